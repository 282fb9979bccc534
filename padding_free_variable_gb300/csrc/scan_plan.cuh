// scan_plan.cuh -- a plan with the tables that the gated linear recurrence adds to it.
#pragma once

#include "common.cuh"

namespace lstm {

constexpr int kScanPiece = 256;         // shortest piece that a sequence is cut into where its pieces run side by side
constexpr int kScanChunk = 64;          // steps between the states that are kept for the backward pass

struct ScanTables {
    int64_t chunks = 0;                 // pieces of at most kScanChunk steps of all sequences
    // sequences cut into pieces of kScanPiece << level steps, the last level uncut (every sequence has a piece, if an empty one)
    int32_t levels = 0;
    int32_t level_first[24] = {};       // first entry of the level in d_pieces
    int32_t level_count[25] = {};
    const int4* d_pieces = nullptr;     // (slot, piece, length of the sequence, entry of the slot's first piece in its level by slot)
    const int32_t* d_chunk = nullptr;   // [B+1] first chunk of each slot (both in the allocation of the plan's d_len)
};

// What every plan handle points to.
struct ScanPlan : lstm_plan {
    ScanTables scan;
};

}  // namespace lstm
