"""Which rows the block norms read in groups of eight from a multiple of eight values in memory (odd widths): no group that
is read whole may begin before its tensor or end behind it.  The library's own rule is asked, the kernels' index
arithmetic is done over on the host."""
import os
import subprocess

from padding_free_variable_gb300 import build as pbuild

PROGRAM = r"""
#include <cstdio>
#include <cstring>
#include "block_norm.cuh"

int main()
{
    using namespace lstm;
    long taken = 0, bad = 0;
    for (int layer = 0; layer < 2; ++layer)
        for (int D = 1; D <= 70; ++D)
            for (int pad : {0, 8, 24})
                for (int64_t rows = 1; rows <= 20; ++rows) {
                    NormArgs a;
                    memset((void*)&a, 0, sizeof a);
                    float* const p = (float*)4096;      // aligned, never read
                    a.D = D; a.rows = rows; a.post = a.pre = layer ? LSTM_NORM_LAYER : LSTM_NORM_RMS; a.gate = LSTM_GATE_SILU;
                    a.w.w_post = a.w.scale = a.w.w_pre = p;
                    if (layer) a.w.b_post = a.w.b_pre = p;
                    a.x = a.y = a.g = a.dn = a.dx_out = p;
                    a.x_out = a.n = a.dx = a.dy = a.dg = p;
                    a.ldy = a.ldg = a.lddy = a.lddg = D + pad;
                    if (!norm_shifted(a)) continue;
                    ++taken;
                    for (int64_t ld : {(int64_t)D, (int64_t)D + pad})
                        for (int64_t r = 0; r < rows; ++r) {
                            const int shift = (int)((uint64_t)r * (unsigned)D & 7u);
                            for (int at = -shift; at < D; at += 8) {
                                const bool whole = at >= 0 && at + 8 <= D;
                                if (!whole && r == rows - 1) continue;      // the last row's ends are read value by value
                                const int64_t from = r * ld + at;
                                if (from % 8 || from < 0 || from + 8 > (rows - 1) * ld + D) {
                                    if (bad++ < 5) printf("width %d, %ld rows of stride %ld: row %ld reads %ld to %ld\n", D, (long)rows, (long)ld, (long)r, (long)from, (long)from + 7);
                                }
                            }
                        }
                }
    printf("taken %ld bad %ld\n", taken, bad);
    return bad || !taken;
}
"""


def test_no_group_is_read_beyond_its_tensor(tmp_path):
    lib = pbuild.build()
    src, exe = tmp_path / "reach.cu", tmp_path / "reach"
    src.write_text(PROGRAM)
    cmd = [pbuild.nvcc()] + pbuild.ARCH + pbuild.NVCC_FLAGS + [str(src), "-o", str(exe), lib, "-Xlinker", "-rpath=" + os.path.dirname(lib)]
    done = subprocess.run(cmd, capture_output=True, text=True)
    assert done.returncode == 0, done.stderr
    done = subprocess.run([str(exe)], capture_output=True, text=True)
    assert done.returncode == 0, done.stdout + done.stderr
