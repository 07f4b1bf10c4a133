"""What the int8 products load, and which tile shape they take, decided on the
host (no GPU): the functions of csrc/gemm_i8_plan.h, which the kernels and
their launches call too, in a small C++ program, and the loads of the built
library.

A read past an operand cannot be seen in a result (A counts as zero past K), so
it is looked for here.
"""
import os
import re
import shutil
import subprocess

import pytest

import moe_expert_layer_topk_amd as moe

CSRC = os.path.join(os.path.dirname(moe.LIB_PATH), "csrc")
OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"


def _run_cpp(tmp_path, body):
    """Compiles and runs a main() with this body; it prints what it finds wrong."""
    src, exe = tmp_path / "plan.cpp", tmp_path / "plan"
    src.write_text('#include "gemm_i8_plan.h"\n#include <cstdio>\n#include <initializer_list>\nusing namespace moe;\n'
                   "int main() {\n" + body + "\n    return 0;\n}\n")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    return subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout


def test_loads_stay_inside_the_operand(tmp_path):
    """Every lane offset of a tile of up to 256 rows, at every K position of
    the loops and past them (the prologue's, a step of zeros, retired loads):
    what the record count admits lies inside the operand, and what the sums
    need is admitted, at its own address."""
    out = _run_cpp(tmp_path, """
    long checked = 0;
    for (int K : {16, 32, 80, 112, 128, 144, 240, 256, 400, 512, 1040, 2064, 131056})
        for (int rows : {1, 2, 31, 32, 33, 64, 127, 128, 255, 256, 257, 1000}) {
            const size_t n = (size_t)rows * K;
            for (int k0 = 0; k0 < K + 1024; k0 += K > 4096 && k0 > 1024 && k0 < K - 1024 ? 12800 : 128)
                for (int on = 0; on < 2; ++on) {
                    const uint32_t left = records_from(records(n), on ? k0 : NOWHERE);
                    for (int r = 0; r < 256; ++r)
                        for (int at = 0; at < 128; at += 16) {
                            const uint32_t o = row_offset(r, rows - 1, K, at);
                            const bool admitted = o < left;
                            ++checked;
                            if (admitted && (!on || (size_t)k0 + o + 16 > n))
                                return printf("past the end: K %d rows %d k0 %d on %d row %d at %d\\n", K, rows, k0, on, r, at), 0;
                            const int real = r < rows ? r : rows - 1;
                            if (on && k0 + at < K && (!admitted || (size_t)k0 + o != (size_t)real * K + k0 + at))
                                return printf("not loaded: K %d rows %d k0 %d row %d at %d\\n", K, rows, k0, r, at), 0;
                        }
                }
        }
    // operands past 4 GiB from a tile's first row on: every offset a tile can have stays below the count
    if (records_from(records((size_t)1 << 40), 131056) < 257 * 131056 || records_from(records((size_t)1 << 40), NOWHERE) != 0)
        return printf("count of a large operand\\n"), 0;
    if (records((size_t)1 << 40) % 16) return printf("a count inside an access\\n"), 0;
    printf("ok %ld\\n", checked);""")
    assert out.startswith("ok "), out


def test_every_documented_size_has_a_launch(tmp_path):
    """Up to 2^30 rows on either side (gated: 2^31 B rows) the picked shape's
    launch holds fewer than 2^32 threads, and sizes that had one keep theirs."""
    out = _run_cpp(tmp_path, """
    int shapes[S_COUNT] = {};
    for (long long cus : {256, 304, 64})
        for (int K : {16, 128, 256, 2048, 131056})
            for (int few : {1, 2, 5, 7, 8, 31, 32, 33, 64, 200, 256, 300})
                for (int e = 0; e <= 30; ++e)
                    for (int d = -3; d <= 3; d += 3)
                        for (int side = 0; side < 3; ++side) {
                            // a; b; b of a gated product, whose gate and up rows both count
                            const long long many = (1LL << e) + d;
                            if (many < 1 || many > 1LL << 30 || (many + 15) / 16 * ((few + 7) / 8) >= 1LL << 31) continue;
                            const int M = side == 0 ? (int)many : few;
                            const long long rows_b = side == 0 ? few : side == 1 ? many : 2 * many;
                            const int s = pick_shape(M, rows_b, K, cus);
                            const long long tiles = shape_tiles(s, M, rows_b), threads = tiles * 64 * split_waves(s, tiles <= cus);
                            ++shapes[s];
                            if (threads >= 1LL << 32) return printf("%d x %lld x %d, %lld CUs: shape %d, %lld threads\\n", M, rows_b, K, cus, s, threads), 0;
                        }
    for (int i = 0; i < S_COUNT; ++i)
        if (!shapes[i]) return printf("shape %d is never picked\\n", i), 0;
    const struct { int M, N, K, s; } known[] = {{1, 2048, 2048, S_32x32}, {32, 2048, 512, S_32x64}, {333, 1000, 4112, S_32x64}, {400, 2048, 2048, S_64x64},
        {2048, 2048, 2048, S_128x128}, {16384, 256, 7168, S_128x128}, {16384, 2048, 2048, S_256x256}};
    for (const auto& k : known)
        if (pick_shape(k.M, k.N, k.K, 256) != k.s) return printf("%d x %d x %d: %d\\n", k.M, k.N, k.K, pick_shape(k.M, k.N, k.K, 256)), 0;
    printf("ok\\n");""")
    assert out.startswith("ok"), out


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="no disassembler for the built kernels")
def test_no_load_counts_on_the_scalar_offset(tmp_path):
    """The buffer loads of the built library have a scalar offset of 0, so that the
    bounds check compares the lane's offset alone (with another one its
    descriptions disagree)."""
    if not os.path.exists(moe.LIB_PATH):
        from moe_expert_layer_topk_amd.build import build
        build()
    lib = tmp_path / "lib.so"
    shutil.copy(moe.LIB_PATH, lib)
    subprocess.run([OBJDUMP, "--offloading", str(lib)], check=True, capture_output=True, cwd=tmp_path)
    loads, other = 0, set()
    for f in sorted(tmp_path.glob("lib.so*gfx950*")):
        text = subprocess.run([OBJDUMP, "-d", str(f)], check=True, capture_output=True, text=True).stdout
        for m in re.finditer(r"\bbuffer_load\w+ [^\n]*?s\[\d+:\d+\], (\w+) offen[^\n]* lds", text):
            loads += 1
            if m.group(1) != "0":
                other.add(m.group(0))
    assert loads > 100
    assert not other, sorted(other)[:4]
