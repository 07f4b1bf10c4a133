"""Which tile shape an e4m3 product takes (csrc/gemm_i8_plan.h, in a small C++
program on the host): every size that is documented has a launch, and the shapes
that the kernels have."""
import os
import subprocess

import moe_expert_layer_topk_amd as moe

CSRC = os.path.join(os.path.dirname(moe.LIB_PATH), "csrc")


def test_every_documented_size_has_a_launch(tmp_path):
    src, exe = tmp_path / "plan.cpp", tmp_path / "plan"
    src.write_text("""#include "gemm_i8_plan.h"
#include <cstdio>
#include <initializer_list>
using namespace moe;
int main() {
    int shapes[2][S_COUNT] = {};
    for (int f32 = 0; f32 < 2; ++f32)
        for (long long cus : {256, 304, 64})
            for (int K : {16, 128, 256, 2048, 131056})
                for (int few : {1, 2, 5, 7, 8, 31, 32, 33, 64, 200, 256, 300})
                    for (int e = 0; e <= 30; ++e)
                        for (int d = -3; d <= 3; d += 3)
                            for (int side = 0; side < 3 - f32; ++side) {
                                const long long many = (1LL << e) + d;
                                if (many < 1 || many > 1LL << 30 || (many + 15) / 16 * ((few + 7) / 8) >= 1LL << 31) continue;
                                const int M = side == 0 ? (int)many : few;
                                const long long rows_b = side == 0 ? few : side == 1 ? many : 2 * many;
                                const int s = pick_shape(f32 ? kShapesFp8F32 : kShapesFp8, M, rows_b, K, cus);
                                const long long tiles = shape_tiles(s, M, rows_b), threads = tiles * 64 * split_waves(s, tiles <= cus);
                                ++shapes[f32][s];
                                if (threads >= 1LL << 32) return printf("%d x %lld x %d, %lld CUs: shape %d\\n", M, rows_b, K, cus, s), 0;
                                if (f32 && s == S_256x256) return printf("fp32 outputs have no 256 x 256 tile\\n"), 0;
                            }
    for (int f32 = 0; f32 < 2; ++f32)
        for (int i = f32; i < S_COUNT; ++i)
            if (!shapes[f32][i]) return printf("shape %d is never picked (%d)\\n", i, f32), 0;
    const struct { int f32, M, N, K, s; } known[] = {{0, 1, 2048, 2048, S_32x32}, {0, 16384, 2048, 2048, S_256x256}, {0, 2048, 2048, 2048, S_128x128},
        {1, 8, 131072, 2048, S_32x64}, {1, 16384, 2048, 2048, S_128x128}};
    for (const auto& k : known)
        if (pick_shape(k.f32 ? kShapesFp8F32 : kShapesFp8, k.M, k.N, k.K, 256) != k.s)
            return printf("%d x %d x %d: %d\\n", k.M, k.N, k.K, pick_shape(k.f32 ? kShapesFp8F32 : kShapesFp8, k.M, k.N, k.K, 256)), 0;
    printf("ok\\n");
}
""")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    assert out.startswith("ok"), out
