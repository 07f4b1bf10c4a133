"""What moe_sample makes of top_k (csrc/sample_plan.h, evaluated by the compiler on
the host, which refuses a sum that does not fit an int): the whole range of int32."""
import os
import subprocess

import moe_expert_layer_topk_amd as moe

CSRC = os.path.join(os.path.dirname(moe.LIB_PATH), "csrc")
INCLUDE = os.path.join(os.path.dirname(os.path.dirname(moe.LIB_PATH)), "include")


def test_top_k_of_any_int(tmp_path):
    src = tmp_path / "plan.cpp"
    src.write_text("""#include "sample_plan.h"
using namespace moe;
constexpr int LARGEST = 0x7FFFFFFF, CHUNK = 4096;
template <int K>
constexpr bool holds() {
    constexpr int k = kept_by_count(K);
    // all of a chunk's candidates are looked at as they would be with sums in 64 bits
    constexpr int none = 0, some = 64 + 2 * 20 + 1;
    static_assert(worth_parts(none, k) == (k && none > 2LL * K + 64) && worth_parts(some, k) == (k && some > 2LL * K + 64) &&
                  worth_parts(CHUNK, k) == (k && CHUNK > 2LL * K + 64), "parts");
    return K <= 0 ? k == 0 : K <= MOE_SAMPLE_MAX_COLS ? k == K : k == MOE_SAMPLE_MAX_COLS;
}
static_assert(holds<-LARGEST - 1>() && holds<-1>() && holds<0>() && holds<1>() && holds<2>() && holds<20>() && holds<2015>() && holds<2016>() &&
              holds<CHUNK>() && holds<MOE_SAMPLE_MAX_COLS - 1>() && holds<MOE_SAMPLE_MAX_COLS>() && holds<MOE_SAMPLE_MAX_COLS + 1>() &&
              holds<(1 << 30) - 33>() && holds<(1 << 30) - 32>() && holds<(1 << 30)>() && holds<LARGEST>(), "top_k");
int main() {}
""")
    got = subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-fsyntax-only", "-I", CSRC, "-I", INCLUDE, str(src)], capture_output=True, text=True)
    assert got.returncode == 0, got.stderr
