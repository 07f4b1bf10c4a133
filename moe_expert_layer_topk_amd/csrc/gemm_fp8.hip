// e4m3 matrix products with a power of two per row and 128 columns of A and an
// fp32 scale per 128 x 128 block of B, and the gated form.
//
// gemm: out[m][n] = sum_j sb[n / 128][j] 2^(sa[m][j] - 127) sum_{k in block j} a[m][k] b[n][k] (+ bias[n]) (+ add[m][n])
// glu:  the same product with the rows of w13; h = silu(g) u in the epilogue
//
// bf16 outputs: a block's sum is one FP8 matrix instruction (K = 128), which
// takes A's scale as an operand. It aligns the products of each group of its K
// at the largest one's exponent and drops what lies 14 bits and more below
// (measured: 2^16 - 2^16 + 2^3 gives 2^3, + 2^2 gives 0), which is well below
// bf16's own step: 1.1e-4 of the output's norm, where bf16 rounds 1.7e-3 off.
// fp32 outputs would show it (1.1e-5 .. 1.5e-5 of the norm), so their codes are
// widened to bf16, exactly, for the bf16 instruction, which drops 25 bits below.
// The running sum over the blocks is fp32, one fused multiply-add per block.
#include "moe_common.h"
#include "moe_kernels.h"

namespace moe {

struct Fp8Args {
    const uint8_t* a;
    const uint8_t* sa;
    const uint8_t* b;
    const float* sb;
    const float* bias;        // may be null
    const void* add;          // may be null; the output's type
    void* out;
    int M, N, K;              // N: output columns (glu: inter; b then has 2N rows)
};

// codes 8 i .. 8 i + 7 of a fragment as bf16
__device__ __forceinline__ bf16x8 widen(const i32x8& f, int i) {
    i32x4 w;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t lo, hi;
        e4m3x4_to_bf16x4((uint32_t)f[2 * i + h], lo, hi);
        w[2 * h] = (int)lo;
        w[2 * h + 1] = (int)hi;
    }
    return __builtin_bit_cast(bf16x8, w);
}
// 2^(b - 127), NaN for 255
__device__ __forceinline__ float e8m0_f32(uint32_t b) {
    return __uint_as_float(b == 255 ? 0x7FC00000u : b == 0 ? 0x00400000u : b << 23);
}

// One wave a 16 x 16 tile, fragments straight from memory.
template <bool GLU, bool F32>
__global__ void __launch_bounds__(64) gemm_fp8_kernel(Fp8Args p, int tiles_m, int tiles) {
    const int lane = lane_id(), m = lane & 15, q = lane >> 4;
    for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int row0 = t % tiles_m * 16, col0 = t / tiles_m * 16;
    const int KB = (p.K + 127) / 128;
    const int ra = min(row0 + m, p.M - 1), cb = min(col0 + m, p.N - 1);
    const uint8_t* pa = p.a + (size_t)ra * p.K;
    const uint8_t* pb = p.b + (size_t)cb * p.K;
    const uint8_t* pu = pb + (size_t)p.N * p.K;
    const float* sb = p.sb + (size_t)(col0 / 128) * KB;
    const float* su = sb + (size_t)((p.N + 127) / 128) * KB;
    // 32 K bytes of a row: chunks q and 4 + q of the block's eight; zero past K
    auto frag = [&](const uint8_t* r, int j) __attribute__((always_inline)) {
        i32x8 f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int k = 128 * j + 64 * h + 16 * q;
            const i32x4 v = k < p.K ? *(const i32x4*)(r + k) : i32x4{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < 4; ++i) f[4 * h + i] = v[i];
        }
        return f;
    };
    f32x4 g = {0, 0, 0, 0}, u = {0, 0, 0, 0};
    for (int j = 0; j < KB; ++j) {
        const i32x8 fa = frag(pa, j);
        const int e = p.sa[(size_t)ra * KB + j];
        if (F32) {
            const i32x8 fb = frag(pb, j);
            f32x4 x = {0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < 4; ++i) x = mfma_bf16_16x16x32(widen(fa, i), widen(fb, i), x);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                g[i] = __builtin_fmaf(x[i] * e8m0_f32(p.sa[(size_t)min(row0 + 4 * q + i, p.M - 1) * KB + j]), sb[j], g[i]);
            continue;
        }
        const f32x4 x = mfma_fp8_16x16x128(fa, frag(pb, j), f32x4{0, 0, 0, 0}, e, 127);
#pragma unroll
        for (int i = 0; i < 4; ++i) g[i] = __builtin_fmaf(x[i], sb[j], g[i]);
        if (GLU) {
            const f32x4 y = mfma_fp8_16x16x128(fa, frag(pu, j), f32x4{0, 0, 0, 0}, e, 127);
#pragma unroll
            for (int i = 0; i < 4; ++i) u[i] = __builtin_fmaf(y[i], su[j], u[i]);
        }
    }
    // register i: row 4 q + i, column m
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = row0 + 4 * q + i, c = col0 + m;
        if (r >= p.M || c >= p.N) continue;
        const size_t o = (size_t)r * p.N + c;
        float v = g[i];
        if (GLU) v = v / (1.0f + __expf(-v)) * u[i];
        else {
#pragma clang fp contract(off)
            if (p.bias) v += p.bias[c];
            if (p.add) v += F32 ? ((const float*)p.add)[o] : bf16_to_f32(((const uint16_t*)p.add)[o]);
        }
        if (F32) ((float*)p.out)[o] = v;
        else ((__bf16*)p.out)[o] = (__bf16)v;
    }
    }
}

template <bool GLU, bool F32>
static hipError_t launch_any(const Fp8Args& p, int kid, hipStream_t stream) {
    const int tm = (p.M + 15) / 16, tn = (p.N + 15) / 16;
    const int tiles = tm * tn;                                   // (fewer than 2^30)
    return launch_kernel(kid, stream, gemm_fp8_kernel<GLU, F32>, dim3((unsigned)min(tiles, 1 << 20)), dim3(64), 0, p, tm, tiles);
}

hipError_t launch_gemm_fp8(const uint8_t* a, const uint8_t* sa, const uint8_t* b, const float* sb, const float* bias,
                           const void* add, int M, int N, int K, bool f32, void* out, bool aligned, hipStream_t stream) {
    const Fp8Args p{a, sa, b, sb, bias, add, out, M, N, K};
    return f32 ? launch_any<false, true>(p, K_GEMM_FP8, stream) : launch_any<false, false>(p, K_GEMM_FP8, stream);
}

hipError_t launch_glu_fp8(const uint8_t* a, const uint8_t* sa, const uint8_t* w13, const float* s13, int M, int I, int K,
                          uint16_t* h, bool aligned, hipStream_t stream) {
    const Fp8Args p{a, sa, w13, s13, nullptr, nullptr, h, M, I, K};
    return launch_any<true, false>(p, K_GLU_FP8, stream);
}

}  // namespace moe
