// int8 matrix products with a scale per token and channel, and the gated form.
//
// gemm: out[m][n] = (sum_k a[m][k] b[n][k]) sa[m] sb[n] (+ bias[n]) (+ add[m][n])
// glu:  the same product with the rows of w13; h = silu(g) u in the epilogue
//
// Sums are int32 and exact (K <= 131056 keeps |sum| <= 2^31 - 2^18), so their
// order, and how K is split, does not change a bit of the output.
//
// Rows of A and B are K-contiguous: both operands of v_mfma_i32_*_i8 take 16
// consecutive K bytes of one row per lane, and A and B only have to agree on
// which K bytes a lane holds.
#include "moe_common.h"
#include "moe_kernels.h"

namespace moe {

typedef int i32x16 __attribute__((ext_vector_type(16)));

struct GemmArgs {
    const int8_t* a;
    const float* sa;
    const int8_t* b;
    const float* sb;
    const float* bias;        // may be null
    const void* add;          // may be null; the output's type
    void* out;
    int M, N, K;              // N: output columns (glu: inter; b then has 2N rows)
    int vec;                  // output (and add) rows take vector accesses of a lane's columns
};

__device__ const uint8_t g_zero16[16] = {0};            // source of K bytes past a row's end

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    typedef float f2 __attribute__((ext_vector_type(2)));
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2){a, b}, b2));
}
__device__ __forceinline__ float glu_h(float g, float u) { return g / (1.0f + __expf(-g)) * u; }

// Workgroup barrier that waits for the wave's LDS traffic only (the fence of
// __syncthreads() would drain the direct-to-LDS loads in flight).
static __device__ __forceinline__ void barrier_lds() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);                // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// NC adjacent output columns of one row
template <int NC, bool F32>
__device__ __forceinline__ void store_cols(const GemmArgs& p, int row, int col, float (&v)[NC]) {
    const size_t o = (size_t)row * p.N + col;
    if (p.vec) {                                        // N % NC == 0: all NC columns or none
        if (col >= p.N) return;
        if (F32) {
            if (p.add) {
#pragma unroll
                for (int n = 0; n < NC; ++n) v[n] += ((const float*)p.add + o)[n];
            }
#pragma unroll
            for (int n = 0; n < NC; ++n) ((float*)p.out + o)[n] = v[n];
            return;
        }
        uint32_t w[NC / 2];
        if (p.add) {
#pragma unroll
            for (int h = 0; h < NC / 2; ++h) w[h] = *(const uint32_t*)((const uint16_t*)p.add + o + 2 * h);
#pragma unroll
            for (int h = 0; h < NC / 2; ++h) {
                v[2 * h] += __uint_as_float(w[h] << 16);
                v[2 * h + 1] += __uint_as_float(w[h] & 0xFFFF0000u);
            }
        }
#pragma unroll
        for (int h = 0; h < NC / 2; ++h) w[h] = pack_bf16(v[2 * h], v[2 * h + 1]);
        uint16_t* d = (uint16_t*)p.out + o;
        if constexpr (NC == 2) *(uint32_t*)d = w[0];
        else if constexpr (NC == 4) *(uint2*)d = make_uint2(w[0], w[1]);
        else *(uint4*)d = make_uint4(w[0], w[1], w[2], w[3]);
        return;
    }
#pragma unroll
    for (int n = 0; n < NC; ++n) {
        if (col + n >= p.N) continue;
        if (F32) {
            if (p.add) v[n] += ((const float*)p.add)[o + n];
            ((float*)p.out)[o + n] = v[n];
        } else {
            if (p.add) v[n] += bf16_to_f32(((const uint16_t*)p.add)[o + n]);
            ((uint16_t*)p.out)[o + n] = (uint16_t)pack_bf16(v[n], 0.f);
        }
    }
}

// ------------------------------------------------------------------ tiles
// TM x TN outputs (glu: TN rows of B = TN / 2 columns of h) by WM x WN waves,
// K in steps of 128 bytes through a ring of R LDS stages of TM + TN rows.
// A stage row's 16-byte chunk c sits at c ^ ((row / 2) & 7): 16-byte fragment
// reads of 32 (or 16) consecutive rows then meet every bank once.
// B fragment f = nw NF + n, row m holds output column nw 32 NF + NF m + n, so
// the columns a lane accumulates are adjacent (glu: the first half of a wave's
// fragments are gate rows, the second the matching up rows).
template <int TM, int TN, int WM, int WN, int R, bool GLU, bool F32>
__global__ void __launch_bounds__(64 * WM * WN) gemm_tile_kernel(GemmArgs p, int tiles_m, int tiles_n) {
    constexpr int WAVES = WM * WN;
    constexpr int MF = TM / WM / 32, NF = TN / WN / 32;
    constexpr int STAGE = (TM + TN) * 128;
    constexpr int LA = TM / 8 / WAVES, LB = TN / 8 / WAVES;      // 8-row loads per wave and step
    constexpr int OUTN = GLU ? TN / 2 : TN;                      // output columns of a tile
    constexpr int NC = GLU ? NF / 2 : NF;                        // adjacent output columns of a lane
    static_assert(MF >= 1 && NC >= 1 && LA >= 1 && LB >= 1 && TM % (8 * WAVES) == 0 && TN % (8 * WAVES) == 0, "tile");
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    float* s_sa = (float*)(smem + R * STAGE);
    float* s_sb = s_sa + TM;                                     // TN scales (glu: gate, then up)
    float* s_bias = s_sb + TN;
    const int lane = lane_id();
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int mw = wv / WN, nw = wv % WN;

    // tile of this workgroup: each XCD takes a run of consecutive tiles
    // (blocks are dealt to the 8 XCDs in turn), and runs go down groups of 8
    // row panels, so an XCD's L2 serves a few panels of A and B at a time
    const int total = tiles_m * tiles_n;
    int L;
    {
        const int x = blockIdx.x & 7, i = blockIdx.x >> 3, per = total >> 3, rem = total & 7;
        L = x * per + min(x, rem) + i;
    }
    const int GM = 8;
    const int grp = L / (GM * tiles_n), first = grp * GM, gsz = min(GM, tiles_m - first);
    const int tm = first + (L - grp * GM * tiles_n) % gsz, tn = (L - grp * GM * tiles_n) / gsz;
    const int row0 = tm * TM, col0 = tn * OUTN;

    // ---- load side: load j of this wave fills stage rows 8 (wv LA + j) ..
    // (A; B after TM rows likewise); lane i: row i / 8 of them, chunk
    // (i % 8) ^ ((row / 2) & 7) of its source row
    const int K = p.K, S = (K + 127) / 128;
    const int sub = lane >> 3;
    auto chunk = [&](int r8) { return 16 * ((lane & 7) ^ ((4 * r8 + (lane >> 4)) & 7)); };   // r8: row / 8
    uint32_t oA[LA], oB[LB];
    const uint8_t* bB[LB];
    const uint8_t* bA = (const uint8_t*)p.a + (size_t)row0 * K;
#pragma unroll
    for (int j = 0; j < LA; ++j) {
        const int r8 = wv * LA + j;
        oA[j] = (uint32_t)min(8 * r8 + sub, p.M - 1 - row0) * K + chunk(r8);
    }
#pragma unroll
    for (int j = 0; j < LB; ++j) {
        const int r8 = wv * LB + j, f = r8 / 4, m = 8 * (r8 & 3) + sub;
        const int w = f / NF, n = f % NF;
        const int c = w * 32 * NC + NC * m + n % NC;             // output column in the tile
        bB[j] = (const uint8_t*)p.b + ((size_t)col0 + (GLU && n >= NC ? p.N : 0)) * K;
        oB[j] = (uint32_t)min(c, p.N - 1 - col0) * K + chunk(r8);
    }
    auto issue = [&](int s) __attribute__((always_inline)) {
        uint8_t* st = smem + (s % R) * STAGE;
        const int k0 = s * 128;
        if (k0 + 128 <= K) {
#pragma unroll
            for (int j = 0; j < LA; ++j) lds_dma16(bA + k0 + oA[j], st + 1024 * (wv * LA + j));
#pragma unroll
            for (int j = 0; j < LB; ++j) lds_dma16(bB[j] + k0 + oB[j], st + TM * 128 + 1024 * (wv * LB + j));
        } else {                                                 // K ends inside this step
#pragma unroll
            for (int j = 0; j < LA; ++j)
                lds_dma16(k0 + chunk(wv * LA + j) < K ? bA + k0 + oA[j] : g_zero16, st + 1024 * (wv * LA + j));
#pragma unroll
            for (int j = 0; j < LB; ++j)
                lds_dma16(k0 + chunk(wv * LB + j) < K ? bB[j] + k0 + oB[j] : g_zero16,
                          st + TM * 128 + 1024 * (wv * LB + j));
        }
    };

    // ---- scales into LDS (no wait of their own: they precede the first stage)
    for (int i = wv; i < TM / 64; i += WAVES)
        lds_dma4(p.sa + min(row0 + 64 * i + lane, p.M - 1), (uint8_t*)(s_sa + 64 * i));
    for (int i = wv; i < TN / 64; i += WAVES) {
        const int c = 64 * i + lane;
        const int n = GLU ? min(col0 + c % OUTN, p.N - 1) + (c >= OUTN ? p.N : 0) : min(col0 + c, p.N - 1);
        lds_dma4(p.sb + n, (uint8_t*)(s_sb + 64 * i));
        if (!GLU && p.bias) lds_dma4(p.bias + n, (uint8_t*)(s_bias + 64 * i));
    }
    // a step past the end fills its ring slot with zeros, so every step has
    // the same number of loads to count (and the slot is not read)
    auto fill = [&](int s) __attribute__((always_inline)) {
        if (s < S) {
            issue(s);
            return;
        }
        uint8_t* st = smem + (s % R) * STAGE;
#pragma unroll
        for (int j = 0; j < LA + LB; ++j) lds_dma16(g_zero16, st + 1024 * (wv * (LA + LB) + j));
    };
#pragma unroll
    for (int s = 0; s < R - 1; ++s) fill(s);

    // ---- multiply
    i32x16 acc[MF][NF];
#pragma unroll
    for (int a = 0; a < MF; ++a)
#pragma unroll
        for (int n = 0; n < NF; ++n)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[a][n][i] = 0;
    const int m = lane & 31, hi = lane >> 5, sw = (m >> 1) & 7;
    for (int s = 0; s < S; ++s) {
        wait_vmcnt<(R - 2) * (LA + LB)>();                       // stage s landed (this wave's part)
        barrier_lds();                                           // ... everyone's; and everyone has read stage s - 1
        if (R > 2 || s + 1 < S) fill(s + R - 1);
        const uint8_t* st = smem + (s % R) * STAGE;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            const int off = m * 128 + (((2 * ks + hi) ^ sw) << 4);
            i32x4 fa[MF], fb[NF];
#pragma unroll
            for (int a = 0; a < MF; ++a) fa[a] = *(const i32x4*)(st + (mw * MF + a) * 4096 + off);
#pragma unroll
            for (int n = 0; n < NF; ++n) fb[n] = *(const i32x4*)(st + TM * 128 + (nw * NF + n) * 4096 + off);
#pragma unroll
            for (int a = 0; a < MF; ++a)
#pragma unroll
                for (int n = 0; n < NF; ++n)
                    acc[a][n] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fa[a], fb[n], acc[a][n], 0, 0, 0);
        }
    }
    wait_vmcnt<0>();

    // ---- epilogue: lane (m, hi), register i of fragment (a, n): row
    // 32 (mw MF + a) + 8 (i / 4) + 4 hi + i % 4, column NC m + n of the wave's
    const int cw = nw * 32 * NC + NC * m, col = col0 + cw;
    float sb[NF], bias[NC];
#pragma unroll
    for (int n = 0; n < NF; ++n) sb[n] = s_sb[(GLU && n >= NC ? OUTN : 0) + cw + n % NC];
#pragma unroll
    for (int n = 0; n < NC; ++n) bias[n] = !GLU && p.bias ? s_bias[cw + n] : 0.f;
#pragma unroll
    for (int a = 0; a < MF; ++a)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int r = 32 * (mw * MF + a) + 8 * (i / 4) + 4 * hi + i % 4;
            const float sa = s_sa[r];
            float v[NC];
#pragma unroll
            for (int n = 0; n < NC; ++n) {
                if constexpr (GLU) v[n] = glu_h((float)acc[a][n][i] * sa * sb[n], (float)acc[a][n + NC][i] * sa * sb[n + NC]);
                else v[n] = (float)acc[a][n][i] * sa * sb[n] + bias[n];
            }
            if (row0 + r < p.M) store_cols<NC, F32>(p, row0 + r, col, v);
        }
}

// ------------------------------------------------------------------ few rows
// Up to 16 MF rows: the weights are streamed once, straight into registers.
// A workgroup owns 16 rows of B (glu: 8 gate and the matching 8 up rows); its
// waves split K in runs of 64 bytes and add their int32 sums in LDS.
template <int MF, int WAVES, bool GLU, bool F32>
__global__ void __launch_bounds__(64 * WAVES) gemm_rows_kernel(GemmArgs p) {
    __shared__ int s_acc[WAVES][MF][256];
    const int lane = lane_id(), wv = threadIdx.x / 64;
    const int m = lane & 15, q = lane >> 4;
    constexpr int OUTN = GLU ? 8 : 16;
    const int col0 = blockIdx.x * OUTN;
    const int c = min(col0 + (GLU ? m & 7 : m), p.N - 1);
    const uint8_t* rb = (const uint8_t*)p.b + ((size_t)c + (GLU && m >= 8 ? p.N : 0)) * p.K;
    const uint8_t* ra[MF];
#pragma unroll
    for (int a = 0; a < MF; ++a) ra[a] = (const uint8_t*)p.a + (size_t)min(16 * a + m, p.M - 1) * p.K;
    i32x4 acc[MF];
#pragma unroll
    for (int a = 0; a < MF; ++a) acc[a] = i32x4{0, 0, 0, 0};
    const int U = (p.K + 63) / 64;
#pragma unroll 4
    for (int u = wv; u < U; u += WAVES) {
        const int k = 64 * u + 16 * q;
        const bool in = k < p.K;
        const i32x4 fb = *(const i32x4*)(in ? rb + k : g_zero16);
#pragma unroll
        for (int a = 0; a < MF; ++a) {
            const i32x4 fa = *(const i32x4*)(in ? ra[a] + k : g_zero16);
            acc[a] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fa, fb, acc[a], 0, 0, 0);
        }
    }
#pragma unroll
    for (int a = 0; a < MF; ++a)
#pragma unroll
        for (int i = 0; i < 4; ++i) s_acc[wv][a][16 * (4 * q + i) + m] = acc[a][i];
    __syncthreads();
    for (int t = threadIdx.x; t < 16 * MF * OUTN; t += 64 * WAVES) {
        const int row = t / OUTN, n = t % OUTN, e = 16 * (row & 15) + n;
        if (row >= p.M || col0 + n >= p.N) continue;
        int g = 0, u = 0;
        for (int w = 0; w < WAVES; ++w) {
            g += s_acc[w][row >> 4][e];
            if (GLU) u += s_acc[w][row >> 4][e + 8];
        }
        const float sa = p.sa[row];
        float v = (float)g * sa * p.sb[col0 + n];
        if constexpr (GLU) v = glu_h(v, (float)u * sa * p.sb[p.N + col0 + n]);
        else if (p.bias) v += p.bias[col0 + n];
        const size_t o = (size_t)row * p.N + col0 + n;
        if (F32) {
            if (p.add) v += ((const float*)p.add)[o];
            ((float*)p.out)[o] = v;
        } else {
            if (p.add) v += bf16_to_f32(((const uint16_t*)p.add)[o]);
            ((uint16_t*)p.out)[o] = (uint16_t)pack_bf16(v, 0.f);
        }
    }
}

// ------------------------------------------------------------------ launch
template <int TM, int TN, int WM, int WN, int R, bool GLU, bool F32>
static hipError_t launch_tile(GemmArgs p, int kid, hipStream_t stream) {
    constexpr int OUTN = GLU ? TN / 2 : TN, NC = (GLU ? TN / 2 : TN) / WN / 32;
    constexpr int SMEM = R * (TM + TN) * 128 + 4 * (TM + 2 * TN);
    hipError_t e = hipFuncSetAttribute((const void*)gemm_tile_kernel<TM, TN, WM, WN, R, GLU, F32>,
                                       hipFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e != hipSuccess) return e;
    p.vec = p.vec && p.N % NC == 0;
    const int tm = (p.M + TM - 1) / TM, tn = (p.N + OUTN - 1) / OUTN;
    MOE_LAUNCH(kid, stream, (gemm_tile_kernel<TM, TN, WM, WN, R, GLU, F32>), dim3((unsigned)(tm * tn)),
               dim3(64 * WM * WN), SMEM, stream, p, tm, tn);
    return hipGetLastError();
}

template <int MF, int WAVES, bool GLU, bool F32>
static hipError_t launch_few(const GemmArgs& p, int kid, hipStream_t stream) {
    MOE_LAUNCH(kid, stream, (gemm_rows_kernel<MF, WAVES, GLU, F32>), dim3((unsigned)((p.N + (GLU ? 7 : 15)) / (GLU ? 8 : 16))),
               dim3(64 * WAVES), 0, stream, p);
    return hipGetLastError();
}

template <bool GLU, bool F32>
static hipError_t launch_any(const GemmArgs& p, int kid, hipStream_t stream) {
    if (p.M <= 16) return launch_few<1, 16, GLU, F32>(p, kid, stream);
    if (p.M <= 32) return launch_few<2, 16, GLU, F32>(p, kid, stream);
    return launch_tile<256, 256, 4, 2, 2, GLU, F32>(p, kid, stream);
}

hipError_t launch_gemm_i8(const int8_t* a, const float* sa, const int8_t* b, const float* sb, const float* bias,
                          const void* add, int M, int N, int K, bool f32, void* out, bool vec, hipStream_t stream) {
    const GemmArgs p{a, sa, b, sb, bias, add, out, M, N, K, vec};
    return f32 ? launch_any<false, true>(p, K_GEMM_I8, stream) : launch_any<false, false>(p, K_GEMM_I8, stream);
}

hipError_t launch_glu_i8(const int8_t* a, const float* sa, const int8_t* w13, const float* s13, int M, int I, int K,
                         uint16_t* h, bool vec, hipStream_t stream) {
    const GemmArgs p{a, sa, w13, s13, nullptr, nullptr, h, M, I, K, vec};
    return launch_any<true, false>(p, K_GLU_I8, stream);
}

}  // namespace moe
