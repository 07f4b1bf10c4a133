// e4m3 matrix products with a power of two per row and 128 columns of A and an
// fp32 scale per 128 x 128 block of B, and the gated form.
//
// gemm: out[m][n] = sum_j sb[n / 128][j] 2^(sa[m][j] - 127) sum_{k in block j} a[m][k] b[n][k] (+ bias[n]) (+ add[m][n])
// glu:  the same product with the rows of w13; h = silu(g) u in the epilogue
//
// bf16 outputs: a block's sum is one FP8 matrix instruction (K = 128), which
// takes A's scale as an operand. It aligns the products of each group of its K
// at the largest one's exponent and drops what lies 14 bits and more below
// (measured: 2^16 - 2^16 + 2^3 gives 2^3, + 2^2 gives 0). Before their rounding the
// sums are 1.5e-5 of the outputs' norm off on codes of normal values and 5.8e-5 on
// codes with heavy tails (normal values times e^(1.5 n)); rounding to bf16 costs
// 1.7e-3, and the error of the rounded outputs is within 1% of what it is with
// exact sums: a few outputs in a thousand are the neighbouring bf16 value, which is
// 1.9e-4 .. 4.8e-4 of the norm. The bf16 instruction's sums would take four
// instructions for one (16384 x 2048 x 2048 145 us for 66). fp32 outputs would show
// the loss (theirs are 1e-7 off), so their codes are widened to bf16, exactly, for
// the bf16 instruction, which drops 25 bits below.
// The running sum over the blocks is fp32, one fused multiply-add per block.
//
// A step of 128 K bytes is a block of the scales. Tiles start at multiples of
// their own width, so a wave's columns lie in one block of B's rows (gated: its
// gate columns, and its up columns, whose blocks are counted from their own
// first row), and B's scale is one number per wave and step.
#include "moe_common.h"
#include "moe_kernels.h"
#include "gemm_tile.h"

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
    int lines;                // output rows are whole 128-byte lines (and add's address is 16-byte aligned)
    int words;                // rows of sa start at multiples of four bytes
};

// 2^(b - 127), NaN for 255
__device__ __forceinline__ float e8m0_f32(uint32_t b) {
    return __uint_as_float(b == 255 ? 0x7FC00000u : b == 0 ? 0x00400000u : b << 23);
}
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
__device__ __forceinline__ i32x8 join(const i32x4& lo, const i32x4& hi) {
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}
// a block's products of two fragments, one a scale operand S of A's; byte A of sa
template <int A>
__device__ __forceinline__ f32x4 mfma_block(const i32x8& a, const i32x8& b, int sa) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f32x4{0, 0, 0, 0}, 0, 0, A, sa, 0, 127);
}

// ------------------------------------------------------------------ tiles
// The layout, the stream of K steps and the loads are those of the int8 tiles:
// TM x TN outputs (glu: TN rows of B = TN / 2 columns of h) by WM x WN waves, R
// LDS stages of TM + TN rows of 128 bytes, a stage row's 16-byte chunk c at c ^
// ((row / 2) & 7), B fragment f = nw NF + n, row m holding output column nw 16
// NC + NC m + n.
// A lane's fragment row is 32 bytes, chunks q and 4 + q (both operands alike, so
// which K bytes share an instruction's place does not matter; a block has one
// scale). A's fragments of a step are in registers, two of B's beside them; each
// is read into the registers that its predecessor's last instruction has just
// taken. Block sums wait for their multiply-add while three more instructions
// are issued.
// At the last but one of B's fragments every fragment of the step is read: past
// the barrier there its stage is refilled with the step R ahead and the next
// step's fragments are read.
// Scales: rows' bytes and blocks' floats for 16 steps at a time, loaded two steps
// ahead, in LDS by the barrier before they are read. [step][64 rows][m] is a
// dword with rows m, 16 + m, 32 + m and 48 + m, the instruction's four byte places.
// What it reaches (us; the rate of 2 M N K operations; medians of calls on a few
// inputs in turn): 4096 x 8192 x 8192 235 (2340 TFLOP/s; 226 .. 247 over all runs, 247
// with new inputs before each call), 16384 x 2048 x 2048 66 (2090; 66 .. 70), gated
// 16384 x 512 x 2048 32.4 (2120; 32 .. 34), 8192^3 463 (2370). A
// library product of the same codes with one scale for the whole tensor takes
// 173, 54.5, (29 without the gate) and 341 in windows of 50 ms and more (its first
// milliseconds are slower). Matrix pipes are busy 58% of the clocks, at 1.9 GHz. Power
// is a part of it (198 us instead of 235 on codes of zero, at 2.4 GHz), not
// all: the library takes 130 there. The rest stands between the matrix
// instructions and is not told apart: four multiply-adds that a block's scale costs
// for each of 32 clocks, reads of fragments, a barrier a step. 256 x 256 tiles read
// 411 MB of L2 misses there for 101 MB of operands (last-level cache).
// Tried without gain: the multiply-add 2 or 4 instructions behind, B's next
// fragment one instruction earlier (233 us), wave priorities on this tile, steps with
// their branches taken out into copies (spills). fp32 outputs on 128 x 128 tiles:
// 4096 x 2048 x 2048 40 us (865 TFLOP/s), 16384 x 2048 x 2048 145 (945), four bf16
// instructions for one; a library bf16 product reaches 1470 at the second size. The codes
// are widened again in every wave and tile that reads them.
// K's end: chunks past it are set to zero in LDS by the lanes that loaded them
// (zero times a NaN code from the next row would be NaN).
constexpr int SCALE_STEPS = 16;

template <int TM, int TN, int WM, int WN, int R, bool GLU, bool F32, bool ANY>
__global__ void __launch_bounds__(64 * WM * WN, 2) gemm_fp8_tile_kernel(Fp8Args p, int tiles_m, int tiles_n) {
    constexpr int WAVES = WM * WN;
    constexpr int MF = TM / WM / 16, NF = TN / WN / 16;
    constexpr int STAGE = (TM + TN) * 128;
    constexpr int LA = TM / 8 / WAVES, LB = TN / 8 / WAVES;      // 8-row loads per wave and step
    constexpr int OUTN = GLU ? TN / 2 : TN;                      // output columns of a tile
    constexpr int NC = GLU ? NF / 2 : NF;                        // adjacent output columns of a lane
    constexpr int SCALES = SCALE_STEPS * (TM + 8);               // bytes of 16 steps' scales
    constexpr int NL = LA + LB, NK = MF * NF;                    // loads, instructions of a step
    constexpr int DEPTH = 3, BAR = (NF - 2) * MF;                // instructions between a block sum and its multiply-add; the barrier's
    static_assert(MF == 4 && NF >= 4 && NF % 4 == 0 && TM * 2 == 64 * WAVES && TN % (8 * WAVES) == 0, "tile");
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    uint8_t* s_scale = smem + R * STAGE;                         // two of them
    float* s_bias = (float*)(s_scale + 2 * SCALES);              // two tiles' worth
    const int lane = lane_id();
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int mw = wv / WN, nw = wv % WN;
    const int K = p.K, KB = (K + 127) / 128, S = max(2, KB);     // (a second step past K multiplies zeros)

    // this workgroup's tiles: a run of consecutive ones on each XCD, going down groups of 8 row panels
    const int total = tiles_m * tiles_n;
    const int xcd = blockIdx.x & 7, idx = blockIdx.x >> 3, per_x = gridDim.x >> 3;
    const int per = total >> 3, rem = total & 7;
    const int start = xcd * per + min(xcd, rem), cnt = per + (xcd < rem ? 1 : 0);
    const int nj = cnt > idx ? (cnt - idx + per_x - 1) / per_x : 0;
    if (nj == 0) return;
    auto place = [&](int j, int& row0, int& col0) __attribute__((always_inline)) {
        const int L = start + idx + per_x * j;
        const int grp = L / (8 * tiles_n), first = grp * 8, gsz = min(8, tiles_m - first), r = L - first * tiles_n;
        row0 = (first + r % gsz) * TM;
        col0 = r / gsz * OUTN;
    };

    // ---- load side
    auto opaque_lane = [&]() __attribute__((always_inline)) {
        int l = lane_id();
        asm volatile("" : "+v"(l));
        return l;
    };
    uint32_t oA[LA], oB[LB];
    Operand bA, bB, bU;                                          // A, B (glu: its gate rows), glu's up rows
    int row0 = 0, col0 = 0, row1, col1;                          // the tile being multiplied; the one being loaded
    auto setup = [&](int j) __attribute__((always_inline)) {
        place(j, row1, col1);
        const int ln = opaque_lane(), sub = ln >> 3, ch0 = 16 * ((ln & 7) ^ (ln >> 4));   // (odd 8-row groups: chunk ^ 64)
        bA.set(p.a + (size_t)row1 * K, (size_t)(p.M - row1) * K);
        bB.set(p.b + (size_t)col1 * K, (size_t)(p.N - col1) * K);
        if (GLU) bU.set(p.b + ((size_t)p.N + col1) * K, (size_t)(p.N - col1) * K);
#pragma unroll
        for (int i = 0; i < LA; ++i) {
            const int r8 = wv * LA + i;
            oA[i] = row_offset(8 * r8 + sub, p.M - 1 - row1, K, ch0 ^ (64 * (r8 & 1)));
        }
#pragma unroll
        for (int i = 0; i < LB; ++i) {
            const int r8 = wv * LB + i, f = r8 / 2, m = 8 * (r8 & 1) + sub;
            const int w = f / NF, n = f % NF;
            const int c = w * 16 * NC + NC * m + n % NC;         // output column in the tile
            oB[i] = row_offset(c, p.N - 1 - col1, K, ch0 ^ (64 * (r8 & 1)));
        }
    };
    auto bias = [&](int slot) __attribute__((always_inline)) {
        if (GLU) return;
        const int ln = opaque_lane();
        for (int i = wv; i < TN / 64; i += WAVES) {
            const int n = min(col1 + 64 * i + ln, p.N - 1);
            lds_dma4(p.bias ? p.bias + n : &g_no_bias, (uint8_t*)(s_bias + slot * TN + 64 * i));
        }
    };
    auto dst_of = [&](int st, int l) __attribute__((always_inline)) {
        return smem + st * STAGE + (l < LA ? 1024 * (wv * LA + l) : TM * 128 + 1024 * (wv * LB + l - LA));
    };
    // load l of the 128 K bytes from k0 on (NOWHERE: no access) into stage st
    auto dma = [&](int k0, int st, int l) __attribute__((always_inline)) {
        const int j = l < LA ? l : 0, i = l < LA ? 0 : l - LA;
        if (l < LA) bA.load_lds(dst_of(st, l), oA[j], k0);
        else if (GLU && (wv * LB + i) / 2 % NF >= NC) bU.load_lds(dst_of(st, l), oB[i], k0);
        else bB.load_lds(dst_of(st, l), oB[i], k0);
    };
    // step s's chunks past K, in the stage that this wave's loads have filled
    auto end_of_k = [&](int s, int st) __attribute__((always_inline)) {
        if (128 * (s + 1) <= K) return;
        const int ln = opaque_lane(), ch0 = 16 * ((ln & 7) ^ (ln >> 4));
#pragma unroll
        for (int l = 0; l < NL; ++l) {
            const int r8 = l < LA ? wv * LA + l : wv * LB + l - LA;
            if (128 * s + (ch0 ^ (64 * (r8 & 1))) >= K) *(i32x4*)(dst_of(st, l) + 16 * ln) = i32x4{0, 0, 0, 0};
        }
    };
    // scales of steps s0 .. s0 + 15 of the tile being loaded: a thread has eight of a row's bytes, two dwords, and one block's float
    uint32_t sc[2];
    float sf = 0.f;
    auto scales_load = [&](int s0) __attribute__((always_inline)) {
        const int t = wv * 64 + opaque_lane(), at = s0 + 8 * (t & 1);
        const uint8_t* src = p.sa + (size_t)min(row1 + (t >> 1), p.M - 1) * KB;
        // (steps past the last one: any of the row's bytes, for products of zeros)
        if (p.words) {
#pragma unroll
            for (int h = 0; h < 2; ++h) sc[h] = *(const uint32_t*)(src + min(at + 4 * h, KB - 4));
        } else {
            uint32_t b[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) b[i] = src[min(at + i, KB - 1)];
#pragma unroll
            for (int h = 0; h < 2; ++h) sc[h] = b[4 * h] | b[4 * h + 1] << 8 | b[4 * h + 2] << 16 | b[4 * h + 3] << 24;
        }
        if (t < 2 * SCALE_STEPS) {
            // block t / 16: of the tile's columns (glu: of its gate columns, of its up columns)
            const int nb = (p.N + 127) / 128, c = GLU ? col1 / 128 + (t / SCALE_STEPS) * nb : min(col1 / 128 + t / SCALE_STEPS, nb - 1);
            const int s = s0 + t % SCALE_STEPS;
            sf = s < KB ? p.sb[(size_t)c * KB + s] : 0.f;
        }
    };
    auto scales_store = [&](int slot) __attribute__((always_inline)) {
        const int t = wv * 64 + opaque_lane(), row = t >> 1;
        uint8_t* to = s_scale + slot * SCALES + (8 * (t & 1) * (TM / 64) + row / 64) * 64 + (F32 ? row & 63 : (row & 15) * 4 + ((row >> 4) & 3));
#pragma unroll
        for (int i = 0; i < 8; ++i) to[i * TM] = (uint8_t)(sc[i / 4] >> (8 * (i % 4)));
        if (t < 2 * SCALE_STEPS) *(float*)(s_scale + slot * SCALES + SCALE_STEPS * TM + 4 * t) = sf;
    };

    // ---- multiply side
    f32x4 acc[MF][NF];
    auto zero_acc = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int a = 0; a < MF; ++a)
#pragma unroll
            for (int n = 0; n < NF; ++n) acc[a][n] = f32x4{0, 0, 0, 0};
    };
    const int lo = (lane & 15) * 128 + (((lane >> 4) ^ ((lane >> 1) & 7)) << 4);     // chunk q; chunk 4 + q at ^ 64
    const int loA = lo + mw * MF * 2048, loB = lo + TM * 128 + nw * NF * 2048;
    i32x8 fa[MF], fb[2];
    auto read_a = [&](int off, int a) __attribute__((always_inline)) {
        fa[a] = join(*(const i32x4*)(smem + loA + off + a * 2048), *(const i32x4*)(smem + (loA ^ 64) + off + a * 2048));
    };
    auto read_b = [&](int off, int n) __attribute__((always_inline)) {
        fb[n % 2] = join(*(const i32x4*)(smem + loB + off + n * 2048), *(const i32x4*)(smem + (loB ^ 64) + off + n * 2048));
    };
    int e[F32 ? MF : 1];                                         // scales of row m of each fragment; F32: of rows 4 q .. of one
    float f0 = 0.f, f1 = 0.f;
    // this wave's scales of step s (slot: of its 16 steps)
    auto read_scales = [&](int s, int slot) __attribute__((always_inline)) {
        const uint8_t* at = s_scale + slot * SCALES;
        const int i = s % SCALE_STEPS;
        if constexpr (F32) {
#pragma unroll
            for (int a = 0; a < MF; ++a) e[a] = *(const int*)(at + (i * (TM / 64) + mw) * 64 + 16 * a + 4 * (lane >> 4));
        } else e[0] = *(const int*)(at + (i * (TM / 64) + mw) * 64 + 4 * (lane & 15));
        const float* f = (const float*)(at + SCALE_STEPS * TM);
        f0 = f[(!GLU && TN > 128 ? nw * NF * 16 / 128 * SCALE_STEPS : 0) + i];
        if (GLU) f1 = f[SCALE_STEPS + i];
    };
    auto opaque_stage = [&](int st) __attribute__((always_inline)) {
        int off = st * STAGE;
        asm volatile("" : "+s"(off));
        return off;
    };
    // Step s in stage st; then stage st is loaded from K position k0 and the
    // fragments of the step after it are read. `pending`: scales loaded during
    // the step before go to LDS slot `put`; `fetch` >= 0: those from that step on are
    // loaded. nstep, nslot: the next step and its scales' slot.
    auto step = [&](int st, int nstep, int nslot, int k0, bool pending, int put, int fetch) __attribute__((always_inline)) {
        const int cur = opaque_stage(st), nxt_st = R == 2 ? st ^ 1 : (st + 1) % R, nxt = opaque_stage(nxt_st);
        int e0[F32 ? MF : 1];
#pragma unroll
        for (int a = 0; a < (F32 ? MF : 1); ++a) e0[a] = e[a];
        const float g0 = f0, g1 = f1;
        f32x4 x[DEPTH + 1];
        bf16x8 wa[F32 ? MF : 1][4], wb[4];
        if constexpr (F32) {
#pragma unroll
            for (int a = 0; a < MF; ++a)
#pragma unroll
                for (int i = 0; i < 4; ++i) wa[a][i] = widen(fa[a], i);
        }
        auto fma = [&](int k) __attribute__((always_inline)) {
            const int n = k / MF, a = k % MF;
            const float s = GLU && n >= NC ? g1 : g0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float y = x[k % (DEPTH + 1)][i];
                if constexpr (F32) y *= e8m0_f32((uint32_t)e0[a] >> (8 * i) & 255);
                acc[a][n][i] = __builtin_fmaf(y, s, acc[a][n][i]);
            }
            asm volatile("" : "+v"(acc[a][n]));
        };
        // the instructions up to k stay before the branch that follows (the
        // compiler would move them past it, to their multiply-adds, and hold the
        // fragments of two steps)
        auto issued = [&](int k) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < DEPTH; ++i) asm volatile("" : "+v"(x[(k - i) % (DEPTH + 1)]));
        };
        if (TM == 128) __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int k = 0; k < NK; ++k) {
            const int n = k / MF, a = k % MF;
            f32x4& y = x[k % (DEPTH + 1)];
            if constexpr (F32) {
                if (a == 0) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) wb[i] = widen(fb[n % 2], i);
                }
                y = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < 4; ++i) y = mfma_bf16_16x16x32(wa[a][i], wb[i], y);
            } else {
                if (a == 0) y = mfma_block<0>(fa[a], fb[n % 2], e0[0]);
                if (a == 1) y = mfma_block<1>(fa[a], fb[n % 2], e0[0]);
                if (a == 2) y = mfma_block<2>(fa[a], fb[n % 2], e0[0]);
                if (a == 3) y = mfma_block<3>(fa[a], fb[n % 2], e0[0]);
            }
            __builtin_amdgcn_sched_barrier(0);
            if (k >= DEPTH) fma(k - DEPTH);
            if (k == BAR) {
                if (TM == 128) __builtin_amdgcn_s_setprio(0);
                wait_vmcnt<(R - 2) * NL>();
                issued(k);
                if (pending) scales_store(put);
                end_of_k(nstep, nxt_st);
                barrier_lds();
                read_scales(nstep, nslot);
            }
            if (a == MF - 1) {
                if (n + 2 < NF) read_b(cur, n + 2);
                else read_b(nxt, n + 2 - NF);
            }
            if (n == NF - 1) read_a(nxt, a);
#pragma unroll
            for (int l = 0; l < NL; ++l)
                if (BAR + 1 + l * (NK - 1 - BAR) / NL == k) dma(k0, st, l);
            __builtin_amdgcn_sched_barrier(0);
        }
        issued(NK - 1);
        if (fetch >= 0) scales_load(fetch);
#pragma unroll
        for (int k = NK - DEPTH; k < NK; ++k) fma(k);
    };
    auto rows_out = [&](const float* md, auto with_add) __attribute__((always_inline)) {
        constexpr bool ADD = decltype(with_add)::value;
        const int ln = opaque_lane(), m = ln & 15, q = ln >> 4;
        const int cw = nw * 16 * NC + NC * m, col = col0 + cw;
        const bool full = ANY ? col + NC <= p.N : col < p.N;     // all of the lane's columns exist
        float bs[NC];
#pragma unroll
        for (int n = 0; n < NC; ++n) bs[n] = GLU ? -0.f : md[cw + n];
        // lane (m, q), register i of fragment (a, n): row 16 (mw MF + a) + 4 q + i
        auto values = [&](int a, int i, float (&v)[NC]) __attribute__((always_inline)) {
#pragma unroll
            for (int n = 0; n < NC; ++n) {
                if constexpr (GLU) v[n] = glu_h(acc[a][n][i], acc[a][n + NC][i]);
                else v[n] = acc[a][n][i] + bs[n];
            }
        };
#pragma unroll
        for (int a = 0; a < MF; ++a) {
            // the addends of NB rows are loaded together (rows and columns past
            // the output: from inside it, and dropped)
            constexpr int AB = F32 ? 2 : 4;
            Cols<NC, F32, ANY> plus[ADD ? AB : 1];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (ADD) {
                    if (i % AB == 0) {
#pragma unroll
                        for (int b = 0; b < AB; ++b) {
                            const int row = min(row0 + 16 * (mw * MF + a) + 4 * q + i + b, p.M - 1);
                            if (!ANY) plus[b].load(p.add, (size_t)row * p.N + (full ? col : 0));
                            else {
                                plus[b] = {};
                                if (full) plus[b].load(p.add, (size_t)row * p.N + col);
                            }
                        }
                    }
                }
                const int row = row0 + 16 * (mw * MF + a) + 4 * q + i;
                float v[NC];
                values(a, i, v);
                if constexpr (ADD) {
                    plus[i % AB].add_to(v);
                    // (used outside the masked store, or the wait for the addends sinks into it and into the next step loop)
#pragma unroll
                    for (int n = 0; n < NC; ++n) asm volatile("" : "+v"(v[n]));
                }
                if (row < p.M && full) Cols<NC, F32, ANY>::store(p.out, (size_t)row * p.N + col, v);
            }
        }
        // a wave in which the output's rows end inside a lane: that lane's columns
        if (!ANY || __ballot(!full && col < p.N) == 0) return;
        constexpr int RB = NC <= 4 ? 4 : 1;
#pragma unroll
        for (int a = 0; a < MF; ++a) {
#pragma unroll
            for (int i0 = 0; i0 < 4; i0 += RB) {
                const int row = row0 + 16 * (mw * MF + a) + 4 * q + i0;
                float v[RB][NC];
                __builtin_amdgcn_sched_barrier(0);       // (every row's values at once, or those of the loop above, would spill)
#pragma unroll
                for (int n = 0; n < NC; ++n) asm volatile("" : "+v"(bs[n]));
#pragma unroll
                for (int i = 0; i < RB; ++i) values(a, i0 + i, v[i]);
                if (full) continue;
                if constexpr (ADD) {
#pragma unroll
                    for (int i = 0; i < RB; ++i) add_each<NC, F32>(p, row + i, col, v[i]);
                }
#pragma unroll
                for (int i = 0; i < RB; ++i)
                    if (row + i < p.M) store_each<NC, F32>(p, row + i, col, v[i]);
            }
        }
    };
    auto epilogue = [&](int slot) __attribute__((always_inline)) {
        const float* md = s_bias + slot * TN;
        if (!GLU && p.add) rows_out(md, IC<!GLU>{});
        else rows_out(md, IC<0>{});
    };

    setup(0);
    bias(0);
    scales_load(0);
    scales_store(0);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int l = 0; l < NL; ++l) dma(128 * r, r, l);
    zero_acc();
    wait_vmcnt<(R - 1) * NL>();
    end_of_k(0, 0);
    barrier_lds();
    read_scales(0, 0);
#pragma unroll
    for (int a = 0; a < MF; ++a) read_a(opaque_stage(0), a);
    read_b(opaque_stage(0), 0);
    read_b(opaque_stage(0), 1);
    __builtin_amdgcn_s_waitcnt(0xC07F);                          // (lgkmcnt(0): left open, it would be waited for in every step)
    int st = 0, slot = 0;                                        // slot: of the scales of the step being multiplied
    bool pending = false;
    if constexpr (R > 2) {                                       // (one tile a workgroup)
        row0 = row1;
        col0 = col1;
#pragma clang loop unroll(disable)
        for (int s = 0; s < S; ++s, st = (st + 1) % R) {
            const bool turn = (s + 1) % SCALE_STEPS == 0, ask = (s + 2) % SCALE_STEPS == 0 && s + 2 < S;
            step(st, s + 1, slot ^ turn, s + R < S ? (s + R) * 128 : NOWHERE, pending, slot ^ 1, ask ? s + 2 : -1);
            slot ^= turn;
            pending = ask;
        }
        epilogue(0);
        return;
    }
#pragma clang loop unroll(disable)
    for (int j = 0; j < nj; ++j) {
        row0 = row1;
        col0 = col1;
        const int more = j + 1 < nj;
#pragma clang loop unroll(disable)
        for (int s = 0; s < S; ++s, st ^= 1) {
            const bool next = s == S - 2 && more, last = s == S - 1;
            if (next) setup(j + 1);                              // every load of tile j is out
            const bool turn = last || (s + 1) % SCALE_STEPS == 0;
            const bool ask = next || ((s + 2) % SCALE_STEPS == 0 && s + 2 < S);
            step(st, last ? 0 : s + 1, slot ^ turn, s + 2 < S ? (s + 2) * 128 : more ? (s + 2 - S) * 128 : NOWHERE, pending,
                 slot ^ 1, ask ? (next ? 0 : s + 2) : -1);
            slot ^= turn;
            pending = ask;
            if (next) bias((j + 1) & 1);
        }
        epilogue(j & 1);
        zero_acc();
    }
}

// ------------------------------------------------------------------ few tiles
// Smaller tiles, as in the int8 products: the waves of a workgroup share one TM x
// TN tile and take turns at its blocks of 128 K bytes, each with a stage of its
// own and no barrier in the loop; their fp32 sums meet in LDS, added in the
// waves' order. The instruction's rows are columns of the output here and its
// columns rows: a lane then has one row of A, whose scale byte it loads with the stage.
// 1 x 2048 x 2048 3.6 us (launch and first latency), 8 x 131072 x 2048 with fp32
// outputs 53.5 us from memory (5.1 TB/s, a copy's rate), 333 x 1000 x 4112 fp32 10.8 us:
// 176 tiles of 32 x 64 on 256 CUs, 66 MB from L2 to LDS, 26% of the vector unit for
// the widening.
template <int TM, int TN, int WK, bool GLU, bool F32>
__global__ void __launch_bounds__(64 * WK) gemm_fp8_split_kernel(Fp8Args p, int tiles_m, int tiles_n) {
    constexpr int MF = TM / 16, NF = TN / 16;
    constexpr int STAGE = (TM + TN) * 128;                       // 128 K bytes of the tile's rows
    constexpr int LD = (TM + TN) / 8;                            // 8-row loads of a stage
    constexpr int OUTN = GLU ? TN / 2 : TN;
    static_assert(TM * TN * 4 <= STAGE, "the waves' sums fit their stages");
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    float* s_bias = (float*)(smem + WK * STAGE);
    const int lane = lane_id();
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    // consecutive tiles share their B rows (the tall operand: the weights) on one XCD
    int L;
    {
        const int total = tiles_m * tiles_n;
        const int x = blockIdx.x & 7, i = blockIdx.x >> 3, per = total >> 3, rem = total & 7;
        L = x * per + min(x, rem) + i;
    }
    const int row0 = (L % tiles_m) * TM, col0 = (L / tiles_m) * OUTN;
    const int K = p.K, KB = (K + 127) / 128;

    // load j: 8 stage rows; lane i row i / 8 of them, chunk (i % 8) ^ ((row / 2) & 7)
    uint8_t* stage = smem + wv * STAGE;
    Operand bA, bB, bU;                                          // A, B (glu: its gate rows), glu's up rows
    bA.set(p.a + (size_t)row0 * K, (size_t)(p.M - row0) * K);
    bB.set(p.b + (size_t)col0 * K, (size_t)(p.N - col0) * K);
    if (GLU) bU.set(p.b + ((size_t)p.N + col0) * K, (size_t)(p.N - col0) * K);
    uint32_t off[LD];
#pragma unroll
    for (int j = 0; j < LD; ++j) {
        const int r = 8 * j + (lane >> 3), ch = 16 * ((lane & 7) ^ ((4 * j + (lane >> 4)) & 7));
        if (8 * j < TM) off[j] = row_offset(r, p.M - 1 - row0, K, ch);
        else off[j] = row_offset(r - TM - (GLU && 8 * j - TM >= OUTN ? OUTN : 0), p.N - 1 - col0, K, ch);
    }
    const int m = lane & 15, q = lane >> 4;
    const uint8_t* psa[MF];
#pragma unroll
    for (int a = 0; a < MF; ++a) psa[a] = p.sa + (size_t)min(row0 + 16 * a + m, p.M - 1) * KB;
    const float* psb = p.sb + (size_t)(col0 / 128) * KB;
    const float* psu = psb + (size_t)((p.N + 127) / 128) * KB;
    uint32_t e[MF];
    float f0, f1 = 0.f;
    auto fill = [&](int seg) __attribute__((always_inline)) {
#pragma unroll
        for (int a = 0; a < MF; ++a) e[a] = psa[a][seg];
        f0 = psb[seg];
        if (GLU) f1 = psu[seg];
#pragma unroll
        for (int j = 0; j < LD; ++j)
            (8 * j < TM ? bA : GLU && 8 * j - TM >= OUTN ? bU : bB).load_lds(stage + 1024 * j, off[j], seg * 128);
    };
    if (!GLU && p.bias) {
        for (int i = wv; i < (TN + 63) / 64; i += WK) lds_dma4(p.bias + min(col0 + 64 * i + lane, p.N - 1), (uint8_t*)(s_bias + 64 * i));
    }
    if (wv < KB) fill(wv);

    f32x4 acc[MF][NF];
#pragma unroll
    for (int a = 0; a < MF; ++a)
#pragma unroll
        for (int n = 0; n < NF; ++n) acc[a][n] = f32x4{0, 0, 0, 0};
    const int lo = m * 128 + ((q ^ ((m >> 1) & 7)) << 4);        // chunk q of fragment row m; chunk 4 + q at ^ 64
    for (int seg = wv; seg < KB; seg += WK) {
        wait_vmcnt<0>();
        asm volatile("" ::: "memory");                           // no read of the stage before the wait
        if (128 * (seg + 1) > K) {                               // chunks past K count as zero (NaN codes of the next row would not)
#pragma unroll
            for (int j = 0; j < LD; ++j)
                if (128 * seg + 16 * ((lane & 7) ^ ((4 * j + (lane >> 4)) & 7)) >= K)
                    *(i32x4*)(stage + 1024 * j + 16 * lane) = i32x4{0, 0, 0, 0};
        }
        i32x8 fa[MF], fb[NF];
#pragma unroll
        for (int a = 0; a < MF; ++a) fa[a] = join(*(const i32x4*)(stage + lo + a * 2048), *(const i32x4*)(stage + (lo ^ 64) + a * 2048));
#pragma unroll
        for (int n = 0; n < NF; ++n)
            fb[n] = join(*(const i32x4*)(stage + TM * 128 + lo + n * 2048), *(const i32x4*)(stage + TM * 128 + (lo ^ 64) + n * 2048));
        uint32_t ec[MF];
#pragma unroll
        for (int a = 0; a < MF; ++a) ec[a] = e[a];
        const float g0 = f0, g1 = f1;
        // the fragments are in registers before their stage is refilled
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(0xC07F);                      // lgkmcnt(0)
        __builtin_amdgcn_sched_barrier(0);
        if (seg + WK < KB) fill(seg + WK);
        if constexpr (F32) {
            bf16x8 wa[MF][4];
            float s[MF];
#pragma unroll
            for (int a = 0; a < MF; ++a) {
                s[a] = e8m0_f32(ec[a]);
#pragma unroll
                for (int i = 0; i < 4; ++i) wa[a][i] = widen(fa[a], i);
            }
#pragma unroll
            for (int n = 0; n < NF; ++n) {
                f32x4 x[MF];
#pragma unroll
                for (int a = 0; a < MF; ++a) x[a] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bf16x8 wb = widen(fb[n], i);
#pragma unroll
                    for (int a = 0; a < MF; ++a) x[a] = mfma_bf16_16x16x32(wb, wa[a][i], x[a]);
                }
#pragma unroll
                for (int a = 0; a < MF; ++a)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[a][n][i] = __builtin_fmaf(x[a][i] * s[a], g0, acc[a][n][i]);
            }
        } else {
#pragma unroll
            for (int n = 0; n < NF; ++n)
#pragma unroll
                for (int a = 0; a < MF; ++a) {
                    const f32x4 x = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb[n], fa[a], f32x4{0, 0, 0, 0}, 0, 0, 0, 127, 0, (int)ec[a]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[a][n][i] = __builtin_fmaf(x[i], GLU && n >= NF / 2 ? g1 : g0, acc[a][n][i]);
                }
        }
    }
    wait_vmcnt<0>();                                             // (a wave without a segment: its bias)
    barrier_lds();
    // output row 16 a + m, columns 16 n + 4 q ..: four columns c sit at c ^ the row, so that 16 rows meet every bank
    float* s_acc = (float*)smem;
    constexpr int QT = TN / 4;
#pragma unroll
    for (int a = 0; a < MF; ++a)
#pragma unroll
        for (int n = 0; n < NF; ++n)
            *(f32x4*)(s_acc + wv * TM * TN + (16 * a + m) * TN + 4 * ((4 * n + q) ^ (m & (QT - 1)))) = acc[a][n];
    barrier_lds();
    constexpr int QN = OUTN / 4;                                 // groups of 4 output columns of a row
#pragma unroll 2
    for (int t = threadIdx.x; t < TM * QN; t += 64 * WK) {
        const int r = t / QN, c = t % QN * 4;
        if (row0 + r >= p.M) continue;
        f32x4 g = {0, 0, 0, 0}, u = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < WK; ++w) {
            const float* s = s_acc + w * TM * TN + r * TN;
            g += *(const f32x4*)(s + 4 * ((c / 4) ^ (r & 15 & (QT - 1))));
            if (GLU) u += *(const f32x4*)(s + 4 * (((c + OUTN) / 4) ^ (r & 15 & (QT - 1))));
        }
        float v[4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            if constexpr (GLU) v[n] = glu_h(g[n], u[n]);
            else v[n] = p.bias ? g[n] + s_bias[c + n] : g[n];
        }
        const size_t o = (size_t)(row0 + r) * p.N + col0 + c;
        if (p.lines) {
            if (col0 + c >= p.N) continue;
            if (!GLU && p.add) {
                Cols<4, F32> plus;
                plus.load(p.add, o);
                plus.add_to(v);
            }
            Cols<4, F32>::store(p.out, o, v);
        } else if (col0 + c + 4 <= p.N) {
            if (!GLU && p.add) {
                Cols<4, F32, true> plus;
                plus.load(p.add, o);
                plus.add_to(v);
            }
            Cols<4, F32, true>::store(p.out, o, v);
        } else {
            if (!GLU && p.add) add_each<4, F32>(p, row0 + r, col0 + c, v);
            store_each<4, F32>(p, row0 + r, col0 + c, v);
        }
    }
}

// ------------------------------------------------------------------ launch
template <int TM, int TN, int WM, int WN, int R, bool GLU, bool F32, bool ANY>
static hipError_t launch_tile(const Fp8Args& p, int dev, int kid, hipStream_t stream) {
    constexpr int OUTN = GLU ? TN / 2 : TN;
    constexpr int SMEM = R * (TM + TN) * 128 + 2 * SCALE_STEPS * (TM + 8) + 8 * TN;
    constexpr int PER_CU = 163840 / SMEM < 8 / (WM * WN) ? 163840 / SMEM : 8 / (WM * WN);
    static std::atomic<uint64_t> done{0};
    const hipError_t e = allow_lds((const void*)gemm_fp8_tile_kernel<TM, TN, WM, WN, R, GLU, F32, ANY>, SMEM, dev, done);
    if (e != hipSuccess) return e;
    const int tm = (p.M + TM - 1) / TM, tn = (p.N + OUTN - 1) / OUTN;
    const int slots = (device_cus(dev) * PER_CU + 7) / 8 * 8, grid = min(slots, (tm * tn + 7) / 8 * 8);
    return launch_kernel(kid, stream, gemm_fp8_tile_kernel<TM, TN, WM, WN, R, GLU, F32, ANY>, dim3((unsigned)grid),
                         dim3(64 * WM * WN), SMEM, p, tm, tn);
}

template <int TM, int TN, int WK, bool GLU, bool F32>
static hipError_t launch_split(const Fp8Args& p, int dev, int kid, hipStream_t stream) {
    constexpr int OUTN = GLU ? TN / 2 : TN;
    constexpr int SMEM = WK * (TM + TN) * 128 + 256 * ((TN + 63) / 64);
    static std::atomic<uint64_t> done{0};
    const hipError_t e = allow_lds((const void*)gemm_fp8_split_kernel<TM, TN, WK, GLU, F32>, SMEM, dev, done);
    if (e != hipSuccess) return e;
    const int tm = (p.M + TM - 1) / TM, tn = (p.N + OUTN - 1) / OUTN;
    return launch_kernel(kid, stream, gemm_fp8_split_kernel<TM, TN, WK, GLU, F32>, dim3((unsigned)(tm * tn)),
                         dim3(64 * WK), SMEM, p, tm, tn);
}

template <bool GLU, bool F32>
static hipError_t launch_any(const Fp8Args& p, int kid, hipStream_t stream) {
    int dev = 0;
    const hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    const long long cus = device_cus(dev), rows_b = (long long)p.N * (GLU ? 2 : 1);
    const int shape = pick_shape(F32 ? kShapesFp8F32 : kShapesFp8, p.M, rows_b, p.K, cus);
    const bool few = shape_tiles(shape, p.M, rows_b) <= cus;             // at most one tile a CU
    if constexpr (!F32) {
        if (shape == S_256x256)
            return p.lines ? launch_tile<256, 256, 4, 2, 2, GLU, false, false>(p, dev, kid, stream)
                           : launch_tile<256, 256, 4, 2, 2, GLU, false, true>(p, dev, kid, stream);
    }
    if (shape == S_128x128) {
        if (few)
            return p.lines ? launch_tile<128, 128, 2, 2, 4, GLU, F32, false>(p, dev, kid, stream)
                           : launch_tile<128, 128, 2, 2, 4, GLU, F32, true>(p, dev, kid, stream);
        return p.lines ? launch_tile<128, 128, 2, 2, 2, GLU, F32, false>(p, dev, kid, stream)
                       : launch_tile<128, 128, 2, 2, 2, GLU, F32, true>(p, dev, kid, stream);
    }
    switch (shape) {
        case S_32x64:
            return few ? launch_split<32, 64, split_waves(S_32x64, true), GLU, F32>(p, dev, kid, stream)
                       : launch_split<32, 64, split_waves(S_32x64, false), GLU, F32>(p, dev, kid, stream);
        case S_32x32: return launch_split<32, 32, split_waves(S_32x32, false), GLU, F32>(p, dev, kid, stream);
        default:
            return few ? launch_split<64, 64, split_waves(S_64x64, true), GLU, F32>(p, dev, kid, stream)
                       : launch_split<64, 64, split_waves(S_64x64, false), GLU, F32>(p, dev, kid, stream);
    }
}

hipError_t launch_gemm_fp8(const uint8_t* a, const uint8_t* sa, const uint8_t* b, const float* sb, const float* bias,
                           const void* add, int M, int N, int K, bool f32, void* out, bool aligned, hipStream_t stream) {
    const Fp8Args p{a, sa, b, sb, bias, add, out, M, N, K, aligned && whole_lines(out, N, f32 ? 4 : 2),
                    (uintptr_t)sa % 4 == 0 && (K + 127) / 128 % 4 == 0};
    return f32 ? launch_any<false, true>(p, K_GEMM_FP8, stream) : launch_any<false, false>(p, K_GEMM_FP8, stream);
}

hipError_t launch_glu_fp8(const uint8_t* a, const uint8_t* sa, const uint8_t* w13, const float* s13, int M, int I, int K,
                          uint16_t* h, bool aligned, hipStream_t stream) {
    const Fp8Args p{a, sa, w13, s13, nullptr, nullptr, h, M, I, K, aligned && whole_lines(h, I, 2),
                    (uintptr_t)sa % 4 == 0 && (K + 127) / 128 % 4 == 0};
    return launch_any<true, false>(p, K_GLU_FP8, stream);
}

}  // namespace moe
