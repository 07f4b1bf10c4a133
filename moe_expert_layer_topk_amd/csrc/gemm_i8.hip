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
#include "gemm_tile.h"

namespace moe {

struct GemmArgs {
    const int8_t* a;
    const float* sa;
    const int8_t* b;
    const float* sb;
    const float* bias;        // may be null
    const void* add;          // may be null; the output's type
    void* out;
    int M, N, K;              // N: output columns (glu: inter; b then has 2N rows)
    int lines;                // output rows are whole 128-byte lines (and add's address is 16-byte aligned)
};

// One output before its addend, in this order in every kernel, so that its bits
// do not depend on the tile: the sum in fp32, the row's scale, the column's
// scale and the bias in one rounding. Addends come after it, and the compiler
// may not draw their addition into the product (contract(off) there).
__device__ __forceinline__ float scaled(int sum, float sa, float sb, float bias) {
    return __builtin_fmaf((float)sum * sa, sb, bias);
}

// ------------------------------------------------------------------ tiles
// TM x TN outputs (glu: TN rows of B = TN / 2 columns of h) by WM x WN waves,
// K in steps of 128 bytes through R LDS stages of TM + TN rows, each step two
// sub-steps of 64 bytes.
// A stage row's 16-byte chunk c sits at c ^ ((row / 2) & 7): 16-byte fragment
// reads of 16 consecutive rows then meet every bank once.
// B fragment f = nw NF + n, row m holds output column nw 16 NC + NC m + n (NC
// = NF), so the columns a lane accumulates are adjacent (glu: NC = NF / 2; the
// first half of a wave's fragments are gate rows, the second the matching up
// rows).
// Persistent: a workgroup's tiles form one stream of K steps. Sub-step 0's
// instructions run while sub-step 1's fragments are read. In sub-step 1 every
// fragment of the step is in registers; past a barrier its stage is refilled
// with the step R ahead (R = 2: the next tile's first ones at a tile's end, so
// they land during the epilogue) and the next step's first fragments are read.
// R = 4 has a loop of its own for one tile a workgroup: the loop over tiles
// with it took 14.5 us at 2048^3 instead of 12.7.
//
// Bound by the chip's power: on random codes the loop runs at 1.6-1.9 GHz
// (2.4 GHz on zeros, 1.4 times as fast), with the matrix pipe busy 75% of the
// clocks at 4096 x 8192 x 8192, 61% at 16384 x 2048 x 2048 and 55% at gated 16384
// x 512 x 2048, where two tiles' prologues and epilogues a CU count. So
// what counts is energy per output: 16x16x64 instructions (registers only: 3950
// TOPS on random codes; 32x32x32: 2920), tiles as large as LDS allows, few
// instructions beside the matrix ones. 8192^3: 409 us, 2690 TOPS (a library product with int32 output on the same card 457-465 us); 4096
// x 8192 x 8192 210 us (253); 16384 x 2048 x 2048 61 us (81); gated 16384 x 512
// x 2048 30.4 us. Measured without gain: 256 x 128 tiles with three stages, four
// 128 x 128 waves (the compiler spills), places of the barrier and the loads
// between the matrix instructions.
template <int TM, int TN, int WM, int WN, int R, bool GLU, bool F32, bool ANY>
__global__ void __launch_bounds__(64 * WM * WN, 2) gemm_tile_kernel(GemmArgs p, int tiles_m, int tiles_n) {
    constexpr int WAVES = WM * WN;
    constexpr int MF = TM / WM / 16, NF = TN / WN / 16;
    constexpr int STAGE = (TM + TN) * 128;
    constexpr int LA = TM / 8 / WAVES, LB = TN / 8 / WAVES;      // 8-row loads per wave and step
    constexpr int OUTN = GLU ? TN / 2 : TN;                      // output columns of a tile
    constexpr int NC = GLU ? NF / 2 : NF;                        // adjacent output columns of a lane
    constexpr int META = TM + 2 * TN;                            // floats: row scales, column scales, bias
    static_assert(LA >= 1 && LB >= 1 && TM % (8 * WAVES) == 0 && TN % (8 * WAVES) == 0 && TM % 64 == 0 && TN % 64 == 0, "tile");
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    float* s_meta = (float*)(smem + R * STAGE);                  // two tiles' worth
    const int lane = lane_id();
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int mw = wv / WN, nw = wv % WN;
    const int K = p.K, S = max(2, (K + 127) / 128);             // (a second step past K multiplies zeros)

    // this workgroup's tiles: start + idx + per_x j, j < nj. Each XCD takes a
    // run of consecutive tiles (blocks are dealt to the 8 XCDs in turn), and
    // runs go down groups of 8 row panels, so an XCD's L2 serves a few panels
    // of A and B at a time
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

    // ---- load side: load j of this wave fills stage rows 8 (wv LA + j) ..
    // (A; B after TM rows likewise); lane i: row i / 8 of them, chunk
    // (i % 8) ^ ((row / 2) & 7) of its source row. Buffer loads: 32-bit lane
    // offsets from the tile's first row, the K position in the descriptor, no
    // vector address arithmetic in the step loop. A step that K ends in runs on
    // into the next row, and past the operand's end the buffer's bounds check
    // drops the access, as it does for every access of a step past K in the
    // last row: the multiply side zeroes A there.
    // (Per-lane constants used once a tile are formed there, from an opaque copy
    // of the lane id: held across the step loop they would spill.)
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
    // the loaded tile's scales into metadata slot `slot`
    auto meta = [&](int slot) __attribute__((always_inline)) {
        const int ln = opaque_lane();
        float* md = s_meta + slot * META;
        for (int i = wv; i < TM / 64; i += WAVES)
            lds_dma4(p.sa + min(row1 + 64 * i + ln, p.M - 1), (uint8_t*)(md + 64 * i));
        for (int i = wv; i < TN / 64; i += WAVES) {
            const int c = 64 * i + ln;
            const int n = GLU ? min(col1 + c % OUTN, p.N - 1) + (c >= OUTN ? p.N : 0) : min(col1 + c, p.N - 1);
            lds_dma4(p.sb + n, (uint8_t*)(md + TM + 64 * i));
            if (!GLU) lds_dma4(p.bias ? p.bias + n : &g_no_bias, (uint8_t*)(md + TM + TN + 64 * i));
        }
    };
    // load l of the 128 K bytes from k0 on (NOWHERE: no access) into stage st
    auto dma = [&](int k0, int st, int l) __attribute__((always_inline)) {
        const int j = l < LA ? l : 0, i = l < LA ? 0 : l - LA;
        uint8_t* dst = smem + st * STAGE + (l < LA ? 1024 * (wv * LA + j) : TM * 128 + 1024 * (wv * LB + i));
        if (l < LA) bA.load_lds(dst, oA[j], k0);
        else if (GLU && (wv * LB + i) / 2 % NF >= NC) bU.load_lds(dst, oB[i], k0);
        else bB.load_lds(dst, oB[i], k0);
    };

    // ---- multiply side: lane (m, q) holds 16 K bytes of fragment row m, chunk 4 u + q in sub-step u
    i32x4 acc[MF][NF];
    auto zero_acc = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int a = 0; a < MF; ++a)
#pragma unroll
            for (int n = 0; n < NF; ++n) acc[a][n] = i32x4{0, 0, 0, 0};
    };
    // (sub-step 1's chunk is sub-step 0's ^ 4: byte offset ^ 64)
    const int lo = (lane & 15) * 128 + (((lane >> 4) ^ ((lane >> 1) & 7)) << 4);
    i32x4 fa[2][MF], fb[2][NF];
    constexpr int NK = MF * NF, NR = MF + NF, NL = LA + LB;
    // this lane's bytes of its wave's first A and B fragment, sub-step u of stage st
    const int loA = lo + mw * MF * 2048, loB = lo + TM * 128 + nw * NF * 2048;
    auto frags = [&](int st, int u) __attribute__((always_inline)) {
        int off = st * STAGE;
        asm volatile("" : "+s"(off));
        return make_int2((loA ^ (64 * u)) + off, (loB ^ (64 * u)) + off);
    };
    // fragment i of sub-step u, in the order the instructions take them
    auto read = [&](int2 f, int u, int i) __attribute__((always_inline)) {
        if (i == 0) fa[u][0] = *(const i32x4*)(smem + f.x);
        else if (i <= NF) fb[u][i - 1] = *(const i32x4*)(smem + f.y + (i - 1) * 2048);
        else fa[u][i - NF] = *(const i32x4*)(smem + f.x + (i - NF) * 2048);
    };
    // A is zero past K (s: the step; 16-byte chunk 4 u + lane / 16 of it)
    auto cut = [&](int s, int u) __attribute__((always_inline)) {
        if (128 * (s + 1) <= K) return;
        const bool out = 128 * s + 64 * u + 16 * (opaque_lane() >> 4) >= K;
#pragma unroll
        for (int a = 0; a < MF; ++a)
#pragma unroll
            for (int i = 0; i < 4; ++i) fa[u][a][i] = out ? 0 : fa[u][a][i];
    };
    // sub-step 0 of step s: multiply, and read sub-step 1 behind the first instructions
    auto half0 = [&](int s, int st) __attribute__((always_inline)) {
        const int2 f = frags(st, 1);
        cut(s, 0);
        // two workgroups on a CU: the one in its first half, which waits for
        // nothing, goes first (4096 x 2048 x 2048 19.6 -> 18.3 us; with one the
        // order does not matter)
        if (TM == 128) __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int k = 0; k < NK; ++k) {
            acc[k / NF][k % NF] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fa[0][k / NF], fb[0][k % NF], acc[k / NF][k % NF], 0, 0, 0);
            if (k < NR) read(f, 1, k);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // sub-step 1: after BAR instructions every wave's reads of the stage are
    // done and the other stage has landed; then that stage's first fragments
    // are read and this one is refilled (the loads spread over the rest)
    constexpr int BAR = 2;
    constexpr int LS = (NK - BAR) / NL > 0 ? (NK - BAR) / NL : 1;
    auto half1 = [&](int s, int st, int k0) __attribute__((always_inline)) {
        const int2 f = frags(R == 2 ? st ^ 1 : (st + 1) % R, 0);
        cut(s, 1);
        if (TM == 128) __builtin_amdgcn_s_setprio(0);
#pragma unroll
        for (int k = 0; k < NK; ++k) {
            acc[k / NF][k % NF] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fa[1][k / NF], fb[1][k % NF], acc[k / NF][k % NF], 0, 0, 0);
            if (k == BAR - 1) {
                wait_vmcnt<(R - 2) * NL>();
                barrier_lds();
            }
            if (k >= BAR - 1 && k - BAR + 1 < NR) read(f, 0, k - BAR + 1);
            if (k >= BAR && (k - BAR) % LS == 0 && (k - BAR) / LS < NL) dma(k0, st, (k - BAR) / LS);
            __builtin_amdgcn_sched_barrier(0);
        }
        static_assert((NK - 1 - BAR) / LS >= NL - 1 && NK - BAR + 1 > NR, "every load and read has its instruction");
    };
    auto rows_out = [&](const float* md, auto with_add) __attribute__((always_inline)) {
        constexpr bool ADD = decltype(with_add)::value;
        const int ln = opaque_lane(), m = ln & 15, q = ln >> 4;
        const int cw = nw * 16 * NC + NC * m, col = col0 + cw;
        const bool full = ANY ? col + NC <= p.N : col < p.N;     // all of the lane's columns exist
        float sb[NF], bias[NC];
#pragma unroll
        for (int n = 0; n < NF; ++n) sb[n] = md[TM + (GLU && n >= NC ? OUTN : 0) + cw + n % NC];
#pragma unroll
        for (int n = 0; n < NC; ++n) bias[n] = GLU ? -0.f : md[TM + TN + cw + n];
        // lane (m, q), register i of fragment (a, n): row 16 (mw MF + a) + 4 q + i
        auto values = [&](int a, int i, float sa, float (&v)[NC]) __attribute__((always_inline)) {
#pragma unroll
            for (int n = 0; n < NC; ++n) {
                v[n] = scaled(acc[a][n][i], sa, sb[n], bias[n]);
                if constexpr (GLU) v[n] = glu_h(v[n], scaled(acc[a][n + NC][i], sa, sb[n + NC], -0.f));
            }
        };
#pragma unroll
        for (int a = 0; a < MF; ++a) {
            const f32x4 sa = *(const f32x4*)(md + 16 * (mw * MF + a) + 4 * q);
            // the addends of NB rows are loaded together (rows and columns past
            // the output: from inside it, and dropped)
            constexpr int NB = F32 ? 2 : 4;
            Cols<NC, F32, ANY> plus[ADD ? NB : 1];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (ADD) {
                    if (i % NB == 0) {
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
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
                values(a, i, sa[i], v);
                if constexpr (ADD) {
                    plus[i % NB].add_to(v);
                    // used outside the masked store: otherwise the wait for
                    // the addends sinks into it, and where no lane stores
                    // they stay in flight and the step loop waits, every
                    // step, before it reuses their registers (226 -> 242 us
                    // at 4096 x 8192 x 8192, which has no addend)
#pragma unroll
                    for (int n = 0; n < NC; ++n) asm volatile("" : "+v"(v[n]));
                }
                if (row < p.M && full) Cols<NC, F32, ANY>::store(p.out, (size_t)row * p.N + col, v);
            }
        }
        // a wave in which the output's rows end inside a lane: that lane's
        // columns (the addends of RB rows before their stores, which could be
        // the same memory: one after the other, each would wait for memory)
        if (!ANY || __ballot(!full && col < p.N) == 0) return;
        constexpr int RB = NC <= 4 ? 4 : 1;
#pragma unroll
        for (int a = 0; a < MF; ++a) {
            const f32x4 sa = *(const f32x4*)(md + 16 * (mw * MF + a) + 4 * q);
#pragma unroll
            for (int i0 = 0; i0 < 4; i0 += RB) {
                const int row = row0 + 16 * (mw * MF + a) + 4 * q + i0;
                float v[RB][NC];
                __builtin_amdgcn_sched_barrier(0);       // (every row's values at once would spill)
#pragma unroll
                for (int i = 0; i < RB; ++i) values(a, i0 + i, sa[i0 + i], v[i]);
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
        const float* md = s_meta + slot * META;
        if (!GLU && p.add) rows_out(md, IC<!GLU>{});
        else rows_out(md, IC<0>{});
    };

    setup(0);
    meta(0);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int l = 0; l < NL; ++l) dma(128 * r, r, l);
    zero_acc();
    wait_vmcnt<(R - 1) * NL>();
    barrier_lds();
#pragma unroll
    for (int i = 0; i < NR; ++i) read(frags(0, 0), 0, i);
    int st = 0;
    if constexpr (R > 2) {                                       // (one tile a workgroup)
        row0 = row1;
        col0 = col1;
        for (int s = 0; s < S; ++s, st = (st + 1) % R) {
            half0(s, st);
            half1(s, st, s + R < S ? (s + R) * 128 : NOWHERE);
        }
        epilogue(0);
        return;
    }
    for (int j = 0; j < nj; ++j) {
        row0 = row1;
        col0 = col1;
        const int more = j + 1 < nj;
        for (int s = 0; s < S; ++s, st ^= 1) {
            half0(s, st);
            const bool next = s == S - 2 && more;
            if (next) setup(j + 1);                              // every load of tile j is out
            half1(s, st, s + 2 < S ? (s + 2) * 128 : more ? (s + 2 - S) * 128 : NOWHERE);
            if (next) meta((j + 1) & 1);                         // (after half1's wait and barrier)
        }
        epilogue(j & 1);
        zero_acc();
    }
}

// ------------------------------------------------------------------ few tiles
// Smaller tiles, for outputs that large tiles would spread over too few CUs.
// The waves of a workgroup share one TM x TN tile and take turns at its K
// segments of 128 bytes: wave k multiplies segments k, k + WK, ... of the whole
// tile, which reads half as much LDS per matrix instruction as splitting the
// tile (a 64 x 64 tile in four 32 x 32 quarters), and their int32 sums meet in
// LDS at the end, where the epilogue takes them in row order.
// Each wave has a stage of its own, fills it, waits for its own loads alone and
// refills it once the fragments are in registers: no barrier in the loop, and
// waves that drift apart cover each other's waits. One stage and more waves, or
// more workgroups on a CU, beat more stages (a barrier for each step and four
// shared stages: 333 x 1000 x 4112 9.8 us, this 8.9; 256 x 2048 x 2048 5.6 and
// 5.0; 481 x 2496 x 1632 10.9 and 9.6; two or three stages a wave in between).
// With one row the weights stream at HBM's rate: 1 x 8192 x 8192 takes 13.3 us,
// 5.05 TB/s, with twelve weight matrices in turn (a 1 GiB copy on the same card:
// 5.1), and 10.7 us where the one matrix of 67 MB stays in the last-level cache.
// Below 2048 x 2048 most of it is launch and first latency (4.0 us). With more
// rows, bound by L2 to LDS loads (about 50 bytes a clock and CU). A kernel that
// streamed B straight into registers for up to 32 rows was no faster at one
// row and up to 1.4 times slower at 16.
template <int TM, int TN, int WK, bool GLU, bool F32>
__global__ void __launch_bounds__(64 * WK) gemm_split_kernel(GemmArgs p, int tiles_m, int tiles_n) {
    constexpr int MF = TM / 32, NF = TN / 32;
    constexpr int STAGE = (TM + TN) * 128;                       // 128 K bytes of the tile's rows
    constexpr int LD = (TM + TN) / 8;                            // 8-row loads of a stage
    constexpr int OUTN = GLU ? TN / 2 : TN;
    static_assert(TM * TN * 4 <= STAGE, "the waves' sums fit their stages");
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    float* s_sa = (float*)(smem + WK * STAGE);
    float* s_sb = s_sa + 64 * ((TM + 63) / 64);
    float* s_bias = s_sb + 64 * ((TN + 63) / 64);
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
    const int K = p.K, segs = (K + 127) / 128;

    // load j: 8 stage rows; lane i row i / 8 of them, chunk (i % 8) ^ ((row / 2)
    // & 7). A segment that K ends in runs on into the next row, and past the
    // operand's end nothing is read: the multiply side zeroes A there.
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
    auto fill = [&](int seg) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < LD; ++j)
            (8 * j < TM ? bA : GLU && 8 * j - TM >= OUTN ? bU : bB).load_lds(stage + 1024 * j, off[j], seg * 128);
    };
    for (int i = wv; i < (TM + 63) / 64; i += WK)
        lds_dma4(p.sa + min(row0 + 64 * i + lane, p.M - 1), (uint8_t*)(s_sa + 64 * i));
    for (int i = wv; i < (TN + 63) / 64; i += WK) {
        const int c = 64 * i + lane;
        const int n = GLU ? min(col0 + c % OUTN, p.N - 1) + (c >= OUTN && c < TN ? p.N : 0) : min(col0 + c, p.N - 1);
        lds_dma4(p.sb + n, (uint8_t*)(s_sb + 64 * i));
        if (!GLU && p.bias) lds_dma4(p.bias + n, (uint8_t*)(s_bias + 64 * i));
    }
    if (wv < segs) fill(wv);

    i32x16 acc[MF][NF];
#pragma unroll
    for (int a = 0; a < MF; ++a)
#pragma unroll
        for (int n = 0; n < NF; ++n)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[a][n][i] = 0;
    const int m = lane & 31, hi = lane >> 5;
    // lane (m, hi) holds 16 K bytes of fragment row m, chunk 2 u + hi of sub-step u
    int lo[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) lo[u] = m * 128 + (((2 * u + hi) ^ ((m >> 1) & 7)) << 4);
    for (int seg = wv; seg < segs; seg += WK) {
        wait_vmcnt<0>();
        asm volatile("" ::: "memory");                           // no read of the stage before the wait
        i32x4 fa[4][MF], fb[4][NF];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
#pragma unroll
            for (int a = 0; a < MF; ++a) fa[u][a] = *(const i32x4*)(stage + lo[u] + a * 4096);
#pragma unroll
            for (int n = 0; n < NF; ++n) fb[u][n] = *(const i32x4*)(stage + lo[u] + TM * 128 + n * 4096);
        }
        if (128 * (seg + 1) > K) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const bool out = 128 * seg + 32 * u + 16 * hi >= K;
#pragma unroll
                for (int a = 0; a < MF; ++a)
#pragma unroll
                    for (int i = 0; i < 4; ++i) fa[u][a][i] = out ? 0 : fa[u][a][i];
            }
        }
        // the fragments are in registers before their stage is refilled
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(0xC07F);                      // lgkmcnt(0)
        __builtin_amdgcn_sched_barrier(0);
        if (seg + WK < segs) fill(seg + WK);
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int a = 0; a < MF; ++a)
#pragma unroll
                for (int n = 0; n < NF; ++n)
                    acc[a][n] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fa[u][a], fb[u][n], acc[a][n], 0, 0, 0);
    }
    wait_vmcnt<0>();                                             // (a wave without a segment: its scales)
    barrier_lds();
    int* s_acc = (int*)smem;
#pragma unroll
    for (int a = 0; a < MF; ++a)
#pragma unroll
        for (int n = 0; n < NF; ++n)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                s_acc[wv * TM * TN + (32 * a + 8 * (i / 4) + 4 * hi + i % 4) * TN + 32 * n + m] = acc[a][n][i];
    barrier_lds();
    constexpr int QN = OUTN / 4;                                 // groups of 4 output columns of a row
#pragma unroll 2
    for (int t = threadIdx.x; t < TM * QN; t += 64 * WK) {
        const int r = t / QN, c = t % QN * 4;
        if (row0 + r >= p.M) continue;
        i32x4 g = {0, 0, 0, 0}, u = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < WK; ++w) {
            g += *(const i32x4*)(s_acc + w * TM * TN + r * TN + c);
            if (GLU) u += *(const i32x4*)(s_acc + w * TM * TN + r * TN + c + OUTN);
        }
        const float sa = s_sa[r];
        float v[4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            v[n] = scaled(g[n], sa, s_sb[c + n], !GLU && p.bias ? s_bias[c + n] : -0.f);
            if constexpr (GLU) v[n] = glu_h(v[n], scaled(u[n], sa, s_sb[OUTN + c + n], -0.f));
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
static hipError_t launch_tile(const GemmArgs& p, int dev, int kid, hipStream_t stream) {
    constexpr int OUTN = GLU ? TN / 2 : TN;
    constexpr int SMEM = R * (TM + TN) * 128 + 8 * (TM + 2 * TN);
    constexpr int PER_CU = 163840 / SMEM < 8 / (WM * WN) ? 163840 / SMEM : 8 / (WM * WN);
    static std::atomic<uint64_t> done{0};
    const hipError_t e = allow_lds((const void*)gemm_tile_kernel<TM, TN, WM, WN, R, GLU, F32, ANY>, SMEM, dev, done);
    if (e != hipSuccess) return e;
    const int tm = (p.M + TM - 1) / TM, tn = (p.N + OUTN - 1) / OUTN;
    const int slots = (device_cus(dev) * PER_CU + 7) / 8 * 8, grid = min(slots, (tm * tn + 7) / 8 * 8);
    return launch_kernel(kid, stream, gemm_tile_kernel<TM, TN, WM, WN, R, GLU, F32, ANY>, dim3((unsigned)grid),
                         dim3(64 * WM * WN), SMEM, p, tm, tn);
}

template <int TM, int TN, int WK, bool GLU, bool F32>
static hipError_t launch_split(const GemmArgs& p, int dev, int kid, hipStream_t stream) {
    constexpr int OUTN = GLU ? TN / 2 : TN;
    constexpr int SMEM = WK * (TM + TN) * 128 + 256 * ((TM + 63) / 64 + 2 * ((TN + 63) / 64));
    static std::atomic<uint64_t> done{0};
    const hipError_t e = allow_lds((const void*)gemm_split_kernel<TM, TN, WK, GLU, F32>, SMEM, dev, done);
    if (e != hipSuccess) return e;
    const int tm = (p.M + TM - 1) / TM, tn = (p.N + OUTN - 1) / OUTN;
    return launch_kernel(kid, stream, gemm_split_kernel<TM, TN, WK, GLU, F32>, dim3((unsigned)(tm * tn)),
                         dim3(64 * WK), SMEM, p, tm, tn);
}

template <bool GLU, bool F32>
static hipError_t launch_any(const GemmArgs& p, int kid, hipStream_t stream) {
    int dev = 0;
    const hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    const long long cus = device_cus(dev), rows_b = (long long)p.N * (GLU ? 2 : 1);
    const int shape = pick_shape(p.M, rows_b, p.K, cus);
    const bool few = shape_tiles(shape, p.M, rows_b) <= cus;             // at most one tile a CU
    switch (shape) {
        case S_256x256:
            return p.lines ? launch_tile<256, 256, 4, 2, 2, GLU, F32, false>(p, dev, kid, stream)
                           : launch_tile<256, 256, 4, 2, 2, GLU, F32, true>(p, dev, kid, stream);
        case S_128x128:
            // at most one tile a CU: one stage in flight does not cover a load
            // (us with two stages / with four: 16384 x 256 x 7168 52.9 / 41.4,
            // 2048 x 2048 x 8192 42.0 / 36.4, 2048^3 14.2 / 12.7, 2048 x 2048 x
            // 512 6.6 / 6.7); with more, two of two stages share the CU's LDS
            if (few)
                return p.lines ? launch_tile<128, 128, 2, 2, 4, GLU, F32, false>(p, dev, kid, stream)
                               : launch_tile<128, 128, 2, 2, 4, GLU, F32, true>(p, dev, kid, stream);
            return p.lines ? launch_tile<128, 128, 2, 2, 2, GLU, F32, false>(p, dev, kid, stream)
                           : launch_tile<128, 128, 2, 2, 2, GLU, F32, true>(p, dev, kid, stream);
        case S_64x64:
            return few ? launch_split<64, 64, split_waves(S_64x64, true), GLU, F32>(p, dev, kid, stream)
                       : launch_split<64, 64, split_waves(S_64x64, false), GLU, F32>(p, dev, kid, stream);
        case S_32x64:
            return few ? launch_split<32, 64, split_waves(S_32x64, true), GLU, F32>(p, dev, kid, stream)
                       : launch_split<32, 64, split_waves(S_32x64, false), GLU, F32>(p, dev, kid, stream);
        default: return launch_split<32, 32, split_waves(S_32x32, false), GLU, F32>(p, dev, kid, stream);
    }
}

hipError_t launch_gemm_i8(const int8_t* a, const float* sa, const int8_t* b, const float* sb, const float* bias,
                          const void* add, int M, int N, int K, bool f32, void* out, bool aligned, hipStream_t stream) {
    const GemmArgs p{a, sa, b, sb, bias, add, out, M, N, K, aligned && whole_lines(out, N, f32 ? 4 : 2)};
    return f32 ? launch_any<false, true>(p, K_GEMM_I8, stream) : launch_any<false, false>(p, K_GEMM_I8, stream);
}

hipError_t launch_glu_i8(const int8_t* a, const float* sa, const int8_t* w13, const float* s13, int M, int I, int K,
                         uint16_t* h, bool aligned, hipStream_t stream) {
    const GemmArgs p{a, sa, w13, s13, nullptr, nullptr, h, M, I, K, aligned && whole_lines(h, I, 2)};
    return launch_any<true, false>(p, K_GLU_I8, stream);
}

}  // namespace moe
