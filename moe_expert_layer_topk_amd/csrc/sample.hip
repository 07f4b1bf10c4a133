// One token per row of logits: temperature, top-k, top-p, min-p and the draw
// from a given random number.
//
// The kept tokens are a prefix of the order (logit falling, id rising), so one
// border, a (logit, id), describes them: every token before it or equal to it,
// with w >= min_p. The draw is a search in the sums of their weights by id.
//
// chunk kernel: one workgroup for each 4096 logits, which it reads once and
// holds in registers. It writes the chunk's largest and smallest logit, its
// weight and, for rows with a filter, the tokens that the filter could keep, in the
// order of their ids. A chunk can tell from itself alone, with m its largest
// logit, S its weight (relative to m), V the row's length:
//   top_k: a token that k tokens of the chunk precede is out;
//   min_p: the row's largest logit is m at least, so w < min_p relative to m is out;
//   top_p: at least (1 - top_p) of the weight lies at and behind the last kept
//     token, on at most V tokens that weigh no more than it, so w < (1 - top_p) S / V is out.
// With top_k and top_p only the first holds: top_p's share is one of the weight
// of all k tokens. A chunk writes no more than its share of a row's LIST; where
// it has more candidates, it writes the first of the order and the largest
// logit that it left out.
// finish kernel: one workgroup a row. Counts and weights of 2048 equal parts of
// the candidates' range say which part holds a border, and its tokens, put in
// order, where. It holds if it lies before every logit that was left out
// (nearly always, with a filter); else (a top_p or min_p that keeps thousands of
// tokens) the chunks' weights by steps of an eighth of the temperature say in
// which step it lies, and the row is read again for that step's tokens; and where
// these are too many (equal logits), the same is done with all of the row's. No
// filter: the chunk that the draw falls into is read again.
//
// Weights are fp64, sums of them fp64 in a fixed order; the parts' and the steps'
// weights are summed with atomics, and therefore as integers (multiples of 2^-42 of
// the largest weight).
//
// What bounds it: rows x 131072 logits want the copy's rate, 5 TB/s, and the chunk
// kernel's vector unit is busy before that. 256 x 131072 fp32 (134 MB, 26.6 us to
// copy), vector instructions of a wave for its 16 logits a lane, us of the two kernels:
//   greedy              334   25 +  5   the logit's place in the order, a largest one in 64 bits
//   no filter           521   37 +  7   an exponential, 20 instructions a logit (14 of them fp64)
//   top_k of 50         486   34 + 10   no exponential but the choice of candidates: by the listing 190 for
//                                       their writes (one predicated for each element), 100 for the bound by the
//                                       threads' largest, 60 for the mask, 36 for the places, 37 for the row's parameters
//   top_p alone        1358   81 + 43   exponentials, a 64-bit addition in LDS for each logit's step, then candidates
//   all four            614   42 + 14   four fifths of these rows have top_k: as that, and parts where candidates are many
// The row kernels of top_p alone wait for one workgroup that reads a row again
// (thousands of kept tokens); likewise 52..57 us with all four, and 62..70 where one of
// the rows keeps thousands. The bf16 row kernels spill 8 vector registers (224 bytes of
// scratch a lane; the fp32 ones spill scalars alone, 160 bytes): 256 x 131072 with
// top_k and top_p, rows without top_k among them, 48 + 43 us, fp32 48 + 36. More rows
// than CUs are a second round of workgroups that have a CU each (100 KB of LDS): 512 x
// 16000 21 + 36. One row of 131072 is launch and
// latency: 12 us with top_k of 20 (chunks 7, row 5..12), 19 with several hundred, 40
// where thousands are kept; up to 4096 logits are one kernel, 6 us. (One workgroup
// of 1024 threads for a row of any length took 1580 us at 131072, chunks of
// 16384 logits 26 us where those of 4096 take 19.)
#include "moe_common.h"
#include "moe_kernels.h"
#include "gemm_tile.h"
#include "sample_plan.h"

namespace moe {

constexpr int ST = 1024;                                         // threads of a finish workgroup
constexpr int CHUNK = 4096;                                      // logits of a chunk
constexpr int MAX_CHUNKS = MOE_SAMPLE_MAX_COLS / CHUNK;
constexpr int LIST = 4096;                                       // candidates of a row
constexpr int RUN = LIST / ST;                                   // of a thread
constexpr int BINS = 2048;
constexpr double ONE = 4398046511104.0;                          // 2^42: the sum of 2^20 weights stays below 2^63
constexpr float INF = __builtin_inff();
constexpr int STEPS = 256;                                       // a chunk's steps of an eighth of the temperature

struct Chunk {
    double sum;               // weight relative to `top`
    float top, low;           // largest (+inf: NaN or +inf among them) and smallest logit that is not -inf
    float cut;                // largest candidate that is not written; -inf: all are
    int n;                    // candidates that are
};

// larger float, larger key; zeros of both signs are one value
__device__ __forceinline__ uint32_t logit_key(float f) {
    const uint32_t b = __float_as_uint(f + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_logit(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k); }
// a token's place in the order: larger comes first
__device__ __forceinline__ uint64_t place_of(float x, int id) { return (uint64_t)logit_key(x) << 32 | (uint32_t)~id; }
__device__ __forceinline__ float place_logit(uint64_t p) { return key_logit((uint32_t)(p >> 32)); }
__device__ __forceinline__ int place_id(uint64_t p) { return (int)~(uint32_t)p; }

// 2^(i / 32)
__device__ const double g_two[32] = {
    1.0, 1.0218971486541166, 1.0442737824274138, 1.0671404006768237,
    1.0905077326652577, 1.1143867425958924, 1.1387886347566916, 1.1637248587775775,
    1.189207115002721, 1.215247359980469, 1.241857812073484, 1.2690509571917332,
    1.2968395546510096, 1.3252366431597413, 1.3542555469368927, 1.383909881963832,
    1.4142135623730951, 1.4451808069770467, 1.4768261459394993, 1.5091644275934228,
    1.5422108254079407, 1.5759808451078865, 1.6104903319492543, 1.645755478153965,
    1.681792830507429, 1.718619298122478, 1.7562521603732995, 1.7947090750031072,
    1.8340080864093424, 1.8741676341103, 1.9152065613971474, 1.9571441241754002};
// e^(d inv) for d <= 0, scale = 32 inv / ln 2: 2^(n / 32) e^r with |r| <= ln 2 / 64
// and Taylor's polynomial of e^r to r^5 (the rest is below 3e-15); 1 for 0, 0
// far below 2^-1022. `two`: the table in LDS (32 entries, 64 banks), where it saves
// six of the eleven steps that a whole power of two would leave to the polynomial.
__device__ __forceinline__ double exp_neg(double d, double scale, const double* two) {
    // (bounded first: y - n of an unbounded product may be contracted to what the product's
    // rounding left, 1e70 and more, and r^5 of that to infinity)
    const double y = fmax(d * scale, -40000.0), n = __builtin_rint(y);
    const double r = (y - n) * 0.0216608493924982909;            // ln 2 / 32
    double f = 1.0 / 120.0;
    f = __builtin_fma(f, r, 1.0 / 24.0);
    f = __builtin_fma(f, r, 1.0 / 6.0);
    f = __builtin_fma(f, r, 0.5);
    f = __builtin_fma(f, r, 1.0);
    f = __builtin_fma(f, r, 1.0);
    const int e = (int)n;
    return __builtin_ldexp(f * two[e & 31], e >> 5);
}

// e^((x - top) inv), 0 for -inf (below the bound, also times 0). (Without a branch: in
// one for each element the chains of a thread's elements wait for themselves; 16 of
// them 5600 -> 3100 clocks.)
__device__ __forceinline__ double weight_of(float x, double top, double scale, const double* two) {
    return exp_neg((double)x - top, scale, two);
}
// a weight's mass: the nearest multiple of 2^-42, from where 2^52 + w 2^42 has its bits
__device__ __forceinline__ uint64_t mass_of(double w) {
    return __builtin_bit_cast(uint64_t, __builtin_fma(w, ONE, 4503599627370496.0)) & 0xFFFFFFFFFFFFFull;
}

// a row's parameters
struct Request {
    double scale, top_p, min_p;// 32 / (ln 2 temperature), 0 for infinity
    float temperature;
    int k;                     // 0: off
    bool bad, p_on, m_on;
    __device__ __forceinline__ Request(const SampleArgs& a, int r) {
        temperature = a.temperature ? a.temperature[r] : 1.f;
        const float u = a.u[r], tp = a.top_p ? a.top_p[r] : 1.f, mp = a.min_p ? a.min_p[r] : 0.f;
        bad = !(u >= 0.f && u <= 1.f) || !(temperature >= 0.f) || tp != tp || !(mp <= 1.f);
        scale = temperature > 0.f ? 46.16624130844682903552 / (double)temperature : 0.0;
        k = temperature == 0.f ? 1 : a.top_k ? kept_by_count(a.top_k[r]) : 0;
        top_p = tp > 0.f ? tp : 0.f;
        min_p = mp > 0.f ? mp : 0.f;
        p_on = tp < 1.f && k != 1;
        m_on = mp > 0.f && k != 1;
    }
    // The step that a logit is in: they are an eighth of the temperature wide and the
    // same for every chunk. Monotone in x; clamped where an int would not hold it.
    __device__ __forceinline__ int step(float x) const {
        return (int)floorf(fminf(fmaxf(x * (8.f / temperature), -1e9f), 1e9f));
    }
    // a logit below which the weight does not reach w beside a logit of m (the
    // hardware's logarithm and fp32's steps are far within the 1e-5)
    __device__ __forceinline__ float least(float m, double w) const {
        const float f = (float)w;
        if (!(f > 0.f) || temperature == INF) return -INF;
        const float d = __builtin_amdgcn_logf(f) * 0.693147181f * temperature;
        return m + d - (fabsf(m) + fabsf(d) + temperature) * 1e-5f;
    }
    // with `m` the largest logit and `sum` the weight of (a part of) the row:
    // tokens below are not kept, or weigh less than 2^-46 of the largest
    __device__ __forceinline__ float floor(float m, double sum, int V) const {
        double w = 1.0 / 70368744177664.0;
        if (!(k && p_on)) {
            if (m_on) w = fmax(w, min_p);
            if (p_on) w = fmax(w, (1.0 - top_p) * sum / V);
        }
        return least(m, fmin(w, 1.0));
    }
};

// four consecutive logits from element i on, which the row has
template <bool F32>
__device__ __forceinline__ void load_four(const void* row, int i, float (&x)[4]) {
    typedef uint32_t w4 __attribute__((ext_vector_type(4)));
    typedef uint32_t w2 __attribute__((ext_vector_type(2)));
    typedef w4 place4 __attribute__((aligned(4)));
    typedef w2 place2 __attribute__((aligned(2)));
    if (F32) {
        const w4 v = *(const place4*)((const float*)row + i);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = __uint_as_float(v[j]);
    } else {
        const w2 v = *(const place2*)((const uint16_t*)row + i);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = __uint_as_float(j & 1 ? v[j / 2] & 0xFFFF0000u : v[j / 2] << 16);
    }
}
// N fours, `step` elements apart, -inf from element V on. Where all of `all`
// elements from `base` on are there (the same for a wave), the loads go out
// together, without a branch for each.
template <bool F32, int N>
__device__ __forceinline__ void load_fours(const void* row, int i, int step, int base, int all, int V, float (&x)[N][4]) {
    if (base + all <= V) {
#pragma unroll
        for (int n = 0; n < N; ++n) load_four<F32>(row, i + n * step, x[n]);
    } else {
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int e = i + n * step + j;
                x[n][j] = e < V ? (F32 ? ((const float*)row)[e] : bf16_to_f32(((const uint16_t*)row)[e])) : -INF;
            }
    }
}

// ---- over a wave by lane moves in the vector unit
// (lanes that get nothing: `none`; ZERO: 0, which a move within rows gives by itself)
template <int CTRL, int ROWS, bool ZERO, typename T>
__device__ __forceinline__ T moved(T v, T none) {
    constexpr bool FILL = ZERO && ROWS == 0xF;
    if constexpr (sizeof(T) == 4) {
        return __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, none), __builtin_bit_cast(int, v), CTRL, ROWS, 0xF, FILL));
    } else {
        const int2 a = __builtin_bit_cast(int2, v), b = __builtin_bit_cast(int2, none);
        return __builtin_bit_cast(T, make_int2(__builtin_amdgcn_update_dpp(b.x, a.x, CTRL, ROWS, 0xF, FILL),
                                               __builtin_amdgcn_update_dpp(b.y, a.y, CTRL, ROWS, 0xF, FILL)));
    }
}
struct Plus {
    static constexpr bool ZERO = true;
    template <typename T>
    __device__ __forceinline__ static T of(T x, T y) { return x + y; }
    template <typename T>
    __device__ __forceinline__ static T none() { return (T)0; }
};
struct Most {
    static constexpr bool ZERO = false;
    template <typename T>
    __device__ __forceinline__ static T of(T x, T y) { return x > y ? x : y; }
    template <typename T>
    __device__ __forceinline__ static T none() { return __is_same(T, float) ? (T)-INF : (T)(__is_same(T, int) ? -0x7FFFFFFF - 1 : 0); }
};
struct Least {
    static constexpr bool ZERO = false;
    template <typename T>
    __device__ __forceinline__ static T of(T x, T y) { return x < y ? x : y; }
    template <typename T>
    __device__ __forceinline__ static T none() { return __is_same(T, float) ? (T)INF : __is_same(T, int) ? (T)0x7FFFFFFF : (T)~0ull; }
};
// over the lanes (ROW: the lanes of a row of 16) up to and with this one. Largest and
// smallest floats in one instruction a step: a lane that gets nothing keeps its value.
// (A lane move may read a register two wait states after it is written.)
#define MOE_SCAN(OP, CTRL, ROWS) asm("s_nop 1\n\t" OP " %0, %0, %0 " CTRL " row_mask:" ROWS " bank_mask:0xf" : "+v"(v))
template <typename F, bool ROW = false, typename T>
__device__ __forceinline__ T wave_scan(T v) {
    if constexpr (__is_same(T, float) && __is_same(F, Most)) {
        MOE_SCAN("v_max_f32_dpp", "row_shr:1", "0xf");
        MOE_SCAN("v_max_f32_dpp", "row_shr:2", "0xf");
        MOE_SCAN("v_max_f32_dpp", "row_shr:4", "0xf");
        MOE_SCAN("v_max_f32_dpp", "row_shr:8", "0xf");
        if (!ROW) MOE_SCAN("v_max_f32_dpp", "row_bcast:15", "0xa");
        if (!ROW) MOE_SCAN("v_max_f32_dpp", "row_bcast:31", "0xc");
        return v;
    }
    if constexpr (__is_same(T, float) && __is_same(F, Least)) {
        MOE_SCAN("v_min_f32_dpp", "row_shr:1", "0xf");
        MOE_SCAN("v_min_f32_dpp", "row_shr:2", "0xf");
        MOE_SCAN("v_min_f32_dpp", "row_shr:4", "0xf");
        MOE_SCAN("v_min_f32_dpp", "row_shr:8", "0xf");
        if (!ROW) MOE_SCAN("v_min_f32_dpp", "row_bcast:15", "0xa");
        if (!ROW) MOE_SCAN("v_min_f32_dpp", "row_bcast:31", "0xc");
        return v;
    }
    const T none = F::template none<T>();
    v = F::of(moved<0x111, 0xF, F::ZERO>(v, none), v);           // from 1, 2, 4, 8 lanes below in the row of 16
    v = F::of(moved<0x112, 0xF, F::ZERO>(v, none), v);
    v = F::of(moved<0x114, 0xF, F::ZERO>(v, none), v);
    v = F::of(moved<0x118, 0xF, F::ZERO>(v, none), v);
    if (ROW) return v;
    v = F::of(moved<0x142, 0xA, F::ZERO>(v, none), v);           // rows 0 and 2 into 1 and 3
    v = F::of(moved<0x143, 0xC, F::ZERO>(v, none), v);           // the lower half's into the upper
    return v;
}
#undef MOE_SCAN
template <typename T>
__device__ __forceinline__ T of_lane(T v, int lane) {
    if constexpr (sizeof(T) == 4) return __builtin_bit_cast(T, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
    else {
        const int2 a = __builtin_bit_cast(int2, v);
        return __builtin_bit_cast(T, make_int2(__builtin_amdgcn_readlane(a.x, lane), __builtin_amdgcn_readlane(a.y, lane)));
    }
}
template <typename F, typename T>
__device__ __forceinline__ T wave_all(T v) { return of_lane(wave_scan<F>(v), 63); }

// ---- over a workgroup of NT threads. A value a wave goes through `s`, which no
// call may use that is less than one barrier away.
// `s` holds a value for each wave: those of all
template <int NT, typename F, typename T>
__device__ __forceinline__ T of_waves(const T* s) {
    if constexpr (NT / 64 <= 4) {
        T v = s[0];
#pragma unroll
        for (int i = 1; i < NT / 64; ++i) v = F::of(v, s[i]);
        return v;
    }
    const int l = lane_id() & 15;
    return of_lane(wave_scan<F, true>(l < NT / 64 ? s[l] : F::template none<T>()), 15);
}
template <int NT, typename F, typename T>
__device__ __forceinline__ T block_all(T v, void* s) {
    v = wave_scan<F>(v);
    if (lane_id() == 63) ((T*)s)[threadIdx.x / 64] = v;
    __syncthreads();
    return of_waves<NT, F>((const T*)s);
}
// sum over the threads up to and with this one; that of all
template <int NT, typename T>
__device__ __forceinline__ T block_sums(T v, T& all, void* s) {
    v = wave_scan<Plus>(v);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    if (lane_id() == 63) ((T*)s)[wave] = v;
    __syncthreads();
    if constexpr (NT / 64 <= 4) {
        T before = 0;
        all = 0;
#pragma unroll
        for (int i = 0; i < NT / 64; ++i) {
            const T w = ((const T*)s)[i];
            if (i < wave) before += w;
            all += w;
        }
        return before + v;
    }
    const int l = lane_id() & 15;
    const T w = wave_scan<Plus, true>(l < NT / 64 ? ((const T*)s)[l] : (T)0);
    all = of_lane(w, 15);
    return wave ? of_lane(w, wave - 1) + v : v;
}

// equal parts of [low, top], the largest logits first (part: monotone in x)
template <int N>
struct Parts {
    float top, scale;
    __device__ __forceinline__ Parts(float t, float low) : top(t), scale(t > low ? (float)N / (t - low) : 0.f) {}
    __device__ __forceinline__ int of(float x) const { return (int)fminf((top - x) * scale, (float)(N - 1)); }
};
// The first part up to and with which the counts reach `want` (-1: they never do), and how many lie before it.
// A barrier before the call; s: two places for block_sums, at: two for the result.
template <int NT, int N>
__device__ __forceinline__ int part_of_count(const uint32_t* cnt, uint32_t want, uint32_t& before, void* s, int* at) {
    constexpr int R = N / NT;
    uint32_t c[R], own = 0, all;
#pragma unroll
    for (int i = 0; i < R; ++i) own += c[i] = cnt[R * threadIdx.x + i];
    uint32_t start = block_sums<NT>(own, all, s) - own;
    if (all < want) return -1;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        if (start < want && want <= start + c[i]) {
            at[0] = R * threadIdx.x + i;
            at[1] = (int)start;
        }
        start += c[i];
    }
    __syncthreads();
    before = (uint32_t)at[1];
    return at[0];
}

// n <= LIST places in LDS, largest first; n rounded up to a power of two with zeros. Barriers before and behind.
__device__ __forceinline__ void sort_places(uint64_t* p, int n) {
    int size = 64;
    while (size < n) size <<= 1;
    for (int i = n + threadIdx.x; i < size; i += ST) p[i] = 0;
    for (int run = 2; run <= size; run <<= 1)
        for (int d = run >> 1; d > 0; d >>= 1) {
            __syncthreads();
            for (int t = threadIdx.x; t < size / 2; t += ST) {
                const int i = 2 * t - (t & (d - 1)), j = i + d;
                const uint64_t x = p[i], y = p[j];
                if ((x < y) == ((i & run) == 0)) {
                    p[i] = y;
                    p[j] = x;
                }
            }
        }
    __syncthreads();
}

// (fmaxf first makes its operands quiet, one instruction each)
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
    float r;
    asm("v_min3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}

// ------------------------------------------------------------------ a chunk
constexpr int CHUNK_BINS = 1024;
struct ChunkShared {
    double two[32];
    uint64_t mass[STEPS];
    uint32_t cnt[CHUNK_BINS];
    uint64_t s[7][16];
    int at[2];
    int part[16];
};

// NT threads with E logits each; `share`: how many candidates may be written
template <bool F32, int NT, int E>
__device__ __forceinline__ void sample_chunk(const SampleArgs& a, int r, int c, int share, Chunk* info, uint64_t* list, uint64_t* steps, ChunkShared& s) {
    constexpr int NV = E / 4, SW = NT / 64;
    static_assert(NT * E == CHUNK && NV <= 4, "chunk");
    const void* row = (const uint8_t*)a.logits + (size_t)r * a.stride * (F32 ? 4 : 2);
    const int V = a.V, c0 = c * CHUNK, t = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(t / 64);
    float x[NV][4];
    load_fours<F32>(row, c0 + 4 * t, 4 * NT, c0, CHUNK, V, x);
    const Request q(a, r);
    for (int i = t; i < CHUNK_BINS; i += NT) s.cnt[i] = 0;
    for (int i = t; i < STEPS; i += NT) s.mass[i] = 0;
    if (t < 32) s.two[t] = g_two[t];
    const bool filter = q.k || q.p_on || q.m_on;
    float top = -INF, low = INF;
    bool nan = false;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        top = max3(top, max3(x[j][0], x[j][1], x[j][2]), x[j][3]);
        nan |= __builtin_isunordered(x[j][0], x[j][1]) || __builtin_isunordered(x[j][2], x[j][3]);
    }
    if (nan) top = INF;
    const float mine_top = top;
    if (filter) {
#pragma unroll
        for (int j = 0; j < NV; ++j) low = min3(low, min3(x[j][0], x[j][1], x[j][2]), x[j][3]);
        if (__ballot(low == -INF)) {
            low = INF;
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    if (x[j][v] > -INF) low = fminf(low, x[j][v]);
        }
    }
    {
        const float wt = wave_scan<Most>(top), wl = wave_scan<Least>(low);
        if (lane_id() == 63) {
            ((float*)s.s[0])[wave] = wt;
            ((float*)s.s[1])[wave] = wl;
        }
        __syncthreads();
        top = of_waves<NT, Most>((const float*)s.s[0]);
        low = of_waves<NT, Least>((const float*)s.s[1]);
    }
    Chunk out{0.0, top, low, -INF, 0};
    if (q.bad || !(top < INF) || top == -INF) {
        if (t == 0) *info = out;
        return;
    }
    if (q.k == 1) {                                              // the first token of the order
        uint64_t best = 0;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v) best = Most::of(best, place_of(x[j][v], c0 + (j * NT + t) * 4 + v));
        best = block_all<NT, Most>(best, s.s[2]);
        if (t == 0) {
            list[0] = best;
            out.n = 1;
            *info = out;
        }
        return;
    }
    // the chunk's weight, where the row's is needed (with top_k its candidates have it; min_p alone: likewise)
    if (q.k == 0 && (q.p_on || !q.m_on)) {
        // (top_p: by steps below the largest logit's too, for a border among many tokens)
        const int first = q.step(top);
        double sum = 0.0;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (__ballot(x[j][0] > -INF || x[j][1] > -INF || x[j][2] > -INF || x[j][3] > -INF)) {
                double w[4];
#pragma unroll
                for (int v = 0; v < 4; ++v) sum += w[v] = weight_of(x[j][v], top, q.scale, s.two);
                if (q.p_on && steps) {
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        const int i = first - q.step(x[j][v]);
                        if (i < STEPS) atomicAdd((unsigned long long*)&s.mass[i], (unsigned long long)mass_of(w[v]));
                    }
                }
            }
        out.sum = block_all<NT, Plus>(sum, s.s[2]);
        if (q.p_on && steps)
            for (int i = t; i < STEPS; i += NT) steps[i] = s.mass[i];
    }
    if (!filter) {
        if (t == 0) *info = out;
        return;
    }
    float floor = fmaxf(q.floor(top, out.sum, V), low);
    // top_k: k threads' largest logits are k tokens, so what lies below the k-th
    // largest of these is out (about as much as below the k-th token, for a
    // sixteenth of the additions that all tokens would take)
    if (q.k && q.k <= NT / 2) {
        const Parts<CHUNK_BINS> part(top, floor);
        const int b = part.of(mine_top);
        const bool one = mine_top >= floor;
        if (one) atomicAdd(&s.cnt[b], 1u);
        __syncthreads();
        uint32_t before;
        const int last = part_of_count<NT, CHUNK_BINS>(s.cnt, (uint32_t)q.k, before, s.s[4], s.at);
        if (one) s.cnt[b] = 0;                                   // (counted again below; every thread has read)
        if (last >= 0 && last < CHUNK_BINS - 1) {                // (the last part has all that lies lower, or all of a range too small for a scale)
            const float d = (float)(last + 1) / part.scale;
            floor = fmaxf(floor, top - d - (fabsf(top) + d) * 1e-6f);
        }
    }
    // Candidates: from `floor` on, bit 4 j + v. In the order of their ids: [vector][wave][lane][element].
    uint32_t mine = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v) mine |= (uint32_t)(x[j][v] >= floor) << (4 * j + v);
    int at[NV], total;
    auto places = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < NV; j += 2) {                        // (counts of two vectors in one scan: 256 at most)
            const uint32_t c = __popc(mine >> (4 * j) & 15) | (j + 1 < NV ? __popc(mine >> (4 * j + 4) & 15) << 16 : 0), e = wave_scan<Plus>(c);
            at[j] = (e - c) & 0xFFFF;
            if (lane_id() == 63) s.part[j * SW + wave] = e & 0xFFFF;
            if (j + 1 < NV) {
                at[j + 1 < NV ? j + 1 : 0] = (e - c) >> 16;
                if (lane_id() == 63) s.part[(j + 1 < NV ? j + 1 : 0) * SW + wave] = e >> 16;
            }
        }
        __syncthreads();
        static_assert(NV * SW == 16, "a lane each");
        const int end = wave_scan<Plus, true>(s.part[lane_id() & 15]);
        total = of_lane(end, 15);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int i = j * SW + wave;
            at[j] += i ? of_lane(end, i - 1) : 0;
        }
    };
    places();
    // More than the share, or than a few times k: those of the parts up to the k-th
    // (what is left out then is out), or of as many parts as fit the share.
    if (total > share || worth_parts(total, q.k)) {
        const Parts<CHUNK_BINS> part(top, floor);
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v)
                if (mine >> (4 * j + v) & 1) atomicAdd(&s.cnt[part.of(x[j][v])], 1u);
        __syncthreads();
        uint32_t before;
        const int want = q.k ? min(q.k, share) : share;
        int last = part_of_count<NT, CHUNK_BINS>(s.cnt, (uint32_t)want, before, s.s[6], s.at);
        if (last >= 0) {
            const bool fits = (int)(before + s.cnt[last]) <= share;
            if (!fits) --last;
            float cut = -INF;
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    if ((mine >> (4 * j + v) & 1) && part.of(x[j][v]) > last) {
                        cut = fmaxf(cut, x[j][v]);
                        mine &= ~(1u << (4 * j + v));
                    }
            if (!fits || !q.k || q.k > share) out.cut = block_all<NT, Most>(cut, s.s[5]);
            places();
        }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        int to = at[j];
#pragma unroll
        for (int v = 0; v < 4; ++v)
            if (mine >> (4 * j + v) & 1) list[to++] = place_of(x[j][v], c0 + (j * NT + t) * 4 + v);
    }
    out.n = total;
    if (t == 0) *info = out;
}

// ------------------------------------------------------------------ a row
struct RowShared {
    double two[32];
    uint64_t list[LIST];      // candidates by id
    uint64_t sorted[LIST];    // a part's tokens; the groups' sums of a draw
    uint32_t cnt[BINS];
    uint64_t mass[BINS];
    double share[MAX_CHUNKS], above[MAX_CHUNKS];                 // a chunk's weights' unit in the row's; its kept weight in whole steps
    uint64_t kept[MAX_CHUNKS];                                   // ... in the border's step, as a mass
    int shift[MAX_CHUNKS];
    uint64_t s[16][16];
    double got[2];
    uint64_t before[2];
    int at[2], hit[1], part[16];
    int n;
};

// the least `first` of the workgroup's threads, if there is none (0x7FFFFFFF) the largest `last`
__device__ __forceinline__ int choose(int first, int last, RowShared& s) {
    first = wave_all<Least>(first);
    last = wave_all<Most>(last);
    const int wave = threadIdx.x / 64;
    if (lane_id() == 0) {
        ((int*)s.s[8])[wave] = first;
        ((int*)s.s[9])[wave] = last;
    }
    __syncthreads();
    first = of_waves<ST, Least>((const int*)s.s[8]);
    last = of_waves<ST, Most>((const int*)s.s[9]);
    return first != 0x7FFFFFFF ? first : last;
}

// The lowest id in [lo, hi) (lo a multiple of four) up to and with which the
// weights exceed `aim` (past their sum: the last id with a weight), -1 if there
// is no weight. aim(sum) gives it. The id is left in s.hit[0], the sum in
// s.got[1] and the id's weight in s.got[0].
template <bool F32, typename W, typename A>
__device__ __forceinline__ void draw(const void* row, int lo, int hi, W weight, A aim, RowShared& s) {
    double* sums = (double*)s.sorted;                            // of 256 ids each, LIST of them at most
    const int t = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(t / 64);
    const int groups = (hi - lo + 255) / 256;
    __syncthreads();
    constexpr int D = 8;                                         // loads in flight
    for (int g0 = wave; g0 < groups; g0 += D * (ST / 64)) {
        float x[D][4];
        const int base = lo + g0 * 256;
        load_fours<F32>(row, base + 4 * lane, 256 * (ST / 64), base, 256 * (ST / 64) * (D - 1) + 256, hi, x);
#pragma unroll
        for (int d = 0; d < D; ++d) {
            const int g = g0 + d * (ST / 64), id = lo + g * 256 + lane * 4;
            if (g >= groups) break;
            double w = 0.0;
#pragma unroll
            for (int v = 0; v < 4; ++v) w += weight(x[d][v], id + v);
            w = wave_scan<Plus>(w);
            if (lane == 63) sums[g] = w;
        }
    }
    if (t == 0) s.hit[0] = -1;
    __syncthreads();
    // a run of groups for each thread
    const int run = (groups + ST - 1) / ST, g0 = min(t * run, groups), g1 = min(g0 + run, groups);
    double own = 0.0, total;
    for (int g = g0; g < g1; ++g) own += sums[g];
    const double end = block_sums<ST>(own, total, s.s[0]);
    const double want = aim(total);
    // the group: the first one whose end exceeds the aim, else the last one with a weight
    int first = 0x7FFFFFFF, last = -1;
    {
        double e = end - own;
        for (int g = g0; g < g1; ++g) {
            e += sums[g];
            if (sums[g] > 0.0) {
                last = g;
                if (e > want) first = min(first, g);
            }
        }
    }
    const int g = choose(first, last, s);
    if (g >= g0 && g < g1) {
        double e = end - own;
        for (int i = g0; i < g; ++i) e += sums[i];
        s.got[0] = e;
    }
    if (t == 0) s.got[1] = total;
    __syncthreads();
    if (g < 0) return;                                           // (s.hit[0] is -1)
    if (wave == 0) {
        const double start = s.got[0];
        float x[1][4];
        const int id = lo + g * 256 + lane * 4;
        load_fours<F32>(row, id, 0, lo + g * 256, 256, hi, x);
        double w[4], sum = 0.0;
#pragma unroll
        for (int v = 0; v < 4; ++v) sum += w[v] = weight(x[0][v], id + v);
        double e = start + (wave_scan<Plus>(sum) - sum);
        int at = -1, any = -1;
        double wa = 0.0, wy = 0.0;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            e += w[v];
            if (w[v] > 0.0) {
                any = id + v;
                wy = w[v];
                if (e > want && at < 0) {
                    at = id + v;
                    wa = w[v];
                }
            }
        }
        const uint64_t hit = __ballot(at >= 0), some = __ballot(any >= 0);
        const int from = hit ? __ffsll((long long)hit) - 1 : 63 - __clzll((long long)some);
        if (lane == from) {
            s.hit[0] = hit ? at : any;
            s.got[0] = hit ? wa : wy;
        }
    }
    __syncthreads();
}

// A lane's chunks of a row: lane, 64 + lane, ...
template <typename F>
__device__ __forceinline__ void each_chunk(int chunks, F f) {
    for (int c0 = 0; c0 < chunks; c0 += 64) f(c0 + lane_id(), c0 + lane_id() < chunks);
}

// The draw from the kept tokens, those from place `least` on, whose weight in chunk
// c is kept(c, in): the chunk that the aim falls into (past the sum: the last with
// a weight), read again.
template <bool F32, typename K, typename W>
__device__ __forceinline__ void draw_by_chunks(const SampleArgs& a, int r, const void* row, int chunks, K kept, W weight, double total, uint64_t least,
                                               RowShared& s) {
    const int V = a.V, t = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(t / 64);
    const double u = a.u[r];
    const double aim = u * total;
    double sum = 0.0, before = 0.0;
    int at = -1;
    each_chunk(chunks, [&](int c, bool in) __attribute__((always_inline)) {
        const double w = kept(c, in), end = sum + wave_scan<Plus>(w);
        const uint64_t some = __ballot(w > 0.0), hit = some & __ballot(end > aim);
        if (at < 0 || !(sum > aim)) {
            const int l = hit ? __ffsll((long long)hit) - 1 : some ? 63 - __clzll((long long)some) : -1;
            if (l >= 0) {
                at = c - lane + l;
                before = l ? of_lane(end, l - 1) : sum;
            }
        }
        sum = of_lane(end, 63);
    });
    constexpr int NV = CHUNK / (4 * ST);
    const int id0 = max(at, 0) * CHUNK;                          // (there is a weight: the largest logit's is 1)
    float x[NV][4];
    load_fours<F32>(row, id0 + 4 * t, 4 * ST, id0, CHUNK, V, x);
    // sums up to each lane's four, of each [vector][wave]
    double w[NV][4], ends[NV];
#pragma unroll
    for (int g = 0; g < NV; ++g) {
        double own = 0.0;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            w[g][v] = 0.0;
            if (place_of(x[g][v], id0 + 4 * (g * ST + t) + v) < least) x[g][v] = -INF;
        }
        if (__ballot(x[g][0] > -INF || x[g][1] > -INF || x[g][2] > -INF || x[g][3] > -INF)) {
#pragma unroll
            for (int v = 0; v < 4; ++v) own += w[g][v] = weight(x[g][v]);
        }
        ends[g] = wave_scan<Plus>(own);
        if (lane == 63) ((double*)s.s[4])[g * (ST / 64) + wave] = ends[g];
        ends[g] -= own;
    }
    __syncthreads();
    static_assert(NV * (ST / 64) == 16, "a lane each");
    const double part = ((const double*)s.s[4])[lane & 15], upto = before + wave_scan<Plus, true>(part);
    int first = 0x7FFFFFFF, last = -1;
    double pf = 0.0, pl = 0.0;
#pragma unroll
    for (int g = 0; g < NV; ++g) {
        const int i = g * (ST / 64) + wave;
        double y = (i ? of_lane(upto, i - 1) : before) + ends[g];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int id = 4 * (g * ST + t) + v;
            y += w[g][v];
            if (w[g][v] > 0.0) {
                last = id;
                pl = w[g][v];
                if (y > aim && id < first) {
                    first = id;
                    pf = w[g][v];
                }
            }
        }
    }
    const int chosen = choose(first, last, s);
    if (chosen == first || (chosen == last && first == 0x7FFFFFFF)) {            // (the token's thread)
        a.ids[r] = id0 + chosen;
        if (a.p) a.p[r] = (float)((chosen == first ? pf : pl) / total);
    }
}

// The border of the tokens that each(f) calls f(logit, id) for, by counts and masses
// of equal parts of [from, top], which fill(parts) adds up. share_of: the weight that
// top_p is a share of (0: that of these tokens, or of those that top_k leaves).
// False if the border may lie behind left_out. ALL: there may be more tokens in a
// part than can be sorted; nth(key, n) then finds the n-th id (the last, of fewer)
// with a logit's key. A barrier before; s.cnt and s.mass are zero.
template <bool ALL, typename M, typename E, typename F, typename N>
__device__ __forceinline__ bool find_border(const Request& q, float top, float from, double share_of, float left_out, M mass, E each, F fill, N nth,
                                            uint64_t& border, RowShared& s) {
    const int t = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(t / 64);
    const Parts<BINS> parts(top, from);
    border = 0;
    // counts and masses of the parts
    const bool both = q.p_on;
    fill(parts);
    __syncthreads();
    constexpr int R = BINS / ST;
    uint64_t own = 0, ends = 0, whole = 0;                   // masses of this thread's parts, up to and with them, of all
    if (both) {
#pragma unroll
        for (int i = 0; i < R; ++i) own += s.mass[R * t + i];
        ends = block_sums<ST>(own, whole, s.s[5]);
        if (share_of > 0.0) whole = (uint64_t)__builtin_ceil(share_of * ONE);
    }
    bool found = q.k || both || !(left_out > -INF);
    for (int stage = 0; stage < 2 && found; ++stage) {       // top_k, then top_p
        if (stage == 0 ? !q.k : !both) continue;
        // The part, and what lies before it: tokens; masses.
        int b = -1;
        uint64_t want;
        if (stage == 0) {
            uint32_t before;
            b = part_of_count<ST, BINS>(s.cnt, (uint32_t)q.k, before, s.s[6], s.at);
            want = q.k - before;
            if (b >= 0 && t == b / R) {
                uint64_t x = ends - own;
                for (int i = R * t; i < b; ++i) x += s.mass[i];
                s.before[0] = x;
            }
        } else {
            const double part = __builtin_ceil(q.top_p * (double)whole);
            want = part < 1.0 ? 1 : (uint64_t)part;
            __syncthreads();
            if (t == 0) s.at[0] = -1;
            __syncthreads();
            if (ends - own < want && want <= ends) {
                uint64_t start = ends - own;
                int i = R * t;
                while (start + s.mass[i] < want) start += s.mass[i++];
                s.at[0] = i;
                s.before[1] = start;
            }
            __syncthreads();
            b = s.at[0];
            if (b >= 0) want -= s.before[1];
        }
        if (b < 0) {                                         // never reached: all of them, or candidates left out
            found = !(left_out > -INF);
            continue;
        }
        // In that part: the last token that lies before `want` tokens (the last
        // one whose masses before it stay below `want`; the first one always),
        // and the mass up to and with it.
        uint64_t place, kept;
        if (t == 0) s.n = 0;
        __syncthreads();
        each([&](float x, int id) __attribute__((always_inline)) {
            if (parts.of(x) == b) {
                const int at = atomicAdd(&s.n, 1);
                if (at < LIST) s.sorted[at] = place_of(x, id);
            }
        });
        __syncthreads();
        const int m = s.n;
        if (m <= 64) {                                           // one wave: each token against all
            if (wave == 0) {
                const uint64_t mine = lane < m ? s.sorted[lane] : 0;
                const uint64_t w = lane < m ? mass(place_logit(mine)) : 0;
                uint64_t before = 0;
                for (int i = 0; i < m; ++i) {
                    const uint64_t wo = stage ? of_lane(w, i) : 1;
                    before += of_lane(mine, i) > mine ? wo : 0;
                }
                const bool in = lane < m && (before < want || before == 0);      // (the first, and others behind masses of zero)
                kept = wave_all<Plus>(in ? w : 0);
                place = wave_all<Least>(in ? mine : ~0ull);
                if (lane == 0) {
                    s.s[1][0] = kept;
                    s.s[1][1] = place;
                }
            }
            __syncthreads();
            kept = s.s[1][0];
            place = s.s[1][1];
        } else if (m <= LIST) {
            sort_places(s.sorted, m);
            uint64_t w[RUN], sum = 0, all_of;
#pragma unroll
            for (int i = 0; i < RUN; ++i) {
                w[i] = RUN * t + i < m ? mass(place_logit(s.sorted[RUN * t + i])) : 0;
                sum += w[i];
            }
            uint64_t before = block_sums<ST>(sum, all_of, s.s[1]) - sum, in = 0;
            int keep = 0;
#pragma unroll
            for (int i = 0; i < RUN; ++i) {
                const int at = RUN * t + i;
                if (at < m && ((stage ? before : (uint64_t)at) < want || at == 0)) {
                    keep = at + 1;
                    in += w[i];
                }
                before += w[i];
            }
            keep = block_all<ST, Most>(keep, s.s[2]);
            kept = block_all<ST, Plus>(in, s.s[3]);
            place = s.sorted[keep - 1];
        } else if constexpr (ALL) {
            // more than can be sorted (the row's logits, then): halve the range of keys until one is left
            uint32_t lo = ~0u, hi = 0;
            each([&](float x, int) __attribute__((always_inline)) {
                if (parts.of(x) == b) {
                    lo = min(lo, logit_key(x));
                    hi = max(hi, logit_key(x));
                }
            });
            lo = block_all<ST, Least>(lo, s.s[1]);
            hi = block_all<ST, Most>(hi, s.s[2]);
            // the smallest key with less than `want` above it; last of all what lies above that, and its mass
            uint64_t above, above_mass;
            if (want == 0) want = 1;
            for (bool last = false;;) {
                last = lo >= hi;
                const uint32_t mid = last ? lo : lo + (hi - lo) / 2;
                uint64_t n_above = 0, m_above = 0;
                each([&](float x, int) __attribute__((always_inline)) {
                    if (parts.of(x) == b && logit_key(x) > mid) {
                        ++n_above;
                        m_above += mass(x);
                    }
                });
                __syncthreads();
                above = block_all<ST, Plus>(n_above, s.s[3]);
                above_mass = block_all<ST, Plus>(m_above, s.s[4]);
                if (last) break;
                if ((stage ? above_mass : above) < want) hi = mid;
                else lo = mid + 1;
            }
            // of the tokens with that key the first by id
            const uint32_t key = lo;
            const uint64_t each_one = mass(key_logit(key)), left = want - (stage ? above_mass : above);
            const double ties = !stage ? (double)left : each_one ? (double)((left + each_one - 1) / each_one) : (double)MOE_SAMPLE_MAX_COLS;
            nth(key, ties);
            kept = above_mass + (uint64_t)fmin(ties, s.got[1]) * each_one;
            place = (uint64_t)key << 32 | (uint32_t)~s.hit[0];
        } else {                                             // (LIST candidates are sorted)
            place = kept = 0;
        }
        border = Most::of(border, place);
        found = place_logit(place) > left_out;
        if (stage == 0) whole = s.before[0] + kept;
    }
    return found;
}

// Rows whose border may lie behind the candidates.
template <bool F32>
__device__ __forceinline__ void sample_many_row(const SampleArgs& a, int r, int chunks, const Chunk* info, const uint64_t* steps, float top, float low, double all,
                                                RowShared& s) {
    const void* row = (const uint8_t*)a.logits + (size_t)r * a.stride * (F32 ? 4 : 2);
    const int V = a.V, t = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(t / 64);
    const Request q(a, r);
    const double u = a.u[r];
    const double zmax = top;
    auto weight = [&](float x) __attribute__((always_inline)) { return weight_of(x, zmax, q.scale, s.two); };
    auto mass = [&](float x) __attribute__((always_inline)) { return mass_of(weight(x)); };
    uint64_t border = 0;
    __syncthreads();
    // ---- top_p alone, with many tokens: the chunks' weights by steps say in which
    // step the border lies; that step's tokens, taken from the row, and 2048 equal
    // parts of them, where. min_p's border lies in a step as well: the kept tokens are
    // those of the steps above the first of the two steps, and some of its own. False
    // where the step's tokens are too many.
    auto by_steps = [&](uint64_t& border) __attribute__((always_inline)) {
        const int first = q.step(top);
        each_chunk(chunks, [&](int c, bool in) __attribute__((always_inline)) {
            if (wave || !in) return;
            const Chunk k = info[c];
            s.share[c] = k.sum > 0.0 ? exp_neg((double)k.top - zmax, q.scale, s.two) * (1.0 / ONE) : 0.0;
            s.shift[c] = k.sum > 0.0 ? min(first - q.step(k.top), STEPS) : STEPS;
            s.kept[c] = 0;
        });
        for (int i = t; i < BINS; i += ST) s.mass[i] = 0;
        if (t == 0) s.n = 0, s.at[0] = -1;
        __syncthreads();
        // the row's steps (from its largest logit's on), up to the one that reaches `want`
        // (a fourth of the chunks a thread, eight loads together)
        // (more than nothing, so that with top_p of 0 the border is the first token too: its weight is 1)
        const double want = fmax(q.top_p * all, 1.0 / ONE);
        double own = 0.0, total;
        double* parts_of = (double*)s.sorted;
        for (int c0 = t / STEPS; c0 < chunks; c0 += 32) {
            uint64_t w[8];
            const int i = t % STEPS;
#pragma unroll
            for (int d = 0; d < 8; ++d) {
                const int c = min(c0 + 4 * d, chunks - 1);
                w[d] = steps[(size_t)c * STEPS + max(i - s.shift[c], 0)];
            }
#pragma unroll
            for (int d = 0; d < 8; ++d) {
                const int c = min(c0 + 4 * d, chunks - 1);
                if (c0 + 4 * d < chunks && i >= s.shift[c]) own += s.share[c] * (double)w[d];
            }
        }
        static_assert(ST == 4 * STEPS, "a fourth of the chunks each");
        parts_of[t] = own;
        __syncthreads();
        own = t < STEPS ? (parts_of[t] + parts_of[STEPS + t]) + (parts_of[2 * STEPS + t] + parts_of[3 * STEPS + t]) : 0.0;
        const double end = block_sums<ST>(own, total, s.s[10]), start = end - own;
        if (own > 0.0 && start < want && want <= end) {          // (roundings could let two threads do it: the first one)
            atomicMax(&s.at[0], STEPS - t);
        }
        __syncthreads();
        const int bp = STEPS - s.at[0];                          // (none: past the last one)
        int b = bp;
        if (q.m_on) {
            // logits on both sides of min_p's border, by more than their own roundings; in one step, or not certain
            const float below = q.least(top, q.min_p), above = below + 2.f * (top - below + fabsf(top) + q.temperature) * 1e-5f;
            const int bm = first - q.step(fminf(above, top));
            if (bm < first - q.step(below)) return false;
            b = min(b, bm);
        }
        if (b >= STEPS) return false;
        if (t == b) s.got[0] = start;
        const int in_step = first - b;
        if (in_step <= -1000000000 || in_step >= 1000000000) return false;       // (step()'s bounds)
        // each chunk's weight above that step: four of a lane's steps, of four chunks together
        for (int c0 = wave; c0 < chunks; c0 += 4 * (ST / 64)) {
            typedef uint64_t u64x2 __attribute__((ext_vector_type(2)));
            u64x2 w[4][2];
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                const u64x2* at = (const u64x2*)(steps + (size_t)min(c0 + d * (ST / 64), chunks - 1) * STEPS + 4 * lane);
                w[d][0] = at[0];
                w[d][1] = at[1];
            }
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                const int c = c0 + d * (ST / 64);
                if (c >= chunks) break;
                const int n = b - s.shift[c] - 4 * lane;
                uint64_t sum = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) sum += i < n ? w[d][i / 2][i % 2] : 0;
                sum = wave_all<Plus>(sum);
                if (lane == 0) s.above[c] = s.share[c] * (double)sum;
            }
        }
        // the step's tokens
        uint64_t* tokens = s.list;                               // (and s.sorted behind it)
        const float slope = 8.f / q.temperature, in_this = (float)in_step;
        constexpr int D = 8;                                     // loads in flight; one addition for a wave's tokens of them
        float x[D][4], next[D][4];
        load_fours<F32>(row, 4 * t, ST * 4, 0, D * ST * 4, V, next);
        for (int base = 0; base < V; base += D * ST * 4) {
#pragma unroll
            for (int d = 0; d < D; ++d)
#pragma unroll
                for (int v = 0; v < 4; ++v) x[d][v] = next[d][v];
            const int ahead = base + D * ST * 4;
            if (ahead < V) load_fours<F32>(row, ahead + 4 * t, ST * 4, ahead, D * ST * 4, V, next);
            uint32_t mine = 0;
#pragma unroll
            for (int d = 0; d < D; ++d)
#pragma unroll
                for (int v = 0; v < 4; ++v) mine |= (uint32_t)(floorf(x[d][v] * slope) == in_this) << (4 * d + v);   // (step(), within its bounds)
            const int count = __popc(mine), upto = wave_scan<Plus>(count), all_of = of_lane(upto, 63);
            if (all_of == 0) continue;
            int at = 0;
            if (lane == 0) at = atomicAdd(&s.n, all_of);
            at = of_lane(at, 0) + upto - count;
            // (their ids: a lane has few of its 32, and where it would have to branch for each of them with its logit, that took thrice the time)
            for (; mine; mine &= mine - 1, ++at) {
                const int i = __ffs((int)mine) - 1;
                if (at < 2 * LIST) tokens[at] = (uint32_t)(base + 4 * t + (i / 4) * ST * 4 + i % 4);
            }
        }
        __syncthreads();
        const int n = s.n;
        if (n > 2 * LIST) return false;
        {
            // with their logits, in the order of the tokens
            float y[2 * RUN];
#pragma unroll
            for (int d = 0; d < 2 * RUN; ++d) {
                const int i = t + d * ST;
                if (i < n) y[d] = F32 ? ((const float*)row)[tokens[i]] : bf16_to_f32(((const uint16_t*)row)[tokens[i]]);
            }
#pragma unroll
            for (int d = 0; d < 2 * RUN; ++d) {
                const int i = t + d * ST;
                if (i < n) tokens[i] = place_of(y[d], (int)tokens[i]);
            }
            __syncthreads();
        }
        auto sum_kept = [&](uint64_t border) __attribute__((always_inline)) {
            for (int i = t; i < n; i += ST) {
                const double w = weight(place_logit(tokens[i]));
                if (tokens[i] >= border && w >= q.min_p)
                    atomicAdd((unsigned long long*)&s.kept[place_id(tokens[i]) / CHUNK], (unsigned long long)mass_of(w));
            }
            __syncthreads();
        };
        if (b < bp) {                                            // (min_p's alone)
            border = 0;
            sum_kept(border);
            return true;
        }
        // their range, in parts; the part that reaches what is left of `want`
        uint64_t hi = 0, lo = ~0ull;
        for (int i = t; i < n; i += ST) {
            hi = Most::of(hi, tokens[i]);
            lo = Least::of(lo, tokens[i]);
        }
        hi = block_all<ST, Most>(hi, s.s[11]);
        lo = block_all<ST, Least>(lo, s.s[12]);
        const Parts<BINS> parts(place_logit(hi), place_logit(lo));
        for (int i = t; i < n; i += ST) {
            const float x = place_logit(tokens[i]);
            atomicAdd((unsigned long long*)&s.mass[parts.of(x)], (unsigned long long)mass(x));
        }
        if (t == 0) s.n = 0, s.at[0] = -1;
        __syncthreads();
        const double left = __builtin_ceil((want - s.got[0]) * ONE);
        const uint64_t rest = left < 1.0 ? 1 : (uint64_t)left;
        constexpr int R = BINS / ST;
        uint64_t mine = 0, whole;
#pragma unroll
        for (int i = 0; i < R; ++i) mine += s.mass[R * t + i];
        const uint64_t ends = block_sums<ST>(mine, whole, s.s[13]);
        const uint64_t need = Least::of(rest, whole);            // (roundings; whole > 0: the step has a weight)
        if (ends - mine < need && need <= ends) {
            uint64_t upto = ends - mine;
            int i = R * t;
            while (upto + s.mass[i] < need) upto += s.mass[i++];
            s.at[0] = i;
            s.before[0] = upto;
        }
        __syncthreads();
        const int p = s.at[0];
        if (p < 0) return false;
        const uint64_t in_part = need - s.before[0];
        // that part's tokens in order, as many as a wave holds; more where logits are equal
        uint64_t* few = s.s[0];
        constexpr int FEW = 64;
        for (int i = t; i < n; i += ST)
            if (parts.of(place_logit(tokens[i])) == p) {
                const int at = atomicAdd(&s.n, 1);
                if (at < FEW) few[at] = tokens[i];
            }
        __syncthreads();
        const int m = s.n;
        if (m <= FEW) {
            const uint64_t e = lane < m ? few[lane] : 0;
            const uint64_t w = lane < m ? mass(place_logit(e)) : 0;
            uint64_t before = 0;
            for (int i = 0; i < m; ++i) before += of_lane(e, i) > e ? of_lane(w, i) : 0;
            border = wave_all<Least>(lane < m && (before < in_part || before == 0) ? e : ~0ull);
        } else {
            // equal logits (else: the row's): as many of the lowest ids as the mass takes
            hi = 0, lo = ~0ull;
            for (int i = t; i < n; i += ST) {
                const uint64_t e = tokens[i];
                if (parts.of(place_logit(e)) != p) continue;
                hi = Most::of(hi, e);
                lo = Least::of(lo, e);
            }
            hi = block_all<ST, Most>(hi, s.s[11]);
            lo = block_all<ST, Least>(lo, s.s[12]);
            if (hi >> 32 != lo >> 32) return false;
            const uint64_t each_one = mass(place_logit(hi));
            const int ties = each_one ? (int)Least::of((in_part + each_one - 1) / each_one, (uint64_t)m) : m;
            const int width = (V + BINS - 1) / BINS;             // ids of a bin: 512 at most
            for (int i = t; i < n; i += ST)
                if (tokens[i] >> 32 == hi >> 32) atomicAdd(&s.cnt[place_id(tokens[i]) / width], 1u);
            if (t == 0) s.n = 0;
            __syncthreads();
            uint32_t before;
            const int bin = part_of_count<ST, BINS>(s.cnt, (uint32_t)ties, before, s.s[15], s.at);
            uint64_t* same = s.mass;
            for (int i = t; i < n; i += ST)
                if (tokens[i] >> 32 == hi >> 32 && place_id(tokens[i]) / width == bin) same[atomicAdd(&s.n, 1)] = tokens[i];
            __syncthreads();
            const int k = s.n;
            if (t < k) {
                int rank = 0;
                for (int i = 0; i < k; ++i) rank += same[i] > same[t];
                if (rank == ties - (int)before - 1) s.before[1] = same[t];
            }
            __syncthreads();
            border = s.before[1];
        }
        sum_kept(border);
        return true;
    };

    if (q.k == 0 && q.p_on && steps && by_steps(border)) {
        auto kept = [&](int c, bool in) __attribute__((always_inline)) { return in ? s.above[c] + (double)s.kept[c] * (1.0 / ONE) : 0.0; };
        double total = 0.0;
        each_chunk(chunks, [&](int c, bool in) __attribute__((always_inline)) { total += wave_all<Plus>(kept(c, in)); });
        auto kept_weight = [&](float x) __attribute__((always_inline)) {
            const double w = weight(x);
            return w >= q.min_p ? w : 0.0;
        };
        return draw_by_chunks<F32>(a, r, row, chunks, kept, kept_weight, total, border, s);
    }

    // ---- the row's logits (but those of 2^-46 of the largest weight and less)
    __syncthreads();
    for (int i = t; i < BINS; i += ST) {
        s.cnt[i] = 0;
        s.mass[i] = 0;
    }
    __syncthreads();
    const float bottom = fmaxf(q.least(top, 1.0 / 70368744177664.0), low);
    auto each = [&](auto f) __attribute__((always_inline)) {
        constexpr int D = 4;                                     // loads in flight
        for (int i = t * 4; i < V; i += D * ST * 4) {
            float x[D][4];
            load_fours<F32>(row, i, ST * 4, i - 4 * t, D * ST * 4, V, x);
#pragma unroll
            for (int d = 0; d < D; ++d)
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    if (x[d][v] >= bottom) f(x[d][v], i + d * ST * 4 + v);
        }
    };
    border = 0;
    if (q.k || q.p_on)
        find_border<true>(q, top, bottom, 0.0, -INF, mass, each,
                          [&](const Parts<BINS>& parts) __attribute__((always_inline)) {
                              each([&](float x, int) __attribute__((always_inline)) {
                                  const int b = parts.of(x);
                                  if (q.k) atomicAdd(&s.cnt[b], 1u);
                                  if (q.p_on) atomicAdd((unsigned long long*)&s.mass[b], (unsigned long long)mass(x));
                              });
                          },
                          [&](uint32_t key, double ties) __attribute__((always_inline)) {
                              draw<F32>(row, 0, V, [&](float x, int) __attribute__((always_inline)) { return x > -INF && logit_key(x) == key ? 1.0 : 0.0; },
                                        [&](double sum) { return fmin(ties, sum) - 1.0; }, s);
                          },
                          border, s);
    draw<F32>(row, 0, V, [&](float x, int id) __attribute__((always_inline)) {
                  const double w = weight(x);
                  return x >= bottom && place_of(x, id) >= border && w >= q.min_p ? w : 0.0;
              }, [&](double sum) { return u * sum; }, s);
    if (t == 0) {
        a.ids[r] = s.hit[0];
        if (a.p) a.p[r] = (float)(s.got[0] / s.got[1]);
    }
}

// (parameters arrive in a lane's registers)
template <typename T>
__device__ __forceinline__ T uniform(T v) { return of_lane(v, 0); }
using KernelArgs = const __attribute__((address_space(4))) SampleArgs;
// A function of its own, so that its registers do not weigh on the others (the kernel
// with it inside spilled 77), and the program's end, so that it saves none of them
// (with a return it began with 8 us of stores). From `args`, the kernel's arguments.
template <bool F32>
__device__ __noinline__ __attribute__((noreturn)) void sample_many(const KernelArgs* args, int r, int chunks, const Chunk* info, const uint64_t* steps,
                                                                   float top, float low, double all) {
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    const SampleArgs a = *(const SampleArgs*)uniform(args);
    sample_many_row<F32>(a, uniform(r), uniform(chunks), uniform(info), uniform(steps), uniform(top), uniform(low), uniform(all), *(RowShared*)smem);
    __builtin_amdgcn_endpgm();
}

// `listed`: the row's one chunk has left its candidates in s.list
template <bool F32>
__device__ __forceinline__ void sample_finish(const SampleArgs& a, int r, int chunks, int share, const Chunk* info, const uint64_t* lists, const uint64_t* steps,
                                              bool listed, RowShared& s) {
    const void* row = (const uint8_t*)a.logits + (size_t)r * a.stride * (F32 ? 4 : 2);
    const int V = a.V, t = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(t / 64);
    // candidates, four of a chunk in a row for each thread (memory behind the last one is the lists' own)
    uint64_t e[RUN];
    int n4[RUN / 4];
#pragma unroll
    for (int g = 0; g < RUN / 4; ++g) {
        const int slot = 4 * (g * ST + t), c = min(slot / share, chunks - 1), i = slot - c * share;
        n4[g] = 0;
        if (slot < chunks * share) {
            n4[g] = info[c].n - i;
#pragma unroll
            for (int v = 0; v < 4; ++v) e[4 * g + v] = listed ? s.list[i + v] : lists[(size_t)c * share + i + v];
        }
    }
    // every wave puts the chunks together for itself
    float top = -INF, low = INF, cut = -INF;
    each_chunk(chunks, [&](int c, bool in) __attribute__((always_inline)) {
        if (!in) return;
        const Chunk k = info[c];
        top = fmaxf(top, k.top);
        low = fminf(low, k.low);
        cut = fmaxf(cut, k.cut);
    });
    const Request q(a, r);
    const double u = a.u[r];
    for (int i = t; i < BINS; i += ST) {
        s.cnt[i] = 0;
        s.mass[i] = 0;
    }
    if (t < 32) s.two[t] = g_two[t];
    __syncthreads();
    top = wave_all<Most>(top);
    low = wave_all<Least>(low);
    cut = wave_all<Most>(cut);
    auto give = [&](int id, double p) __attribute__((always_inline)) {
        if (t == 0) {
            a.ids[r] = id;
            if (a.p) a.p[r] = (float)p;
            if (id < 0 && a.err) atomicAdd(a.err, 1);
        }
    };
    if (q.bad || !(top < INF) || top == -INF) return give(-1, 0.0);
    const double zmax = top;
    auto weight = [&](float x) __attribute__((always_inline)) { return weight_of(x, zmax, q.scale, s.two); };
    auto mass = [&](float x) __attribute__((always_inline)) { return mass_of(weight(x)); };

    if (q.k == 1) {
        uint64_t best = 0;
#pragma unroll
        for (int i = 0; i < RUN; ++i)
            if (i % 4 < n4[i / 4]) best = Most::of(best, e[i]);
        return give(place_id(block_all<ST, Most>(best, s.s[4])), 1.0);
    }
    // the row's weight from the chunks', where they have it
    double all = 0.0;
    const bool pure = q.k == 0 && !q.p_on && !q.m_on;
    auto scaled = [&](int c, bool in) __attribute__((always_inline)) {
        if (!in || !(info[c].sum > 0.0)) return 0.0;
        return info[c].sum * exp_neg((double)info[c].top - zmax, q.scale, s.two);
    };
    if (q.k == 0 && (q.p_on || pure)) each_chunk(chunks, [&](int c, bool in) __attribute__((always_inline)) { all += wave_all<Plus>(scaled(c, in)); });
    if (pure) return draw_by_chunks<F32>(a, r, row, chunks, scaled, weight, all, 0, s);          // no filter

    // ---- few candidates
    const float least = q.floor(top, all, V), floor = fmaxf(least, low);
    float from = floor;                                          // (about) the least candidate
    bool in[RUN];
    int n;
    // those that f(i) names of the thread's, into s.list in the order of their ids (barriers before and behind)
    auto collect = [&](auto f) __attribute__((always_inline)) {
        int to[RUN / 4];
#pragma unroll
        for (int g = 0; g < RUN / 4; ++g) {
            int before = 0, count = 0;
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                in[4 * g + v] = f(4 * g + v);
                const uint64_t b = __ballot(in[4 * g + v]);
                before += __popcll(b & lanemask_lt());
                count += __popcll(b);
            }
            to[g] = before;
            if (lane == 0) s.part[g * (ST / 64) + wave] = count;
        }
        __syncthreads();
        static_assert(RUN / 4 * (ST / 64) == 16, "a lane each");
        const int end = wave_scan<Plus, true>(s.part[lane & 15]);
        n = of_lane(end, 15);
#pragma unroll
        for (int g = 0; g < RUN / 4; ++g) {
            const int i = g * (ST / 64) + wave;
            int at = to[g] + (i ? of_lane(end, i - 1) : 0);
#pragma unroll
            for (int v = 0; v < 4; ++v)
                if (in[4 * g + v]) s.list[at++] = e[4 * g + v];
        }
    };
    collect([&](int i) __attribute__((always_inline)) { return i % 4 < n4[i / 4] && place_logit(e[i]) >= floor; });
    // more than one wave can put in order: the parts up to the k-th first
    auto candidates = [&](auto f) __attribute__((always_inline)) {
#pragma unroll
        for (int v = 0; v < RUN; ++v)
            if (in[v]) f(place_logit(e[v]), place_id(e[v]));
    };
    if (q.k && n > 64 && n > q.k) {
        const Parts<BINS> parts(top, floor);
        candidates([&](float x, int) __attribute__((always_inline)) { atomicAdd(&s.cnt[parts.of(x)], 1u); });
        __syncthreads();
        uint32_t before;
        const int last = part_of_count<ST, BINS>(s.cnt, (uint32_t)q.k, before, s.s[10], s.at);
        collect([&](int v) __attribute__((always_inline)) { return in[v] && parts.of(place_logit(e[v])) <= last; });
        from = fmaxf(floor, top - (float)(last + 1) / parts.scale);
        for (int i = t; i < BINS; i += ST) s.cnt[i] = 0;
    }
    __syncthreads();
    if (n <= 64 && !(cut >= least)) {
        if (wave) return;
        // a candidate a lane: how many, and what weight, the others have that lie before it
        const uint64_t mine = lane < n ? s.list[lane] : 0;
        const double w = lane < n ? weight(place_logit(mine)) : 0.0;
        double before = 0.0;
        int rank = 0;
        for (int i = 0; i < n; ++i) {
            const bool first = of_lane(mine, i) > mine;
            rank += first;
            before += first ? of_lane(w, i) : 0.0;
        }
        bool keep = lane < n && (!q.k || rank < q.k);
        const double whole = q.k ? wave_all<Plus>(keep ? w : 0.0) : all;
        keep = keep && (!q.p_on || before < q.top_p * whole || rank == 0) && w >= q.min_p;
        const double end = wave_scan<Plus>(keep ? w : 0.0), total = of_lane(end, 63), aim = u * total;
        const uint64_t some = __ballot(keep && w > 0.0), hit = some & __ballot(end > aim);
        const int l = hit ? __ffsll((long long)hit) - 1 : 63 - __clzll((long long)some);
        return give(place_id(of_lane(mine, l)), of_lane(w, l) / total);
    }
    // ---- the border, among the candidates
    uint64_t border;                                             // the last kept place (before min_p)
    const float left_out = cut >= least ? cut : -INF;
    const bool sure = find_border<false>(q, top, from, q.k == 0 ? all : 0.0, left_out, mass, candidates,
                                         [&](const Parts<BINS>& parts) __attribute__((always_inline)) {
                                             uint64_t w[RUN];    // (all of a thread's before its branches)
                                             bool any = false;
#pragma unroll
                                             for (int v = 0; v < RUN; ++v) {
                                                 w[v] = 0;
                                                 any |= in[v];
                                             }
                                             if (q.p_on && __ballot(any)) {
#pragma unroll
                                                 for (int v = 0; v < RUN; ++v) w[v] = mass(in[v] ? place_logit(e[v]) : top);
                                             }
#pragma unroll
                                             for (int v = 0; v < RUN; ++v)
                                                 if (in[v]) {
                                                     const int b = parts.of(place_logit(e[v]));
                                                     if (q.k) atomicAdd(&s.cnt[b], 1u);
                                                     if (q.p_on) atomicAdd((unsigned long long*)&s.mass[b], (unsigned long long)w[v]);
                                                 }
                                         },
                                         [](uint32_t, double) {}, border, s);
    if (!sure) sample_many<F32>((KernelArgs*)__builtin_amdgcn_kernarg_segment_ptr(), r, chunks, info, steps, top, low, all);
    // the draw by id: a run of the list for each thread
    __syncthreads();
    const int run = (n + ST - 1) / ST, i0 = min(t * run, n), i1 = min(i0 + run, n);
    auto kept = [&](int i) __attribute__((always_inline)) {
        const uint64_t at = s.list[i];
        const double w = weight(place_logit(at));
        return at >= border && w >= q.min_p ? w : 0.0;
    };
    double sum = 0.0, total;
    for (int i = i0; i < i1; ++i) sum += kept(i);
    double x = block_sums<ST>(sum, total, s.s[7]) - sum;
    const double aim = u * total;
    int first = 0x7FFFFFFF, last = -1;
    if (sum > 0.0)
        for (int i = i0; i < i1; ++i) {
            const double w = kept(i);
            x += w;
            if (w > 0.0) {
                last = i;
                if (x > aim) first = min(first, i);
            }
        }
    const uint64_t chosen = s.list[choose(first, last, s)];
    give(place_id(chosen), weight(place_logit(chosen)) / total);
}

constexpr int CHUNK_THREADS = 256;
template <bool F32>
__global__ void __launch_bounds__(CHUNK_THREADS, 6) sample_chunk_kernel(SampleArgs a, int chunks, int share, Chunk* info, uint64_t* lists, uint64_t* steps) {
    __shared__ ChunkShared s;
    const long long n = (long long)a.B * chunks;
    for (long long i = blockIdx.x; i < n; i += gridDim.x) {
        sample_chunk<F32, CHUNK_THREADS, CHUNK / CHUNK_THREADS>(a, (int)(i / chunks), (int)(i % chunks), share, info + i, lists + i * share,
                                                               steps + i * STEPS, s);
        __syncthreads();
    }
}
template <bool F32>
__global__ void __launch_bounds__(ST) sample_finish_kernel(SampleArgs a, int chunks, int share, const Chunk* info, const uint64_t* lists,
                                                           const uint64_t* steps) {
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    const size_t i = (size_t)blockIdx.x * chunks;
    sample_finish<F32>(a, blockIdx.x, chunks, share, info + i, lists + i * share, steps + i * STEPS, false, *(RowShared*)smem);
}
// rows of one chunk
struct OneShared {
    RowShared row;
    ChunkShared chunk;
    Chunk info;
};
template <bool F32>
__global__ void __launch_bounds__(ST) sample_row_kernel(SampleArgs a) {
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    OneShared& s = *(OneShared*)smem;
    sample_chunk<F32, ST, CHUNK / ST>(a, blockIdx.x, 0, LIST, &s.info, s.row.list, nullptr, s.chunk);
    __syncthreads();
    sample_finish<F32>(a, blockIdx.x, 1, LIST, &s.info, nullptr, nullptr, true, s.row);
}

static int chunks_of(int V) { return (V + CHUNK - 1) / CHUNK; }
static int share_of(int chunks) { return LIST / chunks / 4 * 4; }
static size_t info_bytes(int B, int V) { return ((size_t)B * chunks_of(V) * sizeof(Chunk) + 255) / 256 * 256; }
size_t sample_workspace_bytes(int B, int V) {
    const int chunks = chunks_of(V);
    if (chunks == 1) return 0;
    return info_bytes(B, V) + (size_t)B * chunks * (share_of(chunks) + STEPS) * 8;
}

template <bool F32>
static hipError_t launch(const SampleArgs& a, void* ws, hipStream_t stream) {
    const int chunks = chunks_of(a.V), share = share_of(chunks);
    Chunk* info = (Chunk*)ws;
    uint64_t* lists = (uint64_t*)((uint8_t*)ws + info_bytes(a.B, a.V));
    uint64_t* steps = lists + (size_t)a.B * chunks * share;
    static_assert(sizeof(OneShared) <= 163840, "LDS");
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    static std::atomic<uint64_t> done[2];
    if (chunks == 1) {
        e = allow_lds((const void*)sample_row_kernel<F32>, sizeof(OneShared), dev, done[0]);
        if (e != hipSuccess) return e;
        return launch_kernel(K_SAMPLE, stream, sample_row_kernel<F32>, dim3((unsigned)a.B), dim3(ST), sizeof(OneShared), a);
    }
    e = allow_lds((const void*)sample_finish_kernel<F32>, sizeof(RowShared), dev, done[1]);
    if (e != hipSuccess) return e;
    const long long n = (long long)a.B * chunks;
    e = launch_kernel(K_SAMPLE, stream, sample_chunk_kernel<F32>, dim3((unsigned)(n < (1 << 20) ? n : 1 << 20)), dim3(CHUNK_THREADS), 0, a,
                      chunks, share, info, lists, steps);
    if (e != hipSuccess) return e;
    return launch_kernel(K_SAMPLE, stream, sample_finish_kernel<F32>, dim3((unsigned)a.B), dim3(ST), sizeof(RowShared), a, chunks, share,
                         (const Chunk*)info, (const uint64_t*)lists, (const uint64_t*)steps);
}
hipError_t launch_sample(const SampleArgs& a, bool f32, void* ws, hipStream_t stream) {
    return f32 ? launch<true>(a, ws, stream) : launch<false>(a, ws, stream);
}

}  // namespace moe
