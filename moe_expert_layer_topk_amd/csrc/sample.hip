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
// finish kernel: one workgroup a row. Candidates are sorted in LDS, borders come
// from prefix sums, and hold if they lie before every logit that was left out
// (nearly always, with a filter). No filter: the chunk that the draw falls into
// is read again. Else (a top_p that keeps thousands of tokens) the row is read
// again: counts and weights of 2048 equal parts of the logits' range, the
// tokens of the part that holds the border sorted, the kept weight by id.
//
// Weights are fp64, sums of them fp64 in a fixed order; the parts' weights are
// summed with atomics, and therefore as integers (multiples of 2^-42 of the
// largest weight).
#include "moe_common.h"
#include "moe_kernels.h"
#include "gemm_tile.h"

namespace moe {

constexpr int ST = 1024;                                         // threads of a finish workgroup
constexpr int CHUNK = 4096;                                      // logits of a chunk
constexpr int MAX_CHUNKS = MOE_SAMPLE_MAX_COLS / CHUNK;
constexpr int LIST = 4096;                                       // candidates of a row
constexpr int BINS = 2048;
constexpr double ONE = 4398046511104.0;                          // 2^42: the sum of 2^20 weights stays below 2^63
constexpr float INF = __builtin_inff();

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

// e^x for x <= 0: 2^n e^r with |r| <= ln 2 / 2 and Taylor's polynomial of e^r to
// r^11 (the rest is below 7e-15); 1 for 0, 0 below 2^-1022
__device__ __forceinline__ double exp_neg(double x) {
    const double n = __builtin_rint(x * 1.4426950408889634074);
    const double r = __builtin_fma(n, -0.693147180559945309417, x);
    double y = 1.0 / 39916800.0;
    y = __builtin_fma(y, r, 1.0 / 3628800.0);
    y = __builtin_fma(y, r, 1.0 / 362880.0);
    y = __builtin_fma(y, r, 1.0 / 40320.0);
    y = __builtin_fma(y, r, 1.0 / 5040.0);
    y = __builtin_fma(y, r, 1.0 / 720.0);
    y = __builtin_fma(y, r, 1.0 / 120.0);
    y = __builtin_fma(y, r, 1.0 / 24.0);
    y = __builtin_fma(y, r, 1.0 / 6.0);
    y = __builtin_fma(y, r, 0.5);
    y = __builtin_fma(y, r, 1.0);
    y = __builtin_fma(y, r, 1.0);
    const int e = n < -1022.0 ? 0 : (int)n + 1023;
    return e ? y * __longlong_as_double((long long)e << 52) : 0.0;
}

// a row's parameters
struct Request {
    double inv, top_p, min_p;  // 1 / temperature (0 for infinity)
    float temperature;
    int k;                     // 0: off
    bool bad, p_on, m_on;
    __device__ __forceinline__ Request(const SampleArgs& a, int r) {
        temperature = a.temperature ? a.temperature[r] : 1.f;
        const float u = a.u[r], tp = a.top_p ? a.top_p[r] : 1.f, mp = a.min_p ? a.min_p[r] : 0.f;
        bad = !(u >= 0.f && u <= 1.f) || !(temperature >= 0.f) || tp != tp || !(mp <= 1.f);
        inv = temperature > 0.f ? 1.0 / (double)temperature : 0.0;
        k = temperature == 0.f ? 1 : a.top_k ? max(a.top_k[r], 0) : 0;
        top_p = tp > 0.f ? tp : 0.f;
        min_p = mp > 0.f ? mp : 0.f;
        p_on = tp < 1.f && k != 1;
        m_on = mp > 0.f && k != 1;
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

// N consecutive logits from element i on, -inf past the row's end
template <bool F32, int N>
__device__ __forceinline__ void load_logits(const void* row, int i, int V, float (&x)[N]) {
    typedef uint32_t w4 __attribute__((ext_vector_type(N)));
    typedef uint32_t w2 __attribute__((ext_vector_type(N / 2)));
    typedef w4 place4 __attribute__((aligned(4)));
    typedef w2 place2 __attribute__((aligned(2)));
    if (i + N <= V) {
        if (F32) {
            const w4 v = *(const place4*)((const float*)row + i);
#pragma unroll
            for (int j = 0; j < N; ++j) x[j] = __uint_as_float(v[j]);
        } else {
            const w2 v = *(const place2*)((const uint16_t*)row + i);
#pragma unroll
            for (int j = 0; j < N; ++j) x[j] = __uint_as_float(j & 1 ? v[j / 2] & 0xFFFF0000u : v[j / 2] << 16);
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j)
            x[j] = i + j < V ? (F32 ? ((const float*)row)[i + j] : bf16_to_f32(((const uint16_t*)row)[i + j])) : -INF;
    }
}

// ---- over a wave by lane moves in the vector unit
template <int CTRL, int ROWS, typename T>
__device__ __forceinline__ T moved(T v, T none) {
    if constexpr (sizeof(T) == 4) {
        return __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, none), __builtin_bit_cast(int, v), CTRL, ROWS, 0xF, false));
    } else {
        const int2 a = __builtin_bit_cast(int2, v), b = __builtin_bit_cast(int2, none);
        return __builtin_bit_cast(T, make_int2(__builtin_amdgcn_update_dpp(b.x, a.x, CTRL, ROWS, 0xF, false),
                                               __builtin_amdgcn_update_dpp(b.y, a.y, CTRL, ROWS, 0xF, false)));
    }
}
struct Plus {
    template <typename T>
    __device__ __forceinline__ static T of(T x, T y) { return x + y; }
    template <typename T>
    __device__ __forceinline__ static T none() { return (T)0; }
};
struct Most {
    template <typename T>
    __device__ __forceinline__ static T of(T x, T y) { return x > y ? x : y; }
    template <typename T>
    __device__ __forceinline__ static T none() { return __is_same(T, float) ? (T)-INF : (T)(__is_same(T, int) ? -0x7FFFFFFF - 1 : 0); }
};
struct Least {
    template <typename T>
    __device__ __forceinline__ static T of(T x, T y) { return x < y ? x : y; }
    template <typename T>
    __device__ __forceinline__ static T none() { return __is_same(T, float) ? (T)INF : __is_same(T, int) ? (T)0x7FFFFFFF : (T)~0ull; }
};
// over the lanes up to and with this one
template <typename F, typename T>
__device__ __forceinline__ T wave_scan(T v) {
    const T none = F::template none<T>();
    v = F::of(moved<0x111, 0xF>(v, none), v);                    // from 1, 2, 4, 8 lanes below in the row of 16
    v = F::of(moved<0x112, 0xF>(v, none), v);
    v = F::of(moved<0x114, 0xF>(v, none), v);
    v = F::of(moved<0x118, 0xF>(v, none), v);
    v = F::of(moved<0x142, 0xA>(v, none), v);                    // rows 0 and 2 into 1 and 3
    v = F::of(moved<0x143, 0xC>(v, none), v);                    // the lower half's into the upper
    return v;
}
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
template <int NT, typename F, typename T>
__device__ __forceinline__ T block_all(T v, void* s) {
    v = wave_scan<F>(v);
    if (lane_id() == 63) ((T*)s)[threadIdx.x / 64] = v;
    __syncthreads();
    const int l = lane_id() & 15;
    return of_lane(wave_scan<F>(l < NT / 64 ? ((const T*)s)[l] : F::template none<T>()), 15);
}
// sum over the threads up to and with this one; that of all
template <int NT, typename T>
__device__ __forceinline__ T block_sums(T v, T& all, void* s) {
    v = wave_scan<Plus>(v);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    if (lane_id() == 63) ((T*)s)[wave] = v;
    __syncthreads();
    const int l = lane_id() & 15;
    const T w = wave_scan<Plus>(l < NT / 64 ? ((const T*)s)[l] : (T)0);
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

// ------------------------------------------------------------------ a chunk
constexpr int CHUNK_BINS = 1024;
struct ChunkShared {
    uint32_t cnt[CHUNK_BINS];
    uint64_t s[8][16];
    int at[2];
    int part[4][16];
};

// NT threads with E logits each; `share`: how many candidates may be written
template <bool F32, int NT, int E>
__device__ void sample_chunk(const SampleArgs& a, int r, int c, int share, Chunk* info, uint64_t* list, ChunkShared& s) {
    constexpr int NV = E / 4, SW = NT / 64;
    static_assert(NT * E == CHUNK && NV <= 4, "chunk");
    const void* row = (const uint8_t*)a.logits + (size_t)r * a.stride * (F32 ? 4 : 2);
    const int V = a.V, c0 = c * CHUNK, t = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(t / 64);
    float x[NV][4];
#pragma unroll
    for (int j = 0; j < NV; ++j) load_logits<F32>(row, c0 + (j * NT + t) * 4, V, x[j]);
    const Request q(a, r);
    for (int i = t; i < CHUNK_BINS; i += NT) s.cnt[i] = 0;
    float top = -INF, low = INF;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const float y = x[j][v] == x[j][v] ? x[j][v] : INF;
            top = fmaxf(top, y);
            if (y > -INF) low = fminf(low, y);
        }
    {
        const float wt = wave_scan<Most>(top), wl = wave_scan<Least>(low);
        if (lane_id() == 63) {
            ((float*)s.s[0])[wave] = wt;
            ((float*)s.s[1])[wave] = wl;
        }
        __syncthreads();
        const int l = lane_id() & 15;
        top = of_lane(wave_scan<Most>(l < SW ? ((const float*)s.s[0])[l] : -INF), 15);
        low = of_lane(wave_scan<Least>(l < SW ? ((const float*)s.s[1])[l] : INF), 15);
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
        double sum = 0.0;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v) sum += x[j][v] == -INF ? 0.0 : exp_neg(((double)x[j][v] - (double)top) * q.inv);
        out.sum = block_all<NT, Plus>(sum, s.s[2]);
    }
    if (q.k == 0 && !q.p_on && !q.m_on) {
        if (t == 0) *info = out;
        return;
    }
    const float floor = fmaxf(q.floor(top, out.sum, V), low);
    // Candidates: from `least` on. More than the share, or than a few times k:
    // those of the parts up to the k-th (what is left out then is out), or of as
    // many parts as fit the share.
    auto count = [&](auto f) __attribute__((always_inline)) {
        int n = 0;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v) n += f(x[j][v]);
        return n;
    };
    const int all = block_all<NT, Plus>(count([&](float y) { return y >= floor; }), s.s[3]);
    const Parts<CHUNK_BINS> part(top, floor);
    int last = CHUNK_BINS;
    if (all > share || (q.k && all > 2 * q.k + 64)) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v)
                if (x[j][v] >= floor) atomicAdd(&s.cnt[part.of(x[j][v])], 1u);
        __syncthreads();
        uint32_t before;
        const int want = q.k ? min(q.k, share) : share;
        last = part_of_count<NT, CHUNK_BINS>(s.cnt, (uint32_t)want, before, s.s[4], s.at);
        if (last < 0) last = CHUNK_BINS;
        else {
            const bool fits = (int)(before + s.cnt[last]) <= share;
            if (!fits) --last;
            if (!fits || !q.k || q.k > share) {
                float cut = -INF;
#pragma unroll
                for (int j = 0; j < NV; ++j)
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        if (x[j][v] >= floor && part.of(x[j][v]) > last) cut = fmaxf(cut, x[j][v]);
                out.cut = block_all<NT, Most>(cut, s.s[5]);
            }
        }
    }
    // in the order of their ids: [vector][wave][lane][element]
    auto in = [&](float y) { return y >= floor && part.of(y) <= last; };
    int at[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        int before = 0, n = 0;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const uint64_t b = __ballot(in(x[j][v]));
            before += __popcll(b & lanemask_lt());
            n += __popcll(b);
        }
        at[j] = before;
        if (lane_id() == 0) s.part[j][wave] = n;
    }
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int w = 0; w < SW; ++w) {
            if (w == wave) at[j] += total;
            total += s.part[j][w];
        }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        int to = at[j];
#pragma unroll
        for (int v = 0; v < 4; ++v)
            if (in(x[j][v])) list[to++] = place_of(x[j][v], c0 + (j * NT + t) * 4 + v);
    }
    out.n = total;
    if (t == 0) *info = out;
}

// ------------------------------------------------------------------ a row
struct RowShared {
    uint64_t list[LIST];      // candidates by id
    uint64_t sorted[LIST];    // ... by place; wave sums of a draw
    uint32_t cnt[BINS];
    uint64_t mass[BINS];
    double ends[MAX_CHUNKS];  // weight up to and with a chunk
    uint64_t s[16][16];
    double got[2];
    uint64_t border[2];
    int at[2], hit[2];
    int n;
};

// The lowest id in [lo, hi) (lo a multiple of four) up to and with which the
// weights exceed `aim` (past their sum: the last id with a weight), -1 if there
// is no weight. aim(sum) gives it. The id is left in s.hit[0], the sum in
// s.got[1] and the id's weight in s.got[0].
template <bool F32, typename W, typename A>
__device__ void draw(const void* row, int lo, int hi, W weight, A aim, RowShared& s) {
    double* sums = (double*)s.sorted;                            // of 256 ids each, LIST of them at most
    const int t = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(t / 64);
    const int groups = (hi - lo + 255) / 256;
    __syncthreads();
    for (int g = wave; g < groups; g += ST / 64) {
        float x[4];
        const int id = lo + g * 256 + lane * 4;
        load_logits<F32>(row, id, hi, x);
        double w = 0.0;
#pragma unroll
        for (int v = 0; v < 4; ++v) w += weight(x[v], id + v);
        w = wave_scan<Plus>(w);
        if (lane == 63) sums[g] = w;
    }
    if (t == 0) s.hit[0] = s.hit[1] = -1;
    __syncthreads();
    // a run of groups for each thread
    const int run = (groups + ST - 1) / ST, g0 = min(t * run, groups), g1 = min(g0 + run, groups);
    double own = 0.0, total;
    for (int g = g0; g < g1; ++g) own += sums[g];
    const double end = block_sums<ST>(own, total, s.s[0]);
    const double want = aim(total);
    // the group: the first one whose end exceeds the aim, else the last one with a weight
    {
        double e = end - own;
        for (int g = g0; g < g1; ++g) {
            const double before = e;
            e += sums[g];
            if (sums[g] > 0.0) {
                atomicMax(&s.hit[1], g);
                if (e > want && before <= want) atomicMax(&s.hit[0], g);
            }
        }
    }
    __syncthreads();
    const int found = s.hit[0], last = s.hit[1], g = found >= 0 ? found : last;
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
        float x[4];
        const int id = lo + g * 256 + lane * 4;
        load_logits<F32>(row, id, hi, x);
        double w[4], sum = 0.0;
#pragma unroll
        for (int v = 0; v < 4; ++v) sum += w[v] = weight(x[v], id + v);
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

template <bool F32>
__device__ void sample_finish(const SampleArgs& a, int r, int chunks, int share, const Chunk* info, const uint64_t* lists, RowShared& s) {
    const void* row = (const uint8_t*)a.logits + (size_t)r * a.stride * (F32 ? 4 : 2);
    const int V = a.V, t = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(t / 64);
    // four candidates of a chunk for each thread (memory behind the last one is the lists' own)
    const int c4 = min(4 * t / share, chunks - 1), i4 = 4 * t - c4 * share;
    uint64_t e[4];
    int n4 = 0;
    if (4 * t < chunks * share) {
        n4 = info[c4].n;
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = lists[(size_t)c4 * share + i4 + i];
    }
    Chunk mine{0.0, -INF, INF, -INF, 0};
    if (t < chunks) mine = info[t];
    const Request q(a, r);
    const double u = a.u[r];
    auto give = [&](int id, double p) {
        if (t == 0) {
            a.ids[r] = id;
            if (a.p) a.p[r] = (float)p;
            if (id < 0 && a.err) atomicAdd(a.err, 1);
        }
    };
    for (int i = t; i < BINS; i += ST) s.cnt[i] = 0;
    float top, low, cut;
    {
        const float wt = wave_scan<Most>(mine.top), wl = wave_scan<Least>(mine.low), wc = wave_scan<Most>(mine.cut);
        if (lane_id() == 63) {
            ((float*)s.s[1])[wave] = wt;
            ((float*)s.s[2])[wave] = wl;
            ((float*)s.s[3])[wave] = wc;
        }
        __syncthreads();
        const int l = lane_id() & 15;
        top = of_lane(wave_scan<Most>(((const float*)s.s[1])[l]), 15);
        low = of_lane(wave_scan<Least>(((const float*)s.s[2])[l]), 15);
        cut = of_lane(wave_scan<Most>(((const float*)s.s[3])[l]), 15);
    }
    if (q.bad || !(top < INF) || top == -INF) return give(-1, 0.0);
    const double zmax = top;
    auto weight = [&](float x) { return x == -INF ? 0.0 : exp_neg(((double)x - zmax) * q.inv); };

    if (q.k == 1) {
        uint64_t best = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i4 + i < n4) best = Most::of(best, e[i]);
        return give(place_id(block_all<ST, Most>(best, s.s[4])), 1.0);
    }
    // the row's weight from the chunks'
    double all;
    const double part = t < chunks && mine.sum > 0.0 ? mine.sum * exp_neg(((double)mine.top - zmax) * q.inv) : 0.0;
    const double end = block_sums<ST>(part, all, s.s[5]);
    if (q.k == 0 && !q.p_on && !q.m_on) {
        // no filter: the chunk that the aim falls into (past the sum: the last with a weight)
        if (t < chunks) s.ends[t] = end;
        if (t == 0) s.at[0] = s.at[1] = -1;
        __syncthreads();
        const double aim = u * all;
        if (part > 0.0) {
            atomicMax(&s.at[1], t);
            if (s.ends[t] > aim && (t == 0 || s.ends[t - 1] <= aim)) atomicMax(&s.at[0], t);
        }
        __syncthreads();
        const int c = s.at[0] >= 0 ? s.at[0] : s.at[1];
        const double before = c ? s.ends[c - 1] : 0.0;
        draw<F32>(row, c * CHUNK, min((c + 1) * CHUNK, V), [&](float x, int) { return weight(x); },
                  [&](double) { return aim - before; }, s);
        return give(s.hit[0], s.got[0] / all);
    }

    // ---- few candidates
    const float least = q.floor(top, all, V), floor = fmaxf(least, low);
    const Parts<BINS> parts(top, floor);
    uint64_t border = 0;                                         // the last kept place (before min_p)
    {
        bool in[4];
        int own = 0, n;
#pragma unroll
        for (int i = 0; i < 4; ++i) own += in[i] = i4 + i < n4 && place_logit(e[i]) >= floor;
        int to = block_sums<ST>(own, n, s.s[6]);
        if (q.k && n > 2 * q.k + 64) {                           // those of the parts up to the k-th
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (in[i]) atomicAdd(&s.cnt[parts.of(place_logit(e[i]))], 1u);
            __syncthreads();
            uint32_t before;
            const int last = part_of_count<ST, BINS>(s.cnt, (uint32_t)q.k, before, s.s[7], s.at);
            own = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) own += in[i] = in[i] && parts.of(place_logit(e[i])) <= last;
            to = block_sums<ST>(own, n, s.s[8]);
        }
        to -= own;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (in[i]) {
                s.list[to] = e[i];
                s.sorted[to++] = e[i];
            }
        __syncthreads();
        if (n) sort_places(s.sorted, n);
        // a run of four of the order for each thread
        int keep = q.k ? min(n, q.k) : n;
        bool sure = !(cut >= least);                             // nothing that counts was left out
        if (q.k && !sure) sure = n >= q.k && place_logit(s.sorted[q.k - 1]) > cut;
        const bool reach = sure;
        if (q.p_on && n) {
            double w[4], sum = 0.0, total;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                w[i] = 4 * t + i < keep ? weight(place_logit(s.sorted[4 * t + i])) : 0.0;
                sum += w[i];
            }
            double before = block_sums<ST>(sum, total, s.s[9]) - sum;
            const double want = q.top_p * (q.k ? total : all);
            int m = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (4 * t + i < keep && (before < want || 4 * t + i == 0)) m = 4 * t + i + 1;
                before += w[i];
            }
            m = block_all<ST, Most>(m, s.s[10]);
            // (k off, candidates left out: the border has to lie among those that are here, before all of the others)
            if (!q.k && !reach) sure = total >= want && place_logit(s.sorted[m - 1]) > cut;
            keep = m;
        }
        if (sure) {
            border = s.sorted[keep - 1];
            // the draw by id
            double w[4], sum = 0.0, total;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                w[i] = 0.0;
                if (4 * t + i < n && s.list[4 * t + i] >= border) {
                    w[i] = weight(place_logit(s.list[4 * t + i]));
                    if (w[i] < q.min_p) w[i] = 0.0;
                }
                sum += w[i];
            }
            if (t == 0) s.hit[0] = 0x7FFFFFFF, s.hit[1] = -1;
            double x = block_sums<ST>(sum, total, s.s[11]) - sum;
            const double aim = u * total;
            int first = 0x7FFFFFFF, last = -1;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x += w[i];
                if (w[i] > 0.0) {
                    last = 4 * t + i;
                    if (x > aim) first = min(first, 4 * t + i);
                }
            }
            if (last >= 0) atomicMax(&s.hit[1], last);
            if (first != 0x7FFFFFFF) atomicMin(&s.hit[0], first);
            __syncthreads();
            const uint64_t chosen = s.list[s.hit[0] != 0x7FFFFFFF ? s.hit[0] : s.hit[1]];
            return give(place_id(chosen), weight(place_logit(chosen)) / total);
        }
    }

    // ---- many: over the row again. Logits 2^-46 of the largest weight and less do not count.
    auto mass = [&](float x) { return (uint64_t)__builtin_rint(weight(x) * ONE); };
    const float bottom = fmaxf(q.least(top, 1.0 / 70368744177664.0), low);
    const Parts<BINS> every(top, bottom);
    auto each = [&](auto f) {
        for (int i = t * 4; i < V; i += ST * 4) {
            float x[4];
            load_logits<F32>(row, i, V, x);
#pragma unroll
            for (int v = 0; v < 4; ++v)
                if (x[v] >= bottom) f(x[v], i + v);
        }
    };
    if (q.k || q.p_on) {
        __syncthreads();
        for (int i = t; i < BINS; i += ST) {
            s.cnt[i] = 0;
            s.mass[i] = 0;
        }
        __syncthreads();
        each([&](float x, int) {
            const int b = every.of(x);
            atomicAdd(&s.cnt[b], 1u);
            atomicAdd((unsigned long long*)&s.mass[b], (unsigned long long)mass(x));
        });
        __syncthreads();
        // the tokens of part b that lie before (mass: whose masses before them stay below) `want`, the first one always:
        // the last of them, and all their mass
        auto border_in = [&](int b, uint64_t want, bool by_mass, uint64_t& kept) -> uint64_t {
            const int m = (int)s.cnt[b];
            if (t == 0) s.n = 0;
            __syncthreads();
            if (m <= LIST) {
                each([&](float x, int id) {
                    if (every.of(x) == b) s.sorted[atomicAdd(&s.n, 1)] = place_of(x, id);
                });
                __syncthreads();
                sort_places(s.sorted, m);
                uint64_t w[4], own = 0, all_of;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    w[i] = 4 * t + i < m ? mass(place_logit(s.sorted[4 * t + i])) : 0;
                    own += w[i];
                }
                uint64_t before = block_sums<ST>(own, all_of, s.s[1]) - own, in = 0;
                int keep = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int at = 4 * t + i;
                    if (at < m && ((by_mass ? before : (uint64_t)at) < want || at == 0)) {
                        keep = at + 1;
                        in += w[i];
                    }
                    before += w[i];
                }
                keep = block_all<ST, Most>(keep, s.s[2]);
                kept = block_all<ST, Plus>(in, s.s[3]);
                return s.sorted[keep - 1];
            }
            // more than can be sorted: halve the range of keys until one is left
            uint32_t lo = ~0u, hi = 0;
            each([&](float x, int) {
                if (every.of(x) == b) {
                    lo = min(lo, logit_key(x));
                    hi = max(hi, logit_key(x));
                }
            });
            lo = block_all<ST, Least>(lo, s.s[1]);
            hi = block_all<ST, Most>(hi, s.s[2]);
            auto above = [&](uint32_t key, bool masses) {
                uint64_t v = 0;
                each([&](float x, int) {
                    if (every.of(x) == b && logit_key(x) > key) v += masses ? mass(x) : 1;
                });
                __syncthreads();
                return block_all<ST, Plus>(v, s.s[3]);
            };
            if (want == 0) want = 1;
            while (lo < hi) {                                    // the smallest key with less than `want` above it
                const uint32_t mid = lo + (hi - lo) / 2;
                if (above(mid, by_mass) < want) hi = mid;
                else lo = mid + 1;
            }
            // of the tokens with that key the first by id
            const uint64_t each_one = by_mass ? mass(key_logit(lo)) : 1, left = want - above(lo, by_mass);
            const uint64_t ties = each_one ? (left + each_one - 1) / each_one : (uint64_t)V;
            const uint32_t key = lo;
            kept = above(lo, true);
            draw<F32>(row, 0, V, [&](float x, int) { return x > -INF && logit_key(x) == key ? 1.0 : 0.0; },
                      [&](double sum) { return fmin((double)ties, sum) - 1.0; }, s);
            kept += (uint64_t)fmin((double)ties, s.got[1]) * mass(key_logit(key));
            return (uint64_t)key << 32 | (uint32_t)~s.hit[0];
        };
        // masses of this thread's two parts, and up to and with them
        const uint64_t first = s.mass[2 * t], second = s.mass[2 * t + 1];
        uint64_t whole;
        const uint64_t ends = block_sums<ST>(first + second, whole, s.s[4]);
        if (q.k) {
            uint32_t before;
            const int b = part_of_count<ST, BINS>(s.cnt, (uint32_t)q.k, before, s.s[5], s.at);
            if (b >= 0) {
                if (t == b / 2) s.border[0] = ends - (b & 1 ? second : first + second);
                __syncthreads();
                uint64_t kept;
                border = border_in(b, q.k - before, false, kept);
                whole = s.border[0] + kept;
            }
        }
        if (q.p_on) {
            const double x = __builtin_ceil(q.top_p * (double)whole);
            const uint64_t want = x < 1.0 ? 1 : (uint64_t)x;
            const uint64_t start = ends - first - second;
            __syncthreads();
            if (t == 0) s.at[0] = 0;
            __syncthreads();
            if (start < want && want <= ends) {
                const bool later = start + first < want;
                s.at[0] = 2 * t + later;
                s.border[1] = later ? start + first : start;
            }
            __syncthreads();
            uint64_t kept;
            const int b = s.at[0];
            const uint64_t p = border_in(b, want - s.border[1], true, kept);
            border = Most::of(border, p);
        }
    }
    draw<F32>(row, 0, V, [&](float x, int id) {
                  if (!(x >= bottom) || place_of(x, id) < border) return 0.0;
                  const double w = weight(x);
                  return w >= q.min_p ? w : 0.0;
              }, [&](double sum) { return u * sum; }, s);
    give(s.hit[0], s.got[0] / s.got[1]);
}

constexpr int CHUNK_THREADS = 256;
template <bool F32>
__global__ void __launch_bounds__(CHUNK_THREADS) sample_chunk_kernel(SampleArgs a, int chunks, int share, Chunk* info, uint64_t* lists) {
    __shared__ ChunkShared s;
    const long long n = (long long)a.B * chunks;
    for (long long i = blockIdx.x; i < n; i += gridDim.x) {
        sample_chunk<F32, CHUNK_THREADS, CHUNK / CHUNK_THREADS>(a, (int)(i / chunks), (int)(i % chunks), share, info + i, lists + i * share, s);
        __syncthreads();
    }
}
template <bool F32>
__global__ void __launch_bounds__(ST) sample_finish_kernel(SampleArgs a, int chunks, int share, const Chunk* info, const uint64_t* lists) {
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    const size_t i = (size_t)blockIdx.x * chunks;
    sample_finish<F32>(a, blockIdx.x, chunks, share, info + i, lists + i * share, *(RowShared*)smem);
}
// rows of one chunk
template <bool F32>
__global__ void __launch_bounds__(ST) sample_row_kernel(SampleArgs a, int share, Chunk* info, uint64_t* lists) {
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    const size_t i = blockIdx.x;
    sample_chunk<F32, ST, CHUNK / ST>(a, (int)i, 0, share, info + i, lists + i * share, *(ChunkShared*)smem);
    __syncthreads();
    sample_finish<F32>(a, (int)i, 1, share, info + i, lists + i * share, *(RowShared*)smem);
}

static int chunks_of(int V) { return (V + CHUNK - 1) / CHUNK; }
static int share_of(int chunks) { return LIST / chunks / 4 * 4; }
static size_t info_bytes(int B, int V) { return ((size_t)B * chunks_of(V) * sizeof(Chunk) + 255) / 256 * 256; }
size_t sample_workspace_bytes(int B, int V) {
    const int chunks = chunks_of(V);
    return info_bytes(B, V) + (size_t)B * chunks * share_of(chunks) * 8;
}

template <bool F32>
static hipError_t launch(const SampleArgs& a, void* ws, hipStream_t stream) {
    const int chunks = chunks_of(a.V), share = share_of(chunks);
    Chunk* info = (Chunk*)ws;
    uint64_t* lists = (uint64_t*)((uint8_t*)ws + info_bytes(a.B, a.V));
    static_assert(sizeof(RowShared) <= 163840 && sizeof(ChunkShared) <= sizeof(RowShared), "LDS");
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    static std::atomic<uint64_t> done[2];
    if (chunks == 1) {
        e = allow_lds((const void*)sample_row_kernel<F32>, sizeof(RowShared), dev, done[0]);
        if (e != hipSuccess) return e;
        return launch_kernel(K_SAMPLE, stream, sample_row_kernel<F32>, dim3((unsigned)a.B), dim3(ST), sizeof(RowShared), a, share, info, lists);
    }
    e = allow_lds((const void*)sample_finish_kernel<F32>, sizeof(RowShared), dev, done[1]);
    if (e != hipSuccess) return e;
    const long long n = (long long)a.B * chunks;
    e = launch_kernel(K_SAMPLE, stream, sample_chunk_kernel<F32>, dim3((unsigned)(n < (1 << 20) ? n : 1 << 20)), dim3(CHUNK_THREADS), 0, a,
                      chunks, share, info, lists);
    if (e != hipSuccess) return e;
    return launch_kernel(K_SAMPLE, stream, sample_finish_kernel<F32>, dim3((unsigned)a.B), dim3(ST), sizeof(RowShared), a, chunks, share,
                         (const Chunk*)info, (const uint64_t*)lists);
}
hipError_t launch_sample(const SampleArgs& a, bool f32, void* ws, hipStream_t stream) {
    return f32 ? launch<true>(a, ws, stream) : launch<false>(a, ws, stream);
}

}  // namespace moe
