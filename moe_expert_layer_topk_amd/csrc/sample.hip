// One token per row of logits: temperature, top-k, top-p, min-p and the draw
// from a given random number.
//
// The kept tokens are a prefix of the order (logit falling, id rising), so one
// border, a (logit, id), describes them: every token before it or equal to it,
// with w >= min_p. The draw is a search in the sums of their weights by id.
//
// chunk kernel: one workgroup for each 1024 E logits, which it reads once and
// holds in registers. It writes the chunk's largest and smallest logit, its weight and,
// for rows with a filter, the tokens that the filter could keep, in the order of
// their ids. A chunk can tell from itself alone, with m its largest logit, S its
// weight (relative to m), V the row's length:
//   top_k: a token that k tokens of the chunk precede is out;
//   min_p: the row's largest logit is m at least, so w < min_p relative to m is out;
//   top_p: at least (1 - top_p) of the weight lies at and behind the last kept
//     token, on at most V tokens that weigh no more than it, so w < (1 - top_p) S / V is out.
// With top_k and top_p only the first holds: top_p's share is one of the weight
// of all k tokens.
// finish kernel: one workgroup a row. Few candidates (nearly always, with a
// filter): sorted in LDS, borders from prefix sums. No filter: the chunk that
// the draw falls into is read again. Else (a top_p that keeps thousands of
// tokens) the row is read again: counts and weights of 2048 equal parts of
// the logits' range, the tokens of the part that holds the border sorted, the
// kept weight by id.
//
// Weights are fp64, sums of them fp64 in a fixed order; the parts' weights are
// summed with atomics, and therefore as integers (multiples of 2^-42 of the
// largest weight).
#include "moe_common.h"
#include "moe_kernels.h"
#include "gemm_tile.h"

namespace moe {

constexpr int ST = 1024, SW = ST / 64;                           // threads, waves of a workgroup
constexpr int CAP = 1536;                                        // candidates of a chunk that are written
constexpr int LIST = 4096;                                       // candidates of a row that are sorted
constexpr int BINS = 2048;
constexpr int MAX_CHUNKS = 256;
constexpr double ONE = 4398046511104.0;                          // 2^42: the sum of 2^20 weights stays below 2^63
constexpr float INF = __builtin_inff();

struct Chunk {
    double sum;               // weight relative to `top`
    float top, low;           // largest (+inf: NaN or +inf among them) and smallest logit that is not -inf
    int n;                    // candidates, CAP + 1 for more than CAP
    int pad;
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
    // the smallest logit whose weight could reach w beside a logit of m, rounded down
    __device__ __forceinline__ float least(float m, double w) const {
        if (!(w > 0.0) || temperature == INF) return -INF;
        const double d = log(w) * temperature;
        return (float)((double)m + d - (fabs((double)m) + fabs(d)) * 1e-6);
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

// ---- over the workgroup; `s` holds one value a wave and is free again after the next barrier
template <typename T, typename F>
__device__ __forceinline__ T block_reduce(T v, F f, T* s) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = f(v, (T)__shfl_xor(v, o, 64));
    __syncthreads();
    if (lane_id() == 0) s[threadIdx.x / 64] = v;
    __syncthreads();
    v = s[lane_id() & (SW - 1)];
#pragma unroll
    for (int o = SW / 2; o > 0; o >>= 1) v = f(v, (T)__shfl_xor(v, o, 64));
    return v;
}
struct Plus {
    template <typename T>
    __device__ __forceinline__ T operator()(T x, T y) const { return x + y; }
};
struct Most {
    template <typename T>
    __device__ __forceinline__ T operator()(T x, T y) const { return x > y ? x : y; }
};
struct Least {
    template <typename T>
    __device__ __forceinline__ T operator()(T x, T y) const { return x < y ? x : y; }
};
// sum over the threads up to and with this one
template <typename T>
__device__ __forceinline__ T block_sums(T v, T* s) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const T y = __shfl_up(v, o, 64);
        if (lane_id() >= o) v += y;
    }
    __syncthreads();
    if (lane_id() == 63) s[threadIdx.x / 64] = v;
    __syncthreads();
    T w = s[lane_id() & (SW - 1)];
#pragma unroll
    for (int o = 1; o < SW; o <<= 1) {
        const T y = __shfl_up(w, o, SW);
        if ((lane_id() & (SW - 1)) >= o) w += y;
    }
    const int wave = threadIdx.x / 64;
    const T before = __shfl(w, max(wave - 1, 0), 64);
    return wave ? before + v : v;
}

// equal parts of [low, top], the largest logits first (part: monotone in x)
struct Parts {
    float top, scale;
    __device__ __forceinline__ Parts(float t, float low) : top(t), scale(t > low ? (float)BINS / (t - low) : 0.f) {}
    __device__ __forceinline__ int of(float x) const { return (int)fminf((top - x) * scale, (float)(BINS - 1)); }
};
// the first part up to and with which the counts reach `want`, -1 if they never do; how many lie before it
__device__ __forceinline__ int part_of_count(const uint32_t* cnt, uint32_t want, uint32_t& before, uint32_t* s, int* s_at) {
    const uint32_t a = cnt[2 * threadIdx.x], b = cnt[2 * threadIdx.x + 1];
    const uint32_t end = block_sums(a + b, s);
    if (threadIdx.x == 0) s_at[0] = -1;
    __syncthreads();
    const uint32_t start = end - a - b;
    if (start < want && want <= end) {
        const bool second = start + a < want;
        s_at[0] = 2 * threadIdx.x + second;
        s_at[1] = (int)(second ? start + a : start);
    }
    __syncthreads();
    before = (uint32_t)s_at[1];
    const int at = s_at[0];
    __syncthreads();
    return at;
}

// n <= LIST places in LDS, largest first; n rounded up to a power of two with zeros
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
struct ChunkShared {
    uint32_t cnt[BINS];
    double sum[SW];
    uint64_t best[SW];
    float f[SW];
    uint32_t u[SW];
    int at[2];
    int part[16][SW];
};

template <bool F32, int E>
__device__ void sample_chunk(const SampleArgs& a, int r, int c, Chunk* info, uint2* list, ChunkShared& s) {
    constexpr int NV = E / 4;
    const void* row = (const uint8_t*)a.logits + (size_t)r * a.stride * (F32 ? 4 : 2);
    const int V = a.V, c0 = c * ST * E, t = threadIdx.x, wave = t / 64;
    const Request q(a, r);
    float x[NV][4];
#pragma unroll
    for (int j = 0; j < NV; ++j) load_logits<F32>(row, c0 + (j * ST + t) * 4, V, x[j]);
    float top = -INF, low = INF;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const float y = x[j][v] == x[j][v] ? x[j][v] : INF;
            top = fmaxf(top, y);
            if (y > -INF) low = fminf(low, y);
        }
    const float own = top;                                       // the thread's largest
    top = block_reduce(top, Most(), s.f);
    Chunk out{0.0, top, 0.f, 0, 0};
    if (q.bad || !(top < INF) || top == -INF) {
        if (t == 0) *info = out;
        return;
    }
    if (q.k == 1) {                                              // the first token of the order
        uint64_t best = 0;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v) best = Most()(best, place_of(x[j][v], c0 + (j * ST + t) * 4 + v));
        best = block_reduce(best, Most(), s.best);
        if (t == 0) {
            list[0] = make_uint2((uint32_t)best, (uint32_t)(best >> 32));
            out.n = 1;
            *info = out;
        }
        return;
    }
    out.low = low = block_reduce(low, Least(), s.f);
    // the chunk's weight, where the row's is needed (with top_k its candidates have it; min_p alone: likewise)
    if (q.k == 0 && (q.p_on || !q.m_on)) {
        double sum = 0.0;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v) sum += x[j][v] == -INF ? 0.0 : exp_neg(((double)x[j][v] - (double)top) * q.inv);
        out.sum = block_reduce(sum, Plus(), s.sum);
    }
    if (q.k == 0 && !q.p_on && !q.m_on) {
        if (t == 0) *info = out;
        return;
    }
    float floor = -INF;
    if (!(q.k && q.p_on)) {
        if (q.m_on) floor = q.least(top, q.min_p);
        if (q.p_on) floor = fmaxf(floor, q.least(top, (1.0 - q.top_p) * out.sum / V));
    }
    bool in[NV][4];
    int n = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            in[j][v] = x[j][v] > -INF && x[j][v] >= floor;
            n += in[j][v];
        }
    if (q.k) {
        // more of them than a few times k: those of the parts up to the k-th. (1024
        // threads' largest bound the first 1024 tokens from below.)
        const int all = block_reduce(n, Plus(), (int*)s.u);
        if (all > 2 * q.k + 64) {
            const float least = block_reduce(own, Least(), s.f);
            const Parts part(top, fmaxf(floor, q.k <= ST && least > -INF ? least : low));
            for (int i = t; i < BINS; i += ST) s.cnt[i] = 0;
            __syncthreads();
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    if (in[j][v] && (q.k > ST || x[j][v] >= least)) atomicAdd(&s.cnt[part.of(x[j][v])], 1u);
            __syncthreads();
            uint32_t before;
            const int last = part_of_count(s.cnt, (uint32_t)q.k, before, s.u, s.at);
            if (last >= 0) {
#pragma unroll
                for (int j = 0; j < NV; ++j)
#pragma unroll
                    for (int v = 0; v < 4; ++v) in[j][v] = in[j][v] && (q.k > ST || x[j][v] >= least) && part.of(x[j][v]) <= last;
            }
        }
    }
    // candidates in the order of their ids: [vector][wave][lane][element]
    int at[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        int before = 0, count = 0;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const uint64_t b = __ballot(in[j][v]);
            before += __popcll(b & lanemask_lt());
            count += __popcll(b);
        }
        at[j] = before;
        if (lane_id() == 0) s.part[j][wave] = count;
    }
    __syncthreads();
    int total = 0, start[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int w = 0; w < SW; ++w) {
            if (w == wave) start[j] = total;
            total += s.part[j][w];
        }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        int to = start[j] + at[j];
#pragma unroll
        for (int v = 0; v < 4; ++v)
            if (in[j][v]) {
                if (to < CAP) list[to] = make_uint2(~(uint32_t)(c0 + (j * ST + t) * 4 + v), logit_key(x[j][v]));
                ++to;
            }
    }
    out.n = min(total, CAP + 1);
    if (t == 0) *info = out;
}

// ------------------------------------------------------------------ a row
struct RowShared {
    uint64_t list[LIST];      // candidates by id
    uint64_t sorted[LIST];    // ... by place; wave sums of a draw
    uint32_t cnt[BINS];
    uint64_t mass[BINS];
    double ends[MAX_CHUNKS];  // weight up to and with a chunk
    int first[MAX_CHUNKS + 1];
    double sum[SW];
    uint64_t best[SW];
    float f[SW];
    uint32_t u[SW];
    int at[2];
    int n;
    double d;
};

// The lowest id in [lo, hi) (lo a multiple of four) up to and with which the
// weights exceed `aim` (past their sum: the last id with a weight), -1 if there
// is no weight. aim(sum) gives it. Returned in s.at[0], the sum in s.d and the
// id's weight in s.sum[0], to all threads.
template <bool F32, typename W, typename A>
__device__ void draw(const void* row, int lo, int hi, W weight, A aim, RowShared& s) {
    double* sums = (double*)s.sorted;                            // of 256 ids each, LIST of them
    const int t = threadIdx.x, lane = lane_id(), wave = t / 64;
    const int groups = (hi - lo + 255) / 256;
    __syncthreads();
    for (int g = wave; g < groups; g += SW) {
        float x[4];
        const int id = lo + g * 256 + lane * 4;
        load_logits<F32>(row, id, hi, x);
        double w = 0.0;
#pragma unroll
        for (int v = 0; v < 4; ++v) w += weight(x[v], id + v);
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) w += __shfl_xor(w, o, 64);
        if (lane == 0) sums[g] = w;
    }
    __syncthreads();
    // a run of groups for each thread
    const int run = (groups + ST - 1) / ST, g0 = min(t * run, groups), g1 = min(g0 + run, groups);
    double own = 0.0;
    for (int g = g0; g < g1; ++g) own += sums[g];
    const double end = block_sums(own, s.sum);
    __syncthreads();
    if (t == ST - 1) s.d = end;
    if (t == 0) s.at[0] = s.at[1] = -1;
    __syncthreads();
    const double total = s.d, want = aim(total);
    // the group: the first one whose end exceeds the aim, else the last one with a weight
    {
        double e = end - own;
        for (int g = g0; g < g1; ++g) {
            const double before = e;
            e += sums[g];
            if (sums[g] > 0.0) {
                atomicMax(&s.at[1], g);
                if (e > want && before <= want) atomicMax(&s.at[0], g);
            }
        }
    }
    __syncthreads();
    const int found = s.at[0], last = s.at[1], g = found >= 0 ? found : last;
    if (g >= g0 && g < g1) {
        double e = end - own;
        for (int i = g0; i < g; ++i) e += sums[i];
        s.sum[1] = e;
    }
    __syncthreads();
    const double start = s.sum[1];
    __syncthreads();
    if (g < 0) return;                                           // (s.at[0] is -1)
    if (wave == 0) {
        float x[4];
        const int id = lo + g * 256 + lane * 4;
        load_logits<F32>(row, id, hi, x);
        double w[4], sum = 0.0;
#pragma unroll
        for (int v = 0; v < 4; ++v) sum += w[v] = weight(x[v], id + v);
        double e = sum;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const double y = __shfl_up(e, o, 64);
            if (lane >= o) e += y;
        }
        e = start + (e - sum);
        int at = 0x7FFFFFFF, any = -1;
        double wa = 0.0, wy = 0.0;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            e += w[v];
            if (w[v] > 0.0) {
                any = id + v;
                wy = w[v];
                if (e > want && at == 0x7FFFFFFF) {
                    at = id + v;
                    wa = w[v];
                }
            }
        }
        const uint64_t hit = __ballot(at != 0x7FFFFFFF), some = __ballot(any >= 0);
        const int from = hit ? __ffsll((long long)hit) - 1 : 63 - __clzll((long long)some);
        if (lane == from) {
            s.at[0] = hit ? at : any;
            s.sum[0] = hit ? wa : wy;
        }
    }
    __syncthreads();
}

template <bool F32>
__device__ void sample_finish(const SampleArgs& a, int r, int chunks, int chunk_size, const Chunk* info, const uint2* lists, RowShared& s) {
    const void* row = (const uint8_t*)a.logits + (size_t)r * a.stride * (F32 ? 4 : 2);
    const int V = a.V, t = threadIdx.x;
    const Request q(a, r);
    const double u = a.u[r];
    auto give = [&](int id, double p) {
        if (t == 0) {
            a.ids[r] = id;
            if (a.p) a.p[r] = (float)p;
            if (id < 0 && a.err) atomicAdd(a.err, 1);
        }
    };
    Chunk mine{0.0, -INF, INF, 0, 0};
    if (t < chunks) mine = info[t];
    const float top = block_reduce(mine.top, Most(), s.f);
    if (q.bad || !(top < INF) || top == -INF) return give(-1, 0.0);
    if (mine.top == -INF) mine.low = INF;                        // (a chunk without a token)
    const int n_all = block_reduce(mine.n, Plus(), (int*)s.u);
    const bool over = block_reduce(mine.n, Most(), (int*)s.u) > CAP;
    const double zmax = top;
    auto weight = [&](float x) { return x == -INF ? 0.0 : exp_neg(((double)x - zmax) * q.inv); };

    if (q.k == 1) {
        uint64_t best = 0;
        if (t < chunks && mine.n) {
            const uint2 e = lists[(size_t)t * CAP];
            best = (uint64_t)e.y << 32 | e.x;
        }
        best = block_reduce(best, Most(), s.best);
        return give(place_id(best), 1.0);
    }
    // the row's weight from the chunks'
    const double part = t < chunks && mine.sum > 0.0 ? mine.sum * exp_neg(((double)mine.top - zmax) * q.inv) : 0.0;
    const double end = block_sums(part, s.sum);
    __syncthreads();
    if (t < chunks) s.ends[t] = end;
    if (t == ST - 1) s.d = end;
    __syncthreads();
    const double all = s.d;
    if (q.k == 0 && !q.p_on && !q.m_on) {
        // no filter: the chunk that the aim falls into (past the sum: the last with a weight)
        const double aim = u * all;
        if (t == 0) s.at[0] = s.at[1] = -1;
        __syncthreads();
        if (t < chunks && part > 0.0) {
            atomicMax(&s.at[1], t);
            if (s.ends[t] > aim && (t == 0 || s.ends[t - 1] <= aim)) atomicMax(&s.at[0], t);
        }
        __syncthreads();
        const int c = s.at[0] >= 0 ? s.at[0] : s.at[1];
        const double before = c ? s.ends[c - 1] : 0.0;
        draw<F32>(row, c * chunk_size, min((c + 1) * chunk_size, V), [&](float x, int) { return weight(x); },
                  [&](double) { return aim - before; }, s);
        return give(s.at[0], s.sum[0] / all);
    }

    // ---- few candidates
    // where candidate i of the row lies: chunk c with first[c] <= i < first[c + 1]
    bool listed = !over;
    int n = 0;
    if (listed) {
        const int fe = block_sums(mine.n, (int*)s.u);
        if (t < chunks) s.first[t + 1] = fe;
        if (t == 0) s.first[0] = 0;
        __syncthreads();
        auto candidate = [&](int i) {
            int lo = 0, hi = chunks;
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (s.first[mid] <= i) lo = mid;
                else hi = mid;
            }
            const uint2 e = lists[(size_t)lo * CAP + i - s.first[lo]];
            return (uint64_t)e.y << 32 | e.x;
        };
        float floor = -INF;
        if (!(q.k && q.p_on)) {
            if (q.m_on) floor = q.least(top, q.min_p);
            if (q.p_on) floor = fmaxf(floor, q.least(top, (1.0 - q.top_p) * all / V));
        }
        // top_k of several chunks' firsts: the parts up to the k-th
        int last = BINS;
        float low = INF;
        for (int i = t; i < n_all; i += ST) low = fminf(low, place_logit(candidate(i)));
        const Parts cut(top, block_reduce(low, Least(), s.f));
        if (q.k && n_all > 2 * q.k + 64) {
            for (int i = t; i < BINS; i += ST) s.cnt[i] = 0;
            __syncthreads();
            for (int i = t; i < n_all; i += ST) {
                const float x = place_logit(candidate(i));
                if (x >= floor) atomicAdd(&s.cnt[cut.of(x)], 1u);
            }
            __syncthreads();
            uint32_t before;
            last = part_of_count(s.cnt, (uint32_t)q.k, before, s.u, s.at);
            if (last < 0) last = BINS;
        }
        for (int i0 = 0; i0 < n_all; i0 += ST) {                 // in the order of the ids
            uint64_t e = 0;
            bool in = false;
            if (i0 + t < n_all) {
                e = candidate(i0 + t);
                const float x = place_logit(e);
                in = x >= floor && cut.of(x) <= last;
            }
            const int to = block_sums((int)in, (int*)s.u);
            if (in && n + to <= LIST) s.list[n + to - 1] = e;
            if (t == ST - 1) s.n = to;
            __syncthreads();
            n += s.n;
        }
        listed = n <= LIST;
    }
    uint64_t border = 0;                                         // the last kept place (before min_p)
    if (listed) {
        __syncthreads();
        for (int i = t; i < n; i += ST) s.sorted[i] = s.list[i];
        __syncthreads();
        sort_places(s.sorted, n);
        int keep = q.k ? min(n, q.k) : n;
        // a run of the order for each thread
        constexpr int RUN = LIST / ST;
        if (q.p_on) {
            const int run = (n + ST - 1) / ST, i0 = min(t * run, keep), i1 = min(i0 + run, keep);
            double w[RUN], own = 0.0;
#pragma unroll
            for (int i = 0; i < RUN; ++i) {
                w[i] = i0 + i < i1 ? weight(place_logit(s.sorted[i0 + i])) : 0.0;
                own += w[i];
            }
            const double e = block_sums(own, s.sum);
            __syncthreads();
            if (t == ST - 1) s.d = e;
            __syncthreads();
            const double want = q.top_p * (q.k ? s.d : all);
            double before = e - own;
            int m = 0;
#pragma unroll
            for (int i = 0; i < RUN; ++i) {
                if (i0 + i < i1 && (before < want || i0 + i == 0)) m = i0 + i + 1;
                before += w[i];
            }
            keep = block_reduce(m, Most(), (int*)s.u);
        }
        border = s.sorted[keep - 1];
        // the draw by id
        const int run = (n + ST - 1) / ST, i0 = min(t * run, n), i1 = min(i0 + run, n);
        double w[RUN], own = 0.0;
#pragma unroll
        for (int i = 0; i < RUN; ++i) {
            w[i] = 0.0;
            if (i0 + i < i1 && s.list[i0 + i] >= border) {
                w[i] = weight(place_logit(s.list[i0 + i]));
                if (w[i] < q.min_p) w[i] = 0.0;
            }
            own += w[i];
        }
        const double e = block_sums(own, s.sum);
        __syncthreads();
        if (t == ST - 1) s.d = e;
        if (t == 0) s.at[0] = 0x7FFFFFFF, s.at[1] = -1;
        __syncthreads();
        const double total = s.d, aim = u * total;
        double sum = e - own;
#pragma unroll
        for (int i = 0; i < RUN; ++i) {
            sum += w[i];
            if (w[i] > 0.0) {
                atomicMax(&s.at[1], i0 + i);
                if (sum > aim) atomicMin(&s.at[0], i0 + i);
            }
        }
        __syncthreads();
        const int at = s.at[0] != 0x7FFFFFFF ? s.at[0] : s.at[1];
        const uint64_t chosen = s.list[at];
        return give(place_id(chosen), weight(place_logit(chosen)) / total);
    }

    // ---- many: over the row again. Logits 2^-46 of the largest weight and less do not count.
    const float lowest = block_reduce(mine.low, Least(), s.f);
    const float floor = fmaxf(lowest, q.least(top, 1.0 / 70368744177664.0));
    const Parts parts(top, floor);
    auto mass = [&](float x) { return (uint64_t)__builtin_rint(weight(x) * ONE); };
    auto each = [&](auto f) {
        for (int i = t * 4; i < V; i += ST * 4) {
            float x[4];
            load_logits<F32>(row, i, V, x);
#pragma unroll
            for (int v = 0; v < 4; ++v)
                if (x[v] >= floor) f(x[v], i + v);
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
            const int b = parts.of(x);
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
                    if (parts.of(x) == b) s.sorted[atomicAdd(&s.n, 1)] = place_of(x, id);
                });
                __syncthreads();
                sort_places(s.sorted, m);
                constexpr int RUN = LIST / ST;
                const int run = (m + ST - 1) / ST, i0 = min(t * run, m), i1 = min(i0 + run, m);
                uint64_t w[RUN], own = 0;
#pragma unroll
                for (int i = 0; i < RUN; ++i) {
                    w[i] = i0 + i < i1 ? mass(place_logit(s.sorted[i0 + i])) : 0;
                    own += w[i];
                }
                uint64_t before = block_sums(own, s.best) - own, in = 0;
                int keep = 0;
#pragma unroll
                for (int i = 0; i < RUN; ++i) {
                    if (i0 + i < i1 && ((by_mass ? before : (uint64_t)(i0 + i)) < want || i0 + i == 0)) {
                        keep = i0 + i + 1;
                        in += w[i];
                    }
                    before += w[i];
                }
                keep = block_reduce(keep, Most(), (int*)s.u);
                kept = block_reduce(in, Plus(), s.best);
                return s.sorted[keep - 1];
            }
            // more than can be sorted: halve the range of keys until one is left
            uint32_t lo = ~0u, hi = 0;
            each([&](float x, int) {
                if (parts.of(x) == b) {
                    lo = min(lo, logit_key(x));
                    hi = max(hi, logit_key(x));
                }
            });
            lo = block_reduce(lo, Least(), s.u);
            hi = block_reduce(hi, Most(), s.u);
            auto above = [&](uint32_t key, bool masses) {
                uint64_t v = 0;
                each([&](float x, int) {
                    if (parts.of(x) == b && logit_key(x) > key) v += masses ? mass(x) : 1;
                });
                return block_reduce(v, Plus(), s.best);
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
            kept += (uint64_t)fmin((double)ties, s.d) * mass(key_logit(key));
            return (uint64_t)key << 32 | (uint32_t)~s.at[0];
        };
        // masses up to and with each part
        auto mass_end = [&](uint64_t& first) {
            first = s.mass[2 * t];
            return block_sums(first + s.mass[2 * t + 1], s.best);
        };
        uint64_t first, whole;
        const uint64_t ends = mass_end(first);
        __syncthreads();
        if (t == ST - 1) s.best[0] = ends;
        __syncthreads();
        whole = s.best[0];
        __syncthreads();
        if (q.k) {
            uint32_t before;
            const int b = part_of_count(s.cnt, (uint32_t)q.k, before, s.u, s.at);
            if (b >= 0) {
                if (t == b / 2) s.best[0] = ends - s.mass[b] - (b & 1 ? 0 : s.mass[b + 1]);
                __syncthreads();
                const uint64_t over_b = s.best[0];
                __syncthreads();
                uint64_t kept;
                border = border_in(b, q.k - before, false, kept);
                whole = over_b + kept;
            }
        }
        if (q.p_on) {
            const double x = __builtin_ceil(q.top_p * (double)whole);
            const uint64_t want = x < 1.0 ? 1 : (uint64_t)x;
            if (t == 0) s.at[0] = 0;
            __syncthreads();
            const uint64_t start = ends - first - s.mass[2 * t + 1];
            if (start < want && want <= ends) {
                const bool second = start + first < want;
                s.at[0] = 2 * t + second;
                s.best[0] = second ? start + first : start;
            }
            __syncthreads();
            const int b = s.at[0];
            const uint64_t before = s.best[0];
            __syncthreads();
            uint64_t kept;
            const uint64_t p = border_in(b, want - before, true, kept);
            border = Most()(border, p);
        }
    }
    draw<F32>(row, 0, V, [&](float x, int id) {
                  if (!(x >= floor) || place_of(x, id) < border) return 0.0;
                  const double w = weight(x);
                  return w >= q.min_p ? w : 0.0;
              }, [&](double sum) { return u * sum; }, s);
    give(s.at[0], s.sum[0] / s.d);
}

template <bool F32, int E>
__global__ void __launch_bounds__(ST) sample_chunk_kernel(SampleArgs a, int chunks, Chunk* info, uint2* lists) {
    __shared__ ChunkShared s;
    const long long n = (long long)a.B * chunks;
    for (long long i = blockIdx.x; i < n; i += gridDim.x) {
        sample_chunk<F32, E>(a, (int)(i / chunks), (int)(i % chunks), info + i, lists + i * CAP, s);
        __syncthreads();
    }
}
template <bool F32>
__global__ void __launch_bounds__(ST) sample_finish_kernel(SampleArgs a, int chunks, int chunk_size, const Chunk* info, const uint2* lists) {
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    const size_t i = (size_t)blockIdx.x * chunks;
    sample_finish<F32>(a, blockIdx.x, chunks, chunk_size, info + i, lists + i * CAP, *(RowShared*)smem);
}
// rows of one chunk
template <bool F32, int E>
__global__ void __launch_bounds__(ST) sample_row_kernel(SampleArgs a, Chunk* info, uint2* lists) {
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    const size_t i = blockIdx.x;
    sample_chunk<F32, E>(a, (int)i, 0, info + i, lists + i * CAP, *(ChunkShared*)smem);
    __syncthreads();
    sample_finish<F32>(a, (int)i, 1, ST * E, info + i, lists + i * CAP, *(RowShared*)smem);
}

// Logits of a thread of the chunk kernel: 4 where 16 would leave CUs without a chunk.
static int chunk_elems(int B, int V) { return (long long)B * ((V + ST * 16 - 1) / (ST * 16)) >= 256 || V > ST * 4 * MAX_CHUNKS ? 16 : 4; }
static int chunks_of(int B, int V) {
    const int e = chunk_elems(B, V);
    return (V + ST * e - 1) / (ST * e);
}
size_t sample_workspace_bytes(int B, int V) {
    const size_t n = (size_t)B * chunks_of(B, V);
    return (n * sizeof(Chunk) + 255) / 256 * 256 + n * CAP * sizeof(uint2);
}

template <bool F32>
static hipError_t launch(const SampleArgs& a, void* ws, hipStream_t stream) {
    const int e = chunk_elems(a.B, a.V), chunks = chunks_of(a.B, a.V);
    const size_t n = (size_t)a.B * chunks;
    Chunk* info = (Chunk*)ws;
    uint2* lists = (uint2*)((uint8_t*)ws + (n * sizeof(Chunk) + 255) / 256 * 256);
    static_assert(sizeof(RowShared) <= 163840 && sizeof(ChunkShared) <= sizeof(RowShared), "LDS");
    int dev = 0;
    hipError_t st = hipGetDevice(&dev);
    if (st != hipSuccess) return st;
    if (chunks == 1) {
        static std::atomic<uint64_t> done[2];
        const auto kernel = e == 16 ? sample_row_kernel<F32, 16> : sample_row_kernel<F32, 4>;
        st = allow_lds((const void*)kernel, sizeof(RowShared), dev, done[e == 16]);
        if (st != hipSuccess) return st;
        return launch_kernel(K_SAMPLE, stream, kernel, dim3((unsigned)a.B), dim3(ST), sizeof(RowShared), a, info, lists);
    }
    const auto kernel = e == 16 ? sample_chunk_kernel<F32, 16> : sample_chunk_kernel<F32, 4>;
    st = launch_kernel(K_SAMPLE, stream, kernel, dim3((unsigned)(n < (1u << 21) ? n : 1u << 21)), dim3(ST), 0, a, chunks, info, lists);
    if (st != hipSuccess) return st;
    static std::atomic<uint64_t> done{0};
    st = allow_lds((const void*)sample_finish_kernel<F32>, sizeof(RowShared), dev, done);
    if (st != hipSuccess) return st;
    return launch_kernel(K_SAMPLE, stream, sample_finish_kernel<F32>, dim3((unsigned)a.B), dim3(ST), sizeof(RowShared), a, chunks, ST * e,
                         (const Chunk*)info, (const uint2*)lists);
}
hipError_t launch_sample(const SampleArgs& a, bool f32, void* ws, hipStream_t stream) {
    return f32 ? launch<true>(a, ws, stream) : launch<false>(a, ws, stream);
}

}  // namespace moe
