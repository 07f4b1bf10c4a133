// One token per row of logits: temperature, top-k, top-p, min-p and the draw
// from a given random number.
//
// The kept tokens are a prefix of the order (logit falling, id rising), so they
// are described by a border: every key above `key`, and the first `ties` tokens
// by id of those that have it. Keys are the logits' bits in an order-preserving
// form; weights are integers (2^42 exp(z - max z), rounded), so that sums are
// exact and have no order.
#include "moe_common.h"
#include "moe_kernels.h"

namespace moe {

int sample_max_cols() { return MOE_SAMPLE_MAX_COLS; }

constexpr int SAMPLE_THREADS = 1024;
constexpr double SAMPLE_ONE = 4398046511104.0;                   // 2^42: the sum of 2^20 weights stays below 2^63

// larger float, larger key; zeros of both signs are one value; -inf 0x007FFFFF, NaN of either sign outside (-inf, +inf)
__device__ __forceinline__ uint32_t logit_key(float f) {
    const uint32_t b = __float_as_uint(f + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_logit(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k); }
constexpr uint32_t KEY_NONE = 0x007FFFFFu, KEY_INF = 0xFF800000u;

template <bool F32>
struct Logits {
    const void* row;
    __device__ __forceinline__ uint32_t key(int i) const {
        return logit_key(F32 ? ((const float*)row)[i] : bf16_to_f32(((const uint16_t*)row)[i]));
    }
};

template <typename T, typename F>
__device__ __forceinline__ T block_reduce(T v, F f, T* s) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = f(v, (T)__shfl_xor(v, o, 64));
    __syncthreads();
    if (lane_id() == 0) s[threadIdx.x / 64] = v;
    __syncthreads();
    v = s[0];
    for (int i = 1; i < SAMPLE_THREADS / 64; ++i) v = f(v, s[i]);
    return v;
}
// sum over the threads before this one
__device__ __forceinline__ uint64_t block_before(uint64_t v, uint64_t* s) {
    uint64_t x = v;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const uint64_t y = __shfl_up(x, o, 64);
        if (lane_id() >= o) x += y;
    }
    __syncthreads();
    if (lane_id() == 63) s[threadIdx.x / 64] = x;
    __syncthreads();
    for (int i = 0; i < (int)threadIdx.x / 64; ++i) x += s[i];
    return x - v;
}

template <bool F32>
__global__ void __launch_bounds__(SAMPLE_THREADS) sample_kernel(SampleArgs a) {
    __shared__ uint64_t s_sum[SAMPLE_THREADS / 64];
    const int r = blockIdx.x, t = threadIdx.x, V = a.V;
    const Logits<F32> L{(const uint8_t*)a.logits + (size_t)r * a.stride * (F32 ? 4 : 2)};
    auto plus = [](uint64_t x, uint64_t y) { return x + y; };
    auto most = [](uint64_t x, uint64_t y) { return x > y ? x : y; };
    const double u = a.u[r], temp = a.temperature ? a.temperature[r] : 1.0, min_p = a.min_p ? a.min_p[r] : 0.0;
    const double top_p = a.top_p ? a.top_p[r] : 1.0;
    int top_k = a.top_k ? a.top_k[r] : 0;
    bool bad = !(u >= 0.0 && u <= 1.0) || !(temp >= 0.0) || !(min_p <= 1.0) || top_p != top_p;

    uint64_t top = 0;                                            // the largest key; NaN first
    uint64_t n = 0;                                              // tokens that are not masked
    for (int i = t; i < V; i += SAMPLE_THREADS) {
        const uint32_t k = L.key(i);
        top = most(top, k >= KEY_INF || k < KEY_NONE ? 1ull << 32 : k);
        n += k != KEY_NONE;
    }
    top = block_reduce(top, most, s_sum);
    n = block_reduce(n, plus, s_sum);
    bad |= top >= KEY_INF || top == KEY_NONE;
    if (bad) {
        if (t == 0) {
            a.ids[r] = -1;
            if (a.p) a.p[r] = 0.f;
            if (a.err) atomicAdd(a.err, 1);
        }
        return;
    }
    const double zmax = key_logit((uint32_t)top), inv = temp > 0.0 ? 1.0 / temp : 0.0;
    if (temp == 0.0) top_k = 1;
    auto weight = [&](uint32_t k) { return k == KEY_NONE ? 0.0 : exp(((double)key_logit(k) - zmax) * inv); };
    auto mass = [&](uint32_t k) { return (uint64_t)rint(weight(k) * SAMPLE_ONE); };

    // tokens above key k, and their mass
    auto above = [&](uint32_t k, bool masses) {
        uint64_t v = 0;
        for (int i = t; i < V; i += SAMPLE_THREADS) {
            const uint32_t x = L.key(i);
            if (x > k) v += masses ? mass(x) : 1;
        }
        return block_reduce(v, plus, s_sum);
    };
    // the smallest key with fewer than `want` above it
    auto border = [&](uint64_t want, bool masses, uint32_t lo) {
        uint32_t hi = (uint32_t)top;                             // nothing is above top
        while (lo < hi) {
            const uint32_t mid = lo + (hi - lo) / 2;
            if (above(mid, masses) < want) hi = mid;
            else lo = mid + 1;
        }
        return lo;
    };
    uint32_t key = KEY_NONE + 1;                                 // everything unmasked
    uint64_t ties = ~0ull;
    if (top_k > 0 && (uint64_t)top_k < n) {
        key = border(top_k, false, key);
        ties = top_k - above(key, false);
    }
    if (top_p < 1.0 && temp > 0.0) {
        uint64_t all = above(key, true), at = 0;
        for (int i = t; i < V; i += SAMPLE_THREADS) at += L.key(i) == key;
        at = block_reduce(at, plus, s_sum);
        all += (ties < at ? ties : at) * mass(key);
        const double want = top_p > 0.0 ? ceil(top_p * (double)all) : 1.0;
        const uint64_t w = want < 1.0 ? 1 : (uint64_t)want;
        const uint32_t k2 = border(w, true, key);
        const uint64_t m = mass(k2), more = m ? (w - above(k2, true) + m - 1) / m : ~0ull;
        ties = k2 > key || more < ties ? more : ties;
        key = k2;
    }

    // the draw: thread t has a run of ids
    const int run = (V + SAMPLE_THREADS - 1) / SAMPLE_THREADS, i0 = min(t * run, V), i1 = min(i0 + run, V);
    uint64_t at = 0;
    for (int i = i0; i < i1; ++i) at += L.key(i) == key;
    const uint64_t before = block_before(at, s_sum);
    auto kept = [&](uint32_t k, uint64_t& rank) {
        const bool in = k > key || (k == key && rank < ties);
        rank += k == key;
        return in && weight(k) >= min_p ? mass(k) : 0;
    };
    uint64_t rank = before, own = 0;
    for (int i = i0; i < i1; ++i) own += kept(L.key(i), rank);
    const uint64_t start = block_before(own, s_sum), all = block_reduce(own, plus, s_sum);
    uint64_t aim = (uint64_t)(u * (double)all);
    if (aim >= all) aim = all - 1;
    if (start <= aim && aim < start + own) {
        rank = before;
        uint64_t sum = start;
        for (int i = i0; i < i1; ++i) {
            const uint32_t k = L.key(i);
            sum += kept(k, rank);
            if (sum > aim) {
                a.ids[r] = i;
                if (a.p) a.p[r] = (float)(weight(k) * SAMPLE_ONE / (double)all);
                break;
            }
        }
    }
}

size_t sample_workspace_bytes(int B, int V) { return 0; }

hipError_t launch_sample(const SampleArgs& a, bool f32, void* ws, hipStream_t stream) {
    return f32 ? launch_kernel(K_SAMPLE, stream, sample_kernel<true>, dim3((unsigned)a.B), dim3(SAMPLE_THREADS), 0, a)
               : launch_kernel(K_SAMPLE, stream, sample_kernel<false>, dim3((unsigned)a.B), dim3(SAMPLE_THREADS), 0, a);
}

}  // namespace moe
