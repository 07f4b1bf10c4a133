// Pieces that the tiled products share (gemm_i8.hip, gemm_fp8.hip): outputs and
// addends of a lane's columns, bounds-checked loads to LDS, launch helpers.
#pragma once
#include "moe_common.h"
#include "gemm_i8_plan.h"

#include <atomic>

namespace moe {

typedef int i32x16 __attribute__((ext_vector_type(16)));

static __device__ const float g_no_bias = -0.0f;               // (x + -0 is x for every x, zeros of both signs too)

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    typedef float f2 __attribute__((ext_vector_type(2)));
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2){a, b}, b2));
}
// silu(g) u; the hardware's base-2 exponential and reciprocal are within one
// step of fp32 each, and a sigmoid below 2^-126 (g below -87.3) is 0, less than
// 2^-126 |g u| of h (the correctly rounded division costs ten instructions more
// in an epilogue that no matrix instruction hides: gated 16384 x 512 x 2048
// 37.2 us with it)
__device__ __forceinline__ float glu_h(float g, float u) {
    return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.44269504088896341f)) * u;   // (g u first could overflow)
}

// Workgroup barrier that waits for the wave's LDS traffic only (the fence of
// __syncthreads() would drain the direct-to-LDS loads in flight).
static __device__ __forceinline__ void barrier_lds() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);                // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// NC adjacent output columns of one row, all of them inside it, in accesses of
// up to 16 bytes. !ANY: rows are whole 128-byte lines. Outputs are written once
// and not read here, so they are stored past the caches' order of use, and a
// launch does not end by writing back what its last tiles left in L2 (16384 x
// 2048 x 512 with the addend 39 -> 35 us, gated 16384 x 512 x 2048 31.4 ->
// 30.2, others the same).
// ANY: rows of any length that start at any element. Here such stores would
// write parts of lines to memory one by one (15007 x 1928 x 128 32 us, stored
// through L2 19; 10357 x 752 x 208 with the addend 11.2 and 10.2). Accesses
// that are not aligned to their size are split by the memory pipeline, which
// is still fewer than one for each value (5324 x 437 x 1408 with the addend
// 24.2 us one by one, 16.3 so; 4096 x 1999 x 2048 25.1 and 21.5).
template <int NC, bool F32, bool ANY = false>
struct Cols {
    typedef uint32_t word __attribute__((ext_vector_type(NC == 2 && !F32 ? 1 : NC * (F32 ? 4 : 2) / 4 < 4 ? NC * (F32 ? 4 : 2) / 4 : 4)));
    typedef word place __attribute__((aligned(ANY ? (F32 ? 4 : 2) : sizeof(word))));
    static constexpr int W = sizeof(word) / 4;                   // dwords of an access
    static constexpr int NW = NC * (F32 ? 4 : 2) / (4 * W);      // accesses
    word w[NW];
    __device__ __forceinline__ void load(const void* p, size_t o) {
        const place* q = (const place*)((const uint8_t*)p + o * (F32 ? 4 : 2));
#pragma unroll
        for (int h = 0; h < NW; ++h) w[h] = q[h];
    }
    __device__ __forceinline__ void add_to(float (&v)[NC]) const {
#pragma clang fp contract(off)
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            if (F32) v[n] += __uint_as_float(w[n / W][n % W]);
            else {
                const uint32_t d = w[n / 2 / W][n / 2 % W];
                v[n] += __uint_as_float(n & 1 ? d & 0xFFFF0000u : d << 16);
            }
        }
    }
    __device__ __forceinline__ static void store(void* p, size_t o, const float (&v)[NC]) {
        Cols c;
#pragma unroll
        for (int d = 0; d < NW * W; ++d) {
            if (F32) c.w[d / W][d % W] = __float_as_uint(v[d]);
            else c.w[d / W][d % W] = pack_bf16(v[2 * d], v[2 * d + 1]);
        }
        place* q = (place*)((uint8_t*)p + o * (F32 ? 4 : 2));
#pragma unroll
        for (int h = 0; h < NW; ++h) {
            if (ANY) q[h] = c.w[h];
            else __builtin_nontemporal_store(c.w[h], q + h);
        }
    }
};
// the columns of them that exist, one by one: addends, outputs. Up to four
// columns load without a branch (past the row's end its last addend), so that
// no load waits in a branch of its own (10357 x 755 x 208 with the addend 18.5
// -> 14.5 us); with eight the addresses would take registers from the step loop
// of a 256 x 256 tile (8192 x 8191 x 8192 408 -> 452 us).
template <int NC, bool F32, typename Args>
__device__ __forceinline__ void add_each(const Args& p, int row, int col, float (&v)[NC]) {
#pragma clang fp contract(off)
    const size_t o = (size_t)min(row, p.M - 1) * p.N;
#pragma unroll
    for (int n = 0; n < NC; ++n) {
        if (NC > 4 && col + n >= p.N) continue;
        const size_t i = o + min(col + n, p.N - 1);
        v[n] += F32 ? ((const float*)p.add)[i] : bf16_to_f32(((const uint16_t*)p.add)[i]);
    }
}
template <int NC, bool F32, typename Args>
__device__ __forceinline__ void store_each(const Args& p, int row, int col, const float (&v)[NC]) {
    const size_t o = (size_t)row * p.N + col;
#pragma unroll
    for (int n = 0; n < NC; ++n) {
        if (col + n >= p.N) continue;
        if (F32) ((float*)p.out)[o + n] = v[n];
        else ((uint16_t*)p.out)[o + n] = (uint16_t)pack_bf16(v[n], 0.f);
    }
}

template <int V>
struct IC {
    static constexpr int value = V;
};

// Rows of an operand from a tile's first one on, as a buffer: accesses past its
// end return nothing. Each K position has a descriptor of its own, based there
// and holding the records that are left, and no scalar offset. The check that
// drops an access then compares the lane's offset alone, which every
// description of it agrees on; of a scalar offset the compiler's intrinsic says
// that it is left out of the check, the MI300 instruction set that it is taken
// off the record count, and neither what happens where it exceeds that count.
struct Operand {
    const uint8_t* p;
    int bytes;
    __device__ __forceinline__ void set(const void* first, size_t n) {
        p = (const uint8_t*)first;
        bytes = records(n);
    }
    // 16 bytes a lane, from lane offset o at K position k, to dst + 16 lane
    __device__ __forceinline__ void load_lds(uint8_t* dst, uint32_t o, int k) const {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            __builtin_amdgcn_make_buffer_rsrc((void*)(p + k), 0, records_from(bytes, k), 0x00027000),
            (__attribute__((address_space(3))) void*)dst, 16, (int)o, 0, 0, 0);
    }
};

// Raises a kernel's dynamic LDS limit, once for each device (the call costs
// more than the launch's other checks together; racing callers repeat it).
static hipError_t allow_lds(const void* kernel, int bytes, int dev, std::atomic<uint64_t>& done) {
    const uint64_t bit = 1ull << (dev & 63);
    if (dev < 64 && (done.load(std::memory_order_relaxed) & bit)) return hipSuccess;
    const hipError_t e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == hipSuccess && dev < 64) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

static bool whole_lines(const void* p, int cols, int size) { return ((uintptr_t)p | (uintptr_t)cols * size) % 128 == 0; }

}  // namespace moe
