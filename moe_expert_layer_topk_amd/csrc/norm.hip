// Row operators ahead of the 8-bit products: residual addition + RMS norm with
// optional 8-bit rows, and the int8 row quantizer on its own.
//
// norm:  v = x + res, r = 1 / sqrt(mean(v^2) + eps), y = v r w, all in fp32;
//        sum = bf16(v), y = bf16(y), codes from the fp32 y: every output is
//        rounded once.
// int8:  m = max(max|y|, 2^-100), scale = m / 127, code = rint(y (127 / m)).
//        The floor keeps 127 / m finite and needs no special case for a row of
//        zeros. Maxima are taken over the bit patterns of |y| as integers:
//        they order like the values, with infinity and NaN above all of them,
//        so a row holding either is found by the same reduction (scale NaN,
//        codes 0: an int8 code cannot carry it).
// e4m3:  per 128 columns, the power-of-two scale of moe_quant_act; a group
//        holding infinity or NaN gets the E8M0 NaN byte and codes 0.
//
// Bound by HBM: each input is read once and each output written once. A row
// stays in registers between the reductions and the stores (so the outputs
// may be the inputs' own memory): one pass, up to 16384 columns.
#include "moe_common.h"
#include "moe_kernels.h"

namespace moe {

struct NormArgs {
    const uint16_t* x;
    const uint16_t* res;      // may be null
    const float* w;           // may be null
    float eps;
    int rows, cols, qmode;
    uint16_t* sum;            // may be null
    uint16_t* y;              // may be null
    uint8_t* codes;
    void* scales;
};

constexpr float NORM_FLOOR = 0x1p-100f;

// two fp32 -> packed bf16, round to nearest even, NaN kept
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    typedef float f2 __attribute__((ext_vector_type(2)));
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2){a, b}, b2));
}
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o, 64));
    return v;
}

// Reductions over the TPR threads of a row (64: one wave; 256: the workgroup,
// through four LDS words that no other reduction of the kernel uses).
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* s) {
    v = wave_sum(v);
    if (TPR == 64) return v;
    if (lane_id() == 0) s[threadIdx.x / 64] = v;
    __syncthreads();
    return (s[0] + s[1]) + (s[2] + s[3]);
}
template <int TPR>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* s) {
    v = wave_max_u32(v);
    if (TPR == 64) return v;
    if (lane_id() == 0) s[threadIdx.x / 64] = v;
    __syncthreads();
    return max(max(s[0], s[1]), max(s[2], s[3]));
}

// int8 scale and multiplier of a row from the bits of its largest |value|
__device__ __forceinline__ void i8_scale(uint32_t amax_bits, float* scale, float* inv) {
    if (amax_bits >= 0x7F800000u) {
        *scale = __uint_as_float(0x7FC00000u);
        *inv = 0.f;
        return;
    }
    const float m = fmaxf(__uint_as_float(amax_bits), NORM_FLOOR);
    *scale = m / 127.0f;
    *inv = 127.0f / m;
}
// the low byte of the result is the code (inv = 0: a row that holds NaN or
// infinity, whose products here may be NaN)
__device__ __forceinline__ int i8_code(float v, float inv) {
    const float c = fminf(fmaxf(rintf(v * inv), -127.f), 127.f);
    return inv == 0.f ? 0 : (int)c;
}

// Rows of 16-byte vectors: TPR threads per row, NV vectors of 8 per thread.
template <int TPR, int NV, bool NORM>
__global__ void __launch_bounds__(256) norm_vec_kernel(NormArgs p) {
    __shared__ float s_sum[4];
    __shared__ uint32_t s_max[4];
    const int t = threadIdx.x % TPR;
    const long row = (long)blockIdx.x * (256 / TPR) + threadIdx.x / TPR;
    if (TPR == 64 && row >= p.rows) return;             // whole waves; no barrier follows
    const size_t base = (size_t)row * p.cols;
    const int nvec = p.cols / 8;
    i32x4 xr[NV], rr[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int i = t + j * TPR;
        xr[j] = rr[j] = i32x4{0, 0, 0, 0};
        if (i < nvec) {
            xr[j] = __builtin_nontemporal_load((const i32x4*)(p.x + base) + i);
            if (NORM && p.res) rr[j] = __builtin_nontemporal_load((const i32x4*)(p.res + base) + i);
        }
    }
    float v[NV][8];
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            v[j][2 * d] = __uint_as_float((uint32_t)xr[j][d] << 16);
            v[j][2 * d + 1] = __uint_as_float((uint32_t)xr[j][d] & 0xFFFF0000u);
            if (NORM) {
                v[j][2 * d] += __uint_as_float((uint32_t)rr[j][d] << 16);
                v[j][2 * d + 1] += __uint_as_float((uint32_t)rr[j][d] & 0xFFFF0000u);
                ss = fmaf(v[j][2 * d], v[j][2 * d], ss);
                ss = fmaf(v[j][2 * d + 1], v[j][2 * d + 1], ss);
            }
        }
    if (NORM) {
        const float r = rsqrtf(row_sum<TPR>(ss, s_sum) / (float)p.cols + p.eps);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int i = t + j * TPR;
            if (i >= nvec) continue;
            if (p.sum) {
                i32x4 o;
#pragma unroll
                for (int d = 0; d < 4; ++d) o[d] = (int)pack_bf16(v[j][2 * d], v[j][2 * d + 1]);
                *((i32x4*)(p.sum + base) + i) = o;
            }
            f32x4 w0 = {1, 1, 1, 1}, w1 = {1, 1, 1, 1};
            if (p.w) {
                w0 = *((const f32x4*)p.w + 2 * i);
                w1 = *((const f32x4*)p.w + 2 * i + 1);
            }
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                v[j][d] = v[j][d] * r * w0[d];
                v[j][4 + d] = v[j][4 + d] * r * w1[d];
            }
            if (p.y) {
                i32x4 o;
#pragma unroll
                for (int d = 0; d < 4; ++d) o[d] = (int)pack_bf16(v[j][2 * d], v[j][2 * d + 1]);
                *((i32x4*)(p.y + base) + i) = o;
            }
        }
    }
    if (p.qmode == MOE_Q_I8_ROW) {
        uint32_t am = 0;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int d = 0; d < 8; ++d) am = max(am, abs_bits(v[j][d]));   // (absent vectors hold zeros)
        float scale, inv;
        i8_scale(row_max<TPR>(am, s_max), &scale, &inv);
        if (t == 0) ((float*)p.scales)[row] = scale;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int i = t + j * TPR;
            if (i >= nvec) continue;
            uint32_t o[2] = {0, 0};
#pragma unroll
            for (int d = 0; d < 8; ++d) o[d / 4] |= (uint32_t)(i8_code(v[j][d], inv) & 0xFF) << (8 * (d % 4));
            *((uint2*)(p.codes + base) + i) = make_uint2(o[0], o[1]);
        }
    } else if (p.qmode == MOE_Q_FP8_G128_POW2) {
        // 16 consecutive lanes hold a group of 128 columns (cols % 128 == 0:
        // a group's vectors are all present or all absent)
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int i = t + j * TPR;
            uint32_t am = 0;
#pragma unroll
            for (int d = 0; d < 8; ++d) am = max(am, abs_bits(v[j][d]));
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) am = max(am, (uint32_t)__shfl_xor((int)am, o, 64));
            if (i >= nvec) continue;
            const bool bad = am >= 0x7F800000u;
            int s = bad ? 0 : pow2_exponent_448(__uint_as_float(am));
            s = s < -127 ? -127 : (s > 127 ? 127 : s);
            uint32_t o[2];
#pragma unroll
            for (int h = 0; h < 2; ++h)
                o[h] = f32x2_to_e4m3(ldexpf(v[j][4 * h], -s), ldexpf(v[j][4 * h + 1], -s)) |
                       (f32x2_to_e4m3(ldexpf(v[j][4 * h + 2], -s), ldexpf(v[j][4 * h + 3], -s)) << 16);
            *((uint2*)(p.codes + base) + i) = bad ? make_uint2(0, 0) : make_uint2(o[0], o[1]);
            if ((i & 15) == 0) ((uint8_t*)p.scales)[(size_t)row * (p.cols / 128) + i / 16] = (uint8_t)(bad ? 255 : s + 127);
        }
    }
}

// Rows whose length or address is no multiple of 16 bytes: one element per
// thread and step, a workgroup per row.
template <int NE, bool NORM>
__global__ void __launch_bounds__(256) norm_elem_kernel(NormArgs p) {
    __shared__ float s_sum[4];
    __shared__ uint32_t s_max[4];
    const int t = threadIdx.x;
    const size_t row = blockIdx.x, base = row * p.cols;
    float v[NE];
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < NE; ++j) {
        const int i = t + j * 256;
        v[j] = 0.f;
        if (i < p.cols) {
            v[j] = bf16_to_f32(p.x[base + i]);
            if (NORM && p.res) v[j] += bf16_to_f32(p.res[base + i]);
        }
        ss = fmaf(v[j], v[j], ss);
    }
    if (NORM) {
        const float r = rsqrtf(row_sum<256>(ss, s_sum) / (float)p.cols + p.eps);
#pragma unroll
        for (int j = 0; j < NE; ++j) {
            const int i = t + j * 256;
            if (i >= p.cols) continue;
            if (p.sum) p.sum[base + i] = (uint16_t)pack_bf16(v[j], 0.f);
            v[j] = v[j] * r * (p.w ? p.w[i] : 1.f);
            if (p.y) p.y[base + i] = (uint16_t)pack_bf16(v[j], 0.f);
        }
    }
    if (p.qmode == MOE_Q_I8_ROW) {
        uint32_t am = 0;
#pragma unroll
        for (int j = 0; j < NE; ++j) am = max(am, abs_bits(v[j]));
        float scale, inv;
        i8_scale(row_max<256>(am, s_max), &scale, &inv);
        if (t == 0) ((float*)p.scales)[row] = scale;
#pragma unroll
        for (int j = 0; j < NE; ++j) {
            const int i = t + j * 256;
            if (i < p.cols) p.codes[base + i] = (uint8_t)i8_code(v[j], inv);
        }
    }
}

int norm_max_cols() { return 16384; }

template <bool NORM>
static hipError_t launch_rows(const NormArgs& p, bool vec, int kid, hipStream_t stream) {
    const dim3 b(256);
    const unsigned R = (unsigned)p.rows;
    if (!vec) {
        if (p.cols <= 2048) MOE_LAUNCH(kid, stream, (norm_elem_kernel<8, NORM>), dim3(R), b, 0, stream, p);
        else MOE_LAUNCH(kid, stream, (norm_elem_kernel<64, NORM>), dim3(R), b, 0, stream, p);
        return hipGetLastError();
    }
    const int nvec = p.cols / 8;
    if (nvec <= 256 && p.rows >= 1024) {
        const dim3 g((R + 3) / 4);
        if (nvec <= 64) MOE_LAUNCH(kid, stream, (norm_vec_kernel<64, 1, NORM>), g, b, 0, stream, p);
        else if (nvec <= 128) MOE_LAUNCH(kid, stream, (norm_vec_kernel<64, 2, NORM>), g, b, 0, stream, p);
        else MOE_LAUNCH(kid, stream, (norm_vec_kernel<64, 4, NORM>), g, b, 0, stream, p);
    } else if (nvec <= 256) MOE_LAUNCH(kid, stream, (norm_vec_kernel<256, 1, NORM>), dim3(R), b, 0, stream, p);
    else if (nvec <= 512) MOE_LAUNCH(kid, stream, (norm_vec_kernel<256, 2, NORM>), dim3(R), b, 0, stream, p);
    else if (nvec <= 1024) MOE_LAUNCH(kid, stream, (norm_vec_kernel<256, 4, NORM>), dim3(R), b, 0, stream, p);
    else MOE_LAUNCH(kid, stream, (norm_vec_kernel<256, 8, NORM>), dim3(R), b, 0, stream, p);
    return hipGetLastError();
}

hipError_t launch_norm(const uint16_t* x, const uint16_t* res, const float* w, float eps, int rows, int cols, int qmode,
                       uint16_t* sum, uint16_t* y, uint8_t* codes, void* scales, bool vec, hipStream_t stream) {
    return launch_rows<true>(NormArgs{x, res, w, eps, rows, cols, qmode, sum, y, codes, scales}, vec, K_NORM, stream);
}

hipError_t launch_quant_rows(const uint16_t* x, int rows, int cols, int8_t* codes, float* scales, bool vec,
                             hipStream_t stream) {
    return launch_rows<false>(NormArgs{x, nullptr, nullptr, 0.f, rows, cols, MOE_Q_I8_ROW, nullptr, nullptr,
                                       (uint8_t*)codes, scales}, vec, K_QUANT_ROWS, stream);
}

}  // namespace moe
