// Row operators ahead of the 8-bit products: residual addition + RMS norm with
// optional 8-bit rows, the int8 row quantizer on its own, and the way back from
// 8-bit rows to bf16.
//
// norm:  v = x + res (fp32), r = 1 / sqrt(mean(v^2) + eps), y = v r w;
//        sum = bf16(v), y = bf16(y), codes from the unrounded y.
// int8:  m = max(max|y|, 2^-100), scale = m / 127, code = rint(127 y / m).
//        The floor keeps 127 / m finite and needs no special case for a row of
//        zeros.
// e4m3:  per 128 columns, the power-of-two scale of moe_quant_act.
//
// The squares' sum, r and y are fp64, and so is every code that could depend on
// it: a code changes where its argument passes a border, so an error of 2^-24
// would change some ten codes in a million. int8 codes are formed in fp32
// first, and again in fp64 where their argument lies near a border, ties to the
// even code. e4m3 codes
// come from y rounded to odd, which a second rounding to fewer bits leaves
// correctly rounded.
// Rows of int8 read from bf16 (quant_rows): with 8-bit mantissas X and M and x
// j binades below m, 127 x / m = 127 X / (M 2^j) is a border exactly, or at
// least 2^-16 of itself away from it (the least distance is 1 / 502 at j = 1,
// 1 / 64768 at j = 8; from j = 9 on it is below 1 / 2). That is 2^8 half steps of fp32,
// so rounding the fp64 product to fp32 first puts the exact ties back on the
// border and moves nothing else across one.
// A row (e4m3: a group) that holds NaN or infinity gets codes 0 and a NaN scale
// (e4m3: the E8M0 NaN byte): an 8-bit code cannot carry them.
//
// Bound by HBM: each input is read once and each output written once. A row
// stays in registers between the reductions and the stores (so the outputs
// may be the inputs' own memory): one pass, up to 16384 columns. 16384 x 2048
// with the residual, both bf16 outputs and int8 rows: 55 us, 5.5 TB/s (a 1 GiB
// copy on the same card: 5.1; with fp32 arithmetic 51 us); without 8-bit rows
// 45 us. Reading a row twice would have added a third to its bytes.
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
    double inv_cols;
};

constexpr double NORM_FLOOR = 0x1p-100;

// two fp32 -> packed bf16, round to nearest even, NaN kept
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    typedef float f2 __attribute__((ext_vector_type(2)));
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2){a, b}, b2));
}

// The largest |value| seen, and the largest upper word of an |value| as an
// integer: at or above 0x7FF00000 where one was NaN or infinite (the maximum
// of two floating-point values leaves a NaN out).
struct Peak {
    double m = 0.0;
    uint32_t hi = 0;
    __device__ __forceinline__ void add(double u) {
        m = fmax(m, fabs(u));
        hi = max(hi, (uint32_t)(__builtin_bit_cast(uint64_t, u) >> 32) & 0x7FFFFFFFu);
    }
};

// Reductions of a wave by lane moves in the vector unit (a step through LDS
// waits some 100 clocks: 16384 x 512 with int8 rows 19.0 us, these 17.8; int8
// rows alone 6887 x 1200 10.6 and 9.7).
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_sum_step(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, ROWS, 0xF, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, ROWS, 0xF, false);
    return v + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double wave_sum_f64(double v) {
    v = dpp_sum_step<0x111, 0xF>(v);   // row_shr:1
    v = dpp_sum_step<0x112, 0xF>(v);   // row_shr:2
    v = dpp_sum_step<0x114, 0xF>(v);   // row_shr:4
    v = dpp_sum_step<0x118, 0xF>(v);   // row_shr:8  -> lane 15 of each row holds the row's sum
    v = dpp_sum_step<0x142, 0xA>(v);   // row_bcast:15 into rows 1 and 3
    v = dpp_sum_step<0x143, 0xC>(v);   // row_bcast:31 into rows 2 and 3 -> lane 63 holds the sum
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, 63);
    return __builtin_bit_cast(double, (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), 63) << 32 | lo);
}
// largest of 16 consecutive lanes (a group of 128 columns), in each of them
__device__ __forceinline__ uint32_t group_max_u32(uint32_t v) {
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));     // quad_perm [1,0,3,2]
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));     // quad_perm [2,3,0,1]
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x124, 0xF, 0xF, true));    // row_ror:4
    return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x128, 0xF, 0xF, true)); // row_ror:8
}

// Sum over the TPR threads of a row (64: one wave; 256: the workgroup, through
// four LDS words that no other reduction of the kernel uses).
template <int TPR>
__device__ __forceinline__ double row_sum(double v, double* s) {
    v = wave_sum_f64(v);
    if (TPR == 64) return v;
    if (lane_id() == 0) s[threadIdx.x / 64] = v;
    __syncthreads();
    return (s[0] + s[1]) + (s[2] + s[3]);
}

// 1 / sqrt(a) and 1 / a to a few 2^-52: the hardware's estimates (2^-24 and
// better) and two Newton steps
__device__ __forceinline__ double rsqrt_f64(double a) {
    double r = __builtin_amdgcn_rsq(a);
#pragma unroll
    for (int i = 0; i < 2; ++i) r = fma(0.5 * r, fma(-a * r, r, 1.0), r);
    return a == __builtin_inf() ? 0.0 : r;
}
__device__ __forceinline__ double rcp_f64(double a) {
    double r = __builtin_amdgcn_rcp(a);
#pragma unroll
    for (int i = 0; i < 2; ++i) r = fma(r, fma(-a, r, 1.0), r);
    return r;
}

// int8 scale of a row and the multiplier of its v w values, from the threads'
// peaks of |v w| and the row's r (both positive: rounding keeps their order).
// mul 0: the row holds NaN or infinity, or a value past fp32. quick: mul in
// fp32, or 0 where a product of it could leave fp32's normal range.
template <int TPR>
__device__ __forceinline__ void i8_scale(Peak p, double r, double* s_max, uint32_t* s_bad, float* scale, double* mul, float* quick) {
    uint32_t bad = __ballot(p.hi >= 0x7FF00000u) != 0;
    // (of positive doubles the bits keep the order)
    p.m = __builtin_bit_cast(double, wave_max_u64_dpp(__builtin_bit_cast(uint64_t, p.m)));
    if (TPR != 64) {
        if (lane_id() == 0) {
            s_max[threadIdx.x / 64] = p.m;
            s_bad[threadIdx.x / 64] = bad;
        }
        __syncthreads();
        p.m = fmax(fmax(s_max[0], s_max[1]), fmax(s_max[2], s_max[3]));
        bad = s_bad[0] | s_bad[1] | s_bad[2] | s_bad[3];
    }
    const double m = fmax(p.m * r, NORM_FLOOR);
    // (r is 0 or NaN only where a value of the row, or the sum of its squares, was not finite)
    if (bad || !(r > 0.0) || m > 3.4028234663852886e38) {
        *scale = __uint_as_float(0x7FC00000u);
        *mul = 0.0;
        *quick = 0.f;
        return;
    }
    *scale = (float)(m * (1.0 / 127.0));
    *mul = r * (127.0 * rcp_f64(m));
    *quick = p.m >= 0x1p-100 && p.m <= 0x1p+120 ? (float)*mul : 0.f;
}
// the low byte of the result is the code. u * mul is within 2^-43 of 127 y / m
// (|.| <= 127); in rows without weights, and with weights that are powers of
// two, r drops out of that and it can be a border exactly, so it is rounded to a
// multiple of 2^-40 first, which puts those ties back (adding 3/2 2^12, whose
// step that is, and taking it off again).
template <bool NORM>
__device__ __forceinline__ int i8_code(double u, double mul) {
    if (mul == 0.0) return 0;
    return NORM ? (int)rint((u * mul + 0x1.8p12) - 0x1.8p12) : (int)rintf((float)(u * mul));
}
// y rounded to odd at 20 mantissa bits: the upper word, its last bit set where
// the lower is not zero (exact in fp32 down to its smallest normal value)
__device__ __forceinline__ float to_odd(double y) {
    const uint64_t b = __builtin_bit_cast(uint64_t, y);
    const uint32_t hi = (uint32_t)(b >> 32) | ((uint32_t)b != 0 ? 1u : 0u);
    return (float)__builtin_bit_cast(double, (uint64_t)hi << 32);
}

// Rows of 16-byte vectors: TPR threads per row, NV vectors of 8 per thread.
// SHIFT: the rows' length is no multiple of 8. Vectors then lie on the
// tensors' own 16-byte grid (all tensors start on it, so a row is shifted
// alike in each of them); the first and the last of a row may hold elements of
// the rows beside it, which count as zeros and are not written, and the last
// of the whole tensor may end past it, where it is read one by one.
template <int TPR, int NV, bool NORM, bool SHIFT>
__global__ void __launch_bounds__(256) norm_vec_kernel(NormArgs p) {
    __shared__ double s_sum[4], s_max[4];
    __shared__ uint32_t s_bad[4];
    const int t = threadIdx.x % TPR;
    const long row = (long)blockIdx.x * (256 / TPR) + threadIdx.x / TPR;
    if (TPR == 64 && row >= p.rows) return;             // whole waves; no barrier follows
    const int off = SHIFT ? (int)(((size_t)row * p.cols) & 7) : 0;
    const size_t base = (size_t)row * p.cols - off;     // of the row's first vector
    const int end = off + p.cols;                       // the row's elements: [off, end) from there
    const int nvec = SHIFT ? (end + 7) / 8 : p.cols / 8;
    // vector i holds elements of this row only
    auto whole = [&](int i) { return !SHIFT || (8 * i >= off && 8 * i + 8 <= end); };
    auto load = [&](const uint16_t* src, int i) __attribute__((always_inline)) {
        if (SHIFT && base + 8 * i + 8 > (size_t)p.rows * p.cols) {
            i32x4 x = {0, 0, 0, 0};                     // (past the end: its last value, dropped below)
#pragma unroll
            for (int d = 0; d < 8; ++d)
                x[d / 2] |= (int)((uint32_t)src[min(base + 8 * i + d, (size_t)p.rows * p.cols - 1)] << (16 * (d & 1)));
            return x;
        }
        return __builtin_nontemporal_load((const i32x4*)(src + base) + i);
    };
    auto store8 = [&](uint16_t* dst, int i, const i32x4& o) __attribute__((always_inline)) {
        if (whole(i)) *((i32x4*)(dst + base) + i) = o;
        else
            for (int d = 0; d < 8; ++d)
                if (8 * i + d >= off && 8 * i + d < end) dst[base + 8 * i + d] = (uint16_t)((uint32_t)o[d / 2] >> (16 * (d & 1)));
    };
    i32x4 xr[NV], rr[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int i = t + j * TPR;
        xr[j] = rr[j] = i32x4{0, 0, 0, 0};
        if (i < nvec) {
            xr[j] = load(p.x, i);
            if (NORM && p.res) rr[j] = load(p.res, i);
        }
    }
    float v[NV][8];                                     // (absent vectors hold zeros)
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            v[j][2 * d] = __uint_as_float((uint32_t)xr[j][d] << 16);
            v[j][2 * d + 1] = __uint_as_float((uint32_t)xr[j][d] & 0xFFFF0000u);
            if (NORM) {
                v[j][2 * d] += __uint_as_float((uint32_t)rr[j][d] << 16);
                v[j][2 * d + 1] += __uint_as_float((uint32_t)rr[j][d] & 0xFFFF0000u);
            }
        }
    if (SHIFT) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int d = 0; d < 8; ++d) {
                const int e = 8 * (t + j * TPR) + d;
                if (e < off || e >= end) v[j][d] = 0.f;
            }
    }
    double r = 1.0;
    if (NORM) {
        double ss = 0.0;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int d = 0; d < 8; ++d) ss = fma((double)v[j][d], (double)v[j][d], ss);
        r = rsqrt_f64(fma(row_sum<TPR>(ss, s_sum), p.inv_cols, (double)p.eps));
    }
    // the weights of vector j
    auto weights = [&](int j, float (&w)[8]) __attribute__((always_inline)) {
        int i = min(t + j * TPR, nvec - 1);
        asm volatile("" : "+v"(i));                     // (loaded again where they are needed again)
        if (SHIFT && p.cols < 8) {
#pragma unroll
            for (int d = 0; d < 8; ++d) w[d] = p.w[min(max(8 * i + d - off, 0), p.cols - 1)];
            return;
        }
        // vectors that reach past the row: the eight weights at its end,
        // rotated into place (loads in a branch of their own would wait there)
        const int at = 8 * i - off, in = SHIFT ? min(max(at, 0), p.cols - 8) : at;
        typedef f32x4 f32x4_dword __attribute__((aligned(4)));       // (vector loads need whole dwords only)
        f32x4 w0 = *(const f32x4_dword*)(p.w + in), w1 = *(const f32x4_dword*)(p.w + in + 4);
        if (SHIFT && __ballot(at != in)) {
            const int by = at - in;
            if (by & 1) {
                const float x = w0[0];
                w0 = f32x4{w0[1], w0[2], w0[3], w1[0]};
                w1 = f32x4{w1[1], w1[2], w1[3], x};
            }
            if (by & 2) {
                const f32x4 x = w0;
                w0 = f32x4{w0[2], w0[3], w1[0], w1[1]};
                w1 = f32x4{w1[2], w1[3], x[0], x[1]};
            }
            if (by & 4) {
                const f32x4 x = w0;
                w0 = w1;
                w1 = x;
            }
        }
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            w[d] = w0[d];
            w[4 + d] = w1[d];
        }
    };
    // v w of vector j (exact: two 24-bit factors), formed again where it is
    // needed; y is that times r
    auto vw_of = [&](int j, double (&u)[8]) __attribute__((always_inline)) {
#pragma unroll
        for (int d = 0; d < 8; ++d) {
            asm volatile("" : "+v"(v[j][d]));           // (converted again, not kept as a double)
            u[d] = (double)v[j][d];
        }
        if (NORM && p.w) {
            float w[8];
            weights(j, w);
#pragma unroll
            for (int d = 0; d < 8; ++d) u[d] *= (double)w[d];
        }
    };
    Peak peak;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        if (j * TPR >= nvec) break;
        const int i = t + j * TPR;
        double u[8];
        vw_of(j, u);
        if (NORM && i < nvec) {
            if (p.sum) {
                i32x4 o;
#pragma unroll
                for (int d = 0; d < 4; ++d) o[d] = (int)pack_bf16(v[j][2 * d], v[j][2 * d + 1]);
                store8(p.sum, i, o);
            }
            if (p.y) {
                i32x4 o;
#pragma unroll
                for (int d = 0; d < 4; ++d) o[d] = (int)pack_bf16((float)(u[2 * d] * r), (float)(u[2 * d + 1] * r));
                store8(p.y, i, o);
            }
        }
        if (p.qmode == MOE_Q_I8_ROW) {
#pragma unroll
            for (int d = 0; d < 8; ++d) peak.add(u[d]);
        } else if (NORM && !SHIFT && p.qmode == MOE_Q_FP8_G128_POW2) {
            // 16 consecutive lanes hold a group of 128 columns (cols % 128 ==
            // 0: a group's vectors are all present or all absent)
            float z[8];
            uint32_t gm = 0;
#pragma unroll
            for (int d = 0; d < 8; ++d) {
                z[d] = to_odd(u[d] * r);
                gm = max(gm, __float_as_uint(z[d]) & 0x7FFFFFFFu);
            }
            gm = group_max_u32(gm);
            if (i >= nvec) continue;
            const bool bad = gm >= 0x7F800000u;
            int s = bad ? 0 : pow2_exponent_448(__uint_as_float(gm));
            s = s < -127 ? -127 : (s > 127 ? 127 : s);
            int down = s;
            // Values below fp32's normal ones can have a code in such groups: again
            // from 2^24 y. (The wave's vectors, and the factor formed here: a branch
            // of single lanes took 26 registers more, 16384 x 2048 55 -> 58 us.)
            if (__ballot(s <= -116)) {
                double up = s <= -116 ? 0x1p24 : 1.0;
                asm volatile("" : "+v"(up));
                up *= r;
#pragma unroll
                for (int d = 0; d < 8; ++d) z[d] = to_odd(u[d] * up);
                down = s <= -116 ? s + 24 : s;
            }
            uint32_t o[2];
#pragma unroll
            for (int h = 0; h < 2; ++h)
                o[h] = f32x2_to_e4m3(ldexpf(z[4 * h], -down), ldexpf(z[4 * h + 1], -down)) |
                       (f32x2_to_e4m3(ldexpf(z[4 * h + 2], -down), ldexpf(z[4 * h + 3], -down)) << 16);
            *((uint2*)(p.codes + base) + i) = bad ? make_uint2(0, 0) : make_uint2(o[0], o[1]);
            if ((i & 15) == 0) ((uint8_t*)p.scales)[(size_t)row * (p.cols / 128) + i / 16] = (uint8_t)(bad ? 255 : s + 127);
        }
    }
    if (p.qmode == MOE_Q_I8_ROW) {
        float scale;
        double mul;                                     // 127 r / m: what v w is multiplied by
        float quick;
        i8_scale<TPR>(peak, r, s_max, s_bad, &scale, &mul, &quick);
        if (t == 0) ((float*)p.scales)[row] = scale;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (j * TPR >= nvec) break;
            const int i = t + j * TPR;
            // In fp32 first: z is within 3 2^-24 of its value, so the code is
            // certain where z is 2^-22 of itself and more away from a border
            // (z + 3 2^22 is rounded to an integer, in its low byte).
            float w[8];
            if (NORM && p.w) weights(j, w);
            bool redo = quick == 0.f;
            uint32_t f[8], o[2];
#pragma unroll
            for (int d = 0; d < 8; ++d) {
                const float z = (NORM && p.w ? v[j][d] * w[d] : v[j][d]) * quick, n = z + 12582912.f;
                redo |= fmaf(fabsf(z), 0x1p-22f, fabsf(z - (n - 12582912.f))) > 0.5f;
                f[d] = __float_as_uint(n);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)                 // (byte 0 of each)
                o[h] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(f[4 * h + 3], f[4 * h + 2], 0x0C0C0400u),
                                             __builtin_amdgcn_perm(f[4 * h + 1], f[4 * h], 0x0C0C0400u), 0x05040100u);
            if (__ballot(redo)) {                       // the wave's vectors again, in fp64
                double u[8];
                vw_of(j, u);
                o[0] = o[1] = 0;
#pragma unroll
                for (int d = 0; d < 8; ++d) o[d / 4] |= (uint32_t)(i8_code<NORM>(u[d], mul) & 0xFF) << (8 * (d % 4));
            }
            if (i >= nvec) continue;
            if (whole(i)) *((uint2*)(p.codes + base) + i) = make_uint2(o[0], o[1]);
            else
                for (int d = 0; d < 8; ++d)
                    if (8 * i + d >= off && 8 * i + d < end) p.codes[base + 8 * i + d] = (uint8_t)(o[d / 4] >> (8 * (d % 4)));
        }
    }
}

// Rows whose address is no multiple of 16 bytes (or that the vector kernel has
// no room for): one element per thread and step, a workgroup per row.
template <int NE, bool NORM>
__global__ void __launch_bounds__(256) norm_elem_kernel(NormArgs p) {
    __shared__ double s_sum[4], s_max[4];
    __shared__ uint32_t s_bad[4];
    const int t = threadIdx.x;
    const size_t row = blockIdx.x, base = row * p.cols;
    float v[NE];
    double r = 1.0, ss = 0.0;
#pragma unroll
    for (int j = 0; j < NE; ++j) {
        const int i = t + j * 256;
        v[j] = 0.f;
        if (i < p.cols) {
            v[j] = bf16_to_f32(p.x[base + i]);
            if (NORM && p.res) v[j] += bf16_to_f32(p.res[base + i]);
        }
    }
    if (NORM) {
#pragma unroll
        for (int j = 0; j < NE; ++j) ss = fma((double)v[j], (double)v[j], ss);
        r = rsqrt_f64(fma(row_sum<256>(ss, s_sum), p.inv_cols, (double)p.eps));
    }
    auto vw_of = [&](int j) __attribute__((always_inline)) {
        asm volatile("" : "+v"(v[j]));                  // (converted again, not kept as a double)
        return (double)v[j] * (NORM && p.w ? (double)p.w[min(t + j * 256, p.cols - 1)] : 1.0);
    };
    Peak peak;
#pragma unroll
    for (int j = 0; j < NE; ++j) {
        const int i = t + j * 256;
        const double u = vw_of(j);
        peak.add(u);
        if (!NORM || i >= p.cols) continue;
        if (p.sum) p.sum[base + i] = (uint16_t)pack_bf16(v[j], 0.f);
        if (p.y) p.y[base + i] = (uint16_t)pack_bf16((float)(u * r), 0.f);
    }
    if (p.qmode == MOE_Q_I8_ROW) {
        float scale;
        double mul;
        float quick;
        i8_scale<256>(peak, r, s_max, s_bad, &scale, &mul, &quick);
        if (t == 0) ((float*)p.scales)[row] = scale;
#pragma unroll
        for (int j = 0; j < NE; ++j) {
            const int i = t + j * 256;
            if (i < p.cols) p.codes[base + i] = (uint8_t)i8_code<NORM>(vw_of(j), mul);
        }
    }
}

// ------------------------------------------------------------------ 8-bit rows -> bf16
// 8 values per thread (ELEM: one, where an address is not aligned), over the
// whole tensor: code * scale in fp32, rounded once. SHIFT (int8, cols no
// multiple of 8): 8 values may belong to two rows or more; the division that
// finds the row, and the walk over rows, cost little beside one value a thread
// (5708 x 5878: 47 us so, 16.5 with 8).
template <int QMODE, bool ELEM, bool SHIFT>
__global__ void __launch_bounds__(256) dequant_rows_kernel(const uint8_t* codes, const void* scales, int cols, size_t n,
                                                           uint16_t* out) {
    // (the caller keeps the number of vectors below 2^32, and that of values too where they are counted)
    const uint32_t iv = blockIdx.x * 256u + threadIdx.x;
    const size_t i = (size_t)iv * (ELEM ? 1 : 8);
    if (i >= n) return;
    const uint32_t row = ELEM || SHIFT ? (uint32_t)i / (uint32_t)cols : iv / (uint32_t)(cols / 8);
    float sc;
    if (QMODE == MOE_Q_I8_ROW) sc = ((const float*)scales)[row];
    else {
        const uint8_t e = ((const uint8_t*)scales)[i / 128];             // (rows are whole groups)
        sc = e == 255 ? __uint_as_float(0x7FC00000u) : ldexpf(1.0f, (int)e - 127);
    }
    if (ELEM) {
        out[i] = (uint16_t)pack_bf16((float)(int8_t)codes[i] * sc, 0.f);
        return;
    }
    float s[8];
#pragma unroll
    for (int d = 0; d < 8; ++d) s[d] = sc;
    if (SHIFT) {
        uint32_t r = row, c = (uint32_t)i - row * (uint32_t)cols;
        if (c + 8 > (uint32_t)cols) {
#pragma unroll
            for (int d = 0; d < 8; ++d) {
                if (c == (uint32_t)cols) {
                    c = 0;
                    if (i + d < n) sc = ((const float*)scales)[++r];
                }
                s[d] = sc;
                ++c;
            }
        }
        if (i + 8 > n) {                                                 // the tensor ends in this vector
            for (int d = 0; i + d < n; ++d) out[i + d] = (uint16_t)pack_bf16((float)(int8_t)codes[i + d] * s[d], 0.f);
            return;
        }
    }
    const uint2 c = *(const uint2*)(codes + i);
    i32x4 o;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        const uint32_t w = (d < 2 ? c.x : c.y) >> (16 * (d & 1));
        const float a = QMODE == MOE_Q_I8_ROW ? (float)(int8_t)w : e4m3_to_f32(w & 0xFF);
        const float b = QMODE == MOE_Q_I8_ROW ? (float)(int8_t)(w >> 8) : e4m3_to_f32((w >> 8) & 0xFF);
        o[d] = (int)pack_bf16(a * s[2 * d], b * s[2 * d + 1]);
    }
    *(i32x4*)(out + i) = o;
}

int norm_max_cols() { return 16384; }

// A wave per row needs no exchange through LDS and leaves no threads idle on
// short rows; a workgroup per row spreads few rows over more CUs. Measured (us,
// a wave / a workgroup a row): int8 rows alone 8192 x 512 4.9 / 9.9, 2048 x 512
// 4.1 / 4.2; norm with int8 rows 1024 x 512 4.9 / 5.2, 512 x 768 4.6 / 4.4, 1024
// x 2048 9.2 / 6.3, 2048 x 2048 13.2 / 10.8, 4096 x 1536 14.6 / 15.9, 4096 x 1032
// 13.9 / 14.4, 16384 x 2048 54.8 / 56.5.
template <bool NORM, bool SHIFT>
static hipError_t launch_vec(const NormArgs& p, int nvec, int kid, hipStream_t stream) {
    const dim3 b(256), R((unsigned)p.rows), R4(((unsigned)p.rows + 3) / 4);
    if (nvec <= 256 && p.rows >= (nvec <= 128 ? 1024 : 2049)) {
        if (nvec <= 64) return launch_kernel(kid, stream, norm_vec_kernel<64, 1, NORM, SHIFT>, R4, b, 0, p);
        else if (nvec <= 128) return launch_kernel(kid, stream, norm_vec_kernel<64, 2, NORM, SHIFT>, R4, b, 0, p);
        else return launch_kernel(kid, stream, norm_vec_kernel<64, 4, NORM, SHIFT>, R4, b, 0, p);
    } else if (nvec <= 256) return launch_kernel(kid, stream, norm_vec_kernel<256, 1, NORM, SHIFT>, R, b, 0, p);
    else if (nvec <= 512) return launch_kernel(kid, stream, norm_vec_kernel<256, 2, NORM, SHIFT>, R, b, 0, p);
    else if (nvec <= 1024) return launch_kernel(kid, stream, norm_vec_kernel<256, 4, NORM, SHIFT>, R, b, 0, p);
    else return launch_kernel(kid, stream, norm_vec_kernel<256, 8, NORM, SHIFT>, R, b, 0, p);
}

template <bool NORM>
static hipError_t launch_rows(const NormArgs& p, bool aligned, int kid, hipStream_t stream) {
    const int nvec = (p.cols + 14) / 8;                          // vectors of a shifted row at most
    if (aligned && p.cols % 8 == 0) return launch_vec<NORM, false>(p, p.cols / 8, kid, stream);
    if (aligned && nvec <= 2048) return launch_vec<NORM, true>(p, nvec, kid, stream);
    const dim3 b(256), R((unsigned)p.rows);
    if (p.cols <= 2048) return launch_kernel(kid, stream, norm_elem_kernel<8, NORM>, R, b, 0, p);
    else return launch_kernel(kid, stream, norm_elem_kernel<64, NORM>, R, b, 0, p);
}

hipError_t launch_norm(const uint16_t* x, const uint16_t* res, const float* w, float eps, int rows, int cols, int qmode,
                       uint16_t* sum, uint16_t* y, uint8_t* codes, void* scales, bool aligned, hipStream_t stream) {
    return launch_rows<true>(NormArgs{x, res, w, eps, rows, cols, qmode, sum, y, codes, scales, 1.0 / cols}, aligned, K_NORM, stream);
}

hipError_t launch_quant_rows(const uint16_t* x, int rows, int cols, int8_t* codes, float* scales, bool aligned,
                             hipStream_t stream) {
    return launch_rows<false>(NormArgs{x, nullptr, nullptr, 0.f, rows, cols, MOE_Q_I8_ROW, nullptr, nullptr,
                                       (uint8_t*)codes, scales, 1.0 / cols}, aligned, K_QUANT_ROWS, stream);
}

hipError_t launch_dequant_rows(const uint8_t* codes, const void* scales, int rows, int cols, int qmode, uint16_t* out,
                               bool aligned, hipStream_t stream) {
    const size_t n = (size_t)rows * cols;
    const dim3 g((unsigned)((n + (aligned ? 2047 : 255)) / (aligned ? 2048 : 256))), b(256);
    if (qmode == MOE_Q_FP8_G128_POW2)
        return launch_kernel(K_DEQUANT_ROWS, stream, dequant_rows_kernel<MOE_Q_FP8_G128_POW2, false, false>, g, b, 0, codes, scales, cols, n, out);
    else if (!aligned)
        return launch_kernel(K_DEQUANT_ROWS, stream, dequant_rows_kernel<MOE_Q_I8_ROW, true, false>, g, b, 0, codes, scales, cols, n, out);
    else if (cols % 8)
        return launch_kernel(K_DEQUANT_ROWS, stream, dequant_rows_kernel<MOE_Q_I8_ROW, false, true>, g, b, 0, codes, scales, cols, n, out);
    else
        return launch_kernel(K_DEQUANT_ROWS, stream, dequant_rows_kernel<MOE_Q_I8_ROW, false, false>, g, b, 0, codes, scales, cols, n, out);
}

}  // namespace moe
