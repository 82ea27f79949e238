// Activations of the MLP operators and their row passes: the INT8 rows of a
// float32 or bfloat16 input, and the scaled FP16 rows of a gradient.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace w4a8 {
namespace mlp {

// ------------------------------------------------------------- activations ---
// Everything in float32. The logistic function is taken from
// t = exp(-|z|) in (0, 1], so nothing overflows, and 1 - s(z) = s(-z) comes
// without cancellation. The fast exponential is off by at most 2 + 1.173 |z|
// ulp: some 20 ulp of s where s is still above 2^-24, less than 2^-24 absolute
// in z s beyond. The tanh
// form of GELU is z s(2 t(z)) by 1 + tanh(a) = 2 s(2a).
struct Logistic {
    float s, c;  // s(z) and 1 - s(z)
};
__device__ __forceinline__ Logistic logistic(float z) {
    const float t = __expf(-fabsf(z));
    const float r = __fdividef(1.0f, 1.0f + t);
    const float q = t * r;
    return z >= 0.0f ? Logistic{r, q} : Logistic{q, r};
}

constexpr float GELU_C = 0.7978845608028654f;   // sqrt(2 / pi)
constexpr float GELU_A = 0.044715f;
constexpr float RSQRT_2PI = 0.3989422804014327f;

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
    if constexpr (ACT == W4A8_ACT_NONE) return z;
    if constexpr (ACT == W4A8_ACT_RELU) return z > 0.0f ? z : 0.0f;
    if constexpr (ACT == W4A8_ACT_SILU) return z * logistic(z).s;
    if constexpr (ACT == W4A8_ACT_GELU) return z * normcdff(z);
    if constexpr (ACT == W4A8_ACT_GELU_TANH) {
        const float t = GELU_C * __fmaf_rn(GELU_A * z * z, z, z);
        return z * logistic(2.0f * t).s;
    }
    return z;
}

// The activation by its code: for places that finish few values.
__device__ __noinline__ float act_any(int act, float z) {
    switch (act) {
        case W4A8_ACT_RELU: return act_value<W4A8_ACT_RELU>(z);
        case W4A8_ACT_SILU: return act_value<W4A8_ACT_SILU>(z);
        case W4A8_ACT_GELU: return act_value<W4A8_ACT_GELU>(z);
        case W4A8_ACT_GELU_TANH: return act_value<W4A8_ACT_GELU_TANH>(z);
        default: return z;
    }
}

// The activation and its derivative at z (ReLU's derivative at 0 is 0).
template <int ACT>
__device__ __forceinline__ void act_value_grad(float z, float &a, float &d) {
    a = z;
    d = 1.0f;
    if constexpr (ACT == W4A8_ACT_RELU) {
        a = z > 0.0f ? z : 0.0f;
        d = z > 0.0f ? 1.0f : 0.0f;
    } else if constexpr (ACT == W4A8_ACT_SILU) {
        const Logistic l = logistic(z);
        a = z * l.s;
        d = l.s * __fmaf_rn(z, l.c, 1.0f);
    } else if constexpr (ACT == W4A8_ACT_GELU) {
        const float p = normcdff(z);
        a = z * p;
        d = __fmaf_rn(z * RSQRT_2PI, expf(-0.5f * z * z), p);
    } else if constexpr (ACT == W4A8_ACT_GELU_TANH) {
        const float z2 = z * z;
        const Logistic l = logistic(2.0f * GELU_C * __fmaf_rn(GELU_A * z2, z, z));
        a = z * l.s;
        d = __fmaf_rn(z * l.s * l.c, 2.0f * GELU_C * __fmaf_rn(3.0f * GELU_A, z2, 1.0f), l.s);
    }
}

// ---------------------------------------------------------- typed elements ---
// Rows of T (float or __nv_bfloat16) that an earlier kernel may still be
// writing when this one starts: coherent loads, as ld_dep in common.cuh.
__device__ __forceinline__ float ld_elem(const float *p) { return ld_dep(p); }
__device__ __forceinline__ float ld_elem(const __nv_bfloat16 *p) {
    uint16_t v;
    asm volatile("ld.global.u16 %0, [%1];" : "=h"(v) : "l"(p));
    return __uint_as_float((uint32_t)v << 16);
}
__device__ __forceinline__ void unpack_bf16x2(uint32_t w, float &lo, float &hi) {
    lo = __uint_as_float(w << 16);
    hi = __uint_as_float(w & 0xFFFF0000u);
}
// Eight consecutive elements; vec: the address is 16-byte aligned.
__device__ __forceinline__ void ld_elem8(const float *p, float (&v)[8]) {
    const float4 a = ld_dep_f4(p), b = ld_dep_f4(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void ld_elem8(const __nv_bfloat16 *p, float (&v)[8]) {
    const uint4 a = ld_dep_v4(p);
    unpack_bf16x2(a.x, v[0], v[1]);
    unpack_bf16x2(a.y, v[2], v[3]);
    unpack_bf16x2(a.z, v[4], v[5]);
    unpack_bf16x2(a.w, v[6], v[7]);
}
// Elements i..i+7 of a row of n, zeros past its end.
template <typename T>
__device__ __forceinline__ void ld_row8(const T *row, int i, int n, bool vec, float (&v)[8]) {
    if (vec && i + 8 <= n) {
        ld_elem8(row + i, v);
        return;
    }
#pragma unroll
    for (int b = 0; b < 8; ++b) v[b] = i + b < n ? ld_elem(row + i + b) : 0.0f;
}
__device__ __forceinline__ void st_elem(float *p, float v) { *p = v; }
__device__ __forceinline__ void st_elem(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// Maximum of one value per thread over the block, known to every thread.
template <int THREADS>
__device__ __forceinline__ float block_max(float a, float *red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    if (lane == 0) red[warp] = a;
    __syncthreads();
    float m = red[0];
#pragma unroll
    for (int i = 1; i < THREADS / 32; ++i) m = fmaxf(m, red[i]);
    __syncthreads();
    return m;
}

// --------------------------------------------------------------- INT8 rows ---
// The codes of eight consecutive values (scale s): word 0 = k0 k2 k4 k6, word
// 1 = k1 k3 k5 k7. x s lies within 127 plus one rounding, so adding 1.5 2^23
// rounds it to the nearest integer, ties to even, in the low bits (act_code8's
// value; the clamp never binds) at two full-rate instructions a value, where
// a conversion to integer runs at a quarter of the rate.
__device__ __forceinline__ uint2 row_codes8(const float (&v)[8], float s) {
    uint32_t q[8];
#pragma unroll
    for (int b = 0; b < 8; ++b) q[b] = __float_as_uint(__fadd_rn(__fmul_rn(v[b], s), 12582912.0f));
    const uint32_t e0 = __byte_perm(q[0], q[2], 0x0040), e1 = __byte_perm(q[4], q[6], 0x0040);
    const uint32_t o0 = __byte_perm(q[1], q[3], 0x0040), o1 = __byte_perm(q[5], q[7], 0x0040);
    return make_uint2(__byte_perm(e0, e1, 0x5410), __byte_perm(o0, o1, 0x5410));
}

// Step 3 of the layer on rows of T: the arithmetic of k_act_quant (the same
// scales and codes for the same float32 values; a bfloat16 is widened
// exactly), codes stored in the k-permuted order of the nibble unpack (k0 k2
// k4 k6 k1 k3 k5 k7 in every 8), the bytes from K to ldq zero. One block per
// row; a row of up to THREADS x 8 x UNITS elements stays in registers between
// the abs-max and the codes, a longer one is read twice. Bound: reading X.
template <typename T, int THREADS, int UNITS>
__global__ void __launch_bounds__(THREADS)
k_quant_rows(const T *X, int M, int K, int ldx, int8_t *__restrict__ Xq, int ldq, float *__restrict__ sx,
             int vec) {
    __shared__ float red[THREADS / 32];
    // as in k_act_quant: dependents start only once all earlier work is done,
    // so they may read static weights ahead of their own wait
    griddep_wait();
    griddep_launch_dependents();
    const int units = ldq / 8;
    const bool in_regs = units <= THREADS * UNITS;
    for (int m = blockIdx.x; m < M; m += gridDim.x) {
        const T *x = X + (size_t)m * ldx;
        uint2 *row = reinterpret_cast<uint2 *>(Xq + (size_t)m * ldq);
        float v[UNITS][8], amax = 0.0f;
        if (in_regs) {
#pragma unroll
            for (int i = 0; i < UNITS; ++i) {
                ld_row8(x, 8 * ((int)threadIdx.x + i * THREADS), K, vec != 0, v[i]);
#pragma unroll
                for (int b = 0; b < 8; ++b) amax = fmaxf(amax, fabsf(v[i][b]));
            }
        } else {
            for (int u = threadIdx.x; u < units; u += THREADS) {
                float w[8];
                ld_row8(x, 8 * u, K, vec != 0, w);
#pragma unroll
                for (int b = 0; b < 8; ++b) amax = fmaxf(amax, fabsf(w[b]));
            }
        }
        const float s = act_scale_from_amax(block_max<THREADS>(amax, red));
        if (threadIdx.x == 0) sx[m] = s;
        if (in_regs) {
#pragma unroll
            for (int i = 0; i < UNITS; ++i) {
                const int u = threadIdx.x + i * THREADS;
                if (u < units) row[u] = row_codes8(v[i], s);
            }
        } else {
            for (int u = threadIdx.x; u < units; u += THREADS) {
                float w[8];
                ld_row8(x, 8 * u, K, vec != 0, w);
                row[u] = row_codes8(w, s);
            }
        }
    }
}

// ----------------------------------------------------------- gradient rows ---
// The operand of the gradient product: v[m][n] = dz[m][n] / sw[n] (the gated
// form has two segments, gate then up, each `seg` columns, zero past N), held
// in FP16 with one power of two per row: p[m][n] = fp16(v 2^e[m]), with the
// row's abs-max at 2^14..2^15. A value then rounds by at most 2^-11 of itself
// down to 2^-28 of the row's maximum (and by 2^-39 of the maximum below), and
// the INT4 codes are exact in FP16, so the product is eight times closer
// than with bfloat16 rows at the same tensor-core rate. With LO a second
// plane holds fp16(v 2^e - p): 22 bits, for float32 gradients.
template <bool GLU, typename T>
struct GradIn {
    const T *dy;      // [M][lddy]: gradient of the output
    const T *z, *u;   // [M][ldz]: saved pre-activations (z: gate, or the linear's z; null without activation)
    const float *sw, *su;
    int N, lddy, ldz;
    // the segments' values of column n in row m, before the scales
    template <int ACT>
    __device__ __forceinline__ void dz(int m, int n, float &a, float &b) const {
        const float dyv = ld_elem(dy + (size_t)m * lddy + n);
        if constexpr (GLU) {
            float av, dv;
            act_value_grad<ACT>(ld_elem(z + (size_t)m * ldz + n), av, dv);
            a = dyv * ld_elem(u + (size_t)m * ldz + n) * dv;
            b = dyv * av;
        } else {
            b = 0.0f;
            a = dyv;
            if constexpr (ACT != W4A8_ACT_NONE) {
                float av, dv;
                act_value_grad<ACT>(ld_elem(z + (size_t)m * ldz + n), av, dv);
                a = dyv * dv;
            }
        }
    }
};

// Power of two that brings a row's abs-max into [2^14, 2^15) and its inverse
// (1 for a zero or non-finite row; exponents clamped to normal floats).
__device__ __forceinline__ void row_power(float amax, float &s, float &rs) {
    const int ex = (int)((__float_as_uint(amax) >> 23) & 0xFFu);  // biased exponent
    int e = (ex == 0 && amax == 0.0f) || ex == 255 ? 0 : 14 - (ex - 127);
    e = min(max(e, -126), 126);
    s = __uint_as_float((uint32_t)(127 + e) << 23);
    rs = __uint_as_float((uint32_t)(127 - e) << 23);
}

constexpr int GR_THREADS = 256;

template <bool GLU, bool LO, int ACT, typename T>
__global__ void __launch_bounds__(GR_THREADS)
k_grad_rows(GradIn<GLU, T> in, int M, int seg, __half *__restrict__ P, float *__restrict__ rs) {
    __shared__ float red[GR_THREADS / 32];
    griddep_wait();
    griddep_launch_dependents();
    const int width = GLU ? 2 * seg : seg;
    for (int m = blockIdx.x; m < M; m += gridDim.x) {
        float amax = 0.0f;
        for (int n = threadIdx.x; n < in.N; n += GR_THREADS) {
            float a, b;
            in.template dz<ACT>(m, n, a, b);
            amax = fmaxf(amax, fabsf(__fdiv_rn(a, ld_dep(in.sw + n))));
            if constexpr (GLU) amax = fmaxf(amax, fabsf(__fdiv_rn(b, ld_dep(in.su + n))));
        }
        float s, r;
        row_power(block_max<GR_THREADS>(amax, red), s, r);
        if (threadIdx.x == 0) rs[m] = r;
        __half *hi = P + (size_t)m * width, *lo = hi + (size_t)M * width;
        auto put = [&](int i, float v) {
            const __half h = __float2half_rn(v);
            hi[i] = h;
            if constexpr (LO) lo[i] = __float2half_rn(v - __half2float(h));
        };
        for (int n = threadIdx.x; n < seg; n += GR_THREADS) {
            float a = 0.0f, b = 0.0f;
            if (n < in.N) {
                in.template dz<ACT>(m, n, a, b);
                a = __fdiv_rn(a, ld_dep(in.sw + n)) * s;
                if constexpr (GLU) b = __fdiv_rn(b, ld_dep(in.su + n)) * s;
            }
            put(n, a);
            if constexpr (GLU) put(seg + n, b);
        }
    }
}

// Bias gradients: column sums of dz. Block (column block of 32, row slice):
// each of 8 warps adds every eighth row of the slice, the warps' sums meet in
// shared memory in a fixed order, and a second kernel adds the slices in
// order, so a run repeats bit for bit. Sums are float32 over at most
// BG_ROWS / 8 rows, then 8, then the slices.
constexpr int BG_ROWS = 256;

template <bool GLU, int ACT, typename T>
__global__ void __launch_bounds__(256)
k_bias_grad_part(GradIn<GLU, T> in, int M, float *__restrict__ part) {
    __shared__ float red[GLU ? 2 : 1][8][33];
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n = blockIdx.x * 32 + lane;
    const int m1 = min(M, ((int)blockIdx.y + 1) * BG_ROWS);
    float sa = 0.0f, sb = 0.0f;
    if (n < in.N) {
        for (int m = blockIdx.y * BG_ROWS + warp; m < m1; m += 8) {
            float a, b;
            in.template dz<ACT>(m, n, a, b);
            sa += a;
            sb += b;
        }
    }
    red[0][warp][lane] = sa;
    if constexpr (GLU) red[1][warp][lane] = sb;
    __syncthreads();
    if (warp < (GLU ? 2 : 1) && n < in.N) {
        float t = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) t += red[warp][w][lane];
        part[((size_t)blockIdx.y * (GLU ? 2 : 1) + warp) * in.N + n] = t;
    }
}

// db[n] (and for the gated form dbu[n]) = sum over slices; null: not wanted.
__global__ void __launch_bounds__(256)
k_bias_grad_sum(const float *part, int slices, int segs, int N, float *dba, float *dbb) {
    griddep_wait();
    griddep_launch_dependents();
    const int n = blockIdx.x * 256 + threadIdx.x;
    float *out = blockIdx.y == 0 ? dba : dbb;
    if (n >= N || out == nullptr) return;
    float t = 0.0f;
    for (int s = 0; s < slices; ++s) t += ld_dep(part + ((size_t)s * segs + blockIdx.y) * N + n);
    out[n] = t;
}

}  // namespace mlp
}  // namespace w4a8
