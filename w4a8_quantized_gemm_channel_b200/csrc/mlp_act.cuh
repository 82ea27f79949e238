// Activations of the MLP operators and their row passes: the INT8 rows of a
// float32 or bfloat16 input, and the scaled FP16 rows of a gradient.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace w4a8 {
namespace mlp {

// ------------------------------------------------------------- activations ---
// Everything in float32, in few instructions: an epilogue's exponentials,
// reciprocals and conversions share one pipe at an eighth of the ALU's rate, so
// each activation takes one of the first two each. The hardware exponential
// (2 ulp) of a product rounded before it is off by 2 ulp + |argument| 2^-24:
// some 20 ulp where the activation's tail is still above 2^-24, and less than
// 2^-24 absolute beyond.
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float LOG2E = 1.4426950408889634f;
constexpr float GELU_C = 0.7978845608028654f;   // sqrt(2 / pi)
constexpr float GELU_A = 0.044715f;
constexpr float RSQRT_2PI = 0.3989422804014327f;

// exp(-2t) = 2^(z (c1 + c2 z^2)) of the tanh form, t = sqrt(2/pi)(z + 0.044715 z^3):
// 1 + tanh(t) = 2 / (1 + exp(-2t)).
__device__ __forceinline__ float gelu_tanh_arg(float z) {
    return z * __fmaf_rn(-2.0f * GELU_C * GELU_A * LOG2E, z * z, -2.0f * GELU_C * LOG2E);
}

// e = exp(-z^2 / 2) and Phi(-|z|) = e g(|z|): g(x) = erfcx(x / sqrt(2)) / 2 is
// smooth in t = 1 / (1 + 0.3 x), here the polynomial of degree 8 in t with the
// least relative error over 0 <= x <= 14 (5.8e-8; 7 2^-24 evaluated in float32),
// found by reweighted least squares against float64 erfcx. The tail keeps its
// relative accuracy, so z Phi(z) has no cancellation for negative z.
__device__ __forceinline__ float normal_tail(float z, float &e) {
    const float x = fabsf(z), t = rcp_fast(__fmaf_rn(0.3f, x, 1.0f));
    e = exp2_fast(-0.5f * LOG2E * (x * x));
    float g = 0.0383782896f;
    g = __fmaf_rn(g, t, -0.169166112f);
    g = __fmaf_rn(g, t, 0.228660081f);
    g = __fmaf_rn(g, t, -0.0765064774f);
    g = __fmaf_rn(g, t, 0.142535524f);
    g = __fmaf_rn(g, t, 0.0946835229f);
    g = __fmaf_rn(g, t, 0.121920342f);
    g = __fmaf_rn(g, t, 0.119487689f);
    g = __fmaf_rn(g, t, 7.168876e-06f);
    return e * g;
}

// z / (1 + e) with e = exp(-..): an overflowing e gives the limit 0.
template <int ACT>
__device__ __forceinline__ float act_value(float z) {
    if constexpr (ACT == W4A8_ACT_NONE) return z;
    if constexpr (ACT == W4A8_ACT_RELU) return z > 0.0f ? z : 0.0f;
    if constexpr (ACT == W4A8_ACT_SILU) return z * rcp_fast(1.0f + exp2_fast(-LOG2E * z));
    if constexpr (ACT == W4A8_ACT_GELU) {
        float e;
        const float q = normal_tail(z, e);
        return z * (z < 0.0f ? q : 1.0f - q);
    }
    if constexpr (ACT == W4A8_ACT_GELU_TANH) return z * rcp_fast(1.0f + exp2_fast(gelu_tanh_arg(z)));
    return z;
}

// s(a) and 1 - s(a) of the logistic function, -a log2(e) given: e = exp(-a),
// s = 1 / (1 + e), 1 - s = e s without cancellation, or 1 where s has become 0.
struct Logistic {
    float s, c;
};
__device__ __forceinline__ Logistic logistic2(float minus_a_log2e) {
    const float e = exp2_fast(minus_a_log2e), s = rcp_fast(1.0f + e);
    return Logistic{s, s > 0.0f ? e * s : 1.0f};
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
        const Logistic l = logistic2(-LOG2E * z);
        a = z * l.s;
        d = l.s * __fmaf_rn(z, l.c, 1.0f);
    } else if constexpr (ACT == W4A8_ACT_GELU) {
        float e;
        const float q = normal_tail(z, e), p = z < 0.0f ? q : 1.0f - q;
        a = z * p;
        d = __fmaf_rn(z * RSQRT_2PI, e, p);
    } else if constexpr (ACT == W4A8_ACT_GELU_TANH) {
        const Logistic l = logistic2(gelu_tanh_arg(z));
        a = z * l.s;
        // (a l.c is 0 long before z^2 overflows; the cap keeps the product a number)
        d = __fmaf_rn(a * l.c, 2.0f * GELU_C * __fmaf_rn(3.0f * GELU_A, fminf(z * z, 1e30f), 1.0f), l.s);
    }
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

// Eight elements as loaded.
template <typename T>
struct Raw8 {
    uint4 r[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T *row, int i, int n, bool vec) {
        if (vec && i + 8 <= n) {
            r[0] = ld_dep_v4(row + i);
            if constexpr (sizeof(T) == 4) r[1] = ld_dep_v4(row + i + 4);
            return;
        }
        float v[8];
        ld_row8(row, i, n, false, v);
        if constexpr (sizeof(T) == 4) {
            r[0] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
            r[1] = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
        } else {  // widened bfloat16: the upper halves
            r[0] = make_uint4(__byte_perm(__float_as_uint(v[0]), __float_as_uint(v[1]), 0x7632),
                              __byte_perm(__float_as_uint(v[2]), __float_as_uint(v[3]), 0x7632),
                              __byte_perm(__float_as_uint(v[4]), __float_as_uint(v[5]), 0x7632),
                              __byte_perm(__float_as_uint(v[6]), __float_as_uint(v[7]), 0x7632));
        }
    }
    __device__ __forceinline__ void values(float (&v)[8]) const {
        if constexpr (sizeof(T) == 4) {
            v[0] = __uint_as_float(r[0].x); v[1] = __uint_as_float(r[0].y);
            v[2] = __uint_as_float(r[0].z); v[3] = __uint_as_float(r[0].w);
            v[4] = __uint_as_float(r[1].x); v[5] = __uint_as_float(r[1].y);
            v[6] = __uint_as_float(r[1].z); v[7] = __uint_as_float(r[1].w);
        } else {
            unpack_bf16x2(r[0].x, v[0], v[1]);
            unpack_bf16x2(r[0].y, v[2], v[3]);
            unpack_bf16x2(r[0].z, v[4], v[5]);
            unpack_bf16x2(r[0].w, v[6], v[7]);
        }
    }
};

// Step 3 of the layer on rows of T: the arithmetic of k_act_quant (the same
// scales and codes for the same float32 values; a bfloat16 is widened
// exactly), codes stored in the k-permuted order of the nibble unpack (k0 k2
// k4 k6 k1 k3 k5 k7 in every 8), the bytes from K to ldq zero. Bound: reading X.
//
// One block per row, the row's bytes kept as loaded between the two steps: few
// registers, so many blocks per SM whose loads, reductions and stores overlap.
// Rows of up to 8 THREADS UNITS values fit (12288 in the widest form); longer
// ones are read twice. A bfloat16 call of 2048 rows and 256 channels takes 36.6
// us at K = 12288, 51.1 at 12304, 84.8 at 28672.
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
    auto peak = [](const Raw8<T> &r, float a) {
        float v[8];
        r.values(v);
#pragma unroll
        for (int b = 0; b < 8; ++b) a = fmaxf(a, fabsf(v[b]));
        return a;
    };
    for (int m = blockIdx.x; m < M; m += gridDim.x) {
        const T *x = X + (size_t)m * ldx;
        uint2 *row = reinterpret_cast<uint2 *>(Xq + (size_t)m * ldq);
        Raw8<T> raw[UNITS];
        float amax = 0.0f;
        if (in_regs) {
#pragma unroll
            for (int i = 0; i < UNITS; ++i)
                if ((int)threadIdx.x + i * THREADS < units) raw[i].load(x, 8 * ((int)threadIdx.x + i * THREADS), K, vec != 0);
#pragma unroll
            for (int i = 0; i < UNITS; ++i)
                if ((int)threadIdx.x + i * THREADS < units) amax = peak(raw[i], amax);
        } else {
            for (int u = threadIdx.x; u < units; u += THREADS) {
                raw[0].load(x, 8 * u, K, vec != 0);
                amax = peak(raw[0], amax);
            }
        }
        const float s = act_scale_from_amax(block_max<THREADS>(amax, red));
        if (threadIdx.x == 0) sx[m] = s;
        if (in_regs) {
#pragma unroll
            for (int i = 0; i < UNITS; ++i) {
                const int u = threadIdx.x + i * THREADS;
                float v[8];
                raw[i].values(v);
                if (u < units) row[u] = row_codes8(v, s);
            }
        } else {
            for (int u = threadIdx.x; u < units; u += THREADS) {
                float v[8];
                raw[0].load(x, 8 * u, K, vec != 0);
                raw[0].values(v);
                row[u] = row_codes8(v, s);
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
    int vec;          // the rows' eight-element pieces are 16-byte aligned
    // the operands of columns n..n+7 in row m, as loaded; zeros past N
    struct Piece {
        Raw8<T> d, g, w;
    };
    template <int ACT>
    __device__ __forceinline__ void load(int m, int n, Piece &p) const {
        p.d.load(dy + (size_t)m * lddy, n, N, vec != 0);
        if (GLU || ACT != W4A8_ACT_NONE) p.g.load(z + (size_t)m * ldz, n, N, vec != 0);
        if constexpr (GLU) p.w.load(u + (size_t)m * ldz, n, N, vec != 0);
    }
    // the segments' values there, before the scales
    template <int ACT>
    __device__ __forceinline__ static void values(const Piece &p, float (&a)[8], float (&b)[8]) {
        float d[8], g[8], w[8];
        p.d.values(d);
        if constexpr (GLU || ACT != W4A8_ACT_NONE) p.g.values(g);
        if constexpr (GLU) p.w.values(w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            a[i] = d[i];
            b[i] = 0.0f;
            if constexpr (GLU || ACT != W4A8_ACT_NONE) {
                float av, dv;
                act_value_grad<ACT>(g[i], av, dv);
                a[i] = GLU ? d[i] * w[i] * dv : d[i] * dv;
                if constexpr (GLU) b[i] = d[i] * av;
            }
        }
    }
    template <int ACT>
    __device__ __forceinline__ void dz8(int m, int n, float (&a)[8], float (&b)[8]) const {
        Piece p;
        load<ACT>(m, n, p);
        values<ACT>(p, a, b);
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

// One block per row: the values go to shared memory as float32 while the
// row's abs-max is taken, then out as FP16. (HELD false: rows whose values do
// not fit are computed twice.) v = dz / sw by a fast reciprocal, 2 ulp. Bound:
// HBM, (1 + saved) N T read and 2 N bytes per segment and plane written.
constexpr int GR_THREADS = 512;
constexpr int GR_HELD_MAX = 220 * 1024;  // bytes of values a block may hold

template <bool GLU, bool LO, bool HELD, int ACT, typename T>
__global__ void __launch_bounds__(GR_THREADS)
k_grad_rows(GradIn<GLU, T> in, int M, int seg, __half *__restrict__ P, float *__restrict__ rs) {
    __shared__ float red[GR_THREADS / 32];
    extern __shared__ __align__(16) float held[];  // HELD: [segments][seg]
    griddep_wait();
    griddep_launch_dependents();
    const int width = GLU ? 2 * seg : seg;
    // v of columns n..n+7: dz / sw
    const bool swv = (reinterpret_cast<uintptr_t>(in.sw) & 15) == 0;
    const bool suv = GLU && (reinterpret_cast<uintptr_t>(in.su) & 15) == 0;
    using Piece = typename GradIn<GLU, T>::Piece;
    auto values = [&](const Piece &p, int n, float (&a)[8], float (&b)[8]) {
        float s[8];
        ld_row8(in.sw, n, in.N, swv, s);
        in.template values<ACT>(p, a, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] *= rcp_fast(s[i]);
        if constexpr (GLU) {
            ld_row8(in.su, n, in.N, suv, s);
#pragma unroll
            for (int i = 0; i < 8; ++i) b[i] *= rcp_fast(s[i]);
        }
        if (n + 8 > in.N) {  // past the row's end: 0 times the reciprocal of nothing
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (n + i >= in.N) a[i] = b[i] = 0.0f;
        }
    };
    auto keep = [&](int i, const float (&v)[8]) {
        *reinterpret_cast<float4 *>(held + i) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4 *>(held + i + 4) = make_float4(v[4], v[5], v[6], v[7]);
    };
    auto kept = [&](int i, float (&v)[8]) {
        const float4 x = *reinterpret_cast<const float4 *>(held + i), y = *reinterpret_cast<const float4 *>(held + i + 4);
        v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
        v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
    };
    // (gated: the next piece travels while one is computed, 68.6 -> 62.7 us at
    // 2048 x 11008; with one segment those registers cost a resident block, 16.3 -> 21.4
    // us at 2048 x 4096, so each piece is loaded when it comes)
    Piece next;
    const int n0 = 8 * threadIdx.x;
    if (GLU && n0 < seg) in.template load<ACT>(blockIdx.x, n0, next);
    for (int m = blockIdx.x; m < M; m += gridDim.x) {
        float amax = 0.0f;
        for (int n = n0; n < seg; n += 8 * GR_THREADS) {
            float a[8], b[8];
            Piece p;
            if constexpr (GLU) {
                p = next;
                if (n + 8 * GR_THREADS < seg) in.template load<ACT>(m, n + 8 * GR_THREADS, next);
                else if (m + gridDim.x < M) in.template load<ACT>(m + gridDim.x, n0, next);
            } else {
                in.template load<ACT>(m, n, p);
            }
            values(p, n, a, b);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                amax = fmaxf(amax, fabsf(a[i]));
                if constexpr (GLU) amax = fmaxf(amax, fabsf(b[i]));
            }
            if constexpr (HELD) {
                keep(n, a);
                if constexpr (GLU) keep(seg + n, b);
            }
        }
        float s, r;
        row_power(block_max<GR_THREADS>(amax, red), s, r);
        if (threadIdx.x == 0) rs[m] = r;
        __half *hi = P + (size_t)m * width, *lo = hi + (size_t)M * width;
        auto put = [&](int i, const float (&v)[8]) {
            __half2 h[4], l[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float x = v[2 * j] * s, y = v[2 * j + 1] * s;
                h[j] = __floats2half2_rn(x, y);
                if constexpr (LO) {
                    const float2 f = __half22float2(h[j]);
                    l[j] = __floats2half2_rn(x - f.x, y - f.y);
                }
            }
            *reinterpret_cast<uint4 *>(hi + i) = *reinterpret_cast<const uint4 *>(h);
            if constexpr (LO) *reinterpret_cast<uint4 *>(lo + i) = *reinterpret_cast<const uint4 *>(l);
        };
        for (int n = n0; n < seg; n += 8 * GR_THREADS) {  // a thread's own pieces
            float a[8], b[8];
            if constexpr (HELD) {
                kept(n, a);
                if constexpr (GLU) kept(seg + n, b);
            } else {
                Piece p;
                in.template load<ACT>(m, n, p);
                values(p, n, a, b);
            }
            put(n, a);
            if constexpr (GLU) put(seg + n, b);
        }
    }
}

// Bias gradients: column sums of dz. Block (64 columns, slice of BG_ROWS rows):
// 64 row groups of 8 lanes x 8 columns each take every 64th row of the slice,
// their sums are added in a fixed order, so a run repeats bit for bit. One
// slice writes the result; more leave partial sums that k_bias_grad_sum adds
// in order. Sums are float32 over at most BG_ROWS / 64 rows, then 64, then the
// slices. Bound: HBM, the rows read once more; at few rows the launch, hence
// one where one slice covers them. Beside a gradient of 2048 x 4096 x 11008
// (M, K, N) in bfloat16 it adds 35 us (GELU), gated 50 us (SiLU).
constexpr int BG_ROWS = 256, BG_COLS = 64, BG_GROUPS = 64;

template <bool GLU, int ACT, typename T>
__global__ void __launch_bounds__(512)
k_bias_grad(GradIn<GLU, T> in, int M, float *part, float *dba, float *dbb) {
    constexpr int SEGS = GLU ? 2 : 1;
    __shared__ float red[SEGS][BG_GROUPS][BG_COLS + 1];
    griddep_wait();
    griddep_launch_dependents();
    const int c = threadIdx.x & 7, g = threadIdx.x >> 3;
    const int n0 = blockIdx.x * BG_COLS, n = n0 + 8 * c;
    const int slices = (M + BG_ROWS - 1) / BG_ROWS;
    for (int slice = blockIdx.y; slice < slices; slice += gridDim.y) {
        const int m1 = min(M, (slice + 1) * BG_ROWS);
        float sa[8] = {}, sb[8] = {};
        if (n < in.N) {
#pragma unroll 4
            for (int m = slice * BG_ROWS + g; m < m1; m += BG_GROUPS) {
                float a[8], b[8];
                in.template dz8<ACT>(m, n, a, b);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    sa[i] += a[i];
                    sb[i] += b[i];
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            red[0][g][8 * c + i] = sa[i];
            if constexpr (GLU) red[1][g][8 * c + i] = sb[i];
        }
        __syncthreads();
        const int col = threadIdx.x % BG_COLS, s = threadIdx.x / BG_COLS;
        if (s < SEGS && n0 + col < in.N) {
            float t = 0.0f;
#pragma unroll 16
            for (int w = 0; w < BG_GROUPS; ++w) t += red[s][w][col];
            float *out = s == 0 ? dba : dbb;
            if (slices > 1) part[((size_t)slice * SEGS + s) * in.N + n0 + col] = t;
            else if (out != nullptr) out[n0 + col] = t;
        }
        __syncthreads();
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
#pragma unroll 8
    for (int s = 0; s < slices; ++s) t += ld_dep(part + ((size_t)s * segs + blockIdx.y) * N + n);
    out[n] = t;
}

}  // namespace mlp
}  // namespace w4a8
