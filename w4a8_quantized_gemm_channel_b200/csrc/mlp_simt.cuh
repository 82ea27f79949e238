// CUDA-core form of the MLP operators: any shape, used for tiny problems.
#pragma once

#include "mlp_act.cuh"

namespace w4a8 {
namespace mlp {

// What one projection reads: packed codes, channel scales, bias or null.
struct Proj {
    const uint8_t *Wp;
    const float *sw;
    const float *bias;
};

// Arguments of a forward call's epilogue. Rows of T; R, Z, U may be null.
// linear: Y = act(z) + R, Z = z. gated: Y = act(g) u, Z = g, U = u.
struct EpiArgs {
    const void *R;
    void *Y, *Z, *U;
    int ldr, ldy, ldz;
};

// z = acc / (sx sw) + b as acc ((1/sx) (1/sw)) + b, the product with acc and
// the sum in one rounding. The reciprocals meet first: their product is what
// one unit of acc weighs, so it overflows only where the result does. (With
// acc / sx first, up to 2^31 times the row's abs-max, rows of 1e35 gave
// infinities for results of 1e35.)
__device__ __forceinline__ float dequant(float acc, float rsx, float rsw, float b) {
    return __fmaf_rn(acc, __fmul_rn(rsx, rsw), b);
}

// One thread per output. The row is in the k-permuted order, so a packed word
// of eight codes meets two words of it: two dp4a on sign-extended nibbles.
// FUSED (K <= SIMT_FUSED_K): a block quantizes its row into shared memory
// first, so a tiny call is one launch; otherwise Xq and sx are the row pass's.
constexpr int SIMT_FUSED_K = 4096;

template <bool GLU, bool FUSED, int ACT, typename T>
__global__ void __launch_bounds__(128)
k_mlp_simt(const T *X, int ldx, int vec, const int8_t *Xq, int M, int K, int ldq, const float *sx, Proj a, Proj b,
           int ldp, int N, EpiArgs e) {
    __shared__ uint2 codes[FUSED ? SIMT_FUSED_K / 8 : 1];
    __shared__ float red[4];
    griddep_launch_dependents();
    griddep_wait();
    const int n = blockIdx.x * 128 + threadIdx.x, nn = min(n, N - 1);
    const float ra = __frcp_rn(ld_dep(a.sw + nn)), ba = a.bias ? ld_dep(a.bias + nn) : 0.0f;
    const float rb = GLU ? __frcp_rn(ld_dep(b.sw + nn)) : 0.0f, bb = GLU && b.bias ? ld_dep(b.bias + nn) : 0.0f;
    const uint32_t *wa = reinterpret_cast<const uint32_t *>(a.Wp + (size_t)nn * ldp);
    const uint32_t *wb = GLU ? reinterpret_cast<const uint32_t *>(b.Wp + (size_t)nn * ldp) : wa;
    auto ld32 = [](const uint32_t *p) {
        uint32_t v;
        asm volatile("ld.global.u32 %0, [%1];" : "=r"(v) : "l"(p));
        return v;
    };
    const int units = (K + 7) / 8;
    for (int m = blockIdx.y; m < M; m += gridDim.y) {
        float s;
        if constexpr (FUSED) {
            const T *x = X + (size_t)m * ldx;
            float v[8], amax = 0.0f;
            for (int u = threadIdx.x; u < units; u += 128) {
                ld_row8(x, 8 * u, K, vec != 0, v);
#pragma unroll
                for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
            }
            s = act_scale_from_amax(block_max<128>(amax, red));  // its barriers also end the last row's reads
            for (int u = threadIdx.x; u < units; u += 128) {
                if (units > 128) ld_row8(x, 8 * u, K, vec != 0, v);
                codes[u] = row_codes8(v, s);
            }
            __syncthreads();
        } else {
            s = ld_dep(sx + m);
        }
        const uint32_t *x = reinterpret_cast<const uint32_t *>(Xq + (size_t)m * ldq);
        int32_t ca = 0, cb = 0;
        for (int w = 0; w < units; ++w) {
            uint2 q;
            if constexpr (FUSED) q = codes[w];
            else q = make_uint2(ld32(x + 2 * w), ld32(x + 2 * w + 1));
            uint32_t lo, hi;
            unpack_s4x8(ld32(wa + w), lo, hi);
            ca = __dp4a((int)lo, (int)q.x, __dp4a((int)hi, (int)q.y, ca));
            if constexpr (GLU) {
                unpack_s4x8(ld32(wb + w), lo, hi);
                cb = __dp4a((int)lo, (int)q.x, __dp4a((int)hi, (int)q.y, cb));
            }
        }
        if (n >= N) continue;
        const float rx = __frcp_rn(s);
        const float z = dequant(__int2float_rn(ca), rx, ra, ba);
        float y = act_value<ACT>(z);
        if constexpr (GLU) {
            const float u = dequant(__int2float_rn(cb), rx, rb, bb);
            y *= u;
            if (e.U) st_elem(static_cast<T *>(e.U) + (size_t)m * e.ldz + n, u);
        } else {
            if (e.R) y += ld_elem(static_cast<const T *>(e.R) + (size_t)m * e.ldr + n);
        }
        if (e.Z) st_elem(static_cast<T *>(e.Z) + (size_t)m * e.ldz + n, z);
        st_elem(static_cast<T *>(e.Y) + (size_t)m * e.ldy + n, y);
    }
}

// dX[m][k] = rs[m] sum_s sum_n P[m][s seg + n] q_s[n][k]: one thread per row
// and eight k (a packed word per n), float32 sums. planes: 1, or 2 with the
// low parts of P behind its M rows.
template <typename T>
__global__ void __launch_bounds__(128)
k_grad_simt(const __half *P, const float *rs, int M, int N, int seg, int segs, int planes, const uint8_t *Wa,
            const uint8_t *Wb, int ldp, int K, T *dX, int lddx) {
    griddep_launch_dependents();
    griddep_wait();
    const int w = blockIdx.x * 128 + threadIdx.x;
    if (8 * w >= K) return;
    const size_t width = (size_t)segs * seg;
    for (int m = blockIdx.y; m < M; m += gridDim.y) {
        float acc[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
        for (int s = 0; s < segs; ++s) {
            const uint8_t *W = (s ? Wb : Wa) + 4 * (size_t)w;
            const __half *p = P + (size_t)m * width + (size_t)s * seg;
            for (int n = 0; n < N; ++n) {
                uint16_t h;
                uint32_t q;
                asm volatile("ld.global.u16 %0, [%1];" : "=h"(h) : "l"(p + n));
                asm volatile("ld.global.u32 %0, [%1];" : "=r"(q) : "l"(W + (size_t)n * ldp));
                float v = __half2float(__ushort_as_half(h));
                if (planes == 2) {
                    asm volatile("ld.global.u16 %0, [%1];" : "=h"(h) : "l"(p + (size_t)M * width + n));
                    v += __half2float(__ushort_as_half(h));
                }
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    acc[j] = __fmaf_rn(v, (float)((int)((q >> (4 * j) & 15u) ^ 8u) - 8), acc[j]);
            }
        }
        const float r = ld_dep(rs + m);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (8 * w + j < K) st_elem(dX + (size_t)m * lddx + 8 * w + j, acc[j] * r);
    }
}

}  // namespace mlp
}  // namespace w4a8
