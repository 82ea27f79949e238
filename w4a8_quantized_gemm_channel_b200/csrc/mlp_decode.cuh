// Few-row form of the MLP operators' forward calls (M <= 16): the packed
// weights stream once through shared memory, everything else happens beside
// the stream.
//
// Bound: HBM, N K / 2 bytes per projection. The block is that of k_decode_ring
// (decode_bulk.cuh): one producer thread keeps a ring of TMA stages full (16
// packed rows x up to 2 KB each), 8 consumer warps multiply a stage with the
// INT8 rows on the legacy integer tensor-core path, 16 q nibbles, K <= 131072.
//
// Gated form: a stage holds 8 gate rows and the same 8 up rows, so that the
// m16n8k32 product leaves a channel's two projections in one thread's
// accumulators and one thread finishes act(g) u; nothing is exchanged beyond
// the sum over the warps.
//
// The INT8 rows come from the row pass, or (FUSED, few values) from X itself:
// every block quantizes all rows, the values held in registers between the
// abs-max and the codes, which saves the launch of the row pass. Rows sit in
// shared memory in the k-permuted order of the nibble masks.
#pragma once

#include "decode_bulk.cuh"
#include "mlp_act.cuh"
#include "mlp_simt.cuh"

namespace w4a8 {
namespace mlp {

constexpr int DEC_TOK = 16;                 // rows at most
constexpr int DEC_RING = 12;                // ring slots at most
constexpr int DEC_RED = 2;                  // groups whose warp sums may be waiting to be added
constexpr int DEC_THREADS = dbulk::THREADS + 32;  // 8 consumer warps, the producer, the finishing warp
constexpr int DEC_CONSUMERS = dbulk::CONSUMERS;

struct DecArgs {
    const void *X;       // FUSED: rows of T
    const int8_t *Xq;    // else: INT8 rows (permuted order) and scales
    const float *sx;
    int ldx, ldq, vec;
    int M, K, N;
    Proj a, b;
    EpiArgs e;
    int act, ring, early, max_sb;
};

// Stages of a row's packed bytes: nst stages of sb bytes (a multiple of 64),
// activation rows pitch bytes apart (all k of the stages + 16).
struct DecGeo {
    int kp, sb, nst, pitch;
    __host__ __device__ DecGeo(int K, int max_sb) {
        kp = packed_row_bytes(K);
        const int kp64 = (kp + 63) / 64 * 64;
        sb = kp64 < max_sb ? kp64 : max_sb;
        nst = (kp + sb - 1) / sb;
        pitch = 2 * sb * nst + 16;
    }
    __host__ __device__ int stage_bytes() const { return 16 * sb; }
};

template <int NTG>
struct DecSmem {
    uint64_t full[DEC_RING], empty[DEC_RING];
    uint64_t rfull[DEC_RED], rfree[DEC_RED];
    float part[8][dbulk::CONSUMER_WARPS];
    float rsx[8 * NTG];
    int32_t red[DEC_RED][dbulk::CONSUMER_WARPS][16][8 * NTG + 1];
    int abort;
};
// A block's static shared memory, up to where the dynamic part begins.
template <int NTG>
constexpr int dec_static() { return ((int)sizeof(DecSmem<NTG>) + 1023) / 1024 * 1024 + 1024; }
constexpr int DEC_SM_SMEM = 226 * 1024;  // what blocks may take of an SM's shared memory

// Quantize the M <= R rows of X (J units of 8 values per thread and row) into
// xs, all rows at once: one round of loads, one barrier for the abs-maxima.
template <int R, int J, typename T>
__device__ __forceinline__ void dec_quantize(const DecArgs &p, int ks, int pitch, int8_t *xs,
                                             float (*part)[dbulk::CONSUMER_WARPS], float *rsx, int tid) {
    Raw8<T> raw[R][J];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int j = 0; j < J; ++j)  // rows past the last repeat it
            raw[r][j].load(static_cast<const T *>(p.X) + (size_t)min(r, p.M - 1) * p.ldx,
                           8 * (tid + DEC_CONSUMERS * j), p.K, p.vec != 0);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        float a = 0.0f, v[8];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            raw[r][j].values(v);
#pragma unroll
            for (int b = 0; b < 8; ++b) a = fmaxf(a, fabsf(v[b]));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
        if ((tid & 31) == 0) part[r][tid >> 5] = a;
    }
    ptx::bar_sync(1, DEC_CONSUMERS);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (r >= p.M) break;
        float a = part[r][0], v[8];
#pragma unroll
        for (int w = 1; w < dbulk::CONSUMER_WARPS; ++w) a = fmaxf(a, part[r][w]);
        const float s = act_scale_from_amax(a);
        if (tid == 0) rsx[r] = __frcp_rn(s);
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int k = 8 * (tid + DEC_CONSUMERS * j);
            raw[r][j].values(v);
            if (k < ks) *reinterpret_cast<uint2 *>(xs + (size_t)r * pitch + k) = row_codes8(v, s);  // zeros past K
        }
    }
}

// MMAs of one stage for NTG groups of 8 rows: chunks of 64 packed bytes (128 k)
// warp, warp + 8, ...; xs: the INT8 rows, pitch bytes apart, at the stage's k.
template <int NTG>
__device__ __forceinline__ void dec_stage(int32_t (&acc)[NTG][2][4], const uint8_t *st, int sb, const int8_t *xs,
                                          int pitch, int M, int g, int t, int warp) {
    const int cps = sb / 64;
#pragma unroll 2
    for (int c = warp; c < cps; c += dbulk::CONSUMER_WARPS) {
        const uint4 wa = ptx::lds128(st + g * sb + 64 * c + 16 * t);
        const uint4 wb = ptx::lds128(st + (g + 8) * sb + 64 * c + 16 * t);
        const uint32_t pa[4] = {wa.x, wa.y, wa.z, wa.w}, pb[4] = {wb.x, wb.y, wb.z, wb.w};
        uint4 x[NTG][2];
#pragma unroll
        for (int i = 0; i < NTG; ++i) {
            const int8_t *xp = xs + (size_t)(8 * i + g) * pitch + 128 * c + 32 * t;
            const bool ok = 8 * i + g < M;
            x[i][0] = ok ? ptx::lds128(xp) : make_uint4(0, 0, 0, 0);
            x[i][1] = ok ? ptx::lds128(xp + 16) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            constexpr uint32_t H = 0xF0F0F0F0u;
            const uint32_t alo = (pa[j] << 4) & H, ahi = pa[j] & H, blo = (pb[j] << 4) & H, bhi = pb[j] & H;
#pragma unroll
            for (int i = 0; i < NTG; ++i) {
                const uint4 &v = x[i][j >> 1];
                mma_s8_16832(acc[i][j & 1], alo, blo, ahi, bhi, (j & 1) ? v.z : v.x, (j & 1) ? v.w : v.y);
            }
        }
    }
}

// J > 0: FUSED, M <= R rows with J units of 8 values per thread and row. J = 0: INT8 rows.
template <bool GLU, int NTG, int R, int J, typename T>
__global__ void __launch_bounds__(DEC_THREADS, 2)
k_mlp_decode(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b, const DecArgs p) {
    constexpr int TOK = 8 * NTG;
    constexpr int CH = GLU ? 8 : 16;  // channels per group of 16 packed rows
    __shared__ DecSmem<NTG> sm;
    extern __shared__ __align__(1024) uint8_t dyn_smem[];
    const DecGeo geo(p.K, p.max_sb);
    const int sb = geo.sb, nst = geo.nst, pitch = geo.pitch, stage_bytes = geo.stage_bytes(), ks = pitch - 16;
    int8_t *xs = reinterpret_cast<int8_t *>(dyn_smem + (size_t)p.ring * stage_bytes);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int groups = (p.N + CH - 1) / CH;
    const int my_groups = (groups - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;
    const int items = my_groups * nst;
    volatile int *abort = &sm.abort;

    if (tid == 0) {
        for (int s = 0; s < p.ring; ++s) {
            ptx::mbar_init(&sm.full[s], 1);
            ptx::mbar_init(&sm.empty[s], dbulk::CONSUMER_WARPS);
        }
        for (int s = 0; s < DEC_RED; ++s) {
            ptx::mbar_init(&sm.rfull[s], dbulk::CONSUMER_WARPS);
            ptx::mbar_init(&sm.rfree[s], 1);
        }
        sm.abort = 0;
        ptx::fence_mbar_init();
    }
    __syncthreads();
    griddep_launch_dependents();

    if (warp == dbulk::CONSUMER_WARPS) {
        // ------------------------------------------------- producer (lane 0)
        int issued = 0;
        auto issue = [&](int it) {
            const int j = it / nst, s = it - j * nst, slot = it % p.ring;
            const int n0 = ((int)blockIdx.x + j * (int)gridDim.x) * CH;
            uint8_t *dst = dyn_smem + (size_t)slot * stage_bytes;
            ptx::mbar_arrive_expect_tx(&sm.full[slot], (uint32_t)stage_bytes);
            ptx::tma_load_2d(dst, &tm_a, s * (sb / 8), n0, &sm.full[slot]);
            if constexpr (GLU) ptx::tma_load_2d(dst + 8 * sb, &tm_b, s * (sb / 8), n0, &sm.full[slot]);
            ++issued;
        };
        const int pre = min(p.ring, items);
        if (lane == 0) {
            ptx::prefetch_tensormap(&tm_a);
            if (p.early)
                for (int it = 0; it < pre; ++it) issue(it);
        }
        __syncwarp();  // a lane waiting in griddepcontrol.wait holds its warp
        griddep_wait();
        if (lane != 0) return;
        for (int it = issued; it < items; ++it) {
            // a slot is free once every consumer warp arrived on its last use
            if (it >= p.ring && !ptx::mbar_wait(&sm.empty[it % p.ring], (uint32_t)(it / p.ring - 1) & 1u, abort)) break;
            issue(it);
        }
        // the block may exit only when every copy it issued has landed
        for (int it = max(0, issued - p.ring); it < issued; ++it)
            ptx::mbar_wait_drain(&sm.full[it % p.ring], (uint32_t)(it / p.ring) & 1u);
        return;
    }

    if (warp == dbulk::CONSUMER_WARPS + 1) {
        // -------------------------------------------------- finishing warp
        // A group's sums over K meet in shared memory; the consumers only leave
        // them there and go on, this warp adds them up and finishes the outputs
        // (channel i % CH, row i / CH), its operands fetched a group ahead.
        constexpr int OUTS = CH * TOK / 32;  // outputs per lane
        const int ch = lane % CH;
        griddep_wait();
        float sa, ba, sc, bb, r[OUTS];
        auto fetch = [&](int j) {
            const int n = min(((int)blockIdx.x + j * (int)gridDim.x) * CH + ch, p.N - 1);
            sa = ld_dep(p.a.sw + n);
            ba = p.a.bias ? ld_dep(p.a.bias + n) : 0.0f;
            sc = GLU ? ld_dep(p.b.sw + n) : 1.0f;
            bb = GLU && p.b.bias ? ld_dep(p.b.bias + n) : 0.0f;
            if (!GLU && p.e.R) {
#pragma unroll
                for (int o = 0; o < OUTS; ++o)
                    r[o] = ld_elem(static_cast<const T *>(p.e.R) +
                                   (size_t)min((32 * o + lane) / CH, p.M - 1) * p.e.ldr + n);
            }
        };
        if (my_groups > 0) fetch(0);
        for (int j = 0; j < my_groups; ++j) {
            const int n = ((int)blockIdx.x + j * (int)gridDim.x) * CH + ch, rb = j % DEC_RED;
            const float ra = __frcp_rn(sa) * 0.0625f, rc = __frcp_rn(sc) * 0.0625f;  // the sums hold 16 x the product
            if (!__all_sync(0xffffffffu, ptx::mbar_wait(&sm.rfull[rb], (uint32_t)(j / DEC_RED) & 1u, abort))) return;
            const float b0 = ba, b1 = bb;
            float res[OUTS];
#pragma unroll
            for (int o = 0; o < OUTS; ++o) res[o] = r[o];
            if (j + 1 < my_groups) fetch(j + 1);
#pragma unroll
            for (int o = 0; o < OUTS; ++o) {
                const int tk = (32 * o + lane) / CH;
                if (tk >= p.M || n >= p.N) continue;
                int32_t ca = 0, cb = 0;
#pragma unroll
                for (int w = 0; w < dbulk::CONSUMER_WARPS; ++w) {
                    ca += sm.red[rb][w][ch][tk];
                    if constexpr (GLU) cb += sm.red[rb][w][8 + ch][tk];
                }
                const float rx = sm.rsx[tk];
                const float z = dequant(__int2float_rn(ca), rx, ra, b0), u = GLU ? dequant(__int2float_rn(cb), rx, rc, b1) : 0.0f;
                float y = act_any(p.act, z);
                if constexpr (GLU) y *= u;
                else if (p.e.R) y += res[o];
                st_elem(static_cast<T *>(p.e.Y) + (size_t)tk * p.e.ldy + n, y);
                if (p.e.Z) {
                    st_elem(static_cast<T *>(p.e.Z) + (size_t)tk * p.e.ldz + n, z);
                    if constexpr (GLU) st_elem(static_cast<T *>(p.e.U) + (size_t)tk * p.e.ldz + n, u);
                }
            }
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&sm.rfree[rb]);
        }
        return;
    }

    // -------------------------------------------------------------- consumers
    const int g = lane >> 2, t = lane & 3;
    griddep_wait();
    if constexpr (J > 0) {
        dec_quantize<R, J, T>(p, ks, pitch, xs, sm.part, sm.rsx, tid);
    } else {
        const int per = ks / 16, have = min(p.ldq, ks) / 16;
#pragma unroll 4
        for (int i = tid; i < p.M * per; i += DEC_CONSUMERS) {
            const int r = i / per, c = i - r * per;
            *reinterpret_cast<uint4 *>(xs + (size_t)r * pitch + 16 * c) =
                c < have ? ld_dep_v4(p.Xq + (size_t)r * p.ldq + 16 * c) : make_uint4(0, 0, 0, 0);
        }
        if (tid < p.M) sm.rsx[tid] = __frcp_rn(ld_dep(p.sx + tid));
    }
    ptx::bar_sync(1, DEC_CONSUMERS);

    for (int j = 0; j < my_groups; ++j) {
        int32_t acc[NTG][2][4];
#pragma unroll
        for (int i = 0; i < NTG; ++i)
#pragma unroll
            for (int q = 0; q < 2; ++q) acc[i][q][0] = acc[i][q][1] = acc[i][q][2] = acc[i][q][3] = 0;
        for (int s = 0; s < nst; ++s) {
            const int it = j * nst + s, slot = it % p.ring;
            if (!__all_sync(0xffffffffu, ptx::mbar_wait(&sm.full[slot], (uint32_t)(it / p.ring) & 1u, abort))) return;
            dec_stage<NTG>(acc, dyn_smem + (size_t)slot * stage_bytes, sb, xs + 2 * sb * s, pitch, p.M, g, t, warp);
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&sm.empty[slot]);
        }
        const int rb = j % DEC_RED;
        if (!__all_sync(0xffffffffu, ptx::mbar_wait(&sm.rfree[rb], ((uint32_t)(j / DEC_RED) & 1u) ^ 1u, abort))) return;
        // C fragments: rows g, g + 8, columns 2t, 2t + 1
#pragma unroll
        for (int i = 0; i < NTG; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                sm.red[rb][warp][g + 8 * (q >> 1)][8 * i + 2 * t + (q & 1)] = acc[i][0][q] + acc[i][1][q];
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&sm.rfull[rb]);
    }
}

// ------------------------------------------------------------- host side ---

struct DecPlan {
    bool ok;        // the kernel can run the shape
    bool preferred; // and is faster than the tensor-core form
    int units;      // FUSED: units of 8 values per thread and row (1, 2, 4, 8), 0: INT8 rows
    int rows;       // FUSED: M rounded up to a power of two
    int grid, ring, max_sb;
    size_t smem;
};

// Two blocks per SM where their rings hold at least 48 KB each (one block's 8
// warps alone do not keep up with the stream: 20.5 against 15.4 us at M = 8,
// K = 4096, N = 11008, gated), one otherwise or where there are no more groups
// than SMs. Stages of up to 2048 or 1024 packed bytes per row, whichever
// leaves more bytes in flight beside the activation rows. FUSED while all rows are at most eight
// units of 8 values per thread (2048 values a unit): beyond that every block's
// pass over X costs more than the row pass's launch.
inline DecPlan dec_plan(int M, int K, int N, int ch, int sms) {
    DecPlan d = {};
    if (M < 1 || M > DEC_TOK || K > dbulk::X16_MAX_K) return d;
    const long long groups = (N + ch - 1) / ch;
    const long long fixed = (M <= 8 ? dec_static<1>() : dec_static<2>()) + 1024;
    for (int per_sm = groups > sms ? 2 : 1; per_sm >= 1 && !d.ok; --per_sm) {
        long long best = per_sm == 2 ? 48 * 1024 - 1 : 0;
        for (int max_sb = 2048; max_sb >= 1024; max_sb /= 2) {
            const DecGeo geo(K, max_sb);
            const long long xs = (long long)M * geo.pitch;
            const long long grid = groups < (long long)per_sm * sms ? groups : (long long)per_sm * sms;
            const long long items = (groups + grid - 1) / grid * geo.nst;
            const long long fit = (DEC_SM_SMEM / per_sm - fixed - xs) / geo.stage_bytes();
            long long ring = fit < DEC_RING ? fit : DEC_RING;
            ring = ring < items ? ring : items;
            if (fit < 2 || fit * geo.stage_bytes() <= best) continue;
            best = fit * geo.stage_bytes();
            d.ok = true;
            // Past 8 rows (two MMAs a chunk) one block per SM falls behind the
            // tensor cores on long layers: 39.7 against 22.6 us at M = 16,
            // K = 4096, N = 28672; two blocks (22.9 / 23.0 at M = 9) or a layer
            // of two groups per SM (10.7 / 12.4 at N = 4096) do not.
            d.preferred = M <= 8 || per_sm == 2 || groups <= 2LL * sms;
            d.grid = (int)grid;
            d.ring = (int)ring;
            d.max_sb = max_sb;
            d.smem = (size_t)(ring * geo.stage_bytes() + xs);
            int j = 1;
            while (j * 8 * DEC_CONSUMERS < geo.pitch - 16) j *= 2;
            d.rows = M <= 1 ? 1 : M <= 2 ? 2 : M <= 4 ? 4 : 8;
            d.units = M <= 8 && j * d.rows <= 8 ? j : 0;
        }
    }
    return d;
}

template <bool GLU, int NTG, int R, int J, typename T>
w4a8_status launch_decode(const DecPlan &d, DecArgs p, int ldp, cudaStream_t s) {
    auto kern = k_mlp_decode<GLU, NTG, R, J, T>;
    constexpr int limit = 227 * 1024 - dec_static<NTG>();
    if (!raise_smem_limit(reinterpret_cast<const void *>(kern), limit)) return W4A8_ERR_CUDA;
    const DecGeo geo(p.K, d.max_sb);
    CUtensorMap ta, tb;
    auto map = [&](CUtensorMap *m, const uint8_t *W) {  // packed rows as 8-byte elements
        return tc::make_map_2d(m, CU_TENSOR_MAP_DATA_TYPE_UINT64, W, (uint64_t)(geo.kp / 8), (uint64_t)p.N,
                               (uint64_t)ldp, (uint32_t)(geo.sb / 8), GLU ? 8 : 16, CU_TENSOR_MAP_SWIZZLE_NONE);
    };
    if (!map(&ta, p.a.Wp) || !map(&tb, p.b.Wp)) return W4A8_ERR_CUDA;
    p.ring = d.ring;
    p.max_sb = d.max_sb;
    return from_cuda(launch_pdl(kern, dim3(d.grid), dim3(DEC_THREADS), d.smem, s, ta, tb, p));
}

template <bool GLU, typename T>
w4a8_status launch_decode_any(const DecPlan &d, const DecArgs &p, int ldp, cudaStream_t s) {
#define W4A8_DEC(R, J) \
    if (d.rows == R && d.units == J) return launch_decode<GLU, 1, R, J, T>(d, p, ldp, s);
    W4A8_DEC(1, 1) W4A8_DEC(1, 2) W4A8_DEC(1, 4) W4A8_DEC(1, 8) W4A8_DEC(2, 1) W4A8_DEC(2, 2) W4A8_DEC(2, 4)
    W4A8_DEC(4, 1) W4A8_DEC(4, 2) W4A8_DEC(8, 1)
#undef W4A8_DEC
    if (p.M <= 8) return launch_decode<GLU, 1, 1, 0, T>(d, p, ldp, s);
    return launch_decode<GLU, 2, 1, 0, T>(d, p, ldp, s);
}

}  // namespace mlp
}  // namespace w4a8
