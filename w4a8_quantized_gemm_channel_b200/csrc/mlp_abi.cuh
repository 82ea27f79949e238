// Entry points of the MLP operators (w4a8_linear_act, w4a8_glu and their
// gradients): argument checks, workspace layout, kernel selection, launches.
// Included at the end of w4a8_abi.cu, whose helpers it uses.
#pragma once

#include <climits>

#include "mlp_gemm.cuh"
#include "mlp_decode.cuh"

namespace w4a8 {
namespace {

inline bool io_bf16(unsigned flags) { return (flags & W4A8_IO_BF16) != 0; }
inline size_t io_size(unsigned flags) { return io_bf16(flags) ? 2 : 4; }
inline bool io_aligned(const void *p, unsigned flags) {
    return (reinterpret_cast<uintptr_t>(p) & (io_size(flags) - 1)) == 0;
}
// Rows whose eight-element pieces are 16-byte aligned.
inline bool io_vec(const void *p, int ld, unsigned flags) {
    return aligned16(p) && ((size_t)ld * io_size(flags)) % 16 == 0;
}

// What every MLP call, and the size query for it, checks about sizes and flags.
w4a8_status check_sizes(int M, int K, int N, unsigned flags) {
    if (M < 0 || K < 1 || K > W4A8_ACT_MAX_K || N < 1) return W4A8_ERR_INVALID_ARG;
    if (M >= 1 << 30 || N >= 1 << 30) return W4A8_ERR_INVALID_ARG;  // two of them fit an int
    if (flags & ~(W4A8_IO_BF16 | W4A8_STATIC_WEIGHTS | W4A8_PATH_MASK)) return W4A8_ERR_INVALID_ARG;
    return W4A8_OK;
}
// What every MLP call checks besides, and about one projection.
w4a8_status check_mlp(int M, int K, int N, int ldp, int act, unsigned flags) {
    if (check_sizes(M, K, N, flags) != W4A8_OK) return W4A8_ERR_INVALID_ARG;
    if (ldp < (K + 1) / 2 || ldp % 16 != 0) return W4A8_ERR_INVALID_ARG;
    if (act < W4A8_ACT_NONE || act > W4A8_ACT_GELU_TANH) return W4A8_ERR_INVALID_ARG;
    return W4A8_OK;
}
w4a8_status check_proj(const uint8_t *Wp, const float *sw, const float *vec) {
    if (!Wp || !sw || !aligned16(Wp) || !aligned4(sw) || (vec && !aligned4(vec))) return W4A8_ERR_INVALID_ARG;
    return W4A8_OK;
}
// The gradient's operand rows hold a segment per projection, N rounded up to
// the product's step of 128; the kernels count their columns in an int.
bool grad_rows_fit(int N, int segs) { return ((long long)N + 127) / 128 * 128 * segs <= INT_MAX; }
// A row array of `cols` columns: required ones must be there when there are rows.
bool rows_ok(const void *p, int ld, int cols, bool required, int M, unsigned flags) {
    if (!p) return !required || M == 0;
    return ld >= cols && io_aligned(p, flags);
}

// One instantiation per activation and row type: f<ACT, T>().
template <typename F>
w4a8_status by_act(int act, F &&f) {
    switch (act) {
        case W4A8_ACT_NONE: return f(std::integral_constant<int, W4A8_ACT_NONE>{});
        case W4A8_ACT_RELU: return f(std::integral_constant<int, W4A8_ACT_RELU>{});
        case W4A8_ACT_SILU: return f(std::integral_constant<int, W4A8_ACT_SILU>{});
        case W4A8_ACT_GELU: return f(std::integral_constant<int, W4A8_ACT_GELU>{});
        default: return f(std::integral_constant<int, W4A8_ACT_GELU_TANH>{});
    }
}

// ----------------------------------------------------------------- forward ---
template <typename T>
w4a8_status launch_quant_rows(const void *X, int M, int K, int ldx, const Workspace &ws, unsigned flags,
                              cudaStream_t s) {
    const int vec = io_vec(X, ldx, flags);
    const dim3 grid(M < 65535 ? M : 65535);
    const T *x = static_cast<const T *>(X);
    cudaError_t e;
    if (K <= 2048)
        e = launch_pdl(mlp::k_quant_rows<T, 128, 2>, grid, dim3(128), 0, s, x, M, K, ldx, ws.xq, ws.ldq, ws.sx, vec);
    else if (K <= 4096)
        e = launch_pdl(mlp::k_quant_rows<T, 256, 2>, grid, dim3(256), 0, s, x, M, K, ldx, ws.xq, ws.ldq, ws.sx, vec);
    else
        e = launch_pdl(mlp::k_quant_rows<T, 256, 6>, grid, dim3(256), 0, s, x, M, K, ldx, ws.xq, ws.ldq, ws.sx, vec);
    return from_cuda(e);
}

// Forward workspace: the INT8 rows and scales, then the partial tiles' slots.
uint8_t *ws_parts(const Workspace &ws, int M) {
    const uintptr_t end = reinterpret_cast<uintptr_t>(ws.sx) + sizeof(float) * (size_t)M;
    return reinterpret_cast<uint8_t *>((end + 255) & ~uintptr_t(255));
}
size_t forward_workspace(int M, int K, int N, bool glu) {
    return workspace_bytes_for(M, K, nullptr) + mlp::forward_plan(M, K, N, glu).part_bytes + 256;
}

// Few products, and short sums: the CUDA-core forms, whose launch is the
// cheapest. One thread walks a whole sum there, about 6.4 us per 1000 k and
// 130 us per 1000 n of a gradient, so long ones go to the other forms.
// Measured in a graph, CUDA cores against the decode (M <= 16) or tensor-core
// form, float32. Forward: M 1, N 10: 2.4 / 2.5 us at K 128, 3.3 / 2.4 at K 256,
// 27.5 / 3.2 at K 4096; M 4, N 4: 3.2 / 3.4 at K 256, 4.5 / 3.4 at K 512; M 8, N 4:
// 4.6 / 5.1 at K 512, 7.2 / 5.1 at K 1024; M 20, N 4: 4.7 / 6.7 at K 512. Gradient,
// M 1, K 10: 5.4 / 6.7 us at N 16, 7.7 / 6.5 at N 32, 842 / 18 at N 6500; M 128, K 2:
// 5.7 / 8.3 at N 16, 7.8 / 8.3 at N 32, 11.9 / 8.3 at N 64.
bool mlp_tiny(int M, int K, int N, int segs) { return (double)M * N * K * segs < 65536.0; }
bool forward_tiny(int M, int K, int N, int segs) {
    return mlp_tiny(M, K, N, segs) && K <= (M <= 2 ? 128 : M <= 4 ? 256 : 512);
}
bool grad_tiny(int M, int K, int N, int segs) { return mlp_tiny(M, K, N, segs) && segs * (long long)N <= 24; }

template <bool GLU, typename T>
w4a8_status mlp_forward(const void *X, int M, int K, int ldx, const mlp::Proj &a, const mlp::Proj &b, int ldp, int N,
                        int act, const mlp::EpiArgs &ea, unsigned flags, const Workspace &ws, cudaStream_t s) {
    const int sms = device_info().sm_count;
    const bool early = (flags & W4A8_STATIC_WEIGHTS) != 0;
    unsigned path = flags & W4A8_PATH_MASK;
    const mlp::DecPlan dec = mlp::dec_plan(M, K, N, GLU ? 8 : 16, sms);
    if (path == W4A8_PATH_AUTO)
        path = forward_tiny(M, K, N, GLU ? 2 : 1) ? W4A8_PATH_GENERIC
               : dec.preferred                         ? W4A8_PATH_DECODE
                                                       : W4A8_PATH_TC;
    if (path != W4A8_PATH_GENERIC && path != W4A8_PATH_DECODE && path != W4A8_PATH_TC) return W4A8_ERR_UNSUPPORTED;
    if (path == W4A8_PATH_DECODE && !dec.ok) return W4A8_ERR_UNSUPPORTED;
    if (path != W4A8_PATH_GENERIC && tc::encode_fn() == nullptr) return W4A8_ERR_UNSUPPORTED;
    const bool fused = path == W4A8_PATH_DECODE ? dec.units > 0
                                                : path == W4A8_PATH_GENERIC && K <= mlp::SIMT_FUSED_K;
    w4a8_status st = W4A8_OK;
    if (!fused) st = launch_quant_rows<T>(X, M, K, ldx, ws, flags, s);
    if (st != W4A8_OK) return st;
    if (path == W4A8_PATH_DECODE) {
        // behind the row pass the weights are settled: it lets dependents
        // start only once all earlier work has completed
        const mlp::DecArgs p = {X, ws.xq, ws.sx, ldx, ws.ldq, io_vec(X, ldx, flags), M, K, N, a, b, ea, act, 0,
                                early || !fused};
        st = mlp::launch_decode_any<GLU, T>(dec, p, ldp, s);
        if (st != W4A8_OK) return st;
        t_last_path = W4A8_PATH_DECODE;
        t_last_launches = fused ? 1 : 2;
        t_last_kernel = "k_mlp_decode";
        return W4A8_OK;
    }
    if (path == W4A8_PATH_TC) {
        const int stages = (K + 255) / 256;
        const mlp::PairPlan plan = mlp::forward_plan(M, K, N, GLU);
        const mlp::PairArgs p = {M, N, K, stages, stages, ws.sx, a, b, ea, act, 0, nullptr};
        const mlp::PairCall c = {a.Wp, b.Wp, N, K, ldp, ws.xq, M, ws.ldq};
        st = by_act(act, [&](auto A) {
            return mlp::launch_pair_any<GLU ? mlp::FWD_GLU : mlp::FWD_LINEAR, decltype(A)::value, T>(
                plan, p, c, ws_parts(ws, M), s);
        });
        if (st != W4A8_OK) return st;
        t_last_path = W4A8_PATH_TC;
        t_last_launches = plan.split ? 3 : 2;
        t_last_kernel = "k_mlp_pair";
        return W4A8_OK;
    }
    st = by_act(act, [&](auto A) {
        const dim3 grid((N + 127) / 128, M < 65535 ? M : 65535);
        auto kern = fused ? mlp::k_mlp_simt<GLU, true, decltype(A)::value, T>
                          : mlp::k_mlp_simt<GLU, false, decltype(A)::value, T>;
        return from_cuda(launch_pdl(kern, grid, dim3(128), 0, s, static_cast<const T *>(X), ldx,
                                    (int)io_vec(X, ldx, flags), ws.xq, M, K, ws.ldq, ws.sx, a, b, ldp, N, ea));
    });
    if (st != W4A8_OK) return st;
    t_last_path = W4A8_PATH_GENERIC;
    t_last_launches = fused ? 1 : 2;
    t_last_kernel = "k_mlp_simt";
    return W4A8_OK;
}

// Checks shared by the two forward calls once their own are done; `run` on OK.
template <bool GLU>
w4a8_status mlp_forward_call(const void *X, int M, int K, int ldx, const mlp::Proj &a, const mlp::Proj &b, int ldp,
                             int N, int act, const mlp::EpiArgs &ea, unsigned flags, void *workspace,
                             size_t workspace_bytes, cudaStream_t s) {
    if (M == 0) { t_last_launches = 0; t_last_kernel = ""; return W4A8_OK; }
    if (!workspace || !aligned16(workspace)) return W4A8_ERR_WORKSPACE;
    if (workspace_bytes < w4a8_act_workspace_size(M, K, N, GLU ? 2 : 1, flags)) return W4A8_ERR_WORKSPACE;
    if (!device_info().ok) return W4A8_ERR_UNSUPPORTED;
    const Workspace ws = carve_workspace(workspace, M, K);
    return io_bf16(flags) ? mlp_forward<GLU, __nv_bfloat16>(X, M, K, ldx, a, b, ldp, N, act, ea, flags, ws, s)
                          : mlp_forward<GLU, float>(X, M, K, ldx, a, b, ldp, N, act, ea, flags, ws, s);
}

// --------------------------------------------------------------- gradients ---
// Workspace: the FP16 rows (one plane, two for float32), their powers of two,
// and the bias gradients' partial sums, each on a 256-byte boundary.
struct GradWorkspace {
    int seg;     // columns of a segment: N rounded up to the product's k step
    int planes;
    size_t p_bytes, rs_bytes, part_bytes;
    mlp::PairPlan plan;
    __half *P;
    float *rs, *part;
    void *tiles;    // the product's partial tiles
    size_t total() const { return p_bytes + rs_bytes + part_bytes + plan.part_bytes + 256; }
    void carve(void *base) {
        uintptr_t p = (reinterpret_cast<uintptr_t>(base) + 255) & ~uintptr_t(255);
        P = reinterpret_cast<__half *>(p);
        rs = reinterpret_cast<float *>(p + p_bytes);
        part = reinterpret_cast<float *>(p + p_bytes + rs_bytes);
        tiles = reinterpret_cast<void *>(p + p_bytes + rs_bytes + part_bytes);
    }
};

GradWorkspace grad_layout(int M, int K, int N, int segs, unsigned flags) {
    GradWorkspace g = {};
    g.seg = round_up(N, 128);
    g.planes = io_bf16(flags) ? 1 : 2;
    g.p_bytes = round256((size_t)g.planes * M * segs * g.seg * sizeof(__half));
    g.rs_bytes = round256((size_t)M * sizeof(float));
    g.part_bytes = round256((size_t)((M + mlp::BG_ROWS - 1) / mlp::BG_ROWS) * segs * N * sizeof(float));
    g.plan = mlp::grad_plan(M, K, segs, g.seg, g.planes == 2);
    return g;
}

template <bool GLU, typename T>
w4a8_status mlp_grad(const mlp::GradIn<GLU, T> &in, int M, const uint8_t *Wa, const uint8_t *Wb, int ldp, int K,
                     int act, unsigned flags, void *dX, int lddx, float *dba, float *dbb, const GradWorkspace &ws,
                     cudaStream_t s) {
    constexpr int SEGS = GLU ? 2 : 1;
    constexpr bool LO = std::is_same<T, float>::value;
    const int N = in.N;
    unsigned path = flags & W4A8_PATH_MASK;
    if (path == W4A8_PATH_AUTO) path = grad_tiny(M, K, N, SEGS) ? W4A8_PATH_GENERIC : W4A8_PATH_TC;
    if (path != W4A8_PATH_GENERIC && path != W4A8_PATH_TC) return W4A8_ERR_UNSUPPORTED;
    if (path == W4A8_PATH_TC && tc::encode_fn() == nullptr) return W4A8_ERR_UNSUPPORTED;
    unsigned launches = 0;
    w4a8_status st = by_act(act, [&](auto A) {
        constexpr int ACT = decltype(A)::value;
        if (dba || dbb) {
            const int slices = (M + mlp::BG_ROWS - 1) / mlp::BG_ROWS;
            cudaError_t e = launch_pdl(mlp::k_bias_grad<GLU, ACT, T>,
                                       dim3((N + mlp::BG_COLS - 1) / mlp::BG_COLS, slices < 65535 ? slices : 65535),
                                       dim3(512), 0, s, in, M, ws.part, dba, dbb);
            ++launches;
            if (e == cudaSuccess && slices > 1) {
                e = launch_pdl(mlp::k_bias_grad_sum, dim3((N + 255) / 256, SEGS), dim3(256), 0, s,
                               (const float *)ws.part, slices, SEGS, N, dba, dbb);
                ++launches;
            }
            if (e != cudaSuccess) return (w4a8_status)W4A8_ERR_CUDA;
        }
        const size_t bytes = (size_t)SEGS * ws.seg * sizeof(float);
        const bool held = bytes <= (size_t)mlp::GR_HELD_MAX;
        auto kern = held ? mlp::k_grad_rows<GLU, LO, true, ACT, T> : mlp::k_grad_rows<GLU, LO, false, ACT, T>;
        if (held && !raise_smem_limit(reinterpret_cast<const void *>(kern), mlp::GR_HELD_MAX))
            return (w4a8_status)W4A8_ERR_CUDA;
        return from_cuda(launch_pdl(kern, dim3(M < 65535 ? M : 65535), dim3(mlp::GR_THREADS), held ? bytes : 0, s, in,
                                    M, ws.seg, ws.P, ws.rs));
    });
    if (st != W4A8_OK) return st;
    if (path == W4A8_PATH_TC) {
        const int seg_stages = ws.seg / (LO ? 64 : 128);
        const mlp::PairArgs p = {M, K, N, seg_stages, SEGS * seg_stages, ws.rs, {}, {},
                                 {nullptr, dX, nullptr, nullptr, 0, lddx, 0}, 0, 0, nullptr};
        const mlp::PairCall c = {Wa, Wb, N, K, ldp, ws.P, ws.planes * M, SEGS * ws.seg};
        st = mlp::launch_pair_any<LO ? mlp::BWD_TWO : mlp::BWD_ONE, W4A8_ACT_NONE, T>(ws.plan, p, c, ws.tiles, s);
        if (st != W4A8_OK) return st;
        t_last_path = W4A8_PATH_TC;
        t_last_launches = launches + (ws.plan.split ? 3 : 2);
        t_last_kernel = "k_mlp_pair";
        return W4A8_OK;
    }
    const dim3 grid(((K + 7) / 8 + 127) / 128, M < 65535 ? M : 65535);
    cudaError_t e = launch_pdl(mlp::k_grad_simt<T>, grid, dim3(128), 0, s, (const __half *)ws.P, (const float *)ws.rs,
                               M, N, ws.seg, SEGS, ws.planes, Wa, Wb, ldp, K, static_cast<T *>(dX), lddx);
    if (e != cudaSuccess) return W4A8_ERR_CUDA;
    t_last_path = W4A8_PATH_GENERIC;
    t_last_launches = launches + 2;
    t_last_kernel = "k_grad_simt";
    return W4A8_OK;
}

template <bool GLU>
w4a8_status mlp_grad_call(const void *dY, int M, int N, int lddy, const void *Z, const void *U, int ldz,
                          const uint8_t *Wa, const float *sa, const uint8_t *Wb, const float *sb, int ldp, int K,
                          int act, unsigned flags, void *dX, int lddx, float *dba, float *dbb, void *workspace,
                          size_t workspace_bytes, cudaStream_t s) {
    if (M == 0) {  // no rows: the bias gradients are empty sums
        cudaError_t e = cudaSuccess;
        if (dba) e = cudaMemsetAsync(dba, 0, sizeof(float) * (size_t)N, s);
        if (e == cudaSuccess && dbb) e = cudaMemsetAsync(dbb, 0, sizeof(float) * (size_t)N, s);
        t_last_launches = 0;
        t_last_kernel = "";
        return from_cuda(e);
    }
    if (!workspace || !aligned16(workspace)) return W4A8_ERR_WORKSPACE;
    if (workspace_bytes < w4a8_grad_workspace_size(M, K, N, GLU ? 2 : 1, flags)) return W4A8_ERR_WORKSPACE;
    if (!device_info().ok) return W4A8_ERR_UNSUPPORTED;
    GradWorkspace ws = grad_layout(M, K, N, GLU ? 2 : 1, flags);
    ws.carve(workspace);
    auto run = [&](auto elem) {
        using T = decltype(elem);
        const mlp::GradIn<GLU, T> in = {static_cast<const T *>(dY), static_cast<const T *>(Z),
                                        static_cast<const T *>(U), sa, sb, N, lddy, ldz,
                                        io_vec(dY, lddy, flags) && (!Z || io_vec(Z, ldz, flags)) &&
                                            (!U || io_vec(U, ldz, flags))};
        return mlp_grad<GLU, T>(in, M, Wa, Wb, ldp, K, act, flags, dX, lddx, dba, dbb, ws, s);
    };
    return io_bf16(flags) ? run(__nv_bfloat16()) : run(float());
}

}  // namespace
}  // namespace w4a8

extern "C" {

size_t w4a8_act_workspace_size(int M, int K, int N, int projections, unsigned flags) {
    if (check_sizes(M, K, N, flags) != W4A8_OK || projections < 1 || projections > 2) return 0;
    return forward_workspace(M, K, N, projections == 2);
}

size_t w4a8_grad_workspace_size(int M, int K, int N, int projections, unsigned flags) {
    if (check_sizes(M, K, N, flags) != W4A8_OK || projections < 1 || projections > 2) return 0;
    if (!grad_rows_fit(N, projections)) return 0;
    return grad_layout(M, K, N, projections, flags).total();
}

w4a8_status w4a8_linear_act(const void *X, int M, int K, int ldx, const uint8_t *Wp, int ldp, const float *sw, int N,
                            const float *bias, int act, const void *R, int ldr, unsigned flags, void *Y, int ldy,
                            void *Z, int ldz, void *workspace, size_t workspace_bytes, void *stream) {
    w4a8_status st = check_mlp(M, K, N, ldp, act, flags);
    if (st == W4A8_OK) st = check_proj(Wp, sw, bias);
    if (st != W4A8_OK) return st;
    if (!rows_ok(X, ldx, K, true, M, flags) || !rows_ok(Y, ldy, N, true, M, flags) ||
        !rows_ok(R, ldr, N, false, M, flags) || !rows_ok(Z, ldz, N, false, M, flags))
        return W4A8_ERR_INVALID_ARG;
    const mlp::Proj a = {Wp, sw, bias};
    const mlp::EpiArgs ea = {R, Y, Z, nullptr, ldr, ldy, ldz};
    return mlp_forward_call<false>(X, M, K, ldx, a, a, ldp, N, act, ea, flags, workspace, workspace_bytes,
                                   static_cast<cudaStream_t>(stream));
}

w4a8_status w4a8_glu(const void *X, int M, int K, int ldx, const uint8_t *Wg, const float *sg, const uint8_t *Wu,
                     const float *su, int ldp, int N, const float *bg, const float *bu, int act, unsigned flags,
                     void *H, int ldh, void *G, void *U, int ldgu, void *workspace, size_t workspace_bytes,
                     void *stream) {
    w4a8_status st = check_mlp(M, K, N, ldp, act, flags);
    if (st == W4A8_OK) st = check_proj(Wg, sg, bg);
    if (st == W4A8_OK) st = check_proj(Wu, su, bu);
    if (st != W4A8_OK) return st;
    if (!rows_ok(X, ldx, K, true, M, flags) || !rows_ok(H, ldh, N, true, M, flags) || (!G != !U) ||
        !rows_ok(G, ldgu, N, false, M, flags) || !rows_ok(U, ldgu, N, false, M, flags))
        return W4A8_ERR_INVALID_ARG;
    const mlp::Proj a = {Wg, sg, bg}, b = {Wu, su, bu};
    const mlp::EpiArgs ea = {nullptr, H, G, U, 0, ldh, ldgu};
    return mlp_forward_call<true>(X, M, K, ldx, a, b, ldp, N, act, ea, flags, workspace, workspace_bytes,
                                  static_cast<cudaStream_t>(stream));
}

w4a8_status w4a8_linear_act_grad(const void *dY, int M, int N, int lddy, const void *Z, int ldz, const uint8_t *Wp,
                                 int ldp, const float *sw, int K, int act, unsigned flags, void *dX, int lddx,
                                 float *dbias, void *workspace, size_t workspace_bytes, void *stream) {
    w4a8_status st = check_mlp(M, K, N, ldp, act, flags);
    if (st == W4A8_OK) st = check_proj(Wp, sw, dbias);
    if (st != W4A8_OK) return st;
    if (act == W4A8_ACT_NONE) Z = nullptr;
    if (!rows_ok(dY, lddy, N, true, M, flags) || !rows_ok(Z, ldz, N, act != W4A8_ACT_NONE, M, flags) ||
        !rows_ok(dX, lddx, K, true, M, flags))
        return W4A8_ERR_INVALID_ARG;
    return mlp_grad_call<false>(dY, M, N, lddy, Z, nullptr, ldz, Wp, sw, Wp, sw, ldp, K, act, flags, dX, lddx, dbias,
                                nullptr, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

w4a8_status w4a8_glu_grad(const void *dH, int M, int N, int lddh, const void *G, const void *U, int ldgu,
                          const uint8_t *Wg, const float *sg, const uint8_t *Wu, const float *su, int ldp, int K,
                          int act, unsigned flags, void *dX, int lddx, float *dbg, float *dbu, void *workspace,
                          size_t workspace_bytes, void *stream) {
    w4a8_status st = check_mlp(M, K, N, ldp, act, flags);
    if (st == W4A8_OK) st = check_proj(Wg, sg, dbg);
    if (st == W4A8_OK) st = check_proj(Wu, su, dbu);
    if (st != W4A8_OK) return st;
    if (!grad_rows_fit(N, 2)) return W4A8_ERR_INVALID_ARG;
    if (!rows_ok(dH, lddh, N, true, M, flags) || !rows_ok(G, ldgu, N, true, M, flags) ||
        !rows_ok(U, ldgu, N, true, M, flags) || !rows_ok(dX, lddx, K, true, M, flags))
        return W4A8_ERR_INVALID_ARG;
    return mlp_grad_call<true>(dH, M, N, lddh, G, U, ldgu, Wg, sg, Wu, su, ldp, K, act, flags, dX, lddx, dbg, dbu,
                               workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
