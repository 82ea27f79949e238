// Tensor-core form of the MLP operators: a CTA pair (tcgen05.mma cta_group::2)
// computes tiles of 256 weight-side rows x NT tokens with both operands in
// shared memory. One kernel serves both directions:
//
//  forward   D[channel][token] = sum_k 16 q[n][k] xq[m][k], kind::i8, INT32.
//            A: widened codes, k-major; B: the INT8 rows, k-major.
//            Epilogue: dequantize, bias, activation, residual; or for the
//            gated form both projections of a channel meet in registers.
//  gradient  D[k][token] = sum_n q[n][k] P[m][n], kind::f16, float32.
//            A: the codes in FP16, MN-major: a packed row holds one n and
//            runs along k, which is D's row axis, so the one stored copy of
//            the weights serves both directions without a transpose; B: the
//            scaled FP16 gradient rows (k_grad_rows), n-major. For float32
//            rows a second B tile holds the low parts and shares the
//            widened weights.
//
// Bound: the tensor pipe at many tokens, the packed weights' stream at few.
//
// Why both operands sit in shared memory (256 tokens and the gradient; see
// Shape::A_TMEM for the others). With the widened weights in TMEM
// the accumulators and the weight slots share its 512 columns, which caps the
// tile at 160 tokens, and the stores into TMEM slow the MMAs down. Here two
// 256-column accumulators fill TMEM, an MMA is 128 tensor cycles long, and per
// SM and 128 cycles the pair moves 20 KB (forward; 18 KB gradient) through
// shared memory: A and B reads of 4 KB each, 4 KB of B arriving, 2 KB (1 KB) of
// packed weights in and out, 4 KB of widened weights written.
//
// Per CTA: 128 rows of A and half of the tile's tokens. Three rings: packed
// weights and tokens (TMA, freed by the widening and by the MMAs), widened
// weights. Warp 0 loads weights, warp 2 tokens, warp 1 issues the MMAs (in the
// leader), warps 4-11 widen, warps 12-19 run the epilogue of one tile while the
// next one's MMAs run (two accumulators), warp 3 stores what they stage. No load
// is multicast. Every wait is bounded, as in gemm_tc_pair.cuh, whose pair
// protocol this follows.
//
// Measured on B200 (product alone, M = 2048): gated K = 8192, N = 28672 560 us,
// 3434 TOPS; gated K = 4096, N = 11008 119 us, 3116 TOPS; linear K = 11008,
// N = 4096 65 us, 2847 TOPS (1.73 rounds of tiles in two); gradient of the same
// layer 123 us, 1502 TFLOP/s.
//
// Gated rows. The 32 TMEM lanes of an epilogue warp hold 16 gate and the same
// 16 up channels (the widening warps place the rows so), and one shuffle per
// two outputs brings a channel's pair together: lanes 0-15 finish a unit's first
// 8 tokens, lanes 16-31 the others.
#pragma once

#include "gemm_tc_pair.cuh"
#include "mlp_act.cuh"
#include "mlp_simt.cuh"

namespace w4a8 {
namespace mlp {

enum { FWD_LINEAR = 0, FWD_GLU = 1, BWD_ONE = 2, BWD_TWO = 3 };  // BWD_TWO: two planes of B (float32 rows)

constexpr int ROWS_CTA = 128;                  // A rows per CTA
constexpr int SUB_BYTES = ROWS_CTA * 128;      // widened sub-tile: 128 rows x 128 k INT8, or 128 k x 64 n FP16
constexpr int EPI_SMEM = 32768;                // output staging
constexpr int CONV_GROUPS = 2, GROUP_WARPS = 4;
constexpr int CONV_WARPS = CONV_GROUPS * GROUP_WARPS;
constexpr int FIRST_CONV = 4, FIRST_EPI = FIRST_CONV + CONV_WARPS;
constexpr int EPI_GROUPS = 2;                  // warpgroups of the epilogue, units in turn
constexpr int UNIT = 16;                       // tokens of an epilogue unit
constexpr int PAIR_THREADS = 32 * (FIRST_EPI + 4 * EPI_GROUPS);
// named barriers: all epilogue warps; a group; a group's staging set free, written
constexpr int BAR_EPI = 1, BAR_GROUP = 2, BAR_FREE = 4, BAR_STAGED = 8;

// A stage is 8 MMAs: two sub-tiles of the contraction (128 k, or 64 n, each),
// or one sub-tile against two planes. (With stages of 4 MMAs the issuing
// thread's wait and commit per stage left the pipe idle a fifth of the time.)
template <int MODE, int NT>
struct Shape {
    static constexpr bool FWD = MODE == FWD_LINEAR || MODE == FWD_GLU;
    static constexpr int PLANES = MODE == BWD_TWO ? 2 : 1;
    static constexpr int SUBS = 2 / PLANES;
    static constexpr int SUB = FWD ? 128 : 64;                  // contraction per sub-tile
    static constexpr int STEP = SUBS * SUB;                     // contraction per stage
    static constexpr int P_SUB = FWD ? 128 * 64 : 64 * 64;      // packed bytes per sub-tile
    static constexpr int P_BYTES = SUBS * P_SUB;
    static constexpr int A_BYTES = SUBS * SUB_BYTES;
    // Float32 gradients: an accumulator takes this many stages (256 n) and the
    // epilogue adds it to a sum in registers, rounded to nearest. The tensor
    // core's own adder truncates, an error that grows with the length of the
    // sum (1.4e-9 of the result per n: 1.8e-6 at 1001 n, against 0.5e-6 for
    // rounded additions).
    static constexpr int CHUNK = PLANES == 2 ? 4 : 1 << 30;
    static constexpr int B_TILE = NT / 2 * 128;                 // one sub-tile or plane of the tokens
    static constexpr int B_BYTES = 2 * B_TILE;
    // Where the widened weights go. With few tokens the MMAs of a stage read as
    // much of A as with many, and A's way through shared memory (written and
    // read, 64 KB a stage) is most of its traffic and sets the pace: 600 ns a
    // stage with 64 tokens. The accumulators then leave TMEM free, so the
    // forward forms of 128 and 64 tokens keep A there (tcgen05.st, no shared
    // memory). The gradient's A is MN-major, which only shared memory can hold.
    static constexpr bool A_TMEM = FWD && NT < 256;
    static constexpr int A_COLS = STEP / 4;                     // TMEM columns of a stage of A
    static constexpr int D_COLS = A_TMEM ? NT : 256;            // columns per accumulator
    // Slots per ring: widened stages, tokens, and as many of packed weights as
    // fit, up to eight: their loads come from HBM. (Two widened stages instead
    // of three cost the gradient a fifth at 64 and 128 tokens.)
    static constexpr int A_SLOTS = A_TMEM ? 4 : SUBS == 2 && NT == 256 ? 2 : 3;
    static constexpr int B_SLOTS = A_TMEM ? 4 : 3;
    static constexpr int A_SMEM = A_TMEM ? 0 : A_SLOTS * A_BYTES;
    static constexpr int REST = 232448 - 1024 - EPI_SMEM - 2048 - A_SMEM - B_SLOTS * B_BYTES - (A_TMEM ? 1024 : 0);
    static constexpr int P_SLOTS = REST / P_BYTES < 8 ? REST / P_BYTES : 8;
    static_assert(!A_TMEM || 2 * NT + A_SLOTS * A_COLS <= 512, "TMEM budget");
    static_assert(P_SLOTS >= 2, "packed stages");
    // Widening: both groups on every stage (half each), which has a stage
    // ready soonest, or, where the MMAs of a stage are shorter than its
    // widening, the groups on every second stage, which hides the latencies of
    // one behind the other.
    static constexpr bool TURNS = NT < 256;
    static constexpr int WARPS_PER_STAGE = TURNS ? GROUP_WARPS : CONV_WARPS;
    static_assert(B_SLOTS >= A_SLOTS && P_SLOTS >= A_SLOTS, "A-slot reuse waits on a token slot's barrier");
};

template <int MODE, int NT>
struct alignas(1024) PairSmem {
    using S = Shape<MODE, NT>;
    uint8_t b[S::B_SLOTS][S::B_BYTES];
    uint8_t a[S::A_TMEM ? 1 : S::A_SLOTS][S::A_TMEM ? 1024 : S::A_BYTES];
    uint8_t packed[S::P_SLOTS][S::P_BYTES];
    uint8_t epi[EPI_SMEM];
    uint64_t pfull[S::P_SLOTS];   // packed weights landed
    uint64_t pfree[S::P_SLOTS];   // packed weights read (the stage's widening warps)
    uint64_t bfull[S::B_SLOTS];   // this CTA's tokens landed
    uint64_t empty[S::B_SLOTS];   // MMAs of the stage finished (both CTAs)
    uint64_t ready[S::A_SLOTS];   // leader: both CTAs' operands there (their widening warps)
    uint64_t acc_full[2];         // accumulator ready (both CTAs)
    uint64_t acc_empty[2];        // leader: both CTAs' epilogues drained (16 warps)
    uint64_t done;                // every MMA finished (both CTAs)
    alignas(16) float tok[NT];    // 1/sx (forward) or the row's power of two
    uint32_t tmem_base;
    int abort;
    int stop;                     // the epilogue gave up
    uint32_t sink[CONV_WARPS];    // see give_back
};

struct PairArgs {
    int M;              // tokens
    int N;              // rows of D: channels per projection, or K of the gradient
    int depth;          // contraction per segment: K, or the gradient's N
    int seg_stages;     // stages per segment
    int stages;         // stages per tile (one segment, or two: the gated gradient)
    const float *tok;   // sx, or the rows' powers of two
    Proj a, b;
    EpiArgs e;          // gradient: Y = dX
    int act, tma_out;
    uint32_t *parts;    // split calls: accumulators of partial tiles, else null
};

// The tiles' stages in one row, tile after tile, as the pairs share them out.
// Whole tiles in turn; or, split, an equal run of stages per pair, whose first
// and last tiles may be partial: their accumulators go to the pair's two
// slots (2 pair: the run's first segment, 2 pair + 1: its last) and
// k_mlp_join adds them up and finishes the tile.
struct Run {
    int tile, s0, s1;            // the current segment: stages [s0, s1) of a tile
    long long at, end;           // split: position in the row, the run's end
    int stages, num_tiles, step;
    bool split, first;
    __device__ __forceinline__ Run(const PairArgs &p, int num_tiles_, int pair, int npairs)
        : stages(p.stages), num_tiles(num_tiles_), step(npairs), split(p.parts != nullptr), first(true) {
        const long long all = (long long)num_tiles_ * p.stages;
        at = split ? all * pair / npairs : (long long)pair * p.stages;
        end = split ? all * (pair + 1) / npairs : all;
        locate();
    }
    __device__ __forceinline__ void locate() {
        tile = (int)(at / stages);
        s0 = (int)(at - (long long)tile * stages);
        s1 = split && end - at < stages - s0 ? s0 + (int)(end - at) : stages;
    }
    __device__ __forceinline__ bool valid() const { return at < end; }
    __device__ __forceinline__ bool partial() const { return s1 - s0 != stages; }
    __device__ __forceinline__ int slot(int pair) const { return 2 * pair + (first ? 0 : 1); }
    __device__ __forceinline__ void next() {
        at += split ? s1 - s0 : (long long)step * stages;
        first = false;
        if (valid()) locate();
    }
    // all stages of the run
    __device__ __forceinline__ int total() const {
        return split ? (int)(end - at) : (int)((end - at + (long long)step * stages - 1) / ((long long)step * stages)) * stages;
    }
};

// ---- the MMA with both operands in shared memory ----
template <bool FWD>
__device__ __forceinline__ void mma_ss2(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    if constexpr (FWD)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
            "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
            "r"(accumulate)
            : "memory");
}

// Instruction descriptor of kind::f16: D float32 (bits 4-5 = 1), A and B FP16
// (0), A MN-major (bit 15), B k-major, N >> 3 and M >> 4 as for kind::i8.
__host__ __device__ constexpr uint32_t idesc_f16_mn(int m, int n) {
    return (1u << 4) | (1u << 15) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// Shared-memory descriptor of the MN-major FP16 operand in 128-byte swizzled
// rows: a row is 64 elements along M for one n, eight rows (n) an atom of
// 1024 bytes, the next 64 elements along M `block` bytes further.
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr, uint32_t block) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)((block >> 4) & 0x3FFFu) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

// One lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t v;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(v));
    return v != 0;
}
// A bounded wait of the whole warp with one outcome for all its lanes.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort) {
    if (__all_sync(0xffffffffu, ptx::mbar_try_wait(bar, parity))) return true;
    return __all_sync(0xffffffffu, ptx::mbar_wait(bar, parity, abort));
}
// Untiled bulk store of this CTA's shared memory (16-byte aligned, a multiple of 16 bytes).
__device__ __forceinline__ void bulk_s2g(void *dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(ptx::smem_addr(src)),
                 "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void bar_arrive(int id, int count) {
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(count) : "memory");
}
__device__ __forceinline__ void bulk_wait_read_0() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void sts128(void *p, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(ptx::smem_addr(p)), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}

// ---------------------------------------------------------------- widening ---
// A thread's 16-byte pieces (32 codes) of a stage, in two steps: the loads and
// the widening with its stores. A packed sub-tile is a 64-byte swizzled box
// (16-byte chunk c of row s at chunk c ^ ((s >> 1) & 3)); widened sub-tiles
// are 128-byte swizzled.
//
// Forward: half g of a stage is sub-tile g, a thread has one A row r of it.
// Nibbles stay in the high half of their byte (16 q), in the order the INT8
// rows are stored in.
// Gated: A rows 32 w + 0..15 are gate channels 16 w + .., 32 w + 16..31 the
// same up channels (the packed tile holds 64 gate rows, then 64 up rows).
//
// Gradient: a thread takes chunks c of packed row n (one n, 128 k): c = tid / 64
// and that + 2 of sub-tile g (half g), or with two planes (one sub-tile)
// c = 2 g + tid / 64.
// Nibble u of q + 8 is put under the FP16 exponent of 1024 (1024 + u, exact)
// and 1032 is subtracted. Masking words of eight codes gives them in the order
// k0 k4 k1 k5 k2 k6 k3 k7, undone by the epilogue's row index.
template <int MODE>
constexpr int pieces() { return MODE == BWD_TWO ? 1 : MODE == BWD_ONE ? 2 : 4; }

// A load done exactly once: an ordinary one might be repeated at its use
// instead of keeping the registers, after its slot has been given back.
__device__ __forceinline__ uint4 lds128_once(const void *p) {
    uint4 v;
    asm volatile("ld.volatile.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(ptx::smem_addr(p))
                 : "memory");
    return v;
}

// WHOLE: the group takes the whole stage, its other half's pieces after its own.
template <int MODE, bool WHOLE>
__device__ __forceinline__ void load_pieces(uint4 (&v)[pieces<MODE>() * (WHOLE ? 2 : 1)], const uint8_t *packed, int g,
                                            int tid) {
#pragma unroll
    for (int h = 0; h < (WHOLE ? 2 : 1); ++h) {
        const int half = WHOLE ? h : g;
        if constexpr (MODE == FWD_LINEAR || MODE == FWD_GLU) {
            const int r = tid, s = MODE == FWD_GLU ? ((r & 16) << 2) + ((r >> 5) << 4) + (r & 15) : r;
            const uint8_t *row = packed + half * (128 * 64) + s * 64;
#pragma unroll
            for (int c = 0; c < 4; ++c) v[4 * h + c] = lds128_once(row + 16 * (c ^ ((s >> 1) & 3)));
        } else {
            const int n = tid & 63, c = tid >> 6;
            const uint8_t *row = packed + (MODE == BWD_ONE ? half * (64 * 64) : 0) + n * 64;
            if constexpr (MODE == BWD_ONE) {
                v[2 * h] = lds128_once(row + 16 * (c ^ ((n >> 1) & 3)));
                v[2 * h + 1] = lds128_once(row + 16 * ((c + 2) ^ ((n >> 1) & 3)));
            } else {
                v[h] = lds128_once(row + 16 * ((2 * half + c) ^ ((n >> 1) & 3)));
            }
        }
    }
}

// Gives a packed slot back once this warp's loads of v have returned: every
// lane votes on a value that depends on each of its loads, and lane 0 stores
// the outcome before it arrives. (An mbarrier arrive does not wait for loads
// in flight; behind loads that were merely issued it let the slot be refilled
// under them.)
template <int N>
__device__ __forceinline__ void give_back(uint64_t *bar, uint32_t *sink, const uint4 (&v)[N], int lane) {
    uint32_t d = v[0].x;
#pragma unroll
    for (int i = 1; i < N; ++i) d ^= v[i].x;
    const uint32_t all = __ballot_sync(0xffffffffu, d & 1u);
    if (lane == 0) {
        asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(ptx::smem_addr(sink)), "r"(all) : "memory");
        ptx::mbar_arrive(bar);
    }
}

__device__ __forceinline__ void widen_chunk(const uint4 &v, uint8_t *slot, int n, int c) {
    const __half2 off = __floats2half2_rn(1032.0f, 1032.0f);
    const uint32_t p[4] = {v.x, v.y, v.z, v.w};
    uint8_t *row = slot + (c >> 1) * (64 * 128) + n * 128;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t t = ((p[w] >> (4 * j)) & 0x000F000Fu) ^ 0x64086408u;
            const __half2 h = __hsub2(*reinterpret_cast<__half2 *>(&t), off);
            o[j] = *reinterpret_cast<const uint32_t *>(&h);
        }
        sts128(row + 16 * ((4 * (c & 1) + w) ^ (n & 7)), o[0], o[1], o[2], o[3]);
    }
}

template <int MODE, bool WHOLE>
__device__ __forceinline__ void widen_pieces(const uint4 (&v)[pieces<MODE>() * (WHOLE ? 2 : 1)], uint8_t *slot, int g,
                                             int tid) {
#pragma unroll
    for (int h = 0; h < (WHOLE ? 2 : 1); ++h) {
        const int half = WHOLE ? h : g;
        if constexpr (MODE == FWD_LINEAR || MODE == FWD_GLU) {
            const int r = tid;
            uint8_t *row = slot + half * SUB_BYTES + r * 128;
            constexpr uint32_t H = 0xF0F0F0F0u;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const uint4 &w = v[4 * h + c];
                sts128(row + 16 * ((2 * c) ^ (r & 7)), (w.x << 4) & H, w.x & H, (w.y << 4) & H, w.y & H);
                sts128(row + 16 * ((2 * c + 1) ^ (r & 7)), (w.z << 4) & H, w.z & H, (w.w << 4) & H, w.w & H);
            }
        } else if constexpr (MODE == BWD_ONE) {
            widen_chunk(v[2 * h], slot + half * SUB_BYTES, tid & 63, tid >> 6);
            widen_chunk(v[2 * h + 1], slot + half * SUB_BYTES, tid & 63, (tid >> 6) + 2);
        } else {
            widen_chunk(v[h], slot, tid & 63, 2 * half + (tid >> 6));
        }
    }
}

// A whole forward stage of row r to TMEM lane r (the thread's), 4 INT8 a column.
__device__ __forceinline__ void widen_tmem(const uint4 (&v)[8], uint32_t taddr) {
    constexpr uint32_t H = 0xF0F0F0F0u;
    ptx::tc_fence_after();  // behind the wait for the MMAs that read the slot
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t o[32];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const uint32_t p[4] = {v[4 * h + c].x, v[4 * h + c].y, v[4 * h + c].z, v[4 * h + c].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                o[8 * c + 2 * j] = (p[j] << 4) & H;
                o[8 * c + 2 * j + 1] = p[j] & H;
            }
        }
        ptx::tmem_st_32x32b_x32(taddr + 32 * h, o);
    }
    ptx::tmem_wait_st();
    ptx::tc_fence_before();
}

// ---------------------------------------------------------------- epilogue ---
// A unit (16 tokens) of one TMEM lane, written to the staging tiles [16][COLS]
// of T at `st` (shared address of this thread's column in the first row; the
// saved pre-activations' tiles follow `tile` bytes apart). Every choice is a template argument: branches per element made this
// loop several times slower.
// (The stores carry no memory clobber: they would order every table load
// behind them. The barrier that publishes a tile has one.)
template <int N>
__device__ __forceinline__ void sts_column(uint32_t a, int row, const float (&v)[N], float) {
#pragma unroll
    for (int j = 0; j < N; ++j) asm volatile("st.shared.f32 [%0], %1;" ::"r"(a + j * row), "f"(v[j]));
}
template <int N>
__device__ __forceinline__ void sts_column(uint32_t a, int row, const float (&v)[N], __nv_bfloat16) {
#pragma unroll
    for (int j = 0; j < N; j += 2)  // one conversion rounds two values
        asm volatile(
            "{\n\t.reg .b16 lo, hi;\n\t.reg .b32 w;\n\tcvt.rn.bf16x2.f32 w, %3, %2;\n\tmov.b32 {lo, hi}, w;\n\t"
            "st.shared.b16 [%0], lo;\n\tst.shared.b16 [%1], hi;\n\t}" ::"r"(a + j * row),
            "r"(a + (j + 1) * row), "f"(v[j]), "f"(v[j + 1]));
}
__device__ __forceinline__ void load_tokens(float (&t)[16], const float *tok) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 q = reinterpret_cast<const float4 *>(tok)[i];
        t[4 * i] = q.x; t[4 * i + 1] = q.y; t[4 * i + 2] = q.z; t[4 * i + 3] = q.w;
    }
}

template <int ACT, bool GLU, bool SAVE, bool RES, typename T>
__device__ __forceinline__ void fwd_unit(const uint32_t (&v)[16], const float (&r)[16], const float *tok, float rsw,
                                         float b, int lane, uint32_t st, int tile) {
    constexpr int ROW = (GLU ? 64 : 128) * (int)sizeof(T);
    float z[16];
    load_tokens(z, tok);
#pragma unroll
    for (int j = 0; j < 16; ++j) z[j] = dequant(__int2float_rn((int32_t)v[j]), z[j], rsw, b);
    if constexpr (GLU) {
        // lanes 0-15 finish tokens 0-7 of the unit, lanes 16-31 tokens 8-15
        const bool gate = lane < 16;
        const uint32_t at = st + (gate ? 0 : 8 * ROW);
        float g[8], u[8], h[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float got = __shfl_xor_sync(0xffffffffu, gate ? z[8 + j] : z[j], 16);
            g[j] = gate ? z[j] : got;
            u[j] = gate ? got : z[8 + j];
            h[j] = act_value<ACT>(g[j]) * u[j];
        }
        sts_column(at, ROW, h, T());
        if constexpr (SAVE) {
            sts_column(at + tile, ROW, g, T());
            sts_column(at + 2 * tile, ROW, u, T());
        }
    } else {
        float y[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            y[j] = act_value<ACT>(z[j]);
            if constexpr (RES) y[j] += r[j];
        }
        sts_column(st, ROW, y, T());
        if constexpr (SAVE) sts_column(st + tile, ROW, z, T());
    }
}

template <int ACT, bool GLU, typename T>
__device__ __forceinline__ void fwd_unit_any(bool save, bool res, const uint32_t (&v)[16], const float (&r)[16],
                                             const float *tok, float rsw, float b, int lane, uint32_t st, int tile) {
    if (GLU || !res) {
        if (save) fwd_unit<ACT, GLU, true, false, T>(v, r, tok, rsw, b, lane, st, tile);
        else fwd_unit<ACT, GLU, false, false, T>(v, r, tok, rsw, b, lane, st, tile);
    } else {
        if (save) fwd_unit<ACT, GLU, true, true, T>(v, r, tok, rsw, b, lane, st, tile);
        else fwd_unit<ACT, GLU, false, true, T>(v, r, tok, rsw, b, lane, st, tile);
    }
}

// A staged unit to memory by a group's four warps, where the arrays'
// alignment does not allow the TMA store.
template <int COLS, typename T>
__device__ __forceinline__ void copy_out(const uint8_t *stg, void *out, int ld, int m0, int M, int n0, int N, int et) {
    constexpr int STEP = 128 / COLS;  // rows per pass of the group
    const T *s = reinterpret_cast<const T *>(stg) + et;
    const int r0 = et / COLS, n = n0 + et % COLS;
    if (n >= N) return;
    T *o = static_cast<T *>(out) + (size_t)(m0 + r0) * ld + n;
    T v[UNIT / STEP];
#pragma unroll
    for (int i = 0; i < UNIT / STEP; ++i) v[i] = s[128 * i];
#pragma unroll
    for (int i = 0; i < UNIT / STEP; ++i)
        if (m0 + r0 + i * STEP < M) o[(size_t)(i * STEP) * ld] = v[i];
}

// Staging of a call: each group owns half of EPI_SMEM, as one set of tiles or
// two sets of half that size. A partial tile's unit (raw accumulators, all 128
// lanes) takes 8 KB of a set.
constexpr int RAW_UNIT = UNIT * ROWS_CTA * 4;
template <int MODE, typename T>
struct Staging {
    static constexpr int COLS = MODE == FWD_GLU ? 64 : 128;
    static constexpr int TILE = UNIT * COLS * (int)sizeof(T);
    int outs, sets;
    __device__ __forceinline__ explicit Staging(const EpiArgs &e) {
        outs = 1 + ((MODE == FWD_LINEAR || MODE == FWD_GLU) && e.Z ? (MODE == FWD_GLU ? 2 : 1) : 0);
        sets = outs * TILE <= EPI_SMEM / EPI_GROUPS / 2 ? 2 : 1;
    }
    __device__ __forceinline__ uint8_t *at(uint8_t *epi, int group, int set) const {
        return epi + group * (EPI_SMEM / EPI_GROUPS) + set * (EPI_SMEM / EPI_GROUPS / 2);
    }
};
static_assert(Staging<FWD_LINEAR, float>::TILE * 2 * EPI_GROUPS <= EPI_SMEM &&
              Staging<FWD_GLU, float>::TILE * 3 * EPI_GROUPS <= EPI_SMEM &&
              RAW_UNIT * 2 * EPI_GROUPS <= EPI_SMEM, "one set of every call fits, and two of raw units");

// Where a partial tile's unit goes: slot, CTA of the pair, unit; rows of 128 lanes.
template <int NT>
__host__ __device__ constexpr size_t part_offset(int slot, int rank, int unit) {
    return (((size_t)slot * 2 + rank) * (NT / UNIT) + unit) * (UNIT * ROWS_CTA);
}

// ACT is a template argument of the kernel (none for the gradient): one kernel
// with all activations behind a switch ran the epilogue-bound shapes 13 to 18 %
// slower (M 4096, K 256).
template <int MODE, int NT, int ACT, typename T>
__global__ void __launch_bounds__(PAIR_THREADS, 1)
k_mlp_pair(const __grid_constant__ CUtensorMap tm_wa, const __grid_constant__ CUtensorMap tm_wb,
           const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_y,
           const __grid_constant__ CUtensorMap tm_z, const __grid_constant__ CUtensorMap tm_u, const PairArgs p) {
    using S = Shape<MODE, NT>;
    constexpr bool FWD = S::FWD, GLU = MODE == FWD_GLU;
    constexpr int A_SLOTS = S::A_SLOTS, B_SLOTS = S::B_SLOTS, HT = NT / 2;
    constexpr int TILE_ROWS = GLU ? ROWS_CTA : 2 * ROWS_CTA;  // output columns per pair tile
    extern __shared__ uint8_t smem_raw[];
    auto &sm = *reinterpret_cast<PairSmem<MODE, NT> *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    // warp-uniform by construction, so that what the MMA warp computes from it
    // stays on the uniform datapath, where tcgen05 takes its operands from
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int rank = (int)ptx::cluster_ctarank();
    const int pair = (int)blockIdx.x >> 1, npairs = (int)gridDim.x >> 1;
    const int tiles_m = (p.M + NT - 1) / NT, tiles_n = (p.N + TILE_ROWS - 1) / TILE_ROWS;
    const int num_tiles = tiles_m * tiles_n;
    const Run run0(p, num_tiles, pair, npairs);
    const int total = run0.valid() ? run0.total() : 0;
    volatile int *abort = &sm.abort;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S::P_SLOTS; ++s) {
            ptx::mbar_init(&sm.pfull[s], 1);
            ptx::mbar_init(&sm.pfree[s], S::WARPS_PER_STAGE);
        }
        for (int s = 0; s < B_SLOTS; ++s) {
            ptx::mbar_init(&sm.bfull[s], 1);
            ptx::mbar_init(&sm.empty[s], 1);
        }
        for (int a = 0; a < A_SLOTS; ++a) ptx::mbar_init(&sm.ready[a], 2 * S::WARPS_PER_STAGE);
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(&sm.acc_full[b], 1);
            ptx::mbar_init(&sm.acc_empty[b], 2 * 4 * EPI_GROUPS);
        }
        ptx::mbar_init(&sm.done, 1);
        sm.abort = 0;
        sm.stop = 0;
        ptx::fence_mbar_init();
        ptx::prefetch_tensormap(&tm_wa);
        ptx::prefetch_tensormap(&tm_x);
    }
    if (warp == 1) {
        tcp::tmem_alloc2(&sm.tmem_base, 512);
        tcp::tmem_relinquish2();
    }
    ptx::tc_fence_before();
    // both CTAs' barriers initialized and TMEM allocated before any remote use
    ptx::cluster_arrive_release();
    ptx::cluster_wait_acquire();
    ptx::tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, sm.tmem_base, 0);

    // Packed weights of stage st of a tile. Sub-tiles past the contraction's
    // end are zero-filled by the loads' bounds.
    auto load_weights = [&](int slot, int n_tile, int st) {
        ptx::mbar_arrive_expect_tx(&sm.pfull[slot], S::P_BYTES);
#pragma unroll
        for (int u = 0; u < S::SUBS; ++u) {
            uint8_t *dst = sm.packed[slot] + u * S::P_SUB;
            if constexpr (MODE == FWD_LINEAR) {
                ptx::tma_load_2d(dst, &tm_wa, 64 * (S::SUBS * st + u), n_tile * 256 + rank * 128, &sm.pfull[slot]);
            } else if constexpr (GLU) {
                const int n0 = n_tile * 128 + rank * 64;
                ptx::tma_load_2d(dst, &tm_wa, 64 * (S::SUBS * st + u), n0, &sm.pfull[slot]);
                ptx::tma_load_2d(dst + 4096, &tm_wb, 64 * (S::SUBS * st + u), n0, &sm.pfull[slot]);
            } else {
                const bool second = st >= p.seg_stages;
                ptx::tma_load_2d(dst, second ? &tm_wb : &tm_wa, n_tile * 128 + rank * 64,
                                 64 * (S::SUBS * (second ? st - p.seg_stages : st) + u), &sm.pfull[slot]);
            }
        }
    };
    // The first stages' packed tiles are requested before the dependency wait:
    // the row pass before this kernel lets it start only once all earlier work
    // is done, so the weights are settled. The tokens are read after the wait.
    const int pre_w = min(S::P_SLOTS, total);
    if (warp == 0 && lane == 0) {
        Run r = run0;
        for (int it = 0, st = r.s0; it < pre_w; ++it) {
            load_weights(it, r.tile / tiles_m, st);
            if (++st == r.s1) {
                r.next();
                st = r.s0;
            }
        }
    }
    __syncwarp();
    griddep_launch_dependents();
    griddep_wait();

    if (warp == 0 || warp == 2) {
        // ------------------------------------- TMA producers (each CTA: its halves)
        // Warp 0: packed weights, freed as soon as they are widened. Warp 2:
        // tokens, freed by the MMAs.
        if (lane == 0) {
            const bool w = warp == 0;
            const int slots = w ? S::P_SLOTS : B_SLOTS;
            uint64_t *full = w ? sm.pfull : sm.bfull, *freed = w ? sm.pfree : sm.empty;
            int slot = 0, it = 0;
            uint32_t phase = 0, issued = (1u << pre_w) - 1u, last_par = 0;
            if (!w) issued = 0;
            bool ok = true;
            for (Run r = run0; r.valid() && ok; r.next()) {
                const int n_tile = r.tile / tiles_m;
                const int m0 = (r.tile % tiles_m) * NT + rank * HT;
                for (int st = r.s0; st < r.s1; ++st, ++it) {
                    if (!w || it >= pre_w) {
                        if (!ptx::mbar_wait(&freed[slot], phase ^ 1, abort)) { ok = false; break; }
                        if (w) {
                            load_weights(slot, n_tile, st);
                        } else {
                            ptx::mbar_arrive_expect_tx(&sm.bfull[slot], S::B_BYTES);
#pragma unroll
                            for (int u = 0; u < 2; ++u)
                                ptx::tma_load_2d(sm.b[slot] + u * S::B_TILE, &tm_x,
                                                 S::STEP * st + (S::SUBS == 2 ? u * S::SUB : 0),
                                                 m0 + (S::PLANES == 2 ? u * p.M : 0), &sm.bfull[slot]);
                        }
                    }
                    issued |= 1u << slot;
                    last_par = (last_par & ~(1u << slot)) | (phase << slot);
                    if (++slot == slots) { slot = 0; phase ^= 1; }
                }
            }
            // Drain: every load this thread issued lands before the CTA exits.
            if (!ok)
                for (int s = 0; s < slots; ++s)
                    if (issued & (1u << s)) ptx::mbar_wait_drain(&full[s], (last_par >> s) & 1u);
        }
    } else if (warp == 1) {
        // ---------------------------------------------------- MMA issuer (leader only)
        // The widening warps of both CTAs arrive on ready only after the
        // tokens of the same stage have landed in their CTA.
        // The whole warp runs the loop and one elected lane issues: descriptors
        // and addresses are then uniform values. (With one lane in a branch of
        // its own each MMA took about 100 cycles to issue and a commit 400.)
        if (rank == 0) {
            const bool one = elect_one();
            constexpr uint32_t idesc = FWD ? ptx::idesc_i8(256, NT) : idesc_f16_mn(256, NT);
            // descriptors count 16-byte units, so a step is an addition
            const uint64_t a0 = FWD ? ptx::sdesc_k_sw128(ptx::smem_addr(sm.a[0]))
                                    : sdesc_mn_sw128(ptx::smem_addr(sm.a[0]), 64 * 128);
            const uint64_t b0 = ptx::sdesc_k_sw128(ptx::smem_addr(sm.b[0]));
            constexpr uint32_t A_STEP = FWD ? 32 : 2048;  // bytes per MMA along the contraction
            int slot = 0, as = 0, buf = 0;
            uint32_t aphase = 0, bphase = 0;
            bool ok = true;
            for (Run r = run0; r.valid() && ok; r.next()) {
                uint32_t d = 0;
                int seg_st = r.s0 >= p.seg_stages ? r.s0 - p.seg_stages : r.s0;
                int left = p.depth - S::STEP * seg_st;
                for (int st = r.s0; st < r.s1; ++st) {
                    const bool fresh = (st - r.s0) % S::CHUNK == 0;  // a new accumulator
                    ok = !fresh || warp_wait(&sm.acc_empty[buf], bphase ^ 1u, abort);
                    ok = ok && warp_wait(&sm.ready[as], aphase, abort);
                    if (!ok) break;
                    d = tmem + (uint32_t)(buf * S::D_COLS);
                    const uint32_t ta = tmem + (uint32_t)(2 * NT + as * S::A_COLS);
                    ptx::tc_fence_after();
                    const uint64_t a = a0 + (uint32_t)(as * S::A_BYTES / 16), b = b0 + (uint32_t)(slot * S::B_BYTES / 16);
                    auto mma = [&](int i) {
                        const int sub = S::SUBS == 2 ? i >> 2 : 0, kk = i & 3;
                        const uint64_t ad = a + (uint32_t)((sub * SUB_BYTES + kk * A_STEP) / 16);
                        const uint64_t bd = b + (uint32_t)(((i >> 2) * S::B_TILE + 32 * kk) / 16);
                        if constexpr (S::A_TMEM) {
                            if (one) tcp::mma_i8_ts2(d, ta + 8 * i, bd, idesc, !fresh || i != 0);
                        } else {
                            if (one) mma_ss2<FWD>(d, ad, bd, idesc, !fresh || i != 0);
                        }
                    };
#pragma unroll
                    for (int i = 0; i < 4; ++i) mma(i);
                    if (S::SUBS == 1 || left > S::SUB) {  // else the second sub-tile lies past the contraction's end
#pragma unroll
                        for (int i = 4; i < 8; ++i) mma(i);
                    }
                    if (one) tcp::mma_commit2_both(&sm.empty[slot]);
                    left -= S::STEP;
                    if (++seg_st == p.seg_stages) { seg_st = 0; left = p.depth; }
                    if (++slot == B_SLOTS) slot = 0;
                    if (++as == A_SLOTS) { as = 0; aphase ^= 1u; }
                    if (st + 1 == r.s1 || (st + 1 - r.s0) % S::CHUNK == 0) {
                        if (one) tcp::mma_commit2_both(&sm.acc_full[buf]);
                        if (++buf == 2) { buf = 0; bphase ^= 1u; }
                    }
                }
            }
            if (total > 0 && one) tcp::mma_commit2_both(&sm.done);
        }
    } else if (warp >= FIRST_CONV && warp < FIRST_EPI) {
        // ---------------------------------------------------- widening (each CTA: its 128 rows)
        const int grp = (warp - FIRST_CONV) / GROUP_WARPS;
        const int tid = (threadIdx.x - 32 * FIRST_CONV) % (32 * GROUP_WARPS);
        constexpr int STRIDE = S::TURNS ? CONV_GROUPS : 1;   // stages from one of this group's to its next
        constexpr int PIECES = pieces<MODE>() * (S::TURNS ? 2 : 1);
        const int it0 = S::TURNS ? grp : 0;
        int ps = it0, bs = it0, as = it0 % A_SLOTS;
        int old = (it0 + B_SLOTS - A_SLOTS) % B_SLOTS;        // the token slot of iteration it - A_SLOTS
        uint32_t pphase = 0, bphase = 0;
        uint32_t ophase = it0 >= A_SLOTS ? 0 : 1;             // below 0 it has the parity before the first
        for (int it = it0; it < total; it += STRIDE) {
            // The packed bytes come into registers, and their slot is given
            // back, before the wait for the A slot: what follows the MMAs' end
            // is only the widening and its stores.
            // (A group that takes every second stage waits for the A slot first:
            // all stages up to it - A_SLOTS are then done, among them the last
            // ones in its packed and token slots, so the parity of its own waits
            // cannot be mistaken for a phase that the other group consumes.)
            if (S::TURNS && it >= A_SLOTS && !warp_wait(&sm.empty[old], ophase, abort)) break;
            if (!warp_wait(&sm.pfull[ps], pphase, abort)) break;
            uint4 v[PIECES];
            load_pieces<MODE, S::TURNS>(v, sm.packed[ps], grp, tid);
            give_back<PIECES>(&sm.pfree[ps], &sm.sink[warp - FIRST_CONV], v, lane);
            if (!warp_wait(&sm.bfull[bs], bphase, abort)) break;
            // the A slot was last read by the MMAs of iteration it - A_SLOTS
            if (!S::TURNS && it >= A_SLOTS && !warp_wait(&sm.empty[old], ophase, abort)) break;
            if constexpr (S::A_TMEM) {
                widen_tmem(v, tmem + ((uint32_t)(32 * (warp & 3)) << 16) + (uint32_t)(2 * NT + as * S::A_COLS));
            } else {
                widen_pieces<MODE, S::TURNS>(v, sm.a[as], grp, tid);
                tcp::fence_proxy_async_smem();  // the slot's generic writes, before the MMA reads them
            }
            __syncwarp();
            if (lane == 0) tcp::mbar_arrive_leader(&sm.ready[as]);
            if ((ps += STRIDE) >= S::P_SLOTS) { ps -= S::P_SLOTS; pphase ^= 1u; }
            if ((bs += STRIDE) >= B_SLOTS) { bs -= B_SLOTS; bphase ^= 1u; }
            if ((old += STRIDE) >= B_SLOTS) { old -= B_SLOTS; ophase ^= 1u; }
            if ((as += STRIDE) >= A_SLOTS) as -= A_SLOTS;
        }
    } else if (warp >= FIRST_EPI) {
        // ---------------------------------------------------- epilogue (each CTA: its 128 TMEM lanes)
        // Two groups of four warps (one per quarter of the lanes) take units of
        // 16 tokens in turn.
        const int q = warp & 3, eg = (warp - FIRST_EPI) >> 2;
        const int ea = threadIdx.x - 32 * FIRST_EPI, et = ea & 127;
        const Staging<MODE, T> sg(p.e);
        constexpr int COLS = sg.COLS, TILE = sg.TILE;
        // this thread's output column inside the CTA's COLS (the gradient's
        // rows come in the order of the widening masks)
        const int col = GLU ? 16 * q + (lane & 15)
                            : FWD ? et : (et & ~7) | ((et & 7) >> 1) | ((et & 1) << 2);
        const uint32_t lane_base = (uint32_t)(q * 32) << 16;
        const bool res = FWD && !GLU && p.e.R != nullptr;
        int buf = 0, set = 0;
        uint32_t acc_phase = 0;
        for (Run run = run0; run.valid(); run.next()) {
            const int n_tile = run.tile / tiles_m, m_base = (run.tile % tiles_m) * NT;
            const int n_base = n_tile * TILE_ROWS + rank * COLS, n = n_base + col;
            const bool n_ok = n < p.N, partial = run.partial();
            if (ea < NT) {
                const float t = m_base + ea < p.M ? ld_dep(p.tok + m_base + ea) : 1.0f;
                sm.tok[ea] = FWD ? __frcp_rn(t) : t;
            }
            float rsw = 1.0f, b = 0.0f;
            if constexpr (FWD) {
                const bool up = GLU && lane >= 16;
                const float *sw = up ? p.b.sw : p.a.sw, *bias = up ? p.b.bias : p.a.bias;
                rsw = n_ok ? __frcp_rn(ld_dep(sw + n)) * 0.0625f : 1.0f;  // the accumulator holds 16 x the sum
                b = n_ok && bias ? ld_dep(bias + n) : 0.0f;
            }
            // A unit's values, from TMEM or summed, through its staging tiles.
            auto finish = [&](int c0, const uint32_t (&v)[16]) {
                const int m0 = m_base + c0;
                if (m0 >= p.M) return;
                // the set is free: the store warp has seen its last stores read
                ptx::bar_sync(BAR_FREE + 2 * eg + set, 160);
                uint8_t *stg = sg.at(sm.epi, eg, set);
                const uint32_t st = ptx::smem_addr(stg) + (uint32_t)(col * (int)sizeof(T));
                float r[16];
                if (res && !partial) {  // indexes past the edges repeat the last row or column
                    const T *R = static_cast<const T *>(p.e.R) + min(n, p.N - 1);
#pragma unroll
                    for (int j = 0; j < 16; ++j) r[j] = ld_elem(R + (size_t)min(m0 + j, p.M - 1) * p.e.ldr);
                }
                const float *tok = sm.tok + c0;
                if (partial) {
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        asm volatile("st.shared.u32 [%0], %1;" ::"r"(ptx::smem_addr(stg) + (uint32_t)(j * ROWS_CTA + et) * 4),
                                     "r"(v[j]));
                } else if constexpr (FWD) {
                    fwd_unit_any<ACT, GLU, T>(p.e.Z != nullptr, res, v, r, tok, rsw, b, lane, st, TILE);
                } else {
                    float y[16];
                    load_tokens(y, tok);
#pragma unroll
                    for (int j = 0; j < 16; ++j) y[j] *= __uint_as_float(v[j]);
                    sts_column(st, COLS * (int)sizeof(T), y, T());
                }
                if (p.tma_out || partial) {
                    tcp::fence_proxy_async_smem();  // the staging writes, before the store reads them
                } else {
                    ptx::bar_sync(BAR_GROUP + eg, 128);
                    copy_out<COLS, T>(stg, p.e.Y, p.e.ldy, m0, p.M, n_base, p.N, et);
                    if (sg.outs > 1) copy_out<COLS, T>(stg + TILE, p.e.Z, p.e.ldz, m0, p.M, n_base, p.N, et);
                    if (sg.outs > 2) copy_out<COLS, T>(stg + 2 * TILE, p.e.U, p.e.ldz, m0, p.M, n_base, p.N, et);
                }
                bar_arrive(BAR_STAGED + 2 * eg + set, 160);
                if (sg.sets == 2) set ^= 1;
            };
            auto load_unit = [&](int c0, uint32_t (&v)[16]) {
                ptx::tmem_ld_32x32b_x16(tmem + lane_base + (uint32_t)(buf * S::D_COLS + c0), v);
                ptx::tmem_wait_ld();
            };
            auto drained = [&]() {
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) tcp::mbar_arrive_leader(&sm.acc_empty[buf]);
                if (++buf == 2) { buf = 0; acc_phase ^= 1; }
            };
            // One decision for all warps (the first time, this barrier also
            // publishes the table).
            auto acc_ready = [&]() {
                const bool got = ptx::bar_and(BAR_EPI, 128 * EPI_GROUPS, ptx::mbar_wait(&sm.acc_full[buf], acc_phase, abort));
                ptx::tc_fence_after();
                return got;
            };
            bool alive = acc_ready();
            if constexpr (S::PLANES == 2) {
                constexpr int MINE = NT / (UNIT * EPI_GROUPS);  // this group's units
                float sum[MINE][16];
#pragma unroll
                for (int i = 0; i < MINE; ++i)
#pragma unroll
                    for (int j = 0; j < 16; ++j) sum[i][j] = 0.0f;
                for (int st = run.s0; alive && st < run.s1; st += S::CHUNK) {
                    if (st > run.s0) alive = acc_ready();
                    if (!alive) break;
#pragma unroll
                    for (int i = 0; i < MINE; ++i) {
                        uint32_t v[16];
                        load_unit(UNIT * (eg + EPI_GROUPS * i), v);
#pragma unroll
                        for (int j = 0; j < 16; ++j) sum[i][j] += __uint_as_float(v[j]);
                    }
                    drained();
                }
                if (alive) {
#pragma unroll
                    for (int i = 0; i < MINE; ++i) {
                        uint32_t v[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) v[j] = __float_as_uint(sum[i][j]);
                        finish(UNIT * (eg + EPI_GROUPS * i), v);
                    }
                }
            } else if (alive) {
#pragma unroll 1
                for (int c0 = UNIT * eg; c0 < NT && m_base + c0 < p.M; c0 += UNIT * EPI_GROUPS) {
                    uint32_t v[16];
                    load_unit(c0, v);
                    finish(c0, v);
                }
                drained();
            }
            if (!alive) {
                sm.stop = 1;  // let the store warp leave too
                bar_arrive(BAR_STAGED + 2 * eg + set, 160);
                break;
            }
            ptx::bar_sync(BAR_EPI, 128 * EPI_GROUPS);  // the table is rewritten next tile
        }
    } else if (warp == 3) {
        // ---------------------------------------------------- output stores
        // Its own warp, so that neither the store's issue nor the wait for the
        // staging tiles to be read holds the epilogue up. Units in order: the
        // groups in turn, each group's sets in turn. (Units that the epilogue
        // has copied out itself only pass through.)
        const Staging<MODE, T> sg(p.e);
        constexpr int COLS = sg.COLS, TILE = sg.TILE;
        int unit[EPI_GROUPS] = {};  // units each group has had
        for (int i = 0; i < EPI_GROUPS * sg.sets; ++i) bar_arrive(BAR_FREE + 2 * (i % EPI_GROUPS) + i / EPI_GROUPS, 160);
        bool stop = false;
        for (Run run = run0; run.valid() && !stop; run.next()) {
            const int n_base = (run.tile / tiles_m) * TILE_ROWS + rank * COLS, m_base = (run.tile % tiles_m) * NT;
            const int units = (min(NT, p.M - m_base) + UNIT - 1) / UNIT;
            for (int i = 0; i < units; ++i) {
                const int eg = i % EPI_GROUPS, m0 = m_base + i * UNIT;
                const int set = sg.sets == 2 ? unit[eg] & 1 : 0;
                ptx::bar_sync(BAR_STAGED + 2 * eg + set, 160);
                stop = sm.stop != 0;
                if (stop) break;
                if (lane == 0) {
                    const uint8_t *stg = sg.at(sm.epi, eg, set);
                    if (run.partial()) {
                        bulk_s2g(p.parts + part_offset<NT>(run.slot(pair), rank, i), stg, RAW_UNIT);
                    } else if (p.tma_out && n_base < p.N) {
                        tcp::tma_store_2d(&tm_y, stg, n_base, m0);
                        if (sg.outs > 1) tcp::tma_store_2d(&tm_z, stg + TILE, n_base, m0);
                        if (sg.outs > 2) tcp::tma_store_2d(&tm_u, stg + 2 * TILE, n_base, m0);
                    }
                    tcp::bulk_commit_group();
                    // one set: this unit has been read; two: every earlier one
                    if (sg.sets == 2) tcp::bulk_wait_read_1();
                    else bulk_wait_read_0();
                }
                __syncwarp();
                // so the group's only set, or the one of its previous unit, is free
                if (sg.sets == 1) bar_arrive(BAR_FREE + 2 * eg, 160);
                else if (unit[eg] > 0) bar_arrive(BAR_FREE + 2 * eg + (set ^ 1), 160);
                ++unit[eg];
            }
        }
        // the output stores have completed before the CTA exits
        if (lane == 0) tcp::bulk_wait_all();
    }

    // Every MMA of the pair has finished before TMEM is released.
    if (warp == 1) {
        if (total > 0 && lane == 0) ptx::mbar_wait_drain(&sm.done, 0);
        __syncwarp();
    }
    ptx::tc_fence_before();
    __syncthreads();
    // the pair meets before TMEM is released and before either CTA exits
    ptx::cluster_arrive_release();
    ptx::cluster_wait_acquire();
    ptx::tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        tcp::tmem_dealloc2(tmem, 512);
    }
}

// Finishes the tiles that k_mlp_pair left in parts. Block (b, unit): the tile
// that holds the boundary between the runs of pairs b and b + 1, if b is the
// first boundary inside it; JOIN tokens; thread: a TMEM lane of one of the
// pair's CTAs. Parts are added in the order of their stages, so results
// repeat bit for bit (INT32 sums are exact anyway).
constexpr int JOIN = 4;
static_assert(UNIT % JOIN == 0, "a block's tokens lie in one unit");
template <int MODE, int NT, typename T>
__global__ void __launch_bounds__(256)
k_mlp_join(const PairArgs p, int npairs) {
    constexpr bool FWD = Shape<MODE, NT>::FWD, GLU = MODE == FWD_GLU;
    constexpr int COLS = GLU ? 64 : 128, TILE_ROWS = 2 * COLS;
    griddep_launch_dependents();
    griddep_wait();
    const int tiles_m = (p.M + NT - 1) / NT, tiles_n = (p.N + TILE_ROWS - 1) / TILE_ROWS;
    const long long all = (long long)tiles_m * tiles_n * p.stages;
    auto bound = [&](int i) { return all * i / npairs; };  // where pair i's run begins
    const int b = blockIdx.x, unit = blockIdx.y * JOIN / UNIT, j0 = blockIdx.y * JOIN % UNIT;
    const long long x = bound(b + 1);
    const int tile = (int)(x / p.stages);
    const long long t0 = (long long)tile * p.stages, t1 = t0 + p.stages;
    if (x == t0 || x >= all || bound(b) > t0) return;  // no tile inside, or an earlier boundary's
    const int m0 = (tile % tiles_m) * NT + unit * UNIT + j0;
    if (m0 >= p.M) return;
    const int rank = threadIdx.x >> 7, et = threadIdx.x & 127, lane = et & 31;
    // the parts: the tile is the first of its run except, perhaps, in run b
    const int parts = (int)((t1 * npairs + all - 1) / all) - b;
    const uint32_t *src = p.parts + part_offset<NT>(2 * b, rank, unit) + (size_t)j0 * ROWS_CTA + et;
    constexpr size_t SLOT = part_offset<NT>(1, 0, 0);
    uint32_t v[JOIN];
    for (int q0 = 0; q0 < parts; q0 += 4) {  // four parts' loads in flight, added in order
        uint32_t w[4][JOIN];
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int j = 0; j < JOIN; ++j)
                if (q0 + q < parts) {
                    const size_t slot = q0 + q == 0 ? (bound(b) < t0 ? 1 : 0) : 2 * (size_t)(q0 + q);
                    asm volatile("ld.global.u32 %0, [%1];" : "=r"(w[q][j]) : "l"(src + slot * SLOT + j * ROWS_CTA));
                }
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int j = 0; j < JOIN; ++j)
                if (q0 + q < parts) {
                    if (q0 + q == 0) v[j] = w[q][j];
                    else if constexpr (FWD) v[j] += w[q][j];
                    else v[j] = __float_as_uint(__uint_as_float(v[j]) + __uint_as_float(w[q][j]));
                }
    }
    const int col = GLU ? 16 * (et >> 5) + (lane & 15) : FWD ? et : (et & ~7) | ((et & 7) >> 1) | ((et & 1) << 2);
    const int n = (tile / tiles_m) * TILE_ROWS + rank * COLS + col;
    const bool n_ok = n < p.N;
    const bool up = GLU && lane >= 16;
    float rsw = 1.0f, bias = 0.0f;
    if constexpr (FWD) {
        const Proj &w = up ? p.b : p.a;
        rsw = n_ok ? __frcp_rn(ld_dep(w.sw + n)) * 0.0625f : 1.0f;
        bias = n_ok && w.bias ? ld_dep(w.bias + n) : 0.0f;
    }
    const int rows = min(JOIN, p.M - m0);
    float t[JOIN], z[JOIN], u[JOIN];
#pragma unroll
    for (int j = 0; j < JOIN; ++j) t[j] = ld_dep(p.tok + m0 + min(j, rows - 1));
    if constexpr (FWD) {
#pragma unroll
        for (int j = 0; j < JOIN; ++j) {
            z[j] = dequant(__int2float_rn((int32_t)v[j]), __frcp_rn(t[j]), rsw, bias);
            u[j] = GLU ? __shfl_xor_sync(0xffffffffu, z[j], 16) : 0.0f;
        }
        if (up || !n_ok) return;
        if (!GLU && p.e.R) {
            const T *R = static_cast<const T *>(p.e.R) + (size_t)m0 * p.e.ldr + n;
#pragma unroll
            for (int j = 0; j < JOIN; ++j) u[j] = j < rows ? ld_elem(R + (size_t)j * p.e.ldr) : 0.0f;
        }
        auto finish = [&](auto A) {
            T *Y = static_cast<T *>(p.e.Y) + (size_t)m0 * p.e.ldy + n;
#pragma unroll
            for (int j = 0; j < JOIN; ++j) {
                const float a = act_value<decltype(A)::value>(z[j]);
                if (j < rows) st_elem(Y + (size_t)j * p.e.ldy, GLU ? a * u[j] : a + u[j]);
            }
        };
        switch (p.act) {
            case W4A8_ACT_NONE: finish(std::integral_constant<int, W4A8_ACT_NONE>{}); break;
            case W4A8_ACT_RELU: finish(std::integral_constant<int, W4A8_ACT_RELU>{}); break;
            case W4A8_ACT_SILU: finish(std::integral_constant<int, W4A8_ACT_SILU>{}); break;
            case W4A8_ACT_GELU: finish(std::integral_constant<int, W4A8_ACT_GELU>{}); break;
            default: finish(std::integral_constant<int, W4A8_ACT_GELU_TANH>{}); break;
        }
        if (p.e.Z) {
#pragma unroll
            for (int j = 0; j < JOIN; ++j) {
                if (j >= rows) break;
                st_elem(static_cast<T *>(p.e.Z) + (size_t)(m0 + j) * p.e.ldz + n, z[j]);
                if constexpr (GLU) st_elem(static_cast<T *>(p.e.U) + (size_t)(m0 + j) * p.e.ldz + n, u[j]);
            }
        }
    } else {
        if (!n_ok) return;
        T *Y = static_cast<T *>(p.e.Y) + (size_t)m0 * p.e.ldy + n;
#pragma unroll
        for (int j = 0; j < JOIN; ++j)
            if (j < rows) st_elem(Y + (size_t)j * p.e.ldy, __uint_as_float(v[j]) * t[j]);
    }
}

// ------------------------------------------------------------- host side ---

// CTA pairs of a launch: one per two of the B200's 148 SMs. A property of the
// plan (the partial tiles' slots depend on it), not of the device at hand:
// with fewer SMs the pairs run one after another, none waits for another.
constexpr int PAIRS = 74;

// Token tile and sharing of a call, by estimated time. Whole tiles: the first
// tile's stages, then per round the longer of a tile's stages and its epilogue
// (beside the next one's stages), then the last epilogue. Measured per stage
// of 8 MMAs: about 750 ns with 256 tokens, 460 with 128, 400 with 64 (the
// float32 gradient's a quarter more); the epilogue about 26 ns a token and
// 0.8 us a tile. Shared: equal runs of stages, the join's launch, the partial
// tiles written and read (2 x 74 slots; some 16 us with 256 tokens); taken
// only where the estimate gains a tenth: with long sums the card's power
// limit, not the idle pairs, sets the pace (2048 x 28672 x 4096: 210 us shared,
// whole tiles 188).
struct PairPlan {
    int nt;
    bool split;
    size_t part_bytes;
};
inline PairPlan pair_plan(int M, int rows, int tile_rows, int stages, bool two = false) {
    PairPlan best = {256, false, 0};
    double best_t = -1.0;
    const int cand[3] = {256, 128, 64};
    const double stage_ns[3] = {750.0, 460.0, 400.0};
    for (int i = two ? 1 : 0; i < 3; ++i) {  // two planes: the sums of 256 tokens do not fit the registers
        const int nt = cand[i];
        const long long tiles = (long long)((M + nt - 1) / nt) * ((rows + tile_rows - 1) / tile_rows);
        const double main = stages * stage_ns[i], epi = 800.0 + 26.0 * nt;
        const double whole = main + (double)((tiles - 1) / PAIRS) * (main > epi ? main : epi) + epi;
        if (best_t < 0 || whole < best_t) {
            best_t = whole;
            best = {nt, false, 0};
        }
        const size_t slot = (size_t)256 * nt * 4;
        const double share = 1.1 * ((double)((tiles * stages + PAIRS - 1) / PAIRS) * stage_ns[i] + 2.0 * epi +
                                    3000.0 + 16000.0 * nt / 256.0);
        if (tiles * stages >= PAIRS && share < best_t) {
            best_t = share;
            best = {nt, true, 2 * PAIRS * slot};
        }
    }
    return best;
}
// Stages of a call: forward 256 k, gradient 128 n (64 for two planes) per segment.
inline PairPlan forward_plan(int M, int K, int N, bool glu) { return pair_plan(M, N, glu ? 128 : 256, (K + 255) / 256); }
inline PairPlan grad_plan(int M, int K, int segs, int seg, bool two) {
    return pair_plan(M, K, 256, segs * (seg / (two ? 64 : 128)), two);
}

// What a launch needs beside PairArgs: the operands' shapes.
struct PairCall {
    const uint8_t *Wa, *Wb;
    int w_rows, k, ldp;          // packed rows, their codes and stride
    const void *X;               // INT8 rows [M][ldq], or FP16 rows [planes M][width]
    int x_rows, x_inner;         // rows and row elements (= stride) of X
};

template <int MODE, int NT, int ACT, typename T>
w4a8_status launch_pair(PairArgs p, const PairCall &c, cudaStream_t stream) {
    using S = Shape<MODE, NT>;
    constexpr bool GLU = MODE == FWD_GLU;
    constexpr int COLS = GLU ? 64 : 128, TILE_ROWS = 2 * COLS;
    auto kern = k_mlp_pair<MODE, NT, ACT, T>;
    const int smem = (int)sizeof(PairSmem<MODE, NT>) + 1024;
    if (!raise_smem_limit(reinterpret_cast<const void *>(kern), smem)) return W4A8_ERR_CUDA;
    CUtensorMap wa, wb, x, out[3];
    memset(out, 0, sizeof(out));
    const uint32_t box_rows = S::FWD ? (GLU ? 64 : 128) : 64;
    // A row's own bytes, not its stride: of the last row of a column range of a
    // wider array the stride reaches past the array's end.
    auto map_w = [&](CUtensorMap *m, const uint8_t *W) {
        return tc::make_map_u8(m, W, (uint64_t)packed_row_bytes(c.k), (uint64_t)c.w_rows, (uint64_t)c.ldp, 64,
                               box_rows, CU_TENSOR_MAP_SWIZZLE_64B);
    };
    if (!map_w(&wa, c.Wa) || !map_w(&wb, c.Wb)) return W4A8_ERR_CUDA;
    const size_t xsz = S::FWD ? 1 : 2;
    if (!tc::make_map_2d(&x, S::FWD ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, c.X,
                         (uint64_t)c.x_inner, (uint64_t)c.x_rows, (uint64_t)c.x_inner * xsz, 128 / xsz, NT / 2,
                         CU_TENSOR_MAP_SWIZZLE_128B))
        return W4A8_ERR_CUDA;
    // Outputs go through tensor maps where every array's base, row stride and
    // row of N outputs end on 16-byte boundaries (the store's bounds check on
    // the inner dimension works in 16-byte units); directly otherwise.
    void *const arr[3] = {p.e.Y, p.e.Z, p.e.U};
    const int ld[3] = {p.e.ldy, p.e.ldz, p.e.ldz};
    bool tma = (size_t)p.N * sizeof(T) % 16 == 0;
    for (int i = 0; i < 3; ++i)
        if (arr[i]) tma = tma && aligned16(arr[i]) && (size_t)ld[i] * sizeof(T) % 16 == 0;
    const CUtensorMapDataType t = sizeof(T) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
    for (int i = 0; i < 3 && tma; ++i)
        if (arr[i])
            tma = tc::make_map_2d(&out[i], t, arr[i], (uint64_t)p.N, (uint64_t)p.M, (uint64_t)ld[i] * sizeof(T), COLS,
                                  UNIT, CU_TENSOR_MAP_SWIZZLE_NONE);
    p.tma_out = tma;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(PAIR_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const long long tiles = (long long)((p.M + NT - 1) / NT) * ((p.N + TILE_ROWS - 1) / TILE_ROWS);
    const long long pairs = p.parts || tiles > PAIRS ? PAIRS : tiles;
    cfg.gridDim = dim3((unsigned)(2 * pairs));
    cudaError_t e = cudaLaunchKernelEx(&cfg, kern, wa, wb, x, out[0], out[1], out[2], p);
    if (e == cudaSuccess && p.parts)
        e = launch_pdl(k_mlp_join<MODE, NT, T>, dim3(PAIRS - 1, (unsigned)((p.M < NT ? p.M : NT) + JOIN - 1) / JOIN),
                       dim3(256), 0, stream, p, PAIRS);
    return from_cuda(e);
}

template <int MODE, int ACT, typename T>
w4a8_status launch_pair_any(const PairPlan &plan, PairArgs p, const PairCall &c, void *parts, cudaStream_t s) {
    p.parts = plan.split ? static_cast<uint32_t *>(parts) : nullptr;
    if constexpr (MODE != BWD_TWO)
        if (plan.nt == 256) return launch_pair<MODE, 256, ACT, T>(p, c, s);
    if (plan.nt == 128) return launch_pair<MODE, 128, ACT, T>(p, c, s);
    return launch_pair<MODE, 64, ACT, T>(p, c, s);
}

}  // namespace mlp
}  // namespace w4a8
