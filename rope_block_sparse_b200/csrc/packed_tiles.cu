// Attention over packed sequences on tcgen05 (h3a_packed_attention): whole
// prompts and pieces of prompts, causal or not, with grouped heads.
//
// The queries that share a kv head are the rows of one matrix: row r of a
// 128-row tile is query r / group, head r % group of the kv head's group, so a
// tile holds T = 128 / group queries (rounded down) of all the group's heads
// and K and V are loaded once for the whole group.  The tensor map of Q has the
// group as a dimension, so one TMA box {32 channels, group, 1, T} is one
// swizzled chunk of such a tile.  One CTA owns one or two consecutive tiles (of T
// queries) of one sequence and kv head and one part of its keys (all of them
// unless there are too few tiles to fill the GPU); packed_plan.cu decides.
//
// Which sequence a CTA belongs to is found without a schedule made beforehand:
// with `span` queries a CTA, sequence s may use the CTAs from floor(starts_q[s] /
// span) + s on, which is ascending in s and leaves each sequence at least the
// ceil(lq / span) that it needs; at most `seqs` CTAs find nothing to do.  Later
// CTAs of a sequence see more keys when causal, so they are taken in descending
// order and a sequence's kv heads side by side, so that the longest CTAs of a
// sequence come first (against one kv head behind the other: one prompt of 2,048,
// 32/8 heads x 128, 40.7 us / 58.6, of 4,096 143 / 160, 24 up to 300 28.9 / 30.9;
// pieces of 509 tokens behind 12,000, 28/4 x 96, 146 / 143).  The producer's warp finds the work and starts the first
// loads while the others set up barriers and TMEM.
//
// The pipeline is that of attention.cu (which see for the measurements behind
// it).  The first four or eight warps are softmax warps (warpgroup t = tile t,
// thread = row), then come four with a role each: the TMA producer with K and V
// rings of 64-byte swizzled chunks; the issuer of QK^T (with P over S, of PV too);
// the issuer of PV where P has a buffer of its own; and the one that looks over V.
// S_t = Q_t K^T and O_t += P_t V accumulate in TMEM in fp32; the softmax is online
// in fp32 against a row reference that moves only when the maximum grew by 2^8; P
// is rounded to the element type for the PV MMA, whose error (half a step relative
// a weight) is that of rounding O once more.  What is different:
//   - the first tile of a CTA may need fewer steps than the second (n[0] <=
//     n[1], causal); it then simply stops earlier;
//   - every row has its own number of keys; a step whose 128 keys all rows of a
//     warp attend skips the comparison;
//   - V is looked over.  In a step where some row does not attend some key, a
//     weight of zero times an infinity or NaN in V would be NaN; the last warp
//     clears such values in shared memory before PV may read them (the barrier
//     v_ready) and notes it, and the epilogue adds them back to the rows that
//     do attend them.  Only the last one to three steps of a CTA are looked
//     over; in the others the warp passes the barrier on.
//
// What bounds it: long sequences the softmax's exponentials and the tensor core
// together (two tiles, 128 keys: 2,048 clk of MUFU and at head_dim 128 as many of
// MMA; one prompt of 16,384, 32/8 heads x 128: 2.0 ms at the clock that
// the power cap leaves, 1.08 PFLOP/s; 1.75 ms before the cap takes hold); short
// ones a CTA's beginning and end, about 4 us (24 prompts up to 300, the same
// heads: 29 us, 8.4 of them HBM's).  A step takes 2,600 to 3,000 clk at head_dim 96.
#include "fastmath.cuh"
#include "h3a_internal.h"
#include "half16.cuh"
#include "prompt_internal.h"
#include "sm100.cuh"

namespace h3a {
namespace {

constexpr int kChunkBytes = 128 * 64;  // 128 rows x 32 channels, 64-byte swizzle
constexpr uint32_t kSwizzle64 = 4;
__host__ __device__ constexpr uint32_t col_s(int t) { return t ? 128u : 0u; }

// A CTA of TILES query tiles, by head dimension.  Two tiles share every K and V
// tile and hide each other's softmax: one CTA a multiprocessor.  One tile is
// half of everything, so that two CTAs fit and hide each other's beginning and
// end, which is what short sequences consist of.
template <int D_, int TILES>
struct Geo {
    static constexpr int D = D_, kTiles = TILES;
    static constexpr int kSoftmaxWarps = 4 * TILES;  // a warpgroup per query tile
    static constexpr int kProducerWarp = kSoftmaxWarps, kMmaWarp = kSoftmaxWarps + 1, kPvWarp = kSoftmaxWarps + 2;
    static constexpr int kThreads = 32 * (kSoftmaxWarps + 4);
    static constexpr int kCtas = TILES == 1 ? 2 : 1;  // per multiprocessor
    // Register split (setmaxnreg): the softmax warpgroups hold a 128-value row each.
    static constexpr uint32_t kRegsLaunch = (65536 / kCtas / kThreads) / 8 * 8;
    static constexpr uint32_t kRegsSoftmax = 200, kRegsOther = TILES == 1 ? 56 : 80;
    static_assert(kSoftmaxWarps * 32 * kRegsSoftmax + 128 * kRegsOther <= kThreads * kRegsLaunch, "register split");
    static constexpr int kChunks = D / 32;
    static constexpr int kTileBytes = kChunks * kChunkBytes;
    static constexpr int kStages = TILES == 1 ? (D == 64 ? 2 : 1) : D == 64 ? 5 : D == 96 ? 3 : 2;
    static constexpr int kKSteps = D / 16;
    // TMEM: S_0 (S_1), O_0 (O_1), and where it fits a P buffer of 64 columns that
    // the tiles take in turn; else P_t is written over S_t.
    static constexpr uint32_t kTmemCols = 256 * TILES;
    __host__ __device__ static constexpr uint32_t col_o(int t) { return 128u * TILES + (t ? D : 0); }
    static constexpr uint32_t kColP = 128u * TILES + TILES * D;
    static constexpr bool kSepP = kColP + 64 <= kTmemCols;
};

// What one CTA works on.
struct Work {
    PackedSeq s;
    int kvh, split;
    int t0;        // first query of tile 0, in the sequence
    int queries;   // queries of the sequence that count
    int begin;     // first key of the part
    int end0, end1;  // one past the last key any row of tile 0, 1 attends in this part
    int n0, n1;      // 128-key steps of tile 0, 1
    int last;        // the tile with the most steps: 1 if it exists, else 0
    int clean;       // steps before the first in which some row does not attend some key
    int none;        // no work
    __device__ __forceinline__ int end(int t) const { return t ? end1 : end0; }
    __device__ __forceinline__ int n(int t) const { return t ? n1 : n0; }
    __device__ __forceinline__ int steps() const { return last ? n1 : n0; }
};

// What the issuing threads' loops need of it, in registers.
struct Steps {
    int n0, n1, last;
    __device__ __forceinline__ explicit Steps(const Work& w) : n0(w.n0), n1(w.n1), last(w.last) {}
    __device__ __forceinline__ int n(int t) const { return t ? n1 : n0; }
    __device__ __forceinline__ int steps() const { return last ? n1 : n0; }
};

template <class G>
struct Smem {
    static constexpr int kStages = G::kStages;
    uint8_t q[G::kTiles][G::kTileBytes];
    uint8_t k[kStages][G::kTileBytes];
    uint8_t v[kStages][G::kTileBytes];
    uint64_t q_full[2];
    uint64_t k_full[kStages], k_empty[kStages];
    uint64_t v_full[kStages], v_ready[kStages], v_empty[kStages];
    uint64_t s_full[2], p_full[2], o_done[2];
    uint64_t s_read[2];   // separate P: S_t has been read into registers
    uint64_t pv_done[2];  // separate P: PV_t(j) has completed (P buffer free)
    uint64_t mma_drain, pv_drain;
    Work work;  // in shared memory: what is needed after the main loop does not sit in registers during it
    int64_t place[G::kSoftmaxWarps][32];  // where each softmax warp's rows go, in elements; -1: nowhere
    uint32_t tmem_base;
    int abort_flag;
    int never;      // stays 0: abort flag for waits that must ignore an abort
    int nonfinite;  // a value of V was cleared
};

struct TileArgs {
    PackedArgs p;
    int pairs;     // CTAs a kv head may have over all sequences
    int per_tile;  // T: queries of a tile
    int* status;
    uint64_t timeout_ns;
};

__device__ __forceinline__ void raise_timeout(const TileArgs& a, volatile int* abort_flag) {
    *abort_flag = 1;
    atomicOr(a.status, kDevTimeout);
}

__device__ __forceinline__ uint64_t kmajor_base(const uint8_t* tile) {
    return smem_desc(smem_u32(tile), 16, 512, kSwizzle64);
}
__host__ __device__ constexpr uint32_t kmajor_step(int s) {
    return static_cast<uint32_t>(((s >> 1) * kChunkBytes + (s & 1) * 32) >> 4);
}
__device__ __forceinline__ uint64_t mnmajor_base(const uint8_t* tile) {
    return smem_desc(smem_u32(tile), kChunkBytes, 512, kSwizzle64);
}
__host__ __device__ constexpr uint32_t mnmajor_step(int s) { return static_cast<uint32_t>((s * 16 * 64) >> 4); }

// Instruction descriptor of kind::f16 with fp32 accumulation; both operands bf16 or both fp16.
template <bool FP16>
constexpr uint32_t idesc(int M, int N, int a_mn, int b_mn) {
    return idesc_bf16_f32(M, N, a_mn, b_mn) & ~(FP16 ? (1u << 7) | (1u << 10) : 0u);
}

// Finds this CTA's work; false if there is none.  The whole warp takes part: 32
// sequences are tried at a time, each with all its entries, since a trip to
// memory is what this takes.
__device__ __forceinline__ bool find_work(const TileArgs& a, int tiles, Work& w) {
    const int lane = threadIdx.x & 31;
    const int at = blockIdx.x / a.p.kv_heads, pair = a.pairs - 1 - at;
    w.kvh = blockIdx.x - at * a.p.kv_heads;
    w.split = blockIdx.y;
    const uint32_t span = tiles * a.per_tile;
    int lo = 0, hi = a.p.seqs;  // the last sequence in [lo, hi) whose pairs start at or before this one
    PackedSeq mine;
    int first;
    for (;;) {
        const int step = (hi - lo + 31) / 32, probe = lo + lane * step;
        mine = packed_seq(a.p, min(probe, a.p.seqs - 1));
        first = static_cast<int>(static_cast<uint32_t>(mine.q0) / span) + probe;
        // lane 0 stands for lo itself
        const uint32_t yes = __ballot_sync(0xffffffffu, lane == 0 || (probe < hi && first <= pair));
        const int winner = 31 - __clz(yes);
        if (step == 1) {
            w.s.q0 = __shfl_sync(0xffffffffu, mine.q0, winner);
            w.s.k0 = __shfl_sync(0xffffffffu, mine.k0, winner);
            w.s.lq = __shfl_sync(0xffffffffu, mine.lq, winner);
            w.s.lk = __shfl_sync(0xffffffffu, mine.lk, winner);
            first = __shfl_sync(0xffffffffu, first, winner);
            break;
        }
        lo += winner * step;
        hi = min(hi, lo + step);
    }
    const int64_t t0 = static_cast<int64_t>(pair - first) * static_cast<int>(span);
    w.queries = static_cast<int>(min(static_cast<int64_t>(w.s.lq), a.p.max_q));
    if (t0 < 0 || t0 >= w.queries) return false;
    w.t0 = static_cast<int>(t0);
    w.last = tiles == 2 && w.t0 + a.per_tile < w.queries ? 1 : 0;
    w.begin = 0;
    w.end1 = w.n1 = 0;
    for (int t = 0; t <= w.last; ++t) {
        const int last_query = min(w.t0 + (t + 1) * a.per_tile, w.queries) - 1;
        const int64_t limit = packed_limit(a.p, w.s, last_query);
        const int64_t begin = min(static_cast<int64_t>(w.split) * a.p.chunk, int64_t(0x7fffffff) & ~int64_t(127));
        const int64_t end = w.split + 1 == a.p.splits ? limit : min(limit, begin + a.p.chunk);
        w.begin = static_cast<int>(begin);
        const int n = end > begin ? static_cast<int>((end - begin + 127) / 128) : 0;
        (t ? w.end1 : w.end0) = static_cast<int>(end);
        (t ? w.n1 : w.n0) = n;
    }
    const int least = packed_limit(a.p, w.s, w.t0);
    w.clean = least > w.begin ? (least - w.begin) / 128 : 0;
    // later parts without keys are not read; the first one also stands for a row without any
    return w.split == 0 || w.steps() > 0;
}

// The loads of one step of K or V into buffer `stage`.
template <class G>
__device__ __forceinline__ void load_kv(uint8_t* tile, const CUtensorMap* map, uint64_t* full, const Work& w, int j) {
    mbar_arrive_expect_tx(full, G::kTileBytes);
    const int row = static_cast<int>(w.s.k0) + w.begin + j * 128;
    for (int c = 0; c < G::kChunks; ++c) tma_load_4d(tile + c * kChunkBytes, map, full, 32 * c, w.kvh, row, 0);
}

template <class G>
__device__ __forceinline__ void load_q(Smem<G>& sm, const TileArgs& a, const CUtensorMap* map, const Work& w, int t) {
    mbar_arrive_expect_tx(&sm.q_full[t], G::kChunks * 64u * static_cast<uint32_t>(a.per_tile * a.p.group));
    const int row = static_cast<int>(w.s.q0) + w.t0 + t * a.per_tile;
    for (int c = 0; c < G::kChunks; ++c) tma_load_4d(sm.q[t] + c * kChunkBytes, map, &sm.q_full[t], 32 * c, 0, w.kvh, row);
}

// The first loads, before the CTA's other warps are ready: the first K behind the
// first Q, since the first MMA waits for these two.  A tile without steps needs no
// Q (its rows' zeros go out through that memory).
template <class G>
__device__ __forceinline__ void load_first(Smem<G>& sm, const TileArgs& a, const Work& w, const CUtensorMap* tq, const CUtensorMap* tk,
                                           const CUtensorMap* tv) {
    if (w.n0 > 0) load_q(sm, a, tq, w, 0);
    if (w.steps() == 0) return;
    load_kv<G>(sm.k[0], tk, &sm.k_full[0], w, 0);
    if (w.n1 > 0) load_q(sm, a, tq, w, G::kTiles - 1);
    load_kv<G>(sm.v[0], tv, &sm.v_full[0], w, 0);
}

template <class G>
__device__ void producer(Smem<G>& sm, const TileArgs& a, const Work& w, const CUtensorMap* tk, const CUtensorMap* tv,
                         volatile int* abort_flag) {
    const int n = w.steps();
    bool ok = true;
    int issued_k = min(n, 1), issued_v = issued_k;
    uint32_t stage = G::kStages > 1 ? 1 : 0, phase = G::kStages > 1 ? 0 : 1;
    for (int j = 1; j < n; ++j) {
        if (!(ok = mbar_wait(&sm.k_empty[stage], phase ^ 1u, abort_flag, a.timeout_ns))) break;
        load_kv<G>(sm.k[stage], tk, &sm.k_full[stage], w, j);
        ++issued_k;
        if (!(ok = mbar_wait(&sm.v_empty[stage], phase ^ 1u, abort_flag, a.timeout_ns))) break;
        load_kv<G>(sm.v[stage], tv, &sm.v_full[stage], w, j);
        ++issued_v;
        if (++stage == G::kStages) {
            stage = 0;
            phase ^= 1u;
        }
    }
    if (!ok) raise_timeout(a, abort_flag);
    // Drain: every load issued must have landed before the CTA may exit.
    volatile int* never = &sm.never;
    if (w.n0 > 0) mbar_wait(&sm.q_full[0], 0u, never, a.timeout_ns);
    if (w.n1 > 0) mbar_wait(&sm.q_full[1], 0u, never, a.timeout_ns);
    for (int i = max(0, issued_k - G::kStages); i < issued_k; ++i)
        mbar_wait(&sm.k_full[i % G::kStages], (i / G::kStages) & 1u, never, a.timeout_ns);
    for (int i = max(0, issued_v - G::kStages); i < issued_v; ++i)
        mbar_wait(&sm.v_full[i % G::kStages], (i / G::kStages) & 1u, never, a.timeout_ns);
}

// The last warp: passes each V tile on, cleared of infinities and NaN where some row
// does not attend some key of the step.
template <class G, bool FP16>
__device__ void scan_values(Smem<G>& sm, const TileArgs& a, const Work& w, volatile int* abort_flag) {
    const int lane = threadIdx.x & 31, n = w.steps(), clean = w.clean;
    uint32_t stage = 0, phase = 0;
    for (int j = 0; j < n; ++j) {
        if (!__all_sync(0xffffffffu, mbar_wait(&sm.v_full[stage], phase, abort_flag, a.timeout_ns))) {
            if (lane == 0) raise_timeout(a, abort_flag);
            return;
        }
        if (j >= clean) {
            // 0 * x is NaN for the values looked for and changes nothing else
            uint4* tile = reinterpret_cast<uint4*>(sm.v[stage]);
            uint32_t sum[4] = {0, 0, 0, 0};
#pragma unroll 8
            for (int i = lane; i < G::kTileBytes / 16; i += 32) {
                const uint4 x = tile[i];
                sum[0] = Half16<FP16>::add_zero_times(x.x, sum[0]), sum[1] = Half16<FP16>::add_zero_times(x.y, sum[1]);
                sum[2] = Half16<FP16>::add_zero_times(x.z, sum[2]), sum[3] = Half16<FP16>::add_zero_times(x.w, sum[3]);
            }
            if (nonfinite_halves<FP16>(sum[0]) | nonfinite_halves<FP16>(sum[1]) | nonfinite_halves<FP16>(sum[2]) |
                nonfinite_halves<FP16>(sum[3])) {
                for (int i = lane; i < G::kTileBytes / 16; i += 32) {
                    uint4 x = tile[i];
                    x.x = finite_or_zero<FP16>(x.x, nonfinite_halves<FP16>(x.x));
                    x.y = finite_or_zero<FP16>(x.y, nonfinite_halves<FP16>(x.y));
                    x.z = finite_or_zero<FP16>(x.z, nonfinite_halves<FP16>(x.z));
                    x.w = finite_or_zero<FP16>(x.w, nonfinite_halves<FP16>(x.w));
                    tile[i] = x;
                }
                *reinterpret_cast<volatile int*>(&sm.nonfinite) = 1;
            }
            fence_proxy_async_shared();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.v_ready[stage]);
        if (++stage == G::kStages) {
            stage = 0;
            phase ^= 1u;
        }
    }
}

struct MmaState {
    uint64_t dq0, dq1, dk, dv;  // base descriptors: Q tiles, K stage 0, V stage 0
};

// S_t(j) = Q_t K(j)^T.  The first tile of a step waits for K, the last one releases it.
template <class G, bool FP16>
__device__ __forceinline__ bool issue_qk(Smem<G>& sm, const TileArgs& a, const Steps& w, const MmaState& st,
                                         uint32_t tmem, int t, int j, volatile int* abort_flag) {
    const uint32_t stage = static_cast<uint32_t>(j) % G::kStages, phase = (static_cast<uint32_t>(j) / G::kStages) & 1u;
    if (!mbar_wait(&sm.k_full[stage], phase, abort_flag, a.timeout_ns)) return false;
    tc_fence_after_sync();
    constexpr uint32_t id = idesc<FP16>(128, 128, 0, 0);
    const uint64_t dq = t ? st.dq1 : st.dq0, dk = st.dk + stage * (G::kTileBytes >> 4);
    const uint32_t d = tmem + col_s(t);
#pragma unroll
    for (int s = 0; s < G::kKSteps; ++s) mma_ss(d, dq + kmajor_step(s), dk + kmajor_step(s), id, s > 0 ? 1u : 0u);
    tc_commit(&sm.s_full[t]);
    if (t == w.last) tc_commit(&sm.k_empty[stage]);
    return true;
}

// O_t += P_t(j) V(j).
template <class G, bool FP16>
__device__ __forceinline__ bool issue_pv(Smem<G>& sm, const TileArgs& a, const Steps& w, const MmaState& st,
                                         uint32_t tmem, int t, int j, volatile int* abort_flag) {
    const uint32_t stage = static_cast<uint32_t>(j) % G::kStages, phase = (static_cast<uint32_t>(j) / G::kStages) & 1u;
    if (!mbar_wait(&sm.v_ready[stage], phase, abort_flag, a.timeout_ns)) return false;
    tc_fence_after_sync();
    constexpr uint32_t id = idesc<FP16>(128, G::D, 0, 1);
    const uint64_t dv = st.dv + stage * (G::kTileBytes >> 4);
    const uint32_t d = tmem + G::col_o(t), pa = tmem + (G::kSepP ? G::kColP : col_s(t));
    mma_ts(d, pa, dv, id, j > 0 ? 1u : 0u);
#pragma unroll
    for (int s = 1; s < 8; ++s) mma_ts(d, pa + 8 * s, dv + mnmajor_step(s), id, 1u);
    if (t == w.last) tc_commit(&sm.v_empty[stage]);
    return true;
}

// Separate P: QK^T and PV touch disjoint TMEM and have a thread each.
template <class G, bool FP16>
__device__ void qk_issuer(Smem<G>& sm, const TileArgs& a, const Work& work, uint32_t tmem, volatile int* abort_flag) {
    const Steps w(work);
    if (w.steps() == 0) return;
    MmaState st;
    st.dq0 = kmajor_base(sm.q[0]);
    st.dq1 = kmajor_base(sm.q[G::kTiles - 1]);
    st.dk = kmajor_base(sm.k[0]);
    bool ok = true;
    for (int j = 0; j < w.steps() && ok; ++j)
        for (int t = 0; t <= w.last && ok; ++t) {
            if (j >= w.n(t)) continue;
            ok = j == 0 ? mbar_wait(&sm.q_full[t], 0u, abort_flag, a.timeout_ns)
                        : mbar_wait(&sm.s_read[t], static_cast<uint32_t>((j - 1) & 1), abort_flag, a.timeout_ns);
            if (!ok) break;
            tc_fence_after_sync();
            ok = issue_qk<G, FP16>(sm, a, w, st, tmem, t, j, abort_flag);
        }
    if (!ok) raise_timeout(a, abort_flag);
    // Drain: every MMA this thread issued must have completed before TMEM is released.
    tc_commit(&sm.mma_drain);
    mbar_wait(&sm.mma_drain, 0u, &sm.never, a.timeout_ns);
}

template <class G, bool FP16>
__device__ void pv_issuer(Smem<G>& sm, const TileArgs& a, const Work& work, uint32_t tmem, volatile int* abort_flag) {
    const Steps w(work);
    if (w.steps() == 0) return;
    MmaState st;
    st.dv = mnmajor_base(sm.v[0]);
    bool ok = true;
    for (int j = 0; j < w.steps() && ok; ++j)
        for (int t = 0; t <= w.last && ok; ++t) {
            if (j >= w.n(t)) continue;
            ok = mbar_wait(&sm.p_full[t], static_cast<uint32_t>(j & 1), abort_flag, a.timeout_ns);
            if (!ok) break;
            tc_fence_after_sync();
            ok = issue_pv<G, FP16>(sm, a, w, st, tmem, t, j, abort_flag);
            if (!ok) break;
            tc_commit(&sm.pv_done[t]);
            if (j + 1 == w.n(t)) tc_commit(&sm.o_done[t]);
        }
    if (!ok) raise_timeout(a, abort_flag);
    tc_commit(&sm.pv_drain);
    mbar_wait(&sm.pv_drain, 0u, &sm.never, a.timeout_ns);
}

// P over S: one thread, PV_t(j) then QK_t(j+1) per tile (the QK overwrites the
// columns the PV reads; MMAs of one thread complete in issue order).
template <class G, bool FP16>
__device__ void mma_issuer(Smem<G>& sm, const TileArgs& a, const Work& work, uint32_t tmem, volatile int* abort_flag) {
    const Steps w(work);
    if (w.steps() == 0) return;
    MmaState st;
    st.dq0 = kmajor_base(sm.q[0]);
    st.dq1 = kmajor_base(sm.q[G::kTiles - 1]);
    st.dk = kmajor_base(sm.k[0]);
    st.dv = mnmajor_base(sm.v[0]);
    bool ok = true;
    for (int t = 0; t <= w.last && ok; ++t)
        if (w.n(t) > 0)
            ok = mbar_wait(&sm.q_full[t], 0u, abort_flag, a.timeout_ns) && issue_qk<G, FP16>(sm, a, w, st, tmem, t, 0, abort_flag);
    for (int j = 0; j < w.steps() && ok; ++j)
        for (int t = 0; t <= w.last && ok; ++t) {
            if (j >= w.n(t)) continue;
            ok = mbar_wait(&sm.p_full[t], static_cast<uint32_t>(j & 1), abort_flag, a.timeout_ns);
            if (!ok) break;
            tc_fence_after_sync();
            ok = issue_pv<G, FP16>(sm, a, w, st, tmem, t, j, abort_flag);
            if (!ok) break;
            if (j + 1 < w.n(t))
                ok = issue_qk<G, FP16>(sm, a, w, st, tmem, t, j + 1, abort_flag);
            else
                tc_commit(&sm.o_done[t]);
        }
    if (!ok) raise_timeout(a, abort_flag);
    tc_commit(&sm.mma_drain);
    mbar_wait(&sm.mma_drain, 0u, &sm.never, a.timeout_ns);
}

__device__ __forceinline__ uint32_t (&slice32(uint32_t* x))[32] { return *reinterpret_cast<uint32_t(*)[32]>(x); }
__device__ __forceinline__ uint32_t (&slice16(uint32_t* x))[16] { return *reinterpret_cast<uint32_t(*)[16]>(x); }

// O row *= alpha.  Out of line: it runs only when a row's maximum grew by more than 2^8.
template <class G>
__device__ __noinline__ void rescale_o(uint32_t tO, float alpha) {
#pragma unroll 1
    for (int cc = 0; cc < G::kChunks; ++cc) {
        uint32_t o[32];
        tmem_ld_x32(tO + 32u * cc, o);
        tmem_wait_ld_x32(o);
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
        tmem_st_x32(tO + 32u * cc, o);
    }
}

// Adds the infinities and NaN that 32 channels of V hold among keys [from, to)
// to o: what was cleared, for a row that attends those keys.
template <bool FP16>
__device__ __noinline__ void add_nonfinite(float* o, const uint16_t* v, int64_t vn, int from, int to) {
    for (int key = from; key < to; ++key) {
        const uint32_t* p = reinterpret_cast<const uint32_t*>(v + key * vn);
        for (int i = 0; i < 16; ++i) {
            const uint32_t x = p[i];
            if (nonfinite_halves<FP16>(x) == 0) continue;
            float lo, hi;
            Half16<FP16>::unpack(x, lo, hi);
            o[2 * i] += isfinite(lo) ? 0.f : lo;
            o[2 * i + 1] += isfinite(hi) ? 0.f : hi;
        }
    }
}

// Softmax of query tile t: thread r owns row r (TMEM lane r), all 128 keys of a step.
template <class G, bool FP16>
__device__ void softmax_group(Smem<G>& sm, const TileArgs& a, const Work& w, uint32_t tmem, int t, volatile int* abort_flag) {
    using H = Half16<FP16>;
    constexpr int D = G::D;
    constexpr bool kSep = G::kSepP;
    const int lane = threadIdx.x & 31;
    const int quarter = (threadIdx.x >> 5) & 3;  // TMEM lanes [32*quarter, 32*quarter + 32)
    const int row = quarter * 32 + lane;
    const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tS = tmem + lane_addr + col_s(t);
    const uint32_t tO = tmem + lane_addr + G::col_o(t);
    const uint32_t tP = tmem + lane_addr + G::kColP;
    const int n = w.n(t), n0 = w.n0, last = w.last;
    // the row's query in the sequence, -1 if it has none
    auto query_of_row = [&]() {
        const int query = w.t0 + t * a.per_tile + row / a.p.group;
        return row < a.per_tile * a.p.group && query < w.queries ? query : -1;
    };
    // Keys of the tile that the row attends.  Rows that are no query's see what the
    // tile sees (and are not written), so that they do not cost their warp the
    // comparisons.
    auto limit_of = [&](int query) { return query >= 0 ? min(packed_limit(a.p, w.s, query), w.end(t)) : w.end(t); };
    const bool in = G::kTiles == 1 && query_of_row() >= 0;
    int valid = max(limit_of(query_of_row()) - w.begin, 0);  // keys of the step and behind that the row attends
    // Separate P: before this tile writes the shared P buffer at step j, the PV
    // that last read it must have completed -- the other tile's of step j - 1
    // (tile 0) or j (tile 1) as long as that tile runs, else this tile's own of
    // step j - 1.  It was issued after PV_t(j-1), so O_t is stable too.  The
    // wait names a phase at most one ahead of the barrier's last completed one.
    auto wait_p_buffer = [&](int j) -> bool {
        const bool other = t == 0 ? last == 1 : j < n0;
        const int u = other ? 1 - t : t;
        const int ph = other && t == 1 ? j : j - 1;
        if (ph < 0) return true;
        const bool r = __all_sync(0xffffffffu, mbar_wait(&sm.pv_done[u], static_cast<uint32_t>(ph & 1), abort_flag, a.timeout_ns));
        if (r) tc_fence_after_sync();
        return r;
    };
    const float c = a.p.scale_log2;
    float m_used = -INFINITY;  // row reference of scaled logits (log2 units); -inf: no key yet
    float l = 0.f;
    bool ok = true;
    for (int j = 0; j < n; ++j, valid -= 128) {
        if (!__all_sync(0xffffffffu, mbar_wait(&sm.s_full[t], static_cast<uint32_t>(j & 1), abort_flag, a.timeout_ns))) {
            ok = false;
            break;
        }
        tc_fence_after_sync();
        // Moves the reference to the step's maximum mx where it must (and O with
        // it): at the first step, and when a row's maximum grew by 2^8 or it had no
        // key before.  O_t must be stable then: with P over S the commit behind
        // s_full covers PV_t(j-1); with a separate P buffer, its wait does.
        bool p_free = false;
        auto refer = [&](float mx) -> bool {
            if (j == 0) {
                m_used = mx;
                return true;
            }
            const bool need = mx - m_used > 8.0f;
            if (__any_sync(0xffffffffu, need)) {
                if constexpr (kSep) {
                    if (!wait_p_buffer(j)) return false;
                    p_free = true;
                }
                float alpha = 1.0f;
                if (need) {
                    alpha = ex2_approx(m_used - mx);
                    m_used = mx;
                }
                l *= alpha;
                rescale_o<G>(tO, alpha);
            }
            return true;
        };
        auto s_is_read = [&]() {
            if constexpr (kSep) {
                // S_t is in registers: release it for QK_t(j+1)
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.s_read[t]);
            }
        };
        uint64_t acc[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
        const uint64_t c2 = f2(c, c);
        const bool partly = __any_sync(0xffffffffu, valid < 128);  // some row does not attend some key
        if (G::kTiles == 2 || !partly) {
            // the row in registers, all of it unrolled
            uint32_t x[128];
            float pm[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int q = 0; q < 2; ++q) tmem_ld_x32(tS + 32u * q, slice32(x + 32 * q));
#pragma unroll
            for (int q = 0; q < 2; ++q) tmem_wait_ld_x32(slice32(x + 32 * q));
#pragma unroll
            for (int q = 2; q < 4; ++q) tmem_ld_x32(tS + 32u * q, slice32(x + 32 * q));
            if (G::kTiles == 2 && partly) {
#pragma unroll
                for (int i = 0; i < 64; ++i)
                    if (i >= valid) x[i] = __float_as_uint(-INFINITY);
            }
            // first half's max while the second half loads
#pragma unroll
            for (int i = 0; i < 32; ++i)
                pm[i & 3] = max3(pm[i & 3], __uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]));
#pragma unroll
            for (int q = 2; q < 4; ++q) tmem_wait_ld_x32(slice32(x + 32 * q));
            s_is_read();
            if (G::kTiles == 2 && partly) {
#pragma unroll
                for (int i = 64; i < 128; ++i)
                    if (i >= valid) x[i] = __float_as_uint(-INFINITY);
            }
#pragma unroll
            for (int i = 32; i < 64; ++i)
                pm[i & 3] = max3(pm[i & 3], __uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]));
            if (!(ok = refer(c * fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3]))))) break;
            const float ref = m_used == -INFINITY ? 0.f : m_used;  // no key yet: weights 2^-inf = 0
            const uint64_t nm2 = f2(-ref, -ref);
#pragma unroll
            for (int i = 0; i < 64; ++i) {
                float a0, a1;
                f2_split(f2_fma(f2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), c2, nm2), a0, a1);
                const float p0 = ex2_approx(a0), p1 = ex2_approx(a1);
                acc[i & 1] = f2_add(acc[i & 1], f2(p0, p1));
                x[i] = H::pack(p0, p1);
                if constexpr (!kSep)
                    if ((i & 15) == 15) tmem_st_x16(tS + (i - 15), slice16(x + (i - 15)));
            }
            if constexpr (kSep) {
                if (!p_free && !(ok = wait_p_buffer(j))) break;
                tmem_st_x32(tP, slice32(x));
                tmem_st_x32(tP + 32u, slice32(x + 32));
            }
        } else {
            // One tile, where the keys end or the diagonal passes: 32 columns at a
            // time, as far as any row of the warp attends them, S read once for the
            // maximum and once for the weights.  Not unrolled: a short sequence
            // runs through this once or twice, and fetching the instructions is
            // then most of what it costs.  (16 prompts of up to 1,000, 16 heads x
            // 64: 39.0 us against 45.6 by the row in registers.  With two tiles,
            // which take turns at the tensor core, the longer step costs more than
            // it saves: 52.2 us against 46.9.)
            const int top = __reduce_max_sync(0xffffffffu, in ? min(max(valid, 0), 128) : 0);
            float mx = -INFINITY;
#pragma unroll 1
            for (int k = 0; k < top; k += 32) {
                uint32_t x[32];
                tmem_ld_x32(tS + k, x);
                tmem_wait_ld_x32(x);
#pragma unroll
                for (int i = 0; i < 32; ++i) mx = fmaxf(mx, k + i < valid ? __uint_as_float(x[i]) : -INFINITY);
            }
            if (!(ok = refer(c * mx))) break;
            const float ref = m_used == -INFINITY ? 0.f : m_used;
            const uint64_t nm2 = f2(-ref, -ref);
            if constexpr (kSep)
                if (!p_free && !(ok = wait_p_buffer(j))) break;
#pragma unroll 1
            for (int k = 0; k < 128; k += 32) {
                uint32_t x[32];
                if (k < top) {
                    tmem_ld_x32(tS + k, x);
                    tmem_wait_ld_x32(x);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float a0, a1;
                        f2_split(f2_fma(f2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), c2, nm2), a0, a1);
                        const float p0 = k + 2 * i < valid ? ex2_approx(a0) : 0.f, p1 = k + 2 * i + 1 < valid ? ex2_approx(a1) : 0.f;
                        acc[i & 1] = f2_add(acc[i & 1], f2(p0, p1));
                        x[i] = H::pack(p0, p1);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[i] = 0;
                }
                tmem_st_x16((kSep ? tP : tS) + k / 2, slice16(x));  // P over S: behind what was read last
            }
            s_is_read();
        }
        float s0, s1, s2, s3;
        f2_split(acc[0], s0, s1);
        f2_split(acc[1], s2, s3);
        l += (s0 + s1) + (s2 + s3);
        // one arrival per warp: every lane's TMEM stores are complete and fenced
        tmem_wait_st();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full[t]);
    }
    if (ok && n > 0) ok = __all_sync(0xffffffffu, mbar_wait(&sm.o_done[t], 0u, abort_flag, a.timeout_ns));
    if (!ok) {
        raise_timeout(a, abort_flag);
        return;
    }
    // what the rows' end needs is worked out again: it does not sit in registers during the loop
    const int query = query_of_row();
    const bool there = query >= 0;
    if ((n == 0 && w.split > 0) || !__any_sync(0xffffffffu, there)) return;
    tc_fence_after_sync();
    const bool cleared = *reinterpret_cast<volatile int*>(&sm.nonfinite) != 0;
    const float inv_l = l == 0.f ? 0.f : 1.0f / l;
    const float lse2 = l == 0.f ? -INFINITY : m_used + log2f(l);
    const int head = w.kvh * a.p.group + row % a.p.group;
    const int64_t tok = w.s.q0 + query, qh = tok * a.p.heads + head;
    const bool split = a.p.splits > 1;
    // A warp's 32 rows go out through the Q tile's shared memory (no MMA reads
    // it any more), 64 bytes of each at a time, four lanes a row: a thread's own row
    // would be written 16 bytes here and 16 there.  16-byte pieces are swizzled by
    // the row so that neither side collides.
    const int64_t rows = a.p.total_q * a.p.heads;
    int64_t* places = sm.place[t * 4 + quarter];
    places[lane] = !there ? -1 : split ? (w.split * rows + qh) * D : tok * a.p.on + head * a.p.oh;
    __syncwarp();
    int64_t at[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) at[i] = places[i * 8 + lane / 4];
    uint4* stage = reinterpret_cast<uint4*>(sm.q[t]) + quarter * 32 * (D / 8);
    const int mine = lane * 4, turn = (lane >> 1) & 3;
    auto theirs = [&](int i) { return (i * 8 + lane / 4) * 4 + ((lane & 3) ^ ((lane >> 3) & 3)); };
    // what was cleared, for a row that attends it
    auto restore = [&](uint32_t* x, int channel) {
        float tmp[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) tmp[i] = __uint_as_float(x[i]);
        add_nonfinite<FP16>(tmp, static_cast<const uint16_t*>(a.p.v) + w.s.k0 * a.p.vn + w.kvh * a.p.vh + channel, a.p.vn,
                            w.begin + 128 * w.clean, limit_of(query));
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(tmp[i]);
    };
    if (!split) {
        uint32_t x[D];
        if (n > 0) {
#pragma unroll
            for (int cc = 0; cc < G::kChunks; ++cc) tmem_ld_x32(tO + 32u * cc, slice32(x + 32 * cc));
#pragma unroll
            for (int cc = 0; cc < G::kChunks; ++cc) tmem_wait_ld_x32(slice32(x + 32 * cc));
        } else {
#pragma unroll
            for (int i = 0; i < D; ++i) x[i] = 0;
        }
#pragma unroll
        for (int cc = 0; cc < G::kChunks; ++cc) {
#pragma unroll
            for (int i = 32 * cc; i < 32 * cc + 32; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * inv_l);
            if (cleared && there) restore(x + 32 * cc, 32 * cc);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t h[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    h[e] = H::pack(__uint_as_float(x[32 * cc + 8 * i + 2 * e]), __uint_as_float(x[32 * cc + 8 * i + 2 * e + 1]));
                stage[128 * cc + mine + (i ^ turn)] = make_uint4(h[0], h[1], h[2], h[3]);
            }
        }
        __syncwarp();
#pragma unroll
        for (int cc = 0; cc < G::kChunks; ++cc)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 v = stage[128 * cc + theirs(i)];
                if (at[i] >= 0) reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.p.o) + at[i] + 32 * cc)[lane & 3] = v;
            }
    } else {
#pragma unroll 1
        for (int cc = 0; cc < G::kChunks; ++cc) {
            uint32_t x[32];
            if (n > 0) {
                tmem_ld_x32(tO + 32u * cc, x);
                tmem_wait_ld_x32(x);
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = 0;
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * inv_l);
            if (cleared && there) restore(x, 32 * cc);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    stage[128 * h + mine + (i ^ turn)] =
                        make_uint4(x[16 * h + 4 * i], x[16 * h + 4 * i + 1], x[16 * h + 4 * i + 2], x[16 * h + 4 * i + 3]);
            }
            __syncwarp();
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint4 v = stage[128 * h + theirs(i)];
                    if (at[i] >= 0) reinterpret_cast<uint4*>(a.p.part_o + at[i] + 32 * cc + 16 * h)[lane & 3] = v;
                }
            __syncwarp();
        }
    }
    if (there) {
        if (split)
            a.p.part_lse[w.split * rows + qh] = lse2;
        else if (a.p.lse)
            a.p.lse[qh] = lse2 * 0.6931471805599453f;
    }
}

template <class G, bool FP16>
__global__ void __launch_bounds__(G::kThreads, G::kCtas)
    packed_tiles_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                        const __grid_constant__ CUtensorMap tv, const __grid_constant__ TileArgs a) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = smem_u32(smem_raw);
    Smem<G>& sm = *reinterpret_cast<Smem<G>*>(smem_raw + (((base + 1023u) & ~1023u) - base));
    const int warp = threadIdx.x >> 5;
    if (warp == G::kProducerWarp) {
        // the work and its first loads, while the other warps set up the rest
        if ((threadIdx.x & 31) == 0) {
            prefetch_tensor_map(&tq);
            prefetch_tensor_map(&tk);
            prefetch_tensor_map(&tv);
            for (int t = 0; t < 2; ++t) mbar_init(&sm.q_full[t], 1);
            for (int s = 0; s < G::kStages; ++s) {
                mbar_init(&sm.k_full[s], 1);
                mbar_init(&sm.k_empty[s], 1);
                mbar_init(&sm.v_full[s], 1);
                mbar_init(&sm.v_ready[s], 1);
                mbar_init(&sm.v_empty[s], 1);
            }
            fence_barrier_init();
        }
        __syncwarp();
        wait_for_previous();
        Work mine;
        mine.none = !find_work(a, G::kTiles, mine);
        if ((threadIdx.x & 31) == 0) {
            if (!mine.none) load_first<G>(sm, a, mine, &tq, &tk, &tv);
            sm.work = mine;
        }
    } else if (warp == G::kMmaWarp) {
        tmem_alloc(&sm.tmem_base, G::kTmemCols);
        tmem_relinquish();
        let_next_start();  // not before: see launch_early
    } else if (threadIdx.x == 0) {
        for (int t = 0; t < 2; ++t) {
            mbar_init(&sm.s_full[t], 1);
            mbar_init(&sm.p_full[t], 4);  // one arrival per softmax warp of the tile
            mbar_init(&sm.o_done[t], 1);
            mbar_init(&sm.s_read[t], 4);
            mbar_init(&sm.pv_done[t], 1);
        }
        mbar_init(&sm.mma_drain, 1);
        mbar_init(&sm.pv_drain, 1);
        sm.abort_flag = 0;
        sm.never = 0;
        sm.nonfinite = 0;
        fence_barrier_init();
    }
    __syncwarp();
    if (warp != G::kProducerWarp) wait_for_previous();
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const Work& w = sm.work;
    const uint32_t tmem = sm.tmem_base;
    volatile int* abort_flag = &sm.abort_flag;

    if (w.none) {
        // nothing to do
    } else if (warp < G::kSoftmaxWarps) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(G::kRegsSoftmax));
        const int t = warp >> 2;
        if (t <= w.last) softmax_group<G, FP16>(sm, a, w, tmem, t, abort_flag);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(G::kRegsOther));
        const bool one = (threadIdx.x & 31) == 0;
        if (warp == G::kProducerWarp) {
            if (one) producer<G>(sm, a, w, &tk, &tv, abort_flag);
        } else if (warp == G::kMmaWarp) {
            if (one) {
                if constexpr (G::kSepP)
                    qk_issuer<G, FP16>(sm, a, w, tmem, abort_flag);
                else
                    mma_issuer<G, FP16>(sm, a, w, tmem, abort_flag);
            }
        } else if (warp == G::kPvWarp) {
            if constexpr (G::kSepP)
                if (one) pv_issuer<G, FP16>(sm, a, w, tmem, abort_flag);
        } else {
            scan_values<G, FP16>(sm, a, w, abort_flag);
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == G::kMmaWarp) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, G::kTmemCols);
    }
}

template <class G, bool FP16>
cudaError_t run(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const TileArgs& a, cudaStream_t st) {
    constexpr size_t smem = sizeof(Smem<G>) + 1024;  // + alignment slack
    static_assert((smem + 1024) * G::kCtas <= 233472, "shared memory of a multiprocessor");
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(packed_tiles_kernel<G, FP16>), static_cast<int>(smem), done);
    if (e != cudaSuccess) return e;
    const dim3 grid(static_cast<unsigned>(a.pairs) * a.p.kv_heads, a.p.splits);
    return launch_early(packed_tiles_kernel<G, FP16>, grid, G::kThreads, smem, st, tq, tk, tv, a);
}

template <int TILES>
cudaError_t run(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const TileArgs& a, int d, bool fp16,
                cudaStream_t st) {
    switch (d) {
        case 64: return fp16 ? run<Geo<64, TILES>, true>(tq, tk, tv, a, st) : run<Geo<64, TILES>, false>(tq, tk, tv, a, st);
        case 96: return fp16 ? run<Geo<96, TILES>, true>(tq, tk, tv, a, st) : run<Geo<96, TILES>, false>(tq, tk, tv, a, st);
        default: return fp16 ? run<Geo<128, TILES>, true>(tq, tk, tv, a, st) : run<Geo<128, TILES>, false>(tq, tk, tv, a, st);
    }
}

}  // namespace

cudaError_t launch_packed_tiles(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const PackedArgs& p,
                                int d, bool fp16, int tiles, int* status, uint64_t timeout_ns, cudaStream_t st) {
    TileArgs a;
    a.p = p;
    a.pairs = static_cast<int>(packed_tile_groups(p.total_q, p.seqs, p.group, tiles));
    a.per_tile = packed_queries_per_tile(p.group);
    a.status = status;
    a.timeout_ns = timeout_ns;
    return tiles == 1 ? run<1>(tq, tk, tv, a, d, fp16, st) : run<2>(tq, tk, tv, a, d, fp16, st);
}

}  // namespace h3a
