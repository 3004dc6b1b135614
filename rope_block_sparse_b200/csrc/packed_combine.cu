// Joins the parts of sequences' keys (h3a_packed_attention): for every (query,
// head), o = sum_p w_p o_p / sum_p w_p with w_p = 2^(lse_p - max lse).  WARPS warps
// a row, each taking every WARPS-th part and keeping a running maximum: one
// where a row has few parts and there are many rows, four where a few rows have
// many.  Latency is what this costs, not bytes (the parts are fp32 and stay in
// L2): it takes two trips to memory, one for the row's sequence and its parts'
// places, one for four parts' log-sum-exps and rows together.
#include "half16.cuh"
#include "prompt_internal.h"

namespace h3a {
namespace {

constexpr int kThreads = 128;
constexpr int kAhead = 4;  // parts a warp has in flight

template <int D, bool FP16, int WARPS>
__global__ void __launch_bounds__(kThreads) packed_combine_kernel(const __grid_constant__ PackedArgs a) {
    using H = Half16<FP16>;
    constexpr int kPer = D / 32;  // channels a lane
    constexpr int kRows = kThreads / 32 / WARPS;
    __shared__ float joined[WARPS][D];
    __shared__ float joined_top[WARPS], joined_sum[WARPS];
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) % WARPS, row = (threadIdx.x >> 5) / WARPS;
    early_start();
    const int64_t qh = static_cast<int64_t>(blockIdx.x) * kRows + row;
    const int64_t n = qh / a.heads;
    const int head = static_cast<int>(qh - n * a.heads);
    if (n >= a.total_q) return;
    // the sequence of row n, the last one that starts at or before it, with all
    // its entries: 32 are tried at a time
    PackedSeq s;
    int2 ends = make_int2(0, 0);
    for (int lo = 0, hi = a.seqs;;) {
        const int step = (hi - lo + 31) / 32, probe = lo + lane * step, at = min(probe, a.seqs - 1);
        const PackedSeq mine = packed_seq(a, at);
        int2 mine_ends = ends;
        if (a.streams > 0) mine_ends = a.part_slots[at];
        const uint32_t yes = __ballot_sync(0xffffffffu, lane == 0 || (probe < hi && mine.q0 <= n));
        const int winner = 31 - __clz(yes);
        if (step == 1) {
            s.q0 = __shfl_sync(0xffffffffu, mine.q0, winner);
            s.k0 = 0;
            s.lq = __shfl_sync(0xffffffffu, mine.lq, winner);
            s.lk = __shfl_sync(0xffffffffu, mine.lk, winner);
            ends.x = __shfl_sync(0xffffffffu, mine_ends.x, winner);
            ends.y = __shfl_sync(0xffffffffu, mine_ends.y, winner);
            break;
        }
        lo += winner * step;
        hi = min(hi, lo + step);
    }
    const int queries = static_cast<int>(min(static_cast<int64_t>(s.lq), a.max_q));
    if (n < s.q0 || n - s.q0 >= queries) return;
    const int query = static_cast<int>(n - s.q0);
    // Part p's row is first + p * step (but for a stream's part 0: row0).
    int parts;
    int64_t row0, first, step;
    if (a.streams > 0) {
        const int kvh = head / a.group, r = query * a.group + head % a.group;
        const bool keys = packed_limit(a, s, queries - 1) > 0;
        if (keys && ends.x < 0) return;  // finished by one CTA
        // the parts after a sequence's first one begin their stretch
        parts = keys ? (ends.y >> 1) - (ends.x >> 1) + 1 : 0;
        row0 = packed_part_slot(a, ends.x, kvh) * kRowSlots + r;
        first = packed_part_slot(a, ends.x & ~1, kvh) * kRowSlots + r;
        step = packed_part_slot(a, 2, 0) * kRowSlots;
    } else {
        parts = min(a.splits, max(1, (packed_limit(a, s, query) + a.chunk - 1) / a.chunk));
        row0 = first = qh;
        step = a.total_q * a.heads;
    }
    float top = -INFINITY, sum = 0.f, acc[kPer] = {};
    for (int p = warp; p < parts; p += kAhead * WARPS) {
        float lse[kAhead], v[kAhead][kPer];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int part = p + u * WARPS;
            lse[u] = -INFINITY;
#pragma unroll
            for (int i = 0; i < kPer; ++i) v[u][i] = 0.f;
            if (part < parts) {
                const int64_t at = part == 0 ? row0 : first + part * step;
                lse[u] = a.part_lse[at];
#pragma unroll
                for (int i = 0; i < kPer; ++i) v[u][i] = a.part_o[at * D + lane + 32 * i];
            }
        }
        const float before = top;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) top = fmaxf(top, lse[u]);
        const float ref = top == -INFINITY ? 0.f : top;
        const float keep = exp2f(before - ref);
        sum *= keep;
#pragma unroll
        for (int i = 0; i < kPer; ++i) acc[i] *= keep;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const float w = exp2f(lse[u] - ref);
            sum += w;
#pragma unroll
            for (int i = 0; i < kPer; ++i) acc[i] = fmaf(w, v[u][i], acc[i]);
        }
    }
    if (WARPS > 1) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) joined[warp][lane + 32 * i] = acc[i];
        if (lane == 0) {
            joined_top[warp] = top;
            joined_sum[warp] = sum;
        }
        __syncthreads();  // all of the block's warps share the row
        if (warp != 0) return;
#pragma unroll
        for (int w = 1; w < WARPS; ++w) top = fmaxf(top, joined_top[w]);
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) acc[i] = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            const float f = exp2f(joined_top[w] - (top == -INFINITY ? 0.f : top));
            sum = fmaf(f, joined_sum[w], sum);
#pragma unroll
            for (int i = 0; i < kPer; ++i) acc[i] = fmaf(f, joined[w][lane + 32 * i], acc[i]);
        }
    }
    const float ref = top == -INFINITY ? 0.f : top;
    const float inv = sum == 0.f ? 0.f : 1.0f / sum;
    uint16_t* dst = static_cast<uint16_t*>(a.o) + n * a.on + head * a.oh + lane;
#pragma unroll
    for (int i = 0; i < kPer; ++i) dst[32 * i] = static_cast<uint16_t>(H::pack(acc[i] * inv, 0.f));
    if (a.lse && lane == 0) a.lse[qh] = sum == 0.f ? -INFINITY : (ref + log2f(sum)) * 0.6931471805599453f;
}

template <int D, bool FP16, int WARPS>
cudaError_t run(const PackedArgs& a, cudaStream_t st) {
    const int64_t rows = a.total_q * a.heads, per = kThreads / 32 / WARPS;
    return launch_early(packed_combine_kernel<D, FP16, WARPS>, dim3(static_cast<unsigned>((rows + per - 1) / per)), kThreads, 0, st, a);
}

template <int D>
cudaError_t run(const PackedArgs& a, bool fp16, cudaStream_t st) {
    if (a.streams > 8 * a.seqs || a.splits > 8) return fp16 ? run<D, true, 4>(a, st) : run<D, false, 4>(a, st);
    return fp16 ? run<D, true, 1>(a, st) : run<D, false, 1>(a, st);
}

}  // namespace

cudaError_t launch_packed_combine(const PackedArgs& a, int d, bool fp16, cudaStream_t st) {
    if (a.total_q == 0) return cudaSuccess;
    switch (d) {
        case 64: return run<64>(a, fp16, st);
        case 96: return run<96>(a, fp16, st);
        default: return run<128>(a, fp16, st);
    }
}

}  // namespace h3a
