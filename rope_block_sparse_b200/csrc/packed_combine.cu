// Joins the parts of split keys (h3a_packed_attention): for every (query,
// head), o = sum_s w_s o_s / sum_s w_s with w_s = 2^(lse_s - max lse), over the
// parts that cover the query's keys.  One warp a row; the parts' rows are fp32
// and stay in L2 between the two launches.
#include "half16.cuh"
#include "prompt_internal.h"

namespace h3a {
namespace {

constexpr int kThreads = 128;

template <int D, bool FP16>
__global__ void __launch_bounds__(kThreads) packed_combine_kernel(const PackedArgs a) {
    using H = Half16<FP16>;
    constexpr int kPer = D / 32;  // channels a lane
    const int lane = threadIdx.x & 31;
    const int64_t qh = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t n = qh / a.heads;
    const int head = static_cast<int>(qh % a.heads);
    if (n >= a.total_q) return;
    // the sequence of row n: the last one that starts at or before it
    if (n < __ldg(a.starts_q) || n >= __ldg(a.starts_q + a.seqs)) return;
    int lo = 0, hi = a.seqs;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(a.starts_q + mid) <= n) lo = mid; else hi = mid;
    }
    const PackedSeq s = packed_seq(a, lo);
    if (n < s.q0 || n - s.q0 >= min(static_cast<int64_t>(s.lq), a.max_q)) return;
    const int limit = packed_limit(a, s, static_cast<int>(n - s.q0));
    const int parts = min(a.splits, max(1, (limit + a.chunk - 1) / a.chunk));
    const int64_t step = a.total_q * a.heads;
    float top = -INFINITY;
    for (int p = lane; p < parts; p += 32) top = fmaxf(top, a.part_lse[p * step + qh]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float ref = top == -INFINITY ? 0.f : top;
    float acc[kPer] = {}, sum = 0.f;
    for (int p = 0; p < parts; ++p) {
        const float w = exp2f(a.part_lse[p * step + qh] - ref);
        if (w == 0.f) continue;
        sum += w;
        const float* src = a.part_o + (p * step + qh) * D + lane;
#pragma unroll
        for (int i = 0; i < kPer; ++i) acc[i] = fmaf(w, src[32 * i], acc[i]);
    }
    const float inv = sum == 0.f ? 0.f : 1.0f / sum;
    uint16_t* dst = static_cast<uint16_t*>(a.o) + n * a.on + head * a.oh + lane;
#pragma unroll
    for (int i = 0; i < kPer; ++i) dst[32 * i] = static_cast<uint16_t>(H::pack(acc[i] * inv, 0.f));
    if (a.lse && lane == 0) a.lse[qh] = sum == 0.f ? -INFINITY : (ref + log2f(sum)) * 0.6931471805599453f;
}

template <int D>
cudaError_t run(const PackedArgs& a, bool fp16, cudaStream_t st) {
    const int64_t warps = a.total_q * a.heads, per = kThreads / 32;
    const unsigned grid = static_cast<unsigned>((warps + per - 1) / per);
    if (fp16)
        packed_combine_kernel<D, true><<<grid, kThreads, 0, st>>>(a);
    else
        packed_combine_kernel<D, false><<<grid, kThreads, 0, st>>>(a);
    return cudaGetLastError();
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
