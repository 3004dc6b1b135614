// Joins the parts of split keys (h3a_packed_attention): for every (query,
// head), o = sum_s w_s o_s / sum_s w_s with w_s = 2^(lse_s - max lse), over the
// parts that cover the query's keys.  WARPS warps a row, each taking every
// WARPS-th part: one where a row has few parts and there are many rows, four
// where a few rows have many (a long cache split over the GPU: 16,000 keys of
// 32/8 heads x 128 in 84 parts took 42 us with one).  The weights are worked out
// first, one lane a part, so that the rows' loads do not wait for one another;
// the parts' rows are fp32 and stay in L2 between the two launches.
#include "half16.cuh"
#include "prompt_internal.h"

namespace h3a {
namespace {

constexpr int kThreads = 128;
constexpr int kMostParts = 256;  // packed_plan's limit

template <int D, bool FP16, int WARPS>
__global__ void __launch_bounds__(kThreads) packed_combine_kernel(const __grid_constant__ PackedArgs a) {
    using H = Half16<FP16>;
    constexpr int kPer = D / 32;  // channels a lane
    constexpr int kRows = kThreads / 32 / WARPS;
    __shared__ float weight[kRows][kMostParts];
    __shared__ float joined[WARPS][D];
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) % WARPS, row = (threadIdx.x >> 5) / WARPS;
    // launched while the parts are still computed (run): wait for them
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t qh = static_cast<int64_t>(blockIdx.x) * kRows + row;
    const int64_t n = qh / a.heads;
    const int head = static_cast<int>(qh % a.heads);
    if (n >= a.total_q) return;
    // the sequence of row n: the last one that starts at or before it
    if (n < __ldg(a.starts_q) || n >= __ldg(a.starts_q + a.seqs)) return;
    int lo = 0, hi = a.seqs;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, probe = lo + lane * step;
        const uint32_t yes = __ballot_sync(0xffffffffu, lane == 0 || (probe < hi && __ldg(a.starts_q + probe) <= n));
        lo += (31 - __clz(yes)) * step;
        hi = min(hi, lo + step);
    }
    const PackedSeq s = packed_seq(a, lo);
    if (n < s.q0 || n - s.q0 >= min(static_cast<int64_t>(s.lq), a.max_q)) return;
    const int limit = packed_limit(a, s, static_cast<int>(n - s.q0));
    const int parts = min(a.splits, max(1, (limit + a.chunk - 1) / a.chunk));
    const int64_t step = a.total_q * a.heads;
    // every warp of the row works out all weights: the sum needs no barrier then
    float top = -INFINITY;
    for (int p = lane; p < parts; p += 32) top = fmaxf(top, a.part_lse[p * step + qh]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float ref = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
    for (int p = lane; p < parts; p += 32) {
        const float w = exp2f(a.part_lse[p * step + qh] - ref);
        sum += w;
        if (p % WARPS == warp) weight[row][p] = w;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    __syncwarp();
    float acc[kPer] = {};
#pragma unroll 4
    for (int p = warp; p < parts; p += WARPS) {
        const float w = weight[row][p];
        const float* src = a.part_o + (p * step + qh) * D + lane;
#pragma unroll
        for (int i = 0; i < kPer; ++i) acc[i] = fmaf(w, src[32 * i], acc[i]);
    }
    if (WARPS > 1) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) joined[warp][lane + 32 * i] = acc[i];
        __syncthreads();  // all of the block's warps share the row
        if (warp != 0) return;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            acc[i] = 0.f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) acc[i] += joined[w][lane + 32 * i];
        }
    }
    const float inv = sum == 0.f ? 0.f : 1.0f / sum;
    uint16_t* dst = static_cast<uint16_t*>(a.o) + n * a.on + head * a.oh + lane;
#pragma unroll
    for (int i = 0; i < kPer; ++i) dst[32 * i] = static_cast<uint16_t>(H::pack(acc[i] * inv, 0.f));
    if (a.lse && lane == 0) a.lse[qh] = sum == 0.f ? -INFINITY : (ref + log2f(sum)) * 0.6931471805599453f;
}

template <int D, bool FP16, int WARPS>
cudaError_t run(const PackedArgs& a, cudaStream_t st) {
    const int64_t rows = a.total_q * a.heads, per = kThreads / 32 / WARPS;
    // Programmatic dependent launch: this kernel's CTAs are set up while the last
    // parts are computed.
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(static_cast<unsigned>((rows + per - 1) / per));
    c.blockDim = dim3(kThreads);
    c.stream = st;
    c.attrs = &early;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, packed_combine_kernel<D, FP16, WARPS>, a);
}

template <int D>
cudaError_t run(const PackedArgs& a, bool fp16, cudaStream_t st) {
    if (a.splits > 8) return fp16 ? run<D, true, 4>(a, st) : run<D, false, 4>(a, st);
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
