// Launchers of the prompt side's operators, shared between the C-ABI front end
// (h3a_api.cu) and the kernel translation units.  Not part of the public
// interface.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <atomic>
#include <cstddef>
#include <cstdint>

#include "h3a.h"

namespace h3a {

constexpr int kSms = 148;  // B200

// Lets `kernel` use `bytes` of dynamic shared memory, once per device and kernel
// (`done`: a bit for each device, of its own for each kernel).
cudaError_t allow_smem(const void* kernel, int bytes, std::atomic<uint64_t>& done);

// Programmatic dependent launch.  The prompt side's kernels are launched with
// launch_early and call early_start, or its two halves, before they touch global
// memory: their CTAs may then be set up while the stream's kernel before them
// still runs, and begin the moment it is complete and its writes are visible.
// They let the kernel after them do the same as soon as all their own CTAs have
// started; a kernel that allocates TMEM, when all its CTAs have theirs: columns
// that a CTA of the next launch took first would be held until this launch ends.
template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, const A&... args) {
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = grid;
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = smem;
    c.stream = st;
    c.attrs = &early;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, kernel, args...);
}
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void early_start() {
    let_next_start();
    wait_for_previous();
}

// One-dimensional rotary positions (rope.cu).  A side with heads == 0 is absent.
struct RopeSide {
    const void* x;
    void* y;
    int64_t sn, sh, on, oh;  // element strides of input and output
    int heads;
};
cudaError_t launch_rope(const RopeSide& q, const RopeSide& k, int head_dim, bool fp16, const int32_t* positions,
                        int64_t tokens, const h3a_rope_plan& plan, bool inverse, cudaStream_t st);

// Residual addition + RMS norm (rmsnorm.cu).
struct RmsNormArgs {
    const void* x;
    const void* f;  // null: no residual
    const float* gamma;
    void* h;
    void* y;
    float* scales;
    int64_t xs, fs, hs, ys;  // row strides, elements
    int64_t rows;
    int width;
    float eps;
};
constexpr int kRmsNormMaxWidth = 16384;
cudaError_t launch_residual_rmsnorm(const RmsNormArgs& a, bool fp16, h3a_scales scales, cudaStream_t st);

// Attention over packed sequences (packed_tiles.cu, packed_rows.cu, packed_combine.cu).
struct PackedArgs {
    const void *q, *k, *v;
    void* o;
    float* lse;  // [total_q, heads] or null
    const int32_t *starts_q, *starts_k, *lengths_k;
    int64_t qn, qh, kn, kh, vn, vh, on, oh;  // element strides
    int64_t total_q, total_k;
    int64_t max_q;           // queries of a sequence past this are left alone
    int seqs, heads, kv_heads, group;
    int causal;
    float scale_log2;  // logit scale * log2(e)
    // Parts of sequences' keys, joined by launch_packed_combine: normalised fp32
    // rows and their log-sum-exps (log2 units).
    // Tile kernel: parts of `chunk` keys (the last of `splits` takes what
    // remains), row (split * total_q + query) * heads + head.
    // Row kernel: `streams` stretches of all keys (0: a CTA takes whole sequences
    // and nothing is joined) have two parts each, 2 i of the sequence in which
    // stretch i begins and 2 i + 1 of the one in which it ends, kRowSlots rows for
    // every kv head; part_slots has each sequence's first and last part, or -1
    // when it needs no joining.
    int splits, chunk, streams;
    float* part_o;
    float* part_lse;
    int2* part_slots;
};
// What a sequence's entry of the index arrays means, cut to the tensors.
struct PackedSeq {
    int64_t q0, k0;
    int lq, lk;
};
__device__ __forceinline__ PackedSeq packed_seq(const PackedArgs& a, int s) {
    PackedSeq r;
    const int64_t tq = a.total_q, tk = a.total_k;
    const int64_t q0 = min(max(static_cast<int64_t>(__ldg(a.starts_q + s)), int64_t(0)), tq);
    const int64_t q1 = min(max(static_cast<int64_t>(__ldg(a.starts_q + s + 1)), q0), tq);
    const int64_t k0 = min(max(static_cast<int64_t>(__ldg(a.starts_k + s)), int64_t(0)), tk);
    const int64_t nk = a.lengths_k ? static_cast<int64_t>(__ldg(a.lengths_k + s))
                                   : static_cast<int64_t>(__ldg(a.starts_k + s + 1)) - k0;
    r.q0 = q0;
    r.k0 = k0;
    r.lq = static_cast<int>(q1 - q0);
    r.lk = static_cast<int>(min(max(nk, int64_t(0)), tk - k0));
    return r;
}
// Keys that query i of the sequence attends: the first `packed_limit` of it.
__device__ __forceinline__ int packed_limit(const PackedArgs& a, const PackedSeq& s, int i) {
    if (!a.causal) return s.lk;
    const int64_t n = static_cast<int64_t>(i) + 1 + s.lk - s.lq;
    return static_cast<int>(min(max(n, int64_t(0)), static_cast<int64_t>(s.lk)));
}

constexpr int kRowSlots = 16;  // rows of a part of the row kernel
// Where the row kernel's part is, in units of kRowSlots rows.
__device__ __forceinline__ int64_t packed_part_slot(const PackedArgs& a, int part, int kvh) {
    return static_cast<int64_t>(part) * a.kv_heads + kvh;
}

// How a call is carried out (packed_plan.cu).
struct PackedPlan {
    int tiles;  // 128-row tiles a CTA on tcgen05 (packed_tiles.cu): 1 or 2; 0: 16 rows (packed_rows.cu)
    int splits, chunk, streams;
};
PackedPlan packed_plan(const h3a_packed_desc& d);
// CTAs of the row kernel that a multiprocessor holds.
constexpr int packed_rows_ctas(int d) { return d == 64 ? 4 : 2; }
// Whether so few CTAs of whole sequences take eight warps each.
constexpr bool packed_rows_few(int d, int64_t ctas) { return ctas <= kSms * (d == 64 ? 2 : 1); }
// Queries in a 128-row tile, and the CTAs of `tiles` tiles that hold every sequence's.
int packed_queries_per_tile(int group);
int64_t packed_tile_groups(int64_t total_q, int seqs, int group, int tiles);

// At most kRowSlots rows (queries x group) of each sequence and kv head.
cudaError_t launch_packed_rows(const PackedArgs& a, int d, bool fp16, cudaStream_t st);
// Tensor maps: q as {d, group, kv_heads, total_q} with a {32, group, 1,
// packed_queries_per_tile} box, k and v as {d, kv_heads, total_k} with {32, 1,
// 128} boxes, 64-byte swizzle.
cudaError_t launch_packed_tiles(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const PackedArgs& p,
                                int d, bool fp16, int tiles, int* status, uint64_t timeout_ns, cudaStream_t st);
cudaError_t launch_packed_combine(const PackedArgs& a, int d, bool fp16, cudaStream_t st);

}  // namespace h3a
