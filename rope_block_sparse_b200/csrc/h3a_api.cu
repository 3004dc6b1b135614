// C-ABI front end of libh3a: argument validation, tensor-map encoding and
// launches on the caller's stream.  Nothing here allocates device memory; the
// only device state is the per-device status word below (and the copy of it
// that the last read took).
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>
#include <string>

#include "h3a.h"
#include "h3a_internal.h"
#include "prompt_internal.h"

// Sticky per-device status word: kernels OR error bits into it.
__device__ int g_h3a_status_word;
// What the last read of the status word took out of it.
__device__ int g_h3a_status_taken;

// Reads and clears the status word in one atomic step, so that an error a
// kernel on another stream ORs in at the same moment is either taken by this
// read or left for the next one -- never lost.
__global__ void status_take_kernel() { g_h3a_status_taken = atomicExch(&g_h3a_status_word, 0); }

namespace h3a {
namespace {

constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s per pipeline wait
constexpr int kMaxDevices = 64;

thread_local std::string g_last_cuda_error;

h3a_status cuda_fail(cudaError_t e) {
    g_last_cuda_error = std::string(cudaGetErrorName(e)) + ": " + cudaGetErrorString(e);
    return H3A_ERR_CUDA;
}

// Device address of g_h3a_status_word, resolved once per device.
std::mutex g_status_mu;
// Serialises readers of g_h3a_status_taken (one per process at a time).
std::mutex g_take_mu;
int* g_status_ptr[kMaxDevices] = {};

h3a_status status_word(int** out) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e);
    if (dev < 0 || dev >= kMaxDevices) return H3A_ERR_UNSUPPORTED;
    std::lock_guard<std::mutex> lock(g_status_mu);
    if (g_status_ptr[dev] == nullptr) {
        void* p = nullptr;
        e = cudaGetSymbolAddress(&p, g_h3a_status_word);
        if (e != cudaSuccess) return cuda_fail(e);
        g_status_ptr[dev] = static_cast<int*>(p);
    }
    *out = g_status_ptr[dev];
    return H3A_OK;
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
std::once_flag g_encode_once;
EncodeTiledFn g_encode = nullptr;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Validates a Q/K/V/O descriptor.  Fills `s` on success.  head_dim 96 for
// every call; the router and attention also take 128 (wide_ok).
h3a_status check_desc(const h3a_qkv_desc* d, Shape* s, bool wide_ok = false) {
    if (d == nullptr) return H3A_ERR_INVALID_ARG;
    if (d->head_dim != kHeadDim && !(wide_ok && d->head_dim == kHeadDimWide)) return H3A_ERR_UNSUPPORTED;
    if (d->B < 1 || d->N < 1 || d->heads < 1) return H3A_ERR_INVALID_ARG;
    if (d->stride_b < 0 || d->stride_n < 0 || d->stride_h < 0) return H3A_ERR_INVALID_ARG;
    if ((d->stride_b % 8) || (d->stride_n % 8) || (d->stride_h % 8)) return H3A_ERR_INVALID_ARG;
    if (d->heads > 1 && d->stride_h < d->head_dim) return H3A_ERR_INVALID_ARG;
    if (d->N > 1 && d->stride_n < d->head_dim) return H3A_ERR_INVALID_ARG;
    // byte strides must stay within the tensor-map limit (2^40)
    const int64_t lim = (int64_t(1) << 39);
    if (d->stride_b >= lim || d->stride_n >= lim || d->stride_h >= lim) return H3A_ERR_UNSUPPORTED;
    s->B = d->B;
    s->N = d->N;
    s->heads = d->heads;
    s->d = d->head_dim;
    s->sb = d->stride_b;
    s->sn = d->stride_n;
    s->sh = d->stride_h;
    return H3A_OK;
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Router workspace: the fp32 block means of Q, [B, heads, nblk, d], then those
// of K stored channel-major, [B, heads, d, pooled_k_stride(nblk)], each half
// starting on a 256-byte boundary.
size_t pooled_q_bytes(const Shape& s, int nblk) {
    return align256(static_cast<size_t>(s.B) * s.heads * nblk * s.d * sizeof(float));
}
size_t pooled_k_bytes(const Shape& s, int nblk) {
    return align256(static_cast<size_t>(s.B) * s.heads * s.d * pooled_k_stride(nblk) * sizeof(float));
}

}  // namespace

namespace {
// Tiled tensor map over a [B, N, heads, d] bf16 tensor (d contiguous) with the
// given box and swizzle; elements outside the tensor read as zero.
cudaError_t encode_qkv_map(CUtensorMap* map, const void* base, const Shape& s, const cuuint32_t (&box)[4],
                           CUtensorMapSwizzle swizzle) {
    std::call_once(g_encode_once, []() {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            g_encode = reinterpret_cast<EncodeTiledFn>(fn);
    });
    if (g_encode == nullptr) return cudaErrorNotSupported;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(s.d), static_cast<cuuint64_t>(s.heads),
                                static_cast<cuuint64_t>(s.N), static_cast<cuuint64_t>(s.B)};
    // byte strides of dims 1..3; a size-1 dim gets a nominal (unused) stride
    auto stride_or = [](int64_t st, int64_t fallback) { return static_cast<cuuint64_t>((st > 0 ? st : fallback) * 2); };
    const cuuint64_t strides[3] = {stride_or(s.sh, s.d), stride_or(s.sn, s.d), stride_or(s.sb, s.d)};
    const cuuint32_t elem_strides[4] = {1, 1, 1, 1};
    CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box,
                          elem_strides, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}
}  // namespace

cudaError_t make_qkv_tensor_map(CUtensorMap* map, const void* base, const Shape& s) {
    const cuuint32_t box[4] = {32, 1, 128, 1};
    return encode_qkv_map(map, base, s, box, CU_TENSOR_MAP_SWIZZLE_64B);
}

cudaError_t make_head_slice_tensor_map(CUtensorMap* map, const void* base, const Shape& s) {
    const cuuint32_t box[4] = {static_cast<cuuint32_t>(kHeadDim), static_cast<cuuint32_t>(kPrologueSliceHeads), 1, 1};
    return encode_qkv_map(map, base, s, box, CU_TENSOR_MAP_SWIZZLE_NONE);
}

// Tensor maps of the packed tile kernel (see launch_packed_tiles).  Without
// keys, k and v may be null: q stands in, and no step reads it.
static cudaError_t make_packed_tensor_maps(const h3a_packed_desc& d, const void* q, const void* k, const void* v,
                                           CUtensorMap* tq, CUtensorMap* tk, CUtensorMap* tv) {
    const int group = d.heads / d.kv_heads;
    // a dimension of size one is not stepped: any valid stride
    auto step = [&](int64_t stride, int64_t size) { return size > 1 ? stride : static_cast<int64_t>(d.head_dim); };
    const int64_t qh = step(d.q_stride_h, d.heads);
    const Shape sq{static_cast<int>(d.total_q), d.kv_heads, group, d.head_dim, step(d.q_stride_n, d.total_q), qh * group, qh};
    const cuuint32_t box[4] = {32, static_cast<cuuint32_t>(group), 1, static_cast<cuuint32_t>(packed_queries_per_tile(group))};
    cudaError_t e = encode_qkv_map(tq, q, sq, box, CU_TENSOR_MAP_SWIZZLE_64B);
    for (int i = 0; i < 2 && e == cudaSuccess; ++i) {
        const int64_t sn = step(i ? d.v_stride_n : d.k_stride_n, d.total_k), sh = step(i ? d.v_stride_h : d.k_stride_h, d.kv_heads);
        const int rows = d.total_k > 0 ? static_cast<int>(d.total_k) : 1;
        const Shape s{1, rows, d.total_k > 0 ? d.kv_heads : 1, d.head_dim, d.head_dim, sn, sh};
        e = make_qkv_tensor_map(i ? tv : tk, d.total_k > 0 ? (i ? v : k) : q, s);
    }
    return e;
}

}  // namespace h3a

using namespace h3a;

namespace {

// Shared checks of the router's shape, sparsity and workspace; on success
// fills nblk, k and the two pooled halves of the workspace.
h3a_status route_setup(const Shape& s, double sparsity, int32_t block, const void* workspace, size_t ws_bytes,
                       int* nblk, int64_t* kk, float** pq, float** pk) {
    if (block != kBlock) return H3A_ERR_UNSUPPORTED;
    if (!(sparsity >= 0.0 && sparsity < 1.0)) return H3A_ERR_INVALID_ARG;
    *nblk = (s.N + kBlock - 1) / kBlock;
    if (*nblk > route_max_blocks(s.d)) return H3A_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(s.B) * s.heads > 65535) return H3A_ERR_UNSUPPORTED;
    const size_t half = pooled_q_bytes(s, *nblk);
    if (workspace == nullptr || !aligned16(workspace) || ws_bytes < half + pooled_k_bytes(s, *nblk))
        return H3A_ERR_WORKSPACE;
    *kk = h3a_route_k(*nblk, sparsity);
    *pq = static_cast<float*>(const_cast<void*>(workspace));
    *pk = reinterpret_cast<float*>(static_cast<char*>(const_cast<void*>(workspace)) + half);
    return H3A_OK;
}

// Shared checks of the prologue's arguments.
h3a_status prologue_check(const void* q, const void* k, const h3a_qkv_desc* d, const float* gamma_q,
                          const float* gamma_k, h3a_grid grid, double theta, float eps, const void* q_out,
                          const void* k_out, Shape* s) {
    h3a_status rc = check_desc(d, s);
    if (rc != H3A_OK) return rc;
    if (!q || !k || !gamma_q || !gamma_k || !q_out || !k_out) return H3A_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(q_out) || !aligned16(k_out)) return H3A_ERR_INVALID_ARG;
    if (!(reinterpret_cast<uintptr_t>(gamma_q) % 4 == 0 && reinterpret_cast<uintptr_t>(gamma_k) % 4 == 0))
        return H3A_ERR_INVALID_ARG;
    if (grid.T < 1 || grid.H < 1 || grid.W < 1) return H3A_ERR_INVALID_ARG;
    if (static_cast<int64_t>(grid.T) * grid.H * grid.W != d->N) return H3A_ERR_INVALID_ARG;
    if (!(eps >= 0.0f) || !(theta > 0.0)) return H3A_ERR_INVALID_ARG;
    return H3A_OK;
}

bool known(h3a_dtype t) { return t == H3A_BF16 || t == H3A_FP16; }

// Strides of a [rows, heads, d] tensor: multiples of 8 elements that step over
// what lies inside them.  A dimension of size one is not stepped: any stride.
bool strides_ok(int64_t sn, int64_t sh, int64_t rows, int64_t heads, int64_t d) {
    return (heads <= 1 || (sh >= d && sh % 8 == 0)) && (rows <= 1 || (sn >= d && sn % 8 == 0));
}

h3a_status rope_plan_check(int32_t rotary_dim, const h3a_rope_plan* plan, double amplitude) {
    if (!plan || rotary_dim < 2 || rotary_dim % 2 || !std::isfinite(static_cast<float>(amplitude))) return H3A_ERR_INVALID_ARG;
    return rotary_dim > 2 * H3A_ROPE_MAX_PAIRS ? H3A_ERR_UNSUPPORTED : H3A_OK;
}

// Radians per position as a 64-bit fraction of a turn, modulo 1.
uint64_t turns_of(double frequency) {
    const double turns = frequency / 6.283185307179586476925;
    const double part = turns - std::floor(turns);  // exact: [0, 1]
    return static_cast<uint64_t>(std::fmod(std::ldexp(part, 64), 18446744073709551616.0));
}

// The logit scale in the kernels' log2 units.
float packed_scale_log2(const h3a_packed_desc& d) {
    const double scale = d.scale == 0.0f ? 1.0 / std::sqrt(static_cast<double>(d.head_dim)) : d.scale;
    return static_cast<float>(scale * 1.4426950408889634);
}

// Checks a packed descriptor and lays out its partial rows.
struct PackedRoom {
    size_t o, lse, all;  // bytes of the partial rows, up to their log-sum-exps' end, and of everything
};
h3a_status packed_check(const h3a_packed_desc* d, PackedPlan* plan, PackedRoom* room) {
    if (d == nullptr || !known(d->dtype)) return H3A_ERR_INVALID_ARG;
    if (d->seqs < 1 || d->heads < 1 || d->kv_heads < 1 || d->heads % d->kv_heads) return H3A_ERR_INVALID_ARG;
    if (d->total_q < 0 || d->total_k < 0 || d->max_q < 0 || d->max_k < 0) return H3A_ERR_INVALID_ARG;
    if (!(d->scale >= 0.0f) || (d->scale > 0.0f && !std::isfinite(packed_scale_log2(*d)))) return H3A_ERR_INVALID_ARG;
    if (d->head_dim != 64 && d->head_dim != 96 && d->head_dim != 128) return H3A_ERR_UNSUPPORTED;
    if (d->heads / d->kv_heads > 128) return H3A_ERR_UNSUPPORTED;
    const int64_t lim = int64_t(1) << 31;
    if (d->total_q >= lim || d->total_k >= lim) return H3A_ERR_UNSUPPORTED;
    // byte strides must stay within the tensor-map limit (2^40)
    for (int64_t s : {d->q_stride_n, d->q_stride_h * (d->heads / d->kv_heads), d->k_stride_n, d->k_stride_h, d->v_stride_n,
                      d->v_stride_h})
        if (s >= (int64_t(1) << 39)) return H3A_ERR_UNSUPPORTED;
    if (!strides_ok(d->q_stride_n, d->q_stride_h, d->total_q, d->heads, d->head_dim) ||
        !strides_ok(d->k_stride_n, d->k_stride_h, d->total_k, d->kv_heads, d->head_dim) ||
        !strides_ok(d->v_stride_n, d->v_stride_h, d->total_k, d->kv_heads, d->head_dim) ||
        !strides_ok(d->o_stride_n, d->o_stride_h, d->total_q, d->heads, d->head_dim))
        return H3A_ERR_INVALID_ARG;
    *plan = packed_plan(*d);
    const int group = d->heads / d->kv_heads;
    const double columns = plan->tiles ? static_cast<double>(packed_tile_groups(d->total_q, d->seqs, group, plan->tiles))
                                       : std::max(d->seqs, plan->streams);
    const double grid = columns * d->kv_heads;
    const double rows = static_cast<double>(d->total_q) * d->heads;
    if (grid >= static_cast<double>(lim) || rows >= static_cast<double>(lim)) return H3A_ERR_UNSUPPORTED;
    *room = PackedRoom{};
    if (plan->splits > 1 || plan->streams > 0) {
        const size_t parts = plan->streams > 0 ? static_cast<size_t>(plan->streams) * d->kv_heads * 2 * kRowSlots
                                               : static_cast<size_t>(plan->splits) * static_cast<size_t>(d->total_q) * d->heads;
        room->o = align256(parts * d->head_dim * sizeof(float));
        room->lse = room->o + align256(parts * sizeof(float));
        room->all = room->lse + (plan->streams > 0 ? align256(static_cast<size_t>(d->seqs) * sizeof(int2)) : 0);
    }
    return H3A_OK;
}

}  // namespace

extern "C" {

const char* h3a_status_string(h3a_status s) {
    switch (s) {
        case H3A_OK: return "H3A_OK";
        case H3A_ERR_INVALID_ARG: return "H3A_ERR_INVALID_ARG";
        case H3A_ERR_UNSUPPORTED: return "H3A_ERR_UNSUPPORTED";
        case H3A_ERR_CUDA: return "H3A_ERR_CUDA";
        case H3A_ERR_TIMEOUT: return "H3A_ERR_TIMEOUT";
        case H3A_ERR_WORKSPACE: return "H3A_ERR_WORKSPACE";
    }
    return "H3A_ERR_UNKNOWN";
}

const char* h3a_last_cuda_error_string(void) { return g_last_cuda_error.c_str(); }

h3a_status h3a_qk_norm_rope(const void* q, const void* k, const h3a_qkv_desc* d, const float* gamma_q,
                            const float* gamma_k, h3a_grid grid, double theta, float eps, void* q_out, void* k_out,
                            h3a_stream_t stream) {
    Shape s;
    h3a_status rc = prologue_check(q, k, d, gamma_q, gamma_k, grid, theta, eps, q_out, k_out, &s);
    if (rc != H3A_OK) return rc;
    cudaError_t e = launch_qk_norm_rope(q, k, q_out, k_out, gamma_q, gamma_k, s, grid.T, grid.H, grid.W, theta, eps,
                                        reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? H3A_OK : cuda_fail(e);
}

double h3a_step_sparsity(int32_t step, int32_t first_sparse_step, double sparsity) {
    if (step < 1 || first_sparse_step < 1 || !(sparsity >= 0.0 && sparsity < 1.0)) return -1.0;
    return step >= first_sparse_step ? sparsity : 0.0;
}

h3a_status h3a_qk_fullnorm_rope(const void* q, const void* k, const h3a_qkv_desc* d, const float* gamma_q,
                                const float* gamma_k, h3a_grid grid, double theta, float eps, void* q_out,
                                void* k_out, h3a_stream_t stream) {
    Shape s;
    h3a_status rc = prologue_check(q, k, d, gamma_q, gamma_k, grid, theta, eps, q_out, k_out, &s);
    if (rc != H3A_OK) return rc;
    if (!aligned16(gamma_q) || !aligned16(gamma_k)) return H3A_ERR_INVALID_ARG;  // read as float4
    // one CTA per token, each holding its token's rows in registers
    if (s.heads > 74 || static_cast<int64_t>(s.B) * s.N >= (int64_t(1) << 31)) return H3A_ERR_UNSUPPORTED;
    cudaError_t e = launch_qk_fullnorm_rope(q, k, q_out, k_out, gamma_q, gamma_k, s, grid.H, grid.W, theta, eps,
                                            reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? H3A_OK : cuda_fail(e);
}

int64_t h3a_route_k(int64_t nkv, double sparsity) {
    if (nkv < 1 || !(sparsity >= 0.0 && sparsity < 1.0)) return -1;
    int64_t kk = static_cast<int64_t>(std::ceil((1.0 - sparsity) * static_cast<double>(nkv) - 1e-9));
    if (kk < 1) kk = 1;
    if (kk > nkv) kk = nkv;
    return kk;
}

h3a_status h3a_route_workspace_size(const h3a_qkv_desc* d, int32_t block, size_t* bytes) {
    Shape s;
    h3a_status rc = check_desc(d, &s, true);
    if (rc != H3A_OK) return rc;
    if (bytes == nullptr) return H3A_ERR_INVALID_ARG;
    if (block != kBlock) return H3A_ERR_UNSUPPORTED;
    const int nblk = (s.N + kBlock - 1) / kBlock;
    *bytes = pooled_q_bytes(s, nblk) + pooled_k_bytes(s, nblk);
    return H3A_OK;
}

h3a_status h3a_route(const void* q, const void* k, const h3a_qkv_desc* d, double sparsity, int32_t block,
                     int32_t* block_idx, int64_t* k_out, void* workspace, size_t ws_bytes, h3a_stream_t stream) {
    Shape s;
    h3a_status rc = check_desc(d, &s, true);
    if (rc != H3A_OK) return rc;
    if (block != kBlock) return H3A_ERR_UNSUPPORTED;
    if (!q || !k || !block_idx) return H3A_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || (reinterpret_cast<uintptr_t>(block_idx) & 3u)) return H3A_ERR_INVALID_ARG;
    int nblk;
    int64_t kk;
    float *pq, *pk;
    rc = route_setup(s, sparsity, block, workspace, ws_bytes, &nblk, &kk, &pq, &pk);
    if (rc != H3A_OK) return rc;
    if (k_out) *k_out = kk;
    cudaError_t e = launch_route(q, k, s, nblk, static_cast<int>(kk), pq, pk, block_idx,
                                 reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? H3A_OK : cuda_fail(e);
}

h3a_status h3a_qk_norm_rope_pool(const void* q, const void* k, const h3a_qkv_desc* d, const float* gamma_q,
                                 const float* gamma_k, h3a_grid grid, double theta, float eps, void* q_out,
                                 void* k_out, void* workspace, size_t ws_bytes, h3a_stream_t stream) {
    Shape s;
    h3a_status rc = prologue_check(q, k, d, gamma_q, gamma_k, grid, theta, eps, q_out, k_out, &s);
    if (rc != H3A_OK) return rc;
    const int nblk = (s.N + kBlock - 1) / kBlock;
    if (s.B > 65535 || (s.heads + kPrologueSliceHeads - 1) / kPrologueSliceHeads > 65535) return H3A_ERR_UNSUPPORTED;
    const size_t half = pooled_q_bytes(s, nblk);
    if (workspace == nullptr || !aligned16(workspace) || ws_bytes < half + pooled_k_bytes(s, nblk))
        return H3A_ERR_WORKSPACE;
    float* pq = static_cast<float*>(workspace);
    float* pk = reinterpret_cast<float*>(static_cast<char*>(workspace) + half);
    int* status = nullptr;
    rc = status_word(&status);
    if (rc != H3A_OK) return rc;
    CUtensorMap tq, tk;
    cudaError_t e = make_head_slice_tensor_map(&tq, q, s);
    if (e == cudaSuccess) e = make_head_slice_tensor_map(&tk, k, s);
    if (e != cudaSuccess) return cuda_fail(e);
    e = launch_qk_norm_rope_pool(tq, tk, q_out, k_out, gamma_q, gamma_k, s, grid.H, grid.W, theta, eps, pq, pk,
                                 status, kWaitLimitNs, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? H3A_OK : cuda_fail(e);
}

h3a_status h3a_route_pooled(const h3a_qkv_desc* d, double sparsity, int32_t block, int32_t* block_idx,
                            int64_t* k_out, const void* workspace, size_t ws_bytes, h3a_stream_t stream) {
    Shape s;
    h3a_status rc = check_desc(d, &s);
    if (rc != H3A_OK) return rc;
    if (!block_idx || (reinterpret_cast<uintptr_t>(block_idx) & 3u)) return H3A_ERR_INVALID_ARG;
    int nblk;
    int64_t kk;
    float *pq, *pk;
    rc = route_setup(s, sparsity, block, workspace, ws_bytes, &nblk, &kk, &pq, &pk);
    if (rc != H3A_OK) return rc;
    if (k_out) *k_out = kk;
    cudaError_t e = launch_route_scores(pq, pk, s, nblk, static_cast<int>(kk), block_idx,
                                        reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? H3A_OK : cuda_fail(e);
}

h3a_status h3a_attention(const void* q, const void* k, const void* v, const h3a_qkv_desc* d,
                         const int32_t* block_idx, int32_t k_blocks, int32_t block, float scale, void* o,
                         h3a_stream_t stream) {
    Shape s;
    h3a_status rc = check_desc(d, &s, true);
    if (rc != H3A_OK) return rc;
    if (block != kBlock) return H3A_ERR_UNSUPPORTED;
    if (!q || !k || !v || !o) return H3A_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return H3A_ERR_INVALID_ARG;
    if (!(scale >= 0.0f) || !std::isfinite(scale)) return H3A_ERR_INVALID_ARG;
    const int nblk = (s.N + kBlock - 1) / kBlock;
    if (block_idx != nullptr) {
        if ((reinterpret_cast<uintptr_t>(block_idx) & 3u) || k_blocks < 1 || k_blocks > nblk)
            return H3A_ERR_INVALID_ARG;
    }
    const int64_t grid = static_cast<int64_t>(s.B) * s.heads * ((nblk + 1) / 2);
    if (grid >= (int64_t(1) << 31)) return H3A_ERR_UNSUPPORTED;
    if (scale == 0.0f) scale = static_cast<float>(1.0 / std::sqrt(static_cast<double>(s.d)));
    int* status = nullptr;
    rc = status_word(&status);
    if (rc != H3A_OK) return rc;
    CUtensorMap tq, tk, tv;
    cudaError_t e = make_qkv_tensor_map(&tq, q, s);
    if (e == cudaSuccess) e = make_qkv_tensor_map(&tk, k, s);
    if (e == cudaSuccess) e = make_qkv_tensor_map(&tv, v, s);
    if (e != cudaSuccess) return cuda_fail(e);
    e = launch_attention(tq, tk, tv, o, s, block_idx, k_blocks, scale, status, kWaitLimitNs,
                         reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? H3A_OK : cuda_fail(e);
}

h3a_status h3a_residual_adaln(const void* x, const void* f, const float* gate, const float* shift,
                              const float* scale, int32_t B, int64_t rows, int32_t width, float eps, void* h_out,
                              void* y_out, h3a_stream_t stream) {
    if (B < 1 || rows < 0 || width < 8) return H3A_ERR_INVALID_ARG;
    if (width % 8) return H3A_ERR_INVALID_ARG;
    if (width > residual_adaln_max_width()) return H3A_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(B) * rows >= (int64_t(1) << 31)) return H3A_ERR_UNSUPPORTED;
    if (!x || !shift || !scale || !y_out) return H3A_ERR_INVALID_ARG;
    if (f && (!gate || !h_out)) return H3A_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(shift) || !aligned16(scale) || !aligned16(y_out)) return H3A_ERR_INVALID_ARG;
    if ((f && !aligned16(f)) || (gate && !aligned16(gate)) || (h_out && !aligned16(h_out)))
        return H3A_ERR_INVALID_ARG;
    if (!(eps >= 0.0f)) return H3A_ERR_INVALID_ARG;
    cudaError_t e = launch_residual_adaln(x, f, f ? gate : nullptr, shift, scale, B, rows, width, eps,
                                          f ? h_out : nullptr, y_out, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? H3A_OK : cuda_fail(e);
}

h3a_status h3a_swiglu(const void* in, int64_t rows, int32_t ffn_width, void* out, h3a_stream_t stream) {
    if (rows < 0 || ffn_width < 8 || (ffn_width % 8)) return H3A_ERR_INVALID_ARG;
    if (!in || !out || !aligned16(in) || !aligned16(out)) return H3A_ERR_INVALID_ARG;
    cudaError_t e = launch_swiglu(in, rows, ffn_width, out, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? H3A_OK : cuda_fail(e);
}

h3a_status h3a_residual_diff(const void* cur, const void* prev, int64_t n, double threshold, void* workspace,
                             size_t ws_bytes, double* rel_out, int32_t* reuse_out, h3a_stream_t stream) {
    if (n < 8 || (n % 8)) return H3A_ERR_INVALID_ARG;
    if (!cur || !prev || !rel_out || !aligned16(cur) || !aligned16(prev)) return H3A_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(rel_out) & 7u) || (reinterpret_cast<uintptr_t>(reuse_out) & 3u))
        return H3A_ERR_INVALID_ARG;
    if (!(threshold >= 0.0)) return H3A_ERR_INVALID_ARG;
    if (workspace == nullptr || !aligned16(workspace) || ws_bytes < residual_diff_workspace_bytes())
        return H3A_ERR_WORKSPACE;
    cudaError_t e = launch_residual_diff(cur, prev, n, threshold, workspace, rel_out, reuse_out,
                                         reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? H3A_OK : cuda_fail(e);
}

h3a_status h3a_rope_plan_from(int32_t rotary_dim, int32_t interleaved, const double* frequencies, double amplitude,
                              h3a_rope_plan* plan) {
    const h3a_status rc = rope_plan_check(rotary_dim, plan, amplitude);
    if (rc != H3A_OK) return rc;
    if (!frequencies) return H3A_ERR_INVALID_ARG;
    for (int j = 0; j < rotary_dim / 2; ++j)
        if (!std::isfinite(frequencies[j])) return H3A_ERR_INVALID_ARG;
    std::memset(plan, 0, sizeof(*plan));
    plan->pairs = rotary_dim / 2;
    plan->interleaved = interleaved ? 1 : 0;
    plan->amplitude = static_cast<float>(amplitude);
    for (int j = 0; j < plan->pairs; ++j) plan->turns[j] = turns_of(frequencies[j]);
    return H3A_OK;
}

h3a_status h3a_rope_plan_scaled(int32_t rotary_dim, int32_t interleaved, double theta, h3a_rope_scaling scaling,
                                double factor, int64_t original_length, double low_turns, double high_turns,
                                double amplitude, h3a_rope_plan* plan) {
    const h3a_status rc = rope_plan_check(rotary_dim, plan, amplitude);
    if (rc != H3A_OK) return rc;
    if (!(theta > 0.0) || !std::isfinite(theta) || !(factor > 0.0) || !std::isfinite(factor))
        return H3A_ERR_INVALID_ARG;
    if (scaling < H3A_ROPE_PLAIN || scaling > H3A_ROPE_PARTS) return H3A_ERR_INVALID_ARG;
    if (scaling == H3A_ROPE_PARTS &&
        (original_length < 1 || !std::isfinite(low_turns) || !std::isfinite(high_turns) || !(high_turns > low_turns)))
        return H3A_ERR_INVALID_ARG;
    const double r = rotary_dim;
    if (scaling == H3A_ROPE_BASE && rotary_dim > 2) theta *= std::pow(factor, r / (r - 2.0));
    if (!std::isfinite(theta)) return H3A_ERR_INVALID_ARG;
    double f[H3A_ROPE_MAX_PAIRS];
    for (int j = 0; j < rotary_dim / 2; ++j) {
        f[j] = std::pow(theta, -2.0 * j / r);
        if (scaling == H3A_ROPE_LINEAR) f[j] /= factor;
        if (scaling == H3A_ROPE_PARTS) {
            const double n = static_cast<double>(original_length) * f[j] / 6.283185307179586476925;
            const double w = std::fmin(std::fmax((n - low_turns) / (high_turns - low_turns), 0.0), 1.0);
            f[j] *= w + (1.0 - w) / factor;
        }
    }
    return h3a_rope_plan_from(rotary_dim, interleaved, f, amplitude, plan);
}

h3a_status h3a_rope(const void* q, void* q_out, const h3a_heads_desc* dq, const void* k, void* k_out,
                    const h3a_heads_desc* dk, h3a_dtype dtype, const int32_t* positions, int64_t tokens,
                    const h3a_rope_plan* plan, int32_t inverse, h3a_stream_t stream) {
    if (!dq || !plan || !known(dtype) || tokens < 0 || (k && !dk)) return H3A_ERR_INVALID_ARG;
    if (plan->pairs < 1 || plan->pairs > H3A_ROPE_MAX_PAIRS) return H3A_ERR_INVALID_ARG;
    const int sides = k ? 2 : 1;
    int64_t heads = 0;
    RopeSide side[2] = {};
    for (int i = 0; i < sides; ++i) {
        const h3a_heads_desc& d = i ? *dk : *dq;
        const void* x = i ? k : q;
        void* y = i ? k_out : q_out;
        if (d.heads < 1 || d.head_dim < 2 * plan->pairs || d.head_dim % 8 || d.head_dim != dq->head_dim)
            return H3A_ERR_INVALID_ARG;
        if (!strides_ok(d.stride_n, d.stride_h, tokens, d.heads, d.head_dim) ||
            !strides_ok(d.out_stride_n, d.out_stride_h, tokens, d.heads, d.head_dim))
            return H3A_ERR_INVALID_ARG;
        if (tokens > 0 && (!x || !y)) return H3A_ERR_INVALID_ARG;
        if (!aligned16(x) || !aligned16(y)) return H3A_ERR_INVALID_ARG;
        if (x == y && (d.stride_n != d.out_stride_n || d.stride_h != d.out_stride_h)) return H3A_ERR_INVALID_ARG;
        side[i] = RopeSide{x, y, d.stride_n, d.stride_h, d.out_stride_n, d.out_stride_h, d.heads};
        heads += d.heads;
    }
    if (dq->head_dim > 512 || tokens >= (int64_t(1) << 31) || heads > 32768) return H3A_ERR_UNSUPPORTED;
    if (tokens == 0) return H3A_OK;
    if (!positions || (reinterpret_cast<uintptr_t>(positions) & 3u)) return H3A_ERR_INVALID_ARG;
    cudaError_t e = launch_rope(side[0], side[1], dq->head_dim, dtype == H3A_FP16, positions, tokens, *plan, inverse != 0,
                                reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? H3A_OK : cuda_fail(e);
}

h3a_status h3a_residual_rmsnorm(const void* x, int64_t x_stride, const void* f, int64_t f_stride, const float* gamma,
                                int64_t rows, int32_t width, h3a_dtype dtype, float eps, h3a_scales scales,
                                void* h_out, int64_t h_stride, void* y_out, int64_t y_stride, float* scales_out,
                                h3a_stream_t stream) {
    if (rows < 0 || width < 8 || width % 8 || !known(dtype) || !(eps >= 0.0f)) return H3A_ERR_INVALID_ARG;
    if (scales < H3A_SCALES_NONE || scales > H3A_SCALES_GROUP) return H3A_ERR_INVALID_ARG;
    auto stride_ok = [&](int64_t s) { return s % 8 == 0 && s >= width; };
    if (!stride_ok(x_stride) || !stride_ok(y_stride) || (f && (!stride_ok(f_stride) || !stride_ok(h_stride))))
        return H3A_ERR_INVALID_ARG;
    if (width > kRmsNormMaxWidth || rows >= (int64_t(1) << 31)) return H3A_ERR_UNSUPPORTED;
    if (rows == 0) return H3A_OK;
    if (!x || !gamma || !y_out || (f && !h_out)) return H3A_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(gamma) || !aligned16(y_out) || (f && (!aligned16(f) || !aligned16(h_out))))
        return H3A_ERR_INVALID_ARG;
    if (f && ((h_out == x && h_stride != x_stride) || (h_out == f && h_stride != f_stride))) return H3A_ERR_INVALID_ARG;
    if (scales != H3A_SCALES_NONE && (!scales_out || (reinterpret_cast<uintptr_t>(scales_out) & 3u)))
        return H3A_ERR_INVALID_ARG;
    const RmsNormArgs a{x, f, gamma, f ? h_out : nullptr, y_out, scales_out, x_stride, f_stride, h_stride, y_stride, rows, width, eps};
    cudaError_t e = launch_residual_rmsnorm(a, dtype == H3A_FP16, scales, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? H3A_OK : cuda_fail(e);
}

h3a_status h3a_packed_attention_workspace_size(const h3a_packed_desc* d, size_t* bytes) {
    PackedPlan plan;
    PackedRoom room;
    const h3a_status rc = packed_check(d, &plan, &room);
    if (rc != H3A_OK) return rc;
    if (bytes == nullptr) return H3A_ERR_INVALID_ARG;
    *bytes = room.all;
    return H3A_OK;
}

h3a_status h3a_packed_attention(const void* q, const void* k, const void* v, const h3a_packed_desc* d,
                                const int32_t* starts_q, const int32_t* starts_k, const int32_t* lengths_k, void* o,
                                float* lse, void* workspace, size_t ws_bytes, h3a_stream_t stream) {
    PackedPlan plan;
    PackedRoom room;
    h3a_status rc = packed_check(d, &plan, &room);
    if (rc != H3A_OK) return rc;
    if (d->total_q == 0 || d->max_q == 0) return H3A_OK;  // no query, nothing to write
    if (!q || !o || (d->total_k > 0 && (!k || !v)) || !starts_q || !starts_k) return H3A_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return H3A_ERR_INVALID_ARG;
    for (const void* p : {static_cast<const void*>(starts_q), static_cast<const void*>(starts_k),
                          static_cast<const void*>(lengths_k), static_cast<const void*>(lse)})
        if (reinterpret_cast<uintptr_t>(p) & 3u) return H3A_ERR_INVALID_ARG;
    if (room.all > 0 && (!workspace || !aligned16(workspace) || ws_bytes < room.all)) return H3A_ERR_WORKSPACE;
    PackedArgs a{};
    a.q = q, a.k = k, a.v = v, a.o = o, a.lse = lse;
    a.starts_q = starts_q, a.starts_k = starts_k, a.lengths_k = lengths_k;
    a.qn = d->q_stride_n, a.qh = d->q_stride_h, a.kn = d->k_stride_n, a.kh = d->k_stride_h;
    a.vn = d->v_stride_n, a.vh = d->v_stride_h, a.on = d->o_stride_n, a.oh = d->o_stride_h;
    a.total_q = d->total_q, a.total_k = d->total_k, a.max_q = d->max_q;
    a.seqs = d->seqs, a.heads = d->heads, a.kv_heads = d->kv_heads, a.group = d->heads / d->kv_heads;
    a.causal = d->causal != 0;
    a.scale_log2 = packed_scale_log2(*d);
    a.splits = plan.splits, a.chunk = plan.chunk, a.streams = plan.streams;
    if (room.all > 0) {
        a.part_o = static_cast<float*>(workspace);
        a.part_lse = reinterpret_cast<float*>(static_cast<char*>(workspace) + room.o);
        a.part_slots = reinterpret_cast<int2*>(static_cast<char*>(workspace) + room.lse);
    }
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (plan.tiles) {
        int* status = nullptr;
        rc = status_word(&status);
        if (rc != H3A_OK) return rc;
        CUtensorMap tq, tk, tv;
        e = make_packed_tensor_maps(*d, q, k, v, &tq, &tk, &tv);
        if (e == cudaSuccess)
            e = launch_packed_tiles(tq, tk, tv, a, d->head_dim, d->dtype == H3A_FP16, plan.tiles, status, kWaitLimitNs, st);
    } else {
        e = launch_packed_rows(a, d->head_dim, d->dtype == H3A_FP16, st);
    }
    if (e == cudaSuccess && room.all > 0) e = launch_packed_combine(a, d->head_dim, d->dtype == H3A_FP16, st);
    return e == cudaSuccess ? H3A_OK : cuda_fail(e);
}

h3a_status h3a_last_device_error(h3a_stream_t stream) {
    int* status = nullptr;
    h3a_status rc = status_word(&status);
    if (rc != H3A_OK) return rc;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    std::lock_guard<std::mutex> lock(g_take_mu);
    // after everything already queued on `stream`: take the word, then copy it out
    status_take_kernel<<<1, 1, 0, st>>>();
    cudaError_t e = cudaGetLastError();
    int word = 0;
    if (e == cudaSuccess) e = cudaMemcpyFromSymbolAsync(&word, g_h3a_status_taken, sizeof(int), 0,
                                                        cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    if (e != cudaSuccess) return cuda_fail(e);
    return (word & kDevTimeout) ? H3A_ERR_TIMEOUT : H3A_OK;
}

h3a_status h3a_selftest_wait_timeout(uint32_t limit_us, h3a_stream_t stream) {
    int* status = nullptr;
    h3a_status rc = status_word(&status);
    if (rc != H3A_OK) return rc;
    rc = h3a_last_device_error(stream);  // start from a clear word
    if (rc == H3A_ERR_CUDA) return rc;
    cudaError_t e = launch_selftest_wait(static_cast<uint64_t>(limit_us) * 1000ull, status,
                                         reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e);
    return h3a_last_device_error(stream);
}

h3a_status h3a_selftest_mma(const void* a, const void* b, float* s_out, float* r_out, h3a_stream_t stream) {
    if (!a || !b || !s_out || !r_out) return H3A_ERR_INVALID_ARG;
    if (!aligned16(a) || !aligned16(b) || !aligned16(s_out) || !aligned16(r_out)) return H3A_ERR_INVALID_ARG;
    int* status = nullptr;
    h3a_status rc = status_word(&status);
    if (rc != H3A_OK) return rc;
    Shape s{1, 128, 1, kHeadDim, 128 * kHeadDim, kHeadDim, kHeadDim};
    CUtensorMap ta, tb;
    cudaError_t e = make_qkv_tensor_map(&ta, a, s);
    if (e == cudaSuccess) e = make_qkv_tensor_map(&tb, b, s);
    if (e != cudaSuccess) return cuda_fail(e);
    e = launch_selftest_mma(ta, tb, s_out, r_out, status, kWaitLimitNs, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? H3A_OK : cuda_fail(e);
}

h3a_status h3a_selftest_exp2(const float* x, float* y, int32_t n, h3a_stream_t stream) {
    if (n < 0 || (n > 0 && (!x || !y))) return H3A_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(x) & 3u) || (reinterpret_cast<uintptr_t>(y) & 3u)) return H3A_ERR_INVALID_ARG;
    cudaError_t e = launch_selftest_exp2(x, y, n, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? H3A_OK : cuda_fail(e);
}

}  // extern "C"
