// Attention over packed sequences, few query rows at a time: single tokens
// over caches (h3a_packed_attention; the tile kernel in packed_tiles.cu takes
// calls with more rows).
//
// The queries that share a kv head are the rows of one matrix: row r of a
// sequence is query r / group, head r % group of the kv head's group, at most
// 16 (the M of mma.m16n8k16).  A CTA's warps take units of 16 keys in turn, each
// with a cp.async pipeline of its own through shared memory, so no barrier
// stands between load and use:
//   S = Q K^T (Q in registers), online softmax in fp32 (log2 domain, running
//   row maximum m and sum l), O = alpha O + P V with P rounded to the element
//   type straight from S's registers.
// At the end the warps' (m, l, O) are joined through shared memory.  HBM-bound:
// K and V are read once; one unit is 16 keys x (K + V) = 8 KB at head_dim 128.
//
// Work: blocks of 64 keys of all sequences, one behind the other.  Short
// sequences get a CTA each (and kv head).  Long or few ones are streamed: the
// blocks are cut into equal stretches, whatever sequences they run through, as
// many as make the GPU's CTAs with one for each kv head, so that neither a long
// sequence nor a short batch leaves part of the GPU idle; a sequence that lies
// in one stretch is finished there, the others' parts go to the workspace and
// are joined by packed_combine.cu.  The kv heads of a stretch run side by side:
// their rows of a key lie behind one another in memory, and apart in time they
// are 256 bytes here and there (16,000 keys of 8 kv heads x 128 by stretches of
// single heads: 20.5 us, side by side 16).  Measured, with the joining: 47 caches of
// up to 16,384 keys, 32/8 heads x 128, 1.11 GB: 176 to 188 us, 5.9 to 6.3 TB/s = 0.90
// to 0.96 of a copy; 8 of up to 900, 16 heads x 64: 7.6 to 8.4 us, of which HBM takes 1.3 and
// a launch 1.6 to 2.0; what the others go to is not known (more units on their way did not
// shorten it).
//
// Keys no row attends are read as zeros (cp.async with a source size of 0), so
// what lies behind a sequence is never touched.  Where some rows attend a key
// and others do not (causal, several queries), an infinity or NaN in V would
// reach the others as 0 * NaN: such a unit's V fragments have their non-finite
// values set to zero, and the end adds those back to exactly the rows that
// attend them.
#include "half16.cuh"
#include "prompt_internal.h"

namespace h3a {
namespace {

constexpr int kWarps = 4;    // of a streamed CTA
constexpr int kUnit = 16;    // keys a warp takes at a time
// One unit on its way while one is in work: 2 CTAs x 4 warps x 8 KB = 64 KB a
// multiprocessor cover the latency, and more requests at a time only disturb one
// another (47 caches of up to 16,384 keys: 183 us; with two units on their way 198,
// with three 203).
constexpr int kStages = 2;

// A CTA of W warps.
template <int D, int W>
struct Geo {
    static constexpr int kPitch = D * 2 + 16;  // an odd multiple of 16 bytes: ldmatrix rows hit distinct banks
    static constexpr int kTile = kUnit * kPitch;
    static constexpr int kChunks = D / 8;      // 16-byte chunks of a key
    static constexpr int kStageBytes = 2 * kTile;
    static constexpr int kPipeBytes = W * kStages * kStageBytes;
    static constexpr int kJoinPitch = D + 4;
    static constexpr int kJoinBytes = (W * 16 * kJoinPitch + W * 16 * 2) * 4;
    static constexpr int kSmem = kPipeBytes > kJoinBytes ? kPipeBytes : kJoinBytes;
    static_assert(D % 16 == 0 && (kUnit * kChunks) % 32 == 0, "head_dim");
};

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// 16 bytes global -> shared; zeros when `bytes` is 0 (nothing is read then)
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
template <bool FP16>
__device__ __forceinline__ void mma_16x8x16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (FP16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

constexpr int kBlockKeys = kUnit * kWarps;  // 64: what the work is counted in

// Queries of the sequence that count, and blocks of its keys that any of them attends.
__device__ __forceinline__ int counted_queries(const PackedArgs& a, const PackedSeq& s) {
    return static_cast<int>(min(static_cast<int64_t>(s.lq), a.max_q));
}
__device__ __forceinline__ int key_blocks(const PackedArgs& a, const PackedSeq& s) {
    const int queries = counted_queries(a, s);
    return queries == 0 ? 0 : (packed_limit(a, s, queries - 1) + kBlockKeys - 1) / kBlockKeys;
}

// Keys [begin, end) of one (sequence, kv head), and where the result goes.
struct Segment {
    int kvh, begin, end;
    int64_t slot;  // part's slot, or -1: the end result
};

// found[2]: a warp cleared a value of V, in turns (0 at the first call) so that one
// is set back while nobody uses it.
template <int D, bool FP16, int W>
__device__ __forceinline__ void attend(const PackedArgs& a, const PackedSeq& s, const Segment& g, uint8_t* smem, int* found, int turn) {
    using G = Geo<D, W>;
    using H = Half16<FP16>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int queries = counted_queries(a, s);
    const int rows = queries * a.group;  // at most 16
    const int least = packed_limit(a, s, 0);
    const int begin = g.begin, end = g.end, kvh = g.kvh;

    // Q: rows lane / 4 and lane / 4 + 8 of the A fragments
    const int ra = lane >> 2;
    int limit[2];
    uint32_t qf[D / 16][4];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int r = ra + 8 * e;
        const bool in = r < rows;
        const int query = in ? r / a.group : 0, head = in ? r % a.group : 0;
        limit[e] = in ? packed_limit(a, s, query) : 0;
        const uint16_t* p = static_cast<const uint16_t*>(a.q) + (s.q0 + query) * a.qn + (static_cast<int64_t>(kvh) * a.group + head) * a.qh;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            const int c = ks * 16 + 2 * (lane & 3);
            qf[ks][e] = in ? *reinterpret_cast<const uint32_t*>(p + c) : 0u;
            qf[ks][e + 2] = in ? *reinterpret_cast<const uint32_t*>(p + c + 8) : 0u;
        }
    }

    const uint32_t pipe = smem_addr(smem) + warp * (kStages * G::kStageBytes);
    const uint16_t* kbase = static_cast<const uint16_t*>(a.k) + s.k0 * a.kn + kvh * a.kh;
    const uint16_t* vbase = static_cast<const uint16_t*>(a.v) + s.k0 * a.vn + kvh * a.vh;
    auto load = [&](int key0, int stage) {
        if (key0 < end) {
            const uint32_t dk = pipe + stage * G::kStageBytes;
#pragma unroll
            for (int it = 0; it < kUnit * G::kChunks / 32; ++it) {
                const int i = it * 32 + lane, row = i / G::kChunks, c = i % G::kChunks;
                const int key = key0 + row;
                const bool in = key < end;
                const int64_t kk = in ? key : 0;
                const uint32_t off = row * G::kPitch + c * 16;
                cp_async16(dk + off, kbase + kk * a.kn + c * 8, in ? 16u : 0u);
                cp_async16(dk + G::kTile + off, vbase + kk * a.vn + c * 8, in ? 16u : 0u);
            }
        }
        cp_async_commit();  // an empty group keeps the count
    };

    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    bool nonfinite = false;
    constexpr int kStride = kUnit * W;
    int next = begin + warp * kUnit;
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i, next += kStride) load(next, i);
    int stage = 0;
    for (int key0 = begin + warp * kUnit; key0 < end; key0 += kStride, next += kStride) {
        cp_async_wait<kStages - 2>();
        __syncwarp();
        load(next, stage == 0 ? kStages - 1 : stage - 1);
        const uint32_t kt = pipe + stage * G::kStageBytes, vt = kt + G::kTile;
        // S = Q K^T: n-tiles of keys 0-7 and 8-15
        float c[2][4] = {};
        const int mi = lane >> 3, mr = lane & 7;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            uint32_t b[4];
            ldmatrix_x4(kt + ((mi >> 1) * 8 + mr) * G::kPitch + ks * 32 + (mi & 1) * 16, b);
            mma_16x8x16<FP16>(c[0], qf[ks], b[0], b[1]);
            mma_16x8x16<FP16>(c[1], qf[ks], b[2], b[3]);
        }
        const bool partly = key0 + kUnit > least;  // some row does not attend some key of the unit
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                c[t][e] *= a.scale_log2;
                if (partly && key0 + t * 8 + 2 * (lane & 3) + (e & 1) >= min(limit[e >> 1], end)) c[t][e] = -INFINITY;
                mx[e >> 1] = fmaxf(mx[e >> 1], c[t][e]);
            }
        float alpha[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
            mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
            mx[e] = fmaxf(mx[e], m[e]);
            const float ref = mx[e] == -INFINITY ? 0.f : mx[e];  // no key yet: every weight is exp2(-inf) = 0
            alpha[e] = exp2_fast(m[e] - ref);
            m[e] = mx[e];
            l[e] *= alpha[e];
            mx[e] = ref;
        }
        uint32_t p[4];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                c[t][e] = exp2_fast(c[t][e] - mx[e >> 1]);
                l[e >> 1] += c[t][e];
            }
            p[2 * t] = H::pack(c[t][0], c[t][1]);
            p[2 * t + 1] = H::pack(c[t][2], c[t][3]);
        }
        if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                o[i][0] *= alpha[0], o[i][1] *= alpha[0];
                o[i][2] *= alpha[1], o[i][3] *= alpha[1];
            }
        }
#pragma unroll
        for (int dt = 0; dt < D / 16; ++dt) {
            uint32_t b[4];
            ldmatrix_x4_trans(vt + ((mi & 1) * 8 + mr) * G::kPitch + dt * 32 + (mi >> 1) * 16, b);
            if (partly) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t bad = nonfinite_halves<FP16>(b[i]);
                    nonfinite |= bad != 0;
                    b[i] = finite_or_zero<FP16>(b[i], bad);
                }
            }
            mma_16x8x16<FP16>(o[2 * dt], p, b[0], b[1]);
            mma_16x8x16<FP16>(o[2 * dt + 1], p, b[2], b[3]);
        }
        stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    cp_async_wait<0>();
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
    }
    if (nonfinite) found[turn] = 1;
    __syncthreads();  // every warp is done with its pipeline: the join reuses it
    if (threadIdx.x == 0) found[turn ^ 1] = 0;
    float* jo = reinterpret_cast<float*>(smem);
    float* jm = jo + W * 16 * G::kJoinPitch;
    float* jl = jm + W * 16;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
        float* d = jo + (warp * 16 + ra) * G::kJoinPitch + i * 8 + 2 * (lane & 3);
        *reinterpret_cast<float2*>(d) = make_float2(o[i][0], o[i][1]);
        *reinterpret_cast<float2*>(d + 8 * G::kJoinPitch) = make_float2(o[i][2], o[i][3]);
    }
    if ((lane & 3) == 0) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            jm[warp * 16 + ra + 8 * e] = m[e];
            jl[warp * 16 + ra + 8 * e] = l[e];
        }
    }
    __syncthreads();
    // 2 W threads a row, every 2 W-th group of four channels each
    constexpr int kTeam = 2 * W;
    const int row = threadIdx.x / kTeam;
    if (row < rows) {
        const int query = row / a.group;
        const int64_t n = s.q0 + query;
        const int head = kvh * a.group + row % a.group;
        float top = -INFINITY, w[W], sum = 0.f;
    #pragma unroll
        for (int i = 0; i < W; ++i) top = fmaxf(top, jm[i * 16 + row]);
        const float ref = top == -INFINITY ? 0.f : top;
    #pragma unroll
        for (int i = 0; i < W; ++i) {
            w[i] = exp2_fast(jm[i * 16 + row] - ref);
            sum += w[i] * jl[i * 16 + row];
        }
        const float inv = sum == 0.f ? 0.f : 1.0f / sum;
        const float lse2 = sum == 0.f ? -INFINITY : ref + log2f(sum);
        const int64_t qh = n * a.heads + head;
        const int limit_row = min(packed_limit(a, s, query), end);
        for (int c = (threadIdx.x % kTeam) * 4; c < D; c += 4 * kTeam) {
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    #pragma unroll
            for (int i = 0; i < W; ++i) {
                const float4 v = *reinterpret_cast<const float4*>(jo + (i * 16 + row) * G::kJoinPitch + c);
                acc.x = fmaf(w[i], v.x, acc.x), acc.y = fmaf(w[i], v.y, acc.y);
                acc.z = fmaf(w[i], v.z, acc.z), acc.w = fmaf(w[i], v.w, acc.w);
            }
            acc.x *= inv, acc.y *= inv, acc.z *= inv, acc.w *= inv;
            if (found[turn]) {
                // the units whose V was cleared: from the first key some row does not attend
                const int from = max(begin, begin + (least - begin) / kUnit * kUnit);
                for (int key = from; key < limit_row; ++key) {
                    const uint2 raw = *reinterpret_cast<const uint2*>(vbase + static_cast<int64_t>(key) * a.vn + c);
                    float x[4];
                    H::unpack(raw.x, x[0], x[1]);
                    H::unpack(raw.y, x[2], x[3]);
                    acc.x += isfinite(x[0]) ? 0.f : x[0], acc.y += isfinite(x[1]) ? 0.f : x[1];
                    acc.z += isfinite(x[2]) ? 0.f : x[2], acc.w += isfinite(x[3]) ? 0.f : x[3];
                }
            }
            if (g.slot >= 0) {
                *reinterpret_cast<float4*>(a.part_o + (g.slot * kRowSlots + row) * D + c) = acc;
            } else {
                uint16_t* dst = static_cast<uint16_t*>(a.o) + n * a.on + head * a.oh + c;
                *reinterpret_cast<uint2*>(dst) = make_uint2(H::pack(acc.x, acc.y), H::pack(acc.z, acc.w));
            }
        }
        if (threadIdx.x % kTeam == 0) {
            if (g.slot >= 0)
                a.part_lse[g.slot * kRowSlots + row] = lse2;
            else if (a.lse)
                a.lse[qh] = lse2 * 0.6931471805599453f;
        }
    }
    __syncthreads();  // the next segment reuses the shared memory
}

// A CTA a (sequence, kv head).
template <int D, bool FP16, int W>
__global__ void __launch_bounds__(32 * W, W == kWarps ? packed_rows_ctas(D) : 1) packed_rows_kernel(const __grid_constant__ PackedArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int found[2];
    if (threadIdx.x == 0) found[0] = found[1] = 0;
    early_start();
    __syncthreads();
    const PackedSeq s = packed_seq(a, blockIdx.x / a.kv_heads);
    const int queries = counted_queries(a, s);
    if (queries == 0) return;
    attend<D, FP16, W>(a, s, {static_cast<int>(blockIdx.x % a.kv_heads), 0, packed_limit(a, s, queries - 1), -1}, smem, found, 0);
}

// An equal stretch of all key blocks a CTA.
template <int D, bool FP16>
__global__ void __launch_bounds__(32 * kWarps, packed_rows_ctas(D)) packed_stream_kernel(const __grid_constant__ PackedArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int found[2];
    __shared__ int64_t sums[kWarps];
    __shared__ int64_t start_blocks;  // blocks before the sequence the stretch starts in
    __shared__ int start_seq;
    early_start();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // Blocks of all sequences: each thread counts a run of them, then a scan.
    const int run = (a.seqs + (32 * kWarps) - 1) / (32 * kWarps);
    const int first = threadIdx.x * run, last = min(first + run, a.seqs);
    int64_t mine = 0;
    for (int i = first; i < last; ++i) mine += key_blocks(a, packed_seq(a, i));
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
    }
    if (lane == 31) sums[warp] = upto;
    if (threadIdx.x == 0) found[0] = found[1] = 0;
    __syncthreads();
    int64_t all = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        if (i < warp) upto += sums[i];
        all += sums[i];
    }
    // two blocks at least: a stretch has a beginning and an end
    const int64_t stretch = max((all + a.streams - 1) / a.streams, int64_t(2));
    const int kvh = blockIdx.x % a.kv_heads, stream = blockIdx.x / a.kv_heads;
    int64_t at = stream * stretch;
    const int64_t to = min(at + stretch, all);
    if (at >= to) return;
    if (upto - mine <= at && at < upto) {
        int64_t before = upto - mine;
        int i = first;
        for (;; ++i) {
            const int n = key_blocks(a, packed_seq(a, i));
            if (at < before + n) break;
            before += n;
        }
        start_seq = i;
        start_blocks = before;
    }
    __syncthreads();
    int seq = start_seq;
    PackedSeq s = packed_seq(a, seq);
    int blocks = key_blocks(a, s);
    int block = static_cast<int>(at - start_blocks);
    for (int slot = 0, turn = 0;; slot = 1, turn ^= 1) {
        const int count = static_cast<int>(min(static_cast<int64_t>(blocks - block), to - at));
        const int end = min((block + count) * kBlockKeys, packed_limit(a, s, counted_queries(a, s) - 1));
        // only a stretch's first and last sequence can be a part
        const int part = count == blocks ? -1 : stream * 2 + slot;
        attend<D, FP16, kWarps>(a, s, {kvh, block * kBlockKeys, end, part < 0 ? -1 : packed_part_slot(a, part, kvh)}, smem, found, turn);
        if (threadIdx.x == 0 && kvh == 0) {
            if (block == 0) a.part_slots[seq].x = part;
            if (block + count == blocks) a.part_slots[seq].y = part;
        }
        at += count;
        if (at >= to) return;
        block = 0;
        do {  // there are blocks left, so a sequence that has some follows
            s = packed_seq(a, ++seq);
            blocks = key_blocks(a, s);
        } while (blocks == 0);
    }
}

template <int D, bool FP16, int W, bool STREAM>
cudaError_t launch(const PackedArgs& a, cudaStream_t st) {
    constexpr int smem = Geo<D, W>::kSmem;
    static std::atomic<uint64_t> done{0};
    constexpr auto kernel = STREAM ? packed_stream_kernel<D, FP16> : packed_rows_kernel<D, FP16, W>;
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), smem, done);
    if (e != cudaSuccess) return e;
    const int64_t grid = static_cast<int64_t>(STREAM ? a.streams : a.seqs) * a.kv_heads;
    return launch_early(kernel, dim3(static_cast<unsigned>(grid)), 32 * W, smem, st, a);
}

template <int D, bool FP16>
cudaError_t run(const PackedArgs& a, cudaStream_t st) {
    if (a.streams > 0) return launch<D, FP16, kWarps, true>(a, st);
    // Few CTAs: each takes its keys faster with more warps (us, four warps against
    // eight: 8 x 16 heads x 64 up to 900 keys 8.95 / 7.63, 16 x 8 x 128 up to 700
    // 12.3 / 10.8, but 16 x 16 x 128, 256 CTAs, 13.9 / 15.8)
    if (packed_rows_few(D, static_cast<int64_t>(a.seqs) * a.kv_heads)) return launch<D, FP16, 8, false>(a, st);
    return launch<D, FP16, kWarps, false>(a, st);
}

}  // namespace

cudaError_t launch_packed_rows(const PackedArgs& a, int d, bool fp16, cudaStream_t st) {
    switch (d) {
        case 64: return fp16 ? run<64, true>(a, st) : run<64, false>(a, st);
        case 96: return fp16 ? run<96, true>(a, st) : run<96, false>(a, st);
        default: return fp16 ? run<128, true>(a, st) : run<128, false>(a, st);
    }
}

}  // namespace h3a
