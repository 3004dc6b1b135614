// One-dimensional rotary positions over q and k of packed prompts or single
// tokens (the prompt side's counterpart of the 3D prologue in prologue.cu).
//
//   (a', b') = A (a cos th - b sin th, a sin th + b cos th),
//   th = 2 pi frac(position * turns_j)
//
// turns_j is a 64-bit fixed-point fraction of a turn per position, so the
// product modulo 2^64 is the angle's exact place on the circle for any int32
// position; its top 32 bits feed sincospi.  HBM-bound: every element is read
// and written once, 4 bytes.
//
// A thread owns one slot of a head -- VEC pairs, as two vectors of VEC elements
// -- for every head of its token, so cos and sin are computed once per token
// and slot and stay in registers.  VEC is the largest power of two (at most 8,
// 16-byte vectors) that divides the number of pairs: both vectors of a slot
// are then aligned in either layout.
#include "half16.cuh"
#include "prompt_internal.h"

namespace h3a {
namespace {

template <int VEC>
struct Vec;
template <>
struct Vec<8> {
    using Raw = uint4;
};
template <>
struct Vec<4> {
    using Raw = uint2;
};
template <>
struct Vec<2> {
    using Raw = uint32_t;
};
template <>
struct Vec<1> {
    using Raw = uint16_t;
};

template <bool FP16, int VEC>
__device__ __forceinline__ void unpack(const typename Vec<VEC>::Raw& r, float (&x)[VEC]) {
    if constexpr (VEC == 1) {
        float hi;
        Half16<FP16>::unpack(r, x[0], hi);
    } else {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&r);
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) Half16<FP16>::unpack(w[i], x[2 * i], x[2 * i + 1]);
    }
}

template <bool FP16, int VEC>
__device__ __forceinline__ typename Vec<VEC>::Raw pack(const float (&x)[VEC]) {
    typename Vec<VEC>::Raw r;
    if constexpr (VEC == 1) {
        r = static_cast<uint16_t>(Half16<FP16>::pack(x[0], 0.f));
    } else {
        uint32_t* w = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) w[i] = Half16<FP16>::pack(x[2 * i], x[2 * i + 1]);
    }
    return r;
}

struct RopeArgs {
    RopeSide side[2];
    const int32_t* positions;
    int64_t tokens;
    int head_dim;
    int slots;          // rotated slots, then (out of place) copied ones
    int heads_at_once;  // heads a block works on side by side
    int heads_per_block;
    bool inverse;
    h3a_rope_plan plan;
};

constexpr int kAhead = 4;  // heads whose loads a thread has in flight

template <bool FP16, int VEC>
__global__ void __launch_bounds__(288) rope_kernel(const __grid_constant__ RopeArgs a) {
    using Raw = typename Vec<VEC>::Raw;
    using T = uint16_t;
    const int slot = threadIdx.x % a.slots;
    const int lane_head = threadIdx.x / a.slots;
    if (lane_head >= a.heads_at_once) return;
    const int rotated = a.plan.pairs / VEC;
    const bool turn = slot < rotated;
    // channels of the slot's two vectors; a copied slot's second one may lie past the head
    int ca, cb;
    if (!turn) {
        ca = 2 * a.plan.pairs + (slot - rotated) * 2 * VEC;
        cb = ca + VEC;
    } else if (a.plan.interleaved) {
        ca = slot * 2 * VEC;
        cb = ca + VEC;
    } else {
        ca = slot * VEC;
        cb = a.plan.pairs + ca;
    }
    const bool has_b = cb < a.head_dim;
    uint64_t turns[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) turns[i] = turn ? a.plan.turns[slot * VEC + i] : 0;
    const int nq = a.side[0].heads, heads = nq + a.side[1].heads;
    const int h0 = blockIdx.y * a.heads_per_block + lane_head;
    const int h1 = min(heads, (static_cast<int>(blockIdx.y) + 1) * a.heads_per_block);

    for (int64_t n = blockIdx.x; n < a.tokens; n += gridDim.x) {
        float c[VEC], s[VEC];
        const int64_t position = __ldg(a.positions + n);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            // signed half turns in [-1, 1)
            const int top = static_cast<int>((static_cast<uint64_t>(position) * turns[i]) >> 32);
            sincospif(static_cast<float>(top) * 0x1p-31f, &s[i], &c[i]);
            c[i] *= a.plan.amplitude;
            s[i] *= a.inverse ? -a.plan.amplitude : a.plan.amplitude;
        }
        for (int h = h0; h < h1; h += kAhead * a.heads_at_once) {
            Raw ra[kAhead], rb[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int hu = h + u * a.heads_at_once;
                if (hu >= h1) break;
                const bool is_k = hu >= nq;
                const RopeSide& sd = a.side[is_k];
                const T* x = static_cast<const T*>(sd.x) + n * sd.sn + (hu - (is_k ? nq : 0)) * sd.sh;
                ra[u] = *reinterpret_cast<const Raw*>(x + ca);
                if (has_b) rb[u] = *reinterpret_cast<const Raw*>(x + cb);
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int hu = h + u * a.heads_at_once;
                if (hu >= h1) break;
                const bool is_k = hu >= nq;
                const RopeSide& sd = a.side[is_k];
                T* y = static_cast<T*>(sd.y) + n * sd.on + (hu - (is_k ? nq : 0)) * sd.oh;
                if (turn) {
                    float xa[VEC], xb[VEC], ya[VEC], yb[VEC];
                    unpack<FP16, VEC>(ra[u], xa);
                    unpack<FP16, VEC>(rb[u], xb);
                    if (a.plan.interleaved) {
                        // the two vectors are 2 * VEC consecutive channels: pair i is elements 2i and 2i + 1
#pragma unroll
                        for (int i = 0; i < VEC; ++i) {
                            const float p = 2 * i < VEC ? xa[(2 * i) % VEC] : xb[(2 * i) % VEC];
                            const float q = 2 * i + 1 < VEC ? xa[(2 * i + 1) % VEC] : xb[(2 * i + 1) % VEC];
                            const float p1 = fmaf(p, c[i], -(q * s[i])), q1 = fmaf(p, s[i], q * c[i]);
                            (2 * i < VEC ? ya : yb)[(2 * i) % VEC] = p1;
                            (2 * i + 1 < VEC ? ya : yb)[(2 * i + 1) % VEC] = q1;
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < VEC; ++i) {
                            ya[i] = fmaf(xa[i], c[i], -(xb[i] * s[i]));
                            yb[i] = fmaf(xa[i], s[i], xb[i] * c[i]);
                        }
                    }
                    ra[u] = pack<FP16, VEC>(ya);
                    rb[u] = pack<FP16, VEC>(yb);
                }
                *reinterpret_cast<Raw*>(y + ca) = ra[u];
                if (has_b) *reinterpret_cast<Raw*>(y + cb) = rb[u];
            }
        }
    }
}

template <bool FP16, int VEC>
cudaError_t run(RopeArgs& a, bool copies, cudaStream_t st) {
    const int rest = a.head_dim - 2 * a.plan.pairs;
    a.slots = a.plan.pairs / VEC + (copies ? (rest + 2 * VEC - 1) / (2 * VEC) : 0);
    const int threads = a.slots <= 128 ? 128 : (a.slots + 31) / 32 * 32;
    const int heads = a.side[0].heads + a.side[1].heads;
    a.heads_at_once = threads / a.slots;
    const int steps = (heads + a.heads_at_once - 1) / a.heads_at_once;
    // A token's heads stay with one block, which computes its cos and sin once,
    // unless that leaves multiprocessors without work.
    constexpr int64_t kBlocks = kSms * 16;
    int64_t parts = kBlocks / (a.tokens > 0 ? a.tokens : 1);
    parts = parts < 1 ? 1 : parts > steps ? steps : parts;
    a.heads_per_block = static_cast<int>((steps + parts - 1) / parts) * a.heads_at_once;
    const dim3 grid(static_cast<unsigned>(a.tokens < kBlocks ? a.tokens : kBlocks),
                    static_cast<unsigned>((heads + a.heads_per_block - 1) / a.heads_per_block));
    rope_kernel<FP16, VEC><<<grid, threads, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeSide& q, const RopeSide& k, int head_dim, bool fp16, const int32_t* positions,
                        int64_t tokens, const h3a_rope_plan& plan, bool inverse, cudaStream_t st) {
    if (tokens == 0) return cudaSuccess;
    RopeArgs a;
    a.side[0] = q;
    a.side[1] = k;
    a.positions = positions;
    a.tokens = tokens;
    a.head_dim = head_dim;
    a.inverse = inverse;
    a.plan = plan;
    // channels past the rotated ones are copied unless every side works in place
    const bool copies = (q.x != q.y) || (k.heads > 0 && k.x != k.y);
    const int p = plan.pairs;
    if (p % 8 == 0) return fp16 ? run<true, 8>(a, copies, st) : run<false, 8>(a, copies, st);
    if (p % 4 == 0) return fp16 ? run<true, 4>(a, copies, st) : run<false, 4>(a, copies, st);
    if (p % 2 == 0) return fp16 ? run<true, 2>(a, copies, st) : run<false, 2>(a, copies, st);
    return fp16 ? run<true, 1>(a, copies, st) : run<false, 1>(a, copies, st);
}

}  // namespace h3a
