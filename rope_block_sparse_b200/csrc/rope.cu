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
// An item is one head of one token; the threads of a group take a slot of it
// each (see Mode).  A block takes a chunk of ITEMS items a group: it loads
// them, computes the (cos, sin) of the chunk's tokens once into shared memory
// while the loads are in flight, rotates and stores.
#include "half16.cuh"
#include "prompt_internal.h"

namespace h3a {
namespace {

// What a slot is, by the number of pairs and the layout.
enum Mode {
    kPaired8,     // a multiple of 8 pairs: two vectors of 8 channels that hold 8 whole pairs
    kPaired4,     // a multiple of 4: the same with vectors of 4 channels
    kNeighbours,  // interleaved, any number: one vector of 8 channels, 4 whole pairs
    // halves, any number: one vector of 8 channels, whose partners lie `pairs`
    // channels away at any alignment and come through shared memory
    kHalvesAny,
};
template <Mode MODE>
constexpr bool kPaired = MODE == kPaired8 || MODE == kPaired4;
template <Mode MODE>
constexpr int kVec = MODE == kPaired4 ? 4 : 8;  // channels of a vector
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

struct RopeArgs {
    RopeSide side[2];
    const int32_t* positions;
    int64_t items;       // tokens * heads of both sides
    int heads;           // of both sides
    int head_dim;
    uint32_t heads_inv;  // ceil(2^32 / heads), for the quotient of small numbers
    uint32_t row_inv;    // the same of a token's row of angles
    int slots;           // threads of a group
    int groups;          // items a block works on side by side
    bool inverse;
    h3a_rope_plan plan;
};

// n / d by inv = ceil(2^32 / d): exact while n * d < 2^32
__device__ __forceinline__ uint32_t quotient(uint32_t n, uint32_t inv, uint32_t d) {
    return d == 1 ? n : __umulhi(n, inv);
}

template <bool FP16, int VEC>
__device__ __forceinline__ void unpack(const typename Vec<VEC>::Raw& r, float (&x)[VEC]) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&r);
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) Half16<FP16>::unpack(w[i], x[2 * i], x[2 * i + 1]);
}

template <bool FP16, int VEC>
__device__ __forceinline__ typename Vec<VEC>::Raw pack(const float (&x)[VEC]) {
    typename Vec<VEC>::Raw r;
    uint32_t* w = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) w[i] = Half16<FP16>::pack(x[2 * i], x[2 * i + 1]);
    return r;
}

// Angles a slot reads of its token's row.
template <Mode MODE>
constexpr int kAngles = MODE == kPaired8 || MODE == kHalvesAny ? 8 : 4;
// Rotated slots of a head: what follows is copied.
template <Mode MODE>
__host__ __device__ __forceinline__ int rotated_slots(int pairs) {
    return kPaired<MODE> ? pairs / kVec<MODE> : (2 * pairs + 7) / 8;
}
// Place of a slot's angle e in the row: two angles of neighbouring slots lie 16
// bytes apart, so that a warp's 16-byte loads do not collide.
__device__ __forceinline__ int angle_at(int slot, int e, int rotated) { return ((e >> 1) * rotated + slot) * 2 + (e & 1); }

// Blocks in flight and queued per multiprocessor.  8,192 tokens of 40 heads x 128:
// 31.5 us at 8, 28.8 at 16, 27.6 at 32 (one chunk each then); as it stands 26.9 (168
// MB, 6.2 TB/s = 0.95 of a copy).  30,011 tokens of 32 heads x 96, half rotated: 57.1 us
// (369 MB, 6.5 TB/s).  Angles per thread instead of per chunk took 37 and 97 us.  The
// same 8,192 tokens with 25 rotated pairs: 31.9 us as neighbours, 40.8 as halves
// (kHalvesAny: eight 2-byte shared loads a vector), 43.2 with 63 pairs.
constexpr int kBlocksPerSm = 32;
constexpr int kThreads = 128;

template <bool FP16, Mode MODE, int ITEMS>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
    constexpr int VEC = kVec<MODE>;
    using Raw = typename Vec<VEC>::Raw;
    extern __shared__ __align__(16) float2 angles[];  // [token][row of angles], then (kHalvesAny) the items' heads
    __shared__ uint64_t turns[H3A_ROPE_MAX_PAIRS];
    const int pairs = a.plan.pairs, rotated = rotated_slots<MODE>(pairs), row = rotated * kAngles<MODE>;
    // Parameters indexed by thread: read through their address, since constant
    // loads of unlike addresses are served one after the other.
    for (int i = threadIdx.x; i < pairs; i += kThreads)
        asm volatile("ld.u64 %0, [%1];" : "=l"(turns[i]) : "l"(&a.plan.turns[i]));

    early_start();

    const int slot = threadIdx.x % a.slots;
    const int group = threadIdx.x / a.slots;
    const bool busy = group < a.groups, turn = slot < rotated;
    // first channels of the slot's vectors; a copied slot's second one may lie past the head
    const bool halves = kPaired<MODE> && turn && !a.plan.interleaved;
    const int ca = slot * (kPaired<MODE> && !halves ? 2 * VEC : VEC);
    const int cb = halves ? pairs + ca : ca + VEC;
    const bool has_b = kPaired<MODE> && cb < a.head_dim;
    const int nq = a.side[0].heads;
    const uint32_t per_chunk = ITEMS * a.groups;

    for (int64_t first = static_cast<int64_t>(blockIdx.x) * per_chunk; first < a.items;
         first += static_cast<int64_t>(gridDim.x) * per_chunk) {
        const int64_t token0 = first / a.heads;
        const uint32_t into = static_cast<uint32_t>(first - token0 * a.heads);  // head of the chunk's first item
        const uint32_t items = static_cast<uint32_t>(min(static_cast<int64_t>(per_chunk), a.items - first));
        const uint32_t tokens = quotient(into + items - 1, a.heads_inv, a.heads) + 1;
        uint16_t* staged = reinterpret_cast<uint16_t*>(angles + static_cast<size_t>(tokens) * row);
        Raw ra[ITEMS], rb[ITEMS];
#pragma unroll
        for (int u = 0; u < ITEMS; ++u) {
            const uint32_t item = u * a.groups + group;
            if (!busy || item >= items) break;
            const uint32_t t = quotient(into + item, a.heads_inv, a.heads), h = into + item - t * a.heads;
            const RopeSide& sd = a.side[h >= nq];
            const uint16_t* x = static_cast<const uint16_t*>(sd.x) + (token0 + t) * sd.sn + (h >= nq ? h - nq : h) * sd.sh;
            ra[u] = *reinterpret_cast<const Raw*>(x + ca);
            if (has_b) rb[u] = *reinterpret_cast<const Raw*>(x + cb);
        }
        __syncthreads();  // turns are there; the last chunk's angles are no longer read
        for (uint32_t i = threadIdx.x; i < tokens * row; i += kThreads) {
            const uint32_t t = quotient(i, a.row_inv, row), c = i - t * row;
            const int64_t position = __ldg(a.positions + token0 + t);
            const int pair = MODE == kHalvesAny && static_cast<int>(c) >= pairs ? c - pairs : c;
            // signed half turns in [-1, 1); angles past the last pair are not read
            const int top = pair < pairs ? static_cast<int>((static_cast<uint64_t>(position) * turns[pair]) >> 32) : 0;
            float s, cosine;
            sincospif(static_cast<float>(top) * 0x1p-31f, &s, &cosine);
            s *= a.inverse ? -a.plan.amplitude : a.plan.amplitude;
            if (MODE == kHalvesAny && static_cast<int>(c) < pairs) s = -s;  // by channel: x cos + partner * s
            angles[t * row + angle_at(c / kAngles<MODE>, c % kAngles<MODE>, rotated)] = make_float2(cosine * a.plan.amplitude, s);
        }
        if (MODE == kHalvesAny) {
#pragma unroll
            for (int u = 0; u < ITEMS; ++u) {
                const uint32_t item = u * a.groups + group;
                if (!busy || item >= items) break;
                if (turn) *reinterpret_cast<Raw*>(staged + (item * rotated + slot) * 8) = ra[u];
            }
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < ITEMS; ++u) {
            const uint32_t item = u * a.groups + group;
            if (!busy || item >= items) break;
            const uint32_t t = quotient(into + item, a.heads_inv, a.heads), h = into + item - t * a.heads;
            const RopeSide& sd = a.side[h >= nq];
            uint16_t* y = static_cast<uint16_t*>(sd.y) + (token0 + t) * sd.on + (h >= nq ? h - nq : h) * sd.oh;
            if (turn) {
                float c[kAngles<MODE>], s[kAngles<MODE>], xa[VEC], ya[VEC];
#pragma unroll
                for (int e = 0; e < kAngles<MODE>; e += 2) {
                    const float4 v = *reinterpret_cast<const float4*>(angles + t * row + angle_at(slot, e, rotated));
                    c[e] = v.x, s[e] = v.y, c[e + 1] = v.z, s[e + 1] = v.w;
                }
                unpack<FP16, VEC>(ra[u], xa);
                if constexpr (kPaired<MODE>) {
                    float xb[VEC], yb[VEC];
                    unpack<FP16, VEC>(rb[u], xb);
                    if (a.plan.interleaved) {
                        // consecutive vectors: pair i is their elements 2i and 2i + 1
#pragma unroll
                        for (int i = 0; i < VEC; ++i) {
                            const float p = 2 * i < VEC ? xa[(2 * i) % VEC] : xb[(2 * i) % VEC];
                            const float q = 2 * i < VEC ? xa[(2 * i + 1) % VEC] : xb[(2 * i + 1) % VEC];
                            (2 * i < VEC ? ya : yb)[(2 * i) % VEC] = fmaf(p, c[i], -(q * s[i]));
                            (2 * i < VEC ? ya : yb)[(2 * i + 1) % VEC] = fmaf(p, s[i], q * c[i]);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < VEC; ++i) {
                            ya[i] = fmaf(xa[i], c[i], -(xb[i] * s[i]));
                            yb[i] = fmaf(xa[i], s[i], xb[i] * c[i]);
                        }
                    }
                    rb[u] = pack<FP16, VEC>(yb);
                } else if constexpr (MODE == kNeighbours) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        ya[2 * i] = fmaf(xa[2 * i], c[i], -(xa[2 * i + 1] * s[i]));
                        ya[2 * i + 1] = fmaf(xa[2 * i], s[i], xa[2 * i + 1] * c[i]);
                    }
                } else {
                    const uint16_t* head = staged + item * rotated * 8;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int ch = ca + i, partner = ch < pairs ? ch + pairs : ch - pairs;
                        float p, none;
                        Half16<FP16>::unpack(head[partner], p, none);
                        ya[i] = fmaf(xa[i], c[i], p * s[i]);
                    }
                }
                const Raw done = pack<FP16, VEC>(ya);
                if (!kPaired<MODE> && ca + 8 > 2 * pairs) {
                    // the vector in which the rotated channels end: the rest as it was, two channels a word
                    const uint32_t* from = reinterpret_cast<const uint32_t*>(&done);
                    uint32_t* w = reinterpret_cast<uint32_t*>(&ra[u]);
#pragma unroll
                    for (int i = 0; i < VEC / 2; ++i) w[i] = ca + 2 * i < 2 * pairs ? from[i] : w[i];
                } else {
                    ra[u] = done;
                }
            }
            *reinterpret_cast<Raw*>(y + ca) = ra[u];
            if (has_b) *reinterpret_cast<Raw*>(y + cb) = rb[u];
        }
    }
}

uint32_t inverse_of(int d) { return static_cast<uint32_t>(((uint64_t(1) << 32) + d - 1) / d); }

template <bool FP16, Mode MODE, int ITEMS>
cudaError_t launch(const RopeArgs& a, cudaStream_t st) {
    const int rotated = rotated_slots<MODE>(a.plan.pairs), row = rotated * kAngles<MODE>;
    const int per_chunk = ITEMS * a.groups;
    const int64_t chunks = (a.items + per_chunk - 1) / per_chunk, most = static_cast<int64_t>(kSms) * kBlocksPerSm;
    const size_t tokens = (per_chunk + a.heads - 2) / a.heads + 1;  // that a chunk may touch
    // at most 35 KB of angles and 8 KB of heads
    const size_t smem = tokens * row * sizeof(float2) + (MODE == kHalvesAny ? static_cast<size_t>(per_chunk) * rotated * 16 : 0);
    return launch_early(rope_kernel<FP16, MODE, ITEMS>, dim3(static_cast<unsigned>(chunks < most ? chunks : most)), kThreads, smem, st, a);
}

template <bool FP16, Mode MODE>
cudaError_t run(RopeArgs& a, bool copies, cudaStream_t st) {
    const int rotated = rotated_slots<MODE>(a.plan.pairs);
    constexpr int channels = kPaired<MODE> ? 2 * kVec<MODE> : 8;  // of a slot
    a.slots = copies ? (a.head_dim + channels - 1) / channels : rotated;
    a.groups = kThreads / a.slots;
    a.row_inv = inverse_of(rotated * kAngles<MODE>);
    // Few items: one a group, so that they spread over the GPU.  Many: enough
    // loads in flight a thread, and the angles shared by more heads.
    if (a.items <= static_cast<int64_t>(kSms) * 8 * a.groups) return launch<FP16, MODE, 1>(a, st);
    return launch<FP16, MODE, 4>(a, st);
}

template <bool FP16>
cudaError_t run(RopeArgs& a, bool copies, cudaStream_t st) {
    if (a.plan.pairs % 8 == 0) return run<FP16, kPaired8>(a, copies, st);
    if (a.plan.pairs % 4 == 0) return run<FP16, kPaired4>(a, copies, st);
    return a.plan.interleaved ? run<FP16, kNeighbours>(a, copies, st) : run<FP16, kHalvesAny>(a, copies, st);
}

}  // namespace

cudaError_t launch_rope(const RopeSide& q, const RopeSide& k, int head_dim, bool fp16, const int32_t* positions,
                        int64_t tokens, const h3a_rope_plan& plan, bool inverse, cudaStream_t st) {
    if (tokens == 0) return cudaSuccess;
    RopeArgs a;
    a.side[0] = q;
    a.side[1] = k;
    a.positions = positions;
    a.heads = q.heads + k.heads;
    a.items = tokens * a.heads;
    a.heads_inv = inverse_of(a.heads);
    a.head_dim = head_dim;
    a.inverse = inverse;
    a.plan = plan;
    // channels past the rotated ones are copied unless every side works in place
    const bool copies = (q.x != q.y) || (k.heads > 0 && k.x != k.y);
    return fp16 ? run<true>(a, copies, st) : run<false>(a, copies, st);
}

}  // namespace h3a
