// The residual's addition and the root-mean-square norm of the prompt side, to
// 16 bits or to e4m3 with scales (h3a_residual_rmsnorm):
//
//   h = x + f (rounded once),  y = h * r * gamma,  r = 1 / sqrt(mean(h^2) + eps),
//   e4m3: scale = max(max|y|, 2^-100) / 448 per row or group of 128 channels.
//
// HBM-bound: x and f are read once, h and y written once (7 bytes a channel
// with the residual and e4m3).  `lanes` threads hold a row in registers, VPT
// vectors of eight channels each: a part of a warp for narrow rows, a whole CTA
// for wide ones.  They go on to their next row (persistent grid): gamma stays
// in registers, and the rows to come are on their way meanwhile.  Those of a
// wide row with its residual wait in registers, one row ahead; the others come
// through shared memory by cp.async, two rows ahead, into slots that belong to
// the thread that reads them, so that no barrier stands between copy and use.
// (One way for both: 200,000 rows of 96 with residual take 42 us by registers
// and 24 through shared memory, 8,000 of 8,192 without 49 and 43, but 8,192 of
// 4,096 with it 39.7 and 42.)  The sum of squares and max|h * gamma| are reduced
// together (one barrier a row, none for parts of a warp); max|y| is r times the
// latter.  Divisions are taken once a row or group, as reciprocals: y / scale is then two
// roundings from the quotient instead of one, 2^-24 against e4m3's 2^-4, and a value on
// the border of two codes may take the other one.
// Measured: 124,992 rows of 5,376 with residual and row scales 784 us (4.70 GB,
// 6.0 TB/s = 0.91 of a copy), 8,192 of 4,096 with group scales 40.6 us (0.89).
#include <algorithm>

#include "half16.cuh"
#include "prompt_internal.h"

namespace h3a {
namespace {

constexpr float kE4m3Most = 448.f;
constexpr float kLeastAmax = 0x1p-100f;
constexpr int kStages = 3;

// max that keeps a NaN of either side
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ void copy16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))), "l"(src)
                 : "memory");
}

// LANES: threads of a row, a power of two up to 32, or 0 for the whole CTA
template <int VPT, int LANES, bool FP16, int SCALES, bool RES>
__global__ void __launch_bounds__(LANES ? 128 : 512) residual_rmsnorm_kernel(const RmsNormArgs a) {
    using H = Half16<FP16>;
    constexpr int kOf = RES ? 2 : 1;       // vectors a channel vector is made from
    constexpr bool kRing = LANES || !RES;  // rows to come wait in shared memory, else in registers
    extern __shared__ uint4 ring[];        // [stage][VPT][x, f][thread]
    uint4 ahead[VPT][kOf];
    __shared__ float red[2][2][16];   // [row parity][sum of squares, max][warp]
    const int nvec = a.width / 8, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int warps = blockDim.x >> 5;
    const int step = LANES ? LANES : blockDim.x;
    const int mine = LANES ? threadIdx.x & (LANES - 1) : threadIdx.x;
    const int64_t rows_at_once = LANES ? static_cast<int64_t>(gridDim.x) * (blockDim.x / step) : gridDim.x;
    const uint16_t* x = static_cast<const uint16_t*>(a.x);
    const uint16_t* f = static_cast<const uint16_t*>(a.f);
    int64_t row = LANES ? static_cast<int64_t>(blockIdx.x) * (blockDim.x / step) + threadIdx.x / step : blockIdx.x;
    auto slot = [&](int stage, int u, int of) -> uint4& { return ring[((stage * VPT + u) * kOf + of) * blockDim.x + threadIdx.x]; };
    auto fetch = [&](int64_t r, int stage) {
        if (r < a.rows) {
#pragma unroll
            for (int u = 0; u < VPT; ++u) {
                const int v = mine + u * step;
                if (v >= nvec) continue;
                const uint4* px = reinterpret_cast<const uint4*>(x + r * a.xs) + v;
                const uint4* pf = reinterpret_cast<const uint4*>(f + r * a.fs) + v;
                if constexpr (kRing) {
                    copy16(&slot(stage, u, 0), px);
                    if (RES) copy16(&slot(stage, u, kOf - 1), pf);
                } else {
                    ahead[u][0] = __ldcs(px);
                    if (RES) ahead[u][kOf - 1] = __ldcs(pf);
                }
            }
        }
        if (kRing) asm volatile("cp.async.commit_group;" ::: "memory");  // an empty group keeps the count
    };
    early_start();
#pragma unroll
    for (int i = 0; i < (kRing ? kStages - 1 : 1); ++i) fetch(row + i * rows_at_once, i);
    float g[VPT][8];
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
        const int v = mine + u * step;
        float4 g0 = make_float4(0.f, 0.f, 0.f, 0.f), g1 = g0;
        if (v < nvec) {
            g0 = __ldg(reinterpret_cast<const float4*>(a.gamma) + 2 * v);
            g1 = __ldg(reinterpret_cast<const float4*>(a.gamma) + 2 * v + 1);
        }
        g[u][0] = g0.x, g[u][1] = g0.y, g[u][2] = g0.z, g[u][3] = g0.w;
        g[u][4] = g1.x, g[u][5] = g1.y, g[u][6] = g1.z, g[u][7] = g1.w;
    }
    const float inv_width = 1.0f / static_cast<float>(a.width);
    // every row of a warp's lanes runs as long as one of them has a row left: the reductions are of the whole warp
    const int64_t rounds = (a.rows - (LANES ? static_cast<int64_t>(blockIdx.x) * (blockDim.x / step) : row) + rows_at_once - 1) / rows_at_once;
    int stage = 0;
    for (int64_t round = 0; round < rounds; ++round, row += rows_at_once) {
        const bool there = !LANES || row < a.rows;
        if (kRing) {
            fetch(row + (kStages - 1) * rows_at_once, stage == 0 ? kStages - 1 : stage - 1);
            asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
        }
        float y[VPT][8];  // h * gamma
        float sum = 0.f, most = 0.f;
        float group_most[VPT];
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            const int v = mine + u * step;
            const bool in = there && v < nvec;
            const uint4 xr = !in ? make_uint4(0, 0, 0, 0) : kRing ? slot(stage, u, 0) : ahead[u][0];
            uint32_t w[4] = {xr.x, xr.y, xr.z, xr.w};
            if (RES) {
                const uint4 fr = !in ? make_uint4(0, 0, 0, 0) : kRing ? slot(stage, u, kOf - 1) : ahead[u][kOf - 1];
                const uint32_t wf[4] = {fr.x, fr.y, fr.z, fr.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float lo, hi, flo, fhi;
                    H::unpack(w[i], lo, hi);
                    H::unpack(wf[i], flo, fhi);
                    w[i] = H::pack(lo + flo, hi + fhi);  // the statistics use the rounded values
                }
                if (in) reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.h) + row * a.hs)[v] = make_uint4(w[0], w[1], w[2], w[3]);
            }
            group_most[u] = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float lo, hi;
                H::unpack(w[i], lo, hi);
                sum = fmaf(lo, lo, sum);
                sum = fmaf(hi, hi, sum);
                y[u][2 * i] = lo * g[u][2 * i];
                y[u][2 * i + 1] = hi * g[u][2 * i + 1];
                if (SCALES != H3A_SCALES_NONE)
                    group_most[u] = max_nan(group_most[u], max_nan(fabsf(y[u][2 * i]), fabsf(y[u][2 * i + 1])));
            }
            if (SCALES == H3A_SCALES_ROW) most = max_nan(most, group_most[u]);
        }
        if (!kRing) fetch(row + rows_at_once, 0);  // in flight while this row is reduced and written
#pragma unroll
        for (int o = (LANES ? LANES : 32) / 2; o > 0; o >>= 1) {
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (SCALES == H3A_SCALES_ROW) most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, o));
        }
        if (!LANES) {
            // rows alternate between two buffers: whoever still reads this one
            // has not passed the next row's barrier
            const int parity = round & 1;
            if (lane == 0) {
                red[parity][0][warp] = sum;
                if (SCALES == H3A_SCALES_ROW) red[parity][1][warp] = most;
            }
            __syncthreads();
            sum = lane < warps ? red[parity][0][lane] : 0.f;
            if (SCALES == H3A_SCALES_ROW) most = lane < warps ? red[parity][1][lane] : 0.f;
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) {
                sum += __shfl_xor_sync(0xffffffffu, sum, o);
                if (SCALES == H3A_SCALES_ROW) most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, o));
            }
            sum = __shfl_sync(0xffffffffu, sum, 0);
            if (SCALES == H3A_SCALES_ROW) most = __shfl_sync(0xffffffffu, most, 0);
        }
        const float r = rsqrtf(fmaf(sum, inv_width, a.eps));
        // What turns y = h * gamma * r into what is rounded.  Not multiplied into r: with
        // small rows (r large) and a group of zeros (scale least) their product overflows.
        float q = 1.f;
        if (SCALES == H3A_SCALES_ROW) {
            const float scale = max_nan(most * r, kLeastAmax) * (1.0f / kE4m3Most);
            q = __frcp_rn(scale);
            if (there && mine == 0) a.scales[row] = scale;
        }
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            const int v = mine + u * step;
            if (SCALES == H3A_SCALES_GROUP) {
                // a group of 128 channels is 16 neighbouring threads (or all of a row that has fewer)
                float m = group_most[u];
#pragma unroll
                for (int o = LANES && LANES < 16 ? LANES / 2 : 8; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
                const float scale = max_nan(m * r, kLeastAmax) * (1.0f / kE4m3Most);
                q = __frcp_rn(scale);
                if (there && v < nvec && (v & 15) == 0) a.scales[row * ((nvec + 15) / 16) + v / 16] = scale;
            }
            if (!there || v >= nvec) continue;
#pragma unroll
            for (int i = 0; i < 8; ++i) y[u][i] *= r;
            if (SCALES == H3A_SCALES_NONE) {
                uint4 w;
                w.x = H::pack(y[u][0], y[u][1]);
                w.y = H::pack(y[u][2], y[u][3]);
                w.z = H::pack(y[u][4], y[u][5]);
                w.w = H::pack(y[u][6], y[u][7]);
                reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.y) + row * a.ys)[v] = w;
            } else {
                uint2 w;
                w.x = pack_e4m3x2(y[u][0] * q, y[u][1] * q) | pack_e4m3x2(y[u][2] * q, y[u][3] * q) << 16;
                w.y = pack_e4m3x2(y[u][4] * q, y[u][5] * q) | pack_e4m3x2(y[u][6] * q, y[u][7] * q) << 16;
                reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.y) + row * a.ys)[v] = w;
            }
        }
        stage = stage + 1 == kStages ? 0 : stage + 1;
    }
}

template <int VPT, int LANES, bool FP16, int SCALES, bool RES>
cudaError_t launch(const RmsNormArgs& a, int threads, cudaStream_t st) {
    constexpr bool ring = LANES || !RES;
    const int smem = ring ? kStages * VPT * (RES ? 2 : 1) * threads * 16 : 0;
    if (smem > 47 << 10) {  // 48 KB with the static array
        static std::atomic<uint64_t> done{0};
        constexpr int most = kStages * (RES ? 2 : 1) * kRmsNormMaxWidth * 2;
        const cudaError_t e = allow_smem(reinterpret_cast<const void*>(residual_rmsnorm_kernel<VPT, LANES, FP16, SCALES, RES>), most, done);
        if (e != cudaSuccess) return e;
    }
    // persistent: about as many CTAs as registers and shared memory let a multiprocessor hold
    const int per_sm = std::max(1, ring ? std::min(2048 / threads, (200 << 10) / smem) : 1024 / threads);
    const int64_t rows = LANES ? threads / LANES : 1;
    const int64_t grid = std::min<int64_t>((a.rows + rows - 1) / rows, kSms * per_sm);
    return launch_early(residual_rmsnorm_kernel<VPT, LANES, FP16, SCALES, RES>, dim3(static_cast<unsigned>(grid)), threads, smem, st, a);
}

template <int VPT, int LANES, bool FP16>
cudaError_t run(const RmsNormArgs& a, h3a_scales scales, int threads, cudaStream_t st) {
    switch (scales) {
        case H3A_SCALES_ROW:
            return a.f ? launch<VPT, LANES, FP16, H3A_SCALES_ROW, true>(a, threads, st)
                       : launch<VPT, LANES, FP16, H3A_SCALES_ROW, false>(a, threads, st);
        case H3A_SCALES_GROUP:
            return a.f ? launch<VPT, LANES, FP16, H3A_SCALES_GROUP, true>(a, threads, st)
                       : launch<VPT, LANES, FP16, H3A_SCALES_GROUP, false>(a, threads, st);
        default:
            return a.f ? launch<VPT, LANES, FP16, H3A_SCALES_NONE, true>(a, threads, st)
                       : launch<VPT, LANES, FP16, H3A_SCALES_NONE, false>(a, threads, st);
    }
}

template <int VPT, int LANES>
cudaError_t run(const RmsNormArgs& a, bool fp16, h3a_scales scales, int threads, cudaStream_t st) {
    return fp16 ? run<VPT, LANES, true>(a, scales, threads, st) : run<VPT, LANES, false>(a, scales, threads, st);
}

}  // namespace

cudaError_t launch_residual_rmsnorm(const RmsNormArgs& a, bool fp16, h3a_scales scales, cudaStream_t st) {
    if (a.rows == 0) return cudaSuccess;
    const int nvec = a.width / 8;
    // up to 1,024 channels a warp or part of one
    // (groups of 16 vectors must not be spread over a thread's vectors)
    if (nvec <= 8) return run<1, 8>(a, fp16, scales, 128, st);
    if (nvec <= 16) return run<1, 16>(a, fp16, scales, 128, st);
    if (nvec <= 32) return run<2, 16>(a, fp16, scales, 128, st);
    if (nvec <= 64) return run<2, 32>(a, fp16, scales, 128, st);
    if (nvec <= 96) return run<3, 0>(a, fp16, scales, 32, st);
    if (nvec <= 128) return run<4, 0>(a, fp16, scales, 32, st);
    // then a CTA a row, with the fewest idle vector slots
    auto threads_of = [&](int vpt) { return ((nvec + vpt - 1) / vpt + 31) / 32 * 32; };
    int vpt = 4, best = 1 << 30;
    for (int c = 2; c <= 4; ++c) {
        if (threads_of(c) > 512) continue;
        const int idle = threads_of(c) * c - nvec;
        if (idle < best) best = idle, vpt = c;
    }
    switch (vpt) {
        case 2: return run<2, 0>(a, fp16, scales, threads_of(2), st);
        case 3: return run<3, 0>(a, fp16, scales, threads_of(3), st);
        default: return run<4, 0>(a, fp16, scales, threads_of(4), st);
    }
}

}  // namespace h3a
