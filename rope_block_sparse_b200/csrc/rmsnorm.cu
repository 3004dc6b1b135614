// The residual's addition and the root-mean-square norm of the prompt side, to
// 16 bits or to e4m3 with scales (h3a_residual_rmsnorm):
//
//   h = x + f (rounded once),  y = h * r * gamma,  r = 1 / sqrt(mean(h^2) + eps),
//   e4m3: scale = max(max|y|, 2^-100) / 448 per row or group of 128 channels.
//
// HBM-bound: x and f are read once, h and y written once (7 bytes a channel
// with the residual and e4m3).  A CTA holds a row in registers, VPT vectors of
// eight channels a thread, and goes on to its next row (persistent grid):
// gamma stays in registers and the next row's loads are issued before this
// row's reduction, so they are in flight while it is normalised.  The sum of
// squares and max|h * gamma| are reduced together, one barrier a row; max|y|
// is r times the latter.
#include "half16.cuh"
#include "prompt_internal.h"

namespace h3a {
namespace {

constexpr float kE4m3Most = 448.f;
constexpr float kLeastAmax = 0x1p-100f;

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

template <int VPT, bool FP16, int SCALES>
__global__ void __launch_bounds__(512) residual_rmsnorm_kernel(const RmsNormArgs a) {
    using H = Half16<FP16>;
    __shared__ float red[2][2][16];  // [row parity][sum of squares, max][warp]
    const int nvec = a.width / 8, step = blockDim.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int warps = blockDim.x >> 5;
    const uint16_t* x = static_cast<const uint16_t*>(a.x);
    const uint16_t* f = static_cast<const uint16_t*>(a.f);
    float g[VPT][8];
    uint4 xr[VPT], fr[VPT];
    int64_t row = blockIdx.x;
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
        const int v = threadIdx.x + u * step;
        xr[u] = fr[u] = make_uint4(0, 0, 0, 0);
        if (v < nvec) {
            xr[u] = __ldcs(reinterpret_cast<const uint4*>(x + row * a.xs) + v);
            if (f) fr[u] = __ldcs(reinterpret_cast<const uint4*>(f + row * a.fs) + v);
            const float4 g0 = __ldg(reinterpret_cast<const float4*>(a.gamma) + 2 * v);
            const float4 g1 = __ldg(reinterpret_cast<const float4*>(a.gamma) + 2 * v + 1);
            g[u][0] = g0.x, g[u][1] = g0.y, g[u][2] = g0.z, g[u][3] = g0.w;
            g[u][4] = g1.x, g[u][5] = g1.y, g[u][6] = g1.z, g[u][7] = g1.w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) g[u][i] = 0.f;
        }
    }
    const float inv_width = 1.0f / static_cast<float>(a.width);
    for (int parity = 0; row < a.rows; parity ^= 1) {
        float y[VPT][8];  // h, then h * gamma
        float sum = 0.f, most = 0.f;
        float group_most[VPT];
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            const int v = threadIdx.x + u * step;
            uint32_t w[4] = {xr[u].x, xr[u].y, xr[u].z, xr[u].w};
            const uint32_t wf[4] = {fr[u].x, fr[u].y, fr[u].z, fr[u].w};
            group_most[u] = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float lo, hi;
                H::unpack(w[i], lo, hi);
                if (f) {
                    float flo, fhi;
                    H::unpack(wf[i], flo, fhi);
                    w[i] = H::pack(lo + flo, hi + fhi);
                    H::unpack(w[i], lo, hi);  // the statistics use the rounded values
                }
                sum = fmaf(lo, lo, sum);
                sum = fmaf(hi, hi, sum);
                y[u][2 * i] = lo * g[u][2 * i];
                y[u][2 * i + 1] = hi * g[u][2 * i + 1];
                if (SCALES != H3A_SCALES_NONE)
                    group_most[u] = max_nan(group_most[u], max_nan(fabsf(y[u][2 * i]), fabsf(y[u][2 * i + 1])));
            }
            if (SCALES == H3A_SCALES_ROW) most = max_nan(most, group_most[u]);
            if (f && v < nvec)
                reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.h) + row * a.hs)[v] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        const int64_t next = row + gridDim.x;
        if (next < a.rows) {
#pragma unroll
            for (int u = 0; u < VPT; ++u) {
                const int v = threadIdx.x + u * step;
                if (v < nvec) {
                    xr[u] = __ldcs(reinterpret_cast<const uint4*>(x + next * a.xs) + v);
                    if (f) fr[u] = __ldcs(reinterpret_cast<const uint4*>(f + next * a.fs) + v);
                }
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (SCALES == H3A_SCALES_ROW) most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, o));
        }
        if (warps > 1) {
            // rows alternate between two buffers: whoever still reads this one
            // has not passed the next row's barrier
            if (lane == 0) {
                red[parity][0][warp] = sum;
                if (SCALES == H3A_SCALES_ROW) red[parity][1][warp] = most;
            }
            __syncthreads();
            sum = lane < warps ? red[parity][0][lane] : 0.f;
            if (SCALES == H3A_SCALES_ROW) most = lane < warps ? red[parity][1][lane] : 0.f;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                sum += __shfl_xor_sync(0xffffffffu, sum, o);
                if (SCALES == H3A_SCALES_ROW) most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, o));
            }
        }
        const float r = 1.0f / sqrtf(fmaf(sum, inv_width, a.eps));
        float scale = 0.f;
        if (SCALES == H3A_SCALES_ROW) {
            scale = max_nan(most * r, kLeastAmax) / kE4m3Most;
            if (threadIdx.x == 0) a.scales[row] = scale;
        }
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            const int v = threadIdx.x + u * step;
            if (SCALES == H3A_SCALES_GROUP) {
                // a group of 128 channels is 16 neighbouring lanes
                float m = group_most[u];
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
                scale = max_nan(m * r, kLeastAmax) / kE4m3Most;
                if (v < nvec && (lane & 15) == 0) a.scales[row * ((nvec + 15) / 16) + v / 16] = scale;
            }
            if (v >= nvec) continue;
            if (SCALES == H3A_SCALES_NONE) {
                uint4 w;
                w.x = H::pack(y[u][0] * r, y[u][1] * r);
                w.y = H::pack(y[u][2] * r, y[u][3] * r);
                w.z = H::pack(y[u][4] * r, y[u][5] * r);
                w.w = H::pack(y[u][6] * r, y[u][7] * r);
                reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.y) + row * a.ys)[v] = w;
            } else {
                const float inv = 1.0f / scale;
                uint2 w;
                w.x = pack_e4m3x2(y[u][0] * r * inv, y[u][1] * r * inv) | pack_e4m3x2(y[u][2] * r * inv, y[u][3] * r * inv) << 16;
                w.y = pack_e4m3x2(y[u][4] * r * inv, y[u][5] * r * inv) | pack_e4m3x2(y[u][6] * r * inv, y[u][7] * r * inv) << 16;
                reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.y) + row * a.ys)[v] = w;
            }
        }
        row = next;
    }
}

template <int VPT, bool FP16, int SCALES>
cudaError_t run(const RmsNormArgs& a, int threads, cudaStream_t st) {
    // enough CTAs to fill the registers; more only wait their turn
    const int per_sm = threads >= 512 ? 2 : threads >= 256 ? 4 : threads >= 128 ? 6 : 1024 / threads;
    const int64_t grid = a.rows < kSms * per_sm ? a.rows : kSms * per_sm;
    residual_rmsnorm_kernel<VPT, FP16, SCALES><<<static_cast<unsigned>(grid), threads, 0, st>>>(a);
    return cudaGetLastError();
}

template <int VPT, bool FP16>
cudaError_t run(const RmsNormArgs& a, h3a_scales scales, int threads, cudaStream_t st) {
    switch (scales) {
        case H3A_SCALES_ROW: return run<VPT, FP16, H3A_SCALES_ROW>(a, threads, st);
        case H3A_SCALES_GROUP: return run<VPT, FP16, H3A_SCALES_GROUP>(a, threads, st);
        default: return run<VPT, FP16, H3A_SCALES_NONE>(a, threads, st);
    }
}

template <int VPT>
cudaError_t run(const RmsNormArgs& a, bool fp16, h3a_scales scales, int threads, cudaStream_t st) {
    return fp16 ? run<VPT, true>(a, scales, threads, st) : run<VPT, false>(a, scales, threads, st);
}

}  // namespace

cudaError_t launch_residual_rmsnorm(const RmsNormArgs& a, bool fp16, h3a_scales scales, cudaStream_t st) {
    if (a.rows == 0) return cudaSuccess;
    const int nvec = a.width / 8;
    auto threads_of = [&](int vpt) { return ((nvec + vpt - 1) / vpt + 31) / 32 * 32; };
    // one warp a row up to 1,024 channels, else the fewest idle vector slots
    int vpt = 1;
    if (nvec <= 128) {
        vpt = (nvec + 31) / 32;
    } else {
        int best = 1 << 30;
        for (int c = 2; c <= 4; ++c) {
            if (threads_of(c) > 512) continue;
            const int idle = threads_of(c) * c - nvec;
            if (idle < best) best = idle, vpt = c;
        }
    }
    const int threads = threads_of(vpt);
    switch (vpt) {
        case 1: return run<1>(a, fp16, scales, threads, st);
        case 2: return run<2>(a, fp16, scales, threads, st);
        case 3: return run<3>(a, fp16, scales, threads, st);
        default: return run<4>(a, fp16, scales, threads, st);
    }
}

}  // namespace h3a
