// How an h3a_packed_attention call is carried out: which kernel, and into how
// many parts a sequence's keys are cut.  Host only; goes by the descriptor's
// sizes, so the workspace size follows from the descriptor alone.
#include <algorithm>
#include <cmath>

#include "prompt_internal.h"

#ifndef ONE_TILE_KEYS
#define ONE_TILE_KEYS -1
#endif
#ifndef JOINUS
#define JOINUS 3.0
#endif
namespace h3a {

cudaError_t allow_smem(const void* kernel, int bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}

int packed_queries_per_tile(int group) { return 128 / group; }

int64_t packed_tile_groups(int64_t total_q, int seqs, int group, int tiles) {
    return total_q / (tiles * packed_queries_per_tile(group)) + seqs;
}

namespace {

// Parts for the row kernel: what is estimated to end first.  Two CTAs a
// multiprocessor take 64 keys in about 0.4 us each, a CTA's beginning and end
// about 2 us; joining the parts is a second launch.
int64_t row_splits(const h3a_packed_desc& d, int64_t max_k) {
    const double base = static_cast<double>(d.seqs) * d.kv_heads, units = static_cast<double>((max_k + 63) / 64);
    int64_t best = 1;
    double least = 0;
    for (int64_t s = 1; s <= 256 && s <= units; s += s < 16 ? 1 : s / 8) {
        const double waves = std::max(1.0, base * s / (2 * kSms));
        const double us = waves * (std::ceil(units / s) * 0.4 + 2.0) + (s > 1 ? JOINUS + 0.03 * s : 0.0);
        if (s == 1 || us < 0.9 * least) {
            best = s;
            least = us;
        }
    }
    return best;
}

}  // namespace

PackedPlan packed_plan(const h3a_packed_desc& d) {
    PackedPlan p{};
    const int group = d.heads / d.kv_heads;
    const int64_t max_q = std::min(d.max_q, d.total_q), max_k = std::min(d.max_k, d.total_k);
    // Up to 16 rows (queries x heads of a group) fit one mma.m16n8k16 tile of
    // the row kernel, which then reads the keys once; more go to the 128-row
    // tiles of the tcgen05 kernel.
    // One tile a CTA for short sequences, two for long ones (us, one against two;
    // 16 prompts): 32/8 heads x 128 up to 300 keys 21.8 / 24.1, 700 51.6 / 53.1, 1,000
    // 77.9 / 76.8; 28/4 x 96 up to 700 40.3 / 41.1, 1,000 60.5 / 59.2; 16 x 64 up to
    // 2,000 87.9 / 98.3, but one prompt of 16,000 792 / 771.
    const int64_t one_tile = ONE_TILE_KEYS >= 0 ? ONE_TILE_KEYS : d.head_dim == 64 ? 4096 : 768;
    p.tiles = max_q * group <= 16 ? 0 : max_k <= one_tile ? 1 : 2;
    int64_t splits, chunk;
    if (p.tiles) {
        // a part for every multiprocessor without work, each of at least 512
        // keys (a part costs each of its rows an fp32 row written and read)
        const int64_t pairs = std::max<int64_t>(1, (d.total_q + 2 * packed_queries_per_tile(group) - 1) / (2 * packed_queries_per_tile(group)));
        const int64_t work = pairs * d.kv_heads;
        splits = std::min(kSms / std::max<int64_t>(work, 1), max_k / 512);
        splits = std::max<int64_t>(1, std::min<int64_t>(splits, 64));
        chunk = ((max_k + splits - 1) / splits + 127) / 128 * 128;
    } else {
        splits = row_splits(d, max_k);
        chunk = ((max_k + splits - 1) / splits + 63) / 64 * 64;
    }
    p.splits = static_cast<int>(std::max<int64_t>(1, splits));
    p.chunk = static_cast<int>(std::max<int64_t>(128, std::min<int64_t>(chunk, int64_t(1) << 30)));
    return p;
}

}  // namespace h3a
