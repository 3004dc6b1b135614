// How an h3a_packed_attention call is carried out: which kernel, and into how
// many parts a sequence's keys are cut.  Host only; goes by the descriptor's
// sizes, so the workspace size follows from the descriptor alone.
#include <algorithm>
#include <cmath>

#include "prompt_internal.h"

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

// Parts for the tile kernel: what is estimated to end first.  With too few tiles
// for the GPU, parts put the other multiprocessors to work; every part costs its
// CTA a beginning and an end (about four 128-key steps), each of its rows an
// fp32 row written and read, and the call a second launch.
int64_t tile_splits(const h3a_packed_desc& d, int tiles, int64_t max_q, int64_t max_k) {
    const int group = d.heads / d.kv_heads, span = tiles * packed_queries_per_tile(group);
    const double slots = kSms * (tiles == 1 ? 2 : 1);
    // every sequence's last CTA is half full on average
    const double base = (static_cast<double>(d.total_q) / span + 0.5 * d.seqs) * d.kv_heads;
    const double steps = static_cast<double>((max_k + 127) / 128);
    // what a tile has to do on average: causal queries see what lies before them,
    // and of several sequences most are shorter than the longest
    double mean = d.causal && max_k > 0 ? steps * (1.0 - 0.5 * std::min(1.0, static_cast<double>(max_q) / max_k)) : steps;
    if (d.seqs > 1) mean *= 0.6;
    const double step_us = 1.8;
    const double rows_us = static_cast<double>(d.total_q) * d.heads * d.head_dim * 8 / 4e6;
    int64_t best = 1;
    double least = 0;
    for (int64_t s = 1; s <= 64 && (s == 1 || steps / s >= 2); ++s) {
        const double longest = std::ceil(steps / s) + 4, waves = base * s / slots;
        const double units = waves <= 1 ? longest : std::max(longest, waves * (mean / s + 4) + 0.25 * longest);
        const double us = units * step_us + (s > 1 ? 4 + rows_us * s : 0);
        // a clear gain only: the lengths are guessed, and tiles come in whole numbers
        if (s == 1 || us < (best == 1 ? 0.75 : 0.97) * least) {
            best = s;
            least = us;
        }
    }
    return best;
}

// Stretches that the row kernel's keys are cut into (packed_rows.cu), 0 for a CTA
// a sequence and kv head: where that would leave the GPU idle for longer than
// joining parts takes.
int row_streams(const h3a_packed_desc& d, int64_t max_k) {
    const double base = static_cast<double>(d.seqs) * d.kv_heads;
    const int slots = kSms * packed_rows_ctas(d.head_dim);
    const double blocks = static_cast<double>((max_k + 63) / 64);  // of the longest sequence
    // A CTA takes 64 keys in 0.006 us a channel, one of eight warps in 0.8 of it.
    // Around them 3 us, streamed 8 to 11 (the stretches to find, the second
    // launch, more ends with more sequences); ragged sequences are half as long as
    // the longest on average.  Measured (us, a CTA each against streamed): 8
    // sequences x 16 heads x 64 up to 900 keys 7.6 / 11.8, 1 x 8 x 64 of 2,000 12.1 /
    // 8.0, 16 x 8 x 128 up to 700 10.8 / 12.6, up to 3,000 28.1 / 24.3, 1 x 8 x 128 of
    // 4,000 41.1 / 10.6.
    const double block_us = 0.006 * d.head_dim;
    const double few = packed_rows_few(d.head_dim, static_cast<int64_t>(base)) ? 0.8 : 1.0;
    const double whole = 3 + std::max(1.0, base / slots) * blocks * block_us * few;
    const double streamed = 8 + 3 * std::min(1.0, base / 64) + std::max(2.0, 0.5 * blocks * base / slots) * block_us;
    if (whole <= streamed) return 0;
    // one for each kv head: as many as fill one to three rounds of the GPU best
    int best = 1;
    double most = 0;
    for (int rounds = 1; rounds <= 3; ++rounds) {
        const int n = std::max(1, rounds * slots / d.kv_heads);
        const double used = static_cast<double>(n) * d.kv_heads / (std::ceil(static_cast<double>(n) * d.kv_heads / slots) * slots);
        if (used > most + 0.05) {
            best = n;
            most = used;
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
    // One tile a CTA for short sequences, two for long ones (us, one against two):
    // 64 prompts, 28/4 heads x 96, up to 250 keys 37.6 / 43.2; 24, 32/8 x 128, up to 300
    // 29.0 / 29.6; 16 up to 400 26.5 / 25.6, up to 700 47.5 / 43.4; 5, 16 x 128, up to
    // 350 12.4 / 10.1; 16 x 64: 8 up to 2,000 48.4 / 51.8, one of 6,000 112.7 / 114.9, one
    // of 16,000 792 / 771.  And one where no sequence's queries fill more: 16 pieces of
    // up to 8 tokens behind 4,000, 32/8 x 128, 42.4 / 50.3, 32 up to 16 behind 3,000, 28/4
    // x 96, 27.3 / 32.8.  The 320 keys come from head_dim 128; at 96, whose two-tile form has
    // a P buffer of its own, the figures above are all there is.
    const int64_t one_tile = d.head_dim == 64 ? 8192 : 320;
    const bool one = max_k <= one_tile || max_q <= packed_queries_per_tile(group);
    p.tiles = max_q * group <= kRowSlots ? 0 : one ? 1 : 2;
    int64_t splits = 1, chunk = max_k;
    if (p.tiles) {
        splits = tile_splits(d, p.tiles, max_q, max_k);
        chunk = ((max_k + splits - 1) / splits + 127) / 128 * 128;
    } else {
        p.streams = row_streams(d, max_k);
    }
    p.splits = static_cast<int>(splits);
    p.chunk = static_cast<int>(std::max<int64_t>(128, std::min<int64_t>(chunk, int64_t(1) << 30)));
    return p;
}

}  // namespace h3a
