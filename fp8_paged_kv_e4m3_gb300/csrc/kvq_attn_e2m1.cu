// kvq_attn_e2m1.cu -- attention over E2M1 pools: the choice of kernel, splits and
// merge, and the mma.sync kernel's instances at head_dim 128.
#include <cmath>

#include "kvq_attn_e2m1.cuh"

namespace kvq {

// whether a call runs on the tcgen05 kernel, which takes the same time for any number of rows up to 32.  Up to 16
// rows the mma.sync kernel is faster (32 x 8192: 51 us against 68; ragged 108 against 136), beyond them slower
// (32 rows: 89 us against 68; ragged 210 against 137).
static bool e2m1_uses_tc(int head_dim, int rows, bool topk) { return head_dim == 128 && rows > 16 && !topk; }

// The numbers of splits worth a look: those that fill k whole waves of `resident` CTAs, and `most`.
template <typename F>
static void e2m1_each_filling(int64_t pairs, int64_t resident, int32_t most, F f)
{
    for (int64_t k = 1; k <= 16; ++k) {
        const int64_t s = k * resident / pairs;
        if (s >= most) break;
        if (s >= 1) f(int32_t(s), k);
    }
    f(most, (pairs * most + resident - 1) / resident);
}

int32_t e2m1_splits(int head_dim, bool topk, int32_t batch, int32_t num_kv_heads, int rows, int32_t max_pages, int32_t most)
{
    const int64_t pairs = int64_t(batch) * num_kv_heads;
    int32_t best = most;
    if (e2m1_uses_tc(head_dim, rows, topk)) {
        // A CTA costs about 8 us beside 2 us per tile of 128 tokens (two CTAs per SM), which for full
        // sequences gives waves * (tiles / splits * 2 + 8); of the numbers within a tenth of the least, the
        // largest, which balances varied lengths best (64 sequences of 1K to 32K: 3, 4, 6 splits 138, 137, 145 us;
        // 32 x 8192: 2, 4, 6 splits 69, 75, 83 us).
        const int64_t resident = int64_t(device_sm_count()) * (rows <= 32 ? 2 : 1);
        const double tiles = (max_pages + 31) / 32;
        auto cost = [&](int32_t s, int64_t waves) { return double(waves) * (std::ceil(tiles / s) * 2.0 + 8.0); };
        double least = HUGE_VAL;
        e2m1_each_filling(pairs, resident, most, [&](int32_t s, int64_t w) { least = std::fmin(least, cost(s, w)); });
        e2m1_each_filling(pairs, resident, most, [&](int32_t s, int64_t w) {
            if (cost(s, w) <= 1.1 * least) best = s;
        });
        return best;
    }
    if (topk) return most;   // lists and whole contexts side by side: varied work again
    const int64_t resident = e2m1_resident(rows);
    auto score = [&](int32_t s, int64_t waves) { return double(pairs * s) / double(waves * resident) / (1.0 + 0.01 * s); };
    // Up to 8 splits balance a batch of varied lengths by their number, so that fewer (3/5 of them at least) have to
    // fill their waves better by a quarter.  128 pairs: 16 rows x 8192, 7 instead of 8, 53 -> 51 us (contexts of 410 to
    // 8192 35 -> 31); 8 rows x 6000, 4 instead of 6, 32 -> 28 us (300 to 6000 16.7 -> 17.5).
    const int32_t fewest = most > 8 ? (most / 4 > 8 ? most / 4 : 8) : (3 * most + 4) / 5;
    double least = most > 8 ? 0.0 : 1.25 * score(most, (pairs * most + resident - 1) / resident);
    e2m1_each_filling(pairs, resident, most, [&](int32_t s, int64_t waves) {
        if (s >= fewest && score(s, waves) > least) {
            least = score(s, waves);
            best = s;
        }
    });
    return best;
}

cudaError_t launch_attention_e2m1(int head_dim, AttnArgs a, cudaStream_t stream, bool *merged)
{
    *merged = false;
    if (a.batch == 0) return cudaSuccess;
    if (e2m1_uses_tc(head_dim, a.rows, a.topk_idx != nullptr)) return launch_attention_e2m1_tc(a, stream);
    const int64_t ctas = int64_t(a.batch) * a.num_kv_heads * a.num_splits;
    // On a grid of several waves the sequences come longest first, so that the short ones fill its end
    // (B 64, 1K to 32K: 102 -> 85 us, with 16 rows 138 -> 110).  Every CTA classifies the lengths first, which
    // costs more than it brings where a sequence is in many pieces already (B 4 x 262144, 76 splits: 91 -> 101 us).
    a.longest_first = a.batch > 1 && a.num_splits <= 16 && ctas > e2m1_resident(a.rows);
    // Up to 8 splits are merged by their cluster, while the grid is resident at once: a CTA then waits
    // at its end for the other splits of its (sequence, kv head), which finish at about the same time,
    // instead of a second kernel that waits for all (B 32 x 4096: 21.8 -> 20.4 us).  On a grid of several
    // waves it would hold a slot that the next wave needs (B 32 x 8192, 32 rows: 91 -> 106 us).
    *merged = a.out && !a.topk_idx && a.num_splits <= 8 && ctas <= e2m1_resident(a.rows);
    return head_dim == 128 ? launch_e2m1_dim<128>(a, *merged, stream) : launch_attention_e2m1_d64(a, *merged, stream);
}

}  // namespace kvq
