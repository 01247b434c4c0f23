// The plan of a prefix_attn call, from its sizes alone: which kernel takes which
// rows and keys, the key splits, and the workspace that holds their partials.
// Host code without CUDA, so that every size can be checked without a GPU.
#pragma once

#include <cstddef>
#include <cstdint>

namespace qkvf {

constexpr int kPlanPage = 16;            // slots of a page
constexpr int kPaTile = 128;             // query rows of one tcgen05.mma tile
constexpr int kPaMaxSplits = 128;        // key splits of a tile, prefix and own keys each
constexpr int kPrKeys = 64, kPrPages = kPrKeys / kPlanPage;   // keys of a block of the rows kernel

// Keys of a block of the tile kernel
constexpr int pa_tile_keys(int head_dim) { return head_dim == 64 ? 128 : 64; }

struct PaPlan {
    int small, pre_rows, tiles, pair, own_tile, own_rows, own_tiles, sp, ss, sp_max, ss_max;
};

// What the tables have room for may be far more than the requests' keys: for
// the sake of the own keys, the prefix never takes more than this times its own
// shortest time (64 rows x 8 KV heads over 32K, up to 1K own keys, in tables of 32K:
// 56.5 us, and 247 without this bound).
constexpr double kPaWithin = 1.35;

// The split (1..most) that ends soonest when `units` row tiles times the
// splits run in waves of `workers`, each taking blocks / split steps and about
// `over` steps of start and end.
inline int pa_split(int64_t units, int64_t workers, int64_t blocks, int most, double over)
{
    int best = 1;
    double least = 1e300;
    for (int s = 1; s <= most; ++s) {
        const double cost = (double)((units * s + workers - 1) / workers) * ((double)((blocks + s - 1) / s) + over);
        if (cost < least * 0.999) {
            least = cost;
            best = s;
        }
    }
    return best;
}

// The same where `others` CTAs of other_blocks steps follow in the grid: they
// run on the workers that the prefix's last wave leaves, and behind it.  (8
// rows against 8 heads of 64 and 128K keys: 45.5 us; 54.5 with the prefix alone
// dealt to all workers and the own keys' 8 CTAs in a wave of their own.)
inline int pa_rows_split(int64_t units, int64_t workers, int64_t blocks, int most, int64_t others, int64_t other_blocks)
{
    const double over = 6.0, other = (double)other_blocks + over;
    const auto each = [&](int s) { return (double)((blocks + s - 1) / s) + over; };
    const auto waves = [&](int s) { return (units * s + workers - 1) / workers; };
    double shortest = 1e300;
    for (int s = 1; s <= most; ++s) shortest = waves(s) * each(s) < shortest ? waves(s) * each(s) : shortest;
    int best = 1;
    double least = 1e300;
    for (int s = 1; s <= most; ++s) {
        if (waves(s) * each(s) > kPaWithin * shortest) continue;
        const int64_t left = others - (int64_t)((double)(waves(s) * workers - units * s) * (each(s) < other ? 1.0 : each(s) / other));
        const double cost = waves(s) * each(s) + (left > 0 ? (double)((left + workers - 1) / workers) * other : 0.0);
        if (cost < least * 0.999) {
            least = cost;
            best = s;
        }
    }
    return best;
}

// Splits that some plan of this many row tiles may use (without any: one)
inline int pa_most(int64_t units, int64_t workers, int64_t blocks)
{
    if (units < 1) return 1;
    int64_t most = (2 * workers + units - 1) / units;
    if (most > blocks) most = blocks;
    if (most > kPaMaxSplits) most = kPaMaxSplits;
    return most < 1 ? 1 : (int)most;
}

// The tile kernel's split: its steps of `step` us each, the own keys' work
// (`rest`, SM microseconds) on the SMs it leaves free meanwhile and behind it,
// and `merge` us a split to write and join.  With 64 rows x 8 KV heads over 32K
// and up to 1K own keys each, 9 splits (144 CTAs) take 60.8 us and 7 (112) 59.7
// to 61.4; with 33 rows x 4 KV heads of 128 over 16K, 38 splits 30.5 and 18
// 26.1.
inline int pa_tile_split(int64_t units, int64_t blocks, int most, int sms, bool pair, double step, double rest, double merge)
{
    const auto ctas = [&](int s) { return pair ? units * s : (units * s + 1) / 2; };
    const auto tile = [&](int s) {
        return (double)((ctas(s) + sms - 1) / sms) * ((double)((blocks + s - 1) / s) * step + 5.0);
    };
    double shortest = 1e300;
    for (int s = 1; s <= most; ++s) shortest = tile(s) < shortest ? tile(s) : shortest;
    int best = 1;
    double least = 1e300;
    for (int s = 1; s <= most; ++s) {
        if (tile(s) > kPaWithin * shortest) continue;
        double left = rest - (ctas(s) < sms ? (double)(sms - ctas(s)) * tile(s) : 0.0);
        if (left < 0.0) left = 0.0;
        const double cost = tile(s) + left / sms + (rest > 0.0 ? 5.0 * left / rest : 0.0) + merge * s;
        if (cost < least * 0.999) {
            least = cost;
            best = s;
        }
    }
    return best;
}

inline PaPlan pa_plan(int num_reqs, int q_len, int q_heads, int nkv, int head_dim, int prefix_blocks, int max_blocks, int sms)
{
    const int group = q_heads / nkv;
    const int64_t all = (int64_t)num_reqs * q_len * group;   // rows of a KV head
    PaPlan pl;
    // The rows kernel takes the prefix too while its tensor work hides behind
    // the tile kernel's start: up to 4 MB of it a KV head and 32 MB in all, or
    // with one fragment of 16 rows at any length (there 14 us over 128K keys of
    // one head, and 18 in the tile kernel).  32 rows against 8 heads of 64: 6.3
    // us over 2K keys and 15.9 over 16K (tile kernel 9.3 and 17.6), but 26.3
    // over 32K and 44 over 64K (22 and 32).
    const int64_t wide_blocks = (int64_t)prefix_blocks * (head_dim / 64);
    pl.small = all <= 16 || (all <= 64 && wide_blocks <= 1024 && nkv * wide_blocks <= 8192);
    pl.pre_rows = all <= 16 ? 16 : 64;
    pl.tiles = (int)((all + kPaTile - 1) / kPaTile);
    pl.pair = !pl.small && pl.tiles > 1;
    // A request's own keys go to the tile kernel from more than half a tile of
    // rows and 512 keys on: 16 requests x 16 tokens x 64 heads of 64 over 4K keys
    // and up to 256 own 42.5 us in the rows kernel and 44.1 here, 1024 own 54.4
    // and 50.7, 4096 own 90 and 64.7; one request of 512 tokens over 8192 keys 281
    // and 110.  Half a tile or less stays with the rows kernel, although lengths
    // of 2K and more would be better off here (16 requests x 8 tokens, lengths of
    // half the table's width to all of it: 43.9 us and 34.7 at 4096, 77 and 53 at
    // 8192): short ones are not (16.3 and 18.6 at 600; 4 requests over a 4K prefix
    // 19.3 and 25.7), and the rule knows the table's width only, which serving
    // programs set by the longest request they take.
    const bool many = all > 64 && q_len * group > 64;
    pl.own_tile = many && max_blocks > 32;
    pl.own_rows = pl.own_tile ? kPaTile : q_len * group <= 16 ? 16 : 64;
    pl.own_tiles = (q_len * group + pl.own_rows - 1) / pl.own_rows;
    const bool wide = pl.own_rows == 64 || (pl.small && pl.pre_rows == 64);
    const int ctas = wide ? (head_dim == 64 ? 3 : 2) : (head_dim == 64 ? 4 : 3);   // of the rows kernel, per SM
    const int tile_pages = pa_tile_keys(head_dim) / kPlanPage;
    const int ppb = pl.small ? kPrPages : tile_pages, opb = pl.own_tile ? tile_pages : kPrPages;   // pages of a block
    const int64_t nb = (prefix_blocks + ppb - 1) / ppb, no = (max_blocks + opb - 1) / opb;
    const int64_t units = (int64_t)(pl.pair ? (pl.tiles + 1) / 2 : 1) * nkv;
    const int64_t workers = pl.small ? ctas * sms : pl.pair ? sms : 2 * sms;
    const int64_t own = (int64_t)num_reqs * nkv * pl.own_tiles, own_workers = pl.own_tile ? 2 * sms : ctas * sms;
    const int ss_most = pa_most(own, own_workers, no);
    pl.ss = pa_split(own, own_workers, no, ss_most, 6.0);
    pl.ss_max = ss_most;
    if (pl.own_tile) {   // (a narrower table may go to the rows kernel: one bound for both)
        const int64_t small = (int64_t)num_reqs * nkv * ((q_len * group + 63) / 64);
        const int m = pa_most(small, (head_dim == 64 ? 3 : 2) * (int64_t)sms, (max_blocks + kPrPages - 1) / kPrPages);
        if (m > pl.ss_max) pl.ss_max = m;
    }
    if (pl.small) {
        pl.sp = pa_rows_split(units, workers, nb, pa_most(units, workers, nb), max_blocks > 0 ? own * pl.ss : 0,
                              (no + pl.ss - 1) / pl.ss);
    } else {
        // an item's start and its blocks; two of the tile kernel's run side by side
        const double start = pl.own_tile ? 2.0 : 0.6;
        const double stage = pl.own_tile ? 0.3 : (pl.own_rows == 64 ? 2.5 : 1.0) * (head_dim == 64 ? 0.2 : 0.4);
        pl.sp = pa_tile_split(units, nb, pa_most(units, workers, nb), sms, pl.pair, head_dim == 64 ? 1.05 : 0.84,
                              max_blocks > 0 ? (double)own * pl.ss * start + (double)own * no * stage : 0.0,
                              (double)all * nkv * head_dim * 4 / 2e6);
    }
    // (up to 64 rows a narrower prefix may go to the other kernel: one bound for both)
    pl.sp_max = all <= 64 ? pa_most(nkv, 4 * (int64_t)sms, (prefix_blocks + kPrPages - 1) / kPrPages) : pa_most(units, workers, nb);
    return pl;
}

// Partials: (sp_max + ss_max) x rows of O, maximum and sum, in FP32.  The
// bounds grow with the tables' widths, so a workspace serves narrower ones.
inline size_t pa_workspace(const PaPlan &pl, int64_t rows, int head_dim)
{
    return (size_t)rows * (pl.sp_max + pl.ss_max) * (head_dim * 4 + 8) + 256;
}

}  // namespace qkvf
