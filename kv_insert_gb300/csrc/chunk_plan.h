// How a chunk_attn call's work is dealt: the requests' rows in blocks, every
// block's keys for every KV head, one line of work cut into equal parts.  Plain
// arithmetic, so that every batch can be checked without a GPU.
#pragma once

#include <cmath>
#include <cstdint>

#ifdef __CUDACC__
#define CH_HD __host__ __device__ __forceinline__
#else
#define CH_HD inline
#endif

namespace qkvf {

constexpr int kChKeys = 128;     // keys of a step
constexpr int kChRows = 256;     // rows (token, q head of the KV head) of a block: two tiles
constexpr int kChTile = 128;     // rows of one tile; a block of no more has one

// An item is one block of a request's rows against its keys, for one KV head.
// Its cost: the keys its last row sees, and kChOver keys' worth of start and
// end, in keys x q heads (so that a block's own 256 rows are 256 of them).  A
// block of one tile shares its keys between the two groups of warps that
// otherwise take a tile each: 3 of 4 of a whole block's cost a key.  (kChOver
// 448 / 576 / 704: 468 / 472 / 475 us for three prompts of up to 8192 tokens, 208 /
// 208 / 210 for chunks beside single tokens, 103 / 104 / 103 for 64 single tokens;
// 192, with a slower start of an item, a fifth more than the best.)
constexpr int kChOver = 448;
constexpr int kChWhole = 4, kChHalf = 3;

struct ChRequest {
    int row0, n, L;   // first token, new tokens (none: 0 or less), keys
};

// A place in the line of work: block b of request r for KV head g, from its key step k on
struct ChPos {
    int r, g, b, k;
};

// (A request's rows, n times the group, are at most 2^30.  What the warps of
// chunk_tile_kernel compute of an item is in 32 bits: a 64-bit division is a
// subroutine call, and those do not go with setmaxnreg.)
CH_HD int ch_blocks(int n, int group) { return n > 0 ? (n * group + kChRows - 1) / kChRows : 0; }

CH_HD int ch_rows(int n, int group, int b)   // of block b
{
    const int left = n * group - b * kChRows;
    return left < kChRows ? left : kChRows;
}

// Keys that a block's last row sees (none: 0), and the steps that hold them
CH_HD int ch_keys(const ChRequest &q, int group, int b)
{
    const int keys = q.L - q.n + (b * kChRows + ch_rows(q.n, group, b) - 1) / group + 1;
    return keys > 0 ? keys : 0;
}
CH_HD int ch_steps(int keys) { return (keys + kChKeys - 1) / kChKeys; }

// The first b blocks' cost (all of two tiles), and block b's
CH_HD int64_t ch_before(const ChRequest &q, int group, int b)
{
    const int64_t ctx = q.L > q.n ? q.L - q.n : 0, each = (int64_t)group * (kChOver + ctx);
    return kChWhole * (each * b + (int64_t)(kChRows / 2) * b * ((int64_t)b + 1));
}
CH_HD int64_t ch_cost(const ChRequest &q, int group, int b)
{
    const int64_t ctx = q.L > q.n ? q.L - q.n : 0;
    return (ch_rows(q.n, group, b) > kChTile ? kChWhole : kChHalf) *
           ((int64_t)group * (kChOver + ctx) + (int64_t)kChRows * ((int64_t)b + 1));
}

// A sum of costs.  A call's own are below 2^57; starts that go up and down, where
// the same tokens count again and again, stop at 2^61.
CH_HD int64_t ch_add(int64_t a, int64_t b)
{
    const int64_t most = int64_t(1) << 61;
    return a + b < most ? a + b : most;
}

// A request's cost for one KV head
CH_HD int64_t ch_request_cost(const ChRequest &q, int group)
{
    const int blocks = ch_blocks(q.n, group);
    return blocks ? ch_before(q, group, blocks - 1) + ch_cost(q, group, blocks - 1) : 0;
}

// The place `off` into a request's cost (0 <= off < nkv times that)
CH_HD ChPos ch_locate(const ChRequest &q, int group, int r, int64_t off)
{
    ChPos at;
    const int64_t per = ch_request_cost(q, group);
    const int last = ch_blocks(q.n, group) - 1;
    at.r = r;
    at.g = (int)(off / per);
    off -= at.g * per;
    if (off >= ch_before(q, group, last)) {
        at.b = last;
    } else {   // 128 b^2 + (each + 128) b = off / 4, then exactly
        const int64_t ctx = q.L > q.n ? q.L - q.n : 0;
        const float each = (float)((int64_t)group * (kChOver + ctx) + kChRows / 2), o = (float)(off / kChWhole);
        // (the root without the difference of two large numbers)
        at.b = (int)(2.f * o / (each + sqrtf(each * each + 4.f * (kChRows / 2) * o)));
        if (at.b > last - 1) at.b = last - 1;
        while (at.b > 0 && ch_before(q, group, at.b) > off) --at.b;
        while (at.b < last - 1 && ch_before(q, group, at.b + 1) <= off) ++at.b;
    }
    const int steps = ch_steps(ch_keys(q, group, at.b));
    at.k = (int)((off - ch_before(q, group, at.b)) * steps / ch_cost(q, group, at.b));
    return at;
}

// Where part c of `parts` of a line of cost `total` starts
CH_HD int64_t ch_part(int64_t total, int parts, int c)
{
    return total / parts * c + total % parts * c / parts;
}

CH_HD bool ch_same_item(const ChPos &a, const ChPos &b) { return a.r == b.r && a.g == b.g && a.b == b.b; }
CH_HD bool ch_reached(const ChPos &a, const ChPos &b)   // a at or behind b
{
    return a.r != b.r ? a.r > b.r : a.g != b.g ? a.g > b.g : a.b != b.b ? a.b > b.b : a.k >= b.k;
}

// Steps [k0, k1) of an item of `steps` (0 of 0: rows that see no key)
struct ChPiece {
    ChPos at;
    int k1, steps;
};

// The piece at `at` of request q, of what ends at `end`; false: no part of the
// item is left there.  Moves `at` to the next item, of request r + 1 at g = b =
// k = 0 after the request's last.
CH_HD bool ch_take(const ChRequest &q, int group, int nkv, ChPos &at, const ChPos &end, ChPiece &piece)
{
    piece.at = at;
    piece.steps = ch_steps(ch_keys(q, group, at.b));
    const bool ends = ch_same_item(at, end);
    piece.k1 = ends ? end.k : piece.steps;
    if (ends) {
        at = end;
    } else {
        at.k = 0;
        if (++at.b == ch_blocks(q.n, group)) {
            at.b = 0;
            if (++at.g == nkv) {
                at.g = 0;
                ++at.r;
            }
        }
    }
    return piece.k1 > piece.at.k || (piece.steps == 0 && !ends);
}

// ---- key_weights: blocks of keys against the rows that see them ---------------

constexpr int kKwKeys = 256;   // keys of a block: two tensor-memory tiles

// A request's tokens that count (the last n) and its keys; `tokens` of a step.
// Block b's keys are seen by tokens from L - 256 b or n from the end on; it costs
// those, and `over` tokens' worth of loading the keys.
CH_HD int kw_blocks(const ChRequest &q) { return (int)(((int64_t)q.L + kKwKeys - 1) / kKwKeys); }
CH_HD int kw_seen(const ChRequest &q, int b) { return q.n < q.L - b * kKwKeys ? q.n : q.L - b * kKwKeys; }
CH_HD int kw_steps(const ChRequest &q, int b, int tokens) { return (kw_seen(q, b) + tokens - 1) / tokens; }

CH_HD int64_t kw_before(const ChRequest &q, int b, int over)   // the first b blocks' cost
{
    const int64_t flat = q.L > q.n ? (q.L - q.n) / kKwKeys + 1 : 1;   // blocks that all n see
    const int64_t f = b < flat ? b : flat, m = b - f;
    const int64_t ends = (int64_t)q.L * m - kKwKeys / 2 * ((int64_t)b * (b - 1) - f * (f - 1));
    return (int64_t)over * b + (q.n < q.L ? q.n : q.L) * f + (m > 0 ? ends : 0);
}
CH_HD int64_t kw_cost(const ChRequest &q, int b, int over) { return (int64_t)over + kw_seen(q, b); }
CH_HD int64_t kw_request_cost(const ChRequest &q, int over) { return q.n < 0 || q.L <= 0 ? 0 : kw_before(q, kw_blocks(q), over); }

CH_HD ChPos kw_locate(const ChRequest &q, int r, int64_t off, int tokens, int over)
{
    ChPos at;
    const int64_t per = kw_request_cost(q, over);
    const int last = kw_blocks(q) - 1;
    at.r = r;
    at.g = (int)(off / per);
    off -= at.g * per;
    // bisection: 25 steps at most
    int lo = 0, hi = last;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (kw_before(q, mid, over) <= off) lo = mid;
        else hi = mid - 1;
    }
    at.b = lo;
    at.k = (int)((off - kw_before(q, at.b, over)) * kw_steps(q, at.b, tokens) / kw_cost(q, at.b, over));
    return at;
}

// As ch_take, of one request's blocks of keys
CH_HD bool kw_take(const ChRequest &q, int tokens, int nkv, ChPos &at, const ChPos &end, ChPiece &piece)
{
    piece.at = at;
    piece.steps = kw_steps(q, at.b, tokens);
    const bool ends = ch_same_item(at, end);
    piece.k1 = ends ? end.k : piece.steps;
    if (ends) {
        at = end;
    } else {
        at.k = 0;
        if (++at.b == kw_blocks(q)) {
            at.b = 0;
            if (++at.g == nkv) {
                at.g = 0;
                ++at.r;
            }
        }
    }
    return piece.k1 > piece.at.k || (piece.steps == 0 && !ends);
}

}  // namespace qkvf
