// chunk_attn: attention of each request's new tokens over its paged keys
// (included by qkv_front.cu after norm_rope.cuh: one translation unit).
//
// Request r brings the rows starts[r] .. starts[r + 1] - 1 of q, n of them, and
// has L keys, its new tokens' among them.  Its token i sees keys j <= L - n + i:
//   s = scale q . k;  out = sum exp(s - m) v / sum exp(s - m);  lse = ln sum exp(s).
//
// chunk_tile_kernel, one CTA per SM.  A request's rows (token, q head of a KV
// head) are cut into blocks of 256, two tensor-memory tiles, each the work of a
// group of four softmax warps (a thread per row) and an MMA warp; both tiles
// take the same keys, 128 a step, from one ring that two producer warps fill, one
// with K and one with V (TMA, a swizzled box of every page each).  The producer of
// K also hands the CTA's items out.  A block of 128 rows or
// fewer (decode) is one tile whose even steps are the first group's and whose
// odd ones the second's, joined at its end.  Lengths are on the device:
// chunk_plan_kernel, one CTA, adds the requests' costs up and cuts the line of
// work into equal parts (chunk_plan.h), a CTA's each, which start and end in the
// middle of a block's keys too.  A block that several CTAs share leaves partials (m, sum exp(s - m),
// sum exp(s - m) v) in the workspace, at most two a CTA, and chunk_merge_kernel
// joins them in order.
//
// S = Q K^T goes to tensor memory and the weights back over it, as the A operand
// of O += P V.  With heads of 64 the weights take the outer half of S's columns
// and the next S the other ones, made meanwhile; with heads of 128 S, O and the
// weights fill tensor memory, and the next S follows the product.
//
// The producer of V looks at it before its product where a step ends behind the
// keys or holds keys that not every row of the block sees: slots behind the keys
// become 0, and so do infinities and NaN among the others (0 x infinity is not
// 0), which are added at the block's end for the rows that see them.
//
// What bounds it: for long rows the step of 256 x 128 (3,100 to 3,600 clocks with
// heads of 128, of them 2,048 of products, the rest softmax and hand-overs that
// do not overlap them): three prompts of up to 8192 tokens, 8 x 4 heads of 128,
// 468 us, 1.2 PFLOP/s.  For single tokens bytes: 64 requests of up to 4096 keys,
// 103 us, 5.6 TB/s.  A CTA's warps run six programs: their code has to stay in
// the instruction cache (157 KB to half, with the producers of K and V split in
// the same step: 667 to 595 us, 142 to 120).

#include "chunk_plan.h"

namespace qkvf {

constexpr int kChMaxTokens = 1 << 24;

struct RaggedParams {
    const void *q;
    const void *kv_cache;
    const int32_t *starts, *block_table, *context_lens;
    void *out;
    float *lse;             // chunk_attn: written; key_weights: read
    const float *weights;   // key_weights: [R][nkv][16 max_blocks]
    float *out_weights;
    int64_t num_pages;
    int64_t q_ts, q_hs;
    float *ws_o;            // chunk_attn: partial O [2 parts][256][D]
    float2 *ws_ml;          // (maximum in log2 units, sum; below 0: void) [2 parts][256]
    ChPos *ws_pos;          // [parts + 1]: where every part starts
    unsigned long long wait_limit_ns;
    int T, R, max_blocks, q_heads, nkv, group;
    int parts;
    int window;
    float decay;
    float scale_log2;
    int zero;
};

// Request r, n <= 0 where it has no rows or is left alone; flag: raise the
// status bit of a bad one
__device__ __forceinline__ ChRequest ragged_request(const RaggedParams &p, int b, int e, int L, bool flag)
{
    ChRequest q;
    q.row0 = b;
    q.n = e - b;
    q.L = L;
    const bool bad = b < 0 || e < b || e > p.T || L > p.max_blocks * kPageSlots;
    if (bad || L < 0) {
        if (bad && flag) atomicOr(&g_status, QKVF_STATUS_BAD_REQUEST);
        q.n = -1;
    }
    return q;
}
__device__ __forceinline__ ChRequest ragged_request(const RaggedParams &p, int r, bool flag)
{
    return ragged_request(p, p.starts[r], p.starts[r + 1], p.context_lens[r], flag);
}

// ---- shapes -----------------------------------------------------------------

constexpr int kChThreads = 384;   // 2 softmax groups of 4 warps, producers of K and of V, 2 MMA warps
constexpr int kChPages = kChKeys / kPageSlots;
constexpr int kChLooks = 8;       // barriers of looked-at V in turn: more than the ring holds steps
constexpr int kChItems = 4;       // items handed out and not done with
static_assert(kChTile == kPaTile, "tiles as in prefix_attn");

// A unit of the ring is K or V of one step
template <int D>
struct ChShape {
    static constexpr int nb = D / 64;                          // 64-column blocks of K or V
    static constexpr uint32_t page_bytes = kPageSlots * 2 * D; // one box
    static constexpr uint32_t unit_bytes = kChPages * page_bytes;
    static constexpr int units = D == 64 ? 12 : 5;
    static constexpr uint32_t q_bytes = kChTile * 2 * D;
    // tensor memory: a group's S and weights (three units of 64 columns, or S
    // alone with the weights over it), then both groups' O
    static constexpr bool over = D == 128;
    static constexpr uint32_t sp_cols = over ? kChKeys : 3 * kChKeys / 2;
    static constexpr uint32_t tO = 2 * sp_cols, cols = 512;
    static_assert(tO + 2 * D <= cols, "tensor memory");
};

// ---- the items of a part ------------------------------------------------------

// (Known to the compiler as one value a warp: what follows from such values stays
// in uniform registers, which the operands of products and copies need.)
__device__ __forceinline__ int ch_uniform(int x) { return __reduce_max_sync(0xffffffffu, x); }

// Steps of one block's keys, as the producer of K hands them to the other warps
struct ChItem {
    int r, g, b, k;          // request, KV head, block, first step
    int n;                   // steps here (0: rows that see no key; -1: the part's end)
    int of;                  // the block's steps in all
    int rows;                // of the block
    int keys, all;           // keys that some row sees, and that every row sees
    int row0, tokens, L;     // the request's
    int look_from, look0;    // V is looked at from that step on; look0 + step: which look it is
    int bad, dropped;        // a page outside the cache; values of V left out
    __device__ __forceinline__ bool single() const { return rows <= kChTile; }
    __device__ __forceinline__ bool mine(int step, int w) const { return !single() || (step & 1) == w; }
    __device__ __forceinline__ int pages(int step) const   // of a step, with keys
    {
        return min(kChPages, (keys + kPageSlots - 1) / kPageSlots - (k + step) * kChPages);
    }
    __device__ __forceinline__ bool whole() const { return n == of; }
};
static_assert(sizeof(ChItem) == 64, "four 16-byte words");

// The next item of a part (by one warp); looks: steps before it whose V is looked at
__device__ __forceinline__ ChItem ch_next(const RaggedParams &p, ChPos &at, const ChPos &end, int &looks)
{
    ChItem it = {};
    it.n = -1;
    while (!ch_reached(at, end)) {
        const ChRequest q = ragged_request(p, ch_uniform(p.starts[at.r]), ch_uniform(p.starts[at.r + 1]), ch_uniform(p.context_lens[at.r]), false);
        if (q.n <= 0) {
            at = {at.r + 1, 0, 0, 0};
            continue;
        }
        ChPiece piece;
        if (!ch_take(q, p.group, p.nkv, at, end, piece)) continue;
        it.r = piece.at.r;
        it.g = piece.at.g;
        it.b = piece.at.b;
        it.k = piece.at.k;
        it.n = piece.k1 - piece.at.k;
        it.of = piece.steps;
        it.rows = ch_rows(q.n, p.group, it.b);
        it.keys = ch_keys(q, p.group, it.b);
        it.all = q.L - q.n + it.b * kChRows / p.group + 1;
        it.row0 = q.row0;
        it.tokens = q.n;
        it.L = q.L;
        // a step's V is looked at if it ends behind the keys, or some rows do not see all of it
        it.look_from = max(0, min(it.n, max(min(it.all, it.keys), 0) / kChKeys - it.k));
        it.look0 = looks - it.look_from;
        looks += it.n - it.look_from;
        break;
    }
    return it;
}

struct ChSmem {   // offsets from the 1024-byte aligned base
    uint32_t q, ring, full, empty, vready, qready, sfull, sfree, pready, pvdone, odone, drain, tmem, dead, ifull, iempty, items, join, total;
};

template <int D>
__host__ __device__ constexpr ChSmem ch_smem()
{
    using Sh = ChShape<D>;
    ChSmem L = {};
    uint32_t off = 0;
    L.q = off;
    off += 2 * Sh::q_bytes;
    L.ring = off;
    off += Sh::units * Sh::unit_bytes;
    L.full = off;
    off += Sh::units * 8;
    L.empty = off;
    off += Sh::units * 8;
    L.vready = off;
    off += kChLooks * 8;
    L.qready = off;
    off += 16;
    L.sfull = off;
    off += 16;
    L.sfree = off;
    off += 16;
    L.pready = off;   // [block % 2][group]
    off += 32;
    L.pvdone = off;
    off += 16;
    L.odone = off;
    off += 16;
    L.drain = off;
    off += 16;
    L.tmem = off;
    off += 8;
    L.dead = off;
    off += 8;
    L.ifull = off;
    off += kChItems * 8;
    L.iempty = off;
    off += kChItems * 8;
    off = (off + 15) / 16 * 16;
    L.items = off;
    off += kChItems * sizeof(ChItem);
    L.join = off;      // the second group's maxima and sums
    off += 8 * kChTile;
    L.total = off + 1024;
    return L;
}

__device__ __forceinline__ void ch_load_page(uint32_t dst, const CUtensorMap *m, uint32_t bar, int block, int c4)
{
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %3, %5, %3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(0), "r"(c4), "r"(block)
        : "memory");
}

// Tensor memory into registers.  The wait stands in the same statement as the
// loads: they write their registers behind the compiler's back, and what it put
// in between (a register spilled or moved) would take or lose a value.
#define CH_REGS16(a, i) PA_REGS8(a, i), PA_REGS8(a, i + 8)
#define CH_REGS64(a) CH_REGS16(a, 0), CH_REGS16(a, 16), CH_REGS16(a, 32), CH_REGS16(a, 48)

__device__ __forceinline__ void ch_load64(uint32_t addr, uint32_t (&a)[64])
{
    asm volatile(
        "{\n"
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32, %33, %34, %35, %36, %37, "
        "%38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, "
        "%60, %61, %62, %63}, [%64];\n"
        "tcgen05.wait::ld.sync.aligned;\n"
        "}\n"
        : CH_REGS64(a)
        : "r"(addr)
        : "memory");
}

__device__ __forceinline__ void ch_load16(uint32_t addr, uint32_t (&a)[16])
{
    asm volatile(
        "{\n"
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
        "[%16];\n"
        "tcgen05.wait::ld.sync.aligned;\n"
        "}\n"
        : CH_REGS16(a, 0)
        : "r"(addr)
        : "memory");
}

__device__ __forceinline__ void ch_load32(uint32_t addr, uint32_t (&a)[32])
{
    asm volatile(
        "{\n"
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
        "tcgen05.wait::ld.sync.aligned;\n"
        "}\n"
        : CH_REGS16(a, 0), CH_REGS16(a, 16)
        : "r"(addr)
        : "memory");
}

// pa_wait in few instructions: the kernel's code has to stay in the instruction
// cache (below)
__device__ __forceinline__ void ch_wait(uint32_t bar, uint32_t parity, volatile int *dead, unsigned long long limit_ns, bool honour)
{
    unsigned long long start = 0;
#pragma unroll 1
    while (!mbar_try_wait(bar, parity)) {
        const unsigned long long now = global_ns();
        if (start == 0) start = now;
        if (now - start > limit_ns) {
            *dead = 1;
            atomicOr(&g_status, QKVF_STATUS_WAIT_TIMEOUT);
            return;
        }
        if (honour && *dead) return;
    }
}

// 1 / x and log2 x on the special-function unit, within 2^-22: functions with
// a slow path are subroutine calls there
__device__ __forceinline__ float ch_rcp(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float ch_lg2(float x)
{
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Both softmax groups (named barrier 1)
__device__ __forceinline__ void ch_groups_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// V row of key j of a request; null: its page is outside the cache
template <int D>
__device__ __forceinline__ const uint16_t *ch_value_row(const RaggedParams &p, int r, int g, int j)
{
    const int page = p.block_table[(int64_t)r * p.max_blocks + j / kPageSlots];
    if (page < 0 || page >= p.num_pages) return nullptr;
    const int64_t slot = ((int64_t)page * p.nkv + g) * kPageSlots + j % kPageSlots;
    return static_cast<const uint16_t *>(p.kv_cache) + slot * (2 * D) + D;
}

template <class E, int D>
struct ChTile {
    using Sh = ChShape<D>;
    static constexpr int NU = Sh::units, U = kChKeys / 2;
    static constexpr ChSmem LY = ch_smem<D>();
    const CUtensorMap *map;
    const RaggedParams &p;
    uint8_t *smem;
    uint32_t sb;
    int lane;

    __device__ __forceinline__ volatile int *dead_flag() const { return reinterpret_cast<volatile int *>(smem + LY.dead); }
    __device__ __forceinline__ bool dead() const { return dead_flag()[0] != 0; }
    __device__ __forceinline__ void wait(uint32_t bar, int n) const   // until phase n of bar is complete
    {
        ch_wait(sb + bar, (uint32_t)n & 1, dead_flag(), p.wait_limit_ns, true);
    }
    // Item `seq`: its place, and by its values (at the part's end n is -1).  Items
    // come and go whether or not a wait gave up: every warp sees all of them.
    __device__ __forceinline__ ChItem *place(int seq) const { return reinterpret_cast<ChItem *>(smem + LY.items) + seq % kChItems; }
    __device__ __forceinline__ ChItem item(int seq) const
    {
        ch_wait(sb + LY.ifull + 8 * (seq % kChItems), (uint32_t)(seq / kChItems) & 1, dead_flag(), p.wait_limit_ns, false);
        __syncwarp();
        const int *x = reinterpret_cast<const int *>(place(seq));
        ChItem it = {};
        it.r = ch_uniform(x[0]);
        it.g = ch_uniform(x[1]);
        it.b = ch_uniform(x[2]);
        it.k = ch_uniform(x[3]);
        it.n = ch_uniform(x[4]);
        it.of = ch_uniform(x[5]);
        it.rows = ch_uniform(x[6]);
        it.keys = ch_uniform(x[7]);
        it.all = ch_uniform(x[8]);
        it.row0 = ch_uniform(x[9]);
        it.tokens = ch_uniform(x[10]);
        it.L = ch_uniform(x[11]);
        it.look_from = ch_uniform(x[12]);
        it.look0 = ch_uniform(x[13]);
        return it;
    }
    __device__ __forceinline__ void done(int seq) const   // this warp is, with item seq
    {
        __syncwarp();
        if (lane == 0) mbar_arrive(sb + LY.iempty + 8 * (seq % kChItems));
    }
    // V unit u of a step
    __device__ __forceinline__ void wait_value(const ChItem &it, int step, int u) const
    {
        if (step >= it.look_from) {
            const int n = it.look0 + step;
            wait(LY.vready + 8 * (n % kChLooks), n / kChLooks);
        } else {
            wait(LY.full + 8 * (u % NU), u / NU);
        }
    }
    __device__ __forceinline__ uint32_t unit(int u) const { return LY.ring + (u % NU) * Sh::unit_bytes; }

    // ---- produce: K (kV = 0) or V (1) of every step; K's warp hands out the
    // items, V's looks at V where that is due ----
    __device__ __forceinline__ void produce(int kV, ChPos at, const ChPos &end) const
    {
        if (lane == 0) tma_prefetch_map(map);
        int u = kV, looks = 0;
        bool ok = true, bad_any = false;
#pragma unroll 1
        for (int seq = 0;; ++seq) {
            ChItem it;
            if (kV) {
                it = item(seq);
                if (it.n > 0) fetch(it);
            } else {
                it = ch_next(p, at, end, looks);
                if (seq >= kChItems)
                    ch_wait(sb + LY.iempty + 8 * (seq % kChItems), (uint32_t)(seq / kChItems - 1) & 1, dead_flag(), p.wait_limit_ns, false);
                __syncwarp();
                if (lane == 0) {
                    *place(seq) = it;
                    mbar_arrive(sb + LY.ifull + 8 * (seq % kChItems));
                }
                __syncwarp();
            }
            if (it.n < 0) break;
            const int32_t *table = p.block_table + (int64_t)it.r * p.max_blocks;
            const int pg0 = it.k * kChPages, pg1 = min((it.k + it.n) * kChPages, (it.keys + kPageSlots - 1) / kPageSlots);
            int next = pg0 + lane < pg1 ? table[pg0 + lane] : 0;
#pragma unroll 1
            for (int c = pg0; c < pg1 && ok; c += 32) {
                int page = next;
                if (c + 32 + lane < pg1) next = table[c + 32 + lane];
                bool bad = false;
                if (c + lane < pg1 && (page < 0 || page >= p.num_pages)) {   // flagged, page 0 in its place
                    bad = true;
                    page = 0;
                }
                if (__any_sync(0xffffffffu, bad)) {   // seen by the softmax before the item's end
                    bad_any = true;
                    *reinterpret_cast<volatile int *>(&place(seq)->bad) = 1;
                    __syncwarp();
                }
                const int box = page * p.nkv + it.g;
#pragma unroll 1
                for (int s0 = c; s0 < min(c + 32, pg1); s0 += kChPages, u += 2) {
                    const int n = min(kChPages, pg1 - s0);
                    if (u >= NU) wait(LY.empty + 8 * (u % NU), u / NU - 1);
                    __syncwarp();
                    ok = !__any_sync(0xffffffffu, dead());
                    if (!ok) break;
                    const uint32_t bar = sb + LY.full + 8 * (u % NU), dst = sb + unit(u);
                    if (pa_elect()) mbar_expect_tx(bar, (uint32_t)n * Sh::page_bytes);
                    __syncwarp();
#pragma unroll 1
                    for (int i = 0; i < n; ++i) {   // page i: its box is lane s0 - c + i's
                        const int c4 = ch_uniform(lane == s0 - c + i ? box : INT_MIN);
                        if (pa_elect()) ch_load_page(dst + i * Sh::page_bytes, map, bar, kV * Sh::nb, c4);
                    }
                    __syncwarp();
                    const int step = (s0 - pg0) / kChPages;
                    if (kV && step >= it.look_from) {
                        wait(LY.full + 8 * (u % NU), u / NU);
                        __syncwarp();
                        if (look(it, step, smem + unit(u))) *reinterpret_cast<volatile int *>(&place(seq)->dropped) = 1;
                        __syncwarp();
                        if (lane == 0) mbar_arrive(sb + LY.vready + 8 * ((it.look0 + step) % kChLooks));
                    }
                }
            }
            if (kV) done(seq);
        }
        if (lane == 0) {
            if (bad_any) atomicOr(&g_status, QKVF_STATUS_BAD_REQUEST);
            if (dead())   // our copies land before the CTA leaves
                for (int k = max(kV, u - 2 * NU); k < u; k += 2)
                    if (k >= u - NU) ch_wait(sb + LY.full + 8 * (k % NU), (uint32_t)((k / NU) & 1), dead_flag(), p.wait_limit_ns, false);
        }
        __syncwarp();
    }
    // The item's rows of q into L2, some steps before they are loaded
    __device__ __forceinline__ void fetch(const ChItem &it) const
    {
#pragma unroll 1
        for (int i = lane; i < it.rows * Sh::nb; i += 32) {
            const int mr = it.b * kChRows + i / Sh::nb, tok = mr / p.group, head = it.g * p.group + mr - tok * p.group;
            const uint16_t *row = static_cast<const uint16_t *>(p.q) + ((int64_t)it.row0 + tok) * p.q_ts + head * p.q_hs;
            asm volatile("prefetch.global.L2 [%0];" ::"l"(row + i % Sh::nb * 64));
        }
    }
    // The V rows of a step: 0 behind the keys; not finite, among those that some
    // row does not see: 0, and true
    __device__ __forceinline__ bool look(const ChItem &it, int step, uint8_t *at) const
    {
        const int k0 = (it.k + step) * kChKeys, from = max(min(it.all, it.keys) - k0, 0), keys = min(it.keys - k0, kChKeys);
        const int to = (keys + kPageSlots - 1) / kPageSlots * kPageSlots;
        bool found = false, wrote = false;
#pragma unroll 2
        for (int c = from * (D / 8) + lane; c < to * (D / 8); c += 32) {
            const int key = c / (D / 8), ch = c % (D / 8);   // (a row's 16-byte chunks in any order)
            uint4 *x = reinterpret_cast<uint4 *>(at + (key >> 3) * (Sh::nb * 1024) + (ch / 8) * 1024 + (key & 7) * 128 + (ch & 7) * 16);
            const uint4 v = *x;
            uint4 m = make_uint4(~0u, ~0u, ~0u, ~0u);
            if (key < keys) {
                m = make_uint4(pa_not_finite<E>(v.x), pa_not_finite<E>(v.y), pa_not_finite<E>(v.z), pa_not_finite<E>(v.w));
                found |= (m.x | m.y | m.z | m.w) != 0;
            }
            if (m.x | m.y | m.z | m.w) {
                wrote = true;
                *x = make_uint4(v.x & ~m.x, v.y & ~m.y, v.z & ~m.z, v.w & ~m.w);
            }
        }
        if (__any_sync(0xffffffffu, wrote)) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        return __any_sync(0xffffffffu, found);
    }

    // ---- multiply: group w's S = Q K^T and O += P V ----
    __device__ __forceinline__ void multiply(int W) const
    {
        ChItem it;
        int u0 = 0, items = 0, blk = 0;   // units before the item; items and steps of this group
        const uint64_t qd = pa_desc(sb + LY.q + W * Sh::q_bytes, 16, 1024);
        const uint64_t kd0 = pa_desc(sb + LY.ring, 16, Sh::nb * 1024);
        const uint64_t vd0 = pa_desc(sb + LY.ring, 1024, Sh::nb * 1024);
        const uint32_t dSP = W * Sh::sp_cols, dO = Sh::tO + W * D;
        // S of the step whose K is unit u, the item's `nth` of this group
        const auto scores = [&](int u, int nth) {
            wait(LY.full + 8 * (u % NU), u / NU);
            // the columns S takes: the weights before (one, or two steps ago) are
            // multiplied (an item's end has waited for all of its products), and
            // the last S is read (over: the product's end says so too)
            if (Sh::over && nth > 0) wait(LY.pvdone + 8 * W, blk - 1);
            if (!Sh::over) {
                if (nth > 1) wait(LY.pvdone + 8 * W, blk - 2);
                if (blk > 0) wait(LY.sfree + 8 * W, blk - 1);
            }
            __syncwarp();
            tc_fence_after();
            const uint64_t kd = kd0 + (uint32_t)(u % NU) * (Sh::unit_bytes / 16);
            const uint32_t dS = dSP + (Sh::over ? 0 : (blk & 1) * U);
            if (pa_elect()) {
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
                    umma_bf16(dS, qd + (i / 4) * (kChTile * 8) + (i % 4) * 2, kd + (i / 4) * 64 + (i % 4) * 2,
                              pa_idesc<E>(kChKeys, false), i != 0);
                umma_commit(sb + LY.sfull + 8 * W);
                umma_commit(sb + LY.empty + 8 * (u % NU));
            }
            __syncwarp();
            ++blk;
        };
        const auto values = [&](int b, int step, uint32_t acc) {   // O += P V of this group's step b
            const int u = u0 + 2 * step + 1, pages = it.pages(step);
            wait_value(it, step, u);
            wait(LY.pready + 16 * (b & 1) + 8 * W, b >> 1);
            __syncwarp();
            tc_fence_after();
            const uint64_t vd = vd0 + (uint32_t)(u % NU) * (Sh::unit_bytes / 16);
            const uint32_t dP = dSP + (Sh::over ? 0 : (b & 1) * 2 * U);
            if (pa_elect()) {
#pragma unroll
                for (int i = 0; i < kChPages; ++i)
                    if (i < pages)
                        pa_umma_ts(dO, dP + 8 * i, vd + i * (Sh::page_bytes / 16), pa_idesc<E>(D, true), i > 0 ? 1u : acc);
                umma_commit(sb + LY.pvdone + 8 * W);
                umma_commit(sb + LY.empty + 8 * (u % NU));
            }
            __syncwarp();
        };
        // The other group's step: its units pass here too, in order, so that no
        // phase of a barrier is missed
        const auto pass = [&](int step) {
            const int u = u0 + 2 * step;
            wait(LY.full + 8 * (u % NU), u / NU);
            wait_value(it, step, u + 1);
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(sb + LY.empty + 8 * (u % NU));
                mbar_arrive(sb + LY.empty + 8 * ((u + 1) % NU));
            }
        };
#pragma unroll 1
        for (int seq = 0;; ++seq) {
            it = item(seq);
            if (it.n < 0) break;
            const int n = it.n;
            int before = -1, nth = 0;   // the step whose product is due
#pragma unroll 1
            for (int s = 0; s <= n; ++s) {   // (n: the last product)
                if (s < n && !it.mine(s, W)) {
                    pass(s);
                    continue;
                }
                if (s == n && nth == 0) break;   // no step was this group's
                if (nth == 0) wait(LY.qready + 8 * W, items++);
                if (!Sh::over && s < n) scores(u0 + 2 * s, nth);
                if (nth > 0) values(s < n && !Sh::over ? blk - 2 : blk - 1, before, nth > 1);
                if (Sh::over && s < n) scores(u0 + 2 * s, nth);
                before = s;
                ++nth;
            }
            if (nth > 0) {
                if (pa_elect()) umma_commit(sb + LY.odone + 8 * W);
                __syncwarp();
                if (lane == 0) mbar_arrive(sb + LY.odone + 8 * W);   // with the flags of bad pages and values left out
            }
            u0 += 2 * n;
            done(seq);
        }
        // every MMA of this warp is done before tensor memory is freed (the same
        // lane is elected each time: commits cover the MMAs of one thread)
        if (pa_elect()) umma_commit(sb + LY.drain + 8 * W);
        __syncwarp();
        if (lane == 0) ch_wait(sb + LY.drain + 8 * W, 0, dead_flag(), p.wait_limit_ns, false);
        __syncwarp();
    }

    // A warp's 32 rows of Q or the output in accesses of whole rows
    static constexpr int kRowsAtOnce = 32 / (D / 8), kRowTurns = 32 / kRowsAtOnce;
    // 16-byte chunk c of a row of a Q tile
    static __device__ __forceinline__ uint4 *chunk(uint8_t *tile, int row, int c)
    {
        return reinterpret_cast<uint4 *>(tile + (c / 8) * (kChTile * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4));
    }

    // ---- softmax: thread = row of group w's tile ----
    __device__ __forceinline__ void softmax(int w, int wq) const
    {
        const int row = 32 * wq + lane;
        const uint32_t lane_base = (uint32_t)(32 * wq) << 16;
        const uint32_t aSP = w * Sh::sp_cols + lane_base, aO = Sh::tO + w * D + lane_base;
        uint8_t *sq = smem + LY.q + w * Sh::q_bytes;
        int blk = 0, items = 0;
        const uint64_t cc = f2_pack(p.scale_log2, p.scale_log2);
#pragma unroll 1
        for (int seq = 0;; ++seq) {
            const ChItem it = item(seq);
            if (it.n < 0) break;
            const bool single = it.single();
            const int n = it.n, by = single ? 2 : 1, first = single ? w : 0;
            const int m = (single ? 0 : w * kChTile) + row;   // the thread's row of the block
            const bool active = 32 * wq + (single ? 0 : w * kChTile) < it.rows, valid = m < it.rows;
            const int mr = it.b * kChRows + m, tok = mr / p.group, head = it.g * p.group + mr - tok * p.group;
            const int64_t grow = ((int64_t)it.row0 + tok) * p.q_heads + head;   // output row
            const int limit = valid ? it.L - it.tokens + tok + 1 : 0;           // keys that the row sees
            if (n == 0) {   // rows that see no key
                if (valid && (!single || w == 0)) put_none(grow, true);
                done(seq);
                continue;
            }
            float mu = -INFINITY, l = 0.f;
            if (first < n) {
                if (active) {   // the previous item is done: its Q is no longer read
                    const uint16_t *src = valid ? static_cast<const uint16_t *>(p.q) + ((int64_t)it.row0 + tok) * p.q_ts + head * p.q_hs
                                                : nullptr;
#pragma unroll 4
                    for (int i = 0; i < kRowTurns; ++i) {   // whole rows: few lines an access
                        const int r = i * kRowsAtOnce + lane / (D / 8), c = lane % (D / 8);
                        const uint16_t *x = reinterpret_cast<const uint16_t *>(__shfl_sync(0xffffffffu, (unsigned long long)src, r));
                        // (all of them on their way at once; zeros for a row of none)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(chunk(sq, 32 * wq + r, c))),
                                     "l"(x ? x + c * 8 : static_cast<const uint16_t *>(p.q)), "r"(x ? 16 : 0)
                                     : "memory");
                    }
                    asm volatile("cp.async.wait_all;" ::: "memory");
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                }
                mbar_arrive(sb + LY.qready + 8 * w);
                const auto arrive = [&](uint32_t bar) {   // for this warp, which has left tensor memory
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(sb + bar);
                };
                // (two barriers in turn: S of step b says that the weights of step
                // b - 2 have been multiplied, so that phase has been seen)
                const auto pready = [&](int b) { return LY.pready + 16 * (b & 1) + 8 * w; };
                // The weights of a step, against the maximum so far.  Later scores may
                // exceed it as long as a step's weights stay below a limit in sum (so
                // no maximum is taken per step); otherwise it follows, O is rescaled
                // and the weights are formed again.  An item's first step starts there.
#pragma unroll 1
                for (int s = first; s < n; s += by, ++blk) {
                    wait(LY.sfull + 8 * w, blk);
                    __syncwarp();
                    if (active) {
                        tc_fence_after();
                        const int outer = Sh::over ? 0 : blk & 1;   // the half of the keys in S's outer unit
                        const uint32_t aOut = aSP + 2 * outer * U;
                        uint32_t so[U], sm[U], po[U / 2], pm[U / 2];
                        const int left = limit - (it.k + s) * kChKeys;   // keys of the step that the row sees
                        if (__any_sync(0xffffffffu, valid && left < kChKeys)) hide(aSP + (Sh::over ? 0 : outer * U), left);
                        bool follow = s == first;
                        float sum = INFINITY;
                        ch_load64(aSP + U, sm);
#pragma unroll 1
                        for (bool again = false;; again = true) {
                            ch_load64(aOut, so);   // (not overwritten yet)
                            if (!Sh::over && !again) arrive(LY.sfree + 8 * w);
                            if (follow) {
                                // (only this row's own scores move it, not a neighbour's)
                                const float top = fmaf(pa_max(so, pa_max(sm, -INFINITY)), p.scale_log2, -PaWeight<E>::below);
                                const bool grew = top > mu && !(sum < PaWeight<E>::most);
                                const float al = grew ? a2_ex2(mu - top) : 1.f;
                                if (grew) mu = top;
                                l *= al;
                                if (s != first) rescale(w, blk - 1, aO, al);
                            }
                            const float base = mu == -INFINITY ? 0.f : -mu;
                            sum = pa_weights<E>(so, po, cc, base);
                            sum += pa_weights<E>(sm, pm, cc, base);
                            if (follow || !__any_sync(0xffffffffu, !(sum < PaWeight<E>::most))) break;
                            follow = true;
                        }
                        l += sum;
                        pa_tmem_st<U / 2>(aOut + outer * (U / 2), po);
                        pa_tmem_st<U / 2>(aOut + (outer ^ 1) * (U / 2), pm);
                        pa_tmem_st_wait();
                    } else if (!Sh::over) {
                        arrive(LY.sfree + 8 * w);
                    }
                    arrive(pready(blk));
                }
                wait(LY.odone + 8 * w, items++);
                __syncwarp();
                tc_fence_after();
            }
            finish(it, seq, w, row, m, active, valid, grow, limit, mu, l, aO);
            tc_fence_before();
            done(seq);
        }
    }

    // The scores from column `left` on become -infinity, whatever their slots
    // hold (in a loop over tensor memory: steps that need it are few)
    __device__ __forceinline__ void hide(uint32_t aS, int left) const
    {
#pragma unroll 1
        for (int c = 0; c < kChKeys; c += 16) {
            uint32_t t[16];
            ch_load16(aS + c, t);
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (c + e >= left) t[e] = 0xff800000u;
            pa_tmem_st16(aS + c, t);
        }
        pa_tmem_st_wait();
    }

    // O times al, behind the product of step b
    __device__ __forceinline__ void rescale(int w, int b, uint32_t aO, float al) const
    {
        wait(LY.pvdone + 8 * w, b);
        __syncwarp();
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
            uint32_t o[16];
            ch_load16(aO + c, o);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * al);
            pa_tmem_st16(aO + c, o);
        }
    }

    // A row without keys, or of a skipped request
    __device__ __forceinline__ void put_none(int64_t grow, bool seen) const
    {
        uint4 *out = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.out) + grow * D);
#pragma unroll
        for (int c = 0; c < D / 8; ++c) out[c] = make_uint4(0u, 0u, 0u, 0u);
        if (seen && p.lse) p.lse[grow] = -INFINITY;
    }

    // The item's rows: joined if the groups shared them, then the output, or a partial
    __device__ __forceinline__ void finish(const ChItem &it, int seq, int w, int row, int m, bool active, bool valid, int64_t grow, int limit,
                                           float mu, float l, uint32_t aO) const
    {
        const bool joined = it.single() && it.n > 1;
        float4 *shared = reinterpret_cast<float4 *>(smem + LY.q);      // [D / 4][128]: the whole Q area, whose products are done
        float2 *shared_ml = reinterpret_cast<float2 *>(smem + LY.join);
        if (it.single() && w == 1) {
            if (!joined) return;
            ch_groups_sync();   // both groups' products are done
            if (active) {
                shared_ml[row] = make_float2(mu, l);
#pragma unroll 1
                for (int c = 0; c < D; c += 16) {
                    uint32_t o[16];
                    ch_load16(aO + c, o);
#pragma unroll
                    for (int e = 0; e < 16; e += 4)
                        shared[(c + e) / 4 * kChTile + row] = make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]),
                                                                         __uint_as_float(o[e + 2]), __uint_as_float(o[e + 3]));
                }
            }
            ch_groups_sync();   // written
            ch_groups_sync();   // and read
            return;
        }
        float al0 = 1.f, al1 = 0.f;
        if (joined) {
            ch_groups_sync();
            ch_groups_sync();
            if (active) {
                const float2 other = shared_ml[row];
                const float top = fmaxf(mu, other.x), base = top == -INFINITY ? 0.f : top;
                al0 = a2_ex2(mu - base);
                al1 = a2_ex2(other.x - base);
                l = l * al0 + other.y * al1;
                mu = top;
            }
        }
        uint8_t *sq = smem + LY.q + w * Sh::q_bytes;
        if (active && !__any_sync(0xffffffffu, dead())) {
            const volatile ChItem *flags = place(seq);
            const bool dropped = flags->dropped, bad = flags->bad;
            const bool whole = it.whole();
            const int part = 2 * blockIdx.x + (it.k == 0);
            float *po = p.ws_o + ((int64_t)part * kChRows + m) * D;
            const float inv = ch_rcp(l);   // (a sum of a row that sees a key is far above the subnormals)
            uint16_t *out = static_cast<uint16_t *>(p.out) + grow * D;
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
                uint32_t o[16];
                __syncwarp();
                ch_load16(aO + c, o);
                if (joined) {
#pragma unroll
                    for (int e = 0; e < 16; e += 4) {
                        const float4 y = shared[(c + e) / 4 * kChTile + row];
                        o[e] = __float_as_uint(fmaf(__uint_as_float(o[e]), al0, y.x * al1));
                        o[e + 1] = __float_as_uint(fmaf(__uint_as_float(o[e + 1]), al0, y.y * al1));
                        o[e + 2] = __float_as_uint(fmaf(__uint_as_float(o[e + 2]), al0, y.z * al1));
                        o[e + 3] = __float_as_uint(fmaf(__uint_as_float(o[e + 3]), al0, y.w * al1));
                    }
                }
                if (valid && !whole) {
#pragma unroll
                    for (int e = 0; e < 16; e += 4)
                        *reinterpret_cast<uint4 *>(po + c + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                } else if (valid && !bad) {
#pragma unroll
                    for (int e = 0; e < 16; e += 8) {
                        uint32_t y[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            y[i] = l == 0.f ? 0u : E::pack(__uint_as_float(o[e + 2 * i]) * inv, __uint_as_float(o[e + 2 * i + 1]) * inv);
                        uint4 *dst = joined ? reinterpret_cast<uint4 *>(out + c + e) : chunk(sq, row, (c + e) / 8);
                        *dst = make_uint4(y[0], y[1], y[2], y[3]);
                    }
                }
            }
            if (whole && !joined) {   // by way of the Q tile: whole rows an access
                __syncwarp();
                const unsigned long long mine = (unsigned long long)(valid && !bad ? out : nullptr);
#pragma unroll 4
                for (int i = 0; i < kRowTurns; ++i) {
                    const int r = i * kRowsAtOnce + lane / (D / 8), c = lane % (D / 8);
                    uint4 *y = reinterpret_cast<uint4 *>(__shfl_sync(0xffffffffu, mine, r));
                    if (y) y[c] = *chunk(sq, (row & ~31) + r, c);
                }
                __syncwarp();
            }
            if (dropped && valid && !bad) {   // what is not finite, to the rows that see it
                const int to = min(min(it.keys, (it.k + it.n) * kChKeys), limit);
#pragma unroll 1
                for (int key = max(it.all, it.k * kChKeys); key < to; ++key) {
                    const uint16_t *v = ch_value_row<D>(p, it.r, it.g, key);
#pragma unroll 1
                    for (int d = 0; v && d < D; ++d)
                        if (pa_not_finite<E>(v[d])) {
                            if (whole)
                                out[d] = E::put(E::get(out[d]) + E::get(v[d]));
                            else
                                po[d] += E::get(v[d]);
                        }
                }
            }
            if (valid && !whole)
                p.ws_ml[(int64_t)part * kChRows + m] = make_float2(mu, bad ? -1.f : l);
            else if (valid && bad && p.zero)
                put_none(grow, false);
            else if (valid && !bad && p.lse)
                p.lse[grow] = l == 0.f ? -INFINITY : (mu + ch_lg2(l)) * 0.6931471805599453f;
        }
        if (joined) ch_groups_sync();   // the Q area is the next item's
    }
};

// Where every part of the line of work starts: the requests' costs added up (a
// thread's run of requests each), then a part a thread.
constexpr int kChPlanThreads = 1024;

// cost(r, flag, request): request r's cost (flag: raise the status bit of a bad
// one) and what locate needs; locate(request, r, off): the place that far into it
template <class Cost, class Locate>
__device__ __forceinline__ void ch_plan(const RaggedParams &p, Cost cost, Locate locate)
{
    __shared__ int64_t before[kChPlanThreads + 1], warps[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (p.R + kChPlanThreads - 1) / kChPlanThreads, r0 = tid * per, r1 = min(p.R, r0 + per);
    ChRequest q;
    int64_t upto = 0;
    for (int r = r0; r < r1; ++r) upto = ch_add(upto, cost(r, true, q));
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto = ch_add(upto, y);
    }
    if (lane == 31) warps[warp] = upto;
    __syncthreads();
    if (warp == 0) {
        int64_t v = warps[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v = ch_add(v, y);
        }
        warps[lane] = v;
    }
    __syncthreads();
    if (warp > 0) upto = ch_add(upto, warps[warp - 1]);
    before[tid + 1] = upto;
    if (tid == 0) before[0] = 0;
    __syncthreads();
    const int64_t total = before[kChPlanThreads];
    for (int c = tid; c <= p.parts; c += kChPlanThreads) {
        ChPos at = {p.R, 0, 0, 0};
        int64_t off = ch_part(total, p.parts, c);
        if (off < total) {
            int lo = 0, hi = kChPlanThreads - 1;   // the last thread whose run starts at or before it
            while (lo < hi) {
                const int mid = (lo + hi + 1) / 2;
                if (before[mid] <= off) lo = mid;
                else hi = mid - 1;
            }
            off -= before[lo];
            for (int r = lo * per; r < min(p.R, lo * per + per); ++r) {
                const int64_t own = cost(r, false, q);
                if (off < own) {
                    at = locate(q, r, off);
                    break;
                }
                off -= own;
            }
        }
        p.ws_pos[c] = at;
    }
}

__global__ void __launch_bounds__(kChPlanThreads) chunk_plan_kernel(const __grid_constant__ RaggedParams p)
{
    if (threadIdx.x == 0) griddep_launch_dependents();
    griddep_wait();
    const auto cost = [&](int r, bool flag, ChRequest &q) {
        q = ragged_request(p, r, flag);
        return p.nkv * ch_request_cost(q, p.group);
    };
    ch_plan(p, cost, [&](const ChRequest &q, int r, int64_t off) { return ch_locate(q, p.group, r, off); });
}

template <class E, int D>
__global__ void __launch_bounds__(kChThreads, 1)
    chunk_tile_kernel(const __grid_constant__ CUtensorMap tmKV, const __grid_constant__ RaggedParams p)
{
    using Sh = ChShape<D>;
    constexpr ChSmem LY = ch_smem<D>();
    extern __shared__ uint8_t ch_smem_dyn[];
    uint8_t *smem = ch_smem_dyn + ((1024u - (smem_u32(ch_smem_dyn) & 1023u)) & 1023u);
    const uint32_t sb = smem_u32(smem);
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) griddep_launch_dependents();
    griddep_wait();   // every input comes from the kernels before this one
    ChPos begin, end;   // (as in ChItem: one value a warp)
    {
        const int *x = reinterpret_cast<const int *>(p.ws_pos + blockIdx.x);
        begin = {ch_uniform(x[0]), ch_uniform(x[1]), ch_uniform(x[2]), ch_uniform(x[3])};
        end = {ch_uniform(x[4]), ch_uniform(x[5]), ch_uniform(x[6]), ch_uniform(x[7])};
    }
    if (ch_reached(begin, end)) return;   // no work is left for this part
    if (threadIdx.x == 0) {
        for (int i = 0; i < Sh::units; ++i) {
            mbar_init(sb + LY.full + 8 * i, 1);
            mbar_init(sb + LY.empty + 8 * i, 2);
        }
        for (int i = 0; i < kChLooks; ++i) mbar_init(sb + LY.vready + 8 * i, 1);
        for (int w = 0; w < 2; ++w) {
            mbar_init(sb + LY.qready + 8 * w, 128);
            mbar_init(sb + LY.sfull + 8 * w, 1);
            mbar_init(sb + LY.sfree + 8 * w, 4);
            mbar_init(sb + LY.pready + 8 * w, 4);
            mbar_init(sb + LY.pready + 16 + 8 * w, 4);
            mbar_init(sb + LY.pvdone + 8 * w, 1);
            mbar_init(sb + LY.odone + 8 * w, 2);
            mbar_init(sb + LY.drain + 8 * w, 1);
        }
        *reinterpret_cast<volatile int *>(smem + LY.dead) = 0;
        for (int i = 0; i < kChItems; ++i) {
            mbar_init(sb + LY.ifull + 8 * i, 1);
            mbar_init(sb + LY.iempty + 8 * i, 11);   // all warps but the one that hands them out
        }
        fence_barrier_init();
    }
    // all of tensor memory (one CTA per SM): it starts at column 0
    if (warp == 0) a2_tmem_alloc<Sh::cols>(sb + LY.tmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const ChTile<E, D> tile{&tmKV, p, smem, sb, lane};
    // a softmax thread holds a row's whole S: its groups take registers from the
    // other warpgroup (256 x 216 + 128 x 72 = 384 x 168, what the launch has)
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        tile.softmax(warp >> 2, warp & 3);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp < 10)
            tile.produce(ch_uniform(warp - 8), begin, end);
        else
            tile.multiply(ch_uniform(warp - 10));
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) a2_tmem_dealloc<Sh::cols>(0u);
}

// Joins the partials of the item that part blockIdx.x leaves to the next ones,
// a warp per row, the parts in order; and clears the rows of an output without
// earlier contents that no request has.
constexpr int kChMergeThreads = 256, kChMergeY = 8;   // 32 rows a CTA

template <class E, int D>
__global__ void __launch_bounds__(kChMergeThreads) chunk_merge_kernel(const __grid_constant__ RaggedParams p)
{
    if (threadIdx.x == 0) griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    using V = typename std::conditional<D == 128, float4, float2>::type;   // a lane's columns
    if (p.zero)
        for (int64_t t = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 8 + warp; t < p.T; t += (int64_t)gridDim.x * gridDim.y * 8) {
            int lo = 0, hi = p.R;   // the last request that starts at or before t
            while (lo < hi) {
                const int mid = (lo + hi + 1) / 2;
                if (p.starts[mid] <= t) lo = mid;
                else hi = mid - 1;
            }
            if (lo < p.R && p.starts[lo] <= t && t < p.starts[lo + 1] && ragged_request(p, lo, false).n > 0) continue;
            uint4 *out = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.out) + t * p.q_heads * D);
            for (int64_t i = lane; i < (int64_t)p.q_heads * D / 8; i += 32) out[i] = make_uint4(0u, 0u, 0u, 0u);
        }
    const int c = blockIdx.x;
    const ChPos here = p.ws_pos[c], next = p.ws_pos[c + 1];
    if (next.k == 0 || (ch_same_item(here, next) && here.k > 0)) return;   // none, or an earlier part's
    const ChRequest q = ragged_request(p, next.r, false);
    int last = c + 1;   // the part that ends it
    while (ch_same_item(p.ws_pos[last + 1], next)) ++last;
    const int rows = ch_rows(q.n, p.group, next.b);
    for (int m = blockIdx.y * 8 + warp; m < rows; m += gridDim.y * 8) {
        const auto slot = [&](int part) { return ((int64_t)2 * part + (part == c)) * kChRows + m; };
        float top = -INFINITY;
        bool bad = false;
        for (int i = c + lane; i <= last; i += 32) {   // (a part without a step of it left nothing)
            if (i > c && i < last && p.ws_pos[i].k == p.ws_pos[i + 1].k) continue;
            const float2 ml = p.ws_ml[slot(i)];
            bad |= ml.y < 0.f;
            top = fmaxf(top, ml.x);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        bad = __any_sync(0xffffffffu, bad);
        const int mr = next.b * kChRows + m, tok = mr / p.group;
        const int64_t grow = ((int64_t)q.row0 + tok) * p.q_heads + next.g * p.group + mr - tok * p.group;
        uint16_t *out = static_cast<uint16_t *>(p.out) + grow * D + lane * (D / 32);
        if (bad) {
            for (int e = 0; p.zero && e < D / 32; ++e) out[e] = 0;
            continue;
        }
        const float base = top == -INFINITY ? 0.f : top;
        float o[D / 32] = {}, l = 0.f;
#pragma unroll 4
        for (int i = c; i <= last; ++i) {
            if (i > c && i < last && p.ws_pos[i].k == p.ws_pos[i + 1].k) continue;
            const float2 ml = p.ws_ml[slot(i)];
            const V y = *reinterpret_cast<const V *>(p.ws_o + slot(i) * D + lane * (D / 32));
            const float al = a2_ex2(ml.x - base);
            if (ml.x == -INFINITY && ml.y == 0.f) continue;   // no key of it seen
            l = fmaf(ml.y, al, l);
            o[0] = fmaf(y.x, al, o[0]);
            o[1] = fmaf(y.y, al, o[1]);
            if constexpr (D == 128) {
                o[2] = fmaf(y.z, al, o[2]);
                o[3] = fmaf(y.w, al, o[3]);
            }
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int e = 0; e < D / 32; e += 2)
            *reinterpret_cast<uint32_t *>(out + e) = l == 0.f ? 0u : E::pack(o[e] * inv, o[e + 1] * inv);
        if (p.lse && lane == 0) p.lse[grow] = l == 0.f ? -INFINITY : (base + log2f(l)) * 0.6931471805599453f;
    }
}

template <class E, int D>
bool prepare_chunk_kernel()
{
    static_assert(ch_smem<D>().total <= (uint32_t)kMaxSmemPerCta, "shared memory");
    return cudaFuncSetAttribute((const void *)chunk_tile_kernel<E, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)ch_smem<D>().total) == cudaSuccess;
}

bool prepare_chunk_kernels()
{
    return prepare_chunk_kernel<Bf16, 64>() && prepare_chunk_kernel<Bf16, 128>() && prepare_chunk_kernel<Fp16, 64>() &&
           prepare_chunk_kernel<Fp16, 128>();
}

// The cache as in encode_prefix_map, in boxes of K or V of one page of one KV
// head: 8-slot groups of its 64-column blocks, 1 KB each
int encode_chunk_map(const void *kv_cache, int64_t num_pages, int nkv, int head_dim, bool bf16, CUtensorMap *m)
{
    const cuuint64_t slot = (cuuint64_t)head_dim * 4;   // bytes of a slot
    const cuuint64_t dims[5] = {64, 8, (cuuint64_t)head_dim / 32, 2, (cuuint64_t)num_pages * nkv};
    const cuuint64_t strides[4] = {slot, 128, 8 * slot, kPageSlots * slot};
    const cuuint32_t box[5] = {64, 8, (cuuint32_t)head_dim / 64, 2, 1};
    const cuuint32_t es[5] = {1, 1, 1, 1, 1};
    return g_encode(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 5, (void *)kv_cache,
                    dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? QKVF_OK
               : QKVF_ERR_CUDA;
}

template <class E, int D>
int launch_chunk(const CUtensorMap &map, const RaggedParams &prm, void *stream)
{
    int rc = launch_pdl(chunk_plan_kernel, dim3(1), dim3(kChPlanThreads), 0, stream, prm);
    if (rc != QKVF_OK) return rc;
    rc = launch_pdl(chunk_tile_kernel<E, D>, dim3((unsigned)prm.parts), dim3(kChThreads), (size_t)ch_smem<D>().total,
                              stream, map, prm);
    if (rc != QKVF_OK) return rc;
    return launch_pdl(chunk_merge_kernel<E, D>, dim3((unsigned)prm.parts, kChMergeY), dim3(kChMergeThreads), 0, stream, prm);
}

// ---- host -------------------------------------------------------------------

const char *check_ragged_shape(int T, int num_reqs, int q_heads, int num_kv_heads, int head_dim, int max_blocks, int *code)
{
    *code = QKVF_ERR_TOKENS;
    if (num_reqs < 0 || num_reqs > kPaMaxRequests) return "num_reqs must be 0..65535";
    if (T < 0 || T > kChMaxTokens) return "T must be 0..2^24 tokens";
    *code = QKVF_ERR_LAYOUT;
    if (head_dim != 64 && head_dim != 128) return "head_dim must be 64 or 128";
    if (num_kv_heads < 1 || num_kv_heads > 64) return "num_kv_heads must be 1..64";
    if (q_heads < num_kv_heads || q_heads % num_kv_heads || q_heads / num_kv_heads > kPaMaxGroup)
        return "q_heads must be 1..64 times num_kv_heads";
    *code = QKVF_ERR_SIZES;
    if (max_blocks < 1 || max_blocks > (1 << 20)) return "max_blocks must be 1..2^20";
    if ((int64_t)T * q_heads > (int64_t(1) << 30)) return "T * q_heads must be <= 2^30";
    *code = QKVF_OK;
    return nullptr;
}

const char *check_ragged_args(const void *q, int64_t q_ts, int64_t q_hs, const void *kv_cache, int64_t num_pages,
                              const int32_t *starts, const int32_t *block_table, int max_blocks, const int32_t *context_lens,
                              int T, int num_reqs, int q_heads, int num_kv_heads, int head_dim, float scale, int dtype,
                              const void *workspace, int *code)
{
    dtype = dtype_of(dtype);
    if (const char *why = check_ragged_shape(T, num_reqs, q_heads, num_kv_heads, head_dim, max_blocks, code)) return why;
    *code = QKVF_ERR_LAYOUT;
    if (dtype != QKVF_DTYPE_BF16 && dtype != QKVF_DTYPE_FP16) return "dtype must be bf16 or fp16";
    if (!stride_ok(q_ts) || !stride_ok(q_hs) || q_ts % 8 || q_hs % 8)
        return "q's strides must be multiples of 8 elements, 0..2^36";
    *code = QKVF_ERR_SIZES;
    if (num_pages < 1 || num_pages > (int64_t(1) << 31) / num_kv_heads) return "num_pages * num_kv_heads must be 1..2^31";
    *code = QKVF_ERR_ARG;
    if (!(scale > 0.f) || !(scale <= 1e6f)) return "scale must be in (0, 1e6]";
    *code = QKVF_OK;
    if (num_reqs == 0 && T == 0) return nullptr;
    *code = QKVF_ERR_NULL;
    if ((T > 0 && !q) || !kv_cache || !starts || !workspace || (num_reqs > 0 && (!block_table || !context_lens)))
        return "a required pointer is NULL";
    *code = QKVF_ERR_ALIGN;
    if (!aligned(q, 16) || !aligned(kv_cache, 16)) return "q and kv_cache must be 16-byte aligned";
    if (!aligned(starts, 4) || !aligned(context_lens, 4) || !aligned(block_table, 4))
        return "the starts, tables and lengths must be 4-byte aligned";
    if (!aligned(workspace, 256)) return "the workspace must be 256-byte aligned";
    *code = QKVF_OK;
    return nullptr;
}

// Whether one of the outputs (and the workspace) overlaps an input or another of them
bool ragged_overlap(const RaggedParams &p, int head_dim, const void *const *outs, const size_t *sizes, int n, const void *in,
                    size_t in_bytes)
{
    const View vq = p.T > 0 ? view_of(p.q, p.T, p.q_ts, p.q_heads, p.q_hs, head_dim, 2) : View{};
    const void *parts[] = {vq.ptr, p.kv_cache, p.context_lens, p.block_table, p.starts, in};
    const size_t bytes[] = {vq.extent, (size_t)p.num_pages * p.nkv * kPageSlots * 2 * head_dim * 2, (size_t)p.R * 4,
                            (size_t)p.R * p.max_blocks * 4, (size_t)(p.R + 1) * 4, in_bytes};
    for (int o = 0; o < n; ++o) {
        if (!sizes[o]) continue;
        for (int i = 0; i < 6; ++i)
            if (bytes[i] && overlap(parts[i], bytes[i], outs[o], sizes[o])) return true;
        for (int i = 0; i < o; ++i)
            if (sizes[i] && overlap(outs[i], sizes[i], outs[o], sizes[o])) return true;
    }
    return false;
}

const char *check_chunk_args(const RaggedParams &p, int head_dim, float scale, int dtype, const void *workspace,
                             size_t workspace_bytes, int *code)
{
    if (const char *why = check_ragged_args(p.q, p.q_ts, p.q_hs, p.kv_cache, p.num_pages, p.starts, p.block_table,
                                            p.max_blocks, p.context_lens, p.T, p.R, p.q_heads, p.nkv, head_dim, scale,
                                            dtype, workspace, code))
        return why;
    if (p.R == 0 && p.T == 0) return nullptr;
    *code = QKVF_ERR_NULL;
    if (p.T > 0 && !p.out) return "a required pointer is NULL";
    *code = QKVF_ERR_ALIGN;
    if (!aligned(p.out, 16)) return "out must be 16-byte aligned";
    if (!aligned(p.lse, 4)) return "lse must be 4-byte aligned";
    *code = QKVF_ERR_ARG;
    const size_t rows = (size_t)p.T * p.q_heads;
    const void *outs[] = {p.out, p.lse, workspace};
    const size_t sizes[] = {rows * head_dim * 2, p.lse ? rows * 4 : 0, workspace_bytes};
    if (ragged_overlap(p, head_dim, outs, sizes, 3, nullptr, 0)) return "out, lse or the workspace overlaps another argument";
    *code = QKVF_OK;
    return nullptr;
}

RaggedParams ragged_params(const void *q, int64_t q_ts, int64_t q_hs, const void *kv_cache, int64_t num_pages,
                           const int32_t *starts, const int32_t *block_table, int max_blocks, const int32_t *context_lens,
                           int T, int num_reqs, int q_heads, int num_kv_heads, float scale, int dtype)
{
    RaggedParams p = {};
    p.q = q;
    p.q_ts = q_ts;
    p.q_hs = q_hs;
    p.kv_cache = kv_cache;
    p.num_pages = num_pages;
    p.starts = starts;
    p.block_table = block_table;
    p.max_blocks = max_blocks;
    p.context_lens = context_lens;
    p.T = T;
    p.R = num_reqs;
    p.q_heads = q_heads;
    p.nkv = num_kv_heads;
    p.group = num_kv_heads > 0 ? q_heads / num_kv_heads : 0;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.zero = zero_skipped(dtype);
    return p;
}

// Two partials a part, their maxima and sums, the parts' starts
size_t chunk_workspace(int head_dim, int sms)
{
    const size_t slots = (size_t)2 * sms;
    return slots * kChRows * (head_dim * 4 + 8) + ((size_t)(sms + 1) * sizeof(ChPos) + 255) / 256 * 256;
}

}  // namespace qkvf

extern "C" {

size_t chunk_attn_workspace_bytes(int T, int num_reqs, int q_heads, int num_kv_heads, int head_dim, int max_blocks)
{
    int code;
    if (qkvf::check_ragged_shape(T, num_reqs, q_heads, num_kv_heads, head_dim, max_blocks, &code)) return 0;
    qkvf::DeviceState *d;
    return qkvf::probe_device(&d) == QKVF_OK ? qkvf::chunk_workspace(head_dim, d->sms) : 0;
}

const char *chunk_attn_unsupported(const void *q, int64_t q_token_stride, int64_t q_head_stride, const void *kv_cache,
                                   int64_t num_pages, const int32_t *starts, const int32_t *block_table, int max_blocks,
                                   const int32_t *context_lens, int T, int num_reqs, int q_heads, int num_kv_heads,
                                   int head_dim, float scale, int dtype, void *out, float *lse, const void *workspace,
                                   size_t workspace_bytes)
{
    qkvf::RaggedParams prm = qkvf::ragged_params(q, q_token_stride, q_head_stride, kv_cache, num_pages, starts, block_table,
                                                 max_blocks, context_lens, T, num_reqs, q_heads, num_kv_heads, scale, dtype);
    prm.out = out;
    prm.lse = lse;
    int code;
    const char *why = qkvf::check_chunk_args(prm, head_dim, scale, dtype, workspace, workspace_bytes, &code);
    if (why) return why;
    qkvf::DeviceState *d;
    const int rc = qkvf::probe_device(&d);
    if (rc != QKVF_OK) return qkv_front_strerror(rc);
    return T > 0 && workspace_bytes < qkvf::chunk_workspace(head_dim, d->sms) ? "the workspace is too small" : nullptr;
}

int chunk_attn(const void *q, int64_t q_token_stride, int64_t q_head_stride, const void *kv_cache, int64_t num_pages,
               const int32_t *starts, const int32_t *block_table, int max_blocks, const int32_t *context_lens, int T,
               int num_reqs, int q_heads, int num_kv_heads, int head_dim, float scale, int dtype, void *out, float *lse,
               void *workspace, size_t workspace_bytes, void *stream)
{
    qkvf::RaggedParams prm = qkvf::ragged_params(q, q_token_stride, q_head_stride, kv_cache, num_pages, starts, block_table,
                                                 max_blocks, context_lens, T, num_reqs, q_heads, num_kv_heads, scale, dtype);
    prm.out = out;
    prm.lse = lse;
    int code;
    if (qkvf::check_chunk_args(prm, head_dim, scale, dtype, workspace, workspace_bytes, &code)) return code;
    if (T == 0) return QKVF_OK;
    qkvf::DeviceState *d;
    const int rc = qkvf::probe_device(&d);
    if (rc != QKVF_OK) return rc;
    if (workspace_bytes < qkvf::chunk_workspace(head_dim, d->sms)) return QKVF_ERR_SIZES;
    const bool bf16 = qkvf::dtype_of(dtype) == QKVF_DTYPE_BF16;
    CUtensorMap map;
    const int mrc = qkvf::encode_chunk_map(kv_cache, num_pages, num_kv_heads, head_dim, bf16, &map);
    if (mrc != QKVF_OK) return mrc;
    prm.wait_limit_ns = qkvf::g_wait_limit_ns;
    prm.parts = d->sms;
    prm.ws_o = static_cast<float *>(workspace);
    prm.ws_ml = reinterpret_cast<float2 *>(prm.ws_o + (size_t)2 * d->sms * qkvf::kChRows * head_dim);
    prm.ws_pos = reinterpret_cast<qkvf::ChPos *>(prm.ws_ml + (size_t)2 * d->sms * qkvf::kChRows);
    if (bf16)
        return head_dim == 64 ? qkvf::launch_chunk<qkvf::Bf16, 64>(map, prm, stream)
                              : qkvf::launch_chunk<qkvf::Bf16, 128>(map, prm, stream);
    return head_dim == 64 ? qkvf::launch_chunk<qkvf::Fp16, 64>(map, prm, stream)
                          : qkvf::launch_chunk<qkvf::Fp16, 128>(map, prm, stream);
}

int chunk_attn_packed(const int64_t *args, void *stream)
{
    if (!args) return QKVF_ERR_NULL;
    qkvf::Words w(args);
    const int mb = w.i(7), T = w.i(9), R = w.i(10), q_heads = w.i(11), nkv = w.i(12), dim = w.i(13), dtype = w.i(15);
    if (!w.ok) return QKVF_ERR_SIZES;
    return chunk_attn(w.p<void>(0), args[1], args[2], w.p<void>(3), args[4], w.p<int32_t>(5), w.p<int32_t>(6), mb,
                      w.p<int32_t>(8), T, R, q_heads, nkv, dim, (float)w.d(14), dtype, w.p<void>(16), w.p<float>(17),
                      w.p<void>(18), (size_t)args[19], stream);
}

}  // extern "C"
