// key_weights: the attention weight that each cached key received (included by
// qkv_front.cu after chunk_attn.cuh: one translation unit).
//
// With token i of a request's n (its last `window`, where that is given) seeing
// keys j <= L - n + i:
//   w[j] = decay w[j] + sum over those tokens and the KV head's q heads of exp(s - lse),  s = scale q . k.
//
// key_tile_kernel, one CTA per SM: blocks of 256 keys of one KV head, two tiles
// of 128 that stay in shared memory, against all rows that see them, up to 128 a
// step.  S is formed transposed (keys x rows, K as the first operand), so a
// thread's row of tensor memory is one key and its sum needs no other thread; the
// rows' lse are the same for all threads.  Work is dealt as in chunk_attn
// (chunk_plan.h): every CTA an equal part, a block of keys shared by several CTAs
// leaves sums in the workspace that key_merge_kernel adds in order.
//
// Rows arrive by TMA, as many whole tokens of the KV head's q heads as a step
// has room for; lse beside them.  Rows of a step that no token of the request
// has, and rows of lse -infinity, are not counted, whatever they hold.
//
// What bounds it: with many rows not the exponentials (29 % of their unit; half of
// them left out changes nothing) nor any other unit (issue 39 %, products 33 %),
// but most likely a thread's chain of load from tensor memory, wait and weights,
// with two computing warps a scheduler (64 tokens x 4 heads a KV head of 128, 2
// requests of up to 32K keys: 37 us; a choice row by row costs 7 more); with single
// tokens the 2,500 clocks of instructions that every role spends on a block (16
// requests of up to 8K keys, 8 x 8 heads of 64: 34 us, 2.4 TB/s of keys).  Plan
// and merge are 5 and 3 to 4 us of each.

namespace qkvf {

struct KeyParams {
    RaggedParams r;
    float *ws;       // sums [2 parts][256]
    int *ws_bad;     // [2 parts]: such a sum is void
    int tokens;      // of a step
    int rows;        // tokens * group
    int over;        // cost of a block of keys beside its rows, in tokens
};

constexpr int kKwThreads = 384;   // 2 groups of 4 warps, a tile each; producers of keys and of rows; the MMA warp
constexpr int kKwItems = 4;

template <int D>
struct KwShape {
    static constexpr int nb = D / 64;
    static constexpr uint32_t page_bytes = kPageSlots * 2 * D, tile_bytes = kChPages * page_bytes;
    static constexpr int tiles = D == 64 ? 8 : 4;       // ring of key tiles
    static constexpr uint32_t rows_bytes = kChTile * 2 * D;
    static constexpr int blocks = D == 64 ? 4 : 2;      // ring of steps' rows
};

struct KwItem {
    int r, g, b, k, n, of;       // as in ChItem (n 0: no rows; -1: the end)
    int row0, tokens, L;         // the request's tokens that count, its keys
    int first;                   // the block's first step's first token
    int bad, pad[5];
    __device__ __forceinline__ int keys(int tile) const { return min(kChTile, L - b * kKwKeys - tile * kChTile); }
};
static_assert(sizeof(KwItem) == 64, "four 16-byte words");

struct KwSmem {
    uint32_t keys, rows, lse, out, kfull, kempty, rfull, rempty, sfull, sfree, ifull, iempty, drain, tmem, dead, items, total;
};

template <int D>
__host__ __device__ constexpr KwSmem kw_smem()
{
    using Sh = KwShape<D>;
    KwSmem L = {};
    uint32_t off = 0;
    L.keys = off;
    off += Sh::tiles * Sh::tile_bytes;
    L.rows = off;
    off += Sh::blocks * Sh::rows_bytes;
    L.lse = off;
    off += Sh::blocks * kChTile * 4;
    L.out = off;     // whether a step has rows that are left out (lse -infinity)
    off += Sh::blocks * 4;
    L.kfull = off;
    off += Sh::tiles * 8;
    L.kempty = off;
    off += Sh::tiles * 8;
    L.rfull = off;
    off += Sh::blocks * 8;
    L.rempty = off;
    off += Sh::blocks * 8;
    L.sfull = off;   // [tile][step % 2]
    off += 32;
    L.sfree = off;
    off += 32;
    L.ifull = off;
    off += kKwItems * 8;
    L.iempty = off;
    off += kKwItems * 8;
    L.drain = off;
    off += 8;
    L.tmem = off;
    off += 8;
    L.dead = off;
    off += 16;
    L.items = off;
    off += kKwItems * sizeof(KwItem);
    L.total = off + 1024;
    return L;
}

// A request's tokens that count: n < 0 where it is left alone
__device__ __forceinline__ ChRequest kw_request(const RaggedParams &p, int b, int e, int L, bool flag)
{
    ChRequest q = ragged_request(p, b, e, L, flag);
    if (p.window > 0 && q.n > p.window) {
        q.row0 += q.n - p.window;
        q.n = p.window;
    }
    return q;
}

// (q: the request of number qr, kept from one item to the next)
__device__ __forceinline__ KwItem kw_next(const KeyParams &kp, ChPos &at, const ChPos &end, ChRequest &q, int &qr)
{
    const RaggedParams &p = kp.r;
    KwItem it = {};
    it.n = -1;
    while (!ch_reached(at, end)) {
        if (at.r != qr) {
            qr = at.r;
            q = kw_request(p, ch_uniform(p.starts[at.r]), ch_uniform(p.starts[at.r + 1]), ch_uniform(p.context_lens[at.r]), false);
        }
        if (q.n < 0 || q.L <= 0) {
            at = {at.r + 1, 0, 0, 0};
            continue;
        }
        ChPiece piece;
        if (!kw_take(q, kp.tokens, p.nkv, at, end, piece)) continue;
        it.r = piece.at.r;
        it.g = piece.at.g;
        it.b = piece.at.b;
        it.k = piece.at.k;
        it.n = piece.k1 - piece.at.k;
        it.of = piece.steps;
        it.row0 = q.row0;
        it.tokens = q.n;
        it.L = q.L;
        it.first = q.n - kw_seen(q, it.b);
        break;
    }
    return it;
}

__device__ __forceinline__ void kw_load_rows(uint32_t dst, const CUtensorMap *m, uint32_t bar, int block, int head, int token)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(0), "r"(block), "r"(head), "r"(token)
        : "memory");
}

// S^T = K Q^T: 128 keys x n rows
template <class E>
__device__ __forceinline__ uint32_t kw_idesc(int n)
{
    constexpr uint32_t fmt = E::is_bf16 ? 1u : 0u;
    return 1u << 4 | fmt << 7 | fmt << 10 | (uint32_t)(n >> 3) << 17 | (uint32_t)(kChTile >> 4) << 24;
}

template <class E, int D>
struct KwTile {
    using Sh = KwShape<D>;
    static constexpr KwSmem LY = kw_smem<D>();
    const CUtensorMap *key_map, *row_map;
    const KeyParams &kp;
    uint8_t *smem;
    uint32_t sb;
    int lane;

    __device__ __forceinline__ volatile int *dead_flag() const { return reinterpret_cast<volatile int *>(smem + LY.dead); }
    __device__ __forceinline__ bool dead() const { return dead_flag()[0] != 0; }
    __device__ __forceinline__ void wait(uint32_t bar, int n, bool honour = true) const   // until phase n of bar is complete
    {
        ch_wait(sb + bar, (uint32_t)n & 1, dead_flag(), kp.r.wait_limit_ns, honour);
    }
    __device__ __forceinline__ KwItem *place(int seq) const { return reinterpret_cast<KwItem *>(smem + LY.items) + seq % kKwItems; }
    __device__ __forceinline__ KwItem item(int seq) const
    {
        wait(LY.ifull + 8 * (seq % kKwItems), seq / kKwItems, false);
        __syncwarp();
        const int *x = reinterpret_cast<const int *>(place(seq));
        KwItem it = {};
        it.r = ch_uniform(x[0]);
        it.g = ch_uniform(x[1]);
        it.b = ch_uniform(x[2]);
        it.k = ch_uniform(x[3]);
        it.n = ch_uniform(x[4]);
        it.of = ch_uniform(x[5]);
        it.row0 = ch_uniform(x[6]);
        it.tokens = ch_uniform(x[7]);
        it.L = ch_uniform(x[8]);
        it.first = ch_uniform(x[9]);
        return it;
    }
    __device__ __forceinline__ void done(int seq) const
    {
        __syncwarp();
        if (lane == 0) mbar_arrive(sb + LY.iempty + 8 * (seq % kKwItems));
    }
    // The first token of an item's step
    __device__ __forceinline__ int token(const KwItem &it, int step) const { return it.first + (it.k + step) * kp.tokens; }

    // ---- the keys of every item, and the items ----
    // Hands item seq out and copies its keys; false at the end
    __device__ __forceinline__ bool copy(int seq, const KwItem &it, int pages, int page, int &t, bool &ok, bool &bad_any) const
    {
        const RaggedParams &p = kp.r;
        if (seq >= kKwItems) wait(LY.iempty + 8 * (seq % kKwItems), seq / kKwItems - 1, false);
        __syncwarp();
        if (lane == 0) {
            *place(seq) = it;
            mbar_arrive(sb + LY.ifull + 8 * (seq % kKwItems));
        }
        __syncwarp();
        if (it.n < 0) return false;
        bool bad = false;
        if (lane < pages && (page < 0 || page >= p.num_pages)) {   // flagged, page 0 in its place
            bad = true;
            page = 0;
        }
        if (__any_sync(0xffffffffu, bad)) {   // seen before the item's end
            bad_any = true;
            *reinterpret_cast<volatile int *>(&place(seq)->bad) = 1;
            __syncwarp();
        }
        const int box = page * p.nkv + it.g;
#pragma unroll 1
        for (int half = 0; half * kChPages < pages; ++half, ++t) {
            const int n = min(kChPages, pages - half * kChPages), st = t % Sh::tiles;
            if (ok && t >= Sh::tiles) wait(LY.kempty + 8 * st, t / Sh::tiles - 1);
            __syncwarp();
            ok = ok && !__any_sync(0xffffffffu, dead());
            if (!ok) break;
            const uint32_t bar = sb + LY.kfull + 8 * st;
            int c4[kChPages];   // (all of them first: one at a time each waits for the one before)
#pragma unroll
            for (int i = 0; i < kChPages; ++i) c4[i] = ch_uniform(lane == half * kChPages + i ? box : INT_MIN);
            if (pa_elect()) {
                mbar_expect_tx(bar, (uint32_t)n * Sh::page_bytes);
#pragma unroll
                for (int i = 0; i < kChPages; ++i)
                    if (i < n) ch_load_page(sb + LY.keys + st * Sh::tile_bytes + i * Sh::page_bytes, key_map, bar, 0, c4[i]);
            }
            __syncwarp();
        }
        return true;
    }

    __device__ __forceinline__ void produce_keys(ChPos at, const ChPos &end) const
    {
        const RaggedParams &p = kp.r;
        if (lane == 0) tma_prefetch_map(key_map);
        int t = 0;   // tiles so far
        bool ok = true, bad_any = false;
        // an item and its pages are looked up while the one before is copied
        // (a chain of two reads from memory, longer than the copy's issue)
        ChRequest q = {};
        int qr = -1, pages = 0, page = 0;
        KwItem it = {};
#pragma unroll 1
        for (int seq = -1;; ++seq) {
            const KwItem next = kw_next(kp, at, end, q, qr);
            const int pg0 = next.b * (kKwKeys / kPageSlots);
            const int next_pages = next.n > 0 ? min(2 * kChPages, (next.L + kPageSlots - 1) / kPageSlots - pg0) : 0;
            const int next_page = lane < next_pages ? p.block_table[(int64_t)next.r * p.max_blocks + pg0 + lane] : 0;
            if (seq >= 0 && !copy(seq, it, pages, page, t, ok, bad_any)) break;
            it = next;
            pages = next_pages;
            page = next_page;
        }
        if (lane == 0) {
            if (bad_any) atomicOr(&g_status, QKVF_STATUS_BAD_REQUEST);
            if (dead())   // our copies land before the CTA leaves
                for (int k = max(0, t - Sh::tiles); k < t; ++k) wait(LY.kfull + 8 * (k % Sh::tiles), k / Sh::tiles, false);
        }
        __syncwarp();
    }

    // ---- the rows of every step, and their lse ----
    __device__ __forceinline__ void produce_rows() const
    {
        const RaggedParams &p = kp.r;
        if (lane == 0 && p.T > 0) tma_prefetch_map(row_map);
        int s = 0;   // steps so far
        bool ok = true;
#pragma unroll 1
        for (int seq = 0;; ++seq) {
            const KwItem it = item(seq);
            if (it.n < 0) break;
#pragma unroll 1
            for (int i = 0; i < it.n; ++i, ++s) {
                const int st = s % Sh::blocks, t0 = token(it, i);
                float lse[kChTile / 32];
#pragma unroll
                for (int e = 0; e < kChTile / 32; ++e) {
                    const int m = 32 * e + lane, tok = t0 + m / p.group;
                    const bool in = m < kp.rows && tok < it.tokens;
                    lse[e] = in ? p.lse[((int64_t)it.row0 + tok) * p.q_heads + it.g * p.group + m % p.group] : -INFINITY;
                }
                if (ok && s >= Sh::blocks) wait(LY.rempty + 8 * st, s / Sh::blocks - 1);
                __syncwarp();
                ok = ok && !__any_sync(0xffffffffu, dead());
                if (!ok) break;
                const uint32_t bar = sb + LY.rfull + 8 * st;
                float *dst = reinterpret_cast<float *>(smem + LY.lse) + st * kChTile;
#pragma unroll
                for (int e = 0; e < kChTile / 32; ++e)   // a row that sees no key (-infinity) adds nothing to any
                    dst[32 * e + lane] = lse[e] == -INFINITY ? -INFINITY : -lse[e];
                bool out = false;   // (here: until now the loads were on their way)
#pragma unroll
                for (int e = 0; e < kChTile / 32; ++e) {
                    const int m = 32 * e + lane;
                    out |= lse[e] == -INFINITY && m < kp.rows && t0 + m / p.group < it.tokens;
                }
                out = __any_sync(0xffffffffu, out);
                if (lane == 0) reinterpret_cast<int *>(smem + LY.out)[st] = out;
                __syncwarp();
                if (lane == 0) mbar_arrive(bar);
                if (pa_elect()) {
                    mbar_expect_tx(bar, (uint32_t)(Sh::nb * 128 * kp.rows));
                    for (int c = 0; c < Sh::nb; ++c)
                        kw_load_rows(sb + LY.rows + st * Sh::rows_bytes + c * (kChTile * 128), row_map, bar, c, it.g * p.group, it.row0 + t0);
                }
                __syncwarp();
            }
            done(seq);
        }
        if (lane == 0 && dead())
            for (int k = max(0, s - Sh::blocks); k < s; ++k) wait(LY.rfull + 8 * (k % Sh::blocks), k / Sh::blocks, false);
        __syncwarp();
    }

    // ---- multiply ----
    __device__ __forceinline__ void multiply() const
    {
        const uint64_t kd0 = pa_desc(sb + LY.keys, 16, Sh::nb * 1024), rd0 = pa_desc(sb + LY.rows, 16, 1024);
        const uint32_t idesc = kw_idesc<E>((kp.rows + 15) / 16 * 16);
        int t = 0, s = 0, n0 = 0, n1 = 0;   // tiles and steps so far; S tiles of each half
#pragma unroll 1
        for (int seq = 0;; ++seq) {
            const KwItem it = item(seq);
            if (it.n < 0) break;
            if (it.n == 0) {
                done(seq);
                continue;
            }
            const int tiles = it.keys(1) > 0 ? 2 : 1;
#pragma unroll 1
            for (int i = 0; i < it.n; ++i, ++s) {
                wait(LY.rfull + 8 * (s % Sh::blocks), s / Sh::blocks);
                const uint64_t rd = rd0 + (uint32_t)(s % Sh::blocks) * (Sh::rows_bytes / 16);
#pragma unroll 1
                for (int h = 0; h < tiles; ++h) {
                    const int st = (t + h) % Sh::tiles, n = h ? n1++ : n0++;
                    if (i == 0) wait(LY.kfull + 8 * st, (t + h) / Sh::tiles);
                    if (n > 1) wait(LY.sfree + 16 * h + 8 * (n & 1), n / 2 - 1);
                    __syncwarp();
                    tc_fence_after();
                    const uint64_t kd = kd0 + (uint32_t)st * (Sh::tile_bytes / 16);
                    if (pa_elect()) {
#pragma unroll
                        for (int c = 0; c < D / 16; ++c)
                            umma_bf16((uint32_t)(2 * h + (n & 1)) * kChTile, kd + (c / 4) * 64 + (c % 4) * 2,
                                      rd + (c / 4) * (kChTile * 8) + (c % 4) * 2, idesc, c != 0);
                        umma_commit(sb + LY.sfull + 16 * h + 8 * (n & 1));
                        if (h == tiles - 1) umma_commit(sb + LY.rempty + 8 * (s % Sh::blocks));
                        if (i == it.n - 1) umma_commit(sb + LY.kempty + 8 * st);
                    }
                    __syncwarp();
                }
            }
            t += tiles;
            done(seq);
        }
        if (pa_elect()) umma_commit(sb + LY.drain);
        __syncwarp();
        if (lane == 0) wait(LY.drain, 0, false);
        __syncwarp();
    }

    // The weights of rows from c on, of one key: added up (all 32 of them, or of 16 those from..rows - 1: the
    // choice row by row costs more than the weights; out: and without those of lse -infinity, whose scores
    // may be NaN)
    template <bool all, bool out>
    __device__ __forceinline__ float weigh_rows(uint32_t aS, const float *lse, int c, int from, int rows, uint64_t scale2) const
    {
        const uint64_t log2e = f2_pack(1.4426950408889634f, 1.4426950408889634f);
        constexpr int count = all ? 32 : 16;
        uint32_t x[count];
        if constexpr (all)
            ch_load32(aS + c, x);
        else
            ch_load16(aS + c, x);
        uint64_t acc[2] = {0, 0};
#pragma unroll
        for (int e = 0; e < count; e += 4) {
            const float4 z = *reinterpret_cast<const float4 *>(lse + c + e);
            float y[4];
            // the difference first: near 0 the weight then has all of its bits
            f2_unpack(f2_mul(f2_fma(f2_pack(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), scale2, f2_pack(z.x, z.y)), log2e), y[0], y[1]);
            f2_unpack(f2_mul(f2_fma(f2_pack(__uint_as_float(x[e + 2]), __uint_as_float(x[e + 3])), scale2, f2_pack(z.z, z.w)), log2e), y[2], y[3]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                y[i] = a2_ex2(y[i]);
                if (!all && (c + e + i < from || c + e + i >= rows)) y[i] = 0.f;
                if (out && (i == 0 ? z.x : i == 1 ? z.y : i == 2 ? z.z : z.w) == -INFINITY) y[i] = 0.f;
            }
            acc[0] = f2_add(acc[0], f2_pack(y[0], y[1]));
            acc[1] = f2_add(acc[1], f2_pack(y[2], y[3]));
        }
        float a, b;
        f2_unpack(f2_add(acc[0], acc[1]), a, b);
        return a + b;
    }

    // ---- the weights: thread = key of half h's tile ----
    __device__ __forceinline__ void weigh(int h, int wq) const
    {
        const RaggedParams &p = kp.r;
        const int key = 32 * wq + lane;
        const uint32_t aS = (uint32_t)(2 * h) * kChTile + ((uint32_t)(32 * wq) << 16);
        const float scale = p.scale_log2 * 0.6931471805599453f;
        const uint64_t scale2 = f2_pack(scale, scale);
        int s = 0, n = 0;
#pragma unroll 1
        for (int seq = 0;; ++seq) {
            const KwItem it = item(seq);
            if (it.n < 0) break;
            const int keys = it.keys(h), j = it.b * kKwKeys + h * kChTile + key;   // the thread's key
            const int64_t place_of = ((int64_t)it.r * p.nkv + it.g) * p.max_blocks * kPageSlots + j;
            const bool whole = it.n == it.of && key < keys;
            // (on its way while the rows are weighed)
            const float held = p.decay != 0.f && whole ? p.weights[place_of] : 0.f;
            float total = 0.f;
#pragma unroll 1
            for (int i = 0; i < it.n; ++i, ++s) {
                wait(LY.rfull + 8 * (s % Sh::blocks), s / Sh::blocks);   // (every phase is seen: it gives the rows free too)
                __syncwarp();
                if (keys > 0) {
                    const int t0 = token(it, i), rows = min(kp.rows, (it.tokens - t0) * p.group);
                    // the first row that sees the key
                    const int from = (j - (it.L - it.tokens) - t0) * p.group;
                    const bool out = reinterpret_cast<const volatile int *>(smem + LY.out)[s % Sh::blocks] != 0;
                    const bool plain = !__any_sync(0xffffffffu, from > 0 || out);
                    const float *lse = reinterpret_cast<const float *>(smem + LY.lse) + (s % Sh::blocks) * kChTile;
                    wait(LY.sfull + 16 * h + 8 * (n & 1), n / 2);
                    __syncwarp();
                    tc_fence_after();
                    float sum = 0.f;
                    int c = 0;
#pragma unroll 1
                    for (; plain && c + 32 <= rows; c += 32)
                        sum += weigh_rows<true, false>(aS + (n & 1) * kChTile, lse, c, from, rows, scale2);
#pragma unroll 1
                    for (; !out && c < rows; c += 16)
                        sum += weigh_rows<false, false>(aS + (n & 1) * kChTile, lse, c, from, rows, scale2);
#pragma unroll 1
                    for (; c < rows; c += 16) sum += weigh_rows<false, true>(aS + (n & 1) * kChTile, lse, c, from, rows, scale2);
                    total += sum;
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(sb + LY.sfree + 16 * h + 8 * (n & 1));
                    ++n;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(sb + LY.rempty + 8 * (s % Sh::blocks));
            }
            if (!__any_sync(0xffffffffu, dead())) {
                const bool bad = reinterpret_cast<const volatile KwItem *>(place(seq))->bad;
                if (it.n < it.of) {   // a part of the rows
                    const int part = 2 * blockIdx.x + (it.k == 0);
                    kp.ws[(int64_t)part * kKwKeys + h * kChTile + key] = total;
                    if (h == 0 && key == 0) kp.ws_bad[part] = bad;
                } else if (key < keys && !bad) {
                    p.out_weights[place_of] = p.decay == 0.f ? total : fmaf(p.decay, held, total);
                }
            }
            done(seq);
        }
    }
};

template <class E, int D>
__global__ void __launch_bounds__(kKwThreads, 1)
    key_tile_kernel(const __grid_constant__ CUtensorMap keys, const __grid_constant__ CUtensorMap rows, const __grid_constant__ KeyParams kp)
{
    using Sh = KwShape<D>;
    constexpr KwSmem LY = kw_smem<D>();
    extern __shared__ uint8_t kw_smem_dyn[];
    uint8_t *smem = kw_smem_dyn + ((1024u - (smem_u32(kw_smem_dyn) & 1023u)) & 1023u);
    const uint32_t sb = smem_u32(smem);
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) griddep_launch_dependents();
    griddep_wait();   // every input comes from the kernels before this one
    ChPos begin, end;
    {
        const int *x = reinterpret_cast<const int *>(kp.r.ws_pos + blockIdx.x);
        begin = {ch_uniform(x[0]), ch_uniform(x[1]), ch_uniform(x[2]), ch_uniform(x[3])};
        end = {ch_uniform(x[4]), ch_uniform(x[5]), ch_uniform(x[6]), ch_uniform(x[7])};
    }
    if (ch_reached(begin, end)) return;   // no work is left for this part
    if (threadIdx.x == 0) {
        for (int i = 0; i < Sh::tiles; ++i) {
            mbar_init(sb + LY.kfull + 8 * i, 1);
            mbar_init(sb + LY.kempty + 8 * i, 1);
        }
        for (int i = 0; i < Sh::blocks; ++i) {
            mbar_init(sb + LY.rfull + 8 * i, 2);    // lse, and the rows' bytes
            mbar_init(sb + LY.rempty + 8 * i, 9);   // the products, and 8 warps done with lse
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(sb + LY.sfull + 8 * i, 1);
            mbar_init(sb + LY.sfree + 8 * i, 4);
        }
        for (int i = 0; i < kKwItems; ++i) {
            mbar_init(sb + LY.ifull + 8 * i, 1);
            mbar_init(sb + LY.iempty + 8 * i, 10);   // all working warps but the one that hands them out
        }
        mbar_init(sb + LY.drain, 1);
        *reinterpret_cast<volatile int *>(smem + LY.dead) = 0;
        fence_barrier_init();
    }
    if (warp == 0) a2_tmem_alloc<512>(sb + LY.tmem);   // all of it: it starts at column 0
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const KwTile<E, D> tile{&keys, &rows, kp, smem, sb, lane};
    if (warp < 8)
        tile.weigh(ch_uniform(warp >> 2), ch_uniform(warp & 3));
    else if (warp == 8)
        tile.produce_keys(begin, end);
    else if (warp == 9)
        tile.produce_rows();
    else if (warp == 10)
        tile.multiply();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) a2_tmem_dealloc<512>(0u);
}

// Where every part starts (as chunk_plan_kernel)
__global__ void __launch_bounds__(kChPlanThreads) key_plan_kernel(const __grid_constant__ KeyParams kp)
{
    if (threadIdx.x == 0) griddep_launch_dependents();
    griddep_wait();
    const RaggedParams &p = kp.r;
    const auto cost = [&](int r, bool flag, ChRequest &q) {
        q = kw_request(p, p.starts[r], p.starts[r + 1], p.context_lens[r], flag);
        return p.nkv * kw_request_cost(q, kp.over);
    };
    ch_plan(p, cost, [&](const ChRequest &q, int r, int64_t off) { return kw_locate(q, r, off, kp.tokens, kp.over); });
}

// The block of keys that part blockIdx.x leaves to the next ones: the parts' sums in order
__global__ void __launch_bounds__(kKwKeys) key_merge_kernel(const __grid_constant__ KeyParams kp)
{
    if (threadIdx.x == 0) griddep_launch_dependents();
    griddep_wait();
    const RaggedParams &p = kp.r;
    const int c = blockIdx.x;
    const ChPos here = p.ws_pos[c], next = p.ws_pos[c + 1];
    if (next.k == 0 || (ch_same_item(here, next) && here.k > 0)) return;   // none, or an earlier part's
    const ChRequest q = kw_request(p, p.starts[next.r], p.starts[next.r + 1], p.context_lens[next.r], false);
    float total = 0.f;
    bool bad = false;
    for (int i = c;; ++i) {
        const bool last = !ch_same_item(p.ws_pos[i + 1], next);
        if (i == c || last || p.ws_pos[i].k != p.ws_pos[i + 1].k) {   // (a part without a step of it left nothing)
            const int part = 2 * i + (i == c);
            total += kp.ws[(int64_t)part * kKwKeys + threadIdx.x];
            bad |= kp.ws_bad[part] != 0;
        }
        if (last) break;
    }
    const int j = next.b * kKwKeys + threadIdx.x;
    if (bad || j >= q.L) return;
    const int64_t at = ((int64_t)next.r * p.nkv + next.g) * p.max_blocks * kPageSlots + j;
    p.out_weights[at] = p.decay == 0.f ? total : fmaf(p.decay, p.weights[at], total);
}

// ---- host -------------------------------------------------------------------

template <class E, int D>
bool prepare_key_kernel()
{
    static_assert(kw_smem<D>().total <= (uint32_t)kMaxSmemPerCta, "shared memory");
    return cudaFuncSetAttribute((const void *)key_tile_kernel<E, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)kw_smem<D>().total) == cudaSuccess;
}

bool prepare_key_kernels()
{
    return prepare_key_kernel<Bf16, 64>() && prepare_key_kernel<Bf16, 128>() && prepare_key_kernel<Fp16, 64>() &&
           prepare_key_kernel<Fp16, 128>();
}

// q as 64 columns, the head's 64-column blocks, heads, tokens: a box is one such
// block of a KV head's q heads of `tokens` tokens, 128 bytes a row
int encode_rows_map(const RaggedParams &p, int head_dim, int tokens, bool bf16, CUtensorMap *m)
{
    // (a dimension of one element has no stride of its own)
    const cuuint64_t hs = p.q_heads > 1 ? (cuuint64_t)p.q_hs * 2 : (cuuint64_t)head_dim * 2;
    const cuuint64_t ts = p.T > 1 ? (cuuint64_t)p.q_ts * 2 : (cuuint64_t)head_dim * 2;
    const cuuint64_t dims[4] = {64, (cuuint64_t)head_dim / 64, (cuuint64_t)p.q_heads, (cuuint64_t)p.T};
    const cuuint64_t strides[3] = {128, hs, ts};
    const cuuint32_t box[4] = {64, 1, (cuuint32_t)p.group, (cuuint32_t)tokens};
    const cuuint32_t es[4] = {1, 1, 1, 1};
    return g_encode(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, (void *)p.q, dims, strides,
                    box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? QKVF_OK
               : QKVF_ERR_CUDA;
}

// Two sums a part, whether they are void, the parts' starts
size_t key_weights_workspace(int sms)
{
    const size_t slots = (size_t)2 * sms;
    return slots * (kKwKeys * 4 + 4) + ((size_t)(sms + 1) * sizeof(ChPos) + 255) / 256 * 256 + 256;
}

// Tokens of a step: as many as 128 rows hold, and no more than the requests have
// on average (single tokens: no rows beside their own are fetched)
KeyParams key_params(RaggedParams p, void *workspace, int sms)
{
    KeyParams kp = {};
    const int most = kChTile / p.group, mean = p.R > 0 ? (p.T + p.R - 1) / p.R : 1;
    kp.tokens = mean < 1 ? 1 : mean < most ? mean : most;
    kp.rows = kp.tokens * p.group;
    kp.over = 3 * most;
    const size_t slots = (size_t)2 * sms;
    kp.ws = static_cast<float *>(workspace);
    kp.ws_bad = reinterpret_cast<int *>(kp.ws + slots * kKwKeys);
    p.ws_pos = reinterpret_cast<ChPos *>(kp.ws_bad + (slots + 3) / 4 * 4);
    p.parts = sms;
    p.wait_limit_ns = g_wait_limit_ns;
    kp.r = p;
    return kp;
}

template <class E, int D>
int launch_key_weights(const CUtensorMap &keys, const CUtensorMap &rows, const KeyParams &kp, void *stream)
{
    int rc = launch_pdl(key_plan_kernel, dim3(1), dim3(kChPlanThreads), 0, stream, kp);
    if (rc != QKVF_OK) return rc;
    rc = launch_pdl(key_tile_kernel<E, D>, dim3((unsigned)kp.r.parts), dim3(kKwThreads), (size_t)kw_smem<D>().total, stream, keys,
                    rows, kp);
    if (rc != QKVF_OK) return rc;
    return launch_pdl(key_merge_kernel, dim3((unsigned)kp.r.parts), dim3(kKwKeys), 0, stream, kp);
}

const char *check_key_weights_args(const RaggedParams &p, int head_dim, float scale, int dtype, const void *workspace,
                                   size_t workspace_bytes, int *code)
{
    if (const char *why = check_ragged_args(p.q, p.q_ts, p.q_hs, p.kv_cache, p.num_pages, p.starts, p.block_table,
                                            p.max_blocks, p.context_lens, p.T, p.R, p.q_heads, p.nkv, head_dim, scale,
                                            dtype, workspace, code))
        return why;
    *code = QKVF_ERR_LAYOUT;
    if ((p.T > 1 && p.q_ts == 0) || (p.q_heads > 1 && p.q_hs == 0)) return "q's strides must be above 0";
    *code = QKVF_ERR_ARG;
    if (p.window < 0) return "window must be 0 (every token) or more";
    if (!(p.decay >= 0.f) || !(p.decay <= 1.f)) return "decay must be in [0, 1]";
    *code = QKVF_OK;
    if (p.R == 0) return nullptr;
    *code = QKVF_ERR_NULL;
    if ((p.T > 0 && !p.lse) || !p.out_weights || (p.decay != 0.f && !p.weights)) return "a required pointer is NULL";
    *code = QKVF_ERR_ALIGN;
    if (!aligned(p.lse, 4) || !aligned(p.weights, 4) || !aligned(p.out_weights, 4))
        return "lse and the weights must be 4-byte aligned";
    *code = QKVF_ERR_ARG;
    const size_t w_bytes = (size_t)p.R * p.nkv * p.max_blocks * kPageSlots * 4, rows = (size_t)p.T * p.q_heads;
    if (p.weights && p.weights != p.out_weights && overlap(p.weights, w_bytes, p.out_weights, w_bytes))
        return "out overlaps weights without being weights";
    if (p.weights && workspace_bytes && overlap(p.weights, w_bytes, workspace, workspace_bytes))
        return "out or the workspace overlaps another argument";
    const void *outs[] = {p.out_weights, workspace};
    const size_t sizes[] = {w_bytes, workspace_bytes};
    if (ragged_overlap(p, head_dim, outs, sizes, 2, p.lse, rows * 4)) return "out or the workspace overlaps another argument";
    *code = QKVF_OK;
    return nullptr;
}

}  // namespace qkvf

extern "C" {

size_t key_weights_workspace_bytes(int T, int num_reqs, int q_heads, int num_kv_heads, int head_dim, int max_blocks)
{
    int code;
    if (qkvf::check_ragged_shape(T, num_reqs, q_heads, num_kv_heads, head_dim, max_blocks, &code)) return 0;
    qkvf::DeviceState *d;
    return qkvf::probe_device(&d) == QKVF_OK ? qkvf::key_weights_workspace(d->sms) : 0;
}

const char *key_weights_unsupported(const void *q, int64_t q_token_stride, int64_t q_head_stride, const void *kv_cache,
                                    int64_t num_pages, const float *lse, const int32_t *starts, const int32_t *block_table,
                                    int max_blocks, const int32_t *context_lens, int T, int num_reqs, int q_heads,
                                    int num_kv_heads, int head_dim, int window, float decay, float scale, int dtype,
                                    const float *weights, float *out, const void *workspace, size_t workspace_bytes)
{
    qkvf::RaggedParams prm = qkvf::ragged_params(q, q_token_stride, q_head_stride, kv_cache, num_pages, starts, block_table,
                                                 max_blocks, context_lens, T, num_reqs, q_heads, num_kv_heads, scale, dtype);
    prm.lse = const_cast<float *>(lse);
    prm.weights = weights;
    prm.out_weights = out;
    prm.window = window;
    prm.decay = decay;
    int code;
    const char *why = qkvf::check_key_weights_args(prm, head_dim, scale, dtype, workspace, workspace_bytes, &code);
    if (why) return why;
    qkvf::DeviceState *d;
    const int rc = qkvf::probe_device(&d);
    if (rc != QKVF_OK) return qkv_front_strerror(rc);
    return num_reqs > 0 && workspace_bytes < qkvf::key_weights_workspace(d->sms) ? "the workspace is too small" : nullptr;
}

int key_weights(const void *q, int64_t q_token_stride, int64_t q_head_stride, const void *kv_cache, int64_t num_pages,
                const float *lse, const int32_t *starts, const int32_t *block_table, int max_blocks,
                const int32_t *context_lens, int T, int num_reqs, int q_heads, int num_kv_heads, int head_dim, int window,
                float decay, float scale, int dtype, const float *weights, float *out, void *workspace,
                size_t workspace_bytes, void *stream)
{
    qkvf::RaggedParams prm = qkvf::ragged_params(q, q_token_stride, q_head_stride, kv_cache, num_pages, starts, block_table,
                                                 max_blocks, context_lens, T, num_reqs, q_heads, num_kv_heads, scale, dtype);
    prm.lse = const_cast<float *>(lse);
    prm.weights = weights;
    prm.out_weights = out;
    prm.window = window;
    prm.decay = decay;
    int code;
    if (qkvf::check_key_weights_args(prm, head_dim, scale, dtype, workspace, workspace_bytes, &code)) return code;
    if (num_reqs == 0) return QKVF_OK;
    qkvf::DeviceState *d;
    const int rc = qkvf::probe_device(&d);
    if (rc != QKVF_OK) return rc;
    if (workspace_bytes < qkvf::key_weights_workspace(d->sms)) return QKVF_ERR_SIZES;
    const bool bf16 = qkvf::dtype_of(dtype) == QKVF_DTYPE_BF16;
    CUtensorMap keys, rows = {};
    int mrc = qkvf::encode_chunk_map(kv_cache, num_pages, num_kv_heads, head_dim, bf16, &keys);
    if (mrc != QKVF_OK) return mrc;
    qkvf::KeyParams kp = qkvf::key_params(prm, workspace, d->sms);
    if (T > 0) mrc = qkvf::encode_rows_map(prm, head_dim, kp.tokens, bf16, &rows);
    if (mrc != QKVF_OK) return mrc;
    if (bf16)
        return head_dim == 64 ? qkvf::launch_key_weights<qkvf::Bf16, 64>(keys, rows, kp, stream)
                              : qkvf::launch_key_weights<qkvf::Bf16, 128>(keys, rows, kp, stream);
    return head_dim == 64 ? qkvf::launch_key_weights<qkvf::Fp16, 64>(keys, rows, kp, stream)
                          : qkvf::launch_key_weights<qkvf::Fp16, 128>(keys, rows, kp, stream);
}

int key_weights_packed(const int64_t *args, void *stream)
{
    if (!args) return QKVF_ERR_NULL;
    qkvf::Words w(args);
    const int mb = w.i(8), T = w.i(10), R = w.i(11), q_heads = w.i(12), nkv = w.i(13), dim = w.i(14), window = w.i(15),
              dtype = w.i(18);
    if (!w.ok) return QKVF_ERR_SIZES;
    return key_weights(w.p<void>(0), args[1], args[2], w.p<void>(3), args[4], w.p<float>(5), w.p<int32_t>(6), w.p<int32_t>(7),
                       mb, w.p<int32_t>(9), T, R, q_heads, nkv, dim, window, (float)w.d(16), (float)w.d(17), dtype,
                       w.p<float>(19), w.p<float>(20), w.p<void>(21), (size_t)args[22], stream);
}

}  // extern "C"
