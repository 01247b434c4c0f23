// prefix_attn: decode attention of requests that share a prefix (included by
// qkv_front.cu: one translation unit).
//
// Row (request r, token i of its q_len, q head h) attends to the shared
// prefix's keys 0 .. P - 1 and to its request's own keys j <= L_r - q_len + i,
// under one softmax:
//   s = scale q . k;  out = sum exp(s - m) v / sum exp(s - m);  lse = ln sum exp(s).
// Both key ranges are split; every split leaves a partial (m, sum exp(s - m),
// sum exp(s - m) v), m near its own maximum, per row in the workspace, in FP32, and a merge joins them:
//   out = sum_k e^(m_k - M) o_k / sum_k e^(m_k - M) l_k,  M = max_k m_k.
//
// Three kernels, the second and third PDL-launched behind the first:
//  * prefix_tile_kernel: all requests' rows against the prefix in tiles of 128
//    rows on tcgen05, one CTA per SM.  Two groups of four softmax warps (a
//    thread per row), each group on its own tile, both on the same key blocks
//    (one tile: on two halves of the keys); two producer warps (TMA, a
//    swizzled box per page) and an MMA warp per group.  S = Q K^T goes to
//    tensor memory, the weights back into S's columns as the A operand of
//    O += P V, so neither passes through shared memory.
//  * prefix_rows_kernel: each request's own keys, and a prefix that few rows
//    share, in tiles of 16 or 64 rows with mma.sync, two to four CTAs per SM.
//    Many short key lists want many small CTAs in flight; it starts beside the
//    tile kernel on the SMs that one leaves (its split is chosen with that work
//    in mind) and follows on all of them.  Long own keys of many rows a request
//    take the tile kernel instead, one item a group.
//  * prefix_merge_kernel: a row's partials, 1 to 16 warps a row.
//
// What bounds it.  A prefix of many rows is a dense product: 512 rows x 8 KV
// heads of 64 over 32K keys are 34 GFLOP, 17.8 us at the 1930 TFLOP/s measured
// for bf16, with 10 us of bytes.  A step of the tile kernel (two tiles against
// 128 keys) takes ~1830 clocks: 1024 of them are the least that its 32768
// exponentials need (8 a clock and scheduler), 1050 the tensor pipe's work
// beside them, and the rest the hand-overs between softmax and MMA warps
// (160 - 275 clocks each), which the two groups' warps on a scheduler spend
// at the same time.  64 x 64 heads of 64 over 128K keys run in 123 us (1120
// TFLOP/s); the 32K call with up to 1K own keys per request in 56.4 us.  With few
// rows the keys' bytes bound it: 8 rows x 8 KV heads of 128 over 128K keys take
// 83 us, 80.3 at the copy rate.  Short calls are two launches: 5.8 us.

#include <type_traits>

#include "prefix_plan.h"

namespace qkvf {

constexpr int kPaMaxRequests = 65535;
constexpr int kPaMaxQLen = 1024;
constexpr int kPaMaxGroup = 64;          // q heads per KV head
constexpr int kPaThreads = 384;          // 2 softmax groups of 4 warps, 2 producer warps, 2 MMA warps

// Weights are 2^(s - mu), mu some bits below the row's maximum: in fp16, whose
// normal numbers end at 2^-14, a weight of 1 for the maximum would leave keys 14
// bits below it fewer and fewer bits, and keys 25 below it none, while they
// still count in the sum (one early key that takes most of the weight, in front
// of thousands that make the output).  bf16 has the range of FP32.
// 8 bits: in the tile kernel a row's weights of a block may add up to `most`
// before mu follows, and a block of 128 equal scores stays below that.  It leaves
// fp16 8 bits of growth where bf16 has 14: 64 rows x 8 KV heads over
// 32K keys take 56 us in either for scores of a standard deviation of 1 or 2, 65
// and 55 for one of 4, 71 and 67 for one of 8.
template <class E>
struct PaWeight {
    static constexpr float below = E::is_bf16 ? 0.f : 8.f, most = E::is_bf16 ? 16384.f : 61440.f;
};

// Shapes by head width: a block of keys is one ring stage (K and V, 32 KB)
// and one S tile; each of the two rings holds `slots` of them.
template <int D>
struct PaShape {
    static constexpr int keys = pa_tile_keys(D);
    static constexpr int pages = keys / kPageSlots;
    static constexpr int slots = D == 64 ? 3 : 2;
    static constexpr int nblk = 2 * D / 64;                    // 64-column blocks of a slot: K then V
    static constexpr uint32_t page_bytes = kPageSlots * 4 * D; // one box
    static constexpr uint32_t stage_bytes = pages * page_bytes;
    static constexpr uint32_t q_bytes = kPaTile * 2 * D;
    // tensor memory columns: three units of keys / 2 columns a group for S and
    // the weights, then both groups' O
    static constexpr uint32_t tSP = 0, tO = 3 * keys, cols = 512;
    static_assert(tO + 2 * D <= cols && stage_bytes == 32768, "tensor memory and ring");
};

struct PaSmem {   // offsets from the 1024-byte aligned base
    uint32_t q, ring, full, empty, qready, sfull, sfree, pready, pvdone, odone, drain, tmem, flags, total;
};

template <int D>
__host__ __device__ constexpr PaSmem pa_smem()
{
    using Sh = PaShape<D>;
    PaSmem L = {};
    uint32_t off = 0;
    L.q = off;
    off += 2 * Sh::q_bytes;
    L.ring = off;
    off += 2 * Sh::slots * Sh::stage_bytes;
    L.full = off;
    off += 2 * Sh::slots * 8;
    L.empty = off;
    off += 2 * Sh::slots * 8;
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
    L.flags = off;
    off += 32;
    L.total = off + 1024;
    return L;
}

struct PrefixParams {
    const void *q;
    const int32_t *prefix_pages;
    const int32_t *prefix_len;
    const int32_t *block_table;
    const int32_t *context_lens;
    void *out;
    float *lse;
    float *ws_o;      // partial O [split][row][D], prefix splits first
    float2 *ws_ml;    // partial (mu in log2 units, sum) [row][split]
    int64_t num_pages;
    int64_t q_ts, q_hs;
    unsigned long long wait_limit_ns;
    int prefix_blocks, max_blocks;
    int R, q_len, q_heads, nkv, group;
    int rows;         // R * q_len * q_heads
    int tiles;        // 128-row tiles of a KV head's rows (the tile kernel)
    int pair;         // both groups of a CTA on one key stream
    int small, pre_rows;       // the prefix's rows are few: the rows kernel's, in a tile of pre_rows
    int own_tile;              // the own keys are the tile kernel's too
    int own_rows, own_tiles;   // rows of one tile of a request's rows, tiles of a request
    int sp, ss;       // key splits of the prefix and of a request's own keys
    float scale_log2;
    const void *kv_cache;
    int zero;         // rows left alone have zeros in out instead
};

// One unit of work: a tile of query rows against a range of key blocks
struct PaItem {
    const int32_t *pages;
    int g;           // KV head
    int tok0;        // first token of the row set the tile is cut from
    int row0, rows;  // the tile's first row in that set, and its rows
    int kb0, kb1;    // key blocks
    int keys;        // keys that some row of the tile sees
    int limit0;      // keys that token 0 of the row set sees; later tokens see `step` more each
    int step;
    int all;         // keys that every row of the tile sees
    int split;       // partial slot
};

// past: past L1, in a kernel that starts without a wait of its own (elsewhere
// L1 is worth having: 64 requests' own keys without a prefix 20.3 us and 21.2, 33
// rows x 4 KV heads of 128 over 16K 21.6 and 22.6)
template <class T>
__device__ __forceinline__ T pa_load(const T *ptr, bool past) { return past ? __ldcg(ptr) : *ptr; }

__device__ __forceinline__ int pa_prefix_len(const PrefixParams &p, bool past)
{
    if (p.prefix_blocks == 0) return 0;
    const int P = pa_load(p.prefix_len, past);
    return P > p.prefix_blocks * kPageSlots ? -1 : P;
}

// The nb key blocks of a row set dealt evenly to min(splits, nb) splits; the
// splits behind those are empty
__device__ __forceinline__ void pa_deal(PaItem &it, int nb, int splits, int s)
{
    const int n = min(splits, nb);
    it.kb0 = s < n ? (int)((int64_t)s * nb / n) : 0;
    it.kb1 = s < n ? (int)((int64_t)(s + 1) * nb / n) : 0;
}

// The prefix: tile `tile` (of `tile_rows` rows) of KV head g, split s, blocks of KB keys
template <int KB>
__device__ __forceinline__ PaItem pa_prefix_item(const PrefixParams &p, int P, int tile_rows, int tile, int g, int s)
{
    PaItem it;
    it.pages = p.prefix_pages;
    it.g = g;
    it.tok0 = 0;
    it.row0 = tile * tile_rows;
    it.rows = min(tile_rows, p.R * p.q_len * p.group - it.row0);
    it.keys = P;
    it.limit0 = P;
    it.step = 0;
    it.all = P;
    it.split = s;
    pa_deal(it, (P + KB - 1) / KB, p.sp, s);
    return it;
}

// Keys that some row of a request's tile sees: its last token's (none of a
// padding request's: its length, any negative number, enters no sum)
__device__ __forceinline__ int pa_own_keys(const PrefixParams &p, int L, int tile)
{
    if (L < 0 || L > p.max_blocks * kPageSlots) return 0;
    const int last = min(p.q_len - 1, (tile * p.own_rows + p.own_rows - 1) / p.group);
    return max(0, L - p.q_len + last + 1);
}

// A request's own keys: tile `tile` of request r's rows of KV head g, split s
template <int KB>
__device__ __forceinline__ PaItem pa_own_item(const PrefixParams &p, int P, int L, int r, int tile, int g, int s)
{
    PaItem it;
    it.pages = p.block_table + (size_t)r * p.max_blocks;
    it.g = g;
    it.tok0 = r * p.q_len;
    it.row0 = tile * p.own_rows;
    it.rows = min(p.own_rows, p.q_len * p.group - it.row0);
    it.keys = P < 0 ? 0 : pa_own_keys(p, L, tile);
    it.limit0 = max(L, 0) - p.q_len + 1;
    it.step = 1;
    it.all = it.limit0 + it.row0 / p.group;
    it.split = p.sp + s;
    pa_deal(it, (it.keys + KB - 1) / KB, p.ss, s);
    return it;
}

// The tile kernel's work in order.  The prefix's, pair: a CTA's two groups take
// the same key blocks against the two tiles of a 256-row block (a second tile
// that does not exist has rows <= 0); otherwise the only tile's splits go to 2
// gridDim.x groups.  The own keys': one item a group.
template <int D, bool kOwn>
struct PaWork {
    const PrefixParams &p;
    int P, w, idx, end, stride;
    __device__ __forceinline__ PaWork(const PrefixParams &prm, int prefix, int group) : p(prm), P(prefix), w(group)
    {
        if (kOwn) {
            idx = 2 * blockIdx.x + w;
            stride = end = p.R * p.nkv * p.own_tiles * p.ss;
        } else {
            idx = p.pair ? blockIdx.x : 2 * blockIdx.x + w;
            stride = p.pair ? gridDim.x : 2 * gridDim.x;
            end = P > 0 ? (p.pair ? (p.tiles + 1) / 2 : 1) * p.nkv * p.sp : 0;
        }
    }
    __device__ __forceinline__ bool next(PaItem &it)   // the next item with key blocks
    {
        for (; idx < end; idx += stride) {
            if (kOwn) {
                const int g = idx % p.nkv, rest = idx / p.nkv, r = rest % p.R, ts = rest / p.R;
                const int L = __reduce_max_sync(0xffffffffu, __ldcg(p.context_lens + r));
                it = pa_own_item<PaShape<D>::keys>(p, P, L, r, ts % p.own_tiles, g, ts / p.own_tiles);
            } else {
                const int rb = p.pair ? (p.tiles + 1) / 2 : 1, tile = p.pair ? 2 * (idx % rb) + w : 0, gs = idx / rb;
                it = pa_prefix_item<PaShape<D>::keys>(p, P, kPaTile, tile, gs % p.nkv, gs / p.nkv);
            }
            if (it.kb1 > it.kb0) {
                idx += stride;
                return true;
            }
        }
        return false;
    }
};

// Ring position of a group's step n: with pair the steps alternate between
// the two rings, otherwise they stay in ring w
template <int NS>
struct PaRing {
    int w, pair, n = 0;
    int st, use;   // stage and how often it was used before
    __device__ __forceinline__ PaRing(int group, int both) : w(group), pair(both) {}
    __device__ __forceinline__ void take()
    {
        const int ring = pair ? n & 1 : w, k = pair ? n >> 1 : n;
        ++n;
        st = ring * NS + k % NS;
        use = k / NS;
    }
};

// Until the phase of this parity completes, at most limit_ns: then flags[0] is
// set, every later wait of the CTA that honours it is short, and its results
// are void.  (In line: a function call does not go with setmaxnreg.)
__device__ __forceinline__ void pa_wait(uint32_t bar, uint32_t parity, volatile int *flags, unsigned long long limit_ns,
                                        bool honour = true)
{
    unsigned long long start = 0;
#pragma unroll 1
    for (int i = 1; !mbar_try_wait(bar, parity); ++i) {
        if (i & 63) continue;
        if (honour && flags[0]) return;
        const unsigned long long now = global_ns();
        if (start == 0) {
            start = now;
        } else if (now - start > limit_ns) {
            flags[0] = 1;
            atomicOr(&g_status, QKVF_STATUS_WAIT_TIMEOUT);
            return;
        }
    }
}

// One lane of a converged warp, known to the compiler as one (its operands of
// tcgen05 instructions then stay in uniform registers)
__device__ __forceinline__ bool pa_elect()
{
    uint32_t mine;
    asm volatile(
        "{\n"
        ".reg .pred p;\n"
        "elect.sync _|p, 0xffffffff;\n"
        "selp.u32 %0, 1, 0, p;\n"
        "}\n"
        : "=r"(mine));
    return mine != 0;
}

// ---- tensor memory, 32 lanes x 32 columns per warp -------------------------

#define PA_REGS8(a, i) "=r"(a[i]), "=r"(a[i + 1]), "=r"(a[i + 2]), "=r"(a[i + 3]), "=r"(a[i + 4]), "=r"(a[i + 5]), "=r"(a[i + 6]), "=r"(a[i + 7])
#define PA_IN8(a, i) "r"(a[i]), "r"(a[i + 1]), "r"(a[i + 2]), "r"(a[i + 3]), "r"(a[i + 4]), "r"(a[i + 5]), "r"(a[i + 6]), "r"(a[i + 7])

__device__ __forceinline__ void pa_tmem_ld32(uint32_t addr, uint32_t *r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : PA_REGS8(r, 0), PA_REGS8(r, 8), PA_REGS8(r, 16), PA_REGS8(r, 24)
        : "r"(addr));
}

__device__ __forceinline__ void pa_tmem_st16(uint32_t addr, const uint32_t *r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(addr),
        PA_IN8(r, 0), PA_IN8(r, 8)
        : "memory");
}

template <int N>
__device__ __forceinline__ void pa_tmem_st(uint32_t addr, const uint32_t *r)
{
#pragma unroll
    for (int c = 0; c < N; c += 16) pa_tmem_st16(addr + c, r + c);
}

// N scores of this thread's row (and N more)
template <int N>
__device__ __forceinline__ void pa_load_scores(uint32_t addr, uint32_t *s)
{
#pragma unroll
    for (int c = 0; c < N; c += 32) pa_tmem_ld32(addr + c, s + c);
    tmem_ld_wait();
}
template <int N>
__device__ __forceinline__ void pa_issue_scores(uint32_t addr, uint32_t *s, uint32_t addr2, uint32_t *s2)
{
#pragma unroll
    for (int c = 0; c < N; c += 32) {
        pa_tmem_ld32(addr + c, s + c);
        pa_tmem_ld32(addr2 + c, s2 + c);
    }
}

// Behind the wait for a load: no use of its registers moves ahead of here
template <int N>
__device__ __forceinline__ void pa_loaded(uint32_t (&s)[N])
{
#pragma unroll
    for (int c = 0; c < N; c += 8)
        asm volatile("" : "+r"(s[c]), "+r"(s[c + 1]), "+r"(s[c + 2]), "+r"(s[c + 3]), "+r"(s[c + 4]), "+r"(s[c + 5]),
                     "+r"(s[c + 6]), "+r"(s[c + 7]));
}

// The scores from `limit` on become -infinity, whatever their slots hold
template <int N>
__device__ __forceinline__ void pa_hide(uint32_t (&s)[N], int limit)
{
#pragma unroll
    for (int c = 0; c < N; ++c)
        if (c >= limit) s[c] = 0xff800000u;
}

__device__ __forceinline__ void pa_tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D += A B with A (the weights) in tensor memory
__device__ __forceinline__ void pa_umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n"
        ".reg .pred p;\n"
        "setp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n"
        "}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Descriptor of a 128-byte-swizzled operand: `sbo` bytes between 8-row groups
// (8-key groups of V), `lbo` bytes between 64-column blocks of V
__device__ __forceinline__ uint64_t pa_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo)
{
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)(lbo >> 4) << 16 | (uint64_t)(sbo >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

__device__ __forceinline__ void pa_load_page(uint32_t dst, const CUtensorMap *m, uint32_t bar, int c4)
{
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %3, %3, %3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(0), "r"(c4)
        : "memory");
}

// kind::f16, FP32 accumulator, M = 128: bf16 or fp16 operands, B MN-major for V
template <class E>
__device__ __forceinline__ constexpr uint32_t pa_idesc(int n, bool b_mn)
{
    constexpr uint32_t fmt = E::is_bf16 ? 1u : 0u;
    return 1u << 4 | fmt << 7 | fmt << 10 | (b_mn ? 1u << 16 : 0u) | (uint32_t)(n >> 3) << 17 |
           (uint32_t)(kPaTile >> 4) << 24;
}

__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

template <int N>
__device__ __forceinline__ float pa_max(const uint32_t (&s)[N], float m)
{
    float a = m, b = m;
#pragma unroll
    for (int c = 0; c < N; c += 4) {
        a = fmaxf(fmaxf(a, __uint_as_float(s[c])), __uint_as_float(s[c + 1]));
        b = fmaxf(fmaxf(b, __uint_as_float(s[c + 2])), __uint_as_float(s[c + 3]));
    }
    return fmaxf(a, b);
}

// The weights 2^(scale s + base) of N scores, rounded and packed in pairs; returns their sum
template <class E, int N>
__device__ __forceinline__ float pa_weights(const uint32_t (&s)[N], uint32_t (&pk)[N / 2], uint64_t scale2, float base)
{
    const uint64_t nb2 = f2_pack(base, base);
    uint64_t sum[2] = {0, 0};
#pragma unroll
    for (int c = 0; c < N; c += 2) {
        float a, b;
        f2_unpack(f2_fma(f2_pack(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), scale2, nb2), a, b);
        a = a2_ex2(a);
        b = a2_ex2(b);
        sum[(c >> 1) & 1] = f2_add(sum[(c >> 1) & 1], f2_pack(a, b));
        pk[c / 2] = E::pack(a, b);
    }
    float a, b;
    f2_unpack(f2_add(sum[0], sum[1]), a, b);
    return a + b;
}

// A key that only later rows of a tile see has the weight 0 in the others, and
// a V of it that is not finite must not meet that weight (0 x infinity is not
// 0).  Among the keys from it.all on such values become 0 before the product,
// and the rows that see the key have them added when the item is done.  (16
// requests x 8 tokens x 64 heads of 64 over up to 1K own keys: 19.3 us, and 18.6
// without looking; over 8K shared keys besides 42.3 and 41.4.)

// The halves of two packed values that are infinite or NaN, as a mask
template <class E>
__device__ __forceinline__ uint32_t pa_not_finite(uint32_t v)
{
    constexpr uint32_t exponent = E::is_bf16 ? 0x7f807f80u : 0x7c007c00u;
    return __vcmpeq2(v & exponent, exponent);
}

// By one warp: whether the V rows of keys `from` .. `to` - 1 of the pages at
// `pages` (as TMA lays them out) hold something not finite; kDrop: which
// becomes 0
template <class E, int D, bool kDrop>
__device__ __forceinline__ bool pa_find_not_finite(uint8_t *pages, int from, int to)
{
    constexpr int rows8 = D / 32 * 1024;   // bytes of 8 slots, K and V
    bool found = false;
#pragma unroll 1
    for (int c = from * (D / 8) + (threadIdx.x & 31); c < to * (D / 8); c += 32) {
        const int key = c / (D / 8), ch = c % (D / 8);   // (a row's 16-byte chunks in any order)
        uint4 *at = reinterpret_cast<uint4 *>(pages + (key >> 3) * rows8 + (D / 64 + ch / 8) * 1024 + (key & 7) * 128 + (ch & 7) * 16);
        const uint4 v = *at;
        const uint32_t x = pa_not_finite<E>(v.x), y = pa_not_finite<E>(v.y), z = pa_not_finite<E>(v.z), u = pa_not_finite<E>(v.w);
        if (x | y | z | u) {
            found = true;
            if (kDrop) *at = make_uint4(v.x & ~x, v.y & ~y, v.z & ~z, v.w & ~u);
        }
    }
    found = __any_sync(0xffffffffu, found);
    if (kDrop && found) {
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
    }
    return found;
}

// V row of own key `key` of the item's KV head, past L1; null: its page is outside the cache
template <int D>
__device__ __forceinline__ const uint32_t *pa_value_row(const PrefixParams &p, const PaItem &it, int key)
{
    const int page = __ldcg(it.pages + key / kPageSlots);
    if (page < 0 || page >= p.num_pages) return nullptr;
    const int64_t slot = ((int64_t)page * p.nkv + it.g) * kPageSlots + key % kPageSlots;
    return reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(p.kv_cache) + slot * (2 * D) + D);
}

// (a, b) += those of two packed values that are not finite
template <class E>
__device__ __forceinline__ void pa_add_not_finite(uint32_t v, float &a, float &b)
{
    const uint32_t m = pa_not_finite<E>(v);
    if (m & 0xffffu) a += E::lo(v);
    if (m & 0xffff0000u) b += E::hi(v);
}

// The roles of the tile kernel's warps.  Every loop over items and blocks is
// the same in each of them.
template <class E, int D, bool kOwn>
struct PaTile {
    using Sh = PaShape<D>;
    using Work = PaWork<D, kOwn>;
    static constexpr int KB = Sh::keys, NS = Sh::slots, U = KB / 2;
    // Each S is loaded before the weights ahead of it are handed over: 64 rows
    // x 8 KV heads of 8 over 128K keys 129.6 us, and 135.4 without.  With blocks of
    // 64 keys S would not be there yet: 8 heads of 128 over 32K 70.5 us, 62.5 without.
    static constexpr bool kAhead = D == 64;
    static constexpr PaSmem LY = pa_smem<D>();
    const CUtensorMap *map;
    const PrefixParams &p;
    uint8_t *smem;
    uint32_t sb;
    int lane;

    // The prefix's length, the same register for the whole warp.  What a role's
    // first item needs besides is fetched beside it.
    __device__ __forceinline__ int length() const { return __reduce_max_sync(0xffffffffu, pa_prefix_len(p, kOwn)); }
    __device__ __forceinline__ volatile int *flags() const { return reinterpret_cast<volatile int *>(smem + LY.flags); }
    __device__ __forceinline__ void wait(uint32_t bar, int n) const   // until phase n of bar is complete
    {
        pa_wait(sb + bar, (uint32_t)n & 1, flags(), p.wait_limit_ns);
    }
    __device__ __forceinline__ bool dead() const { return flags()[0] != 0; }
    __device__ __forceinline__ int pair() const { return kOwn ? 0 : p.pair; }
    // A page outside the cache, as producer w has flagged: of the prefix's it voids every row
    __device__ __forceinline__ bool bad(int w) const { return kOwn ? flags()[1 + w] : flags()[1] | flags()[2]; }
    __device__ __forceinline__ int pages_from(const PaItem &it, int block) const   // of a block, with keys
    {
        return min(Sh::pages, (it.keys + kPageSlots - 1) / kPageSlots - block * Sh::pages);
    }

    // ---- produce: ring w's blocks, one 128-byte-swizzled box per page ----
    __device__ __forceinline__ void produce(int w) const
    {
        if (lane == 0) tma_prefetch_map(map);
        PaItem it;
        int guess = -1, entry = 0;   // the first entries as of a full table
        if (!kOwn && Work(p, p.prefix_blocks * kPageSlots, w).next(it)) {
            guess = it.kb0 * Sh::pages;
            if (guess + lane < p.prefix_blocks) entry = pa_load(it.pages + guess + lane, kOwn);
        }
        Work work(p, length(), w);
        bool ok = true;
        PaRing<NS> ring(w, pair());
        int mine = 0;   // steps loaded into this ring
        unsigned bad_any = 0u;
        while (ok && work.next(it)) {
            const int pg0 = it.kb0 * Sh::pages;
            const int pg1 = min(it.kb1 * Sh::pages, (it.keys + kPageSlots - 1) / kPageSlots);
            int next = pg0 + lane < pg1 ? (pg0 == guess ? entry : pa_load(it.pages + pg0 + lane, kOwn)) : 0;
            for (int c = pg0; c < pg1 && ok; c += 32) {
                int page = next;
                if (c + 32 + lane < pg1) next = pa_load(it.pages + c + 32 + lane, kOwn);
                bool bad = false;
                if (c + lane < pg1 && (page < 0 || page >= p.num_pages)) {   // flagged, page 0 in its place
                    bad = true;
                    page = 0;
                }
                if (__any_sync(0xffffffffu, bad)) {   // seen by the softmax before these keys' products are
                    bad_any = 1u;
                    flags()[1 + w] = 1;
                    __syncwarp();
                }
                for (int b0 = c; b0 < min(c + 32, pg1); b0 += Sh::pages) {
                    ring.take();
                    const int st = ring.st;
                    if (st / NS != w) continue;   // the other producer's
                    const int n = min(Sh::pages, pg1 - b0);
                    if (ring.use > 0) wait(LY.empty + 8 * st, ring.use - 1);
                    __syncwarp();
                    ok = !__any_sync(0xffffffffu, dead());
                    if (!ok) break;
                    if (lane == 0) mbar_expect_tx(sb + LY.full + 8 * st, (uint32_t)n * Sh::page_bytes);
                    __syncwarp();
                    ++mine;
                    const int i = c + lane - b0;
                    if (i >= 0 && i < n)
                        pa_load_page(sb + LY.ring + st * Sh::stage_bytes + i * Sh::page_bytes, map,
                                     sb + LY.full + 8 * st, page * p.nkv + it.g);
                }
            }
        }
        if (lane == 0) {
            if (bad_any) atomicOr(&g_status, QKVF_STATUS_BAD_REQUEST);
            if (dead())   // our copies land before the CTA leaves
                for (int j = max(0, mine - NS); j < mine; ++j)
                    pa_wait(sb + LY.full + 8 * (w * NS + j % NS), (uint32_t)((j / NS) & 1), flags(), p.wait_limit_ns, false);
        }
        __syncwarp();
    }

    // ---- multiply: group W's S = Q K^T and O += P V ----------------------
    template <int W>
    __device__ __forceinline__ void multiply() const
    {
        Work work(p, length(), W);
        PaItem it;
        PaRing<NS> ring(W, pair());
        int items = 0, blk = 0;   // items and blocks of this group so far
        const uint64_t qd = pa_desc(sb + LY.q + W * Sh::q_bytes, 16, 1024);
        const uint64_t kd0 = pa_desc(sb + LY.ring, 16, Sh::nblk * 1024);
        const uint64_t vd0 = pa_desc(sb + LY.ring + (D / 64) * 1024, 1024, Sh::nblk * 1024);
        constexpr uint32_t dSP = Sh::tSP + W * 3 * U, dO = Sh::tO + W * D;
        while (work.next(it)) {
            const int n = it.kb1 - it.kb0;
            if (it.rows <= 0) {   // no second tile: hand the blocks back
                for (int j = 0; j < n; ++j) {
                    ring.take();
                    wait(LY.full + 8 * ring.st, ring.use);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(sb + LY.empty + 8 * ring.st);
                }
                continue;
            }
            wait(LY.qready + 8 * W, items++);
            int st_prev = 0, pages_prev = 0;
            // the first block with keys that some rows do not see
            const int partly_from = kOwn && it.all < it.keys ? max(it.all, 0) / KB - it.kb0 : n;
            for (int j = 0; j <= n; ++j) {
                int st = 0, pages = 0;
                if (j < n) {   // S of block j
                    ring.take();
                    st = ring.st;
                    pages = pages_from(it, it.kb0 + j);
                    // S of the block before has been read, and the weights of the
                    // one before that, whose columns this S takes (an item's end
                    // has waited for all of its products)
                    wait(LY.full + 8 * st, ring.use);
                    if (j > 1) wait(LY.pvdone + 8 * W, blk - 2);
                    if (blk > 0) wait(LY.sfree + 8 * W, blk - 1);
                    __syncwarp();
                    tc_fence_after();
                    // descriptors: constant steps (16 bytes each) from the tile's first
                    const uint64_t kd = kd0 + (uint32_t)st * (Sh::stage_bytes / 16);
                    const uint32_t dS = dSP + (blk & 1) * U;
                    if (pa_elect()) {
#pragma unroll
                        for (int i = 0; i < D / 16; ++i)
                            umma_bf16(dS, qd + (i / 4) * (kPaTile * 8) + (i % 4) * 2, kd + (i / 4) * 64 + (i % 4) * 2,
                                      pa_idesc<E>(KB, false), i != 0);
                        umma_commit(sb + LY.sfull + 8 * W);
                    }
                    __syncwarp();
                    ++blk;
                }
                if (j > 0) {   // O += P V of block j - 1
                    const int b = j < n ? blk - 2 : blk - 1;
                    if (kOwn && j > partly_from) {   // while its weights are being made
                        const int k0 = (it.kb0 + j - 1) * KB;
                        if (pa_find_not_finite<E, D, true>(smem + LY.ring + st_prev * Sh::stage_bytes, max(it.all - k0, 0), min(it.keys - k0, KB)))
                            flags()[3 + W] = 1;
                    }
                    wait(LY.pready + 16 * (b & 1) + 8 * W, b >> 1);
                    __syncwarp();
                    tc_fence_after();
                    const uint64_t vd = vd0 + (uint32_t)st_prev * (Sh::stage_bytes / 16);
                    const uint32_t dP = dSP + (b & 1) * 2 * U;
                    const uint32_t acc = j > 1;   // the item's first product overwrites O
                    if (pages_prev == Sh::pages) {
                        if (pa_elect()) {
#pragma unroll
                            for (int i = 0; i < Sh::pages; ++i)
                                pa_umma_ts(dO, dP + 8 * i, vd + i * (Sh::page_bytes / 16), pa_idesc<E>(D, true), i > 0 ? 1u : acc);
                            umma_commit(sb + LY.pvdone + 8 * W);
                            umma_commit(sb + LY.empty + 8 * st_prev);
                        }
                    } else if (pa_elect()) {
                        for (int i = 0; i < pages_prev; ++i)
                            pa_umma_ts(dO, dP + 8 * i, vd + i * (Sh::page_bytes / 16), pa_idesc<E>(D, true), i > 0 ? 1u : acc);
                        umma_commit(sb + LY.pvdone + 8 * W);
                        umma_commit(sb + LY.empty + 8 * st_prev);
                    }
                    __syncwarp();
                }
                st_prev = st;
                pages_prev = pages;
            }
            if (pa_elect()) umma_commit(sb + LY.odone + 8 * W);
            __syncwarp();
            if (kOwn && lane == 0) mbar_arrive(sb + LY.odone + 8 * W);   // with the flag of values dropped
        }
        // every MMA of this warp is done before tensor memory is freed (the same
        // lane is elected each time: commits cover the MMAs of one thread)
        if (pa_elect()) umma_commit(sb + LY.drain + 8 * W);
        __syncwarp();
        if (lane == 0) pa_wait(sb + LY.drain + 8 * W, 0, flags(), p.wait_limit_ns, false);
        __syncwarp();
    }

    // ---- softmax: thread = row of group w's tile -------------------------
    // S of even blocks lies in units 0 and 1 of the group's three (KB / 2
    // columns each), of odd ones in 1 and 2.  The weights take the outer unit's
    // columns; the middle one and the unit at the other end are free for the
    // next S while this block's weights are still being made.
    __device__ __forceinline__ void softmax(int w, int wq) const
    {
        const int row = 32 * wq + lane;
        const uint32_t lane_base = (uint32_t)(32 * wq) << 16;
        const uint32_t aSP = Sh::tSP + w * 3 * U + lane_base, aO = Sh::tO + w * D + lane_base;
        uint8_t *sq = smem + LY.q + w * Sh::q_bytes;
        if (!kOwn) {   // the first item's rows of q into L2
            const int idx = p.pair ? blockIdx.x : 2 * blockIdx.x + w, rb = p.pair ? (p.tiles + 1) / 2 : 1;
            const int m = (p.pair ? 2 * (idx % rb) + w : 0) * kPaTile + row, tok = m / p.group;
            const char *q = reinterpret_cast<const char *>(static_cast<const uint16_t *>(p.q) + tok * p.q_ts +
                                                           (idx / rb % p.nkv * p.group + m - tok * p.group) * p.q_hs);
            if (tok < p.R * p.q_len)
                for (int c = 0; c < 2 * D; c += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(q + c));
        }
        Work work(p, length(), w);
        PaItem it;
        PaRing<NS> ring(w, pair());
        int blk = 0, items = 0;
        const uint64_t cc = f2_pack(p.scale_log2, p.scale_log2);
        while (work.next(it)) {
            const int n = it.kb1 - it.kb0;
            if (it.rows <= 0) {
                ring.n += n;
                continue;
            }
            const bool active = 32 * wq < it.rows, valid = row < it.rows;
            const int m = it.row0 + row, tok = m / p.group, head = it.g * p.group + m - tok * p.group;
            const int64_t grow = (int64_t)(it.tok0 + tok) * p.q_heads + head;   // output row
            if (active) {   // the previous item is done: its Q is no longer read
                const uint4 *src = reinterpret_cast<const uint4 *>(
                    static_cast<const uint16_t *>(p.q) + (it.tok0 + tok) * p.q_ts + head * p.q_hs);
                uint4 v[D / 8];
#pragma unroll
                for (int c = 0; c < D / 8; ++c) v[c] = valid ? pa_load(src + c, kOwn) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                for (int c = 0; c < D / 8; ++c)
                    *reinterpret_cast<uint4 *>(sq + (c / 8) * (kPaTile * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4)) = v[c];
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            }
            mbar_arrive(sb + LY.qready + 8 * w);
            // S of block j: the item's keys in it
            const auto scores = [&](int j) {
                wait(LY.sfull + 8 * w, blk);
                __syncwarp();
                tc_fence_after();
                int keys = KB;
                if (j == n - 1 && it.keys < it.kb1 * KB) {
                    keys = it.keys - (it.kb1 - 1) * KB;
                    zero_tail(ring, keys, row);
                }
                ++ring.n;
                return keys;
            };
            const auto arrive = [&](uint32_t bar) {   // for this warp, which has left tensor memory
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(sb + bar);
            };
            // (two barriers in turn: S of block b says that the weights of block
            // b - 2 have been multiplied, so that phase has been seen)
            const auto pready = [&](int b) { return LY.pready + 16 * (b & 1) + 8 * w; };
            float mu = -INFINITY, l = 0.f;
            uint32_t so[U], sm[U];
            int keys = KB, outer = 0;   // of the block; the half of the keys in the outer unit
            // The weights of block j, against the maximum so far.  Later scores
            // may exceed it as long as a block's weights stay below a limit in sum
            // (so no maximum is taken per block); otherwise it follows and O is
            // rescaled.  An item's first block starts there.
            const auto weigh = [&](int j) {
                const uint32_t aOut = aSP + 2 * outer * U;
                uint32_t po[U / 2], pm[U / 2];
                int left = keys;   // keys of the block that the row sees
                if (kOwn && valid) left = min(left, it.limit0 + it.step * tok - (it.kb0 + j) * KB);
                const bool hide = kOwn ? __any_sync(0xffffffffu, left < KB) : left < KB;
                if (hide) {
                    pa_hide(so, left - outer * U);
                    pa_hide(sm, left - (outer ^ 1) * U);
                }
                float base = -mu, sum = INFINITY;
                for (bool again = false;; again = true) {
                    if (again || j > 0) {
                        sum = pa_weights<E>(so, po, cc, base);
                        sum += pa_weights<E>(sm, pm, cc, base);
                        if (again || !__any_sync(0xffffffffu, !(sum < PaWeight<E>::most))) break;
                        pa_load_scores<U>(aOut, so);   // not overwritten yet
                        pa_loaded(so);
                        if (hide) pa_hide(so, left - outer * U);
                    }
                    // (only this row's own scores move it, not a neighbour's)
                    const float top = fmaf(pa_max(so, pa_max(sm, -INFINITY)), p.scale_log2, -PaWeight<E>::below);
                    const bool grew = top > mu && !(sum < PaWeight<E>::most);
                    const float al = grew ? a2_ex2(mu - top) : 1.f;
                    if (grew) mu = top;
                    base = mu == -INFINITY ? 0.f : -mu;
                    l *= al;
                    if (j > 0) {
                        wait(LY.pvdone + 8 * w, blk - 1);
                        __syncwarp();
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < D; c += 16) {
                            uint32_t o[16];
                            tmem_ld_x16(aO + c, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * al);
                            pa_tmem_st16(aO + c, o);
                        }
                    }
                }
                l += sum;
                pa_tmem_st<U / 2>(aOut + outer * (U / 2), po);
                pa_tmem_st<U / 2>(aOut + (outer ^ 1) * (U / 2), pm);
            };
            const auto load = [&]() {
                pa_issue_scores<U>(aSP + 2 * outer * U, so, aSP + U, sm);
            };
            const auto loaded = [&]() {
                tmem_ld_wait();
                pa_loaded(so);
                pa_loaded(sm);
                arrive(LY.sfree + 8 * w);
            };
            if (kAhead && active) {
                keys = scores(0);
                outer = blk & 1;
                load();
                loaded();
                for (int j = 0;; ++j) {
                    weigh(j);
                    const uint32_t ready = pready(blk++);
                    if (j == n - 1) {
                        pa_tmem_st_wait();
                        arrive(ready);
                        break;
                    }
                    keys = scores(j + 1);
                    outer ^= 1;
                    load();   // on its way to registers while the weights land
                    pa_tmem_st_wait();
                    arrive(ready);
                    loaded();
                }
            } else {
                for (int j = 0; j < n; ++j, ++blk) {
                    keys = scores(j);
                    outer = blk & 1;
                    if (active) {
                        load();
                        loaded();
                        weigh(j);
                        pa_tmem_st_wait();
                    } else {
                        arrive(LY.sfree + 8 * w);
                    }
                    arrive(pready(blk));
                }
            }
            // (not on pvdone, whose last two phases may both be open)
            wait(LY.odone + 8 * w, items++);
            __syncwarp();
            if (active && !__any_sync(0xffffffffu, dead())) {
                tc_fence_after();
                float *dst = p.ws_o + ((int64_t)it.split * p.rows + grow) * D;
                const bool dropped = kOwn && flags()[3 + w];
#pragma unroll
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[32];
                    pa_tmem_ld32(aO + c, o);
                    tmem_ld_wait();
                    if (kOwn && dropped) {
                        const int end = min(min(it.keys, it.kb1 * KB), valid ? it.limit0 + it.step * tok : 0);
#pragma unroll 1
                        for (int key = max(it.all, it.kb0 * KB); key < end; ++key) {
                            const uint32_t *v = pa_value_row<D>(p, it, key);
                            if (!v) continue;
#pragma unroll
                            for (int e = 0; e < 32; e += 2) {
                                float a = __uint_as_float(o[e]), b = __uint_as_float(o[e + 1]);
                                pa_add_not_finite<E>(__ldcg(v + (c + e) / 2), a, b);
                                o[e] = __float_as_uint(a);
                                o[e + 1] = __float_as_uint(b);
                            }
                        }
                        __syncwarp();
                    }
                    if (valid)
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            __stcg(reinterpret_cast<uint4 *>(dst + c + e), make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]));
                }
                tc_fence_before();
                // a sum below zero: a page outside the cache, which voids every row
                if (valid) __stcg(p.ws_ml + grow * (p.sp + p.ss) + it.split, make_float2(mu, bad(w) ? -1.f : l));
            }
        }
    }

    // The V rows of an item's last page behind its keys (of `keys` in the
    // block): whatever they hold must not meet a zero weight
    __device__ __forceinline__ void zero_tail(PaRing<NS> ring, int keys, int row) const
    {
        const int s0 = keys & (kPageSlots - 1), pg = keys / kPageSlots;
        if (s0 == 0) return;
        ring.take();
        wait(LY.full + 8 * ring.st, ring.use);
        uint8_t *page = smem + LY.ring + ring.st * Sh::stage_bytes + pg * Sh::page_bytes;
        for (int c = row; c < (kPageSlots - s0) * (D / 8); c += 128) {
            const int s = s0 + c / (D / 8), ch = c % (D / 8);
            *reinterpret_cast<uint4 *>(page + (s >> 3) * (Sh::nblk * 1024) + (D / 64 + ch / 8) * 1024 + (s & 7) * 128 +
                                       (ch & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
    }
};

template <class E, int D, bool kOwn>
__global__ void __launch_bounds__(kPaThreads, 1)
    prefix_tile_kernel(const __grid_constant__ CUtensorMap tmKV, const __grid_constant__ PrefixParams p)
{
    using Sh = PaShape<D>;
    constexpr PaSmem LY = pa_smem<D>();
    extern __shared__ uint8_t pa_smem_dyn[];
    uint8_t *smem = pa_smem_dyn + ((1024u - (smem_u32(pa_smem_dyn) & 1023u)) & 1023u);
    const uint32_t sb = smem_u32(smem);
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;

    // The own keys' CTAs behind the prefix's: as in the rows kernel, every input
    // is in L2 and read past L1, and only the grid as a whole must not end before
    // that one.
    const bool behind = kOwn && p.prefix_blocks > 0, last = blockIdx.x == gridDim.x - 1;
    if (kOwn) {
        if (threadIdx.x == 0) griddep_launch_dependents();
        if (!behind) griddep_wait();
        PaItem it;
        const int P = pa_prefix_len(p, kOwn);
        const bool any = PaWork<D, kOwn>(p, P, 0).next(it) | PaWork<D, kOwn>(p, P, 1).next(it);
        if (!any) {   // requests without keys
            if (behind && last) griddep_wait();
            return;
        }
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2 * Sh::slots; ++i) {
            mbar_init(sb + LY.full + 8 * i, 1);
            mbar_init(sb + LY.empty + 8 * i, !kOwn && p.pair ? 2 : 1);   // the groups that read the stage
        }
        for (int w = 0; w < 2; ++w) {
            mbar_init(sb + LY.qready + 8 * w, 128);
            mbar_init(sb + LY.sfull + 8 * w, 1);
            mbar_init(sb + LY.sfree + 8 * w, 4);
            mbar_init(sb + LY.pready + 8 * w, 4);
            mbar_init(sb + LY.pready + 16 + 8 * w, 4);
            mbar_init(sb + LY.pvdone + 8 * w, 1);
            mbar_init(sb + LY.odone + 8 * w, kOwn ? 2 : 1);
            mbar_init(sb + LY.drain + 8 * w, 1);
        }
        // a wait gave up; a page outside the cache, by producer; values not finite
        // among keys that not every row sees, by group
        for (int i = 0; i < (kOwn ? 5 : 3); ++i) reinterpret_cast<volatile int *>(smem + LY.flags)[i] = 0;
        fence_barrier_init();
    }
    // all of tensor memory (one CTA per SM): it starts at column 0
    if (warp == 0) a2_tmem_alloc<Sh::cols>(sb + LY.tmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (!kOwn) {
        griddep_wait();   // every input comes from the kernels before this one
        // released only now: the kernel behind this one reads the same inputs
        // without a wait of its own
        if (threadIdx.x == 0) griddep_launch_dependents();
    }
    const PaTile<E, D, kOwn> tile{&tmKV, p, smem, sb, lane};
    // a softmax thread holds a row's whole S: its groups take registers from the
    // other warpgroup (256 x 208 + 128 x 88 = 384 x 168, what the launch has)
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        tile.softmax(warp >> 2, warp & 3);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (warp < 10)
            tile.produce(warp - 8);
        else if (warp == 10)
            tile.template multiply<0>();
        else
            tile.template multiply<1>();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) a2_tmem_dealloc<Sh::cols>(0u);
    if (behind && last) griddep_wait();
}

// ---- few rows: mma.sync over small CTAs ------------------------------------
//
// A tile of 16 or 64 rows against a range of its own key blocks: four warps
// and a producer per CTA, several CTAs per SM, so that many short key lists
// are in flight at once.  16 rows: warp w takes page w of each 64-key stage
// and the four partials are joined in shared memory; 64 rows: warp w takes
// rows 16 w .. against every page.

constexpr int kPrThreads = 160;
static_assert(kPlanPage == kPageSlots, "prefix_plan.h");

template <int D>
struct PrShape {
    static constexpr int slots = D == 64 ? 3 : 2;
    static constexpr int nblk = 2 * D / 64;
    static constexpr uint32_t page_bytes = kPageSlots * 4 * D;
    static constexpr uint32_t stage_bytes = kPrPages * page_bytes;
    static constexpr uint32_t ring_bytes = slots * stage_bytes;
    // barriers full and empty, one of values cleared, pages outside the cache by
    // stage, two flags: a wait gave up, values were cleared
    static constexpr uint32_t smem = ring_bytes + slots * 20 + 16 + 1024;
    static constexpr int ostride = D + 4;   // floats per row of a warp's partial, over the ring
    static_assert(4 * 16 * (ostride + 2) * 4 <= ring_bytes, "the warps' partials fit the ring");
};

template <int D, int RT>
constexpr int pr_ctas_per_sm()
{
    return RT == 16 ? (D == 64 ? 4 : 3) : (D == 64 ? 3 : 2);
}

template <class E>
__device__ __forceinline__ void pr_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if constexpr (E::is_bf16)
        mma_bf16_16816(d, a[0], a[1], a[2], a[3], b0, b1);
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
            "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Whether the tile kernel runs in front of the rows kernel
__device__ __forceinline__ bool pr_behind(const PrefixParams &p) { return !p.small && p.prefix_blocks > 0; }

// One item against its key blocks: RT = 16 or 64 rows.  kTokens: some rows may
// see fewer keys than others (requests of several tokens; without the code for
// that 64 requests' own keys take 21.2 us instead of 21.4, and with a 32K prefix
// 54.5 instead of 55.5).
template <class E, int D, int RT, bool kTokens>
__device__ __forceinline__ void pr_item(const CUtensorMap &tmKV, const PrefixParams &p, const PaItem &it, int first_entry,
                                        uint8_t *smem)
{
    using Sh = PrShape<D>;
    constexpr int NS = Sh::slots, NP = RT == 16 ? 1 : kPrPages;
    const uint32_t sb = smem_u32(smem), full0 = sb + Sh::ring_bytes, empty0 = full0 + 8 * NS, cleared = empty0 + 8 * NS;
    volatile int *slot_bad = reinterpret_cast<volatile int *>(smem + Sh::ring_bytes + 16 * NS + 8);
    volatile int *flags = slot_bad + NS;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const auto wait = [&](uint32_t bar, int n) {
        return mbar_try_wait(bar, (uint32_t)n & 1) || bounded_wait(bar, (uint32_t)n & 1, flags, p.wait_limit_ns, true);
    };
    const int g = it.g;
    const int32_t *pages = it.pages;
    const int n = it.kb1 - it.kb0;   // stages
    const int pg0 = it.kb0 * kPrPages;
    const int pg1 = min(it.kb1 * kPrPages, (it.keys + kPageSlots - 1) / kPageSlots);

    const int gq = lane >> 2, t = lane & 3;
    float o[D / 8][4], m_a = -INFINITY, m_b = -INFINITY, l_a = 0.f, l_b = 0.f;
    int bad = 0;
    bool ok = true;
    const int row_a = (RT == 64 ? 16 * warp : 0) + gq, row_b = row_a + 8;
    if (warp == 4) {
        // ---- produce ---------------------------------------------------------
        const uint64_t policy = policy_evict_first();   // these keys are read once
        unsigned bad_any = 0u;
        bool stop = false;
        int j = 0;
        int next = pg0 + lane < pg1 ? (pg0 == 0 ? first_entry : __ldcg(pages + pg0 + lane)) : 0;
        for (int c = pg0; c < pg1 && !stop; c += 32) {
            int page = next;
            if (c + 32 + lane < pg1) next = __ldcg(pages + c + 32 + lane);
            bool wrong = false;
            if (c + lane < pg1 && (page < 0 || page >= p.num_pages)) {   // flagged, page 0 in its place
                wrong = true;
                page = 0;
            }
            const unsigned bads = __ballot_sync(0xffffffffu, wrong);
            bad_any |= bads;
            for (int b0 = c; b0 < min(c + 32, pg1); b0 += kPrPages, ++j) {
                const int st = j % NS, use = j / NS, np_ = min(kPrPages, pg1 - b0);
                int okl = 1;
                if (lane == 0) {
                    okl = use == 0 || wait(empty0 + 8 * st, use - 1);
                    if (okl) {
                        slot_bad[st] = (bads >> (b0 - c)) & 15u;
                        mbar_expect_tx(full0 + 8 * st, (uint32_t)np_ * Sh::page_bytes);
                    }
                }
                if (!__shfl_sync(0xffffffffu, okl, 0)) {
                    stop = true;
                    break;
                }
                const int i = c + lane - b0;
                if (i >= 0 && i < np_)
                    tma_load_page(sb + st * Sh::stage_bytes + i * Sh::page_bytes, &tmKV, full0 + 8 * st, page * p.nkv + g, policy);
            }
        }
        if (lane == 0) {
            if (bad_any) atomicOr(&g_status, QKVF_STATUS_BAD_REQUEST);
            if (flags[0])
                for (int k = max(0, j - NS); k < j; ++k)
                    bounded_wait(full0 + 8 * (k % NS), (uint32_t)((k / NS) & 1), flags, p.wait_limit_ns, false);
        }
        __syncwarp();
    } else {
        // ---- compute: rows gq and gq + 8 of the warp's 16, mma.sync layout ----
        const int ma = it.row0 + row_a, mb = it.row0 + row_b, ta = ma / p.group, tb = mb / p.group;
        const bool va = row_a < it.rows, vb = row_b < it.rows;
        uint32_t qa[D / 16][4];
        const bool past = pr_behind(p);
        {
            const uint16_t *qp = static_cast<const uint16_t *>(p.q);
            const uint16_t *pa = qp + (it.tok0 + ta) * p.q_ts + (g * p.group + ma - ta * p.group) * p.q_hs + 2 * t;
            const uint16_t *pb = qp + (it.tok0 + tb) * p.q_ts + (g * p.group + mb - tb * p.group) * p.q_hs + 2 * t;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                qa[k][0] = va ? pa_load(reinterpret_cast<const uint32_t *>(pa + 16 * k), past) : 0u;
                qa[k][1] = vb ? pa_load(reinterpret_cast<const uint32_t *>(pb + 16 * k), past) : 0u;
                qa[k][2] = va ? pa_load(reinterpret_cast<const uint32_t *>(pa + 16 * k + 8), past) : 0u;
                qa[k][3] = vb ? pa_load(reinterpret_cast<const uint32_t *>(pb + 16 * k + 8), past) : 0u;
            }
        }
#pragma unroll
        for (int d = 0; d < D / 8; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[d][e] = 0.f;
        const int lim_a = it.limit0 + it.step * ta, lim_b = it.limit0 + it.step * tb;
        const bool rows_here = RT == 16 || 16 * warp < it.rows;
        // the first stage with keys that some rows do not see
        const int partly_from = kTokens && it.all < it.keys ? max(it.all, 0) / kPrKeys - it.kb0 : n;
        for (int j = 0; j < n; ++j) {
            const int st = j % NS;
            ok = __all_sync(0xffffffffu, wait(full0 + 8 * st, j / NS));
            if (!ok) break;
            bad |= slot_bad[st];
            const int left = pg1 - pg0 - j * kPrPages;   // pages from this stage on
            if (kTokens && j >= partly_from) {
                uint8_t *stage = smem + st * Sh::stage_bytes;
                const int k0 = (it.kb0 + j) * kPrKeys, k1 = k0 + warp * kPageSlots;
                // the warp's page; where the other warps read it too, all of them look through
                // the stage, and find the same, before any changes it (two phases a stage)
                const bool clear = RT == 16 || pa_find_not_finite<E, D, false>(stage, max(it.all - k0, 0), min(it.keys - k0, kPrKeys));
                if (RT == 64 && clear) {
                    if (lane == 0) mbar_arrive(cleared);
                    ok = __all_sync(0xffffffffu, wait(cleared, 0));
                    if (!ok) break;
                }
                if (clear && pa_find_not_finite<E, D, true>(stage + warp * Sh::page_bytes, max(it.all - k1, 0), min(it.keys - k1, kPageSlots)))
                    flags[1] = 1;
                if (RT == 64 && clear) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(cleared);
                    ok = __all_sync(0xffffffffu, wait(cleared, 1));
                    if (!ok) break;
                }
            }
            const int b_lo = RT == 16 ? warp : 0;         // the warp's pages of the stage: b_lo ..
            if (rows_here && b_lo < left) {
                const uint32_t base = sb + st * Sh::stage_bytes + b_lo * Sh::page_bytes;
                const int key0 = (it.kb0 + j) * kPrKeys + b_lo * kPageSlots;
                float sc[2 * NP][4];
#pragma unroll
                for (int b = 0; b < NP; ++b) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int e = 0; e < 4; ++e) sc[2 * b + h][e] = 0.f;
                    if (b < left)
#pragma unroll
                        for (int k = 0; k < D / 16; ++k) {
                            const int ch = 2 * k + ((lane >> 3) & 1);   // 8-dim chunk; key lane % 8 (+ 8 for lanes 16 ..)
                            uint32_t b0, b1, b2, b3;
                            ldsm_x4(base + b * Sh::page_bytes + (lane >> 4) * (Sh::nblk * 1024) + (ch >> 3) * 1024 +
                                        (lane & 7) * 128 + (((ch & 7) ^ (lane & 7)) << 4),
                                    b0, b1, b2, b3);
                            pr_mma<E>(sc[2 * b], qa[k], b0, b1);
                            pr_mma<E>(sc[2 * b + 1], qa[k], b2, b3);
                        }
                }
                if (__any_sync(0xffffffffu, min(lim_a, lim_b) < key0 + NP * kPageSlots))
#pragma unroll
                    for (int b = 0; b < 2 * NP; ++b)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (key0 + 8 * b + 2 * t + (e & 1) >= (e >= 2 ? lim_b : lim_a)) sc[b][e] = -INFINITY;
                float mx_a = -INFINITY, mx_b = -INFINITY;
#pragma unroll
                for (int b = 0; b < 2 * NP; ++b) {
                    mx_a = fmaxf(fmaxf(mx_a, sc[b][0]), sc[b][1]);
                    mx_b = fmaxf(fmaxf(mx_b, sc[b][2]), sc[b][3]);
                }
#pragma unroll
                for (int off = 1; off <= 2; off <<= 1) {
                    mx_a = fmaxf(mx_a, __shfl_xor_sync(0xffffffffu, mx_a, off));
                    mx_b = fmaxf(mx_b, __shfl_xor_sync(0xffffffffu, mx_b, off));
                }
                const float mn_a = fmaxf(m_a, fmaf(mx_a, p.scale_log2, -PaWeight<E>::below)),
                            mn_b = fmaxf(m_b, fmaf(mx_b, p.scale_log2, -PaWeight<E>::below));
                const float base_a = mn_a == -INFINITY ? 0.f : mn_a, base_b = mn_b == -INFINITY ? 0.f : mn_b;
                if (__any_sync(0xffffffffu, mn_a != m_a || mn_b != m_b)) {
                    const float al_a = a2_ex2(m_a - base_a), al_b = a2_ex2(m_b - base_b);
                    l_a *= al_a;
                    l_b *= al_b;
#pragma unroll
                    for (int d = 0; d < D / 8; ++d) {
                        o[d][0] *= al_a;
                        o[d][1] *= al_a;
                        o[d][2] *= al_b;
                        o[d][3] *= al_b;
                    }
                    m_a = mn_a;
                    m_b = mn_b;
                }
#pragma unroll
                for (int b = 0; b < 2 * NP; ++b) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[b][e] = a2_ex2(fmaf(sc[b][e], p.scale_log2, e >= 2 ? -base_b : -base_a));
                    l_a += sc[b][0] + sc[b][1];
                    l_b += sc[b][2] + sc[b][3];
                }
#pragma unroll
                for (int b = 0; b < NP; ++b)
                    if (b < left) {
                        const uint32_t pf[4] = {E::pack(sc[2 * b][0], sc[2 * b][1]), E::pack(sc[2 * b][2], sc[2 * b][3]),
                                                E::pack(sc[2 * b + 1][0], sc[2 * b + 1][1]), E::pack(sc[2 * b + 1][2], sc[2 * b + 1][3])};
                        // V rows behind the keys, whatever they hold, must not
                        // meet a zero weight: b0 / b2 hold keys 2t, 2t + 1 of
                        // the page, b1 / b3 keys 8 + 2t, 9 + 2t
                        const int in = it.keys - (key0 + b * kPageSlots);
                        uint32_t m0 = 0xffffffffu, m1 = 0xffffffffu;
                        if (in < kPageSlots) {
                            m0 = (2 * t < in ? 0xffffu : 0u) | (2 * t + 1 < in ? 0xffff0000u : 0u);
                            m1 = (2 * t + 8 < in ? 0xffffu : 0u) | (2 * t + 9 < in ? 0xffff0000u : 0u);
                        }
#pragma unroll
                        for (int k = 0; k < D / 16; ++k) {
                            const int ch = 2 * k + (lane >> 4);   // key lane % 8 (+ 8 for lanes 8 .. 15, 24 ..)
                            uint32_t b0, b1, b2, b3;
                            ldsm_x4_trans(base + b * Sh::page_bytes + ((lane >> 3) & 1) * (Sh::nblk * 1024) +
                                              (D / 64 + (ch >> 3)) * 1024 + (lane & 7) * 128 + (((ch & 7) ^ (lane & 7)) << 4),
                                          b0, b1, b2, b3);
                            pr_mma<E>(o[2 * k], pf, b0 & m0, b1 & m1);
                            pr_mma<E>(o[2 * k + 1], pf, b2 & m0, b3 & m1);
                        }
                    }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty0 + 8 * st);
        }
        if (kTokens && partly_from < n && __any_sync(0xffffffffu, flags[1] != 0)) {
            const int end = min(it.keys, it.kb1 * kPrKeys);
#pragma unroll 1
            for (int key = max(it.all, it.kb0 * kPrKeys); key < end; ++key) {
                if (RT == 16 && (key / kPageSlots) % kPrPages != warp) continue;   // another warp's page
                const uint32_t *v = pa_value_row<D>(p, it, key);
                if (!v) continue;
#pragma unroll
                for (int d = 0; d < D / 8; ++d) {
                    const uint32_t x = __ldcg(v + 4 * d + t);
                    if (key < lim_a) pa_add_not_finite<E>(x, o[d][0], o[d][1]);
                    if (key < lim_b) pa_add_not_finite<E>(x, o[d][2], o[d][3]);
                }
            }
        }
#pragma unroll
        for (int off = 1; off <= 2; off <<= 1) {
            l_a += __shfl_xor_sync(0xffffffffu, l_a, off);
            l_b += __shfl_xor_sync(0xffffffffu, l_b, off);
        }
    }
    const int64_t head0 = (int64_t)it.tok0 * p.q_heads + (int64_t)g * p.group;
    const auto out_row = [&](int row) {   // output row of row `row` of the tile
        const int m = it.row0 + row, tok = m / p.group;
        return head0 + (int64_t)tok * p.q_heads + (m - tok * p.group);
    };
    float *ws = p.ws_o + (int64_t)it.split * p.rows * D;
    const int splits = p.sp + p.ss;
    if constexpr (RT == 64) {
        if (warp < 4 && ok) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int row = half ? row_b : row_a;
                if (row < it.rows) {
                    const int64_t gr = out_row(row);
#pragma unroll
                    for (int d = 0; d < D / 8; ++d)
                        __stcg(reinterpret_cast<float2 *>(ws + gr * D + 8 * d + 2 * t), make_float2(o[d][2 * half], o[d][2 * half + 1]));
                    if (t == 0) __stcg(p.ws_ml + gr * splits + it.split, make_float2(half ? m_b : m_a, bad ? -1.f : (half ? l_b : l_a)));
                }
            }
        }
    } else {
        // join the four warps' partials over the drained ring, in warp order
        __syncthreads();
        float *part = reinterpret_cast<float *>(smem), *ml = part + 4 * 16 * Sh::ostride;
        if (warp < 4) {
            float *mine = part + warp * 16 * Sh::ostride;
#pragma unroll
            for (int d = 0; d < D / 8; ++d) {
                *reinterpret_cast<float2 *>(mine + gq * Sh::ostride + 8 * d + 2 * t) = make_float2(o[d][0], o[d][1]);
                *reinterpret_cast<float2 *>(mine + (gq + 8) * Sh::ostride + 8 * d + 2 * t) = make_float2(o[d][2], o[d][3]);
            }
            if (t == 0) {
                *reinterpret_cast<float2 *>(ml + 2 * (16 * warp + gq)) = make_float2(m_a, l_a);
                *reinterpret_cast<float2 *>(ml + 2 * (16 * warp + gq + 8)) = make_float2(m_b, l_b);
            }
        }
        __syncthreads();
        const int row = threadIdx.x >> 3, c = threadIdx.x & 7;   // 8 threads a row
        if (row < it.rows && row < 16 && !flags[0]) {
            float f[4], M = -INFINITY, l = 0.f;
#pragma unroll
            for (int w = 0; w < 4; ++w) M = fmaxf(M, ml[2 * (16 * w + row)]);
            const float base = M == -INFINITY ? 0.f : M;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                f[w] = a2_ex2(ml[2 * (16 * w + row)] - base);
                l = fmaf(ml[2 * (16 * w + row) + 1], f[w], l);
            }
            const int64_t gr = out_row(row);
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const float4 v = *reinterpret_cast<const float4 *>(part + (16 * w + row) * Sh::ostride + 32 * k + 4 * c);
                    x.x = fmaf(v.x, f[w], x.x);
                    x.y = fmaf(v.y, f[w], x.y);
                    x.z = fmaf(v.z, f[w], x.z);
                    x.w = fmaf(v.w, f[w], x.w);
                }
                __stcg(reinterpret_cast<float4 *>(ws + gr * D + 32 * k + 4 * c), x);
            }
            if (c == 0) __stcg(p.ws_ml + gr * splits + it.split, make_float2(M, bad ? -1.f : l));
        }
    }
}

// Prefix items (where the prefix's rows are few: p.small) in tiles of RTP
// rows, then the requests' own keys in tiles of RTO.
template <class E, int D, int RTP, int RTO, bool kTokens>
__global__ void __launch_bounds__(kPrThreads, pr_ctas_per_sm<D, (RTP > RTO ? RTP : RTO)>())
    prefix_rows_kernel(const __grid_constant__ CUtensorMap tmKV, const __grid_constant__ PrefixParams p)
{
    using Sh = PrShape<D>;
    constexpr int NS = Sh::slots;
    extern __shared__ uint8_t pr_smem_dyn[];
    uint8_t *smem = pr_smem_dyn + ((1024u - (smem_u32(pr_smem_dyn) & 1023u)) & 1023u);
    const uint32_t full0 = smem_u32(smem) + Sh::ring_bytes, empty0 = full0 + 8 * NS;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(full0 + 8 * i, 1);
            mbar_init(empty0 + 8 * i, 4);
        }
        mbar_init(empty0 + 8 * NS, 4);
        for (int i = 0; i < 2; ++i) reinterpret_cast<volatile int *>(smem + Sh::ring_bytes + 16 * NS + 8)[NS + i] = 0;
        fence_barrier_init();
        griddep_launch_dependents();
    }
    __syncthreads();
    // Behind the tile kernel every input is already in L2 (that kernel has
    // waited for the kernels that write it before this one could start), and
    // only the grid as a whole must not end before it: the last CTA waits, at
    // its end.  A CTA without a wait of its own may find an older copy of a line
    // in its SM's L1, so q, the lengths and the tables are read past it (keys
    // come by TMA, from L2).
    const bool behind = pr_behind(p);
    if (!behind) griddep_wait();

    int idx = blockIdx.x;
    const int np = p.small && p.prefix_blocks > 0 ? p.nkv * p.sp : 0;
    const bool own = idx >= np;
    idx -= own ? np : 0;
    const int g = idx % p.nkv, rest = idx / p.nkv;
    const int r = own ? rest % p.R : 0, ts = own ? rest / p.R : 0;
    const int tile = own ? ts % p.own_tiles : 0, split = own ? ts / p.own_tiles : rest;
    const int32_t *pages = own ? p.block_table + (size_t)r * p.max_blocks : p.prefix_pages;
    // the first split starts at page 0: its entries need not wait for a length
    int first_entry = 0;
    if (warp == 4 && split == 0 && lane < (own ? p.max_blocks : p.prefix_blocks)) first_entry = __ldcg(pages + lane);
    const int P = pa_prefix_len(p, true), L = own ? __ldcg(p.context_lens + r) : 0;
    const PaItem it = own ? pa_own_item<kPrKeys>(p, P, L, r, tile, g, split) : pa_prefix_item<kPrKeys>(p, max(P, 0), RTP, 0, g, split);
    if (it.kb1 > it.kb0) {
        if constexpr (RTP == RTO) {
            pr_item<E, D, RTO, kTokens>(tmKV, p, it, first_entry, smem);
        } else {
            if (own)
                pr_item<E, D, RTO, kTokens>(tmKV, p, it, first_entry, smem);
            else
                pr_item<E, D, RTP, false>(tmKV, p, it, first_entry, smem);
        }
    }
    if (behind && blockIdx.x == gridDim.x - 1) griddep_wait();
}

// Joins a row's partials: kWarps warps a row, D / 4 lanes a partial, the
// partials dealt round robin.  The lengths, the maxima and sums and the first
// partials' O are loaded side by side, before it is known which of the slots
// hold keys (the others' contents are not used).  Sums in a fixed order: the
// same bits every time.
constexpr int kPaMergeAhead = 6;   // partials in flight per lane

__host__ __device__ constexpr int pa_merge_threads(int warps) { return warps > 4 ? 32 * warps : 128; }

template <class E, int D, int kWarps>
__global__ void __launch_bounds__(pa_merge_threads(kWarps)) prefix_merge_kernel(const __grid_constant__ PrefixParams p)
{
    constexpr int LPR = D / 4, PAR = kWarps * 32 / LPR, kRows = pa_merge_threads(kWarps) / (32 * kWarps);
    __shared__ float weight[kRows][2 * kPaMaxSplits];
    __shared__ float4 part[kRows][kWarps][32];
    if (threadIdx.x == 0) griddep_launch_dependents();
    griddep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rl = warp / kWarps, wr = warp % kWarps;   // the row of the CTA, the warp of the row
    const int row = blockIdx.x * kRows + rl;
    if (kWarps == 1 && row >= p.rows) return;   // (with more warps the CTA is one row)
    const int t = row / p.q_heads, h = row - t * p.q_heads, r = p.q_len == 1 ? t : t / p.q_len;
    const int slots = p.sp + p.ss;
    const float2 *ml = p.ws_ml + (int64_t)row * slots;
    const int first = wr * (32 / LPR) + lane / LPR, d = lane % LPR;   // this lane's first slot, its 4 columns
    const float4 *src = reinterpret_cast<const float4 *>(p.ws_o + (int64_t)row * D) + d;
    const int64_t step = (int64_t)p.rows * (D / 4);
    const int P = pa_prefix_len(p, false), L = p.context_lens[r];
    float2 v[2 * kPaMaxSplits / 32];
#pragma unroll
    for (int i = 0; i < 2 * kPaMaxSplits / 32; ++i)
        if (lane + 32 * i < slots) v[i] = __ldcg(ml + lane + 32 * i);
    float4 x[kPaMergeAhead];
#pragma unroll
    for (int i = 0; i < kPaMergeAhead; ++i)
        if (first + i * PAR < slots) x[i] = __ldcg(src + (first + i * PAR) * step);
    const auto skip = [&]() {
        if (p.zero && wr == 0 && lane < LPR)
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + (int64_t)row * D + 4 * d) = make_uint2(0u, 0u);
    };
    if (L < 0 && P >= 0) return skip();   // a padding request
    if (P < 0 || L > p.max_blocks * kPageSlots) {
        if (lane == 0 && wr == 0) atomicOr(&g_status, QKVF_STATUS_BAD_REQUEST);
        return skip();
    }
    const int own = pa_own_keys(p, L, p.own_tiles == 1 ? 0 : ((t - r * p.q_len) * p.group + h % p.group) / p.own_rows);
    const int pkeys = p.small ? kPrKeys : PaShape<D>::keys;
    const int okeys = p.own_tile ? PaShape<D>::keys : kPrKeys;
    const int np = min(p.sp, (P + pkeys - 1) / pkeys), no = p.sp + min(p.ss, (own + okeys - 1) / okeys);
    const auto holds = [&](int s) { return s < np || (s >= p.sp && s < no); };
    float M = -INFINITY;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 2 * kPaMaxSplits / 32; ++i)
        if (32 * i < slots) {
            if (!holds(lane + 32 * i)) v[i] = make_float2(-INFINITY, 0.f);
            M = fmaxf(M, v[i].x);
            bad |= v[i].y < 0.f;
        }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    if (__any_sync(0xffffffffu, bad)) return skip();   // a page outside the cache
    const float base = M == -INFINITY ? 0.f : M;
    float l = 0.f;
#pragma unroll
    for (int i = 0; i < 2 * kPaMaxSplits / 32; ++i)
        if (32 * i < slots) {
            const float f = exp2f(v[i].x - base);
            if (wr == 0) weight[rl][lane + 32 * i] = f;
            l = fmaf(v[i].y, f, l);
        }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
    if (kWarps == 1)
        __syncwarp();
    else
        __syncthreads();
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = first; s0 < slots; s0 += kPaMergeAhead * PAR) {
        if (s0 != first)
#pragma unroll
            for (int i = 0; i < kPaMergeAhead; ++i)
                if (holds(s0 + i * PAR)) x[i] = __ldcg(src + (s0 + i * PAR) * step);
#pragma unroll
        for (int i = 0; i < kPaMergeAhead; ++i)
            if (holds(s0 + i * PAR)) {
                const float f = weight[rl][s0 + i * PAR];
                o.x = fmaf(x[i].x, f, o.x);
                o.y = fmaf(x[i].y, f, o.y);
                o.z = fmaf(x[i].z, f, o.z);
                o.w = fmaf(x[i].w, f, o.w);
            }
    }
    if constexpr (LPR == 16) {
        o.x += __shfl_xor_sync(0xffffffffu, o.x, 16);
        o.y += __shfl_xor_sync(0xffffffffu, o.y, 16);
        o.z += __shfl_xor_sync(0xffffffffu, o.z, 16);
        o.w += __shfl_xor_sync(0xffffffffu, o.w, 16);
    }
    if constexpr (kWarps > 1) {
        part[rl][wr][lane] = o;
        __syncthreads();
        if (wr > 0) return;
#pragma unroll
        for (int w = 1; w < kWarps; ++w) {
            const float4 y = part[rl][w][lane];
            o.x += y.x;
            o.y += y.y;
            o.z += y.z;
            o.w += y.w;
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const uint2 y = l == 0.f ? make_uint2(0u, 0u) : make_uint2(E::pack(o.x * inv, o.y * inv), E::pack(o.z * inv, o.w * inv));
    if (lane < LPR) *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + (int64_t)row * D + 4 * d) = y;
    if (p.lse && lane == 0) p.lse[row] = l == 0.f ? -INFINITY : (base + log2f(l)) * 0.6931471805599453f;
}

// ---- host: launch (splits and workspace: prefix_plan.h) ---------------------

template <class E, int D, int RTP, int RTO>
bool prepare_rows_kernel()
{
    constexpr auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
    return cudaFuncSetAttribute((const void *)prefix_rows_kernel<E, D, RTP, RTO, false>, attr, (int)PrShape<D>::smem) == cudaSuccess &&
           cudaFuncSetAttribute((const void *)prefix_rows_kernel<E, D, RTP, RTO, true>, attr, (int)PrShape<D>::smem) == cudaSuccess;
}

template <class E, int D>
bool prepare_prefix_kernel()
{
    static_assert(pa_smem<D>().total <= (uint32_t)kMaxSmemPerCta, "shared memory");
    constexpr auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
    return cudaFuncSetAttribute((const void *)prefix_tile_kernel<E, D, false>, attr, (int)pa_smem<D>().total) == cudaSuccess &&
           cudaFuncSetAttribute((const void *)prefix_tile_kernel<E, D, true>, attr, (int)pa_smem<D>().total) == cudaSuccess &&
           prepare_rows_kernel<E, D, 16, 16>() && prepare_rows_kernel<E, D, 64, 16>() && prepare_rows_kernel<E, D, 64, 64>();
}

bool prepare_prefix_kernels()
{
    return prepare_prefix_kernel<Bf16, 64>() && prepare_prefix_kernel<Bf16, 128>() &&
           prepare_prefix_kernel<Fp16, 64>() && prepare_prefix_kernel<Fp16, 128>();
}

// The cache as dim 0 = 64 columns of a slot, dim 1 = slot % 8, dim 2 = the
// slot's 64-column blocks (K, then V), dim 3 = slot / 8, dim 4 = (page, KV
// head): a box is one page of one KV head, its 8-slot groups of every block 1
// KB each and equally far apart from page to page.
int encode_prefix_map(const void *kv_cache, int64_t num_pages, int nkv, int head_dim, bool bf16, CUtensorMap *m)
{
    const cuuint64_t slot = (cuuint64_t)head_dim * 4;   // bytes of a slot
    const cuuint64_t dims[5] = {64, 8, (cuuint64_t)head_dim / 32, 2, (cuuint64_t)num_pages * nkv};
    const cuuint64_t strides[4] = {slot, 128, 8 * slot, kPageSlots * slot};
    const cuuint32_t box[5] = {64, 8, (cuuint32_t)head_dim / 32, 2, 1};
    const cuuint32_t es[5] = {1, 1, 1, 1, 1};
    return g_encode(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 5, (void *)kv_cache,
                    dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? QKVF_OK
               : QKVF_ERR_CUDA;
}

template <class E, int D>
int launch_prefix(const CUtensorMap &map, const PrefixParams &prm, int sms, void *stream)
{
    int rc = QKVF_OK;
    if (!prm.small && prm.prefix_blocks > 0) {
        int64_t grid = (int64_t)prm.nkv * prm.sp;
        grid = prm.pair ? grid * ((prm.tiles + 1) / 2) : (grid + 1) / 2;
        if (grid > sms) grid = sms;
        rc = launch_pdl(prefix_tile_kernel<E, D, false>, dim3((unsigned)grid), dim3(kPaThreads), (size_t)pa_smem<D>().total,
                        stream, map, prm);
        if (rc != QKVF_OK) return rc;
    }
    const int64_t items = (prm.small && prm.prefix_blocks > 0 ? (int64_t)prm.nkv * prm.sp : 0) +
                          (prm.max_blocks > 0 ? (int64_t)prm.R * prm.nkv * prm.own_tiles * prm.ss : 0);
    if (items > 0 && prm.own_tile) {
        rc = launch_pdl(prefix_tile_kernel<E, D, true>, dim3((unsigned)((items + 1) / 2)), dim3(kPaThreads),
                        (size_t)pa_smem<D>().total, stream, map, prm);
        if (rc != QKVF_OK) return rc;
    } else if (items > 0) {
        const bool tokens = prm.q_len > 1 && prm.max_blocks > 0;
        const auto rows = [&](auto several) {
            constexpr bool k = decltype(several)::value;
            return prm.own_rows == 64                ? prefix_rows_kernel<E, D, 64, 64, k>
                   : prm.small && prm.pre_rows == 64 ? prefix_rows_kernel<E, D, 64, 16, k>
                                                     : prefix_rows_kernel<E, D, 16, 16, k>;
        };
        rc = launch_pdl(tokens ? rows(std::true_type()) : rows(std::false_type()),
                        dim3((unsigned)items), dim3(kPrThreads), (size_t)PrShape<D>::smem, stream, map, prm);
        if (rc != QKVF_OK) return rc;
    }
    // Several warps a row where there are more partials than one warp has in
    // flight and few rows: with 4096 rows of 128 and 10 partials one is faster;
    // 8 rows of 64 with 128 partials of a 128K prefix take 14.3 us in all with
    // sixteen, 17.5 with eight; 256 rows with 65 partials 16.8 and 14.8.
    constexpr int ahead = kPaMergeAhead * 32 / (D / 4);   // a warp's
    const int splits = prm.sp + prm.ss;
    const int64_t rows = prm.rows;
    const int warps = splits <= ahead || rows > 16 * sms          ? 1
                      : splits <= 4 * ahead || rows > 4 * sms ? 4
                      : rows > sms                            ? 8
                                                              : 16;
    return launch_pdl(warps == 1   ? prefix_merge_kernel<E, D, 1>
                      : warps == 4 ? prefix_merge_kernel<E, D, 4>
                      : warps == 8 ? prefix_merge_kernel<E, D, 8>
                                   : prefix_merge_kernel<E, D, 16>,
                      dim3((unsigned)(warps == 1 ? (rows + 3) / 4 : rows)), dim3(pa_merge_threads(warps)), 0, stream, prm);
}

const char *check_prefix_shape(int num_reqs, int q_len, int q_heads, int num_kv_heads, int head_dim,
                               int prefix_blocks, int max_blocks, int *code)
{
    *code = QKVF_ERR_TOKENS;
    if (num_reqs < 0 || num_reqs > kPaMaxRequests) return "num_reqs must be 0..65535";
    if (q_len < 1 || q_len > kPaMaxQLen) return "q_len must be 1..1024";
    *code = QKVF_ERR_LAYOUT;
    if (head_dim != 64 && head_dim != 128) return "head_dim must be 64 or 128";
    if (num_kv_heads < 1 || num_kv_heads > 64) return "num_kv_heads must be 1..64";
    if (q_heads < num_kv_heads || q_heads % num_kv_heads || q_heads / num_kv_heads > kPaMaxGroup)
        return "q_heads must be 1..64 times num_kv_heads";
    *code = QKVF_ERR_SIZES;
    if (prefix_blocks < 0 || prefix_blocks > (1 << 24) || max_blocks < 0 || max_blocks > (1 << 24))
        return "prefix_blocks and max_blocks must be 0..2^24";
    if ((int64_t)num_reqs * q_len * q_heads > (int64_t(1) << 24)) return "num_reqs * q_len * q_heads must be <= 2^24";
    *code = QKVF_OK;
    return nullptr;
}

const char *check_prefix_args(const void *q, int64_t q_ts, int64_t q_hs, const void *kv_cache, int64_t num_pages,
                              const int32_t *prefix_pages, int prefix_blocks, const int32_t *prefix_len,
                              const int32_t *block_table, int max_blocks, const int32_t *context_lens,
                              int num_reqs, int q_len, int q_heads, int num_kv_heads, int head_dim, float scale,
                              int dtype, const void *out, const float *lse, const void *workspace,
                              size_t workspace_bytes, int *code)
{
    dtype = dtype_of(dtype);
    if (const char *why = check_prefix_shape(num_reqs, q_len, q_heads, num_kv_heads, head_dim, prefix_blocks,
                                             max_blocks, code))
        return why;
    *code = QKVF_ERR_LAYOUT;
    if (dtype != QKVF_DTYPE_BF16 && dtype != QKVF_DTYPE_FP16) return "dtype must be bf16 or fp16";
    if (!stride_ok(q_ts) || !stride_ok(q_hs) || q_ts % 8 || q_hs % 8)
        return "q's strides must be multiples of 8 elements, 0..2^36";
    *code = QKVF_ERR_SIZES;
    if (num_pages < 1 || num_pages > (int64_t(1) << 31) / num_kv_heads) return "num_pages * num_kv_heads must be 1..2^31";
    *code = QKVF_ERR_ARG;
    if (!(scale > 0.f) || !(scale <= 1e6f)) return "scale must be in (0, 1e6]";
    *code = QKVF_OK;
    if (num_reqs == 0) return nullptr;
    *code = QKVF_ERR_NULL;
    if (!q || !kv_cache || !context_lens || !out || !workspace || (max_blocks > 0 && !block_table) ||
        (prefix_blocks > 0 && (!prefix_pages || !prefix_len)))
        return "a required pointer is NULL";
    *code = QKVF_ERR_ALIGN;
    if (!aligned(q, 16) || !aligned(kv_cache, 16) || !aligned(out, 16)) return "q, kv_cache and out must be 16-byte aligned";
    if (!aligned(context_lens, 4) || !aligned(block_table, 4) || !aligned(prefix_pages, 4) ||
        !aligned(prefix_len, 4) || !aligned(lse, 4))
        return "the tables, lengths and lse must be 4-byte aligned";
    if (!aligned(workspace, 256)) return "the workspace must be 256-byte aligned";
    *code = QKVF_ERR_ARG;
    const size_t rows = (size_t)num_reqs * q_len * q_heads;
    const View vq = view_of(q, num_reqs * q_len, q_ts, q_heads, q_hs, head_dim, 2);
    const void *parts[] = {vq.ptr, kv_cache, context_lens, block_table, prefix_pages, prefix_len, out, lse, workspace};
    const size_t bytes[] = {vq.extent, (size_t)num_pages * num_kv_heads * kPageSlots * 2 * head_dim * 2,
                            (size_t)num_reqs * 4, (size_t)num_reqs * max_blocks * 4, (size_t)prefix_blocks * 4,
                            prefix_blocks > 0 ? (size_t)4 : 0, rows * head_dim * 2, lse ? rows * 4 : 0, workspace_bytes};
    for (int o = 6; o < 9; ++o)   // each output and the workspace against everything before it
        for (int i = 0; i < o; ++i)
            if (overlap(parts[i], bytes[i], parts[o], bytes[o])) return "out, lse or the workspace overlaps another argument";
    *code = QKVF_OK;
    return nullptr;
}

}  // namespace qkvf

extern "C" {

size_t prefix_attn_workspace_bytes(int num_reqs, int q_len, int q_heads, int num_kv_heads, int head_dim,
                                   int prefix_blocks, int max_blocks)
{
    int code;
    if (qkvf::check_prefix_shape(num_reqs, q_len, q_heads, num_kv_heads, head_dim, prefix_blocks, max_blocks, &code))
        return 0;
    qkvf::DeviceState *d;
    if (qkvf::probe_device(&d) != QKVF_OK) return 0;
    return qkvf::pa_workspace(qkvf::pa_plan(num_reqs, q_len, q_heads, num_kv_heads, head_dim, prefix_blocks, max_blocks, d->sms),
                              (int64_t)num_reqs * q_len * q_heads, head_dim);
}

const char *prefix_attn_unsupported(const void *q, int64_t q_token_stride, int64_t q_head_stride,
                                    const void *kv_cache, int64_t num_pages, const int32_t *prefix_pages,
                                    int prefix_blocks, const int32_t *prefix_len, const int32_t *block_table,
                                    int max_blocks, const int32_t *context_lens, int num_reqs, int q_len,
                                    int q_heads, int num_kv_heads, int head_dim, float scale, int dtype,
                                    const void *out, const float *lse, const void *workspace,
                                    size_t workspace_bytes)
{
    int code;
    const char *why = qkvf::check_prefix_args(q, q_token_stride, q_head_stride, kv_cache, num_pages, prefix_pages,
                                              prefix_blocks, prefix_len, block_table, max_blocks, context_lens,
                                              num_reqs, q_len, q_heads, num_kv_heads, head_dim, scale, dtype, out,
                                              lse, workspace, workspace_bytes, &code);
    if (why) return why;
    if (num_reqs == 0) return nullptr;
    qkvf::DeviceState *d;
    const int rc = qkvf::probe_device(&d);
    if (rc != QKVF_OK) return qkv_front_strerror(rc);
    return workspace_bytes < prefix_attn_workspace_bytes(num_reqs, q_len, q_heads, num_kv_heads, head_dim,
                                                         prefix_blocks, max_blocks)
               ? "the workspace is too small"
               : nullptr;
}

int prefix_attn(const void *q, int64_t q_token_stride, int64_t q_head_stride, const void *kv_cache,
                int64_t num_pages, const int32_t *prefix_pages, int prefix_blocks, const int32_t *prefix_len,
                const int32_t *block_table, int max_blocks, const int32_t *context_lens, int num_reqs, int q_len,
                int q_heads, int num_kv_heads, int head_dim, float scale, int dtype, void *out, float *lse,
                void *workspace, size_t workspace_bytes, void *stream)
{
    int code;
    if (qkvf::check_prefix_args(q, q_token_stride, q_head_stride, kv_cache, num_pages, prefix_pages, prefix_blocks,
                                prefix_len, block_table, max_blocks, context_lens, num_reqs, q_len, q_heads,
                                num_kv_heads, head_dim, scale, dtype, out, lse, workspace, workspace_bytes, &code))
        return code;
    if (num_reqs == 0) return QKVF_OK;
    qkvf::DeviceState *d;
    int rc = qkvf::probe_device(&d);
    if (rc != QKVF_OK) return rc;
    const qkvf::PaPlan pl = qkvf::pa_plan(num_reqs, q_len, q_heads, num_kv_heads, head_dim, prefix_blocks, max_blocks, d->sms);
    if (workspace_bytes < qkvf::pa_workspace(pl, (int64_t)num_reqs * q_len * q_heads, head_dim)) return QKVF_ERR_SIZES;
    const bool bf16 = qkvf::dtype_of(dtype) == QKVF_DTYPE_BF16;
    CUtensorMap map;
    rc = qkvf::encode_prefix_map(kv_cache, num_pages, num_kv_heads, head_dim, bf16, &map);
    if (rc != QKVF_OK) return rc;
    qkvf::PrefixParams prm = {};
    prm.q = q;
    prm.kv_cache = kv_cache;
    prm.zero = qkvf::zero_skipped(dtype);
    prm.prefix_pages = prefix_pages;
    prm.prefix_len = prefix_len;
    prm.block_table = block_table;
    prm.context_lens = context_lens;
    prm.out = out;
    prm.lse = lse;
    prm.num_pages = num_pages;
    prm.q_ts = q_token_stride;
    prm.q_hs = q_head_stride;
    prm.wait_limit_ns = qkvf::g_wait_limit_ns;
    prm.prefix_blocks = prefix_blocks;
    prm.max_blocks = max_blocks;
    prm.R = num_reqs;
    prm.q_len = q_len;
    prm.q_heads = q_heads;
    prm.nkv = num_kv_heads;
    prm.group = q_heads / num_kv_heads;
    prm.rows = num_reqs * q_len * q_heads;
    prm.tiles = pl.tiles;
    prm.small = pl.small;
    prm.pre_rows = pl.pre_rows;
    prm.own_tile = pl.own_tile;
    prm.own_rows = pl.own_rows;
    prm.own_tiles = pl.own_tiles;
    prm.sp = pl.sp;
    prm.ss = pl.ss;
    prm.pair = pl.pair;
    prm.scale_log2 = scale * 1.4426950408889634f;
    prm.ws_o = static_cast<float *>(workspace);
    prm.ws_ml = reinterpret_cast<float2 *>(prm.ws_o + (size_t)prm.rows * (pl.sp + pl.ss) * head_dim);
    if (bf16)
        return head_dim == 64 ? qkvf::launch_prefix<qkvf::Bf16, 64>(map, prm, d->sms, stream)
                              : qkvf::launch_prefix<qkvf::Bf16, 128>(map, prm, d->sms, stream);
    return head_dim == 64 ? qkvf::launch_prefix<qkvf::Fp16, 64>(map, prm, d->sms, stream)
                          : qkvf::launch_prefix<qkvf::Fp16, 128>(map, prm, d->sms, stream);
}

int prefix_attn_packed(const int64_t *args, void *stream)
{
    if (!args) return QKVF_ERR_NULL;
    qkvf::Words w(args);
    const int prefix_blocks = w.i(6), max_blocks = w.i(9), R = w.i(11), q_len = w.i(12), q_heads = w.i(13), nkv = w.i(14),
              dim = w.i(15), dtype = w.i(17);
    if (!w.ok) return QKVF_ERR_SIZES;
    return prefix_attn(w.p<void>(0), args[1], args[2], w.p<void>(3), args[4], w.p<int32_t>(5), prefix_blocks, w.p<int32_t>(7),
                       w.p<int32_t>(8), max_blocks, w.p<int32_t>(10), R, q_len, q_heads, nkv, dim, (float)w.d(16), dtype,
                       w.p<void>(18), w.p<float>(19), w.p<void>(20), (size_t)args[21], stream);
}

}  // extern "C"
