// kv_evict: keep the keys of largest weight of every request and KV head,
// and move them together (included by qkv_front.cu after chunk_attn.cuh: one
// translation unit).
//
// Of a request's L keys the last `recent` stay, and of the others the keep -
// recent of largest weight, the lower index first among equals; kept keys keep
// their order.  Two kernels:
//  * evict_select_kernel, a CTA per (request, KV head): the smallest kept
//    weight by up to four passes over its bits (8, 11, 11 and 2 at a time, a
//    histogram each; no more once the digits found are taken whole), then one
//    ordered pass that numbers the kept keys and moves their weights.  A row's
//    weights are read once, into shared memory (the first 18,432 of them).
//    What bounds it is one CTA's instructions and barriers (64 rows of 9,000 to
//    16,384 keys, 2,048 kept: 15 us, of them 3 to load, 2.7 a pass and 4 for the
//    numbering; the weights read from memory in every pass: 19).
//  * evict_move_kernel copies K | V slots.  Into other pages every slot is on
//    its own; in place a kept key only ever moves down, so a CTA takes some
//    columns of all slots and reads each round of slots before it writes them.
//    The first is bound by its bytes (64 rows of 2,048 kept keys of 128, 134 MB:
//    20 us), the second by its rounds, one after another with a barrier each (36).

namespace qkvf {

constexpr int kEvThreads = 1024, kEvBins = 2048;
constexpr int kEvFirst = 256;      // bins of the first pass, 32 copies of each
constexpr int kEvCached = 18432;   // weights of a row kept in shared memory (72 KB beside 32 KB of bins: two CTAs an SM)
constexpr int kEvMaxKeep = 1 << 24;

struct EvictParams {
    void *kv_cache;
    const float *weights;
    float *out_weights;
    const int32_t *block_table, *out_table;
    const int32_t *context_lens;
    int32_t *out_lens;
    int32_t *kept;
    int64_t num_pages;
    int max_blocks, out_blocks;
    int R, nkv, dim, keep, recent;
    int in_place;
};

// Weights in the order of unsigned numbers: -0 is 0 (the sum), and NaN, which a
// sum makes 0x7fffffff, above everything
__device__ __forceinline__ uint32_t ev_key(float w)
{
    const uint32_t u = __float_as_uint(__fadd_rn(w, 0.f));
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

// Where chunk c of four weights lies in shared memory: neither neighbours nor
// chunks at a distance of 2 or 4 meet in a bank
__device__ __forceinline__ int ev_chunk(int c) { return c ^ ((c >> 3) & 3); }

// Sum over the warp's lanes up to this one
__device__ __forceinline__ uint32_t ev_scan(uint32_t v)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    return v;
}

// One more at `bin` (an address in shared memory) where `on`
__device__ __forceinline__ void ev_count(uint32_t bin, bool on)
{
    asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %1, 0;\n @p red.shared.add.u32 [%0], 1;\n}" ::"r"(bin), "r"((uint32_t)on)
                 : "memory");
}

extern __shared__ __align__(16) float ev_weights[];

__global__ void __launch_bounds__(kEvThreads) evict_select_kernel(const __grid_constant__ EvictParams p)
{
    __shared__ uint32_t bins[kEvFirst * 32];
    __shared__ uint32_t warp_sums[2][32];   // a barrier apart: the next sums take the other row
    __shared__ uint32_t found[2][3];        // the digit, the keys above it, whether it is taken whole
    if (threadIdx.x == 0) griddep_launch_dependents();
    for (int i = threadIdx.x; i < kEvFirst * 32; i += kEvThreads) bins[i] = 0u;
    griddep_wait();
    const int r = blockIdx.x / p.nkv, g = blockIdx.x % p.nkv, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row = blockIdx.x;
    const float *w = p.weights + row * p.max_blocks * kPageSlots;
    float *ow = p.out_weights + row * p.out_blocks * kPageSlots;
    int32_t *kept = p.kept + row * p.keep;
    const int L = p.context_lens[r], n = min(L, p.keep);
    bool bad = L > p.max_blocks * kPageSlots;
    const int cached = bad ? 0 : min(max(L, 0), kEvCached);
    const uint32_t cache = smem_u32(ev_weights), bins0 = smem_u32(bins);
    if ((reinterpret_cast<uintptr_t>(w) & 15) == 0) {   // (a row's end is a multiple of 16 bytes as well)
        for (int c = tid; c * 4 < cached; c += kEvThreads)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(cache + ev_chunk(c) * 16), "l"(w + c * 4) : "memory");
    } else {
        for (int j = tid; j < cached; j += kEvThreads)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(cache + ev_chunk(j >> 2) * 16 + (j & 3) * 4), "l"(w + j)
                         : "memory");
    }
    // a page outside the cache leaves the request alone, in every KV head
    if (L > 0 && !bad) {
        const int32_t *from = p.block_table + (int64_t)r * p.max_blocks, *to = p.out_table + (int64_t)r * p.out_blocks;
        for (int i = tid; i < (L + kPageSlots - 1) / kPageSlots; i += kEvThreads) bad |= from[i] < 0 || from[i] >= p.num_pages;
        for (int i = tid; i < (n + kPageSlots - 1) / kPageSlots; i += kEvThreads) bad |= to[i] < 0 || to[i] >= p.num_pages;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (__syncthreads_or(bad) || L < 0) {
        if (L >= 0 && tid == 0 && g == 0) atomicOr(&g_status, QKVF_STATUS_BAD_REQUEST);
        for (int i = tid; i < p.keep; i += kEvThreads) kept[i] = -1;
        return;
    }
    // weights 4 c .. 4 c + 3 (those from L on are anything)
    const auto four = [&](int c, float (&v)[4]) {
        if (c * 4 < cached) {
            const float4 x = *reinterpret_cast<const float4 *>(ev_weights + ev_chunk(c) * 4);
            v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = c * 4 + e < L ? w[c * 4 + e] : 0.f;
        }
    };
    for (int i = n + tid; i < p.keep; i += kEvThreads) kept[i] = -1;
    // the keys to choose from, and how many of them
    const int old = L - min(p.recent, L), take = n - (L - old);
    uint32_t prefix = 0u, mask = 0u;
    int above = 0, turn = 0;   // keys of larger weight than `prefix` so far
    if (take == 0) {           // none: more than any weight, and no equal of it taken
        prefix = mask = 0xffffffffu;
    } else if (take < old) {
#pragma unroll 1
        for (int pass = 0, shift = 24; pass < 4; ++pass, turn ^= 1) {
            // the first digit is mostly the same: a lane has its own copy of the bins (sums of one address take turns)
            const int bits = pass == 0 ? 8 : pass < 3 ? 11 : 2, copies = pass == 0 ? 5 : 0;
            if (pass > 0) shift -= bits;
            const int turned = shift - copies - 2;   // to where a bin's address has the digit
            const uint32_t bin0 = bins0 + (pass == 0 ? lane * 4 : 0), digits = ((1u << bits) - 1u) << (copies + 2);
            for (int c = tid; c * 4 < old; c += kEvThreads) {
                float v[4];
                four(c, v);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t k = ev_key(v[e]);
                    ev_count(bin0 + (__funnelshift_r(k, k, turned) & digits), c * 4 + e < old && (k & mask) == prefix);
                }
            }
            __syncthreads();
            // from the largest digit down, two a thread: where the number to take is reached
            int top;
            uint32_t c0 = 0u, c1 = 0u;
            if (pass == 0) {   // four threads a digit, the first of them holds its count
                top = kEvFirst - 1 - tid / 4;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    uint32_t &bin = bins[top * 32 + (tid & 3) * 8 + ((i + tid / 4) & 7)];
                    c0 += bin;
                    bin = 0u;
                }
                c0 += __shfl_xor_sync(0xffffffffu, c0, 1);
                c0 += __shfl_xor_sync(0xffffffffu, c0, 2);
                if (tid & 3) c0 = 0u;
            } else {
                top = kEvBins - 1 - 2 * tid;
                c0 = bins[top], c1 = bins[top - 1];
                bins[top] = bins[top - 1] = 0u;
            }
            const uint32_t all = __reduce_add_sync(0xffffffffu, c0 + c1);
            if (lane == 0) warp_sums[turn][warp] = all;
            __syncthreads();
            const uint32_t lower = above + __reduce_add_sync(0xffffffffu, lane < warp ? warp_sums[turn][lane] : 0u);
            if ((int)lower < take && take <= (int)(lower + all)) {   // one warp has it
                const uint32_t upto = lower + ev_scan(c0 + c1), before = upto - c0 - c1;
                if ((int)before < take && take <= (int)upto) {
                    const bool second = (int)(before + c0) < take;
                    found[turn][0] = second ? top - 1 : top;
                    found[turn][1] = second ? before + c0 : before;
                    found[turn][2] = take == (int)(second ? upto : before + c0);
                }
            }
            __syncthreads();
            prefix |= found[turn][0] << shift;
            mask |= ((1u << bits) - 1u) << shift;
            above = (int)found[turn][1];
            if (found[turn][2]) break;   // every key of these digits stays: the others do not matter
        }
        turn ^= 1;
    }
    const int ties = take - above;   // of the digits of `prefix`, in order
    const bool all = take >= old;
    if (!(all && p.in_place)) {
        // a thread takes neighbouring keys, up to 16 of them a round, and lists
        // the kept ones in shared memory: written from the threads themselves,
        // 16 stores of a few lanes each, the round took a fifth longer
        uint16_t *list = reinterpret_cast<uint16_t *>(bins);
        const int each = min(4, (L + kEvThreads * 4 - 1) / (kEvThreads * 4));
        int sure = 0, equal = 0;   // kept for their weight or age, and ties, before this round
        for (int j0 = 0; j0 < L; j0 += kEvThreads * 4 * each, turn ^= 1) {
            const int own = tid * 4 * each, j = j0 + own;
            uint32_t yes = 0u, maybe = 0u;
#pragma unroll 1
            for (int i = 0; i < each && j + i * 4 < L; ++i) {
                float v[4];
                four(j / 4 + i, v);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t k = ev_key(v[e]) & mask, bit = 1u << e << (i * 4);
                    if (all || j + i * 4 + e >= old || k > prefix) yes |= bit;
                    if (k == prefix) maybe |= bit;
                }
            }
            const uint32_t in = L - j >= 16 ? 0xffffu : (1u << max(L - j, 0)) - 1u;
            yes &= in;
            maybe &= in & ~yes;
            const uint32_t mine = ((uint32_t)__popc(yes) << 16) + __popc(maybe);   // (at most 16384 of a kind in a round)
            const uint32_t upto = ev_scan(mine);
            if (lane == 31) warp_sums[turn][warp] = upto;
            __syncthreads();
            const uint32_t others = warp_sums[turn][lane];
            const uint32_t at = __reduce_add_sync(0xffffffffu, lane < warp ? others : 0u) + upto - mine;
            const uint32_t total = __reduce_add_sync(0xffffffffu, others);
            const int before = min(equal, ties);   // ties kept before this round
            int t = equal + (int)(at & 0xffffu), dst = (int)(at >> 16) + min(t, ties) - before;
            for (uint32_t m = yes | maybe; m; m &= m - 1u) {
                const int e = __ffs(m) - 1;
                const bool tie = maybe >> e & 1u;
                if (!tie || t < ties) list[dst++] = (uint16_t)(own + e);
                t += tie;
            }
            __syncthreads();
            const int base = sure + before;
            equal += (int)(total & 0xffffu);
            sure += (int)(total >> 16);
            const int count = sure + min(equal, ties) - base;
            for (int i0 = 0; i0 < count; i0 += kEvThreads) {
                const int i = i0 + tid, src = i < count ? j0 + list[i] : 0;
                float v = 0.f;
                if (i < count) v = src < cached ? ev_weights[ev_chunk(src >> 2) * 4 + (src & 3)] : w[src];
                __syncthreads();   // in place a kept key only ever moves down: what is written now is read
                if (i < count) {
                    kept[base + i] = src;
                    ow[base + i] = v;
                }
            }
        }
    } else {
        for (int i = tid; i < n; i += kEvThreads) kept[i] = i;
    }
    __syncthreads();
    const int end = p.in_place ? L : p.out_blocks * kPageSlots;
    for (int i = n + tid; i < end; i += kEvThreads) ow[i] = 0.f;
}

__device__ __forceinline__ uint4 *ev_slot(const EvictParams &p, const int32_t *table, int g, int key)
{
    const int64_t slot = ((int64_t)table[key / kPageSlots] * p.nkv + g) * kPageSlots + key % kPageSlots;
    return reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.kv_cache) + slot * (2 * p.dim));
}

constexpr int kEvMoveThreads = 256, kEvMoveEach = 4, kEvSlice = 4;   // in place: 64 bytes of every slot a CTA

// blockIdx.x: a run of slots (other pages) or some columns of all of them (in place)
__global__ void __launch_bounds__(kEvMoveThreads) evict_move_kernel(const __grid_constant__ EvictParams p)
{
    if (threadIdx.x == 0) griddep_launch_dependents();
    griddep_wait();
    const int64_t row = blockIdx.y + (int64_t)blockIdx.z * gridDim.y;
    if (row >= (int64_t)p.R * p.nkv) return;
    const int r = (int)(row / p.nkv), g = (int)(row % p.nkv), tid = threadIdx.x;
    const int32_t *kept = p.kept + row * p.keep;
    const int32_t *from = p.block_table + (int64_t)r * p.max_blocks, *to = p.out_table + (int64_t)r * p.out_blocks;
    const int chunks = p.dim / 4;   // 16-byte chunks of a slot
    if (blockIdx.x == 0 && g == 0 && tid == 0) {
        const int L = p.context_lens[r];
        if (L == 0 || (L > 0 && kept[0] >= 0)) p.out_lens[r] = min(L, p.keep);
    }
    const int width = p.in_place ? min(kEvSlice, chunks - (int)blockIdx.x * kEvSlice) : chunks;
    const int c0 = p.in_place ? blockIdx.x * kEvSlice : 0;
    const int per = kEvMoveThreads / width, i0 = tid / width, c = c0 + tid % width;   // slots at a time
    const int64_t step = (int64_t)per * kEvMoveEach;
    const int64_t first = p.in_place ? 0 : blockIdx.x * step, last = p.in_place ? p.keep : min((int64_t)p.keep, first + step);
    for (int64_t b = first; b < last; b += step) {
        uint4 v[kEvMoveEach];
        int src[kEvMoveEach];
#pragma unroll
        for (int e = 0; e < kEvMoveEach; ++e) {
            const int64_t i = b + e * per + i0;
            src[e] = i0 < per && i < last ? kept[i] : -1;
            if (p.in_place && src[e] == (int)i) src[e] = -1;
        }
#pragma unroll
        for (int e = 0; e < kEvMoveEach; ++e)
            if (src[e] >= 0) v[e] = ev_slot(p, from, g, src[e])[c];
        if (p.in_place) __syncthreads();   // the round is read before it is written
#pragma unroll
        for (int e = 0; e < kEvMoveEach; ++e)
            if (src[e] >= 0) ev_slot(p, to, g, (int)(b + e * per + i0))[c] = v[e];
    }
}

bool prepare_evict_kernel()
{
    return cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kEvCached * (int)sizeof(float)) ==
           cudaSuccess;
}

const char *check_evict_args(const void *kv_cache, int64_t num_pages, const float *weights, const int32_t *block_table,
                             int max_blocks, const int32_t *context_lens, int num_reqs, int num_kv_heads, int head_dim,
                             int keep, int recent, const int32_t *out_table, int out_blocks, const float *out_weights,
                             const int32_t *out_lens, const int32_t *kept, int *code)
{
    *code = QKVF_ERR_TOKENS;
    if (num_reqs < 0 || num_reqs > kPaMaxRequests) return "num_reqs must be 0..65535";
    *code = QKVF_ERR_LAYOUT;
    if (head_dim < 8 || head_dim > kRopeMaxDim || head_dim % 8) return "head_dim must be a multiple of 8, 8..512";
    if (num_kv_heads < 1 || num_kv_heads > 1024) return "num_kv_heads must be 1..1024";
    *code = QKVF_ERR_SIZES;
    if (num_pages < 1 || num_pages > (int64_t(1) << 31)) return "num_pages must be 1..2^31";
    if (max_blocks < 1 || max_blocks > (1 << 20) || out_blocks < 1 || out_blocks > (1 << 20))
        return "max_blocks and out_blocks must be 1..2^20";
    if (keep < 1 || keep > kEvMaxKeep || recent < 0 || recent > keep) return "keep must be 1..2^24 and recent 0..keep";
    *code = QKVF_OK;
    if (num_reqs == 0) return nullptr;
    *code = QKVF_ERR_NULL;
    if (!kv_cache || !weights || !block_table || !context_lens || !out_table || !out_weights || !out_lens || !kept)
        return "a required pointer is NULL";
    *code = QKVF_ERR_ALIGN;
    if (!aligned(kv_cache, 16)) return "kv_cache must be 16-byte aligned";
    if (!aligned(weights, 4) || !aligned(block_table, 4) || !aligned(context_lens, 4) || !aligned(out_table, 4) ||
        !aligned(out_weights, 4) || !aligned(out_lens, 4) || !aligned(kept, 4))
        return "the weights, tables, lengths and kept must be 4-byte aligned";
    *code = QKVF_ERR_ARG;
    const bool same = out_table == block_table;
    if ((out_weights == weights) != same || (out_lens == context_lens) != same || (same && out_blocks != max_blocks))
        return "the table, weights and lengths must all be in place, or none of them";
    *code = QKVF_ERR_SIZES;
    if (!same && (int64_t)out_blocks * kPageSlots < keep) return "out_table has less room than keep";
    *code = QKVF_ERR_ARG;
    const size_t rows = (size_t)num_reqs * num_kv_heads;
    const void *parts[] = {block_table, weights, context_lens, out_table, out_weights, out_lens, kv_cache, kept};
    const size_t bytes[] = {(size_t)num_reqs * max_blocks * 4, rows * max_blocks * kPageSlots * 4, (size_t)num_reqs * 4,
                            (size_t)num_reqs * out_blocks * 4, rows * out_blocks * kPageSlots * 4, (size_t)num_reqs * 4,
                            (size_t)num_pages * num_kv_heads * kPageSlots * 2 * head_dim * 2, rows * keep * 4};
    for (int o = 4; o < 8; ++o)   // what is written against everything before it
        for (int i = 0; i < o; ++i) {
            if (same && i + 3 == o && o < 6) continue;   // itself
            if (overlap(parts[i], bytes[i], parts[o], bytes[o])) return "an output overlaps another argument";
        }
    if (!same && overlap(parts[3], bytes[3], parts[0], bytes[0])) return "out_table overlaps block_table";
    *code = QKVF_OK;
    return nullptr;
}

}  // namespace qkvf

extern "C" {

const char *kv_evict_unsupported(void *kv_cache, int64_t num_pages, const float *weights, const int32_t *block_table,
                                 int max_blocks, const int32_t *context_lens, int num_reqs, int num_kv_heads,
                                 int head_dim, int keep, int recent, const int32_t *out_table, int out_blocks,
                                 float *out_weights, int32_t *out_lens, int32_t *kept)
{
    int code;
    const char *why = qkvf::check_evict_args(kv_cache, num_pages, weights, block_table, max_blocks, context_lens, num_reqs,
                                             num_kv_heads, head_dim, keep, recent, out_table, out_blocks, out_weights,
                                             out_lens, kept, &code);
    if (why) return why;
    qkvf::DeviceState *d;
    const int rc = qkvf::probe_device(&d);
    return rc == QKVF_OK ? nullptr : qkv_front_strerror(rc);
}

int kv_evict(void *kv_cache, int64_t num_pages, const float *weights, const int32_t *block_table, int max_blocks,
             const int32_t *context_lens, int num_reqs, int num_kv_heads, int head_dim, int keep, int recent,
             const int32_t *out_table, int out_blocks, float *out_weights, int32_t *out_lens, int32_t *kept,
             void *stream)
{
    int code;
    if (qkvf::check_evict_args(kv_cache, num_pages, weights, block_table, max_blocks, context_lens, num_reqs, num_kv_heads,
                               head_dim, keep, recent, out_table, out_blocks, out_weights, out_lens, kept, &code))
        return code;
    if (num_reqs == 0) return QKVF_OK;
    qkvf::DeviceState *d;
    int rc = qkvf::probe_device(&d);
    if (rc != QKVF_OK) return rc;
    qkvf::EvictParams prm = {};
    prm.kv_cache = kv_cache;
    prm.weights = weights;
    prm.out_weights = out_weights;
    prm.block_table = block_table;
    prm.out_table = out_table;
    prm.context_lens = context_lens;
    prm.out_lens = out_lens;
    prm.kept = kept;
    prm.num_pages = num_pages;
    prm.max_blocks = max_blocks;
    prm.out_blocks = out_blocks;
    prm.R = num_reqs;
    prm.nkv = num_kv_heads;
    prm.dim = head_dim;
    prm.keep = keep;
    prm.recent = recent;
    prm.in_place = out_table == block_table;
    const int64_t rows = (int64_t)num_reqs * num_kv_heads;
    const int64_t cached = (int64_t)max_blocks * qkvf::kPageSlots;
    rc = qkvf::launch_pdl(qkvf::evict_select_kernel, dim3((unsigned)rows), dim3(qkvf::kEvThreads),
                          (cached < qkvf::kEvCached ? cached : qkvf::kEvCached) * sizeof(float), stream, prm);
    if (rc != QKVF_OK) return rc;
    const int chunks = head_dim / 4, step = qkvf::kEvMoveThreads / chunks * qkvf::kEvMoveEach;
    const int x = prm.in_place ? (chunks + qkvf::kEvSlice - 1) / qkvf::kEvSlice : (keep + step - 1) / step;
    const int64_t y = rows < 32768 ? rows : 32768;
    return qkvf::launch_pdl(qkvf::evict_move_kernel, dim3((unsigned)x, (unsigned)y, (unsigned)((rows + y - 1) / y)),
                            dim3(qkvf::kEvMoveThreads), 0, stream, prm);
}

int kv_evict_packed(const int64_t *args, void *stream)
{
    if (!args) return QKVF_ERR_NULL;
    qkvf::Words w(args);
    const int mb = w.i(4), R = w.i(6), nkv = w.i(7), dim = w.i(8), keep = w.i(9), recent = w.i(10), ob = w.i(12);
    if (!w.ok) return QKVF_ERR_SIZES;
    return kv_evict(w.p<void>(0), args[1], w.p<float>(2), w.p<int32_t>(3), mb, w.p<int32_t>(5), R, nkv, dim, keep, recent,
                    w.p<int32_t>(11), ob, w.p<float>(13), w.p<int32_t>(14), w.p<int32_t>(15), stream);
}

}  // extern "C"
