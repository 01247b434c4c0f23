// kv_evict: keep the keys of largest weight of every request and KV head,
// and move them together (included by qkv_front.cu after chunk_attn.cuh: one
// translation unit).
//
// Of a request's L keys the last `recent` stay, and of the others the keep -
// recent of largest weight, the lower index first among equals; kept keys keep
// their order.  Two kernels:
//  * evict_select_kernel, a CTA per (request, KV head): the smallest kept
//    weight by three passes over its bits (11, 11 and 10 at a time, a histogram
//    each), then one ordered pass that numbers the kept keys and moves their
//    weights.
//  * evict_move_kernel copies K | V slots.  Into other pages every slot is on
//    its own; in place a kept key only ever moves down, so a CTA takes some
//    columns of all slots and reads each round of slots before it writes them.

namespace qkvf {

constexpr int kEvThreads = 1024, kEvEach = 4, kEvBins = 2048;
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

// Weights in the order of unsigned numbers: -0 is 0, NaN above everything
__device__ __forceinline__ uint32_t ev_key(float w)
{
    const uint32_t u = __float_as_uint(w + 0.f);
    if (w != w) return 0xffffffffu;
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

// Inclusive sum over the block's threads before and with this one; total: of all
__device__ __forceinline__ uint64_t ev_scan(uint64_t v, uint64_t *warp_sums, uint64_t &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    __syncthreads();   // the sums of the scan before are read
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    if (warp == 0) {
        uint64_t s = warp_sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint64_t y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        warp_sums[lane] = s;
    }
    __syncthreads();
    total = warp_sums[31];
    return v + (warp ? warp_sums[warp - 1] : 0);
}

__global__ void __launch_bounds__(kEvThreads) evict_select_kernel(const __grid_constant__ EvictParams p)
{
    __shared__ uint32_t bins[kEvBins];
    __shared__ uint64_t warp_sums[32];
    __shared__ uint32_t found[2];   // the digit, and the keys of higher digits
    __shared__ int bad;
    if (threadIdx.x == 0) griddep_launch_dependents();
    griddep_wait();
    const int r = blockIdx.x / p.nkv, g = blockIdx.x % p.nkv, tid = threadIdx.x;
    const int64_t row = blockIdx.x;
    const float *w = p.weights + row * p.max_blocks * kPageSlots;
    float *ow = p.out_weights + row * p.out_blocks * kPageSlots;
    int32_t *kept = p.kept + row * p.keep;
    const int L = p.context_lens[r], n = min(L, p.keep);
    // a page outside the cache leaves the request alone, in every KV head
    if (tid == 0) bad = L > p.max_blocks * kPageSlots;
    __syncthreads();
    if (L > 0 && !bad) {
        const int32_t *from = p.block_table + (int64_t)r * p.max_blocks, *to = p.out_table + (int64_t)r * p.out_blocks;
        bool out = false;
        for (int i = tid; i < (L + kPageSlots - 1) / kPageSlots; i += kEvThreads) out |= from[i] < 0 || from[i] >= p.num_pages;
        for (int i = tid; i < (n + kPageSlots - 1) / kPageSlots; i += kEvThreads) out |= to[i] < 0 || to[i] >= p.num_pages;
        if (out) bad = 1;
    }
    __syncthreads();
    if (bad || L < 0) {
        if (bad && tid == 0 && g == 0) atomicOr(&g_status, QKVF_STATUS_BAD_REQUEST);
        for (int i = tid; i < p.keep; i += kEvThreads) kept[i] = -1;
        return;
    }
    for (int i = n + tid; i < p.keep; i += kEvThreads) kept[i] = -1;
    // the keys to choose from, and how many of them
    const int old = L - min(p.recent, L), take = n - (L - old);
    uint32_t prefix = 0u, mask = 0u;
    int above = 0;   // keys of larger weight than `prefix` so far
    if (take < old) {
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, width = pass == 2 ? 1024 : 2048;
            for (int i = tid; i < width; i += kEvThreads) bins[i] = 0u;
            __syncthreads();
            for (int j = tid; j < old; j += kEvThreads) {
                const uint32_t k = ev_key(w[j]);
                if ((k & mask) == prefix) atomicAdd(&bins[(k >> shift) & (width - 1)], 1u);
            }
            __syncthreads();
            // from the largest digit down: where the number to take is reached
            const int per = width / kEvThreads, top = width - 1 - tid * per;
            uint32_t c0 = bins[top], c1 = per == 2 ? bins[top - 1] : 0u;
            uint64_t total;
            const uint32_t upto = above + (uint32_t)ev_scan(c0 + c1, warp_sums, total), before = upto - c0 - c1;
            if ((int)before < take && take <= (int)upto) {
                const bool second = (int)(before + c0) < take;
                found[0] = second ? top - 1 : top;
                found[1] = second ? before + c0 : before;
            }
            if (take == 0 && tid == 0) {   // none of them: above every digit
                found[0] = width - 1;
                found[1] = 0;
            }
            __syncthreads();
            prefix |= found[0] << shift;
            mask |= (uint32_t)(width - 1) << shift;
            above = (int)found[1];
            __syncthreads();
        }
    }
    const int ties = take - above;   // of weight `prefix` itself, in order
    const bool all = take >= old;
    if (!(all && p.in_place)) {
        uint64_t base = 0;   // kept for their weight or age in the high half, ties in the low one
        for (int j0 = 0; j0 < L; j0 += kEvThreads * kEvEach) {
            const int j = j0 + tid * kEvEach;
            float v[kEvEach];
            uint64_t mine = 0;
            uint32_t kind[kEvEach];
#pragma unroll
            for (int e = 0; e < kEvEach; ++e) {
                v[e] = j + e < L ? w[j + e] : 0.f;
                kind[e] = 0;
                if (j + e < L) {
                    const uint32_t k = ev_key(v[e]);
                    kind[e] = all || j + e >= old || k > prefix ? 2 : k == prefix ? 1 : 0;
                }
                mine += kind[e] == 2 ? uint64_t(1) << 32 : kind[e];
            }
            uint64_t total;
            uint64_t at = base + ev_scan(mine, warp_sums, total) - mine;   // (and every weight of the round is read)
#pragma unroll
            for (int e = 0; e < kEvEach; ++e) {
                const int tied = (int)(uint32_t)at;
                const bool keep = kind[e] == 2 || (kind[e] == 1 && tied < ties);
                if (keep) {
                    const int dst = (int)(at >> 32) + min(tied, ties);
                    kept[dst] = j + e;
                    ow[dst] = v[e];
                }
                at += kind[e] == 2 ? uint64_t(1) << 32 : kind[e];
            }
            base += total;
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
    rc = qkvf::launch_pdl(qkvf::evict_select_kernel, dim3((unsigned)rows), dim3(qkvf::kEvThreads), 0, stream, prm);
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
