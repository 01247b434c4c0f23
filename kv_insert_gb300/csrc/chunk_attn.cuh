// chunk_attn: attention of each request's new tokens over its paged keys, and
// key_weights: what each key received of it (included by qkv_front.cu after
// norm_rope.cuh: one translation unit).
//
// Request r brings the rows starts[r] .. starts[r + 1] - 1 of q, n of them, and
// has L keys, its new tokens' among them.  Its token i sees keys j <= L - n + i:
//   s = scale q . k;  out = sum exp(s - m) v / sum exp(s - m);  lse = ln sum exp(s).
// key_weights: w[j] = decay w[j] + sum over tokens and the KV head's q heads of
// exp(s - lse).

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
    int T, R, max_blocks, q_heads, nkv, group;
    int window;
    float decay;
    float scale_log2;
    int zero;
};

// A request's rows and keys; n < 0: left alone
struct RaggedRequest {
    int row0, n, L;
};

__device__ __forceinline__ RaggedRequest ragged_request(const RaggedParams &p, int r)
{
    RaggedRequest q;
    const int b = p.starts[r], e = p.starts[r + 1];
    q.L = p.context_lens[r];
    q.row0 = b;
    q.n = e - b;
    const bool bad = b < 0 || e < b || e > p.T || q.L > p.max_blocks * kPageSlots;
    if (bad || q.L < 0) {
        if (bad) atomicOr(&g_status, QKVF_STATUS_BAD_REQUEST);
        q.n = -1;
    }
    return q;
}

template <class E, int D>
__device__ __forceinline__ float ragged_dot(const uint16_t *k, const float *q, int lane)
{
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) s = fmaf(q[i], E::get(k[lane + 32 * i]), s);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

template <class E, int D>
__global__ void __launch_bounds__(128) chunk_rows_kernel(const __grid_constant__ RaggedParams p)
{
    if (threadIdx.x == 0) griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (row >= (int64_t)p.T * p.q_heads) return;
    const int t = (int)(row / p.q_heads), h = (int)(row % p.q_heads), g = h / p.group;
    uint16_t *out = static_cast<uint16_t *>(p.out) + row * D;
    int lo = 0, hi = p.R;   // the last request that starts at or before t
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (p.starts[mid] <= t) lo = mid;
        else hi = mid - 1;
    }
    bool ok = lo < p.R && p.starts[lo] <= t && t < p.starts[lo + 1];
    RaggedRequest q = {0, -1, 0};
    if (ok) q = ragged_request(p, lo);
    ok = q.n >= 0;
    if (blockIdx.x == 0)   // each request's starts and length, flagged once
        for (int r = threadIdx.x; r < p.R; r += 128) ragged_request(p, r);
    float acc[D / 32] = {}, m = -INFINITY, l = 0.f, part = 0.f, qv[D / 32];   // part: of up to 64 keys
    if (ok) {
        const uint16_t *qp = static_cast<const uint16_t *>(p.q) + t * p.q_ts + h * p.q_hs;
        for (int i = 0; i < D / 32; ++i) qv[i] = E::get(qp[lane + 32 * i]);
        const int end = q.L - q.n + (t - q.row0) + 1;
        for (int j = 0; j < end; ++j) {
            const int page = p.block_table[(int64_t)lo * p.max_blocks + j / kPageSlots];
            if (page < 0 || page >= p.num_pages) {
                ok = false;
                atomicOr(&g_status, QKVF_STATUS_BAD_REQUEST);
                break;
            }
            const uint16_t *k = static_cast<const uint16_t *>(p.kv_cache) +
                                (((int64_t)page * p.nkv + g) * kPageSlots + j % kPageSlots) * (2 * D);
            const float s = ragged_dot<E, D>(k, qv, lane) * p.scale_log2, mn = fmaxf(m, s);
            const float al = exp2f(m - mn), w = exp2f(s - mn);
            m = mn;
            part = part * al + w;
            l *= al;
            if (j % 64 == 63) {
                l += part;
                part = 0.f;
            }
            for (int i = 0; i < D / 32; ++i) acc[i] = fmaf(w, E::get(k[D + lane + 32 * i]), acc[i] * al);
        }
    }
    if (!ok) {
        for (int i = 0; p.zero && i < D / 32; ++i) out[lane + 32 * i] = 0;
        return;
    }
    l += part;
    for (int i = 0; i < D / 32; ++i) out[lane + 32 * i] = E::put(l == 0.f ? 0.f : acc[i] / l);
    if (p.lse && lane == 0) p.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

template <class E, int D>
__global__ void __launch_bounds__(128) key_rows_kernel(const __grid_constant__ RaggedParams p)
{
    if (threadIdx.x == 0) griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, r = blockIdx.z, g = blockIdx.y;
    const int j = blockIdx.x * 4 + (threadIdx.x >> 5);
    const RaggedRequest q = ragged_request(p, r);
    if (q.n < 0 || j >= q.L) return;
    const int page = p.block_table[(int64_t)r * p.max_blocks + j / kPageSlots];
    if (page < 0 || page >= p.num_pages) {
        atomicOr(&g_status, QKVF_STATUS_BAD_REQUEST);
        return;
    }
    const uint16_t *k = static_cast<const uint16_t *>(p.kv_cache) +
                        (((int64_t)page * p.nkv + g) * kPageSlots + j % kPageSlots) * (2 * D);
    float sum = 0.f;
    const int n = p.window ? min(q.n, p.window) : q.n;
    for (int i = max(q.n - n, j - (q.L - q.n)); i < q.n; ++i) {
        const int t = q.row0 + i;
        for (int h = g * p.group; h < (g + 1) * p.group; ++h) {
            float qv[D / 32];
            for (int d = 0; d < D / 32; ++d)
                qv[d] = E::get((static_cast<const uint16_t *>(p.q) + t * p.q_ts + h * p.q_hs)[lane + 32 * d]);
            const float lse = p.lse[(int64_t)t * p.q_heads + h];
            const float s = ragged_dot<E, D>(k, qv, lane);
            if (lse > -INFINITY) sum += exp2f(fmaf(s, p.scale_log2, -lse * 1.4426950408889634f));
        }
    }
    if (lane == 0) {
        const int64_t at = ((int64_t)r * p.nkv + g) * p.max_blocks * kPageSlots + j;
        p.out_weights[at] = p.decay == 0.f ? sum : fmaf(p.decay, p.weights[at], sum);
    }
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

const char *check_key_weights_args(const RaggedParams &p, int head_dim, float scale, int dtype, const void *workspace,
                                   size_t workspace_bytes, int *code)
{
    if (const char *why = check_ragged_args(p.q, p.q_ts, p.q_hs, p.kv_cache, p.num_pages, p.starts, p.block_table,
                                            p.max_blocks, p.context_lens, p.T, p.R, p.q_heads, p.nkv, head_dim, scale,
                                            dtype, workspace, code))
        return why;
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

size_t chunk_workspace(int head_dim, int sms) { return 512; }
size_t key_weights_workspace(int head_dim, int sms) { return 512; }

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
    const dim3 grid((unsigned)(((int64_t)T * q_heads + 3) / 4));
    return qkvf::launch_pdl(bf16 ? head_dim == 64 ? qkvf::chunk_rows_kernel<qkvf::Bf16, 64> : qkvf::chunk_rows_kernel<qkvf::Bf16, 128>
                                 : head_dim == 64 ? qkvf::chunk_rows_kernel<qkvf::Fp16, 64> : qkvf::chunk_rows_kernel<qkvf::Fp16, 128>,
                            grid, dim3(128), 0, stream, prm);
}

size_t key_weights_workspace_bytes(int T, int num_reqs, int q_heads, int num_kv_heads, int head_dim, int max_blocks)
{
    int code;
    if (qkvf::check_ragged_shape(T, num_reqs, q_heads, num_kv_heads, head_dim, max_blocks, &code)) return 0;
    qkvf::DeviceState *d;
    return qkvf::probe_device(&d) == QKVF_OK ? qkvf::key_weights_workspace(head_dim, d->sms) : 0;
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
    return num_reqs > 0 && workspace_bytes < qkvf::key_weights_workspace(head_dim, d->sms) ? "the workspace is too small" : nullptr;
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
    if (workspace_bytes < qkvf::key_weights_workspace(head_dim, d->sms)) return QKVF_ERR_SIZES;
    const bool bf16 = qkvf::dtype_of(dtype) == QKVF_DTYPE_BF16;
    const dim3 grid((unsigned)(max_blocks * qkvf::kPageSlots / 4), (unsigned)num_kv_heads, (unsigned)num_reqs);
    return qkvf::launch_pdl(bf16 ? head_dim == 64 ? qkvf::key_rows_kernel<qkvf::Bf16, 64> : qkvf::key_rows_kernel<qkvf::Bf16, 128>
                                 : head_dim == 64 ? qkvf::key_rows_kernel<qkvf::Fp16, 64> : qkvf::key_rows_kernel<qkvf::Fp16, 128>,
                            grid, dim3(128), 0, stream, prm);
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
