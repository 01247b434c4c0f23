// prefix_attn: decode attention of requests that share a prefix (included by
// qkv_front.cu: one translation unit).
//
// Row (request r, token i of its q_len, q head h) attends to the shared
// prefix's keys 0 .. P - 1 and to its request's own keys j <= L_r - q_len + i,
// under one softmax:
//   s = scale q . k;  out = sum exp(s - m) v / sum exp(s - m);  lse = ln sum exp(s).

namespace qkvf {

constexpr int kPaMaxRequests = 65535;
constexpr int kPaMaxQLen = 1024;
constexpr int kPaMaxGroup = 64;   // q heads per KV head

struct PrefixParams {
    const void *q;
    const void *kv_cache;
    const int32_t *prefix_pages;
    const int32_t *prefix_len;
    const int32_t *block_table;
    const int32_t *context_lens;
    void *out;
    float *lse;
    int64_t num_pages;
    int64_t q_ts, q_hs;
    int prefix_blocks, max_blocks;
    int R, q_len, q_heads, nkv, dim;
    float scale;
};

constexpr int kPaWarps = 4;

// One warp per row: lane l scores key 32 c + l of chunk c, then every lane
// accumulates dims l, l + 32, ... of the weighted V rows.
template <class E, int D>
__global__ void __launch_bounds__(32 * kPaWarps) prefix_attn_kernel(const PrefixParams p)
{
    __shared__ float qs[kPaWarps][D];
    if (threadIdx.x == 0) griddep_launch_dependents();
    griddep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * kPaWarps + warp;
    if (row >= (int64_t)p.R * p.q_len * p.q_heads) return;
    const int t = (int)(row / p.q_heads), h = (int)(row % p.q_heads), r = t / p.q_len, i = t % p.q_len;
    const int g = h / (p.q_heads / p.nkv);
    const int L = p.context_lens[r], P = p.prefix_blocks > 0 ? *p.prefix_len : 0;
    if (L < 0) return;   // a padding request
    bool bad = L > p.max_blocks * kPageSlots || P < 0 || P > p.prefix_blocks * kPageSlots;
    const int32_t *bt = p.block_table + (size_t)r * p.max_blocks;
    if (!bad) {
        for (int b = lane; b < (P + kPageSlots - 1) / kPageSlots; b += 32)
            bad |= p.prefix_pages[b] < 0 || p.prefix_pages[b] >= p.num_pages;
        for (int b = lane; b < (L + kPageSlots - 1) / kPageSlots; b += 32) bad |= bt[b] < 0 || bt[b] >= p.num_pages;
    }
    if (__any_sync(0xffffffffu, bad)) {
        if (lane == 0) atomicOr(&g_status, QKVF_STATUS_BAD_REQUEST);
        return;
    }
    const uint16_t *q = static_cast<const uint16_t *>(p.q) + t * p.q_ts + h * p.q_hs;
    for (int d = lane; d < D; d += 32) qs[warp][d] = E::get(q[d]) * p.scale;
    __syncwarp();
    float m = -INFINITY, l = 0.f, o[D / 32];
#pragma unroll
    for (int k = 0; k < D / 32; ++k) o[k] = 0.f;
    for (int part = 0; part < 2; ++part) {
        const int32_t *pages = part == 0 ? p.prefix_pages : bt;
        const int keys = part == 0 ? P : max(0, L - p.q_len + i + 1);
        for (int c = 0; c < keys; c += 32) {
            const int j = c + lane;
            const uint16_t *kv = static_cast<const uint16_t *>(p.kv_cache);
            float s = -INFINITY;
            if (j < keys) {
                kv += (((int64_t)pages[j / kPageSlots] * p.nkv + g) * kPageSlots + j % kPageSlots) * (2 * D);
                s = 0.f;
                for (int d = 0; d < D; ++d) s = fmaf(qs[warp][d], E::get(kv[d]), s);
            }
            float mx = s;
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
            const float mn = fmaxf(m, mx), base = mn == -INFINITY ? 0.f : mn;
            const float w = j < keys ? expf(s - base) : 0.f, al = expf(m - base);
            float sum = w;
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            l = l * al + sum;
            m = mn;
#pragma unroll
            for (int k = 0; k < D / 32; ++k) o[k] *= al;
            for (int jj = 0; jj < 32 && c + jj < keys; ++jj) {
                const float wj = __shfl_sync(0xffffffffu, w, jj);
                const uint16_t *vj = reinterpret_cast<const uint16_t *>(
                    __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(kv), jj));
#pragma unroll
                for (int k = 0; k < D / 32; ++k) o[k] = fmaf(wj, E::get(vj[D + 32 * k + lane]), o[k]);
            }
        }
    }
    uint16_t *out = static_cast<uint16_t *>(p.out) + row * D;
#pragma unroll
    for (int k = 0; k < D / 32; ++k) out[32 * k + lane] = E::put(l == 0.f ? 0.f : o[k] / l);
    if (p.lse && lane == 0) p.lse[row] = l == 0.f ? -INFINITY : m + logf(l);
}

size_t prefix_attn_workspace(int num_reqs, int q_len, int q_heads, int nkv, int head_dim, int prefix_blocks,
                             int max_blocks)
{
    (void)num_reqs, (void)q_len, (void)q_heads, (void)nkv, (void)head_dim, (void)prefix_blocks, (void)max_blocks;
    return 256;
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
    if ((int64_t)num_reqs * q_len * q_heads > (int64_t(1) << 26)) return "num_reqs * q_len * q_heads must be <= 2^26";
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
    if (const char *why = check_prefix_shape(num_reqs, q_len, q_heads, num_kv_heads, head_dim, prefix_blocks,
                                             max_blocks, code))
        return why;
    *code = QKVF_ERR_LAYOUT;
    if (dtype != QKVF_DTYPE_BF16 && dtype != QKVF_DTYPE_FP16) return "dtype must be bf16 or fp16";
    if (!stride_ok(q_ts) || !stride_ok(q_hs) || q_ts % 8 || q_hs % 8)
        return "q's strides must be multiples of 8 elements, 0..2^36";
    *code = QKVF_ERR_SIZES;
    if (num_pages < 1 || num_pages * num_kv_heads > (int64_t(1) << 31)) return "num_pages * num_kv_heads must be 1..2^31";
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
    *code = QKVF_ERR_SIZES;
    const size_t need = prefix_attn_workspace(num_reqs, q_len, q_heads, num_kv_heads, head_dim, prefix_blocks, max_blocks);
    if (need == 0 || workspace_bytes < need) return "the workspace is too small";
    *code = QKVF_ERR_ARG;
    const size_t rows = (size_t)num_reqs * q_len * q_heads;
    const View vq = view_of(q, num_reqs * q_len, q_ts, q_heads, q_hs, head_dim, 2);
    const void *parts[] = {vq.ptr, kv_cache, context_lens, block_table, prefix_pages, prefix_len, out, lse, workspace};
    const size_t bytes[] = {vq.extent, (size_t)num_pages * num_kv_heads * kPageSlots * 2 * head_dim * 2,
                            (size_t)num_reqs * 4, (size_t)num_reqs * max_blocks * 4, (size_t)prefix_blocks * 4,
                            prefix_blocks > 0 ? (size_t)4 : 0, rows * head_dim * 2, lse ? rows * 4 : 0, need};
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
    return qkvf::prefix_attn_workspace(num_reqs, q_len, q_heads, num_kv_heads, head_dim, prefix_blocks, max_blocks);
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
    qkvf::DeviceState *d;
    const int rc = qkvf::probe_device(&d);
    return rc == QKVF_OK ? nullptr : qkv_front_strerror(rc);
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
    const int rc = qkvf::probe_device(&d);
    if (rc != QKVF_OK) return rc;
    qkvf::PrefixParams prm = {};
    prm.q = q;
    prm.kv_cache = kv_cache;
    prm.prefix_pages = prefix_pages;
    prm.prefix_len = prefix_len;
    prm.block_table = block_table;
    prm.context_lens = context_lens;
    prm.out = out;
    prm.lse = lse;
    prm.num_pages = num_pages;
    prm.q_ts = q_token_stride;
    prm.q_hs = q_head_stride;
    prm.prefix_blocks = prefix_blocks;
    prm.max_blocks = max_blocks;
    prm.R = num_reqs;
    prm.q_len = q_len;
    prm.q_heads = q_heads;
    prm.nkv = num_kv_heads;
    prm.dim = head_dim;
    prm.scale = scale;
    const int64_t rows = (int64_t)num_reqs * q_len * q_heads;
    auto kernel = dtype == QKVF_DTYPE_BF16
                      ? (head_dim == 64 ? qkvf::prefix_attn_kernel<qkvf::Bf16, 64> : qkvf::prefix_attn_kernel<qkvf::Bf16, 128>)
                      : (head_dim == 64 ? qkvf::prefix_attn_kernel<qkvf::Fp16, 64> : qkvf::prefix_attn_kernel<qkvf::Fp16, 128>);
    return qkvf::launch_pdl(kernel, dim3((unsigned)((rows + qkvf::kPaWarps - 1) / qkvf::kPaWarps)),
                            dim3(32 * qkvf::kPaWarps), 0, stream, prm);
}

}  // extern "C"
