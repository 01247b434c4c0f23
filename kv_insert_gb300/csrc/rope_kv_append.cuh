// rope_kv_append: rotate a step's q and k heads and write its k and v heads
// into the paged cache, for any head width, rotary layout and strides
// (included by qkv_front.cu after rope.cuh: one translation unit).
//
// The kernels are rope.cuh's, over the heads q, k and v of a token: k head g
// goes to the K half and v head g to the V half of slot slots[t] of KV head g,
// as in qknorm_rope_kv_insert (which also norms, for one fixed layout).

namespace qkvf {

const char *check_append_args(const void *q, int64_t q_ts, int64_t q_hs, const void *k, int64_t k_ts,
                              int64_t k_hs, const void *v, int64_t v_ts, int64_t v_hs,
                              const int64_t *positions, const int64_t *slots, const float *cos_sin,
                              int64_t cos_sin_rows, void *q_out, int64_t o_ts, int64_t o_hs, void *kv_cache,
                              int64_t num_pages, int T, int q_heads, int num_kv_heads, int head_dim, int rot_dim,
                              int layout, int dtype, int *code)
{
    dtype = dtype_of(dtype);
    *code = QKVF_ERR_TOKENS;
    if (T < 0 || T > kRopeMaxTokens) return "T must be 0..16777216 tokens";
    *code = QKVF_ERR_LAYOUT;
    if (dtype != QKVF_DTYPE_BF16 && dtype != QKVF_DTYPE_FP16) return "dtype must be bf16 or fp16";
    if (q_heads < 0 || q_heads > kRopeMaxHeads) return "q_heads must be 0..4096";
    if (num_kv_heads < 1 || num_kv_heads > 1024) return "num_kv_heads must be 1..1024";
    if (head_dim < 8 || head_dim > kRopeMaxDim || head_dim % 8) return "head_dim must be a multiple of 8, 8..512";
    if (rot_dim < 2 || rot_dim > head_dim || rot_dim % 2) return "rot_dim must be even, 2..head_dim";
    if (layout != QKVF_ROPE_INTERLEAVED && layout != QKVF_ROPE_HALF) return "layout must be interleaved or half";
    if (!stride_ok(q_ts) || !stride_ok(q_hs) || !stride_ok(k_ts) || !stride_ok(k_hs) || !stride_ok(v_ts) ||
        !stride_ok(v_hs) || !stride_ok(o_ts) || !stride_ok(o_hs))
        return "strides must be 0..2^36 elements";
    if (q_heads > 0 && !view_distinct(T, o_ts, q_heads, o_hs, head_dim)) return "q_out's strides make its heads overlap";
    *code = QKVF_ERR_SIZES;
    if (cos_sin_rows < 1 || cos_sin_rows > (int64_t(1) << 40)) return "cos_sin_rows must be >= 1";
    if (num_pages < 1 || num_pages > (int64_t(1) << 36)) return "num_pages must be >= 1";
    *code = QKVF_OK;
    if (T == 0) return nullptr;
    *code = QKVF_ERR_NULL;
    if (!k || !v || !positions || !slots || !cos_sin || !kv_cache || (q_heads > 0 && (!q || !q_out)))
        return "a required pointer is NULL";
    *code = QKVF_ERR_ALIGN;
    if (!aligned(k, 2) || !aligned(v, 2) || (q_heads > 0 && (!aligned(q, 2) || !aligned(q_out, 2))))
        return "q, k, v and q_out must be aligned to their elements";
    if (!aligned(cos_sin, 16) || !aligned(kv_cache, 16)) return "cos_sin and kv_cache must be 16-byte aligned";
    if (!aligned(positions, 8) || !aligned(slots, 8)) return "positions and slots must be 8-byte aligned int64";
    *code = QKVF_ERR_ARG;
    const size_t cache_b = (size_t)num_pages * num_kv_heads * kPageSlots * 2 * head_dim * 2;
    const size_t cs_b = (size_t)cos_sin_rows * rot_dim * 4, idx_b = (size_t)T * 8;
    const View vk = view_of(k, T, k_ts, num_kv_heads, k_hs, head_dim, 2);
    const View vv = view_of(v, T, v_ts, num_kv_heads, v_hs, head_dim, 2);
    if (overlap(vk.ptr, vk.extent, kv_cache, cache_b) || overlap(vv.ptr, vv.extent, kv_cache, cache_b) ||
        overlap(cos_sin, cs_b, kv_cache, cache_b) || overlap(positions, idx_b, kv_cache, cache_b) ||
        overlap(slots, idx_b, kv_cache, cache_b))
        return "an input overlaps kv_cache";
    if (q_heads > 0) {
        const View vq = view_of(q, T, q_ts, q_heads, q_hs, head_dim, 2);
        const View vo = view_of(q_out, T, o_ts, q_heads, o_hs, head_dim, 2);
        if (overlap(vq.ptr, vq.extent, kv_cache, cache_b) || overlap(vo.ptr, vo.extent, kv_cache, cache_b))
            return "q or q_out overlaps kv_cache";
        const bool same = q == q_out && (T == 1 || q_ts == o_ts) && (q_heads == 1 || q_hs == o_hs);
        if (!same && views_overlap(vq, vo)) return "q_out overlaps q without being q";
        if (views_overlap(vk, vo) || views_overlap(vv, vo) || overlap(cos_sin, cs_b, vo.ptr, vo.extent) ||
            overlap(positions, idx_b, vo.ptr, vo.extent) || overlap(slots, idx_b, vo.ptr, vo.extent))
            return "an input overlaps q_out";
    }
    *code = QKVF_OK;
    return nullptr;
}

}  // namespace qkvf

extern "C" {

const char *rope_kv_append_unsupported(const void *q, int64_t q_token_stride, int64_t q_head_stride,
                                       const void *k, int64_t k_token_stride, int64_t k_head_stride,
                                       const void *v, int64_t v_token_stride, int64_t v_head_stride,
                                       const int64_t *positions, const int64_t *slots, const float *cos_sin,
                                       int64_t cos_sin_rows, void *q_out, int64_t q_out_token_stride,
                                       int64_t q_out_head_stride, void *kv_cache, int64_t num_pages, int T,
                                       int q_heads, int num_kv_heads, int head_dim, int rot_dim, int layout,
                                       int dtype)
{
    int code;
    const char *why = qkvf::check_append_args(
        q, q_token_stride, q_head_stride, k, k_token_stride, k_head_stride, v, v_token_stride, v_head_stride,
        positions, slots, cos_sin, cos_sin_rows, q_out, q_out_token_stride, q_out_head_stride, kv_cache,
        num_pages, T, q_heads, num_kv_heads, head_dim, rot_dim, layout, dtype, &code);
    if (why) return why;
    qkvf::DeviceState *d;
    const int rc = qkvf::probe_device(&d);
    return rc == QKVF_OK ? nullptr : qkv_front_strerror(rc);
}

int rope_kv_append(const void *q, int64_t q_token_stride, int64_t q_head_stride, const void *k,
                   int64_t k_token_stride, int64_t k_head_stride, const void *v, int64_t v_token_stride,
                   int64_t v_head_stride, const int64_t *positions, const int64_t *slots, const float *cos_sin,
                   int64_t cos_sin_rows, void *q_out, int64_t q_out_token_stride, int64_t q_out_head_stride,
                   void *kv_cache, int64_t num_pages, int T, int q_heads, int num_kv_heads, int head_dim,
                   int rot_dim, int layout, int dtype, void *stream)
{
    int code;
    if (qkvf::check_append_args(q, q_token_stride, q_head_stride, k, k_token_stride, k_head_stride, v,
                                v_token_stride, v_head_stride, positions, slots, cos_sin, cos_sin_rows, q_out,
                                q_out_token_stride, q_out_head_stride, kv_cache, num_pages, T, q_heads,
                                num_kv_heads, head_dim, rot_dim, layout, dtype, &code))
        return code;
    if (T == 0) return QKVF_OK;
    qkvf::DeviceState *d;
    const int rc = qkvf::probe_device(&d);
    if (rc != QKVF_OK) return rc;
    qkvf::RopeParams prm = {};
    prm.q = q;
    prm.k = k;
    prm.v = v;
    prm.out = q_out;
    prm.kv_cache = kv_cache;
    prm.positions = positions;
    prm.slots = slots;
    prm.cos_sin = cos_sin;
    prm.cos_rows = cos_sin_rows;
    prm.slot_end = num_pages * qkvf::kPageSlots;
    prm.q_ts = q_token_stride;
    prm.q_hs = q_head_stride;
    prm.k_ts = k_token_stride;
    prm.k_hs = k_head_stride;
    prm.v_ts = v_token_stride;
    prm.v_hs = v_head_stride;
    prm.o_ts = q_out_token_stride;
    prm.o_hs = q_out_head_stride;
    prm.T = T;
    prm.q_heads = q_heads;
    prm.nkv = num_kv_heads;
    prm.dim = head_dim;
    prm.rot = rot_dim;
    prm.in_place = q == q_out;
    prm.zero = qkvf::zero_skipped(dtype);
    dtype = qkvf::dtype_of(dtype);
    prm.sign = 1.f;
    const bool half = layout == QKVF_ROPE_HALF;
    return dtype == QKVF_DTYPE_BF16 ? qkvf::launch_rope<qkvf::Bf16>(prm, half, d->sms, stream)
                                    : qkvf::launch_rope<qkvf::Fp16>(prm, half, d->sms, stream);
}

int rope_kv_append_packed(const int64_t *args, void *stream)
{
    if (!args) return QKVF_ERR_NULL;
    qkvf::Words w(args);
    const int T = w.i(18), q_heads = w.i(19), nkv = w.i(20), dim = w.i(21), rot = w.i(22), layout = w.i(23), dtype = w.i(24);
    if (!w.ok) return QKVF_ERR_SIZES;
    return rope_kv_append(w.p<void>(0), args[1], args[2], w.p<void>(3), args[4], args[5], w.p<void>(6), args[7], args[8],
                          w.p<int64_t>(9), w.p<int64_t>(10), w.p<float>(11), args[12], w.p<void>(13), args[14], args[15],
                          w.p<void>(16), args[17], T, q_heads, nkv, dim, rot, layout, dtype, stream);
}

}  // extern "C"
