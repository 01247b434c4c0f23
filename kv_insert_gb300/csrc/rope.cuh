// rope_table, rope: rotary positions for any head layout (included by
// qkv_front.cu: one translation unit).
//
// A pair (a, b) of a head's columns is turned by its position's angle p f_i:
//   (a, b) -> (a c - b s, b c + a s),   c = cos(p f_i), s = sin(p f_i),
// pairs being columns (2i, 2i + 1) (interleaved) or (i, i + rot / 2) (half) of
// the head's first rot columns; the columns behind them are copied.  The
// gradient of a rotation is the turn by -p f_i: the same kernel with s negated.

namespace qkvf {

constexpr int kRopeMaxTokens = 1 << 24;
constexpr int kRopeMaxHeads = 4096;
constexpr int kRopeMaxDim = 512;
constexpr int64_t kMaxStride = int64_t(1) << 36;   // elements; extents then stay far below 2^63 bytes

// ---- element types ---------------------------------------------------------

__host__ __device__ inline int dtype_bytes(int dtype) { return dtype == QKVF_DTYPE_FP32 ? 4 : 2; }

struct Bf16 {
    using store = uint16_t;
    static __device__ __forceinline__ float get(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
    static __device__ __forceinline__ uint16_t put(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }
    static constexpr bool is_bf16 = true;
    static __device__ __forceinline__ uint32_t pack(float lo, float hi)
    {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
};
struct Fp16 {
    using store = uint16_t;
    static __device__ __forceinline__ float get(uint16_t v) { return __half2float(__ushort_as_half(v)); }
    static __device__ __forceinline__ uint16_t put(float v) { return __half_as_ushort(__float2half_rn(v)); }
    static constexpr bool is_bf16 = false;
    static __device__ __forceinline__ uint32_t pack(float lo, float hi)
    {
        const __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
};
struct Fp32 {
    using store = float;
    static __device__ __forceinline__ float get(float v) { return v; }
    static __device__ __forceinline__ float put(float v) { return v; }
};

// ---- strided [tokens, heads, dim] views ------------------------------------

// A view's extent in bytes, and its rows for the overlap test: the dimension
// with the larger stride is the outer one, `span` bytes of each of its rows
// may be touched.
struct View {
    const void *ptr;
    size_t extent;
    size_t outer;   // outer stride in bytes (0: a single row)
    size_t span;
};

View view_of(const void *ptr, int T, int64_t ts, int heads, int64_t hs, int dim, int elt)
{
    View v;
    v.ptr = ptr;
    const int64_t st = T > 1 ? ts : 0, sh = heads > 1 ? hs : 0;
    const bool token_outer = st >= sh;
    const int64_t inner = token_outer ? (int64_t)(heads - 1) * sh : (int64_t)(T - 1) * st;
    const int64_t outer = token_outer ? (int64_t)(T - 1) * st : (int64_t)(heads - 1) * sh;
    v.span = (size_t)(inner + dim) * elt;
    v.extent = (size_t)(inner + outer + dim) * elt;
    v.outer = (size_t)(token_outer ? st : sh) * elt;
    return v;
}

// Whether two views may share a byte.  Views of one packed buffer (equal
// outer strides, each row's bytes within a stride) are compared column by
// column; anything else by its whole extent.
bool views_overlap(const View &a, const View &b)
{
    if (!overlap(a.ptr, a.extent, b.ptr, b.extent)) return false;
    if (a.outer != b.outer || a.outer == 0 || a.span > a.outer || b.span > b.outer) return true;
    const uintptr_t pa = (uintptr_t)a.ptr, pb = (uintptr_t)b.ptr;
    const size_t off = pb >= pa ? (pb - pa) % a.outer : (a.outer - (pa - pb) % a.outer) % a.outer;
    return off < a.span || off + b.span > a.outer;
}

// A view whose elements are all different addresses (an output must be one)
bool view_distinct(int T, int64_t ts, int heads, int64_t hs, int dim)
{
    if (T > 1 && heads > 1) {
        if (ts >= hs) return hs >= dim && ts >= (int64_t)(heads - 1) * hs + dim;
        return ts >= dim && hs >= (int64_t)(T - 1) * ts + dim;
    }
    return (T <= 1 || ts >= dim) && (heads <= 1 || hs >= dim);
}

bool stride_ok(int64_t s) { return s >= 0 && s <= kMaxStride; }

// ---- the table -------------------------------------------------------------

constexpr int kRtMaxPairs = kRopeMaxDim / 2;

// Each pair's frequency in turns per position as a 64-bit fraction: a
// position's angle is the low 64 bits of position * rate, exact modulo one
// turn however far the position (a 32-bit product of both would lose the
// angle beyond 2^24 / f positions).
struct RopeTableParams {
    float *table;
    int64_t first;
    int64_t rows;
    int half;
    float magnitude;
    uint64_t rate[kRtMaxPairs];
};

__global__ void __launch_bounds__(256) rope_table_kernel(const __grid_constant__ RopeTableParams p)
{
    if (threadIdx.x == 0) griddep_launch_dependents();
    griddep_wait();
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x)
        for (int i = threadIdx.x; i < p.half; i += blockDim.x) {
            const uint64_t phase = (uint64_t)(p.first + row) * p.rate[i];
            // twice the signed fraction of a turn: [-1, 1) half turns
            const float h = __ll2float_rn((long long)phase) * 0x1p-63f;
            float sn, cs;
            sincospif(h, &sn, &cs);
            float *dst = p.table + row * (2 * p.half);
            dst[i] = cs * p.magnitude;
            dst[p.half + i] = sn * p.magnitude;
        }
}

const char *check_rope_table_args(const float *table, int64_t first, int64_t rows, int rot_dim, double base,
                                  int scaling, double factor, int64_t original_len, double slow, double fast,
                                  double magnitude, int *code)
{
    *code = QKVF_ERR_LAYOUT;
    if (rot_dim < 2 || rot_dim > kRopeMaxDim || rot_dim % 2) return "rot_dim must be even, 2..512";
    *code = QKVF_ERR_SIZES;
    if (rows < 0 || first < 0 || rows > (int64_t(1) << 32) || first > (int64_t(1) << 40))
        return "rows must be 0..2^32 and the first position 0..2^40";
    *code = QKVF_ERR_ARG;
    if (!(base > 1.0) || !(base <= 1e30)) return "base must be in (1, 1e30]";
    if (scaling < QKVF_ROPE_NONE || scaling > QKVF_ROPE_RAMP) return "unknown scaling";
    if (scaling != QKVF_ROPE_NONE && (!(factor >= 1.0) || !(factor <= 1e9))) return "factor must be in [1, 1e9]";
    if (scaling == QKVF_ROPE_BASE && rot_dim < 4) return "base scaling needs a rot_dim of 4 or more";
    if (scaling == QKVF_ROPE_RAMP && (original_len < 1 || !(slow >= 0.0) || !(fast > slow) || !(fast <= 1e9)))
        return "ramp scaling needs original_len >= 1 and 0 <= slow < fast";
    if (!(magnitude > 0.0) || !(magnitude <= 1e6)) return "magnitude must be in (0, 1e6]";
    *code = QKVF_OK;
    if (rows == 0) return nullptr;
    *code = QKVF_ERR_NULL;
    if (!table) return "the table pointer is NULL";
    *code = QKVF_ERR_ALIGN;
    if (!aligned(table, 16)) return "the table must be 16-byte aligned";
    *code = QKVF_OK;
    return nullptr;
}

// ---- the rotation ----------------------------------------------------------

struct RopeParams {
    const void *x;
    void *out;
    const int64_t *positions;
    const float *cos_sin;
    int64_t cos_rows;
    int64_t x_ts, x_hs, o_ts, o_hs;   // strides in elements
    int T, heads, dim, rot;
    int half_layout;
    float sign;      // -1: the gradient
    int in_place;    // the columns behind rot are already where they belong
};

// (a, b) turned: each result is two FP32 products and a sum, rounded once more
// to the output's type
__device__ __forceinline__ void rope_pair(float a, float b, float c, float s, float &ya, float &yb)
{
    ya = fmaf(a, c, -(b * s));
    yb = fmaf(b, c, a * s);
}

// One CTA per token (round robin), one pair or one copied column per thread.
template <class E>
__global__ void __launch_bounds__(256) rope_kernel(const RopeParams p)
{
    using S = typename E::store;
    if (threadIdx.x == 0) griddep_launch_dependents();
    griddep_wait();
    const int half = p.rot >> 1, units = half + (p.in_place ? 0 : p.dim - p.rot);
    for (int t = blockIdx.x; t < p.T; t += gridDim.x) {
        const int64_t pos = p.positions[t];
        if (pos < 0 || pos >= p.cos_rows) {
            if (threadIdx.x == 0) atomicOr(&g_status, QKVF_STATUS_BAD_POSITION);
            continue;
        }
        const float *row = p.cos_sin + pos * p.rot;
        for (int u = threadIdx.x; u < units * p.heads; u += blockDim.x) {
            const int h = u / units, i = u % units;
            const S *src = static_cast<const S *>(p.x) + t * p.x_ts + h * p.x_hs;
            S *dst = static_cast<S *>(p.out) + t * p.o_ts + h * p.o_hs;
            if (i < half) {
                const int ca = p.half_layout ? i : 2 * i, cb = p.half_layout ? i + half : 2 * i + 1;
                float ya, yb;
                rope_pair(E::get(src[ca]), E::get(src[cb]), row[i], p.sign * row[half + i], ya, yb);
                dst[ca] = E::put(ya);
                dst[cb] = E::put(yb);
            } else {
                dst[p.rot + i - half] = src[p.rot + i - half];
            }
        }
    }
}

const char *check_rope_args(const void *x, int64_t x_ts, int64_t x_hs, const int64_t *positions,
                            const float *cos_sin, int64_t cos_sin_rows, void *out, int64_t o_ts, int64_t o_hs,
                            int T, int heads, int head_dim, int rot_dim, int layout, int inverse, int dtype,
                            int *code)
{
    *code = QKVF_ERR_TOKENS;
    if (T < 0 || T > kRopeMaxTokens) return "T must be 0..16777216 tokens";
    *code = QKVF_ERR_LAYOUT;
    if (dtype < QKVF_DTYPE_BF16 || dtype > QKVF_DTYPE_FP32) return "dtype must be bf16, fp16 or fp32";
    if (heads < 1 || heads > kRopeMaxHeads) return "heads must be 1..4096";
    if (head_dim < 2 || head_dim > kRopeMaxDim) return "head_dim must be 2..512";
    if (rot_dim < 2 || rot_dim > head_dim || rot_dim % 2) return "rot_dim must be even, 2..head_dim";
    if (layout != QKVF_ROPE_INTERLEAVED && layout != QKVF_ROPE_HALF) return "layout must be interleaved or half";
    if (!stride_ok(x_ts) || !stride_ok(x_hs) || !stride_ok(o_ts) || !stride_ok(o_hs))
        return "strides must be 0..2^36 elements";
    if (!view_distinct(T, o_ts, heads, o_hs, head_dim)) return "out's strides make its heads overlap";
    *code = QKVF_ERR_ARG;
    if (inverse != 0 && inverse != 1) return "inverse must be 0 or 1";
    *code = QKVF_ERR_SIZES;
    if (cos_sin_rows < 1 || cos_sin_rows > (int64_t(1) << 40)) return "cos_sin_rows must be >= 1";
    *code = QKVF_OK;
    if (T == 0) return nullptr;
    *code = QKVF_ERR_NULL;
    if (!x || !positions || !cos_sin || !out) return "a required pointer is NULL";
    *code = QKVF_ERR_ALIGN;
    const int elt = dtype_bytes(dtype);
    if (!aligned(x, elt) || !aligned(out, elt)) return "x and out must be aligned to their elements";
    if (!aligned(cos_sin, 16)) return "cos_sin must be 16-byte aligned";
    if (!aligned(positions, 8)) return "positions must be 8-byte aligned int64";
    *code = QKVF_ERR_ARG;
    const View vx = view_of(x, T, x_ts, heads, x_hs, head_dim, elt);
    const View vo = view_of(out, T, o_ts, heads, o_hs, head_dim, elt);
    const bool same = x == out && (T == 1 || x_ts == o_ts) && (heads == 1 || x_hs == o_hs);
    if (!same && views_overlap(vx, vo)) return "out overlaps x without being x";
    if (overlap(positions, (size_t)T * 8, out, vo.extent) ||
        overlap(cos_sin, (size_t)cos_sin_rows * rot_dim * 4, out, vo.extent))
        return "an input overlaps out";
    *code = QKVF_OK;
    return nullptr;
}

// Launch with PDL on `stream`; every kernel here waits for the kernel before
// it ahead of its first load or store.
template <class... Args>
int launch_pdl(void (*kernel)(Args...), dim3 grid, dim3 block, size_t smem, void *stream, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = g_pdl ? 1 : 0;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) {
        (void)cudaGetLastError();
        return QKVF_ERR_CUDA;
    }
    return QKVF_OK;
}

}  // namespace qkvf

extern "C" {

const char *rope_table_unsupported(const float *table, int64_t first, int64_t rows, int rot_dim, double base,
                                   int scaling, double factor, int64_t original_len, double slow, double fast,
                                   double magnitude)
{
    int code;
    const char *why = qkvf::check_rope_table_args(table, first, rows, rot_dim, base, scaling, factor,
                                                  original_len, slow, fast, magnitude, &code);
    if (why) return why;
    qkvf::DeviceState *d;
    const int rc = qkvf::probe_device(&d);
    return rc == QKVF_OK ? nullptr : qkv_front_strerror(rc);
}

int rope_table(float *table, int64_t first, int64_t rows, int rot_dim, double base, int scaling, double factor,
               int64_t original_len, double slow, double fast, double magnitude, void *stream)
{
    int code;
    if (qkvf::check_rope_table_args(table, first, rows, rot_dim, base, scaling, factor, original_len, slow,
                                    fast, magnitude, &code))
        return code;
    if (rows == 0) return QKVF_OK;
    qkvf::DeviceState *d;
    const int rc = qkvf::probe_device(&d);
    if (rc != QKVF_OK) return rc;
    qkvf::RopeTableParams prm;
    prm.table = table;
    prm.first = first;
    prm.rows = rows;
    prm.half = rot_dim / 2;
    prm.magnitude = (float)magnitude;
    if (scaling == QKVF_ROPE_BASE) base *= pow(factor, rot_dim / (rot_dim - 2.0));
    constexpr double kTurn = 6.283185307179586476925286766559;
    for (int i = 0; i < prm.half; ++i) {
        double f = pow(base, -2.0 * i / rot_dim);
        if (scaling == QKVF_ROPE_LINEAR) f /= factor;
        if (scaling == QKVF_ROPE_RAMP) {
            double g = ((double)original_len * f / kTurn - slow) / (fast - slow);
            g = g < 0.0 ? 0.0 : (g > 1.0 ? 1.0 : g);
            f = (1.0 - g) * f / factor + g * f;
        }
        prm.rate[i] = (uint64_t)ldexp(f / kTurn, 64);   // f <= 1: below 2^62
    }
    const int64_t most = (int64_t)d->sms * 8;
    return qkvf::launch_pdl(qkvf::rope_table_kernel, dim3((unsigned)(rows < most ? rows : most)), dim3(256), 0,
                            stream, prm);
}

const char *rope_unsupported(const void *x, int64_t x_token_stride, int64_t x_head_stride,
                             const int64_t *positions, const float *cos_sin, int64_t cos_sin_rows, void *out,
                             int64_t out_token_stride, int64_t out_head_stride, int T, int heads, int head_dim,
                             int rot_dim, int layout, int inverse, int dtype)
{
    int code;
    const char *why = qkvf::check_rope_args(x, x_token_stride, x_head_stride, positions, cos_sin, cos_sin_rows,
                                            out, out_token_stride, out_head_stride, T, heads, head_dim, rot_dim,
                                            layout, inverse, dtype, &code);
    if (why) return why;
    qkvf::DeviceState *d;
    const int rc = qkvf::probe_device(&d);
    return rc == QKVF_OK ? nullptr : qkv_front_strerror(rc);
}

int rope(const void *x, int64_t x_token_stride, int64_t x_head_stride, const int64_t *positions,
         const float *cos_sin, int64_t cos_sin_rows, void *out, int64_t out_token_stride,
         int64_t out_head_stride, int T, int heads, int head_dim, int rot_dim, int layout, int inverse,
         int dtype, void *stream)
{
    int code;
    if (qkvf::check_rope_args(x, x_token_stride, x_head_stride, positions, cos_sin, cos_sin_rows, out,
                              out_token_stride, out_head_stride, T, heads, head_dim, rot_dim, layout, inverse,
                              dtype, &code))
        return code;
    if (T == 0) return QKVF_OK;
    qkvf::DeviceState *d;
    const int rc = qkvf::probe_device(&d);
    if (rc != QKVF_OK) return rc;
    qkvf::RopeParams prm = {};
    prm.x = x;
    prm.out = out;
    prm.positions = positions;
    prm.cos_sin = cos_sin;
    prm.cos_rows = cos_sin_rows;
    prm.x_ts = x_token_stride;
    prm.x_hs = x_head_stride;
    prm.o_ts = out_token_stride;
    prm.o_hs = out_head_stride;
    prm.T = T;
    prm.heads = heads;
    prm.dim = head_dim;
    prm.rot = rot_dim;
    prm.half_layout = layout == QKVF_ROPE_HALF;
    prm.sign = inverse ? -1.f : 1.f;
    prm.in_place = x == out;
    const int64_t most = (int64_t)d->sms * 8;
    const dim3 grid((unsigned)(T < most ? T : most));
    auto kernel = dtype == QKVF_DTYPE_BF16   ? qkvf::rope_kernel<qkvf::Bf16>
                  : dtype == QKVF_DTYPE_FP16 ? qkvf::rope_kernel<qkvf::Fp16>
                                             : qkvf::rope_kernel<qkvf::Fp32>;
    return qkvf::launch_pdl(kernel, grid, dim3(256), 0, stream, prm);
}

}  // extern "C"
