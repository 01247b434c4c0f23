// rope_table, rope: rotary positions for any head layout (included by
// qkv_front.cu: one translation unit).
//
// A pair (a, b) of a head's columns is turned by its position's angle p f_i:
//   (a, b) -> (a c - b s, b c + a s),   c = cos(p f_i), s = sin(p f_i),
// pairs being columns (2i, 2i + 1) (interleaved) or (i, i + rot / 2) (half) of
// the head's first rot columns; the columns behind them are copied.  The
// gradient of a rotation is the turn by -p f_i: the same kernel with s negated.
//
// Bound by bytes: 16384 tokens x 32 heads of 128 (bf16) take 41.4 us, the
// copy rate; 4096 tokens of 8 KV heads of 64 into the cache 15.4 us (12.7 at
// the copy rate); a table of 131072 x 128 13.3 us (10.0; its sines and cosines
// are the rest); 4099 x 25 heads of 80 (fp16, 32 columns rotated) 8.5 us, of
// which 5.0 are bytes and ~2.4 the launch's start and first loads, as in every
// call of a few tokens.

namespace qkvf {

constexpr int kRopeMaxTokens = 1 << 24;
constexpr int kRopeMaxHeads = 4096;
constexpr int kRopeMaxDim = 512;
constexpr int64_t kMaxStride = int64_t(1) << 36;   // elements; extents then stay far below 2^63 bytes

// ---- element types ---------------------------------------------------------

__host__ __device__ inline int dtype_bytes(int dtype) { return dtype == QKVF_DTYPE_FP32 ? 4 : 2; }

// A dtype argument without and with its flag
inline int dtype_of(int arg) { return arg & ~QKVF_DTYPE_ZERO_SKIPPED; }
inline bool zero_skipped(int arg) { return arg & QKVF_DTYPE_ZERO_SKIPPED; }

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
    static __device__ __forceinline__ float lo(uint32_t v) { return get((uint16_t)v); }
    static __device__ __forceinline__ float hi(uint32_t v) { return get((uint16_t)(v >> 16)); }
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
    static __device__ __forceinline__ float lo(uint32_t v) { return get((uint16_t)v); }
    static __device__ __forceinline__ float hi(uint32_t v) { return get((uint16_t)(v >> 16)); }
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

// Each pair's frequency in turns per position as a 64-bit fraction, from a
// double: a position's angle is the low 64 bits of position * rate.  The product
// loses nothing however far the position, so the angle is off by the
// frequency's own error alone, about position f 2^-51 radians (a 32-bit
// product would lose the angle beyond 2^24 / f positions).
struct RopeTableParams {
    float *table;
    int64_t first;
    int64_t rows;
    int half;
    float magnitude;
    uint64_t rate[kRtMaxPairs];
};

// A thread keeps one pair and walks the rows: the next row's phase is a 64-bit
// sum.  The phase's top 32 bits, signed, are its angle in 2^-31 half turns, and
// rounded to fp32 for the sine and cosine (2^-25 half turns at most).
__global__ void __launch_bounds__(256) rope_table_kernel(const __grid_constant__ RopeTableParams p)
{
    if (threadIdx.x == 0) griddep_launch_dependents();
    griddep_wait();
    const int per = 256 / p.half;   // rows of a CTA at a time
    const int r = threadIdx.x / p.half, i = threadIdx.x - r * p.half;
    if (r >= per) return;
    const int64_t row0 = (int64_t)blockIdx.x * per + r, step = (int64_t)gridDim.x * per;
    const uint64_t rate = p.rate[i];
    uint64_t phase = (uint64_t)(p.first + row0) * rate;
    const uint64_t turn = (uint64_t)step * rate;
    float *dst = p.table + row0 * (2 * p.half) + i;
    for (int64_t row = row0; row < p.rows; row += step, phase += turn, dst += step * (2 * p.half)) {
        float sn, cs;
        sincospif((float)(int)(uint32_t)(phase >> 32) * 0x1p-31f, &sn, &cs);
        dst[0] = cs * p.magnitude;
        dst[p.half] = sn * p.magnitude;
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

// One call of rope (nkv = 0) or of rope_kv_append: the heads of a token in the
// order q, k, v.  q is rotated into out, k into the K half of the token's
// cache slot, v copied into the V half.
struct RopeParams {
    const void *q, *k, *v;
    void *out;
    void *kv_cache;
    const int64_t *positions;
    const int64_t *slots;
    const float *cos_sin;
    int64_t cos_rows;
    int64_t slot_end;
    int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, o_ts, o_hs;   // strides in elements
    int T, q_heads, nkv, dim, rot;
    int in_place;    // out is q: the columns behind rot are where they belong
    float sign;      // -1: the gradient
    // the vector kernel's threads: unit u of a head group of a token
    int units, q_groups, groups, tokens;   // units of a head, head groups of q and of all, tokens of a grid row
    int q_per, kv_per;                     // heads of a group
    uint32_t unit_m, unit_s, group_m, group_s;
    int zero;        // a token left alone has zeros in out instead
};

// n / d for n < 2^31 by a product and a shift
void fast_div(uint32_t d, uint32_t *m, uint32_t *s)
{
    uint32_t l = 0;
    while ((uint64_t(1) << l) < d) ++l;
    *s = l;
    *m = (uint32_t)(((uint64_t(1) << 32) * ((uint64_t(1) << l) - d)) / d + 1);
}
__device__ __forceinline__ uint32_t div_by(uint32_t n, uint32_t m, uint32_t s) { return (__umulhi(n, m) + n) >> s; }

// (a, b) turned: a product and a fused sum in FP32, rounded once more to the
// output's type
__device__ __forceinline__ void rope_pair(float a, float b, float c, float s, float &ya, float &yb)
{
    ya = fmaf(a, c, -(b * s));
    yb = fmaf(b, c, a * s);
}

// A token's indices: whether its heads are rotated and its slot written, with
// the status bits of those that are not.  `first`: the thread that reports.
struct RopeToken {
    const float *row;   // its cos | sin row, null: leave the token alone
    int64_t slot;       // the element offset of its slot for KV head 0, or -1
};

__device__ __forceinline__ RopeToken rope_token(const RopeParams &p, int64_t pos, int64_t slot, bool first)
{
    RopeToken k;
    const bool pos_ok = pos >= 0 && pos < p.cos_rows;
    k.row = pos_ok ? p.cos_sin + pos * p.rot : nullptr;
    k.slot = pos_ok && slot >= 0 && slot < p.slot_end
                 ? ((slot / kPageSlots) * p.nkv * kPageSlots + slot % kPageSlots) * (2 * (int64_t)p.dim)
                 : -1;
    if (first && (!pos_ok || slot >= p.slot_end))
        atomicOr(&g_status, (pos_ok ? 0u : QKVF_STATUS_BAD_POSITION) | (slot >= p.slot_end ? QKVF_STATUS_BAD_SLOT : 0u));
    return k;
}

// Head h of token t: where it is read and written; dst null: not at all
template <class S>
__device__ __forceinline__ void rope_head(const RopeParams &p, int64_t t, int h, const RopeToken &k, const S *&src, S *&dst)
{
    if (h < p.q_heads) {
        src = static_cast<const S *>(p.q) + t * p.q_ts + h * p.q_hs;
        dst = static_cast<S *>(p.out) + t * p.o_ts + h * p.o_hs;
    } else {
        const bool is_v = h >= p.q_heads + p.nkv;
        const int g = h - p.q_heads - (is_v ? p.nkv : 0);
        src = is_v ? static_cast<const S *>(p.v) + t * p.v_ts + g * p.v_hs : static_cast<const S *>(p.k) + t * p.k_ts + g * p.k_hs;
        dst = k.slot < 0 ? nullptr
                         : static_cast<S *>(p.kv_cache) + k.slot + (int64_t)g * kPageSlots * 2 * p.dim + (is_v ? p.dim : 0);
    }
}

// The 16-byte kernels' threads: every row starts on 16 bytes, a thread takes
// the same columns of kHeads neighbouring heads of a token (all q, all k or
// all v), so that the token's cos | sin values are read once for them and that
// many loads are in flight.  q_per, kv_per: heads of a group (kHeads, or dealt
// evenly); kg: k's groups.
template <class S>
struct RopeHeads {
    const S *src;
    S *dst;
    int64_t src_step, dst_step;
    int h0, n;
    bool is_q, is_v;
    __device__ __forceinline__ RopeHeads(const RopeParams &p, int64_t t, int grp, int q_per, int kv_per, int kg)
    {
        int count = p.q_heads, per = q_per;
        is_q = grp < p.q_groups;
        is_v = false;
        h0 = grp * per;
        src = static_cast<const S *>(p.q) + t * p.q_ts;
        dst = static_cast<S *>(p.out) + t * p.o_ts;
        src_step = p.q_hs;
        dst_step = p.o_hs;
        if (!is_q) {
            is_v = grp >= p.q_groups + kg;
            per = kv_per;
            h0 = (grp - p.q_groups - (is_v ? kg : 0)) * per;
            count = p.nkv;
            src = is_v ? static_cast<const S *>(p.v) + t * p.v_ts : static_cast<const S *>(p.k) + t * p.k_ts;
            src_step = is_v ? p.v_hs : p.k_hs;
            dst_step = (int64_t)kPageSlots * 2 * p.dim;
        }
        src += h0 * src_step;
        n = min(per, count - h0);
    }
    // Where the heads are written, once the token's indices are known; false: nowhere
    __device__ __forceinline__ bool place(const RopeParams &p, const RopeToken &tok)
    {
        if (!tok.row) return false;
        if (!is_q) {
            if (tok.slot < 0) return false;
            dst = static_cast<S *>(p.kv_cache) + tok.slot + (is_v ? p.dim : 0);
        }
        dst += h0 * dst_step;
        return true;
    }
    // Of q heads that have no place (no row): zeros, 16 bytes from column c on
    __device__ __forceinline__ void clear(const RopeParams &p, int c)
    {
        if (p.zero && is_q)
#pragma unroll 1
            for (int i = 0; i < n; ++i) *reinterpret_cast<uint4 *>(dst + (h0 + i) * dst_step + c) = make_uint4(0u, 0u, 0u, 0u);
    }
};

template <class E>
union RopeChunk {
    static constexpr int vec = 16 / sizeof(typename E::store);
    uint4 v;
    typename E::store e[vec];
};

// A unit is one 16-byte chunk of a head (interleaved pairs), or chunk u of the
// first half of its rotated columns with its partner in the second (half
// pairs; the chunks behind the rotated columns are units of their own).  Four
// CTAs per SM (64 registers): 4096 tokens of 12 heads of 128 5.5 us, and 6.8 with
// the 72 registers that the compiler would take and three; a single wave of
// CTAs pays for it (512 tokens of 72 heads of 64: 3.9 us, and 3.4).
template <class E, bool kHalf, int kHeads>
__global__ void __launch_bounds__(256, 4) rope_vec_kernel(const __grid_constant__ RopeParams p)
{
    using S = typename E::store;
    using Chunk = RopeChunk<E>;
    constexpr int vec = Chunk::vec, pairs = kHalf ? vec : vec / 2;   // rotation pairs of a unit
    if (threadIdx.x == 0) griddep_launch_dependents();
    griddep_wait();
    const uint32_t lin = blockIdx.x * 256 + threadIdx.x;
    const uint32_t rest = div_by(lin, p.unit_m, p.unit_s), u = lin - rest * p.units;
    const uint32_t tl = div_by(rest, p.group_m, p.group_s), grp = rest - tl * p.groups;
    const int64_t t = (int64_t)blockIdx.y * p.tokens + tl;
    if ((int)tl >= p.tokens || t >= p.T) return;
    const int64_t pos = p.positions[t], slot = p.nkv ? p.slots[t] : -1;
    const int half = p.rot >> 1;
    const bool rotated = kHalf ? (int)u < half / vec : (int)u * pairs < half;
    const int c0 = kHalf && !rotated ? half / vec + u : u;   // the unit's first chunk
    RopeHeads<S> hd(p, t, grp, p.q_per, p.kv_per, (p.groups - p.q_groups) >> 1);
    const S *src = hd.src + c0 * vec;
    Chunk x[kHeads], y[kHalf ? kHeads : 1];
#pragma unroll
    for (int i = 0; i < kHeads; ++i)
        if (i < hd.n) {
            x[i].v = *reinterpret_cast<const uint4 *>(src + i * hd.src_step);
            if (kHalf && rotated) y[kHalf ? i : 0].v = *reinterpret_cast<const uint4 *>(src + i * hd.src_step + half);
        }
    const RopeToken tok = rope_token(p, pos, slot, u == 0 && grp == 0);
    if (!hd.place(p, tok)) {
        hd.clear(p, c0 * vec);
        if (kHalf && rotated) hd.clear(p, c0 * vec + half);
        return;
    }
    S *dst = hd.dst + c0 * vec;
    if (!rotated || hd.is_v) {
        if (hd.is_q && p.in_place) return;
#pragma unroll
        for (int i = 0; i < kHeads; ++i)
            if (i < hd.n) {
                *reinterpret_cast<uint4 *>(dst + i * hd.dst_step) = x[i].v;
                if (kHalf && rotated) *reinterpret_cast<uint4 *>(dst + i * hd.dst_step + half) = y[kHalf ? i : 0].v;
            }
        return;
    }
    float c[pairs], s[pairs];
    const int i0 = u * pairs;
    if (pairs % 4 == 0 && p.rot % 8 == 0) {   // both halves of the row on 16 bytes
#pragma unroll
        for (int i = 0; i + 4 <= pairs; i += 4) {
            *reinterpret_cast<float4 *>(c + i) = *reinterpret_cast<const float4 *>(tok.row + i0 + i);
            *reinterpret_cast<float4 *>(s + i) = *reinterpret_cast<const float4 *>(tok.row + half + i0 + i);
        }
    } else {
#pragma unroll
        for (int i = 0; i < pairs; ++i) {
            const bool in = i0 + i < half;
            c[i] = in ? tok.row[i0 + i] : 1.f;
            s[i] = in ? tok.row[half + i0 + i] : 0.f;
        }
    }
#pragma unroll
    for (int i = 0; i < pairs; ++i) s[i] *= p.sign;
    const int whole = kHalf ? pairs : min(pairs, half - i0);   // the rotated columns may end in a chunk
#pragma unroll
    for (int i = 0; i < kHeads; ++i)
        if (i < hd.n) {
            Chunk &a = x[i], &b = kHalf ? y[kHalf ? i : 0] : x[i];
#pragma unroll
            for (int k = 0; k < pairs; ++k)
                if (kHalf || k < whole) {
                    const int ia = kHalf ? k : 2 * k, ib = kHalf ? k : 2 * k + 1;
                    float ya, yb;
                    rope_pair(E::get(a.e[ia]), E::get(b.e[ib]), c[k], s[k], ya, yb);
                    a.e[ia] = E::put(ya);
                    b.e[ib] = E::put(yb);
                }
            *reinterpret_cast<uint4 *>(dst + i * hd.dst_step) = x[i].v;
            if (kHalf) *reinterpret_cast<uint4 *>(dst + i * hd.dst_step + half) = y[kHalf ? i : 0].v;
        }
}

// Half pairs whose distance is not whole chunks: the CTA's heads (256 / units
// whole groups of 8) go through shared memory.  Global memory moves in 16-byte
// chunks; in between, a warp takes 32 neighbouring pairs of a group's heads, so
// that cos, sin and both columns are neighbouring words for its lanes.  kZero: a
// call with p.zero (11704 x 43 x 128, 82 rotated: 65.8 us, and 62.1 without the
// code for it).
constexpr int kRopeStagedHeads = 8;

template <class E, bool kZero>
__global__ void __launch_bounds__(256) rope_staged_kernel(const __grid_constant__ RopeParams p)
{
    using S = typename E::store;
    constexpr int vec = RopeChunk<E>::vec, kHeads = kRopeStagedHeads;
    __shared__ uint4 stage[256 * kHeads];
    __shared__ const float *table[256];   // a group's cos | sin row (null: nothing to turn)
    if (threadIdx.x == 0) griddep_launch_dependents();
    griddep_wait();
    const int per = 256 / p.units;
    const int r = div_by(threadIdx.x, p.unit_m, p.unit_s), u = threadIdx.x - r * p.units;
    const uint32_t rest = blockIdx.x * per + r;
    const uint32_t tl = div_by(rest, p.group_m, p.group_s), grp = rest - tl * p.groups;
    const int64_t t = (int64_t)blockIdx.y * p.tokens + tl;
    const bool mine = r < per && (int)tl < p.tokens && t < p.T;
    const int64_t pos = mine ? p.positions[t] : -1, slot = mine && p.nkv ? p.slots[t] : -1;
    RopeHeads<S> hd(p, mine ? t : 0, mine ? grp : 0, kHeads, kHeads, (p.nkv + kHeads - 1) / kHeads);
    uint4 *rows = stage + r * kHeads * p.units + u;   // the group's heads, p.units chunks each
    if (mine) {
        uint4 x[kHeads];
#pragma unroll
        for (int i = 0; i < kHeads; ++i)
            if (i < hd.n) x[i] = *reinterpret_cast<const uint4 *>(hd.src + i * hd.src_step + u * vec);
#pragma unroll
        for (int i = 0; i < kHeads; ++i)
            if (i < hd.n) rows[i * p.units] = x[i];
    }
    bool put = false;
    if (mine) {
        const RopeToken tok = rope_token(p, pos, slot, u == 0 && grp == 0);
        put = hd.place(p, tok);
        if (!put && kZero) hd.clear(p, u * vec);
        if (u == 0) table[r] = put && !hd.is_v ? tok.row : nullptr;
    } else if (r < per && u == 0) {
        table[r] = nullptr;
    }
    __syncthreads();
    const int half = p.rot >> 1, blocks = (half + 31) / 32;
    for (int w = threadIdx.x >> 5; w < per * blocks; w += 8) {
        const int g = w / blocks, i = (w - g * blocks) * 32 + (threadIdx.x & 31);
        const float *row = table[g];
        if (!row || i >= half) continue;
        const float c = row[i], s = p.sign * row[half + i];
        S *e = reinterpret_cast<S *>(stage + g * kHeads * p.units) + i;   // heads past the group's last: unread
#pragma unroll
        for (int k = 0; k < kHeads; ++k) {
            S *a = e + k * p.dim;
            float ya, yb;
            rope_pair(E::get(a[0]), E::get(a[half]), c, s, ya, yb);
            a[0] = E::put(ya);
            a[half] = E::put(yb);
        }
    }
    __syncthreads();
    if (!put || (hd.is_q && p.in_place && u * vec >= p.rot)) return;
#pragma unroll
    for (int i = 0; i < kHeads; ++i)
        if (i < hd.n) *reinterpret_cast<uint4 *>(hd.dst + i * hd.dst_step + u * vec) = rows[i * p.units];
}

// Element kernel, for rows off the 16-byte grid: lanes over a head's pairs and
// copied columns, warps over the token's heads.
template <class E>
__global__ void __launch_bounds__(256) rope_element_kernel(const __grid_constant__ RopeParams p, int half_layout)
{
    using S = typename E::store;
    if (threadIdx.x == 0) griddep_launch_dependents();
    griddep_wait();
    const int half = p.rot >> 1, tail = p.dim - p.rot, heads = p.q_heads + 2 * p.nkv;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        const RopeToken tok = rope_token(p, p.positions[t], p.nkv ? p.slots[t] : -1, threadIdx.x == 0);
        if (!tok.row) {
            for (int h = warp; p.zero && h < p.q_heads; h += 8)
                for (int i = lane; i < p.dim; i += 32) (static_cast<S *>(p.out) + t * p.o_ts + h * p.o_hs)[i] = S(0);
            continue;
        }
        for (int h = warp; h < heads; h += 8) {
            const S *src;
            S *dst;
            rope_head<S>(p, t, h, tok, src, dst);
            if (!dst) continue;
            const bool copy_all = h >= p.q_heads + p.nkv;
            if (!copy_all)
                for (int i = lane; i < half; i += 32) {
                    const int ca = half_layout ? i : 2 * i, cb = half_layout ? i + half : 2 * i + 1;
                    float ya, yb;
                    rope_pair(E::get(src[ca]), E::get(src[cb]), tok.row[i], p.sign * tok.row[half + i], ya, yb);
                    dst[ca] = E::put(ya);
                    dst[cb] = E::put(yb);
                }
            if (copy_all)
                for (int i = lane; i < p.dim; i += 32) dst[i] = src[i];
            else if (tail && !(h < p.q_heads && p.in_place))
                for (int i = lane; i < tail; i += 32) dst[p.rot + i] = src[p.rot + i];
        }
    }
}

const char *check_rope_args(const void *x, int64_t x_ts, int64_t x_hs, const int64_t *positions,
                            const float *cos_sin, int64_t cos_sin_rows, void *out, int64_t o_ts, int64_t o_hs,
                            int T, int heads, int head_dim, int rot_dim, int layout, int inverse, int dtype,
                            int *code)
{
    dtype = dtype_of(dtype);
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

// The grid of a 16-byte kernel: `units` columns' threads a head group, groups
// of `heads` heads, `whole` head groups a CTA (0: threads dealt without gaps)
dim3 rope_grid(RopeParams &prm, int units, int heads, int whole)
{
    prm.units = units;
    prm.q_groups = (prm.q_heads + heads - 1) / heads;
    const int kv_groups = (prm.nkv + heads - 1) / heads;
    prm.groups = prm.q_groups + 2 * kv_groups;
    // the vector kernel's, dealt evenly: 25 heads as 7, 7, 7, 4 rather than 8, 8,
    // 8, 1 (4096 tokens of 9 heads of 128: 4.3 us, and 6.1 as 8 and 1)
    prm.q_per = prm.q_groups ? (prm.q_heads + prm.q_groups - 1) / prm.q_groups : 0;
    prm.kv_per = kv_groups ? (prm.nkv + kv_groups - 1) / kv_groups : 0;
    fast_div(prm.units, &prm.unit_m, &prm.unit_s);
    fast_div(prm.groups, &prm.group_m, &prm.group_s);
    const int64_t most = (int64_t(1) << 30) / ((int64_t)units * prm.groups);   // a grid row's tokens
    prm.tokens = (int)(prm.T < most ? prm.T : most);
    const int64_t work = (int64_t)prm.tokens * prm.groups;
    const int64_t ctas = whole ? (work + whole - 1) / whole : (work * units + 255) / 256;
    return dim3((unsigned)ctas, (unsigned)((prm.T + prm.tokens - 1) / prm.tokens));
}

template <class E, bool kHalf, int kHeads>
int launch_rope_vec(RopeParams &prm, void *stream)
{
    const int units = (kHalf ? prm.dim - prm.rot / 2 : prm.dim) / RopeChunk<E>::vec;
    const dim3 grid = rope_grid(prm, units, kHeads, 0);
    return launch_pdl(rope_vec_kernel<E, kHalf, kHeads>, grid, dim3(256), 0, stream, prm);
}

// Rows that all start on 16 bytes take a 16-byte kernel: whole chunks where
// the half layout's partner of a chunk is a chunk (16384 x 32 x 128 bf16:
// 41.4 us, the copy peak), otherwise through shared memory (11704 x 43 x 128,
// 82 of them rotated: 62.2 us, and 106.8 us in the element kernel).  Several
// heads a thread where there are several (with one head of 256 a token and
// 100000 tokens 60.5 us, against 30.9 with one or two).  Rows off the 16-byte
// grid go element by element.
template <class E>
int launch_rope(RopeParams &prm, bool half_layout, int sms, void *stream)
{
    constexpr int vec = RopeChunk<E>::vec;
    const auto whole = [&](const void *ptr, int64_t ts, int64_t hs, int heads) {
        return heads == 0 || (aligned(ptr, 16) && (prm.T == 1 || ts % vec == 0) && (heads == 1 || hs % vec == 0));
    };
    if (prm.dim % vec == 0 && whole(prm.q, prm.q_ts, prm.q_hs, prm.q_heads) &&
        whole(prm.out, prm.o_ts, prm.o_hs, prm.q_heads) && whole(prm.k, prm.k_ts, prm.k_hs, prm.nkv) &&
        whole(prm.v, prm.v_ts, prm.v_hs, prm.nkv)) {
        if (half_layout && prm.rot / 2 % vec) {
            const int units = prm.dim / vec, per = 256 / units;
            const dim3 grid = rope_grid(prm, units, kRopeStagedHeads, per);
            return launch_pdl(prm.zero ? rope_staged_kernel<E, true> : rope_staged_kernel<E, false>, grid, dim3(256), 0, stream, prm);
        }
        const bool few = (prm.q_heads > prm.nkv ? prm.q_heads : prm.nkv) <= 2;
        if (half_layout) return few ? launch_rope_vec<E, true, 1>(prm, stream) : launch_rope_vec<E, true, 4>(prm, stream);
        return few ? launch_rope_vec<E, false, 2>(prm, stream) : launch_rope_vec<E, false, 8>(prm, stream);
    }
    const int64_t most = (int64_t)sms * 8;
    return launch_pdl(rope_element_kernel<E>, dim3((unsigned)(prm.T < most ? prm.T : most)), dim3(256), 0, stream, prm,
                      (int)half_layout);
}

// A packed call's arguments, one 64-bit word each
struct Words {
    const int64_t *a;
    bool ok;   // every int so far fits one
    explicit Words(const int64_t *words) : a(words), ok(true) {}
    int i(int k)
    {
        ok &= a[k] == (int64_t)(int)a[k];
        return (int)a[k];
    }
    double d(int k) const
    {
        double v;
        memcpy(&v, a + k, 8);
        return v;
    }
    template <class T>
    T *p(int k) const { return reinterpret_cast<T *>((uintptr_t)a[k]); }
};

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
    const int per = 256 / prm.half;
    const int64_t want = (rows + per - 1) / per, most = (int64_t)d->sms * 8;
    return qkvf::launch_pdl(qkvf::rope_table_kernel, dim3((unsigned)(want < most ? want : most)), dim3(256), 0,
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
    prm.q = x;
    prm.out = out;
    prm.positions = positions;
    prm.cos_sin = cos_sin;
    prm.cos_rows = cos_sin_rows;
    prm.q_ts = x_token_stride;
    prm.q_hs = x_head_stride;
    prm.o_ts = out_token_stride;
    prm.o_hs = out_head_stride;
    prm.T = T;
    prm.q_heads = heads;
    prm.dim = head_dim;
    prm.rot = rot_dim;
    prm.in_place = x == out;
    prm.zero = qkvf::zero_skipped(dtype);
    dtype = qkvf::dtype_of(dtype);
    prm.sign = inverse ? -1.f : 1.f;
    const bool half = layout == QKVF_ROPE_HALF;
    return dtype == QKVF_DTYPE_BF16   ? qkvf::launch_rope<qkvf::Bf16>(prm, half, d->sms, stream)
           : dtype == QKVF_DTYPE_FP16 ? qkvf::launch_rope<qkvf::Fp16>(prm, half, d->sms, stream)
                                      : qkvf::launch_rope<qkvf::Fp32>(prm, half, d->sms, stream);
}

int rope_table_packed(const int64_t *args, void *stream)
{
    if (!args) return QKVF_ERR_NULL;
    qkvf::Words w(args);
    const int rot_dim = w.i(3), scaling = w.i(5);
    if (!w.ok) return QKVF_ERR_SIZES;
    return rope_table(w.p<float>(0), args[1], args[2], rot_dim, w.d(4), scaling, w.d(6), args[7], w.d(8), w.d(9),
                      w.d(10), stream);
}

int rope_packed(const int64_t *args, void *stream)
{
    if (!args) return QKVF_ERR_NULL;
    qkvf::Words w(args);
    const int T = w.i(9), heads = w.i(10), dim = w.i(11), rot = w.i(12), layout = w.i(13), inverse = w.i(14), dtype = w.i(15);
    if (!w.ok) return QKVF_ERR_SIZES;
    return rope(w.p<void>(0), args[1], args[2], w.p<int64_t>(3), w.p<float>(4), args[5], w.p<void>(6), args[7], args[8],
                T, heads, dim, rot, layout, inverse, dtype, stream);
}

}  // extern "C"
