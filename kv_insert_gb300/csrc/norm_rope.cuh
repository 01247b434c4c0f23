// norm_rope, norm_rope_backward, norm_rope_kv_append: the RMS norm of every
// head with a weight, and its rotation, in one pass (included by qkv_front.cu
// after rope_kv_append.cuh: one translation unit).
//
// A head's row x of D columns, r = (mean x^2 + eps)^(-1/2), and R(p) the turn
// of its first rot columns by the token's position (rope.cuh):
//   y = R(p) (w * x r).
// Its gradients, with g' = R(-p) g, u = w * g' and mean over the D columns:
//   dx = r u - x r^3 mean(u * x),   dw = sum over tokens and heads of g' * x r,
// the second term as (x r) (r (r mean(u * x))): r^3 by itself leaves FP32 for
// rows of 1e13 and more, or of 1e-13 and less with a small eps, dx does not.
// r is formed again from x, which dx and dw need anyway: nothing is kept
// between the two directions.
//
// A group of P lanes takes a head, a unit of two 16-byte chunks a lane (two
// units for the widest), with the chunks' weights in registers; the sums over a
// head are shuffles within the group.  A unit's chunks are neighbours, or in the
// half layout a chunk and its partner, so no column crosses lanes; half pairs
// whose distance is no whole chunk go through shared memory.  Rows off the
// 16-byte grid take a warp per head element by element.

namespace qkvf {

struct NormParams {
    RopeParams r;             // heads, strides, positions, table, cache
    const void *qw, *kw;      // weights of q (x) and k heads, or null
    int qw_fp32, kw_fp32;     // their type: fp32, otherwise the heads'
    float eps;
    int lanes, lane_m;        // P, and 2^16 / P rounded up
    int warp_groups;          // groups of a warp (lanes behind the last one idle)
    // the gradient: r.q is the output's gradient, r.out x's gradient
    const void *x;
    int64_t x_ts, x_hs;
    float *part;              // [ctas][dim] sums of g' * x r (null: no weight gradient)
};

// Weights of a 16-byte chunk's columns from c on (1 without a weight)
template <class E, int n>
__device__ __forceinline__ void norm_weights(const void *w, int fp32, int c, float (&out)[n])
{
    if (!w) {
#pragma unroll
        for (int i = 0; i < n; ++i) out[i] = 1.f;
    } else if (fp32) {
#pragma unroll
        for (int i = 0; i < n; i += 4) *reinterpret_cast<float4 *>(out + i) = *reinterpret_cast<const float4 *>(static_cast<const float *>(w) + c + i);
    } else {
        RopeChunk<E> v;
        v.v = *reinterpret_cast<const uint4 *>(static_cast<const typename E::store *>(w) + c);
#pragma unroll
        for (int i = 0; i < n; ++i) out[i] = E::get(v.e[i]);
    }
}

template <class E>
__device__ __forceinline__ float norm_weight(const void *w, int fp32, int c)
{
    return !w ? 1.f : fp32 ? static_cast<const float *>(w)[c] : E::get(static_cast<const typename E::store *>(w)[c]);
}

// cos and sin of `pairs` pairs from i0 on (beyond the rotated ones: no turn)
template <int pairs>
__device__ __forceinline__ void norm_angles(const float *row, int rot, int i0, float sign, float (&c)[pairs], float (&s)[pairs])
{
    const int half = rot >> 1;
    if (pairs % 4 == 0 && rot % 8 == 0 && i0 + pairs <= half) {   // both halves of the row on 16 bytes
#pragma unroll
        for (int i = 0; i + 4 <= pairs; i += 4) {
            *reinterpret_cast<float4 *>(c + i) = *reinterpret_cast<const float4 *>(row + i0 + i);
            *reinterpret_cast<float4 *>(s + i) = *reinterpret_cast<const float4 *>(row + half + i0 + i);
        }
    } else {
#pragma unroll
        for (int i = 0; i < pairs; ++i) {
            const bool in = i0 + i < half;
            c[i] = in ? row[i0 + i] : 1.f;
            s[i] = in ? row[half + i0 + i] : 0.f;
        }
    }
#pragma unroll
    for (int i = 0; i < pairs; ++i) s[i] *= sign;
}

// Pairs (2i, 2i + 1); pairs (i, i + rot / 2) whose distance is whole chunks; the
// same at any distance, by way of shared memory
enum NormPairs { kNormInterleaved = 0, kNormHalf = 1, kNormStaged = 2 };

// A lane's unit u of a head: two chunks, at columns a and b (the second may not
// exist), whose pairs are within the unit but for kNormStaged
template <class E, int kPairs>
struct NormUnit {
    static constexpr int vec = RopeChunk<E>::vec;
    int a, b;        // first columns
    int i0, whole;   // first pair, pairs turned
    bool in, two;    // the unit exists; it has a second chunk
    __device__ __forceinline__ NormUnit(const RopeParams &p, int u)
    {
        const int half = p.rot >> 1, h = kPairs == kNormHalf ? half / vec : 0;   // units of two chunks that turn together
        in = u < p.units;
        if (u < h) {
            a = u * vec;
            b = a + half;
        } else {
            a = 2 * (h + (u - h)) * vec;
            b = a + vec;
        }
        two = b < p.dim;
        i0 = u * vec;
        whole = kPairs == kNormHalf ? (u < h ? vec : 0) : max(0, min(vec, half - i0));
    }
};

// A chunk's values, and back: two at a time, as are the sums and products on
// them (one by one the gradients of 8192 x 32 x 128 take 54 us instead of 50)
template <class E, int vec>
__device__ __forceinline__ void norm_unpack(const RopeChunk<E> &x, float (&v)[vec])
{
    if constexpr (vec == 8) {
        const uint32_t w[4] = {x.v.x, x.v.y, x.v.z, x.v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = E::lo(w[i]);
            v[2 * i + 1] = E::hi(w[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < vec; ++i) v[i] = E::get(x.e[i]);
    }
}
template <class E, int vec>
__device__ __forceinline__ uint4 norm_pack(const float (&v)[vec])
{
    if constexpr (vec == 8)
        return make_uint4(E::pack(v[0], v[1]), E::pack(v[2], v[3]), E::pack(v[4], v[5]), E::pack(v[6], v[7]));
    else
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}
__device__ __forceinline__ uint64_t norm_two(const float *v) { return f2_pack(v[0], v[1]); }

// Turn a unit's values in place
template <class E, int kPairs, int vec>
__device__ __forceinline__ void norm_turn(float (&a)[vec], float (&b)[vec], const float *c, const float *s, int whole)
{
    if constexpr (kPairs == kNormHalf) {   // all of its pairs, or none
        if (whole > 0)
#pragma unroll
            for (int k = 0; k < vec; k += 2) {
                const uint64_t x = norm_two(a + k), y = norm_two(b + k), cc = norm_two(c + k);
                f2_unpack(f2_fma(x, cc, f2_mul(y, f2_pack(-s[k], -s[k + 1]))), a[k], a[k + 1]);
                f2_unpack(f2_fma(y, cc, f2_mul(x, norm_two(s + k))), b[k], b[k + 1]);
            }
    } else {
#pragma unroll
        for (int k = 0; k < vec; ++k)
            if (k < whole) {
                if (k < vec / 2)
                    rope_pair(a[2 * k], a[2 * k + 1], c[k], s[k], a[2 * k], a[2 * k + 1]);
                else
                    rope_pair(b[2 * k - vec], b[2 * k + 1 - vec], c[k], s[k], b[2 * k - vec], b[2 * k + 1 - vec]);
            }
    }
}

// kNormStaged: column c of a head whose values are in `row`, turned.  `own` is
// its value, w the partner's weight (times r).
template <class E>
__device__ __forceinline__ float norm_turn_staged(const typename E::store *row, const float *angles, int half, float sign, int c, float own,
                                                  const void *weight, int fp32, float r)
{
    if (c >= 2 * half) return own;
    const bool second = c >= half;
    const int i = second ? c - half : c, q = second ? i : c + half;
    const float other = E::get(row[q]) * r * norm_weight<E>(weight, fp32, q), sn = sign * angles[half + i];
    return fmaf(own, angles[i], second ? other * sn : -(other * sn));
}

// A thread's place: its lane within its group (units: none of it), and the
// group within its CTA.  (div: lane / P, exact below 32)
struct NormPlace {
    int sl, sub;
    __device__ __forceinline__ explicit NormPlace(const NormParams &p)
    {
        const int lane = threadIdx.x & 31, grp = (lane * p.lane_m) >> 16;
        const bool in = grp < p.warp_groups;
        sl = in ? lane - grp * p.lanes : p.r.units;
        sub = (threadIdx.x >> 5) * p.warp_groups + (in ? grp : 0);
    }
};

// The sum over `lanes` neighbouring lanes (a power of two), in each of them
__device__ __forceinline__ float norm_sum(float v, int lanes)
{
    for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The sum over a group, in each of its lanes (the whole warp calls)
__device__ __forceinline__ float norm_group_sum(float v, const NormParams &p, int sl)
{
    if ((p.lanes & (p.lanes - 1)) == 0) return norm_sum(v, p.lanes);
    for (int o = 16; o > 0; o >>= 1) {   // lane 0 of the group gathers it
        if (o >= p.lanes) continue;
        const float y = __shfl_down_sync(0xffffffffu, v, o);
        if (sl + o < p.lanes) v += y;
    }
    return __shfl_sync(0xffffffffu, v, ((threadIdx.x & 31) - sl) & 31);
}

// One group of lanes takes kHeads neighbouring heads of a token: two CTAs an SM
// with four heads a lane have 64 KB on their way at first, and nothing while they
// compute and store (8192 tokens of 32 heads of 128, 134 MB: 28 to 30 us, 4.5 to
// 4.8 TB/s, with 44 % of the issue slots used; in fp32, 268 MB: 43 us, 6.2 TB/s;
// three CTAs with two heads a lane 31 us).
template <class E, int kPairs, int kHeads, int kUnits>
__global__ void __launch_bounds__(256, 2) norm_vec_kernel(const __grid_constant__ NormParams p)
{
    using S = typename E::store;
    using Chunk = RopeChunk<E>;
    using Unit = NormUnit<E, kPairs>;
    constexpr int vec = Chunk::vec;
    __shared__ uint4 stage[kPairs == kNormStaged ? 256 * 2 * kHeads * kUnits : 1];
    if (threadIdx.x == 0) griddep_launch_dependents();
    griddep_wait();
    const RopeParams &r = p.r;
    const NormPlace at(p);
    const int sl = at.sl;
    const uint32_t lin = blockIdx.x * (8 * p.warp_groups) + at.sub;
    const uint32_t tl = div_by(lin, r.group_m, r.group_s), grp = lin - tl * r.groups;
    const int64_t t = (int64_t)blockIdx.y * r.tokens + tl;
    const bool mine = (int)tl < r.tokens && t < r.T;
    const int64_t pos = mine ? r.positions[t] : -1, slot = mine && r.nkv ? r.slots[t] : -1;
    RopeHeads<S> hd(r, mine ? t : 0, mine ? grp : 0, r.q_per, r.kv_per, (r.groups - r.q_groups) >> 1);
    if (!mine) hd.n = 0;
    Chunk x[kUnits][kHeads], y[kUnits][kHeads];
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
        const Unit un(r, sl + k * p.lanes);
#pragma unroll
        for (int i = 0; i < kHeads; ++i) {
            x[k][i].v = y[k][i].v = make_uint4(0u, 0u, 0u, 0u);
            if (un.in && i < hd.n) {
                x[k][i].v = *reinterpret_cast<const uint4 *>(hd.src + i * hd.src_step + un.a);
                if (un.two) y[k][i].v = *reinterpret_cast<const uint4 *>(hd.src + i * hd.src_step + un.b);
            }
        }
    }
    const RopeToken tok = mine ? rope_token(r, pos, slot, sl == 0 && grp == 0) : RopeToken{nullptr, -1};
    const bool put = mine && hd.place(r, tok);
    const void *w = hd.is_q ? p.qw : p.kw;
    const int wf = hd.is_q ? p.qw_fp32 : p.kw_fp32;
    // (on their way beside the chunks; after the sums they cost 2 us of 30 at 8192 x 32 x 128)
    float c[kUnits][vec], s[kUnits][vec], wa[kUnits][vec], wb[kUnits][vec];
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
        const Unit un(r, sl + k * p.lanes);
        if (!un.in || !put || hd.is_v) continue;
        if (kPairs != kNormStaged && un.whole > 0) norm_angles<vec>(tok.row, r.rot, un.i0, 1.f, c[k], s[k]);
        norm_weights<E>(w, wf, un.a, wa[k]);
        norm_weights<E>(un.two ? w : nullptr, wf, un.b, wb[k]);
    }
    float rs[kHeads];
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
        uint64_t sum = 0;
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
            float a[vec], b[vec];
            norm_unpack<E>(x[k][i], a);
            norm_unpack<E>(y[k][i], b);
#pragma unroll
            for (int e = 0; e < vec; e += 2) {
                const uint64_t a2 = norm_two(a + e), b2 = norm_two(b + e);
                sum = f2_fma(b2, b2, f2_fma(a2, a2, sum));
            }
        }
        float s0, s1;
        f2_unpack(sum, s0, s1);
        rs[i] = rsqrtf(fmaf(norm_group_sum(s0 + s1, p, sl), 1.f / (float)r.dim, p.eps));   // every lane of the warp is here
    }
    S *rows = reinterpret_cast<S *>(stage) + (size_t)at.sub * kHeads * r.dim;   // the group's heads
    if (kPairs == kNormStaged) {
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
            const Unit un(r, sl + k * p.lanes);
#pragma unroll
            for (int i = 0; i < kHeads; ++i)
                if (un.in) {
                    *reinterpret_cast<uint4 *>(rows + i * r.dim + un.a) = x[k][i].v;
                    if (un.two) *reinterpret_cast<uint4 *>(rows + i * r.dim + un.b) = y[k][i].v;
                }
        }
        __syncwarp();   // (a group is within a warp)
    }
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
        const Unit un(r, sl + k * p.lanes);
        if (!un.in || !mine) continue;
        if (!put) {
            hd.clear(r, un.a);
            if (un.two) hd.clear(r, un.b);
            continue;
        }
        if (hd.is_v) {
#pragma unroll
            for (int i = 0; i < kHeads; ++i)
                if (i < hd.n) {
                    *reinterpret_cast<uint4 *>(hd.dst + i * hd.dst_step + un.a) = x[k][i].v;
                    if (un.two) *reinterpret_cast<uint4 *>(hd.dst + i * hd.dst_step + un.b) = y[k][i].v;
                }
            continue;
        }
#pragma unroll
        for (int i = 0; i < kHeads; ++i)
            if (i < hd.n) {
                float a[vec], b[vec];
                norm_unpack<E>(x[k][i], a);
                norm_unpack<E>(y[k][i], b);
                const uint64_t r2 = f2_pack(rs[i], rs[i]);
#pragma unroll
                for (int e = 0; e < vec; e += 2) {
                    f2_unpack(f2_mul(f2_mul(norm_two(a + e), r2), norm_two(wa[k] + e)), a[e], a[e + 1]);
                    f2_unpack(f2_mul(f2_mul(norm_two(b + e), r2), norm_two(wb[k] + e)), b[e], b[e + 1]);
                }
                if (kPairs == kNormStaged) {
                    const int half = r.rot >> 1;
#pragma unroll
                    for (int e = 0; e < vec; ++e) {
                        a[e] = norm_turn_staged<E>(rows + i * r.dim, tok.row, half, 1.f, un.a + e, a[e], w, wf, rs[i]);
                        if (un.two) b[e] = norm_turn_staged<E>(rows + i * r.dim, tok.row, half, 1.f, un.b + e, b[e], w, wf, rs[i]);
                    }
                } else {
                    norm_turn<E, kPairs>(a, b, c[k], s[k], un.whole);
                }
                *reinterpret_cast<uint4 *>(hd.dst + i * hd.dst_step + un.a) = norm_pack<E>(a);
                if (un.two) *reinterpret_cast<uint4 *>(hd.dst + i * hd.dst_step + un.b) = norm_pack<E>(b);
            }
    }
}

// Element kernel, for rows off the 16-byte grid: a warp per head
template <class E>
__global__ void __launch_bounds__(256) norm_element_kernel(const __grid_constant__ NormParams p, int half_layout)
{
    using S = typename E::store;
    if (threadIdx.x == 0) griddep_launch_dependents();
    griddep_wait();
    const RopeParams &r = p.r;
    const int half = r.rot >> 1, heads = r.q_heads + 2 * r.nkv;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int64_t t = blockIdx.x; t < r.T; t += gridDim.x) {
        const RopeToken tok = rope_token(r, r.positions[t], r.nkv ? r.slots[t] : -1, threadIdx.x == 0);
        if (!tok.row) {
            for (int h = warp; r.zero && h < r.q_heads; h += 8)
                for (int i = lane; i < r.dim; i += 32) (static_cast<S *>(r.out) + t * r.o_ts + h * r.o_hs)[i] = S(0);
            continue;
        }
        for (int h = warp; h < heads; h += 8) {
            const S *src;
            S *dst;
            rope_head<S>(r, t, h, tok, src, dst);
            if (!dst) continue;
            if (h >= r.q_heads + r.nkv) {
                for (int i = lane; i < r.dim; i += 32) dst[i] = src[i];
                continue;
            }
            const bool is_q = h < r.q_heads;
            const void *w = is_q ? p.qw : p.kw;
            const int wf = is_q ? p.qw_fp32 : p.kw_fp32;
            float ss = 0.f;
            for (int i = lane; i < r.dim; i += 32) {
                const float v = E::get(src[i]);
                ss = fmaf(v, v, ss);
            }
            const float rs = rsqrtf(fmaf(norm_sum(ss, 32), 1.f / (float)r.dim, p.eps));   // (the whole head is read)
            for (int i = lane; i < half; i += 32) {
                const int ca = half_layout ? i : 2 * i, cb = half_layout ? i + half : 2 * i + 1;
                float ya, yb;
                rope_pair(E::get(src[ca]) * rs * norm_weight<E>(w, wf, ca), E::get(src[cb]) * rs * norm_weight<E>(w, wf, cb),
                          tok.row[i], tok.row[half + i], ya, yb);
                dst[ca] = E::put(ya);
                dst[cb] = E::put(yb);
            }
            for (int i = r.rot + lane; i < r.dim; i += 32) dst[i] = E::put(E::get(src[i]) * rs * norm_weight<E>(w, wf, i));
        }
    }
}

// ---- the gradients ----------------------------------------------------------
//
// A lane keeps its unit while its group walks over the heads, so the weight's
// gradient adds up in registers; a CTA joins its groups in shared memory in
// order and leaves one row of sums, and norm_dw_kernel adds the CTAs' rows in
// order: a call repeats bitwise.  The next heads' chunks are on their way to
// shared memory while one is computed (four: 128 KB an SM); two CTAs an SM.
// Bound by neither bytes nor issue (46 % of the slots; 35 % with 25 heads of 80)
// but by each round's chain: the head, then its angles, then two sums by
// shuffles.  8192 tokens of 32 heads of 128 (201 MB): 50 us, 4.0 TB/s, and 3 for
// norm_dw_kernel behind it (5 alone); in fp32 (403 MB) 83 us with it.

constexpr int kNormAhead = 4;

__device__ __forceinline__ void norm_fetch(uint4 *dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

template <class E, int kPairs, int kUnits>
__global__ void __launch_bounds__(256, kUnits == 1 ? 2 : 1) norm_back_vec_kernel(const __grid_constant__ NormParams p)
{
    using S = typename E::store;
    using Chunk = RopeChunk<E>;
    using Unit = NormUnit<E, kPairs>;
    constexpr int vec = Chunk::vec;
    extern __shared__ float norm_dw[];   // [groups of the CTA][dim]; kNormStaged: before that their heads
    if (threadIdx.x == 0) griddep_launch_dependents();
    griddep_wait();
    const RopeParams &r = p.r;
    const NormPlace at(p);
    const int sl = at.sl, sub = at.sub, subs = 8 * p.warp_groups;
    const float inv_dim = 1.f / (float)r.dim;
    float wa[kUnits][vec], wb[kUnits][vec], da[kUnits][vec], db[kUnits][vec];
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
        const Unit un(r, sl + k * p.lanes);
#pragma unroll
        for (int e = 0; e < vec; ++e) wa[k][e] = wb[k][e] = da[k][e] = db[k][e] = 0.f;
        if (un.in) norm_weights<E>(p.qw, p.qw_fp32, un.a, wa[k]);
        if (un.in && un.two) norm_weights<E>(p.qw, p.qw_fp32, un.b, wb[k]);
    }
    const int64_t rows = (int64_t)r.T * r.q_heads, step = (int64_t)gridDim.x * subs;
    // A lane's chunks of the next heads on their way to shared memory: [turn][chunk][thread]
    uint4 *ahead = reinterpret_cast<uint4 *>(norm_dw + (size_t)subs * r.dim) + threadIdx.x;
    // a walk over the group's heads (a 64-bit division a head would cost as much as its sums)
    const int dt = (int)(step / r.q_heads), dh = (int)(step - (int64_t)dt * r.q_heads);
    struct Walk {
        int t, h;
    };
    const auto advance = [&](Walk &w) {
        w.t += dt;
        w.h += dh;
        if (w.h >= r.q_heads) {
            w.h -= r.q_heads;
            ++w.t;
        }
    };
    const int64_t row00 = (int64_t)blockIdx.x * subs + sub;
    Walk now = {(int)(row00 / r.q_heads), (int)(row00 % r.q_heads)}, next = now;
    const auto fetch = [&](int turn) {
        if (next.t < r.T) {
            const S *gp = static_cast<const S *>(r.q) + next.t * r.q_ts + next.h * r.q_hs;
            const S *xp = static_cast<const S *>(p.x) + next.t * p.x_ts + next.h * p.x_hs;
#pragma unroll
            for (int k = 0; k < kUnits; ++k) {
                const Unit un(r, sl + k * p.lanes);
                uint4 *dst = ahead + (turn * kUnits + k) * (4 * 256);
                if (!un.in) continue;
                norm_fetch(dst, gp + un.a);
                norm_fetch(dst + 512, xp + un.a);
                if (un.two) {
                    norm_fetch(dst + 256, gp + un.b);
                    norm_fetch(dst + 768, xp + un.b);
                }
            }
        }
        advance(next);
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll 1
    for (int i = 0; i < kNormAhead; ++i) fetch(i);
    int64_t pos = now.t < r.T ? r.positions[now.t] : -1;
    int turn = 0;
    // (the same number of rounds for every group: shuffles take whole warps)
#pragma unroll 1
    for (int64_t row0 = (int64_t)blockIdx.x * subs; row0 < rows; row0 += step) {
        const bool mine = now.t < r.T;
        struct {
            int64_t pos;
            int t, h;
            Chunk ga[kUnits], gb[kUnits], xa[kUnits], xb[kUnits];
        } cur;
        cur.t = now.t;
        cur.h = now.h;
        cur.pos = pos;
        advance(now);
        if (now.t < r.T) pos = r.positions[now.t];
        asm volatile("cp.async.wait_group %0;" ::"n"(kNormAhead - 1) : "memory");
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
            const Unit un(r, sl + k * p.lanes);
            const uint4 *src = ahead + (turn * kUnits + k) * (4 * 256), none = make_uint4(0u, 0u, 0u, 0u);
            const bool one = mine && un.in, two = one && un.two;
            cur.ga[k].v = one ? src[0] : none;
            cur.gb[k].v = two ? src[256] : none;
            cur.xa[k].v = one ? src[512] : none;
            cur.xb[k].v = two ? src[768] : none;
        }
        fetch(turn);   // into the place just read
        turn = turn == kNormAhead - 1 ? 0 : turn + 1;
        const RopeToken tok = mine ? rope_token(r, cur.pos, -1, sl == 0 && cur.h == 0) : RopeToken{nullptr, -1};
        S *row = reinterpret_cast<S *>(norm_dw) + (size_t)sub * r.dim;
        if (kPairs == kNormStaged) {
            __syncwarp();   // the head before is read
#pragma unroll
            for (int k = 0; k < kUnits; ++k) {
                const Unit un(r, sl + k * p.lanes);
                if (un.in) *reinterpret_cast<uint4 *>(row + un.a) = cur.ga[k].v;
                if (un.in && un.two) *reinterpret_cast<uint4 *>(row + un.b) = cur.gb[k].v;
            }
            __syncwarp();
        }
        float g[kUnits][vec], g2[kUnits][vec];
        uint64_t squares = 0, dots = 0;
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
            const Unit un(r, sl + k * p.lanes);
            if (!un.in || !tok.row) continue;
            norm_unpack<E>(cur.ga[k], g[k]);
            norm_unpack<E>(cur.gb[k], g2[k]);
            if (kPairs == kNormStaged) {
                const int half = r.rot >> 1;
#pragma unroll
                for (int e = 0; e < vec; ++e) {
                    g[k][e] = norm_turn_staged<E>(row, tok.row, half, -1.f, un.a + e, g[k][e], nullptr, 0, 1.f);
                    if (un.two) g2[k][e] = norm_turn_staged<E>(row, tok.row, half, -1.f, un.b + e, g2[k][e], nullptr, 0, 1.f);
                }
            } else if (un.whole > 0) {
                float c[vec], s[vec];
                norm_angles<vec>(tok.row, r.rot, un.i0, -1.f, c, s);
                norm_turn<E, kPairs>(g[k], g2[k], c, s, un.whole);
            }
            float x[vec], x2[vec];
            norm_unpack<E>(cur.xa[k], x);
            norm_unpack<E>(cur.xb[k], x2);
#pragma unroll
            for (int e = 0; e < vec; e += 2) {
                const uint64_t u = norm_two(x + e), v = norm_two(x2 + e);
                squares = f2_fma(v, v, f2_fma(u, u, squares));
                dots = f2_fma(f2_mul(norm_two(g2[k] + e), norm_two(wb[k] + e)), v,
                              f2_fma(f2_mul(norm_two(g[k] + e), norm_two(wa[k] + e)), u, dots));
            }
        }
        float ss, dot, odd;
        f2_unpack(squares, ss, odd);
        ss = norm_group_sum(ss + odd, p, sl);
        f2_unpack(dots, dot, odd);
        dot = norm_group_sum(dot + odd, p, sl);
        const float rs = rsqrtf(fmaf(ss, inv_dim, p.eps)), back = rs * (rs * dot * inv_dim);
        S *dst = static_cast<S *>(r.out) + cur.t * r.o_ts + cur.h * r.o_hs;
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
            const Unit un(r, sl + k * p.lanes);
            if (!un.in || !mine) continue;
            if (!tok.row) {
                if (r.zero) {
                    *reinterpret_cast<uint4 *>(dst + un.a) = make_uint4(0u, 0u, 0u, 0u);
                    if (un.two) *reinterpret_cast<uint4 *>(dst + un.b) = make_uint4(0u, 0u, 0u, 0u);
                }
                continue;
            }
            float x[vec], y[vec];
            const uint64_t r2 = f2_pack(rs, rs), back2 = f2_pack(-back, -back);
            const auto half = [&](const Chunk &xs, const float (&gs)[vec], const float (&ws)[vec], float (&ds)[vec]) {
                norm_unpack<E>(xs, x);
#pragma unroll
                for (int e = 0; e < vec; e += 2) {
                    const uint64_t n2 = f2_mul(norm_two(x + e), r2), gg = norm_two(gs + e);
                    f2_unpack(f2_fma(gg, n2, norm_two(ds + e)), ds[e], ds[e + 1]);
                    f2_unpack(f2_fma(n2, back2, f2_mul(r2, f2_mul(gg, norm_two(ws + e)))), y[e], y[e + 1]);
                }
            };
            half(cur.xa[k], g[k], wa[k], da[k]);
            *reinterpret_cast<uint4 *>(dst + un.a) = norm_pack<E>(y);
            if (un.two) {
                half(cur.xb[k], g2[k], wb[k], db[k]);
                *reinterpret_cast<uint4 *>(dst + un.b) = norm_pack<E>(y);
            }
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (!p.part) return;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
        const Unit un(r, sl + k * p.lanes);
        if (!un.in) continue;
#pragma unroll
        for (int e = 0; e < vec; ++e) {
            norm_dw[sub * r.dim + un.a + e] = da[k][e];
            if (un.two) norm_dw[sub * r.dim + un.b + e] = db[k][e];
        }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < r.dim; c += 256) {
        float v = 0.f;
        for (int i = 0; i < subs; ++i) v += norm_dw[i * r.dim + c];
        p.part[(int64_t)blockIdx.x * r.dim + c] = v;
    }
}

template <class E>
__global__ void __launch_bounds__(256) norm_back_element_kernel(const __grid_constant__ NormParams p, int half_layout)
{
    using S = typename E::store;
    extern __shared__ float norm_dw[];   // [8 warps][dim], a lane's columns its own
    if (threadIdx.x == 0) griddep_launch_dependents();
    griddep_wait();
    const RopeParams &r = p.r;
    const int half = r.rot >> 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float *dw = norm_dw + warp * r.dim;
    for (int i = lane; i < r.dim; i += 32) dw[i] = 0.f;
    __syncwarp();
    const int64_t rows = (int64_t)r.T * r.q_heads, step = (int64_t)gridDim.x * 8;
    const int dt = (int)(step / r.q_heads), dh = (int)(step - (int64_t)dt * r.q_heads);
    int64_t t = ((int64_t)blockIdx.x * 8 + warp) / r.q_heads;
    int h = (int)(((int64_t)blockIdx.x * 8 + warp) % r.q_heads);
    for (int64_t row = (int64_t)blockIdx.x * 8 + warp; row < rows; row += step, t += dt + (h + dh >= r.q_heads),
                 h += dh - (h + dh >= r.q_heads ? r.q_heads : 0)) {
        const S *gp = static_cast<const S *>(r.q) + t * r.q_ts + h * r.q_hs;
        const S *xp = static_cast<const S *>(p.x) + t * p.x_ts + h * p.x_hs;
        S *dst = static_cast<S *>(r.out) + t * r.o_ts + h * r.o_hs;
        const RopeToken tok = rope_token(r, r.positions[t], -1, lane == 0 && h == 0);
        if (!tok.row) {
            for (int i = lane; r.zero && i < r.dim; i += 32) dst[i] = S(0);
            continue;
        }
        // pair i of a lane, g turned back; or the column behind the rotated ones
        const auto each = [&](auto use) {
            for (int i = lane; i < half; i += 32) {
                const int ca = half_layout ? i : 2 * i, cb = half_layout ? i + half : 2 * i + 1;
                float a, b;
                rope_pair(E::get(gp[ca]), E::get(gp[cb]), tok.row[i], -tok.row[half + i], a, b);
                use(ca, a, cb, b);
            }
            for (int i = r.rot + lane; i < r.dim; i += 32) use(i, E::get(gp[i]), -1, 0.f);
        };
        float ss = 0.f, dot = 0.f;
        const auto add = [&](int c, float g) {
            const float x = E::get(xp[c]);
            ss = fmaf(x, x, ss);
            dot = fmaf(g * norm_weight<E>(p.qw, p.qw_fp32, c), x, dot);
        };
        each([&](int ca, float a, int cb, float b) {
            add(ca, a);
            if (cb >= 0) add(cb, b);
        });
        ss = norm_sum(ss, 32);
        dot = norm_sum(dot, 32);   // (the whole row is read before any of it is written)
        const float inv_dim = 1.f / (float)r.dim;
        const float rs = rsqrtf(fmaf(ss, inv_dim, p.eps)), back = rs * (rs * dot * inv_dim);
        const auto put = [&](int c, float g) {
            const float n = E::get(xp[c]) * rs;
            dw[c] = fmaf(g, n, dw[c]);
            dst[c] = E::put(fmaf(-n, back, rs * (g * norm_weight<E>(p.qw, p.qw_fp32, c))));
        };
        each([&](int ca, float a, int cb, float b) {
            put(ca, a);
            if (cb >= 0) put(cb, b);
        });
    }
    if (!p.part) return;
    __syncthreads();
    for (int c = threadIdx.x; c < r.dim; c += 256) {
        float v = 0.f;
        for (int i = 0; i < 8; ++i) v += norm_dw[i * r.dim + c];
        p.part[(int64_t)blockIdx.x * r.dim + c] = v;
    }
}

// The weight's gradient from the CTAs' rows: 32 warps take every 32nd row of 32
// columns, joined in order
__global__ void __launch_bounds__(1024) norm_dw_kernel(const float *part, int rows, int dim, void *out, int dtype)
{
    __shared__ float sums[32][32];
    if (threadIdx.x == 0) griddep_launch_dependents();
    griddep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = blockIdx.x * 32 + lane;
    float v = 0.f;
    if (c < dim)
#pragma unroll 4
        for (int i = warp; i < rows; i += 32) v += part[(int64_t)i * dim + c];
    sums[warp][lane] = v;
    __syncthreads();
    if (warp > 0 || c >= dim) return;
    v = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += sums[i][lane];
    if (dtype == QKVF_DTYPE_FP32)
        static_cast<float *>(out)[c] = v;
    else
        static_cast<uint16_t *>(out)[c] = dtype == QKVF_DTYPE_BF16 ? Bf16::put(v) : Fp16::put(v);
}

// ---- host -------------------------------------------------------------------

template <class E, int kPairs>
bool prepare_norm_kernel()
{
    constexpr auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
    constexpr int smem = 16384 + kNormAhead * 4 * 256 * 16;
    return cudaFuncSetAttribute((const void *)norm_back_vec_kernel<E, kPairs, 1>, attr, smem) == cudaSuccess &&
           cudaFuncSetAttribute((const void *)norm_back_vec_kernel<E, kPairs, 2>, attr, smem + kNormAhead * 4 * 256 * 16) == cudaSuccess;
}

template <class E>
bool prepare_norm_kernel()
{
    return prepare_norm_kernel<E, kNormInterleaved>() && prepare_norm_kernel<E, kNormHalf>() && prepare_norm_kernel<E, kNormStaged>();
}

bool prepare_norm_kernels() { return prepare_norm_kernel<Bf16>() && prepare_norm_kernel<Fp16>() && prepare_norm_kernel<Fp32>(); }

constexpr int kNormBackCtas = 2;   // per SM

int64_t norm_back_ctas(int64_t rows, int sms)
{
    const int64_t most = (int64_t)sms * kNormBackCtas, want = (rows + 7) / 8;
    return want < most ? want : most;
}

// The lanes of a head for its units: a power of two, at most 32, or as many as
// units where a warp holds more heads so (5 units: six heads instead of four;
// the sum over a head is one shuffle longer then).  That many lanes against a
// power of two, us in graphs, 16.4 MB of 25 heads, bf16, forward | backward:
//   3 units (48)  11.0 12.6 | 22.4 22.4      9 (144)  12.6 15.1 | 23.4 27.1
//   5 (80)        11.1 12.9 | 22.6 25.6     10 (160)  10.9 12.7 | 22.4 25.2
//   6 (96)        10.8 12.6 | 22.1 23.2
int norm_lanes(NormParams &prm, int units)
{
    int lanes = 1;
    while (lanes < units && lanes < 32) lanes *= 2;
    if (units < 32 && 32 / units > 32 / lanes) lanes = units;
    prm.r.units = units;
    prm.lanes = lanes;
    prm.lane_m = (65536 + lanes - 1) / lanes;
    prm.warp_groups = 32 / lanes;
    return (units + lanes - 1) / lanes;   // units of a lane
}

// Whether the 16-byte kernels take rows
template <class E>
bool norm_whole(const NormParams &prm)
{
    constexpr int vec = RopeChunk<E>::vec;
    const RopeParams &r = prm.r;
    const auto whole = [&](const void *ptr, int64_t ts, int64_t hs, int heads) {
        return heads == 0 || !ptr || (aligned(ptr, 16) && (r.T == 1 || ts % vec == 0) && (heads == 1 || hs % vec == 0));
    };
    return r.dim % vec == 0 && whole(r.q, r.q_ts, r.q_hs, r.q_heads) && whole(r.out, r.o_ts, r.o_hs, r.q_heads) &&
           whole(r.k, r.k_ts, r.k_hs, r.nkv) && whole(r.v, r.v_ts, r.v_hs, r.nkv) && whole(prm.x, prm.x_ts, prm.x_hs, r.q_heads) &&
           aligned(prm.qw, 16) && aligned(prm.kw, 16);
}

// How pairs lie, and the units of a head (two chunks each)
template <class E>
int norm_pairs(const NormParams &prm, bool half_layout, int *units)
{
    constexpr int vec = RopeChunk<E>::vec;
    const int chunks = prm.r.dim / vec, h = half_layout && prm.r.rot / 2 % vec == 0 ? prm.r.rot / 2 / vec : 0;
    *units = h + (chunks - 2 * h + 1) / 2;
    return !half_layout ? kNormInterleaved : h ? kNormHalf : kNormStaged;
}

template <class E, int kPairs, int kHeads, int kUnits>
int launch_norm_vec(NormParams &prm, void *stream)
{
    RopeParams &r = prm.r;
    r.q_groups = (r.q_heads + kHeads - 1) / kHeads;
    const int kv_groups = (r.nkv + kHeads - 1) / kHeads;
    r.groups = r.q_groups + 2 * kv_groups;
    r.q_per = r.q_groups ? (r.q_heads + r.q_groups - 1) / r.q_groups : 0;
    r.kv_per = kv_groups ? (r.nkv + kv_groups - 1) / kv_groups : 0;
    fast_div(r.groups, &r.group_m, &r.group_s);
    const int64_t most = (int64_t(1) << 30) / r.groups / prm.lanes;   // a grid row's tokens: its threads below 2^30
    r.tokens = (int)(r.T < most ? r.T : most);
    const int64_t rows = (int64_t)r.tokens * r.groups, per = 8 * prm.warp_groups;   // groups of a grid row, of a CTA
    const dim3 grid((unsigned)((rows + per - 1) / per), (unsigned)((r.T + r.tokens - 1) / r.tokens));
    return launch_pdl(norm_vec_kernel<E, kPairs, kHeads, kUnits>, grid, dim3(256), 0, stream, prm);
}

template <class E, int kPairs>
int launch_norm_pairs(NormParams &prm, int units, void *stream)
{
    return norm_lanes(prm, units) == 1 ? launch_norm_vec<E, kPairs, 4, 1>(prm, stream) : launch_norm_vec<E, kPairs, 2, 2>(prm, stream);
}

template <class E>
int launch_norm(NormParams &prm, bool half_layout, int sms, void *stream)
{
    if (norm_whole<E>(prm)) {
        int units;
        const int pairs = norm_pairs<E>(prm, half_layout, &units);
        return pairs == kNormInterleaved ? launch_norm_pairs<E, kNormInterleaved>(prm, units, stream)
               : pairs == kNormHalf      ? launch_norm_pairs<E, kNormHalf>(prm, units, stream)
                                         : launch_norm_pairs<E, kNormStaged>(prm, units, stream);
    }
    const int64_t most = (int64_t)sms * 8;
    return launch_pdl(norm_element_kernel<E>, dim3((unsigned)(prm.r.T < most ? prm.r.T : most)), dim3(256), 0, stream, prm,
                      (int)half_layout);
}

template <class E, int kPairs>
int launch_norm_back_pairs(NormParams &prm, int units, int64_t ctas, void *stream)
{
    const int per = norm_lanes(prm, units);
    const size_t smem = (size_t)(8 * prm.warp_groups) * prm.r.dim * 4 + (size_t)kNormAhead * per * 4 * 256 * 16;   // 16 KB at most, and 64 a unit
    return launch_pdl(per == 1 ? norm_back_vec_kernel<E, kPairs, 1> : norm_back_vec_kernel<E, kPairs, 2>, dim3((unsigned)ctas),
                      dim3(256), smem, stream, prm);
}

template <class E>
int launch_norm_back(NormParams &prm, bool half_layout, int sms, void *grad_weight, int grad_weight_dtype, void *stream)
{
    const int64_t ctas = norm_back_ctas((int64_t)prm.r.T * prm.r.q_heads, sms);
    int rc;
    if (norm_whole<E>(prm)) {
        int units;
        const int pairs = norm_pairs<E>(prm, half_layout, &units);
        rc = pairs == kNormInterleaved ? launch_norm_back_pairs<E, kNormInterleaved>(prm, units, ctas, stream)
             : pairs == kNormHalf      ? launch_norm_back_pairs<E, kNormHalf>(prm, units, ctas, stream)
                                       : launch_norm_back_pairs<E, kNormStaged>(prm, units, ctas, stream);
    } else {
        rc = launch_pdl(norm_back_element_kernel<E>, dim3((unsigned)ctas), dim3(256), (size_t)8 * prm.r.dim * 4, stream, prm,
                        (int)half_layout);
    }
    if (rc != QKVF_OK || !grad_weight) return rc;
    return launch_pdl(norm_dw_kernel, dim3((unsigned)((prm.r.dim + 31) / 32)), dim3(1024), 0, stream,
                      (const float *)prm.part, (int)ctas, prm.r.dim, grad_weight, grad_weight_dtype);
}

// A weight: of the heads' type or fp32, over nothing that the call writes
const char *check_norm_weight(const void *w, int weight_dtype, int dtype, int head_dim, const void *out, size_t out_bytes, int *code)
{
    *code = QKVF_ERR_LAYOUT;
    if (weight_dtype != dtype_of(dtype) && weight_dtype != QKVF_DTYPE_FP32) return "a weight must be of the heads' type or fp32";
    *code = QKVF_ERR_ALIGN;
    if (!aligned(w, dtype_bytes(weight_dtype))) return "a weight must be aligned to its elements";
    *code = QKVF_ERR_ARG;
    if (w && out && overlap(w, (size_t)head_dim * dtype_bytes(weight_dtype), out, out_bytes)) return "a weight overlaps an output";
    *code = QKVF_OK;
    return nullptr;
}

bool norm_eps_ok(float eps) { return eps >= 0.f && eps <= 1.f; }

const char *check_norm_args(const void *x, int64_t x_ts, int64_t x_hs, const void *weight, int weight_dtype,
                            const int64_t *positions, const float *cos_sin, int64_t cos_sin_rows, void *out,
                            int64_t o_ts, int64_t o_hs, int T, int heads, int head_dim, int rot_dim, int layout,
                            float eps, int dtype, int *code)
{
    if (const char *why = check_rope_args(x, x_ts, x_hs, positions, cos_sin, cos_sin_rows, out, o_ts, o_hs, T, heads,
                                          head_dim, rot_dim, layout, 0, dtype, code))
        return why;
    *code = QKVF_ERR_ARG;
    if (!norm_eps_ok(eps)) return "eps must be in [0, 1]";
    const size_t out_b = T > 0 ? view_of(out, T, o_ts, heads, o_hs, head_dim, dtype_bytes(dtype_of(dtype))).extent : 0;
    return check_norm_weight(weight, weight_dtype, dtype, head_dim, out, out_b, code);
}

const char *check_norm_back_args(const void *grad, int64_t g_ts, int64_t g_hs, const void *x, int64_t x_ts, int64_t x_hs,
                                 const void *weight, int weight_dtype, const int64_t *positions, const float *cos_sin,
                                 int64_t cos_sin_rows, void *grad_x, int64_t dx_ts, int64_t dx_hs, void *grad_weight,
                                 int grad_weight_dtype, int T, int heads, int head_dim, int rot_dim, int layout, float eps,
                                 int dtype, const void *workspace, size_t workspace_bytes, int *code)
{
    if (const char *why = check_norm_args(grad, g_ts, g_hs, weight, weight_dtype, positions, cos_sin, cos_sin_rows, grad_x,
                                          dx_ts, dx_hs, T, heads, head_dim, rot_dim, layout, eps, dtype, code))
        return why;
    *code = QKVF_ERR_LAYOUT;
    if (!stride_ok(x_ts) || !stride_ok(x_hs)) return "strides must be 0..2^36 elements";
    if (grad_weight && grad_weight_dtype != dtype_of(dtype) && grad_weight_dtype != QKVF_DTYPE_FP32)
        return "the weight's gradient must be of the heads' type or fp32";
    *code = QKVF_ERR_ARG;
    if (grad_weight && !weight) return "a gradient of no weight";
    *code = QKVF_ERR_ALIGN;
    if (!aligned(grad_weight, dtype_bytes(grad_weight_dtype))) return "the weight's gradient must be aligned to its elements";
    *code = QKVF_OK;
    if (T == 0 && !grad_weight) return nullptr;
    const int elt = dtype_bytes(dtype_of(dtype));
    *code = QKVF_ERR_NULL;
    if ((T > 0 && !x) || (T > 0 && grad_weight && !workspace)) return "a required pointer is NULL";
    *code = QKVF_ERR_ALIGN;
    if (!aligned(x, elt)) return "x must be aligned to its elements";
    if (!aligned(workspace, 256)) return "the workspace must be 256-byte aligned";
    *code = QKVF_ERR_ARG;
    const View vx = T > 0 ? view_of(x, T, x_ts, heads, x_hs, head_dim, elt) : View{};
    const View vg = T > 0 ? view_of(grad, T, g_ts, heads, g_hs, head_dim, elt) : View{};
    const View vd = T > 0 ? view_of(grad_x, T, dx_ts, heads, dx_hs, head_dim, elt) : View{};
    if (T > 0 && views_overlap(vx, vd)) return "grad_x overlaps x";
    const size_t dw_b = grad_weight ? (size_t)head_dim * dtype_bytes(grad_weight_dtype) : 0;
    const void *in[] = {vg.ptr, vx.ptr, weight, positions, cos_sin, vd.ptr, grad_weight};
    const size_t bytes[] = {vg.extent, vx.extent, weight ? (size_t)head_dim * dtype_bytes(weight_dtype) : 0, (size_t)T * 8,
                            T > 0 ? (size_t)cos_sin_rows * rot_dim * 4 : 0, vd.extent, dw_b};
    for (int i = 0; i < 6; ++i)
        if (dw_b && bytes[i] && overlap(in[i], bytes[i], grad_weight, dw_b)) return "the weight's gradient overlaps another argument";
    for (int i = 0; i < 7; ++i)
        if (grad_weight && T > 0 && bytes[i] && overlap(in[i], bytes[i], workspace, workspace_bytes))
            return "the workspace overlaps another argument";
    *code = QKVF_OK;
    return nullptr;
}

size_t norm_back_workspace(int64_t T, int heads, int head_dim, int sms)
{
    const size_t n = (size_t)norm_back_ctas(T * heads, sms) * head_dim * 4;
    return (n + 255) / 256 * 256;
}

const char *check_norm_append_args(const void *q, int64_t q_ts, int64_t q_hs, const void *k, int64_t k_ts, int64_t k_hs,
                                   const void *v, int64_t v_ts, int64_t v_hs, const void *q_weight, const void *k_weight,
                                   int weight_dtype, const int64_t *positions, const int64_t *slots, const float *cos_sin,
                                   int64_t cos_sin_rows, void *q_out, int64_t o_ts, int64_t o_hs, void *kv_cache,
                                   int64_t num_pages, int T, int q_heads, int num_kv_heads, int head_dim, int rot_dim,
                                   int layout, float eps, int dtype, int *code)
{
    if (const char *why = check_append_args(q, q_ts, q_hs, k, k_ts, k_hs, v, v_ts, v_hs, positions, slots, cos_sin,
                                            cos_sin_rows, q_out, o_ts, o_hs, kv_cache, num_pages, T, q_heads, num_kv_heads,
                                            head_dim, rot_dim, layout, dtype, code))
        return why;
    *code = QKVF_ERR_ARG;
    if (!norm_eps_ok(eps)) return "eps must be in [0, 1]";
    const size_t cache_b = T > 0 ? (size_t)num_pages * num_kv_heads * kPageSlots * 2 * head_dim * 2 : 0;
    const size_t out_b = T > 0 && q_heads > 0 ? view_of(q_out, T, o_ts, q_heads, o_hs, head_dim, 2).extent : 0;
    for (const void *w : {q_weight, k_weight}) {
        if (const char *why = check_norm_weight(w, weight_dtype, dtype, head_dim, kv_cache, cache_b, code)) return why;
        if (const char *why = check_norm_weight(w, weight_dtype, dtype, head_dim, out_b ? q_out : nullptr, out_b, code)) return why;
    }
    return nullptr;
}

}  // namespace qkvf

extern "C" {

const char *norm_rope_unsupported(const void *x, int64_t x_token_stride, int64_t x_head_stride, const void *weight,
                                  int weight_dtype, const int64_t *positions, const float *cos_sin,
                                  int64_t cos_sin_rows, void *out, int64_t out_token_stride, int64_t out_head_stride,
                                  int T, int heads, int head_dim, int rot_dim, int layout, float eps, int dtype)
{
    int code;
    const char *why = qkvf::check_norm_args(x, x_token_stride, x_head_stride, weight, weight_dtype, positions, cos_sin,
                                            cos_sin_rows, out, out_token_stride, out_head_stride, T, heads, head_dim,
                                            rot_dim, layout, eps, dtype, &code);
    if (why) return why;
    qkvf::DeviceState *d;
    const int rc = qkvf::probe_device(&d);
    return rc == QKVF_OK ? nullptr : qkv_front_strerror(rc);
}

int norm_rope(const void *x, int64_t x_token_stride, int64_t x_head_stride, const void *weight, int weight_dtype,
              const int64_t *positions, const float *cos_sin, int64_t cos_sin_rows, void *out, int64_t out_token_stride,
              int64_t out_head_stride, int T, int heads, int head_dim, int rot_dim, int layout, float eps, int dtype,
              void *stream)
{
    int code;
    if (qkvf::check_norm_args(x, x_token_stride, x_head_stride, weight, weight_dtype, positions, cos_sin, cos_sin_rows,
                              out, out_token_stride, out_head_stride, T, heads, head_dim, rot_dim, layout, eps, dtype,
                              &code))
        return code;
    if (T == 0) return QKVF_OK;
    qkvf::DeviceState *d;
    const int rc = qkvf::probe_device(&d);
    if (rc != QKVF_OK) return rc;
    qkvf::NormParams prm = {};
    prm.r.q = x;
    prm.r.out = out;
    prm.r.positions = positions;
    prm.r.cos_sin = cos_sin;
    prm.r.cos_rows = cos_sin_rows;
    prm.r.q_ts = x_token_stride;
    prm.r.q_hs = x_head_stride;
    prm.r.o_ts = out_token_stride;
    prm.r.o_hs = out_head_stride;
    prm.r.T = T;
    prm.r.q_heads = heads;
    prm.r.dim = head_dim;
    prm.r.rot = rot_dim;
    prm.r.zero = qkvf::zero_skipped(dtype);
    prm.qw = weight;
    prm.qw_fp32 = weight_dtype == QKVF_DTYPE_FP32;
    prm.eps = eps;
    dtype = qkvf::dtype_of(dtype);
    const bool half = layout == QKVF_ROPE_HALF;
    return dtype == QKVF_DTYPE_BF16   ? qkvf::launch_norm<qkvf::Bf16>(prm, half, d->sms, stream)
           : dtype == QKVF_DTYPE_FP16 ? qkvf::launch_norm<qkvf::Fp16>(prm, half, d->sms, stream)
                                      : qkvf::launch_norm<qkvf::Fp32>(prm, half, d->sms, stream);
}

size_t norm_rope_backward_workspace_bytes(int T, int heads, int head_dim)
{
    if (T < 0 || T > qkvf::kRopeMaxTokens || heads < 1 || heads > qkvf::kRopeMaxHeads || head_dim < 2 ||
        head_dim > qkvf::kRopeMaxDim)
        return 0;
    qkvf::DeviceState *d;
    return qkvf::probe_device(&d) == QKVF_OK ? qkvf::norm_back_workspace(T, heads, head_dim, d->sms) : 0;
}

const char *norm_rope_backward_unsupported(const void *grad_out, int64_t grad_token_stride, int64_t grad_head_stride,
                                           const void *x, int64_t x_token_stride, int64_t x_head_stride,
                                           const void *weight, int weight_dtype, const int64_t *positions,
                                           const float *cos_sin, int64_t cos_sin_rows, void *grad_x,
                                           int64_t grad_x_token_stride, int64_t grad_x_head_stride, void *grad_weight,
                                           int grad_weight_dtype, int T, int heads, int head_dim, int rot_dim,
                                           int layout, float eps, int dtype, const void *workspace,
                                           size_t workspace_bytes)
{
    int code;
    const char *why = qkvf::check_norm_back_args(grad_out, grad_token_stride, grad_head_stride, x, x_token_stride,
                                                 x_head_stride, weight, weight_dtype, positions, cos_sin, cos_sin_rows,
                                                 grad_x, grad_x_token_stride, grad_x_head_stride, grad_weight,
                                                 grad_weight_dtype, T, heads, head_dim, rot_dim, layout, eps, dtype,
                                                 workspace, workspace_bytes, &code);
    if (why) return why;
    qkvf::DeviceState *d;
    const int rc = qkvf::probe_device(&d);
    if (rc != QKVF_OK) return qkv_front_strerror(rc);
    return T > 0 && grad_weight && workspace_bytes < qkvf::norm_back_workspace(T, heads, head_dim, d->sms)
               ? "the workspace is too small"
               : nullptr;
}

int norm_rope_backward(const void *grad_out, int64_t grad_token_stride, int64_t grad_head_stride, const void *x,
                       int64_t x_token_stride, int64_t x_head_stride, const void *weight, int weight_dtype,
                       const int64_t *positions, const float *cos_sin, int64_t cos_sin_rows, void *grad_x,
                       int64_t grad_x_token_stride, int64_t grad_x_head_stride, void *grad_weight,
                       int grad_weight_dtype, int T, int heads, int head_dim, int rot_dim, int layout, float eps,
                       int dtype, void *workspace, size_t workspace_bytes, void *stream)
{
    int code;
    if (qkvf::check_norm_back_args(grad_out, grad_token_stride, grad_head_stride, x, x_token_stride, x_head_stride,
                                   weight, weight_dtype, positions, cos_sin, cos_sin_rows, grad_x, grad_x_token_stride,
                                   grad_x_head_stride, grad_weight, grad_weight_dtype, T, heads, head_dim, rot_dim,
                                   layout, eps, dtype, workspace, workspace_bytes, &code))
        return code;
    if (T == 0 && !grad_weight) return QKVF_OK;
    qkvf::DeviceState *d;
    const int rc = qkvf::probe_device(&d);
    if (rc != QKVF_OK) return rc;
    if (T == 0)   // no token: a gradient of zeros
        return qkvf::launch_pdl(qkvf::norm_dw_kernel, dim3((unsigned)((head_dim + 31) / 32)), dim3(1024), 0, stream,
                                (const float *)nullptr, 0, head_dim, grad_weight, grad_weight_dtype);
    if (grad_weight && workspace_bytes < qkvf::norm_back_workspace(T, heads, head_dim, d->sms)) return QKVF_ERR_SIZES;
    qkvf::NormParams prm = {};
    prm.r.q = grad_out;
    prm.r.out = grad_x;
    prm.r.positions = positions;
    prm.r.cos_sin = cos_sin;
    prm.r.cos_rows = cos_sin_rows;
    prm.r.q_ts = grad_token_stride;
    prm.r.q_hs = grad_head_stride;
    prm.r.o_ts = grad_x_token_stride;
    prm.r.o_hs = grad_x_head_stride;
    prm.r.T = T;
    prm.r.q_heads = heads;
    prm.r.dim = head_dim;
    prm.r.rot = rot_dim;
    prm.r.zero = qkvf::zero_skipped(dtype);
    prm.x = x;
    prm.x_ts = x_token_stride;
    prm.x_hs = x_head_stride;
    prm.qw = weight;
    prm.qw_fp32 = weight_dtype == QKVF_DTYPE_FP32;
    prm.eps = eps;
    prm.part = grad_weight ? static_cast<float *>(workspace) : nullptr;
    dtype = qkvf::dtype_of(dtype);
    const bool half = layout == QKVF_ROPE_HALF;
    return dtype == QKVF_DTYPE_BF16
               ? qkvf::launch_norm_back<qkvf::Bf16>(prm, half, d->sms, grad_weight, grad_weight_dtype, stream)
           : dtype == QKVF_DTYPE_FP16
               ? qkvf::launch_norm_back<qkvf::Fp16>(prm, half, d->sms, grad_weight, grad_weight_dtype, stream)
               : qkvf::launch_norm_back<qkvf::Fp32>(prm, half, d->sms, grad_weight, grad_weight_dtype, stream);
}

const char *norm_rope_kv_append_unsupported(
    const void *q, int64_t q_token_stride, int64_t q_head_stride, const void *k, int64_t k_token_stride,
    int64_t k_head_stride, const void *v, int64_t v_token_stride, int64_t v_head_stride, const void *q_weight,
    const void *k_weight, int weight_dtype, const int64_t *positions, const int64_t *slots, const float *cos_sin,
    int64_t cos_sin_rows, void *q_out, int64_t q_out_token_stride, int64_t q_out_head_stride, void *kv_cache,
    int64_t num_pages, int T, int q_heads, int num_kv_heads, int head_dim, int rot_dim, int layout, float eps, int dtype)
{
    int code;
    const char *why = qkvf::check_norm_append_args(
        q, q_token_stride, q_head_stride, k, k_token_stride, k_head_stride, v, v_token_stride, v_head_stride, q_weight,
        k_weight, weight_dtype, positions, slots, cos_sin, cos_sin_rows, q_out, q_out_token_stride, q_out_head_stride,
        kv_cache, num_pages, T, q_heads, num_kv_heads, head_dim, rot_dim, layout, eps, dtype, &code);
    if (why) return why;
    qkvf::DeviceState *d;
    const int rc = qkvf::probe_device(&d);
    return rc == QKVF_OK ? nullptr : qkv_front_strerror(rc);
}

int norm_rope_kv_append(const void *q, int64_t q_token_stride, int64_t q_head_stride, const void *k,
                        int64_t k_token_stride, int64_t k_head_stride, const void *v, int64_t v_token_stride,
                        int64_t v_head_stride, const void *q_weight, const void *k_weight, int weight_dtype,
                        const int64_t *positions, const int64_t *slots, const float *cos_sin, int64_t cos_sin_rows,
                        void *q_out, int64_t q_out_token_stride, int64_t q_out_head_stride, void *kv_cache,
                        int64_t num_pages, int T, int q_heads, int num_kv_heads, int head_dim, int rot_dim, int layout,
                        float eps, int dtype, void *stream)
{
    int code;
    if (qkvf::check_norm_append_args(q, q_token_stride, q_head_stride, k, k_token_stride, k_head_stride, v,
                                     v_token_stride, v_head_stride, q_weight, k_weight, weight_dtype, positions, slots,
                                     cos_sin, cos_sin_rows, q_out, q_out_token_stride, q_out_head_stride, kv_cache,
                                     num_pages, T, q_heads, num_kv_heads, head_dim, rot_dim, layout, eps, dtype, &code))
        return code;
    if (T == 0) return QKVF_OK;
    qkvf::DeviceState *d;
    const int rc = qkvf::probe_device(&d);
    if (rc != QKVF_OK) return rc;
    qkvf::NormParams prm = {};
    qkvf::RopeParams &r = prm.r;
    r.q = q;
    r.k = k;
    r.v = v;
    r.out = q_out;
    r.kv_cache = kv_cache;
    r.positions = positions;
    r.slots = slots;
    r.cos_sin = cos_sin;
    r.cos_rows = cos_sin_rows;
    r.slot_end = num_pages * qkvf::kPageSlots;
    r.q_ts = q_token_stride;
    r.q_hs = q_head_stride;
    r.k_ts = k_token_stride;
    r.k_hs = k_head_stride;
    r.v_ts = v_token_stride;
    r.v_hs = v_head_stride;
    r.o_ts = q_out_token_stride;
    r.o_hs = q_out_head_stride;
    r.T = T;
    r.q_heads = q_heads;
    r.nkv = num_kv_heads;
    r.dim = head_dim;
    r.rot = rot_dim;
    r.zero = qkvf::zero_skipped(dtype);
    prm.qw = q_weight;
    prm.kw = k_weight;
    prm.qw_fp32 = prm.kw_fp32 = weight_dtype == QKVF_DTYPE_FP32;
    prm.eps = eps;
    const bool half = layout == QKVF_ROPE_HALF;
    return qkvf::dtype_of(dtype) == QKVF_DTYPE_BF16 ? qkvf::launch_norm<qkvf::Bf16>(prm, half, d->sms, stream)
                                                    : qkvf::launch_norm<qkvf::Fp16>(prm, half, d->sms, stream);
}

int norm_rope_packed(const int64_t *args, void *stream)
{
    if (!args) return QKVF_ERR_NULL;
    qkvf::Words w(args);
    const int wd = w.i(4), T = w.i(11), heads = w.i(12), dim = w.i(13), rot = w.i(14), layout = w.i(15), dtype = w.i(17);
    if (!w.ok) return QKVF_ERR_SIZES;
    return norm_rope(w.p<void>(0), args[1], args[2], w.p<void>(3), wd, w.p<int64_t>(5), w.p<float>(6), args[7], w.p<void>(8),
                     args[9], args[10], T, heads, dim, rot, layout, (float)w.d(16), dtype, stream);
}

int norm_rope_backward_packed(const int64_t *args, void *stream)
{
    if (!args) return QKVF_ERR_NULL;
    qkvf::Words w(args);
    const int wd = w.i(7), dwd = w.i(15), T = w.i(16), heads = w.i(17), dim = w.i(18), rot = w.i(19), layout = w.i(20),
              dtype = w.i(22);
    if (!w.ok) return QKVF_ERR_SIZES;
    return norm_rope_backward(w.p<void>(0), args[1], args[2], w.p<void>(3), args[4], args[5], w.p<void>(6), wd,
                              w.p<int64_t>(8), w.p<float>(9), args[10], w.p<void>(11), args[12], args[13], w.p<void>(14), dwd, T,
                              heads, dim, rot, layout, (float)w.d(21), dtype, w.p<void>(23), (size_t)args[24], stream);
}

int norm_rope_kv_append_packed(const int64_t *args, void *stream)
{
    if (!args) return QKVF_ERR_NULL;
    qkvf::Words w(args);
    const int wd = w.i(11), T = w.i(21), q_heads = w.i(22), nkv = w.i(23), dim = w.i(24), rot = w.i(25), layout = w.i(26),
              dtype = w.i(28);
    if (!w.ok) return QKVF_ERR_SIZES;
    return norm_rope_kv_append(w.p<void>(0), args[1], args[2], w.p<void>(3), args[4], args[5], w.p<void>(6), args[7], args[8],
                               w.p<void>(9), w.p<void>(10), wd, w.p<int64_t>(12), w.p<int64_t>(13), w.p<float>(14), args[15],
                               w.p<void>(16), args[17], args[18], w.p<void>(19), args[20], T, q_heads, nkv, dim, rot, layout,
                               (float)w.d(27), dtype, stream);
}

}  // extern "C"
