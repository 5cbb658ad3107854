// Norm of queries and keys for each head with the position rotation in the
// same pass, its gradient, and the rotation's table.
//
// Forward, for a head x of D columns at a token of position p:
//   r = 1 / sqrt(mean(x^2) + eps),  y = x r w,
//   (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin)  for the R/2 pairs.
// Backward: rotate the output's gradient by the negative angles to dy, then
//   dw = sum over rows of dy x r,  g = dy w,  dx = r (g - x r mean(g x r)).
// Both are bound by memory: the forward reads and writes each element once,
// the backward reads two and writes one.  The mean square is computed again
// in the backward because x is read there anyway.
//
// Vector path: a head is cut into units of two 8-element vectors that hold
// whole rotation pairs (half layout: columns 8u.. and R/2 + 8u..; interleaved:
// 16 consecutive columns; unrotated columns: 16 consecutive), one unit a lane,
// so the rotation needs no exchange between lanes and the two sums of a head
// are butterflies over G = 4 to 32 lanes.  A warp holds 32 / G heads of one
// token at a time, keeps the token's cosines and sines and the weight in
// registers over the token's heads, and issues the loads of two heads before
// it uses the first.
#include <cuda_runtime.h>

#include "ops_internal.h"

namespace {

using tide::from_f32;
using tide::load8;
using tide::op_aligned;
using tide::op_fail;
using tide::store8;
using tide::to_f32;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxHeadDim = 4096;
constexpr int kMaxVecHeadDim = 512;
constexpr int kGenericSmem = 40 * 1024;  // weight-gradient sums of the generic backward

// Strided heads of one tensor.
template <typename T>
struct Heads {
    T *p;
    int64_t st, sh;
    __device__ T *row(int64_t t, int h) const { return p + t * st + h * sh; }
};

// Queries or keys of a call.
template <typename T>
struct Part {
    Heads<T> x, d, out;  // input; output's gradient (backward); output or input's gradient
    const T *w;
    int heads;
    int heads_per_item;
    int64_t items;       // tokens * ceil(heads / heads_per_item)
    float *partial;      // backward: weight-gradient sums, one row of D for each block
    int blocks;          // backward: blocks that work on this part
};

template <typename T>
struct QkArgs {
    Part<T> part[2];
    int64_t tokens;
    int D, R;
    int64_t max_position;
    const float *table;
    const void *positions;
    int position_bytes;
    float eps;
};

template <typename T>
__device__ __forceinline__ int64_t position_of(const QkArgs<T> &a, int64_t t)
{
    const int64_t p = a.position_bytes == 8 ? static_cast<const int64_t *>(a.positions)[t]
                                            : int64_t(static_cast<const int32_t *>(a.positions)[t]);
    return p >= 0 && p < a.max_position ? p : -1;
}

// Where a lane's unit lies in a head (see the top of the file).
struct Unit {
    int off0, off1, ci;
    bool has0, has1, rot;
};
template <bool IL>
__device__ __forceinline__ Unit unit_of(int u, int D, int R)
{
    Unit n;
    const int nrot = R / 16;
    n.rot = u < nrot;
    n.off0 = n.rot ? (IL ? 16 * u : 8 * u) : R + 16 * (u - nrot);
    n.off1 = n.rot && !IL ? R / 2 + 8 * u : n.off0 + 8;
    n.has0 = n.off0 < D;
    n.has1 = n.off1 < D;
    n.ci = 8 * u;
    return n;
}

template <typename T>
__device__ __forceinline__ void load_unit(const T *row, const Unit &n, bool on, float (&v)[16])
{
#pragma unroll
    for (int i = 0; i < 16; ++i)
        v[i] = 0.f;
    if (on && n.has0)
        load8(row + n.off0, v);
    if (on && n.has1)
        load8(row + n.off1, v + 8);
}
template <typename T>
__device__ __forceinline__ void store_unit(T *row, const Unit &n, bool on, const float (&v)[16])
{
    if (on && n.has0)
        store8(row + n.off0, v);
    if (on && n.has1)
        store8(row + n.off1, v + 8);
}

// Cosines and sines of a unit's eight pairs.
template <typename T>
__device__ __forceinline__ void load_angles(const QkArgs<T> &a, int64_t t, const Unit &n, float (&c)[8], float (&s)[8])
{
    if (!n.rot)
        return;
    const int64_t pos = position_of(a, t);
    if (pos < 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            c[i] = s[i] = __int_as_float(0x7fffffff);
        return;
    }
    const float *row = a.table + pos * a.R;
    load8(row + n.ci, c);
    load8(row + a.R / 2 + n.ci, s);
}

// (a, b) -> (a c - b s, b c + a s), with s negated for the way back.
template <bool IL, bool BACK>
__device__ __forceinline__ void rotate(float (&v)[16], const float (&c)[8], const float (&s)[8])
{
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float &x = v[IL ? 2 * j : j], &y = v[IL ? 2 * j + 1 : 8 + j];
        const float sj = BACK ? -s[j] : s[j];
        const float nx = __fmaf_rn(x, c[j], -__fmul_rn(y, sj));
        y = __fmaf_rn(y, c[j], __fmul_rn(x, sj));
        x = nx;
    }
}

template <int G>
__device__ __forceinline__ float group_sum(float x)
{
#pragma unroll
    for (int o = G / 2; o > 0; o /= 2)
        x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

template <int G>
__device__ __forceinline__ float inv_rms(const float (&v)[16], int D, float eps)
{
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        ss = __fmaf_rn(v[i], v[i], ss);
    return rsqrtf(__fdividef(group_sum<G>(ss), float(D)) + eps);
}

template <typename T, int G, bool IL>
__global__ void __launch_bounds__(kThreads) qk_forward_kernel(const QkArgs<T> a)
{
    constexpr int kRows = 32 / G;  // heads of one step of a warp
    const int lane = threadIdx.x & 31, g = lane / G;
    const Unit n = unit_of<IL>(lane % G, a.D, a.R);
    int64_t item = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const int which = item >= a.part[0].items;
    if (which)
        item -= a.part[0].items;
    const Part<T> &p = a.part[which];
    if (item >= p.items)
        return;
    const int chunks = (p.heads + p.heads_per_item - 1) / p.heads_per_item;
    const int64_t t = item / chunks;
    const int h0 = int(item - t * chunks) * p.heads_per_item;
    const int h1 = min(p.heads, h0 + p.heads_per_item);

    float c[8], s[8], w[16];
    load_angles(a, t, n, c, s);
    if (p.w)
        load_unit(p.w, n, true, w);
    for (int hb = h0; hb < h1; hb += 2 * kRows) {
        const int h[2] = {hb + g, hb + kRows + g};
        float v[2][16];
#pragma unroll
        for (int k = 0; k < 2; ++k)
            load_unit(p.x.row(t, h[k]), n, h[k] < h1, v[k]);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (p.w) {
                const float r = inv_rms<G>(v[k], a.D, a.eps);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    v[k][i] = v[k][i] * r * w[i];
            }
            if (n.rot)
                rotate<IL, false>(v[k], c, s);
            store_unit(p.out.row(t, h[k]), n, h[k] < h1, v[k]);
        }
    }
}

template <typename T, int G, bool IL>
__global__ void __launch_bounds__(kThreads) qk_backward_kernel(const QkArgs<T> a)
{
    constexpr int kRows = 32 / G;
    __shared__ float sums[kThreads / G][16 * G];
    const int lane = threadIdx.x & 31, g = lane / G, u = lane % G;
    const Unit n = unit_of<IL>(u, a.D, a.R);
    const int which = int(blockIdx.x) >= a.part[0].blocks;
    const Part<T> &p = a.part[which];
    const int block = int(blockIdx.x) - (which ? a.part[0].blocks : 0);
    const int chunks = (p.heads + p.heads_per_item - 1) / p.heads_per_item;

    float w[16], acc[16];
#pragma unroll
    for (int i = 0; i < 16; ++i)
        acc[i] = 0.f;
    if (p.w)
        load_unit(p.w, n, true, w);
    for (int64_t item = int64_t(block) * kWarps + (threadIdx.x >> 5); item < p.items;
         item += int64_t(p.blocks) * kWarps) {
        const int64_t t = item / chunks;
        const int h0 = int(item - t * chunks) * p.heads_per_item;
        const int h1 = min(p.heads, h0 + p.heads_per_item);
        float c[8], s[8];
        load_angles(a, t, n, c, s);
        for (int hb = h0; hb < h1; hb += kRows) {
            const int h = hb + g;
            float d[16], x[16];
            load_unit(p.d.row(t, h), n, h < h1, d);
            if (p.w)
                load_unit(p.x.row(t, h), n, h < h1, x);
            if (n.rot)
                rotate<IL, true>(d, c, s);
            if (p.w) {
                const float r = inv_rms<G>(x, a.D, a.eps);
                float m = 0.f;
                if (h >= h1) {  // an idle group's gradient is 0, even where its token's angles are NaN
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        d[i] = x[i] = 0.f;
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    x[i] *= h < h1 ? r : 0.f;
                    acc[i] = __fmaf_rn(d[i], x[i], acc[i]);
                    d[i] *= w[i];
                    m = __fmaf_rn(d[i], x[i], m);
                }
                m = __fdividef(group_sum<G>(m), float(a.D));
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    d[i] = r * __fmaf_rn(-x[i], m, d[i]);
            }
            store_unit(p.out.row(t, h), n, h < h1, d);
        }
    }
    if (!p.w)
        return;
    const int row = (threadIdx.x >> 5) * kRows + g;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (n.has0)
            sums[row][n.off0 + i] = acc[i];
        if (n.has1)
            sums[row][n.off1 + i] = acc[8 + i];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.D; i += kThreads) {
        float x = 0.f;
        for (int k = 0; k < kThreads / G; ++k)
            x += sums[k][i];
        p.partial[int64_t(block) * a.D + i] = x;
    }
}

// Generic path (any D up to 4096, any alignment): a warp for each head, a
// lane for every 32nd pair or unrotated column, the head read once for its
// sums and again for its output.
struct Cols {
    int a, b;  // columns of a pair; b < 0: an unrotated column
};
template <bool IL>
__device__ __forceinline__ Cols cols_of(int i, int R)
{
    if (i >= R / 2)
        return {i + R / 2, -1};
    return IL ? Cols{2 * i, 2 * i + 1} : Cols{i, i + R / 2};
}

__device__ __forceinline__ float warp_sum(float x) { return group_sum<32>(x); }

template <typename T, bool IL, bool GRAD>
__global__ void __launch_bounds__(kThreads) qk_generic_kernel(const QkArgs<T> a)
{
    extern __shared__ float sums[];  // GRAD: [warps][D]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int which = int(blockIdx.x) >= a.part[0].blocks;
    const Part<T> &p = a.part[which];
    const int block = int(blockIdx.x) - (which ? a.part[0].blocks : 0);
    const int n = a.D - a.R / 2;
    float *mine = sums + warp * a.D;
    if (GRAD && p.w)
        for (int i = lane; i < a.D; i += 32)
            mine[i] = 0.f;
    __syncwarp();
    for (int64_t item = int64_t(block) * warps + warp; item < p.items; item += int64_t(p.blocks) * warps) {
        const int64_t t = item / p.heads;
        const int h = int(item - t * p.heads);
        const T *x = p.x.row(t, h);
        const T *d = GRAD ? p.d.row(t, h) : nullptr;
        T *out = p.out.row(t, h);
        const int64_t pos = a.R ? position_of(a, t) : -1;
        const float *cs = a.table + (pos < 0 ? 0 : pos) * a.R;
        const float bad = __int_as_float(0x7fffffff);
        float r = 1.f, m = 0.f;
        if (p.w) {
            float ss = 0.f;
            for (int i = lane; i < a.D; i += 32) {
                const float f = to_f32(x[i]);
                ss = __fmaf_rn(f, f, ss);
            }
            r = rsqrtf(__fdividef(warp_sum(ss), float(a.D)) + a.eps);
        }
        // The (rotated back) output's gradient of a pair.
        auto grad = [&](const Cols &k, int i, float &da, float &db) {
            da = to_f32(d[k.a]);
            db = 0.f;
            if (k.b >= 0) {
                db = to_f32(d[k.b]);
                const float c = pos < 0 ? bad : cs[i], s = pos < 0 ? bad : cs[a.R / 2 + i];
                const float na = __fmaf_rn(da, c, __fmul_rn(db, s));
                db = __fmaf_rn(db, c, -__fmul_rn(da, s));
                da = na;
            }
        };
        if (GRAD && p.w) {
            for (int i = lane; i < n; i += 32) {
                const Cols k = cols_of<IL>(i, a.R);
                float da, db;
                grad(k, i, da, db);
                const float xa = to_f32(x[k.a]) * r;
                mine[k.a] = __fmaf_rn(da, xa, mine[k.a]);
                m = __fmaf_rn(da * to_f32(p.w[k.a]), xa, m);
                if (k.b >= 0) {
                    const float xb = to_f32(x[k.b]) * r;
                    mine[k.b] = __fmaf_rn(db, xb, mine[k.b]);
                    m = __fmaf_rn(db * to_f32(p.w[k.b]), xb, m);
                }
            }
            m = __fdividef(warp_sum(m), float(a.D));
        }
        for (int i = lane; i < n; i += 32) {
            const Cols k = cols_of<IL>(i, a.R);
            if (GRAD) {
                float da, db;
                grad(k, i, da, db);
                if (p.w) {
                    da = r * __fmaf_rn(-(to_f32(x[k.a]) * r), m, da * to_f32(p.w[k.a]));
                    if (k.b >= 0)
                        db = r * __fmaf_rn(-(to_f32(x[k.b]) * r), m, db * to_f32(p.w[k.b]));
                }
                out[k.a] = from_f32<T>(da);
                if (k.b >= 0)
                    out[k.b] = from_f32<T>(db);
            } else {
                float ya = to_f32(x[k.a]), yb = k.b >= 0 ? to_f32(x[k.b]) : 0.f;
                if (p.w) {
                    ya = ya * r * to_f32(p.w[k.a]);
                    if (k.b >= 0)
                        yb = yb * r * to_f32(p.w[k.b]);
                }
                if (k.b >= 0) {
                    const float c = pos < 0 ? bad : cs[i], s = pos < 0 ? bad : cs[a.R / 2 + i];
                    const float na = __fmaf_rn(ya, c, -__fmul_rn(yb, s));
                    out[k.b] = from_f32<T>(__fmaf_rn(yb, c, __fmul_rn(ya, s)));
                    ya = na;
                }
                out[k.a] = from_f32<T>(ya);
            }
        }
    }
    if (!GRAD || !p.w)
        return;
    __syncthreads();
    for (int i = threadIdx.x; i < a.D; i += blockDim.x) {
        float x = 0.f;
        for (int k = 0; k < warps; ++k)
            x += sums[k * a.D + i];
        p.partial[int64_t(block) * a.D + i] = x;
    }
}

// dw = sum of the blocks' rows, in a fixed order: 32 columns a block, 32
// slices of the rows each.
template <typename T>
__global__ void __launch_bounds__(1024) qk_weight_grad_kernel(const float *pq, int nq, T *dq, const float *pk, int nk,
                                                              T *dk, int D)
{
    __shared__ float sums[32][33];
    const float *p = blockIdx.y ? pk : pq;
    const int n = blockIdx.y ? nk : nq;
    T *out = blockIdx.y ? dk : dq;
    if (!out)
        return;
    const int col = blockIdx.x * 32 + threadIdx.x;
    float x = 0.f;
    if (col < D)
        for (int i = threadIdx.y; i < n; i += 32)
            x += p[int64_t(i) * D + col];
    sums[threadIdx.y][threadIdx.x] = x;
    __syncthreads();
    x = group_sum<32>(sums[threadIdx.x][threadIdx.y]);
    const int c2 = blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 0 && c2 < D)
        out[c2] = from_f32<T>(x);
}

__global__ void rope_table_kernel(int64_t n, int half, double base, int scaling, double factor, double low,
                                  double high, double original, float *table)
{
    const int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i >= n * half)
        return;
    const int64_t p = i / half;
    const int k = int(i - p * half);
    double f = pow(base, -2.0 * k / (2.0 * half));
    if (scaling == 1) {
        f /= factor;
    } else if (scaling == 2) {
        const double turns = original * f / 6.283185307179586;  // original / wavelength
        if (turns < low)
            f /= factor;
        else if (turns <= high) {
            const double mix = (turns - low) / (high - low);
            f = (1.0 - mix) * f / factor + mix * f;
        }
    }
    double s, c;
    sincos(double(p) * f, &s, &c);
    table[p * 2 * half + k] = float(c);
    table[p * 2 * half + half + k] = float(s);
}

size_t elem_bytes(int dtype) { return dtype == TIDE_DTYPE_F32 ? 4 : 2; }

tide_status_t check_desc(const tide_qk_t *qk)
{
    if (!qk)
        return op_fail(TIDE_ERR_INVALID_ARG, "qk is NULL");
    if (qk->dtype != TIDE_DTYPE_BF16 && qk->dtype != TIDE_DTYPE_F32)
        return op_fail(TIDE_ERR_UNSUPPORTED, "dtype %d is not implemented", qk->dtype);
    if (qk->tokens < 0 || qk->q_heads < 0 || qk->k_heads < 0 || qk->q_heads > (1 << 20) || qk->k_heads > (1 << 20))
        return op_fail(TIDE_ERR_INVALID_ARG, "tokens %lld, q_heads %d, k_heads %d", (long long)qk->tokens, qk->q_heads,
                       qk->k_heads);
    if (qk->head_dim < 1 || qk->head_dim > kMaxHeadDim)
        return op_fail(TIDE_ERR_INVALID_ARG, "head_dim %d outside [1, %d]", qk->head_dim, kMaxHeadDim);
    if (qk->rotary_dim < 0 || qk->rotary_dim > qk->head_dim || qk->rotary_dim % 2)
        return op_fail(TIDE_ERR_INVALID_ARG, "rotary_dim %d: need an even number in [0, head_dim = %d]",
                       qk->rotary_dim, qk->head_dim);
    if (!(qk->eps >= 0.f) || qk->eps > 1e30f)
        return op_fail(TIDE_ERR_INVALID_ARG, "eps %g", double(qk->eps));
    const int64_t most = int64_t(0x7fffffff) * kWarps / 2;  // items of one launch
    if (qk->tokens > 0 && (int64_t(qk->q_heads) > most / qk->tokens || int64_t(qk->k_heads) > most / qk->tokens))
        return op_fail(TIDE_ERR_INVALID_ARG, "tokens %lld times heads is over %lld", (long long)qk->tokens,
                       (long long)most);
    if (qk->rotary_dim > 0 && qk->tokens > 0) {
        if (qk->position_bytes != 4 && qk->position_bytes != 8)
            return op_fail(TIDE_ERR_INVALID_ARG, "position_bytes %d: need 4 or 8", qk->position_bytes);
        if (!qk->table || !qk->positions || qk->max_position < 1 || qk->max_position > tide::kMaxExtent / kMaxHeadDim)
            return op_fail(TIDE_ERR_INVALID_ARG, "a rotation needs a table, positions and max_position >= 1");
        if (!op_aligned(qk->table, 4) || !op_aligned(qk->positions, size_t(qk->position_bytes)))
            return op_fail(TIDE_ERR_ALIGNMENT, "table or positions not aligned to their element size");
    }
    for (const void *w : {qk->q_weight, qk->k_weight})
        if (w && !op_aligned(w, elem_bytes(qk->dtype)))
            return op_fail(TIDE_ERR_ALIGNMENT, "a weight is not aligned to its element size");
    return TIDE_OK;
}

// A tensor of heads: pointer, alignment, strides; an output's rows must be apart.
tide_status_t check_heads(const tide_qk_t *qk, const tide_heads_t *x, int heads, bool output, const char *name)
{
    if (heads == 0 || qk->tokens == 0)
        return TIDE_OK;
    if (!x || !x->data)
        return op_fail(TIDE_ERR_INVALID_ARG, "%s is NULL", name);
    if (!op_aligned(x->data, elem_bytes(qk->dtype)))
        return op_fail(TIDE_ERR_ALIGNMENT, "%s is not aligned to its element size", name);
    if (x->token_stride < 0 || x->head_stride < 0 || !tide::op_extent_ok(qk->tokens, x->token_stride) ||
        !tide::op_extent_ok(heads, x->head_stride))
        return op_fail(TIDE_ERR_INVALID_ARG, "%s has bad strides", name);
    if (output) {
        const bool many_t = qk->tokens > 1, many_h = heads > 1;
        bool apart = (!many_t || x->token_stride >= qk->head_dim) && (!many_h || x->head_stride >= qk->head_dim);
        if (apart && many_t && many_h) {
            const int64_t d = qk->head_dim;
            apart = x->token_stride >= x->head_stride ? x->token_stride >= (heads - 1) * x->head_stride + d
                                                      : x->head_stride >= (qk->tokens - 1) * x->token_stride + d;
        }
        if (!apart)
            return op_fail(TIDE_ERR_INVALID_ARG, "rows of %s overlap", name);
    }
    return TIDE_OK;
}

bool vec_rows(const tide_qk_t *qk, const tide_heads_t *x, int heads)
{
    if (heads == 0)
        return true;
    const int64_t v = 16 / int64_t(elem_bytes(qk->dtype));
    return op_aligned(x->data, 16) && (qk->tokens < 2 || x->token_stride % v == 0) &&
           (heads < 2 || x->head_stride % v == 0);
}

// 16-byte rows whose rotated part is whole units: the vector path.
bool vec_shape(const tide_qk_t *qk)
{
    return qk->head_dim <= kMaxVecHeadDim && qk->head_dim % 8 == 0 && qk->rotary_dim % 16 == 0 &&
           (qk->rotary_dim == 0 || op_aligned(qk->table, 16)) && (!qk->q_weight || op_aligned(qk->q_weight, 16)) &&
           (!qk->k_weight || op_aligned(qk->k_weight, 16));
}

// Lanes of one head: the power of two that holds its units.
int lanes_of(const tide_qk_t *qk)
{
    const int units = qk->rotary_dim / 16 + (qk->head_dim - qk->rotary_dim + 15) / 16;
    int g = 4;
    while (g < units)
        g *= 2;
    return g;
}

template <typename T>
Heads<T> heads_of(const tide_heads_t *x)
{
    return x ? Heads<T>{static_cast<T *>(x->data), x->token_stride, x->head_stride} : Heads<T>{nullptr, 0, 0};
}

// Blocks of the backward for queries and for keys: four a SM, shared by heads.
void grad_blocks(const tide_qk_t *qk, int sms, int *q, int *k)
{
    const int64_t all = int64_t(sms) * 4, heads = int64_t(qk->q_heads) + qk->k_heads;
    int64_t nq = heads ? (all * qk->q_heads + heads - 1) / heads : 0;
    int64_t nk = all - nq;
    if (qk->k_heads > 0 && nk < 1)
        nk = 1;
    *q = int(qk->q_heads > 0 ? std::min(nq, qk->tokens * qk->q_heads) : 0);
    *k = int(qk->k_heads > 0 ? std::min(nk, qk->tokens * qk->k_heads) : 0);
}

template <typename T>
QkArgs<T> make_args(const tide_qk_t *qk)
{
    QkArgs<T> a = {};
    a.tokens = qk->tokens;
    a.D = qk->head_dim;
    a.R = qk->rotary_dim;
    a.max_position = qk->max_position;
    a.table = qk->table;
    a.positions = qk->positions;
    a.position_bytes = qk->position_bytes;
    a.eps = qk->eps;
    a.part[0].w = static_cast<const T *>(qk->q_weight);
    a.part[1].w = static_cast<const T *>(qk->k_weight);
    a.part[0].heads = qk->q_heads;
    a.part[1].heads = qk->k_heads;
    return a;
}

template <typename T, int G>
void launch_forward(const QkArgs<T> &a, bool il, unsigned grid, cudaStream_t st)
{
    if (il)
        qk_forward_kernel<T, G, true><<<grid, kThreads, 0, st>>>(a);
    else
        qk_forward_kernel<T, G, false><<<grid, kThreads, 0, st>>>(a);
}
template <typename T, int G>
void launch_backward(const QkArgs<T> &a, bool il, unsigned grid, cudaStream_t st)
{
    if (il)
        qk_backward_kernel<T, G, true><<<grid, kThreads, 0, st>>>(a);
    else
        qk_backward_kernel<T, G, false><<<grid, kThreads, 0, st>>>(a);
}

template <typename T, bool GRAD>
void launch_generic(const QkArgs<T> &a, bool il, cudaStream_t st)
{
    int warps = kWarps;
    if (GRAD)
        warps = std::max(1, std::min(warps, kGenericSmem / (4 * a.D)));
    const size_t smem = GRAD ? size_t(warps) * a.D * 4 : 0;
    const unsigned grid = unsigned(a.part[0].blocks + a.part[1].blocks);
    if (il)
        qk_generic_kernel<T, true, GRAD><<<grid, warps * 32, smem, st>>>(a);
    else
        qk_generic_kernel<T, false, GRAD><<<grid, warps * 32, smem, st>>>(a);
}

template <typename T>
tide_status_t forward(const tide_qk_t *qk, const tide_heads_t *q, const tide_heads_t *k, const tide_heads_t *qo,
                      const tide_heads_t *ko, cudaStream_t st)
{
    QkArgs<T> a = make_args<T>(qk);
    const tide_heads_t *in[2] = {q, k}, *out[2] = {qo, ko};
    bool vec = vec_shape(qk);
    for (int i = 0; i < 2; ++i) {
        Part<T> &p = a.part[i];
        p.x = heads_of<T>(in[i]);
        p.out = heads_of<T>(out[i]);
        vec = vec && vec_rows(qk, in[i], p.heads) && vec_rows(qk, out[i], p.heads);
    }
    if (!vec) {
        for (Part<T> &p : a.part) {
            p.items = qk->tokens * p.heads;
            p.blocks = int(std::min<int64_t>((p.items + kWarps - 1) / kWarps, 1 << 20));
        }
        launch_generic<T, false>(a, qk->interleaved, st);
        return tide::op_launched("qk_norm_rope");
    }
    const int g = lanes_of(qk);
    for (Part<T> &p : a.part) {
        // All heads of a token in one warp reuse its angles; few tokens are spread over more warps instead.
        p.heads_per_item = qk->tokens >= 4096 ? std::max(p.heads, 1) : 32 / g;
        p.items = qk->tokens * ((p.heads + p.heads_per_item - 1) / p.heads_per_item);
    }
    const unsigned grid = unsigned((a.part[0].items + a.part[1].items + kWarps - 1) / kWarps);
    switch (g) {
    case 4: launch_forward<T, 4>(a, qk->interleaved, grid, st); break;
    case 8: launch_forward<T, 8>(a, qk->interleaved, grid, st); break;
    case 16: launch_forward<T, 16>(a, qk->interleaved, grid, st); break;
    default: launch_forward<T, 32>(a, qk->interleaved, grid, st); break;
    }
    return tide::op_launched("qk_norm_rope");
}

template <typename T>
tide_status_t backward(const tide_qk_t *qk, const tide_heads_t *dqo, const tide_heads_t *dko, const tide_heads_t *q,
                       const tide_heads_t *k, const tide_heads_t *dq, const tide_heads_t *dk, T *dwq, T *dwk,
                       float *partial, cudaStream_t st)
{
    QkArgs<T> a = make_args<T>(qk);
    const tide_heads_t *in[2] = {q, k}, *grad[2] = {dqo, dko}, *out[2] = {dq, dk};
    bool vec = vec_shape(qk);
    for (int i = 0; i < 2; ++i) {
        Part<T> &p = a.part[i];
        p.x = heads_of<T>(p.w ? in[i] : nullptr);
        p.d = heads_of<T>(grad[i]);
        p.out = heads_of<T>(out[i]);
        vec = vec && (!p.w || vec_rows(qk, in[i], p.heads)) && vec_rows(qk, grad[i], p.heads) &&
              vec_rows(qk, out[i], p.heads);
    }
    grad_blocks(qk, tide::op_sm_count(), &a.part[0].blocks, &a.part[1].blocks);
    a.part[0].partial = partial;
    a.part[1].partial = partial + int64_t(a.part[0].blocks) * a.D;
    const unsigned grid = unsigned(a.part[0].blocks + a.part[1].blocks);
    if (!vec) {
        for (Part<T> &p : a.part)
            p.items = qk->tokens * p.heads;
        if (grid)
            launch_generic<T, true>(a, qk->interleaved, st);
    } else if (grid) {
        const int g = lanes_of(qk);
        for (Part<T> &p : a.part) {
            p.heads_per_item = qk->tokens >= 4096 ? std::max(p.heads, 1) : 32 / g;
            p.items = qk->tokens * ((p.heads + p.heads_per_item - 1) / p.heads_per_item);
        }
        switch (g) {
        case 4: launch_backward<T, 4>(a, qk->interleaved, grid, st); break;
        case 8: launch_backward<T, 8>(a, qk->interleaved, grid, st); break;
        case 16: launch_backward<T, 16>(a, qk->interleaved, grid, st); break;
        default: launch_backward<T, 32>(a, qk->interleaved, grid, st); break;
        }
    }
    if (grid)
        if (const tide_status_t s = tide::op_launched("qk_norm_rope_grad"))
            return s;
    if (!dwq && !dwk)
        return TIDE_OK;
    qk_weight_grad_kernel<T><<<dim3(unsigned((a.D + 31) / 32), 2), dim3(32, 32), 0, st>>>(
        a.part[0].partial, a.part[0].blocks, dwq, a.part[1].partial, a.part[1].blocks, dwk, a.D);
    return tide::op_launched("qk_norm_rope_grad: weights");
}

}  // namespace

extern "C" {

tide_status_t tide_rope_table(int64_t max_position, int32_t rotary_dim, double base, int32_t scaling, double factor,
                              double low_freq_factor, double high_freq_factor, double original, float *table,
                              void *stream)
{
    tide::record_error("");
    if (max_position < 0 || rotary_dim < 2 || rotary_dim % 2 || rotary_dim > kMaxHeadDim)
        return op_fail(TIDE_ERR_INVALID_ARG, "max_position %lld, rotary_dim %d", (long long)max_position, rotary_dim);
    if (!(base > 0) || scaling < 0 || scaling > 2 || (scaling && !(factor > 0)) ||
        (scaling == 2 && (!(low_freq_factor > 0) || !(high_freq_factor > low_freq_factor) || !(original > 0))))
        return op_fail(TIDE_ERR_INVALID_ARG, "base, scaling or its factors out of range");
    if (max_position > int64_t(0x7fffffff) * 256 / (rotary_dim / 2))
        return op_fail(TIDE_ERR_INVALID_ARG, "max_position %lld", (long long)max_position);
    if (max_position == 0)
        return TIDE_OK;
    if (!table)
        return op_fail(TIDE_ERR_INVALID_ARG, "table is NULL");
    if (!op_aligned(table, 4))
        return op_fail(TIDE_ERR_ALIGNMENT, "table is not aligned to its element size");
    const tide::NvtxRange range("tide_rope_table");
    const int64_t n = max_position * (rotary_dim / 2);
    rope_table_kernel<<<unsigned((n + 255) / 256), 256, 0, static_cast<cudaStream_t>(stream)>>>(
        max_position, rotary_dim / 2, base, scaling, factor, low_freq_factor, high_freq_factor, original, table);
    return tide::op_launched("rope_table");
}

tide_status_t tide_qk_norm_rope(const tide_qk_t *qk, const tide_heads_t *q, const tide_heads_t *k,
                                const tide_heads_t *q_out, const tide_heads_t *k_out, void *stream)
{
    tide::record_error("");
    tide_status_t s = check_desc(qk);
    if (!s)
        s = check_heads(qk, q, qk->q_heads, false, "q");
    if (!s)
        s = check_heads(qk, k, qk->k_heads, false, "k");
    if (!s)
        s = check_heads(qk, q_out, qk->q_heads, true, "q_out");
    if (!s)
        s = check_heads(qk, k_out, qk->k_heads, true, "k_out");
    if (s || qk->tokens == 0 || (qk->q_heads == 0 && qk->k_heads == 0))
        return s;
    const tide::NvtxRange range("tide_qk_norm_rope");
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return qk->dtype == TIDE_DTYPE_F32 ? forward<float>(qk, q, k, q_out, k_out, st)
                                       : forward<__nv_bfloat16>(qk, q, k, q_out, k_out, st);
}

int64_t tide_qk_norm_rope_grad_workspace(const tide_qk_t *qk)
{
    tide::record_error("");
    if (check_desc(qk))
        return -1;
    int nq, nk;
    grad_blocks(qk, tide::op_sm_count(), &nq, &nk);
    return std::max<int64_t>(256, (int64_t(nq) + nk) * qk->head_dim * 4);
}

tide_status_t tide_qk_norm_rope_grad(const tide_qk_t *qk, const tide_heads_t *dq_out, const tide_heads_t *dk_out,
                                     const tide_heads_t *q, const tide_heads_t *k, const tide_heads_t *dq,
                                     const tide_heads_t *dk, void *dq_weight, void *dk_weight, void *workspace,
                                     int64_t workspace_bytes, void *stream)
{
    tide::record_error("");
    tide_status_t s = check_desc(qk);
    if (!s)
        s = check_heads(qk, dq_out, qk->q_heads, false, "dq_out");
    if (!s)
        s = check_heads(qk, dk_out, qk->k_heads, false, "dk_out");
    if (!s && qk->q_weight)
        s = check_heads(qk, q, qk->q_heads, false, "q");
    if (!s && qk->k_weight)
        s = check_heads(qk, k, qk->k_heads, false, "k");
    if (!s)
        s = check_heads(qk, dq, qk->q_heads, true, "dq");
    if (!s)
        s = check_heads(qk, dk, qk->k_heads, true, "dk");
    if (s)
        return s;
    if (!qk->q_weight != !dq_weight || !qk->k_weight != !dk_weight)
        return op_fail(TIDE_ERR_INVALID_ARG, "a weight's gradient goes with the weight: both or neither");
    if ((dq_weight && !op_aligned(dq_weight, elem_bytes(qk->dtype))) ||
        (dk_weight && !op_aligned(dk_weight, elem_bytes(qk->dtype))))
        return op_fail(TIDE_ERR_ALIGNMENT, "a weight's gradient is not aligned to its element size");
    if (workspace_bytes < tide_qk_norm_rope_grad_workspace(qk) || !workspace)
        return op_fail(TIDE_ERR_INVALID_ARG, "workspace of %lld bytes: need %lld", (long long)workspace_bytes,
                       (long long)tide_qk_norm_rope_grad_workspace(qk));
    if (!op_aligned(workspace, 256))
        return op_fail(TIDE_ERR_ALIGNMENT, "workspace is not 256-byte aligned");
    const tide::NvtxRange range("tide_qk_norm_rope_grad");
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    float *partial = static_cast<float *>(workspace);
    if (qk->dtype == TIDE_DTYPE_F32)
        return backward<float>(qk, dq_out, dk_out, q, k, dq, dk, static_cast<float *>(dq_weight),
                               static_cast<float *>(dk_weight), partial, st);
    return backward<__nv_bfloat16>(qk, dq_out, dk_out, q, k, dq, dk, static_cast<__nv_bfloat16 *>(dq_weight),
                                   static_cast<__nv_bfloat16 *>(dk_weight), partial, st);
}

}  // extern "C"
