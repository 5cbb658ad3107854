// Softmax attention of whole prompts over packed sequences, and its gradient.
//
//   s_rc = scale q_r k_c  for the keys c that row r sees,
//   lse_r = log sum_c exp(s_rc),  o_r = sum_c exp(s_rc - lse_r) v_c
//   p = exp(s - lse),  delta_r = do_r o_r,  dp_rc = do_r v_c,  ds = p (dp - delta),
//   dq_r = scale sum_c ds_rc k_c,  dk_c = scale sum_r ds_rc q_r,  dv_c = sum_r p_rc do_r
#include <cuda_runtime.h>

#include <algorithm>

#include "ops_internal.h"

namespace {

using tide::op_aligned;
using tide::op_fail;
using bf16 = __nv_bfloat16;

constexpr int kMaxHeadDim = 128;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr unsigned kAll = 0xffffffffu;

// A tensor of heads: rows of D contiguous elements on 16-byte boundaries.
struct Heads {
    bf16 *p;
    int64_t ts, hs;
    __host__ __device__ bf16 *row(int64_t t, int64_t h) const { return p + t * ts + h * hs; }
};

// [a, b): what a row sees, or which rows see a key; empty: a >= b.
struct Span {
    int a, b;
};

struct Problem {
    const void *offsets;  // NULL: one sequence
    int offset_bytes, n;  // n sequences
    int T, Hq, Hk, D, causal;
    float scale;

    __device__ int64_t offset(int i) const
    {
        return offset_bytes == 8 ? static_cast<const int64_t *>(offsets)[i]
                                 : int64_t(static_cast<const int32_t *>(offsets)[i]);
    }
    // The sequence of token t, cut to [0, T); empty if it belongs to none.  Whatever the offsets hold, nothing
    // outside them is read and what comes out lies in [0, T).
    __device__ Span sequence(int t) const
    {
        if (t < 0 || t >= T)
            return {0, 0};
        if (!offsets)
            return {0, T};
        int lo = -1, hi = n;  // offset(lo) <= t < offset(hi)
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (offset(mid) <= t)
                lo = mid;
            else
                hi = mid;
        }
        if (lo < 0)
            return {0, 0};
        const int64_t a = max(int64_t(0), offset(lo)), b = min(int64_t(T), offset(lo + 1));
        return a <= t && t < b ? Span{int(a), int(b)} : Span{0, 0};
    }
    __device__ Span keys_of(int r) const
    {
        const Span s = sequence(r);
        return {s.a, causal ? min(s.b, r + 1) : s.b};
    }
    __device__ Span rows_of(int c) const
    {
        const Span s = sequence(c);
        return {causal ? max(s.a, c) : s.a, s.b};
    }
};

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ---------------------------------------------------------------- rows by themselves
//
// One row (or key) a lane, by the formulas, over what it sees and nothing else.

__device__ float dot_row(const bf16 *a, const bf16 *b, int D)
{
    float s = 0.f;
    for (int d = 0; d < D; d += 8) {
        float x[8], y[8];
        tide::load8(a + d, x);
        tide::load8(b + d, y);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            s = fmaf(x[i], y[i], s);
    }
    return s;
}

// The union of a warp's spans.
__device__ Span warp_span(Span s)
{
    const bool some = s.a < s.b;
    return {__reduce_min_sync(kAll, some ? s.a : 0x7fffffff), __reduce_max_sync(kAll, some ? s.b : 0)};
}

// log2 of the sum of 2^(c s) over the span, -inf if it is empty.
__device__ float row_lse2(const bf16 *q, const Heads &k, int hk, Span see, int D, float c)
{
    const Span all = warp_span(see);
    float top = -INFINITY, sum = 0.f;
    for (int j = all.a; j < all.b; ++j) {
        if (j < see.a || j >= see.b)
            continue;
        const float s = dot_row(q, k.row(j, hk), D) * c;
        const float m = fmaxf(top, s), at = isinf(m) ? 0.f : m;
        sum = sum * exp2_fast(top - at) + exp2_fast(s - at);
        top = m;
    }
    return see.a < see.b ? (isinf(top) ? 0.f : top) + log2f(sum) : -INFINITY;
}

__device__ void row_forward(const bf16 *q, const Heads &k, const Heads &v, int hk, Span see, int D, float c, float lse2,
                            bf16 *o)
{
    const Span all = warp_span(see);
    for (int d0 = 0; d0 < D; d0 += 8) {
        float acc[8] = {};
        for (int j = all.a; j < all.b; ++j) {
            if (j < see.a || j >= see.b)
                continue;
            const float p = exp2_fast(dot_row(q, k.row(j, hk), D) * c - lse2);
            float x[8];
            tide::load8(v.row(j, hk) + d0, x);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                acc[i] = fmaf(p, x[i], acc[i]);
        }
        if (o)
            tide::store8(o + d0, acc);
    }
}

__global__ void __launch_bounds__(128) forward_simple(Problem pr, Heads q, Heads k, Heads v, Heads o, float *lse)
{
    const int r = blockIdx.x * 128 + threadIdx.x, h = blockIdx.y, hk = h / (pr.Hq / pr.Hk);
    const Span see = r < pr.T ? pr.keys_of(r) : Span{0, 0};
    const bool mine = r < pr.T;
    const bf16 *qr = q.row(mine ? r : 0, h);
    const float c = pr.scale * kLog2e, lse2 = row_lse2(qr, k, hk, see, pr.D, c);
    row_forward(qr, k, v, hk, see, pr.D, c, lse2, mine ? o.row(r, h) : nullptr);
    if (mine)
        lse[int64_t(h) * pr.T + r] = lse2 * kLn2;
}

// delta [Hq][T] = sum over d of do * o.
__global__ void __launch_bounds__(256) delta_kernel(Problem pr, Heads dout, Heads o, float *delta)
{
    const int64_t i = (int64_t(blockIdx.x) * 256 + threadIdx.x) / 16;  // 16 lanes a row
    const int at = threadIdx.x % 16 * 8;
    const int64_t t = i / pr.Hq;
    const int h = int(i % pr.Hq);
    float s = 0.f;
    if (t < pr.T && at < pr.D) {
        float x[8], y[8];
        tide::load8(dout.row(t, h) + at, x);
        tide::load8(o.row(t, h) + at, y);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            s = fmaf(x[j], y[j], s);
    }
#pragma unroll
    for (int w = 8; w > 0; w /= 2)
        s += __shfl_xor_sync(kAll, s, w);
    if (t < pr.T && at == 0)
        delta[int64_t(h) * pr.T + t] = s;
}

__device__ void row_dq(const bf16 *q, const bf16 *dout, const Heads &k, const Heads &v, int hk, Span see, int D, float c,
                       float scale, float lse2, float delta, bf16 *dq)
{
    const Span all = warp_span(see);
    for (int d0 = 0; d0 < D; d0 += 8) {
        float acc[8] = {};
        for (int j = all.a; j < all.b; ++j) {
            if (j < see.a || j >= see.b)
                continue;
            const float p = exp2_fast(dot_row(q, k.row(j, hk), D) * c - lse2);
            const float ds = p * (dot_row(dout, v.row(j, hk), D) - delta);
            float x[8];
            tide::load8(k.row(j, hk) + d0, x);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                acc[i] = fmaf(ds, x[i], acc[i]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            acc[i] *= scale;
        if (dq)
            tide::store8(dq + d0, acc);
    }
}

__device__ void row_dkv(const Problem &pr, const bf16 *k, const bf16 *v, const Heads &q, const Heads &dout, int hk, Span see,
                        float c, const float *lse, const float *delta, bf16 *dk, bf16 *dv)
{
    const Span all = warp_span(see);
    const int group = pr.Hq / pr.Hk, D = pr.D;
    for (int d0 = 0; d0 < D; d0 += 8) {
        float ak[8] = {}, av[8] = {};
        for (int h = hk * group; h < (hk + 1) * group; ++h)
            for (int r = all.a; r < all.b; ++r) {
                if (r < see.a || r >= see.b)
                    continue;
                const int64_t i = int64_t(h) * pr.T + r;
                const float p = exp2_fast(dot_row(q.row(r, h), k, D) * c - lse[i] * kLog2e);
                const float ds = p * (dot_row(dout.row(r, h), v, D) - delta[i]);
                float x[8], y[8];
                tide::load8(q.row(r, h) + d0, x);
                tide::load8(dout.row(r, h) + d0, y);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    ak[j] = fmaf(ds, x[j], ak[j]);
                    av[j] = fmaf(p, y[j], av[j]);
                }
            }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            ak[i] *= pr.scale;
        if (dk) {
            tide::store8(dk + d0, ak);
            tide::store8(dv + d0, av);
        }
    }
}

__global__ void __launch_bounds__(128) dq_simple(Problem pr, Heads q, Heads k, Heads v, Heads dout, const float *lse,
                                                 const float *delta, Heads dq)
{
    const int r = blockIdx.x * 128 + threadIdx.x, h = blockIdx.y, hk = h / (pr.Hq / pr.Hk);
    const bool mine = r < pr.T;
    const Span see = mine ? pr.keys_of(r) : Span{0, 0};
    const int64_t t = mine ? r : 0, i = int64_t(h) * pr.T + t;
    row_dq(q.row(t, h), dout.row(t, h), k, v, hk, see, pr.D, pr.scale * kLog2e, pr.scale, lse[i] * kLog2e, delta[i],
           mine ? dq.row(r, h) : nullptr);
}

__global__ void __launch_bounds__(128) dkv_simple(Problem pr, Heads q, Heads k, Heads v, Heads dout, const float *lse,
                                                  const float *delta, Heads dk, Heads dv)
{
    const int c = blockIdx.x * 128 + threadIdx.x, h = blockIdx.y;
    const bool mine = c < pr.T;
    const Span see = mine ? pr.rows_of(c) : Span{0, 0};
    const int64_t t = mine ? c : 0;
    row_dkv(pr, k.row(t, h), v.row(t, h), q, dout, h, see, pr.scale * kLog2e, lse, delta, mine ? dk.row(c, h) : nullptr,
            mine ? dv.row(c, h) : nullptr);
}

// ---------------------------------------------------------------- host

tide_status_t check_desc(const tide_attention_t *at)
{
    if (!at)
        return op_fail(TIDE_ERR_INVALID_ARG, "at is NULL");
    if (at->tokens < 0 || at->tokens > 0x7fffffff - 512)
        return op_fail(TIDE_ERR_INVALID_ARG, "tokens %lld", (long long)at->tokens);
    if (at->k_heads < 1 || at->q_heads < 1 || at->q_heads > 65535 || at->q_heads % at->k_heads)
        return op_fail(TIDE_ERR_INVALID_ARG, "q_heads %d, k_heads %d: need a multiple, at most 65535", at->q_heads,
                       at->k_heads);
    if (at->tokens * at->q_heads > int64_t(1) << 34)
        return op_fail(TIDE_ERR_INVALID_ARG, "tokens %lld times q_heads %d is above 2^34", (long long)at->tokens,
                       at->q_heads);
    if (at->head_dim < 8 || at->head_dim % 8)
        return op_fail(TIDE_ERR_INVALID_ARG, "head_dim %d: need a multiple of 8", at->head_dim);
    if (at->head_dim > kMaxHeadDim)
        return op_fail(TIDE_ERR_UNSUPPORTED, "head_dim %d: at most %d", at->head_dim, kMaxHeadDim);
    if (!(at->scale > 0.f) || at->scale > 3.0e38f)
        return op_fail(TIDE_ERR_INVALID_ARG, "scale %g: need a positive number", double(at->scale));
    if (at->offsets) {
        if (at->sequences < 0 || at->sequences > 0x7ffffffe)
            return op_fail(TIDE_ERR_INVALID_ARG, "sequences %lld", (long long)at->sequences);
        if (at->offset_bytes != 4 && at->offset_bytes != 8)
            return op_fail(TIDE_ERR_INVALID_ARG, "offset_bytes %d: need 4 or 8", at->offset_bytes);
        if (!op_aligned(at->offsets, size_t(at->offset_bytes)))
            return op_fail(TIDE_ERR_ALIGNMENT, "offsets are not aligned to their size");
    }
    return TIDE_OK;
}

tide_status_t check_heads(const tide_attention_t *at, const tide_heads_t *x, int heads, bool output, const char *name)
{
    if (at->tokens == 0)
        return TIDE_OK;
    if (!x || !x->data)
        return op_fail(TIDE_ERR_INVALID_ARG, "%s is NULL", name);
    const bool many_t = at->tokens > 1, many_h = heads > 1;
    const int64_t limit = int64_t(1) << 38;  // a tensor map's strides are below 2^40 bytes
    if ((many_t && (x->token_stride < 1 || x->token_stride > limit)) ||
        (many_h && (x->head_stride < 1 || x->head_stride > limit)))
        return op_fail(TIDE_ERR_INVALID_ARG, "%s has bad strides", name);
    if (!op_aligned(x->data, 16) || (many_t && x->token_stride % 8) || (many_h && x->head_stride % 8))
        return op_fail(TIDE_ERR_ALIGNMENT, "rows of %s are not on 16-byte boundaries", name);
    if (output) {
        const int64_t d = at->head_dim;
        bool apart = (!many_t || x->token_stride >= d) && (!many_h || x->head_stride >= d);
        if (apart && many_t && many_h)
            apart = x->token_stride >= x->head_stride ? x->token_stride >= (heads - 1) * x->head_stride + d
                                                      : x->head_stride >= (at->tokens - 1) * x->token_stride + d;
        if (!apart)
            return op_fail(TIDE_ERR_INVALID_ARG, "rows of %s overlap", name);
    }
    return TIDE_OK;
}

tide_status_t check_floats(const tide_attention_t *at, const float *p, const char *name)
{
    if (at->tokens && !p)
        return op_fail(TIDE_ERR_INVALID_ARG, "%s is NULL", name);
    return op_aligned(p, 4) ? TIDE_OK : op_fail(TIDE_ERR_ALIGNMENT, "%s is not aligned to its element size", name);
}

Problem problem_of(const tide_attention_t *at)
{
    Problem p = {};
    p.offsets = at->offsets, p.offset_bytes = at->offset_bytes, p.n = int(at->sequences);
    p.T = int(at->tokens), p.Hq = at->q_heads, p.Hk = at->k_heads, p.D = at->head_dim;
    p.causal = at->causal != 0, p.scale = at->scale;
    return p;
}

// Strides of dimensions of one element are not looked at: any will do.
Heads heads_of(const tide_attention_t *at, const tide_heads_t *x, int heads)
{
    return {static_cast<bf16 *>(x->data), at->tokens > 1 ? x->token_stride : int64_t(at->head_dim),
            heads > 1 ? x->head_stride : int64_t(at->head_dim)};
}

}  // namespace

extern "C" {

tide_status_t tide_attention(const tide_attention_t *at, const tide_heads_t *q, const tide_heads_t *k,
                             const tide_heads_t *v, const tide_heads_t *o, float *lse, void *stream)
{
    tide::record_error("");
    tide_status_t s = check_desc(at);
    if (!s)
        s = check_heads(at, q, at->q_heads, false, "q");
    if (!s)
        s = check_heads(at, k, at->k_heads, false, "k");
    if (!s)
        s = check_heads(at, v, at->k_heads, false, "v");
    if (!s)
        s = check_heads(at, o, at->q_heads, true, "o");
    if (!s)
        s = check_floats(at, lse, "lse");
    if (s || at->tokens == 0)
        return s;
    const tide::NvtxRange range("tide_attention");
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const Problem p = problem_of(at);
    forward_simple<<<dim3(unsigned((p.T + 127) / 128), unsigned(p.Hq)), 128, 0, st>>>(
        p, heads_of(at, q, p.Hq), heads_of(at, k, p.Hk), heads_of(at, v, p.Hk), heads_of(at, o, p.Hq), lse);
    return tide::op_launched("attention");
}

int64_t tide_attention_grad_workspace(const tide_attention_t *at)
{
    tide::record_error("");
    if (check_desc(at))
        return -1;
    return std::max<int64_t>(256, at->tokens * at->q_heads * 4);
}

tide_status_t tide_attention_grad(const tide_attention_t *at, const tide_heads_t *dout, const tide_heads_t *q,
                                  const tide_heads_t *k, const tide_heads_t *v, const tide_heads_t *o,
                                  const float *lse, const tide_heads_t *dq, const tide_heads_t *dk,
                                  const tide_heads_t *dv, void *workspace, int64_t workspace_bytes, void *stream)
{
    tide::record_error("");
    tide_status_t s = check_desc(at);
    const struct {
        const tide_heads_t *x;
        bool q, output;
        const char *name;
    } all[] = {{dout, true, false, "do"}, {q, true, false, "q"},  {k, false, false, "k"},  {v, false, false, "v"},
               {o, true, false, "o"},     {dq, true, true, "dq"}, {dk, false, true, "dk"}, {dv, false, true, "dv"}};
    for (const auto &a : all)
        if (!s)
            s = check_heads(at, a.x, a.q ? at->q_heads : at->k_heads, a.output, a.name);
    if (!s)
        s = check_floats(at, lse, "lse");
    if (s || at->tokens == 0)
        return s;
    const int64_t need = tide_attention_grad_workspace(at);
    if (!workspace || workspace_bytes < need)
        return op_fail(TIDE_ERR_INVALID_ARG, "workspace of %lld bytes: need %lld", (long long)workspace_bytes,
                       (long long)need);
    if (!op_aligned(workspace, 256))
        return op_fail(TIDE_ERR_ALIGNMENT, "workspace is not 256-byte aligned");
    const tide::NvtxRange range("tide_attention_grad");
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const Problem p = problem_of(at);
    float *delta = static_cast<float *>(workspace);
    const Heads hq = heads_of(at, q, p.Hq), hk = heads_of(at, k, p.Hk), hv = heads_of(at, v, p.Hk);
    const Heads hd = heads_of(at, dout, p.Hq);
    delta_kernel<<<unsigned((int64_t(p.T) * p.Hq + 15) / 16), 256, 0, st>>>(p, hd, heads_of(at, o, p.Hq), delta);
    s = tide::op_launched("attention_grad: delta");
    if (s)
        return s;
    const unsigned tiles = unsigned((p.T + 127) / 128);
    dkv_simple<<<dim3(tiles, unsigned(p.Hk)), 128, 0, st>>>(p, hq, hk, hv, hd, lse, delta, heads_of(at, dk, p.Hk),
                                                           heads_of(at, dv, p.Hk));
    s = tide::op_launched("attention_grad: dk, dv");
    if (s)
        return s;
    dq_simple<<<dim3(tiles, unsigned(p.Hq)), 128, 0, st>>>(p, hq, hk, hv, hd, lse, delta, heads_of(at, dq, p.Hq));
    return tide::op_launched("attention_grad: dq");
}

}  // extern "C"
