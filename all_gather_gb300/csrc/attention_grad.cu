// Gradient of softmax attention over packed sequences.
//
//   p = exp(s - lse),  delta_r = do_r o_r,  dp_rc = do_r v_c,  ds = p (dp - delta),
//   dq_r = scale sum_c ds_rc k_c,  dk_c = scale sum_r ds_rc q_r,  dv_c = sum_r p_rc do_r
#include "attention.h"

namespace {

using namespace tide::attn;
using tide::op_aligned;
using tide::op_fail;

__device__ int g_timed_out;

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

}  // namespace

namespace tide {
namespace attn {

cudaError_t grad_timed_out(int *seen, cudaStream_t st) { return take_flag(g_timed_out, seen, st); }

}  // namespace attn
}  // namespace tide

extern "C" {

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
