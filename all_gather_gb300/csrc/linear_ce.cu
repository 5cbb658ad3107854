// Softmax cross entropy of a vocabulary head and its gradient, without the
// logits in memory.
//
//   z = x W^T,  lse_t = log sum_v exp(z_tv),  loss_t = lse_t - z_t,target
//   dz = (exp(z - lse) - [v = target]) dloss,  dx = dz W,  dW = dz^T x
//
// The loss takes tiles of the logits as they are made: each tile leaves, for
// each of its rows, its maximum m and sum s of exp(z - m), and a second kernel
// joins a row's pairs in a fixed order.  The gradient makes the logits again,
// a piece of the vocabulary at a time, and keeps only that piece's dz.
#include <cuda_runtime.h>

#include "ops_internal.h"

namespace {

using tide::op_aligned;
using tide::op_fail;
using tide::to_f32;
using bf16 = __nv_bfloat16;

constexpr int kTile = 64, kStep = 16, kThreads = 256;
constexpr int64_t kPieceBytes = int64_t(256) << 20;  // dz of one piece of the vocabulary
constexpr int64_t kMinPiece = 8192;

// target of a token: its column, -1 = ignored, -2 = outside the vocabulary
struct Targets {
    const void *p;
    int bytes;
    int64_t ignore, vocab;
    __device__ int64_t get(int64_t t) const
    {
        const int64_t y = bytes == 8 ? static_cast<const int64_t *>(p)[t]
                                     : int64_t(static_cast<const int32_t *>(p)[t]);
        return y == ignore ? -1 : y < 0 || y >= vocab ? -2 : y;
    }
};

struct Operand {
    const bf16 *p;
    int64_t row, k;  // strides of the tile's rows (or columns) and of the sum
};

enum Epilogue { kStats, kDz, kAdd, kStore };

struct Gemm {
    Operand a, b;
    int64_t M, N, K;
    int64_t v0;          // first vocabulary column of this piece
    Targets y;
    float2 *part;        // kStats: [column tiles][M]
    float *zy;           // kStats: logit of the target
    const float *lse, *dloss;
    bf16 *out;           // kDz, kStore
    int64_t out_stride;
    float *acc;          // kAdd: [M][N], added to unless `first`
    int first;
};

template <int E>
__global__ void __launch_bounds__(kThreads) gemm_kernel(const Gemm g)
{
    __shared__ float as[kStep][kTile + 1], bs[kStep][kTile + 1];
    __shared__ float cs[E == kStats ? kTile : 1][kTile + 1];
    const int64_t m0 = int64_t(blockIdx.y) * kTile, n0 = int64_t(blockIdx.x) * kTile;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float c[4][4] = {};
    for (int64_t k0 = 0; k0 < g.K; k0 += kStep) {
        for (int i = threadIdx.x; i < kTile * kStep; i += kThreads) {
            const int k = i % kStep, r = i / kStep;
            const bool in_k = k0 + k < g.K;
            as[k][r] = in_k && m0 + r < g.M ? to_f32(g.a.p[(m0 + r) * g.a.row + (k0 + k) * g.a.k]) : 0.f;
            bs[k][r] = in_k && n0 + r < g.N ? to_f32(g.b.p[(n0 + r) * g.b.row + (k0 + k) * g.b.k]) : 0.f;
        }
        __syncthreads();
        for (int k = 0; k < kStep; ++k)
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j)
                    c[i][j] = __fmaf_rn(as[k][ty * 4 + i], bs[k][tx * 4 + j], c[i][j]);
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i) {
        const int64_t m = m0 + ty * 4 + i;
        for (int j = 0; j < 4; ++j) {
            const int64_t n = n0 + tx * 4 + j;
            if (E == kStats) {
                cs[ty * 4 + i][tx * 4 + j] = c[i][j];
            } else if (m < g.M && n < g.N) {
                if (E == kDz) {
                    const int64_t y = g.y.get(m);
                    float d = 0.f;
                    if (y != -1) {
                        d = (expf(c[i][j] - g.lse[m]) - (g.v0 + n == y ? 1.f : 0.f)) * g.dloss[m];
                        if (y == -2)
                            d = __int_as_float(0x7fffffff);
                    }
                    g.out[m * g.out_stride + n] = __float2bfloat16_rn(d);
                } else if (E == kAdd) {
                    float *p = g.acc + m * g.N + n;
                    *p = g.first ? c[i][j] : *p + c[i][j];
                } else {
                    g.out[m * g.out_stride + n] = __float2bfloat16_rn(c[i][j]);
                }
            }
        }
    }
    if (E != kStats)
        return;
    __syncthreads();
    const int r = threadIdx.x;
    if (r >= kTile || m0 + r >= g.M)
        return;
    const int64_t t = m0 + r, y = g.y.get(t);
    const int cols = int(min(int64_t(kTile), g.N - n0));
    float top = -INFINITY, sum = 0.f;
    for (int j = 0; j < cols; ++j) {
        top = fmaxf(top, cs[r][j]);
        if (n0 + j == y)
            g.zy[t] = cs[r][j];
    }
    const float at = isinf(top) ? 0.f : top;
    for (int j = 0; j < cols; ++j)
        sum += expf(cs[r][j] - at);
    g.part[int64_t(blockIdx.x) * g.M + t] = make_float2(top, sum);
}

__global__ void __launch_bounds__(256) join_kernel(const float2 *part, int64_t tiles, int64_t T, const float *zy,
                                                   Targets y, float *loss, float *lse)
{
    const int64_t t = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (t >= T)
        return;
    float top = -INFINITY, sum = 0.f;
    for (int64_t i = 0; i < tiles; ++i)
        top = fmaxf(top, part[i * T + t].x);
    for (int64_t i = 0; i < tiles; ++i) {
        const float2 p = part[i * T + t];
        sum += p.x == top ? p.y : p.y * expf(p.x - top);
    }
    const float l = logf(sum) + (isinf(top) ? 0.f : top);
    const int64_t v = y.get(t);
    lse[t] = l;
    loss[t] = v == -1 ? 0.f : v == -2 ? __int_as_float(0x7fffffff) : l - zy[t];
}

__global__ void __launch_bounds__(256) round_kernel(const float *acc, int64_t T, int64_t H, bf16 *out, int64_t stride)
{
    const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (i < T * H)
        out[i / H * stride + i % H] = __float2bfloat16_rn(acc[i]);
}

int64_t round_up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

tide_status_t check_desc(const tide_ce_t *ce)
{
    if (!ce)
        return op_fail(TIDE_ERR_INVALID_ARG, "ce is NULL");
    if (ce->tokens < 0 || ce->tokens > 0x7fffffff - 512 || ce->vocab < 1 || ce->vocab > 0x7fffffff - 512 ||
        ce->hidden < 1 || ce->hidden > (1 << 20))
        return op_fail(TIDE_ERR_INVALID_ARG, "tokens %lld, vocab %lld, hidden %lld", (long long)ce->tokens,
                       (long long)ce->vocab, (long long)ce->hidden);
    if (ce->target_bytes != 4 && ce->target_bytes != 8)
        return op_fail(TIDE_ERR_INVALID_ARG, "target_bytes %d: need 4 or 8", ce->target_bytes);
    if (!tide::op_extent_ok(ce->tokens, ce->x_stride) || !tide::op_extent_ok(ce->vocab, ce->weight_stride) ||
        (ce->tokens > 1 && ce->x_stride < ce->hidden) || (ce->vocab > 1 && ce->weight_stride < ce->hidden))
        return op_fail(TIDE_ERR_INVALID_ARG, "x_stride %lld, weight_stride %lld for hidden %lld",
                       (long long)ce->x_stride, (long long)ce->weight_stride, (long long)ce->hidden);
    return TIDE_OK;
}

tide_status_t check_data(const tide_ce_t *ce)
{
    if (!ce->weight || (ce->tokens > 0 && (!ce->x || !ce->targets)))
        return op_fail(TIDE_ERR_INVALID_ARG, "x, weight or targets is NULL");
    if (!op_aligned(ce->weight, 2) || !op_aligned(ce->x, 2) || !op_aligned(ce->targets, size_t(ce->target_bytes)))
        return op_fail(TIDE_ERR_ALIGNMENT, "x, weight or targets is not aligned to its element size");
    return TIDE_OK;
}

tide_status_t check_workspace(const void *workspace, int64_t have, int64_t need)
{
    if (!workspace || have < need)
        return op_fail(TIDE_ERR_INVALID_ARG, "workspace of %lld bytes: need %lld", (long long)have, (long long)need);
    if (!op_aligned(workspace, 256))
        return op_fail(TIDE_ERR_ALIGNMENT, "workspace is not 256-byte aligned");
    return TIDE_OK;
}

int64_t piece_of(const tide_ce_t *ce)
{
    const int64_t fit = kPieceBytes / 2 / std::max<int64_t>(ce->tokens, 1) / 256 * 256;
    return std::min(round_up(ce->vocab, 256), std::max(kMinPiece, fit));
}

dim3 grid_of(int64_t M, int64_t N) { return dim3(unsigned((N + kTile - 1) / kTile), unsigned((M + kTile - 1) / kTile)); }

Gemm base(const tide_ce_t *ce)
{
    Gemm g = {};
    g.y = {ce->targets, ce->target_bytes, ce->ignore_index, ce->vocab};
    return g;
}

}  // namespace

extern "C" {

int64_t tide_ce_loss_workspace(const tide_ce_t *ce)
{
    tide::record_error("");
    if (check_desc(ce))
        return -1;
    const int64_t tiles = (ce->vocab + kTile - 1) / kTile;
    return 256 + round_up(tiles * ce->tokens * 8, 256) + round_up(ce->tokens * 4, 256);
}

tide_status_t tide_ce_loss(const tide_ce_t *ce, float *loss, float *lse, void *workspace, int64_t workspace_bytes,
                           void *stream)
{
    tide::record_error("");
    tide_status_t s = check_desc(ce);
    if (!s)
        s = check_data(ce);
    if (s || ce->tokens == 0)
        return s;
    if (!loss || !lse)
        return op_fail(TIDE_ERR_INVALID_ARG, "loss or lse is NULL");
    if (!op_aligned(loss, 4) || !op_aligned(lse, 4))
        return op_fail(TIDE_ERR_ALIGNMENT, "loss or lse is not aligned to its element size");
    s = check_workspace(workspace, workspace_bytes, tide_ce_loss_workspace(ce));
    if (s)
        return s;
    const tide::NvtxRange range("tide_ce_loss");
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int64_t T = ce->tokens, V = ce->vocab, tiles = (V + kTile - 1) / kTile;
    Gemm g = base(ce);
    g.a = {static_cast<const bf16 *>(ce->x), ce->x_stride, 1};
    g.b = {static_cast<const bf16 *>(ce->weight), ce->weight_stride, 1};
    g.M = T, g.N = V, g.K = ce->hidden;
    g.part = static_cast<float2 *>(workspace);
    g.zy = reinterpret_cast<float *>(static_cast<char *>(workspace) + round_up(tiles * T * 8, 256));
    gemm_kernel<kStats><<<grid_of(T, V), kThreads, 0, st>>>(g);
    if ((s = tide::op_launched("ce_loss")))
        return s;
    join_kernel<<<unsigned((T + 255) / 256), 256, 0, st>>>(g.part, tiles, T, g.zy, g.y, loss, lse);
    return tide::op_launched("ce_loss: join");
}

int64_t tide_ce_grad_workspace(const tide_ce_t *ce)
{
    tide::record_error("");
    if (check_desc(ce))
        return -1;
    return 256 + round_up(ce->tokens * piece_of(ce) * 2, 256) + round_up(ce->tokens * ce->hidden * 4, 256);
}

tide_status_t tide_ce_grad(const tide_ce_t *ce, const float *lse, const float *dloss, void *dx, int64_t dx_stride,
                           void *dweight, int64_t dweight_stride, void *workspace, int64_t workspace_bytes,
                           void *stream)
{
    tide::record_error("");
    tide_status_t s = check_desc(ce);
    if (!s)
        s = check_data(ce);
    if (s)
        return s;
    if (!dweight || (ce->tokens > 0 && (!lse || !dloss || !dx)))
        return op_fail(TIDE_ERR_INVALID_ARG, "lse, dloss, dx or dweight is NULL");
    if (!op_aligned(lse, 4) || !op_aligned(dloss, 4) || !op_aligned(dx, 2) || !op_aligned(dweight, 2))
        return op_fail(TIDE_ERR_ALIGNMENT, "lse, dloss, dx or dweight is not aligned to its element size");
    if (!tide::op_extent_ok(ce->tokens, dx_stride) || !tide::op_extent_ok(ce->vocab, dweight_stride) ||
        (ce->tokens > 1 && dx_stride < ce->hidden) || (ce->vocab > 1 && dweight_stride < ce->hidden))
        return op_fail(TIDE_ERR_INVALID_ARG, "dx_stride %lld, dweight_stride %lld for hidden %lld",
                       (long long)dx_stride, (long long)dweight_stride, (long long)ce->hidden);
    s = check_workspace(workspace, workspace_bytes, tide_ce_grad_workspace(ce));
    if (s)
        return s;
    const tide::NvtxRange range("tide_ce_grad");
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int64_t T = ce->tokens, V = ce->vocab, H = ce->hidden, piece = piece_of(ce);
    const bf16 *x = static_cast<const bf16 *>(ce->x), *w = static_cast<const bf16 *>(ce->weight);
    bf16 *dz = static_cast<bf16 *>(workspace);
    float *acc = reinterpret_cast<float *>(static_cast<char *>(workspace) + round_up(T * piece * 2, 256));
    for (int64_t v0 = 0; v0 < V; v0 += piece) {
        const int64_t n = std::min(piece, V - v0);
        Gemm g = base(ce);
        g.v0 = v0;
        if (T > 0) {
            g.a = {x, ce->x_stride, 1};
            g.b = {w + v0 * ce->weight_stride, ce->weight_stride, 1};
            g.M = T, g.N = n, g.K = H;
            g.lse = lse, g.dloss = dloss, g.out = dz, g.out_stride = piece;
            gemm_kernel<kDz><<<grid_of(g.M, g.N), kThreads, 0, st>>>(g);
            if ((s = tide::op_launched("ce_grad: dz")))
                return s;
            g.a = {dz, piece, 1};
            g.b = {w + v0 * ce->weight_stride, 1, ce->weight_stride};
            g.M = T, g.N = H, g.K = n;
            g.acc = acc, g.first = v0 == 0;
            gemm_kernel<kAdd><<<grid_of(g.M, g.N), kThreads, 0, st>>>(g);
            if ((s = tide::op_launched("ce_grad: dx")))
                return s;
        }
        g.a = {dz, 1, piece};
        g.b = {x, 1, ce->x_stride};
        g.M = n, g.N = H, g.K = T;
        g.out = static_cast<bf16 *>(dweight) + v0 * dweight_stride, g.out_stride = dweight_stride;
        gemm_kernel<kStore><<<grid_of(g.M, g.N), kThreads, 0, st>>>(g);
        if ((s = tide::op_launched("ce_grad: dweight")))
            return s;
    }
    if (T == 0)
        return TIDE_OK;
    round_kernel<<<unsigned((T * H + 255) / 256), 256, 0, st>>>(acc, T, H, static_cast<bf16 *>(dx), dx_stride);
    return tide::op_launched("ce_grad: rounding");
}

tide_status_t tide_ops_device_status(void *stream)
{
    tide::record_error("");
    const cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? TIDE_OK : op_fail(TIDE_ERR_CUDA, "synchronise: %s", cudaGetErrorString(e));
}

}  // extern "C"
