// Layer norm of rows, or without its centre the root-mean-square norm, and its
// gradient.
//
//   m = mean(x) (0 without the centre),  r = 1 / sqrt(mean((x - m)^2) + eps),
//   n = (x - m) r,  y = n w + b
//   g = dy w:  dx = r (g - mean(g) - n mean(g n)),  dw = sum over rows of dy n,
//   db = sum over rows of dy  (mean(g): only with the centre)
//
// A group of warps has a row in registers, so x (and dy) are read once; the
// second moment is taken around the mean that is already known, which keeps
// its digits where the mean is large.  The gradient takes its three sums in
// one go after the mean: sum(g n) = r sum(g (x - m)).  Statistics are computed
// again there rather than kept: x has to be read anyway.
//
// A thread keeps its columns for all rows of its group, so it adds up their dw
// and db in registers; the groups' shares go to the workspace and a second
// kernel adds them in a fixed order.
#include <cuda_runtime.h>

#include <algorithm>

#include "ops_internal.h"

namespace {

using tide::op_aligned;
using tide::op_fail;
using bf16 = __nv_bfloat16;

constexpr unsigned kAll = 0xffffffffu;
constexpr int kMaxWarps = 32;  // of a row

template <typename T>
struct Args {
    int64_t rows;
    int cols, center;
    float eps;
    const T *x, *dy, *w, *b;
    T *out;
    int64_t xs, dys, outs;
    float *partial;  // [groups][2][cols]: shares of dw, db
};

// ---------------------------------------------------------------- a row in registers

// U units of eight elements a thread.  Rows on 16-byte boundaries: unit u of
// thread t is elements 8 (u N + t) to + 7 of the row, N threads; others: its
// element i is number (8 u + i) N + t, so that neighbours read neighbours.
template <bool VEC>
__device__ __forceinline__ int column(int u, int i, int t, int n)
{
    return VEC ? 8 * (u * n + t) + i : (8 * u + i) * n + t;
}

// Eight elements as they lie in memory.
template <typename T>
struct Raw {
    uint4 v[sizeof(T) / 2];
};

__device__ __forceinline__ void unpack(const Raw<bf16> &raw, float *f);
__device__ __forceinline__ void unpack(const Raw<float> &raw, float *f);

// Unit u of a thread, from memory.
template <typename T, bool VEC>
__device__ __forceinline__ Raw<T> load_unit(const T *p, int cols, int u, int t, int n)
{
    Raw<T> raw;
    if (VEC) {
        const int c = column<VEC>(u, 0, t, n);
#pragma unroll
        for (int k = 0; k < int(sizeof(T) / 2); ++k)
            raw.v[k] = c < cols ? __ldg(reinterpret_cast<const uint4 *>(p + c) + k) : make_uint4(0, 0, 0, 0);
    } else {
        T e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = column<VEC>(u, i, t, n);
            e[i] = c < cols ? p[c] : T(0.f);
        }
        raw = *reinterpret_cast<Raw<T> *>(e);
    }
    return raw;
}

// Rows on their way to the threads that will work on them: a thread copies its
// own units to shared memory (cp.async) two rows ahead, and waits for nobody
// else's.  Where rows are not on 16-byte boundaries it loads them when it needs
// them.
constexpr int kStages = 3;
template <typename T, bool VEC, int U, int TENSORS>
struct Stream {
    static constexpr int kPieces = sizeof(T) / 2;                  // of 16 bytes a unit
    static constexpr int kStage = TENSORS * U * kPieces * 16;      // bytes a thread
    uint32_t at;                                                   // of the thread's first piece
    int pitch;                                                     // between pieces
    int stage;

    __device__ __forceinline__ Stream(uint32_t smem) : at(smem + threadIdx.x * 16), pitch(int(blockDim.x) * 16), stage(0) {}
    __device__ __forceinline__ void fetch(const T *const (&rows)[TENSORS], bool some, int ahead, int cols, int t, int n)
    {
        if (!VEC)
            return;
        const uint32_t to = at + uint32_t((stage + ahead) % kStages) * TENSORS * U * kPieces * pitch;
        if (some) {
#pragma unroll
            for (int k = 0; k < TENSORS; ++k)
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int c = column<VEC>(u, 0, t, n);
                    if (c < cols)
#pragma unroll
                        for (int i = 0; i < kPieces; ++i)
                            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                             to + uint32_t((k * U + u) * kPieces + i) * pitch),
                                         "l"(reinterpret_cast<const uint4 *>(rows[k] + c) + i)
                                         : "memory");
                }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    // The current row's units as fp32; what lies behind its end is 0.
    __device__ __forceinline__ void take(const T *const (&rows)[TENSORS], int cols, int t, int n, float (&f)[TENSORS][U][8])
    {
        if (VEC)
            asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
        const uint32_t from = at + uint32_t(stage) * TENSORS * U * kPieces * pitch;
#pragma unroll
        for (int k = 0; k < TENSORS; ++k)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                Raw<T> raw;
                if (VEC) {
                    const bool in = column<VEC>(u, 0, t, n) < cols;
#pragma unroll
                    for (int i = 0; i < kPieces; ++i) {
                        uint4 &v = raw.v[i];
                        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                                     : "r"(from + uint32_t((k * U + u) * kPieces + i) * pitch)
                                     : "memory");
                        if (!in)
                            v = make_uint4(0, 0, 0, 0);
                    }
                } else {
                    raw = load_unit<T, VEC>(rows[k], cols, u, t, n);
                }
                unpack(raw, f[k][u]);
            }
        stage = stage + 1 == kStages ? 0 : stage + 1;
    }
};

__device__ __forceinline__ void unpack(const Raw<bf16> &raw, float *f)
{
    const uint32_t w[4] = {raw.v[0].x, raw.v[0].y, raw.v[0].z, raw.v[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void unpack(const Raw<float> &raw, float *f)
{
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        f[4 * k] = __uint_as_float(raw.v[k].x), f[4 * k + 1] = __uint_as_float(raw.v[k].y);
        f[4 * k + 2] = __uint_as_float(raw.v[k].z), f[4 * k + 3] = __uint_as_float(raw.v[k].w);
    }
}
template <typename T, bool VEC>
__device__ __forceinline__ void store_unit(T *p, int cols, int u, int t, int n, const float *f)
{
    if (VEC) {
        const int c = column<VEC>(u, 0, t, n);
        if (c < cols)
            tide::store8(p + c, f);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = column<VEC>(u, i, t, n);
            if (c < cols)
                p[c] = tide::from_f32<T>(f[i]);
        }
    }
}

// A group: `warps` warps of the block that work on one row.
struct Group {
    int warps, index, t, n;  // its number in the block; the thread's number in it, of n
    float *shared;           // [2][warps][4]

    // Sums over the group, to all of its threads.  Two buffers in turn: who writes one again has met all
    // others at the barrier that follows their reading of it.
    template <int K>
    __device__ __forceinline__ void sum(float (&s)[K], int turn) const
    {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int o = 16; o > 0; o /= 2)
                s[k] += __shfl_xor_sync(kAll, s[k], o);
        if (warps == 1)
            return;
        float *buf = shared + turn * warps * 4;
        if (t % 32 == 0)
#pragma unroll
            for (int k = 0; k < K; ++k)
                buf[t / 32 * 4 + k] = s[k];
        asm volatile("bar.sync %0, %1;" ::"r"(index + 1), "r"(n) : "memory");
#pragma unroll
        for (int k = 0; k < K; ++k)
            s[k] = buf[k];
        for (int w = 1; w < warps; ++w)
#pragma unroll
            for (int k = 0; k < K; ++k)
                s[k] += buf[w * 4 + k];
    }
};

__device__ __forceinline__ Group group_of(int warps, float *shared)
{
    const int n = warps * 32, index = int(threadIdx.x) / n;
    return {warps, index, int(threadIdx.x) % n, n, shared + index * warps * 8};
}

// THREADS: of a block at most, with BLOCKS of them on an SM.
template <typename T, bool VEC, int U, int THREADS, int BLOCKS>
__global__ void __launch_bounds__(THREADS, BLOCKS) forward_kernel(Args<T> a, int warps)
{
    extern __shared__ uint4 ring[];
    __shared__ float shared[kMaxWarps * 8];
    const Group g = group_of(warps, shared);
    const int64_t step = int64_t(gridDim.x) * (blockDim.x / g.n);
    const float inv = 1.f / float(a.cols);
    Stream<T, VEC, U, 1> in(uint32_t(__cvta_generic_to_shared(ring)));
    int64_t row = int64_t(blockIdx.x) * (blockDim.x / g.n) + g.index;
    auto fetch = [&](int64_t r, int ahead) {
        const T *const rows[1] = {a.x + r * a.xs};
        in.fetch(rows, r < a.rows, ahead, a.cols, g.t, g.n);
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i)
        fetch(row + i * step, i);
    for (; row < a.rows; row += step) {
        fetch(row + (kStages - 1) * step, kStages - 1);
        float x[1][U][8], mean[1] = {0.f}, var[1] = {0.f};
        const T *const rows[1] = {a.x + row * a.xs};
        in.take(rows, a.cols, g.t, g.n, x);
        auto &f = x[0];
        if (a.center) {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    mean[0] += f[u][i];
            g.sum(mean, 0);
            mean[0] *= inv;
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                f[u][i] -= mean[0];
                if (column<VEC>(u, VEC ? 0 : i, g.t, g.n) < a.cols)
                    var[0] = fmaf(f[u][i], f[u][i], var[0]);
            }
        g.sum(var, 1);
        const float r = 1.f / sqrtf(fmaf(var[0], inv, a.eps));
        T *out = a.out + row * a.outs;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float k[8], s[8];
            if (a.w)
                unpack(load_unit<T, VEC>(a.w, a.cols, u, g.t, g.n), k);
            if (a.b)
                unpack(load_unit<T, VEC>(a.b, a.cols, u, g.t, g.n), s);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                f[u][i] *= r;
                if (a.w)
                    f[u][i] = a.b ? fmaf(f[u][i], k[i], s[i]) : f[u][i] * k[i];
                else if (a.b)
                    f[u][i] += s[i];
            }
            store_unit<T, VEC>(out, a.cols, u, g.t, g.n, f[u]);
        }
    }
}

template <typename T, bool VEC, int U, int THREADS, int BLOCKS>
__global__ void __launch_bounds__(THREADS, BLOCKS) backward_kernel(Args<T> a, int warps)
{
    extern __shared__ uint4 ring[];
    __shared__ float shared[kMaxWarps * 8];
    const Group g = group_of(warps, shared);
    const int groups = blockDim.x / g.n;
    const int64_t step = int64_t(gridDim.x) * groups;
    const float inv = 1.f / float(a.cols);
    Stream<T, VEC, U, 2> in(uint32_t(__cvta_generic_to_shared(ring)));
    float dw[U][8] = {}, db[U][8] = {};
    const int64_t first = int64_t(blockIdx.x) * groups + g.index;
    auto fetch = [&](int64_t r, int ahead) {
        const T *const rows[2] = {a.x + r * a.xs, a.dy + r * a.dys};
        in.fetch(rows, r < a.rows, ahead, a.cols, g.t, g.n);
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i)
        fetch(first + i * step, i);
    for (int64_t row = first; row < a.rows; row += step) {
        fetch(row + (kStages - 1) * step, kStages - 1);
        float both[2][U][8], mean[1] = {0.f}, s[3] = {0.f, 0.f, 0.f};
        const T *const rows[2] = {a.x + row * a.xs, a.dy + row * a.dys};
        in.take(rows, a.cols, g.t, g.n, both);
        auto &f = both[0], &d = both[1];
        if (a.center) {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    mean[0] += f[u][i];
            g.sum(mean, 0);
            mean[0] *= inv;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float k[8];
            if (a.w)
                unpack(load_unit<T, VEC>(a.w, a.cols, u, g.t, g.n), k);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (column<VEC>(u, VEC ? 0 : i, g.t, g.n) >= a.cols)
                    continue;
                f[u][i] -= mean[0];
                const float gi = a.w ? d[u][i] * k[i] : d[u][i];
                s[0] = fmaf(f[u][i], f[u][i], s[0]);
                s[1] += gi;
                s[2] = fmaf(gi, f[u][i], s[2]);
            }
        }
        g.sum(s, 1);
        const float r = 1.f / sqrtf(fmaf(s[0], inv, a.eps));
        const float along = s[2] * r * inv, level = a.center ? s[1] * inv : 0.f;
        T *out = a.out + row * a.outs;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float k[8], y[8];
            if (a.w)
                unpack(load_unit<T, VEC>(a.w, a.cols, u, g.t, g.n), k);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float n = f[u][i] * r, gi = a.w ? d[u][i] * k[i] : d[u][i];
                y[i] = r * (fmaf(-n, along, gi) - level);
                dw[u][i] = fmaf(d[u][i], n, dw[u][i]);
                db[u][i] += d[u][i];
            }
            store_unit<T, VEC>(out, a.cols, u, g.t, g.n, y);
        }
    }
    if (!a.partial)
        return;
    float *p = a.partial + (int64_t(blockIdx.x) * groups + g.index) * 2 * a.cols;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = column<VEC>(u, i, g.t, g.n);
            if (c < a.cols) {
                if (a.w)
                    p[c] = dw[u][i];
                if (a.b)
                    p[a.cols + c] = db[u][i];
            }
        }
}

// ---------------------------------------------------------------- rows that do not fit

__device__ float block_sum(float s, float *shared)
{
#pragma unroll
    for (int o = 16; o > 0; o /= 2)
        s += __shfl_xor_sync(kAll, s, o);
    __syncthreads();
    if (threadIdx.x % 32 == 0)
        shared[threadIdx.x / 32] = s;
    __syncthreads();
    s = shared[0];
    for (int w = 1; w < int(blockDim.x / 32); ++w)
        s += shared[w];
    return s;
}

// A block a row, which is read again for each sum.
template <typename T, bool GRAD>
__global__ void __launch_bounds__(1024) wide_kernel(Args<T> a)
{
    __shared__ float shared[32];
    const float inv = 1.f / float(a.cols);
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T *x = a.x + row * a.xs, *dy = GRAD ? a.dy + row * a.dys : nullptr;
        float mean = 0.f, s0 = 0.f, s1 = 0.f, s2 = 0.f;
        if (a.center) {
            for (int c = threadIdx.x; c < a.cols; c += blockDim.x)
                mean += tide::to_f32(x[c]);
            mean = block_sum(mean, shared) * inv;
        }
        for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
            const float f = tide::to_f32(x[c]) - mean;
            s0 = fmaf(f, f, s0);
            if (GRAD) {
                const float gi = a.w ? tide::to_f32(dy[c]) * tide::to_f32(a.w[c]) : tide::to_f32(dy[c]);
                s1 += gi;
                s2 = fmaf(gi, f, s2);
            }
        }
        const float r = 1.f / sqrtf(fmaf(block_sum(s0, shared), inv, a.eps));
        float along = 0.f, level = 0.f;
        if (GRAD) {
            level = a.center ? block_sum(s1, shared) * inv : 0.f;
            along = block_sum(s2, shared) * r * inv;
        }
        T *out = a.out + row * a.outs;
        float *p = GRAD && a.partial ? a.partial + int64_t(blockIdx.x) * 2 * a.cols : nullptr;
        const bool first = row == blockIdx.x;
        for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
            const float n = (tide::to_f32(x[c]) - mean) * r;
            if (!GRAD) {
                float y = a.w ? n * tide::to_f32(a.w[c]) : n;
                if (a.b)
                    y = a.w ? fmaf(n, tide::to_f32(a.w[c]), tide::to_f32(a.b[c])) : n + tide::to_f32(a.b[c]);
                out[c] = tide::from_f32<T>(y);
                continue;
            }
            const float d = tide::to_f32(dy[c]), gi = a.w ? d * tide::to_f32(a.w[c]) : d;
            out[c] = tide::from_f32<T>(r * (fmaf(-n, along, gi) - level));
            if (p) {  // this thread's columns of this block's share
                p[c] = first ? d * n : fmaf(d, n, p[c]);
                p[a.cols + c] = first ? d : p[a.cols + c] + d;
            }
        }
    }
}

// dw, db [cols] from the groups' shares: 32 columns a block, 32 groups at a time.
template <typename T>
__global__ void __launch_bounds__(1024) weight_grad_kernel(const float *partial, int groups, int cols, T *dw, T *db)
{
    __shared__ float shared[32][33];
    const int c = blockIdx.x * 32 + threadIdx.x % 32, y = threadIdx.x / 32, which = blockIdx.y;
    T *out = which ? db : dw;
    if (!out)
        return;
    float s = 0.f;
    if (c < cols)
#pragma unroll 4
        for (int g = y; g < groups; g += 32)
            s += partial[(int64_t(g) * 2 + which) * cols + c];
    shared[y][threadIdx.x % 32] = s;
    __syncthreads();
    s = shared[threadIdx.x % 32][y];  // a column a warp
#pragma unroll
    for (int o = 16; o > 0; o /= 2)
        s += __shfl_xor_sync(kAll, s, o);
    const int cc = blockIdx.x * 32 + y;
    if (threadIdx.x % 32 == 0 && cc < cols)
        out[cc] = tide::from_f32<T>(s);
}

// ---------------------------------------------------------------- host

size_t elem_bytes(int dtype) { return dtype == TIDE_DTYPE_F32 ? 4 : 2; }

tide_status_t check_desc(const tide_norm_t *n)
{
    if (!n)
        return op_fail(TIDE_ERR_INVALID_ARG, "norm is NULL");
    if (n->rows < 0 || n->rows > tide::kMaxExtent || n->cols < 1 || n->cols > (1 << 24))
        return op_fail(TIDE_ERR_INVALID_ARG, "rows %lld, cols %lld", (long long)n->rows, (long long)n->cols);
    if (n->dtype != TIDE_DTYPE_BF16 && n->dtype != TIDE_DTYPE_F32)
        return op_fail(TIDE_ERR_UNSUPPORTED, "dtype %d", n->dtype);
    if (!(n->eps >= 0.f) || n->eps > 3.0e38f)
        return op_fail(TIDE_ERR_INVALID_ARG, "eps %g", double(n->eps));
    if (!op_aligned(n->weight, elem_bytes(n->dtype)) || !op_aligned(n->bias, elem_bytes(n->dtype)))
        return op_fail(TIDE_ERR_ALIGNMENT, "weight or bias is not aligned to its element size");
    return TIDE_OK;
}

tide_status_t check_rows(const tide_norm_t *n, const void *p, int64_t stride, bool output, const char *name)
{
    if (n->rows == 0)
        return TIDE_OK;
    if (!p)
        return op_fail(TIDE_ERR_INVALID_ARG, "%s is NULL", name);
    if (!op_aligned(p, elem_bytes(n->dtype)))
        return op_fail(TIDE_ERR_ALIGNMENT, "%s is not aligned to its element size", name);
    if (n->rows > 1 && (stride < (output ? n->cols : 0) || !tide::op_extent_ok(n->rows, stride)))
        return op_fail(TIDE_ERR_INVALID_ARG, "%s has stride %lld for %lld columns", name, (long long)stride,
                       (long long)n->cols);
    return TIDE_OK;
}

// How rows are shared out: units a thread, warps a row, rows a block, blocks.
struct Shape {
    bool wide, vec;
    int units, warps, groups, blocks;
};

// A thread has 64 bytes of a row of one tensor, 32 of one of two.
Shape shape_of(const tide_norm_t *n, bool grad, bool vec)
{
    Shape s = {};
    s.vec = vec;
    s.units = (n->dtype == TIDE_DTYPE_F32 ? 2 : 4) / (grad ? 2 : 1);
    s.warps = int((n->cols + 256 * s.units - 1) / (256 * s.units));
    s.wide = s.warps > kMaxWarps;
    if (s.wide)
        s.warps = kMaxWarps;
    s.groups = std::max(1, 8 / s.warps);
    const int threads = s.warps * s.groups * 32;
    const int per_sm = threads <= 256 ? grad ? 2 : 3 : threads <= 320 ? 2 : 1;
    s.blocks = int(std::max<int64_t>(1, std::min<int64_t>((n->rows + s.groups - 1) / s.groups,
                                                          int64_t(std::max(tide::op_sm_count(), 1)) * per_sm)));
    return s;
}

bool rows_aligned(const void *p, int64_t stride, int64_t rows, size_t elem)
{
    return op_aligned(p, 16) && (rows < 2 || stride * int64_t(elem) % 16 == 0);
}

template <typename T>
Args<T> args_of(const tide_norm_t *n, const void *x, int64_t xs, void *out, int64_t outs)
{
    Args<T> a = {};
    a.rows = n->rows, a.cols = int(n->cols), a.center = n->center != 0, a.eps = n->eps;
    a.w = static_cast<const T *>(n->weight), a.b = static_cast<const T *>(n->bias);
    a.x = static_cast<const T *>(x), a.xs = xs, a.out = static_cast<T *>(out), a.outs = outs;
    return a;
}

template <auto KERNEL, typename T>
tide_status_t launch_ring(const Args<T> &a, const Shape &s, int bytes, const char *what, cudaStream_t st)
{
    const int threads = s.warps * s.groups * 32, smem = bytes * kStages * threads;
    const cudaError_t e = tide::op_allow_smem<KERNEL>(200 * 1024);
    if (e != cudaSuccess)
        return op_fail(TIDE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
    KERNEL<<<unsigned(s.blocks), unsigned(threads), smem, st>>>(a, s.warps);
    return tide::op_launched(what);
}

template <typename T, bool GRAD, bool VEC>
tide_status_t launch_shape(const Args<T> &a, const Shape &s, const char *what, cudaStream_t st)
{
    constexpr int U = 8 / int(sizeof(T)) / (GRAD ? 2 : 1), kBytes = VEC ? 64 : 0;
    const int threads = s.warps * s.groups * 32;
    if constexpr (GRAD) {
        return threads <= 256   ? launch_ring<backward_kernel<T, VEC, U, 256, 2>>(a, s, kBytes, what, st)
               : threads <= 320 ? launch_ring<backward_kernel<T, VEC, U, 320, 2>>(a, s, kBytes, what, st)
               : threads <= 512 ? launch_ring<backward_kernel<T, VEC, U, 512, 1>>(a, s, kBytes, what, st)
                                : launch_ring<backward_kernel<T, VEC, U, 1024, 1>>(a, s, kBytes, what, st);
    } else {
        return threads <= 256   ? launch_ring<forward_kernel<T, VEC, U, 256, 3>>(a, s, kBytes, what, st)
               : threads <= 320 ? launch_ring<forward_kernel<T, VEC, U, 320, 2>>(a, s, kBytes, what, st)
               : threads <= 512 ? launch_ring<forward_kernel<T, VEC, U, 512, 1>>(a, s, kBytes, what, st)
                                : launch_ring<forward_kernel<T, VEC, U, 1024, 1>>(a, s, kBytes, what, st);
    }
}

template <typename T, bool GRAD>
tide_status_t launch(const Args<T> &a, const Shape &s, const char *what, cudaStream_t st)
{
    if (s.wide) {
        wide_kernel<T, GRAD><<<unsigned(s.blocks), 1024, 0, st>>>(a);
        return tide::op_launched(what);
    }
    return s.vec ? launch_shape<T, GRAD, true>(a, s, what, st) : launch_shape<T, GRAD, false>(a, s, what, st);
}

template <typename T>
tide_status_t backward(const tide_norm_t *n, const Args<T> &a, const Shape &s, void *dw, void *db, cudaStream_t st)
{
    if (n->rows)
        if (const tide_status_t e = launch<T, true>(a, s, "layer_norm_grad", st))
            return e;
    if (!dw && !db)
        return TIDE_OK;
    weight_grad_kernel<T><<<dim3(unsigned((n->cols + 31) / 32), 2), 1024, 0, st>>>(
        a.partial, n->rows ? s.blocks * (s.wide ? 1 : s.groups) : 0, a.cols, static_cast<T *>(dw), static_cast<T *>(db));
    return tide::op_launched("layer_norm_grad: weight");
}

}  // namespace

extern "C" {

tide_status_t tide_layer_norm(const tide_norm_t *norm, const void *x, int64_t x_stride, void *y, int64_t y_stride,
                              void *stream)
{
    tide::record_error("");
    tide_status_t s = check_desc(norm);
    if (!s)
        s = check_rows(norm, x, x_stride, false, "x");
    if (!s)
        s = check_rows(norm, y, y_stride, true, "y");
    if (s || norm->rows == 0)
        return s;
    const tide::NvtxRange range("tide_layer_norm");
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const size_t e = elem_bytes(norm->dtype);
    const bool vec = norm->cols % 8 == 0 && rows_aligned(x, x_stride, norm->rows, e) &&
                     rows_aligned(y, y_stride, norm->rows, e) && op_aligned(norm->weight, 16) && op_aligned(norm->bias, 16);
    const Shape shape = shape_of(norm, false, vec);
    if (norm->dtype == TIDE_DTYPE_F32)
        return launch<float, false>(args_of<float>(norm, x, x_stride, y, y_stride), shape, "layer_norm", st);
    return launch<bf16, false>(args_of<bf16>(norm, x, x_stride, y, y_stride), shape, "layer_norm", st);
}

int64_t tide_layer_norm_grad_workspace(const tide_norm_t *norm)
{
    tide::record_error("");
    if (check_desc(norm))
        return -1;
    if (!norm->weight && !norm->bias)
        return 0;
    const Shape s = shape_of(norm, true, false);
    return std::max<int64_t>(256, int64_t(s.blocks) * s.groups * 2 * norm->cols * 4);
}

tide_status_t tide_layer_norm_grad(const tide_norm_t *norm, const void *dy, int64_t dy_stride, const void *x,
                                   int64_t x_stride, void *dx, int64_t dx_stride, void *dweight, void *dbias,
                                   void *workspace, int64_t workspace_bytes, void *stream)
{
    tide::record_error("");
    tide_status_t s = check_desc(norm);
    if (!s)
        s = check_rows(norm, dy, dy_stride, false, "dy");
    if (!s)
        s = check_rows(norm, x, x_stride, false, "x");
    if (!s)
        s = check_rows(norm, dx, dx_stride, true, "dx");
    if (s)
        return s;
    if (!norm->weight != !dweight || !norm->bias != !dbias)
        return op_fail(TIDE_ERR_INVALID_ARG, "a gradient goes with its weight or bias: both or neither");
    const size_t e = elem_bytes(norm->dtype);
    if (!op_aligned(dweight, e) || !op_aligned(dbias, e))
        return op_fail(TIDE_ERR_ALIGNMENT, "dweight or dbias is not aligned to its element size");
    const int64_t need = tide_layer_norm_grad_workspace(norm);
    if (workspace_bytes < need || (need && !workspace))
        return op_fail(TIDE_ERR_INVALID_ARG, "workspace of %lld bytes: need %lld", (long long)workspace_bytes,
                       (long long)need);
    if (!op_aligned(workspace, 256))
        return op_fail(TIDE_ERR_ALIGNMENT, "workspace is not 256-byte aligned");
    const tide::NvtxRange range("tide_layer_norm_grad");
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int64_t T = norm->rows;
    const bool vec = norm->cols % 8 == 0 && rows_aligned(x, x_stride, T, e) && rows_aligned(dy, dy_stride, T, e) &&
                     rows_aligned(dx, dx_stride, T, e) && op_aligned(norm->weight, 16);
    const Shape shape = shape_of(norm, true, vec);
    float *partial = need ? static_cast<float *>(workspace) : nullptr;
    if (norm->dtype == TIDE_DTYPE_F32) {
        Args<float> a = args_of<float>(norm, x, x_stride, dx, dx_stride);
        a.dy = static_cast<const float *>(dy), a.dys = dy_stride, a.partial = partial;
        return backward(norm, a, shape, dweight, dbias, st);
    }
    Args<bf16> a = args_of<bf16>(norm, x, x_stride, dx, dx_stride);
    a.dy = static_cast<const bf16 *>(dy), a.dys = dy_stride, a.partial = partial;
    return backward(norm, a, shape, dweight, dbias, st);
}

}  // extern "C"
