// SwiGLU that keeps gate and up in 8 bits for the backward pass, and its
// gradient from the 8-bit values.
//
//   forward:  h = g s u, s = 1 / (1 + exp(-g));
//             for each 128 columns of a row: e with amax 2^(127 - e) <= 448,
//             smallest; code = e4m3(x 2^(127 - e))
//   backward: dg = dh u s (1 + g (1 - s)),  du = dh g s,  h = g s u.
//
// The scale is a power of two, so scaling is exact and the code is one
// rounding to nearest even of the value.  e4m3 rather than int8: a block may
// hold values a hundred times its others, which a common integer step would
// round to zero.
//
// Both are bound by memory (bf16: 8 bytes an element forward, 10 backward); the
// forward has some 25 instructions an element to hide under it, so it works on
// pairs of values where it can.  Sixteen lanes take one block, eight elements
// each, so a block's maximum is four exchanges and every load and store is a
// whole vector; a warp takes two neighbouring blocks of a row and steps down
// the rows, with the next row's loads on their way.  Rows that are not on
// 16-byte boundaries, or whose length is not a multiple of 8, take the same
// kernel with single elements, 16 columns apart in a lane.
//
// Measured (bf16, 16384 x 14336): forward 295 us, 6.4 TB/s, 96% of the copy
// rate (386 us with a warp a block pair and 64-bit divisions for each, where
// 78% of the issue slots were busy); gradient 354 us, 6.6 TB/s, 99.5%.  fp32
// rows of 1003 columns: 5.9 us for 1001 (17 us with 8 neighbouring elements a
// lane, whose loads did not coalesce).
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>

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
constexpr int kBlock = TIDE_CKPT8_BLOCK;
constexpr int kWarpsPerSm = 64;
constexpr uint32_t kInfBits = 0x7f800000u;

// 1 / (1 + exp(-g)) from exp(-|g|), so that nothing overflows and small
// results keep their precision.  bf16 takes the fast exponential and reciprocal
// (about 2^-22), far below its rounding; the exponential is made 2^24 too large
// and scaled back, which keeps results under 2^-126 without the instruction's
// own scaling.
template <typename T>
__device__ __forceinline__ float sigmoid(float g)
{
    if constexpr (sizeof(T) == 2) {
        float e, r;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(__fmaf_rn(fabsf(g), -1.4426950408889634f, 24.f)));
        e *= 5.9604644775390625e-8f;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
        return (g < 0.f ? e : 1.f) * r;
    } else {
        const float e = expf(-fabsf(g));
        return (g < 0.f ? e : 1.f) / (1.f + e);
    }
}

// A lane's eight elements of a block as they lie in memory.  VEC: columns c to
// c + 7; otherwise c, c + 16, ..., c + 112.  Columns from `cols` on read as 0.
template <bool VEC, typename T>
struct Eight {
    float f[8];
    __device__ __forceinline__ void load(const T *row, int64_t c, int64_t cols)
    {
        if constexpr (VEC) {
            if (c < cols) {
                load8(row + c, f);
                return;
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = !VEC && c + 16 * i < cols ? to_f32(row[c + 16 * i]) : 0.f;
    }
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = f[i];
    }
    // Largest magnitude as bits; infinities and NaN are above all others.
    __device__ __forceinline__ uint32_t top() const
    {
        uint32_t t = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            t = max(t, __float_as_uint(f[i]) & 0x7fffffffu);
        return t;
    }
};
template <>
struct Eight<true, __nv_bfloat16> {  // packed until they are needed
    uint4 w;
    __device__ __forceinline__ void load(const __nv_bfloat16 *row, int64_t c, int64_t cols)
    {
        w = c < cols ? *reinterpret_cast<const uint4 *>(row + c) : make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(x[i] << 16);
            v[2 * i + 1] = __uint_as_float(x[i] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ uint32_t top() const
    {
        auto mag = [](uint32_t x) {
            x &= 0x7fff7fffu;
            return *reinterpret_cast<const __nv_bfloat162 *>(&x);
        };
        const __nv_bfloat162 t =
            __hmax2_nan(__hmax2_nan(mag(w.x), mag(w.y)), __hmax2_nan(mag(w.z), mag(w.w)));
        const uint32_t b = *reinterpret_cast<const uint32_t *>(&t);
        return max(b << 16, b & 0xffff0000u);
    }
};

template <bool VEC, typename T>
__device__ __forceinline__ void store_cols(T *row, int64_t c, int64_t cols, const float (&v)[8])
{
    if constexpr (VEC) {
        if (c < cols)
            store8(row + c, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + 16 * i < cols)
                row[c + 16 * i] = from_f32<T>(v[i]);
    }
}
template <bool VEC>
__device__ __forceinline__ uint2 load_codes(const uint8_t *row, int64_t c, int64_t cols)
{
    uint32_t w[2] = {0, 0};
    if constexpr (VEC) {
        if (c < cols)
            return *reinterpret_cast<const uint2 *>(row + c);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + 16 * i < cols)
                w[i / 4] |= uint32_t(row[c + 16 * i]) << (8 * (i % 4));
    }
    return make_uint2(w[0], w[1]);
}
template <bool VEC>
__device__ __forceinline__ void store_codes(uint8_t *row, int64_t c, int64_t cols, uint2 q)
{
    if constexpr (VEC) {
        if (c < cols)
            *reinterpret_cast<uint2 *>(row + c) = q;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + 16 * i < cols)
                row[c + 16 * i] = uint8_t((i < 4 ? q.x : q.y) >> (8 * (i % 4)));
    }
}

__device__ __forceinline__ uint32_t block_max(uint32_t x)
{
#pragma unroll
    for (int o = 8; o > 0; o /= 2)
        x = max(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

// Codes of a lane's eight values and the exponent of their block (16 lanes),
// whose largest magnitude is `top`.
__device__ __forceinline__ uint2 encode(float (&v)[8], uint32_t top, int &exponent)
{
    if (__any_sync(0xffffffffu, top >= kInfBits)) {  // infinities or NaN: they do not count, and become NaN
        uint32_t t = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t b = __float_as_uint(v[i]) & 0x7fffffffu;
            t = max(t, b < kInfBits ? b : 0u);
            if (b >= kInfBits)
                v[i] = __int_as_float(0x7fffffff);
        }
        top = block_max(t);
    }
    // amax = f 2^(E - 127), 1 <= f < 2, and 448 = 1.75 2^8: e - 127 = E - 127 - 8, one more if f > 1.75.
    // Subnormal amax has E = 0 and ends at the smallest exponent either way.
    const int e = top == 0 ? 127 : max(int((top + 0x1fffffu) >> 23) - 8, 1);
    exponent = e;
    const float scale = __uint_as_float(uint32_t(254 - e) << 23);  // 2^(127 - e), e in [1, 247]
    uint32_t w[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        uint16_t lo, hi;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(v[4 * k + 1] * scale), "f"(v[4 * k] * scale));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(v[4 * k + 3] * scale), "f"(v[4 * k + 2] * scale));
        w[k] = uint32_t(hi) << 16 | lo;
    }
    return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void decode(uint2 q, int exponent, float (&v)[8])
{
    const float scale = __uint_as_float(uint32_t(exponent) << 23);  // exponents are >= 1
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w = (i < 2 ? q.x : q.y) >> (16 * (i % 2));
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(w & 0xffffu), __NV_E4M3);
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
        v[2 * i] = f.x * scale;
        v[2 * i + 1] = f.y * scale;
    }
}

template <typename T>
struct SwigluArgs {
    int64_t rows, cols;
    int64_t row_step;   // rows from one of a warp to its next
    int blocks, pairs;  // blocks of a row, and pairs of blocks
    const T *gate, *up, *dh;
    int64_t gate_stride, up_stride, dh_stride;
    T *h, *dgate, *dup;
    int64_t h_stride, dgate_stride, dup_stride;
    uint8_t *g8, *ge, *u8, *ue;
};

// A lane's place: its warp's first row, its block and its first column.
struct Place {
    int64_t row;
    int block;
    int64_t c;
};
template <bool VEC, typename T>
__device__ __forceinline__ Place place_of(const SwigluArgs<T> &a)
{
    const int lane = threadIdx.x & 31;
    const int64_t warp = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    Place p;
    p.row = warp / a.pairs;
    p.block = 2 * int(warp - p.row * a.pairs) + lane / 16;
    p.c = int64_t(p.block) * kBlock + (VEC ? 8 : 1) * (lane % 16);
    return p;
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) swiglu_forward_kernel(const SwigluArgs<T> a)
{
    const Place p = place_of<VEC>(a);
    if (p.row >= a.row_step)
        return;
    const bool writes = threadIdx.x % 16 == 0 && p.block < a.blocks;
    Eight<VEC, T> gate, up;
    gate.load(a.gate + p.row * a.gate_stride, p.c, a.cols);
    up.load(a.up + p.row * a.up_stride, p.c, a.cols);
    for (int64_t row = p.row; row < a.rows; row += a.row_step) {
        float g[8], u[8], h[8];
        gate.get(g);
        up.get(u);
        const uint32_t tg = block_max(gate.top()), tu = block_max(up.top());
        const int64_t next = row + a.row_step;
        if (next < a.rows) {
            gate.load(a.gate + next * a.gate_stride, p.c, a.cols);
            up.load(a.up + next * a.up_stride, p.c, a.cols);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            h[i] = g[i] * sigmoid<T>(g[i]) * u[i];
        store_cols<VEC>(a.h + row * a.h_stride, p.c, a.cols, h);
        int eg, eu;
        const uint2 qg = encode(g, tg, eg), qu = encode(u, tu, eu);
        store_codes<VEC>(a.g8 + row * a.cols, p.c, a.cols, qg);
        store_codes<VEC>(a.u8 + row * a.cols, p.c, a.cols, qu);
        if (writes) {
            a.ge[row * a.blocks + p.block] = uint8_t(eg);
            a.ue[row * a.blocks + p.block] = uint8_t(eu);
        }
    }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) swiglu_backward_kernel(const SwigluArgs<T> a)
{
    const Place p = place_of<VEC>(a);
    if (p.row >= a.row_step || p.block >= a.blocks)
        return;
    Eight<VEC, T> dh;
    uint2 qg, qu;
    int eg, eu;
    auto load = [&](int64_t row) {
        qg = load_codes<VEC>(a.g8 + row * a.cols, p.c, a.cols);
        qu = load_codes<VEC>(a.u8 + row * a.cols, p.c, a.cols);
        dh.load(a.dh + row * a.dh_stride, p.c, a.cols);
        eg = a.ge[row * a.blocks + p.block];
        eu = a.ue[row * a.blocks + p.block];
    };
    load(p.row);
    for (int64_t row = p.row; row < a.rows; row += a.row_step) {
        float g[8], u[8], d[8], x[8], s[8];
        dh.get(d);
        decode(qg, eg, g);
        decode(qu, eu, u);
        if (row + a.row_step < a.rows)
            load(row + a.row_step);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            s[i] = sigmoid<T>(g[i]);
            x[i] = d[i] * u[i] * s[i] * __fmaf_rn(g[i], 1.f - s[i], 1.f);
        }
        store_cols<VEC>(a.dgate + row * a.dgate_stride, p.c, a.cols, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            s[i] *= g[i];
            x[i] = d[i] * s[i];
        }
        store_cols<VEC>(a.dup + row * a.dup_stride, p.c, a.cols, x);
        if (!a.h)
            continue;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = s[i] * u[i];
        store_cols<VEC>(a.h + row * a.h_stride, p.c, a.cols, x);
    }
}

size_t elem_bytes(int dtype) { return dtype == TIDE_DTYPE_F32 ? 4 : 2; }

tide_status_t check_shape(int64_t rows, int64_t cols, int32_t dtype, const tide_ckpt8_t *ckpt)
{
    if (dtype != TIDE_DTYPE_BF16 && dtype != TIDE_DTYPE_F32)
        return op_fail(TIDE_ERR_UNSUPPORTED, "dtype %d is not implemented", dtype);
    if (rows < 0 || cols < 0 || !tide::op_extent_ok(rows, cols) || !tide::op_extent_ok(cols, 1))
        return op_fail(TIDE_ERR_INVALID_ARG, "rows %lld, cols %lld", (long long)rows, (long long)cols);
    if (rows > 0 && cols > 0) {
        const int64_t pairs = (cols + 2 * kBlock - 1) / (2 * kBlock);
        if (pairs > 0x3fffffff || pairs > int64_t(0x7fffffff) * kWarps / rows)
            return op_fail(TIDE_ERR_INVALID_ARG, "rows %lld x cols %lld is over one launch", (long long)rows,
                           (long long)cols);
        if (!ckpt || !ckpt->gate_codes || !ckpt->gate_exps || !ckpt->up_codes || !ckpt->up_exps)
            return op_fail(TIDE_ERR_INVALID_ARG, "a checkpoint pointer is NULL");
    }
    return TIDE_OK;
}

tide_status_t check_rows(const void *p, int64_t stride, int64_t rows, int64_t cols, int32_t dtype, bool output,
                         const char *name)
{
    if (rows == 0 || cols == 0)
        return TIDE_OK;
    if (!p)
        return op_fail(TIDE_ERR_INVALID_ARG, "%s is NULL", name);
    if (!op_aligned(p, elem_bytes(dtype)))
        return op_fail(TIDE_ERR_ALIGNMENT, "%s is not aligned to its element size", name);
    if (stride < 0 || !tide::op_extent_ok(rows, stride) || (output && rows > 1 && stride < cols))
        return op_fail(TIDE_ERR_INVALID_ARG, "%s has row stride %lld for %lld columns", name, (long long)stride,
                       (long long)cols);
    return TIDE_OK;
}

bool vec_rows(const void *p, int64_t stride, int64_t rows, int32_t dtype)
{
    return op_aligned(p, 16) && (rows < 2 || stride % (16 / int64_t(elem_bytes(dtype))) == 0);
}
bool vec_ckpt(const tide_ckpt8_t *k, int64_t cols)
{
    return cols % 8 == 0 && op_aligned(k->gate_codes, 8) && op_aligned(k->up_codes, 8);
}

template <typename T>
SwigluArgs<T> make_args(int64_t rows, int64_t cols, const tide_ckpt8_t *k)
{
    SwigluArgs<T> a = {};
    a.rows = rows;
    a.cols = cols;
    a.blocks = int((cols + kBlock - 1) / kBlock);
    a.pairs = (a.blocks + 1) / 2;
    // As many warps as the SMs hold, and some more to even out their ends.
    const int64_t warps = int64_t(std::max(tide::op_sm_count(), 1)) * kWarpsPerSm;
    a.row_step = std::min(rows, std::max<int64_t>(1, warps / a.pairs));
    a.g8 = static_cast<uint8_t *>(k->gate_codes);
    a.ge = static_cast<uint8_t *>(k->gate_exps);
    a.u8 = static_cast<uint8_t *>(k->up_codes);
    a.ue = static_cast<uint8_t *>(k->up_exps);
    return a;
}

template <typename T>
tide_status_t forward(int64_t rows, int64_t cols, bool vec, const void *gate, int64_t gs, const void *up, int64_t us,
                      void *h, int64_t hs, const tide_ckpt8_t *k, cudaStream_t st)
{
    SwigluArgs<T> a = make_args<T>(rows, cols, k);
    a.gate = static_cast<const T *>(gate), a.gate_stride = gs;
    a.up = static_cast<const T *>(up), a.up_stride = us;
    a.h = static_cast<T *>(h), a.h_stride = hs;
    const unsigned grid = unsigned((a.row_step * a.pairs + kWarps - 1) / kWarps);
    if (vec)
        swiglu_forward_kernel<T, true><<<grid, kThreads, 0, st>>>(a);
    else
        swiglu_forward_kernel<T, false><<<grid, kThreads, 0, st>>>(a);
    return tide::op_launched("swiglu_ckpt8");
}

template <typename T>
tide_status_t backward(int64_t rows, int64_t cols, bool vec, const tide_ckpt8_t *k, const void *dh, int64_t ds,
                       void *dgate, int64_t gs, void *dup, int64_t us, void *h, int64_t hs, cudaStream_t st)
{
    SwigluArgs<T> a = make_args<T>(rows, cols, k);
    a.dh = static_cast<const T *>(dh), a.dh_stride = ds;
    a.dgate = static_cast<T *>(dgate), a.dgate_stride = gs;
    a.dup = static_cast<T *>(dup), a.dup_stride = us;
    a.h = static_cast<T *>(h), a.h_stride = hs;
    const unsigned grid = unsigned((a.row_step * a.pairs + kWarps - 1) / kWarps);
    if (vec)
        swiglu_backward_kernel<T, true><<<grid, kThreads, 0, st>>>(a);
    else
        swiglu_backward_kernel<T, false><<<grid, kThreads, 0, st>>>(a);
    return tide::op_launched("swiglu_ckpt8_grad");
}

}  // namespace

extern "C" {

tide_status_t tide_swiglu_ckpt8(int64_t rows, int64_t cols, int32_t dtype, const void *gate, int64_t gate_stride,
                                const void *up, int64_t up_stride, void *h, int64_t h_stride,
                                const tide_ckpt8_t *ckpt, void *stream)
{
    tide::record_error("");
    tide_status_t s = check_shape(rows, cols, dtype, ckpt);
    if (!s)
        s = check_rows(gate, gate_stride, rows, cols, dtype, false, "gate");
    if (!s)
        s = check_rows(up, up_stride, rows, cols, dtype, false, "up");
    if (!s)
        s = check_rows(h, h_stride, rows, cols, dtype, true, "h");
    if (s || rows == 0 || cols == 0)
        return s;
    const tide::NvtxRange range("tide_swiglu_ckpt8");
    const bool vec = vec_ckpt(ckpt, cols) && vec_rows(gate, gate_stride, rows, dtype) &&
                     vec_rows(up, up_stride, rows, dtype) && vec_rows(h, h_stride, rows, dtype);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dtype == TIDE_DTYPE_F32)
        return forward<float>(rows, cols, vec, gate, gate_stride, up, up_stride, h, h_stride, ckpt, st);
    return forward<__nv_bfloat16>(rows, cols, vec, gate, gate_stride, up, up_stride, h, h_stride, ckpt, st);
}

tide_status_t tide_swiglu_ckpt8_grad(int64_t rows, int64_t cols, int32_t dtype, const tide_ckpt8_t *ckpt,
                                     const void *dh, int64_t dh_stride, void *dgate, int64_t dgate_stride, void *dup,
                                     int64_t dup_stride, void *h, int64_t h_stride, void *stream)
{
    tide::record_error("");
    tide_status_t s = check_shape(rows, cols, dtype, ckpt);
    if (!s)
        s = check_rows(dh, dh_stride, rows, cols, dtype, false, "dh");
    if (!s)
        s = check_rows(dgate, dgate_stride, rows, cols, dtype, true, "dgate");
    if (!s)
        s = check_rows(dup, dup_stride, rows, cols, dtype, true, "dup");
    if (!s && h)
        s = check_rows(h, h_stride, rows, cols, dtype, true, "h");
    if (s || rows == 0 || cols == 0)
        return s;
    const tide::NvtxRange range("tide_swiglu_ckpt8_grad");
    const bool vec = vec_ckpt(ckpt, cols) && vec_rows(dh, dh_stride, rows, dtype) &&
                     vec_rows(dgate, dgate_stride, rows, dtype) && vec_rows(dup, dup_stride, rows, dtype) &&
                     (!h || vec_rows(h, h_stride, rows, dtype));
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dtype == TIDE_DTYPE_F32)
        return backward<float>(rows, cols, vec, ckpt, dh, dh_stride, dgate, dgate_stride, dup, dup_stride, h, h_stride,
                               st);
    return backward<__nv_bfloat16>(rows, cols, vec, ckpt, dh, dh_stride, dgate, dgate_stride, dup, dup_stride, h,
                                   h_stride, st);
}

}  // extern "C"
