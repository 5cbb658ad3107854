// Helpers shared by the training-step operators: argument errors, launch
// checks and element types.  Not part of the C ABI.
#pragma once

#include <cuda_bf16.h>

#include <cstdarg>
#include <cstdio>

#include "tide_internal.h"

namespace tide {

// Record the detail that tide_last_error() reports and return the status.
__attribute__((format(printf, 2, 3))) inline tide_status_t op_fail(tide_status_t st, const char *fmt, ...)
{
    char buf[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    record_error(buf);
    return st;
}

// Status of the launch that was just made, counted if it was accepted.
inline tide_status_t op_launched(const char *what)
{
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return op_fail(TIDE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
    g_launches.fetch_add(1);
    return TIDE_OK;
}

inline bool op_aligned(const void *p, size_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

// SM count of the current device (looked up once per device).
inline int op_sm_count()
{
    static std::atomic<int> known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
        return 0;
    int n = known[dev].load(std::memory_order_relaxed);
    if (!n && cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess)
        known[dev].store(n, std::memory_order_relaxed);
    return n;
}

// Lets a kernel have `bytes` of dynamic shared memory; asked for once on each device.
template <auto KERNEL>
cudaError_t op_allow_smem(int bytes)
{
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && done.load(std::memory_order_relaxed) >> dev & 1))
        return e;
    e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64)
        done.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
    return e;
}

// Sizes are kept below 2^60 elements so that byte offsets fit 64 bits.
constexpr int64_t kMaxExtent = int64_t(1) << 60;
inline bool op_extent_ok(int64_t n, int64_t stride)
{
    return stride <= kMaxExtent && (n <= 1 || stride <= kMaxExtent / n);
}

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// Eight consecutive elements as fp32; `p` is 16-byte aligned.
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float *f)
{
    const uint4 v = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void load8(const float *p, float *f)
{
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
    f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float *f)
{
    *reinterpret_cast<uint4 *>(p) =
        make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}
__device__ __forceinline__ void store8(float *p, const float *f)
{
    reinterpret_cast<float4 *>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}

// Rows that do not start on 16-byte boundaries, by whole aligned pieces.

// Bytes `phase` (0 to 15) to phase + 15 of 32.
__device__ __forceinline__ void shift_bytes(const uint32_t (&w)[8], uint32_t phase, uint32_t (&out)[4])
{
    uint32_t a[6], b[5];
#pragma unroll
    for (int i = 0; i < 6; ++i)
        a[i] = phase & 8 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i)
        b[i] = phase & 4 ? a[i + 1] : a[i];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        out[i] = __funnelshift_r(b[i], b[i + 1], 8 * (phase & 3));
}

// The 16 bytes at `p`, of which those before `end` count (at least one; the rest
// is whatever lies there or 0): read as the aligned 16-byte pieces that hold a
// byte that counts, so that nothing is touched that shares no piece with one.
__device__ __forceinline__ void load16_any(const void *p, const void *end, uint32_t (&out)[4])
{
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    const uint32_t phase = uint32_t(at & 15);
    const uint4 *q = reinterpret_cast<const uint4 *>(at - phase);
    const uint4 x = q[0];
    uint4 y = make_uint4(0, 0, 0, 0);
    if (phase && reinterpret_cast<uintptr_t>(q + 1) < reinterpret_cast<uintptr_t>(end))
        y = q[1];
    const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    shift_bytes(w, phase, out);
}

}  // namespace tide
