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
// are butterflies over G = 4 to 32 lanes.  A warp takes 32 / G heads of one
// token at a time (a step).  Persistent warps copy their next three (or two) steps
// into shared memory (cp.async, every lane its own vectors, so nothing waits
// for another warp), which keeps enough bytes on their way from few warps with
// many registers; a token's angles come along with its first step.  Products
// run on pairs of fp32 (f32x2), with the weight folded into the cosines and
// sines once a token: three instructions a pair.
//
// Measured (bf16, 32768 tokens of 32 + 4 heads of 128): forward 104 us, 5.8 TB/s,
// 88% of the copy rate, with 60% of the issue slots busy; gradient 139.5 us with
// its weights, 6.5 TB/s, 98%.  Loads straight into registers, a warp a token,
// took 213 and 268 us: at 96 to 127 registers too few warps wait at a time.
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
    int heads_per_item;  // forward: queries, then keys
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

template <int G>
__device__ __forceinline__ float group_sum(float x)
{
#pragma unroll
    for (int o = G / 2; o > 0; o /= 2)
        x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Two fp32 values in one 64-bit register pair.
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pair(float lo, float hi)
{
    return f32x2(__float_as_uint(hi)) << 32 | __float_as_uint(lo);
}
__device__ __forceinline__ float lo_of(f32x2 x) { return __uint_as_float(uint32_t(x)); }
__device__ __forceinline__ float hi_of(f32x2 x) { return __uint_as_float(uint32_t(x >> 32)); }
__device__ __forceinline__ f32x2 swapped(f32x2 x) { return x >> 32 | x << 32; }
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b)
{
    f32x2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c)
{
    f32x2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// Steps of a warp's ring: four, or three where four would leave a SM one block
// instead of two (fp32 gradients, 18 KB a warp: 1003 tokens of 7 + 3 heads of 96
// 14.3 us with four, 12.3 with three).
template <typename T>
__host__ __device__ constexpr int depth_of(int tensors)
{
    return sizeof(T) * tensors > 4 ? 3 : 4;
}

__device__ __forceinline__ void copy16(void *dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(uint32_t(__cvta_generic_to_shared(dst))), "l"(src)
                 : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Sixteen elements of a unit as pairs.
__device__ __forceinline__ void unpack8(const uint4 *q, int stride, f32x2 *v, const __nv_bfloat16 *)
{
    const uint4 x = q[0];
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
__device__ __forceinline__ void unpack8(const uint4 *q, int stride, f32x2 *v, const float *)
{
    const uint4 x = q[0], y = q[stride];
    v[0] = f32x2(x.y) << 32 | x.x, v[1] = f32x2(x.w) << 32 | x.z;
    v[2] = f32x2(y.y) << 32 | y.x, v[3] = f32x2(y.w) << 32 | y.z;
}
template <typename T>
__device__ __forceinline__ void store_unit(T *row, const Unit &n, const f32x2 (&v)[8])
{
    float f[16];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        f[2 * i] = lo_of(v[i]), f[2 * i + 1] = hi_of(v[i]);
    if (n.has0)
        store8(row + n.off0, f);
    if (n.has1)
        store8(row + n.off1, f + 8);
}
// A weight's elements of a unit (0 outside the head).
template <typename T>
__device__ __forceinline__ void load_weight(const T *w, const Unit &n, f32x2 (&v)[8])
{
    float f[16];
#pragma unroll
    for (int i = 0; i < 16; ++i)
        f[i] = 0.f;
    if (n.has0)
        load8(w + n.off0, f);
    if (n.has1)
        load8(w + n.off1, f + 8);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = pair(f[2 * i], f[2 * i + 1]);
}

// The other member of each element's rotation pair.
template <bool IL>
__device__ __forceinline__ f32x2 partner(const f32x2 (&v)[8], int i)
{
    return IL ? swapped(v[i]) : v[i ^ 4];
}

// A warp's list of items (a token, or some of its heads): every `step`-th from
// `first`, `count` in all.  Lane j holds the table row of the j-th item of 32,
// and of the 32 after them, so that no item waits for its position.
template <typename T>
struct Items {
    int64_t first, step;
    int count, chunks, per_item, heads;
    int now, next, block;
    __device__ int position(const QkArgs<T> &a, int n) const
    {
        return a.R && n < count ? int(position_of(a, (first + n * step) / chunks)) : -1;
    }
    __device__ void start(const QkArgs<T> &a, int64_t first_, int64_t step_, int heads_, int per_item_)
    {
        first = first_, step = step_, heads = heads_, per_item = per_item_;
        chunks = (heads + per_item - 1) / per_item;
        const int64_t items = a.tokens * chunks;
        count = first < items ? int((items - first + step - 1) / step) : 0;
        block = 0;
        now = position(a, threadIdx.x & 31);
        next = position(a, (threadIdx.x & 31) + 32);
    }
    // Row of the table for the n-th item (-1: outside); n grows by at most one from call to call.
    __device__ int row(const QkArgs<T> &a, int n)
    {
        if (n / 32 != block) {
            block = n / 32;
            now = next;
            next = position(a, (block + 1) * 32 + (threadIdx.x & 31));
        }
        return __shfl_sync(0xffffffffu, now, n % 32);
    }
    // Token, first head and end of the n-th item.
    __device__ int64_t enter(int n, int &h0, int &h1) const
    {
        int64_t t = first + n * step;
        h0 = 0;
        if (chunks > 1) {
            const int64_t item = t;
            t = item / chunks;
            h0 = int(item - t * chunks) * per_item;
        }
        h1 = min(heads, h0 + per_item);
        return t;
    }
};

// Cosines and sines of a unit's pairs out of a token's row in shared memory,
// as factors of an element and of its partner; back: of the reverse rotation.
template <bool IL, bool BACK>
__device__ __forceinline__ void angle_factors(const float *row, int R, const Unit &n, bool bad, f32x2 (&c2)[8],
                                              f32x2 (&s2)[8])
{
    float c[8], s[8];
    if (n.rot) {
        load8(row + n.ci, c);
        load8(row + R / 2 + n.ci, s);
    }
    if (bad) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            c[j] = s[j] = __int_as_float(0x7fffffff);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (IL) {
            c2[i] = pair(c[i], c[i]);
            s2[i] = BACK ? pair(s[i], -s[i]) : pair(-s[i], s[i]);
        } else {
            const int j = 2 * (i & 3);
            c2[i] = pair(c[j], c[j + 1]);
            s2[i] = (i < 4) == BACK ? pair(s[j], s[j + 1]) : pair(-s[j], -s[j + 1]);
        }
    }
}

template <int G>
__device__ __forceinline__ float inv_rms(const f32x2 (&v)[8], float inv_d, float eps)
{
    f32x2 ss = mul2(v[0], v[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i)
        ss = fma2(v[i], v[i], ss);
    return rsqrtf(__fmaf_rn(group_sum<G>(lo_of(ss) + hi_of(ss)), inv_d, eps));
}

// Bytes of a warp's ring: steps of `tensors` tensors, and as many rows of angles.
template <typename T>
__host__ __device__ constexpr int ring_bytes(int tensors, int G)
{
    return depth_of<T>(tensors) * (tensors * 2 * int(sizeof(T)) / 2 * 512 + G * 64);
}

// Pieces that a lane's unit does not have read as 0 out of every slot.
__device__ __forceinline__ void clear_missing(uint4 *ring, int lane, int pieces, int per_vector, const Unit &n)
{
    for (int i = 0; i < pieces; ++i)
        if (!(i / per_vector % 2 ? n.has1 : n.has0))
            ring[i * 32 + lane] = make_uint4(0, 0, 0, 0);
}

template <typename T, int G, bool IL>
__global__ void __launch_bounds__(kThreads, 2) qk_forward_kernel(const QkArgs<T> a)
{
    constexpr int kRows = 32 / G;       // heads of a step
    constexpr int kVec = sizeof(T) / 2; // 16-byte pieces of eight elements
    constexpr int kSlot = 2 * kVec * 32, kDepth = depth_of<T>(1);
    extern __shared__ uint4 smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane / G;
    uint4 *ring = smem + warp * (ring_bytes<T>(1, G) / 16);
    float *angles = reinterpret_cast<float *>(ring + kDepth * kSlot);
    ring += lane;
    const Unit n = unit_of<IL>(lane % G, a.D, a.R);
    const float inv_d = 1.f / float(a.D);
    const int hq = a.part[0].heads;
    Items<T> items;
    items.start(a, int64_t(blockIdx.x) * kWarps + warp, int64_t(gridDim.x) * kWarps, hq + a.part[1].heads,
                a.heads_per_item);
    clear_missing(ring - lane, lane, kDepth * 2 * kVec, kVec, n);

    // The next step to fetch: its item, first head, the lane's row.
    int fn = 0, fh = 0, fh1 = 0, slot_f = 0;
    int64_t ft = 0, fd = 0;
    const T *fp = nullptr;
    uint32_t bad_bits = 0;  // bit n % 32: the n-th item's position is outside the table
    auto aim = [&](int h) {
        const Part<T> &p = a.part[h >= hq];
        fp = p.x.row(ft, h >= hq ? h - hq : h);
        fd = kRows * p.x.sh;
    };
    auto next_item = [&] {
        if (fn < items.count) {
            ft = items.enter(fn, fh, fh1);
            aim(fh + g);
        }
    };
    bool fresh = true;
    auto fetch = [&] {
        if (fn < items.count) {
            const int h = fh + g;
            if (h < fh1) {
                uint4 *to = ring + slot_f * kSlot;
#pragma unroll
                for (int k = 0; k < kVec; ++k) {
                    if (n.has0)
                        copy16(to + k * 32, fp + n.off0 + k * 4);
                    if (n.has1)
                        copy16(to + (kVec + k) * 32, fp + n.off1 + k * 4);
                }
            }
            if (fresh && a.R) {
                const int pos = items.row(a, fn);
                const uint32_t bit = 1u << (fn % 32);
                bad_bits = pos < 0 ? bad_bits | bit : bad_bits & ~bit;
                if (pos >= 0) {
                    const float *row = a.table + int64_t(pos) * a.R;
                    float *to = angles + (fn % kDepth) * G * 16;
                    for (int i = lane; i < a.R / 4; i += 32)
                        copy16(to + 4 * i, row + 4 * i);
                }
            }
            fresh = false;
            fh += kRows;
            if (fh >= fh1) {
                ++fn;
                fresh = true;
                next_item();
            } else if (h < hq && h + kRows >= hq) {
                aim(h + kRows);
            } else {
                fp += fd;
            }
        }
        copies_end();
        slot_f = slot_f + 1 == kDepth ? 0 : slot_f + 1;
    };
    next_item();
#pragma unroll 1
    for (int i = 0; i < kDepth - 1; ++i)
        fetch();

    int slot = 0;
    for (int i = 0; i < items.count; ++i) {
        int h, h1;
        const int64_t t = items.enter(i, h, h1);
        f32x2 c2[8], s2[8];
        const T *w = nullptr;
        T *to = nullptr;
        int64_t d = 0;
        int part = -1;
        for (int left = h1 - h - g, hh = h + g; h < h1; h += kRows, hh += kRows, left -= kRows) {
            copies_wait<kDepth - 2>();
            __syncwarp();
            if (left > 0 && part != (hh >= hq)) {  // a token's first queries, or keys: angles and weight into factors
                part = hh >= hq;
                const Part<T> &p = a.part[part];
                to = p.out.row(t, hh - (part ? hq : 0));
                d = kRows * p.out.sh;
                w = p.w;
                angle_factors<IL, false>(angles + (i % kDepth) * G * 16, a.R, n, bad_bits >> (i % 32) & 1, c2, s2);
                if (w) {
                    f32x2 f[8];
                    load_weight(w, n, f);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        c2[j] = n.rot ? mul2(c2[j], f[j]) : f[j];
                        s2[j] = mul2(s2[j], partner<IL>(f, j));
                    }
                }
            }
            f32x2 v[8], y[8];
            unpack8(ring + slot * kSlot, 32, v, static_cast<const T *>(nullptr));
            unpack8(ring + slot * kSlot + kVec * 32, 32, v + 4, static_cast<const T *>(nullptr));
            const float r = inv_rms<G>(v, inv_d, a.eps);
            if (n.rot) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    y[j] = fma2(v[j], c2[j], mul2(partner<IL>(v, j), s2[j]));
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    y[j] = w ? mul2(v[j], c2[j]) : v[j];
            }
            if (w) {
                const f32x2 r2 = pair(r, r);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    y[j] = mul2(y[j], r2);
            }
            if (left > 0) {  // a group without a head has worked on an old step
                store_unit(to, n, y);
                to += d;
            }
            __syncwarp();
            slot = slot + 1 == kDepth ? 0 : slot + 1;
            fetch();
        }
    }
    copies_wait<0>();
}

template <typename T, int G, bool IL>
__global__ void __launch_bounds__(kThreads, 2) qk_backward_kernel(const QkArgs<T> a)
{
    constexpr int kRows = 32 / G;
    constexpr int kVec = sizeof(T) / 2;
    constexpr int kSlot = 4 * kVec * 32, kDepth = depth_of<T>(2);
    extern __shared__ uint4 smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane / G;
    uint4 *ring = smem + warp * (ring_bytes<T>(2, G) / 16);
    float *angles = reinterpret_cast<float *>(ring + kDepth * kSlot);
    ring += lane;
    const Unit n = unit_of<IL>(lane % G, a.D, a.R);
    const float inv_d = 1.f / float(a.D);
    const int which = int(blockIdx.x) >= a.part[0].blocks;
    const Part<T> &p = a.part[which];
    const int block = int(blockIdx.x) - (which ? a.part[0].blocks : 0);
    const bool norm = p.w != nullptr;

    f32x2 w[8], acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        acc[i] = 0;
    if (norm)
        load_weight(p.w, n, w);
    Items<T> items;
    items.start(a, int64_t(block) * kWarps + warp, int64_t(p.blocks) * kWarps, p.heads, p.heads_per_item);
    clear_missing(ring - lane, lane, kDepth * 4 * kVec, kVec, n);

    int fn = 0, fh = 0, fh1 = 0, slot_f = 0;
    const T *fd = nullptr, *fx = nullptr;
    uint32_t bad_bits = 0;
    const int64_t step_d = kRows * p.d.sh, step_x = kRows * p.x.sh, step_out = kRows * p.out.sh;
    auto next_item = [&] {
        if (fn < items.count) {
            const int64_t t = items.enter(fn, fh, fh1);
            fd = p.d.row(t, fh + g);
            fx = p.x.row(t, fh + g);
        }
    };
    bool fresh = true;
    auto fetch = [&] {
        if (fn < items.count) {
            if (fh + g < fh1) {
                uint4 *to = ring + slot_f * kSlot;
#pragma unroll
                for (int k = 0; k < kVec; ++k) {
                    if (n.has0)
                        copy16(to + k * 32, fd + n.off0 + k * 4);
                    if (n.has1)
                        copy16(to + (kVec + k) * 32, fd + n.off1 + k * 4);
                    if (norm && n.has0)
                        copy16(to + (2 * kVec + k) * 32, fx + n.off0 + k * 4);
                    if (norm && n.has1)
                        copy16(to + (3 * kVec + k) * 32, fx + n.off1 + k * 4);
                }
            }
            if (fresh && a.R) {
                const int pos = items.row(a, fn);
                const uint32_t bit = 1u << (fn % 32);
                bad_bits = pos < 0 ? bad_bits | bit : bad_bits & ~bit;
                if (pos >= 0) {
                    const float *row = a.table + int64_t(pos) * a.R;
                    float *to = angles + (fn % kDepth) * G * 16;
                    for (int i = lane; i < a.R / 4; i += 32)
                        copy16(to + 4 * i, row + 4 * i);
                }
            }
            fresh = false;
            fh += kRows;
            fd += step_d;
            fx += step_x;
            if (fh >= fh1) {
                ++fn;
                fresh = true;
                next_item();
            }
        }
        copies_end();
        slot_f = slot_f + 1 == kDepth ? 0 : slot_f + 1;
    };
    next_item();
#pragma unroll 1
    for (int i = 0; i < kDepth - 1; ++i)
        fetch();

    int slot = 0;
    for (int i = 0; i < items.count; ++i) {
        int h, h1;
        const int64_t t = items.enter(i, h, h1);
        T *to = p.out.row(t, h + g);
        f32x2 c2[8], s2[8];
        bool first = true;
        for (; h < h1; h += kRows) {
            copies_wait<kDepth - 2>();
            __syncwarp();
            if (first)
                angle_factors<IL, true>(angles + (i % kDepth) * G * 16, a.R, n, bad_bits >> (i % 32) & 1, c2, s2);
            first = false;
            const bool on = h + g < h1;
            const uint4 *from = ring + slot * kSlot;
            f32x2 d[8], y[8];
            unpack8(from, 32, d, static_cast<const T *>(nullptr));
            unpack8(from + kVec * 32, 32, d + 4, static_cast<const T *>(nullptr));
            if (n.rot) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    y[j] = fma2(d[j], c2[j], mul2(partner<IL>(d, j), s2[j]));
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    y[j] = d[j];
            }
            if (norm) {
                f32x2 x[8];
                unpack8(from + 2 * kVec * 32, 32, x, static_cast<const T *>(nullptr));
                unpack8(from + 3 * kVec * 32, 32, x + 4, static_cast<const T *>(nullptr));
                if (h + kRows > h1 && !on) {  // a group without a head adds nothing to the weight's gradient
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        x[j] = y[j] = 0;
                }
                const float r = inv_rms<G>(x, inv_d, a.eps);
                const f32x2 r2 = pair(r, r);
                f32x2 m2 = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    x[j] = mul2(x[j], r2);
                    acc[j] = fma2(y[j], x[j], acc[j]);
                    y[j] = mul2(y[j], w[j]);
                    m2 = fma2(y[j], x[j], m2);
                }
                const float m = -group_sum<G>(lo_of(m2) + hi_of(m2)) * inv_d;
                m2 = pair(m, m);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    y[j] = mul2(fma2(x[j], m2, y[j]), r2);
            }
            if (on)
                store_unit(to, n, y);
            to += step_out;
            __syncwarp();
            slot = slot + 1 == kDepth ? 0 : slot + 1;
            fetch();
        }
    }
    copies_wait<0>();
    if (!norm)
        return;
    __syncthreads();  // the ring is free: the lanes' sums go through it
    float *sums = reinterpret_cast<float *>(smem);
    const int row = warp * kRows + g;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int off = i < 4 ? n.off0 + 2 * i : n.off1 + 2 * (i - 4);
        if (i < 4 ? n.has0 : n.has1) {
            sums[row * 16 * G + off] = lo_of(acc[i]);
            sums[row * 16 * G + off + 1] = hi_of(acc[i]);
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.D; i += kThreads) {
        float x = 0.f;
        for (int k = 0; k < kThreads / G; ++k)
            x += sums[k * 16 * G + i];
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
    if (col < D) {
#pragma unroll 4
        for (int i = threadIdx.y; i < n; i += 32)
            x += p[int64_t(i) * D + col];
    }
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
        if (!qk->table || !qk->positions || qk->max_position < 1 || qk->max_position > 0x7fffffff)
            return op_fail(TIDE_ERR_INVALID_ARG, "a rotation needs a table, positions and max_position in [1, 2^31)");
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

// Heads of one warp's item: all of a token, or whole steps of fewer where that
// leaves warps without an item.
int heads_per_item(int heads, int rows, int64_t tokens, int64_t warps)
{
    const int64_t steps = (heads + rows - 1) / rows, want = std::max<int64_t>(1, warps / std::max<int64_t>(tokens, 1));
    return int((steps + std::min(steps, want) - 1) / std::min(steps, want)) * rows;
}

// Blocks of the backward for queries and for keys, shared by their
// steps of four heads and one more for each token's own work.
// per_sm: two for the vector kernel; eight for the generic one, whose warps keep
// nothing in flight beyond their own head.
constexpr int kVecPerSm = 2, kGenericPerSm = 8;
void grad_blocks(const tide_qk_t *qk, int sms, int per_sm, int *q, int *k)
{
    const int64_t all = int64_t(sms) * per_sm;
    const int64_t wq = qk->q_heads ? qk->q_heads + 4 : 0, wk = qk->k_heads ? qk->k_heads + 4 : 0;
    int64_t nq = wq + wk ? (all * wq + wq + wk - 1) / (wq + wk) : 0;
    int64_t nk = all - nq;
    if (qk->k_heads > 0 && nk < 1)
        nk = 1;
    // a block that gets a step of at least one of its warps
    *q = int(qk->q_heads > 0 ? std::min(nq, (qk->tokens * qk->q_heads + kWarps - 1) / kWarps) : 0);
    *k = int(qk->k_heads > 0 ? std::min(nk, (qk->tokens * qk->k_heads + kWarps - 1) / kWarps) : 0);
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

// Starts a vector kernel with its rings.
template <auto KERNEL, typename T>
tide_status_t launch_vec(const QkArgs<T> &a, unsigned grid, int smem, const char *what, cudaStream_t st)
{
    const cudaError_t e = tide::op_allow_smem<KERNEL>(smem);
    if (e != cudaSuccess)
        return op_fail(TIDE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
    KERNEL<<<grid, kThreads, size_t(smem), st>>>(a);
    return tide::op_launched(what);
}
template <typename T, int G>
tide_status_t launch_forward(const QkArgs<T> &a, bool il, unsigned grid, cudaStream_t st)
{
    constexpr int smem = kWarps * ring_bytes<T>(1, G);
    return il ? launch_vec<qk_forward_kernel<T, G, true>>(a, grid, smem, "qk_norm_rope", st)
              : launch_vec<qk_forward_kernel<T, G, false>>(a, grid, smem, "qk_norm_rope", st);
}
template <typename T, int G>
tide_status_t launch_backward(const QkArgs<T> &a, bool il, unsigned grid, cudaStream_t st)
{
    constexpr int smem = std::max(kWarps * ring_bytes<T>(2, G), kThreads * 16 * 4);
    return il ? launch_vec<qk_backward_kernel<T, G, true>>(a, grid, smem, "qk_norm_rope_grad", st)
              : launch_vec<qk_backward_kernel<T, G, false>>(a, grid, smem, "qk_norm_rope_grad", st);
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
    // All heads of a token in one warp reuse its angles; few tokens are spread over more warps instead.
    const int g = lanes_of(qk), heads = qk->q_heads + qk->k_heads, rows = 32 / g;
    const int64_t blocks = int64_t(tide::op_sm_count()) * 2;
    a.heads_per_item = heads_per_item(heads, rows, qk->tokens, blocks * kWarps);
    const int64_t items = qk->tokens * ((heads + a.heads_per_item - 1) / a.heads_per_item);
    const unsigned grid = unsigned(std::min((items + kWarps - 1) / kWarps, blocks));
    switch (g) {
    case 4: return launch_forward<T, 4>(a, qk->interleaved, grid, st);
    case 8: return launch_forward<T, 8>(a, qk->interleaved, grid, st);
    case 16: return launch_forward<T, 16>(a, qk->interleaved, grid, st);
    default: return launch_forward<T, 32>(a, qk->interleaved, grid, st);
    }
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
    grad_blocks(qk, tide::op_sm_count(), vec ? kVecPerSm : kGenericPerSm, &a.part[0].blocks, &a.part[1].blocks);
    a.part[0].partial = partial;
    a.part[1].partial = partial + int64_t(a.part[0].blocks) * a.D;
    const unsigned grid = unsigned(a.part[0].blocks + a.part[1].blocks);
    if (!vec) {
        for (Part<T> &p : a.part)
            p.items = qk->tokens * p.heads;
        if (grid) {
            launch_generic<T, true>(a, qk->interleaved, st);
            if (const tide_status_t s = tide::op_launched("qk_norm_rope_grad"))
                return s;
        }
    } else if (grid) {
        const int g = lanes_of(qk);
        for (Part<T> &p : a.part) {
            p.heads_per_item = heads_per_item(std::max(p.heads, 1), 32 / g, qk->tokens, int64_t(p.blocks) * kWarps);
            p.items = qk->tokens * ((p.heads + p.heads_per_item - 1) / p.heads_per_item);
        }
        tide_status_t s = TIDE_OK;
        switch (g) {
        case 4: s = launch_backward<T, 4>(a, qk->interleaved, grid, st); break;
        case 8: s = launch_backward<T, 8>(a, qk->interleaved, grid, st); break;
        case 16: s = launch_backward<T, 16>(a, qk->interleaved, grid, st); break;
        default: s = launch_backward<T, 32>(a, qk->interleaved, grid, st); break;
        }
        if (s)
            return s;
    }
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
    if (!qk->q_weight && !qk->k_weight)
        return 0;
    int nq, nk;
    grad_blocks(qk, tide::op_sm_count(), kGenericPerSm, &nq, &nk);  // what rows will be on is not known here
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
    const int64_t need = tide_qk_norm_rope_grad_workspace(qk);
    if (workspace_bytes < need || (need && !workspace))
        return op_fail(TIDE_ERR_INVALID_ARG, "workspace of %lld bytes: need %lld", (long long)workspace_bytes,
                       (long long)need);
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
