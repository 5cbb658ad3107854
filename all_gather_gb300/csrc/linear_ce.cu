// Softmax cross entropy of a vocabulary head and its gradient, without the
// logits in memory.
//
//   z = x W^T,  lse_t = log sum_v exp(z_tv),  loss_t = lse_t - z_t,target
//   dz = (exp(z - lse) - [v = target]) dloss,  dx = dz W,  dW = dz^T x
//
// The loss takes tiles of the logits as they are made: each tile leaves, for
// each of its tokens, its maximum m and sum s of exp(z - m), the target's logit
// left out, and a second kernel joins a token's pairs in a fixed order.  That
// kernel also takes the target's logit, as a dot product of its own: the tensor
// cores cut the last bits of their sums towards zero, which averages out in lse
// but not in a single logit (8192 x 131072 x 4096: the loss is 9e-7 off, 1.4e-6
// with the tensor cores').  With z_t in one form only, the loss is
//   log(1 + sum over v != t of exp(z_v - z_t)),
// which no rounding makes negative and which keeps its digits where the target
// dominates and lse - z_t would cancel (4096 columns, z_t = 30: 2e-4 off).
//
// The gradient makes the logits again, a piece of the vocabulary at a time, and
// keeps only that piece's dz, rounded to bf16: the products take operands of
// one type, and its error is that of rounding x or W once more.  dz is kept
// relative to the largest |dloss|, which the results are multiplied by at their
// end: the usual dloss, the same for all tokens, would else put its own
// rounding on every term, where it does not average out.  The target's own dz,
// p - 1, is expm1(z_t - lse) of the same dot product: from the tensor cores'
// logit it would be off by their cut, 2e-4 at z_t = 30, which is more than a
// well-predicted token's whole gradient.
//
// All products run in one persistent kernel, a pair of blocks (two SMs) on tiles
// of 256 rows and up to 256 columns: in each block a thread fetches 64 columns
// of both operands at a time into a ring of swizzled tiles (TMA), one thread of
// the pair issues the tensor-core products into one of two accumulators in
// tensor memory, and eight warps of each block work on the other one.  The rows
// are the vocabulary's (the hidden columns', for dx) and the tile's columns are
// tokens: 256 rows suit sizes that are large anyway, and the columns can be
// fitted to the number of tokens, from 32.  A result warp turns its 32 x 32
// logits over in shared memory and has a token a thread.  The operand whose
// rows are the summed dimension (W for dx, dz and x for dW) is read as it lies,
// MN-major, so nothing is transposed in memory.
//
// Bound by the tensor cores for many tokens and by the weight's bytes for few.
// Measured: loss 8192 x 131072 x 4096 4.93 ms, 1,785 TFLOP/s (the clock held at
// 1.7 GHz by the power limit; 128 x 256 tiles of single blocks 5.69 ms); 64 x
// 131072 x 4096 162 us, 6.6 TB/s; 7 x 32768 x 2048 29 us, 4.6 TB/s.  Gradient
// 4096 x 131072 x 4096 7.68 ms, 1,718 TFLOP/s (single blocks 9.5 ms); 513 x
// 50001 x 2048 238 us, 1,324 TFLOP/s.
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "ops_internal.h"
#include "umma.h"

namespace {

using tide::op_aligned;
using tide::op_fail;
using bf16 = __nv_bfloat16;
namespace um = tide::umma;

constexpr int kM = 128, kN = 256, kK = 64;  // a block's rows, the pair's columns at most, a step of the sum
constexpr int kABytes = kM * kK * 2;        // a block's share of a step: its rows of A, and half of B's columns
constexpr int kRingBytes = 192 * 1024;
constexpr int kMaxStages = 10;              // six at 256 columns (four: 5% slower)
constexpr int kOutWarps = 8;                // warps that work on results
constexpr int kOutTile = 4096;              // a warp's results on their way out
constexpr int kSmemBytes = kRingBytes + kOutWarps * kOutTile + 1024;  // 1024: alignment
constexpr int kThreads = 64 + 32 * kOutWarps;                         // fetch, products, results
constexpr int kTmemCols = 512;                       // two accumulators of 256 columns
constexpr int kGroupM = 16;                          // row tiles that share a sweep over the columns, in L2 (4 and 64: same)
constexpr int64_t kPieceBytes = int64_t(256) << 20;  // dz of one piece of the vocabulary
constexpr int64_t kMinPiece = 8192;
constexpr int kMaxSplits = 64;
constexpr float kLog2e = 1.4426950408889634f;

// Set when a bounded wait of a product runs out; read and cleared by
// tide_ops_device_status.
__device__ int g_timed_out;

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

// What becomes of a tile: statistics of its tokens; dz; a share of dx; dW.
enum Epilogue { kStats, kDz, kAdd, kStore };

struct Gemm {
    CUtensorMap a, b, c;  // c: kDz and kStore: out; kAdd: sums, as [splits][M][N]
    int64_t M, N, K;
    int one_copy;        // MN-major operands: blocks of 64 columns come in one copy (3-d maps)
    int tiles_m, tiles_n, splits, steps;  // steps of the sum in all
    int tile_n;          // columns of a tile: a multiple of 32, of 128 for kStore
    int stages;          // of the ring
    int sums, sum_cols;  // kStats: accumulators that take a tile's steps in turn, and how far apart they are
    int64_t v0;          // first vocabulary row of this piece
    Targets y;
    float2 *part;        // kStats: [128-row tiles][N]
    const float *lse, *dloss, *unit, *miss;  // unit: what dz is relative to; miss: p - 1 of each token's target
    bf16 *out;           // kStore
    int64_t out_stride;
    int out_tiles;       // its rows are on 16-byte boundaries: stored as tiles
    int first;           // kAdd: the sums are written, not added to
    uint64_t wait_ns;
    int skip_fill;       // TIDE_DEBUG_SKIP_FILL
};

// exp of a difference of logits.  The difference is taken before the factor
// log2(e): folded into one multiply-add with a rounded log2(e) z it would be
// off by the rounding of z, and overflow for the largest z.  Results under
// 2^-126 are 0 (ftz), which spares the instruction's scaling of subnormals.
__device__ __forceinline__ float exp_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * kLog2e));
    return y;
}

struct Work {
    int m, n, split, s0, s1;  // tile, share of the sum, its steps
};
__device__ __forceinline__ Work work_of(const Gemm &g, int64_t i)
{
    Work w;
    const int64_t tiles = int64_t(g.tiles_m) * g.tiles_n;
    w.split = int(i / tiles);
    i -= w.split * tiles;
    const int64_t group = i / (int64_t(kGroupM) * g.tiles_n);
    const int rows = min(kGroupM, g.tiles_m - int(group) * kGroupM);
    i -= group * kGroupM * g.tiles_n;
    w.n = int(i / rows);
    w.m = int(group) * kGroupM + int(i % rows);
    const int64_t s = g.steps;
    w.s0 = int(s * w.split / g.splits);
    w.s1 = int(s * (w.split + 1) / g.splits);
    return w;
}

// Maximum and sum of exp(z - maximum) of 32 logits, of which the first `count`
// count.  An infinite maximum stands for itself: exp(z) is 0 or infinite.
__device__ __forceinline__ float2 stats_of(const uint32_t (&v)[32], int count)
{
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < 32; ++i)
        if (i < count)
            top = fmaxf(top, __uint_as_float(v[i]));
    const float at = isinf(top) ? 0.f : top;
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
        if (i < count)
            a += exp_fast(__uint_as_float(v[i]) - at);
        if (i + 1 < count)
            b += exp_fast(__uint_as_float(v[i + 1]) - at);
    }
    return make_float2(top, a + b);
}
__device__ __forceinline__ float2 join(float2 a, float2 b)
{
    const float top = fmaxf(a.x, b.x);
    return make_float2(top, (a.x == top ? a.y : a.y * exp_fast(a.x - top)) +
                                (b.x == top ? b.y : b.y * exp_fast(b.x - top)));
}

// A warp's 32 x 32 fp32 values turned over in its 4 KB of shared memory: from
// a row a lane to a column a lane.  The 16-byte pieces of a row are swizzled by
// its number, so neither side meets a bank twice.
__device__ __forceinline__ void turn_over(uint32_t tile, int lane, uint32_t (&v)[32])
{
#pragma unroll
    for (int j = 0; j < 8; ++j)
        um::store_shared16(tile + lane * 128 + ((j ^ (lane & 7)) << 4), v[4 * j], v[4 * j + 1], v[4 * j + 2],
                           v[4 * j + 3]);
    __syncwarp();
#pragma unroll
    for (int r = 0; r < 32; ++r)
        v[r] = um::load_shared4(tile + r * 128 + (((lane / 4) ^ (r & 7)) << 4) + lane % 4 * 4);
    __syncwarp();
}

template <int E>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1) gemm_kernel(const __grid_constant__ Gemm g)
{
    constexpr bool kAMn = E == kAdd || E == kStore, kBMn = E == kStore;  // operands that are MN-major
    extern __shared__ uint8_t smem_raw[];
    const uint32_t ring = (um::smem_addr(smem_raw) + 1023) / 1024 * 1024;
    __shared__ uint64_t bars[2 * kMaxStages + 5];
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int gave_up;
    __shared__ int pair_gave_up, fills;  // told at the end: a block of the pair gave up; stages that this one filled
    const uint32_t full = um::smem_addr(bars), empty = full + 8 * kMaxStages;
    const uint32_t acc_full = empty + 8 * kMaxStages, acc_empty = acc_full + 16, drained = acc_empty + 16;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = int(um::cluster_rank());  // block 0 of a pair issues the products
    const int cols_b = g.tile_n / 2, stage_bytes = kABytes + cols_b * kK * 2;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kMaxStages; ++i) {
            um::mbar_init(full + 8 * i, 1);
            um::mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            um::mbar_init(acc_full + 8 * i, 1);
            um::mbar_init(acc_empty + 8 * i, kOutWarps * 2);
        }
        um::mbar_init(drained, 1);
        um::fence_barrier_init();
        gave_up = pair_gave_up = 0;
        um::prefetch_map(&g.a);
        um::prefetch_map(&g.b);
    }
    if (warp == 1)
        um::tmem_alloc(um::smem_addr(&tmem_slot), kTmemCols);
    um::fence_before();
    __syncthreads();
    um::cluster_sync();
    um::fence_after();
    const uint32_t tmem = tmem_slot;
    const int64_t works = int64_t(g.tiles_m) * g.tiles_n * g.splits;
    const int64_t first = blockIdx.x / 2, step = gridDim.x / 2;
    int stage = 0, turns = 0;  // of the fetch warp: ring position, and how often the ring went round

    // The two loops below set the pace of every step of the sum, a few hundred cycles: operand layouts are known at
    // compile time, addresses run along, and whether MN-major blocks come in one copy is settled outside.
    if (warp == 0) {
        const bool leader = um::elected();
        const uint32_t full0 = um::cluster_addr(full, 0);  // both blocks' copies count at block 0's barriers
        const uint32_t tx = uint32_t(stage_bytes) * 2;
        auto fetch = [&](auto copies) {
            constexpr bool one_copy = decltype(copies)::value;
            uint32_t at = ring, bar = 0;  // the stage's memory, and its barrier's offset
            for (int64_t i = first; i < works; i += step) {
                const Work w = work_of(g, i);
                const int m = (w.m * 2 + rank) * kM, n = w.n * g.tile_n + rank * cols_b;
                for (int k = w.s0 * kK; k < w.s1 * kK; k += kK) {
                    if (!um::mbar_wait(empty + bar, (turns & 1) ^ 1, &gave_up, g.wait_ns))
                        return;
                    if (leader) {
                        if (rank == 0)
                            um::mbar_expect(full + bar, tx);
                        if (!kAMn) {
                            um::tma_load_2d(at, &g.a, k, m, full0 + bar);
                        } else if (one_copy) {
                            um::tma_load_3d(at, &g.a, 0, k, m / 64, full0 + bar);
                        } else {
                            for (int j = 0; j < kM / 64; ++j)
                                um::tma_load_2d(at + j * 64 * kK * 2, &g.a, m + j * 64, k, full0 + bar);
                        }
                        if (!kBMn) {
                            um::tma_load_2d(at + kABytes, &g.b, k, n, full0 + bar);
                        } else if (one_copy) {
                            um::tma_load_3d(at + kABytes, &g.b, 0, k, n / 64, full0 + bar);
                        } else {
                            for (int j = 0; j < cols_b / 64; ++j)
                                um::tma_load_2d(at + kABytes + j * 64 * kK * 2, &g.b, n + j * 64, k, full0 + bar);
                        }
                    }
                    at += stage_bytes, bar += 8;
                    if (++stage == g.stages)
                        stage = 0, ++turns, at = ring, bar = 0;
                }
            }
        };
        if ((kAMn || kBMn) && g.one_copy)
            fetch(std::true_type{});
        else
            fetch(std::false_type{});
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0) {
            const bool leader = um::elected();
            const uint32_t idesc = um::instr_desc(kM * 2, g.tile_n, kAMn, kBMn);
            constexpr uint32_t a_step = (kAMn ? 2048 : 32) >> 4, b_step = (kBMn ? 2048 : 32) >> 4;  // 16 of the sum
            const uint64_t a0 = um::operand_desc(ring, kAMn, 64 * kK * 2);
            const uint64_t b0 = um::operand_desc(ring + kABytes, kBMn, 64 * kK * 2);
            const uint32_t stage_units = uint32_t(stage_bytes) >> 4;
            int stage = 0, phase = 0, buf = 0, buf_phase = 0;
            uint32_t at = 0, bar = 0;
            bool ok = true;
            if (g.skip_fill && first == 0)  // nothing arrives at this barrier before the end
                ok = um::mbar_wait(drained, 0, &gave_up, g.wait_ns);
            for (int64_t i = first; ok && i < works; i += step) {
                const Work w = work_of(g, i);
                if (!(ok = um::mbar_wait<true>(acc_empty + 8 * buf, buf_phase ^ 1, &gave_up, g.wait_ns)))
                    break;
                um::fence_after();
                const uint32_t d0 = tmem + buf * kN;
                uint32_t d = d0;
                int turn = 0;
                bool add = false;
                for (int s = w.s0; s < w.s1; ++s) {
                    if (!(ok = um::mbar_wait(full + bar, phase, &gave_up, g.wait_ns)))
                        break;
                    um::fence_after();
                    if (leader) {
#pragma unroll
                        for (int k = 0; k < kK / 16; ++k)
                            um::mma_bf16(d, a0 + at + k * a_step, b0 + at + k * b_step, idesc, add || k > 0);
                        um::mma_commit(empty + bar);
                    }
                    if (E == kStats) {
                        d += g.sum_cols;
                        if (++turn == g.sums)
                            turn = 0, d = d0, add = true;
                    } else {
                        add = true;
                    }
                    at += stage_units, bar += 8;
                    if (++stage == g.stages)
                        stage = 0, phase ^= 1, at = 0, bar = 0;
                }
                __syncwarp();
                if (ok && leader)
                    um::mma_commit(acc_full + 8 * buf);
                if (++buf == 2)
                    buf = 0, buf_phase ^= 1;
            }
            __syncwarp();
            if (!ok && leader) {  // wait for the products in flight before the accumulators and tiles go
                g_timed_out = 1;
                um::mma_commit(drained);
                const uint64_t t0 = um::now_ns();
                while (!um::mbar_try(drained, 0) && um::now_ns() - t0 < g.wait_ns) {
                }
            }
        }
        __syncwarp();
    } else {
        // A warp reads the tensor-memory lanes of its number modulo 4; the first four warps take the first half of
        // the tile's columns, the others the rest.
        const int quarter = warp % 4, half = (warp - 2) / 4;
        const int half_n = (g.tile_n / 2 + 31) / 32 * 32;
        const int width = half ? g.tile_n - half_n : half_n;
        const uint32_t outs = ring + kRingBytes, out = outs + (warp - 2) * kOutTile;
        const uint32_t acc_done = um::cluster_addr(acc_empty, 0);
        const float unit = E == kStore || E == kDz ? *g.unit : 1.f;
        int buf = 0, buf_phase = 0, out_at = 0;
        int64_t i = first;
        for (; i < works; i += step) {
            const Work w = work_of(g, i);
            const int64_t m0 = (int64_t(w.m) * 2 + rank) * kM + quarter * 32, m = m0 + lane;
            const int64_t n0 = int64_t(w.n) * g.tile_n + half * half_n;
            const int rows = int(max(int64_t(0), min(int64_t(32), g.M - m0)));  // of the warp's
            // Before the wait, the lane's token of each 32 columns: kStats and kDz: target (as a row of the warp's);
            // kDz: lse, factor, the target's dz.
            int64_t hit[4];
            float lse[4], scale[4], dz_hit[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int64_t t = n0 + k * 32 + lane;
                int64_t y = -1;
                if ((E == kStats || E == kDz) && k * 32 < width && t < g.N)
                    y = g.y.get(t);
                hit[k] = y - g.v0 - m0;
                lse[k] = INFINITY, scale[k] = 0.f, dz_hit[k] = 0.f;  // an ignored token: exp(z - lse) = 0
                if (E == kDz && y != -1) {
                    lse[k] = g.lse[t];
                    scale[k] = y == -2 ? __int_as_float(0x7fffffff) : __fdiv_rn(g.dloss[t], unit);
                    dz_hit[k] = g.miss[t] * scale[k];
                }
            }
            bool ready = um::mbar_wait<false, 100>(acc_full + 8 * buf, buf_phase, &gave_up, g.wait_ns);
            if (E == kStats)  // the warps that meet at a barrier below leave together, should one's wait have run out
                ready = um::group_all(1 + half, 128, ready);
            if (!ready) {
                g_timed_out = 1;
                break;
            }
            um::fence_after();
            const uint32_t d = tmem + (uint32_t(quarter * 32) << 16) + buf * kN + half * half_n;
            float2 stats[4];  // kStats: of the lane's token in each 32 columns
#pragma unroll
            for (int c = 0; c < kN / 2; c += 32) {
                const int64_t n = n0 + c;
                const int cols = c < width ? int(min(int64_t(32), g.N - n)) : 0;
                stats[c / 32] = make_float2(-INFINITY, 0.f);
                if (cols <= 0)
                    continue;
                uint32_t v[32];
                um::tmem_load32(d + c, v);
                um::tmem_wait_load();
                if (E == kStats) {
                    const int sums = min(g.sums, w.s1 - w.s0);
                    for (int k = 1; k < sums; ++k) {
                        uint32_t u[32];
                        um::tmem_load32(d + k * g.sum_cols + c, u);
                        um::tmem_wait_load();
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            v[j] = __float_as_uint(__uint_as_float(v[j]) + __uint_as_float(u[j]));
                    }
                }
                if (E == kStats) {
                    turn_over(out, lane, v);  // v[r]: vocabulary row m0 + r of the lane's token
                    const int64_t at = hit[c / 32];
                    if (__any_sync(0xffffffffu, at >= 0 && at < 32)) {  // its target: joined later
#pragma unroll
                        for (int r = 0; r < 32; ++r)
                            if (at == r)
                                v[r] = __float_as_uint(-INFINITY);
                    }
                    stats[c / 32] = stats_of(v, rows);
                } else if (E == kAdd) {
                    if (lane == 0)
                        um::stores_read<0>();
                    __syncwarp();
                    if (w.s0 == w.s1) {  // a last piece shorter than its splits: nothing was summed
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            v[j] = 0;
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        um::store_shared16(out + lane * 128 + ((j ^ (lane & 7)) << 4), v[4 * j], v[4 * j + 1],
                                           v[4 * j + 2], v[4 * j + 3]);
                    um::fence_copies();
                    __syncwarp();
                    if (lane == 0 && rows > 0) {
                        if (g.first)
                            um::tma_store_3d(&g.c, out, int(n), int(m0), w.split);
                        else
                            um::tma_add_3d(&g.c, out, int(n), int(m0), w.split);
                        um::stores_end();
                    }
                } else {
                    // Tiles of 32 rows of 64 bytes, two in turn, their 16-byte pieces swizzled by bits 1 and 2 of the
                    // row's number.
                    const uint32_t tile = out + out_at * (kOutTile / 2);
                    if (E == kDz || g.out_tiles) {
                        if (lane == 0)
                            um::stores_read<1>();
                        __syncwarp();
                    }
                    if (E == kDz) {
                        // Lane j has the target, lse and factor of token n + j; everyone gets them in turn.
                        const int64_t at = hit[c / 32];
                        const uint32_t hits = __ballot_sync(0xffffffffu, at >= 0 && at < 32);
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            const float l = __shfl_sync(0xffffffffu, lse[c / 32], j);
                            const float f = __shfl_sync(0xffffffffu, scale[c / 32], j);
                            v[j] = __float_as_uint(exp_fast(__uint_as_float(v[j]) - l) * f);
                        }
                        if (hits) {  // targets among the warp's rows: apart, so that the loop above has no branches
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (hits >> j & 1) {
                                    const int r = __shfl_sync(0xffffffffu, int(at), j);
                                    const float f = __shfl_sync(0xffffffffu, dz_hit[c / 32], j);
                                    if (lane == r)
                                        v[j] = __float_as_uint(f);
                                }
                        }
                        // A row of the tile is a token: two bytes of it a lane.
                        const uint32_t piece = uint32_t(lane) / 8, byte = uint32_t(lane) % 8 * 2;
#pragma unroll
                        for (int j = 0; j < 32; j += 2) {
                            const uint32_t f = tide::pack_bf16(__uint_as_float(v[j]), __uint_as_float(v[j + 1]));
                            const uint32_t to = tile + j * 64 + ((piece ^ (j / 2 & 3)) << 4) + byte;
                            um::store_shared2(to, uint16_t(f));
                            um::store_shared2(to + 64, uint16_t(f >> 16));
                        }
                    } else {
                        uint32_t f[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            f[j] = tide::pack_bf16(__uint_as_float(v[2 * j]) * unit, __uint_as_float(v[2 * j + 1]) * unit);
                        if (g.out_tiles) {
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                um::store_shared16(tile + lane * 64 + ((j ^ (lane / 2 & 3)) << 4), f[4 * j],
                                                   f[4 * j + 1], f[4 * j + 2], f[4 * j + 3]);
                        } else if (lane < rows) {
                            uint16_t *p = reinterpret_cast<uint16_t *>(g.out) + m * g.out_stride + n;
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (j < cols)
                                    p[j] = uint16_t(f[j / 2] >> (16 * (j % 2)));
                        }
                    }
                    if (E == kDz || g.out_tiles) {
                        um::fence_copies();
                        __syncwarp();
                        if (lane == 0 && rows > 0) {
                            um::tma_store_2d(&g.c, tile, int(E == kDz ? m0 : n), int(E == kDz ? n : m0));
                            um::stores_end();
                        }
                        out_at ^= 1;
                    }
                }
            }
            um::fence_before();
            __syncwarp();
            if (lane == 0)
                um::mbar_arrive_cluster(acc_done + 8 * buf);
            if (E == kStats) {  // join the block's four shares of 32 rows, 32 tokens a warp
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    um::store_shared8(out + (k * 32 + lane) * 8, __float_as_uint(stats[k].x),
                                      __float_as_uint(stats[k].y));
                um::group_sync(1 + half, 128);
                float2 s = make_float2(-INFINITY, 0.f);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t x, y;
                    um::load_shared8(outs + (half * 4 + k) * kOutTile + (quarter * 32 + lane) * 8, x, y);
                    s = join(s, make_float2(__uint_as_float(x), __uint_as_float(y)));
                }
                const int64_t t = n0 + quarter * 32 + lane;
                if (quarter * 32 < width && t < g.N)
                    g.part[(int64_t(w.m) * 2 + rank) * g.N + t] = s;
                um::group_sync(1 + half, 128);
            }
            if (++buf == 2)
                buf = 0, buf_phase ^= 1;
        }
        if (lane == 0)
            um::stores_read<0>();
        __syncwarp();
        if (i < works) {  // a wait has run out: this tile and the later ones become NaN (0x7fff7fff: so is either half)
            for (int j = 0; j < kOutTile / 512; ++j)
                um::store_shared16(out + j * 512 + lane * 16, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
            um::fence_copies();
            __syncwarp();
            for (; i < works; i += step) {
                const Work w = work_of(g, i);
                const int64_t m0 = (int64_t(w.m) * 2 + rank) * kM + quarter * 32;
                const int64_t n0 = int64_t(w.n) * g.tile_n + half * half_n;
                if (E == kStats) {
                    const int64_t t = n0 + quarter * 32 + lane;
                    if (quarter * 32 < width && t < g.N)
                        g.part[(int64_t(w.m) * 2 + rank) * g.N + t] = make_float2(-INFINITY, __int_as_float(0x7fffffff));
                    continue;
                }
                for (int c = 0; c < width; c += 32) {
                    const int64_t n = n0 + c;
                    if (n >= g.N || m0 >= g.M)
                        continue;
                    if (E == kStore && !g.out_tiles) {
                        for (int64_t j = n; j < min(n + 32, g.N); ++j)
                            if (m0 + lane < g.M)
                                reinterpret_cast<uint16_t *>(g.out)[(m0 + lane) * g.out_stride + j] = 0x7fff;
                    } else if (lane == 0) {
                        if (E == kAdd && g.first)
                            um::tma_store_3d(&g.c, out, int(n), int(m0), w.split);
                        else if (E == kAdd)
                            um::tma_add_3d(&g.c, out, int(n), int(m0), w.split);
                        else
                            um::tma_store_2d(&g.c, out, int(E == kDz ? m0 : n), int(E == kDz ? n : m0));
                    }
                }
            }
            if (lane == 0) {
                um::stores_end();
                um::stores_read<0>();
            }
            __syncwarp();
        }
    }
    um::fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && gave_up) {
        for (int r = 0; r < 2; ++r)
            um::store_cluster(um::cluster_addr(um::smem_addr(&pair_gave_up), r), 1);
    }
    if (threadIdx.x == 0)
        fills = turns * g.stages + stage;
    um::cluster_sync();
    if (pair_gave_up) {  // the pair's copies in flight land, for as long as another wait, before its memory goes
        if (threadIdx.x == 0 && rank == 0) {
            const int mine = fills, theirs = um::load_cluster(um::cluster_addr(um::smem_addr(&fills), 1));
            const uint64_t t0 = um::now_ns();
            for (int k = 0; k < g.stages; ++k) {
                const int times = (max(mine, theirs) - k + g.stages - 1) / g.stages;  // fills of this stage
                if ((mine - k + g.stages - 1) / g.stages < times)  // the other block was ahead: its bytes alone
                    um::mbar_expect(full + 8 * k, uint32_t(stage_bytes));
                while (times > 0 && !um::mbar_try(full + 8 * k, (times - 1) & 1) && um::now_ns() - t0 < g.wait_ns) {
                }
            }
        }
        um::cluster_sync();
    }
    um::fence_after();
    if (warp == 1)
        um::tmem_free(tmem, kTmemCols);
}

// Rows that the tiled copies cannot take (16-byte boundaries) go into the
// workspace first, `pitch` elements (a multiple of 8) apart; what lies between
// them is not read as part of a row.
__global__ void __launch_bounds__(256) align_kernel(const bf16 *in, int64_t stride, int64_t rows, int64_t cols,
                                                    bf16 *out, int64_t pitch)
{
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const bf16 *row = in + r * stride;
        for (int64_t c = 8 * threadIdx.x; c < cols; c += 8 * 256) {
            uint32_t w[4];
            tide::load16_any(row + c, row + cols, w);
            *reinterpret_cast<uint4 *>(out + r * pitch + c) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

// The way back: rows `pitch` elements apart to rows on any boundary, by aligned
// 16-byte pieces between a row's first and last few elements.
__global__ void __launch_bounds__(256) unalign_kernel(const bf16 *in, int64_t pitch, int64_t rows, int64_t cols,
                                                      bf16 *out, int64_t stride)
{
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const bf16 *from = in + r * pitch;
        bf16 *to = out + r * stride;
        const int64_t head = min(cols, int64_t((16 - (reinterpret_cast<uintptr_t>(to) & 15)) % 16 / 2));
        const int64_t whole = (cols - head) / 8, tail = head + 8 * whole;
        for (int64_t i = threadIdx.x; i < whole; i += 256) {
            uint32_t w[4];
            tide::load16_any(from + head + 8 * i, from + cols, w);
            *reinterpret_cast<uint4 *>(to + head + 8 * i) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        if (threadIdx.x < head)
            to[threadIdx.x] = from[threadIdx.x];
        if (tail + threadIdx.x < cols)
            to[tail + threadIdx.x] = from[tail + threadIdx.x];
    }
}

// A lane's share of the dot product of two rows on 16-byte boundaries, of which
// its warp takes part `part` of `parts`.
__device__ __forceinline__ float dot_share(const bf16 *a, const bf16 *b, int H, int lane, int part, int parts)
{
    float z = 0.f;
    const int whole = H / 8;
    for (int i = part * 32 + lane; i < whole; i += 32 * parts) {
        float p[8], q[8];
        tide::load8(a + 8 * i, p);
        tide::load8(b + 8 * i, q);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            z = __fmaf_rn(p[k], q[k], z);
    }
    if (part == 0 && whole * 8 + lane < H)
        z = __fmaf_rn(tide::to_f32(a[whole * 8 + lane]), tide::to_f32(b[whole * 8 + lane]), z);
    return z;
}

// Joins the pairs (maximum, sum) of `rows` neighbouring tokens a block, 256 /
// rows slices of the vocabulary tiles each, and takes their targets' logits, a
// warp a token or, where there are fewer than eight, a part of one.
__global__ void __launch_bounds__(256) join_kernel(const float2 *part, int tiles, int64_t T, int rows, Targets y,
                                                   const bf16 *x, int64_t x_stride, const bf16 *w, int64_t w_stride,
                                                   int H, float *loss, float *lse)
{
    __shared__ float2 slices[256];
    __shared__ float dots[32];
    const int64_t t0 = int64_t(blockIdx.x) * rows;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int parts = rows < 8 ? 8 / rows : 1;
    for (int r = rows < 8 ? warp % rows : warp; r < rows; r += 8) {
        const int64_t v = t0 + r < T ? y.get(t0 + r) : -1;
        float z = 0.f;
        if (v >= 0)
            z = dot_share(x + (t0 + r) * x_stride, w + v * w_stride, H, lane, rows < 8 ? warp / rows : 0, parts);
#pragma unroll
        for (int o = 16; o > 0; o /= 2)
            z += __shfl_xor_sync(0xffffffffu, z, o);
        if (lane == 0)
            dots[rows < 8 ? warp : r] = z;
    }

    const int row = threadIdx.x % rows, slice = threadIdx.x / rows, n = 256 / rows;
    const int64_t t = t0 + row;
    float2 s = make_float2(-INFINITY, 0.f);
    if (t < T) {
        int i = slice;
        for (; i + 3 * n < tiles; i += 4 * n) {
            float2 p[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                p[k] = part[int64_t(i + k * n) * T + t];
            s = join(s, join(join(p[0], p[1]), join(p[2], p[3])));
        }
        for (; i < tiles; i += n)
            s = join(s, part[int64_t(i) * T + t]);
    }
    slices[threadIdx.x] = s;
    for (int half = n / 2; half > 0; half /= 2) {
        __syncthreads();
        if (slice < half)
            slices[threadIdx.x] = s = join(s, slices[threadIdx.x + half * rows]);
    }
    __syncthreads();
    if (slice > 0 || t >= T)
        return;
    float z = dots[row];
    for (int k = 1; k < parts; ++k)  // rows < 8: parts of a token are `rows` warps apart
        z += dots[row + k * rows];
    // s has every logit but the target's, if there is one.
    const int64_t v = y.get(t);
    float l, e = 0.f;
    if (v < 0 || !isfinite(z)) {
        l = logf(s.y) + (isinf(s.x) ? 0.f : s.x);
        if (v >= 0) {
            if (!(z < 0.f) && !isnan(l))
                l = z;
            e = l - z;
        } else if (v == -2) {
            e = __int_as_float(0x7fffffff);
        }
    } else if (s.x <= z) {
        e = log1pf(s.y * expf(s.x - z));
        l = z + e;
    } else {
        e = logf(s.y + expf(z - s.x));
        l = s.x + e;
        e += s.x - z;
    }
    lse[t] = l;
    loss[t] = e;
}

// Block 0: what dz is kept relative to: the largest finite |dloss| of the tokens
// that count, 1 if that is 0.  The others, a token each: its hidden state into
// the workspace, rows `pitch` (a multiple of 8) apart on 16-byte boundaries, and
// p - 1 of its target (0 where there is none).  An ignored token's row becomes
// zeroes, for its dz is 0, and 0 times what it holds need not be.
// ALIGNED: x and weight have their rows on 16-byte boundaries, and H % 8 = 0.
// Bound by loads that wait for one another: 513 x 2048 takes 4.4 us, with a
// warp a token 7.5 us.
template <bool ALIGNED>
__global__ void __launch_bounds__(256) prepare_kernel(const float *dloss, Targets y, int64_t T, float *unit,
                                                      const bf16 *x, int64_t x_stride, const bf16 *w, int64_t w_stride,
                                                      int H, const float *lse, float *miss, bf16 *out, int64_t pitch)
{
    __shared__ float shares[8];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    if (blockIdx.x) {
        const int64_t t = int64_t(blockIdx.x) - 1, v = y.get(t);
        const float l = lse[t];
        const bf16 *a = x + t * x_stride, *b = w + max(v, int64_t(0)) * w_stride;
        float z = 0.f;
        for (int c = 8 * threadIdx.x; c < H; c += 8 * 256) {
            uint32_t p[4], q[4];
            if constexpr (ALIGNED) {
                const uint4 i = *reinterpret_cast<const uint4 *>(a + c), j = *reinterpret_cast<const uint4 *>(b + c);
                p[0] = i.x, p[1] = i.y, p[2] = i.z, p[3] = i.w;
                q[0] = j.x, q[1] = j.y, q[2] = j.z, q[3] = j.w;
            } else {
                tide::load16_any(a + c, a + H, p);
                tide::load16_any(b + c, b + H, q);
            }
            const uint32_t kept = v == -1 ? 0 : ~0u;
            *reinterpret_cast<uint4 *>(out + t * pitch + c) =
                make_uint4(p[0] & kept, p[1] & kept, p[2] & kept, p[3] & kept);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t high = k % 2 ? 0xffff0000u : 0xffffu, up = k % 2 ? 0 : 16;
                if (ALIGNED || c + k < H)
                    z = __fmaf_rn(__uint_as_float((p[k / 2] & high) << up), __uint_as_float((q[k / 2] & high) << up), z);
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o /= 2)
            z += __shfl_xor_sync(0xffffffffu, z, o);
        if (lane == 0)
            shares[warp] = z;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int k = 1; k < 8; ++k)
                z += shares[k];
            miss[t] = v < 0 ? 0.f : expm1f(z - l);
        }
        return;
    }
    float top = 0.f;
#pragma unroll 8
    for (int64_t t = threadIdx.x; t < T; t += 256) {
        const float d = fabsf(dloss[t]);
        if (y.get(t) != -1 && d > top && d < INFINITY)
            top = d;
    }
#pragma unroll
    for (int o = 16; o > 0; o /= 2)
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0)
        shares[warp] = top;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int k = 1; k < 8; ++k)
            top = fmaxf(top, shares[k]);
        *unit = top > 0.f ? top : 1.f;
    }
}

// dx [T, H] = sum of the splits, in order, of the sums [H][T] (rows `pitch`
// apart), times their unit: blocks of 32 x 32, turned over in shared memory.
__global__ void __launch_bounds__(256) round_kernel(const float *acc, int splits, int64_t T, int64_t H, int64_t pitch,
                                                    const float *unit_, bf16 *out, int64_t stride)
{
    const float unit = *unit_;
    __shared__ float tile[32][33];
    const int64_t t0 = int64_t(blockIdx.x) * 32, h0 = int64_t(blockIdx.y) * 32;
    const int lane = threadIdx.x % 32, row = threadIdx.x / 32;
#pragma unroll
    for (int r = row; r < 32; r += 8) {
        float x = 0.f;
        if (t0 + lane < T && h0 + r < H) {
            const float *p = acc + (h0 + r) * pitch + t0 + lane;
#pragma unroll 4
            for (int s = 0; s < splits; ++s)
                x += p[s * H * pitch];
        }
        tile[r][lane] = x * unit;
    }
    __syncthreads();
#pragma unroll
    for (int r = row; r < 32; r += 8)
        if (t0 + r < T && h0 + lane < H)
            out[(t0 + r) * stride + h0 + lane] = __float2bfloat16_rn(tile[lane][r]);
}

int64_t round_up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

// Rows apart, and less than the 2^40 bytes that a tensor map takes.
bool stride_ok(int64_t rows, int64_t stride, int64_t cols)
{
    return tide::op_extent_ok(rows, stride) && (rows < 2 || (stride >= cols && stride < int64_t(1) << 39));
}

tide_status_t check_desc(const tide_ce_t *ce)
{
    if (!ce)
        return op_fail(TIDE_ERR_INVALID_ARG, "ce is NULL");
    if (ce->tokens < 0 || ce->tokens > 0x7fffffff - 512 || ce->vocab < 1 || ce->vocab > 0x7fffffff - 512 ||
        ce->hidden < 1 || ce->hidden > (1 << 20))
        return op_fail(TIDE_ERR_INVALID_ARG, "tokens %lld, vocab %lld, hidden %lld", (long long)ce->tokens,
                       (long long)ce->vocab, (long long)ce->hidden);
    if (ce->debug & ~(TIDE_DEBUG_SHORT_WAIT | TIDE_DEBUG_SKIP_FILL))
        return op_fail(TIDE_ERR_INVALID_ARG, "unknown debug bits 0x%x", ce->debug);
    if (ce->target_bytes != 4 && ce->target_bytes != 8)
        return op_fail(TIDE_ERR_INVALID_ARG, "target_bytes %d: need 4 or 8", ce->target_bytes);
    if (!stride_ok(ce->tokens, ce->x_stride, ce->hidden) || !stride_ok(ce->vocab, ce->weight_stride, ce->hidden))
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

// ---------------------------------------------------------------- host

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled()
{
    static const EncodeTiled fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return fn;
}

// A row-major bf16 matrix.
struct Mat {
    const bf16 *p;
    int64_t rows, cols, stride;
    int64_t readable = 0;  // columns that may be read, if more than cols
    int64_t blocks_of_64() const { return readable ? readable / 64 : cols % 64 ? 0 : cols / 64; }
};

bool rows_aligned(const void *p, int64_t stride, int64_t rows)
{
    return op_aligned(p, 16) && (rows < 2 || stride % 8 == 0);
}

tide_status_t encode(CUtensorMap *map, CUtensorMapDataType type, int rank, void *p, const cuuint64_t *dims,
                     const cuuint64_t *strides, const cuuint32_t *box, CUtensorMapSwizzle swizzle)
{
    const cuuint32_t step[3] = {1, 1, 1};
    const CUresult r = encode_tiled()(map, type, cuuint32_t(rank), p, dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return op_fail(TIDE_ERR_CUDA, "cuTensorMapEncodeTiled: %d", int(r));
    return TIDE_OK;
}

// Tensor map whose copies are `box_rows` rows of `box_cols` columns (64, or 32);
// what lies outside the matrix reads as 0 and is not written.
tide_status_t make_map(CUtensorMap *map, const Mat &m, int box_rows, int box_cols = 64)
{
    const cuuint64_t dims[2] = {cuuint64_t(m.cols), cuuint64_t(m.rows)};
    const cuuint64_t strides[1] = {cuuint64_t(m.rows < 2 ? (m.cols + 7) / 8 * 16 : m.stride * 2)};
    const cuuint32_t box[2] = {cuuint32_t(box_cols), cuuint32_t(box_rows)};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<bf16 *>(m.p), dims, strides, box,
                  box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}

// An MN-major operand whose copies are `blocks` blocks of 64 columns by 64 rows:
// one copy where the plain map takes one a block.  Its last block of columns is
// whole, so they have to be a multiple of 64 that may be read.
tide_status_t make_block_map(CUtensorMap *map, const Mat &m, int blocks)
{
    const cuuint64_t dims[3] = {64, cuuint64_t(m.rows), cuuint64_t(m.blocks_of_64())};
    const cuuint64_t strides[2] = {cuuint64_t(m.rows < 2 ? m.blocks_of_64() * 128 : m.stride * 2), 128};
    const cuuint32_t box[3] = {64, kK, cuuint32_t(blocks)};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<bf16 *>(m.p), dims, strides, box,
                  CU_TENSOR_MAP_SWIZZLE_128B);
}

// The same for fp32 sums [splits][rows][cols] with rows `pitch` apart: 32 rows of 32 columns.
tide_status_t make_acc_map(CUtensorMap *map, float *p, int64_t splits, int64_t rows, int64_t cols, int64_t pitch)
{
    const cuuint64_t dims[3] = {cuuint64_t(cols), cuuint64_t(rows), cuuint64_t(splits)};
    const cuuint64_t strides[2] = {cuuint64_t(pitch * 4), cuuint64_t(rows * pitch * 4)};
    const cuuint32_t box[3] = {32, 32, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, p, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

Gemm base(const tide_ce_t *ce)
{
    Gemm g = {};
    g.y = {ce->targets, ce->target_bytes, ce->ignore_index, ce->vocab};
    g.splits = 1;
    g.wait_ns = ce->debug & TIDE_DEBUG_SHORT_WAIT ? tide::kShortWaitBudgetNs : tide::kWaitBudgetNs;
    g.skip_fill = (ce->debug & TIDE_DEBUG_SKIP_FILL) != 0;
    return g;
}

// Columns of a tile and shares of the sum for a product of `tiles_m` row tiles,
// N columns and `steps` steps: those of the shortest rounds.  A step takes as
// long as its columns and a fixed part, no less than what the fetch of its rows
// takes, and a tile's end another four steps'.  Shares are tried where they
// fill one to eight rounds.
void shape_of(int64_t tiles_m, int64_t N, int64_t steps, int unit, int max_splits, int *tile_n, int *splits)
{
    const int64_t pairs = std::max(tide::op_sm_count() / 2, 1);
    const int most = int(std::min<int64_t>(max_splits, steps / 4 + 1));
    double best = 1e300;
    for (int n = kN; n >= std::min(unit, 128); n -= unit) {
        const int64_t tiles = std::max<int64_t>(1, tiles_m * ((N + n - 1) / n));
        const double step = std::max(n, 96) + 32;
        int last = 0;
        for (int r = 0; r <= 8; ++r) {  // r = 0: one share
            const int s = r == 0 ? 1 : int(std::min<int64_t>(most, r * pairs / tiles));
            if (s <= last)
                continue;
            last = s;
            const double time = double((tiles * s + pairs - 1) / pairs) * (double(steps) / s * step + 4 * 288);
            if (time < best * 0.99)
                best = time, *tile_n = n, *splits = s;
            if (s == most)
                break;
        }
    }
}

// C[M, N] = sum over k of A B.  A K-major operand is given with its rows as the
// tile's dimension, an MN-major one with its rows as the summed one.
template <int E>
tide_status_t launch(Gemm &g, const Mat &a, const Mat &b, const char *what, cudaStream_t st)
{
    constexpr bool a_mn = E == kAdd || E == kStore, b_mn = E == kStore;
    g.M = a_mn ? a.cols : a.rows;
    g.N = b_mn ? b.cols : b.rows;
    g.K = a_mn ? a.rows : a.cols;
    g.steps = int((g.K + kK - 1) / kK);
    g.tiles_m = int((g.M + 2 * kM - 1) / (2 * kM));
    if (E != kAdd)
        shape_of(g.tiles_m, g.N, g.steps, E == kStore ? 128 : 32, 1, &g.tile_n, &g.splits);
    g.tiles_n = int((g.N + g.tile_n - 1) / g.tile_n);
    // The tensor cores cut each addition's last bits, so a long chain drifts towards zero (by 1 to 2e-6 over 4096
    // columns).  Where a tile leaves tensor memory free, the loss takes its steps in two to eight chains.
    g.sums = 1;
    while (E == kStats && g.sums * 2 * g.tile_n <= kN)
        g.sums *= 2;
    g.sum_cols = kN / g.sums;
    g.stages = std::min(kMaxStages, kRingBytes / (kABytes + g.tile_n / 2 * kK * 2));
    g.one_copy = a_mn && a.blocks_of_64() > 0 && (!b_mn || b.blocks_of_64() > 0);
    tide_status_t s = g.one_copy ? make_block_map(&g.a, a, kM / 64) : make_map(&g.a, a, a_mn ? kK : kM);
    if (!s)
        s = g.one_copy && b_mn ? make_block_map(&g.b, b, g.tile_n / 128) : make_map(&g.b, b, b_mn ? kK : g.tile_n / 2);
    if (!s && E == kStore && g.out_tiles)
        s = make_map(&g.c, {g.out, g.M, g.N, g.out_stride}, 32, 32);
    if (s)
        return s;
    const int64_t works = int64_t(g.tiles_m) * g.tiles_n * g.splits;
    const unsigned grid = unsigned(std::min<int64_t>(works, std::max(tide::op_sm_count() / 2, 1))) * 2;
    gemm_kernel<E><<<grid, kThreads, kSmemBytes, st>>>(g);
    return tide::op_launched(what);
}

// What the products need besides good arguments, asked for before a call
// enqueues anything.
template <int... E>
tide_status_t get_ready()
{
    if (!encode_tiled())
        return op_fail(TIDE_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
    cudaError_t e = cudaSuccess;
    ((e = e == cudaSuccess ? tide::op_allow_smem<gemm_kernel<E>>(kSmemBytes) : e), ...);
    return e == cudaSuccess ? TIDE_OK : op_fail(TIDE_ERR_CUDA, "ce: %s", cudaGetErrorString(e));
}

// Where a call's scratch data lies in its workspace, in bytes.
struct Layout {
    int64_t x = -1, w = -1, pitch = 0;  // aligned copies of x (always for the gradient) and weight, where needed
    int64_t part = 0;                   // loss
    int64_t dz = 0, acc = 0, unit = 0, miss = 0, piece = 0, acc_pitch = 0;  // gradient
    int splits = 1, tile_n = kN;        // of dx
    int64_t bytes = 0;
    int64_t take(int64_t n)
    {
        const int64_t at = bytes;
        bytes += round_up(n, 256);
        return at;
    }
};

Layout layout_of(const tide_ce_t *ce, bool grad)
{
    Layout l;
    l.pitch = round_up(ce->hidden, 8);
    if (grad || !rows_aligned(ce->x, ce->x_stride, ce->tokens))
        l.x = l.take(ce->tokens * l.pitch * 2);
    if (!rows_aligned(ce->weight, ce->weight_stride, ce->vocab))
        l.w = l.take(ce->vocab * l.pitch * 2);
    if (grad) {
        l.piece = piece_of(ce);
        l.acc_pitch = round_up(ce->tokens, 4);
        const int64_t sum = std::max<int64_t>(l.acc_pitch * ce->hidden * 4, 1);
        shape_of((ce->hidden + 2 * kM - 1) / (2 * kM), ce->tokens, (std::min(l.piece, ce->vocab) + kK - 1) / kK, 32,
                 int(std::max<int64_t>(1, std::min<int64_t>(kMaxSplits, kPieceBytes / sum))), &l.tile_n, &l.splits);
        l.dz = l.take(ce->tokens * l.piece * 2);
        l.acc = l.take(sum * l.splits);
        l.unit = l.take(4);
        l.miss = l.take(ce->tokens * 4);
    } else {
        l.part = l.take((ce->vocab + 2 * kM - 1) / (2 * kM) * 2 * ce->tokens * 8);
    }
    l.bytes = std::max<int64_t>(l.bytes, 256);
    return l;
}

tide_status_t align_rows(Mat &m, char *workspace, int64_t at, int64_t pitch, cudaStream_t st)
{
    if (at < 0 || m.rows == 0)
        return TIDE_OK;
    bf16 *out = reinterpret_cast<bf16 *>(workspace + at);
    align_kernel<<<unsigned(std::min<int64_t>(m.rows, 1 << 20)), 256, 0, st>>>(m.p, m.stride, m.rows, m.cols, out,
                                                                             pitch);
    m.p = out, m.stride = pitch;
    return tide::op_launched("ce: aligned rows");
}

}  // namespace

extern "C" {

int64_t tide_ce_loss_workspace(const tide_ce_t *ce)
{
    tide::record_error("");
    return check_desc(ce) ? -1 : layout_of(ce, false).bytes;
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
    const Layout l = layout_of(ce, false);
    s = check_workspace(workspace, workspace_bytes, l.bytes);
    if (!s)
        s = get_ready<kStats>();
    if (s)
        return s;
    const tide::NvtxRange range("tide_ce_loss");
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    char *ws = static_cast<char *>(workspace);
    const int64_t T = ce->tokens, V = ce->vocab, H = ce->hidden;
    Mat x = {static_cast<const bf16 *>(ce->x), T, H, ce->x_stride};
    Mat w = {static_cast<const bf16 *>(ce->weight), V, H, ce->weight_stride};
    s = align_rows(x, ws, l.x, l.pitch, st);
    if (!s)
        s = align_rows(w, ws, l.w, l.pitch, st);
    if (s)
        return s;
    Gemm g = base(ce);
    g.part = reinterpret_cast<float2 *>(ws + l.part);
    s = launch<kStats>(g, w, x, "ce_loss", st);
    if (s)
        return s;
    int rows = 32;  // few rows: more slices of each, and more blocks
    while (rows > 1 && T / rows < 128)
        rows /= 2;
    join_kernel<<<unsigned((T + rows - 1) / rows), 256, 0, st>>>(g.part, 2 * g.tiles_m, T, rows, g.y, x.p, x.stride, w.p,
                                                               w.stride, int(H), loss, lse);
    return tide::op_launched("ce_loss: join");
}

int64_t tide_ce_grad_workspace(const tide_ce_t *ce)
{
    tide::record_error("");
    return check_desc(ce) ? -1 : layout_of(ce, true).bytes;
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
    if (!stride_ok(ce->tokens, dx_stride, ce->hidden) || !stride_ok(ce->vocab, dweight_stride, ce->hidden))
        return op_fail(TIDE_ERR_INVALID_ARG, "dx_stride %lld, dweight_stride %lld for hidden %lld",
                       (long long)dx_stride, (long long)dweight_stride, (long long)ce->hidden);
    const Layout l = layout_of(ce, true);
    s = check_workspace(workspace, workspace_bytes, l.bytes);
    if (!s)
        s = get_ready<kDz, kAdd, kStore>();
    if (s)
        return s;
    const tide::NvtxRange range("tide_ce_grad");
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    char *ws = static_cast<char *>(workspace);
    const int64_t T = ce->tokens, V = ce->vocab, H = ce->hidden;
    if (T == 0) {  // nothing to sum
        const cudaError_t e = cudaMemset2DAsync(dweight, size_t(V > 1 ? dweight_stride : H) * 2, 0, size_t(H) * 2,
                                                size_t(V), st);
        return e == cudaSuccess ? TIDE_OK : op_fail(TIDE_ERR_CUDA, "ce_grad: %s", cudaGetErrorString(e));
    }
    Mat x = {static_cast<const bf16 *>(ce->x), T, H, ce->x_stride};
    Mat w = {static_cast<const bf16 *>(ce->weight), V, H, ce->weight_stride};
    bf16 *dz = reinterpret_cast<bf16 *>(ws + l.dz), *rows = reinterpret_cast<bf16 *>(ws + l.x);
    float *acc = reinterpret_cast<float *>(ws + l.acc), *unit = reinterpret_cast<float *>(ws + l.unit);
    float *miss = reinterpret_cast<float *>(ws + l.miss);
    s = align_rows(w, ws, l.w, l.pitch, st);
    if (s)
        return s;
    const bool aligned = H % 8 == 0 && rows_aligned(x.p, x.stride, T);  // w is, here
    (aligned ? prepare_kernel<true> : prepare_kernel<false>)<<<unsigned(1 + T), 256, 0, st>>>(
        dloss, base(ce).y, T, unit, x.p, x.stride, w.p, w.stride, int(H), lse, miss, rows, l.pitch);
    s = tide::op_launched("ce_grad: rows");
    x.p = rows, x.stride = l.pitch;
    for (int64_t v0 = 0; !s && v0 < V; v0 += l.piece) {
        const int64_t n = std::min(l.piece, V - v0);
        const Mat wp = {w.p + v0 * w.stride, n, H, w.stride}, dzp = {dz, T, n, l.piece, l.piece};
        Gemm g = base(ce);
        g.v0 = v0;
        g.lse = lse, g.dloss = dloss, g.unit = unit, g.miss = miss;
        s = make_map(&g.c, dzp, 32, 32);
        if (!s)
            s = launch<kDz>(g, wp, x, "ce_grad: dz", st);
        if (s)
            return s;
        g.first = v0 == 0, g.splits = l.splits, g.tile_n = l.tile_n;
        s = make_acc_map(&g.c, acc, l.splits, H, T, l.acc_pitch);
        if (!s)
            s = launch<kAdd>(g, wp, dzp, "ce_grad: dx", st);
        if (s)
            return s;
        bf16 *dwp = static_cast<bf16 *>(dweight) + v0 * dweight_stride;
        g.out = dwp, g.out_stride = dweight_stride;
        g.out_tiles = H % 8 == 0 && rows_aligned(g.out, dweight_stride, V);  // tiles are stored by 16 bytes
        // Rows on other boundaries go through the weight's aligned copy, if there is one: this piece of it has been
        // used.  Single stores from the result warps take eight times as long (20 x 50001 x 2047: 989 us in all, 278 this way).
        const bool staged = !g.out_tiles && l.w >= 0;
        if (staged) {
            g.out = reinterpret_cast<bf16 *>(ws + l.w) + v0 * l.pitch, g.out_stride = l.pitch;
            g.out_tiles = 1;
        }
        s = launch<kStore>(g, dzp, x, "ce_grad: dweight", st);
        if (!s && staged) {
            unalign_kernel<<<unsigned(std::min<int64_t>(n, 1 << 20)), 256, 0, st>>>(g.out, l.pitch, n, H, dwp,
                                                                                  dweight_stride);
            s = tide::op_launched("ce_grad: dweight's rows");
        }
    }
    if (s)
        return s;
    round_kernel<<<dim3(unsigned((T + 31) / 32), unsigned((H + 31) / 32)), 256, 0, st>>>(
        acc, l.splits, T, H, l.acc_pitch, unit, static_cast<bf16 *>(dx), dx_stride);
    return tide::op_launched("ce_grad: rounding");
}

tide_status_t tide_ops_device_status(void *stream)
{
    tide::record_error("");
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    int seen = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(&seen, g_timed_out, sizeof seen, 0, cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess)
        e = cudaStreamSynchronize(st);
    if (e == cudaSuccess && seen) {
        const int zero = 0;
        e = cudaMemcpyToSymbolAsync(g_timed_out, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, st);
        if (e == cudaSuccess)
            e = cudaStreamSynchronize(st);
    }
    if (e != cudaSuccess)
        return op_fail(TIDE_ERR_CUDA, "operators' status: %s", cudaGetErrorString(e));
    return seen ? op_fail(TIDE_ERR_TIMEOUT, "a bounded device-side wait expired") : TIDE_OK;
}

}  // extern "C"
