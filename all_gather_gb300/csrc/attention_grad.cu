// Gradient of softmax attention over packed sequences.
//
//   p = exp(s - lse),  delta_r = do_r o_r,  dp_rc = do_r v_c,  ds = p (dp - delta),
//   dq_r = scale sum_c ds_rc k_c,  dk_c = scale sum_r ds_rc q_r,  dv_c = sum_r p_rc do_r
//
// Two passes over the pairs of tiles, one that holds 128 keys and sums dk and
// dv over the rows that see them (and over the query heads that share them),
// one that holds 128 rows and sums dq over their keys.  That makes seven
// products of a pair where five would do, s and dp twice, but every sum has one
// owner: no partial result goes through memory, nothing is added out of order,
// and no operand is written to shared memory by threads.
//
// Both are one kernel.  A block holds two resident tiles (k and v, or q and do),
// and two rings bring the streamed ones (X: q, or k; Y: do, or v):
//   S = R0 X^T, D = R1 Y^T  in tensor memory, a resident row a lane;
//   P = exp(S - lse) and dS = P (D - delta), made by eight warps, a row a
//   thread and half the columns, and written as bf16 over S and D, from where
//   the tensor cores take them as operands:  dv += P Y,  dk or dq += dS X.
// While P is made the tensor cores work on dS of the step before, and the other
// way around.
//
// Masks, tiles and rows that are not finite: as in the forward pass.
#include "attention.h"

namespace {

using namespace tide::attn;
using tide::op_aligned;
using tide::op_fail;
namespace um = tide::umma;

constexpr int kThreads = 384;  // eight warps for the elements, four that fetch, multiply, fetch lse and delta, and idle
constexpr int kRowRegs = 224, kOtherRegs = 56;  // registers a thread, of 168 at the launch: (2 * 224 + 56) * 128 = 168 * 384
constexpr int kClaims = 8;     // of a block's last items, kept for a wait that runs out

// Set when a bounded wait runs out.
__device__ int g_timed_out;

struct Backward {
    CUtensorMap r0, r1, x, y;  // keys: k, v, q, do; rows: q, do, k, v
    Problem pr;
    Heads q, k, v, dout;
    Heads out0, out1;  // keys: dv, dk; rows: -, dq
    const float *lse, *delta;
    int items;  // tiles times heads
    uint64_t wait_ns;
    int skip_fill;  // TIDE_DEBUG_SKIP_FILL
};

struct Item {
    int number;  // -1: no more
    Tiles tiles;  // streamed
};
template <bool KEYS>
__device__ __forceinline__ void place_of(const Backward &f, int item, int &head, int &t0)
{
    const int heads = KEYS ? f.pr.Hk : f.pr.Hq, tile = item / heads;  // the longest of a causal sequence first
    head = item % heads;
    t0 = (KEYS ? tile : f.items / heads - 1 - tile) * kTile;
}
template <bool KEYS>
__device__ __forceinline__ Span span_of(const Problem &pr, int t)
{
    return KEYS ? pr.rows_of(t) : pr.keys_of(t);
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

// One output row a lane (dv, dk or dq of token t), by itself, over what it sees only; lanes with an empty span take no
// part.  Columns [d0, d1).  Ends early where every element is NaN already.
enum Which { kDv, kDk, kDq };
__device__ __forceinline__ void row_alone(Which which, const Backward &f, int t, int head, Span see, int d0, int d1, bf16 *out)
{
    const Problem &pr = f.pr;
    const Span all = warp_span(see);
    const bool mine = see.a < see.b;
    const int group = pr.Hq / pr.Hk, D = pr.D;
    const float c = pr.scale * kLog2e;
    const int h0 = which == kDq ? head : head * group, h1 = which == kDq ? head + 1 : h0 + group;
#pragma unroll 1
    for (int d = d0; d < d1; d += 16) {
        float acc[16] = {};
        bool more = mine;
#pragma unroll 1
        for (int h = h0; h < h1; ++h)
#pragma unroll 1
            for (int j = all.a; j < all.b && __any_sync(kAll, more); ++j) {
                if (j < see.a || j >= see.b)
                    continue;
                const int r = which == kDq ? t : j, key = which == kDq ? j : t, hk = h / group;
                const int64_t i = int64_t(h) * pr.T + r;
                const float p = exp2_fast(fmaf(dot_row(f.q.row(r, h), f.k.row(key, hk), D), c, -f.lse[i] * kLog2e));
                const float w = which == kDv ? p : p * (dot_row(f.dout.row(r, h), f.v.row(key, hk), D) - f.delta[i]);
                const bf16 *from = which == kDv ? f.dout.row(r, h) : which == kDk ? f.q.row(r, h) : f.k.row(key, hk);
                more = false;
#pragma unroll
                for (int e = 0; e < 16; e += 8) {
                    float x[8];
                    if (d + e < d1)
                        tide::load8(from + d + e, x);
#pragma unroll
                    for (int m = 0; m < 8; ++m)
                        if (d + e < d1) {
                            acc[e + m] = fmaf(w, x[m], acc[e + m]);
                            more = more || !isnan(acc[e + m]);
                        }
                }
            }
#pragma unroll
        for (int e = 0; e < 16; e += 8)
            if (mine && d + e < d1) {
                float x[8];
#pragma unroll
                for (int m = 0; m < 8; ++m)
                    x[m] = which == kDv ? acc[e + m] : acc[e + m] * pr.scale;
                tide::store8(out + d + e, x);
            }
    }
}

// W: columns of a head in shared and tensor memory, 64 or 128.  KEYS: the resident tile is one of keys.
template <int W, bool KEYS>
__global__ void __launch_bounds__(kThreads, 1) backward_kernel(const __grid_constant__ Backward f)
{
    constexpr int kHalves = W / 64, kTileBytes = kHalves * kHalf;
    // X waits from S to dS X, Y at most from D to P Y; at W = 128 five stages are what fits
    constexpr int kXs = 3, kYs = 2;
    constexpr uint32_t kS = 0, kD = 128, kAcc0 = 256, kAcc1 = 384;  // columns of tensor memory; rows: a second D at kAcc0
    extern __shared__ uint8_t smem_raw[];
    const uint32_t resident = (um::smem_addr(smem_raw) + 1023) / 1024 * 1024;
    const uint32_t xs = resident + 2 * kTileBytes, ys = xs + kXs * kTileBytes;
    __shared__ uint64_t bars[2 * kXs + 2 * kYs + 23];
    __shared__ alignas(16) uint4 answer;
    __shared__ alignas(16) float lse_of[2][kTile], delta_of[kTile];  // keys: of a step's rows, -lse in log2, and -delta
    __shared__ Item items[2];
    __shared__ int claims[kClaims], claimed, done[8];  // done: items of each of the eight warps
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int gave_up;
    const uint32_t x_full = um::smem_addr(bars), x_empty = x_full + 8 * kXs, y_full = x_empty + 8 * kXs,
                   y_empty = y_full + 8 * kYs, rest = y_empty + 8 * kYs;
    const uint32_t r_full = rest, r_empty = rest + 8, s_full = rest + 16, p_ready = rest + 24, d_full = rest + 32,
                   ds_ready = rest + 48, acc_full = rest + 64, acc_free = rest + 72, item_full = rest + 80,
                   item_empty = rest + 96, lse_full = rest + 112, lse_empty = rest + 128, delta_full = rest + 144,
                   delta_empty = rest + 152, asked = rest + 160, drained = rest + 168, never = rest + 176;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const Problem &pr = f.pr;
    const int group = pr.Hq / pr.Hk;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kXs; ++i)
            um::mbar_init(x_full + 8 * i, 1), um::mbar_init(x_empty + 8 * i, 1);
        for (int i = 0; i < kYs; ++i)
            um::mbar_init(y_full + 8 * i, 1), um::mbar_init(y_empty + 8 * i, 1);
        for (int i = 0; i < 2; ++i) {
            um::mbar_init(d_full + 8 * i, 1);
            um::mbar_init(ds_ready + 8 * i, 8);  // rows: a warp may be a step ahead of another one
            um::mbar_init(item_full + 8 * i, 1);
            um::mbar_init(item_empty + 8 * i, KEYS ? 10 : 9);
            um::mbar_init(lse_full + 8 * i, 1);
            um::mbar_init(lse_empty + 8 * i, 8);
        }
        um::mbar_init(r_full, 1);
        um::mbar_init(r_empty, 1);
        um::mbar_init(s_full, 1);
        um::mbar_init(p_ready, 8);
        um::mbar_init(acc_full, 1);
        um::mbar_init(acc_free, 8);
        um::mbar_init(delta_full, 1);
        um::mbar_init(delta_empty, 8);
        um::mbar_init(asked, 1);
        um::mbar_init(drained, 1);
        um::mbar_init(never, 1);
        um::fence_barrier_init();
        gave_up = 0, claimed = 0, answer = make_uint4(0, 0, 0, 0);
        um::fence_copies();
        um::prefetch_map(&f.r0);
        um::prefetch_map(&f.r1);
        um::prefetch_map(&f.x);
        um::prefetch_map(&f.y);
    }
    if (threadIdx.x < 8)
        done[threadIdx.x] = 0;
    if (warp == 9)
        um::tmem_alloc_own(um::smem_addr(&tmem_slot), 512);
    um::fence_before();
    __syncthreads();
    um::fence_after();
    const uint32_t tmem = tmem_slot;
    auto wait = [&](uint32_t bar, uint32_t parity) { return um::mbar_wait(bar, parity, &gave_up, f.wait_ns); };

    if (warp >= 8) {
        um::fewer_registers<kOtherRegs>();
        if (warp == 8) {
            const bool leader = um::elected();
            int number = blockIdx.x, slot = 0, turn = 0, xi = 0, x_phase = 0, yi = 0, y_phase = 0, taken = 0;
            int x_fills = 0, y_fills = 0, r_fills = 0;  // copies under way at most: the last of each place
            bool ok = true;
            while (ok) {
                if (lane == 0) {
                    claims[taken % kClaims] = number;
                    claimed = taken + 1;
                }
                ++taken;
                if (leader)
                    um::ask_next_block(um::smem_addr(&answer), asked);
                int head, t0;
                place_of<KEYS>(f, number, head, t0);
                // which tiles are streamed: what the resident ones see or are seen by, four tokens a lane
                Span see = {0x7fffffff, 0};
#pragma unroll 1
                for (int t = t0 + lane; t < t0 + kTile; t += 32) {
                    const Span s = span_of<KEYS>(pr, t);
                    if (s.a < s.b)
                        see = {min(see.a, s.a), max(see.b, s.b)};
                }
                const Tiles tiles = tiles_of(warp_span(see));
                if (!(ok = wait(item_empty + 8 * slot, turn ^ 1)))
                    break;
                if (lane == 0) {
                    items[slot] = {number, tiles};
                    um::mbar_arrive(item_full + 8 * slot);
                }
                if (++slot == 2)
                    slot = 0, turn ^= 1;
                if (tiles.a < tiles.b) {
                    if (!(ok = wait(r_empty, (r_fills & 1) ^ 1)))
                        break;
                    if (leader) {
                        um::mbar_expect(r_full, 2 * kTileBytes);
                        load_tile(resident, &f.r0, kHalves, head, t0, r_full);
                        load_tile(resident + kTileBytes, &f.r1, kHalves, head, t0, r_full);
                    }
                    ++r_fills;
                }
                const int h0 = KEYS ? head * group : head / group, h1 = KEYS ? h0 + group : h0 + 1;
                bool skip = f.skip_fill && number == 0;  // this item's first streamed tile never comes
                for (int h = h0; ok && h < h1; ++h)
                    for (int j = tiles.a; j < tiles.b; ++j) {
                        if (!(ok = wait(x_empty + 8 * xi, x_phase ^ 1)))
                            break;
                        if (skip) {
                            ok = wait(never, 0);  // nothing arrives there
                            break;
                        }
                        if (leader) {
                            um::mbar_expect(x_full + 8 * xi, kTileBytes);
                            load_tile(xs + xi * kTileBytes, &f.x, kHalves, h, j * kTile, x_full + 8 * xi);
                        }
                        ++x_fills;
                        if (++xi == kXs)
                            xi = 0, x_phase ^= 1;
                        if (!(ok = wait(y_empty + 8 * yi, y_phase ^ 1)))
                            break;
                        if (leader) {
                            um::mbar_expect(y_full + 8 * yi, kTileBytes);
                            load_tile(ys + yi * kTileBytes, &f.y, kHalves, h, j * kTile, y_full + 8 * yi);
                        }
                        ++y_fills;
                        if (++yi == kYs)
                            yi = 0, y_phase ^= 1;
                    }
                if (!ok || !(ok = wait(asked, (taken - 1) & 1)))
                    break;
                number = um::next_block(um::smem_addr(&answer));
                um::fence_copies();
                __syncwarp();
                if (number < 0)
                    break;
            }
            if (ok && (ok = wait(item_empty + 8 * slot, turn ^ 1))) {
                if (lane == 0) {
                    items[slot].number = -1;
                    um::mbar_arrive(item_full + 8 * slot);
                }
            }
            if (!ok) {
                // The answer that is under way, and the copies: neither may find the block gone.
                auto land = [&](uint32_t bar, uint32_t parity) {
                    const uint64_t began = um::now_ns();
                    while (!um::mbar_try(bar, parity) && um::now_ns() - began < f.wait_ns) {
                    }
                };
                land(asked, (taken - 1) & 1);
                const int more = um::next_block(um::smem_addr(&answer));
                if (lane == 0 && more >= 0 && more != number) {
                    claims[taken % kClaims] = more;
                    claimed = taken + 1;
                }
                for (int i = max(0, x_fills - kXs); i < x_fills; ++i)
                    land(x_full + 8 * (i % kXs), (i / kXs) & 1);
                for (int i = max(0, y_fills - kYs); i < y_fills; ++i)
                    land(y_full + 8 * (i % kYs), (i / kYs) & 1);
                if (r_fills)
                    land(r_full, (r_fills - 1) & 1);
            }
            __syncwarp();
        } else if (warp == 9) {
            const bool leader = um::elected();
            const int dn = (pr.D + 15) / 16 * 16, ksteps = dn / 16;
            const uint32_t idesc_s = um::instr_desc(kTile, kTile, false, false);
            const uint32_t idesc_acc = um::instr_desc(kTile, dn, false, true);
            // rows of a resident tile times those of a streamed one
            auto pairs = [&](uint32_t d, uint32_t r, uint32_t streamed, uint32_t bar) {
                um::fence_after();
                if (leader) {
                    const uint64_t a = um::operand_desc(r, false, 0), b = um::operand_desc(streamed, false, 0);
                    for (int i = 0; i < ksteps; ++i) {
                        const uint32_t off = ((i % 4) * 32 + (i / 4) * kHalf) >> 4;
                        um::mma_own(tmem + d, a + off, b + off, idesc_s, i > 0);
                    }
                    um::mma_commit_own(bar);
                }
            };
            // a sum over a streamed tile's rows, with P or dS, whose halves are 64 columns apart
            auto sum = [&](uint32_t d, uint32_t p, uint32_t streamed, bool add, uint32_t bar) {
                um::fence_after();
                if (leader) {
                    const uint64_t b = um::operand_desc(streamed, true, kHalf);
#pragma unroll
                    for (int i = 0; i < kTile / 16; ++i)
                        um::mma_own_tmem(tmem + d, tmem + p + (i / 4) * 64 + i % 4 * 8, b + i * (2048 >> 4), idesc_acc,
                                         add || i > 0);
                    um::mma_commit_own(bar);
                }
            };
            int slot = 0, turn = 0, x_of_s = 0, xs_phase = 0, x_of_sum = 0, y_of_d = 0, yd_phase = 0, y_of_sum = 0;
            uint32_t r_phase = 0, p_phase = 0, ds_phase = 0, acc_phase = 0;
            bool ok = true;
            while (ok) {
                if (!(ok = wait(item_full + 8 * slot, turn)))
                    break;
                const Item it = items[slot];
                __syncwarp();
                if (lane == 0)
                    um::mbar_arrive(item_empty + 8 * slot);
                if (++slot == 2)
                    slot = 0, turn ^= 1;
                if (it.number < 0)
                    break;
                const int steps = (it.tiles.b - it.tiles.a) * (KEYS ? group : 1);
                if (steps == 0)
                    continue;
                if (!(ok = wait(r_full, r_phase)))
                    break;
                r_phase ^= 1;
                auto make_s = [&] {
                    if (!(ok = wait(x_full + 8 * x_of_s, xs_phase)))
                        return;
                    pairs(kS, resident, xs + x_of_s * kTileBytes, s_full);
                    if (++x_of_s == kXs)
                        x_of_s = 0, xs_phase ^= 1;
                };
                auto make_d = [&](int n) {
                    if (!(ok = wait(y_full + 8 * y_of_d, yd_phase)))
                        return;
                    const int b = KEYS ? 0 : n & 1;
                    pairs(kD + b * 128, resident + kTileBytes, ys + y_of_d * kTileBytes, d_full + 8 * b);
                    if (!KEYS && leader)  // its only use
                        um::mma_commit_own(y_empty + 8 * y_of_d);
                    if (n == steps - 1 && leader)
                        um::mma_commit_own(r_empty);
                    if (++y_of_d == kYs)
                        y_of_d = 0, yd_phase ^= 1;
                };
                make_s();
                if (ok)
                    make_d(0);
                for (int n = 0; ok && n < steps; ++n) {
                    if (n == 0) {
                        if (!(ok = wait(acc_free, acc_phase ^ 1)))
                            break;
                        acc_phase ^= 1;
                    }
                    if (!(ok = wait(p_ready, p_phase)))
                        break;
                    p_phase ^= 1;
                    if (KEYS) {
                        sum(kAcc0, kS, ys + y_of_sum * kTileBytes, n > 0, y_empty + 8 * y_of_sum);
                        if (++y_of_sum == kYs)
                            y_of_sum = 0;
                    }
                    if (n + 1 < steps) {
                        make_s();
                        if (!KEYS && ok)
                            make_d(n + 1);
                        if (!ok)
                            break;
                    }
                    const int b = KEYS ? 0 : n & 1;
                    if (!(ok = wait(ds_ready + 8 * b, ds_phase >> b & 1)))
                        break;
                    ds_phase ^= 1 << b;
                    sum(kAcc1, kD + b * 128, xs + x_of_sum * kTileBytes, n > 0, x_empty + 8 * x_of_sum);
                    if (++x_of_sum == kXs)
                        x_of_sum = 0;
                    if (KEYS && n + 1 < steps)
                        make_d(n + 1);
                }
                if (ok && leader)
                    um::mma_commit_own(acc_full);
            }
            __syncwarp();
            if (leader) {  // nothing may be under way when the accumulators go
                um::mma_commit_own(drained);
                const uint64_t began = um::now_ns();
                while (!um::mbar_try(drained, 0) && um::now_ns() - began < f.wait_ns) {
                }
            }
            __syncwarp();
        } else if (KEYS && warp == 10) {
            int slot = 0, turn = 0, at = 0;
            uint32_t phase = 0, delta_phase = 0;
            bool ok = true;
            while (ok) {
                if (!(ok = wait(item_full + 8 * slot, turn)))
                    break;
                const Item it = items[slot];
                __syncwarp();
                if (lane == 0)
                    um::mbar_arrive(item_empty + 8 * slot);
                if (++slot == 2)
                    slot = 0, turn ^= 1;
                if (it.number < 0)
                    break;
                int head, t0;
                place_of<KEYS>(f, it.number, head, t0);
                for (int h = head * group; ok && h < (head + 1) * group; ++h)
                    for (int j = it.tiles.a; j < it.tiles.b; ++j) {
                        float l[4], d[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int r = j * kTile + i * 32 + lane;
                            const int64_t from = int64_t(h) * pr.T + r;
                            l[i] = r < pr.T ? f.lse[from] : 0.f;
                            d[i] = r < pr.T ? f.delta[from] : 0.f;
                        }
                        if (!(ok = wait(lse_empty + 8 * at, phase ^ 1)))
                            break;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            lse_of[at][i * 32 + lane] = -l[i] * kLog2e;
                        __syncwarp();
                        if (lane == 0)
                            um::mbar_arrive(lse_full + 8 * at);
                        if (!(ok = wait(delta_empty, delta_phase ^ 1)))
                            break;
                        delta_phase ^= 1;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            delta_of[i * 32 + lane] = -d[i];
                        __syncwarp();
                        if (lane == 0)
                            um::mbar_arrive(delta_full);
                        if (++at == 2)
                            at = 0, phase ^= 1;
                    }
            }
        }
    } else {
        um::more_registers<kRowRegs>();
        const int half = warp / 4, quarter = warp % 4;
        const uint32_t lanes = tmem + (uint32_t(quarter * 32) << 16);
        const float c = pr.scale * kLog2e;
        int slot = 0, turn = 0, at = 0;
        uint32_t s_phase = 0, d_phase = 0, lse_phase = 0, delta_phase = 0, acc_phase = 0;
        bool ok = true;
        for (;;) {
            if (!wait(item_full + 8 * slot, turn))
                break;
            const Item it = items[slot];
            __syncwarp();
            if (lane == 0)
                um::mbar_arrive(item_empty + 8 * slot);
            if (++slot == 2)
                slot = 0, turn ^= 1;
            if (it.number < 0)
                break;
            int head, t0;
            place_of<KEYS>(f, it.number, head, t0);
            const int t = t0 + quarter * 32 + lane;
            const Span see = span_of<KEYS>(pr, t);
            float lse2 = 0.f, delta = 0.f;  // rows: negated
            if (!KEYS && t < pr.T) {
                const int64_t from = int64_t(head) * pr.T + t;
                lse2 = -f.lse[from] * kLog2e;
                delta = -f.delta[from];
            }
            __syncwarp();  // the search for the sequence took lanes apart
            const int steps = (it.tiles.b - it.tiles.a) * (KEYS ? group : 1);
            int j = it.tiles.a;
            for (int n = 0; n < steps; ++n) {
                const int first = j * kTile + half * 64;  // token of this thread's first column
                if (++j == it.tiles.b)
                    j = it.tiles.a;
                const int a = see.a - first, b = see.b - first;
                const bool masked = __any_sync(kAll, a > 0 || b < 64);
                if (!(ok = wait(s_full, s_phase)))
                    break;
                s_phase ^= 1;
                um::fence_after();
                uint32_t v[2][32];
                um::tmem_load32(lanes + kS + half * 64, v[0]);
                um::tmem_load32(lanes + kS + half * 64 + 32, v[1]);
                um::tmem_wait_load();
                if (!KEYS) {  // S is not written over: free for the next one
                    um::fence_before();
                    __syncwarp();
                    if (lane == 0)
                        um::mbar_arrive(p_ready);
                } else if (!(ok = wait(lse_full + 8 * at, lse_phase))) {
                    break;
                }
                float2 p[32];
                const float2 cc = make_float2(c, c);
#pragma unroll
                for (int x = 0; x < 32; ++x) {
                    float2 l = make_float2(lse2, lse2);
                    if (KEYS)
                        l = *reinterpret_cast<const float2 *>(&lse_of[at][half * 64 + 2 * x]);
                    p[x] = um::fma2(make_float2(__uint_as_float(v[x / 16][x % 16 * 2]),
                                                __uint_as_float(v[x / 16][x % 16 * 2 + 1])), cc, l);
                    p[x].x = exp2_fast(p[x].x), p[x].y = exp2_fast(p[x].y);
                }
                if (masked) {
#pragma unroll
                    for (int x = 0; x < 32; ++x) {
                        p[x].x = 2 * x >= a && 2 * x < b ? p[x].x : 0.f;
                        p[x].y = 2 * x + 1 >= a && 2 * x + 1 < b ? p[x].y : 0.f;
                    }
                }
                if (KEYS) {
                    uint32_t w[32];
#pragma unroll
                    for (int x = 0; x < 32; ++x)
                        w[x] = tide::pack_bf16(p[x].x, p[x].y);
                    um::tmem_store32(lanes + kS + half * 64, w);
                    um::tmem_wait_store();
                    um::fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        um::mbar_arrive(p_ready);
                        um::mbar_arrive(lse_empty + 8 * at);
                    }
                    if (++at == 2)
                        at = 0, lse_phase ^= 1;
                    if (!(ok = wait(delta_full, delta_phase)))
                        break;
                    delta_phase ^= 1;
                }
                const int buf = KEYS ? 0 : n & 1;
                if (!(ok = wait(d_full + 8 * buf, d_phase >> buf & 1)))
                    break;
                d_phase ^= 1 << buf;
                um::fence_after();
                const uint32_t d_at = lanes + kD + buf * 128 + half * 64;
                um::tmem_load32(d_at, v[0]);
                um::tmem_load32(d_at + 32, v[1]);
                um::tmem_wait_load();
                uint32_t w[32];
#pragma unroll
                for (int x = 0; x < 32; ++x) {
                    float2 d = make_float2(delta, delta);
                    if (KEYS)
                        d = *reinterpret_cast<const float2 *>(&delta_of[half * 64 + 2 * x]);
                    d = um::add2(make_float2(__uint_as_float(v[x / 16][x % 16 * 2]),
                                             __uint_as_float(v[x / 16][x % 16 * 2 + 1])), d);
                    p[x] = um::mul2(p[x], d);
                }
                if (masked) {  // 0 times what is not finite
#pragma unroll
                    for (int x = 0; x < 32; ++x) {
                        p[x].x = 2 * x >= a && 2 * x < b ? p[x].x : 0.f;
                        p[x].y = 2 * x + 1 >= a && 2 * x + 1 < b ? p[x].y : 0.f;
                    }
                }
#pragma unroll
                for (int x = 0; x < 32; ++x)
                    w[x] = tide::pack_bf16(p[x].x, p[x].y);
                um::tmem_store32(d_at, w);
                um::tmem_wait_store();
                um::fence_before();
                __syncwarp();
                if (lane == 0) {
                    um::mbar_arrive(ds_ready + 8 * buf);
                    if (KEYS)
                        um::mbar_arrive(delta_empty);
                }
            }
            if (!ok)
                break;
            // Keys: the first four warps have dv, the others dk; rows: half the columns of dq each.
            constexpr int kCols = KEYS ? W : W / 2;
            const int d0 = KEYS ? 0 : half * kCols;
            const bool some = see.a < see.b;
            bf16 *out = (KEYS && half == 0 ? f.out0 : f.out1).row(min(t, pr.T - 1), head);
            if (steps) {
                if (!(ok = wait(acc_full, acc_phase)))
                    break;
                acc_phase ^= 1;
                um::fence_after();
                uint32_t o[kCols / 32][32];
#pragma unroll
                for (int i = 0; i < kCols / 32; ++i)
                    um::tmem_load32(lanes + (KEYS && half == 0 ? kAcc0 : kAcc1) + d0 + 32 * i, o[i]);
                um::tmem_wait_load();
                um::fence_before();
                __syncwarp();
                if (lane == 0)
                    um::mbar_arrive(acc_free);
                const float by = KEYS && half == 0 ? 1.f : pr.scale;
                bool odd = false;  // not finite
#pragma unroll
                for (int d = 0; d < kCols; d += 8) {
                    float x[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        x[i] = __uint_as_float(o[d / 32][d % 32 + i]);
                        odd = odd || !(fabsf(x[i]) < INFINITY);
                        x[i] = some ? x[i] * by : 0.f;
                    }
                    if (d0 + d < pr.D && t < pr.T)
                        tide::store8(out + d0 + d, x);
                }
                odd = odd && some;
                if (__any_sync(kAll, odd))
                    row_alone(!KEYS ? kDq : half ? kDk : kDv, f, odd ? t : 0, head, odd ? see : Span{0, 0}, d0,
                              min(d0 + kCols, pr.D), out);
            } else if (t < pr.T) {
                const float x[8] = {};
                for (int d = d0; d < min(d0 + kCols, pr.D); d += 8)
                    tide::store8(out + d, x);
            }
            if (lane == 0)
                ++done[warp];
        }
    }
    um::fence_before();
    __syncthreads();
    um::fence_after();
    if (gave_up) {  // what was claimed and not finished is NaN
        if (threadIdx.x == 0)
            g_timed_out = 1;
        if (warp < 8)
            for (int i = done[warp]; i < claimed; ++i) {
                int head, t0;
                place_of<KEYS>(f, claims[i % kClaims], head, t0);
                const int t = t0 + threadIdx.x % kTile, half = warp / 4;
                if (t >= pr.T)
                    continue;
                bf16 *out = (KEYS && half == 0 ? f.out0 : f.out1).row(t, head);
                const int d0 = KEYS ? 0 : half * (W / 2), d1 = KEYS ? pr.D : min(d0 + W / 2, pr.D);
                for (int d = d0; d < d1; ++d)
                    out[d] = __float2bfloat16_rn(__int_as_float(0x7fffffff));
            }
    }
    if (warp == 9)
        um::tmem_free_own(tmem, 512);
}

template <int W, bool KEYS>
tide_status_t launch(const Backward &f, cudaStream_t st)
{
    constexpr int smem = 7 * (W / 64) * kHalf + 1024;  // 1024: alignment
    const cudaError_t e = tide::op_allow_smem<backward_kernel<W, KEYS>>(smem);
    if (e != cudaSuccess)
        return op_fail(TIDE_ERR_CUDA, "attention_grad: %s", cudaGetErrorString(e));
    backward_kernel<W, KEYS><<<unsigned(f.items), kThreads, smem, st>>>(f);
    return tide::op_launched("attention_grad");
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
    if (!tide::encode_tiled())
        return op_fail(TIDE_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
    const tide::NvtxRange range("tide_attention_grad");
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    float *delta = static_cast<float *>(workspace);
    Backward f = {};
    f.pr = problem_of(at);
    const Problem &p = f.pr;
    f.q = heads_of(at, q, p.Hq), f.k = heads_of(at, k, p.Hk), f.v = heads_of(at, v, p.Hk);
    f.dout = heads_of(at, dout, p.Hq);
    f.lse = lse, f.delta = delta;
    f.wait_ns = wait_of(at);
    f.skip_fill = (at->debug & TIDE_DEBUG_SKIP_FILL) != 0;
    CUtensorMap mq, mk, mv, md;
    s = heads_map(&mq, f.q, p.T, p.Hq, p.D);
    if (!s)
        s = heads_map(&mk, f.k, p.T, p.Hk, p.D);
    if (!s)
        s = heads_map(&mv, f.v, p.T, p.Hk, p.D);
    if (!s)
        s = heads_map(&md, f.dout, p.T, p.Hq, p.D);
    if (s)
        return s;
    delta_kernel<<<unsigned((int64_t(p.T) * p.Hq + 15) / 16), 256, 0, st>>>(p, f.dout, heads_of(at, o, p.Hq), delta);
    s = tide::op_launched("attention_grad: delta");
    if (s)
        return s;
    const int tiles = (p.T + kTile - 1) / kTile;
    f.r0 = mk, f.r1 = mv, f.x = mq, f.y = md;
    f.out0 = heads_of(at, dv, p.Hk), f.out1 = heads_of(at, dk, p.Hk);
    f.items = tiles * p.Hk;
    s = p.D <= 64 ? launch<64, true>(f, st) : launch<128, true>(f, st);
    if (s)
        return s;
    f.r0 = mq, f.r1 = md, f.x = mk, f.y = mv;
    f.out1 = heads_of(at, dq, p.Hq);
    f.items = tiles * p.Hq;
    return p.D <= 64 ? launch<64, false>(f, st) : launch<128, false>(f, st);
}

}  // extern "C"
