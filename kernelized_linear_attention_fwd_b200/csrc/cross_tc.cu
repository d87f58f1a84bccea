// Cross attention with KATA weights on the tensor cores (bf16, d in {16, 32, 64},
// read as 64 by the tensor maps, which fill the columns past d with zeros).
//
//   s = q.k,  w = s^2,  l = sum_s w,  y = (sum_s w v) / l              (0 if l = 0)
//
// and, with D = dy.y and p = dy.v for the gradient dy of y,
//
//   ds = 2 s (p - D) / l,   dq = sum_s ds k,   dk = sum_t ds q,   dv = sum_t (w / l) dy.
//
// One kernel, three modes.  Each keeps 128-row tiles of its accumulators in
// tensor memory, walks the other axis in blocks, and forms per block
//
//   forward  rows = queries  S = Q K^T (128 keys)                     O  += bf16(w) V
//   dq       rows = queries  S = Q K^T, P = dY V^T (64 keys)          dQ += bf16(s (p - D)) K
//   dkv      rows = keys     S = K Q^T, P = V dY^T (64 queries)       dV += bf16(w / l) dY
//                                                                     dK += bf16(ds) Q
//
// The weights are polynomial: no running maximum, no rescaling, so pieces of a
// long axis add up, and the backward pass recomputes s exactly as the forward
// did.  dq and dk, dv are formed by separate passes, each tile owned by one CTA:
// 14 d flops per (query, key) instead of 10, but no atomics, so results do not
// depend on order.
//
// Roundings to bf16: the weights (and ds) that go back into the tensor cores as
// operands, once each.  The denominator sums the rounded weights, so the rows
// remain convex combinations of values: with one visible key y = v exactly and,
// D being formed from the same y in fp32, the gradient of q and k is then zero up
// to fp32 rounding instead of up to bf16 rounding.
//
// Schedule.  The work is a line of units, one per (128-row tile, column block),
// sequence by sequence; every CTA of the persistent grid takes an equal stretch
// of it (cross_sched.cuh), whatever the lengths, and walks the stretch item by
// item (forward, dq: two tiles, which share the columns they read; dkv: one tile).
// An item that a stretch boundary cuts is written as partial sums and joined
// (cross.cu).  Warp 8 loads (TMA), warp 9 issues the products S and P into one of
// three score buffers of 128 columns, warps 0-3 and 4-7 turn scores into weights,
// stored over the scores, and warps 10 and 11 issue the products that accumulate.  The two
// halves (warps 0-3, 4-7) take the two tiles of an item; items of one tile go to
// them in turn, each with its own accumulator, so that one's epilogue overlaps the
// other's steps; in dkv they take the steps of the one tile in turn.
#include <cuda_bf16.h>

#include "cross_sched.cuh"
#include "kata_internal.cuh"
#include "sm100.cuh"
#include "tmap.cuh"

namespace kata {
namespace {

using namespace kata::sm100;

constexpr int kXThreads = 384;
constexpr int kXTma = 8, kXScore = 9, kXAcc = 10;  // and 11
constexpr int kXTile = 128;  // rows of a tile

template <int MODE>
struct XCfg {
    static constexpr int kBlk = cross_tc_cols(MODE);           // columns of a step
    static constexpr int kTiles = cross_tc_tiles(MODE);        // tiles of an item
    static constexpr int kRowOps = MODE == kCrossFwd ? 1 : 2;  // row operands
    static constexpr int kSlot = kRowOps * kTiles * 16384;     // bytes of an item's row operands
    static constexpr int kOp = kBlk * 128;                     // bytes of one column operand
    static constexpr int kStage = 2 * kOp;
    static constexpr int kStages = MODE == kCrossFwd ? 5 : MODE == kCrossDq ? 6 : 8;
    static constexpr int kStat = MODE == kCrossDkv ? 512 : 0;  // -D and 1 / l of the step's queries
    static constexpr int kSmem = 2 * kSlot + kStages * (kStage + kStat) + 1024;
    static constexpr int kBufs = 3;
    static constexpr uint32_t kBuf0 = 128;  // first score buffer's column; accumulators 0 .. 127
};

struct XBars {
    uint64_t qfull[2], qempty[2], full[8], empty[8], bfree[3], ofull[2], ofree[2], drain[3];
    // scores formed and weights stored, per half and buffer: a half (and the warp
    // that accumulates for it) waits for its own steps only, so with one barrier
    // per buffer it could fall two phases behind the other half's steps and take
    // a completed phase for its own.  (dkv: weights of either half in pfull[0], as
    // both accumulating warps wait for every step.)
    uint64_t sfull[2][3], pfull[2][3];
};

// Place in a ring and the parity of its current round.
struct XRing {
    int i = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int n) {
        if (++i == n) {
            i = 0;
            phase ^= 1;
        }
    }
};

struct XArgs {
    XSched sched;
    int d, stat_stride;
    long long BH;
    __nv_bfloat16 *o0, *o1;  // forward: out; dq: dq; dkv: dv, dk
    float *y, *den;          // forward exports
    float *part, *part_l;    // partial sums of cut items
    const float *delta, *rden;
    int *status;
};

__device__ __forceinline__ uint64_t desc_at(uint64_t d, uint32_t bytes) { return d + (bytes >> 4); }

// Bulk copy of `bytes` (a multiple of 16, both ends 16-byte aligned) into shared memory.
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// Writes 64 accumulated columns of a row (the first d of them) times `scale` as
// bf16, and unrounded to y if given.
__device__ __forceinline__ void store_row(__nv_bfloat16 *dst, float *y, const uint32_t *o, float scale, int d) {
    const uint64_t sc = f32x2_pack(__float_as_uint(scale), __float_as_uint(scale));
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        if (8 * c >= d) break;
        uint64_t p[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) p[x] = f32x2_mul(f32x2_pack(o[8 * c + 2 * x], o[8 * c + 2 * x + 1]), sc);
        *reinterpret_cast<uint4 *>(dst + 8 * c) = make_uint4(f32x2_to_bf16x2(p[0]), f32x2_to_bf16x2(p[1]),
                                                             f32x2_to_bf16x2(p[2]), f32x2_to_bf16x2(p[3]));
        if (y) {
            *reinterpret_cast<float4 *>(y + 8 * c) =
                make_float4(f32x2_lo(p[0]), f32x2_hi(p[0]), f32x2_lo(p[1]), f32x2_hi(p[1]));
            *reinterpret_cast<float4 *>(y + 8 * c + 4) =
                make_float4(f32x2_lo(p[2]), f32x2_hi(p[2]), f32x2_lo(p[3]), f32x2_hi(p[3]));
        }
    }
}

__device__ __forceinline__ void store_part(float *dst, const uint32_t *o, int d) {
#pragma unroll
    for (int c = 0; c < 16; ++c) {
        if (4 * c >= d) break;
        *reinterpret_cast<uint4 *>(dst + 4 * c) = make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
    }
}

// Rows without a visible key, which no unit covers: zeros.  Tile by tile over the
// grid, by the 8 warps of the two halves.
template <int MODE>
__device__ void zero_dead_rows(const XArgs &a, int warp, int lane) {
    const XSched &sc = a.sched;
    if (!sc.key_lengths) return;
    const int tiles = (sc.rows + kXTile - 1) / kXTile;
    const long long n = a.BH * tiles;
    for (long long x = blockIdx.x * 8LL + warp; x < n; x += gridDim.x * 8LL) {
        const int bh = (int)(x / tiles), r0 = (int)(x % tiles) * kXTile;
        const int live = cross_length(sc.key_lengths, bh / sc.Hkv, sc.Tk);
        if (MODE == kCrossDkv ? r0 < live : live > 0) continue;
        const long long row = (long long)bh * sc.rows + r0;
        const int rows = min(kXTile, sc.rows - r0);
        const uint4 z = make_uint4(0u, 0u, 0u, 0u);
        for (int c = lane; c < rows * a.d / 8; c += 32) {
            reinterpret_cast<uint4 *>(a.o0 + row * a.d)[c] = z;
            if (MODE == kCrossDkv) reinterpret_cast<uint4 *>(a.o1 + row * a.d)[c] = z;
            if (MODE == kCrossFwd && a.y) {
                reinterpret_cast<uint4 *>(a.y + row * a.d)[2 * c] = z;
                reinterpret_cast<uint4 *>(a.y + row * a.d)[2 * c + 1] = z;
            }
        }
        if (MODE == kCrossFwd && a.den)
            for (int c = lane; c < rows; c += 32) a.den[row + c] = 0.f;
    }
}

template <int MODE>
__global__ void __launch_bounds__(kXThreads, 1)
cross_tc_kernel(const __grid_constant__ CUtensorMap tm_r0, const __grid_constant__ CUtensorMap tm_r1,
                const __grid_constant__ CUtensorMap tm_c0, const __grid_constant__ CUtensorMap tm_c1,
                const XArgs a) {
    using C = XCfg<MODE>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ XBars bars;
    __shared__ XRange range;
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;

    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sm_ring = sm + 2 * C::kSlot;
    uint8_t *sm_stat = sm_ring + C::kStages * C::kStage;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;

    if (tid == 0) {
        abort_flag = 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.qfull[i], 1);
            mbar_init(&bars.qempty[i], 1);
            mbar_init(&bars.ofull[i], 1);
            mbar_init(&bars.ofree[i], 4);
            mbar_init(&bars.drain[i], 1);
        }
        mbar_init(&bars.drain[2], 1);
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&bars.full[i], 1);
            mbar_init(&bars.empty[i], 1);
        }
        for (int i = 0; i < C::kBufs; ++i) {
            mbar_init(&bars.sfull[0][i], 1);
            mbar_init(&bars.sfull[1][i], 1);
            mbar_init(&bars.pfull[0][i], 4);
            mbar_init(&bars.pfull[1][i], 4);
            mbar_init(&bars.bfree[i], MODE == kCrossDkv ? 2 : 1);
        }
        fence_mbarrier_init();
    }
    if (warp == kXScore) {
        tmem_alloc(&tmem_base, 512);
        tmem_relinquish();
    }
    if (warp == kXTma) {
        if (lane == 0) {
            tma_prefetch_desc(&tm_r0);
            tma_prefetch_desc(&tm_c0);
            tma_prefetch_desc(&tm_c1);
        }
        __syncwarp();
        const XRange r = x_range<MODE>(a.sched, blockIdx.x, gridDim.x, lane);
        if (lane == 0) range = r;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = tmem_base;
    volatile int *abort = &abort_flag;
    XIter<MODE> iter(a.sched, range);
    XItem it;

    if (warp == kXTma) {
        // ------------------------------------------------------------ loads
        if (lane == 0) {
            int nq = 0, ns = 0;  // items and stages loaded
            bool ok = true;
            while (ok && iter.next(it)) {
                const int qb = nq & 1;
                ok = mbar_wait(&bars.qempty[qb], ((nq >> 1) & 1) ^ 1, abort);
                if (!ok) break;
                mbar_arrive_expect_tx(&bars.qfull[qb], it.n_tiles * C::kRowOps * 16384);
                for (int t = 0; t < it.n_tiles; ++t) {
                    uint8_t *dst = sm + qb * C::kSlot + t * 16384;
                    tma_load_3d(dst, &tm_r0, &bars.qfull[qb], 0, it.r0 + kXTile * t, it.bh);
                    if (C::kRowOps == 2)
                        tma_load_3d(dst + C::kTiles * 16384, &tm_r1, &bars.qfull[qb], 0, it.r0 + kXTile * t, it.bh);
                }
                ++nq;
                for (int b = 0; b < it.n_blk; ++b) {
                    const int s = ns % C::kStages;
                    ok = mbar_wait(&bars.empty[s], ((ns / C::kStages) & 1) ^ 1, abort);
                    if (!ok) break;
                    const int col = (it.b0 + b) * C::kBlk;
                    uint8_t *dst = sm_ring + s * C::kStage;
                    // boxes of 64 columns; of the forward's second half only what is visible
                    const int boxes = C::kBlk == 128 && it.cols - col > 64 ? 2 : 1;
                    mbar_arrive_expect_tx(&bars.full[s], boxes * 16384 + C::kStat);
                    for (int x = 0; x < boxes; ++x) {
                        tma_load_3d(dst + x * 8192, &tm_c0, &bars.full[s], 0, col + 64 * x, it.bh);
                        tma_load_3d(dst + C::kOp + x * 8192, &tm_c1, &bars.full[s], 0, col + 64 * x, it.bh);
                    }
                    if (MODE == kCrossDkv) {
                        const long long o = (long long)it.bh * a.stat_stride + col;
                        bulk_load(sm_stat + s * C::kStat, a.delta + o, 256, &bars.full[s]);
                        bulk_load(sm_stat + s * C::kStat + 256, a.rden + o, 256, &bars.full[s]);
                    }
                    ++ns;
                }
            }
            // every load issued must have landed before the CTA exits
            for (int x = nq > 2 ? nq - 2 : 0; x < nq; ++x) mbar_wait_issued(&bars.qfull[x & 1], (x >> 1) & 1);
            for (int x = ns > C::kStages ? ns - C::kStages : 0; x < ns; ++x)
                mbar_wait_issued(&bars.full[x % C::kStages], (x / C::kStages) & 1);
        }
    } else if (warp == kXScore) {
        // ------------------------------------------------------------ products that form scores
        if (lane == 0) {
            const uint32_t id = idesc_bf16(128, C::kBlk, 0, 0);
            const uint64_t dR = desc_sw128(smem_u32(sm), 16, 1024);
            const uint64_t dC = desc_sw128(smem_u32(sm_ring), 16, 1024);
            const int n_ks = a.d / 16;  // the head's own coordinates: the columns past d are zeros
            XRing stage, buf;
            int j = 0, n = 0;  // items, steps
            // per score buffer (4 bits): the stage + 1 that its current step is the last to
            // read, or 0.  A buffer found free releases that stage, which saves the
            // accumulating warps a commit per block.
            uint32_t release = 0;
            bool ok = true;
            while (ok && iter.next(it)) {
                const int qb = j & 1;
                const uint64_t r0 = desc_at(dR, qb * C::kSlot);
                ok = mbar_wait(&bars.qfull[qb], (j >> 1) & 1, abort);
                for (int b = 0; b < it.n_blk && ok; ++b) {
                    const uint64_t c = desc_at(dC, stage.i * C::kStage);
                    ok = mbar_wait(&bars.full[stage.i], stage.phase, abort);
                    for (int t = 0; t < it.n_tiles && ok; ++t, ++n) {
                        const int x = buf.i;
                        const uint32_t col = tm + C::kBuf0 + 128 * x;
                        const uint64_t r = desc_at(r0, t * 16384);
                        uint64_t *sfull = &bars.sfull[x_half<MODE>(it, t, j, n)][x];
                        const uint32_t done = (release >> (4 * x)) & 15u;
                        release = (release & ~(15u << (4 * x))) |
                                  ((t == it.n_tiles - 1 ? stage.i + 1u : 0u) << (4 * x));
                        ok = mbar_wait(&bars.bfree[x], buf.phase ^ 1, abort);  // the first round passes at once
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            if (ks < n_ks) mma_ss(col, desc_at(r, 32 * ks), desc_at(c, 32 * ks), id, ks > 0);
                        if (MODE != kCrossFwd) {
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks)
                                if (ks < n_ks)
                                    mma_ss(col + 64, desc_at(r, C::kTiles * 16384 + 32 * ks),
                                           desc_at(c, C::kOp + 32 * ks), id, ks > 0);
                        }
                        mma_commit(sfull);
                        if (done) mbar_arrive(&bars.empty[done - 1]);
                        buf.next(C::kBufs);
                    }
                    stage.next(C::kStages);
                }
                if (!ok) break;
                mma_commit(&bars.qempty[qb]);
                ++j;
            }
            mma_commit(&bars.drain[0]);
            mbar_wait_issued(&bars.drain[0], 0);
        }
    } else if (warp >= kXAcc) {
        // ------------------------------------------------------------ products that accumulate
        // One warp per accumulator (forward, dq: the half's tile; dkv: dv and dk), so
        // that one's waits and overhead pass while the other issues, and every
        // accumulator is added to in the order of the steps.
        if (lane == 0) {
            const int me = warp - kXAcc;
            const uint32_t id = idesc_bf16(128, 64, 0, 1);
            const bool second = MODE == kCrossFwd || (MODE == kCrossDkv && me == 0);  // the column operand used
            const uint64_t dC = desc_at(desc_sw128(smem_u32(sm_ring), 8192, 1024), second ? C::kOp : 0);
            const uint32_t acc = tm + 64 * me;
            const uint32_t w_off = MODE == kCrossDkv && me == 1 ? 64 : 0;  // where its weights lie in a buffer
            XRing stage, buf;
            const int ph = MODE == kCrossDkv ? 0 : me;
            uint32_t ophase = 1;  // the accumulator's first use passes at once
            uint32_t pphase = 0;  // parity of the next of this warp's uses of each buffer
            int j = 0, n = 0;
            bool ok = true;
            while (ok && iter.next(it)) {
                const bool mine = MODE == kCrossDkv || it.n_tiles == 2 || (j & 1) == me;
                for (int b = 0; b < it.n_blk && ok; ++b) {
                    const uint64_t c = desc_at(dC, stage.i * C::kStage);
                    for (int t = 0; t < it.n_tiles; ++t, ++n) {
                        if (mine && (MODE == kCrossDkv || it.n_tiles == 1 || t == me)) {
                            const uint32_t col = tm + C::kBuf0 + 128 * buf.i + w_off;
                            if (b == 0) {
                                ok = mbar_wait(&bars.ofree[me], ophase, abort);
                                if (!ok) break;
                                ophase ^= 1;
                            }
                            ok = mbar_wait(&bars.pfull[ph][buf.i], (pphase >> buf.i) & 1, abort);
                            if (!ok) break;
                            pphase ^= 1u << buf.i;
                            tc_fence_after();
#pragma unroll
                            for (int ks = 0; ks < C::kBlk / 16; ++ks)
                                mma_ts(acc, col + 8 * ks, desc_at(c, 2048 * ks), id, b > 0 || ks > 0);
                            mma_commit(&bars.bfree[buf.i]);
                            if (b == it.n_blk - 1) mma_commit(&bars.ofull[me]);
                        }
                        buf.next(C::kBufs);
                    }
                    stage.next(C::kStages);
                }
                ++j;
            }
            mma_commit(&bars.drain[1 + me]);
            mbar_wait_issued(&bars.drain[1 + me], 0);
        }
    } else {
        // ------------------------------------------------------------ weights and epilogue
        const int half = warp / 4, qd = warp % 4;
        const int row = 32 * qd + lane;
        const uint32_t lane_base = static_cast<uint32_t>(32 * qd) << 16;
        const uint32_t acc = tm + 64 * half + lane_base;
        const int rows = a.sched.rows;
        int j = 0, ns = 0, n = 0;
        uint32_t uses = 0, sphase = 0;  // sphase: parity of this half's next use of each buffer
        bool ok = true;
        zero_dead_rows<MODE>(a, warp, lane);
        __syncwarp();
        while (ok && iter.next(it)) {
            // forward, dq: the tile this half takes, if any
            const int t = MODE == kCrossDkv ? 0 : it.n_tiles == 2 ? half : (j & 1) == half ? 0 : -1;
            const int r = it.r0 + kXTile * t + row;
            const long long gr = (long long)it.bh * rows + r;
            float l = 0.f, ndelta = 0.f;
            if (MODE == kCrossDq && t >= 0 && r < rows) ndelta = a.delta[(long long)it.bh * a.stat_stride + r];
            // this half's steps: forward, dq: one per block, at its tile; dkv: every second step
            const int first = MODE == kCrossDkv ? (n + half) & 1 : t < 0 ? it.n_blk : 0;
            for (int b = first; b < it.n_blk && ok; b += MODE == kCrossDkv ? 2 : 1) {
                const int m = n + b * it.n_tiles + t;
                const int x = m % C::kBufs, s = (ns + b) % C::kStages;
                const uint32_t fpar = ((ns + b) / C::kStages) & 1;
                const uint32_t buf = tm + C::kBuf0 + 128 * x + lane_base;
                ok = __all_sync(0xffffffffu, mbar_wait(&bars.sfull[half][x], (sphase >> x) & 1, abort));
                if (!ok) break;
                sphase ^= 1u << x;
                tc_fence_after();
                const int lim = it.cols - (it.b0 + b) * C::kBlk;  // columns below lim are visible
                if constexpr (MODE == kCrossFwd) {
                    uint64_t acc2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t v[64], p[32];
                        tmem_ld32(buf + 64 * h, v);
                        tmem_ld32(buf + 64 * h + 32, v + 32);
                        tmem_ld_wait();
                        if (lim < 128) {
#pragma unroll
                            for (int y = 0; y < 64; ++y) v[y] = 64 * h + y < lim ? v[y] : 0u;
                        }
#pragma unroll
                        for (int y = 0; y < 32; ++y) {
                            const uint64_t s2 = f32x2_pack(v[2 * y], v[2 * y + 1]);
                            p[y] = f32x2_to_bf16x2(f32x2_mul(s2, s2));
                            acc2[y & 3] = f32x2_add(acc2[y & 3], f32x2_pack(p[y] << 16, p[y] & 0xFFFF0000u));
                        }
                        tmem_st32(buf + 32 * h, p);
                    }
                    const uint64_t z = f32x2_add(f32x2_add(acc2[0], acc2[1]), f32x2_add(acc2[2], acc2[3]));
                    l += f32x2_lo(z) + f32x2_hi(z);
                } else if constexpr (MODE == kCrossDq) {
                    const uint64_t nd = f32x2_pack(__float_as_uint(ndelta), __float_as_uint(ndelta));
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t v[32], g[32], p[16];
                        tmem_ld32(buf + 32 * h, v);
                        tmem_ld32(buf + 64 + 32 * h, g);
                        tmem_ld_wait();
                        if (lim < 64) {
#pragma unroll
                            for (int y = 0; y < 32; ++y) {
                                v[y] = 32 * h + y < lim ? v[y] : 0u;
                                g[y] = 32 * h + y < lim ? g[y] : 0u;
                            }
                        }
#pragma unroll
                        for (int y = 0; y < 16; ++y)
                            p[y] = f32x2_to_bf16x2(f32x2_mul(f32x2_pack(v[2 * y], v[2 * y + 1]),
                                                             f32x2_add(f32x2_pack(g[2 * y], g[2 * y + 1]), nd)));
                        tmem_st16(buf + 16 * h, p);
                    }
                } else {
                    // -D and 1 / l of the step's queries (zeros past the last one)
                    ok = __all_sync(0xffffffffu, mbar_wait(&bars.full[s], fpar, abort));
                    if (!ok) break;
                    const float4 *sd = reinterpret_cast<const float4 *>(sm_stat + s * C::kStat);
                    const float4 *sr = sd + 16;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t v[32], g[32], p[16], e[16];
                        tmem_ld32(buf + 32 * h, v);
                        tmem_ld32(buf + 64 + 32 * h, g);
                        tmem_ld_wait();
#pragma unroll
                        for (int y = 0; y < 8; ++y) {
                            const float4 fd = sd[8 * h + y], fr = sr[8 * h + y];
#pragma unroll
                            for (int z = 0; z < 2; ++z) {
                                const uint64_t s2 = f32x2_pack(v[4 * y + 2 * z], v[4 * y + 2 * z + 1]);
                                const uint64_t g2 = f32x2_pack(g[4 * y + 2 * z], g[4 * y + 2 * z + 1]);
                                const uint64_t d2 =
                                    f32x2_pack(__float_as_uint(z ? fd.z : fd.x), __float_as_uint(z ? fd.w : fd.y));
                                const uint64_t r2 =
                                    f32x2_pack(__float_as_uint(z ? fr.z : fr.x), __float_as_uint(z ? fr.w : fr.y));
                                const uint64_t sr2 = f32x2_mul(s2, r2);
                                p[2 * y + z] = f32x2_to_bf16x2(f32x2_mul(s2, sr2));
                                e[2 * y + z] = f32x2_to_bf16x2(f32x2_mul(sr2, f32x2_add(g2, d2)));  // ds / 2
                            }
                        }
                        tmem_st16(buf + 16 * h, p);
                        tmem_st16(buf + 64 + 16 * h, e);
                    }
                }
                // Rows past the visible keys of the operand that the weights multiply may
                // hold anything (NaN times a zero weight is NaN): cleared in the block
                // where the visible keys end, by every warp of both halves before it
                // hands its weights over.
                if (MODE != kCrossDkv && lim < C::kBlk) {
                    ok = __all_sync(0xffffffffu, mbar_wait(&bars.full[s], fpar, abort));
                    if (!ok) break;
                    uint8_t *op = sm_ring + s * C::kStage + (MODE == kCrossFwd ? C::kOp : 0);
                    for (int k = lim + qd; k < C::kBlk; k += 4)
                        *reinterpret_cast<uint32_t *>(op + k * 128 + lane * 4) = 0u;
                    fence_proxy_async_smem();
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    // the accumulating warp reads the stage without waiting for it
                    ok = mbar_wait(&bars.full[s], fpar, abort);
                    if (ok) mbar_arrive(&bars.pfull[MODE == kCrossDkv ? 0 : half][x]);
                }
                ok = __shfl_sync(0xffffffffu, ok, 0);
            }
            if (!ok) break;
            if (t >= 0) {
                uint32_t o[64];
                ok = __all_sync(0xffffffffu, mbar_wait(&bars.ofull[half], uses & 1, abort));
                if (!ok) break;
                ++uses;
                tc_fence_after();
                tmem_ld32(acc, o);
                tmem_ld32(acc + 32, o + 32);
                tmem_ld_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.ofree[half]);
                if (MODE == kCrossDkv && r >= it.live) {  // keys past the visible ones, whatever they hold
#pragma unroll
                    for (int c = 0; c < 64; ++c) o[c] = 0u;
                }
                if (r < rows) {
                    if (it.part >= 0) {
                        // cut item: row of the piece's slot (dkv: dv's rows, then dk's)
                        const long long pr = x_part_row<MODE>(a.sched, it.part) + kXTile * t + row +
                                             (MODE == kCrossDkv ? kXTile * half : 0);
                        store_part(a.part + pr * a.d, o, a.d);
                        if (MODE == kCrossFwd) a.part_l[pr] = l;
                    } else if (MODE == kCrossFwd) {
                        store_row(a.o0 + gr * a.d, a.y ? a.y + gr * a.d : nullptr, o, cross_recip(l), a.d);
                        if (a.den) a.den[gr] = l;
                    } else if (MODE == kCrossDq) {
                        store_row(a.o0 + gr * a.d, nullptr, o, 2.f * a.rden[(long long)it.bh * a.stat_stride + r],
                                  a.d);
                    } else {
                        store_row((half ? a.o1 : a.o0) + gr * a.d, nullptr, o, half ? 2.f : 1.f, a.d);
                    }
                }
                __syncwarp();
            }
            n += it.n_blk * it.n_tiles;
            ns += it.n_blk;
            ++j;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kXScore) tmem_dealloc(tm, 512);
    if (tid == 0 && abort_flag) atomicCAS(a.status, 0, (int)KATA_ERR_TIMEOUT);
}

template <int MODE>
cudaError_t launch_mode(const CrossPlan &p, const CrossIo &io, cudaStream_t st) {
    using C = XCfg<MODE>;
    char *ws = static_cast<char *>(io.ws);
    XArgs a{};
    a.sched = p.sched[MODE];
    a.sched.key_lengths = io.key_lengths;
    a.d = p.d;
    a.stat_stride = p.R_pad;
    a.BH = p.BH;
    a.o0 = static_cast<__nv_bfloat16 *>(MODE == kCrossFwd ? io.out : MODE == kCrossDq ? io.dq : io.dv);
    a.o1 = static_cast<__nv_bfloat16 *>(io.dk);
    a.y = io.y;
    a.den = io.den;
    a.part = reinterpret_cast<float *>(ws + p.ws_part[MODE]);
    a.part_l = reinterpret_cast<float *>(ws + p.ws_part_l);
    a.delta = reinterpret_cast<const float *>(ws + p.ws_delta);
    a.rden = reinterpret_cast<const float *>(ws + p.ws_rden);
    a.status = device_status_ptr();
    if (!a.status) return cudaErrorUnknown;
    const void *r0 = MODE == kCrossDkv ? io.k : io.q, *r1 = MODE == kCrossDkv ? io.v : io.dout;
    const void *c0 = MODE == kCrossDkv ? io.q : io.k, *c1 = MODE == kCrossDkv ? io.dout : io.v;
    if (MODE == kCrossFwd) r1 = r0;
    CUtensorMap maps[4];
    const void *base[4] = {r0, r1, c0, c1};
    for (int m = 0; m < 4; ++m) {
        const uint64_t n = m < 2 ? a.sched.rows : a.sched.cols, w = 2 * (uint64_t)p.d;
        const uint64_t dims[3] = {(uint64_t)p.d, n, (uint64_t)p.BH}, strides[2] = {w, w * n};
        const uint32_t box[3] = {64, m < 2 ? (uint32_t)kXTile : 64u, 1};
        if (!make_tmap_bf16(&maps[m], base[m], 3, dims, strides, box)) return cudaErrorInvalidValue;
    }
    const cudaError_t e = smem_opt_in_once<cross_tc_kernel<MODE>>(C::kSmem);
    if (e != cudaSuccess) return e;
    ProfScope prof(MODE == kCrossFwd ? "cross_fwd" : MODE == kCrossDq ? "cross_dq" : "cross_dkv", st);
    cross_tc_kernel<MODE><<<p.sched[MODE].grid, kXThreads, C::kSmem, st>>>(maps[0], maps[1], maps[2], maps[3], a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cross_tc(CrossMode mode, const CrossPlan &p, const CrossIo &io, cudaStream_t st) {
    switch (mode) {
        case kCrossFwd: return launch_mode<kCrossFwd>(p, io, st);
        case kCrossDq: return launch_mode<kCrossDq>(p, io, st);
        default: return launch_mode<kCrossDkv>(p, io, st);
    }
}

}  // namespace kata
