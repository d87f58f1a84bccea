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
// Schedule.  A persistent CTA of 11 warps walks items (problem, 256 rows, piece of
// the other axis): warp 8 loads (TMA), warp 9 issues the products S and P into one
// of three (dkv: two) score buffers of 128 columns, warps 0-3 and 4-7 turn the
// scores of row tile 0 and 1 into weights, stored over the scores, and warp 10
// issues the products that accumulate.  An item of one tile alternates between
// the two halves, so its epilogue overlaps the next item's steps.
#include <cuda_bf16.h>

#include "kata_internal.cuh"
#include "sm100.cuh"
#include "tmap.cuh"

namespace kata {
namespace {

using namespace kata::sm100;

constexpr int kXThreads = 352;
constexpr int kXTma = 8, kXScore = 9, kXAcc = 10;
constexpr int kXTile = 128;  // rows of a tile
constexpr int kXRows = 256;  // rows of an item (two tiles)

template <int MODE>
struct XCfg {
    static constexpr int kBlk = MODE == kCrossFwd ? 128 : 64;  // columns of a step
    static constexpr int kRowOps = MODE == kCrossFwd ? 1 : 2;  // row operands
    static constexpr int kSlot = kRowOps * 2 * 16384;          // bytes of an item's row operands
    static constexpr int kOp = kBlk * 128;                     // bytes of one column operand
    static constexpr int kStage = 2 * kOp;
    static constexpr int kStages = MODE == kCrossFwd ? 5 : MODE == kCrossDq ? 6 : 5;
    static constexpr int kStat = MODE == kCrossDkv ? 512 : 0;  // D and 1 / l of the step's queries
    static constexpr int kSmem = 2 * kSlot + kStages * (kStage + kStat) + 1024;
    static constexpr int kBufs = MODE == kCrossDkv ? 2 : 3;
    static constexpr uint32_t kAccCols = MODE == kCrossDkv ? 128 : 64;  // accumulator columns per tile
    static constexpr uint32_t kBuf0 = 2 * kAccCols;                     // first score buffer's column
};

struct XBars {
    uint64_t qfull[2], qempty[2], full[6], empty[6], pfull[3], bfree[3], ofull[2], ofree[2], drain[2];
    // scores formed, per half and buffer: a half waits for its own steps only, so
    // with one barrier per buffer it could fall two phases behind the other
    // half's steps (items of one tile) and take a completed phase for its own
    uint64_t sfull[2][3];
};

struct XArgs {
    int rows, cols, Hkv, tiles, splits, n_items, Tk, d, stat_stride;
    long long BH;
    const int *key_lengths;
    __nv_bfloat16 *o0, *o1;  // forward: out; dq: dq; dkv: dv, dk
    float *y, *den;          // forward exports
    float *part, *part_l;    // partial sums (splits > 1)
    const float *delta, *rden;
    int *status;
};

struct XItem {
    int bh, r0, n_tiles, split, c0, n_blk;
    int live;  // forward, dq: visible columns; dkv: visible rows
};

template <int MODE>
__device__ __forceinline__ XItem x_item(const XArgs &a, int i) {
    XItem it;
    it.split = i % a.splits;
    const int x = i / a.splits;
    it.bh = x / a.tiles;
    it.r0 = (x % a.tiles) * kXRows;
    it.live = cross_length(a.key_lengths, it.bh / a.Hkv, a.Tk);
    const int cols = MODE == kCrossDkv ? a.cols : it.live;
    const int rows = MODE == kCrossDkv ? it.live : a.rows;
    it.n_tiles = rows > it.r0 + kXTile ? 2 : rows > it.r0 ? 1 : 0;
    const int blocks = (cols + XCfg<MODE>::kBlk - 1) / XCfg<MODE>::kBlk;
    const int piece = (blocks + a.splits - 1) / a.splits;
    it.c0 = it.split * piece * XCfg<MODE>::kBlk;
    it.n_blk = it.n_tiles ? max(0, min(piece, blocks - it.split * piece)) : 0;
    return it;
}

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

template <int MODE>
__global__ void __launch_bounds__(kXThreads, 1)
cross_tc_kernel(const __grid_constant__ CUtensorMap tm_r0, const __grid_constant__ CUtensorMap tm_r1,
                const __grid_constant__ CUtensorMap tm_c0, const __grid_constant__ CUtensorMap tm_c1,
                const XArgs a) {
    using C = XCfg<MODE>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ XBars bars;
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
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&bars.full[i], 1);
            mbar_init(&bars.empty[i], 1);
        }
        for (int i = 0; i < C::kBufs; ++i) {
            mbar_init(&bars.sfull[0][i], 1);
            mbar_init(&bars.sfull[1][i], 1);
            mbar_init(&bars.pfull[i], 4);
            mbar_init(&bars.bfree[i], 1);
        }
        fence_mbarrier_init();
    }
    if (warp == kXScore) {
        tmem_alloc(&tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = tmem_base;
    volatile int *abort = &abort_flag;

    if (warp == kXTma) {
        // ------------------------------------------------------------ loads
        if (lane == 0) {
            int nq = 0, ns = 0;  // items and stages loaded
            bool ok = true;
            for (int i = blockIdx.x; i < a.n_items && ok; i += gridDim.x) {
                const XItem it = x_item<MODE>(a, i);
                if (it.n_blk == 0) continue;
                const int qb = nq & 1;
                ok = mbar_wait(&bars.qempty[qb], ((nq >> 1) & 1) ^ 1, abort);
                if (!ok) break;
                mbar_arrive_expect_tx(&bars.qfull[qb], it.n_tiles * C::kRowOps * 16384);
                for (int t = 0; t < it.n_tiles; ++t) {
                    uint8_t *dst = sm + qb * C::kSlot + t * 16384;
                    tma_load_3d(dst, &tm_r0, &bars.qfull[qb], 0, it.r0 + kXTile * t, it.bh);
                    if (C::kRowOps == 2)
                        tma_load_3d(dst + 32768, &tm_r1, &bars.qfull[qb], 0, it.r0 + kXTile * t, it.bh);
                }
                ++nq;
                for (int b = 0; b < it.n_blk; ++b) {
                    const int s = ns % C::kStages;
                    ok = mbar_wait(&bars.empty[s], ((ns / C::kStages) & 1) ^ 1, abort);
                    if (!ok) break;
                    const int col = it.c0 + b * C::kBlk;
                    mbar_arrive_expect_tx(&bars.full[s], C::kStage + C::kStat);
                    tma_load_3d(sm_ring + s * C::kStage, &tm_c0, &bars.full[s], 0, col, it.bh);
                    tma_load_3d(sm_ring + s * C::kStage + C::kOp, &tm_c1, &bars.full[s], 0, col, it.bh);
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
            int j = 0, ns = 0, n = 0;   // items, stages, steps
            bool ok = true;
            for (int i = blockIdx.x; i < a.n_items && ok; i += gridDim.x) {
                const XItem it = x_item<MODE>(a, i);
                if (it.n_blk == 0) continue;
                const int qb = j & 1;
                ok = mbar_wait(&bars.qfull[qb], (j >> 1) & 1, abort);
                for (int b = 0; b < it.n_blk && ok; ++b, ++ns) {
                    const int s = ns % C::kStages;
                    ok = mbar_wait(&bars.full[s], (ns / C::kStages) & 1, abort);
                    for (int t = 0; t < it.n_tiles && ok; ++t, ++n) {
                        const int x = n % C::kBufs, u = n / C::kBufs;
                        if (u > 0) ok = mbar_wait(&bars.bfree[x], (u - 1) & 1, abort);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t buf = tm + C::kBuf0 + 128 * x;
                        const uint64_t r = desc_at(dR, qb * C::kSlot + t * 16384), c = desc_at(dC, s * C::kStage);
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            if (ks < n_ks) mma_ss(buf, desc_at(r, 32 * ks), desc_at(c, 32 * ks), id, ks > 0);
                        if (MODE != kCrossFwd) {
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks)
                                if (ks < n_ks)
                                    mma_ss(buf + 64, desc_at(r, 32768 + 32 * ks), desc_at(c, C::kOp + 32 * ks), id,
                                           ks > 0);
                        }
                        mma_commit(&bars.sfull[it.n_tiles == 2 ? t : (j & 1)][x]);
                    }
                }
                if (!ok) break;
                mma_commit(&bars.qempty[qb]);
                ++j;
            }
            mma_commit(&bars.drain[0]);
            mbar_wait_issued(&bars.drain[0], 0);
        }
    } else if (warp == kXAcc) {
        // ------------------------------------------------------------ products that accumulate
        if (lane == 0) {
            const uint32_t id = idesc_bf16(128, 64, 0, 1);
            const uint64_t dC = desc_sw128(smem_u32(sm_ring), 8192, 1024);
            int j = 0, ns = 0, n = 0;
            uint32_t uses[2] = {0, 0};
            bool ok = true;
            for (int i = blockIdx.x; i < a.n_items && ok; i += gridDim.x) {
                const XItem it = x_item<MODE>(a, i);
                if (it.n_blk == 0) continue;
                for (int b = 0; b < it.n_blk && ok; ++b, ++ns) {
                    const int s = ns % C::kStages;
                    for (int t = 0; t < it.n_tiles; ++t, ++n) {
                        const int half = it.n_tiles == 2 ? t : (j & 1);
                        const int x = n % C::kBufs, u = n / C::kBufs;
                        if (b == 0) {
                            const uint32_t k = uses[half]++;
                            if (k > 0) ok = mbar_wait(&bars.ofree[half], (k - 1) & 1, abort);
                            if (!ok) break;
                        }
                        ok = mbar_wait(&bars.pfull[x], u & 1, abort);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t acc = tm + C::kAccCols * half, buf = tm + C::kBuf0 + 128 * x;
                        const uint64_t c0 = desc_at(dC, s * C::kStage), c1 = desc_at(c0, C::kOp);
#pragma unroll
                        for (int ks = 0; ks < C::kBlk / 16; ++ks)
                            mma_ts(acc, buf + 8 * ks, desc_at(MODE == kCrossDq ? c0 : c1, 2048 * ks), id,
                                   b > 0 || ks > 0);
                        if (MODE == kCrossDkv) {
#pragma unroll
                            for (int ks = 0; ks < C::kBlk / 16; ++ks)
                                mma_ts(acc + 64, buf + 64 + 8 * ks, desc_at(c0, 2048 * ks), id, b > 0 || ks > 0);
                        }
                        mma_commit(&bars.bfree[x]);
                        if (t == it.n_tiles - 1) mma_commit(&bars.empty[s]);
                        if (b == it.n_blk - 1) mma_commit(&bars.ofull[half]);
                    }
                }
                ++j;
            }
            mma_commit(&bars.drain[1]);
            mbar_wait_issued(&bars.drain[1], 0);
        }
    } else {
        // ------------------------------------------------------------ weights and epilogue
        const int half = warp / 4, qd = warp % 4;
        const int row = 32 * qd + lane;
        const uint32_t lane_base = static_cast<uint32_t>(32 * qd) << 16;
        const uint32_t acc = tm + C::kAccCols * half + lane_base;
        int j = 0, ns = 0, n = 0;
        uint32_t uses = 0, sphase = 0;  // sphase: parity of this half's next use of each buffer
        bool ok = true;
        for (int i = blockIdx.x; i < a.n_items && ok; i += gridDim.x) {
            const XItem it = x_item<MODE>(a, i);
            const int t = it.n_blk == 0 || it.n_tiles == 2 ? half : ((j & 1) == half ? 0 : 1);
            const int r = it.r0 + kXTile * t + row;
            const bool on = it.n_blk > 0 && t < it.n_tiles;
            const long long gr = (long long)it.bh * a.rows + r;
            float l = 0.f, delta = 0.f;
            if (MODE == kCrossDq && on && r < a.rows) delta = a.delta[(long long)it.bh * a.stat_stride + r];
            for (int b = 0; on && b < it.n_blk && ok; ++b) {
                const int m = n + b * it.n_tiles + (it.n_tiles == 2 ? t : 0);
                const int x = m % C::kBufs, s = (ns + b) % C::kStages;
                const uint32_t fpar = ((ns + b) / C::kStages) & 1;
                const uint32_t buf = tm + C::kBuf0 + 128 * x + lane_base;
                ok = __all_sync(0xffffffffu, mbar_wait(&bars.sfull[half][x], (sphase >> x) & 1, abort));
                if (!ok) break;
                sphase ^= 1u << x;
                tc_fence_after();
                const int lim = it.live - (it.c0 + b * C::kBlk);  // columns below lim are visible
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
                    const uint64_t nd = f32x2_pack(__float_as_uint(-delta), __float_as_uint(-delta));
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
                    // D and 1 / l of the step's queries (zeros past the last one)
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
                                const uint64_t d2 = f32x2_pack(__float_as_uint(z ? -fd.z : -fd.x),
                                                               __float_as_uint(z ? -fd.w : -fd.y));
                                const uint64_t r2 = f32x2_pack(__float_as_uint(z ? fr.z : fr.x),
                                                               __float_as_uint(z ? fr.w : fr.y));
                                const uint64_t sr2 = f32x2_mul(s2, r2);
                                p[2 * y + z] = f32x2_to_bf16x2(f32x2_mul(s2, sr2));
                                e[2 * y + z] = f32x2_to_bf16x2(
                                    f32x2_mul(f32x2_add(sr2, sr2), f32x2_add(g2, d2)));
                            }
                        }
                        tmem_st16(buf + 16 * h, p);
                        tmem_st16(buf + 64 + 16 * h, e);
                    }
                }
                // Masked rows of the operand that the weights multiply may hold
                // anything (NaN times a zero weight is NaN): cleared in the block
                // where the visible keys end.  Every warp of both halves clears its
                // share before it hands its weights over.
                if (MODE != kCrossDkv && lim < C::kBlk && it.live < a.cols) {
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
                    if (ok) mbar_arrive(&bars.pfull[x]);
                }
                ok = __shfl_sync(0xffffffffu, ok, 0);
            }
            if (!ok) break;
            uint32_t o[64];
            if (on) {
                ok = __all_sync(0xffffffffu, mbar_wait(&bars.ofull[half], uses & 1, abort));
                if (!ok) break;
                ++uses;
                tc_fence_after();
                tmem_ld32(acc, o);
                tmem_ld32(acc + 32, o + 32);
                tmem_ld_wait();
            } else {
#pragma unroll
                for (int c = 0; c < 64; ++c) o[c] = 0u;
            }
            const bool in = r < a.rows;
            // dkv: rows past the visible keys get zeros whatever they hold
            const bool dead = MODE == kCrossDkv && r >= it.live;
            if constexpr (MODE == kCrossDkv) {
                if (dead) {
#pragma unroll
                    for (int c = 0; c < 64; ++c) o[c] = 0u;
                }
                const long long base = (long long)it.split * 2 * a.BH * a.rows + gr;
                if (in) {
                    if (a.splits > 1)
                        store_part(a.part + base * a.d, o, a.d);
                    else
                        store_row(a.o0 + gr * a.d, nullptr, o, 1.f, a.d);
                }
                __syncwarp();
                uint32_t e[64];
                if (on) {
                    tmem_ld32(acc + 64, e);
                    tmem_ld32(acc + 96, e + 32);
                    tmem_ld_wait();
                }
                if (!on || dead) {
#pragma unroll
                    for (int c = 0; c < 64; ++c) e[c] = 0u;
                }
                if (in) {
                    if (a.splits > 1)
                        store_part(a.part + (base + a.BH * a.rows) * a.d, e, a.d);
                    else
                        store_row(a.o1 + gr * a.d, nullptr, e, 1.f, a.d);
                }
            } else if (in) {
                if (a.splits > 1) {
                    const long long pr = (long long)it.split * a.BH * a.rows + gr;
                    store_part(a.part + pr * a.d, o, a.d);
                    if (MODE == kCrossFwd) a.part_l[pr] = l;
                } else if (MODE == kCrossFwd) {
                    store_row(a.o0 + gr * a.d, a.y ? a.y + gr * a.d : nullptr, o, cross_recip(l), a.d);
                    if (a.den) a.den[gr] = l;
                } else {
                    store_row(a.o0 + gr * a.d, nullptr, o, 2.f * a.rden[(long long)it.bh * a.stat_stride + r], a.d);
                }
            }
            if (on) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.ofree[half]);
            }
            if (it.n_blk > 0) {
                n += it.n_blk * it.n_tiles;
                ns += it.n_blk;
                ++j;
            }
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
    a.rows = MODE == kCrossDkv ? p.Tk : p.R;
    a.cols = MODE == kCrossDkv ? p.R : p.Tk;
    a.Hkv = p.Hkv;
    a.tiles = (a.rows + kXRows - 1) / kXRows;
    a.splits = p.splits[MODE];
    a.n_items = (int)(p.BH * a.tiles * a.splits);
    a.Tk = p.Tk;
    a.d = p.d;
    a.stat_stride = p.R_pad;
    a.BH = p.BH;
    a.key_lengths = io.key_lengths;
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
        const uint64_t n = m < 2 ? a.rows : a.cols, w = 2 * (uint64_t)p.d;
        const uint64_t dims[3] = {(uint64_t)p.d, n, (uint64_t)p.BH}, strides[2] = {w, w * n};
        const uint32_t box[3] = {64, m < 2 ? (uint32_t)kXTile : (uint32_t)C::kBlk, 1};
        if (!make_tmap_bf16(&maps[m], base[m], 3, dims, strides, box)) return cudaErrorInvalidValue;
    }
    const cudaError_t e = smem_opt_in_once<cross_tc_kernel<MODE>>(C::kSmem);
    if (e != cudaSuccess) return e;
    const int grid = a.n_items < tc::num_sms() ? a.n_items : tc::num_sms();
    ProfScope prof(MODE == kCrossFwd ? "cross_fwd" : MODE == kCrossDq ? "cross_dq" : "cross_dkv", st);
    cross_tc_kernel<MODE><<<grid, kXThreads, C::kSmem, st>>>(maps[0], maps[1], maps[2], maps[3], a);
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
