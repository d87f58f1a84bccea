// Cross attention with KATA weights on the tensor cores (bf16, d in {16, 32, 64},
// read as 64 by the tensor maps, which fill the columns past d with zeros).
//
//   s = q.k,  w = s^2,  l = sum_s w,  y = (sum_s w v) / l              (0 if l = 0)
//
// and, with D = dy.y and p = dy.v for the gradient dy of y,
//
//   ds = 2 s (p - D) / l,   dq = sum_s ds k,   dk = sum_t ds q,   dv = sum_t (w / l) dy.
//
// Every pass keeps 128-row tiles of its accumulators in tensor memory, walks the
// other axis in blocks of 128 and forms per block
//
//   forward (here)   rows = queries  S = Q K^T             O  += bf16(w) V
//   dq  (_bwd.cu)    rows = queries  S = Q K^T, P = dY V^T  dQ += bf16(s (p - D)) K
//   dkv (_bwd.cu)    rows = keys     S = K Q^T, P = V dY^T  dV += bf16(w / l) dY
//                                                           dK += bf16(ds / 2) Q
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
// item.  An item that a stretch boundary cuts is written as partial sums and
// joined (cross.cu).  A forward item is two tiles, which share the keys and values
// they read.  Warp 8 loads (TMA), warp 9 issues the products that form scores into
// one of three score buffers of 128 columns, warps 0-3 and 4-7 turn the scores of
// one tile each into weights, stored over the scores, and warps 10 and 11 issue the
// products that accumulate.  Items of one tile go to the two halves in turn, each
// with its own accumulator, so that one's epilogue overlaps the other's steps.
#include "cross_tc.cuh"

namespace kata {
namespace {

constexpr int kXThreads = 384;
constexpr int kXTma = 8, kXScore = 9, kXAcc = 10;  // and 11
constexpr int kBlk = 128;                           // keys of a step
constexpr int kSlot = 2 * 16384;                    // bytes of an item's queries
constexpr int kOp = kBlk * 128;                     // bytes of a block's keys (or values)
constexpr int kStage = 2 * kOp;
constexpr int kStages = 5;
constexpr int kSmem = 2 * kSlot + kStages * kStage + 1024;
constexpr int kBufs = 3;
constexpr uint32_t kBuf0 = 128;  // first score buffer's column; the halves' accumulators lie at 0 and 64

struct XBars {
    uint64_t qfull[2], qempty[2], full[kStages], empty[kStages], bfree[kBufs], ofull[2], ofree[2], drain[3];
    // scores formed and weights stored, per half and buffer: a half (and the warp
    // that accumulates for it) waits for its own steps only, so with one barrier
    // per buffer it could fall two phases behind the other half's steps and take
    // a completed phase for its own.
    uint64_t sfull[2][kBufs], pfull[2][kBufs];
};

// SPLIT: the weights as two bf16 numbers each (high and low part), which takes twice
// the products that accumulate: the forward of a training step with d <= 32.  Its y
// gives the backward pass D = dy.y, and an error of D enters every key's gradient
// with one sign: next to the other roundings it is as 1 / sqrt(d).  Error of dq
// relative to exact, rms, without and with (0.00166 of it the output's rounding):
// d = 16 0.0026, 0.0025; d = 32 0.0025, 0.0024; d = 64 0.0024, 0.0024.  For d = 64 it
// would take the forward of 2048 queries on 4096 keys from 125 to 202 us.
template <bool SPLIT>
__global__ void __launch_bounds__(kXThreads, 1)
cross_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const XArgs a) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ XBars bars;
    __shared__ XRange range;
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;

    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sm_ring = sm + 2 * kSlot;
    uint8_t *sm_stat = sm_ring + kStages * kStage;
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
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&bars.full[i], 1);
            mbar_init(&bars.empty[i], 1);
        }
        for (int i = 0; i < kBufs; ++i) {
            mbar_init(&bars.sfull[0][i], 1);
            mbar_init(&bars.sfull[1][i], 1);
            mbar_init(&bars.pfull[0][i], 4);
            mbar_init(&bars.pfull[1][i], 4);
            mbar_init(&bars.bfree[i], 1);
        }
        fence_mbarrier_init();
    }
    if (warp == kXScore) {
        tmem_alloc(&tmem_base, 512);
        tmem_relinquish();
    }
    if (warp == kXTma) {
        if (lane == 0) {
            tma_prefetch_desc(&tm_q);
            tma_prefetch_desc(&tm_k);
            tma_prefetch_desc(&tm_v);
        }
        __syncwarp();
        const XRange r = x_range<kCrossFwd>(a.sched, blockIdx.x, gridDim.x, lane);
        if (lane == 0) range = r;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_wait();  // what ran before has ended: memory may be read and written
    const uint32_t tm = tmem_base;
    volatile int *abort = &abort_flag;
    XIter<kCrossFwd> iter(a.sched, range);
    XItem it;

    if (warp == kXTma) {
        // ------------------------------------------------------------ loads
        if (lane == 0) {
            if (!a.sched.whole) a.pieces[blockIdx.x] = XIter<kCrossFwd>::first(a.sched, range);
            int nq = 0, ns = 0;  // items and stages loaded
            bool ok = true;
            while (ok && iter.next(it)) {
                const int qb = nq & 1;
                ok = mbar_wait(&bars.qempty[qb], ((nq >> 1) & 1) ^ 1, abort);
                if (!ok) break;
                mbar_arrive_expect_tx(&bars.qfull[qb], it.n_tiles * 16384);
                for (int t = 0; t < it.n_tiles; ++t)
                    tma_load_3d(sm + qb * kSlot + t * 16384, &tm_q, &bars.qfull[qb], 0, it.r0 + kXTile * t, it.bh);
                ++nq;
                for (int b = 0; b < it.n_blk; ++b) {
                    const int s = ns % kStages;
                    ok = mbar_wait(&bars.empty[s], ((ns / kStages) & 1) ^ 1, abort);
                    if (!ok) break;
                    const int col = (it.b0 + b) * kBlk;
                    uint8_t *dst = sm_ring + s * kStage;
                    // boxes of 64 keys, the second if it holds a visible one
                    const int boxes = it.cols - col > 64 ? 2 : 1;
                    mbar_arrive_expect_tx(&bars.full[s], boxes * 16384);
                    for (int x = 0; x < boxes; ++x) {
                        tma_load_3d(dst + x * 8192, &tm_k, &bars.full[s], 0, col + 64 * x, it.bh);
                        tma_load_3d(dst + kOp + x * 8192, &tm_v, &bars.full[s], 0, col + 64 * x, it.bh);
                    }
                    ++ns;
                }
            }
            // every load issued must have landed before the CTA exits
            for (int x = nq > 2 ? nq - 2 : 0; x < nq; ++x) mbar_wait_issued(&bars.qfull[x & 1], (x >> 1) & 1);
            for (int x = ns > kStages ? ns - kStages : 0; x < ns; ++x)
                mbar_wait_issued(&bars.full[x % kStages], (x / kStages) & 1);
        }
    } else if (warp == kXScore) {
        // ------------------------------------------------------------ products that form scores
        if (lane == 0) {
            const uint32_t id = idesc_bf16(128, kBlk, 0, 0);
            const uint64_t dR = desc_sw128(smem_u32(sm), 16, 1024);
            const uint64_t dC = desc_sw128(smem_u32(sm_ring), 16, 1024);
            const int n_ks = a.d / 16;  // the head's own coordinates: the columns past d are zeros
            XRing stage, buf;
            int j = 0, n = 0;  // items, steps
            // per score buffer (4 bits): the stage + 1 that its current step, of a second tile,
            // is the last to read, or 0.  A buffer found free releases that stage.
            uint32_t release = 0;
            bool ok = true;
            while (ok && iter.next(it)) {
                const int qb = j & 1;
                const uint64_t r0 = desc_at(dR, qb * kSlot);
                ok = mbar_wait(&bars.qfull[qb], (j >> 1) & 1, abort);
                for (int b = 0; b < it.n_blk && ok; ++b) {
                    const uint64_t c = desc_at(dC, stage.i * kStage);
                    ok = mbar_wait(&bars.full[stage.i], stage.phase, abort);
                    for (int t = 0; t < it.n_tiles && ok; ++t, ++n) {
                        const int x = buf.i;
                        const uint32_t col = tm + kBuf0 + 128 * x;
                        const uint64_t r = desc_at(r0, t * 16384);
                        uint64_t *sfull = &bars.sfull[x_half(it, t, j)][x];
                        const uint32_t done = (release >> (4 * x)) & 15u;
                        release = (release & ~(15u << (4 * x))) | ((t == 1 ? stage.i + 1u : 0u) << (4 * x));
                        ok = mbar_wait(&bars.bfree[x], buf.phase ^ 1, abort);  // the first round passes at once
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            if (ks < n_ks) mma_ss(col, desc_at(r, 32 * ks), desc_at(c, 32 * ks), id, ks > 0);
                        mma_commit(sfull);
                        if (done) mbar_arrive(&bars.empty[done - 1]);
                        buf.next(kBufs);
                    }
                    stage.next(kStages);
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
        // One warp per accumulator, so that one's waits and overhead pass while the
        // other issues, and every accumulator is added to in the order of the steps.
        if (lane == 0) {
            const int me = warp - kXAcc;
            const uint32_t id = idesc_bf16(128, a.d, 0, 1);  // the head's own columns
            const uint64_t dV = desc_sw128(smem_u32(sm_ring + kOp), 8192, 1024);
            const uint32_t acc = tm + 64 * me;
            XRing stage, buf;
            uint32_t ophase = 1;  // the accumulator's first use passes at once
            uint32_t pphase = 0;  // parity of the next of this warp's uses of each buffer
            int j = 0, n = 0;
            bool ok = true;
            while (ok && iter.next(it)) {
                const bool mine = it.n_tiles == 2 || (j & 1) == me;
                for (int b = 0; b < it.n_blk && ok; ++b) {
                    const uint64_t c = desc_at(dV, stage.i * kStage);
                    for (int t = 0; t < it.n_tiles; ++t, ++n) {
                        if (mine && (it.n_tiles == 1 || t == me)) {
                            const uint32_t col = tm + kBuf0 + 128 * buf.i;
                            if (b == 0) {
                                ok = mbar_wait(&bars.ofree[me], ophase, abort);
                                if (!ok) break;
                                ophase ^= 1;
                            }
                            ok = mbar_wait(&bars.full[stage.i], stage.phase, abort) &&
                                 mbar_wait(&bars.pfull[me][buf.i], (pphase >> buf.i) & 1, abort);
                            if (!ok) break;
                            pphase ^= 1u << buf.i;
                            tc_fence_after();
#pragma unroll
                            for (int ks = 0; ks < kBlk / 16; ++ks)
                                mma_ts(acc, col + (SPLIT ? 32 * (ks / 2) + 8 * (ks % 2) : 8 * ks), desc_at(c, 2048 * ks),
                                       id, b > 0 || ks > 0);
                            if (SPLIT) {
#pragma unroll
                                for (int ks = 0; ks < kBlk / 16; ++ks)
                                    mma_ts(acc, col + 32 * (ks / 2) + 8 * (ks % 2) + 16, desc_at(c, 2048 * ks), id, 1);
                            }
                            mma_commit(&bars.bfree[buf.i]);
                            // an item of one tile, whose steps wait for loads: its stage is free at
                            // once (with two tiles the scores' warp knows when both are done)
                            if (it.n_tiles == 1) mma_commit(&bars.empty[stage.i]);
                            if (b == it.n_blk - 1) mma_commit(&bars.ofull[me]);
                        }
                        buf.next(kBufs);
                    }
                    stage.next(kStages);
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
        zero_dead_rows<kCrossFwd>(a, warp, 8, lane);
        __syncwarp();
        while (ok && iter.next(it)) {
            // the tile this half takes, if any
            const int t = it.n_tiles == 2 ? half : (j & 1) == half ? 0 : -1;
            const int r = it.r0 + kXTile * t + row;
            const long long gr = (long long)it.bh * rows + r;
            float l = 0.f;
            for (int b = t < 0 ? it.n_blk : 0; b < it.n_blk && ok; ++b) {
                const int m = n + b * it.n_tiles + t;
                const int x = m % kBufs, s = (ns + b) % kStages;
                const uint32_t fpar = ((ns + b) / kStages) & 1;
                const uint32_t buf = tm + kBuf0 + 128 * x + lane_base;
                ok = __all_sync(0xffffffffu, mbar_wait(&bars.sfull[half][x], (sphase >> x) & 1, abort));
                if (!ok) break;
                sphase ^= 1u << x;
                tc_fence_after();
                const int lim = it.cols - (it.b0 + b) * kBlk;  // columns below lim are visible
                uint64_t acc2[4] = {0ull, 0ull, 0ull, 0ull};
                if constexpr (SPLIT) {
#pragma unroll
                    for (int h = 0; h < 4; ++h) {  // 32 scores: 16 columns of high parts, 16 of low ones
                        uint32_t v[32], p[16];
                        tmem_ld32(buf + 32 * h, v);
                        tmem_ld_wait();
#pragma unroll
                        for (int y = 0; y < 32; ++y) v[y] = 32 * h + y < lim ? v[y] : 0u;
#pragma unroll
                        for (int y = 0; y < 16; ++y) {
                            const uint64_t s2 = f32x2_pack(v[2 * y], v[2 * y + 1]), w2 = f32x2_mul(s2, s2);
                            p[y] = f32x2_to_bf16x2(w2);
                            const uint64_t hi = f32x2_pack(p[y] << 16, p[y] & 0xFFFF0000u);
                            const uint32_t q = f32x2_to_bf16x2(f32x2_add(w2, hi ^ 0x8000000080000000ull));
                            v[y] = q;
                            acc2[y & 3] = f32x2_add(acc2[y & 3], f32x2_add(hi, f32x2_pack(q << 16, q & 0xFFFF0000u)));
                        }
                        tmem_st16(buf + 32 * h, p);
                        tmem_st16(buf + 32 * h + 16, v);
                    }
                } else
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
                // Values past the visible keys may be anything (NaN times a zero weight is
                // NaN): cleared in the block where the visible keys end, by every warp of
                // both halves before it hands its weights over.
                if (lim < kBlk) {
                    ok = __all_sync(0xffffffffu, mbar_wait(&bars.full[s], fpar, abort));
                    if (!ok) break;
                    uint8_t *op = sm_ring + s * kStage + kOp;
                    for (int k = lim + qd; k < kBlk; k += 4)
                        *reinterpret_cast<uint32_t *>(op + k * 128 + lane * 4) = 0u;
                    fence_proxy_async_smem();
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.pfull[half][x]);
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
                if (r < rows) {
                    if (it.part >= 0) {  // cut item: the row of the piece's slot
                        const long long pr = x_part_row(a.sched, it.part) + kXTile * t + row;
                        store_part(a.part + pr * a.d, o, a.d);
                        a.part_l[pr] = l;
                    } else {
                        store_row(a.o0 + gr * a.d, a.y ? a.y + gr * a.d : nullptr, o, cross_recip(l), a.d);
                        if (a.den) a.den[gr] = l;
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

}  // namespace

cudaError_t launch_cross_fwd_tc(const CrossPlan &p, const CrossIo &io, cudaStream_t st) {
    XLaunch x;
    cudaError_t e = x_launch(kCrossFwd, p, io, x);
    if (e != cudaSuccess) return e;
    const bool split = io.y && p.d <= 32;
    e = split ? smem_opt_in_once<cross_fwd_kernel<true>>(kSmem) : smem_opt_in_once<cross_fwd_kernel<false>>(kSmem);
    if (e != cudaSuccess) return e;
    auto *kernel = split ? cross_fwd_kernel<true> : cross_fwd_kernel<false>;
    ProfScope prof("cross_fwd", st);
    kernel<<<x.a.sched.grid, kXThreads, kSmem, st>>>(x.maps[0], x.maps[2], x.maps[3], x.a);
    return cudaGetLastError();
}

}  // namespace kata
