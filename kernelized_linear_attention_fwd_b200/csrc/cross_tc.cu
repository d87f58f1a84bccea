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
//   forward  rows = queries  S = Q K^T              O  += bf16(w) V
//   dq       rows = queries  S = Q K^T, P = dY V^T  dQ += bf16(s (p - D)) K
//   dkv      rows = keys     S = K Q^T, P = V dY^T  dV += bf16(w / l) dY
//                                                   dK += bf16(ds / 2) Q
//
// The weights are polynomial: no running maximum, no rescaling, so pieces of a
// long axis add up, and the backward pass recomputes s exactly as the forward
// did.  dq and dk, dv are formed by separate passes, each tile owned by one CTA:
// 14 d flops per (query, key) instead of 10, but no atomics, so results do not
// depend on order.
//
// Roundings to bf16: the weights (and ds) that go back into the tensor cores as
// operands, once each (or twice, SPLIT below).  The denominator is the product of the same rounded weights
// with a column of ones, in 16 columns more of the product with the values (which
// the 128-row operand's read pays for anyway), so that y is a convex combination of
// values to fp32: with one visible key y = v and, D being formed from the same y,
// the gradient of q and k is zero up to fp32 rounding instead of up to bf16
// rounding.  (8192 queries, 16384 keys, 8 heads: 295 us with the rounded weights summed
// by the warps, 265 us with the unrounded ones, 258 us this way.)
//
// Times in this file compare variants in short bursts, 20 launches of a captured graph,
// at the step that they were measured.  As it stands that prompt takes 243 us so, and 273
// to 289 us in an unbroken run, where the power cap lowers the clock.
//
// Schedule.  The work is a line of units, one per (128-row tile, column block),
// sequence by sequence; every CTA of the persistent grid takes an equal stretch
// of it (cross_sched.cuh), whatever the lengths, and walks the stretch item by
// item.  An item that a stretch boundary cuts is written as partial sums and
// joined (cross.cu).
//
// A step is one tile against one block.  Tensor memory holds
//
//   0 .. 127       accumulators: forward: O and l; dq: two of 64 columns, items in
//                  turn; dkv: dV and dK
//   128, 256       S of successive steps (forward: and 384); the weights replace it:
//                  per 16 scores 8 columns of w or ds (SPLIT: and 8 of low parts), or 8 of
//                  w / l and 8 of ds (SPLIT: their low parts 128 columns on, in the second
//                  region, which there is none of then)
//   384            dq, dkv: P, free again once the warps have read it
//
// so the next step's S is formed while this step's scores are turned, its P right
// after them, and a step's accumulation overlaps the next one's scores.  128-column
// score products run at the full rate (N = 64 ones pay for reading the 128-row
// operand twice as often: a 64-column form of the backward passes took 1.6 times as
// long).  One warp loads (TMA), one issues S, one P, one or two (dkv) accumulate.
// 16 warps turn scores into weights, 32 columns each of their 32 rows (dkv with 8 warps
// of 64 columns took 207 us where 16 take 189: 4 sequences of 16 heads, 2048 queries,
// 4096 keys, ragged); dq, with half of dkv's arithmetic, has 8 (143 us; 16: 147), and the
// forward, with a quarter, 8 (256 us; 16: 258).
#include "cross_tc.cuh"

namespace kata {
namespace {

// GROUPS: of 4 warps that turn scores into weights; the other warps come behind them.
template <int MODE, int GROUPS, bool SPLIT>
struct XCfg {
    static constexpr bool kFwd = MODE == kCrossFwd, kDkv = MODE == kCrossDkv;
    static constexpr int kGroups = GROUPS;
    static constexpr int kTma = 4 * kGroups, kS = kTma + 1, kP = kFwd ? -1 : kTma + 2, kAcc = kTma + (kFwd ? 2 : 3);
    static constexpr int kThreads = 32 * (kFwd ? kAcc + 1 : kAcc + 2);
    static constexpr int kCols = kXCols / kGroups;  // columns of a step that a group turns
    static constexpr int kRowOps = kFwd ? 1 : 2;
    static constexpr int kSlot = kRowOps * 16384;  // an item's row operands
    static constexpr int kOp = kXCols * 128;       // one column operand of a block
    static constexpr int kStage = 2 * kOp;
    static constexpr int kStages = kFwd ? 5 : 4;
    static constexpr int kStat = kDkv ? 1024 : 0;  // -D and 1 / l of the block's queries
    static constexpr int kOnes = kFwd ? 16384 : 0;  // a 128 x 64 operand of ones
    static constexpr int kSmem = 2 * kSlot + kStages * (kStage + kStat) + kOnes + 1024;
    // tensor memory: accumulators in columns 0 .. 127, regions of S, the one of P
    static constexpr int kRegions = kFwd ? 3 : kDkv && SPLIT ? 1 : 2;
    static constexpr uint32_t kLow = kDkv ? 128 : 8;  // SPLIT: from a part to its low part
    static constexpr uint32_t kColS = 128, kColP = 384;
};

// What two numbers lose by their rounding to bf16, as bf16.
__device__ __forceinline__ uint32_t low_part(uint64_t x, uint32_t rounded) {
    return f32x2_to_bf16x2(
        f32x2_add(x, f32x2_pack(rounded << 16, rounded & 0xFFFF0000u) ^ 0x8000000080000000ull));
}

template <typename C>
struct XBars {
    uint64_t qfull[2], qempty[2], full[C::kStages], empty[C::kStages];
    // per S region: scores formed (S and P of the step), weights stored, products done;
    // P read
    uint64_t sfull[C::kRegions], wfull[C::kRegions], sfree[C::kRegions], pfree;
    uint64_t ofull[2], ofree[2], drain[4];
};

// SPLIT: what goes back into the products (w, ds, w / l) as two bf16 numbers each, a
// high and a low part, which takes twice the products that accumulate.  Used by
// training steps (CrossPlan::split) where the rounding of one number would show, and by
// the forward of few rows:
//
// - The forward, d <= 32: its y gives the backward pass D = dy.y, and an error of D
//   enters every key's gradient with one sign: next to the other roundings it is as
//   1 / sqrt(d).  Also with up to 256 keys, whose roundings do not average out.
//   For d = 64 and many keys it would take half as long again (2048 queries on 4096 keys)
//   for an error of dq of 0.0024 either way.
// - dq, d = 16: dq is orthogonal to q, as y does not depend on q's length, while the
//   errors of ds lie mostly along q: 0.0025 of dq, rms (0.00166 of it the output's
//   rounding), without, 0.0017 with it.
// - dq and dkv with up to 32 rows or 32 keys: few roundings enter a sum, and with two
//   keys, say, p and D cancel (1.6 to 2.4 times the output's own rounding without).
// - Any forward of up to 32 rows: outputs so few show single roundings.
template <int MODE, int GROUPS, bool SPLIT>
__device__ __forceinline__ void cross_tc(const CUtensorMap &tm_r0, const CUtensorMap &tm_r1, const CUtensorMap &tm_c0,
                                         const CUtensorMap &tm_c1, const XArgs &a, int cta) {
    using C = XCfg<MODE, GROUPS, SPLIT>;
    constexpr bool kFwd = C::kFwd, kDkv = C::kDkv;
    extern __shared__ uint8_t smem_raw[];
    __shared__ XBars<C> bars;
    __shared__ XRange range;
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;

    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sm_ring = sm + 2 * C::kSlot;
    uint8_t *sm_stat = sm_ring + C::kStages * C::kStage, *sm_ones = sm_stat;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;

    if (kFwd) {
        for (int x = tid; x < C::kOnes / 4; x += C::kThreads) reinterpret_cast<uint32_t *>(sm_ones)[x] = 0x3F803F80u;
        fence_proxy_async_smem();
    }
    if (tid == 0) {
        abort_flag = 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.qfull[i], 1);
            mbar_init(&bars.qempty[i], C::kRowOps);  // the warps that form scores
            mbar_init(&bars.ofull[i], 1);
            mbar_init(&bars.ofree[i], 4 * C::kGroups / (kDkv ? 2 : 1));
        }
        for (int i = 0; i < 4; ++i) mbar_init(&bars.drain[i], 1);
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&bars.full[i], 1);
            mbar_init(&bars.empty[i], 1);
        }
        for (int i = 0; i < C::kRegions; ++i) {
            mbar_init(&bars.sfull[i], C::kRowOps);
            mbar_init(&bars.wfull[i], 4 * C::kGroups);
            mbar_init(&bars.sfree[i], kDkv ? 2 : 1);
        }
        mbar_init(&bars.pfree, 4 * C::kGroups);
        fence_mbarrier_init();
    }
    if (warp == C::kS) {
        tmem_alloc(&tmem_base, 512);
        tmem_relinquish();
    }
    if (warp == C::kTma) {
        if (lane == 0) {
            tma_prefetch_desc(&tm_r0);
            if (!kFwd) tma_prefetch_desc(&tm_r1);
            tma_prefetch_desc(&tm_c0);
            tma_prefetch_desc(&tm_c1);
        }
        __syncwarp();
        const XRange r = x_range<MODE>(a.sched, cta, lane);
        if (lane == 0) range = r;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_wait();  // what ran before has ended: memory may be read and written
    const uint32_t tm = tmem_base;
    volatile int *abort = &abort_flag;
    XIter<MODE> iter(a.sched, range, cta);
    XItem it;

    if (warp == C::kTma) {
        // ------------------------------------------------------------ loads
        if (lane == 0) {
            if (!a.sched.whole) a.pieces[cta] = XIter<MODE>::first(a.sched, range);
            int nq = 0, ns = 0;  // items and stages loaded
            XRing stage;
            bool ok = true;
            while (ok && iter.next(it)) {
                const int qb = nq & 1;
                ok = mbar_wait(&bars.qempty[qb], ((nq >> 1) & 1) ^ 1, abort);
                if (!ok) break;
                mbar_arrive_expect_tx(&bars.qfull[qb], C::kSlot);
                tma_load_3d(sm + qb * C::kSlot, &tm_r0, &bars.qfull[qb], 0, it.r0, it.bh);
                if (!kFwd) tma_load_3d(sm + qb * C::kSlot + 16384, &tm_r1, &bars.qfull[qb], 0, it.r0, it.bh);
                ++nq;
                for (int b = 0; b < it.n_blk; ++b) {
                    const int s = stage.i;
                    ok = mbar_wait(&bars.empty[s], stage.phase ^ 1, abort);
                    if (!ok) break;
                    const int col = (it.b0 + b) * kXCols;
                    uint8_t *dst = sm_ring + s * C::kStage;
                    // boxes of 64 columns; of keys, a second one without a visible key is skipped
                    const int boxes = kDkv || it.cols - col > 64 ? 2 : 1;
                    mbar_arrive_expect_tx(&bars.full[s], boxes * 16384 + (kDkv ? C::kStat : 0));
                    for (int x = 0; x < boxes; ++x) {
                        tma_load_3d(dst + x * 8192, &tm_c0, &bars.full[s], 0, col + 64 * x, it.bh);
                        tma_load_3d(dst + C::kOp + x * 8192, &tm_c1, &bars.full[s], 0, col + 64 * x, it.bh);
                    }
                    if (kDkv) {
                        const long long o = (long long)it.bh * a.stat_stride + col;
                        bulk_load(sm_stat + s * C::kStat, a.delta + o, 512, &bars.full[s]);
                        bulk_load(sm_stat + s * C::kStat + 512, a.rden + o, 512, &bars.full[s]);
                    }
                    ++ns;
                    stage.next(C::kStages);
                }
            }
            // every load issued must have landed before the CTA exits
            for (int x = nq > 2 ? nq - 2 : 0; x < nq; ++x) mbar_wait_issued(&bars.qfull[x & 1], (x >> 1) & 1);
            for (int x = ns > C::kStages ? ns - C::kStages : 0; x < ns; ++x)
                mbar_wait_issued(&bars.full[x % C::kStages], (x / C::kStages) & 1);
        }
    } else if (warp == C::kS || warp == C::kP) {
        // ------------------------------------------------------------ products that form S, P
        if (lane == 0) {
            const int me = warp - C::kS;
            const uint32_t id = idesc_bf16(128, 128, 0, 0);
            const uint64_t dR = desc_sw128(smem_u32(sm + 16384 * me), 16, 1024);
            const uint64_t dC = desc_sw128(smem_u32(sm_ring + C::kOp * me), 16, 1024);
            const int n_ks = a.d / 16;  // the head's own coordinates: the columns past d are zeros
            XRing stage, buf;           // buf: the step's S region
            uint32_t pphase = 1;        // P's region: the first use passes at once
            int j = 0;
            uint32_t release = 0;  // warp C::kS, per S region (4 bits): the stage + 1 its step reads
            bool ok = true;
            while (ok && iter.next(it)) {
                const int qb = j & 1;
                const uint64_t r = desc_at(dR, qb * C::kSlot);
                ok = mbar_wait(&bars.qfull[qb], (j >> 1) & 1, abort);
                for (int b = 0; b < it.n_blk && ok; ++b) {
                    const uint64_t c = desc_at(dC, stage.i * C::kStage);
                    const uint32_t col = tm + (me == 0 ? C::kColS + 128 * buf.i : C::kColP);
                    const uint32_t done = (release >> (4 * buf.i)) & 15u;
                    release = (release & ~(15u << (4 * buf.i))) | ((stage.i + 1u) << (4 * buf.i));
                    ok = mbar_wait(&bars.full[stage.i], stage.phase, abort) &&
                         (me == 0 ? mbar_wait(&bars.sfree[buf.i], buf.phase ^ 1, abort)
                                  : mbar_wait(&bars.pfree, pphase, abort));
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        if (ks < n_ks) mma_ss(col, desc_at(r, 32 * ks), desc_at(c, 32 * ks), id, ks > 0);
                    mma_commit(&bars.sfull[buf.i]);
                    // a region found free: every product of the step that used it is done, so
                    // its stage is (P of that step was formed before its weights)
                    if (me == 0 && done) mbar_arrive(&bars.empty[done - 1]);
                    buf.next(C::kRegions);
                    pphase ^= 1;
                    stage.next(C::kStages);
                }
                if (!ok) break;
                mma_commit(&bars.qempty[qb]);
                ++j;
            }
            mma_commit(&bars.drain[me]);
            mbar_wait_issued(&bars.drain[me], 0);
        }
    } else if (warp >= C::kAcc) {
        // ------------------------------------------------------------ products that accumulate
        if (lane == 0 && (kDkv || warp == C::kAcc)) {
            const int me = warp - C::kAcc;  // dkv: 0: dV from w / l and dY, 1: dK from ds and Q
            // the head's own columns; forward: the block's values and, 64 columns on, ones, whose
            // product with the weights is the denominator
            const uint32_t id = idesc_bf16(128, kFwd ? 80 : a.d, 0, 1);
            const uint8_t *op = sm_ring + (kFwd || (kDkv && me == 0) ? C::kOp : 0);
            const uint64_t dC = desc_sw128(smem_u32(op), kFwd ? smem_u32(sm_ones) - smem_u32(op) : 8192, 1024);
            XRing stage, buf, acc;  // acc: dq: the accumulator of the item
            uint32_t ophase = 1;    // forward, dkv: the accumulator's first use passes at once
            bool ok = true;
            while (ok && iter.next(it)) {
                const int o = MODE == kCrossDq ? acc.i : me;
                ok = mbar_wait(&bars.ofree[o], MODE == kCrossDq ? acc.phase ^ 1 : ophase, abort);
                for (int b = 0; b < it.n_blk && ok; ++b) {
                    uint64_t c = desc_at(dC, stage.i * C::kStage);
                    // the ones stay where they are: the distance to them shrinks
                    if (kFwd) c -= static_cast<uint64_t>((stage.i * C::kStage) >> 4) << 16;
                    const uint32_t w = tm + C::kColS + 128 * buf.i + 8 * me;
                    // that the stage has landed is the warps' wait in the forward, whose steps this
                    // warp bounds (256 us here, 245 there), and this warp's in dq and dkv
                    ok = (kFwd || mbar_wait(&bars.full[stage.i], stage.phase, abort)) &&
                         mbar_wait(&bars.wfull[buf.i], buf.phase, abort);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)
                        mma_ts(tm + 64 * o, w + 16 * ks, desc_at(c, 2048 * ks), id, b > 0 || ks > 0);
                    if (SPLIT) {
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks)
                            mma_ts(tm + 64 * o, w + 16 * ks + C::kLow, desc_at(c, 2048 * ks), id, 1);
                    }
                    mma_commit(&bars.sfree[buf.i]);
                    buf.next(C::kRegions);
                    stage.next(C::kStages);
                }
                if (!ok) break;
                mma_commit(&bars.ofull[o]);
                ophase ^= 1;
                acc.next(2);
            }
            mma_commit(&bars.drain[2 + me]);
            mbar_wait_issued(&bars.drain[2 + me], 0);
        }
    } else {
        // ------------------------------------------------------------ weights and epilogue
        const int grp = warp / 4, qd = warp % 4;
        const int row = 32 * qd + lane;
        const uint32_t lane_base = static_cast<uint32_t>(32 * qd) << 16;
        const int rows = a.sched.rows;
        const uint32_t tP = tm + C::kColP + C::kCols * grp + lane_base;
        XRing stage, buf, acc;
        uint32_t ophase = 0;
        bool ok = true;
        zero_dead_rows<MODE>(a, cta, warp, 4 * C::kGroups, lane);
        __syncwarp();
        while (ok && iter.next(it)) {
            const int r = it.r0 + row;
            const long long gr = (long long)it.bh * rows + r, gs = (long long)it.bh * a.stat_stride + r;
            const float ndelta = MODE == kCrossDq && r < rows ? a.delta[gs] : 0.f;
            const uint64_t nd = f32x2_pack(__float_as_uint(ndelta), __float_as_uint(ndelta));
            for (int b = 0; b < it.n_blk; ++b) {
                const int s = stage.i;
                const uint32_t tS = tm + C::kColS + 128 * buf.i + C::kCols * grp + lane_base;
                // of this group's columns, those visible (dkv masks none)
                const int lim = it.cols - (it.b0 + b) * kXCols - C::kCols * grp;
                if constexpr (kDkv) {
                    // the block's -D and 1 / l (zeros past the last query)
                    ok = __all_sync(0xffffffffu, mbar_wait(&bars.full[s], stage.phase, abort));
                    if (!ok) break;
                }
                ok = __all_sync(0xffffffffu, mbar_wait(&bars.sfull[buf.i], buf.phase, abort));
                if (!ok) break;
                tc_fence_after();
                if constexpr (kFwd) {
#pragma unroll
                    for (int g = 0; g < C::kCols / 32; ++g) {
                        uint32_t v[32];
                        tmem_ld32(tS + 32 * g, v);
                        tmem_ld_wait();
                        if (lim < C::kCols) {
#pragma unroll
                            for (int y = 0; y < 32; ++y) v[y] = 32 * g + y < lim ? v[y] : 0u;
                        }
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t w[8], e[8];
#pragma unroll
                            for (int y = 0; y < 8; ++y) {
                                const uint64_t s2 = f32x2_pack(v[16 * h + 2 * y], v[16 * h + 2 * y + 1]);
                                const uint64_t w2 = f32x2_mul(s2, s2);
                                w[y] = f32x2_to_bf16x2(w2);
                                if (SPLIT) e[y] = low_part(w2, w[y]);
                            }
                            tmem_st8(tS + 32 * g + 16 * h, w);
                            if (SPLIT) tmem_st8(tS + 32 * g + 16 * h + C::kLow, e);
                        }
                    }
                } else if constexpr (kDkv) {
                    // Fragment layout: -D and 1 / l of 8 queries serve the thread's 4 rows.  (One
                    // row per thread would read all 32 columns' of each from shared memory.)
                    static_assert(!kDkv || C::kCols == 32, "fragment loads of 32 columns");
                    const float2 *sd = reinterpret_cast<const float2 *>(sm_stat + s * C::kStat) +
                                       (C::kCols * grp) / 2 + lane % 4;
                    // P first, all of it: the next step's may then be formed under this one's arithmetic
                    uint32_t g[32];
                    tmem_ld_16x256b_x4(tP, g);
                    tmem_ld_16x256b_x4(tP + (16u << 16), g + 16);
                    tmem_ld_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars.pfree);
                    float2 fd[4], fr[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        fd[j] = sd[4 * j];
                        fr[j] = sd[64 + 4 * j];
                    }
#pragma unroll
                    for (int u = 0; u < 2; ++u) {  // lanes 0 .. 15, 16 .. 31
                        const uint32_t tSu = tS + (static_cast<uint32_t>(16 * u) << 16);
                        uint32_t v[16];
                        tmem_ld_16x256b_x4(tSu, v);
                        tmem_ld_wait();
#pragma unroll
                        for (int h = 0; h < 2; ++h) {  // 16 columns: 8 of w / l, 8 of ds / 2
                            uint32_t w[4], e[4], wl[4], el[4];
#pragma unroll
                            for (int y = 0; y < 4; ++y) {
                                const int j = 2 * h + y / 2, c = 8 * h + 2 * y;
                                const uint64_t s2 = f32x2_pack(v[c], v[c + 1]);
                                const uint64_t g2 = f32x2_pack(g[16 * u + c], g[16 * u + c + 1]);
                                const uint64_t d2 = f32x2_pack(__float_as_uint(fd[j].x), __float_as_uint(fd[j].y));
                                const uint64_t r2 = f32x2_pack(__float_as_uint(fr[j].x), __float_as_uint(fr[j].y));
                                const uint64_t sr2 = f32x2_mul(s2, r2);
                                const uint64_t w2 = f32x2_mul(s2, sr2), e2 = f32x2_mul(sr2, f32x2_add(g2, d2));
                                w[y] = f32x2_to_bf16x2(w2);
                                e[y] = f32x2_to_bf16x2(e2);
                                if (SPLIT) {
                                    wl[y] = low_part(w2, w[y]);
                                    el[y] = low_part(e2, e[y]);
                                }
                            }
                            if (SPLIT) {
                                tmem_st_16x128b_x2(tSu + 16 * h + C::kLow, wl);
                                tmem_st_16x128b_x2(tSu + 16 * h + 8 + C::kLow, el);
                            }
                            tmem_st_16x128b_x2(tSu + 16 * h, w);
                            tmem_st_16x128b_x2(tSu + 16 * h + 8, e);
                        }
                    }
                } else {
#pragma unroll
                    for (int h = 0; h < C::kCols / 16; ++h) {
                        uint32_t v[16], g[16], w[8], e[8];
                        tmem_ld16(tP + 16 * h, g);
                        tmem_ld16(tS + 16 * h, v);
                        tmem_ld_wait();
                        if (h == C::kCols / 16 - 1) {  // P is read: the next step's may be formed
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&bars.pfree);
                        }
                        if (lim < C::kCols) {
#pragma unroll
                            for (int y = 0; y < 16; ++y) {
                                v[y] = 16 * h + y < lim ? v[y] : 0u;
                                g[y] = 16 * h + y < lim ? g[y] : 0u;
                            }
                        }
#pragma unroll
                        for (int y = 0; y < 8; ++y) {
                            const uint64_t e2 = f32x2_mul(f32x2_pack(v[2 * y], v[2 * y + 1]),
                                                          f32x2_add(f32x2_pack(g[2 * y], g[2 * y + 1]), nd));
                            w[y] = f32x2_to_bf16x2(e2);
                            if (SPLIT) e[y] = low_part(e2, w[y]);
                        }
                        tmem_st8(tS + 16 * h, w);
                        if (SPLIT) tmem_st8(tS + 16 * h + C::kLow, e);
                    }
                }
                // keys (forward: values) past the visible ones may be anything (NaN times a zero
                // weight is NaN): cleared in the block where the visible keys end
                if (!kDkv && lim < C::kCols) {
                    ok = __all_sync(0xffffffffu, mbar_wait(&bars.full[s], stage.phase, abort));
                    if (!ok) break;
                    uint8_t *op = sm_ring + s * C::kStage + (kFwd ? C::kOp : 0) + C::kCols * grp * 128;
                    for (int k = max(lim, 0) + qd; k < C::kCols; k += 4)
                        *reinterpret_cast<uint32_t *>(op + k * 128 + lane * 4) = 0u;
                    fence_proxy_async_smem();
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (kFwd) ok = mbar_wait(&bars.full[s], stage.phase, abort);
                    if (ok) mbar_arrive(&bars.wfull[buf.i]);
                }
                if (kFwd) ok = __shfl_sync(0xffffffffu, ok, 0);
                if (kFwd && !ok) break;
                buf.next(C::kRegions);
                stage.next(C::kStages);
            }
            if (!ok) break;
            // this group's columns of the item's accumulators: forward, dq: 64 / groups of
            // them; dkv: the first groups dV's, the others dK's
            constexpr int N = kDkv ? 128 / C::kGroups : 64 / C::kGroups;
            const int ob = kDkv ? grp / (C::kGroups / 2) : kFwd ? 0 : acc.i;
            const int c0 = kDkv ? N * (grp % (C::kGroups / 2)) : N * grp;
            uint32_t o[64];
            ok = __all_sync(0xffffffffu, mbar_wait(&bars.ofull[ob], MODE == kCrossDq ? acc.phase : ophase, abort));
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < N; c += 16) tmem_ld16(tm + 64 * ob + c0 + c + lane_base, o + c);
            uint32_t den[8];  // forward: the denominator, in each of the 16 columns from 64 on
            if (kFwd) tmem_ld8(tm + 64 + lane_base, den);
            tmem_ld_wait();
            const float l = kFwd ? __uint_as_float(den[0]) : 0.f;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.ofree[ob]);
            if (kDkv && r >= it.live) {  // keys past the visible ones, whatever they hold
#pragma unroll
                for (int c = 0; c < N; ++c) o[c] = 0u;
            }
            if (r < rows && c0 < a.d) {
                const int nc = min(N, a.d - c0);
                if (it.part >= 0) {  // cut item: the row of the piece's slot (dkv: dv's rows, then dk's)
                    const long long pr = x_part_row(a.sched, it.part) + row + (kDkv ? kXTile * ob : 0);
                    store_part(a.part + pr * a.d + c0, o, nc);
                    if (kFwd && grp == 0) a.part_l[pr] = l;
                } else if (kFwd) {
                    store_row(a.o0 + gr * a.d + c0, a.y ? a.y + gr * a.d + c0 : nullptr, o, cross_recip(l), nc);
                    if (a.den && grp == 0) a.den[gr] = l;
                } else {
                    const float f = !kDkv ? 2.f * a.rden[gs] : ob ? 2.f : 1.f;
                    store_row((kDkv && ob ? a.o1 : a.o0) + gr * a.d + c0, nullptr, o, f, nc);
                }
            }
            __syncwarp();
            ophase ^= 1;
            acc.next(2);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == C::kS) tmem_dealloc(tm, 512);
    if (tid == 0 && abort_flag) atomicCAS(a.status, 0, (int)KATA_ERR_TIMEOUT);
}

constexpr int x_groups(int mode) { return mode == kCrossDkv ? 4 : 2; }

template <int MODE, bool SPLIT>
__global__ void __launch_bounds__(XCfg<MODE, x_groups(MODE), SPLIT>::kThreads, 1)
cross_tc_kernel(const __grid_constant__ XLaunch x) {
    cross_tc<MODE, x_groups(MODE), SPLIT>(x.maps[0], x.maps[1], x.maps[2], x.maps[3], x.a, blockIdx.x);
}

// dq and dkv side by side, the SMs shared out by their work: for problems so small
// that a launch's start and end count (two sequences of 8 query heads on 2 key
// heads, 1021 queries, 1999 keys, d = 32: 19 and 25 us and a join each, or 37 us and one
// join).
template <bool SPLIT_Q, bool SPLIT_KV>
__global__ void __launch_bounds__(XCfg<kCrossDkv, 4, SPLIT_KV>::kThreads, 1)
cross_tc_both(const __grid_constant__ XLaunch q, const __grid_constant__ XLaunch kv) {
    if ((int)blockIdx.x < kv.a.sched.grid)
        cross_tc<kCrossDkv, 4, SPLIT_KV>(kv.maps[0], kv.maps[1], kv.maps[2], kv.maps[3], kv.a, blockIdx.x);
    else
        cross_tc<kCrossDq, 4, SPLIT_Q>(q.maps[0], q.maps[1], q.maps[2], q.maps[3], q.a,
                                     blockIdx.x - kv.a.sched.grid);
}

template <int MODE, bool SPLIT>
cudaError_t launch_mode(const CrossPlan &p, const CrossIo &io, cudaStream_t st) {
    using C = XCfg<MODE, x_groups(MODE), SPLIT>;
    XLaunch x;
    cudaError_t e = x_launch(static_cast<CrossMode>(MODE), p, io, x);
    if (e != cudaSuccess) return e;
    if ((e = smem_opt_in_once<cross_tc_kernel<MODE, SPLIT>>(C::kSmem)) != cudaSuccess) return e;
    ProfScope prof(MODE == kCrossFwd ? "cross_fwd" : MODE == kCrossDq ? "cross_dq" : "cross_dkv", st);
    if (MODE == kCrossFwd) {  // the call's first kernel
        cross_tc_kernel<MODE, SPLIT><<<x.a.sched.grid, C::kThreads, C::kSmem, st>>>(x);
        return cudaGetLastError();
    }
    return launch_dependent(cross_tc_kernel<MODE, SPLIT>, dim3(x.a.sched.grid), (unsigned)C::kThreads, C::kSmem, st, x);
}

template <bool SPLIT_Q, bool SPLIT_KV>
cudaError_t launch_backward(const CrossPlan &p, const CrossIo &io, cudaStream_t st) {
    if (!p.together) {
        const cudaError_t e = launch_mode<kCrossDq, SPLIT_Q>(p, io, st);
        return e != cudaSuccess ? e : launch_mode<kCrossDkv, SPLIT_KV>(p, io, st);
    }
    using C = XCfg<kCrossDkv, 4, SPLIT_KV>;
    XLaunch q, kv;
    cudaError_t e = x_launch(kCrossDq, p, io, q);
    if (e == cudaSuccess) e = x_launch(kCrossDkv, p, io, kv);
    if (e == cudaSuccess) e = smem_opt_in_once<cross_tc_both<SPLIT_Q, SPLIT_KV>>(C::kSmem);
    if (e != cudaSuccess) return e;
    ProfScope prof("cross_bwd", st);
    return launch_dependent(cross_tc_both<SPLIT_Q, SPLIT_KV>, dim3(q.a.sched.grid + kv.a.sched.grid), (unsigned)C::kThreads,
                            C::kSmem, st, q, kv);
}

}  // namespace

cudaError_t launch_cross_tc_forward(const CrossPlan &p, const CrossIo &io, cudaStream_t st) {
    const bool split = io.y ? p.split[kCrossFwd] : p.R <= kSplitRows;
    return split ? launch_mode<kCrossFwd, true>(p, io, st) : launch_mode<kCrossFwd, false>(p, io, st);
}
cudaError_t launch_cross_tc_backward(const CrossPlan &p, const CrossIo &io, cudaStream_t st) {
    if (p.split[kCrossDkv]) return launch_backward<true, true>(p, io, st);
    return p.split[kCrossDq] ? launch_backward<true, false>(p, io, st) : launch_backward<false, false>(p, io, st);
}

}  // namespace kata
