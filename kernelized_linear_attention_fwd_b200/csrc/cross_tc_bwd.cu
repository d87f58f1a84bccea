// Backward passes of cross attention on the tensor cores (formulas, roundings and
// work distribution: cross_tc.cu).
//
// A step is a 128-row tile against a block of 128 columns: two products form the
// scores S and P (128 columns of tensor memory each), 8 warps turn them into bf16
// weights, and one (dq) or two (dkv) products accumulate.  Tensor memory holds
//
//   0 .. 127    accumulators: dq: two of 64 columns, items in turn; dkv: dV, dK
//   128, 256    S of even and odd steps; the weights replace it: per 16 scores 8
//               columns of ds (dq) or of w / l and 8 of ds (dkv)
//   384         P, free again once the warps have read it
//
// so the next step's S is formed while this step's scores are turned, its P right
// after them, and a step's accumulation overlaps the next one's scores.  128-column
// score products run at the full rate (N = 64 ones pay for reading the 128-row
// operand twice as often: a 64-column form of these kernels took 1.6 times as long).
// One warp loads, one issues S, one P, two accumulate (dq: one).  dkv has 16 warps
// to turn scores into weights, 32 columns each of their 32 rows (8 warps of 64 columns
// took 207 us where 16 take 189: 4 heads-batches of 16 heads, 2048 queries, 4096 keys,
// ragged); dq, with half the arithmetic, has 8 (143 us; 16: 147).
#include "cross_tc.cuh"

namespace kata {
namespace {

// Groups of 4 warps that turn scores into weights, and the other warps behind them.
template <int MODE>
struct BCfg {
    static constexpr int kGroups = MODE == kCrossDq ? 2 : 4;
    static constexpr int kThreads = 32 * (4 * kGroups + 5);
    static constexpr int kTma = 4 * kGroups, kS = kTma + 1, kP = kTma + 2, kAcc = kTma + 3;
    static constexpr int kCols = kXCols / kGroups;  // columns of a step that a group turns
};
constexpr int kBSlot = 2 * 16384;    // an item's two row operands
constexpr int kBOp = kXCols * 128;   // one column operand of a block
constexpr int kBStage = 2 * kBOp;
constexpr int kBStat = 1024;         // dkv: -D and 1 / l of the block's queries
constexpr int kBStages = 4;
constexpr int kBSmem = 2 * kBSlot + kBStages * (kBStage + kBStat) + 1024;
constexpr uint32_t kBColS = 128, kBColP = 384;

struct BBars {
    uint64_t qfull[2], qempty[2], full[kBStages], empty[kBStages];
    // per S region: scores formed, weights stored, products done; P formed, P read
    uint64_t sfull[2], wfull[2], sfree[2], pfull, pfree;
    uint64_t ofull[2], ofree[2], drain[4];
};

template <int MODE>
__global__ void __launch_bounds__(BCfg<MODE>::kThreads, 1)
cross_bwd_kernel(const __grid_constant__ CUtensorMap tm_r0, const __grid_constant__ CUtensorMap tm_r1,
                 const __grid_constant__ CUtensorMap tm_c0, const __grid_constant__ CUtensorMap tm_c1,
                 const XArgs a) {
    constexpr bool kDkv = MODE == kCrossDkv;
    using Cfg = BCfg<MODE>;
    constexpr int kBGroups = Cfg::kGroups, kBCols = Cfg::kCols;
    constexpr int kBTma = Cfg::kTma, kBS = Cfg::kS, kBP = Cfg::kP, kBAcc = Cfg::kAcc;
    extern __shared__ uint8_t smem_raw[];
    __shared__ BBars bars;
    __shared__ XRange range;
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;

    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sm_ring = sm + 2 * kBSlot;
    uint8_t *sm_stat = sm_ring + kBStages * kBStage;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;

    if (tid == 0) {
        abort_flag = 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.qfull[i], 1);
            mbar_init(&bars.qempty[i], 2);  // both score warps
            mbar_init(&bars.sfull[i], 1);
            mbar_init(&bars.wfull[i], 4 * kBGroups);
            mbar_init(&bars.sfree[i], kDkv ? 2 : 1);
            mbar_init(&bars.ofull[i], 1);
            mbar_init(&bars.ofree[i], 4 * kBGroups / (kDkv ? 2 : 1));
        }
        for (int i = 0; i < 4; ++i) mbar_init(&bars.drain[i], 1);
        for (int i = 0; i < kBStages; ++i) {
            mbar_init(&bars.full[i], 1);
            mbar_init(&bars.empty[i], 1);
        }
        mbar_init(&bars.pfull, 1);
        mbar_init(&bars.pfree, 4 * kBGroups);
        fence_mbarrier_init();
    }
    if (warp == kBS) {
        tmem_alloc(&tmem_base, 512);
        tmem_relinquish();
    }
    if (warp == kBTma) {
        if (lane == 0) {
            tma_prefetch_desc(&tm_r0);
            tma_prefetch_desc(&tm_r1);
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
    griddep_wait();  // what ran before has ended: memory may be read and written
    const uint32_t tm = tmem_base;
    volatile int *abort = &abort_flag;
    XIter<MODE> iter(a.sched, range);
    XItem it;

    if (warp == kBTma) {
        // ------------------------------------------------------------ loads
        if (lane == 0) {
            if (!a.sched.whole) a.pieces[blockIdx.x] = XIter<MODE>::first(a.sched, range);
            int nq = 0, ns = 0;  // items and stages loaded
            XRing stage;
            bool ok = true;
            while (ok && iter.next(it)) {
                const int qb = nq & 1;
                ok = mbar_wait(&bars.qempty[qb], ((nq >> 1) & 1) ^ 1, abort);
                if (!ok) break;
                mbar_arrive_expect_tx(&bars.qfull[qb], kBSlot);
                tma_load_3d(sm + qb * kBSlot, &tm_r0, &bars.qfull[qb], 0, it.r0, it.bh);
                tma_load_3d(sm + qb * kBSlot + 16384, &tm_r1, &bars.qfull[qb], 0, it.r0, it.bh);
                ++nq;
                for (int b = 0; b < it.n_blk; ++b) {
                    const int s = stage.i;
                    ok = mbar_wait(&bars.empty[s], stage.phase ^ 1, abort);
                    if (!ok) break;
                    const int col = (it.b0 + b) * kXCols;
                    uint8_t *dst = sm_ring + s * kBStage;
                    // boxes of 64 columns; dq skips a second one without a visible key
                    const int boxes = kDkv || it.cols - col > 64 ? 2 : 1;
                    mbar_arrive_expect_tx(&bars.full[s], boxes * 16384 + (kDkv ? kBStat : 0));
                    for (int x = 0; x < boxes; ++x) {
                        tma_load_3d(dst + x * 8192, &tm_c0, &bars.full[s], 0, col + 64 * x, it.bh);
                        tma_load_3d(dst + kBOp + x * 8192, &tm_c1, &bars.full[s], 0, col + 64 * x, it.bh);
                    }
                    if (kDkv) {
                        const long long o = (long long)it.bh * a.stat_stride + col;
                        bulk_load(sm_stat + s * kBStat, a.delta + o, 512, &bars.full[s]);
                        bulk_load(sm_stat + s * kBStat + 512, a.rden + o, 512, &bars.full[s]);
                    }
                    ++ns;
                    stage.next(kBStages);
                }
            }
            // every load issued must have landed before the CTA exits
            for (int x = nq > 2 ? nq - 2 : 0; x < nq; ++x) mbar_wait_issued(&bars.qfull[x & 1], (x >> 1) & 1);
            for (int x = ns > kBStages ? ns - kBStages : 0; x < ns; ++x)
                mbar_wait_issued(&bars.full[x % kBStages], (x / kBStages) & 1);
        }
    } else if (warp == kBS || warp == kBP) {
        // ------------------------------------------------------------ products that form S, P
        if (lane == 0) {
            const int me = warp - kBS;
            const uint32_t id = idesc_bf16(128, 128, 0, 0);
            const uint64_t dR = desc_sw128(smem_u32(sm + 16384 * me), 16, 1024);
            const uint64_t dC = desc_sw128(smem_u32(sm_ring + kBOp * me), 16, 1024);
            const int n_ks = a.d / 16;  // the head's own coordinates: the columns past d are zeros
            XRing stage, buf;           // buf: S region (two), or the one of P
            int j = 0;
            uint32_t release = 0;  // warp kBS, per S region (4 bits): the stage + 1 its step reads
            bool ok = true;
            while (ok && iter.next(it)) {
                const int qb = j & 1;
                const uint64_t r = desc_at(dR, qb * kBSlot);
                ok = mbar_wait(&bars.qfull[qb], (j >> 1) & 1, abort);
                for (int b = 0; b < it.n_blk && ok; ++b) {
                    const uint64_t c = desc_at(dC, stage.i * kBStage);
                    const uint32_t col = tm + (me == 0 ? kBColS + 128 * buf.i : kBColP);
                    const uint32_t done = (release >> (4 * buf.i)) & 15u;
                    release = (release & ~(15u << (4 * buf.i))) | ((stage.i + 1u) << (4 * buf.i));
                    ok = mbar_wait(&bars.full[stage.i], stage.phase, abort) &&
                         mbar_wait(me == 0 ? &bars.sfree[buf.i] : &bars.pfree, buf.phase ^ 1, abort);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        if (ks < n_ks) mma_ss(col, desc_at(r, 32 * ks), desc_at(c, 32 * ks), id, ks > 0);
                    mma_commit(me == 0 ? &bars.sfull[buf.i] : &bars.pfull);
                    // a region found free: every product of the step that used it is done, so
                    // its stage is (P of that step was formed before its weights)
                    if (me == 0 && done) mbar_arrive(&bars.empty[done - 1]);
                    buf.next(me == 0 ? 2 : 1);
                    stage.next(kBStages);
                }
                if (!ok) break;
                mma_commit(&bars.qempty[qb]);
                ++j;
            }
            mma_commit(&bars.drain[me]);
            mbar_wait_issued(&bars.drain[me], 0);
        }
    } else if (warp >= kBAcc) {
        // ------------------------------------------------------------ products that accumulate
        if (lane == 0 && (kDkv || warp == kBAcc)) {
            const int me = warp - kBAcc;  // dkv: 0: dV from w / l and dY, 1: dK from ds and Q
            const uint32_t id = idesc_bf16(128, a.d, 0, 1);  // the head's own columns
            const uint64_t dC = desc_sw128(smem_u32(sm_ring + (kDkv && me == 0 ? kBOp : 0)), 8192, 1024);
            XRing stage, buf, acc;  // acc: dq, the accumulator of the item
            uint32_t ophase = 1;    // dkv: the accumulator's first use passes at once
            bool ok = true;
            while (ok && iter.next(it)) {
                const int o = kDkv ? me : acc.i;
                ok = mbar_wait(&bars.ofree[o], kDkv ? ophase : acc.phase ^ 1, abort);
                for (int b = 0; b < it.n_blk && ok; ++b) {
                    const uint64_t c = desc_at(dC, stage.i * kBStage);
                    const uint32_t w = tm + kBColS + 128 * buf.i + 8 * me;
                    ok = mbar_wait(&bars.full[stage.i], stage.phase, abort) &&
                         mbar_wait(&bars.wfull[buf.i], buf.phase, abort);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)
                        mma_ts(tm + 64 * o, w + 16 * ks, desc_at(c, 2048 * ks), id, b > 0 || ks > 0);
                    mma_commit(&bars.sfree[buf.i]);
                    buf.next(2);
                    stage.next(kBStages);
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
        const uint32_t tP = tm + kBColP + kBCols * grp + lane_base;
        XRing stage, buf, acc;
        uint32_t pphase = 0, ophase = 0;
        bool ok = true;
        zero_dead_rows<MODE>(a, warp, 4 * kBGroups, lane);
        __syncwarp();
        while (ok && iter.next(it)) {
            const int r = it.r0 + row;
            const long long gr = (long long)it.bh * rows + r, gs = (long long)it.bh * a.stat_stride + r;
            const float ndelta = !kDkv && r < rows ? a.delta[gs] : 0.f;
            const uint64_t nd = f32x2_pack(__float_as_uint(ndelta), __float_as_uint(ndelta));
            for (int b = 0; b < it.n_blk; ++b) {
                const int s = stage.i;
                const uint32_t tS = tm + kBColS + 128 * buf.i + kBCols * grp + lane_base;
                // of this group's columns, those visible (dkv masks none)
                const int lim = it.cols - (it.b0 + b) * kXCols - kBCols * grp;
                if constexpr (kDkv) {
                    // the block's -D and 1 / l (zeros past the last query)
                    ok = __all_sync(0xffffffffu, mbar_wait(&bars.full[s], stage.phase, abort));
                    if (!ok) break;
                }
                ok = __all_sync(0xffffffffu, mbar_wait(&bars.sfull[buf.i], buf.phase, abort) &&
                                                 mbar_wait(&bars.pfull, pphase, abort));
                if (!ok) break;
                tc_fence_after();
                if constexpr (kDkv) {
                    // Fragment layout: -D and 1 / l of 8 queries serve the thread's 4 rows.  (One
                    // row per thread would read all 32 columns' of each from shared memory.)
                    static_assert(!kDkv || kBCols == 32, "fragment loads of 32 columns");
                    const float2 *sd = reinterpret_cast<const float2 *>(sm_stat + s * kBStat) +
                                       (kBCols * grp) / 2 + lane % 4;
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
                            uint32_t w[4], e[4];
#pragma unroll
                            for (int y = 0; y < 4; ++y) {
                                const int j = 2 * h + y / 2, c = 8 * h + 2 * y;
                                const uint64_t s2 = f32x2_pack(v[c], v[c + 1]);
                                const uint64_t g2 = f32x2_pack(g[16 * u + c], g[16 * u + c + 1]);
                                const uint64_t d2 = f32x2_pack(__float_as_uint(fd[j].x), __float_as_uint(fd[j].y));
                                const uint64_t r2 = f32x2_pack(__float_as_uint(fr[j].x), __float_as_uint(fr[j].y));
                                const uint64_t sr2 = f32x2_mul(s2, r2);
                                w[y] = f32x2_to_bf16x2(f32x2_mul(s2, sr2));
                                e[y] = f32x2_to_bf16x2(f32x2_mul(sr2, f32x2_add(g2, d2)));
                            }
                            tmem_st_16x128b_x2(tSu + 16 * h, w);
                            tmem_st_16x128b_x2(tSu + 16 * h + 8, e);
                        }
                    }
                } else {
#pragma unroll
                    for (int h = 0; h < kBCols / 16; ++h) {
                        uint32_t v[16], g[16], w[8];
                        tmem_ld16(tP + 16 * h, g);
                        tmem_ld16(tS + 16 * h, v);
                        tmem_ld_wait();
                        if (h == kBCols / 16 - 1) {  // P is read: the next step's may be formed
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&bars.pfree);
                        }
                        if (lim < kBCols) {
#pragma unroll
                            for (int y = 0; y < 16; ++y) {
                                v[y] = 16 * h + y < lim ? v[y] : 0u;
                                g[y] = 16 * h + y < lim ? g[y] : 0u;
                            }
                        }
#pragma unroll
                        for (int y = 0; y < 8; ++y)
                            w[y] = f32x2_to_bf16x2(f32x2_mul(f32x2_pack(v[2 * y], v[2 * y + 1]),
                                                             f32x2_add(f32x2_pack(g[2 * y], g[2 * y + 1]), nd)));
                        tmem_st8(tS + 16 * h, w);
                    }
                }
                // dq: keys past the visible ones may be anything (NaN times a zero weight is
                // NaN): cleared in the block where the visible keys end
                if (!kDkv && lim < kBCols) {
                    ok = __all_sync(0xffffffffu, mbar_wait(&bars.full[s], stage.phase, abort));
                    if (!ok) break;
                    uint8_t *op = sm_ring + s * kBStage + kBCols * grp * 128;
                    for (int k = max(lim, 0) + qd; k < kBCols; k += 4)
                        *reinterpret_cast<uint32_t *>(op + k * 128 + lane * 4) = 0u;
                    fence_proxy_async_smem();
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.wfull[buf.i]);
                pphase ^= 1;
                buf.next(2);
                stage.next(kBStages);
            }
            if (!ok) break;
            // this group's columns of the item's accumulators: dq: 64 / groups of them; dkv: the
            // first groups dV's, the others dK's
            constexpr int N = kDkv ? 128 / kBGroups : 64 / kBGroups;
            const int ob = kDkv ? grp / (kBGroups / 2) : acc.i;
            const int c0 = kDkv ? N * (grp % (kBGroups / 2)) : N * grp;
            uint32_t o[64];
            ok = __all_sync(0xffffffffu, mbar_wait(&bars.ofull[ob], kDkv ? ophase : acc.phase, abort));
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < N; c += 16) tmem_ld16(tm + 64 * ob + c0 + c + lane_base, o + c);
            tmem_ld_wait();
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
    if (warp == kBS) tmem_dealloc(tm, 512);
    if (tid == 0 && abort_flag) atomicCAS(a.status, 0, (int)KATA_ERR_TIMEOUT);
}

template <int MODE>
cudaError_t launch_mode(const CrossPlan &p, const CrossIo &io, cudaStream_t st) {
    XLaunch x;
    cudaError_t e = x_launch(static_cast<CrossMode>(MODE), p, io, x);
    if (e != cudaSuccess) return e;
    if ((e = smem_opt_in_once<cross_bwd_kernel<MODE>>(kBSmem)) != cudaSuccess) return e;
    ProfScope prof(MODE == kCrossDq ? "cross_dq" : "cross_dkv", st);
    return launch_dependent(cross_bwd_kernel<MODE>, dim3(x.a.sched.grid), (unsigned)BCfg<MODE>::kThreads, kBSmem, st,
                            x.maps[0], x.maps[1], x.maps[2], x.maps[3], x.a);
}

}  // namespace

cudaError_t launch_cross_bwd_tc(CrossMode mode, const CrossPlan &p, const CrossIo &io, cudaStream_t st) {
    return mode == kCrossDq ? launch_mode<kCrossDq>(p, io, st) : launch_mode<kCrossDkv>(p, io, st);
}

}  // namespace kata
