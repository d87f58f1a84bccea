// Cross attention: the steps around the main kernels (cross_tc.cu, cross_f32.cu)
// that both types share: the backward pass's row statistics, and the joins of
// partial sums when a long axis was split over several CTAs.
#include <cuda_bf16.h>

#include "cross_sched.cuh"
#include "kata_internal.cuh"
#include "sm100.cuh"

namespace kata {
namespace {

// Row statistics of the backward pass: delta = -dy.y (y the forward's unrounded
// output) and 1 / den (0 for a row without weight), zeros in the padding up to
// R_pad.
__device__ __forceinline__ float dot8(const float *a, const float4 &x, const float4 &y) {
    const float4 u = *reinterpret_cast<const float4 *>(a), v = *reinterpret_cast<const float4 *>(a + 4);
    float s = u.x * x.x;
    s = fmaf(u.y, x.y, s);
    s = fmaf(u.z, x.z, s);
    s = fmaf(u.w, x.w, s);
    s = fmaf(v.x, y.x, s);
    s = fmaf(v.y, y.y, s);
    s = fmaf(v.z, y.z, s);
    return fmaf(v.w, y.w, s);
}
__device__ __forceinline__ float dot8(const __nv_bfloat16 *a, const float4 &x, const float4 &y) {
    const uint4 w = *reinterpret_cast<const uint4 *>(a);
    const float u[8] = {__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                        __uint_as_float(w.y & 0xFFFF0000u), __uint_as_float(w.z << 16),
                        __uint_as_float(w.z & 0xFFFF0000u), __uint_as_float(w.w << 16),
                        __uint_as_float(w.w & 0xFFFF0000u)};
    return dot8(u, x, y);
}

template <typename T>
__global__ void __launch_bounds__(256)
cross_stats_kernel(const T *dout, const float *y, const float *den, float *delta, float *rden, long long BH, int R,
                   int R_pad, int d) {
    const int lanes = d / 8, sub = threadIdx.x % lanes, per = 256 / lanes;  // 8 columns a lane
    const long long n = BH * R_pad, rows = (n + per - 1) / per;
    sm100::griddep_launch_dependents();
    for (long long b = blockIdx.x; b < rows; b += gridDim.x) {  // every warp whole, for the shuffles
        const long long x = b * per + threadIdx.x / lanes, bh = x / R_pad;
        const int r = (int)(x - bh * R_pad);
        float s = 0.f, rd = 0.f;
        if (x < n && r < R) {
            const long long o = (bh * R + r) * d + 8 * sub;
            const float4 *yy = reinterpret_cast<const float4 *>(y + o);
            s = dot8(dout + o, yy[0], yy[1]);
            rd = cross_recip(den[bh * R + r]);
        }
        for (int l = lanes / 2; l > 0; l >>= 1) s += __shfl_xor_sync(0xffffffffu, s, l);
        if (sub == 0 && x < n) {
            delta[x] = -s;
            rden[x] = rd;
        }
    }
}

// Joins the pieces of a row: sum over splits in order, by G groups of 16 threads
// each (thread = 4 columns), then the groups in order.  kJoinDen: divided by the
// summed denominators (forward; y and den exported if given); kJoinRow: times
// 2 / l of the row (dq); kJoinPlain: as is (dk, dv).
enum Join { kJoinDen, kJoinRow, kJoinPlain };
template <typename T, int JOIN, int G>
__global__ void __launch_bounds__(256)
cross_join_kernel(const float *part, const float *part_l, const float *rden, T *out, float *y, float *den,
                  long long n_rows, long long split_stride, int splits, int R, int R_pad, int d) {
    constexpr int kRows = 16 / G;
    __shared__ float4 red[16][16];
    __shared__ float red_l[16];
    sm100::griddep_wait();
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16, g = ty % G, c = 4 * tx;
    const long long row = (long long)blockIdx.x * kRows + ty / G;
    const bool on = row < n_rows;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
    if (on && c < d) {
#pragma unroll 4
        for (int x = g; x < splits; x += G) {
            const float4 v = *reinterpret_cast<const float4 *>(part + (x * split_stride + row) * d + c);
            s.x += v.x;
            s.y += v.y;
            s.z += v.z;
            s.w += v.w;
            if (JOIN == kJoinDen) l += part_l[x * split_stride + row];
        }
    }
    if (G > 1) {
        red[ty][tx] = s;
        if (JOIN == kJoinDen && tx == 0) red_l[ty] = l;
        __syncthreads();
        if (g > 0) return;
        s = red[ty][tx];
        l = JOIN == kJoinDen ? red_l[ty] : 0.f;
        for (int x = 1; x < G; ++x) {
            const float4 v = red[ty + x][tx];
            s.x += v.x;
            s.y += v.y;
            s.z += v.z;
            s.w += v.w;
            if (JOIN == kJoinDen) l += red_l[ty + x];
        }
    }
    if (!on || c >= d) return;
    float f = 1.f;
    if (JOIN == kJoinDen) f = cross_recip(l);
    if (JOIN == kJoinRow) f = 2.f * rden[row / R * R_pad + row % R];
    s.x *= f;
    s.y *= f;
    s.z *= f;
    s.w *= f;
    const long long o = row * d + c;
    store_out(out, o, s.x);
    store_out(out, o + 1, s.y);
    store_out(out, o + 2, s.z);
    store_out(out, o + 3, s.w);
    if (JOIN == kJoinDen) {
        if (y) *reinterpret_cast<float4 *>(y + o) = s;
        if (den && c == 0) den[row] = l;
    }
}

template <typename T, int JOIN>
cudaError_t launch_join(const CrossPlan &p, CrossMode mode, const float *part, const float *part_l,
                        const float *rden, void *out, float *y, float *den, long long n_rows,
                        long long split_stride, cudaStream_t st) {
    const int s = p.splits[mode];
    ProfScope prof("cross_join", st);
    const bool many = s > 8;
    return launch_dependent(many ? cross_join_kernel<T, JOIN, 16> : cross_join_kernel<T, JOIN, 1>,
                            dim3((unsigned)(many ? n_rows : (n_rows + 15) / 16)), 256u, 0, st, part, part_l, rden,
                            static_cast<T *>(out), y, den, n_rows, split_stride, s, p.R, p.R_pad, p.d);
}

// Joins the items that the schedule of the tensor cores and of few rows cut (cross_sched.cuh).  Grid x: the
// stretch boundaries c = 1 .. G - 1; the block of the first boundary inside an item
// adds the item's pieces in order: the end of CTA c - 1's stretch, then the starts
// of the later CTAs' up to the item's end, as the CTAs have recorded them.  A block
// of 256 threads takes 16 / G16 rows (grid y), thread = 4 columns of a row and every
// G16-th piece.
template <typename T, int MODE, int G16>
__global__ void __launch_bounds__(256)
cross_cut_join_kernel(const XSched s, const XPiece *pieces, const float *part, const float *part_l, const float *rden,
                     T *o0, T *o1, float *y, float *den, int grid, int R_pad, int d) {
    constexpr int kRows = 16 / G16;
    __shared__ float4 red[16][16];
    __shared__ float red_l[16];
    sm100::griddep_wait();
    const int c = blockIdx.x + 1, lane = threadIdx.x % 32;
    const XPiece me = pieces[c], prev = pieces[c - 1];
    const bool same = prev.bh == me.bh && prev.r0 == me.r0;
    if (me.bh < 0 || !me.cont || (same && prev.cont)) return;
    const int slot0 = 2 * (c - 1) + (same ? 0 : 1);  // the item began that CTA's stretch, or ended it
    int n = 2;                                       // pieces
    if (!me.last)
        for (int x = c + 1;; x += 32) {  // up to the CTA that reaches the item's end
            const bool end = x + lane >= grid || pieces[x + lane].last;
            const unsigned m = __ballot_sync(0xffffffffu, end);
            if (m) {
                n = x + __ffs(m) - c + 1;
                break;
            }
        }
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16, g = ty % G16, col = 4 * tx;
    const int row = blockIdx.y * kRows + ty / G16;  // of the slot
    // dkv: rows 0 .. 127 of a slot are dv's, the others dk's
    const int r = me.r0 + (MODE == kCrossDkv ? row % 128 : row);
    const bool on = r < s.rows && row < s.slot_rows && col < d;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
    if (on) {
#pragma unroll 4
        for (int x = g; x < n; x += G16) {
            const long long pr = (x == 0 ? slot0 : 2LL * (c - 1 + x)) * s.slot_rows + row;
            const float4 w = *reinterpret_cast<const float4 *>(part + pr * d + col);
            v.x += w.x;
            v.y += w.y;
            v.z += w.z;
            v.w += w.w;
            if (MODE == kCrossFwd) l += part_l[pr];
        }
    }
    if (G16 > 1) {
        red[ty][tx] = v;
        if (MODE == kCrossFwd && tx == 0) red_l[ty] = l;
        __syncthreads();
        if (g > 0) return;
        for (int x = 1; x < G16; ++x) {
            const float4 w = red[ty + x][tx];
            v.x += w.x;
            v.y += w.y;
            v.z += w.z;
            v.w += w.w;
        }
        if (MODE == kCrossFwd) {
            l = red_l[ty];
            for (int x = 1; x < G16; ++x) l += red_l[ty + x];
        }
    }
    if (!on) return;
    float f = 1.f;
    if (MODE == kCrossFwd) f = cross_recip(l);
    if (MODE == kCrossDq) f = 2.f * rden[(long long)me.bh * R_pad + r];
    if (MODE == kCrossDkv && row >= 128) f = 2.f;
    v.x *= f;
    v.y *= f;
    v.z *= f;
    v.w *= f;
    const long long gr = (long long)me.bh * s.rows + r, o = gr * d + col;
    T *dst = MODE == kCrossDkv && row >= 128 ? o1 : o0;
    store_out(dst, o, v.x);
    store_out(dst, o + 1, v.y);
    store_out(dst, o + 2, v.z);
    store_out(dst, o + 3, v.w);
    if (MODE == kCrossFwd) {
        if (y) *reinterpret_cast<float4 *>(y + o) = v;
        if (den && col == 0) den[gr] = l;
    }
}

template <typename T, int MODE>
cudaError_t launch_cut_join(const CrossPlan &p, const CrossIo &io, cudaStream_t st) {
    const XSched &s = p.sched[MODE];
    if (cross_whole(s, io) || s.grid == 1) return cudaSuccess;
    char *ws = static_cast<char *>(io.ws);
    const float *part = reinterpret_cast<const float *>(ws + p.ws_part[MODE]);
    const float *part_l = reinterpret_cast<const float *>(ws + p.ws_part_l);
    const float *rden = reinterpret_cast<const float *>(ws + p.ws_rden);
    T *o0 = static_cast<T *>(MODE == kCrossFwd ? io.out : MODE == kCrossDq ? io.dq : io.dv);
    T *o1 = static_cast<T *>(io.dk);
    // few rows: an item is cut into many pieces, which 16 threads share per 4 columns
    const bool few = s.slot_rows <= 64;
    const dim3 grid(s.grid - 1, few ? s.slot_rows : (s.slot_rows + 15) / 16);
    const XPiece *pieces = reinterpret_cast<const XPiece *>(ws + p.ws_pieces[MODE]);
    ProfScope prof("cross_join", st);
    return launch_dependent(few ? cross_cut_join_kernel<T, MODE, 16> : cross_cut_join_kernel<T, MODE, 1>, grid, 256u, 0, st, s,
                            pieces, part, part_l, rden, o0, o1, io.y, io.den, s.grid, p.R_pad, p.d);
}

cudaError_t launch_main(CrossMode mode, const CrossPlan &p, const CrossIo &io, cudaStream_t st) {
    if (mode == kCrossFwd && p.few) return launch_cross_few(p, io, st);
    if (p.dtype != KATA_BF16) return launch_cross_f32(mode, p, io, st);
    return launch_cross_tc(mode, p, io, st);
}

template <typename T>
cudaError_t forward(const CrossPlan &p, const CrossIo &io, cudaStream_t st) {
    cudaError_t e = launch_main(kCrossFwd, p, io, st);
    if (e == cudaSuccess && (p.few || p.dtype == KATA_BF16)) return launch_cut_join<T, kCrossFwd>(p, io, st);
    if (e != cudaSuccess || p.splits[kCrossFwd] == 1) return e;
    const char *ws = static_cast<const char *>(io.ws);
    return launch_join<T, kJoinDen>(p, kCrossFwd, reinterpret_cast<const float *>(ws + p.ws_part[kCrossFwd]),
                                    reinterpret_cast<const float *>(ws + p.ws_part_l), nullptr, io.out, io.y, io.den,
                                    p.BH * p.R, p.BH * p.R, st);
}

template <typename T>
cudaError_t backward(const CrossPlan &p, const CrossIo &io, cudaStream_t st) {
    char *ws = static_cast<char *>(io.ws);
    float *delta = reinterpret_cast<float *>(ws + p.ws_delta), *rden = reinterpret_cast<float *>(ws + p.ws_rden);
    {
        ProfScope prof("cross_stats", st);
        const long long per = 256 / (p.d / 8), blocks = (p.BH * p.R_pad + per - 1) / per, most = 16LL * kPlanSms;
        cross_stats_kernel<T><<<(unsigned)(blocks < most ? blocks : most), 256, 0, st>>>(
            static_cast<const T *>(io.dout), io.y, io.den, delta, rden, p.BH, p.R, p.R_pad, p.d);
    }
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if ((e = launch_main(kCrossDq, p, io, st)) != cudaSuccess) return e;
    if (p.dtype == KATA_BF16) {
        if ((e = launch_cut_join<T, kCrossDq>(p, io, st)) != cudaSuccess) return e;
        if ((e = launch_main(kCrossDkv, p, io, st)) != cudaSuccess) return e;
        return launch_cut_join<T, kCrossDkv>(p, io, st);
    }
    if (p.splits[kCrossDq] > 1) {
        e = launch_join<T, kJoinRow>(p, kCrossDq, reinterpret_cast<const float *>(ws + p.ws_part[kCrossDq]), nullptr,
                                     rden, io.dq, nullptr, nullptr, p.BH * p.R, p.BH * p.R, st);
        if (e != cudaSuccess) return e;
    }
    if ((e = launch_main(kCrossDkv, p, io, st)) != cudaSuccess) return e;
    if (p.splits[kCrossDkv] > 1) {
        const float *part = reinterpret_cast<const float *>(ws + p.ws_part[kCrossDkv]);
        const long long n = p.BH * p.Tk;
        e = launch_join<T, kJoinPlain>(p, kCrossDkv, part, nullptr, nullptr, io.dv, nullptr, nullptr, n, 2 * n, st);
        if (e != cudaSuccess) return e;
        e = launch_join<T, kJoinPlain>(p, kCrossDkv, part + n * p.d, nullptr, nullptr, io.dk, nullptr, nullptr, n,
                                       2 * n, st);
    }
    return e;
}

}  // namespace

cudaError_t launch_cross_forward(const CrossPlan &p, const CrossIo &io, cudaStream_t st) {
    return p.dtype == KATA_BF16 ? forward<__nv_bfloat16>(p, io, st) : forward<float>(p, io, st);
}
cudaError_t launch_cross_backward(const CrossPlan &p, const CrossIo &io, cudaStream_t st) {
    return p.dtype == KATA_BF16 ? backward<__nv_bfloat16>(p, io, st) : backward<float>(p, io, st);
}

}  // namespace kata
