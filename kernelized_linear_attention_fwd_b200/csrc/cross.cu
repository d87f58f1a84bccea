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
__device__ __forceinline__ float dot8(const float4 &u, const float4 &v, const float4 &x, const float4 &y) {
    float s = u.x * x.x;
    s = fmaf(u.y, x.y, s);
    s = fmaf(u.z, x.z, s);
    s = fmaf(u.w, x.w, s);
    s = fmaf(v.x, y.x, s);
    s = fmaf(v.y, y.y, s);
    s = fmaf(v.z, y.z, s);
    return fmaf(v.w, y.w, s);
}
__device__ __forceinline__ float dot8(const float *a, const float4 &x, const float4 &y) {
    const float4 *u = reinterpret_cast<const float4 *>(a);
    return dot8(u[0], u[1], x, y);
}
__device__ __forceinline__ float dot8(const __nv_bfloat16 *a, const float4 &x, const float4 &y) {
    const uint4 w = *reinterpret_cast<const uint4 *>(a);
    const float4 u = make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u),
                                 __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u));
    const float4 v = make_float4(__uint_as_float(w.z << 16), __uint_as_float(w.z & 0xFFFF0000u),
                                 __uint_as_float(w.w << 16), __uint_as_float(w.w & 0xFFFF0000u));
    return dot8(u, v, x, y);
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

// The joins of the fp32 kernels' pieces.  Sum over splits in order, by G groups of 16
// threads each (thread = 4 columns), then the groups in order.  kJoinDen: divided by
// the summed denominators (forward; y and den exported if given); kJoinRow: times
// 2 / l of the row (dq); kJoinPlain: as is (dk, dv).
enum Join { kJoinDen, kJoinRow, kJoinPlain };
struct SplitJob {
    const float *part, *part_l, *rden;
    float *out, *y, *den;
    long long n_rows, split_stride;
    int splits, R, R_pad, d;
};
template <int JOIN, int G>
__device__ void split_join(const SplitJob &j) {
    const float *part = j.part, *part_l = j.part_l, *rden = j.rden;
    float *out = j.out, *y = j.y, *den = j.den;
    const long long n_rows = j.n_rows, split_stride = j.split_stride;
    const int splits = j.splits, R = j.R, R_pad = j.R_pad, d = j.d;
    constexpr int kRows = 16 / G;
    __shared__ float4 red[16][16];
    __shared__ float red_l[16];
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
    *reinterpret_cast<float4 *>(out + o) = s;
    if (JOIN == kJoinDen) {
        if (y) *reinterpret_cast<float4 *>(y + o) = s;
        if (den && c == 0) den[row] = l;
    }
}

template <int G>
__global__ void __launch_bounds__(256)
split_join_forward(const SplitJob j) {
    sm100::griddep_wait();
    split_join<kJoinDen, G>(j);
}
// Grid z: dq, dv, dk (those with one piece are not joined: no rows).
template <int G>
__global__ void __launch_bounds__(256)
split_join_backward(const SplitJob q, const SplitJob v, const SplitJob k) {
    sm100::griddep_wait();
    if (blockIdx.z == 0)
        split_join<kJoinRow, G>(q);
    else
        split_join<kJoinPlain, G>(blockIdx.z == 1 ? v : k);
}
unsigned split_join_blocks(const SplitJob &j, int G) { return (unsigned)((j.n_rows + 16 / G - 1) / (16 / G)); }

// Joins the items that the schedule of the tensor cores and of few rows cut
// (cross_sched.cuh).  Grid x: the stretch boundaries c = 1 .. G - 1; the block of the first boundary inside an item
// adds the item's pieces in order: the end of CTA c - 1's stretch, then the starts
// of the later CTAs' up to the item's end, as the CTAs have recorded them.  A block
// of 256 threads takes 16 / G16 rows (grid y), thread = 4 columns of a row and every
// G16-th piece.
template <typename T>
struct CutJob {
    XSched s;
    const XPiece *pieces;
    const float *part, *part_l, *rden;
    T *o0, *o1;
    float *y, *den;
    int R_pad, d;
};
template <typename T, int MODE, int G16>
__device__ void cut_join(const CutJob<T> &j) {
    const XSched &s = j.s;
    const XPiece *pieces = j.pieces;
    const float *part = j.part, *part_l = j.part_l, *rden = j.rden;
    T *o0 = j.o0, *o1 = j.o1;
    float *y = j.y, *den = j.den;
    const int R_pad = j.R_pad, d = j.d, grid = s.grid;
    constexpr int kRows = 16 / G16;
    __shared__ float4 red[16][16];
    __shared__ float red_l[16];
    const int c = blockIdx.x + 1, lane = threadIdx.x % 32;
    if (c >= grid || (int)blockIdx.y * kRows >= s.slot_rows) return;
    const XPiece me = pieces[c], prev = pieces[c - 1];
    const bool same = prev.bh == me.bh && prev.r0 == me.r0;
    if (me.bh < 0 || !me.cont || (same && prev.cont)) return;
    const int slot0 = 2 * (c - 1) + (same ? 0 : 1);  // the item began that CTA's stretch, or ended it
    int n = 2;                                       // pieces
    if (!me.last)
        for (int x = c + 1, k = 4; k == 4; x += 128) {  // up to the CTA that reaches the item's end
            bool end[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) end[i] = x + 32 * i + lane >= grid || pieces[x + 32 * i + lane].last;
#pragma unroll
            for (int i = 3; i >= 0; --i) {
                const unsigned m = __ballot_sync(0xffffffffu, end[i]);
                if (m) {
                    n = x + 32 * i + __ffs(m) - c + 1;
                    k = i;
                }
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
#pragma unroll 8
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

// G16: as many threads per 4 columns as 16 where an item has few rows and so many
// pieces.
template <typename T, int G16>
__global__ void __launch_bounds__(256)
cut_join_forward(const CutJob<T> j) {
    sm100::griddep_wait();
    cut_join<T, kCrossFwd, G16>(j);
}
// Grid z: dq, dkv (grid 1: none cut).
template <typename T, int G16>
__global__ void __launch_bounds__(256)
cut_join_backward(const CutJob<T> q, const CutJob<T> kv) {
    sm100::griddep_wait();
    if (blockIdx.z == 0)
        cut_join<T, kCrossDq, G16>(q);
    else
        cut_join<T, kCrossDkv, 1>(kv);
}

template <typename T>
CutJob<T> cut_job(CrossMode mode, const CrossPlan &p, const CrossIo &io) {
    char *ws = static_cast<char *>(io.ws);
    CutJob<T> j;
    j.s = p.sched[mode];
    if (cross_whole(j.s, io)) j.s.grid = 1;  // nothing is cut
    j.pieces = reinterpret_cast<const XPiece *>(ws + p.ws_pieces[mode]);
    j.part = reinterpret_cast<const float *>(ws + p.ws_part[mode]);
    j.part_l = reinterpret_cast<const float *>(ws + p.ws_part_l);
    j.rden = reinterpret_cast<const float *>(ws + p.ws_rden);
    j.o0 = static_cast<T *>(mode == kCrossFwd ? io.out : mode == kCrossDq ? io.dq : io.dv);
    j.o1 = static_cast<T *>(io.dk);
    j.y = io.y;
    j.den = io.den;
    j.R_pad = p.R_pad;
    j.d = p.d;
    return j;
}
template <typename T>
dim3 cut_grid(const CutJob<T> &j, bool few) {
    return dim3(j.s.grid - 1, few ? j.s.slot_rows : (j.s.slot_rows + 15) / 16);
}

SplitJob split_job(CrossMode mode, const CrossPlan &p, const CrossIo &io) {
    const char *ws = static_cast<const char *>(io.ws);
    const long long n = p.BH * (mode == kCrossDkv ? p.Tk : p.R);
    SplitJob j;
    j.part = reinterpret_cast<const float *>(ws + p.ws_part[mode]);
    j.part_l = reinterpret_cast<const float *>(ws + p.ws_part_l);
    j.rden = reinterpret_cast<const float *>(ws + p.ws_rden);
    j.out = static_cast<float *>(mode == kCrossFwd ? io.out : mode == kCrossDq ? io.dq : io.dv);
    j.y = io.y;
    j.den = io.den;
    j.splits = p.splits[mode];
    j.n_rows = j.splits > 1 ? n : 0;
    j.split_stride = mode == kCrossDkv ? 2 * n : n;
    j.R = p.R;
    j.R_pad = p.R_pad;
    j.d = p.d;
    return j;
}

template <typename T>
cudaError_t forward(const CrossPlan &p, const CrossIo &io, cudaStream_t st) {
    const cudaError_t e = p.few                     ? launch_cross_few(p, io, st)
                          : p.dtype == KATA_BF16 ? launch_cross_tc_forward(p, io, st)
                                                 : launch_cross_f32_forward(p, io, st);
    if (e != cudaSuccess) return e;
    ProfScope prof("cross_join", st);
    if (p.few || p.dtype == KATA_BF16) {
        const CutJob<T> j = cut_job<T>(kCrossFwd, p, io);
        if (j.s.grid == 1) return cudaSuccess;
        const bool few = j.s.slot_rows <= 64;
        return launch_dependent(few ? cut_join_forward<T, 16> : cut_join_forward<T, 1>, cut_grid(j, few), 256u, 0, st,
                                j);
    }
    const SplitJob j = split_job(kCrossFwd, p, io);
    if (j.n_rows == 0) return cudaSuccess;
    const bool many = j.splits > 8;
    return launch_dependent(many ? split_join_forward<16> : split_join_forward<1>,
                            dim3(split_join_blocks(j, many ? 16 : 1)), 256u, 0, st, j);
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
    e = p.dtype == KATA_BF16 ? launch_cross_tc_backward(p, io, st) : launch_cross_f32_backward(p, io, st);
    if (e != cudaSuccess) return e;
    ProfScope prof("cross_join", st);
    if (p.dtype == KATA_BF16) {
        const CutJob<T> q = cut_job<T>(kCrossDq, p, io), kv = cut_job<T>(kCrossDkv, p, io);
        const bool few = q.s.slot_rows <= 64;
        dim3 grid = cut_grid(q, few);
        const dim3 g = cut_grid(kv, false);
        if (g.x > 0) grid = dim3(g.x > grid.x ? g.x : grid.x, g.y > grid.y ? g.y : grid.y, 2);
        if (grid.x == 0) return cudaSuccess;
        return launch_dependent(few ? cut_join_backward<T, 16> : cut_join_backward<T, 1>, grid, 256u, 0, st, q, kv);
    }
    const SplitJob q = split_job(kCrossDq, p, io), v = split_job(kCrossDkv, p, io);
    SplitJob k = v;
    k.part = v.part + (v.split_stride / 2) * p.d;
    k.out = static_cast<float *>(io.dk);
    const int G = q.splits > 8 || v.splits > 8 ? 16 : 1;
    const unsigned nq = split_join_blocks(q, G), nv = split_join_blocks(v, G);
    if (nq == 0 && nv == 0) return cudaSuccess;
    return launch_dependent(G == 16 ? split_join_backward<16> : split_join_backward<1>,
                            dim3(nq > nv ? nq : nv, 1, nv > 0 ? 3 : 1), 256u, 0, st, q, v, k);
}

}  // namespace

cudaError_t launch_cross_forward(const CrossPlan &p, const CrossIo &io, cudaStream_t st) {
    return p.dtype == KATA_BF16 ? forward<__nv_bfloat16>(p, io, st) : forward<float>(p, io, st);
}
cudaError_t launch_cross_backward(const CrossPlan &p, const CrossIo &io, cudaStream_t st) {
    return p.dtype == KATA_BF16 ? backward<__nv_bfloat16>(p, io, st) : backward<float>(p, io, st);
}

}  // namespace kata
