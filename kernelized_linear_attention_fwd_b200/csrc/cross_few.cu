// Cross attention forward for few rows (at most 4 per key head: decode steps), bf16
// and fp32, on the CUDA cores: y = sum_s w v / sum_s w, w = (q.k)^2.
//
// Bound by reading the keys and values once.  64 sequences of 1501 keys and less, 16
// heads, one query (270 MB): 45 us, 6.0 TB/s, against 60 us on the tensor cores, whose
// one group of warps per item takes longer over 128 rows of scores than their
// block's loads.  Past 4 rows the registers of the rows' accumulators crowd out the
// loads in flight (8 rows, 2 key heads of 131072 keys: 63 us against 18 there).
//
// The work is cut as in the tensor-core kernels (cross_sched.cuh): CTAs of 8 warps
// take equal stretches of 128-key blocks.  d / 8 lanes hold 8 coordinates each of a
// key, a warp 32 / (d / 8) keys at a time; per block every warp has its 16 keys' loads
// in flight.  Scores are summed over a key's lanes by shuffles; the accumulators of
// the keys' lanes and of the warps are added once per piece.
#include <cuda_bf16.h>

#include "cross_sched.cuh"
#include "kata_internal.cuh"
#include "sm100.cuh"

namespace kata {
namespace {

using namespace kata::sm100;

constexpr int kFWarps = 8;

struct FArgs {
    XSched sched;
    long long BH;
    const void *q, *k, *v;
    void *out;
    float *y, *den, *part, *part_l;
    XPiece *pieces;
};

// 8 consecutive elements as 4 fp32 pairs.
struct Raw8 {
    uint4 a, b;  // b: fp32 only
};
__device__ __forceinline__ Raw8 load8(const __nv_bfloat16 *p) { return {__ldg(reinterpret_cast<const uint4 *>(p)), {}}; }
__device__ __forceinline__ Raw8 load8(const float *p) {
    return {__ldg(reinterpret_cast<const uint4 *>(p)), __ldg(reinterpret_cast<const uint4 *>(p) + 1)};
}
template <typename T>
__device__ __forceinline__ void pairs(const Raw8 &r, uint64_t (&x)[4]) {
    if (sizeof(T) == 2) {
        x[0] = f32x2_pack(r.a.x << 16, r.a.x & 0xFFFF0000u);
        x[1] = f32x2_pack(r.a.y << 16, r.a.y & 0xFFFF0000u);
        x[2] = f32x2_pack(r.a.z << 16, r.a.z & 0xFFFF0000u);
        x[3] = f32x2_pack(r.a.w << 16, r.a.w & 0xFFFF0000u);
    } else {
        x[0] = f32x2_pack(r.a.x, r.a.y);
        x[1] = f32x2_pack(r.a.z, r.a.w);
        x[2] = f32x2_pack(r.b.x, r.b.y);
        x[3] = f32x2_pack(r.b.z, r.b.w);
    }
}

// RB: rows computed (the rows rounded up to 1, 2, 4).
template <typename T, int D, int RB>
__global__ void __launch_bounds__(32 * kFWarps, few_per_sm(RB))
cross_few_kernel(const FArgs a) {
    constexpr int L = D / 8, KW = 32 / L;           // lanes of a key, keys of a warp
    constexpr int N = kXCols / (kFWarps * KW);      // key groups of a warp per block
    constexpr int U = N < 4 ? N : 4;                // of them in flight
    __shared__ XRange range;
    __shared__ float red[kFWarps][RB][D], red_l[kFWarps][RB];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, key = lane / L, c = 8 * (lane % L);
    if (warp == 0) {
        const XRange r = x_range<kCrossFwd>(a.sched, blockIdx.x, lane);
        if (lane == 0) range = r;
    }
    __syncthreads();
    const int rows = a.sched.rows;
    if (threadIdx.x == 0 && !a.sched.whole) a.pieces[blockIdx.x] = XIter<kCrossFwd>::first(a.sched, range);
    // sequences without a visible key, which no unit covers
    if (a.sched.key_lengths)
        for (long long bh = blockIdx.x; bh < a.BH; bh += gridDim.x) {
            if (cross_length(a.sched.key_lengths, (int)(bh / a.sched.Hkv), a.sched.Tk) > 0) continue;
            for (int x = threadIdx.x; x < rows * D; x += 32 * kFWarps) {
                store_out(static_cast<T *>(a.out), bh * rows * D + x, 0.f);
                if (a.y) a.y[bh * rows * D + x] = 0.f;
                if (a.den && x < rows) a.den[bh * rows + x] = 0.f;
            }
        }
    XIter<kCrossFwd> iter(a.sched, range, blockIdx.x);
    XItem it;
    while (iter.next(it)) {
        const T *kp = static_cast<const T *>(a.k) + (long long)it.bh * a.sched.cols * D + c;
        const T *vp = static_cast<const T *>(a.v) + (long long)it.bh * a.sched.cols * D + c;
        uint64_t q[RB][4], o[RB][4];
        float l[RB];
#pragma unroll
        for (int r = 0; r < RB; ++r) {
            Raw8 x = {};
            if (r < rows) x = load8(static_cast<const T *>(a.q) + ((long long)it.bh * rows + r) * D + c);
            pairs<T>(x, q[r]);
            l[r] = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) o[r][e] = 0ull;
        }
        for (int b = 0; b < it.n_blk; ++b) {
            const int s0 = (it.b0 + b) * kXCols + warp * KW + key;
#pragma unroll
            for (int n0 = 0; n0 < N; n0 += U) {
                Raw8 kr[U], vr[U];
                bool on[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int s = s0 + (n0 + u) * kFWarps * KW;
                    on[u] = s < it.cols;
                    kr[u] = Raw8{};
                    vr[u] = Raw8{};  // nothing of a masked key is read
                    if (on[u]) {
                        kr[u] = load8(kp + (long long)s * D);
                        vr[u] = load8(vp + (long long)s * D);
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    uint64_t kx[4], vx[4];
                    pairs<T>(kr[u], kx);
                    pairs<T>(vr[u], vx);
                    float s[RB];
#pragma unroll
                    for (int r = 0; r < RB; ++r) {
                        const uint64_t t = f32x2_fma(
                            q[r][3], kx[3], f32x2_fma(q[r][2], kx[2], f32x2_fma(q[r][1], kx[1], f32x2_mul(q[r][0], kx[0]))));
                        s[r] = f32x2_lo(t) + f32x2_hi(t);
                    }
#pragma unroll
                    for (int x = L / 2; x > 0; x >>= 1)
#pragma unroll
                        for (int r = 0; r < RB; ++r) s[r] += __shfl_xor_sync(0xffffffffu, s[r], x);
#pragma unroll
                    for (int r = 0; r < RB; ++r) {
                        const float w = s[r] * s[r];
                        l[r] += w;
                        const uint64_t w2 = f32x2_pack(__float_as_uint(w), __float_as_uint(w));
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[r][e] = f32x2_fma(w2, vx[e], o[r][e]);
                    }
                }
            }
        }
        // the keys' lanes, then the warps
        float f[RB][8];
#pragma unroll
        for (int r = 0; r < RB; ++r) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                f[r][2 * e] = f32x2_lo(o[r][e]);
                f[r][2 * e + 1] = f32x2_hi(o[r][e]);
            }
#pragma unroll
            for (int x = L; x < 32; x <<= 1) {
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], x);
#pragma unroll
                for (int e = 0; e < 8; ++e) f[r][e] += __shfl_xor_sync(0xffffffffu, f[r][e], x);
            }
        }
        __syncthreads();  // the last piece's sums are read
        if (key == 0) {
#pragma unroll
            for (int r = 0; r < RB; ++r) {
                *reinterpret_cast<float4 *>(&red[warp][r][c]) = make_float4(f[r][0], f[r][1], f[r][2], f[r][3]);
                *reinterpret_cast<float4 *>(&red[warp][r][c + 4]) = make_float4(f[r][4], f[r][5], f[r][6], f[r][7]);
                if (lane == 0) red_l[warp][r] = l[r];
            }
        }
        __syncthreads();
        for (int x = threadIdx.x; x < rows * D; x += 32 * kFWarps) {
            const int r = x / D, e = x % D;
            float s = 0.f, den = 0.f;
#pragma unroll
            for (int w = 0; w < kFWarps; ++w) {
                s += red[w][r][e];
                den += red_l[w][r];
            }
            if (it.part >= 0) {
                const long long pr = x_part_row(a.sched, it.part) + r;
                a.part[pr * D + e] = s;
                if (e == 0) a.part_l[pr] = den;
            } else {
                const long long gr = (long long)it.bh * rows + r;
                s *= cross_recip(den);
                store_out(static_cast<T *>(a.out), gr * D + e, s);
                if (a.y) a.y[gr * D + e] = s;
                if (a.den && e == 0) a.den[gr] = den;
            }
        }
    }
}

template <typename T, int D, int RB>
cudaError_t launch_rb(const CrossPlan &p, const CrossIo &io, cudaStream_t st) {
    char *ws = static_cast<char *>(io.ws);
    FArgs a{};
    a.sched = p.sched[kCrossFwd];
    a.sched.key_lengths = io.key_lengths;
    a.sched.whole = cross_whole(p.sched[kCrossFwd], io);
    a.BH = p.BH;
    a.q = io.q;
    a.k = io.k;
    a.v = io.v;
    a.out = io.out;
    a.y = io.y;
    a.den = io.den;
    a.part = reinterpret_cast<float *>(ws + p.ws_part[kCrossFwd]);
    a.part_l = reinterpret_cast<float *>(ws + p.ws_part_l);
    a.pieces = reinterpret_cast<XPiece *>(ws + p.ws_pieces[kCrossFwd]);
    ProfScope prof("cross_few", st);
    cross_few_kernel<T, D, RB><<<a.sched.grid, 32 * kFWarps, 0, st>>>(a);
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_d(const CrossPlan &p, const CrossIo &io, cudaStream_t st) {
    if (p.R == 1) return launch_rb<T, D, 1>(p, io, st);
    if (p.R == 2) return launch_rb<T, D, 2>(p, io, st);
    return launch_rb<T, D, 4>(p, io, st);
}

template <typename T>
cudaError_t launch_t(const CrossPlan &p, const CrossIo &io, cudaStream_t st) {
    switch (p.d) {
        case 16: return launch_d<T, 16>(p, io, st);
        case 32: return launch_d<T, 32>(p, io, st);
        default: return launch_d<T, 64>(p, io, st);
    }
}

}  // namespace

cudaError_t launch_cross_few(const CrossPlan &p, const CrossIo &io, cudaStream_t st) {
    return p.dtype == KATA_BF16 ? launch_t<__nv_bfloat16>(p, io, st) : launch_t<float>(p, io, st);
}

}  // namespace kata
