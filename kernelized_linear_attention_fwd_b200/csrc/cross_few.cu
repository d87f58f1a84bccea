// Cross attention forward for few rows per key head (decode steps), on the register
// level: y = sum_s w v / sum_s w, w = (q.k)^2.  Up to 2 rows in bf16 and 4 in fp32 on
// the CUDA cores; 3 to 16 rows in bf16 by register-level tensor products (further down).
//
// Bound by reading the keys and values once.  64 sequences of 1501 keys and less, 16
// heads, one query (270 MB): 45 us, 6.0 TB/s, against 60 us on the tensor cores, whose
// one group of warps per item takes longer over 128 rows of scores than their
// block's loads; in fp32 (540 MB) 114 us, 4.7 TB/s, of 2 rows a key head on half as many
// 85, of 4 on a quarter 41.  Past 4 rows the registers of the rows' accumulators crowd out the
// loads in flight (8 rows, 2 key heads of 131072 keys: 63 us).
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

// This CTA's stretch of the work, its first piece noted, and its share of the sequences
// without a visible key, which no unit covers.
template <typename T, int D>
__device__ __forceinline__ void few_begin(const FArgs &a, XRange &range) {
    if (threadIdx.x < 32) {
        const XRange r = x_range<kCrossFwd>(a.sched, blockIdx.x, threadIdx.x);
        if (threadIdx.x == 0) range = r;
    }
    __syncthreads();
    const int rows = a.sched.rows;
    if (threadIdx.x == 0 && !a.sched.whole) a.pieces[blockIdx.x] = XIter<kCrossFwd>::first(a.sched, range);
    if (a.sched.key_lengths)
        for (long long bh = blockIdx.x; bh < a.BH; bh += gridDim.x) {
            if (cross_length(a.sched.key_lengths, (int)(bh / a.sched.Hkv), a.sched.Tk) > 0) continue;
            for (int x = threadIdx.x; x < rows * D; x += 32 * kFWarps) {
                store_out(static_cast<T *>(a.out), bh * rows * D + x, 0.f);
                if (a.y) a.y[bh * rows * D + x] = 0.f;
                if (a.den && x < rows) a.den[bh * rows + x] = 0.f;
            }
        }
}

// The warps' sums of an item or piece, added and written.
template <typename T, int D, int RB>
__device__ __forceinline__ void few_end(const FArgs &a, const XItem &it, const float (&red)[kFWarps][RB][D],
                                        const float (&red_l)[kFWarps][RB]) {
    const int rows = a.sched.rows;
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

// RB: rows computed (the rows rounded up to 1, 2, and in fp32 4).
template <typename T, int D, int RB>
__global__ void __launch_bounds__(32 * kFWarps, few_per_sm(RB))
cross_few_kernel(const FArgs a) {
    constexpr int L = D / 8, KW = 32 / L;           // lanes of a key, keys of a warp
    constexpr int N = kXCols / (kFWarps * KW);      // key groups of a warp per block
    constexpr int U = N < 4 ? N : 4;                // of them in flight
    __shared__ XRange range;
    __shared__ __align__(16) float red[kFWarps][RB][D];
    __shared__ float red_l[kFWarps][RB];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, key = lane / L, c = 8 * (lane % L);
    few_begin<T, D>(a, range);
    const int rows = a.sched.rows;
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
        few_end<T, D, RB>(a, it, red, red_l);
    }
}

// Three to 16 rows (decode steps with shared key heads), bf16: the products are
// register-level ones (m16n8k16), whose 16 rows are the rows, so that a key's operands go from
// memory to registers once and stay there.  A lane loads D / 4 coordinates of a key, in
// one run; the coordinates' order within a product is free, so these words are the score
// product's operand as they lie, and transposed 8 x 8 (movmatrix) the value product's.
// The weights go back as two bf16 numbers, high and low part; the denominator is the sum of
// both.  A warp has 16 keys of the next block in flight while it works on one.  2 key heads
// of 131072 keys, 8 rows (67 MB, which stay in L2): 12.1 us, and 6 for the join of 296 pieces; on the
// 128-row tiles 15.5 and 4.7 with the weights as precise.  One CTA of 16 warps per SM: 18 us.
// 4 rows on 64 x 4 key heads of 1500 keys (98 MB, in L2 too), with the join: 35 us on the CUDA
// cores, 24 so; 1 and 2 rows are 5% slower so.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// W words of a row.
template <int W>
__device__ __forceinline__ void load_words(uint32_t (&w)[W], const __nv_bfloat16 *p, bool on) {
    if constexpr (W == 2) {
        const uint2 v = on ? __ldg(reinterpret_cast<const uint2 *>(p)) : make_uint2(0u, 0u);
        w[0] = v.x;
        w[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {
            const uint4 v = on ? __ldg(reinterpret_cast<const uint4 *>(p) + i) : make_uint4(0u, 0u, 0u, 0u);
            w[4 * i] = v.x;
            w[4 * i + 1] = v.y;
            w[4 * i + 2] = v.z;
            w[4 * i + 3] = v.w;
        }
    }
}

template <int D>
__global__ void __launch_bounds__(32 * kFWarps, few_per_sm(16))
cross_rows_kernel(const FArgs a) {
    using T = __nv_bfloat16;
    constexpr int W = D / 8;  // words of a lane: D / 4 coordinates
    static_assert(kXCols == 16 * kFWarps, "a warp takes 16 keys of a block");
    __shared__ XRange range;
    __shared__ __align__(16) float red[kFWarps][16][D];
    __shared__ float red_l[kFWarps][16];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, c = (lane % 4) * (D / 4);
    few_begin<T, D>(a, range);
    const int rows = a.sched.rows;
    XIter<kCrossFwd> iter(a.sched, range, blockIdx.x);
    XItem it;
    while (iter.next(it)) {
        const T *kp = static_cast<const T *>(a.k) + (long long)it.bh * a.sched.cols * D + c;
        const T *vp = static_cast<const T *>(a.v) + (long long)it.bh * a.sched.cols * D + c;
        uint32_t q[2][W];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            load_words<W>(q[i], static_cast<const T *>(a.q) + ((long long)it.bh * rows + g + 8 * i) * D + c,
                          g + 8 * i < rows);
        float o[W][4], l[2] = {0.f, 0.f};  // rows g, g + 8: coordinates c + 2 j, c + 2 j + 1 of o[j]
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
        uint32_t k[2][W], v[2][W];  // keys g, g + 8 of the warp's 16
        auto load = [&](int b) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int s = (it.b0 + b) * kXCols + 16 * warp + 8 * i + g;
                const bool on = b < it.n_blk && s < it.cols;  // nothing of a masked key is read
                load_words<W>(k[i], kp + (long long)s * D, on);
                load_words<W>(v[i], vp + (long long)s * D, on);
            }
        };
        load(0);
        for (int b = 0; b < it.n_blk; ++b) {
            float s[2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int e = 0; e < 4; ++e) s[i][e] = 0.f;
#pragma unroll
                for (int x = 0; x < W; x += 2) mma(s[i], q[0][x], q[1][x], q[0][x + 1], q[1][x + 1], k[i][x], k[i][x + 1]);
            }
            uint32_t vt[2][W];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < W; ++j) vt[i][j] = transposed(v[i][j]);
            load(b + 1);
            uint32_t hi[4], lo[4];  // rows g, g + 8 of keys 0 .. 7, then of keys 8 .. 15
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x = s[i / 2][2 * (i & 1)], y = s[i / 2][2 * (i & 1) + 1], wx = x * x, wy = y * y;
                hi[i] = pack_bf16x2(wx, wy);
                const float hx = __uint_as_float(hi[i] << 16), hy = __uint_as_float(hi[i] & 0xFFFF0000u);
                lo[i] = pack_bf16x2(wx - hx, wy - hy);
                l[i & 1] += (hx + __uint_as_float(lo[i] << 16)) + (hy + __uint_as_float(lo[i] & 0xFFFF0000u));
            }
#pragma unroll
            for (int j = 0; j < W; ++j) {
                mma(o[j], lo[0], lo[1], lo[2], lo[3], vt[0][j], vt[1][j]);
                mma(o[j], hi[0], hi[1], hi[2], hi[3], vt[0][j], vt[1][j]);
            }
        }
        __syncthreads();  // the last piece's sums are read
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int j = 0; j < W; ++j)
                *reinterpret_cast<float2 *>(&red[warp][g + 8 * i][c + 2 * j]) = make_float2(o[j][2 * i], o[j][2 * i + 1]);
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
            if (lane % 4 == 0) red_l[warp][g + 8 * i] = l[i];
        }
        __syncthreads();
        few_end<T, D, 16>(a, it, red, red_l);
    }
}

template <typename T, int D, int RB>
cudaError_t launch_rb(const CrossPlan &p, const CrossIo &io, cudaStream_t st) {  // RB = 16: cross_rows_kernel
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
    if constexpr (RB == 16)
        cross_rows_kernel<D><<<a.sched.grid, 32 * kFWarps, 0, st>>>(a);
    else
        cross_few_kernel<T, D, RB><<<a.sched.grid, 32 * kFWarps, 0, st>>>(a);
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_d(const CrossPlan &p, const CrossIo &io, cudaStream_t st) {
    if (p.R == 1) return launch_rb<T, D, 1>(p, io, st);
    if (p.R == 2) return launch_rb<T, D, 2>(p, io, st);
    return launch_rb<T, D, sizeof(T) == 2 ? 16 : 4>(p, io, st);
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
