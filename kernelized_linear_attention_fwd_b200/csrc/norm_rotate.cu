// Per-head RMS norm of queries and keys with the rotation by position, and its
// gradient (entry points kata_qk_norm_rotate, kata_qk_norm_rotate_backward).
//
// One row is a head's d coordinates x at one token:
//
//     r = 1 / sqrt(mean_i x_i^2 + eps),  u = r x,  z = w . u,
//     (y_a, y_b) = (z_a cos t - z_b sin t, z_a sin t + z_b cos t)
//
// for each of the n_rot pairs (a, b), t = position * inv_freq[pair]; the other
// coordinates pass.  With g the gradient turned back by the same angles,
//
//     dw = sum over rows of g . u,    dx = r (w . g - u mean_i(w_i g_i u_i)).
//
// The data is read token-major with strides, as a projection leaves it, and the
// outputs are written head-major, as the attention calls read it, so no copy
// sits between the two.
//
// Layout.  A row is d / 8 lanes of 8 elements each: 4 pairs (a_j, b_j), so that a
// rotation needs no exchange between lanes.  Pairs of neighbours (2p, 2p + 1)
// make the lane's 8 elements contiguous; pairs (p, p + n) make them two runs of
// 4, from each half.  A warp takes one token and walks its heads, 32 / (d / 8)
// of them at a time.  The angles depend on the token only: lane p computes
// the one of pair p (at most 32), and the warp shares them through shared
// memory.  When there are fewer tokens than the GPU holds warps, the heads of
// a token are spread over several warps (grid.y).
#include <cuda_bf16.h>

#include "kata_internal.cuh"
#include "sm100.cuh"

namespace kata {
namespace {

using namespace kata::sm100;

constexpr int kNormWarps = 8;

// A lane's 4 pairs (a_j, b_j) of a row as packed fp32: a = (a_0 a_1), (a_2 a_3), b
// likewise, whichever way the pairs lie in memory; all arithmetic is on these.
struct Pairs {
    uint64_t a[2], b[2];
};

__device__ __forceinline__ uint32_t lo16(uint32_t w) { return w << 16; }
__device__ __forceinline__ uint32_t hi16(uint32_t w) { return w & 0xFFFF0000u; }
__device__ __forceinline__ uint64_t both(float x) { return f32x2_pack(__float_as_uint(x), __float_as_uint(x)); }

// The 8 elements of a lane in memory: two vectors of 4 at offsets o0 and o1
// (half-split pairs: a_0 .. a_3 and b_0 .. b_3; neighbouring pairs: a_0 b_0 a_1 b_1
// and a_2 b_2 a_3 b_3).
template <typename T, bool INTER>
struct Row8;
template <bool INTER>
struct Row8<__nv_bfloat16, INTER> {
    uint2 v[2];
    __device__ __forceinline__ void load(const __nv_bfloat16 *row, int o0, int o1) {
        v[0] = __ldg(reinterpret_cast<const uint2 *>(row + o0));
        v[1] = __ldg(reinterpret_cast<const uint2 *>(row + o1));
    }
    __device__ __forceinline__ void zero() { v[0] = v[1] = make_uint2(0u, 0u); }
    __device__ __forceinline__ Pairs get() const {
        Pairs p;
        if (INTER) {
            p.a[0] = f32x2_pack(lo16(v[0].x), lo16(v[0].y));
            p.b[0] = f32x2_pack(hi16(v[0].x), hi16(v[0].y));
            p.a[1] = f32x2_pack(lo16(v[1].x), lo16(v[1].y));
            p.b[1] = f32x2_pack(hi16(v[1].x), hi16(v[1].y));
        } else {
            p.a[0] = f32x2_pack(lo16(v[0].x), hi16(v[0].x));
            p.a[1] = f32x2_pack(lo16(v[0].y), hi16(v[0].y));
            p.b[0] = f32x2_pack(lo16(v[1].x), hi16(v[1].x));
            p.b[1] = f32x2_pack(lo16(v[1].y), hi16(v[1].y));
        }
        return p;
    }
    __device__ __forceinline__ static void store(__nv_bfloat16 *row, int o0, int o1, const Pairs &p) {
        uint2 w[2];
        if (INTER) {
            w[0] = make_uint2(pack_bf16x2(f32x2_lo(p.a[0]), f32x2_lo(p.b[0])),
                              pack_bf16x2(f32x2_hi(p.a[0]), f32x2_hi(p.b[0])));
            w[1] = make_uint2(pack_bf16x2(f32x2_lo(p.a[1]), f32x2_lo(p.b[1])),
                              pack_bf16x2(f32x2_hi(p.a[1]), f32x2_hi(p.b[1])));
        } else {
            w[0] = make_uint2(f32x2_to_bf16x2(p.a[0]), f32x2_to_bf16x2(p.a[1]));
            w[1] = make_uint2(f32x2_to_bf16x2(p.b[0]), f32x2_to_bf16x2(p.b[1]));
        }
        *reinterpret_cast<uint2 *>(row + o0) = w[0];
        *reinterpret_cast<uint2 *>(row + o1) = w[1];
    }
};
template <bool INTER>
struct Row8<float, INTER> {
    uint4 v[2];
    __device__ __forceinline__ void load(const float *row, int o0, int o1) {
        v[0] = __ldg(reinterpret_cast<const uint4 *>(row + o0));
        v[1] = __ldg(reinterpret_cast<const uint4 *>(row + o1));
    }
    __device__ __forceinline__ void zero() { v[0] = v[1] = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ Pairs get() const {
        Pairs p;
        if (INTER) {
            p.a[0] = f32x2_pack(v[0].x, v[0].z);
            p.b[0] = f32x2_pack(v[0].y, v[0].w);
            p.a[1] = f32x2_pack(v[1].x, v[1].z);
            p.b[1] = f32x2_pack(v[1].y, v[1].w);
        } else {
            p.a[0] = f32x2_pack(v[0].x, v[0].y);
            p.a[1] = f32x2_pack(v[0].z, v[0].w);
            p.b[0] = f32x2_pack(v[1].x, v[1].y);
            p.b[1] = f32x2_pack(v[1].z, v[1].w);
        }
        return p;
    }
    __device__ __forceinline__ static void store(float *row, int o0, int o1, const Pairs &p) {
        const float a0 = f32x2_lo(p.a[0]), a1 = f32x2_hi(p.a[0]), a2 = f32x2_lo(p.a[1]), a3 = f32x2_hi(p.a[1]);
        const float b0 = f32x2_lo(p.b[0]), b1 = f32x2_hi(p.b[0]), b2 = f32x2_lo(p.b[1]), b3 = f32x2_hi(p.b[1]);
        *reinterpret_cast<float4 *>(row + o0) = INTER ? make_float4(a0, b0, a1, b1) : make_float4(a0, a1, a2, a3);
        *reinterpret_cast<float4 *>(row + o1) = INTER ? make_float4(a2, b2, a3, b3) : make_float4(b0, b1, b2, b3);
    }
};

// A lane's offsets in a row.
template <int D, bool INTER>
struct Lane {
    int p0, o0, o1;  // first pair; the two runs of 4 elements

    __device__ __forceinline__ explicit Lane(int lane, int n_rot) {
        p0 = 4 * (lane % (D / 8));
        if (INTER) {
            o0 = 2 * p0;
            o1 = o0 + 4;
        } else if (p0 < n_rot) {
            o0 = p0;
            o1 = p0 + n_rot;
        } else {  // coordinates that pass: any cover of [2 n_rot, D) by runs of 4
            o0 = p0 + n_rot;
            o1 = p0 + D / 2;
        }
    }
    // element e of the row's run order (a_0 .. a_3, b_0 .. b_3) in memory
    __device__ __forceinline__ int at(int e) const {
        const int j = e & 3;
        if (INTER) return 2 * (p0 + j) + e / 4;
        return (e < 4 ? o0 : o1) + j;
    }
};

// Cosine and sine of the angles of one token's pairs, shared by the warp through
// `buf`: pair `lane` is worked out here.  position * inv_freq is taken in 64 bits,
// reduced to a fraction of a turn there (at position 2^31 that still leaves 2^-22
// of a turn), and only the fraction's sine and cosine are 32-bit.
__device__ __forceinline__ void share_angles(float2 *buf, int lane, long long pos, double turn_freq, int n_rot) {
    __syncwarp();
    float2 cs = make_float2(1.f, 0.f);  // pairs that do not turn
    if (lane < n_rot) {
        const double turns = (double)pos * turn_freq;
        sincospif((float)(2.0 * (turns - rint(turns))), &cs.y, &cs.x);
    }
    buf[lane] = cs;
    __syncwarp();
}

// Sum over the lanes of one row.
template <int D>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = D / 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Dot product of a lane's 8 elements.
__device__ __forceinline__ float dot8(const Pairs &x, const Pairs &y) {
    const uint64_t t = f32x2_fma(
        x.b[1], y.b[1], f32x2_fma(x.b[0], y.b[0], f32x2_fma(x.a[1], y.a[1], f32x2_mul(x.a[0], y.a[0]))));
    return f32x2_lo(t) + f32x2_hi(t);
}

// Row groups that a warp loads at a time: 2 KB, of the input or of input and gradient.
__host__ __device__ constexpr int norm_groups(bool backward, int size) { return (backward ? 4 : 8) / size; }
// Blocks per SM (64 and 80 registers a thread).
__host__ __device__ constexpr int norm_per_sm(bool backward) { return backward ? 2 : 3; }

template <typename T>
struct NormArgs {
    const T *x[2];       // queries, keys: element (b, t, h, 0) at b sb + t st + h sh
    long long sb[2], st[2], sh[2];
    T *y[2];             // [B, H, T, D]
    const float *w[2];   // [D] or null (ones)
    int H[2];
    // backward
    const T *gy[2];      // [B, H, T, D]
    T *dx[2];            // strided
    long long db[2], dt[2], dh[2];
    float *partial;      // [gridDim.x * gridDim.y][2][D]
    const float *inv_freq;
    const long long *pos;  // position of (b, t) at pos[b * pos_stride + t]; null: t
    long long pos_stride;
    int T_, n_rot;
    long long tokens;  // B T
    float eps;
};

// A warp loads up to U row groups at a time; what is left of a token's heads goes
// group by group.  The arithmetic is packed (fp32 pairs) and the forward's gains are
// folded into the angles once per token and tensor: 139 us without either for 65536
// tokens of 16 + 16 heads of 64 (537 MB), 95 us so, 5.7 TB/s.  The gradient (32768
// tokens of 16 + 4 heads, 252 MB) takes 70 us, 3.6 TB/s: half of its warps' time is
// waiting for loads, and neither more warps of fewer registers, nor more rows at a
// time, nor loading a set of rows ahead across tokens changed it (70 to 76 us).
template <typename T, int D, bool INTER, bool BWD>
__global__ void __launch_bounds__(32 * kNormWarps, norm_per_sm(BWD))
norm_rotate_kernel(const NormArgs<T> a) {
    constexpr int kLanes = D / 8, kRows = 32 / kLanes, U = norm_groups(BWD, sizeof(T));
    using Row = Row8<T, INTER>;
    __shared__ float2 cs_buf[kNormWarps][32];
    __shared__ float w_buf[2][D];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, sub = lane / kLanes;
    const Lane<D, INTER> L(lane, a.n_rot);
    const double turn_freq = lane < a.n_rot ? (double)a.inv_freq[lane] * 0.15915494309189533577 : 0.0;
    for (int x = threadIdx.x; x < 2 * D; x += 32 * kNormWarps) {
        const float *src = x < D ? a.w[0] : a.w[1];
        (&w_buf[0][0])[x] = src ? src[x % D] : 1.f;
    }
    __syncthreads();
    Pairs dw[2] = {};

    // this warp's tokens, every n_warps-th, as (b, t)
    const int n_warps = gridDim.x * kNormWarps, tok0 = blockIdx.x * kNormWarps + warp;
    const int step_b = n_warps / a.T_, step_t = n_warps - step_b * a.T_;
    int b = tok0 / a.T_, t = tok0 - b * a.T_;
    int left = tok0 < a.tokens ? (int)((a.tokens - tok0 + n_warps - 1) / n_warps) : 0;
    auto position = [&](int bb, int tt) { return a.pos ? a.pos[bb * a.pos_stride + tt] : (long long)tt; };
    long long pos = left > 0 ? position(b, t) : 0;
    for (; left > 0; --left) {
        share_angles(cs_buf[warp], lane, pos, turn_freq, a.n_rot);
        // the next token's place and position, a token ahead
        int nb = b + step_b, nt = t + step_t;
        if (nt >= a.T_) {
            nt -= a.T_;
            ++nb;
        }
        if (left > 1) pos = position(nb, nt);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const int H = a.H[m];
            if (H == 0) continue;
            Pairs w, c, s;  // c in a: cosine; s in a: sine, in b: -sine
            {
                const float4 u = *reinterpret_cast<const float4 *>(&cs_buf[warp][L.p0]);
                const float4 v = *reinterpret_cast<const float4 *>(&cs_buf[warp][L.p0 + 2]);
                c.a[0] = f32x2_pack(__float_as_uint(u.x), __float_as_uint(u.z));
                c.a[1] = f32x2_pack(__float_as_uint(v.x), __float_as_uint(v.z));
                s.a[0] = f32x2_pack(__float_as_uint(u.y), __float_as_uint(u.w));
                s.a[1] = f32x2_pack(__float_as_uint(v.y), __float_as_uint(v.w));
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    s.b[i] = s.a[i] ^ 0x8000000080000000ull;
                    w.a[i] = f32x2_pack(__float_as_uint(w_buf[m][L.at(2 * i)]),
                                        __float_as_uint(w_buf[m][L.at(2 * i + 1)]));
                    w.b[i] = f32x2_pack(__float_as_uint(w_buf[m][L.at(4 + 2 * i)]),
                                        __float_as_uint(w_buf[m][L.at(5 + 2 * i)]));
                }
            }
            Pairs ca, cb;  // forward: y_a = x_a ca.a + x_b cb.a, y_b = x_a ca.b + x_b cb.b
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                ca.a[i] = f32x2_mul(c.a[i], w.a[i]);
                cb.a[i] = f32x2_mul(s.b[i], w.b[i]);
                ca.b[i] = f32x2_mul(s.a[i], w.a[i]);
                cb.b[i] = f32x2_mul(c.a[i], w.b[i]);
            }
            const int h0 = blockIdx.y * (U * kRows) + sub, stride = gridDim.y * (U * kRows);
            const long long sh = a.sh[m] * kRows, yh = (long long)a.T_ * D * kRows;
            const T *px = a.x[m] + b * a.sb[m] + t * a.st[m] + h0 * a.sh[m];
            const long long y0 = (((long long)b * H + h0) * a.T_ + t) * D;

            auto work = [&](const Row &rx, const Row &rg, T *dst, bool on) {
                Pairs x = rx.get(), o;
                const float r = rsqrtf(fmaf(row_sum<D>(dot8(x, x)), 1.f / D, a.eps));
                const uint64_t r2 = both(r);
                if (!BWD) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        o.a[i] = f32x2_mul(f32x2_fma(x.a[i], ca.a[i], f32x2_mul(x.b[i], cb.a[i])), r2);
                        o.b[i] = f32x2_mul(f32x2_fma(x.a[i], ca.b[i], f32x2_mul(x.b[i], cb.b[i])), r2);
                    }
                } else {
                    const Pairs y = rg.get();
                    Pairs g;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        // the gradient turned back
                        g.a[i] = f32x2_fma(y.a[i], c.a[i], f32x2_mul(y.b[i], s.a[i]));
                        g.b[i] = f32x2_fma(y.b[i], c.a[i], f32x2_mul(y.a[i], s.b[i]));
                        x.a[i] = f32x2_mul(x.a[i], r2);  // u
                        x.b[i] = f32x2_mul(x.b[i], r2);
                        dw[m].a[i] = f32x2_fma(g.a[i], x.a[i], dw[m].a[i]);
                        dw[m].b[i] = f32x2_fma(g.b[i], x.b[i], dw[m].b[i]);
                        g.a[i] = f32x2_mul(g.a[i], w.a[i]);
                        g.b[i] = f32x2_mul(g.b[i], w.b[i]);
                    }
                    const uint64_t nm2 = both(row_sum<D>(dot8(g, x)) * (-1.f / D));
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        o.a[i] = f32x2_mul(f32x2_fma(nm2, x.a[i], g.a[i]), r2);
                        o.b[i] = f32x2_mul(f32x2_fma(nm2, x.b[i], g.b[i]), r2);
                    }
                }
                if (on) Row::store(dst, L.o0, L.o1, o);
            };

            T *po = BWD ? a.dx[m] + b * a.db[m] + t * a.dt[m] + h0 * a.dh[m] : a.y[m] + y0;
            const long long oh = BWD ? a.dh[m] * kRows : yh;
            const T *pg = BWD ? a.gy[m] + y0 : nullptr;
            int h = h0;
            for (; h - sub + U * kRows <= H; h += stride) {
                Row rx[U], rg[BWD ? U : 1];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    rx[u].load(px + u * sh, L.o0, L.o1);
                    if (BWD) rg[u].load(pg + u * yh, L.o0, L.o1);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) work(rx[u], rg[BWD ? u : 0], po + u * oh, true);
                px += gridDim.y * (U * sh);
                po += gridDim.y * (U * oh);
                if (BWD) pg += gridDim.y * (U * yh);
            }
            // the set of groups that reaches past the last head, if it is this block's
            for (int u = 0; u < U && h - sub < H; ++u, h += kRows) {
                Row rx, rg;
                const bool on = h < H;
                rx.zero();
                rg.zero();
                if (on) {
                    rx.load(px, L.o0, L.o1);
                    if (BWD) rg.load(pg, L.o0, L.o1);
                }
                work(rx, rg, po, on);
                px += sh;
                po += oh;
                if (BWD) pg += yh;
            }
        }
        b = nb;
        t = nt;
    }
    if (BWD) {
        // the block's sum of dw: lanes of one column, then warps, always in this order
        __shared__ float red[kNormWarps][2][D];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint64_t q = e < 4 ? dw[m].a[(e & 3) / 2] : dw[m].b[(e & 3) / 2];
                float v = e & 1 ? f32x2_hi(q) : f32x2_lo(q);
#pragma unroll
                for (int o = kLanes; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
                if (sub == 0) red[warp][m][L.at(e)] = v;
            }
        __syncthreads();
        if (threadIdx.x < 2 * D) {
            float v = 0.f;
#pragma unroll
            for (int x = 0; x < kNormWarps; ++x) v += (&red[x][0][0])[threadIdx.x];
            a.partial[((long long)blockIdx.y * gridDim.x + blockIdx.x) * (2 * D) + threadIdx.x] = v;
        }
    }
}

// dw = sum of the blocks' partial sums, in a fixed order: a CTA per 16 columns,
// thread (g, c) adds the blocks g, g + 64, ... of column c, then one warp per column
// adds the 64 groups.
template <int D>
__global__ void __launch_bounds__(1024)
norm_dw_kernel(const float *partial, int n, float *dwq, float *dwk) {
    constexpr int C = 16, G = 1024 / C;  // columns and groups of a CTA
    __shared__ float red[G][C + 1];
    const int c = threadIdx.x % C, g = threadIdx.x / C, col = blockIdx.x * C + c;
    float v = 0.f;
#pragma unroll 10
    for (int i = g; i < n; i += G) v += partial[(long long)i * (2 * D) + col];
    red[g][c] = v;
    __syncthreads();
    if (threadIdx.x < 32 * C) {  // warp x: the groups of column x, always in this order
        const int x = threadIdx.x / 32, l = threadIdx.x % 32;
        v = red[l][x] + red[l + 32][x];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        const int k = blockIdx.x * C + x;
        float *dst = k < D ? dwq : dwk;
        if (l == 0 && dst) dst[k % D] = v;
    }
}

// Blocks of the launch: as many as hold the tokens, at most what the SMs hold at a time;
// if the tokens fill less than that, the heads are spread over grid.y.
template <typename T, int D, bool INTER, bool BWD>
cudaError_t launch_one(const NormRotate &p, cudaStream_t st) {
    NormArgs<T> a;
    for (int m = 0; m < 2; ++m) {
        a.x[m] = static_cast<const T *>(p.x[m]);
        a.y[m] = static_cast<T *>(p.y[m]);
        a.w[m] = p.w[m];
        a.H[m] = p.H[m];
        a.sb[m] = p.xs[m][0];
        a.st[m] = p.xs[m][1];
        a.sh[m] = p.xs[m][2];
        a.gy[m] = static_cast<const T *>(p.gy[m]);
        a.dx[m] = static_cast<T *>(p.dx[m]);
        a.db[m] = p.ds[m][0];
        a.dt[m] = p.ds[m][1];
        a.dh[m] = p.ds[m][2];
    }
    a.partial = static_cast<float *>(p.ws);
    a.inv_freq = p.inv_freq;
    a.pos = p.positions;
    a.pos_stride = p.pos_stride;
    a.T_ = p.T;
    a.n_rot = p.n_rot;
    a.tokens = (long long)p.B * p.T;
    a.eps = p.eps;
    const dim3 grid = norm_rotate_grid(p);
    {
        ProfScope prof(BWD ? "norm_rotate_bwd" : "norm_rotate", st);
        norm_rotate_kernel<T, D, INTER, BWD><<<grid, 32 * kNormWarps, 0, st>>>(a);
    }
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !BWD || (!p.dw[0] && !p.dw[1])) return e;
    ProfScope prof("norm_dw", st);
    norm_dw_kernel<D><<<2 * D / 16, 1024, 0, st>>>(a.partial, (int)(grid.x * grid.y), p.dw[0], p.dw[1]);
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_d(const NormRotate &p, cudaStream_t st) {
    if (p.backward)
        return p.interleaved ? launch_one<T, D, true, true>(p, st) : launch_one<T, D, false, true>(p, st);
    return p.interleaved ? launch_one<T, D, true, false>(p, st) : launch_one<T, D, false, false>(p, st);
}

template <typename T>
cudaError_t launch_t(const NormRotate &p, cudaStream_t st) {
    switch (p.d) {
        case 16: return launch_d<T, 16>(p, st);
        case 32: return launch_d<T, 32>(p, st);
        default: return launch_d<T, 64>(p, st);
    }
}

}  // namespace

dim3 norm_rotate_grid(const NormRotate &p) {
    const long long tokens = (long long)p.B * p.T;
    const long long blocks = (tokens + kNormWarps - 1) / kNormWarps;
    const long long full = (long long)norm_per_sm(p.backward) * kPlanSms;
    const int gx = (int)(blocks < full ? blocks : full);
    // row groups a warp could leave to others
    const int rows = norm_groups(p.backward, p.dtype == KATA_BF16 ? 2 : 4) * (256 / p.d);
    const int hm = p.H[0] > p.H[1] ? p.H[0] : p.H[1];
    const int groups = (hm + rows - 1) / rows;
    int gy = (int)(full / gx);
    if (gy > groups) gy = groups;
    if (gy < 1) gy = 1;
    return dim3(gx, gy);
}

cudaError_t launch_norm_rotate(const NormRotate &p, cudaStream_t st) {
    return p.dtype == KATA_BF16 ? launch_t<__nv_bfloat16>(p, st) : launch_t<float>(p, st);
}

}  // namespace kata
