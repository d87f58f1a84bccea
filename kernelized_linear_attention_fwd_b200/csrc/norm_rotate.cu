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

namespace kata {
namespace {

constexpr int kNormWarps = 8;

template <typename T>
struct Vec4;
template <>
struct Vec4<float> {
    using V = float4;
};
template <>
struct Vec4<__nv_bfloat16> {
    using V = uint2;
};

__device__ __forceinline__ void unpack4(const float4 &v, float *x) {
    x[0] = v.x;
    x[1] = v.y;
    x[2] = v.z;
    x[3] = v.w;
}
__device__ __forceinline__ void unpack4(const uint2 &v, float *x) {
    x[0] = __uint_as_float(v.x << 16);
    x[1] = __uint_as_float(v.x & 0xFFFF0000u);
    x[2] = __uint_as_float(v.y << 16);
    x[3] = __uint_as_float(v.y & 0xFFFF0000u);
}
__device__ __forceinline__ void pack4(const float *x, float4 &v) { v = make_float4(x[0], x[1], x[2], x[3]); }
__device__ __forceinline__ void pack4(const float *x, uint2 &v) {
    __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
    v.x = *reinterpret_cast<uint32_t *>(&a);
    v.y = *reinterpret_cast<uint32_t *>(&b);
}

// The 8 elements of a lane as two vectors of 4 (half-split pairs: a_0..a_3 and
// b_0..b_3; neighbouring pairs: a_0 b_0 a_1 b_1 and a_2 b_2 a_3 b_3).
template <typename T>
struct Row8 {
    typename Vec4<T>::V v[2];
    __device__ __forceinline__ void load(const T *row, int o0, int o1) {
        v[0] = __ldg(reinterpret_cast<const typename Vec4<T>::V *>(row + o0));
        v[1] = __ldg(reinterpret_cast<const typename Vec4<T>::V *>(row + o1));
    }
    __device__ __forceinline__ void store(T *row, int o0, int o1) const {
        *reinterpret_cast<typename Vec4<T>::V *>(row + o0) = v[0];
        *reinterpret_cast<typename Vec4<T>::V *>(row + o1) = v[1];
    }
    __device__ __forceinline__ void get(float *x) const {
        unpack4(v[0], x);
        unpack4(v[1], x + 4);
    }
    __device__ __forceinline__ void set(const float *x) {
        pack4(x, v[0]);
        pack4(x + 4, v[1]);
    }
};

// Positions in x[8] of the pair j's members.
template <bool INTER>
__device__ __forceinline__ constexpr int pa(int j) {
    return INTER ? 2 * j : j;
}
template <bool INTER>
__device__ __forceinline__ constexpr int pb(int j) {
    return INTER ? 2 * j + 1 : j + 4;
}

// The lane's offsets in a row and its four angles.
template <int D, bool INTER>
struct Lane {
    int o0, o1;
    float c[4], s[4];

    __device__ __forceinline__ explicit Lane(int lane, int n_rot) {
        const int p0 = 4 * (lane % (D / 8));
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

    // Angle of pair `lane` for this token, shared through `buf` (one per warp).
    // position * inv_freq is taken in 64 bits, reduced to a fraction of a turn
    // there (at position 2^31 that still leaves 2^-22 of a turn), and only the
    // fraction's sine and cosine are 32-bit.
    __device__ __forceinline__ void angles(float2 *buf, int lane, long long pos, double turn_freq, int n_rot) {
        __syncwarp();
        if (lane < n_rot) {
            const double turns = (double)pos * turn_freq;
            float2 cs;
            sincospif((float)(2.0 * (turns - rint(turns))), &cs.y, &cs.x);
            buf[lane] = cs;
        }
        __syncwarp();
        const int p0 = 4 * (lane % (D / 8));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool on = p0 + j < n_rot;
            const float2 cs = on ? buf[p0 + j] : make_float2(1.f, 0.f);
            c[j] = cs.x;
            s[j] = cs.y;
        }
    }
};

// Sum over the lanes of one row.
template <int D>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = D / 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

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

// U row groups in flight per warp: at U = 4 a lane has 4 (forward) loads of 16
// bytes outstanding, about 128 KB per SM at 64 warps.
template <typename T, int D, bool INTER, bool BWD>
__global__ void __launch_bounds__(32 * kNormWarps, BWD ? 3 : 4)
norm_rotate_kernel(const NormArgs<T> a) {
    constexpr int kLanes = D / 8, kRows = 32 / kLanes, U = BWD ? 2 : 4;
    __shared__ float2 cs_buf[kNormWarps][32];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, sub = lane / kLanes;
    Lane<D, INTER> L(lane, a.n_rot);
    const double turn_freq = lane < a.n_rot ? (double)a.inv_freq[lane] * 0.15915494309189533577 : 0.0;
    __shared__ float w_buf[2][D];
    for (int x = threadIdx.x; x < 2 * D; x += 32 * kNormWarps) {
        const float *src = x < D ? a.w[0] : a.w[1];
        (&w_buf[0][0])[x] = src ? src[x % D] : 1.f;
    }
    __syncthreads();
    float dw[2][8] = {};

    const long long n_warps = (long long)gridDim.x * kNormWarps;
    for (long long tok = (long long)blockIdx.x * kNormWarps + warp; tok < a.tokens; tok += n_warps) {
        const long long b = tok / a.T_, t = tok - b * a.T_;
        if (a.n_rot > 0)
            L.angles(cs_buf[warp], lane, a.pos ? a.pos[b * a.pos_stride + t] : t, turn_freq, a.n_rot);
        else
            L.angles(cs_buf[warp], lane, 0, 0.0, 0);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const int H = a.H[m];
            float w[8];
            *reinterpret_cast<float4 *>(w) = *reinterpret_cast<const float4 *>(&w_buf[m][L.o0]);
            *reinterpret_cast<float4 *>(w + 4) = *reinterpret_cast<const float4 *>(&w_buf[m][L.o1]);
            const T *xt = a.x[m] + b * a.sb[m] + t * a.st[m];
            const long long yt = (b * H * a.T_ + t) * D;  // head h adds h T D
            for (int h0 = blockIdx.y * (U * kRows); h0 < H; h0 += gridDim.y * (U * kRows)) {
                Row8<T> rx[U], rg[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int h = h0 + u * kRows + sub;
                    if (h < H) {
                        rx[u].load(xt + h * a.sh[m], L.o0, L.o1);
                        if (BWD) rg[u].load(a.gy[m] + yt + (long long)h * a.T_ * D, L.o0, L.o1);
                    } else {
                        const float zero[8] = {};
                        rx[u].set(zero);
                        if (BWD) rg[u].set(zero);
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int h = h0 + u * kRows + sub;
                    float x[8], o[8];
                    rx[u].get(x);
                    float ss = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
                    const float r = rsqrtf(fmaf(row_sum<D>(ss), 1.f / D, a.eps));
                    if (!BWD) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) x[e] *= w[e];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float za = x[pa<INTER>(j)], zb = x[pb<INTER>(j)];
                            o[pa<INTER>(j)] = r * fmaf(za, L.c[j], -zb * L.s[j]);
                            o[pb<INTER>(j)] = r * fmaf(za, L.s[j], zb * L.c[j]);
                        }
                        rx[u].set(o);
                        if (h < H) rx[u].store(a.y[m] + yt + (long long)h * a.T_ * D, L.o0, L.o1);
                    } else {
                        float g[8];
                        rg[u].get(g);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {  // the gradient turned back
                            const float ya = g[pa<INTER>(j)], yb = g[pb<INTER>(j)];
                            g[pa<INTER>(j)] = fmaf(ya, L.c[j], yb * L.s[j]);
                            g[pb<INTER>(j)] = fmaf(yb, L.c[j], -ya * L.s[j]);
                        }
                        float dot = 0.f;
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            x[e] *= r;  // u
                            dw[m][e] = fmaf(g[e], x[e], dw[m][e]);
                            g[e] *= w[e];
                            dot = fmaf(g[e], x[e], dot);
                        }
                        const float mean = row_sum<D>(dot) * (1.f / D);
#pragma unroll
                        for (int e = 0; e < 8; ++e) o[e] = r * fmaf(-mean, x[e], g[e]);
                        rx[u].set(o);
                        if (h < H)
                            rx[u].store(a.dx[m] + b * a.db[m] + t * a.dt[m] + h * a.dh[m], L.o0, L.o1);
                    }
                }
            }
        }
    }
    if (BWD) {
        // the block's sum of dw: lanes of one column, then warps, always in this order
        __shared__ float red[kNormWarps][2][D];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float v = dw[m][e];
#pragma unroll
                for (int o = kLanes; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
                if (sub == 0) red[warp][m][(e < 4 ? L.o0 : L.o1) + (e & 3)] = v;
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

// Blocks of the launch: as many as hold the tokens, at most 4 per SM (32 warps);
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
    const long long full = 4LL * kPlanSms;
    const int gx = (int)(blocks < full ? blocks : full);
    // row groups a warp could leave to others
    const int rows = (p.backward ? 2 : 4) * (256 / p.d);
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
