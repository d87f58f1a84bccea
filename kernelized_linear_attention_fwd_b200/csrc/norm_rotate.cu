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
    __device__ __forceinline__ void load_shared(uint32_t at0, uint32_t at1) {
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v[0].x), "=r"(v[0].y) : "r"(at0));
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v[1].x), "=r"(v[1].y) : "r"(at1));
    }
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
    __device__ __forceinline__ void load_shared(uint32_t at0, uint32_t at1) {
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v[0].x), "=r"(v[0].y), "=r"(v[0].z), "=r"(v[0].w) : "r"(at0));
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v[1].x), "=r"(v[1].y), "=r"(v[1].z), "=r"(v[1].w) : "r"(at1));
    }
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

// A lane's gains of one tensor, in the row's run order.
template <int D, bool INTER>
__device__ __forceinline__ Pairs gains(const float *w, const Lane<D, INTER> &L) {
    Pairs p;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        p.a[i] = f32x2_pack(__float_as_uint(w[L.at(2 * i)]), __float_as_uint(w[L.at(2 * i + 1)]));
        p.b[i] = f32x2_pack(__float_as_uint(w[L.at(4 + 2 * i)]), __float_as_uint(w[L.at(5 + 2 * i)]));
    }
    return p;
}

// The turn of a lane's pairs: cosine (c), sine (s) and its negative (n).
struct Turn {
    uint64_t c[2], s[2], n[2];
};
__device__ __forceinline__ Turn turn_of(const float2 (&cs)[4]) {
    Turn t;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        t.c[i] = f32x2_pack(__float_as_uint(cs[2 * i].x), __float_as_uint(cs[2 * i + 1].x));
        t.s[i] = f32x2_pack(__float_as_uint(cs[2 * i].y), __float_as_uint(cs[2 * i + 1].y));
        t.n[i] = t.s[i] ^ 0x8000000080000000ull;
    }
    return t;
}

// One row's share of a lane.  Forward: x normed, times the gains and turned, m the
// turn with the gains folded in: out_a = x_a m.a + x_b m.b, out_b = x_a k.a + x_b k.b.
template <int D>
__device__ __forceinline__ Pairs row_forward(const Pairs &x, const Pairs &m, const Pairs &k, float eps) {
    const uint64_t r2 = both(rsqrtf(fmaf(row_sum<D>(dot8(x, x)), 1.f / D, eps)));
    Pairs o;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        o.a[i] = f32x2_mul(f32x2_fma(x.a[i], m.a[i], f32x2_mul(x.b[i], m.b[i])), r2);
        o.b[i] = f32x2_mul(f32x2_fma(x.a[i], k.a[i], f32x2_mul(x.b[i], k.b[i])), r2);
    }
    return o;
}
__device__ __forceinline__ void fold(const Turn &t, const Pairs &w, Pairs &m, Pairs &k) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        m.a[i] = f32x2_mul(t.c[i], w.a[i]);
        m.b[i] = f32x2_mul(t.n[i], w.b[i]);
        k.a[i] = f32x2_mul(t.s[i], w.a[i]);
        k.b[i] = f32x2_mul(t.c[i], w.b[i]);
    }
}
// Backward: the input's gradient from the output's, y; dw gains the row's share.  With
// t = r g: dw += t x, dx = w t - x r^2 mean(w t x).
template <int D>
__device__ __forceinline__ Pairs row_backward(const Pairs &x, const Pairs &y, const Turn &t, const Pairs &w, Pairs &dw,
                                              float eps) {
    const float r = rsqrtf(fmaf(row_sum<D>(dot8(x, x)), 1.f / D, eps));
    const uint64_t r2 = both(r);
    Pairs g, o;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        // the gradient turned back
        g.a[i] = f32x2_fma(y.a[i], t.c[i], f32x2_mul(y.b[i], t.s[i]));
        g.b[i] = f32x2_fma(y.b[i], t.c[i], f32x2_mul(y.a[i], t.n[i]));
        g.a[i] = f32x2_mul(g.a[i], r2);
        g.b[i] = f32x2_mul(g.b[i], r2);
        dw.a[i] = f32x2_fma(g.a[i], x.a[i], dw.a[i]);
        dw.b[i] = f32x2_fma(g.b[i], x.b[i], dw.b[i]);
        g.a[i] = f32x2_mul(g.a[i], w.a[i]);
        g.b[i] = f32x2_mul(g.b[i], w.b[i]);
    }
    const uint64_t c = both(row_sum<D>(dot8(g, x)) * (r * (-1.f / D)) * r);  // no r^2: it may overflow
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        o.a[i] = f32x2_fma(c, x.a[i], g.a[i]);
        o.b[i] = f32x2_fma(c, x.b[i], g.b[i]);
    }
    return o;
}

// The block's sum of dw into its row of `partial`: lanes of one column, then warps,
// always in this order.
template <int D, bool INTER>
__device__ __forceinline__ void store_dw(const Pairs (&dw)[2], const Lane<D, INTER> &L, float *partial) {
    __shared__ float red[kNormWarps][2][D];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint64_t q = e < 4 ? dw[m].a[(e & 3) / 2] : dw[m].b[(e & 3) / 2];
            float v = e & 1 ? f32x2_hi(q) : f32x2_lo(q);
#pragma unroll
            for (int o = D / 8; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            if (lane < D / 8) red[warp][m][L.at(e)] = v;
        }
    __syncthreads();
    if (threadIdx.x < 2 * D) {
        float v = 0.f;
#pragma unroll
        for (int x = 0; x < kNormWarps; ++x) v += (&red[x][0][0])[threadIdx.x];
        partial[threadIdx.x] = v;
    }
}

// Row groups of a set, which a warp loads at a time: 2 KB, of the input or of input and
// gradient.
__host__ __device__ constexpr int norm_groups(bool backward, int size) { return (backward ? 4 : 8) / size; }
// Blocks per SM (80 and 128 registers a thread).
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

// cp.async of N bytes; zeros if not `on` (the address is then not read).
template <int N>
__device__ __forceinline__ void async_copy(uint32_t dst, const void *src, bool on) {
    const int n = on ? N : 0;
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(n) : "memory");
}
template <int N>
__device__ __forceinline__ void async_copy(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N) : "memory");
}
__device__ __forceinline__ void async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

constexpr int kSetBytes = 2048, kNormStages = 3;
constexpr int kNormRing = kNormWarps * kNormStages * kSetBytes;

// A warp walks its tokens' sets of U row groups and loads two sets ahead, across
// tensors and tokens, into a ring in shared memory of which every lane reads what it
// copied itself (so nothing but its own copies is waited for); the gradient with sets of
// twice the rows and the ring of four sets: no faster.  Loads into registers, one set at
// a time, took 95 us for 65536 tokens of 16 + 16 heads of 64 (537 MB; so 87 us, 6.2 TB/s), and
// 72 us for the gradient of 32768 tokens of 16 + 4 heads (252 MB; so 60 us, 4.2 TB/s: its
// arithmetic keeps two thirds of the issue slots busy; in fp32, 503 MB, 87 us, 5.8 TB/s).
// The arithmetic is packed (fp32 pairs) and the forward's gains are folded into the angles
// once per token and tensor (139 us without either).

template <typename T, int D, bool INTER, bool BWD>
__global__ void __launch_bounds__(32 * kNormWarps, norm_per_sm(BWD))
norm_rotate_kernel(const NormArgs<T> a) {
    constexpr int kLanes = D / 8, kRows = 32 / kLanes, U = norm_groups(BWD, sizeof(T));
    using Row = Row8<T, INTER>;
    __shared__ __align__(16) float2 cs_buf[kNormWarps][32];
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

    extern __shared__ __align__(16) uint8_t ring[];
    constexpr int V = 4 * sizeof(T), X = BWD ? 2 : 1;  // bytes of a run; tensors read
    static_assert(U * X * 2 * V * 32 == kSetBytes, "size of a set");
    // a stage: group by group two runs of x, then of the gradient, each 32 lanes side by side
    const uint32_t ring_at = smem_u32(ring) + warp * (kNormStages * kSetBytes) + lane * V;

    // this warp's tokens, every n_warps-th, as (b, t); a token's sets: U groups of its
    // queries, every gridDim.y-th, then of its keys
    const int n_warps = gridDim.x * kNormWarps, tok0 = blockIdx.x * kNormWarps + warp;
    const int step_b = n_warps / a.T_, step_t = n_warps - step_b * a.T_;
    int b = tok0 / a.T_, t = tok0 - b * a.T_;
    int left = tok0 < a.tokens ? (int)((a.tokens - tok0 + n_warps - 1) / n_warps) : 0;
    int n_sets[2];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        const int all = (a.H[m] + U * kRows - 1) / (U * kRows);
        n_sets[m] = (all - (int)blockIdx.y + (int)gridDim.y - 1) / (int)gridDim.y;
    }
    auto step = [&](int &bb, int &tt) {
        bb += step_b;
        tt += step_t;
        if (tt >= a.T_) {
            tt -= a.T_;
            ++bb;
        }
    };
    // the set to be loaded next: its token, how many of its tensor are left, its first head
    // and rows
    int lb = b, lt = t, l_left = n_sets[0] + n_sets[1] > 0 ? left : 0, lm = n_sets[0] > 0 ? 0 : 1, li = 0, lh = 0;
    const T *lx = nullptr, *lg = nullptr;
    uint32_t l_at = ring_at;
    auto load_tensor = [&]() {  // the first set of the token's tensor lm
        li = n_sets[lm];
        lh = (int)blockIdx.y * (U * kRows);
        lx = a.x[lm] + lb * a.sb[lm] + lt * a.st[lm] + (lh + sub) * a.sh[lm] + L.o0;
        if (BWD) lg = a.gy[lm] + (((long long)lb * a.H[lm] + lh + sub) * a.T_ + lt) * D + L.o0;
    };
    if (l_left > 0) load_tensor();
    const int run = L.o1 - L.o0;
    const long long yh = (long long)a.T_ * D * kRows;
    auto load_next = [&]() {
        if (l_left > 0) {
            const long long sh = a.sh[lm] * kRows;
            const int H = a.H[lm];
            if (lh + U * kRows <= H) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const T *x = lx + u * sh;
                    async_copy<V>(l_at + (u * 2 * X) * (32 * V), x);
                    async_copy<V>(l_at + (u * 2 * X + 1) * (32 * V), x + run);
                    if (BWD) {
                        const T *g = lg + u * yh;
                        async_copy<V>(l_at + (u * 2 * X + 2) * (32 * V), g);
                        async_copy<V>(l_at + (u * 2 * X + 3) * (32 * V), g + run);
                    }
                }
            } else {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const bool on = lh + u * kRows + sub < H;
                    const T *x = on ? lx + u * sh : a.x[lm];
                    async_copy<V>(l_at + (u * 2 * X) * (32 * V), x, on);
                    async_copy<V>(l_at + (u * 2 * X + 1) * (32 * V), on ? x + run : x, on);
                    if (BWD) {
                        const T *g = on ? lg + u * yh : a.gy[lm];
                        async_copy<V>(l_at + (u * 2 * X + 2) * (32 * V), g, on);
                        async_copy<V>(l_at + (u * 2 * X + 3) * (32 * V), on ? g + run : g, on);
                    }
                }
            }
            if (--li > 0) {
                lh += gridDim.y * (U * kRows);
                lx += gridDim.y * (U * sh);
                if (BWD) lg += gridDim.y * (U * yh);
            } else {
                if (lm == 0 && n_sets[1] > 0) {
                    lm = 1;
                } else {
                    lm = n_sets[0] > 0 ? 0 : 1;
                    step(lb, lt);
                    --l_left;
                }
                if (l_left > 0) load_tensor();
            }
        }
        async_commit();
        l_at = l_at == ring_at + (kNormStages - 1) * kSetBytes ? ring_at : l_at + kSetBytes;
    };
#pragma unroll
    for (int x = 0; x < kNormStages - 1; ++x) load_next();
    uint32_t r_at = ring_at;  // the stage read
    auto position = [&](int bb, int tt) { return a.pos ? a.pos[bb * a.pos_stride + tt] : (long long)tt; };
    long long pos = left > 0 ? position(b, t) : 0;
    for (; left > 0; --left) {
        share_angles(cs_buf[warp], lane, pos, turn_freq, a.n_rot);
        // the next token's place and position, a token ahead
        int nb = b, nt = t;
        step(nb, nt);
        if (left > 1) pos = position(nb, nt);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const int H = a.H[m];
            if (n_sets[m] <= 0) continue;
            const float4 u0 = *reinterpret_cast<const float4 *>(&cs_buf[warp][L.p0]);
            const float4 u1 = *reinterpret_cast<const float4 *>(&cs_buf[warp][L.p0 + 2]);
            const float2 cs[4] = {{u0.x, u0.y}, {u0.z, u0.w}, {u1.x, u1.y}, {u1.z, u1.w}};
            const Turn turn = turn_of(cs);
            const Pairs w = gains(w_buf[m], L);
            Pairs fm, fk;
            if (!BWD) fold(turn, w, fm, fk);
            int h = blockIdx.y * (U * kRows);
            const long long oh = BWD ? a.dh[m] * kRows : (long long)a.T_ * D * kRows;
            T *po = BWD ? a.dx[m] + b * a.db[m] + t * a.dt[m] + (h + sub) * a.dh[m]
                        : a.y[m] + (((long long)b * H + h + sub) * a.T_ + t) * D;
            for (int i = 0; i < n_sets[m]; ++i) {
                load_next();
                async_wait<kNormStages - 1>();
                auto work = [&](int u, bool on) {
                    Row rx, rg;
                    rx.load_shared(r_at + (u * 2 * X) * (32 * V), r_at + (u * 2 * X + 1) * (32 * V));
                    Pairs o;
                    if constexpr (BWD) {
                        rg.load_shared(r_at + (u * 2 * X + 2) * (32 * V), r_at + (u * 2 * X + 3) * (32 * V));
                        o = row_backward<D>(rx.get(), rg.get(), turn, w, dw[m], a.eps);
                    } else {
                        o = row_forward<D>(rx.get(), fm, fk, a.eps);
                    }
                    if (on) Row::store(po + u * oh, L.o0, L.o1, o);
                };
                if (h + U * kRows <= H) {
#pragma unroll
                    for (int u = 0; u < U; ++u) work(u, true);
                } else {
                    for (int u = 0; u < U && h + u * kRows < H; ++u) work(u, h + u * kRows + sub < H);
                }
                r_at = r_at == ring_at + (kNormStages - 1) * kSetBytes ? ring_at : r_at + kSetBytes;
                h += gridDim.y * (U * kRows);
                po += gridDim.y * (U * oh);
            }
        }
        b = nb;
        t = nt;
    }
    async_wait<0>();
    if constexpr (BWD)
        store_dw(dw, L, a.partial + ((long long)blockIdx.y * gridDim.x + blockIdx.x) * (2 * D));
}

// The same for few heads: a warp takes G row groups of each tensor at once, which are
// all heads of a token, or with one group those of several consecutive tokens, 2^hs
// rows to a token.  A token's rows are loaded together, a turn ahead, and each lane
// works out its own four angles.  Forward / gradient of 60000 tokens, us, above and so: 2
// groups, 8 + 8 heads of 64, 68 / 79 and 51 / 87 (so the gradient is not done so), 6 + 3 heads
// 62 / 79 and 45 / 71, 16 + 16 heads of 32 67 / 79 and 51 / 83; 1 group, 4 + 4 heads of 64, 56 / 70 and
// 35 / 50.  4 groups, 12 + 12 heads, take 82 us above and 80 so.
template <typename T, int D, bool INTER, bool BWD, int G>
__global__ void __launch_bounds__(32 * kNormWarps, 2)
norm_rotate_packed_kernel(const NormArgs<T> a, int hs) {
    constexpr int kLanes = D / 8, kRows = 32 / kLanes;
    using Row = Row8<T, INTER>;
    __shared__ float w_buf[2][D];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, sub = lane / kLanes;
    const Lane<D, INTER> L(lane, a.n_rot);
    double freq[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        freq[j] = L.p0 + j < a.n_rot ? (double)a.inv_freq[L.p0 + j] * 0.15915494309189533577 : 0.0;
    for (int x = threadIdx.x; x < 2 * D; x += 32 * kNormWarps) {
        const float *src = x < D ? a.w[0] : a.w[1];
        (&w_buf[0][0])[x] = src ? src[x % D] : 1.f;
    }
    __syncthreads();
    Pairs dw[2] = {};
    const int per = kRows >> hs, h = sub & ((1 << hs) - 1);  // tokens of a warp, the lane's head
    const long long step = (long long)gridDim.x * kNormWarps * per;
    const int step_b = (int)(step / a.T_), step_t = (int)(step - (long long)step_b * a.T_);
    long long tok = ((long long)blockIdx.x * kNormWarps + warp) * per;  // the warp's first token
    const long long mine = tok + (sub >> hs);
    int b = (int)(mine / a.T_), t = (int)(mine - (long long)b * a.T_);
    struct Data {
        Row x[2][G], g[BWD ? 2 : 1][BWD ? G : 1];
        long long pos;
    };
    auto load = [&](int bb, int tt, bool on, Data &d) {
        d.pos = on && a.n_rot > 0 ? (a.pos ? a.pos[bb * a.pos_stride + tt] : (long long)tt) : 0;
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int u = 0; u < G; ++u) {
                const int hu = h + u * kRows;
                d.x[m][u].zero();
                if (BWD) d.g[m][u].zero();
                if (on && hu < a.H[m]) {
                    d.x[m][u].load(a.x[m] + bb * a.sb[m] + tt * a.st[m] + hu * a.sh[m], L.o0, L.o1);
                    if (BWD)
                        d.g[m][u].load(a.gy[m] + (((long long)bb * a.H[m] + hu) * a.T_ + tt) * D, L.o0, L.o1);
                }
            }
    };
    Data d;
    if (tok < a.tokens) load(b, t, mine < a.tokens, d);
    for (; tok < a.tokens; tok += step) {
        int nb = b + step_b, nt = t + step_t;
        if (nt >= a.T_) {
            nt -= a.T_;
            ++nb;
        }
        const long long at = tok + (sub >> hs);
        Data n;
        load(nb, nt, at + step < a.tokens, n);
        float2 cs[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const double turns = (double)d.pos * freq[j];
            sincospif((float)(2.0 * (turns - rint(turns))), &cs[j].y, &cs[j].x);
        }
        const Turn turn = turn_of(cs);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            if (a.H[m] == 0) continue;
            const Pairs w = gains(w_buf[m], L);
            Pairs fm, fk;
            if (!BWD) fold(turn, w, fm, fk);
#pragma unroll
            for (int u = 0; u < G; ++u) {
                if (u > 0 && u * kRows >= a.H[m]) break;
                const int hu = h + u * kRows;
                Pairs o;
                if constexpr (BWD)
                    o = row_backward<D>(d.x[m][u].get(), d.g[m][u].get(), turn, w, dw[m], a.eps);
                else
                    o = row_forward<D>(d.x[m][u].get(), fm, fk, a.eps);
                if (at < a.tokens && hu < a.H[m]) {
                    T *po = BWD ? a.dx[m] + b * a.db[m] + t * a.dt[m] + hu * a.dh[m]
                                : a.y[m] + (((long long)b * a.H[m] + hu) * a.T_ + t) * D;
                    Row::store(po, L.o0, L.o1, o);
                }
            }
        }
        d = n;
        b = nb;
        t = nt;
    }
    if constexpr (BWD) store_dw(dw, L, a.partial + (long long)blockIdx.x * (2 * D));
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

int max_heads(const NormRotate &p) { return p.H[0] > p.H[1] ? p.H[0] : p.H[1]; }

// log2 of the rows that a token takes in the packed kernel; -1: too many heads for it.
// The forward takes two row groups, the gradient one (the figures are at the kernel).
int norm_packed(const NormRotate &p) {
    const int hm = max_heads(p), rows = 256 / p.d;
    int hs = 0;
    while ((1 << hs) < hm && (1 << hs) < rows) ++hs;
    return hm <= (p.backward ? rows : 2 * rows) ? hs : -1;
}

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
        const int hs = norm_packed(p);
        if (hs >= 0 && max_heads(p) <= 256 / D)
            norm_rotate_packed_kernel<T, D, INTER, BWD, 1><<<grid, 32 * kNormWarps, 0, st>>>(a, hs);
        else if (!BWD && hs >= 0)
            norm_rotate_packed_kernel<T, D, INTER, false, 2><<<grid, 32 * kNormWarps, 0, st>>>(a, hs);
        else {
            const cudaError_t e = smem_opt_in_once<norm_rotate_kernel<T, D, INTER, BWD>>(kNormRing);
            if (e != cudaSuccess) return e;
            norm_rotate_kernel<T, D, INTER, BWD><<<grid, 32 * kNormWarps, kNormRing, st>>>(a);
        }
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

// Blocks of the launch: as many as hold the tokens, at most what the SMs hold at a
// time; if the tokens of the unpacked kernel fill less than that, the heads are spread
// over grid.y.  The same for both types, as the workspace is.
dim3 norm_rotate_grid(const NormRotate &p) {
    const long long tokens = (long long)p.B * p.T;
    const int hs = norm_packed(p);
    const long long full = (long long)(hs >= 0 ? 2 : norm_per_sm(p.backward)) * kPlanSms;
    const long long per = kNormWarps * (hs >= 0 ? (256 / p.d) >> hs : 1);  // tokens of a block
    const long long blocks = (tokens + per - 1) / per;
    const int gx = (int)(blocks < full ? blocks : full);
    if (hs >= 0) return dim3(gx);
    const int rows = norm_groups(p.backward, 2) * (256 / p.d);  // row groups a warp could leave to others
    const int hm = max_heads(p);
    int gy = (int)(full / gx);
    if (gy > (hm + rows - 1) / rows) gy = (hm + rows - 1) / rows;
    return dim3(gx, gy < 1 ? 1 : gy);
}

cudaError_t launch_norm_rotate(const NormRotate &p, cudaStream_t st) {
    return p.dtype == KATA_BF16 ? launch_t<__nv_bfloat16>(p, st) : launch_t<float>(p, st);
}

}  // namespace kata
