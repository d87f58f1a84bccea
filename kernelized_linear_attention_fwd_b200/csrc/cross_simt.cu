// Cross attention with KATA weights in fp32 on the CUDA cores (formulas and modes:
// cross_tc.cu).  A CTA of 256 threads owns 16 RT rows and walks the other axis in
// blocks of 64 columns: thread (ty, tx) forms the scores of rows ty RT + i and
// columns tx + 16 j, stores the weights in shared memory, and accumulates D / 16
// columns of the same rows.  Bound by the FFMA pipe (4 d flops per pair and
// product pass); RT = 1 keeps short row counts from computing 64 rows.
//
// Every block's sum is formed on its own and then added to the total, so that a
// chain of additions is 64 long inside a block and Tk / 64 long across blocks.
#include "kata_internal.cuh"

namespace kata {
namespace {

constexpr int kCols = 64;
constexpr int kPs = kCols + 4;  // row stride of the weights

struct SArgs {
    int rows, cols, Hkv, tiles, splits, Tk, stat_stride;
    long long BH;
    const int *key_lengths;
    const float *r0, *r1, *c0, *c1;
    float *o0, *o1, *y, *den, *part, *part_l;
    const float *delta, *rden;
};

template <int D, int MODE, int RT>
constexpr int simt_smem() {
    constexpr int TR = 16 * RT, S = D + 4;
    return 4 * (TR * S * (MODE == kCrossFwd ? 1 : 2) + 2 * kCols * S + TR * kPs * (MODE == kCrossDkv ? 2 : 1) +
                2 * kCols);
}

// n rows of D floats into shared memory, rows from `live` on as zeros.
template <int D>
__device__ __forceinline__ void load_tile(float *dst, const float *src, int n, int live) {
    for (int x = threadIdx.x; x < n * (D / 4); x += 256) {
        const int r = x / (D / 4), c = 4 * (x % (D / 4));
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < live) v = *reinterpret_cast<const float4 *>(src + (long long)r * D + c);
        *reinterpret_cast<float4 *>(dst + r * (D + 4) + c) = v;
    }
}

// s[i][j] = row (ty RT + i) of `a` times row (tx + 16 j) of `b`.
template <int D, int RT>
__device__ __forceinline__ void dots(float (&s)[RT][4], const float *a, const float *b, int ty, int tx) {
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
    for (int k = 0; k < D; k += 4) {
        float4 x[RT], y[4];
#pragma unroll
        for (int i = 0; i < RT; ++i) x[i] = *reinterpret_cast<const float4 *>(a + (ty * RT + i) * (D + 4) + k);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4 *>(b + (tx + 16 * j) * (D + 4) + k);
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] = fmaf(x[i].x, y[j].x, s[i][j]);
                s[i][j] = fmaf(x[i].y, y[j].y, s[i][j]);
                s[i][j] = fmaf(x[i].z, y[j].z, s[i][j]);
                s[i][j] = fmaf(x[i].w, y[j].w, s[i][j]);
            }
    }
}

// acc[i][c] += sum over the block's columns of w[ty RT + i][.] times b[.][tx D / 16 + c].
template <int D, int RT>
__device__ __forceinline__ void accumulate(float (&acc)[RT][D / 16], const float *w, const float *b, int ty, int tx) {
    constexpr int N = D / 16;
    float s[RT][N] = {};
#pragma unroll 4
    for (int j = 0; j < kCols; j += 4) {
        float4 p[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) p[i] = *reinterpret_cast<const float4 *>(w + (ty * RT + i) * kPs + j);
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
            float v[N];
#pragma unroll
            for (int c = 0; c < N; ++c) v[c] = b[(j + jj) * (D + 4) + tx * N + c];
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                const float f = jj == 0 ? p[i].x : jj == 1 ? p[i].y : jj == 2 ? p[i].z : p[i].w;
#pragma unroll
                for (int c = 0; c < N; ++c) s[i][c] = fmaf(f, v[c], s[i][c]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int c = 0; c < N; ++c) acc[i][c] += s[i][c];
}

template <int D, int MODE, int RT>
__global__ void __launch_bounds__(256)
cross_simt_kernel(const SArgs a) {
    constexpr int TR = 16 * RT, S = D + 4, N = D / 16;
    extern __shared__ float sm[];
    float *R0 = sm, *R1 = R0 + TR * S;  // R1: backward only
    float *C0 = R0 + TR * S * (MODE == kCrossFwd ? 1 : 2), *C1 = C0 + kCols * S;
    float *P = C1 + kCols * S, *E = P + TR * kPs;  // E: dkv only
    float *sd = P + TR * kPs * (MODE == kCrossDkv ? 2 : 1), *sr = sd + kCols;

    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    const int split = blockIdx.x % a.splits, x = blockIdx.x / a.splits;
    const int bh = x / a.tiles, r0 = (x % a.tiles) * TR;
    const int live = cross_length(a.key_lengths, bh / a.Hkv, a.Tk);
    const int rows = MODE == kCrossDkv ? live : a.rows, cols = MODE == kCrossDkv ? a.cols : live;
    const int blocks = rows > r0 ? (cols + kCols - 1) / kCols : 0;
    const int piece = (blocks + a.splits - 1) / a.splits;
    const int b0 = split * piece, b1 = min(blocks, b0 + piece);
    const long long row0 = (long long)bh * a.rows + r0, col0 = (long long)bh * a.cols;

    float acc0[RT][N] = {}, acc1[RT][N] = {}, l[RT] = {}, delta[RT] = {};  // delta: -D
    if (b0 < b1) {
        load_tile<D>(R0, a.r0 + row0 * D, TR, rows - r0);
        if (MODE != kCrossFwd) load_tile<D>(R1, a.r1 + row0 * D, TR, rows - r0);
    }
    if (MODE == kCrossDq) {
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const int r = r0 + ty * RT + i;
            if (r < a.rows) delta[i] = a.delta[(long long)bh * a.stat_stride + r];
        }
    }
    for (int b = b0; b < b1; ++b) {
        const int c0 = b * kCols;
        __syncthreads();  // the last block's operands are read
        load_tile<D>(C0, a.c0 + (col0 + c0) * D, kCols, cols - c0);
        load_tile<D>(C1, a.c1 + (col0 + c0) * D, kCols, cols - c0);
        if (MODE == kCrossDkv && threadIdx.x < kCols) {
            sd[threadIdx.x] = a.delta[(long long)bh * a.stat_stride + c0 + threadIdx.x];
            sr[threadIdx.x] = a.rden[(long long)bh * a.stat_stride + c0 + threadIdx.x];
        }
        __syncthreads();
        float s[RT][4], g[RT][4];
        dots<D, RT>(s, R0, C0, ty, tx);
        if (MODE != kCrossFwd) dots<D, RT>(g, R1, C1, ty, tx);
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            float lb = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int o = (ty * RT + i) * kPs + tx + 16 * j;
                if (MODE == kCrossFwd) {
                    const float w = s[i][j] * s[i][j];
                    lb += w;
                    P[o] = w;
                } else if (MODE == kCrossDq) {
                    P[o] = s[i][j] * (g[i][j] + delta[i]);
                } else {
                    const float t = s[i][j] * sr[tx + 16 * j];
                    P[o] = s[i][j] * t;
                    E[o] = 2.f * t * (g[i][j] + sd[tx + 16 * j]);
                }
            }
            l[i] += lb;
        }
        __syncthreads();
        accumulate<D, RT>(acc0, P, MODE == kCrossDq ? C0 : C1, ty, tx);
        if (MODE == kCrossDkv) accumulate<D, RT>(acc1, E, C0, ty, tx);
    }
    if (MODE == kCrossFwd) {
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
    }
    const long long n_rows = a.BH * a.rows;
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        const int r = r0 + ty * RT + i;
        if (r >= a.rows) continue;
        const long long gr = (long long)bh * a.rows + r;
        if (a.splits > 1) {
            const long long pr = (MODE == kCrossDkv ? 2 : 1) * split * n_rows + gr;
#pragma unroll
            for (int c = 0; c < N; ++c) {
                a.part[pr * D + tx * N + c] = acc0[i][c];
                if (MODE == kCrossDkv) a.part[(pr + n_rows) * D + tx * N + c] = acc1[i][c];
            }
            if (MODE == kCrossFwd && tx == 0) a.part_l[pr] = l[i];
            continue;
        }
        float f = 1.f;
        if (MODE == kCrossFwd) f = cross_recip(l[i]);
        if (MODE == kCrossDq) f = 2.f * a.rden[(long long)bh * a.stat_stride + r];
#pragma unroll
        for (int c = 0; c < N; ++c) {
            const float v = acc0[i][c] * f;
            a.o0[gr * D + tx * N + c] = v;
            if (MODE == kCrossFwd && a.y) a.y[gr * D + tx * N + c] = v;
            if (MODE == kCrossDkv) a.o1[gr * D + tx * N + c] = acc1[i][c];
        }
        if (MODE == kCrossFwd && a.den && tx == 0) a.den[gr] = l[i];
    }
}

template <int D, int MODE, int RT>
cudaError_t launch_one(const CrossPlan &p, const CrossIo &io, cudaStream_t st) {
    const char *ws = static_cast<const char *>(io.ws);
    auto f = [](const void *x) { return static_cast<const float *>(x); };
    auto w = [&](size_t o) { return reinterpret_cast<float *>(const_cast<char *>(ws) + o); };
    SArgs a{};
    a.rows = MODE == kCrossDkv ? p.Tk : p.R;
    a.cols = MODE == kCrossDkv ? p.R : p.Tk;
    a.Hkv = p.Hkv;
    a.tiles = (a.rows + 16 * RT - 1) / (16 * RT);
    a.splits = p.splits[MODE];
    a.Tk = p.Tk;
    a.stat_stride = p.R_pad;
    a.BH = p.BH;
    a.key_lengths = io.key_lengths;
    a.r0 = f(MODE == kCrossDkv ? io.k : io.q);
    a.r1 = f(MODE == kCrossDkv ? io.v : io.dout);
    a.c0 = f(MODE == kCrossDkv ? io.q : io.k);
    a.c1 = f(MODE == kCrossDkv ? io.dout : io.v);
    a.o0 = static_cast<float *>(MODE == kCrossFwd ? io.out : MODE == kCrossDq ? io.dq : io.dv);
    a.o1 = static_cast<float *>(io.dk);
    a.y = io.y;
    a.den = io.den;
    a.part = w(p.ws_part[MODE]);
    a.part_l = w(p.ws_part_l);
    a.delta = w(p.ws_delta);
    a.rden = w(p.ws_rden);
    constexpr int smem = simt_smem<D, MODE, RT>();
    const cudaError_t e = smem_opt_in_once<cross_simt_kernel<D, MODE, RT>>(smem);
    if (e != cudaSuccess) return e;
    ProfScope prof(MODE == kCrossFwd ? "cross_fwd_simt" : MODE == kCrossDq ? "cross_dq_simt" : "cross_dkv_simt", st);
    cross_simt_kernel<D, MODE, RT><<<(unsigned)(p.BH * a.tiles * a.splits), 256, smem, st>>>(a);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(CrossMode mode, const CrossPlan &p, const CrossIo &io, cudaStream_t st) {
    if (mode == kCrossDq) return launch_one<D, kCrossDq, 4>(p, io, st);
    if (mode == kCrossDkv) return launch_one<D, kCrossDkv, 4>(p, io, st);
    return cross_simt_rows(mode, p) == 16 ? launch_one<D, kCrossFwd, 1>(p, io, st)
                                          : launch_one<D, kCrossFwd, 4>(p, io, st);
}

}  // namespace

int cross_simt_rows(CrossMode mode, const CrossPlan &p) { return mode == kCrossFwd && p.R <= 16 ? 16 : 64; }

cudaError_t launch_cross_simt(CrossMode mode, const CrossPlan &p, const CrossIo &io, cudaStream_t st) {
    switch (p.d) {
        case 16: return launch_d<16>(mode, p, io, st);
        case 32: return launch_d<32>(mode, p, io, st);
        default: return launch_d<64>(mode, p, io, st);
    }
}

}  // namespace kata
