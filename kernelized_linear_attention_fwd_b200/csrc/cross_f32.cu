// Cross attention with KATA weights in fp32 (formulas and modes: cross_tc.cu), on the
// tensor cores with every fp32 operand as the sum of three bf16 numbers (the published
// splitting of Henry, Tang and Heinecke, "Leveraging the bfloat16 Artificial Intelligence
// Datatype For Higher-Precision Computations", ARITH 2019):
//
//   x = h + m + l,  h = bf16(x), m = bf16(x - h), l = bf16(x - h - m)
//
// (8 + 8 + 8 significant bits; both differences are exact), so that
//
//   x y = h h' + (h m' + m h') + (h l' + m m' + l h')  up to 2^-24 |x y|:
//
// six products of exact bf16 pairs summed in fp32.  The five small ones come before
// h h', so that only a block's last few additions round at the sum's own size, and
// every block's sum is formed on its own and then added to the total in fp32.  Error
// against exact, rms: 1.5e-7 to 1.9e-7 (the same in plain fp32 products: 2.4e-7).
//
// A CTA of 4 warps owns 64 rows and walks the other axis in blocks of 64 columns, whose
// operands it splits into three planes of shared memory as it loads them.  A warp
// holds 16 rows: scores and accumulators are fragments in registers, and the weights,
// formed in the scores' fragments, are the operand of the next product as they lie.
// The register-level products (mma.sync) suit tiles this small, whose split takes
// the arithmetic of all the warps: tcgen05 would need the three planes of the
// weights in tensor memory beside their scores, 192 columns where a step of the bf16
// kernel has 128.  Measured (8 heads, 2048 queries and keys, d = 64): forward 153 us,
// gradient 475 us, which is 56 and 63 TFLOP/s of fp32 products (the CUDA cores' form of
// this kernel: 279 and 915 us, bound by its shared-memory reads; 8192 queries and keys:
// 2.02 and 6.7 ms, 68 and 72 TFLOP/s).  The register-level products' pipe is 66 to 74%
// active; six products at the bf16 rate of tcgen05 would allow some 275 TFLOP/s, so this
// path is a choice of simplicity for a precision that serves small training, not a limit.
// (With twice as many chains of products side by side: the same.)
#include <cuda_bf16.h>

#include "kata_internal.cuh"
#include "sm100.cuh"

namespace kata {
namespace {

using namespace kata::sm100;

constexpr int kN = kF32Tile;           // rows of a CTA, columns of a block
constexpr int kPlane = kN * 128;       // bytes: rows of 64 bf16, 16-byte chunks swizzled by row
constexpr int kOperand = 3 * kPlane;
constexpr int kThreads = 128;

template <int MODE>
constexpr int f32_smem() {
    return ((MODE == kCrossFwd ? 1 : 2) + 2) * kOperand + (MODE == kCrossDkv ? 2 * kN * 4 : 0);
}

struct FArgs {
    int rows, cols, Hkv, tiles, splits, Tk, stat_stride;
    long long BH;
    const int *key_lengths;
    const float *r0, *r1, *c0, *c1;
    float *o0, *o1, *y, *den, *part, *part_l;
    const float *delta, *rden;  // -D, 1 / l
};

// Byte offset of 16-byte chunk `chunk` of row `row` in a plane.
__device__ __forceinline__ uint32_t at(int row, int chunk) { return row * 128 + ((chunk ^ (row & 7)) << 4); }

// Two fp32 values as three bf16 pairs.
__device__ __forceinline__ void split2(float x, float y, uint32_t &h, uint32_t &m, uint32_t &l) {
    h = pack_bf16x2(x, y);
    x -= __uint_as_float(h << 16);
    y -= __uint_as_float(h & 0xFFFF0000u);
    m = pack_bf16x2(x, y);
    x -= __uint_as_float(m << 16);
    y -= __uint_as_float(m & 0xFFFF0000u);
    l = pack_bf16x2(x, y);
}

// N times 64 rows of D floats into three planes each, rows from `live` on as zeros.  All
// loads are issued before the first is split: the wait for memory is the same for one
// operand and for four.
struct Source {
    uint8_t *dst;
    const float *src;
    int live;
};
template <int D, int N>
__device__ __forceinline__ void load_planes(const Source (&op)[N]) {
    constexpr int K = kN * (D / 4) / kThreads;
    float4 v[N][K];
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int x = threadIdx.x + k * kThreads, r = x / (D / 4), c = x % (D / 4);
            v[n][k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < op[n].live) v[n][k] = *reinterpret_cast<const float4 *>(op[n].src + (long long)r * D + 4 * c);
        }
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int x = threadIdx.x + k * kThreads, r = x / (D / 4), c = x % (D / 4);
            uint2 p[3];
            split2(v[n][k].x, v[n][k].y, p[0].x, p[1].x, p[2].x);
            split2(v[n][k].z, v[n][k].w, p[0].y, p[1].y, p[2].y);
            const uint32_t o = at(r, c / 2) + 8 * (c & 1);
#pragma unroll
            for (int i = 0; i < 3; ++i) *reinterpret_cast<uint2 *>(op[n].dst + i * kPlane + o) = p[i];
        }
}

__device__ __forceinline__ void ldm(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldm_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The five small products of two 8-column tiles, smallest first; planes h, m, l.
__device__ __forceinline__ void mma_small(float (&c0)[4], float (&c1)[4], const uint32_t (&a)[3][4],
                                          const uint32_t (&b)[3][4]) {
    constexpr int ia[5] = {2, 0, 1, 1, 0}, ib[5] = {0, 2, 1, 0, 1};
#pragma unroll
    for (int i = 0; i < 5; ++i) {
        mma(c0, a[ia[i]], b[ib[i]][0], b[ib[i]][1]);
        mma(c1, a[ia[i]], b[ib[i]][2], b[ib[i]][3]);
    }
}

// s[j] = rows r0 .. r0 + 15 of `a` times the 8 rows of column tile j of `b`, both
// [64][D] in planes.
template <int D>
__device__ __forceinline__ void scores(float (&s)[8][4], uint32_t a, uint32_t b, int r0, int lane) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[j][e] = 0.f;
    const int ra = r0 + (lane & 15), ca = lane >> 4;
    const int rb = (lane & 7) + ((lane >> 4) << 3), cb = (lane >> 3) & 1;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
        uint32_t fa[3][4];
#pragma unroll
        for (int p = 0; p < 3; ++p) ldm(fa[p], a + p * kPlane + at(ra, 2 * k + ca));
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            uint32_t fb[3][4];
#pragma unroll
            for (int p = 0; p < 3; ++p) ldm(fb[p], b + p * kPlane + at(rb + 8 * j, 2 * k + cb));
            mma_small(s[j], s[j + 1], fa, fb);
        }
    }
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {  // h h'
        uint32_t fa[4];
        ldm(fa, a + at(ra, 2 * k + ca));
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            uint32_t fb[4];
            ldm(fb, b + at(rb + 8 * j, 2 * k + cb));
            mma(s[j], fa, fb[0], fb[1]);
            mma(s[j + 1], fa, fb[2], fb[3]);
        }
    }
}

// acc[j] += weights (fragments of 16 rows and 64 columns, given by w(tile, e)) times
// column tile j of `b` [64][D] in planes.
template <int D, typename W>
__device__ __forceinline__ void accumulate(float (&acc)[D / 8][4], W w, uint32_t b, int lane) {
    float t[D / 8][4];
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) t[j][e] = 0.f;
    const int rb = lane & 15, cb = lane >> 4;
    uint32_t hi[4][4];
#pragma unroll
    for (int k = 0; k < kN / 16; ++k) {
        uint32_t fa[3][4];
#pragma unroll
        for (int x = 0; x < 4; ++x)  // rows g, g + 8 of tile 2k, then of tile 2k + 1
            split2(w(2 * k + x / 2, 2 * (x & 1)), w(2 * k + x / 2, 2 * (x & 1) + 1), fa[0][x], fa[1][x], fa[2][x]);
#pragma unroll
        for (int x = 0; x < 4; ++x) hi[k][x] = fa[0][x];
#pragma unroll
        for (int j = 0; j < D / 8; j += 2) {
            uint32_t fb[3][4];
#pragma unroll
            for (int p = 0; p < 3; ++p) ldm_t(fb[p], b + p * kPlane + at(16 * k + rb, j + cb));
            mma_small(t[j], t[j + 1], fa, fb);
        }
    }
#pragma unroll
    for (int k = 0; k < kN / 16; ++k)
#pragma unroll
        for (int j = 0; j < D / 8; j += 2) {
            uint32_t fb[4];
            ldm_t(fb, b + at(16 * k + rb, j + cb));
            mma(t[j], hi[k], fb[0], fb[1]);
            mma(t[j + 1], hi[k], fb[2], fb[3]);
        }
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][e] += t[j][e];
}

template <int D, int MODE>
__device__ __forceinline__ void cross_f32(const FArgs &a, int cta, uint8_t *sm) {
    uint8_t *R0 = sm, *R1 = R0 + kOperand;  // R1: backward only
    uint8_t *C0 = R0 + (MODE == kCrossFwd ? 1 : 2) * kOperand, *C1 = C0 + kOperand;
    float *sd = reinterpret_cast<float *>(C1 + kOperand), *sr = sd + kN;  // dkv only

    const int lane = threadIdx.x % 32, w0 = threadIdx.x / 32 * 16;  // the warp's first row
    const int g = lane / 4, q = 2 * (lane % 4);                     // fragment row and first column
    const int split = cta % a.splits, x = cta / a.splits;
    const int bh = x / a.tiles, r0 = (x % a.tiles) * kN;
    const int live = cross_length(a.key_lengths, bh / a.Hkv, a.Tk);
    const int rows = MODE == kCrossDkv ? live : a.rows, cols = MODE == kCrossDkv ? a.cols : live;
    const int blocks = rows > r0 ? (cols + kN - 1) / kN : 0;
    const int piece = (blocks + a.splits - 1) / a.splits;
    const int b0 = split * piece, b1 = min(blocks, b0 + piece);
    const long long row0 = (long long)bh * a.rows + r0, col0 = (long long)bh * a.cols;

    float acc0[D / 8][4] = {}, acc1[MODE == kCrossDkv ? D / 8 : 1][4] = {};
    float l[2] = {0.f, 0.f}, delta[2] = {0.f, 0.f};  // of rows w0 + g and w0 + g + 8
    if (MODE == kCrossDq) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = r0 + w0 + g + 8 * i;
            if (r < a.rows) delta[i] = a.delta[(long long)bh * a.stat_stride + r];
        }
    }
    for (int b = b0; b < b1; ++b) {
        const int c0 = b * kN;
        const Source s0 = {C0, a.c0 + (col0 + c0) * D, cols - c0}, s1 = {C1, a.c1 + (col0 + c0) * D, cols - c0};
        __syncthreads();  // the last block's operands are read
        if (b > b0) {
            load_planes<D>({s0, s1});
        } else if constexpr (MODE == kCrossFwd) {
            load_planes<D>({{R0, a.r0 + row0 * D, rows - r0}, s0, s1});
        } else {
            load_planes<D>({{R0, a.r0 + row0 * D, rows - r0}, {R1, a.r1 + row0 * D, rows - r0}, s0, s1});
        }
        if (MODE == kCrossDkv && threadIdx.x < kN) {
            sd[threadIdx.x] = a.delta[(long long)bh * a.stat_stride + c0 + threadIdx.x];
            sr[threadIdx.x] = a.rden[(long long)bh * a.stat_stride + c0 + threadIdx.x];
        }
        __syncthreads();
        float s[8][4];
        scores<D>(s, smem_u32(R0), smem_u32(C0), w0, lane);
        if constexpr (MODE == kCrossFwd) {
            float lb[2] = {0.f, 0.f};
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[j][e] *= s[j][e];
                    lb[e / 2] += s[j][e];
                }
            l[0] += lb[0];
            l[1] += lb[1];
            accumulate<D>(acc0, [&](int j, int e) { return s[j][e]; }, smem_u32(C1), lane);
        } else {
            float p[8][4];
            scores<D>(p, smem_u32(R1), smem_u32(C1), w0, lane);
            if constexpr (MODE == kCrossDq) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[j][e] *= p[j][e] + delta[e / 2];
                accumulate<D>(acc0, [&](int j, int e) { return s[j][e]; }, smem_u32(C0), lane);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float2 d2 = *reinterpret_cast<const float2 *>(sd + 8 * j + q);
                    const float2 r2 = *reinterpret_cast<const float2 *>(sr + 8 * j + q);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float t = s[j][e] * (e & 1 ? r2.y : r2.x);
                        p[j][e] = 2.f * t * (p[j][e] + (e & 1 ? d2.y : d2.x));
                        s[j][e] *= t;
                    }
                }
                accumulate<D>(acc0, [&](int j, int e) { return s[j][e]; }, smem_u32(C1), lane);
                accumulate<D>(acc1, [&](int j, int e) { return p[j][e]; }, smem_u32(C0), lane);
            }
        }
    }
    if (MODE == kCrossFwd) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
        }
    }
    const long long n_rows = a.BH * a.rows;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = r0 + w0 + g + 8 * i;
        if (r >= a.rows) continue;
        const long long gr = (long long)bh * a.rows + r;
        const bool cut = a.splits > 1;
        const long long pr = (MODE == kCrossDkv ? 2 : 1) * split * n_rows + gr;
        float f = 1.f;
        if (!cut && MODE == kCrossFwd) f = cross_recip(l[i]);
        if (!cut && MODE == kCrossDq) f = 2.f * a.rden[(long long)bh * a.stat_stride + r];
        // padded keys beside the last visible one: zeros, also where a query that is not finite
        // turned their zero products into NaN (the length is read again: a register less above)
        const bool dead = MODE == kCrossDkv && r >= cross_length(a.key_lengths, bh / a.Hkv, a.Tk);
        float *o = cut ? a.part + pr * D : a.o0 + gr * D;
        float *o1 = MODE == kCrossDkv ? (cut ? a.part + (pr + n_rows) * D : a.o1 + gr * D) : nullptr;
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
            const float2 v = dead ? make_float2(0.f, 0.f) : make_float2(acc0[j][2 * i] * f, acc0[j][2 * i + 1] * f);
            *reinterpret_cast<float2 *>(o + 8 * j + q) = v;
            if (MODE == kCrossFwd && !cut && a.y) *reinterpret_cast<float2 *>(a.y + gr * D + 8 * j + q) = v;
            if constexpr (MODE == kCrossDkv)
                *reinterpret_cast<float2 *>(o1 + 8 * j + q) =
                    dead ? make_float2(0.f, 0.f) : make_float2(acc1[j][2 * i], acc1[j][2 * i + 1]);
        }
        if (MODE == kCrossFwd && q == 0) {
            if (cut)
                a.part_l[pr] = l[i];
            else if (a.den)
                a.den[gr] = l[i];
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 2)
cross_f32_forward(const FArgs a) {
    extern __shared__ __align__(128) uint8_t sm[];
    cross_f32<D, kCrossFwd>(a, blockIdx.x, sm);
}
// dq and dkv in one launch, dkv's longer CTAs first: neither needs the other, and the
// SMs that one leaves idle go to the other.
template <int D>
__global__ void __launch_bounds__(kThreads, 2)
cross_f32_backward(const FArgs q, const FArgs kv, int n_kv) {
    extern __shared__ __align__(128) uint8_t sm[];
    griddep_wait();
    if ((int)blockIdx.x < n_kv)
        cross_f32<D, kCrossDkv>(kv, blockIdx.x, sm);
    else
        cross_f32<D, kCrossDq>(q, blockIdx.x - n_kv, sm);
}

FArgs f32_args(CrossMode mode, const CrossPlan &p, const CrossIo &io) {
    const char *ws = static_cast<const char *>(io.ws);
    const bool dkv = mode == kCrossDkv;
    auto f = [](const void *x) { return static_cast<const float *>(x); };
    auto w = [&](size_t o) { return reinterpret_cast<float *>(const_cast<char *>(ws) + o); };
    FArgs a{};
    a.rows = dkv ? p.Tk : p.R;
    a.cols = dkv ? p.R : p.Tk;
    a.Hkv = p.Hkv;
    a.tiles = (a.rows + kN - 1) / kN;
    a.splits = p.splits[mode];
    a.Tk = p.Tk;
    a.stat_stride = p.R_pad;
    a.BH = p.BH;
    a.key_lengths = io.key_lengths;
    a.r0 = f(dkv ? io.k : io.q);
    a.r1 = f(dkv ? io.v : io.dout);
    a.c0 = f(dkv ? io.q : io.k);
    a.c1 = f(dkv ? io.dout : io.v);
    a.o0 = static_cast<float *>(mode == kCrossFwd ? io.out : mode == kCrossDq ? io.dq : io.dv);
    a.o1 = static_cast<float *>(io.dk);
    a.y = io.y;
    a.den = io.den;
    a.part = w(p.ws_part[mode]);
    a.part_l = w(p.ws_part_l);
    a.delta = w(p.ws_delta);
    a.rden = w(p.ws_rden);
    return a;
}
unsigned f32_grid(const FArgs &a) { return (unsigned)(a.BH * a.tiles * a.splits); }

template <int D>
cudaError_t launch_forward(const CrossPlan &p, const CrossIo &io, cudaStream_t st) {
    const FArgs a = f32_args(kCrossFwd, p, io);
    constexpr int smem = f32_smem<kCrossFwd>();
    const cudaError_t e = smem_opt_in_once<cross_f32_forward<D>>(smem);
    if (e != cudaSuccess) return e;
    ProfScope prof("cross_fwd_f32", st);
    cross_f32_forward<D><<<f32_grid(a), kThreads, smem, st>>>(a);  // the call's first kernel
    return cudaGetLastError();
}
template <int D>
cudaError_t launch_backward(const CrossPlan &p, const CrossIo &io, cudaStream_t st) {
    const FArgs q = f32_args(kCrossDq, p, io), kv = f32_args(kCrossDkv, p, io);
    constexpr int smem = f32_smem<kCrossDkv>();
    const cudaError_t e = smem_opt_in_once<cross_f32_backward<D>>(smem);
    if (e != cudaSuccess) return e;
    ProfScope prof("cross_bwd_f32", st);
    return launch_dependent(cross_f32_backward<D>, dim3(f32_grid(kv) + f32_grid(q)), (unsigned)kThreads, smem, st, q,
                            kv, (int)f32_grid(kv));
}

}  // namespace

cudaError_t launch_cross_f32_forward(const CrossPlan &p, const CrossIo &io, cudaStream_t st) {
    switch (p.d) {
        case 16: return launch_forward<16>(p, io, st);
        case 32: return launch_forward<32>(p, io, st);
        default: return launch_forward<64>(p, io, st);
    }
}
cudaError_t launch_cross_f32_backward(const CrossPlan &p, const CrossIo &io, cudaStream_t st) {
    switch (p.d) {
        case 16: return launch_backward<16>(p, io, st);
        case 32: return launch_backward<32>(p, io, st);
        default: return launch_backward<64>(p, io, st);
    }
}

}  // namespace kata
