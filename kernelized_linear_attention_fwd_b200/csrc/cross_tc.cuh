// Parts of the tensor-core kernel of cross attention (cross_tc.cu): arguments, tensor
// maps, and what reads and writes rows.
#pragma once

#include <cuda_bf16.h>

#include "cross_sched.cuh"
#include "kata_internal.cuh"
#include "sm100.cuh"
#include "tmap.cuh"

namespace kata {

using namespace kata::sm100;

// Place in a ring and the parity of its current round.
struct XRing {
    int i = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int n) {
        if (++i == n) {
            i = 0;
            phase ^= 1;
        }
    }
};

struct XArgs {
    XSched sched;
    int d, stat_stride;
    long long BH;
    __nv_bfloat16 *o0, *o1;  // forward: out; dq: dq; dkv: dv, dk
    float *y, *den;          // forward exports
    float *part, *part_l;    // partial sums of cut items
    XPiece *pieces;          // every CTA's first piece
    const float *delta, *rden;
    int *status;
};

__device__ __forceinline__ uint64_t desc_at(uint64_t d, uint32_t bytes) { return d + (bytes >> 4); }

// Bulk copy of `bytes` (a multiple of 16, both ends 16-byte aligned) into shared memory.
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// Writes 64 accumulated columns of a row (the first d of them) times `scale` as
// bf16, and unrounded to y if given.
__device__ __forceinline__ void store_row(__nv_bfloat16 *dst, float *y, const uint32_t *o, float scale, int d) {
    const uint64_t sc = f32x2_pack(__float_as_uint(scale), __float_as_uint(scale));
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        if (8 * c >= d) break;
        uint64_t p[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) p[x] = f32x2_mul(f32x2_pack(o[8 * c + 2 * x], o[8 * c + 2 * x + 1]), sc);
        *reinterpret_cast<uint4 *>(dst + 8 * c) = make_uint4(f32x2_to_bf16x2(p[0]), f32x2_to_bf16x2(p[1]),
                                                             f32x2_to_bf16x2(p[2]), f32x2_to_bf16x2(p[3]));
        if (y) {
            *reinterpret_cast<float4 *>(y + 8 * c) =
                make_float4(f32x2_lo(p[0]), f32x2_hi(p[0]), f32x2_lo(p[1]), f32x2_hi(p[1]));
            *reinterpret_cast<float4 *>(y + 8 * c + 4) =
                make_float4(f32x2_lo(p[2]), f32x2_hi(p[2]), f32x2_lo(p[3]), f32x2_hi(p[3]));
        }
    }
}

__device__ __forceinline__ void store_part(float *dst, const uint32_t *o, int d) {
#pragma unroll
    for (int c = 0; c < 16; ++c) {
        if (4 * c >= d) break;
        *reinterpret_cast<uint4 *>(dst + 4 * c) = make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
    }
}

// Rows without a visible key, which no unit covers: zeros.  Tile by tile over the
// mode's CTAs, by the n_warps warps of each that call it.
template <int MODE>
__device__ void zero_dead_rows(const XArgs &a, int cta, int warp, int n_warps, int lane) {
    const XSched &sc = a.sched;
    if (!sc.key_lengths) return;
    const int tiles = (sc.rows + kXTile - 1) / kXTile;
    const long long n = a.BH * tiles;
    for (long long x = (long long)cta * n_warps + warp; x < n; x += (long long)sc.grid * n_warps) {
        const int bh = (int)(x / tiles), r0 = (int)(x % tiles) * kXTile;
        const int live = cross_length(sc.key_lengths, bh / sc.Hkv, sc.Tk);
        if (MODE == kCrossDkv ? r0 < live : live > 0) continue;
        const long long row = (long long)bh * sc.rows + r0;
        const int rows = min(kXTile, sc.rows - r0);
        const uint4 z = make_uint4(0u, 0u, 0u, 0u);
        for (int c = lane; c < rows * a.d / 8; c += 32) {
            reinterpret_cast<uint4 *>(a.o0 + row * a.d)[c] = z;
            if (MODE == kCrossDkv) reinterpret_cast<uint4 *>(a.o1 + row * a.d)[c] = z;
            if (MODE == kCrossFwd && a.y) {
                reinterpret_cast<uint4 *>(a.y + row * a.d)[2 * c] = z;
                reinterpret_cast<uint4 *>(a.y + row * a.d)[2 * c + 1] = z;
            }
        }
        if (MODE == kCrossFwd && a.den)
            for (int c = lane; c < rows; c += 32) a.den[row + c] = 0.f;
    }
}

// Arguments and tensor maps (row operands r0, r1, column operands c0, c1) of a mode.
struct XLaunch {
    CUtensorMap maps[4];
    XArgs a;
};
inline cudaError_t x_launch(CrossMode mode, const CrossPlan &p, const CrossIo &io, XLaunch &x) {
    char *ws = static_cast<char *>(io.ws);
    XArgs &a = x.a;
    a = XArgs{};
    a.sched = p.sched[mode];
    a.sched.key_lengths = io.key_lengths;
    a.sched.whole = cross_whole(p.sched[mode], io);
    a.d = p.d;
    a.stat_stride = p.R_pad;
    a.BH = p.BH;
    a.o0 = static_cast<__nv_bfloat16 *>(mode == kCrossFwd ? io.out : mode == kCrossDq ? io.dq : io.dv);
    a.o1 = static_cast<__nv_bfloat16 *>(io.dk);
    a.y = io.y;
    a.den = io.den;
    a.part = reinterpret_cast<float *>(ws + p.ws_part[mode]);
    a.part_l = reinterpret_cast<float *>(ws + p.ws_part_l);
    a.pieces = reinterpret_cast<XPiece *>(ws + p.ws_pieces[mode]);
    a.delta = reinterpret_cast<const float *>(ws + p.ws_delta);
    a.rden = reinterpret_cast<const float *>(ws + p.ws_rden);
    a.status = device_status_ptr();
    if (!a.status) return cudaErrorUnknown;
    const void *r0 = mode == kCrossDkv ? io.k : io.q, *r1 = mode == kCrossDkv ? io.v : io.dout;
    const void *c0 = mode == kCrossDkv ? io.q : io.k, *c1 = mode == kCrossDkv ? io.dout : io.v;
    if (mode == kCrossFwd) r1 = r0;
    const void *base[4] = {r0, r1, c0, c1};
    for (int m = 0; m < 4; ++m) {
        const uint64_t n = m < 2 ? a.sched.rows : a.sched.cols, w = 2 * (uint64_t)p.d;
        const uint64_t dims[3] = {(uint64_t)p.d, n, (uint64_t)p.BH}, strides[2] = {w, w * n};
        const uint32_t box[3] = {64, m < 2 ? (uint32_t)kXTile : 64u, 1};
        if (!make_tmap_bf16(&x.maps[m], base[m], 3, dims, strides, box)) return cudaErrorInvalidValue;
    }
    return cudaSuccess;
}

}  // namespace kata
