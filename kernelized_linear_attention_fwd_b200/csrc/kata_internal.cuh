// Internal declarations shared by the CUDA translation units of libkata.
// Not part of the public ABI (that is include/kata.h).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <initializer_list>
#include <mutex>

#include "../../include/kata.h"

namespace kata {

// ---------------------------------------------------------------------------
// Packed symmetric feature rows.
//
// phi(x) = vec(x x^T) has dk^2 entries but only dk(dk+1)/2 distinct ones:
// (q.k)^2 = sum_i q_i^2 k_i^2 + 2 sum_{i<j} q_i q_j k_i k_j.  The state is kept
// on the half triangle i <= j (row r enumerates (i, j) with i outer), storing
// the plain sums sum_s k_si k_sj v_s; the weight c_ij (1 on the diagonal, 2
// off it) is applied on the query side at readout.
// ---------------------------------------------------------------------------
__host__ __device__ constexpr int packed_rows(int d) { return d * (d + 1) / 2; }

__host__ __device__ inline int packed_row_start(int d, int i) { return i * d - (i * (i - 1)) / 2; }

__host__ __device__ inline void packed_row_ij(int d, int r, int &i, int &j) {
    int a = 0;
    while (r >= d - a) {
        r -= d - a;
        ++a;
    }
    i = a;
    j = a + r;
}

// KATA-Mg with G factors of P = DK / G coordinates each: only pairs (i, j)
// inside one factor carry state.  The packed rows are the G factors' own
// packed rows one after the other: row r = f * Rp + r', Rp = P (P + 1) / 2,
// is the pair (f P + i', f P + j') of the factor's row r' = (i', j').  G = 1
// is the layout above.
__host__ __device__ constexpr int packed_rows_g(int d, int G) { return G * packed_rows(d / G); }

__host__ __device__ inline void packed_row_ij_g(int d, int G, int r, int &i, int &j) {
    const int P = d / G, Rp = packed_rows(P), f = r / Rp;
    packed_row_ij(P, r - f * Rp, i, j);
    i += f * P;
    j += f * P;
}

// Packed row of the pair (i, j), i <= j, both in one factor.
__host__ __device__ inline int packed_row_index_g(int d, int G, int i, int j) {
    const int P = d / G, f = i / P;
    return f * packed_rows(P) + packed_row_start(P, i - f * P) + (j - i);
}

// ---------------------------------------------------------------------------
// Forward plan: segment length, number of segments, workspace layout.
// ---------------------------------------------------------------------------
// kTensorCore: bf16 heads of d = 64, and of d = 16 or 32 read as 64 by the
// tensor maps (TMA fills the columns past d with zeros, which add nothing to
// any product or sum; the output store writes only the first d columns) and
// run on the two-factor layout (Plan::tc_g).
enum class Path : int { kSimt = 0, kTensorCore = 1 };

struct Plan {
    int B, H, T, dk, dv, C;
    kata_dtype dtype;
    long long BH;
    int L;      // segment length (tokens), a multiple of C and of 128; T in the quadratic plan
    int n_seg;  // ceil(T / L)
    int R;      // packed feature rows (of d = 64 on the tensor-core path)
    int g = 1;  // rank-one PSD factors per head (KATA-Mg; 1 = the single factor)
    // Factors of the tensor-core layout the kernels run: g, except that a
    // single-factor head of d <= 32 runs the two-factor layout (its
    // coordinates 32-63, read as zeros, form a second factor that contributes
    // nothing), which holds its state in 1152 rows instead of 2176.
    int tc_g = 1;
    Path path;
    // workspace (bytes from the base, all 256-byte aligned)
    size_t ws_seg_state;  // fp32 per-segment states, exclusive prefix after the scan
    size_t ws_total;      // fp32 total state (packed), when needed
    size_t ws_extra;      // path-specific
    size_t ws_aux;        // path-specific (unused)
    size_t ws_bytes;
};

// Fills `p`; returns KATA_OK or the error the forward must return.  small_tc:
// bf16 heads of d < 64 run the tensor-core kernels (read as 64 by the tensor
// maps); without it (KATA-Mg, whose factors split the head at d / 2) they
// take the fp32 CUDA-core path.
kata_status make_plan(int B, int H, int T, int dk, int dv, int C, kata_dtype dtype, Plan &p,
                      bool small_tc = true);
// The plan of the quadratic form: one segment of T tokens, no workspace.
kata_status make_quadratic_plan(int B, int H, int T, int dk, int dv, kata_dtype dtype, Plan &p);

// Device address of the status word that kernels set when an on-device check
// fails (one per device; resolved on first use with that device current).
int *device_status_ptr();

// Argument checks shared by the entry points.
inline size_t align_up(size_t x) { return (x + 255) / 256 * 256; }
inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool overlaps(const void *a, size_t na, const void *b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

// True when every non-null pointer is memory of the current device (or
// managed memory).  Host memory and another device's memory are rejected, so
// a call given them returns an error instead of launching kernels that would
// fault.  Checked after every other host-side check.
bool device_ptrs_ok(std::initializer_list<const void *> ptrs);

// Kernel timing (include/kata_profile.h): no-ops unless profiling is enabled.
int prof_begin(const char *name, cudaStream_t st);
void prof_end(int ev, cudaStream_t st);

struct ProfScope {
    int ev;
    cudaStream_t st;
    ProfScope(const char *name, cudaStream_t s) : ev(prof_begin(name, s)), st(s) {}
    ~ProfScope() { prof_end(ev, st); }
};

// Opt-in dynamic shared memory of a kernel, set once per device: the
// attribute lasts for the life of the context, and setting it on every launch
// costs host time that small launches cannot hide.
// The per-device record is guarded, so host threads may make first calls at
// the same time.
template <auto Kernel>
cudaError_t smem_opt_in_once(int bytes) {
    static std::mutex mu;
    static int set_bytes[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lk(mu);
    if (dev >= 0 && dev < 64 && set_bytes[dev] == bytes) return cudaSuccess;
    e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev >= 0 && dev < 64) set_bytes[dev] = bytes;
    return e;
}

// Launches `kernel` as a programmatic dependent of the call's previous kernel: its
// launch overlaps that kernel's end, and it must execute griddepcontrol.wait before
// it reads or writes what earlier work touches.
template <typename... Exp, typename... Act>
cudaError_t launch_dependent(void (*kernel)(Exp...), dim3 grid, unsigned block, int smem, cudaStream_t st,
                             Act... args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Exp>(args)...);
}

// Element loads as fp32.
__device__ __forceinline__ float load_f32(const float *p, long long i) { return p[i]; }
__device__ __forceinline__ float load_f32(const __nv_bfloat16 *p, long long i) {
    return __bfloat162float(p[i]);
}
__device__ __forceinline__ void store_out(float *p, long long i, float x) { p[i] = x; }
__device__ __forceinline__ void store_out(__nv_bfloat16 *p, long long i, float x) {
    p[i] = __float2bfloat16_rn(x);
}

// Initial state of a forward: the sum of n dense states, S [B, H, d*d, d]
// and Z [B, H, d, d] fp32 (d = the plan's dk); input m starts s_stride
// (z_stride) floats after input m - 1.  n = 0: the forward starts from the
// empty state.
struct InitState {
    const float *s = nullptr;
    const float *z = nullptr;
    int n = 0;
    long long s_stride = 0, z_stride = 0;
};

// Launchers (return cudaSuccess or the launch error).  out == nullptr skips
// the readout (state only: state_out and z_out are then required).
cudaError_t launch_simt_forward(const Plan &p, const void *q, const void *k, const void *v,
                                void *out, float *state_out, float *z_out, const InitState &init,
                                void *ws, cudaStream_t st);
namespace tc {
// Tensor-core path (bf16, d = dv in {16, 32, 64}, computed as 64): workspace
// layout and launcher.
// reuse_seg: the workspace already holds every segment's state, written by a
// state-only launch for the same keys, values and sizes; skip building them.
void plan_tc_workspace(Plan &p);
cudaError_t launch_tc_forward(const Plan &p, const void *q, const void *k, const void *v,
                              void *out, float *state_out, float *z_out, const InitState &init,
                              void *ws, cudaStream_t st, bool reuse_seg = false);
// Streaming multiprocessors of the current device (cached).
int num_sms();
}  // namespace tc

// Streaming multiprocessors that launch and workspace plans are made for: a
// constant, so that a workspace's size depends on the call's arguments only.
constexpr int kPlanSms = 148;

// Head norm with rotation (norm_rotate.cu); index 0 the queries, 1 the keys
// (H[1] = 0: no keys).
struct NormRotate {
    bool backward = false, interleaved = false;
    int B, T, d, n_rot;
    int H[2];
    kata_dtype dtype;
    float eps;
    const void *x[2];
    long long xs[2][3];  // strides of batch, token, head (elements)
    void *y[2];
    const float *w[2];
    const float *inv_freq;
    const long long *positions;
    long long pos_stride;
    const void *gy[2];
    void *dx[2];
    long long ds[2][3];
    float *dw[2];
    void *ws;  // backward: grid blocks x 2 d floats
};
dim3 norm_rotate_grid(const NormRotate &p);
cudaError_t launch_norm_rotate(const NormRotate &p, cudaStream_t st);

// Cross attention (cross_tc.cu for bf16, cross_f32.cu for fp32, cross_few.cu for few
// rows).  The query
// heads that share a key head are consecutive in memory, so they are the rows of
// one problem: BH = B Hkv problems of R = (H / Hkv) Tq rows and Tk keys.
enum CrossMode : int { kCrossFwd = 0, kCrossDq = 1, kCrossDkv = 2 };
// Work of one mode on the tensor cores (cross_sched.cuh).
struct XSched {
    int B, Hkv, rows, cols, Tk;
    const int *key_lengths;
    int grid;
    int min_share;  // fewest units a CTA takes
    int whole;      // cut at item boundaries only: 2: always, 1: if the lengths are equal
    int slot_rows;  // rows of a cut piece's partial sums
};
struct CrossPlan {
    int B, H, Hkv, Tq, Tk, d;
    kata_dtype dtype;
    long long BH;
    int R;             // rows per problem
    int R_pad;         // R rounded up to 128: row stride of the statistics
    bool few;          // forward by launch_cross_few
    bool split[3];      // bf16, per CrossMode, in training: operands as two bf16 numbers
    int splits[3];     // fp32, per CrossMode: pieces of the summed axis (1: no join)
    XSched sched[3];   // bf16, per CrossMode, and few
    bool together;     // bf16: dq and dkv in one launch
    // workspace (bytes)
    size_t ws_part[3];  // partial sums of each mode
    size_t ws_part_l;   // forward: partial denominators
    size_t ws_pieces[3];  // bf16: every CTA's first piece
    size_t ws_delta;    // backward: [BH][R_pad] -(dy.y), then [BH][R_pad] 1 / den
    size_t ws_rden;
    size_t ws_fwd_bytes, ws_bwd_bytes;
};
struct CrossIo {
    const void *q, *k, *v, *dout;
    const int *key_lengths;  // [B] or null
    void *out;
    float *y, *den;          // forward: nullable exports; backward: inputs
    void *dq, *dk, *dv;
    void *ws;
};
inline int cross_whole(const XSched &s, const CrossIo &io) { return s.whole == 2 || (s.whole && !io.key_lengths); }
cudaError_t launch_cross_forward(const CrossPlan &p, const CrossIo &io, cudaStream_t st);
cudaError_t launch_cross_backward(const CrossPlan &p, const CrossIo &io, cudaStream_t st);
// One mode's main kernel: forward of at most kFewRows (bf16: kFewRowsBf16) rows per key
// head; others in bf16 and in fp32.
constexpr int kSplitRows = 32;  // bf16: up to so many rows or keys, operands as two bf16 numbers
constexpr int kFewRows = 4, kFewRowsBf16 = 16;
// CTAs per SM of those kernels for this many rows (64, 80, 128 registers a thread).
__host__ __device__ constexpr int few_per_sm(int rows) { return rows == 1 ? 4 : rows == 2 ? 3 : 2; }
cudaError_t launch_cross_few(const CrossPlan &p, const CrossIo &io, cudaStream_t st);
cudaError_t launch_cross_tc_forward(const CrossPlan &p, const CrossIo &io, cudaStream_t st);
cudaError_t launch_cross_tc_backward(const CrossPlan &p, const CrossIo &io, cudaStream_t st);  // dq and dkv
cudaError_t launch_cross_f32_forward(const CrossPlan &p, const CrossIo &io, cudaStream_t st);
cudaError_t launch_cross_f32_backward(const CrossPlan &p, const CrossIo &io, cudaStream_t st);  // dq and dkv
// Rows of a CTA and columns of a block of the fp32 kernels.
constexpr int kF32Tile = 64;

// Keys that sequence b may attend to: its length, within [0, Tk].
__device__ __forceinline__ int cross_length(const int *key_lengths, int b, int Tk) {
    return key_lengths ? min(max(__ldg(key_lengths + b), 0), Tk) : Tk;
}
// 1 / den, and 0 for a row without weight.  Sums below the smallest normal number count as
// none: their reciprocals overflow, and one such query would make every key's gradient
// infinite or NaN.
__device__ __forceinline__ float cross_recip(float den) { return den < 1.17549435e-38f ? 0.f : 1.f / den; }

// Decode step on the dense (d^2 rows) or packed (d(d+1)/2 rows) state layout.
cudaError_t launch_decode(int B, int H, int dk, int dv, kata_dtype dtype, const void *q,
                          const void *k, const void *v, void *out, float *state, float *z,
                          bool packed, cudaStream_t st);
// The decode step of KATA-Mg with g factors on the dense layout (g = 1: the
// dense step above).
cudaError_t launch_decode_mg(int B, int H, int dk, int g, kata_dtype dtype, const void *q,
                             const void *k, const void *v, void *out, float *state, float *z,
                             cudaStream_t st);
// Dense <-> packed state conversion (pack: dense -> packed).
cudaError_t launch_state_convert(bool pack, int B, int H, int dk, const float *src_s,
                                 const float *src_z, float *dst_s, float *dst_z, cudaStream_t st);

}  // namespace kata
