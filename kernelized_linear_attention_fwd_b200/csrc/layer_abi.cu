// C ABI of the head norm with rotation and of cross attention: argument checks,
// plans and dispatch.  Declarations and the contract: include/kata.h.
#include <math.h>

#include "cross_sched.cuh"
#include "kata_internal.cuh"

namespace kata {
namespace {

// ---------------------------------------------------------------------------
// Head norm with rotation
// ---------------------------------------------------------------------------
size_t norm_workspace_bytes(const NormRotate &p) {
    const dim3 g = norm_rotate_grid(p);
    return align_up((size_t)g.x * g.y * 2 * p.d * sizeof(float));
}

// Sizes; fills what the grid and the workspace depend on.
kata_status norm_sizes(int B, int T, int Hq, int Hk, int d, kata_dtype dtype, NormRotate &p) {
    if (B < 1 || T < 1 || Hq < 1 || Hk < 0 || d < 1) return KATA_ERR_INVALID_ARG;
    if (dtype != KATA_F32 && dtype != KATA_BF16) return KATA_ERR_UNSUPPORTED;
    if (d != 16 && d != 32 && d != 64) return KATA_ERR_UNSUPPORTED;
    // a warp's step past the last token, and a block row's past the last head (of at most 444
    // block rows of 64 heads), fit
    const int most = 0x7fffffff - (1 << 17);
    if (B > most || T > most || Hq > most || Hk > most) return KATA_ERR_UNSUPPORTED;
    if ((long long)B * T > (1LL << 40) / ((long long)Hq + Hk)) return KATA_ERR_UNSUPPORTED;
    p.B = B;
    p.T = T;
    p.H[0] = Hq;
    p.H[1] = Hk;
    p.d = d;
    p.dtype = dtype;
    return KATA_OK;
}

// Strides of a [B, T, H, d] tensor: non-negative, 16-byte multiples along axes
// longer than 1 (others are not used and kept as 0), spans within 2^46 elements.
bool norm_strides(const NormRotate &p, int m, const int64_t *s, long long (&out)[3]) {
    const long long n[3] = {p.B, p.T, p.H[m]};
    const int per16 = p.dtype == KATA_BF16 ? 8 : 4;
    if (!s) return false;
    for (int i = 0; i < 3; ++i) {
        out[i] = 0;
        if (n[i] == 1) continue;
        if (s[i] < 0 || s[i] % per16 != 0) return false;
        if (s[i] > (1LL << 46) / n[i]) return false;
        out[i] = s[i];
    }
    return true;
}

size_t norm_span(const NormRotate &p, int m, const long long (&s)[3]) {
    const long long e = (p.B - 1) * s[0] + (p.T - 1) * s[1] + (p.H[m] - 1) * s[2] + p.d;
    return (size_t)e * (p.dtype == KATA_BF16 ? 2 : 4);
}

// A strided box of rows, its axes by falling stride.
struct Rows {
    long long s[3], n[3];
    int axes = 0;
    long long d;
    // elements from the first to behind the last, of the axes from `i` on
    long long span(int i) const {
        long long e = d;
        for (; i < axes; ++i) e += (n[i] - 1) * s[i];
        return e;
    }
};
Rows rows_of(const NormRotate &p, int m, const long long (&s)[3]) {
    const long long n[3] = {p.B, p.T, p.H[m]};
    Rows r;
    r.d = p.d;
    for (int i = 0; i < 3; ++i) {
        if (n[i] == 1) continue;
        int k = r.axes++;
        for (; k > 0 && r.s[k - 1] < s[i]; --k) {
            r.s[k] = r.s[k - 1];
            r.n[k] = r.n[k - 1];
        }
        r.s[k] = s[i];
        r.n[k] = n[i];
    }
    return r;
}

// No two rows share memory: every axis steps over all that the shorter ones cover.
bool rows_disjoint(const Rows &r) {
    for (int i = 0; i < r.axes; ++i)
        if (r.s[i] < r.span(i + 1)) return false;
    return true;
}

// No row of a (axes from i on) meets one of b (from j on), which starts `off` elements
// behind it.  The longest step moves one against the other; where it belongs to both, only
// the difference m of their places on it counts: off + m step.  Each place at which the
// rest of the two could meet is looked into.  With rows that do not overlap themselves
// there are two at most on a shared step; a box that meets more of the other's steps is
// taken for overlapping.
bool boxes_apart(const Rows &a, int i, const Rows &b, int j, long long off) {
    if (off >= a.span(i) || -off >= b.span(j)) return true;
    if (i == a.axes && j == b.axes) return false;
    const long long sa = i < a.axes ? a.s[i] : 0, sb = j < b.axes ? b.s[j] : 0, step = sa > sb ? sa : sb;
    if (step < 1) return false;
    const int ia = i + (sa == step), jb = j + (sb == step);
    // they can meet for -eb < off + m step < ea
    const long long ea = a.span(ia), eb = b.span(jb);
    auto floor_div = [](long long x, long long y) { return x >= 0 ? x / y : -((y - 1 - x) / y); };
    long long lo = floor_div(-eb - off, step) + 1, hi = floor_div(ea - 1 - off, step);
    const long long m0 = ia > i ? 1 - a.n[i] : 0, m1 = jb > j ? b.n[j] - 1 : 0;
    if (lo < m0) lo = m0;
    if (hi > m1) hi = m1;
    if (hi - lo > 1) return false;
    for (long long m = lo; m <= hi; ++m)
        if (!boxes_apart(a, ia, b, jb, off + m * step)) return false;
    return true;
}

// dq and dk (each without overlap of its own rows) share no row: in separate buffers, or
// slices of one in whatever order of batch, tokens and heads.
bool slices_disjoint(const NormRotate &p) {
    const long long es = p.dtype == KATA_BF16 ? 2 : 4;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(p.dx[0]), a1 = reinterpret_cast<uintptr_t>(p.dx[1]);
    const int lo = a0 <= a1 ? 0 : 1;
    const uintptr_t gap = lo == 0 ? a1 - a0 : a0 - a1;
    if (gap >= norm_span(p, lo, p.ds[lo])) return true;
    return boxes_apart(rows_of(p, lo, p.ds[lo]), 0, rows_of(p, 1 - lo, p.ds[1 - lo]), 0, (long long)gap / es);
}

// Checks shared by both directions; y of the backward pass are the gradients.
kata_status norm_common(NormRotate &p, const void *q, const void *k, const float *q_weight, const float *k_weight,
                        const float *inv_freq, const int64_t *positions, int n_rot, const int64_t *q_strides,
                        const int64_t *k_strides, int64_t pos_stride, float eps, int interleaved) {
    if (n_rot < 0 || n_rot > p.d / 2) return KATA_ERR_INVALID_ARG;
    if (!interleaved && n_rot % 4 != 0) return KATA_ERR_UNSUPPORTED;
    if (!(eps > 0.f) || isinf(eps)) return KATA_ERR_INVALID_ARG;
    if (!q || (p.H[1] > 0) != (k != nullptr)) return KATA_ERR_INVALID_ARG;
    if (n_rot > 0 && !inv_freq) return KATA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(q_weight) || !aligned16(k_weight) || !aligned16(inv_freq))
        return KATA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(positions) & 7u) != 0) return KATA_ERR_INVALID_ARG;
    if (positions && (pos_stride < 0 || pos_stride > (1LL << 40))) return KATA_ERR_INVALID_ARG;
    if (!norm_strides(p, 0, q_strides, p.xs[0])) return KATA_ERR_INVALID_ARG;
    for (long long &s : p.xs[1]) s = 0;
    if (k && !norm_strides(p, 1, k_strides, p.xs[1])) return KATA_ERR_INVALID_ARG;
    p.interleaved = interleaved != 0;
    p.n_rot = n_rot;
    p.eps = eps;
    p.x[0] = q;
    p.x[1] = k;
    p.w[0] = q_weight;
    p.w[1] = k_weight;
    p.inv_freq = inv_freq;
    p.positions = reinterpret_cast<const long long *>(positions);
    p.pos_stride = pos_stride;
    for (int m = 0; m < 2; ++m) {
        p.y[m] = p.dx[m] = nullptr;
        p.gy[m] = nullptr;
        p.dw[m] = nullptr;
        for (long long &s : p.ds[m]) s = 0;
    }
    p.ws = nullptr;
    return KATA_OK;
}

size_t dense_bytes(const NormRotate &p, int m) {
    return (size_t)p.B * p.T * p.H[m] * p.d * (p.dtype == KATA_BF16 ? 2 : 4);
}

// Whether [o, o + n) touches any of the call's inputs.
bool hits_inputs(const NormRotate &p, const void *o, size_t n) {
    for (int m = 0; m < 2; ++m) {
        if (p.x[m] && overlaps(o, n, p.x[m], norm_span(p, m, p.xs[m]))) return true;
        if (p.w[m] && overlaps(o, n, p.w[m], (size_t)p.d * 4)) return true;
        if (p.gy[m] && overlaps(o, n, p.gy[m], dense_bytes(p, m))) return true;
    }
    if (p.n_rot > 0 && overlaps(o, n, p.inv_freq, (size_t)p.n_rot * 4)) return true;
    return p.positions && overlaps(o, n, p.positions, 8 * ((size_t)(p.B - 1) * p.pos_stride + p.T));
}

// ---------------------------------------------------------------------------
// Cross attention
// ---------------------------------------------------------------------------
// fp32: pieces of the summed axis, none empty: 1 when the items fill the SMs, else the
// number that gives the busiest SM the least to do, counting a block as 1, what a CTA
// does besides its blocks (loading its rows, storing its sums) as 1, and two CTAs that
// share an SM as 1.3 times one (4096 queries and keys, one head: one CTA an SM 111 us,
// two 85).
int cross_splits(long long items, long long blocks) {
    if (items >= 2 * kPlanSms) return 1;
    long long best = 1, best_cost = 0;
    for (long long piece = blocks; piece >= 1; piece = piece > 64 ? piece - piece / 16 : piece - 1) {
        const long long s = (blocks + piece - 1) / piece;
        const long long n = (items * s + kPlanSms - 1) / kPlanSms, cost = (n / 2 * 13 + n % 2 * 10) * (piece + 1);
        if (best_cost == 0 || cost < best_cost) {
            best = s;
            best_cost = cost;
        }
    }
    return (int)best;
}

// The tensor cores' schedule of one mode.  Items are cut unless that gains little:
// - whole = 2: items at most 4 units long (below that a CTA's start and the join cost
//   more than the steps saved), or 16 and more of them per SM;
// - whole = 1: equal lengths and whole items, dealt evenly, that leave the busiest SM at
//   most 3% above the average.  (Lengths that differ put stretches of whole items up
//   to an item apart.)
bool cross_sched(const CrossPlan &p, CrossMode m, int rows, int cols, int sms, XSched &s) {
    const long long tiles = (rows + kXTile - 1) / kXTile, blocks = (cols + kXCols - 1) / kXCols;
    const long long items = p.BH * tiles;
    if (items >= (1LL << 31) || items > (1LL << 62) / blocks) return false;
    const long long units = items * blocks;
    s.B = p.B;
    s.Hkv = p.Hkv;
    s.rows = rows;
    s.cols = cols;
    s.Tk = p.Tk;
    s.key_lengths = nullptr;
    // CTAs that run at a time, and the fewest units worth one
    const int full = m == kCrossFwd && p.few ? few_per_sm(p.R) * kPlanSms : sms, least = m == kCrossFwd && p.few ? 2 : 4;
    const long long rounds = (items + full - 1) / full;
    const bool tiny = items < full && blocks <= least;
    s.whole = tiny || items >= 16 * full ? 2 : rounds * full * 100 <= items * 103 ? 1 : 0;
    s.min_share = s.whole == 2 ? 1 : least;
    const long long most = s.whole == 2 ? items : (units + least - 1) / least;
    s.grid = (int)(most < full ? most : full);
    const int most_rows = m == kCrossDkv ? 256 : 128;  // dkv: dv's 128 rows and dk's
    s.slot_rows = m != kCrossDkv && rows < most_rows ? rows : most_rows;
    return true;
}

kata_status cross_plan(int B, int H, int Hkv, int Tq, int Tk, int d, kata_dtype dtype, CrossPlan &p) {
    if (B < 1 || H < 1 || Hkv < 1 || Tq < 1 || Tk < 1 || d < 1 || H % Hkv != 0) return KATA_ERR_INVALID_ARG;
    if (dtype != KATA_F32 && dtype != KATA_BF16) return KATA_ERR_UNSUPPORTED;
    if (d != 16 && d != 32 && d != 64) return KATA_ERR_UNSUPPORTED;
    const long long rows = (long long)(H / Hkv) * Tq, most = 0x7fffffffLL - 256;
    if (rows >= most || Tk >= most) return KATA_ERR_UNSUPPORTED;
    p.B = B;
    p.H = H;
    p.Hkv = Hkv;
    p.Tq = Tq;
    p.Tk = Tk;
    p.d = d;
    p.dtype = dtype;
    p.BH = (long long)B * Hkv;
    if (p.BH > (1LL << 40) / rows || p.BH > (1LL << 40) / Tk) return KATA_ERR_UNSUPPORTED;
    p.R = (int)rows;
    p.R_pad = (p.R + 127) / 128 * 128;
    const size_t stat = align_up((size_t)p.BH * p.R_pad * 4);
    p.ws_delta = 0;
    p.ws_rden = stat;
    size_t off = 2 * stat;
    p.few = p.R <= (dtype == KATA_BF16 ? kFewRowsBf16 : kFewRows);
    // dq and dkv in one launch while each would take an SM less than some 32 steps; the
    // SMs go by the steps' times, about 1 : 1.4
    const long long rt = (p.R + kXTile - 1) / kXTile, kt = (Tk + kXTile - 1) / kXTile;
    p.together = dtype == KATA_BF16 && p.BH < kPlanSms * 32 / rt / kt;
    const int sms_q = kPlanSms * 5 / 12;
    // Where the error of a training step's rounded weights shows (cross_tc.cu): the
    // forward of heads up to 32 or of few keys (256 keys: 57 us, 66 so, for 3 sequences of
    // 16 heads and 4000 queries), dq of heads of 16, everything if few rows meet in a
    // sum (16 rows on 4000 keys, 48 heads: backward 79 us, 89 so).
    const bool few_terms = p.R <= kSplitRows || Tk <= kSplitRows;
    p.split[kCrossFwd] = d <= 32 || Tk <= 256 || few_terms;
    p.split[kCrossDq] = d == 16 || few_terms;
    p.split[kCrossDkv] = few_terms;
    for (const CrossMode m : {kCrossFwd, kCrossDq, kCrossDkv}) {
        const long long n = m == kCrossDkv ? Tk : p.R, c = m == kCrossDkv ? p.R : Tk;
        size_t part_rows = 0;  // rows of partial sums
        const bool cut = dtype == KATA_BF16 || (m == kCrossFwd && p.few);
        if (cut) {
            const int sms = !p.together || m == kCrossFwd ? kPlanSms : m == kCrossDq ? sms_q : kPlanSms - sms_q;
            if (!cross_sched(p, m, (int)n, (int)c, sms, p.sched[m])) return KATA_ERR_UNSUPPORTED;
            part_rows = p.sched[m].whole == 2 ? 0 : (size_t)p.sched[m].grid * 2 * p.sched[m].slot_rows;
            p.splits[m] = 1;
        } else {
            const long long items = p.BH * ((n + kF32Tile - 1) / kF32Tile);
            if (items >= most / 2) return KATA_ERR_UNSUPPORTED;  // dq's and dkv's share a grid
            p.splits[m] = cross_splits(items, (c + kF32Tile - 1) / kF32Tile);
            if (p.splits[m] > 1) part_rows = (size_t)p.splits[m] * p.BH * n * (m == kCrossDkv ? 2 : 1);
        }
        const size_t part = align_up(part_rows * d * 4);
        const size_t pieces = cut && part ? align_up(p.sched[m].grid * sizeof(XPiece)) : 0;
        if (m == kCrossFwd) {
            p.ws_part[m] = 0;
            p.ws_part_l = part;
            p.ws_pieces[m] = part + align_up(part_rows * 4);
            p.ws_fwd_bytes = p.ws_pieces[m] + pieces;
        } else {
            p.ws_part[m] = off;
            p.ws_pieces[m] = off + part;
            off += part + pieces;
        }
    }
    p.ws_bwd_bytes = off;
    return KATA_OK;
}

kata_status cross_workspace(size_t need, const void *ws, size_t bytes) {
    if (need == 0) return KATA_OK;
    if (!ws || bytes < need || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return KATA_ERR_WORKSPACE;
    return KATA_OK;
}

// A range of memory, for the overlap checks.
struct Range {
    const void *p;
    size_t n;
};
// Every output present lies apart from the inputs and from the other outputs.
bool apart(std::initializer_list<Range> outs, std::initializer_list<Range> ins) {
    for (const Range &o : outs) {
        if (!o.p) continue;
        for (const Range &i : ins)
            if (i.p && overlaps(o.p, o.n, i.p, i.n)) return false;
        for (const Range &x : outs)
            if (&x != &o && x.p && overlaps(o.p, o.n, x.p, x.n)) return false;
    }
    return true;
}

}  // namespace
}  // namespace kata

using namespace kata;

extern "C" {

kata_status kata_qk_norm_rotate(const void *q, const void *k, void *q_out, void *k_out, const float *q_weight,
                                const float *k_weight, const float *inv_freq, const int64_t *positions, int B,
                                int T, int Hq, int Hk, int d, int n_rot, const int64_t *q_strides,
                                const int64_t *k_strides, int64_t pos_stride, float eps, int interleaved,
                                kata_dtype dtype, kata_stream_t stream) {
    NormRotate p;
    kata_status s = norm_sizes(B, T, Hq, Hk, d, dtype, p);
    if (s != KATA_OK) return s;
    s = norm_common(p, q, k, q_weight, k_weight, inv_freq, positions, n_rot, q_strides, k_strides, pos_stride, eps,
                    interleaved);
    if (s != KATA_OK) return s;
    if (!q_out || (k != nullptr) != (k_out != nullptr) || !aligned16(q_out) || !aligned16(k_out))
        return KATA_ERR_INVALID_ARG;
    p.y[0] = q_out;
    p.y[1] = k_out;
    if (hits_inputs(p, q_out, dense_bytes(p, 0)) || (k && hits_inputs(p, k_out, dense_bytes(p, 1))))
        return KATA_ERR_INVALID_ARG;
    if (k && overlaps(q_out, dense_bytes(p, 0), k_out, dense_bytes(p, 1))) return KATA_ERR_INVALID_ARG;
    if (!device_ptrs_ok({q, k, q_out, k_out, q_weight, k_weight, n_rot ? inv_freq : nullptr, positions}))
        return KATA_ERR_INVALID_ARG;
    return launch_norm_rotate(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? KATA_OK : KATA_ERR_CUDA;
}

size_t kata_qk_norm_rotate_backward_workspace_bytes(int B, int T, int Hq, int Hk, int d) {
    NormRotate p;
    if (norm_sizes(B, T, Hq, Hk, d, KATA_F32, p) != KATA_OK) return 0;
    p.backward = true;
    return norm_workspace_bytes(p);
}

kata_status kata_qk_norm_rotate_backward(const void *dq_out, const void *dk_out, const void *q, const void *k,
                                         const float *q_weight, const float *k_weight, const float *inv_freq,
                                         const int64_t *positions, void *dq, void *dk, float *dq_weight,
                                         float *dk_weight, int B, int T, int Hq, int Hk, int d, int n_rot,
                                         const int64_t *q_strides, const int64_t *k_strides,
                                         const int64_t *dq_strides, const int64_t *dk_strides, int64_t pos_stride,
                                         float eps, int interleaved, kata_dtype dtype, void *workspace,
                                         size_t workspace_bytes, kata_stream_t stream) {
    NormRotate p;
    kata_status s = norm_sizes(B, T, Hq, Hk, d, dtype, p);
    if (s != KATA_OK) return s;
    p.backward = true;
    s = norm_common(p, q, k, q_weight, k_weight, inv_freq, positions, n_rot, q_strides, k_strides, pos_stride, eps,
                    interleaved);
    if (s != KATA_OK) return s;
    const void *gy[2] = {dq_out, dk_out};
    void *dx[2] = {dq, dk};
    float *dw[2] = {dq_weight, dk_weight};
    const int64_t *ds[2] = {dq_strides, dk_strides};
    for (int m = 0; m < 2; ++m) {
        if (p.x[m] ? !gy[m] || !dx[m] : gy[m] || dx[m] || dw[m]) return KATA_ERR_INVALID_ARG;
        if (!aligned16(gy[m]) || !aligned16(dx[m]) || !aligned16(dw[m])) return KATA_ERR_INVALID_ARG;
        p.gy[m] = gy[m];
        p.dx[m] = dx[m];
        p.dw[m] = dw[m];
        if (p.x[m] && (!norm_strides(p, m, ds[m], p.ds[m]) || !rows_disjoint(rows_of(p, m, p.ds[m]))))
            return KATA_ERR_INVALID_ARG;
    }
    for (int m = 0; m < 2; ++m) {
        if (!p.x[m]) continue;
        const size_t n = norm_span(p, m, p.ds[m]);
        if (hits_inputs(p, p.dx[m], n)) return KATA_ERR_INVALID_ARG;
        for (int o = 0; o < 2; ++o) {
            if (!p.dw[o]) continue;
            if (overlaps(p.dw[o], (size_t)d * 4, p.dx[m], n)) return KATA_ERR_INVALID_ARG;
        }
        if (p.dw[m] && hits_inputs(p, p.dw[m], (size_t)d * 4)) return KATA_ERR_INVALID_ARG;
    }
    if (p.x[1] && !slices_disjoint(p)) return KATA_ERR_INVALID_ARG;
    if (p.dw[0] && p.dw[1] && overlaps(p.dw[0], (size_t)d * 4, p.dw[1], (size_t)d * 4)) return KATA_ERR_INVALID_ARG;
    s = cross_workspace(norm_workspace_bytes(p), workspace, workspace_bytes);
    if (s != KATA_OK) return s;
    p.ws = workspace;
    if (!device_ptrs_ok({q, k, dq_out, dk_out, dq, dk, dq_weight, dk_weight, q_weight, k_weight,
                         n_rot ? inv_freq : nullptr, positions, workspace}))
        return KATA_ERR_INVALID_ARG;
    return launch_norm_rotate(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? KATA_OK : KATA_ERR_CUDA;
}

size_t kata_cross_forward_workspace_bytes(int B, int H, int Hkv, int Tq, int Tk, int d, kata_dtype dtype) {
    CrossPlan p;
    return cross_plan(B, H, Hkv, Tq, Tk, d, dtype, p) == KATA_OK ? p.ws_fwd_bytes : 0;
}

kata_status kata_cross_forward(const void *q, const void *k, const void *v, const int32_t *key_lengths, void *out,
                               int B, int H, int Hkv, int Tq, int Tk, int d, kata_dtype dtype, float *y_out,
                               float *den_out, void *workspace, size_t workspace_bytes, kata_stream_t stream) {
    CrossPlan p;
    kata_status s = cross_plan(B, H, Hkv, Tq, Tk, d, dtype, p);
    if (s != KATA_OK) return s;
    if (!q || !k || !v || !out) return KATA_ERR_INVALID_ARG;
    for (const void *x : {q, k, v, (const void *)out, (const void *)y_out, (const void *)den_out})
        if (!aligned16(x)) return KATA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(key_lengths) & 3u) != 0) return KATA_ERR_INVALID_ARG;
    const size_t es = dtype == KATA_BF16 ? 2 : 4, nq = (size_t)p.BH * p.R, nk = (size_t)p.BH * Tk;
    if (!apart({{out, nq * d * es}, {y_out, nq * d * 4}, {den_out, nq * 4}},
               {{q, nq * d * es}, {k, nk * d * es}, {v, nk * d * es}, {key_lengths, (size_t)B * 4}}))
        return KATA_ERR_INVALID_ARG;
    s = cross_workspace(p.ws_fwd_bytes, workspace, workspace_bytes);
    if (s != KATA_OK) return s;
    if (!device_ptrs_ok({q, k, v, key_lengths, out, y_out, den_out, p.ws_fwd_bytes ? workspace : nullptr}))
        return KATA_ERR_INVALID_ARG;
    CrossIo io{};
    io.q = q;
    io.k = k;
    io.v = v;
    io.key_lengths = key_lengths;
    io.out = out;
    io.y = y_out;
    io.den = den_out;
    io.ws = workspace;
    return launch_cross_forward(p, io, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? KATA_OK
                                                                                              : KATA_ERR_CUDA;
}

size_t kata_cross_backward_workspace_bytes(int B, int H, int Hkv, int Tq, int Tk, int d, kata_dtype dtype) {
    CrossPlan p;
    return cross_plan(B, H, Hkv, Tq, Tk, d, dtype, p) == KATA_OK ? p.ws_bwd_bytes : 0;
}

kata_status kata_cross_backward(const void *dout, const void *q, const void *k, const void *v, const float *y,
                                const float *den, const int32_t *key_lengths, void *dq, void *dk, void *dv, int B,
                                int H, int Hkv, int Tq, int Tk, int d, kata_dtype dtype, void *workspace,
                                size_t workspace_bytes, kata_stream_t stream) {
    CrossPlan p;
    kata_status s = cross_plan(B, H, Hkv, Tq, Tk, d, dtype, p);
    if (s != KATA_OK) return s;
    for (const void *x : {dout, q, k, v, (const void *)y, (const void *)den, (const void *)dq, (const void *)dk,
                          (const void *)dv})
        if (!x || !aligned16(x)) return KATA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(key_lengths) & 3u) != 0) return KATA_ERR_INVALID_ARG;
    const size_t es = dtype == KATA_BF16 ? 2 : 4, nq = (size_t)p.BH * p.R, nk = (size_t)p.BH * Tk;
    if (!apart({{dq, nq * d * es}, {dk, nk * d * es}, {dv, nk * d * es}},
               {{dout, nq * d * es}, {q, nq * d * es}, {k, nk * d * es}, {v, nk * d * es}, {y, nq * d * 4},
                {den, nq * 4}, {key_lengths, (size_t)B * 4}}))
        return KATA_ERR_INVALID_ARG;
    s = cross_workspace(p.ws_bwd_bytes, workspace, workspace_bytes);
    if (s != KATA_OK) return s;
    if (!device_ptrs_ok({dout, q, k, v, y, den, key_lengths, dq, dk, dv, workspace})) return KATA_ERR_INVALID_ARG;
    CrossIo io{};
    io.q = q;
    io.k = k;
    io.v = v;
    io.dout = dout;
    io.key_lengths = key_lengths;
    io.y = const_cast<float *>(y);
    io.den = const_cast<float *>(den);
    io.dq = dq;
    io.dk = dk;
    io.dv = dv;
    io.ws = workspace;
    return launch_cross_backward(p, io, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? KATA_OK
                                                                                               : KATA_ERR_CUDA;
}

}  // extern "C"
