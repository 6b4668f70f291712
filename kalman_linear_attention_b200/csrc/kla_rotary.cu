// kla_rotary.cu -- host side of the queries' and keys' norm with the position
// rotation (kla_qk_norm_rotary_*, kla_rotary_forward of include/kla.h):
// argument checks, vector widths and launches of the kernels in
// kla_rotary.cuh.
#include "kla_rotary.cuh"

#include <algorithm>
#include <cmath>
#include <utility>

namespace {

using namespace kla_mixer;

// Heads of a token that a group of lanes takes one after another, with the
// cos and sin that it holds (B=4, T=4096, 32 + 8 heads of 128, bf16: 69 us with
// 8, 78 with 4, 70 with 16; 16 heads of 16: 146 us, 141 and 226), where there
// are two items at least for each warp of a full GPU (B=8, T=2048, 16 + 16 heads
// of 128: 56 us, 61 with four; the first shape's backward pass 103 us, 109
// with one).
constexpr int kRotaryRows = 8, kRotaryItems = 2;

constexpr int64_t kMaxRow = 1 << 29;  // elements of a token

// What one call works on, checked: everything but the tensors.
struct Call {
    RotaryParams prm = {};
    kla_dtype_t dtype = KLA_F32;
    int64_t B = 0, T = 0, D = 0;
    int vec = 1, upl = 1;
};

kla_status_t check_call(kla_dtype_t dtype, const double *inv_freq, int64_t rot_dim, int interleaved, float scale,
                        const int64_t *positions, int64_t position_stride, int64_t position0, int64_t B, int64_t T,
                        int64_t D, Call *c) {
    if (B < 0 || T < 0 || D < 0 || D > KLA_ROTARY_MAX_D) return KLA_ERR_INVALID_ARG;
    if (!dtype_ok(dtype)) return KLA_ERR_UNSUPPORTED_DTYPE;
    if (rot_dim < 0 || rot_dim > D || rot_dim % 2 != 0 || (rot_dim > 0 && !inv_freq) ||
        (interleaved != 0 && interleaved != 1) || !std::isfinite(scale) || position_stride < 0)
        return KLA_ERR_INVALID_ARG;
    int64_t tokens = 0;
    if (!mul_ok(B, T, &tokens)) return KLA_ERR_INVALID_ARG;
    RotaryParams &p = c->prm;
    p.inv_freq = inv_freq;
    p.positions = positions;
    p.position_stride = position_stride;
    p.position0 = position0;
    p.T = T;
    p.tokens = tokens;
    p.scale = scale;
    p.sign = 1.f;
    p.D = (int)D;
    p.half = (int)(rot_dim / 2);
    p.interleaved = interleaved;
    c->dtype = dtype;
    c->B = B;
    c->T = T;
    c->D = D;
    return KLA_OK;
}

// One strided input [B, T, heads, D] (strides null: dense); *bytes is what it
// spans.  A stride along an axis of one element does not matter.
bool set_input(const Call &c, const void *x, const int64_t *strides, int64_t heads, RotaryTensor *t, int64_t *bytes) {
    if (heads < 0 || heads > INT32_MAX) return false;
    int64_t row = 0, batch = 0, all = 0, span = 0;
    // heads and elements of a token are counted in 32 bits, up to two steps past the last
    if (!mul_ok(heads, c.D, &row) || row > kMaxRow || !mul_ok(row, c.T, &batch) || !mul_ok(batch, c.B, &all) ||
        !mul_ok(all, 4, &span))
        return false;
    t->x = x;
    t->heads = (int)heads;
    t->sb = strides ? strides[0] : batch;
    t->st = strides ? strides[1] : row;
    t->sh = strides ? strides[2] : c.D;
    if (c.B <= 1) t->sb = 0;
    if (c.T <= 1) t->st = 0;
    if (heads <= 1) t->sh = 0;
    if (t->sb < 0 || t->st < 0 || t->sh < 0) return false;
    *bytes = 0;
    if (all == 0) return true;
    int64_t eb = 0, et = 0, eh = 0;
    if (!mul_ok(t->sb, c.B - 1, &eb) || !mul_ok(t->st, c.T - 1, &et) || !mul_ok(t->sh, heads - 1, &eh)) return false;
    const int64_t most = INT64_MAX / 8;
    if (eb > most - c.D || et > most - c.D - eb || eh > most - c.D - eb - et) return false;
    *bytes = (eb + et + eh + c.D) * dtype_size(c.dtype);
    return true;
}

// The widest vector (16 bytes at most) on which the arrays start and that
// divides the strides and a row, and with pairs of halves also the halves and
// the rest of the row.
void choose_vec(Call *c, int tensors) {
    const int64_t e = dtype_size(c->dtype);
    const int64_t rest = c->D - 2 * c->prm.half;
    const bool halves = c->prm.half > 0 && !c->prm.interleaved;
    auto fits = [&](int v) {
        if (c->D % v != 0 || (halves && (c->prm.half % v != 0 || rest % v != 0))) return false;
        for (int i = 0; i < tensors; ++i) {
            const RotaryTensor &t = c->prm.t[i];
            if (t.sb % v != 0 || t.st % v != 0 || t.sh % v != 0) return false;
            for (const void *p : {t.x, t.gy, (const void *)t.y})
                if (p && !aligned(p, v * e)) return false;
        }
        return true;
    };
    c->vec = (int)(16 / e);
    while (c->vec > 1 && !fits(c->vec)) c->vec /= 2;
    c->prm.units = (int)((c->D + 2 * c->vec - 1) / (2 * c->vec));
    // narrow vectors: four units a lane, so that a row is not spread over more
    // lanes than its size is worth
    const int least = c->vec > 2 ? 1 : 4;
    int lanes = 1;
    while (lanes < 32 && lanes * least < c->prm.units) lanes *= 2;
    c->prm.lanes = lanes;
    c->upl = (c->prm.units + lanes - 1) / lanes;
}

// How warps share a tensor's tokens and heads.  A group takes kRotaryRows
// heads of a token where there are tokens enough to fill the SMs with warps,
// fewer where there are not.  At most as many CTAs as are resident at once;
// the tensors share them by their rows and what an item costs beyond its rows
// (about two rows' time: cos and sin, the first copies).  Items are whole, so the
// warps with one more than the others set the time: B=4, T=4096, 32 + 8 heads of
// 128 has 6.006 items of the queries for a warp, and 10.04 of the keys; the
// rotation of T=16384, 8 heads 2.31.
void choose_items(Call *c, int tensors, bool backward) {
    const int64_t cap = (int64_t)sm_count() * rotary_resident(c->vec, c->upl, backward);
    const int64_t warps = kRotaryThreads / 32, abreast = 32 / c->prm.lanes;
    const int64_t fill = cap * warps;
    int64_t work[2] = {0, 0}, need[2] = {0, 0};
    for (int i = 0; i < tensors; ++i) {
        RotaryTensor &t = c->prm.t[i];
        const int64_t h = t.heads;
        if (h == 0 || c->prm.tokens == 0) continue;
        // heads that a warp takes at once: few, so that a group has many heads
        // and cos and sin serve them all; more where warps would be idle
        int64_t n = 1;
        while (n < abreast && n < h &&
               (n * kRotaryRows < h || c->prm.tokens * n < kRotaryItems * fill * abreast))
            n *= 2;
        t.abreast = (int)n;
        const int64_t shares = (c->prm.tokens + abreast / n - 1) / (abreast / n);
        const int64_t most = (h + n - 1) / n;  // one head a group
        int64_t splits = (most + kRotaryRows - 1) / kRotaryRows;
        splits = std::max(splits, std::min(most, fill / std::max<int64_t>(1, shares)));
        t.splits = (int)splits;
        const int64_t items = shares > kMaxGrid ? kMaxGrid : shares * splits;  // enough to fill any grid
        need[i] = (items + warps - 1) / warps;
        work[i] = items * ((most + splits - 1) / splits + 2);
    }
    const double all = (double)work[0] + (double)work[1];
    for (int i = 0; i < tensors; ++i)
        if (need[i] > 0)
            c->prm.t[i].ctas = (unsigned)(need[0] + need[1] <= cap
                                              ? need[i]
                                              : std::min(need[i], std::max<int64_t>(1, (int64_t)(cap * (work[i] / all)))));
}

// Pairs of cos and sin that a warp makes at once: those of its tokens.
int table_pairs(const Call &c) {
    int most = 0;
    for (const RotaryTensor &t : c.prm.t)
        if (t.ctas > 0) most = std::max(most, 32 / c.prm.lanes / t.abreast * c.prm.half);
    return most;
}

template <typename T, int VEC, int UPL, bool NORM, bool BACKWARD>
cudaError_t launch(const Call &c, cudaStream_t st) {
    const unsigned grid = c.prm.t[0].ctas + c.prm.t[1].ctas;
    if (grid == 0) return cudaSuccess;
    const int pairs = table_pairs(c);
    size_t smem = (kRotaryThreads / 32) * (size_t)RotaryShared<T, VEC, UPL, BACKWARD>::warp_bytes(pairs);
    if (BACKWARD) smem = std::max(smem, (size_t)(kRotaryThreads / 32) * c.prm.D * sizeof(float));  // the weights' sums
    auto kernel = kla_rotary_kernel<T, VEC, UPL, NORM, BACKWARD>;
    if (smem > 48 * 1024) {  // leave to use it, once for each device, kernel and size reached
        static std::mutex mu;
        static size_t allowed[256] = {};
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e == cudaSuccess && (dev < 0 || dev >= 256)) e = cudaErrorInvalidDevice;
        if (e != cudaSuccess) return e;
        std::lock_guard<std::mutex> lock(mu);
        if (allowed[dev] < smem) {
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
            if (e != cudaSuccess) return e;
            allowed[dev] = smem;
        }
    }
    kernel<<<grid, kRotaryThreads, smem, st>>>(c.prm, pairs);
    return cudaGetLastError();
}

// Units a lane: one, two or four where that is enough, else as many as the
// longest row has.
template <typename T, int VEC, bool NORM, bool BACKWARD>
cudaError_t launch_vec(const Call &c, cudaStream_t st) {
    constexpr int MOST = KLA_ROTARY_MAX_D / (2 * VEC) / 32;
    if constexpr (VEC > 2) {
        if (c.upl == 1) return launch<T, VEC, 1, NORM, BACKWARD>(c, st);
        if (c.upl == 2) return launch<T, VEC, 2, NORM, BACKWARD>(c, st);
    }
    if (MOST > 4 && c.upl <= 4) return launch<T, VEC, MOST < 4 ? MOST : 4, NORM, BACKWARD>(c, st);
    return launch<T, VEC, MOST, NORM, BACKWARD>(c, st);
}

template <typename T, bool NORM, bool BACKWARD>
cudaError_t launch_type(const Call &c, cudaStream_t st) {
    if constexpr (sizeof(T) == 2)
        if (c.vec == 8) return launch_vec<T, 8, NORM, BACKWARD>(c, st);
    if (c.vec == 4) return launch_vec<T, 4, NORM, BACKWARD>(c, st);
    if (c.vec == 2) return launch_vec<T, 2, NORM, BACKWARD>(c, st);
    return launch_vec<T, 1, NORM, BACKWARD>(c, st);
}

template <bool NORM, bool BACKWARD>
cudaError_t launch_call(const Call &c, cudaStream_t st) {
    return c.dtype == KLA_F32 ? launch_type<float, NORM, BACKWARD>(c, st)
                              : launch_type<__nv_bfloat16, NORM, BACKWARD>(c, st);
}

// Bytes that a call's positions span.
Range positions_range(const Call &c, const int64_t *positions) {
    if (!positions || c.prm.tokens == 0) return Range{0, 0};
    int64_t n = 0;
    if (!mul_ok(c.prm.position_stride, c.B - 1, &n) || n > INT64_MAX / 16 - c.T) n = INT64_MAX / 16 - c.T;
    return range_of(positions, 8 * (n + c.T));
}

// CTAs of a backward call at most.
int64_t backward_cap() { return (int64_t)sm_count() * kRotaryBackwardCtas; }

}  // namespace

KLA_API kla_status_t kla_rotary_forward(const void *x, const int64_t *x_strides, kla_dtype_t dtype,
                                        const double *inv_freq, int64_t rot_dim, int interleaved, float scale,
                                        int inverse, const int64_t *positions, int64_t position_stride,
                                        int64_t position0, void *out, int64_t B, int64_t T, int64_t H, int64_t D,
                                        void *stream) {
    Call c;
    const kla_status_t bad = check_call(dtype, inv_freq, rot_dim, interleaved, scale, positions, position_stride,
                                        position0, B, T, D, &c);
    if (bad != KLA_OK) return bad;
    int64_t bytes = 0;
    if (!set_input(c, x, x_strides, H, &c.prm.t[0], &bytes) || (inverse != 0 && inverse != 1))
        return KLA_ERR_INVALID_ARG;
    if (bytes == 0) return KLA_OK;
    if (!x || !out) return KLA_ERR_INVALID_ARG;
    const int64_t n = c.prm.tokens * H * D * dtype_size(dtype);
    const Range outs[1] = {range_of(out, n)};
    const Range ins[3] = {range_of(x, bytes), range_of(inv_freq, 4 * rot_dim), positions_range(c, positions)};
    if (any_overlap(outs, 1, ins, 3)) return KLA_ERR_INVALID_ARG;
    c.prm.t[0].y = out;
    if (inverse) c.prm.sign = -1.f;
    choose_vec(&c, 1);
    choose_items(&c, 1, false);
    return launch_call<false, false>(c, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KLA_OK : KLA_ERR_CUDA;
}

KLA_API kla_status_t kla_qk_norm_rotary_forward(const void *q, const int64_t *q_strides, const void *k,
                                                const int64_t *k_strides, kla_dtype_t dtype, const float *q_weight,
                                                const float *k_weight, float eps, const double *inv_freq,
                                                int64_t rot_dim, int interleaved, float scale,
                                                const int64_t *positions, int64_t position_stride,
                                                int64_t position0, void *q_out, void *k_out, int64_t B, int64_t T,
                                                int64_t Hq, int64_t Hk, int64_t D, void *stream) {
    Call c;
    const kla_status_t bad = check_call(dtype, inv_freq, rot_dim, interleaved, scale, positions, position_stride,
                                        position0, B, T, D, &c);
    if (bad != KLA_OK) return bad;
    int64_t qb = 0, kb = 0;
    if (!(eps >= 0.f) || !std::isfinite(eps) || !set_input(c, q, q_strides, Hq, &c.prm.t[0], &qb) ||
        !set_input(c, k, k_strides, Hk, &c.prm.t[1], &kb))
        return KLA_ERR_INVALID_ARG;
    if (qb == 0 && kb == 0) return KLA_OK;
    if ((qb && (!q || !q_out)) || (kb && (!k || !k_out))) return KLA_ERR_INVALID_ARG;
    const int64_t e = dtype_size(dtype);
    const Range outs[2] = {range_of(q_out, c.prm.tokens * Hq * D * e), range_of(k_out, c.prm.tokens * Hk * D * e)};
    const Range ins[6] = {range_of(q, qb), range_of(k, kb), range_of(q_weight, 4 * D), range_of(k_weight, 4 * D),
                          range_of(inv_freq, 4 * rot_dim), positions_range(c, positions)};
    if (any_overlap(outs, 2, ins, 6)) return KLA_ERR_INVALID_ARG;
    c.prm.eps = eps;
    c.prm.t[0].y = q_out;
    c.prm.t[1].y = k_out;
    c.prm.t[0].w = q_weight;
    c.prm.t[1].w = k_weight;
    choose_vec(&c, 2);
    choose_items(&c, 2, false);
    return launch_call<true, false>(c, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KLA_OK : KLA_ERR_CUDA;
}

KLA_API kla_status_t kla_qk_norm_rotary_backward_workspace_size(int64_t Hq, int64_t Hk, int64_t D, size_t *bytes) {
    if (!bytes || Hq < 0 || Hk < 0 || D < 0 || D > KLA_ROTARY_MAX_D) return KLA_ERR_INVALID_ARG;
    *bytes = Hq + Hk > 0 ? (size_t)(backward_cap() + 2) * (size_t)D * sizeof(float) : 0;
    return KLA_OK;
}

KLA_API kla_status_t kla_qk_norm_rotary_backward(
    const void *q, const int64_t *q_strides, const void *k, const int64_t *k_strides, kla_dtype_t dtype,
    const float *q_weight, const float *k_weight, float eps, const double *inv_freq, int64_t rot_dim,
    int interleaved, float scale, const int64_t *positions, int64_t position_stride, int64_t position0,
    const void *g_q, const void *g_k, void *grad_q, void *grad_k, float *grad_q_weight, float *grad_k_weight,
    int64_t B, int64_t T, int64_t Hq, int64_t Hk, int64_t D, void *workspace, size_t workspace_bytes,
    void *stream) {
    Call c;
    const kla_status_t bad = check_call(dtype, inv_freq, rot_dim, interleaved, scale, positions, position_stride,
                                        position0, B, T, D, &c);
    if (bad != KLA_OK) return bad;
    int64_t qb = 0, kb = 0;
    if (!(eps >= 0.f) || !std::isfinite(eps) || !set_input(c, q, q_strides, Hq, &c.prm.t[0], &qb) ||
        !set_input(c, k, k_strides, Hk, &c.prm.t[1], &kb))
        return KLA_ERR_INVALID_ARG;
    if (D == 0) return KLA_OK;
    // a tensor without rows, or of which nothing is wanted, is left out
    const bool do_q = qb && (grad_q || grad_q_weight), do_k = kb && (grad_k || grad_k_weight);
    if ((do_q && (!q || !g_q)) || (do_k && (!k || !g_k))) return KLA_ERR_INVALID_ARG;
    const int64_t e = dtype_size(dtype);
    const int64_t nq = c.prm.tokens * Hq * D * e, nk = c.prm.tokens * Hk * D * e;
    const Range outs[5] = {range_of(grad_q, nq), range_of(grad_k, nk), range_of(grad_q_weight, 4 * D),
                           range_of(grad_k_weight, 4 * D), range_of(workspace, (int64_t)workspace_bytes)};
    const Range ins[8] = {range_of(q, qb), range_of(k, kb), range_of(g_q, nq), range_of(g_k, nk),
                          range_of(q_weight, 4 * D), range_of(k_weight, 4 * D),
                          range_of(inv_freq, 4 * rot_dim), positions_range(c, positions)};
    if (any_overlap(outs, 5, ins, 8)) return KLA_ERR_INVALID_ARG;
    const bool sums = (do_q && grad_q_weight) || (do_k && grad_k_weight);
    if (sums) {
        size_t need = 0;
        kla_qk_norm_rotary_backward_workspace_size(Hq, Hk, D, &need);
        if (!workspace || workspace_bytes < need) return KLA_ERR_WORKSPACE_TOO_SMALL;
        if (!aligned(workspace, 256)) return KLA_ERR_MISALIGNED;
    }
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // the gradient of a weight that no row has used
    if (grad_q_weight && !qb && cudaMemsetAsync(grad_q_weight, 0, 4 * (size_t)D, st) != cudaSuccess)
        return KLA_ERR_CUDA;
    if (grad_k_weight && !kb && cudaMemsetAsync(grad_k_weight, 0, 4 * (size_t)D, st) != cudaSuccess)
        return KLA_ERR_CUDA;
    c.prm.eps = eps;
    c.prm.sign = -1.f;
    RotaryTensor *t = c.prm.t;
    t[0].gy = g_q; t[0].y = grad_q; t[0].w = q_weight;
    t[1].gy = g_k; t[1].y = grad_k; t[1].w = k_weight;
    if (!do_q) t[0] = RotaryTensor{};
    if (!do_k) t[1] = RotaryTensor{};
    if (!do_q && !do_k) return KLA_OK;
    choose_vec(&c, 2);
    choose_items(&c, 2, true);
    float *partial = static_cast<float *>(workspace);
    if (do_q && grad_q_weight) t[0].partial = partial;
    if (do_k && grad_k_weight) t[1].partial = partial + (int64_t)t[0].ctas * D;
    if (launch_call<true, true>(c, st) != cudaSuccess) return KLA_ERR_CUDA;
    if (sums) {
        RotaryReduceParams r = {};
        const int columns = (int)((D + 31) / 32);
        r.partial[0] = t[0].partial; r.partial[1] = t[1].partial;
        r.out[0] = grad_q_weight; r.out[1] = grad_k_weight;
        r.rows[0] = t[0].ctas; r.rows[1] = t[1].ctas;
        r.D = (int)D;
        r.ctas = t[0].partial ? columns : 0;
        const int grid = r.ctas + (t[1].partial ? columns : 0);
        kla_rotary_reduce_kernel<<<grid, dim3(32, 32), 0, st>>>(r);
        if (cudaGetLastError() != cudaSuccess) return KLA_ERR_CUDA;
    }
    return KLA_OK;
}
