// kla_gated.cu -- host side of the gated linear recurrence (kla_gated_scan_*
// of include/kla.h): argument checks, tiling and launches of the kernels in
// kla_gated.cuh.
#include "kla_gated.cuh"

#include <algorithm>
#include <type_traits>

namespace {

using namespace kla_mixer;

bool gate_ok(kla_gate_t g) { return g == KLA_GATE_CHANNEL || g == KLA_GATE_HEAD; }

struct Sizes {
    int64_t HN = 0, C = 0, rows = 0, n = 0;  // H*N, B*H*N, B*T*H, B*T*H*N
    int64_t gates = 0;                       // elements of f
};
bool sizes(int64_t B, int64_t T, int64_t H, int64_t N, kla_gate_t gate, Sizes *s) {
    int64_t bt = 0, bytes = 0;
    if (T < 0 || !mul_ok(H, N, &s->HN) || !mul_ok(B, s->HN, &s->C) || !mul_ok(B, T, &bt) ||
        !mul_ok(bt, H, &s->rows) || !mul_ok(bt, s->HN, &s->n) || !mul_ok(s->n, 4, &bytes) ||
        !mul_ok(s->rows, 4, &bytes))
        return false;
    s->gates = gate == KLA_GATE_HEAD ? s->rows : s->n;
    return true;
}

// Tokens of a lane in a round: 2 KB (bf16, shared gates, forward) to 8 KB (shared
// gates, backward) of a warp's rows in flight, two channels a lane.  Measured
// beside the other choice, on the long shape (B=1, T=65536, 32 x 128) and an
// ordinary one (B=8, T=2048, 16 x 128):
//   shared gates, forward   fp32 long 382 us, 494 with 8; bf16 ordinary 42, 50;
//                 backward  619, 711; 64, 72
//   fp32, forward           ordinary 67, 73 with 16; long 526, 487
//         backward          107, 123 with 8; 947, 848
//   bf16, forward, where an SM has one CTA at most (`few`: no more tiles than
//         SMs)              T=32768, 32 x 128, 189, 199 with 12
//         where it has more ordinary 49.7, 52.6 with 16
//         backward          ordinary 79.7, 82.4 with 4
template <typename Tin, bool HEAD, bool BACKWARD>
constexpr int tokens_of_lane(bool few) {
    if (HEAD) return 16;
    if (BACKWARD) return sizeof(Tin) == 4 ? 4 : 8;
    return sizeof(Tin) == 4 ? 8 : few ? 16 : 12;
}
int tokens_of_lane(kla_dtype_t dt, bool head, bool backward, bool few) {
    using bf16 = __nv_bfloat16;
    if (dt == KLA_F32)
        return head ? backward ? tokens_of_lane<float, true, true>(few) : tokens_of_lane<float, true, false>(few)
                    : backward ? tokens_of_lane<float, false, true>(few) : tokens_of_lane<float, false, false>(few);
    return head ? backward ? tokens_of_lane<bf16, true, true>(few) : tokens_of_lane<bf16, true, false>(few)
                : backward ? tokens_of_lane<bf16, false, true>(few) : tokens_of_lane<bf16, false, false>(few);
}

struct Launch {
    GatedTiles g;
    int64_t tiles;
    int vec, S, copy, W, C, group;
    bool few;  // no more tiles than SMs
};

// The arrays of a call: those whose rows are read through shared memory
// (in), and those that are only written.
struct Array {
    const void *p;
    int64_t size;  // of an element
    bool in;
};

// Tiles of 32 / S x vec channels.  Tiles run on over the heads of a batch row,
// unless a gate is shared by a head whose channels and a tile's do not divide
// one another (or by heads so small that a tile would have more of them than
// its warps have room for): then each head has tiles of its own, so that the
// sum over its channels stays within whole tiles.
void tile(int64_t B, int64_t H, int64_t N, bool head, int vec, int S, Launch *l) {
    const int64_t cw = 32 / S * vec;
    const bool own = head && N % cw != 0 && (cw % N != 0 || cw / N > kGatedHeads / S);
    l->vec = vec;
    l->S = S;
    l->g.seg = own ? N : H * N;
    l->g.per_seg = (l->g.seg + cw - 1) / cw;
    l->g.per_row = l->g.per_seg * (own ? H : 1);
    l->tiles = B * l->g.per_row;
    l->group = head && !own && N < cw ? (int)(N / vec) : 32 / S;
}

// How the rows of tiles of segments of `seg` channels can be copied.
int copy_of(int64_t HN, int64_t seg, const Array *arrays, int n) {
    bool wide = seg == HN || seg % 8 == 0, start = true;
    for (int i = 0; i < n; ++i)
        if (arrays[i].in && arrays[i].p) {
            wide = wide && HN * arrays[i].size % 16 == 0;
            start = start && aligned(arrays[i].p, 16);
        }
    return start ? wide ? WIDE : SHIFT : NARROW;
}

// Warps that an SM holds at once, by registers and by shared memory
// (rows and gates of a warp, as GatedStage has them).
struct Resident {
    kla_dtype_t dt;
    bool head, backward;
    int64_t tokens(bool few) const { return tokens_of_lane(dt, head, backward, few); }
    // bytes of a warp's rows in one round
    int64_t stage(const Launch &l) const {
        const int64_t e = dtype_size(dt), L = tokens(l.few), S = l.S;
        const int64_t pad = l.copy == SHIFT ? 16 : 0, cw = 32 / S * l.vec, apart = S > 1 ? cw : 0;
        const int64_t wide = S * (L * (4 * cw + pad) + 4 * apart), in = S * (L * (e * cw + pad) + e * apart);
        return (backward ? 2 * wide : in) + (head ? 0 : in);
    }
    int64_t warps(const Launch &l) const {
        const int64_t bytes =
            kGatedRounds * stage(l) + (head ? tokens(l.few) * kGatedHeads * 4 : 0) + 512 * l.vec;
        return std::min<int64_t>(65536 / (32 * (backward ? kGatedBackwardRegs : kGatedRegs)) / 4 * 4,
                                 226 * 1024 / bytes);
    }
};

// The widest tiles of which there are enough: 0.8 of the SMs, or 1.5 of them
// with one channel a lane.  Measured, forward and backward: shared gates, the
// long fp32 shape, 128 tiles of 32 channels 380 and 616 us, 256 of 16 440 and 904;
// B=2, T=5001, 12 x 80, 120 tiles 21 and 37, 240 27 and 51.  Near the edge, fp32,
// T=4096, 112 tiles of 64 channels 63 and 109, as 224 of 32 59 and 102 (shared
// gates 51 and 72, 43 and 78); 120 tiles 64 and 111, as 240 64 and 107 (53 and 72,
// 48 and 76).  Rows that start on 16 bytes, and on pairs of channels in every
// array, take two channels a lane (half the instructions for a channel, and two
// chains of multiply-adds side by side), others one; a warp's lanes in 1, 2, 4 or
// (fp32) 8 parts.
template <typename F>
Launch plan(int64_t B, int64_t T, int64_t H, int64_t N, const Array *arrays, int n, const F &resident) {
    Launch l;
    const bool head = resident.head;
    const int64_t HN = H * N, sms = sm_count();
    l.g.T = T; l.g.H = H; l.g.N = N; l.g.HN = HN;
    bool pairs = HN % 2 == 0 && (!head || N % 2 == 0);
    for (int i = 0; i < n; ++i) pairs = pairs && aligned(arrays[i].p, 2 * arrays[i].size);
    constexpr int kForms[7][2] = {{2, 1}, {2, 2}, {2, 4}, {2, 8}, {1, 1}, {1, 2}, {1, 4}};
    bool any = false;
    for (const auto &form : kForms) {
        const int vec = form[0], S = form[1];
        Launch k = l;
        tile(B, H, N, head, vec, S, &k);
        k.copy = copy_of(HN, k.g.seg, arrays, n);
        if (vec == 2 ? !pairs || k.copy != WIDE : any) continue;
        if (vec == 1 && k.copy == WIDE) k.copy = SHIFT;
        // Parts whose rows are no shorter than a sector of memory in the inputs'
        // type: bf16 in 4 parts at most (T=65536, 2 x 64, backward: shared gates
        // 64 us, 86 with 8; a gate for each channel 78, 79; B=8, T=8192: 33, 41;
        // forward 41 us, 39 with 8; 45, 47; 23, 27)
        k.few = k.tiles <= sms;
        const int64_t L = resident.tokens(k.few);
        if (S > 1 && (k.copy == NARROW || (T + L - 1) / L < S || (vec == 2 && 64 / S * dtype_size(resident.dt) < 32)))
            continue;
        l = k;
        any = any || vec == 2;
        if (vec == 2 ? 5 * l.tiles >= 4 * sms : 2 * l.tiles >= 3 * sms) break;
    }
    const int64_t R = l.S * resident.tokens(l.few), chunks = (T + R - 1) / R;  // of a warp
    const int64_t held = resident.warps(l);
    l.C = 1;
    // 8 warps (B=8, T=2048, 16 x 128, two CTAs an SM: bf16 50 us, 55 with 12, 51
    // with 6; fp32 66, 74 and 64; shared gates 42, 41 and 47)
    l.W = (int)std::min({(int64_t)8, held, chunks});
    if (3 * l.tiles <= 2 * sms) {
        // few tiles all the same: clusters, until there are more CTAs than SMs
        while (l.C < kGatedMaxCluster && l.tiles * l.C <= sms && (int64_t)l.C * l.W < chunks) l.C *= 2;
    } else if (l.few && chunks >= 32 * kGatedMaxWarps) {
        // one CTA an SM, and a long sequence: as many warps as have 64 KB of
        // rows in a round (the long fp32 shape: 512 us with 16 against 602
        // with 8, backward 932 against 1123; shared gates 397 against 422; T=32768
        // in bf16 197 against 206).  B=1, 16 x 128 in bf16, four parts: of 256
        // chunks 74 us with 16, 58 with 8, of 384 105 and 84; above the limit
        // 512 137 and 111, backward 179 and 183
        l.W = (int)std::max<int64_t>(
            l.W, std::min({(int64_t)kGatedMaxWarps, held, 64 * 1024 / resident.stage(l)}));
    }
    // many tiles: fewer warps each, so that all are resident at once (CTAs
    // that had to wait for others would run alone at the end)
    if (l.C == 1) l.W = (int)std::max<int64_t>(1, std::min<int64_t>(l.W, held / ((l.tiles + sms - 1) / sms)));
    return l;
}

// How a call runs.  A gate for each head of one channel is a gate for each
// channel; the arrays of gates shared by a head are read element by element.
Launch plan_forward(int64_t B, int64_t T, int64_t H, int64_t N, kla_dtype_t dt, kla_gate_t gate, const void *f,
                    const void *x, const float *h) {
    const bool head = gate == KLA_GATE_HEAD && N > 1;
    const int64_t e = dtype_size(dt);
    const Array arrays[3] = {{x, e, true}, {h, 4, false}, {f, e, true}};
    return plan(B, T, H, N, arrays, head ? 2 : 3, Resident{dt, head, false});
}
Launch plan_backward(int64_t B, int64_t T, int64_t H, int64_t N, kla_dtype_t dt, kla_gate_t gate, const void *f,
                     const float *h, const float *g_h, const void *grad_f, const void *grad_x) {
    const bool head = gate == KLA_GATE_HEAD && N > 1;
    const int64_t e = dtype_size(dt);
    const Array arrays[5] = {{g_h, 4, true}, {grad_f ? h : nullptr, 4, true}, {grad_x, e, false},
                             {f, e, true}, {grad_f, e, false}};
    return plan(B, T, H, N, arrays, head ? 3 : 5, Resident{dt, head, true});
}

// Tiles (of cw channels) of a head whose gate gradients the reduce kernel adds up.
int64_t parts_of(int64_t N, int cw) { return (N + cw - 1) / cw; }

template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), int64_t grid, int threads, int cluster, size_t smem, cudaStream_t stream,
                   A &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.dynamicSmemBytes = smem;
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

// Leave for a kernel to use all the shared memory that its largest CTA needs,
// once for each device.
template <auto KERNEL>
cudaError_t allow_smem(int smem) {
    static std::mutex mu;
    static bool done[256] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 256) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (done[dev]) return cudaSuccess;
    e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    done[dev] = e == cudaSuccess;
    return e;
}

template <int VEC>
constexpr int smem_bytes(int stage, int W, int C) {
    return W * (stage + GatedPairs<VEC>::BYTES) + (C > 1 ? C * GatedPairs<VEC>::BYTES : 0);
}

template <auto KERNEL, int VEC, typename Params>
cudaError_t run(const Launch &l, int stage, const Params &prm, cudaStream_t st) {
    const cudaError_t e = allow_smem<KERNEL>(
        std::min(227 * 1024, smem_bytes<VEC>(stage, kGatedMaxWarps, kGatedMaxCluster)));
    if (e != cudaSuccess) return e;
    return launch(KERNEL, l.tiles * l.C, 32 * l.W, l.C, (size_t)smem_bytes<VEC>(stage, l.W, l.C), st, prm);
}

template <typename Tin, int VEC, int S, bool HEAD, int COPY, int L>
cudaError_t run_tokens(const Launch &l, const GatedParams &prm, cudaStream_t st) {
    constexpr int STAGE = GatedStage<Tin, VEC, S, HEAD, L, COPY, false>::WARP;
    return run<kla_gated_forward_kernel<Tin, VEC, S, HEAD, L, COPY>, VEC>(l, STAGE, prm, st);
}
template <typename Tin, int VEC, int S, bool HEAD, int COPY, int L>
cudaError_t run_tokens(const Launch &l, const GatedBackwardParams &prm, cudaStream_t st) {
    constexpr int STAGE = GatedStage<Tin, VEC, S, HEAD, L, COPY, true>::WARP;
    return run<kla_gated_backward_kernel<Tin, VEC, S, HEAD, L, COPY>, VEC>(l, STAGE, prm, st);
}
template <typename Tin, int VEC, int S, bool HEAD, int COPY, typename Params>
cudaError_t run_scan(const Launch &l, const Params &prm, cudaStream_t st) {
    constexpr bool BACKWARD = std::is_same_v<Params, GatedBackwardParams>;
    return l.few ? run_tokens<Tin, VEC, S, HEAD, COPY, tokens_of_lane<Tin, HEAD, BACKWARD>(true)>(l, prm, st)
                 : run_tokens<Tin, VEC, S, HEAD, COPY, tokens_of_lane<Tin, HEAD, BACKWARD>(false)>(l, prm, st);
}
// The forms that plan() chooses from.
template <typename Tin, bool HEAD, typename Params>
cudaError_t run_form(const Launch &l, const Params &prm, cudaStream_t st) {
    if (l.copy == NARROW) return run_scan<Tin, 1, 1, HEAD, NARROW>(l, prm, st);
    if (l.copy == SHIFT)
        return l.S == 1   ? run_scan<Tin, 1, 1, HEAD, SHIFT>(l, prm, st)
               : l.S == 2 ? run_scan<Tin, 1, 2, HEAD, SHIFT>(l, prm, st)
                          : run_scan<Tin, 1, 4, HEAD, SHIFT>(l, prm, st);
    if constexpr (sizeof(Tin) == 4)
        if (l.S == 8) return run_scan<Tin, 2, 8, HEAD, WIDE>(l, prm, st);
    return l.S == 1   ? run_scan<Tin, 2, 1, HEAD, WIDE>(l, prm, st)
           : l.S == 2 ? run_scan<Tin, 2, 2, HEAD, WIDE>(l, prm, st)
                      : run_scan<Tin, 2, 4, HEAD, WIDE>(l, prm, st);
}
template <typename Params>
cudaError_t run_type(const Launch &l, kla_dtype_t dt, bool head, const Params &prm, cudaStream_t st) {
    if (dt == KLA_F32) return head ? run_form<float, true>(l, prm, st) : run_form<float, false>(l, prm, st);
    return head ? run_form<__nv_bfloat16, true>(l, prm, st) : run_form<__nv_bfloat16, false>(l, prm, st);
}

template <typename Tin>
int step_vec(const GatedStepParams &prm, bool head) {
    const int64_t e = (int64_t)sizeof(Tin);
    const bool ok = prm.C % 4 == 0 && (!head || prm.N % 4 == 0) && (head || aligned(prm.f, 4 * e)) &&
                    aligned(prm.x, 4 * e) && aligned(prm.h, 16) && aligned(prm.out, 16);
    return ok ? 4 : 1;
}

template <typename Tin>
cudaError_t run_step(const GatedStepParams &prm, bool head, cudaStream_t st) {
    const int vec = step_vec<Tin>(prm, head);
    const int64_t work = (prm.C + vec - 1) / vec;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)std::min<int64_t>((work + 255) / 256, (int64_t)sm_count() * 8));
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (vec == 4)
        return head ? cudaLaunchKernelEx(&cfg, kla_gated_step_kernel<Tin, 4, true>, prm)
                    : cudaLaunchKernelEx(&cfg, kla_gated_step_kernel<Tin, 4, false>, prm);
    return head ? cudaLaunchKernelEx(&cfg, kla_gated_step_kernel<Tin, 1, true>, prm)
                : cudaLaunchKernelEx(&cfg, kla_gated_step_kernel<Tin, 1, false>, prm);
}

}  // namespace

KLA_API kla_status_t kla_gated_scan_forward(const void *f, const void *x, kla_dtype_t in_dtype, kla_gate_t gate,
                                            const float *h0, float *h, int64_t B, int64_t T, int64_t H, int64_t N,
                                            void *stream) {
    if (B < 0 || T < 0 || H < 0 || N < 0 || !gate_ok(gate)) return KLA_ERR_INVALID_ARG;
    if (!dtype_ok(in_dtype)) return KLA_ERR_UNSUPPORTED_DTYPE;
    Sizes s;
    if (!sizes(B, T, H, N, gate, &s)) return KLA_ERR_INVALID_ARG;
    if (s.n == 0) return KLA_OK;
    if (!f || !x || !h) return KLA_ERR_INVALID_ARG;
    const int64_t e = dtype_size(in_dtype);
    const Range outs[1] = {range_of(h, 4 * s.n)};
    const Range ins[3] = {range_of(f, e * s.gates), range_of(x, e * s.n), range_of(h0, 4 * s.C)};
    if (any_overlap(outs, 1, ins, 3)) return KLA_ERR_INVALID_ARG;

    const bool head = gate == KLA_GATE_HEAD && N > 1;
    const Launch l = plan_forward(B, T, H, N, in_dtype, gate, f, x, h);
    if (l.tiles > kMaxGrid / l.C) return KLA_ERR_INVALID_ARG;
    GatedParams prm;
    prm.g = l.g;
    prm.f = f; prm.x = x; prm.h0 = h0; prm.h = h; prm.n = s.n;
    return run_type(l, in_dtype, head, prm, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KLA_OK : KLA_ERR_CUDA;
}

KLA_API kla_status_t kla_gated_scan_plan(int64_t B, int64_t T, int64_t H, int64_t N, kla_dtype_t in_dtype,
                                         kla_gate_t gate, int backward, kla_gated_plan_t *out) {
    if (!out || B < 0 || T < 0 || H < 0 || N < 0 || !gate_ok(gate) || (backward != 0 && backward != 1))
        return KLA_ERR_INVALID_ARG;
    if (!dtype_ok(in_dtype)) return KLA_ERR_UNSUPPORTED_DTYPE;
    Sizes s;
    if (!sizes(B, T, H, N, gate, &s)) return KLA_ERR_INVALID_ARG;
    *out = kla_gated_plan_t{};
    if (s.n == 0) return KLA_OK;
    alignas(16) static const float any[4] = {};  // only where it lies is looked at
    const Launch l = backward ? plan_backward(B, T, H, N, in_dtype, gate, any, any, any, any, any)
                              : plan_forward(B, T, H, N, in_dtype, gate, any, any, any);
    out->tiles = l.tiles;
    out->channels = 32 / l.S * l.vec;
    out->parts = l.S;
    out->tokens = tokens_of_lane(in_dtype, gate == KLA_GATE_HEAD && N > 1, backward, l.few);
    out->warps = l.W;
    out->cluster = l.C;
    out->whole_rows = l.copy == WIDE;
    const int64_t round = (int64_t)l.C * l.W * l.S * out->tokens;
    out->rounds = (T + round - 1) / round;
    return KLA_OK;
}

KLA_API kla_status_t kla_gated_scan_step(const void *f, const void *x, kla_dtype_t in_dtype, kla_gate_t gate,
                                         const float *h, float *h_out, int64_t B, int64_t H, int64_t N,
                                         void *stream) {
    if (B < 0 || H < 0 || N < 0 || !gate_ok(gate)) return KLA_ERR_INVALID_ARG;
    if (!dtype_ok(in_dtype)) return KLA_ERR_UNSUPPORTED_DTYPE;
    Sizes s;
    if (!sizes(B, 1, H, N, gate, &s)) return KLA_ERR_INVALID_ARG;
    if (s.n == 0) return KLA_OK;
    if (!f || !x || !h || !h_out) return KLA_ERR_INVALID_ARG;
    const int64_t e = dtype_size(in_dtype);
    const Range outs[1] = {range_of(h_out, 4 * s.n)};
    // in place (h_out == h) each thread reads its channels before it writes them
    const Range ins[3] = {range_of(f, e * s.gates), range_of(x, e * s.n),
                          range_of(h == h_out ? nullptr : h, 4 * s.n)};
    if (any_overlap(outs, 1, ins, 3)) return KLA_ERR_INVALID_ARG;
    GatedStepParams prm;
    prm.f = f; prm.x = x; prm.h = h; prm.out = h_out; prm.C = s.n; prm.N = N;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool head = gate == KLA_GATE_HEAD;
    const cudaError_t err =
        in_dtype == KLA_F32 ? run_step<float>(prm, head, st) : run_step<__nv_bfloat16>(prm, head, st);
    return err == cudaSuccess ? KLA_OK : KLA_ERR_CUDA;
}

KLA_API kla_status_t kla_gated_scan_backward_workspace_size(int64_t B, int64_t T, int64_t H, int64_t N,
                                                            kla_dtype_t in_dtype, kla_gate_t gate, size_t *bytes) {
    if (!bytes || B < 0 || T < 0 || H < 0 || N < 0 || !gate_ok(gate)) return KLA_ERR_INVALID_ARG;
    if (!dtype_ok(in_dtype)) return KLA_ERR_UNSUPPORTED_DTYPE;
    Sizes s;
    if (!sizes(B, T, H, N, gate, &s)) return KLA_ERR_INVALID_ARG;
    *bytes = 0;
    if (gate == KLA_GATE_HEAD && s.n > 0) {
        const int64_t parts = parts_of(N, 8);  // the narrowest tiles
        if (parts > 1) *bytes = (size_t)(4 * parts * s.rows);
    }
    return KLA_OK;
}

KLA_API kla_status_t kla_gated_scan_backward(const void *f, kla_dtype_t in_dtype, kla_gate_t gate, const float *h0,
                                             const float *h, const float *g_h, void *grad_f, void *grad_x,
                                             float *grad_h0, int64_t B, int64_t T, int64_t H, int64_t N,
                                             void *workspace, size_t workspace_bytes, void *stream) {
    size_t need = 0;
    const kla_status_t ws = kla_gated_scan_backward_workspace_size(B, T, H, N, in_dtype, gate, &need);
    if (ws != KLA_OK) return ws;
    Sizes s;
    sizes(B, T, H, N, gate, &s);
    const bool unused = s.C == 0 && s.gates > 0 && grad_f;  // gates of heads without channels
    if ((s.C == 0 && !unused) || (!grad_f && !grad_x && !grad_h0)) return KLA_OK;
    if (s.n > 0 && (!f || !g_h || (grad_f && !h))) return KLA_ERR_INVALID_ARG;
    const int64_t e = dtype_size(in_dtype);
    const Range outs[4] = {range_of(grad_f, e * s.gates), range_of(grad_x, e * s.n), range_of(grad_h0, 4 * s.C),
                           range_of(workspace, (int64_t)workspace_bytes)};
    const Range ins[4] = {range_of(f, e * s.gates), range_of(h0, 4 * s.C), range_of(h, 4 * s.n),
                          range_of(g_h, 4 * s.n)};
    if (any_overlap(outs, 4, ins, 4)) return KLA_ERR_INVALID_ARG;
    if (grad_f && need) {
        if (!workspace || workspace_bytes < need) return KLA_ERR_WORKSPACE_TOO_SMALL;
        if (!aligned(workspace, 256)) return KLA_ERR_MISALIGNED;
    }
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (unused)  // no state depends on them
        return cudaMemsetAsync(grad_f, 0, (size_t)(e * s.gates), st) == cudaSuccess ? KLA_OK : KLA_ERR_CUDA;
    if (T == 0) {  // no token: the loss does not depend on the entering state
        if (!grad_h0) return KLA_OK;
        return cudaMemsetAsync(grad_h0, 0, (size_t)(4 * s.C), st) == cudaSuccess ? KLA_OK : KLA_ERR_CUDA;
    }

    const bool head = gate == KLA_GATE_HEAD && N > 1;
    const Launch l = plan_backward(B, T, H, N, in_dtype, gate, f, h, g_h, grad_f, grad_x);
    if (l.tiles > kMaxGrid / l.C) return KLA_ERR_INVALID_ARG;
    const int64_t parts = head ? parts_of(N, 32 / l.S * l.vec) : 1;
    GatedBackwardParams prm;
    prm.g = l.g;
    prm.f = f; prm.h0 = h0; prm.h = h; prm.gh = g_h;
    prm.gf = grad_f; prm.gx = grad_x; prm.gh0 = grad_h0;
    prm.partial = grad_f && parts > 1 ? static_cast<float *>(workspace) : nullptr;
    prm.gates = s.rows;
    prm.n = s.n;
    prm.group = l.group;
    cudaError_t err = run_type(l, in_dtype, head, prm, st);
    if (err == cudaSuccess && prm.partial) {
        const unsigned grid = (unsigned)std::min<int64_t>((s.rows + 255) / 256, (int64_t)sm_count() * 8);
        if (in_dtype == KLA_F32)
            kla_gated_reduce_kernel<float><<<grid, 256, 0, st>>>(prm.partial, static_cast<float *>(grad_f), s.rows,
                                                                 (int)parts);
        else
            kla_gated_reduce_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(
                prm.partial, static_cast<__nv_bfloat16 *>(grad_f), s.rows, (int)parts);
        err = cudaGetLastError();
    }
    return err == cudaSuccess ? KLA_OK : KLA_ERR_CUDA;
}
