// kla_gated.cuh -- the gated linear recurrence with given gates (sm_100a).
//
//   h_t = f_t h_{t-1} + x_t,   h_{-1} = h0
//
// for every channel (b, h, n) independently; the gate f is per channel, or
// shared by the N channels of a head.  Two tokens compose into one of the
// same kind, (f2, x2) after (f1, x1) = (f2 f1, f2 x1 + x2), so a span of
// tokens is summed up by the pair (A, z) = (product of gates, state left by
// a zero entry), and the state after it is A h + z.
//
// A CTA (or a cluster of C CTAs) owns a tile of 32 x VEC channels of one
// batch row for the whole sequence, and walks it in rounds of C x W x L
// tokens: warp w of a CTA takes L consecutive tokens, each lane VEC
// neighbouring channels.  Per round
//
//   1. every warp asks for its rows of the next round, by asynchronous copies
//      into shared memory (two rounds of it) of 16 bytes a lane, several rows
//      at once (WIDE), or, where rows do not start on 16 bytes, of each lane's
//      own channels; copies of 4 bytes a lane throughout took a third longer.
//      Nothing waits but the warp for its own copies.  Gates shared by a head
//      go through registers, one round ahead, a token a lane;
//   2. it composes its tokens of this round (two multiply-adds a token) and
//      leaves (A, z) in shared memory;
//   3. after one barrier each warp runs through the W pairs with the state
//      that left the previous round: the value on reaching its own pair is
//      its entry, the last one the next round's entry;
//   4. it replays its L tokens from the entry (one multiply-add a token) and
//      stores the states straight from registers.
//
// With few channels the sequence itself has to fill the GPU: a cluster of C
// CTAs then shares the tile, its ranks taking consecutive spans of W x L
// tokens; each rank writes its span's composed pair into every rank's shared
// memory, and one cluster barrier a round replaces any hand-over through
// global memory: no workspace, no flags, no waiting loops, one launch, and
// the same result from run to run.
//
// The backward pass is the same recurrence in reverse time,
//   E_t = dL/dh_t = g_t + f_{t+1} E_{t+1},
//   dL/dx_t = E_t,  dL/df_t = E_t h_{t-1},  dL/dh0 = f_0 E_0,
// on rows of f and h that are shifted by one token against g.
//
// States, products and sums are fp32; the gradients of f and x are rounded
// once to the inputs' type on store.
#pragma once

#include "kla_mixer.h"

namespace kla_mixer {

constexpr int kGatedMaxWarps = 8;
// CTAs per SM that the kernels' registers leave room for.
#ifndef KLA_GATED_MINB
#define KLA_GATED_MINB 3
#endif
#ifndef KLA_GATED_BACKWARD_MINB
#define KLA_GATED_BACKWARD_MINB 2
#endif
constexpr int kGatedMaxCluster = 8;

struct GatedTiles {
    int64_t T, H, N, HN;
    int64_t seg;      // channels that tiles may not straddle: H*N, or N (gates shared by odd-sized heads)
    int64_t per_seg;  // tiles per segment
    int64_t per_row;  // tiles per batch row
};

struct GatedParams {
    GatedTiles g;
    const void *f, *x;
    const float *h0;
    float *h;
};

// Where a tile lies: batch row, first channel, end of its segment.
struct TileAt {
    int64_t b, c0, end;
};
__device__ __forceinline__ TileAt tile_at(const GatedTiles &g, int64_t tile, int cw) {
    TileAt a;
    a.b = tile / g.per_row;
    const int64_t in_row = tile - a.b * g.per_row;
    const int64_t s = in_row / g.per_seg;
    a.c0 = s * g.seg + (in_row - s * g.per_seg) * cw;
    a.end = (s + 1) * g.seg;
    return a;
}

__device__ __forceinline__ unsigned cluster_rank() {
    unsigned r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ unsigned cluster_size() {
    unsigned r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Store to the same shared-memory variable of cluster rank `rank`.
__device__ __forceinline__ void store_remote(float2 *p, unsigned rank, float2 v) {
    const unsigned local = static_cast<unsigned>(__cvta_generic_to_shared(p));
    unsigned remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(rank));
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(remote), "f"(v.x), "f"(v.y) : "memory");
}

// The pairs (A, z) of a round's warps, and of a cluster's CTAs; double-buffered,
// so that one barrier a round is enough (a buffer is written again two rounds
// later, behind the barrier of the round between).
template <int VEC>
struct GatedPairs {
    using Pairs = float2[VEC][32];
    Pairs *warp;  // [2][W]
    Pairs *cta;   // [2][C]
    static constexpr int BYTES = 2 * (int)sizeof(Pairs);  // of a warp, or of a CTA of a cluster
};

// Step 2 and 3 above: leave this warp's pair, meet the others, and return
// the state entering this warp's tokens in `entry`; `carry` goes from the
// round's entry to its exit.  Called by all warps of the CTA (cluster).
template <int VEC, bool CLUSTER>
__device__ __forceinline__ void exchange(const GatedPairs<VEC> &sh, int buf, int w, int W, int lane, unsigned rank,
                                         unsigned C, const float (&A)[VEC], const float (&z)[VEC],
                                         float (&carry)[VEC], float (&entry)[VEC]) {
#pragma unroll
    for (int v = 0; v < VEC; ++v) sh.warp[buf * W + w][v][lane] = make_float2(A[v], z[v]);
    __syncthreads();
    if constexpr (!CLUSTER) {
        for (int i = 0; i < W; ++i) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                if (i == w) entry[v] = carry[v];
                const float2 p = sh.warp[buf * W + i][v][lane];
                carry[v] = fmaf(p.x, carry[v], p.y);
            }
        }
    } else {
        float pa[VEC], pz[VEC], ta[VEC], tz[VEC];  // of the warps before this one, of all
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            ta[v] = 1.f;
            tz[v] = 0.f;
        }
        for (int i = 0; i < W; ++i) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                if (i == w) {
                    pa[v] = ta[v];
                    pz[v] = tz[v];
                }
                const float2 p = sh.warp[buf * W + i][v][lane];
                tz[v] = fmaf(p.x, tz[v], p.y);
                ta[v] *= p.x;
            }
        }
        for (unsigned c = w; c < C; c += W)
#pragma unroll
            for (int v = 0; v < VEC; ++v)
                store_remote(&sh.cta[buf * C + rank][v][lane], c, make_float2(ta[v], tz[v]));
        cluster_barrier();
        float mine[VEC];
        for (unsigned c = 0; c < C; ++c) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                if (c == rank) mine[v] = carry[v];
                const float2 p = sh.cta[buf * C + c][v][lane];
                carry[v] = fmaf(p.x, carry[v], p.y);
            }
        }
#pragma unroll
        for (int v = 0; v < VEC; ++v) entry[v] = fmaf(pa[v], mine[v], pz[v]);
    }
}

// The row strides, opaque to the optimiser: it would otherwise carry a pointer
// for each of a round's rows from round to round (over 240 registers).
__device__ __forceinline__ int64_t opaque(int64_t x) {
    asm volatile("" : "+l"(x));
    return x;
}

// A vector on its way through shared memory: an asynchronous copy, or, for a
// single 16-bit element, a plain one.
template <typename T, int V>
__device__ __forceinline__ void bring(T *to, const T *from) {
    if constexpr (V * sizeof(T) >= 4)
        copy_async<V * sizeof(T)>(static_cast<unsigned>(__cvta_generic_to_shared(to)), from);
    else
        *to = *from;
}
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> pack_at(const T *p) {
    return *reinterpret_cast<const Pack<T, V> *>(p);
}
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> pack_of(float x) {
    Pack<T, V> p;
#pragma unroll
    for (int v = 0; v < V; ++v) p.v[v] = from_float<T>(x);
    return p;
}

// Copies of a warp's rows [0, L) x 32 VEC channels into `to`, those of them in
// [lo, hi); row i starts at from + i * step (step is negative in reverse
// time), at the tile's first channel; `width` channels of it are there.
template <typename T, int VEC, int L, bool WIDE>
__device__ __forceinline__ void bring_rows(T *to, const T *from, int64_t step, int lo, int hi, int width) {
    const int lane = threadIdx.x & 31;
    if constexpr (WIDE) {
        constexpr int E = 16 / (int)sizeof(T);      // elements a lane
        constexpr int LANES = 32 * VEC / E;         // lanes a row
        constexpr int ROWS = 32 / LANES;            // rows at once
        const int col = lane % LANES * E;
        int i = lane / LANES;
        const T *p = from + i * step + col;
        T *q = to + i * 32 * VEC + col;
#pragma unroll
        for (int k = 0; k < L / ROWS; ++k, i += ROWS, p += ROWS * step, q += ROWS * 32 * VEC)
            if (i >= lo && i < hi && col < width) bring<T, E>(q, p);
    } else {
        // a lane past the last channel copies the last ones
        const int col = lane * VEC < width ? lane * VEC : width - VEC;
        const T *p = from + col;
        T *q = to + lane * VEC;
#pragma unroll
        for (int i = 0; i < L; ++i, p += step, q += 32 * VEC)
            if (i >= lo && i < hi) bring<T, VEC>(q, p);
    }
}

// Gates shared by heads: those of a warp's L tokens and up to kGatedHeads heads
// of the tile, a few in each lane, one round ahead.
constexpr int kGatedHeads = 8;
template <typename Tin, int L>
struct HeadGates {
    static constexpr int N = L * kGatedHeads / 32;
    Tin ahead[N];

    // Token i of head k: at from + i * step + k, where lo <= i < hi.
    __device__ __forceinline__ void ask(const Tin *from, int64_t step, int heads, int lo, int hi) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int i = (n * 32 + lane) % L, k = (n * 32 + lane) / L;
            if (n * 32 < heads * L) {  // uniform
                ahead[n] = from_float<Tin>(1.f);
                if (k < heads && i >= lo && i < hi) ahead[n] = from[i * step + k];
            }
        }
    }
    // Into shared memory, in fp32: [heads][L].
    __device__ __forceinline__ void give(float *to, int heads) const {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int n = 0; n < N; ++n)
            if (n * 32 + lane < heads * L) to[n * 32 + lane] = to_float(ahead[n]);
    }
};

// Shared memory of a warp, in bytes: two rounds of its rows, and the gates
// shared by heads.
template <typename Tin, int VEC, bool HEAD, int L, bool BACKWARD>
struct GatedStage {
    static constexpr int X = 0;                                                  // rows of x, or of g
    static constexpr int H = X + 32 * L * VEC * (BACKWARD ? 4 : (int)sizeof(Tin));  // rows of h
    static constexpr int F = H + (BACKWARD ? 32 * L * VEC * 4 : 0);              // rows of f
    static constexpr int BYTES = F + (HEAD ? 0 : 32 * L * VEC * (int)sizeof(Tin));
    static constexpr int GATES = 2 * BYTES;
    static constexpr int WARP = GATES + (HEAD ? L * kGatedHeads * 4 : 0);
};

// The gates of a round, by token: floats of the lane's head, or packs of the
// rows in shared memory.  Tokens that are not there leave the state as it is.
template <typename Tin, int VEC, bool HEAD>
struct GateRow {
    const float *head;  // HEAD: of the lane's head
    const Tin *rows;    // else: of the lane's channels
    int lo, hi;         // tokens that are there
    __device__ __forceinline__ float at(int i, int v) const {
        if constexpr (HEAD) return head[i];
        return i >= lo && i < hi ? to_float(pack_at<Tin, VEC>(rows + i * 32 * VEC).v[v]) : 1.f;
    }
};

// Grid: tiles x C CTAs of 32 x W threads.  Dynamic shared memory: GatedStage of
// each warp, then the pairs.
template <typename Tin, int VEC, bool HEAD, int L, bool WIDE, bool CLUSTER>
__global__ void __launch_bounds__(32 * kGatedMaxWarps, KLA_GATED_MINB) kla_gated_forward_kernel(const GatedParams prm) {
    using Stage = GatedStage<Tin, VEC, HEAD, L, false>;
    using Pairs = typename GatedPairs<VEC>::Pairs;
    extern __shared__ __align__(16) unsigned char shared[];
    const GatedTiles &g = prm.g;
    const int lane = threadIdx.x & 31;
    const int w = threadIdx.x >> 5;
    const int W = blockDim.x >> 5;
    const unsigned C = CLUSTER ? cluster_size() : 1u;
    const unsigned rank = CLUSTER ? cluster_rank() : 0u;
    const TileAt at = tile_at(g, blockIdx.x / C, 32 * VEC);
    const int64_t c = at.c0 + lane * VEC;
    const bool valid = c < at.end;
    const int width = at.end - at.c0 < 32 * VEC ? (int)(at.end - at.c0) : 32 * VEC;
    const int64_t row0 = at.b * g.T;
    const int64_t head0 = HEAD ? at.c0 / g.N : 0;
    const int heads = HEAD ? (int)((at.c0 + width - 1) / g.N - head0) + 1 : 0;
    const Tin *f = static_cast<const Tin *>(prm.f) + (HEAD ? row0 * g.H + head0 : row0 * g.HN + at.c0);
    const Tin *x = static_cast<const Tin *>(prm.x) + row0 * g.HN + at.c0;
    float *h = prm.h + row0 * g.HN + c;
    unsigned char *const mine = shared + w * Stage::WARP;
    float *const gates = reinterpret_cast<float *>(mine + Stage::GATES);
    Pairs *const pairs = reinterpret_cast<Pairs *>(shared + W * Stage::WARP);
    const GatedPairs<VEC> sh{pairs, pairs + 2 * W};

    float carry[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) carry[v] = prm.h0 && valid ? prm.h0[at.b * g.HN + c + v] : 0.f;

    const int64_t span = (int64_t)W * L;
    const int64_t rounds = (g.T + span * C - 1) / (span * C);
    HeadGates<Tin, L> ahead;
    auto ask = [&](int64_t r) {
        const int64_t hn = opaque(g.HN), t0 = (r * C + rank) * span + w * L;
        const int nv = (int)(g.T - t0 < L ? g.T - t0 : L);
        unsigned char *const to = mine + (r & 1) * Stage::BYTES;
        bring_rows<Tin, VEC, L, WIDE>(reinterpret_cast<Tin *>(to + Stage::X), x + t0 * hn, hn, 0, nv, width);
        if constexpr (HEAD)
            ahead.ask(f + t0 * g.H, g.H, heads, 0, nv);
        else
            bring_rows<Tin, VEC, L, WIDE>(reinterpret_cast<Tin *>(to + Stage::F), f + t0 * hn, hn, 0, nv, width);
        copies_commit();
    };
    ask(0);
    if (CLUSTER) cluster_barrier();  // every rank runs before its shared memory is written

#pragma unroll 1
    for (int64_t r = 0; r < rounds; ++r) {
        const int64_t hn = opaque(g.HN), t0 = (r * C + rank) * span + w * L;
        const int nv = (int)(g.T - t0 < L ? g.T - t0 : L);
        const unsigned char *const from = mine + (r & 1) * Stage::BYTES;
        __syncwarp();  // the other stage and the gates have been read
        if (HEAD) ahead.give(gates, heads);
        if (r + 1 < rounds) {
            ask(r + 1);
            copies_wait<1>();
        } else {
            copies_wait<0>();
        }
        __syncwarp();
        const GateRow<Tin, VEC, HEAD> fs{gates + (HEAD && valid ? (c / g.N - head0) * L : 0),
                                         reinterpret_cast<const Tin *>(from + Stage::F) + lane * VEC, 0, nv};
        const Tin *const xs = reinterpret_cast<const Tin *>(from + Stage::X) + lane * VEC;
        auto x_at = [&](int i) { return i < nv ? pack_at<Tin, VEC>(xs + i * 32 * VEC) : pack_of<Tin, VEC>(0.f); };
        float A[VEC], z[VEC], entry[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            A[v] = 1.f;
            z[v] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const Pack<Tin, VEC> xi = x_at(i);
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const float fv = fs.at(i, v);
                A[v] *= fv;
                z[v] = fmaf(fv, z[v], to_float(xi.v[v]));
            }
        }
        exchange<VEC, CLUSTER>(sh, (int)(r & 1), w, W, lane, rank, C, A, z, carry, entry);
        float *ht = h + t0 * hn;
#pragma unroll
        for (int i = 0; i < L; ++i, ht += hn) {
            const Pack<Tin, VEC> xi = x_at(i);
            Pack<float, VEC> o;
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                entry[v] = fmaf(fs.at(i, v), entry[v], to_float(xi.v[v]));
                o.v[v] = entry[v];
            }
            if (valid && i < nv) store_cs<float, VEC>(ht, o);
        }
    }
}

struct GatedBackwardParams {
    GatedTiles g;
    const void *f;
    const float *h0, *h, *gh;
    void *gf, *gx;
    float *gh0;
    float *partial;  // [tiles of a head][B, T, H]: sums over a tile, where a head has several
    int64_t gates;   // B * T * H
    int group;       // lanes that share a head (HEAD): 32, or N / VEC below it
};

// Sums of L values over the lanes of groups of `group` lanes (a power of two),
// in a fixed order: halves of the values change hands at each step, so that
// every lane ends with the sums of its own share of them.
template <int L>
struct GroupSums {
    float x[L];
    int first;  // this lane's share: values first .. first + count - 1
    int count;
    bool writes;  // among the lanes with the same share, the one that writes

    __device__ __forceinline__ void run(int group) {
        const int lane = threadIdx.x & 31;
        first = 0;
        count = L;
        writes = true;
#pragma unroll
        for (int k = 0; k < 5; ++k) {
            const int o = group >> (k + 1);
            if (o == 0) continue;
            const bool up = lane & o;
            const int half = (L >> k) >> 1;
            if (half > 0) {
#pragma unroll
                for (int j = 0; j < half; ++j) {
                    const float give = up ? x[j] : x[half + j];
                    const float keep = up ? x[half + j] : x[j];
                    x[j] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                }
                first += up ? half : 0;
                count = half;
            } else {
                x[0] += __shfl_xor_sync(0xffffffffu, x[0], o);
                writes = writes && !up;
            }
        }
    }
};

// Grid: tiles x C CTAs of 32 x W threads; token s of the kernel is T-1-s.
// Dynamic shared memory as in the forward kernel.
template <typename Tin, int VEC, bool HEAD, int L, bool WIDE, bool CLUSTER>
__global__ void __launch_bounds__(32 * kGatedMaxWarps, KLA_GATED_BACKWARD_MINB)
kla_gated_backward_kernel(const GatedBackwardParams prm) {
    using Stage = GatedStage<Tin, VEC, HEAD, L, true>;
    using Pairs = typename GatedPairs<VEC>::Pairs;
    extern __shared__ __align__(16) unsigned char shared[];
    const GatedTiles &g = prm.g;
    const int lane = threadIdx.x & 31;
    const int w = threadIdx.x >> 5;
    const int W = blockDim.x >> 5;
    const unsigned C = CLUSTER ? cluster_size() : 1u;
    const unsigned rank = CLUSTER ? cluster_rank() : 0u;
    const TileAt at = tile_at(g, blockIdx.x / C, 32 * VEC);
    const int64_t c = at.c0 + lane * VEC;
    const bool valid = c < at.end;
    const int width = at.end - at.c0 < 32 * VEC ? (int)(at.end - at.c0) : 32 * VEC;
    const int64_t row0 = at.b * g.T;
    const int64_t head0 = HEAD ? at.c0 / g.N : 0;
    const int heads = HEAD ? (int)((at.c0 + width - 1) / g.N - head0) + 1 : 0;
    const Tin *f = static_cast<const Tin *>(prm.f) + (HEAD ? row0 * g.H + head0 : row0 * g.HN + at.c0);
    const float *gh = prm.gh + row0 * g.HN + at.c0;
    const float *h = prm.gf ? prm.h + row0 * g.HN + at.c0 : nullptr;
    const float *h0 = prm.h0 && valid ? prm.h0 + at.b * g.HN + c : nullptr;
    Tin *gx = prm.gx ? static_cast<Tin *>(prm.gx) + row0 * g.HN + c : nullptr;
    Tin *gf = prm.gf && !HEAD ? static_cast<Tin *>(prm.gf) + row0 * g.HN + c : nullptr;
    unsigned char *const mine = shared + w * Stage::WARP;
    float *const gates = reinterpret_cast<float *>(mine + Stage::GATES);
    Pairs *const pairs = reinterpret_cast<Pairs *>(shared + W * Stage::WARP);
    const GatedPairs<VEC> sh{pairs, pairs + 2 * W};

    float carry[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) carry[v] = 0.f;

    const int64_t span = (int64_t)W * L;
    const int64_t rounds = (g.T + span * C - 1) / (span * C);
    HeadGates<Tin, L> ahead;
    // of token t: g; h of token t - 1 (none before the first); f of token t + 1
    // (none after the last)
    auto ask = [&](int64_t r) {
        const int64_t hn = opaque(g.HN), s0 = (r * C + rank) * span + w * L;
        const int nv = (int)(g.T - s0 < L ? g.T - s0 : L);
        const int64_t tl = g.T - 1 - s0;  // the chunk's last token; it walks down
        unsigned char *const to = mine + (r & 1) * Stage::BYTES;
        bring_rows<float, VEC, L, WIDE>(reinterpret_cast<float *>(to + Stage::X), gh + tl * hn, -hn, 0, nv, width);
        if (h)
            bring_rows<float, VEC, L, WIDE>(reinterpret_cast<float *>(to + Stage::H), h + (tl - 1) * hn, -hn, 0,
                                            tl < nv ? (int)tl : nv, width);
        if constexpr (HEAD)
            ahead.ask(f + (tl + 1) * g.H, -g.H, heads, s0 > 0 ? 0 : 1, nv);
        else
            bring_rows<Tin, VEC, L, WIDE>(reinterpret_cast<Tin *>(to + Stage::F), f + (tl + 1) * hn, -hn,
                                          s0 > 0 ? 0 : 1, nv, width);
        copies_commit();
    };
    ask(0);
    if (CLUSTER) cluster_barrier();

#pragma unroll 1
    for (int64_t r = 0; r < rounds; ++r) {
        const int64_t hn = opaque(g.HN), s0 = (r * C + rank) * span + w * L;
        const int nv = (int)(g.T - s0 < L ? g.T - s0 : L);
        const int64_t tl = g.T - 1 - s0;
        const unsigned char *const from = mine + (r & 1) * Stage::BYTES;
        __syncwarp();  // the other stage and the gates have been read
        if (HEAD) ahead.give(gates, heads);
        if (r + 1 < rounds) {
            ask(r + 1);
            copies_wait<1>();
        } else {
            copies_wait<0>();
        }
        __syncwarp();
        const GateRow<Tin, VEC, HEAD> fs{gates + (HEAD && valid ? (c / g.N - head0) * L : 0),
                                         reinterpret_cast<const Tin *>(from + Stage::F) + lane * VEC, s0 > 0 ? 0 : 1, nv};
        const float *const gs = reinterpret_cast<const float *>(from + Stage::X) + lane * VEC;
        const float *const hs = reinterpret_cast<const float *>(from + Stage::H) + lane * VEC;
        auto g_at = [&](int i) { return i < nv ? pack_at<float, VEC>(gs + i * 32 * VEC) : pack_of<float, VEC>(0.f); };
        float A[VEC], z[VEC], entry[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            A[v] = 1.f;
            z[v] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const Pack<float, VEC> gi = g_at(i);
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const float fv = fs.at(i, v);
                A[v] *= fv;
                z[v] = fmaf(fv, z[v], gi.v[v]);
            }
        }
        exchange<VEC, CLUSTER>(sh, (int)(r & 1), w, W, lane, rank, C, A, z, carry, entry);
        GroupSums<L> sum;  // HEAD: this lane's share of the shared gate's gradient
        Tin *gxt = gx + tl * hn;
        Tin *gft = gf + tl * hn;
#pragma unroll
        for (int i = 0; i < L; ++i, gxt -= hn, gft -= hn) {
            const Pack<float, VEC> gi = g_at(i);
            Pack<float, VEC> before = pack_of<float, VEC>(0.f);
            if (h && i < nv) {
                if (i < tl)
                    before = pack_at<float, VEC>(hs + i * 32 * VEC);
                else if (h0)
#pragma unroll
                    for (int v = 0; v < VEC; ++v) before.v[v] = h0[v];
            }
            Pack<Tin, VEC> ox, of;
            sum.x[i] = 0.f;
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                entry[v] = fmaf(fs.at(i, v), entry[v], gi.v[v]);
                ox.v[v] = from_float<Tin>(entry[v]);
                if (HEAD)
                    sum.x[i] = fmaf(entry[v], before.v[v], sum.x[i]);
                else
                    of.v[v] = from_float<Tin>(entry[v] * before.v[v]);
            }
            if (HEAD && !valid) sum.x[i] = 0.f;
            if (valid && i < nv) {
                if (gx) store_cs<Tin, VEC>(gxt, ox);
                if (!HEAD && gf) store_cs<Tin, VEC>(gft, of);
            }
        }
        if (prm.gh0 && tl + 1 == nv && nv > 0 && valid) {  // this chunk ended at token 0
            const Tin *const f0 = f + (HEAD ? c / g.N - head0 : lane * VEC);
#pragma unroll
            for (int v = 0; v < VEC; ++v)
                prm.gh0[at.b * g.HN + c + v] = to_float(f0[HEAD ? 0 : v]) * entry[v];
        }
        if (HEAD && prm.gf) {
            sum.run(prm.group);
            const int64_t k = at.c0 + (lane & ~(prm.group - 1)) * VEC;  // the group's first channel
            if (k < at.end && sum.writes) {
                const int64_t head = k / g.N;
                const int64_t j = prm.partial ? (at.c0 - head * g.N) / (32 * VEC) : 0;
#pragma unroll
                for (int i = 0; i < L; ++i) {
                    if (i >= sum.count || sum.first + i >= nv) continue;
                    const int64_t at_gate = (row0 + tl - sum.first - i) * g.H + head;
                    if (prm.partial)
                        prm.partial[j * prm.gates + at_gate] = sum.x[i];
                    else
                        static_cast<Tin *>(prm.gf)[at_gate] = from_float<Tin>(sum.x[i]);
                }
            }
        }
    }
}

// The gradient of a gate shared by several tiles: their sums, added in order.
template <typename Tin>
__global__ void __launch_bounds__(256) kla_gated_reduce_kernel(const float *partial, Tin *gf, int64_t gates,
                                                               int parts) {
    for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < gates; i += (int64_t)gridDim.x * blockDim.x) {
        float s = 0.f;
        for (int j = 0; j < parts; ++j) s += partial[j * gates + i];
        gf[i] = from_float<Tin>(s);
    }
}

// One decode token: h' = f h + x, V channels per thread.  Bound by HBM (or by
// the launch): consecutive steps overlap through programmatic dependent
// launch, with nothing but the launch itself ahead of the wait.
struct GatedStepParams {
    const void *f, *x;
    const float *h;
    float *out;
    int64_t C, N;
};
template <typename Tin, int V, bool HEAD>
__global__ void __launch_bounds__(256) kla_gated_step_kernel(const GatedStepParams prm) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr int FV = HEAD ? 1 : V;
    for (int64_t i = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) * V; i < prm.C;
         i += (int64_t)gridDim.x * blockDim.x * V) {
        const Pack<Tin, FV> f = load_cs<Tin, FV>(static_cast<const Tin *>(prm.f) + (HEAD ? i / prm.N : i));
        const Pack<Tin, V> x = load_cs<Tin, V>(static_cast<const Tin *>(prm.x) + i);
        Pack<float, V> h = *reinterpret_cast<const Pack<float, V> *>(prm.h + i);
#pragma unroll
        for (int v = 0; v < V; ++v) h.v[v] = fmaf(to_float(f.v[HEAD ? 0 : v]), h.v[v], to_float(x.v[v]));
        *reinterpret_cast<Pack<float, V> *>(prm.out + i) = h;
    }
}

}  // namespace kla_mixer
