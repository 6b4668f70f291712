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
//   1. every warp loads its L rows of f and x into registers: all the loads
//      of the round are in flight at once, rows of 32 x VEC elements,
//      coalesced, with no demand on alignment beyond the vector's;
//   2. it composes them (two multiply-adds a token) and leaves (A, z) in
//      shared memory;
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

// The pairs (A, z) of a round, and of a cluster's CTAs; double-buffered, so
// that one barrier a round is enough (a buffer is written again two rounds
// later, behind the barrier of the round between).
template <int VEC>
struct GatedShared {
    float2 warp[2][kGatedMaxWarps][VEC][32];
    float2 cta[2][kGatedMaxCluster][VEC][32];
};

// Step 2 and 3 above: leave this warp's pair, meet the others, and return
// the state entering this warp's tokens in `entry`; `carry` goes from the
// round's entry to its exit.  Called by all warps of the CTA (cluster).
template <int VEC, bool CLUSTER>
__device__ __forceinline__ void exchange(GatedShared<VEC> &sh, int buf, int w, int W, int lane, unsigned rank,
                                         unsigned C, const float (&A)[VEC], const float (&z)[VEC],
                                         float (&carry)[VEC], float (&entry)[VEC]) {
#pragma unroll
    for (int v = 0; v < VEC; ++v) sh.warp[buf][w][v][lane] = make_float2(A[v], z[v]);
    __syncthreads();
    if constexpr (!CLUSTER) {
        for (int i = 0; i < W; ++i) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                if (i == w) entry[v] = carry[v];
                const float2 p = sh.warp[buf][i][v][lane];
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
                const float2 p = sh.warp[buf][i][v][lane];
                tz[v] = fmaf(p.x, tz[v], p.y);
                ta[v] *= p.x;
            }
        }
        for (unsigned c = w; c < C; c += W)
#pragma unroll
            for (int v = 0; v < VEC; ++v)
                store_remote(&sh.cta[buf][rank][v][lane], c, make_float2(ta[v], tz[v]));
        cluster_barrier();
        float mine[VEC];
        for (unsigned c = 0; c < C; ++c) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                if (c == rank) mine[v] = carry[v];
                const float2 p = sh.cta[buf][c][v][lane];
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

// Grid: tiles x C CTAs of 32 x W threads.
template <typename Tin, int VEC, bool HEAD, int L, bool CLUSTER>
__global__ void __launch_bounds__(32 * kGatedMaxWarps, KLA_GATED_MINB) kla_gated_forward_kernel(const GatedParams prm) {
    __shared__ GatedShared<VEC> sh;
    const GatedTiles &g = prm.g;
    const int lane = threadIdx.x & 31;
    const int w = threadIdx.x >> 5;
    const int W = blockDim.x >> 5;
    const unsigned C = CLUSTER ? cluster_size() : 1u;
    const unsigned rank = CLUSTER ? cluster_rank() : 0u;
    const TileAt at = tile_at(g, blockIdx.x / C, 32 * VEC);
    int64_t c = at.c0 + lane * VEC;
    const bool valid = c < at.end;
    if (!valid) c = at.end - VEC;  // reads a neighbour's channels, stores nothing
    const int64_t gates = HEAD ? g.H : g.HN;
    const int64_t row0 = at.b * g.T;
    const Tin *f = static_cast<const Tin *>(prm.f) + row0 * gates + (HEAD ? c / g.N : c);
    const Tin *x = static_cast<const Tin *>(prm.x) + row0 * g.HN + c;
    float *h = prm.h + row0 * g.HN + c;
    constexpr int FV = HEAD ? 1 : VEC;  // gates per lane and token

    float carry[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) carry[v] = prm.h0 ? prm.h0[at.b * g.HN + c + v] : 0.f;
    if (CLUSTER) cluster_barrier();  // every rank runs before its shared memory is written

    const int64_t span = (int64_t)W * L;
    const int64_t rounds = (g.T + span * C - 1) / (span * C);
#pragma unroll 1
    for (int64_t r = 0; r < rounds; ++r) {
        const int64_t hn = opaque(g.HN), gn = HEAD ? opaque(g.H) : hn;
        const int64_t t0 = (r * C + rank) * span + w * L;
        const int64_t left = g.T - t0;
        const int nv = left >= L ? L : left > 0 ? (int)left : 0;
        Pack<Tin, FV> fr[L];
        Pack<Tin, VEC> xr[L];
        const Tin *ft = f + t0 * gn;
        const Tin *xt = x + t0 * hn;
        if (nv == L) {
#pragma unroll
            for (int i = 0; i < L; ++i, ft += gn, xt += hn) {
                fr[i] = load_cs<Tin, FV>(ft);
                xr[i] = load_cs<Tin, VEC>(xt);
            }
        } else {  // tokens past the end leave the state as it is: f = 1, x = 0
#pragma unroll
            for (int i = 0; i < L; ++i, ft += gn, xt += hn) {
#pragma unroll
                for (int v = 0; v < FV; ++v) fr[i].v[v] = from_float<Tin>(1.f);
#pragma unroll
                for (int v = 0; v < VEC; ++v) xr[i].v[v] = from_float<Tin>(0.f);
                if (i < nv) {
                    fr[i] = load_cs<Tin, FV>(ft);
                    xr[i] = load_cs<Tin, VEC>(xt);
                }
            }
        }
        float A[VEC], z[VEC], entry[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            A[v] = 1.f;
            z[v] = 0.f;
#pragma unroll
            for (int i = 0; i < L; ++i) {
                const float fv = to_float(fr[i].v[HEAD ? 0 : v]);
                A[v] *= fv;
                z[v] = fmaf(fv, z[v], to_float(xr[i].v[v]));
            }
        }
        exchange<VEC, CLUSTER>(sh, (int)(r & 1), w, W, lane, rank, C, A, z, carry, entry);
        float *ht = h + t0 * hn;
#pragma unroll
        for (int i = 0; i < L; ++i, ht += hn) {
            Pack<float, VEC> o;
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                entry[v] = fmaf(to_float(fr[i].v[HEAD ? 0 : v]), entry[v], to_float(xr[i].v[v]));
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

// Grid: tiles x C CTAs of 32 x W threads; token s of the kernel is T-1-s.
template <typename Tin, int VEC, bool HEAD, int L, bool CLUSTER>
__global__ void __launch_bounds__(32 * kGatedMaxWarps, KLA_GATED_BACKWARD_MINB) kla_gated_backward_kernel(const GatedBackwardParams prm) {
    __shared__ GatedShared<VEC> sh;
    const GatedTiles &g = prm.g;
    const int lane = threadIdx.x & 31;
    const int w = threadIdx.x >> 5;
    const int W = blockDim.x >> 5;
    const unsigned C = CLUSTER ? cluster_size() : 1u;
    const unsigned rank = CLUSTER ? cluster_rank() : 0u;
    const int64_t tile = blockIdx.x / C;
    const TileAt at = tile_at(g, tile, 32 * VEC);
    int64_t c = at.c0 + lane * VEC;
    const bool valid = c < at.end;
    if (!valid) c = at.end - VEC;
    const int64_t gates = HEAD ? g.H : g.HN;
    const int64_t row0 = at.b * g.T;
    const int64_t head = HEAD ? c / g.N : 0;
    const Tin *f = static_cast<const Tin *>(prm.f) + row0 * gates + (HEAD ? head : c);
    const float *gh = prm.gh + row0 * g.HN + c;
    const float *h = prm.gf ? prm.h + row0 * g.HN + c : nullptr;
    const float *h0 = prm.h0 ? prm.h0 + at.b * g.HN + c : nullptr;
    Tin *gx = prm.gx ? static_cast<Tin *>(prm.gx) + row0 * g.HN + c : nullptr;
    Tin *gf = prm.gf && !HEAD ? static_cast<Tin *>(prm.gf) + row0 * gates + c : nullptr;
    constexpr int FV = HEAD ? 1 : VEC;

    float carry[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) carry[v] = 0.f;
    if (CLUSTER) cluster_barrier();

    const int64_t span = (int64_t)W * L;
    const int64_t rounds = (g.T + span * C - 1) / (span * C);
#pragma unroll 1
    for (int64_t r = 0; r < rounds; ++r) {
        const int64_t hn = opaque(g.HN), gn = HEAD ? opaque(g.H) : hn;
        const int64_t s0 = (r * C + rank) * span + w * L;
        const int64_t left = g.T - s0;
        const int nv = left >= L ? L : left > 0 ? (int)left : 0;
        const int64_t tl = g.T - 1 - s0;  // the chunk's last token; it walks down to tl - nv + 1
        Pack<Tin, FV> fr[L];              // f of token t + 1
        Pack<float, VEC> gr[L], hr[L];    // g of token t, h of token t - 1
        const Tin *ft = f + (tl + 1) * gn;
        const float *gt = gh + tl * hn;
        const float *ht = h + (tl - 1) * hn;
        if (nv == L && s0 > 0 && tl >= L) {  // every shifted row exists
#pragma unroll
            for (int i = 0; i < L; ++i, ft -= gn, gt -= hn, ht -= hn) {
                fr[i] = load_cs<Tin, FV>(ft);
                gr[i] = load_cs<float, VEC>(gt);
                if (h) hr[i] = load_cs<float, VEC>(ht);
            }
        } else {
#pragma unroll
            for (int i = 0; i < L; ++i, ft -= gn, gt -= hn, ht -= hn) {
                const int64_t t = tl - i;
                const bool on = i < nv;
#pragma unroll
                for (int v = 0; v < FV; ++v) fr[i].v[v] = from_float<Tin>(1.f);
#pragma unroll
                for (int v = 0; v < VEC; ++v) gr[i].v[v] = hr[i].v[v] = 0.f;
                if (on && t + 1 < g.T) fr[i] = load_cs<Tin, FV>(ft);
                if (on) gr[i] = load_cs<float, VEC>(gt);
                if (on && h) {
                    if (t > 0)
                        hr[i] = load_cs<float, VEC>(ht);
                    else if (h0)
#pragma unroll
                        for (int v = 0; v < VEC; ++v) hr[i].v[v] = h0[v];
                }
            }
        }
        float A[VEC], z[VEC], entry[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            A[v] = 1.f;
            z[v] = 0.f;
#pragma unroll
            for (int i = 0; i < L; ++i) {
                const float fv = to_float(fr[i].v[HEAD ? 0 : v]);
                A[v] *= fv;
                z[v] = fmaf(fv, z[v], gr[i].v[v]);
            }
        }
        exchange<VEC, CLUSTER>(sh, (int)(r & 1), w, W, lane, rank, C, A, z, carry, entry);
        float sum[L];  // HEAD: this lane's share of the shared gate's gradient
        Tin *gxt = gx + tl * hn;
        Tin *gft = gf + tl * hn;
#pragma unroll
        for (int i = 0; i < L; ++i, gxt -= hn, gft -= hn) {
            Pack<Tin, VEC> ox, of;
            sum[i] = 0.f;
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                entry[v] = fmaf(to_float(fr[i].v[HEAD ? 0 : v]), entry[v], gr[i].v[v]);
                ox.v[v] = from_float<Tin>(entry[v]);
                if (HEAD)
                    sum[i] = fmaf(entry[v], hr[i].v[v], sum[i]);
                else
                    of.v[v] = from_float<Tin>(entry[v] * hr[i].v[v]);
            }
            if (valid && i < nv) {
                if (gx) store_cs<Tin, VEC>(gxt, ox);
                if (!HEAD && gf) store_cs<Tin, VEC>(gft, of);
            }
        }
        if (prm.gh0 && tl - nv == -1 && nv > 0 && valid) {  // this chunk ended at token 0
            const Pack<Tin, FV> f0 = load_cs<Tin, FV>(f);
#pragma unroll
            for (int v = 0; v < VEC; ++v)
                prm.gh0[at.b * g.HN + c + v] = to_float(f0.v[HEAD ? 0 : v]) * entry[v];
        }
        if (HEAD && prm.gf) {
            // sum over the lanes of a head, in a fixed order
#pragma unroll
            for (int i = 0; i < L; ++i) {
                if (!valid) sum[i] = 0.f;
                for (int o = prm.group >> 1; o > 0; o >>= 1) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o);
            }
            const int in_group = lane & (prm.group - 1);
            if (at.c0 + (int64_t)(lane - in_group) * VEC < at.end) {  // a head of this tile
#pragma unroll
                for (int i = 0; i < L; ++i) {
                    if (i >= nv || (i & (prm.group - 1)) != in_group) continue;
                    const int64_t at_gate = (row0 + tl - i) * g.H + head;
                    if (prm.partial) {
                        const int64_t j = (at.c0 - head * g.N) / (32 * VEC);
                        prm.partial[j * prm.gates + at_gate] = sum[i];
                    } else {
                        static_cast<Tin *>(prm.gf)[at_gate] = from_float<Tin>(sum[i]);
                    }
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
