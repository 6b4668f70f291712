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
// A CTA (or a cluster of C CTAs) owns a tile of 32 / S x VEC channels of one
// batch row for the whole sequence, and walks it in rounds of C x W x S x L
// tokens: warp w of a CTA takes S L consecutive tokens, each lane L of them
// and VEC neighbouring channels (with few channels S parts of a warp's lanes
// take narrower rows, so that there are more tiles).  Per round
//
//   1. every warp asks for its rows of the next round, by asynchronous copies
//      of 16 bytes a lane into shared memory (two rounds of it), several rows
//      at once.  Where rows do not start on 16 bytes (SHIFT) the aligned
//      pieces around them are copied and read at an offset.  Nothing waits but
//      the warp for its own copies.  (Copies of each lane's own 4 bytes took a
//      third longer.)  Gates shared by a head go through registers, one round
//      ahead, a token a lane;
//   2. it composes its tokens of this round (two multiply-adds a token) and
//      leaves (A, z) in shared memory;
//   3. after one barrier each warp runs through the W pairs with the state
//      that left the previous round: the value on reaching its own pair is
//      its entry, the last one the next round's entry;
//   4. it replays its L tokens from the entry (one multiply-add a token) and
//      stores the states straight from registers.
//
// With few channels the sequence itself has to fill the GPU: a cluster of C
// CTAs then shares the tile, its ranks taking consecutive spans of W x S x L
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
// Every element is read and written once: HBM is the floor.  Copies reach 6.46
// TB/s; the scan of B=1, T=65536, 32 x 128 in fp32 takes 510 to 535 us (0.93 to
// 0.98 of that), its backward pass 930 to 950 (0.88 to 0.89), the bf16 scan of
// B=8, T=2048, 16 x 128 49.7 us (0.84) and 79.5 backward (0.91).  What bounds the
// rest is the chain of rounds, whose copies, barrier and exchange the 8 warps
// of a lone CTA do not hide (B=2, T=5001, 12 x 80, shared gates, 120 tiles: 10
// rounds of 1.6 us, 21 us forward and 37 backward, 0.58 and 0.49).
//
// States, products and sums are fp32; the gradients of f and x are rounded
// once to the inputs' type on store.
#pragma once

#include "kla_mixer.h"

namespace kla_mixer {

constexpr int kGatedMaxWarps = 16;
// Rounds of rows that a warp holds: the present one, and one asked for.  With
// two asked for, of 8 tokens a lane, a bf16 gate for each channel took as long
// for B=8, T=2048, 16 x 128 (49 us) and 227 us against 195 for B=1, T=32768,
// 32 x 128; fp32 took 76 us against 66.
constexpr int kGatedRounds = 2;
// Registers of a thread, forward and backward: 24 and 16 warps on an SM.
constexpr int kGatedRegs = 80, kGatedBackwardRegs = 120;
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
    int64_t n;  // B * T * H * N
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

// Steps 2 and 3 above: from every lane's pair to the state entering its
// tokens, in `entry`; `carry` goes from the round's entry to its exit.  The S
// parts of a warp's tokens are composed by lane exchange first.  Called by all
// warps of the CTA (cluster).
template <int VEC, int S>
__device__ __forceinline__ void exchange(const GatedPairs<VEC> &sh, int buf, int w, int W, unsigned rank, unsigned C,
                                         float (&A)[VEC], float (&z)[VEC], float (&carry)[VEC], float (&entry)[VEC]) {
    constexpr int LW = 32 / S;
    const int lane = threadIdx.x & 31, ch = lane % LW, sub = lane / LW;
    float ba[VEC], bz[VEC];  // of the parts before this lane's
    if constexpr (S > 1) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
#pragma unroll
            for (int d = 1; d < S; d *= 2) {
                const float pa = __shfl_up_sync(0xffffffffu, A[v], d * LW);
                const float pz = __shfl_up_sync(0xffffffffu, z[v], d * LW);
                if (sub >= d) {
                    z[v] = fmaf(A[v], pz, z[v]);
                    A[v] *= pa;
                }
            }
            ba[v] = __shfl_up_sync(0xffffffffu, A[v], LW);
            bz[v] = __shfl_up_sync(0xffffffffu, z[v], LW);
            if (sub == 0) {
                ba[v] = 1.f;
                bz[v] = 0.f;
            }
        }
    }
    if (S == 1 || sub == S - 1)
#pragma unroll
        for (int v = 0; v < VEC; ++v) sh.warp[buf * W + w][v][ch] = make_float2(A[v], z[v]);
    __syncthreads();
    if (C == 1) {
#pragma unroll 4
        for (int i = 0; i < W; ++i) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                if (i == w) entry[v] = carry[v];
                const float2 p = sh.warp[buf * W + i][v][ch];
                carry[v] = fmaf(p.x, carry[v], p.y);
            }
        }
    } else {
        float pa[VEC], pz[VEC], ta[VEC], tz[VEC];  // of the warps before this one, of all
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            pa[v] = ta[v] = 1.f;
            pz[v] = tz[v] = 0.f;
        }
#pragma unroll 4
        for (int i = 0; i < W; ++i) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                if (i == w) {
                    pa[v] = ta[v];
                    pz[v] = tz[v];
                }
                const float2 p = sh.warp[buf * W + i][v][ch];
                tz[v] = fmaf(p.x, tz[v], p.y);
                ta[v] *= p.x;
            }
        }
        if (S == 1 || sub == 0)
            for (unsigned c = w; c < C; c += W)
#pragma unroll
                for (int v = 0; v < VEC; ++v)
                    store_remote(&sh.cta[buf * C + rank][v][ch], c, make_float2(ta[v], tz[v]));
        cluster_barrier();
#pragma unroll 4
        for (unsigned c = 0; c < C; ++c) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                if (c == rank) entry[v] = carry[v];
                const float2 p = sh.cta[buf * C + c][v][ch];
                carry[v] = fmaf(p.x, carry[v], p.y);
            }
        }
#pragma unroll
        for (int v = 0; v < VEC; ++v) entry[v] = fmaf(pa[v], entry[v], pz[v]);
    }
    if constexpr (S > 1)
#pragma unroll
        for (int v = 0; v < VEC; ++v) entry[v] = fmaf(ba[v], entry[v], bz[v]);
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

struct Yes {
    static constexpr bool value = true;
};
struct No {
    static constexpr bool value = false;
};

// How rows come to shared memory: rows that all start on 16 bytes; rows that
// start anywhere, of an array that starts on 16 bytes; and any array (each
// lane its own channel, 16-bit elements by plain loads).
enum { WIDE = 0, SHIFT = 1, NARROW = 2 };

// A warp's S x L rows of CW channels in shared memory.  The S parts' rows are
// set apart by a row's width, so that lanes of different parts do not meet in
// one bank.
template <typename T, int S, int L, int CW, int COPY>
struct Rows {
    static constexpr int R = S * L;
    static constexpr int PITCH = CW * (int)sizeof(T) + (COPY == SHIFT ? 16 : 0);  // bytes
    static constexpr int PART = L * PITCH + (S > 1 ? CW * (int)sizeof(T) : 0);
    static constexpr int BYTES = S * PART;
    static __device__ __forceinline__ int at(int i) { return S == 1 ? i * PITCH : i / L * PART + i % L * PITCH; }

    // Ask for rows [lo, hi) (FULL: all of them, and all channels) into `to`.
    // Row i starts at element `first` + i * step of `base`, an array of `size`
    // elements, and has `width` channels.
    template <bool FULL>
    static __device__ __forceinline__ void ask(unsigned char *to, const T *base, int64_t size, int64_t first,
                                               int64_t step, int lo, int hi, int width) {
        const int lane = threadIdx.x & 31;
        if constexpr (COPY == WIDE) {
            constexpr int E = 16 / (int)sizeof(T);  // elements a lane
            constexpr int LANES = CW / E;           // lanes a row
            constexpr int ROWS = 32 / LANES;        // rows at once
            const int col = lane % LANES * E;
            int i = lane / LANES;
            const T *p = base + first + i * step + col;
#pragma unroll
            for (int k = 0; k < R / ROWS; ++k, i += ROWS, p += ROWS * step)
                if (FULL || (i >= lo && i < hi && col < width))
                    bring<T, E>(reinterpret_cast<T *>(to + at(i) + col * (int)sizeof(T)), p);
        } else if constexpr (COPY == SHIFT) {
            // pieces of 16 bytes from the one that holds the row's first
            // element; of the array's last piece what is there
            constexpr int E = 16 / (int)sizeof(T);
            constexpr int PIECES = CW / E + 1;
            constexpr int ALL = R * PIECES;
#pragma unroll
            for (int k = 0; k < (ALL + 31) / 32; ++k) {
                const int n = k * 32 + lane, i = n / PIECES, piece = n % PIECES;
                if (n >= ALL || i < lo || i >= hi) continue;
                const int64_t first_of = first + i * step;
                const int64_t from = first_of - (first_of & (E - 1)) + piece * E;
                if (from >= first_of + width) continue;
                const int64_t left = size - from;
                copy_async_part(static_cast<unsigned>(__cvta_generic_to_shared(to + at(i) + piece * 16)), base + from,
                                left < E ? (int)left * (int)sizeof(T) : 16);
            }
        } else {
            static_assert(COPY != NARROW || CW == 32, "a channel a lane");
            const int col = lane < width ? lane : width - 1;  // past the last channel: the last one
            const T *p = base + first + col;
#pragma unroll
            for (int i = 0; i < R; ++i, p += step)
                if (FULL || (i >= lo && i < hi)) bring<T, 1>(reinterpret_cast<T *>(to + at(i)) + lane, p);
        }
    }
    // Byte offset of row i's first element from the start of its row.
    static __device__ __forceinline__ int shift(int64_t first, int64_t step, int i) {
        if constexpr (COPY != SHIFT) return 0;
        constexpr int E = 16 / (int)sizeof(T);
        // the low bits alone: offsets past 32 bits wrap
        return (int)(((unsigned)first + (unsigned)i * (unsigned)step) & (unsigned)(E - 1)) * (int)sizeof(T);
    }
};

// Gates shared by heads: those of a warp's R = S L tokens and up to kGatedHeads
// / S heads of the tile, a few in each lane, one round ahead.
constexpr int kGatedHeads = 8;
template <typename Tin, int S, int L, int ROUNDS>
struct HeadGates {
    static constexpr int R = S * L;
    static constexpr int N = L * kGatedHeads / 32;
    Tin ahead[ROUNDS - 1][N];

    // Make room for the next round's.
    __device__ __forceinline__ void shift() {
#pragma unroll
        for (int k = 0; k + 1 < ROUNDS - 1; ++k)
#pragma unroll
            for (int n = 0; n < N; ++n) ahead[k][n] = ahead[k + 1][n];
    }
    // Token i of head k: at from + i * step + k, where lo <= i < hi.
    __device__ __forceinline__ void ask(const Tin *from, int64_t step, int heads, int lo, int hi) {
        const int lane = threadIdx.x & 31;
        Tin(&last)[N] = ahead[ROUNDS - 2];
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int i = (n * 32 + lane) % R, k = (n * 32 + lane) / R;
            if (n * 32 < heads * R) {  // uniform
                last[n] = from_float<Tin>(1.f);
                if (k < heads && i >= lo && i < hi) last[n] = from[i * step + k];
            }
        }
    }
    // Into shared memory, in fp32: [heads][R].
    __device__ __forceinline__ void give(float *to, int heads) const {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int n = 0; n < N; ++n)
            if (n * 32 + lane < heads * R) to[n * 32 + lane] = to_float(ahead[0][n]);
    }
};

// Shared memory of a warp, in bytes: its rounds of rows, and the gates
// shared by heads.
template <typename Tin, int VEC, int S, bool HEAD, int L, int COPY, bool BACKWARD>
struct GatedStage {
    static constexpr int CW = 32 / S * VEC;
    using In = Rows<Tin, S, L, CW, COPY>;
    using Wide = Rows<float, S, L, CW, COPY>;
    static constexpr int X = 0;                                         // rows of x, or of g
    static constexpr int H = X + (BACKWARD ? Wide::BYTES : In::BYTES);  // rows of h
    static constexpr int F = H + (BACKWARD ? Wide::BYTES : 0);          // rows of f
    static constexpr int BYTES = F + (HEAD ? 0 : In::BYTES);
    static constexpr int ROUNDS = kGatedRounds;
    static constexpr int GATES = ROUNDS * BYTES;
    static constexpr int WARP = GATES + (HEAD ? L * kGatedHeads * 4 : 0);
    static_assert(BYTES % 16 == 0 && WARP % 16 == 0, "16-byte pieces");
};

// Grid: tiles x C CTAs of 32 x W threads.  Dynamic shared memory: GatedStage of
// each warp, then the pairs.
template <typename Tin, int VEC, int S, bool HEAD, int L, int COPY>
__global__ void __maxnreg__(kGatedRegs)
kla_gated_forward_kernel(const GatedParams prm) {
    using Stage = GatedStage<Tin, VEC, S, HEAD, L, COPY, false>;
    using In = typename Stage::In;
    using Pairs = typename GatedPairs<VEC>::Pairs;
    constexpr int LW = 32 / S, R = S * L;
    extern __shared__ __align__(16) unsigned char shared[];
    const GatedTiles &g = prm.g;
    const int lane = threadIdx.x & 31, ch = lane % LW, sub = lane / LW;
    const int w = threadIdx.x >> 5;
    const int W = blockDim.x >> 5;
    const unsigned C = cluster_size();
    const unsigned rank = cluster_rank();
    const TileAt at = tile_at(g, blockIdx.x / C, Stage::CW);
    const int64_t c = at.c0 + ch * VEC;
    const bool valid = c < at.end;
    const int width = at.end - at.c0 < Stage::CW ? (int)(at.end - at.c0) : Stage::CW;
    const int64_t row0 = at.b * g.T;
    const int64_t head0 = HEAD ? at.c0 / g.N : 0;
    const int heads = HEAD ? (int)((at.c0 + width - 1) / g.N - head0) + 1 : 0;
    const Tin *const f = static_cast<const Tin *>(prm.f);
    const Tin *const x = static_cast<const Tin *>(prm.x);
    float *const h = prm.h + ch * VEC;
    unsigned char *const mine = shared + w * Stage::WARP;
    float *const gates = reinterpret_cast<float *>(mine + Stage::GATES);
    Pairs *const pairs = reinterpret_cast<Pairs *>(shared + W * Stage::WARP);
    const GatedPairs<VEC> sh{pairs, pairs + 2 * W};

    float carry[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) carry[v] = prm.h0 && valid ? prm.h0[at.b * g.HN + c + v] : 0.f;

    // where this warp is in a round: the first element of its rows, their
    // gates, and the tokens from there to the end (none when not positive)
    const int64_t t0 = (int64_t)(rank * W + w) * R, round = (int64_t)C * W * R;
    const int64_t rounds = (g.T + round - 1) / round;
    const bool whole = width == Stage::CW;
    HeadGates<Tin, S, L, Stage::ROUNDS> ahead;
    auto ask_rows = [&](auto full, int buf, int64_t first, const Tin *gate_rows, int64_t left) {
        constexpr bool FULL = decltype(full)::value;
        const int64_t hn = opaque(g.HN);
        const int nv = FULL ? R : (int)(left < R ? left : R);
        unsigned char *const to = mine + buf * Stage::BYTES;
        In::template ask<FULL>(to + Stage::X, x, prm.n, first, hn, 0, nv, width);
        if constexpr (HEAD)
            ahead.ask(gate_rows, g.H, heads, 0, nv);
        else
            In::template ask<FULL>(to + Stage::F, f, prm.n, first, hn, 0, nv, width);
        copies_commit();
    };
    // FULL rounds of a warp, all of whose tokens and channels are there, take
    // code without their tests (a third of the instructions)
    auto ask = [&](int buf, int64_t first, const Tin *gate_rows, int64_t left) {
        whole && left >= R ? ask_rows(Yes{}, buf, first, gate_rows, left) : ask_rows(No{}, buf, first, gate_rows, left);
    };
    auto run = [&](auto full_, int buf, int parity, int64_t first, int64_t left_of_warp) {
        constexpr bool FULL = decltype(full_)::value;
        const int64_t hn = opaque(g.HN);
        const int64_t left = left_of_warp - sub * L;  // of this lane's tokens
        const int nv = FULL ? L : (int)(left < L ? left : L);
        const unsigned char *const from = mine + buf * Stage::BYTES;
        // tokens that are not there leave the state as it is: f = 1, x = 0
        const int at_lane = sub * In::PART + ch * VEC * (int)sizeof(Tin);
        [[maybe_unused]] const float *const gate = gates + (HEAD && valid ? (c / g.N - head0) * R : 0) + sub * L;
        auto pack = [&](int part, int i) {
            return pack_at<Tin, VEC>(reinterpret_cast<const Tin *>(from + part + at_lane + i * In::PITCH +
                                                                   In::shift(first, hn, sub * L + i)));
        };
        auto x_at = [&](int i) { return FULL || i < nv ? pack(Stage::X, i) : pack_of<Tin, VEC>(0.f); };
        auto f_at = [&](int i, float (&to)[VEC]) {
            if constexpr (HEAD) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) to[v] = pack_at<float, 4>(gate + i / 4 * 4).v[i % 4];
            } else {
                const Pack<Tin, VEC> p = FULL || i < nv ? pack(Stage::F, i) : pack_of<Tin, VEC>(1.f);
#pragma unroll
                for (int v = 0; v < VEC; ++v) to[v] = to_float(p.v[v]);
            }
        };
        float A[VEC], z[VEC], entry[VEC], fi[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            A[v] = 1.f;
            z[v] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const Pack<Tin, VEC> xi = x_at(i);
            f_at(i, fi);
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                A[v] *= fi[v];
                z[v] = fmaf(fi[v], z[v], to_float(xi.v[v]));
            }
        }
        exchange<VEC, S>(sh, parity, w, W, rank, C, A, z, carry, entry);
        float *ht = h + first + sub * L * hn;
#pragma unroll
        for (int i = 0; i < L; ++i, ht += hn) {
            const Pack<Tin, VEC> xi = x_at(i);
            f_at(i, fi);
            Pack<float, VEC> o;
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                entry[v] = fmaf(fi[v], entry[v], to_float(xi.v[v]));
                o.v[v] = entry[v];
            }
            if (FULL || (valid && i < nv)) store_cs<float, VEC>(ht, o);
        }
    };

    int64_t first = (row0 + t0) * g.HN + at.c0, left = g.T - t0;
    int64_t first_asked = first, left_asked = left;
    const Tin *gate_rows = HEAD ? f + (row0 + t0) * g.H + head0 : nullptr;
    const int64_t first_step = round * g.HN, gate_step = HEAD ? round * g.H : 0;
    // the rounds asked for are `asked` ahead of the present one
    int64_t asked = 0;
    int to_buf = 0;
    auto ask_next = [&]() {
        if (HEAD) ahead.shift();
        if (asked < rounds) {
            ask(to_buf, first_asked, gate_rows, left_asked);
            first_asked += first_step;
            gate_rows += gate_step;
            left_asked -= round;
        } else {
            copies_commit();
        }
        ++asked;
        to_buf = to_buf == Stage::ROUNDS - 1 ? 0 : to_buf + 1;
    };
#pragma unroll
    for (int k = 0; k < Stage::ROUNDS - 1; ++k) ask_next();
    if (C > 1) cluster_barrier();  // every rank runs before its shared memory is written
    int buf = 0;
#pragma unroll 1
    for (int64_t r = 0; r < rounds; ++r, first += first_step, left -= round) {
        __syncwarp();  // the stage to fill and the gates have been read
        if (HEAD) ahead.give(gates, heads);
        ask_next();
        copies_wait<Stage::ROUNDS - 1>();
        __syncwarp();
        // all warps of a CTA take the same branch: its barriers stand in both
        whole && left >= (W - w) * R ? run(Yes{}, buf, (int)(r & 1), first, left)
                                     : run(No{}, buf, (int)(r & 1), first, left);
        buf = buf == Stage::ROUNDS - 1 ? 0 : buf + 1;
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
    int64_t n;       // B * T * H * N
    int group;       // lanes that share a head (HEAD): 32 / S, or N / VEC below it
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
template <typename Tin, int VEC, int S, bool HEAD, int L, int COPY>
__global__ void __maxnreg__(kGatedBackwardRegs)
kla_gated_backward_kernel(const GatedBackwardParams prm) {
    using Stage = GatedStage<Tin, VEC, S, HEAD, L, COPY, true>;
    using In = typename Stage::In;
    using Wide = typename Stage::Wide;
    using Pairs = typename GatedPairs<VEC>::Pairs;
    constexpr int LW = 32 / S, R = S * L;
    extern __shared__ __align__(16) unsigned char shared[];
    const GatedTiles &g = prm.g;
    const int lane = threadIdx.x & 31, ch = lane % LW, sub = lane / LW;
    const int w = threadIdx.x >> 5;
    const int W = blockDim.x >> 5;
    const unsigned C = cluster_size();
    const unsigned rank = cluster_rank();
    const TileAt at = tile_at(g, blockIdx.x / C, Stage::CW);
    const int64_t c = at.c0 + ch * VEC;
    const bool valid = c < at.end;
    const int width = at.end - at.c0 < Stage::CW ? (int)(at.end - at.c0) : Stage::CW;
    const int64_t row0 = at.b * g.T;
    const int64_t head0 = HEAD ? at.c0 / g.N : 0;
    const int heads = HEAD ? (int)((at.c0 + width - 1) / g.N - head0) + 1 : 0;
    const Tin *const f = static_cast<const Tin *>(prm.f);
    const float *const h = prm.gf ? prm.h : nullptr;
    const float *const h0 = prm.h0 && valid ? prm.h0 + at.b * g.HN + c : nullptr;
    Tin *const gx = static_cast<Tin *>(prm.gx);
    Tin *const gf = HEAD ? nullptr : static_cast<Tin *>(prm.gf);
    unsigned char *const mine = shared + w * Stage::WARP;
    float *const gates = reinterpret_cast<float *>(mine + Stage::GATES);
    Pairs *const pairs = reinterpret_cast<Pairs *>(shared + W * Stage::WARP);
    const GatedPairs<VEC> sh{pairs, pairs + 2 * W};

    float carry[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) carry[v] = 0.f;

    // as in the forward kernel, in reverse time: the first of a warp's rows is
    // its last token's, and `left` counts the tokens from there down to the first
    const int64_t t0 = (int64_t)(rank * W + w) * R, round = (int64_t)C * W * R;
    const int64_t rounds = (g.T + round - 1) / round;
    const bool whole = width == Stage::CW;
    HeadGates<Tin, S, L, Stage::ROUNDS> ahead;
    // of token t: g; h of token t - 1 (none before the first); f of token t + 1
    // (none after the last)
    auto ask_rows = [&](auto full, int buf, int64_t first, const Tin *gate_rows, int64_t left) {
        constexpr bool FULL = decltype(full)::value;
        const int64_t hn = opaque(g.HN);
        const int nv = FULL ? R : (int)(left < R ? left : R);
        const int lo = FULL || left < g.T ? 0 : 1, before = FULL ? R : (int)(left - 1 < R ? left - 1 : R);
        unsigned char *const to = mine + buf * Stage::BYTES;
        Wide::template ask<FULL>(to + Stage::X, prm.gh, prm.n, first, -hn, 0, nv, width);
        if (h) Wide::template ask<FULL>(to + Stage::H, h, prm.n, first - hn, -hn, 0, before, width);
        if constexpr (HEAD)
            ahead.ask(gate_rows, -g.H, heads, lo, nv);
        else
            In::template ask<FULL>(to + Stage::F, f, prm.n, first + hn, -hn, lo, nv, width);
        copies_commit();
    };
    // FULL: as in the forward kernel, with the tokens before and after
    auto ask = [&](int buf, int64_t first, const Tin *gate_rows, int64_t left) {
        whole && left < g.T && left > R ? ask_rows(Yes{}, buf, first, gate_rows, left) : ask_rows(No{}, buf, first, gate_rows, left);
    };
    auto run = [&](auto full_, int buf, int parity, int64_t first, int64_t left_of_warp) {
        constexpr bool FULL = decltype(full_)::value;
        const int64_t hn = opaque(g.HN);
        const int64_t tl = left_of_warp - 1 - sub * L;  // this lane's last token
        const int nv = FULL ? L : (int)(tl + 1 < L ? tl + 1 : L);
        [[maybe_unused]] const bool at_end = !FULL && left_of_warp == g.T && sub == 0;  // its last token is the sequence's
        const unsigned char *const from = mine + buf * Stage::BYTES;
        [[maybe_unused]] const int at_in = sub * In::PART + ch * VEC * (int)sizeof(Tin);
        const int at_wide = sub * Wide::PART + ch * VEC * 4;
        [[maybe_unused]] const float *const gate = gates + (HEAD && valid ? (c / g.N - head0) * R : 0) + sub * L;
        auto wide = [&](int part, int64_t row, int i) {
            return pack_at<float, VEC>(reinterpret_cast<const float *>(from + part + at_wide + i * Wide::PITCH +
                                                                       Wide::shift(row, -hn, sub * L + i)));
        };
        auto g_at = [&](int i) { return FULL || i < nv ? wide(Stage::X, first, i) : pack_of<float, VEC>(0.f); };
        auto f_at = [&](int i, float (&to)[VEC]) {
            if constexpr (HEAD) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) to[v] = pack_at<float, 4>(gate + i / 4 * 4).v[i % 4];
            } else {
                Pack<Tin, VEC> p = pack_of<Tin, VEC>(1.f);
                if (FULL || (i < nv && !(at_end && i == 0)))
                    p = pack_at<Tin, VEC>(reinterpret_cast<const Tin *>(from + Stage::F + at_in + i * In::PITCH +
                                                                        In::shift(first + hn, -hn, sub * L + i)));
#pragma unroll
                for (int v = 0; v < VEC; ++v) to[v] = to_float(p.v[v]);
            }
        };
        float A[VEC], z[VEC], entry[VEC], fi[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            A[v] = 1.f;
            z[v] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const Pack<float, VEC> gi = g_at(i);
            f_at(i, fi);
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                A[v] *= fi[v];
                z[v] = fmaf(fi[v], z[v], gi.v[v]);
            }
        }
        exchange<VEC, S>(sh, parity, w, W, rank, C, A, z, carry, entry);
        GroupSums<L> sum;  // HEAD: this lane's share of the shared gate's gradient
        const int64_t out = first - sub * L * hn + ch * VEC;
        Tin *gxt = gx + out;
        Tin *gft = gf + out;
#pragma unroll
        for (int i = 0; i < L; ++i, gxt -= hn, gft -= hn) {
            const Pack<float, VEC> gi = g_at(i);
            f_at(i, fi);
            Pack<float, VEC> before = pack_of<float, VEC>(0.f);
            if (h) {
                if (FULL || (i < nv && i < tl))
                    before = wide(Stage::H, first - hn, i);
                else if (i < nv && h0)
#pragma unroll
                    for (int v = 0; v < VEC; ++v) before.v[v] = h0[v];
            }
            Pack<Tin, VEC> ox, of;
            sum.x[i] = 0.f;
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                entry[v] = fmaf(fi[v], entry[v], gi.v[v]);
                ox.v[v] = from_float<Tin>(entry[v]);
                if (HEAD)
                    sum.x[i] = fmaf(entry[v], before.v[v], sum.x[i]);
                else
                    of.v[v] = from_float<Tin>(entry[v] * before.v[v]);
            }
            if (HEAD && !FULL && !valid) sum.x[i] = 0.f;
            if (FULL || (valid && i < nv)) {
                if (gx) store_cs<Tin, VEC>(gxt, ox);
                if (!HEAD && gf) store_cs<Tin, VEC>(gft, of);
            }
        }
        if (!FULL && prm.gh0 && nv > 0 && tl + 1 == nv && valid) {  // this lane ended at token 0
            const Tin *const f0 = f + (HEAD ? row0 * g.H + c / g.N : row0 * g.HN + c);
#pragma unroll
            for (int v = 0; v < VEC; ++v)
                prm.gh0[at.b * g.HN + c + v] = to_float(f0[HEAD ? 0 : v]) * entry[v];
        }
        if (HEAD && prm.gf) {
            sum.run(prm.group);
            const int64_t k = at.c0 + (ch & ~(prm.group - 1)) * VEC;  // the group's first channel
            if (sum.writes && (FULL || k < at.end)) {
                const int64_t head = k / g.N;
                const int64_t at_gate = (row0 + tl - sum.first) * g.H + head;
                float *const part =
                    prm.partial ? prm.partial + (at.c0 - head * g.N) / Stage::CW * prm.gates + at_gate : nullptr;
                Tin *const gate_out = static_cast<Tin *>(prm.gf) + at_gate;
#pragma unroll
                for (int i = 0; i < L; ++i) {
                    if (i >= sum.count) break;
                    if (!FULL && sum.first + i >= nv) break;
                    if (part)
                        part[-i * g.H] = sum.x[i];
                    else
                        gate_out[-i * g.H] = from_float<Tin>(sum.x[i]);
                }
            }
        }
    };

    int64_t first = (row0 + g.T - 1 - t0) * g.HN + at.c0, left = g.T - t0;
    int64_t first_asked = first, left_asked = left;
    const Tin *gate_rows = HEAD ? f + (row0 + g.T - t0) * g.H + head0 : nullptr;
    const int64_t first_step = -round * g.HN, gate_step = HEAD ? -round * g.H : 0;
    // the rounds asked for are `asked` ahead of the present one
    int64_t asked = 0;
    int to_buf = 0;
    auto ask_next = [&]() {
        if (HEAD) ahead.shift();
        if (asked < rounds) {
            ask(to_buf, first_asked, gate_rows, left_asked);
            first_asked += first_step;
            gate_rows += gate_step;
            left_asked -= round;
        } else {
            copies_commit();
        }
        ++asked;
        to_buf = to_buf == Stage::ROUNDS - 1 ? 0 : to_buf + 1;
    };
#pragma unroll
    for (int k = 0; k < Stage::ROUNDS - 1; ++k) ask_next();
    if (C > 1) cluster_barrier();
    int buf = 0;
#pragma unroll 1
    for (int64_t r = 0; r < rounds; ++r, first += first_step, left -= round) {
        __syncwarp();  // the stage to fill and the gates have been read
        if (HEAD) ahead.give(gates, heads);
        ask_next();
        copies_wait<Stage::ROUNDS - 1>();
        __syncwarp();
        // all warps of a CTA take the same branch: its barriers stand in both
        whole && left + w * R < g.T && left > (W - w) * R ? run(Yes{}, buf, (int)(r & 1), first, left)
                                                          : run(No{}, buf, (int)(r & 1), first, left);
        buf = buf == Stage::ROUNDS - 1 ? 0 : buf + 1;
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
