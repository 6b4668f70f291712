// kla_rotary.cuh -- the RMS norm of queries and keys for each head with the
// position rotation in the same pass, its backward pass, and the rotation
// alone (sm_100a).
//
// For a row x of D elements (one head of one token at position s), with a
// weight w (1 where there is none):
//
//   r = 1 / sqrt(mean(x^2) + eps),   n_d = w_d x_d r,   y = R(s) n,
//
// where R(s) turns the first rot elements pairwise: pair i, (n_i,
// n_{i + rot/2}) or the neighbours (n_2i, n_{2i+1}), by the angle s
// inv_freq_i, times `scale`; the other elements pass.  Without the norm, n =
// x.  The inverse rotation (angle negated, same scale) is also the transpose,
// so with g' = R(s)^T dL/dy and u = w g':
//
//   dL/dw_d = sum over rows of g'_d x_d r,
//   dL/dx_d = r (u_d - x_d r^2 mean(u x)).
//
// Every element is read and written once, so HBM is the floor: 52 us for B=4,
// T=4096, 32 + 8 heads of 128 in bf16, of which the norm with the rotation
// takes 69 us (4.9 TB/s, 0.75 of a copy), its backward pass 103 (0.76), the
// rotation of the queries alone 49 (0.84); fp32 rows reach 0.85.  Instructions
// come next to it (0.58 to 0.67 of the issue slots): conversions, the products
// with w and r, the turns and the exchanges of the sum of squares are a few
// instructions for each pair of elements, which 4 bytes of traffic in bf16
// leave little time for.  Rows of a few elements (D = 16: 0.57) pay for the
// row's own work.  A
// row belongs to a group of lanes (a power of two, at most a warp), and a
// warp to one token, or to several where a token's heads do not fill it: its
// lanes form the tokens' cos and sin together, in shared memory, and each
// lane then keeps those of its own elements in registers while its group goes
// through its heads one after another.  Rows come through a ring in shared
// memory by asynchronous copies, RING - 1 of them ahead; each lane copies and
// reads its own vectors only, so that there is nothing to wait for but its
// own copies.  The sum of squares is a few lane exchanges.  Warps share
// nothing (but for the weights' gradients, added up at the end).  Arithmetic
// is in packed pairs of fp32 where it can be.
//
// A lane holds two vectors of VEC elements (or UPL times that): one from each
// half of the rotated part, or, with neighbouring pairs, any two; both members
// of a pair are in the same lane.  (Where the halves do not allow vectors, as
// when their length is odd, wider vectors whose lanes found the partners in
// shared memory took 1.2 to 2.4 times as long as narrow ones.)
//
// Angles: the product of position and frequency in 64 bits, reduced there to
// a fraction of a turn, so that far positions lose little (at 10^9 less than
// 4e-7 of a radian); the rounding of that fraction to 32 bits is given back to
// first order.
#pragma once

#include "kla_mixer.h"

namespace kla_mixer {

constexpr int kRotaryThreads = 256;
// CTAs of an SM, by the registers that they leave a thread: 80 forward, 128
// backward (the gradient's rows, and the weights' sums).  B=4, T=4096, 32 + 8
// heads of 128, bf16: forward 69 us with 3, 71 with 2, 92 with 4 (spills);
// backward 103 us with 2, 144 with 1, 218 with 3 (spills).
constexpr int kRotaryCtas = 3, kRotaryBackwardCtas = 2;
// Rows in flight and in use (up to 16 elements a lane): forward 69 us with 3,
// 75 with 2, 69 with 4; backward 103, 109 and 105.
constexpr int kRotaryRing = 3;

__host__ __device__ constexpr int rotary_resident(int vec, int upl, bool backward) {
    return vec * upl > 8 ? 1 : backward || upl > 1 ? kRotaryBackwardCtas : kRotaryCtas;
}

struct RotaryTensor {
    const void *x, *gy;      // input; gradient of the output (backward)
    void *y;                 // output; gradient of the input (backward)
    const float *w;          // weight or null
    float *partial;          // [CTAs of this tensor][D]: sums of the weight's gradient, or null
    int64_t sb, st, sh;      // strides of x in elements; y and gy are dense
    int heads;
    int abreast;             // heads of a token that a warp takes at once (a power of two)
    int splits;              // warps that share a token's heads
    unsigned ctas;           // of this tensor
};

struct RotaryParams {
    RotaryTensor t[2];
    const double *inv_freq;
    const int64_t *positions;  // or null: position0 + t
    int64_t position_stride, position0;
    int64_t T, tokens;         // tokens = B * T
    float eps, scale, sign;    // sign of the sine: -1 for the inverse
    int D, half, interleaved;
    int lanes;                 // of a row
    int units;                 // of a row: pairs of VEC-element vectors
};

// scale (cos, sign sin) of a position times a frequency.
__device__ __forceinline__ float2 turn(const RotaryParams &prm, double at, int pair) {
    const double turns = at * (prm.inv_freq[pair] * 0.15915494309189533577);  // 1 / 2 pi
    const double r = turns - rint(turns);
    const float f = (float)r;
    float s, c;
    sincospif(2.f * f, &s, &c);
    const float d = (float)(r - (double)f) * 6.28318530717958648f;
    return make_float2(prm.scale * fmaf(-s, d, c), prm.sign * prm.scale * fmaf(c, d, s));
}

// Elements of unit u: two vectors of VEC at a and b (b >= D: there is none).
// The units' first vectors lie side by side, and so do their second ones:
// what the lanes of a group ask for at once is contiguous.
struct Unit {
    int a, b;
};
template <int VEC>
__device__ __forceinline__ Unit unit_at(const RotaryParams &prm, int u) {
    const int turned = prm.interleaved ? 0 : prm.half / VEC;  // units of the two halves
    if (u < turned) return Unit{u * VEC, prm.half + u * VEC};
    if (VEC == 1 && prm.interleaved) return Unit{2 * u, 2 * u + 1};     // a pair
    const int k = u - turned, rest = prm.units - turned;
    return Unit{2 * turned * VEC + k * VEC, 2 * turned * VEC + (rest + k) * VEC};
}

// A lane's vector of VEC elements in fp32: packed pairs (VEC = 1: the second
// of the pair is not used).
template <int VEC>
struct Lane {
    static constexpr int N = VEC > 1 ? VEC / 2 : 1;
    float2 v[N];
};

template <int VEC>
__device__ __forceinline__ Lane<VEC> unpack(const float *p) {
    Lane<VEC> x;
    const Pack<float, VEC> r = *reinterpret_cast<const Pack<float, VEC> *>(p);
#pragma unroll
    for (int j = 0; j < Lane<VEC>::N; ++j) x.v[j] = make_float2(r.v[VEC > 1 ? 2 * j : 0], VEC > 1 ? r.v[2 * j + 1] : 0.f);
    return x;
}
template <int VEC>
__device__ __forceinline__ Lane<VEC> unpack(const __nv_bfloat16 *p) {
    Lane<VEC> x;
    if constexpr (VEC == 1) {
        x.v[0] = make_float2(__bfloat162float(*p), 0.f);
    } else {
        const Pack<unsigned, VEC / 2> r = *reinterpret_cast<const Pack<unsigned, VEC / 2> *>(p);
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j)  // two bf16 a word: their bits are the upper halves of fp32
            x.v[j] = make_float2(__uint_as_float(r.v[j] << 16), __uint_as_float(r.v[j] & 0xffff0000u));
    }
    return x;
}

template <int VEC>
__device__ __forceinline__ void store_lane(float *p, const Lane<VEC> &x) {
    Pack<float, VEC> r;
#pragma unroll
    for (int j = 0; j < VEC; ++j) r.v[j] = j & 1 ? x.v[j / 2].y : x.v[j / 2].x;
    store_cs<float, VEC>(p, r);
}
template <int VEC>
__device__ __forceinline__ void store_lane(__nv_bfloat16 *p, const Lane<VEC> &x) {
    if constexpr (VEC == 1) {
        *p = __float2bfloat16_rn(x.v[0].x);
    } else {
        Pack<__nv_bfloat162, VEC / 2> r;
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) r.v[j] = __float22bfloat162_rn(x.v[j]);
        store_cs<__nv_bfloat162, VEC / 2>(reinterpret_cast<__nv_bfloat162 *>(p), r);
    }
}

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// What a lane's elements are turned by, for one token: y_a = A a + B b, y_b =
// C a + D b for the pairs (a_j, b_j) of two halves; for neighbours the same of
// each (x_2i, x_2i+1), the pairs of the first vector, then of the second.
// FOLD: with the weights in them; else D = A.
template <int VEC, bool FOLD>
struct Turns {
    static constexpr int N = Lane<VEC>::N;
    float2 A[N], B[N], C[N], D[FOLD ? N : 1];

    // From the token's table of `half` pairs and the weights of a and b.
    __device__ __forceinline__ void take(const RotaryParams &prm, const float2 *table, const Unit &k,
                                         const Lane<VEC> &wa, const Lane<VEC> &wb) {
        auto set = [](float2 &to, int j, float x) {
            if (VEC == 1)  // a pair's second half is not used: zeros, which add nothing to a sum
                to = make_float2(x, 0.f);
            else if (j & 1)
                to.y = x;
            else
                to.x = x;
        };
        auto get = [](const Lane<VEC> &w, int j) { return j & 1 ? w.v[j / 2].y : w.v[j / 2].x; };
        const bool neighbours = VEC > 1 && prm.interleaved;
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            const int pair = !prm.interleaved ? k.a + j : VEC == 1 ? k.a / 2 : j < N ? k.a / 2 + j : k.b / 2 + j - N;
            const float2 t = pair < prm.half ? table[pair] : make_float2(1.f, 0.f);
            const float2 w = j < N ? wa.v[j % N] : wb.v[j % N];
            const float first = FOLD ? neighbours ? w.x : get(wa, j) : 1.f;
            const float second = FOLD ? neighbours ? w.y : get(wb, j) : 1.f;
            set(A[j / 2], j, first * t.x);
            set(B[j / 2], j, -second * t.y);
            set(C[j / 2], j, first * t.y);
            if constexpr (FOLD) set(D[j / 2], j, second * t.x);
        }
    }

    // Turn a lane's elements in place.
    __device__ __forceinline__ void apply(const RotaryParams &prm, const Unit &k, Lane<VEC> &a, Lane<VEC> &b) const {
        auto d = [&](int j) { return FOLD ? D[j % (FOLD ? N : 1)] : A[j]; };
        if (VEC == 1 || !prm.interleaved) {
            if (k.a < (prm.interleaved ? 2 * prm.half : prm.half)) {
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const float2 u = a.v[j], v = b.v[j];
                    a.v[j] = __ffma2_rn(u, A[j], __fmul2_rn(v, B[j]));
                    b.v[j] = __ffma2_rn(u, C[j], __fmul2_rn(v, d(j)));
                }
            } else if (FOLD) {
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    a.v[j] = __fmul2_rn(a.v[j], A[j]);
                    b.v[j] = __fmul2_rn(b.v[j], d(j));
                }
            }
        } else {
            auto pick = [](float2 from, int j) { return j & 1 ? from.y : from.x; };
            auto one = [&](float2 &x, int pair, int j) {
                const float pa = pick(A[j / 2], j), pd = pick(d(j / 2), j);
                if (pair < prm.half)
                    x = make_float2(fmaf(x.x, pa, x.y * pick(B[j / 2], j)), fmaf(x.x, pick(C[j / 2], j), x.y * pd));
                else if (FOLD)
                    x = make_float2(x.x * pa, x.y * pd);
            };
#pragma unroll
            for (int j = 0; j < N; ++j) {
                one(a.v[j], k.a / 2 + j, j);
                one(b.v[j], k.b / 2 + j, N + j);
            }
        }
    }
};

__device__ __forceinline__ float row_sum(float x, int lanes) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        if (o < lanes) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Shared memory of a warp: the ring (vector by vector, lane by lane), and the
// table.
template <typename T, int VEC, int UPL, bool BACKWARD>
struct RotaryShared {
    static constexpr int BYTES = VEC * (int)sizeof(T);  // of a vector
    static constexpr bool ASYNC = BYTES >= 4;
    static constexpr int VECTORS = 2 * UPL * (BACKWARD ? 2 : 1);  // of a lane and row
    static constexpr int RING = VEC * UPL > 8 ? 2 : kRotaryRing;
    static constexpr int SLOT = VECTORS * 32 * BYTES;
    static constexpr int TABLE_OFF = RING * SLOT;
    __host__ __device__ static constexpr int warp_bytes(int table_pairs) {
        return TABLE_OFF + (table_pairs * 8 + 15) / 16 * 16;
    }
};

// Grid: the CTAs of the first tensor, then those of the second.  An item is
// 32 / lanes / abreast tokens and one of `splits` shares of their heads; the
// warps of a tensor's CTAs take items in turn.  UPL: units per lane.
template <typename T, int VEC, int UPL, bool NORM, bool BACKWARD>
__global__ void __launch_bounds__(kRotaryThreads, rotary_resident(VEC, UPL, BACKWARD))
kla_rotary_kernel(const RotaryParams prm, const int table_pairs) {
    using Sh = RotaryShared<T, VEC, UPL, BACKWARD>;
    using Row = Lane<VEC>;
    constexpr int N = Row::N;
    constexpr bool FOLD = NORM && !BACKWARD;
    extern __shared__ __align__(16) unsigned char shared[];
    const bool second = blockIdx.x >= prm.t[0].ctas;
    const RotaryTensor x = second ? prm.t[1] : prm.t[0];
    const unsigned cta = blockIdx.x - (second ? prm.t[0].ctas : 0u);
    const int warp = threadIdx.x >> 5;
    const int lanes = prm.lanes;
    const int lane = threadIdx.x & (lanes - 1);
    const int group = (threadIdx.x & 31) / lanes;   // of the warp
    const int abreast = x.abreast;
    const int tokens_abreast = 32 / lanes / abreast;
    const int sub_token = group / abreast;
    const int sub_head = group & (abreast - 1);
    unsigned char *const mine = shared + warp * Sh::warp_bytes(table_pairs);
    T *const ring = reinterpret_cast<T *>(mine) + (threadIdx.x & 31) * VEC;  // this lane's first vector
    const unsigned ring_at = static_cast<unsigned>(__cvta_generic_to_shared(ring));
    float2 *const table = reinterpret_cast<float2 *>(mine + Sh::TABLE_OFF) + sub_token * prm.half;

    Unit unit[UPL];
    Row ga[UPL], gb[UPL];      // the weight's gradient over this lane's rows
    bool on[UPL], two[UPL];
#pragma unroll
    for (int u = 0; u < UPL; ++u) {
        const int k = lane + u * lanes;
        unit[u] = unit_at<VEC>(prm, k);
        on[u] = k < prm.units;
        two[u] = on[u] && unit[u].b < prm.D;
#pragma unroll
        for (int j = 0; j < N; ++j) ga[u].v[j] = gb[u].v[j] = both(0.f);
    }
    // the weight at a lane's elements
    auto weights = [&](int u, Row &wa, Row &wb) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            wa.v[j] = wb.v[j] = both(1.f);
            if (NORM && x.w) {
                if (on[u]) wa.v[j].x = __ldg(x.w + unit[u].a + 2 * j);
                if (two[u]) wb.v[j].x = __ldg(x.w + unit[u].b + 2 * j);
                if (VEC > 1 && on[u]) wa.v[j].y = __ldg(x.w + unit[u].a + 2 * j + 1);
                if (VEC > 1 && two[u]) wb.v[j].y = __ldg(x.w + unit[u].b + 2 * j + 1);
            }
        }
    };
    Row wa[BACKWARD ? UPL : 1], wb[BACKWARD ? UPL : 1];
    if constexpr (BACKWARD) {
#pragma unroll
        for (int u = 0; u < UPL; ++u) weights(u, wa[u], wb[u]);
    }
    // zeros where no row will be read: vectors without elements, rows past the last
#pragma unroll
    for (int i = 0; i < Sh::RING * Sh::VECTORS; ++i)
        *reinterpret_cast<typename Raw<Sh::BYTES>::type *>(ring + i * 32 * VEC) = {};

    const float inv_d = 1.f / (float)prm.D;
    const int head_step = x.splits * abreast;
    const int turns = (x.heads + head_step - 1) / head_step;  // rows of a group and item
    const int64_t step = (int64_t)head_step * x.sh;
    const int dense_step = head_step * prm.D;
    const int last = x.heads - 1;
    const int64_t shares = (prm.tokens + tokens_abreast - 1) / tokens_abreast;
    const unsigned warps = x.ctas * (kRotaryThreads / 32);
    const unsigned me = cta * (kRotaryThreads / 32) + warp;

    int split = (int)(me % (unsigned)x.splits);
#pragma unroll 1
    for (int64_t share = me / (unsigned)x.splits; share < shares;) {
        const int64_t first = share * tokens_abreast + sub_token;
        const bool have = first < prm.tokens;
        const int64_t token = have ? first : prm.tokens - 1;
        const int64_t b = prm.tokens <= 0xffffffffll ? (int64_t)((unsigned)token / (unsigned)prm.T) : token / prm.T;
        const int64_t t = token - b * prm.T;
        int head = split * abreast + sub_head;
        const T *const in = static_cast<const T *>(x.x) + b * x.sb + t * x.st;
        const T *const gin = static_cast<const T *>(x.gy) + token * x.heads * prm.D;
        T *py = static_cast<T *>(x.y) + (token * x.heads + head) * prm.D;

        // rows past the last are not read (their slot keeps what it held) and not stored
        int ahead = head;
        unsigned slot = 0;
        const T *px = in + head * x.sh;
        const T *pg = gin + head * prm.D;
        auto fetch = [&]() {
            if (ahead <= last) {
                auto copy = [&](int vector, const T *from) {
                    if constexpr (Sh::ASYNC)
                        copy_async<Sh::BYTES>(ring_at + slot + vector * 32 * Sh::BYTES, from);
                    else
                        ring[(slot / Sh::BYTES) + vector * 32 * VEC] = *from;
                };
#pragma unroll
                for (int u = 0; u < UPL; ++u) {
                    if (on[u]) copy(2 * u, px + unit[u].a);
                    if (two[u]) copy(2 * u + 1, px + unit[u].b);
                    if constexpr (BACKWARD) {
                        if (on[u]) copy(2 * (UPL + u), pg + unit[u].a);
                        if (two[u]) copy(2 * (UPL + u) + 1, pg + unit[u].b);
                    }
                }
            }
            ahead += head_step;
            px += step;
            pg += dense_step;
            slot = slot == (Sh::RING - 1) * Sh::SLOT ? 0 : slot + Sh::SLOT;
        };
#pragma unroll
        for (int i = 0; i < Sh::RING - 1; ++i) {
            if (i < turns) fetch();
            copies_commit();
        }
        Turns<VEC, FOLD> turn_of[UPL];
        if (prm.half > 0) {
            __syncwarp();
            const double at = (double)(prm.positions ? prm.positions[b * prm.position_stride + t] : prm.position0 + t);
            for (int i = sub_head * lanes + lane; i < prm.half; i += abreast * lanes) table[i] = turn(prm, at, i);
            __syncwarp();
        }
#pragma unroll
        for (int u = 0; u < UPL; ++u) {
            Row pa, pb;
#pragma unroll
            for (int j = 0; j < N; ++j) pa.v[j] = pb.v[j] = both(1.f);
            if (FOLD) weights(u, pa, pb);
            turn_of[u].take(prm, table, unit[u], pa, pb);
        }
        const T *row = ring;
#pragma unroll 1
        for (int i = 0; i < turns; ++i) {
            copies_wait<Sh::RING - 2>();
            const bool live = have && head <= last;
            Row va[UPL], vb[UPL], ua[UPL], ub[UPL];
#pragma unroll
            for (int u = 0; u < UPL; ++u) {
                va[u] = unpack<VEC>(row + 2 * u * 32 * VEC);
                vb[u] = unpack<VEC>(row + (2 * u + 1) * 32 * VEC);
                if constexpr (BACKWARD) {
                    ua[u] = unpack<VEC>(row + 2 * (UPL + u) * 32 * VEC);
                    ub[u] = unpack<VEC>(row + (2 * (UPL + u) + 1) * 32 * VEC);
                }
            }
            row = row == ring + (Sh::RING - 1) * (Sh::VECTORS * 32 * VEC) ? ring : row + Sh::VECTORS * 32 * VEC;
            if (i + Sh::RING - 1 < turns) fetch();
            copies_commit();
            float r = 1.f;
            if (NORM) {
                float2 ss = both(0.f);
#pragma unroll
                for (int u = 0; u < UPL; ++u)
#pragma unroll
                    for (int j = 0; j < N; ++j)
                        ss = __ffma2_rn(va[u].v[j], va[u].v[j], __ffma2_rn(vb[u].v[j], vb[u].v[j], ss));
                r = rsqrtf(fmaf(row_sum(ss.x + ss.y, lanes), inv_d, prm.eps));
            }
            if constexpr (!BACKWARD) {
#pragma unroll
                for (int u = 0; u < UPL; ++u) {
                    turn_of[u].apply(prm, unit[u], va[u], vb[u]);
                    if (NORM) {
#pragma unroll
                        for (int j = 0; j < N; ++j) {
                            va[u].v[j] = __fmul2_rn(va[u].v[j], both(r));
                            vb[u].v[j] = __fmul2_rn(vb[u].v[j], both(r));
                        }
                    }
                    if (live && on[u]) store_lane<VEC>(py + unit[u].a, va[u]);
                    if (live && two[u]) store_lane<VEC>(py + unit[u].b, vb[u]);
                }
            } else {
                // with p = g' x:  dw += r p,  dx = r (w g' - x (r mean(w p)) r)
                float2 dot = both(0.f);
                const float2 rl = both(live ? r : 0.f);
#pragma unroll
                for (int u = 0; u < UPL; ++u) {
                    turn_of[u].apply(prm, unit[u], ua[u], ub[u]);
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        const float2 pa = __fmul2_rn(ua[u].v[j], va[u].v[j]), pb = __fmul2_rn(ub[u].v[j], vb[u].v[j]);
                        ga[u].v[j] = __ffma2_rn(pa, rl, ga[u].v[j]);
                        gb[u].v[j] = __ffma2_rn(pb, rl, gb[u].v[j]);
                        dot = __ffma2_rn(pa, wa[u].v[j], __ffma2_rn(pb, wb[u].v[j], dot));
                    }
                }
                if (x.y) {
                    // r m is as large as w g', r as 1 / x: neither r^2 nor r^3,
                    // out of fp32's range for rows of 1e15, stands alone
                    const float m = row_sum(dot.x + dot.y, lanes) * inv_d;
                    const float2 k = both(-(r * m) * r), rr = both(r);
#pragma unroll
                    for (int u = 0; u < UPL; ++u) {
#pragma unroll
                        for (int j = 0; j < N; ++j) {
                            ua[u].v[j] = __fmul2_rn(rr, __ffma2_rn(va[u].v[j], k, __fmul2_rn(wa[u].v[j], ua[u].v[j])));
                            ub[u].v[j] = __fmul2_rn(rr, __ffma2_rn(vb[u].v[j], k, __fmul2_rn(wb[u].v[j], ub[u].v[j])));
                        }
                        if (live && on[u]) store_lane<VEC>(py + unit[u].a, ua[u]);
                        if (live && two[u]) store_lane<VEC>(py + unit[u].b, ub[u]);
                    }
                }
            }
            head += head_step;
            py += dense_step;
        }
        copies_wait<0>();
        share += warps / (unsigned)x.splits;
        split += (int)(warps % (unsigned)x.splits);
        if (split >= x.splits) {
            split -= x.splits;
            ++share;
        }
    }

    if constexpr (BACKWARD) {
        // the weight's gradient: over the groups of a warp by lane exchange,
        // over the warps through shared memory, in a fixed order
        if (!x.partial) return;
        float *const sums = reinterpret_cast<float *>(shared);  // [warps][D]
        __syncthreads();
#pragma unroll
        for (int u = 0; u < UPL; ++u)
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                float sa = j & 1 ? ga[u].v[j / 2].y : ga[u].v[j / 2].x;
                float sb = j & 1 ? gb[u].v[j / 2].y : gb[u].v[j / 2].x;
                for (int o = lanes; o < 32; o <<= 1) {
                    sa += __shfl_xor_sync(0xffffffffu, sa, o);
                    sb += __shfl_xor_sync(0xffffffffu, sb, o);
                }
                if ((threadIdx.x & 31) < lanes) {
                    if (on[u]) sums[warp * prm.D + unit[u].a + j] = sa;
                    if (two[u]) sums[warp * prm.D + unit[u].b + j] = sb;
                }
            }
        __syncthreads();
        for (int d = threadIdx.x; d < prm.D; d += blockDim.x) {
            float s = 0.f;
            for (int w = 0; w < (int)(blockDim.x >> 5); ++w) s += sums[w * prm.D + d];
            x.partial[(int64_t)cta * prm.D + d] = s;
        }
    }
}

// The CTAs' sums of the weights' gradients, added in a fixed order.  Grid: 32
// elements a CTA, the first tensor's, then the second's; 32 x 32 threads.
struct RotaryReduceParams {
    const float *partial[2];
    float *out[2];
    unsigned rows[2];
    int D, ctas;  // ctas: of the first tensor
};
__global__ void __launch_bounds__(1024) kla_rotary_reduce_kernel(const RotaryReduceParams prm) {
    __shared__ float sums[32][33];
    const bool second = (int)blockIdx.x >= prm.ctas;
    const int first = ((int)blockIdx.x - (second ? prm.ctas : 0)) * 32;
    const float *partial = second ? prm.partial[1] : prm.partial[0];
    const unsigned rows = second ? prm.rows[1] : prm.rows[0];
    float *out = second ? prm.out[1] : prm.out[0];
    const int d = first + threadIdx.x;
    float s = 0.f;
    if (d < prm.D)
        for (unsigned r = threadIdx.y; r < rows; r += 32) s += partial[(int64_t)r * prm.D + d];
    sums[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    s = row_sum(sums[threadIdx.x][threadIdx.y], 32);
    const int e = first + threadIdx.y;
    if (threadIdx.x == 0 && e < prm.D) out[e] = s;
}

}  // namespace kla_mixer
