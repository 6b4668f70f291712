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
// Every element is read and written once: the kernels are bound by HBM.  A
// row belongs to a group of lanes (a power of two, at most a warp); the sum
// of squares is a few lane exchanges and nothing goes through shared memory
// but the table of cos and sin, which a CTA makes once for its tokens and
// uses for all of their heads.  A lane holds whole pairs: VEC elements from
// each half of the rotated part, or 2 VEC neighbours.
//
// Angles: the product of position and frequency in 64 bits, reduced there to
// a fraction of a turn, so that far positions lose nothing; the rounding of
// that fraction to 32 bits is given back to first order.
#pragma once

#include "kla_mixer.h"

namespace kla_mixer {

constexpr int kRotaryThreads = 256;
constexpr int kRotaryTable = 2048;  // pairs of cos and sin that a CTA holds (16 KB)

struct RotaryTensor {
    const void *x, *gy;      // input; gradient of the output (backward)
    void *y;                 // output; gradient of the input (backward)
    const float *w;          // weight or null
    float *partial;          // [CTAs of this tensor][D]: sums of the weight's gradient, or null
    int64_t sb, st, sh;      // strides of x in elements; y and gy are dense
    int heads;
    int tokens_per_cta;
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

// (cos, sin) of 2 pi times a number of turns.
__device__ __forceinline__ float2 turn(double turns) {
    const double r = turns - rint(turns);
    const float f = (float)r;
    float s, c;
    sincospif(2.f * f, &s, &c);
    const float d = (float)(r - (double)f) * 6.28318530717958648f;
    return make_float2(fmaf(-s, d, c), fmaf(c, d, s));
}

// The table of a CTA's tokens [first, first + n).
__device__ __forceinline__ void rotary_table(const RotaryParams &prm, float2 *table, int64_t first, int n) {
    for (int i = threadIdx.x; i < n * prm.half; i += blockDim.x) {
        const int k = i / prm.half;
        const int64_t token = first + k;
        const int64_t b = token / prm.T;
        const int64_t t = token - b * prm.T;
        const int64_t at = prm.positions ? prm.positions[b * prm.position_stride + t] : prm.position0 + t;
        const float2 cs = turn((double)at * (prm.inv_freq[i - k * prm.half] * 0.15915494309189533577));
        table[i] = make_float2(prm.scale * cs.x, prm.sign * prm.scale * cs.y);
    }
}

// Elements of unit u: two vectors of VEC at a and b (b >= D: there is none),
// and the table entry of their first pair (negative: they pass).
struct Unit {
    int a, b, pair;
};
template <int VEC>
__device__ __forceinline__ Unit unit_at(const RotaryParams &prm, int u) {
    Unit k;
    const int turned = prm.half / VEC;
    if (u < turned) {
        k.pair = u * VEC;
        k.a = prm.interleaved ? 2 * u * VEC : u * VEC;
        k.b = prm.interleaved ? k.a + VEC : prm.half + u * VEC;
    } else {
        k.pair = -1;
        k.a = 2 * prm.half + 2 * (u - turned) * VEC;
        k.b = k.a + VEC;
    }
    return k;
}

// Turn the pairs of a unit in place.
template <int VEC>
__device__ __forceinline__ void rotate(float (&a)[VEC], float (&b)[VEC], const float2 *cs, bool interleaved) {
    auto pair = [](float &x, float &y, float2 c) {
        const float u = x, v = y;
        x = fmaf(u, c.x, -v * c.y);
        y = fmaf(u, c.y, v * c.x);
    };
    if (VEC == 1 || !interleaved) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) pair(a[j], b[j], cs[j]);
    } else {
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) {
            pair(a[2 * j], a[2 * j + 1], cs[j]);
            pair(b[2 * j], b[2 * j + 1], cs[VEC / 2 + j]);
        }
    }
}

template <typename T, int VEC>
__device__ __forceinline__ void load_row(float (&to)[VEC], const T *p, bool on) {
    if (on) {
        const Pack<T, VEC> r = load_cs<T, VEC>(p);
#pragma unroll
        for (int j = 0; j < VEC; ++j) to[j] = to_float(r.v[j]);
    } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) to[j] = 0.f;
    }
}
template <typename T, int VEC>
__device__ __forceinline__ void store_row(T *p, const float (&from)[VEC]) {
    Pack<T, VEC> r;
#pragma unroll
    for (int j = 0; j < VEC; ++j) r.v[j] = from_float<T>(from[j]);
    store_cs<T, VEC>(p, r);
}

__device__ __forceinline__ float row_sum(float x, int lanes) {
    for (int o = lanes >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Grid: the CTAs of the first tensor, then those of the second; each CTA
// takes blocks of tokens_per_cta tokens, `ctas` blocks apart.  UPL: units per
// lane.  Shared memory: the table, and (backward) the warps' weight sums.
template <typename T, int VEC, int UPL, bool NORM, bool BACKWARD>
__global__ void __launch_bounds__(kRotaryThreads) kla_rotary_kernel(const RotaryParams prm) {
    extern __shared__ float2 table[];
    const int which = blockIdx.x >= prm.t[0].ctas;
    const RotaryTensor &x = which ? prm.t[1] : prm.t[0];
    const unsigned cta = blockIdx.x - (which ? prm.t[0].ctas : 0u);
    const int lanes = prm.lanes;
    const int lane = threadIdx.x & (lanes - 1);
    const int group = threadIdx.x / lanes;
    const int groups = blockDim.x / lanes;
    const int warp_group = (threadIdx.x & ~31) / lanes;  // of the warp's first lane

    Unit unit[UPL];
    float wa[UPL][VEC], wb[UPL][VEC];      // the weight at this lane's elements
    float ga[UPL][VEC], gb[UPL][VEC];      // its gradient over this lane's rows
    bool on[UPL], two[UPL];
#pragma unroll
    for (int u = 0; u < UPL; ++u) {
        const int k = lane + u * lanes;
        unit[u] = unit_at<VEC>(prm, k);
        on[u] = k < prm.units;
        two[u] = on[u] && unit[u].b < prm.D;
        if (NORM) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                wa[u][j] = x.w && on[u] ? x.w[unit[u].a + j] : 1.f;
                wb[u][j] = x.w && two[u] ? x.w[unit[u].b + j] : 1.f;
                ga[u][j] = gb[u][j] = 0.f;
            }
        }
    }
    const float inv_d = 1.f / (float)prm.D;

    for (int64_t first = (int64_t)cta * x.tokens_per_cta; first < prm.tokens;
         first += (int64_t)x.ctas * x.tokens_per_cta) {
        const int64_t left = prm.tokens - first;
        const int n = left < x.tokens_per_cta ? (int)left : x.tokens_per_cta;
        if (first != (int64_t)cta * x.tokens_per_cta) __syncthreads();  // the table's last readers
        rotary_table(prm, table, first, n);
        __syncthreads();
        const int rows = n * x.heads;
        // whole warps run on while one of their groups has a row
        for (int base = warp_group, row = group; base < rows; base += groups, row += groups) {
            const bool live = row < rows;
            const int k = live ? row / x.heads : 0;
            const int head = live ? row - k * x.heads : 0;
            const int64_t token = first + k;
            const int64_t b = token / prm.T;
            const T *px = static_cast<const T *>(x.x) + b * x.sb + (token - b * prm.T) * x.st + head * x.sh;
            const int64_t dense = (token * x.heads + head) * prm.D;
            float va[UPL][VEC], vb[UPL][VEC];
            if (NORM || !BACKWARD) {
#pragma unroll
                for (int u = 0; u < UPL; ++u) {
                    load_row<T, VEC>(va[u], px + unit[u].a, live && on[u]);
                    load_row<T, VEC>(vb[u], px + unit[u].b, live && two[u]);
                }
            }
            float r = 1.f;
            if (NORM) {
                float ss = 0.f;
#pragma unroll
                for (int u = 0; u < UPL; ++u)
#pragma unroll
                    for (int j = 0; j < VEC; ++j) ss = fmaf(va[u][j], va[u][j], fmaf(vb[u][j], vb[u][j], ss));
                r = rsqrtf(fmaf(row_sum(ss, lanes), inv_d, prm.eps));
                if (!live) r = 0.f;  // no row: eps = 0 would make it infinite, and the weight's sum NaN
            }
            T *py = static_cast<T *>(x.y) + dense;
            if constexpr (!BACKWARD) {
#pragma unroll
                for (int u = 0; u < UPL; ++u) {
                    if (NORM) {
#pragma unroll
                        for (int j = 0; j < VEC; ++j) {
                            va[u][j] *= r * wa[u][j];
                            vb[u][j] *= r * wb[u][j];
                        }
                    }
                    if (on[u] && unit[u].pair >= 0)
                        rotate<VEC>(va[u], vb[u], table + k * prm.half + unit[u].pair, prm.interleaved);
                    if (live && on[u]) store_row<T, VEC>(py + unit[u].a, va[u]);
                    if (live && two[u]) store_row<T, VEC>(py + unit[u].b, vb[u]);
                }
            } else {
                const T *pg = static_cast<const T *>(x.gy) + dense;
                float ua[UPL][VEC], ub[UPL][VEC];
                float dot = 0.f;
#pragma unroll
                for (int u = 0; u < UPL; ++u) {
                    load_row<T, VEC>(ua[u], pg + unit[u].a, live && on[u]);
                    load_row<T, VEC>(ub[u], pg + unit[u].b, live && two[u]);
                }
#pragma unroll
                for (int u = 0; u < UPL; ++u) {
                    if (on[u] && unit[u].pair >= 0)
                        rotate<VEC>(ua[u], ub[u], table + k * prm.half + unit[u].pair, prm.interleaved);
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        va[u][j] *= r;
                        vb[u][j] *= r;
                        ga[u][j] = fmaf(ua[u][j], va[u][j], ga[u][j]);
                        gb[u][j] = fmaf(ub[u][j], vb[u][j], gb[u][j]);
                        ua[u][j] *= wa[u][j];
                        ub[u][j] *= wb[u][j];
                        dot = fmaf(ua[u][j], va[u][j], fmaf(ub[u][j], vb[u][j], dot));
                    }
                }
                if (!x.y) continue;  // uniform: only the weight's gradient is wanted
                const float m = row_sum(dot, lanes) * inv_d;
#pragma unroll
                for (int u = 0; u < UPL; ++u) {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        ua[u][j] = r * fmaf(-va[u][j], m, ua[u][j]);
                        ub[u][j] = r * fmaf(-vb[u][j], m, ub[u][j]);
                    }
                    if (live && on[u]) store_row<T, VEC>(py + unit[u].a, ua[u]);
                    if (live && two[u]) store_row<T, VEC>(py + unit[u].b, ub[u]);
                }
            }
        }
    }

    if constexpr (BACKWARD) {
        // the weight's gradient: over the groups of a warp by lane exchange,
        // over the warps through shared memory, in a fixed order
        if (!x.partial) return;
        float *sums = reinterpret_cast<float *>(table);  // [warps][D]
        __syncthreads();
        const int warp = threadIdx.x >> 5;
#pragma unroll
        for (int u = 0; u < UPL; ++u)
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                for (int o = lanes; o < 32; o <<= 1) {
                    ga[u][j] += __shfl_xor_sync(0xffffffffu, ga[u][j], o);
                    gb[u][j] += __shfl_xor_sync(0xffffffffu, gb[u][j], o);
                }
                if ((threadIdx.x & 31) < lanes) {
                    if (on[u]) sums[warp * prm.D + unit[u].a + j] = ga[u][j];
                    if (two[u]) sums[warp * prm.D + unit[u].b + j] = gb[u][j];
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
