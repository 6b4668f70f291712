// kla_mixer.h -- what the translation units of the mixer operators share
// (kla_gated.cu, kla_rotary.cu): host-side argument checks in the manner of
// kla.cu, and the few device helpers that do not need kla_device.cuh (which
// owns device globals and is compiled into kla.cu alone).
#pragma once

#include "kla.h"

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#define KLA_API extern "C" __attribute__((visibility("default")))

namespace kla_mixer {

// ---- host ------------------------------------------------------------------
inline bool mul_ok(int64_t a, int64_t b, int64_t *out) {
    if (a < 0 || b < 0) return false;
    if (a != 0 && b > INT64_MAX / a) return false;
    *out = a * b;
    return true;
}

inline bool dtype_ok(kla_dtype_t d) { return d == KLA_F32 || d == KLA_BF16; }
inline int64_t dtype_size(kla_dtype_t d) { return d == KLA_BF16 ? 2 : 4; }

struct Range {
    uintptr_t lo, hi;
};
inline Range range_of(const void *p, int64_t bytes) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return Range{lo, p ? lo + (uintptr_t)bytes : lo};
}

// Any two of `outs` overlap, or any output overlaps any input.
inline bool any_overlap(const Range *outs, int n_out, const Range *ins, int n_in) {
    auto hit = [](const Range &x, const Range &y) {
        return x.lo != x.hi && y.lo != y.hi && x.lo < y.hi && y.lo < x.hi;
    };
    for (int i = 0; i < n_out; ++i) {
        for (int j = i + 1; j < n_out; ++j)
            if (hit(outs[i], outs[j])) return true;
        for (int j = 0; j < n_in; ++j)
            if (hit(outs[i], ins[j])) return true;
    }
    return false;
}

inline bool aligned(const void *p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % (uintptr_t)bytes == 0; }

// Multiprocessors of the current device.
inline int sm_count() {
    static std::mutex mu;
    static int count[256] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 256) return 148;
    std::lock_guard<std::mutex> lock(mu);
    if (count[dev] == 0) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
        count[dev] = n;
    }
    return count[dev];
}

constexpr int64_t kMaxGrid = 0x7fffffff;

// ---- device ----------------------------------------------------------------
// V consecutive elements of type T as one aligned load or store.
template <typename T, int V>
struct alignas(V * sizeof(T)) Pack {
    T v[V];
};

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T> __device__ __forceinline__ T from_float(float x);
template <> __device__ __forceinline__ float from_float<float>(float x) { return x; }
// round to nearest even, once, from the fp32 result
template <> __device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) {
    return __float2bfloat16_rn(x);
}

// Streaming (evict-first) load and store of a pack: every element of these
// operators is read and written once.
template <int BYTES> struct Raw;
template <> struct Raw<2> { using type = unsigned short; };
template <> struct Raw<4> { using type = unsigned; };
template <> struct Raw<8> { using type = uint2; };
template <> struct Raw<16> { using type = uint4; };
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load_cs(const T *p) {
    using R = typename Raw<V * sizeof(T)>::type;
    const R r = __ldcs(reinterpret_cast<const R *>(p));
    return *reinterpret_cast<const Pack<T, V> *>(&r);
}
template <typename T, int V>
__device__ __forceinline__ void store_cs(T *p, const Pack<T, V> &x) {
    using R = typename Raw<V * sizeof(T)>::type;
    __stcs(reinterpret_cast<R *>(p), *reinterpret_cast<const R *>(&x));
}

// Asynchronous copy of BYTES (4, 8 or 16) to the shared-memory address `at`.
template <int BYTES>
__device__ __forceinline__ void copy_async(unsigned at, const void *from) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(from) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(at), "l"(from), "n"(BYTES) : "memory");
}
// The same of the first `bytes` (up to 16) of 16; the rest becomes zero.
__device__ __forceinline__ void copy_async_part(unsigned at, const void *from, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at), "l"(from), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

}  // namespace kla_mixer
