// Device helpers of the token operators: element types in 16-byte pieces, and
// the owner of a token in a batch of sequences.  gfx950 only.
#pragma once

#include <cstdint>

#include <hip/hip_runtime.h>

#include "token_internal.h"

namespace bevpool {

constexpr int kLanes = 64;

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x8 __attribute__((ext_vector_type(8)));

template <int DT> struct Elem;
template <> struct Elem<kF32> { using type = float; };
template <> struct Elem<kF16> { using type = _Float16; };
template <> struct Elem<kBF16> { using type = __bf16; };
template <> struct Elem<kE4M3> { using type = uint8_t; };

// Eight consecutive elements as floats (16-byte aligned address).
template <int DT>
__device__ __forceinline__ f32x8 load8(const typename Elem<DT>::type *p)
{
    if constexpr (DT == kF32) {
        const f32x4 a = *reinterpret_cast<const f32x4 *>(p);
        const f32x4 b = *reinterpret_cast<const f32x4 *>(p + 4);
        return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    } else if constexpr (DT == kF16) {
        return __builtin_convertvector(*reinterpret_cast<const f16x8 *>(p), f32x8);
    } else {
        return __builtin_convertvector(*reinterpret_cast<const bf16x8 *>(p), f32x8);
    }
}

// Four e4m3 codes of four floats within the format's range, rounded to
// nearest-even; NaN gives its code.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d)
{
    int w = 0;
    w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, w, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
    return uint32_t(w);
}

// Rounds eight floats to DT (nearest-even) and stores them.
template <int DT>
__device__ __forceinline__ void store8(typename Elem<DT>::type *p, f32x8 v)
{
    if constexpr (DT == kF32) {
        *reinterpret_cast<f32x4 *>(p) = __builtin_shufflevector(v, v, 0, 1, 2, 3);
        *reinterpret_cast<f32x4 *>(p + 4) = __builtin_shufflevector(v, v, 4, 5, 6, 7);
    } else if constexpr (DT == kF16) {
        *reinterpret_cast<f16x8 *>(p) = __builtin_convertvector(v, f16x8);
    } else if constexpr (DT == kBF16) {
        *reinterpret_cast<bf16x8 *>(p) = __builtin_convertvector(v, bf16x8);
    } else {
        u32x2 w;
        w.x = e4m3x4(v[0], v[1], v[2], v[3]);
        w.y = e4m3x4(v[4], v[5], v[6], v[7]);
        *reinterpret_cast<u32x2 *>(p) = w;
    }
}

__device__ __forceinline__ int clip(int v, int lo, int hi) { return v < lo ? lo : (v > hi ? hi : v); }

// The number of s in [1, n] with key(s) <= x, by the whole wave: each step
// asks 64 evenly spaced keys and keeps the gap that holds the boundary.
// key is non-decreasing; for any other the answer is still within [0, n].
template <typename Key>
__device__ __forceinline__ int count_upto(int n, int64_t x, Key key)
{
    const int lane = int(threadIdx.x) & (kLanes - 1);
    int lo = 1, len = n;                      // the boundary lies in [lo, lo + len]
    while (len > kLanes) {
        const int step = (len + kLanes - 1) / kLanes;
        const int at = lo + (lane + 1) * step - 1;
        const bool in = at < lo + len;
        const int c = __popcll(__ballot(in && key(in ? at : lo) <= x));
        const int used = c * step;
        lo += used;
        len = len - used < step ? len - used : step;
    }
    const bool in = lane < len;
    return lo - 1 + __popcll(__ballot(in && key(in ? lo + lane : 1) <= x));
}

}  // namespace bevpool
