// How the Newton-Schulz steps hold their matrices in fp16: what is stored is the
// true value times a power of two (of X a factor of its own for every matrix and
// step), so that neither end of fp16's range is near.
#pragma once

#include <cuda_bf16.h>
#include <math.h>

namespace moe {
namespace grp {

// A and B stored over true values, and X's factor once its singular values are
// near 1.
constexpr float kSX = 8192.f, kSA = 8192.f, kSB = 2048.f;

// A bound on the singular values of X after a step, from one before it.
__host__ __device__ inline float next_bound(float u, float a, float b, float c)
{
    const float s = u * u;
    return fminf(u * (fabsf(a) + s * (fabsf(b) + s * fabsf(c))), 1e3f);
}

// X's factor over kSX, as a power of two, where its singular values are at most u.
// They start at |G| / (|G| + eps): an update far below eps would vanish under kSX,
// and with it the result, about |a| to the number of steps times what X was.
__device__ __forceinline__ int x_shift(float u)
{
    if (!(u > 0.f) || u >= 0.5f)
        return 0;
    return (int)fminf(floorf(-log2f(u)), 100.f);
}
__device__ __forceinline__ float power2(int k) { return __int_as_float((127 + k) << 23); }

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f(float v) { return v; }
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }

}  // namespace grp
}  // namespace moe
