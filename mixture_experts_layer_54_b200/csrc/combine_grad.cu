// Gradients of the gated combine y[t] = sum_j gate[t, j] Y_perm[row(t, j)]
// over kept assignments ("Lab 18 - Mixture of experts", section 1: y = sum of
// g_i FFN_i(x)):
//   dY_perm[row(t, j)] = gate[t, j] dy[t],   dgate[t, j] = <dy[t], Y_perm[row(t, j)]>.
// Bound by memory: dy read once, each kept row of Y_perm read and of dY_perm
// written once.  One block per token: a thread holds 16 bytes of dy[t] in
// registers and takes all k rows' pieces at the same place, every row's load in
// flight before the first use; the k dot products (fp32) are summed over the
// block in a fixed order.
#include "internal.cuh"

namespace moe {

namespace {

constexpr int CT = 128;   // threads

template <typename T>
struct Vec;
template <>
struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void load(const uint4 &u, float *f)
    {
        f[0] = __uint_as_float(u.x), f[1] = __uint_as_float(u.y);
        f[2] = __uint_as_float(u.z), f[3] = __uint_as_float(u.w);
    }
    static __device__ __forceinline__ uint4 pack(const float *f)
    {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                          __float_as_uint(f[3]));
    }
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void load(const uint4 &u, float *f)
    {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float *f)
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<uint32_t *>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

template <typename T, int K>
__global__ void __launch_bounds__(CT)
    combine_grad_kernel(int tokens, int d, int E, int rows, const T *dy, const T *Y,
                        const float *gates, const int32_t *topk, const int32_t *pos,
                        const uint8_t *keep, const int32_t *offsets, T *dY, float *dgates)
{
    using V = Vec<T>;
    __shared__ float part[CT / 32][K];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, nv = d / V::N;
    pdl_wait();
    pdl_trigger();
    for (int t = blockIdx.x; t < tokens; t += gridDim.x) {
        int row[K];
        float gate[K], dot[K];
#pragma unroll
        for (int j = 0; j < K; ++j) {
            const int64_t a = (int64_t)t * K + j;
            const int e = topk[a];
            int r = -1;   // dropped, or outside the buffers: no row
            if (keep[a] && e >= 0 && e < E) {
                r = offsets[e] + pos[a];
                if (r < 0 || r >= rows)
                    r = -1;
            }
            row[j] = r;
            gate[j] = gates[a];
            dot[j] = 0.f;
        }
        const uint4 *dyv = reinterpret_cast<const uint4 *>(dy + (int64_t)t * d);
        for (int i = tid; i < nv; i += CT) {
            uint4 y[K];
#pragma unroll
            for (int j = 0; j < K; ++j)
                y[j] = row[j] >= 0
                           ? reinterpret_cast<const uint4 *>(Y + (int64_t)row[j] * d)[i]
                           : make_uint4(0, 0, 0, 0);
            float g[V::N];
            V::load(dyv[i], g);
#pragma unroll
            for (int j = 0; j < K; ++j) {
                if (row[j] < 0)
                    continue;
                float f[V::N], o[V::N];
                V::load(y[j], f);
#pragma unroll
                for (int c = 0; c < V::N; ++c) {
                    dot[j] = fmaf(g[c], f[c], dot[j]);
                    o[c] = gate[j] * g[c];
                }
                reinterpret_cast<uint4 *>(dY + (int64_t)row[j] * d)[i] = V::pack(o);
            }
        }
#pragma unroll
        for (int j = 0; j < K; ++j) {
#pragma unroll
            for (int s = 16; s; s >>= 1)
                dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], s);
            if (lane == 0)
                part[warp][j] = dot[j];
        }
        __syncthreads();
        if (tid < K) {
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < CT / 32; ++w)
                sum += part[w][tid];
            dgates[(int64_t)t * K + tid] = sum;
        }
        __syncthreads();
    }
}

template <typename T, int K>
cudaError_t launch(const moe_config &c, const void *dy, const void *Y, const float *gates,
                   const int32_t *topk, const int32_t *pos, const uint8_t *keep,
                   const int32_t *offsets, void *dY, float *dgates, cudaStream_t s)
{
    const int blocks = c.T < 65535 * 16 ? c.T : 65535 * 16;
    return launch_pdl(combine_grad_kernel<T, K>, dim3(blocks), dim3(CT), 0, s, (int)c.T, (int)c.d,
                      (int)c.E, (int)perm_rows(c), static_cast<const T *>(dy),
                      static_cast<const T *>(Y), gates, topk, pos, keep, offsets,
                      static_cast<T *>(dY), dgates);
}

template <typename T>
cudaError_t launch_k(const moe_config &c, const void *dy, const void *Y, const float *gates,
                     const int32_t *topk, const int32_t *pos, const uint8_t *keep,
                     const int32_t *offsets, void *dY, float *dgates, cudaStream_t s)
{
    switch (c.k) {
    case 1: return launch<T, 1>(c, dy, Y, gates, topk, pos, keep, offsets, dY, dgates, s);
    case 2: return launch<T, 2>(c, dy, Y, gates, topk, pos, keep, offsets, dY, dgates, s);
    case 3: return launch<T, 3>(c, dy, Y, gates, topk, pos, keep, offsets, dY, dgates, s);
    case 4: return launch<T, 4>(c, dy, Y, gates, topk, pos, keep, offsets, dY, dgates, s);
    case 5: return launch<T, 5>(c, dy, Y, gates, topk, pos, keep, offsets, dY, dgates, s);
    case 6: return launch<T, 6>(c, dy, Y, gates, topk, pos, keep, offsets, dY, dgates, s);
    case 7: return launch<T, 7>(c, dy, Y, gates, topk, pos, keep, offsets, dY, dgates, s);
    case 8: return launch<T, 8>(c, dy, Y, gates, topk, pos, keep, offsets, dY, dgates, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_combine_grad(const moe_config &c, const void *dy, const void *Y_perm,
                                const float *gates, const int32_t *topk, const int32_t *pos,
                                const uint8_t *keep, const int32_t *offsets, void *dY_perm,
                                float *dgates, cudaStream_t s)
{
    return c.dtype == MOE_DTYPE_BF16
               ? launch_k<__nv_bfloat16>(c, dy, Y_perm, gates, topk, pos, keep, offsets, dY_perm,
                                         dgates, s)
               : launch_k<float>(c, dy, Y_perm, gates, topk, pos, keep, offsets, dY_perm, dgates,
                                 s);
}

}  // namespace moe
