// fp32 grouped products on the CUDA cores.  The fp32 layer is the small one the
// router's precision is checked with, so the kernel is a plain shared-memory
// tile (64 x 64 outputs, 16 of K, 16 outputs a thread) for any strides; fp32
// FMAs in K order, so results do not depend on the launch.
#include "grouped_simt.cuh"

namespace moe {
namespace grp {

namespace {

constexpr int TM = 64, TN = 64, TK = 16;

__global__ void __launch_bounds__(256) simt_kernel(const Simt p)
{
    __shared__ float As[TK][TM + 4], Bs[TK][TN + 4];
    const int g = blockIdx.z, tid = threadIdx.x;
    pdl_wait();
    pdl_trigger();
    if (p.clear && blockIdx.x + blockIdx.y + blockIdx.z == 0 && tid == 0)
        *p.clear = 0;
    int M = p.M, K = p.K, m_base = 0, k_base = 0;
    if (p.mode == RAGGED_M)
        group_rows(p.offsets, p.rows, p.n_rows, g, &m_base, &M);
    else if (p.mode == RAGGED_K)
        group_rows(p.offsets, p.rows, p.n_rows, g, &k_base, &K);
    const float *A = p.a + g * p.a_group + m_base * p.a_m + k_base * p.a_k;
    const float *B = p.b + g * p.b_group + k_base * p.b_k;
    const int64_t c0 = g * p.c_group + m_base * p.c_m;
    const int n0 = blockIdx.x * TN, tx = tid & 15, ty = tid >> 4;
    // consecutive threads along the contiguous index of each operand
    const bool ak = p.a_k == 1, bk = p.b_k == 1;
    for (int m0 = blockIdx.y * TM; m0 < M; m0 += gridDim.y * TM) {
        float acc[4][4] = {};
        for (int k0 = 0; k0 < K; k0 += TK) {
#pragma unroll
            for (int i = 0; i < TM * TK / 256; ++i) {
                const int e = tid + 256 * i;
                const int m = ak ? e / TK : e % TM, k = ak ? e % TK : e / TM;
                As[k][m] = m0 + m < M && k0 + k < K
                               ? A[(int64_t)(m0 + m) * p.a_m + (int64_t)(k0 + k) * p.a_k]
                               : 0.f;
                const int n = bk ? e / TK : e % TN, kk = bk ? e % TK : e / TN;
                Bs[kk][n] = n0 + n < p.N && k0 + kk < K
                                ? B[(int64_t)(n0 + n) * p.b_n + (int64_t)(k0 + kk) * p.b_k]
                                : 0.f;
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < TK; ++k) {
                const float4 a = *reinterpret_cast<const float4 *>(&As[k][ty * 4]);
                const float4 b = *reinterpret_cast<const float4 *>(&Bs[k][tx * 4]);
                const float av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
            }
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
                if (m < M && n < p.N) {
                    const int64_t o = c0 + (int64_t)m * p.c_m + n;
                    p.c[o] = p.add ? p.add[o] + acc[i][j] : acc[i][j];
                }
            }
    }
}

__global__ void __launch_bounds__(256)
    act_grad_kernel(int act, int64_t n, const float *u, const float *v, const float *dh, float *h,
                    float *du, float *dv)
{
    pdl_wait();
    pdl_trigger();
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll) {
        const float a = u[i], g = dh[i];
        if (act == MOE_ACT_GELU) {
            const float cdf = 0.5f * (1.f + erff(a * 0.70710678118654752f));
            h[i] = a * cdf;
            du[i] = g * (cdf + a * 0.39894228040143268f * expf(-0.5f * a * a));
        } else {
            const float s = 1.f / (1.f + expf(-a)), as = a * s, b = v[i];
            h[i] = as * b;
            dv[i] = g * as;
            du[i] = g * b * (s + as * (1.f - s));
        }
    }
}

}  // namespace

cudaError_t launch_simt(const Simt &p, cudaStream_t s)
{
    const int64_t m = p.mode == RAGGED_M ? p.n_rows : p.M;
    int64_t my = ceil_div(m, TM);
    if (p.mode == RAGGED_M)   // twice the mean group; longer groups loop
        my = ceil_div(2 * m, (int64_t)p.groups * TM) < my ? ceil_div(2 * m, (int64_t)p.groups * TM)
                                                          : my;
    if (my < 1)
        return cudaSuccess;
    if (my > 16384)
        my = 16384;
    return launch_pdl(simt_kernel, dim3((unsigned)ceil_div(p.N, TN), (unsigned)my, p.groups),
                      dim3(256), 0, s, p);
}

cudaError_t launch_act_grad(int act, int64_t n, const float *u, const float *v, const float *dh,
                            float *h, float *du, float *dv, cudaStream_t s)
{
    if (n < 1)
        return cudaSuccess;
    const int64_t blocks = ceil_div(n, 256) < 4096 ? ceil_div(n, 256) : 4096;
    return launch_pdl(act_grad_kernel, dim3((unsigned)blocks), dim3(256), 0, s, act, n, u, v, dh,
                      h, du, dv);
}

}  // namespace grp
}  // namespace moe
