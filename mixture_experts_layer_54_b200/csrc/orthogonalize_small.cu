// Orthogonalised updates of small matrices: one block holds a whole matrix and
// runs every Newton-Schulz step in shared memory and TMEM (fifteen launches of
// the stacked products and their round trips through memory took 98 us for 4 of
// 64 x 32; this kernel's time is in the phases' latencies).
//
// X is p x q with p <= q (a tall G is read and written transposed), as two fp16
// terms hi + lo in the layout the tensor cores read: 64-column blocks of 128
// rows x 128 bytes, 128-byte swizzle; rows and columns past p and q are zero.
// The same bytes serve as the K-major operand of A = X X^T and as the MN-major
// operand of X = B X.  A step is three phases, each one tcgen05.mma sequence of
// hi hi + hi lo + lo hi (22 bits, so results are those of fp32 arithmetic) and
// one pass of the eight warps over the accumulator:
//   A = X X^T;  B = a I + b A + c A A;  X = B X.
// A and B share one buffer of 128 x 128 in two terms.
#include "grouped.cuh"
#include "orthogonalize.cuh"

#include <cuda_fp16.h>
#include <math.h>

namespace moe {
namespace grp {

using namespace tc;

namespace {

__device__ int32_t g_gave_up;   // MOE_ERR_DEVICE_TIMEOUT after any call here gave up

constexpr int BLOCK = 128 * 128;                            // bytes of 64 columns of one term
constexpr int THREADS = 256;

struct SmallParams {
    const void *G;
    __nv_bfloat16 *U;
    int m, n, steps;
    float a, b, c, eps, scale;
    int32_t *status;
};

// byte offset of (row, col) in a term
__device__ __forceinline__ uint32_t place(int row, int col)
{
    return (uint32_t)(col >> 6) * BLOCK + row * 128 + ((((col >> 3) & 7) ^ (row & 7)) << 4) +
           (col & 7) * 2;
}

// 16 values of a row, as hi + lo, to columns col .. col + 15 of both terms
__device__ __forceinline__ void put16(uint8_t *hi, uint8_t *lo, int row, int col, const float *v)
{
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        uint32_t h[4], l[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float x0 = v[8 * g + 2 * j], x1 = v[8 * g + 2 * j + 1];
            const __half2 a = __floats2half2_rn(x0, x1);
            const float2 f = __half22float2(a);
            const __half2 d = __floats2half2_rn(x0 - f.x, x1 - f.y);
            h[j] = *reinterpret_cast<const uint32_t *>(&a);
            l[j] = *reinterpret_cast<const uint32_t *>(&d);
        }
        const uint32_t o = place(row, col + 8 * g);
        *reinterpret_cast<uint4 *>(hi + o) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4 *>(lo + o) = make_uint4(l[0], l[1], l[2], l[3]);
    }
}

// the values of both terms at columns col .. col + 15 of a row
__device__ __forceinline__ void get16(const uint8_t *hi, const uint8_t *lo, int row, int col,
                                      float *v)
{
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        const uint32_t o = place(row, col + 8 * g);
        const uint4 h = *reinterpret_cast<const uint4 *>(hi + o);
        const uint4 l = *reinterpret_cast<const uint4 *>(lo + o);
        const uint32_t hw[4] = {h.x, h.y, h.z, h.w}, lw[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&hw[j]));
            const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&lw[j]));
            v[8 * g + 2 * j] = x.x + y.x;
            v[8 * g + 2 * j + 1] = x.y + y.y;
        }
    }
}

__host__ __device__ constexpr uint32_t tmem_cols(int blocks) { return blocks <= 2 ? 256 : 512; }

template <typename T>
__global__ void __launch_bounds__(THREADS, 1) ns_small_kernel(const SmallParams s)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~uintptr_t(1023));
    const bool wide = s.m <= s.n;
    const int p = wide ? s.m : s.n, q = wide ? s.n : s.m, mn = s.m * s.n;
    const int qb = (q + 63) / 64, pb = (p + 63) / 64;     // 64-column blocks of X and of A
    uint8_t *xh = smem, *xl = xh + qb * BLOCK, *sh = xl + qb * BLOCK, *sl = sh + pb * BLOCK;
    __shared__ uint64_t bar_mem;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    __shared__ double part[THREADS / 32];
    __shared__ float s_mul, s_over, s_size;
    __shared__ int again;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t bar = smem_u32(&bar_mem);
    const Ctl ctl{&abort_flag, s.status, 2000000000ull};
    if (tid == 0) {
        mbar_init(bar, 1);
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    // 128 columns of A, the blocks of X: 256 or 512.  The launch asks for enough
    // shared memory that no more blocks share an SM than its TMEM holds.
    const uint32_t cols = tmem_cols(qb);
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&tmem_slot)),
                     "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    for (int i = tid; i < 2 * (qb + pb) * BLOCK / 16; i += THREADS)
        reinterpret_cast<uint4 *>(smem)[i] = make_uint4(0, 0, 0, 0);
    pdl_wait();
    pdl_trigger();
    if (blockIdx.x == 0 && tid == 0)
        *s.status = 0;

    // |G| and X = G / (|G| + eps), times its factor
    const T *G = static_cast<const T *>(s.G) + (int64_t)blockIdx.x * mn;
    float acc[4] = {};
    for (int i = tid; i < mn; i += 4 * THREADS) {
        float f[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
            f[u] = i + u * THREADS < mn ? to_f<T>(G[i + u * THREADS]) : 0.f;
#pragma unroll
        for (int u = 0; u < 4; ++u)
            acc[u] = fmaf(f[u], f[u], acc[u]);
    }
    auto warp_sums = [&](double v) {
#pragma unroll
        for (int o = 16; o; o >>= 1)
            v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == 0)
            part[warp] = v;
    };
    auto block_sum = [&]() {
        double v = part[0];
        for (int i = 1; i < THREADS / 32; ++i)
            v += part[i];
        return v;
    };
    warp_sums((double)acc[0] + acc[1] + acc[2] + acc[3]);
    tc_fence_before();
    __syncthreads();   // also: shared memory zeroed, barrier and TMEM ready
    tc_fence_after();
    double v = 0;
    if (tid == 0) {
        v = block_sum();
        again = !(v >= 1e-20 && v <= 1e38);   // some squares may have left fp32's range
    }
    __syncthreads();
    if (again) {
        double w = 0;
        for (int i = tid; i < mn; i += THREADS) {
            const double x = (double)to_f<T>(G[i]);
            w += x * x;
        }
        warp_sums(w);
        __syncthreads();
        if (tid == 0)
            v = block_sum();
    }
    if (tid == 0) {
        const double size = sqrt(v), norm = size + (double)s.eps;
        // G times a power of two near kSX / |G| (exact), then the rest of the factor
        double mul = 1.0;
        if (isfinite(norm) && norm > 0)
            mul = exp2((double)min(max(13 - (int)ceil(log2(size > 0 ? size : norm)), -126), 126));
        s_mul = (float)mul;
        s_size = norm > 0 ? (float)(size / norm) : 0.f;
        s_over = (float)(isfinite(norm) ? (double)kSX * power2(x_shift(s_size)) / (mul * norm) : nan(""));
    }
    __syncthreads();
    const float mul = s_mul, over = s_over;
    float bound = s_size;         // of X's singular values
    int shift = x_shift(bound);   // X's factor is kSX times this power of two
    for (int i = tid; i < mn; i += THREADS) {
        const int r = i / s.n, c = i - r * s.n;
        const uint32_t o = wide ? place(r, c) : place(c, r);
        const float x = to_f<T>(G[i]) * mul * over;
        const __half h = __float2half_rn(x);
        *reinterpret_cast<__half *>(xh + o) = h;
        *reinterpret_cast<__half *>(xl + o) = __float2half_rn(x - __half2float(h));
    }
    const uint32_t tmem = tmem_slot;
    const uint32_t t_s = tmem, t_x = tmem + 128;   // A and A A; X
    const uint32_t idesc = (1u << 4) | (8u << 24);   // fp16 operands, fp32 sums, 128 rows
    const int pk = (p + 15) / 16, qk = (q + 15) / 16;
    const uint32_t ax[2] = {smem_u32(xh), smem_u32(xl)}, as[2] = {smem_u32(sh), smem_u32(sl)};
    const int row = 32 * (warp & 3) + lane, half = warp >> 2;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const bool rows = 32 * (warp & 3) < p;   // this warp's rows hold some of X's
    uint32_t parity = 0;
    bool ok = true;

    // X, A or B written by all: visible to the tensor cores before the next phase
    auto written = [&]() {
        fence_async_smem();
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
    };
    // the phase's products are done (the same answer for all threads; false when
    // a wait ran out)
    auto done = [&]() {
        const int got = wait_bar(bar, parity, ctl);
        parity ^= 1u;
        tc_fence_after();
        return __syncthreads_and(got) != 0;
    };
    // d = a a^T over `steps` steps of 16 columns
    auto square = [&](uint32_t d, const uint32_t *t, int steps) {
        const uint32_t id = idesc | ((uint32_t)(pk * 16 >> 3) << 17);
        bool first = true;
        for (int term = 0; term < 3; ++term)
            for (int k = 0; k < steps; ++k) {
                const uint32_t o = (uint32_t)(k >> 2) * BLOCK + (k & 3) * 32;
                mma<1>(d, sdesc_sw128(t[term == 2] + o), sdesc_sw128(t[term == 1] + o), id,
                       first ? 0u : 1u);
                first = false;
            }
        mma_commit(bar);
    };

    for (int i = 0; ok && i < s.steps; ++i) {
        const bool last = i + 1 == s.steps;
        const int was = shift;
        bound = next_bound(bound, s.a, s.b, s.c);
        shift = x_shift(bound);
        written();
        if (tid == 0)
            square(t_s, ax, qk);
        if (!(ok = done()))
            break;
        const float fa = kSA / (kSX * kSX) * power2(-was) * power2(-was);
        if (rows)
            for (int c = 16 * half; c < 16 * pk; c += 32) {
                float f[16];
                tmem_ld16(t_s + lanes + c, f);
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    f[j] *= fa;
                put16(sh, sl, row, c, f);
            }
        written();
        if (tid == 0)
            square(t_s, as, pk);
        if (!(ok = done()))
            break;
        if (rows)
            for (int c = 16 * half; c < 16 * pk; c += 32) {
                float f[16], g[16];
                tmem_ld16(t_s + lanes + c, f);
                get16(sh, sl, row, c, g);
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    f[j] = s.c * kSB / (kSA * kSA) * f[j] + s.b * kSB / kSA * g[j];
                    if (c + j == row && row < p)
                        f[j] += s.a * kSB;
                }
                put16(sh, sl, row, c, f);
            }
        written();
        if (tid == 0) {
            for (int n0 = 0; n0 < qb; n0 += 4) {   // up to 256 columns at a time
                const uint32_t id = idesc | (1u << 16) |
                                    ((uint32_t)(min(4, qb - n0) * 64 >> 3) << 17);
                bool first = true;
                for (int term = 0; term < 3; ++term)
                    for (int k = 0; k < pk; ++k) {
                        const uint32_t oa = (uint32_t)(k >> 2) * BLOCK + (k & 3) * 32;
                        const uint32_t ob = (uint32_t)n0 * BLOCK + k * 2048;
                        mma<1>(t_x + n0 * 64, sdesc_sw128(as[term == 2] + oa),
                               sdesc_mn(ax[term == 1] + ob, BLOCK), id, first ? 0u : 1u);
                        first = false;
                    }
            }
            mma_commit(bar);
        }
        if (!(ok = done()))
            break;
        if (rows) {
            const float f0 = (last ? s.scale / kSX : power2(shift)) / kSB * power2(-was);
            for (int c = 16 * half; c < 16 * qk; c += 32) {
                float f[16];
                tmem_ld16(t_x + lanes + c, f);
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    f[j] *= f0;
                if (!last) {
                    put16(xh, xl, row, c, f);
                } else if (row < p) {
                    __nv_bfloat16 *U = s.U + (int64_t)blockIdx.x * mn;
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (c + j < q)
                            U[wide ? row * s.n + c + j : (c + j) * s.n + row] =
                                __float2bfloat16_rn(f[j]);
                }
            }
        }
    }
    if (!ok && tid == 0) {   // what was issued still has to end before TMEM is freed
        wait_bar(bar, parity ^ 1u, ctl, false);
    }
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && abort_flag)
        atomicExch(&g_gave_up, (int32_t)MOE_ERR_DEVICE_TIMEOUT);
    if (warp == 0) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols)
                     : "memory");
    }
}

int small_smem(int m, int n)
{
    const int p = m < n ? m : n, q = m < n ? n : m;
    const int need = 2 * ((p + 63) / 64 + (q + 63) / 64) * BLOCK + 1024;
    const int least = (tmem_cols((q + 63) / 64) == 256 ? 112 : 116) * 1024;   // two blocks an SM, or one
    return need > least ? need : least;
}

}  // namespace

cudaError_t gave_up_small(int32_t **word)
{
    return cudaGetSymbolAddress(reinterpret_cast<void **>(word), g_gave_up);
}

// X in two terms, A in two: what fits in a block's shared memory, and 128 rows
bool orthogonalize_is_small(int m, int n)
{
    const int p = m < n ? m : n, q = m < n ? n : m;
    return p <= 128 && q <= 320;
}

cudaError_t launch_orthogonalize_small(bool bf16, int E, int m, int n, const void *G, int steps,
                                       float a, float b, float c, float eps, float scale, void *U,
                                       int32_t *status, cudaStream_t s)
{
    const SmallParams p{G, static_cast<__nv_bfloat16 *>(U), m, n, steps, a, b, c, eps, scale,
                        status};
    const int smem = small_smem(m, n);
    auto kern = bf16 ? ns_small_kernel<__nv_bfloat16> : ns_small_kernel<float>;
    cudaError_t err = raise_smem_limit((const void *)kern, smem);
    if (err != cudaSuccess)
        return err;
    return launch_pdl(kern, dim3(E), dim3(THREADS), smem, s, p);
}

}  // namespace grp
}  // namespace moe
