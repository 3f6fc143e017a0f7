// Orthogonalised updates of matrices of few rows or columns (p <= 56) that are too
// long for the one-block form.  Their singular values lie together, and where the
// steps amplify them the fp16 roundings of the stacked products, alike in all of
// them, came out as 7.5e-3 (4 x 637) and 4.2e-3 (32 x 700) of the result.
//
// All matrices of the steps are polynomials of X X^T (X is p x q, a tall G read
// transposed), so the steps run on p x p alone, in double:
//   S = G G^T;  n = sqrt(trace S) + eps;  A = S / n^2, P = I;
//   steps of  B = a I + b A + c A A,  P = B P,  A = B A B;  U = scale P G / n.
// G is read twice and nothing else of its size is: three launches, the first bound
// by double FMAs (p p q), the second by one block's (4 p^3 a step), the third by
// fp32 FMAs (p p q).  Against the stacked products: 8 of 56 x 4096 155 us from 180,
// 64 of 56 x 1024 201 from 193, 1 of 8 x 4096 30 from 133.
#include "orthogonalize.cuh"

#include "internal.cuh"

namespace moe {
namespace grp {

namespace {

constexpr int THREADS = 256;
constexpr int SLICE = 32;   // columns of X at a time in the first launch

struct GramParams {
    const void *G;
    __nv_bfloat16 *U;
    int m, n, steps, parts, ld;   // ld: p rounded up to 4
    float a, b, c, eps, scale;
    double *sums;                 // [E][parts][ld][ld]
    float *P;                     // [E][ld][ld]: P scale / (2^k n)
    float *mul;                   // [E][2]: 2^k as two factors, |G| 2^k near 1
    int32_t *status;
};

// Row (column) i of a thread's 4 x 4 values: two neighbours in either half of the
// matrix, so that 16-byte reads of neighbouring threads are neighbours too.
__device__ __forceinline__ int place4(int t, int i, int ld) { return 2 * t + (i & 1) + (i >> 1) * (ld / 2); }

// acc += x y^T of the 4 x 4 values (r, c) for one contraction index: its rows of x
// and y, ld wide.
__device__ __forceinline__ void outer(const double *x, const double *y, int r, int c, int ld,
                                      double (&acc)[4][4])
{
    double f[4], g[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const double2 u = *reinterpret_cast<const double2 *>(x + place4(r, 2 * h, ld));
        const double2 v = *reinterpret_cast<const double2 *>(y + place4(c, 2 * h, ld));
        f[2 * h] = u.x, f[2 * h + 1] = u.y;
        g[2 * h] = v.x, g[2 * h + 1] = v.y;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc[i][j] = fma(f[i], g[j], acc[i][j]);
}

// The first product: this block's columns' part of G G^T, 4 x 4 values a thread.
template <typename T>
__global__ void __launch_bounds__(THREADS) gram_kernel(const GramParams s)
{
    __shared__ __align__(16) double x[SLICE][64];
    const bool wide = s.m <= s.n;
    const int p = wide ? s.m : s.n, q = wide ? s.n : s.m, nb = s.ld / 4, tid = threadIdx.x;
    const int r = tid / nb, c = tid % nb;
    pdl_wait();
    pdl_trigger();
    if (blockIdx.x + blockIdx.y == 0 && tid == 0)
        *s.status = 0;
    const T *G = static_cast<const T *>(s.G) + (int64_t)blockIdx.y * s.m * s.n;
    const int each = (q + s.parts * SLICE - 1) / (s.parts * SLICE) * SLICE;
    const int64_t first = (int64_t)blockIdx.x * each;
    const int64_t end = first + each < q ? first + each : q;
    double acc[4][4] = {};
    for (int64_t q0 = first; q0 < end; q0 += SLICE) {
        __syncthreads();
        for (int i = tid; i < SLICE * s.ld; i += THREADS) {
            // neighbouring threads along the contiguous index
            const int k = wide ? i % SLICE : i / s.ld, j = wide ? i / SLICE : i % s.ld;
            const bool in = j < p && q0 + k < end;
            x[k][j] = in ? (double)to_f<T>(wide ? G[(int64_t)j * s.n + q0 + k] : G[(q0 + k) * s.n + j])
                         : 0.;
        }
        __syncthreads();
        if (r < nb)
#pragma unroll 4
            for (int k = 0; k < SLICE; ++k)
                outer(x[k], x[k], r, c, s.ld, acc);
    }
    if (r < nb) {
        double *out = s.sums + ((int64_t)blockIdx.y * s.parts + blockIdx.x) * s.ld * s.ld;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                out[place4(r, i, s.ld) * s.ld + place4(c, j, s.ld)] = acc[i][j];
    }
}

// out(i, j, (x y)(i, j)) of two symmetric matrices that commute (so x is read along
// its rows as well), pitch ld; the block's threads take 4 x 4 values each.
template <typename F>
__device__ __forceinline__ void product(const double *x, const double *y, int ld, F out)
{
    const int nb = ld / 4, t = threadIdx.x;
    if (t < nb * nb) {
        const int r = t / nb, c = t % nb;
        double acc[4][4] = {};
#pragma unroll 4
        for (int k = 0; k < ld; ++k)
            outer(x + k * ld, y + k * ld, r, c, ld, acc);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                out(place4(r, i, ld), place4(c, j, ld), acc[i][j]);
    }
    __syncthreads();
}

__global__ void __launch_bounds__(THREADS) gram_steps_kernel(const GramParams s)
{
    extern __shared__ __align__(16) double mats[];
    const int p = s.m < s.n ? s.m : s.n, ld = s.ld, size = ld * ld, tid = threadIdx.x;
    double *A = mats, *B = A + size, *P = B + size, *T = P + size;
    __shared__ double inv, factor;
    pdl_wait();
    pdl_trigger();
    const double *sums = s.sums + (int64_t)blockIdx.x * s.parts * size;
    for (int i = tid; i < size; i += THREADS) {
        double v = 0;
        for (int k = 0; k < s.parts; ++k)
            v += sums[(int64_t)k * size + i];
        A[i] = v;
    }
    __syncthreads();
    if (tid == 0) {
        double v = 0;
        for (int i = 0; i < p; ++i)
            v += A[i * ld + i];
        const double len = sqrt(v), norm = len + (double)s.eps;
        int k = 0;
        if (isfinite(norm) && norm > 0)
            k = -(int)ceil(log2(len > 0 ? len : norm));
        const int k0 = min(max(k, -126), 126);
        s.mul[2 * blockIdx.x] = (float)exp2((double)k0);
        s.mul[2 * blockIdx.x + 1] = (float)exp2((double)(k - k0));
        inv = 1 / norm;   // zero with eps = 0: NaN as the formula has it
        // an infinity or NaN in G: the whole update is NaN
        factor = isfinite(norm) ? (double)s.scale / (exp2((double)k) * norm) : nan("");
    }
    __syncthreads();
    for (int i = tid; i < size; i += THREADS)
        A[i] = A[i] * inv * inv;
    __syncthreads();
    for (int step = 0; step < s.steps; ++step) {
        product(A, A, ld, [&](int i, int j, double v) {
            B[i * ld + j] = (i == j && i < p ? (double)s.a : 0.) + (double)s.b * A[i * ld + j] +
                            (double)s.c * v;
        });
        if (step > 0) {
            product(B, P, ld, [&](int i, int j, double v) { T[i * ld + j] = v; });
            double *t = P;
            P = T;
            T = t;
        } else {   // P was the identity
            for (int i = tid; i < size; i += THREADS)
                P[i] = B[i];
        }
        if (step + 1 < s.steps) {
            product(B, A, ld, [&](int i, int j, double v) { T[i * ld + j] = v; });
            product(T, B, ld, [&](int i, int j, double v) { A[i * ld + j] = v; });
        }
    }
    for (int i = tid; i < size; i += THREADS)
        s.P[(int64_t)blockIdx.x * size + i] = (float)(P[i] * factor);
}

// U = P G: a thread takes 16 of the p values of one column (of a quarter, a half or
// all of the block's threads' columns).
template <typename T>
__global__ void __launch_bounds__(THREADS) gram_apply_kernel(const GramParams s)
{
    __shared__ __align__(16) float P[64 * 64];
    __shared__ float x[64 * 64];            // [p][columns]
    const bool wide = s.m <= s.n;
    const int p = wide ? s.m : s.n, q = wide ? s.n : s.m, tid = threadIdx.x;
    const int groups = p > 32 ? 4 : p > 16 ? 2 : 1, cols = THREADS / groups;
    pdl_wait();
    pdl_trigger();
    const int64_t e = blockIdx.y, at = e * s.m * s.n, q0 = (int64_t)blockIdx.x * cols;
    const int n = q - q0 < cols ? (int)(q - q0) : cols;
    const T *G = static_cast<const T *>(s.G) + at;
    __nv_bfloat16 *U = s.U + at;
    const float mul = s.mul[2 * e], mul2 = s.mul[2 * e + 1];
    for (int i = tid; i < 64 * 64; i += THREADS) {   // pitch 64; rows and columns past p: 0
        const int j = i >> 6, k = i & 63;
        P[i] = j < p && k < p ? s.P[(e * s.ld + j) * s.ld + k] : 0.f;
    }
    for (int i = tid; i < p * n; i += THREADS) {
        const int j = wide ? i / n : i % p, c = wide ? i % n : i / p;
        x[j * cols + c] = to_f<T>(wide ? G[(int64_t)j * s.n + q0 + c] : G[q0 * s.n + i]) * mul * mul2;
    }
    __syncthreads();
    const int c = tid % cols, r = tid / cols * 16;
    float acc[16] = {};
    if (c < n)
        for (int k = 0; k < p; ++k) {
            const float v = x[k * cols + c];
            const float4 *row = reinterpret_cast<const float4 *>(P + k * 64 + r);   // symmetric
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 w = row[i];
                acc[4 * i] = fmaf(w.x, v, acc[4 * i]);
                acc[4 * i + 1] = fmaf(w.y, v, acc[4 * i + 1]);
                acc[4 * i + 2] = fmaf(w.z, v, acc[4 * i + 2]);
                acc[4 * i + 3] = fmaf(w.w, v, acc[4 * i + 3]);
            }
        }
    if (wide) {
        if (c < n)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (r + i < p)
                    U[(int64_t)(r + i) * s.n + q0 + c] = __float2bfloat16_rn(acc[i]);
        return;
    }
    // the columns of X are U's rows, one run of n p values: out through shared memory
    __syncthreads();
    __nv_bfloat16 *stage = reinterpret_cast<__nv_bfloat16 *>(x);
    if (c < n)
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (r + i < p)
                stage[c * p + r + i] = __float2bfloat16_rn(acc[i]);
    __syncthreads();
    for (int i = tid; i < n * p; i += THREADS)
        U[q0 * s.n + i] = stage[i];
}

struct GramBufs {
    int32_t *status;
    double *sums;
    float *P, *mul;
    int parts, ld;
    size_t bytes;
};

GramBufs carve(int64_t E, int m, int n, void *ws)
{
    const int p = m < n ? m : n, q = m < n ? n : m;
    GramBufs b;
    b.ld = (p + 3) & ~3;
    // slices of 256 columns, until all matrices together have about 512
    const int64_t most = 512 / E > 1 ? 512 / E : 1, want = ceil_div(q, 256);
    b.parts = (int)(want < most ? want : most);
    char *base = static_cast<char *>(ws);
    size_t off = 0;
    auto take = [&](size_t bytes) {
        void *r = base ? base + off : nullptr;
        off = align_up(off + bytes, 256);
        return r;
    };
    b.status = static_cast<int32_t *>(take(256));
    b.sums = static_cast<double *>(take((size_t)E * b.parts * b.ld * b.ld * 8));
    b.P = static_cast<float *>(take((size_t)E * b.ld * b.ld * 4));
    b.mul = static_cast<float *>(take((size_t)E * 8));
    b.bytes = off;
    return b;
}

}  // namespace

// What the stacked products cannot hold to 2e-3; from 57 on they do, and are the
// faster of the two.  growth: P is held in fp32 for the last product, so where a
// singular value is zero the result is off by growth 2^-24; the quintic's six steps
// are 1670.  (X itself, which the stacked products keep, stays bounded however many
// steps there are.)
bool orthogonalize_is_gram(int m, int n, double growth)
{
    return (m < n ? m : n) <= 56 && growth <= 2048;
}

size_t orthogonalize_gram_bytes(int64_t E, int m, int n) { return carve(E, m, n, nullptr).bytes; }

cudaError_t launch_orthogonalize_gram(bool bf16, int E, int m, int n, const void *G, int steps,
                                      float a, float b, float c, float eps, float scale, void *U,
                                      void *ws, cudaStream_t s)
{
    const GramBufs w = carve(E, m, n, ws);
    const GramParams p{G,      static_cast<__nv_bfloat16 *>(U), m, n, steps, w.parts, w.ld, a, b, c, eps, scale,
                       w.sums, w.P, w.mul, w.status};
    const int smem = 4 * w.ld * w.ld * 8, lo = m < n ? m : n, q = m < n ? n : m;
    const int cols = THREADS / (lo > 32 ? 4 : lo > 16 ? 2 : 1);
    cudaError_t err = raise_smem_limit((const void *)gram_steps_kernel, smem);
    if (err == cudaSuccess)
        err = launch_pdl(bf16 ? gram_kernel<__nv_bfloat16> : gram_kernel<float>, dim3(w.parts, E),
                         dim3(THREADS), 0, s, p);
    if (err == cudaSuccess)
        err = launch_pdl(gram_steps_kernel, dim3(E), dim3(THREADS), smem, s, p);
    if (err == cudaSuccess)
        err = launch_pdl(bf16 ? gram_apply_kernel<__nv_bfloat16> : gram_apply_kernel<float>,
                         dim3((unsigned)ceil_div(q, cols), E), dim3(THREADS), 0, s, p);
    return err;
}

}  // namespace grp
}  // namespace moe
