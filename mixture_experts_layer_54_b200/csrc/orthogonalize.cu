// Orthogonalised updates of stacked expert matrices by Newton-Schulz products:
//   X = G / (|G|_F + eps), then `steps` times  A = X X^T (X^T X when X is
//   tall), X = a X + (b A + c A A) X (a X + X (b A + c A A)),
// which drives the singular values towards 1 and keeps the singular vectors.
//
// Bound by the tensor cores.  The products run on the fp16 pipe (the rate of
// bf16, 3 more bits) on fp16 copies of X, A and B = b A + c A A with powers of
// two as scales (orthogonalize.cuh), so nothing is near the ends of fp16's range
// while the singular values stay below about 2.8.  A step multiplies small singular
// values by a = 3.4, so what a rounding of X (2^-11) leaves among them in the
// first of five steps comes out 140 times as large: 2e-2 of the result for an
// update of rank 32, measured.  That noise only passes through a X, since B
// multiplies those directions by almost nothing; so X is held as two fp16
// terms (hi + lo, 22 bits), a X takes both and the products only hi.  The
// result is then within 2e-3 of the 64-bit one (2-norm; 1.4e-3 for noise, 6e-4
// for decaying spectra, 1.8e-3 for rank 32), at the cost of one product each,
// where two terms in every product cost 2.6 times as much for 8e-4.  a hi comes
// with the product, as a on B's diagonal (one array less to read in its
// epilogue: 8 to 6 bytes an element), and the last step reads hi alone: near
// singular value 1 the same X in both places is the more exact.  A bf16 G times
// a power of two is exact in one term (but for elements below 2^-30 of its norm).
// A and B are symmetric: only tiles on or below the diagonal are computed and
// mirrored.
#include "grouped.cuh"
#include "orthogonalize.cuh"

#include <cuda_fp16.h>
#include <math.h>
#include <string.h>

namespace moe {
namespace grp {

namespace {

constexpr int kMaxParts = 256;

inline int64_t up8(int64_t v) { return (v + 7) / 8 * 8; }

// 8 consecutive elements from p (`vec`: p is 16-byte aligned), n of them valid
template <typename T>
__device__ __forceinline__ void load8(const T *p, int n, bool vec, float *f)
{
    if (vec && n >= 8) {
        if (sizeof(T) == 2) {
            const uint4 u = *reinterpret_cast<const uint4 *>(p);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = __uint_as_float(w[i] << 16);
                f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float4 u = reinterpret_cast<const float4 *>(p)[h];
                f[4 * h] = u.x, f[4 * h + 1] = u.y, f[4 * h + 2] = u.z, f[4 * h + 3] = u.w;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = i < n ? to_f<T>(p[i]) : 0.f;
    }
}

// Whether a sum of squares taken in fp32 can be wrong: some overflowed, or the
// sum is so small that those which vanished (2^-149 each) could matter.
__device__ __forceinline__ bool squares_outside(double v) { return !(v >= 1e-20 && v <= 1e38); }

// Sums of squares of `parts` slices of each matrix (fp32 in a thread, then
// double over the block; fixed order).  Four 8-element pieces of a thread are
// in flight at a time.  A slice whose squares leave fp32's range is summed again
// in double.
template <typename T>
__global__ void __launch_bounds__(256)
    square_sums_kernel(const T *G, int64_t mn, int parts, bool vec, double *out)
{
    pdl_wait();
    pdl_trigger();
    const int e = blockIdx.y;
    const T *g = G + e * mn;
    const int64_t step = parts * 2048ll;
    float acc[4] = {};
    for (int64_t i = (blockIdx.x * 256ll + threadIdx.x) * 8; i < mn; i += 4 * step) {
        float f[4][8];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int64_t o = i + u * step;
            const int n = mn - o < 8 ? (int)(mn - o) : 8;
            load8(g + (n > 0 ? o : 0), n, vec, f[u]);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                acc[u] = fmaf(f[u][j], f[u][j], acc[u]);
    }
    __shared__ double part[8];
    __shared__ int again;
    auto block_sum = [&](double v) {   // thread 0's answer is the block's
#pragma unroll
        for (int s = 16; s; s >>= 1)
            v += __shfl_xor_sync(0xffffffffu, v, s);
        if ((threadIdx.x & 31) == 0)
            part[threadIdx.x >> 5] = v;
        __syncthreads();
        if (threadIdx.x == 0)
            for (int i = 1; i < 8; ++i)
                v += part[i];
        return v;
    };
    double v = block_sum((double)acc[0] + acc[1] + acc[2] + acc[3]);
    if (threadIdx.x == 0)
        again = squares_outside(v);
    __syncthreads();
    if (again) {
        v = 0;
        for (int64_t i = (blockIdx.x * 256ll + threadIdx.x) * 8; i < mn; i += step)
            for (int64_t j = i; j < i + 8 && j < mn; ++j) {
                const double x = (double)to_f<T>(g[j]);
                v += x * x;
            }
        v = block_sum(v);
    }
    if (threadIdx.x == 0)
        out[e * kMaxParts + blockIdx.x] = v;
}

struct Coeffs {
    float a, b, c;
};

// X = G 2^k as one or two fp16 terms, 2^k the power of two that brings |G| into
// (kSX / 2, kSX]; scale[e] = 2^k (|G| + eps) is then what X stands over.  scale[i E
// + e], from i = 1 on, is X's factor before step i.
// Rows of a multiple of 8 elements are one run of them; others go row by row.
template <typename T>
__global__ void __launch_bounds__(256)
    scale_kernel(const T *G, int m, int n, int64_t ld, int parts, bool vec, const double *sums,
                 float eps, Coeffs co, int steps, __half *hi, __half *lo, float *scale)
{
    pdl_wait();
    pdl_trigger();
    const int e = blockIdx.y;
    __shared__ float s_mul[2];   // 2^k as two factors: k may pass fp32's exponents
    if (threadIdx.x < 32) {
        double v = 0;
        for (int i = threadIdx.x; i < parts; i += 32)
            v += sums[e * kMaxParts + i];
#pragma unroll
        for (int s = 16; s; s >>= 1)
            v += __shfl_xor_sync(0xffffffffu, v, s);
        if (threadIdx.x == 0) {
            const double size = sqrt(v), norm = size + (double)eps;
            double sc = norm;   // zero with eps = 0: 0 / 0 as the formula has it
            int k = 0;
            if (isfinite(norm) && norm > 0) {
                k = 13 - (int)ceil(log2(size > 0 ? size : norm));
                k = min(k, 100 - (int)ceil(log2(norm)));   // sc stays in fp32's range
                sc = exp2((double)k) * norm;
            } else if (!isfinite(norm)) {
                sc = nan("");   // an infinity or NaN in G: the whole update is NaN
            }
            const int k0 = min(max(k, -126), 126);
            s_mul[0] = (float)exp2((double)k0);
            s_mul[1] = (float)exp2((double)(k - k0));
            if (blockIdx.x == 0) {
                scale[e] = (float)sc;
                float u = norm > 0 ? (float)(size / norm) : 0.f;
                for (int i = 1; i < steps; ++i) {
                    u = next_bound(u, co.a, co.b, co.c);
                    scale[(int64_t)i * gridDim.y + e] = kSX * power2(x_shift(u));
                }
            }
        }
    }
    __syncthreads();
    const float mul = s_mul[0], mul2 = s_mul[1];
    const int cpr = (int)(ld / 8);
    const int64_t chunks = (int64_t)m * cpr;
    const bool flat = n == ld;
    const T *g = G + (int64_t)e * m * n;
    __half *oh = hi + (int64_t)e * m * ld, *ol = lo ? lo + (int64_t)e * m * ld : nullptr;
    const int64_t step = gridDim.x * 256ll;
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < chunks; i += 2 * step) {
        float f[2][8];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int64_t k = i + u * step;
            if (k < chunks) {
                if (flat) {
                    load8(g + 8 * k, 8, vec, f[u]);
                } else {
                    const int64_t r = k / cpr;
                    const int c = (int)(k - r * cpr) * 8;
                    load8(g + r * n + c, n - c < 8 ? n - c : 8, vec, f[u]);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int64_t k = i + u * step;
            if (k >= chunks)
                break;
            uint32_t h[4], l[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float x0 = f[u][2 * j] * mul * mul2, x1 = f[u][2 * j + 1] * mul * mul2;
                const __half2 a = __floats2half2_rn(x0, x1);
                const float2 b = __half22float2(a);
                const __half2 d = __floats2half2_rn(x0 - b.x, x1 - b.y);
                h[j] = *reinterpret_cast<const uint32_t *>(&a);
                l[j] = *reinterpret_cast<const uint32_t *>(&d);
            }
            *reinterpret_cast<uint4 *>(oh + 8 * k) = make_uint4(h[0], h[1], h[2], h[3]);
            if (ol)
                *reinterpret_cast<uint4 *>(ol + 8 * k) = make_uint4(l[0], l[1], l[2], l[3]);
        }
    }
}

// Tiles of E products of M x N over K: a round of 256 x 256 tiles on SM pairs
// costs its contraction (0.8 us for 128, bound by the loads, and as much for 128
// x 128 tiles on single SMs) and 8 us at its end, where the small tiles take 4;
// four times as many of them go two to a pair.
Tiles ns_tiles(int E, int M, int N, int K, bool sym)
{
    auto rounds = [&](int t, int units) {
        const int64_t r = ceil_div(M, t), c = ceil_div(N, t);
        return ceil_div(E * (sym ? r * (r + 1) / 2 : r * c), units);
    };
    const int sms = device_sms();
    const double k = 0.8 * ceil_div(K, 128);
    return rounds(256, sms / 2) * (k + 8) <= rounds(128, sms) * (k + 4) ? PAIR_256 : ONE_128;
}

struct Bufs {
    int32_t *status;
    unsigned long long *counters;
    float *partial;
    double *sums;
    float *scale;
    __half *X[2][2], *A, *B;   // X: [ping-pong][hi, lo]
    size_t bytes;
};

Bufs carve(int64_t E, int64_t m, int64_t n, int steps, void *ws)
{
    Bufs b;
    char *base = static_cast<char *>(ws);
    size_t off = 0;
    auto take = [&](size_t bytes) {
        void *p = base ? base + off : nullptr;
        off = align_up(off + bytes, 256);
        return p;
    };
    const int64_t p = m < n ? m : n;
    const size_t x = (size_t)(E * m * up8(n)) * 2, a = (size_t)(E * p * up8(p)) * 2;
    b.status = static_cast<int32_t *>(take(256));
    b.counters = static_cast<unsigned long long *>(take(kCounterBytes));
    b.partial = static_cast<float *>(take(kPartialBytes));
    b.sums = static_cast<double *>(take((size_t)E * kMaxParts * 8));
    b.scale = static_cast<float *>(take((size_t)steps * E * 4));
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2; ++j)
            b.X[i][j] = static_cast<__half *>(take(steps > 1 || i + j == 0 ? x : 0));
    b.A = static_cast<__half *>(take(a));
    b.B = static_cast<__half *>(take(a));
    b.bytes = off;
    return b;
}

}  // namespace

bool orthogonalize_is_small(int m, int n);
cudaError_t launch_orthogonalize_small(bool bf16, int E, int m, int n, const void *G, int steps,
                                       float a, float b, float c, float eps, float scale, void *U,
                                       int32_t *status, cudaStream_t s);

bool orthogonalize_is_gram(int m, int n, double growth);
size_t orthogonalize_gram_bytes(int64_t E, int m, int n);
cudaError_t launch_orthogonalize_gram(bool bf16, int E, int m, int n, const void *G, int steps,
                                      float a, float b, float c, float eps, float scale, void *U,
                                      void *ws, cudaStream_t s);

size_t orthogonalize_bytes(int64_t E, int64_t m, int64_t n, int steps)
{
    if (orthogonalize_is_small((int)m, (int)n))
        return 256;   // the status word alone
    const size_t bytes = carve(E, m, n, steps, nullptr).bytes;
    // the coefficients decide between the two
    const size_t gram = orthogonalize_is_gram((int)m, (int)n, 1)
                            ? orthogonalize_gram_bytes(E, (int)m, (int)n) : 0;
    return bytes > gram ? bytes : gram;
}

cudaError_t launch_orthogonalize(bool bf16, int E, int m, int n, const void *G, int steps,
                                 float a, float b, float c, double growth, float eps, float scale,
                                 void *U, void *ws, cudaStream_t s)
{
    if (orthogonalize_is_small(m, n))
        return launch_orthogonalize_small(bf16, E, m, n, G, steps, a, b, c, eps, scale, U,
                                          static_cast<int32_t *>(ws), s);
    if (orthogonalize_is_gram(m, n, growth))
        return launch_orthogonalize_gram(bf16, E, m, n, G, steps, a, b, c, eps, scale, U, ws, s);
    Bufs w = carve(E, m, n, steps, ws);
    const int64_t mn = (int64_t)m * n, ldx = up8(n);
    const bool wide = m <= n;
    const int p = wide ? m : n, q = wide ? n : m;
    const int64_t lda = up8(p);
    const int esz = bf16 ? 2 : 4;
    const bool al = (reinterpret_cast<uintptr_t>(G) & 15u) == 0;
    const int64_t want = ceil_div(mn, 256 * 8 * 4);
    const int64_t cap = ceil_div(device_sms() * 6, E);   // a few blocks an SM over all matrices
    const int64_t most_parts = cap < kMaxParts ? cap : kMaxParts;
    const int parts = (int)(want < 1 ? 1 : (want > most_parts ? most_parts : want));
    const bool vsum = al && mn * esz % 16 == 0, vrow = al && (int64_t)n * esz % 16 == 0;
    int64_t cblocks = ceil_div((int64_t)m * (ldx / 8), 256);
    const int64_t most = ceil_div(device_sms() * 16, E);
    cblocks = cblocks > most ? most : cblocks;
    // X0 needs its low half unless G is bf16 (exact in one term) or this is the only step
    const bool lo0 = !bf16 && steps > 1;
    const Coeffs co{a, b, c};
    cudaError_t err = clear_for_replay(w.counters, s);
    if (err != cudaSuccess)
        return err;
    if (bf16) {
        const __nv_bfloat16 *g = static_cast<const __nv_bfloat16 *>(G);
        err = launch_pdl(square_sums_kernel<__nv_bfloat16>, dim3(parts, E), dim3(256), 0, s, g, mn,
                         parts, vsum, w.sums);
        if (err == cudaSuccess)
            err = launch_pdl(scale_kernel<__nv_bfloat16>, dim3((unsigned)cblocks, E), dim3(256), 0,
                             s, g, m, n, ldx, parts, vrow, (const double *)w.sums, eps, co, steps,
                             w.X[0][0], lo0 ? w.X[0][1] : nullptr, w.scale);
    } else {
        const float *g = static_cast<const float *>(G);
        err = launch_pdl(square_sums_kernel<float>, dim3(parts, E), dim3(256), 0, s, g, mn, parts,
                         vsum, w.sums);
        if (err == cudaSuccess)
            err = launch_pdl(scale_kernel<float>, dim3((unsigned)cblocks, E), dim3(256), 0, s, g, m,
                             n, ldx, parts, vrow, (const double *)w.sums, eps, co, steps,
                             w.X[0][0], lo0 ? w.X[0][1] : nullptr, w.scale);
    }
    if (err != cudaSuccess)
        return err;
    const int box = b_box(EPI_NS, PAIR_256), sk = stage_k(EPI_NS, PAIR_256);   // the same for ONE_128
    const bool nw = is_wide(n), pw = is_wide(p);
    int cur = 0;
    for (int i = 0; i < steps; ++i, cur ^= 1) {
        const bool last = i + 1 == steps;
        __half *X = w.X[cur][0], *Xlo = !last && (i > 0 || lo0) ? w.X[cur][1] : nullptr;
        bool ok = true;
        Params P;
        memset(&P, 0, sizeof P);
        P.nsets = 1;
        P.fp16 = 1;
        P.counters = w.counters;
        P.partial = w.partial;
        P.partial_bytes = kPartialBytes;
        P.status = w.status;
        P.clear_status = i == 0;
        Set &t = P.set[0];
        t.mode = DENSE;
        t.groups = E;
        t.a_grouped = t.b_grouped = 1;
        t.segs = t.period = 1;

        // A = X X^T (X^T X)
        t.M = t.N = p;
        t.K = q;
        t.sym = 1;
        t.a_wide = t.b_wide = nw;
        if (wide) {
            ok &= map_k(&t.a[0], X, m, n, ldx, E, m * ldx, 128, sk, nw);
            ok &= map_k(&t.b[0], X, m, n, ldx, E, m * ldx, box, sk, nw);
        } else {
            ok &= map_mn(&t.a[0], X, m, n, ldx, E, m * ldx, sk, 128, nw);
            ok &= map_mn(&t.b[0], X, m, n, ldx, E, m * ldx, sk, box, nw);
        }
        t.out = w.A;
        t.ld = (int)lda;
        t.out_group = p * lda;
        const float *scale_i = w.scale + (int64_t)i * E;
        t.alpha = kSA;
        t.scale = scale_i;
        t.scale_pow = 2;
        if (!ok)
            return cudaErrorInvalidValue;
        if ((err = launch_tc(P, EPI_NS, wide ? A_K_B_K : A_MN_B_MN,
                             ns_tiles(E, p, p, q, true), s)) != cudaSuccess)
            return err;

        // B = a I + b A + c A A
        P.clear_status = 0;
        t.K = p;
        t.a_wide = t.b_wide = pw;
        ok &= map_k(&t.a[0], w.A, p, p, lda, E, p * lda, 128, sk, pw);
        ok &= map_k(&t.b[0], w.A, p, p, lda, E, p * lda, box, sk, pw);
        t.out = w.B;
        t.alpha = c * kSB / (kSA * kSA);
        t.beta = b * kSB / kSA;
        t.diag = a * kSB;
        t.base = w.A;
        t.base_ld = (int)lda;
        t.base_group = p * lda;
        t.scale = nullptr;
        if (!ok)
            return cudaErrorInvalidValue;
        if ((err = launch_tc(P, EPI_NS, A_K_B_K, ns_tiles(E, p, p, p, true), s)) != cudaSuccess)
            return err;

        // X = B hi + a lo (hi B + a lo)
        t.sym = 0;
        t.diag = 0.f;
        t.M = m;
        t.N = n;
        t.a_wide = wide ? pw : nw;
        t.b_wide = wide ? nw : pw;
        if (wide) {
            ok &= map_k(&t.a[0], w.B, p, p, lda, E, p * lda, 128, sk, pw);
            ok &= map_mn(&t.b[0], X, m, n, ldx, E, m * ldx, sk, box, nw);
        } else {
            ok &= map_k(&t.a[0], X, m, n, ldx, E, m * ldx, 128, sk, nw);
            ok &= map_k(&t.b[0], w.B, p, p, lda, E, p * lda, box, sk, pw);
        }
        t.alpha = (last ? scale : 1.f) / kSB;
        t.beta = a;   // with lo, which the last step does without
        t.scale = scale_i;
        t.scale_to = last ? nullptr : scale_i + E;
        t.scale_pow = 1;
        t.base = Xlo;
        t.base_ld = (int)ldx;
        t.base_group = m * ldx;
        t.out = last ? U : w.X[cur ^ 1][0];
        t.out2 = i + 2 < steps ? w.X[cur ^ 1][1] : nullptr;   // the last step reads hi alone
        t.out_bf16 = last;
        t.ld = last ? n : (int)ldx;
        t.out_group = last ? mn : m * ldx;
        if (!ok)
            return cudaErrorInvalidValue;
        if ((err = launch_tc(P, EPI_NS, wide ? A_K_B_MN : A_K_B_K,
                             ns_tiles(E, m, n, p, false), s)) != cudaSuccess)
            return err;
    }
    return cudaSuccess;
}

}  // namespace grp
}  // namespace moe
