// Host side of the expert training calls of include/moe_b200.h: argument
// checks, workspace carving and launches.  As in api.cu nothing here allocates
// or synchronises, and an invalid call launches nothing.
#include "grouped_simt.cuh"

#include <math.h>
#include <string.h>

namespace moe {

cudaError_t launch_combine_grad(const moe_config &c, const void *dy, const void *Y_perm,
                                const float *gates, const int32_t *topk, const int32_t *pos,
                                const uint8_t *keep, const int32_t *offsets, void *dY_perm,
                                float *dgates, cudaStream_t s);

namespace grp {
size_t orthogonalize_bytes(int64_t E, int64_t m, int64_t n, int steps);
cudaError_t launch_orthogonalize(bool bf16, int E, int m, int n, const void *G, int steps, float a,
                                 float b, float c, double growth, float eps, float scale, void *U,
                                 void *ws, cudaStream_t s);
// The words that say that a bounded wait ran out on this device.
cudaError_t gave_up_grouped(int32_t **word);
cudaError_t gave_up_small(int32_t **word);
cudaError_t launch_grouped_probe(unsigned long long timeout_ns, cudaStream_t s);
}  // namespace grp

using namespace grp;

namespace {

constexpr size_t kStatusBytes = 256;
// workspace of the grouped products in bf16: status word, counters and parts of
// cut tiles
constexpr size_t kGroupedBytes = kStatusBytes + kCounterBytes + kPartialBytes;
constexpr int kMaxShared = 64;   // shared experts of one backward call (tile table)

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

moe_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

cudaError_t clear_word(void *ws, cudaStream_t s) { return cudaMemsetAsync(ws, 0, 4, s); }

struct Table {
    const int32_t *offsets, *rows;
    int n_rows;
};

Params tc_params(const Table &t, void *ws, bool clear)
{
    Params p;
    memset(&p, 0, sizeof p);
    p.offsets = t.offsets;
    p.rows = t.rows;
    p.n_rows = t.n_rows;
    p.status = static_cast<int32_t *>(ws);
    p.clear_status = clear;
    return p;
}

// Lets a launch cut tiles, with the scratch behind the status word.
void set_cut(Params &p, void *ws)
{
    char *base = static_cast<char *>(ws);
    p.counters = reinterpret_cast<unsigned long long *>(base + kStatusBytes);
    p.partial = reinterpret_cast<float *>(base + kStatusBytes + kCounterBytes);
    p.partial_bytes = kPartialBytes;
}

// Tiles for `rows` rows in `groups` groups of about the same length, n columns.
// A round of tiles costs its loads, 64 KB a stage and SM either way, so 256 x 256
// on SM pairs take over where they need fewer rounds than 128 x 128: past 128
// rows a group (8 x 200 rows through 4096 x 4096: 70 us against 92; 8 x 100: 68
// against 61).  The hidden gradients' single-SM tiles load 96 KB for 64.
Tiles row_tiles(int64_t rows, int64_t groups, int64_t n, bool hidden)
{
    const int64_t each = ceil_div(rows, groups), sms = device_sms();
    const int64_t pair = ceil_div(groups * ceil_div(each, 256) * ceil_div(n, hidden ? 128 : 256),
                                  sms / 2);
    const int64_t one = ceil_div(groups * ceil_div(each, 128) * ceil_div(n, 128), sms);
    return (hidden ? 2 * pair < 3 * one : pair < one) ? PAIR_256 : ONE_128;
}
// Weight gradients: 256 x 256 tiles once the matrix fills them.
Tiles dw_tiles(int64_t M, int64_t N) { return M >= 256 && N >= 256 ? PAIR_256 : ONE_128; }

// y [R, N] = x [R, K] W[g]^T, or with back: dx [R, K] = dy [R, N] W[g].
cudaError_t rows_tc(const Table &t, int G, int64_t R, int N, int K, const void *in, const void *W,
                    void *out, bool back, void *status, cudaStream_t s)
{
    Params p = tc_params(t, status, true);
    // Few rows a group: the weights' bytes are the work.  8 groups through 4096 x 4096
    // on 32-row tiles against 128: 55 us against 60 for 16 rows each, as for 0 to 32 rows;
    // 256 through 2048 x 1024: 192 against 212, 188 against 198.  Groups of 0 to 48 (64 to
    // 69 us against 48 to 60, 275 against 215) have a second tile where 128 rows do with one.
    const Tiles tiles = R <= 16ll * G ? ONE_32 : row_tiles(R, G, back ? K : N, false);
    Set &a = p.set[0];
    p.nsets = 1;
    a.mode = RAGGED_M;
    a.groups = G;
    a.N = back ? K : N;
    a.K = back ? N : K;
    a.segs = a.period = 1;
    a.b_grouped = 1;
    a.ld = a.N;
    a.out = out;
    const int sk = stage_k(EPI_ROWS, tiles), box = b_box(EPI_ROWS, tiles);
    a.a_wide = is_wide(a.K);
    a.b_wide = is_wide(K);
    bool ok = map_k(&a.a[0], in, R, a.K, a.K, 1, 0, tiles == ONE_32 ? 32 : 128, sk, a.a_wide);
    if (back)
        ok &= map_mn(&a.b[0], W, N, K, K, G, (int64_t)N * K, sk, box, a.b_wide);
    else
        ok &= map_k(&a.b[0], W, N, K, K, G, (int64_t)N * K, box, sk, a.b_wide);
    if (tiles == ONE_128) {
        a.has_few = 1;
        ok &= map_k(&a.a_few, in, R, a.K, a.K, 1, 0, 32, sk, false);
    }
    if (!ok)
        return cudaErrorInvalidValue;
    set_cut(p, status);
    if (may_cut(a.K)) {
        const cudaError_t e = clear_for_replay(p.counters, s);
        if (e != cudaSuccess)
            return e;
    }
    return launch_tc(p, EPI_ROWS, back ? A_K_B_MN : A_K_B_K, tiles, s);
}

// One weight-gradient set: out[g] (M x N) (= add +) sum_r a[r, :]^T b[r, :].
bool dw_set(Set &t, int mode, int groups, int64_t rows, int M, int N, const void *a, bool a_grouped,
            const void *b, bool b_grouped, const void *add, void *out, bool f32, Tiles tiles)
{
    t.mode = mode;
    t.groups = groups;
    t.M = M;
    t.N = N;
    t.K = mode == DENSE ? (int)rows : 0;
    t.segs = t.period = 1;
    t.a_grouped = a_grouped;
    t.b_grouped = b_grouped;
    t.ld = N;
    t.out_group = (int64_t)M * N;
    t.add = add;
    t.out = out;
    t.out_f32 = f32;
    // no rows: nothing is loaded, the maps only have to be valid
    const int64_t r = rows > 0 ? rows : 1;
    const void *pa = rows > 0 ? a : out, *pb = rows > 0 ? b : out;
    const int sk = stage_k(EPI_DW, tiles);
    t.a_wide = is_wide(M);
    t.b_wide = is_wide(N);
    return map_mn(&t.a[0], pa, r, M, M, a_grouped ? groups : 1, r * M, sk, 128, t.a_wide) &&
           map_mn(&t.b[0], pb, r, N, N, b_grouped ? groups : 1, r * N, sk, b_box(EPI_DW, tiles),
                  t.b_wide);
}

Simt simt_rows(const Table &t, int mode, int G, int M, int N, int K, const float *in,
               int64_t in_group, const float *W, bool back, float *out, int64_t out_group,
               const float *add)
{
    Simt p;
    memset(&p, 0, sizeof p);
    p.mode = mode;
    p.groups = G;
    p.M = M;
    p.N = back ? K : N;
    p.K = back ? N : K;
    p.a = in;
    p.a_m = p.K;
    p.a_k = 1;
    p.a_group = in_group;
    p.b = W;
    p.b_group = (int64_t)N * K;
    p.b_n = back ? 1 : K;
    p.b_k = back ? K : 1;
    p.c = out;
    p.c_m = p.N;
    p.c_group = out_group;
    p.add = add;
    p.offsets = t.offsets;
    p.rows = t.rows;
    p.n_rows = t.n_rows;
    return p;
}

Simt simt_dw(const Table &t, int mode, int G, int rows, int M, int N, const float *a,
             int64_t a_group, const float *b, int64_t b_group, const float *add, float *out)
{
    Simt p;
    memset(&p, 0, sizeof p);
    p.mode = mode;
    p.groups = G;
    p.M = M;
    p.N = N;
    p.K = mode == DENSE ? rows : 0;
    p.a = a;
    p.a_m = 1;
    p.a_k = M;
    p.a_group = a_group;
    p.b = b;
    p.b_n = 1;
    p.b_k = N;
    p.b_group = b_group;
    p.c = out;
    p.c_m = N;
    p.c_group = (int64_t)M * N;
    p.add = add;
    p.offsets = t.offsets;
    p.rows = t.rows;
    p.n_rows = t.n_rows;
    return p;
}

moe_status check_grouped(int32_t dtype, int32_t G, int64_t R, int32_t N, int32_t K)
{
    if (dtype != MOE_DTYPE_F32 && dtype != MOE_DTYPE_BF16)
        return MOE_ERR_DTYPE;
    if (G < 1 || G > kMaxE || R < 0 || R > INT32_MAX / 2 || N < 1 || K < 1 || N > 1 << 20 ||
        K > 1 << 20)
        return MOE_ERR_SHAPE;
    if (dtype == MOE_DTYPE_BF16 && (N % 8 || K % 8))
        return MOE_ERR_SHAPE;   // 16-byte rows for TMA
    return MOE_OK;
}

size_t grouped_bytes(int32_t dtype)
{
    return dtype == MOE_DTYPE_BF16 ? kGroupedBytes : kStatusBytes;
}

moe_status check_ws(const void *ws, size_t bytes, size_t need)
{
    if (!ws)
        return MOE_ERR_NULL;
    if (!aligned(ws, 256))
        return MOE_ERR_ALIGN;
    return bytes < need ? MOE_ERR_WORKSPACE : MOE_OK;
}

// fp32: nothing waits on the device, and the workspace is only the status word
moe_status check_grouped_ws(int32_t dtype, const void *ws, size_t bytes)
{
    if (dtype == MOE_DTYPE_F32 && !ws)
        return MOE_OK;
    return check_ws(ws, bytes, grouped_bytes(dtype));
}

moe_status rows_call(int32_t dtype, int32_t G, int64_t R, int32_t N, int32_t K, const void *in,
                     const void *W, const int32_t *offsets, const int32_t *rows, void *out,
                     void *ws, size_t ws_bytes, moe_stream_t stream, bool back)
{
    moe_status st = check_grouped(dtype, G, R, N, K);
    if (st != MOE_OK)
        return st;
    if (!W || !offsets || (R > 0 && (!in || !out)))
        return MOE_ERR_NULL;
    const uintptr_t al = dtype == MOE_DTYPE_BF16 ? 16 : 4;
    if (!aligned(in, al) || !aligned(W, al) || !aligned(out, al))
        return MOE_ERR_ALIGN;
    if ((st = check_grouped_ws(dtype, ws, ws_bytes)) != MOE_OK)
        return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const Table t{offsets, rows, (int)R};
    if (R == 0)
        return ws ? cuda_status(clear_word(ws, s)) : MOE_OK;
    if (dtype == MOE_DTYPE_BF16)
        return cuda_status(rows_tc(t, G, R, N, K, in, W, out, back, ws, s));
    Simt p = simt_rows(t, RAGGED_M, G, 0, N, K, static_cast<const float *>(in), 0,
                       static_cast<const float *>(W), back, static_cast<float *>(out), 0, nullptr);
    p.clear = static_cast<int32_t *>(ws);
    return cuda_status(launch_simt(p, s));
}

// Whether every X, X X^T and a I + b A + c A A of `steps` steps stays inside fp16 as
// they are stored (times 8192, 8192 and 2048), for singular values from 0 to 1 at
// the start: p(x) = x g(x^2), g(s) = a + b s + c s^2, at the ends of the interval and
// where p' or g' is zero.  *growth: the most that all steps together multiply a
// singular value by.
bool steps_in_range(double a, double b, double c, int steps, double *growth)
{
    double u = 1;
    *growth = 1;
    for (int i = 0; i < steps; ++i) {
        if (!(u <= 2.8))   // 8192 u^2 <= 64225
            return false;
        double top = 0, most = fabs(a);
        auto look = [&](double s) {
            if (!(s >= 0 && s <= u * u))
                return;
            const double g = fabs(a + s * (b + s * c));
            most = g > most ? g : most;
            top = sqrt(s) * g > top ? sqrt(s) * g : top;
        };
        look(u * u);
        look(-b / (2 * c));
        const double q = sqrt(9 * b * b - 20 * a * c);   // p' = a + 3 b s + 5 c s^2
        look((-3 * b + q) / (10 * c));
        look((-3 * b - q) / (10 * c));
        look(-a / (3 * b));                              // c = 0
        if (!(most <= 31))   // 2048 g <= 63488
            return false;
        *growth *= most;
        u = top;
    }
    return true;
}

// Scratch of the FFN backward: hidden activations and their gradients, and in
// fp32 also u, v and dh (in bf16 those never leave the accumulators).
struct FfnScratch {
    void *h, *du, *dv, *hs, *dus, *dvs;
    size_t bytes;
};

FfnScratch carve_ffn(const moe_config &c, void *ws)
{
    FfnScratch f;
    char *base = static_cast<char *>(ws);
    size_t off = kStatusBytes;
    auto take = [&](size_t bytes) {
        void *p = base ? base + off : nullptr;
        off = align_up(off + bytes, 256);
        return p;
    };
    const size_t e = dtype_bytes(c.dtype);
    if (c.dtype == MOE_DTYPE_BF16)
        off = kGroupedBytes;
    const size_t r = (size_t)perm_rows(c) * c.d_ff * e;
    const size_t q = c.n_shared > 0 ? (size_t)c.n_shared * c.T * c.d_ff_shared * e : 0;
    const bool swiglu = c.act == MOE_ACT_SWIGLU;
    f.h = take(r);
    f.du = take(r);
    f.dv = take(swiglu ? r : 0);
    f.hs = take(q);
    f.dus = take(q);
    f.dvs = take(swiglu ? q : 0);
    f.bytes = off;
    return f;
}

struct FfnArgs {
    const void *x_perm, *dY, *W1, *W3, *W2, *x, *dy, *Ws1, *Ws3, *Ws2;
    void *dx, *dW1, *dW3, *dW2, *dxs, *dWs1, *dWs3, *dWs2;
};

cudaError_t ffn_grad_tc(const moe_config &c, const Table &t, const FfnArgs &a, const FfnScratch &f,
                        bool f32, bool acc, void *status, cudaStream_t s)
{
    const int64_t R = t.n_rows;
    const int d = c.d, F = c.d_ff, E = c.E, S = c.n_shared, Fs = c.d_ff_shared, T = c.T;
    const bool swiglu = c.act == MOE_ACT_SWIGLU, shared = S > 0 && T > 0;
    const Tiles hid = row_tiles((int64_t)T * c.k, E, F, true);
    const Tiles tiles = row_tiles((int64_t)T * c.k, E, d, false);
    const Epi epi = swiglu ? EPI_SWIGLU : EPI_GELU;
    cudaError_t e;
    bool ok = true;

    // h, du, dv from x and dy
    Params p = tc_params(t, status, true);
    const int ubox = b_box(epi, hid), ask = stage_k(epi, hid);   // widths: multiples of 64
    auto act_set = [&](Set &v, int mode, int groups, int64_t rows, int cols, const void *in,
                       const void *dout, const void *w1, const void *w3, const void *w2, void *h,
                       void *du, void *dv) {
        v.mode = mode;
        v.groups = groups;
        v.M = mode == DENSE ? (int)rows : 0;
        v.N = cols;
        v.K = d;
        v.segs = v.period = 2;
        v.b_grouped = 1;
        v.ld = cols;
        v.out_group = rows * cols;
        v.out = h;
        v.out2 = du;
        v.out3 = dv;
        v.a_wide = v.b_wide = 1;
        ok &= map_k(&v.a[0], dout, rows, d, d, 1, 0, 128, ask, true);
        ok &= map_k(&v.a[1], in, rows, d, d, 1, 0, 128, ask, true);
        ok &= map_k(&v.b[0], w1, cols, d, d, groups, (int64_t)cols * d, ubox, ask, true);
        ok &= map_mn(&v.b[1], w2, d, cols, cols, groups, (int64_t)cols * d, ask, dh_box(hid),
                     true);
        if (swiglu)
            ok &= map_k(&v.b3, w3, cols, d, d, groups, (int64_t)cols * d, ubox, ask, true);
    };
    act_set(p.set[0], RAGGED_M, E, R, F, a.x_perm, a.dY, a.W1, a.W3, a.W2, f.h, f.du, f.dv);
    p.nsets = 1;
    if (shared) {
        act_set(p.set[1], DENSE, S, T, Fs, a.x, a.dy, a.Ws1, a.Ws3, a.Ws2, f.hs, f.dus, f.dvs);
        p.nsets = 2;
    }
    if (!ok)
        return cudaErrorInvalidValue;
    set_cut(p, status);   // not for these tiles, which are whole, but for the calls' below
    if ((e = clear_for_replay(p.counters, s)) != cudaSuccess)
        return e;
    if ((e = launch_tc(p, epi, A_K_B_K, hid, s)) != cudaSuccess)
        return e;

    // dx = du W1 (+ dv W3); shared: summed over the experts in the accumulator
    p = tc_params(t, status, false);
    auto dx_set = [&](Set &v, int mode, int groups, int64_t rows, int cols, const void *du,
                      const void *dv, const void *w1, const void *w3, void *out) {
        v.mode = mode;
        v.groups = mode == DENSE ? 1 : groups;
        v.M = mode == DENSE ? (int)rows : 0;
        v.N = d;
        v.K = cols;
        v.period = swiglu ? 2 : 1;
        v.segs = v.period * (mode == DENSE ? groups : 1);
        v.seg_grouped = mode == DENSE;
        v.a_grouped = mode == DENSE;
        v.b_grouped = 1;
        v.ld = d;
        v.out = out;
        const int ag = mode == DENSE ? groups : 1, sk = stage_k(EPI_ROWS, tiles);
        const int box = b_box(EPI_ROWS, tiles);
        v.a_wide = v.b_wide = 1;
        ok &= map_k(&v.a[0], du, rows, cols, cols, ag, rows * cols, 128, sk, true);
        ok &= map_mn(&v.b[0], w1, cols, d, d, groups, (int64_t)cols * d, sk, box, true);
        if (swiglu) {
            ok &= map_k(&v.a[1], dv, rows, cols, cols, ag, rows * cols, 128, sk, true);
            ok &= map_mn(&v.b[1], w3, cols, d, d, groups, (int64_t)cols * d, sk, box, true);
        }
    };
    dx_set(p.set[0], RAGGED_M, E, R, F, f.du, f.dv, a.W1, a.W3, a.dx);
    p.nsets = 1;
    if (shared) {
        dx_set(p.set[1], DENSE, S, T, Fs, f.dus, f.dvs, a.Ws1, a.Ws3, a.dxs);
        p.nsets = 2;
    }
    if (!ok)
        return cudaErrorInvalidValue;
    set_cut(p, status);
    if ((e = launch_tc(p, EPI_ROWS, A_K_B_MN, tiles, s)) != cudaSuccess)
        return e;

    // weight gradients
    p = tc_params(t, status, false);
    int n = 0;
    const Tiles wt = dw_tiles(F, d);
    auto add = [&](void *out) { return acc ? out : nullptr; };
    ok &= dw_set(p.set[n++], RAGGED_K, E, R, F, d, f.du, false, a.x_perm, false, add(a.dW1), a.dW1,
                 f32, wt);
    if (swiglu)
        ok &= dw_set(p.set[n++], RAGGED_K, E, R, F, d, f.dv, false, a.x_perm, false, add(a.dW3),
                     a.dW3, f32, wt);
    ok &= dw_set(p.set[n++], RAGGED_K, E, R, d, F, a.dY, false, f.h, false, add(a.dW2), a.dW2, f32, wt);
    if (S > 0) {
        ok &= dw_set(p.set[n++], DENSE, S, T, Fs, d, f.dus, true, a.x, false, add(a.dWs1), a.dWs1,
                     f32, wt);
        if (swiglu)
            ok &= dw_set(p.set[n++], DENSE, S, T, Fs, d, f.dvs, true, a.x, false, add(a.dWs3),
                         a.dWs3, f32, wt);
        ok &= dw_set(p.set[n++], DENSE, S, T, d, Fs, a.dy, false, f.hs, true, add(a.dWs2), a.dWs2,
                     f32, wt);
    }
    p.nsets = n;
    if (!ok)
        return cudaErrorInvalidValue;
    set_cut(p, status);
    return launch_tc(p, EPI_DW, A_MN_B_MN, wt, s);
}

// fp32: the same gradients one product at a time; h holds u until the
// activation gradient, du holds dh, dv holds v.
cudaError_t ffn_grad_simt(const moe_config &c, const Table &t, const FfnArgs &a,
                          const FfnScratch &f, bool acc, void *status, cudaStream_t s)
{
    const bool swiglu = c.act == MOE_ACT_SWIGLU;
    const int d = c.d;
    cudaError_t e = cudaSuccess;
    auto run = [&](Simt p) {
        p.clear = static_cast<int32_t *>(status);   // the first launch clears it
        status = nullptr;
        if (e == cudaSuccess)
            e = launch_simt(p, s);
    };
    auto F32 = [](const void *p) { return static_cast<const float *>(p); };
    auto M32 = [](void *p) { return static_cast<float *>(p); };
    auto half = [&](int mode, int G, int64_t rows, int F, const void *in, const void *dout,
                    const void *W1, const void *W3, const void *W2, void *h, void *du, void *dv,
                    void *dx, void *dW1, void *dW3, void *dW2) {
        const bool dense = mode == DENSE;
        const int M = dense ? (int)rows : 0;
        const int64_t og = dense ? rows * F : 0;   // hidden buffers: one slab per shared expert
        run(simt_rows(t, mode, G, M, F, d, F32(in), 0, F32(W1), false, M32(h), og, nullptr));
        if (swiglu)
            run(simt_rows(t, mode, G, M, F, d, F32(in), 0, F32(W3), false, M32(dv), og, nullptr));
        // dh = dy W2: W2 [d, F] with its rows as the contraction
        run(simt_rows(t, mode, G, M, d, F, F32(dout), 0, F32(W2), true, M32(du), og, nullptr));
        if (e == cudaSuccess)
            e = launch_act_grad(c.act, (dense ? G : 1) * rows * F, F32(h), F32(dv), F32(du), M32(h),
                                M32(du), M32(dv), s);
        // shared experts add up in dx one after the other
        for (int g = 0; g < (dense ? G : 1); ++g) {
            const int64_t w = (int64_t)g * F * d;
            const int gs = dense ? 1 : G;
            run(simt_rows(t, mode, gs, M, F, d, F32(du) + g * og, 0, F32(W1) + w, true, M32(dx), 0,
                          g ? F32(dx) : nullptr));
            if (swiglu)
                run(simt_rows(t, mode, gs, M, F, d, F32(dv) + g * og, 0, F32(W3) + w, true,
                              M32(dx), 0, F32(dx)));
        }
        const int wm = dense ? DENSE : RAGGED_K;
        run(simt_dw(t, wm, G, (int)rows, F, d, F32(du), og, F32(in), 0, acc ? F32(dW1) : nullptr,
                    M32(dW1)));
        if (swiglu)
            run(simt_dw(t, wm, G, (int)rows, F, d, F32(dv), og, F32(in), 0,
                        acc ? F32(dW3) : nullptr, M32(dW3)));
        run(simt_dw(t, wm, G, (int)rows, d, F, F32(dout), 0, F32(h), og, acc ? F32(dW2) : nullptr,
                    M32(dW2)));
    };
    half(RAGGED_M, c.E, t.n_rows, c.d_ff, a.x_perm, a.dY, a.W1, a.W3, a.W2, f.h, f.du, f.dv, a.dx,
         a.dW1, a.dW3, a.dW2);
    if (c.n_shared > 0)
        half(DENSE, c.n_shared, c.T, c.d_ff_shared, a.x, a.dy, a.Ws1, a.Ws3, a.Ws2, f.hs, f.dus,
             f.dvs, a.dxs, a.dWs1, a.dWs3, a.dWs2);
    return e;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_grouped_workspace_size(int32_t dtype, int32_t G, int64_t R, int32_t N, int32_t K)
{
    return check_grouped(dtype, G, R, N, K) == MOE_OK ? grouped_bytes(dtype) : 0;
}

moe_status moe_grouped_matmul(int32_t dtype, int32_t G, int64_t R, int32_t N, int32_t K,
                              const void *x, const void *W, const int32_t *offsets,
                              const int32_t *rows, void *y, void *ws, size_t ws_bytes,
                              moe_stream_t stream)
{
    return rows_call(dtype, G, R, N, K, x, W, offsets, rows, y, ws, ws_bytes, stream, false);
}

moe_status moe_grouped_matmul_dx(int32_t dtype, int32_t G, int64_t R, int32_t N, int32_t K,
                                 const void *dy, const void *W, const int32_t *offsets,
                                 const int32_t *rows, void *dx, void *ws, size_t ws_bytes,
                                 moe_stream_t stream)
{
    return rows_call(dtype, G, R, N, K, dy, W, offsets, rows, dx, ws, ws_bytes, stream, true);
}

moe_status moe_grouped_matmul_dw(int32_t dtype, int32_t G, int64_t R, int32_t N, int32_t K,
                                 const void *dy, const void *x, const int32_t *offsets,
                                 const int32_t *rows, int32_t dw_dtype, const void *add, void *dW,
                                 void *ws, size_t ws_bytes, moe_stream_t stream)
{
    moe_status st = check_grouped(dtype, G, R, N, K);
    if (st != MOE_OK)
        return st;
    if ((dw_dtype != MOE_DTYPE_F32 && dw_dtype != MOE_DTYPE_BF16) ||
        (dtype == MOE_DTYPE_F32 && dw_dtype != MOE_DTYPE_F32))
        return MOE_ERR_DTYPE;
    if (!dW || !offsets || (R > 0 && (!dy || !x)))
        return MOE_ERR_NULL;
    const uintptr_t al = dtype == MOE_DTYPE_BF16 ? 16 : 4;
    if (!aligned(dy, al) || !aligned(x, al) || !aligned(dW, al) || !aligned(add, al))
        return MOE_ERR_ALIGN;
    if ((st = check_grouped_ws(dtype, ws, ws_bytes)) != MOE_OK)
        return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const Table t{offsets, rows, (int)R};
    if (dtype == MOE_DTYPE_F32) {
        Simt p = simt_dw(t, RAGGED_K, G, 0, N, K, static_cast<const float *>(dy), 0,
                         static_cast<const float *>(x), 0, static_cast<const float *>(add),
                         static_cast<float *>(dW));
        p.clear = static_cast<int32_t *>(ws);
        return cuda_status(launch_simt(p, s));
    }
    Params p = tc_params(t, ws, true);
    const Tiles tiles = dw_tiles(N, K);
    p.nsets = 1;
    if (!dw_set(p.set[0], RAGGED_K, G, R, N, K, dy, false, x, false, add, dW,
                dw_dtype == MOE_DTYPE_F32, tiles))
        return MOE_ERR_CUDA;
    set_cut(p, ws);
    if (may_cut(R)) {
        const cudaError_t e = clear_for_replay(p.counters, s);
        if (e != cudaSuccess)
            return MOE_ERR_CUDA;
    }
    return cuda_status(launch_tc(p, EPI_DW, A_MN_B_MN, tiles, s));
}

moe_status moe_combine_backward(const moe_config *cfg, const void *dy, const void *Y_perm,
                                const float *gates, const int32_t *topk_idx, const int32_t *pos,
                                const uint8_t *keep, const int32_t *offsets, void *dY_perm,
                                float *dgates, moe_stream_t stream)
{
    moe_status st = moe_validate(cfg);
    if (st != MOE_OK)
        return st;
    if (cfg->T == 0)
        return MOE_OK;
    if (!dy || !Y_perm || !gates || !topk_idx || !pos || !keep || !offsets || !dY_perm || !dgates)
        return MOE_ERR_NULL;
    if (!aligned(dy, 16) || !aligned(Y_perm, 16) || !aligned(dY_perm, 16))
        return MOE_ERR_ALIGN;
    return cuda_status(launch_combine_grad(*cfg, dy, Y_perm, gates, topk_idx, pos, keep, offsets,
                                           dY_perm, dgates,
                                           reinterpret_cast<cudaStream_t>(stream)));
}

size_t moe_ffn_backward_workspace_size(const moe_config *cfg)
{
    return moe_validate(cfg) == MOE_OK ? carve_ffn(*cfg, nullptr).bytes : 0;
}

moe_status moe_expert_ffn_backward(const moe_config *cfg, const void *x_perm,
                                   const int32_t *offsets, const int32_t *kept,
                                   const void *dY_perm, const void *W1, const void *W3,
                                   const void *W2, const void *x, const void *dY_shared,
                                   const void *Ws1, const void *Ws3, const void *Ws2,
                                   void *dx_perm, void *dW1, void *dW3, void *dW2,
                                   void *dx_shared, void *dWs1, void *dWs3, void *dWs2,
                                   int32_t dw_dtype, int32_t accumulate, void *ws,
                                   size_t ws_bytes, moe_stream_t stream)
{
    moe_status st = moe_validate(cfg);
    if (st != MOE_OK)
        return st;
    const moe_config &c = *cfg;
    const bool swiglu = c.act == MOE_ACT_SWIGLU, shared = c.n_shared > 0;
    if ((dw_dtype != MOE_DTYPE_F32 && dw_dtype != MOE_DTYPE_BF16) ||
        (c.dtype == MOE_DTYPE_F32 && dw_dtype != MOE_DTYPE_F32))
        return MOE_ERR_DTYPE;
    if (c.n_shared > kMaxShared)
        return MOE_ERR_SHAPE;
    if (!x_perm || !offsets || !kept || !dY_perm || !W1 || !W2 || !dx_perm || !dW1 || !dW2 ||
        (swiglu && (!W3 || !dW3)))
        return MOE_ERR_NULL;
    if (shared && (!Ws1 || !Ws2 || !dWs1 || !dWs2 || (swiglu && (!Ws3 || !dWs3)) ||
                   (c.T > 0 && (!x || !dY_shared || !dx_shared))))
        return MOE_ERR_NULL;
    const FfnArgs a{x_perm, dY_perm, W1, W3, W2, x, dY_shared, Ws1, Ws3, Ws2,
                    dx_perm, dW1, dW3, dW2, dx_shared, dWs1, dWs3, dWs2};
    const void *ptrs[] = {a.x_perm, a.dY, a.W1, a.W3, a.W2, a.x, a.dy, a.Ws1, a.Ws3, a.Ws2,
                          a.dx, a.dW1, a.dW3, a.dW2, a.dxs, a.dWs1, a.dWs3, a.dWs2};
    for (const void *p : ptrs)
        if (!aligned(p, 16))
            return MOE_ERR_ALIGN;
    const FfnScratch f = carve_ffn(c, ws);
    if ((st = check_ws(ws, ws_bytes, f.bytes)) != MOE_OK)
        return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const Table t{offsets, kept, (int)perm_rows(c)};
    if (c.dtype == MOE_DTYPE_BF16)
        return cuda_status(ffn_grad_tc(c, t, a, f, dw_dtype == MOE_DTYPE_F32, accumulate != 0, ws,
                                       s));
    return cuda_status(ffn_grad_simt(c, t, a, f, accumulate != 0, ws, s));
}

moe_status moe_training_status(int32_t *status, moe_stream_t stream)
{
    if (!status)
        return MOE_ERR_NULL;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    int32_t *word[2], seen[2] = {0, 0};
    if (gave_up_grouped(&word[0]) != cudaSuccess || gave_up_small(&word[1]) != cudaSuccess)
        return MOE_ERR_CUDA;
    for (int i = 0; i < 2; ++i)
        if (cudaMemcpyAsync(&seen[i], word[i], 4, cudaMemcpyDeviceToHost, s) != cudaSuccess)
            return MOE_ERR_CUDA;
    if (cudaStreamSynchronize(s) != cudaSuccess)
        return MOE_ERR_CUDA;
    *status = seen[0] ? seen[0] : seen[1];
    return MOE_OK;
}

moe_status moe_clear_training_status(moe_stream_t stream)
{
    int32_t *word[2];
    if (gave_up_grouped(&word[0]) != cudaSuccess || gave_up_small(&word[1]) != cudaSuccess)
        return MOE_ERR_CUDA;
    for (int i = 0; i < 2; ++i)
        if (clear_word(word[i], reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
            return MOE_ERR_CUDA;
    return MOE_OK;
}

moe_status moe_probe_training_timeout(uint64_t timeout_ns, moe_stream_t stream)
{
    if (timeout_ns > 2000000000ull)
        return MOE_ERR_SHAPE;
    return cuda_status(launch_grouped_probe(timeout_ns, reinterpret_cast<cudaStream_t>(stream)));
}

size_t moe_orthogonalize_workspace_size(int32_t E, int32_t m, int32_t n, int32_t steps)
{
    if (E < 1 || E > kEntries || m < 1 || n < 1 || m > 1 << 20 || n > 1 << 20 || steps < 1 || steps > 32)
        return 0;
    return orthogonalize_bytes(E, m, n, steps);
}

moe_status moe_orthogonalize(int32_t dtype, int32_t E, int32_t m, int32_t n, const void *G,
                             int32_t steps, const float *coeffs, float eps, float scale, void *U,
                             void *ws, size_t ws_bytes, moe_stream_t stream)
{
    if (dtype != MOE_DTYPE_F32 && dtype != MOE_DTYPE_BF16)
        return MOE_ERR_DTYPE;
    const size_t need = moe_orthogonalize_workspace_size(E, m, n, steps);
    if (need == 0)
        return MOE_ERR_SHAPE;
    if (!G || !U || !coeffs)
        return MOE_ERR_NULL;
    for (int i = 0; i < 3; ++i)
        if (!isfinite(coeffs[i]))
            return MOE_ERR_SHAPE;
    if (!(eps >= 0.f) || !isfinite(eps) || !isfinite(scale))
        return MOE_ERR_SHAPE;
    if (!aligned(G, dtype == MOE_DTYPE_BF16 ? 2 : 4) || !aligned(U, 2))
        return MOE_ERR_ALIGN;
    const moe_status st = check_ws(ws, ws_bytes, need);
    if (st != MOE_OK)
        return st;
    double growth;
    if (!steps_in_range(coeffs[0], coeffs[1], coeffs[2], steps, &growth))
        return MOE_ERR_SHAPE;
    return cuda_status(launch_orthogonalize(dtype == MOE_DTYPE_BF16, E, m, n, G, steps, coeffs[0],
                                            coeffs[1], coeffs[2], growth, eps, scale, U, ws,
                                            reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
