// Grouped matrix products on the 5th-generation tensor cores, for operands of
// either storage order: y = x W^T, dx = dy W, dW = dy^T x over the ragged
// expert segments, the hidden gradients of the expert FFNs, and the stacked
// products of the Newton-Schulz steps.
//
// One persistent, warp-specialised kernel (TMA -> shared memory ->
// tcgen05.mma -> TMEM -> registers -> global).  PAIR tiles take a 2-CTA
// cluster: 256 output rows (128 a CTA) x BN columns, each CTA loading its rows
// of A and half the rows of B.  A stage is 128 of K, one TMA instruction for each
// operand where the contiguous extent is a multiple of 64 (the tensor is then
// described as blocks of 64 columns and the box takes two), two otherwise: their
// number bounds the loads.  Operands whose contraction index is the row
// index of the stored matrix (W in dx, both in dW) are read as they lie: boxes
// of 64 contiguous elements x a stage's contraction rows, and the MMA takes
// them as MN-major, so nothing is transposed in memory.
//
// Ragged contractions (dW): a group's rows end anywhere, and what follows
// belongs to the next group or to nobody (it may hold NaN, so it cannot be
// multiplied by zeros).  The MMA stops at the 16-row step holding the last
// row; a warp of its own waits for that stage's copies and clears the up to 15
// rows behind it in shared memory before handing the stage over, while the
// loads go on to the next tile (5.3 us a tile of two rows when the loading warp
// did it in turn).
//
// The tensor cores truncate when they add to an fp32 accumulator, a bias of
// about 2e-8 of the sum for every 16 rows (measured: 1.6e-6 after 1536 rows,
// where fp32 rounding alone leaves 3e-7), so a weight gradient over many rows
// is summed in accumulators of 512 rows each, which the epilogue adds up in
// registers (round to nearest) while the next one fills: 128 values a thread.
// Products and input gradients, which end in bf16, take accumulators of 8192 past
// that (1e-5; a single one left 2e-5 at 14336 and 1e-3 at 2^20), in kernels of their
// own: with the sums' code and registers contractions of 256 to 8192 took 2 to 5%
// longer.  u, v and dh (over the layer's width) and the stacks keep a single one.
//
// Work is dealt as tiles, one to each CTA (pair) in turn.  Where the last round
// would leave most of them idle (or, with few rows, every round), the tiles of
// the last rounds are cut along the contraction: each part leaves its fp32
// accumulators in the workspace, and the warp that finishes a tile's part last
// adds the parts up in their order and stores the rows, so the result does not
// depend on who was last.  split_plan() weighs the rounds saved against that.
//
// Output rows go from registers to memory, each masked by the group's end: rows
// behind it are neither written nor read.  (Out by TMA through the 2 KB a warp
// that the ring leaves, weight gradients took 1.2 times as long: a warp waits for
// its piece to be read before the next.)
//
// Roles: warp 0 loads, warp 1 issues the MMAs (and owns TMEM), the last eight
// are the epilogue (warp w reads TMEM lanes 32 (w mod 4) .. +31, the first four
// of them the first half of the columns).  Every wait is bounded; on expiry the CTA sets
// MOE_ERR_DEVICE_TIMEOUT, every role leaves its loop, copies in flight are
// awaited (bounded too), TMEM is freed and the kernel returns.
#include "grouped.cuh"

#include <cuda_fp16.h>
#include <stddef.h>
#include <string.h>
#include <time.h>

#include <atomic>

namespace moe {
namespace grp {

using namespace tc;

namespace {

__device__ int32_t g_gave_up;   // MOE_ERR_DEVICE_TIMEOUT after any call here gave up

constexpr int EPI_WARPS = 8;
constexpr uint32_t TMEM_COLS = 512;
constexpr int STG_WARP = 32 * 64;        // staging tile of an epilogue warp: 32 rows of 64 bytes
constexpr int RING_BYTES = 192 * 1024;
constexpr int kLongRows = 8192;          // EPI_ROWS_LONG: contraction in one accumulator

// AR: rows of A a CTA takes, 128, or 32 for groups of few rows: the MMA's other
// rows read on into the next bytes of the ring, their results are never stored,
// and the ring holds 5 x 32 KB of weights instead of 3 x 32.
template <int CTAS, int BN, int EPI, int AR>
struct Shape {
    static constexpr bool ACT = EPI == EPI_GELU || EPI == EPI_SWIGLU;
    static constexpr bool ROWS = EPI == EPI_ROWS || EPI == EPI_ROWS_LONG;
    static constexpr int BM = AR * CTAS;
    static constexpr int A_BYTES = AR * 128;             // AR rows x 64 elements
    static constexpr int FIRST_EPI = EPI == EPI_DW ? 3 : 2;   // first of the epilogue warps
    static constexpr int THREADS = 32 * (FIRST_EPI + EPI_WARPS);
    static constexpr int MMA_M = 128 * CTAS;
    // epilogue warps of a CTA that have rows, and floats of a cut tile's part
    static constexpr int ROW_WARPS = 2 * (AR / 32);
    static constexpr int PART = BM * BN;
    // accumulator columns of the widest B tile (ACT: u, with v beside it)
    static constexpr int BNB = EPI == EPI_SWIGLU ? 2 * BN : BN;
    static constexpr int B_ROWS = BNB / CTAS;            // B rows of one CTA
    static constexpr int B_BYTES = B_ROWS * 128;         // of 64 contraction elements
    static constexpr int SUB = A_BYTES + B_BYTES;
    // 128 of K a stage where three stages fit: half the barrier round trips
    static constexpr int KSUB = 6 * SUB <= RING_BYTES ? 2 : 1;
    static constexpr int STAGES = AR < 128 ? 5 : RING_BYTES / (KSUB * SUB);
    static constexpr int BK = 64 * KSUB;
    static constexpr int MN_BLOCK = BK * 128;            // 64 columns of an MN-major stage
    static constexpr int OFF_B = STAGES * KSUB * A_BYTES;
    static constexpr bool STAGED = EPI == EPI_NS;   // rows of odd pitch go through shared memory
    static constexpr int OFF_STG = OFF_B + STAGES * KSUB * B_BYTES;
    static constexpr int OFF_BAR = OFF_STG + (STAGED ? EPI_WARPS * STG_WARP : 0);
    static constexpr int OFF_TAB = OFF_BAR + 256;
    static constexpr int SMEM = OFF_TAB + 8 * kMaxE + 4 * (kEntries + 4) + 1024;   // + alignment slack
    // contraction summed in one accumulator before the epilogue adds it, in
    // registers, to the tile's running sum (0: all of it)
    static constexpr int CHUNK = EPI == EPI_DW ? 512 : EPI == EPI_ROWS_LONG ? kLongRows : 0;
    static constexpr int CHUNK_BLOCKS = CHUNK > 0 ? CHUNK / BK : 1;
    // TMEM columns.  Plain: two accumulators of BN.  GELU: u and dh, twice.
    // SwiGLU: u | v once (256 columns), dh twice behind it.
    static constexpr int DH_COL = EPI == EPI_SWIGLU ? 2 * BN : BN;
};

struct Tile {
    int set, g;
    int m0, n0;        // first output row (in the group) and column
    int mg;            // output rows of the group
    int row0;          // first row of the group in the tall buffers (RAGGED_M)
    int k0, klen;      // contraction: first index and length
    int kbs;           // its blocks of BK, for one segment
    int b0, b1;        // the blocks of this part, over all segments
    int part, parts;   // which of how many parts of a tile
    int cut;           // number among the cut tiles
};

// The first `whole` tiles are items by themselves; every later one is `parts`
// items, one for each part of its contraction.
struct Plan {
    int whole, parts, items;
};

// Tiles of entry (set, g).
template <int BM, int BN>
__device__ __forceinline__ int entry_tiles(const Set &s, const int2 *span, int g)
{
    const int m = s.mode == RAGGED_M ? span[g].y : s.M;
    const int mt = (m + BM - 1) / BM, nt = (s.N + BN - 1) / BN;
    if (!s.sym)
        return mt * nt;
    int n = 0;
    for (int i = 0; i < mt; ++i)
        n += min(nt, (i + 1) * (BM / BN));
    return n;
}

// A plan for `tiles` tiles of `kb` contraction blocks each on `units` CTAs or
// pairs, `most` cut items at most.  Costs in blocks (0.8 us): an item's epilogue
// 2; a cut tile 3 to leave and 3.5 a part to add up.  Lane i of a warp tries i parts
// for the tiles of the last round, or of the last two, or for all.
template <int CTAS>
__device__ __forceinline__ Plan split_plan(int tiles, int kb, int units, int most, int lane)
{
    const int rounds = tiles / units;
    const int parts = 1 + (lane & 15);
    float best = 1e30f;
    int whole = tiles;
    if (lane == 0) {
        best = (float)((tiles + units - 1) / units) * (kb + 2);
    } else if (parts > 1 && 2 * parts <= kb) {
        // lanes 1..15: tiles past the last full round; 17..31: one round more
        const int full = lane < 16 ? rounds : rounds - 1;
        const int cut = tiles - full * units;
        if (full >= 0 && cut > 0 && (int64_t)cut * parts <= most) {
            best = (float)full * (kb + 2) +
                   (float)((cut * parts + units - 1) / units) * ((kb + parts - 1) / parts + 2) + 3 +
                   3.5f * parts;
            whole = full * units;
        }
    }
    float low = best;
#pragma unroll
    for (int s = 16; s; s >>= 1)
        low = fminf(low, __shfl_xor_sync(0xffffffffu, low, s));
    const int from = __ffs(__ballot_sync(0xffffffffu, best == low)) - 1;
    Plan pl;
    pl.whole = __shfl_sync(0xffffffffu, whole, from);
    pl.parts = __shfl_sync(0xffffffffu, parts, from);
    pl.items = pl.whole + (tiles - pl.whole) * pl.parts;
    return pl;
}

// i / d for 0 <= i < 2^24, d > 0
__device__ __forceinline__ int div_small(int i, int d)
{
    int q = (int)__fdividef((float)i, (float)d);
    const int r = i - q * d;
    return r < 0 ? q - 1 : (r >= d ? q + 1 : q);
}

template <int BM, int BN, int BK, int SETS>
__device__ __forceinline__ Tile decode(const ParamsOf<SETS> &p, const int *tstart, const int2 *span,
                                       const Plan &pl, int item)
{
    Tile t;
    int tile = item;
    t.part = 0;
    t.parts = 1;
    t.cut = 0;
    if (item >= pl.whole) {
        t.cut = div_small(item - pl.whole, pl.parts);
        t.part = item - pl.whole - t.cut * pl.parts;
        t.parts = pl.parts;
        tile = pl.whole + t.cut;
    }
    int lo = 0, hi = p.entries;   // last entry with tstart <= tile
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (tstart[mid] <= tile)
            lo = mid;
        else
            hi = mid;
    }
    int set = 0;
    while (set + 1 < p.nsets && p.set[set + 1].ent0 <= lo)
        ++set;
    const Set &s = p.set[set];
    t.set = set;
    t.g = lo - s.ent0;
    t.mg = s.M;
    t.row0 = 0;
    t.k0 = 0;
    t.klen = s.K;
    if (s.mode == RAGGED_M)
        t.row0 = span[t.g].x, t.mg = span[t.g].y;
    else if (s.mode == RAGGED_K)
        t.k0 = span[t.g].x, t.klen = span[t.g].y;
    t.kbs = (t.klen + BK - 1) / BK;
    const int blocks = t.kbs * s.segs;
    t.b0 = 0;
    t.b1 = blocks;
    if (t.parts > 1) {
        t.b0 = (int)((int64_t)blocks * t.part / t.parts);
        t.b1 = (int)((int64_t)blocks * (t.part + 1) / t.parts);
    }
    int i = tile - tstart[lo];
    const int nt = (s.N + BN - 1) / BN;
    if (s.sym) {
        int r = 0;
        for (;; ++r) {
            const int c = min(nt, (r + 1) * (BM / BN));
            if (i < c)
                break;
            i -= c;
        }
        t.m0 = r * BM;
        t.n0 = i * BN;
    } else {
        const int mt = (t.mg + BM - 1) / BM;
        const int n = i < 1 << 24 ? div_small(i, mt) : i / mt;
        t.m0 = (i - n * mt) * BM;
        t.n0 = n * BN;
    }
    return t;
}

// Whether a contraction's last block of `rem` rows ends inside a 16-row step,
// so that rows behind it have to be cleared.
template <int BK>
__device__ __forceinline__ bool ragged_tail(int rem)
{
    return rem < BK && (rem & 15);
}

template <int CTAS>
__device__ __forceinline__ void commit_all(uint32_t bar)
{
    if (CTAS == 2)
        mma_commit_pair(bar);
    else
        mma_commit(bar);
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap *m)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
}

// PAIR: the barrier may be the other CTA's
template <bool PAIR>
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap *m, uint32_t bar, int c0,
                                         int c1, int c2, int c3)
{
    if (PAIR)
        asm volatile(
            "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
            : "memory");
}

// Arrive on the leader's barrier with `bytes` to come by TMA.  Nothing this
// thread wrote has to be seen by the waiter, so the arrival is relaxed (with a
// release at cluster scope for every stage 16384 rows through 8 x 4096 x 14336
// took 1820 us instead of 1390).
template <int CTAS>
__device__ __forceinline__ void arrive_bytes(uint32_t bar, uint32_t bytes)
{
    if (CTAS == 2)
        asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::
                         "r"(bar),
                     "r"(bytes)
                     : "memory");
    else
        mbar_expect_tx(bar, bytes);
}

// Arrive on the leader's barrier after this warp's own writes to the stage.
template <int CTAS>
__device__ __forceinline__ void arrive_written(uint32_t bar)
{
    if (CTAS == 2)
        asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
                     : "memory");
    else
        mbar_arrive(bar);
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b)
{
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t *>(&h);
}

// Every lane stores its own row, 32 bytes at a time where the rows start on
// 32-byte boundaries (whole sectors), else 16.
__device__ __forceinline__ void st32(void *p, const uint32_t *w)
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}
__device__ __forceinline__ void st16(void *p, const uint32_t *w)
{
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void ld32(const void *p, uint32_t *w)
{
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]),
                   "=r"(w[6]), "=r"(w[7])
                 : "l"(p)
                 : "memory");
}

// n 32-byte pieces of a row, those that begin before byte `end`
template <int N>
__device__ __forceinline__ void load_row(const uint8_t *p, int end, int bytes, uint32_t *w)
{
#pragma unroll
    for (int c = 0; c < N; ++c) {
        if (bytes == 32) {
            if (32 * c < end)
                ld32(p + 32 * c, w + 8 * c);
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (32 * c + 16 * h < end) {
                    const uint4 u = *reinterpret_cast<const uint4 *>(p + 32 * c + 16 * h);
                    w[8 * c + 4 * h] = u.x, w[8 * c + 4 * h + 1] = u.y;
                    w[8 * c + 4 * h + 2] = u.z, w[8 * c + 4 * h + 3] = u.w;
                }
        }
    }
}
// n 32-byte pieces of a row, those that begin before byte `end`
template <int N>
__device__ __forceinline__ void store_row(uint8_t *p, int end, int bytes, const uint32_t *w)
{
#pragma unroll
    for (int c = 0; c < N; ++c) {
        if (bytes == 32) {
            if (32 * c < end)
                st32(p + 32 * c, w + 8 * c);
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (32 * c + 16 * h < end)
                    st16(p + 32 * c + 16 * h, w + 8 * c + 4 * h);
        }
    }
}

// 4 x 4 transpose of blocks of W words over four neighbouring lanes: lane q of
// them holds row q's blocks 0..3 before, block q of rows 0..3 after.
template <int W>
__device__ __forceinline__ void transpose_blocks(uint32_t (&w)[4][W], int lane)
{
    const bool b0 = lane & 1, b1 = lane & 2;
#pragma unroll
    for (int j = 0; j < W; ++j) {
#pragma unroll
        for (int k = 0; k < 4; k += 2) {   // blocks k, k + 1 with the odd/even neighbour
            const uint32_t o = __shfl_xor_sync(0xffffffffu, b0 ? w[k][j] : w[k + 1][j], 1);
            if (b0)
                w[k][j] = o;
            else
                w[k + 1][j] = o;
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {      // blocks k, k + 2 with the neighbour two lanes on
            const uint32_t o = __shfl_xor_sync(0xffffffffu, b1 ? w[k][j] : w[k + 2][j], 2);
            if (b1)
                w[k][j] = o;
            else
                w[k + 2][j] = o;
        }
    }
}

// 32 columns of packed 16-bit values of this lane's row: four lanes trade 16-byte
// blocks, so that a row's 64 bytes leave in one instruction.  out: row 0 of the
// warp, first column; rv rows and cv columns (a multiple of 8) are stored.
__device__ __forceinline__ void store_traded(const uint32_t *v, uint16_t *out, int64_t ld, int lane,
                                             int rv, int cv)
{
    uint32_t w[4][4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            w[k][j] = v[4 * k + j];
    transpose_blocks(w, lane);
    const int r0 = lane & ~3, c = 8 * (lane & 3);
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (r0 + k < rv && c < cv)
            st16(out + (r0 + k) * ld + c, w[k]);
}

// This lane's row of N sums (plus the addend) to fp32 or bf16.  at: element
// (row 0 of the warp, first column); rv rows and cols columns are stored.
// Without an addend four lanes trade blocks first, so that a row's 128 bytes
// leave in one instruction: lanes storing 32 bytes of a row each cost the load
// and store unit 32 lines an instruction (313 us instead of 393, two rows an expert
// into 8 x 4096 x 14336).  With an addend each lane keeps its row: the trades and
// the addend together do not fit the registers (196 us instead of 157, 64 groups
// of 1536 rows added in fp32).
template <int N>
__device__ __forceinline__ void store_sums(const Set &s, const float (&sum)[N], int64_t at, int lane,
                                           int rv, int cols, int bytes)
{
    if (s.add) {
        if (lane >= rv)
            return;
        const int esz = s.out_f32 ? 4 : 2;
        const int64_t o = (at + (int64_t)lane * s.ld) * esz;
        uint8_t *out = static_cast<uint8_t *>(s.out) + o;
        const uint8_t *add = static_cast<const uint8_t *>(s.add) + o;
#pragma unroll
        for (int i = 0; i < N / 16; ++i) {   // 16 columns at a time
            const float *v = sum + 16 * i;
            const int end = (cols - 16 * i) * esz;
            uint32_t w[16];
            if (s.out_f32) {
                load_row<2>(add + 64 * i, end, bytes, w);
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    w[j] = __float_as_uint(v[j] + __uint_as_float(w[j]));
                store_row<2>(out + 64 * i, end, bytes, w);
            } else {
                load_row<1>(add + 32 * i, end, bytes, w);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    w[j] = pack_bf16(v[2 * j] + __uint_as_float(w[j] << 16),
                                     v[2 * j + 1] + __uint_as_float(w[j] & 0xffff0000u));
                store_row<1>(out + 32 * i, end, bytes, w);
            }
        }
        return;
    }
    const int q = lane & 3, r0 = lane & ~3;
    if (!s.out_f32) {
        uint16_t *out = static_cast<uint16_t *>(s.out) + at;
#pragma unroll
        for (int i = 0; i < N / 64; ++i) {
            if (64 * i >= cols)
                break;
            uint32_t w[4][8];
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    w[k][j] = pack_bf16(sum[64 * i + 16 * k + 2 * j], sum[64 * i + 16 * k + 2 * j + 1]);
            transpose_blocks(w, lane);
            const int c = 64 * i + 16 * q;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint16_t *p = out + (int64_t)(r0 + k) * s.ld + c;
                if (r0 + k >= rv)
                    continue;
                if (bytes == 32) {
                    if (c < cols)
                        st32(p, w[k]);
                } else {
                    if (c < cols)
                        st16(p, w[k]);
                    if (c + 8 < cols)
                        st16(p + 8, w[k] + 4);
                }
            }
        }
        return;
    }
    float *out = static_cast<float *>(s.out) + at;
#pragma unroll
    for (int i = 0; i < N / 32; ++i) {
        if (32 * i >= cols)
            break;
        uint32_t w[4][8];
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                w[k][j] = __float_as_uint(sum[32 * i + 8 * k + j]);
        transpose_blocks(w, lane);
        const int c = 32 * i + 8 * q;
        if (c >= cols)
            continue;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float *p = out + (int64_t)(r0 + k) * s.ld + c;
            if (r0 + k >= rv)
                continue;
            if (bytes == 32) {
                st32(p, w[k]);
            } else {
                st16(p, w[k]);
                st16(p + 4, w[k] + 4);
            }
        }
    }
}

// The same to rows of any alignment, through a tile in shared memory: a warp
// writes one row's 32 values at a time.  out: column 0 of row 0; rv rows and cv columns are stored.
__device__ __forceinline__ void store_odd(uint8_t *stg, int lane, const uint32_t *w, uint16_t *out,
                                          int64_t ld, int rv, int cv)
{
    __syncwarp();
#pragma unroll
    for (int ch = 0; ch < 4; ++ch)
        *reinterpret_cast<uint4 *>(stg + lane * 64 + ((ch ^ ((lane >> 1) & 3)) << 4)) =
            make_uint4(w[4 * ch], w[4 * ch + 1], w[4 * ch + 2], w[4 * ch + 3]);
    __syncwarp();
#pragma unroll 8
    for (int r = 0; r < 32; ++r)
        if (r < rv && lane < cv)
            out[r * ld + lane] = *reinterpret_cast<const uint16_t *>(
                stg + r * 64 + (((lane >> 3) ^ ((r >> 1) & 3)) << 4) + (lane & 7) * 2);
}

// The loading warp has issued `n` stages.  Bounded by the time from one stage to the
// next: the tails may lie any number of tiles apart, so a limit on the whole wait
// would give up on a launch longer than that with nothing wrong.
__device__ __forceinline__ bool wait_loaded(const volatile int *loaded, int n, const Ctl &c)
{
    int seen = *loaded;
    uint64_t t0 = global_ns();
    while (seen < n) {
        __nanosleep(64);
        const int now = *loaded;
        if (now != seen) {
            seen = now;
            t0 = global_ns();
        } else if (*c.abort) {
            return false;
        } else if (global_ns() - t0 > c.timeout_ns) {
            give_up(c);
            return false;
        }
    }
    return true;
}

// This warp's part of a cut tile is written; true for the last of the parts,
// which then sees them all.  The counter's upper 48 bits are the launch's tag:
// any other tag there (what the memory held before) counts as zero, so nothing
// has to be cleared first, but before a replay (clear_for_replay).
__device__ __forceinline__ bool last_part(unsigned long long *count, unsigned long long tag,
                                          int parts, int lane)
{
    __threadfence();
    __syncwarp();
    int last = 0;
    if (lane == 0) {
        unsigned long long seen = *reinterpret_cast<volatile unsigned long long *>(count), now;
        for (;;) {   // one of at most 16 parts: some other part got through on every failure
            const unsigned long long n = (seen >> 16 == tag ? seen & 0xffff : 0) + 1;
            last = n == (unsigned long long)parts;
            now = atomicCAS(count, seen, last ? 0 : tag << 16 | n);
            if (now == seen)
                break;
            seen = now;
        }
    }
    // lane 0 saw the other parts arrive; a shuffle alone orders no memory, so the
    // other lanes' reads of those parts wait for lane 0 here
    last = __shfl_sync(0xffffffffu, last, 0);
    __syncwarp();
    __threadfence();
    return last;
}

// 32 columns of a cut tile's row, its parts added in their order.
__device__ __forceinline__ void add_parts(const float4 *from, int64_t step, int parts, float *v)
{
#pragma unroll
    for (int j = 0; j < 32; ++j)
        v[j] = 0.f;
#pragma unroll 1
    for (int k = 0; k < parts; ++k, from += step) {
        float4 f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            f[j] = __ldcg(from + 32 * j);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[4 * j] += f[j].x, v[4 * j + 1] += f[j].y;
            v[4 * j + 2] += f[j].z, v[4 * j + 3] += f[j].w;
        }
    }
}

__device__ __forceinline__ uint32_t pack_fp16(float a, float b)
{
    __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t *>(&h);
}
__device__ __forceinline__ float2 unpack_fp16(uint32_t u)
{
    return __half22float2(*reinterpret_cast<__half2 *>(&u));
}

// The mirrored place of 32 columns (w: pairs of columns of this lane's row):
// out points at column 0's place for row 0 of the warp.  Two exchanges give a
// lane one column's values for four rows, so a warp stores 64-byte pieces, 8
// bytes a lane.  rv rows and cv columns are valid (the pitch covers rv rounded
// up to 4).
__device__ __forceinline__ void store_mirror(const uint32_t *w, uint16_t *out, int64_t ld, int lane,
                                             int rv, int cv)
{
    uint32_t y[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const uint32_t o = __shfl_xor_sync(0xffffffffu, w[j], 1);
        y[j] = lane & 1 ? __byte_perm(o, w[j], 0x7632) : __byte_perm(w[j], o, 0x5410);
    }
    const bool up = lane & 2;
    const int r = lane & ~3;
#pragma unroll
    for (int j = 0; j < 16; j += 2) {
        const uint32_t o = __shfl_xor_sync(0xffffffffu, up ? y[j] : y[j + 1], 2);
        const int col = 2 * j + (up ? 2 : 0) + (lane & 1);
        if (r < rv && col < cv)
            *reinterpret_cast<uint2 *>(out + col * ld + r) =
                up ? make_uint2(o, y[j + 1]) : make_uint2(y[j], o);
    }
}

template <int CTAS, int BN, bool A_MN, bool B_MN, int EPI, int AR, int SETS>
__global__ void __launch_bounds__(Shape<CTAS, BN, EPI, AR>::THREADS, 1)
    grouped_kernel(const __grid_constant__ ParamsOf<SETS> p)
{
    using S = Shape<CTAS, BN, EPI, AR>;
    constexpr bool ACT = S::ACT;
    constexpr int STAGES = S::STAGES, KSUB = S::KSUB, BM = S::BM, A_BYTES = S::A_BYTES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~uintptr_t(1023));
    const uint32_t sA = smem_u32(smem), sB = smem_u32(smem + S::OFF_B);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + S::OFF_BAR);
    const uint32_t bar0 = smem_u32(bars);
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
    auto tfull_bar = [&](int a) { return bar0 + 8u * (2 * STAGES + a); };
    auto tempty_bar = [&](int a) { return bar0 + 8u * (2 * STAGES + 2 + a); };
    const uint32_t drain_bar = bar0 + 8u * (2 * STAGES + 4);
    auto tail_bar = [&](int s) { return bar0 + 8u * (2 * STAGES + 5 + s); };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + S::OFF_BAR + 8 * (3 * STAGES + 5));
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    volatile int *loaded = abort_flag + 1;   // EPI_DW: stages issued, for the tails' warp
    int2 *span = reinterpret_cast<int2 *>(smem + S::OFF_TAB);   // [groups] first row, rows
    int *tstart = reinterpret_cast<int *>(span + kMaxE);        // [entries + 1]
    int *plan_slot = tstart + kEntries + 1;                     // the Plan

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CTAS == 2 ? cluster_rank() : 0;
    const bool leader = rank == 0;
    const int unit = blockIdx.x / CTAS, units = gridDim.x / CTAS;
    const Ctl ctl{abort_flag, p.status, p.timeout_ns};

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full_bar(s), CTAS);   // each CTA's producer, with its bytes
            mbar_init(empty_bar(s), 1);
            mbar_init(tail_bar(s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(tfull_bar(a), 1);
            mbar_init(tempty_bar(a), CTAS * EPI_WARPS);
        }
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        *loaded = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        if (CTAS == 2) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                             smem_u32(tmem_slot)),
                         "r"(TMEM_COLS)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                             smem_u32(tmem_slot)),
                         "r"(TMEM_COLS)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
    }
    if (threadIdx.x == 0) {
        prefetch_map(&p.set[0].a[0]);
        prefetch_map(&p.set[0].b[0]);
    }
    // Without a segment table the tiles are known before the launch before is done:
    // with that, the maps fetched here and the arguments of one set, the 15 launches of
    // a 256 x 256 update take 117 us instead of 135.
    const bool ragged = p.set[0].mode != DENSE;
    if (ragged) {
        pdl_wait();
        pdl_trigger();
        // all groups' reads in flight at once
        for (int g = threadIdx.x; g < p.set[0].groups; g += S::THREADS)
            group_rows(p.offsets, p.rows, p.n_rows, g, &span[g].x, &span[g].y);
        __syncthreads();
    }
    if (warp == 2) {
        // the tile table: running sum of the entries' tiles
        int base = 0;
        for (int e0 = 0; e0 < p.entries; e0 += 32) {
            const int e = e0 + lane;
            int n = 0;
            if (e < p.entries) {
                int set = 0;
                while (set + 1 < p.nsets && p.set[set + 1].ent0 <= e)
                    ++set;
                n = entry_tiles<BM, BN>(p.set[set], span, e - p.set[set].ent0);
            }
            int sum = n;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, sum, d);
                if (lane >= d)
                    sum += o;
            }
            if (e < p.entries)
                tstart[e] = base + sum - n;
            base += __shfl_sync(0xffffffffu, sum, 31);
        }
        Plan pl{base, 1, base};
        if (p.partial && base > 0) {
            // contraction blocks of a tile, averaged over the first set's groups
            const Set &s = p.set[0];
            int k = s.K;
            if (s.mode == RAGGED_K) {
                k = 0;
                for (int g = lane; g < s.groups; g += 32)
                    k += span[g].y;
#pragma unroll
                for (int d = 16; d; d >>= 1)
                    k += __shfl_xor_sync(0xffffffffu, k, d);
                k /= s.groups;
            }
            pl = split_plan<CTAS>(base, s.segs * ((k + S::BK - 1) / S::BK), units,
                                  p.partial_bytes / (S::PART * 4), lane);
        }
        if (lane == 0) {
            tstart[p.entries] = base;
            plan_slot[0] = pl.whole, plan_slot[1] = pl.parts, plan_slot[2] = pl.items;
        }
    }
    tc_fence_before();
    if (CTAS == 2)
        cluster_sync();   // barriers initialised in both CTAs, TMEM allocated, table ready
    else
        __syncthreads();
    tc_fence_after();
    const Plan pl{plan_slot[0], plan_slot[1], plan_slot[2]};
    const int total = pl.items;
    const uint32_t tmem_base = *tmem_slot;
    if (!ragged) {
        pdl_wait();
        pdl_trigger();
    }
    if (p.clear_status && blockIdx.x == 0 && threadIdx.x == 0)
        *p.status = 0;

    if (warp == 0) {
        // ================= loads (both CTAs) =================
        int stage = 0, stages = 0;
        uint32_t phase = 0;
        int issued = 0;
        uint32_t last_phase = 0;   // bit s: phase of stage s's last use
        bool ok = true;
        Tile next;
        if (unit < total)
            next = decode<BM, BN, S::BK>(p, tstart, span, pl, unit);
        for (int tile = unit; ok && tile < total; tile += units) {
            const Tile t = next;
            bool ahead = false;   // the next tile is looked up behind this one's first stage
            const Set &s = p.set[t.set];
            const int m_row = t.m0 + (int)rank * AR + (s.mode == RAGGED_M ? t.row0 : 0);
            int sg = t.kbs > 0 ? t.b0 / t.kbs : 0, kb = t.b0 - sg * t.kbs;
            while (ok && sg * t.kbs + kb < t.b1) {
                const int ph = ACT ? sg : sg % s.period;
                const int bi = ACT ? 1 - sg : ph;
                const int grp = !ACT && s.seg_grouped ? sg / s.period : t.g;
                const int ga = s.a_grouped ? grp : 0, gb = s.b_grouped ? grp : 0;
                const bool uv = EPI == EPI_SWIGLU && sg == 1;
                const bool b_mn = ACT ? sg == 0 : B_MN;
                // B rows of this CTA, and their first
                const int b_rows = ACT ? (uv ? S::B_ROWS : BN / CTAS) : S::B_ROWS;
                const int b_row = t.n0 + (uv && CTAS == 2 ? 0 : (int)rank * (BN / CTAS));
                // a tile of few rows loads no more than 32 (the MMA's other rows are
                // whatever the stage holds; they are never stored)
                const bool few = S::ROWS && s.has_few && t.mg - t.m0 <= 32;
                const int a_rows = few ? 32 : AR;
                const CUtensorMap *am = few ? &s.a_few : &s.a[ph];
                const CUtensorMap *bm = uv && rank == 1 ? &s.b3 : &s.b[bi];
                const int end = min(t.kbs, t.b1 - sg * t.kbs);
                for (; kb < end; ++kb) {
                    int okw = lane == 0 ? (wait_bar(empty_bar(stage), phase ^ 1u, ctl) ? 1 : 0) : 1;
                    if (!__shfl_sync(0xffffffffu, okw, 0)) {
                        ok = false;
                        break;
                    }
                    const int rem = t.klen - kb * S::BK;
                    const int nks = rem >= S::BK ? KSUB : (rem + 63) / 64;
                    const bool a_wide = !few && s.a_wide, b_wide = s.b_wide;
                    // K-major: nks pieces of 64 of K; MN-major: BK rows
                    const uint32_t bytes =
                        (uint32_t)((A_MN || a_wide ? KSUB : nks) * a_rows * 128 +
                                   (b_mn || b_wide ? KSUB : nks) * b_rows * 128);
                    const uint32_t fb = CTAS == 2 ? map_to_rank(full_bar(stage), 0)
                                                  : full_bar(stage);
                    const uint32_t sa = sA + stage * KSUB * A_BYTES;
                    const uint32_t sb = sB + stage * KSUB * S::B_BYTES;
                    const int kc = t.k0 + kb * S::BK;
                    // rows behind the group's last must be cleared before use
                    const bool tail = EPI == EPI_DW && s.mode == RAGGED_K && ragged_tail<S::BK>(rem);
                    if (lane == 0) {
                        if (tail)
                            mbar_expect_tx(tail_bar(stage), bytes);
                        else
                            arrive_bytes<CTAS>(fb, bytes);
                        auto load = [&](uint32_t dst, const CUtensorMap *m, int c0, int c1, int c2,
                                        int c3) {
                            if (EPI == EPI_DW && tail)
                                load_box<false>(dst, m, tail_bar(stage), c0, c1, c2, c3);
                            else
                                load_box<CTAS == 2>(dst, m, fb, c0, c1, c2, c3);
                        };
                        if (a_wide) {
                            load(sa, am, 0, A_MN ? kc : m_row, (A_MN ? m_row : kc) / 64, ga);
                        } else if (A_MN) {
                            load(sa, am, m_row, kc, 0, ga);
                            load(sa + S::MN_BLOCK, am, m_row + 64, kc, 0, ga);
                        } else {
                            for (int ks = 0; ks < nks; ++ks)
                                load(sa + ks * A_BYTES, am, kc + ks * 64, m_row, 0, ga);
                        }
                        if (b_wide) {
                            load(sb, bm, 0, b_mn ? kc : b_row, (b_mn ? b_row : kc) / 64, gb);
                            if (uv && CTAS == 1)
                                load(sb + BN * 128, &s.b3, 0, b_row, kc / 64, gb);
                        } else if (b_mn) {
                            for (int b = 0; b < b_rows / 64; ++b)
                                load(sb + b * S::MN_BLOCK, bm, b_row + b * 64, kc, 0, gb);
                        } else {
                            for (int ks = 0; ks < nks; ++ks) {
                                load(sb + ks * S::B_BYTES, bm, kc + ks * 64, b_row, 0, gb);
                                if (uv && CTAS == 1)
                                    load(sb + ks * S::B_BYTES + BN * 128, &s.b3, kc + ks * 64,
                                         b_row, 0, gb);
                            }
                        }
                    }
                    if (EPI == EPI_DW && lane == 0)
                        *loaded = ++stages;
                    if (!ahead && tile + units < total)
                        next = decode<BM, BN, S::BK>(p, tstart, span, pl, tile + units);
                    ahead = true;
                    issued |= 1 << stage;
                    last_phase = (last_phase & ~(1u << stage)) | (phase << stage);
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                ++sg;
                kb = 0;
            }
            if (!ahead && tile + units < total)   // an empty contraction
                next = decode<BM, BN, S::BK>(p, tstart, span, pl, tile + units);
        }
        // the leader's full barriers count both CTAs' bytes: drain there
        if (leader && lane == 0)
            for (int s = 0; s < STAGES; ++s)
                if (issued >> s & 1)
                    wait_bar<true>(full_bar(s), last_phase >> s & 1, ctl, false);
    } else if (warp == 1) {
        // ================= MMA issue (leader CTA only) =================
        if (lane == 0 && leader) {
            const uint32_t fmt = p.fp16 ? 0u : (1u << 7) | (1u << 10);
            const uint32_t idesc0 = (1u << 4) | fmt | ((uint32_t)(S::MMA_M >> 4) << 24);
            int stage = 0;
            uint32_t phase = 0;
            int it = 0;
            bool ok = true, any = false;
            Tile next;
            if (unit < total)
                next = decode<BM, BN, S::BK>(p, tstart, span, pl, unit);
            for (int tile = unit; ok && tile < total; tile += units, ++it) {
                const Tile t = next;
                bool ahead = false;
                const Set &s = p.set[t.set];
                int slot = it & 1;
                if (!wait_bar(tempty_bar(slot), ((it >> 1) & 1) ^ 1u, ctl)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                bool first = true;
                int sg = t.kbs > 0 ? t.b0 / t.kbs : 0, kb = t.b0 - sg * t.kbs, n = 0;
                while (ok && sg * t.kbs + kb < t.b1) {
                    const bool uv = EPI == EPI_SWIGLU && sg == 1;
                    const bool b_mn = ACT ? sg == 0 : B_MN;
                    uint32_t d = tmem_base;
                    if (!ACT)
                        d += slot * BN;
                    else if (EPI == EPI_GELU)
                        d += slot * 2 * BN + (sg == 0 ? S::DH_COL : 0);
                    else
                        d += sg == 0 ? S::DH_COL + slot * BN : 0;
                    if (ACT)
                        first = true;
                    if (uv && it > 0) {
                        // u | v has one slot: the previous tile's epilogue must be done
                        if (!wait_bar(tempty_bar(slot ^ 1), ((it - 1) >> 1) & 1, ctl)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                    }
                    const uint32_t idesc = idesc0 | (A_MN ? 1u << 15 : 0u) |
                                           (b_mn ? 1u << 16 : 0u) |
                                           ((uint32_t)((uv ? 2 * BN : BN) >> 3) << 17);
                    const int end = min(t.kbs, t.b1 - sg * t.kbs);
                    for (; kb < end; ++kb, ++n) {
                        if (S::CHUNK > 0 && n > 0 && n % S::CHUNK_BLOCKS == 0) {
                            // this accumulator is full: on to the other one
                            commit_all<CTAS>(tfull_bar(slot));
                            ++it;
                            slot = it & 1;
                            d = tmem_base + slot * BN;
                            first = true;
                            if (!wait_bar(tempty_bar(slot), ((it >> 1) & 1) ^ 1u, ctl)) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
                        }
                        const int rem = t.klen - kb * S::BK;
                        // a cleared tail: the other CTA's threads wrote to the stage too
                        const bool got = A_MN && rem < S::BK
                                             ? wait_bar<true>(full_bar(stage), phase, ctl)
                                             : wait_bar(full_bar(stage), phase, ctl);
                        if (!got) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const int steps = rem >= S::BK ? S::BK / 16 : (rem + 15) / 16;
#pragma unroll
                        for (int st = 0; st < S::BK / 16; ++st) {
                            if (st >= steps)
                                break;
                            const int ks = st >> 2, kk = st & 3;
                            const uint32_t a = sA + stage * KSUB * A_BYTES;
                            const uint32_t b = sB + stage * KSUB * S::B_BYTES;
                            mma<CTAS>(d,
                                      A_MN ? sdesc_mn(a + st * 2048, S::MN_BLOCK)
                                           : sdesc_sw128(a + ks * A_BYTES + kk * 32),
                                      b_mn ? sdesc_mn(b + st * 2048, S::MN_BLOCK)
                                           : sdesc_sw128(b + ks * S::B_BYTES + kk * 32),
                                      idesc, first ? 0u : 1u);
                            first = false;
                        }
                        commit_all<CTAS>(empty_bar(stage));
                        any = true;
                        if (!ahead && tile + units < total)
                            next = decode<BM, BN, S::BK>(p, tstart, span, pl, tile + units);
                        ahead = true;
                        if (++stage == STAGES) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                    ++sg;
                    kb = 0;
                }
                if (!ok)
                    break;
                if (!ahead && tile + units < total)   // an empty contraction
                    next = decode<BM, BN, S::BK>(p, tstart, span, pl, tile + units);
                commit_all<CTAS>(tfull_bar(slot));
                any = true;
            }
            if (any) {
                if (CTAS == 2)
                    mma_commit_local2(drain_bar);
                else
                    mma_commit(drain_bar);
                wait_bar(drain_bar, 0, ctl, false);
            }
        }
    } else if (EPI == EPI_DW && warp == 2) {
        // ================= ragged tails (both CTAs) =================
        int blocks = 0;          // stages used by the tiles before
        uint32_t parity = 0;     // bit s: phase of stage s's next tail
        bool ok = true;
        for (int tile = unit; ok && tile < total; tile += units) {
            const Tile t = decode<BM, BN, S::BK>(p, tstart, span, pl, tile);
            const int rem = t.klen - (t.kbs - 1) * S::BK;
            blocks += t.b1 - t.b0;
            if (p.set[t.set].mode != RAGGED_K || t.b1 == t.b0 || t.b1 != t.kbs ||
                !ragged_tail<S::BK>(rem))
                continue;
            const int stage = (blocks - 1) % STAGES;
            ok = lane > 0 || wait_loaded(loaded, blocks, ctl);
            ok = __all_sync(0xffffffffu, ok) && wait_bar(tail_bar(stage), parity >> stage & 1, ctl);
            ok = __all_sync(0xffffffffu, ok);
            parity ^= 1u << stage;
            // 128 bytes a row, so 8 lanes a row: four rows of a box at a time
            const uint32_t at = (uint32_t)(rem + (lane >> 3)) * 128 + (lane & 7) * 16;
            const int rows = 16 - (rem & 15);
            for (int box = 0; box < 2 + S::B_ROWS / 64; ++box) {
                const uint32_t dst = box < 2 ? sA + stage * KSUB * A_BYTES + box * S::MN_BLOCK
                                             : sB + stage * KSUB * S::B_BYTES +
                                                   (box - 2) * S::MN_BLOCK;
#pragma unroll
                for (int r = 0; r < 16; r += 4)
                    if (r + (lane >> 3) < rows)
                        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(dst + at +
                                                                                       r * 128),
                                     "r"(0)
                                     : "memory");
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0)
                arrive_written<CTAS>(CTAS == 2 ? map_to_rank(full_bar(stage), 0) : full_bar(stage));
        }
    } else if (warp >= S::FIRST_EPI) {
        // ================= epilogue (eight warps, both CTAs) =================
        const int q = warp & 3, half = (warp - S::FIRST_EPI) >> 2;
        uint8_t *stg = smem + S::OFF_STG + (S::STAGED ? warp - S::FIRST_EPI : 0) * STG_WARP;
        int it = 0;
        for (int tile = unit; tile < total; tile += units, ++it) {
            const Tile t = decode<BM, BN, S::BK>(p, tstart, span, pl, tile);
            const Set &s = p.set[t.set];
            int slot = it & 1;
            const int m = t.m0 + (int)rank * 128 + q * 32;   // first row, in the group
            // rows of it from there on, in this tile
            const int rv = AR < 128 && q > 0 ? 0 : t.mg - m;
            const int c_end = rv > 0 ? min((half + 1) * (BN / 2), s.N - t.n0) : 0;
            // base is read a chunk ahead: the first before the products are done
            uint32_t base[EPI == EPI_NS ? 16 : 1];
            const bool based = EPI == EPI_NS && s.base && lane < rv;
            float alpha = s.alpha, beta = s.beta;
            const uint8_t *from = reinterpret_cast<const uint8_t *>(
                static_cast<const __half *>(s.base) + (int64_t)t.g * s.base_group +
                (int64_t)(m + lane) * s.base_ld + t.n0);
            if constexpr (EPI == EPI_DW) {
                // the addend's lines on their way to L2 while the products run
                if (s.add && lane < rv) {
                    const int esz = s.out_f32 ? 4 : 2, c = half * (BN / 2);
                    const uint8_t *row = static_cast<const uint8_t *>(s.add) +
                                         ((int64_t)t.g * s.out_group +
                                          (int64_t)(m + lane) * s.ld + t.n0 + c) * esz;
                    for (int b = 0; b < (c_end - c) * esz; b += 128)
                        asm volatile("prefetch.global.L2 [%0];" ::"l"(row + b));
                }
            }
            if constexpr (EPI == EPI_NS) {
                const int c = half * (BN / 2);
                if (based && c < c_end)
                    load_row<2>(from + 2 * c, 2 * (s.N - t.n0 - c), s.base_bytes, base);
                if (s.scale) {
                    const float sc = s.scale[t.g], to = s.scale_to ? s.scale_to[t.g] : 1.f;
                    alpha = s.scale_pow == 2 ? alpha / sc / sc : alpha * to / sc;
                    beta = beta * to / sc;
                }
            }
            if (!wait_bar(tfull_bar(slot), (it >> 1) & 1, ctl))
                break;
            tc_fence_after();
            const uint32_t tq = tmem_base + ((uint32_t)(q * 32) << 16);
            // element (first row of the warp, first column of the tile) of the output
            const int64_t row = m + (s.mode == RAGGED_M ? t.row0 : 0);
            const int64_t at0 = (s.mode == RAGGED_M ? 0 : (int64_t)t.g * s.out_group) +
                                row * s.ld + t.n0;
            const int bytes = s.bytes;
            // a cut tile's parts: 32 rows x BN / 2 columns of this warp, 4 columns of
            // a lane together
            const int wid = (int)rank * S::ROW_WARPS + half * (AR / 32) + q;
            const int64_t part_step = S::PART / 4;
            float4 *part0 = reinterpret_cast<float4 *>(p.partial) +
                            ((int64_t)t.cut * t.parts + t.part) * part_step +
                            (int64_t)wid * (BN / 8) * 32;
            unsigned long long *count = p.counters + t.cut * (CTAS * S::ROW_WARPS) + wid;
            if constexpr (S::CHUNK > 0) {
                float sum[BN / 2];
                if (t.b0 == t.b1) {   // nothing was accumulated: an empty group's sum
#pragma unroll
                    for (int i = 0; i < BN / 2; ++i)
                        sum[i] = 0.f;
                } else {
#pragma unroll
                    for (int i = 0; i < BN / 64; ++i)
                        tmem_ld32(tq + slot * BN + half * (BN / 2) + 32 * i, sum + 32 * i);
                }
                bool ok = true;
                for (int k = S::CHUNK_BLOCKS; k < t.b1 - t.b0; k += S::CHUNK_BLOCKS) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (CTAS == 2)
                            mbar_arrive_remote(map_to_rank(tempty_bar(slot), 0));
                        else
                            mbar_arrive(tempty_bar(slot));
                    }
                    ++it;
                    slot = it & 1;
                    if (!wait_bar(tfull_bar(slot), (it >> 1) & 1, ctl)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
#pragma unroll
                    for (int i = 0; i < BN / 32; ++i) {
                        float v[16];
                        tmem_ld16(tq + slot * BN + half * (BN / 2) + 16 * i, v);
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            sum[16 * i + j] += v[j];
                    }
                }
                if (!ok)
                    break;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {   // the sums are in registers: release TMEM before the stores
                    if (CTAS == 2)
                        mbar_arrive_remote(map_to_rank(tempty_bar(slot), 0));
                    else
                        mbar_arrive(tempty_bar(slot));
                }
                if (t.parts > 1) {
                    if (rv <= 0)
                        continue;
                    float4 *at = part0 + lane;
#pragma unroll
                    for (int i = 0; i < BN / 8; ++i)
                        at[32 * i] = make_float4(sum[4 * i], sum[4 * i + 1], sum[4 * i + 2],
                                                 sum[4 * i + 3]);
                    if (!last_part(count, p.tag, t.parts, lane))
                        continue;
                    const float4 *from = part0 + lane - t.part * part_step;
#pragma unroll
                    for (int i = 0; i < BN / 2; i += 32)
                        add_parts(from + 8 * i, part_step, t.parts, sum + i);
                }
                if constexpr (EPI == EPI_DW) {
                    if (rv > 0)
                        store_sums<BN / 2>(s, sum, at0 + half * (BN / 2), lane,
                                           rv, c_end - half * (BN / 2), bytes);
                } else {
#pragma unroll
                    for (int i = 0; i < BN / 64; ++i) {
                        const int c = half * (BN / 2) + 32 * i;
                        uint32_t w[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            w[j] = pack_bf16(sum[32 * i + 2 * j], sum[32 * i + 2 * j + 1]);
                        if (c < c_end)
                            store_traded(w, static_cast<uint16_t *>(s.out) + at0 + c, s.ld, lane, rv,
                                         s.N - t.n0 - c);
                    }
                }
                continue;
            }
            bool released = false;
            auto release = [&]() {   // this warp is done with the accumulator
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (CTAS == 2)
                        mbar_arrive_remote(map_to_rank(tempty_bar(slot), 0));
                    else
                        mbar_arrive(tempty_bar(slot));
                }
            };
            if (!ACT && t.parts > 1) {
                if (rv > 0) {
#pragma unroll
                    for (int i = 0; i < BN / 64; ++i) {
                        float v[32];
                        tmem_ld32(tq + slot * BN + half * (BN / 2) + 32 * i, v);
                        if (t.b0 == t.b1) {   // a part of a short contraction may be empty
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                v[j] = 0.f;
                        }
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            part0[(8 * i + j) * 32 + lane] =
                                make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                    }
                }
                release();
                released = true;
                if (rv <= 0 || !last_part(count, p.tag, t.parts, lane))
                    continue;
            }
#pragma unroll 1
            for (int c = half * (BN / 2); c < c_end; c += 32) {
                const int cv = s.N - t.n0 - c;
                const int64_t at = at0 + c;
                float v[32];
                uint32_t w[16];
                if constexpr (ACT) {
                    // u = x W1^T, v = x W3^T, dh = dy W2; h = act(u) (v), and the
                    // gradients of u and v:
                    //   GELU    h = u Phi(u); du = dh (Phi(u) + u phi(u))
                    //   SwiGLU  h = u s v, s = 1 / (1 + e^-u);
                    //           du = dh v s (1 + u (1 - s)), dv = dh u s
                    // h, du and dv are rounded to bf16 here, as the forward rounds its h: they
                    // are the next products' operands on the tensor cores.  Against 64 bits
                    // the gradients are off by 2.4e-3 (2-norm); held in fp32 until the end
                    // they would be by 1.7e-3, at twice the products that take them.
                    const uint32_t tu = tq + c + (EPI == EPI_GELU ? slot * 2 * BN : 0);
                    const uint32_t tdh = tq + c + S::DH_COL + slot * (EPI == EPI_GELU ? 2 * BN : BN);
                    float dh[32];
                    tmem_ld32(tu, v);
                    tmem_ld32(tdh, dh);
                    if constexpr (EPI == EPI_GELU) {
                        uint32_t g[16];
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            float h[2], du[2];
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const float u = v[i + j];
                                const float cdf = 0.5f * (1.f + erff(u * 0.70710678118654752f));
                                h[j] = u * cdf;
                                du[j] = dh[i + j] *
                                        (cdf + u * 0.39894228040143268f * __expf(-0.5f * u * u));
                            }
                            w[i / 2] = pack_bf16(h[0], h[1]);
                            g[i / 2] = pack_bf16(du[0], du[1]);
                        }
                        store_traded(w, static_cast<uint16_t *>(s.out) + at, s.ld, lane, rv, cv);
                        store_traded(g, static_cast<uint16_t *>(s.out2) + at, s.ld, lane, rv, cv);
                    } else {
                        float x3[32];
                        tmem_ld32(tu + BN, x3);
                        uint32_t g[16], k[16];
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            float h[2], du[2], dv[2];
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const float u = v[i + j];
                                const float sg = __fdividef(1.f, 1.f + __expf(-u));
                                const float us = u * sg;
                                h[j] = us * x3[i + j];
                                dv[j] = dh[i + j] * us;
                                du[j] = dh[i + j] * x3[i + j] * (sg + us * (1.f - sg));
                            }
                            w[i / 2] = pack_bf16(h[0], h[1]);
                            g[i / 2] = pack_bf16(du[0], du[1]);
                            k[i / 2] = pack_bf16(dv[0], dv[1]);
                        }
                        store_traded(w, static_cast<uint16_t *>(s.out) + at, s.ld, lane, rv, cv);
                        store_traded(g, static_cast<uint16_t *>(s.out2) + at, s.ld, lane, rv, cv);
                        store_traded(k, static_cast<uint16_t *>(s.out3) + at, s.ld, lane, rv, cv);
                    }
                } else {
                    if (t.parts > 1) {
                        add_parts(part0 + lane - t.part * part_step + (c - half * (BN / 2)) * 8,
                                  part_step, t.parts, v);
                    } else {
                        tmem_ld32(tq + slot * BN + c, v);
                    }
                    if constexpr (S::ROWS) {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
                        store_traded(w, static_cast<uint16_t *>(s.out) + at, s.ld, lane, rv, cv);
                    } else if constexpr (EPI == EPI_NS) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            v[i] *= alpha;
                        if (based) {
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const float2 f = unpack_fp16(base[i]);
                                v[2 * i] += beta * f.x;
                                v[2 * i + 1] += beta * f.y;
                            }
                            if (c + 32 < c_end)
                                load_row<2>(from + 2 * (c + 32), 2 * (cv - 32), s.base_bytes, base);
                        }
                        if (s.diag != 0.f && t.n0 + c < m + 32 && m < t.n0 + c + 32) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                v[i] += t.n0 + c + i == m + lane ? s.diag : 0.f;
                        }
                        uint16_t *hi = static_cast<uint16_t *>(s.out) + at;
                        if (s.out_bf16) {
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
                            if (bytes >= 16)
                                store_traded(w, hi, s.ld, lane, rv, cv);
                            else
                                store_odd(stg, lane, w, hi, s.ld, rv, cv);
                            continue;
                        }
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            w[i] = pack_fp16(v[2 * i], v[2 * i + 1]);
                        // columns past N up to the pitch's multiple of 8 are written too
                        const int cw = (cv + 7) & ~7;
                        store_traded(w, hi, s.ld, lane, rv, cw);
                        if (s.out2) {
                            uint32_t lw[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const float2 f = unpack_fp16(w[i]);
                                lw[i] = pack_fp16(v[2 * i] - f.x, v[2 * i + 1] - f.y);
                            }
                            store_traded(lw, static_cast<uint16_t *>(s.out2) + at, s.ld, lane, rv,
                                         cw);
                        }
                        if (s.sym && t.n0 + BN <= t.m0)
                            store_mirror(w,
                                         static_cast<uint16_t *>(s.out) +
                                             (int64_t)t.g * s.out_group +
                                             (int64_t)(t.n0 + c) * s.ld + m,
                                         s.ld, lane, rv, cv);
                    }
                }
            }
            if (!released)
                release();
        }
    }

    // ---- tear-down: all CTAs done with TMEM before it is freed ----
    tc_fence_before();
    __syncthreads();
    if (CTAS == 2)
        cluster_sync();
    if (threadIdx.x == 0 && *abort_flag)
        atomicExch(&g_gave_up, (int32_t)MOE_ERR_DEVICE_TIMEOUT);
    if (warp == 1) {
        tc_fence_after();
        if (CTAS == 2)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                         "r"(TMEM_COLS)
                         : "memory");
        else
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                         "r"(TMEM_COLS)
                         : "memory");
    }
}

// One bounded wait on a barrier that nothing arrives on (diagnostic).
__global__ void probe_kernel(unsigned long long timeout_ns)
{
    __shared__ uint64_t bar;
    __shared__ int abort_flag;
    mbar_init(smem_u32(&bar), 1);
    abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    const Ctl ctl{&abort_flag, &g_gave_up, timeout_ns};
    wait_bar(smem_u32(&bar), 0, ctl);
}

__global__ void __launch_bounds__(1024) clear_counters_kernel(unsigned long long *counters)
{
    pdl_wait();
    pdl_trigger();
    counters[blockIdx.x * 1024 + threadIdx.x] = 0;
}

template <int CTAS, int BN, bool A_MN, bool B_MN, int EPI, int SETS, int AR = 128>
cudaError_t launch_sets(const Params &all, cudaStream_t s)
{
    ParamsOf<SETS> p;   // the last member is shorter
    static_assert(offsetof(ParamsOf<SETS>, set) == offsetof(Params, set), "layout");
    memcpy(&p, &all, sizeof p);
    using S = Shape<CTAS, BN, EPI, AR>;
    static_assert(S::SMEM <= 232448, "shared memory");
    // mn_box_rows: the rows of a stage
    static_assert(S::BK == (CTAS == 1 && EPI == EPI_SWIGLU ? 64 : 128), "stage");
    static_assert(S::DH_COL + 2 * BN <= 512 || !S::ACT, "TMEM");
    // the counters of the most tiles that are cut at a time
    static_assert(kPartialBytes / (S::PART * 4) / 2 * CTAS * S::ROW_WARPS * 8 <= kCounterBytes,
                  "counters");
    auto kern = grouped_kernel<CTAS, BN, A_MN, B_MN, EPI, AR, SETS>;
    cudaError_t err = raise_smem_limit((const void *)kern, S::SMEM);
    if (err != cudaSuccess)
        return err;
    int units = device_sms();
    if (CTAS == 2) {
        err = cached_active_clusters((const void *)kern, S::THREADS, S::SMEM, 2, &units);
        if (err != cudaSuccess)
            return err;
        if (units < 1)
            return cudaErrorInvalidConfiguration;
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CTAS;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(CTAS * units);
    cfg.blockDim = dim3(S::THREADS);
    cfg.dynamicSmemBytes = S::SMEM;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = CTAS == 2 ? 2 : 1;
    err = cudaLaunchKernelEx(&cfg, kern, p);
    return err != cudaSuccess ? err : cudaGetLastError();
}

// Stacks and products are one set; hidden gradients and the FFN's dx a ragged and
// perhaps a shared one; weight gradients one, or up to six of an FFN.
template <int CTAS, int BN, bool A_MN, bool B_MN, int EPI, int AR = 128>
cudaError_t launch_one(const Params &p, cudaStream_t s)
{
    constexpr bool rows = EPI == EPI_ROWS || EPI == EPI_ROWS_LONG;
    constexpr int most = EPI == EPI_DW ? kSets
                         : EPI == EPI_NS || (rows && (!B_MN || AR < 128)) ? 1 : 2;
    if (p.nsets > most)
        return cudaErrorInvalidValue;
    if (most > 1 && !(EPI == EPI_GELU || EPI == EPI_SWIGLU) && p.nsets == 1)
        return launch_sets<CTAS, BN, A_MN, B_MN, EPI, 1, AR>(p, s);
    return launch_sets<CTAS, BN, A_MN, B_MN, EPI, most, AR>(p, s);
}

template <int EPI>
cudaError_t launch_rows(const Params &p, Layout layout, Tiles tiles, cudaStream_t s)
{
    const bool pair = tiles == PAIR_256;
    if (tiles == ONE_32)
        return layout == A_K_B_MN ? launch_one<1, 128, false, true, EPI, 32>(p, s)
                                  : launch_one<1, 128, false, false, EPI, 32>(p, s);
    if (layout == A_K_B_MN)
        return pair ? launch_one<2, 256, false, true, EPI>(p, s)
                    : launch_one<1, 128, false, true, EPI>(p, s);
    return pair ? launch_one<2, 256, false, false, EPI>(p, s)
                : launch_one<1, 128, false, false, EPI>(p, s);
}

constexpr int kBnAct = 128;

// [groups, rows, cols] 2-byte elements, row pitch ld, as (64, rows, cols / 64,
// groups) with boxes of `blocks` blocks of 64 columns (wide), or as (cols, rows,
// 1, groups) with boxes of 64 columns.
bool map_4d(CUtensorMap *m, const void *base, int64_t rows, int64_t cols, int64_t ld,
            int64_t groups, int64_t group_stride, int box_rows, int blocks)
{
    EncodeTiled enc = encoder();
    if (!enc)
        return false;
    const bool wide = blocks > 0;
    const cuuint64_t far = (cuuint64_t)(group_stride > 0 ? group_stride : rows * ld) * 2;
    cuuint64_t dims[4] = {(cuuint64_t)(wide ? 64 : cols), (cuuint64_t)rows,
                          (cuuint64_t)(wide ? cols / 64 : 1), (cuuint64_t)groups};
    cuuint64_t strides[3] = {(cuuint64_t)ld * 2, wide ? 128 : far, far};
    cuuint32_t box[4] = {64, (cuuint32_t)box_rows, (cuuint32_t)(wide ? blocks : 1), 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool map_k(CUtensorMap *m, const void *base, int64_t rows, int64_t cols, int64_t ld,
           int64_t groups, int64_t group_stride, int box_rows, int stage_k, bool wide)
{
    return map_4d(m, base, rows, cols, ld, groups, group_stride, box_rows,
                  wide ? stage_k / 64 : 0);
}

bool map_mn(CUtensorMap *m, const void *base, int64_t rows, int64_t cols, int64_t ld,
            int64_t groups, int64_t group_stride, int stage_k, int box_cols, bool wide)
{
    return map_4d(m, base, rows, cols, ld, groups, group_stride, stage_k, wide ? box_cols / 64 : 0);
}

int b_box(Epi epi, Tiles tiles)   // SwiGLU: a box of W1 and one of W3
{
    return epi == EPI_GELU && tiles == PAIR_256 ? kBnAct / 2 : 128;
}

int dh_box(Tiles tiles) { return tiles == PAIR_256 ? kBnAct / 2 : kBnAct; }

int stage_k(Epi epi, Tiles tiles) { return epi == EPI_SWIGLU && tiles != PAIR_256 ? 64 : 128; }

cudaError_t gave_up_grouped(int32_t **word)
{
    return cudaGetSymbolAddress(reinterpret_cast<void **>(word), g_gave_up);
}

cudaError_t launch_grouped_probe(unsigned long long timeout_ns, cudaStream_t s)
{
    probe_kernel<<<1, 1, 0, s>>>(timeout_ns);
    return cudaGetLastError();
}

cudaError_t clear_for_replay(unsigned long long *counters, cudaStream_t s)
{
    static_assert(kCounterBytes % (8 * 1024) == 0, "counters");
    cudaStreamCaptureStatus capture;
    const cudaError_t err = cudaStreamIsCapturing(s, &capture);
    if (err != cudaSuccess || capture == cudaStreamCaptureStatusNone)
        return err;
    return launch_pdl(clear_counters_kernel, dim3(kCounterBytes / (8 * 1024)), dim3(1024), 0, s,
                      counters);
}

cudaError_t launch_tc(Params &p, Epi epi, Layout layout, Tiles tiles, cudaStream_t s)
{
    int ents = 0;
    int64_t longest = 0;   // contraction
    for (int i = 0; i < p.nsets; ++i) {
        Set &v = p.set[i];
        if ((int64_t)v.segs * v.K > longest)
            longest = (int64_t)v.segs * v.K;
        v.ent0 = ents;
        // what every row of every output (and addend) is aligned to
        const int64_t esz = epi == EPI_DW && v.out_f32 ? 4 : 2;
        const uint64_t all = (uint64_t)(v.ld * esz) | (uint64_t)(v.out_group * esz) |
                             reinterpret_cast<uint64_t>(v.out) |
                             reinterpret_cast<uint64_t>(v.out2) |
                             reinterpret_cast<uint64_t>(v.out3) |
                             reinterpret_cast<uint64_t>(v.add);
        v.bytes = all % 32 == 0 ? 32 : (all % 16 == 0 ? 16 : 2);
        const uint64_t base = (uint64_t)(v.base_ld * 2) | (uint64_t)(v.base_group * 2) |
                              reinterpret_cast<uint64_t>(v.base);
        v.base_bytes = base % 32 == 0 ? 32 : 16;
        ents += v.groups;
    }
    if (ents > kEntries)
        return cudaErrorInvalidValue;
    p.entries = ents;
    if (epi == EPI_GELU || epi == EPI_SWIGLU)
        p.partial = nullptr;   // u, v and dh are not cut
    p.timeout_ns = 2000000000ull;
    static std::atomic<unsigned long long> calls{(unsigned long long)time(nullptr) << 20};
    p.tag = (calls.fetch_add(1) * 0x9E3779B97F4A7C15ull) >> 16 | 1;
    const bool pair = tiles == PAIR_256;
    switch (epi) {
    case EPI_GELU:
        return pair ? launch_one<2, kBnAct, false, false, EPI_GELU>(p, s)
                    : launch_one<1, kBnAct, false, false, EPI_GELU>(p, s);
    case EPI_SWIGLU:
        return pair ? launch_one<2, kBnAct, false, false, EPI_SWIGLU>(p, s)
                    : launch_one<1, kBnAct, false, false, EPI_SWIGLU>(p, s);
    case EPI_DW:
        return pair ? launch_one<2, 256, true, true, EPI_DW>(p, s)
                    : launch_one<1, 128, true, true, EPI_DW>(p, s);
    case EPI_ROWS:
    case EPI_ROWS_LONG:
        return longest > kLongRows ? launch_rows<EPI_ROWS_LONG>(p, layout, tiles, s)
                                   : launch_rows<EPI_ROWS>(p, layout, tiles, s);
    case EPI_NS:
        if (layout == A_K_B_MN)
            return pair ? launch_one<2, 256, false, true, EPI_NS>(p, s)
                        : launch_one<1, 128, false, true, EPI_NS>(p, s);
        if (layout == A_MN_B_MN)
            return pair ? launch_one<2, 256, true, true, EPI_NS>(p, s)
                        : launch_one<1, 128, true, true, EPI_NS>(p, s);
        return pair ? launch_one<2, 256, false, false, EPI_NS>(p, s)
                    : launch_one<1, 128, false, false, EPI_NS>(p, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace grp
}  // namespace moe
