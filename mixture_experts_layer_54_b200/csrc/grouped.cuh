// Grouped matrix products shared by the expert training calls: what a launch
// is told (grouped_tc.cu runs it on the tensor cores, grouped_simt.cu in fp32).
#pragma once

#include "internal.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace grp {

// Which extent of a group the segment table gives.
//   RAGGED_M: its output rows are rows [offsets[g], offsets[g] + rows[g]) of
//             one tall buffer (products with the expert's weights);
//   RAGGED_K: its contraction runs over those rows (weight gradients);
//   DENSE:    every group has the same extents (shared experts, stacks).
enum Mode { RAGGED_M = 0, RAGGED_K = 1, DENSE = 2 };

constexpr int kSets = 6;
constexpr int kEntries = 1024;   // (set, group) pairs of a launch
// Scratch of cut tiles: the parts, and the counters (most tiles cut at a time:
// as many as parts fit, at least two parts each).
constexpr int kPartialBytes = 32 << 20;
constexpr int kCounterBytes = kPartialBytes / (128 * 128 * 4) / 2 * 8 * 8;

// One family of products of a launch: out[g] = sum over K segments of A B^T.
struct Set {
    // Segment i of a tile's contraction multiplies operand pair i % period; with
    // seg_grouped both operands' group is i / period.
    CUtensorMap a[2], b[2];
    CUtensorMap a_few;           // a[0] in boxes of 32 rows, if has_few (ONE_128, one segment)
    CUtensorMap b3;              // EPI_SWIGLU: W3 (b[0] = W1, b[1] = W2)
    int mode, groups, ent0;      // ent0: first entry of the tile table
    int M, N, K;                 // output rows (not RAGGED_M), columns, contraction (not RAGGED_K)
    int segs, period, seg_grouped, has_few;
    int a_grouped, b_grouped;    // 1: the operand has one matrix per group
    int a_wide, b_wide;          // 1: one box is a whole stage (all segments')
    int sym;                     // 1: out is symmetric; only tiles on or below the diagonal
    int ld;                      // row pitch of out (elements)
    int64_t out_group;           // elements between the groups' outputs (not RAGGED_M)
    void *out;                   // EPI_GELU / EPI_SWIGLU: h
    void *out2, *out3;           // EPI_GELU / EPI_SWIGLU: du, dv; EPI_NS: out2
    const void *add;             // EPI_DW, nullable: added before the rounding
    int out_f32;                 // EPI_DW
    // EPI_NS: val = alpha acc + beta base (+ diag on the diagonal), stored as fp16
    // (out2: what the rounding lost, as another fp16) or as bf16
    const void *base;            // nullable
    float diag;
    int base_ld, out_bf16;
    int64_t base_group;
    float alpha, beta;
    const float *scale;          // nullable: alpha / scale[g]^scale_pow, beta / scale[g]
    const float *scale_to;       // nullable: alpha and beta times scale_to[g]
    int scale_pow;
    int bytes, base_bytes;       // alignment of the rows (32, 16 or 2), found at launch
};

// A kernel takes as many sets as its launches have: six are 6 KB of arguments.
template <int SETS>
struct __align__(64) ParamsOf {
    int nsets, entries;          // set 0 is the ragged one, if any is
    const int32_t *offsets;      // [G + 1]
    const int32_t *rows;         // [G], nullable: offsets[g + 1] - offsets[g]
    int n_rows;                  // rows of the tall buffers; the table is held inside them
    int fp16;                    // operands are fp16 (else bf16)
    // scratch of tiles cut along their contraction: parts' accumulators, and a
    // counter for each warp of each cut tile (any contents, but a captured launch's
    // counters are cleared first: clear_for_replay).  NULL: no tile is cut
    float *partial;
    unsigned long long *counters;
    int partial_bytes;
    unsigned long long tag;      // of this launch in the counters
    int32_t *status;
    int clear_status;
    unsigned long long timeout_ns;
    Set set[SETS];
};
using Params = ParamsOf<kSets>;

// First row and row count of group g, held inside the buffers whatever the
// table says.
__device__ __forceinline__ void group_rows(const int32_t *offsets, const int32_t *rows, int n_rows,
                                           int g, int *start, int *count)
{
    const int lo = min(max(offsets[g], 0), n_rows), hi = min(max(offsets[g + 1], lo), n_rows);
    *start = lo;
    *count = rows ? min(max(rows[g], 0), hi - lo) : hi - lo;
}

// MN-major operand, 128-byte swizzle: 64 contiguous elements per 128-byte row,
// one row per contraction index; 8-row groups 1024 bytes apart (stride offset),
// blocks of 64 elements `block` bytes apart (leading offset).
__device__ __forceinline__ uint64_t sdesc_mn(uint32_t saddr, uint32_t block)
{
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(block >> 4) << 16) |
           ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

template <int CTAS>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                    uint32_t accumulate)
{
    if (CTAS == 2)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
}

// Epilogues: EPI_ROWS bf16 rows; EPI_DW fp32 or bf16 with an addend; EPI_NS
// the Newton-Schulz stores; EPI_GELU / EPI_SWIGLU the hidden activations and
// their gradients.  EPI_ROWS_LONG is launch_tc's own choice for EPI_ROWS.
enum Epi { EPI_ROWS = 0, EPI_DW = 1, EPI_NS = 2, EPI_GELU = 3, EPI_SWIGLU = 4, EPI_ROWS_LONG = 5 };

// Operand layouts: MN = the contraction index is the row index of the stored
// matrix (its other index is contiguous), K = the contraction is contiguous.
enum Layout { A_K_B_K = 0, A_K_B_MN = 1, A_MN_B_MN = 2 };

// PAIR_256: 256 x 256 on SM pairs (hidden gradients: 256 x 128); ONE_128: 128 x
// 128 and ONE_32: 32 x 128 (EPI_ROWS alone) on single SMs.
enum Tiles { PAIR_256, ONE_128, ONE_32 };

cudaError_t launch_tc(Params &p, Epi epi, Layout layout, Tiles tiles, cudaStream_t s);

// The counters of cut tiles go by the tag of their launch, a new one for every call
// of launch_tc.  A captured launch keeps its tag, so what a replay that gave up left
// in the counters would count as the next replay's: while the stream is being
// captured this clears them, once before the launches of a call (0.5 to 1.7 us of a
// replay; nothing otherwise).
cudaError_t clear_for_replay(unsigned long long *counters, cudaStream_t s);
// Whether tiles of this contraction may be cut at all: four blocks at least
// (split_plan).
inline bool may_cut(int64_t contraction) { return contraction > 3 * 128; }

// Maps of a [groups, rows, cols] 2-byte tensor with row pitch ld (group_stride in
// elements) for the operand's role: K-major (cols is the contraction), boxes of
// box_rows; MN-major (rows is the contraction), boxes of box_cols.  wide: cols is
// a multiple of 64 and one box is a whole stage (a_wide, b_wide of the Set).
bool map_k(CUtensorMap *m, const void *base, int64_t rows, int64_t cols, int64_t ld,
           int64_t groups, int64_t group_stride, int box_rows, int stage_k, bool wide);
bool map_mn(CUtensorMap *m, const void *base, int64_t rows, int64_t cols, int64_t ld,
            int64_t groups, int64_t group_stride, int stage_k, int box_cols, bool wide);
inline bool is_wide(int64_t cols) { return cols % 64 == 0; }
// Of launches of this shape: B's rows a box (A's: 128, or 32 on ONE_32), those of
// W2 in the hidden gradients, and the contraction a stage holds.
int b_box(Epi epi, Tiles tiles);
int dh_box(Tiles tiles);
int stage_k(Epi epi, Tiles tiles);

}  // namespace grp
}  // namespace moe
