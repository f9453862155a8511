// The dense feed-forward operators' internal interface: dense.cpp checks a
// call and describes its matrix products, the k_dense*.hip launchers run them.
#pragma once

#include "arg_checks.h"
#include "ecf_internal.h"

namespace ecf {

// One matrix product with its epilogue:
//   acc_g[m][n] = sum_s sum_k A_s(m, k) B(n, k),  s < ksegs, k < K
// A_s(m, k) is a[s][m * lda + k], or a[s][k * lda + m] with a_t; B likewise.
//  - gated:       b[0] and b[1] give two sums over the one A; the epilogue joins them
//  - ksegs == 2:  a[0] . b[0] + a[1] . b[1], both K long
//  - mhalves == 2: a[h] gives out[h], h = 0, 1 (two products that share B)
// At most one of the three holds.
struct DenseGemm {
    int dtype;  // of A, B, bias and saved pre-activations: ECF_F32, ECF_BF16 or ECF_F16
    bool a_t, b_t;
    const void *a[2], *b[2];
    int64_t lda, ldb;
    bool a_padded;  // rows of A go on with zeros to the next multiple of 8 elements
    int M, N, K;
    int ksegs, mhalves;
    bool gated;
    // epilogue: z = acc + bias; save <- z; out = act(z) + res, gated: act(z_0) * z_1
    int act, out_dtype;
    const void *bias[2];
    const void *res;  // in out_dtype; not gated
    int64_t ldres;
    void *out[2];
    int64_t ldout;
    void *save[2];
    int64_t ldsave;
    // backward products in fp16: what undoes the scale of A (see DenseGrad), a power of
    // two per row of the output, [half][M]; null: none
    const float *unscale;
    bool stream_out;  // set by the launcher: the output does not fit the caches
};
// ws: `room` bytes for the partial sums of a split K (may be null where that is 0); a
// plan that needs more is not taken
int launch_dense_gemm(const DenseGemm &g, void *ws, size_t room, hipStream_t st);
// Column sums still to be joined over the row blocks of launch_dense_grad: fp32
// partial [row_blocks][n I], the first I columns into out[0], the others into out[1]
// (each may be null).  A block takes 64 columns.
struct DenseColsum {
    const float *partial;
    int row_blocks, I, n, out_dtype;
    void *out[2];
    int blocks;  // 0: nothing to join
};
// The products of a backward pass, dx (n-contiguous B) and dW (m- and n-contiguous;
// either may be null), and the column sums, in one launch or more.
int launch_dense_backward(const DenseGemm *gx, const DenseGemm *gw, const DenseColsum &sums, void *ws, size_t room,
                          hipStream_t st);

// ---- which kernel a product takes (dense_plan.cpp) ----------------------------------

// A product in tiles: the tile, the splits of K, and whether operands can go straight
// to LDS.
struct DensePlan {
    int tile;  // index into the launcher's tiles
    int splits;
    bool dma;
};
struct DenseTile {
    int bm, bn;
};
DenseTile dense_tile(int dtype, bool dma, int tile);
// x W^T of at most kFewTokens rows as a stream of the weights (k_dense_few.hip): weight
// rows per block, groups of as many tokens (1, 2 or 4), waves per block.  It needs no
// workspace.  Up to kAlwaysFew rows of kAlwaysFewX elements together it is the faster
// way, unless 16-bit rows start at odd elements; elsewhere the estimates decide (16
// tokens, 2 x 1024 rows in bf16: streamed and in tiles 9.2 and 10.6 us of K 4096, 15.5
// and 13.1 of K 8192, whose x every block reads).
struct DenseFew {
    int rows, groups, waves;
};
constexpr int kFewTokens = 64, kAlwaysFew = 16;
constexpr int64_t kAlwaysFewX = 1 << 17;
bool few_needs_no_room(int64_t T, int64_t in);
constexpr int kFewWaves = 8;              // most waves per block
struct DenseChoice {
    enum Kind { kFew, kShort, kTiles } kind;
    DensePlan tiles;
    DenseFew few;
};
// room: bytes of workspace for partial sums, dense_partials of which the choice needs
size_t dense_partials(const DenseGemm &g, int splits);
DenseChoice choose_gemm(const DenseGemm &g, int cus, size_t room);
// Both products of a backward pass in one launch, where that is the faster way.
struct DensePair {
    DensePlan x;
    int splits_w;
    size_t at_w;  // dW's partial sums lie this far behind dx's
};
bool choose_pair(const DenseGemm &gx, const DenseGemm &gw, int cus, size_t room, DensePair *out);

int launch_dense_few(const DenseGemm &g, const DenseFew &f, hipStream_t st);
// The most workspace that any plan of a product with M x N outputs in each plane over
// K (ksegs times) asks for: fp32 sums of its splits, 0 where K is too short to split.
constexpr size_t kDensePartialBytes = (size_t)32 << 20;
size_t dense_gemm_ws(int64_t M, int64_t N, int64_t K, int ksegs, int planes);

// dz rows of the backward passes, in the operands' type: dz[t][i] (linear), or
// da = dz[t][i] and db = dz[T + t][i] (gated).  Columns from I to the pitch, the next
// multiple of 8, are zeroed.  With sums, the columns are added up:
// into `sums` where one row block covers all tokens, else per row block into
// partial [block][1 or 2][I], and `left` says what is still to be joined.
struct DenseGrad {
    int dtype, dout_dtype, act;
    bool gated;
    const void *dout, *a, *b;  // linear: a = z (null when act is none)
    int64_t lddout, ldab;
    int T, I;
    void *dz;  // null: column sums only
    int64_t pitch;
    bool want_sums;
    void *sums[2];  // each may be null
    int sums_dtype;
    float *partial;
    // fp16: da, db and dz may lie outside the type's range although the products made
    // of them do not (an fp32 dy of 1e-9 or 1e6; a dh b over 65504).  With `scaled` they
    // are held twice, times powers of two: `dz`, of which dx is made, row by row (da and
    // db of a token together), `dz_w`, of which dW is made, column by column (either may
    // be null: not wanted).  The power puts the largest finite value of the row (column)
    // at 2^14 to 2^15.  Values within 2^-28 of that one keep all their bits, what is below
    // 2^-39 of it is lost, and no row of dx or dW hangs on the gradients of another.
    // (A linear dz of an fp16 dy leaves the range by slopes of up to 1.13 only, but half
    // of it, which needs no pass, is one bit short in the subnormals.)
    bool scaled;
    void *dz_w;
    uint32_t *row_tops, *col_tops;    // the largest of each tile: [column block][T], [row block][1 or 2][I]
    float *row_inverse, *col_inverse; // the inverse powers: [T], [1 or 2][I]
};
// column blocks of any call
int64_t dense_grad_col_blocks(int64_t I);
// the most row blocks of any call with up to T tokens
int64_t dense_grad_max_row_blocks(int64_t T);
int launch_dense_grad(const DenseGrad &g, DenseColsum *left, hipStream_t st);

}  // namespace ecf
