// loss_products.h -- the matrix products of the output-layer losses
// (loss_products.cu), as output_loss.cu launches them.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "chain.h"

namespace txl {

// One call's rows, as the kernels see them.
struct LossRows {
    const int64_t *target;     // cross entropy: the rows' own column, of weight 1; else NULL and
    int *col;                  // [rows][K] listed columns: those of even 64-column chunks of the vocabulary
                               // ascending, then those of odd ones, then kNoColumn
    int *even;                 // [rows] how many of the former
    float *p;                  // [rows][K] their weights
    float *ent;                // [rows] sum_k p log p
    int K, vocab;
    float t;                   // temperature
    const float *lse, *dloss;  // [rows] (backward)
};
constexpr int kNoColumn = INT32_MAX;   // an invalid list entry: sorts behind every column
constexpr float kLn2 = 0.693147180559945309f;
__device__ __forceinline__ int target_column(const LossRows &r, long i)
{
    const int64_t y = r.target[i];
    return y >= 0 && y < r.vocab ? (int)y : kNoColumn;
}
// t * dloss; 0 for a row without a valid entry (`any`) or a finite logit
__device__ __forceinline__ float row_factor(const LossRows &r, long i, bool any)
{
    return any && r.lse[i] != -INFINITY ? r.t * r.dloss[i] : 0.f;
}

// A row's loss and lse by the lanes of a warp, from its sum l of 2^(y - ref)
// over the vocabulary and y at its listed columns.
__device__ __forceinline__ void row_loss(const LossRows &r, const float *ysel, float ref, float l, float t2, long row, int lane,
                                         float *loss, float *lse)
{
    const float y_lse = ref + log2f(l);
    float dot = 0.f;
    int any = 0;
    if (r.target) {
        any = target_column(r, row) != kNoColumn;
        if (any && lane == 0) dot = y_lse - __ldcg(ysel + row);
    } else {
        for (int k = lane; k < r.K; k += 32) {
            if (r.col[row * r.K + k] == kNoColumn) continue;
            any = 1;
            const float p = r.p[row * r.K + k];
            if (p != 0.f) dot += p * (y_lse - __ldcg(ysel + row * r.K + k));
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        dot += __shfl_xor_sync(0xffffffffu, dot, o);
        any |= __shfl_xor_sync(0xffffffffu, any, o);
    }
    if (lane == 0) {
        lse[row] = y_lse * kLn2;
        loss[row] = any && y_lse != -INFINITY ? t2 * ((r.target ? 0.f : r.ent[row]) + kLn2 * dot) : 0.f;
    }
}

// A bf16 matrix in device memory, [pieces][rows][cols] with `pitch` elements
// between rows (a multiple of 8, 16-byte aligned base).  One piece holds
// bf16 values; three hold fp32 values as the exact sum of their pieces.
struct LossMatrix {
    const void *base;
    long pitch, piece_stride;
    int rows, cols, pieces;
};

// How a launch divides its work (from sizes and the number of SMs alone).
struct LossTiling {
    int cg;             // CTAs per tile: 2 for more than 128 rows, else 1
    int bn;             // output columns per tile
    int tiles_m, tiles_n;
    int strip;          // vocabulary passes: tiles of one row block that a CTA (pair) does in a row
    int splits;         // gradients: parts of the long axis, each into a slot of its own
    bool turned;        // dh: computed as W^T dz^T
    bool first;         // gradients: dealt out before the other (the longer items)
    int ahead;          // ... items of the other that go to the CTAs without a last item of this one
};

// Vocabulary pass over rows x cols logits; *us its estimated time.
LossTiling vocab_tiling(int rows, int cols, int d, int parts, double *us = nullptr);
inline int vocab_strips(const LossTiling &t) { return (t.tiles_n + t.strip - 1) / t.strip; }
constexpr int kSlotsPerStrip = 2;      // the halves of a tile's columns are kept apart

// The launch that makes dh += dz W and dW = dz^T h of one vocabulary piece of
// `cols` columns (`whole`: the columns of the call's other pieces, whose dh
// slots it adds to with dh_slots); returns its estimated time in us.
// dh_splits fixes dh's splits (0: free).
double gradient_tiling(int rows, int d, int cols, int whole, int parts, bool dh_slots, int dh_splits, LossTiling *dh,
                       LossTiling *dw);
// The bf16 parts that dz is kept in.  For many bf16 rows one: a product's error
// from dz's rounding averages out over the rows to that of its own rounding.
// Few rows leave some elements with hardly more than one rounding, so up to
// 128 keep what it takes off as a second part (dW of 8 rows 2.6e-3 off in the
// mean with one part, 1.7e-3 with two and as rounded from the exact one).
// The products take these parts as further rows of dz (dz_rows() in all).
// 128 x 768 x 90326 tokens, both directions: 156 us, with one part 138.
inline int dz_parts(int rows, int parts) { return parts == 3 ? 3 : rows > 128 ? 1 : 2; }
inline int dz_rows(int rows, int parts) { return parts == 3 ? rows : rows * dz_parts(rows, parts); }
// Columns of the backward's vocabulary pieces: at most `most`, a multiple of
// kLossPieceUnit unless it is the whole vocabulary.
constexpr int kLossPieceUnit = 256;
int gradient_piece(int rows, int d, int vocab, int parts, int most);

// part[2 * strip + half][row] = (maximum, sum of 2^(y - maximum)) over the
// columns, y = alpha (h . w + bias); ysel[row][k] = y at the listed columns
// (vocabulary column = v0 + column of w).  bias: of w's columns, 16-byte
// aligned, or NULL.  With loss and lse (cross entropy whose vocabulary is one
// strip) the rows' results are written instead of part.
cudaError_t launch_loss_lse(const LossMatrix &h, const LossMatrix &w, const float *bias, int v0, float alpha,
                            const LossRows &r, float *ysel, float2 *part, float *loss, float *lse, const LossTiling &t, cudaStream_t s);

// dz = coef (2^(y - l2) - listed weights), in dz's pieces; dbpart[row / 32][column]
// (pitch dz.pitch) the columns' sums over 32 rows each, when given.
cudaError_t launch_loss_dz(const LossMatrix &h, const LossMatrix &w, const float *bias, int v0, float alpha,
                           const LossRows &r, const LossMatrix &dz, float *dbpart, const LossTiling &t,
                           cudaStream_t s);

// out(m, n) = sum_k a(m, k) b(k, n).  a is stored [m][k], or [k][m] with
// a_t; b is stored [k][n], or [n][k] with b_t; out [m][n], or [n][m] with
// out_t.  f32 selects fp32 output; it then has `splits` slots of slot_stride
// elements (the sum of which is the product), added to what they hold with
// `add`.  One or two of them per launch, with one cg.
struct LossOutput {
    void *base;
    long pitch, slot_stride;
    bool f32, add;
    bool tma;           // rows that TMA stores can address (slots are); else elements are stored one or two at a time
};
struct LossContraction {
    LossMatrix a, b;
    bool a_t, b_t, out_t;
    int m, n, k;
    LossOutput out;
    LossTiling t;
};
cudaError_t launch_loss_gradients(const LossContraction *jobs, int n, int parts, cudaStream_t s);

// The losses of a handful of rows on the CUDA cores (loss_few.cu), where the
// tensor-core kernel would need a copy of the weights.
constexpr int kFewColumns = 1024;   // widest d_model
struct FewShape {
    int tok, slots;    // tokens per chunk, chunks in the ring
    int per, blocks;   // tokens per block
    int groups;        // of threads that take a chunk's tokens in turn (backward)
    bool joined;       // forward: the blocks are a cluster, which writes losses
};
// false: sizes for the tensor-core kernel.  w_ok: w is 16-byte aligned.
bool few_shape(int rows, int d, int vocab, bool f32, bool w_ok, bool backward, FewShape *s);
struct FewCall {
    const void *h, *w;
    const float *bias;
    LossRows r;
    int rows, d, vocab;
    FewShape s;
    bool f32, backward;
    float alpha;
    float *ysel;         // forward: as launch_loss_lse
    float2 *part;        // ... [blocks][rows]
    float t2, *loss, *lse_out; // ... of a joined shape
    void *dh, *dw;       // backward; each and db may be NULL
    float *db, *dh_part; // dh_part: [blocks * groups][rows][d]
};
cudaError_t launch_loss_few(const FewCall &a, cudaStream_t s);
// error words of loss_few.cu and loss_products.cu (*word stays as it is before the first launch)
cudaError_t read_and_clear_few_error(unsigned int *word, cudaStream_t s);
cudaError_t read_and_clear_loss_error(unsigned int *word, cudaStream_t s);

}  // namespace txl
