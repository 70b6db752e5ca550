// head.hpp -- arguments and launchers of the output head's losses (declared for
// model_api.cpp, which validates, and for the kernels).
//
// A head's logits l = scale * x W^T are never written. Every kernel works on
// rows: the tokens that have something to learn, in order, so that tokens
// without a label cost nothing and whatever lies in them reaches no sum.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm_core.hpp"

namespace mg {

// What a call's tokens ask for: k entries each of the vocabulary (a label, or
// a teacher's choices).
struct HeadRows {
    int64_t T;            // tokens
    const int *count;     // rows, on the device; null: every token is a row
    const int *token;     // the token of each row; null: itself
    const void *ids;      // [T][k], 32 or 64 bits each
    int ids64, k;
    int64_t V;
};

// One product of x's rows with `p.N` rows of W from entry v0 on.
struct HeadTileArgs {
    ProbLd p;             // A: x, B: W's piece, K: their width
    HeadRows r;
    int64_t v0;
    float scale;
    int group_m;
    // forward: of each row and each tile of the vocabulary the largest l and
    // the sum of exp(l - that), base 2; the logits of the row's own entries
    float2 *parts;        // [tiles of the vocabulary][T]
    float *picked;        // [T][k]
    // backward: the gradient of the logits, d_loss * grad_scale *
    // ((mass + 2 z lse) softmax(l) - weight of the entry) * *raise, in the type
    const float *lse, *mass, *weights, *d_loss, *raise;
    float z, grad_scale;
    char *grad;           // [rows][ld_grad]
    int64_t ld_grad;
};

// dx (rows of tokens) or dw (rows of W) from the gradient of the logits.
struct HeadOutArgs {
    ProbLd p;             // M or K is the count of rows where `count` is given
    const int *count;
    const int *token;     // dx: the token of each row
    int splits;           // dx: units that share a tile's K, each with a slot of its own
    float *slots;         // dx: [tile][split] partial sums over pieces, fragment order
    int first, last;      // dx: no sums yet; this call's units finish their tile
    const float *lower;   // the sums' factor, inverse of `raise`
    char *out;
    int64_t ld_out, cols; // columns that exist (p.N may be padded)
    int group_m;
};

enum HeadTileId { HEAD_256 = 0, HEAD_128 = 1, HEAD_64 = 2, HEAD_32 = 3 };
struct HeadTileDim { int bm, bn, per_cu; };
constexpr HeadTileDim kHeadTiles[] = {{256, 256, 1}, {128, 128, 2}, {64, 128, 2}, {32, 128, 2}};

// Per type (kernels_head_f16.hip, kernels_head_bf16.hip). stats and grad: any
// tile; dx and dw: HEAD_256 or HEAD_128.
struct HeadLaunch {
    hipError_t (*stats)(int tile, const HeadTileArgs &a, int grid, hipStream_t st);
    hipError_t (*grad)(int tile, const HeadTileArgs &a, int grid, hipStream_t st);
    hipError_t (*dx)(int tile, const HeadOutArgs &a, int grid, hipStream_t st);
    hipError_t (*dx_finish)(int tile, const HeadOutArgs &a, int grid, hipStream_t st);
    hipError_t (*dw)(int tile, const HeadOutArgs &a, int grid, hipStream_t st);
};
const HeadLaunch &head_launch_f16();
const HeadLaunch &head_launch_bf16();

// The kernels around the products (kernels_head.hip).

// Rows of 16-bit elements, padded with zeros: out[i][0 .. ld_out).
hipError_t launch_head_pad(const void *src, int64_t ld, int64_t rows, int64_t cols, void *out, int64_t ld_out,
                           hipStream_t st);

// A teacher's entries: ids [T][k] and logits of any float type, to weights that
// sum to 1 (mass 1; 0 and no weights where a token has no entry, NaN where an id
// lies past the vocabulary). Entries of one id become one; merged ids are -1.
hipError_t launch_head_teacher(const int32_t *ids, const void *logits, int type, int64_t ld_logits, float inv_tau,
                               int64_t T, int k, int64_t V, int32_t *out_ids, float *weights, float *mass,
                               hipStream_t st);

struct HeadSelectArgs {
    HeadRows r;           // count and token are written
    int64_t ignore;
    const float *mass;    // teacher: rows whose mass is 0 have nothing to learn
    const float *d_loss;  // backward: nor have rows whose d_loss is 0
    const float *lse;
    float z, grad_scale;
    int fp16;             // of `raise`: the type's range is to be used
    const void *x;        // rows of 16-bit elements, packed into out with zeros behind
    int64_t ldx, H, Hp;
    void *out;
    int *count, *token;
    float *raise;         // {raise, its inverse}
    // rows with nothing to learn
    float *loss, *lse_out, *picked;   // forward: 0
    void *dx;             // backward: 0, packed [T][H]
};
hipError_t launch_head_select(const HeadSelectArgs &a, hipStream_t st);

struct HeadJoinArgs {
    HeadRows r;
    int64_t ignore;
    int tiles;
    const float2 *parts;
    const float *weights, *mass;   // teacher
    float *picked;
    float z, tau2;
    float *loss, *lse;
};
hipError_t launch_head_join(const HeadJoinArgs &a, hipStream_t st);

__device__ __forceinline__ int64_t head_id(const HeadRows &r, int64_t e) {
    return r.ids64 ? static_cast<const int64_t *>(r.ids)[e] : static_cast<const int32_t *>(r.ids)[e];
}
__device__ __forceinline__ int head_rows(const int *count, int64_t T) { return uniform(count ? *count : (int)T); }

}  // namespace mg
