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
    const void *ids;      // [T][k], 32 or 64 bits each; a teacher's in ascending order, those < 0 behind
    int ids64, k;
    int64_t V;
    // A teacher's: of each token how many ids lie below each span of 2^shift
    // entries of the vocabulary, [T][spans + 1]; null where k is 1.
    uint16_t *below;
    int shift, spans;
};
// Spans as narrow as the narrowest tile, as long as there are not too many.
constexpr int HEAD_MIN_SHIFT = 7, HEAD_MAX_SPANS = 4096;
inline int head_shift(int64_t V) {
    int s = HEAD_MIN_SHIFT;
    while ((V >> s) >= HEAD_MAX_SPANS) ++s;
    return s;
}
inline int head_spans(int64_t V) { return (int)((V - 1) >> head_shift(V)) + 1; }

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
    float *slots;         // dx: [unit] sums over pieces, in the order of fragments
    int first, last;      // dx: the first piece, the last one
    int pieces, plan_ipt; // dx: of the call; k-tiles of its first piece
    const float *lower;   // the sums' factor, inverse of `raise`
    char *out;
    int64_t ld_out, cols; // columns that exist (p.N may be padded)
    int group_m;
};

enum HeadTileId { HEAD_256 = 0, HEAD_128 = 1, HEAD_64 = 2, HEAD_32 = 3 };
struct HeadTileDim { int bm, bn, per_cu; };
constexpr HeadTileDim kHeadTiles[] = {{256, 256, 1}, {128, 128, 2}, {64, 128, 2}, {32, 128, 2}};

// What a round of the two larger tiles takes, in hundredths of a us, as
// measured on bf16 products of 100 to 4096 rows (1 to 16 rounds, 2 to 64
// k-tiles): a k-tile, what a tile costs beside them (fill, statistics; with an
// output to write), writing a tile's sums to a slot or reading them, and of the
// kernel that adds slots, one of them.
struct HeadTileTime { int k_tile, stats, output, slot, add; };
constexpr HeadTileTime kHeadTimes[] = {{175, 1000, 1500, 500, 7}, {114, 250, 450, 250, 2}};

// What dx takes where s units share each of its tiles along K. A tile's sums
// wait in slots between pieces of the vocabulary, or until they are added.
constexpr int HEAD_CUS = 256;
constexpr uint32_t HEAD_MAX_SPLITS = 32, HEAD_MIN_SHARE = 8;   // units a tile; k-tiles a unit
__host__ __device__ inline uint64_t head_dx_time(int tile, uint32_t tiles, uint32_t s, uint32_t ipt, bool pieces) {
    const HeadTileTime t = kHeadTimes[tile];
    const uint32_t room = (uint32_t)(HEAD_CUS * kHeadTiles[tile].per_cu);
    const uint64_t rounds = (tiles * s + room - 1) / room;
    const uint64_t unit = (uint64_t)t.k_tile * ((ipt + s - 1) / s) + t.output + (pieces ? 2 * t.slot : s > 1 ? t.slot : 0);
    return rounds * unit + (s > 1 ? (uint64_t)tiles * s * t.add + 300 : 0);
}
// Whether a number of units is worth looking at: with four rounds of tiles and
// more the last one matters less than the slots.
__host__ __device__ inline bool head_may_split(int tile, uint32_t tiles, uint32_t s, uint32_t ipt) {
    return s == 1 || (tiles < (uint32_t)(4 * HEAD_CUS * kHeadTiles[tile].per_cu) && s <= HEAD_MAX_SPLITS && s * HEAD_MIN_SHARE <= ipt);
}
// The fastest, the smaller of equals. The device knows how many tiles the rows
// make; the host needs the most units that any number of rows leads to.
inline uint32_t head_splits(int tile, uint32_t tiles, uint32_t ipt, bool pieces) {
    uint32_t best = 1;
    for (uint32_t s = 2; head_may_split(tile, tiles, s, ipt); ++s)
        if (head_dx_time(tile, tiles, s, ipt, pieces) < head_dx_time(tile, tiles, best, ipt, pieces)) best = s;
    return best;
}
// The same by a wave, a number a lane.
__device__ __forceinline__ int head_splits_wave(int tile, uint32_t tiles, uint32_t ipt, bool pieces) {
    const uint32_t s = (threadIdx.x & 63) + 1;
    uint64_t v = ~0ull;
    if (head_may_split(tile, tiles, s, ipt)) v = head_dx_time(tile, tiles, s, ipt, pieces) * 64 + (s - 1);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        const uint64_t w = __shfl_xor((unsigned long long)v, o);
        v = w < v ? w : v;
    }
    return uniform((int)(v & 63)) + 1;
}

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
// lies past the vocabulary). Entries of one id become one; they are sorted by
// id, with -1 for those that do not exist behind. r.below is written.
struct HeadTeacherArgs {
    const int32_t *ids;   // [T][k]
    const void *logits;
    int64_t ld_logits;
    float inv_tau;
    HeadRows r;
    int32_t *out_ids;
    float *weights, *mass;
};
hipError_t launch_head_teacher(int type, const HeadTeacherArgs &a, hipStream_t st);

// Tokens whose rows are counted by a launch before the one that picks them, and
// how many such counts there are (none of few tokens).
constexpr int64_t HEAD_CHUNK = 1024, HEAD_ALONE = 4096;
__host__ __device__ inline int64_t head_counts(int64_t T) { return T <= HEAD_ALONE ? 0 : (T + HEAD_CHUNK - 1) / HEAD_CHUNK; }

struct HeadSelectArgs {
    HeadRows r;           // count and token are written
    int64_t ignore;
    const float *mass;    // teacher: rows whose mass is 0 have nothing to learn
    const float *d_loss;  // backward: nor have rows whose d_loss is 0
    const float *lse;
    float z, grad_scale;
    int below;            // write r.below, of rows
    int fp16;             // of `raise`: the type's range is to be used
    const void *x;        // rows of 16-bit elements, packed into out with zeros behind
    int64_t ldx, H, Hp;
    void *out;
    int *count, *token;
    int *counts;          // [head_counts(T)], null if that is 0
    float2 *largest;      // the same
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
// A wave writes a token's row of `below` from its sorted ids in LDS: a lane
// searches for the first of its spans and walks on from there.
__device__ __forceinline__ void head_below(const HeadRows &r, int64_t t, const int32_t *ids, int lane) {
    const int per = r.spans / 64 + 1, first = lane * per, last = min(first + per, r.spans + 1);
    int lo = 0, hi = first < last ? r.k : 0;   // the first entry that is missing or not below
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        const int32_t id = ids[mid];
        if (id >= 0 && id < (int64_t)first << r.shift) lo = mid + 1;
        else hi = mid;
    }
    for (int g = first; g < last; ++g) {
        for (; lo < r.k; ++lo) {
            const int32_t id = ids[lo];
            if (id < 0 || id >= (int64_t)g << r.shift) break;
        }
        r.below[t * (r.spans + 1) + g] = (uint16_t)lo;
    }
}
__device__ __forceinline__ int head_rows(const int *count, int64_t T) { return uniform(count ? *count : (int)T); }

}  // namespace mg
