// expert.hpp -- launchers of the expert order's operators (declared for
// model_api.cpp, which validates).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mg {

// How a list of slots is cut for sorting: parts of `chunk` slots, a workgroup
// each. One part is counted and placed by one launch, more by two: 4096 slots of
// 64 experts 6.1 us or 2.3 + 4.5 and a launch between, 8192 9.3 or 2.3 + 4.9, 16384
// 16.1 or 2.3 + 4.9 (parts of 4096: 2.9 + 7.0), 65536 55 or 2.3 + 5.8 (2.9 + 7.8).
struct ExpertCut {
    int64_t chunk, parts;
};
constexpr int64_t EXPERT_ONE = 4096, EXPERT_CHUNK = 1024, EXPERT_PARTS = 256;
inline ExpertCut expert_cut(int64_t slots) {
    int64_t chunk = EXPERT_CHUNK;
    if (slots <= EXPERT_ONE) chunk = slots > 0 ? slots : 1;
    else if (slots > chunk * EXPERT_PARTS) chunk = (slots + EXPERT_PARTS - 1) / EXPERT_PARTS;
    chunk = (chunk + 1023) / 1024 * 1024;   // whole waves' runs of 64
    return {chunk, slots > 0 ? (slots + chunk - 1) / chunk : 1};
}

struct ExpertSortArgs {
    const void *ids;     // [slots], 32 or 64 bits each
    int ids64;
    int64_t slots, chunk;
    int experts, parts, bits;   // bits of the largest expert
    int *counts;         // [parts][experts], where there is more than one part
    int32_t *offsets, *row_of;
};
hipError_t launch_expert_sort(const ExpertSortArgs &a, hipStream_t st);

struct ExpertRowsArgs {
    int64_t tokens, cols;
    int top_k, experts;
    const int32_t *offsets, *row_of;
    const void *x;       // [tokens]: gather's input, the gradient of combine's output
    void *out;           // [tokens]: combine's output
    const void *rows;    // [tokens * top_k]: combine's input
    void *rows_out;      // [tokens * top_k]: gather's output, the gradient of combine's input
    int64_t ld_x, ld_out, ld_rows, ld_rows_out;
    const float *weights;
    float *d_weights;
};
hipError_t launch_expert_gather(int type, const ExpertRowsArgs &a, hipStream_t st);
hipError_t launch_expert_combine(int type, const ExpertRowsArgs &a, hipStream_t st);
hipError_t launch_expert_combine_backward(int type, const ExpertRowsArgs &a, hipStream_t st);

}  // namespace mg
