// Beam search: selection over beams x vocabulary, and reordering of rows.
#pragma once

#include "kernels.cuh"

namespace rlt {

constexpr int kMaxBeams = 64;

// include/rlt.h: rlt_beam_select
template <typename T>
[[nodiscard]]
cudaError_t launch_beam_select(const T* logits, const float* scores, const uint8_t* finished,
                               int eos, float temperature, int groups, int beams, int vocab,
                               int k, int32_t* parents, int32_t* tokens, float* new_scores,
                               uint8_t* new_finished, cudaStream_t st);

// One buffer whose rows are reordered: `planes` planes per row, and in each the
// bytes of blocks [first, last): block = `unit` bytes, first = start / page,
// last = ceil(len / page), start = from[row] and len = pos[row] where given.
struct ReorderSeg {
    uint8_t* base;
    int64_t row, plane;         // strides in bytes
    int64_t unit;               // bytes of one block
    const int32_t* pos;         // per row lengths on the device, or null
    int64_t start, len;         // the least of from, the largest of pos, where given
    int planes, page;
    const int32_t* from = nullptr;      // per row starts on the device, or null (with page = 1)
};
constexpr int kMaxSegs = 8;
// Rows g*beams + i <- g*beams + parents[g*beams + i], every segment in one launch.
[[nodiscard]]
cudaError_t launch_reorder(const ReorderSeg* segs, int n_segs, const int32_t* parents, int groups,
                           int beams, cudaStream_t st);

}  // namespace rlt
