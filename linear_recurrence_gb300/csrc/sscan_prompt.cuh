// Parameters and launches of the packed selective scan, shared by its kernels
// (sscan_prompt_kernel.cuh) and the entry point (sscan_prompt.cu).
#pragma once

#include "block_utils.cuh"

namespace sscan {

constexpr int kPromptTile = 16;           // tokens staged at a time (32 in the scan's direct form)
constexpr int kSegStep = 16;              // segments are whole tiles of 16
constexpr float kCutBits = 26.f;          // a border leaves out what decayed below 2^-26: a quarter of an fp32 rounding of what entered
constexpr int kPromptWarps = 4;           // warps of a scan CTA
constexpr int kEndStates = 4;             // states whose end values a warp finds together

struct PromptParams {
    const void* u;
    const void* delta;
    const float* A;
    const void* B;
    const void* C;
    const float* D;
    const void* z;
    const float* bias;
    float* state;
    void* out;
    long long dim;
    int tokens, N;
    int seg_tokens, segments;
    int softplus;
    bool narrow;  // four states of one channel a thread
    // scratch of a split: per segment, the end state [dim, N], the carried-in
    // request's saved initial state [dim, N], and sum of dt [dim, groups of 4 states],
    // infinite where the group's states had decayed before the segment's start
    float* h_end;
    float* h_first;
    float* dt_sum;
    Requests req;
};

// Both passes of a call for rows of T, whole 16-byte vectors (ALIGNED) or not.
template <typename T, bool ALIGNED>
cudaError_t prompt_launch(const PromptParams& p, cudaStream_t st);
extern template cudaError_t prompt_launch<float, true>(const PromptParams&, cudaStream_t);
extern template cudaError_t prompt_launch<float, false>(const PromptParams&, cudaStream_t);
extern template cudaError_t prompt_launch<bf16, true>(const PromptParams&, cudaStream_t);
extern template cudaError_t prompt_launch<bf16, false>(const PromptParams&, cudaStream_t);

}  // namespace sscan
