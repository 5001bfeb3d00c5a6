// The packed scan's kernels for fp32 rows, whole 16-byte vectors (one
// translation unit a form, so that they compile in parallel).
#include "sscan_prompt_kernel.cuh"

namespace sscan {
template cudaError_t prompt_launch<float, true>(const PromptParams&, cudaStream_t);
}  // namespace sscan
