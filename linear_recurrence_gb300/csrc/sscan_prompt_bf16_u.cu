// The packed scan's kernels for bf16 rows, any alignment (one
// translation unit a form, so that they compile in parallel).
#include "sscan_prompt_kernel.cuh"

namespace sscan {
template cudaError_t prompt_launch<bf16, false>(const PromptParams&, cudaStream_t);
}  // namespace sscan
