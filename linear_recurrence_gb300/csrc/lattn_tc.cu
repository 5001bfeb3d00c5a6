// Launches of the linear attention kernels on the tensor cores (lattn_tc.cuh).
#include "lattn_tc.cuh"

namespace sscan {
namespace {

template <int KD, int MODE>
cudaError_t walk(const LattnParams& p, int pieces, cudaStream_t st) {
    constexpr unsigned bytes = MODE == WALK_OUT ? TcWalkSmem<KD>::bytes : TcWalkSmem<KD>::few_bytes;
    const cudaError_t e = cudaFuncSetAttribute(lattn_tc_walk<KD, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    return launch(lattn_tc_walk<KD, MODE>, dim3((unsigned)(p.heads * p.vtiles), (unsigned)pieces, (unsigned)p.batch), dim3(kTcThreads), bytes,
                  st, false, p);
}
template <int KD>
cudaError_t walk_all(const LattnParams& p, cudaStream_t st) {
    cudaError_t e = cudaSuccess;
    if (p.pieces > 1) e = walk<KD, WALK_ENDS>(p, p.pieces - 1, st);
    return e != cudaSuccess ? e : walk<KD, WALK_OUT>(p, p.pieces, st);
}

}  // namespace

cudaError_t lattn_tc_walk_launch(const LattnParams& p, cudaStream_t st) {
    return p.N <= 64 ? walk_all<64>(p, st) : walk_all<128>(p, st);
}

}  // namespace sscan
