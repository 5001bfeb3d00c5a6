// Launches of the linear attention kernels on the FP32 units (lattn_simt.cuh).
#include "lattn_simt.cuh"

namespace sscan {
namespace {

template <typename K>
cudaError_t with_smem(K kernel, size_t bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <typename T, int KD, int MODE>
cudaError_t walk(const LattnParams& p, int pieces, bool after, cudaStream_t st) {
    const size_t smem = sizeof(float) * (KD * kLdv + 64 * (KD + 4) + 2 * 64 * kLdv + (MODE == WALK_OUT ? 2 * KD * kLdv : 0));
    const cudaError_t e = with_smem(lattn_walk<T, KD, MODE>, smem);
    if (e != cudaSuccess) return e;
    return launch(lattn_walk<T, KD, MODE>, dim3((unsigned)(p.heads * p.vtiles), (unsigned)pieces, (unsigned)p.batch), dim3(256), smem, st, after, p);
}
// (after: not the first kernel of its call, which begins while the one before it ends)
template <typename T, int KD>
cudaError_t walk_all(const LattnParams& p, cudaStream_t st) {
    cudaError_t e = cudaSuccess;
    if (p.pieces > 1) e = walk<T, KD, WALK_ENDS>(p, p.pieces - 1, p.apart, st);
    return e != cudaSuccess ? e : walk<T, KD, WALK_OUT>(p, p.pieces, p.apart || p.pieces > 1, st);
}
template <typename T>
cudaError_t walk_keys(const LattnParams& p, cudaStream_t st) {
    return p.N <= 64 ? walk_all<T, 64>(p, st) : walk_all<T, 128>(p, st);
}

template <typename T, int KD, bool STEPS>
cudaError_t grad(const LattnParams& p, cudaStream_t st) {
    const size_t smem = sizeof(float) * (2 * KD * kLd + 4 * 64 * kLd + 2 * 64 * (KD + 1));
    const cudaError_t e = with_smem(lattn_grad<T, KD, STEPS>, smem);
    if (e != cudaSuccess) return e;
    return launch(lattn_grad<T, KD, STEPS>, dim3((unsigned)p.chunks, (unsigned)(p.groups * p.subsets), (unsigned)p.batch), dim3(256), smem, st, true, p);
}

template <typename T, int KD>
cudaError_t grad_all(const LattnParams& p, cudaStream_t st) {
    constexpr bool FEW = sizeof(T) == 2;  // bf16 has one chunk at most
    cudaError_t e = cudaSuccess;
    if constexpr (!FEW)
        if (p.pieces > 1) e = walk<T, KD, WALK_ENDS>(p, p.pieces - 1, false, st);
    if (e == cudaSuccess) e = walk<T, KD, WALK_STATES>(p, p.pieces, p.pieces > 1, st);
    if constexpr (!FEW)
        if (e == cudaSuccess && p.pieces > 1) e = walk<T, KD, WALK_DENDS>(p, p.pieces - 1, true, st);
    if (e == cudaSuccess) e = walk<T, KD, WALK_DSTATES>(p, p.pieces, true, st);
    if (e != cudaSuccess) return e;
    return p.delta != nullptr ? grad<T, KD, true>(p, st) : grad<T, KD, false>(p, st);
}
template <typename T>
cudaError_t grad_keys(const LattnParams& p, cudaStream_t st) {
    return p.N <= 64 ? grad_all<T, 64>(p, st) : grad_all<T, 128>(p, st);
}

}  // namespace

cudaError_t lattn_walk_launch(const LattnParams& p, cudaStream_t st) {
    return walk_keys<float>(p, st);
}
cudaError_t lattn_grad_launch(const LattnParams& p, int dtype, cudaStream_t st) {
    return dtype == SSCAN_F32 ? grad_keys<float>(p, st) : grad_keys<bf16>(p, st);
}
cudaError_t lattn_parts_launch(const LattnParams& p, int dtype, cudaStream_t st) {
    const long long n = (long long)p.batch * p.groups * p.N * p.L, ctas = div_up(2 * n, 256);
    const dim3 grid((unsigned)(ctas < 4096 ? ctas : 4096));
    if (dtype == SSCAN_F32)
        return launch(lattn_add_parts<float>, grid, dim3(256), 0, st, true, p.dq_part, p.dk_part, static_cast<float*>(p.dq),
                      static_cast<float*>(p.dk), n, p.subsets);
    return launch(lattn_add_parts<bf16>, grid, dim3(256), 0, st, true, p.dq_part, p.dk_part, static_cast<bf16*>(p.dq),
                  static_cast<bf16*>(p.dk), n, p.subsets);
}
cudaError_t lattn_heads_launch(const LattnParams& p, float* dA, float* dbias, float* dD, cudaStream_t st) {
    return launch(lattn_add_heads, dim3((unsigned)p.heads, 3), dim3(256), 0, st, true, p.head_part, dA, dbias, dD, p.heads,
                  (long long)p.batch * p.chunks);
}

}  // namespace sscan
