// Copying, forking, compacting and freeing rows of a state cache:
//
//   cache[l][dst[i]] = what cache[l][src[i]] held before the call (zeros where src[i] < 0)
//
// for every layer l and move i at once, in place: a row may be the source of
// some moves and the target of another, in any order (a compaction, a permutation of
// beams).  Rows are independent along their bytes, so a CTA owns a stripe of all rows: it
// reads the stripe of every source into shared memory, and only then writes the
// targets.  No order among CTAs matters, and every byte is read and written once, which is
// the floor: HBM bandwidth bounds it.
#include <stdio.h>

#include "block_utils.cuh"

namespace {

struct MoveParams {
    char* cache;
    const int *src, *dst;
    int* status;
    long long layers, rows, row_bytes;
    int moves, stripe, stripes;  // bytes of a stripe (a multiple of the unit), stripes a row
};

template <typename U>
__global__ void __launch_bounds__(256) state_move_kernel(const MoveParams p) {
    extern __shared__ __align__(16) char held[];
    const int unit = (int)sizeof(U), per = p.stripe / unit;
    if (blockIdx.x == 0) {
        bool bad = false;
        for (int i = threadIdx.x; i < p.moves; i += 256) bad |= p.src[i] >= p.rows || p.dst[i] >= p.rows;
        if (bad) *p.status = SSCAN_ERR_INVALID;
    }
    for (long long item = blockIdx.x; item < p.layers * p.stripes; item += gridDim.x) {
        const long long layer = item / p.stripes, at = item % p.stripes * p.stripe;
        const long long left = (p.row_bytes - at) / unit;
        const int n = left < per ? (int)left : per;
        char* base = p.cache + layer * p.rows * p.row_bytes + at;
        U* mine = reinterpret_cast<U*>(held);
        __syncthreads();  // the stripe before is written
        for (int i = threadIdx.x; i < p.moves * per; i += 256) {
            const int move = i / per, j = i % per, from = __ldg(p.src + move), to = __ldg(p.dst + move);
            if (j >= n || to < 0 || to >= p.rows) continue;
            U x = {};
            if (from >= 0 && from < p.rows) x = *reinterpret_cast<const U*>(base + from * p.row_bytes + (long long)j * unit);
            mine[i] = x;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < p.moves * per; i += 256) {
            const int move = i / per, j = i % per, from = __ldg(p.src + move), to = __ldg(p.dst + move);
            if (j >= n || to < 0 || to >= p.rows || from >= p.rows) continue;
            *reinterpret_cast<U*>(base + to * p.row_bytes + (long long)j * unit) = mine[i];
        }
    }
}

template <typename U>
cudaError_t run(MoveParams& p, cudaStream_t st) {
    const int unit = (int)sizeof(U);
    // whole lines where they fit
    long long stripe = (long long)(96 * 1024) / p.moves / unit * unit;
    if (stripe < unit) stripe = unit;
    if (stripe > 512) stripe = 512;
    if (stripe > p.row_bytes) stripe = p.row_bytes;
    p.stripe = (int)stripe;
    p.stripes = (int)sscan::div_up(p.row_bytes, stripe);
    const size_t smem = (size_t)p.moves * stripe;
    const cudaError_t e = cudaFuncSetAttribute(state_move_kernel<U>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const long long items = p.layers * p.stripes;
    return sscan::launch(state_move_kernel<U>, dim3((unsigned)(items < (1 << 20) ? items : (1 << 20))), dim3(256), smem, st, false, p);
}

}  // namespace

extern "C" int state_move(void* cache, const int32_t* src, const int32_t* dst, int64_t moves, int64_t layers, int64_t rows,
                          int64_t row_bytes, void* stream) {
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    sscan::record_call(0, st, "rejected");
    const long long lim = 1LL << 30;
    if (moves < 0 || moves > STATE_MOVE_MAX || layers < 0 || layers > lim || rows < 0 || rows > lim || row_bytes < 0 || row_bytes > (1LL << 34) ||
        (layers && rows && row_bytes && (rows > (1LL << 44) / layers || row_bytes > (1LL << 44) / (layers * rows))))
        return SSCAN_ERR_INVALID;
    if (moves == 0 || layers == 0 || rows == 0 || row_bytes == 0) {
        sscan::record_call(0, st, "empty");
        return SSCAN_OK;
    }
    if (!cache || !src || !dst) return SSCAN_ERR_INVALID;
    int* status = sscan::device_status_word();
    if (status == nullptr) return sscan::finish(cudaErrorUnknown);
    MoveParams p = {};
    p.cache = static_cast<char*>(cache); p.src = src; p.dst = dst; p.status = status;
    p.layers = layers; p.rows = rows; p.row_bytes = row_bytes; p.moves = (int)moves;
    sscan::record_call(1, st, "state move");
    if (row_bytes % 16 == 0 && sscan::is_aligned(cache, 16)) return sscan::finish(run<uint4>(p, st));
    if (row_bytes % 4 == 0 && sscan::is_aligned(cache, 4)) return sscan::finish(run<unsigned>(p, st));
    if (row_bytes % 2 == 0 && sscan::is_aligned(cache, 2)) return sscan::finish(run<unsigned short>(p, st));
    return sscan::finish(run<unsigned char>(p, st));
}
