// Copying, forking, compacting and freeing rows of a state cache:
//
//   cache[l][dst[i]] = what cache[l][src[i]] held before the call (zeros where src[i] < 0)
//
// for every layer l and move i at once, in place: a row may be the source of
// some moves and the target of another, in any order (a compaction, a permutation of
// beams).  Rows are independent along their bytes, so a CTA owns a stripe of all rows: it
// reads the stripe of every source into shared memory, and only then writes the
// targets.  No order among CTAs matters, and every byte is read and written once, which is
// the floor: HBM bandwidth bounds it.  Rows of whole 16-byte vectors go by bulk copies in both directions,
// all of a stripe's on the way at once (160 moves of 2.6 MB rows in two layers: 229 us, by
// loads and stores of threads 580; the floor is 251); others by threads.
#include <stdio.h>

#include "block_utils.cuh"
#include "tc_utils.cuh"

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

__global__ void __launch_bounds__(128) state_move_bulk(const MoveParams p) {
    extern __shared__ __align__(128) char held[];  // a stripe of zeros, then one a move
    __shared__ uint64_t bar;
    if (blockIdx.x == 0) {
        bool bad = false;
        for (int i = threadIdx.x; i < p.moves; i += 128) bad |= p.src[i] >= p.rows || p.dst[i] >= p.rows;
        if (bad) *p.status = SSCAN_ERR_INVALID;
    }
    const long long layer = blockIdx.x / p.stripes, at = blockIdx.x % p.stripes * (long long)p.stripe;
    const unsigned bytes = (unsigned)(p.row_bytes - at < p.stripe ? p.row_bytes - at : p.stripe);
    char* base = p.cache + layer * p.rows * p.row_bytes + at;
    if (threadIdx.x == 0) {
        sscan::mbar_init(&bar, 128);
        sscan::mbar_fence_init();
    }
    for (int i = threadIdx.x; i < p.stripe / 16; i += 128) reinterpret_cast<uint4*>(held)[i] = make_uint4(0u, 0u, 0u, 0u);
    sscan::fence_proxy_async_smem();
    __syncthreads();
    unsigned mine = 0;
    for (int i = threadIdx.x; i < p.moves; i += 128) {
        const int from = __ldg(p.src + i), to = __ldg(p.dst + i);
        if (to >= 0 && to < p.rows && from >= 0 && from < p.rows) mine += bytes;
    }
    sscan::mbar_arrive_expect_tx(&bar, mine);
    for (int i = threadIdx.x; i < p.moves; i += 128) {
        const int from = __ldg(p.src + i), to = __ldg(p.dst + i);
        if (to >= 0 && to < p.rows && from >= 0 && from < p.rows)
            sscan::bulk_load(held + (long long)(i + 1) * p.stripe, base + from * p.row_bytes, bytes, &bar);
    }
    // nothing is written before everything is read
    if (!sscan::mbar_wait_bounded(&bar, 0)) {
        *p.status = SSCAN_ERR_TIMEOUT;
        sscan::mbar_wait_bounded(&bar, 0);  // once more for what is in flight
        return;
    }
    for (int i = threadIdx.x; i < p.moves; i += 128) {
        const int from = __ldg(p.src + i), to = __ldg(p.dst + i);
        if (to >= 0 && to < p.rows && from < p.rows) sscan::bulk_store(base + to * p.row_bytes, held + (from < 0 ? 0 : (long long)(i + 1) * p.stripe), bytes);
    }
    sscan::bulk_store_wait();
}

// The shared memory that a call may ask for.  The limit belongs to the kernel, not to a call: were it set to
// each call's own size, a call of few moves on another host thread could lower it between the set-up of one
// of many and its launch, which would then fail.
constexpr int kBulkShared = 200 * 1024;
template <typename U>
constexpr int kUnitShared = STATE_MOVE_MAX * (int)sizeof(U) > 96 * 1024 ? STATE_MOVE_MAX * (int)sizeof(U) : 96 * 1024;

// Stripes of whole 16-byte vectors: as long as shared memory holds, and short enough for four CTAs an SM where rows are small
// (160 moves: 229 us, in half of it 240, a quarter 267).
cudaError_t run_bulk(MoveParams& p, cudaStream_t st) {
    long long stripe = (long long)kBulkShared / (p.moves + 1) / 16 * 16;
    const long long spread = sscan::div_up(p.layers * p.row_bytes, 4 * 152 * 16) * 16;
    if (stripe > spread) stripe = spread;
    if (stripe < 128) stripe = 128;
    if (stripe > 4096) stripe = 4096;
    while (stripe > 16 && (p.moves + 1) * stripe > kBulkShared) stripe -= 16;
    p.stripe = (int)stripe;
    p.stripes = (int)sscan::div_up(p.row_bytes, stripe);
    const size_t smem = (size_t)(p.moves + 1) * stripe;
    const cudaError_t e = cudaFuncSetAttribute(state_move_bulk, cudaFuncAttributeMaxDynamicSharedMemorySize, kBulkShared);
    if (e != cudaSuccess) return e;
    return sscan::launch(state_move_bulk, dim3((unsigned)(p.layers * p.stripes)), dim3(128), smem, st, false, p);
}

template <typename U>
cudaError_t run(MoveParams& p, cudaStream_t st) {
    const int unit = (int)sizeof(U);
    // whole lines where they fit (kUnitShared: 96 KB of them, or one unit of the most moves)
    long long stripe = (long long)(96 * 1024) / p.moves / unit * unit;
    if (stripe < unit) stripe = unit;
    if (stripe > 512) stripe = 512;
    if (stripe > p.row_bytes) stripe = p.row_bytes;
    p.stripe = (int)stripe;
    p.stripes = (int)sscan::div_up(p.row_bytes, stripe);
    const size_t smem = (size_t)p.moves * stripe;
    const cudaError_t e = cudaFuncSetAttribute(state_move_kernel<U>, cudaFuncAttributeMaxDynamicSharedMemorySize, kUnitShared<U>);
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
    if (row_bytes % 16 == 0 && sscan::is_aligned(cache, 16)) {
        // (a grid of more CTAs than the hardware takes, with shortest stripes: by threads)
        if (layers * sscan::div_up(row_bytes, 16) <= 0x7fffffffLL) return sscan::finish(run_bulk(p, st));
        return sscan::finish(run<uint4>(p, st));
    }
    if (row_bytes % 4 == 0 && sscan::is_aligned(cache, 4)) return sscan::finish(run<unsigned>(p, st));
    if (row_bytes % 2 == 0 && sscan::is_aligned(cache, 2)) return sscan::finish(run<unsigned short>(p, st));
    return sscan::finish(run<unsigned char>(p, st));
}
