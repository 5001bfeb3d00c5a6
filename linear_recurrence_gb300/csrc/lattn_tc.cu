// Launches of the linear attention kernels on the tensor cores (lattn_tc.cuh).
#include "lattn_tc.cuh"

namespace sscan {
// defined in sscan_fwd_tma.cu
bool tma_encode_rows(CUtensorMap* map, const void* base, long long L, long long rows, long long sets, long long batch,
                     long long row_stride, long long batch_stride, int box_rows);

namespace {

bool tma_rows(const void* base, long long row, long long batch_stride, int batch) {
    return is_aligned(base, 16) && row > 0 && row % 8 == 0 && (batch == 1 || (batch_stride > 0 && batch_stride % 8 == 0));
}

// Tensor maps of q and k; rows that TMA cannot take are copied into *copy, which the
// caller frees on the stream.
cudaError_t make_maps(const LattnParams& p, TcMaps& maps, void** copy, cudaStream_t st) {
    const void* base[2] = {p.q, p.k};
    long long row[2] = {p.qd, p.kd}, batch[2] = {p.qb, p.kb};
    const bool fine[2] = {tma_rows(p.q, p.qd, p.qb, p.batch), tma_rows(p.k, p.kd, p.kb, p.batch)};
    if (!fine[0] || !fine[1]) {
        TcCopy c = {};
        c.rows = (long long)p.groups * p.N;
        c.to_stride = (p.L + 7) / 8 * 8;
        c.batch = p.batch;
        c.L = p.L;
        const size_t each = (size_t)p.batch * c.rows * c.to_stride;
        const int count = (fine[0] ? 0 : 1) + (fine[1] ? 0 : 1);
        cudaError_t e = scratch_alloc(copy, count * each * sizeof(bf16), st);
        if (e != cudaSuccess) return e;
        bf16* to = static_cast<bf16*>(*copy);
        for (int i = 0; i < 2; ++i) {
            if (fine[i]) continue;
            c.from[i] = static_cast<const bf16*>(base[i]);
            c.to[i] = to;
            c.batch_stride[i] = batch[i];
            c.row_stride[i] = row[i];
            base[i] = to;
            row[i] = c.to_stride;
            batch[i] = c.rows * c.to_stride;
            to += each;
        }
        const long long gx = div_up(p.L, 2048), gy = div_up(p.batch * c.rows, 4);
        e = launch(lattn_tc_copy, dim3((unsigned)gx, (unsigned)(gy < 65535 ? gy : 65535), 2), dim3(256), 0, st, false, c);
        if (e != cudaSuccess) return e;
    }
    CUtensorMap* to[2] = {&maps.q, &maps.k};
    for (int i = 0; i < 2; ++i) {
        // with one batch its stride only has to be a valid one
        const long long b = p.batch == 1 ? row[i] * p.groups * p.N : batch[i];
        if (!tma_encode_rows(to[i], base[i], p.L, p.N, p.groups, p.batch, row[i], b, p.N <= 64 ? 64 : 128)) return cudaErrorInvalidValue;
    }
    return cudaSuccess;
}

template <int KD, int MODE>
cudaError_t walk(const LattnParams& p, const TcMaps& maps, int pieces, cudaStream_t st) {
    constexpr unsigned bytes = MODE == WALK_OUT ? TcWalkSmem<KD>::bytes : TcWalkSmem<KD>::few_bytes;
    const cudaError_t e = cudaFuncSetAttribute(lattn_tc_walk<KD, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    return launch(lattn_tc_walk<KD, MODE>, dim3((unsigned)(p.heads * p.vtiles), (unsigned)pieces, (unsigned)p.batch), dim3(kTcThreads), bytes,
                  st, false, p, maps);
}
template <int KD>
cudaError_t walk_all(const LattnParams& p, const TcMaps& maps, cudaStream_t st) {
    cudaError_t e = cudaSuccess;
    if (p.pieces > 1) e = walk<KD, WALK_ENDS>(p, maps, p.pieces - 1, st);
    return e != cudaSuccess ? e : walk<KD, WALK_OUT>(p, maps, p.pieces, st);
}

}  // namespace

bool lattn_tc_copies(const LattnParams& p) {
    return !tma_rows(p.q, p.qd, p.qb, p.batch) || !tma_rows(p.k, p.kd, p.kb, p.batch);
}

cudaError_t lattn_tc_walk_launch(const LattnParams& p, cudaStream_t st) {
    TcMaps maps = {};
    void* copy = nullptr;
    cudaError_t e = p.L > 0 ? make_maps(p, maps, &copy, st) : cudaSuccess;
    if (e == cudaSuccess) e = p.N <= 64 ? walk_all<64>(p, maps, st) : walk_all<128>(p, maps, st);
    if (copy != nullptr) {
        const cudaError_t ef = cudaFreeAsync(copy, st);
        if (e == cudaSuccess) e = ef;
    }
    return e;
}

}  // namespace sscan
