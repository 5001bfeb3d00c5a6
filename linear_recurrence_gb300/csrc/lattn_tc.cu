// Launches of the linear attention kernels on the tensor cores (lattn_tc.cuh).
#include "lattn_tc_grad.cuh"

namespace sscan {
// defined in sscan_fwd_tma.cu
bool tma_encode_rows(CUtensorMap* map, const void* base, long long L, long long rows, long long sets, long long batch,
                     long long row_stride, long long batch_stride, int box_rows);

namespace {

bool tma_rows(const void* base, long long row, long long batch_stride, int batch) {
    return is_aligned(base, 16) && row > 0 && row % 8 == 0 && (batch == 1 || (batch_stride > 0 && batch_stride % 8 == 0));
}

// An input's rows for TMA: `sets` of `rows` rows a batch.
struct TcInput {
    const void* base;
    long long row_stride, batch_stride;
    int rows, sets, box;
};

// Tensor maps of up to two inputs; rows that TMA cannot take are copied into *copy, which
// the caller frees on the stream.
cudaError_t make_maps(const TcInput (&in)[2], CUtensorMap* const (&maps)[2], int batch, int L, void** copy, cudaStream_t st) {
    TcInput x[2] = {in[0], in[1]};
    TcCopy c = {};
    size_t bytes[2] = {0, 0};
    for (int i = 0; i < 2; ++i) {
        if (tma_rows(x[i].base, x[i].row_stride, x[i].batch_stride, batch)) continue;
        bytes[i] = (size_t)batch * x[i].sets * x[i].rows * ((L + 7) / 8 * 8) * sizeof(bf16);
    }
    if (bytes[0] + bytes[1] > 0) {
        cudaError_t e = scratch_alloc(copy, bytes[0] + bytes[1], st);
        if (e != cudaSuccess) return e;
        c.to_stride = (L + 7) / 8 * 8;
        c.batch = batch;
        c.L = L;
        char* to = static_cast<char*>(*copy);
        long long most = 0;
        for (int i = 0; i < 2; ++i) {
            if (bytes[i] == 0) continue;
            c.from[i] = static_cast<const bf16*>(x[i].base);
            c.to[i] = reinterpret_cast<bf16*>(to);
            c.batch_stride[i] = x[i].batch_stride;
            c.row_stride[i] = x[i].row_stride;
            c.rows[i] = (long long)x[i].sets * x[i].rows;
            x[i].base = to;
            x[i].row_stride = c.to_stride;
            x[i].batch_stride = c.rows[i] * c.to_stride;
            if (c.rows[i] > most) most = c.rows[i];
            to += bytes[i];
        }
        const long long gx = div_up(L, 2048), gy = div_up(batch * most, 4);
        e = launch(lattn_tc_copy, dim3((unsigned)gx, (unsigned)(gy < 65535 ? gy : 65535), 2), dim3(256), 0, st, false, c);
        if (e != cudaSuccess) return e;
    }
    for (int i = 0; i < 2; ++i) {
        // with one batch its stride only has to be a valid one
        const long long b = batch == 1 ? x[i].row_stride * x[i].sets * x[i].rows : x[i].batch_stride;
        if (!tma_encode_rows(maps[i], x[i].base, L, x[i].rows, x[i].sets, batch, x[i].row_stride, b, x[i].box)) return cudaErrorInvalidValue;
    }
    return cudaSuccess;
}
cudaError_t make_qk_maps(const LattnParams& p, TcMaps& maps, void** copy, cudaStream_t st) {
    const int box = p.N <= 64 ? 64 : 128;
    const TcInput in[2] = {{p.q, p.qd, p.qb, p.N, p.groups, box}, {p.k, p.kd, p.kb, p.N, p.groups, box}};
    CUtensorMap* const to[2] = {&maps.q, &maps.k};
    return make_maps(in, to, p.batch, p.L, copy, st);
}

template <int KD, int MODE, bool APART = false>
cudaError_t walk(const LattnParams& p, const TcMaps& maps, int pieces, bool after, cudaStream_t st) {
    constexpr unsigned bytes = MODE == WALK_OUT ? TcWalkSmem<KD>::bytes : TcWalkSmem<KD>::few_bytes;
    const cudaError_t e = cudaFuncSetAttribute(lattn_tc_walk<KD, MODE, APART>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    return launch(lattn_tc_walk<KD, MODE, APART>, dim3((unsigned)(p.heads * p.vtiles), (unsigned)pieces, (unsigned)p.batch), dim3(kTcThreads), bytes,
                  st, after, p, maps);
}
// (after: not the first kernel of its call, which begins while the one before it ends)
template <int KD, bool APART>
cudaError_t walk_all(const LattnParams& p, const TcMaps& maps, bool after, cudaStream_t st) {
    cudaError_t e = cudaSuccess;
    if (p.pieces > 1) e = walk<KD, WALK_ENDS, APART>(p, maps, p.pieces - 1, after, st);
    return e != cudaSuccess ? e : walk<KD, WALK_OUT, APART>(p, maps, p.pieces, after || p.pieces > 1, st);
}
template <int KD>
cudaError_t walk_any(const LattnParams& p, const TcMaps& maps, bool after, cudaStream_t st) {
    return p.apart ? walk_all<KD, true>(p, maps, true, st) : walk_all<KD, false>(p, maps, after, st);
}

template <int KD>
cudaError_t grad(const LattnParams& p, const TcMaps& maps, const TcGradMaps& gmaps, bool after, cudaStream_t st) {
    cudaError_t e = cudaSuccess;
    if (p.pieces > 1) e = walk<KD, WALK_ENDS>(p, maps, p.pieces - 1, after, st);
    if (e == cudaSuccess) e = walk<KD, WALK_STATES>(p, maps, p.pieces, after || p.pieces > 1, st);
    if (e == cudaSuccess && p.pieces > 1) e = walk<KD, WALK_DENDS>(p, maps, p.pieces - 1, true, st);
    if (e == cudaSuccess) e = walk<KD, WALK_DSTATES>(p, maps, p.pieces, true, st);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(lattn_tc_grad<KD>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)TcGradSmem<KD>::bytes);
    if (e != cudaSuccess) return e;
    return launch(lattn_tc_grad<KD>, dim3((unsigned)p.chunks, (unsigned)(p.groups * p.subsets), (unsigned)p.batch), dim3(kGradThreads),
                  TcGradSmem<KD>::bytes, st, true, p, gmaps);
}

}  // namespace

int lattn_tc_grad_copies(const LattnParams& p) {
    const bool v = tma_rows(p.v, p.vd, p.vb, p.batch), u = tma_rows(p.dout, p.L, (long long)p.heads * p.P * p.L, p.batch);
    return (lattn_tc_copies(p) ? 1 : 0) + (v && u ? 0 : 1);
}

cudaError_t lattn_tc_grad_launch(const LattnParams& p, cudaStream_t st) {
    TcMaps maps = {};
    TcGradMaps gmaps = {};
    void *copy = nullptr, *copy_v = nullptr;
    cudaError_t e = make_qk_maps(p, maps, &copy, st);
    if (e == cudaSuccess) {
        gmaps.q = maps.q;
        gmaps.k = maps.k;
        const TcInput in[2] = {{p.v, p.vd, p.vb, p.P, p.heads, 64}, {p.dout, p.L, (long long)p.heads * p.P * p.L, p.P, p.heads, 64}};
        CUtensorMap* const to[2] = {&gmaps.v, &gmaps.dout};
        e = make_maps(in, to, p.batch, p.L, &copy_v, st);
    }
    const bool after = copy != nullptr || copy_v != nullptr;
    if (e == cudaSuccess) e = p.N <= 64 ? grad<64>(p, maps, gmaps, after, st) : grad<128>(p, maps, gmaps, after, st);
    void* const copies[2] = {copy, copy_v};
    for (void* c : copies) {
        if (c == nullptr) continue;
        const cudaError_t ef = cudaFreeAsync(c, st);
        if (e == cudaSuccess) e = ef;
    }
    return e;
}

bool lattn_tc_copies(const LattnParams& p) {
    return !tma_rows(p.q, p.qd, p.qb, p.batch) || !tma_rows(p.k, p.kd, p.kb, p.batch);
}

cudaError_t lattn_tc_walk_launch(const LattnParams& p, cudaStream_t st) {
    TcMaps maps = {};
    void* copy = nullptr;
    cudaError_t e = p.L > 0 ? make_qk_maps(p, maps, &copy, st) : cudaSuccess;
    if (e == cudaSuccess) e = p.N <= 64 ? walk_any<64>(p, maps, copy != nullptr, st) : walk_any<128>(p, maps, copy != nullptr, st);
    if (copy != nullptr) {
        const cudaError_t ef = cudaFreeAsync(copy, st);
        if (e == cudaSuccess) e = ef;
    }
    return e;
}

}  // namespace sscan
