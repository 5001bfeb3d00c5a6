// Linear attention with a decay for each head on the FP32 units (formulas:
// lattn.cuh): the walk over the chunks and the gradients of one chunk.  256
// threads as 16 x 16; a product of [M, K] by [N, K] gives each thread the outputs
// (ty + 16 i, tx + 16 j), operands read from shared memory with any strides, one
// odd so that the 16 rows or columns of a half warp lie in different banks.
//
// The FP32 units and the shared memory that feeds them bound these: 2047 tokens x 8 heads of 64 x 64,
// forward and gradients 167 us, of which the gradients of the chunks 60 (256 CTAs in two rounds of one an SM; issue
// slots busy for 48%), the forward walk 32, the walks for states 15 each, for the parts of time before them
// 12 to 14 each (28 to 43% of the issue slots: one warp or two a scheduler).  Without time split for so few heads: 759 us.
#pragma once

#include "lattn.cuh"

namespace sscan {

template <int RM, int RN>
__device__ __forceinline__ void tile_mm(float (&acc)[RM][RN], const float* a, int am, int ak, const float* b, int bn, int bk,
                                        int depth) {
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    a += ty * am;
    b += tx * bn;
#pragma unroll 4
    for (int k = 0; k < depth; ++k) {
        float x[RM], y[RN];
#pragma unroll
        for (int i = 0; i < RM; ++i) x[i] = a[16 * i * am + k * ak];
#pragma unroll
        for (int j = 0; j < RN; ++j) y[j] = b[16 * j * bn + k * bk];
#pragma unroll
        for (int i = 0; i < RM; ++i)
#pragma unroll
            for (int j = 0; j < RN; ++j) acc[i][j] = fmaf(x[i], y[j], acc[i][j]);
    }
}
// The same with operands that lie [K][M] and [K][N], rows of 16-byte vectors: a thread's
// outputs are (4 ty + 64 a + i, 4 tx + 64 c + j), and a step of the sum takes one vector for
// four rows or columns, which keeps the FP32 units fed: 16 multiply-adds for two loads.
template <int RA, int RB>
__device__ __forceinline__ void tile_mm4(float (&acc)[4 * RA][4 * RB], const float* a, int lda, const float* b, int ldb, int depth) {
    a += 4 * (threadIdx.x >> 4);
    b += 4 * (threadIdx.x & 15);
#pragma unroll 4
    for (int k = 0; k < depth; ++k) {
        float x[4 * RA], y[4 * RB];
#pragma unroll
        for (int i = 0; i < RA; ++i) load4_smem(a + k * lda + 64 * i, *reinterpret_cast<float(*)[4]>(x + 4 * i));
#pragma unroll
        for (int j = 0; j < RB; ++j) load4_smem(b + k * ldb + 64 * j, *reinterpret_cast<float(*)[4]>(y + 4 * j));
#pragma unroll
        for (int i = 0; i < 4 * RA; ++i)
#pragma unroll
            for (int j = 0; j < 4 * RB; ++j) acc[i][j] = fmaf(x[i], y[j], acc[i][j]);
    }
}
template <int RM, int RN>
__device__ __forceinline__ void clear(float (&acc)[RM][RN]) {
#pragma unroll
    for (int i = 0; i < RM; ++i)
#pragma unroll
        for (int j = 0; j < RN; ++j) acc[i][j] = 0.f;
}

constexpr int kLd = kChunk + 1;  // leading dimension of rows of a chunk's tokens

// rows x kChunk values of channels [0, real) at tokens [t0, t0 + len) into dst [rows][kLd]; zeros elsewhere
// (sixteen loads of a thread on the way at once: one after the other they took most of a chunk's time)
template <int LD, typename T>
__device__ __forceinline__ void stage_rows(float* dst, const T* src, long long stride, int rows, int real, int t0, int len) {
    const int col = threadIdx.x & 63, first = threadIdx.x >> 6;
#pragma unroll 1
    for (int r0 = 0; r0 < rows; r0 += 64) {
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int r = r0 + first + 4 * i;
            x[i] = r < real && col < len ? to_f32(src[r * stride + t0 + col]) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) dst[(r0 + first + 4 * i) * LD + col] = x[i];
    }
}
template <typename T>
__device__ __forceinline__ void stage(float* dst, const T* src, long long stride, int rows, int real, int t0, int len) {
    stage_rows<kLd>(dst, src, stride, rows, real, t0, len);
}

// The same with rows of kLdv values; and a transposed copy [kChunk][ld] of such rows, times
// weight[token] where given: 32 x 32 values at a time along their diagonals, so that neither
// reads nor writes meet in a bank.
constexpr int kLdv = kChunk + 4;
template <typename T>
__device__ __forceinline__ void stage_vec(float* dst, const T* src, long long stride, int rows, int real, int t0, int len) {
    stage_rows<kLdv>(dst, src, stride, rows, real, t0, len);
}
__device__ __forceinline__ void transpose(float* dst, int ld, const float* src, int rows, const float* weight) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int block = warp; block < rows / 32 * 2; block += 8) {
        const int r0 = block >> 1 << 5, c0 = (block & 1) << 5;
#pragma unroll 8
        for (int i = 0; i < 32; ++i) {
            const int r = r0 + lane, c = c0 + ((lane + i) & 31);
            dst[c * ld + r] = src[r * kLdv + c] * (weight != nullptr ? weight[c] : 1.f);
        }
    }
}

// Steps of a chunk's tokens and their sums, by the first warp: dt (0 beyond len), run = T, rest = R.
struct ChunkSteps {
    float dt[kChunk], run[kChunk], low[kChunk], rest[kChunk];  // low: what run's roundings left out
};
template <typename T>
__device__ __forceinline__ void stage_steps(ChunkSteps& c, const LattnParams& p, long long at, int head, int len) {
    if (threadIdx.x >= 32) return;
    const int lane = threadIdx.x;
    float x[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int t = 2 * lane + i;
        x[i] = t < len ? lattn_step_of<T>(p, at + t, head) : 0.f;
        c.dt[t] = x[i];
    }
    Sum2 up = Sum2{x[0], 0.f} + Sum2{x[1], 0.f};
    float down = x[0] + x[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Sum2 u = shfl_up2(up, o);
        const float d = __shfl_down_sync(0xffffffffu, down, o);
        if (lane >= o) up = u + up;
        if (lane + o < 32) down += d;
    }
    const Sum2 before = shfl_up2(up, 1);
    const float behind = __shfl_down_sync(0xffffffffu, down, 1);
    const float a = lane < 31 ? behind : 0.f;
    const Sum2 first = (lane ? before : Sum2{0.f, 0.f}) + Sum2{x[0], 0.f}, second = first + Sum2{x[1], 0.f};
    c.run[2 * lane] = first.h;
    c.low[2 * lane] = first.l;
    c.run[2 * lane + 1] = second.h;
    c.low[2 * lane + 1] = second.l;
    c.rest[2 * lane] = a + x[1];
    c.rest[2 * lane + 1] = a;
}

// The slopes of a chunk's tokens and their sums in two terms, by the second warp.
struct ChunkSlopes {
    float slope[kChunk], sum[kChunk], low[kChunk];
};
template <typename T>
__device__ __forceinline__ void stage_slopes(ChunkSlopes& c, const LattnParams& p, long long at, int head, int len) {
    if (threadIdx.x < 32 || threadIdx.x >= 64) return;
    const int lane = threadIdx.x - 32;
    float x[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int t = 2 * lane + i;
        x[i] = t < len ? lattn_slope_of<T>(p, at + t, head) : 0.f;
        c.slope[t] = x[i];
    }
    Sum2 up = Sum2{x[0], 0.f} + Sum2{x[1], 0.f};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Sum2 u = shfl_up2(up, o);
        if (lane >= o) up = u + up;
    }
    const Sum2 before = shfl_up2(up, 1);
    const Sum2 first = (lane ? before : Sum2{0.f, 0.f}) + Sum2{x[0], 0.f}, second = first + Sum2{x[1], 0.f};
    c.sum[2 * lane] = first.h;
    c.low[2 * lane] = first.l;
    c.sum[2 * lane + 1] = second.h;
    c.low[2 * lane + 1] = second.l;
}

// One tile of 64 value channels of a head walks the chunks of a piece of time,
// its state [64][KD] in registers (value channel 4 tx + j, key channel 4 ty + 64 (i / 4) + i % 4).
//   WALK_ENDS     the state behind the piece, into p.ends (first pass of a time split)
//   WALK_OUT      outputs and final states
//   WALK_STATES   the state before each chunk, into p.starts
//   WALK_DSTATES  from the end: the gradient of the state behind each chunk, into p.dends
//   WALK_DENDS    from the end: the gradient of the state before the piece, into p.ends
// The outputs' part of the state takes it from shared memory.
template <typename T, int KD, int MODE>
__global__ void __launch_bounds__(256) lattn_walk(const LattnParams p) {
    constexpr int RK = KD / 16;
    constexpr bool REV = MODE == WALK_DSTATES || MODE == WALK_DENDS, END = MODE == WALK_ENDS || MODE == WALK_DENDS;
    constexpr int LK = KD + 4;
    extern __shared__ __align__(16) float smem[];
    float* Ks = smem;              // [KD][kLdv]
    float* Kt = Ks + KD * kLdv;    // [64][LK] weighted
    float* Vt = Kt + 64 * LK;      // [64][kLdv], token by channel
    float* Ps = Vt + 64 * kLdv;    // [64][kLdv]: values, then scores, then outputs
    float* Qs = Ps + 64 * kLdv;    // [KD][kLdv]  (outputs only)
    float* Ss = Qs + KD * kLdv;    // [KD][kLdv]
    __shared__ ChunkSteps c;
    __shared__ float weight[kChunk];
    griddep_wait();  // (launched while the kernel before it in the call ends)
    const int tile = blockIdx.x, head = tile / p.vtiles, v0 = (tile % p.vtiles) * kValueTile;
    const int w = blockIdx.y, b = blockIdx.z;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int group = head / (p.heads / p.groups), pv = min(kValueTile, p.P - v0);
    const float a = p.A[head] * kLog2e, skip = p.D != nullptr ? p.D[head] : 0.f;
    const T* q = static_cast<const T*>(p.q) + b * p.qb + (long long)group * p.N * p.qd;
    const T* k = static_cast<const T*>(p.k) + b * p.kb + (long long)group * p.N * p.kd;
    const T* v = static_cast<const T*>(p.v) + b * p.vb + ((long long)head * p.P + v0) * p.vd;
    if (REV) {  // the gradients' walk: q and do take the places of k and v
        k = q;
        v = static_cast<const T*>(p.dout) + ((long long)b * p.heads * p.P + (long long)head * p.P + v0) * p.L;
    }
    const long long vd = REV ? p.L : p.vd, kd = REV ? p.qd : p.kd;
    const long long steps = b * p.tb + head * p.td;
    const long long tile_size = (long long)kValueTile * KD, tiles = (long long)p.heads * p.vtiles;
    auto piece_tile = [&](float* base, int piece) { return base + (((long long)piece * p.batch + b) * tiles + tile) * tile_size; };
    float s[RK][4];

    // a state row's [P][N] of this head and tile: four key channels at once where N and the row allow it
    const bool fours = p.N % 4 == 0 && ((reinterpret_cast<uintptr_t>(p.s_in) | reinterpret_cast<uintptr_t>(p.s_out) |
                                         reinterpret_cast<uintptr_t>(p.ds_in) | reinterpret_cast<uintptr_t>(p.ds_out)) & 15u) == 0;
    auto load_state = [&](const float* row) {
#pragma unroll
        for (int a4 = 0; a4 < RK / 4; ++a4)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n = 4 * ty + 64 * a4, d = 4 * tx + j;
                const float* at = row + ((long long)head * p.P + v0 + d) * p.N + n;
                const bool in = row != nullptr && d < pv;
                if (fours) {
                    const float4 x = in && n < p.N ? *reinterpret_cast<const float4*>(at) : make_float4(0.f, 0.f, 0.f, 0.f);
                    s[4 * a4][j] = x.x; s[4 * a4 + 1][j] = x.y; s[4 * a4 + 2][j] = x.z; s[4 * a4 + 3][j] = x.w;
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[4 * a4 + i][j] = in && n + i < p.N ? at[i] : 0.f;
                }
            }
    };
    auto store_state = [&](float* row) {
#pragma unroll
        for (int a4 = 0; a4 < RK / 4; ++a4)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n = 4 * ty + 64 * a4, d = 4 * tx + j;
                if (d >= pv) continue;
                float* at = row + ((long long)head * p.P + v0 + d) * p.N + n;
                if (fours) {
                    if (n < p.N) *reinterpret_cast<float4*>(at) = make_float4(s[4 * a4][j], s[4 * a4 + 1][j], s[4 * a4 + 2][j], s[4 * a4 + 3][j]);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (n + i < p.N) at[i] = s[4 * a4 + i][j];
                }
            }
    };
    // tiles in scratch lie [key channel][64 value channels], so that a half warp's vectors follow one another
    auto store_tile = [&](float* to) {
#pragma unroll
        for (int i = 0; i < RK; ++i)
            *reinterpret_cast<float4*>(to + (4 * ty + 64 * (i >> 2) + (i & 3)) * kValueTile + 4 * tx) = make_float4(s[i][0], s[i][1], s[i][2], s[i][3]);
    };
    auto load_tile = [&](const float* from, float decay) {
#pragma unroll
        for (int i = 0; i < RK; ++i) {
            const float4 x = *reinterpret_cast<const float4*>(from + (4 * ty + 64 * (i >> 2) + (i & 3)) * kValueTile + 4 * tx);
            s[i][0] = fmaf(s[i][0], decay, x.x);
            s[i][1] = fmaf(s[i][1], decay, x.y);
            s[i][2] = fmaf(s[i][2], decay, x.z);
            s[i][3] = fmaf(s[i][3], decay, x.w);
        }
    };

    float total = 0.f;  // steps since the piece's start
    auto chunk = [&](int t0, int len) {
        __syncthreads();  // the chunk before still reads the buffers
        stage_steps<T>(c, p, steps + t0, head, len);
        stage_vec(Ks, k, kd, KD, p.N, t0, len);
        stage_vec(Ps, v, vd, kValueTile, pv, t0, len);
        if (MODE == WALK_OUT) {
            stage_vec(Qs, q, p.qd, KD, p.N, t0, len);
#pragma unroll
            for (int i = 0; i < RK; ++i) *reinterpret_cast<float4*>(Ss + (4 * ty + 64 * (i >> 2) + (i & 3)) * kLdv + 4 * tx) = make_float4(s[i][0], s[i][1], s[i][2], s[i][3]);
        }
        __syncthreads();
        if (MODE == WALK_STATES) store_tile(p.starts + (((long long)b * tiles + tile) * p.chunks + t0 / kChunk) * tile_size);
        if (MODE == WALK_DSTATES) store_tile(p.dends + (((long long)b * tiles + tile) * p.chunks + t0 / kChunk) * tile_size);
        if (threadIdx.x < kChunk) {
            const int t = threadIdx.x;
            weight[t] = REV ? p.scale * ex2(a * c.run[t]) : c.dt[t] * ex2(a * c.rest[t]);
        }
        const float all = c.run[kChunk - 1];
        total += all;
        transpose(Vt, kLdv, Ps, kValueTile, nullptr);
        __syncthreads();
        transpose(Kt, LK, Ks, KD, weight);
        if (MODE == WALK_OUT) {
            float acc[4][4], o[4][4];
            clear(acc);
            tile_mm4<1, 1>(acc, Qs, kLdv, Ks, kLdv, p.N);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int u = 4 * tx + j;
                float f[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int t = 4 * ty + i;
                    f[i] = t >= u ? p.scale * acc[i][j] * ex2(a * ((c.run[t] - c.run[u]) + (c.low[t] - c.low[u]))) * c.dt[u] : 0.f;
                    if (t == u) f[i] += skip;
                }
                *reinterpret_cast<float4*>(Ps + u * kLdv + 4 * ty) = make_float4(f[0], f[1], f[2], f[3]);
            }
            clear(o);
            tile_mm4<1, 1>(o, Qs, kLdv, Ss, kLdv, p.N);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float f = p.scale * ex2(a * c.run[4 * ty + i]);
#pragma unroll
                for (int j = 0; j < 4; ++j) o[i][j] *= f;
            }
            __syncthreads();
            tile_mm4<1, 1>(o, Ps, kLdv, Vt, kLdv, kChunk);
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 4; ++j) *reinterpret_cast<float4*>(Ps + (4 * tx + j) * kLdv + 4 * ty) = make_float4(o[0][j], o[1][j], o[2][j], o[3][j]);
        }
        __syncthreads();
        if (MODE == WALK_OUT) {
            T* out = static_cast<T*>(p.o) + ((long long)b * p.heads * p.P + (long long)head * p.P + v0) * p.L + t0;
            for (int r = threadIdx.x >> 6; r < pv; r += 4)
                if ((threadIdx.x & 63) < len) out[(long long)r * p.L + (threadIdx.x & 63)] = from_f32<T>(Ps[r * kLdv + (threadIdx.x & 63)]);
        }
        const float decay = ex2(a * all);
#pragma unroll
        for (int i = 0; i < RK; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i][j] *= decay;
        tile_mm4<RK / 4, 1>(s, Kt, LK, Vt, kLdv, kChunk);
    };
    auto walk = [&](int from, int to) {
        if (REV) {
            for (int t = (to - 1) / kChunk * kChunk; t >= from; t -= kChunk) chunk(t, min(kChunk, to - t));
        } else {
            for (int t = from; t < to; t += kChunk) chunk(t, min(kChunk, to - t));
        }
    };
    // the state that enters piece w, where a request began in piece `first`
    auto enter = [&](int first) {
#pragma unroll
        for (int i = 0; i < RK; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
        for (int i = first; i < w; ++i)
            load_tile(piece_tile(p.ends, i), i == first ? 0.f : ex2(a * p.sums[((long long)i * p.batch + b) * p.heads + head]));
    };
    auto leave = [&]() {
        store_tile(piece_tile(p.ends, w));
        if (threadIdx.x == 0 && v0 == 0) p.sums[((long long)w * p.batch + b) * p.heads + head] = total;
    };

    if (!p.packed) {
        const long long row = (long long)b * p.heads * p.P * p.N;
        const float* init = REV ? p.ds_in : p.s_in;
        float* last = REV ? p.ds_out : p.s_out;
        // pieces of the reversed walk count from the end
        const int whole = (p.L + kChunk - 1) / kChunk * kChunk;
        const int from = REV ? max(0, whole - (w + 1) * p.span) : w * p.span;
        const int to = REV ? min(p.L, whole - w * p.span) : min(p.L, (w + 1) * p.span);
        if (w == 0 || END) load_state(w == 0 && init != nullptr ? init + row : nullptr);
        else enter(0);
        walk(from, to);
        if (END) leave();
        else if (w == p.pieces - 1 && last != nullptr) store_state(last + row);
        return;
    }
    const long long row_size = (long long)p.heads * p.P * p.N;
    const int from = part_begin(p, w), to = part_begin(p, w + 1);
    if (MODE == WALK_ENDS) {
        // only what crosses the end of this piece of time counts
        int r = p.req.find(to - 1);
        const Piece x = piece_at(p.req, r, to - 1);
        if (x.end <= to || (p.apart && r >= 0 && r < p.req.requests && x.end - x.begin <= kLattnShort)) return;
        const bool begins = x.begin >= from;
        load_state(begins && x.has ? p.s_in + x.row * row_size : nullptr);
        if (begins) store_tile(piece_tile(p.aside, w));
        walk(max(from, x.begin), to);
        leave();
        return;
    }
    if (w == 0 && blockIdx.x == 0 && threadIdx.x < 32) p.req.check(threadIdx.x, 32);
    if (w == 0) {  // empty requests: a row that does not continue starts from zeros
        for (int r = 0; !p.apart && r < p.req.requests; ++r) {
            if (p.req.offset(r + 1) > p.req.offset(r)) continue;
            const int row = p.req.slot(r);
            if (row < 0 || p.req.continues(r)) continue;
            load_state(nullptr);
            store_state(p.s_out + row * row_size);
        }
    }
    if (from >= to) return;
    int r = p.req.find(from);
    Piece x;
    for (int t = from; next_piece(p.req, p.apart, r, t, to, x);) {
        const int end = min(x.end, to);
        if (x.begin < from && t == from) {
            enter(part_of(p, x.begin));
        } else if (x.end > to && p.pieces > 1) {
#pragma unroll
            for (int i = 0; i < RK; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
            load_tile(piece_tile(p.aside, w), 0.f);
        } else {
            load_state(x.has ? p.s_in + x.row * row_size : nullptr);
        }
        walk(t, end);
        if (x.end <= to && x.row >= 0) store_state(p.s_out + x.row * row_size);
        t = end;
    }
}

// sums over the 16 threads of a row, and over the 16 rows of threads of a column
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The gradients of one chunk, for a subset of the heads that share a set of
// queries and keys: dq and dk are summed over them in registers, so that no two
// CTAs add to the same value.  dt, T and R as in the walk.  STEPS: with delta, so that there are slopes.
template <typename T, int KD, bool STEPS>
__global__ void __launch_bounds__(256) lattn_grad(const LattnParams p) {
    constexpr int RK = KD / 16;
    constexpr int LS = KD + 1;
    extern __shared__ float smem[];
    float* Qs = smem;             // [KD][kLd]
    float* Ks = Qs + KD * kLd;    // [KD][kLd]
    float* Vs = Ks + KD * kLd;    // [64][kLd]
    float* Us = Vs + 64 * kLd;    // [64][kLd] do
    float* Es = Us + 64 * kLd;    // [64][kLd]
    float* Fs = Es + 64 * kLd;    // [64][kLd]
    float* Ss = Fs + 64 * kLd;    // [64][LS] state before the chunk
    float* Ds = Ss + 64 * LS;     // [64][LS] gradient of the state behind it
    __shared__ ChunkSteps c;
    __shared__ float rows[kChunk], cols[8][kChunk], diag[kChunk], xs[kChunk], ys[kChunk];
    __shared__ ChunkSlopes z;
    __shared__ float wide[8], das[8], dbs[8], state_dot, skip_sum;
    griddep_wait();
    const int t0 = blockIdx.x * kChunk, len = min(kChunk, p.L - t0), b = blockIdx.z;
    const int group = blockIdx.y / p.subsets, subset = blockIdx.y % p.subsets, per = p.heads / p.groups;
    const int h0 = group * per + (int)((long long)per * subset / p.subsets), h1 = group * per + (int)((long long)per * (subset + 1) / p.subsets);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long tiles = (long long)p.heads * p.vtiles, tile_size = (long long)kValueTile * KD;
    stage(Qs, static_cast<const T*>(p.q) + b * p.qb + (long long)group * p.N * p.qd, p.qd, KD, p.N, t0, len);
    stage(Ks, static_cast<const T*>(p.k) + b * p.kb + (long long)group * p.N * p.kd, p.kd, KD, p.N, t0, len);
    float dq[4][RK], dk[4][RK], qk[4][4];
    clear(dq);
    clear(dk);
    clear(qk);
    __syncthreads();
    tile_mm(qk, Qs, 1, kLd, Ks, 1, kLd, p.N);
    for (int head = h0; head < h1; ++head) {
        const float a = p.A[head] * kLog2e, skip = p.D != nullptr ? p.D[head] : 0.f;
        __syncthreads();
        stage_steps<T>(c, p, b * p.tb + head * p.td + t0, head, len);
        if (STEPS) stage_slopes<T>(z, p, b * p.tb + head * p.td + t0, head, len);
        if (threadIdx.x < kChunk) rows[threadIdx.x] = diag[threadIdx.x] = xs[threadIdx.x] = ys[threadIdx.x] = 0.f;
        for (int i = threadIdx.x; i < 8 * kChunk; i += 256) (&cols[0][0])[i] = 0.f;
        if (threadIdx.x == 0) state_dot = skip_sum = 0.f;
        float da = 0.f, db = 0.f;  // the pairs' part of dA, and of ddelta_bias without the rate
        for (int vt = 0; vt < p.vtiles; ++vt) {
            const int v0 = vt * kValueTile, pv = min(kValueTile, p.P - v0);
            const long long out_row = (long long)b * p.heads * p.P + (long long)head * p.P + v0;
            const long long at = (((long long)b * tiles + head * p.vtiles + vt) * p.chunks + blockIdx.x) * tile_size;
            __syncthreads();
            stage(Vs, static_cast<const T*>(p.v) + b * p.vb + ((long long)head * p.P + v0) * p.vd, p.vd, kValueTile, pv, t0, len);
            stage(Us, static_cast<const T*>(p.dout) + out_row * p.L, p.L, kValueTile, pv, t0, len);
            float dot = 0.f;
#pragma unroll 8
            for (int j = 0; j < kValueTile * KD / 256; ++j) {
                const int i = threadIdx.x + 256 * j;
                const float x = p.starts[at + i], y = p.dends[at + i];
                Ss[i % kValueTile * LS + i / kValueTile] = x;
                Ds[i % kValueTile * LS + i / kValueTile] = y;
                dot = fmaf(x, y, dot);
            }
            dot = warp_sum(dot);
            if (lane == 0) wide[warp] = dot;
            __syncthreads();
            if (threadIdx.x == 0) {
                float sum = 0.f;
                for (int i = 0; i < 8; ++i) sum += wide[i];
                state_dot += ex2(a * c.run[kChunk - 1]) * sum;
            }
            float g[4][4];
            clear(g);
            tile_mm(g, Us, 1, kLd, Vs, 1, kLd, kValueTile);
            float col[4] = {0.f, 0.f, 0.f, 0.f}, skips = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = ty + 16 * i;
                float row = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int u = tx + 16 * j;
                    const float time = (c.run[t] - c.run[u]) + (c.low[t] - c.low[u]), e = t >= u ? p.scale * ex2(a * time) : 0.f;
                    const float f = t >= u ? e * qk[i][j] : 0.f;
                    const float pair = t >= u ? f * g[i][j] : 0.f;
                    Es[t * kLd + u] = t >= u ? e * g[i][j] * c.dt[u] : 0.f;
                    Fs[t * kLd + u] = f;
                    if (t == u) {
                        diag[t] += pair;
                        skips += g[i][j];
                    } else {
                        const float weighted = pair * c.dt[u];
                        row += weighted;
                        da = t > u ? fmaf(weighted, time, da) : da;
                        if (STEPS) db = t > u ? fmaf(weighted, (z.sum[t] - z.sum[u]) + (z.low[t] - z.low[u]), db) : db;
                        col[j] += pair;
                    }
                }
                row = row_sum(row);
                if (tx == 0) rows[t] += row;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                col[j] += __shfl_xor_sync(0xffffffffu, col[j], 16);
                if (lane < 16) cols[warp][tx + 16 * j] += col[j];
            }
            skips = warp_sum(skips);
            __syncthreads();
            if (lane == 0) wide[warp] = skips;
            tile_mm(dq, Es, kLd, 1, Ks, kLd, 1, kChunk);
            tile_mm(dk, Es, 1, kLd, Qs, kLd, 1, kChunk);
            float r[4][RK];
            clear(r);
            tile_mm(r, Us, 1, kLd, Ss, 1, LS, kValueTile);  // S^T do
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = ty + 16 * i;
                const float f = p.scale * ex2(a * c.run[t]);
                float x = 0.f;
#pragma unroll
                for (int j = 0; j < RK; ++j) {
                    r[i][j] *= f;
                    x = fmaf(r[i][j], Qs[(tx + 16 * j) * kLd + t], x);
                    dq[i][j] += r[i][j];
                }
                x = row_sum(x);
                if (tx == 0) xs[t] += x;
            }
            clear(r);
            tile_mm(r, Vs, 1, kLd, Ds, 1, LS, kValueTile);  // dS'^T v
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = ty + 16 * i;
                const float f = c.dt[t] * ex2(a * c.rest[t]);
#pragma unroll
                for (int j = 0; j < RK; ++j) dk[i][j] = fmaf(r[i][j], f, dk[i][j]);
            }
            float dv[4][4];
            clear(dv);
            tile_mm(dv, Ks, 1, kLd, Ds, LS, 1, p.N);  // dS' k
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = ty + 16 * i;
                const float f = ex2(a * c.rest[t]);
                float y = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    dv[i][j] *= f;
                    y = fmaf(dv[i][j], Vs[(tx + 16 * j) * kLd + t], y);
                }
                y = row_sum(y);
                if (tx == 0) ys[t] += y;
            }
            tile_mm(dv, Fs, 1, kLd, Us, kLd, 1, kChunk);
            __syncthreads();
            if (threadIdx.x == 0)
                for (int i = 0; i < 8; ++i) skip_sum += wide[i];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int t = ty + 16 * i, d = tx + 16 * j;
                    Es[d * kLd + t] = fmaf(c.dt[t], dv[i][j], skip * Us[d * kLd + t]);
                }
            __syncthreads();
            T* out = static_cast<T*>(p.dv) + out_row * p.L + t0;
            for (int d = threadIdx.x >> 6; d < pv; d += 4)
                if ((threadIdx.x & 63) < len) out[(long long)d * p.L + (threadIdx.x & 63)] = from_f32<T>(Es[d * kLd + (threadIdx.x & 63)]);
        }
        da = warp_sum(da);
        db = warp_sum(db);
        if (lane == 0) das[warp] = da;
        if (lane == 0) dbs[warp] = db;
        __syncthreads();
        if (threadIdx.x < 32) {
            // two tokens a lane: sums from the end of (rows - columns + X), from the start of dt Y
            float m[2], y[2], w[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int t = 2 * lane + i;
                float column = 0.f;
                for (int j = 0; j < 8; ++j) column += cols[j][t];
                w[i] = column + diag[t] + ys[t];
                m[i] = rows[t] - c.dt[t] * column + xs[t];
                y[i] = c.dt[t] * ys[t];
            }
            float down = m[0] + m[1], up = y[0] + y[1];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float d = __shfl_down_sync(0xffffffffu, down, o), u = __shfl_up_sync(0xffffffffu, up, o);
                if (lane + o < 32) down += d;
                if (lane >= o) up += u;
            }
            const float behind = __shfl_down_sync(0xffffffffu, down, 1), before = __shfl_up_sync(0xffffffffu, up, 1);
            float g[2];
            const float e = lane < 31 ? behind : 0.f, s = lane ? before : 0.f;
            g[1] = m[1] + e + (s + y[0]) + state_dot;
            g[0] = m[0] + m[1] + e + s + state_dot;
            // dA as its terms by the time that they span (lattn.cuh)
            float dA = (lane < 8 ? das[lane] : 0.f) + (lane == 0 ? state_dot * c.run[kChunk - 1] : 0.f);
            float timed = 0.f, dbias = 0.f;
            if (STEPS) timed = (lane < 8 ? dbs[lane] : 0.f) + (lane == 0 ? state_dot * z.sum[kChunk - 1] : 0.f);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int t = 2 * lane + i;
                if (t >= len) continue;
                dA += fmaf(xs[t], c.run[t], y[i] * c.rest[t]);
                if (STEPS) timed += fmaf(xs[t], z.sum[t], y[i] * (z.sum[kChunk - 1] - z.sum[t]));
                float dd = fmaf(p.A[head], g[i], w[i]);
                if (STEPS) {
                    dd *= z.slope[t];
                    dbias = fmaf(z.slope[t], w[i], dbias);
                    static_cast<T*>(p.ddelta)[((long long)b * p.heads + head) * p.L + t0 + t] = from_f32<T>(dd);
                }
            }
            dA = warp_sum(dA);
            dbias = warp_sum(fmaf(p.A[head], timed, dbias));
            if (lane == 0) {
                const long long all = (long long)p.batch * p.chunks, at = (long long)b * p.chunks + blockIdx.x;
                p.head_part[head * all + at] = dA;
                p.head_part[((long long)p.heads + head) * all + at] = dbias;
                p.head_part[((long long)2 * p.heads + head) * all + at] = skip_sum;
            }
        }
    }
    // dq and dk [KD][tokens]
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        __syncthreads();
        float* buf = which ? Ks : Qs;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < RK; ++j) buf[(tx + 16 * j) * kLd + ty + 16 * i] = which ? dk[i][j] : dq[i][j];
        __syncthreads();
        const long long at = ((long long)b * p.groups * p.N + (long long)group * p.N) * p.L + t0;
        float* part = which ? p.dk_part : p.dq_part;
        T* out = static_cast<T*>(which ? p.dk : p.dq);
        const int col = threadIdx.x & 63;
        if (col >= len) continue;
        for (int n = threadIdx.x >> 6; n < p.N; n += 4) {
            if (part != nullptr) part[(long long)subset * p.batch * p.groups * p.N * p.L + at + (long long)n * p.L + col] = buf[n * kLd + col];
            else out[at + (long long)n * p.L + col] = from_f32<T>(buf[n * kLd + col]);
        }
    }
}

// dq and dk from their parts, in the order of the subsets
template <typename T>
__global__ void __launch_bounds__(256) lattn_add_parts(const float* a, const float* b, T* x, T* y, long long n, int parts) {
    griddep_wait();
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < 2 * n; i += (long long)gridDim.x * 256) {
        const float* from = i < n ? a + i : b + (i - n);
        float sum = 0.f;
        for (int j = 0; j < parts; ++j) sum += from[j * n];
        if (i < n) x[i] = from_f32<T>(sum);
        else y[i - n] = from_f32<T>(sum);
    }
}
// dA, ddelta_bias and dD from their parts: one CTA a head and output, sums in a fixed order
__global__ void __launch_bounds__(256) lattn_add_heads(const float* part, float* dA, float* dbias, float* dD, int heads, long long all) {
    __shared__ float sums[8];
    griddep_wait();
    float* to = blockIdx.y == 0 ? dA : blockIdx.y == 1 ? dbias : dD;
    if (to == nullptr) return;
    const float* from = part + ((long long)blockIdx.y * heads + blockIdx.x) * all;
    float s = 0.f;
    for (long long i = threadIdx.x; i < all; i += 256) s += from[i];
    s = warp_sum(s);
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < 8; ++i) s += sums[i];
        to[blockIdx.x] = s;
    }
}

}  // namespace sscan
