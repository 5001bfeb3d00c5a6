// RMS norms around a layer's scan on sm_103a.
//
// addnorm, before the layer, on token rows [rows, width]:
//   r = residual + scale * x   (kept, fp32)
//   y = r * rstd * w,          rstd = 1 / sqrt(mean(r^2) + eps)
//
// gatenorm, after the scan, over the channels of y [batch, dim, L] (the scan's
// channel-major layout) or [rows, dim] (single tokens), in `groups` equal parts:
//   gate first:  v = y * silu(z),  out = v * rstd(v) * w
//   norm first:  out = y * rstd(y) * w * silu(z)
//
// Gradients.  With n = v * rstd and q the gradient of n (the upstream gradient
// times w, and times the gate when the norm comes first):
//   dv = rstd * (q - n * mean(q * n)),   dw = sum over tokens of (upstream * n)
//
// All of it is a few operations a value, so HBM bandwidth bounds it: each
// input should be read once and each output written once.  Sums are fp32.
// Measured, of the copy rate: addnorm 8192 x 2560 bf16 with an fp32 residual forward
// 36.3 us (102%), backward 54.9 + 6.0 us (82%); gatenorm 4 x 2048 x 2048 bf16 forward 26
// us (57%), backward 41 + 4 us (55%).
#include <cooperative_groups.h>
#include <stdio.h>

#include <algorithm>
#include <initializer_list>

#include "block_utils.cuh"

namespace {

namespace cg = cooperative_groups;
using sscan::bf16;
using sscan::VecOf;

// Elements between a row and the 16-byte boundary at or below it.
template <typename T>
__device__ __forceinline__ int phase_of(const T* p) {
    return (int)((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T));
}

// ---- token rows -------------------------------------------------------------

// A CTA owns one row at a time: thread i holds vectors i, i + threads, ... (V
// of them) in registers, so the row is read once.
template <int NUM>
__device__ __forceinline__ void cta_sum(float (&v)[NUM], float* shared) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
    for (int i = 0; i < NUM; ++i) v[i] = sscan::warp_sum(v[i]);
    if (warps == 1) return;
    __syncthreads();  // the row before may still read
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < NUM; ++i) shared[i * 32 + warp] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NUM; ++i) v[i] = sscan::warp_sum(lane < warps ? shared[i * 32 + lane] : 0.f);
}

// The thread's i-th vector, or past the row's end its last one, whose values are
// then not used (its owner may be writing r over it): loads without a
// branch between them are under way together (4096 x 2049 bf16, eight single values a
// thread: 60 us forward and backward, 107 with the branch).
__device__ __forceinline__ int clamped(int i, int vecs) {
    const int at = threadIdx.x + i * blockDim.x;
    return at < vecs ? at : vecs - 1;
}

template <typename T, int E>
__device__ __forceinline__ void load_vec(const T* p, float (&v)[E]) {
    if constexpr (E == 1) {
        v[0] = sscan::to_f32(*p);
    } else if constexpr (sizeof(T) * E == 32) {  // fp32 beside bf16 vectors
        float lo[4], hi[4];
        sscan::widen(reinterpret_cast<const uint4*>(p)[0], lo, static_cast<float*>(nullptr));
        sscan::widen(reinterpret_cast<const uint4*>(p)[1], hi, static_cast<float*>(nullptr));
#pragma unroll
        for (int i = 0; i < 4; ++i) { v[i] = lo[i]; v[4 + i] = hi[i]; }
    } else {
        sscan::widen(*reinterpret_cast<const uint4*>(p), v, static_cast<T*>(nullptr));
    }
}
template <typename T, int E>
__device__ __forceinline__ void store_vec(T* p, const float (&v)[E]) {
    if constexpr (E == 1) {
        *p = sscan::from_f32<T>(v[0]);
    } else if constexpr (sizeof(T) * E == 32) {
        reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *reinterpret_cast<uint4*>(p) = sscan::narrow(v, static_cast<T*>(nullptr));
    }
}

// The widest CTA of a row kernel: 16384 columns are 512 threads of four
// 8-element vectors, and 1024 threads of four 4-element or sixteen single ones.
template <int E> constexpr int kRowThreads = E == 8 ? 512 : 1024;

struct AddNormParams {
    const void* x;          // [rows, width]
    const float* residual;  // [rows, width] or NULL
    const float* w;
    void* y;
    float* r;               // residual after the addition
    const void* dy;
    const float* dr;        // gradient of r, or NULL
    void* dx;
    float* dresidual;
    float* parts;           // [CTAs, width] weight-gradient sums
    long long rows;
    int width;
    float scale, eps;
};

template <typename T, int E, int V>
__global__ void __launch_bounds__(kRowThreads<E>) addnorm_fwd_kernel(const AddNormParams p) {
    __shared__ float shared[32];
    const int vecs = p.width / E;
    for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const T* x = static_cast<const T*>(p.x) + row * p.width;
        float a[V][E], r[V][E], sum[1] = {0.f};
#pragma unroll
        for (int i = 0; i < V; ++i) load_vec<T, E>(x + (long long)clamped(i, vecs) * E, a[i]);
        if (p.residual != nullptr) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                load_vec<float, E>(p.residual + row * p.width + (long long)clamped(i, vecs) * E, r[i]);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int j = 0; j < E; ++j) r[i][j] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int at = threadIdx.x + i * blockDim.x;
            if (at >= vecs) break;
#pragma unroll
            for (int j = 0; j < E; ++j) {
                r[i][j] = fmaf(p.scale, a[i][j], r[i][j]);
                sum[0] = fmaf(r[i][j], r[i][j], sum[0]);
            }
            store_vec<float, E>(p.r + row * p.width + (long long)at * E, r[i]);
        }
        cta_sum(sum, shared);
        const float rstd = rsqrtf(sum[0] / (float)p.width + p.eps);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int at = threadIdx.x + i * blockDim.x;
            if (at >= vecs) break;
            float w[E];
            load_vec<float, E>(p.w + at * E, w);
#pragma unroll
            for (int j = 0; j < E; ++j) r[i][j] *= rstd * w[j];
            store_vec<T, E>(static_cast<T*>(p.y) + row * p.width + (long long)at * E, r[i]);
        }
    }
}

// Persistent CTAs: a thread keeps the weight-gradient sums of its columns over
// all the CTA's rows and writes them once, as one row of p.parts.
template <typename T, int E, int V>
__global__ void __launch_bounds__(kRowThreads<E>) addnorm_bwd_kernel(const AddNormParams p) {
    __shared__ float shared[64];
    const int vecs = p.width / E;
    float dw[V][E];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < E; ++j) dw[i][j] = 0.f;
    for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
        float r[V][E], g[V][E], d[V][E], sum[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < V; ++i) {  // every load of the row before the first sum
            if (V == 1 && threadIdx.x >= vecs) break;
            const long long from = row * p.width + (long long)(V == 1 ? threadIdx.x : clamped(i, vecs)) * E;
            load_vec<float, E>(p.r + from, r[i]);
            load_vec<T, E>(static_cast<const T*>(p.dy) + from, g[i]);
            if (V > 1) continue;
            if (p.dr != nullptr) {
                load_vec<float, E>(p.dr + from, d[i]);
            } else {
#pragma unroll
                for (int j = 0; j < E; ++j) d[i][j] = 0.f;
            }
        }
        if (V > 1) {
            if (p.dr != nullptr) {
#pragma unroll
                for (int i = 0; i < V; ++i) load_vec<float, E>(p.dr + row * p.width + (long long)clamped(i, vecs) * E, d[i]);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i)
#pragma unroll
                    for (int j = 0; j < E; ++j) d[i][j] = 0.f;
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int at = threadIdx.x + i * blockDim.x;
            if (at >= vecs) break;
            float w[E];
            load_vec<float, E>(p.w + at * E, w);
#pragma unroll
            for (int j = 0; j < E; ++j) {
                sum[0] = fmaf(r[i][j], r[i][j], sum[0]);
                sum[1] = fmaf(g[i][j] * w[j], r[i][j], sum[1]);
            }
        }
        cta_sum(sum, shared);
        const float rstd = rsqrtf(sum[0] / (float)p.width + p.eps);
        const float c = sum[1] / (float)p.width * rstd * rstd;  // dr = dr_out + rstd * (dy w - r c)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int at = threadIdx.x + i * blockDim.x;
            if (at >= vecs) break;
            float w[E];
            load_vec<float, E>(p.w + at * E, w);
#pragma unroll
            for (int j = 0; j < E; ++j) {
                dw[i][j] = fmaf(g[i][j], r[i][j] * rstd, dw[i][j]);
                d[i][j] = fmaf(rstd, fmaf(-r[i][j], c, g[i][j] * w[j]), d[i][j]);
            }
            if (p.dresidual != nullptr) store_vec<float, E>(p.dresidual + row * p.width + (long long)at * E, d[i]);
#pragma unroll
            for (int j = 0; j < E; ++j) d[i][j] *= p.scale;
            store_vec<T, E>(static_cast<T*>(p.dx) + row * p.width + (long long)at * E, d[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int at = threadIdx.x + i * blockDim.x;
        if (at >= vecs) break;
        store_vec<float, E>(p.parts + (long long)blockIdx.x * p.width + at * E, dw[i]);
    }
    sscan::griddep_launch_dependents();
}

// out[c] = sum over rows of parts[row, c], in a fixed order: a CTA takes 32
// columns, or eight (a sector of a row) and more rows at a time where 32 would
// leave SMs without a CTA (4560 rows of 113 columns: 12.5 us against 37; 8192
// columns: 5.0 us with 32, 10.6 with eight).
template <int kSumCols>
__global__ void __launch_bounds__(1024) column_sum_kernel(const float* parts, float* out, long long rows, long long cols) {
    __shared__ float part[kSumCols][33];
    constexpr int kBatch = 8, kStep = 1024 / kSumCols;  // rows of a thread under way, rows of a step
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, column = lane % kSumCols;
    const long long c = (long long)blockIdx.x * kSumCols + column;
    sscan::griddep_wait();
    float a = 0.f;
    if (c < cols) {
        for (long long r0 = threadIdx.x / kSumCols; r0 < rows; r0 += kStep * kBatch) {
            float v[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) v[k] = r0 + kStep * k < rows ? parts[(r0 + kStep * k) * cols + c] : 0.f;
#pragma unroll
            for (int k = 0; k < kBatch; ++k) a += v[k];
        }
    }
#pragma unroll
    for (int o = 16; o >= kSumCols; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    if (lane < kSumCols) part[column][warp] = a;
    __syncthreads();
    const long long mine = (long long)blockIdx.x * kSumCols + warp;
    if (warp < kSumCols) {
        a = sscan::warp_sum(part[warp][lane]);
        if (lane == 0 && mine < cols) out[mine] = a;
    }
}

struct GateParams {
    const void* y;
    const void* z;
    const float* w;
    const void* dout;
    void* out;
    void* dy;
    void* dz;
    float* parts;   // weight-gradient sums of each (batch, token tile): [tiles, dim]
    long long batch, dim, len, groups;
    int size, share;  // channels of a group, and of a CTA of its cluster
    long long z_batch_stride, z_dim_stride;
    float eps;
};

// One row of a group: CTA per (row, group) of [rows, dim].
template <typename T, int E, int V, bool NORM_FIRST>
__global__ void __launch_bounds__(kRowThreads<E>) gatenorm_rows_kernel(const GateParams p) {
    __shared__ float shared[32];
    const int size = p.size;
    const unsigned groups = (unsigned)p.groups;
    const long long row = groups == 1 ? blockIdx.x : blockIdx.x / groups;
    const long long first = groups == 1 ? 0 : (long long)(blockIdx.x % groups) * size;
    const int vecs = size / E;
    const T* y = static_cast<const T*>(p.y) + row * p.dim + first;
    const T* z = static_cast<const T*>(p.z) + row * p.z_batch_stride + first;
    T* out = static_cast<T*>(p.out) + row * p.dim + first;
    float v[V][E], gate[V][E], sum[1] = {0.f};
#pragma unroll
    for (int i = 0; i < V; ++i) {
        load_vec<T, E>(y + (long long)clamped(i, vecs) * E, v[i]);
        load_vec<T, E>(z + (long long)clamped(i, vecs) * E, gate[i]);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (threadIdx.x + i * blockDim.x >= vecs) break;
#pragma unroll
        for (int j = 0; j < E; ++j) {
            gate[i][j] *= sscan::fast_sigmoid(gate[i][j]);
            if (!NORM_FIRST) v[i][j] *= gate[i][j];
            sum[0] = fmaf(v[i][j], v[i][j], sum[0]);
        }
    }
    cta_sum(sum, shared);
    const float rstd = rsqrtf(sum[0] / (float)size + p.eps);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int at = threadIdx.x + i * blockDim.x;
        if (at >= vecs) break;
        float w[E];
        load_vec<float, E>(p.w + first + (long long)at * E, w);
#pragma unroll
        for (int j = 0; j < E; ++j) {
            v[i][j] *= rstd * w[j];
            if (NORM_FIRST) v[i][j] *= gate[i][j];
        }
        store_vec<T, E>(out + (long long)at * E, v[i]);
    }
}

// ---- channel-major ----------------------------------------------------------
//
// The norm runs across rows that lie L elements apart, so a token's values come
// in pieces of as many bytes as the tile has tokens.  gatenorm_cluster_kernel
// reads them once: a cluster of CTAs holds a tile of all the group's channels in shared
// memory (each CTA its share of the channels), sums the squares, exchanges
// the sums through distributed shared memory, and finishes from what it holds.
// gatenorm_tile_kernel takes the groups too wide for that: it walks the
// channels twice.

// Threads of a CTA.  A thread's own cost (addresses, reductions) is worth about
// four vectors of work, so more threads repeat it and fewer leave the SM short
// of warps (4 x 2048 x 2048 bf16, forward and backward: 67.8 us; 76.9 with 128,
// 106.8 with 512).
constexpr int kGateThreads = 256;

// Column sums of a tile meet here: [partial][sum][token].
template <int NUM, int TT, int PARTS>
struct alignas(16) GateSums {
    float part[PARTS][NUM][TT];
    float cta[NUM][TT];    // over the CTA's channels, read by its cluster
    float total[NUM][TT];
};

// Tiles are 64 bytes of every row: 4 threads of 16 bytes (E tokens) a row.
// ALIGNED: rows of whole 16-byte vectors, staged and stored as such.  Otherwise
// a row is staged from the 16-byte boundary before it, a thread puts its tokens
// together from shared words, and results leave through the row's own place in
// shared memory, one token a lane.
template <typename T, bool ALIGNED, bool NORM_FIRST, bool BWD>
__global__ void __launch_bounds__(kGateThreads, ALIGNED ? (BWD ? 4 : 6) : (BWD ? 3 : 4)) gatenorm_cluster_kernel(const GateParams p) {
    constexpr int E = VecOf<T>::E;
    constexpr int TX = 4, TT = TX * E;            // threads across a row, tokens of a tile
    constexpr int RY = kGateThreads / TX;         // rows at a time
    constexpr int kChunks = TX + (ALIGNED ? 0 : 1);
    constexpr int kArrays = BWD ? 3 : 2;
    constexpr int NUM = BWD ? 2 : 1;
    constexpr int PARTS = kGateThreads / 32;
    __shared__ GateSums<NUM, TT, PARTS> sums;
    extern __shared__ __align__(16) unsigned char raw_rows[];
    uint4* rows = reinterpret_cast<uint4*>(raw_rows);  // [array][channel][chunk]

    cg::cluster_group cluster = cg::this_cluster();
    const unsigned ranks = cluster.num_blocks(), rank = cluster.block_rank();
    const unsigned tiles = (unsigned)((p.len + TT - 1) / TT), tile = blockIdx.x >> (31 - __clz((int)ranks));
    const long long b = blockIdx.z, group = blockIdx.y;
    const int size = p.size, share = p.share;
    const int first = (int)rank * share < size ? (int)rank * share : size;
    const int count = size - first < share ? size - first : share;  // the CTA's channels
    const long long d0 = group * size + first;
    const long long t0 = (long long)tile * TT;
    const T* src[3] = {static_cast<const T*>(p.y) + b * p.dim * p.len + d0 * p.len + t0,
                       static_cast<const T*>(p.z) + b * p.z_batch_stride + d0 * p.z_dim_stride + t0,
                       BWD ? static_cast<const T*>(p.dout) + b * p.dim * p.len + d0 * p.len + t0 : nullptr};
    const long long stride[3] = {p.len, p.z_dim_stride, p.len};
    const int left = p.len - t0 < TT ? (int)(p.len - t0) : TT;  // tokens of this tile
    // elements between a row and the 16-byte boundary before it
    int phase0[3], phase_step[3];
#pragma unroll
    for (int a = 0; a < kArrays; ++a) {
        phase0[a] = phase_of(src[a]);
        phase_step[a] = (int)stride[a];
    }
    auto phase = [&](int a, int r) { return (phase0[a] + (int)((unsigned)r * (unsigned)phase_step[a])) & (E - 1); };
#pragma unroll
    for (int a = 0; a < kArrays; ++a) {
        if (ALIGNED) {
            const int c = threadIdx.x % TX;
            const int bytes = c * E < left ? 16 : 0;
            const T* from = src[a] + threadIdx.x / TX * stride[a] + (bytes ? c * E : 0);
            uint4* to = rows + a * share * kChunks + threadIdx.x;
#pragma unroll 4
            for (int r = threadIdx.x / TX; r < count; r += RY) {
                sscan::cp_async16(to, from, bytes);
                to += kGateThreads;
                from += RY * stride[a];
            }
        } else {
            // whole chunks, with whatever lies beside the tile's tokens in them, but
            // for those that reach outside the array
            const T* lo = static_cast<const T*>(a == 0 ? p.y : a == 1 ? p.z : p.dout);
            const T* hi = lo + (p.batch - 1) * (a == 1 ? p.z_batch_stride : p.dim * p.len) + (p.dim - 1) * stride[a] + p.len;
            for (int i = threadIdx.x; i < count * kChunks; i += kGateThreads) {
                const int r = i / kChunks, c = i % kChunks;
                const T* from = src[a] + r * stride[a] + c * E - phase(a, r);
                uint4* to = rows + (a * share + r) * kChunks + c;
                if (from >= lo && from + E <= hi) {
                    sscan::cp_async16(to, from, 16);
                } else {
                    T* one = reinterpret_cast<T*>(to);
#pragma unroll 1
                    for (int j = 0; j < E; ++j)
                        one[j] = from + j >= lo && from + j < hi ? from[j] : sscan::from_f32<T>(0.f);
                }
            }
        }
    }
    sscan::cp_async_commit();
    sscan::cp_async_wait<0>();
    __syncthreads();

    const int tx = threadIdx.x % TX, ry = threadIdx.x / TX, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // the thread's tokens of row r of array a
    auto read = [&](int a, int r, float (&v)[E]) {
        const uint4* row = rows + (a * share + r) * kChunks;
        uint4 q;
        if constexpr (ALIGNED) {
            q = row[tx];
        } else {
            const int at = phase(a, r) + tx * E;
            const unsigned* word = reinterpret_cast<const unsigned*>(row) + at * (int)sizeof(T) / 4;
            if constexpr (E == 4) {
                q = make_uint4(word[0], word[1], word[2], word[3]);
            } else {
                const unsigned odd = (at & 1) * 16;  // an odd token is the upper half of its word
                // (the word after the last token is read only where it holds one)
                const unsigned last = odd ? word[4] : 0u;
                q = make_uint4(__funnelshift_r(word[0], word[1], odd), __funnelshift_r(word[1], word[2], odd),
                               __funnelshift_r(word[2], word[3], odd), __funnelshift_r(word[3], last, odd));
            }
        }
        sscan::widen(q, v, static_cast<T*>(nullptr));
        if (!ALIGNED && left < TT) {  // past the row's end lies another row
#pragma unroll
            for (int j = 0; j < E; ++j)
                if (tx * E + j >= left) v[j] = 0.f;
        }
    };
    float sum[NUM][E];
#pragma unroll
    for (int i = 0; i < NUM; ++i)
#pragma unroll
        for (int j = 0; j < E; ++j) sum[i][j] = 0.f;
    // Forward: y * silu(z) in fp32 takes the place of y and z, which is as large,
    // so that the gate is computed once.  Every thread walks the same number of
    // rows: a row's four threads read it before one of them writes.
    for (int r0 = 0; r0 < count; r0 += RY) {
        const int r = r0 + ry;
        const bool in = r < count;
        float v[E], g[E], q[E], w = 0.f;
        if (in) {
            read(0, r, v);
            read(1, r, g);
            if constexpr (BWD) {
                read(2, r, q);
                w = __ldg(p.w + d0 + r);
            }
        }
        if (!BWD && !ALIGNED) __syncwarp();
        if (!in) continue;
#pragma unroll
        for (int j = 0; j < E; ++j) {
            g[j] *= sscan::fast_sigmoid(g[j]);
            if (NORM_FIRST) sum[0][j] = fmaf(v[j], v[j], sum[0][j]);
            if (!NORM_FIRST || !BWD) v[j] *= g[j];
            if (!NORM_FIRST) sum[0][j] = fmaf(v[j], v[j], sum[0][j]);
            if constexpr (BWD) sum[1][j] = fmaf(NORM_FIRST ? q[j] * w * g[j] : q[j] * w, v[j], sum[1][j]);
        }
        if constexpr (!BWD) {
#pragma unroll
            for (int i = 0; i < E / 4; ++i)
                rows[(i * share + r) * kChunks + tx] = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
                                                                  __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3]));
        }
    }
    // The warp's eight rows: each exchange with the lane 16, 8 and 4 away halves
    // the tokens that a lane still sums (with four tokens the last one only adds),
    // so the 8 tokens take 7 shuffles and end one to a lane.
#pragma unroll
    for (int i = 0; i < NUM; ++i) {
        int token = tx * E;
#pragma unroll
        for (int n = E / 2, o = 16; o >= TX; o >>= 1, n >>= 1) {
            if (n > 0) {
                const bool upper = (lane & o) != 0;
#pragma unroll
                for (int j = 0; j < n; ++j) {
                    const float give = upper ? sum[i][j] : sum[i][j + n], keep = upper ? sum[i][j + n] : sum[i][j];
                    sum[i][j] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                }
                token += upper ? n : 0;
            } else {
                sum[i][0] += __shfl_xor_sync(0xffffffffu, sum[i][0], o);
            }
        }
        sums.part[warp][i][token] = sum[i][0];
    }
    __syncthreads();
    if (threadIdx.x < NUM * TT) {
        const int i = threadIdx.x / TT, t = threadIdx.x % TT;
        float a = 0.f;
#pragma unroll
        for (int k = 0; k < PARTS; ++k) a += sums.part[k][i][t];
        sums.cta[i][t] = a;
    }
    cluster.sync();
    if (threadIdx.x < NUM * TT) {
        float a = 0.f;
        for (unsigned k = 0; k < ranks; ++k) a += cluster.map_shared_rank(&sums.cta[0][0], k)[threadIdx.x];
        const int t = threadIdx.x % TT;
        a *= 1.f / (float)size;
        // 1 / sqrt(mean of squares + eps) (0 past the row's end), mean of q * v
        sums.total[threadIdx.x / TT][t] = threadIdx.x >= TT ? a : t < left ? rsqrtf(a + p.eps) : 0.f;
    }
    __syncthreads();
    // Results of the warp's 32 / TX rows: a thread's tokens as one vector, or,
    // unaligned, laid over the row's place in array a and stored one token a lane.
    const bool on = tx * E < left;
    auto write = [&](T* out, int a, int r0, int r, bool in, const float (&v)[E]) {
        if constexpr (ALIGNED) {
            if (in && on) store_vec<T, E>(out + r * p.len + tx * E, v);
        } else {
            if (in) rows[(a * share + r) * kChunks + tx] = sscan::narrow(v, static_cast<T*>(nullptr));
            __syncwarp();
            const int t = lane % TT;
#pragma unroll
            for (int k = lane / TT; k < 32 / TX; k += 32 / TT) {
                const int rk = r0 + warp * (32 / TX) + k;
                if (rk < count && t < left) out[rk * p.len + t] = reinterpret_cast<const T*>(rows + (a * share + rk) * kChunks)[t];
            }
        }
    };
    const long long base = b * p.dim * p.len + d0 * p.len + t0;
    float rstd[E];
#pragma unroll
    for (int j = 0; j < E; ++j) rstd[j] = sums.total[0][tx * E + j];
    if constexpr (!BWD) {
        T* out = static_cast<T*>(p.out) + base;
        for (int r0 = 0; r0 < count; r0 += RY) {
            const int r = r0 + ry;
            const bool in = r < count;
            float v[E];
            if (in) {
                const float w = __ldg(p.w + d0 + r);
#pragma unroll
                for (int i = 0; i < E / 4; ++i) {
                    const uint4 q = rows[(i * share + r) * kChunks + tx];
                    v[4 * i] = __uint_as_float(q.x); v[4 * i + 1] = __uint_as_float(q.y);
                    v[4 * i + 2] = __uint_as_float(q.z); v[4 * i + 3] = __uint_as_float(q.w);
                }
#pragma unroll
                for (int j = 0; j < E; ++j) v[j] *= rstd[j] * w;
            }
            if (!ALIGNED) __syncwarp();
            write(out, 0, r0, r, in, v);
            if (!ALIGNED) __syncwarp();
        }
    } else {
        T* dy = static_cast<T*>(p.dy) + base;
        T* dz = static_cast<T*>(p.dz) + base;
        float mean[E];  // mean of q * n
#pragma unroll
        for (int j = 0; j < E; ++j) mean[j] = sums.total[NUM - 1][tx * E + j] * rstd[j];
        float* parts = p.parts + (b * tiles + tile) * p.dim + d0;
        for (int r0 = 0; r0 < count; r0 += RY) {
            const int r = r0 + ry;
            const bool in = r < count;
            float v[E], g[E], q[E], dw = 0.f;
            if (in) {
                const float w = __ldg(p.w + d0 + r);
                read(0, r, v);
                read(1, r, g);
                read(2, r, q);
#pragma unroll
                for (int j = 0; j < E; ++j) {
                    const float s = sscan::fast_sigmoid(g[j]);
                    const float gate = g[j] * s, dsilu = fmaf(gate, 1.f - s, s);
                    const float up = NORM_FIRST ? q[j] * gate : q[j];  // gradient of n * w
                    const float n = (NORM_FIRST ? v[j] : v[j] * gate) * rstd[j];
                    const float dv = rstd[j] * fmaf(-n, mean[j], up * w);
                    dw = fmaf(up, n, dw);
                    g[j] = (NORM_FIRST ? q[j] * n * w : dv * v[j]) * dsilu;
                    v[j] = NORM_FIRST ? dv : dv * gate;
                }
            }
            if (!ALIGNED) __syncwarp();  // the rows have been read
            write(dy, 0, r0, r, in, v);
            write(dz, 1, r0, r, in, g);
            if (!ALIGNED) __syncwarp();
            dw = sscan::warp_sum<TX>(dw);
            if (in && tx == 0) parts[r] = dw;
        }
        sscan::griddep_launch_dependents();
    }
    // no CTA leaves while another may read its sums (nothing else needs to be
    // seen, so this does not wait for the stores)
    asm volatile("barrier.cluster.arrive.relaxed.aligned;\nbarrier.cluster.wait.aligned;\n" ::: "memory");
}

// A CTA owns 32 tokens of one (batch, group) and walks the group's channels
// twice: TX threads of E consecutive tokens by 256 / TX channels at a time.
constexpr int kTileTokens = 32;

template <typename T, int E>
__device__ __forceinline__ void load_tokens(const T* p, long long t, long long len, float (&v)[E]) {
    if constexpr (E == 1) {
        v[0] = t < len ? sscan::to_f32(p[t]) : 0.f;
    } else {
        if (t < len) {
            sscan::widen(*reinterpret_cast<const uint4*>(p + t), v, static_cast<T*>(nullptr));
        } else {
#pragma unroll
            for (int j = 0; j < E; ++j) v[j] = 0.f;
        }
    }
}
template <typename T, int E>
__device__ __forceinline__ void store_tokens(T* p, long long t, long long len, const float (&v)[E]) {
    if (t >= len) return;
    if constexpr (E == 1) p[t] = sscan::from_f32<T>(v[0]);
    else *reinterpret_cast<uint4*>(p + t) = sscan::narrow(v, static_cast<T*>(nullptr));
}

// Sum a[NUM][E] over the CTA's channel lanes, for each token; every thread gets its tokens' sums.
template <int E, int NUM>
__device__ __forceinline__ void channel_sum(float (&a)[NUM][E], float (*shared)[kTileTokens]) {
    constexpr int TX = kTileTokens / E;
    const int tx = threadIdx.x % TX, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < NUM; ++i)
#pragma unroll
        for (int j = 0; j < E; ++j)
#pragma unroll
            for (int o = 16; o >= TX; o >>= 1) a[i][j] += __shfl_xor_sync(0xffffffffu, a[i][j], o);
#pragma unroll
    for (int i = 0; i < NUM; ++i) {
        if (lane < TX) {
#pragma unroll
            for (int j = 0; j < E; ++j) shared[i * 8 + warp][tx * E + j] = a[i][j];
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NUM; ++i)
#pragma unroll
        for (int j = 0; j < E; ++j) {
            float s = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) s += shared[i * 8 + k][tx * E + j];
            a[i][j] = s;
        }
}

template <typename T, int E, bool NORM_FIRST, bool BWD>
__global__ void __launch_bounds__(256) gatenorm_tile_kernel(const GateParams p) {
    constexpr int TX = kTileTokens / E, CY = 256 / TX;
    __shared__ float shared[16][kTileTokens];
    const long long tiles = (p.len + kTileTokens - 1) / kTileTokens;
    const long long tile = blockIdx.x % tiles, b = blockIdx.x / tiles / p.groups, group = blockIdx.x / tiles % p.groups;
    const long long size = p.dim / p.groups, first = group * size;
    const int tx = threadIdx.x % TX, cy = threadIdx.x / TX;
    const long long t = tile * kTileTokens + tx * E;
    const T* y = static_cast<const T*>(p.y) + b * p.dim * p.len;
    const T* z = static_cast<const T*>(p.z) + b * p.z_batch_stride;
    const T* dout = static_cast<const T*>(p.dout) + b * p.dim * p.len;
    constexpr int NUM = BWD ? 2 : 1;
    float sum[NUM][E];
#pragma unroll
    for (int i = 0; i < NUM; ++i)
#pragma unroll
        for (int j = 0; j < E; ++j) sum[i][j] = 0.f;
    for (long long d = first + cy; d < first + size; d += CY) {
        float v[E], g[E];
        load_tokens<T, E>(y + d * p.len, t, p.len, v);
        if (!NORM_FIRST || BWD) load_tokens<T, E>(z + d * p.z_dim_stride, t, p.len, g);
#pragma unroll
        for (int j = 0; j < E; ++j) {
            if (!NORM_FIRST || BWD) g[j] *= sscan::fast_sigmoid(g[j]);
            if (!NORM_FIRST) v[j] *= g[j];
            sum[0][j] = fmaf(v[j], v[j], sum[0][j]);
        }
        if constexpr (BWD) {
            const float w = __ldg(p.w + d);
            float q[E];
            load_tokens<T, E>(dout + d * p.len, t, p.len, q);
#pragma unroll
            for (int j = 0; j < E; ++j) {
                q[j] *= w;
                if (NORM_FIRST) q[j] *= g[j];
                sum[1][j] = fmaf(q[j], v[j], sum[1][j]);
            }
        }
    }
    channel_sum<E, NUM>(sum, shared);
    float rstd[E];
#pragma unroll
    for (int j = 0; j < E; ++j) rstd[j] = t + j < p.len ? rsqrtf(sum[0][j] / (float)size + p.eps) : 0.f;
    if constexpr (!BWD) {
        T* out = static_cast<T*>(p.out) + b * p.dim * p.len;
        for (long long d = first + cy; d < first + size; d += CY) {
            float v[E], g[E];
            const float w = __ldg(p.w + d);
            load_tokens<T, E>(y + d * p.len, t, p.len, v);
            load_tokens<T, E>(z + d * p.z_dim_stride, t, p.len, g);
#pragma unroll
            for (int j = 0; j < E; ++j) v[j] *= g[j] * sscan::fast_sigmoid(g[j]) * rstd[j] * w;
            store_tokens<T, E>(out + d * p.len, t, p.len, v);
        }
    } else {
        T* dy = static_cast<T*>(p.dy) + b * p.dim * p.len;
        T* dz = static_cast<T*>(p.dz) + b * p.dim * p.len;
        float mean[E];  // mean of q * n
#pragma unroll
        for (int j = 0; j < E; ++j) mean[j] = sum[1][j] * rstd[j] / (float)size;
        float* parts = p.parts + (b * tiles + tile) * p.dim;
        // every thread walks the same number of channels: the warp sums below need them all
        for (long long d0 = first; d0 < first + size; d0 += CY) {
            const bool on = d0 + cy < first + size;
            const long long d = on ? d0 + cy : first + size - 1;
            float v[E], g[E], q[E], dw = 0.f;
            const float w = __ldg(p.w + d);
            load_tokens<T, E>(y + d * p.len, t, p.len, v);
            load_tokens<T, E>(z + d * p.z_dim_stride, t, p.len, g);
            load_tokens<T, E>(dout + d * p.len, t, p.len, q);
            float oy[E], oz[E];
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const float s = sscan::fast_sigmoid(g[j]);
                const float gate = g[j] * s, dsilu = s * fmaf(g[j], 1.f - s, 1.f);
                const float up = NORM_FIRST ? q[j] * gate : q[j];         // gradient of n * w
                const float n = (NORM_FIRST ? v[j] : v[j] * gate) * rstd[j];
                const float dv = rstd[j] * fmaf(-n, mean[j], up * w);
                dw = fmaf(up, n, dw);
                oy[j] = NORM_FIRST ? dv : dv * gate;
                oz[j] = (NORM_FIRST ? q[j] * n * w : dv * v[j]) * dsilu;
            }
            if (on) {
                store_tokens<T, E>(dy + d * p.len, t, p.len, oy);
                store_tokens<T, E>(dz + d * p.len, t, p.len, oz);
            }
#pragma unroll
            for (int o = TX / 2; o > 0; o >>= 1) dw += __shfl_xor_sync(0xffffffffu, dw, o);
            if (on && tx == 0) parts[d] = dw;
        }
        sscan::griddep_launch_dependents();
    }
}

// ---- host side --------------------------------------------------------------

constexpr long long kBig = 1LL << 40;
constexpr long long kGridMax = (1LL << 31) - 1;

bool sizes_ok(long long a, long long b, long long c) {
    return a >= 0 && b >= 0 && c >= 0 && a <= kBig && b <= kBig && c <= kBig && (!a || b <= kBig / a) &&
           (!(a * b) || c <= kBig / (a * b));
}

// Threads and vectors a thread for a row of `vecs` vectors of E elements: the
// fewest vectors a thread (1, 2, 4; four times that many single elements) for
// which the row fits 512 threads.  One vector a thread leaves registers for three backward CTAs an
// SM (8192 x 2560 bf16: backward 54.6 us, against 62.8 with two vectors in
// half the threads; forward 36.5 against 39.0).  Four single elements are few
// loads under way: eight from 1024 on (4096 x 1753 bf16 forward and backward
// 52 us, against 65 with four).
struct RowPlan { int threads, v; };
constexpr long long kOneVec = 512;
template <int E>
RowPlan plan_row(long long vecs) {
    const int m = E == 1 ? 4 : 1;
    int v = 4;
    if (vecs <= (E == 1 ? 1024 : kOneVec)) v = 1;
    else if (vecs <= 2 * kOneVec * m) v = 2;
    return {(int)sscan::div_up(sscan::div_up(vecs, v * m), 32) * 32, v};
}

cudaError_t column_sum(const float* parts, float* out, long long rows, long long cols, cudaStream_t st) {
    const bool wide = cols >= 152 * 32;
    return sscan::launch(wide ? column_sum_kernel<32> : column_sum_kernel<8>, dim3((unsigned)sscan::div_up(cols, wide ? 32 : 8)),
                         dim3(1024), 0, st, true, parts, out, rows, cols);
}

template <typename T, int E>
cudaError_t addnorm_fwd_launch(const AddNormParams& p, cudaStream_t st) {
    constexpr int M = E == 1 ? 4 : 1;
    const RowPlan pl = plan_row<E>(p.width / E);
    const dim3 grid((unsigned)(p.rows < kGridMax ? p.rows : kGridMax)), block(pl.threads);
    if (pl.v == 1) return sscan::launch(addnorm_fwd_kernel<T, E, M>, grid, block, 0, st, false, p);
    if (pl.v == 2) return sscan::launch(addnorm_fwd_kernel<T, E, 2 * M>, grid, block, 0, st, false, p);
    return sscan::launch(addnorm_fwd_kernel<T, E, 4 * M>, grid, block, 0, st, false, p);
}
template <typename T, int E>
cudaError_t addnorm_bwd_launch(const AddNormParams& p, const RowPlan& pl, int ctas, cudaStream_t st) {
    constexpr int M = E == 1 ? 4 : 1;
    const dim3 grid(ctas), block(pl.threads);
    if (pl.v == 1) return sscan::launch(addnorm_bwd_kernel<T, E, M>, grid, block, 0, st, false, p);
    if (pl.v == 2) return sscan::launch(addnorm_bwd_kernel<T, E, 2 * M>, grid, block, 0, st, false, p);
    return sscan::launch(addnorm_bwd_kernel<T, E, 4 * M>, grid, block, 0, st, false, p);
}
template <typename T, int E, bool NF>
cudaError_t gatenorm_rows_launch(const GateParams& p, cudaStream_t st) {
    constexpr int M = E == 1 ? 4 : 1;
    const RowPlan pl = plan_row<E>(p.dim / p.groups / E);
    const dim3 grid((unsigned)(p.batch * p.groups)), block(pl.threads);
    if (pl.v == 1) return sscan::launch(gatenorm_rows_kernel<T, E, M, NF>, grid, block, 0, st, false, p);
    if (pl.v == 2) return sscan::launch(gatenorm_rows_kernel<T, E, 2 * M, NF>, grid, block, 0, st, false, p);
    return sscan::launch(gatenorm_rows_kernel<T, E, 4 * M, NF>, grid, block, 0, st, false, p);
}
// Shared memory of a CTA's share at most, which is also every form's opt-in limit: the
// limit belongs to the kernel, not to the call, so all calls set the same one
// (host threads may be between their set-up and their launch).
constexpr long long kGateShared = 212 * 1024;

// CTAs of the cluster that shares a tile of a channel-major call, or 0 for the
// walk that reads its inputs twice.  The smallest cluster that leaves an SM room
// for several CTAs' shares (bf16 2048 channels: eight CTAs of 256), or the largest at all; a
// larger one while the grid leaves SMs idle.
template <typename T, bool BWD>
int gate_ranks(const GateParams& p, bool vec) {
    const long long size = p.dim / p.groups, tiles = sscan::div_up(p.len, 64 / (int)sizeof(T)) * p.batch * p.groups;
    auto bytes = [&](long long ranks) { return (BWD ? 3 : 2) * sscan::div_up(size, ranks) * (vec ? 64 : 80); };
    int ranks = 1;
    while (ranks < 8 && (bytes(ranks) > (BWD ? 52 : 36) * 1024 || (tiles * ranks < 304 && size / ranks >= 64))) ranks *= 2;
    // (groups and batch are the grid's second and third dimensions)
    return bytes(ranks) <= kGateShared && tiles * ranks <= kGridMax && p.groups <= 65535 && p.batch <= 65535 ? ranks : 0;
}
long long gate_part_rows(const GateParams& p, int ranks, int esz) {
    return p.batch * sscan::div_up(p.len, ranks > 0 ? 64 / esz : kTileTokens);
}

template <typename T, bool ALIGNED, bool NF, bool BWD>
cudaError_t gatenorm_cluster_launch(const GateParams& p0, int ranks, cudaStream_t st) {
    GateParams p = p0;
    p.size = (int)(p.dim / p.groups);
    p.share = (int)sscan::div_up(p.size, ranks);
    auto kernel = gatenorm_cluster_kernel<T, ALIGNED, NF, BWD>;
    const size_t smem = (size_t)((BWD ? 3 : 2) * p.share * (ALIGNED ? 64 : 80));
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kGateShared);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(sscan::div_up(p.len, 64 / (int)sizeof(T)) * ranks), (unsigned)p.groups, (unsigned)p.batch);
    cfg.blockDim = dim3(kGateThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ranks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}
template <typename T, bool ALIGNED, bool NF, bool BWD>
cudaError_t gatenorm_launch_as(const GateParams& p, int ranks, cudaStream_t st) {
    if (ranks > 0) return gatenorm_cluster_launch<T, ALIGNED, NF, BWD>(p, ranks, st);
    const dim3 grid((unsigned)(sscan::div_up(p.len, kTileTokens) * p.batch * p.groups));
    return sscan::launch(gatenorm_tile_kernel<T, ALIGNED ? VecOf<T>::E : 1, NF, BWD>, grid, dim3(256), 0, st, false, p);
}
template <typename T, bool BWD>
cudaError_t gatenorm_launch(const GateParams& p, int ranks, bool vec, bool norm_first, cudaStream_t st) {
    if (vec)
        return norm_first ? gatenorm_launch_as<T, true, true, BWD>(p, ranks, st) : gatenorm_launch_as<T, true, false, BWD>(p, ranks, st);
    return norm_first ? gatenorm_launch_as<T, false, true, BWD>(p, ranks, st) : gatenorm_launch_as<T, false, false, BWD>(p, ranks, st);
}

bool aligned_all(std::initializer_list<const void*> ptrs) {
    for (const void* p : ptrs)
        if (!sscan::is_aligned(p, 16)) return false;
    return true;
}

// CTAs of the persistent backward: what 152 SMs hold at about 60 registers a
// thread, 960 threads each (54.6 us as above; 63.3 with 640, 67.6 with 1280,
// which come in a second wave)
int bwd_ctas(long long rows, int threads) {
    const long long ctas = 152LL * std::max(1, 960 / threads);
    return (int)std::min(rows, ctas);
}

}  // namespace

extern "C" int addnorm_fwd(const void* x, const float* residual, const float* weight, void* y, float* residual_out,
                           int64_t rows, int64_t width, float scale, float eps, int dtype, void* stream) {
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    sscan::record_call(0, st, "rejected");
    if ((dtype != SSCAN_F32 && dtype != SSCAN_BF16) || !sizes_ok(rows, width, 1) || width < 1 || width > BLOCKNORM_MAX_WIDTH)
        return SSCAN_ERR_INVALID;
    if (rows == 0) {
        sscan::record_call(0, st, "empty");
        return SSCAN_OK;
    }
    if (!x || !weight || !y || !residual_out) return SSCAN_ERR_INVALID;
    AddNormParams p = {};
    p.x = x; p.residual = residual; p.w = weight; p.y = y; p.r = residual_out;
    p.rows = rows; p.width = (int)width; p.scale = scale; p.eps = eps;
    const bool vec = width % (dtype == SSCAN_F32 ? 4 : 8) == 0 && aligned_all({x, residual, weight, y, residual_out});
    sscan::record_call(1, st, vec ? "addnorm fwd vec=1" : "addnorm fwd vec=0");
    if (dtype == SSCAN_F32)
        return sscan::finish(vec ? addnorm_fwd_launch<float, 4>(p, st) : addnorm_fwd_launch<float, 1>(p, st));
    return sscan::finish(vec ? addnorm_fwd_launch<bf16, 8>(p, st) : addnorm_fwd_launch<bf16, 1>(p, st));
}

extern "C" int addnorm_bwd(const float* residual_out, const float* weight, const void* dy, const float* dresidual_out,
                           void* dx, float* dresidual, float* dweight, int64_t rows, int64_t width, float scale,
                           float eps, int dtype, void* stream) {
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    sscan::record_call(0, st, "rejected");
    if ((dtype != SSCAN_F32 && dtype != SSCAN_BF16) || !sizes_ok(rows, width, 1) || width < 1 || width > BLOCKNORM_MAX_WIDTH)
        return SSCAN_ERR_INVALID;
    if (!dweight || (rows && (!residual_out || !weight || !dy || !dx))) return SSCAN_ERR_INVALID;
    if (rows == 0) {
        sscan::record_call(0, st, "empty: dweight = 0");
        return sscan::finish(cudaMemsetAsync(dweight, 0, (size_t)width * sizeof(float), st));
    }
    AddNormParams p = {};
    p.r = const_cast<float*>(residual_out); p.w = weight; p.dy = dy; p.dr = dresidual_out; p.dx = dx;
    p.dresidual = dresidual; p.rows = rows; p.width = (int)width; p.scale = scale; p.eps = eps;
    const bool vec = width % (dtype == SSCAN_F32 ? 4 : 8) == 0 &&
                     aligned_all({residual_out, weight, dy, dresidual_out, dx, dresidual});
    const RowPlan pl = dtype == SSCAN_F32 ? (vec ? plan_row<4>(width / 4) : plan_row<1>(width))
                                          : (vec ? plan_row<8>(width / 8) : plan_row<1>(width));
    const int ctas = bwd_ctas(rows, pl.threads);
    void* parts = nullptr;
    cudaError_t e = sscan::scratch_alloc(&parts, (size_t)ctas * width * sizeof(float), st);
    if (e != cudaSuccess) return sscan::finish(e);
    p.parts = static_cast<float*>(parts);
    sscan::record_call(2, st, vec ? "addnorm bwd vec=1" : "addnorm bwd vec=0");
    if (dtype == SSCAN_F32) e = vec ? addnorm_bwd_launch<float, 4>(p, pl, ctas, st) : addnorm_bwd_launch<float, 1>(p, pl, ctas, st);
    else e = vec ? addnorm_bwd_launch<bf16, 8>(p, pl, ctas, st) : addnorm_bwd_launch<bf16, 1>(p, pl, ctas, st);
    if (e == cudaSuccess) e = column_sum(p.parts, dweight, ctas, width, st);
    const cudaError_t ef = cudaFreeAsync(parts, st);
    return sscan::finish(e != cudaSuccess ? e : ef);
}

namespace {
bool gate_ok(long long batch, long long dim, long long len, long long groups, int dtype, int flags) {
    return (dtype == SSCAN_F32 || dtype == SSCAN_BF16) && sizes_ok(batch, dim, len) && groups >= 1 &&
           (flags & ~GATENORM_NORM_FIRST) == 0 && dim % groups == 0 &&
           (!batch || !dim || groups * batch <= kGridMax / sscan::div_up(len > 0 ? len : 1, 16)) && dim <= kGridMax;
}
void record_gate(const char* what, int launches, int ranks, bool vec, cudaStream_t st) {
    char plan[64];
    snprintf(plan, sizeof(plan), "gatenorm %s cluster=%d vec=%d", what, ranks, vec ? 1 : 0);
    sscan::record_call(launches, st, plan);
}
}  // namespace

extern "C" int gatenorm_fwd(const void* y, const void* z, const float* weight, void* out, int64_t batch, int64_t dim,
                            int64_t seqlen, int64_t groups, int64_t z_batch_stride, int64_t z_dim_stride, float eps,
                            int dtype, int flags, void* stream) {
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    sscan::record_call(0, st, "rejected");
    if (!gate_ok(batch, dim, seqlen, groups, dtype, flags) || z_batch_stride < 0 || z_dim_stride < 0)
        return SSCAN_ERR_INVALID;
    if (batch == 0 || dim == 0 || seqlen == 0) {
        sscan::record_call(0, st, "empty");
        return SSCAN_OK;
    }
    if (!y || !z || !weight || !out) return SSCAN_ERR_INVALID;
    GateParams p = {};
    p.y = y; p.z = z; p.w = weight; p.out = out;
    p.batch = batch; p.dim = dim; p.len = seqlen; p.groups = groups;
    p.z_batch_stride = z_batch_stride; p.z_dim_stride = z_dim_stride; p.eps = eps;
    const int e = dtype == SSCAN_F32 ? 4 : 8;
    const bool vec = seqlen % e == 0 && z_batch_stride % e == 0 && z_dim_stride % e == 0 && aligned_all({y, z, out});
    const bool nf = (flags & GATENORM_NORM_FIRST) != 0;
    const int ranks = dtype == SSCAN_F32 ? gate_ranks<float, false>(p, vec) : gate_ranks<bf16, false>(p, vec);
    record_gate("fwd", 1, ranks, vec, st);
    return sscan::finish(dtype == SSCAN_F32 ? gatenorm_launch<float, false>(p, ranks, vec, nf, st)
                                            : gatenorm_launch<bf16, false>(p, ranks, vec, nf, st));
}

extern "C" int gatenorm_bwd(const void* y, const void* z, const float* weight, const void* dout, void* dy, void* dz,
                            float* dweight, int64_t batch, int64_t dim, int64_t seqlen, int64_t groups,
                            int64_t z_batch_stride, int64_t z_dim_stride, float eps, int dtype, int flags,
                            void* stream) {
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    sscan::record_call(0, st, "rejected");
    if (!gate_ok(batch, dim, seqlen, groups, dtype, flags) || z_batch_stride < 0 || z_dim_stride < 0)
        return SSCAN_ERR_INVALID;
    if (dim == 0) {
        sscan::record_call(0, st, "empty");
        return SSCAN_OK;
    }
    if (!dweight) return SSCAN_ERR_INVALID;
    if (batch == 0 || seqlen == 0) {
        sscan::record_call(0, st, "empty: dweight = 0");
        return sscan::finish(cudaMemsetAsync(dweight, 0, (size_t)dim * sizeof(float), st));
    }
    if (!y || !z || !weight || !dout || !dy || !dz) return SSCAN_ERR_INVALID;
    GateParams p = {};
    p.y = y; p.z = z; p.w = weight; p.dout = dout; p.dy = dy; p.dz = dz;
    p.batch = batch; p.dim = dim; p.len = seqlen; p.groups = groups;
    p.z_batch_stride = z_batch_stride; p.z_dim_stride = z_dim_stride; p.eps = eps;
    const int e = dtype == SSCAN_F32 ? 4 : 8;
    const bool vec = seqlen % e == 0 && z_batch_stride % e == 0 && z_dim_stride % e == 0 && aligned_all({y, z, dout, dy, dz});
    const int ranks = dtype == SSCAN_F32 ? gate_ranks<float, true>(p, vec) : gate_ranks<bf16, true>(p, vec);
    const long long part_rows = gate_part_rows(p, ranks, dtype == SSCAN_F32 ? 4 : 2);
    void* parts = nullptr;
    cudaError_t err = sscan::scratch_alloc(&parts, (size_t)(part_rows * dim) * sizeof(float), st);
    if (err != cudaSuccess) return sscan::finish(err);
    p.parts = static_cast<float*>(parts);
    record_gate("bwd", 2, ranks, vec, st);
    const bool nf = (flags & GATENORM_NORM_FIRST) != 0;
    err = dtype == SSCAN_F32 ? gatenorm_launch<float, true>(p, ranks, vec, nf, st)
                             : gatenorm_launch<bf16, true>(p, ranks, vec, nf, st);
    if (err == cudaSuccess) err = column_sum(p.parts, dweight, part_rows, dim, st);
    const cudaError_t ef = cudaFreeAsync(parts, st);
    return sscan::finish(err != cudaSuccess ? err : ef);
}

extern "C" int gatenorm_step(const void* y, const void* z, const float* weight, void* out, int64_t rows, int64_t dim,
                             int64_t groups, int64_t z_stride, float eps, int dtype, int flags, void* stream) {
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    sscan::record_call(0, st, "rejected");
    if (!gate_ok(rows, dim, 1, groups, dtype, flags) || z_stride < 0) return SSCAN_ERR_INVALID;
    if (rows == 0 || dim == 0) {
        sscan::record_call(0, st, "empty");
        return SSCAN_OK;
    }
    if (!y || !z || !weight || !out) return SSCAN_ERR_INVALID;
    GateParams p = {};
    p.y = y; p.z = z; p.w = weight; p.out = out;
    p.batch = rows; p.dim = dim; p.len = 1; p.groups = groups;
    p.z_batch_stride = z_stride; p.eps = eps;
    const long long size = dim / groups;
    p.size = (int)size;
    const int e = dtype == SSCAN_F32 ? 4 : 8;
    const bool vec = size % e == 0 && z_stride % e == 0 && aligned_all({y, z, weight, out});
    if (size > BLOCKNORM_MAX_WIDTH) return SSCAN_ERR_INVALID;
    const bool nf = (flags & GATENORM_NORM_FIRST) != 0;
    sscan::record_call(1, st, vec ? "gatenorm step vec=1" : "gatenorm step vec=0");
    if (dtype == SSCAN_F32) {
        if (vec) return sscan::finish(nf ? gatenorm_rows_launch<float, 4, true>(p, st) : gatenorm_rows_launch<float, 4, false>(p, st));
        return sscan::finish(nf ? gatenorm_rows_launch<float, 1, true>(p, st) : gatenorm_rows_launch<float, 1, false>(p, st));
    }
    if (vec) return sscan::finish(nf ? gatenorm_rows_launch<bf16, 8, true>(p, st) : gatenorm_rows_launch<bf16, 8, false>(p, st));
    return sscan::finish(nf ? gatenorm_rows_launch<bf16, 1, true>(p, st) : gatenorm_rows_launch<bf16, 1, false>(p, st));
}
