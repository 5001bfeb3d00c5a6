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
        float r[V][E], sum[1] = {0.f};
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int at = threadIdx.x + i * blockDim.x;
            if (at >= vecs) break;
            float a[E];
            load_vec<T, E>(x + (long long)at * E, a);
            if (p.residual != nullptr) {
                load_vec<float, E>(p.residual + row * p.width + (long long)at * E, r[i]);
#pragma unroll
                for (int j = 0; j < E; ++j) r[i][j] = fmaf(p.scale, a[j], r[i][j]);
            } else {
#pragma unroll
                for (int j = 0; j < E; ++j) r[i][j] = p.scale * a[j];
            }
#pragma unroll
            for (int j = 0; j < E; ++j) sum[0] = fmaf(r[i][j], r[i][j], sum[0]);
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
            const int at = threadIdx.x + i * blockDim.x;
            if (at >= vecs) break;
            load_vec<float, E>(p.r + row * p.width + (long long)at * E, r[i]);
            load_vec<T, E>(static_cast<const T*>(p.dy) + row * p.width + (long long)at * E, g[i]);
            if (p.dr != nullptr) {
                load_vec<float, E>(p.dr + row * p.width + (long long)at * E, d[i]);
            } else {
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

// out[c] = sum over rows of parts[row, c], in a fixed order: 32 warps take
// every 32nd row of 32 columns, then meet in shared memory.
__global__ void __launch_bounds__(1024) column_sum_kernel(const float* parts, float* out, long long rows, long long cols) {
    __shared__ float part[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long c = (long long)blockIdx.x * 32 + lane;
    sscan::griddep_wait();
    float a = 0.f;
    if (c < cols) {
#pragma unroll 4
        for (long long r = warp; r < rows; r += 32) a += parts[r * cols + c];
    }
    part[lane][warp] = a;
    __syncthreads();
    a = sscan::warp_sum(part[warp][lane]);  // column `warp` of the 32
    const long long mine = (long long)blockIdx.x * 32 + warp;
    if (lane == 0 && mine < cols) out[mine] = a;
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
    long long z_batch_stride, z_dim_stride;
    float eps;
};

// One row of a group: CTA per (row, group) of [rows, dim].
template <typename T, int E, int V, bool NORM_FIRST>
__global__ void __launch_bounds__(kRowThreads<E>) gatenorm_rows_kernel(const GateParams p) {
    __shared__ float shared[32];
    const long long size = p.dim / p.groups;
    const long long row = blockIdx.x / p.groups, first = blockIdx.x % p.groups * size;
    const int vecs = (int)(size / E);
    const T* y = static_cast<const T*>(p.y) + row * p.dim + first;
    const T* z = static_cast<const T*>(p.z) + row * p.z_batch_stride + first;
    T* out = static_cast<T*>(p.out) + row * p.dim + first;
    float v[V][E], gate[V][E], sum[1] = {0.f};
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int at = threadIdx.x + i * blockDim.x;
        if (at >= vecs) break;
        load_vec<T, E>(y + (long long)at * E, v[i]);
        load_vec<T, E>(z + (long long)at * E, gate[i]);
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

// Column sums of a tile meet here: [partial][sum][token].
template <int NUM, int TT, int PARTS>
struct GateSums {
    float part[PARTS][NUM][TT];
    float cta[NUM][TT];    // over the CTA's channels, read by its cluster
    float total[NUM][TT];
};

// T: I/O type; TT: tokens of a tile; ALIGNED: rows of whole 16-byte vectors (a
// thread then takes E consecutive tokens of a row, otherwise one).
template <typename T, int TT, bool ALIGNED, bool NORM_FIRST, bool BWD>
__global__ void __launch_bounds__(256) gatenorm_cluster_kernel(const GateParams p) {
    constexpr int E = VecOf<T>::E;
    constexpr int N = ALIGNED ? E : 1;            // tokens of a thread
    constexpr int TX = TT / N;                    // threads across a row
    constexpr int RY = 256 / TX;                  // rows at a time
    constexpr int kChunks = TT / E + (ALIGNED ? 0 : 1);
    constexpr int kArrays = BWD ? 3 : 2;
    constexpr int NUM = BWD ? 2 : 1;
    constexpr int PARTS = TX > 32 ? RY : 8;
    __shared__ GateSums<NUM, TT, PARTS> sums;
    extern __shared__ __align__(16) unsigned char raw_rows[];
    uint4* rows = reinterpret_cast<uint4*>(raw_rows);  // [array][channel][chunk]

    cg::cluster_group cluster = cg::this_cluster();
    const unsigned ranks = cluster.num_blocks(), rank = cluster.block_rank();
    const unsigned tiles = (unsigned)((p.len + TT - 1) / TT);
    const unsigned id = blockIdx.x / ranks;
    const unsigned tile = id % tiles;
    const long long b = id / tiles / p.groups, group = id / tiles % p.groups;
    const int size = (int)(p.dim / p.groups);
    const int share = (size + (int)ranks - 1) / (int)ranks;
    const int first = (int)rank * share < size ? (int)rank * share : size;
    const int count = size - first < share ? size - first : share;  // the CTA's channels
    const long long d0 = group * size + first;
    const long long t0 = (long long)tile * TT;
    const T* src[3] = {static_cast<const T*>(p.y) + b * p.dim * p.len + d0 * p.len + t0,
                       static_cast<const T*>(p.z) + b * p.z_batch_stride + d0 * p.z_dim_stride + t0,
                       BWD ? static_cast<const T*>(p.dout) + b * p.dim * p.len + d0 * p.len + t0 : nullptr};
    const long long stride[3] = {p.len, p.z_dim_stride, p.len};
    const int left = p.len - t0 < TT ? (int)(p.len - t0) : TT;  // tokens of this tile
#pragma unroll
    for (int a = 0; a < kArrays; ++a) {
        if (ALIGNED) {  // 256 / kChunks rows at a time
            const int c = threadIdx.x % kChunks;
            const int bytes = c * E < left ? 16 : 0;
            const T* from = src[a] + threadIdx.x / kChunks * stride[a] + (bytes ? c * E : 0);
            uint4* to = rows + a * share * kChunks + threadIdx.x;
#pragma unroll 4
            for (int r = threadIdx.x / kChunks; r < count; r += 256 / kChunks) {
                sscan::cp_async16(to, from, bytes);
                to += 256;
                from += 256 / kChunks * stride[a];
            }
        } else {
            for (int i = threadIdx.x; i < count * kChunks; i += 256) {
                const int r = i / kChunks, c = i % kChunks;
                const T* row = src[a] + r * stride[a];
                uint4* to = rows + (a * share + r) * kChunks + c;
                const int at = c * E - phase_of(row);  // token of the chunk's first element
                if (at >= 0 && at + E <= left) {
                    sscan::cp_async16(to, row + at, 16);
                } else {
                    T* one = reinterpret_cast<T*>(to);
#pragma unroll
                    for (int j = 0; j < E; ++j)
                        one[j] = at + j >= 0 && at + j < left ? row[at + j] : sscan::from_f32<T>(0.f);
                }
            }
        }
    }
    sscan::cp_async_commit();
    sscan::cp_async_wait<0>();
    __syncthreads();

    const int tx = threadIdx.x % TX, ry = threadIdx.x / TX, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto read = [&](int a, int r, float (&v)[N]) {
        if constexpr (ALIGNED) {
            sscan::widen(rows[(a * share + r) * kChunks + tx], v, static_cast<T*>(nullptr));
        } else {
            const T* row = reinterpret_cast<const T*>(rows + (a * share + r) * kChunks);
            v[0] = sscan::to_f32(row[phase_of(src[a] + r * stride[a]) + tx]);
        }
    };
    float sum[NUM][N];
#pragma unroll
    for (int i = 0; i < NUM; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j) sum[i][j] = 0.f;
    // forward, aligned: y * silu(z) in fp32 takes the place of y and z, which
    // is as large, so that the gate is computed once
    constexpr bool kKeep = !BWD && ALIGNED;
#pragma unroll 2
    for (int r = ry; r < count; r += RY) {
        float v[N], g[N];
        read(0, r, v);
        if (!NORM_FIRST || BWD || kKeep) read(1, r, g);
#pragma unroll
        for (int j = 0; j < N; ++j) {
            if (!NORM_FIRST || BWD || kKeep) g[j] *= sscan::fast_sigmoid(g[j]);
            if (NORM_FIRST) sum[0][j] = fmaf(v[j], v[j], sum[0][j]);
            if (!NORM_FIRST || kKeep) v[j] *= g[j];
            if (!NORM_FIRST) sum[0][j] = fmaf(v[j], v[j], sum[0][j]);
        }
        if constexpr (kKeep) {
#pragma unroll
            for (int i = 0; i < N / 4; ++i)
                rows[(i * share + r) * kChunks + tx] = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
                                                                  __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3]));
        }
        if constexpr (BWD) {
            const float w = __ldg(p.w + d0 + r);
            float q[N];
            read(2, r, q);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                q[j] *= w;
                if (NORM_FIRST) q[j] *= g[j];
                sum[1][j] = fmaf(q[j], v[j], sum[1][j]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < NUM; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j) {
#pragma unroll
            for (int o = 16; o >= TX; o >>= 1) sum[i][j] += __shfl_xor_sync(0xffffffffu, sum[i][j], o);
            if (lane < TX) sums.part[TX > 32 ? ry : warp][i][tx * N + j] = sum[i][j];
        }
    __syncthreads();
    for (int i = threadIdx.x; i < NUM * TT; i += 256) {
        float a = 0.f;
#pragma unroll
        for (int k = 0; k < PARTS; ++k) a += sums.part[k][i / TT][i % TT];
        sums.cta[i / TT][i % TT] = a;
    }
    cluster.sync();
    for (int i = threadIdx.x; i < NUM * TT; i += 256) {
        float a = 0.f;
        for (unsigned k = 0; k < ranks; ++k) a += cluster.map_shared_rank(&sums.cta[0][0], k)[i];
        sums.total[i / TT][i % TT] = a;
    }
    __syncthreads();
    float rstd[N], mean[N];  // 1 / sqrt(mean of squares + eps), mean of q * n
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const bool on = tx * N + j < left;
        rstd[j] = on ? rsqrtf(sums.total[0][tx * N + j] / (float)size + p.eps) : 0.f;
        mean[j] = BWD ? sums.total[NUM - 1][tx * N + j] * rstd[j] / (float)size : 0.f;
    }
    const bool on = tx * N < left;
    if constexpr (!BWD) {
        T* out = static_cast<T*>(p.out) + b * p.dim * p.len + d0 * p.len + t0 + tx * N;
#pragma unroll 2
        for (int r = ry; r < count; r += RY) {
            float v[N];
            const float w = __ldg(p.w + d0 + r);
            if constexpr (kKeep) {
#pragma unroll
                for (int i = 0; i < N / 4; ++i) {
                    const uint4 q = rows[(i * share + r) * kChunks + tx];
                    v[4 * i] = __uint_as_float(q.x); v[4 * i + 1] = __uint_as_float(q.y);
                    v[4 * i + 2] = __uint_as_float(q.z); v[4 * i + 3] = __uint_as_float(q.w);
                }
            } else {
                float g[N];
                read(0, r, v);
                read(1, r, g);
#pragma unroll
                for (int j = 0; j < N; ++j) v[j] *= g[j] * sscan::fast_sigmoid(g[j]);
            }
#pragma unroll
            for (int j = 0; j < N; ++j) v[j] *= rstd[j] * w;
            if (on) store_vec<T, N>(out + r * p.len, v);
        }
    } else {
        T* dy = static_cast<T*>(p.dy) + b * p.dim * p.len + d0 * p.len + t0 + tx * N;
        T* dz = static_cast<T*>(p.dz) + b * p.dim * p.len + d0 * p.len + t0 + tx * N;
        // a tile wider than a warp leaves one row of weight sums for each half
        constexpr int kHalves = TX > 32 ? TX / 32 : 1;
        float* parts = p.parts + ((b * tiles + tile) * kHalves + (TX > 32 ? warp % kHalves : 0)) * p.dim + d0;
        // every thread walks the same number of channels: the warp sums below need them all
        for (int r0 = 0; r0 < count; r0 += RY) {
            const bool in = r0 + ry < count;
            const int r = in ? r0 + ry : count - 1;
            float v[N], g[N], q[N], dw = 0.f;
            const float w = __ldg(p.w + d0 + r);
            read(0, r, v);
            read(1, r, g);
            read(2, r, q);
            float oy[N], oz[N];
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float s = sscan::fast_sigmoid(g[j]);
                const float gate = g[j] * s, dsilu = s * fmaf(g[j], 1.f - s, 1.f);
                const float up = NORM_FIRST ? q[j] * gate : q[j];  // gradient of n * w
                const float n = (NORM_FIRST ? v[j] : v[j] * gate) * rstd[j];
                const float dv = rstd[j] * fmaf(-n, mean[j], up * w);
                dw = fmaf(up, n, dw);
                oy[j] = NORM_FIRST ? dv : dv * gate;
                oz[j] = (NORM_FIRST ? q[j] * n * w : dv * v[j]) * dsilu;
            }
            if (in && on) {
                store_vec<T, N>(dy + r * p.len, oy);
                store_vec<T, N>(dz + r * p.len, oz);
            }
            dw = sscan::warp_sum<(TX < 32 ? TX : 32)>(dw);
            if (in && lane % (TX < 32 ? TX : 32) == 0) parts[r] = dw;
        }
        sscan::griddep_launch_dependents();
    }
    cluster.sync();  // no CTA leaves while another reads its sums
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
// half the threads; forward 36.5 against 39.0).
struct RowPlan { int threads, v; };
constexpr long long kOneVec = 512;
template <int E>
RowPlan plan_row(long long vecs) {
    const int m = E == 1 ? 4 : 1;
    int v = 4;
    if (vecs <= kOneVec * m) v = 1;
    else if (vecs <= 2LL * kOneVec * m) v = 2;
    return {(int)sscan::div_up(sscan::div_up(vecs, v * m), 32) * 32, v};
}

cudaError_t column_sum(const float* parts, float* out, long long rows, long long cols, cudaStream_t st) {
    return sscan::launch(column_sum_kernel, dim3((unsigned)sscan::div_up(cols, 32)), dim3(1024), 0, st, true, parts, out,
                         rows, cols);
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
// How a channel-major call runs: a cluster of `ranks` CTAs with `tokens`
// tokens a tile, or (ranks 0) the walk that reads its inputs twice.
struct GatePlan {
    int ranks, tokens;
    long long part_rows;  // rows of weight-gradient sums
};
// Rows of 128 bytes where the CTAs' shares of a tile leave room for two (three
// forward) CTAs an SM, else of 64 bytes, up to one CTA an SM; the smallest
// cluster that does, or a larger one while the grid leaves SMs idle.
template <typename T, bool BWD>
GatePlan plan_gate(const GateParams& p, bool vec) {
    const long long size = p.dim / p.groups;
    const int wide = 128 / (int)sizeof(T);
    auto bytes = [&](long long ranks, int tokens) {
        return (BWD ? 3 : 2) * sscan::div_up(size, ranks) * (tokens * (long long)sizeof(T) + (vec ? 0 : 16));
    };
    auto part_rows = [&](int tokens) { return p.batch * sscan::div_up(p.len, tokens) * (vec || tokens <= 32 ? 1 : tokens / 32); };
    const long long roomy = BWD ? 104 * 1024 : 70 * 1024, most = 216 * 1024;
    for (const long long limit : {roomy, most})
        for (int tokens = wide; tokens >= wide / 2; tokens /= 2)
            for (int ranks = 1; ranks <= 8; ranks *= 2) {
                if (bytes(ranks, tokens) > limit) continue;
                const long long tiles = sscan::div_up(p.len, tokens) * p.batch * p.groups;
                while (ranks < 8 && tiles * ranks < 304 && size / ranks >= 64) ranks *= 2;
                if (tiles * ranks > kGridMax) break;
                return {ranks, tokens, part_rows(tokens)};
            }
    return {0, kTileTokens, part_rows(kTileTokens)};
}

template <typename T, int TT, bool ALIGNED, bool NF, bool BWD>
cudaError_t gatenorm_cluster_launch(const GateParams& p, int ranks, cudaStream_t st) {
    auto kernel = gatenorm_cluster_kernel<T, TT, ALIGNED, NF, BWD>;
    const long long share = sscan::div_up(p.dim / p.groups, ranks);
    const size_t smem = (size_t)((BWD ? 3 : 2) * share * (TT * (long long)sizeof(T) + (ALIGNED ? 0 : 16)));
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(sscan::div_up(p.len, TT) * p.batch * p.groups * ranks));
    cfg.blockDim = dim3(256);
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
cudaError_t gatenorm_launch_as(const GateParams& p, const GatePlan& pl, cudaStream_t st) {
    constexpr int wide = 128 / (int)sizeof(T);
    if (pl.ranks > 0)
        return pl.tokens == wide ? gatenorm_cluster_launch<T, wide, ALIGNED, NF, BWD>(p, pl.ranks, st)
                                 : gatenorm_cluster_launch<T, wide / 2, ALIGNED, NF, BWD>(p, pl.ranks, st);
    const dim3 grid((unsigned)(sscan::div_up(p.len, kTileTokens) * p.batch * p.groups));
    return sscan::launch(gatenorm_tile_kernel<T, ALIGNED ? VecOf<T>::E : 1, NF, BWD>, grid, dim3(256), 0, st, false, p);
}
template <typename T, bool BWD>
cudaError_t gatenorm_launch(const GateParams& p, const GatePlan& pl, bool vec, bool norm_first, cudaStream_t st) {
    if (vec)
        return norm_first ? gatenorm_launch_as<T, true, true, BWD>(p, pl, st) : gatenorm_launch_as<T, true, false, BWD>(p, pl, st);
    return norm_first ? gatenorm_launch_as<T, false, true, BWD>(p, pl, st) : gatenorm_launch_as<T, false, false, BWD>(p, pl, st);
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
void record_gate(const char* what, int launches, const GatePlan& pl, bool vec, cudaStream_t st) {
    char plan[64];
    snprintf(plan, sizeof(plan), "gatenorm %s cluster=%d tokens=%d vec=%d", what, pl.ranks, pl.tokens, vec ? 1 : 0);
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
    const GatePlan pl = dtype == SSCAN_F32 ? plan_gate<float, false>(p, vec) : plan_gate<bf16, false>(p, vec);
    record_gate("fwd", 1, pl, vec, st);
    return sscan::finish(dtype == SSCAN_F32 ? gatenorm_launch<float, false>(p, pl, vec, nf, st)
                                            : gatenorm_launch<bf16, false>(p, pl, vec, nf, st));
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
    const GatePlan pl = dtype == SSCAN_F32 ? plan_gate<float, true>(p, vec) : plan_gate<bf16, true>(p, vec);
    void* parts = nullptr;
    cudaError_t err = sscan::scratch_alloc(&parts, (size_t)(pl.part_rows * dim) * sizeof(float), st);
    if (err != cudaSuccess) return sscan::finish(err);
    p.parts = static_cast<float*>(parts);
    record_gate("bwd", 2, pl, vec, st);
    const bool nf = (flags & GATENORM_NORM_FIRST) != 0;
    err = dtype == SSCAN_F32 ? gatenorm_launch<float, true>(p, pl, vec, nf, st)
                             : gatenorm_launch<bf16, true>(p, pl, vec, nf, st);
    if (err == cudaSuccess) err = column_sum(p.parts, dweight, pl.part_rows, dim, st);
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
