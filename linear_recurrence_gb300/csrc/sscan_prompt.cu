// Selective scan over packed prompts with a state cache, on sm_103a.
//
// The tokens of several requests lie end to end along the time axis; each
// request's recurrence starts from its cache row (or zeros) and leaves its
// last state there:
//   h_t[n] = exp(dt_t*A[d,n]) * h_{t-1}[n] + dt_t*u_t*B_t[n],   y_t = sum_n C_t[n]*h_t[n] + D*u_t
// with dt = delta, or softplus(delta + bias), and y gated by silu(z) where given.
//
// The packed axis is cut into equal segments, whatever the requests' lengths,
// so that ragged prompts load the GPU evenly.  A state that crosses a segment
// border is found first, by a pass that walks each segment backwards:
//   h_end[n] = sum_t exp(A[n] * S_t) * dt_t*u_t*B_t[n],   S_t = sum of dt after t in the segment
// has no step-to-step dependence, and once A[n]*S_t < -kCutBits*ln 2 for a warp's
// states and channels, the rest of the segment contributes less than 2^-kCutBits of
// what it adds up and the walk ends.  Decay rates grow with n, so
// most states need a few dozen tokens.  The scan pass then starts every
// segment from the composed states of the ones before (again only as far back
// as they matter), writes each output once, rounded once, and needs no
// correction afterwards.  Steps dt must be >= 0 for the cut-off to hold (the
// domain of the scan's time splits everywhere in this library); rates A >= 0 never
// meet it and are followed to the request's start.
//
// An element (token, channel, state) takes one exponential and four fp32
// operations in the scan pass, which bounds it by issue slots: 152 SMs x 128
// lanes / 5 at 2.07 GHz is 8.06 T elements/s; bytes are a tenth of that time.
#include <stdio.h>

#include "block_utils.cuh"

namespace {

using sscan::bf16;
using sscan::Requests;
using sscan::VecOf;

constexpr int kTile = 16;                 // tokens staged at a time
constexpr int kPitch = kTile + 4;         // floats per staged row: 16-byte reads of 8 rows meet all banks once
constexpr float kCutBits = 40.f;          // 2^-40 of the sum: below fp32 resolution with 16 bits to spare
constexpr int kStates = 8;                // states of a thread in the scan pass
constexpr int kChannels = 2;              // channels of a thread in the scan pass
constexpr int kWarps = 4;                 // warps of a scan CTA

struct PromptParams {
    const void* u;
    const void* delta;
    const float* A;
    const void* B;
    const void* C;
    const float* D;
    const void* z;
    const float* bias;
    float* state;
    void* out;
    long long dim;
    int tokens, N;
    int seg_tokens, segments;
    int softplus;
    // scratch of a split: per segment, the end state [dim, N], the carried-in
    // request's saved initial state [dim, N], and sum of dt [dim, groups of 4 states]
    float* h_end;
    float* h_first;
    float* dt_sum;
    Requests req;
};

// Raw elements of one row around [t0, t0 + kTile), as they lie in memory:
// 16-byte chunks from the boundary at or below the first.  The row's first
// token then sits `phase` elements into the staged row.
template <typename T> constexpr int kRawPitch = kTile + (16 / (int)sizeof(T));
template <typename T> constexpr int kRawChunks = kRawPitch<T> * (int)sizeof(T) / 16;
template <typename T>
__device__ __forceinline__ int row_phase(const T* p) {
    return (int)((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T));
}
// One chunk of a row starting at element `row` + t0 (t0 a multiple of kTile):
// asynchronous when it lies inside [lo, hi), element by element at the
// tensor's ends.
template <typename T>
__device__ __forceinline__ void stage_chunk(T* dst, const T* first, int chunk, const T* lo, const T* hi) {
    constexpr int E = VecOf<T>::E;
    const T* src = reinterpret_cast<const T*>(reinterpret_cast<uintptr_t>(first) & ~(uintptr_t)15u) + chunk * E;
    if (src >= lo && src + E <= hi) {
        sscan::cp_async16(dst + chunk * E, src, 16);
    } else {
#pragma unroll
        for (int j = 0; j < E; ++j) dst[chunk * E + j] = src + j >= lo && src + j < hi ? src[j] : sscan::from_f32<T>(0.f);
    }
}

// ---- states at segment ends -------------------------------------------------

// A CTA takes 32 channels of one segment; warp w the states 4w .. 4w+3 of all
// of them (lane = channel), so that warps of fast-decaying states stop early.
constexpr int kEndStates = 4;

template <typename T>
struct EndShared {
    alignas(16) T u[2][32][kRawPitch<T>];
    alignas(16) T d[2][32][kRawPitch<T>];
    alignas(16) float dt[32][kPitch];
    alignas(16) float du[32][kPitch];
    alignas(16) float B[kTile][64];
};

template <typename T>
__global__ void __launch_bounds__(512) sscan_prompt_ends_kernel(const PromptParams p) {
    __shared__ EndShared<T> sh;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, threads = blockDim.x;
    const int seg = blockIdx.y;
    const long long d0 = (long long)blockIdx.x * 32;
    const long long d = d0 + lane < p.dim ? d0 + lane : p.dim - 1;
    const bool mine = d0 + lane < p.dim;
    const int begin = seg * p.seg_tokens;
    const int end = begin + p.seg_tokens;  // a border inside the tokens: the last segment is not walked
    if (blockIdx.x == 0 && seg == 0) p.req.check(threadIdx.x, threads);
    sscan::griddep_launch_dependents();
    // the request that crosses the border, if any
    const int s = p.req.find(end - 1);
    const bool in_request = s >= 0 && s < p.req.requests;
    int from = s < 0 ? 0 : p.req.offset(s);
    const int until = s < 0 ? p.req.offset(0) : in_request ? p.req.offset(s + 1) : p.tokens;
    if (until <= end) return;  // it ends at the border: nothing is carried
    const bool starts_here = from >= begin;
    const int stop = starts_here ? from : begin;

    const int n0 = warp * kEndStates;
    float a[kEndStates], h[kEndStates], amax = -INFINITY;
#pragma unroll
    for (int i = 0; i < kEndStates; ++i) {
        a[i] = n0 + i < p.N ? p.A[d * p.N + n0 + i] * sscan::kLog2e : -INFINITY;
        amax = fmaxf(amax, a[i]);
        if (a[i] == -INFINITY) a[i] = 0.f;
        h[i] = 0.f;
    }
    float S = 0.f;
    const T* u = static_cast<const T*>(p.u);
    const T* delta = static_cast<const T*>(p.delta);
    const T* Bm = static_cast<const T*>(p.B);
    const T* hi = u + p.dim * p.tokens;
    const T* dhi = delta + p.dim * p.tokens;
    auto stage = [&](int t0, int buf) {
        for (int i = threadIdx.x; i < 32 * kRawChunks<T>; i += threads) {
            const int r = i / kRawChunks<T>, c = i % kRawChunks<T>;
            const long long dr = d0 + r < p.dim ? d0 + r : p.dim - 1;
            const T* ru = u + dr * p.tokens + t0;
            const T* rd = delta + dr * p.tokens + t0;
            stage_chunk(sh.u[buf][r], ru, c, u, hi);
            stage_chunk(sh.d[buf][r], rd, c, delta, dhi);
        }
        sscan::cp_async_commit();
    };
    bool done = n0 >= p.N;
    int t0 = (end - 1) / kTile * kTile, buf = 0;
    stage(t0, 0);
    for (; t0 + kTile > stop; t0 -= kTile, buf ^= 1) {
        if (t0 > stop) stage(t0 - kTile, buf ^ 1);
        else sscan::cp_async_commit();
        sscan::cp_async_wait<1>();
        __syncthreads();
        for (int i = threadIdx.x; i < 32 * kTile; i += threads) {
            const int r = i / kTile, j = i % kTile, t = t0 + j;
            const long long dr = d0 + r < p.dim ? d0 + r : p.dim - 1;
            float dt = 0.f, du = 0.f;
            if (t >= stop && t < end) {
                dt = sscan::to_f32(sh.d[buf][r][row_phase(delta + dr * p.tokens + t0) + j]);
                if (p.bias != nullptr) dt += __ldg(p.bias + dr);
                if (p.softplus) dt = sscan::softplus_f32(dt);
                du = dt * sscan::to_f32(sh.u[buf][r][row_phase(u + dr * p.tokens + t0) + j]);
            }
            sh.dt[r][j] = dt;
            sh.du[r][j] = du;
        }
        for (int i = threadIdx.x; i < p.N * kTile; i += threads) {
            const int n = i / kTile, j = i % kTile, t = t0 + j;
            sh.B[j][n] = t >= stop && t < end ? sscan::to_f32(Bm[(long long)n * p.tokens + t]) : 0.f;
        }
        for (int i = threadIdx.x; i < kTile * 64; i += threads)  // states past N
            if (i % 64 >= p.N) sh.B[i / 64][i % 64] = 0.f;
        __syncthreads();
        if (!done) {
#pragma unroll
            for (int j4 = kTile - 4; j4 >= 0; j4 -= 4) {
                float dt[4], du[4];
                sscan::load4_smem(&sh.dt[lane][j4], dt);
                sscan::load4_smem(&sh.du[lane][j4], du);
#pragma unroll
                for (int j = 3; j >= 0; --j) {
                    float b[4];
                    sscan::load4_smem(&sh.B[j4 + j][n0], b);
#pragma unroll
                    for (int i = 0; i < kEndStates; ++i) h[i] = fmaf(sscan::ex2(a[i] * S), du[j] * b[i], h[i]);
                    S += dt[j];
                }
            }
            done = __all_sync(0xffffffffu, !mine || amax * S < -kCutBits);
        }
        if (__syncthreads_and(done)) break;
    }
    sscan::cp_async_wait<0>();
    const int slot = in_request && starts_here ? p.req.slot(s) : -1;
    const bool cont = slot >= 0 && p.req.continues(s);
    if (n0 < p.N && mine) {
        const long long at = ((long long)seg * p.dim + d) * p.N + n0;
#pragma unroll
        for (int i = 0; i < kEndStates; ++i) {
            if (n0 + i >= p.N) break;
            float first = 0.f;
            if (starts_here) {  // kept for the scan pass, which may find the cache row already updated
                if (cont) first = p.state[((long long)slot * p.dim + d) * p.N + n0 + i];
                p.h_first[at + i] = first;
                if (cont) h[i] = fmaf(sscan::ex2(a[i] * S), first, h[i]);
            }
            p.h_end[at + i] = h[i];
        }
        const int groups = (p.N + kEndStates - 1) / kEndStates;
        p.dt_sum[((long long)seg * p.dim + d) * groups + warp] = S;
    }
}

// ---- the scan ----------------------------------------------------------------

// P lanes share a channel (8 states each); a thread advances 2 channels, so
// that a B or C value read from shared memory serves two elements.  A warp's
// channels are its own from staging to the store: only B and C are shared by
// the CTA.
template <typename T, int P, bool GATED>
struct ScanShared {
    static constexpr int kRows = 32 / P * kChannels;  // channels of a warp
    alignas(16) T u[kWarps][2][kRows][kRawPitch<T>];
    alignas(16) T d[kWarps][2][kRows][kRawPitch<T>];
    alignas(16) T z[kWarps][2][GATED ? kRows : 1][kRawPitch<T>];
    alignas(16) float dt[kWarps][kRows][kPitch];
    alignas(16) float du[kWarps][kRows][kPitch];  // dt * u, then the outputs
    alignas(16) float B[2][kTile][P * kStates];
    alignas(16) float C[2][kTile][P * kStates];
};

template <typename T, int P, bool GATED>
__global__ void __launch_bounds__(kWarps * 32) sscan_prompt_kernel(const PromptParams p) {
    using Sh = ScanShared<T, P, GATED>;
    constexpr int kRows = Sh::kRows, NP = P * kStates, kThreads = kWarps * 32;
    extern __shared__ __align__(16) unsigned char raw_shared[];
    Sh& sh = *reinterpret_cast<Sh*>(raw_shared);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int seg = blockIdx.y;
    const long long d0 = ((long long)blockIdx.x * kWarps + warp) * kRows;  // the warp's first channel
    const int part = lane % P, n0 = part * kStates;
    const int row0 = lane / P;  // the thread's channels: rows row0 and row0 + 32 / P
    const int begin = seg * p.seg_tokens;
    const int end = begin + p.seg_tokens < p.tokens ? begin + p.seg_tokens : p.tokens;
    const T* u = static_cast<const T*>(p.u);
    const T* delta = static_cast<const T*>(p.delta);
    const T* z = static_cast<const T*>(p.z);
    const T* Bm = static_cast<const T*>(p.B);
    const T* Cm = static_cast<const T*>(p.C);
    T* out = static_cast<T*>(p.out);
    const long long total = p.dim * p.tokens;
    auto row_of = [&](int r) { return d0 + r < p.dim ? d0 + r : p.dim - 1; };

    auto stage = [&](int t0, int buf) {
        for (int i = lane; i < kRows * kRawChunks<T>; i += 32) {
            const int r = i / kRawChunks<T>, c = i % kRawChunks<T>;
            const long long at = row_of(r) * p.tokens + t0;
            stage_chunk(sh.u[warp][buf][r], u + at, c, u, u + total);
            stage_chunk(sh.d[warp][buf][r], delta + at, c, delta, delta + total);
            if (GATED) stage_chunk(sh.z[warp][buf][r], z + at, c, z, z + total);
        }
        sscan::cp_async_commit();
    };
    // B and C of a tile: read into registers a tile ahead, stored transposed
    constexpr int kBC = NP * kTile / kThreads;
    float bq[kBC], cq[kBC];
    auto fetch_bc = [&](int t0) {
#pragma unroll
        for (int i = 0; i < kBC; ++i) {
            const int at = threadIdx.x + i * kThreads, n = at / kTile, t = t0 + at % kTile;
            const bool on = n < p.N && t < p.tokens;
            bq[i] = on ? sscan::to_f32(Bm[(long long)n * p.tokens + t]) : 0.f;
            cq[i] = on ? sscan::to_f32(Cm[(long long)n * p.tokens + t]) : 0.f;
        }
    };
    auto store_bc = [&](int buf) {
#pragma unroll
        for (int i = 0; i < kBC; ++i) {
            const int at = threadIdx.x + i * kThreads;
            sh.B[buf][at % kTile][at / kTile] = bq[i];
            sh.C[buf][at % kTile][at / kTile] = cq[i];
        }
    };
    if (p.segments == 1 && blockIdx.x == 0) p.req.check(threadIdx.x, kThreads);
    stage(begin, 0);
    fetch_bc(begin);
    store_bc(0);

    long long ch[kChannels];
    bool mine[kChannels];
    float a[kChannels][kStates], h[kChannels][kStates];
#pragma unroll
    for (int c = 0; c < kChannels; ++c) {
        const long long d = d0 + row0 + c * (32 / P);
        mine[c] = d < p.dim;
        ch[c] = mine[c] ? d : p.dim - 1;
#pragma unroll
        for (int i = 0; i < kStates; ++i) {
            a[c][i] = n0 + i < p.N ? p.A[ch[c] * p.N + n0 + i] * sscan::kLog2e : 0.f;
            h[c][i] = 0.f;
        }
    }
    auto load_state = [&](const float* from) {  // [dim, N]
#pragma unroll
        for (int c = 0; c < kChannels; ++c)
#pragma unroll
            for (int i = 0; i < kStates; ++i) h[c][i] = n0 + i < p.N ? from[ch[c] * p.N + n0 + i] : 0.f;
    };
    auto keep_state = [&](int s) {
        if (s < 0 || s >= p.req.requests) return;
        const int slot = p.req.slot(s);
        if (slot < 0) return;
#pragma unroll
        for (int c = 0; c < kChannels; ++c)
#pragma unroll
            for (int i = 0; i < kStates; ++i)
                if (mine[c] && n0 + i < p.N) p.state[((long long)slot * p.dim + ch[c]) * p.N + n0 + i] = h[c][i];
    };
    // the state of request s before its first token, at a token of this segment
    auto enter = [&](int s) {
        const int slot = s >= 0 && s < p.req.requests && p.req.continues(s) ? p.req.slot(s) : -1;
        if (slot < 0) {
#pragma unroll
            for (int c = 0; c < kChannels; ++c)
#pragma unroll
                for (int i = 0; i < kStates; ++i) h[c][i] = 0.f;
        } else if (p.req.offset(s + 1) > begin + p.seg_tokens) {
            load_state(p.h_first + (long long)seg * p.dim * p.N);  // another CTA writes its cache row
        } else {
            load_state(p.state + (long long)slot * p.dim * p.N);
        }
    };

    sscan::griddep_wait();  // the end states, and the cache rows they were read from
    if (seg == 0) {  // requests without tokens that begin anew: their state is zero
        for (int s = 0; s < p.req.requests && p.req.has != nullptr; ++s)
            if (p.req.offset(s + 1) <= p.req.offset(s) && !p.req.continues(s)) keep_state(s);
    }
    int cur = p.req.find(begin);
    auto start_of = [&](int s) { return s < 0 ? 0 : p.req.offset(s); };
    auto end_of = [&](int s) { return s < 0 ? p.req.offset(0) : s < p.req.requests ? p.req.offset(s + 1) : p.tokens; };
    if (start_of(cur) >= begin) {
        enter(cur);
    } else {
        // compose the segments before, from the nearest, down to the one where
        // the request starts
        const int first = start_of(cur) / p.seg_tokens;
        const int groups = (p.N + kEndStates - 1) / kEndStates;
        float e[kChannels][kStates];  // exponents of the decay so far
#pragma unroll
        for (int c = 0; c < kChannels; ++c)
#pragma unroll
            for (int i = 0; i < kStates; ++i) e[c][i] = 0.f;
        for (int g = seg - 1; g >= first; --g) {
            bool live = false;
#pragma unroll
            for (int c = 0; c < kChannels; ++c) {
                const long long at = ((long long)g * p.dim + ch[c]);
#pragma unroll
                for (int i = 0; i < kStates; ++i) {
                    if (n0 + i >= p.N) continue;
                    h[c][i] = fmaf(sscan::ex2(e[c][i]), p.h_end[at * p.N + n0 + i], h[c][i]);
                    e[c][i] = fmaf(a[c][i], p.dt_sum[at * groups + (n0 + i) / kEndStates], e[c][i]);
                    live |= e[c][i] >= -kCutBits;
                }
            }
            if (!__any_sync(0xffffffffu, live)) break;
        }
    }
    int next = end_of(cur);  // the next token that begins another request

    for (int t0 = begin, buf = 0; t0 < end; t0 += kTile, buf ^= 1) {
        const bool more = t0 + kTile < end;
        if (more) {
            stage(t0 + kTile, buf ^ 1);
            fetch_bc(t0 + kTile);
        } else {
            sscan::cp_async_commit();
        }
        sscan::cp_async_wait<1>();
        __syncwarp();
        for (int i = lane; i < kRows * kTile; i += 32) {
            const int r = i / kTile, j = i % kTile;
            const long long dr = row_of(r);
            float dt = sscan::to_f32(sh.d[warp][buf][r][row_phase(delta + dr * p.tokens + t0) + j]);
            if (p.bias != nullptr) dt += __ldg(p.bias + dr);
            if (p.softplus) dt = sscan::softplus_f32(dt);
            sh.dt[warp][r][j] = dt;
            sh.du[warp][r][j] = dt * sscan::to_f32(sh.u[warp][buf][r][row_phase(u + dr * p.tokens + t0) + j]);
        }
        __syncthreads();  // B and C of this tile
        const int limit = end - t0 < kTile ? end - t0 : kTile;
#pragma unroll 1
        for (int j4 = 0; j4 < limit; j4 += 4) {
            float dt[kChannels][4], du[kChannels][4], y[kChannels][4];
#pragma unroll
            for (int c = 0; c < kChannels; ++c) {
                sscan::load4_smem(&sh.dt[warp][row0 + c * (32 / P)][j4], dt[c]);
                sscan::load4_smem(&sh.du[warp][row0 + c * (32 / P)][j4], du[c]);
            }
            const bool border = next < t0 + j4 + 4 || t0 + j4 + 4 > end;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                bool skip = false;
                if (border) {
                    skip = t0 + j4 + j >= end;
                    if (!skip && t0 + j4 + j == next) {
                        keep_state(cur);
                        cur = p.req.find(next);
                        enter(cur);
                        next = end_of(cur);
                    }
                }
                float b[kStates], cc[kStates];
#pragma unroll
                for (int i = 0; i < kStates; i += 4) {
                    const float4 bv = *reinterpret_cast<const float4*>(&sh.B[buf][j4 + j][n0 + i]);
                    const float4 cv = *reinterpret_cast<const float4*>(&sh.C[buf][j4 + j][n0 + i]);
                    b[i] = bv.x; b[i + 1] = bv.y; b[i + 2] = bv.z; b[i + 3] = bv.w;
                    cc[i] = cv.x; cc[i + 1] = cv.y; cc[i + 2] = cv.z; cc[i + 3] = cv.w;
                }
#pragma unroll
                for (int c = 0; c < kChannels; ++c) {
                    y[c][j] = 0.f;
                    if (skip) continue;
#pragma unroll
                    for (int i = 0; i < kStates; ++i) {
                        h[c][i] = fmaf(sscan::ex2(dt[c][j] * a[c][i]), h[c][i], du[c][j] * b[i]);
                        y[c][j] = fmaf(cc[i], h[c][i], y[c][j]);
                    }
                }
            }
#pragma unroll
            for (int c = 0; c < kChannels; ++c)
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int o = 1; o < P; o <<= 1) y[c][j] += __shfl_xor_sync(0xffffffffu, y[c][j], o);
            // the lanes of a channel have all read du; its place takes the outputs
            if (part == 0) {
#pragma unroll
                for (int c = 0; c < kChannels; ++c)
                    *reinterpret_cast<float4*>(&sh.du[warp][row0 + c * (32 / P)][j4]) =
                        make_float4(y[c][0], y[c][1], y[c][2], y[c][3]);
            }
        }
        __syncwarp();
        for (int i = lane; i < kRows * kTile; i += 32) {
            const int r = i / kTile, j = i % kTile, t = t0 + j;
            if (t >= end || d0 + r >= p.dim) continue;
            const long long at = (d0 + r) * p.tokens;
            float y = sh.du[warp][r][j];
            if (p.D != nullptr) y = fmaf(__ldg(p.D + d0 + r), sscan::to_f32(sh.u[warp][buf][r][row_phase(u + at + t0) + j]), y);
            if (GATED) {
                const float g = sscan::to_f32(sh.z[warp][buf][r][row_phase(z + at + t0) + j]);
                y *= g * sscan::fast_sigmoid(g);
            }
            out[at + t] = sscan::from_f32<T>(y);
        }
        if (more) store_bc(buf ^ 1);
        __syncwarp();
    }
    if (next == end) keep_state(cur);
}

// ---- host side ----------------------------------------------------------------

constexpr long long kBig = 1LL << 40;
constexpr long long kIntMax = 1LL << 30;  // token, request and channel numbers are 32-bit on the device

bool sizes_ok(long long a, long long b, long long c) {
    return a >= 0 && b >= 0 && c >= 0 && a <= kBig && b <= kBig && c <= kBig && (!a || b <= kBig / a) &&
           (!(a * b) || c <= kBig / (a * b));
}

template <typename T, int P, bool GATED>
cudaError_t run_scan(const PromptParams& p, bool dependent, cudaStream_t st) {
    constexpr size_t bytes = sizeof(ScanShared<T, P, GATED>);
    static_assert(bytes <= 227 * 1024, "shared memory of a CTA");
    const cudaError_t e = cudaFuncSetAttribute(sscan_prompt_kernel<T, P, GATED>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)sscan::div_up(p.dim, kWarps * ScanShared<T, P, GATED>::kRows), (unsigned)p.segments);
    return sscan::launch(sscan_prompt_kernel<T, P, GATED>, grid, dim3(kWarps * 32), bytes, st, dependent, p);
}
template <typename T, int P>
cudaError_t run_gated(const PromptParams& p, bool dependent, cudaStream_t st) {
    return p.z != nullptr ? run_scan<T, P, true>(p, dependent, st) : run_scan<T, P, false>(p, dependent, st);
}
template <typename T>
cudaError_t run_all(const PromptParams& p, cudaStream_t st) {
    cudaError_t e = cudaSuccess;
    const bool split = p.segments > 1;
    if (split) {
        const dim3 grid((unsigned)sscan::div_up(p.dim, 32), (unsigned)(p.segments - 1));
        e = sscan::launch(sscan_prompt_ends_kernel<T>, grid, dim3(32 * (unsigned)sscan::div_up(p.N, kEndStates)), 0, st,
                          false, p);
        if (e != cudaSuccess) return e;
    }
    if (p.N <= 8) return run_gated<T, 1>(p, split, st);
    if (p.N <= 16) return run_gated<T, 2>(p, split, st);
    if (p.N <= 32) return run_gated<T, 4>(p, split, st);
    return run_gated<T, 8>(p, split, st);
}

}  // namespace

extern "C" int sscan_prompt(const void* u, const void* delta, const float* A, const void* B, const void* C,
                            const float* D, const void* z, const float* delta_bias, const int32_t* cu_seqlens,
                            const int32_t* slots, const uint8_t* has_state, float* state, void* out, int64_t requests,
                            int64_t num_slots, int64_t dim, int64_t tokens, int64_t dstate, int dtype, int flags,
                            int segments, void* stream) {
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    sscan::record_call(0, st, "rejected");
    if (dtype != SSCAN_F32 && dtype != SSCAN_BF16) return SSCAN_ERR_INVALID;
    if (dstate < 1 || dstate > sscan_max_dstate() || segments < 0 || (flags & ~SSCAN_DELTA_SOFTPLUS)) return SSCAN_ERR_INVALID;
    if (!sizes_ok(1, dim, tokens) || !sizes_ok(num_slots, dim, dstate) || !sizes_ok(1, tokens, dstate)) return SSCAN_ERR_INVALID;
    if (requests < 0 || requests > kIntMax || tokens > kIntMax || num_slots > kIntMax || dim > kIntMax ||
        (slots == nullptr && requests > num_slots))
        return SSCAN_ERR_INVALID;
    if (dim == 0 || (requests == 0 && tokens == 0)) {
        sscan::record_call(0, st, "empty");
        return SSCAN_OK;
    }
    if (!cu_seqlens || (num_slots && !state) || !A || (tokens && (!u || !delta || !B || !C || !out))) return SSCAN_ERR_INVALID;
    int* status = sscan::device_status_word();
    if (status == nullptr) return sscan::finish(cudaErrorUnknown);
    PromptParams p = {};
    p.u = u; p.delta = delta; p.A = A; p.B = B; p.C = C; p.D = D; p.z = z; p.bias = delta_bias; p.state = state; p.out = out;
    p.dim = dim; p.tokens = (int)tokens; p.N = (int)dstate;
    p.softplus = flags & SSCAN_DELTA_SOFTPLUS;
    p.req = Requests{cu_seqlens, slots, has_state, (int)requests, (int)num_slots, (int)tokens, status};
    const int lanes = dstate <= 8 ? 1 : dstate <= 16 ? 2 : dstate <= 32 ? 4 : 8;
    const long long tiles = sscan::div_up(dim, kWarps * (32 / lanes) * kChannels);
    long long want = segments;
    if (want == 0) want = sscan::div_up(3 * 152, tiles);  // about three CTAs on every SM
    long long chunks = sscan::div_up(tokens > 0 ? tokens : 1, kTile);
    long long per = sscan::div_up(chunks, want < 1 ? 1 : want);
    if (segments == 0 && per < 4) per = 4;
    if (per > chunks) per = chunks;
    while (sscan::div_up(chunks, per) > 65535) per *= 2;
    p.seg_tokens = (int)(per * kTile);
    p.segments = (int)sscan::div_up(chunks, per);
    void* scratch = nullptr;
    if (p.segments > 1) {
        const size_t cells = (size_t)p.segments * (size_t)dim;
        const size_t groups = (size_t)sscan::div_up(dstate, kEndStates);
        const cudaError_t e = sscan::scratch_alloc(&scratch, cells * (2 * (size_t)dstate + groups) * sizeof(float), st);
        if (e != cudaSuccess) return sscan::finish(e);
        p.h_end = static_cast<float*>(scratch);
        p.h_first = p.h_end + cells * (size_t)dstate;
        p.dt_sum = p.h_first + cells * (size_t)dstate;
    }
    char plan[96];
    snprintf(plan, sizeof(plan), "sscan prompt lanes=%d segments=%d of %d", lanes, p.segments, p.seg_tokens);
    sscan::record_call(p.segments > 1 ? 2 : 1, st, plan);
    cudaError_t e = dtype == SSCAN_F32 ? run_all<float>(p, st) : run_all<bf16>(p, st);
    if (scratch != nullptr) {
        const cudaError_t ef = cudaFreeAsync(scratch, st);
        if (e == cudaSuccess) e = ef;
    }
    return sscan::finish(e);
}
