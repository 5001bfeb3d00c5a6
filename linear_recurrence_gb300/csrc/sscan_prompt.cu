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
constexpr float kCutBits = 30.f;          // 2^-30 of the sum: a 64th of an fp32 rounding
constexpr int kStates = 8;                // states of a thread in the scan pass
constexpr int kChannels = 2;              // channels of a thread in the scan pass
constexpr int kWarps = 4;                 // warps of a scan CTA
// CTAs an SM holds by registers: four (128 registers a thread) but for one
// lane a channel, whose 64 rows a warp leave room for two by shared memory.
template <int P> constexpr int kResident = P == 1 ? 2 : 4;

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

// Offset of tokens j .. j+3 (j a multiple of 4) of row r in an fp32 tile of
// kTile floats a row: the row's four 16-byte pieces are permuted by the row, so
// that eight neighbouring rows' pieces of the same tokens lie in distinct banks.
__device__ __forceinline__ int piece(int r, int j) { return r * kTile + (j ^ ((r >> 1 & 3) << 2)); }

// A row's elements [t0, t0 + kTile) are staged as they lie in memory.  ALIGNED
// (rows of whole 16-byte vectors): exactly those.  Otherwise 16-byte chunks
// from the boundary at or below the first, which then sits `phase` elements
// into the staged row; the phase depends on the row, not on t0.
template <typename T, bool ALIGNED> constexpr int kRawPitch = kTile + (ALIGNED ? 0 : 16 / (int)sizeof(T));
template <typename T, bool ALIGNED> constexpr int kRawChunks = kTile * (int)sizeof(T) / 16 + (ALIGNED ? 0 : 1);

template <typename T>
struct RawRows {
    const T* base;   // row 0 of the CTA's (or warp's) rows
    const T* lo;     // the whole array: [lo, hi)
    const T* hi;
    int tokens;
    int phase0;
    __device__ __forceinline__ RawRows(const void* array, long long row0, long long rows, int n)
        : base(static_cast<const T*>(array) + row0 * n), lo(static_cast<const T*>(array)), hi(lo + rows * n), tokens(n),
          phase0((int)((reinterpret_cast<uintptr_t>(base) & 15u) / sizeof(T))) {}
    __device__ __forceinline__ int phase(int r) const {
        return (phase0 + (int)((unsigned)r * (unsigned)tokens)) & (VecOf<T>::E - 1);
    }
    // chunk c of row r at t0 of an unaligned array, asynchronously where it lies inside the array
    __device__ __forceinline__ void stage(T* dst, int r, int c, int t0) const {
        constexpr int E = VecOf<T>::E;
        const T* src = base + (long long)r * tokens + t0 + c * E - phase(r);
        if (src >= lo && src + E <= hi) {
            sscan::cp_async16(dst + c * E, src, 16);
        } else {
#pragma unroll
            for (int j = 0; j < E; ++j)
                dst[c * E + j] = src + j >= lo && src + j < hi ? src[j] : sscan::from_f32<T>(0.f);
        }
    }
    // four values from token j on
    template <bool ALIGNED>
    __device__ __forceinline__ void read4(const T* row, int r, int j, float (&v)[4]) const {
        if (ALIGNED) {
            sscan::load4_smem(row + j, v);
        } else {
            const T* at = row + phase(r) + j;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = sscan::to_f32(at[i]);
        }
    }
};

__device__ __forceinline__ void store4(float* p, const float (&v)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(bf16* p, const float (&v)[4]) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(v[0], v[1]), hi = __floats2bfloat162_rn(v[2], v[3]);
    *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const unsigned*>(&lo), *reinterpret_cast<const unsigned*>(&hi));
}

// ---- states at segment ends -------------------------------------------------

// A CTA takes 32 channels of one segment; warp w the states 4w .. 4w+3 of all
// of them (lane = channel), so that warps of fast-decaying states stop early.
constexpr int kEndStates = 4;

template <typename T, bool ALIGNED>
struct EndShared {
    alignas(16) T u[2][32][kRawPitch<T, ALIGNED>];
    alignas(16) T d[2][32][kRawPitch<T, ALIGNED>];
    alignas(16) float dt[32 * kTile];
    alignas(16) float du[32 * kTile];
    alignas(16) float B[kTile][64];
};

template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(512) sscan_prompt_ends_kernel(const PromptParams p) {
    __shared__ EndShared<T, ALIGNED> sh;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, threads = blockDim.x;
    const int seg = blockIdx.y;
    const long long d0 = (long long)blockIdx.x * 32;
    const int rows = p.dim - d0 < 32 ? (int)(p.dim - d0) : 32;
    const bool mine = lane < rows;
    const long long d = d0 + (mine ? lane : rows - 1);
    const int begin = seg * p.seg_tokens;
    const int end = begin + p.seg_tokens;  // a border inside the tokens: the last segment is not walked
    if (blockIdx.x == 0 && seg == 0) p.req.check(threadIdx.x, threads);
    sscan::griddep_launch_dependents();
    // the request that crosses the border, if any
    const int s = p.req.find(end - 1);
    const bool in_request = s >= 0 && s < p.req.requests;
    const int from = s < 0 ? 0 : p.req.offset(s);
    const int until = s < 0 ? p.req.offset(0) : in_request ? p.req.offset(s + 1) : p.tokens;
    if (until <= end) return;  // it ends at the border: nothing is carried
    const bool starts_here = from >= begin;
    const int stop = starts_here ? from : begin;

    const int n0 = warp * kEndStates;
    float a[kEndStates], h[kEndStates], amax = -INFINITY;
#pragma unroll
    for (int i = 0; i < kEndStates; ++i) {
        a[i] = n0 + i < p.N ? p.A[d * p.N + n0 + i] * sscan::kLog2e : 0.f;
        if (n0 + i < p.N) amax = fmaxf(amax, a[i]);
        h[i] = 0.f;
    }
    float S = 0.f;
    const RawRows<T> u(p.u, d0, p.dim, p.tokens), delta(p.delta, d0, p.dim, p.tokens);
    const T* Bm = static_cast<const T*>(p.B);
    constexpr int kChunks = kRawChunks<T, ALIGNED>;
    auto stage = [&](int t0, int buf) {
        for (int i = threadIdx.x; i < 32 * kChunks; i += threads) {
            const int r = i / kChunks, c = i % kChunks;
            if (r >= rows) continue;
            if (ALIGNED) {
                if (t0 + c * VecOf<T>::E >= p.tokens) continue;
                const long long at = (long long)r * p.tokens + t0 + c * VecOf<T>::E;
                sscan::cp_async16(&sh.u[buf][r][c * VecOf<T>::E], u.base + at, 16);
                sscan::cp_async16(&sh.d[buf][r][c * VecOf<T>::E], delta.base + at, 16);
            } else {
                u.stage(sh.u[buf][r], r, c, t0);
                delta.stage(sh.d[buf][r], r, c, t0);
            }
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
        for (int i = threadIdx.x; i < 32 * (kTile / 4); i += threads) {
            const int r = i / (kTile / 4), j4 = i % (kTile / 4) * 4;
            if (r >= rows) continue;
            float dt[4], du[4];
            delta.template read4<ALIGNED>(sh.d[buf][r], r, j4, dt);
            u.template read4<ALIGNED>(sh.u[buf][r], r, j4, du);
            const float bias = p.bias != nullptr ? __ldg(p.bias + d0 + r) : 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                dt[j] += bias;
                if (p.softplus) dt[j] = sscan::softplus_f32(dt[j]);
                du[j] *= dt[j];
                const int t = t0 + j4 + j;
                if (t < stop || t >= end) dt[j] = du[j] = 0.f;
            }
            *reinterpret_cast<float4*>(&sh.dt[piece(r, j4)]) = make_float4(dt[0], dt[1], dt[2], dt[3]);
            *reinterpret_cast<float4*>(&sh.du[piece(r, j4)]) = make_float4(du[0], du[1], du[2], du[3]);
        }
        const int padded = (p.N + kEndStates - 1) / kEndStates * kEndStates;
        for (int i = threadIdx.x; i < padded * kTile; i += threads) {
            const int n = i / kTile, j = i % kTile, t = t0 + j;
            sh.B[j][n] = n < p.N && t >= stop && t < end ? sscan::to_f32(Bm[(long long)n * p.tokens + t]) : 0.f;
        }
        __syncthreads();
        if (!done) {
#pragma unroll
            for (int j4 = kTile - 4; j4 >= 0; j4 -= 4) {
                float dt[4], du[4];
                sscan::load4_smem(&sh.dt[piece(lane, j4)], dt);
                sscan::load4_smem(&sh.du[piece(lane, j4)], du);
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
// the CTA.  Per tile a warp widens its rows to fp32 dt and dt * u (with bias
// and softplus), advances its states over them, and finishes its outputs
// (skip term, gate, rounding) from the fp32 sums.
template <typename T, int P, bool GATED, bool ALIGNED>
struct ScanShared {
    static constexpr int kRows = 32 / P * kChannels;  // channels of a warp
    alignas(16) T u[kWarps][2][kRows][kRawPitch<T, ALIGNED>];
    alignas(16) T d[kWarps][2][kRows][kRawPitch<T, ALIGNED>];
    alignas(16) T z[kWarps][2][GATED ? kRows : 1][kRawPitch<T, ALIGNED>];
    alignas(16) float dt[kWarps][kRows * kTile];
    alignas(16) float du[kWarps][kRows * kTile];  // dt * u, then the outputs
    alignas(16) float B[2][kTile][P * kStates];
    alignas(16) float C[2][kTile][P * kStates];
    float D[kWarps][kRows];
    float bias[kWarps][kRows];
};

template <typename T, int P, bool GATED, bool ALIGNED>
__global__ void __launch_bounds__(kWarps * 32, kResident<P>) sscan_prompt_kernel(const PromptParams p) {
    using Sh = ScanShared<T, P, GATED, ALIGNED>;
    constexpr int kRows = Sh::kRows, NP = P * kStates, kThreads = kWarps * 32;
    extern __shared__ __align__(16) unsigned char raw_shared[];
    Sh& sh = *reinterpret_cast<Sh*>(raw_shared);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int seg = blockIdx.y;
    const long long d0 = ((long long)blockIdx.x * kWarps + warp) * kRows;  // the warp's first channel
    const int rows = p.dim - d0 < kRows ? (p.dim > d0 ? (int)(p.dim - d0) : 0) : kRows;
    const int part = lane % P, n0 = part * kStates;
    // the thread's channels: neighbouring rows, which odd parts hold in the
    // opposite order, so that one exchange gives each of two lanes the other's
    // share of the channel that it keeps
    auto row_of = [&](int c) { return P == 1 ? lane + 32 * c : lane / P * kChannels + (part & 1 ? kChannels - 1 - c : c); };
    const int begin = seg * p.seg_tokens;
    const int end = begin + p.seg_tokens < p.tokens ? begin + p.seg_tokens : p.tokens;
    const RawRows<T> u(p.u, d0, p.dim, p.tokens), delta(p.delta, d0, p.dim, p.tokens),
        z(GATED ? p.z : p.u, d0, p.dim, p.tokens);
    const T* Bm = static_cast<const T*>(p.B);
    const T* Cm = static_cast<const T*>(p.C);
    T* out_lane = static_cast<T*>(p.out) + (d0 + lane / 4) * p.tokens + lane % 4 * 4;
    constexpr int kChunks = kRawChunks<T, ALIGNED>;

    // aligned rows: the warp stages 32 / kChunks rows at a time, from per-lane
    // offsets that move with the tile
    constexpr int kStep = ALIGNED ? 32 / kChunks : 1;
    const long long lane_at = (long long)(lane / kChunks) * p.tokens + lane % kChunks * VecOf<T>::E;
    const long long step_at = (long long)kStep * p.tokens;
    auto stage = [&](int t0, int buf) {
        if (ALIGNED) {
            const int to = lane / kChunks * kTile + lane % kChunks * VecOf<T>::E;
            const bool on = t0 + lane % kChunks * VecOf<T>::E < p.tokens;  // past a row's end nothing is used
#pragma unroll
            for (int k = 0; k < (kRows + kStep - 1) / kStep; ++k) {
                if (!on || lane / kChunks + k * kStep >= rows) continue;
                const long long from = lane_at + k * step_at + t0;
                sscan::cp_async16(&sh.u[warp][buf][k * kStep][0] + to, u.base + from, 16);
                sscan::cp_async16(&sh.d[warp][buf][k * kStep][0] + to, delta.base + from, 16);
                if (GATED) sscan::cp_async16(&sh.z[warp][buf][k * kStep][0] + to, z.base + from, 16);
            }
        } else {
#pragma unroll 2
            for (int i = lane; i < kRows * kChunks; i += 32) {
                const int r = i / kChunks, c = i % kChunks;
                if (r >= rows) continue;
                u.stage(sh.u[warp][buf][r], r, c, t0);
                delta.stage(sh.d[warp][buf][r], r, c, t0);
                if (GATED) z.stage(sh.z[warp][buf][r], r, c, t0);
            }
        }
        sscan::cp_async_commit();
    };
    // B and C of a tile: read into registers a tile ahead, stored transposed
    constexpr int kBC = NP * kTile / kThreads, kBCRows = kThreads / kTile;
    const int bc_n = threadIdx.x / kTile, bc_j = threadIdx.x % kTile;
    const long long bc_at = (long long)bc_n * p.tokens + bc_j, bc_step = (long long)kBCRows * p.tokens;
    float bq[kBC], cq[kBC];
    auto fetch_bc = [&](int t0) {
        const bool on = t0 + bc_j < p.tokens;
#pragma unroll
        for (int i = 0; i < kBC; ++i) {
            const long long from = bc_at + i * bc_step + t0;
            bq[i] = on && bc_n + i * kBCRows < p.N ? sscan::to_f32(Bm[from]) : 0.f;
            cq[i] = on && bc_n + i * kBCRows < p.N ? sscan::to_f32(Cm[from]) : 0.f;
        }
    };
    auto store_bc = [&](int buf) {
#pragma unroll
        for (int i = 0; i < kBC; ++i) {
            sh.B[buf][bc_j][bc_n + i * kBCRows] = bq[i];
            sh.C[buf][bc_j][bc_n + i * kBCRows] = cq[i];
        }
    };
    if (p.segments == 1 && blockIdx.x == 0) p.req.check(threadIdx.x, kThreads);
    stage(begin, 0);
    fetch_bc(begin);
    store_bc(0);
    for (int r = lane; r < kRows; r += 32) {
        sh.D[warp][r] = p.D != nullptr && r < rows ? __ldg(p.D + d0 + r) : 0.f;
        sh.bias[warp][r] = p.bias != nullptr && r < rows ? __ldg(p.bias + d0 + r) : 0.f;
    }

    int row[kChannels];
    long long ch[kChannels];
    float a[kChannels][kStates], h[kChannels][kStates];
#pragma unroll
    for (int c = 0; c < kChannels; ++c) {
        row[c] = row_of(c);
        ch[c] = d0 + row[c] < p.dim ? d0 + row[c] : p.dim - 1;
#pragma unroll
        for (int i = 0; i < kStates; ++i) {
            a[c][i] = n0 + i < p.N ? p.A[ch[c] * p.N + n0 + i] * sscan::kLog2e : 0.f;
            h[c][i] = 0.f;
        }
    }
    auto read_states = [&](const float* from, float (&v)[kStates]) {
#pragma unroll
        for (int i = 0; i < kStates; i += 4) {
            const float4 q = *reinterpret_cast<const float4*>(from + n0 + i);
            v[i] = q.x; v[i + 1] = q.y; v[i + 2] = q.z; v[i + 3] = q.w;
        }
    };
    // The sum over a channel's lanes of its partial outputs: `mine` is this
    // lane's share of the channel it keeps, `other` its share of the one that
    // its neighbour keeps (the mirrored register).
    constexpr int kKept = P == 1 ? kChannels : kChannels / 2;
    auto channel_sum = [&](float mine, float other) {
        if (P == 1) return mine;
        mine += __shfl_xor_sync(0xffffffffu, other, 1);
#pragma unroll
        for (int o = 2; o < P; o <<= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
        return mine;
    };
    auto keep_state = [&](int s) {
        if (s < 0 || s >= p.req.requests) return;
        const int slot = p.req.slot(s);
        if (slot < 0) return;
#pragma unroll
        for (int c = 0; c < kChannels; ++c)
#pragma unroll
            for (int i = 0; i < kStates; ++i)
                if (row[c] < rows && n0 + i < p.N) p.state[((long long)slot * p.dim + ch[c]) * p.N + n0 + i] = h[c][i];
    };
    // the state of request s before its first token, at a token of this segment
    auto enter = [&](int s) {
        const int slot = s >= 0 && s < p.req.requests && p.req.continues(s) ? p.req.slot(s) : -1;
        const float* from = nullptr;
        if (slot >= 0)  // a request that crosses the border has its cache row written by another CTA
            from = p.req.offset(s + 1) > begin + p.seg_tokens ? p.h_first + (long long)seg * p.dim * p.N
                                                              : p.state + (long long)slot * p.dim * p.N;
#pragma unroll
        for (int c = 0; c < kChannels; ++c)
#pragma unroll
            for (int i = 0; i < kStates; ++i)
                h[c][i] = from != nullptr && n0 + i < p.N ? from[ch[c] * p.N + n0 + i] : 0.f;
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
#pragma unroll
        for (int k = 0; k < kRows; k += 8) {  // 8 rows at a time, four lanes a row
            const int r = k + lane / 4, j4 = lane % 4 * 4;
            float dt[4], du[4];
            delta.template read4<ALIGNED>(sh.d[warp][buf][r], r, j4, dt);
            u.template read4<ALIGNED>(sh.u[warp][buf][r], r, j4, du);
            if (p.bias != nullptr) {
                const float bias = sh.bias[warp][r];
#pragma unroll
                for (int j = 0; j < 4; ++j) dt[j] += bias;
            }
            if (p.softplus) {
#pragma unroll
                for (int j = 0; j < 4; ++j) dt[j] = sscan::softplus_f32(dt[j]);
            }
            const int to = k * kTile + piece(lane / 4, j4);  // a row's permutation repeats every 8 rows
            *reinterpret_cast<float4*>(&sh.dt[warp][to]) = make_float4(dt[0], dt[1], dt[2], dt[3]);
            *reinterpret_cast<float4*>(&sh.du[warp][to]) =
                make_float4(dt[0] * du[0], dt[1] * du[1], dt[2] * du[2], dt[3] * du[3]);
        }
        __syncthreads();  // B and C of this tile
        const int limit = end - t0 < kTile ? end - t0 : kTile;
#pragma unroll 1
        for (int j4 = 0; j4 < limit; j4 += 4) {
            if (next >= t0 + j4 + 4 && t0 + j4 + 4 <= end) {
                float dt[kChannels][4], du[kChannels][4], y[kChannels][4];
#pragma unroll
                for (int c = 0; c < kChannels; ++c) {
                    sscan::load4_smem(&sh.dt[warp][piece(row[c], j4)], dt[c]);
                    sscan::load4_smem(&sh.du[warp][piece(row[c], j4)], du[c]);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float b[kStates], cc[kStates];
                    read_states(sh.B[buf][j4 + j], b);
                    read_states(sh.C[buf][j4 + j], cc);
#pragma unroll
                    for (int c = 0; c < kChannels; ++c) {
                        y[c][j] = 0.f;
#pragma unroll
                        for (int i = 0; i < kStates; ++i) {
                            h[c][i] = fmaf(sscan::ex2(dt[c][j] * a[c][i]), h[c][i], du[c][j] * b[i]);
                            y[c][j] = fmaf(cc[i], h[c][i], y[c][j]);
                        }
                    }
                }
#pragma unroll
                for (int c = 0; c < kKept; ++c)
#pragma unroll
                    for (int j = 0; j < 4; ++j) y[c][j] = channel_sum(y[c][j], y[kChannels - 1 - c][j]);
                // the lanes of a channel have read its dt * u, which feeds the sums: the outputs take its place
                if (part < 2) {
#pragma unroll
                    for (int c = 0; c < kKept; ++c)
                        *reinterpret_cast<float4*>(&sh.du[warp][piece(row[c], j4)]) = make_float4(y[c][0], y[c][1], y[c][2], y[c][3]);
                }
            } else {
                // a request begins among these tokens, or the tokens end: one at a time
#pragma unroll 1
                for (int j = j4; j < j4 + 4 && t0 + j < end; ++j) {
                    if (t0 + j == next) {
                        keep_state(cur);
                        cur = p.req.find(next);
                        enter(cur);
                        next = end_of(cur);
                    }
                    float b[kStates], cc[kStates], y[kChannels];
                    read_states(sh.B[buf][j], b);
                    read_states(sh.C[buf][j], cc);
#pragma unroll
                    for (int c = 0; c < kChannels; ++c) {
                        const float dt = sh.dt[warp][piece(row[c], j4) + j - j4], du = sh.du[warp][piece(row[c], j4) + j - j4];
                        y[c] = 0.f;
#pragma unroll
                        for (int i = 0; i < kStates; ++i) {
                            h[c][i] = fmaf(sscan::ex2(dt * a[c][i]), h[c][i], du * b[i]);
                            y[c] = fmaf(cc[i], h[c][i], y[c]);
                        }
                    }
#pragma unroll
                    for (int c = 0; c < kKept; ++c) y[c] = channel_sum(y[c], y[kChannels - 1 - c]);
                    if (part < 2) {
#pragma unroll
                        for (int c = 0; c < kKept; ++c) sh.du[warp][piece(row[c], j4) + j - j4] = y[c];
                    }
                }
            }
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < kRows; k += 8) {
            const int r = k + lane / 4, j4 = lane % 4 * 4;
            if (r >= rows || t0 + j4 >= end) continue;
            float y[4], v[4];
            sscan::load4_smem(&sh.du[warp][k * kTile + piece(lane / 4, j4)], y);
            if (p.D != nullptr) {
                const float D = sh.D[warp][r];
                u.template read4<ALIGNED>(sh.u[warp][buf][r], r, j4, v);
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] = fmaf(D, v[j], y[j]);
            }
            if (GATED) {
                z.template read4<ALIGNED>(sh.z[warp][buf][r], r, j4, v);
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] *= v[j] * sscan::fast_sigmoid(v[j]);
            }
            // unaligned rows leave through shared memory (dt is done with), so
            // that neighbouring lanes store neighbouring tokens
            store4(ALIGNED ? out_lane + (long long)k * p.tokens + t0 : reinterpret_cast<T*>(sh.dt[warp] + r * kTile) + j4, y);
        }
        if (!ALIGNED) {
            __syncwarp();
            const int j = lane % kTile;
            T* to = static_cast<T*>(p.out) + (d0 + lane / kTile) * p.tokens + t0 + j;
#pragma unroll 4
            for (int r = lane / kTile; r < rows; r += 32 / kTile, to += 32 / kTile * (long long)p.tokens)
                if (t0 + j < end) *to = reinterpret_cast<const T*>(sh.dt[warp] + r * kTile)[j];
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

template <typename T, int P, bool GATED, bool ALIGNED>
cudaError_t run_scan(const PromptParams& p, cudaStream_t st) {
    constexpr size_t bytes = sizeof(ScanShared<T, P, GATED, ALIGNED>);
    static_assert(bytes <= 227 * 1024, "shared memory of a CTA");
    const cudaError_t e = cudaFuncSetAttribute(sscan_prompt_kernel<T, P, GATED, ALIGNED>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)sscan::div_up(p.dim, kWarps * ScanShared<T, P, GATED, ALIGNED>::kRows), (unsigned)p.segments);
    return sscan::launch(sscan_prompt_kernel<T, P, GATED, ALIGNED>, grid, dim3(kWarps * 32), bytes, st, p.segments > 1, p);
}
template <typename T, int P, bool ALIGNED>
cudaError_t run_gated(const PromptParams& p, cudaStream_t st) {
    return p.z != nullptr ? run_scan<T, P, true, ALIGNED>(p, st) : run_scan<T, P, false, ALIGNED>(p, st);
}
template <typename T, bool ALIGNED>
cudaError_t run_all(const PromptParams& p, cudaStream_t st) {
    if (p.segments > 1) {
        const dim3 grid((unsigned)sscan::div_up(p.dim, 32), (unsigned)(p.segments - 1));
        const dim3 block(32 * (unsigned)sscan::div_up(p.N, kEndStates));
        const cudaError_t e = sscan::launch(sscan_prompt_ends_kernel<T, ALIGNED>, grid, block, 0, st, false, p);
        if (e != cudaSuccess) return e;
    }
    if (p.N <= 8) return run_gated<T, 1, ALIGNED>(p, st);
    if (p.N <= 16) return run_gated<T, 2, ALIGNED>(p, st);
    if (p.N <= 32) return run_gated<T, 4, ALIGNED>(p, st);
    return run_gated<T, 8, ALIGNED>(p, st);
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
    if (want == 0) want = (4 * 152) / tiles;  // one wave of four CTAs an SM
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
    const bool aligned = tokens % (dtype == SSCAN_F32 ? 4 : 8) == 0 && sscan::is_aligned(u, 16) &&
                         sscan::is_aligned(delta, 16) && sscan::is_aligned(z, 16) && sscan::is_aligned(out, 16);
    cudaError_t e = dtype == SSCAN_F32 ? (aligned ? run_all<float, true>(p, st) : run_all<float, false>(p, st))
                                       : (aligned ? run_all<bf16, true>(p, st) : run_all<bf16, false>(p, st));
    if (scratch != nullptr) {
        const cudaError_t ef = cudaFreeAsync(scratch, st);
        if (e == cudaSuccess) e = ef;
    }
    return sscan::finish(e);
}
