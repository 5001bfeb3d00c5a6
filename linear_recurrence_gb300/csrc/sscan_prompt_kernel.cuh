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
// has no step-to-step dependence, and once A[n]*S_t < -kCutBits*ln 2 in every
// channel of a warp, what the rest of the segment put into the state has decayed
// below 2^-kCutBits of its size and is left out: the state is done.  Decay rates usually grow with n, so most states
// take a few dozen tokens.  The scan pass then starts every segment from the
// composed states of the ones before (again only as far back as they matter),
// writes each output once, rounded once, and needs no correction afterwards.
// Steps dt must be >= 0 for the cut-off to hold (the domain of the scan's time
// splits everywhere in this library); rates A >= 0 never meet it and are
// followed to the request's start.
//
// An element (token, channel, state) takes one exponential and four fp32
// operations in the scan pass, which bounds it by issue slots: 152 SMs x 128
// lanes / 5 at 2.07 GHz is 8.06 T elements/s; the bytes take about as long in
// fp32 and a half of it in bf16.  Measured: 65536 x 1536 x 16 fp32 543 us for
// the call: 404 of the scan pass, which issues 105 instructions a token and
// warp where the arithmetic is 80, at 66% of the issue slots, and 135 of the
// end states, bound by the latency of the slowest states' walks at 44% of the
// DRAM rate (they read most of u and delta once more); 8209 x 2048 x 16 bf16 with options, rows of odd
// length, 180 us, 123 and 53 (about 165 instructions a token and warp:
// widening, softplus and gate).
#pragma once

#include <type_traits>

#include "row_pieces.cuh"
#include "sscan_prompt.cuh"

namespace sscan {

// CTAs an SM should hold by registers.  16 states a thread need about 160
// registers to read the next tokens ahead: three CTAs (8209 x 2048 bf16: 208 us,
// against 273 with two and 243 with four of 128 registers, in the segments that
// suit each), or the two that the direct form's longer tiles leave room for, as does
// one lane a channel, whose warps have 64 rows.
template <int P, int kStates, bool DIRECT>
constexpr int kResident = kStates == 4 ? 6 : P == 1 || DIRECT ? 2 : 3;

// Offset of tokens j .. j+3 (j a multiple of 4) of row r in an fp32 tile of
// kPromptTile floats a row: the row's four 16-byte pieces are permuted by the row, so
// that eight neighbouring rows' pieces of the same tokens lie in distinct banks.
__device__ __forceinline__ int piece(int r, int j) { return r * kPromptTile + (j ^ ((r >> 1 & 3) << 2)); }

// A row's elements [t0, t0 + kPromptTile) are staged as they lie in memory.  ALIGNED
// (rows of whole 16-byte vectors): exactly those.  Otherwise 16-byte chunks
// from the boundary at or below the first, which then sits `phase` elements
// into the staged row; the phase depends on the row, not on t0.
// PAD: a row is read by one lane alone, and rows 16 bytes longer than a tile
// keep neighbouring lanes' reads out of each other's banks.
template <typename T, int TILE, bool PAD> constexpr int kRawPitch = TILE + (PAD ? 16 / (int)sizeof(T) : 0);
template <typename T, int TILE, bool ALIGNED> constexpr int kRawChunks = TILE * (int)sizeof(T) / 16 + (ALIGNED ? 0 : 1);

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
    // Chunk c of row r at t0 of an unaligned array.  edge: it may reach outside
    // the array (row_pieces.cuh), and is then put together one value at a time.
    __device__ __forceinline__ void stage(T* dst, int r, int c, int t0, bool edge) const {
        constexpr int E = VecOf<T>::E;
        const T* src = base + (long long)r * tokens + t0 + c * E - phase(r);
        if (!edge || (src >= lo && src + E <= hi)) {
            sscan::cp_async16(dst + c * E, src, 16);
        } else {
#pragma unroll
            for (int j = 0; j < E; ++j)
                dst[c * E + j] = src + j >= lo && src + j < hi ? src[j] : sscan::from_f32<T>(0.f);
        }
    }
};
// Four values from token j on of a staged row with the given phase.
template <bool ALIGNED, typename T>
__device__ __forceinline__ void read4(const T* row, int phase, int j, float (&v)[4]) {
    if (ALIGNED) {
        sscan::load4_smem(row + j, v);
    } else {
        const T* at = row + phase + j;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = sscan::to_f32(at[i]);
    }
}

__device__ __forceinline__ void store4(float* p, const float (&v)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(bf16* p, const float (&v)[4]) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(v[0], v[1]), hi = __floats2bfloat162_rn(v[2], v[3]);
    *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const unsigned*>(&lo), *reinterpret_cast<const unsigned*>(&hi));
}

// A load that stays where it is written (the compiler would move it to its use).
__device__ __forceinline__ void load_now(const float* p, float& v) {
    asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v) : "l"(p));
}
__device__ __forceinline__ void load_now(const bf16* p, bf16& v) {
    unsigned short w;
    asm volatile("ld.global.nc.u16 %0, [%1];" : "=h"(w) : "l"(p));
    v = __ushort_as_bfloat16(w);
}

// ---- states at segment ends -------------------------------------------------

// A warp takes 32 channels (lane = channel) and 4 consecutive states of one
// segment, and walks it back on its own: it stages its own rows and B, meets
// no barrier, and drops each state as it decays.  Warps of the slowest states
// come first in the grid, as they walk furthest; the others' rows are then in
// the L2.  (With the four state groups' warps in one CTA over shared rows, every
// group waited for the slowest at each tile's barriers: 345 us instead of 223
// on 65536 x 1536 fp32 in 50 segments.  8 or 16 states a warp convert each step
// once for more states, and leave too few warps: that call takes 587 and 603 us
// instead of 558.  The scan pass is not launched before the
// last walk ends: its CTAs would move in beside the walks, and some SMs get
// fewer than their share, 217 us instead of 183 on 8209 x 2048 bf16 with options.)
constexpr int kEndWarps = 4;  // warps of a CTA: neighbouring channels, the same states

// A lane reads its own row, one value at a time where rows start anywhere.  The
// rows whose start lies at the same place of a 16-byte chunk are eight (bf16)
// or four (fp32) apart; every eighth row is moved on so that their reads meet
// in no bank.
template <typename T> constexpr int kEndPitch = kRawPitch<T, kPromptTile, true>;
template <typename T> constexpr int kEndShift = sizeof(T) == 4 ? 4 : 16;
template <typename T>
__device__ __forceinline__ int end_row(int r) { return r * kEndPitch<T> + r / 8 * kEndShift<T>; }

template <typename T>
struct EndShared {
    alignas(16) T u[kEndWarps][2][32 * kEndPitch<T> + 3 * kEndShift<T>];
    alignas(16) T d[kEndWarps][2][32 * kEndPitch<T> + 3 * kEndShift<T>];
    alignas(16) float B[kEndWarps][2][kEndStates][kPromptTile];
};

template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(kEndWarps * 32) sscan_prompt_ends_kernel(const PromptParams p) {
    extern __shared__ __align__(16) unsigned char raw_shared[];
    EndShared<T>& sh = *reinterpret_cast<EndShared<T>*>(raw_shared);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int seg = blockIdx.y, n0 = blockIdx.z * kEndStates;
    const long long d0 = ((long long)blockIdx.x * kEndWarps + warp) * 32;
    if (blockIdx.x == 0 && seg == 0 && n0 == 0) p.req.check(threadIdx.x, kEndWarps * 32);
    if (d0 >= p.dim) return;
    const int rows = p.dim - d0 < 32 ? (int)(p.dim - d0) : 32;
    const bool mine = lane < rows;
    const long long d = d0 + (mine ? lane : rows - 1);
    const int begin = seg * p.seg_tokens;
    const int end = begin + p.seg_tokens;  // a border inside the tokens: the last segment is not walked
    // the request that crosses the border, if any
    const int s = p.req.find(end - 1);
    const bool in_request = s >= 0 && s < p.req.requests;
    const int from = s < 0 ? 0 : p.req.offset(s);
    const int until = s < 0 ? p.req.offset(0) : in_request ? p.req.offset(s + 1) : p.tokens;
    if (until <= end) return;  // it ends at the border: nothing is carried
    const bool starts_here = from >= begin;
    const int stop = starts_here ? from : begin;

    float a[kEndStates], h[kEndStates];
    unsigned live = 0u;  // states that some channel of the warp still needs
#pragma unroll
    for (int i = 0; i < kEndStates; ++i) {
        a[i] = n0 + i < p.N ? p.A[d * p.N + n0 + i] * sscan::kLog2e : 0.f;
        if (n0 + i < p.N) live |= 1u << i;
        h[i] = 0.f;
    }
    const float bias = p.bias != nullptr ? __ldg(p.bias + d) : 0.f;
    float S = 0.f;
    const RawRows<T> u(p.u, d0, p.dim, p.tokens), delta(p.delta, d0, p.dim, p.tokens);
    const int u_phase = u.phase(lane), d_phase = delta.phase(lane);
    constexpr int kChunks = kRawChunks<T, kPromptTile, ALIGNED>, E = VecOf<T>::E;
    // lane's part of a tile of B: token lane % kPromptTile of every second state from lane / kPromptTile
    const int bj = lane % kPromptTile, bn = lane / kPromptTile;
    const T* Bm = static_cast<const T*>(p.B) + (long long)(n0 + bn) * p.tokens + bj;
    const long long b_step = (long long)(32 / kPromptTile) * p.tokens;
    const long long lane_at = (long long)(lane / kChunks) * p.tokens + lane % kChunks * E;
    auto stage = [&](int t0, int buf) {
        if (ALIGNED) {
            constexpr int kStep = 32 / kChunks;
#pragma unroll
            for (int k = 0; k < 32; k += kStep) {
                const int r = k + lane / kChunks;
                if (r >= rows || t0 + lane % kChunks * E >= p.tokens) continue;
                const long long at = lane_at + (long long)k * p.tokens + t0;
                sscan::cp_async16(&sh.u[warp][buf][end_row<T>(r) + lane % kChunks * E], u.base + at, 16);
                sscan::cp_async16(&sh.d[warp][buf][end_row<T>(r) + lane % kChunks * E], delta.base + at, 16);
            }
        } else {
            const bool edge = inner_at_edge(d0, rows, p.dim, p.tokens, t0, kPromptTile, E);  // (its tiles end at the border)
#pragma unroll
            for (int k = 0; k < kChunks; ++k) {
                const int r = (lane + 32 * k) / kChunks, c = (lane + 32 * k) % kChunks;
                if (r >= rows) continue;
                u.stage(&sh.u[warp][buf][end_row<T>(r)], r, c, t0, edge);
                delta.stage(&sh.d[warp][buf][end_row<T>(r)], r, c, t0, edge);
            }
        }
        sscan::cp_async_commit();
    };
    // B goes through registers, loaded a tile ahead; tokens of another request,
    // and states past N, contribute nothing
    constexpr int kBRows = 32 / kPromptTile, kB = kEndStates / kBRows;
    T bq[kB];
    auto fetch_b = [&](int t0) {
        const bool on = t0 + bj >= stop && t0 + bj < end;
#pragma unroll
        for (int i = 0; i < kB; ++i) {
            bq[i] = sscan::from_f32<T>(0.f);
            if (on && n0 + bn + i * kBRows < p.N) load_now(Bm + i * b_step + t0, bq[i]);
        }
    };
    auto store_b = [&](int buf) {
#pragma unroll
        for (int i = 0; i < kB; ++i) sh.B[warp][buf][bn + i * kBRows][bj] = sscan::to_f32(bq[i]);
    };
    int t0 = (end - 1) / kPromptTile * kPromptTile, buf = 0;
    stage(t0, 0);
    fetch_b(t0);
    store_b(0);
    for (; t0 + kPromptTile > stop; t0 -= kPromptTile, buf ^= 1) {
        if (t0 > stop) {
            fetch_b(t0 - kPromptTile);
            stage(t0 - kPromptTile, buf ^ 1);
        } else {
            sscan::cp_async_commit();
        }
        sscan::cp_async_wait<1>();
        __syncwarp();
        const bool whole = t0 >= stop && t0 + kPromptTile <= end;
        float after[kPromptTile], du[kPromptTile];  // sum of dt after each token; dt * u
#pragma unroll
        for (int j4 = kPromptTile - 4; j4 >= 0; j4 -= 4) {
            float dt[4], u4[4];
            read4<ALIGNED>(&sh.d[warp][buf][end_row<T>(lane)], d_phase, j4, dt);
            read4<ALIGNED>(&sh.u[warp][buf][end_row<T>(lane)], u_phase, j4, u4);
            if (p.softplus) {
#pragma unroll
                for (int j = 0; j < 4; ++j) dt[j] = sscan::softplus_f32(dt[j] + bias);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) dt[j] += bias;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) u4[j] *= dt[j];
            if (!whole) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (t0 + j4 + j < stop || t0 + j4 + j >= end) dt[j] = u4[j] = 0.f;
            }
#pragma unroll
            for (int j = 3; j >= 0; --j) {
                after[j4 + j] = S;
                S += dt[j];
                du[j4 + j] = u4[j];
            }
        }
        // of the states up to the highest that is needed, without a branch between
        // them: their loads and exponentials overlap (65536 x 1536 fp32: 133 us
        // against 144 with a test per state; with the rows' conversion inside each copy of the code
        // 65 us instead of 52 on 8209 x 2048 bf16 with options, for instruction fetches)
        static_assert(kEndStates == 4, "the counts below");
        auto walk = [&](auto count) {
#pragma unroll
            for (int j4 = kPromptTile - 4; j4 >= 0; j4 -= 4)
#pragma unroll
                for (int i = 0; i < decltype(count)::value; ++i) {
                    float b[4];
                    sscan::load4_smem(&sh.B[warp][buf][i][j4], b);
#pragma unroll
                    for (int j = 3; j >= 0; --j)
                        h[i] = fmaf(sscan::ex2(a[i] * after[j4 + j]), du[j4 + j] * b[j], h[i]);
                }
        };
        if (live > 7u) walk(std::integral_constant<int, 4>());
        else if (live > 3u) walk(std::integral_constant<int, 3>());
        else if (live > 1u) walk(std::integral_constant<int, 2>());
        else walk(std::integral_constant<int, 1>());
#pragma unroll
        for (int i = 0; i < kEndStates; ++i)
            if (__all_sync(0xffffffffu, !mine || a[i] * S < -kCutBits)) live &= ~(1u << i);
        if (live == 0u) break;
        if (t0 > stop) store_b(buf ^ 1);
        __syncwarp();  // every lane has read the buffers that the next tile but one fills
    }
    sscan::cp_async_wait<0>();
    if (!mine) return;
    // A walk that ended early has seen a part of the steps only: what lies before
    // (the initial state, the segments before) is dropped with the rest, not
    // weighted with the part's decay.
    const bool all = live != 0u;
    const int slot = in_request && starts_here ? p.req.slot(s) : -1;
    const bool cont = slot >= 0 && p.req.continues(s);
    const long long at = ((long long)seg * p.dim + d) * p.N + n0;
#pragma unroll
    for (int i = 0; i < kEndStates; ++i) {
        if (n0 + i >= p.N) break;
        float first = 0.f;
        if (starts_here) {  // kept for the scan pass, which may find the cache row already updated
            if (cont) first = p.state[((long long)slot * p.dim + d) * p.N + n0 + i];
            p.h_first[at + i] = first;
            if (cont && all) h[i] = fmaf(sscan::ex2(a[i] * S), first, h[i]);
        }
        p.h_end[at + i] = h[i];
    }
    p.dt_sum[((long long)seg * p.dim + d) * gridDim.z + blockIdx.z] = all ? S : INFINITY;
}

// ---- the scan ----------------------------------------------------------------

// P lanes share a channel, kStates states each, and a thread advances
// kChannels channels: wide threads 8 states of 2 channels, so that a B or C
// value read from shared memory serves two elements, narrow ones 4 of one, for calls of few
// tokens.  A warp's channels are its own from staging to the store: only B and C
// are shared by the CTA.  Per tile a warp widens its rows to fp32 dt and dt * u
// (with bias and softplus), advances its states over them, and finishes its
// outputs (skip term, gate, rounding) from the fp32 sums.
template <typename T, int P, int kStates, int kChannels, bool OPT, bool ALIGNED>
struct ScanShared {
    static constexpr int kRows = 32 / P * kChannels;  // channels of a warp
    static constexpr bool kDirect = sizeof(T) == 4 && ALIGNED && !OPT && kChannels == 2;
    static constexpr int kTile = kDirect ? 2 * kPromptTile : kPromptTile;
    static constexpr int kPitch = kRawPitch<T, kTile, kDirect || !ALIGNED>;
    static constexpr int kBPitch = kTile + 4;  // the lanes of a channel read distinct banks
    alignas(16) T u[kPromptWarps][2][kRows][kPitch];
    alignas(16) T d[kPromptWarps][2][kRows][kPitch];
    alignas(16) T z[kPromptWarps][2][OPT ? kRows : 1][kPitch];
    alignas(16) float dt[kPromptWarps][kDirect ? 4 : kRows * kTile];
    alignas(16) float du[kPromptWarps][kDirect ? 4 : kRows * kTile];  // dt * u, then the outputs
    alignas(16) float B[2][P * kStates][kBPitch];
    alignas(16) float C[2][P * kStates][kBPitch];
    float D[kPromptWarps][kRows];
    float bias[kPromptWarps][kRows];
};

template <typename T, int P, int kStates, int kChannels, bool OPT, bool ALIGNED>
__global__ void __launch_bounds__(kPromptWarps * 32, kResident<P, kStates, sizeof(T) == 4 && ALIGNED && !OPT && kChannels == 2>)
    sscan_prompt_kernel(const PromptParams p) {
    using Sh = ScanShared<T, P, kStates, kChannels, OPT, ALIGNED>;
    constexpr int kRows = Sh::kRows, NP = P * kStates, kThreads = kPromptWarps * 32;
    // plain fp32 rows need no widening: the lanes read them as they were staged
    // and store their channels' outputs themselves
    constexpr bool kDirect = Sh::kDirect;
    constexpr int kTile = Sh::kTile;
    const bool gated = OPT && p.z != nullptr;
    extern __shared__ __align__(16) unsigned char raw_shared[];
    Sh& sh = *reinterpret_cast<Sh*>(raw_shared);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int seg = blockIdx.y;
    const long long d0 = ((long long)blockIdx.x * kPromptWarps + warp) * kRows;  // the warp's first channel
    const int rows = p.dim - d0 < kRows ? (p.dim > d0 ? (int)(p.dim - d0) : 0) : kRows;
    const int part = lane % P;
    auto state_of = [&](int i) { return i * P + part; };  // neighbouring lanes read neighbouring rows of B and C
    // the thread's channels: neighbouring rows, which odd parts hold in the
    // opposite order, so that one exchange gives each of two lanes the other's
    // share of the channel that it keeps
    auto row_of = [&](int c) { return P == 1 ? lane + 32 * c : lane / P * kChannels + (part & 1 ? kChannels - 1 - c : c); };
    constexpr bool kSwap = P > 1 && kChannels > 1;  // (one channel a thread: all its lanes get the whole sum)
    const int begin = seg * p.seg_tokens;
    const int end = begin + p.seg_tokens < p.tokens ? begin + p.seg_tokens : p.tokens;
    const RawRows<T> u(p.u, d0, p.dim, p.tokens), delta(p.delta, d0, p.dim, p.tokens),
        z(gated ? p.z : p.u, d0, p.dim, p.tokens);
    // of the rows lane / 4 + 8 k that a lane converts: 8 rows on, a phase is the same again
    const int u_phase = u.phase(lane / 4), d_phase = delta.phase(lane / 4), z_phase = z.phase(lane / 4);
    const T* Bm = static_cast<const T*>(p.B);
    const T* Cm = static_cast<const T*>(p.C);
    T* out_lane = static_cast<T*>(p.out) + (d0 + lane / 4) * p.tokens + lane % 4 * 4;
    constexpr int kChunks = kRawChunks<T, kTile, ALIGNED>;

    // aligned rows: the warp stages 32 / kChunks rows at a time, from per-lane
    // offsets that move with the tile
    constexpr int kStep = ALIGNED ? 32 / kChunks : 1;
    const long long lane_at = (long long)(lane / kChunks) * p.tokens + lane % kChunks * VecOf<T>::E;
    const long long step_at = (long long)kStep * p.tokens;
    const int last_inner = last_inner_tile(d0, rows, p.dim, p.tokens, kTile, VecOf<T>::E);
    auto stage = [&](int t0, int buf) {
        if (ALIGNED) {
            const int to = lane / kChunks * Sh::kPitch + lane % kChunks * VecOf<T>::E;
            const bool on = t0 + lane % kChunks * VecOf<T>::E < p.tokens;  // past a row's end nothing is used
#pragma unroll
            for (int k = 0; k < (kRows + kStep - 1) / kStep; ++k) {
                if (!on || lane / kChunks + k * kStep >= rows) continue;
                const long long from = lane_at + k * step_at + t0;
                sscan::cp_async16(&sh.u[warp][buf][k * kStep][0] + to, u.base + from, 16);
                sscan::cp_async16(&sh.d[warp][buf][k * kStep][0] + to, delta.base + from, 16);
                if (gated) sscan::cp_async16(&sh.z[warp][buf][k * kStep][0] + to, z.base + from, 16);
            }
        } else {
            const bool edge = at_edge(t0, last_inner);
#pragma unroll 1
            for (int i = lane; i < kRows * kChunks; i += 32) {
                const int r = i / kChunks, c = i % kChunks;
                if (r >= rows) continue;
                u.stage(sh.u[warp][buf][r], r, c, t0, edge);
                delta.stage(sh.d[warp][buf][r], r, c, t0, edge);
                if (gated) z.stage(sh.z[warp][buf][r], r, c, t0, edge);
            }
        }
        sscan::cp_async_commit();
    };
    // B and C of a tile: read into registers a tile ahead, widened into shared memory
    constexpr int kBCRows = kThreads / kTile, kBC = NP / kBCRows;
    static_assert(NP % kBCRows == 0, "whole rows of B and C a step");
    const int bc_n = threadIdx.x / kTile, bc_j = threadIdx.x % kTile;
    const long long bc_at = (long long)bc_n * p.tokens + bc_j, bc_step = (long long)kBCRows * p.tokens;
    // (aligned fp32 rows go there by themselves)
    constexpr bool kCopyBC = sizeof(T) == 4 && ALIGNED;
    constexpr int kBCChunks = NP * (kTile / 4);  // 16-byte pieces of a tile of B
    T bq[kBC], cq[kBC];
    auto fetch_bc = [&](int t0, int buf) {
        if constexpr (kCopyBC) {
            for (int i = threadIdx.x; i < kBCChunks; i += kThreads) {
                const int n = i / (kTile / 4), j = i % (kTile / 4) * 4;
                if (n >= p.N || t0 + j >= p.tokens) continue;
                const long long from = (long long)n * p.tokens + t0 + j;
                sscan::cp_async16(&sh.B[buf][n][j], Bm + from, 16);
                sscan::cp_async16(&sh.C[buf][n][j], Cm + from, 16);
            }
        } else {
            const bool on = t0 + bc_j < p.tokens;
#pragma unroll
            for (int i = 0; i < kBC; ++i) {
                const long long from = bc_at + i * bc_step + t0;
                bq[i] = cq[i] = sscan::from_f32<T>(0.f);
                if (on && bc_n + i * kBCRows < p.N) {
                    load_now(Bm + from, bq[i]);
                    load_now(Cm + from, cq[i]);
                }
            }
        }
    };
    auto store_bc = [&](int buf) {
        if (kCopyBC) return;
#pragma unroll
        for (int i = 0; i < kBC; ++i) {
            sh.B[buf][bc_n + i * kBCRows][bc_j] = sscan::to_f32(bq[i]);
            sh.C[buf][bc_n + i * kBCRows][bc_j] = sscan::to_f32(cq[i]);
        }
    };
    if (p.segments == 1 && blockIdx.x == 0) p.req.check(threadIdx.x, kThreads);
    fetch_bc(begin, 0);
    stage(begin, 0);
    store_bc(0);
    if (kCopyBC) {  // states past N: zero rows
        for (int i = threadIdx.x; i < NP * kTile; i += kThreads)
            if (i / kTile >= p.N)
                sh.B[0][i / kTile][i % kTile] = sh.B[1][i / kTile][i % kTile] = sh.C[0][i / kTile][i % kTile] =
                    sh.C[1][i / kTile][i % kTile] = 0.f;
    }
    for (int r = lane; r < kRows; r += 32) {
        sh.D[warp][r] = p.D != nullptr && r < rows ? __ldg(p.D + d0 + r) : 0.f;
        sh.bias[warp][r] = p.bias != nullptr && r < rows ? __ldg(p.bias + d0 + r) : 0.f;
    }

    int row[kChannels];
    long long ch[kChannels];
    float a[kChannels][kStates], h[kChannels][kStates], skip[kChannels];
#pragma unroll
    for (int c = 0; c < kChannels; ++c) {
        row[c] = row_of(c);
        ch[c] = d0 + row[c] < p.dim ? d0 + row[c] : p.dim - 1;
        skip[c] = kDirect && p.D != nullptr ? __ldg(p.D + ch[c]) : 0.f;
#pragma unroll
        for (int i = 0; i < kStates; ++i) {
            a[c][i] = state_of(i) < p.N ? p.A[ch[c] * p.N + state_of(i)] * sscan::kLog2e : 0.f;
            h[c][i] = 0.f;
        }
    }
    // The sum over a channel's lanes of its partial outputs: `mine` is this
    // lane's share of the channel it keeps, `other` its share of the one that
    // its neighbour keeps (the mirrored register).
    constexpr int kKept = kSwap ? kChannels / 2 : kChannels;
    const bool writes = part < (kSwap ? 2 : 1);
    auto channel_sum = [&](float mine, float other) {
        if (kSwap) mine += __shfl_xor_sync(0xffffffffu, other, 1);
#pragma unroll
        for (int o = kSwap ? 2 : 1; o < P; o <<= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
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
                if (row[c] < rows && state_of(i) < p.N) p.state[((long long)slot * p.dim + ch[c]) * p.N + state_of(i)] = h[c][i];
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
                h[c][i] = from != nullptr && state_of(i) < p.N ? from[ch[c] * p.N + state_of(i)] : 0.f;
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
                    const int n = state_of(i);
                    if (n >= p.N) continue;
                    h[c][i] = fmaf(sscan::ex2(e[c][i]), p.h_end[at * p.N + n], h[c][i]);
                    e[c][i] = fmaf(a[c][i], p.dt_sum[at * groups + n / kEndStates], e[c][i]);
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
            if (!kCopyBC) fetch_bc(t0 + kTile, buf ^ 1);
            stage(t0 + kTile, buf ^ 1);
        } else {
            sscan::cp_async_commit();
        }
        sscan::cp_async_wait<1>();
        __syncwarp();
#pragma unroll
        for (int k = 0; k < (kDirect ? 0 : kRows); k += 8) {  // 8 rows at a time, four lanes a row
            const int r = k + lane / 4, j4 = lane % 4 * 4;
            if (kRows < 8 && r >= kRows) break;
            float dt[4], du[4];
            read4<ALIGNED>(sh.d[warp][buf][r], d_phase, j4, dt);
            read4<ALIGNED>(sh.u[warp][buf][r], u_phase, j4, du);
            if (OPT) {
                const float bias = sh.bias[warp][r];
                if (p.softplus) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) dt[j] = sscan::softplus_f32(dt[j] + bias);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) dt[j] += bias;
                }
            }
            const int to = k * kTile + piece(lane / 4, j4);  // a row's permutation repeats every 8 rows
            *reinterpret_cast<float4*>(&sh.dt[warp][to]) = make_float4(dt[0], dt[1], dt[2], dt[3]);
            *reinterpret_cast<float4*>(&sh.du[warp][to]) =
                make_float4(dt[0] * du[0], dt[1] * du[1], dt[2] * du[2], dt[3] * du[3]);
        }
        __syncthreads();  // B and C of this tile; every warp is done with those of the last
        if (kCopyBC && more) {
            fetch_bc(t0 + kTile, buf ^ 1);
            cp_async_commit();
        }
        const int limit = end - t0 < kTile ? end - t0 : kTile;
        float nd[kChannels][4], nu[kChannels][4];  // dt and u (or dt * u) of the next four tokens
        auto read_next = [&](int j4) {
#pragma unroll
            for (int c = 0; c < kChannels; ++c) {
                if constexpr (kDirect) {
                    sscan::load4_smem(&sh.d[warp][buf][row[c]][j4], nd[c]);
                    sscan::load4_smem(&sh.u[warp][buf][row[c]][j4], nu[c]);
                } else {
                    sscan::load4_smem(&sh.dt[warp][piece(row[c], j4)], nd[c]);
                    sscan::load4_smem(&sh.du[warp][piece(row[c], j4)], nu[c]);
                }
            }
        };
        read_next(0);
#pragma unroll 2
        for (int j4 = 0; j4 < limit; j4 += 4) {
            if (next >= t0 + j4 + 4 && t0 + j4 + 4 <= end) {
                float dt[kChannels][4], du[kChannels][4], y[kChannels][4], u4[kDirect ? kChannels : 1][4];
#pragma unroll
                for (int c = 0; c < kChannels; ++c)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        dt[c][j] = nd[c][j];
                        if (kDirect) u4[kDirect ? c : 0][j] = nu[c][j];
                        du[c][j] = kDirect ? nd[c][j] * nu[c][j] : nu[c][j];
                        y[c][j] = 0.f;
                    }
                if (j4 + 4 < kTile) read_next(j4 + 4);
#pragma unroll
                for (int i = 0; i < kStates; ++i) {
                    float b[4], cc[4];
                    sscan::load4_smem(&sh.B[buf][state_of(i)][j4], b);
                    sscan::load4_smem(&sh.C[buf][state_of(i)][j4], cc);
#pragma unroll
                    for (int c = 0; c < kChannels; ++c)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            h[c][i] = fmaf(sscan::ex2(dt[c][j] * a[c][i]), h[c][i], du[c][j] * b[j]);
                            y[c][j] = fmaf(cc[j], h[c][i], y[c][j]);
                        }
                }
#pragma unroll
                for (int c = 0; c < kKept; ++c)
#pragma unroll
                    for (int j = 0; j < 4; ++j) y[c][j] = channel_sum(y[c][j], y[kChannels - 1 - c][j]);
                // the lanes of a channel have read its dt * u, which feeds the sums: the outputs take its place
                if constexpr (kDirect) {
#pragma unroll
                    for (int c = 0; c < kKept; ++c) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) y[c][j] = fmaf(skip[c], u4[c][j], y[c][j]);
                        if (writes && row[c] < rows) store4(static_cast<T*>(p.out) + ch[c] * p.tokens + t0 + j4, y[c]);
                    }
                } else if (writes) {
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
                    float y[kChannels];
#pragma unroll
                    for (int c = 0; c < kChannels; ++c) {
                        float dt, du;
                        if constexpr (kDirect) {
                            dt = sscan::to_f32(sh.d[warp][buf][row[c]][j]);
                            du = dt * sscan::to_f32(sh.u[warp][buf][row[c]][j]);
                        } else {
                            dt = sh.dt[warp][piece(row[c], j4) + j - j4];
                            du = sh.du[warp][piece(row[c], j4) + j - j4];
                        }
                        y[c] = 0.f;
#pragma unroll
                        for (int i = 0; i < kStates; ++i) {
                            h[c][i] = fmaf(sscan::ex2(dt * a[c][i]), h[c][i], du * sh.B[buf][state_of(i)][j]);
                            y[c] = fmaf(sh.C[buf][state_of(i)][j], h[c][i], y[c]);
                        }
                    }
#pragma unroll
                    for (int c = 0; c < kKept; ++c) y[c] = channel_sum(y[c], y[kChannels - 1 - c]);
                    if (writes) {
#pragma unroll
                        for (int c = 0; c < kKept; ++c) {
                            if constexpr (kDirect) {
                                const float at_u = sscan::to_f32(sh.u[warp][buf][row[c]][j]);
                                if (row[c] < rows)
                                    static_cast<T*>(p.out)[ch[c] * p.tokens + t0 + j] = sscan::from_f32<T>(fmaf(skip[c], at_u, y[c]));
                            } else {
                                sh.du[warp][piece(row[c], j4) + j - j4] = y[c];
                            }
                        }
                    }
                }
                if (j4 + 4 < limit) read_next(j4 + 4);
            }
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < (kDirect ? 0 : kRows); k += 8) {
            const int r = k + lane / 4, j4 = lane % 4 * 4;
            if (r >= rows || t0 + j4 >= end) continue;
            float y[4], v[4];
            sscan::load4_smem(&sh.du[warp][k * kTile + piece(lane / 4, j4)], y);
            if (p.D != nullptr) {
                const float D = sh.D[warp][r];
                read4<ALIGNED>(sh.u[warp][buf][r], u_phase, j4, v);
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] = fmaf(D, v[j], y[j]);
            }
            if (gated) {
                read4<ALIGNED>(sh.z[warp][buf][r], z_phase, j4, v);
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

template <typename T, int P, int kStates, int kChannels, bool OPT, bool ALIGNED>
cudaError_t run_scan(const PromptParams& p, cudaStream_t st) {
    using Sh = ScanShared<T, P, kStates, kChannels, OPT, ALIGNED>;
    static_assert(sizeof(Sh) <= 227 * 1024, "shared memory of a CTA");
    auto kernel = sscan_prompt_kernel<T, P, kStates, kChannels, OPT, ALIGNED>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Sh));
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)sscan::div_up(p.dim, kPromptWarps * Sh::kRows), (unsigned)p.segments);
    return sscan::launch(kernel, grid, dim3(kPromptWarps * 32), sizeof(Sh), st, p.segments > 1, p);
}
template <typename T, int P, int kStates, int kChannels, bool ALIGNED>
cudaError_t run_opt(const PromptParams& p, cudaStream_t st) {
    return p.z != nullptr || p.bias != nullptr || p.softplus ? run_scan<T, P, kStates, kChannels, true, ALIGNED>(p, st)
                                                             : run_scan<T, P, kStates, kChannels, false, ALIGNED>(p, st);
}
template <typename T, bool ALIGNED>
cudaError_t prompt_launch(const PromptParams& p, cudaStream_t st) {
    if (p.segments > 1) {
        const dim3 grid((unsigned)sscan::div_up(p.dim, 32 * kEndWarps), (unsigned)(p.segments - 1),
                        (unsigned)sscan::div_up(p.N, kEndStates));
        static_assert(sizeof(EndShared<T>) <= 48 * 1024, "shared memory without opting in");
        const cudaError_t e = sscan::launch(sscan_prompt_ends_kernel<T, ALIGNED>, grid, dim3(32 * kEndWarps),
                                            sizeof(EndShared<T>), st, false, p);
        if (e != cudaSuccess) return e;
    }
    // four states of one channel a thread where the tokens are too few for the
    // wide threads to fill the GPU, else eight states of two channels
    if (p.narrow) {
        if (p.N <= 8) return run_opt<T, 2, 4, 1, ALIGNED>(p, st);
        if (p.N <= 16) return run_opt<T, 4, 4, 1, ALIGNED>(p, st);
        if (p.N <= 32) return run_opt<T, 8, 4, 1, ALIGNED>(p, st);
        return run_opt<T, 16, 4, 1, ALIGNED>(p, st);
    }
    if (p.N <= 8) return run_opt<T, 1, 8, 2, ALIGNED>(p, st);
    if (p.N <= 16) return run_opt<T, 2, 8, 2, ALIGNED>(p, st);
    if (p.N <= 32) return run_opt<T, 4, 8, 2, ALIGNED>(p, st);
    return run_opt<T, 8, 8, 2, ALIGNED>(p, st);
}

}  // namespace sscan
