// Short causal depthwise convolution on sm_103a: the W-tap filter that runs
// before the selective scan of a layer.
//
//   c[d,t] = bias[d] + sum_{k<W} w[d,k] * x[d, t-(W-1)+k],   y = c * sigmoid(c) (SiLU) or c
//
// Inputs before a sequence's first token come from its state (the last W-1
// inputs before it, oldest first) or are zero.  Forward, gradients, packed
// prompts over a state cache, and single tokens.
//
// Every form reads x once and writes y once, with about 2W + 8 operations a
// value, so HBM bandwidth is the floor; instructions come close behind it (a
// 16-byte bf16 window of 8 values takes about 183 of them, 40 for the SiLU).
// Time is contiguous in a row: a thread owns a 16-byte window of it and takes
// the W-1 inputs before its window from its left neighbour in the warp by
// shuffles; sums are fp32, outputs are rounded once.  Measured: 16411 x 5120
// packed bf16 tokens 80 us (62% of the copy rate); 4 x 2048 x 2048 bf16
// forward 18.0 and gradients 27.4 us (55% and 54%); single tokens 256 x 5120 6.6 us.
#include <type_traits>

#include "block_utils.cuh"

namespace {

using sscan::bf16;
using sscan::Requests;
using sscan::VecOf;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct Rows {  // [batch, dim, len] rows with unit time stride
    long long batch_stride, dim_stride;
};

// Elements before the first 16-byte boundary at or below p.
template <typename T>
__device__ __forceinline__ int phase_of(const T* p) {
    return (int)((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T));
}

// x[t0 .. t0+E-1] of a row of n tokens, zero outside it.  VEC: t0 is on a
// 16-byte boundary, and only windows across the row's ends go one value at a
// time (out of line: inlined, their predicated instructions tripled the kernels').
template <typename T>
__device__ __noinline__ uint4 load_edge(const T* row, int t0, int n) {
    constexpr int E = VecOf<T>::E;
    float v[E];
#pragma unroll
    for (int j = 0; j < E; ++j) v[j] = t0 + j >= 0 && t0 + j < n ? sscan::to_f32(row[t0 + j]) : 0.f;
    return sscan::narrow(v, static_cast<T*>(nullptr));
}
template <typename T>
__device__ __noinline__ void store_edge(T* row, int t0, int n, uint4 q) {
    constexpr int E = VecOf<T>::E;
    float v[E];
    sscan::widen(q, v, static_cast<T*>(nullptr));
#pragma unroll
    for (int j = 0; j < E; ++j)
        if (t0 + j >= 0 && t0 + j < n) row[t0 + j] = sscan::from_f32<T>(v[j]);
}
// INSIDE: the caller knows that the window lies inside the row.
template <typename T, bool VEC, bool INSIDE>
__device__ __forceinline__ uint4 load_raw(const T* row, int t0, int n) {
    constexpr int E = VecOf<T>::E;
    if (VEC && (INSIDE || (t0 >= 0 && t0 + E <= n))) return __ldg(reinterpret_cast<const uint4*>(row + t0));
    if (t0 + E <= 0 || t0 >= n) return make_uint4(0u, 0u, 0u, 0u);
    return load_edge(row, t0, n);
}
template <typename T, bool VEC, bool INSIDE, int E = VecOf<T>::E>
__device__ __forceinline__ void store_window(T* row, int t0, int n, const float (&v)[E]) {
    const uint4 q = sscan::narrow(v, static_cast<T*>(nullptr));
    if (VEC && (INSIDE || (t0 >= 0 && t0 + E <= n))) *reinterpret_cast<uint4*>(row + t0) = q;
    else if (t0 + E > 0 && t0 < n) store_edge(row, t0, n, q);
}
// The inputs before a sequence put into a window that reaches back over its start.
template <typename T, int H, int E = VecOf<T>::E>
__device__ __noinline__ uint4 put_before(uint4 q, const T* x0, int t0) {
    float v[E];
    sscan::widen(q, v, static_cast<T*>(nullptr));
#pragma unroll
    for (int j = 0; j < E; ++j)
        if (t0 + j < 0 && t0 + j >= -H) v[j] = sscan::to_f32(x0[H + t0 + j]);
    return sscan::narrow(v, static_cast<T*>(nullptr));
}
// W weights of channel d.
template <int W>
__device__ __forceinline__ void load_weights(const float* w, long long d, bool vec, float (&v)[W]) {
    if (W == 4 && vec) {
        const float4 q = __ldg(reinterpret_cast<const float4*>(w) + d);
        v[0] = q.x; v[1] = q.y; v[2] = q.z; v[W - 1] = q.w;
    } else {
#pragma unroll
        for (int k = 0; k < W; ++k) v[k] = __ldg(w + d * W + k);
    }
}

// ---- forward ---------------------------------------------------------------

struct ConvParams {
    const void* x;
    const float* w;
    const float* bias;
    const void* x0;    // batch form: [batch, dim, W-1] or NULL
    void* final_state; // batch form: [batch, dim, W-1] or NULL
    void* state;       // packed form: the cache
    void* y;           // contiguous
    long long batch, dim, len;
    Rows xs;
    int silu;
    bool w_aligned;  // weight rows of four are 16-byte vectors
    unsigned strips, groups;  // grid = strips x channel groups x batch
    int strip_tiles;          // tiles of 31 windows that a warp takes one after another
    bool flat;                // the grid has one dimension
    Requests req;
};

// What request s leaves in channel d of its cache row: its last inputs, or
// what the row (or zeros) held where it has fewer than W-1.
template <typename T, int W>
__device__ __forceinline__ void keep_state(const ConvParams& p, const T* xrow, long long d, int s) {
    constexpr int H = W - 1;
    const int slot = p.req.slot(s);
    if (slot < 0) return;
    const int begin = p.req.offset(s), end = p.req.offset(s + 1);
    T* st = static_cast<T*>(p.state) + ((long long)slot * p.dim + d) * H;
    const bool cont = p.req.continues(s);
    T keep[H];
#pragma unroll
    for (int j = 0; j < H; ++j) {
        const int back = end - begin - H + j;  // token of the request, or before it
        keep[j] = back >= 0 ? xrow[begin + back]
                  : cont && H + back >= 0 && H + back < H ? st[H + back]
                                                          : sscan::from_f32<T>(0.f);
    }
#pragma unroll
    for (int j = 0; j < H; ++j) st[j] = keep[j];
}

// Whether request s leaves its cache row to the kernel after this one (>= 0):
// it has no tokens, or begins so near a strip's end that its first tokens may
// lie in two strips (by up to W-1 tokens and a row's phase).  Otherwise the CTA
// of the strip that it begins in alone reads its old state.
template <int E>
__device__ __forceinline__ int apart(const ConvParams& p, int s) {
    const int at = p.req.offset(s), span = p.strip_tiles * 31 * E;
    if (p.req.offset(s + 1) <= at) return 0;
    return at % span - (span - 16);
}

// A warp walks a strip of one row, 32 consecutive windows (a tile) at a time
// with the next two tiles' loads under way: lane 0's window only supplies the inputs
// before lane 1's, so a tile is 31 windows (3% of the loads, and no lane takes
// another path).  A strip makes the row's addresses, phase and weights once for
// several tiles: with one tile a warp that was half of the instructions,
// and instructions, not bytes, set the time.  The packed form first runs over its
// strips as one sequence; the CTA then computes the first W-1 outputs of each
// request that begins there again, from the request's state.
// VEC: every row of x and y has the same phase against 16-byte boundaries
// (the windows then start on them).
constexpr int kMaxStrip = 8;  // tiles of a strip

// INSIDE: the tile's windows lie inside the row, and no inputs before it count.
template <typename T, int W, bool VEC, bool INSIDE>
__device__ __forceinline__ void conv_tile(const ConvParams& p, uint4 raw, const float (&w)[W], float bias, T* yrow,
                                          long long row, int t0, int len) {
    constexpr int E = VecOf<T>::E;
    constexpr int H = W - 1;  // inputs before a window
    float v[H + E], own[E];
    if (!INSIDE && p.x0 != nullptr && t0 < 0) raw = put_before<T, H>(raw, static_cast<const T*>(p.x0) + row * H, t0);
    sscan::widen(raw, own, static_cast<T*>(nullptr));
#pragma unroll
    for (int j = 0; j < E; ++j) v[H + j] = own[j];
#pragma unroll
    for (int j = 0; j < H; ++j) v[j] = __shfl_up_sync(0xffffffffu, v[E + j], 1);
    float out[E];
#pragma unroll
    for (int j = 0; j < E; ++j) {
        float c = bias;
#pragma unroll
        for (int k = 0; k < W; ++k) c = fmaf(w[k], v[j + k], c);
        out[j] = c;
    }
    if (p.silu) {
#pragma unroll
        for (int j = 0; j < E; ++j) out[j] *= sscan::fast_sigmoid(out[j]);
    }
    if ((threadIdx.x & 31) > 0) store_window<T, VEC, INSIDE>(yrow, t0, len, out);
}

// (Six CTAs an SM: 16411 x 5120 packed bf16 tokens 72.1 us, against 76.4 at the
// five that the compiler's registers left; eight spill.)
template <typename T, int W, bool PACKED, bool VEC>
__global__ void __launch_bounds__(kThreads, 6) sconv_fwd_kernel(const __grid_constant__ ConvParams p) {
    constexpr int E = VecOf<T>::E;
    constexpr int H = W - 1;
    constexpr int kTile = 31 * E;  // tokens of a tile
    __shared__ int begun[PACKED ? kMaxStrip * kTile + 16 : 1], begun_count;  // requests that begin in or just before the strip
    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5;
    // (a division costs as much as a tile's loads and stores: three grid
    // dimensions unless a call exceeds two of them)
    unsigned strip = blockIdx.x, group = blockIdx.y;
    long long b = blockIdx.z;
    if (p.flat) {
        strip = blockIdx.x % p.strips;
        group = blockIdx.x / p.strips % p.groups;
        b = blockIdx.x / p.strips / p.groups;
    }
    const int begin = (int)strip * p.strip_tiles * kTile, span = p.strip_tiles * kTile;
    const long long cta0 = (long long)group * kWarps;  // the CTA's first channel
    const long long d = cta0 + warp;
    const int len = (int)p.len;
    const T* xrow = static_cast<const T*>(p.x) + b * p.xs.batch_stride + d * p.xs.dim_stride;
    const long long row = b * p.dim + d;
    if (PACKED) {
        if (threadIdx.x == 0) begun_count = 0;
        __syncthreads();
        // requests with tokens, and the tokens after the last request, that
        // begin at begin - E - H or later; each begins at a token of its own
        for (int s = threadIdx.x; s <= p.req.requests; s += kThreads) {
            const int at = p.req.offset(s), until = s < p.req.requests ? p.req.offset(s + 1) : len;
            if (at < until && at > begin - E - H && at < begin + span) {
                const int i = atomicAdd(&begun_count, 1);
                if (i < kMaxStrip * kTile + 16) begun[i] = s;
            }
        }
        if (strip == 0 && group == 0) p.req.check(threadIdx.x, kThreads);
        if (p.strips > 1) sscan::griddep_launch_dependents();
    }
    if (d < p.dim) {
        T* yrow = static_cast<T*>(p.y) + row * p.len;
        const int lead = VEC ? phase_of(xrow) : 0;  // of the row's first window before the tile
        const int stop = begin + span < len + lead ? begin + span : len + lead;
        // lane 0's window begins up to 2E - 1 before the tile
        const unsigned insides = VEC && len >= kTile + 2 * E ? (unsigned)(len - kTile - 2 * E) + 1u : 0u;
        auto inside = [&](int at) { return VEC && (unsigned)(at - 2 * E) < insides; };
        auto load = [&](int at) {
            const int t0 = at + (lane - 1) * E - lead;
            return inside(at) ? load_raw<T, VEC, true>(xrow, t0, len) : load_raw<T, VEC, false>(xrow, t0, len);
        };
        uint4 now = load(begin), next = now;
        if (begin + kTile < stop) next = load(begin + kTile);
        float w[W];
        load_weights<W>(p.w, d, p.w_aligned, w);
        const float bias = p.bias != nullptr ? __ldg(p.bias + d) : 0.f;
        for (int at = begin; at < stop; at += kTile) {
            const uint4 raw = now;
            now = next;
            if (at + 2 * kTile < stop) next = load(at + 2 * kTile);
            const int t0 = at + (lane - 1) * E - lead;
            if (inside(at)) conv_tile<T, W, VEC, true>(p, raw, w, bias, yrow, row, t0, len);
            else conv_tile<T, W, VEC, false>(p, raw, w, bias, yrow, row, t0, len);
        }
        if (!PACKED && p.final_state != nullptr && strip == 0 && lane < H) {
            const int t = len - H + lane;
            static_cast<T*>(p.final_state)[row * H + lane] =
                t >= 0 ? xrow[t] : p.x0 != nullptr ? static_cast<const T*>(p.x0)[row * H + H + t] : sscan::from_f32<T>(0.f);
        }
    }
    if (PACKED) {
        __syncthreads();
        const int n = begun_count < kMaxStrip * kTile + 16 ? begun_count : kMaxStrip * kTile + 16;
        for (int i = threadIdx.x; i < n * kWarps * H; i += kThreads) {
            const int dist = i % H, s = begun[i / H / kWarps];
            const long long c = cta0 + i / H % kWarps;
            if (c >= p.dim) continue;
            const T* xc = static_cast<const T*>(p.x) + c * p.xs.dim_stride;
            const int at = p.req.offset(s), t = at + dist;
            const int mine0 = begin - (VEC ? phase_of(xc) : 0);
            const int until = s < p.req.requests ? p.req.offset(s + 1) : len;
            if (t >= until || t < mine0 || t >= mine0 + span) continue;
            const int slot = s < p.req.requests && p.req.continues(s) ? p.req.slot(s) : -1;
            const T* st = static_cast<const T*>(p.state) + ((long long)slot * p.dim + c) * H;
            float a = p.bias != nullptr ? __ldg(p.bias + c) : 0.f;
#pragma unroll
            for (int k = 0; k < W; ++k) {
                const int back = dist - H + k;  // token of the request, or before it
                const float tap = back >= 0 ? sscan::to_f32(xc[at + back]) : slot >= 0 ? sscan::to_f32(st[H + back]) : 0.f;
                a = fmaf(__ldg(p.w + c * W + k), tap, a);
            }
            static_cast<T*>(p.y)[c * p.len + t] = sscan::from_f32<T>(p.silu ? a * sscan::fast_sigmoid(a) : a);
        }
        // the cache rows of requests whose states no other CTA reads, and this one has read
        __syncthreads();
        const long long c = cta0 + threadIdx.x % kWarps;
        const T* xc = static_cast<const T*>(p.x) + c * p.xs.dim_stride;
        const bool all = p.strips == 1;
        for (int i = threadIdx.x / kWarps; i < (all ? p.req.requests : n) && c < p.dim; i += kThreads / kWarps) {
            const int s = all ? i : begun[i];
            if (all || (s < p.req.requests && p.req.offset(s) >= begin && apart<E>(p, s) < 0))
                keep_state<T, W>(p, xc, c, s);
        }
    }
}

// The cache rows that the kernel above left (16411 tokens of 48 requests: the
// call takes 82 us when this kernel updates all of them): one thread per (request,
// channel), after it in the same stream.
template <typename T, int W>
__global__ void __launch_bounds__(kThreads) sconv_state_kernel(const __grid_constant__ ConvParams p) {
    const long long d = (long long)blockIdx.x * kThreads + threadIdx.x;
    sscan::griddep_wait();
    if (d >= p.dim) return;
    for (int s = blockIdx.y; s < p.req.requests; s += gridDim.y)
        if (p.len == 0 || apart<VecOf<T>::E>(p, s) >= 0)
            keep_state<T, W>(p, static_cast<const T*>(p.x) + d * p.xs.dim_stride, d, s);
}

// ---- gradients -------------------------------------------------------------
//
//   dc[t] = dy[t] * silu'(c[t]),  silu'(c) = s (1 + c (1 - s)),  s = sigmoid(c)
//   dx[t] = sum_k w[k] dc[t + (W-1) - k]  (+ the final state's gradient)
//   dw[k] = sum_{b,t} dc[t] x[t - (W-1) + k],   dbias = sum_{b,t} dc[t]
//
// One CTA owns one channel: its warps walk pieces of 30 windows of the
// channel's rows in every batch (lane 0's window supplies the inputs before
// lane 1's, lane 31's the W-1 values of dc after lane 30's), each loading the
// next piece before it works on the last.  c is recomputed from x.  The sums
// over batch and time stay in registers and meet in shared memory in a fixed
// order, so the gradients do not depend on scheduling.
struct ConvBwdParams {
    const void* x;
    const float* w;
    const float* bias;
    const void* x0;
    const void* dy;            // contiguous
    const void* dfinal;        // [batch, dim, W-1] or NULL
    void* dx;                  // contiguous
    float* dw;
    float* dbias;              // or NULL
    void* dx0;                 // [batch, dim, W-1] or NULL
    long long batch, dim, len;
    Rows xs;
    int silu;
    bool w_aligned;  // weight rows of four are 16-byte vectors
};

constexpr int kBwdMost = 512;  // threads of a channel's CTA at most

template <typename T, int W, bool VEC>
__global__ void __launch_bounds__(kBwdMost, 2) sconv_bwd_kernel(const __grid_constant__ ConvBwdParams p) {
    constexpr int E = VecOf<T>::E;
    constexpr int H = W - 1;
    constexpr int STEP = 30 * E;
    __shared__ float part[kBwdMost / 32][W + 1];
    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const long long d = blockIdx.x;
    float w[W];
    const float bias = p.bias != nullptr ? __ldg(p.bias + d) : 0.f;
    load_weights<W>(p.w, d, p.w_aligned, w);
    auto silu_slope = [](float c) {
        const float s = sscan::fast_sigmoid(c);
        return s * fmaf(c, 1.f - s, 1.f);
    };
    float dw[W], db = 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) dw[k] = 0.f;
    const int len = (int)p.len;
    const int pieces = (len + E - 1 + STEP - 1) / STEP;  // E - 1: the row's phase
    // this warp's pieces in order, and the rows they lie in
    int piece = warp, bi = 0;
    const T* xrow = static_cast<const T*>(p.x) + d * p.xs.dim_stride;
    const T* dyrow = static_cast<const T*>(p.dy) + d * p.len;
    T* dxrow = static_cast<T*>(p.dx) + d * p.len;
    const long long next_row = p.dim * p.len;
    auto settle = [&]() {
        while (piece >= pieces && bi < p.batch) {
            piece -= pieces;
            ++bi;
            xrow += p.xs.batch_stride;
            dyrow += next_row;
            dxrow += next_row;
        }
        return bi < p.batch;
    };
    auto start = [&]() { return piece * STEP + (lane - 1) * E - (VEC ? phase_of(xrow) : 0); };
    const unsigned insides = VEC && len >= 33 * E + H ? (unsigned)(len - 33 * E - H) + 1u : 0u;
    auto inside = [&]() { return VEC && (unsigned)(piece * STEP - 2 * E) < insides; };
    uint4 xraw, graw;
    auto fetch = [&](int t0) {
        if (inside()) {
            xraw = load_raw<T, VEC, true>(xrow, t0, len);
            graw = load_raw<T, VEC, true>(dyrow, t0, len);
        } else {
            xraw = load_raw<T, VEC, false>(xrow, t0, len);
            graw = load_raw<T, VEC, false>(dyrow, t0, len);
        }
    };
    // One piece, and the next one's loads.  INSIDE: all its windows lie inside
    // the row, before the last H tokens, and no inputs before it count (as
    // predicated blocks the exceptions cost a fifth of the instructions).
    bool more = pieces > 0 && settle();
    int t0 = 0;
    if (more) fetch(t0 = start());
    auto work = [&](auto inside_tag) {
        constexpr bool INSIDE = decltype(inside_tag)::value;
        const int t = t0;
        T* const to = dxrow;
        const long long at = bi * p.dim + d;
        float v[H + E], dc[E + H], own[E], g[E];
        if (!INSIDE && p.x0 != nullptr && t < 0) xraw = put_before<T, H>(xraw, static_cast<const T*>(p.x0) + at * H, t);
        sscan::widen(xraw, own, static_cast<T*>(nullptr));
        sscan::widen(graw, g, static_cast<T*>(nullptr));
        piece += warps;
        more = settle();
        if (more) fetch(t0 = start());
#pragma unroll
        for (int j = 0; j < E; ++j) v[H + j] = own[j];
#pragma unroll
        for (int j = 0; j < H; ++j) v[j] = __shfl_up_sync(0xffffffffu, v[E + j], 1);
#pragma unroll
        for (int j = 0; j < E; ++j) {
            float c = bias;
#pragma unroll
            for (int k = 0; k < W; ++k) c = fmaf(w[k], v[j + k], c);
            dc[j] = c;
        }
        if (p.silu) {
#pragma unroll
            for (int j = 0; j < E; ++j) dc[j] = g[j] * silu_slope(dc[j]);
        } else {
#pragma unroll
            for (int j = 0; j < E; ++j) dc[j] = g[j];
        }
        if (!INSIDE) {  // nothing comes back from outside the row
#pragma unroll
            for (int j = 0; j < E; ++j)
                if (t + j < 0 || t + j >= len) dc[j] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < H; ++j) dc[E + j] = __shfl_down_sync(0xffffffffu, dc[j], 1);
        float dx[E];
#pragma unroll
        for (int j = 0; j < E; ++j) {
            float a = 0.f;
#pragma unroll
            for (int k = 0; k < W; ++k) a = fmaf(w[k], dc[j + H - k], a);
            dx[j] = a;
        }
        if (!INSIDE && p.dfinal != nullptr && t + E > len - H) {
            const T* df = static_cast<const T*>(p.dfinal) + at * H;
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const int back = t + j - (len - H);
                if (t + j >= 0 && back >= 0 && back < H) dx[j] += sscan::to_f32(df[back]);
            }
        }
        if (lane > 0 && lane < 31) {
#pragma unroll
            for (int j = 0; j < E; ++j) {
                // (outside the row dc is zero, but an input beside it may be infinite)
                if (!INSIDE && (t + j < 0 || t + j >= len)) continue;
                db += dc[j];
#pragma unroll
                for (int k = 0; k < W; ++k) dw[k] = fmaf(dc[j], v[j + k], dw[k]);
            }
            store_window<T, VEC, INSIDE>(to, t, len, dx);
        }
    };
    while (more) {
        if (inside()) work(std::true_type{});
        else work(std::false_type{});
    }
    if (p.dx0 != nullptr) {
        // gradients of the inputs before the sequence: the first tokens' dc
        for (long long b = threadIdx.x; b < p.batch; b += blockDim.x) {
            const T* xrow = static_cast<const T*>(p.x) + b * p.xs.batch_stride + d * p.xs.dim_stride;
            const long long row = b * p.dim + d;
            const T* dyrow = static_cast<const T*>(p.dy) + row * p.len;
            float dc[H];
            for (int t = 0; t < H; ++t) {
                dc[t] = 0.f;
                if (t >= p.len) continue;
                float c = bias;
                for (int k = 0; k < W; ++k) {
                    const int at = t - H + k;
                    const float tap = at >= 0 ? sscan::to_f32(xrow[at])
                                      : p.x0 != nullptr ? sscan::to_f32(static_cast<const T*>(p.x0)[row * H + H + at]) : 0.f;
                    c = fmaf(w[k], tap, c);
                }
                dc[t] = sscan::to_f32(dyrow[t]) * (p.silu ? silu_slope(c) : 1.f);
            }
            for (int j = 0; j < H; ++j) {  // x[j - H]
                float a = 0.f;
                for (int t = 0; t < H; ++t) {
                    const int k = j - t;  // t = (j - H) + H - k
                    if (k >= 0) a = fmaf(w[k], dc[t], a);
                }
                const long long back = j - p.len;  // its place in the final state when the sequence is short
                if (p.dfinal != nullptr && back >= 0) a += sscan::to_f32(static_cast<const T*>(p.dfinal)[row * H + back]);
                static_cast<T*>(p.dx0)[row * H + j] = sscan::from_f32<T>(a);
            }
        }
    }
#pragma unroll
    for (int k = 0; k < W; ++k) {
        dw[k] = sscan::warp_sum(dw[k]);
        if (lane == 0) part[warp][k] = dw[k];
    }
    db = sscan::warp_sum(db);
    if (lane == 0) part[warp][W] = db;
    __syncthreads();
    if (threadIdx.x <= W) {
        float a = 0.f;
        for (int i = 0; i < warps; ++i) a += part[i][threadIdx.x];
        if (threadIdx.x < W) p.dw[d * W + threadIdx.x] = a;
        else if (p.dbias != nullptr) p.dbias[d] = a;
    }
}

// ---- single tokens ---------------------------------------------------------

struct ConvStepParams {
    const void* x;
    const float* w;
    const float* bias;
    void* state;
    void* y;
    long long batch, dim, x_stride;
    int silu;
    Requests req;
};

// A thread owns V consecutive channels of R tokens: the W-1 cached inputs of
// a token are V*(W-1) consecutive values of its cache row.  All R tokens' rows are on the
// way before the first is used, and the weights are read once for them.
// V = a 16-byte vector, or 1.
constexpr int kStepThreads = 128;

template <typename T, int W, int V, int R>
__global__ void __launch_bounds__(kStepThreads) sconv_step_kernel(const __grid_constant__ ConvStepParams p) {
    constexpr int H = W - 1;
    constexpr int E = VecOf<T>::E;
    const long long d = ((long long)blockIdx.x * kStepThreads + threadIdx.x) * V;
    if (blockIdx.x == 0 && blockIdx.y == 0) p.req.check(threadIdx.x, kStepThreads);
    if (d >= p.dim) return;
    for (long long b0 = (long long)blockIdx.y * R; b0 < p.batch; b0 += (long long)gridDim.y * R) {
        int slot[R];
#pragma unroll
        for (int r = 0; r < R; ++r) slot[r] = b0 + r < p.batch ? p.req.slot((int)(b0 + r)) : -1;
        if constexpr (V > 1) {
            uint4 xq[R], old[R][H];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const uint4* st = reinterpret_cast<const uint4*>(static_cast<const T*>(p.state) + ((long long)slot[r] * p.dim + d) * H);
                xq[r] = make_uint4(0u, 0u, 0u, 0u);
                if (b0 + r < p.batch)
                    xq[r] = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(p.x) + (b0 + r) * p.x_stride + d));
#pragma unroll
                for (int i = 0; i < H; ++i) old[r][i] = slot[r] >= 0 ? st[i] : make_uint4(0u, 0u, 0u, 0u);
            }
            float w[V][W], bias[V];  // V * W consecutive weights, V biases
#pragma unroll
            for (int i = 0; i < V * W; i += 4) {
                const float4 q = __ldg(reinterpret_cast<const float4*>(p.w + d * W + i));
                w[i / W][i % W] = q.x; w[(i + 1) / W][(i + 1) % W] = q.y;
                w[(i + 2) / W][(i + 2) % W] = q.z; w[(i + 3) / W][(i + 3) % W] = q.w;
            }
#pragma unroll
            for (int i = 0; i < V; i += 4) {
                float4 q = make_float4(0.f, 0.f, 0.f, 0.f);
                if (p.bias != nullptr) q = __ldg(reinterpret_cast<const float4*>(p.bias + d + i));
                bias[i] = q.x; bias[i + 1] = q.y; bias[i + 2] = q.z; bias[i + 3] = q.w;
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (b0 + r >= p.batch) break;
                float xv[E], out[E], was[H][E];
                sscan::widen(xq[r], xv, static_cast<T*>(nullptr));
#pragma unroll
                for (int i = 0; i < H; ++i) sscan::widen(old[r][i], was[i], static_cast<T*>(nullptr));
                // input k of channel c is value c * H + k of the row
#pragma unroll
                for (int c = 0; c < V; ++c) {
                    float a = fmaf(w[c][H], xv[c], bias[c]);
#pragma unroll
                    for (int k = 0; k < H; ++k) a = fmaf(w[c][k], was[(c * H + k) / E][(c * H + k) % E], a);
                    out[c] = p.silu ? a * sscan::fast_sigmoid(a) : a;
                }
                *reinterpret_cast<uint4*>(static_cast<T*>(p.y) + (b0 + r) * p.dim + d) =
                    sscan::narrow(out, static_cast<T*>(nullptr));
                if (slot[r] < 0) continue;
                // the cached inputs move up by one; the token's own comes last
                uint4* st = reinterpret_cast<uint4*>(static_cast<T*>(p.state) + ((long long)slot[r] * p.dim + d) * H);
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    float now[E];
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const int c = (i * E + e) / H, k = (i * E + e) % H, from = c * H + k + 1;
                        now[e] = k + 1 < H ? was[from / E < H ? from / E : 0][from % E] : xv[c];
                    }
                    st[i] = sscan::narrow(now, static_cast<T*>(nullptr));
                }
            }
        } else {
            const float bias = p.bias != nullptr ? __ldg(p.bias + d) : 0.f;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (b0 + r >= p.batch) break;
                T* st = static_cast<T*>(p.state) + ((long long)slot[r] * p.dim + d) * H;
                T old[H];
#pragma unroll
                for (int k = 0; k < H; ++k) old[k] = slot[r] >= 0 ? st[k] : sscan::from_f32<T>(0.f);
                const T xv = static_cast<const T*>(p.x)[(b0 + r) * p.x_stride + d];
                float a = fmaf(__ldg(p.w + d * W + H), sscan::to_f32(xv), bias);
#pragma unroll
                for (int k = 0; k < H; ++k) a = fmaf(__ldg(p.w + d * W + k), sscan::to_f32(old[k]), a);
                static_cast<T*>(p.y)[(b0 + r) * p.dim + d] = sscan::from_f32<T>(p.silu ? a * sscan::fast_sigmoid(a) : a);
                if (slot[r] >= 0) {
#pragma unroll
                    for (int k = 0; k < H; ++k) st[k] = k + 1 < H ? old[k + 1] : xv;
                }
            }
        }
    }
}

// ---- host side --------------------------------------------------------------

constexpr long long kBig = 1LL << 40;
constexpr long long kIntMax = 1LL << 30;  // token, request and channel numbers are 32-bit on the device

bool sizes_ok(long long a, long long b, long long c) {
    return a >= 0 && b >= 0 && c >= 0 && a <= kBig && b <= kBig && c <= kBig && (!a || b <= kBig / a) &&
           (!(a * b) || c <= kBig / (a * b));
}

// Whether every row of x and of a contiguous [batch, dim, len] array lies the
// same way against 16-byte boundaries.
bool same_phase(const void* x, const void* y, Rows xs, long long batch, long long dim, long long len, int esz) {
    const long long e = 16 / esz;
    const uintptr_t ax = reinterpret_cast<uintptr_t>(x), ay = reinterpret_cast<uintptr_t>(y);
    return (ax - ay) % 16 == 0 && ax % esz == 0 && (dim <= 1 || (xs.dim_stride - len) % e == 0) &&
           (batch <= 1 || (xs.batch_stride - dim * len) % e == 0);
}

// Tiles of 31 windows of a row, and how many a warp takes: up to eight while
// the warps still fill the SMs twice, at 40 each (4 x 2048 x 2048 bf16: 18.5 us;
// 19.6 when they need fill them once, 19.2 four times).
long long tiles_of(const ConvParams& p, bool vec, int window) {
    return sscan::div_up(p.len + (vec ? window - 1 : 0), 31LL * window);
}
int strip_tiles(const ConvParams& p, bool vec, int window) {
    const long long tiles = tiles_of(p, vec, window);
    int n = 1;
    while (n < kMaxStrip && n < tiles && p.batch * p.dim * tiles / (n + 1) >= 2 * 40 * 152) ++n;
    return n;
}

template <typename T, int W, bool PACKED>
cudaError_t run_fwd(const ConvParams& p0, bool vec, cudaStream_t st) {
    ConvParams p = p0;
    constexpr int E = VecOf<T>::E;
    p.strip_tiles = strip_tiles(p, vec, E);
    p.strips = (unsigned)sscan::div_up(tiles_of(p, vec, E), p.strip_tiles);
    p.groups = (unsigned)sscan::div_up(p.dim, kWarps);
    p.w_aligned = sscan::is_aligned(p.w, 16);
    p.flat = p.groups > 65535 || p.batch > 65535;
    const dim3 grid = p.flat ? dim3((unsigned)((long long)p.strips * p.groups * p.batch)) : dim3(p.strips, p.groups, (unsigned)p.batch);
    if (vec) return sscan::launch(sconv_fwd_kernel<T, W, PACKED, true>, grid, dim3(kThreads), 0, st, false, p);
    return sscan::launch(sconv_fwd_kernel<T, W, PACKED, false>, grid, dim3(kThreads), 0, st, false, p);
}
template <typename T, int W>
cudaError_t run_state(const ConvParams& p0, bool vec, bool dependent, cudaStream_t st) {
    ConvParams p = p0;
    p.strip_tiles = strip_tiles(p, vec, VecOf<T>::E);  // the strips of the kernel before it
    const dim3 grid((unsigned)sscan::div_up(p.dim, kThreads), (unsigned)(p.req.requests < 65535 ? p.req.requests : 65535));
    return sscan::launch(sconv_state_kernel<T, W>, grid, dim3(kThreads), 0, st, dependent, p);
}
template <typename T, int W>
cudaError_t run_bwd(const ConvBwdParams& p0, bool vec, cudaStream_t st) {
    ConvBwdParams p = p0;
    p.w_aligned = sscan::is_aligned(p.w, 16);
    // four warps a channel (2048 channels of 4 x 2048 tokens: 27.7 us; 30.7 with
    // eight, whose pieces do not come out even), more where the channels alone
    // would leave SMs idle
    const dim3 grid((unsigned)p.dim), block(p.dim >= 8 * 152 ? 128 : p.dim >= 2 * 152 ? 256 : kBwdMost);
    if (vec) return sscan::launch(sconv_bwd_kernel<T, W, true>, grid, block, 0, st, false, p);
    return sscan::launch(sconv_bwd_kernel<T, W, false>, grid, block, 0, st, false, p);
}
template <typename T, int W, int R>
cudaError_t run_tokens(const ConvStepParams& p, bool vec, cudaStream_t st) {
    constexpr int E = VecOf<T>::E;
    const long long gx = sscan::div_up(p.dim, (long long)kStepThreads * (vec ? E : 1)), gy = sscan::div_up(p.batch, R);
    const dim3 grid((unsigned)gx, (unsigned)(gy < 65535 ? gy : 65535));
    if (vec) return sscan::launch(sconv_step_kernel<T, W, E, R>, grid, dim3(kStepThreads), 0, st, false, p);
    return sscan::launch(sconv_step_kernel<T, W, 1, R>, grid, dim3(kStepThreads), 0, st, false, p);
}
template <typename T, int W>
cudaError_t run_step(const ConvStepParams& p, bool vec, cudaStream_t st) {
    // two tokens a thread where that leaves every SM a few CTAs
    const long long ctas = p.batch * sscan::div_up(p.dim, (long long)kStepThreads * (vec ? VecOf<T>::E : 1));
    return ctas >= 8 * 152 ? run_tokens<T, W, 2>(p, vec, st) : run_tokens<T, W, 1>(p, vec, st);
}

// F<T, W>(args...) for the dtype and width (2 .. 4)
#define SCONV_DISPATCH(F, ...)                                                        \
    (dtype == SSCAN_F32 ? (width == 2   ? F(float, 2)(__VA_ARGS__)                    \
                           : width == 3 ? F(float, 3)(__VA_ARGS__)                    \
                                        : F(float, 4)(__VA_ARGS__))                   \
                        : (width == 2   ? F(bf16, 2)(__VA_ARGS__)                     \
                           : width == 3 ? F(bf16, 3)(__VA_ARGS__)                     \
                                        : F(bf16, 4)(__VA_ARGS__)))
#define SCONV_FWD(T, W) run_fwd<T, W, false>
#define SCONV_PACKED(T, W) run_fwd<T, W, true>
#define SCONV_STATE(T, W) run_state<T, W>
#define SCONV_BWD(T, W) run_bwd<T, W>
#define SCONV_STEP(T, W) run_step<T, W>

// Channels, and the forward kernel's CTAs, fit a grid's first dimension.
bool grid_ok(long long batch, long long dim, long long len) {
    return dim <= kIntMax && batch <= kIntMax && len <= kIntMax &&
           sscan::div_up(len + 8, 124) <= kIntMax / (sscan::div_up(dim, kWarps) * (batch > 0 ? batch : 1));
}
bool common_ok(long long width, int dtype, int flags) {
    return (dtype == SSCAN_F32 || dtype == SSCAN_BF16) && width >= 2 && width <= SCONV_MAX_WIDTH &&
           (flags & ~SCONV_SILU) == 0;
}

}  // namespace

extern "C" int sconv_fwd(const void* x, const float* weight, const float* bias, const void* x0, void* y,
                         void* final_state, int64_t batch, int64_t dim, int64_t seqlen, int64_t width,
                         int64_t x_batch_stride, int64_t x_dim_stride, int dtype, int flags, void* stream) {
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    sscan::record_call(0, st, "rejected");
    if (!common_ok(width, dtype, flags) || !sizes_ok(batch, dim, seqlen)) return SSCAN_ERR_INVALID;
    if (x_batch_stride < 0 || x_dim_stride < 0 || (dim && !grid_ok(batch, dim, seqlen))) return SSCAN_ERR_INVALID;
    if (batch == 0 || dim == 0) {
        sscan::record_call(0, st, "empty");
        return SSCAN_OK;
    }
    if (seqlen == 0) {  // the state passes through
        const size_t bytes = (size_t)(batch * dim * (width - 1)) * (dtype == SSCAN_F32 ? 4 : 2);
        sscan::record_call(0, st, "sconv seqlen 0: final_state = x0");
        if (final_state == nullptr || final_state == x0) return SSCAN_OK;
        return sscan::finish(x0 ? cudaMemcpyAsync(final_state, x0, bytes, cudaMemcpyDeviceToDevice, st)
                                : cudaMemsetAsync(final_state, 0, bytes, st));
    }
    if (!x || !weight || !y) return SSCAN_ERR_INVALID;
    ConvParams p = {};
    p.x = x; p.w = weight; p.bias = bias; p.x0 = x0; p.final_state = final_state; p.y = y;
    p.batch = batch; p.dim = dim; p.len = seqlen;
    p.xs = Rows{x_batch_stride, x_dim_stride};
    p.silu = flags & SCONV_SILU;
    const bool vec = same_phase(x, y, p.xs, batch, dim, seqlen, dtype == SSCAN_F32 ? 4 : 2);
    sscan::record_call(1, st, vec ? "sconv fwd vec=1" : "sconv fwd vec=0");
    return sscan::finish(SCONV_DISPATCH(SCONV_FWD, p, vec, st));
}

extern "C" int sconv_bwd(const void* x, const float* weight, const float* bias, const void* x0, const void* dy,
                         const void* dfinal_state, void* dx, float* dweight, float* dbias, void* dx0, int64_t batch,
                         int64_t dim, int64_t seqlen, int64_t width, int64_t x_batch_stride, int64_t x_dim_stride,
                         int dtype, int flags, void* stream) {
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    sscan::record_call(0, st, "rejected");
    if (!common_ok(width, dtype, flags) || !sizes_ok(batch, dim, seqlen)) return SSCAN_ERR_INVALID;
    if (x_batch_stride < 0 || x_dim_stride < 0 || (dim && !grid_ok(batch, dim, seqlen))) return SSCAN_ERR_INVALID;
    if (dim == 0) {
        sscan::record_call(0, st, "empty");
        return SSCAN_OK;
    }
    if (!weight || !dweight || (batch && seqlen && (!x || !dy || !dx))) return SSCAN_ERR_INVALID;
    ConvBwdParams p = {};
    p.x = x; p.w = weight; p.bias = bias; p.x0 = x0; p.dy = dy; p.dfinal = dfinal_state;
    p.dx = dx; p.dw = dweight; p.dbias = dbias; p.dx0 = dx0;
    p.batch = batch; p.dim = dim; p.len = seqlen;
    p.xs = Rows{x_batch_stride, x_dim_stride};
    p.silu = flags & SCONV_SILU;
    const int esz = dtype == SSCAN_F32 ? 4 : 2;
    const bool vec = same_phase(x, dy, p.xs, batch, dim, seqlen, esz) && same_phase(x, dx, p.xs, batch, dim, seqlen, esz);
    sscan::record_call(1, st, vec ? "sconv bwd vec=1" : "sconv bwd vec=0");
    return sscan::finish(SCONV_DISPATCH(SCONV_BWD, p, vec, st));
}

extern "C" int sconv_prompt(const void* x, const float* weight, const float* bias, const int32_t* cu_seqlens,
                            const int32_t* slots, const uint8_t* has_state, void* state, void* y, int64_t requests,
                            int64_t num_slots, int64_t dim, int64_t tokens, int64_t width, int64_t x_dim_stride,
                            int dtype, int flags, void* stream) {
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    sscan::record_call(0, st, "rejected");
    if (!common_ok(width, dtype, flags) || !sizes_ok(1, dim, tokens) || !sizes_ok(num_slots, dim, width))
        return SSCAN_ERR_INVALID;
    if (x_dim_stride < 0 || requests < 0 || requests > kIntMax || tokens > kIntMax || num_slots > kIntMax ||
        (slots == nullptr && requests > num_slots) || (dim && !grid_ok(1, dim, tokens)))
        return SSCAN_ERR_INVALID;
    if (dim == 0 || (requests == 0 && tokens == 0)) {
        sscan::record_call(0, st, "empty");
        return SSCAN_OK;
    }
    if (!weight || !cu_seqlens || (num_slots && !state) || (tokens && (!x || !y))) return SSCAN_ERR_INVALID;
    ConvParams p = {};
    p.x = x; p.w = weight; p.bias = bias; p.state = state; p.y = y;
    p.batch = 1; p.dim = dim; p.len = tokens;
    p.xs = Rows{0, x_dim_stride};
    p.silu = flags & SCONV_SILU;
    int* status = sscan::device_status_word();
    if (status == nullptr) return sscan::finish(cudaErrorUnknown);
    p.req = Requests{cu_seqlens, slots, has_state, (int)requests, (int)num_slots, (int)tokens, status};
    const bool vec = same_phase(x, y, p.xs, 1, dim, tokens, dtype == SSCAN_F32 ? 4 : 2);
    // where one strip holds all tokens the convolution's CTAs update the whole cache
    const int window = dtype == SSCAN_F32 ? 4 : 8;
    const bool state_pass = requests > 0 && (tokens == 0 || tiles_of(p, vec, window) > strip_tiles(p, vec, window));
    sscan::record_call((tokens > 0) + state_pass, st, vec ? "sconv prompt vec=1" : "sconv prompt vec=0");
    cudaError_t e = cudaSuccess;
    if (tokens > 0) e = SCONV_DISPATCH(SCONV_PACKED, p, vec, st);
    if (e == cudaSuccess && state_pass) e = SCONV_DISPATCH(SCONV_STATE, p, vec, tokens > 0, st);
    return sscan::finish(e);
}

extern "C" int sconv_step(const void* x, const float* weight, const float* bias, const int32_t* slots, void* state,
                          void* y, int64_t batch, int64_t num_slots, int64_t dim, int64_t width, int64_t x_stride,
                          int dtype, int flags, void* stream) {
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    sscan::record_call(0, st, "rejected");
    if (!common_ok(width, dtype, flags) || !sizes_ok(batch, dim, width) || !sizes_ok(num_slots, dim, width))
        return SSCAN_ERR_INVALID;
    if (x_stride < 0 || batch > kIntMax || num_slots > kIntMax || (slots == nullptr && batch > num_slots) ||
        dim > kIntMax)
        return SSCAN_ERR_INVALID;
    if (batch == 0 || dim == 0) {
        sscan::record_call(0, st, "empty");
        return SSCAN_OK;
    }
    if (!x || !weight || !y || (num_slots && !state)) return SSCAN_ERR_INVALID;
    ConvStepParams p = {};
    p.x = x; p.w = weight; p.bias = bias; p.state = state; p.y = y;
    p.batch = batch; p.dim = dim; p.x_stride = x_stride;
    p.silu = flags & SCONV_SILU;
    int* status = sscan::device_status_word();
    if (status == nullptr) return sscan::finish(cudaErrorUnknown);
    p.req = Requests{nullptr, slots, nullptr, (int)batch, (int)num_slots, 0, status};
    const int e = dtype == SSCAN_F32 ? 4 : 8;
    const bool vec = dim % e == 0 && (batch == 1 || x_stride % e == 0) && sscan::is_aligned(x, 16) &&
                     sscan::is_aligned(y, 16) && sscan::is_aligned(state, 16) && sscan::is_aligned(weight, 16) &&
                     sscan::is_aligned(bias, 16);
    sscan::record_call(1, st, vec ? "sconv step vec=1" : "sconv step vec=0");
    return sscan::finish(SCONV_DISPATCH(SCONV_STEP, p, vec, st));
}
