// RMS norms of queries and keys for each head, with the rotation by position in
// the same pass, on sm_103a.  Per token and head, over its D channels:
//
//   y = x * rstd * w,   rstd = 1 / sqrt(mean(x^2) + eps)
//   channels i and i + r of y, i < r, turn by the angle pos * freq[i]:
//   out_i = y_i cos - y_{i+r} sin,   out_{i+r} = y_{i+r} cos + y_i sin
//
// (r = the number of frequencies; channels from 2r on stay as they are).  Gradients, from
// the upstream gradient turned back, u, with n = x * rstd and g = u * w:
//
//   dx = rstd * (g - n * mean(g * n)),   dw = sum over tokens and heads of u * n
//
// Angles.  An angle is needed modulo one turn, and pos is an integer, so the
// frequency counts only by the fraction of a turn that it adds per position: that fraction
// as a 64-bit integer times pos, modulo 2^64, is the angle without any rounding of its
// own, however far the position (2^-64 of a turn times pos from the fraction's
// rounding, for frequencies up to 2^44 either way).  In fp32 pos * freq would be off by 2^-24 of the whole
// angle: 0.03 rad at position 500,000.
//
// A few operations a value: HBM should bound it; by measurement the issue of instructions and
// the sums' exchanges do.  Layout [batch, heads * D, L]: a warp takes V vectors of 16 bytes of tokens
// of one head at a time, all channels in registers: lane = vector x channels (32 / V lanes share
// them, each with pairs that turn together), so that the sums over channels stay in the warp and
// inputs are read once.  A CTA takes a run of heads, tile of 32 tokens by tile, and forms a tile's cosines
// and sines once, in shared memory.  4 x 2048 tokens x 32 heads of 128 in bf16: forward 35 us
// (3.8 TB/s), gradients 67 us (3.0 TB/s); 8209 tokens x 48 heads, rows off 16-byte boundaries, 74 us
// (2.7 TB/s); with tiles of 64 tokens for six heads, and one value an operation, 49, 101 and 137 us; three CTAs
// an SM in the forward pass 45 us: their registers spill.
#include <stdio.h>

#include "block_utils.cuh"
#include "piece_loads.cuh"

namespace {

using sscan::bf16;

constexpr int kTile = 32;   // tokens of a tile
constexpr int kWarps = 8;

struct QkParams {
    const void* x[2];   // q, k
    const void* dy[2];
    void* y[2];         // outputs, or dq and dk
    const float* w[2];
    float* dw[2];
    float* parts;       // [ctas][2][D]
    const int* pos;     // [batch][L]
    const float* freq;  // [r]
    long long xb[2], xd[2];  // batch and channel strides of q and k
    int heads[2];
    long long batch, L;
    int D, r;
    long long per;      // (tile, head) units of a CTA, tile by tile, a tile's queries before its keys
    float eps;
};

// The fraction of a turn that a frequency adds per position, in units of 2^-64.  1 / (2 pi) stands in two
// doubles, 107 bits, so that what the product's rounding leaves out counts as well: in one double the fraction would be off
// by 2^-54 of all turns, 1e-5 rad at position 2^31 for a frequency of 100.  Whole turns drop out of both parts,
// which are signed, so that a small one keeps its bits.  2^-64 off for |freq| up to 2^44.
__device__ __forceinline__ unsigned long long turn_of(float freq) {
    const double f = (double)freq, high = 0.15915494309189535, low = -9.839338337591243e-18;  // 1 / (2 pi)
    const double t = f * high, rest = fma(f, low, fma(f, high, -t));
    const double unit = 18446744073709551616.0;
    return (unsigned long long)__double2ll_rn((t - rint(t)) * unit) + (unsigned long long)__double2ll_rn((rest - rint(rest)) * unit);
}
// The upper half of (turn * pos) modulo 2^64 as it stands, signed: [-1/2, 1/2) of a turn to 2^-32.
__device__ __forceinline__ void cos_sin(unsigned long long turn, int pos, float& c, float& s) {
    const unsigned lo = (unsigned)turn, hi = (unsigned)(turn >> 32);
    const unsigned a = hi * (unsigned)pos + __umulhi(lo, (unsigned)pos) - (pos < 0 ? lo : 0u);
    sincospif(__int2float_rn((int)a) * 4.656612873077393e-10f, &s, &c);  // 2^-31 half turns
}

// Two values at a time.
struct Two {
    unsigned long long v;
    __device__ __forceinline__ float x() const { return __uint_as_float((unsigned)v); }
    __device__ __forceinline__ float y() const { return __uint_as_float((unsigned)(v >> 32)); }
};
__device__ __forceinline__ Two two(float x, float y) {
    return Two{(unsigned long long)__float_as_uint(x) | (unsigned long long)__float_as_uint(y) << 32};
}
__device__ __forceinline__ Two operator*(Two a, Two b) {
    Two d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
    return d;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
    Two d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return d;
}
__device__ __forceinline__ void widen2(const uint4& v, Two (&f)[4], bf16*) {
    const unsigned w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = two(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
__device__ __forceinline__ void widen2(const uint4& v, Two (&f)[2], float*) {
    f[0] = two(__uint_as_float(v.x), __uint_as_float(v.y));
    f[1] = two(__uint_as_float(v.z), __uint_as_float(v.w));
}
template <typename T, int E>
__device__ __forceinline__ uint4 narrow2(const Two (&f)[E / 2]) {
    float v[E];
#pragma unroll
    for (int i = 0; i < E / 2; ++i) { v[2 * i] = f[i].x(); v[2 * i + 1] = f[i].y(); }
    return sscan::narrow(v, (T*)nullptr);
}

// One vector of tokens of a channel; VEC: rows lie on 16-byte boundaries.
template <bool VEC>
__device__ __forceinline__ uint4 load_tokens(const float* p, int have) {
    if (VEC && have == 4) return __ldg(reinterpret_cast<const uint4*>(p));
    const unsigned* w = reinterpret_cast<const unsigned*>(p);
    return make_uint4(have > 0 ? __ldg(w) : 0u, have > 1 ? __ldg(w + 1) : 0u, have > 2 ? __ldg(w + 2) : 0u, have > 3 ? __ldg(w + 3) : 0u);
}
template <typename T, bool VEC>
__device__ __forceinline__ void store_tokens(T* p, int have, const uint4& v) {
    constexpr int E = sscan::VecOf<T>::E;
    if (VEC && have == E) {
        *reinterpret_cast<uint4*>(p) = v;
        return;
    }
    const unsigned w[4] = {v.x, v.y, v.z, v.w};
    if (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < have) reinterpret_cast<unsigned*>(p)[i] = w[i];
        return;
    }
    unsigned short* to = reinterpret_cast<unsigned short*>(p);
#pragma unroll
    for (int i = 0; i < E; ++i)
        if (i < have) to[i] = (unsigned short)(w[i / 2 % 4] >> (16 * (i & 1)));
}
// Sums over the 32 / V lanes that share a vector's channels, for each of its E tokens:
// halving exchanges leave a lane with one token's sum, which all then read from it.
template <int V, int E>
__device__ __forceinline__ float channel_sum(float (&v)[E]) {
    const int lane = threadIdx.x & 31;
    int m = 16;
#pragma unroll
    for (int n = E / 2; n > 0; n >>= 1) {
        const bool high = (lane & m) != 0;
#pragma unroll
        for (int j = 0; j < n; ++j) {
            const float give = high ? v[j] : v[j + n], keep = high ? v[j + n] : v[j];
            v[j] = keep + __shfl_xor_sync(0xffffffffu, give, m);
        }
        m >>= 1;
    }
    for (; m >= V; m >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], m);
    return v[0];
}
// (E = 8: token bits 0..2 are lane bits 2..4; E = 4: 3..4)
template <int E>
__device__ __forceinline__ int held_token() { return (threadIdx.x & 31) / (E == 8 ? 4 : 8); }
template <int V, int E>
__device__ __forceinline__ float of_token(float v, int e) {
    return __shfl_sync(0xffffffffu, v, (threadIdx.x & (V - 1)) + (E == 8 ? 4 * e : 8 * e));
}

// A frequency's cosines and sines, four tokens' of each in turn; the pad keeps the lanes of a quarter
// warp, four frequencies by two vectors, in different banks.
constexpr int kTableRow = 2 * kTile + 4;

// bf16 rows that lie anywhere pass through shared memory, both ways: the warps that share a head copy
// a tile's rows by the aligned vectors around them, the next head's while one is worked on, and write
// results by whole words of a row.  Rows eight apart lie at one offset from a 16-byte boundary
// whatever their stride, so a thread takes every eighth row.  Aligned rows come that way as well, for the
// head that is fetched ahead (forward 38 -> 35 us), and are stored straight.  (Straight from registers every store of a word
// touched 16 rows' lines and every vector took two loads: 8209 tokens x 48 heads of 128 took 121 us.)
constexpr int kStageRow = kTile + 8;  // values of a row: a tile's and what the alignment adds

// where the rows lie behind the weights and sums, in floats from the sums on
template <bool BWD>
__host__ __device__ constexpr int stage_at(int D) {
    return (BWD ? 2 * kWarps * D : 0) + (D & 1) * 2;
}

// V: vectors of a row in a warp; KP: pairs of channels a lane, 64 / V * KP >= D
template <typename T, int V, int KP, bool BWD, bool VEC>
__global__ void __launch_bounds__(256, KP <= 4 ? 2 : 1) qknorm_kernel(const QkParams p) {
    constexpr int E = sscan::VecOf<T>::E, kSpan = V * E, kSets = kTile / kSpan, kHeads = kWarps / kSets, kShares = 32 / V;
    constexpr bool STAGED = sizeof(T) == 2, OUT_STAGED = STAGED && !VEC;
    extern __shared__ __align__(16) float table[];  // [r + 1][kTableRow]: the last turns nothing; weights [2][D]; sums [2][kWarps][D]; rows
    __shared__ unsigned long long turns[128];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, vector = lane & (V - 1), share = lane / V;
    const int all = p.heads[0] + p.heads[1];
    const long long tiles = (p.L + kTile - 1) / kTile, units = p.batch * tiles * all;
    float* weights = table + (p.r + 1) * kTableRow;
    float* sums = weights + 2 * p.D;
    // rows of this warp's head: those of x, then upstream gradients or results (gradients go where x was)
    const int slot = warp / kSets, slot_warp = warp % kSets;
    bf16* stage = reinterpret_cast<bf16*>(sums + stage_at<BWD>(p.D)) + slot * (BWD || !VEC ? 2 : 1) * p.D * kStageRow;
    bf16* second = stage + p.D * kStageRow;
    auto together = [&] { asm volatile("bar.sync %0, %1;\n" ::"r"(slot + 1), "n"(32 * kSets) : "memory"); };
    // a lane's channels: pairs (q, q + r) that turn, then pairs of neighbours that do not; -1: none
    auto channel = [&](int i) {
        const int q = share + kShares * (i >> 1), c = q < p.r ? q + (i & 1) * p.r : 2 * q + (i & 1);
        return c < p.D && 2 * q < p.D ? c : -1;
    };
    float dw[BWD ? 2 * KP : 1];
    int held = -1;  // whose weights' gradients dw holds
    auto flush = [&](int to) {
        if (held >= 0) {
#pragma unroll
            for (int i = 0; i < (BWD ? 2 * KP : 0); ++i) {
                float s = dw[i];
#pragma unroll
                for (int m = 1; m < V; m <<= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
                const int c = channel(i);
                if (vector == 0 && c >= 0) sums[(held * kWarps + warp) * p.D + c] += s;
            }
        }
#pragma unroll
        for (int i = 0; i < (BWD ? 2 * KP : 1); ++i) dw[i] = 0.f;
        held = to;
    };
    if (BWD)
        for (int i = threadIdx.x; i < 2 * kWarps * p.D; i += 256) sums[i] = 0.f;
    for (int i = threadIdx.x; i < 2 * p.D; i += 256) {
        const float* w = p.w[i / p.D];
        weights[i] = w != nullptr ? w[i % p.D] : 0.f;
    }
    for (int i = threadIdx.x; i < kTableRow; i += 256) table[p.r * kTableRow + i] = (i & 4) ? 0.f : 1.f;
    // (no loop over at most 128 of them: unrolled, it took registers from the gradients, 75 us for 72)
    if (threadIdx.x < p.r) turns[threadIdx.x] = turn_of(p.freq[threadIdx.x]);
    const long long last = min(units, ((long long)blockIdx.x + 1) * p.per);
    for (long long unit = blockIdx.x * p.per; unit < last;) {
        const int h0 = (int)(unit % all), h1 = (int)min((long long)all, h0 + (last - unit));
        const long long tile = unit / all % tiles, b = unit / all / tiles;
        const long long t0 = tile * kTile;
        unit += h1 - h0;
        __syncthreads();
        for (int i = threadIdx.x; i < p.r * kTile; i += 256) {
            const int f = i / kTile, t = i % kTile;
            float c = 1.f, s = 0.f;
            if (t0 + t < p.L) cos_sin(turns[f], p.pos[b * p.L + t0 + t], c, s);
            float* to = table + f * kTableRow + (t / 4) * 8 + t % 4;
            to[0] = c;
            to[4] = s;
        }
        __syncthreads();
        const int at = (warp % kSets) * kSpan + vector * E;  // the lane's first token in the tile
        const long long left = p.L - t0 - at;
        const int have = left <= 0 ? 0 : left < E ? (int)left : E;
        // a head's rows of this tile on their way
        const int n = (int)min((long long)kTile, p.L - t0);
        auto fetch = [&](const void* from, long long first, long long stride, const T* end, bf16* to) {
            const bf16* lo = static_cast<const bf16*>(from);
            const int j = lane & 7;
            for (int c8 = slot_warp * 4 + (lane >> 3); c8 < 8; c8 += 4 * kSets) {
                const bf16* row = lo + first + c8 * stride;
                const int phase = (int)sscan::phase8(row);
                if (j >= kStageRow / 8 || 8 * j >= phase + n || c8 >= p.D) continue;
                const bf16* at = row - phase + 8 * j;
                bf16* s = to + c8 * kStageRow + 8 * j;
                const int times = (p.D - c8 + 7) / 8;
                if (at >= lo && at + (times - 1) * 8 * stride + 8 <= reinterpret_cast<const bf16*>(end)) {
#pragma unroll 4
                    for (int m = 0; m < times; ++m, at += 8 * stride, s += 8 * kStageRow) sscan::cp_async16(s, at, 16);
                } else {  // a vector reaches out of the tensor
                    for (int m = 0; m < times; ++m, at += 8 * stride, s += 8 * kStageRow)
                        for (int e = 0; e < 8; ++e)
                            if (at + e >= lo && at + e < reinterpret_cast<const bf16*>(end)) s[e] = at[e];
                }
            }
            sscan::cp_async_commit();
        };
        auto fetch_x = [&](int h) {
            const int which = h >= p.heads[0], head = which ? h - p.heads[0] : h;
            const long long last_row = (p.batch - 1) * p.xb[which] + ((long long)p.heads[which] * p.D - 1) * p.xd[which];
            fetch(p.x[which], b * p.xb[which] + (long long)head * p.D * p.xd[which] + t0, p.xd[which],
                  static_cast<const T*>(p.x[which]) + last_row + p.L, stage);
        };
        auto fetch_dy = [&](int h) {
            const int which = h >= p.heads[0], head = which ? h - p.heads[0] : h;
            const long long rows = (long long)p.heads[which] * p.D;
            fetch(p.dy[which], (b * rows + (long long)head * p.D) * p.L + t0, p.L, static_cast<const T*>(p.dy[which]) + p.batch * rows * p.L, second);
        };
        if (STAGED && h0 + slot < h1) {
            fetch_x(h0 + slot);
            if (BWD) fetch_dy(h0 + slot);
        }
        for (int h = h0 + slot; h < h1; h += kHeads) {
            const int which = h >= p.heads[0], head = which ? h - p.heads[0] : h, heads = p.heads[which];
            if (BWD && which != held) flush(which);
            const long long row = (b * heads + head) * p.D, xd = p.xd[which];
            const T* x = static_cast<const T*>(p.x[which]) + b * p.xb[which] + (long long)head * p.D * xd + t0 + at;
            T* out = static_cast<T*>(p.y[which]) + row * p.L + t0 + at;
            const float* w = weights + which * p.D;
            uint4 xv[2 * KP], uv[BWD ? 2 * KP : 2];
            const T* dy0 = static_cast<const T*>(p.dy[which]);
            if constexpr (STAGED) {
                sscan::cp_async_wait<0>();
                together();
                auto take = [&](uint4& to, const bf16* row, const T* global, int c) {
                    const uint4* from = reinterpret_cast<const uint4*>(row + (c < 0 ? 0 : c) * kStageRow + at);
                    to = VEC ? from[0] : sscan::piece_shift(sscan::Piece8{from[0], from[1]}, sscan::phase8(reinterpret_cast<const bf16*>(global)));
                    if (c < 0 || have < E) to = sscan::keep_values(to, 0, c < 0 ? 0 : have);
                };
#pragma unroll
                for (int i = 0; i < 2 * KP; ++i) {
                    const int c = channel(i);
                    take(xv[i], stage, x + c * xd, c);
                    if constexpr (BWD) take(uv[i], second, dy0 + (row + c) * p.L + t0, c);
                }
                together();
                if (h + kHeads < h1) {
                    if (BWD) fetch_dy(h + kHeads);
                    if (!BWD || VEC) fetch_x(h + kHeads);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 2 * KP; ++i) {
                    const int c = channel(i);
                    xv[i] = load_tokens<VEC>(x + c * xd, c < 0 ? 0 : have);
                    if constexpr (BWD) uv[i] = load_tokens<VEC>(dy0 + (row + c) * p.L + t0 + at, c < 0 ? 0 : have);
                }
            }
            const Two minus = two(-1.f, -1.f);
            Two sq[E / 2], gn[E / 2];
#pragma unroll
            for (int e = 0; e < E / 2; ++e) sq[e] = gn[e] = two(0.f, 0.f);
            // cosines and sines of pair k
            auto turn = [&](int k, Two (&c)[E / 2], Two (&s)[E / 2]) {
                const int q = share + kShares * k;
                const float* from = table + (q < p.r ? q : p.r) * kTableRow + 2 * at;
#pragma unroll
                for (int e = 0; e < E / 2; e += 2) {
                    const float4 a = *reinterpret_cast<const float4*>(from + 4 * e), d = *reinterpret_cast<const float4*>(from + 4 * e + 4);
                    c[e] = two(a.x, a.y); c[e + 1] = two(a.z, a.w);
                    s[e] = two(d.x, d.y); s[e + 1] = two(d.z, d.w);
                }
            };
            auto weight = [&](int i) { const int c = channel(i); const float v = c < 0 ? 0.f : w[c]; return two(v, v); };
            // upstream gradients of pair k, turned back
            auto upstream = [&](int k, Two (&a)[E / 2], Two (&d)[E / 2]) {
                Two ya[E / 2], yd[E / 2], c[E / 2], s[E / 2];
                widen2(uv[BWD ? 2 * k : 0], ya, (T*)nullptr);
                widen2(uv[BWD ? 2 * k + 1 : 1], yd, (T*)nullptr);
                turn(k, c, s);
#pragma unroll
                for (int e = 0; e < E / 2; ++e) {
                    a[e] = fma2(ya[e], c[e], yd[e] * s[e]);
                    d[e] = fma2(ya[e] * s[e], minus, yd[e] * c[e]);
                }
            };
#pragma unroll
            for (int k = 0; k < KP; ++k) {
                Two a[E / 2], d[E / 2];
                widen2(xv[2 * k], a, (T*)nullptr);
                widen2(xv[2 * k + 1], d, (T*)nullptr);
#pragma unroll
                for (int e = 0; e < E / 2; ++e) sq[e] = fma2(a[e], a[e], fma2(d[e], d[e], sq[e]));
                if constexpr (BWD) {
                    Two ua[E / 2], ud[E / 2];
                    upstream(k, ua, ud);
                    const Two wa = weight(2 * k), wd = weight(2 * k + 1);
#pragma unroll
                    for (int e = 0; e < E / 2; ++e) gn[e] = fma2(ua[e] * wa, a[e], fma2(ud[e] * wd, d[e], gn[e]));
                }
            }
            // What the second pass takes is widened and turned again: kept from the first it
            // would fill the registers twice over.
#pragma unroll
            for (int i = 0; i < 2 * KP; ++i) {
                asm volatile("" : "+r"(xv[i].x), "+r"(xv[i].y), "+r"(xv[i].z), "+r"(xv[i].w) : : "memory");
                if constexpr (BWD) asm volatile("" : "+r"(uv[i].x), "+r"(uv[i].y), "+r"(uv[i].z), "+r"(uv[i].w) : : "memory");
            }
            float one[E];
#pragma unroll
            for (int e = 0; e < E; ++e) one[e] = e & 1 ? sq[e / 2].y() : sq[e / 2].x();
            // (a token behind the last has no norm: with eps = 0 an infinite one would enter the weights' sums as 0 * inf)
            const float square = channel_sum<V, E>(one);
            const float scale = !BWD || held_token<E>() < have ? 1.f / sqrtf(square / (float)p.D + p.eps) : 0.f;
            float mean = 0.f;
            if (BWD) {  // n * mean(g n) = x * rstd^2 * mean(g x)
#pragma unroll
                for (int e = 0; e < E; ++e) one[e] = e & 1 ? gn[e / 2].y() : gn[e / 2].x();
                mean = -scale * scale * (channel_sum<V, E>(one) / (float)p.D);
            }
            Two rstd[E / 2], m[E / 2];
#pragma unroll
            for (int e = 0; e < E / 2; ++e) {
                rstd[e] = two(of_token<V, E>(scale, 2 * e), of_token<V, E>(scale, 2 * e + 1));
                if (BWD) m[e] = two(of_token<V, E>(mean, 2 * e), of_token<V, E>(mean, 2 * e + 1));
            }
#pragma unroll
            for (int k = 0; k < KP; ++k) {
                Two a[E / 2], d[E / 2];
                widen2(xv[2 * k], a, (T*)nullptr);
                widen2(xv[2 * k + 1], d, (T*)nullptr);
                const Two wa = weight(2 * k), wd = weight(2 * k + 1);
                if constexpr (BWD) {
                    Two ua[E / 2], ud[E / 2], na = two(0.f, 0.f), nd = two(0.f, 0.f);
                    upstream(k, ua, ud);
#pragma unroll
                    for (int e = 0; e < E / 2; ++e) {
                        na = fma2(ua[e], a[e] * rstd[e], na);
                        nd = fma2(ud[e], d[e] * rstd[e], nd);
                        a[e] = rstd[e] * fma2(a[e], m[e], ua[e] * wa);
                        d[e] = rstd[e] * fma2(d[e], m[e], ud[e] * wd);
                    }
                    dw[BWD ? 2 * k : 0] += na.x() + na.y();
                    dw[BWD ? 2 * k + 1 : 0] += nd.x() + nd.y();
                } else {
                    Two c[E / 2], s[E / 2];
                    turn(k, c, s);
#pragma unroll
                    for (int e = 0; e < E / 2; ++e) {
                        const Two ya = a[e] * (rstd[e] * wa), yd = d[e] * (rstd[e] * wd);
                        a[e] = fma2(yd * s[e], minus, ya * c[e]);
                        d[e] = fma2(yd, c[e], ya * s[e]);
                    }
                }
                if constexpr (OUT_STAGED) {
                    const int ca = channel(2 * k), cd = channel(2 * k + 1);
                    bf16* going = BWD ? stage : second;
                    if (ca >= 0) *reinterpret_cast<uint4*>(going + ca * kStageRow + at) = narrow2<T, E>(a);
                    if (cd >= 0) *reinterpret_cast<uint4*>(going + cd * kStageRow + at) = narrow2<T, E>(d);
                } else {
                    const int ca = channel(2 * k), cd = channel(2 * k + 1);
                    store_tokens<T, VEC>(out + ca * p.L, ca < 0 ? 0 : have, narrow2<T, E>(a));
                    store_tokens<T, VEC>(out + cd * p.L, cd < 0 ? 0 : have, narrow2<T, E>(d));
                }
            }
            if constexpr (OUT_STAGED) {
                together();
                // a half warp a row, a word a lane; rows four apart lie in different banks
                const int j = lane & 15;
#pragma unroll
                for (int u = 0; u < 4 / kSets; ++u) {
                    const int c8 = 4 * (lane >> 4) + slot_warp * (4 / kSets) + u;
                    unsigned short* to = reinterpret_cast<unsigned short*>(static_cast<bf16*>(p.y[which]) + (row + c8) * p.L + t0);
                    const unsigned* words = reinterpret_cast<const unsigned*>((BWD ? stage : second) + c8 * kStageRow) + j;
                    const int odd = (int)(reinterpret_cast<uintptr_t>(to) >> 1) & 1, t = 2 * j + odd;
                    const bool first = odd && j == 0, both = t + 1 < n, one = t + 1 == n;
                    for (int c = c8; c < p.D; c += 8, to += 8 * p.L, words += 4 * kStageRow) {
                        const unsigned low = words[0], word = odd ? __funnelshift_r(low, words[1], 16) : low;
                        if (both) *reinterpret_cast<unsigned*>(to + t) = word;
                        if (one) to[t] = (unsigned short)word;
                        if (first) to[0] = (unsigned short)low;
                    }
                }
                if (BWD) {
                    together();
                    if (h + kHeads < h1) fetch_x(h + kHeads);
                }
            }
        }
    }
    if constexpr (BWD) {  // two rows of sums a CTA: over the vectors, then over the warps in order
        flush(-1);
        __syncthreads();
        for (int c = threadIdx.x; c < 2 * p.D; c += 256) {
            float s = 0.f;
            for (int i = 0; i < kWarps; ++i) s += sums[(c / p.D * kWarps + i) * p.D + c % p.D];
            p.parts[(long long)blockIdx.x * 2 * p.D + c] = s;
        }
    }
}

// weight gradients from two rows of sums a CTA, in their order
__global__ void __launch_bounds__(256) qknorm_add(const float* parts, float* a, float* b, int D, int rows) {
    __shared__ float part[8][32];
    sscan::griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float* to = blockIdx.y ? b : a;
    if (to == nullptr) return;
    float s = 0.f;
    if (c < D)
        for (int r = warp; r < rows; r += 8) s += parts[(2LL * r + blockIdx.y) * D + c];
    part[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < D) {
        for (int i = 1; i < 8; ++i) s += part[i][lane];
        to[c] = s;
    }
}

// Single tokens: [batch, heads * D], a warp a head.
template <typename T>
__global__ void __launch_bounds__(256) qknorm_step_kernel(const QkParams p) {
    extern __shared__ float table[];  // [8 warps][D]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int all = p.heads[0] + p.heads[1];
    float* mine = table + warp * p.D;
    const long long items = p.batch * all;
    for (long long item = (long long)blockIdx.x * 8 + warp; item < items; item += (long long)gridDim.x * 8) {
        const int h = (int)(item % all);
        const long long b = item / all;
        const int which = h >= p.heads[0], head = which ? h - p.heads[0] : h;
        const T* x = static_cast<const T*>(p.x[which]) + b * p.xb[which] + (long long)head * p.D;
        T* out = static_cast<T*>(p.y[which]) + (b * p.heads[which] + head) * p.D;
        float sq = 0.f;
        for (int i = lane; i < p.D; i += 32) {
            const float v = sscan::to_f32(x[i]);
            mine[i] = v;
            sq = fmaf(v, v, sq);
        }
        const float rstd = 1.f / sqrtf(sscan::warp_sum(sq) / (float)p.D + p.eps);
        __syncwarp();
        for (int i = lane; i < p.D; i += 32) {
            float y = mine[i] * rstd * __ldg(p.w[which] + i);
            if (i < 2 * p.r) {
                const int f = i < p.r ? i : i - p.r, o = i < p.r ? i + p.r : i - p.r;
                float c, s;
                cos_sin(turn_of(p.freq[f]), p.pos[b], c, s);
                const float other = mine[o] * rstd * __ldg(p.w[which] + o);
                y = i < p.r ? fmaf(y, c, -other * s) : fmaf(y, c, other * s);
            }
            out[i] = sscan::from_f32<T>(y);
        }
        __syncwarp();
    }
}

constexpr long long kBig = 1LL << 40;
constexpr long long kIntMax = 1LL << 30;
bool sizes_ok(long long batch, long long qh, long long kh, long long D, long long L, long long rot, int dtype) {
    if (dtype != SSCAN_F32 && dtype != SSCAN_BF16) return false;
    if (D < 1 || D > QKNORM_MAX_DIM || rot < 0 || 2 * rot > D || qh < 0 || kh < 0 || batch < 0 || L < 0) return false;
    if (qh + kh > (1 << 20) || batch > kIntMax || L > kIntMax) return false;
    const long long c = (qh + kh) * D;
    return !batch || !L || !c || (batch <= kBig / L && c <= kBig / (batch * L));
}
bool strides_ok(const int64_t* s, int n) {
    if (s == nullptr) return false;
    for (int i = 0; i < n; ++i)
        if (s[i] < 0 || s[i] > kBig) return false;
    return true;
}

// Shared memory of a call: the table, weights, sums and rows; a head of one channel more never takes less
template <typename T, int V, bool BWD, bool VEC>
constexpr size_t shared_bytes(int D, int r) {
    constexpr bool STAGED = sizeof(T) == 2;
    constexpr int slots = kWarps / (kTile / (V * sscan::VecOf<T>::E));
    return ((size_t)(r + 1) * kTableRow + 2 * D + stage_at<BWD>(D)) * sizeof(float) +
           (STAGED ? (size_t)slots * (BWD || !VEC ? 2 : 1) * D * kStageRow * sizeof(bf16) : 0);
}
template <typename T, int V, int KP, bool BWD, bool VEC>
cudaError_t run_rows(QkParams& p, long long ctas, cudaStream_t st) {
    const size_t smem = shared_bytes<T, V, BWD, VEC>(p.D, p.r);
    // The limit belongs to the kernel, not to a call: set to each call's own size, a narrow call on another host
    // thread could lower it between a wide call's set-up and its launch, which would then fail.
    constexpr int widest = 64 / V * KP;
    const cudaError_t e = cudaFuncSetAttribute(qknorm_kernel<T, V, KP, BWD, VEC>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)shared_bytes<T, V, BWD, VEC>(widest, widest / 2));
    if (e != cudaSuccess) return e;
    return sscan::launch(qknorm_kernel<T, V, KP, BWD, VEC>, dim3((unsigned)ctas), dim3(256), smem, st, false, p);
}
template <typename T, int V, int KP, bool BWD>
cudaError_t run_tiles(QkParams& p, long long ctas, cudaStream_t st) {
    constexpr int E = sscan::VecOf<T>::E;
    bool vec = p.L % E == 0;
    for (int i = 0; i < 2; ++i) {
        if (p.heads[i] == 0) continue;
        vec = vec && p.xb[i] % E == 0 && p.xd[i] % E == 0 && sscan::is_aligned(p.x[i], 16) && sscan::is_aligned(p.y[i], 16) &&
              (!BWD || sscan::is_aligned(p.dy[i], 16));
    }
    return vec ? run_rows<T, V, KP, BWD, true>(p, ctas, st) : run_rows<T, V, KP, BWD, false>(p, ctas, st);
}
template <typename T, bool BWD>
cudaError_t run_dim(QkParams& p, long long ctas, cudaStream_t st) {
    if (p.D <= 64) return run_tiles<T, 4, 4, BWD>(p, ctas, st);
    if (p.D <= 128) return run_tiles<T, 2, 4, BWD>(p, ctas, st);
    return run_tiles<T, 2, 8, BWD>(p, ctas, st);
}
void fill(QkParams& p, const void* q, const void* k, const float* qw, const float* kw, const int32_t* pos, const float* freq,
          void* qo, void* ko, int64_t batch, int64_t qh, int64_t kh, int64_t D, int64_t L, int64_t rot, float eps) {
    p.x[0] = q; p.x[1] = k; p.w[0] = qw; p.w[1] = kw; p.y[0] = qo; p.y[1] = ko;
    p.pos = pos; p.freq = freq;
    p.heads[0] = (int)qh; p.heads[1] = (int)kh;
    p.batch = batch; p.L = L; p.D = (int)D; p.r = (int)rot; p.eps = eps;
}
// CTAs for one wave, each with as many units: a multiple of 8, the most heads that a CTA takes at once.
long long plan(QkParams& p, int resident) {
    const long long units = p.batch * sscan::div_up(p.L, kTile) * (p.heads[0] + p.heads[1]);
    const long long each = sscan::div_up(units, (long long)resident * 152);
    p.per = (each + 7) / 8 * 8;
    return sscan::div_up(units, p.per);
}
}  // namespace

extern "C" int qknorm_fwd(const void* q, const void* k, const float* q_weight, const float* k_weight, const int32_t* positions,
                          const float* inv_freq, void* q_out, void* k_out, int64_t batch, int64_t q_heads, int64_t k_heads,
                          int64_t head_dim, int64_t seqlen, int64_t rotated, const int64_t* strides, float eps, int dtype,
                          void* stream) {
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    sscan::record_call(0, st, "rejected");
    if (!sizes_ok(batch, q_heads, k_heads, head_dim, seqlen, rotated, dtype) || !strides_ok(strides, 4)) return SSCAN_ERR_INVALID;
    if (batch == 0 || seqlen == 0 || q_heads + k_heads == 0) {
        sscan::record_call(0, st, "empty");
        return SSCAN_OK;
    }
    if ((q_heads && (!q || !q_weight || !q_out)) || (k_heads && (!k || !k_weight || !k_out)) || (rotated && (!positions || !inv_freq)))
        return SSCAN_ERR_INVALID;
    QkParams p = {};
    fill(p, q, k, q_weight, k_weight, positions, inv_freq, q_out, k_out, batch, q_heads, k_heads, head_dim, seqlen, rotated, eps);
    p.xb[0] = strides[0]; p.xd[0] = strides[1]; p.xb[1] = strides[2]; p.xd[1] = strides[3];
    const long long ctas = plan(p, head_dim <= 128 ? 2 : 1);
    sscan::record_call(1, st, "qknorm fwd");
    return sscan::finish(dtype == SSCAN_F32 ? run_dim<float, false>(p, ctas, st) : run_dim<bf16, false>(p, ctas, st));
}

extern "C" int qknorm_bwd(const void* q, const void* k, const float* q_weight, const float* k_weight, const int32_t* positions,
                          const float* inv_freq, const void* dq_out, const void* dk_out, void* dq, void* dk, float* dq_weight,
                          float* dk_weight, int64_t batch, int64_t q_heads, int64_t k_heads, int64_t head_dim, int64_t seqlen,
                          int64_t rotated, const int64_t* strides, float eps, int dtype, void* stream) {
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    sscan::record_call(0, st, "rejected");
    if (!sizes_ok(batch, q_heads, k_heads, head_dim, seqlen, rotated, dtype) || !strides_ok(strides, 4)) return SSCAN_ERR_INVALID;
    if ((q_heads && !dq_weight) || (k_heads && !dk_weight)) return SSCAN_ERR_INVALID;
    if (batch == 0 || seqlen == 0 || q_heads + k_heads == 0) {
        sscan::record_call(0, st, "empty: weight gradients = 0");
        cudaError_t e = cudaSuccess;
        if (dq_weight) e = cudaMemsetAsync(dq_weight, 0, (size_t)head_dim * sizeof(float), st);
        if (e == cudaSuccess && dk_weight) e = cudaMemsetAsync(dk_weight, 0, (size_t)head_dim * sizeof(float), st);
        return sscan::finish(e);
    }
    if ((q_heads && (!q || !q_weight || !dq_out || !dq)) || (k_heads && (!k || !k_weight || !dk_out || !dk)) ||
        (rotated && (!positions || !inv_freq)))
        return SSCAN_ERR_INVALID;
    QkParams p = {};
    fill(p, q, k, q_weight, k_weight, positions, inv_freq, dq, dk, batch, q_heads, k_heads, head_dim, seqlen, rotated, eps);
    p.xb[0] = strides[0]; p.xd[0] = strides[1]; p.xb[1] = strides[2]; p.xd[1] = strides[3];
    p.dy[0] = dq_out; p.dy[1] = dk_out;
    const long long ctas = plan(p, head_dim <= 128 ? 2 : 1);
    void* parts = nullptr;
    cudaError_t e = sscan::scratch_alloc(&parts, (size_t)ctas * 2 * head_dim * sizeof(float), st);
    if (e != cudaSuccess) return sscan::finish(e);
    p.parts = static_cast<float*>(parts);
    sscan::record_call(2, st, "qknorm bwd");
    e = dtype == SSCAN_F32 ? run_dim<float, true>(p, ctas, st) : run_dim<bf16, true>(p, ctas, st);
    if (e == cudaSuccess)
        e = sscan::launch(qknorm_add, dim3((unsigned)sscan::div_up(head_dim, 32), 2), dim3(256), 0, st, true, p.parts, dq_weight, dk_weight,
                          p.D, (int)ctas);
    const cudaError_t ef = cudaFreeAsync(parts, st);
    return sscan::finish(e != cudaSuccess ? e : ef);
}

extern "C" int qknorm_step(const void* q, const void* k, const float* q_weight, const float* k_weight, const int32_t* positions,
                           const float* inv_freq, void* q_out, void* k_out, int64_t batch, int64_t q_heads, int64_t k_heads,
                           int64_t head_dim, int64_t rotated, int64_t q_stride, int64_t k_stride, float eps, int dtype,
                           void* stream) {
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    sscan::record_call(0, st, "rejected");
    if (!sizes_ok(batch, q_heads, k_heads, head_dim, 1, rotated, dtype) || q_stride < 0 || k_stride < 0) return SSCAN_ERR_INVALID;
    if (batch == 0 || q_heads + k_heads == 0) {
        sscan::record_call(0, st, "empty");
        return SSCAN_OK;
    }
    if ((q_heads && (!q || !q_weight || !q_out)) || (k_heads && (!k || !k_weight || !k_out)) || (rotated && (!positions || !inv_freq)))
        return SSCAN_ERR_INVALID;
    QkParams p = {};
    fill(p, q, k, q_weight, k_weight, positions, inv_freq, q_out, k_out, batch, q_heads, k_heads, head_dim, 1, rotated, eps);
    p.xb[0] = q_stride; p.xb[1] = k_stride;
    const long long ctas = sscan::div_up(batch * (q_heads + k_heads), 8);
    const size_t smem = (size_t)8 * head_dim * sizeof(float);
    sscan::record_call(1, st, "qknorm step");
    const dim3 grid((unsigned)(ctas < (1 << 20) ? ctas : (1 << 20)));
    return sscan::finish(dtype == SSCAN_F32 ? sscan::launch(qknorm_step_kernel<float>, grid, dim3(256), smem, st, false, p)
                                            : sscan::launch(qknorm_step_kernel<bf16>, grid, dim3(256), smem, st, false, p));
}
