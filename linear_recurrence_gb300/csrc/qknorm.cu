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
// rounding).  In fp32 pos * freq would be off by 2^-24 of the whole angle: 0.03 rad at
// position 500,000.
//
// A few operations a value: HBM bandwidth bounds it.  Layout [batch, heads * D, L]: a warp
// takes V vectors of 16 bytes of tokens of one head at a time, all channels in registers: lane =
// vector x channels (32 / V lanes share them, each with pairs that turn together), so that the
// sums over channels stay in the warp and inputs are read once.  Cosines and sines of a
// tile of 64 tokens are formed once in shared memory, for several heads.  (With 8 warps sharing a head's
// channels and one value a load, 8209 tokens x 48 heads of 128 took 312 us.)
#include <stdio.h>

#include "block_utils.cuh"
#include "piece_loads.cuh"

namespace {

using sscan::bf16;

constexpr int kTile = 64;   // tokens of a tile
constexpr int kWarps = 8;

struct QkParams {
    const void* x[2];   // q, k
    const void* dy[2];
    void* y[2];         // outputs, or dq and dk
    const float* w[2];
    float* dw[2];
    float* parts;       // [ctas][D]
    const int* pos;     // [batch][L]
    const float* freq;  // [r]
    long long xb[2], xd[2];  // batch and channel strides of q and k
    int heads[2];
    long long batch, L;
    int D, r, per;      // per: heads that share a tile's cosines and sines
    int ctas[2];        // of queries, of keys
    float eps;
};

// The fraction of a turn that a frequency adds per position, in units of 2^-64.
__device__ __forceinline__ unsigned long long turn_of(float freq) {
    const double t = (double)freq * 0.15915494309189533577;  // 1 / (2 pi)
    const double f = t - floor(t);                            // [0, 1]
    return f >= 1.0 ? 0ull : __double2ull_rz(f * 18446744073709551616.0);
}
__device__ __forceinline__ void cos_sin(unsigned long long turn, int pos, float& c, float& s) {
    const long long a = (long long)(turn * (unsigned long long)(long long)pos);  // signed: [-1/2, 1/2) of a turn
    sincospif(__ll2float_rn(a) * 1.0842021724855044e-19f, &s, &c);             // 2^-63 half turns
}

// One vector of tokens of a channel; VEC: rows lie on 16-byte boundaries.
template <typename T, bool VEC>
__device__ __forceinline__ uint4 load_tokens(const T* p, int have, const T* lo, const T* hi) {
    constexpr int E = sscan::VecOf<T>::E;
    if (VEC && have == E) return __ldg(reinterpret_cast<const uint4*>(p));
    unsigned w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < E; ++i) {
        if (i >= have) continue;
        if (sizeof(T) == 4) w[i % 4] = __ldg(reinterpret_cast<const unsigned*>(p) + i);
        else w[i / 2 % 4] |= (unsigned)__ldg(reinterpret_cast<const unsigned short*>(p) + i) << (16 * (i & 1));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
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
    if (have == E) {  // words where they lie on 4 bytes
        if ((reinterpret_cast<uintptr_t>(p) & 2u) == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) reinterpret_cast<unsigned*>(to)[i] = w[i];
        } else {
            to[0] = (unsigned short)w[0];
#pragma unroll
            for (int i = 0; i < 3; ++i) reinterpret_cast<unsigned*>(to + 1)[i] = __funnelshift_r(w[i], w[i + 1], 16);
            to[7] = (unsigned short)(w[3] >> 16);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < E; ++i)
        if (i < have) to[i] = (unsigned short)(w[i / 2 % 4] >> (16 * (i & 1)));
}
// all of a thread's vectors of one array: rows that lie anywhere come by two vectors and a shift
template <typename T, int KP, bool VEC>
struct Rows {
    template <typename Row>
    static __device__ __forceinline__ void load(uint4 (&x)[2 * KP], const T* base, Row row, int have, const T* lo, const T* hi) {
        if constexpr (VEC || sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 2 * KP; ++i) {
                const long long at = row(i);
                x[i] = at >= 0 ? load_tokens<T, VEC>(base + at, have, lo, hi) : make_uint4(0u, 0u, 0u, 0u);
            }
        } else {
            constexpr int kAtOnce = 8;
#pragma unroll
            for (int i = 0; i < 2 * KP; i += kAtOnce) {
                sscan::Piece8 y[kAtOnce];
#pragma unroll
                for (int j = 0; j < kAtOnce; ++j) {
                    const long long at = row(i + j);
                    sscan::piece_load(y[j], base + (at < 0 ? 0 : at), at < 0 ? 0 : have, lo, hi);
                }
#pragma unroll
                for (int j = 0; j < kAtOnce; ++j) {
                    const long long at = row(i + j);
                    x[i + j] = sscan::piece_take(y[j], base + (at < 0 ? 0 : at), at < 0 ? 0 : have, lo, hi);
                }
            }
        }
    }
};

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
template <int V, int E>
__device__ __forceinline__ float of_token(float v, int e) {  // E = 8: token bits 0..2 are lane bits 2..4; E = 4: 3..4
    return __shfl_sync(0xffffffffu, v, (threadIdx.x & (V - 1)) + (E == 8 ? 4 * e : 8 * e));
}

constexpr int kTableRow = 2 * kTile + 4;  // a frequency's cosines, sines and a pad that keeps lanes in different banks

// V: vectors of a row in a warp; KP: pairs of channels a lane, 64 / V * KP >= D
template <typename T, int V, int KP, bool BWD, bool VEC>
__global__ void __launch_bounds__(256, KP <= 4 && !BWD ? 2 : 1) qknorm_kernel(const QkParams p) {
    constexpr int E = sscan::VecOf<T>::E, kSpan = V * E, kSets = kTile / kSpan, kHeads = kWarps / kSets, kShares = 32 / V;
    extern __shared__ float table[];  // [r][kTableRow]
    __shared__ unsigned long long turns[128];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, vector = lane & (V - 1), share = lane / V;
    const int which = (int)blockIdx.x >= p.ctas[0];
    const int block = which ? blockIdx.x - p.ctas[0] : blockIdx.x;
    const int heads = p.heads[which], tiles = (int)((p.L + kTile - 1) / kTile), strips = (heads + p.per - 1) / p.per;
    const T* x0 = static_cast<const T*>(p.x[which]);
    const T* x1 = x0 + (p.batch - 1) * p.xb[which] + ((long long)heads * p.D - 1) * p.xd[which] + p.L;
    const T* dy0 = BWD ? static_cast<const T*>(p.dy[which]) : nullptr;
    const T* dy1 = BWD ? dy0 + p.batch * heads * p.D * p.L : nullptr;
    const long long xd = p.xd[which];
    // a lane's channels: pairs (q, q + r) that turn, then pairs of neighbours that do not; -1: none
    auto channel = [&](int i) {
        const int q = share + kShares * (i >> 1), c = q < p.r ? q + (i & 1) * p.r : 2 * q + (i & 1);
        return c < p.D && 2 * q < p.D ? c : -1;
    };
    float dw[BWD ? 2 * KP : 1];
    if (BWD) {
#pragma unroll
        for (int i = 0; i < (BWD ? 2 * KP : 1); ++i) dw[i] = 0.f;
    }
    for (int i = threadIdx.x; i < p.r; i += 256) turns[i] = turn_of(p.freq[i]);
    __syncthreads();
    for (long long item = block; item < p.batch * tiles * strips; item += p.ctas[which]) {
        const int strip = (int)(item % strips);
        const long long tile = item / strips % tiles, b = item / strips / tiles;
        const long long t0 = tile * kTile;
        __syncthreads();
        for (int i = threadIdx.x; i < p.r * kTile; i += 256) {
            const int f = i / kTile, t = i % kTile;
            float c = 1.f, s = 0.f;
            if (t0 + t < p.L) cos_sin(turns[f], p.pos[b * p.L + t0 + t], c, s);
            table[f * kTableRow + t] = c;
            table[f * kTableRow + kTile + t] = s;
        }
        __syncthreads();
        const int at = (warp % kSets) * kSpan + vector * E;  // the lane's first token in the tile
        const long long left = p.L - t0 - at;
        const int have = left <= 0 ? 0 : left < E ? (int)left : E;
        const int h1 = min(heads, (strip + 1) * p.per);
        for (int head = strip * p.per + warp / kSets; head < h1; head += kHeads) {
            const long long row = (b * heads + head) * p.D;
            const T* x = x0 + b * p.xb[which] + (long long)head * p.D * xd + t0 + at;
            T* out = static_cast<T*>(p.y[which]) + row * p.L + t0 + at;
            uint4 xv[2 * KP], uv[BWD ? 2 * KP : 2];
            auto x_row = [&](int i) { const int c = channel(i); return c < 0 || have == 0 ? -1LL : c * xd; };
            auto y_row = [&](int i) { const int c = channel(i); return c < 0 || have == 0 ? -1LL : c * p.L; };
            Rows<T, KP, VEC>::load(xv, x, x_row, have, x0, x1);
            if constexpr (BWD) Rows<T, KP, VEC>::load(uv, dy0 + row * p.L + t0 + at, y_row, have, dy0, dy1);
            float sq[E], gn[E];
#pragma unroll
            for (int e = 0; e < E; ++e) sq[e] = gn[e] = 0.f;
            // cosines and sines of pair k (1 and 0 where it does not turn)
            auto turn = [&](int k, float (&c)[E], float (&s)[E]) {
                const int q = share + kShares * k;
                const bool turns_ = q < p.r;
                const float* from = table + (turns_ ? q : 0) * kTableRow + at;
#pragma unroll
                for (int e = 0; e < E; e += 4) {
                    const float4 a = *reinterpret_cast<const float4*>(from + e), d = *reinterpret_cast<const float4*>(from + kTile + e);
                    c[e] = turns_ ? a.x : 1.f; c[e + 1] = turns_ ? a.y : 1.f; c[e + 2] = turns_ ? a.z : 1.f; c[e + 3] = turns_ ? a.w : 1.f;
                    s[e] = turns_ ? d.x : 0.f; s[e + 1] = turns_ ? d.y : 0.f; s[e + 2] = turns_ ? d.z : 0.f; s[e + 3] = turns_ ? d.w : 0.f;
                }
            };
            auto weight = [&](int i) { const int c = channel(i); return c < 0 ? 0.f : __ldg(p.w[which] + c); };
            // upstream gradients of pair k, turned back
            auto upstream = [&](int k, float (&a)[E], float (&d)[E]) {
                float ya[E], yd[E], c[E], s[E];
                sscan::widen(uv[BWD ? 2 * k : 0], ya, (T*)nullptr);
                sscan::widen(uv[BWD ? 2 * k + 1 : 1], yd, (T*)nullptr);
                if (p.r > 0) turn(k, c, s);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    a[e] = p.r > 0 ? fmaf(ya[e], c[e], yd[e] * s[e]) : ya[e];
                    d[e] = p.r > 0 ? fmaf(yd[e], c[e], -ya[e] * s[e]) : yd[e];
                }
            };
#pragma unroll
            for (int k = 0; k < KP; ++k) {
                float a[E], d[E];
                sscan::widen(xv[2 * k], a, (T*)nullptr);
                sscan::widen(xv[2 * k + 1], d, (T*)nullptr);
#pragma unroll
                for (int e = 0; e < E; ++e) sq[e] = fmaf(a[e], a[e], fmaf(d[e], d[e], sq[e]));
                if constexpr (BWD) {
                    float ua[E], ud[E];
                    upstream(k, ua, ud);
                    const float wa = weight(2 * k), wd = weight(2 * k + 1);
#pragma unroll
                    for (int e = 0; e < E; ++e) gn[e] = fmaf(ua[e] * wa, a[e], fmaf(ud[e] * wd, d[e], gn[e]));
                }
            }
            // What the second pass takes is widened and turned again: kept from the first it
            // would fill the registers twice over.
#pragma unroll
            for (int i = 0; i < 2 * KP; ++i) {
                asm volatile("" : "+r"(xv[i].x), "+r"(xv[i].y), "+r"(xv[i].z), "+r"(xv[i].w) : : "memory");
                if constexpr (BWD) asm volatile("" : "+r"(uv[i].x), "+r"(uv[i].y), "+r"(uv[i].z), "+r"(uv[i].w) : : "memory");
            }
            const float mine = channel_sum<V, E>(sq);
            const float scale = 1.f / sqrtf(mine / (float)p.D + p.eps);
            float mean = 0.f;
            if (BWD) mean = scale * scale * (channel_sum<V, E>(gn) / (float)p.D);  // n * mean(g n) = x * rstd^2 * mean(g x)
            float rstd[E], m[E];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                rstd[e] = of_token<V, E>(scale, e);
                m[e] = BWD ? of_token<V, E>(mean, e) : 0.f;
            }
#pragma unroll
            for (int k = 0; k < KP; ++k) {
                float a[E], d[E];
                sscan::widen(xv[2 * k], a, (T*)nullptr);
                sscan::widen(xv[2 * k + 1], d, (T*)nullptr);
                const float wa = weight(2 * k), wd = weight(2 * k + 1);
                if constexpr (BWD) {
                    float ua[E], ud[E];
                    upstream(k, ua, ud);
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        dw[BWD ? 2 * k : 0] = fmaf(ua[e], a[e] * rstd[e], dw[BWD ? 2 * k : 0]);
                        dw[BWD ? 2 * k + 1 : 0] = fmaf(ud[e], d[e] * rstd[e], dw[BWD ? 2 * k + 1 : 0]);
                        a[e] = rstd[e] * fmaf(ua[e], wa, -a[e] * m[e]);
                        d[e] = rstd[e] * fmaf(ud[e], wd, -d[e] * m[e]);
                    }
                } else {
                    float c[E], s[E];
                    if (p.r > 0) turn(k, c, s);
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const float ya = a[e] * (rstd[e] * wa), yd = d[e] * (rstd[e] * wd);
                        a[e] = p.r > 0 ? fmaf(ya, c[e], -yd * s[e]) : ya;
                        d[e] = p.r > 0 ? fmaf(yd, c[e], ya * s[e]) : yd;
                    }
                }
                const long long ra = y_row(2 * k), rd = y_row(2 * k + 1);
                if (ra >= 0) store_tokens<T, VEC>(out + ra, have, sscan::narrow(a, (T*)nullptr));
                if (rd >= 0) store_tokens<T, VEC>(out + rd, have, sscan::narrow(d, (T*)nullptr));
            }
        }
    }
    if constexpr (BWD) {  // one row of sums a CTA: over the vectors, then over the warps in order
        __shared__ float sums[kWarps][2 * kShares * KP];
#pragma unroll
        for (int i = 0; i < 2 * KP; ++i) {
            float s = dw[i];
#pragma unroll
            for (int m = 1; m < V; m <<= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
            const int c = channel(i);
            if (vector == 0 && c >= 0) sums[warp][c] = s;
        }
        __syncthreads();
        for (int c = threadIdx.x; c < p.D; c += 256) {
            float s = 0.f;
            for (int i = 0; i < kWarps; ++i) s += sums[i][c];
            p.parts[(long long)blockIdx.x * p.D + c] = s;
        }
    }
}

// weight gradients from one row of sums a CTA, in their order: those of q first
__global__ void __launch_bounds__(256) qknorm_add(const float* parts, float* a, float* b, int D, int rows_a, int rows_b) {
    __shared__ float part[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    const int first = blockIdx.y ? rows_a : 0, rows = blockIdx.y ? rows_b : rows_a;
    float* to = blockIdx.y ? b : a;
    if (to == nullptr) return;
    float s = 0.f;
    if (c < D)
        for (int r = warp; r < rows; r += 8) s += parts[(long long)(first + r) * D + c];
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

template <typename T, int V, int KP, bool BWD, bool VEC>
cudaError_t run_rows(QkParams& p, cudaStream_t st) {
    const size_t smem = (size_t)(p.r > 0 ? p.r : 1) * kTableRow * sizeof(float);
    const cudaError_t e = cudaFuncSetAttribute(qknorm_kernel<T, V, KP, BWD, VEC>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return sscan::launch(qknorm_kernel<T, V, KP, BWD, VEC>, dim3((unsigned)(p.ctas[0] + p.ctas[1])), dim3(256), smem, st, false, p);
}
template <typename T, int V, int KP, bool BWD>
cudaError_t run_tiles(QkParams& p, cudaStream_t st) {
    constexpr int E = sscan::VecOf<T>::E;
    bool vec = p.L % E == 0;
    for (int i = 0; i < 2; ++i) {
        if (p.heads[i] == 0) continue;
        vec = vec && p.xb[i] % E == 0 && p.xd[i] % E == 0 && sscan::is_aligned(p.x[i], 16) && sscan::is_aligned(p.y[i], 16) &&
              (!BWD || sscan::is_aligned(p.dy[i], 16));
    }
    return vec ? run_rows<T, V, KP, BWD, true>(p, st) : run_rows<T, V, KP, BWD, false>(p, st);
}
template <typename T, bool BWD>
cudaError_t run_dim(QkParams& p, cudaStream_t st) {
    if (p.D <= 64) return run_tiles<T, 4, 4, BWD>(p, st);
    if (p.D <= 128) return run_tiles<T, 2, 4, BWD>(p, st);
    return run_tiles<T, 2, 8, BWD>(p, st);
}
void fill(QkParams& p, const void* q, const void* k, const float* qw, const float* kw, const int32_t* pos, const float* freq,
          void* qo, void* ko, int64_t batch, int64_t qh, int64_t kh, int64_t D, int64_t L, int64_t rot, float eps) {
    p.x[0] = q; p.x[1] = k; p.w[0] = qw; p.w[1] = kw; p.y[0] = qo; p.y[1] = ko;
    p.pos = pos; p.freq = freq;
    p.heads[0] = (int)qh; p.heads[1] = (int)kh;
    p.batch = batch; p.L = L; p.D = (int)D; p.r = (int)rot; p.eps = eps;
}
// Heads that share a tile's cosines and sines: up to 16, fewer while there are not four
// items an SM; then CTAs for queries and for keys by their numbers of heads.
int plan(QkParams& p, int resident) {
    const long long all = p.heads[0] + p.heads[1], tiles = p.batch * sscan::div_up(p.L, kTile);
    long long per = all * tiles / (4 * 152);
    p.per = (int)(per < 4 ? 4 : per > 16 ? 16 : per);
    const long long items[2] = {tiles * sscan::div_up(p.heads[0], p.per), tiles * sscan::div_up(p.heads[1], p.per)};
    const long long most = (long long)resident * 152;  // one wave
    for (int i = 0; i < 2; ++i) {
        long long n = items[0] + items[1] <= most ? items[i] : most * p.heads[i] / all;
        if (n < 1 && items[i] > 0) n = 1;
        p.ctas[i] = (int)n;
    }
    return p.ctas[0] + p.ctas[1];
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
    plan(p, head_dim <= 128 ? 2 : 1);
    sscan::record_call(1, st, "qknorm fwd");
    return sscan::finish(dtype == SSCAN_F32 ? run_dim<float, false>(p, st) : run_dim<bf16, false>(p, st));
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
    const int ctas = plan(p, 1);
    void* parts = nullptr;
    cudaError_t e = sscan::scratch_alloc(&parts, (size_t)ctas * head_dim * sizeof(float), st);
    if (e != cudaSuccess) return sscan::finish(e);
    p.parts = static_cast<float*>(parts);
    sscan::record_call(2, st, "qknorm bwd");
    e = dtype == SSCAN_F32 ? run_dim<float, true>(p, st) : run_dim<bf16, true>(p, st);
    if (e == cudaSuccess)
        e = sscan::launch(qknorm_add, dim3((unsigned)sscan::div_up(head_dim, 32), 2), dim3(256), 0, st, false, p.parts, dq_weight, dk_weight,
                          p.D, p.ctas[0], p.ctas[1]);
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
