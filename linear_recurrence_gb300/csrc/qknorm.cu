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
// A few operations a value: HBM bandwidth bounds it.  Layout [batch, heads * D, L]: 64
// tokens of a head are a tile, lane = two tokens, 8 warps share the channels; cosines and
// sines of the tile's tokens are formed once, for several heads.
#include <stdio.h>

#include "block_utils.cuh"

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
    float* parts;       // [ctas][2][D]
    const int* pos;     // [batch][L]
    const float* freq;  // [r]
    long long xb[2], xd[2];  // batch and channel strides of q and k
    int heads[2];
    long long batch, L;
    int D, r, per;      // heads a CTA takes on
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

// Channel of a warp's i-th pair: pairs (i, i + r) first, then single channels.
// Slots 0 .. D-1 in the order of the work: slot 2i -> i, 2i+1 -> i + r for i < r, slot j >= 2r -> j.
template <typename T, int CH, bool BWD>  // CH: slots a warp (even), kWarps * CH >= D
__global__ void __launch_bounds__(256) qknorm_kernel(const QkParams p) {
    extern __shared__ float table[];  // cos and sin [r][2][kTile]
    __shared__ unsigned long long turns[128];
    __shared__ float sums[2][kWarps][kTile];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int tiles = (int)((p.L + kTile - 1) / kTile);
    const int all = p.heads[0] + p.heads[1], strips = (all + p.per - 1) / p.per;
    float dw[BWD ? 2 : 1][BWD ? CH : 1];
    if (BWD) {
#pragma unroll
        for (int i = 0; i < (BWD ? CH : 1); ++i) dw[0][i] = dw[BWD][i] = 0.f;
    }
    for (int i = threadIdx.x; i < p.r; i += 256) turns[i] = turn_of(p.freq[i]);
    __syncthreads();
    for (long long item = blockIdx.x; item < p.batch * tiles * strips; item += gridDim.x) {
        const int strip = (int)(item % strips);
        const long long tile = item / strips % tiles, b = item / strips / tiles;
        const long long t0 = tile * kTile;
        __syncthreads();
        for (int i = threadIdx.x; i < p.r * kTile; i += 256) {
            const int f = i / kTile, t = i % kTile;
            float c = 1.f, s = 0.f;
            if (t0 + t < p.L) cos_sin(turns[f], p.pos[b * p.L + t0 + t], c, s);
            table[2 * f * kTile + t] = c;
            table[(2 * f + 1) * kTile + t] = s;
        }
        __syncthreads();
        const int h1 = min(all, (strip + 1) * p.per);
        for (int h = strip * p.per; h < h1; ++h) {
            const int which = h >= p.heads[0], head = which ? h - p.heads[0] : h;
            const T* x = static_cast<const T*>(p.x[which]) + b * p.xb[which] + (long long)head * p.D * p.xd[which] + t0;
            const long long row = (b * p.heads[which] + head) * p.D;
            const T* dy = BWD ? static_cast<const T*>(p.dy[which]) + row * p.L + t0 : nullptr;
            T* out = static_cast<T*>(p.y[which]) + row * p.L + t0;
            float v[CH][2], u[BWD ? CH : 1][2], sq[2] = {0.f, 0.f}, gn[2] = {0.f, 0.f};
            auto channel = [&](int i) {
                const int slot = warp * CH + i;
                return slot < 2 * p.r ? (slot & 1 ? p.r : 0) + (slot >> 1) : slot;
            };
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const bool in = warp * CH + i < p.D;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int t = lane + 32 * e;
                    const bool ok = in && t0 + t < p.L;
                    v[i][e] = ok ? sscan::to_f32(x[channel(i) * p.xd[which] + t]) : 0.f;
                    if (BWD) u[BWD ? i : 0][e] = ok ? sscan::to_f32(dy[channel(i) * p.L + t]) : 0.f;
                }
            }
            if (BWD) {  // turn the upstream gradient back
#pragma unroll
                for (int i = 0; i < (BWD ? CH : 0); i += 2) {
                    const int slot = warp * CH + i;
                    if (slot >= 2 * p.r) continue;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float c = table[slot * kTile + lane + 32 * e], s = table[(slot + 1) * kTile + lane + 32 * e];
                        const float a = u[i][e], d = u[i + 1][e];
                        u[i][e] = fmaf(a, c, d * s);
                        u[i + 1][e] = fmaf(d, c, -a * s);
                    }
                }
            }
            float w[CH];
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                w[i] = warp * CH + i < p.D ? __ldg(p.w[which] + channel(i)) : 0.f;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    sq[e] = fmaf(v[i][e], v[i][e], sq[e]);
                    if (BWD) gn[e] = fmaf(u[BWD ? i : 0][e] * w[i], v[i][e], gn[e]);
                }
            }
            __syncthreads();  // the head before still reads the sums
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                sums[0][warp][lane + 32 * e] = sq[e];
                if (BWD) sums[1][warp][lane + 32 * e] = gn[e];
            }
            __syncthreads();
            float rstd[2], m[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float a = 0.f, g = 0.f;
#pragma unroll
                for (int i = 0; i < kWarps; ++i) {
                    a += sums[0][i][lane + 32 * e];
                    if (BWD) g += sums[1][i][lane + 32 * e];
                }
                rstd[e] = 1.f / sqrtf(a / (float)p.D + p.eps);
                m[e] = rstd[e] * rstd[e] * (g / (float)p.D);  // n * mean(g n) = x * rstd^2 * mean(g x)
            }
#pragma unroll
            for (int i = 0; i < CH; i += 2) {
                const int slot = warp * CH + i;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float a, d;
                    if (BWD) {
                        const int j = BWD ? i : 0, l = BWD ? i + 1 : 0;
                        dw[BWD ? which : 0][j] = fmaf(u[j][e], v[i][e] * rstd[e], dw[BWD ? which : 0][j]);
                        dw[BWD ? which : 0][l] = fmaf(u[l][e], v[i + 1][e] * rstd[e], dw[BWD ? which : 0][l]);
                        a = rstd[e] * (u[j][e] * w[i] - v[i][e] * m[e]);
                        d = rstd[e] * (u[l][e] * w[i + 1] - v[i + 1][e] * m[e]);
                    } else {
                        a = v[i][e] * rstd[e] * w[i];
                        d = v[i + 1][e] * rstd[e] * w[i + 1];
                        if (slot < 2 * p.r) {
                            const float c = table[slot * kTile + lane + 32 * e], s = table[(slot + 1) * kTile + lane + 32 * e];
                            const float y = a;
                            a = fmaf(y, c, -d * s);
                            d = fmaf(d, c, y * s);
                        }
                    }
                    if (t0 + lane + 32 * e < p.L) {
                        if (slot < p.D) out[channel(i) * p.L + lane + 32 * e] = sscan::from_f32<T>(a);
                        if (slot + 1 < p.D) out[channel(i + 1) * p.L + lane + 32 * e] = sscan::from_f32<T>(d);
                    }
                }
            }
        }
    }
    if (BWD) {
#pragma unroll
        for (int which = 0; which < 2; ++which)
#pragma unroll
            for (int i = 0; i < (BWD ? CH : 0); ++i) {
                const float s = sscan::warp_sum(dw[BWD ? which : 0][i]);
                const int slot = warp * CH + i;
                if (lane == 0 && slot < p.D)
                    p.parts[((long long)blockIdx.x * 2 + which) * p.D + (slot < 2 * p.r ? (slot & 1 ? p.r : 0) + (slot >> 1) : slot)] = s;
            }
    }
}

// weight gradients from one row of sums a CTA, in their order
__global__ void __launch_bounds__(256) qknorm_add(const float* parts, float* a, float* b, int D, int rows) {
    __shared__ float part[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < 2 * D)
        for (int r = warp; r < rows; r += 8) s += parts[(long long)r * 2 * D + c];
    part[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < 2 * D) {
        for (int i = 1; i < 8; ++i) s += part[i][lane];
        if (c < D && a != nullptr) a[c] = s;
        if (c >= D && b != nullptr) b[c - D] = s;
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

template <typename T, int CH, bool BWD>
cudaError_t run_tiles(QkParams& p, int ctas, cudaStream_t st) {
    const size_t smem = (size_t)p.r * 2 * kTile * sizeof(float);
    const cudaError_t e = cudaFuncSetAttribute(qknorm_kernel<T, CH, BWD>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return sscan::launch(qknorm_kernel<T, CH, BWD>, dim3((unsigned)ctas), dim3(256), smem, st, false, p);
}
template <typename T, bool BWD>
cudaError_t run_dim(QkParams& p, int ctas, cudaStream_t st) {
    if (p.D <= 64) return run_tiles<T, 8, BWD>(p, ctas, st);
    if (p.D <= 128) return run_tiles<T, 16, BWD>(p, ctas, st);
    return run_tiles<T, 32, BWD>(p, ctas, st);
}
void fill(QkParams& p, const void* q, const void* k, const float* qw, const float* kw, const int32_t* pos, const float* freq,
          void* qo, void* ko, int64_t batch, int64_t qh, int64_t kh, int64_t D, int64_t L, int64_t rot, float eps) {
    p.x[0] = q; p.x[1] = k; p.w[0] = qw; p.w[1] = kw; p.y[0] = qo; p.y[1] = ko;
    p.pos = pos; p.freq = freq;
    p.heads[0] = (int)qh; p.heads[1] = (int)kh;
    p.batch = batch; p.L = L; p.D = (int)D; p.r = (int)rot; p.eps = eps;
}
// Heads that share a tile's cosines and sines: as many as leave two CTAs an SM.
int plan(QkParams& p) {
    const long long all = p.heads[0] + p.heads[1], tiles = p.batch * sscan::div_up(p.L, kTile);
    long long per = all * tiles / (2 * 152);
    p.per = (int)(per < 1 ? 1 : per > 16 ? 16 : per);
    const long long items = tiles * sscan::div_up(all, p.per);
    return (int)(items < 4 * 152 ? items : 4 * 152);
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
    const int ctas = plan(p);
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
    const int ctas = plan(p);
    void* parts = nullptr;
    cudaError_t e = sscan::scratch_alloc(&parts, (size_t)ctas * 2 * head_dim * sizeof(float), st);
    if (e != cudaSuccess) return sscan::finish(e);
    p.parts = static_cast<float*>(parts);
    sscan::record_call(2, st, "qknorm bwd");
    e = dtype == SSCAN_F32 ? run_dim<float, true>(p, ctas, st) : run_dim<bf16, true>(p, ctas, st);
    if (e == cudaSuccess)
        e = sscan::launch(qknorm_add, dim3((unsigned)sscan::div_up(2 * head_dim, 32)), dim3(256), 0, st, false, p.parts, dq_weight, dk_weight,
                          p.D, ctas);
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
