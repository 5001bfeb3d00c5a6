// One token of every request through linear attention with a decay for each
// head, over a cache of states:
//
//   S <- e^(A dt) S + dt v k^T,   o = scale * S q + D v       S [P, N] a head
//
// A request with a negative cache row is padding: computed from a zero state,
// nothing kept.  The fp32 states are read and written once, 8 bytes for about 5
// operations, so HBM bandwidth bounds the step.  A warp owns rows (value
// channels) of one head and request: Q lanes share a row of N states, 16 bytes a
// lane, and its R rows are all on the way before the first is used.
#include "lattn.cuh"

namespace {

using sscan::bf16;
using sscan::Requests;

struct StepParams {
    const void *q, *k, *v, *delta;
    const float *A, *D, *bias;
    float* state;
    void* o;
    long long qs, ks, vs, ts;  // row strides
    long long batch;
    int heads, groups, N, P, softplus;
    float scale;
    Requests req;
};

// VEC: N is a multiple of 4 and the cache's rows are 16-byte aligned.
//
// Four CTAs an SM: more bytes on the way cost more in DRAM turns between reads and writes than
// they hide (256 x 80 heads of 64 x 128, 8 rows a warp: 3 CTAs 246 us, 4 220, 5 254, 6 299; 16
// rows 265, 4 rows at 6 CTAs 257; the floor is 201).
template <typename T, int Q, int R, bool VEC>
__global__ void __launch_bounds__(256, 4) lattn_step_kernel(const StepParams p) {
    constexpr int ROWS = 32 / Q * R;  // value channels of a warp
    const int lane = threadIdx.x & 31, sub = lane / Q, n0 = lane % Q * 4;
    const int strips = (p.P + ROWS - 1) / ROWS;
    const long long item = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (blockIdx.x == 0 && blockIdx.y == 0) p.req.check(threadIdx.x, 256);
    if (item >= (long long)p.heads * strips) return;
    const int head = (int)(item / strips), d0 = (int)(item % strips) * ROWS + sub;
    const int group = head / (p.heads / p.groups);
    const float a = __ldg(p.A + head) * sscan::kLog2e, skip = p.D != nullptr ? __ldg(p.D + head) : 0.f;
    for (long long b = blockIdx.y; b < p.batch; b += gridDim.y) {
        const int slot = p.req.slot((int)b);
        float* row = p.state + (((long long)(slot < 0 ? 0 : slot) * p.heads + head) * p.P) * p.N + n0;
        float s[R][4];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int d = d0 + r * (32 / Q);
#pragma unroll
            for (int i = 0; i < 4; ++i) s[r][i] = 0.f;
            if (slot < 0 || d >= p.P || n0 >= p.N) continue;
            if (VEC) {
                const float4 x = __ldcs(reinterpret_cast<const float4*>(row + (long long)d * p.N));
                s[r][0] = x.x; s[r][1] = x.y; s[r][2] = x.z; s[r][3] = x.w;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) if (n0 + i < p.N) s[r][i] = row[(long long)d * p.N + i];
            }
        }
        float k[4], q[4], dt = 1.f;
        const T* qp = static_cast<const T*>(p.q) + b * p.qs + (long long)group * p.N + n0;
        const T* kp = static_cast<const T*>(p.k) + b * p.ks + (long long)group * p.N + n0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            q[i] = n0 + i < p.N ? sscan::to_f32(qp[i]) : 0.f;
            k[i] = n0 + i < p.N ? sscan::to_f32(kp[i]) : 0.f;
        }
        if (p.delta != nullptr) {
            dt = sscan::to_f32(static_cast<const T*>(p.delta)[b * p.ts + head]);
            if (p.bias != nullptr) dt += __ldg(p.bias + head);
            if (p.softplus) dt = sscan::softplus_f32(dt);
        }
        const float decay = sscan::ex2(a * dt);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int d = d0 + r * (32 / Q);
            const float v = d < p.P ? sscan::to_f32(static_cast<const T*>(p.v)[b * p.vs + (long long)head * p.P + d]) : 0.f;
            float y = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[r][i] = fmaf(decay, s[r][i], dt * v * k[i]);
                y = fmaf(s[r][i], q[i], y);
            }
            if (slot >= 0 && d < p.P && n0 < p.N) {
                if (VEC) {
                    __stcs(reinterpret_cast<float4*>(row + (long long)d * p.N), make_float4(s[r][0], s[r][1], s[r][2], s[r][3]));
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) if (n0 + i < p.N) row[(long long)d * p.N + i] = s[r][i];
                }
            }
            y = sscan::warp_sum<Q>(y);
            if (lane % Q == 0 && d < p.P)
                static_cast<T*>(p.o)[(b * p.heads + head) * p.P + d] = sscan::from_f32<T>(fmaf(skip, v, p.scale * y));
        }
    }
}

template <typename T, int Q, int R>
cudaError_t run_lanes(const StepParams& p, bool vec, cudaStream_t st) {
    const long long items = (long long)p.heads * sscan::div_up(p.P, 32 / Q * R);
    const dim3 grid((unsigned)sscan::div_up(items, 8), (unsigned)(p.batch < 65535 ? p.batch : 65535));
    if (vec) return sscan::launch(lattn_step_kernel<T, Q, R, true>, grid, dim3(256), 0, st, false, p);
    return sscan::launch(lattn_step_kernel<T, Q, R, false>, grid, dim3(256), 0, st, false, p);
}
template <typename T>
cudaError_t run_step(const StepParams& p, bool vec, cudaStream_t st) {
    if (p.N <= 16) return run_lanes<T, 4, 2>(p, vec, st);
    if (p.N <= 32) return run_lanes<T, 8, 4>(p, vec, st);
    if (p.N <= 64) return run_lanes<T, 16, 8>(p, vec, st);
    return run_lanes<T, 32, 8>(p, vec, st);
}

// Sums of R values over Q lanes, of which lane's share is that of value lane % Q / (Q / R): each
// exchange halves the values that a lane still carries, 9 shuffles for 8 values over 32 lanes and not 40.
template <int Q, int R>
__device__ __forceinline__ float sum_rows(float (&y)[R], int lane) {
#pragma unroll
    for (int h = R / 2, m = Q / 2; h > 0; h /= 2, m /= 2) {
        const bool upper = (lane & m) != 0;
#pragma unroll
        for (int i = 0; i < h; ++i) {
            const float give = upper ? y[i] : y[i + h];
            y[i] = (upper ? y[i + h] : y[i]) + __shfl_xor_sync(0xffffffffu, give, m);
        }
    }
#pragma unroll
    for (int m = Q / R / 2; m > 0; m /= 2) y[0] += __shfl_xor_sync(0xffffffffu, y[0], m);
    return y[0];
}

// A request of at most kLattnShort tokens of a packed axis, token by token: a CTA takes one
// head of one request, its q, k, v and steps in shared memory, and its warps hold the state's rows as
// above.  The chunks of the walks cost a request of any length some 6 us of an SM; here it costs its
// state's way through HBM and the scan's arithmetic (8192 tokens x 32 heads of 64 x 128 in 1024
// requests: 853 us, by chunks 1519; in 4096: 1820, 6146; the states alone take 321 and 1285 us.  With
// a sum over the lanes for each row and token it took 1245 and 2138).
template <typename T, int Q, int R, bool VEC>
__global__ void __launch_bounds__(256, 4) lattn_short_kernel(const __grid_constant__ sscan::LattnParams p) {
    constexpr int ROWS = 32 / Q * R, S = sscan::kLattnShort;
    extern __shared__ __align__(16) float smem[];
    const int ld = (p.N + 3) / 4 * 4 + 4;
    float* qs = smem;              // [S][ld]
    float* ks = qs + S * ld;       // [S][ld]
    float* vs = ks + S * ld;       // [P][S + 1]
    float* os = vs + p.P * (S + 1);  // [P][S + 1]
    __shared__ float dts[S];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / Q, n0 = lane % Q * 4;
    const int head = blockIdx.x, group = head / (p.heads / p.groups), strips = (p.P + ROWS - 1) / ROWS;
    const float a = __ldg(p.A + head) * sscan::kLog2e, skip = p.D != nullptr ? __ldg(p.D + head) : 0.f;
    const T* q = static_cast<const T*>(p.q) + (long long)group * p.N * p.qd;
    const T* k = static_cast<const T*>(p.k) + (long long)group * p.N * p.kd;
    const T* v = static_cast<const T*>(p.v) + (long long)head * p.P * p.vd;
    const int j0 = threadIdx.x & (S - 1), c0 = threadIdx.x / S;
    for (int s = blockIdx.y; s < p.req.requests; s += gridDim.y) {
        const int begin = p.req.offset(s), len = p.req.offset(s + 1) - begin;
        if (len > S) continue;
        const int slot = p.req.slot(s);
        if (len <= 0) {  // no tokens: a row that does not continue starts from zeros
            if (slot < 0 || p.req.continues(s)) continue;
            float* row = p.s_out + ((long long)slot * p.heads + head) * p.P * p.N;
            for (int i = threadIdx.x; i < p.P * p.N; i += 256) row[i] = 0.f;
            continue;
        }
        const bool has = slot >= 0 && p.req.continues(s);
        __syncthreads();  // the request before is written
        const bool in = j0 < len;
        for (int n = c0; n < ld; n += 256 / S) {
            qs[j0 * ld + n] = in && n < p.N ? sscan::to_f32(q[n * p.qd + begin + j0]) : 0.f;
            ks[j0 * ld + n] = in && n < p.N ? sscan::to_f32(k[n * p.kd + begin + j0]) : 0.f;
        }
        for (int d = c0; d < p.P; d += 256 / S) vs[d * (S + 1) + j0] = in ? sscan::to_f32(v[d * p.vd + begin + j0]) : 0.f;
        if (threadIdx.x < len) dts[threadIdx.x] = sscan::lattn_step_of<T>(p, head * p.td + begin + threadIdx.x, head);
        bool staged = false;
        for (int strip = warp; strip < (strips + 7) / 8 * 8; strip += 8) {
            const int d0 = strip * ROWS + sub;
            float* row = p.s_out + (((long long)(slot < 0 ? 0 : slot) * p.heads + head) * p.P) * p.N + n0;
            float st[R][4];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int d = d0 + r * (32 / Q);
#pragma unroll
                for (int i = 0; i < 4; ++i) st[r][i] = 0.f;
                if (!has || d >= p.P || n0 >= p.N) continue;
                if (VEC) {
                    const float4 x = __ldcs(reinterpret_cast<const float4*>(row + (long long)d * p.N));
                    st[r][0] = x.x; st[r][1] = x.y; st[r][2] = x.z; st[r][3] = x.w;
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) if (n0 + i < p.N) st[r][i] = row[(long long)d * p.N + i];
                }
            }
            if (!staged) __syncthreads();  // (each warp passes here once: strips are whole rounds of the 8 warps)
            staged = true;
            for (int t = 0; t < len; ++t) {
                float kv[4] = {0.f, 0.f, 0.f, 0.f}, qv[4] = {0.f, 0.f, 0.f, 0.f};
                if (n0 < p.N) {
                    sscan::load4_smem(ks + t * ld + n0, kv);
                    sscan::load4_smem(qs + t * ld + n0, qv);
                }
                const float dt = dts[t], decay = sscan::ex2(a * dt);
#pragma unroll
                for (int i = 0; i < 4; ++i) kv[i] *= dt;
                float y[R];
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const int d = d0 + r * (32 / Q);
                    const float x = d < p.P ? vs[d * (S + 1) + t] : 0.f;
                    y[r] = 0.f;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        st[r][i] = fmaf(decay, st[r][i], x * kv[i]);
                        y[r] = fmaf(st[r][i], qv[i], y[r]);
                    }
                }
                const float sum = sum_rows<Q, R>(y, lane);
                const int d = d0 + lane % Q / (Q / R) * (32 / Q);
                if (lane % (Q / R) == 0 && d < p.P) os[d * (S + 1) + t] = fmaf(skip, vs[d * (S + 1) + t], p.scale * sum);
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int d = d0 + r * (32 / Q);
                if (slot < 0 || d >= p.P || n0 >= p.N) continue;
                if (VEC) {
                    __stcs(reinterpret_cast<float4*>(row + (long long)d * p.N), make_float4(st[r][0], st[r][1], st[r][2], st[r][3]));
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) if (n0 + i < p.N) row[(long long)d * p.N + i] = st[r][i];
                }
            }
        }
        __syncthreads();
        T* out = static_cast<T*>(p.o) + (long long)head * p.P * p.L + begin;
        if (in)
            for (int d = c0; d < p.P; d += 256 / S) out[(long long)d * p.L + j0] = sscan::from_f32<T>(os[d * (S + 1) + j0]);
    }
}

// Shared memory of a call: queries, keys, values and outputs
constexpr size_t short_bytes(int N, int P) {
    return sizeof(float) * (2 * sscan::kLattnShort * ((N + 3) / 4 * 4 + 4) + 2 * P * (sscan::kLattnShort + 1));
}
template <typename T, int Q, int R, bool VEC>
cudaError_t run_short_as(const sscan::LattnParams& p, cudaStream_t st) {
    const size_t smem = short_bytes(p.N, p.P);
    // The limit belongs to the kernel, not to a call: set to each call's own size, a narrow call on another host
    // thread could lower it between a wide call's set-up and its launch, which would then fail.
    const cudaError_t e = cudaFuncSetAttribute(lattn_short_kernel<T, Q, R, VEC>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)short_bytes(4 * Q, LATTN_MAX_VALUE));
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)p.heads, (unsigned)(p.req.requests < 65535 ? p.req.requests : 65535));
    return sscan::launch(lattn_short_kernel<T, Q, R, VEC>, grid, dim3(256), smem, st, false, p);
}
template <typename T, int Q, int R>
cudaError_t run_short_rows(const sscan::LattnParams& p, cudaStream_t st) {
    return p.N % 4 == 0 && sscan::is_aligned(p.s_out, 16) ? run_short_as<T, Q, R, true>(p, st) : run_short_as<T, Q, R, false>(p, st);
}
template <typename T>
cudaError_t run_short(const sscan::LattnParams& p, cudaStream_t st) {
    if (p.N <= 16) return run_short_rows<T, 4, 2>(p, st);
    if (p.N <= 32) return run_short_rows<T, 8, 4>(p, st);
    if (p.N <= 64) return run_short_rows<T, 16, 8>(p, st);
    return run_short_rows<T, 32, 8>(p, st);
}

}  // namespace

cudaError_t sscan::lattn_short_launch(const LattnParams& p, int dtype, cudaStream_t st) {
    return dtype == SSCAN_F32 ? run_short<float>(p, st) : run_short<bf16>(p, st);
}

extern "C" int lattn_step(const void* q, const void* k, const void* v, const float* A, const void* delta, const float* D,
                          const float* delta_bias, const int32_t* slots, float* state, void* o, int64_t batch,
                          int64_t num_slots, int64_t heads, int64_t groups, int64_t key, int64_t value, int64_t q_stride,
                          int64_t k_stride, int64_t v_stride, int64_t delta_stride, float scale, int dtype, int flags,
                          void* stream) {
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    sscan::record_call(0, st, "rejected");
    if ((dtype != SSCAN_F32 && dtype != SSCAN_BF16) || (flags & ~SSCAN_DELTA_SOFTPLUS) != 0) return SSCAN_ERR_INVALID;
    const long long lim = 1LL << 28;  // 32-bit channel, request and row numbers on the device
    if (key < 1 || key > LATTN_MAX_KEY || value < 1 || value > LATTN_MAX_VALUE || groups < 1 || heads < 0 || heads > 65535 ||
        heads % groups != 0 || batch < 0 || batch > lim || num_slots < 0 || num_slots > lim || q_stride < 0 || k_stride < 0 ||
        v_stride < 0 || delta_stride < 0 || (slots == nullptr && batch > num_slots))
        return SSCAN_ERR_INVALID;
    if (batch == 0 || heads == 0) {
        sscan::record_call(0, st, "empty");
        return SSCAN_OK;
    }
    if (!q || !k || !v || !A || !o || (num_slots && !state)) return SSCAN_ERR_INVALID;
    int* status = sscan::device_status_word();
    if (status == nullptr) return sscan::finish(cudaErrorUnknown);
    StepParams p = {};
    p.q = q; p.k = k; p.v = v; p.delta = delta; p.A = A; p.D = D; p.bias = delta_bias; p.state = state; p.o = o;
    p.qs = q_stride; p.ks = k_stride; p.vs = v_stride; p.ts = delta_stride;
    p.batch = batch; p.heads = (int)heads; p.groups = (int)groups; p.N = (int)key; p.P = (int)value;
    p.softplus = flags & SSCAN_DELTA_SOFTPLUS; p.scale = scale;
    p.req = Requests{nullptr, slots, nullptr, (int)batch, (int)num_slots, 0, status};
    const bool vec = key % 4 == 0 && sscan::is_aligned(state, 16);
    sscan::record_call(1, st, vec ? "lattn step vec=1" : "lattn step vec=0");
    return sscan::finish(dtype == SSCAN_F32 ? run_step<float>(p, vec, st) : run_step<bf16>(p, vec, st));
}
