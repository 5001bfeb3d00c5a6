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

}  // namespace

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
