// Single-token selective-scan update over a state cache, on sm_103a: one
// decode step for a batch of requests whose states lie in rows of a larger
// cache, with the options of the scan inside.
//
//   dt = delta, or softplus(delta + bias)
//   h[n] <- exp(dt*A[d,n]) * h[n] + dt*u*B[n],   y = (sum_n C[n]*h[n] + D[d]*u) * silu(z)
//
// A request with a negative cache row is padding: it is computed from a zero
// state and keeps none.  The fp32 state is read and written once, 8 bytes per
// (request, channel, state) against about 7 operations, so HBM bandwidth bounds
// the step: a thread owns up to two groups of 4 consecutive states (16-byte
// loads and stores, both in flight together) and the threads of a channel sum their parts by
// shuffles.
#include "block_utils.cuh"

namespace {

using sscan::bf16;
using sscan::Requests;

struct StepParams {
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
    long long batch, z_stride;
    int dim, N, softplus;
    Requests req;
};

__device__ __forceinline__ void load4(const float* p, float (&v)[4]) {
    const float4 q = __ldg(reinterpret_cast<const float4*>(p));
    v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
}
__device__ __forceinline__ void load4(const bf16* p, float (&v)[4]) {
    const uint2 q = __ldg(reinterpret_cast<const uint2*>(p));
    v[0] = __uint_as_float(q.x << 16); v[1] = __uint_as_float(q.x & 0xffff0000u);
    v[2] = __uint_as_float(q.y << 16); v[3] = __uint_as_float(q.y & 0xffff0000u);
}

// Q threads a channel, G groups of 4 states a thread (states 4*(q + Q*g) ..).
// VEC: N is a multiple of 4 and every row of states, A, B and C is aligned for 4 values at once.
template <typename T, int Q, int G, bool VEC>
__global__ void __launch_bounds__(256) sscan_step_slots_kernel(const StepParams p) {
    const long long tid = (long long)blockIdx.x * 256 + threadIdx.x;
    const int q = (int)(tid % Q);
    const bool valid = tid / Q < p.dim;
    const long long d = valid ? tid / Q : p.dim - 1;
    if (blockIdx.x == 0 && blockIdx.y == 0) p.req.check(threadIdx.x, 256);
    for (long long b = blockIdx.y; b < p.batch; b += gridDim.y) {
        const int slot = p.req.slot((int)b);
        float* row = p.state + ((long long)(slot < 0 ? 0 : slot) * p.dim + d) * p.N;
        const long long at = b * p.dim + d;
        float h[G][4];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const int n0 = 4 * (q + Q * g);
#pragma unroll
            for (int i = 0; i < 4; ++i) h[g][i] = 0.f;
            if (slot < 0 || !valid || n0 >= p.N) continue;
            if (VEC) {
                const float4 v = *reinterpret_cast<const float4*>(row + n0);
                h[g][0] = v.x; h[g][1] = v.y; h[g][2] = v.z; h[g][3] = v.w;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) if (n0 + i < p.N) h[g][i] = row[n0 + i];
            }
        }
        float dt = sscan::to_f32(static_cast<const T*>(p.delta)[at]);
        const float u = sscan::to_f32(static_cast<const T*>(p.u)[at]);
        if (p.bias != nullptr) dt += __ldg(p.bias + d);
        if (p.softplus) dt = sscan::softplus_f32(dt);
        const float du = dt * u, dl = dt * sscan::kLog2e;
        const T* B = static_cast<const T*>(p.B) + b * p.N;
        const T* C = static_cast<const T*>(p.C) + b * p.N;
        const float* A = p.A + d * p.N;
        float y = 0.f;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const int n0 = 4 * (q + Q * g);
            if (n0 >= p.N) continue;
            float a[4], bv[4], cv[4];
            if (VEC) {
                load4(A + n0, a);
                load4(B + n0, bv);
                load4(C + n0, cv);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bool on = n0 + i < p.N;
                    a[i] = on ? A[n0 + i] : 0.f;
                    bv[i] = on ? sscan::to_f32(B[n0 + i]) : 0.f;
                    cv[i] = on ? sscan::to_f32(C[n0 + i]) : 0.f;
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (!VEC && n0 + i >= p.N) continue;
                h[g][i] = fmaf(sscan::ex2(dl * a[i]), h[g][i], du * bv[i]);
                y = fmaf(cv[i], h[g][i], y);
            }
            if (slot < 0 || !valid) continue;
            if (VEC) {
                *reinterpret_cast<float4*>(row + n0) = make_float4(h[g][0], h[g][1], h[g][2], h[g][3]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) if (n0 + i < p.N) row[n0 + i] = h[g][i];
            }
        }
        y = sscan::warp_sum<Q>(y);
        if (q == 0 && valid) {
            if (p.D != nullptr) y = fmaf(__ldg(p.D + d), u, y);
            if (p.z != nullptr) {
                const float g = sscan::to_f32(static_cast<const T*>(p.z)[b * p.z_stride + d]);
                y *= g * sscan::fast_sigmoid(g);
            }
            static_cast<T*>(p.out)[at] = sscan::from_f32<T>(y);
        }
    }
}

template <typename T, int Q, int G>
cudaError_t run_step(const StepParams& p, bool vec, cudaStream_t st) {
    const dim3 grid((unsigned)sscan::div_up((long long)p.dim * Q, 256), (unsigned)(p.batch < 65535 ? p.batch : 65535));
    if (vec) return sscan::launch(sscan_step_slots_kernel<T, Q, G, true>, grid, dim3(256), 0, st, false, p);
    return sscan::launch(sscan_step_slots_kernel<T, Q, G, false>, grid, dim3(256), 0, st, false, p);
}
template <typename T>
cudaError_t run_all(const StepParams& p, bool vec, cudaStream_t st) {
    if (p.N <= 4) return run_step<T, 1, 1>(p, vec, st);
    if (p.N <= 8) return run_step<T, 1, 2>(p, vec, st);
    if (p.N <= 16) return run_step<T, 2, 2>(p, vec, st);
    if (p.N <= 32) return run_step<T, 4, 2>(p, vec, st);
    return run_step<T, 8, 2>(p, vec, st);
}

}  // namespace

extern "C" int sscan_step_slots(const void* u, const void* delta, const float* A, const void* B, const void* C,
                                const float* D, const void* z, const float* delta_bias, const int32_t* slots,
                                float* state, void* out, int64_t batch, int64_t num_slots, int64_t dim, int64_t dstate,
                                int64_t z_stride, int dtype, int flags, void* stream) {
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    sscan::record_call(0, st, "rejected");
    if (dtype != SSCAN_F32 && dtype != SSCAN_BF16) return SSCAN_ERR_INVALID;
    if (dstate < 1 || dstate > sscan_max_dstate() || (flags & ~SSCAN_DELTA_SOFTPLUS)) return SSCAN_ERR_INVALID;
    const long long lim = 1LL << 28;  // 32-bit channel, request and row numbers on the device
    if (batch < 0 || dim < 0 || num_slots < 0 || z_stride < 0 || batch > lim || dim > lim || num_slots > lim ||
        (slots == nullptr && batch > num_slots))
        return SSCAN_ERR_INVALID;
    if (batch == 0 || dim == 0) {
        sscan::record_call(0, st, "empty");
        return SSCAN_OK;
    }
    if (!u || !delta || !A || !B || !C || !out || (num_slots && !state)) return SSCAN_ERR_INVALID;
    int* status = sscan::device_status_word();
    if (status == nullptr) return sscan::finish(cudaErrorUnknown);
    StepParams p = {};
    p.u = u; p.delta = delta; p.A = A; p.B = B; p.C = C; p.D = D; p.z = z; p.bias = delta_bias;
    p.state = state; p.out = out; p.batch = batch; p.z_stride = z_stride;
    p.dim = (int)dim; p.N = (int)dstate; p.softplus = flags & SSCAN_DELTA_SOFTPLUS;
    p.req = Requests{nullptr, slots, nullptr, (int)batch, (int)num_slots, 0, status};
    const unsigned align = dtype == SSCAN_F32 ? 16 : 8;
    const bool vec = dstate % 4 == 0 && sscan::is_aligned(state, 16) && sscan::is_aligned(A, 16) &&
                     sscan::is_aligned(B, align) && sscan::is_aligned(C, align);
    sscan::record_call(1, st, vec ? "step slots vec=1" : "step slots vec=0");
    return sscan::finish(dtype == SSCAN_F32 ? run_all<float>(p, vec, st) : run_all<bf16>(p, vec, st));
}
