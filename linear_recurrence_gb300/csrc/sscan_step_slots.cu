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
// shuffles.  A state is touched once a step, so it passes through the L2 marked
// to be replaced first (256 x 5120 x 16: 31.0 us, against 34.5 without the marks).
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

// Q threads a channel, G groups of 4 states a thread (states 4*(q + Q*g) ..),
// R requests a thread: their states are all on the way before the first is
// used, and A is read once for them.
// VEC: N is a multiple of 4 and every row of states, A, B and C is aligned for 4 values at once.
template <typename T, int Q, int G, int R, bool VEC>
__global__ void __launch_bounds__(256) sscan_step_slots_kernel(const StepParams p) {
    const long long tid = (long long)blockIdx.x * 256 + threadIdx.x;
    const int q = (int)(tid % Q);
    const bool valid = tid / Q < p.dim;
    const long long d = valid ? tid / Q : p.dim - 1;
    if (blockIdx.x == 0 && blockIdx.y == 0) p.req.check(threadIdx.x, 256);
    for (long long b0 = (long long)blockIdx.y * R; b0 < p.batch; b0 += (long long)gridDim.y * R) {
        int slot[R];
        float h[R][G][4], dt[R], u[R], z[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const long long b = b0 + r < p.batch ? b0 + r : p.batch - 1;
            slot[r] = b0 + r < p.batch && valid ? p.req.slot((int)b) : -1;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float* row = p.state + ((long long)(slot[r] < 0 ? 0 : slot[r]) * p.dim + d) * p.N;
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const int n0 = 4 * (q + Q * g);
#pragma unroll
                for (int i = 0; i < 4; ++i) h[r][g][i] = 0.f;
                if (slot[r] < 0 || n0 >= p.N) continue;
                if (VEC) {
                    const float4 v = __ldcs(reinterpret_cast<const float4*>(row + n0));
                    h[r][g][0] = v.x; h[r][g][1] = v.y; h[r][g][2] = v.z; h[r][g][3] = v.w;
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) if (n0 + i < p.N) h[r][g][i] = row[n0 + i];
                }
            }
            const long long b = b0 + r < p.batch ? b0 + r : p.batch - 1, at = b * p.dim + d;
            dt[r] = sscan::to_f32(static_cast<const T*>(p.delta)[at]);
            u[r] = sscan::to_f32(static_cast<const T*>(p.u)[at]);
            z[r] = p.z != nullptr ? sscan::to_f32(static_cast<const T*>(p.z)[b * p.z_stride + d]) : 0.f;
        }
        const float bias = p.bias != nullptr ? __ldg(p.bias + d) : 0.f;
        const float skip = p.D != nullptr ? __ldg(p.D + d) : 0.f;
        const float* A = p.A + d * p.N;
        float a[G][4], y[R];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const int n0 = 4 * (q + Q * g);
#pragma unroll
            for (int i = 0; i < 4; ++i) a[g][i] = 0.f;
            if (n0 >= p.N) continue;
            if (VEC) {
                load4(A + n0, a[g]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) if (n0 + i < p.N) a[g][i] = A[n0 + i];
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const long long b = b0 + r < p.batch ? b0 + r : p.batch - 1;
            float* row = p.state + ((long long)(slot[r] < 0 ? 0 : slot[r]) * p.dim + d) * p.N;
            dt[r] += bias;
            if (p.softplus) dt[r] = sscan::softplus_f32(dt[r]);
            const float du = dt[r] * u[r], dl = dt[r] * sscan::kLog2e;
            const T* B = static_cast<const T*>(p.B) + b * p.N;
            const T* C = static_cast<const T*>(p.C) + b * p.N;
            y[r] = 0.f;
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const int n0 = 4 * (q + Q * g);
                if (n0 >= p.N) continue;
                float bv[4], cv[4];
                if (VEC) {
                    load4(B + n0, bv);
                    load4(C + n0, cv);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        bv[i] = n0 + i < p.N ? sscan::to_f32(B[n0 + i]) : 0.f;
                        cv[i] = n0 + i < p.N ? sscan::to_f32(C[n0 + i]) : 0.f;
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (!VEC && n0 + i >= p.N) continue;
                    h[r][g][i] = fmaf(sscan::ex2(dl * a[g][i]), h[r][g][i], du * bv[i]);
                    y[r] = fmaf(cv[i], h[r][g][i], y[r]);
                }
                if (slot[r] < 0) continue;
                if (VEC) {
                    __stcs(reinterpret_cast<float4*>(row + n0), make_float4(h[r][g][0], h[r][g][1], h[r][g][2], h[r][g][3]));
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) if (n0 + i < p.N) row[n0 + i] = h[r][g][i];
                }
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            y[r] = fmaf(skip, u[r], sscan::warp_sum<Q>(y[r]));
            if (q == 0 && valid && b0 + r < p.batch) {
                if (p.z != nullptr) y[r] *= z[r] * sscan::fast_sigmoid(z[r]);
                static_cast<T*>(p.out)[(b0 + r) * p.dim + d] = sscan::from_f32<T>(y[r]);
            }
        }
    }
}

template <typename T, int Q, int G, int R>
cudaError_t run_rows(const StepParams& p, bool vec, cudaStream_t st) {
    const long long gy = sscan::div_up(p.batch, R);
    const dim3 grid((unsigned)sscan::div_up((long long)p.dim * Q, 256), (unsigned)(gy < 65535 ? gy : 65535));
    if (vec) return sscan::launch(sscan_step_slots_kernel<T, Q, G, R, true>, grid, dim3(256), 0, st, false, p);
    return sscan::launch(sscan_step_slots_kernel<T, Q, G, R, false>, grid, dim3(256), 0, st, false, p);
}
template <typename T, int Q, int G>
cudaError_t run_step(const StepParams& p, bool vec, cudaStream_t st) {
    // two requests a thread once that still leaves eight CTAs an SM (256 x 5120
    // x 16, before the marks on the state: 34.5 us; one request 39.0, four 41.7)
    const long long ctas = p.batch * sscan::div_up((long long)p.dim * Q, 256);
    return ctas >= 16 * 152 ? run_rows<T, Q, G, 2>(p, vec, st) : run_rows<T, Q, G, 1>(p, vec, st);
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
