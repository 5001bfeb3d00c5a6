// Helpers shared by the kernels around the scan (short convolution, packed
// scan, block norms): 16-byte vectors widened to fp32, activations, warp sums,
// bounds-checked request tables and programmatic dependent launches.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/sscan.h"
#include "device_utils.cuh"

namespace sscan {
// defined in sscan_abi.cu
void record_call(int launches, cudaStream_t stream, const char* plan);
void record_error(cudaError_t e);
cudaError_t scratch_alloc(void** ptr, size_t bytes, cudaStream_t stream);
int* device_status_word();

constexpr float kLog2e = 1.4426950408889634f;

// Elements of a 16-byte vector.
template <typename T> struct VecOf;
template <> struct VecOf<float> { static constexpr int E = 4; };
template <> struct VecOf<bf16> { static constexpr int E = 8; };

// 16 bytes widened to fp32 (and back, rounded to nearest even).
__device__ __forceinline__ void widen(const uint4& q, float (&v)[4], float*) {
    v[0] = __uint_as_float(q.x); v[1] = __uint_as_float(q.y);
    v[2] = __uint_as_float(q.z); v[3] = __uint_as_float(q.w);
}
__device__ __forceinline__ void widen(const uint4& q, float (&v)[8], bf16*) {
    const unsigned w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint4 narrow(const float (&v)[4], float*) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}
__device__ __forceinline__ uint4 narrow(const float (&v)[8], bf16*) {
    unsigned w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const unsigned*>(&p);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// sigmoid and softplus on the exponent unit.  sigmoid(x) = 1 / (1 + 2^(-x log2 e));
// for x below about -88 the exponential overflows to infinity and the result
// is 0, its limit.
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float fast_sigmoid(float x) { return rcp(1.f + ex2(-x * kLog2e)); }
// log(1 + e^x) = max(x, 0) + log(1 + e) with e = e^-|x| in (0, 1], and
// log(1 + e) = e * p(e), p the polynomial of degree 8 that meets log(1 + e) / e
// at the Chebyshev nodes of [0, 1], its coefficients rounded to fp32: 9.3e-8 of it
// off at most, 2e-7 with the rounding of the steps.  e adds the exponent unit's
// 2.4e-7 and the rounding of its exponent, which grows with |x| (7.3e-8 of e a unit):
// for negative x the result is within 6e-7 + 7.3e-8 |x| of itself, down to
// x = -87, where e is flushed to zero.
__device__ __forceinline__ float softplus_f32(float x) {
    const float e = ex2(-fabsf(x) * kLog2e);
    float p = fmaf(e, 0.0051261018961668015f, -0.029074065387248993f);
    p = fmaf(p, e, 0.0775160863995552f);
    p = fmaf(p, e, -0.13602247834205627f);
    p = fmaf(p, e, 0.19076880812644958f);
    p = fmaf(p, e, -0.2483539879322052f);
    p = fmaf(p, e, 0.3331812024116516f);
    p = fmaf(p, e, -0.4999944567680359f);
    p = fmaf(p, e, 0.9999999403953552f);
    return fmaf(e, p, fmaxf(x, 0.f));
}

template <int LANES = 32>
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// ---- request tables of packed calls ---------------------------------------
//
// A packed call lays the tokens of `requests` prompts end to end; prompt s owns
// tokens [cu[s], cu[s+1]).  The tables live on the device, so the host cannot
// check them: every kernel clamps what it reads from them to the arrays'
// bounds, and the device status word records a table that needed it.
struct Requests {
    const int* cu;             // [requests + 1]
    const int* slots;          // [requests] cache rows, or NULL: request s uses row s
    const unsigned char* has;  // [requests] continues from its cached state, or NULL: all do
    int requests;
    int num_slots;
    int tokens;
    int* status;

    __device__ __forceinline__ int offset(int s) const {
        const int v = __ldg(cu + s);
        return v < 0 ? 0 : v > tokens ? tokens : v;
    }
    // cache row of request s, or -1 when it keeps no state
    __device__ __forceinline__ int slot(int s) const {
        const int v = slots != nullptr ? __ldg(slots + s) : s;
        return v >= num_slots ? -1 : v;
    }
    __device__ __forceinline__ bool continues(int s) const { return has == nullptr || __ldg(has + s) != 0; }
    // the last request that starts at or before token t (skipping the empty
    // ones that start there too), or -1 / requests when t lies in none
    __device__ __forceinline__ int find(int t) const {
        int lo = -1, hi = requests;  // cu[lo] <= t < cu[hi]
        if (t >= offset(requests)) return requests;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (offset(mid) <= t) lo = mid; else hi = mid;
        }
        return lo;
    }
    // record entries of requests [first, first + step, ...] that lie outside the arrays
    __device__ __forceinline__ void check(int first, int step) const {
        bool bad = false;
        for (int s = first; s < requests; s += step) {
            if (cu != nullptr) {
                const int a = __ldg(cu + s), b = __ldg(cu + s + 1);
                bad |= a < 0 || b < a || b > tokens;
            }
            bad |= slots != nullptr && __ldg(slots + s) >= num_slots;
        }
        if (bad) *status = SSCAN_ERR_INVALID;
    }
};

// Launch as a programmatic dependent of the kernel before it on the stream
// (dependent == true; the kernel calls griddep_wait before it touches what
// that one writes) or as an ordinary kernel.
template <typename... KArgs, typename... Args>
inline cudaError_t launch(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, bool dependent,
                          Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = dependent ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

inline int finish(cudaError_t e) {
    if (e == cudaSuccess) return SSCAN_OK;
    record_error(e);
    return SSCAN_ERR_CUDA;
}
inline bool is_aligned(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1u)) == 0; }
inline long long div_up(long long a, long long b) { return (a + b - 1) / b; }

}  // namespace sscan
