// Entry points of linear attention with a decay for each head (kernels:
// lattn_simt.cuh; single tokens: lattn_step.cu).
#include <stdio.h>

#include "lattn.cuh"

namespace {
using sscan::kChunk;
using sscan::kValueTile;
using sscan::LattnParams;

constexpr long long kBig = 1LL << 40;
constexpr long long kIntMax = 1LL << 30;  // token, request and channel numbers are 32-bit on the device
constexpr long long kGridYZ = 65535;
constexpr long long kSms = 152;

bool product_ok(long long a, long long b, long long c) {
    return a >= 0 && b >= 0 && c >= 0 && a <= kBig && b <= kBig && c <= kBig && (!a || b <= kBig / a) &&
           (!(a * b) || c <= kBig / (a * b));
}

// Sizes and strides that every call shares.
bool sizes_ok(long long batch, long long heads, long long groups, long long key, long long value, long long len, int dtype,
              int flags) {
    return (dtype == SSCAN_F32 || dtype == SSCAN_BF16) && (flags & ~SSCAN_DELTA_SOFTPLUS) == 0 && key >= 1 &&
           key <= LATTN_MAX_KEY && value >= 1 && value <= LATTN_MAX_VALUE && groups >= 1 && heads >= 0 && heads <= kGridYZ &&
           heads % groups == 0 && batch >= 0 && batch <= kGridYZ && len >= 0 && len <= kIntMax &&
           product_ok(batch, heads * value, len) && product_ok(batch, groups * key, len);
}

void fill(LattnParams& p, const void* q, const void* k, const void* v, const float* A, const void* delta, const float* D,
          const float* bias, const int64_t* strides, int64_t batch, int64_t heads, int64_t groups, int64_t key, int64_t value,
          int64_t len, float scale, int flags, int chunk) {
    p.q = q; p.k = k; p.v = v; p.A = A; p.delta = delta; p.D = D; p.bias = bias;
    p.qb = strides[0]; p.qd = strides[1]; p.kb = strides[2]; p.kd = strides[3];
    p.vb = strides[4]; p.vd = strides[5]; p.tb = strides[6]; p.td = strides[7];
    p.batch = (int)batch; p.heads = (int)heads; p.groups = (int)groups; p.N = (int)key; p.P = (int)value; p.L = (int)len;
    p.vtiles = (int)sscan::div_up(value, kValueTile);
    p.scale = scale; p.softplus = flags & SSCAN_DELTA_SOFTPLUS;
    p.chunk = chunk;
    p.chunks = (int)sscan::div_up(len, chunk);
    p.pieces = 1; p.span = p.chunks * chunk; p.subsets = 1;
}

bool strides_ok(const int64_t* s, const void* delta) {
    if (s == nullptr) return false;
    for (int i = 0; i < (delta != nullptr ? 8 : 6); ++i)
        if (s[i] < 0 || s[i] > kBig) return false;
    return true;
}

size_t tile_floats(const LattnParams& p) {
    return (size_t)kValueTile * (p.N <= 64 ? 64 : 128);
}

// Parts of time for the walks; `pieces` pins them.  Chosen by what they take, in chunks of one
// CTA.  With the outputs each wave of CTAs walks a part, and takes `ends` to begin and end.  The pass
// before it, which leaves the outputs out, takes 0.7 of what a part holds of the state before the
// next: all of it on one sequence, little where a part holds several requests, as parts then begin
// with one; those parts are up to half as long again.  Joining the states of all parts before
// takes `join` a part, and the pass itself, with its scratch, the host `call`.  (bf16: 24 heads x 65536 tokens: 6
// parts 368 us, 5 433, 7 494, 12 389; 1 head: 32 parts 91 us, 64 74, 100 74, 150 84; 80 heads x 8209
// tokens in 24 requests: 5 parts 233 us, 3 249, 1 326.  fp32, 1 head x 65536: 100 parts 370 us, 150 258.)
void split_time(LattnParams& p, int pieces) {
    const long long tiles = (long long)p.batch * p.heads * p.vtiles, chunks = p.chunks > 0 ? p.chunks : 1;
    if (pieces <= 0) {
        const bool tc = p.chunk == sscan::kTcChunk;
        const double ends = tc ? 2.5 : 0.6, join = tc ? 0.14 : 0.02, call = tc ? 1.5 : 0.5;
        const double request = p.packed && p.req.requests > 0 ? (double)chunks / p.req.requests : (double)chunks;
        const long long most = kSms / tiles > 32 ? kSms / tiles : 32;
        double best = 0;
        for (long long n = 1; n <= most && n <= chunks; ++n) {
            const double part = (double)sscan::div_up(chunks, n);
            const bool several = request <= part / 2;  // requests in a part
            const double before = several ? 0.5 : request < part ? request : part;
            double cost = sscan::div_up(tiles * n, (long long)kSms) * (part + ends);
            if (n > 1) cost += sscan::div_up(tiles * (n - 1), (long long)kSms) * (0.7 * before + ends) + join * n + call + (several ? 0.25 * part : 0);
            if (n == 1 || cost < best) {
                best = cost;
                pieces = (int)n;
            }
        }
    }
    if (pieces > chunks) pieces = (int)chunks;
    if (pieces > kGridYZ) pieces = (int)kGridYZ;
    const long long per = sscan::div_up(chunks, pieces);
    p.pieces = (int)sscan::div_up(chunks, per);
    p.span = (int)(per * p.chunk);
}

// Outputs and final states.
int run_walk(LattnParams& p, int pieces, const char* what, int dtype, cudaStream_t st) {
    const long long tiles = (long long)p.batch * p.heads * p.vtiles;
    split_time(p, pieces);
    void* scratch = nullptr;
    if (p.pieces > 1) {
        const size_t ends = (size_t)p.pieces * tiles * tile_floats(p), sums = (size_t)p.pieces * p.batch * p.heads;
        const cudaError_t e = sscan::scratch_alloc(&scratch, (ends * (p.packed ? 2 : 1) + sums) * sizeof(float), st);
        if (e != cudaSuccess) return sscan::finish(e);
        p.ends = static_cast<float*>(scratch);
        p.aside = p.ends + ends;
        p.sums = p.ends + ends * (p.packed ? 2 : 1);
    }
    char plan[80];
    snprintf(plan, sizeof(plan), "lattn %s pieces=%d", what, p.pieces);
    const bool copies = dtype == SSCAN_BF16 && p.L > 0 && sscan::lattn_tc_copies(p);
    sscan::record_call((p.pieces > 1 ? 2 : 1) + (copies ? 1 : 0) + (p.apart ? 1 : 0), st, plan);
    cudaError_t e = dtype == SSCAN_BF16 ? sscan::lattn_tc_walk_launch(p, st) : sscan::lattn_walk_launch(p, st);
    if (scratch != nullptr) {
        const cudaError_t ef = cudaFreeAsync(scratch, st);
        if (e == cudaSuccess) e = ef;
    }
    return sscan::finish(e);
}
}  // namespace

extern "C" int lattn_fwd(const void* q, const void* k, const void* v, const float* A, const void* delta, const float* D,
                         const float* delta_bias, const float* s0, void* o, float* final_state, int64_t batch, int64_t heads,
                         int64_t groups, int64_t key, int64_t value, int64_t seqlen, const int64_t* strides, float scale,
                         int dtype, int flags, int pieces, void* stream) {
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    sscan::record_call(0, st, "rejected");
    if (!sizes_ok(batch, heads, groups, key, value, seqlen, dtype, flags) || pieces < 0 || !strides_ok(strides, delta)) return SSCAN_ERR_INVALID;
    if (batch == 0 || heads == 0 || (seqlen == 0 && final_state == nullptr)) {
        sscan::record_call(0, st, "empty");
        return SSCAN_OK;
    }
    if (seqlen == 0) {
        const size_t bytes = (size_t)(batch * heads * value * key) * sizeof(float);
        sscan::record_call(0, st, "empty: final_state only");
        return sscan::finish(s0 != nullptr ? cudaMemcpyAsync(final_state, s0, bytes, cudaMemcpyDeviceToDevice, st)
                                           : cudaMemsetAsync(final_state, 0, bytes, st));
    }
    if (!q || !k || !v || !A || !o) return SSCAN_ERR_INVALID;
    int* status = sscan::device_status_word();
    if (status == nullptr) return sscan::finish(cudaErrorUnknown);
    LattnParams p = {};
    p.failed = status;
    fill(p, q, k, v, A, delta, D, delta_bias, strides, batch, heads, groups, key, value, seqlen, scale, flags, dtype == SSCAN_BF16 ? sscan::kTcChunk : kChunk);
    p.o = o; p.s_in = s0; p.s_out = final_state;
    return run_walk(p, pieces, "fwd", dtype, st);
}

extern "C" int lattn_prompt(const void* q, const void* k, const void* v, const float* A, const void* delta, const float* D,
                            const float* delta_bias, const int32_t* cu_seqlens, const int32_t* slots, const uint8_t* has_state,
                            float* state, void* o, int64_t requests, int64_t num_slots, int64_t heads, int64_t groups,
                            int64_t key, int64_t value, int64_t tokens, const int64_t* strides, float scale, int dtype,
                            int flags, int pieces, void* stream) {
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    sscan::record_call(0, st, "rejected");
    if (!sizes_ok(1, heads, groups, key, value, tokens, dtype, flags) || pieces < 0 || !strides_ok(strides, delta)) return SSCAN_ERR_INVALID;
    if (requests < 0 || requests > kIntMax || num_slots < 0 || num_slots > kIntMax || !product_ok(num_slots, heads * value, key) ||
        (slots == nullptr && requests > num_slots))
        return SSCAN_ERR_INVALID;
    if (heads == 0 || (requests == 0 && tokens == 0)) {
        sscan::record_call(0, st, "empty");
        return SSCAN_OK;
    }
    if (!cu_seqlens || (num_slots && !state) || !A || (tokens && (!q || !k || !v || !o))) return SSCAN_ERR_INVALID;
    int* status = sscan::device_status_word();
    if (status == nullptr) return sscan::finish(cudaErrorUnknown);
    LattnParams p = {};
    fill(p, q, k, v, A, delta, D, delta_bias, strides, 1, heads, groups, key, value, tokens, scale, flags, dtype == SSCAN_BF16 ? sscan::kTcChunk : kChunk);
    p.o = o; p.s_in = state; p.s_out = state;
    p.packed = true;
    p.failed = status;
    p.req = sscan::Requests{cu_seqlens, slots, has_state, (int)requests, (int)num_slots, (int)tokens, status};
    // Where requests are short on average some are very short: they go token by token.  (One
    // kernel more costs others about 3 us.)
    p.apart = requests > 1 && tokens <= 128 * requests;
    if (p.apart) {
        const cudaError_t e = sscan::lattn_short_launch(p, dtype, st);
        if (e != cudaSuccess) return sscan::finish(e);
    }
    return run_walk(p, pieces, "prompt", dtype, st);
}

extern "C" int lattn_bwd(const void* q, const void* k, const void* v, const float* A, const void* delta, const float* D,
                         const float* delta_bias, const float* s0, const void* dout, const float* dfinal_state, void* dq,
                         void* dk, void* dv, void* ddelta, float* dA, float* dD, float* ddelta_bias, float* ds0, int64_t batch,
                         int64_t heads, int64_t groups, int64_t key, int64_t value, int64_t seqlen, const int64_t* strides,
                         float scale, int dtype, int flags, void* stream) {
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    sscan::record_call(0, st, "rejected");
    if (!sizes_ok(batch, heads, groups, key, value, seqlen, dtype, flags) || !strides_ok(strides, delta)) return SSCAN_ERR_INVALID;
    if (heads == 0) {
        sscan::record_call(0, st, "empty");
        return SSCAN_OK;
    }
    if (!dA) return SSCAN_ERR_INVALID;
    if (batch == 0 || seqlen == 0) {
        sscan::record_call(0, st, "empty: gradients of no tokens");
        cudaError_t e = cudaMemsetAsync(dA, 0, (size_t)heads * sizeof(float), st);
        if (e == cudaSuccess && dD != nullptr) e = cudaMemsetAsync(dD, 0, (size_t)heads * sizeof(float), st);
        if (e == cudaSuccess && ddelta_bias != nullptr) e = cudaMemsetAsync(ddelta_bias, 0, (size_t)heads * sizeof(float), st);
        const size_t bytes = (size_t)(batch * heads * value * key) * sizeof(float);
        if (e == cudaSuccess && ds0 != nullptr && bytes)
            e = dfinal_state != nullptr ? cudaMemcpyAsync(ds0, dfinal_state, bytes, cudaMemcpyDeviceToDevice, st) : cudaMemsetAsync(ds0, 0, bytes, st);
        return sscan::finish(e);
    }
    if (!q || !k || !v || !A || !dout || !dq || !dk || !dv || (delta && !ddelta)) return SSCAN_ERR_INVALID;
    int* status = sscan::device_status_word();
    if (status == nullptr) return sscan::finish(cudaErrorUnknown);
    LattnParams p = {};
    p.failed = status;
    const bool tc = dtype == SSCAN_BF16 && batch * groups * seqlen > sscan::kLattnFew;
    fill(p, q, k, v, A, delta, D, delta_bias, strides, batch, heads, groups, key, value, seqlen, scale, flags, tc ? sscan::kTcChunk : kChunk);
    p.dout = dout; p.s_in = s0; p.ds_in = dfinal_state; p.ds_out = ds0;
    p.dq = dq; p.dk = dk; p.dv = dv; p.ddelta = ddelta;
    // A group's heads in one CTA need no sum of parts.  Shared out among more CTAs they fill the
    // GPU: as many as make the last CTA end first, a wave of CTAs taking as long as its heads
    // and one more for its beginning and end; a set of parts costs about a quarter of a head (and a
    // sixteenth where a few tokens' parts are small: 1 token x 80 heads 201 -> 107 us).
    const bool few = dtype == SSCAN_BF16 && !tc;
    const long long per = heads / groups, ctas = (long long)p.chunks * groups * batch;
    long long best = 0;
    for (long long s = 1; s <= per && s * groups <= kGridYZ; ++s) {
        const long long waves = sscan::div_up(ctas * s, kSms), cost = (few ? 16 : 4) * waves * (sscan::div_up(per, s) * p.vtiles + 1) + (s > 1 ? s : 0);
        if (s == 1 || cost < best) {
            best = cost;
            p.subsets = (int)s;
        }
    }
    if ((long long)p.groups * p.subsets > kGridYZ) return SSCAN_ERR_INVALID;
    const size_t states = (size_t)batch * heads * p.vtiles * p.chunks * tile_floats(p);
    const size_t part = p.subsets > 1 ? (size_t)p.subsets * batch * groups * key * seqlen : 0;
    const size_t head_part = (size_t)3 * heads * batch * p.chunks;
    split_time(p, 0);
    const size_t ends = p.pieces > 1 ? (size_t)p.pieces * batch * heads * p.vtiles * tile_floats(p) : 0;
    const size_t sums = p.pieces > 1 ? (size_t)p.pieces * batch * heads : 0;
    void* scratch = nullptr;
    cudaError_t e = sscan::scratch_alloc(&scratch, (2 * states + ends + 2 * part + head_part + sums) * sizeof(float), st);
    if (e != cudaSuccess) return sscan::finish(e);
    p.starts = static_cast<float*>(scratch);
    p.dends = p.starts + states;
    p.ends = p.dends + states;
    p.dq_part = part ? p.ends + ends : nullptr;
    p.dk_part = part ? p.dq_part + part : nullptr;
    p.head_part = p.ends + ends + 2 * part;
    p.sums = p.head_part + head_part;
    char plan[80];
    snprintf(plan, sizeof(plan), "lattn bwd subsets=%d pieces=%d", p.subsets, p.pieces);
    sscan::record_call((p.subsets > 1 ? 5 : 4) + (p.pieces > 1 ? 2 : 0) + (tc ? sscan::lattn_tc_grad_copies(p) : 0), st, plan);
    e = tc ? sscan::lattn_tc_grad_launch(p, st) : sscan::lattn_grad_launch(p, dtype, st);
    if (e == cudaSuccess && p.subsets > 1) e = sscan::lattn_parts_launch(p, dtype, st);
    if (e == cudaSuccess) e = sscan::lattn_heads_launch(p, dA, delta != nullptr ? ddelta_bias : nullptr, dD, st);
    const cudaError_t ef = cudaFreeAsync(scratch, st);
    return sscan::finish(e != cudaSuccess ? e : ef);
}
