// Entry point of the packed selective scan (kernels: sscan_prompt_kernel.cuh).
#include <stdio.h>

#include "sscan_prompt.cuh"

namespace {
constexpr long long kBig = 1LL << 40;
constexpr long long kIntMax = 1LL << 30;  // token, request and channel numbers are 32-bit on the device

bool sizes_ok(long long a, long long b, long long c) {
    return a >= 0 && b >= 0 && c >= 0 && a <= kBig && b <= kBig && c <= kBig && (!a || b <= kBig / a) &&
           (!(a * b) || c <= kBig / (a * b));
}

}  // namespace

extern "C" int sscan_prompt(const void* u, const void* delta, const float* A, const void* B, const void* C,
                            const float* D, const void* z, const float* delta_bias, const int32_t* cu_seqlens,
                            const int32_t* slots, const uint8_t* has_state, float* state, void* out, int64_t requests,
                            int64_t num_slots, int64_t dim, int64_t tokens, int64_t dstate, int dtype, int flags,
                            int segments, void* stream) {
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    sscan::record_call(0, st, "rejected");
    if (dtype != SSCAN_F32 && dtype != SSCAN_BF16) return SSCAN_ERR_INVALID;
    if (dstate < 1 || dstate > sscan_max_dstate() || segments < 0 || (flags & ~SSCAN_DELTA_SOFTPLUS)) return SSCAN_ERR_INVALID;
    if (!sizes_ok(1, dim, tokens) || !sizes_ok(num_slots, dim, dstate) || !sizes_ok(1, tokens, dstate)) return SSCAN_ERR_INVALID;
    if (requests < 0 || requests > kIntMax || tokens > kIntMax || num_slots > kIntMax || dim > kIntMax ||
        (slots == nullptr && requests > num_slots))
        return SSCAN_ERR_INVALID;
    if (dim == 0 || (requests == 0 && tokens == 0)) {
        sscan::record_call(0, st, "empty");
        return SSCAN_OK;
    }
    if (!cu_seqlens || (num_slots && !state) || !A || (tokens && (!u || !delta || !B || !C || !out))) return SSCAN_ERR_INVALID;
    int* status = sscan::device_status_word();
    if (status == nullptr) return sscan::finish(cudaErrorUnknown);
    sscan::PromptParams p = {};
    p.u = u; p.delta = delta; p.A = A; p.B = B; p.C = C; p.D = D; p.z = z; p.bias = delta_bias; p.state = state; p.out = out;
    p.dim = dim; p.tokens = (int)tokens; p.N = (int)dstate;
    p.softplus = flags & SSCAN_DELTA_SOFTPLUS;
    p.req = sscan::Requests{cu_seqlens, slots, has_state, (int)requests, (int)num_slots, (int)tokens, status};
    const bool aligned = tokens % (dtype == SSCAN_F32 ? 4 : 8) == 0 && sscan::is_aligned(u, 16) &&
                         sscan::is_aligned(delta, 16) && sscan::is_aligned(B, 16) && sscan::is_aligned(C, 16) &&
                         sscan::is_aligned(z, 16) && sscan::is_aligned(out, 16);
    // A CTA of wide threads covers 128 channels of up to 16 states.  One wave of
    // as many of them as the SMs hold shares the packed axis (65536 x 1536 fp32:
    // 25 segments 545 us, 20 676 us, 28, a second wave, 869 us).  Short segments
    // lose more to the walks back from their ends than the last CTA of an SM
    // gains: the SMs then take one less.
    //   fp32, the direct form: 512 x 8192 in 37 segments of 224 tokens, one CTA an SM,
    //     59 us, 74 of 112 71 us; but 1536 x 8192 25 of 336 122 us, 12 of 688 129 us
    //   unaligned fp32: 700 x 3001 with options 24 of 128 75 us, 47 of 64 91 us;
    //     911 x 1670 18 of 96, one CTA an SM, 52 us, 27 of 64 62 us
    //   bf16 with options: 1024 x 4097 37 of 112, two an SM, 78 us, 52 of 80 86 us,
    //     19 of 224 89 us; but 5120 x 1024 11 of 96 70 us, 6 of 176 76 us
    //   one lane a channel, not direct: 512 x 9001 bf16 141 of 64 54 us, 74 of 128 70 us
    // No segment has less than 64 tokens.  Where those are too few for one CTA
    // an SM, narrow threads spread the work over four times as many warps
    // (5120 channels x 37 tokens: 8 us against 14).
    const bool direct = dtype == SSCAN_F32 && aligned && z == nullptr && delta_bias == nullptr && flags == 0;
    const bool options = z != nullptr || delta_bias != nullptr || flags != 0;
    const int lanes = dstate <= 8 ? 1 : dstate <= 16 ? 2 : dstate <= 32 ? 4 : 8;
    const long long chunks = sscan::div_up(tokens > 0 ? tokens : 1, sscan::kSegStep);
    const long long shortest = 64 / sscan::kSegStep;
    long long tiles = sscan::div_up(dim, sscan::kPromptWarps * (32 / lanes) * 2);
    p.narrow = tiles * sscan::div_up(chunks, shortest) < 152;
    if (p.narrow) tiles = sscan::div_up(dim, sscan::kPromptWarps * (32 / (2 * lanes)));
    // CTAs an SM holds: by registers, or (wider rows of more arrays) by shared memory
    const int resident = p.narrow ? 4 : direct || lanes == 1 || (dtype == SSCAN_F32 && !aligned && options) ? 2 : 3;
    auto per_segment = [&](int ctas) {
        const long long count = (long long)ctas * 152 / tiles;
        return sscan::div_up(chunks, count < 1 ? 1 : count);
    };
    long long per;
    if (segments > 0) {
        per = sscan::div_up(chunks, segments);
    } else {
        int ctas = resident;
        auto long_enough = [&]() { return (resident == 2 ? 160 : ctas == 3 ? 96 : 80) / sscan::kSegStep; };
        while (!p.narrow && (direct || lanes > 1) && ctas > 1 && per_segment(ctas) < long_enough()) --ctas;
        per = per_segment(ctas);
        if (per < shortest) per = shortest;
    }
    if (per > chunks) per = chunks;
    while (sscan::div_up(chunks, per) > 65535) per *= 2;
    p.seg_tokens = (int)(per * sscan::kSegStep);
    p.segments = (int)sscan::div_up(chunks, per);
    void* scratch = nullptr;
    if (p.segments > 1) {
        const size_t cells = (size_t)p.segments * (size_t)dim;
        const size_t groups = (size_t)sscan::div_up(dstate, sscan::kEndStates);
        const cudaError_t e = sscan::scratch_alloc(&scratch, cells * (2 * (size_t)dstate + groups) * sizeof(float), st);
        if (e != cudaSuccess) return sscan::finish(e);
        p.h_end = static_cast<float*>(scratch);
        p.h_first = p.h_end + cells * (size_t)dstate;
        p.dt_sum = p.h_first + cells * (size_t)dstate;
    }
    char plan[96];
    snprintf(plan, sizeof(plan), "sscan prompt lanes=%d%s segments=%d of %d", p.narrow ? 2 * lanes : lanes,
             p.narrow ? " narrow" : "", p.segments, p.seg_tokens);
    sscan::record_call(p.segments > 1 ? 2 : 1, st, plan);
    cudaError_t e;
    if (dtype == SSCAN_F32) e = aligned ? sscan::prompt_launch<float, true>(p, st) : sscan::prompt_launch<float, false>(p, st);
    else e = aligned ? sscan::prompt_launch<sscan::bf16, true>(p, st) : sscan::prompt_launch<sscan::bf16, false>(p, st);
    if (scratch != nullptr) {
        const cudaError_t ef = cudaFreeAsync(scratch, st);
        if (e == cudaSuccess) e = ef;
    }
    return sscan::finish(e);
}
