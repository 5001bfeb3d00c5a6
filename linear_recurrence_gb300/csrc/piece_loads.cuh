// Loads of eight consecutive bf16 values from rows of any alignment.
#pragma once

#include "device_utils.cuh"

namespace sscan {

// Eight values from p on, the first `n` of them (zeros elsewhere), in two steps, so
// that a thread has the loads of several pieces on the way before it uses the
// first.  Where p lies off a 16-byte boundary both vectors around it are read and shifted
// into place; where those would leave [lo, hi), what may be read, values one by one.
struct Piece8 {
    uint4 a, b;
};
__device__ __forceinline__ bool piece_wide(const bf16* p, int n, const bf16* lo, const bf16* hi, unsigned phase) {
    return n > 0 && p - phase >= lo && p - phase + (phase ? 16 : 8) <= hi;
}
__device__ __forceinline__ unsigned phase8(const bf16* p) { return (unsigned)(reinterpret_cast<uintptr_t>(p) & 15u) >> 1; }
__device__ __forceinline__ void piece_load(Piece8& x, const bf16* p, int n, const bf16* lo, const bf16* hi) {
    const unsigned phase = phase8(p);
    const uint4* base = reinterpret_cast<const uint4*>(p - phase);
    const bool wide = piece_wide(p, n, lo, hi, phase);
    x.a = x.b = make_uint4(0u, 0u, 0u, 0u);
    if (wide) x.a = __ldg(base);
    if (wide && phase != 0) x.b = __ldg(base + 1);
}
// eight values from value `phase` of the two vectors on
__device__ __forceinline__ uint4 piece_shift(const Piece8& x, unsigned phase) {
    // words from 2 * (phase / 4) on, then from (phase / 2) % 2 on, then half a word
    const bool two = phase & 4, one = phase & 2;
    const unsigned w0 = two ? x.a.z : x.a.x, w1 = two ? x.a.w : x.a.y, w2 = two ? x.b.x : x.a.z, w3 = two ? x.b.y : x.a.w;
    const unsigned w4 = two ? x.b.z : x.b.x, w5 = two ? x.b.w : x.b.y;
    const unsigned x0 = one ? w1 : w0, x1 = one ? w2 : w1, x2 = one ? w3 : w2, x3 = one ? w4 : w3, x4 = one ? w5 : w4;
    const unsigned s = (phase & 1) * 16;
    return make_uint4(__funnelshift_r(x0, x1, s), __funnelshift_r(x1, x2, s), __funnelshift_r(x2, x3, s), __funnelshift_r(x3, x4, s));
}
// values [first, last) of eight, zeros in place of the others
__device__ __forceinline__ uint4 keep_values(uint4 x, int first, int last) {
    unsigned* w = &x.x;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] &= (2 * i >= first && 2 * i < last ? 0x0000ffffu : 0u) | (2 * i + 1 >= first && 2 * i + 1 < last ? 0xffff0000u : 0u);
    return x;
}
__device__ __forceinline__ uint4 piece_take(const Piece8& x, const bf16* p, int n, const bf16* lo, const bf16* hi) {
    const unsigned phase = phase8(p);
    if (n <= 0) return make_uint4(0u, 0u, 0u, 0u);
    if (!piece_wide(p, n, lo, hi, phase)) {
        unsigned w[4] = {0u, 0u, 0u, 0u};
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
            const unsigned v = (unsigned)__ldg(reinterpret_cast<const unsigned short*>(p) + i) << (16 * (i & 1));
            w[0] |= (i >> 1) == 0 ? v : 0u;
            w[1] |= (i >> 1) == 1 ? v : 0u;
            w[2] |= (i >> 1) == 2 ? v : 0u;
            w[3] |= (i >> 1) == 3 ? v : 0u;
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    return keep_values(piece_shift(x, phase), 0, n);
}
}  // namespace sscan
