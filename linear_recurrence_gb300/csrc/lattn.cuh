// Linear attention with a decay for each head: what its kernels share.
//
// Per head, with queries and keys of N channels, values of P channels, a decay
// rate A and a step dt_t for each token (dt = 1 where none is given):
//
//   S_t = e^(A dt_t) S_{t-1} + dt_t v_t k_t^T      S [P, N]
//   o_t = scale * S_t q_t + D v_t
//
// It is the selective scan with one rate a head, so that time can be cut into
// chunks whose inside is a product of matrices.  In a chunk that begins with
// state S, with T_t the sum of its steps up to and with token t, R_t the sum of
// its steps behind t, and E_ts = e^(A (T_t - T_s)) for s <= t (0 for s > t):
//
//   o_t  = scale * sum_s E_ts dt_s (q_t . k_s) v_s  +  scale * e^(A T_t) S q_t  +  D v_t
//   S'   = e^(A T_end) S + sum_s e^(A R_s) dt_s v_s k_s^T
//
// Gradients, from do and the gradient dS' of the state behind the chunk, with
// F_ts = scale * E_ts (q_t . k_s) and G_ts = do_t . v_s:
//
//   dS     = e^(A T_end) dS' + sum_t scale * e^(A T_t) do_t q_t^T       (of the state before the chunk)
//   dq_t   = scale * (sum_s E_ts G_ts dt_s k_s + e^(A T_t) S^T do_t)
//   dk_s   = sum_t scale * E_ts G_ts dt_s q_t + dt_s e^(A R_s) dS'^T v_s
//   dv_s   = dt_s * (sum_t F_ts do_t + e^(A R_s) dS' k_s) + D do_s
//   weight_s = sum_t F_ts G_ts + Y_s,  Y_s = e^(A R_s) v_s . dS' k_s    (of dt_s as the weight of v_s k_s^T)
//
// The exponent A dt_t stands in every pair around token t: with W_ts = F_ts G_ts dt_s
// its gradient is
//
//   g_t = sum_{t' >= t > s} W_t's + sum_{t' >= t} X_t' + sum_{s < t} dt_s Y_s + e^(A T_end) S . dS'
//   X_t = scale * e^(A T_t) do_t . S q_t
//
// where the first sum is sum_{t' >= t} (sum_{s < t'} W_t's - sum_{t'' > t'} W_t''t'): sums of a chunk only, so
// that a long sequence adds no cancellation.  ddt_t = A g_t + weight_t, dD = sum_t do_t . v_t.
// dA = sum dt_t g_t, summed term by term with the time that each spans,
//
//   dA = sum_{t > s} W_ts (T_t - T_s) + sum_t X_t T_t + sum_s dt_s Y_s R_s + e^(A T_end) S . dS' T_end
//
// since the g of a long step between short ones is what large sums leave over, and the step multiplies it: by
// sum dt_t g_t a rate of -16 with steps from 0.02 to 3 was off by 1.6e-5 in chunks of 64 tokens, 3.2e-5 in chunks of 128.
// ddelta_bias = sum slope_t ddt_t, slope_t the steps' derivative, is summed the same way, with Z_t the sum of
// the slopes up to and with token t in place of T_t (Z_end - Z_s in place of R_s):
//
//   dbias = sum slope_t weight_t + A (sum_{t > s} W_ts (Z_t - Z_s) + sum_t X_t Z_t + sum_s dt_s Y_s (Z_end - Z_s)
//                                     + e^(A T_end) S . dS' Z_end)
//
// (as the sum of slope_t ddt_t it was off by 1e-6 to 6e-6 of the heads' norm, by 1e-5 where a head's terms cancel).
#pragma once

#include "block_utils.cuh"

namespace sscan {

// Tokens of a chunk in the kernels on the FP32 units and on the tensor cores; value channels of a tile.
constexpr int kChunk = 64;
constexpr int kTcChunk = 128;
constexpr int kValueTile = 64;
constexpr int kLattnShort = 16;  // tokens of a request that is taken token by token
// Tokens of a set of queries and keys, over all batches and groups, up to which gradients in bf16 go to the FP32
// units.  dq and dk of so few are few sums over the heads that share them: where one happens to cancel, what the tensor
// cores round each head's weight by (2^-9) is a large part of all there is (2 tokens, 16 heads: off by up to 1.5e-2
// where exact ones rounded once are 1.7e-3).  Many tokens' sums do not cancel all at once.
constexpr int kLattnFew = 16;

// A sum and what its rounding left out.  The exponents between tokens of a chunk are differences of sums
// of steps; where a decay is fast the sums are large and only differences between neighbours count, in dA most:
// from sums in fp32 alone dA of a rate of -16 and steps of 0.8 was off by 1.4e-4 in chunks of 128 tokens, by
// 1.7e-5 in chunks of 64; fp32 outputs of a rate of -8, steps of 0.02 and a 10 at every fifth token by 3.2e-5, where
// two terms leave 1.4e-7.  The outputs in bf16 take one term: what it leaves out, 2^-24 of the sum of |A| dt over a
// chunk, stays below half a step of theirs up to sums of 2^15.
struct Sum2 {
    float h, l;
};
__device__ __forceinline__ Sum2 operator+(const Sum2& a, const Sum2& b) {
    const float s = __fadd_rn(a.h, b.h), v = __fsub_rn(s, a.h);
    const float lost = __fadd_rn(__fsub_rn(a.h, __fsub_rn(s, v)), __fsub_rn(b.h, v));
    return Sum2{s, __fadd_rn(__fadd_rn(a.l, b.l), lost)};
}
__device__ __forceinline__ Sum2 shfl_up2(const Sum2& a, int n) {
    return Sum2{__shfl_up_sync(0xffffffffu, a.h, n), __shfl_up_sync(0xffffffffu, a.l, n)};
}

struct LattnParams {
    const void *q, *k, *v, *delta;  // delta: NULL for steps of one
    const void* dout;
    const float *A, *D, *bias;
    void* o;
    const float* s_in;   // initial states (packed: the cache), or NULL: zeros
    float* s_out;        // final states (packed: the cache), or NULL
    const float* ds_in;  // gradient of the final states, or NULL
    float* ds_out;       // gradient of the initial states, or NULL
    void *dq, *dk, *dv, *ddelta;
    long long qb, qd, kb, kd, vb, vd, tb, td;  // batch and channel strides of q, k, v and delta
    int batch, heads, groups, N, P, L;
    int vtiles;  // tiles of value channels a head
    float scale;
    int softplus;
    // time split: pieces of `span` tokens (of a packed axis: about); what an earlier piece leaves behind
    int pieces, span;
    float* ends;   // [pieces][batch][heads * vtiles][kValueTile][KD] states behind each piece
    float* sums;   // [pieces][batch][heads] their steps
    float* aside;  // as ends: initial states of requests that cross a piece's end
    // gradients: states at every chunk's start, gradients of the states at its end
    float *starts, *dends;  // [batch][heads * vtiles][chunks][kValueTile][KD]
    int chunk, chunks;      // tokens of a chunk, and their number
    int subsets;    // subsets of a group's heads that a CTA each sums dq and dk of
    float *dq_part, *dk_part;  // [subsets][batch][groups * N][L], or NULL: one subset writes dq and dk itself
    float* head_part;          // [3][heads][batch * chunks]: parts of dA, ddelta_bias and dD
    bool packed;
    bool apart;  // requests of at most kLattnShort tokens have a kernel of their own: the walks pass them
    Requests req;
    int* failed;  // the device status word
};

enum WalkMode { WALK_ENDS, WALK_OUT, WALK_STATES, WALK_DSTATES, WALK_DENDS };

// The step of one token, from its delta: softplus(delta + bias), delta + bias, delta or 1.
__device__ __forceinline__ float lattn_step_from(const LattnParams& p, float x, int head) {
    if (p.delta == nullptr) return 1.f;
    if (p.bias != nullptr) x += __ldg(p.bias + head);
    return p.softplus ? softplus_f32(x) : x;
}
template <typename T>
__device__ __forceinline__ float lattn_step_of(const LattnParams& p, long long at, int head) {
    return lattn_step_from(p, p.delta != nullptr ? to_f32(static_cast<const T*>(p.delta)[at]) : 0.f, head);
}

// What a step changes by with its delta (0 without one).
template <typename T>
__device__ __forceinline__ float lattn_slope_of(const LattnParams& p, long long at, int head) {
    if (p.delta == nullptr) return 0.f;
    return p.softplus ? fast_sigmoid(to_f32(static_cast<const T*>(p.delta)[at]) + (p.bias != nullptr ? __ldg(p.bias + head) : 0.f)) : 1.f;
}

// What a CTA walks: one request, or the tokens between two, of a packed axis.
struct Piece {
    int begin, end;  // of the request
    int row;         // its cache row, or -1
    bool has;        // continues from its row
};
// The piece that token t lies in; s: the request to look from (find(t)), moved to it.  r
// answers for the request tables: Requests itself, or a copy of a part of them.
template <typename R>
__device__ __forceinline__ Piece piece_at(const R& r, int& s, int t) {
    Piece w;
    if (s < 0) {
        w.begin = 0; w.end = r.offset(0); w.row = -1; w.has = false;
        if (w.end > t) return w;
        s = 0;
    }
    while (s < r.requests && r.offset(s + 1) <= t) ++s;
    if (s >= r.requests) {
        w.begin = r.offset(r.requests); w.end = r.tokens; w.row = -1; w.has = false;
        return w;
    }
    w.begin = r.offset(s); w.end = r.offset(s + 1);
    w.row = r.slot(s);
    w.has = w.row >= 0 && r.continues(s);
    if (w.row < 0) w.row = -1;
    return w;
}

// Where part w of a packed axis begins: at w * span, or at the end of a request that lies within a
// quarter of a part: what begins with a request needs no states from before.
__device__ __forceinline__ int part_begin(const LattnParams& p, int w) {
    const int t = w * p.span;
    if (w == 0 || t >= p.L) return w == 0 ? 0 : p.L;
    int r = p.req.find(t);
    const Piece x = piece_at(p.req, r, t);
    const int before = t - x.begin, behind = x.end - t;
    if (min(before, behind) > p.span / 4 || min(before, behind) < 0) return t;  // (below zero: offsets that do not ascend)
    return before <= behind ? x.begin : x.end;
}
// the part that token t lies in
__device__ __forceinline__ int part_of(const LattnParams& p, int t) {
    const int w = t / p.span;
    return t < part_begin(p, w) ? w - 1 : t >= part_begin(p, w + 1) ? w + 1 : w;
}

// The next piece that a walk takes, from token t on: short requests that have a kernel of their
// own are passed, 32 at a time by a whole warp.  t moves to the piece; false: none before `to`.
template <typename R>
__device__ __forceinline__ bool next_piece(const R& r, bool apart, int& s, int& t, int to, Piece& w) {
    while (t < to) {
        w = piece_at(r, s, t);
        if (!apart || s < 0 || s >= r.requests || w.end - w.begin > kLattnShort) return true;
        const int lane = threadIdx.x & 31;
        int at = s + 1;
        for (;;) {
            const int i = at + lane;
            const unsigned stop = __ballot_sync(0xffffffffu, i >= r.requests || r.offset(i + 1) - r.offset(i) > kLattnShort);
            if (stop != 0u) {
                at += __ffs(stop) - 1;
                break;
            }
            at += 32;
        }
        s = at < r.requests ? at : r.requests;
        const int begin = r.offset(s);
        t = begin > t ? begin : w.end > t ? w.end : t + 1;  // (forward, whatever the table holds)
    }
    return false;
}

cudaError_t lattn_short_launch(const LattnParams& p, int dtype, cudaStream_t st);
// fp32, and bf16 gradients of very few tokens, on the FP32 units (lattn_simt.cuh)
cudaError_t lattn_walk_launch(const LattnParams& p, cudaStream_t st);
cudaError_t lattn_grad_launch(const LattnParams& p, int dtype, cudaStream_t st);
// sums of parts, whichever kernels they are of
cudaError_t lattn_parts_launch(const LattnParams& p, int dtype, cudaStream_t st);
cudaError_t lattn_heads_launch(const LattnParams& p, float* dA, float* dbias, float* dD, cudaStream_t st);
// bf16 on the tensor cores (lattn_tc.cuh)
cudaError_t lattn_tc_walk_launch(const LattnParams& p, cudaStream_t st);
cudaError_t lattn_tc_grad_launch(const LattnParams& p, cudaStream_t st);
int lattn_tc_grad_copies(const LattnParams& p);  // copies of inputs that it launches first
bool lattn_tc_copies(const LattnParams& p);  // whether its calls copy queries or keys first

}  // namespace sscan
