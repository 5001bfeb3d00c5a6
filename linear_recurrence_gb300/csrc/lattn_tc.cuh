// Linear attention with a decay for each head on the tensor cores, bf16 inputs
// (formulas: lattn.cuh): the walk over the chunks.
//
// A CTA walks the chunks of 128 tokens of one tile of 64 value channels of a
// head.  Inputs lie along time, so a chunk of a channel is a row of 128 values; every
// product takes the same tiles, summed along the rows or across them (tc_utils.cuh):
//
//   QK [t, s]    = q_t . k_s                      q across, k across      (all of a chunk's pairs)
//   OI [t, p]    = S q_t                          q across, state across
//   SD [n, p]    = sum_s k_s (weight_s v_s)       k along, weighted v along
//   O  [t, p]    = D v_t + sum_s P_ts v_s         D and P in tensor memory, v along
//
// with P_ts = scale * E_ts dt_s (q_t . k_s) formed in registers from QK and written over it.  D is
// an fp32 weight: what bf16 holds of it is a diagonal operand of its own, written once, and the rest joins P's
// diagonal (all of D in P would keep 8 bits: outputs off by 2.3e-3 where this leaves 1.7e-3 to 1.9e-3).
// The state lives in the registers of the threads that read SD, in fp32.  Rounded to bf16 are P and the state as operands, one factor of each of
// the two sums that make o (which is bf16 itself), never both factors of one (a second term of P brings
// o to the 1.65e-3 of its own rounding, and 65536 tokens from 366 to 405 us: its code
// crowds the other roles' out of the instruction cache); the weighted
// v is taken in three terms of bf16, all 24 bits of it, because states are fp32.
//
// Warps take roles: 8 form P, outputs and states; 1 brings queries and keys in by TMA
// and forms the steps; 6 bring values in and weight them; 1 issues the products.  TMA
// needs rows that begin on 16 bytes: queries and keys whose rows do not (a packed batch of
// odd length) are copied once to rows that do; chunks begin on multiples of 8 tokens, a
// request's first chunk with up to 7 tokens of the request before it masked.  Values pass
// through registers, to be weighted, and are shifted into place there.
//
// Measured: 4 x 2048 tokens x 32 heads of 64 x 128, forward 49 us, a walk without outputs 36 us
// (3.1 us and 2.3 us a chunk of a CTA); 65536 tokens x 24 heads of 64 x 64, six parts of time, 240 us
// after 132 us for the states before them; 8209 tokens x 80 heads in 24 requests, five parts, 200 us
// after 12 to 22 us.  The tensor pipe is busy for 19 to 30% of that time, the issue slots for 38 to 52%, DRAM
// for 10 to 20%: a chunk is a chain of products, tensor memory read into registers, arithmetic there, and the next
// products, one CTA an SM (shared memory holds one), and the chain's latency bounds it.  What overlaps by now:
// the scores of the next chunk, the weighting of its values, and the outputs of the chunk before.  20 warps, with scores and states
// apart on 80 to 144 registers, took 519 us where 16 take 377: fewer registers made the chain longer.
#pragma once

#include <cuda.h>

#include "lattn.cuh"
#include "piece_loads.cuh"
#include "tc_utils.cuh"

namespace sscan {

static_assert(kTcChunk == kTcTokens, "a row of a tile holds a chunk");
// 8 warps compute, 1 brings queries, keys and steps, 6 bring values, 1 issues
// products: 16 leave 128 registers a thread, so that nothing spills.
constexpr int kTcFront = 8;       // the warp of queries, keys and steps
constexpr int kTcProducers = 6;   // the warps after it
constexpr int kTcWarps = 10 + kTcProducers;
constexpr int kTcThreads = kTcWarps * 32;

struct TcMaps {
    CUtensorMap q, k;
};

// The three terms of bf16 that make up 8 fp32 values: 8 bits each, the first two
// cut off, so that what remains is exact and the third holds all of it.
__device__ __forceinline__ void split3(const float (&f)[8], uint4 (&t)[3]) {
    float r[8];
    unsigned* w0 = &t[0].x;
    unsigned* w1 = &t[1].x;
    unsigned* w2 = &t[2].x;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = f[i] - __uint_as_float(__float_as_uint(f[i]) & 0xffff0000u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w0[i] = __byte_perm(__float_as_uint(f[2 * i]), __float_as_uint(f[2 * i + 1]), 0x7632);
        w1[i] = __byte_perm(__float_as_uint(r[2 * i]), __float_as_uint(r[2 * i + 1]), 0x7632);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] -= __uint_as_float(__float_as_uint(r[i]) & 0xffff0000u);
#pragma unroll
    for (int i = 0; i < 4; ++i) w2[i] = __byte_perm(__float_as_uint(r[2 * i]), __float_as_uint(r[2 * i + 1]), 0x7632);
}

// (Loops below are kept short, and calls inline: the roles' loops run side by side, and with
// all of them unrolled they did not fit the instruction cache together: warps waited for
// instructions 7 of 12.6 cycles an issue; 65536 tokens 585 us, then 450.)

// The chunks that a CTA walks, in order: those of each piece of a packed axis, or of
// one sequence.  APART: short requests have a kernel of their own.  (A kernel of its own: the
// code that passes them, in every role, cost walks without them 17 of 235 us.)
template <bool APART>
struct ChunkWalk {
    const LattnParams& p;
    Piece piece;
    int request, at, stop;  // stop: end of this piece in [.., to)
    int to;
    bool fresh;             // the next chunk begins a piece
    __device__ __forceinline__ ChunkWalk(const LattnParams& params, int from, int until) : p(params), at(from), to(until) {
        fresh = true;
        stop = from;
        request = p.packed && from < until ? p.req.find(from) : 0;
        piece.begin = 0; piece.end = p.L; piece.row = -1; piece.has = false;
    }
    // the next chunk: tokens [base + lead, base + lead + len), base a multiple of 8; false at the end
    __device__ __forceinline__ bool next(int& base, int& lead, int& len, bool& ends) {
        if (at >= to) return false;
        if (fresh) {
            if (APART) {
                if (!next_piece(p.req, true, request, at, to, piece)) return false;
            } else if (p.packed) {
                piece = piece_at(p.req, request, at);
            }
            stop = min(piece.end, to);
        }
        base = at & ~7;
        lead = at & 7;
        len = min(kTcChunk - lead, stop - at);
        at += len;
        ends = at >= stop;
        fresh = ends;
        return true;
    }
};

struct alignas(16) TcSteps {
    float run[kTcChunk];   // A log2(e) T
    float col[kTcChunk];   // scale * dt
    float row[kTcChunk];   // scale * e^(A T)
    float tail[kTcChunk];  // dt e^(A R), or scale * e^(A T) in the gradients' walk
    float decay, total;    // e^(A T_end), T_end
};

// Rows of q and k that TMA cannot take, copied to rows of `to_stride` values (a
// multiple of 8): 8 values a thread.
struct TcCopy {
    const bf16* from[2];
    bf16* to[2];
    long long batch_stride[2], row_stride[2], rows[2];  // rows of a batch
    long long to_stride;
    int batch, L;
};
__global__ void __launch_bounds__(256) lattn_tc_copy(const TcCopy c) {
    const int which = blockIdx.z;
    if (c.from[which] == nullptr) return;
    const bf16* lo = c.from[which];
    const bf16* hi = lo + (c.batch - 1) * c.batch_stride[which] + (c.rows[which] - 1) * c.row_stride[which] + c.L;
    const int t = (blockIdx.x * 256 + threadIdx.x) * 8, n = min(8, c.L - t);
    if (n <= 0) return;
    const long long rows = c.rows[which];
    for (long long r0 = (long long)blockIdx.y * 4; r0 < c.batch * rows; r0 += (long long)gridDim.y * 4) {
        // (one division for four rows: with one a row, twice, 2048 rows of 8209 values took 25 us)
        const long long b0 = c.batch == 1 ? 0 : r0 / rows;
        long long b = b0, r = r0 - b0 * rows;
        const bf16* from[4];
        Piece8 x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool in = b < c.batch;
            from[j] = in ? lo + b * c.batch_stride[which] + r * c.row_stride[which] + t : nullptr;
            piece_load(x[j], in ? from[j] : lo, in ? n : 0, lo, hi);
            if (++r == rows) {
                r = 0;
                ++b;
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (from[j] == nullptr) break;
            *reinterpret_cast<uint4*>(c.to[which] + (r0 + j) * c.to_stride + t) = piece_take(x[j], from[j], n, lo, hi);
        }
    }
}

template <int KD>
struct TcWalkSmem {
    static constexpr unsigned tile = KD * 256;
    static constexpr unsigned q = 0, k = 2 * tile, v = 4 * tile, vt = v + 16384, s = vt + 3 * 16384, steps = s + KD * 128;
    static constexpr unsigned bytes = steps + 4 * sizeof(TcSteps) + 1024;  // and room to begin on 1024 bytes
    // without outputs: keys and weighted values twice, and both terms of a state
    static constexpr unsigned few_image = 2 * tile + 6 * 16384, few_steps = few_image + KD * 256, few_bytes = few_steps + 4 * sizeof(TcSteps) + 1024;
};

struct TcBars {
    uint64_t full_qk[2], full_vt[2], full_v;  // tiles -> issuer and producers
    // products -> compute warps and producers; with the first two the issuer itself
    // arrives too, which passes on the steps that it has seen written
    uint64_t done_qk, done_st[2], done_o;
    uint64_t ready_p, ready_s[2], free_o;  // compute warps -> issuer
    uint64_t last;                      // all products
};

// A wait on a barrier, of a limited number of tries (each of which the hardware
// suspends for a while: seconds in all).  One that gives up marks the CTA: no later
// wait lasts, the walk runs out with meaningless outputs and the status word says so.
constexpr int kTcTries = 1 << 18;
__device__ __forceinline__ void tc_wait(uint64_t* bar, unsigned parity, volatile int* failed, int* status) {
#pragma unroll 1
    for (int i = 0; !mbar_try_wait(bar, parity); ++i) {
        if (*failed) break;
        if (i == kTcTries) {
            *failed = 1;
            *status = SSCAN_ERR_TIMEOUT;
        }
    }
    __syncwarp();  // what follows is for whole warps
}

template <int KD, int MODE, bool APART>
__global__ void __launch_bounds__(kTcThreads, 1) lattn_tc_walk(const __grid_constant__ LattnParams p, const __grid_constant__ TcMaps maps) {
    constexpr bool OUT = MODE == WALK_OUT, REV = MODE == WALK_DSTATES || MODE == WALK_DENDS;
    constexpr bool END = MODE == WALK_ENDS || MODE == WALK_DENDS, KEEP = MODE == WALK_STATES || MODE == WALK_DSTATES;
    using M = TcWalkSmem<KD>;
    extern __shared__ char raw[];
    char* smem = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
    __shared__ TcBars bar;
    __shared__ unsigned tmem_at;
    __shared__ int failed;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    char *qs = smem + M::q, *ks = smem + (OUT ? M::k : 0), *vs = smem + M::v, *vt = smem + (OUT ? M::vt : 2 * M::tile), *ss = smem + M::s;
    char* im = smem + M::few_image;
    TcSteps* steps = reinterpret_cast<TcSteps*>(smem + (OUT ? M::steps : M::few_steps));
    const int tile = blockIdx.x, head = tile / p.vtiles, v0 = (tile % p.vtiles) * kValueTile;
    const int w = blockIdx.y, b = blockIdx.z;
    const int group = head / (p.heads / p.groups), pv = min(kValueTile, p.P - v0);
    const float rate = p.A[head] * kLog2e;
    const long long tiles = (long long)p.heads * p.vtiles;
    const long long dim = (long long)p.heads * p.P, row0 = (long long)head * p.P + v0;
    constexpr unsigned kColumns = OUT ? 512 : 128;
    // Without outputs the first 4 warps bring values too, and the 4 after them keep the whole state.
    constexpr int kFirst = OUT ? 0 : 4, kValueWarps = kTcProducers + kFirst;
    constexpr int SC = OUT ? 32 : 64;  // value channels of a thread's part of the state
    // columns: QK 128 and over them P (half 64 h of its tokens from column 64 h on), D 64, SD 64, OI and O twice 64 each
    constexpr int d_at = 128, oi_at = 256, o_at = 384, sd_at = OUT ? 192 : 0;

    // Every kernel of a call waits here for the one before it, whose last CTAs let it begin.  (Let in by its
    // first ones, it held their SMs' shared memory up: no faster.)
    griddep_wait();
    // what this CTA walks
    int from = w * p.span, to = min(p.L, from + p.span);
    if (REV) {
        const int whole = (p.L + kTcChunk - 1) / kTcChunk * kTcChunk;
        from = max(0, whole - (w + 1) * p.span);
        to = min(p.L, whole - w * p.span);
    }
    if (p.packed && p.pieces > 1) {
        from = part_begin(p, w);
        to = part_begin(p, w + 1);
    }
    const int begin = from;
    Piece cross;  // the request that crosses the end of this part of time (first pass)
    cross.begin = 0; cross.end = p.L; cross.row = -1; cross.has = false;
    if (p.packed && MODE == WALK_ENDS) {
        int r = p.req.find(to - 1);
        cross = piece_at(p.req, r, to - 1);
        if (cross.end <= to || (APART && r >= 0 && r < p.req.requests && cross.end - cross.begin <= kLattnShort)) return;
        from = max(from, cross.begin);
    }

    if (warp == kTcWarps - 1) tc_alloc(&tmem_at, kColumns);
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.full_qk[i], 2);
            mbar_init(&bar.full_vt[i], kValueWarps);
            mbar_init(&bar.done_st[i], 2);
            mbar_init(&bar.ready_s[i], 8 - kFirst);
        }
        mbar_init(&bar.full_v, kTcProducers);
        mbar_init(&bar.done_qk, 2);
        mbar_init(&bar.done_o, 1);
        mbar_init(&bar.last, 1);
        mbar_init(&bar.ready_p, 8);
        mbar_init(&bar.free_o, 8);
        mbar_fence_init();
        failed = 0;
    }
    // rows that no channel fills stay zero
    {
        const int rows = OUT ? 4 * KD + 64 + 3 * 64 : 2 * KD + 6 * 64;
        for (int i = tid; i < rows * 16; i += kTcThreads) reinterpret_cast<uint4*>(smem)[i] = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const unsigned tm = tmem_at;
    auto wait = [&](uint64_t* x, unsigned parity) { tc_wait(x, parity, &failed, p.failed); };
    int t0, lead, len;  // a chunk's tile begins at token t0, its tokens at t0 + lead
    bool ends;
    // chunks of the gradients' walk run backwards: where the one at `at` really lies
    auto reversed = [&](int at) { return REV ? from + (to - 1 - at) / kTcChunk * kTcChunk : at; };

    if (warp >= kFirst && warp < 8) {
        // ---- P, outputs and states --------------------------------------------------
        const int g = OUT ? warp >> 2 : 0, r = (warp & 3) * 32 + lane;  // row of every accumulator, and which half of its columns
        const unsigned mine = tm + ((unsigned)((warp & 3) * 32) << 16);
        // D in two parts: what bf16 holds of it stands on the diagonal of an operand of its own, the rest joins P
        const float D = OUT && p.D != nullptr ? p.D[head] : 0.f, D1 = __bfloat162float(__float2bfloat16_rn(D));
        const float skip = fabsf(D1) <= 3.4e38f ? D - D1 : 0.f;
        float s[SC];  // state of key channel r, value channels 32 g ..
        float total = 0.f;
        const long long tile_size = (long long)kValueTile * KD;
        auto piece_tile = [&](float* base, int piece) { return base + (((long long)piece * p.batch + b) * tiles + tile) * tile_size; };
        // states lie [value channel][key channel]: rows of N in a cache, of KD in scratch
        auto get = [&](const float* from_, int stride, int channels, int keys) {
#pragma unroll
            for (int j = 0; j < SC; ++j) s[j] = r < keys && 32 * g + j < channels ? from_[(32 * g + j) * stride + r] : 0.f;
        };
        auto join = [&](const float* from_, float decay) {  // eight loads at a time: no more fit in registers beside the state
            if (r >= KD) return;
#pragma unroll
            for (int j = 0; j < SC; j += 8) {
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = from_[(32 * g + j + e) * KD + r];
#pragma unroll
                for (int e = 0; e < 8; ++e) s[j + e] = fmaf(s[j + e], decay, x[e]);
            }
        };
        auto put = [&](float* to_, int stride, int channels, int keys) {
#pragma unroll
            for (int j = 0; j < SC; ++j)
                if (r < keys && 32 * g + j < channels) to_[(32 * g + j) * stride + r] = s[j];
        };
        // the state as an operand: rows of 64 value channels in bf16
        auto publish = [&](int i) {
            if (OUT && r < KD) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    *reinterpret_cast<uint4*>(ss + tile_piece(r, 4 * g + q, KD)) =
                        make_uint4(pack_bf16(s[8 * q], s[8 * q + 1]), pack_bf16(s[8 * q + 2], s[8 * q + 3]),
                                   pack_bf16(s[8 * q + 4], s[8 * q + 5]), pack_bf16(s[8 * q + 6], s[8 * q + 7]));
            }
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.ready_s[i & 1]);
        };
        // The state that a piece begins with: a cache's or initial row, what was put aside, or
        // the states behind the parts of time since its request began, joined in order.
        auto begin_piece = [&](const ChunkWalk<APART>& walk, int t) {
            const float* row = nullptr;
            int first = w;  // of the parts to join
            bool beside = false, keep = false;
            if (!p.packed) {
                row = w == 0 ? (REV ? p.ds_in : p.s_in) : nullptr;
                if (row != nullptr) row += b * dim * p.N;
                if (!END) first = 0;
            } else if (MODE == WALK_ENDS) {
                keep = cross.begin >= begin;
                if (keep && cross.has) row = p.s_in + cross.row * dim * p.N;
            } else if (walk.piece.begin < from && t == from) {
                first = part_of(p, walk.piece.begin);
            } else if (walk.piece.end > to && p.pieces > 1) {
                beside = true;
            } else if (walk.piece.has) {
                row = p.s_in + walk.piece.row * dim * p.N;
            }
#pragma unroll
            for (int j = 0; j < SC; ++j) s[j] = 0.f;
            if (beside) row = piece_tile(p.aside, w);
            else if (first < w) row = piece_tile(p.ends, first);
            else if (row != nullptr) row += row0 * p.N;
            const bool scratch = beside || first < w;
            if (row != nullptr) get(row, scratch ? KD : p.N, scratch ? 64 : pv, scratch ? KD : p.N);
#pragma unroll 1
            for (int i = first + 1; i < w; ++i)
                join(piece_tile(p.ends, i), ex2(rate * p.sums[((long long)i * p.batch + b) * p.heads + head]));
            if (keep) put(piece_tile(p.aside, w), KD, 64, KD);
        };
        // states of empty requests: a row that does not continue starts from zeros
        if (p.packed && MODE == WALK_OUT && w == 0) {
            if (tile == 0 && warp == 0) p.req.check(lane, 32);
            for (int i = 0; !APART && i < p.req.requests; ++i) {
                if (p.req.offset(i + 1) > p.req.offset(i)) continue;
                const int row = p.req.slot(i);
                if (row < 0 || p.req.continues(i)) continue;
                float* to_ = p.s_out + (row * dim + row0) * p.N;
                for (int j = tid; j < pv * p.N; j += 256) to_[j] = 0.f;
            }
        }
        // the outputs of chunk i, while the products of the next are under way
        int out_at = 0, out_lead = 0, out_end = 0, last_i = -1;
        const bool even = p.L % 2 == 0 && (reinterpret_cast<uintptr_t>(p.o) & 3u) == 0;
        auto output = [&](int i) {
            const float f = steps[i & 3].row[r];
            bf16* out = static_cast<bf16*>(p.o) + (b * dim + row0 + 32 * g) * p.L + out_at + r;
            const bool pairs = even && out_lead == 0 && out_end == kTcChunk;
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                float o[16], oi[16];
                tc_load16(mine + o_at + (i & 1) * 64 + 32 * g + 16 * h, o);
                tc_load16(mine + oi_at + (i & 1) * 64 + 32 * g + 16 * h, oi);
                tc_wait_loads(o);
                tc_wait_loads(oi);
                if (h == 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.free_o);
                }
                const int d0 = 32 * g + 16 * h;
                unsigned y[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] = pack_bf16(fmaf(oi[2 * j], f, o[2 * j]), fmaf(oi[2 * j + 1], f, o[2 * j + 1]));
                if (pairs) {  // two tokens at once: the even lane of a pair stores one channel, the odd one the next
                    bf16* to_ = out + (16 * h + (lane & 1)) * (long long)p.L - (lane & 1);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const unsigned other = __shfl_xor_sync(0xffffffffu, y[j], 1);
                        const unsigned two = lane & 1 ? __byte_perm(other, y[j], 0x7632) : __byte_perm(y[j], other, 0x5410);
                        if (d0 + 2 * j + (lane & 1) < pv) *reinterpret_cast<unsigned*>(to_) = two;
                        to_ += 2ll * p.L;
                    }
                } else if (r >= out_lead && r < out_end) {
                    unsigned short* to_ = reinterpret_cast<unsigned short*>(out) + 16 * h * (long long)p.L;
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        if (d0 + j < pv) *to_ = (unsigned short)(y[j >> 1] >> (16 * (j & 1)));
                        to_ += p.L;
                    }
                }
            }
        };
        if (OUT) {
            const unsigned mark = __float_as_uint(D1) >> ((r & 1) ? 0 : 16);
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                const int c0 = 32 * g + 8 * h;
                unsigned x[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = c0 + j == r >> 1 ? mark : 0u;
                tc_store8(mine + d_at + c0, x);
            }
            tc_wait_stores();
        }
        ChunkWalk<APART> walk(p, from, to);
        bool more = walk.next(t0, lead, len, ends);
        if (more) {
            begin_piece(walk, t0 + lead);
            publish(0);
        }
        for (int i = 0; more; ++i) {
            const TcSteps& st = steps[i & 3];
            if (KEEP) {
                // both terms of the state before (behind) this chunk, as an operand's image: laid out in shared
                // memory and sent off in one piece
                if (warp == kFirst && lane == 0) bulk_store_wait();
                asm volatile("bar.sync 1, 128;\n" ::: "memory");
                if (r < KD) {
#pragma unroll
                    for (int q = 0; q < SC / 8; ++q) {
                        uint4 hi, lo;
                        unsigned* h = &hi.x;
                        unsigned* l = &lo.x;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float x = s[8 * q + 2 * e], y = s[8 * q + 2 * e + 1];
                            h[e] = pack_bf16(x, y);
                            l[e] = pack_bf16(x - __uint_as_float(h[e] << 16), y - __uint_as_float(h[e] & 0xffff0000u));
                        }
                        *reinterpret_cast<uint4*>(im + tile_piece(r, q, KD)) = hi;
                        *reinterpret_cast<uint4*>(im + KD * 128 + tile_piece(r, q, KD)) = lo;
                    }
                }
                fence_proxy_async_smem();
                asm volatile("bar.sync 1, 128;\n" ::: "memory");
                if (warp == kFirst && lane == 0)
                    bulk_store(reinterpret_cast<char*>(REV ? p.dends : p.starts) +
                                   (((long long)b * tiles + tile) * p.chunks + reversed(t0) / kTcChunk) * tile_size * 4,
                               im, KD * 256);
            }
            if (OUT) {
                wait(&bar.done_qk, i & 1);  // (and with it the products of the chunk before)
                tc_fence_after();
                const float run = st.run[r];
#pragma unroll 1
                for (int h = 0; h < 4; ++h) {
                    const int c0 = 64 * g + 16 * h, behind = c0 - (warp & 3) * 32;  // columns from which token of the warp on
                    unsigned x[8];
                    if (behind > 31) {  // all of these tokens come later
#pragma unroll
                        for (int j = 0; j < 8; ++j) x[j] = 0u;
                    } else {
                        float f[16];
                        tc_load16(mine + c0, f);
                        tc_wait_loads(f);
#pragma unroll
                        for (int j = 0; j < 16; j += 4) {
                            const float4 c = *reinterpret_cast<const float4*>(&st.run[c0 + j]);
                            const float4 d = *reinterpret_cast<const float4*>(&st.col[c0 + j]);
                            f[j] *= ex2(run - c.x) * d.x;
                            f[j + 1] *= ex2(run - c.y) * d.y;
                            f[j + 2] *= ex2(run - c.z) * d.z;
                            f[j + 3] *= ex2(run - c.w) * d.w;
                        }
                        if (c0 == 0 && lead > 0) {  // tokens of the request before
#pragma unroll
                            for (int j = 0; j < 8; ++j) f[j] = j < lead ? 0.f : f[j];
                        }
                        if (behind >= 0) {
#pragma unroll
                            for (int j = 0; j < 16; ++j) f[j] = behind + j < lane ? f[j] : behind + j == lane ? f[j] + skip : 0.f;
                        }
#pragma unroll
                        for (int j = 0; j < 8; ++j) x[j] = pack_bf16(f[2 * j], f[2 * j + 1]);
                    }
                    tc_store8(mine + (c0 & 64) + ((c0 & 63) >> 1), x);  // where this thread's scores were
                }
                tc_wait_stores();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.ready_p);
            }
            // the state behind this chunk; what comes next is looked up before it is waited for
            const int c0 = t0, clead = lead, cend = lead + len;
            const bool cends = ends;
            // where the state goes after the last chunk of a piece
            float* last = nullptr;
            if (END) {
                last = piece_tile(p.ends, w);
            } else if (!p.packed) {
                last = REV ? p.ds_out : p.s_out;
                last = w == p.pieces - 1 && last != nullptr ? last + (b * dim + row0) * p.N : nullptr;
            } else if (walk.piece.end <= to && walk.piece.row >= 0) {
                last = p.s_out + (walk.piece.row * dim + row0) * p.N;
            }
            more = walk.next(t0, lead, len, ends);
            if (cends && more && p.packed && OUT && walk.piece.has) {  // the next request's state, on its way to the L2
                const long long line = (long long)tid * 128;
                if (line < (long long)pv * p.N * 4)
                    asm volatile("prefetch.global.L2 [%0];\n" ::"l"(reinterpret_cast<const char*>(p.s_in + (walk.piece.row * dim + row0) * p.N) + line));
            }
            wait(&bar.done_st[i & 1], (i >> 1) & 1);
            tc_fence_after();
            {
                const float decay = st.decay;
                total += st.total;
#pragma unroll
                for (int h = 0; h < SC / 16; ++h) {
                    float d[16];
                    tc_load16(mine + sd_at + (OUT ? 0 : (i & 1) * 64) + 32 * g + 16 * h, d);
                    tc_wait_loads(d);
#pragma unroll
                    for (int j = 0; j < 16; ++j) s[16 * h + j] = fmaf(s[16 * h + j], decay, d[j]);
                }
            }
            if (cends) {
                if (END && warp == kFirst && lane == 0 && v0 == 0)
                    p.sums[((long long)w * p.batch + b) * p.heads + head] = total;
                if (last != nullptr) put(last, END ? KD : p.N, END ? 64 : pv, END ? KD : p.N);
                if (more) begin_piece(walk, t0 + lead);
            }
            if (more) publish(i + 1);
            if (OUT && i > 0) output(i - 1);
            out_at = c0; out_lead = clead; out_end = cend;
            last_i = i;
        }
        if (KEEP && warp == kFirst && lane == 0) bulk_store_wait();
        if (OUT && last_i >= 0) {
            wait(&bar.done_o, last_i & 1);
            tc_fence_after();
            output(last_i);
        }
    } else if (warp == kTcFront) {
        // ---- queries, keys and steps --------------------------------------------------
        ChunkWalk<APART> walk(p, from, to);
        const CUtensorMap* kmap = REV ? &maps.q : &maps.k;
        const long long rows = b * p.tb + head * p.td;
        int i = 0;
        for (; walk.next(t0, lead, len, ends); ++i) {
            const int t = reversed(t0), first = lead, last = REV ? min(kTcChunk, to - t) : lead + len;
            float x[4], up = 0.f, down;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = 4 * lane + j;
                x[j] = p.delta != nullptr && c >= first && c < last ? to_f32(static_cast<const bf16*>(p.delta)[rows + t + c]) : 0.f;
            }
            if (i >= 2) wait(&bar.done_st[i & 1], ((i - 2) >> 1) & 1);
            if (lane == 0) {
                mbar_arrive_expect_tx(&bar.full_qk[i & 1], (OUT ? 2 : 1) * M::tile);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (OUT) tma_load_4d(qs + (i & 1) * M::tile + h * KD * 128, &maps.q, t + 64 * h, 0, group, b, &bar.full_qk[i & 1]);
                    tma_load_4d(ks + (i & 1) * M::tile + h * KD * 128, kmap, t + 64 * h, 0, group, b, &bar.full_qk[i & 1]);
                }
            }
            __syncwarp();
            TcSteps& st = steps[i & 3];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = 4 * lane + j;
                x[j] = c >= first && c < last ? lattn_step_from(p, x[j], head) : 0.f;
                up += x[j];
            }
            down = up;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float u = __shfl_up_sync(0xffffffffu, up, o), d = __shfl_down_sync(0xffffffffu, down, o);
                if (lane >= o) up += u;
                if (lane + o < 32) down += d;
            }
            float before = __shfl_up_sync(0xffffffffu, up, 1), behind = __shfl_down_sync(0xffffffffu, down, 1);
            if (lane == 0) before = 0.f;
            if (lane == 31) behind = 0.f;
            const float all = __shfl_sync(0xffffffffu, up, 31);
            float run = before;
            // sums from the end, so that small ones near the end keep their bits
            const float rests[4] = {behind + (x[3] + x[2] + x[1]), behind + (x[3] + x[2]), behind + x[3], behind};
            float4 a, c, e, d;
            float* pa = &a.x;
            float* pc = &c.x;
            float* pe = &e.x;
            float* pd = &d.x;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                run += x[j];
                pa[j] = rate * run;
                pc[j] = p.scale * x[j];
                pe[j] = p.scale * ex2(rate * run);
                const bool mine = 4 * lane + j >= first && 4 * lane + j < last;
                pd[j] = !mine ? 0.f : REV ? pe[j] : x[j] * ex2(rate * rests[j]);
            }
            *reinterpret_cast<float4*>(&st.run[4 * lane]) = a;
            *reinterpret_cast<float4*>(&st.col[4 * lane]) = c;
            *reinterpret_cast<float4*>(&st.row[4 * lane]) = e;
            *reinterpret_cast<float4*>(&st.tail[4 * lane]) = d;
            if (lane == 0) {
                st.total = all;
                st.decay = ex2(rate * all);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.full_qk[i & 1]);
        }
        // no copy is in flight when the CTA ends, even after a wait that gave up
        for (int j = max(0, i - 2); j < i; ++j) mbar_wait_bounded(&bar.full_qk[j & 1], (j >> 1) & 1);
    } else if (warp != kTcWarps - 1) {
        // ---- values ----------------------------------------------------------------
        const int id = warp > kTcFront ? tid - 32 * (kTcFront + 1) : tid + 32 * kTcProducers;
        const bf16* v = static_cast<const bf16*>(REV ? p.dout : p.v);
        const long long vd = REV ? p.L : p.vd, vb = REV ? dim * p.L : p.vb;
        const bf16* v1 = v + (p.batch - 1) * vb + (dim - 1) * vd + p.L;  // what may be read ends here
        const bf16* vr = v + b * vb + row0 * vd;
        // a thread takes piece id % 16 (8 tokens) of rows id / 16, + kRows, ..
        const int piece = id & 15, row = id >> 4;
        constexpr int kRows = 2 * kValueWarps;  // rows that these warps fill at once, 16 threads a row
        constexpr int kBatch = (64 + kRows - 1) / kRows, kAhead = OUT ? 1 : 2;
        // kRows is 4 more than a multiple of 8: every other row's pieces swap halves
        static_assert(kRows % 8 == 4, "where a thread's pieces lie");
        const unsigned place = tile_piece(row, piece, 64);
        auto at = [&](char* tile_, int j) { return reinterpret_cast<uint4*>(tile_ + (place ^ ((j & 1) << 6)) + j * kRows * 128); };
        auto arrive = [&](uint64_t* x) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(x);
        };
        ChunkWalk<APART> walk(p, from, to);
        bool more = walk.next(t0, lead, len, ends);
        Piece8 y[kBatch];  // the next chunk's, on the way
        // of this thread's piece, [first, last) belong to the chunk
        auto last_of = [&]() { return min(8, max(0, (REV ? min(kTcChunk, to - reversed(t0)) : lead + len) - 8 * piece)); };
        // Whole chunks of rows on 16-byte boundaries need one vector a piece, whole chunks
        // whose vectors all lie inside the array two and a shift; what is left is looked at piece by piece.
        const bool aligned = vd % 8 == 0 && (reinterpret_cast<uintptr_t>(vr) & 15u) == 0;
        auto whole = [&]() {
            const int t = reversed(t0);
            return lead == 0 && (REV ? to - t >= kTcChunk : len == kTcChunk) &&
                   (aligned || (vr + t - v >= 8 && v1 - (vr + (pv - 1) * vd + t) >= kTcChunk + 8));
        };
        auto load = [&](bool easy) {
            const bf16* src = vr + row * vd + reversed(t0) + 8 * piece;
            const long long next = kRows * vd;
            if (easy && aligned) {
#pragma unroll
                for (int j = 0; j < kBatch; ++j)
                    if (row + j * kRows < pv) y[j].a = __ldg(reinterpret_cast<const uint4*>(src + j * next));
            } else if (easy) {
#pragma unroll
                for (int j = 0; j < kBatch; ++j)
                    if (row + j * kRows < pv) {
                        const uint4* base = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(src + j * next) & ~(uintptr_t)15);
                        y[j].a = __ldg(base);
                        y[j].b = __ldg(base + 1);
                    }
            } else {
                const int last = last_of();
#pragma unroll
                for (int j = 0; j < kBatch; ++j) piece_load(y[j], src + j * next, row + j * kRows < pv ? last : 0, v, v1);
            }
        };
        bool easy = more && whole();
        if (more) load(easy);
        for (int i = 0; more; ++i) {
            const int first = min(8, max(0, lead - 8 * piece)), last = last_of();
            const bool fix = p.packed && (lead > 0 || (lead + len < kTcChunk && t0 + lead + len < p.L)) && last - first < 8;
            uint4 x[kBatch];
            {
                const bf16* src = vr + row * vd + reversed(t0) + 8 * piece;
                const long long next = kRows * vd;
                if (easy && aligned) {
#pragma unroll
                    for (int j = 0; j < kBatch; ++j) x[j] = y[j].a;
                } else if (easy) {
#pragma unroll
                    for (int j = 0; j < kBatch; ++j) x[j] = piece_shift(y[j], phase8(src + j * next));
                } else {
#pragma unroll
                    for (int j = 0; j < kBatch; ++j) {
                        x[j] = piece_take(y[j], src + j * next, row + j * kRows < pv ? last : 0, v, v1);
                        x[j] = keep_values(x[j], first, last);
                    }
                }
            }
            more = walk.next(t0, lead, len, ends);
            easy = more && whole();
            if (more) load(easy);
            wait(&bar.full_qk[i & 1], (i >> 1) & 1);  // the steps' weights are written
            // without outputs there is room for two sets of weighted values
            char* to_ = vt + (OUT ? 0 : (i & 1) * 3 * 16384);
            if (i >= kAhead) wait(&bar.done_st[(i - kAhead) & 1], ((i - kAhead) >> 1) & 1);
            const float4 w0 = *reinterpret_cast<const float4*>(&steps[i & 3].tail[8 * piece]);
            const float4 w1 = *reinterpret_cast<const float4*>(&steps[i & 3].tail[8 * piece + 4]);
            const float wt[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
            // (a thread writes its pieces down and reads them back: a short loop instead of six
            // pieces by name in registers)
#pragma unroll
            for (int j = 0; j < kBatch; ++j)
                if (row + kRows * j < pv) *at(to_, j) = x[j];
#pragma unroll(OUT ? 1 : 4)
            for (int j = 0; row + kRows * j < pv; ++j) {
                float f[8];
                widen(*at(to_, j), f, (bf16*)nullptr);
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] *= wt[e];
                uint4 terms[3];
                split3(f, terms);
#pragma unroll
                for (int term = 0; term < 3; ++term) *at(to_ + term * 16384, j) = terms[term];
            }
            // keys of other requests in this chunk's tile: their products with weights of zero count,
            // so that they must not be infinities or NaN
            if (fix) {
                for (int c = row; c < p.N; c += kRows) {
                    uint4* k_at = reinterpret_cast<uint4*>(ks + (i & 1) * M::tile + tile_piece(c, piece, KD));
                    *k_at = keep_values(*k_at, first, last);
                }
            }
            arrive(&bar.full_vt[i & 1]);
            if (OUT) {
                if (i > 0) wait(&bar.done_o, (i - 1) & 1);
#pragma unroll
                for (int j = 0; j < kBatch; ++j)
                    if (row + kRows * j < pv) *at(vs, j) = x[j];
                arrive(&bar.full_v);
            }
        }
    } else {
        // ---- products -----------------------------------------------------------------
        // descriptors are formed once, a product's operands then lie at constant distances
        const int steps_n = (p.N + 15) / 16;
        const uint64_t q_across = desc_across(smem_addr(qs), KD, 0), k_across = desc_across(smem_addr(ks), KD, 0);
        const uint64_t s_across = desc_across(smem_addr(ss), KD, 0), k_along = desc_along(smem_addr(ks), KD, 0);
        const uint64_t v_along = desc_along(smem_addr(vs), 64, 0), t_along = desc_along(smem_addr(vt), 64, 0);
        auto qk = [&](int i) {
            wait(&bar.full_qk[i & 1], (i >> 1) & 1);
            tc_fence_after();
            if (tc_elect()) {
                const uint64_t buffer = (i & 1) * (M::tile >> 4);
#pragma unroll
                for (int j = 0; j < KD / 16; ++j)
                    if (j < steps_n) tc_mma(tm, q_across + buffer + 128 * j, k_across + buffer + 128 * j, tc_kind(128, 128, true, true), j > 0);
                tc_commit(&bar.done_qk);
                mbar_arrive(&bar.done_qk);
            }
            __syncwarp();
        };
        ChunkWalk<APART> walk(p, from, to);
        bool more = walk.next(t0, lead, len, ends);
        if (more && OUT) qk(0);
        for (int i = 0; more; ++i) {
            const uint64_t buffer = (i & 1) * (M::tile >> 4);
            if (!OUT) wait(&bar.full_qk[i & 1], (i >> 1) & 1);
            // with outputs the state before this chunk; else what frees the columns of the chunk before the last
            if (OUT) wait(&bar.ready_s[i & 1], (i >> 1) & 1);
            else if (i > 0) wait(&bar.ready_s[(i - 1) & 1], ((i - 1) >> 1) & 1);
            if (OUT) {
                if (i > 1) wait(&bar.free_o, i & 1);  // outputs of the chunk before the last are read
                tc_fence_after();
                if (tc_elect()) {
#pragma unroll
                    for (int j = 0; j < KD / 16; ++j)
                        if (j < steps_n)
                            tc_mma(tm + oi_at + (i & 1) * 64, q_across + buffer + 128 * j, s_across + 128 * j, tc_kind(128, 64, true, true), j > 0);
                }
                __syncwarp();
            }
            wait(&bar.full_vt[i & 1], (i >> 1) & 1);
            tc_fence_after();
            if (tc_elect()) {
#pragma unroll 1
                for (int term = 0; term < 3; ++term)
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        tc_mma(tm + sd_at + (OUT ? 0 : (i & 1) * 64), k_along + buffer + (j >> 2) * (KD * 8) + (j & 3) * 2,
                               t_along + (OUT ? 0 : (i & 1) * 3 * 1024) + term * 1024 + (j >> 2) * 512 + (j & 3) * 2, tc_kind(128, 64, false, false), term + j > 0);
                tc_commit(&bar.done_st[i & 1]);
                mbar_arrive(&bar.done_st[i & 1]);
            }
            __syncwarp();
            more = walk.next(t0, lead, len, ends);
            if (OUT) {
                wait(&bar.full_v, i & 1);
                tc_fence_after();
                if (tc_elect()) {  // D's products need no scores (an absent D is zero)
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        tc_mma_ts(tm + o_at + (i & 1) * 64, tm + d_at + 8 * j, v_along + (j >> 2) * 512 + (j & 3) * 2,
                                  tc_kind(128, 64, false, false), j > 0);
                }
                __syncwarp();
                wait(&bar.ready_p, i & 1);
                tc_fence_after();
                if (tc_elect()) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        tc_mma_ts(tm + o_at + (i & 1) * 64, tm + (j >> 2) * 64 + 8 * (j & 3), v_along + (j >> 2) * 512 + (j & 3) * 2,
                                  tc_kind(128, 64, false, false), true);
                    tc_commit(&bar.done_o);
                }
                __syncwarp();
                if (more) {
                    wait(&bar.done_o, i & 1);  // the next scores go where P lies
                    qk(i + 1);
                }
            }
        }
    }
    if (warp == kTcWarps - 1) {  // nothing is in flight when the tensor memory goes back, even after a wait that gave up
        if (tc_elect()) tc_commit(&bar.last);
        __syncwarp();
        mbar_wait_bounded(&bar.last, 0);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kTcWarps - 1) tc_free(tm, kColumns);
}

}  // namespace sscan
