// Gradients of linear attention with a decay for each head on the tensor cores,
// bf16 (formulas: lattn.cuh): one chunk of 128 tokens, for the heads that share a set of
// queries and keys, or a part of them.
//
// The states before all chunks and their gradients behind them come from two walks
// (lattn_tc.cuh), as tiles in two terms of bf16.  A CTA then goes through its heads' tiles of 64 value
// channels, and sums dq and dk over them in tensor memory, so that no two CTAs add to
// the same value.  Per tile, all operands being rows along time (or key channels):
//
//   QK [t, s]   q across, k across        G [t, s]    do across, v across
//   in registers: E_ts = e^(A (T_t - T_s)), F = scale E QK, H = scale E G dt_s, and the sums over
//   rows and columns of F G that the steps' gradients take
//   dq^T [n, t] k along, H along          + (S as rows of n) x (do times scale e^(A T_t))
//   dk^T [n, s] q along, H across         + (dS' as rows of n) x (v times dt_s e^(A R_s))
//   DF [s, p]   F across, do along        DI [s, p]   k across, dS' across (both terms)
//   U [t, p]    q across, S across (both terms)
//
// dv = dt (e^(A R) DI + DF) + D do, X = scale e^(A T) do . U, Y = e^(A R) v . DI.  dq and dk lie
// transposed so that a thread holds consecutive tokens of a channel.
//
// Rounded to bf16 are F, H, the scaled do and v, and S and dS' in dq and dk: one or two factors
// of sums that are rounded to bf16 themselves.  What the fp32 sums dA and ddelta_bias (and through
// them ddelta) are made of is not: QK and G are exact products summed in fp32, and U and DI take
// S and dS' in both terms (2^-16).
//
// Measured: 4 x 2048 tokens x 32 heads of 64 x 128 on one set of queries and keys, 135 us of the 271
// that forward and gradients take (128 CTAs of 16 tiles; 208 MB read, most of it states, 1.9 TB/s).  Issue slots are
// busy for 42%, the tensor pipe for 21%: a tile is two chains of products with registers' work between
// them.  The next tile's steps, states and values come while the tile before is worked on.
#pragma once

#include "lattn_tc.cuh"

namespace sscan {

struct TcGradMaps {
    CUtensorMap q, k, v, dout;
};

// 16 warps compute (with 8 a tile of value channels took 25,000 cycles: 13,800 of
// them in their registers' work, at about 6 cycles an instruction), 1 brings tiles, 1 issues products
constexpr int kGradCompute = 16;
constexpr int kGradWarps = kGradCompute + 2;
constexpr int kGradThreads = kGradWarps * 32;

struct alignas(16) TcGradSteps {
    float run[kTcChunk];   // A log2(e) T
    float low[kTcChunk];   // what its roundings left out
    float dt[kTcChunk];
    float pre[kTcChunk];   // scale * e^(A T)
    float rest[kTcChunk];  // e^(A R)
    float tail[kTcChunk];  // dt * e^(A R)
    float decay;           // e^(A T_end)
};

struct TcGradBars {
    uint64_t full_qk, full, full_s; // tiles of the chunk; a unit's do, v and steps, and its states
    uint64_t done1, done2, done3;   // products: scores; sums and states; the rest
    uint64_t scores_read, ready_ef, ready_scaled, freed;
};

template <int KD>
struct TcGradSmem {
    static constexpr unsigned tile = KD * 256;
    static constexpr unsigned q = 0, k = tile, v = 2 * tile, u = v + 16384;           // u: do
    static constexpr unsigned s = u + 16384, d = s + KD * 256;                        // states and their gradients, both terms
    static constexpr unsigned e = d + KD * 256, f = e + 32768, end = f + 32768;       // H and F; then the scaled tiles
    // H is zero for tokens t < 64 and s >= 64: no product reads it there, and the CTA's
    // steps and sums lie in that quarter
    static constexpr unsigned hole = e + 16384;
    static constexpr unsigned bytes = end + 1024;
};
struct TcGradHole {
    TcGradSteps st;
    float cols[4][kTcChunk], rows[2][kTcChunk], ys[2][kTcChunk], diag[kTcChunk];  // rows: with X
    float dots[kGradCompute], skips[kGradCompute], das[kGradCompute], dbs[kGradCompute];
};
static_assert(sizeof(TcGradHole) <= 8192, "a quarter of H");

// sums over a warp's lanes of 16 columns; lane l holds that of column l / 2
__device__ __forceinline__ float column_sums(float (&v)[16]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int n = 8; n > 0; n >>= 1) {
        const int m = 2 * n;
        const bool high = (lane & m) != 0;
#pragma unroll
        for (int j = 0; j < n; ++j) {
            const float give = high ? v[j] : v[j + n], keep = high ? v[j + n] : v[j];
            v[j] = keep + __shfl_xor_sync(0xffffffffu, give, m);
        }
    }
    return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 1);
}

template <int KD>
__global__ void __launch_bounds__(kGradThreads, 1) lattn_tc_grad(const __grid_constant__ LattnParams p, const __grid_constant__ TcGradMaps maps) {
    using M = TcGradSmem<KD>;
    extern __shared__ char raw[];
    char* smem = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
    __shared__ TcGradBars bar;
    TcGradHole& sums = *reinterpret_cast<TcGradHole*>(smem + M::hole);
    TcGradSteps& st = sums.st;
    __shared__ __align__(16) float slope[kTcChunk], slope_sum[kTcChunk], slope_low[kTcChunk];  // slopes, Z, and what its roundings left out
    __shared__ unsigned tmem_at;
    __shared__ int failed;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int t0 = blockIdx.x * kTcChunk, len = min(kTcChunk, p.L - t0), b = blockIdx.z;
    const int group = blockIdx.y / p.subsets, subset = blockIdx.y % p.subsets, per = p.heads / p.groups;
    const int h0 = group * per + (int)((long long)per * subset / p.subsets), h1 = group * per + (int)((long long)per * (subset + 1) / p.subsets);
    const int units = (h1 - h0) * p.vtiles;
    const long long tiles = (long long)p.heads * p.vtiles;
    auto image = [&](const float* base, int unit) {  // of the states of a unit's tile at this chunk
        return reinterpret_cast<const char*>(base) +
               (((long long)b * tiles + (long long)h0 * p.vtiles + unit) * p.chunks + blockIdx.x) * (KD * 256);
    };
    constexpr int dq_at = 0, dk_at = 128, qk_at = 256, g_at = 384;  // columns; after the scores:
    constexpr int df_at = 256, di_at = 320, u_at = 384;

    griddep_wait();
    if (warp == kGradCompute + 1) tc_alloc(&tmem_at, 512);
    if (tid == 0) {
        mbar_init(&bar.full_qk, 1);
        mbar_init(&bar.full, 2);
        mbar_init(&bar.full_s, 1);
        mbar_init(&bar.done1, 1);
        mbar_init(&bar.done2, 1);
        mbar_init(&bar.done3, 1);
        mbar_init(&bar.scores_read, kGradCompute);
        mbar_init(&bar.ready_ef, kGradCompute);
        mbar_init(&bar.ready_scaled, kGradCompute);
        mbar_init(&bar.freed, kGradCompute);
        mbar_fence_init();
        failed = 0;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const unsigned tm = tmem_at;
    auto wait = [&](uint64_t* x, unsigned parity) { tc_wait(x, parity, &failed, p.failed); };

    if (warp < kGradCompute) {
        // ---- scores, scaled tiles, outputs -------------------------------------------------
        const int g = warp >> 2, r = (warp & 3) * 32 + lane, block = (warp & 3) * 32;
        const unsigned mine = tm + ((unsigned)block << 16);
        float row = 0.f, x = 0.f, y = 0.f, dia = 0.f, dot = 0.f, skip_sum = 0.f, da = 0.f;
        auto arrive = [&](uint64_t* to) {
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(to);
        };
        for (int u = 0; u < units; ++u) {
            const int head = h0 + u / p.vtiles, vt = u % p.vtiles, v0 = vt * kValueTile, pv = min(kValueTile, p.P - v0);
            const float skip = p.D != nullptr ? __ldg(p.D + head) : 0.f;
            if (vt == 0) row = x = y = dia = dot = skip_sum = da = 0.f;
            wait(&bar.full, u & 1);
            wait(&bar.done1, u & 1);
            tc_fence_after();
            const float run = st.run[r], low = st.low[r];
            // two blocks of 16 columns, the second from the last: once it is read, the products that
            // take the scores' place may begin
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                const int c0 = 32 * g + 16 * h, behind = c0 - block;
                float s[16], gg[16];
                const bool later = behind > 31;  // all of these tokens come later
                if (!later) {
                    tc_load16(mine + qk_at + c0, s);
                    tc_load16(mine + g_at + c0, gg);
                    tc_wait_loads(s);
                    tc_wait_loads(gg);
                }
                if (h == 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.scores_read);
                }
                uint4* f_at = reinterpret_cast<uint4*>(smem + M::f + tile_piece(r, c0 >> 3, 128));
                uint4* e_at = reinterpret_cast<uint4*>(smem + M::e + tile_piece(r, c0 >> 3, 128));
                const int swap = ((c0 >> 3) ^ r) & 1 ? -1 : 1;  // where the next piece lies: the pieces of a row are permuted in pairs
                if (later) {
                    f_at[0] = f_at[swap] = make_uint4(0u, 0u, 0u, 0u);
                    if (c0 < 64 || block >= 64) e_at[0] = e_at[swap] = make_uint4(0u, 0u, 0u, 0u);
                    if (vt == 0 && (lane & 1) == 0) sums.cols[warp & 3][c0 + (lane >> 1)] = 0.f;
                    continue;
                }
                unsigned ef[8], ff[8];
#pragma unroll
                for (int j = 0; j < 16; j += 4) {
                    const float4 c = *reinterpret_cast<const float4*>(&st.run[c0 + j]);
                    const float4 l = *reinterpret_cast<const float4*>(&st.low[c0 + j]);
                    const float4 d = *reinterpret_cast<const float4*>(&st.dt[c0 + j]);
                    const float cr[4] = {c.x, c.y, c.z, c.w}, cl[4] = {l.x, l.y, l.z, l.w}, cd[4] = {d.x, d.y, d.z, d.w};
                    float hh[4], f[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int at = behind + j + i;  // column, as a token of the warp
                        const float time = (run - cr[i]) + (low - cl[i]), e = p.scale * ex2(time), gv = gg[j + i];
                        f[i] = e * s[j + i];
                        hh[i] = e * gv * cd[i];
                        float pair = f[i] * gv;
                        if (behind > -16) {  // on the diagonal
                            f[i] = at <= lane ? f[i] : 0.f;
                            hh[i] = at <= lane ? hh[i] : 0.f;
                            if (at == lane) {
                                dia += pair;
                                skip_sum += gv;
                            }
                            pair = at < lane ? pair : 0.f;
                        }
                        s[j + i] = pair;
                        const float weighted = pair * cd[i];
                        row += weighted;
                        da = fmaf(weighted, time, da);
                    }
                    ff[j / 2] = pack_bf16(f[0], f[1]);
                    ff[j / 2 + 1] = pack_bf16(f[2], f[3]);
                    ef[j / 2] = pack_bf16(hh[0], hh[1]);
                    ef[j / 2 + 1] = pack_bf16(hh[2], hh[3]);
                }
                f_at[0] = make_uint4(ff[0], ff[1], ff[2], ff[3]);
                f_at[swap] = make_uint4(ff[4], ff[5], ff[6], ff[7]);
                e_at[0] = make_uint4(ef[0], ef[1], ef[2], ef[3]);
                e_at[swap] = make_uint4(ef[4], ef[5], ef[6], ef[7]);
                const float sum = column_sums(s);
                if ((lane & 1) == 0) {
                    float* to = &sums.cols[warp & 3][c0 + (lane >> 1)];
                    *to = vt == 0 ? sum : *to + sum;
                }
            }
            arrive(&bar.ready_ef);
            // S . dS' while the products are under way
            wait(&bar.full_s, u & 1);
            {
                float sum = 0.f;
#pragma unroll 1
                for (int i = tid; i < KD * 8; i += 32 * kGradCompute) {
                    float a[8], c[8], e[8];
                    widen(*reinterpret_cast<const uint4*>(smem + M::s + i * 16), a, (bf16*)nullptr);
                    widen(*reinterpret_cast<const uint4*>(smem + M::s + KD * 128 + i * 16), e, (bf16*)nullptr);
#pragma unroll
                    for (int j = 0; j < 8; ++j) a[j] += e[j];
                    widen(*reinterpret_cast<const uint4*>(smem + M::d + i * 16), c, (bf16*)nullptr);
                    widen(*reinterpret_cast<const uint4*>(smem + M::d + KD * 128 + i * 16), e, (bf16*)nullptr);
#pragma unroll
                    for (int j = 0; j < 8; ++j) sum = fmaf(a[j], c[j] + e[j], sum);
                }
                dot = fmaf(st.decay, sum, dot);
            }
            wait(&bar.done2, u & 1);
            tc_fence_after();
            // do times scale e^(A T) and v times dt e^(A R), where H and F were: half of the warps each
            {
                const int which = warp >> 3, piece = tid & 15;
                const float* by = (which ? st.tail : st.pre) + 8 * piece;
                const float4 w0 = *reinterpret_cast<const float4*>(by), w1 = *reinterpret_cast<const float4*>(by + 4);
                const float wt[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
                const char* from = smem + (which ? M::v : M::u);
                char* to = smem + (which ? M::f : M::e);
#pragma unroll 2
                for (int c = (tid & 255) >> 4; c < 64; c += 16) {
                    const unsigned at = tile_piece(c, piece, 64);
                    float f[8];
                    widen(*reinterpret_cast<const uint4*>(from + at), f, (bf16*)nullptr);
#pragma unroll
                    for (int j = 0; j < 8; ++j) f[j] *= wt[j];
                    *reinterpret_cast<uint4*>(to + at) = narrow(f, (bf16*)nullptr);
                }
            }
            arrive(&bar.ready_scaled);
            // dv, X and Y: a thread has a token and 16 of the value channels
            {
                const float rest = st.rest[r], dt = st.dt[r];
                const int c0 = 16 * g;
                bf16* out = static_cast<bf16*>(p.dv) + ((long long)b * p.heads * p.P + (long long)head * p.P + v0 + c0) * p.L + t0 + r;
                float xs_ = 0.f, ys_ = 0.f;
                float df[16], di[16], uu[16];
                tc_load16(mine + df_at + c0, df);
                tc_load16(mine + di_at + c0, di);
                tc_load16(mine + u_at + c0, uu);
                tc_wait_loads(df);
                tc_wait_loads(di);
                tc_wait_loads(uu);
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const unsigned at = tile_piece(c0 + j, r >> 3, 64) + (r & 7) * 2;
                    const float dov = __uint_as_float((unsigned)*reinterpret_cast<const unsigned short*>(smem + M::u + at) << 16);
                    const float vv = __uint_as_float((unsigned)*reinterpret_cast<const unsigned short*>(smem + M::v + at) << 16);
                    xs_ = fmaf(uu[j], dov, xs_);
                    ys_ = fmaf(di[j], vv, ys_);
                    const float dv = fmaf(dt, fmaf(rest, di[j], df[j]), skip * dov);
                    if (r < len && c0 + j < pv) *out = __float2bfloat16_rn(dv);
                    out += p.L;
                }
                x = fmaf(st.pre[r], xs_, x);
                y = fmaf(rest, ys_, y);
            }
            if (vt == p.vtiles - 1) {
                // the head's sums: ddelta and parts of dA, ddelta_bias and dD
                if (g >= 2) {
                    sums.rows[g - 2][r] = row + x;
                    sums.ys[g - 2][r] = y;
                }
                if ((r >> 5) == g) sums.diag[r] = dia;
                // dA's terms by the time that they span, here times the rate
                const float end = st.run[kTcChunk - 1];
                da = fmaf(x, run, fmaf(st.dt[r] * y, (end - run) + (st.low[kTcChunk - 1] - low), fmaf(dot, end, da)));
                // ddelta_bias: Z_t - Z_s of a pair as Z_t - Z of the middle of its 32 columns, with the row's sum over these, less
                // Z_s - the same, with the column's: what cancels spans 16 tokens (blocks of 16 columns took 7 us more
                // of 135, pair by pair 15)
                const float z = slope_sum[r], z_end = slope_sum[kTcChunk - 1];
                float db = row * ((z - slope_sum[32 * g + 16]) + (slope_low[r] - slope_low[32 * g + 16]));
                const int mid = (r & ~31) + 16;  // and a quarter of token r's column
                db = fmaf(-(st.dt[r] * sums.cols[g][r]), (z - slope_sum[mid]) + (slope_low[r] - slope_low[mid]), db);
                db = fmaf(x, z, fmaf(st.dt[r] * y, z_end - z, fmaf(dot, z_end, db)));
                const float all_dot = warp_sum(dot), all_skip = warp_sum(skip_sum), all_da = warp_sum(da), all_db = warp_sum(db);
                if (lane == 0) {
                    sums.dots[warp] = all_dot;
                    sums.skips[warp] = all_skip;
                    sums.das[warp] = all_da;
                    sums.dbs[warp] = all_db;
                }
                asm volatile("bar.sync 1, %0;\n" ::"n"(32 * kGradCompute) : "memory");
                if (g < 2) {
                    sums.rows[g][r] += row + x;
                    sums.ys[g][r] += y;
                }
                asm volatile("bar.sync 1, %0;\n" ::"n"(32 * kGradCompute) : "memory");
            }
            const bool finish = warp == 0 && vt == p.vtiles - 1;
            float state_dot = 0.f, skip_all = 0.f, timed = 0.f, sloped = 0.f, m[4], yy[4], w[4], dts[4], sl[4];
            if (finish) {  // all that is read in shared memory, before the next unit may change it
                for (int i = 0; i < kGradCompute; ++i) {
                    state_dot += sums.dots[i];
                    skip_all += sums.skips[i];
                    timed += sums.das[i];
                    sloped += sums.dbs[i];
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int t = 4 * lane + i;
                    const float column = (sums.cols[0][t] + sums.cols[1][t]) + (sums.cols[2][t] + sums.cols[3][t]), yv = sums.ys[0][t] + sums.ys[1][t];
                    dts[i] = st.dt[t];
                    sl[i] = slope[t];
                    w[i] = column + sums.diag[t] + yv;
                    m[i] = (sums.rows[0][t] + sums.rows[1][t]) - dts[i] * column;
                    yy[i] = dts[i] * yv;
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.freed);
            if (finish) {
                // four tokens a lane: sums from the end of (rows - dt columns + X), from the start of dt Y
                float down = (m[0] + m[1]) + (m[2] + m[3]), up = (yy[0] + yy[1]) + (yy[2] + yy[3]);
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const float d = __shfl_down_sync(0xffffffffu, down, o), a = __shfl_up_sync(0xffffffffu, up, o);
                    if (lane + o < 32) down += d;
                    if (lane >= o) up += a;
                }
                float behind = __shfl_down_sync(0xffffffffu, down, 1), before = __shfl_up_sync(0xffffffffu, up, 1);
                if (lane == 31) behind = 0.f;
                if (lane == 0) before = 0.f;
                float gr[4];
#pragma unroll
                for (int i = 3; i >= 0; --i) {
                    behind += m[i];
                    gr[i] = behind;
                }
                float dA = 0.f, dbias = 0.f;
                const float a = __ldg(p.A + head);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int t = 4 * lane + i;
                    gr[i] += before + state_dot;
                    before += yy[i];
                    if (t >= len) continue;
                    dA = fmaf(dts[i], gr[i], dA);
                    float dd = fmaf(a, gr[i], w[i]);
                    if (p.delta != nullptr) {
                        dd *= sl[i];
                        dbias = fmaf(sl[i], w[i], dbias);
                        static_cast<bf16*>(p.ddelta)[((long long)b * p.heads + head) * p.L + t0 + t] = __float2bfloat16_rn(dd);
                    }
                }
                dA = warp_sum(dA);
                // (a rate of zero, or next to it, has no fast decay)
                if (fabsf(a) > 1e-12f) dA = timed / (a * kLog2e);
                dbias = fmaf(a, sloped, warp_sum(dbias));
                if (lane == 0) {
                    const long long all = (long long)p.batch * p.chunks, at = (long long)b * p.chunks + blockIdx.x;
                    p.head_part[head * all + at] = dA;
                    p.head_part[((long long)p.heads + head) * all + at] = dbias;
                    p.head_part[((long long)2 * p.heads + head) * all + at] = skip_all;
                }
            }
        }
        // dq and dk: a thread has a channel and 32 of the tokens
        if (units > 0) {
            wait(&bar.done3, (units - 1) & 1);
            tc_fence_after();
            const bool vec = p.L % 8 == 0 && len == kTcChunk;
#pragma unroll 1
            for (int which = 0; which < 2; ++which) {
                const long long at = ((long long)b * p.groups * p.N + (long long)group * p.N + r) * p.L + t0;
                float* part = which ? p.dk_part : p.dq_part;
                if (part != nullptr) part += (long long)subset * p.batch * p.groups * p.N * p.L + at;
                bf16* out = static_cast<bf16*>(which ? p.dk : p.dq) + at;
                const bool fine = vec && (part != nullptr ? is_aligned16(part) : is_aligned16(out));
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    const int c0 = 32 * g + 16 * h;
                    float s[16];
                    tc_load16(mine + (which ? dk_at : dq_at) + c0, s);
                    tc_wait_loads(s);
                    if (r >= p.N) continue;
                    if (fine && part != nullptr) {
#pragma unroll
                        for (int j = 0; j < 16; j += 4) *reinterpret_cast<float4*>(part + c0 + j) = make_float4(s[j], s[j + 1], s[j + 2], s[j + 3]);
                    } else if (fine) {
#pragma unroll
                        for (int j = 0; j < 16; j += 8)
                            *reinterpret_cast<uint4*>(out + c0 + j) = make_uint4(pack_bf16(s[j], s[j + 1]), pack_bf16(s[j + 2], s[j + 3]),
                                                                                pack_bf16(s[j + 4], s[j + 5]), pack_bf16(s[j + 6], s[j + 7]));
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            if (c0 + j >= len) continue;
                            if (part != nullptr) part[c0 + j] = s[j];
                            else out[c0 + j] = __float2bfloat16_rn(s[j]);
                        }
                    }
                }
            }
        }
    } else if (warp == kGradCompute) {
        // ---- tiles and steps ---------------------------------------------------------
        if (lane == 0 && units > 0) {
            mbar_arrive_expect_tx(&bar.full_qk, 2 * M::tile);
            for (int h = 0; h < 2; ++h) {
                tma_load_4d(smem + M::q + h * KD * 128, &maps.q, t0 + 64 * h, 0, group, b, &bar.full_qk);
                tma_load_4d(smem + M::k + h * KD * 128, &maps.k, t0 + 64 * h, 0, group, b, &bar.full_qk);
            }
        }
        __syncwarp();
        for (int u = 0; u < units; ++u) {
            const int head = h0 + u / p.vtiles, v0 = u % p.vtiles * kValueTile;
            // the unit's steps, in registers until the unit before is done with its own
            const float rate = __ldg(p.A + head) * kLog2e;
            const long long at = b * p.tb + head * p.td + t0;
            float x[4], down = 0.f;
            Sum2 up{0.f, 0.f};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = 4 * lane + j;
                x[j] = c < len ? lattn_step_of<bf16>(p, at + c, head) : 0.f;
                up = up + Sum2{x[j], 0.f};
                down += x[j];
            }
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const Sum2 a = shfl_up2(up, o);
                const float d = __shfl_down_sync(0xffffffffu, down, o);
                if (lane >= o) up = a + up;
                if (lane + o < 32) down += d;
            }
            Sum2 run = shfl_up2(up, 1);
            float behind = __shfl_down_sync(0xffffffffu, down, 1);
            if (lane == 0) run = Sum2{0.f, 0.f};
            if (lane == 31) behind = 0.f;
            const float all = __shfl_sync(0xffffffffu, up.h, 31);
            float runs[4], lows[4], pres[4], ends[4];
            const float rests[4] = {behind + (x[3] + x[2] + x[1]), behind + (x[3] + x[2]), behind + x[3], behind};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = 4 * lane + j;
                run = run + Sum2{x[j], 0.f};
                runs[j] = rate * run.h;
                lows[j] = fmaf(rate, run.h, -runs[j]) + rate * run.l;
                // (tokens behind the last are zeros everywhere; their factors must be finite)
                pres[j] = c < len ? p.scale * ex2(runs[j]) : 0.f;
                ends[j] = c < len ? ex2(rate * rests[j]) : 0.f;
            }
            const float decay = ex2(rate * all);
            // the slopes' sums
            float slopes[4];
            Sum2 zs{0.f, 0.f};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                slopes[j] = 4 * lane + j < len ? lattn_slope_of<bf16>(p, at + 4 * lane + j, head) : 0.f;
                zs = zs + Sum2{slopes[j], 0.f};
            }
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const Sum2 a = shfl_up2(zs, o);
                if (lane >= o) zs = a + zs;
            }
            zs = shfl_up2(zs, 1);
            if (lane == 0) zs = Sum2{0.f, 0.f};
            // the states' tiles are free with the last products, the others once dv is written
            if (u > 0) wait(&bar.done3, (u - 1) & 1);
            if (lane == 0) {
                mbar_arrive_expect_tx(&bar.full_s, 2 * KD * 256);
                bulk_load(smem + M::s, image(p.starts, u), KD * 256, &bar.full_s);
                bulk_load(smem + M::d, image(p.dends, u), KD * 256, &bar.full_s);
            }
            __syncwarp();
            if (u > 0) wait(&bar.freed, (u - 1) & 1);
            if (lane == 0) {
                mbar_arrive_expect_tx(&bar.full, 2 * 16384);
                for (int h = 0; h < 2; ++h) {
                    tma_load_4d(smem + M::v + h * 8192, &maps.v, t0 + 64 * h, v0, head, b, &bar.full);
                    tma_load_4d(smem + M::u + h * 8192, &maps.dout, t0 + 64 * h, v0, head, b, &bar.full);
                }
                if (u + 1 < units) {
                    bulk_prefetch(image(p.starts, u + 1), KD * 256);
                    bulk_prefetch(image(p.dends, u + 1), KD * 256);
                    const int head1 = h0 + (u + 1) / p.vtiles, v1 = (u + 1) % p.vtiles * kValueTile;
                    for (int h = 0; h < 2; ++h) {
                        tma_prefetch_4d(&maps.v, t0 + 64 * h, v1, head1, b);
                        tma_prefetch_4d(&maps.dout, t0 + 64 * h, v1, head1, b);
                    }
                }
            }
            __syncwarp();
            *reinterpret_cast<float4*>(&st.run[4 * lane]) = make_float4(runs[0], runs[1], runs[2], runs[3]);
            *reinterpret_cast<float4*>(&st.low[4 * lane]) = make_float4(lows[0], lows[1], lows[2], lows[3]);
            *reinterpret_cast<float4*>(&st.dt[4 * lane]) = make_float4(x[0], x[1], x[2], x[3]);
            *reinterpret_cast<float4*>(&st.pre[4 * lane]) = make_float4(pres[0], pres[1], pres[2], pres[3]);
            *reinterpret_cast<float4*>(&st.rest[4 * lane]) = make_float4(ends[0], ends[1], ends[2], ends[3]);
            *reinterpret_cast<float4*>(&st.tail[4 * lane]) = make_float4(x[0] * ends[0], x[1] * ends[1], x[2] * ends[2], x[3] * ends[3]);
            if (lane == 0) st.decay = decay;
            float zh[4], zl[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                zs = zs + Sum2{slopes[j], 0.f};
                zh[j] = zs.h;
                zl[j] = zs.l;
            }
            *reinterpret_cast<float4*>(&slope[4 * lane]) = make_float4(slopes[0], slopes[1], slopes[2], slopes[3]);
            *reinterpret_cast<float4*>(&slope_sum[4 * lane]) = make_float4(zh[0], zh[1], zh[2], zh[3]);
            *reinterpret_cast<float4*>(&slope_low[4 * lane]) = make_float4(zl[0], zl[1], zl[2], zl[3]);
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.full);
        }
        // no copy is in flight when the CTA ends, even after a wait that gave up
        if (units > 0) {
            mbar_wait_bounded(&bar.full_qk, 0);
            mbar_wait_bounded(&bar.full, (units - 1) & 1);
            mbar_wait_bounded(&bar.full_s, (units - 1) & 1);
        }
    } else {
        // ---- products -----------------------------------------------------------------
        const int steps_n = (p.N + 15) / 16;
        const unsigned sa = smem_addr(smem);
        const uint64_t q_across = desc_across(sa + M::q, KD, 0), k_across = desc_across(sa + M::k, KD, 0);
        const uint64_t q_along = desc_along(sa + M::q, KD, 0), k_along = desc_along(sa + M::k, KD, 0);
        const uint64_t v_across = desc_across(sa + M::v, 64, 0), u_across = desc_across(sa + M::u, 64, 0), u_along = desc_along(sa + M::u, 64, 0);
        const uint64_t s_across = desc_across(sa + M::s, KD, 0), d_across = desc_across(sa + M::d, KD, 0);
        const uint64_t s_along = desc_along(sa + M::s, KD, 0), d_along = desc_along(sa + M::d, KD, 0);
        const uint64_t e_along = desc_along(sa + M::e, 128, 0), e_across = desc_across(sa + M::e, 128, 0), f_across = desc_across(sa + M::f, 128, 0);
        const uint64_t us_across = desc_across(sa + M::e, 64, 0), vs_across = desc_across(sa + M::f, 64, 0);
        // sixteen values further along a row of a tile of `rows` rows
        auto along = [](int j, int rows) { return (uint64_t)((j >> 2) * (rows * 8) + (j & 3) * 2); };
        if (units > 0) wait(&bar.full_qk, 0);
        for (int u = 0; u < units; ++u) {
            if (u > 0) wait(&bar.freed, (u - 1) & 1);
            tc_fence_after();
            if (tc_elect()) {
#pragma unroll 4
                for (int j = 0; j < steps_n; ++j) tc_mma(tm + qk_at, q_across + 128 * j, k_across + 128 * j, tc_kind(128, 128, true, true), j > 0);
            }
            __syncwarp();
            wait(&bar.full, u & 1);
            tc_fence_after();
            if (tc_elect()) {
#pragma unroll
                for (int j = 0; j < 4; ++j) tc_mma(tm + g_at, u_across + 128 * j, v_across + 128 * j, tc_kind(128, 128, true, true), j > 0);
                tc_commit(&bar.done1);
            }
            __syncwarp();
            wait(&bar.scores_read, u & 1);
            wait(&bar.full_s, u & 1);
            tc_fence_after();
            if (tc_elect()) {
#pragma unroll 1
                for (int term = 0; term < 2; ++term) {
                    const uint64_t off = term * (KD * 8);
#pragma unroll 4
                    for (int j = 0; j < steps_n; ++j) {
                        tc_mma(tm + di_at, k_across + 128 * j, d_across + off + 128 * j, tc_kind(128, 64, true, true), term + j > 0);
                        tc_mma(tm + u_at, q_across + 128 * j, s_across + off + 128 * j, tc_kind(128, 64, true, true), term + j > 0);
                    }
                }
            }
            __syncwarp();
            wait(&bar.ready_ef, u & 1);
            tc_fence_after();
            if (tc_elect()) {
#pragma unroll 4
                for (int i = 0; i < 8; ++i) {
                    // tokens t < 64 have no pairs with s >= 64
                    const int j = i ^ 4;
                    tc_mma(tm + df_at, f_across + 128 * i, u_along + along(i, 64), tc_kind(128, 64, true, false), i > 0);
                    if (i < 4) tc_mma(tm + dq_at, k_along + along(i, KD), e_along + along(i, 128), tc_kind(128, 128, false, false), u + i > 0);
                    else tc_mma(tm + dq_at + 64, k_along + along(i, KD), e_along + along(i, 128) + 512, tc_kind(128, 64, false, false), true);
                    if (i < 4) tc_mma(tm + dk_at, q_along + along(j, KD), e_across + 128 * j, tc_kind(128, 128, false, true), u + i > 0);
                    else tc_mma(tm + dk_at, q_along + along(j, KD), e_across + 128 * j, tc_kind(128, 64, false, true), true);
                }
                tc_commit(&bar.done2);
            }
            __syncwarp();
            wait(&bar.ready_scaled, u & 1);
            tc_fence_after();
            if (tc_elect()) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    tc_mma(tm + dq_at, s_along + 2 * j, us_across + 128 * j, tc_kind(128, 128, false, true), true);
                    tc_mma(tm + dk_at, d_along + 2 * j, vs_across + 128 * j, tc_kind(128, 128, false, true), true);
                }
                tc_commit(&bar.done3);
            }
            __syncwarp();
        }
        if (units > 0) mbar_wait_bounded(&bar.done3, (units - 1) & 1);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kGradCompute + 1) tc_free(tm, 512);
}

}  // namespace sscan
