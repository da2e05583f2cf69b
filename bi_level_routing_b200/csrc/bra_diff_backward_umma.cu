// bra_diff_backward_umma.cu -- gradients of differential attention for bf16 maps with large regions on the
// 5th-generation tensor cores (tcgen05, TMEM accumulators); the formula in bra_diff.cuh, the two passes and what
// passes between them as in bra_diff_backward.cu, the machinery as in bra_diff_umma.cu: eight warps at the exponentials,
// one issuing products, two gathering rows into a ring of stages, one handing landed stages over. Each of the two
// softmax warpgroups takes every other tile with a score buffer of its own, so that one buffer's products run under
// the other's exponentials.
//
// queries: a CTA owns 128 queries. S1, S2 and dP = dout V^T of every key tile are formed twice: first for both
//   softmaxes' maximum and sum and D_i = rowsum(P_i dP), which the warpgroups take over their own tiles and merge, then
//   for dS_i, written as two bf16 terms over S_i and dP in TMEM and multiplied from there: dq_i += dS_i K_i.
// keys: a CTA owns 128 keys and meets the queries that route to them. S_i and dP are formed transposed (keys as
//   rows), so that P1 - lam P2 and dS_i again multiply from where they were scored: dv += (P1 - lam P2)^T dout,
//   dk_i += dS_i^T q_i.
//
// Five products of hd channels, 10 hd operations a query-key pair, and two exponentials are due. Scoring three times and
// the second term of dS make them 20 hd and six. 4096-token maps (4 images, 4 heads of 128) take 1020 us, some 590 the
// queries kernel, where the exponentials (16 a cycle and SM) and the score products share the time, 430 the keys
// kernel, whose products of 32 columns are bound by reading their 128-row operands from shared memory. 512 CTAs
// of one an SM are 3.46 rounds of 148. Precision as in bra_diff_backward.cu.
#include "bra_diff.cuh"

namespace bra {

namespace {

constexpr int kThreads = 384;
constexpr int kOwnBlock = 128 * 128;  // 128 rows x 64 channels
constexpr uint32_t kCols = 512;
constexpr int kBarrierBytes = 512;

// NB: 64-channel blocks of a head; T: rows of a streamed tile (keys, or queries)
template <int NB, int T, int ST> struct BackRing {
    static constexpr int kBlock = T * 128;
    static constexpr int kStage = 2 * NB * kBlock;  // the two streamed arrays
    static constexpr size_t kOwn = (size_t)2 * NB * kOwnBlock;
    static constexpr size_t kRing = (size_t)ST * kStage;
};
constexpr int kKeyTile = 64;  // of the queries kernel
template <int NB> using QueryRing = BackRing<NB, kKeyTile, NB == 1 ? 5 : 4>;
template <int NB> struct KeyPlan {  // of the keys kernel: accumulators of 128 NB columns leave room for two buffers of
    static constexpr int kTile = NB == 1 ? 64 : 32;  // three of these
    static constexpr int kStages = NB == 1 ? 5 : 6;
    using Ring = BackRing<NB, kTile, kStages>;
};

// The lane's 16-byte chunk (of each block) of a row: where it comes from. Halves of d channels are padded with zeros to
// 32 NB for q and k, hd channels to 64 NB for v and dout.
template <int NB> struct Chunk {
    int half[NB], whole[NB];
    bool in_half[NB], in_whole[NB];
    __device__ __forceinline__ Chunk(int lane, int dc)
    {
        const int j = lane & 7;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const int c = j + 8 * nb, m = c / (4 * NB), x = c % (4 * NB);
            in_half[nb] = x < dc;
            half[nb] = in_half[nb] ? 8 * (m * dc + x) : 0;
            in_whole[nb] = c < 2 * dc;
            whole[nb] = in_whole[nb] ? 8 * c : 0;
        }
    }
};

// A warp copies 32 rows (the row of lane l at token `at` of the image, -1: zeros) of two arrays, `split` in halves and
// `run`, to rows r0 .. of the tiles at `dst` and dst + NB blocks.
template <int NB>
__device__ __forceinline__ void gather_rows(const Chunk<NB> &ch, uint32_t dst, int block, int r0, int at, int lane,
                                            const __nv_bfloat16 *split, const __nv_bfloat16 *run, int C)
{
    const int j = lane & 7, sub = lane >> 3;
#pragma unroll
    for (int x = 0; x < 8; ++x) {
        const int tok = __shfl_sync(0xffffffffu, at, 4 * x + sub);
        const int64_t off = (int64_t)max(tok, 0) * C;
        const uint32_t to = dst + sw128(r0 + 4 * x + sub, j);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            cp_async16_or_zero(to + nb * block, split + off + ch.half[nb], tok >= 0 && ch.in_half[nb]);
            cp_async16_or_zero(to + (NB + nb) * block, run + off + ch.whole[nb], tok >= 0 && ch.in_whole[nb]);
        }
    }
}

struct BackBarriers {
    uint64_t *own_full, *own_ready, *full, *ready, *empty, *s_full, *p_full, *drain;
    __device__ __forceinline__ BackBarriers(uint64_t *at, int st)
        : own_full(at), own_ready(at + 1), full(at + 2), ready(full + st), empty(ready + st), s_full(empty + st),
          p_full(s_full + 2), drain(p_full + 2) {}
    __device__ __forceinline__ void init(int st, int copiers)
    {
        mbar_init(own_full, 32);
        mbar_init(own_ready, 1);
        for (int i = 0; i < st; ++i) {
            mbar_init(&full[i], copiers);
            mbar_init(&ready[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
        }
        mbar_init(drain, 1);
        mbar_fence_init();
    }
};

// Warp 11: the CTA's own 128 rows, then a proxy fence between every stage's landing and its use.
template <int NB>
__device__ __forceinline__ void own_rows_and_relay(const DiffArgs &a, const BackBarriers &bar, const Chunk<NB> &ch, uint32_t own,
                                                   const __nv_bfloat16 *split, const __nv_bfloat16 *run, int region, int tok0,
                                                   int lane, int steps, int st)
{
    for (int r0 = 0; r0 < 128; r0 += 32) {
        const int at = tok0 + r0 + lane < a.rs ? token_at(a, region, tok0 + r0 + lane) : -1;
        gather_rows<NB>(ch, own, kOwnBlock, r0, at, lane, split, run, a.C);
    }
    cp_async_arrive(bar.own_full);
    bool alive = steps > 0 && mbar_wait(bar.own_full, 0, a.err);
    fence_async_shared();
    if (lane == 0 && alive) mbar_arrive(bar.own_ready);
    for (int i = 0; i < steps && alive; ++i) {
        alive = mbar_wait(&bar.full[i % st], (uint32_t)((i / st) & 1), a.err);
        fence_async_shared();
        __syncwarp();
        if (lane == 0 && alive) mbar_arrive(&bar.ready[i % st]);
    }
    cp_async_wait_all();
}

// Half a row's (or a whole row's) accumulator columns from TMEM, scaled, rounded and stored: `cols` columns from `t`, of
// which the first `real` are channels of dst.
__device__ __forceinline__ void store_columns(uint32_t t, int cols, int real, float scale, __nv_bfloat16 *dst, bool in)
{
    for (int c = 0; c < cols; c += 32) {
        uint32_t v[32];
        tmem_ld_32x32(t + c, v);
        tmem_wait_ld();
#pragma unroll
        for (int x = 0; x < 32; x += 8) {
            uint32_t pk[4];
#pragma unroll
            for (int y = 0; y < 4; ++y)
                pk[y] = pack_bf16x2(__uint_as_float(v[x + 2 * y]) * scale, __uint_as_float(v[x + 2 * y + 1]) * scale);
            if (in && c + x < real) *reinterpret_cast<uint4 *>(dst + c + x) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
        }
    }
}
__device__ __forceinline__ void store_zeros(int real, __nv_bfloat16 *dst, bool in)
{
    if (in)
        for (int c = 0; c < real; c += 8) *reinterpret_cast<uint4 *>(dst + c) = make_uint4(0, 0, 0, 0);
}

}  // namespace

// ------------------------------------------------------------------ dq, statistics

template <int NB> __global__ void __launch_bounds__(kThreads, 1) diff_backward_queries_umma_kernel(const DiffArgs a)
{
    using L = QueryRing<NB>;
    constexpr int T = kKeyTile, ST = NB == 1 ? 5 : 4, kBlock = L::kBlock, KS = 2 * NB;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sOwn = smem, *sRing = smem + L::kOwn;  // [q, dout][NB], [stage][k, v][NB]
    BackBarriers bar(reinterpret_cast<uint64_t *>(sRing + L::kRing), ST);
    float *part = reinterpret_cast<float *>(sRing + L::kRing + kBarrierBytes);  // [warpgroup][6][128]
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(part + 2 * 6 * 128);
    int *count = reinterpret_cast<int *>(tmem_slot + 1);
    int *bases = count + 3;
    const int warp = uniform((int)(threadIdx.x >> 5)), lane = threadIdx.x & 31;
    if (blockIdx.x < a.B) {
        grid_dependency_wait();
        invert_index<kThreads / 32>(a, blockIdx.x, reinterpret_cast<int *>(smem));
        return;
    }
    const DiffItem it = diff_item(a, blockIdx.x - a.B);

    if (threadIdx.x == 0) bar.init(ST, 64);
    if (warp == 8) {
        tmem_alloc(tmem_slot, kCols);
        tmem_relinquish();
    }
    grid_dependency_wait();
    if (warp == 9) {
        const int n = gather_bases(a, a.idx + ((int64_t)it.b * a.R + it.r) * a.topk, bases, lane);
        if (lane == 0) *count = n;
    }
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    const uint32_t tmem = *tmem_slot;
    const int nkeys = *count * a.rs;
    const int ntiles = (nkeys + T - 1) / T, steps = 2 * ntiles;
    const int64_t image = (int64_t)it.b * a.N * a.C + it.h * a.hd;
    const int region = region_at(a, it.r);
    const int tok0 = it.t * 128;

    if (warp >= 9) {
        const Chunk<NB> ch(lane, a.d / 8);
        if (warp == 11) {
            own_rows_and_relay<NB>(a, bar, ch, smem_u32(sOwn), static_cast<const __nv_bfloat16 *>(a.q) + image,
                                   static_cast<const __nv_bfloat16 *>(a.dout) + image, region, tok0, lane, steps, ST);
        } else {
            const __nv_bfloat16 *gk = static_cast<const __nv_bfloat16 *>(a.k) + image;
            const __nv_bfloat16 *gv = static_cast<const __nv_bfloat16 *>(a.v) + image;
            const int r0 = 32 * (warp - 9);
            for (int i = 0; i < steps; ++i) {
                const int st = i % ST, key = (i < ntiles ? i : i - ntiles) * T + r0 + lane;
                int at = -1;
                if (key < nkeys) {
                    int slot, tok;
                    a.by_rs.divmod(key, slot, tok);
                    at = token_at(a, bases[slot], tok);
                }
                if (!mbar_wait(&bar.empty[st], (uint32_t)(((i / ST) & 1) ^ 1), a.err)) break;
                gather_rows<NB>(ch, smem_u32(sRing + (size_t)st * L::kStage), kBlock, r0, at, lane, gk, gv, a.C);
                cp_async_arrive(&bar.full[st]);
            }
            cp_async_wait_all();
        }
    } else if (warp == 8) {
        // products: S1, S2 and dP of tile i in buffer i & 1 (columns 192 (i & 1) + 0, 64, 128), dq from column 384
        constexpr uint32_t kIdescS = umma_idesc_bf16(128, T, false), kIdescQ = umma_idesc_bf16(128, 32 * NB, true);
        const int n = uniform(ntiles), all = uniform(steps);
        const uint32_t tm = uniform(tmem), own = uniform(desc_low(smem_u32(sOwn))), ring = uniform(desc_low(smem_u32(sRing)));
        const bool leader = elect_one();
        bool alive = all > 0 && mbar_wait(bar.own_ready, 0, a.err);
        int st = 0, next = 0;
        uint32_t phase = 0;
        auto scores = [&](uint32_t buf) {
            const uint32_t rk = ring + next * (L::kStage >> 4), rv = rk + NB * (kBlock >> 4);
            if (leader) {
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks)
                        umma_ss(tm + 192 * buf + 64 * m, own + (NB == 1 ? 4 * m : m * (kOwnBlock >> 4)) + 2 * ks,
                                rk + (NB == 1 ? 4 * m : m * (kBlock >> 4)) + 2 * ks, kIdescS, ks > 0);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        umma_ss(tm + 192 * buf + 128, own + (NB + nb) * (kOwnBlock >> 4) + 2 * ks, rv + nb * (kBlock >> 4) + 2 * ks,
                                kIdescS, nb > 0 || ks > 0);
            }
            if (++next == ST) {
                next = 0;
                phase ^= 1;
            }
        };
        for (int i = 0; i < 2 && i < all && alive; ++i) {
            if (!(alive = mbar_wait(&bar.ready[next], phase, a.err))) break;
            tcgen05_after_sync();
            scores(i);
            if (leader) umma_commit(&bar.s_full[i]);
            __syncwarp();
        }
        for (int i = 0; i < all && alive; ++i) {
            const uint32_t buf = i & 1;
            if (i + 2 < all) alive = mbar_wait(&bar.ready[next], phase, a.err);
            alive = alive && mbar_wait(&bar.p_full[buf], (uint32_t)((i >> 1) & 1), a.err);
            if (!alive) break;
            tcgen05_after_sync();
            if (i >= n && leader) {
                const uint32_t rk = ring + st * (L::kStage >> 4);
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int ks = 0; ks < T / 16; ++ks)
#pragma unroll
                        for (int term = 0; term < 2; ++term)  // dS's high terms over S_m, its low ones over dP
                            umma_ts(tm + 384 + 32 * NB * m,
                                    tm + 192 * buf + (term ? 128 + 32 * (ks / 2) + 16 * m + 8 * (ks % 2) : 64 * m + 8 * ks),
                                    rk + (NB == 1 ? 4 * m : m * (kBlock >> 4)) + 128 * ks, kIdescQ, i > n || ks > 0 || term > 0);
            }
            if (i + 2 < all) scores(buf);
            if (leader) {
                umma_commit(&bar.s_full[buf]);
                umma_commit(&bar.empty[st]);
            }
            __syncwarp();
            if (++st == ST) st = 0;
        }
        if (leader) umma_commit(bar.drain);
        __syncwarp();
        mbar_wait(bar.drain, 0, a.err);
    } else {
        const int g = warp >> 2, row = 32 * (warp & 3) + lane;
        const uint32_t t_row = tmem + ((uint32_t)(32 * (warp & 3)) << 16), t_s = t_row + 192 * g;
        const bool busy = tok0 + 32 * (warp & 3) < a.rs;  // the warp has a query
        const float2 sc = make_float2(a.scale_log2, a.scale_log2);
        bool alive = true;
        float2 mx = make_float2(-INFINITY, -INFINITY), l = make_float2(0.f, 0.f), ed = l;  // of both maps
        auto release = [&] {
            tcgen05_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.p_full[g]);
        };
        int i = g;
        for (; i < ntiles; i += 2) {
            if (!(alive = mbar_wait(&bar.s_full[g], (uint32_t)((i >> 1) & 1), a.err))) break;
            tcgen05_after_sync();
            if (busy) {
#pragma unroll
                for (int c = 0; c < T; c += 32) {
                    uint32_t s1[32], s2[32], dp[32];
                    tmem_ld_32x32(t_s + c, s1);
                    tmem_ld_32x32(t_s + 64 + c, s2);
                    tmem_ld_32x32(t_s + 128 + c, dp);
                    tmem_wait_ld();
                    if ((i + 1) * T > nkeys) {
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            if (i * T + c + x >= nkeys) s1[x] = s2[x] = 0xff800000u;
                    }
                    float t1[2] = {-INFINITY, -INFINITY}, t2[2] = {-INFINITY, -INFINITY};
#pragma unroll
                    for (int x = 0; x < 32; x += 2) {
                        t1[(x >> 1) & 1] = fmax3(t1[(x >> 1) & 1], __uint_as_float(s1[x]), __uint_as_float(s1[x + 1]));
                        t2[(x >> 1) & 1] = fmax3(t2[(x >> 1) & 1], __uint_as_float(s2[x]), __uint_as_float(s2[x + 1]));
                    }
                    const float2 most = make_float2(fmaxf(mx.x, fmaxf(t1[0], t1[1]) * a.scale_log2),
                                                    fmaxf(mx.y, fmaxf(t2[0], t2[1]) * a.scale_log2));
                    const float2 base = make_float2(score_base(most.x), score_base(most.y));
                    const float2 corr = make_float2(fast_exp2(mx.x - base.x), fast_exp2(mx.y - base.y));
                    mx = most;
                    l = __fmul2_rn(l, corr);
                    ed = __fmul2_rn(ed, corr);
                    const float2 nm = make_float2(-base.x, -base.y);
                    float2 la = make_float2(0.f, 0.f), ea = la;
#pragma unroll
                    for (int x = 0; x < 32; ++x) {
                        const float2 z = __ffma2_rn(make_float2(__uint_as_float(s1[x]), __uint_as_float(s2[x])), sc, nm);
                        const float2 e = make_float2(fast_exp2(z.x), fast_exp2(z.y));
                        la = __fadd2_rn(la, e);
                        ea = __ffma2_rn(e, make_float2(__uint_as_float(dp[x]), __uint_as_float(dp[x])), ea);
                    }
                    l = __fadd2_rn(l, la);
                    ed = __fadd2_rn(ed, ea);
                }
            }
            release();
        }
        // the warpgroups' statistics of a row, merged: L = max + log2(sum) and D of each map
        float *mine = part + 6 * 128 * g + row;
        mine[0] = mx.x;
        mine[128] = mx.y;
        mine[256] = l.x;
        mine[384] = l.y;
        mine[512] = ed.x;
        mine[640] = ed.y;
        named_barrier(1, 256);
        float Ls[2], D[2];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const float *x = part + 128 * m + row, *y = x + 6 * 128;
            const float top = fmaxf(x[0], y[0]), base = score_base(top);
            const float wx = fast_exp2(x[0] - base), wy = fast_exp2(y[0] - base);
            const float sum = x[256] * wx + y[256] * wy, num = x[512] * wx + y[512] * wy;
            Ls[m] = log_sum(top, sum, nkeys > 0);
            D[m] = over_sum(num, sum, nkeys > 0);
        }
        const bool in = tok0 + row < a.rs;
        const int token = in ? token_at(a, region, tok0 + row) : 0;
        if (g == 0) {
            if (in) a.stats[((int64_t)it.b * a.heads + it.h) * a.N + token] = make_float4(Ls[0], Ls[1], D[0], D[1]);
            const float dsum = warp_sum(in ? D[1] : 0.f);
            if (lane == 0)
                a.dlam_part[(int64_t)it.h * a.nparts + (((int64_t)it.b * a.R + it.r) * a.tiles + it.t) * 4 + warp] = dsum;
        }
        const float2 nl = make_float2(-Ls[0], -Ls[1]), nd = make_float2(-D[0], -D[1]);
        for (; i < steps && alive; i += 2) {
            if (!(alive = mbar_wait(&bar.s_full[g], (uint32_t)((i >> 1) & 1), a.err))) break;
            tcgen05_after_sync();
            if (busy) {
#pragma unroll
                for (int c = 0; c < T; c += 32) {
                    uint32_t s1[32], s2[32], dp[32];
                    tmem_ld_32x32(t_s + c, s1);
                    tmem_ld_32x32(t_s + 64 + c, s2);
                    tmem_ld_32x32(t_s + 128 + c, dp);
                    tmem_wait_ld();
                    uint32_t w1[16], w2[16], low[32];  // dS1, dS2: high terms; low terms of 1, then of 2
#pragma unroll
                    for (int x = 0; x < 32; x += 2) {
                        float2 ds[2];
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const float dpx = __uint_as_float(dp[x + y]);
                            const float2 z = __ffma2_rn(make_float2(__uint_as_float(s1[x + y]), __uint_as_float(s2[x + y])), sc, nl);
                            ds[y] = __fmul2_rn(make_float2(fast_exp2(z.x), fast_exp2(z.y)), __fadd2_rn(make_float2(dpx, dpx), nd));
                        }
                        const float h0 = bf16_trunc(ds[0].x), h1 = bf16_trunc(ds[1].x);
                        const float g0 = bf16_trunc(ds[0].y), g1 = bf16_trunc(ds[1].y);
                        w1[x / 2] = pack_bf16x2_trunc(h0, h1);
                        w2[x / 2] = pack_bf16x2_trunc(g0, g1);
                        low[x / 2] = pack_bf16x2(ds[0].x - h0, ds[1].x - h1);
                        low[16 + x / 2] = pack_bf16x2(ds[0].y - g0, ds[1].y - g1);
                    }
                    if ((i - ntiles + 1) * T > nkeys) {  // keys past the last one: their rows of k are zeros, their dS must be finite
#pragma unroll
                        for (int x = 0; x < 16; ++x) {
                            const int key = (i - ntiles) * T + c + 2 * x;
                            if (key >= nkeys) w1[x] = w2[x] = low[x] = low[16 + x] = 0u;
                            if (key + 1 == nkeys) {
                                w1[x] &= 0xffffu;
                                w2[x] &= 0xffffu;
                                low[x] &= 0xffffu;
                                low[16 + x] &= 0xffffu;
                            }
                        }
                    }
                    tmem_st_32x16(t_s + c / 2, w1);
                    tmem_st_32x16(t_s + 64 + c / 2, w2);
                    tmem_st_32x32(t_s + 128 + c, low);
                }
                tmem_wait_st();
            }
            release();
        }
        // The commit after the last tile's products. Both warpgroups have seen their last scores by now, so the barrier, one
        // warpgroup's own, cannot be a whole round behind, where its parity would read the same.
        named_barrier(1, 256);
        if (steps > 0 && alive)
            alive = mbar_wait(&bar.s_full[(steps + 1) & 1], (uint32_t)(((steps + 1) >> 1) & 1), a.err);
        tcgen05_after_sync();
        __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.dq) + image + (int64_t)token * a.C + g * a.d;
        if (steps > 0)
            store_columns(t_row + 384 + 32 * NB * g, 32 * NB, a.d, g ? -__ldg(a.lam + it.h) * a.scale : a.scale, dst, in && alive);
        else
            store_zeros(a.d, dst, in);
    }
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    if (warp == 8) tmem_dealloc(tmem, kCols);
}

// ------------------------------------------------------------------ dk, dv, dlam

template <int NB> __global__ void __launch_bounds__(kThreads, 1) diff_backward_keys_umma_kernel(const DiffArgs a)
{
    using L = typename KeyPlan<NB>::Ring;
    constexpr int T = KeyPlan<NB>::kTile, ST = KeyPlan<NB>::kStages, kBlock = L::kBlock, KS = 2 * NB;
    constexpr uint32_t kBuf = 3 * T, kAcc = 6 * T;  // TMEM: buffer u at kBuf u (S1, S2, dP), dv at kAcc, dk after it
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sOwn = smem, *sRing = smem + L::kOwn;  // [k, v][NB], [stage][q, dout][NB]
    float4 *sstat = reinterpret_cast<float4 *>(sRing + L::kRing);  // [stage][T]
    BackBarriers bar(reinterpret_cast<uint64_t *>(sstat + ST * T), ST);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(reinterpret_cast<uint8_t *>(sstat + ST * T) + kBarrierBytes);
    const int warp = uniform((int)(threadIdx.x >> 5)), lane = threadIdx.x & 31;

    grid_dependency_wait();
    if (blockIdx.x < a.heads) {  // dlam of head blockIdx.x, summed in 64 bits in a fixed order
        double *sums = reinterpret_cast<double *>(smem);
        const float *src = a.dlam_part + (int64_t)blockIdx.x * a.nparts;
        double sum = 0.;
        for (int e = threadIdx.x; e < a.nparts; e += kThreads) sum += (double)__ldcg(src + e);
        sums[threadIdx.x] = sum;
        __syncthreads();
        if (threadIdx.x == 0) {
            double total = 0.;
            for (int e = 0; e < kThreads; ++e) total += sums[e];
            a.dlam[blockIdx.x] = (float)-total;
        }
        __syncthreads();
    }
    if (blockIdx.x >= a.nitems) return;
    const DiffItem it = diff_item(a, blockIdx.x);
    if (threadIdx.x == 0) bar.init(ST, T);
    if (warp == 8) {
        tmem_alloc(tmem_slot, kCols);
        tmem_relinquish();
    }
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    const uint32_t tmem = *tmem_slot;
    const int32_t *start = a.start + (int64_t)it.b * (a.R + 1) + it.r;
    const int first = __ldg(start);
    const int nq = (__ldg(start + 1) - first) * a.rs;
    const int steps = (nq + T - 1) / T;
    const int32_t *list = a.list + (int64_t)it.b * a.R * a.topk + first;
    const int64_t image = (int64_t)it.b * a.N * a.C + it.h * a.hd;
    const int region = region_at(a, it.r);
    const int tok0 = it.t * 128;

    if (warp >= 9) {
        const Chunk<NB> ch(lane, a.d / 8);
        if (warp == 11) {
            own_rows_and_relay<NB>(a, bar, ch, smem_u32(sOwn), static_cast<const __nv_bfloat16 *>(a.k) + image,
                                   static_cast<const __nv_bfloat16 *>(a.v) + image, region, tok0, lane, steps, ST);
        } else {
            const __nv_bfloat16 *gq = static_cast<const __nv_bfloat16 *>(a.q) + image;
            const __nv_bfloat16 *gd = static_cast<const __nv_bfloat16 *>(a.dout) + image;
            const float4 *stats = a.stats + ((int64_t)it.b * a.heads + it.h) * a.N;
            // 32 rows to a warp: the halves of a tile of 64, every other tile of 32; a row's address is found one
            // tile ahead of its use (it waits for the list)
            const int r0 = T == 64 ? 32 * (warp - 9) : 0, by = T == 64 ? 1 : 2;
            auto locate = [&](int i) {
                const int query = i * T + r0 + lane;
                if (i >= steps || query >= nq) return -1;
                int slot, tok;
                a.by_rs.divmod(query, slot, tok);
                return token_at(a, region_at(a, __ldg(list + slot)), tok);
            };
            int i = T == 64 ? 0 : warp - 9, at = locate(i);
            for (; i < steps; i += by) {
                const int st = i % ST, ahead = locate(i + by);
                if (!mbar_wait(&bar.empty[st], (uint32_t)(((i / ST) & 1) ^ 1), a.err)) break;
                gather_rows<NB>(ch, smem_u32(sRing + (size_t)st * L::kStage), kBlock, r0, at, lane, gq, gd, a.C);
                cp_async16_or_zero(smem_u32(sstat + st * T + r0 + lane), stats + max(at, 0), at >= 0);
                cp_async_arrive(&bar.full[st]);
                at = ahead;
            }
            cp_async_wait_all();
        }
    } else if (warp == 8) {
        constexpr uint32_t kIdescS = umma_idesc_bf16(128, T, false);
        constexpr uint32_t kIdescV = umma_idesc_bf16(128, 64, true), kIdescK = umma_idesc_bf16(128, 32 * NB, true);
        const int all = uniform(steps);
        const uint32_t tm = uniform(tmem), own = uniform(desc_low(smem_u32(sOwn))), ring = uniform(desc_low(smem_u32(sRing)));
        const bool leader = elect_one();
        bool alive = all > 0 && mbar_wait(bar.own_ready, 0, a.err);
        int st = 0, next = 0;
        uint32_t phase = 0;
        auto scores = [&](uint32_t buf) {
            const uint32_t rq = ring + next * (L::kStage >> 4), rd = rq + NB * (kBlock >> 4);
            if (leader) {
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks)
                        umma_ss(tm + kBuf * buf + T * m, own + (NB == 1 ? 4 * m : m * (kOwnBlock >> 4)) + 2 * ks,
                                rq + (NB == 1 ? 4 * m : m * (kBlock >> 4)) + 2 * ks, kIdescS, ks > 0);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        umma_ss(tm + kBuf * buf + 2 * T, own + (NB + nb) * (kOwnBlock >> 4) + 2 * ks, rd + nb * (kBlock >> 4) + 2 * ks,
                                kIdescS, nb > 0 || ks > 0);
            }
            if (++next == ST) {
                next = 0;
                phase ^= 1;
            }
        };
        for (int i = 0; i < 2 && i < all && alive; ++i) {
            if (!(alive = mbar_wait(&bar.ready[next], phase, a.err))) break;
            tcgen05_after_sync();
            scores(i);
            if (leader) umma_commit(&bar.s_full[i]);
            __syncwarp();
        }
        for (int i = 0; i < all && alive; ++i) {
            const uint32_t buf = i & 1;
            if (i + 2 < all) alive = mbar_wait(&bar.ready[next], phase, a.err);
            alive = alive && mbar_wait(&bar.p_full[buf], (uint32_t)((i >> 1) & 1), a.err);
            if (!alive) break;
            tcgen05_after_sync();
            if (leader) {
                const uint32_t rq = ring + st * (L::kStage >> 4), rd = rq + NB * (kBlock >> 4);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int ks = 0; ks < T / 16; ++ks)
                        umma_ts(tm + kAcc + 64 * nb, tm + kBuf * buf + 2 * T + 8 * ks, rd + nb * (kBlock >> 4) + 128 * ks, kIdescV,
                                i > 0 || ks > 0);
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int ks = 0; ks < T / 16; ++ks)
                        umma_ts(tm + kAcc + 64 * NB + 32 * NB * m, tm + kBuf * buf + T * m + 8 * ks,
                                rq + (NB == 1 ? 4 * m : m * (kBlock >> 4)) + 128 * ks, kIdescK, i > 0 || ks > 0);
            }
            if (i + 2 < all) scores(buf);
            if (leader) {
                umma_commit(&bar.s_full[buf]);
                umma_commit(&bar.empty[st]);
            }
            __syncwarp();
            if (++st == ST) st = 0;
        }
        if (leader) umma_commit(bar.drain);
        __syncwarp();
        mbar_wait(bar.drain, 0, a.err);
    } else {
        const int g = warp >> 2, row = 32 * (warp & 3) + lane;
        const uint32_t t_row = tmem + ((uint32_t)(32 * (warp & 3)) << 16), t_s = t_row + kBuf * g;
        const bool busy = tok0 + 32 * (warp & 3) < a.rs;
        const float2 sc = make_float2(-a.scale_log2, -a.scale_log2), minus = make_float2(-1.f, -1.f);
        const float lam = __ldg(a.lam + it.h);
        bool alive = true;
        for (int i = g; i < steps; i += 2) {
            if (!(alive = mbar_wait(&bar.s_full[g], (uint32_t)((i >> 1) & 1), a.err))) break;
            tcgen05_after_sync();
            if (busy) {
                const float4 *st = sstat + (i % ST) * T;
#pragma unroll
                for (int c = 0; c < T; c += 32) {
                    uint32_t s1[32], s2[32], dp[32];
                    tmem_ld_32x32(t_s + c, s1);
                    tmem_ld_32x32(t_s + T + c, s2);
                    tmem_ld_32x32(t_s + 2 * T + c, dp);
                    tmem_wait_ld();
                    uint32_t w1[16], w2[16], wp[16];
#pragma unroll
                    for (int x = 0; x < 32; x += 2) {
                        float2 ds[2];
                        float pc[2];
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const float4 z = st[c + x + y];  // L1, L2, D1, D2 of the column's query
                            const float dpx = __uint_as_float(dp[x + y]);
                            // L - scale S: the exponent's negative
                            const float2 e = __ffma2_rn(make_float2(__uint_as_float(s1[x + y]), __uint_as_float(s2[x + y])), sc,
                                                        make_float2(z.x, z.y));
                            const float2 p = make_float2(fast_exp2(-e.x), fast_exp2(-e.y));
                            ds[y] = __fmul2_rn(p, __ffma2_rn(make_float2(z.z, z.w), minus, make_float2(dpx, dpx)));
                            pc[y] = fmaf(-lam, p.y, p.x);
                        }
                        w1[x / 2] = pack_bf16x2(ds[0].x, ds[1].x);
                        w2[x / 2] = pack_bf16x2(ds[0].y, ds[1].y);
                        wp[x / 2] = pack_bf16x2(pc[0], pc[1]);
                    }
                    if ((i + 1) * T > nq) {  // columns past the last query
#pragma unroll
                        for (int x = 0; x < 16; ++x) {
                            const int query = i * T + c + 2 * x;
                            if (query >= nq) w1[x] = w2[x] = wp[x] = 0u;
                            if (query + 1 == nq) {
                                w1[x] &= 0xffffu;
                                w2[x] &= 0xffffu;
                                wp[x] &= 0xffffu;
                            }
                        }
                    }
                    tmem_st_32x16(t_s + c / 2, w1);
                    tmem_st_32x16(t_s + T + c / 2, w2);
                    tmem_st_32x16(t_s + 2 * T + c / 2, wp);
                }
                tmem_wait_st();
            }
            tcgen05_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.p_full[g]);
        }
        named_barrier(1, 256);  // as in the queries kernel
        if (steps > 0 && alive)
            alive = mbar_wait(&bar.s_full[(steps + 1) & 1], (uint32_t)(((steps + 1) >> 1) & 1), a.err);
        tcgen05_after_sync();
        const bool in = tok0 + row < a.rs;
        const int64_t off = image + (in ? (int64_t)token_at(a, region, tok0 + row) * a.C : 0);
        __nv_bfloat16 *dk = static_cast<__nv_bfloat16 *>(a.dk) + off, *dv = static_cast<__nv_bfloat16 *>(a.dv) + off;
        if (steps == 0) {
            store_zeros(a.hd, g ? dv : dk, in);
        } else if (g == 0) {
            store_columns(t_row + kAcc + 64 * NB, 32 * NB, a.d, a.scale, dk, in && alive);
            store_columns(t_row + kAcc + 64 * NB + 32 * NB, 32 * NB, a.d, -lam * a.scale, dk + a.d, in && alive);
        } else {
            store_columns(t_row + kAcc, 64 * NB, a.hd, 1.f, dv, in && alive);
        }
    }
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    if (warp == 8) tmem_dealloc(tmem, kCols);
}

// Regions whose 128-row tiles are more than half full. This and the mma.sync kernels, backward: 4 regions of 64
// tokens to a query (4 heads of 64) 160 against 142 us, of 81 tokens 212 against 309, of 100 tokens 244 against
// 360; 4 of 100 tokens, heads of 128, 38 against 75.
static_assert(QueryRing<1>::kOwn + QueryRing<1>::kRing >= (kThreads / 32) * (kMaxRegions + 32) * sizeof(int),
              "the queries kernel's shared memory holds invert_index's");
bool diff_backward_umma_supports(const Geometry &g) { return g.hd % 16 == 0 && g.rs > 64; }

namespace {

template <auto Kernel> cudaError_t launch_with(int grid, size_t smem, const DiffArgs &a, cudaStream_t stream)
{
    const cudaError_t e = grant_shared_memory<Kernel>();
    return e == cudaSuccess ? launch_pdl(Kernel, dim3(grid), dim3(kThreads), smem, stream, a) : e;
}

template <int NB> cudaError_t launch_nb(const DiffArgs &a, int grid, cudaStream_t stream)
{
    using Q = QueryRing<NB>;
    using K = typename KeyPlan<NB>::Ring;
    const cudaError_t e = launch_with<diff_backward_queries_umma_kernel<NB>>(
        a.B + grid, 1024 + Q::kOwn + Q::kRing + kBarrierBytes + 2 * 6 * 128 * 4 + 16 + 4 * (size_t)a.topk, a, stream);
    if (e != cudaSuccess) return e;
    return launch_with<diff_backward_keys_umma_kernel<NB>>(
        grid > a.heads ? grid : a.heads,
        1024 + K::kOwn + K::kRing + (size_t)KeyPlan<NB>::kStages * KeyPlan<NB>::kTile * sizeof(float4) + kBarrierBytes + 16, a, stream);
}

}  // namespace

cudaError_t launch_diff_backward_umma(const DiffArgs &args, cudaStream_t stream)
{
    DiffArgs a = args;
    a.tiles = (a.rs + 127) / 128;
    a.by_tiles = FastDiv::of(a.tiles);
    const long long items = (long long)a.B * a.R * a.tiles * a.heads;
    if (items * 4 + a.B > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    a.nitems = (int)items;
    a.nparts = (int)(items / a.heads * 4);
    return a.hd <= 64 ? launch_nb<1>(a, (int)items, stream) : launch_nb<2>(a, (int)items, stream);
}

}  // namespace bra
