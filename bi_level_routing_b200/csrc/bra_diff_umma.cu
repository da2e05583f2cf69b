// bra_diff_umma.cu -- forward differential attention of bf16 maps on the 5th-generation tensor cores
// (tcgen05, TMEM accumulators), for heads of 16 to 128 channels in multiples of 16 and large regions (see
// bra_diff.cuh for the formula). Heads are padded with zeros to 64 or 128 channels. Two exponentials a query-key
// pair against 6 hd tensor operations: the exponential unit (16 a cycle and SM) is the bound, 1024 cycles for 128
// queries and 64 keys; 16384-token maps (2 images, 2 heads of 64) take 749 us, of which that unit's share is 390.
//
// A CTA owns 128 query tokens of one (image, region, head) and meets the routed keys in tiles of KT: 32 for heads
// of up to 64 channels, whose accumulators leave room in TMEM for two CTAs on an SM (four softmax warps a
// scheduler; one CTA with tiles of 64 takes 776 us there, and 43 instead of 35 us on 256-token regions),
// 64 for larger heads.
//  * warps 0-3 are map 1's softmax, warps 4-7 map 2's; thread t of either owns query row t, i.e. TMEM
//    lane t. It takes its row's scores, follows the running maximum, writes the probabilities as bf16
//    over the first half of its scores, and keeps the row's sum in fp32. The accumulator in TMEM
//    is rescaled only when a row's maximum has grown by more than 2^8 (the probabilities stay relative
//    to an older maximum until then: exact, and far from overflow), so PV products accumulate in place;
//  * warp 8: one elected lane issues the products. S_m = Q_m K_m^T (M = 128, N = KT, K = hd / 2) and
//    O_m += P_m V (M = 128, N = 64 a block, K = KT; P from TMEM). Each map has two score buffers: the
//    scores of the next tile are there when the softmax comes to them;
//  * warps 9-10 gather the key and value rows of the routed regions into a ring of stages by cp.async,
//    128-byte swizzled; regions of any size pack densely, rows past the last key are zeros. A lane finds
//    the address of one row, eight lanes copy it. Warp 11 gathers the query rows and hands the
//    tiles that have landed to warp 8.
// Where there are too few (query tile, head) pairs for the GPU, SPLIT: several CTAs share one, each with a run of its
// keys, and leave both maps' sums of P V, maxima and sums, which a second kernel joins.
// Every wait is bounded (kErrTimeout); no thread leaves before the TMEM is released.
#include "bra_diff.cuh"

namespace bra {

namespace {

constexpr int kThreads = 384;
// Pairs of exponentials out of 32 that go to the exponential unit; the others are polynomials on the FMA
// pipe (16384-token map, 2 images of 2 heads of 64: all 32 778 us, 26 749 us, 20 767 us).
constexpr int kUnitPairs = 26;
constexpr int kQBlock = 128 * 128;       // 128 rows x 64 channels
constexpr int kBarrierBytes = 512;       // room for the mbarriers
constexpr float kGrowth = 8.f;           // log2 of the growth of a maximum that rescales the accumulator

// NB: 64-channel blocks of a head; KT: keys of a tile. TMEM: S of map m, buffer u at KT (2 m + u), O1 at
// 4 KT, O2 after it.
template <int NB, int KT> struct UmmaTile {
    static constexpr int kStages = NB == 1 ? 8 : 5;
    static constexpr int kBlock = KT * 128;
    static constexpr uint32_t kCols = 4 * KT + 128 * NB <= 256 ? 256 : 512;  // an allocation is a power of two
    static size_t bytes(int topk)
    {
        return 1024 + (size_t)NB * (kQBlock + 2 * kStages * kBlock) + kBarrierBytes + 1024 + 16 + 4 * (size_t)topk;
    }
};

}  // namespace

template <int NB, int KT, bool SPLIT>
__global__ void __launch_bounds__(kThreads, KT == 32 ? 2 : 1) diff_attend_umma_kernel(const DiffArgs a)
{
    using L = UmmaTile<NB, KT>;
    constexpr int ST = L::kStages, KS = 2 * NB;  // KS: 16-channel steps of a half head
    constexpr int kBlock = L::kBlock, W = KT / 32;
    constexpr uint32_t kCols = L::kCols;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sQ = smem, *sKV = smem + kQBlock * NB;  // [stage][K, V][NB]
    uint64_t *q_full = reinterpret_cast<uint64_t *>(sKV + (size_t)ST * 2 * NB * kBlock);
    uint64_t *q_ready = q_full + 1, *kv_full = q_ready + 1, *kv_ready = kv_full + ST, *kv_empty = kv_ready + ST;
    uint64_t *s_full = kv_empty + ST;  // [map][buffer]
    uint64_t *p_full = s_full + 4;     // [map][buffer]
    uint64_t *drain = p_full + 4;
    float *sum = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(q_full) + kBarrierBytes);  // [2][128]
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sum + 256);
    int *count = reinterpret_cast<int *>(tmem_slot + 1);
    int *bases = count + 3;
    const int warp = uniform((int)(threadIdx.x >> 5)), lane = threadIdx.x & 31;
    int item = blockIdx.x, split = 0;
    if (SPLIT) a.by_splits.divmod(blockIdx.x, item, split);
    const DiffItem it = diff_item(a, item);

    if (threadIdx.x == 0) {
        mbar_init(q_full, 32);
        mbar_init(q_ready, 1);
        for (int i = 0; i < ST; ++i) {
            mbar_init(&kv_full[i], KT);
            mbar_init(&kv_ready[i], 1);
            mbar_init(&kv_empty[i], 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
        }
        mbar_init(drain, 1);
        mbar_fence_init();
    }
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
    const int key0 = SPLIT ? split * a.per : 0;  // this CTA's first key
    const int nkeys = SPLIT ? min(max(*count * a.rs - key0, 0), a.per) : *count * a.rs;
    const int ntiles = (nkeys + KT - 1) / KT;
    const int64_t image = (int64_t)it.b * a.N * a.C + it.h * a.hd;
    const int region = region_at(a, it.r);
    const int tok0 = it.t * 128;

    if (warp >= 9) {
        // ------------------------------------------------------------- gather
        const int j = lane & 7, sub = lane >> 3;  // this lane's 16-byte chunk (of each block) of rows 4 x + sub
        // where that chunk comes from: halves of d channels padded with zeros to 32 NB for q and k, hd
        // channels padded to 64 NB for v
        const int dc = a.d / 8;
        int c_half[NB];
        bool in_half[NB], in_v[NB];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const int c = j + 8 * nb, m = c / (4 * NB), x = c % (4 * NB);
            in_half[nb] = x < dc;
            c_half[nb] = in_half[nb] ? 8 * (m * dc + x) : 0;
            in_v[nb] = c < 2 * dc;
        }
        if (warp == 11) {
            const __nv_bfloat16 *gq = static_cast<const __nv_bfloat16 *>(a.q) + image;
            for (int r0 = 0; r0 < 128; r0 += 32) {
                const int at = tok0 + r0 + lane < a.rs ? token_at(a, region, tok0 + r0 + lane) : -1;
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const int row = r0 + 4 * x + sub, tok = __shfl_sync(0xffffffffu, at, 4 * x + sub);
                    const __nv_bfloat16 *src = gq + (int64_t)max(tok, 0) * a.C;
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
                        cp_async16_or_zero(smem_u32(sQ + nb * kQBlock) + sw128(row, j), src + c_half[nb], tok >= 0 && in_half[nb]);
                }
            }
            cp_async_arrive(q_full);
            // The copies are generic writes: between their landing and the products' reads stands a proxy
            // fence. Here it holds up nothing but this warp (on the copying side it waits for
            // every copy in flight, on the issuing side it takes 200 cycles a tile).
            bool alive = ntiles > 0 && mbar_wait(q_full, 0, a.err);
            fence_async_shared();
            if (lane == 0 && alive) mbar_arrive(q_ready);
            for (int i = 0; i < ntiles && alive; ++i) {
                alive = mbar_wait(&kv_full[i % ST], (uint32_t)((i / ST) & 1), a.err);
                fence_async_shared();
                __syncwarp();
                if (lane == 0 && alive) mbar_arrive(&kv_ready[i % ST]);
            }
        } else {
            // 32 rows to a warp: the halves of a tile of 64, every other tile of 32
            const __nv_bfloat16 *gk = static_cast<const __nv_bfloat16 *>(a.k) + image;
            const __nv_bfloat16 *gv = static_cast<const __nv_bfloat16 *>(a.v) + image;
            const int r0 = KT == 64 ? 32 * (warp - 9) : 0;
            for (int i = KT == 64 ? 0 : warp - 9; i < ntiles; i += KT == 64 ? 1 : 2) {
                const int st = i % ST, key = i * KT + r0 + lane;
                int at = -1;
                if (key < nkeys) {
                    int slot, tok;
                    a.by_rs.divmod(key0 + key, slot, tok);
                    at = token_at(a, bases[slot], tok);
                }
                if (!mbar_wait(&kv_empty[st], (uint32_t)(((i / ST) & 1) ^ 1), a.err)) break;
                const uint32_t sk = smem_u32(sKV + (size_t)st * 2 * NB * kBlock);
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const int tok = __shfl_sync(0xffffffffu, at, 4 * x + sub);
                    const int64_t off = (int64_t)max(tok, 0) * a.C;
                    const uint32_t dst = sk + sw128(r0 + 4 * x + sub, j);
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
                        cp_async16_or_zero(dst + nb * kBlock, gk + off + c_half[nb], tok >= 0 && in_half[nb]);
                        cp_async16_or_zero(dst + (NB + nb) * kBlock, gv + off + (in_v[nb] ? 8 * j + 64 * nb : 0),
                                           tok >= 0 && in_v[nb]);
                    }
                }
                cp_async_arrive(&kv_full[st]);
            }
        }
        cp_async_wait_all();
    } else if (warp == 8) {
        // ------------------------------------------------------------- products
        constexpr uint32_t kIdescS = umma_idesc_bf16(128, KT, false);
        constexpr uint32_t kIdescPV = umma_idesc_bf16(128, 64, true);
        const int nt = uniform(ntiles);
        const uint32_t tm = uniform(tmem), dq = uniform(desc_low(smem_u32(sQ))), dkv = uniform(desc_low(smem_u32(sKV)));
        const bool leader = elect_one();
        bool alive = nt > 0 && mbar_wait(q_ready, 0, a.err);
        int st = 0, next = 0;  // stages of tile i and of the next tile to form scores of
        uint32_t phase = 0;
        auto scores = [&](int m, uint32_t buf) {  // half m's channels: 64 bytes on in the same rows, or the next block
            const uint32_t hq = NB == 1 ? 4 * m : m * (kQBlock >> 4), hk = NB == 1 ? 4 * m : m * (kBlock >> 4);
            const uint32_t dk = dkv + next * (2 * NB * (kBlock >> 4)) + hk;
            if (leader) {
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
                    umma_ss(tm + KT * (2 * m + buf), dq + hq + 2 * ks, dk + 2 * ks, kIdescS, ks > 0);
            }
        };
        auto advance = [&] {
            if (++next == ST) {
                next = 0;
                phase ^= 1;
            }
        };
        for (int i = 0; i < 2 && i < nt && alive; ++i) {
            if (!(alive = mbar_wait(&kv_ready[next], phase, a.err))) break;
            tcgen05_after_sync();
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                scores(m, i);
                if (leader) umma_commit(&s_full[2 * m + i]);
            }
            __syncwarp();
            advance();
        }
        for (int i = 0; i < nt && alive; ++i) {
            const uint32_t buf = i & 1;
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                if (m == 0 && i + 2 < nt) alive = alive && mbar_wait(&kv_ready[next], phase, a.err);
                alive = alive && mbar_wait(&p_full[2 * m + buf], (uint32_t)((i >> 1) & 1), a.err);
                if (!alive) break;
                tcgen05_after_sync();
                const uint32_t dv = dkv + (st * 2 * NB + NB) * (kBlock >> 4);
                if (leader) {
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                        for (int ks = 0; ks < KT / 16; ++ks)
                            umma_ts(tm + 4 * KT + 64 * (NB * m + nb), tm + KT * (2 * m + buf) + 8 * ks,
                                    dv + nb * (kBlock >> 4) + 128 * ks, kIdescPV, i > 0 || ks > 0);
                }
                // the tile after next takes the buffer whose probabilities were just read (products of one
                // thread run in the order of their issue); the commit says that O_m holds tile i, too
                if (i + 2 < nt) scores(m, buf);
                if (leader) {
                    umma_commit(&s_full[2 * m + buf]);
                    if (m == 1) umma_commit(&kv_empty[st]);
                }
                __syncwarp();
            }
            if (i + 2 < nt) advance();
            if (++st == ST) st = 0;
        }
        // wait for the last commit, so that no arrival lands after this CTA has left
        if (leader) umma_commit(drain);
        __syncwarp();
        mbar_wait(drain, 0, a.err);
    } else {
        // ------------------------------------------------------------- softmax
        const int m = warp >> 2, row = 32 * (warp & 3) + lane;
        const uint32_t t_row = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        const uint32_t t_o = t_row + 4 * KT + 64 * NB * m;
        float mx = -INFINITY, l = 0.f;
        bool alive = true;
        const float2 sc = make_float2(a.scale_log2, a.scale_log2);
        for (int i = 0; i < ntiles; ++i) {
            const uint32_t t_s = t_row + KT * (2 * m + (i & 1));
            if (!(alive = mbar_wait(&s_full[2 * m + (i & 1)], (uint32_t)((i >> 1) & 1), a.err))) break;
            tcgen05_after_sync();
            // The exponentials are taken relative to the maximum so far while this tile's own is still
            // being found; only where it has grown past kGrowth are they taken again.
            uint32_t pw[KT / 2];
            float t;
            float2 ls[2];
            auto probabilities = [&](float base) {
                uint32_t v[W][32];
#pragma unroll
                for (int c = 0; c < W; ++c) tmem_ld_32x32(t_s + 32 * c, v[c]);
                tmem_wait_ld();
                if ((i + 1) * KT > nkeys) {
#pragma unroll
                    for (int c = 0; c < W; ++c)
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            if (i * KT + 32 * c + x >= nkeys) v[c][x] = 0xff800000u;
                }
                const float2 nm = make_float2(base, base);
                float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                ls[0] = ls[1] = make_float2(0.f, 0.f);
#pragma unroll
                for (int x = 0; x < KT / 2; ++x) {
                    const float s0 = __uint_as_float(v[x / 16][(2 * x) % 32]), s1 = __uint_as_float(v[x / 16][(2 * x) % 32 + 1]);
                    const float2 e = __ffma2_rn(make_float2(s0, s1), sc, nm);
                    const float2 p = x * kUnitPairs % 32 < kUnitPairs ? make_float2(fast_exp2(e.x), fast_exp2(e.y)) : poly_exp2(e);
                    top[x & 3] = fmax3_nan(top[x & 3], s0, s1);
                    ls[x & 1] = __fadd2_rn(ls[x & 1], p);
                    pw[x] = pack_bf16x2(p.x, p.y);
                }
                t = fmax3_nan(fmax3_nan(top[0], top[1], top[2]), top[3], top[3]) * a.scale_log2;
            };
            probabilities(mx == -INFINITY ? 0.f : -mx);
            const bool grown = t > mx + kGrowth || (mx == -INFINITY && t != -INFINITY);
            if (__any_sync(0xffffffffu, grown)) {
                const float corr = grown ? fast_exp2(mx - t) : 1.f;
                if (grown) {
                    mx = t;
                    l *= corr;
                }
                if (i > 0) {  // O_m holds the tiles before this one once the next one's scores are there
                    if (!(alive = mbar_wait(&s_full[2 * m + ((i + 1) & 1)], (uint32_t)(((i + 1) >> 1) & 1), a.err))) break;
                    tcgen05_after_sync();
#pragma unroll
                    for (int c = 0; c < 2 * NB; ++c) {
                        uint32_t o[32];
                        tmem_ld_32x32(t_o + 32 * c, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * corr);
                        tmem_st_32x32(t_o + 32 * c, o);
                    }
                    tmem_wait_st();
                }
                probabilities(mx == -INFINITY ? 0.f : -mx);
            }
            if constexpr (KT == 64)
                tmem_st_32x32(t_s, pw);
            else
                tmem_st_32x16(t_s, pw);
            tmem_wait_st();
            const float2 add = __fadd2_rn(ls[0], ls[1]);
            l += t < INFINITY ? add.x + add.y : NAN;  // a NaN or +inf score makes its row NaN
            tcgen05_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[2 * m + (i & 1)]);
        }
        if constexpr (SPLIT) {
            // A sum of -1 is a CTA without keys; scores that are all -inf have a sum of 0 (the polynomial's least values are
            // not one), or NaN where one was NaN.
            const int64_t part = 2 * (int64_t)blockIdx.x + m;
            if (alive && ntiles > 0)
                alive = mbar_wait(&s_full[2 * m + ((ntiles + 1) & 1)], (uint32_t)(((ntiles + 1) >> 1) & 1), a.err);
            tcgen05_after_sync();
            if (alive) a.split_stats[part * 128 + row] = make_float2(mx, ntiles == 0 ? -1.f : mx == -INFINITY && l == l ? 0.f : l);
            float4 *dst = a.split_out + part * (16 * NB * 128) + row;
#pragma unroll
            for (int c = 0; c < 2 * NB; ++c) {
                if (ntiles == 0) break;
                uint32_t o[32];
                tmem_ld_32x32(t_o + 32 * c, o);
                tmem_wait_ld();
                if (!alive) continue;
#pragma unroll
                for (int x = 0; x < 8; ++x)
                    dst[(8 * c + x) * 128] = make_float4(__uint_as_float(o[4 * x]), __uint_as_float(o[4 * x + 1]),
                                                         __uint_as_float(o[4 * x + 2]), __uint_as_float(o[4 * x + 3]));
            }
        } else {
            // out = O1 / l1 - lam O2 / l2: thread `row` of map m's warps writes half m of the row's channels
            sum[128 * m + row] = mx == -INFINITY ? 0.f : l;  // only -inf scores: the polynomial's least values are not a sum
            named_barrier(1, 256);
            for (int x = 0; x < 2 && ntiles > 0 && alive; ++x)  // the commit after the last tile's products
                alive = mbar_wait(&s_full[2 * x + ((ntiles + 1) & 1)], (uint32_t)(((ntiles + 1) >> 1) & 1), a.err);
            tcgen05_after_sync();
            const float l1 = sum[row], l2 = sum[128 + row], lam = __ldg(a.lam + it.h);
            const float w1 = over_sum(1.f, l1, nkeys > 0), w2 = over_sum(-lam, l2, nkeys > 0);
            const bool in = tok0 + row < a.rs;
            __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + image + 32 * NB * m;
            if (in) out += (int64_t)token_at(a, region, tok0 + row) * a.C;
#pragma unroll
            for (int c = 0; c < NB; ++c) {
                uint32_t o1[32], o2[32];
                if (ntiles > 0) {  // the same for the whole CTA: tcgen05.ld is warp-wide
                    tmem_ld_32x32(t_row + 4 * KT + 32 * NB * m + 32 * c, o1);
                    tmem_ld_32x32(t_row + 4 * KT + 64 * NB + 32 * NB * m + 32 * c, o2);
                    tmem_wait_ld();
                }
                if (!in || !alive) continue;
#pragma unroll
                for (int x = 0; x < 32; x += 8) {
                    uint32_t pk[4];
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const int z = x + 2 * y;
                        const float u = fmaf(__uint_as_float(o1[z]), w1, __uint_as_float(o2[z]) * w2);
                        const float w = fmaf(__uint_as_float(o1[z + 1]), w1, __uint_as_float(o2[z + 1]) * w2);
                        pk[y] = ntiles > 0 ? pack_bf16x2(u, w) : 0u;
                    }
                    if (32 * NB * m + 32 * c + x < a.hd) *reinterpret_cast<uint4 *>(out + 32 * c + x) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                }
            }
        }
    }
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    if (warp == 8) tmem_dealloc(tmem, kCols);
}

// A CTA joins 4 channels of an item's 128 rows, a row to a thread: each map's splits relative to the largest of their
// maxima, then out = O1 / l1 - lam O2 / l2. Latency bounds it: the loads of kBatch splits of both maps are all in
// flight at once (one split after the other took 11 us for eight splits of 4096 rows).
template <int NB> __global__ void __launch_bounds__(128) diff_attend_join_kernel(const DiffArgs a)
{
    constexpr int kBatch = 8;
    const int item = blockIdx.x / (a.hd / 4), chunk = blockIdx.x - item * (a.hd / 4);
    const int row = threadIdx.x;
    const DiffItem it = diff_item(a, item);
    grid_dependency_wait();
    const int tok = it.t * 128 + row;
    if (tok >= a.rs) return;
    const float2 *stats = a.split_stats + (int64_t)item * a.splits * 256 + row;
    const float4 *part = a.split_out + (int64_t)item * a.splits * (2 * 16 * NB * 128) + chunk * 128 + row;
    const float lam = __ldg(a.lam + it.h);
    float top[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float4 x[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
    bool some = false;
    for (int s0 = 0; s0 < a.splits; s0 += kBatch) {
        float2 st[kBatch][2];
        float4 o[kBatch][2];
#pragma unroll
        for (int s = 0; s < kBatch; ++s)
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const bool in = s0 + s < a.splits;
                st[s][m] = in ? __ldcg(stats + (2 * (s0 + s) + m) * 128) : make_float2(-INFINITY, -1.f);
                o[s][m] = in ? __ldcg(part + (int64_t)(2 * (s0 + s) + m) * (16 * NB * 128)) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            float most = top[m];
#pragma unroll
            for (int s = 0; s < kBatch; ++s) most = fmaxf(most, st[s][m].x);
            const float corr = top[m] == -INFINITY ? 1.f : fast_exp2(top[m] - most);  // at first there is nothing to scale but 0
            top[m] = most;
            l[m] *= corr;
            x[m] = make_float4(x[m].x * corr, x[m].y * corr, x[m].z * corr, x[m].w * corr);
#pragma unroll
            for (int s = 0; s < kBatch; ++s) {
                if (st[s][m].y == -1.f) continue;
                some = true;
                const float w = st[s][m].x == -INFINITY ? 0.f : fast_exp2(st[s][m].x - most);
                l[m] += st[s][m].x == -INFINITY ? st[s][m].y : st[s][m].y * w;
                x[m].x = fmaf(o[s][m].x, w, x[m].x);
                x[m].y = fmaf(o[s][m].y, w, x[m].y);
                x[m].z = fmaf(o[s][m].z, w, x[m].z);
                x[m].w = fmaf(o[s][m].w, w, x[m].w);
            }
        }
    }
    const float w1 = over_sum(1.f, l[0], some), w2 = over_sum(-lam, l[1], some);
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + ((int64_t)it.b * a.N + token_at(a, region_at(a, it.r), tok)) * a.C +
                         it.h * a.hd + 4 * chunk;
    *reinterpret_cast<uint2 *>(out) = make_uint2(pack_bf16x2(fmaf(x[0].x, w1, x[1].x * w2), fmaf(x[0].y, w1, x[1].y * w2)),
                                                 pack_bf16x2(fmaf(x[0].z, w1, x[1].z * w2), fmaf(x[0].w, w1, x[1].w * w2)));
}

// Any head the register-tiled kernel takes; regions whose query tiles are more than half full, or just
// half with many keys. Both kernels, heads of 64: 4 regions of 64 tokens to a query 36.5 against 41.4 us (16
// images of 16 regions, 4 heads), of 100 tokens 50.8 against 112, of 144 117 against 215; but one
// region of 64 tokens (64 images of 49 regions) 64 against 48.
bool diff_umma_supports(const Geometry &g)
{
    return g.hd % 16 == 0 && (g.rs > 64 || (g.rs == 64 && g.topk >= 4));
}

namespace {

template <int NB, int KT> cudaError_t launch_nb(const DiffArgs &a, int items, cudaStream_t stream)
{
    constexpr auto whole = diff_attend_umma_kernel<NB, KT, false>, part = diff_attend_umma_kernel<NB, KT, true>;
    const bool split = a.splits > 1;
    cudaError_t e = split ? grant_shared_memory<part>() : grant_shared_memory<whole>();
    if (e != cudaSuccess) return e;
    e = launch_pdl(split ? part : whole, dim3(items * a.splits), dim3(kThreads), UmmaTile<NB, KT>::bytes(a.topk), stream, a);
    if (e != cudaSuccess || !split) return e;
    return launch_pdl(diff_attend_join_kernel<NB>, dim3(items * (a.hd / 4)), dim3(128), 0, stream, a);
}

constexpr int key_tile(int hd) { return hd <= 64 ? 32 : 64; }
// Key tiles of a split, at least. One image of one head of 64, whole map: 64 x 64 tokens 68 us in one piece, 28 in splits of
// 16 tiles (29 of 14); 128 x 128 246 and 225. Below, the second launch costs what the split gains: 4 heads of 128,
// 32 x 32 tokens 20.3 in one piece, 17.8 in splits of 4, but 8 regions of 64 tokens to a query (56 x 56, 2 heads) 13.1 and 18.4.
constexpr int kLeastTiles = 16;

// Keys of a split: whole tiles.
int split_keys(int hd, int topk, int rs, int splits)
{
    const int kt = key_tile(hd), tiles = (int)(((long long)topk * rs + kt - 1) / kt);
    return (tiles + splits - 1) / splits * kt;
}

}  // namespace

// One round of the GPU: as many CTAs as fit, kLeastTiles key tiles or more to each.
int diff_umma_splits(const Geometry &g, int num_sms, size_t *scratch)
{
    *scratch = 0;
    const long long items = (long long)g.B * g.R * ((g.rs + 127) / 128) * g.heads;
    const int kt = key_tile(g.hd), nb = g.hd <= 64 ? 1 : 2;
    const long long tiles = ((long long)g.topk * g.rs + kt - 1) / kt;
    long long splits = (long long)num_sms * (nb == 1 ? 2 : 1) / items;
    if (splits > tiles / kLeastTiles) splits = tiles / kLeastTiles;
    if (splits < 2) return 1;
    const int per = split_keys(g.hd, g.topk, g.rs, (int)splits) / kt;
    splits = (tiles + per - 1) / per;
    *scratch = (size_t)(items * splits) * 2 * 128 * (16 * nb * sizeof(float4) + sizeof(float2));
    return (int)splits;
}

cudaError_t launch_diff_attend_umma(const DiffArgs &args, cudaStream_t stream)
{
    DiffArgs a = args;
    a.tiles = (a.rs + 127) / 128;
    a.by_tiles = FastDiv::of(a.tiles);
    const long long items = (long long)a.B * a.R * a.tiles * a.heads;
    if (items > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    a.nitems = (int)items;
    a.by_splits = FastDiv::of(a.splits);
    a.per = split_keys(a.hd, a.topk, a.rs, a.splits);
    return a.hd <= 64 ? launch_nb<1, 32>(a, (int)items, stream) : launch_nb<2, 64>(a, (int)items, stream);
}

}  // namespace bra
