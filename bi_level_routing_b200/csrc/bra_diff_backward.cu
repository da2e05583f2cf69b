// bra_diff_backward.cu -- gradients of differential attention for bf16 maps on mma.sync (formula in
// bra_diff.cuh), heads of 8 to 128 channels in multiples of 8, regions of any size.
//
// Nothing is added in memory, so the gradients are the same bits on every run:
//  queries  the first B CTAs list for each region s the regions that route to it, in the order (region,
//           slot); of the others one group of warps per 16 WPI query tokens of an (image, region, head): a first pass over
//           the routed keys takes both softmaxes' running maximum and sum and, with the same
//           rescaling, D_i = rowsum(P_i dP); a second forms dS_i and sums dq_i = dS_i k_i in
//           registers. It leaves L_i = max + log2(sum) and D_i per query, and its sums of D2;
//  keys     one group of warps per 16 WPI key tokens: over the gathered queries of the regions that
//           route to it, P_i = exp2(scale S_i - L_i), then dv += (P1 - lam P2)^T dout and
//           dk_i += dS_i^T q_i in registers. Scores are formed transposed (keys as rows), so that P and
//           dS leave the product as the A fragments of the next one, without shared memory;
//           the launch's first `heads` CTAs also add up dlam from the partial sums.
//
// Precision: S and dP are exact products of bf16 in fp32 sums, statistics and accumulators are
// fp32. P and, for dk, dS enter the last products as bf16. A row's dS sum to 0, so its roundings meet all of k,
// of which dq keeps only what differs between keys: for dq, dS is two bf16 terms. Each gradient is rounded
// to bf16 once.
//
// Few warps and the latency of their gathers bound it: two kernels of 168 registers a thread, three CTAs (12 warps) an
// SM, for heads of up to 64 channels; above, 242 to 255 registers and two CTAs (8 warps). 64 images of 28 x 28, 2 heads of
// 64, 4 regions of 16 tokens to a query: 83 us, of which the queries kernel takes 40, the keys kernel 43; with 8
// regions 175 us. (The lists in a launch of their own: 88.) Regions of less than 16 tokens leave rows of a warp's tile
// empty: 64 images of 14 x 14, 4 heads of 64, 16 regions of 4 tokens 141 us; of 7 x 7, 8 heads, all 49 one-token regions
// 251 us. One CTA sorts an image's index, and where regions are small and many are routed the queries' launch waits
// for it: one image of 256 one-token regions, all routed, 2 heads, 341 us; of 1024, 5.1 ms, of which the sort takes 4.9.
#include "bra_diff.cuh"

#include <algorithm>

namespace bra {

namespace {

constexpr int kWarps = 4;

constexpr int pow2_at_least(int x)
{
    int p = 1;
    while (p < x) p *= 2;
    return p;
}

template <int DK> struct BackTile {
    static constexpr int kHp = 2 * DK;
    static constexpr int kRow = kHp + 8;  // bf16 per row: an odd number of 16-byte chunks
    static constexpr int kLanes = pow2_at_least(kHp / 8);
    static constexpr int kNk = DK / 16;
};

// The A fragments of rows g and g + 8 (in-region tokens tok0 + ...) of a [.., C] array: NF steps of 16
// channels. split: the two halves of d channels are padded to NF / 2 steps each; else hd channels run on.
template <int NF>
__device__ __forceinline__ void load_rows(const DiffArgs &a, const __nv_bfloat16 *base, int region, int tok0, int lane,
                                          bool split, uint32_t (&f)[NF][4])
{
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
        const int tok = tok0 + g + 8 * hh;
        const bool in = tok < a.rs;
        const __nv_bfloat16 *row = base + (int64_t)(in ? token_at(a, region, tok) : 0) * a.C;
#pragma unroll
        for (int ks = 0; ks < NF; ++ks)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                int c = 16 * ks + 8 * half + 2 * t;
                bool real = in;
                if (split) {
                    const int m = ks >= NF / 2;
                    c -= m * 8 * NF;
                    real = in && c < a.d;
                    c += m * a.d;
                } else {
                    real = in && c < a.hd;
                }
                f[ks][hh + 2 * half] = real ? __ldg(reinterpret_cast<const uint32_t *>(row + c)) : 0u;
            }
    }
}

// acc[nt] += A (NF steps of 16 channels) times the transposed rows of a tile (8 rows per nt), whose
// row 0 lies at shared-memory address r0, for NT column tiles; steps from `first`, f holds NF of them.
template <int NF, int ROW>
__device__ __forceinline__ void rows_product(float (&acc)[4], const uint32_t (&f)[NF][4], uint32_t r0, int nt, int lane,
                                             int first, int steps)
{
#pragma unroll
    for (int ks = 0; ks < steps; ks += 2) {
        uint32_t b[4];
        if (ks + 1 < steps) {
            ldmatrix_x4(r0 + ((8 * nt + (lane & 7)) * ROW + 16 * (first + ks) + 8 * (lane >> 3)) * 2, b[0], b[1], b[2], b[3]);
            mma_bf16_16816(acc, f[first + ks], b[0], b[1]);
            mma_bf16_16816(acc, f[first + ks + 1], b[2], b[3]);
        } else {
            // the last step alone: its two 8 x 8 tiles twice, the second pair unused
            ldmatrix_x4(r0 + ((8 * nt + (lane & 7)) * ROW + 16 * (first + ks) + 8 * ((lane >> 3) & 1)) * 2, b[0], b[1], b[2], b[3]);
            mma_bf16_16816(acc, f[first + ks], b[0], b[1]);
        }
    }
}

// One step of 16 rows as the A operand from two score column tiles.
__device__ __forceinline__ void pack_step(uint32_t (&p)[4], const float (&lo)[4], const float (&hi)[4])
{
    p[0] = pack_bf16x2(lo[0], lo[1]);
    p[1] = pack_bf16x2(lo[2], lo[3]);
    p[2] = pack_bf16x2(hi[0], hi[1]);
    p[3] = pack_bf16x2(hi[2], hi[3]);
}

// The same in two bf16 terms: the values with their low 16 bits cleared, and the rest rounded (16 significant bits in all).
__device__ __forceinline__ void split_step(uint32_t (&hi)[4], uint32_t (&lo)[4], const float (&x)[4], const float (&y)[4])
{
    const float v[8] = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = bf16_trunc(v[2 * i]), b = bf16_trunc(v[2 * i + 1]);
        hi[i] = pack_bf16x2_trunc(a, b);
        lo[i] = pack_bf16x2(v[2 * i] - a, v[2 * i + 1] - b);
    }
}

// A warp's 16 accumulator rows, scaled and rounded, through its own shared-memory rows to
// whole-row stores. Column tiles [0, DK / 8) are the first half's channels, the others the second's
// (split) or the channels run on.
template <int DK>
__device__ __forceinline__ void store_rows(const DiffArgs &a, __nv_bfloat16 *base, int region, int tok0, int lane,
                                           __nv_bfloat16 *rows, const float (&acc)[DK / 4][4], bool split, float s0, float s1)
{
    constexpr int ROW = BackTile<DK>::kRow;
    const int g = lane >> 2, t = lane & 3;
    __syncwarp();
#pragma unroll
    for (int nt = 0; nt < DK / 4; ++nt) {
        const float s = nt < DK / 8 ? s0 : s1;
        *reinterpret_cast<uint32_t *>(rows + g * ROW + 8 * nt + 2 * t) = pack_bf16x2(acc[nt][0] * s, acc[nt][1] * s);
        *reinterpret_cast<uint32_t *>(rows + (g + 8) * ROW + 8 * nt + 2 * t) = pack_bf16x2(acc[nt][2] * s, acc[nt][3] * s);
    }
    __syncwarp();
    constexpr int lanes = BackTile<DK>::kLanes;
    const int j = lane % lanes;
    if (8 * j < a.hd) {
        // where the chunk's two groups of four channels stand in the row
        const int c0 = split && 8 * j >= a.d ? DK + 8 * j - a.d : 8 * j;
        const int c1 = split && 8 * j + 4 >= a.d ? DK + 8 * j + 4 - a.d : 8 * j + 4;
        for (int row = lane / lanes; row < 16; row += 32 / lanes) {
            const int tok = tok0 + row;
            if (tok < a.rs) {
                const uint2 lo = *reinterpret_cast<const uint2 *>(rows + row * ROW + c0);
                const uint2 hi = *reinterpret_cast<const uint2 *>(rows + row * ROW + c1);
                *reinterpret_cast<uint4 *>(base + (int64_t)token_at(a, region, tok) * a.C + 8 * j) = make_uint4(lo.x, lo.y, hi.x, hi.y);
            }
        }
    }
}

}  // namespace

// ------------------------------------------------------------------ dq, statistics

// SINGLE: all keys fit one tile (topk rs <= KT), whose scores stay in registers between the passes.
template <int DK, int WPI, int KT, bool SINGLE>
__global__ void __launch_bounds__(32 * kWarps, SINGLE && DK <= 32 ? 3 : 1) diff_backward_queries_kernel(const DiffArgs a)
{
    constexpr int kStages = SINGLE ? 1 : 2;
    using L = BackTile<DK>;
    constexpr int HP = L::kHp, ROW = L::kRow, NK = L::kNk, NT = KT / 8;
    extern __shared__ float4 smem4[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = warp / WPI, wg = warp % WPI;
    const size_t group_bytes = (size_t)2 * kStages * KT * ROW * 2 + (((size_t)a.topk * 4 + 15) & ~(size_t)15) + 16;
    uint8_t *mine = reinterpret_cast<uint8_t *>(smem4) + group * group_bytes;
    __nv_bfloat16 *tiles = reinterpret_cast<__nv_bfloat16 *>(mine);  // [stage][K, V][KT][ROW]
    int *count = reinterpret_cast<int *>(mine + (size_t)2 * kStages * KT * ROW * 2);
    int *bases = count + 4;
    if (blockIdx.x < a.B) {
        grid_dependency_wait();
        invert_index<kWarps>(a, blockIdx.x, reinterpret_cast<int *>(smem4));
        return;
    }
    const int item = (blockIdx.x - a.B) * (kWarps / WPI) + group;
    if (item >= a.nitems) return;  // the whole group: its barriers are its own
    const DiffItem it = diff_item(a, item);
    grid_dependency_wait();

    if (wg == 0) {
        const int n = gather_bases(a, a.idx + ((int64_t)it.b * a.R + it.r) * a.topk, bases, lane);
        if (lane == 0) *count = n;
    }
    group_barrier<WPI>(group);
    const int nkeys = *count * a.rs;
    const int ntiles = (nkeys + KT - 1) / KT;
    const int64_t image = (int64_t)it.b * a.N * a.C + it.h * a.hd;
    const __nv_bfloat16 *gk = static_cast<const __nv_bfloat16 *>(a.k) + image;
    const __nv_bfloat16 *gv = static_cast<const __nv_bfloat16 *>(a.v) + image;
    auto fetch = [&](int tile, int stage) {
        const int j = lane % L::kLanes, r0 = tile * KT + wg * (KT / WPI);
        __nv_bfloat16 *sk = tiles + (size_t)stage * 2 * KT * ROW + wg * (KT / WPI) * ROW, *sv = sk + KT * ROW;
        warp_rows<KT / WPI, L::kLanes>(
            lane,
            [&](int row) {
                if (r0 + row >= nkeys) return -1;
                int slot, tok;
                a.by_rs.divmod(r0 + row, slot, tok);
                return token_at(a, bases[slot], tok);
            },
            [&](int row, int at) {
                if (j >= HP / 8) return;
                const int64_t off = (int64_t)max(at, 0) * a.C;
                copy_split<DK>(smem_u32(sk + row * ROW), gk + off, j, a.d, at >= 0);
                copy_run(smem_u32(sv + row * ROW), gv + off, j, a.hd, at >= 0);
            });
        cp_async_commit();
    };
    if (ntiles > 0) fetch(0, 0);

    const int g = lane >> 2, t = lane & 3;
    const int region = region_at(a, it.r);
    const int tok0 = it.t * 16 * WPI + 16 * wg;
    uint32_t qf[2 * NK][4], df[2 * NK][4];
    load_rows<2 * NK>(a, static_cast<const __nv_bfloat16 *>(a.q) + image, region, tok0, lane, true, qf);
    load_rows<2 * NK>(a, static_cast<const __nv_bfloat16 *>(a.dout) + image, region, tok0, lane, false, df);
    const int vsteps = (a.hd + 15) / 16;

    float s[2][NT][4], dp[NT][4];
    // S1, S2 and dP of the warp's rows against the tile in `stage`
    auto scores = [&](int tile, int stage) {
        const uint32_t k0 = smem_u32(tiles + (size_t)stage * 2 * KT * ROW);
        const uint32_t v0 = k0 + KT * ROW * 2;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < 4; ++i) s[0][nt][i] = s[1][nt][i] = dp[nt][i] = 0.f;
            rows_product<2 * NK, ROW>(s[0][nt], qf, k0, nt, lane, 0, NK);
            rows_product<2 * NK, ROW>(s[1][nt], qf, k0, nt, lane, NK, NK);
#pragma unroll
            for (int ks = 0; ks < 2 * NK; ks += 2) {
                if (ks >= vsteps) break;
                uint32_t b[4];
                ldmatrix_x4(v0 + ((8 * nt + (lane & 7)) * ROW + 16 * ks + 8 * (lane >> 3)) * 2, b[0], b[1], b[2], b[3]);
                mma_bf16_16816(dp[nt], df[ks], b[0], b[1]);
                if (ks + 1 < vsteps) mma_bf16_16816(dp[nt], df[ks + 1], b[2], b[3]);
            }
        }
        if ((tile + 1) * KT > nkeys) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (tile * KT + 8 * nt + 2 * t + (i & 1) >= nkeys) s[0][nt][i] = s[1][nt][i] = -INFINITY;
        }
    };

    float mx[2][2] = {{-INFINITY, -INFINITY}, {-INFINITY, -INFINITY}};
    float l[2][2] = {{0.f, 0.f}, {0.f, 0.f}}, ed[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
    for (int tile = 0; SINGLE ? tile < 1 : tile < ntiles; ++tile) {
        cp_async_wait_all();
        group_barrier<WPI>(group);
        if (!SINGLE && tile + 1 < ntiles) fetch(tile + 1, (tile + 1) & 1);
        if (SINGLE && ntiles == 0) break;  // no tile: nothing was fetched
        scores(tile, tile & 1);
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                float top = -INFINITY;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) top = fmax3(top, s[m][nt][2 * hh], s[m][nt][2 * hh + 1]);
                const float most = fmaxf(mx[m][hh], quad_max(top) * a.scale_log2), base = score_base(most);
                const float corr = fast_exp2(mx[m][hh] - base);
                mx[m][hh] = most;
                float es = 0.f, eds = 0.f;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float e = fast_exp2(fmaf(s[m][nt][2 * hh + i], a.scale_log2, -base));
                        if (SINGLE) s[m][nt][2 * hh + i] = e;
                        es += e;
                        eds = fmaf(e, dp[nt][2 * hh + i], eds);
                    }
                l[m][hh] = l[m][hh] * corr + es;
                ed[m][hh] = ed[m][hh] * corr + eds;
            }
    }
    // L = max + log2(sum) and D of each row; a query without keys takes part in nothing
    float Ls[2][2], D[2][2];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            const float sum = quad_sum(l[m][hh]), num = quad_sum(ed[m][hh]);
            Ls[m][hh] = log_sum(mx[m][hh], sum, nkeys > 0);
            D[m][hh] = over_sum(num, sum, nkeys > 0);
            l[m][hh] = over_sum(1.f, sum, nkeys > 0);
        }
    float dsum = 0.f;
    float4 *stats = a.stats + ((int64_t)it.b * a.heads + it.h) * a.N;
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
        const int tok = tok0 + g + 8 * hh;
        if (tok < a.rs && t == 0) {
            stats[token_at(a, region, tok)] = make_float4(Ls[0][hh], Ls[1][hh], D[0][hh], D[1][hh]);
            dsum += D[1][hh];
        }
    }
    dsum = warp_sum(dsum);
    if (lane == 0)
        a.dlam_part[(int64_t)it.h * a.nparts + (((int64_t)it.b * a.R + it.r) * a.tiles + it.t) * WPI + wg] = dsum;

    float acc[HP / 8][4];
#pragma unroll
    for (int nt = 0; nt < HP / 8; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[nt][i] = 0.f;
    if (!SINGLE && ntiles > 0) {
        group_barrier<WPI>(group);
        fetch(0, 0);
    }
    for (int tile = 0; SINGLE ? tile < (ntiles > 0) : tile < ntiles; ++tile) {
        if (!SINGLE) {
            cp_async_wait_all();
            group_barrier<WPI>(group);
            if (tile + 1 < ntiles) fetch(tile + 1, (tile + 1) & 1);
            scores(tile, tile & 1);
        }
        const uint32_t k0 = smem_u32(tiles + (size_t)(tile & 1) * 2 * KT * ROW);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float p = SINGLE ? s[m][nt][i] * l[m][i >> 1] : fast_exp2(fmaf(s[m][nt][i], a.scale_log2, -Ls[m][i >> 1]));
                    s[m][nt][i] = p * (dp[nt][i] - D[m][i >> 1]);
                }
#pragma unroll
            for (int ks = 0; ks < KT / 16; ++ks) {
                uint32_t hi[4], lo[4];
                split_step(hi, lo, s[m][2 * ks], s[m][2 * ks + 1]);
#pragma unroll
                for (int np = 0; np < DK / 16; ++np) {
                    uint32_t b[4];
                    ldmatrix_x4_trans(k0 + ((16 * ks + (lane & 15)) * ROW + m * DK + 16 * np + 8 * (lane >> 4)) * 2, b[0],
                                      b[1], b[2], b[3]);
                    mma_bf16_16816(acc[m * (DK / 8) + 2 * np], hi, b[0], b[1]);
                    mma_bf16_16816(acc[m * (DK / 8) + 2 * np + 1], hi, b[2], b[3]);
                    mma_bf16_16816(acc[m * (DK / 8) + 2 * np], lo, b[0], b[1]);
                    mma_bf16_16816(acc[m * (DK / 8) + 2 * np + 1], lo, b[2], b[3]);
                }
            }
        }
    }
    group_barrier<WPI>(group);  // every warp has left the tiles: the rows go through them
    const float lam = __ldg(a.lam + it.h);
    store_rows<DK>(a, static_cast<__nv_bfloat16 *>(a.dq) + image, region, tok0, lane, tiles + (size_t)wg * 16 * ROW, acc,
                   true, a.scale, -lam * a.scale);
}

// ------------------------------------------------------------------ dk, dv, dlam

template <int DK, int WPI, int QT>
__global__ void __launch_bounds__(32 * kWarps, DK <= 32 ? 3 : 1) diff_backward_keys_kernel(const DiffArgs a)
{
    using L = BackTile<DK>;
    constexpr int HP = L::kHp, ROW = L::kRow, NK = L::kNk, NT = QT / 8;
    extern __shared__ float4 smem4[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = warp / WPI, wg = warp % WPI, gtid = threadIdx.x % (32 * WPI);
    constexpr size_t kTileBytes = (size_t)4 * QT * ROW * 2;
    constexpr size_t kKeep = 16 * WPI * ROW * 2;  // the rows on their way out, and room for them when QT is small
    constexpr size_t kBytes = (kTileBytes > kKeep ? kTileBytes : kKeep) + 2 * QT * sizeof(float4);
    uint8_t *mine = reinterpret_cast<uint8_t *>(smem4) + group * kBytes;
    __nv_bfloat16 *tiles = reinterpret_cast<__nv_bfloat16 *>(mine);  // [stage][Q, dO][QT][ROW]
    float4 *sstat = reinterpret_cast<float4 *>(mine + kBytes - 2 * QT * sizeof(float4));  // [stage][QT]
    const int item = blockIdx.x * (kWarps / WPI) + group;
    grid_dependency_wait();
    if (group == 0 && blockIdx.x < a.heads) {  // dlam of head blockIdx.x, summed in 64 bits in a fixed order
        double *part = reinterpret_cast<double *>(smem4);
        const float *src = a.dlam_part + (int64_t)blockIdx.x * a.nparts;
        double sum = 0.;
        for (int e = gtid; e < a.nparts; e += 32 * WPI) sum += (double)__ldcg(src + e);
        part[gtid] = sum;
        group_barrier<WPI>(group);
        if (gtid == 0) {
            double all = 0.;
            for (int e = 0; e < 32 * WPI; ++e) all += part[e];
            a.dlam[blockIdx.x] = (float)-all;
        }
        group_barrier<WPI>(group);
    }
    if (item >= a.nitems) return;  // the whole group
    const DiffItem it = diff_item(a, item);
    const int32_t *start = a.start + (int64_t)it.b * (a.R + 1) + it.r;
    const int first = __ldg(start);
    // the gathered queries: their count passes 31 bits only where a region is named more than
    // 2^31 / rs times, which the launcher refuses
    const int nq = (__ldg(start + 1) - first) * a.rs;
    const int ntiles = (nq + QT - 1) / QT;
    const int32_t *list = a.list + (int64_t)it.b * a.R * a.topk + first;
    const int64_t image = (int64_t)it.b * a.N * a.C + it.h * a.hd;
    const __nv_bfloat16 *gq = static_cast<const __nv_bfloat16 *>(a.q) + image;
    const __nv_bfloat16 *gd = static_cast<const __nv_bfloat16 *>(a.dout) + image;
    const float4 *stats = a.stats + ((int64_t)it.b * a.heads + it.h) * a.N;
    auto fetch = [&](int tile, int stage) {
        const int j = lane % L::kLanes, own = wg * (QT / WPI), r0 = tile * QT + own;
        __nv_bfloat16 *sq = tiles + (size_t)stage * 2 * QT * ROW + own * ROW, *sd = sq + QT * ROW;
        warp_rows<QT / WPI, L::kLanes>(
            lane,
            [&](int row) {
                if (r0 + row >= nq) return -1;
                int slot, tok;
                a.by_rs.divmod(r0 + row, slot, tok);
                return token_at(a, region_at(a, __ldg(list + slot)), tok);
            },
            [&](int row, int at) {
                if (j == 0) cp_async16_or_zero(smem_u32(sstat + stage * QT + own + row), stats + max(at, 0), at >= 0);
                if (j >= HP / 8) return;
                const int64_t off = (int64_t)max(at, 0) * a.C;
                copy_split<DK>(smem_u32(sq + row * ROW), gq + off, j, a.d, at >= 0);
                copy_run(smem_u32(sd + row * ROW), gd + off, j, a.hd, at >= 0);
            });
        cp_async_commit();
    };
    if (ntiles > 0) fetch(0, 0);

    const int t = lane & 3;
    const int region = region_at(a, it.r);
    const int tok0 = it.t * 16 * WPI + 16 * wg;
    uint32_t kf[2 * NK][4], vf[2 * NK][4];
    load_rows<2 * NK>(a, static_cast<const __nv_bfloat16 *>(a.k) + image, region, tok0, lane, true, kf);
    load_rows<2 * NK>(a, static_cast<const __nv_bfloat16 *>(a.v) + image, region, tok0, lane, false, vf);
    const int vsteps = (a.hd + 15) / 16;
    const float lam = __ldg(a.lam + it.h);

    float dk[HP / 8][4], dv[HP / 8][4];
#pragma unroll
    for (int nt = 0; nt < HP / 8; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) dk[nt][i] = dv[nt][i] = 0.f;

    for (int tile = 0; tile < ntiles; ++tile) {
        const int stage = tile & 1;
        cp_async_wait_all();
        group_barrier<WPI>(group);
        if (tile + 1 < ntiles) fetch(tile + 1, stage ^ 1);
        const uint32_t q0 = smem_u32(tiles + (size_t)stage * 2 * QT * ROW);
        const uint32_t d0 = q0 + QT * ROW * 2;
        const float4 *st = sstat + stage * QT;

        float s[2][NT][4], dp[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < 4; ++i) s[0][nt][i] = s[1][nt][i] = dp[nt][i] = 0.f;
            rows_product<2 * NK, ROW>(s[0][nt], kf, q0, nt, lane, 0, NK);
            rows_product<2 * NK, ROW>(s[1][nt], kf, q0, nt, lane, NK, NK);
#pragma unroll
            for (int ks = 0; ks < 2 * NK; ks += 2) {
                if (ks >= vsteps) break;
                uint32_t b[4];
                ldmatrix_x4(d0 + ((8 * nt + (lane & 7)) * ROW + 16 * ks + 8 * (lane >> 3)) * 2, b[0], b[1], b[2], b[3]);
                mma_bf16_16816(dp[nt], vf[ks], b[0], b[1]);
                if (ks + 1 < vsteps) mma_bf16_16816(dp[nt], vf[ks + 1], b[2], b[3]);
            }
            // columns 8 nt + 2 t, + 1 are queries
            const float4 st0 = st[8 * nt + 2 * t], st1 = st[8 * nt + 2 * t + 1];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 z = (i & 1) ? st1 : st0;
                const float p1 = fast_exp2(fmaf(s[0][nt][i], a.scale_log2, -z.x));
                const float p2 = fast_exp2(fmaf(s[1][nt][i], a.scale_log2, -z.y));
                s[0][nt][i] = p1 * (dp[nt][i] - z.z);
                s[1][nt][i] = p2 * (dp[nt][i] - z.w);
                dp[nt][i] = fmaf(-lam, p2, p1);
            }
        }
        if ((tile + 1) * QT > nq) {  // rows past the last query
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (tile * QT + 8 * nt + 2 * t + (i & 1) >= nq) s[0][nt][i] = s[1][nt][i] = dp[nt][i] = 0.f;
        }
#pragma unroll
        for (int ks = 0; ks < QT / 16; ++ks) {
            uint32_t pf[4], s1f[4], s2f[4];
            pack_step(pf, dp[2 * ks], dp[2 * ks + 1]);
            pack_step(s1f, s[0][2 * ks], s[0][2 * ks + 1]);
            pack_step(s2f, s[1][2 * ks], s[1][2 * ks + 1]);
#pragma unroll
            for (int np = 0; np < HP / 16; ++np) {
                const uint32_t off = ((16 * ks + (lane & 15)) * ROW + 16 * np + 8 * (lane >> 4)) * 2;
                uint32_t b[4];
                ldmatrix_x4_trans(q0 + off, b[0], b[1], b[2], b[3]);
                mma_bf16_16816(dk[2 * np], np < NK ? s1f : s2f, b[0], b[1]);
                mma_bf16_16816(dk[2 * np + 1], np < NK ? s1f : s2f, b[2], b[3]);
                if (16 * np < a.hd) {
                    ldmatrix_x4_trans(d0 + off, b[0], b[1], b[2], b[3]);
                    mma_bf16_16816(dv[2 * np], pf, b[0], b[1]);
                    mma_bf16_16816(dv[2 * np + 1], pf, b[2], b[3]);
                }
            }
        }
    }
    group_barrier<WPI>(group);
    __nv_bfloat16 *rows = tiles + (size_t)wg * 16 * ROW;
    store_rows<DK>(a, static_cast<__nv_bfloat16 *>(a.dk) + image, region, tok0, lane, rows, dk, true, a.scale,
                   -lam * a.scale);
    store_rows<DK>(a, static_cast<__nv_bfloat16 *>(a.dv) + image, region, tok0, lane, rows, dv, false, 1.f, 1.f);
}

// ------------------------------------------------------------------ launches

namespace {

size_t round16(size_t x) { return (x + 15) & ~(size_t)15; }

template <auto Kernel> cudaError_t launch_with(int grid, size_t smem, const DiffArgs &a, cudaStream_t stream)
{
    const cudaError_t e = grant_shared_memory<Kernel>();
    if (e != cudaSuccess) return e;
    return launch_pdl(Kernel, dim3(grid), dim3(32 * kWarps), smem, stream, a);
}

template <int DK, int WPI, int KT, bool SINGLE> cudaError_t launch_queries(const DiffArgs &a, int grid, cudaStream_t stream)
{
    constexpr int groups = kWarps / WPI;
    const size_t own = groups * ((size_t)(SINGLE ? 2 : 4) * KT * BackTile<DK>::kRow * 2 + round16((size_t)a.topk * 4) + 16);
    return launch_with<diff_backward_queries_kernel<DK, WPI, KT, SINGLE>>(a.B + grid, std::max(own, invert_bytes(kWarps, a.R)), a,
                                                                          stream);
}

// Query tiles of 16 rows: the gradients' accumulators leave no more registers at three CTAs an SM.
template <int DK, int WPI> cudaError_t launch_one(DiffArgs &a, cudaStream_t stream)
{
    constexpr int ROW = BackTile<DK>::kRow, groups = kWarps / WPI, QT = 16;
    a.tiles = (a.rs + 16 * WPI - 1) / (16 * WPI);
    a.by_tiles = FastDiv::of(a.tiles);
    const long long items = (long long)a.B * a.R * a.tiles * a.heads;
    if (items * WPI + a.B > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    a.nitems = (int)items;
    a.nparts = (int)(items / a.heads * WPI);
    const int grid = (int)((items + groups - 1) / groups);
    const cudaError_t e = DK <= 32 && (long long)a.topk * a.rs <= 64 ? launch_queries<DK, WPI, DK <= 32 ? 64 : 32, DK <= 32>(a, grid, stream)
                                                                     : launch_queries<DK, WPI, 32, false>(a, grid, stream);
    if (e != cudaSuccess) return e;
    constexpr size_t tile = (size_t)4 * QT * ROW * 2, keep = (size_t)16 * WPI * ROW * 2;
    return launch_with<diff_backward_keys_kernel<DK, WPI, QT>>(grid > a.heads ? grid : a.heads,
                       groups * ((tile > keep ? tile : keep) + 2 * QT * sizeof(float4)), a, stream);
}

template <int DK> cudaError_t launch_dk(DiffArgs &a, cudaStream_t stream)
{
    if (a.rs <= 16) return launch_one<DK, 1>(a, stream);
    if (a.rs <= 32) return launch_one<DK, 2>(a, stream);
    return launch_one<DK, 4>(a, stream);
}

}  // namespace

// The query kernels' launches: the partial sums of D2 for each head, one for each warp's rows.
long long diff_backward_parts(const Geometry &g, DiffBackward kernels)
{
    long long per;
    if (kernels == DiffBackward::kUmma)
        per = 4LL * ((g.rs + 127) / 128);
    else if (kernels == DiffBackward::kMma)
        per = g.rs <= 16 ? 1 : g.rs <= 32 ? 2 : 4LL * ((g.rs + 63) / 64);
    else
        per = g.rs <= 16 ? 4 : (long long)diff_simt_warps(g.topk, g.rs) * ((g.rs + 31) / 32);
    return (long long)g.B * g.R * per;
}

void diff_plan(DiffArgs &a, const Geometry &g)
{
    a.B = g.B;
    a.H = g.H;
    a.W = g.W;
    a.C = g.C;
    a.heads = g.heads;
    a.hd = g.hd;
    a.d = g.hd / 2;
    a.n_win = g.n_win;
    a.hr = g.hr;
    a.wr = g.wr;
    a.rs = g.rs;
    a.R = g.R;
    a.topk = g.topk;
    a.N = g.N;
    a.scale = (float)(1.0 / sqrt((double)a.d));
    a.scale_log2 = (float)(1.4426950408889634 / sqrt((double)a.d));
    a.by_rs = FastDiv::of(g.rs);
    a.by_wr = FastDiv::of(g.wr);
    a.by_nwin = FastDiv::of(g.n_win);
    a.by_heads = FastDiv::of(g.heads);
    a.by_R = FastDiv::of(g.R);
    a.by_topk = FastDiv::of(g.topk);
}

cudaError_t launch_diff_backward_mma(const DiffArgs &args, cudaStream_t stream)
{
    DiffArgs a = args;
    if (a.d <= 16) return launch_dk<16>(a, stream);
    if (a.d <= 32) return launch_dk<32>(a, stream);
    if (a.d <= 48) return launch_dk<48>(a, stream);
    return launch_dk<64>(a, stream);
}

}  // namespace bra
