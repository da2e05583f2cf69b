// bra_diff_simt.cu -- differential attention and its gradients of fp32 maps on CUDA cores (formula in bra_diff.cuh), hd a
// multiple of 8 up to 128, regions of any size: 6 hd operations a query-key pair forward (4 hd are due; the two maps'
// sums run apart), 18 hd backward (10 hd are due; both passes score again, one of them twice).
//
// A CTA owns WARPS x RW token rows of one (image, region, head), RW of them a warp's; the tokens they
// meet (keys for the forward pass and dq, queries for dk and dv) come through shared memory in tiles of
// 64, two to a lane. Scores: a lane holds two rows of the tile against the warp's RW rows, whose
// channels are read as broadcasts (RW + 8 shared-memory wavefronts for 8 RW FMAs of a warp, so the
// FMA pipe is the bound from RW = 8 on). The products with the tile's channels turn round: lanes
// over channels, the probabilities of four tile rows read as one broadcast.
// As in bra_diff_backward.cu, nothing is added in memory. Forward, 4 images of 45 x 35, 2 heads of 48, 3 regions
// of 63 tokens to a query: 46 us, a third of the FMA rate. Many keys take warps of four rows, for which both products are
// bound by shared memory (12 wavefronts for 8 cycles of FMA, 8 for 4), and heads of 128 one CTA of eight warps an SM in
// the backward pass: 4 whole maps of 17 x 54, 4 heads of 128, 610 us forward and 2050 us backward, 15
// and 11 % of that rate by the operations due.
#include "bra_diff.cuh"

#include <algorithm>

namespace bra {

namespace {

constexpr int kTileRows = 64;

template <int WARPS, int RW> struct SimtTile {
    static constexpr int kRows = WARPS * RW;
    // floats of shared memory: two tiles, two sets of own rows, NP score planes of each warp
    static size_t floats(int hd, int own, int planes)
    {
        return (size_t)(2 * kTileRows + own * kRows) * (hd + 4) + (size_t)WARPS * planes * RW * kTileRows;
    }
};

// Channels 4 u .. of row `row` of a [rows][hd + 4] tile, or zeros.
__device__ __forceinline__ void stage_vector(float *tile, int hd, int row, int u, const float *src, bool real)
{
    *reinterpret_cast<float4 *>(tile + row * (hd + 4) + 4 * u) =
        real ? __ldg(reinterpret_cast<const float4 *>(src) + u) : make_float4(0.f, 0.f, 0.f, 0.f);
}

// acc[i][0..1] += rows[i] . tile[lane], tile[lane + 32] over channels [c0, c1); packed over pairs of channels
template <int RW>
__device__ __forceinline__ void lane_products(float (&acc)[RW][2], const float *rows, const float *tile, int hd, int lane,
                                              int c0, int c1)
{
    const float *t0 = tile + lane * (hd + 4), *t1 = t0 + 32 * (hd + 4);
    float2 s[RW][2];
#pragma unroll
    for (int i = 0; i < RW; ++i) s[i][0] = s[i][1] = make_float2(0.f, 0.f);
#pragma unroll (RW == 8 ? 1 : 2)
    for (int c = c0; c < c1; c += 4) {
        const float4 x = *reinterpret_cast<const float4 *>(t0 + c), y = *reinterpret_cast<const float4 *>(t1 + c);
#pragma unroll
        for (int i = 0; i < RW; ++i) {
            const float4 q = *reinterpret_cast<const float4 *>(rows + i * (hd + 4) + c);
            const float2 lo = make_float2(q.x, q.y), hi = make_float2(q.z, q.w);
            s[i][0] = __ffma2_rn(lo, make_float2(x.x, x.y), __ffma2_rn(hi, make_float2(x.z, x.w), s[i][0]));
            s[i][1] = __ffma2_rn(lo, make_float2(y.x, y.y), __ffma2_rn(hi, make_float2(y.z, y.w), s[i][1]));
        }
    }
#pragma unroll
    for (int i = 0; i < RW; ++i) {
        acc[i][0] += s[i][0].x + s[i][0].y;
        acc[i][1] += s[i][1].x + s[i][1].y;
    }
}

// o[i][cc] += sum over the tile's rows j of p[i][j] tile[j][lane + 32 cc], packed over pairs of rows; p of channel c is pa
// for c < split, else pb
template <int RW, int NC>
__device__ __forceinline__ void turn_products(float (&o)[RW][NC], const float *pa, const float *pb, int split,
                                              const float *tile, int hd, int lane)
{
#pragma unroll
    for (int cc = 0; cc < NC; ++cc) {
        const int c = min(lane + 32 * cc, hd - 1);
        const float *p = c < split ? pa : pb;
        float2 s[RW];
#pragma unroll
        for (int i = 0; i < RW; ++i) s[i] = make_float2(0.f, 0.f);
#pragma unroll (RW == 8 ? 1 : 2)
        for (int j = 0; j < kTileRows; j += 4) {
            const float2 v0 = make_float2(tile[j * (hd + 4) + c], tile[(j + 1) * (hd + 4) + c]);
            const float2 v1 = make_float2(tile[(j + 2) * (hd + 4) + c], tile[(j + 3) * (hd + 4) + c]);
#pragma unroll
            for (int i = 0; i < RW; ++i) {
                const float4 w = *reinterpret_cast<const float4 *>(p + i * kTileRows + j);
                s[i] = __ffma2_rn(make_float2(w.x, w.y), v0, __ffma2_rn(make_float2(w.z, w.w), v1, s[i]));
            }
        }
#pragma unroll
        for (int i = 0; i < RW; ++i) o[i][cc] += s[i].x + s[i].y;
    }
}

template <int RW, int M> __device__ __forceinline__ void clear(float (&x)[RW][M])
{
#pragma unroll
    for (int i = 0; i < RW; ++i)
#pragma unroll
        for (int j = 0; j < M; ++j) x[i][j] = 0.f;
}

}  // namespace

// Eight warps and the widest heads: 128 registers a thread, so that two CTAs share an SM (4 maps of 17 x 54, 4 heads of 128:
// 607 us, with the five registers more that the compiler takes by itself, and one CTA, 745); else (0) as the compiler chooses.
template <int WARPS, int RW, int NC>
__global__ void __launch_bounds__(32 * WARPS, WARPS == 8 && NC == 4 ? 2 : 0) diff_attend_simt_kernel(const DiffArgs a)
{
    constexpr int ROWS = WARPS * RW, THREADS = 32 * WARPS;
    extern __shared__ float4 smem4[];
    const int hd = a.hd, stride = hd + 4, nvec = hd / 4;
    float *sk = reinterpret_cast<float *>(smem4), *sv = sk + kTileRows * stride, *sq = sv + kTileRows * stride;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float *sp = sq + ROWS * stride + warp * 2 * RW * kTileRows;  // [map][RW][64]
    int *count = reinterpret_cast<int *>(sq + ROWS * stride + WARPS * 2 * RW * kTileRows);
    int *bases = count + 4;
    const DiffItem it = diff_item(a, blockIdx.x);
    const int64_t image = (int64_t)it.b * a.N * a.C + it.h * hd;
    const float *gq = static_cast<const float *>(a.q) + image, *gk = static_cast<const float *>(a.k) + image;
    const float *gv = static_cast<const float *>(a.v) + image;
    const int region = region_at(a, it.r);
    grid_dependency_wait();
    if (warp == 0) {
        const int n = gather_bases(a, a.idx + ((int64_t)it.b * a.R + it.r) * a.topk, bases, lane);
        if (lane == 0) *count = n;
    }
    for (int e = threadIdx.x; e < ROWS * nvec; e += THREADS) {
        const int row = e / nvec, tok = it.t * ROWS + row;
        const bool in = tok < a.rs;
        stage_vector(sq, hd, row, e % nvec, gq + (int64_t)(in ? token_at(a, region, tok) : 0) * a.C, in);
    }
    __syncthreads();
    const int nkeys = *count * a.rs;
    const float *rows = sq + warp * RW * stride;
    const bool busy = it.t * ROWS + warp * RW < a.rs;  // the warp has a row

    float o[2][RW][NC], mx[2][RW], l[2][RW];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        clear<RW, NC>(o[m]);
#pragma unroll
        for (int i = 0; i < RW; ++i) {
            mx[m][i] = -INFINITY;
            l[m][i] = 0.f;
        }
    }
    for (int k0 = 0; k0 < nkeys; k0 += kTileRows) {
        if (k0) __syncthreads();
        for (int e = threadIdx.x; e < kTileRows * nvec; e += THREADS) {
            const int row = e / nvec, key = k0 + row;
            const bool real = key < nkeys;
            int64_t off = 0;
            if (real) {
                int slot, tok;
                a.by_rs.divmod(key, slot, tok);
                off = (int64_t)token_at(a, bases[slot], tok) * a.C;
            }
            stage_vector(sk, hd, row, e % nvec, gk + off, real);
            stage_vector(sv, hd, row, e % nvec, gv + off, real);
        }
        __syncthreads();
        if (!busy) continue;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            float s[RW][2];
            clear<RW, 2>(s);
            lane_products<RW>(s, rows, sk, hd, lane, m * a.d, (m + 1) * a.d);
#pragma unroll
            for (int i = 0; i < RW; ++i) {
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    if (k0 + lane + 32 * x >= nkeys) s[i][x] = -INFINITY;
                const float most = fmaxf(mx[m][i], warp_max(fmaxf(s[i][0], s[i][1])) * a.scale_log2), base = score_base(most);
                const float corr = fast_exp2(mx[m][i] - base);
                mx[m][i] = most;
                const float e0 = fast_exp2(fmaf(s[i][0], a.scale_log2, -base)), e1 = fast_exp2(fmaf(s[i][1], a.scale_log2, -base));
                l[m][i] = l[m][i] * corr + (e0 + e1);
                sp[(m * RW + i) * kTileRows + lane] = e0;
                sp[(m * RW + i) * kTileRows + lane + 32] = e1;
#pragma unroll
                for (int cc = 0; cc < NC; ++cc) o[m][i][cc] *= corr;
            }
        }
        __syncwarp();
#pragma unroll
        for (int m = 0; m < 2; ++m)
            turn_products<RW, NC>(o[m], sp + m * RW * kTileRows, nullptr, hd, sv, hd, lane);
        __syncwarp();
    }
    if (!busy) return;
    const float lam = __ldg(a.lam + it.h);
    float *out = static_cast<float *>(a.out) + image;
#pragma unroll
    for (int i = 0; i < RW; ++i) {
        const int tok = it.t * ROWS + warp * RW + i;
        if (tok >= a.rs) break;
        const float w1 = over_sum(1.f, warp_sum(l[0][i]), nkeys > 0), w2 = over_sum(-lam, warp_sum(l[1][i]), nkeys > 0);
        float *dst = out + (int64_t)token_at(a, region, tok) * a.C;
#pragma unroll
        for (int cc = 0; cc < NC; ++cc) {
            const int c = lane + 32 * cc;
            if (c < hd) dst[c] = (fmaf(o[0][i][cc], w1, o[1][i][cc] * w2));
        }
    }
}

// dq and the statistics (see bra_diff_backward.cu)
template <int WARPS, int RW, int NC>
__global__ void __launch_bounds__(32 * WARPS) diff_backward_queries_simt_kernel(const DiffArgs a)
{
    constexpr int ROWS = WARPS * RW, THREADS = 32 * WARPS;
    extern __shared__ float4 smem4[];
    const int hd = a.hd, stride = hd + 4, nvec = hd / 4;
    float *sk = reinterpret_cast<float *>(smem4), *sv = sk + kTileRows * stride, *sq = sv + kTileRows * stride;
    float *sd = sq + ROWS * stride;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float *sp = sd + ROWS * stride + warp * 2 * RW * kTileRows;
    int *count = reinterpret_cast<int *>(sd + ROWS * stride + WARPS * 2 * RW * kTileRows);
    int *bases = count + 4;
    if (blockIdx.x < a.B) {
        grid_dependency_wait();
        invert_index<WARPS>(a, blockIdx.x, reinterpret_cast<int *>(smem4));
        return;
    }
    const DiffItem it = diff_item(a, blockIdx.x - a.B);
    const int64_t image = (int64_t)it.b * a.N * a.C + it.h * hd;
    const float *gq = static_cast<const float *>(a.q) + image, *gk = static_cast<const float *>(a.k) + image;
    const float *gv = static_cast<const float *>(a.v) + image, *gd = static_cast<const float *>(a.dout) + image;
    const int region = region_at(a, it.r);
    grid_dependency_wait();
    if (warp == 0) {
        const int n = gather_bases(a, a.idx + ((int64_t)it.b * a.R + it.r) * a.topk, bases, lane);
        if (lane == 0) *count = n;
    }
    for (int e = threadIdx.x; e < ROWS * nvec; e += THREADS) {
        const int row = e / nvec, tok = it.t * ROWS + row;
        const bool in = tok < a.rs;
        const int64_t off = (int64_t)(in ? token_at(a, region, tok) : 0) * a.C;
        stage_vector(sq, hd, row, e % nvec, gq + off, in);
        stage_vector(sd, hd, row, e % nvec, gd + off, in);
    }
    __syncthreads();
    const int nkeys = *count * a.rs;
    const float *rows = sq + warp * RW * stride, *drows = sd + warp * RW * stride;
    const bool busy = it.t * ROWS + warp * RW < a.rs;

    auto stage = [&](int k0) {
        for (int e = threadIdx.x; e < kTileRows * nvec; e += THREADS) {
            const int row = e / nvec, key = k0 + row;
            const bool real = key < nkeys;
            int64_t off = 0;
            if (real) {
                int slot, tok;
                a.by_rs.divmod(key, slot, tok);
                off = (int64_t)token_at(a, bases[slot], tok) * a.C;
            }
            stage_vector(sk, hd, row, e % nvec, gk + off, real);
            stage_vector(sv, hd, row, e % nvec, gv + off, real);
        }
    };
    float mx[2][RW], l[2][RW], ed[2][RW];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int i = 0; i < RW; ++i) {
            mx[m][i] = -INFINITY;
            l[m][i] = ed[m][i] = 0.f;
        }
    for (int k0 = 0; k0 < nkeys; k0 += kTileRows) {
        if (k0) __syncthreads();
        stage(k0);
        __syncthreads();
        if (!busy) continue;
        float dp[RW][2];
        clear<RW, 2>(dp);
        lane_products<RW>(dp, drows, sv, hd, lane, 0, hd);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            float s[RW][2];
            clear<RW, 2>(s);
            lane_products<RW>(s, rows, sk, hd, lane, m * a.d, (m + 1) * a.d);
#pragma unroll
            for (int i = 0; i < RW; ++i) {
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    if (k0 + lane + 32 * x >= nkeys) s[i][x] = -INFINITY;
                const float most = fmaxf(mx[m][i], warp_max(fmaxf(s[i][0], s[i][1])) * a.scale_log2), base = score_base(most);
                const float corr = fast_exp2(mx[m][i] - base);
                mx[m][i] = most;
                const float e0 = fast_exp2(fmaf(s[i][0], a.scale_log2, -base)), e1 = fast_exp2(fmaf(s[i][1], a.scale_log2, -base));
                l[m][i] = l[m][i] * corr + (e0 + e1);
                ed[m][i] = ed[m][i] * corr + fmaf(e0, dp[i][0], e1 * dp[i][1]);
            }
        }
    }
    float Ls[2][RW], D[2][RW], dsum = 0.f;
    float4 *stats = a.stats + ((int64_t)it.b * a.heads + it.h) * a.N;
#pragma unroll
    for (int i = 0; i < RW; ++i) {
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const float sum = warp_sum(l[m][i]), num = warp_sum(ed[m][i]);
            Ls[m][i] = log_sum(mx[m][i], sum, nkeys > 0);
            D[m][i] = over_sum(num, sum, nkeys > 0);
        }
        const int tok = it.t * ROWS + warp * RW + i;
        if (tok < a.rs) {
            if (lane == 0) stats[token_at(a, region, tok)] = make_float4(Ls[0][i], Ls[1][i], D[0][i], D[1][i]);
            dsum += D[1][i];
        }
    }
    if (lane == 0)
        a.dlam_part[(int64_t)it.h * a.nparts + (((int64_t)it.b * a.R + it.r) * a.tiles + it.t) * WARPS + warp] = dsum;

    float dq[RW][NC];
    clear<RW, NC>(dq);
    for (int k0 = 0; k0 < nkeys; k0 += kTileRows) {
        if (nkeys > kTileRows) {  // else the only tile is still in place
            __syncthreads();
            stage(k0);
            __syncthreads();
        }
        if (!busy) continue;
        float dp[RW][2];
        clear<RW, 2>(dp);
        lane_products<RW>(dp, drows, sv, hd, lane, 0, hd);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            float s[RW][2];
            clear<RW, 2>(s);
            lane_products<RW>(s, rows, sk, hd, lane, m * a.d, (m + 1) * a.d);
#pragma unroll
            for (int i = 0; i < RW; ++i)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const float p = fast_exp2(fmaf(s[i][x], a.scale_log2, -Ls[m][i]));
                    sp[(m * RW + i) * kTileRows + lane + 32 * x] =
                        k0 + lane + 32 * x < nkeys ? p * (dp[i][x] - D[m][i]) : 0.f;
                }
        }
        __syncwarp();
        turn_products<RW, NC>(dq, sp, sp + RW * kTileRows, a.d, sk, hd, lane);
        __syncwarp();
    }
    if (!busy) return;
    const float s1 = a.scale, s2 = -__ldg(a.lam + it.h) * a.scale;
    float *out = static_cast<float *>(a.dq) + image;
#pragma unroll
    for (int i = 0; i < RW; ++i) {
        const int tok = it.t * ROWS + warp * RW + i;
        if (tok >= a.rs) break;
        float *dst = out + (int64_t)token_at(a, region, tok) * a.C;
#pragma unroll
        for (int cc = 0; cc < NC; ++cc) {
            const int c = lane + 32 * cc;
            if (c < hd) dst[c] = (dq[i][cc] * (c < a.d ? s1 : s2));
        }
    }
}

// dk, dv and dlam (see bra_diff_backward.cu)
template <int WARPS, int RW, int NC>
__global__ void __launch_bounds__(32 * WARPS) diff_backward_keys_simt_kernel(const DiffArgs a)
{
    constexpr int ROWS = WARPS * RW, THREADS = 32 * WARPS;
    extern __shared__ float4 smem4[];
    const int hd = a.hd, stride = hd + 4, nvec = hd / 4;
    float *sq = reinterpret_cast<float *>(smem4), *sd = sq + kTileRows * stride, *sk = sd + kTileRows * stride;
    float *sv = sk + ROWS * stride;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float *sp = sv + ROWS * stride + warp * 3 * RW * kTileRows;  // [P1 - lam P2, dS1, dS2][RW][64]
    grid_dependency_wait();
    if (blockIdx.x < a.heads) {  // dlam of head blockIdx.x, summed in 64 bits in a fixed order
        double *part = reinterpret_cast<double *>(smem4);
        const float *src = a.dlam_part + (int64_t)blockIdx.x * a.nparts;
        double sum = 0.;
        for (int e = threadIdx.x; e < a.nparts; e += THREADS) sum += (double)__ldcg(src + e);
        part[threadIdx.x] = sum;
        __syncthreads();
        if (threadIdx.x == 0) {
            double all = 0.;
            for (int e = 0; e < THREADS; ++e) all += part[e];
            a.dlam[blockIdx.x] = (float)-all;
        }
        __syncthreads();
    }
    if (blockIdx.x >= a.nitems) return;
    const DiffItem it = diff_item(a, blockIdx.x);
    const int64_t image = (int64_t)it.b * a.N * a.C + it.h * hd;
    const float *gq = static_cast<const float *>(a.q) + image, *gk = static_cast<const float *>(a.k) + image;
    const float *gv = static_cast<const float *>(a.v) + image, *gd = static_cast<const float *>(a.dout) + image;
    const float4 *stats = a.stats + ((int64_t)it.b * a.heads + it.h) * a.N;
    const int region = region_at(a, it.r);
    const int32_t *start = a.start + (int64_t)it.b * (a.R + 1) + it.r;
    const int first = __ldg(start);
    const int nq = (__ldg(start + 1) - first) * a.rs;
    const int32_t *list = a.list + (int64_t)it.b * a.R * a.topk + first;
    auto query_at = [&](int query) {
        int slot, tok;
        a.by_rs.divmod(query, slot, tok);
        return token_at(a, region_at(a, __ldg(list + slot)), tok);
    };
    for (int e = threadIdx.x; e < ROWS * nvec; e += THREADS) {
        const int row = e / nvec, tok = it.t * ROWS + row;
        const bool in = tok < a.rs;
        const int64_t off = (int64_t)(in ? token_at(a, region, tok) : 0) * a.C;
        stage_vector(sk, hd, row, e % nvec, gk + off, in);
        stage_vector(sv, hd, row, e % nvec, gv + off, in);
    }
    const float *krows = sk + warp * RW * stride, *vrows = sv + warp * RW * stride;
    const bool busy = it.t * ROWS + warp * RW < a.rs;
    const float lam = __ldg(a.lam + it.h);
    float dk[RW][NC], dv[RW][NC];
    clear<RW, NC>(dk);
    clear<RW, NC>(dv);
    for (int q0 = 0; q0 < nq; q0 += kTileRows) {
        if (q0) __syncthreads();
        for (int e = threadIdx.x; e < kTileRows * nvec; e += THREADS) {
            const int row = e / nvec, query = q0 + row;
            const bool real = query < nq;
            const int64_t off = real ? (int64_t)query_at(query) * a.C : 0;
            stage_vector(sq, hd, row, e % nvec, gq + off, real);
            stage_vector(sd, hd, row, e % nvec, gd + off, real);
        }
        __syncthreads();
        if (!busy) continue;
        float4 st[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int query = q0 + lane + 32 * x;
            st[x] = query < nq ? __ldcg(stats + query_at(query)) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        float dp[RW][2], s1[RW][2], s2[RW][2];
        clear<RW, 2>(dp);
        clear<RW, 2>(s1);
        clear<RW, 2>(s2);
        lane_products<RW>(dp, vrows, sd, hd, lane, 0, hd);
        lane_products<RW>(s1, krows, sq, hd, lane, 0, a.d);
        lane_products<RW>(s2, krows, sq, hd, lane, a.d, hd);
#pragma unroll
        for (int i = 0; i < RW; ++i)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const bool real = q0 + lane + 32 * x < nq;
                const float p1 = fast_exp2(fmaf(s1[i][x], a.scale_log2, -st[x].x));
                const float p2 = fast_exp2(fmaf(s2[i][x], a.scale_log2, -st[x].y));
                float *dst = sp + i * kTileRows + lane + 32 * x;
                dst[0] = real ? fmaf(-lam, p2, p1) : 0.f;
                dst[RW * kTileRows] = real ? p1 * (dp[i][x] - st[x].z) : 0.f;
                dst[2 * RW * kTileRows] = real ? p2 * (dp[i][x] - st[x].w) : 0.f;
            }
        __syncwarp();
        turn_products<RW, NC>(dv, sp, nullptr, hd, sd, hd, lane);
        turn_products<RW, NC>(dk, sp + RW * kTileRows, sp + 2 * RW * kTileRows, a.d, sq, hd, lane);
        __syncwarp();
    }
    if (!busy) return;
    const float w1 = a.scale, w2 = -lam * a.scale;
#pragma unroll
    for (int i = 0; i < RW; ++i) {
        const int tok = it.t * ROWS + warp * RW + i;
        if (tok >= a.rs) break;
        const int64_t off = image + (int64_t)token_at(a, region, tok) * a.C;
#pragma unroll
        for (int cc = 0; cc < NC; ++cc) {
            const int c = lane + 32 * cc;
            if (c < hd) {
                static_cast<float *>(a.dk)[off + c] = (dk[i][cc] * (c < a.d ? w1 : w2));
                static_cast<float *>(a.dv)[off + c] = (dv[i][cc]);
            }
        }
    }
}

namespace {

template <auto Kernel>
cudaError_t launch_with(int grid, int threads, size_t smem, const DiffArgs &a, cudaStream_t stream)
{
    const cudaError_t e = grant_shared_memory<Kernel>();
    if (e != cudaSuccess) return e;
    return launch_pdl(Kernel, dim3(grid), dim3(threads), smem, stream, a);
}

template <int WARPS, int RW, int NC> cudaError_t launch_one(DiffArgs &a, bool backward, cudaStream_t stream)
{
    using L = SimtTile<WARPS, RW>;
    a.tiles = (a.rs + L::kRows - 1) / L::kRows;
    a.by_tiles = FastDiv::of(a.tiles);
    const long long items = (long long)a.B * a.R * a.tiles * a.heads;
    if (items * WARPS + a.B > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    a.nitems = (int)items;
    a.nparts = (int)(items / a.heads * WARPS);
    const size_t tail = 16 + (((size_t)a.topk * 4 + 15) & ~(size_t)15);
    const int grid = (int)items;
    if (!backward)
        return launch_with<diff_attend_simt_kernel<WARPS, RW, NC>>(grid, 32 * WARPS, 4 * L::floats(a.hd, 1, 2) + tail, a,
                           stream);
    const cudaError_t e = launch_with<diff_backward_queries_simt_kernel<WARPS, RW, NC>>(
        a.B + grid, 32 * WARPS, std::max(4 * L::floats(a.hd, 2, 2) + tail, invert_bytes(WARPS, a.R)), a, stream);
    if (e != cudaSuccess) return e;
    return launch_with<diff_backward_keys_simt_kernel<WARPS, RW, NC>>(grid > a.heads ? grid : a.heads, 32 * WARPS,
                       4 * L::floats(a.hd, 2, 3), a, stream);
}

template <int NC> cudaError_t launch_nc(DiffArgs &a, bool backward, cudaStream_t stream)
{
    if (a.rs <= 4) return launch_one<4, 1, NC>(a, backward, stream);
    if (a.rs <= 16) return launch_one<4, 4, NC>(a, backward, stream);
    // CTAs of 32 rows: eight to a warp, whose reads feed the most FMAs, or, for many keys, twice the warps of four rows (3
    // regions of 63 tokens, 48 channels: 47 and 53 us; one of 1024, 64 channels: 148 and 112 us)
    if (diff_simt_warps(a.topk, a.rs) == 4) return launch_one<4, 8, NC>(a, backward, stream);
    return launch_one<8, 4, NC>(a, backward, stream);
}

}  // namespace

cudaError_t launch_diff_simt(const DiffArgs &args, bool backward, cudaStream_t stream)
{
    DiffArgs a = args;
    switch ((a.hd + 31) / 32) {
    case 1: return launch_nc<1>(a, backward, stream);
    case 2: return launch_nc<2>(a, backward, stream);
    case 3: return launch_nc<3>(a, backward, stream);
    default: return launch_nc<4>(a, backward, stream);
    }
}

}  // namespace bra
