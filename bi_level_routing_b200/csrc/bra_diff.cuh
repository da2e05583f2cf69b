// bra_diff.cuh -- what the differential attention kernels share: the call's geometry, the gather of
// a region's routed token rows, and the tile pieces of the bf16 tensor-core kernels.
//
// Differential attention. Head h owns hd = C / heads channels of q, k, v and out. The first d = hd / 2
// channels of its q and k make map 1, the last d map 2; v keeps all hd. For a query of region r, over
// the tokens j of the regions idx[b, r, :],
//   out = (softmax_j(d^-1/2 q1 . k1_j) - lam[h] softmax_j(d^-1/2 q2 . k2_j)) v_j.
// With P1, P2 the two maps, dP = dout V^T and D_i = rowsum(P_i dP) the gradients of sum(dout out) are
//   dS1 = d^-1/2 P1 (dP - D1),  dS2 = -lam d^-1/2 P2 (dP - D2),
//   dq_i = dS_i k_i,  dk_i = dS_i^T q_i,  dv = (P1 - lam P2)^T dout,  dlam = -sum over queries of D2.
#pragma once

#include "bra_device.cuh"
#include "bra_launch.h"

namespace bra {

// Division of 0 <= n < 2^31 by a fixed d >= 1 as a multiplication and a shift: with
// l = ceil(log2 d) and m = floor(2^32 (2^l - d) / d) + 1, n / d = (hi32(n m) + n) >> l.
struct FastDiv {
    uint32_t m, l;
    int d;
    __host__ static FastDiv of(int d)
    {
        uint32_t l = 0;
        while ((1ull << l) < (uint64_t)d) ++l;
        FastDiv f;
        f.m = (uint32_t)(((1ull << 32) * ((1ull << l) - (uint64_t)d)) / (uint64_t)d + 1);
        f.l = l;
        f.d = d;
        return f;
    }
    __device__ __forceinline__ int div(int n) const { return (int)((__umulhi((uint32_t)n, m) + (uint32_t)n) >> l); }
    __device__ __forceinline__ void divmod(int n, int &q, int &r) const
    {
        q = div(n);
        r = n - q * d;
    }
};

struct DiffArgs {
    const void *q, *k, *v, *dout;
    const int32_t *idx;
    const float *lam;
    void *out;
    void *dq, *dk, *dv;     // of the input type
    float *dlam;            // [heads]
    float4 *stats;          // [B, heads, N]: L1, L2 (log2 of each map's normaliser), D1, D2
    float *dlam_part;       // [heads, nparts]: sums of D2, one for each (image, region, query tile, warp)
    int32_t *list;          // [B, R * topk]: for each region, the regions that route to it, in order
    int32_t *start;         // [B, R + 1]: where each region's part of the list starts
    unsigned *err;
    int B, H, W, C, heads, hd, d, n_win, hr, wr, rs, R, topk, N;
    int tiles;      // tiles of a region's tokens
    int nitems;     // work items of the launch
    int nparts;
    int num_sms;
    // the tcgen05 forward pass, an item's keys split over several CTAs
    int splits, per;       // CTAs of an item, keys of one
    float4 *split_out;     // [CTA][map][16-byte chunk][128 rows]: sums of P V
    float2 *split_stats;   // [CTA][map][128 rows]: maximum, sum
    FastDiv by_splits;
    float scale;        // d^-1/2
    float scale_log2;   // d^-1/2 log2(e)
    FastDiv by_rs, by_wr, by_nwin, by_heads, by_tiles, by_R, by_topk;
};

// Warps of a CTA of 32 rows in the CUDA-core kernels of regions above 16 tokens.
inline int diff_simt_warps(int topk, int rs) { return (long long)topk * rs <= 256 ? 4 : 8; }

// Offset y W + x (in tokens, inside an image) of token `tok` of the region whose first token lies at
// `base`.
__device__ __forceinline__ int token_at(const DiffArgs &a, int base, int tok)
{
    int y, x;
    a.by_wr.divmod(tok, y, x);
    return base + y * a.W + x;
}

// Offset of region s's first token.
__device__ __forceinline__ int region_at(const DiffArgs &a, int s)
{
    int ry, rx;
    a.by_nwin.divmod(s, ry, rx);
    return ry * a.hr * a.W + rx * a.wr;
}

// One item of a launch: heads fastest (neighbouring heads' channels share cache lines), then the
// tiles of a region, the regions, the images.
struct DiffItem {
    int h, t, r, b;
};
__device__ __forceinline__ DiffItem diff_item(const DiffArgs &a, int item)
{
    DiffItem it;
    int rest;
    a.by_heads.divmod(item, rest, it.h);
    a.by_tiles.divmod(rest, rest, it.t);
    a.by_R.divmod(rest, it.b, it.r);
    return it;
}

// A warp writes the first-token offsets of the valid regions of idx[b, r, :] to `bases`, in order,
// and returns how many there are; entries outside [0, R) are left out and flagged.
__device__ __forceinline__ int gather_bases(const DiffArgs &a, const int32_t *row, int *bases, int lane)
{
    int n = 0;
    for (int j0 = 0; j0 < a.topk; j0 += 32) {
        const int j = j0 + lane;
        const int s = j < a.topk ? __ldg(row + j) : 0;
        const bool ok = j < a.topk && s >= 0 && s < a.R;
        if (j < a.topk && !ok) flag_error(a.err, kErrIndex);
        const unsigned mask = __ballot_sync(0xffffffffu, ok);
        if (ok) bases[n + __popc(mask & ((1u << lane) - 1u))] = region_at(a, s);
        n += __popc(mask);
    }
    return n;
}

// A 16-byte asynchronous copy, or 16 zero bytes when `real` is false (src is not read then).
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void *src, bool real)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
// Arrives on `bar` once all cp.async copies this thread has issued have landed (the barrier's count
// includes the thread).
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void cp_async8_or_zero(uint32_t dst, const void *src, bool real)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(real ? 8 : 0) : "memory");
}
// 16-byte chunk j of a row in shared memory: the head's two halves of d channels padded with zeros to DK each (q, k), or its hd
// channels run on, zeros after them (v, dout). src: the head's first channel of the token. Halves that are not whole
// 16-byte chunks (d a multiple of 4) are copied in pieces of 8 bytes.
template <int DK>
__device__ __forceinline__ void copy_split(uint32_t row, const __nv_bfloat16 *src, int j, int d, bool real)
{
    const int m = j / (DK / 8), x = 8 * (j % (DK / 8));
    if (d % 8 == 0) {
        cp_async16_or_zero(row + 16 * j, src + (x < d ? m * d + x : 0), real && x < d);
    } else {
        cp_async8_or_zero(row + 16 * j, src + (x < d ? m * d + x : 0), real && x < d);
        cp_async8_or_zero(row + 16 * j + 8, src + (x + 4 < d ? m * d + x + 4 : 0), real && x + 4 < d);
    }
}
__device__ __forceinline__ void copy_run(uint32_t row, const __nv_bfloat16 *src, int j, int hd, bool real)
{
    cp_async16_or_zero(row + 16 * j, src + (8 * j < hd ? 8 * j : 0), real && 8 * j < hd);
}
template <int N> __device__ __forceinline__ void cp_async_wait_but()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// What scores are taken relative to: the running maximum, or 0 while every score so far is -inf, so that exp2(score - base)
// is 0, not NaN. The maximum itself stays -inf then: a 0 in its place would be a floor that later, lower scores cannot
// reach, and below 2^-126 of it they would all count as 0. From a maximum of -inf to any other the sums so far
// (0, or NaN) are multiplied by exp2(-inf - base) = 0.
__device__ __forceinline__ float score_base(float max) { return max == -INFINITY ? 0.f : max; }

// A warp goes through ROWS rows, LANES of its lanes to a row: a lane finds the place of one row (locate(row), -1 for none,
// some dozen instructions), the lanes that copy the row take it from there: copy(row, place).
template <int ROWS, int LANES, typename Locate, typename Copy>
__device__ __forceinline__ void warp_rows(int lane, Locate locate, Copy copy)
{
    static_assert(LANES <= 32 && 32 % LANES == 0, "whole rows to a pass");
#pragma unroll
    for (int r0 = 0; r0 < ROWS; r0 += 32) {
        const int at = r0 + lane < ROWS ? locate(r0 + lane) : -1;
#pragma unroll
        for (int x = 0; x < (ROWS - r0 < 32 ? ROWS - r0 : 32) * LANES; x += 32) {
            const int row = (x + lane) / LANES;
            const int place = __shfl_sync(0xffffffffu, at, row & 31);
            if (r0 + row < ROWS) copy(r0 + row, place);
        }
    }
}

// 2^x of two values on the FMA pipe, for probabilities that are rounded to bf16: x = n + f with n the
// nearest integer (added to 1.5 2^23, where a float's last bit counts ones), 2^f a cubic fitted to least
// relative error on [-1/2, 1/2] (7.5e-5, a 26th of a bf16 rounding), n added to its exponent. x below
// -126.998 counts as that: 1.0013 2^-127 loses its leading one with the exponent, and what is left rounds to 0 in bf16, so
// that a masked key's value counts 0 times. A NaN or +inf x gives some finite value: the caller looks for them in the
// row's maximum.
__device__ __forceinline__ float2 poly_exp2(float2 x)
{
    const float2 magic = make_float2(12582912.f, 12582912.f), back = make_float2(-12582912.f, -12582912.f);
    x = make_float2(fmaxf(x.x, -126.998f), fmaxf(x.y, -126.998f));
    const float2 n = __fadd2_rn(x, magic);
    const float2 m = __fadd2_rn(n, back);
    const float2 f = __ffma2_rn(m, make_float2(-1.f, -1.f), x);
    float2 p = __ffma2_rn(f, make_float2(0.05517120659351349f, 0.05517120659351349f),
                          make_float2(0.24261026084423065f, 0.24261026084423065f));
    p = __ffma2_rn(p, f, make_float2(0.6932609677314758f, 0.6932609677314758f));
    p = __ffma2_rn(p, f, make_float2(0.9999281167984009f, 0.9999281167984009f));
    return make_float2(__uint_as_float(__float_as_uint(p.x) + (__float_as_uint(n.x) << 23)),
                       __uint_as_float(__float_as_uint(p.y) + (__float_as_uint(n.y) << 23)));
}

// ---------------------------------------------------------------- tcgen05, issued by a converged warp
//
// A thread that issues products inside `if (lane == 0)` copies every descriptor from vector to uniform
// registers first (60 cycles a product and 85 a commit were measured); in a converged warp the
// compiler keeps them uniform, and one elected lane issues. uniform() tells it that a value is the same in
// all lanes.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
// Upper and lower half of a descriptor of 128-byte swizzled rows (umma_desc_sw128); x bytes further on is
// + (x >> 4) of the lower half.
constexpr uint32_t kDescHigh = (uint32_t)((1024 >> 4) | (1u << 14) | (2u << 29));
__device__ __forceinline__ uint32_t desc_low(uint32_t saddr) { return ((saddr >> 4) & 0x3FFFu) | (1u << 16); }
// D[tmem] (+)= A[smem] B[smem] and A[tmem] B[smem], bf16 into fp32
__device__ __forceinline__ void umma_ss(uint32_t d, uint32_t a_low, uint32_t b_low, uint32_t idesc, bool add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
        "r"(a_low), "r"(b_low), "r"(idesc), "r"((uint32_t)add), "r"(kDescHigh)
        : "memory");
}
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a_tmem, uint32_t b_low, uint32_t idesc, bool add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 y, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
        "r"(a_tmem), "r"(b_low), "r"(idesc), "r"((uint32_t)add), "r"(kDescHigh)
        : "memory");
}

// A CTA sorts the R * topk routed slots of image b by their region (a stable counting sort): the list of the regions that
// route to each. Warp w owns the slots [w len, (w + 1) len); count[w][s] counts its slots that name s, then holds where
// the first of them goes, so that the list keeps the slots' order. The first B CTAs of the backward pass' first
// launch do this beside the others' queries.
inline size_t invert_bytes(int warps, int R) { return (size_t)warps * (R + 32) * sizeof(int); }
template <int WARPS> __device__ __forceinline__ void invert_index(const DiffArgs &a, int b, int *shared)
{
    int *total = shared, *count = shared + 32 * WARPS;  // [WARPS][R]
    const int R = a.R, topk = a.topk;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n = R * topk, len = (n + WARPS - 1) / WARPS;
    const int begin = min(n, warp * len), end = min(n, begin + len);
    const int32_t *idx = a.idx + (int64_t)b * n;
    int32_t *list = a.list + (int64_t)b * n, *start = a.start + (int64_t)b * (R + 1);
    for (int e = threadIdx.x; e < WARPS * R; e += 32 * WARPS) count[e] = 0;
    __syncthreads();
    int *own = count + warp * R;
    for (int e = begin + lane; e < end; e += 32) {
        const int s = __ldg(idx + e);
        if (s >= 0 && s < R) atomicAdd(own + s, 1);
    }
    __syncthreads();
    // exclusive sums over (region, warp), regions in runs of `per` to a thread
    const int per = (R + 32 * WARPS - 1) / (32 * WARPS);
    const int s0 = min(R, (int)threadIdx.x * per), s1 = min(R, s0 + per);
    int sum = 0;
    for (int s = s0; s < s1; ++s)
        for (int w = 0; w < WARPS; ++w) sum += count[w * R + s];
    total[threadIdx.x] = sum;
    __syncthreads();
    for (int o = 1; o < 32 * WARPS; o *= 2) {
        const int add = (int)threadIdx.x >= o ? total[threadIdx.x - o] : 0;
        __syncthreads();
        total[threadIdx.x] += add;
        __syncthreads();
    }
    int at = total[threadIdx.x] - sum;
    for (int s = s0; s < s1; ++s) {
        start[s] = at;
        for (int w = 0; w < WARPS; ++w) {
            const int c = count[w * R + s];
            count[w * R + s] = at;
            at += c;
        }
    }
    if (threadIdx.x == 32 * WARPS - 1) start[R] = at;
    __syncthreads();
    for (int e0 = begin; e0 < end; e0 += 32) {
        const int e = e0 + lane;
        const int s = e < end ? __ldg(idx + e) : -1;
        const bool ok = s >= 0 && s < R;
        const unsigned same = __match_any_sync(0xffffffffu, ok ? s : -1);
        int slot = 0;
        if (ok) slot = own[s] + __popc(same & ((1u << lane) - 1u));
        __syncwarp();
        if (ok) {
            list[slot] = e / topk;
            if (lane == 31 - __clz(same)) own[s] = slot + 1;
        }
        __syncwarp();
    }
}

// x / sum of a row's probabilities, and the row's max + log2(sum) (so that P = 2^(scale S - that)). A row without keys
// (some = false) has weights 0 and a log of +inf. A row with keys whose sum is not positive held a NaN or +inf score (NaN
// sum) or only -inf ones (sum 0): its softmax is NaN.
__device__ __forceinline__ float over_sum(float x, float sum, bool some) { return sum > 0.f ? x / sum : some ? NAN : 0.f; }
__device__ __forceinline__ float log_sum(float max, float sum, bool some)
{
    return sum > 0.f ? max + log2f(sum) : some ? NAN : INFINITY;
}

__device__ __forceinline__ float quad_max(float x)
{
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}
__device__ __forceinline__ float quad_sum(float x)
{
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    return x + __shfl_xor_sync(0xffffffffu, x, 2);
}
__device__ __forceinline__ float warp_sum(float x)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
__device__ __forceinline__ float warp_max(float x)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

// The barrier of one group of WPI warps of a 4-warp CTA.
template <int WPI> __device__ __forceinline__ void group_barrier(int group)
{
    if (WPI == 1)
        __syncwarp();
    else
        named_barrier(1 + group, 32 * WPI);
}

}  // namespace bra
