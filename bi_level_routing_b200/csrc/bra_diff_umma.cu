// bra_diff_umma.cu -- forward differential attention of bf16 maps on the 5th-generation tensor cores
// (tcgen05, TMEM accumulators), for heads of 64 or 128 channels and regions of at least
// kUmmaRegion tokens (see bra_diff.cuh for the formula). Two exponentials a query-key pair against 6 hd
// tensor operations: from these sizes on the exponential unit (16 a cycle and SM) is the bound.
//
// A CTA owns 128 query tokens of one (image, region, head) and meets the routed keys in tiles of 128:
//  * warps 0-3 are map 1's softmax, warps 4-7 map 2's; thread t of either owns query row t, i.e. TMEM
//    lane t. While one map's scores are formed or its values summed, the other's exponentials run.
//    A thread takes its row's 128 scores, follows the running maximum, writes the probabilities as bf16
//    over the first 64 columns of its scores, and keeps the row's sum in fp32. The accumulator in
//    TMEM is rescaled only when a row's maximum has grown by more than 2^8 (the probabilities stay
//    relative to an older maximum until then: exact, and far from overflow), so PV products
//    accumulate in place;
//  * warp 8: one thread issues the products. S_m = Q_m K_m^T (M = N = 128, K = hd / 2) and
//    O_m += P_m V (M = 128, N = 64 a block, K = 128; P from TMEM), map 1's and map 2's in turn: S_m of
//    the next tile follows O_m of this one at once, since P_m lies over S_m;
//  * warps 9-11 gather the query rows and, into a ring of stages, the key and value rows of the routed
//    regions by cp.async, 128-byte swizzled; regions of any size pack densely, rows past the last key
//    are zeros.
// Every wait is bounded (kErrTimeout); no thread leaves before the TMEM is released.
#include "bra_diff.cuh"

namespace bra {

namespace {

constexpr int kThreads = 384, kLoaders = 96;
constexpr int kBlock = 128 * 128;  // one tile of 128 rows x 64 channels
constexpr uint32_t kCols = 512;    // S1 at 0, S2 at 128, O1 at 256, O2 after it
// Registers a thread after the split; the launcher checks that the launch holds their sum.
constexpr int kManyRegs = 200, kFewRegs = 80;
constexpr float kGrowth = 8.f;     // log2 of the growth of a maximum that rescales the accumulator

template <int NB> struct UmmaTile {
    static constexpr int kStages = NB == 1 ? 4 : 3;
    static size_t bytes(int topk) { return 1024 + (size_t)kBlock * NB * (1 + 2 * kStages) + 256 + 1024 + 16 + 4 * (size_t)topk; }
};

}  // namespace

template <int NB> __global__ void __launch_bounds__(kThreads, 1) diff_attend_umma_kernel(const DiffArgs a)
{
    using L = UmmaTile<NB>;
    constexpr int ST = L::kStages, KS = 2 * NB;  // KS: 16-channel steps of a half head
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sQ = smem, *sKV = smem + kBlock * NB;  // [stage][K, V][NB]
    uint64_t *q_full = reinterpret_cast<uint64_t *>(sKV + (size_t)ST * 2 * NB * kBlock);
    uint64_t *kv_full = q_full + 1, *kv_empty = kv_full + ST;
    uint64_t *s_full = kv_empty + ST, *p_full = s_full + 2, *o_done = p_full + 2, *drain = o_done + 2;
    float *sum = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(q_full) + 256);  // [2][128]
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sum + 256);
    int *count = reinterpret_cast<int *>(tmem_slot + 1);
    int *bases = count + 3;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const DiffItem it = diff_item(a, blockIdx.x);

    if (threadIdx.x == 0) {
        mbar_init(q_full, kLoaders / 32);
        for (int i = 0; i < ST; ++i) {
            mbar_init(&kv_full[i], kLoaders / 32);
            mbar_init(&kv_empty[i], 1);
        }
        for (int m = 0; m < 2; ++m) {
            mbar_init(&s_full[m], 1);
            mbar_init(&p_full[m], 4);
            mbar_init(&o_done[m], 1);
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
    const int nkeys = *count * a.rs;
    const int ntiles = (nkeys + 127) / 128;
    const int64_t image = (int64_t)it.b * a.N * a.C + it.h * a.hd;
    const int region = region_at(a, it.r);
    const int tok0 = it.t * 128;

    // the softmax warps' registers come from the others' (warps 8-11 are one warpgroup)
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
    if (warp >= 9) {
        // ------------------------------------------------------------- gather
        const int tid = threadIdx.x - 288, j = tid & 7;
        const __nv_bfloat16 *gq = static_cast<const __nv_bfloat16 *>(a.q) + image + 8 * j;
        const __nv_bfloat16 *gk = static_cast<const __nv_bfloat16 *>(a.k) + image + 8 * j;
        const __nv_bfloat16 *gv = static_cast<const __nv_bfloat16 *>(a.v) + image + 8 * j;
        if (ntiles > 0) {
            for (int row = tid >> 3; row < 128; row += kLoaders / 8) {
                const bool real = tok0 + row < a.rs;
                const int64_t off = real ? (int64_t)token_at(a, region, tok0 + row) * a.C : 0;
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
                    cp_async16_or_zero(smem_u32(sQ + nb * kBlock) + sw128(row, j), gq + off + 64 * nb, real);
            }
            cp_async_commit();
        }
        // tile i's copies are committed, then tile i - LAG's have landed and are handed over; the queries
        // came before tile 0. LAG = ST - 2: the products release a stage only after they have the
        // next tile, so two tiles must be in hand before the ring's first stage is waited for.
        constexpr int LAG = ST - 2;
        bool alive = true;
        for (int i = 0; i < ntiles + LAG && alive && ntiles > 0; ++i) {
            if (i < ntiles) {
                const int st = i % ST;
                if (!(alive = mbar_wait(&kv_empty[st], (uint32_t)(((i / ST) & 1) ^ 1), a.err))) break;
                uint8_t *sk = sKV + (size_t)st * 2 * NB * kBlock, *sv = sk + NB * kBlock;
                for (int row = tid >> 3; row < 128; row += kLoaders / 8) {
                    const int key = i * 128 + row;
                    const bool real = key < nkeys;
                    int64_t off = 0;
                    if (real) {
                        int slot, tok;
                        a.by_rs.divmod(key, slot, tok);
                        off = (int64_t)token_at(a, bases[slot], tok) * a.C;
                    }
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
                        cp_async16_or_zero(smem_u32(sk + nb * kBlock) + sw128(row, j), gk + off + 64 * nb, real);
                        cp_async16_or_zero(smem_u32(sv + nb * kBlock) + sw128(row, j), gv + off + 64 * nb, real);
                    }
                }
            }
            cp_async_commit();
            cp_async_wait_but<LAG>();
            fence_async_shared();
            __syncwarp();
            if (lane == 0) {
                if (i == LAG) mbar_arrive(q_full);
                if (i >= LAG) mbar_arrive(&kv_full[(i - LAG) % ST]);
            }
        }
        cp_async_wait_all();
    } else {
        // ------------------------------------------------------------- products
        if (lane == 0 && ntiles > 0) {
            constexpr uint32_t kIdescS = umma_idesc_bf16(128, 128, false);
            constexpr uint32_t kIdescPV = umma_idesc_bf16(128, 64, true);
            const uint64_t dq = umma_desc_sw128(smem_u32(sQ)), dkv = umma_desc_sw128(smem_u32(sKV));
            bool alive = mbar_wait(q_full, 0, a.err);
            auto scores = [&](int m, int i) {  // half m's channels: 64 bytes on in the same rows, or the next block
                const uint64_t half = NB == 1 ? 4 * m : (uint64_t)m * (kBlock >> 4);
                const uint64_t dk = dkv + (uint64_t)((i % ST) * 2 * NB) * (kBlock >> 4) + half;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
                    umma_bf16(tmem + 128 * m, dq + half + 2 * ks, dk + 2 * ks, kIdescS, (uint32_t)(ks > 0));
                umma_commit(&s_full[m]);
            };
            if (alive) alive = mbar_wait(&kv_full[0], 0, a.err);
            if (alive) {
                tcgen05_after_sync();
                scores(0, 0);
                scores(1, 0);
            }
            for (int i = 0; i < ntiles && alive; ++i) {
                for (int m = 0; m < 2 && alive; ++m) {
                    if (!(alive = mbar_wait(&p_full[m], (uint32_t)(i & 1), a.err))) break;
                    tcgen05_after_sync();
                    const uint64_t dv = dkv + (uint64_t)((i % ST) * 2 * NB + NB) * (kBlock >> 4);
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks)
                            umma_bf16_ts(tmem + 256 + 64 * (NB * m + nb), tmem + 128 * m + 8 * ks,
                                         dv + (uint64_t)nb * (kBlock >> 4) + 128 * ks, kIdescPV, (uint32_t)(i > 0 || ks > 0));
                    umma_commit(&o_done[m]);
                    if (m == 1) umma_commit(&kv_empty[i % ST]);
                    if (i + 1 < ntiles) {
                        if (m == 0) {
                            if (!(alive = mbar_wait(&kv_full[(i + 1) % ST], (uint32_t)(((i + 1) / ST) & 1), a.err))) break;
                            tcgen05_after_sync();
                        }
                        scores(m, i + 1);
                    }
                }
            }
            // wait for the last commit, so that no arrival lands after this CTA has left
            umma_commit(drain);
            mbar_wait(drain, 0, a.err);
        }
    }
    } else {
        // ------------------------------------------------------------- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kManyRegs));
        const int m = warp >> 2, row = 32 * (warp & 3) + lane;
        const uint32_t t_row = tmem + ((uint32_t)(32 * (warp & 3)) << 16), t_s = t_row + 128 * m;
        const uint32_t t_o = t_row + 256 + 64 * NB * m;
        float mx = -INFINITY, l = 0.f;
        bool alive = true;
        const float2 sc = make_float2(a.scale_log2, a.scale_log2);
        for (int i = 0; i < ntiles; ++i) {
            if (!(alive = mbar_wait(&s_full[m], (uint32_t)(i & 1), a.err))) break;
            tcgen05_after_sync();
            uint32_t v[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld_32x32(t_s + 32 * c, v[c]);
            tmem_wait_ld();
            if ((i + 1) * 128 > nkeys) {
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int x = 0; x < 32; ++x)
                        if (i * 128 + 32 * c + x >= nkeys) v[c][x] = 0xff800000u;
            }
            float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int x = 0; x < 32; x += 2)
#pragma unroll
                for (int c = 0; c < 4; ++c) top[c] = fmax3(top[c], __uint_as_float(v[c][x]), __uint_as_float(v[c][x + 1]));
            const float t = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * a.scale_log2;
            const bool grown = t > mx + kGrowth || (mx == -INFINITY && t != -INFINITY);
            if (__any_sync(0xffffffffu, grown)) {
                const float corr = grown ? fast_exp2(mx - t) : 1.f;
                if (grown) {
                    mx = t;
                    l *= corr;
                }
                if (i > 0) {  // the products so far are complete before they are rescaled
                    if (!(alive = mbar_wait(&o_done[m], (uint32_t)((i - 1) & 1), a.err))) break;
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
            }
            const float base = mx == -INFINITY ? 0.f : -mx;
            const float2 nm = make_float2(base, base);
            float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint32_t pw[32];
#pragma unroll
                for (int x = 0; x < 32; ++x) {
                    const uint32_t s0 = v[2 * half + x / 16][(2 * x) % 32], s1 = v[2 * half + x / 16][(2 * x) % 32 + 1];
                    const float2 e = __ffma2_rn(make_float2(__uint_as_float(s0), __uint_as_float(s1)), sc, nm);
                    const float2 p = make_float2(fast_exp2(e.x), fast_exp2(e.y));
                    ls[x & 1] = __fadd2_rn(ls[x & 1], p);
                    pw[x] = pack_bf16x2(p.x, p.y);
                }
                tmem_st_32x32(t_s + 32 * half, pw);
            }
            tmem_wait_st();
            const float2 add = __fadd2_rn(ls[0], ls[1]);
            l += add.x + add.y;
            tcgen05_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[m]);
        }
        // out = O1 / l1 - lam O2 / l2: thread `row` of map m's warps writes half m of the row's channels
        sum[128 * m + row] = l;
        named_barrier(1, 256);
        if (ntiles > 0 && alive) alive = mbar_wait(&o_done[0], (uint32_t)((ntiles - 1) & 1), a.err);
        if (ntiles > 0 && alive) alive = mbar_wait(&o_done[1], (uint32_t)((ntiles - 1) & 1), a.err);
        tcgen05_after_sync();
        const float l1 = sum[row], l2 = sum[128 + row], lam = __ldg(a.lam + it.h);
        const float w1 = l1 > 0.f ? 1.f / l1 : 0.f, w2 = l2 > 0.f ? -lam / l2 : 0.f;
        const bool in = tok0 + row < a.rs;
        __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + image + 32 * NB * m;
        if (in) out += (int64_t)token_at(a, region, tok0 + row) * a.C;
#pragma unroll
        for (int c = 0; c < NB; ++c) {
            uint32_t o1[32], o2[32];
            if (ntiles > 0) {  // the same for the whole CTA: tcgen05.ld is warp-wide
                tmem_ld_32x32(t_row + 256 + 32 * NB * m + 32 * c, o1);
                tmem_ld_32x32(t_row + 256 + 64 * NB + 32 * NB * m + 32 * c, o2);
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
                *reinterpret_cast<uint4 *>(out + 32 * c + x) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
            }
        }
    }
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    if (warp == 8) tmem_dealloc(tmem, kCols);
}

// From this many tokens a region's query tiles of 128 rows are full enough, and its keys many enough, that
// the tensor-core pipeline beats the register-tiled kernel.
constexpr int kUmmaRegion = 128;

// Heads of 64 or 128 channels; with 128 the ring leaves room for rows of at most 188 routed regions.
bool diff_umma_supports(const Geometry &g)
{
    if (g.rs < kUmmaRegion) return false;
    return (g.hd == 64 && UmmaTile<1>::bytes(g.topk) <= 227 * 1024) || (g.hd == 128 && UmmaTile<2>::bytes(g.topk) <= 227 * 1024);
}

namespace {

template <int NB> cudaError_t launch_nb(const DiffArgs &a, int grid, cudaStream_t stream)
{
    cudaError_t e = grant_shared_memory<diff_attend_umma_kernel<NB>>();
    if (e != cudaSuccess) return e;
    // registers of the launch, as compiled: a split that asks for more would wait forever
    static const int regs = [] {
        cudaFuncAttributes at;
        return cudaFuncGetAttributes(&at, diff_attend_umma_kernel<NB>) == cudaSuccess ? at.numRegs : 0;
    }();
    if (regs * kThreads < 256 * kManyRegs + 128 * kFewRegs) return cudaErrorInvalidConfiguration;
    return launch_pdl(diff_attend_umma_kernel<NB>, dim3(grid), dim3(kThreads), UmmaTile<NB>::bytes(a.topk), stream, a);
}

}  // namespace

cudaError_t launch_diff_attend_umma(const DiffArgs &args, cudaStream_t stream)
{
    DiffArgs a = args;
    a.tiles = (a.rs + 127) / 128;
    a.by_tiles = FastDiv::of(a.tiles);
    const long long items = (long long)a.B * a.R * a.tiles * a.heads;
    if (items > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    a.nitems = (int)items;
    return a.hd == 64 ? launch_nb<1>(a, (int)items, stream) : launch_nb<2>(a, (int)items, stream);
}

}  // namespace bra
