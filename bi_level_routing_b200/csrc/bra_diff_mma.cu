// bra_diff_mma.cu -- forward differential attention of bf16 maps on mma.sync (see bra_diff.cuh for
// the formula), heads of 8 to 128 channels in multiples of 8, regions of any size.
//
// One pass over the routed keys with the running maximum and sum of both softmaxes. A group of WPI
// warps owns 16 WPI query tokens of one (image, region, head); each warp keeps 16 query rows, its
// two score tiles and both maps' 16 x hd accumulators in registers. The routed regions' key and value
// rows are gathered one after the other into tiles of KT rows (regions of any size pack densely) by
// cp.async, the next tile landing while the warps work on the current one. Both maps multiply the
// same value fragment, so V is read from shared memory once for two products.
//
// Precision: products are of bf16 inputs, exact in fp32 sums; scores, maxima, sums and accumulators
// are fp32; P enters the PV product as bf16, its normaliser is summed from the fp32 values; out is
// rounded once.
//
// Latency bounds the routed sizes it serves (a gather, its wait and two dependent products a tile): 64 images of
// 28 x 28, 2 heads of 64, 8 regions of 16 tokens to a query 42 us; 16 images of 28 x 28, 4 heads,
// 4 regions of 49 tokens 40 us.
#include "bra_diff.cuh"

namespace bra {

namespace {

constexpr int kWarps = 4;

constexpr int pow2_at_least(int x)
{
    int p = 1;
    while (p < x) p *= 2;
    return p;
}

template <int DK, int WPI, int KT> struct DiffTile {
    static constexpr int kGroups = kWarps / WPI;
    static constexpr int kHp = 2 * DK;       // padded head channels
    static constexpr int kRow = kHp + 8;     // bf16 per row: an odd number of 16-byte chunks, no ldmatrix conflicts
    static constexpr int kLanes = pow2_at_least(kHp / 8);  // threads that copy one row
    static constexpr size_t group_bytes(int topk) { return (size_t)4 * KT * kRow * 2 + (((size_t)topk * 4 + 15) & ~(size_t)15) + 16; }
};

}  // namespace

template <int DK, int WPI, int KT>
__global__ void __launch_bounds__(32 * kWarps) diff_attend_mma_kernel(const DiffArgs a)
{
    using L = DiffTile<DK, WPI, KT>;
    constexpr int HP = L::kHp, ROW = L::kRow, NK = DK / 16, NT = KT / 8;
    extern __shared__ float4 smem4[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = warp / WPI, wg = warp % WPI;
    uint8_t *mine = reinterpret_cast<uint8_t *>(smem4) + (size_t)group * L::group_bytes(a.topk);
    __nv_bfloat16 *tiles = reinterpret_cast<__nv_bfloat16 *>(mine);  // [stage][K, V][KT][ROW]
    int *count = reinterpret_cast<int *>(mine + (size_t)4 * KT * ROW * 2);
    int *bases = count + 4;
    const int item = blockIdx.x * L::kGroups + group;
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

    const int64_t image = (int64_t)it.b * a.N * a.C + it.h * a.hd;  // first element of this image and head
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

    // the warp's query rows g and g + 8, both maps, as A fragments straight from global memory
    const int g = lane >> 2, t = lane & 3;
    const int region = region_at(a, it.r);
    const int tok0 = it.t * 16 * WPI + 16 * wg;
    uint32_t qf[2][NK][4];
    {
        const __nv_bfloat16 *gq = static_cast<const __nv_bfloat16 *>(a.q) + image;
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            const int tok = tok0 + g + 8 * hh;
            const bool in = tok < a.rs;
            const __nv_bfloat16 *row = gq + (int64_t)(in ? token_at(a, region, tok) : 0) * a.C;
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int ks = 0; ks < NK; ++ks)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const int c = 16 * ks + 8 * half + 2 * t;
                        qf[m][ks][hh + 2 * half] =
                            in && c < a.d ? __ldg(reinterpret_cast<const uint32_t *>(row + m * a.d + c)) : 0u;
                    }
        }
    }

    float o[2][HP / 8][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int nt = 0; nt < HP / 8; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[m][nt][i] = 0.f;
    float mx[2][2] = {{-INFINITY, -INFINITY}, {-INFINITY, -INFINITY}}, l[2][2] = {{0.f, 0.f}, {0.f, 0.f}};

    for (int tile = 0; tile < ntiles; ++tile) {
        const int stage = tile & 1;
        cp_async_wait_all();
        group_barrier<WPI>(group);  // this tile is in place; every warp has left the other stage
        if (tile + 1 < ntiles) fetch(tile + 1, stage ^ 1);
        const uint32_t k0 = smem_u32(tiles + (size_t)stage * 2 * KT * ROW);
        const uint32_t v0 = k0 + KT * ROW * 2;

        float s[2][NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[m][nt][i] = 0.f;
#pragma unroll
            for (int c4 = 0; c4 < HP / 32; ++c4) {  // 32 channels: two steps of 16
                uint32_t b[4];
                ldmatrix_x4(k0 + ((8 * nt + (lane & 7)) * ROW + 32 * c4 + 8 * (lane >> 3)) * 2, b[0], b[1], b[2], b[3]);
                constexpr int n = NK;
                mma_bf16_16816(s[(2 * c4) / n][nt], qf[(2 * c4) / n][(2 * c4) % n], b[0], b[1]);
                mma_bf16_16816(s[(2 * c4 + 1) / n][nt], qf[(2 * c4 + 1) / n][(2 * c4 + 1) % n], b[2], b[3]);
            }
        }
        if ((tile + 1) * KT > nkeys) {  // rows past the last key
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (tile * KT + 8 * nt + 2 * t + (i & 1) >= nkeys) s[0][nt][i] = s[1][nt][i] = -INFINITY;
        }
        uint32_t p[2][KT / 16][4];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            float corr[2];
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                float top = -INFINITY;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) top = fmax3(top, s[m][nt][2 * hh], s[m][nt][2 * hh + 1]);
                const float most = fmaxf(mx[m][hh], quad_max(top) * a.scale_log2), base = score_base(most);
                corr[hh] = fast_exp2(mx[m][hh] - base);
                mx[m][hh] = most;
                float sum = 0.f;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float e = fast_exp2(fmaf(s[m][nt][2 * hh + i], a.scale_log2, -base));
                        s[m][nt][2 * hh + i] = e;
                        sum += e;
                    }
                l[m][hh] = l[m][hh] * corr[hh] + sum;
            }
            // the accumulators follow only when a row's maximum moved, which it seldom does late
            if (__any_sync(0xffffffffu, corr[0] != 1.f || corr[1] != 1.f)) {
#pragma unroll
                for (int nt = 0; nt < HP / 8; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[m][nt][i] *= corr[i >> 1];
            }
#pragma unroll
            for (int ks = 0; ks < KT / 16; ++ks) {
                p[m][ks][0] = pack_bf16x2(s[m][2 * ks][0], s[m][2 * ks][1]);
                p[m][ks][1] = pack_bf16x2(s[m][2 * ks][2], s[m][2 * ks][3]);
                p[m][ks][2] = pack_bf16x2(s[m][2 * ks + 1][0], s[m][2 * ks + 1][1]);
                p[m][ks][3] = pack_bf16x2(s[m][2 * ks + 1][2], s[m][2 * ks + 1][3]);
            }
        }
#pragma unroll
        for (int np = 0; np < HP / 16; ++np) {
            if (16 * np >= a.hd) break;
#pragma unroll
            for (int ks = 0; ks < KT / 16; ++ks) {
                uint32_t b[4];
                ldmatrix_x4_trans(v0 + ((16 * ks + (lane & 15)) * ROW + 16 * np + 8 * (lane >> 4)) * 2, b[0], b[1], b[2], b[3]);
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    mma_bf16_16816(o[m][2 * np], p[m][ks], b[0], b[1]);
                    mma_bf16_16816(o[m][2 * np + 1], p[m][ks], b[2], b[3]);
                }
            }
        }
    }

    // out = O1 / l1 - lam O2 / l2, through shared memory so that whole rows are stored; a query
    // without keys has l = 0 and gets 0
    group_barrier<WPI>(group);
    const float lam = __ldg(a.lam + it.h);
    __nv_bfloat16 *rows = tiles + (size_t)wg * 16 * ROW;
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
        const float w1 = over_sum(1.f, quad_sum(l[0][hh]), nkeys > 0), w2 = over_sum(-lam, quad_sum(l[1][hh]), nkeys > 0);
#pragma unroll
        for (int nt = 0; nt < HP / 8; ++nt) {
            const float x = fmaf(o[0][nt][2 * hh], w1, o[1][nt][2 * hh] * w2);
            const float y = fmaf(o[0][nt][2 * hh + 1], w1, o[1][nt][2 * hh + 1] * w2);
            *reinterpret_cast<uint32_t *>(rows + (g + 8 * hh) * ROW + 8 * nt + 2 * t) = pack_bf16x2(x, y);
        }
    }
    __syncwarp();
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + image;
    constexpr int lanes = L::kLanes < 32 ? L::kLanes : 32;
    const int j = lane % lanes;
    if (8 * j < a.hd)
        for (int row = lane / lanes; row < 16; row += 32 / lanes) {
            const int tok = tok0 + row;
            if (tok < a.rs)
                *reinterpret_cast<uint4 *>(out + (int64_t)token_at(a, region, tok) * a.C + 8 * j) =
                    *reinterpret_cast<const uint4 *>(rows + row * ROW + 8 * j);
        }
}

namespace {

template <int DK, int WPI, int KT> cudaError_t launch_one(DiffArgs &a, cudaStream_t stream)
{
    using L = DiffTile<DK, WPI, KT>;
    a.tiles = (a.rs + 16 * WPI - 1) / (16 * WPI);
    a.by_tiles = FastDiv::of(a.tiles);
    const long long items = (long long)a.B * a.R * a.tiles * a.heads;
    if (items > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    a.nitems = (int)items;
    const size_t smem = L::kGroups * L::group_bytes(a.topk);
    const cudaError_t e = grant_shared_memory<diff_attend_mma_kernel<DK, WPI, KT>>();
    if (e != cudaSuccess) return e;
    const int grid = (int)((items + L::kGroups - 1) / L::kGroups);
    return launch_pdl(diff_attend_mma_kernel<DK, WPI, KT>, dim3(grid), dim3(32 * kWarps), smem, stream, a);
}

// A region of up to 16 tokens is one warp's, of up to 32 two warps' (a group's warps share the tiles it
// gathers, and none may be without rows), larger ones are cut into tiles of 64 rows for four warps.
template <int DK> cudaError_t launch_dk(DiffArgs &a, cudaStream_t stream)
{
    constexpr int KT = DK <= 32 ? 64 : 32;
    if (a.rs <= 16) return launch_one<DK, 1, 32>(a, stream);
    if (a.rs <= 32) return launch_one<DK, 2, 32>(a, stream);
    return launch_one<DK, 4, KT>(a, stream);
}

}  // namespace

cudaError_t launch_diff_attend_mma(const DiffArgs &args, cudaStream_t stream)
{
    DiffArgs a = args;
    if (a.d <= 16) return launch_dk<16>(a, stream);
    if (a.d <= 32) return launch_dk<32>(a, stream);
    if (a.d <= 48) return launch_dk<48>(a, stream);
    return launch_dk<64>(a, stream);
}

}  // namespace bra
