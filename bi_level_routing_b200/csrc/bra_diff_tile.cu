// bra_diff_tile.cu -- forward differential attention of bf16 maps where a query meets at most 64 keys
// (formula in bra_diff.cuh), on mma.sync: every named stage routes so few. All scores of a row are in
// registers at once, so both softmaxes are complete before the product with v, and one product of
// P1 / l1 - lam P2 / l2 serves both maps (bra_diff_mma.cu, whose sums run on, needs two): half the
// PV work, half the accumulators, and twice the CTAs on an SM. Latency bounds these sizes: a CTA is an index
// load, a gather, four products and a store, and the SM overlaps as many CTAs as fit (64 images of 56 x 56,
// one head of 64, one region of 64 tokens to a query: 36 us, 2.8 TB/s; bra_diff_mma.cu 48).
//
// GATHER: a group of WPI warps owns 16 WPI query tokens of one (image, region, head) and the rows of its
// routed regions, as in bra_diff_mma.cu. DENSE (maps of at most 64 tokens in regions of at most 8, where a
// region would fill few of a tile's 16 rows): four warps own all tokens of one (image, head) against all
// tokens, each pair weighted by how often the query's region names the key's (0: no key).
//
// Precision: as bra_diff_mma.cu; the combined probability is rounded to bf16 once.
#include "bra_diff.cuh"

namespace bra {

namespace {

constexpr int kWarps = 4;
constexpr int kTileKeys = 64;

constexpr int pow2_at_least(int x)
{
    int p = 1;
    while (p < x) p *= 2;
    return p;
}

template <int DK, int WPI, int KT, bool DENSE> struct TilePlan {
    static constexpr int kGroups = kWarps / WPI;
    static constexpr int kHp = 2 * DK;
    static constexpr int kRow = kHp + 8;  // bf16 per row: an odd number of 16-byte chunks
    static constexpr int kLanes = pow2_at_least(kHp / 8);
    static constexpr int kRows = KT > 16 * WPI ? KT : 16 * WPI;  // the out rows leave through the K tile
    // K and V tiles, then the region list (16 + 4 topk bytes) or the pair counts (64 x 64 bytes) and a bit for each key
    static constexpr size_t group_bytes(int topk)
    {
        return (size_t)(kRows + KT) * kRow * 2 + (DENSE ? 64 * 64 + 16 : 16 + (((size_t)topk * 4 + 15) & ~(size_t)15));
    }
};

}  // namespace

template <int DK, int WPI, int KT, bool DENSE>
__global__ void __launch_bounds__(32 * kWarps, DK <= 32 ? 4 : 3) diff_attend_tile_kernel(const DiffArgs a)
{
    using L = TilePlan<DK, WPI, KT, DENSE>;
    constexpr int HP = L::kHp, ROW = L::kRow, NK = DK / 16, NT = KT / 8;
    extern __shared__ float4 smem4[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = warp / WPI, wg = warp % WPI, gtid = threadIdx.x % (32 * WPI);
    uint8_t *mine = reinterpret_cast<uint8_t *>(smem4) + (size_t)group * L::group_bytes(a.topk);
    __nv_bfloat16 *sk = reinterpret_cast<__nv_bfloat16 *>(mine), *sv = sk + L::kRows * ROW;
    uint8_t *tail = mine + (size_t)(L::kRows + KT) * ROW * 2;
    int *count = reinterpret_cast<int *>(tail), *bases = count + 4;
    uint32_t *pairs = reinterpret_cast<uint32_t *>(tail);  // [64 queries][64 keys] bytes
    uint32_t *wild = pairs + 64 * 16;                      // [2] keys whose values are not all finite
    const int item = blockIdx.x * L::kGroups + group;
    if (item >= a.nitems) return;  // the whole group: its barriers are its own
    DiffItem it = diff_item(a, item);  // DENSE: the launcher counts one region and one tile
    const int64_t image = (int64_t)it.b * a.N * a.C + it.h * a.hd;
    const __nv_bfloat16 *gk = static_cast<const __nv_bfloat16 *>(a.k) + image;
    const __nv_bfloat16 *gv = static_cast<const __nv_bfloat16 *>(a.v) + image;
    const int region = DENSE ? 0 : region_at(a, it.r);
    const int tok0 = (DENSE ? 0 : it.t * 16 * WPI) + 16 * wg;
    const int ntok = DENSE ? a.N : a.rs;
    auto token = [&](int tok) { return DENSE ? tok : token_at(a, region, tok); };
    if (DENSE)
        for (int e = gtid; e < 64 * 16 + 2; e += 32 * WPI) pairs[e] = 0u;
    grid_dependency_wait();

    int nkeys;
    if (DENSE) {
        nkeys = a.N;
    } else {
        if (wg == 0) {
            const int n = gather_bases(a, a.idx + ((int64_t)it.b * a.R + it.r) * a.topk, bases, lane);
            if (lane == 0) *count = n;
        }
        group_barrier<WPI>(group);
        nkeys = *count * a.rs;
    }
    {
        const int j = lane % L::kLanes, r0 = wg * (KT / WPI);
        warp_rows<KT / WPI, L::kLanes>(
            lane,
            [&](int row) {
                if (r0 + row >= nkeys) return -1;
                if (DENSE) return r0 + row;
                int slot, tok;
                a.by_rs.divmod(r0 + row, slot, tok);
                return token_at(a, bases[slot], tok);
            },
            [&](int row, int at) {
                if (j >= HP / 8) return;
                const int64_t off = (int64_t)max(at, 0) * a.C;
                copy_split<DK>(smem_u32(sk + (r0 + row) * ROW), gk + off, j, a.d, at >= 0);
                copy_run(smem_u32(sv + (r0 + row) * ROW), gv + off, j, a.hd, at >= 0);
            });
        cp_async_commit();
    }
    // the warp's query rows g and g + 8, both maps, as A fragments straight from global memory
    const int g = lane >> 2, t = lane & 3;
    uint32_t qf[2][NK][4];
    {
        const __nv_bfloat16 *gq = static_cast<const __nv_bfloat16 *>(a.q) + image;
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            const int tok = tok0 + g + 8 * hh;
            const bool in = tok < ntok;
            const __nv_bfloat16 *row = gq + (int64_t)(in ? token(tok) : 0) * a.C;
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
    const float lam = __ldg(a.lam + it.h);
    if (DENSE) {
        group_barrier<WPI>(group);  // the counts are cleared
        const int32_t *row = a.idx + (int64_t)it.b * a.R * a.topk;
        constexpr int kAhead = 10;  // index entries in flight for each thread
        for (int e0 = gtid; e0 < a.R * a.topk; e0 += kAhead * 32 * WPI) {
            int named[kAhead];
#pragma unroll
            for (int x = 0; x < kAhead; ++x) {
                const int e = e0 + x * 32 * WPI;
                named[x] = e < a.R * a.topk ? __ldg(row + e) : 0;
            }
#pragma unroll
            for (int x = 0; x < kAhead; ++x) {
                const int e = e0 + x * 32 * WPI, s = named[x];
                if (e >= a.R * a.topk) break;
                if (s < 0 || s >= a.R) {
                    flag_error(a.err, kErrIndex);
                    continue;
                }
                const int from = region_at(a, a.by_topk.div(e)), to = region_at(a, s);
                for (int y = 0; y < a.rs; ++y) {
                    const int query = token_at(a, from, y);
                    for (int z = 0; z < a.rs; ++z) {
                        const int key = token_at(a, to, z);
                        atomicAdd(pairs + query * 16 + (key >> 2), 1u << (8 * (key & 3)));  // at most topk <= 64 of each
                    }
                }
            }
        }
    }
    cp_async_wait_all();
    group_barrier<WPI>(group);
    if (DENSE) {
        // A key's values reach every query's product, 0 times those of a pair that does not meet. Infinities
        // and NaN must not: they are taken out of the tile here and put back, below, for the queries that name them.
        for (int e = gtid; e < KT * (HP / 8); e += 32 * WPI) {
            const int key = e / (HP / 8), c = e % (HP / 8);
            if (8 * c >= a.hd) continue;
            uint4 *at = reinterpret_cast<uint4 *>(sv + key * ROW + 8 * c);
            uint32_t x[4] = {at->x, at->y, at->z, at->w};
            uint32_t found = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t bad = __vcmpeq2(x[i] & 0x7f807f80u, 0x7f807f80u);  // exponents of ones
                found |= bad;
                x[i] &= ~bad;
            }
            if (found) {
                *at = make_uint4(x[0], x[1], x[2], x[3]);
                atomicOr(wild + (key >> 5), 1u << (key & 31));
            }
        }
        group_barrier<WPI>(group);
    }

    const uint32_t k0 = smem_u32(sk), v0 = smem_u32(sv);
    float s[2][NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[m][nt][i] = 0.f;
#pragma unroll
        for (int c4 = 0; c4 < HP / 32; ++c4) {
            uint32_t b[4];
            ldmatrix_x4(k0 + ((8 * nt + (lane & 7)) * ROW + 32 * c4 + 8 * (lane >> 3)) * 2, b[0], b[1], b[2], b[3]);
            constexpr int n = NK;
            mma_bf16_16816(s[(2 * c4) / n][nt], qf[(2 * c4) / n][(2 * c4) % n], b[0], b[1]);
            mma_bf16_16816(s[(2 * c4 + 1) / n][nt], qf[(2 * c4 + 1) / n][(2 * c4 + 1) % n], b[2], b[3]);
        }
        // pairs that do not meet: past the last key, or not named
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            uint32_t named = 0;
            if (DENSE) named = reinterpret_cast<const uint16_t *>(pairs)[(tok0 + g + 8 * hh) * 32 + 4 * nt + t];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const bool none = DENSE ? ((named >> (8 * i)) & 255u) == 0u : 8 * nt + 2 * t + i >= nkeys;
                if (none) s[0][nt][2 * hh + i] = s[1][nt][2 * hh + i] = -INFINITY;
            }
        }
    }
    // s[0] becomes P1 / l1 - lam P2 / l2; a row without keys has l = 0 and becomes 0
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
        float w[2];
        bool keys = false;  // the row has any
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            float top = -INFINITY;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) top = fmax3(top, s[m][nt][2 * hh], s[m][nt][2 * hh + 1]);
            const float base = score_base(quad_max(top) * a.scale_log2);
            float sum = 0.f;
            uint32_t some = 0;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                uint32_t named = 0;
                if (DENSE) named = reinterpret_cast<const uint16_t *>(pairs)[(tok0 + g + 8 * hh) * 32 + 4 * nt + t];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float e = fast_exp2(fmaf(s[m][nt][2 * hh + i], a.scale_log2, -base));
                    if (DENSE) e *= (float)((named >> (8 * i)) & 255u);
                    if (DENSE && m == 0) some |= named;
                    s[m][nt][2 * hh + i] = e;
                    sum += e;
                }
            }
            if (m == 0) {
                some |= __shfl_xor_sync(0xffffffffu, some, 1);
                some |= __shfl_xor_sync(0xffffffffu, some, 2);
                keys = DENSE ? some != 0u : nkeys > 0;
            }
            w[m] = over_sum(m ? -lam : 1.f, quad_sum(sum), keys);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                s[0][nt][2 * hh + i] = fmaf(s[0][nt][2 * hh + i], w[0], s[1][nt][2 * hh + i] * w[1]);
    }
    uint32_t p[KT / 16][4];
#pragma unroll
    for (int ks = 0; ks < KT / 16; ++ks) {
        p[ks][0] = pack_bf16x2(s[0][2 * ks][0], s[0][2 * ks][1]);
        p[ks][1] = pack_bf16x2(s[0][2 * ks][2], s[0][2 * ks][3]);
        p[ks][2] = pack_bf16x2(s[0][2 * ks + 1][0], s[0][2 * ks + 1][1]);
        p[ks][3] = pack_bf16x2(s[0][2 * ks + 1][2], s[0][2 * ks + 1][3]);
    }
    group_barrier<WPI>(group);  // every warp has read K: the out rows go through its tile
    __nv_bfloat16 *rows = sk + (size_t)wg * 16 * ROW;
#pragma unroll
    for (int np = 0; np < HP / 16; ++np) {
        if (16 * np >= a.hd) break;
        float o[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int ks = 0; ks < KT / 16; ++ks) {
            uint32_t b[4];
            ldmatrix_x4_trans(v0 + ((16 * ks + (lane & 15)) * ROW + 16 * np + 8 * (lane >> 4)) * 2, b[0], b[1], b[2], b[3]);
            mma_bf16_16816(o[0], p[ks], b[0], b[1]);
            mma_bf16_16816(o[1], p[ks], b[2], b[3]);
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            *reinterpret_cast<uint32_t *>(rows + g * ROW + 16 * np + 8 * x + 2 * t) = pack_bf16x2(o[x][0], o[x][1]);
            *reinterpret_cast<uint32_t *>(rows + (g + 8) * ROW + 16 * np + 8 * x + 2 * t) = pack_bf16x2(o[x][2], o[x][3]);
        }
    }
    __syncwarp();
    if (DENSE && (wild[0] | wild[1]) != 0u) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            for (int x = 0; x < 16; ++x) {  // key 8 nt + x / 2 against rows of this half
                const int key = 8 * nt + x / 2, hh = x & 1;
                if (!((wild[key >> 5] >> (key & 31)) & 1u)) continue;
                const uint32_t packed = hh ? p[nt / 2][2 * (nt & 1) + 1] : p[nt / 2][2 * (nt & 1)];
                for (int gg = 0; gg < 8; ++gg) {
                    const uint32_t both = __shfl_sync(0xffffffffu, packed, 4 * gg + (key & 7) / 2);
                    const float prob = __uint_as_float((key & 1) ? both & 0xffff0000u : both << 16);
                    const int row = gg + 8 * hh;
                    if (((pairs[(tok0 + row) * 16 + (key >> 2)] >> (8 * (key & 3))) & 255u) == 0u) continue;
                    for (int c = lane; c < a.hd; c += 32) {
                        const float v = __bfloat162float(gv[(int64_t)key * a.C + c]);
                        if (!isfinite(v)) rows[row * ROW + c] = __float2bfloat16_rn(__bfloat162float(rows[row * ROW + c]) + prob * v);
                    }
                }
            }
        __syncwarp();
    }
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + image;
    const int j = lane % L::kLanes;
    if (8 * j < a.hd)
        for (int row = lane / L::kLanes; row < 16; row += 32 / L::kLanes) {
            const int tok = tok0 + row;
            if (tok < ntok)
                *reinterpret_cast<uint4 *>(out + (int64_t)token(tok) * a.C + 8 * j) =
                    *reinterpret_cast<const uint4 *>(rows + row * ROW + 8 * j);
        }
}

bool diff_tile_supports(const Geometry &g) { return (long long)g.topk * g.rs <= kTileKeys; }

namespace {

template <int DK, int WPI, int KT, bool DENSE> cudaError_t launch_one(DiffArgs &a, cudaStream_t stream)
{
    using L = TilePlan<DK, WPI, KT, DENSE>;
    DiffArgs b = a;
    b.tiles = DENSE ? 1 : (a.rs + 16 * WPI - 1) / (16 * WPI);
    b.by_tiles = FastDiv::of(b.tiles);
    if (DENSE) b.by_R = FastDiv::of(1);  // items are (image, head)
    const long long items = (long long)a.B * (DENSE ? 1 : a.R) * b.tiles * a.heads;
    if (items > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    b.nitems = (int)items;
    const cudaError_t e = grant_shared_memory<diff_attend_tile_kernel<DK, WPI, KT, DENSE>>();
    if (e != cudaSuccess) return e;
    const int grid = (int)((items + L::kGroups - 1) / L::kGroups);
    return launch_pdl(diff_attend_tile_kernel<DK, WPI, KT, DENSE>, dim3(grid), dim3(32 * kWarps),
                      L::kGroups * L::group_bytes(a.topk), stream, b);
}

template <int DK> cudaError_t launch_dk(DiffArgs &a, cudaStream_t stream)
{
    const bool few = a.topk * a.rs <= 32;
    // The dense mode from where the gathering warps are more than an SM holds (12): 49 one-token regions, all routed, 8 heads,
    // 1 / 4 / 8 / 64 images: gathered 5.7 / 7.5 / 13.6 / 78.5 us, dense 11.0 / 10.7 / 10.9 / 14.9 us.
    const bool crowded = (long long)a.B * a.R * a.heads > 12LL * a.num_sms;
    if (a.N <= 64 && a.rs <= 8 && crowded) return launch_one<DK, 4, 64, true>(a, stream);
    if (a.rs <= 16) return few ? launch_one<DK, 1, 32, false>(a, stream) : launch_one<DK, 1, 64, false>(a, stream);
    if (a.rs <= 32) return few ? launch_one<DK, 2, 32, false>(a, stream) : launch_one<DK, 2, 64, false>(a, stream);
    return launch_one<DK, 4, 64, false>(a, stream);
}

}  // namespace

cudaError_t launch_diff_attend_tile(const DiffArgs &args, cudaStream_t stream)
{
    DiffArgs a = args;
    if (a.d <= 16) return launch_dk<16>(a, stream);
    if (a.d <= 32) return launch_dk<32>(a, stream);
    if (a.d <= 48) return launch_dk<48>(a, stream);
    return launch_dk<64>(a, stream);
}

}  // namespace bra
