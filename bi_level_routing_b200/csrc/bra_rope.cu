// bra_rope.cu -- rotary positions of q and k. The first 2 axes n channels of every head are `axes`
// blocks of n pairs; pair i of block a is turned by the angle t = position[a] * freqs[i],
//   (u, w) -> mscale (u cos t - w sin t, w cos t + u sin t),
// the inverse by -t (the gradients' way back: the map is linear, its transpose turns by -t and keeps
// mscale). The pairs are (i, i + n) of the block, or (2 i, 2 i + 1) interleaved; the other channels are
// copied. Positions: row and column (axes = 2) or raster number (axes = 1) from an origin, or given per
// token.
//
// The bytes of q and k are the bound. A thread owns one unit of a token's head, 2 VEC channels, and
// its VEC angles, which are the same for every image, head and tensor at that position: it forms sine
// and cosine once and keeps them in registers while it goes through the images, heads and
// tensors of its slice (given positions differ by image, and are formed for each). The angle in turns,
// position * freq / 2 pi, is formed and reduced to [-1/2, 1/2] in 64 bits (fp32 would lose one turn in
// 2^24 at far positions), sine and cosine of the remainder in 32. q and k of 64 images of 56 x 56, 64 channels,
// bf16: 20.3 us from cold, 5.1 TB/s; of 8 images of 128 x 128, 64 channels, fp32, given positions: 23.6 us,
// 5.7 TB/s.
#include "bra_device.cuh"
#include "bra_diff.cuh"
#include "bra_launch.h"

namespace bra {

namespace {

template <int BYTES> struct RopeWord;
template <> struct RopeWord<2> { using type = unsigned short; };
template <> struct RopeWord<4> { using type = uint32_t; };
template <> struct RopeWord<8> { using type = uint2; };
template <> struct RopeWord<16> { using type = uint4; };

// VEC values as one load or store of VEC * sizeof(T) bytes
template <typename T, int VEC> struct RopeVec {
    using Word = typename RopeWord<VEC * sizeof(T)>::type;
    union {
        Word word;
        T value[VEC];
    };
    __device__ __forceinline__ RopeVec() {}
    __device__ __forceinline__ void load(const T *p) { word = *reinterpret_cast<const Word *>(p); }
    __device__ __forceinline__ void store(T *p) const { *reinterpret_cast<Word *>(p) = word; }
};

constexpr int kRopeThreads = 256;

struct RopePlan {
    FastDiv by_units, by_W;
    int units;      // of a head: 2 VEC channels each
    int side;       // heads side by side in a warp, so that it reads whole 128-byte lines
    int turned;     // of them, those that are turned
    int per_block;  // units of one axis' block
    int groups;     // (image, `side` heads) pairs, or groups of heads where positions are given
    int per;        // (tensor, image, head) triples of a CTA
    int64_t threads;  // tokens * units * side
};

}  // namespace

// VEC: elements of one access; GIVEN: positions are read per token (of each image)
template <typename T, int VEC, bool GIVEN>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs a, const RopePlan p)
{
    const int64_t e = (int64_t)blockIdx.x * kRopeThreads + threadIdx.x;
    if (e >= p.threads) return;
    const int64_t tok64 = e / (p.units * p.side);  // of an image; of the whole batch where positions are given
    const int within = (int)(e - tok64 * (p.units * p.side)), hs = within / p.units, u = within - hs * p.units;
    const int stacks = a.heads / p.side;
    const int N = a.H * a.W;
    grid_dependency_wait();

    // the unit's channels: VEC from ca and VEC from cb; its angles: pairs i0 ..
    const bool turned = u < p.turned;
    int ca = 2 * VEC * u, cb = ca + VEC, i0 = 0, axis = 0;
    if (turned) {
        axis = u / p.per_block;
        i0 = (u - axis * p.per_block) * VEC;
        if (!a.interleaved) {
            ca = 2 * a.n * axis + i0;
            cb = ca + a.n;
        }
    }
    float c[VEC], s[VEC];
    if (turned) {
        int64_t at;
        if (GIVEN) {
            at = __ldg(a.pos + tok64 * a.axes + axis);
        } else {
            const int tok = (int)tok64;
            int y, x;
            p.by_W.divmod(tok, y, x);
            at = a.axes == 2 ? (axis ? a.x0 + x : a.y0 + y) : (a.y0 + y) * a.W + a.x0 + x;
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const double turns = (double)at * (double)__ldg(a.freqs + i0 + i) * 0.15915494309189533577;
            const float half_turns = (float)(2.0 * (turns - rint(turns)));
            sincospif(half_turns, &s[i], &c[i]);
            c[i] *= a.mscale;
            s[i] *= a.inverse ? -a.mscale : a.mscale;
        }
    }
    // groups: (image, heads) pairs, heads fastest; all of q, then all of k
    const int64_t first = tok64 * a.C;
    const int64_t per_image = (int64_t)N * a.C;
    constexpr int kBatch = 2;  // triples in flight (64 images of 56 x 56, 64 channels: 20.2 us; 4: 22.6 us)
    const int begin = blockIdx.y * p.per, total = min(p.groups * a.tensors, begin + p.per);
    for (int g0 = begin; g0 < total; g0 += kBatch) {
        RopeVec<T, VEC> va[kBatch], vb[kBatch];
        int64_t off[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int gi = g0 + j;
            if (gi >= total) break;
            const int tensor = gi >= p.groups, pair = gi - tensor * p.groups;
            const int b = GIVEN ? 0 : pair / stacks, h = (pair - b * stacks) * p.side + hs;
            off[j] = b * per_image + first + h * a.hd;
            const T *src = static_cast<const T *>(tensor ? a.k : a.q) + off[j];
            va[j].load(src + ca);
            vb[j].load(src + cb);
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int gi = g0 + j;
            if (gi >= total) break;
            if (turned) {
                if (a.interleaved) {
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {  // pair i: elements 2 i, 2 i + 1 of the unit's 2 VEC
                        T &x = 2 * i < VEC ? va[j].value[(2 * i) % VEC] : vb[j].value[(2 * i) % VEC];
                        T &y = 2 * i + 1 < VEC ? va[j].value[(2 * i + 1) % VEC] : vb[j].value[(2 * i + 1) % VEC];
                        const float fx = to_float(x), fy = to_float(y);
                        x = from_float<T>(fx * c[i] - fy * s[i]);
                        y = from_float<T>(fy * c[i] + fx * s[i]);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        const float fx = to_float(va[j].value[i]), fy = to_float(vb[j].value[i]);
                        va[j].value[i] = from_float<T>(fx * c[i] - fy * s[i]);
                        vb[j].value[i] = from_float<T>(fy * c[i] + fx * s[i]);
                    }
                }
            }
            T *dst = static_cast<T *>(gi >= p.groups ? a.k_out : a.q_out) + off[j];
            va[j].store(dst + ca);
            vb[j].store(dst + cb);
        }
    }
}

namespace {

template <typename T, int VEC> cudaError_t launch_vec(const RopeArgs &a, int num_sms, cudaStream_t stream)
{
    RopePlan p;
    p.units = a.hd / (2 * VEC);
    p.per_block = a.n / VEC;
    p.turned = a.axes * p.per_block;
    p.by_W = FastDiv::of(a.W);
    const bool given = a.pos != nullptr;
    const int64_t tokens = (int64_t)a.H * a.W * (given ? a.B : 1);
    p.side = 1;
    while (a.heads % (2 * p.side) == 0 && 2 * p.side * a.hd * (int)sizeof(T) <= 128) p.side *= 2;
    p.threads = tokens * p.units * p.side;
    const int64_t groups = (int64_t)(given ? 1 : a.B) * (a.heads / p.side);
    if (groups * 2 > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    p.groups = (int)groups;
    const int64_t blocks = (p.threads + kRopeThreads - 1) / kRopeThreads;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    // enough CTAs for eight to an SM; a slice still goes through several (image, head, tensor) triples,
    // so that its angles serve more than one
    int64_t slices = (8LL * num_sms + blocks - 1) / blocks;
    const int64_t most = (groups * a.tensors + 3) / 4;
    if (slices > most) slices = most;
    if (slices > 65535) slices = 65535;
    if (slices < 1) slices = 1;
    p.per = (int)((groups * a.tensors + slices - 1) / slices);
    const dim3 grid((unsigned)blocks, (unsigned)((groups * a.tensors + p.per - 1) / p.per));
    return given ? launch_pdl(rope_kernel<T, VEC, true>, grid, dim3(kRopeThreads), 0, stream, a, p)
                 : launch_pdl(rope_kernel<T, VEC, false>, grid, dim3(kRopeThreads), 0, stream, a, p);
}

}  // namespace

// The widest access that divides a block's pairs and the channels after them. Heads start at multiples
// of hd, so hd's own factors bound the alignment too.
cudaError_t launch_rope(const RopeArgs &a, bool bf16, int num_sms, cudaStream_t stream)
{
    int vec = bf16 ? 8 : 4;
    while (vec > 1 && (a.n % vec || a.hd % (2 * vec))) vec /= 2;
    if (!bf16) {
        if (vec == 4) return launch_vec<float, 4>(a, num_sms, stream);
        if (vec == 2) return launch_vec<float, 2>(a, num_sms, stream);
        return launch_vec<float, 1>(a, num_sms, stream);
    }
    if (vec == 8) return launch_vec<__nv_bfloat16, 8>(a, num_sms, stream);
    if (vec == 4) return launch_vec<__nv_bfloat16, 4>(a, num_sms, stream);
    if (vec == 2) return launch_vec<__nv_bfloat16, 2>(a, num_sms, stream);
    return launch_vec<__nv_bfloat16, 1>(a, num_sms, stream);
}

}  // namespace bra
