// bra_norm.cu -- the norms around a block, fused with its gate and residual, and their gradients.
//
// For every token row of C channels, x the residual stream and h the block's output:
//   s = alpha x + gate * (norm(h) w_post + b_post),    y = norm(s) w_pre + b_pre,
// norm(z) = (z - mean z) / sqrt(mean (z - mean z)^2 + eps) (LayerNorm) or z / sqrt(mean z^2 + eps) (RMS):
// the block's post-norm, its gate and the residual sum, and the next block's pre-norm, in one pass (x and
// h read once, s and y written once). Without w_post the branch is h itself; without h there is only
// y = norm(alpha x) w_pre + b_pre; without w_pre only s. With z^ = norm(z), r its 1 / sqrt(...), and
// N(u, z^, r) = r (u - mean(u) - z^ mean(u z^)) (RMS: without mean(u)), the gradients are
//   dS = ds + N(dy w_pre, s^, r_s),  dx = alpha dS,  dp = gate dS,  dh = N(dp w_post, h^, r_h),
//   dw_pre = sum dy s^, db_pre = sum dy, dgate = sum dS p, dw_post = sum dp h^, db_post = sum dp over rows.
//
// TPR threads hold one row in registers, VPT 16-byte vectors each; the next row's vectors load while
// the current one is worked on. Means are taken before the squares about them (two sums, no
// cancellation), all in fp32. The column sums of the backward pass stay in each thread's registers
// over the rows of its CTA; the CTAs' sums go to a workspace and are added in a fixed order, so the
// result is the same bits on every run.
#include "bra_device.cuh"
#include "bra_launch.h"

namespace bra {

namespace {

template <typename T, int VPT> struct RowVec {
    static constexpr int V = Vec16<T>::N;
    static constexpr int E = V * VPT;
};

// 16-byte loads that do not go through the read-only path (outputs may be the inputs' own buffers)
__device__ __forceinline__ uint4 load16(const void *p)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ uint4 pack16(const float (&f)[4], float)
{
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
__device__ __forceinline__ uint4 pack16(const float (&f)[8], __nv_bfloat16)
{
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

// Sums of K values over the TPR threads of a row. Rows of more than a warp meet in shared memory:
// `red` holds two sets of K values for each warp, used in turn, so one barrier a sum is enough.
template <int TPR, int K> __device__ __forceinline__ void row_sums(float (&v)[K], float *red, int &turn)
{
    constexpr int W = TPR < 32 ? TPR : 32;
#pragma unroll
    for (int o = W / 2; o; o >>= 1)
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    if (TPR > 32) {
        constexpr int kWarps = TPR / 32;
        const int warp = threadIdx.x >> 5;
        float *set = red + turn * 64;
        turn ^= 1;
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int k = 0; k < K; ++k) set[2 * warp + k] = v[k];
        __syncthreads();
        const float *own = set + 2 * (warp / kWarps * kWarps);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) sum += own[2 * w + k];
            v[k] = sum;
        }
    }
}

// z becomes norm(z); returns 1 / sqrt(...). `valid` says which elements lie in the row (whole vectors).
template <int TPR, int V, int VPT>
__device__ __forceinline__ float normalise(float (&z)[V * VPT], const NormArgs &a, int lane, float *red, int &turn)
{
    float sum[1];
    if (a.layer) {
        sum[0] = 0.f;
#pragma unroll
        for (int i = 0; i < V * VPT; ++i) sum[0] += z[i];  // elements past the row are 0
        row_sums<TPR, 1>(sum, red, turn);
        const float mean = sum[0] * a.inv_c;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (lane + i * TPR < a.nvec) {
#pragma unroll
                for (int j = 0; j < V; ++j) z[i * V + j] -= mean;
            }
    }
    sum[0] = 0.f;
#pragma unroll
    for (int i = 0; i < V * VPT; ++i) sum[0] = fmaf(z[i], z[i], sum[0]);
    row_sums<TPR, 1>(sum, red, turn);
    const float r = 1.f / sqrtf(fmaf(sum[0], a.inv_c, a.eps));
#pragma unroll
    for (int i = 0; i < V * VPT; ++i) z[i] *= r;
    return r;
}

// u becomes r (u - mean(u) - z^ mean(u z^)), the mean(u) term for LayerNorm only. Elements past the row
// are 0 in z^ and u and are not stored, so what they become does not matter.
template <int TPR, int E>
__device__ __forceinline__ void norm_back(float (&u)[E], const float (&z)[E], float r, const NormArgs &a, float *red, int &turn)
{
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < E; ++i) {
        sum[0] += u[i];
        sum[1] = fmaf(u[i], z[i], sum[1]);
    }
    row_sums<TPR, 2>(sum, red, turn);
    const float m0 = a.layer ? sum[0] * a.inv_c : 0.f, m1 = sum[1] * a.inv_c;
#pragma unroll
    for (int i = 0; i < E; ++i) u[i] = r * (u[i] - m0 - z[i] * m1);
}

// E values of a channel array at this thread's vectors; `def` where the array is absent or past the row.
template <int TPR, int V, int VPT>
__device__ __forceinline__ void load_channels(float (&w)[V * VPT], const float *p, float def, int nvec, int lane)
{
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < V / 4; ++j) {
            float4 f = make_float4(def, def, def, def);
            if (p && lane + i * TPR < nvec) f = __ldg(reinterpret_cast<const float4 *>(p) + (lane + i * TPR) * (V / 4) + j);
            w[i * V + 4 * j] = f.x;
            w[i * V + 4 * j + 1] = f.y;
            w[i * V + 4 * j + 2] = f.z;
            w[i * V + 4 * j + 3] = f.w;
        }
}

template <typename T, int TPR, int VPT>
__device__ __forceinline__ void load_row(uint4 (&raw)[VPT], const void *base, int64_t row, const NormArgs &a, int lane, bool in)
{
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        raw[i] = make_uint4(0, 0, 0, 0);
        if (in && base && lane + i * TPR < a.nvec)
            raw[i] = load16(static_cast<const T *>(base) + row * a.C + (int64_t)(lane + i * TPR) * Vec16<T>::N);
    }
}

template <typename T, int TPR, int VPT>
__device__ __forceinline__ void store_row(void *base, int64_t row, const NormArgs &a, int lane, const float (&f)[Vec16<T>::N * VPT])
{
    constexpr int V = Vec16<T>::N;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        if (lane + i * TPR < a.nvec) {
            float v[V];
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] = f[i * V + j];
            *reinterpret_cast<uint4 *>(static_cast<T *>(base) + row * a.C + (int64_t)(lane + i * TPR) * V) = pack16(v, T());
        }
}

template <typename T, int VPT> __device__ __forceinline__ void unpack_row(const uint4 (&raw)[VPT], float (&f)[Vec16<T>::N * VPT])
{
#pragma unroll
    for (int i = 0; i < VPT; ++i) Vec16<T>::unpack(raw[i], f + i * Vec16<T>::N);
}

constexpr int block_threads(int tpr) { return tpr > 256 ? tpr : 256; }

}  // namespace

template <typename T, int TPR, int VPT>
__global__ void __launch_bounds__(block_threads(TPR)) norm_residual_kernel(const NormArgs a)
{
    constexpr int V = Vec16<T>::N, E = V * VPT, RPC = block_threads(TPR) / TPR;
    constexpr bool kKeep = E <= 8;  // the channel arrays stay in registers (5 E of them); else they come from L1
    __shared__ float red[128];
    const int lane = threadIdx.x % TPR, grp = threadIdx.x / TPR;
    const int image = blockIdx.x / a.chunks, chunk = blockIdx.x - image * a.chunks;
    const int64_t row0 = (int64_t)image * a.rows;
    const int begin = chunk * a.per, end = min(a.rows, begin + a.per);
    const float *gate = a.gate ? a.gate + (a.gate_images ? (int64_t)image * a.C : 0) : nullptr;
    int turn = 0;
    grid_dependency_wait();
    float wg[kKeep ? E : 1], wp[kKeep ? E : 1], bp[kKeep ? E : 1], wn[kKeep ? E : 1], bn[kKeep ? E : 1];
    if constexpr (kKeep) {
        load_channels<TPR, V, VPT>(wg, gate, 1.f, a.nvec, lane);
        load_channels<TPR, V, VPT>(wp, a.post_w, 1.f, a.nvec, lane);
        load_channels<TPR, V, VPT>(bp, a.post_b, 0.f, a.nvec, lane);
        load_channels<TPR, V, VPT>(wn, a.pre_w, 1.f, a.nvec, lane);
        load_channels<TPR, V, VPT>(bn, a.pre_b, 0.f, a.nvec, lane);
    }
    uint4 xr[VPT], hr[VPT];
    load_row<T, TPR, VPT>(xr, a.x, row0 + begin + grp, a, lane, begin + grp < end);
    load_row<T, TPR, VPT>(hr, a.h, row0 + begin + grp, a, lane, begin + grp < end);
    for (int r = begin; r < end; r += RPC) {
        const int64_t row = row0 + r + grp;
        const bool in = r + grp < end;
        float s[E], p[E];
        unpack_row<T, VPT>(xr, s);
        unpack_row<T, VPT>(hr, p);
        const bool more = r + RPC + grp < end;
        load_row<T, TPR, VPT>(xr, a.x, row + RPC, a, lane, more);
        load_row<T, TPR, VPT>(hr, a.h, row + RPC, a, lane, more);
        if (a.h) {
            if (a.post_w) {
                normalise<TPR, V, VPT>(p, a, lane, red, turn);
                if constexpr (kKeep) {
#pragma unroll
                    for (int i = 0; i < E; ++i) p[i] = fmaf(p[i], wp[i], bp[i]);
                } else {
                    float w[E];
                    load_channels<TPR, V, VPT>(w, a.post_w, 1.f, a.nvec, lane);
#pragma unroll
                    for (int i = 0; i < E; ++i) p[i] *= w[i];
                    if (a.post_b) {
                        load_channels<TPR, V, VPT>(w, a.post_b, 0.f, a.nvec, lane);
#pragma unroll
                        for (int i = 0; i < E; ++i) p[i] += w[i];
                    }
                }
            }
            if (gate) {
                if constexpr (kKeep) {
#pragma unroll
                    for (int i = 0; i < E; ++i) p[i] *= wg[i];
                } else {
                    float w[E];
                    load_channels<TPR, V, VPT>(w, gate, 1.f, a.nvec, lane);
#pragma unroll
                    for (int i = 0; i < E; ++i) p[i] *= w[i];
                }
            }
        }
#pragma unroll
        for (int i = 0; i < E; ++i) s[i] = fmaf(a.alpha, s[i], p[i]);
        if (a.s && in) store_row<T, TPR, VPT>(a.s, row, a, lane, s);
        if (a.pre_w) {
            normalise<TPR, V, VPT>(s, a, lane, red, turn);
            if constexpr (kKeep) {
#pragma unroll
                for (int i = 0; i < E; ++i) s[i] = fmaf(s[i], wn[i], bn[i]);
            } else {
                float w[E];
                load_channels<TPR, V, VPT>(w, a.pre_w, 1.f, a.nvec, lane);
#pragma unroll
                for (int i = 0; i < E; ++i) s[i] *= w[i];
                if (a.pre_b) {
                    load_channels<TPR, V, VPT>(w, a.pre_b, 0.f, a.nvec, lane);
#pragma unroll
                    for (int i = 0; i < E; ++i) s[i] += w[i];
                }
            }
            if (in) store_row<T, TPR, VPT>(a.y, row, a, lane, s);
        }
    }
}

// part [units][5][C]: each CTA's column sums dw_post, db_post, dw_pre, db_pre, dgate
template <typename T, int TPR, int VPT>
__global__ void __launch_bounds__(block_threads(TPR)) norm_residual_backward_kernel(const NormArgs a)
{
    constexpr int V = Vec16<T>::N, E = V * VPT, RPC = block_threads(TPR) / TPR, THREADS = block_threads(TPR);
    __shared__ float red[128];
    extern __shared__ float4 smem4[];
    const int lane = threadIdx.x % TPR, grp = threadIdx.x / TPR;
    const int image = blockIdx.x / a.chunks, chunk = blockIdx.x - image * a.chunks;
    const int64_t row0 = (int64_t)image * a.rows;
    const int begin = chunk * a.per, end = min(a.rows, begin + a.per);
    const float *gate = a.gate ? a.gate + (a.gate_images ? (int64_t)image * a.C : 0) : nullptr;
    int turn = 0;
    grid_dependency_wait();
    float sum[5][E];
#pragma unroll
    for (int k = 0; k < 5; ++k)
#pragma unroll
        for (int i = 0; i < E; ++i) sum[k][i] = 0.f;
    uint4 xr[VPT], hr[VPT], yr[VPT], sr[VPT];
    auto load_all = [&](int64_t row, bool in) {
        load_row<T, TPR, VPT>(xr, a.x, row, a, lane, in);
        load_row<T, TPR, VPT>(hr, a.h, row, a, lane, in);
        load_row<T, TPR, VPT>(yr, a.dy, row, a, lane, in);
        load_row<T, TPR, VPT>(sr, a.ds, row, a, lane, in);
    };
    load_all(row0 + begin + grp, begin + grp < end);
    for (int r = begin; r < end; r += RPC) {
        const int64_t row = row0 + r + grp;
        const bool in = r + grp < end;
        float s[E], hn[E], u[E], dS[E], w[E];
        unpack_row<T, VPT>(xr, s);
        unpack_row<T, VPT>(hr, hn);
        unpack_row<T, VPT>(yr, u);
        unpack_row<T, VPT>(sr, dS);
        load_all(row + RPC, r + RPC + grp < end);
        // the forward pass again: hn = norm(h) (or h), s = alpha x + gate p
        float rh = 1.f;
        if (a.h && a.post_w) rh = normalise<TPR, V, VPT>(hn, a, lane, red, turn);
        auto branch = [&](float (&p)[E]) {  // p = hn w_post + b_post
            if (a.post_w) {
                load_channels<TPR, V, VPT>(w, a.post_w, 0.f, a.nvec, lane);
#pragma unroll
                for (int i = 0; i < E; ++i) p[i] = hn[i] * w[i];
                if (a.post_b) {
                    load_channels<TPR, V, VPT>(w, a.post_b, 0.f, a.nvec, lane);
#pragma unroll
                    for (int i = 0; i < E; ++i) p[i] += w[i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < E; ++i) p[i] = hn[i];
            }
        };
        float p[E];
        branch(p);
        if (gate) load_channels<TPR, V, VPT>(w, gate, 0.f, a.nvec, lane);
#pragma unroll
        for (int i = 0; i < E; ++i) s[i] = fmaf(a.alpha, s[i], gate ? w[i] * p[i] : p[i]);
        if (a.pre_w) {
            const float rs = normalise<TPR, V, VPT>(s, a, lane, red, turn);
            if (in) {
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    sum[2][i] = fmaf(u[i], s[i], sum[2][i]);
                    sum[3][i] += u[i];
                }
            }
            load_channels<TPR, V, VPT>(w, a.pre_w, 0.f, a.nvec, lane);
#pragma unroll
            for (int i = 0; i < E; ++i) u[i] *= w[i];
            norm_back<TPR, E>(u, s, rs, a, red, turn);
#pragma unroll
            for (int i = 0; i < E; ++i) dS[i] += u[i];
        }
        float dx[E];
#pragma unroll
        for (int i = 0; i < E; ++i) dx[i] = a.alpha * dS[i];
        if (in) store_row<T, TPR, VPT>(a.dx, row, a, lane, dx);
        if (a.h) {
            if (gate) {
                load_channels<TPR, V, VPT>(w, gate, 0.f, a.nvec, lane);
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    if (in) sum[4][i] = fmaf(dS[i], p[i], sum[4][i]);
                    dS[i] *= w[i];
                }
            }
            if (a.post_w) {
                if (in) {
#pragma unroll
                    for (int i = 0; i < E; ++i) {
                        sum[0][i] = fmaf(dS[i], hn[i], sum[0][i]);
                        sum[1][i] += dS[i];
                    }
                }
                load_channels<TPR, V, VPT>(w, a.post_w, 0.f, a.nvec, lane);
#pragma unroll
                for (int i = 0; i < E; ++i) dS[i] *= w[i];
                norm_back<TPR, E>(dS, hn, rh, a, red, turn);
            }
            if (in) store_row<T, TPR, VPT>(a.dh, row, a, lane, dS);
        }
    }
    // the CTA's sums: row groups meet in shared memory, a few groups' worth of columns at a time
    float *buf = reinterpret_cast<float *>(smem4);
    float *part = a.part + (int64_t)blockIdx.x * 5 * a.C;
#pragma unroll
    for (int k = 0; k < 5; ++k) {
        if (RPC > 1) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < E; ++i) buf[i * THREADS + threadIdx.x] = sum[k][i];
            __syncthreads();
        }
        if (grp == 0) {
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const int vec = lane + (i / V) * TPR;
                float total = sum[k][i];
                if (RPC > 1)
#pragma unroll 4
                    for (int o = 1; o < RPC; ++o) total += buf[i * THREADS + o * TPR + lane];
                if (vec < a.nvec) part[(int64_t)k * a.C + vec * V + i % V] = total;
            }
        }
    }
}

// Adds the units' column sums, 32 channels and 8 runs of units to a CTA. blockIdx.y: the four weight
// arrays, then the gate (one for each image where it has one).
__global__ void __launch_bounds__(256) norm_column_sums_kernel(const NormArgs a)
{
    __shared__ double sums[8][32];
    const int c = blockIdx.x * 32 + threadIdx.x % 32, run = threadIdx.x / 32;
    const int y = blockIdx.y;
    float *dst = y == 0 ? a.dpost_w : y == 1 ? a.dpost_b : y == 2 ? a.dpre_w : y == 3 ? a.dpre_b : a.dgate;
    grid_dependency_wait();
    if (!dst) return;
    int u0 = 0, u1 = a.units;
    if (y >= 4 && a.gate_images) {
        u0 = (y - 4) * a.chunks;
        u1 = u0 + a.chunks;
        dst += (int64_t)(y - 4) * a.C;
    }
    const float *src = a.part + (int64_t)(y < 4 ? y : 4) * a.C;
    double sum = 0.;
    if (c < a.C)
        for (int u = u0 + run; u < u1; u += 8) sum += (double)__ldcg(src + (int64_t)u * 5 * a.C + c);
    sums[run][threadIdx.x % 32] = sum;
    __syncthreads();
    if (run == 0 && c < a.C) {
        for (int i = 1; i < 8; ++i) sum += sums[i][threadIdx.x];
        dst[c] = (float)sum;
    }
}

bool norm_supports(int C, bool bf16) { return C % (bf16 ? 8 : 4) == 0 && C <= 8192; }

namespace {

// Threads a row and vectors a thread: whole warps' worth of short rows, at most two vectors a thread
// (four in fp32, whose vectors hold half as many channels).
void row_shape(int nvec, int &tpr, int &vpt)
{
    tpr = 4;
    while (tpr < nvec && tpr < 512) tpr *= 2;
    vpt = (nvec + tpr - 1) / tpr;
    if (vpt == 3) vpt = 4;
}

// CTAs: whole rounds of the GPU, each a run of whole row groups of one image (of the whole batch where
// no image has a gate of its own).
void split_rows(NormArgs &a, int threads, int tpr, int ctas)
{
    const int rpc = threads / tpr;
    long long chunks = (ctas + a.images - 1) / a.images;
    const long long most = (a.rows + rpc - 1) / rpc;
    if (chunks > most) chunks = most;
    if (chunks < 1) chunks = 1;
    a.per = (int)((a.rows + chunks - 1) / chunks);
    a.per = (a.per + rpc - 1) / rpc * rpc;
    a.chunks = (a.rows + a.per - 1) / a.per;
    a.units = a.chunks * a.images;
}

template <typename T, int TPR, int VPT> cudaError_t launch_norm(const NormArgs &a, bool backward, cudaStream_t stream)
{
    constexpr int threads = block_threads(TPR);
    if (!backward) return launch_pdl(norm_residual_kernel<T, TPR, VPT>, dim3(a.units), dim3(threads), 0, stream, a);
    const size_t smem = threads > TPR ? sizeof(float) * Vec16<T>::N * VPT * threads : 0;
    cudaError_t e = launch_pdl(norm_residual_backward_kernel<T, TPR, VPT>, dim3(a.units), dim3(threads), smem, stream, a);
    if (e != cudaSuccess) return e;
    return launch_pdl(norm_column_sums_kernel, dim3((a.C + 31) / 32, 4 + (a.gate_images ? a.images : 1)), dim3(256), 0,
                      stream, a);
}

template <typename T> cudaError_t launch_norm_t(const NormArgs &a, int tpr, int vpt, bool backward, cudaStream_t stream)
{
    switch (tpr) {
    case 4: return launch_norm<T, 4, 1>(a, backward, stream);
    case 8: return launch_norm<T, 8, 1>(a, backward, stream);
    case 16: return launch_norm<T, 16, 1>(a, backward, stream);
    case 32: return launch_norm<T, 32, 1>(a, backward, stream);
    case 64: return launch_norm<T, 64, 1>(a, backward, stream);
    case 128: return launch_norm<T, 128, 1>(a, backward, stream);
    case 256: return launch_norm<T, 256, 1>(a, backward, stream);
    default: break;
    }
    if (vpt == 1) return launch_norm<T, 512, 1>(a, backward, stream);
    if (vpt == 2) return launch_norm<T, 512, 2>(a, backward, stream);
    if constexpr (Vec16<T>::N == 4) return launch_norm<T, 512, 4>(a, backward, stream);
    return cudaErrorInvalidConfiguration;
}

}  // namespace

void norm_plan(NormArgs &a, bool backward, int num_sms)
{
    int tpr, vpt;
    row_shape(a.nvec, tpr, vpt);
    const int threads = block_threads(tpr);
    split_rows(a, threads, tpr, num_sms * (backward ? (threads > 256 ? 1 : 2) : 2048 / threads));
}

cudaError_t launch_norm_residual(const NormArgs &a, bool bf16, bool backward, cudaStream_t stream)
{
    int tpr, vpt;
    row_shape(a.nvec, tpr, vpt);
    return bf16 ? launch_norm_t<__nv_bfloat16>(a, tpr, vpt, backward, stream)
                : launch_norm_t<float>(a, tpr, vpt, backward, stream);
}

}  // namespace bra
