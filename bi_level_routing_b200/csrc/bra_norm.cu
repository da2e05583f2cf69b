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
// TPR threads hold one row in registers, VPT 16-byte vectors each; the next rows' vectors land in shared
// memory while the current one is worked on. Means are taken before the squares about them (two sums, no
// cancellation), all in fp32. The weights and the gate are the same for every row of an image, so four
// column sums give all their gradients: A = sum dS h^, S = sum dS, sum dy s^ and sum dy, with
// dgate = w_post A + b_post S, dw_post = sum over images of gate A, db_post = of gate S (S and sum dy only
// where there is a bias). They stay in each thread's registers over the rows of its CTA; the CTAs' sums go to
// a workspace and are added in a fixed order, so the result is the same bits on every run.
//
// The arrays' bytes are the floor (6.56 TB/s copied). Device times, inputs not in L2: 200704 rows of 64 channels
// forward 20.0 us (15.7 at that rate; issue slots are 69 % full), 50176 rows of 128 backward 29.2 us (11.7),
// 8192 rows of 4096 backward 97 us (61.3: each row waits for four sums of its threads), forward 46 us (RMS; 40.9).
#include "bra_device.cuh"
#include "bra_diff.cuh"
#include "bra_launch.h"

namespace bra {

namespace {

constexpr int block_threads(int tpr) { return tpr > 256 ? tpr : 256; }
// CTAs an SM: the kernels' launch bounds, what the grid is planned for, and what their shared memory must let in. Of 256
// threads three in the forward pass (200704 rows of 64 channels: two 21.3 us, three 20.0, four 20.9), two where a
// thread has more than 8 elements, whose channel arrays are in shared memory (8192 rows of 4096, RMS: 45 us; three, with
// one array there and the others from L1, 54), and in the backward pass; of 512 one.
constexpr int sm_ctas(int threads, int elements, bool backward) { return threads > 256 ? 1 : backward || elements > 8 ? 2 : 3; }
constexpr bool sm_holds(int ctas, size_t smem) { return ctas * (smem + 1024) <= 228 * 1024; }  // 1 KB a CTA is the system's

// Row groups in the rings. Forward, 200704 rows of 64 channels: 2 23.8 us, 3 20.0, 4 20.0. Backward, 50176 rows of 128
// channels: 2 32.8 us, 3 29.2, 4 30.1; rows of two vectors a thread hold two CTAs on an SM only with 2 (8192
// rows of 4096: 3 121.8 us, 2 99.4).
constexpr int kForwardStages = 3;
template <int VPT> constexpr int kBackwardStages = VPT == 1 ? 3 : 2;

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
    if constexpr (TPR > 32) {
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

// Element-wise steps on pairs (the packed fp32 instructions halve what is issued).
__device__ __forceinline__ float2 pair(const float *f) { return make_float2(f[0], f[1]); }
__device__ __forceinline__ void put(float *f, float2 v)
{
    f[0] = v.x;
    f[1] = v.y;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
template <int E> __device__ __forceinline__ void times(float (&z)[E], float r)
{
#pragma unroll
    for (int i = 0; i < E; i += 2) put(z + i, __fmul2_rn(pair(z + i), both(r)));
}
template <int E> __device__ __forceinline__ void times(float (&z)[E], const float (&w)[E])
{
#pragma unroll
    for (int i = 0; i < E; i += 2) put(z + i, __fmul2_rn(pair(z + i), pair(w + i)));
}
template <int E> __device__ __forceinline__ void plus(float (&z)[E], const float (&w)[E])
{
#pragma unroll
    for (int i = 0; i < E; i += 2) put(z + i, __fadd2_rn(pair(z + i), pair(w + i)));
}
// z += x y
template <int E> __device__ __forceinline__ void plus_product(float (&z)[E], const float (&x)[E], const float (&y)[E])
{
#pragma unroll
    for (int i = 0; i < E; i += 2) put(z + i, __ffma2_rn(pair(x + i), pair(y + i), pair(z + i)));
}

// z becomes norm(z); returns 1 / sqrt(...). Elements past the row are 0 and stay so.
template <int TPR, int V, int VPT>
__device__ __forceinline__ float normalise(float (&z)[V * VPT], const NormArgs &a, int lane, float *red, int &turn)
{
    constexpr int E = V * VPT;
    float sum[1];
    if (a.layer && TPR <= 32 && a.nvec == TPR * VPT) {
        // Every thread holds E elements: mean and squares about it, merged pair by pair (two sets of n elements with means x and
        // y: the mean (x + y) / 2, the squares' sum grown by (x - y)^2 n / 2), one chain of exchanges instead of two.
        float2 t = make_float2(0.f, 0.f), q = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < E; i += 2) t = __fadd2_rn(t, pair(z + i));
        float mean = (t.x + t.y) * (1.f / E);
#pragma unroll
        for (int i = 0; i < E; i += 2) {
            const float2 d = __fadd2_rn(pair(z + i), both(-mean));
            q = __ffma2_rn(d, d, q);
        }
        float squares = q.x + q.y;
#pragma unroll
        for (int o = 1; o < TPR; o *= 2) {
            const float other = __shfl_xor_sync(0xffffffffu, mean, o);
            const float more = __shfl_xor_sync(0xffffffffu, squares, o);
            const float d = other - mean;
            mean = 0.5f * (mean + other);
            squares = fmaf(d * d, 0.5f * E * o, squares + more);
        }
        const float r = rsqrtf(fmaf(squares, a.inv_c, a.eps));
#pragma unroll
        for (int i = 0; i < E; i += 2) put(z + i, __fmul2_rn(__fadd2_rn(pair(z + i), both(-mean)), both(r)));
        return r;
    }
    if (a.layer) {
        float2 t = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < E; i += 2) t = __fadd2_rn(t, pair(z + i));
        sum[0] = t.x + t.y;
        row_sums<TPR, 1>(sum, red, turn);
        const float mean = sum[0] * a.inv_c;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (lane + i * TPR < a.nvec) {
#pragma unroll
                for (int j = 0; j < V; j += 2) put(z + i * V + j, __fadd2_rn(pair(z + i * V + j), both(-mean)));
            }
    }
    float2 t = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < E; i += 2) t = __ffma2_rn(pair(z + i), pair(z + i), t);
    sum[0] = t.x + t.y;
    row_sums<TPR, 1>(sum, red, turn);
    const float r = rsqrtf(fmaf(sum[0], a.inv_c, a.eps));  // within 2 steps of fp32
    times(z, r);
    return r;
}

// u becomes r (u - mean(u) - z^ mean(u z^)), the mean(u) term for LayerNorm only. Elements past the row are 0 in z^ and u on
// the way in, not on the way out: the caller multiplies them by channel factors of 0 before it sums again.
template <int TPR, int E>
__device__ __forceinline__ void norm_back(float (&u)[E], const float (&z)[E], float r, const NormArgs &a, float *red, int &turn)
{
    float2 t0 = make_float2(0.f, 0.f), t1 = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < E; i += 2) {
        t0 = __fadd2_rn(t0, pair(u + i));
        t1 = __ffma2_rn(pair(u + i), pair(z + i), t1);
    }
    float sum[2] = {t0.x + t0.y, t1.x + t1.y};
    row_sums<TPR, 2>(sum, red, turn);
    const float2 m0 = both(a.layer ? -r * sum[0] * a.inv_c : 0.f), m1 = both(-r * sum[1] * a.inv_c), rr = both(r);
#pragma unroll
    for (int i = 0; i < E; i += 2) put(u + i, __ffma2_rn(pair(z + i), m1, __ffma2_rn(pair(u + i), rr, m0)));
}

// E values of a channel array at this thread's vectors: `def` where the array is absent, 0 past the row (what is multiplied
// by them must stay 0 there: the next sums run over it).
template <int TPR, int V, int VPT>
__device__ __forceinline__ void load_channels(float (&w)[V * VPT], const float *p, float def, int nvec, int lane)
{
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < V / 4; ++j) {
            const bool in = lane + i * TPR < nvec;
            float4 f = in ? make_float4(def, def, def, def) : make_float4(0.f, 0.f, 0.f, 0.f);
            if (p && in) f = __ldg(reinterpret_cast<const float4 *>(p) + (lane + i * TPR) * (V / 4) + j);
            w[i * V + 4 * j] = f.x;
            w[i * V + 4 * j + 1] = f.y;
            w[i * V + 4 * j + 2] = f.z;
            w[i * V + 4 * j + 3] = f.w;
        }
}

// The branch's factor gate * w_post and offset gate * b_post: p = h^ gw + gb.
template <int TPR, int V, int VPT>
__device__ __forceinline__ void load_branch(float (&w)[V * VPT], const float *gate, const float *p, float def, int nvec, int lane)
{
    load_channels<TPR, V, VPT>(w, p, def, nvec, lane);
    if (gate) {
        float g[V * VPT];
        load_channels<TPR, V, VPT>(g, gate, 1.f, nvec, lane);
#pragma unroll
        for (int i = 0; i < V * VPT; ++i) w[i] *= g[i];
    }
}

// A ring of STAGES row groups of ARRAYS input arrays in shared memory. Every thread copies the vectors it will itself read
// (cp.async, no barrier), STAGES - 1 groups ahead: registers could hold one group, too few bytes in flight for
// the memory's latency.
template <typename T, int TPR, int VPT, int ARRAYS, int WANTED> struct RowRing {
    static constexpr int kThreads = block_threads(TPR);
    static constexpr int kGroup = ARRAYS * VPT * kThreads * 16;
    // the widest fp32 rows leave room for fewer: one, if need be, which is copied when it is wanted
    static constexpr int kRoom = 226 * 1024 - (VPT > 1 ? 2 * Vec16<T>::N * VPT * kThreads * 4 : 0);
    static constexpr int kFit = kRoom / kGroup, STAGES = kFit < 1 ? 1 : kFit < WANTED ? kFit : WANTED;
    static constexpr int kAhead = STAGES - 1;
    static constexpr size_t kBytes = (size_t)STAGES * kGroup;
    static_assert(kBytes <= kRoom, "one row group must fit");
    const T *src[ARRAYS];  // this thread's first vector of the next row to fetch
    bool have[ARRAYS];
    uint8_t *mine;
    int64_t step;  // elements from one of the thread's rows to its next
    int vectors;   // of the thread: those of i < VPT with lane + i TPR inside the row
    int put = 0, get = 0;

    __device__ __forceinline__ RowRing(const NormArgs &a, uint8_t *smem, int lane)
        : mine(smem + threadIdx.x * 16), step((int64_t)(kThreads / TPR) * a.C), vectors((a.nvec - lane + TPR - 1) / TPR) {}
    __device__ __forceinline__ void array(int k, const NormArgs &a, const void *base, int64_t row, int lane)
    {
        have[k] = base != nullptr;
        src[k] = static_cast<const T *>(have[k] ? base : a.x) + row * a.C + (int64_t)lane * Vec16<T>::N;
    }
    __device__ __forceinline__ uint8_t *slot(int stage, int array, int i) const
    {
        return mine + (size_t)((stage * ARRAYS + array) * VPT + i) * (kThreads * 16);
    }
    // copies the thread's next row (zeros, reading nothing, where it is not one or an array is absent) and commits
    __device__ __forceinline__ void fetch(bool in)
    {
#pragma unroll
        for (int k = 0; k < ARRAYS; ++k) {
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                cp_async16_or_zero(smem_u32(slot(put, k, i)), src[k] + i * TPR * Vec16<T>::N, in && have[k] && i < vectors);
            src[k] += step;
        }
        cp_async_commit();
        put = put + 1 == STAGES ? 0 : put + 1;
    }
    __device__ __forceinline__ void wait() { cp_async_wait_but<(STAGES > 1 ? STAGES - 2 : 0)>(); }
    __device__ __forceinline__ void read(int k, float (&f)[Vec16<T>::N * VPT]) const
    {
#pragma unroll
        for (int i = 0; i < VPT; ++i) Vec16<T>::unpack(*reinterpret_cast<const uint4 *>(slot(get, k, i)), f + i * Vec16<T>::N);
    }
    __device__ __forceinline__ void next() { get = get + 1 == STAGES ? 0 : get + 1; }
};

// Two channel arrays in shared memory, each thread's own elements where it reads them itself (no barrier): what wide rows
// cannot keep in registers.
template <int TPR, int E> struct Stash {
    static constexpr int kThreads = block_threads(TPR);
    static constexpr size_t kBytes = (size_t)2 * E * kThreads * sizeof(float);
    float4 *mine;
    __device__ __forceinline__ explicit Stash(float *smem) : mine(reinterpret_cast<float4 *>(smem) + threadIdx.x) {}
    __device__ __forceinline__ void write(int k, const float (&w)[E])
    {
#pragma unroll
        for (int i = 0; i < E / 4; ++i)
            mine[(k * (E / 4) + i) * kThreads] = make_float4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
    __device__ __forceinline__ void read(int k, float (&w)[E]) const
    {
#pragma unroll
        for (int i = 0; i < E / 4; ++i) {
            const float4 f = mine[(k * (E / 4) + i) * kThreads];
            w[4 * i] = f.x;
            w[4 * i + 1] = f.y;
            w[4 * i + 2] = f.z;
            w[4 * i + 3] = f.w;
        }
    }
};

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

}  // namespace

template <typename T, int TPR, int VPT>
__global__ void __launch_bounds__(block_threads(TPR), sm_ctas(block_threads(TPR), Vec16<T>::N * VPT, false)) norm_residual_kernel(const NormArgs a)
{
    constexpr int V = Vec16<T>::N, E = V * VPT, RPC = block_threads(TPR) / TPR;
    // the channel arrays stay in registers (4 E of them); else the factors come from shared memory, the biases from L1
    constexpr bool kKeep = E <= 8;
    extern __shared__ float4 smem4[];
    using Ring = RowRing<T, TPR, VPT, 2, kForwardStages>;
    float *red = reinterpret_cast<float *>(smem4) + Ring::kBytes / 4;
    const int lane = threadIdx.x % TPR, grp = threadIdx.x / TPR;
    const int image = blockIdx.x / a.chunks, chunk = blockIdx.x - image * a.chunks;
    const int64_t row0 = (int64_t)image * a.rows;
    const int begin = chunk * a.per, end = min(a.rows, begin + a.per);
    const float *gate = a.gate ? a.gate + (a.gate_images ? (int64_t)image * a.C : 0) : nullptr;
    int turn = 0;
    grid_dependency_wait();
    Ring ring(a, reinterpret_cast<uint8_t *>(smem4), lane);
    ring.array(0, a, a.x, row0 + begin + grp, lane);
    ring.array(1, a, a.h, row0 + begin + grp, lane);
#pragma unroll
    for (int k = 0; k < Ring::kAhead; ++k) ring.fetch(begin + k * RPC + grp < end);
    Stash<TPR, E> stash(red + 128);
    float w[kKeep ? 4 : 1][E];  // gate w_post, gate b_post, w_pre, b_pre
    if constexpr (kKeep) {
        if (a.h) {
            load_branch<TPR, V, VPT>(w[0], gate, a.post_w, 1.f, a.nvec, lane);
            load_branch<TPR, V, VPT>(w[1], a.post_b ? gate : nullptr, a.post_b, 0.f, a.nvec, lane);
        }
        if (a.pre_w) {
            load_channels<TPR, V, VPT>(w[2], a.pre_w, 1.f, a.nvec, lane);
            load_channels<TPR, V, VPT>(w[3], a.pre_b, 0.f, a.nvec, lane);
        }
    } else {
        if (a.h) {
            load_branch<TPR, V, VPT>(w[0], gate, a.post_w, 1.f, a.nvec, lane);
            stash.write(0, w[0]);
        }
        if (a.pre_w) {
            load_channels<TPR, V, VPT>(w[0], a.pre_w, 1.f, a.nvec, lane);
            stash.write(1, w[0]);
        }
    }
    for (int r = begin; r < end; r += RPC) {
        const int64_t row = row0 + r + grp;
        const bool in = r + grp < end;
        float s[E];
        if (Ring::kAhead == 0) ring.fetch(in);
        ring.wait();
        ring.read(0, s);
#pragma unroll
        for (int i = 0; i < E; ++i) s[i] *= a.alpha;
        if (a.h) {
            float p[E];
            ring.read(1, p);
            if (a.post_w) normalise<TPR, V, VPT>(p, a, lane, red, turn);
            if constexpr (kKeep) {
#pragma unroll
                for (int i = 0; i < E; ++i) s[i] += fmaf(p[i], w[0][i], w[1][i]);
            } else {
                stash.read(0, w[0]);
#pragma unroll
                for (int i = 0; i < E; ++i) s[i] = fmaf(p[i], w[0][i], s[i]);
                if (a.post_b) {
                    load_branch<TPR, V, VPT>(w[0], gate, a.post_b, 0.f, a.nvec, lane);
#pragma unroll
                    for (int i = 0; i < E; ++i) s[i] += w[0][i];
                }
            }
        }
        ring.next();
        if (Ring::kAhead > 0) ring.fetch(r + Ring::kAhead * RPC + grp < end);
        if (a.s && in) store_row<T, TPR, VPT>(a.s, row, a, lane, s);
        if (a.pre_w) {
            normalise<TPR, V, VPT>(s, a, lane, red, turn);
            if constexpr (kKeep) {
                times(s, w[2]);
                plus(s, w[3]);
            } else {
                stash.read(1, w[0]);
                times(s, w[0]);
                if (a.pre_b) {
                    load_channels<TPR, V, VPT>(w[0], a.pre_b, 0.f, a.nvec, lane);
                    plus(s, w[0]);
                }
            }
            if (in) store_row<T, TPR, VPT>(a.y, row, a, lane, s);
        }
    }
    cp_async_wait_all();
}

// part [units][4][C]: each CTA's column sums A, sum dy s^, S, sum dy (the last two where BIAS)
template <typename T, int TPR, int VPT, bool BIAS>
__global__ void __launch_bounds__(block_threads(TPR), sm_ctas(block_threads(TPR), Vec16<T>::N * VPT, true)) norm_residual_backward_kernel(const NormArgs a)
{
    constexpr int V = Vec16<T>::N, E = V * VPT, RPC = block_threads(TPR) / TPR, THREADS = block_threads(TPR);
    constexpr int SUMS = BIAS ? 4 : 2;
    constexpr bool kKeep = VPT == 1;  // the channel arrays stay in registers
    extern __shared__ float4 smem4[];
    using Ring = RowRing<T, TPR, VPT, 4, kBackwardStages<VPT>>;
    float *red = reinterpret_cast<float *>(smem4) + Ring::kBytes / 4;
    const int lane = threadIdx.x % TPR, grp = threadIdx.x / TPR;
    const int image = blockIdx.x / a.chunks, chunk = blockIdx.x - image * a.chunks;
    const int64_t row0 = (int64_t)image * a.rows;
    const int begin = chunk * a.per, end = min(a.rows, begin + a.per);
    const float *gate = a.gate ? a.gate + (a.gate_images ? (int64_t)image * a.C : 0) : nullptr;
    int turn = 0;
    grid_dependency_wait();
    Ring ring(a, reinterpret_cast<uint8_t *>(smem4), lane);
    ring.array(0, a, a.x, row0 + begin + grp, lane);
    ring.array(1, a, a.h, row0 + begin + grp, lane);
    ring.array(2, a, a.dy, row0 + begin + grp, lane);
    ring.array(3, a, a.ds, row0 + begin + grp, lane);
#pragma unroll
    for (int k = 0; k < Ring::kAhead; ++k) ring.fetch(begin + k * RPC + grp < end);
    float sum[SUMS][E];
#pragma unroll
    for (int k = 0; k < SUMS; ++k)
#pragma unroll
        for (int i = 0; i < E; ++i) sum[k][i] = 0.f;
    Stash<TPR, E> stash(red + 128);
    float gw[E], gb[kKeep && BIAS ? E : 1], wn[kKeep ? E : 1];
    if constexpr (kKeep) {
        if (a.h) {
            load_branch<TPR, V, VPT>(gw, gate, a.post_w, 1.f, a.nvec, lane);
            if constexpr (BIAS) load_branch<TPR, V, VPT>(gb, a.post_b ? gate : nullptr, a.post_b, 0.f, a.nvec, lane);
        }
        if (a.pre_w) load_channels<TPR, V, VPT>(wn, a.pre_w, 0.f, a.nvec, lane);
    } else {
        if (a.h) {
            load_branch<TPR, V, VPT>(gw, gate, a.post_w, 1.f, a.nvec, lane);
            stash.write(0, gw);
        }
        if (a.pre_w) {
            load_channels<TPR, V, VPT>(gw, a.pre_w, 0.f, a.nvec, lane);
            stash.write(1, gw);
        }
    }
    for (int r = begin; r < end; r += RPC) {
        const int64_t row = row0 + r + grp;
        const bool in = r + grp < end;
        if (Ring::kAhead == 0) ring.fetch(in);
        ring.wait();
        // the forward pass again: hn = norm(h) (or h), s = alpha x + hn gw + gb
        float s[E], hn[E];
        ring.read(0, s);
        times(s, a.alpha);
        float rh = 1.f;
        if (a.h) {
            ring.read(1, hn);
            if (a.post_w) rh = normalise<TPR, V, VPT>(hn, a, lane, red, turn);
            if (!kKeep) stash.read(0, gw);
            plus_product(s, hn, gw);
            if constexpr (BIAS && kKeep) {
                plus(s, gb);
            } else if (BIAS && a.post_b) {
                load_branch<TPR, V, VPT>(gw, gate, a.post_b, 0.f, a.nvec, lane);
                plus(s, gw);
            }
        }
        float dS[E];
        if (a.pre_w) {
            const float rs = normalise<TPR, V, VPT>(s, a, lane, red, turn);
            ring.read(2, dS);
            if (in) {
                plus_product(sum[1], dS, s);
                if (BIAS) plus(sum[SUMS - 1], dS);
            }
            if constexpr (kKeep) {
                times(dS, wn);
            } else {
                stash.read(1, gw);
                times(dS, gw);
            }
            norm_back<TPR, E>(dS, s, rs, a, red, turn);
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) dS[i] = 0.f;
        }
        ring.read(3, s);
        ring.next();
        if (Ring::kAhead > 0) ring.fetch(r + Ring::kAhead * RPC + grp < end);
        plus(dS, s);
#pragma unroll
        for (int i = 0; i < E; ++i) s[i] = dS[i];
        times(s, a.alpha);
        if (in) store_row<T, TPR, VPT>(a.dx, row, a, lane, s);
        if (a.h) {
            if (in) {
                plus_product(sum[0], dS, hn);
                if (BIAS) plus(sum[SUMS - 2], dS);
            }
            if (!kKeep) stash.read(0, gw);
            times(dS, gw);
            if (a.post_w) norm_back<TPR, E>(dS, hn, rh, a, red, turn);
            if (in) store_row<T, TPR, VPT>(a.dh, row, a, lane, dS);
        }
    }
    cp_async_wait_all();
    // the CTA's sums: row groups meet in shared memory
    float *buf = reinterpret_cast<float *>(smem4);
    float *part = a.part + (int64_t)blockIdx.x * 4 * a.C;
#pragma unroll
    for (int k = 0; k < SUMS; ++k) {
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

// The gradients of the weights and the gate from the units' column sums, 32 channels and kRuns runs of images (or, with one
// gate, of units) to a CTA. Few CTAs of many threads: what it takes is the latency of its loads.
constexpr int kRuns = 32;

__global__ void __launch_bounds__(32 * kRuns) norm_column_sums_kernel(const NormArgs a)
{
    __shared__ double sums[4][kRuns][32];
    const int lane = threadIdx.x % 32, c = blockIdx.x * 32 + lane, run = threadIdx.x / 32;
    const bool in = c < a.C;
    const bool bias = a.post_b || a.pre_b;
    double total[4] = {0., 0., 0., 0.};  // sum gate A, sum dy s^, sum gate S, sum dy
    grid_dependency_wait();
    if (in) {
        const float w = a.post_w ? __ldg(a.post_w + c) : 1.f, b = a.post_b ? __ldg(a.post_b + c) : 0.f;
        if (a.gate_images) {
            for (int image = run; image < a.images; image += kRuns) {
                const float g = __ldg(a.gate + (int64_t)image * a.C + c);
                double x[4] = {0., 0., 0., 0.};
#pragma unroll 4
                for (int u = image * a.chunks; u < (image + 1) * a.chunks; ++u)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (k < 2 || bias) x[k] += (double)__ldcg(a.part + ((int64_t)u * 4 + k) * a.C + c);
                a.dgate[(int64_t)image * a.C + c] = (float)(w * x[0] + b * x[2]);
                total[0] += g * x[0];
                total[1] += x[1];
                total[2] += g * x[2];
                total[3] += x[3];
            }
        } else {
#pragma unroll 4
            for (int u = run; u < a.units; u += kRuns)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (k < 2 || bias) total[k] += (double)__ldcg(a.part + ((int64_t)u * 4 + k) * a.C + c);
        }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) sums[k][run][lane] = total[k];
    __syncthreads();
    if (run < 4) {  // warp k adds array k
        double all = 0.;
#pragma unroll 8
        for (int i = 0; i < kRuns; ++i) all += sums[run][i][lane];
        sums[run][0][lane] = all;
    }
    __syncthreads();
    if (run == 0 && in) {
#pragma unroll
        for (int k = 0; k < 4; ++k) total[k] = sums[k][0][lane];
        if (!a.gate_images) {
            const float g = a.gate ? __ldg(a.gate + c) : 1.f;
            const float w = a.post_w ? __ldg(a.post_w + c) : 1.f, b = a.post_b ? __ldg(a.post_b + c) : 0.f;
            if (a.dgate) a.dgate[c] = (float)(w * total[0] + b * total[2]);
            total[0] *= g;
            total[2] *= g;
        }
        if (a.dpost_w) a.dpost_w[c] = (float)total[0];
        if (a.dpre_w) a.dpre_w[c] = (float)total[1];
        if (a.dpost_b) a.dpost_b[c] = (float)total[2];
        if (a.dpre_b) a.dpre_b[c] = (float)total[3];
    }
}

bool norm_supports(int C, bool bf16) { return C % (bf16 ? 8 : 4) == 0 && C <= 8192; }

namespace {

// Threads a row and vectors a thread: a vector a thread up to 256 threads, then two, so that several CTAs
// share an SM and one works while another waits for its rows' sums (8192 bf16 rows of 4096 channels, backward:
// 256 threads of two vectors 100 us, 512 of one 129); 512 threads for the widest rows.
void row_shape(int nvec, int &tpr, int &vpt)
{
    tpr = 4;
    while (tpr < nvec && tpr < 256) tpr *= 2;
    if (nvec > 512) tpr = 512;
    vpt = (nvec + tpr - 1) / tpr;
    if (vpt == 3) vpt = 4;
}

// CTAs of one round of the GPU, each a run of whole row groups of one image (of the whole batch where no image has a
// gate of its own).
void split_rows(NormArgs &a, int threads, int tpr, int ctas)
{
    const int rpc = threads / tpr;
    long long chunks = ctas / a.images;
    const long long most = (a.rows + rpc - 1) / rpc;
    if (chunks > most) chunks = most;
    if (chunks < 1) chunks = 1;
    a.per = (int)((a.rows + chunks - 1) / chunks);
    a.per = (a.per + rpc - 1) / rpc * rpc;
    a.chunks = (a.rows + a.per - 1) / a.per;
    a.units = a.chunks * a.images;
}

template <auto Kernel> cudaError_t launch_with(int threads, size_t smem, const NormArgs &a, cudaStream_t stream)
{
    const cudaError_t e = grant_shared_memory<Kernel>();
    return e == cudaSuccess ? launch_pdl(Kernel, dim3(a.units), dim3(threads), smem, stream, a) : e;
}

template <typename T, int TPR, int VPT> cudaError_t launch_norm(const NormArgs &a, bool backward, cudaStream_t stream)
{
    constexpr int threads = block_threads(TPR);
    constexpr int E = Vec16<T>::N * VPT;
    constexpr size_t red = 128 * sizeof(float);
    constexpr size_t forward = RowRing<T, TPR, VPT, 2, kForwardStages>::kBytes + red + (E > 8 ? Stash<TPR, E>::kBytes : 0);
    static_assert(sm_holds(sm_ctas(threads, E, false), forward), "the planned CTAs fit an SM");
    if (!backward) return launch_with<norm_residual_kernel<T, TPR, VPT>>(threads, forward, a, stream);
    // the ring, later the row groups' column sums
    constexpr size_t ring = RowRing<T, TPR, VPT, 4, kBackwardStages<VPT>>::kBytes;
    constexpr size_t sums = threads > TPR ? sizeof(float) * Vec16<T>::N * VPT * threads : 0;
    constexpr size_t smem = (ring > sums ? ring : sums) + red + (VPT > 1 ? Stash<TPR, E>::kBytes : 0);
    static_assert(sm_holds(sm_ctas(threads, E, true), smem), "the planned CTAs fit an SM");
    cudaError_t e = a.post_b || a.pre_b
                        ? launch_with<norm_residual_backward_kernel<T, TPR, VPT, true>>(threads, smem, a, stream)
                        : launch_with<norm_residual_backward_kernel<T, TPR, VPT, false>>(threads, smem, a, stream);
    if (e != cudaSuccess) return e;
    return launch_pdl(norm_column_sums_kernel, dim3((a.C + 31) / 32), dim3(32 * kRuns), 0, stream, a);
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
    case 256: return vpt == 1 ? launch_norm<T, 256, 1>(a, backward, stream) : launch_norm<T, 256, 2>(a, backward, stream);
    default: break;
    }
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
    split_rows(a, threads, tpr, num_sms * sm_ctas(threads, a.C / a.nvec * vpt, backward));
}

cudaError_t launch_norm_residual(const NormArgs &a, bool bf16, bool backward, cudaStream_t stream)
{
    int tpr, vpt;
    row_shape(a.nvec, tpr, vpt);
    return bf16 ? launch_norm_t<__nv_bfloat16>(a, tpr, vpt, backward, stream)
                : launch_norm_t<float>(a, tpr, vpt, backward, stream);
}

}  // namespace bra
