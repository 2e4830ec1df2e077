// Norms of the heads of q and k with the rotary positions in the same pass, and their gradient.
//
// Per head of a row, r = 1 / sqrt(mean x^2 + eps), n = r x, and
//   y = a R(pos) (w n)                                 (the rotation on its columns, as in attn_rope.cu)
// With g = a R(pos)^T dy the gradient is
//   dw = sum over rows and heads of n g,   dx = r (w g - n mean(n w g)).
// Both move each element once in and once out (the gradient two in) and are bounded by memory.
//
// A group of W lanes, W a power of two, holds a whole head in registers: R items per lane, each two runs of V
// columns that the rotation pairs (item_cols). So the sums over a head are a few shuffles, the head is read once,
// and the next ones are copied to shared memory, every lane's pieces to its own places, while this one is computed. Angles (one set per token, shared by all heads) and
// weights lie in shared memory. A lane keeps its columns over all heads, so the weights' gradient is a sum in its
// registers, joined over the block at the end; a second kernel adds the blocks' sums in a fixed order. No atomics: the
// same call gives the same bytes.
//
// Measured, bf16, 40 heads of 128, 18432 rows: 59.1 us, 6390 GB/s, 0.94 of a copy's rate; the gradient
// of 16384 rows 83-85 us, 6000 GB/s, 0.89. fp32, 32 heads
// of 192, 64 interleaved columns rotated, 8192 rows: 63.3 us, 6360 GB/s, the gradient 97.2 us, 6210 GB/s; 40 heads of 128, 9216 rows: 58.7 us, 6430 GB/s, the
// gradient of 8192 rows 82-84 us. Not kept: heads loaded two or three ahead into registers (forward 75-85 us), four or eight heads of a
// token for each group of lanes with angles and weights in registers (86-93).
#include "attn.h"
#include "launch.cuh"
#include "rows.cuh"

#include <math.h>

namespace attn {
namespace {

constexpr int kNormMaxDim = 1024;
// Blocks of 256 threads that an SM holds, by the items per lane: their registers (64 to 255 per thread).
constexpr int norm_blocks(int items) { return items == 1 ? 4 : 2; }
constexpr int norm_bwd_blocks(int items) { return items == 1 ? 2 : 1; }
// Heads that a group of lanes has in shared memory or on their way there, 32 bytes of a lane for each of its items: two are on their way while one
// is computed. (18432 rows of 40 heads of 128, blocks on an SM x heads: 4 x 3 59.1 us, 4 x 4 59.4, 3 x 4 59.8, 5 x 3 61.4, 5 x 2 63.9, 6 x 3 67.2; one
// head ahead in registers, 5 blocks, 62.6.)
constexpr int kNormFwdStages = 3;
// Heads that a group of lanes of the gradient has in shared memory or on their way there, 64 bytes of a lane for each of its items: with one
// item per lane two are on their way while one is computed (16384 rows of 40 heads of 128: 83 us; one 91, three 90, four 94. fp32 heads
// of 192, three items per lane: one on its way 97.2, two 100; with two blocks on an SM 107).
template <int R>
constexpr int kNormStages = R == 1 ? 3 : 2;
constexpr int kNormItems = 8;      // heads per group of lanes, at least
constexpr int kNormAngles = 8192;  // floats for the angles of a block's tokens, at most
constexpr int kNormShared = 12288; // for them, the weights and the warps' sums (48 KB)

struct NormParams {
    const void* in[2];     // q, k
    const void* grad[2];   // gradients of the outputs (backward)
    void* out[2];          // outputs, or gradients of the inputs
    long long in_stride[2], grad_stride[2], out_stride[2];  // elements between rows
    const float* weight[2];
    float* partial;        // [blocks, 2, d] sums for the weights' gradient, or nullptr
    const int* positions;
    const double* inv_freq;
    RopeCols cols;
    int T, heads[2];
    int tokens;            // tokens per block
    int items, lanes;      // work items per head, lanes per head
    float eps, amplitude, inv_d;
};

// The heads of a block's tokens, taken in turn by the groups of lanes; the indices advance without divisions.
struct HeadWalk {
    int t, h, dt, dh, heads;
    __device__ __forceinline__ HeadWalk(int first, int step, int heads_) : heads(heads_) {
        t = first / heads;
        h = first - t * heads;
        dt = step / heads;
        dh = step - dt * heads;
    }
    __device__ __forceinline__ void next() {
        h += dh;
        t += dt;
        if (h >= heads) h -= heads, ++t;
    }
};

// Sum over a group of W lanes (0: `lanes`).
template <int W>
__device__ __forceinline__ float group_sum(float x, int lanes) {
    if constexpr (W > 0) {
#pragma unroll
        for (int o = W / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    } else {
        for (int o = lanes >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    }
    return x;
}

// Place of element i of a row of n in shared memory: lane j reads elements 8 j .. 8 j + 7 of bf16 rows by two 16-byte loads, which lie in two
// halves of the row, so that neighbouring lanes read neighbouring 16 bytes. (Side by side they conflict in every other bank: forward
// 72 us, the gradient 107 us.) V = 4 and 1 read in order.
template <int V>
__device__ __forceinline__ int spread(int i, int n) {
    return V == 8 ? (i & 4 ? n / 2 : 0) + (i >> 3) * 4 + (i & 3) : i;
}
// Elements V j .. V j + V - 1 of such a row.
template <int V>
__device__ __forceinline__ void load_spread(const float* row, int j, int n, float (&x)[V]) {
    if constexpr (V == 8) {
        float lo[4], hi[4];
        load_angles<4>(row + 4 * j, lo);
        load_angles<4>(row + n / 2 + 4 * j, hi);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = lo[e], x[4 + e] = hi[e];
    } else {
        load_angles<V>(row + V * j, x);
    }
}

// Weights of both tensors into shared memory, ones where there are none: in the order of the columns, rows of d spread.
template <int V>
__device__ __forceinline__ void stage_weights(const NormParams& p, float* w) {
    for (int i = threadIdx.x; i < 2 * p.cols.d; i += blockDim.x) {
        const int k = i >= p.cols.d, c = i - k * p.cols.d;
        const float* from = p.weight[k];
        w[k * p.cols.d + spread<V>(c, p.cols.d)] = from ? from[c] : 1.0f;
    }
}

// cos and sin (times the amplitude) of the block's tokens into cs[token][rot / 2] and sn[token][rot / 2], the rows spread unless the pairs
// are interleaved (whose lanes read four neighbouring ones at a time). Every thread of the block calls it.
template <int V>
__device__ __forceinline__ void stage_angles(const NormParams& p, long long t0, int tokens, bool transpose, float* cs, float* sn) {
    const int half = p.cols.rot / 2;
    if (half == 0) return;
    const int nt = blockDim.x, groups = max(1, nt / half), grp = threadIdx.x / half;
    if (grp >= groups) return;
    for (int i = groups > 1 ? (int)threadIdx.x % half : (int)threadIdx.x; i < half; i += groups > 1 ? half : nt) {
        const double f = p.inv_freq[i];
        const unsigned long long frac = turn_fraction(f);
        const float amp = isfinite(f) ? p.amplitude : __int_as_float(0x7fffffff);  // no angle: NaN
        const int at = p.cols.interleaved ? i : spread<V>(i, half);
        for (int t = groups > 1 ? grp : 0; t < tokens; t += groups) {
            float c, s;
            position_angle(frac, p.positions[t0 + t], c, s);
            cs[t * half + at] = c * amp;
            sn[t * half + at] = (transpose ? -s : s) * amp;
        }
    }
}

// w (r x): r x is at most sqrt(d), where w r may leave fp32 though the result does not.
template <int V>
__device__ __forceinline__ void times(float (&x)[V], const float (&w)[V], float r) {
#pragma unroll
    for (int e = 0; e < V; e += 2) {
        fmul2(x[e], x[e + 1], x[e], x[e + 1], r, r);
        fmul2(x[e], x[e + 1], x[e], x[e + 1], w[e], w[e + 1]);
    }
}

// Pairs (u, w) turned: u c - w s, u s + w c.
template <int V>
__device__ __forceinline__ void turn(float (&u)[V], float (&w)[V], const float (&c)[V], const float (&s)[V]) {
#pragma unroll
    for (int e = 0; e < V; e += 2) {
        float a0, a1, b0, b1;
        fmul2(a0, a1, u[e], u[e + 1], c[e], c[e + 1]);
        fmul2(b0, b1, u[e], u[e + 1], s[e], s[e + 1]);
        ffma2(u[e], u[e + 1], w[e], w[e + 1], -s[e], -s[e + 1], a0, a1);
        ffma2(w[e], w[e + 1], w[e], w[e + 1], c[e], c[e + 1], b0, b1);
    }
}

// Sum of the products over both runs of an item, added to that of two interleaved halves.
template <int V>
__device__ __forceinline__ void add_products(float (&sum)[2], const float (&x)[V], const float (&y)[V]) {
#pragma unroll
    for (int e = 0; e < V; e += 2) ffma2(sum[0], sum[1], x[e], x[e + 1], y[e], y[e + 1], sum[0], sum[1]);
}

// Rotate the pairs of item j.
template <int V>
__device__ __forceinline__ void turn_item(float (&xa)[V], float (&xb)[V], const RopeCols& cols, int j, const float* cs, const float* sn) {
    if (V == 8 && !cols.interleaved) {
        float c[V], s[V];
        load_spread<V>(cs, j, cols.rot / 2, c);
        load_spread<V>(sn, j, cols.rot / 2, s);
        turn<V>(xa, xb, c, s);
    } else {
        rotate_item<V>(xa, xb, cols, j, cs, sn);
    }
}

// Forward for heads that fit into the registers of a group of lanes.
// W > 0: a head is exactly W lanes of R items; 0: p.lanes, the last ones may be idle.
template <typename E, int V, int R, int W>
__global__ void __launch_bounds__(256, norm_blocks(R)) norm_rope_kernel(const __grid_constant__ NormParams p) {
    grid_dependents_launch();
    grid_dependency_wait();
    extern __shared__ __align__(16) float shared[];
    constexpr int kStages = kNormFwdStages;
    const int half = p.cols.rot / 2, d = p.cols.d, H = p.heads[0] + p.heads[1];
    uint4* ring = reinterpret_cast<uint4*>(shared) + threadIdx.x;  // [stage][item][a, b][thread]
    auto piece = [&](int stage, int r, int x) { return ring + ((stage * R + r) * 2 + x) * (int)blockDim.x; };
    float* w = shared + kStages * R * 8 * (int)blockDim.x;
    float* cs = w + 2 * d;
    float* sn = cs + p.tokens * half;
    const long long t0 = (long long)blockIdx.x * p.tokens;
    const int tokens = (int)min((long long)p.tokens, p.T - t0);
    const int lanes = W > 0 ? W : p.lanes, lane = threadIdx.x & (lanes - 1), shift = 31 - __clz(lanes);
    const int groups = blockDim.x >> shift;
    HeadWalk at(threadIdx.x >> shift, groups, H), ahead = at;
    int a[R], b[R];
    bool turned[R], some[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        some[r] = W > 0 || lane + r * lanes < p.items;
        turned[r] = item_cols<V>(p.cols, some[r] ? lane + r * lanes : 0, a[r], b[r]);
    }
    auto load = [&](int stage) {
        if (ahead.t < tokens) {
            const bool k = ahead.h >= p.heads[0];
            const E* src = static_cast<const E*>(k ? p.in[1] : p.in[0]) + (t0 + ahead.t) * (k ? p.in_stride[1] : p.in_stride[0]) +
                           (long long)(k ? ahead.h - p.heads[0] : ahead.h) * d;
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (some[r]) cp_async16(smem_u32(piece(stage, r, 0)), src + a[r], 16), cp_async16(smem_u32(piece(stage, r, 1)), src + b[r], 16);
        }
        cp_async_commit();
        ahead.next();
    };
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) load(s);
    stage_angles<V>(p, t0, tokens, false, cs, sn);
    stage_weights<V>(p, w);
    __syncthreads();
    // (a warp goes on while its first group has a head: the groups of a warp take part in its shuffles)
    const int all = tokens * H;
    int stage = 0;
    for (int i = (threadIdx.x & ~31) >> shift; i < all; i += groups) {
        const bool mine = at.t < tokens;
        const int t = at.t, h = at.h;
        const bool k = h >= p.heads[0];
        cp_async_wait<kStages - 2>();
        float xa[R][V], xb[R][V], ss[2] = {0.0f, 0.0f};  // (a group without a head sums what it finds, for itself)
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (!some[r]) continue;
            unpack<E, V>(*piece(stage, r, 0), xa[r]), unpack<E, V>(*piece(stage, r, 1), xb[r]);
            add_products<V>(ss, xa[r], xa[r]);
            add_products<V>(ss, xb[r], xb[r]);
        }
        at.next();
        load(stage == 0 ? kStages - 1 : stage - 1);
        stage = stage + 1 == kStages ? 0 : stage + 1;
        const float scale = rsqrtf(fmaf(group_sum<W>(ss[0] + ss[1], lanes), p.inv_d, p.eps));
        if (!mine) continue;
        E* dst = static_cast<E*>(k ? p.out[1] : p.out[0]) + (t0 + t) * (k ? p.out_stride[1] : p.out_stride[0]) +
                 (long long)(k ? h - p.heads[0] : h) * d;
        const float* wh = w + (k ? d : 0);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (!some[r]) continue;
            float wa[V], wb[V];
            load_spread<V>(wh, a[r] / V, d, wa);
            load_spread<V>(wh, b[r] / V, d, wb);
            times<V>(xa[r], wa, scale);
            times<V>(xb[r], wb, scale);
            if (turned[r]) turn_item<V>(xa[r], xb[r], p.cols, lane + r * lanes, cs + t * half, sn + t * half);
            store_row<V>(dst + a[r], xa[r]);
            store_row<V>(dst + b[r], xb[r]);
        }
    }
}

// Forward element by element, a warp per head: any alignment and width. The head is read twice (the second time
// from the L1).
template <typename E>
__global__ void __launch_bounds__(256) norm_rope_any_kernel(const __grid_constant__ NormParams p) {
    grid_dependents_launch();
    grid_dependency_wait();
    extern __shared__ __align__(16) float shared[];
    const int half = p.cols.rot / 2, d = p.cols.d, H = p.heads[0] + p.heads[1];
    float* w = shared;
    float* cs = shared + 2 * d;
    float* sn = cs + p.tokens * half;
    const long long t0 = (long long)blockIdx.x * p.tokens;
    const int tokens = (int)min((long long)p.tokens, p.T - t0), lane = threadIdx.x & 31;
    stage_angles<1>(p, t0, tokens, false, cs, sn);
    stage_weights<1>(p, w);
    __syncthreads();
    for (HeadWalk at(threadIdx.x >> 5, blockDim.x >> 5, H); at.t < tokens; at.next()) {
        const int k = at.h >= p.heads[0];
        const int h = k ? at.h - p.heads[0] : at.h;
        const E* src = static_cast<const E*>(p.in[k]) + (t0 + at.t) * p.in_stride[k] + (long long)h * d;
        E* dst = static_cast<E*>(p.out[k]) + (t0 + at.t) * p.out_stride[k] + (long long)h * d;
        float ss = 0.0f;
        for (int i = lane; i < d; i += 32) ss = fmaf((float)src[i], (float)src[i], ss);
        const float scale = rsqrtf(fmaf(group_sum<32>(ss, 32), p.inv_d, p.eps));
        __syncwarp();
        for (int j = lane; j < p.items; j += 32) {
            int a, b;
            const bool turned = item_cols<1>(p.cols, j, a, b);
            float xa[1] = {(float)src[a] * scale * w[k * d + a]}, xb[1] = {(float)src[b] * scale * w[k * d + b]};
            if (turned) rotate_item<1>(xa, xb, p.cols, j, cs + at.t * half, sn + at.t * half);
            store_row<1>(dst + a, xa);
            store_row<1>(dst + b, xb);
        }
    }
}

// The block's sums of the warps' rows [warps][d] to its place.
__device__ __forceinline__ void block_sums(const NormParams& p, const float* rows, int k) {
    __syncthreads();
    const int d = p.cols.d, warps = blockDim.x >> 5;
    float* to = p.partial + ((long long)blockIdx.x * 2 + k) * d;
    for (int c = threadIdx.x; c < d; c += blockDim.x) {
        float s = 0.0f;
        for (int v = 0; v < warps; ++v) s += rows[v * d + c];
        to[c] = s;
    }
    __syncthreads();
}

template <typename E, int V, int R, int W>
__global__ void __launch_bounds__(256, norm_bwd_blocks(R)) norm_rope_bwd_kernel(const __grid_constant__ NormParams p) {
    grid_dependents_launch();
    grid_dependency_wait();
    extern __shared__ __align__(16) float shared[];
    constexpr int kStages = kNormStages<R>;
    const int half = p.cols.rot / 2, d = p.cols.d;
    uint4* ring = reinterpret_cast<uint4*>(shared) + threadIdx.x;  // [stage][item][x a, x b, dy a, dy b][thread]
    auto piece = [&](int stage, int r, int x) { return ring + ((stage * R + r) * 4 + x) * (int)blockDim.x; };
    float* w = shared + kStages * R * 16 * (int)blockDim.x;
    float* rows = w + 2 * d;  // [warps][d]
    float* cs = rows + (blockDim.x >> 5) * d;
    float* sn = cs + p.tokens * half;
    const long long t0 = (long long)blockIdx.x * p.tokens;
    const int tokens = (int)min((long long)p.tokens, p.T - t0);
    const int lanes = W > 0 ? W : p.lanes, lane = threadIdx.x & (lanes - 1), shift = 31 - __clz(lanes);
    const int groups = blockDim.x >> shift;
    int a[R], b[R];
    bool turned[R], some[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        some[r] = W > 0 || lane + r * lanes < p.items;
        turned[r] = item_cols<V>(p.cols, some[r] ? lane + r * lanes : 0, a[r], b[r]);
    }
    HeadWalk ahead(threadIdx.x >> shift, groups, p.heads[0]);
    auto load = [&](int k, int stage) {
        if (ahead.t < tokens) {
            const E* src = static_cast<const E*>(p.in[k]) + (t0 + ahead.t) * p.in_stride[k] + (long long)ahead.h * d;
            const E* grad = static_cast<const E*>(p.grad[k]) + (t0 + ahead.t) * p.grad_stride[k] + (long long)ahead.h * d;
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (some[r]) {
                    cp_async16(smem_u32(piece(stage, r, 0)), src + a[r], 16), cp_async16(smem_u32(piece(stage, r, 1)), src + b[r], 16);
                    cp_async16(smem_u32(piece(stage, r, 2)), grad + a[r], 16), cp_async16(smem_u32(piece(stage, r, 3)), grad + b[r], 16);
                }
        }
        cp_async_commit();
        ahead.next();
    };
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) load(0, s);
    stage_angles<V>(p, t0, tokens, true, cs, sn);
    stage_weights<V>(p, w);
    __syncthreads();
    for (int k = 0; k < 2; ++k) {  // the heads of q, then of k
        if (p.heads[k] == 0) continue;
        HeadWalk at(threadIdx.x >> shift, groups, p.heads[k]);
        float wa_sum[R][V] = {}, wb_sum[R][V] = {};
        const int all = tokens * p.heads[k];
        int stage = 0;
        for (int i = (threadIdx.x & ~31) >> shift; i < all; i += groups) {
            const bool mine = at.t < tokens;
            const int t = at.t, h = at.h;
            cp_async_wait<kStages - 2>();
            float xa[R][V], xb[R][V], ya[R][V], yb[R][V], ss[2] = {0.0f, 0.0f}, dot[2] = {0.0f, 0.0f};
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (!some[r]) continue;
                unpack<E, V>(*piece(stage, r, 0), xa[r]), unpack<E, V>(*piece(stage, r, 1), xb[r]);
                unpack<E, V>(*piece(stage, r, 2), ya[r]), unpack<E, V>(*piece(stage, r, 3), yb[r]);
            }
            at.next();
            load(k, stage == 0 ? kStages - 1 : stage - 1);  // (where the head before this one was)
            stage = stage + 1 == kStages ? 0 : stage + 1;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (!some[r]) continue;
                if (turned[r] && mine) turn_item<V>(ya[r], yb[r], p.cols, lane + r * lanes, cs + t * half, sn + t * half);
                float wa[V], wb[V];
                load_spread<V>(w + k * d, a[r] / V, d, wa);
                load_spread<V>(w + k * d, b[r] / V, d, wb);
                add_products<V>(ss, xa[r], xa[r]);
                add_products<V>(ss, xb[r], xb[r]);
#pragma unroll
                for (int e = 0; e < V; e += 2) {
                    fmul2(wa[e], wa[e + 1], wa[e], wa[e + 1], ya[r][e], ya[r][e + 1]);
                    fmul2(wb[e], wb[e + 1], wb[e], wb[e + 1], yb[r][e], yb[r][e + 1]);
                }
                add_products<V>(dot, xa[r], wa);
                add_products<V>(dot, xb[r], wb);
            }
            const float scale = rsqrtf(fmaf(group_sum<W>(ss[0] + ss[1], lanes), p.inv_d, p.eps));
            const float along = group_sum<W>(dot[0] + dot[1], lanes) * p.inv_d * scale;  // mean(n w g)
            if (!mine) continue;
            E* dst = static_cast<E*>(p.out[k]) + (t0 + t) * p.out_stride[k] + (long long)h * d;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (!some[r]) continue;
                float wa[V], wb[V];
                load_spread<V>(w + k * d, a[r] / V, d, wa);
                load_spread<V>(w + k * d, b[r] / V, d, wb);
                // dx = r (w g - n along); dw += n g. (In this order: r^2 along, and r^2 alone for heads below 10^-19, leave fp32 before dx does.)
                auto finish = [&](float(&x)[V], const float(&y)[V], const float(&wt)[V], float(&w_sum)[V]) {
#pragma unroll
                    for (int e = 0; e < V; e += 2) {
                        float n0, n1, g0, g1;
                        fmul2(n0, n1, x[e], x[e + 1], scale, scale);
                        ffma2(w_sum[e], w_sum[e + 1], n0, n1, y[e], y[e + 1], w_sum[e], w_sum[e + 1]);
                        fmul2(g0, g1, y[e], y[e + 1], wt[e], wt[e + 1]);
                        ffma2(g0, g1, n0, n1, -along, -along, g0, g1);
                        fmul2(x[e], x[e + 1], g0, g1, scale, scale);
                    }
                };
                finish(xa[r], ya[r], wa, wa_sum[r]);
                finish(xb[r], yb[r], wb, wb_sum[r]);
                store_row<V>(dst + a[r], xa[r]);
                store_row<V>(dst + b[r], xb[r]);
            }
        }
        cp_async_wait<0>();
        if (k == 0 && p.heads[1] > 0) {
            ahead = HeadWalk(threadIdx.x >> shift, groups, p.heads[1]);
#pragma unroll
            for (int s = 0; s < kStages - 1; ++s) load(1, s);
        }
        if (!p.partial) continue;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int e = 0; e < V; ++e)
                for (int o = lanes; o < 32; o <<= 1) {
                    wa_sum[r][e] += __shfl_xor_sync(0xffffffffu, wa_sum[r][e], o);
                    wb_sum[r][e] += __shfl_xor_sync(0xffffffffu, wb_sum[r][e], o);
                }
        float* row = rows + (threadIdx.x >> 5) * d;
        if ((threadIdx.x & 31) < lanes) {
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (some[r])
#pragma unroll
                    for (int e = 0; e < V; ++e) row[a[r] + e] = wa_sum[r][e], row[b[r] + e] = wb_sum[r][e];
        }
        block_sums(p, rows, k);
    }
}

// The gradient element by element, a warp per head; its sums for the weights in the warp's row of shared memory.
template <typename E>
__global__ void __launch_bounds__(256) norm_rope_bwd_any_kernel(const __grid_constant__ NormParams p) {
    grid_dependents_launch();
    grid_dependency_wait();
    extern __shared__ __align__(16) float shared[];
    const int half = p.cols.rot / 2, d = p.cols.d, lane = threadIdx.x & 31;
    float* w = shared;
    float* rows = w + 2 * d;
    float* cs = rows + (blockDim.x >> 5) * d;
    float* sn = cs + p.tokens * half;
    const long long t0 = (long long)blockIdx.x * p.tokens;
    const int tokens = (int)min((long long)p.tokens, p.T - t0);
    float* row = rows + (threadIdx.x >> 5) * d;
    stage_angles<1>(p, t0, tokens, true, cs, sn);
    stage_weights<1>(p, w);
    __syncthreads();
    for (int k = 0; k < 2; ++k) {
        if (p.heads[k] == 0) continue;
        for (int i = lane; i < d; i += 32) row[i] = 0.0f;
        __syncwarp();
        for (HeadWalk at(threadIdx.x >> 5, blockDim.x >> 5, p.heads[k]); at.t < tokens; at.next()) {
            const E* src = static_cast<const E*>(p.in[k]) + (t0 + at.t) * p.in_stride[k] + (long long)at.h * d;
            const E* grad = static_cast<const E*>(p.grad[k]) + (t0 + at.t) * p.grad_stride[k] + (long long)at.h * d;
            E* dst = static_cast<E*>(p.out[k]) + (t0 + at.t) * p.out_stride[k] + (long long)at.h * d;
            float ss = 0.0f, dot = 0.0f;
            auto item = [&](int j, int& a, int& b, float (&xa)[1], float (&xb)[1], float (&ya)[1], float (&yb)[1]) {
                const bool turned = item_cols<1>(p.cols, j, a, b);
                xa[0] = (float)src[a], xb[0] = (float)src[b];
                ya[0] = (float)grad[a], yb[0] = (float)grad[b];
                if (turned) rotate_item<1>(ya, yb, p.cols, j, cs + at.t * half, sn + at.t * half);
            };
            int a, b;
            float xa[1], xb[1], ya[1], yb[1];
            for (int j = lane; j < p.items; j += 32) {
                item(j, a, b, xa, xb, ya, yb);
                ss = fmaf(xa[0], xa[0], fmaf(xb[0], xb[0], ss));
                dot = fmaf(xa[0], w[k * d + a] * ya[0], fmaf(xb[0], w[k * d + b] * yb[0], dot));
            }
            const float scale = rsqrtf(fmaf(group_sum<32>(ss, 32), p.inv_d, p.eps));
            const float along = group_sum<32>(dot, 32) * p.inv_d * scale;
            for (int j = lane; j < p.items; j += 32) {
                item(j, a, b, xa, xb, ya, yb);
                xa[0] *= scale, xb[0] *= scale;
                row[a] = fmaf(xa[0], ya[0], row[a]);
                row[b] = fmaf(xb[0], yb[0], row[b]);
                xa[0] = scale * (w[k * d + a] * ya[0] - xa[0] * along);
                xb[0] = scale * (w[k * d + b] * yb[0] - xb[0] * along);
                store_row<1>(dst + a, xa);
                store_row<1>(dst + b, xb);
            }
        }
        if (p.partial) block_sums(p, rows, k);
    }
}

// dw = the blocks' sums added up: 32 columns per block, 32 threads each, joined in a fixed order.
__global__ void __launch_bounds__(1024) norm_weight_sums_kernel(const float* partial, int blocks, int d, float* dq_weight, float* dk_weight) {
    grid_dependency_wait();
    __shared__ float part[32][33];
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5, c = blockIdx.x * 32 + x;
    float s = 0.0f;
    if (c < 2 * d)
        for (int i = y; i < blocks; i += 32) s += partial[(long long)i * 2 * d + c];
    part[y][x] = s;
    __syncthreads();
    s = part[x][y];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const int col = blockIdx.x * 32 + y;
    if (x != 0 || col >= 2 * d) return;
    float* to = col < d ? dq_weight : dk_weight;
    if (to) to[col < d ? col : col - d] = s;
}

// Lanes per head and items per lane with the fewest idle places, of equal ones the fewest items per lane.
void head_shape(int items, int& lanes, int& each) {
    int best = 1 << 30;
    for (int r = 1; r <= 4; ++r) {
        int n = 1;
        while (n < 32 && n * r < items) n *= 2;
        if (n * r >= items && n * r - items < best) best = n * r - items, lanes = n, each = r;
    }
}

template <typename E, int V, int R, int W>
cudaError_t launch_wide(const NormParams& p, bool back, unsigned blocks, unsigned threads, size_t smem, cudaStream_t s) {
    if (back) {
        static std::atomic<bool> attr_set[kMaxAttrDevices];
        const size_t ring = (size_t)kNormStages<R> * R * 64 * threads;
        const cudaError_t e = ensure_smem_attr(norm_rope_bwd_kernel<E, V, R, W>, (int)(kNormStages<R> * R * 64 * 256 + kNormShared * 4), attr_set);
        if (e != cudaSuccess) return e;
        return launch_kernel(norm_rope_bwd_kernel<E, V, R, W>, dim3(blocks), threads, ring + smem, s, {true}, p);
    }
    static std::atomic<bool> attr_set[kMaxAttrDevices];
    const size_t ring = (size_t)kNormFwdStages * R * 32 * threads;
    const cudaError_t e = ensure_smem_attr(norm_rope_kernel<E, V, R, W>, (int)(kNormFwdStages * R * 32 * 256 + kNormShared * 4), attr_set);
    if (e != cudaSuccess) return e;
    return launch_kernel(norm_rope_kernel<E, V, R, W>, dim3(blocks), threads, ring + smem, s, {true}, p);
}

// The common widths have kernels of their own (64, 128 and 256, and with V = 8 items of bf16 192: three items on 4 lanes).
template <typename E, int V>
cudaError_t launch_shape(const NormParams& p, int each, bool back, unsigned blocks, unsigned threads, size_t smem, cudaStream_t s) {
    const bool full = p.items == p.lanes * each;
    if (each == 1 && full && p.lanes == 4) return launch_wide<E, V, 1, 4>(p, back, blocks, threads, smem, s);
    if (each == 1 && full && p.lanes == 8) return launch_wide<E, V, 1, 8>(p, back, blocks, threads, smem, s);
    if (each == 1 && full && p.lanes == 16) return launch_wide<E, V, 1, 16>(p, back, blocks, threads, smem, s);
    if (each == 1) return launch_wide<E, V, 1, 0>(p, back, blocks, threads, smem, s);
    if (each == 2) return launch_wide<E, V, 2, 0>(p, back, blocks, threads, smem, s);
    if (each == 3 && full && p.lanes == (V == 8 ? 4 : 8)) return launch_wide<E, V, 3, V == 8 ? 4 : 8>(p, back, blocks, threads, smem, s);
    if (each == 3) return launch_wide<E, V, 3, 0>(p, back, blocks, threads, smem, s);
    return launch_wide<E, V, 4, 0>(p, back, blocks, threads, smem, s);
}

template <typename E>
cudaError_t launch_norm(NormParams p, bool wide, bool back, int num_sms, float* dq_weight, float* dk_weight, cudaStream_t s) {
    constexpr int V = 16 / sizeof(E);
    int each = 1;
    p.lanes = 32;
    p.items = p.cols.d / 2;
    if (wide) {
        p.items = p.cols.d / (2 * V);
        head_shape(p.items, p.lanes, each);
    }
    const unsigned threads = back && p.cols.d > 512 ? 128 : 256;
    // tokens per block: some heads for every group of lanes, no more than the angles have room for
    const int H = p.heads[0] + p.heads[1], groups = threads / p.lanes;
    long long n = back ? kNormAngles : ((long long)kNormItems * groups + H - 1) / H;
    const int rows = 2 + (back ? (int)threads / 32 : 0);  // of shared memory, besides the angles
    const int angles = kNormShared - rows * p.cols.d < kNormAngles ? kNormShared - rows * p.cols.d : kNormAngles;
    if (p.cols.rot > 0 && n > angles / p.cols.rot) n = angles / p.cols.rot;
    p.tokens = p.T > 0 ? whole_waves(p.T, n, (long long)num_sms * (back ? norm_bwd_blocks(each) : norm_blocks(each))) : 1;
    const long long blocks = ((long long)p.T + p.tokens - 1) / p.tokens;
    const size_t smem = ((size_t)p.tokens * p.cols.rot + (size_t)rows * p.cols.d) * sizeof(float);
    const bool sums = back && (dq_weight || dk_weight);
    cudaError_t e = cudaSuccess;
    void* ws = nullptr;
    if (sums && blocks > 0) {
        cudaMemPool_t pool = nullptr;
        if (current_device_pool(&pool) != ATTN_OK) return cudaErrorUnknown;
        if ((e = cudaMallocFromPoolAsync(&ws, (size_t)blocks * 2 * p.cols.d * sizeof(float), pool, s)) != cudaSuccess) {
            cudaGetLastError();  // (out of memory is no error of the next call)
            return e;
        }
        p.partial = static_cast<float*>(ws);
    }
    if (blocks > 0) {
        if (!wide)
            e = back ? launch_kernel(norm_rope_bwd_any_kernel<E>, dim3((unsigned)blocks), threads, smem, s, {true}, p)
                     : launch_kernel(norm_rope_any_kernel<E>, dim3((unsigned)blocks), threads, smem, s, {true}, p);
        else
            e = launch_shape<E, V>(p, each, back, (unsigned)blocks, threads, smem, s);
    }
    if (e == cudaSuccess && sums) {
        LaunchMode mode;
        mode.dependent = blocks > 0;
        e = launch_kernel(norm_weight_sums_kernel, dim3((unsigned)(2 * p.cols.d + 31) / 32), 1024, 0, s, mode, (const float*)p.partial, (int)blocks,
                          p.cols.d, dq_weight, dk_weight);
    }
    if (ws) cudaFreeAsync(ws, s);
    return e;
}

bool multiple(const void* p, long long bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

// Checks that both directions share; fills p. Tensors of the call: in, (gradients in,) out.
attn_status_t check(NormParams& p, const void* const (&in)[2], const void* const (&grad)[2], void* const (&out)[2],
                    const long long (&in_stride)[2], const long long (&grad_stride)[2], const long long (&out_stride)[2], bool back,
                    const float* q_weight, const float* k_weight, float eps, const int* positions, const double* inv_freq, int T, int Hq,
                    int Hk, int d, int rot_begin, int rot_dim, int elem_type, int interleaved, float amplitude, bool& wide) {
    const int heads[2] = {Hq, Hk};
    for (int i = 0; i < 2; ++i)
        if ((i == 0 || Hk > 0) && (!in[i] || !out[i] || (back && !grad[i]))) return ATTN_ERR_NULL_PTR;
    if (rot_dim != 0 && (!positions || !inv_freq)) return ATTN_ERR_NULL_PTR;
    if (elem_type != ATTN_TYPE_BF16 && elem_type != ATTN_TYPE_F32) return ATTN_ERR_BAD_ARG;
    if ((interleaved != 0 && interleaved != 1) || !isfinite(amplitude) || !isfinite(eps) || eps < 0) return ATTN_ERR_BAD_ARG;
    if (T < 0 || Hq <= 0 || Hk < 0 || Hq > 65535 || Hk > 65535 || d <= 0 || d > kNormMaxDim || d % 2 != 0 || rot_dim < 0 ||
        rot_dim % 2 != 0 || rot_begin < 0 || rot_begin > d - rot_dim)
        return ATTN_ERR_BAD_SHAPE;
    const int size = elem_type == ATTN_TYPE_BF16 ? 2 : 4, V = 16 / size;
    wide = d % (2 * V) == 0 && rot_begin % (2 * V) == 0 && rot_dim % (2 * V) == 0;
    for (int i = 0; i < 2; ++i) {
        p.in[i] = in[i], p.grad[i] = grad[i], p.out[i] = out[i];
        p.in_stride[i] = in_stride[i], p.grad_stride[i] = grad_stride[i], p.out_stride[i] = out_stride[i];
        p.heads[i] = heads[i];
        if (heads[i] == 0) continue;
        // rows of an output may not overlap; those of an input may (stride 0 repeats one row)
        if (in_stride[i] < 0 || (back && grad_stride[i] < 0) || out_stride[i] < (long long)heads[i] * d) return ATTN_ERR_BAD_SHAPE;
        if ((in[i] == out[i] && in_stride[i] != out_stride[i]) || (back && grad[i] == out[i] && grad_stride[i] != out_stride[i]))
            return ATTN_ERR_BAD_SHAPE;
        if (!multiple(in[i], size) || !multiple(out[i], size) || (back && !multiple(grad[i], size))) return ATTN_ERR_ALIGN;
        wide = wide && multiple(in[i], 16) && multiple(out[i], 16) && in_stride[i] % V == 0 && out_stride[i] % V == 0;
        if (back) wide = wide && multiple(grad[i], 16) && grad_stride[i] % V == 0;
    }
    if ((q_weight && !multiple(q_weight, 4)) || (k_weight && !multiple(k_weight, 4))) return ATTN_ERR_ALIGN;
    if (rot_dim != 0 && (!multiple(positions, 4) || !multiple(inv_freq, 8))) return ATTN_ERR_ALIGN;
    p.weight[0] = q_weight, p.weight[1] = k_weight;
    p.partial = nullptr;
    p.positions = positions;
    p.inv_freq = inv_freq;
    p.cols = RopeCols{d, rot_dim ? rot_begin : 0, rot_dim, interleaved};
    p.T = T;
    p.eps = eps;
    p.amplitude = amplitude;
    p.inv_d = 1.0f / (float)d;
    return ATTN_OK;
}

}  // namespace
}  // namespace attn

extern "C" attn_status_t attn_qk_norm_rope(const void* q, const void* k, void* q_out, void* k_out, const float* q_weight,
                                           const float* k_weight, float eps, const int* positions, const double* inv_freq, int T, int Hq,
                                           int Hk, int d, int rot_begin, int rot_dim, long long q_stride, long long k_stride,
                                           long long q_out_stride, long long k_out_stride, int elem_type, int interleaved,
                                           float amplitude, void* stream) {
    using namespace attn;
    NormParams p;
    bool wide = false;
    attn_status_t st = check(p, {q, k}, {nullptr, nullptr}, {q_out, k_out}, {q_stride, k_stride}, {0, 0}, {q_out_stride, k_out_stride}, false,
                             q_weight, k_weight, eps, positions, inv_freq, T, Hq, Hk, d, rot_begin, rot_dim, elem_type, interleaved,
                             amplitude, wide);
    if (st != ATTN_OK || T == 0) return st;
    int* status = nullptr;
    int num_sms = 0;
    if ((st = current_device_info(&status, &num_sms)) != ATTN_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = elem_type == ATTN_TYPE_BF16 ? launch_norm<__nv_bfloat16>(p, wide, false, num_sms, nullptr, nullptr, s)
                                                      : launch_norm<float>(p, wide, false, num_sms, nullptr, nullptr, s);
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

extern "C" attn_status_t attn_qk_norm_rope_bwd(const void* q, const void* k, const void* dq_out, const void* dk_out, const float* q_weight,
                                               const float* k_weight, float eps, const int* positions, const double* inv_freq, void* dq,
                                               void* dk, float* dq_weight, float* dk_weight, int T, int Hq, int Hk, int d, int rot_begin,
                                               int rot_dim, long long q_stride, long long k_stride, long long dq_out_stride,
                                               long long dk_out_stride, long long dq_stride, long long dk_stride, int elem_type,
                                               int interleaved, float amplitude, void* stream) {
    using namespace attn;
    NormParams p;
    bool wide = false;
    attn_status_t st = check(p, {q, k}, {dq_out, dk_out}, {dq, dk}, {q_stride, k_stride}, {dq_out_stride, dk_out_stride},
                             {dq_stride, dk_stride}, true, q_weight, k_weight, eps, positions, inv_freq, T, Hq, Hk, d, rot_begin, rot_dim,
                             elem_type, interleaved, amplitude, wide);
    if (st != ATTN_OK) return st;
    if ((dq_weight && !multiple(dq_weight, 4)) || (dk_weight && !multiple(dk_weight, 4))) return ATTN_ERR_ALIGN;
    if (Hk == 0 && dk_weight) return ATTN_ERR_BAD_ARG;
    if (T == 0 && !dq_weight && !dk_weight) return ATTN_OK;
    int* status = nullptr;
    int num_sms = 0;
    if ((st = current_device_info(&status, &num_sms)) != ATTN_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = elem_type == ATTN_TYPE_BF16 ? launch_norm<__nv_bfloat16>(p, wide, true, num_sms, dq_weight, dk_weight, s)
                                                      : launch_norm<float>(p, wide, true, num_sms, dq_weight, dk_weight, s);
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}
