// Rotary positions: y = a R(pos f) x on the columns [rot_begin, rot_begin + rot_dim) of every head,
// the other columns copied, for the rows of q and k of one call in one launch.
//
// Pair i of a row at position pos turns by the angle pos f_i:
//   (y1, y2) = a (x1 cos - x2 sin, x1 sin + x2 cos);
// R is orthogonal, so the gradient with respect to x is the same rotation by the negative angle
// (transpose). The operator moves each element once in and once out and computes three
// multiply-adds per pair: it is bounded by memory, and the angles must not cost more than that.
// One block takes a few tokens, computes their cosines and sines once into shared memory (shared by
// all heads), and streams the heads through 16-byte loads and stores, the next item's loads ahead of
// this one's stores. Measured: 18432 rows of 40 bf16 heads of 128 in 59.5 us, 6340 GB/s, 0.93 of the
// measured copy rate (65536 rows 1.00); 8192 rows of 32 fp32 heads, 64 of 192 columns rotated, 0.95;
// 64 rows 3.6 us. (Threads that keep their head and columns over the tokens, as in the cache writes,
// need more registers and gave 65 and 74 us for the first two.)
#include "attn.h"
#include "launch.cuh"
#include "rows.cuh"

#include <math.h>

namespace attn {
namespace {

constexpr int kRopeThreads = 256;
// Blocks that an SM holds (48 registers per thread), and items per thread, at most. Measured, us, whole waves of 5
// blocks and items 2: 63.8, 3: 60.2, 4: 59.5, of 6 blocks and items 8: 61.2, 16: 63.7 (18432 rows of 40 bf16 heads of
// 128); of 5 blocks and items 2: 61.0, 4: 62.2, of 6 blocks and items 8: 63.1 (8192 rows of 32 fp32 heads).
constexpr int kRopeBlocks = 5, kRopeItems = 4;
constexpr int kRopeMaxDim = 1024;

struct RopeParams {
    const void *q, *k;
    void *q_out, *k_out;
    long long q_stride, k_stride, q_out_stride, k_out_stride;  // elements between rows
    const int* positions;
    const double* inv_freq;
    RopeCols cols;
    int T, Hq, H;        // rows, query heads, query and key heads
    int tokens;          // tokens per block
    int items;           // work items per head: d / (2 V), or the rotated ones only (in place)
    float amplitude;
    int transpose;
};

// The items of a block of tokens, this thread's ones blockDim apart. Item (t, h, j): token t of the
// block, head h of `heads`, item j of `items` per head, in that order; the indices advance without divisions.
struct ItemWalk {
    int t, h, j, dt, dh, dj, heads, items;
    __device__ __forceinline__ ItemWalk(int heads_, int items_) : heads(heads_), items(items_) {
        const int n = blockDim.x;
        j = threadIdx.x % items;
        h = threadIdx.x / items;
        t = h / heads;
        h -= t * heads;
        dj = n % items;
        dh = n / items;
        dt = dh / heads;
        dh -= dt * heads;
    }
    __device__ __forceinline__ void next() {
        j += dj;
        h += dh;
        t += dt;
        if (j >= items) j -= items, ++h;
        if (h >= heads) h -= heads, ++t;
    }
};

template <typename E, int V>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p) {
    extern __shared__ __align__(16) float angles[];
    const int half = p.cols.rot / 2;
    const long long t0 = (long long)blockIdx.x * p.tokens;
    const int tokens = (int)min((long long)p.tokens, p.T - t0);
    float* cs = angles;
    float* sn = angles + p.tokens * half;
    // An item is loaded while the one before is rotated and stored; the first before the angles are
    // computed, which it does not need.
    typedef typename RawOf<E, V>::type Raw;
    ItemWalk at(p.H, p.items);
    Raw ra, rb;
    auto load = [&]() {
        const bool k = at.h >= p.Hq;
        const E* src = static_cast<const E*>(k ? p.k : p.q) + (t0 + at.t) * (k ? p.k_stride : p.q_stride) +
                       (long long)(k ? at.h - p.Hq : at.h) * p.cols.d;
        int a, b;
        item_cols<V>(p.cols, at.j, a, b);
        ra = load_raw<E, V>(src + a);
        rb = load_raw<E, V>(src + b);
    };
    if (at.t < tokens) load();
    block_angles(p.inv_freq, p.positions + t0, tokens, half, p.amplitude, p.transpose != 0, cs, sn);
    __syncthreads();
    while (at.t < tokens) {
        const int t = at.t, j = at.j;
        const bool k = at.h >= p.Hq;
        E* dst = static_cast<E*>(k ? p.k_out : p.q_out) + (t0 + t) * (k ? p.k_out_stride : p.q_out_stride) +
                 (long long)(k ? at.h - p.Hq : at.h) * p.cols.d;
        float xa[V], xb[V];
        unpack<E, V>(ra, xa);
        unpack<E, V>(rb, xb);
        at.next();
        if (at.t < tokens) load();
        int a, b;
        if (item_cols<V>(p.cols, j, a, b))
            rotate_item<V>(xa, xb, p.cols, j, cs + t * half, sn + t * half);
        store_row<V>(dst + a, xa);
        store_row<V>(dst + b, xb);
    }
}

template <typename E, int V>
cudaError_t launch_rope(RopeParams p, bool in_place, int num_sms, cudaStream_t stream) {
    p.items = (in_place ? p.cols.rot : p.cols.d) / (2 * V);
    const int each = p.H * p.items, most = 8192 / p.cols.rot;  // (the angles of a block's tokens: 32 KB at most)
    const int n = (kRopeItems * kRopeThreads + each - 1) / each;
    p.tokens = whole_waves(p.T, n < most ? n : most, (long long)num_sms * kRopeBlocks);
    const long long blocks = ((long long)p.T + p.tokens - 1) / p.tokens;
    const size_t smem = (size_t)p.tokens * p.cols.rot * sizeof(float);
    return launch_kernel(rope_kernel<E, V>, dim3((unsigned)blocks), kRopeThreads, smem, stream, {}, p);
}

bool multiple(const void* p, long long bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

}  // namespace
}  // namespace attn

extern "C" attn_status_t attn_rope(const void* q, const void* k, void* q_out, void* k_out, const int* positions,
                                   const double* inv_freq, int T, int Hq, int Hk, int d, int rot_begin, int rot_dim,
                                   long long q_stride, long long k_stride, long long q_out_stride, long long k_out_stride,
                                   int elem_type, int interleaved, int transpose, float amplitude, void* stream) {
    using namespace attn;
    if (!q || !q_out || !positions || !inv_freq || (Hk > 0 && (!k || !k_out))) return ATTN_ERR_NULL_PTR;
    if (elem_type != ATTN_TYPE_BF16 && elem_type != ATTN_TYPE_F32) return ATTN_ERR_BAD_ARG;
    if ((interleaved != 0 && interleaved != 1) || (transpose != 0 && transpose != 1) || !isfinite(amplitude))
        return ATTN_ERR_BAD_ARG;
    if (T < 0 || Hq <= 0 || Hk < 0 || Hq > 65535 || Hk > 65535 || d <= 0 || d > kRopeMaxDim || d % 2 != 0 || rot_dim <= 0 ||
        rot_dim % 2 != 0 || rot_begin < 0 || rot_begin > d - rot_dim)
        return ATTN_ERR_BAD_SHAPE;
    const long long wq = (long long)Hq * d, wk = (long long)Hk * d;
    // rows of an output may not overlap; those of an input may (stride 0 repeats one row)
    if (q_stride < 0 || (Hk > 0 && k_stride < 0) || q_out_stride < wq || (Hk > 0 && k_out_stride < wk)) return ATTN_ERR_BAD_SHAPE;
    const int size = elem_type == ATTN_TYPE_BF16 ? 2 : 4;
    if (!multiple(q, size) || !multiple(q_out, size) || !multiple(positions, 4) || !multiple(inv_freq, 8) ||
        (Hk > 0 && (!multiple(k, size) || !multiple(k_out, size))))
        return ATTN_ERR_ALIGN;
    if ((q == q_out && q_stride != q_out_stride) || (Hk > 0 && k == k_out && k_stride != k_out_stride)) return ATTN_ERR_BAD_SHAPE;
    if (T == 0) return ATTN_OK;
    int* status = nullptr;
    int num_sms = 0;
    const attn_status_t st = current_device_info(&status, &num_sms);
    if (st != ATTN_OK) return st;
    RopeParams p;
    p.q = q, p.k = k;
    p.q_out = q_out, p.k_out = k_out;
    p.q_stride = q_stride, p.k_stride = k_stride;
    p.q_out_stride = q_out_stride, p.k_out_stride = k_out_stride;
    p.positions = positions;
    p.inv_freq = inv_freq;
    p.cols = RopeCols{d, rot_begin, rot_dim, interleaved};
    p.T = T;
    p.Hq = Hq;
    p.H = Hq + Hk;
    p.amplitude = amplitude;
    p.transpose = transpose;
    const bool in_place = q == q_out && (Hk == 0 || k == k_out);
    // 16-byte accesses: V elements, whole items on each side of the rotated columns
    const int V = 16 / size;
    bool wide = d % (2 * V) == 0 && rot_begin % (2 * V) == 0 && rot_dim % (2 * V) == 0 && multiple(q, 16) && multiple(q_out, 16) &&
                q_stride % V == 0 && q_out_stride % V == 0;
    if (Hk > 0) wide = wide && multiple(k, 16) && multiple(k_out, 16) && k_stride % V == 0 && k_out_stride % V == 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (elem_type == ATTN_TYPE_BF16)
        e = wide ? launch_rope<__nv_bfloat16, 8>(p, in_place, num_sms, s) : launch_rope<__nv_bfloat16, 1>(p, in_place, num_sms, s);
    else
        e = wide ? launch_rope<float, 4>(p, in_place, num_sms, s) : launch_rope<float, 1>(p, in_place, num_sms, s);
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

// f_i = theta^(-2 i / rot), with the changes for contexts beyond the trained one; see attn.h.
extern "C" attn_status_t attn_rope_freqs(double* inv_freq, double* amplitude, int rot_dim, double theta, int scaling,
                                         double factor, double trained_len, double beta_fast, double beta_slow) {
    if (!inv_freq || !amplitude) return ATTN_ERR_NULL_PTR;
    if (rot_dim <= 0 || rot_dim % 2 != 0 || rot_dim > attn::kRopeMaxDim) return ATTN_ERR_BAD_SHAPE;
    if (!isfinite(theta) || theta <= 0) return ATTN_ERR_BAD_ARG;
    if (scaling != ATTN_ROPE_PLAIN && scaling != ATTN_ROPE_LINEAR && scaling != ATTN_ROPE_NTK && scaling != ATTN_ROPE_YARN)
        return ATTN_ERR_BAD_ARG;
    if (scaling != ATTN_ROPE_PLAIN && !(isfinite(factor) && factor >= 1)) return ATTN_ERR_BAD_ARG;
    if (scaling == ATTN_ROPE_NTK && rot_dim <= 2) return ATTN_ERR_BAD_SHAPE;
    if (scaling == ATTN_ROPE_YARN && !(isfinite(trained_len) && trained_len > 0 && isfinite(beta_fast) && isfinite(beta_slow) &&
                                       beta_fast > beta_slow))
        return ATTN_ERR_BAD_ARG;
    const double base = scaling == ATTN_ROPE_NTK ? theta * pow(factor, (double)rot_dim / (rot_dim - 2)) : theta;
    for (int i = 0; i < rot_dim / 2; ++i) {
        const double f = pow(base, -2.0 * i / rot_dim);
        double out = f;
        if (scaling == ATTN_ROPE_LINEAR) out = f / factor;
        if (scaling == ATTN_ROPE_YARN) {
            const double turns = trained_len * f / 6.283185307179586;
            double keep = (turns - beta_slow) / (beta_fast - beta_slow);
            keep = keep < 0 ? 0 : (keep > 1 ? 1 : keep);
            out = keep * f + (1 - keep) * f / factor;
        }
        inv_freq[i] = out;
    }
    *amplitude = scaling == ATTN_ROPE_YARN ? 0.1 * log(factor) + 1.0 : 1.0;
    return ATTN_OK;
}
