// Writes into and reads from a paged key/value cache, in bf16 or in 8-bit floating point with one
// descale per tensor: code = fp8(x / descale), value = descale * fp8(code).
//
// A write takes the new rows of each sequence, optionally rotates K by its positions (in fp32, so
// that a cached key is rounded once), and stores them at the end of the sequence; a read returns
// the last rows of each sequence as bf16. Both move each element once in and once out and are
// bounded by memory. What a short call costs is the chain of dependent loads from the packed
// row to its page (offsets, length, page table); the rows themselves do not depend on it, so each
// thread loads its first item before the places are known.
//
// Measured: 264 K tokens (8 heads of 128) from e4m3 to bf16 rows in 247 us, 0.97 of the measured copy
// rate; 131072 tokens to a bf16 cache 170 us (0.93), to e4m3 142 us (0.84), with rotation 160 us (0.74); 64
// tokens 4.2 us. What the writes wait for (counters of the 131072-token calls): to bf16 the loads (memory 78 %
// busy, issue slots 32 %); to e4m3 the loads too (70 %, 60 %); rotated to e4m3 no unit is full (62 %, 73 %): with 64
// registers and so 32 warps per SM, loads in flight and instructions to issue cover each other only in part.
#include "attn.h"
#include "launch.cuh"
#include "rows.cuh"

#include <math.h>

namespace attn {
namespace {

constexpr int kCacheThreads = 512;  // at most
constexpr int kCacheMaxTokens = 32;  // tokens per block
// Threads that an SM holds (64 and 32 registers each), and items per thread, at most. Measured, us: 14155 tokens to
// e4m3 with rotation, items 8: 23.1, 12: 22.0, 16: 22.0 (885 blocks, whole waves or not, 24.3); 131072 tokens 8: 163,
// 12: 160; to bf16 8: 169, 12: 170. 14155 tokens read from e4m3 4: 17.7, 8: 20.5; 131072 from bf16 4: 160, 8: 163.
constexpr int kWriteThreads = 1024, kReadThreads = 2048, kWriteItems = 12, kReadItems = 4;

struct CacheParams {
    const __nv_bfloat16* in[2];  // write: k, v
    __nv_bfloat16* out[2];       // read: k, v
    long long stride[2];         // elements between rows of k and v
    uint8_t* cache[2];           // bf16 or 8-bit codes [num_pages * page_size, Hkv, d]
    float descale[2], inv[2];    // inv: 1 / descale, or 0 where divide() has to divide
    PagedRows rows;
    RopeCols cols;               // rot 0: no rotation
    const int* positions;
    const double* inv_freq;
    float amplitude;
    RowShare share;
    int Hkv, items;              // work items per head
};

// Cache rows of tokens [t0, t0 + tokens), a warp for each in turn. Every thread of the block calls it.
__device__ __forceinline__ void find_places(const PagedRows& rows, int t0, int tokens, long long* place) {
    for (int t = threadIdx.x >> 5; t < tokens; t += blockDim.x >> 5) {
        const long long r = paged_row(rows, t0 + t);
        if ((threadIdx.x & 31) == 0) place[t] = r;
    }
}

// Two values to a pair of 8-bit codes (low byte first): nearest even, magnitudes above the largest
// finite one saturate, NaN stays NaN.
template <int FMT>
__device__ __forceinline__ uint32_t fp8x2(float lo, float hi) {
    uint16_t r;
    if (FMT == ATTN_FP8_E4M3)
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two codes to two floats (exact).
template <int FMT>
__device__ __forceinline__ void fp8x2_values(uint32_t two, float& lo, float& hi) {
    uint32_t h2;
    const uint16_t v = (uint16_t)two;
    if (FMT == ATTN_FP8_E4M3)
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(v));
    else
        asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h2) : "h"(v));
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(h2));
}

// x[e] / d rounded to fp32, with inv the rounded 1 / d: the product with inv, corrected by the exact
// remainder (Markstein, "Computation of elementary functions on the IBM RISC System/6000 processor",
// 1990). Far beyond the 8-bit range, where the remainder may overflow or x is not finite, and where inv = 0
// asks for it, by division. (With a division per element the write took 1.4 times as long.)
template <int V>
__device__ __forceinline__ void divide(float (&x)[V], float d, float inv) {
    float q[V], top = 0.0f;
#pragma unroll
    for (int e = 0; e < V; ++e) {
        q[e] = x[e] * inv;
        top = fmaxf(top, fabsf(q[e]));
    }
    if (inv != 0.0f && top < 1e6f) {
#pragma unroll
        for (int e = 0; e < V; ++e) x[e] = fmaf(-fmaf(q[e], d, -x[e]), inv, q[e]);  // (in this order -0 stays -0)
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) x[e] /= d;
    }
}

// V values into the cache at element offset at.
template <int FMT, int V>
__device__ __forceinline__ void store_cache(uint8_t* cache, long long at, float (&x)[V], float descale, float inv) {
    if constexpr (FMT == ATTN_KV_BF16) {
        store_row<V>(reinterpret_cast<__nv_bfloat16*>(cache) + at, x);
    } else {
        divide<V>(x, descale, inv);
        if constexpr (V == 8)
            *reinterpret_cast<uint2*>(cache + at) = make_uint2(fp8x2<FMT>(x[0], x[1]) | (fp8x2<FMT>(x[2], x[3]) << 16),
                                                               fp8x2<FMT>(x[4], x[5]) | (fp8x2<FMT>(x[6], x[7]) << 16));
        else
            cache[at] = (uint8_t)fp8x2<FMT>(x[0], 0.0f);
    }
}

template <int FMT, int V>
__global__ void __launch_bounds__(kCacheThreads) cache_write_kernel(const CacheParams p) {
    extern __shared__ __align__(16) float angles[];
    __shared__ long long place[kCacheMaxTokens];
    typedef typename RawOf<__nv_bfloat16, V>::type Raw;
    const int half = p.cols.rot / 2;
    const long long t0 = (long long)blockIdx.x * p.share.tokens;
    const int tokens = (int)min((long long)p.share.tokens, p.rows.T - t0);
    float* cs = angles;
    float* sn = angles + p.share.tokens * half;
    const int groups = blockDim.x / p.share.width, group = threadIdx.x / p.share.width;
    const int pairs = 2 * p.Hkv * p.items;  // heads of K, then of V
    int pair = threadIdx.x - group * p.share.width;
    bool first = true;
    do {  // (threads without a pair only take part in the angles and places)
        const bool mine = group < groups && pair < pairs;
        const int h = mine ? pair / p.items : 0, j = mine ? pair - h * p.items : 0;
        const bool v = h >= p.Hkv;
        const int head = v ? h - p.Hkv : h;
        const long long stride = v ? p.stride[1] : p.stride[0];
        uint8_t* cache = v ? p.cache[1] : p.cache[0];
        const float descale = v ? p.descale[1] : p.descale[0], inv = v ? p.inv[1] : p.inv[0];
        int a = V * j, b = a + p.cols.d / 2;
        const bool turned = !v && item_cols<V>(p.cols, j, a, b);
        const __nv_bfloat16* src = (v ? p.in[1] : p.in[0]) + (t0 + group) * stride + (long long)head * p.cols.d;
        // an item is loaded while the one before is converted and stored, the first while the places of the
        // tokens are looked up
        Raw ra, rb;
        const int last = mine ? tokens : 0;
        if (group < last) {
            ra = load_raw<__nv_bfloat16, V>(src + a);
            rb = load_raw<__nv_bfloat16, V>(src + b);
        }
        if (first) {
            if (half > 0) block_angles(p.inv_freq, p.positions + t0, tokens, half, p.amplitude, false, cs, sn);
            find_places(p.rows, (int)t0, tokens, place);
            __syncthreads();
            first = false;
        }
        for (int t = group; t < last; t += groups) {
            float xa[V], xb[V];
            unpack<__nv_bfloat16, V>(ra, xa);
            unpack<__nv_bfloat16, V>(rb, xb);
            src += groups * stride;
            if (t + groups < last) {
                ra = load_raw<__nv_bfloat16, V>(src + a);
                rb = load_raw<__nv_bfloat16, V>(src + b);
            }
            if (turned) rotate_item<V>(xa, xb, p.cols, j, cs + t * half, sn + t * half);
            const long long row = place[t];
            if (row < 0) continue;
            const long long to = (row * p.Hkv + head) * p.cols.d;
            store_cache<FMT, V>(cache, to + a, xa, descale, inv);
            store_cache<FMT, V>(cache, to + b, xb, descale, inv);
        }
        pair += p.share.width;
    } while (pair < pairs);
}

// 16 elements per item: one 16-byte load of codes (two of bf16), two 16-byte stores.
template <int FMT>
__global__ void __launch_bounds__(kCacheThreads) cache_read_kernel(const CacheParams p) {
    __shared__ long long place[kCacheMaxTokens];
    const long long t0 = (long long)blockIdx.x * p.share.tokens;
    const int tokens = (int)min((long long)p.share.tokens, p.rows.T - t0);
    find_places(p.rows, (int)t0, tokens, place);
    __syncthreads();
    const int groups = blockDim.x / p.share.width, group = threadIdx.x / p.share.width;
    const int pairs = 2 * p.Hkv * p.items;
    if (group >= groups) return;
    for (int pair = threadIdx.x - group * p.share.width; pair < pairs; pair += p.share.width)
#pragma unroll 2
    for (int t = group; t < tokens; t += groups) {
        const bool kv = pair >= pairs / 2;
        const int c = (kv ? pair - pairs / 2 : pair) * 16;  // element of the row [Hkv, d]
        const long long row = place[t];
        if (row == kRowNone) continue;
        __nv_bfloat16* dst = (kv ? p.out[1] : p.out[0]) + (t0 + t) * (kv ? p.stride[1] : p.stride[0]) + c;
        const uint8_t* cache = kv ? p.cache[1] : p.cache[0];
        uint4 o0 = make_uint4(0, 0, 0, 0), o1 = o0;  // a bad page reads as zeros
        if (row >= 0) {
            const long long e = row * p.Hkv * p.cols.d + c;
            if constexpr (FMT == ATTN_KV_BF16) {
                const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(cache) + e);
                o0 = src[0], o1 = src[1];
            } else {
                const uint4 x = *reinterpret_cast<const uint4*>(cache + e);
                const uint32_t in[4] = {x.x, x.y, x.z, x.w};
                uint32_t out[8];
                const float ds = kv ? p.descale[1] : p.descale[0];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float lo, hi;
                    fp8x2_values<FMT>(in[i / 2] >> (16 * (i & 1)), lo, hi);
                    out[i] = pack_bf16x2(lo * ds, hi * ds);
                }
                o0 = make_uint4(out[0], out[1], out[2], out[3]);
                o1 = make_uint4(out[4], out[5], out[6], out[7]);
            }
        }
        reinterpret_cast<uint4*>(dst)[0] = o0;
        reinterpret_cast<uint4*>(dst)[1] = o1;
    }
}

template <int FMT, int V>
cudaError_t launch_write(CacheParams p, int num_sms, cudaStream_t stream) {
    p.items = p.cols.d / (2 * V);
    p.share = share_rows(p.rows.T, 2 * p.Hkv * p.items, kWriteItems, kCacheMaxTokens, kWriteThreads, num_sms);
    const long long blocks = ((long long)p.rows.T + p.share.tokens - 1) / p.share.tokens;
    const size_t smem = (size_t)p.share.tokens * p.cols.rot * sizeof(float);
    return launch_kernel(cache_write_kernel<FMT, V>, dim3((unsigned)blocks), p.share.threads, smem, stream, {}, p);
}

template <int FMT>
cudaError_t launch_read(CacheParams p, int num_sms, cudaStream_t stream) {
    p.items = p.cols.d / 16;
    p.share = share_rows(p.rows.T, 2 * p.Hkv * p.items, kReadItems, kCacheMaxTokens, kReadThreads, num_sms);
    const long long blocks = ((long long)p.rows.T + p.share.tokens - 1) / p.share.tokens;
    return launch_kernel(cache_read_kernel<FMT>, dim3((unsigned)blocks), p.share.threads, 0, stream, {}, p);
}

bool multiple(const void* p, long long bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

// Checks that both directions share; fills what both use.
attn_status_t check(CacheParams& p, const void* k_cache, const void* v_cache, const void* k, const void* v, long long k_stride,
                    long long v_stride, bool rows_written, const int* page_table, const int* seqlens, const int* cu_seqlens,
                    int page_size, int T, int B, int Hkv, int d, int max_pages, int num_pages, int kv_format, float k_descale,
                    float v_descale) {
    if (!k_cache || !v_cache || !k || !v || !page_table || !seqlens) return ATTN_ERR_NULL_PTR;
    if (kv_format != ATTN_FP8_E4M3 && kv_format != ATTN_FP8_E5M2 && kv_format != ATTN_KV_BF16) return ATTN_ERR_BAD_ARG;
    if (!isfinite(k_descale) || !isfinite(v_descale) || k_descale == 0 || v_descale == 0) return ATTN_ERR_BAD_ARG;
    if (T < 0 || B < 0 || Hkv <= 0 || Hkv > 65535 || d <= 0 || d % 16 != 0 || d > 256 || page_size <= 0 || max_pages <= 0 ||
        num_pages <= 0 || (long long)num_pages * page_size > INT32_MAX || (long long)max_pages * page_size > INT32_MAX)
        return ATTN_ERR_BAD_SHAPE;
    if (!cu_seqlens && T > 0 && (B == 0 || T % B != 0)) return ATTN_ERR_BAD_SHAPE;
    const long long row = (long long)Hkv * d;
    if (k_stride % 8 != 0 || v_stride % 8 != 0 || k_stride < (rows_written ? row : 0) || v_stride < (rows_written ? row : 0))
        return ATTN_ERR_BAD_SHAPE;
    if (!multiple(k_cache, 16) || !multiple(v_cache, 16) || !multiple(k, 16) || !multiple(v, 16) || !multiple(page_table, 4) ||
        !multiple(seqlens, 4) || (cu_seqlens && !multiple(cu_seqlens, 4)))
        return ATTN_ERR_ALIGN;
    p.stride[0] = k_stride, p.stride[1] = v_stride;
    p.cache[0] = static_cast<uint8_t*>(const_cast<void*>(k_cache));
    p.cache[1] = static_cast<uint8_t*>(const_cast<void*>(v_cache));
    p.descale[0] = k_descale, p.descale[1] = v_descale;
    for (int i = 0; i < 2; ++i)  // (beyond these the reciprocal or the remainder could leave the range of fp32)
        p.inv[i] = fabsf(p.descale[i]) > 0x1p-100f && fabsf(p.descale[i]) < 0x1p100f ? 1.0f / p.descale[i] : 0.0f;
    p.rows = PagedRows{page_table, seqlens, cu_seqlens, B, T, max_pages, page_size, num_pages, nullptr};
    p.cols = RopeCols{d, 0, 0, 0};
    p.positions = nullptr;
    p.inv_freq = nullptr;
    p.amplitude = 1.0f;
    p.Hkv = Hkv;
    return ATTN_OK;
}

}  // namespace
}  // namespace attn

extern "C" attn_status_t attn_kv_write_paged(const void* k, const void* v, long long k_stride, long long v_stride, void* k_cache,
                                             void* v_cache, const int* page_table, const int* seqlens, const int* cu_seqlens,
                                             int page_size, int T, int B, int Hkv, int d, int max_pages_per_seq, int num_pages,
                                             int kv_format, float k_descale, float v_descale, const int* positions,
                                             const double* inv_freq, int rot_begin, int rot_dim, int interleaved, float amplitude,
                                             void* stream) {
    using namespace attn;
    CacheParams p;
    attn_status_t st = check(p, k_cache, v_cache, k, v, k_stride, v_stride, false, page_table, seqlens, cu_seqlens, page_size, T, B,
                             Hkv, d, max_pages_per_seq, num_pages, kv_format, k_descale, v_descale);
    if (st != ATTN_OK) return st;
    if (rot_dim != 0) {
        if (!positions || !inv_freq) return ATTN_ERR_NULL_PTR;
        if (rot_dim < 0 || rot_dim % 2 != 0 || rot_begin < 0 || rot_begin > d - rot_dim) return ATTN_ERR_BAD_SHAPE;
        if ((interleaved != 0 && interleaved != 1) || !isfinite(amplitude)) return ATTN_ERR_BAD_ARG;
        if (!multiple(positions, 4) || !multiple(inv_freq, 8)) return ATTN_ERR_ALIGN;
        p.cols = RopeCols{d, rot_begin, rot_dim, interleaved};
        p.positions = positions;
        p.inv_freq = inv_freq;
        p.amplitude = amplitude;
    }
    if (T == 0 || B == 0) return ATTN_OK;
    int num_sms = 0;
    if ((st = current_device_info(&p.rows.status, &num_sms)) != ATTN_OK) return st;
    for (int i = 0; i < 2; ++i) p.in[i] = static_cast<const __nv_bfloat16*>(i ? v : k), p.out[i] = nullptr;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // whole 16-element items on each side of the rotated columns, else pair by pair
    const bool wide = p.cols.begin % 16 == 0 && p.cols.rot % 16 == 0;
    cudaError_t e;
    if (kv_format == ATTN_FP8_E4M3)
        e = wide ? launch_write<ATTN_FP8_E4M3, 8>(p, num_sms, s) : launch_write<ATTN_FP8_E4M3, 1>(p, num_sms, s);
    else if (kv_format == ATTN_FP8_E5M2)
        e = wide ? launch_write<ATTN_FP8_E5M2, 8>(p, num_sms, s) : launch_write<ATTN_FP8_E5M2, 1>(p, num_sms, s);
    else
        e = wide ? launch_write<ATTN_KV_BF16, 8>(p, num_sms, s) : launch_write<ATTN_KV_BF16, 1>(p, num_sms, s);
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

extern "C" attn_status_t attn_kv_read_paged(const void* k_cache, const void* v_cache, void* k, void* v, long long k_stride,
                                            long long v_stride, const int* page_table, const int* seqlens, const int* cu_seqlens,
                                            int page_size, int T, int B, int Hkv, int d, int max_pages_per_seq, int num_pages,
                                            int kv_format, float k_descale, float v_descale, void* stream) {
    using namespace attn;
    CacheParams p;
    attn_status_t st = check(p, k_cache, v_cache, k, v, k_stride, v_stride, true, page_table, seqlens, cu_seqlens, page_size, T, B,
                             Hkv, d, max_pages_per_seq, num_pages, kv_format, k_descale, v_descale);
    if (st != ATTN_OK) return st;
    if (T == 0 || B == 0) return ATTN_OK;
    int num_sms = 0;
    if ((st = current_device_info(&p.rows.status, &num_sms)) != ATTN_OK) return st;
    for (int i = 0; i < 2; ++i) p.in[i] = nullptr, p.out[i] = static_cast<__nv_bfloat16*>(i ? v : k);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = kv_format == ATTN_FP8_E4M3   ? launch_read<ATTN_FP8_E4M3>(p, num_sms, s)
                          : kv_format == ATTN_FP8_E5M2 ? launch_read<ATTN_FP8_E5M2>(p, num_sms, s)
                                                       : launch_read<ATTN_KV_BF16>(p, num_sms, s);
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}
