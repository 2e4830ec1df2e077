// Device helpers that the kernels of the drafted-token attention share: the rows and lengths of a
// sequence, what a row sees, places in the paged cache, and the values taken out of masked tiles.
#pragma once

#include "attn.h"
#include "ptx.cuh"
#include "tree.cuh"

#include <math.h>

namespace attn {
namespace {

__device__ __forceinline__ int cdiv(int a, int b) { return (a + b - 1) / b; }

// Rows and cached tokens of sequence b. False: it has no rows in the output (none given, or offsets
// out of range, which is recorded). A length out of range counts as 0 and is recorded.
struct TreeSeq {
    int q0, n;     // first row of q, rows
    int len, ctx;  // cached tokens, those before the drafted ones
};
__device__ __forceinline__ bool tree_seq(const TreeParams& p, int b, TreeSeq& s) {
    if (p.cu_seqlens) {
        const long long c0 = __ldg(p.cu_seqlens + b), c1 = __ldg(p.cu_seqlens + b + 1);
        if (c0 < 0 || c1 < c0 || c1 > p.T || c1 - c0 > p.max_q) {
            if (threadIdx.x == 0) atomicCAS(p.status, 0, kDevBadIndex);
            return false;
        }
        s.q0 = (int)c0, s.n = (int)(c1 - c0);
    } else {
        s.n = p.T / p.B;
        s.q0 = b * s.n;
    }
    if (s.n == 0) return false;
    int len = __ldg(p.seqlens + b);
    if (len != 0 && (len < s.n || len > (long long)p.max_pages * p.page_size)) {
        if (threadIdx.x == 0) atomicCAS(p.status, 0, kDevBadIndex);
        len = 0;
    }
    s.len = len;
    s.ctx = len - s.n;
    return true;
}

// Work item of a block: sequence, split (-1: the sequence's last one) and head group (kv head * groups +
// row group). False (for the whole block) when it has none. scratch: 2 B + 1 ints of shared memory when
// ranked; every thread calls it.
__device__ __forceinline__ bool tree_item(const TreeParams& p, int* scratch, int& b, int& split, int& hg) {
    const int HG = p.Hkv * p.groups;
    if (p.full_rows < 0 || (int)blockIdx.y < p.full_rows) {
        b = blockIdx.y;
        split = (int)(blockIdx.x / (unsigned)HG);
        hg = (int)(blockIdx.x % (unsigned)HG);
        return true;
    }
    const long long j = (long long)(blockIdx.y - p.full_rows) * gridDim.x + blockIdx.x;
    if (j >= (long long)p.B * HG) return false;
    hg = (int)(j % HG);
    b = (int)(j / HG);
    split = -1;
    if (p.ranked) {
        // the sequence whose last split has rank b in decreasing length (ties: the lower one first)
        const int max_len = p.max_pages * p.page_size;
        int* found = scratch + p.B;
        for (int t = threadIdx.x; t < p.B; t += blockDim.x) {
            const int len = min(max(__ldg(p.seqlens + t), 0), max_len), ns = cdiv(len, p.chunk);
            scratch[t] = len - (ns > 0 ? ns - 1 : 0) * p.chunk;
        }
        __syncthreads();
        for (int t = threadIdx.x; t < p.B; t += blockDim.x) {
            const int mine = scratch[t];
            int rank = 0;
            for (int u = 0; u < p.B; ++u) rank += scratch[u] > mine || (scratch[u] == mine && u < t);
            if (rank == b) *found = t;
        }
        __syncthreads();
        b = *found;
        __syncthreads();  // the scratch has other uses
    }
    return true;
}

// Bits of the keys kb .. kb + 63 that drafted token i of the sequence sees. row: its mask words, or
// nullptr for a chain.
__device__ __forceinline__ unsigned long long tree_window(const unsigned long long* row, int words, int i, int ctx, int len,
                                                          int kb) {
    const int rel = kb - ctx;  // drafted index of bit 0
    unsigned long long w = ~0ull;
    if (rel > -64) {
        if (row) {
            if (rel < 0) {
                w = (__ldg(row) << -rel) | ((1ull << -rel) - 1);
            } else {
                const int x = rel >> 6, sh = rel & 63;
                w = x < words ? __ldg(row + x) >> sh : 0;
                if (sh && x + 1 < words) w |= __ldg(row + x + 1) << (64 - sh);
            }
        } else {
            const int cnt = i - rel + 1;
            w = cnt >= 64 ? ~0ull : (cnt <= 0 ? 0 : (1ull << cnt) - 1);
        }
    }
    const int lim = len - kb;
    if (lim < 64) w &= lim <= 0 ? 0 : (1ull << lim) - 1;
    return w;
}

// Page-table index and slot of token tok (0 <= tok < 2^31).
__device__ __forceinline__ int page_of(const TreeParams& p, int tok, int& slot) {
    const int q = p.ps_magic ? (int)(__umulhi((unsigned)tok, p.ps_magic) >> p.ps_shift) : tok;
    slot = tok - q * p.page_size;
    return q;
}

// Cache row of token tok of a sequence (pt: its row of the page table), or -1 for a page out of range.
__device__ __forceinline__ int cache_row(const TreeParams& p, const int* pt, int tok) {
    int slot;
    const int pg = __ldg(pt + page_of(p, tok, slot));
    if (pg < 0 || pg >= p.num_pages) {
        atomicCAS(p.status, 0, kDevBadIndex);
        return -1;
    }
    return pg * p.page_size + slot;  // < num_pages * page_size <= INT32_MAX
}

template <int FMT>
__device__ __forceinline__ uint32_t fp8x2_f16x2(uint32_t two_codes) {
    const uint16_t v = (uint16_t)two_codes;
    uint32_t d;
    if (FMT == ATTN_FP8_E4M3)
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(v));
    else
        asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(d) : "h"(v));
    return d;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float half_value(uint16_t h) {
    float f;
    asm("cvt.f32.f16 %0, %1;" : "=f"(f) : "h"(h));
    return f;
}

// Value e of a V row in the cache as a float (without the descale).
template <int FMT>
__device__ __forceinline__ float cached_value(const void* cache, long long e) {
    if constexpr (FMT == ATTN_KV_BF16)
        return __bfloat162float(static_cast<const __nv_bfloat16*>(cache)[e]);
    else
        return half_value((uint16_t)fp8x2_f16x2<FMT>(static_cast<const uint8_t*>(cache)[e]));
}

// Sum of the non-finite values in column d of the V rows of tokens [t0, t1) that row i sees: what the
// products left out of the tiles where they took them for zero.
template <int FMT>
__device__ __forceinline__ float nonfinite_sum(const TreeParams& p, const int* pt, const unsigned long long* mrow, int i, const TreeSeq& s,
                               int t0, int t1, int kvh, int D, int d) {
    float sum = 0.0f;
    for (int t = t0; t < t1; ++t) {
        if (!(tree_window(mrow, p.mask_words, i, s.ctx, s.len, t) & 1)) continue;
        const int row = cache_row(p, pt, t);
        if (row < 0) continue;
        const float v = cached_value<FMT>(p.v_cache, ((long long)row * p.Hkv + kvh) * D + d);
        if (!isfinite(v)) sum += v;
    }
    return sum;
}

// Is either 16-bit half of w non-finite (f16 when half_fmt, else bf16)? Mask with ones in the finite
// halves.
__device__ __forceinline__ uint32_t finite_halves(uint32_t w, bool half_fmt) {
    const uint32_t e = half_fmt ? 0x7C00u : 0x7F80u;
    return ((w & e) == e ? 0u : 0xFFFFu) | (((w >> 16) & e) == e ? 0u : 0xFFFF0000u);
}

}  // namespace
}  // namespace attn
