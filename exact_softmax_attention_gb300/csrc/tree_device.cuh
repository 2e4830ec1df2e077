// Device helpers that the kernels of the drafted-token attention share: the rows and lengths of a
// sequence, what a row sees, places in the paged cache, and the values taken out of masked tiles.
#pragma once

#include "attn.h"
#include "ptx.cuh"
#include "tree.cuh"

#include <math.h>

#include <type_traits>

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

// Split size and work item of block `block` where the host left the size open (slots > 0), the same size in
// every block; called by warp 0. The host knows the capacity of the page table only, this the lengths. Of 32
// sizes that need no more than `blocks` blocks it takes the one that ends first, when a block takes as long as
// its tokens and kStart, full splits start first, the others fill the slots that are left, the join of n splits
// takes kJoin n, and blocks that wait for others cost kWait. Lengths and sizes are in units of 64 tokens; least:
// the least size. Measured, batches of 1 to 32 sequences of up to 32768 tokens, equal and ragged: 4% behind the
// best of ten fixed sizes per batch on average, 6% when the page table is four times wider than the lengths need
// (sizes from the capacity alone: 7% and 34%). 40 and 64 sequences (128 cases): 10% behind on average with tight tables,
// 4% ahead with ones four times wider; at worst 61% and 68%, 40 equal ones of 1000 tokens x 4 kv heads in tiles, where 320 blocks
// follow each other in 304 places, which the time above does not count as a second round. It takes 1.3 us, 2.6 us for 64 sequences, the load
// of the lengths included. out: tokens per split, sequence (-1: no work), split (-1: the last one), head group.
__device__ __noinline__ void tree_fit(const int* seqlens, int* chunk_out, int B, int max_len, int HG, int slots, int least,
                                      int block, int blocks, int* out) {
    constexpr float kStart = 6.0f, kJoin = 0.25f, kWait = 1.15f;
    const int lane = threadIdx.x & 31;
    int len[2];  // of sequences 2 lane, 2 lane + 1
#pragma unroll
    for (int x = 0; x < 2; ++x) len[x] = 2 * lane + x < B ? (min(max(__ldg(seqlens + 2 * lane + x), 0), max_len) + 63) >> 6 : 0;
    const float sum = (float)__reduce_add_sync(0xffffffffu, (unsigned)(len[0] + len[1]));
    const int longest = max(1, __reduce_max_sync(0xffffffffu, max(len[0], len[1])));
    const float fHG = (float)HG, fslots = (float)slots;
    // half of the sizes from the even share of a slot upwards, half parts of the longest sequence
    float want = lane < 16 ? __fdividef(sum * fHG, fslots) * (1.0f + 0.125f * lane) : __fdividef((float)longest, (float)(lane - 15));
    want = ceilf(fminf(fmaxf(want, (float)least), (float)max(longest, least)));
    {
        const float inv = __fdividef(1.0f, want);
        const float f0 = (float)len[0], f1 = (float)len[1];
        float full = 0.0f, rest = 0.0f, largest = 0.0f;  // full splits; time and size of the others
        float count = (float)(B - __popc(__ballot_sync(0xffffffffu, len[0] > 0)) - __popc(__ballot_sync(0xffffffffu, len[1] > 0)));
        auto add = [&](float l) {
            const float q = floorf(fmaf(l, inv, 0.5f * inv)), r = fmaf(-q, want, l);
            full += q;
            count += r > 0.0f ? q + 1.0f : q;
            rest += r > 0.0f ? r + kStart : 0.0f;
            largest = fmaxf(largest, r);
        };
#pragma unroll 4
        for (int t = 0; 2 * t < B; ++t) {
            add(__shfl_sync(0xffffffffu, f0, t));
            add(__shfl_sync(0xffffffffu, f1, t));  // (0 behind the last sequence)
        }
        const float fs = full * fHG, waves = floorf(__fdividef(fs, fslots)), over = fs - waves * fslots, one = want + kStart;
        float end = waves * one + fmaxf(over > 0.0f ? one : largest + kStart, __fdividef(rest * fHG, fslots - over));
        end += kJoin * (float)longest * inv;
        count *= fHG;
        if (count > fslots) end *= kWait;
        if (count > (float)blocks) end = INFINITY;
        const unsigned key = __float_as_uint(end), best = __reduce_min_sync(0xffffffffu, key);  // (positive floats)
        want = __shfl_sync(0xffffffffu, want, 31 - __clz(__ballot_sync(0xffffffffu, key == best)));
    }

    // items: the splits of every sequence before its last one, then the last ones, longer ones first if some wait
    int size = (int)want, total, upto, ahead[2], tail[2];  // splits before the last one, size of that
    for (;;) {
        const float inv = __fdividef(1.0f, (float)size);
#pragma unroll
        for (int x = 0; x < 2; ++x) {  // (len - 1) / size, exact after the two corrections
            int q = (int)((float)len[x] * inv), r = len[x] - q * size;
            if (r < 1) --q, r += size;
            if (r > size) ++q, r -= size;
            ahead[x] = len[x] > 0 ? q : 0;
            tail[x] = r;
        }
        upto = ahead[0] + ahead[1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
        }
        total = __shfl_sync(0xffffffffu, upto, 31);
        if ((long long)(total + B) * HG <= blocks) break;
        size = longest;  // no size fitted, or its count was rounded: a split for each sequence does fit
    }
    const int m = (int)((float)block * __fdividef(1.0f, fHG) + 0.5f * __fdividef(1.0f, fHG));  // block / HG (small numbers)
    int rank[2] = {2 * lane, 2 * lane + 1};
    if ((total + B) * HG > slots && m >= total) {  // in four classes
        int above = 0;
        const unsigned below = (1u << lane) - 1;
#pragma unroll
        for (int k = 3; k >= 0; --k) {
            bool in[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) in[x] = 2 * lane + x < B && min(3, 4 * tail[x] / max(1, size)) == k;
            const unsigned b0 = __ballot_sync(0xffffffffu, in[0]), b1 = __ballot_sync(0xffffffffu, in[1]);
            const int at = above + __popc(b0 & below) + __popc(b1 & below);
            if (in[0]) rank[0] = at;
            if (in[1]) rank[1] = at + in[0];
            above += __popc(b0) + __popc(b1);
        }
    }
    upto -= ahead[0] + ahead[1];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        if (2 * lane + x < B && (m < total ? m >= upto && m < upto + ahead[x] : m - total == rank[x])) {
            out[1] = 2 * lane + x;
            out[2] = m < total ? m - upto : -1;
        }
        upto += ahead[x];
    }
    if (lane == 0) {
        out[0] = size * 64;
        if (m >= total + B) out[1] = -1;
        out[3] = block - m * HG;
        if (block == 0) *chunk_out = size * 64;
    }
}

// Work item of a block: tokens per split, sequence, split (-1: the sequence's last one) and head group (kv
// head * groups + row group). False (for the whole block) when it has none. scratch: 4 or, when ranked, B + 1
// ints of shared memory; every thread calls it.
template <bool kCluster>
__device__ __forceinline__ bool tree_item(const TreeParams& p, int* scratch, int& chunk, int& b, int& split, int& hg) {
    const int HG = p.Hkv * p.groups;
    if constexpr (kCluster) {
        chunk = p.chunk;
        b = blockIdx.y;
        split = (int)(blockIdx.x % (unsigned)p.cluster);
        hg = (int)(blockIdx.x / (unsigned)p.cluster);
        return true;
    }
    if (p.slots > 0) {
        if (threadIdx.x < 32)
            tree_fit(p.seqlens, p.ws_chunk, p.B, p.max_pages * p.page_size, HG, p.slots, p.chunk >> 6, blockIdx.x,
                     gridDim.x, scratch);
        __syncthreads();
        chunk = scratch[0], b = scratch[1], split = scratch[2], hg = scratch[3];
        __syncthreads();  // the scratch has other uses
        return b >= 0;
    }
    chunk = p.chunk;
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

// Join of a row's splits by a warp: LSE = log sum_s exp(lse_s), O = sum_s exp(lse_s - LSE) O_s in split order.
// lse_of(i), row_of(i): LSE and D outputs (this lane's ones first) of split i.
template <int D, typename Lse, typename Row>
__device__ __forceinline__ void join_row(int ns, Lse lse_of, Row row_of, __nv_bfloat16* o, float* lse_out) {
    constexpr int PER = D / 32;
    const int lane = threadIdx.x & 31;
    typedef typename std::conditional<D == 128, float4, float2>::type Vec;
    constexpr int kAhead = 8;  // loads in flight; the first ones do not wait for the weights
    Vec v[kAhead];
    auto load = [&](int i) {
#pragma unroll
        for (int x = 0; x < kAhead; ++x) v[x] = i + x < ns ? *reinterpret_cast<const Vec*>(row_of(i + x) + lane * PER) : Vec{};
    };
    load(0);
    // of the first 64 splits, mostly all there are
    const float l0 = lane < ns ? lse_of(lane) : -INFINITY, l1 = lane + 32 < ns ? lse_of(lane + 32) : -INFINITY;
    float mx = fmaxf(l0, l1);
    for (int i = lane + 64; i < ns; i += 32) mx = fmaxf(mx, lse_of(i));
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
    // a split that the row sees nothing of has -inf, zeros as its output and weight 0; a NaN stays
    const float base = mx == -INFINITY ? 0.0f : mx;
    float sum = expf(l0 - base) + expf(l1 - base);
    for (int i = lane + 64; i < ns; i += 32) sum += expf(lse_of(i) - base);
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
    float acc[PER] = {}, lse = -INFINITY;
    if (sum != 0.0f) {
        lse = base + logf(sum);
        float weight = 0.0f;
        for (int i = 0; i < ns; i += kAhead) {
            if (i > 0) load(i);
            if (i % 32 == 0) weight = expf((i == 0 ? l0 : i == 32 ? l1 : i + lane < ns ? lse_of(i + lane) : -INFINITY) - lse);
#pragma unroll
            for (int x = 0; x < kAhead; ++x) {
                const float w = __shfl_sync(0xffffffffu, weight, (i + x) & 31);
                const float* vx = reinterpret_cast<const float*>(&v[x]);
#pragma unroll
                for (int e = 0; e < PER; ++e) acc[e] += w * vx[e];
            }
        }
    }
    if (lane == 0) *lse_out = lse;
#pragma unroll
    for (int e = 0; e < PER; e += 2) *reinterpret_cast<uint32_t*>(o + lane * PER + e) = pack_bf16x2(acc[e], acc[e + 1]);
}

// ---- blocks of a cluster

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The same place of the shared memory of another block.
__device__ __forceinline__ const float* of_block(const float* p, int rank) {
    const float* r;
    asm volatile("mapa.u64 %0, %1, %2;" : "=l"(r) : "l"(p), "r"(rank));
    return r;
}

// Join of the ns splits of R rows by the blocks of a cluster, split i in block i: outputs o_part (rows kStride
// apart) and lse_part of each in its shared memory. Row r of the group is o row first + (r0 + r) / G Hq +
// (r0 + r) % G. Every thread of all blocks calls it. (Not inlined: the kernels' own code stays as short.)
template <int D, int kStride>
__device__ __noinline__ void cluster_join(const float* o_part, const float* lse_part, __nv_bfloat16* o, float* lse, long long first, int r0,
                                          int R, int G, int Hq, int cluster, int ns) {
    __syncwarp();
    cluster_sync();
    const int rank = (int)(blockIdx.x % (unsigned)cluster), warps = blockDim.x >> 5;
    for (int r = rank + cluster * (int)(threadIdx.x >> 5); r < R; r += cluster * warps) {
        const int i = (r0 + r) / G;
        const long long row = first + (long long)i * Hq + (r0 + r - i * G);
        join_row<D>(
            ns, [&](int x) { return *of_block(lse_part + r, x); }, [&](int x) { return of_block(o_part + r * kStride, x); }, o + row * D,
            lse + row);
    }
    cluster_sync();  // a block stays until the others have read its part
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

// Adds to the outputs of a warp's rows (first, first + step, ... < rows of the group that starts at row r0; 32 at
// most) the non-finite values of V of the tokens [t0, t0 + 64) below t_end that each sees: what the products
// left out of the tiles where they took them for zero. Every lane owns D / 32 columns and keeps for each which
// tokens hold infinities and NaN, so the values are read once for all rows. split >= 0: the outputs are those
// of that split in the workspace; -1: the call's; -2: rows part_stride apart from `part` on. (A rare path, out
// of line: the kernels' registers stay as they are.)
template <int D, int FMT>
__device__ __noinline__ void add_nonfinite(const TreeParams& p, int b, int kvh, int r0, int first, int step, int rows, int t0, int t_end,
                                           int split, float* part, int part_stride) {
    constexpr int PER = D / 32;
    const int lane = threadIdx.x & 31;
    TreeSeq s;
    if (!tree_seq(p, b, s)) return;
    const int* pt = p.page_table + (long long)b * p.max_pages;
    unsigned long long seen = 0;  // by row first + lane step
    if (first + lane * step < rows) {
        const int i = (r0 + first + lane * step) / p.G;
        seen = tree_window(p.mask ? p.mask + (long long)(s.q0 + i) * p.mask_words : nullptr, p.mask_words, i, s.ctx, s.len, t0);
        if (t_end - t0 < 64) seen &= (1ull << (t_end - t0)) - 1;
    }
    int row[2];  // of tokens lane and lane + 32
#pragma unroll
    for (int e = 0; e < 2; ++e) row[e] = t0 + lane + 32 * e < t_end ? cache_row(p, pt, t0 + lane + 32 * e) : -1;
    unsigned long long pos[PER] = {}, neg[PER] = {}, nan[PER] = {};
#pragma unroll 4
    for (int t = 0; t < 64; ++t) {
        const int r = __shfl_sync(0xffffffffu, t < 32 ? row[0] : row[1], t & 31);
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            const float v = r >= 0 ? cached_value<FMT>(p.v_cache, ((long long)r * p.Hkv + kvh) * D + lane * PER + e) : 0.0f;
            const unsigned long long bit = 1ull << t;
            pos[e] |= v == INFINITY ? bit : 0;
            neg[e] |= v == -INFINITY ? bit : 0;
            nan[e] |= isnan(v) ? bit : 0;
        }
    }
    for (int k = 0; first + k * step < rows; ++k) {
        const unsigned long long w = __shfl_sync(0xffffffffu, seen, k);
        const int r = first + k * step, i = (r0 + r) / p.G;
        const long long orow = (long long)(s.q0 + i) * p.Hq + kvh * p.G + (r0 + r - i * p.G);
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            float x = 0.0f;
            if (w & pos[e]) x += INFINITY;
            if (w & neg[e]) x -= INFINITY;
            if (w & nan[e]) x = __int_as_float(0x7fffffff);
            if (x == 0.0f) continue;
            x *= p.v_descale;  // (its sign; the weight of a seen token is above 0)
            const int c = lane * PER + e;
            if (split == -1) {
                __nv_bfloat16* to = p.o + orow * D + c;
                *to = __float2bfloat16(__bfloat162float(*to) + x);
            } else if (split == -2) {
                part[r * part_stride + c] += x;
            } else {
                p.ws_o[(orow * p.max_splits + split) * D + c] += x;
            }
        }
    }
}

// Is either 16-bit half of w non-finite (f16 when half_fmt, else bf16)? Mask with ones in the finite
// halves.
__device__ __forceinline__ uint32_t finite_halves(uint32_t w, bool half_fmt) {
    const uint32_t e = half_fmt ? 0x7C00u : 0x7F80u;
    return ((w & e) == e ? 0u : 0xFFFFu) | (((w >> 16) & e) == e ? 0u : 0xFFFF0000u);
}

}  // namespace
}  // namespace attn
