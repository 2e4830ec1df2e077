// Shared by the two kernels that accumulate attention weight per cached token: parameters, the sequences'
// rows and lengths, places in the paged cache.
#pragma once

#include "attn.h"
#include "kernels.cuh"
#include "launch.cuh"
#include "ptx.cuh"

#include <math.h>

namespace attn {

// x / d for 0 <= x < 2^31: multiplier ceil(2^(31+k) / d), k = ceil(log2 d).
struct Divisor {
    int d;
    unsigned magic;
    int shift;
    Divisor() = default;
    explicit Divisor(int divisor) : d(divisor), magic(0), shift(0) {
        if (d == 1) return;
        int k = 0;
        while ((1LL << k) < d) ++k;
        magic = (unsigned)(((1ULL << (31 + k)) + (unsigned long long)d - 1) / (unsigned long long)d);
        shift = k - 1;
    }
#ifdef __CUDACC__
    __device__ __forceinline__ int operator()(int x) const { return magic ? (int)(__umulhi((unsigned)x, magic) >> shift) : x; }
#endif
};

struct ScoreParams {
    const __nv_bfloat16* q;  // [T, Hq, d]
    const float* lse;        // [T, Hq]
    const void* k_cache;     // [num_pages, page_size, Hkv, d], bf16 or 8-bit codes
    float* score;            // [num_pages, Hkv, page_size]
    const int* page_table;   // [B, max_pages]
    const int* seqlens;      // [B], the rows' tokens included
    const int* cu_seqlens;   // [B + 1] or nullptr: T / B rows each
    int B, T, max_q, Hq, Hkv, G, page_size, max_pages, num_pages, num_sms;
    float scale_log2, decay;  // scale (key descale included) times log2(e)
    float unit;              // tiles: -log2(e) / scale_log2
    Divisor by_page;
    int row_heads;           // few rows: kv heads of a block
    int chunk, chunks;       // few rows: tokens per block, blocks of the longest sequence; 0: runs of all tokens there are
    // tiles: [blocks, 2, unit_tok] sums of units that lie in several blocks; 8-bit caches: factor of the scores of each row of q
    float *partial, *factor;
    int unit_tok, unit_shift;    // tokens of a unit: 128, 256 or 512; their logarithm
    int block_tok, head_blocks;  // tokens of a block of rows; blocks of rows of a token (one of the two is 1)
    Divisor by_block_tok;
    Divisor unit_blocks;         // blocks of rows for the tokens of a unit, rounded down, and the division by that
    Divisor grid;                // blocks
    int box_rows;                // rows of a copy of keys through the map (64 or 16, dividing the page size), 1: no map
    int* status;
    unsigned long long watchdog_ns;
};

cudaError_t launch_score_rows(const ScoreParams& p, int d, int kv_format, cudaStream_t stream);
cudaError_t launch_score_tiles(const ScoreParams& p, int d, int kv_format, cudaStream_t stream);

// Rows per kv head (queries x query heads) up to which a warp's products take them; more go to the tiles. A rule on rows and width alone: it is up to 9 %
// off for bf16 keys where there are many heads (8 of 128, 16 and 24 rows), and the other way with one head. Measured, us, products / tiles, 32 x
// U[1333, 4000] tokens: 8 heads of 64, 24 rows, bf16 26.2 / 29.0, e4m3 22.7 / 32.1; 32 rows 30.9 / 29.0, 27.8 / 31.7; one head, 32 rows, 8.4 / 11.3,
// 9.6 / 14.4. 8 heads of 128, 16 rows, 36.4 / 35.6, e4m3 26.6 / 34.2; 24 rows 38.8 / 35.5, 31.7 / 34.5; one head, 24 rows, 9.8 / 12.3, 10.1 / 14.6;
// 8 heads, 32 rows, 63 / 36.
constexpr int score_few_rows(int d) { return d == 64 ? 32 : 24; }

#ifdef __CUDACC__
namespace {

// A load that stays in its place, behind the wait for the kernel before. (Plain loads do as well, but with them the compiler arranged the tile
// kernel so that whole prompts took 129 us, not 126.)
__device__ __forceinline__ int load_in_place(const int* p) {
    int x;
    asm volatile("ld.global.s32 %0, [%1];" : "=r"(x) : "l"(p) : "memory");
    return x;
}

// Rows and cached tokens of sequence b. False: none of its slots are touched (no rows; or a length or offsets out
// of range, which is recorded).
struct ScoreSeq {
    int q0, n;     // first row of q, rows
    int len, ctx;  // cached tokens, those before the rows' own
};
__device__ __forceinline__ bool score_seq(const ScoreParams& p, int b, ScoreSeq& s) {
    long long c0, c1;
    const int len = load_in_place(p.seqlens + b);
    if (p.cu_seqlens) {
        c0 = load_in_place(p.cu_seqlens + b), c1 = load_in_place(p.cu_seqlens + b + 1);
    } else {
        const int n = p.T / p.B;
        c0 = (long long)b * n, c1 = c0 + n;
    }
    const long long n = c1 - c0;
    if (n == 0) return false;
    if (c0 < 0 || n < 0 || c1 > p.T || n > p.max_q || len < n || len > (long long)p.max_pages * p.page_size) {
        atomicCAS(p.status, 0, kDevBadIndex);
        return false;
    }
    s.q0 = (int)c0, s.n = (int)n;
    s.len = len;
    s.ctx = len - s.n;
    return true;
}

// Page-table index and slot of token tok (0 <= tok < 2^31).
__device__ __forceinline__ int score_page(const ScoreParams& p, int tok, int& slot) {
    const int q = p.by_page(tok);
    slot = tok - q * p.page_size;
    return q;
}

// Physical page of a token, or -1 (recorded) for one out of range; pt: the sequence's row of the page table.
__device__ __forceinline__ int score_place(const ScoreParams& p, const int* pt, int tok, int& slot) {
    const int page = pt[score_page(p, tok, slot)];
    if (page >= 0 && page < p.num_pages) return page;
    atomicCAS(p.status, 0, kDevBadIndex);
    return -1;
}

__device__ __forceinline__ float* score_slot(const ScoreParams& p, int page, int slot, int h) {
    return p.score + ((long long)page * p.Hkv + h) * p.page_size + slot;
}

}  // namespace
#endif

}  // namespace attn
