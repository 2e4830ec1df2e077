// Interface between attn_api.cu and attn_tree.cu: attention of drafted tokens over a paged cache.
#pragma once

#include "kernels.cuh"

namespace attn {

struct TreeParams {
    const __nv_bfloat16* q;  // [T, Hq, d]
    const void* k_cache;     // [num_pages, page_size, Hkv, d], bf16 or 8-bit codes
    const void* v_cache;
    const int* page_table;   // [B, max_pages]
    const int* seqlens;      // [B], the drafted tokens included
    const int* cu_seqlens;   // [B + 1] or nullptr: T / B rows each
    const unsigned long long* mask;  // [T, mask_words] or nullptr: a chain
    int mask_words;
    __nv_bfloat16* o;        // [T, Hq, d]
    float* lse;              // [T, Hq]
    float* ws_o;             // [T, Hq, max_splits, d] partial outputs
    float* ws_lse;           // [T, Hq, max_splits]
    int* ws_chunk;           // tokens per split in use, when slots > 0
    int B, T, max_q, Hq, Hkv, G, page_size, max_pages, num_pages;
    int chunk, max_splits;   // tokens per split (a multiple of 64), splits of the longest sequence
    int slots;               // > 0: chunk is the least one; the blocks choose it by the lengths, for so many at once
    int tiles;               // 128-row tiles, not 16-row products
    int cluster;             // > 0: max_splits blocks of a cluster hold the splits of one group and join them themselves
    int groups;              // row groups per kv head (rows: drafted token x query head of the kv head)
    // Work order (tree_grid): grid rows y < full_rows list the splits of sequence y before its last one, the
    // rows after them the last split of every sequence, in decreasing length when ranked. full_rows < 0:
    // row y holds all splits of sequence y. slots > 0: one row, see tree_fit.
    int full_rows, ranked, num_sms;
    // q is multiplied by q_sign (-1, 0, 1) and the scores by |scale|, so that masking and maxima
    // work on scores that grow with q.k for every finite scale (scale 0: q_sign 0, factor 1)
    float q_sign, scale, scale_log2;  // |scale| (key descale included), times log2(e)
    float v_descale, rescale_thr;
    unsigned int ps_magic;   // tok / page_size by multiplication, as in DecodeParams
    int ps_shift;
    int box_rows;            // rows of a box of the maps (64 or 16, dividing the page size), 1: no maps
    int* status;
    unsigned long long watchdog_ns;
};

// 2-D maps over the caches viewed as [num_pages * page_size, Hkv * d], box box_rows rows of 128 bytes
// (64 for 8-bit d = 64).
struct TreeTmaps {
    CUtensorMap k, v;
};

// kv_format: ATTN_KV_BF16, ATTN_FP8_E4M3, ATTN_FP8_E5M2; d 64 or 128.
// tm: the maps when p.tiles and box_rows > 1, else unused.
cudaError_t launch_attn_tree(const TreeParams& p, const TreeTmaps& tm, int d, int kv_format, cudaStream_t stream);
cudaError_t launch_tree_tiles(const TreeParams& p, const TreeTmaps& tm, int d, int kv_format, cudaStream_t stream);

// Sequences up to which the blocks choose the split size by the lengths (two per lane of a warp).
constexpr int kTreeFitSeqs = 64;

// 128-row tiles, or 16-row products? The latter up to 16 rows per kv head, where the cache is read once either way.
// Up to 32 rows they read it twice (once through the L2), but start sooner and need no padding: with d = 64 they are
// faster while an SM has few tokens, by the capacity of the page table (the lengths are not known here). The tiles
// catch up later over codes (they widen V) and where no box divides the pages (one warp copies row by row). Measured,
// 17 to 32 rows, 1 to 64 sequences x 1 to 8 kv heads, full and half-full tables, 16-row products / tiles: pages of 16, codes,
// 850 tokens per SM 17.2 / 18.8 us, 1730 23.9 / 24.2, 3400 38.1 / 37.6, 6900 63.5 / 55.2; bf16 430 13.8 / 15.2, 860 17.0 / 17.3, 1730
// 24.3 / 21.9; pages of 7, codes 3400 36.6 / 37.8, 6900 65.9 / 62.9, bf16 1730 24.0 / 24.3, 3450 40.5 / 39.1 (522 points: 0.3% behind the
// faster one on average, 9% at most: full tables a little below a limit, half-full ones a little above). With more
// sequences the split size does not follow the lengths, and the 16-row products keep their lead only while a sequence and
// kv head have an SM for themselves: 100 sequences of U[100, 1000] x 1 kv head 13.4 / 17.8, 200 x 1 21.2 / 17.1, 200 x 8 102 / 85
// (273 points: 3% behind the faster one on average; 100 sequences of U[20, 100] x 8 24 / 31). With d = 128: 8-bit codes 64 of up
// to 1000 x 8 46 / 34, bf16 48 / 40.
inline bool tree_takes_tiles(long long rows, int d, bool f8, int page_size, int B, int Hkv, long long max_len, int num_sms) {
    if (rows <= 16) return false;
    if (d != 64 || rows > 32) return true;
    const bool boxes = page_size % 16 == 0;
    const long long limit = f8 ? (boxes ? 3400 : 8000) : (boxes ? 1500 : 3400);  // tokens per SM
    return (long long)B * Hkv * max_len > limit * num_sms || (B > kTreeFitSeqs && (long long)B * Hkv > num_sms);
}

// Grid of a split kernel; sets the work order. The last splits are shorter in general: started after all
// others, the longest first, they fill the SMs that the last full-length ones leave idle.
inline dim3 tree_grid(TreeParams& p) {
    const long long HG = (long long)p.Hkv * p.groups;
    if (p.cluster > 0) {
        p.full_rows = -1;
        p.ranked = 0;
        return dim3((unsigned)(p.max_splits * HG), (unsigned)p.B);
    }
    if (p.slots > 0) {  // (blocks without work cost a microsecond or two each, so there are few more than fit at once)
        p.full_rows = 0;
        p.ranked = 0;
        return dim3((unsigned)(p.slots + p.slots / 2));
    }
    const long long X = (p.max_splits > 1 ? p.max_splits - 1 : 1) * HG;
    const long long full = p.max_splits > 1 ? p.B : 0, part = ((long long)p.B * HG + X - 1) / X;
    if (full + part <= 65535) {
        p.full_rows = (int)full;
        // Each block of that part ranks the lengths, which costs it about a microsecond: not when all
        // blocks start at once anyway.
        p.ranked = p.B <= 256 && p.B > 1 && X * (full + part) > 2LL * p.num_sms;
        return dim3((unsigned)X, (unsigned)(full + part));
    }
    p.full_rows = -1;
    p.ranked = 0;
    return dim3((unsigned)(p.max_splits * HG), (unsigned)p.B);
}

// Blocks of the split kernels that share an SM. (64 8-bit codes, up to 8 rows, five, not four: 64 sequences of U[100, 1000]
// 17.0 us, not 20.1, of U[1K, 32K] 197, not 206; with up to 16 rows the registers do not suffice: 242, not 218.)
constexpr int tree_small_blocks(int d, bool f8, int rows) { return d == 128 ? 3 : f8 && rows <= 8 ? 5 : 4; }
constexpr int kTreeTileBlocks = 2;

// Largest cluster that every GPU of this kind can place.
constexpr int kTreeCluster = 8;

// Sets tiles, chunk, max_splits, slots and cluster of p (B, Hkv, G, max_q, max_pages, page_size and num_sms given).
void tree_plan(TreeParams& p, int d, bool f8, int num_splits);

}  // namespace attn
