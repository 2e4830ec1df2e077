// Eviction from a paged cache by accumulated attention weight: which tokens stay (attn_kv_select_paged), and their move to the
// slots that remain (attn_kv_compact_paged).
//
// Selection, one block per (sequence, kv head). Of the tokens between the first `sinks` and the last `recent` the m with the
// largest scores stay, ties to the earlier token. Scores become unsigned keys of the same order, held in shared memory; the m-th largest
// is found by digits of 11, 11 and 10 bits from the top: a histogram of the keys that share the digits found so far, the digit in
// which the count from above passes m. Then a warp's vote per 32 tokens says which stay, in one word. Of the words' counts one
// scan over the block numbers the holes and the tails: a kept token below end = budget - recent stays in its slot, the holes there take in
// order the kept tokens behind it. Bounded by latency and instructions: the loads, a dozen block-wide steps, and per 32 tokens about as many
// instructions. (With neighbouring tokens numbered by one thread each: 64 x 8 rows of 4100-4352 tokens 23 us, 16 x 8 of up to
// 32768 29 us; with keys in registers, four digits of 8 bits, and a numbering per 1024 tokens about 100 us.)
//
// Compaction: row kept[j] -> j with kept[j] >= j. A block lists the slots that get another row, in ascending order, with the
// cache rows of both, and moves them in runs: it loads the rows of a run, then stores them. Every row that it reads later belongs to a slot
// behind the run, and so lies there too: nothing is overwritten that is still needed, and only the loads and the stores of one run
// need a barrier between them. Blocks share nothing: one has a (sequence, kv head) and some 16-byte columns of its rows, fewer columns
// where there are few sequences. Bounded by the memory. (Walking all slots instead of a list took 150 us more in that case.)
#include "attn.h"
#include "kernels.cuh"
#include "launch.cuh"
#include "ptx.cuh"

#include <math.h>
#include <string.h>

namespace attn {
namespace {

constexpr int kLongThreads = 1024;   // selection from more tokens than the shared memory holds
constexpr int kPairs = 4096;         // there: holes paired with tokens at a time
constexpr int kSelectKeys = 49152;   // tokens of a row whose keys the shared memory holds: 210 KB with 12 bytes per 32, and 9 KB besides

struct EvictParams {
    float* score;           // [num_pages, Hkv, page_size]
    uint8_t* cache[2];      // [num_pages, page_size, Hkv, row_bytes]
    const int* page_table;  // [B, max_pages]
    const int* seqlens;     // [B]: cached tokens (selection), tokens that stay (compaction)
    int* kept;              // [B, Hkv, budget]
    int* new_seqlens;       // [B]
    int B, Hkv, page_size, max_pages, num_pages, budget, sinks, recent;
    int most;                // selection: tokens to choose from at most, rounded up to a multiple of 32
    int row_bytes, columns;  // of one kv head; 16-byte columns of K and V that a block moves
    unsigned int ps_magic;  // tok / page_size by multiplication, as in DecodeParams
    int ps_shift;
    int* status;
};

__device__ __forceinline__ int evict_page(const EvictParams& p, int tok, int& slot) {
    const int q = p.ps_magic ? (int)(__umulhi((unsigned)tok, p.ps_magic) >> p.ps_shift) : tok;
    slot = tok - q * p.page_size;
    return q;
}

// Sum over the block before each warp (exclusive) and in all, from the warps' sums; every thread calls it.
__device__ __forceinline__ int warps_before(int mine, int* sums, int& total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __syncthreads();
    if (lane == 0) sums[warp] = mine;
    __syncthreads();
    const int x = lane < (int)(blockDim.x >> 5) ? sums[lane] : 0;
    int upto = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
    }
    total = __shfl_sync(0xffffffffu, upto, 31);
    return __shfl_sync(0xffffffffu, upto - x, warp);
}

// Order of scores as unsigned numbers, 0 for none: NaN above infinity, -0 as 0.
__device__ __forceinline__ uint32_t score_key(float x) {
    if (isnan(x)) return 0xFFFFFFFFu;
    const uint32_t u = __float_as_uint(x + 0.0f);  // (-0 + 0 = 0)
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// What every selection does for a row: lengths, and the tokens that always stay. False: nothing is left to choose.
struct SelectRow {
    int h, len, end, stop, m, n;  // m of n tokens from `sinks` on stay, m < n
    int* kept;
    const int* pt;
};
__device__ __forceinline__ bool select_row(const EvictParams& p, SelectRow& s) {
    const int b = (int)(blockIdx.x / (unsigned)p.Hkv), K = p.budget, tid = threadIdx.x, nt = blockDim.x;
    s.h = (int)(blockIdx.x % (unsigned)p.Hkv);
    s.len = __ldg(p.seqlens + b);
    s.kept = p.kept + (long long)blockIdx.x * K;
    s.pt = p.page_table + (long long)b * p.max_pages;
    const bool bad = s.len < 0 || s.len > (long long)p.max_pages * p.page_size;
    if (tid == 0) {
        if (bad) atomicCAS(p.status, 0, kDevBadIndex);
        if (s.h == 0) p.new_seqlens[b] = bad ? s.len : min(s.len, K);
    }
    if (bad || s.len <= K) {
        for (int j = tid; j < K; j += nt) s.kept[j] = !bad && j < s.len ? j : -1;
        return false;
    }
    s.end = K - p.recent, s.stop = s.len - p.recent;
    for (int j = tid; j < p.sinks; j += nt) s.kept[j] = j;
    for (int j = tid; j < p.recent; j += nt) s.kept[s.end + j] = s.stop + j;
    s.m = s.end - p.sinks, s.n = s.stop - p.sinks;
    return s.m > 0;
}

// Key of token sinks + i.
__device__ __forceinline__ uint32_t key_of(const EvictParams& p, const SelectRow& s, int i) {
    int slot;
    const int page = __ldg(s.pt + evict_page(p, p.sinks + i, slot));
    if (page < 0 || page >= p.num_pages) {
        atomicCAS(p.status, 0, kDevBadIndex);
        return 0;
    }
    return score_key(__ldg(p.score + ((long long)page * p.Hkv + s.h) * p.page_size + slot));
}

// The digit in which the count of the histogram from the top passes `left`, how many of that digit are then left, and of how many. Every
// thread calls it; scratch: 35 words.
template <int kBins>
__device__ __forceinline__ void find_digit(const int* hist, int* scratch, int& digit, int& left, int& of) {
    constexpr int kGroup = kBins / 32, kPer = kGroup / 32;  // bins of a group, of its lanes
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    for (int g = warp; g < 32; g += warps) {  // group g from the top
        int c = 0;
#pragma unroll
        for (int x = 0; x < kPer; ++x) c += hist[kBins - (g + 1) * kGroup + 32 * x + lane];
        c = __reduce_add_sync(0xffffffffu, c);
        if (lane == 0) scratch[g] = c;
    }
    __syncthreads();
    if (warp == 0) {
        auto scan = [&](int x) {  // inclusive
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            return x;
        };
        const int c = scratch[lane], upto = scan(c);
        const int g = __ffs(__ballot_sync(0xffffffffu, upto >= left)) - 1;
        int above = __shfl_sync(0xffffffffu, upto - c, g);
        const int top = kBins - g * kGroup - 1;  // lane l has its bins top - l kPer, ...
        int mine[kPer], sum = 0;
#pragma unroll
        for (int x = 0; x < kPer; ++x) sum += mine[x] = hist[top - lane * kPer - x];
        above += scan(sum) - sum;
#pragma unroll
        for (int x = 0; x < kPer; ++x) {
            if (above < left && above + mine[x] >= left) scratch[32] = top - lane * kPer - x, scratch[33] = left - above, scratch[34] = mine[x];
            above += mine[x];
        }
    }
    __syncthreads();
    digit = scratch[32];
    left = scratch[33];
    of = scratch[34];
}

// Exclusive sum over the block's threads; every thread calls it.
template <typename Sum>
__device__ __forceinline__ Sum block_before(Sum mine, Sum* sums) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    Sum upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Sum y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    Sum x = lane < warp && lane < warps ? sums[lane] : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return upto - mine + x;
}

// QUADS: page_size is a multiple of 4 and score 16-byte aligned.
template <bool QUADS>
__global__ void __launch_bounds__(1024) select_kernel(const __grid_constant__ EvictParams p) {
    grid_dependents_launch();
    extern __shared__ __align__(16) uint32_t keys[];
    __shared__ int hist[2048], scratch[35];
    __shared__ unsigned long long sums[32];
    // behind the keys, per 32 tokens: holes and tails before them, which of them stay
    uint2* ahead = reinterpret_cast<uint2*>(keys + p.most);
    uint32_t* bits = reinterpret_cast<uint32_t*>(ahead + p.most / 32);
    static_assert(2048 >= kSelectKeys / 32, "the histogram also takes the equals among 32 tokens each");
    const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5, warps = nt >> 5;
    auto clear = [&]() {
        for (int i = tid; i < 2048; i += nt) hist[i] = 0;
    };
    clear();
    SelectRow s;
    if (!select_row(p, s)) return;
    const int m = s.m, n = s.n;
    __syncthreads();
    if constexpr (QUADS) {
        // tokens 4 q .. 4 q + 3, on one page
#pragma unroll 8
        for (int q = (p.sinks >> 2) + tid; 4 * q < s.stop; q += nt) {
            int slot;
            const int page = __ldg(s.pt + evict_page(p, 4 * q, slot));
            const bool bad = page < 0 || page >= p.num_pages;
            float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (!bad) x = __ldg(reinterpret_cast<const float4*>(p.score + ((long long)page * p.Hkv + s.h) * p.page_size + slot));
            const float f[4] = {x.x, x.y, x.z, x.w};
            if (bad) atomicCAS(p.status, 0, kDevBadIndex);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = 4 * q + e - p.sinks;
                if (i < 0 || i >= n) continue;
                const uint32_t k = bad ? 0 : score_key(f[e]);
                keys[i] = k;
                atomicAdd(&hist[k >> 21], 1);
            }
        }
    } else {
#pragma unroll 4
        for (int i = tid; i < n; i += nt) {
            const uint32_t k = key_of(p, s, i);
            keys[i] = k;
            atomicAdd(&hist[k >> 21], 1);
        }
    }
    __syncthreads();
    // the m-th largest key, and how many of its equals stay
    int digit, left = m, of;
    find_digit<2048>(hist, scratch, digit, left, of);
    uint32_t found = (uint32_t)digit << 21;
    clear();
    __syncthreads();
    // f(word, its lane's key, is there one) for 32 tokens each, loaded ahead of it
    const int words = (n + 31) >> 5;
    auto each_word = [&](int first, auto f) {
        constexpr int kAhead = 8;
        for (int w = first + warp; w < words; w += kAhead * warps) {
            uint32_t k[kAhead];
#pragma unroll
            for (int x = 0; x < kAhead; ++x) {
                const int i = 32 * (w + x * warps) + lane;
                k[x] = i < n ? keys[i] : 0;
            }
#pragma unroll
            for (int x = 0; x < kAhead; ++x)
                if (w + x * warps < words) f(w + x * warps, k[x], 32 * (w + x * warps) + lane < n);
        }
    };
    each_word(0, [&](int, uint32_t key, bool in) {
        if (in && (key ^ found) >> 21 == 0) atomicAdd(&hist[key >> 10 & 2047], 1);
    });
    __syncthreads();
    find_digit<2048>(hist, scratch, digit, left, of);
    found |= (uint32_t)digit << 10;
    clear();
    __syncthreads();
    each_word(0, [&](int, uint32_t key, bool in) {
        if (in && (key ^ found) >> 10 == 0) atomicAdd(&hist[key & 1023], 1);
    });
    __syncthreads();
    find_digit<1024>(hist, scratch, digit, left, of);
    found |= (uint32_t)digit;

    // which of 32 tokens stay; when not all equals do, those apart
    const bool ties = left < of;
    each_word(0, [&](int w, uint32_t key, bool in) {
        const uint32_t stay = __ballot_sync(0xffffffffu, in && (ties ? key > found : key >= found));
        if (lane == 0) bits[w] = stay;
        if (ties) {
            const uint32_t equal = __ballot_sync(0xffffffffu, in && key == found);
            if (lane == 0) hist[w] = (int)equal;
        }
    });
    __syncthreads();
    // neighbouring words of this thread
    const int each = (words + nt - 1) / nt, w0 = min(words, tid * each), w1 = min(words, w0 + each);
    if (ties) {
        int equals = 0;
        for (int w = w0; w < w1; ++w) equals += __popc(hist[w]);
        int room = left - (int)block_before<unsigned long long>(equals, sums);  // equals that may stay from here on
        for (int w = w0; w < w1 && room > 0; ++w) {
            uint32_t equal = (uint32_t)hist[w];
            for (; equal && room > 0; equal &= equal - 1, --room) bits[w] |= equal & -equal;
        }
        __syncthreads();
    }
    // bits of word w that are tokens below m; behind them
    auto below_m = [&](int w) { return 32 * w + 32 <= m ? ~0u : 32 * w >= m ? 0u : (1u << (m - 32 * w)) - 1; };
    unsigned holes = 0, tails = 0;
    for (int w = w0; w < w1; ++w) holes += __popc(~bits[w] & below_m(w)), tails += __popc(bits[w] & ~below_m(w));
    const unsigned long long before = block_before(((unsigned long long)tails << 32) + holes, sums);
    uint2 upto = make_uint2((unsigned)before, (unsigned)(before >> 32));
    for (int w = w0; w < w1; ++w) {
        ahead[w] = upto;
        upto.x += __popc(~bits[w] & below_m(w)), upto.y += __popc(bits[w] & ~below_m(w));
    }
    __syncthreads();
    // (the keys are done with) the tails in their order, then every slot
    const uint32_t lower = (1u << lane) - 1;
#pragma unroll 4
    for (int w = (m >> 5) + warp; w < words; w += warps) {
        const uint32_t tail = bits[w] & ~below_m(w);
        if (tail >> lane & 1) keys[ahead[w].y + __popc(tail & lower)] = (uint32_t)(32 * w + lane);
    }
    __syncthreads();
#pragma unroll 4
    for (int w = warp; 32 * w < m; w += warps) {
        const uint32_t hole = ~bits[w] & below_m(w);
        const int i = 32 * w + lane;
        if (i < m) s.kept[p.sinks + i] = p.sinks + (hole >> lane & 1 ? (int)keys[ahead[w].x + __popc(hole & lower)] : i);
    }
}

// The same from more tokens: the keys are read again for every step, and the tokens numbered in rounds of one per thread.
__global__ void __launch_bounds__(kLongThreads, 1) select_long_kernel(const __grid_constant__ EvictParams p) {
    grid_dependents_launch();
    __shared__ int hist[2048], scratch[35], sums[32], place[kPairs];
    const int tid = threadIdx.x, lane = tid & 31;
    SelectRow s;
    if (!select_row(p, s)) return;
    const int m = s.m, n = s.n;
    uint32_t found = 0;
    int left = m;
    for (int shift = 21;; shift = shift == 21 ? 10 : 0) {  // digits of 11, 11 and 10 bits
        for (int i = tid; i < 2048; i += kLongThreads) hist[i] = 0;
        __syncthreads();
        for (int i = tid; i < n; i += kLongThreads) {
            const uint32_t k = key_of(p, s, i);
            if (shift == 21 || (k ^ found) >> (shift == 10 ? 21 : 10) == 0) atomicAdd(&hist[shift > 0 ? k >> shift & 2047 : k & 1023], 1);
        }
        __syncthreads();
        int digit, of;
        if (shift > 0)
            find_digit<2048>(hist, scratch, digit, left, of);
        else
            find_digit<1024>(hist, scratch, digit, left, of);
        found |= (uint32_t)digit << shift;
        if (shift == 0) break;
        __syncthreads();
    }
    // holes in turn, kPairs at a time
    const uint32_t below = (1u << lane) - 1;
    for (int first = 0, holes;; first += kPairs) {
        int equals = 0, tails = 0;
        holes = 0;
        for (int base = 0; base < n; base += kLongThreads) {
            const int i = base + tid;
            const uint32_t key = i < n ? key_of(p, s, i) : 0;
            const bool equal = i < n && key == found;
            int total;
            const uint32_t be = __ballot_sync(0xffffffffu, equal);
            const int number = equals + warps_before(__popc(be), sums, total) + __popc(be & below);
            equals += total;
            const bool stay = i < n && (key > found || (equal && number < left));
            const bool hole = i < m && !stay, tail = i >= m && stay;
            if (i < m && stay && first == 0) s.kept[p.sinks + i] = p.sinks + i;
            const uint32_t bh = __ballot_sync(0xffffffffu, hole), bt = __ballot_sync(0xffffffffu, tail);
            const int before = warps_before(__popc(bh) | __popc(bt) << 16, sums, total);
            const int nh = holes + (before & 0xFFFF) + __popc(bh & below) - first, ntl = tails + (before >> 16) + __popc(bt & below) - first;
            holes += total & 0xFFFF;
            tails += total >> 16;
            // (all holes come before the first token behind them, but for those of the same round)
            if (hole && nh >= 0 && nh < kPairs) place[nh] = p.sinks + i;
            __syncthreads();
            if (tail && ntl >= 0 && ntl < kPairs) s.kept[place[ntl]] = p.sinks + i;
        }
        if (holes <= first + kPairs) break;
        __syncthreads();
    }
}

// 16-byte columns of K and V rows, one per lane; kRun rows per thread and run.
constexpr int kCompactThreads = 512, kRun = 8, kMoves = 4096, kLook = kMoves / kCompactThreads;

__global__ void __launch_bounds__(kCompactThreads, 2) compact_kernel(const __grid_constant__ EvictParams p) {
    __shared__ int src[kMoves], dst[kMoves];  // cache rows of the moves listed
    __shared__ unsigned sums[32];
    __shared__ int total;
    grid_dependency_wait();                             // (launched as a programmatic dependent of what is before it)
    const int b = (int)(blockIdx.x / (unsigned)p.Hkv), h = (int)(blockIdx.x % (unsigned)p.Hkv);
    const int n = min(__ldg(p.seqlens + b), p.budget), limit = p.max_pages * p.page_size;
    const int* kept = p.kept + (long long)blockIdx.x * p.budget;
    const int* pt = p.page_table + (long long)b * p.max_pages;
    const int each = p.row_bytes / 16, tid = threadIdx.x;  // columns of K, and of V
    const int lanes = p.columns, col = blockIdx.y * lanes + tid % lanes;
    const int rows = kCompactThreads / lanes, row0 = tid / lanes;
    const bool active = row0 < rows && col < 2 * each;
    uint8_t* cache = p.cache[col >= each] + (long long)h * p.row_bytes + 16 * (col >= each ? col - each : col);
    const long long row_bytes = (long long)p.Hkv * p.row_bytes;
    auto row_of = [&](int tok) {  // -1: a page out of range
        int slot;
        const int page = __ldg(pt + evict_page(p, tok, slot));
        if (page >= 0 && page < p.num_pages) return page * p.page_size + slot;
        atomicCAS(p.status, 0, kDevBadIndex);
        return -1;
    };
    auto sum_of = [&](int row) {  // the score of a cache row
        const int page = row / p.page_size;
        return p.score + ((long long)page * p.Hkv + h) * p.page_size + (row - page * p.page_size);
    };
    for (int j0 = 0; j0 < n; j0 += kMoves) {
        // the slots from j0 on that get another row; neighbouring ones of this thread
        const int first = j0 + tid * kLook;
        int tok[kLook];
        unsigned moves = 0;
#pragma unroll
        for (int x = 0; x < kLook; ++x) tok[x] = first + x < n ? __ldg(kept + first + x) : -1;
#pragma unroll
        for (int x = 0; x < kLook; ++x) {
            if (tok[x] != -1 && (tok[x] < first + x || tok[x] >= limit)) {
                atomicCAS(p.status, 0, kDevBadIndex);
                tok[x] = -1;
            }
            moves += tok[x] > first + x;
        }
        unsigned at = block_before(moves, sums);
        if (tid == kCompactThreads - 1) total = (int)(at + moves);
#pragma unroll
        for (int x = 0; x < kLook; ++x)
            if (tok[x] > first + x) src[at] = tok[x], dst[at++] = first + x;
        __syncthreads();
        const int listed = total;
        for (int i = tid; i < listed; i += kCompactThreads) {
            const int from = row_of(src[i]), to = row_of(dst[i]);
            src[i] = to < 0 ? -1 : from, dst[i] = to;
        }
        __syncthreads();
        for (int i0 = 0; i0 < listed; i0 += rows * kRun) {
            uint4 v[kRun];
#pragma unroll
            for (int x = 0; x < kRun; ++x) {
                const int i = i0 + x * rows + row0;
                if (active && i < listed && src[i] >= 0) v[x] = *reinterpret_cast<const uint4*>(cache + src[i] * row_bytes);
            }
            // (the scores with the first columns, a thread per row)
            const int run = min(rows * kRun, listed - i0);
            constexpr int kSums = kRun / 2;  // (two columns at least: no more rows than that for a thread)
            float sum[kSums];
            auto scores = [&](auto f) {
                if (!p.score || blockIdx.y != 0) return;
#pragma unroll
                for (int x = 0; x < kSums; ++x) {
                    const int i = i0 + x * kCompactThreads + tid;
                    if (x * kCompactThreads + tid < run && src[i] >= 0) f(sum[x], i);
                }
            };
            scores([&](float& f, int i) { f = *sum_of(src[i]); });
            __syncthreads();  // the run is read before any of its slots is written
#pragma unroll
            for (int x = 0; x < kRun; ++x) {
                const int i = i0 + x * rows + row0;
                if (active && i < listed && src[i] >= 0) *reinterpret_cast<uint4*>(cache + dst[i] * row_bytes) = v[x];
            }
            scores([&](float& f, int i) { *sum_of(dst[i]) = f; });
        }
        __syncthreads();  // the list is done with
    }
}

bool multiple(const void* p, long long bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

attn_status_t check_sizes(EvictParams& p, int page_size, int B, int Hkv, int max_pages, int num_pages, int budget) {
    if (B < 0 || B > 65535 || Hkv <= 0 || Hkv > 65535 || page_size <= 0 || max_pages <= 0 || num_pages <= 0 || budget <= 0 ||
        (long long)num_pages * page_size > INT32_MAX || (long long)max_pages * page_size > INT32_MAX / 2 ||
        (long long)B * Hkv > INT32_MAX)
        return ATTN_ERR_BAD_SHAPE;
    p.B = B, p.Hkv = Hkv, p.page_size = page_size, p.max_pages = max_pages, p.num_pages = num_pages, p.budget = budget;
    if (page_size > 1) {  // tok / page_size for tok < 2^31: multiplier ceil(2^(31+k) / page_size), k = ceil(log2 page_size)
        int k = 0;
        while ((1LL << k) < page_size) ++k;
        p.ps_magic = (unsigned)(((1ULL << (31 + k)) + (unsigned long long)page_size - 1) / (unsigned long long)page_size);
        p.ps_shift = k - 1;
    }
    return ATTN_OK;
}

}  // namespace
}  // namespace attn

extern "C" attn_status_t attn_kv_select_paged(const float* score, const int* page_table, const int* seqlens, int* kept, int* new_seqlens,
                                              int page_size, int B, int Hkv, int max_pages_per_seq, int num_pages, int budget, int sinks,
                                              int recent, void* stream) {
    using namespace attn;
    if (!score || !page_table || !seqlens || !kept || !new_seqlens) return ATTN_ERR_NULL_PTR;
    EvictParams p;
    memset(&p, 0, sizeof p);
    attn_status_t st = check_sizes(p, page_size, B, Hkv, max_pages_per_seq, num_pages, budget);
    if (st != ATTN_OK) return st;
    if (sinks < 0 || recent < 0 || (long long)sinks + recent > budget) return ATTN_ERR_BAD_SHAPE;
    if (new_seqlens == seqlens) return ATTN_ERR_BAD_ARG;
    if (!multiple(score, 4) || !multiple(page_table, 4) || !multiple(seqlens, 4) || !multiple(kept, 4) || !multiple(new_seqlens, 4))
        return ATTN_ERR_ALIGN;
    if (B == 0) return ATTN_OK;
    int num_sms = 0;
    if ((st = current_device_info(&p.status, &num_sms)) != ATTN_OK) return st;
    p.score = const_cast<float*>(score);
    p.page_table = page_table;
    p.seqlens = seqlens;
    p.kept = kept;
    p.new_seqlens = new_seqlens;
    p.sinks = sinks, p.recent = recent;
    // tokens to choose from at most
    const long long most = (long long)max_pages_per_seq * page_size - sinks - recent;
    const dim3 grid((unsigned)(B * Hkv));
    cudaError_t e;
    if (most > kSelectKeys) {
        e = launch_kernel(select_long_kernel, grid, kLongThreads, 0, static_cast<cudaStream_t>(stream), {}, p);
    } else {
        // a thread for 8 tokens: the blocks of many short rows share the SMs, long rows have all threads of one
        unsigned threads = 128;
        while (threads < 1024 && threads * 8 < most) threads *= 2;
        static std::atomic<bool> attr_set[2][kMaxAttrDevices];
        const bool quads = page_size % 4 == 0 && multiple(score, 16);
        const auto kernel = quads ? select_kernel<true> : select_kernel<false>;
        p.most = most > 0 ? (int)((most + 31) / 32 * 32) : 0;
        e = ensure_smem_attr(kernel, kSelectKeys / 32 * 140, attr_set[quads]);
        if (e == cudaSuccess) e = launch_kernel(kernel, grid, threads, (size_t)p.most / 32 * 140, static_cast<cudaStream_t>(stream), {}, p);
    }
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

extern "C" attn_status_t attn_kv_compact_paged(void* k_cache, void* v_cache, float* score, const int* kept, const int* new_seqlens,
                                               const int* page_table, int page_size, int B, int Hkv, int d, int max_pages_per_seq,
                                               int num_pages, int budget, int kv_format, void* stream) {
    using namespace attn;
    if (!k_cache || !v_cache || !kept || !new_seqlens || !page_table) return ATTN_ERR_NULL_PTR;
    if (kv_format != ATTN_FP8_E4M3 && kv_format != ATTN_FP8_E5M2 && kv_format != ATTN_KV_BF16) return ATTN_ERR_BAD_ARG;
    EvictParams p;
    memset(&p, 0, sizeof p);
    attn_status_t st = check_sizes(p, page_size, B, Hkv, max_pages_per_seq, num_pages, budget);
    if (st != ATTN_OK) return st;
    if (d <= 0 || d % 16 != 0 || d > 256) return ATTN_ERR_BAD_SHAPE;
    if (!multiple(k_cache, 16) || !multiple(v_cache, 16) || !multiple(score, 4) || !multiple(kept, 4) || !multiple(new_seqlens, 4) ||
        !multiple(page_table, 4))
        return ATTN_ERR_ALIGN;
    if (B == 0) return ATTN_OK;
    int num_sms = 0;
    if ((st = current_device_info(&p.status, &num_sms)) != ATTN_OK) return st;
    p.cache[0] = static_cast<uint8_t*>(k_cache), p.cache[1] = static_cast<uint8_t*>(v_cache);
    p.score = score;
    p.kept = const_cast<int*>(kept);
    p.seqlens = new_seqlens;
    p.page_table = page_table;
    p.row_bytes = kv_format == ATTN_KV_BF16 ? 2 * d : d;
    // All columns of a row in one block; fewer, but whole 32-byte sectors, until there are three blocks for every SM.
    const int all = p.row_bytes / 8;
    p.columns = all;
    while (p.columns > 2 && (long long)B * Hkv * ((all + p.columns - 1) / p.columns) * 2 <= 3LL * num_sms) p.columns = (p.columns + 3) / 4 * 2;
    const unsigned parts = (unsigned)((all + p.columns - 1) / p.columns);
    LaunchMode mode;
    mode.dependent = true;
    const cudaError_t e = launch_kernel(compact_kernel, dim3((unsigned)(B * Hkv), parts), kCompactThreads, 0, static_cast<cudaStream_t>(stream), mode, p);
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}
