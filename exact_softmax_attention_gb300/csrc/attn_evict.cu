// Eviction from a paged cache by accumulated attention weight: which tokens stay (attn_kv_select_paged), and their move to the
// slots that remain (attn_kv_compact_paged).
//
// Selection, one block or cluster of blocks per (sequence, kv head). Of the tokens between the first `sinks` and the last `recent` the m
// with the largest scores stay, ties to the earlier token. Scores become unsigned keys of the same order, held in shared memory; the m-th
// largest is found by digits of 11, 11 and 10 bits from the top: a histogram of the keys that share the digits found so far, the digit
// in which the count from above passes m. Then a lane looks at four neighbouring tokens, a warp at 128, and four votes mark the holes (tokens below
// m that go) and the tails (later ones that stay). One scan over the counts of 128 tokens each numbers the marks in token order, first the holes,
// then the tails, as many of either: hole k takes tail k. Bounded by latency and instructions: the loads, a dozen steps of the whole block,
// and about ten instructions per pass and 32 tokens. Several blocks share a row where rows are long and few: a block counts and marks its part,
// and the others read the counts in its shared memory. (One block for each row, votes on 32 tokens: 16 x 8 rows of up to 32768 tokens 25 us,
// 64 x 8 rows of 4100-4352 tokens 21 us; with keys in registers, four digits of 8 bits, and a numbering per 1024 tokens about 100 us.) Now, on new
// scores in a graph: 8 rows of 1000 tokens 6.6 us (a piece of code per digit instead of a loop: 7.2), 16 x 8 of U[2048, 32768] 20.5, 64 x 8 of
// U[4100, 4352] 18.2.
// Parts and their shared memory go by the page table's capacity, which the host knows, not by the lengths. What that costs in tables much wider than
// the sequences: 64 x 8 rows of 600-1000 tokens 8 us in a tight table, 10 in one of 8192 tokens, 19 in one of 32768, 206 in one of 131072 (four blocks
// a row, one on an SM), 21 in one of 524288, which select_long_kernel takes; 16 x 8 of 1100-4000 tokens 8.4, 7.1, 7.1, 50 and 13; 8 rows of 1000
// tokens 6.5, 11, 16, 15 and 6.
//
// Compaction: row kept[j] -> j with kept[j] >= j. A block lists the slots that get another row, in ascending order, with the
// cache rows of both, and moves them in runs: it loads the rows of a run, then stores them. Every row that it reads later belongs to a slot
// behind the run, and so lies there too: nothing is overwritten that is still needed, and only the loads and the stores of one run
// need a barrier between them. Blocks share nothing: one has a (sequence, kv head) and some 16-byte columns of its rows, fewer columns
// where there are few sequences. Measured on new scores: 16 x 8 x U[2048, 32768] tokens to 2048, bf16 heads of 128, 198011 rows of K and of V
// in and out, 43 us, 4.7 TB/s; 64 x 8 x U[4100, 4352] to 4096, e4m3, 196210 rows, 26.6 us, 3.8 TB/s: the memory, behind the chain list, pages, rows of each
// block, and nothing is loaded while a run is stored. (Walking all slots instead of a list took 150 us more in the first case; blocks of 256 threads,
// three or four on an SM, 47-55 and 29-31 us.)
#include "attn.h"
#include "kernels.cuh"
#include "launch.cuh"
#include "ptx.cuh"

#include <math.h>
#include <string.h>

namespace attn {
namespace {

constexpr int kLongThreads = 1024;  // selection from more tokens than the shared memories of a cluster hold
constexpr int kPairs = 4096;        // there: holes paired with tokens at a time
constexpr int kGroup = 128;         // tokens that a warp looks at
// Groups of a block's part: 512 bytes of keys and 20 of marks and counts each, 33 KB besides (25 KB for one part).
constexpr int kPartGroups = 352, kGroupBytes = kGroup * 4 + 20;
constexpr int kMaxParts = 8;

struct EvictParams {
    float* score;           // [num_pages, Hkv, page_size]
    uint8_t* cache[2];      // [num_pages, page_size, Hkv, row_bytes]
    const int* page_table;  // [B, max_pages]
    const int* seqlens;     // [B]: cached tokens (selection), tokens that stay (compaction)
    int* kept;              // [B, Hkv, budget]
    int* new_seqlens;       // [B]
    int B, Hkv, page_size, max_pages, num_pages, budget, sinks, recent;
    int groups;              // selection: groups of a block's part
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
__device__ __forceinline__ bool select_row(const EvictParams& p, SelectRow& s, int parts = 1, int part = 0) {
    const unsigned row = blockIdx.x / (unsigned)parts;
    const int b = (int)(row / (unsigned)p.Hkv), K = p.budget, tid = part * blockDim.x + threadIdx.x, nt = parts * blockDim.x;
    s.h = (int)(row % (unsigned)p.Hkv);
    s.len = p.seqlens[b];
    s.kept = p.kept + (long long)row * K;
    s.pt = p.page_table + (long long)b * p.max_pages;
    const bool bad = s.len < 0 || s.len > (long long)p.max_pages * p.page_size;
    if (tid == 0) {
        if (bad) atomicCAS(p.status, 0, kDevBadIndex);
        if (s.h == 0) p.new_seqlens[b] = bad ? s.len : min(s.len, K);
    }
    if (bad || s.len <= K) {
        for (unsigned j = tid; j < (unsigned)K; j += nt) s.kept[j] = !bad && j < (unsigned)s.len ? (int)j : -1;  // (j + nt may pass 2^31)
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
    const int page = s.pt[evict_page(p, p.sinks + i, slot)];
    if (page < 0 || page >= p.num_pages) {
        atomicCAS(p.status, 0, kDevBadIndex);
        return 0;
    }
    return score_key(p.score[((long long)page * p.Hkv + s.h) * p.page_size + slot]);
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

// The same place of the shared memory of another block of the cluster.
template <typename T>
__device__ __forceinline__ const T* of_part(const T* p, int rank) {
    const T* r;
    asm volatile("mapa.u64 %0, %1, %2;" : "=l"(r) : "l"(p), "r"(rank));
    return r;
}

// QUADS: page_size is a multiple of 4 and score 16-byte aligned. PARTS: blocks of the cluster that share a row.
template <bool QUADS, int PARTS>
__global__ void __launch_bounds__(1024) select_kernel(const __grid_constant__ EvictParams p) {
    extern __shared__ __align__(16) uint32_t keys[];
    __shared__ __align__(16) int counts[3][2048];
    __shared__ int merged[PARTS > 1 ? 2048 : 1], scratch[35], totals[2];  // totals of this part: equals, marks
    __shared__ unsigned sums[32];
    // behind the keys, per group: four votes (of the lanes' first, second, ... tokens), marks before it
    uint4* votes = reinterpret_cast<uint4*>(keys + p.groups * kGroup);
    unsigned* ahead = reinterpret_cast<unsigned*>(votes + p.groups);
    const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5, warps = nt >> 5;
    const int part = PARTS > 1 ? (int)(blockIdx.x % PARTS) : 0;
    auto all_sync = [&]() {
        if constexpr (PARTS > 1)
            asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
        else
            __syncthreads();
    };
    for (int i = tid; i < 3 * 2048 / 4; i += nt) reinterpret_cast<uint4*>(counts)[i] = make_uint4(0, 0, 0, 0);
    grid_dependents_launch();
    grid_dependency_wait();
    SelectRow s;
    if (!select_row(p, s, PARTS, part)) return;  // (the whole cluster)
    // places count from a multiple of four tokens on: tokens [off, off + n) of these, the first m of them below the row's end
    const int base = p.sinks & ~3, off = p.sinks - base, n = off + s.n, m = off + s.m;
    const int at0 = part * p.groups * kGroup, here = min(p.groups * kGroup, n - at0);  // this part's tokens (maybe none)
    const int groups = here > 0 ? (here + kGroup - 1) / kGroup : 0;
    __syncthreads();
    if constexpr (QUADS) {
#pragma unroll 4
        for (int q = tid; q < groups * (kGroup / 4); q += nt) {
            const int i = at0 + 4 * q;
            uint4 k = make_uint4(0, 0, 0, 0);
            if (i < n) {
                int slot;
                const int page = s.pt[evict_page(p, base + i, slot)];
                if (page >= 0 && page < p.num_pages) {
                    const float4 x = *reinterpret_cast<const float4*>(p.score + ((long long)page * p.Hkv + s.h) * p.page_size + slot);
                    k = make_uint4(score_key(x.x), score_key(x.y), score_key(x.z), score_key(x.w));
                } else {
                    atomicCAS(p.status, 0, kDevBadIndex);
                }
            }
            reinterpret_cast<uint4*>(keys)[q] = k;
        }
    } else {
#pragma unroll 4
        for (int x = tid; x < groups * kGroup; x += nt) {
            keys[x] = at0 + x >= off && at0 + x < n ? key_of(p, s, at0 + x - off) : 0;
        }
    }
    __syncthreads();
    // f(group, the lane's first place, its four keys, which of them are there), the keys loaded one group ahead of it. (Few groups
    // come to a warp: instructions are fetched for nearly every one, so nothing is unrolled that need not be.)
    auto each_group = [&](auto f) {
        uint4 next = make_uint4(0, 0, 0, 0);
        if (warp < groups) next = reinterpret_cast<const uint4*>(keys)[warp * 32 + lane];
#pragma unroll 1
        for (int g = warp; g < groups; g += warps) {
            const uint32_t key[4] = {next.x, next.y, next.z, next.w};
            if (g + warps < groups) next = reinterpret_cast<const uint4*>(keys)[(g + warps) * 32 + lane];
            const int i = at0 + g * kGroup + 4 * lane;
            // bits i .. i + 3 of [off, n)
            const uint32_t there = 15u << min(4, max(0, off - i)) & 15u >> min(4, max(0, i + 4 - n));
            f(g, i, key, there);
        }
    };
    // histogram d of all parts
    auto histogram = [&](int d) -> const int* {
        all_sync();
        if constexpr (PARTS > 1) {
            const int* from[PARTS];
#pragma unroll
            for (int x = 0; x < PARTS; ++x) from[x] = of_part(counts[d], x);
#pragma unroll 2
            for (int i = tid; i < 2048; i += nt) {
                int c = 0;
#pragma unroll
                for (int x = 0; x < PARTS; ++x) c += from[x][i];
                merged[i] = c;
            }
            __syncthreads();
            return merged;
        } else {
            return counts[d];
        }
    };
    // the m-th largest key, and how many of its equals stay
    int left = s.m, of;
    uint32_t found = 0, above = 0;  // the digits found, and their bits
#pragma unroll 1
    for (int d = 0; d < 3; ++d) {  // (a loop: the instructions are fetched once)
        const int shift = d == 0 ? 21 : d == 1 ? 10 : 0;
        const uint32_t mask = d < 2 ? 2047 : 1023;
        each_group([&](int, int, const uint32_t(&key)[4], uint32_t there) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (((key[e] ^ found) & above) == 0 && (there >> e & 1)) atomicAdd(&counts[d][key[e] >> shift & mask], 1);
        });
        int digit;
        find_digit<2048>(histogram(d), scratch, digit, left, of);
        found |= (uint32_t)digit << shift;
        above |= mask << shift;
    }

    // counts of the groups (in ahead) to the counts before them; total[which] is the part's. Returns those of the parts before.
    auto number = [&](int which) {
        __syncthreads();
        const int each = (groups + nt - 1) / nt, g0 = min(groups, tid * each), g1 = min(groups, g0 + each);
        unsigned c = 0;
        for (int g = g0; g < g1; ++g) c += ahead[g];
        unsigned upto = block_before(c, sums);
        if (tid == nt - 1) totals[which] = (int)(upto + c);
        for (int g = g0; g < g1; ++g) {
            const unsigned x = ahead[g];
            ahead[g] = upto;
            upto += x;
        }
        all_sync();
        unsigned before = 0;
        if constexpr (PARTS > 1)
#pragma unroll
            for (int x = 0; x < PARTS - 1; ++x)
                if (x < part) before += (unsigned)of_part(totals, x)[which];
        return before;
    };
    const uint32_t lower = (1u << lane) - 1;
    auto before_lane = [&](const uint4& v) { return __popc(v.x & lower) + __popc(v.y & lower) + __popc(v.z & lower) + __popc(v.w & lower); };
    auto vote4 = [&](uint32_t flags) {
        return make_uint4(__ballot_sync(0xffffffffu, flags & 1), __ballot_sync(0xffffffffu, flags & 2), __ballot_sync(0xffffffffu, flags & 4),
                          __ballot_sync(0xffffffffu, flags & 8));
    };
    const bool ties = left < of;  // not all equals stay
    auto equals = [&](const uint32_t(&key)[4], uint32_t there) {
        uint32_t f = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) f |= (uint32_t)(key[e] == found) << e;
        return f & there;
    };
    unsigned first_equal = 0;
    if (ties) {
        each_group([&](int g, int, const uint32_t(&key)[4], uint32_t there) {
            const uint4 v = vote4(equals(key, there));
            if (lane == 0) ahead[g] = __popc(v.x) + __popc(v.y) + __popc(v.z) + __popc(v.w);
        });
        first_equal = number(0);
    }
    // the marks: tokens below m that go, later ones that stay
    each_group([&](int g, int i, const uint32_t(&key)[4], uint32_t there) {
        uint32_t stay = 0;
        if (!ties) {
#pragma unroll
            for (int e = 0; e < 4; ++e) stay |= (uint32_t)(key[e] >= found) << e;
        } else {
            const uint32_t equal = equals(key, there);
            int rank = (int)(first_equal + ahead[g]) + before_lane(vote4(equal));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                stay |= (uint32_t)(key[e] > found || ((equal >> e & 1) && rank < left)) << e;
                rank += equal >> e & 1;
            }
        }
        uint32_t below = i + 3 < m ? 15u : i >= m ? 0u : (1u << (m - i)) - 1;
        const uint4 v = vote4((stay ^ below) & there);
        __syncwarp();
        if (lane == 0) {
            votes[g] = v;
            ahead[g] = __popc(v.x) + __popc(v.y) + __popc(v.z) + __popc(v.w);
        }
    });
    const unsigned first_mark = number(1);
    // holes in all; the first tail of each part
    unsigned marks = 0, holes;
    if constexpr (PARTS > 1) {
#pragma unroll
        for (int x = 0; x < PARTS; ++x) marks += (unsigned)of_part(totals, x)[1];
    } else {
        marks = (unsigned)totals[1];
    }
    holes = marks / 2;  // (as many as tails)
    // (the keys are done with) this part's tails in their order, from its first one on
    const unsigned first_tail = first_mark > holes ? first_mark : holes;
    auto marked = [&](int g, auto f) {  // f(place, number of the mark before it, is it one)
        const uint4 v = votes[g];
        unsigned rank = first_mark + ahead[g] + before_lane(v);
        const uint32_t bit[4] = {v.x >> lane & 1, v.y >> lane & 1, v.z >> lane & 1, v.w >> lane & 1};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            f(at0 + g * kGroup + 4 * lane + e, rank, bit[e] != 0);
            rank += bit[e];
        }
    };
#pragma unroll 1
    for (int g = max(0, m - at0) / kGroup + warp; g < groups; g += warps)
        marked(g, [&](int i, unsigned rank, bool is) {
            if (is && i >= m) keys[rank - first_tail] = (uint32_t)i;
        });
    all_sync();
    // every slot from `sinks` to the end
    unsigned tail_of[PARTS];  // number of the first tail of each part
    if constexpr (PARTS > 1) {
        unsigned c = 0;
#pragma unroll
        for (int x = 0; x < PARTS; ++x) {
            tail_of[x] = c > holes ? c : holes;
            c += (unsigned)of_part(totals, x)[1];
        }
    }
#pragma unroll 1
    for (int g = warp; g < groups && at0 + g * kGroup < m; g += warps)
        marked(g, [&](int i, unsigned rank, bool is) {
            if (i < off || i >= m) return;
            int from = i;
            if (is) {
                if constexpr (PARTS > 1) {
                    const unsigned want = holes + rank;  // the last part whose tails begin at or before it has it
                    int x = 0;
                    unsigned first = tail_of[0];
#pragma unroll
                    for (int y = 1; y < PARTS; ++y)
                        if (want >= tail_of[y]) x = y, first = tail_of[y];
                    from = (int)of_part(keys, x)[want - first];
                } else {
                    from = (int)keys[rank];
                }
            }
            s.kept[base + i] = base + from;
        });
    if constexpr (PARTS > 1) all_sync();  // a block stays until the others have read its tails
}

// The same from more tokens: the keys are read again for every step, and the tokens numbered in rounds of one per thread.
__global__ void __launch_bounds__(kLongThreads, 1) select_long_kernel(const __grid_constant__ EvictParams p) {
    grid_dependents_launch();
    grid_dependency_wait();
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
    grid_dependents_launch();
    grid_dependency_wait();
    const int b = (int)(blockIdx.x / (unsigned)p.Hkv), h = (int)(blockIdx.x % (unsigned)p.Hkv);
    const int n = min(p.seqlens[b], p.budget), limit = p.max_pages * p.page_size;
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
        const int page = pt[evict_page(p, tok, slot)];
        if (page >= 0 && page < p.num_pages) return page * p.page_size + slot;
        atomicCAS(p.status, 0, kDevBadIndex);
        return -1;
    };
    auto sum_of = [&](int row) {  // the score of a cache row
        const int page = row / p.page_size;
        return p.score + ((long long)page * p.Hkv + h) * p.page_size + (row - page * p.page_size);
    };
    for (unsigned j0 = 0; j0 < (unsigned)max(n, 0); j0 += kMoves) {  // (unsigned: behind the last slots of a bad length j0 is 2^31)
        // the slots from j0 on that get another row; neighbouring ones of this thread
        const int first = (int)j0 + tid * kLook;
        int tok[kLook];
        unsigned moves = 0;
#pragma unroll
        for (int x = 0; x < kLook; ++x) tok[x] = first + x < n ? kept[first + x] : -1;
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

template <int PARTS>
cudaError_t launch_select(EvictParams p, bool quads, long long groups, long long rows, int num_sms, cudaStream_t stream) {
    static std::atomic<bool> attr_set[2][kMaxAttrDevices];
    p.groups = (int)((groups + PARTS - 1) / PARTS);
    // A thread for 8 tokens, but no more than run at once (1024 on an SM, by their registers): 64 x 8 rows of 4100-4352 tokens with 512
    // threads each, two waves of blocks, 22 us.
    unsigned threads = 128;
    while (threads < 1024 && threads * 8 < (unsigned)p.groups * kGroup && rows * PARTS * threads * 2 <= 1024LL * num_sms) threads *= 2;
    const auto kernel = quads ? select_kernel<true, PARTS> : select_kernel<false, PARTS>;
    const cudaError_t e = ensure_smem_attr(kernel, kPartGroups * kGroupBytes, attr_set[quads]);
    if (e != cudaSuccess) return e;
    return launch_kernel(kernel, dim3((unsigned)(rows * PARTS)), threads, (size_t)p.groups * kGroupBytes, stream, {true, PARTS > 1 ? PARTS : 0}, p);
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
    // Places to choose from at most, in groups. A row has the blocks that its keys need room in, and further ones while each still has
    // 2048 places and an SM for itself (its 1024 threads fill the registers: 16 x 8 rows of up to 32768 tokens 25 us, in four parts each 66).
    const long long most = (long long)max_pages_per_seq * page_size - sinks - recent;
    const long long groups = most > 0 ? (most + 3 + kGroup - 1) / kGroup : 1, rows = (long long)B * Hkv;
    int parts = 1;
    while (parts < kMaxParts && groups > (long long)kPartGroups * parts) parts *= 2;
    while (parts < kMaxParts && groups >= 32LL * parts && rows * parts * 2 <= num_sms) parts *= 2;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const bool quads = page_size % 4 == 0 && multiple(score, 16);
    cudaError_t e;
    if (groups > (long long)kPartGroups * parts || rows * parts > INT32_MAX)
        e = launch_kernel(select_long_kernel, dim3((unsigned)rows), kLongThreads, 0, cs, {true}, p);
    else
        e = parts == 1   ? launch_select<1>(p, quads, groups, rows, num_sms, cs)
            : parts == 2 ? launch_select<2>(p, quads, groups, rows, num_sms, cs)
            : parts == 4 ? launch_select<4>(p, quads, groups, rows, num_sms, cs)
                         : launch_select<8>(p, quads, groups, rows, num_sms, cs);
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
