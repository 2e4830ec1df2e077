// Eviction from a paged cache by accumulated attention weight: which tokens stay (attn_kv_select_paged), and their move to the
// slots that remain (attn_kv_compact_paged).
//
// Selection, one block per (sequence, kv head). Of the tokens between the first `sinks` and the last `recent` the m with the
// largest scores stay, ties to the earlier token. Scores become unsigned keys of the same order; the m-th largest key is found by
// digits of 8 bits from the top: a histogram of the keys that share the digits found so far, the digit in which the count from
// above passes m. Then every thread knows of its tokens whether they stay, but for those equal to that key, which
// are numbered in token order. A kept token below end = budget - recent stays in its slot; the holes there, numbered in
// order, take the kept tokens behind end, numbered in order. The keys are read from memory once and held in registers
// when a block's threads have room for them, else read again in every pass. Bounded by latency: a dozen block-wide steps.
//
// Compaction: row kept[j] -> j with kept[j] >= j. A block walks the slots in ascending order: it loads a run of rows,
// then stores them. Every row that it reads later lies at or behind the end of the run, so nothing is overwritten that is still needed,
// and only the loads and the stores of one run need a barrier between them. Blocks share nothing: one has a (sequence, kv head) and
// some 16-byte columns of its rows, fewer columns where there are few sequences. Bounded by the memory.
#include "attn.h"
#include "kernels.cuh"
#include "launch.cuh"

#include <math.h>
#include <string.h>

namespace attn {
namespace {

constexpr int kSelectThreads = 1024;
constexpr int kHeld = 16;  // keys per thread in registers
constexpr int kPairs = 4096;  // holes paired with tokens at a time

struct EvictParams {
    float* score;           // [num_pages, Hkv, page_size]
    uint8_t* cache[2];      // [num_pages, page_size, Hkv, row_bytes]
    const int* page_table;  // [B, max_pages]
    const int* seqlens;     // [B]: cached tokens (selection), tokens that stay (compaction)
    int* kept;              // [B, Hkv, budget]
    int* new_seqlens;       // [B]
    int B, Hkv, page_size, max_pages, num_pages, budget, sinks, recent;
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
    const int x = sums[lane];  // 32 warps
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

__global__ void __launch_bounds__(kSelectThreads, 1) select_kernel(const __grid_constant__ EvictParams p) {
    __shared__ int hist[256], sums[32], digit_at[2], place[kPairs];
    const int tid = threadIdx.x, lane = tid & 31;
    const int b = (int)(blockIdx.x / (unsigned)p.Hkv), h = (int)(blockIdx.x % (unsigned)p.Hkv);
    const int len = __ldg(p.seqlens + b), K = p.budget;
    int* kept = p.kept + (long long)blockIdx.x * K;
    if (len < 0 || len > (long long)p.max_pages * p.page_size) {
        for (int j = tid; j < K; j += kSelectThreads) kept[j] = -1;
        if (tid == 0) {
            atomicCAS(p.status, 0, kDevBadIndex);
            if (h == 0) p.new_seqlens[b] = len;
        }
        return;
    }
    if (h == 0 && tid == 0) p.new_seqlens[b] = min(len, K);
    if (len <= K) {
        for (int j = tid; j < K; j += kSelectThreads) kept[j] = j < len ? j : -1;
        return;
    }
    const int end = K - p.recent, stop = len - p.recent;
    for (int j = tid; j < p.sinks; j += kSelectThreads) kept[j] = j;
    for (int j = tid; j < p.recent; j += kSelectThreads) kept[end + j] = stop + j;
    const int m = end - p.sinks, n = stop - p.sinks;  // m of n tokens stay, m < n
    if (m == 0) return;
    const int* pt = p.page_table + (long long)b * p.max_pages;
    auto key_of = [&](int i) -> uint32_t {  // of token sinks + i
        if (i >= n) return 0;
        int slot;
        const int page = __ldg(pt + evict_page(p, p.sinks + i, slot));
        if (page < 0 || page >= p.num_pages) {
            atomicCAS(p.status, 0, kDevBadIndex);
            return 0;
        }
        return score_key(__ldg(p.score + ((long long)page * p.Hkv + h) * p.page_size + slot));
    };
    uint32_t held[kHeld];
    const bool fits = n <= kHeld * kSelectThreads;
    if (fits) {
#pragma unroll
        for (int x = 0; x < kHeld; ++x) held[x] = key_of(x * kSelectThreads + tid);
    }
    const int rounds = (n + kSelectThreads - 1) / kSelectThreads;
    // f(key, i) for all tokens in rounds of one per thread; every thread takes part in every round
    auto each = [&](auto f) {
        if (fits) {
#pragma unroll
            for (int x = 0; x < kHeld; ++x)
                if (x < rounds) f(held[x], x * kSelectThreads + tid);
        } else {
            for (int x = 0; x < rounds; ++x) f(key_of(x * kSelectThreads + tid), x * kSelectThreads + tid);
        }
    };

    // the m-th largest key, and how many of its equals stay
    uint32_t found = 0;
    int left = m;
    for (int shift = 24; shift >= 0; shift -= 8) {
        if (tid < 256) hist[tid] = 0;
        __syncthreads();
        each([&](uint32_t key, int i) {
            if (i < n && (shift == 24 || (key ^ found) >> (shift + 8) == 0)) atomicAdd(&hist[(key >> shift) & 255], 1);
        });
        __syncthreads();
        if (tid < 32) {  // counts from the top: lane l has digits 255 - 8 l ... 248 - 8 l
            int c[8], sum = 0;
#pragma unroll
            for (int x = 0; x < 8; ++x) sum += c[x] = hist[255 - 8 * lane - x];
            int upto = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += y;
            }
            int above = upto - sum;
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                if (above < left && above + c[x] >= left) digit_at[0] = 255 - 8 * lane - x, digit_at[1] = left - above;
                above += c[x];
            }
        }
        __syncthreads();
        found |= (uint32_t)digit_at[0] << shift;
        left = digit_at[1];
    }

    // In token order: equals of that key stay while their number is below `left`; then the holes and the kept tokens behind
    // `end` are numbered. All of a round's warps are numbered at once.
    uint32_t stays = 0;  // bit x: token x of this thread (when held); else worked out again below
    int equals = 0;      // before this round
    int holes = 0, tails = 0;
    const uint32_t below = (1u << lane) - 1;
    // numbers of a round: equals of this key before this thread
    auto stay = [&](uint32_t key, int i) {
        const bool equal = i < n && key == found;
        const uint32_t ballot = __ballot_sync(0xffffffffu, equal);
        int total;
        const int before = equals + warps_before(__popc(ballot), sums, total) + __popc(ballot & below);
        equals += total;
        return i < n && (key > found || (equal && before < left));
    };
    // holes in turn, kPairs at a time
    for (int first = 0;; first += kPairs) {
        equals = holes = tails = 0;
        int x = 0;
        each([&](uint32_t key, int i) {
            bool s;
            if (first == 0 || !fits) {
                s = stay(key, i);
                if (fits) stays |= (uint32_t)s << x;
            } else {
                s = stays >> x & 1;
            }
            ++x;
            const int tok = p.sinks + i;
            const bool hole = i < n && tok < end && !s, tail = i < n && tok >= end && s;
            if (i < n && tok < end && s && first == 0) kept[tok] = tok;
            int total;
            const uint32_t bh = __ballot_sync(0xffffffffu, hole), bt = __ballot_sync(0xffffffffu, tail);
            const int before = warps_before(__popc(bh) | __popc(bt) << 16, sums, total);
            const int nh = holes + (before & 0xFFFF) + __popc(bh & below) - first, ntl = tails + (before >> 16) + __popc(bt & below) - first;
            holes += total & 0xFFFF;
            tails += total >> 16;
            // (all holes come before the first token behind `end`, but for those of the same round)
            if (hole && nh >= 0 && nh < kPairs) place[nh] = tok;
            __syncthreads();
            if (tail && ntl >= 0 && ntl < kPairs) kept[place[ntl]] = tok;
        });
        if (holes <= first + kPairs) break;
        __syncthreads();
    }
}

// One 16-byte column of K and V rows per lane; kRun rows per thread and run.
constexpr int kCompactThreads = 512, kRun = 8;

__global__ void __launch_bounds__(kCompactThreads) compact_kernel(const __grid_constant__ EvictParams p) {
    const int b = (int)(blockIdx.x / (unsigned)p.Hkv), h = (int)(blockIdx.x % (unsigned)p.Hkv);
    const int n = min(__ldg(p.seqlens + b), p.budget), limit = p.max_pages * p.page_size;
    const int* kept = p.kept + (long long)blockIdx.x * p.budget;
    const int* pt = p.page_table + (long long)b * p.max_pages;
    const int each = p.row_bytes / 16;                        // columns of K, and of V
    const int lanes = p.columns, col = blockIdx.y * lanes + threadIdx.x % lanes;  // 2 each: the score
    const int rows = kCompactThreads / lanes, row0 = threadIdx.x / lanes;
    const bool active = row0 < rows && col < 2 * each + (p.score ? 1 : 0);
    uint8_t* cache = p.cache[col >= each && col < 2 * each];
    const int offset = 16 * (col >= each ? col - each : col);
    // address of token tok's 16 bytes (the score: 4), nullptr for a bad page
    auto at = [&](int tok) -> uint8_t* {
        int slot;
        const int page = __ldg(pt + evict_page(p, tok, slot));
        if (page < 0 || page >= p.num_pages) {
            atomicCAS(p.status, 0, kDevBadIndex);
            return nullptr;
        }
        if (col == 2 * each) return reinterpret_cast<uint8_t*>(p.score + ((long long)page * p.Hkv + h) * p.page_size + slot);
        return cache + (((long long)page * p.page_size + slot) * p.Hkv + h) * p.row_bytes + offset;
    };
    for (int j0 = 0; j0 < n; j0 += rows * kRun) {
        uint4 v[kRun];
        uint8_t* to[kRun];
#pragma unroll
        for (int x = 0; x < kRun; ++x) {
            const int j = j0 + x * rows + row0;
            to[x] = nullptr;
            if (!active || j >= n) continue;
            const int src = __ldg(kept + j);
            if (src == j || src == -1) continue;
            if (src < j || src >= limit) {
                atomicCAS(p.status, 0, kDevBadIndex);
                continue;
            }
            const uint8_t* from = at(src);
            if (!from) continue;
            to[x] = at(j);
            if (col == 2 * each)
                v[x].x = *reinterpret_cast<const uint32_t*>(from);
            else
                v[x] = *reinterpret_cast<const uint4*>(from);
        }
        __syncthreads();  // the run is read before any of its slots is written
#pragma unroll
        for (int x = 0; x < kRun; ++x) {
            if (!to[x]) continue;
            if (col == 2 * each)
                *reinterpret_cast<uint32_t*>(to[x]) = v[x].x;
            else
                *reinterpret_cast<uint4*>(to[x]) = v[x];
        }
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
    const cudaError_t e = launch_kernel(select_kernel, dim3((unsigned)(B * Hkv)), kSelectThreads, 0, static_cast<cudaStream_t>(stream), {}, p);
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
    // all columns of a row in one block, fewer (but whole 32-byte sectors) while there are SMs left
    const int all = p.row_bytes / 8 + (score ? 1 : 0);
    p.columns = all;
    while (p.columns > 2 && (long long)B * Hkv * ((all + p.columns - 1) / p.columns) * 2 <= num_sms) p.columns = (p.columns + 3) / 4 * 2;
    const unsigned parts = (unsigned)((all + p.columns - 1) / p.columns);
    const cudaError_t e = launch_kernel(compact_kernel, dim3((unsigned)(B * Hkv), parts), kCompactThreads, 0, static_cast<cudaStream_t>(stream), {}, p);
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}
