// Attention of drafted tokens over a paged cache for more than 16 rows (drafted tokens x query heads)
// per kv head, in short calls with d = 64 more than 32: 128-row tiles on the tcgen05 tensor cores.
//
// A block takes one (sequence, split of the keys, kv head, 128-row tile) and walks the split's keys in
// tiles of 64. Per tile S = Q K^T (M 128, N 64) and O += P V (M 128, N d), accumulators in tensor
// memory, P as the 16-bit A operand from tensor memory over S; two S buffers, so that the products of a
// tile run during the softmax of the one before. Two blocks share an SM (up to 113 KB of shared memory
// and 256 tensor-memory columns each), so that one block's start, latencies and end are covered by the
// other.
//
// 8-bit caches: K is multiplied as it is (kind::f8f6f4). Q is split into two e4m3 parts after scaling
// each row by a power of two: eight significant bits of bf16 are four and four, so the two parts hold q
// exactly unless an element is more than 2^9 below the row's largest (then it is off by at most 2^-17 of
// that). V is widened to f16 (exact), because P needs more than an 8-bit format: its small values, summed
// over a long context, are not small.
//
// Roles of the warps:
//   warps 0, 2   loads of K and of V: boxes of 64 or 16 rows through tensor maps of the caches viewed as
//                [rows, Hkv d] where the page size is a multiple of that (rows past the end or of a bad
//                page lie outside the map and arrive as zeros), else 16-byte copies of rows that the
//                page table gives. (A tensor copy costs its warp about 66 clocks, so gather copies of
//                four rows, 64 for a 32 KB tile, took 4600.)
//   warps 1, 3   one thread each issues S and P V. (Issued by a whole warp under a predicate, a product
//                costs 70 clocks instead of the 34 to 64 that it takes to execute; and the waits and commits
//                of S and P V in one thread made about 2000 clocks a tile.)
//   warps 4-7    softmax, one row per thread: maximum, conditional rescale of O (only when a maximum
//                grows by more than the threshold), exponentials, P; at the end O / l and the LSE. Warps
//                whose 32 rows are all padding do nothing
//   warp 8       16-bit caches: passes the V tiles on, taking non-finite values out of those that a row
//                may not see in full
//   warps 8-11   8-bit caches: widen the V tiles, taking out non-finite values in the same way
//
// What bounds it. 64 keys of bf16 K and V of a head are 32 KB; the products take 640 clocks of the SM
// (S 8 x 48, bound by the 6 KB of shared memory that each reads, P V 4 x 64). With up to 128 rows the bf16
// form is bounded by the memory: 16 drafted tokens x 4 query heads over 64 sequences of U[1K, 32K] tokens
// take 640 us, 6770 GB/s, 1.00 of the measured copy rate (8 tokens with page size 64: 618 us; page size 1:
// 770 us). 8-bit caches have half the bytes for the same products: 424 us in short bursts, 447 us under steady
// load, where the power limit lowers the clock (0.76, 0.72). No unit is full (tensor pipe 48 % active, memory 52 %, issue
// slots 39 %): a block follows the chain S -> softmax -> P V over two score buffers, and its cost does not fall
// with the rows. More than 128 rows: every further tile reads the cache again through the L2 (64 drafted tokens:
// bf16 904 us, 0.72 of the floor; e4m3 887 us, 0.64). d = 64: half the bytes per key and nearly the same chain
// (64 rows: bf16 343 us, 0.93; e4m3 338 us, 0.47).
// Tried and slower (same case, bf16 / 8-bit, before the work order; this form then took 698 / 584, with S and
// P V in a thread each and raw K 685 / 511): Q in tensor memory with one S buffer 713 / 753, or with S in
// steps of 32 keys 813 / 844 (a product takes 32 clocks at least); one S buffer with two separate P
// 685 / 531; one block of 512 threads per SM with two streams of even and odd tiles 696 / 721. In the present form
// (640 / 440): up to 64 rows copied over the idle softmax warps, each copy with a part of the keys (all of V has to be
// finite then) 1130 / 427; S as a product of M = 64 for them 643 / 450.
#include "launch.cuh"
#include "tree_device.cuh"

#include <float.h>

namespace attn {
namespace {

constexpr int kTileRows = 128;  // rows per block
constexpr int kTileKeys = 64;

template <int D, int FMT>
struct TileLayout {
    static constexpr bool kF8 = FMT != ATTN_KV_BF16;
    static constexpr int kThreads = kF8 ? 384 : 288;
    static constexpr int kQBytes = kTileRows * D * 2;  // 16-bit Q, or its two 8-bit parts
    static constexpr int kChunkQ = kTileRows * 128;    // one [128 rows x 128 bytes] chunk of 16-bit Q
    static constexpr int kTile16 = kTileKeys * D * 2;  // a 16-bit K or V tile
    static constexpr int kChunk16 = kTileKeys * 128;   // one [64 keys x 128 bytes] chunk of it
    static constexpr int kLoad = kF8 ? kTileKeys * D : kTile16;  // a K or V tile as loaded
    static constexpr int kStages = D == 128 ? (kF8 ? 3 : 2) : (kF8 ? 6 : 4);  // loaded K/V tile pairs in flight
    static constexpr int kQOff = 0;
    static constexpr int kRingOff = kQBytes;  // stage s: K tile, V tile
    static constexpr int kWideOff = kRingOff + kStages * 2 * kLoad;  // 8-bit caches: two f16 V tiles
    static constexpr int kBarOff = kWideOff + (kF8 ? 2 * kTile16 : 0);
    // barriers; pairs are [tile parity]
    static constexpr int bQ = 0, bS = 1, bP = 3, bPFree = 5, bWV = 7, bWVFree = 9, bDrain = 11, bLast = 13;
    static constexpr int bK = 14, bV = bK + kStages, bKFree = bV + kStages, bVFree = bKFree + kStages;
    static constexpr int bClean = bVFree + kStages;
    static constexpr int kBars = bClean + kStages;
    // tensor-memory base, abort flag, tiles with odd values, split; sequence, head group, tokens from, to
    static constexpr int kMiscOff = kBarOff + kBars * 8;
    static constexpr int kBytes = kMiscOff + 32;
    // the block's result for the cluster's join, over the tiles when they are done with: [row][kPartRow], LSE
    static constexpr int kPartRow = D + 4, kPartLse = kTileRows * kPartRow * 4;
    static_assert(kPartLse + kTileRows * 4 <= kBarOff, "room for the block's result");
    // at least 80 KB, so that no more than two blocks (256 tensor-memory columns each) share an SM; the
    // dynamic shared memory has to start on a 1024-byte boundary (checked)
    static constexpr int kAlloc = kBytes > 81920 ? kBytes : 81920;
    static_assert(kAlloc <= 115712, "two blocks per SM");
};

constexpr uint32_t kColS = 0, kColO = 128, kCols = 256;  // S buffers at 0 and 64

__device__ __forceinline__ void fence_smem_to_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// A box of rows (columns c .. c + box) from row r on.
__device__ __forceinline__ void copy_box(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int c, int r) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c), "r"(r)
        : "memory");
}

// D (+)= A B of 8-bit operands in shared memory.
__device__ __forceinline__ void mma8_ss(uint32_t d, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// K-major shared-memory descriptor of rows of 64 bytes with the 64-byte swizzle (eight rows are 512 bytes).
__device__ __forceinline__ uint64_t smem_desc_sw64(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)1 << 16 | (uint64_t)(512 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)4 << 61;
}

__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t limit) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, limit));
}

__device__ __forceinline__ void sts128(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void lds128(uint32_t at, uint32_t (&w)[4]) {
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at) : "memory");
}

// Two 8-bit codes in the low (or high) half of w as an f16 pair; e5m2 is the upper byte of an f16.
template <int FMT, int HI>
__device__ __forceinline__ uint32_t widen_pair(uint32_t w) {
    if constexpr (FMT == ATTN_FP8_E5M2)
        return __byte_perm(w, 0, HI ? 0x3424 : 0x1404);
    else
        return fp8x2_f16x2<FMT>(HI ? w >> 16 : w);
}

// Widen the 64-row tile of 8-bit codes at src into f16 at dst (chunks of [64 rows x 128 bytes],
// 128-byte swizzle); thread t of 128. kClean: take non-finite values out, return whether there were any in the
// first `held` rows.
// Eight neighbouring threads take four 16-byte units each of a row pair (at d = 128 the lower units of
// one row and the upper ones of the other), so that neither the loads nor the stores conflict.
template <int D, int FMT, bool kClean>
__device__ __forceinline__ bool widen_tile(uint32_t src, uint32_t dst, int t, int held) {
    constexpr int kHalves = D == 128 ? 2 : 1;  // units per thread and row pair
    constexpr int kPasses = 2;                 // row pairs t / 8 and t / 8 + 16
    const int odd_row = (t >> 2) & 1, row = 2 * (t >> 3) + odd_row, low = t & 3;
    const uint32_t sw = (uint32_t)(row & 7);  // rows advance by 32: the same swizzle
    uint32_t w[kHalves * kPasses][4];  // all loaded before the first is stored
#pragma unroll
    for (int x = 0; x < kHalves * kPasses; ++x) {
        const int u = D == 128 ? low + 4 * (odd_row ^ (x & 1)) : low;
        const int n = D == 128 ? x >> 1 : x;
        // 128-byte rows arrive in the 128-byte swizzle, 64-byte rows in the 64-byte one
        lds128(src + (row + 32 * n) * D + ((D == 128 ? u ^ sw : u ^ ((sw >> 1) & 3)) << 4), w[x]);
    }
    bool odd = false;
#pragma unroll
    for (int x = 0; x < kHalves * kPasses; ++x) {
        const int u = D == 128 ? low + 4 * (odd_row ^ (x & 1)) : low;
        const int n = D == 128 ? x >> 1 : x;
        uint32_t h[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            h[2 * i] = widen_pair<FMT, 0>(w[x][i]);
            h[2 * i + 1] = widen_pair<FMT, 1>(w[x][i]);
        }
        if (kClean) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t keep = finite_halves(h[i], true);
                odd |= keep != 0xFFFFFFFFu && row + 32 * n < held;
                h[i] &= keep;
            }
        }
        const uint32_t to = dst + (u >> 2) * (kTileKeys * 128) + (row + 32 * n) * 128;
        sts128(to + (((2 * (u & 3)) ^ sw) << 4), h[0], h[1], h[2], h[3]);
        sts128(to + (((2 * (u & 3) + 1) ^ sw) << 4), h[4], h[5], h[6], h[7]);
    }
    return odd;
}

// The same with cleaning, for the few tiles that need it (out of line, to leave the loop's registers as they are).
template <int D, int FMT>
__device__ __noinline__ bool widen_clean(uint32_t src, uint32_t dst, int t, int held) {
    return widen_tile<D, FMT, true>(src, dst, t, held);
}

// Non-finite values out of a 16-bit V tile of kBytes bytes at vt, by a warp; true when there were any in the first
// `held` rows (the boxes also bring rows behind the last token).
template <int kBytes>
__device__ __noinline__ bool clean_tile(uint32_t vt, int held) {
    bool odd = false;
#pragma unroll 4
    for (int x = threadIdx.x & 31; x < kBytes / 16; x += 32) {
        uint32_t w[4];
        lds128(vt + 16 * x, w);
        bool bad = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t keep = finite_halves(w[e], false);
            bad |= keep != 0xFFFFFFFFu;
            w[e] &= keep;
        }
        if (bad) sts128(vt + 16 * x, w[0], w[1], w[2], w[3]);
        odd |= bad && ((x >> 3) & (kTileKeys - 1)) < held;
    }
    return odd;
}

// Tiles from this one on (six at most) hold drafted tokens or the end of the sequence.
__device__ __forceinline__ int first_mixed_tile(int ctx, int t_begin) { return ctx <= t_begin ? 0 : (ctx - t_begin) / kTileKeys; }

// What was taken out of V, tile by tile, to the outputs of a softmax warp. item: the block's sequence, head group and
// tokens (from shared memory, so that nothing of this rare path stays in the kernel's registers); odd: bit i for
// mixed tile i; split and part as for add_nonfinite.
template <int D, int FMT>
__device__ __noinline__ void add_odd_values(const TreeParams& p, const int* item, int odd, int split, float* part) {
    const int b = item[0], kvh = item[1] / p.groups, r0 = item[1] % p.groups * kTileRows, first = (threadIdx.x >> 5 & 3) * 32;
    TreeSeq s;
    if (!tree_seq(p, b, s)) return;
    const int rows = min(min(kTileRows, s.n * p.G - r0), first + 32), tile = first_mixed_tile(s.ctx, item[2]);
    if (first >= rows) return;
    for (; odd; odd &= odd - 1)
        add_nonfinite<D, FMT>(p, b, kvh, r0, first, 1, rows, item[2] + (tile + __ffs(odd) - 1) * kTileKeys, item[3], split, part,
                              TileLayout<D, FMT>::kPartRow);
}

// Four values to four e4m3 codes (they are in range and finite).
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | (uint32_t)hi << 16;
}

// Instruction descriptors with fp32 accumulation: 16-bit operands (both f16 or both bf16), and 8-bit
// ones (A e4m3, B e4m3 or e5m2).
__host__ __device__ constexpr uint32_t idesc16(bool f16, uint32_t M, uint32_t N, uint32_t b_mn_major) {
    return (1u << 4) | (f16 ? 0u : (1u << 7) | (1u << 10)) | (b_mn_major << 16) | ((N >> 3) << 17) | ((M >> 4) << 24);
}
__host__ __device__ constexpr uint32_t idesc8(uint32_t b_format, uint32_t M, uint32_t N) {
    return (1u << 4) | (b_format << 10) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

template <int D, int FMT, bool kCluster>
__global__ void __launch_bounds__((TileLayout<D, FMT>::kThreads), 2)
    tree_tile_kernel(const __grid_constant__ TreeParams p, const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV) {
    grid_dependents_launch();
    using L = TileLayout<D, FMT>;
    constexpr bool F8 = L::kF8;
    constexpr int NS = L::kStages;
    extern __shared__ __align__(1024) uint8_t smem[];
    int chunk, b, split, hg;
    if (!tree_item<kCluster>(p, reinterpret_cast<int*>(smem), chunk, b, split, hg)) return;
    const int kvh = hg / p.groups, r0 = (hg % p.groups) * kTileRows;
    TreeSeq s;
    if (!tree_seq(p, b, s)) return;
    const int R = min(kTileRows, s.n * p.G - r0);  // rows of this tile
    if (R <= 0) return;
    const int nsplit = cdiv(s.len, chunk);
    if (split < 0)
        split = nsplit > 0 ? nsplit - 1 : 0;
    else if (p.full_rows >= 0 && split >= nsplit - 1)
        return;  // the last split has its own block
    const int t_begin = split * chunk;
    auto out_row = [&](int r) {
        const int i = (r0 + r) / p.G;
        return (long long)(s.q0 + i) * p.Hq + kvh * p.G + (r0 + r - i * p.G);
    };
    if (s.len == 0) {
        if (split == 0)
            for (int x = threadIdx.x; x < R * D; x += blockDim.x) {
                const long long orow = out_row(x / D);
                p.o[orow * D + x % D] = __float2bfloat16(0.0f);
                if (x % D == 0) p.lse[orow] = -INFINITY;
            }
        return;
    }
    float* part_o = reinterpret_cast<float*>(smem);
    float* part_lse = reinterpret_cast<float*>(smem + L::kPartLse);
    const long long out_first = (long long)s.q0 * p.Hq + kvh * p.G;
    const bool joins = kCluster && nsplit > 1;  // the same in all blocks of a cluster
    if (t_begin >= s.len) {
        if (joins) cluster_join<D, L::kPartRow>(part_o, part_lse, p.o, p.lse, out_first, r0, R, p.G, p.Hq, p.cluster, nsplit);
        return;
    }
    const int t_end = min(s.len, t_begin + chunk);
    const int tiles = cdiv(t_end - t_begin, kTileKeys);

    if (smem_u32(smem) & 1023u) {  // the swizzles count from such boundaries
        if (threadIdx.x == 0) atomicCAS(p.status, 0, kDevTimeout);
        return;
    }
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMiscOff);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMiscOff + 4);
    int* odd_v = reinterpret_cast<int*>(smem + L::kMiscOff + 8);
    volatile int* part_slot = reinterpret_cast<volatile int*>(smem + L::kMiscOff + 12);  // (keeps it out of the registers)
    int* item = reinterpret_cast<int*>(smem + L::kMiscOff + 16);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint64_t wd = p.watchdog_ns;
    const int* pt = p.page_table + (long long)b * p.max_pages;
    // Warps with rows. The rows of padding hold whatever they find in shared and tensor memory: every
    // row of the products depends on its own row of Q and P alone.
    const int row_warps = cdiv(R, 32);
    if (threadIdx.x == 0) {
        mbar_init(&bars[L::bQ], row_warps);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars[L::bS + i], 1);
            mbar_init(&bars[L::bP + i], row_warps);
            mbar_init(&bars[L::bPFree + i], 1);
            mbar_init(&bars[L::bWV + i], 4);
            mbar_init(&bars[L::bWVFree + i], 1);
            mbar_init(&bars[L::bDrain + i], 1);
        }
        mbar_init(&bars[L::bLast], 1);
        for (int i = 0; i < NS; ++i) {
            mbar_init(&bars[L::bK + i], 1);
            mbar_init(&bars[L::bV + i], 1);
            mbar_init(&bars[L::bKFree + i], 1);
            mbar_init(&bars[L::bVFree + i], F8 ? 4 : 1);  // 8-bit: the widening warps; else the products
            mbar_init(&bars[L::bClean + i], 1);
        }
        *abort_flag = 0;
        *odd_v = 0;
        item[0] = b, item[1] = hg, item[2] = t_begin, item[3] = t_end;
        *part_slot = nsplit == 1 ? -1 : joins ? -2 : split;
        fence_mbar_init();
    }
    if (p.box_rows > 1 && warp == 0 && lane == 0) {  // (else there are no maps)
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, kCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t ring = smem_u32(smem + L::kRingOff);
    const int first_mixed = first_mixed_tile(s.ctx, t_begin);

    if (warp == 0 || warp == 2) {
        // ---------------------------------------------------------------- loads of K (warp 0), V (warp 2)
        const bool v = warp == 2;
        uint64_t* full = &bars[v ? L::bV : L::bK];
        uint64_t* free = &bars[v ? L::bVFree : L::bKFree];
        const uint32_t tile = ring + (v ? L::kLoad : 0);
        bool ok = true;
        if (p.box_rows > 1) {
            // boxes: lane -> 16 or 64 rows of one page, and which 128-byte chunk of them
            const CUtensorMap* map = v ? &tmV : &tmK;
            constexpr int kParts = !F8 && D == 128 ? 2 : 1;
            const int per_part = kTileKeys / p.box_rows;
            const bool active = lane < kParts * per_part;
            const int part = lane / per_part, first = (lane - part * per_part) * p.box_rows;
            const int col = kvh * D + part * 64;
            const uint32_t dst = tile + part * L::kChunk16 + first * (F8 ? D : 128);
            const int none = p.num_pages * p.page_size;  // the first row past the cache: zeros
            // the page of the next tile's box is looked up before the copies of this one are issued
            int page = 0, slot = 0;
            bool some = false;
            auto look_up = [&](int i) {
                const int tok = t_begin + i * kTileKeys + first;
                some = active && tok < t_end;
                if (some) page = __ldg(pt + page_of(p, tok, slot));
            };
            look_up(0);
            int issued = 0;
            for (int i = 0; i < tiles; ++i) {
                const int st = i % NS;
                int row = none;
                if (some) {
                    if (page >= 0 && page < p.num_pages)
                        row = page * p.page_size + slot;  // < num_pages * page_size <= INT32_MAX
                    else
                        atomicCAS(p.status, 0, kDevBadIndex);
                }
                if (i + 1 < tiles) look_up(i + 1);
                if (!(ok = wait_all(&free[st], (uint32_t)((i / NS) & 1) ^ 1u, abort_flag, wd))) break;
                if (lane == 0) mbar_arrive_expect_tx(&full[st], L::kLoad);
                __syncwarp();
                if (active) copy_box(dst + st * 2 * L::kLoad, map, &full[st], col, row);
                __syncwarp();
                issued = i + 1;
            }
            if (!ok) {
                // let the copies in flight land before the block can end
                int dummy = 0;
                for (int i = issued > NS ? issued - NS : 0; i < issued; ++i)
                    mbar_wait(&full[i % NS], (uint32_t)((i / NS) & 1), &dummy, 20000000ull);
            }
        } else {
            // other page sizes: each lane finds the cache rows of tokens lane and lane + 32, and copies 16-byte
            // pieces of all rows; a tile is handed over once the copies of the next one are on their way
            constexpr int kRowBytes = F8 ? D : 2 * D, kPieces = kRowBytes / 16, kRows = 32 / kPieces;
            const uint8_t* cache = static_cast<const uint8_t*>(v ? p.v_cache : p.k_cache);
            const int piece = lane % kPieces, sub = lane / kPieces;
            const long long row_bytes = (long long)p.Hkv * kRowBytes;
            const int col = kvh * kRowBytes + piece * 16;
            int page[2], slot[2], n = 0;
            auto look_up = [&](int i) {
                const int tok = t_begin + i * kTileKeys + lane;
                n = tok >= t_end ? 0 : (tok + 32 >= t_end ? 1 : 2);
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (e < n) page[e] = __ldg(pt + page_of(p, tok + 32 * e, slot[e]));
            };
            auto hand_over = [&](int i) {
                fence_smem_to_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&full[i % NS]);
            };
            look_up(0);
            for (int i = 0; i < tiles; ++i) {
                const int st = i % NS;
                int row[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    row[e] = -1;  // no token, or a bad page: zeros
                    if (e < n) {
                        if (page[e] >= 0 && page[e] < p.num_pages)
                            row[e] = page[e] * p.page_size + slot[e];
                        else
                            atomicCAS(p.status, 0, kDevBadIndex);
                    }
                }
                if (i + 1 < tiles) look_up(i + 1);
                if (!(ok = wait_all(&free[st], (uint32_t)((i / NS) & 1) ^ 1u, abort_flag, wd))) break;
#pragma unroll
                for (int it = 0; it < kTileKeys / kRows; ++it) {
                    const int r = it * kRows + sub;
                    const int rr = __shfl_sync(0xffffffffu, row[it * kRows / 32], r & 31);
                    const uint32_t at = tile + st * 2 * L::kLoad +
                                        (kPieces == 16  ? (piece >> 3) * L::kChunk16 + r * 128 + (((piece & 7) ^ (r & 7)) << 4)
                                         : kPieces == 8 ? r * 128 + ((piece ^ (r & 7)) << 4)
                                                        : r * 64 + ((piece ^ ((r >> 1) & 3)) << 4));
                    cp_async16(at, cache + (rr >= 0 ? rr * row_bytes + col : 0), rr >= 0 ? 16u : 0u);
                }
                cp_async_commit();
                if (i > 0) {
                    cp_async_wait<1>();
                    hand_over(i - 1);
                }
            }
            cp_async_wait<0>();
            if (ok) hand_over(tiles - 1);
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------------- S = Q K^T
        // S(i) goes to buffer i & 1, over P(i - 2), once the product with that is complete.
        constexpr uint32_t idS = F8 ? idesc8(FMT == ATTN_FP8_E5M2 ? 1 : 0, kTileRows, kTileKeys) : idesc16(false, kTileRows, kTileKeys, 0);
        const uint32_t q_base = smem_u32(smem + L::kQOff);
        const uint64_t dq = F8 && D == 64 ? smem_desc_sw64(q_base) : smem_desc_sw128(q_base, 16, 1024);
        const uint64_t dk = F8 && D == 64 ? smem_desc_sw64(ring) : smem_desc_sw128(ring, 16, 1024);
        if (lane == 0) {
            auto wait = [&](int bar, uint32_t parity) { return mbar_wait(&bars[bar], parity, abort_flag, wd); };
            bool any = false;
            int st = 0;
            uint32_t par = 0;
            if (wait(L::bQ, 0)) {
                for (int i = 0; i < tiles; ++i) {
                    const int sb = i & 1;
                    if (!wait(L::bPFree + sb, ((uint32_t)(i >> 1) & 1u) ^ 1u) || !wait(L::bK + st, par)) break;
                    tc_fence_after();
                    any = true;
                    const uint64_t kd = dk + (uint64_t)((st * 2 * L::kLoad) >> 4);
                    if constexpr (F8) {
#pragma unroll
                        for (int x = 0; x < 2 * (D / 32); ++x) {  // both parts of Q
                            const int part = x / (D / 32), k = x % (D / 32);
                            mma8_ss(tmem + kColS + 64 * sb, dq + (uint64_t)((part * kTileRows * D + k * 32) >> 4), kd + (uint64_t)((k * 32) >> 4),
                                    idS, x > 0);
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < D / 16; ++k)
                            tc_mma_ss(tmem + kColS + 64 * sb, dq + (uint64_t)(((k >> 2) * L::kChunkQ + (k & 3) * 32) >> 4),
                                      kd + (uint64_t)(((k >> 2) * L::kChunk16 + (k & 3) * 32) >> 4), idS, k > 0);
                    }
                    tc_commit(&bars[L::bS + sb]);
                    tc_commit(&bars[L::bKFree + st]);
                    if (++st == NS) st = 0, par ^= 1u;
                }
            }
            if (any) {
                // every product has completed before the tensor memory is released
                tc_commit(&bars[L::bDrain]);
                int dummy = 0;
                mbar_wait(&bars[L::bDrain], 0, &dummy, 50000000ull);
            }
        }
        __syncwarp();
    } else if (warp == 3) {
        // ---------------------------------------------------------------- O += P V
        constexpr uint32_t idO = idesc16(F8, kTileRows, D, 1);
        const uint64_t dv = smem_desc_sw128(F8 ? smem_u32(smem + L::kWideOff) : ring + L::kLoad, L::kChunk16, 1024);
        if (lane == 0) {
            auto wait = [&](int bar, uint32_t parity) { return mbar_wait(&bars[bar], parity, abort_flag, wd); };
            bool any = false;
            int st = 0;
            uint32_t par = 0;
            for (int i = 0; i < tiles; ++i) {
                const int sb = i & 1;
                const uint32_t half = (uint32_t)(i >> 1) & 1u;
                if (F8 ? !wait(L::bWV + sb, half) : !wait(L::bV + st, par) || !wait(L::bClean + st, par)) break;
                if (!wait(L::bP + sb, half)) break;
                tc_fence_after();
                any = true;
                const uint64_t vd = dv + (uint64_t)((F8 ? sb * L::kTile16 : st * 2 * L::kLoad) >> 4);
#pragma unroll
                for (int k = 0; k < kTileKeys / 16; ++k)
                    tc_mma_ts(tmem + kColO, tmem + kColS + 64 * sb + k * 8, vd + (uint64_t)(k * (2048 >> 4)), idO, i > 0 || k > 0);
                tc_commit(&bars[L::bPFree + sb]);
                tc_commit(F8 ? &bars[L::bWVFree + sb] : &bars[L::bVFree + st]);
                if (i == tiles - 1) tc_commit(&bars[L::bLast]);
                if (++st == NS) st = 0, par ^= 1u;
            }
            if (any) {
                tc_commit(&bars[L::bDrain + 1]);
                int dummy = 0;
                mbar_wait(&bars[L::bDrain + 1], 0, &dummy, 50000000ull);
            }
        }
        __syncwarp();
    } else if (!F8 && warp == 8) {
        // ---------------------------------------------------------------- 16-bit V tiles
        if constexpr (!F8) {
            for (int i = 0; i < tiles; ++i) {
                const int st = i % NS;
                if (!wait_all(&bars[L::bV + st], (uint32_t)((i / NS) & 1), abort_flag, wd)) break;
                if (i >= first_mixed) {
                    const bool odd = clean_tile<L::kTile16>(ring + st * 2 * L::kLoad + L::kLoad, t_end - t_begin - i * kTileKeys);
                    if (odd) atomicOr(odd_v, 1 << (i - first_mixed));
                    __threadfence_block();
                    fence_smem_to_async();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[L::bClean + st]);
            }
        }
    } else if (warp >= 8) {
        // ---------------------------------------------------------------- 8-bit V tiles to f16
        if constexpr (F8) {
            const int t = threadIdx.x & 127;
            const uint32_t wide = smem_u32(smem + L::kWideOff);
            // (two loops and the cleaning out of line: as branches of one loop 431 us became 485, 64 x U[1K, 32K], 16 drafted)
            auto step = [&](int i, auto clean) {
                const int st = i % NS, wb = i & 1;
                if (!wait_all(&bars[L::bV + st], (uint32_t)((i / NS) & 1), abort_flag, wd)) return false;
                if (!wait_all(&bars[L::bWVFree + wb], (uint32_t)((i >> 1) & 1) ^ 1u, abort_flag, wd)) return false;
                const uint32_t src = ring + st * 2 * L::kLoad + L::kLoad, dst = wide + wb * L::kTile16;
                if constexpr (decltype(clean)::value) {
                    if (widen_clean<D, FMT>(src, dst, t, t_end - t_begin - i * kTileKeys)) atomicOr(odd_v, 1 << (i - first_mixed));
                    __threadfence_block();
                } else {
                    widen_tile<D, FMT, false>(src, dst, t, kTileKeys);
                }
                fence_smem_to_async();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bars[L::bWV + wb]);
                    mbar_arrive(&bars[L::bVFree + st]);
                }
                return true;
            };
            int i = 0;
            bool go = true;
            for (; go && i < min(first_mixed, tiles); ++i) go = step(i, std::false_type{});
            for (; go && i < tiles; ++i) go = step(i, std::true_type{});
        }
    } else if (warp - 4 < row_warps) {
        // ---------------------------------------------------------------- softmax and output
        const int quarter = warp & 3;
        const int row = quarter * 32 + lane;
        const bool valid = row < R;
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
        const uint32_t tO = tmem + lane_off + kColO;
        const long long orow = valid ? out_row(row) : 0;
        const int node = valid ? (r0 + row) / p.G : s.n - 1;  // rows of padding see what the last node sees
        const unsigned long long* mrow = p.mask ? p.mask + (long long)(s.q0 + node) * p.mask_words : nullptr;
        float row_scale = 1.0f;  // 8-bit caches: what the row's Q was divided by
        {
            // this thread's row of Q into shared memory, K-major with the swizzle of its row length
            const uint32_t q = smem_u32(smem + L::kQOff);
            const uint4* src = reinterpret_cast<const uint4*>(p.q + orow * D);
            auto load = [&](int c, float (&f)[8]) {
                uint4 x = make_uint4(0, 0, 0, 0);
                if (valid) x = __ldg(src + c);
                const uint32_t in[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    f[2 * e] = __uint_as_float(in[e] << 16) * p.q_sign;
                    f[2 * e + 1] = __uint_as_float(in[e] & 0xFFFF0000u) * p.q_sign;
                }
            };
            if constexpr (!F8) {
#pragma unroll
                for (int c = 0; c < D / 8; ++c) {
                    float f[8];
                    load(c, f);
                    sts128(q + (c >> 3) * L::kChunkQ + row * 128 + (((c & 7) ^ (row & 7)) << 4), pack_bf16x2(f[0], f[1]),
                           pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
                }
            } else {
                // 2^up brings the largest magnitude of the row into [128, 256); a row with a non-finite
                // element becomes NaN
                float top = 0.0f;
                bool finite = true;
#pragma unroll 4
                for (int c = 0; c < D / 8; ++c) {
                    float f[8];
                    load(c, f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        finite = finite && isfinite(f[e]);
                        top = fmaxf(top, fabsf(f[e]));
                    }
                }
                const int up = finite && top > 0.0f ? min(120, 7 - ilogbf(top)) : 0;
                const float mul = finite ? exp2f((float)up) : __int_as_float(0x7fffffff);
                row_scale = exp2f((float)-up);
#pragma unroll 2
                for (int u = 0; u < D / 16; ++u) {  // 16 codes of each part
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float f[8];
                        load(2 * u + c, f);
#pragma unroll
                        for (int e = 0; e < 8; ++e) f[e] *= mul;
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t w = e4m3x4(f[4 * e], f[4 * e + 1], f[4 * e + 2], f[4 * e + 3]);
                            hi[2 * c + e] = w;
                            const uint32_t a = fp8x2_f16x2<ATTN_FP8_E4M3>(w), b = fp8x2_f16x2<ATTN_FP8_E4M3>(w >> 16);
                            lo[2 * c + e] = e4m3x4(f[4 * e] - half_value((uint16_t)a), f[4 * e + 1] - half_value((uint16_t)(a >> 16)),
                                                   f[4 * e + 2] - half_value((uint16_t)b), f[4 * e + 3] - half_value((uint16_t)(b >> 16)));
                        }
                    }
                    const uint32_t at = q + row * D + ((D == 128 ? u ^ (row & 7) : u ^ ((row >> 1) & 3)) << 4);
                    sts128(at, hi[0], hi[1], hi[2], hi[3]);
                    sts128(at + kTileRows * D, lo[0], lo[1], lo[2], lo[3]);
                }
            }
            fence_smem_to_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[L::bQ]);
        }
        // (a product that rounds to 0, or to infinity, would turn masked scores, -inf, or scores of 0 into NaN)
        const float scale = F8 ? fminf(p.scale * row_scale, FLT_MAX) : p.scale;
        const float sl2 = F8 ? fminf(fmaxf(p.scale_log2 * row_scale, 0x1p-126f), FLT_MAX) : p.scale_log2;
        float m = -INFINITY, l = 0.0f;
        bool ok = true;
        for (int i = 0; i < tiles; ++i) {
            const int sb = i & 1;
            const uint32_t tS = tmem + lane_off + kColS + 64 * sb;
            if (!(ok = wait_all(&bars[L::bS + sb], (uint32_t)((i >> 1) & 1), abort_flag, wd))) break;
            tc_fence_after();
            // The row's 64 scores pass through 32 registers, the first half twice: maximum of keys
            // 0-31, maximum and exponentials of 32-63, exponentials of 0-31.
            uint32_t w0 = ~0u, w1 = ~0u;
            if (i >= first_mixed) {
                const unsigned long long w = tree_window(mrow, p.mask_words, node, s.ctx, s.len, t_begin + i * kTileKeys);
                w0 = (uint32_t)w, w1 = (uint32_t)(w >> 32);
            }
            uint32_t x[32];
            auto load_scores = [&](int c0, uint32_t seen) {
                tmem_ld32(tS + c0, x);
                tc_wait_ld();
                reg_fence(x);
                if (i >= first_mixed) {
#pragma unroll
                    for (int c = 0; c < 32; ++c)
                        if (!((seen >> c) & 1)) x[c] = 0xFF800000u;  // -inf
                }
            };
            auto top_score = [&]() {
                float mx[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) mx[e] = fmaxf(__uint_as_float(x[e]), __uint_as_float(x[e + 4]));
#pragma unroll
                for (int c = 8; c < 32; c += 8)
#pragma unroll
                    for (int e = 0; e < 4; ++e) mx[e] = max3f(mx[e], __uint_as_float(x[c + e]), __uint_as_float(x[c + 4 + e]));
                return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
            };
            load_scores(0, w0);
            float mc = fmaxf(m, top_score());
            load_scores(32, w1);
            mc = fmaxf(mc, top_score());
            if (__any_sync(0xffffffffu, (mc - m) * sl2 > p.rescale_thr)) {  // NaN (both -inf) is false
                const float alpha = m == -INFINITY ? 0.0f : ex2_mufu((m - mc) * sl2);
                if (i > 0) {
                    // O += P(i - 1) V is complete before O is rescaled (S(i) was issued before it)
                    if (!(ok = wait_all(&bars[L::bPFree + (sb ^ 1)], (uint32_t)((i - 1) >> 1) & 1u, abort_flag, wd))) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < D; c += 16) {
                        uint32_t o[16];
                        tmem_ld16(tO + c, o);
                        tc_wait_ld();
                        reg_fence(o);
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                        tmem_st16(tO + c, o);
                    }
                }
                l *= alpha;
                m = mc;
            }
            const float neg = m == -INFINITY ? 0.0f : -m * sl2;
            float sum[4] = {0, 0, 0, 0};
            uint32_t pk[16];
            auto exponentials = [&]() {
#pragma unroll
                for (int c = 0; c < 32; c += 2) {
                    float x0, x1;
                    ffma2(x0, x1, __uint_as_float(x[c]), __uint_as_float(x[c + 1]), sl2, sl2, neg, neg);
                    const float p0 = ex2_mufu(x0), p1 = ex2_mufu(x1);
                    const int a = ((c >> 1) & 1) * 2;
                    fadd2(sum[a], sum[a + 1], sum[a], sum[a + 1], p0, p1);
                    pk[c >> 1] = F8 ? pack_half2(p0, p1) : pack_bf16x2(p0, p1);
                }
            };
            exponentials();
            load_scores(0, w0);  // before P of keys 32-63 goes over them
            tmem_st16(tS + 16, pk);
            exponentials();
            tmem_st16(tS, pk);
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[L::bP + sb]);
        }
        if (ok) ok = wait_all(&bars[L::bLast], 0, abort_flag, wd);
        if (ok) {
            tc_fence_after();
            const float inv = l == 0.0f ? 0.0f : p.v_descale / l;
            const bool empty = l == 0.0f;
            const int part = *part_slot;  // split, -1: the only one, -2: for the cluster's join
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                tmem_ld32(tO + c, o);
                tc_wait_ld();
                reg_fence(o);
                float v[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(o[e]);
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = empty ? 0.0f : v[e] * inv;
                if (valid && part == -1) {
                    uint4* dst = reinterpret_cast<uint4*>(p.o + orow * D + c);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        dst[e] = make_uint4(pack_bf16x2(v[8 * e], v[8 * e + 1]), pack_bf16x2(v[8 * e + 2], v[8 * e + 3]),
                                            pack_bf16x2(v[8 * e + 4], v[8 * e + 5]), pack_bf16x2(v[8 * e + 6], v[8 * e + 7]));
                } else if (valid) {
                    float4* dst = reinterpret_cast<float4*>((kCluster ? part_o + row * L::kPartRow : p.ws_o + (orow * p.max_splits + part) * D) + c);
#pragma unroll
                    for (int e = 0; e < 8; ++e) dst[e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
                }
                __syncwarp();
            }
            if (valid) {
                const float lse = empty ? -INFINITY : m * scale + logf(l);
                if (part == -1)
                    p.lse[orow] = lse;
                else if (kCluster)
                    part_lse[row] = lse;
                else
                    p.ws_lse[orow * p.max_splits + part] = lse;
            }
        }
    }

    // -------------------------------------------------------------------- end
    __syncwarp();
    tc_fence_before();
    named_bar_sync(1, L::kThreads);
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, kCols);
    if (threadIdx.x == 0 && *abort_flag) atomicCAS(p.status, 0, kDevTimeout);
    if (warp >= 4 && warp < 8 && *odd_v) add_odd_values<D, FMT>(p, item, *odd_v, *part_slot, part_o);
    if (kCluster && *part_slot == -2) cluster_join<D, L::kPartRow>(part_o, part_lse, p.o, p.lse, out_first, r0, R, p.G, p.Hq, p.cluster, nsplit);
}

template <int D, int FMT, bool kCluster>
cudaError_t launch_tiles(TreeParams p, const TreeTmaps& tm, cudaStream_t stream) {
    constexpr int bytes = TileLayout<D, FMT>::kAlloc;
    static std::atomic<bool> attr_set[kMaxAttrDevices];
    cudaError_t e = ensure_smem_attr(tree_tile_kernel<D, FMT, kCluster>, bytes, attr_set);
    if (e != cudaSuccess) return e;
    p.groups = (int)(((long long)p.max_q * p.G + kTileRows - 1) / kTileRows);
    const dim3 grid = tree_grid(p);
    return launch_kernel(tree_tile_kernel<D, FMT, kCluster>, grid, TileLayout<D, FMT>::kThreads, bytes, stream, {false, p.cluster}, p, tm.k, tm.v);
}

template <int D, bool kCluster>
cudaError_t launch_fmt(const TreeParams& p, const TreeTmaps& tm, int fmt, cudaStream_t stream) {
    return fmt == ATTN_FP8_E4M3   ? launch_tiles<D, ATTN_FP8_E4M3, kCluster>(p, tm, stream)
           : fmt == ATTN_FP8_E5M2 ? launch_tiles<D, ATTN_FP8_E5M2, kCluster>(p, tm, stream)
                                  : launch_tiles<D, ATTN_KV_BF16, kCluster>(p, tm, stream);
}

}  // namespace

cudaError_t launch_tree_tiles(const TreeParams& p, const TreeTmaps& tm, int d, int kv_format, cudaStream_t stream) {
    if (p.cluster > 0)
        return d == 128 ? launch_fmt<128, true>(p, tm, kv_format, stream) : launch_fmt<64, true>(p, tm, kv_format, stream);
    return d == 128 ? launch_fmt<128, false>(p, tm, kv_format, stream) : launch_fmt<64, false>(p, tm, kv_format, stream);
}

}  // namespace attn
