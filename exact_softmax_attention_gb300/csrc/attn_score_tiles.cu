// Attention weight per cached token for more rows per kv head than score_few_rows (the last queries of a prompt, or all of them):
// 128-row tiles on the tcgen05 tensor cores.
//
// The transposed scores S^T = K Q^T have the tokens as rows of the accumulator, so that a thread owns a token: it
// reads its row of S^T from tensor memory, adds exp2(scale s - lse) over the columns, and needs no sum across threads. A unit of
// work is 512 tokens of a (sequence, kv head) (fewer where there would be fewer units than SMs), four accumulator tiles of 128 that share the
// operand Q; a task is a unit times a block of up to 128 rows (as many whole queries times their query heads as fit) that see any of it. The
// tasks of the whole call, in the order sequence, kv head, tokens, rows, are dealt out in equal runs to one persistent block per SM. A unit
// that lies in more than one run leaves partial sums, which a second kernel adds in order.
//
// What bounds it. With d = 128 a task is 4 x 8 products of 128 x 128 x 16 and 65536 exponentials, 2048 clocks of the tensor pipe and of the MUFU,
// for 32 KB of q from the L2 (with units of 256 tokens the L2 was the bound: 153 us for the whole prompts below). Measured: 3300 clocks. The
// products take 92 clocks each, not 64, because both operands come out of shared memory, and a tile's only buffer is held through the products and
// three quarters of the exponentials. Rows that stay the same (up to 128) against new tokens every task are 128 KB of bf16 keys for that, more than
// the memory delivers in the time.
// Whole prompts, 8 x U[512, 4096] tokens, 32/8 heads of 128, bf16: 130 us, 1020 TFLOP/s. Parts left out one by one, three calls in turn (127 us
// then): no exponentials 126, neither them nor the loads of the accumulators 127, an eighth of the products 120, that without exponentials 84. So
// the products take all of the time, the exponentials and loads nearly all, side by side: only less of both would be faster.
// The same over e4m3: 187 us, about 37 of them for the parts of q (151 MB in, as much out). Without exponentials 173, with an eighth of the products 179,
// without loads of the accumulators 174, without reading LSE and factors per column 159: these reads from shared memory cost most.
// The last 32 queries of 16 x U[2K, 16K] cached tokens: bf16 52 us, 5.4 TB/s; e4m3 51 us, heads of 64 44 and 49 us. With any of these parts left out, bf16
// and e4m3 take at most 3 us less: the keys' way into shared memory, and the start.
// Other arrangements, whole prompts, at 138 us then: 32 columns of all tiles to four warps each 179 us; 64 columns of all tiles to four of eight
// warps with their LSE in registers 258; eight warps for every other tile 160; the two product threads in turns 143; later, at 130: keys in
// tensor memory as operand A, products with 64 rows at a time, 161; parts of 32 columns left out in tiles on the diagonal 159; shares of the work
// by the tiles that a task's rows see, instead of by tasks, 133.
//
// The LSE. exp2(c s - l) is exp2(c (s - l / c)): for bf16 keys -l / c comes with the products, as three more columns of q (its bf16 parts) against
// ones, which spares a load from shared memory per column (128 us -> 126). Where the scale does not leave it 24 bits (2^-60 < |c| < 2^60 does), and for
// 8-bit keys, whose rows have factors of their own, it is read per column.
//
// Roles of the warps: 0-15 exponentials and sums, four warps per accumulator tile; 16 and 17 the keys of two tiles each, through tensor
// copies of 64 or 16 rows where the page size is a multiple of that, else by 16-byte copies of rows that the page table gives; 18 the blocks
// of q through tensor copies (one box is the heads of as many queries as fit) and their LSE; 19 and 20 the products of two tiles each,
// issued by one thread: while one waits for its buffer, the other one's products run.
//
// Work split: the tasks are those of the lengths, but the size of a unit and the number of blocks go by the page table's capacity. It makes little
// difference: 32 queries of 4 x U[500, 2000] tokens 9.8 us in a tight table, 9.0 in one of 131072 tokens; of 2000 tokens 7.6 and 8.1; one prompt of
// 1500 tokens 21.6 in both.
//
// Start. 14500 clocks passed before the first product, 5300 in the shares of the work and 2900 in the search of its first task, mostly divisions;
// with multipliers for them, as a programmatic dependent, and with the joining kernel's own search done before it waits: 138 -> 130 us,
// the queries against cached tokens 55.7 -> 52.4.
//
// 8-bit caches: K is multiplied as it is (kind::f8f6f4). A kernel before this one scales each row of q by a power of two and splits
// it into two e4m3 parts: exact unless an element is more than 2^9 below the row's largest (then off by at most 2^-17 of that).
#include "score.cuh"

namespace attn {
namespace {

constexpr int kTileTok = 128, kTiles = 4;   // tokens of an accumulator tile, tiles of a unit at most
constexpr int kUnitTok = kTiles * kTileTok;
constexpr int kBlockRows = 128;             // rows of a task
constexpr int kTileThreads = 21 * 32;
constexpr float kBf16Max = 0x1.FEp127f;
constexpr int kSumWarps = 16, kKeyWarp = 16, kQueryWarp = 18, kProductWarp = 19;

template <int D, int FMT, bool FOLD>
struct ScoreLayout {
    static constexpr bool kF8 = FMT != ATTN_KV_BF16;
    static constexpr int kRow = kF8 ? D : 2 * D;             // bytes of a key
    static constexpr int kBox = kRow < 128 ? kRow : 128;     // bytes of a row in a copy
    static constexpr int kChunk = 128 * kBox;                // [128 rows x 128 (64) bytes]
    static constexpr int kChunks = kRow / kBox;              // of a tile of keys
    static constexpr int kTile = kChunk * kChunks;
    static constexpr int kQChunks = kF8 ? 2 : kChunks;       // of a block of q: its columns, or its two 8-bit parts
    static constexpr int kQ = kQChunks * kChunk;
    static constexpr int kKStages = kTile > 16384 ? 4 : 8;   // tiles of keys
    static constexpr int kQStages = kQ > 16384 ? 2 : 4, kLseStages = kQStages + 2;
    static constexpr int kKOff = 0, kQOff = kKStages * kTile;
    // per row of a block of q: minus the LSE (times log2 e), factor of the scores, last token seen
    static constexpr int kLseOff = kQOff + kQStages * kQ, kLseStage = 3 * kBlockRows * 4;
    // further columns of the operands that give minus the LSE: 16 ones and zeros per token, the three bf16 parts per row of a stage of q
    static constexpr int kFoldK = (kLseOff + kLseStages * kLseStage + 255) / 256 * 256, kFold = FOLD ? 128 * 32 : 0, kFoldQ = kFoldK + kFold;
    static constexpr int kBarOff = kFoldQ + kQStages * kFold;
    static constexpr int bK = 0, bKFree = bK + kKStages, bQ = bKFree + kKStages, bQFree = bQ + kQStages, bL = bQFree + kQStages, bLFree = bL + kLseStages;
    static constexpr int bS = bLFree + kLseStages, bSFree = bS + kTiles, bDrain = bSFree + kTiles, kBars = bDrain + 2;
    // tensor-memory base, abort flag; per lse stage: do rows need their own limits; the plan
    static constexpr int kMiscOff = kBarOff + kBars * 8, kOddOff = kMiscOff + 8, kPlanOff = kOddOff + kLseStages * 4;
    static constexpr int kBytes = kPlanOff + 16;
    static_assert(kBarOff % 8 == 0 && kPlanOff % 8 == 0 && kLseStages % 2 == 0 && kBytes <= 232448, "shared memory of an SM");
};

__device__ __forceinline__ void fence_smem_to_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void copy_box(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int c, int r) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c), "r"(r)
        : "memory");
}

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

// The same for rows of 32 bytes with the 32-byte swizzle.
__device__ __forceinline__ uint64_t smem_desc_sw32(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)1 << 16 | (uint64_t)(256 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)6 << 61;
}

// 16-byte unit u of row r of such rows.
__device__ __forceinline__ uint4* unit32(uint8_t* tile, int r, int u) { return reinterpret_cast<uint4*>(tile + r * 32 + ((u ^ ((r >> 2) & 1)) << 4)); }

// Instruction descriptor, fp32 accumulation, M = 128: bf16 operands, or A in the cache's 8-bit format and B e4m3.
template <int FMT>
__device__ __forceinline__ uint32_t score_idesc(int n) {
    const uint32_t formats = FMT == ATTN_KV_BF16 ? (1u << 7) | (1u << 10) : FMT == ATTN_FP8_E5M2 ? 1u << 7 : 0u;
    return (1u << 4) | formats | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}

// Byte offset of 16-byte unit u of row r in a tile of 128 rows of kRow bytes, swizzled.
template <int kRow>
__device__ __forceinline__ uint32_t unit_at(int r, int u) {
    if constexpr (kRow == 64)
        return r * 64 + ((u ^ ((r >> 1) & 3)) << 4);
    else
        return (u >> 3) * (128 * 128) + r * 128 + (((u & 7) ^ (r & 7)) << 4);
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | (uint32_t)hi << 16;
}

__device__ __forceinline__ void e4m3x4_values(uint32_t w, float (&f)[4]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(i ? w >> 16 : w)));
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}" : "=f"(f[2 * i]), "=f"(f[2 * i + 1]) : "r"(h));
    }
}

// Rows of q for an 8-bit cache: parts [T Hq, 2, D] of e4m3 and the factor of each row's scores. D / 8 threads per row.
template <int D>
__global__ void __launch_bounds__(256) split_q_kernel(const __nv_bfloat16* q, uint8_t* parts, float* factor, long long rows, float scale_log2) {
    grid_dependents_launch();
    constexpr int kUnits = D / 8;
    const long long r = ((long long)blockIdx.x * 256 + threadIdx.x) / kUnits;
    const int u = threadIdx.x % kUnits;
    uint4 w = make_uint4(0, 0, 0, 0);
    if (r < rows) w = reinterpret_cast<const uint4*>(q + r * D)[u];
    const uint32_t e[4] = {w.x, w.y, w.z, w.w};
    uint32_t top = 0;
#pragma unroll
    for (int y = 0; y < 4; ++y) top = max(top, max(e[y] & 0x7FFFu, (e[y] >> 16) & 0x7FFFu));
#pragma unroll
    for (int o = 1; o < kUnits; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (r >= rows) return;
    // 2^up brings the largest magnitude into [128, 256) (biased exponent 127 + 7 + 127 - exponent; the tiniest rows as far as a
    // float reaches)
    const int exponent = (int)(top >> 7);
    float up = 1.0f;
    if (exponent < 255 && top != 0) up = __uint_as_float((unsigned)min(254, 261 - exponent) << 23);
    uint32_t part[2][2];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        float f[4], v[4];
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            f[2 * z] = __uint_as_float(e[2 * y + z] << 16) * up;
            f[2 * z + 1] = __uint_as_float(e[2 * y + z] & 0xFFFF0000u) * up;
        }
        part[0][y] = e4m3x4(f[0], f[1], f[2], f[3]);
        e4m3x4_values(part[0][y], v);
        part[1][y] = e4m3x4(f[0] - v[0], f[1] - v[1], f[2] - v[2], f[3] - v[3]);
    }
    uint2* to = reinterpret_cast<uint2*>(parts + r * 2 * D);
    to[u] = make_uint2(part[0][0], part[0][1]);
    to[kUnits + u] = make_uint2(part[1][0], part[1][1]);
    // a row with a non-finite element gives NaN
    if (u == 0) factor[r] = exponent == 255 ? __int_as_float(0x7fffffff) : scale_log2 / up;
}

// ---- the tasks of a call

// Tasks of one kv head of a sequence. Unit u (tokens from unit_tok u on) is taken with the blocks of rows from first(u) on; blocks that
// do not see it may be among them (when the queries of a block do not divide a unit).
struct SeqTasks {
    int units, blocks;
    long long skip;  // first(u) = max(0, each u - skip)
    int each;        // blocks of a unit's tokens, rounded down
    int cut;         // the first unit that not all blocks see
    __device__ __forceinline__ SeqTasks(const ScoreParams& p, const ScoreSeq& s) {
        units = (s.len + p.unit_tok - 1) >> p.unit_shift;
        blocks = p.by_block_tok(s.n + p.block_tok - 1) * p.head_blocks;
        // token U u is query U u - ctx, in block floor((U u - ctx) / block_tok) >= floor(U / block_tok) u - ceil(ctx / block_tok)
        each = p.unit_blocks.d * p.head_blocks;
        const int before = p.by_block_tok(s.ctx + p.block_tok - 1);
        skip = (long long)before * p.head_blocks;
        cut = p.unit_blocks(before) + 1;
    }
    __device__ __forceinline__ int first(int u) const {
        const long long f = (long long)each * u - skip;
        return f > 0 ? (int)f : 0;
    }
    // tasks of the units before u
    __device__ __forceinline__ long long before(int u) const {
        const long long n = u - cut;  // units of which some blocks are left out
        return (long long)blocks * u - (n > 0 ? each * ((cut + u - 1) * n / 2) - skip * n : 0);
    }
};

// The units of a run in turn, each with the blocks [r, end) of its rows that the run holds.
struct UnitWalk {
    int b, h, u, r, end;
    int left;        // tasks of the run behind this unit
    long long from;  // each u - skip
    bool whole;      // the run holds the first of the unit's tasks
    ScoreSeq s;
    SeqTasks seq;
    __device__ __forceinline__ UnitWalk(const ScoreParams& p, int b_, long long rest, int count) : b(b_), s(), seq(p, s) {
        score_seq(p, b, s);
        seq = SeqTasks(p, s);
        const long long each = seq.before(seq.units);
        h = (int)(rest / each);
        rest -= each * h;
        int lo = 0, hi = seq.units - 1;  // the last unit with before(u) <= rest
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (seq.before(mid) <= rest)
                lo = mid;
            else
                hi = mid - 1;
        }
        u = lo;
        const int behind = (int)(rest - seq.before(u));
        r = seq.first(u) + behind;
        whole = behind == 0;
        from = (long long)seq.each * u - seq.skip;
        left = count;
        cut();
    }
    __device__ __forceinline__ void cut() {
        end = min(seq.blocks, r + left);
        left -= end - r;
    }
    __device__ __forceinline__ bool complete() const { return end == seq.blocks; }
    // On to the next unit (left > 0). Returns whether its first block of q is another one than the last one of this.
    __device__ __forceinline__ bool next(const ScoreParams& p) {
        const int last = end - 1;
        whole = true;
        if (++u < seq.units) {
            from += seq.each;
            r = from > 0 ? (int)from : 0;
            cut();
            return r != last;
        }
        u = r = 0;
        if (++h >= p.Hkv) {
            h = 0;
            do ++b;
            while (!score_seq(p, b, s));
            seq = SeqTasks(p, s);
        }
        from = -seq.skip;
        cut();
        return true;
    }
    // tiles of the unit that there are
    __device__ __forceinline__ int tiles(const ScoreParams& p) const { return min(p.unit_tok, s.len - u * p.unit_tok + kTileTok - 1) / kTileTok; }
    // last token that a block of rows sees
    __device__ __forceinline__ int top(const ScoreParams& p, int i0) const { return s.ctx + min(i0 + p.block_tok, s.n) - 1; }
    // first query of a block, its first head, its rows
    __device__ __forceinline__ int query(const ScoreParams& p, int block) const {
        return p.head_blocks > 1 ? block / p.head_blocks : block * p.block_tok;
    }
    __device__ __forceinline__ int head(const ScoreParams& p, int block) const { return p.head_blocks > 1 ? block % p.head_blocks * kBlockRows : 0; }
    __device__ __forceinline__ int rows(const ScoreParams& p, int block) const {
        if (p.head_blocks > 1) return min(kBlockRows, p.G - head(p, block));
        return min(p.block_tok, s.n - block * p.block_tok) * p.G;
    }
};

// Tasks of sequence b, all kv heads.
__device__ __forceinline__ long long tasks_of(const ScoreParams& p, int b) {
    ScoreSeq s;
    if (!score_seq(p, b, s)) return 0;
    const SeqTasks t(p, s);
    return t.before(t.units) * p.Hkv;
}

// The run of tasks [from, from + count) of block `block`: its first sequence and the task within that. Every thread of the
// block calls it; sums: a word per warp, out: two.
struct TaskRun {
    long long each, from;  // tasks per block; the first one of this
    long long rest;        // tasks of sequence b before it
    int b, count;
};
template <int kThreads>
__device__ __forceinline__ TaskRun task_run(const ScoreParams& p, int block, long long* sums, long long* out) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = p.B <= kThreads ? 1 : (p.B + kThreads - 1) / kThreads, b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
    const long long first = b0 < b1 ? tasks_of(p, b0) : 0;
    long long mine = first;
    for (int b = b0 + 1; b < b1; ++b) mine += tasks_of(p, b);
    long long upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
    }
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    long long total = 0;
    for (int w = 0; w * 32 * per < p.B; ++w) {  // (warps that have sequences)
        if (w == warp) upto += total;
        total += sums[w];
    }
    TaskRun run;
    run.each = total < INT32_MAX - p.grid.d ? p.grid((int)total + p.grid.d - 1) : (total + p.grid.d - 1) / p.grid.d;
    run.from = run.each * block;
    const long long left = total - run.from;
    run.count = (int)(left < run.each ? (left > 0 ? left : 0) : run.each);
    const long long ahead = upto - mine;
    if (run.count > 0 && b0 < b1 && run.from >= ahead && run.from < upto) {
        long long rest = run.from - ahead;
        int b = b0;
        for (long long n = first; rest >= n; n = tasks_of(p, ++b)) rest -= n;
        out[0] = b;
        out[1] = rest;
    }
    __syncthreads();
    run.b = (int)out[0];
    run.rest = out[1];
    return run;
}

template <int D, int FMT, bool FOLD>
__global__ void __launch_bounds__(kTileThreads, 1)
    score_tiles_kernel(const __grid_constant__ ScoreParams p, const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK) {
    using L = ScoreLayout<D, FMT, FOLD>;
    constexpr bool F8 = L::kF8;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMiscOff);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMiscOff + 4);
    int* odd_rows = reinterpret_cast<int*>(smem + L::kOddOff);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint64_t wd = p.watchdog_ns;
    if (smem_u32(smem) & 1023u) {  // (the swizzles count from such boundaries)
        if (threadIdx.x == 0) atomicCAS(p.status, 0, kDevTimeout);
        grid_dependency_wait();
        return;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < L::kKStages; ++i) {
            mbar_init(&bars[L::bK + i], 1);
            mbar_init(&bars[L::bKFree + i], 1);
        }
        for (int i = 0; i < L::kQStages; ++i) {
            mbar_init(&bars[L::bQ + i], FOLD ? 2 : 1);
            mbar_init(&bars[L::bQFree + i], 2);
        }
        for (int i = 0; i < L::kLseStages; ++i) {
            mbar_init(&bars[L::bL + i], 1);
            mbar_init(&bars[L::bLFree + i], kSumWarps);
        }
        for (int i = 0; i < kTiles; ++i) {
            mbar_init(&bars[L::bS + i], 1);
            mbar_init(&bars[L::bSFree + i], 4);
        }
        mbar_init(&bars[L::bDrain], 1);
        mbar_init(&bars[L::bDrain + 1], 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmQ);
        if (p.box_rows > 1) tma_prefetch_desc(&tmK);
    }
    // rows that no copy of q writes are zeros
    if (p.block_tok * p.G < kBlockRows)
        for (int i = threadIdx.x; i < L::kQStages * L::kQ / 16; i += kTileThreads) reinterpret_cast<uint4*>(smem + L::kQOff)[i] = make_uint4(0, 0, 0, 0);
    if (FOLD && threadIdx.x < 256)
        *unit32(smem + L::kFoldK, threadIdx.x >> 1, threadIdx.x & 1) = threadIdx.x & 1 ? make_uint4(0, 0, 0, 0) : make_uint4(0x3F803F80u, 0x3F80u, 0, 0);
    fence_smem_to_async();
    // Nothing that an earlier kernel writes is read before this, and no tensor memory is held that one may still ask for. (8-bit caches: only
    // split_q_kernel can still be running, since that is an ordinary launch. So lengths, pages, keys and old sums are read, and tensor memory is asked
    // for, without a wait; the parts of q and their factors behind one, in the warp that copies them.)
    if (!F8) grid_dependency_wait();
    grid_dependents_launch();
    if (warp == kProductWarp) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    const TaskRun run = task_run<kTileThreads>(p, blockIdx.x, reinterpret_cast<long long*>(smem + L::kLseOff), reinterpret_cast<long long*>(smem + L::kPlanOff));
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if (run.count == 0) {
        if (F8) grid_dependency_wait();
        if (warp == kProductWarp) tmem_dealloc(tmem, 512);
        return;
    }
    const uint32_t base = smem_u32(smem);
    UnitWalk at(p, run.b, run.rest, run.count);

    // The stages of the keys belong to the tiles of a unit, the same number to each, so that one warp fills a stage and one thread
    // multiplies what it holds; its n-th use:
    const int per_tile = L::kKStages * kTileTok / p.unit_tok;
    auto key_stage = [&](int t, int n) { return t * per_tile + (n & (per_tile - 1)); };  // (powers of two)
    auto key_turn = [&](int n) { return (uint32_t)(n / per_tile & 1); };

    if (warp == kKeyWarp || warp == kKeyWarp + 1) {
        // ---------------------------------------------------------------- keys, every other tile
        bool ok = true;
        int uses[2] = {0, 0};  // of the stages of this warp's two tiles
        const CUtensorMap* map = &tmK;
        const int none = p.num_pages * p.page_size;  // the first row past the cache: zeros
        uint64_t* pending = nullptr;                  // the stage whose 16-byte copies may still be on their way
        auto hand_over = [&]() {
            if (!pending) return;
            fence_smem_to_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(pending);
            pending = nullptr;
        };
        while (ok) {
            const int tiles = at.tiles(p);
            const int* pt = p.page_table + (long long)at.b * p.max_pages;
#pragma unroll
            for (int x = 0; x < kTiles / 2; ++x) {
                const int t = warp - kKeyWarp + 2 * x, st = key_stage(t, uses[x]);
                if (!ok || t >= tiles) continue;
                const uint32_t parity = key_turn(uses[x]) ^ 1u;
                const int t0 = at.u * p.unit_tok + t * kTileTok;
                const uint32_t to = base + L::kKOff + st * L::kTile;
                uint64_t* full = &bars[L::bK + st];
                if (p.box_rows > 1) {
                    // lane -> rows of one page, and which columns of them
                    const int boxes = kTileTok / p.box_rows;
                    const int part = lane / boxes, first = (lane - part * boxes) * p.box_rows;
                    const bool active = lane < L::kChunks * boxes;
                    int row = none, slot;
                    if (active && t0 + first < at.s.len) {
                        const int page = score_place(p, pt, t0 + first, slot);
                        if (page >= 0) row = page * p.page_size + slot;
                    }
                    if (!(ok = __all_sync(0xffffffffu, mbar_wait(&bars[L::bKFree + st], parity, abort_flag, wd)))) continue;
                    if (lane == 0) mbar_arrive_expect_tx(full, L::kTile);
                    __syncwarp();
                    if (active) copy_box(to + part * L::kChunk + first * L::kBox, map, full, at.h * D + part * (L::kBox / (F8 ? 1 : 2)), row);
                    __syncwarp();
                } else {
                    // rows of tokens lane, lane + 32, ...; 16-byte pieces of all of them
                    constexpr int kUnits = L::kRow / 16, kStep = 32 / kUnits;
                    int row[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        int slot;
                        const int page = t0 + lane + 32 * e < at.s.len ? score_place(p, pt, t0 + lane + 32 * e, slot) : -1;
                        row[e] = page >= 0 ? page * p.page_size + slot : -1;
                    }
                    // (a stage that is not free yet may wait for what this warp has not handed over)
                    if (!__all_sync(0xffffffffu, mbar_test_wait(&bars[L::bKFree + st], parity))) {
                        cp_async_wait<0>();
                        hand_over();
                        if (!(ok = __all_sync(0xffffffffu, mbar_wait(&bars[L::bKFree + st], parity, abort_flag, wd)))) continue;
                    }
                    const int u = lane % kUnits;
                    const uint8_t* keys = static_cast<const uint8_t*>(p.k_cache) + (long long)at.h * L::kRow + 16 * u;
                    const long long row_bytes = (long long)p.Hkv * L::kRow;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll 8
                        for (int r = lane / kUnits; r < 32; r += kStep) {
                            const int from = __shfl_sync(0xffffffffu, row[e], r);
                            cp_async16(to + unit_at<L::kRow>(32 * e + r, u), keys + (from >= 0 ? from : 0) * row_bytes, from >= 0 ? 16 : 0);
                        }
                    cp_async_commit();
                    if (pending) cp_async_wait<1>();
                    hand_over();
                    pending = full;
                }
                ++uses[x];
            }
            if (!ok || at.left == 0) break;
            at.next(p);
        }
        cp_async_wait<0>();
        hand_over();
        if (!ok) {
            // let the copies in flight land before the block can end
            int dummy = 0;
            for (int x = 0; x < kTiles / 2; ++x)
                for (int n = max(0, uses[x] - per_tile); n < uses[x]; ++n)
                    mbar_wait(&bars[L::bK + key_stage(warp - kKeyWarp + 2 * x, n)], key_turn(n), &dummy, 20000000ull);
        }
    } else if (warp == kQueryWarp) {
        // ---------------------------------------------------------------- blocks of q and their LSE
        if (F8) grid_dependency_wait();  // the parts of q
        const bool by_head = p.head_blocks > 1;
        const uint32_t bytes = (uint32_t)((by_head ? kBlockRows : p.G) * p.block_tok * L::kBox * L::kQChunks);
        int query[4], head[4];  // of rows lane, lane + 32, ... of a block
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int r = lane + 32 * e;
            query[e] = by_head ? 0 : r / p.G;
            head[e] = by_head ? r : r - query[e] * p.G;
        }
        bool ok = true, fresh = true;
        int qn = 0;
        while (ok) {
            for (int r = fresh ? at.r : at.r + 1; r < at.end; ++r) {
                const int st = qn % L::kQStages, ls = qn % L::kLseStages;
                const int i0 = at.query(p, r), h0 = at.head(p, r);
                float l[4], f[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const bool there = query[e] < p.block_tok && i0 + query[e] < at.s.n && h0 + head[e] < p.G;
                    const long long row = (long long)(at.s.q0 + i0 + query[e]) * p.Hq + at.h * p.G + h0 + head[e];
                    l[e] = there ? p.lse[row] : -INFINITY;
                    f[e] = F8 && there ? p.factor[row] : 0.0f;
                }
                if (!(ok = __all_sync(0xffffffffu, mbar_wait(&bars[L::bQFree + st], (uint32_t)(qn / L::kQStages & 1) ^ 1u, abort_flag, wd)))) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&bars[L::bQ + st], bytes);
#pragma unroll
                    for (int c = 0; c < L::kQChunks; ++c)
                        tma_load_3d(smem + L::kQOff + st * L::kQ + c * L::kChunk, &tmQ, &bars[L::bQ + st], c * (L::kBox / (F8 ? 1 : 2)),
                                    at.h * p.G + h0, at.s.q0 + i0);
                }
                __syncwarp();
                if constexpr (FOLD) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        // minus the LSE in units of the products; rows behind the box get weight 0
                        float v = l[e] * p.unit;
                        if (l[e] == -INFINITY) v = query[e] >= p.block_tok ? copysignf(kBf16Max, p.unit) : 0.0f;
                        v = v > kBf16Max ? kBf16Max : v < -kBf16Max ? -kBf16Max : v;
                        const float hi = __bfloat162float(__float2bfloat16_rn(v)), rest = v - hi, mid = __bfloat162float(__float2bfloat16_rn(rest));
                        uint8_t* to = smem + L::kFoldQ + st * L::kFold;
                        *unit32(to, lane + 32 * e, 0) = make_uint4(pack_bf16x2(hi, mid), pack_bf16x2(rest - mid, 0.0f), 0, 0);
                        *unit32(to, lane + 32 * e, 1) = make_uint4(0, 0, 0, 0);
                    }
                    fence_smem_to_async();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars[L::bQ + st]);
                }
                ++qn;
                if (!(ok = __all_sync(0xffffffffu, mbar_wait(&bars[L::bLFree + ls], (uint32_t)((qn - 1) / L::kLseStages & 1) ^ 1u, abort_flag, wd)))) break;
                float* lse2 = reinterpret_cast<float*>(smem + L::kLseOff + ls * L::kLseStage);
                bool odd = false;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int x = lane + 32 * e;
                    // rows behind the box are zeros and get weight 0; others that are not there, or saw nothing, are masked
                    const bool none = l[e] == -INFINITY, behind = query[e] >= p.block_tok;
                    odd = odd || (none && !behind);
                    lse2[x] = none ? (behind ? -INFINITY : 0.0f) : l[e] * -1.4426950408889634f;
                    if (F8) lse2[kBlockRows + x] = none ? 0.0f : f[e];
                    reinterpret_cast<int*>(lse2)[2 * kBlockRows + x] = none ? (behind ? INT32_MAX : -1) : at.s.ctx + i0 + query[e];
                }
                odd = __any_sync(0xffffffffu, odd);
                if (lane == 0) odd_rows[ls] = odd;
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[L::bL + ls]);
            }
            if (at.left == 0) break;
            fresh = at.next(p);
        }
        if (!ok) {
            int dummy = 0;
            for (int x = qn > L::kQStages ? qn - L::kQStages : 0; x < qn; ++x)
                mbar_wait(&bars[L::bQ + x % L::kQStages], (uint32_t)(x / L::kQStages & 1), &dummy, 20000000ull);
        }
    } else if (warp >= kProductWarp) {
        // ---------------------------------------------------------------- products of every other tile
        if (lane == 0) {
            const int mine = warp - kProductWarp;
            auto desc = [&](int off) { return L::kBox == 64 ? smem_desc_sw64(base + off) : smem_desc_sw128(base + off, L::kChunk, 1024); };
            const uint64_t dk = desc(L::kKOff), dq = desc(L::kQOff), fold_k = smem_desc_sw32(base + L::kFoldK), fold_q = smem_desc_sw32(base + L::kFoldQ);
            auto wait = [&](int bar, uint32_t parity) { return mbar_wait(&bars[bar], parity, abort_flag, wd); };
            bool any = false, go = true, fresh = true;
            int qs = 0;                          // stages of q waited for
            int keys[kTiles / 2] = {0, 0};       // uses of the stages of the two tiles' keys
            uint32_t uses[kTiles / 2] = {0, 0};  // of the two tiles' buffers
            while (go) {
                const int tiles = at.tiles(p);
                for (int r = at.r; r < at.end; ++r) {
                    if (fresh) {
                        if (!(go = wait(L::bQ + qs % L::kQStages, qs / L::kQStages & 1))) break;
                        ++qs;
                    }
                    const int st = (qs - 1) % L::kQStages, top = at.top(p, at.query(p, r));
                    const uint64_t qd = dq + (uint64_t)((st * L::kQ) >> 4);
                    const uint32_t idesc = score_idesc<FMT>((at.rows(p, r) + 31) & ~31);
#pragma unroll
                    for (int x = 0; x < kTiles / 2; ++x) {
                        const int t = mine + 2 * x, ks = key_stage(t, keys[x]);
                        if (!go || t >= tiles) continue;
                        if (r == at.r && !(go = wait(L::bK + ks, key_turn(keys[x])))) continue;
                        if (at.u * p.unit_tok + t * kTileTok > top) {  // these rows see nothing of it
                            if (r + 1 == at.end) tc_commit(&bars[L::bKFree + ks]), ++keys[x];
                            continue;
                        }
                        if (!(go = wait(L::bSFree + t, (uses[x]++ & 1) ^ 1u))) continue;
                        tc_fence_after();
                        any = true;
                        const uint32_t d = tmem + (uint32_t)t * 128;
                        const uint64_t kd = dk + (uint64_t)((ks * L::kTile) >> 4);
                        if constexpr (F8) {
#pragma unroll
                            for (int y = 0; y < 2 * (D / 32); ++y) {  // both parts of q
                                const int part = y / (D / 32), k = y % (D / 32);
                                mma8_ss(d, kd + (uint64_t)((k * 32) >> 4), qd + (uint64_t)((part * L::kChunk + k * 32) >> 4), idesc, y > 0);
                            }
                        } else {
#pragma unroll
                            for (int k = 0; k < D / 16; ++k)
                                tc_mma_ss(d, kd + (uint64_t)(((k >> 2) * L::kChunk + (k & 3) * 32) >> 4),
                                          qd + (uint64_t)(((k >> 2) * L::kChunk + (k & 3) * 32) >> 4), idesc, k > 0);
                            if constexpr (FOLD) tc_mma_ss(d, fold_k, fold_q + (uint64_t)((st * L::kFold) >> 4), idesc, 1);
                        }
                        tc_commit(&bars[L::bS + t]);
                        if (r + 1 == at.end) tc_commit(&bars[L::bKFree + ks]), ++keys[x];
                    }
                    if (!go) break;
                    fresh = true;
                    if (r + 1 < at.end) tc_commit(&bars[L::bQFree + st]);
                }
                if (!go || at.left == 0) break;
                fresh = at.next(p);
                if (fresh) tc_commit(&bars[L::bQFree + (qs - 1) % L::kQStages]);
            }
            if (any) {
                // every product has completed before the tensor memory is released
                tc_commit(&bars[L::bDrain + mine]);
                int dummy = 0;
                mbar_wait(&bars[L::bDrain + mine], 0, &dummy, 50000000ull);
            }
        }
        __syncwarp();
    } else if (warp < kSumWarps) {
        // ---------------------------------------------------------------- exponentials and sums
        const int tile = warp >> 2, quarter = warp & 3, mine = tile * kTileTok + quarter * 32 + lane;
        const uint32_t from = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)tile * 128;
        bool go = true, fresh = true;
        int qs = 0;
        uint32_t uses = 0;                // of the tile's buffer
        int piece = at.whole ? 1 : 0;  // place of a partial sum: 0 for the unit that an earlier run began, 1 for the last one
        while (go) {
            const int first = at.u * p.unit_tok + tile * kTileTok, tok = at.u * p.unit_tok + mine;
            const bool there = tile < at.tiles(p);
            float total = 0.0f;
            for (int r = at.r; r < at.end; ++r) {
                if (fresh) ++qs;
                const int ls = (qs - 1) % L::kLseStages, i0 = at.query(p, r), rows = at.rows(p, r);
                // (not the barrier of q: its stage may have been filled twice since)
                if (!(go = __all_sync(0xffffffffu, mbar_wait(&bars[L::bL + ls], (uint32_t)((qs - 1) / L::kLseStages & 1), abort_flag, wd)))) break;
                const float* lse2 = reinterpret_cast<const float*>(smem + L::kLseOff + ls * L::kLseStage);
                const float* factor = lse2 + kBlockRows;
                const int* last = reinterpret_cast<const int*>(lse2 + 2 * kBlockRows);
                if (there && first <= at.top(p, i0)) {
                    // the first row sees the fewest tokens
                    const bool mixed = odd_rows[ls] != 0 || at.s.ctx + i0 < first + kTileTok - 1;
                    if (!(go = __all_sync(0xffffffffu, mbar_wait(&bars[L::bS + tile], uses++ & 1, abort_flag, wd)))) break;
                    tc_fence_after();
                    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    auto add = [&](auto masked) {
#pragma unroll 1
                        for (int c = 0; c < rows; c += 32) {
                            uint32_t x[32];
                            tmem_ld32(from + c, x);
                            tc_wait_ld();
                            reg_fence(x);
                            if (c + 32 >= rows) {  // (the next products need not wait for the last exponentials)
                                tc_fence_before();
                                __syncwarp();
                                if (lane == 0) mbar_arrive(&bars[L::bSFree + tile]);
                            }
#pragma unroll
                            for (int e = 0; e < 32; e += 4) {
                                float y[4];
                                if constexpr (FOLD) {
                                    fmul2(y[0], y[1], __uint_as_float(x[e]), __uint_as_float(x[e + 1]), p.scale_log2, p.scale_log2);
                                    fmul2(y[2], y[3], __uint_as_float(x[e + 2]), __uint_as_float(x[e + 3]), p.scale_log2, p.scale_log2);
                                } else {
                                    const float4 l = *reinterpret_cast<const float4*>(lse2 + c + e);
                                    float4 f = make_float4(p.scale_log2, p.scale_log2, p.scale_log2, p.scale_log2);
                                    if constexpr (F8) f = *reinterpret_cast<const float4*>(factor + c + e);
                                    ffma2(y[0], y[1], __uint_as_float(x[e]), __uint_as_float(x[e + 1]), f.x, f.y, l.x, l.y);
                                    ffma2(y[2], y[3], __uint_as_float(x[e + 2]), __uint_as_float(x[e + 3]), f.z, f.w, l.z, l.w);
                                }
#pragma unroll
                                for (int z = 0; z < 4; ++z) y[z] = ex2_mufu(y[z]);
                                if constexpr (decltype(masked)::value) {
                                    const int4 m = *reinterpret_cast<const int4*>(last + c + e);
                                    y[0] = tok <= m.x ? y[0] : 0.0f;
                                    y[1] = tok <= m.y ? y[1] : 0.0f;
                                    y[2] = tok <= m.z ? y[2] : 0.0f;
                                    y[3] = tok <= m.w ? y[3] : 0.0f;
                                }
                                fadd2(sum[0], sum[1], sum[0], sum[1], y[0], y[1]);
                                fadd2(sum[2], sum[3], sum[2], sum[3], y[2], y[3]);
                            }
                        }
                    };
                    if (mixed)
                        add(std::true_type{});
                    else
                        add(std::false_type{});
                    total += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                }
                fresh = true;
                if (r + 1 < at.end) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars[L::bLFree + ls]);
                }
            }
            if (!go) break;
            if (at.complete() && at.whole) {
                int slot;
                if (tok < at.s.len && mine < p.unit_tok) {
                    const int page = score_place(p, p.page_table + (long long)at.b * p.max_pages, tok, slot);
                    if (page >= 0) {
                        float* to = score_slot(p, page, slot, at.h);
                        *to = p.decay != 0.0f && tok < at.s.ctx ? fmaf(p.decay, *to, total) : total;
                    }
                }
            } else {
                p.partial[((long long)blockIdx.x * 2 + piece) * kUnitTok + mine] = total;
            }
            piece = 1;
            if (at.left == 0) break;
            fresh = at.next(p);
            if (fresh) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[L::bLFree + (qs - 1) % L::kLseStages]);
            }
        }
    }

    // -------------------------------------------------------------------- end
    __syncwarp();
    tc_fence_before();
    named_bar_sync(1, kTileThreads);
    tc_fence_after();
    if (warp == kProductWarp) tmem_dealloc(tmem, 512);
    if (threadIdx.x == 0 && *abort_flag) atomicCAS(p.status, 0, kDevTimeout);
}

// Units that lie in more than one run: the block whose run begins one adds the parts up in order. Before its wait it reads only what
// kernels before score_tiles_kernel wrote, which have ended: every block of that one knows it before it lets this one start.
__global__ void __launch_bounds__(kUnitTok) score_join_kernel(const __grid_constant__ ScoreParams p) {
    __shared__ long long sums[kUnitTok / 32], out[2];
    const TaskRun run = task_run<kUnitTok>(p, blockIdx.x, sums, out);
    // the unit of the run's last task
    bool there = run.count > 0;
    long long begin = 0, end = 0;
    float* to = nullptr;
    float old = 0.0f;
    if (there) {
        long long rest = run.rest + run.count - 1;
        int b = run.b;
        for (long long n; rest >= (n = tasks_of(p, b)); ++b) rest -= n;
        const UnitWalk at(p, b, rest, 1);
        begin = run.from + run.count - 1 - (at.r - at.seq.first(at.u)), end = begin + at.seq.blocks - at.seq.first(at.u);
        const int tok = at.u * p.unit_tok + threadIdx.x;
        there = begin >= run.from && end > run.from + run.count && tok < at.s.len && (int)threadIdx.x < p.unit_tok;
        if (there) {
            int slot;
            const int page = score_place(p, p.page_table + (long long)at.b * p.max_pages, tok, slot);
            there = page >= 0;
            if (there) to = score_slot(p, page, slot, at.h);
            if (there && p.decay != 0.0f && tok < at.s.ctx) old = p.decay * *to;  // (no other block writes it)
        }
    }
    grid_dependency_wait();
    if (!there) return;
    float total = p.partial[((long long)blockIdx.x * 2 + 1) * kUnitTok + threadIdx.x];
    for (long long c = blockIdx.x + 1; c * run.each < end; ++c) total += p.partial[c * 2 * kUnitTok + threadIdx.x];
    *to = old + total;
}

template <int D, int FMT, bool FOLD>
cudaError_t launch_tiles(ScoreParams p, cudaStream_t stream) {
    using L = ScoreLayout<D, FMT, FOLD>;
    constexpr int bytes = L::kBytes, elem = L::kF8 ? 1 : 2;
    static std::atomic<bool> attr_set[kMaxAttrDevices];
    cudaError_t e = ensure_smem_attr(score_tiles_kernel<D, FMT, FOLD>, bytes, attr_set);
    if (e != cudaSuccess) return e;
    p.box_rows = p.page_size % 64 == 0 ? 64 : (p.page_size % 16 == 0 ? 16 : 1);
    // Units of 512 tokens read q half as often as units of 256, but there have to be units (of full tables, or tasks of them) for all SMs.
    const long long blocks = ((long long)p.max_q + p.block_tok - 1) / p.block_tok * p.head_blocks;
    const long long capacity = (long long)p.max_pages * p.page_size, heads = (long long)p.B * p.Hkv;
    p.unit_tok = kUnitTok;
    auto tasks = [&]() { return heads * ((capacity + p.unit_tok - 1) / p.unit_tok) * (blocks < p.num_sms ? blocks : p.num_sms); };
    while (p.unit_tok > kTileTok && tasks() < p.num_sms) p.unit_tok /= 2;
    p.unit_shift = p.unit_tok == 512 ? 9 : p.unit_tok == 256 ? 8 : 7;
    p.unit_blocks = Divisor(p.unit_tok / p.block_tok);
    const unsigned grid = (unsigned)(tasks() < p.num_sms ? tasks() : p.num_sms);  // no more blocks than tasks
    p.grid = Divisor((int)grid);
    // memory of the call: partial sums (unless a unit is one task), factors and parts of q
    const size_t rows = (size_t)p.T * p.Hq;
    const size_t n_partial = blocks > 1 ? (size_t)grid * 2 * kUnitTok : 0, n_factor = L::kF8 ? (rows + 3) / 4 * 4 : 0;
    const size_t ws_bytes = (n_partial + n_factor) * sizeof(float) + (L::kF8 ? rows * 2 * D : 0);
    void* ws = nullptr;
    uint8_t* parts = nullptr;
    if (ws_bytes > 0) {
        cudaMemPool_t pool = nullptr;
        if (current_device_pool(&pool) != ATTN_OK) return cudaErrorUnknown;
        if ((e = cudaMallocFromPoolAsync(&ws, ws_bytes, pool, stream)) != cudaSuccess) {
            cudaGetLastError();  // (out of memory is no error of the next call)
            return e;
        }
        p.partial = static_cast<float*>(ws);
        p.factor = p.partial + n_partial;
        parts = reinterpret_cast<uint8_t*>(p.factor + n_factor);
    }
    CUtensorMap tmQ, tmK;
    const uint64_t q_row = (uint64_t)D * 2;  // bytes of a row of q, in bf16 or in its two parts
    const uint64_t q_dims[3] = {q_row / elem, (uint64_t)p.Hq, (uint64_t)p.T}, q_strides[2] = {q_row, q_row * p.Hq};
    const uint32_t q_box[3] = {(uint32_t)(L::kBox / elem), (uint32_t)(p.G < kBlockRows ? p.G : kBlockRows), (uint32_t)p.block_tok};
    int st = encode_tiled_map(&tmQ, L::kF8 ? (const void*)parts : (const void*)p.q, elem, 3, q_dims, q_strides, q_box);
    if (p.box_rows > 1) {
        const uint64_t k_dims[2] = {(uint64_t)p.Hkv * D, (uint64_t)p.num_pages * p.page_size}, k_strides[1] = {(uint64_t)p.Hkv * D * elem};
        const uint32_t k_box[2] = {(uint32_t)(L::kBox / elem), (uint32_t)p.box_rows};
        if (st == ATTN_OK) st = encode_tiled_map(&tmK, p.k_cache, elem, 2, k_dims, k_strides, k_box);
    } else {
        tmK = tmQ;
    }
    e = st == ATTN_OK ? cudaSuccess : cudaErrorInvalidValue;
    LaunchMode dependent;
    dependent.dependent = true;
    // (split_q_kernel has to be an ordinary launch, not a dependent: the two kernels behind it rely on all earlier work having ended)
    if (L::kF8 && e == cudaSuccess)
        e = launch_kernel(split_q_kernel<D>, dim3((unsigned)((rows * (D / 8) + 255) / 256)), 256, 0, stream, {}, p.q, parts, p.factor, (long long)rows,
                          p.scale_log2);
    if (e == cudaSuccess)
        e = launch_kernel(score_tiles_kernel<D, FMT, FOLD>, dim3(grid), kTileThreads, bytes, stream, dependent, p, tmQ, tmK);
    if (e == cudaSuccess && n_partial > 0) e = launch_kernel(score_join_kernel, dim3(grid), kUnitTok, 0, stream, dependent, p);
    if (ws) cudaFreeAsync(ws, stream);
    return e;
}

template <int D>
cudaError_t launch_fmt(const ScoreParams& p, int fmt, cudaStream_t stream) {
    // Minus the LSE comes with the products where the scale lets it keep its 24 bits in three bf16 parts.
    const bool fold = fabsf(p.scale_log2) > 0x1p-60f && fabsf(p.scale_log2) < 0x1p60f;
    return fmt == ATTN_FP8_E4M3   ? launch_tiles<D, ATTN_FP8_E4M3, false>(p, stream)
           : fmt == ATTN_FP8_E5M2 ? launch_tiles<D, ATTN_FP8_E5M2, false>(p, stream)
           : fold                 ? launch_tiles<D, ATTN_KV_BF16, true>(p, stream)
                                  : launch_tiles<D, ATTN_KV_BF16, false>(p, stream);
}

}  // namespace

cudaError_t launch_score_tiles(const ScoreParams& p_in, int d, int kv_format, cudaStream_t stream) {
    ScoreParams p = p_in;
    // a block of rows: the heads of as many queries as fit, or 128 heads of one
    p.block_tok = p.G <= kBlockRows ? kBlockRows / p.G : 1;
    p.by_block_tok = Divisor(p.block_tok);
    p.head_blocks = (p.G + kBlockRows - 1) / kBlockRows;
    p.unit = (float)(-1.4426950408889634 / (double)p.scale_log2);
    return d == 128 ? launch_fmt<128>(p, kv_format, stream) : launch_fmt<64>(p, kv_format, stream);
}

}  // namespace attn
