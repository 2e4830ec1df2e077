// Attention weight per cached token for more than 16 rows per kv head (the last queries of a prompt, or all of them):
// 128-row tiles on the tcgen05 tensor cores.
//
// The transposed scores S^T = K Q^T have the tokens as rows of the accumulator, so that a thread owns a token: it
// reads its row of S^T from tensor memory, adds exp2(scale s - lse) over the columns, and needs no sum across threads. A unit of
// work is 256 tokens of a (sequence, kv head), two accumulator tiles that share the operand Q; a task is a unit times a
// block of 128 rows (queries x query heads, in the order of q) that see any of it. The tasks of the whole call, in the order
// sequence, kv head, tokens, rows, are dealt out in equal runs to one persistent block per SM. A unit that lies in more than
// one run leaves partial sums, which a second kernel adds in order.
//
// What bounds it. With d = 128 a task is 2 x 8 products of 128 x 128 x 16, 1024 clocks of the tensor pipe, and 32768
// exponentials, 1024 clocks of the MUFU; rows that stay the same (up to 128) against new tokens every task are 64 KB of bf16
// keys for that, more than the memory delivers in the time.
//
// Roles of the warps: 0-3 and 4-7 exponentials and sums, a group per accumulator tile (two buffers each, so that the
// products of a task run during the exponentials of the one before); 8-11 loads (16-byte asynchronous copies of rows that the page
// table gives, so any page size); 12 the products, issued by one thread.
//
// 8-bit caches: K is multiplied as it is (kind::f8f6f4), each row of Q scaled by a power of two and split into two e4m3
// parts: exact unless an element is more than 2^9 below the row's largest (then off by at most 2^-17 of that).
#include "score.cuh"

namespace attn {
namespace {

constexpr int kTileTok = 128, kUnitTok = 2 * kTileTok;  // tokens of an accumulator tile, of a unit
constexpr int kBlockRows = 128;                         // rows of a task
constexpr int kLseStages = 4;
constexpr int kTileThreads = 13 * 32;

template <int D, int FMT>
struct ScoreLayout {
    static constexpr bool kF8 = FMT != ATTN_KV_BF16;
    static constexpr int kRow = kF8 ? D : 2 * D;             // bytes of a key
    static constexpr int kChunk = 128 * (kRow < 128 ? kRow : 128);  // [128 rows x 128 (64) bytes]
    static constexpr int kChunks = kRow > 128 ? 2 : 1;       // of a tile of keys or a 16-bit block of q
    static constexpr int kTile = kChunk * kChunks;
    static constexpr int kQ = kF8 ? 2 * kTile : kTile;       // the block of q, in two parts when 8-bit
    static constexpr int kK = 2 * kTile;                     // keys of a unit
    static constexpr int kKOff = 0;                          // two stages
    static constexpr int kQOff = 2 * kK;                     // two stages
    // per row of a block of q: LSE (times log2 e), factor of the scores, last token seen
    static constexpr int kLseOff = kQOff + 2 * kQ, kLseStage = 3 * kBlockRows * 4;
    static constexpr int kBarOff = kLseOff + kLseStages * kLseStage;
    static constexpr int bK = 0, bKFree = 2, bQ = 4, bQFree = 6, bLFree = 8, bS = bLFree + kLseStages, bSFree = bS + 4;
    static constexpr int bL = bSFree + 4, bDrain = bL + kLseStages, kBars = bDrain + 1;
    // tensor-memory base, abort flag; rows that need their own limits, per lse stage and loading warp; the plan
    static constexpr int kMiscOff = kBarOff + kBars * 8, kOddOff = kMiscOff + 8, kPlanOff = kOddOff + kLseStages * 16;
    static constexpr int kBytes = kPlanOff + 64;
    static_assert(kBarOff % 8 == 0 && kOddOff % 16 == 0 && kBytes <= 232448, "shared memory of an SM");
};

__device__ __forceinline__ void fence_smem_to_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

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

// ---- the tasks of a call

// Tasks of one kv head of a sequence. Unit u (tokens from 256 u on) is seen by the blocks of rows from first(u) on.
struct SeqTasks {
    int units, blocks;
    long long skip;  // first(u) = max(0, 2 G u - skip)
    int G2;
    __device__ __forceinline__ SeqTasks(const ScoreSeq& s, int G) {
        units = (s.len + kUnitTok - 1) / kUnitTok;
        blocks = (int)(((long long)s.n * G + kBlockRows - 1) / kBlockRows);
        // row i G of token 256 u is in block floor((256 u - ctx) G / 128) = 2 G u - ceil(ctx G / 128)
        skip = ((long long)s.ctx * G + kBlockRows - 1) / kBlockRows;
        G2 = 2 * G;
    }
    __device__ __forceinline__ int first(int u) const {
        const long long f = (long long)G2 * u - skip;
        return f > 0 ? (int)f : 0;
    }
    // tasks of the units before u
    __device__ __forceinline__ long long before(int u) const {
        const long long from = skip / G2 + 1;  // the first unit that not all blocks see
        const long long cut = u > from ? (long long)G2 * ((from + u - 1) * (u - from) / 2) - skip * (u - from) : 0;
        return (long long)blocks * u - cut;
    }
};

// Where a task lies: sequence, kv head, unit, block of rows.
struct TaskWalk {
    int b, h, u, r;
    ScoreSeq s;
    SeqTasks seq;
    __device__ __forceinline__ TaskWalk(const ScoreParams& p, int b_, long long rest) : b(b_), s(), seq(s, 1) {
        score_seq(p, b, s);
        seq = SeqTasks(s, p.G);
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
        r = seq.first(u) + (int)(rest - seq.before(u));
    }
    __device__ __forceinline__ bool last_block() const { return r + 1 == seq.blocks; }
    // The next task (there is one). Returns whether the unit changes; q_changes: whether the block of q does.
    __device__ __forceinline__ bool next(const ScoreParams& p, bool& q_changes) {
        const int r0 = r;
        q_changes = true;
        if (++r < seq.blocks) return false;
        if (++u < seq.units) {
            r = seq.first(u);
            q_changes = r != r0;
            return true;
        }
        u = r = 0;
        if (++h < p.Hkv) return true;
        h = 0;
        do ++b;
        while (!score_seq(p, b, s));
        seq = SeqTasks(s, p.G);
        return true;
    }
};

// Tasks of sequence b, all kv heads.
__device__ __forceinline__ long long tasks_of(const ScoreParams& p, int b) {
    ScoreSeq s;
    if (!score_seq(p, b, s)) return 0;
    const SeqTasks t(s, p.G);
    return t.before(t.units) * p.Hkv;
}

// The run of tasks [from, from + count) of block `block`: its first sequence and the task within that. Every thread of the
// block calls it; scratch: 8-byte words for the threads' sums (kWarps) and four results.
struct TaskRun {
    long long each, from, total;  // tasks per block; of this one: its first, and the call's number
    long long rest;               // tasks of sequence b before it
    int b, count;
};
template <int kThreads>
__device__ __forceinline__ TaskRun task_run(const ScoreParams& p, int block, int blocks, long long* sums, long long* out) {
    constexpr int kWarps = kThreads / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (p.B + kThreads - 1) / kThreads, b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) mine += tasks_of(p, b);
    long long upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
    }
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    long long total = 0;
    for (int w = 0; w < kWarps; ++w) {
        if (w == warp) upto += total;
        total += sums[w];
    }
    TaskRun run;
    run.total = total;
    run.each = (total + blocks - 1) / blocks;
    run.from = run.each * block;
    const long long left = total - run.from;
    run.count = (int)(left < run.each ? (left > 0 ? left : 0) : run.each);
    const long long ahead = upto - mine;
    if (run.count > 0 && run.from >= ahead && run.from < upto) {
        long long rest = run.from - ahead;
        int b = b0;
        for (long long n; rest >= (n = tasks_of(p, b)); ++b) rest -= n;
        out[0] = b;
        out[1] = rest;
    }
    __syncthreads();
    run.b = (int)out[0];
    run.rest = out[1];
    return run;
}

template <int D, int FMT>
__global__ void __launch_bounds__(kTileThreads, 1) score_tiles_kernel(const __grid_constant__ ScoreParams p) {
    grid_dependents_launch();
    using L = ScoreLayout<D, FMT>;
    constexpr bool F8 = L::kF8;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
    const TaskRun run = task_run<kTileThreads>(p, blockIdx.x, gridDim.x, reinterpret_cast<long long*>(smem), reinterpret_cast<long long*>(smem + L::kPlanOff));
    if (run.count == 0) return;
    if (smem_u32(smem) & 1023u) {  // the swizzles count from such boundaries
        if (threadIdx.x == 0) atomicCAS(p.status, 0, kDevTimeout);
        return;
    }
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMiscOff);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMiscOff + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint64_t wd = p.watchdog_ns;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars[L::bK + i], 4);
            mbar_init(&bars[L::bKFree + i], 1);
            mbar_init(&bars[L::bQ + i], 4);
            mbar_init(&bars[L::bQFree + i], 1);
        }
        for (int i = 0; i < kLseStages; ++i) {
            mbar_init(&bars[L::bL + i], 4);
            mbar_init(&bars[L::bLFree + i], 8);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&bars[L::bS + i], 1);
            mbar_init(&bars[L::bSFree + i], 4);
        }
        mbar_init(&bars[L::bDrain], 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 12) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t base = smem_u32(smem);
    TaskWalk at(p, run.b, run.rest);
    // stages of units and blocks of q are counted from the first of the run
    unsigned unit = 0, qn = 0;

    if (warp >= 8 && warp < 12) {
        // ---------------------------------------------------------------- loads
        const int tid = threadIdx.x - 256;
        uint64_t *pending = nullptr, *pending_lse = nullptr;  // of the load whose copies may still be on their way
        bool ok = true;
        auto hand_over = [&](auto left) {
            if (!pending) return;
            cp_async_wait<decltype(left)::value>();
            fence_smem_to_async();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(pending);
                if (pending_lse) mbar_arrive(pending_lse);
            }
            pending = pending_lse = nullptr;
        };
        // a stage that is not free yet may wait for what this warp has not handed over
        auto wait_free = [&](uint64_t* bar, uint32_t parity) {
            if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity))) return true;
            hand_over(std::integral_constant<int, 0>{});
            return (bool)__all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, wd));
        };
        bool new_unit = true, new_q = true;
        for (int i = 0; ok; ++i) {
            if (new_unit) {
                const int st = unit & 1;
                if (!(ok = wait_free(&bars[L::bKFree + st], (unit >> 1 & 1u) ^ 1u))) break;
                // a thread copies unit tid % kUnits of rows tid / kUnits, + kStep, ...
                constexpr int kUnits = L::kRow / 16, kStep = 128 / kUnits;
                const int* pt = p.page_table + (long long)at.b * p.max_pages;
                const int t0 = at.u * kUnitTok, u = tid % kUnits;
                const uint8_t* keys = static_cast<const uint8_t*>(p.k_cache) + (long long)at.h * L::kRow + 16 * u;
                const uint32_t to = base + L::kKOff + st * L::kK;
#pragma unroll 8
                for (int r = tid / kUnits; r < kUnitTok; r += kStep) {
                    int slot = 0;
                    const int page = t0 + r < at.s.len ? score_place(p, pt, t0 + r, slot) : -1;
                    const long long row = page >= 0 ? (long long)page * p.page_size + slot : 0;
                    cp_async16(to + (r / kTileTok) * L::kTile + unit_at<L::kRow>(r % kTileTok, u), keys + row * p.Hkv * L::kRow, page >= 0 ? 16 : 0);
                }
                cp_async_commit();
                hand_over(std::integral_constant<int, 1>{});
                pending = &bars[L::bK + st];
                ++unit;
            }
            if (new_q) {
                const int st = qn & 1, ls = qn % kLseStages;
                if (!(ok = wait_free(&bars[L::bQFree + st], (qn >> 1 & 1u) ^ 1u))) break;
                if (!(ok = wait_free(&bars[L::bLFree + ls], (qn / kLseStages & 1u) ^ 1u))) break;
                const int rows = (int)min((long long)kBlockRows, (long long)at.s.n * p.G - (long long)at.r * kBlockRows);
                const int r0 = at.r * kBlockRows;  // (below n G < 2^31)
                auto row_of = [&](int r) {
                    const int i = (r0 + r) / p.G;
                    return (long long)(at.s.q0 + i) * p.Hq + at.h * p.G + (r0 + r - i * p.G);
                };
                float* lse2 = reinterpret_cast<float*>(smem + L::kLseOff + ls * L::kLseStage);
                const uint32_t to = base + L::kQOff + st * L::kQ;
                constexpr int kUnits = D / 8, kStep = 128 / kUnits;
                const int u = tid % kUnits;
                if constexpr (!F8) {
#pragma unroll 4
                    for (int r = tid / kUnits; r < kBlockRows; r += kStep)
                        cp_async16(to + unit_at<L::kRow>(r, u), p.q + row_of(r < rows ? r : 0) * D + 8 * u, r < rows ? 16 : 0);
                } else {
                    // 2^up brings the largest magnitude of the row into [128, 256)
#pragma unroll 4
                    for (int r = tid / kUnits; r < kBlockRows; r += kStep) {
                        uint4 w = make_uint4(0, 0, 0, 0);
                        if (r < rows) w = __ldg(reinterpret_cast<const uint4*>(p.q + row_of(r) * D) + u);
                        const uint32_t e[4] = {w.x, w.y, w.z, w.w};
                        uint32_t top = 0;
#pragma unroll
                        for (int y = 0; y < 4; ++y) top = max(top, max(e[y] & 0x7FFFu, (e[y] >> 16) & 0x7FFFu));
#pragma unroll
                        for (int o = 1; o < kUnits; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                        const int exponent = (int)(top >> 7);
                        // (biased exponent 127 + 7 + 127 - exponent; the tiniest rows as far as a float reaches)
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
                        const uint32_t dst = to + unit_at<L::kRow>(r, u >> 1) + 8 * (u & 1);
#pragma unroll
                        for (int x = 0; x < 2; ++x)
                            asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(dst + x * L::kTile), "r"(part[x][0]), "r"(part[x][1]) : "memory");
                        // a row with a non-finite element gives NaN
                        if (u == 0) lse2[kBlockRows + r] = exponent == 255 ? __int_as_float(0x7fffffff) : p.scale_log2 / up;
                    }
                }
                // LSE and last token of row tid; does any row need its own limit besides the causal one?
                const float l = tid < rows ? __ldg(p.lse + row_of(tid)) : -INFINITY;
                lse2[tid] = l == -INFINITY ? 0.0f : l * 1.4426950408889634f;
                reinterpret_cast<int*>(lse2)[2 * kBlockRows + tid] = l == -INFINITY ? -1 : at.s.ctx + (r0 + tid) / p.G;
                const bool odd = __any_sync(0xffffffffu, l == -INFINITY);
                if (lane == 0) reinterpret_cast<int*>(smem + L::kOddOff)[ls * 4 + (tid >> 5)] = odd;
                cp_async_commit();
                hand_over(std::integral_constant<int, 1>{});
                pending = &bars[L::bQ + st];
                pending_lse = &bars[L::bL + ls];
                ++qn;
            }
            if (i + 1 == run.count) break;
            new_unit = at.next(p, new_q);
        }
        hand_over(std::integral_constant<int, 0>{});
        cp_async_wait<0>();
    } else if (warp == 12) {
        // ---------------------------------------------------------------- products
        if (lane == 0) {
            constexpr bool kNarrow = L::kRow == 64;
            auto desc = [&](int off) { return kNarrow ? smem_desc_sw64(base + off) : smem_desc_sw128(base + off, L::kChunk, 1024); };
            const uint64_t dk = desc(L::kKOff), dq = desc(L::kQOff);
            auto wait = [&](int bar, uint32_t parity) { return mbar_wait(&bars[bar], parity, abort_flag, wd); };
            bool any = false, new_unit = true, new_q = true;
            unsigned units = 0, qs = 0;  // stages waited for
            for (int i = 0;; ++i) {
                if (new_unit) {
                    if (!wait(L::bK + (units & 1), units >> 1 & 1u)) break;
                    ++units;
                }
                if (new_q) {
                    if (!wait(L::bQ + (qs & 1), qs >> 1 & 1u)) break;
                    ++qs;
                }
                const int ks = (units - 1) & 1, st = (qs - 1) & 1, buf = i & 1;
                const int rows = (int)min((long long)kBlockRows, (long long)at.s.n * p.G - (long long)at.r * kBlockRows);
                const uint32_t idesc = score_idesc<FMT>((rows + 31) & ~31);
                bool go = true;
#pragma unroll 1
                for (int t = 0; t < 2 && (go = wait(L::bSFree + 2 * t + buf, (unsigned)(i >> 1 & 1) ^ 1u)); ++t) {
                    tc_fence_after();
                    any = true;
                    const uint32_t d = tmem + (uint32_t)(2 * t + buf) * 128;
                    const uint64_t kd = dk + (uint64_t)((ks * L::kK + t * L::kTile) >> 4), qd = dq + (uint64_t)((st * L::kQ) >> 4);
                    if constexpr (F8) {
#pragma unroll
                        for (int x = 0; x < 2 * (D / 32); ++x) {  // both parts of Q
                            const int part = x / (D / 32), k = x % (D / 32);
                            mma8_ss(d, kd + (uint64_t)((k * 32) >> 4), qd + (uint64_t)((part * L::kTile + k * 32) >> 4), idesc, x > 0);
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < D / 16; ++k)
                            tc_mma_ss(d, kd + (uint64_t)(((k >> 2) * L::kChunk + (k & 3) * 32) >> 4),
                                      qd + (uint64_t)(((k >> 2) * L::kChunk + (k & 3) * 32) >> 4), idesc, k > 0);
                    }
                    tc_commit(&bars[L::bS + 2 * t + buf]);
                }
                if (!go) break;
                if (i + 1 == run.count) break;
                new_unit = at.next(p, new_q);
                if (new_q) tc_commit(&bars[L::bQFree + st]);
                if (new_unit) tc_commit(&bars[L::bKFree + ks]);
            }
            if (any) {
                // every product has completed before the tensor memory is released
                tc_commit(&bars[L::bDrain]);
                int dummy = 0;
                mbar_wait(&bars[L::bDrain], 0, &dummy, 50000000ull);
            }
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------------- exponentials and sums
        const int tile = warp >> 2, quarter = warp & 3, mine = tile * kTileTok + quarter * 32 + lane;
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
        bool new_unit = true, new_q = true, whole = at.r == at.seq.first(at.u);
        int piece = whole ? 1 : 0;  // place of a partial sum: 0 for the unit that an earlier run began, 1 for the last one
        unsigned qs = 0;
        float total = 0.0f;
        for (int i = 0;; ++i) {
            if (new_unit) total = 0.0f;
            if (new_q) ++qs;
            const int ls = (qs - 1) % kLseStages, buf = i & 1;
            const int rows = (int)min((long long)kBlockRows, (long long)at.s.n * p.G - (long long)at.r * kBlockRows);
            const int tok = at.u * kUnitTok + mine, first = at.u * kUnitTok + tile * kTileTok;
            // (not the barrier of q: its stage may have been filled twice since)
            if (!__all_sync(0xffffffffu, mbar_wait(&bars[L::bL + ls], (qs - 1) / kLseStages & 1u, abort_flag, wd))) break;
            const float* lse2 = reinterpret_cast<const float*>(smem + L::kLseOff + ls * L::kLseStage);
            const float* factor = lse2 + kBlockRows;
            const int* last = reinterpret_cast<const int*>(lse2 + 2 * kBlockRows);
            const int4 odd = *reinterpret_cast<const int4*>(smem + L::kOddOff + ls * 16);
            // the first row sees the fewest tokens, the last one the most
            const int top = at.s.ctx + (at.r * kBlockRows + rows - 1) / p.G;
            const bool mixed = (odd.x | odd.y | odd.z | odd.w) != 0 || at.s.ctx + at.r * kBlockRows / p.G < first + kTileTok - 1;
            if (!__all_sync(0xffffffffu, mbar_wait(&bars[L::bS + 2 * tile + buf], (unsigned)(i >> 1 & 1), abort_flag, wd))) break;
            tc_fence_after();
            const uint32_t from = tmem + lane_off + (uint32_t)(2 * tile + buf) * 128;
            float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (first <= top && first < at.s.len) {
#pragma unroll 1
                for (int c = 0; c < rows; c += 32) {
                    uint32_t x[32];
                    tmem_ld32(from + c, x);
                    tc_wait_ld();
                    reg_fence(x);
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        const float4 l = *reinterpret_cast<const float4*>(lse2 + c + e);
                        float4 f = make_float4(p.scale_log2, p.scale_log2, p.scale_log2, p.scale_log2);
                        if constexpr (F8) f = *reinterpret_cast<const float4*>(factor + c + e);
                        float y[4];
                        ffma2(y[0], y[1], __uint_as_float(x[e]), __uint_as_float(x[e + 1]), f.x, f.y, -l.x, -l.y);
                        ffma2(y[2], y[3], __uint_as_float(x[e + 2]), __uint_as_float(x[e + 3]), f.z, f.w, -l.z, -l.w);
#pragma unroll
                        for (int z = 0; z < 4; ++z) y[z] = ex2_mufu(y[z]);
                        if (mixed) {
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
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[L::bSFree + 2 * tile + buf]);
            total += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            const bool end = i + 1 == run.count, complete = at.last_block();
            if (complete || end) {
                if (complete && whole) {
                    int slot;
                    if (tok < at.s.len) {
                        const int page = score_place(p, p.page_table + (long long)at.b * p.max_pages, tok, slot);
                        if (page >= 0) {
                            float* to = score_slot(p, page, slot, at.h);
                            *to = p.decay != 0.0f && tok < at.s.ctx ? fmaf(p.decay, *to, total) : total;
                        }
                    }
                } else {
                    p.partial[((long long)blockIdx.x * 2 + piece) * kUnitTok + mine] = total;
                }
                whole = true;
                piece = 1;
            }
            if (end) break;
            new_unit = at.next(p, new_q);
            if (new_q) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[L::bLFree + ls]);
            }
        }
    }

    // -------------------------------------------------------------------- end
    __syncwarp();
    tc_fence_before();
    named_bar_sync(1, kTileThreads);
    tc_fence_after();
    if (warp == 12) tmem_dealloc(tmem, 512);
    if (threadIdx.x == 0 && *abort_flag) atomicCAS(p.status, 0, kDevTimeout);
}

// Units that lie in more than one run: the block whose run begins one adds the parts up in order.
__global__ void __launch_bounds__(kUnitTok) score_join_kernel(const __grid_constant__ ScoreParams p) {
    __shared__ long long sums[kUnitTok / 32], out[2];
    const TaskRun run = task_run<kUnitTok>(p, blockIdx.x, gridDim.x, sums, out);
    if (run.count == 0) return;
    // the unit of the run's last task
    long long rest = run.rest + run.count - 1;
    int b = run.b;
    for (long long n; rest >= (n = tasks_of(p, b)); ++b) rest -= n;
    const TaskWalk at(p, b, rest);
    const long long begin = run.from + run.count - 1 - (at.r - at.seq.first(at.u)), end = begin + at.seq.blocks - at.seq.first(at.u);
    if (begin < run.from || end <= run.from + run.count) return;
    grid_dependency_wait();
    float total = p.partial[((long long)blockIdx.x * 2 + 1) * kUnitTok + threadIdx.x];
    for (long long c = blockIdx.x + 1; c * run.each < end; ++c) total += p.partial[c * 2 * kUnitTok + threadIdx.x];
    const int tok = at.u * kUnitTok + threadIdx.x;
    if (tok >= at.s.len) return;
    int slot;
    const int page = score_place(p, p.page_table + (long long)at.b * p.max_pages, tok, slot);
    if (page < 0) return;
    float* to = score_slot(p, page, slot, at.h);
    *to = p.decay != 0.0f && tok < at.s.ctx ? fmaf(p.decay, *to, total) : total;
}

template <int D, int FMT>
cudaError_t launch_tiles(ScoreParams p, cudaStream_t stream) {
    constexpr int bytes = ScoreLayout<D, FMT>::kBytes;
    static std::atomic<bool> attr_set[kMaxAttrDevices];
    cudaError_t e = ensure_smem_attr(score_tiles_kernel<D, FMT>, bytes, attr_set);
    if (e != cudaSuccess) return e;
    // no more blocks than there can be tasks
    const long long blocks = ((long long)p.max_q * p.G + kBlockRows - 1) / kBlockRows;
    const long long most = (long long)p.B * p.Hkv * (((long long)p.max_pages * p.page_size + kUnitTok - 1) / kUnitTok) * blocks;
    const unsigned grid = (unsigned)(most < p.num_sms ? most : p.num_sms);
    void* ws = nullptr;
    if (blocks > 1) {  // else a unit is one task
        cudaMemPool_t pool = nullptr;
        if (current_device_pool(&pool) != ATTN_OK) return cudaErrorUnknown;
        if ((e = cudaMallocFromPoolAsync(&ws, (size_t)grid * 2 * kUnitTok * sizeof(float), pool, stream)) != cudaSuccess) {
            cudaGetLastError();  // (out of memory is no error of the next call)
            return e;
        }
        p.partial = static_cast<float*>(ws);
    }
    e = launch_kernel(score_tiles_kernel<D, FMT>, dim3(grid), kTileThreads, bytes, stream, {}, p);
    if (e == cudaSuccess && blocks > 1) {
        LaunchMode mode;
        mode.dependent = true;
        e = launch_kernel(score_join_kernel, dim3(grid), kUnitTok, 0, stream, mode, p);
    }
    if (ws) cudaFreeAsync(ws, stream);
    return e;
}

template <int D>
cudaError_t launch_fmt(const ScoreParams& p, int fmt, cudaStream_t stream) {
    return fmt == ATTN_FP8_E4M3   ? launch_tiles<D, ATTN_FP8_E4M3>(p, stream)
           : fmt == ATTN_FP8_E5M2 ? launch_tiles<D, ATTN_FP8_E5M2>(p, stream)
                                  : launch_tiles<D, ATTN_KV_BF16>(p, stream);
}

}  // namespace

cudaError_t launch_score_tiles(const ScoreParams& p, int d, int kv_format, cudaStream_t stream) {
    return d == 128 ? launch_fmt<128>(p, kv_format, stream) : launch_fmt<64>(p, kv_format, stream);
}

}  // namespace attn
