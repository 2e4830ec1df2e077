// Attention weight per cached token, accumulated: score[t, h] = decay score[t, h] + sum over the rows that see
// token t and the query heads of kv head h of exp(scale q.k - lse); the rows' own tokens have no old sum. This file: argument checks, and the kernel for up to
// score_few_rows rows per kv head (32 of 64 elements, 24 of 128; a decode step has one row times the query heads of a kv head).
//
// With few rows the keys are read once and little is computed with them: the kernel is bounded by the memory. So a
// warp reads K from the cache straight into the operand registers of mma.sync m16n8k16: 16 tokens are the rows of
// A, the queries the columns of B. The order of the columns of K inside the sum is free, as long as q has the same: a
// lane takes the 16 bytes that it loads of a token as its elements of two (8-bit codes: four) products. The next 16
// tokens (narrower rows: 32) are loaded while these are multiplied, and the page table is read one group ahead of them. A block's warps take
// the kv heads of the same tokens, so a cache row is read as a whole.
//
// Measured, 64 sequences of U[1K, 32K] tokens, 32/8 heads of 128: bf16 324-328 us, 6800 GB/s (the rate of a copy); e4m3 182-186 us, 6200 GB/s (loads that
// the warps wait for, 20 on an SM). 48 x U[1, 8000], 1-6 rows of 4 heads x 3 heads of 64, e5m2, pages of 7: 21 us for 41 MB, a
// chain of dependent loads in one wave of blocks (without the exponentials of rows that a sequence has not, or with the keys loaded before the rows:
// no change). 48 x U[5333, 16000] tokens, 8 heads: 16 rows of 64 bf16 88 us, e4m3 67 us (floors 75 and 40); 24 rows of 64 102 and 82 (75, 40); 16 of 128
// 165 and 100 (146, 75); 24 of 128 171 and 117 (146, 75): q's operands in registers leave 12 to 20 warps on an SM, which wait for keys.
//
// Work order. When the blocks of all sequences' full tables run at once, a block has a piece of a sequence. Else the tokens that there are,
// of all sequences one after the other, are dealt out in equal runs to as many blocks as the SMs hold: every SM is busy to the end, however
// ragged the lengths (pieces of 1024 tokens: 64 sequences of U[1K, 32K] x 8 heads of 128 361 us, with e4m3 282 us). What pieces cost where tables are
// much wider than the sequences, which leaves most blocks without tokens: one of 2000 tokens, 8 heads of 128, 4.4 us in a tight table, 7.5 in one of
// 32768, 15.4 in one of 131072; sixteen of U[500, 2000] 9.8 and 10.3.
#include "score.cuh"

#include <float.h>
#include <string.h>

namespace attn {
namespace {

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two 8-bit codes in the low (or high) half of w as an f16 pair; e5m2 is the upper byte of an f16.
template <int FMT>
__device__ __forceinline__ uint32_t widen(uint32_t w, int high) {
    if constexpr (FMT == ATTN_FP8_E5M2) {
        return __byte_perm(w, 0, high ? 0x3424 : 0x1404);
    } else {
        const uint16_t v = (uint16_t)(high ? w >> 16 : w);
        uint32_t d;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(v));
        return d;
    }
}

__device__ __forceinline__ uint32_t half_pair(uint32_t bf16_pair, float factor) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(__uint_as_float(bf16_pair & 0xFFFF0000u) * factor), "f"(__uint_as_float(bf16_pair << 16) * factor));
    return r;
}

constexpr int kRowWarps = 8;  // warps per block, at most

// Tokens of a warp's step in 16s: 2 KB of keys at least. (64 sequences of U[1K, 32K] x 8 heads of 128, e4m3: one 236 us, two 194; 48 of
// U[5333, 16000] x 8 heads of 64, bf16: one 129 us, two 92; e4m3: two 77, four 74, but with 24 rows their registers spill: 29 us, not 26.)
template <int D, bool F8>
constexpr int kRowGroups = D == 128 && !F8 ? 1 : 2;
// Registers of a thread: 80 (24 warps on an SM), 96 (20), 128 (16) or 160 (12), as many warps as do without many spilled registers. (64 sequences of U[1K, 32K] x 8
// heads of 128, e4m3, one row of 4 heads: 80 212 us, 96 186, 128 198, and with two steps loaded ahead instead of one 208. 48 of U[5333, 16000] x 8
// heads of 64, 16 rows: 96 88 us, e4m3 67, 128 96 and 75; 24 rows 132 and 81, 128 102 and 81. Of 128,
// 24 rows, e4m3: 128 142, 160 117; bf16 128 171, 160 191.)
template <int D, bool F8, int NT>
constexpr int kRowRegs = NT == 1 ? (D == 64 || !F8 ? 80 : 96) : D == 64 && NT == 2 ? 96 : D == 128 && F8 && NT == 3 ? 160 : 128;

// Tokens of a sequence in steps of a block.
__device__ __forceinline__ int steps_of(const ScoreParams& p, int b, int step) {
    ScoreSeq s;
    return score_seq(p, b, s) ? (s.len + step - 1) / step : 0;
}

// NT: groups of 8 rows.
template <int D, int FMT, int NT>
__global__ void __maxnreg__((kRowRegs<D, FMT != ATTN_KV_BF16, NT>)) score_rows_kernel(const __grid_constant__ ScoreParams p) {
    grid_dependents_launch();
    grid_dependency_wait();
    constexpr bool F8 = FMT != ATTN_KV_BF16;
    constexpr int TG = kRowGroups<D, F8>, TE = 2 * TG;  // groups of 16 tokens, of 8
    constexpr int kLoads = F8 ? D / 64 : D / 32;     // 16-byte loads of a lane per token
    constexpr int kSteps = D / 16;                   // products
    constexpr int kPer = kSteps / kLoads;            // of each load
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int heads = p.row_heads, warps = blockDim.x >> 5, parts = warps / heads;
    const int h = blockIdx.y * heads + warp % heads, part = warp / heads;
    const int step = 16 * TG * parts;  // tokens of a block's step

    // the block's tokens: [begin, begin + left) steps from sequence b on
    int b, begin, left;
    if (p.chunks > 0) {
        b = (int)(blockIdx.x / (unsigned)p.chunks);
        begin = (int)(blockIdx.x % (unsigned)p.chunks) * (p.chunk / step);
        left = min(p.chunk / step, steps_of(p, b, step) - begin);
    } else {
        __shared__ long long sums[kRowWarps], first[2];
        const int per = (p.B + (int)blockDim.x - 1) / (int)blockDim.x, b0 = min(p.B, (int)threadIdx.x * per), b1 = min(p.B, b0 + per);
        long long mine = 0;
        for (int x = b0; x < b1; ++x) mine += steps_of(p, x, step);
        long long upto = mine, total = 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
        }
        if (lane == 31) sums[warp] = upto;
        __syncthreads();
        for (int w = 0; w < warps; ++w) {
            if (w == warp) upto += total;
            total += sums[w];
        }
        const long long each = (total + gridDim.x - 1) / gridDim.x, from = each * blockIdx.x;
        if (from >= total) return;
        if (from >= upto - mine && from < upto) {
            long long rest = from - (upto - mine);
            int x = b0;
            for (int n; rest >= (n = steps_of(p, x, step)); ++x) rest -= n;
            first[0] = x, first[1] = rest;
        }
        __syncthreads();
        b = (int)first[0];
        begin = (int)first[1];
        left = (int)min(each, total - from);
    }
    if (h >= p.Hkv) return;

    for (; left > 0; ++b, begin = 0) {
        ScoreSeq s;
        if (!score_seq(p, b, s)) continue;
        const int take = min(left, (s.len + step - 1) / step - begin);
        const int t_begin = begin * step, t_end = min(s.len, (begin + take) * step), R = s.n * p.G;
        left -= take;
        const int* pt = p.page_table + (long long)b * p.max_pages;

        // rows g, g + 8, ...: their operands, then for the columns 2 t, 2 t + 1 that this lane gets: factor of the scores, LSE,
        // last token seen
        uint32_t qb[NT][kSteps][2];
        float factor[NT][2], lse2[NT][2];
        int last[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = g + 8 * n, i = r / p.G;
            const bool valid = r < R;
            const uint4* src = reinterpret_cast<const uint4*>(p.q + ((long long)(s.q0 + i) * p.Hq + h * p.G + (r - i * p.G)) * D);
            uint4 w[D / 32];  // bf16: the lane's 8 elements of 32; 8-bit caches: 16 elements of 64
#pragma unroll
            for (int x = 0; x < D / 32; ++x)
                w[x] = valid ? src[F8 ? (x >> 1) * 8 + 2 * t + (x & 1) : 4 * x + t] : make_uint4(0, 0, 0, 0);
            float up = 1.0f;
            if constexpr (F8) {
                // a power of two brings the row's largest magnitude into [2^14, 2^15)
                uint32_t top = 0;
#pragma unroll
                for (int x = 0; x < D / 32; ++x) {
                    const uint32_t e[4] = {w[x].x, w[x].y, w[x].z, w[x].w};
#pragma unroll
                    for (int y = 0; y < 4; ++y) top = max(top, max(e[y] & 0x7FFFu, (e[y] >> 16) & 0x7FFFu));
                }
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // (biased exponent 127 + 14 + 127 - exponent; the tiniest rows as far as a float reaches; 255: not finite)
                const int exponent = (int)(top >> 7);
                if (exponent < 255 && top != 0) up = __uint_as_float((unsigned)min(254, 268 - exponent) << 23);
            }
#pragma unroll
            for (int x = 0; x < D / 32; ++x) {
                const uint32_t e[4] = {w[x].x, w[x].y, w[x].z, w[x].w};
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    qb[n][2 * x + y][0] = F8 ? half_pair(e[2 * y], up) : e[2 * y];
                    qb[n][2 * x + y][1] = F8 ? half_pair(e[2 * y + 1], up) : e[2 * y + 1];
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int rc = 2 * t + e + 8 * n, ic = rc / p.G;
                const float l = rc < R ? p.lse[(long long)(s.q0 + ic) * p.Hq + h * p.G + (rc - ic * p.G)] : -INFINITY;
                last[n][e] = l == -INFINITY ? -1 : s.ctx + ic;  // (such rows saw nothing)
                lse2[n][e] = l == -INFINITY ? 0.0f : l * 1.4426950408889634f;
                const float of_row = __shfl_sync(0xffffffffu, up, (2 * t + e) * 4);
                factor[n][e] = F8 ? p.scale_log2 / of_row : p.scale_log2;
            }
        }

        // Of the step's tokens this lane looks up, and keeps the sum of, token g + 8 t.
        struct Place {
            int page, slot;
        };
        auto look_up = [&](int t0, Place& at) { at.page = t < TE && t0 + g + 8 * t < t_end ? score_place(p, pt, t0 + g + 8 * t, at.slot) : -1; };
        uint4 kv[TE][kLoads];
        float old = 0.0f;
        auto load = [&](const Place& at, int from) {
            const int row = at.page >= 0 ? at.page * p.page_size + at.slot : -1;
#pragma unroll
            for (int e = 0; e < TE; ++e) {
                const int x = __shfl_sync(0xffffffffu, row, (lane & 28) + e);
                const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.k_cache) + ((long long)x * p.Hkv + h) * (F8 ? D : 2 * D));
#pragma unroll
                for (int y = 0; y < kLoads; ++y) kv[e][y] = x >= 0 ? src[4 * y + t] : make_uint4(0, 0, 0, 0);
            }
            if (p.decay != 0.0f) old = row >= 0 && from + g + 8 * t < s.ctx ? p.decay * *score_slot(p, at.page, at.slot, h) : 0.0f;
        };
        Place now, next;
        int t0 = t_begin + 16 * TG * part;
        look_up(t0, now);
        look_up(t0 + step, next);
        load(now, t0);
        for (; t0 < t_end; t0 += step) {
            float acc[TG][NT][4];
#pragma unroll
            for (int c = 0; c < TG; ++c)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[c][n][e] = 0.0f;
#pragma unroll
            for (int c = 0; c < TG; ++c)
#pragma unroll
                for (int x = 0; x < kLoads; ++x) {
                    const uint4 l4 = kv[2 * c][x], h4 = kv[2 * c + 1][x];
                    const uint32_t lo[4] = {l4.x, l4.y, l4.z, l4.w}, hi[4] = {h4.x, h4.y, h4.z, h4.w};
#pragma unroll
                    for (int y = 0; y < kPer; ++y) {
                        uint32_t a[4];
                        if constexpr (F8) {
                            a[0] = widen<FMT>(lo[y], 0), a[1] = widen<FMT>(hi[y], 0);
                            a[2] = widen<FMT>(lo[y], 1), a[3] = widen<FMT>(hi[y], 1);
                        } else {
                            a[0] = lo[2 * y], a[1] = hi[2 * y], a[2] = lo[2 * y + 1], a[3] = hi[2 * y + 1];
                        }
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            if constexpr (F8)
                                mma_f16_16816(acc[c][n], a, qb[n][x * kPer + y][0], qb[n][x * kPer + y][1]);
                            else
                                mma_bf16_16816(acc[c][n], a, qb[n][x * kPer + y][0], qb[n][x * kPer + y][1]);
                        }
                    }
                }
            const float before = old;
            const Place mine = now;
            now = next;
            look_up(t0 + 2 * step, next);
            load(now, t0 + step);
            float sum[TE];
#pragma unroll
            for (int e = 0; e < TE; ++e) sum[e] = 0.0f;
#pragma unroll
            for (int c = 0; c < TG; ++c)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float x0 = ex2_mufu(fmaf(acc[c][n][e], factor[n][e], -lse2[n][e]));
                        const float x1 = ex2_mufu(fmaf(acc[c][n][2 + e], factor[n][e], -lse2[n][e]));
                        sum[2 * c] += t0 + 16 * c + g <= last[n][e] ? x0 : 0.0f;
                        sum[2 * c + 1] += t0 + 16 * c + g + 8 <= last[n][e] ? x1 : 0.0f;
                    }
            // over the columns of the four lanes; lane t keeps tokens g + 8 t
            float total;
            const bool odd = t & 1;
            total = (odd ? sum[1] : sum[0]) + __shfl_xor_sync(0xffffffffu, odd ? sum[0] : sum[1], 1);
            if constexpr (TG == 1) {
                total += __shfl_xor_sync(0xffffffffu, total, 2);
            } else {
                const float upper = (odd ? sum[3] : sum[2]) + __shfl_xor_sync(0xffffffffu, odd ? sum[2] : sum[3], 1);
                total = (t & 2 ? upper : total) + __shfl_xor_sync(0xffffffffu, t & 2 ? total : upper, 2);
            }
            if (mine.page >= 0) *score_slot(p, mine.page, mine.slot, h) = before + total;
        }
    }
}

// Blocks of so many threads of a kernel that an SM of the current device holds; known by device and warps per block. An answer that could not be had
// is not kept: this call goes on with one block, which is slower but right.
template <typename Kernel>
int resident_blocks(Kernel kernel, int device, int threads, std::atomic<int> (&known)[kMaxAttrDevices][kRowWarps + 1]) {
    std::atomic<int>* entry = device >= 0 && device < kMaxAttrDevices ? &known[device][threads / 32] : nullptr;
    int n = entry ? entry->load(std::memory_order_relaxed) : 0;
    if (n > 0) return n;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, 0) != cudaSuccess || n < 1) {
        cudaGetLastError();  // (no error of the next call)
        return 1;
    }
    if (entry) entry->store(n, std::memory_order_relaxed);
    return n;
}

template <int D, int FMT, int NT>
cudaError_t launch_rows(ScoreParams p, cudaStream_t stream) {
    static std::atomic<int> known[kMaxAttrDevices][kRowWarps + 1];
    int device = 0;
    const cudaError_t found = cudaGetDevice(&device);
    if (found != cudaSuccess) return found;
    // Blocks of all heads (8 at most), with as many parts of a step's tokens as fit into 8 warps; smaller ones, of fewer parts or heads, where an SM then
    // holds a quarter more warps. (3 heads of 64, 24 rows, e5m2: blocks of 3 warps, 15 on an SM, 21.2 us, of 6 warps, 12, 24.4. 8 heads of 128, one
    // row of 4 heads, e4m3: blocks of 4 warps, 20, 186 us, of 8, 16, 198; 3 heads of those, 3 warps, 21, 44.8 us, 6 warps, 18, 40.4.)
    auto warps_of = [&](int warps) { return resident_blocks(score_rows_kernel<D, FMT, NT>, device, warps * 32, known) * warps; };
    int heads = p.Hkv < kRowWarps ? p.Hkv : kRowWarps, parts = kRowWarps / heads;
    auto consider = [&](int h, int n) {
        if (warps_of(h * n) * 4 >= warps_of(heads * parts) * 5) heads = h, parts = n;
    };
    for (int n = parts - 1; n > 0; --n) consider(heads, n);
    for (int h = heads / 2; parts == 1 && h > 0 && p.Hkv % h == 0; h /= 2) consider(h, 1);
    p.row_heads = heads;
    const long long groups = (p.Hkv + heads - 1) / heads, capacity = (long long)p.max_pages * p.page_size;
    const int step = 16 * kRowGroups<D, FMT != ATTN_KV_BF16> * parts;
    const long long slots = (long long)p.num_sms * (warps_of(heads * parts) / (heads * parts));
    // pieces of every sequence's table for as many blocks as run at once, a few steps each at least; if that is too many blocks, runs
    long long c = ((long long)p.B * capacity * groups + slots - 1) / slots;
    c = (c + step - 1) / step * step;
    if (c < 2 * step) c = 2 * step;
    const long long pieces = (capacity + c - 1) / c;
    dim3 grid;
    if (pieces * p.B * groups <= slots) {
        p.chunk = (int)c, p.chunks = (int)pieces;
        grid = dim3((unsigned)(pieces * p.B), (unsigned)groups);
    } else {
        p.chunk = p.chunks = 0;
        const long long x = slots / groups;
        grid = dim3((unsigned)(x > 0 ? x : 1), (unsigned)groups);
    }
    return launch_kernel(score_rows_kernel<D, FMT, NT>, grid, (unsigned)(heads * parts * 32), 0, stream, {true}, p);
}

template <int D, int FMT>
cudaError_t launch_nt(const ScoreParams& p, cudaStream_t stream) {
    const long long rows = (long long)p.max_q * p.G;
    return rows <= 8    ? launch_rows<D, FMT, 1>(p, stream)
           : rows <= 16 ? launch_rows<D, FMT, 2>(p, stream)
           : rows <= 24 ? launch_rows<D, FMT, 3>(p, stream)
                        : launch_rows<D, FMT, D == 64 ? 4 : 3>(p, stream);  // (128: no more rows come here)
}

template <int D>
cudaError_t launch_fmt(const ScoreParams& p, int fmt, cudaStream_t stream) {
    return fmt == ATTN_FP8_E4M3   ? launch_nt<D, ATTN_FP8_E4M3>(p, stream)
           : fmt == ATTN_FP8_E5M2 ? launch_nt<D, ATTN_FP8_E5M2>(p, stream)
                                  : launch_nt<D, ATTN_KV_BF16>(p, stream);
}

bool multiple(const void* p, long long bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

}  // namespace

cudaError_t launch_score_rows(const ScoreParams& p, int d, int kv_format, cudaStream_t stream) {
    return d == 128 ? launch_fmt<128>(p, kv_format, stream) : launch_fmt<64>(p, kv_format, stream);
}

}  // namespace attn

extern "C" attn_status_t attn_kv_score_paged(const void* q, const float* lse, const void* k_cache, float* score, const int* page_table,
                                             const int* seqlens, const int* cu_seqlens, int page_size, int T, int B, int max_q, int Hq,
                                             int Hkv, int d, int max_pages_per_seq, int num_pages, float scale, float decay,
                                             int kv_format, float k_descale, void* stream) {
    using namespace attn;
    if (!q || !lse || !k_cache || !score || !page_table || !seqlens) return ATTN_ERR_NULL_PTR;
    if (kv_format != ATTN_FP8_E4M3 && kv_format != ATTN_FP8_E5M2 && kv_format != ATTN_KV_BF16) return ATTN_ERR_BAD_ARG;
    if (!isfinite(k_descale) || !isfinite(decay)) return ATTN_ERR_BAD_ARG;
    if (T < 0 || B < 0 || B > 65535 || max_q < 1 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || Hkv > 65535 || (d != 64 && d != 128) ||
        page_size <= 0 || max_pages_per_seq <= 0 || num_pages <= 0)
        return ATTN_ERR_BAD_SHAPE;
    if ((long long)num_pages * page_size > INT32_MAX) return ATTN_ERR_BAD_SHAPE;  // cache rows are 32-bit indices
    if ((long long)max_pages_per_seq * page_size > INT32_MAX / 2 || (long long)T * Hq > INT32_MAX) return ATTN_ERR_BAD_SHAPE;
    if (!cu_seqlens && T > 0 && (B == 0 || T % B != 0 || T / B > max_q)) return ATTN_ERR_BAD_SHAPE;
    if (!isfinite(scale)) return ATTN_ERR_BAD_SHAPE;
    if (!multiple(q, 16) || !multiple(k_cache, 16) || !multiple(lse, 4) || !multiple(score, 4) || !multiple(page_table, 4) ||
        !multiple(seqlens, 4) || (cu_seqlens && !multiple(cu_seqlens, 4)))
        return ATTN_ERR_ALIGN;
    const double factor = (double)scale * (kv_format == ATTN_KV_BF16 ? 1.0 : (double)k_descale) * 1.4426950408889634;
    if (!(fabs(factor) <= (double)FLT_MAX)) return ATTN_ERR_BAD_ARG;  // a float in the kernels
    if (B == 0 || T == 0) return ATTN_OK;
    ScoreParams p;
    memset(&p, 0, sizeof p);
    const attn_status_t st = current_device_info(&p.status, &p.num_sms);
    if (st != ATTN_OK) return st;
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.lse = lse;
    p.k_cache = k_cache;
    p.score = score;
    p.page_table = page_table;
    p.seqlens = seqlens;
    p.cu_seqlens = cu_seqlens;
    p.B = B, p.T = T;
    p.max_q = cu_seqlens ? (max_q < T ? max_q : T) : T / B;
    p.Hq = Hq, p.Hkv = Hkv, p.G = Hq / Hkv;
    p.page_size = page_size, p.max_pages = max_pages_per_seq, p.num_pages = num_pages;
    p.scale_log2 = (float)factor;
    p.decay = decay;
    p.watchdog_ns = watchdog_ns();
    p.by_page = Divisor(page_size);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = (long long)p.max_q * p.G <= score_few_rows(d) ? launch_score_rows(p, d, kv_format, s) : launch_score_tiles(p, d, kv_format, s);
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}
