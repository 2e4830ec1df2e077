// Attention of the drafted tokens of each sequence over its paged cache (a tree of drafted tokens,
// or a chain), for sm_103a.
//
// Sequence b has len cached tokens, the last n of them the drafted ones. Row (i, h), drafted token i
// and query head h, sees the first len - n tokens and those drafted tokens j whose bit is set in
// mask[i] (no mask: j <= i); o = softmax(scale q k^T) v over what it sees, with the online-softmax
// recurrence. The n G rows of a kv head (G query heads each) are the rows of one product, so one
// pass over the cache serves all drafted tokens. Several blocks share a long sequence (splits of
// its keys) and their partial results are joined by log-sum-exp: by the blocks themselves where they are a
// cluster, through each other's shared memory (few splits, all blocks fit at once), else by a second kernel.
// The cluster saves a workspace and a launch: one sequence of 1000 tokens 12.3 us per call from Python, 15.4
// with the second kernel; in a captured graph both take 10.3 us.
//
// Masked keys contribute exactly nothing, whatever their slots hold: scores are replaced by -inf,
// and in the key tiles where a row may not see every key the non-finite values of V are taken out of
// the product (0 times NaN would be NaN) and added to the rows that do see them at the end. Rows behind the
// last token cost nothing; non-finite values of drafted tokens 15 to 35 us per 64-token tile that holds any (16
// drafted tokens over 4 sequences of 1000, tiles: 12 us without, 44 us with one NaN; few rows 10 and 25).
#include "launch.cuh"
#include "tree_device.cuh"

#include <float.h>

namespace attn {
namespace {

// ------------------------------------------------------------------------------ few rows
//
// One block of four warps per (sequence, split, kv head, group of 16 rows). Each warp streams its own
// 16-token groups through a private cp.async ring of two to four groups (any page size: each row's address
// comes from the page table), and multiplies with mma.sync, whose 16 rows are the group's rows: for
// up to 16 rows per kv head the kernel is bounded by the cache reads, so a wider product would only add work on
// padding (two groups only where tree_takes_tiles says so). 8-bit codes become f16 pairs in registers (exact); the order of d
// inside both products is permuted so that one 16-byte shared load feeds several products.
// Measured, 64 sequences of U[1K, 32K] tokens, 4 query heads on each of 8 kv heads: one token each 597 us
// (7220 GB/s, 1.06 of the measured copy rate, which also writes), four 608 us; e4m3 329 us (6550 GB/s) and
// 353 us, where the conversions and the shared loads of the products take over. One sequence of 1000 tokens:
// one token 7.4 us, four 10.3 us (before the page table was read a group ahead of the copies, and the merge and
// the join had their loads side by side: 11.0 and 16.1).

constexpr int kWarps = 4;
constexpr int kGroup = 16;

template <int D, int GN, int FMT>
struct SmallLayout {
    static constexpr int kElem = FMT == ATTN_KV_BF16 ? 2 : 1;
    // Token groups in flight per warp. With 128 bf16 elements two, so that three blocks share an SM (three groups and
    // two blocks: 64 sequences of U[100, 1000], 4 drafted tokens 36.7 us, not 33.5; of U[1K, 32K] 0.2% faster); with
    // 8-bit codes four (three: 1% slower over long contexts).
    static constexpr int kStages = D == 64 ? 3 : FMT == ATTN_KV_BF16 ? 2 : 4;
    static constexpr int kRow = D * kElem;         // bytes of a cached row of one head
    static constexpr int kTile = kGroup * kRow;    // one K or V stage of a warp
    static constexpr int kChunks = kRow / 16;
    static constexpr int kRing = kWarps * kStages * 2 * kTile;
    static constexpr int kRowO = D + 4;            // floats of a merged row: eight rows' columns in different banks
    static constexpr int kMerge = (kWarps * 16 * kRowO + 2 * kWarps * 16) * 4;
    static constexpr int kPart = kMerge, kPartLse = kPart + 16 * D * 4;  // the block's result for the cluster's join
    static constexpr int kBytes = kRing > kPartLse + 64 ? kRing : kPartLse + 64;
};

// Byte offset of 16-byte chunk c of row r of a stage tile (rows of kChunks chunks, XOR swizzle).
template <int kChunks>
__device__ __forceinline__ uint32_t swz_chunk(int r, int c) {
    constexpr int m = kChunks < 8 ? kChunks - 1 : 7;
    return (uint32_t)(r * kChunks * 16 + ((c ^ (r & m)) << 4));
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&w)[4]) {
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&w)[2]) {
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr) : "memory");
}

// GN: row slots that hold rows (8 or 16). kCluster: the splits of a group are the blocks of a cluster.
template <int D, int GN, int FMT, bool kCluster>
__global__ void __launch_bounds__(kWarps * 32, tree_small_blocks(D, FMT != ATTN_KV_BF16, GN)) tree_small_kernel(const __grid_constant__ TreeParams p) {
    grid_dependents_launch();
    using L = SmallLayout<D, GN, FMT>;
    constexpr bool F8 = FMT != ATTN_KV_BF16;
    constexpr int kStages = L::kStages;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int odd_v;  // a V tile held a non-finite value that was taken out
    int chunk, b, split, hg;
    if (!tree_item<kCluster>(p, reinterpret_cast<int*>(smem), chunk, b, split, hg)) return;
    const int kvh = hg / p.groups, r0 = (hg % p.groups) * 16;
    TreeSeq s;
    if (!tree_seq(p, b, s)) return;
    const int R = min(16, s.n * p.G - r0);  // rows of this group
    if (R <= 0) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nsplit = cdiv(s.len, chunk);
    if (split < 0)
        split = nsplit > 0 ? nsplit - 1 : 0;
    else if (p.full_rows >= 0 && split >= nsplit - 1)
        return;  // the last split has its own block
    const int t_begin = split * chunk;
    // output row of local row r: (s.q0 + i) * Hq + kvh * G + g with (i, g) = divmod(r0 + r, G)
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
    float* part_o = reinterpret_cast<float*>(smem + L::kPart);
    float* part_lse = reinterpret_cast<float*>(smem + L::kPartLse);
    const long long out_first = (long long)s.q0 * p.Hq + kvh * p.G;
    const bool joins = kCluster && nsplit > 1;  // the same in all blocks of a cluster
    if (t_begin >= s.len) {
        if (joins) cluster_join<D, D>(part_o, part_lse, p.o, p.lse, out_first, r0, R, p.G, p.Hq, p.cluster, nsplit);
        return;
    }
    const int t_end = min(s.len, t_begin + chunk);
    if (threadIdx.x == 0) odd_v = 0;
    __syncthreads();

    const int g0 = lane >> 2, qd = lane & 3;
    const bool v0 = g0 < R, v1 = GN == 16 && g0 + 8 < R;
    // what the lane's two rows see among the drafted tokens; rows of padding see every key
    const int i0 = v0 ? (r0 + g0) / p.G : s.n - 1, i1 = v1 ? (r0 + g0 + 8) / p.G : s.n - 1;
    const unsigned long long* mrow0 = p.mask ? p.mask + (long long)(s.q0 + i0) * p.mask_words : nullptr;
    const unsigned long long* mrow1 = p.mask ? p.mask + (long long)(s.q0 + i1) * p.mask_words : nullptr;

    // ---- the warp's ring: token groups t_begin + 16 (warp + 4 i)
    const uint32_t ring = smem_u32(smem) + warp * kStages * 2 * L::kTile;
    const int* pt = p.page_table + (long long)b * p.max_pages;
    const uint8_t* kc = static_cast<const uint8_t*>(p.k_cache);
    const uint8_t* vc = static_cast<const uint8_t*>(p.v_cache);
    constexpr int kRowsPerIter = 32 / L::kChunks;
    const int my_chunk = lane % L::kChunks, my_row = lane / L::kChunks;
    const long long row_bytes = (long long)p.Hkv * L::kRow;
    const int col = kvh * L::kRow + my_chunk * 16;
    const int total = cdiv(t_end - t_begin, kGroup);
    const int mine = total > warp ? cdiv(total - warp, kWarps) : 0;
    auto row_of = [&](int i) {  // cache row of the lane's token of group i; no token or a bad page: zeros
        const int tok = t_begin + kGroup * (warp + kWarps * i) + (lane & 15);
        return i < mine && tok < t_end ? cache_row(p, pt, tok) : -1;
    };
    auto issue = [&](int i, int row) {
        const uint32_t kd = ring + (i % kStages) * 2 * L::kTile, vd = kd + L::kTile;
#pragma unroll
        for (int it = 0; it < kGroup / kRowsPerIter; ++it) {
            const int r = it * kRowsPerIter + my_row;
            const int rr = __shfl_sync(0xffffffffu, row, r);
            const long long off = rr >= 0 ? rr * row_bytes + col : 0;
            const uint32_t n = rr >= 0 ? 16u : 0u;
            cp_async16(kd + swz_chunk<L::kChunks>(r, my_chunk), kc + off, n);
            cp_async16(vd + swz_chunk<L::kChunks>(r, my_chunk), vc + off, n);
        }
    };
    // (the page table is read a group ahead, so that a copy does not wait for it)
    int rows_at[kStages];
#pragma unroll
    for (int i = 0; i < kStages; ++i) rows_at[i] = row_of(i);
    int next_row = rows_at[kStages - 1];
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
        if (i < mine) issue(i, rows_at[i]);
        cp_async_commit();
    }

    // ---- query fragments. 8-bit caches: column 2 qd + e of k-step kk is d = (D/4) qd + 4 kk + e,
    // column 2 qd + 8 + e is that + 2; and f16, after scaling each row by a power of two that brings its largest
    // magnitude into [2^14, 2^15): exact for elements down to 2^-31 of that, within 2^-39 of it for smaller ones. The
    // power goes back into the row's factor of the scores (exactly), so nothing else notices it.
    uint32_t aq[D / 16][4];
    float s0 = p.scale_log2, s1 = p.scale_log2;  // scores of the lane's two rows to exponents of two
    {
        const uint32_t* q0p = reinterpret_cast<const uint32_t*>(p.q + (v0 ? out_row(g0) : 0) * D);
        const uint32_t* q1p = reinterpret_cast<const uint32_t*>(p.q + (v1 ? out_row(g0 + 8) : 0) * D);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            const int c = F8 ? (D / 8) * qd + 2 * kk : kk * 8 + qd, step = F8 ? 1 : 4;
            aq[kk][0] = v0 ? __ldg(q0p + c) : 0u;
            aq[kk][1] = v1 ? __ldg(q1p + c) : 0u;
            aq[kk][2] = v0 ? __ldg(q0p + c + step) : 0u;
            aq[kk][3] = v1 ? __ldg(q1p + c + step) : 0u;
        }
        float mul[2] = {p.q_sign, p.q_sign};
        if constexpr (F8) {
#pragma unroll
            for (int x = 0; x < GN / 8; ++x) {
                uint32_t top = 0;  // the row's largest magnitude, as bf16
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                    for (int e = x; e < 4; e += 2) top = max(top, max(aq[kk][e] & 0x7FFFu, (aq[kk][e] >> 16) & 0x7FFFu));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int up = top == 0 || top >= 0x7F80u ? 0 : min(120, 141 - (int)(top >> 7));
                mul[x] *= __int_as_float((127 + up) << 23);
                // (a factor that rounds to 0, or to infinity, would turn scores of -inf, or 0, into NaN)
                (x ? s1 : s0) = fminf(fmaxf(p.scale_log2 * __int_as_float((127 - up) << 23), 0x1p-126f), FLT_MAX);
            }
        }
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t w = aq[kk][e];
                const float lo = __uint_as_float(w << 16) * mul[e & 1], hi = __uint_as_float(w & 0xFFFF0000u) * mul[e & 1];
                aq[kk][e] = F8 ? pack_half2(lo, hi) : pack_bf16x2(lo, hi);
            }
    }

    constexpr int NH = GN / 8;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;
    float oacc[NH][D / 16][4] = {};
    const int lm_row = (lane & 7) + ((lane >> 4) << 3), lm_par = (lane >> 3) & 1;

    for (int i = 0; i < mine; ++i) {
        cp_async_wait<kStages - 2>();
        __syncwarp();
        if (i + kStages - 1 < mine) {
            issue(i + kStages - 1, next_row);
            next_row = row_of(i + kStages);
        }
        cp_async_commit();
        const uint32_t kt = ring + (i % kStages) * 2 * L::kTile, vt = kt + L::kTile;
        const int g = t_begin + kGroup * (warp + kWarps * i);

        // S = Q K^T: rows of the group x 16 tokens
        float sc[2][4] = {};
        if constexpr (F8) {
            constexpr int W = D / 64;  // 16-byte chunks of K bytes per lane and token
            uint32_t kw[2][W][4];
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int j = 0; j < W; ++j) lds_words(kt + swz_chunk<L::kChunks>(g0 + 8 * nt, W * qd + j), kw[nt][j]);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
                    const uint32_t w = kw[nt][kk >> 2][kk & 3];
                    mma_f16(sc[nt], aq[kk], fp8x2_f16x2<FMT>(w), fp8x2_f16x2<FMT>(w >> 16));
                }
        } else {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                uint32_t b0, b1, b2, b3;
                ldmatrix_x4(kt + swz_chunk<L::kChunks>(lm_row, 2 * kk + lm_par), b0, b1, b2, b3);
                mma_bf16_16816(sc[0], aq[kk], b0, b1);
                mma_bf16_16816(sc[1], aq[kk], b2, b3);
            }
        }
        if (g + kGroup > s.ctx) {  // drafted tokens, or the end of the sequence
            const uint32_t w0 = (uint32_t)tree_window(mrow0, p.mask_words, i0, s.ctx, s.len, g);
            const uint32_t w1 = (uint32_t)tree_window(mrow1, p.mask_words, i1, s.ctx, s.len, g);
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int bit = 2 * qd + 8 * nt + e;
                    if (!((w0 >> bit) & 1)) sc[nt][e] = -INFINITY;
                    if (!((w1 >> bit) & 1)) sc[nt][2 + e] = -INFINITY;
                }
            // take non-finite values out of V (in place; the rows that see them get them at the end)
            bool odd = false;
            for (int c = lane; c < L::kTile / 16; c += 32) {
                uint32_t w[4];
                const uint32_t at = vt + 16 * c;
                lds_words(at, w);
                bool bad = false;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    uint32_t keep;
                    if constexpr (F8) {  // a code is non-finite when its f16 value is
                        const uint32_t lo = finite_halves(fp8x2_f16x2<FMT>(w[x]), true);
                        const uint32_t hi = finite_halves(fp8x2_f16x2<FMT>(w[x] >> 16), true);
                        keep = __byte_perm(lo, hi, 0x6420);
                    } else {
                        keep = finite_halves(w[x], false);
                    }
                    bad |= keep != 0xFFFFFFFFu;
                    w[x] &= keep;
                }
                if (bad)
                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                                 : "memory");
                odd |= bad;
            }
            if (odd) odd_v = 1;
            __syncwarp();
        }

        float mx0 = fmaxf(fmaxf(sc[0][0], sc[0][1]), fmaxf(sc[1][0], sc[1][1]));
        float mx1 = fmaxf(fmaxf(sc[0][2], sc[0][3]), fmaxf(sc[1][2], sc[1][3]));
        mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 1));
        mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 2));
        mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 1));
        mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 2));
        const float mc0 = fmaxf(m0, mx0), mc1 = fmaxf(m1, mx1);
        const bool need = ((mc0 - m0) * s0 > p.rescale_thr) || (GN == 16 && (mc1 - m1) * s1 > p.rescale_thr);
        if (__any_sync(0xffffffffu, need)) {
            const float a0 = m0 == -INFINITY ? 0.0f : ex2_mufu((m0 - mc0) * s0);
            const float a1 = m1 == -INFINITY ? 0.0f : ex2_mufu((m1 - mc1) * s1);
            l0 *= a0, l1 *= a1;
            m0 = mc0, m1 = mc1;
            const int src = qd * 8;  // lane of row 2 qd; O^T columns are rows 2 qd, 2 qd + 1 (+ 8)
#pragma unroll
            for (int nh = 0; nh < NH; ++nh) {
                const float c0 = __shfl_sync(0xffffffffu, nh ? a1 : a0, src);
                const float c1 = __shfl_sync(0xffffffffu, nh ? a1 : a0, src + 4);
#pragma unroll
                for (int mt = 0; mt < D / 16; ++mt) {
                    oacc[nh][mt][0] *= c0;
                    oacc[nh][mt][1] *= c1;
                    oacc[nh][mt][2] *= c0;
                    oacc[nh][mt][3] *= c1;
                }
            }
        }
        const float n0 = m0 == -INFINITY ? 0.0f : -m0 * s0, n1 = m1 == -INFINITY ? 0.0f : -m1 * s1;
        float pr[2][4];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
            pr[nt][0] = ex2_mufu(fmaf(sc[nt][0], s0, n0));
            pr[nt][1] = ex2_mufu(fmaf(sc[nt][1], s0, n0));
            pr[nt][2] = ex2_mufu(fmaf(sc[nt][2], s1, n1));
            pr[nt][3] = ex2_mufu(fmaf(sc[nt][3], s1, n1));
        }
        l0 += (pr[0][0] + pr[0][1]) + (pr[1][0] + pr[1][1]);
        l1 += (pr[0][2] + pr[0][3]) + (pr[1][2] + pr[1][3]);
        // O^T += V^T P^T; P is rounded to the 16-bit type of the product (bf16, or f16 for 8-bit caches)
        uint32_t pb[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const float lo = pr[x & 1][2 * (x >> 1)], hi = pr[x & 1][2 * (x >> 1) + 1];
            pb[x] = F8 ? pack_half2(lo, hi) : pack_bf16x2(lo, hi);
        }
        if constexpr (F8) {
            // tokens 2 qd, 2 qd + 1, 2 qd + 8, 2 qd + 9; bytes [(D/8) g0, (D/8) g0 + D/8) of each
            uint32_t vw[4][D / 32];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int tok = 2 * qd + (t & 1) + 8 * (t >> 1);
                if constexpr (D == 128)
                    lds_words(vt + swz_chunk<L::kChunks>(tok, g0), vw[t]);
                else
                    lds_words(vt + swz_chunk<L::kChunks>(tok, g0 >> 1) + (g0 & 1) * 8, vw[t]);
            }
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt) {
                const uint32_t sel = (mt & 1) ? 0x7362u : 0x5140u;  // bytes 2 j and 2 j + 1 of both tokens
                const uint32_t lo = __byte_perm(vw[0][mt >> 1], vw[1][mt >> 1], sel);
                const uint32_t hi = __byte_perm(vw[2][mt >> 1], vw[3][mt >> 1], sel);
                const uint32_t a[4] = {fp8x2_f16x2<FMT>(lo), fp8x2_f16x2<FMT>(lo >> 16), fp8x2_f16x2<FMT>(hi),
                                       fp8x2_f16x2<FMT>(hi >> 16)};
                mma_f16(oacc[0][mt], a, pb[0], pb[1]);
                if (GN == 16) mma_f16(oacc[NH - 1][mt], a, pb[2], pb[3]);
            }
        } else {
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt) {
                uint32_t a[4];
                ldmatrix_x4_trans(vt + swz_chunk<L::kChunks>(lm_row, 2 * mt + lm_par), a[0], a[1], a[2], a[3]);
                mma_bf16_16816(oacc[0][mt], a, pb[0], pb[1]);
                if (GN == 16) mma_bf16_16816(oacc[NH - 1][mt], a, pb[2], pb[3]);
            }
        }
    }
    cp_async_wait<0>();

    // ---- merge the warps through shared memory: sm_o[warp][row][d], maxima, sums
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    __syncthreads();  // every warp is done with its ring
    float* sm_o = reinterpret_cast<float*>(smem);
    float* sm_m = sm_o + kWarps * GN * L::kRowO;
    float* sm_l = sm_m + kWarps * GN;
    if (qd == 0) {
        sm_m[warp * GN + g0] = F8 ? m0 * s0 : m0;  // (8-bit caches: as an exponent of two, the row's factor included)
        sm_l[warp * GN + g0] = l0;
        if (GN == 16) {
            sm_m[warp * GN + g0 + 8] = F8 ? m1 * s1 : m1;
            sm_l[warp * GN + g0 + 8] = l1;
        }
    }
#pragma unroll
    for (int nh = 0; nh < NH; ++nh)
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt) {
            // rows of O^T: d, in the permuted order of the 8-bit products
            const int d0 = F8 ? (D / 8) * g0 + 2 * mt : mt * 16 + g0, d1 = F8 ? d0 + 1 : d0 + 8;
            float* base = sm_o + (warp * GN + nh * 8 + 2 * qd) * L::kRowO;
            base[d0] = oacc[nh][mt][0];
            base[L::kRowO + d0] = oacc[nh][mt][1];
            base[d1] = oacc[nh][mt][2];
            base[L::kRowO + d1] = oacc[nh][mt][3];
        }
    __syncthreads();
    // four neighbouring elements per thread, so that the rows of a block take few rounds of latency
    constexpr int kPerRow = D / 4, kAtOnce = kWarps * 32 / kPerRow;
    const int d0 = threadIdx.x % kPerRow * 4;
#pragma unroll
    for (int k = 0; k < GN / kAtOnce; ++k) {
        const int r = k * kAtOnce + threadIdx.x / kPerRow;
        if (r >= R) break;
        float mm = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sm_m[w * GN + r]);
        float ll = 0.0f, acc[4] = {};
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            // a warp without a visible key has m = -inf and only zeros (or NaN, which has to stay)
            const float mw = sm_m[w * GN + r];
            const float f = mw == -INFINITY ? 1.0f : ex2_mufu(F8 ? mw - mm : (mw - mm) * p.scale_log2);
            ll += f * sm_l[w * GN + r];
            const float4 o = *reinterpret_cast<const float4*>(sm_o + (w * GN + r) * L::kRowO + d0);
            acc[0] += f * o.x, acc[1] += f * o.y, acc[2] += f * o.z, acc[3] += f * o.w;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = ll == 0.0f ? 0.0f : acc[e] / ll * p.v_descale;
        const float lse = ll == 0.0f ? -INFINITY : mm * (F8 ? 0.6931471805599453f : p.scale) + logf(ll);
        const long long orow = out_row(r);
        if (nsplit == 1) {
            *reinterpret_cast<uint2*>(p.o + orow * D + d0) = make_uint2(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]));
            if (d0 == 0) p.lse[orow] = lse;
        } else if (joins) {
            *reinterpret_cast<float4*>(part_o + r * D + d0) = make_float4(acc[0], acc[1], acc[2], acc[3]);
            if (d0 == 0) part_lse[r] = lse;
        } else {
            *reinterpret_cast<float4*>(p.ws_o + (orow * p.max_splits + split) * D + d0) = make_float4(acc[0], acc[1], acc[2], acc[3]);
            if (d0 == 0) p.ws_lse[orow * p.max_splits + split] = lse;
        }
    }
    if (odd_v) {  // (written before the barriers above; the same for the whole block)
        __syncthreads();
        for (int t = max(t_begin, s.ctx / kGroup * kGroup); t < t_end; t += 64)
            add_nonfinite<D, FMT>(p, b, kvh, r0, warp, kWarps, R, t, t_end, nsplit == 1 ? -1 : joins ? -2 : split, part_o, D);
    }
    if (joins) cluster_join<D, D>(part_o, part_lse, p.o, p.lse, out_first, r0, R, p.G, p.Hq, p.cluster, nsplit);
}

// ------------------------------------------------------------------------------ join of the splits
//
// One warp per output row. Launched as a programmatic dependent of the split kernel; rows of one split are already written.
template <int D>
__global__ void __launch_bounds__(128) tree_combine_kernel(const TreeParams p) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    TreeSeq s;
    const bool rows = tree_seq(p, blockIdx.y, s);
    const long long r = (long long)blockIdx.x * 4 + warp;
    grid_dependency_wait();
    if (!rows || r >= (long long)s.n * p.Hq) return;
    const int ns = cdiv(s.len, p.slots > 0 ? *p.ws_chunk : p.chunk);
    if (ns <= 1) return;
    const long long row = (long long)s.q0 * p.Hq + r;
    const float* wl = p.ws_lse + row * p.max_splits;
    const float* wo = p.ws_o + row * p.max_splits * D;
    join_row<D>(
        ns, [&](int i) { return wl[i]; }, [&](int i) { return wo + (long long)i * D; }, p.o + row * D, p.lse + row);
}

template <int D>
cudaError_t launch_join(const TreeParams& p, cudaStream_t stream) {
    const dim3 grid((unsigned)(((long long)p.max_q * p.Hq + 3) / 4), (unsigned)p.B);
    return launch_kernel(tree_combine_kernel<D>, grid, 128, 0, stream, {true}, p);
}

template <int D, int GN, int FMT, bool kCluster>
cudaError_t launch_small(TreeParams p, cudaStream_t stream) {
    constexpr int bytes = SmallLayout<D, GN, FMT>::kBytes;
    static std::atomic<bool> attr_set[kMaxAttrDevices];
    cudaError_t e = ensure_smem_attr(tree_small_kernel<D, GN, FMT, kCluster>, bytes, attr_set);
    if (e != cudaSuccess) return e;
    p.groups = (int)(((long long)p.max_q * p.G + 15) / 16);
    const dim3 grid = tree_grid(p);
    return launch_kernel(tree_small_kernel<D, GN, FMT, kCluster>, grid, kWarps * 32, bytes, stream, {false, p.cluster}, p);
}

template <int D, int FMT>
cudaError_t launch_rows(const TreeParams& p, cudaStream_t stream) {
    if ((long long)p.max_q * p.G <= 8)
        return p.cluster > 0 ? launch_small<D, 8, FMT, true>(p, stream) : launch_small<D, 8, FMT, false>(p, stream);
    return p.cluster > 0 ? launch_small<D, 16, FMT, true>(p, stream) : launch_small<D, 16, FMT, false>(p, stream);
}

template <int D>
cudaError_t launch_fmt(const TreeParams& p, int fmt, cudaStream_t stream) {
    return fmt == ATTN_FP8_E4M3   ? launch_rows<D, ATTN_FP8_E4M3>(p, stream)
           : fmt == ATTN_FP8_E5M2 ? launch_rows<D, ATTN_FP8_E5M2>(p, stream)
                                  : launch_rows<D, ATTN_KV_BF16>(p, stream);
}

}  // namespace

void tree_plan(TreeParams& p, int d, bool f8, int num_splits) {
    const int B = p.B, Hkv = p.Hkv, rows = p.max_q * p.G, num_sms = p.num_sms;
    const long long lmax = (long long)p.max_pages * p.page_size;
    const bool tiles = tree_takes_tiles(rows, d, f8, p.page_size, B, Hkv, lmax, num_sms);
    p.tiles = tiles;
    const long long groups = (long long)B * Hkv * (tiles ? (rows + 127) / 128 : (rows + 15) / 16);
    const long long slots = (long long)num_sms * (tiles ? kTreeTileBlocks : tree_small_blocks(d, f8, rows));
    const bool fit = num_splits == 0 && groups <= slots && B <= kTreeFitSeqs;
    long long c;
    if (fit) {
        // Fewer (sequence, kv head, row group) groups than blocks that fit at once: the blocks choose by the
        // lengths (tree_fit), as long as the table's capacity leaves anything to choose. The workspace is for
        // sequences that fill an eighth of it.
        c = (lmax * groups + 8 * slots - 1) / (8 * slots);
        if (c < 128) c = 128;
    } else if (num_splits > 0) {
        c = (lmax + num_splits - 1) / num_splits;
    } else if (tiles) {
        // Blocks of 128 rows, two per SM. With fewer (sequence, kv head, row tile) groups than SMs: as many
        // splits as fit at once, at least four of 1024 tokens or more, which balance sequences of different
        // lengths. With enough groups for two blocks per SM: none, because the partial results of 128 rows cost
        // as much traffic as 130 cached tokens of one head and the join is a second launch; the longest
        // sequences start first. In between, a cap of 8192 tokens. Measured, splits -> us: 64 sequences of
        // U[1K, 32K], 16 drafted tokens x 4 query heads x 8 kv heads (512 groups), bf16 1: 633, 2: 650, 4: 644,
        // 8: 668, e4m3 1: 433, 2: 459, 4: 486; 100 of U[100, 4000], 8 drafted tokens x 4 query heads (100
        // groups), bf16 1: 48, 2: 38, 4: 29, 8: 35.
        long long splits = 1, most = 65536;
        if (groups < num_sms) {
            const long long balance = lmax / 1024 < 4 ? lmax / 1024 : 4;
            splits = 2LL * num_sms / groups;
            if (splits < balance) splits = balance;
        }
        if (groups < 2LL * num_sms) most = 8192;
        c = (lmax + splits - 1) / splits;
        if (c < 128) c = 128;
        if (c > most) c = most;
    } else {
        // Blocks of 16 rows, three to five per SM. Many tokens: about 6 items per SM, assuming half-full page
        // tables; fewer: two items per SM, up to 2048 tokens each. Measured, bf16 / e4m3, splits -> us: 64
        // sequences of U[1K, 32K], 4 drafted tokens x 4 query heads x 8 kv heads 2: 624 / 363, 4: 613 / 372,
        // 8: 628 / 372, 16: 655 / 407 (one token each 2: 611 / 345, 4: 601 / 348, 8: 604 / 340); 100 of
        // U[100, 4000], 2 drafted tokens x 4 query heads 1: 49 / 44, 2: 33 / 31, 4: 23 / 23, 8: 27 / 20,
        // 16: 32 / 25.
        const long long tokens = (long long)B * Hkv * lmax;
        c = (tokens + 4LL * num_sms - 1) / (4LL * num_sms) * 2;  // two items per SM
        if (c > 2048) c = 2048;
        const long long many = (tokens / 2 + 6LL * num_sms - 1) / (6LL * num_sms);
        if (c < many) c = many;
        if (c < 128) c = 128;
        if (c > 16384) c = 16384;
    }
    c = (c + 63) / 64 * 64;
    const long long whole = (lmax + 63) / 64 * 64;
    if (c > whole) c = whole;
    if (c < 64) c = 64;
    p.chunk = (int)c;
    p.max_splits = (int)((lmax + c - 1) / c);
    const bool at_once = groups * p.max_splits <= slots;
    p.slots = fit && !at_once ? (int)slots : 0;
    p.cluster = p.max_splits > 1 && p.max_splits <= kTreeCluster && at_once ? p.max_splits : 0;
}

cudaError_t launch_attn_tree(const TreeParams& p_in, const TreeTmaps& tm, int d, int kv_format, cudaStream_t stream) {
    TreeParams p = p_in;
    // tok / page_size for tok < 2^31: multiplier ceil(2^(31+k) / page_size), k = ceil(log2 page_size)
    p.ps_magic = 0;
    p.ps_shift = 0;
    if (p.page_size > 1) {
        int k = 0;
        while ((1LL << k) < p.page_size) ++k;
        p.ps_magic = (unsigned)(((1ULL << (31 + k)) + (unsigned long long)p.page_size - 1) / (unsigned long long)p.page_size);
        p.ps_shift = k - 1;
    }
    cudaError_t e;
    if (p.tiles)
        e = launch_tree_tiles(p, tm, d, kv_format, stream);
    else
        e = d == 128 ? launch_fmt<128>(p, kv_format, stream) : launch_fmt<64>(p, kv_format, stream);
    if (e == cudaSuccess && p.max_splits > 1 && p.cluster == 0) e = d == 128 ? launch_join<128>(p, stream) : launch_join<64>(p, stream);
    return e;
}

}  // namespace attn
