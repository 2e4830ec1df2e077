// Helpers of the row-wise operators (rotary positions, paged cache writes and reads): the angle of
// a position, which columns one work item holds, element packing, and the place of a packed row.
#pragma once

#include "kernels.cuh"
#include "ptx.cuh"

#include <cuda_bf16.h>
#include <stdint.h>

namespace attn {

// Rotary part of a head: columns [begin, begin + rot) of d, pairs (i, i + rot / 2), or with
// interleaved != 0 (2 i, 2 i + 1).
struct RopeCols {
    int d, begin, rot, interleaved;
};

// Work item j of a head (j < d / (2 V)) holds the 2 V columns [a, a + V) and [b, b + V): first the rotated
// ones (then true is returned), a in the lower and b in the upper half of the rotated part, then in the
// same way those that pass through, so that neighbouring items are neighbours in memory. (Single
// interleaved pairs, V = 1, are columns 2 j and 2 j + 1.) V > 1 needs begin and rot to be multiples of 2 V.
template <int V>
__device__ __forceinline__ bool item_cols(const RopeCols& c, int j, int& a, int& b) {
    const int x = V * j, turned = c.rot / 2;
    if (x < turned) {
        a = c.begin + (V == 1 && c.interleaved ? 2 * j : x);
        b = a + (V == 1 && c.interleaved ? 1 : turned);
        return true;
    }
    a = x - turned;
    b = a + (c.d - c.rot) / 2;
    if (a >= c.begin) a += c.rot;
    if (b >= c.begin) b += c.rot;
    return false;
}

// N neighbouring cosines or sines by loads as wide as they allow (aligned to min(16, 4 N) bytes).
template <int N>
__device__ __forceinline__ void load_angles(const float* p, float (&x)[N]) {
    if constexpr (N >= 4) {
#pragma unroll
        for (int e = 0; e < N; e += 4) {
            const float4 w = *reinterpret_cast<const float4*>(p + e);
            x[e] = w.x, x[e + 1] = w.y, x[e + 2] = w.z, x[e + 3] = w.w;
        }
    } else if constexpr (N == 2) {
        const float2 w = *reinterpret_cast<const float2*>(p);
        x[0] = w.x, x[1] = w.y;
    } else {
        x[0] = *p;
    }
}

// Rotate the pairs of item j; cs and sn: cosines and sines of the token, one per pair.
template <int V>
__device__ __forceinline__ void rotate_item(float (&xa)[V], float (&xb)[V], const RopeCols& cols, int j, const float* cs,
                                            const float* sn) {
    if (V == 1 || !cols.interleaved) {
        float c[V], s[V];
        load_angles<V>(cs + V * j, c);
        load_angles<V>(sn + V * j, s);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float u = xa[e], w = xb[e];
            xa[e] = u * c[e] - w * s[e];
            xb[e] = u * s[e] + w * c[e];
        }
    } else if constexpr (V > 1) {  // pairs of adjacent columns: V / 2 in each part
        const int first = V / 2 * j, second = first + cols.rot / 4;
        auto turn = [&](float(&x)[V], int at) {
            float c[V / 2], s[V / 2];
            load_angles<V / 2>(cs + at, c);
            load_angles<V / 2>(sn + at, s);
#pragma unroll
            for (int e = 0; e < V / 2; ++e) {
                const float u = x[2 * e], w = x[2 * e + 1];
                x[2 * e] = u * c[e] - w * s[e];
                x[2 * e + 1] = u * s[e] + w * c[e];
            }
        };
        turn(xa, first);
        turn(xb, second);
    }
}

// A frequency as a 64-bit fraction of a turn per position. The product with an integer position is
// exact modulo one turn in wrapping 64-bit arithmetic, so far positions lose nothing beyond the error of
// the fraction, which is under 2^-63 of a turn for f < 1 (1.5e-9 rad at position 2^31). All in integers: the
// mantissa times 1 / (2 pi) * 2^66, shifted by the exponent; 64-bit floating-point arithmetic is slow on this
// GPU (two results a clock and SM).
__device__ __forceinline__ unsigned long long turn_fraction(double f) {
    const unsigned long long bits = (unsigned long long)__double_as_longlong(f), inv_2pi = 0xA2F9836E4E44152Aull;
    const int exponent = (int)(bits >> 52) & 2047;
    if (exponent == 0) return 0;  // 0, or too small for a bit
    const unsigned long long mantissa = (bits & ((1ull << 52) - 1)) | 1ull << 52;  // f = mantissa * 2^(exponent - 1075)
    const unsigned long long hi = __umul64hi(mantissa, inv_2pi), lo = mantissa * inv_2pi;
    const int shift = 1077 - exponent;  // bits of the product below 2^-64 of a turn
    unsigned long long turns;
    if (shift >= 64)
        turns = shift < 128 ? hi >> (shift - 64) : 0;
    else if (shift > 0)
        turns = hi << (64 - shift) | lo >> shift;
    else
        turns = shift > -64 ? lo << -shift : 0;
    return f < 0 ? 0 - turns : turns;
}

// The quarter turn nearest to the angle is split off in integers too; the rest, at most an eighth of a turn, is
// rounded to fp32, and what that leaves out is added as a rotation by that small angle. So the cosine and sine are
// off by little more than those of sincospif.
__device__ __forceinline__ void position_angle(unsigned long long frac, int pos, float& c, float& s) {
    const unsigned long long phase = frac * (unsigned long long)(long long)pos;  // turns * 2^64
    const unsigned quarter = (unsigned)((phase + (1ull << 61)) >> 62);
    const long long rest = (long long)(phase - ((unsigned long long)quarter << 62));  // [-2^61, 2^61)
    const int top = (int)(rest >> 30);  // 2^-33 half turns, [-2^31, 2^31)
    const float hi = (float)top;
    const float lo = (float)(top - (int)hi) + (float)((int)rest & 0x3FFFFFFF) * 0x1p-30f;
    float c0, s0;
    sincospif(hi * 0x1p-33f, &s0, &c0);
    const float d = lo * 3.657295198e-10f, sx = s0;  // radians: pi * 2^-33
    s0 = fmaf(d, c0, s0);
    c0 = fmaf(-d, sx, c0);
    const float u = quarter & 1 ? -s0 : c0, w = quarter & 1 ? c0 : s0;   // one quarter turn further
    c = quarter & 2 ? -u : u;
    s = quarter & 2 ? -w : w;
}

// cos and sin (times the amplitude) of tokens [0, tokens) of a block into cs[token][rot / 2] and
// sn[token][rot / 2]. Every thread of the block calls it.
__device__ __forceinline__ void block_angles(const double* inv_freq, const int* positions, int tokens, int half,
                                             float amplitude, bool transpose, float* cs, float* sn) {
    const int nt = blockDim.x, groups = max(1, nt / half);
    const int first = threadIdx.x % half, grp = threadIdx.x / half;
    if (grp >= groups) return;
    for (int i = groups > 1 ? first : (int)threadIdx.x; i < half; i += groups > 1 ? half : nt) {
        const double f = inv_freq[i];
        const unsigned long long frac = turn_fraction(f);
        const float amp = isfinite(f) ? amplitude : __int_as_float(0x7fffffff);  // no angle: NaN
        for (int t = groups > 1 ? grp : 0; t < tokens; t += groups) {
            float c, s;
            position_angle(frac, positions[t], c, s);
            cs[t * half + i] = c * amp;
            sn[t * half + i] = (transpose ? -s : s) * amp;
        }
    }
}

// ---- V consecutive elements of a row: as loaded (16 bytes at once when V > 1), and as floats

template <typename E, int V>
struct RawOf {
    static_assert(V * sizeof(E) == 16, "16 bytes");
    typedef uint4 type;
};
template <typename E>
struct RawOf<E, 1> {
    typedef E type;
};

template <typename E, int V>
__device__ __forceinline__ typename RawOf<E, V>::type load_raw(const E* p) {
    return *reinterpret_cast<const typename RawOf<E, V>::type*>(p);
}

template <typename E, int V>
__device__ __forceinline__ void unpack(const typename RawOf<E, V>::type& w, float (&x)[V]) {
    if constexpr (V == 8) {
        const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(r[i] << 16);
            x[2 * i + 1] = __uint_as_float(r[i] & 0xFFFF0000u);
        }
    } else if constexpr (V == 4) {
        x[0] = __uint_as_float(w.x), x[1] = __uint_as_float(w.y), x[2] = __uint_as_float(w.z), x[3] = __uint_as_float(w.w);
    } else {
        x[0] = (float)w;
    }
}

template <int V>
__device__ __forceinline__ void store_row(__nv_bfloat16* p, const float (&x)[V]) {
    if constexpr (V == 8)
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    else
        *p = __float2bfloat16_rn(x[0]);
}

template <int V>
__device__ __forceinline__ void store_row(float* p, const float (&x)[V]) {
    if constexpr (V == 4)
        *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    else
        *p = x[0];
}

// ---- how the threads of a block share the items of its tokens
//
// A token has `pairs` = heads * items per head (head, item) pairs. `width` threads take one pair each (in
// turns, when there are more pairs) and keep it over all tokens of the block, so that heads, columns and
// angles are worked out once; blockDim / width groups of threads take the tokens in turn.
struct RowShare {
    int width, threads;  // threads per token, threads of the block
    int tokens;          // tokens per block
};

// Tokens per block: `most`, fewer where that fills whole waves of `slots` blocks, since a last wave of few blocks
// costs as much as a full one.
inline int whole_waves(int T, long long most, long long slots) {
    if (most < 1) most = 1;
    const long long waves = (T + slots * most - 1) / (slots * most);
    return (int)((T + slots * waves - 1) / (slots * waves));
}

// Tokens for `items` items per thread, `most` at most; `resident` threads fit on an SM.
inline RowShare share_rows(int T, int pairs, int items, int most, int resident, int num_sms) {
    RowShare s;
    const int turns = (pairs + 511) / 512;
    s.width = (pairs + turns - 1) / turns;
    const int groups = s.width >= 256 ? 1 : 256 / s.width;
    s.threads = (s.width * groups + 31) / 32 * 32;
    long long n = ((long long)items * groups + turns - 1) / turns;
    if (n > most) n = most;
    s.tokens = whole_waves(T, n, (long long)num_sms * (resident / s.threads));
    return s;
}

// ---- packed rows of a paged cache

// Sequence of packed row t: the number of sequences that end at or before it. A warp probes 32
// offsets at a time, so 1024 sequences take two rounds of loads. The whole warp calls it.
__device__ __forceinline__ int warp_find_seq(const int* cu, int B, int t) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = B;  // the answer lies in [lo, hi]
    while (lo < hi) {
        const int step = (hi - lo + 31) / 32;
        const long long at = (long long)lo + (long long)(lane + 1) * step - 1;
        const bool before = at < hi && __ldg(cu + at + 1) <= t;
        const int cnt = __popc(__ballot_sync(0xffffffffu, before));
        const long long next = (long long)lo + (long long)cnt * step;
        const long long end = next + step - 1;
        lo = (int)(next < hi ? next : hi);
        hi = (int)(end < hi ? end : hi);
    }
    return lo;
}

// Shared by the cache writes and reads: row t of T belongs to sequence b and is its i-th of n
// rows; it stands for cached token seqlens[b] - n + i.
struct PagedRows {
    const int* page_table;  // [B, max_pages]
    const int* seqlens;     // [B], the n rows included
    const int* cu_seqlens;  // [B + 1] or nullptr: T / B rows each
    int B, T, max_pages, page_size, num_pages;
    int* status;
};

constexpr long long kRowNone = -1;  // no sequence holds the row: it is left as it is
constexpr long long kRowBad = -2;   // a length or page out of range (recorded)

// Cache row of packed row t, or kRowNone / kRowBad. The whole warp calls it.
__device__ __forceinline__ long long paged_row(const PagedRows& p, int t) {
    int b, i, n;
    if (p.cu_seqlens) {
        b = warp_find_seq(p.cu_seqlens, p.B, t);
        if (b >= p.B) return kRowNone;
        const long long c0 = __ldg(p.cu_seqlens + b), c1 = __ldg(p.cu_seqlens + b + 1);
        if (b == 0 && t < c0) return kRowNone;  // rows before the first sequence
        if (t < c0 || t >= c1 || c0 < 0 || c1 > p.T) {  // offsets that decrease or pass the rows
            if ((threadIdx.x & 31) == 0) atomicCAS(p.status, 0, kDevBadIndex);
            return kRowNone;
        }
        i = (int)(t - c0);
        n = (int)(c1 - c0);
    } else {
        n = p.T / p.B;
        b = t / n;
        i = t - b * n;
    }
    const long long len = __ldg(p.seqlens + b);
    const long long at = len - n + i;
    int page = -1;
    if (len >= n && len <= (long long)p.max_pages * p.page_size)
        page = __ldg(p.page_table + (long long)b * p.max_pages + at / p.page_size);
    if (page < 0 || page >= p.num_pages) {
        if ((threadIdx.x & 31) == 0) atomicCAS(p.status, 0, kDevBadIndex);
        return kRowBad;
    }
    return (long long)page * p.page_size + at % p.page_size;
}

}  // namespace attn
