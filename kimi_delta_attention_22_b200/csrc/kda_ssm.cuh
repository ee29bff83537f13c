// kda_ssm.cuh -- device pieces that the selective scan's forward, step and gradient share.
#pragma once

#include "kda_block.cuh"

namespace kda {
namespace ssm {

// softplus(v) = max(v, 0) + log(1 + e), e = e^-|v| <= 1.  With s = e / (2 + e) <= 1/3,
// log(1 + e) = 2 atanh(s) = 2 s (1 + s^2/3 + s^4/5 + ..): the series ends at s^14/15, whose
// remainder is below 2e-9 of the sum, so the value keeps its relative accuracy where e is
// tiny (step sizes of 1e-3 and less), which a logarithm of 1 + e does not.
__device__ __forceinline__ F2 softplus2(F2 v) {
    const F2 e = ex2(mul2(F2{fabsf(v.x), fabsf(v.y)}, both(-kLog2e)));
    const F2 s = mul2(e, rcp(add2(e, both(2.0f)))), q = mul2(s, s);
    F2 p = both(1.0f / 15.0f);
    p = fma2(p, q, both(1.0f / 13.0f));
    p = fma2(p, q, both(1.0f / 11.0f));
    p = fma2(p, q, both(1.0f / 9.0f));
    p = fma2(p, q, both(1.0f / 7.0f));
    p = fma2(p, q, both(1.0f / 5.0f));
    p = fma2(p, q, both(1.0f / 3.0f));
    p = fma2(p, q, both(1.0f));
    return fma2(add2(s, s), p, F2{fmaxf(v.x, 0.0f), fmaxf(v.y, 0.0f)});   // a NaN stays one through e
}
__device__ __forceinline__ float softplus(float v) { return softplus2(F2{v, v}).x; }

// Where row `row` of channel c lies in a tile array [channel][row]: groups of four rows stay
// together (one 16-byte access) and are permuted by the channel, so that neither the staging
// threads (the same channel of eight vectors, four rows) nor the scanning ones (eight
// neighbouring channels, the same rows) meet in a bank.
template <int TT>
__device__ __forceinline__ int cell(int c, int row) {
    return c * TT + ((((row >> 2) ^ (c >> 3) ^ c) & (TT / 4 - 1)) << 2 | (row & 3));
}

// A pair of B or C in shared memory (as stored, two bf16 or two fp32).
__device__ __forceinline__ F2 lds_pair(const float* p) {
    const float2 v = *reinterpret_cast<const float2*>(p);
    return F2{v.x, v.y};
}
__device__ __forceinline__ F2 lds_pair(const __nv_bfloat16* p) {
    const uint32_t v = *reinterpret_cast<const uint32_t*>(p);
    return F2{__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u)};
}

// Four states of B and of C as they lie in shared memory, side by side: [row][lane][B, C][4].
template <typename T, bool BOTH>
struct Quads {
    uint32_t w[(BOTH ? 2 : 1) * sizeof(T)];
    __device__ __forceinline__ void load(const T* p) {
        constexpr int n = (BOTH ? 2 : 1) * (int)sizeof(T);   // words
        if constexpr (n == 2) {
            const uint2 v = *reinterpret_cast<const uint2*>(p);
            w[0] = v.x; w[1] = v.y;
        } else {
#pragma unroll
            for (int k = 0; k < n; k += 4) {
                const uint4 v = reinterpret_cast<const uint4*>(p)[k / 4];
                w[k] = v.x; w[k + 1] = v.y; w[k + 2] = v.z; w[k + 3] = v.w;
            }
        }
    }
    __device__ __forceinline__ F2 get(int which, int m) const {   // pair m of B (0) or C (1)
        if constexpr (sizeof(T) == 2) {
            const uint32_t v = w[which * 2 + m];
            return F2{__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u)};
        } else {
            return F2{__uint_as_float(w[which * 4 + 2 * m]), __uint_as_float(w[which * 4 + 2 * m + 1])};
        }
    }
};

// 8 consecutive channels of one row (those below `n`), as raw words.
template <typename T, bool ALIGNED>
__device__ __forceinline__ Pack<T, 8> load8(const T* p, int n) {
    Pack<T, 8> r = zero_pack<T, 8>();
    if constexpr (ALIGNED) {
        if (n > 0) {
            if constexpr (sizeof(T) == 2) {
                r = load_pack<8>(p);
            } else {
                const Pack<T, 4> a = load_pack<4>(p), b = load_pack<4>(p + 4);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    r.w[i] = a.w[i];
                    r.w[4 + i] = b.w[i];
                }
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) {
                const uint32_t w = load_pack<1>(p + i).w[0];
                if constexpr (sizeof(T) == 2) r.w[i / 2] |= w << (16 * (i & 1));
                else r.w[i] = w;
            }
    }
    return r;
}
template <typename T, bool ALIGNED>
__device__ __forceinline__ void store8(T* p, const float* f, int n) {
    if constexpr (ALIGNED) {
        if (n > 0) {
            if constexpr (sizeof(T) == 2) {
                store_f32<T, 8>(p, f);
            } else {
                store_f32<T, 4>(p, f);
                store_f32<T, 4>(p + 4, f + 4);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) store_f32<T, 1>(p + i, f + i);
    }
}

// Where a CTA's channels lie: CH consecutive channels of one group.
struct ChannelBlock {
    int d0, n, g;   // first channel, channels (<= CH), group
};
template <int CH>
__device__ __forceinline__ ChannelBlock channel_block(int blk, int D, int G) {
    const int dg = D / G, per = (dg + CH - 1) / CH;
    ChannelBlock c;
    c.g = blk / per;
    const int off = (blk - c.g * per) * CH;
    c.d0 = c.g * dg + off;
    c.n = dg - off < CH ? dg - off : CH;
    return c;
}
inline long long channel_blocks(int D, int G, int CH) { return (long long)G * ((D / G + CH - 1) / CH); }

// The sums over a channel's S lanes (lane s of them) of four rows' values, written to
// to[0..3]: lanes swap the halves that they do not keep, so that after two exchanges lane
// s & 3 holds its row, and the remaining lanes are added in full.
template <int S>
__device__ __forceinline__ void lane_sum4(float y0, float y1, float y2, float y3, int s, float* to) {
    if constexpr (S >= 2) {   // lanes with bit 0 keep rows 1 and 3
        const bool up = s & 1;
        const float k0 = up ? y1 : y0, k1 = up ? y3 : y2;
        y0 = k0 + __shfl_xor_sync(0xffffffffu, up ? y0 : y1, 1);
        y1 = k1 + __shfl_xor_sync(0xffffffffu, up ? y2 : y3, 1);
    }
    if constexpr (S >= 4) {   // lanes with bit 1 keep rows 2 and 3
        const bool up = s & 2;
        const float k0 = up ? y1 : y0;
        y0 = k0 + __shfl_xor_sync(0xffffffffu, up ? y0 : y1, 2);
    }
#pragma unroll
    for (int m = 4; m < S; m <<= 1) y0 += __shfl_xor_sync(0xffffffffu, y0, m);
    if constexpr (S == 1) {
        *reinterpret_cast<float4*>(to) = make_float4(y0, y1, y2, y3);
    } else if constexpr (S == 2) {
        to[s] = y0;
        to[2 + s] = y1;
    } else {
        if (s < 4) to[s] = y0;
    }
}

// Rows of the segments that the long axis is cut into (a multiple of the tile's rows), and
// how many; `whole`: one segment is exactly one sequence of a dense batch (or all rows), so
// that no segment starts inside a sequence.
struct Segments {
    long long len, count;
    bool whole;
};

// Whether segment [t0, t1) holds the first row of a sequence: its outgoing state then does
// not depend on its incoming one.  Rows in no sequence count as such.
__device__ __forceinline__ bool starts_inside(const SsmArgs& a, long long t0, long long t1) {
    const SeqRange r = find_seq(a.cu, a.num_seqs, a.M, a.T, t1 - 1);
    return !r.ok || r.b >= t0;
}

}  // namespace ssm
}  // namespace kda
