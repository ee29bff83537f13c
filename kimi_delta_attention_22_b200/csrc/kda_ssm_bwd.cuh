// kda_ssm_bwd.cuh -- gradients of the selective state space scan.
//
// With dy = d_out silu(z) and, from the last row of a sequence back,
//     dh[n]  <- dh[n] + C[n] dy                       (dh starts from d_hT)
//     dC[n]  = sum_d dy h[n],    dB[n] = sum_d dh[n] dt x
//     p      = sum_n dh[n] B[n]
//     w[n]   = dh[n] a[n],  q[n] = w[n] h_prev[n]     (a = e^{dt A})
//     dA[n]  = sum_rows q[n] dt
//     ddt    = sum_n q[n] A[n] + p x,   dx = p dt + Dskip dy
//     dh[n]  <- w[n]                                  (dh0 in front of the first row)
//
// The rows are cut into segments, aligned to the row index.
//   1. summary: every segment alone, scanned once from zero, gives its last state, the
//      gradient that its rows send to the state in front of it (sum_t (prod a) C dy, the
//      running product taken along, so no second exponential), the sum of dt, and both
//      states and sums in front of every 4 rows (checkpoints).
//   2. join: along the segments, forward for the incoming states, backward for the
//      incoming state gradients (the decay over a segment is e^{A sum dt}).
//   3. gradients, all segments in parallel, each from its last 4 rows back: the checkpoint
//      plus the decayed incoming state, then the 4 rows' states and decays into registers,
//      then the 4 rows in reverse.
//   4. sums: of dB and dC over the channel blocks, of dA, dDskip and the bias over segments.
// Two sets of exponentials (and one in 4 rows for the checkpoints) and about 18 fp32
// operations per row, channel and state.  4 x 2048 rows, 2048 channels, 16 states, bf16: 583 us
// (summary 165, join 12, gradients 397, sums 26).  No single pipe bounds it: the gradients kernel
// issues in 54 % of its slots (12 warps per SM, which its 168 registers leave), shared memory is
// half busy, the exponentials take 28 %; the bytes (238 MB) would take 36 us.
//
// Lanes: S lanes of a channel pair, four states each (as two register pairs for the packed
// fp32 instructions); a thread takes two channels, so that B and C are read from shared
// memory once for both and dB, dC are added over both before any exchange.  A CTA of 128
// threads holds 256 / S channels.  Sums over lanes are taken by halving exchanges: a lane
// keeps one half of its values and sends the other.  Where the halves are register pairs or
// channels, lanes on the upper side hold them in swapped order, so that every lane keeps the
// same registers and nothing is selected.
#pragma once

#include <type_traits>

#include "kda_ssm.cuh"

namespace kda {
namespace ssm {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kSub = 4;        // rows between checkpoints

template <int S>
constexpr int channels() { return 2 * kThreads / S; }
template <int S>
constexpr int tile_rows() { return S >= 4 ? 32 : 8 * S; }

// First / last rows of sequences and rows of any sequence, one bit per row of the tile.
struct Events {
    uint32_t first, last, in;
};
__device__ __forceinline__ Events find_events(const SsmArgs& a, long long t0, int rows) {   // whole warps
    Events e;
    const SeqRange r = find_seq(a.cu, a.num_seqs, a.M, a.T, t0 < a.M ? t0 : a.M - 1);
    if (r.ok && t0 >= r.b && t0 + rows <= r.e) {   // the tile inside a sequence, the common case
        e.in = rows == 32 ? 0xffffffffu : (1u << rows) - 1;
        e.first = t0 == r.b ? 1u : 0u;
        e.last = t0 + rows == r.e ? 1u << (rows - 1) : 0u;
        return e;
    }
    const int i = threadIdx.x & 31;
    SeqRange m{0, 0, 0, false};
    if (i < rows && t0 + i < a.M) m = find_seq(a.cu, a.num_seqs, a.M, a.T, t0 + i);
    e.first = __ballot_sync(0xffffffffu, m.ok && m.b == t0 + i);
    e.last = __ballot_sync(0xffffffffu, m.ok && m.e == t0 + i + 1);
    e.in = __ballot_sync(0xffffffffu, m.ok);
    return e;
}

__device__ __forceinline__ F2 shfl2(F2 v, int m) {
    return F2{__shfl_xor_sync(0xffffffffu, v.x, m), __shfl_xor_sync(0xffffffffu, v.y, m)};
}

__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool on) {   // zeros unless `on`
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
                 "r"(on ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_async8(float* dst, const float* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(float* dst, const float* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// One tile of the inputs as loaded: a thread's slots of one row and eight channels each, in
// shared memory that only this thread touches, so that the copies run while the tile before is
// worked on and need no barrier; and its share of B and C in registers.
template <typename T, int S, bool ALIGNED>
struct Raw {
    static constexpr int CH = channels<S>(), TT = tile_rows<S>(), NP = 4 * S;
    static constexpr int VPR = CH / 8, NSLOT = (TT * VPR + kThreads - 1) / kThreads;
    static constexpr int W = sizeof(T) / 2;             // 16-byte words of eight channels
    static constexpr int kBytes = 4 * NSLOT * W * 16 * kThreads;
    static constexpr int BPT = TT * NP / kThreads > 0 ? TT * NP / kThreads : 1;
    static constexpr bool kAhead = BPT <= 8;
    uint4* at;
    T nB[kAhead ? BPT : 1], nC[kAhead ? BPT : 1];
    __device__ __forceinline__ explicit Raw(void* mem) : at(static_cast<uint4*>(mem) + threadIdx.x) {}

    __device__ __forceinline__ void load1(int which, int it, const T* p, int n) {
        uint4* to = at + (which * NSLOT + it) * W * kThreads;
        if constexpr (ALIGNED) {
#pragma unroll
            for (int w = 0; w < W; ++w) cp_async16(to + w * kThreads, n > 0 ? p + w * (16 / sizeof(T)) : p, n > 0);
        } else {
            const Pack<T, 8> v = load8<T, false>(p, n);
#pragma unroll
            for (int w = 0; w < W; ++w) to[w * kThreads] = make_uint4(v.w[4 * w], v.w[4 * w + 1], v.w[4 * w + 2], v.w[4 * w + 3]);
        }
    }
    __device__ __forceinline__ Pack<T, 8> get(int which, int it) const {
        Pack<T, 8> v;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const uint4 u = at[((which * NSLOT + it) * W + w) * kThreads];
            v.w[4 * w] = u.x; v.w[4 * w + 1] = u.y; v.w[4 * w + 2] = u.z; v.w[4 * w + 3] = u.w;
        }
        return v;
    }
    __device__ __forceinline__ void read(int which, int it, float* f) const { unpack<T, 8>(get(which, it), f); }
    __device__ __forceinline__ T bc(const T* p, long long stride, const SsmArgs& a, long long t0, uint32_t in, int e) const {
        const int k = e * kThreads + threadIdx.x, row = k / NP, n = k % NP;
        return row < TT && n < a.N && (in >> (row & 31) & 1) ? p[(t0 + row) * stride + n] : from_f32<T>(0.f);
    }
    __device__ __forceinline__ void load(const SsmArgs& a, const ChannelBlock& cb, long long t0, uint32_t in) {
#pragma unroll
        for (int it = 0; it < NSLOT; ++it) {
            const int slot = it * kThreads + threadIdx.x, row = slot / VPR, c0 = (slot % VPR) * 8;
            const int n = row < TT && (in >> (row & 31) & 1) ? cb.n - c0 : 0;
            // rows and channels that are not read: any address inside the tensors
            const long long t = n > 0 ? t0 + row : t0;
            const int d = n > 0 ? cb.d0 + c0 : cb.d0;
            load1(0, it, static_cast<const T*>(a.x) + t * a.xs + d, n);
            load1(1, it, static_cast<const T*>(a.delta) + t * a.ds + d, n);
            load1(2, it, static_cast<const T*>(a.d_out) + t * a.D + d, n);
            if (a.z != nullptr) load1(3, it, static_cast<const T*>(a.z) + t * a.zs + d, n);
        }
        if constexpr (kAhead) {
            const T* Bp = static_cast<const T*>(a.Bm) + (long long)cb.g * a.N;
            const T* Cp = static_cast<const T*>(a.Cm) + (long long)cb.g * a.N;
#pragma unroll
            for (int e = 0; e < BPT; ++e) {
                nB[e] = bc(Bp, a.bs, a, t0, in, e);
                nC[e] = bc(Cp, a.cs, a, t0, in, e);
            }
        }
    }
    // dt, x (or dt x) and dy into shared memory [channel][row], B and C into theirs; zeros in
    // rows that no sequence covers, which then neither decay nor add anything.
    template <bool TIMES>
    __device__ __forceinline__ void lay(const SsmArgs& a, const ChannelBlock& cb, long long t0, uint32_t in, float* s_dt,
                                        float* s_x, float* s_dy, T* s_B, T* s_C) const {
        const T* Bp = static_cast<const T*>(a.Bm) + (long long)cb.g * a.N;
        const T* Cp = static_cast<const T*>(a.Cm) + (long long)cb.g * a.N;
#pragma unroll
        for (int e = 0; e < BPT; ++e) {
            const int k = e * kThreads + threadIdx.x;
            if (k >= TT * NP) continue;
            s_B[k] = kAhead ? nB[kAhead ? e : 0] : bc(Bp, a.bs, a, t0, in, e);
            s_C[k] = kAhead ? nC[kAhead ? e : 0] : bc(Cp, a.cs, a, t0, in, e);
        }
        cp_async_wait();
#pragma unroll
        for (int it = 0; it < NSLOT; ++it) {
            const int slot = it * kThreads + threadIdx.x, row = slot / VPR, c0 = (slot % VPR) * 8;
            if (row >= TT) break;
            const int n = in >> row & 1 ? cb.n - c0 : 0, d = cb.d0 + c0;
            float xx[8], vv[8], gg[8];
            read(0, it, xx);
            read(1, it, vv);
            read(2, it, gg);
            if (a.z != nullptr) {
                float zz[8];
                read(3, it, zz);
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const F2 q{zz[i], zz[i + 1]}, o = mul2(F2{gg[i], gg[i + 1]}, mul2(q, sigmoid2(q)));
                    gg[i] = o.x;
                    gg[i + 1] = o.y;
                }
            }
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                F2 dt{vv[i], vv[i + 1]};
                if (a.delta_bias)
                    dt = add2(dt, F2{i < n ? __ldg(a.delta_bias + d + i) : 0.f, i + 1 < n ? __ldg(a.delta_bias + d + i + 1) : 0.f});
                if (a.softplus) dt = softplus2(dt);
                if (i >= n) dt.x = 0.f;
                if (i + 1 >= n) dt.y = 0.f;
                const F2 ox = TIMES ? mul2(dt, F2{xx[i], xx[i + 1]}) : F2{xx[i], xx[i + 1]};
                const int o = cell<TT>(c0 + i, row), o2 = cell<TT>(c0 + i + 1, row);
                s_dt[o] = dt.x;
                s_dt[o2] = dt.y;
                s_x[o] = ox.x;
                s_x[o2] = ox.y;
                s_dy[o] = gg[i];
                s_dy[o2] = gg[i + 1];
            }
        }
    }
};

// What the join needs to know of a segment.
constexpr uint8_t kStarts = 1;      // holds a sequence's first row (its last state is its own)
constexpr uint8_t kEnds = 2;        // the sequence of its first row ends in it
constexpr uint8_t kFirst = 4;       // its first row is a sequence's first row

// This thread's channels and states: channel slot k (of two), register pair m (of two).
template <int S>
struct Place {
    static constexpr int CH = channels<S>(), NP = 4 * S;
    int lane, warp, s, csw, sw, d[2];
    bool live[2];
    int ch[2];
    __device__ __forceinline__ Place(const ChannelBlock& cb) {
        const int tid = threadIdx.x;
        lane = tid & 31;
        warp = tid >> 5;
        s = tid % S;
        csw = S >= 2 ? tid & 1 : 0;           // lanes on the upper side of the first channel exchange
        sw = S <= 16 ? tid >> 4 & 1 : 0;      // .. and of the first state exchange
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            ch[k] = tid / S + (k ^ csw) * (CH / 2);
            live[k] = ch[k] < cb.n;
            d[k] = cb.d0 + (live[k] ? ch[k] : 0);
        }
    }
    __device__ __forceinline__ int n(int m) const { return s * 4 + 2 * (m ^ sw); }   // first state of pair m
    // a pair of a caller's [.., D, N] array, at row q
    __device__ __forceinline__ F2 get(const float* p, long long q, const SsmArgs& a, int k, int m) const {
        F2 v{0.f, 0.f};
        if (p == nullptr || !live[k]) return v;
        const float* at = p + (q * a.D + d[k]) * a.N + n(m);
        if (n(m) < a.N) v.x = at[0];
        if (n(m) + 1 < a.N) v.y = at[1];
        return v;
    }
    // A log2(e); -1 for the states that pad N: an infinite step then gives their decay as 0, where
    // e^{inf 0} would be NaN and reach the sums over the states.
    __device__ __forceinline__ F2 rates(const SsmArgs& a, int k, int m) const {
        F2 v = mul2(get(a.A, 0, a, k, m), both(kLog2e));
        if (n(m) >= a.N) v.x = -1.0f;
        if (n(m) + 1 >= a.N) v.y = -1.0f;
        return v;
    }
    __device__ __forceinline__ void put(float* p, long long q, const SsmArgs& a, int k, int m, F2 v) const {
        if (p == nullptr || !live[k]) return;
        float* at = p + (q * a.D + d[k]) * a.N + n(m);
        if (n(m) < a.N) at[0] = v.x;
        if (n(m) + 1 < a.N) at[1] = v.y;
    }
    // the same in a workspace array [.., D, NP]
    __device__ __forceinline__ F2 load(const float* p, long long q, int D, int k, int m) const {
        if (!live[k]) return F2{0.f, 0.f};
        const float2 v = *reinterpret_cast<const float2*>(p + (q * D + d[k]) * NP + n(m));
        return F2{v.x, v.y};
    }
    __device__ __forceinline__ void store(float* p, long long q, int D, int k, int m, F2 v) const {
        if (live[k]) *reinterpret_cast<float2*>(p + (q * D + d[k]) * NP + n(m)) = make_float2(v.x, v.y);
    }
};

template <typename T, int S>
constexpr size_t summary_smem() {
    return Raw<T, S, true>::kBytes + sizeof(float) * 3 * channels<S>() * tile_rows<S>() + sizeof(T) * 2 * tile_rows<S>() * 4 * S;
}

template <typename T, int S, bool ALIGNED>
__global__ void __launch_bounds__(kThreads, 4) ssm_bwd_summary_kernel(SsmArgs a, Segments seg, int nblk, float* hseg,
                                                                     float* rseg, float* dtseg, float* hck, float* dtck,
                                                                     uint8_t* flags) {
    constexpr int CH = channels<S>(), TT = tile_rows<S>(), NP = 4 * S;
    extern __shared__ __align__(16) float sm[];
    Raw<T, S, ALIGNED> raw(sm);
    float *s_dt = sm + Raw<T, S, ALIGNED>::kBytes / 4, *s_u = s_dt + CH * TT, *s_dy = s_u + CH * TT;
    T *s_B = reinterpret_cast<T*>(s_dy + CH * TT), *s_C = s_B + TT * NP;
    const long long sg = blockIdx.x / nblk;
    const ChannelBlock cb = channel_block<CH>(blockIdx.x % nblk, a.D, a.G);
    const Place<S> at(cb);
    if (sg >= seg.count) {   // sequences without rows hand their state's gradient through
        for (long long q = sg - seg.count; q < a.num_seqs; q += gridDim.x / nblk - seg.count) {
            long long b, e;
            if (!check_seq(a.cu, (int)q, a.M, a.T, a.dev_status, b, e) || b != e) continue;
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int m = 0; m < 2; ++m) at.put(a.dh0, q, a, k, m, at.get(a.d_hT, q, a, k, m));
        }
        return;
    }
    const long long t0 = sg * seg.len, t1 = t0 + seg.len < a.M ? t0 + seg.len : a.M;
    F2 A2[2][2], h[2][2], p[2][2], g[2][2];
    float dtsum[2] = {0.f, 0.f};
    bool open = true;   // the first row's sequence goes on: what follows it must not touch g (0 * NaN)
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            A2[k][m] = at.rates(a, k, m);
            h[k][m] = g[k][m] = F2{0.f, 0.f};
            p[k][m] = F2{1.f, 1.f};
        }
    uint8_t f = 0;
    float *ck = hck + t0 / kSub * a.D * NP, *dk = dtck + t0 / kSub * a.D;   // the next checkpoint
    Events ev = find_events(a, t0, TT), evn{0, 0, 0};
    raw.load(a, cb, t0, ev.in);
    for (long long tile = t0; tile < t1; tile += TT, ev = evn) {
        if (tile == t0 && ((ev.first & 1) || !(ev.in & 1))) f |= kFirst;
        if (tile == t0 && !(ev.in & 1)) f |= kEnds;
        if (ev.first) f |= kStarts;
        if (ev.last) f |= kEnds;
        if (tile != t0) __syncthreads();
        raw.template lay<true>(a, cb, tile, ev.in, s_dt, s_u, s_dy, s_B, s_C);
        __syncthreads();
        if (tile + TT < t1) {
            evn = find_events(a, tile + TT, TT);
            raw.load(a, cb, tile + TT, evn.in);
        }
#pragma unroll 1
        for (int i0 = 0; i0 < TT; i0 += kSub) {
            if (tile + i0 >= t1) break;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if (at.live[k]) {
                    *reinterpret_cast<float2*>(ck + at.d[k] * NP + at.n(0)) = make_float2(h[k][0].x, h[k][0].y);
                    *reinterpret_cast<float2*>(ck + at.d[k] * NP + at.n(1)) = make_float2(h[k][1].x, h[k][1].y);
                    if (at.s == 0) dk[at.d[k]] = dtsum[k];
                }
            }
            ck += a.D * NP;
            dk += a.D;
            // four rows, with or without sequences that begin or end there
            auto rows = [&](auto evc, auto goes_on) {
                constexpr bool EV = decltype(evc)::value, OPEN = decltype(goes_on)::value;
#pragma unroll
                for (int i = i0; i < i0 + kSub; i += 4) {
                    float4 d4[2], u4[2], g4[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        d4[k] = *reinterpret_cast<const float4*>(&s_dt[cell<TT>(at.ch[k], i)]);
                        u4[k] = *reinterpret_cast<const float4*>(&s_u[cell<TT>(at.ch[k], i)]);
                        g4[k] = *reinterpret_cast<const float4*>(&s_dy[cell<TT>(at.ch[k], i)]);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (EV && (ev.first >> (i + j) & 1)) {
                            const SeqRange r = find_seq(a.cu, a.num_seqs, a.M, a.T, tile + i + j);
#pragma unroll
                            for (int k = 0; k < 2; ++k)
#pragma unroll
                                for (int m = 0; m < 2; ++m) {
                                    h[k][m] = at.get(a.h0, r.q, a, k, m);
                                }
                            if (tile + i + j > t0) open = false;
                        }
#pragma unroll
                        for (int m = 0; m < 2; ++m) {
                            const F2 B = lds_pair(s_B + (i + j) * NP + at.n(m)), C = lds_pair(s_C + (i + j) * NP + at.n(m));
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const float dt = j == 0 ? d4[k].x : j == 1 ? d4[k].y : j == 2 ? d4[k].z : d4[k].w;
                                const float u = j == 0 ? u4[k].x : j == 1 ? u4[k].y : j == 2 ? u4[k].z : u4[k].w;
                                const float dy = j == 0 ? g4[k].x : j == 1 ? g4[k].y : j == 2 ? g4[k].z : g4[k].w;
                                const F2 e = ex2(mul2(both(dt), A2[k][m]));
                                h[k][m] = fma2(e, h[k][m], mul2(both(u), B));
                                if (EV ? open : OPEN) {
                                    p[k][m] = mul2(p[k][m], e);
                                    g[k][m] = fma2(p[k][m], mul2(both(dy), C), g[k][m]);
                                }
                                if (m == 0) dtsum[k] += dt;
                            }
                        }
                        if (EV && open && (ev.last >> (i + j) & 1)) {
                            const SeqRange r = find_seq(a.cu, a.num_seqs, a.M, a.T, tile + i + j);
#pragma unroll
                            for (int k = 0; k < 2; ++k)
#pragma unroll
                                for (int m = 0; m < 2; ++m) {
                                    g[k][m] = fma2(p[k][m], at.get(a.d_hT, r.q, a, k, m), g[k][m]);
                                }
                            open = false;
                        }
                    }
                }
            };
            if ((ev.first | ev.last) >> i0 & ((1u << kSub) - 1)) rows(std::true_type{}, std::true_type{});
            else if (open) rows(std::false_type{}, std::true_type{});
            else rows(std::false_type{}, std::false_type{});
        }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            at.store(hseg, sg, a.D, k, m, h[k][m]);
            at.store(rseg, sg, a.D, k, m, g[k][m]);
        }
        if (at.s == 0 && at.live[k]) dtseg[sg * a.D + at.d[k]] = dtsum[k];
    }
    if (blockIdx.x % nblk == 0 && threadIdx.x == 0) flags[sg] = f;
}

// y = 0: hseg[k] (segment k's own last state) -> the state in front of it.
// y = 1: rseg[k] (what its rows send to the state in front) -> the gradient of its last state.
// A chain along the segments; eight segments' values are loaded ahead of their use.
__global__ void __launch_bounds__(128) ssm_bwd_join_kernel(SsmArgs a, int NP, long long K, float* hseg, float* rseg,
                                                           const float* dtseg, const uint8_t* flags) {
    constexpr int U = 8;
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x, DN = (long long)a.D * NP;
    if (i >= DN) return;
    const long long d = i / NP;
    const int n = (int)(i - d * NP);
    const float A2 = n < a.N ? a.A[d * a.N + n] * kLog2e : -1.0f;
    const bool fwd = blockIdx.y == 0;
    float* v = fwd ? hseg : rseg;
    float c = 0.f;
    for (long long k0 = 0; k0 < K; k0 += U) {
        float own[U], dec[U];
        uint8_t f[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long k = fwd ? k0 + u : K - 1 - k0 - u;
            const bool in = k0 + u < K;
            own[u] = in ? v[k * DN + i] : 0.f;
            dec[u] = in ? dtseg[k * a.D + d] : 0.f;
            f[u] = in ? flags[k] : 0;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long k = fwd ? k0 + u : K - 1 - k0 - u;
            if (k0 + u >= K) break;
            v[k * DN + i] = c;
            const float through = fmaf(ex2(dec[u] * A2), c, own[u]);
            if (fwd) c = f[u] & kStarts ? own[u] : through;
            else c = f[u] & kFirst ? 0.f : f[u] & kEnds ? own[u] : through;
        }
    }
}

// The sums over a channel's S lanes of four rows' values, in two steps.  Channels first, row by
// row (the lanes of a pair hold the two channels in swapped order): of v[slot] the lane keeps slot
// 0.  Then rows: S = 2 has all four; S >= 4 ends with rows 2 (s & 2) / 2 .. + 1 in r[0], r[1].
template <int S>
__device__ __forceinline__ float channel_exchange(float v0, float v1) {
    return v0 + __shfl_xor_sync(0xffffffffu, v1, 1);
}
template <int S>
__device__ __forceinline__ void row_exchange(const Place<S>& at, float (&r)[4]) {
    if constexpr (S > 2) {
        const bool up = at.s & 2;   // keeps rows 2 and 3
        F2 keep = up ? F2{r[2], r[3]} : F2{r[0], r[1]};
        keep = add2(keep, shfl2(up ? F2{r[0], r[1]} : F2{r[2], r[3]}, 2));
#pragma unroll
        for (int m = 4; m < S; m <<= 1) keep = add2(keep, shfl2(keep, m));
        r[0] = keep.x;
        r[1] = keep.y;
    }
}

// The sums over a warp's channels of a row's dB and dC pairs, written to red[2][NP].
template <int S>
__device__ __forceinline__ void channel_sum(const Place<S>& at, const F2 (&dB)[2], const F2 (&dC)[2], float* red) {
    constexpr int NP = 4 * S;
    const int n0 = at.n(0);
    if constexpr (S == 32) {
        *reinterpret_cast<float4*>(red + n0) = make_float4(dB[0].x, dB[0].y, dB[1].x, dB[1].y);
        *reinterpret_cast<float4*>(red + NP + n0) = make_float4(dC[0].x, dC[0].y, dC[1].x, dC[1].y);
    } else {
        const F2 b = add2(dB[0], shfl2(dB[1], 16)), c = add2(dC[0], shfl2(dC[1], 16));
        if constexpr (S == 16) {
            *reinterpret_cast<float2*>(red + n0) = make_float2(b.x, b.y);
            *reinterpret_cast<float2*>(red + NP + n0) = make_float2(c.x, c.y);
        } else {
            const bool up = at.lane & 8;   // keeps dC
            F2 k = up ? c : b;
            k = add2(k, shfl2(up ? b : c, 8));
            if constexpr (S == 8) {
                *reinterpret_cast<float2*>(red + (up ? NP : 0) + n0) = make_float2(k.x, k.y);
            } else {
                const bool odd = at.lane & 4;   // keeps the pair's second state
                float o = odd ? k.y : k.x;
                o += __shfl_xor_sync(0xffffffffu, odd ? k.x : k.y, 4);
#pragma unroll
                for (int m = 2; m >= S; m >>= 1) o += __shfl_xor_sync(0xffffffffu, o, m);
                if ((at.lane & 3) < S) red[(up ? NP : 0) + n0 + odd] = o;
            }
        }
    }
}

// A thread's own checkpoint (8 floats, two sums of dt) in its slots of shared memory, copied one
// checkpoint ahead of its use.
constexpr int kCk = 10 * kThreads;   // [4 pairs][thread] of float2, then [2][thread]

template <typename T, int S>
constexpr size_t grad_smem() {
    return Raw<T, S, true>::kBytes + sizeof(float) * (3 * channels<S>() * tile_rows<S>() + 2 * kWarps * kSub * 2 * 4 * S + 3 * kCk + 8 * kThreads) +
           sizeof(T) * 2 * tile_rows<S>() * 4 * S;
}

template <typename T, int S, bool ALIGNED>
__global__ void __launch_bounds__(kThreads, 3) ssm_bwd_grad_kernel(SsmArgs a, Segments seg, int nblk, const float* hseg,
                                                                  const float* rseg, const float* hck, const float* dtck,
                                                                  float* part, float* bcpart) {
    constexpr int CH = channels<S>(), TT = tile_rows<S>(), NP = 4 * S, VPR = CH / 8;
    extern __shared__ __align__(16) float sm[];
    Raw<T, S, ALIGNED> raw(sm);
    // dt, x and dy of the tile; as rows are finished, dx, ddelta (without
    // softplus' slope) and y in their place
    float *s_dt = sm + Raw<T, S, ALIGNED>::kBytes / 4, *s_x = s_dt + CH * TT, *s_dy = s_x + CH * TT, *s_red = s_dy + CH * TT;
    float* s_ck = s_red + 2 * kWarps * kSub * 2 * NP;   // two checkpoints, then the segment's incoming state
    T *s_B = reinterpret_cast<T*>(s_ck + 3 * kCk + 8 * kThreads), *s_C = s_B + TT * NP;
    const long long sg = blockIdx.x / nblk;
    const int blk = blockIdx.x % nblk, tid = threadIdx.x;
    const ChannelBlock cb = channel_block<CH>(blk, a.D, a.G);
    const Place<S> at(cb);
    const long long t0 = sg * seg.len, t1 = t0 + seg.len < a.M ? t0 + seg.len : a.M;
    // rows that the segment's incoming state reaches: those of the sequence it is cut out of
    const SeqRange r0 = find_seq(a.cu, a.num_seqs, a.M, a.T, t0);
    const int nrow = (int)(t1 - t0), reach = r0.ok && r0.b < t0 ? (int)(r0.e - t0 < nrow ? r0.e - t0 : nrow) : 0;

    F2 A2[2][2], dh[2][2], dA[2][2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            A2[k][m] = at.rates(a, k, m);
            dh[k][m] = at.load(rseg, sg, a.D, k, m);
            dA[k][m] = F2{0.f, 0.f};
        }
    auto slot = [&](int which, int k, int m) { return s_ck + which * kCk + ((k * 2 + m) * kThreads + tid) * 2; };
    auto slot_dt = [&](int which, int k) { return s_ck + which * kCk + 8 * kThreads + k * kThreads + tid; };
    const float *ck = hck + (t1 - 1) / kSub * a.D * NP, *dk = dtck + (t1 - 1) / kSub * a.D;   // fetched next
    auto fetch = [&](int which) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (at.live[k]) {
                cp_async8(slot(which, k, 0), ck + at.d[k] * NP + at.n(0));
                cp_async8(slot(which, k, 1), ck + at.d[k] * NP + at.n(1));
                cp_async4(slot_dt(which, k), dk + at.d[k]);
            }
        }
        ck -= a.D * NP;
        dk -= a.D;
    };
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const F2 v = at.load(hseg, sg, a.D, k, m), z{0.f, 0.f};
            *reinterpret_cast<float2*>(slot(2, k, m)) = make_float2(v.x, v.y);
            if (!at.live[k])
                for (int w = 0; w < 2; ++w) {
                    *reinterpret_cast<float2*>(slot(w, k, m)) = make_float2(z.x, z.y);
                    *slot_dt(w, k) = 0.f;
                }
        }
    fetch(0);
    F2 sD[S == 1 ? 2 : 1] = {};     // dy x of the rows that this lane finishes
    float skip[2];
    float* s_sb = s_ck + 3 * kCk + tid;   // this thread's sums of ddelta over its rows, [8][thread]
#pragma unroll
    for (int i = 0; i < 8; ++i) s_sb[i * kThreads] = 0.f;
#pragma unroll
    for (int k = 0; k < 2; ++k) skip[k] = a.Dskip && at.live[k] ? a.Dskip[at.d[k]] : 0.f;
    int phase = 0;

    const int last_tile = (nrow - 1) / TT * TT;   // rows count from the segment's first
    Events ev = find_events(a, t0 + last_tile, TT), evn{0, 0, 0};
    raw.load(a, cb, t0 + last_tile, ev.in);
    float* bc = bcpart + ((long long)blk * a.M + t0 + last_tile) * 2 * a.N;   // the tile's dB, dC of this channel block
    for (int tile = last_tile; tile >= 0; tile -= TT, ev = evn, bc -= 2 * TT * a.N) {
        raw.template lay<false>(a, cb, t0 + tile, ev.in, s_dt, s_x, s_dy, s_B, s_C);
        __syncthreads();
#pragma unroll 1
        for (int i0 = TT - kSub; i0 >= 0; i0 -= kSub) {
            if (tile + i0 >= nrow) continue;
            // the state in front of these rows: the checkpoint, and what reaches it of the segment's
            cp_async_wait();
            if (tile + i0 < reach) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const F2 cum = both(*slot_dt(phase, k));
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        float2* v = reinterpret_cast<float2*>(slot(phase, k, m));
                        const float2 in = *reinterpret_cast<const float2*>(slot(2, k, m));
                        const F2 o = fma2(ex2(mul2(cum, A2[k][m])), F2{in.x, in.y}, F2{v->x, v->y});
                        *v = make_float2(o.x, o.y);
                    }
                }
            }
            auto in_front = [&](int k, int m) {
                const float2 v = *reinterpret_cast<const float2*>(slot(phase, k, m));
                return F2{v.x, v.y};
            };
            if (tile + i0 > 0) fetch(phase ^ 1);
            float* red = s_red + (phase * kWarps + at.warp) * kSub * 2 * NP;
            auto rows = [&](auto evc) {
                constexpr bool EV = decltype(evc)::value;
                F2 ha[kSub][2][2], ea[kSub][2][2];
#pragma unroll
                for (int i = 0; i < kSub; i += 4) {
                    float4 d4[2], x4[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        d4[k] = *reinterpret_cast<const float4*>(&s_dt[cell<TT>(at.ch[k], i0 + i)]);
                        x4[k] = *reinterpret_cast<const float4*>(&s_x[cell<TT>(at.ch[k], i0 + i)]);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int r = i + j;
                        SeqRange sr{0, 0, 0, false};
                        const bool first = EV && (ev.first >> (i0 + r) & 1);
                        if (first) sr = find_seq(a.cu, a.num_seqs, a.M, a.T, t0 + tile + i0 + r);
#pragma unroll
                        for (int m = 0; m < 2; ++m) {
                            const F2 B = lds_pair(s_B + (i0 + r) * NP + at.n(m));
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const float dt = j == 0 ? d4[k].x : j == 1 ? d4[k].y : j == 2 ? d4[k].z : d4[k].w;
                                const float x = j == 0 ? x4[k].x : j == 1 ? x4[k].y : j == 2 ? x4[k].z : x4[k].w;
                                F2 hp = r > 0 ? ha[r > 0 ? r - 1 : 0][k][m] : in_front(k, m);
                                if (first) hp = at.get(a.h0, sr.q, a, k, m);
                                ea[r][k][m] = ex2(mul2(both(dt), A2[k][m]));
                                ha[r][k][m] = fma2(ea[r][k][m], hp, mul2(both(dt * x), B));
                            }
                        }
                    }
                }
#pragma unroll
                for (int i = kSub - 4; i >= 0; i -= 4) {
                    float4 d4[2], x4[2], g4[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        d4[k] = *reinterpret_cast<const float4*>(&s_dt[cell<TT>(at.ch[k], i0 + i)]);
                        x4[k] = *reinterpret_cast<const float4*>(&s_x[cell<TT>(at.ch[k], i0 + i)]);
                        g4[k] = *reinterpret_cast<const float4*>(&s_dy[cell<TT>(at.ch[k], i0 + i)]);
                    }
                    constexpr int KO = S == 1 ? 2 : 1;   // channels whose sums a lane ends with
                    float pv[KO][4], qv[KO][4], yv[KO][4];
#pragma unroll
                    for (int j = 3; j >= 0; --j) {
                        const int r = i + j;
                        const bool first = EV && (ev.first >> (i0 + r) & 1), last = EV && (ev.last >> (i0 + r) & 1);
                        SeqRange sr{0, 0, 0, false};
                        if (first || last) sr = find_seq(a.cu, a.num_seqs, a.M, a.T, t0 + tile + i0 + r);
                        F2 B[2], C[2], dB[2], dC[2];
                        float ps[2], qs[2], ys[2];
#pragma unroll
                        for (int m = 0; m < 2; ++m) {
                            B[m] = lds_pair(s_B + (i0 + r) * NP + at.n(m));
                            C[m] = lds_pair(s_C + (i0 + r) * NP + at.n(m));
                        }
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const float dt = j == 0 ? d4[k].x : j == 1 ? d4[k].y : j == 2 ? d4[k].z : d4[k].w;
                            const float x = j == 0 ? x4[k].x : j == 1 ? x4[k].y : j == 2 ? x4[k].z : x4[k].w;
                            const float dy = j == 0 ? g4[k].x : j == 1 ? g4[k].y : j == 2 ? g4[k].z : g4[k].w;
                            const F2 u = both(dt * x);
                            F2 p{0.f, 0.f}, q{0.f, 0.f}, y{0.f, 0.f};
#pragma unroll
                            for (int m = 0; m < 2; ++m) {
                                F2 hp = r > 0 ? ha[r > 0 ? r - 1 : 0][k][m] : in_front(k, m);
                                if (first) hp = at.get(a.h0, sr.q, a, k, m);
                                if (last) dh[k][m] = at.get(a.d_hT, sr.q, a, k, m);
                                dh[k][m] = fma2(C[m], both(dy), dh[k][m]);
                                y = m ? fma2(C[m], ha[r][k][m], y) : mul2(C[m], ha[r][k][m]);
                                dB[m] = k ? fma2(dh[k][m], u, dB[m]) : mul2(dh[k][m], u);
                                dC[m] = k ? fma2(ha[r][k][m], both(dy), dC[m]) : mul2(ha[r][k][m], both(dy));
                                p = m ? fma2(dh[k][m], B[m], p) : mul2(dh[k][m], B[m]);
                                dh[k][m] = mul2(dh[k][m], ea[r][k][m]);
                                const F2 w = mul2(dh[k][m], hp);
                                dA[k][m] = fma2(w, both(dt), dA[k][m]);
                                q = m ? fma2(w, A2[k][m], q) : mul2(w, A2[k][m]);
                                if (first) {
                                    at.put(a.dh0, sr.q, a, k, m, dh[k][m]);
                                    dh[k][m] = F2{0.f, 0.f};
                                }
                            }
                            ps[k] = p.x + p.y;
                            qs[k] = q.x + q.y;
                            ys[k] = y.x + y.y;
                        }
                        if constexpr (S == 1) {
#pragma unroll
                            for (int k = 0; k < KO; ++k) {
                                pv[k][j] = ps[k];
                                qv[k][j] = qs[k];
                                yv[k][j] = ys[k];
                            }
                        } else {
                            pv[0][j] = channel_exchange<S>(ps[0], ps[1]);
                            qv[0][j] = channel_exchange<S>(qs[0], qs[1]);
                            yv[0][j] = channel_exchange<S>(ys[0], ys[1]);
                        }
                        channel_sum<S>(at, dB, dC, red + r * 2 * NP);
                    }
                    // p, q and y over the lanes; the lane that ends with a row (or two, or four) of a
                    // channel finishes it, in place of the row's dt, x and dy, which all lanes have read
                    row_exchange<S>(at, pv[0]);
                    row_exchange<S>(at, qv[0]);
                    row_exchange<S>(at, yv[0]);
#pragma unroll
                    for (int k = 0; k < KO; ++k) {
#pragma unroll
                        for (int w = 0; w < (S >= 4 ? 1 : 2); ++w) {
                            const bool up = S >= 4 ? (at.s & 2) != 0 : w;
                            const F2 dt = up ? F2{d4[k].z, d4[k].w} : F2{d4[k].x, d4[k].y};
                            const F2 x = up ? F2{x4[k].z, x4[k].w} : F2{x4[k].x, x4[k].y};
                            const F2 dy = up ? F2{g4[k].z, g4[k].w} : F2{g4[k].x, g4[k].y};
                            const F2 p{pv[k][2 * w], pv[k][2 * w + 1]}, q{qv[k][2 * w], qv[k][2 * w + 1]}, y{yv[k][2 * w], yv[k][2 * w + 1]};
                            const F2 ox = fma2(p, dt, mul2(both(skip[k]), dy));
                            const F2 ov = fma2(p, x, mul2(q, both(1.0f / kLog2e)));
                            const F2 oy = fma2(both(skip[k]), x, y);
                            sD[k] = fma2(dy, x, sD[k]);
                            if (S < 8 || at.s < 4) {
                                const int o = cell<TT>(at.ch[k], i0 + i) + (up ? 2 : 0);
                                *reinterpret_cast<float2*>(s_dt + o) = make_float2(ox.x, ox.y);
                                *reinterpret_cast<float2*>(s_x + o) = make_float2(ov.x, ov.y);
                                *reinterpret_cast<float2*>(s_dy + o) = make_float2(oy.x, oy.y);
                            }
                        }
                    }
                }
            };
            if ((ev.first | ev.last) >> i0 & ((1u << kSub) - 1)) rows(std::true_type{});
            else rows(std::false_type{});
            __syncthreads();
            for (int k = tid; k < kSub * 2 * NP; k += kThreads) {
                const int r = k / (2 * NP), w = k % (2 * NP) / NP, n = k % NP;
                if (n >= a.N || tile + i0 + r >= nrow) continue;
                float t = 0.f;
#pragma unroll
                for (int x = 0; x < kWarps; ++x) t += s_red[(phase * kWarps + x) * kSub * 2 * NP + k];
                bc[((i0 + r) * 2 + w) * a.N + n] = t;
            }
            phase ^= 1;
        }
        // rows and channels as they were staged: dx, ddelta, dz and the bias' gradient (what the
        // lanes left was written before the last barrier).  The raw inputs are read once more,
        // and the next tile's take their place while these are worked on.
        constexpr int NSLOT = Raw<T, S, ALIGNED>::NSLOT;
        Pack<T, 8> pv[NSLOT], pg[NSLOT], pz[NSLOT];
#pragma unroll
        for (int it = 0; it < NSLOT; ++it) {
            pv[it] = raw.get(1, it);
            pg[it] = raw.get(2, it);
            pz[it] = raw.get(3, it);   // without a z: nothing that is used
        }
        if (tile > 0) {
            evn = find_events(a, t0 + tile - TT, TT);
            raw.load(a, cb, t0 + tile - TT, evn.in);
        }
#pragma unroll
        for (int it = 0; it < NSLOT; ++it) {
            const int slot = it * kThreads + tid, row = slot / VPR, c0 = (slot % VPR) * 8;
            const int cn = max(0, min(8, cb.n - c0)), d = cb.d0 + c0;
            if (row >= TT || !(ev.in >> row & 1) || cn == 0) continue;
            const long long t = t0 + tile + row;
            float dx[8], v[8], z[8], g[8];
            unpack<T, 8>(pv[it], v);
            unpack<T, 8>(pg[it], g);
            unpack<T, 8>(pz[it], z);
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const int o = cell<TT>(c0 + i, row), o2 = cell<TT>(c0 + i + 1, row);
                dx[i] = s_dt[o];
                dx[i + 1] = s_dt[o2];
                F2 ov{s_x[o], s_x[o2]};
                if (a.softplus) {
                    F2 dl{v[i], v[i + 1]};
                    if (a.delta_bias)
                        dl = add2(dl, F2{i < cn ? __ldg(a.delta_bias + d + i) : 0.f, i + 1 < cn ? __ldg(a.delta_bias + d + i + 1) : 0.f});
                    ov = mul2(ov, sigmoid2(dl));
                }
                s_sb[i * kThreads] += ov.x;
                s_sb[(i + 1) * kThreads] += ov.y;
                v[i] = ov.x;
                v[i + 1] = ov.y;
                if (a.z != nullptr) {
                    const F2 zz{z[i], z[i + 1]}, sg1 = sigmoid2(zz);
                    const F2 slope = mul2(sg1, fma2(zz, fma2(sg1, both(-1.0f), both(1.0f)), both(1.0f)));
                    const F2 oz = mul2(mul2(F2{g[i], g[i + 1]}, F2{s_dy[o], s_dy[o2]}), slope);
                    z[i] = oz.x;
                    z[i + 1] = oz.y;
                }
            }
            store8<T, ALIGNED>(static_cast<T*>(a.dx) + t * a.D + d, dx, cn);
            store8<T, ALIGNED>(static_cast<T*>(a.ddelta) + t * a.D + d, v, cn);
            if (a.z != nullptr) store8<T, ALIGNED>(static_cast<T*>(a.dz) + t * a.D + d, z, cn);
        }
        __syncthreads();   // the next tile is laid over this one
    }
    // part[segment]: dA [D][N], dDskip [D], the bias' gradient [D]
    float* pseg = part + sg * ((long long)a.D * a.N + 2 * a.D);
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int m = 0; m < 2; ++m) at.put(pseg, 0, a, k, m, dA[k][m]);
    // dDskip: over the two (S >= 4) lanes that finish a channel's rows
    float* pD = pseg + (long long)a.D * a.N;
#pragma unroll
    for (int k = 0; k < (S == 1 ? 2 : 1); ++k) {
        float t = sD[k].x + sD[k].y;
        if (S >= 4) t += __shfl_xor_sync(0xffffffffu, t, 2);
        if (at.live[k] && at.s < 2) pD[at.d[k]] = t;
    }
    // the bias: a thread's slots all have the same channels; RPP partial sums per channel
    constexpr int RPP = kThreads / VPR;
    const float* s0 = s_ck + 3 * kCk;
    __syncthreads();
    for (int c = tid; c < cb.n; c += kThreads) {
        float t = 0.f;
        for (int r = 0; r < RPP; ++r) t += s0[(c % 8) * kThreads + r * VPR + c / 8];
        pD[a.D + cb.d0 + c] = t;
    }
}

// dB, dC: the channel blocks' partial sums of a row, rounded once.
template <typename T>
__global__ void __launch_bounds__(256) ssm_bwd_bc_kernel(SsmArgs a, int per, const float* bcpart) {
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;   // (row, group, dB or dC, state)
    const long long t = i / ((long long)a.G * 2 * a.N);
    if (t >= a.M) return;
    const int k = (int)(i % ((long long)a.G * 2 * a.N)), g = k / (2 * a.N), w = k % (2 * a.N) / a.N, n = k % a.N;
    if (a.cu != nullptr && !find_seq(a.cu, a.num_seqs, a.M, a.T, t).ok) return;
    const float* p = bcpart + (((long long)g * per * a.M + t) * 2 + w) * a.N + n;
    float s = 0.f;
#pragma unroll 16
    for (int b = 0; b < per; ++b) s += __ldg(p + (long long)b * a.M * 2 * a.N);
    static_cast<T*>(w ? a.dC : a.dB)[(t * a.G + g) * a.N + n] = from_f32<T>(s);
}

struct Layout {
    Segments seg;
    int nblk, per;    // channel blocks in all, per group
    size_t hseg, rseg, dtseg, hck, dtck, part, bcpart, flags, bytes;
};
// Lanes per channel pair (four states per lane).
int lanes_of(int N) { return N <= 4 ? 1 : N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : N <= 64 ? 16 : 32; }
// Segments of 32 to 256 rows: the longest that still give twelve CTAs per SM (of which three or
// four run at a time: the last turn's idle SMs are then a small share).  Every segment costs a
// state, a state gradient and a partial sum of dA.  4 x 2048 rows, 2048 channels: 583 us with 128
// rows, 600 us with 160 (whose turns come out more even), 622 us with 64.
Layout layout(long long M, int D, int N, int G) {
    Layout l;
    const int S = lanes_of(N), CH = 2 * kThreads / S;
    l.per = (D / G + CH - 1) / CH;
    l.nblk = l.per * G;
    l.seg.len = 256;
    while (l.seg.len > 32 && l.nblk * ((M + l.seg.len - 1) / l.seg.len) < 12LL * kSMs) l.seg.len /= 2;
    l.seg.count = (M + l.seg.len - 1) / l.seg.len;
    l.seg.whole = false;
    const long long K = l.seg.count;
    size_t at = 0;
    auto take = [&](size_t n) { const size_t o = at; at += (n + 255) / 256 * 256; return o; };
    const size_t dn = (size_t)D * N, dnp = (size_t)D * 4 * S;
    l.hseg = take(sizeof(float) * K * dnp);
    l.rseg = take(sizeof(float) * K * dnp);
    l.dtseg = take(sizeof(float) * K * D);
    l.hck = take(sizeof(float) * ((M + kSub - 1) / kSub) * dnp);
    l.dtck = take(sizeof(float) * ((M + kSub - 1) / kSub) * D);
    l.part = take(sizeof(float) * (K > 0 ? K : 1) * (dn + 2 * D));
    l.bcpart = take(sizeof(float) * l.nblk * M * 2 * N);
    l.flags = take(K);
    l.bytes = at;
    return l;
}

template <typename T, int S, bool ALIGNED>
cudaError_t go(const SsmArgs& a, cudaStream_t s) {
    const Layout l = layout(a.M, a.D, a.N, a.G);
    const long long K = l.seg.count;
    float* hseg = reinterpret_cast<float*>(a.ws + l.hseg);
    float* rseg = reinterpret_cast<float*>(a.ws + l.rseg);
    float* dtseg = reinterpret_cast<float*>(a.ws + l.dtseg);
    float* hck = reinterpret_cast<float*>(a.ws + l.hck);
    float* dtck = reinterpret_cast<float*>(a.ws + l.dtck);
    float* part = reinterpret_cast<float*>(a.ws + l.part);
    float* bcpart = reinterpret_cast<float*>(a.ws + l.bcpart);
    uint8_t* flags = a.ws + l.flags;
    const long long extra = a.cu != nullptr || a.T == 0 ? (a.num_seqs < 64 ? a.num_seqs : 64) : 0;
    const long long dn = (long long)a.D * a.N, dnp = (long long)a.D * 4 * S, bc = a.M * a.G * 2 * a.N;
    if (l.nblk * (K + extra) > 0x7fffffffLL || (bc + 255) / 256 > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    constexpr size_t sm1 = summary_smem<T, S>(), sm3 = grad_smem<T, S>();
    cudaError_t e = cudaSuccess;
    if (K + extra > 0) {
        auto k1 = ssm_bwd_summary_kernel<T, S, ALIGNED>;
        if ((e = allow_smem(k1, sm1)) != cudaSuccess) return e;
        k1<<<(unsigned)(l.nblk * (K + extra)), kThreads, sm1, s>>>(a, l.seg, l.nblk, hseg, rseg, dtseg, hck, dtck, flags);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    if (K > 0) {
        ssm_bwd_join_kernel<<<dim3((unsigned)((dnp + 127) / 128), 2), 128, 0, s>>>(a, 4 * S, K, hseg, rseg, dtseg, flags);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        auto k3 = ssm_bwd_grad_kernel<T, S, ALIGNED>;
        if ((e = allow_smem(k3, sm3)) != cudaSuccess) return e;
        k3<<<(unsigned)(l.nblk * K), kThreads, sm3, s>>>(a, l.seg, l.nblk, hseg, rseg, hck, dtck, part, bcpart);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        ssm_bwd_bc_kernel<T><<<(unsigned)((bc + 255) / 256), 256, 0, s>>>(a, l.per, bcpart);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    return launch_colsum(part, (int)K, dn, a.dA, a.D, a.dDskip, a.D, a.ddelta_bias, s);
}

template <typename T, bool ALIGNED>
cudaError_t go_n(const SsmArgs& a, cudaStream_t s) {
    switch (lanes_of(a.N)) {
        case 1: return go<T, 1, ALIGNED>(a, s);
        case 2: return go<T, 2, ALIGNED>(a, s);
        case 4: return go<T, 4, ALIGNED>(a, s);
        case 8: return go<T, 8, ALIGNED>(a, s);
        case 16: return go<T, 16, ALIGNED>(a, s);
        default: return go<T, 32, ALIGNED>(a, s);
    }
}

template <typename T>
cudaError_t go_t(const SsmArgs& a, cudaStream_t s) {
    const int el = sizeof(T);
    const long long row = (long long)a.D * el;
    const bool al = (a.D / a.G) % 8 == 0 && vec_ok(a.x, a.xs * el, 16) && vec_ok(a.delta, a.ds * el, 16) &&
                    vec_ok(a.z, a.zs * el, 16) && vec_ok(a.d_out, row, 16) && vec_ok(a.dx, row, 16) &&
                    vec_ok(a.ddelta, row, 16) && vec_ok(a.dz, row, 16);
    return al ? go_n<T, true>(a, s) : go_n<T, false>(a, s);
}

}  // namespace
}  // namespace ssm

}  // namespace kda
