// kda_ssm_fwd.cuh -- selective state space scan: forward over rows.
//
//   dt = softplus(delta + bias),  h[n] <- e^{dt A[n]} h[n] + dt x B[n]
//   y = sum_n h[n] C[n] + Dskip x,  out = y silu(z)
//
// Per row and channel: N exponentials (they depend on the row, the channel and the state,
// so no product of matrices holds them) and about 4 N fp32 operations.  The special-function
// unit gives 16 exponentials per cycle and SM, which bounds the scan; the bytes (x, delta, z,
// out, once each) take about a third of that time at N = 16.
//
// A CTA of 256 threads owns 128 / S channels of one group.  Its first four warps scan: S lanes
// per channel, NS states per lane in registers for all rows.  The other four stage: rows come
// in tiles, of which every thread holds the next one's x, delta and z of one row and eight
// channels in registers while the current tile is scanned; it forms dt and dt x in fp32 and lays
// them down in shared memory [channel][row], where the scan reads four rows at a time, and B and
// C as they are, side by side, once per tile for all channels.  Two tile buffers and four named
// barriers hand the tiles over, so that neither side waits for the other's latencies (243 us with
// one set of warps doing both, 164 us with two).  The sum over a channel's lanes is taken for
// four rows at once (the lanes swap halves, so that two exchanges and one more serve four sums).
// y goes back through shared memory to the thread that holds the row's x and z.
// 4 x 2048 rows, 2048 channels, 16 states, bf16: 140 us; the exponentials alone (and the gate's
// and softplus') would take 74 us, the bytes 21 us.  256 CTAs on 148 SMs are 86 % balanced, and
// on the SMs with two, the two scanning warps of a scheduler are each a chain along the rows.
//
// Too few channels and sequences to fill the SMs: the rows are cut into segments, aligned to
// the row index and not to sequences.  Pass 1 scans every segment from zero (keeping only the
// last state and the sum of dt), a short pass joins them (the decay over a segment is
// e^{A sum dt}), pass 2 scans again from the right state.  This doubles the exponentials, so
// it is used only below three CTAs on five SMs.  32768 packed rows, 1024 channels, 16 states: 422 us
// (summary 183, join 7, final 244 under the profiler; the exponentials twice would take 280).
#pragma once

#include "kda_ssm.cuh"

namespace kda {
namespace ssm {
namespace {

constexpr int kThreads = 128;

template <int S>
constexpr int tile_rows() { return S >= 4 ? 32 : 8 * S; }

// Named barriers between the scanning and the staging warps: FULL + b, tile buffer b holds a
// tile; DONE + b, its scan has ended (y lies in s_y[b], the inputs may be overwritten).
enum { kFull = 1, kDone = 3 };
template <int ID>
__device__ __forceinline__ void bar_sync(int b) {   // the id is an immediate: the CTA then holds 5 barriers, not all 16
    if (b == 0) asm volatile("bar.sync %0, %1;" ::"n"(ID), "n"(2 * kThreads) : "memory");
    else asm volatile("bar.sync %0, %1;" ::"n"(ID + 1), "n"(2 * kThreads) : "memory");
}
template <int ID>
__device__ __forceinline__ void bar_arrive(int b) {
    if (b == 0) asm volatile("bar.arrive %0, %1;" ::"n"(ID), "n"(2 * kThreads) : "memory");
    else asm volatile("bar.arrive %0, %1;" ::"n"(ID + 1), "n"(2 * kThreads) : "memory");
}

template <typename T, int S, int NS, bool ALIGNED, bool SUMMARY>
__global__ void __launch_bounds__(2 * kThreads, 2) ssm_scan_kernel(SsmArgs a, Segments seg, int nblk, float* hseg, float* dtseg) {
    constexpr int CH = kThreads / S, TT = tile_rows<S>(), NP = S * NS;
    constexpr int VPR = CH / 8;                 // threads per staged row
    constexpr int BPT = (TT * NP + kThreads - 1) / kThreads;   // staged elements of B (and C) per thread
    constexpr bool kAhead = BPT <= 8;           // B and C of the next tile wait in registers
    static_assert(TT * VPR <= kThreads && TT % 4 == 0, "tile");
    extern __shared__ __align__(16) float sm[];   // two tile buffers
    constexpr int NBC = SUMMARY ? 1 : 2;        // B, or B and C side by side
    constexpr int kBuf = (SUMMARY ? 2 : 3) * CH * TT + NBC * TT * NP * (int)sizeof(T) / 4;   // floats

    const long long sg = blockIdx.x / nblk;   // segment, or behind them
    const ChannelBlock cb = channel_block<CH>(blockIdx.x % nblk, a.D, a.G);
    const bool scanner = threadIdx.x < kThreads;
    const int tid = threadIdx.x & (kThreads - 1), ch = tid / S, s = tid % S;
    const bool live = ch < cb.n;
    const int d = cb.d0 + (live ? ch : 0);

    if (!SUMMARY && sg >= seg.count) {
        // behind the segments: sequences without rows hand their state through, bounds are checked
        if (!scanner) return;
        for (long long q = sg - seg.count; q < a.num_seqs; q += gridDim.x / nblk - seg.count) {
            long long b, e;
            if (!check_seq(a.cu, (int)q, a.M, a.T, a.dev_status, b, e) || b != e || a.hT == nullptr || !live) continue;
            const long long at = (q * a.D + d) * a.N;
            for (int n = s * NS; n < s * NS + NS && n < a.N; ++n) a.hT[at + n] = a.h0 ? a.h0[at + n] : 0.f;
        }
        return;
    }

    const long long t0 = sg * seg.len;
    const long long t1 = t0 + seg.len < a.M ? t0 + seg.len : a.M;
    SeqRange r{0, 0, 0, false};

    if (!scanner) {
        // ---- staging: this thread's row of the tile and its eight channels
        const int srow = tid / VPR, sc0 = (tid % VPR) * 8;
        const bool stager = tid < TT * VPR;
        const int scn = stager ? max(0, min(8, cb.n - sc0)) : 0;
        const int sd = cb.d0 + sc0;
        const T* xp = static_cast<const T*>(a.x) + sd;
        const T* dp = static_cast<const T*>(a.delta) + sd;
        const T* zp = static_cast<const T*>(a.z) + sd;
        const T* Bp = static_cast<const T*>(a.Bm) + (long long)cb.g * a.N;
        const T* Cp = static_cast<const T*>(a.Cm) + (long long)cb.g * a.N;
        float bias[8], dsk[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            bias[i] = i < scn && a.delta_bias ? a.delta_bias[sd + i] : 0.f;
            dsk[i] = i < scn && a.Dskip ? a.Dskip[sd + i] : 0.f;
        }
        Pack<T, 8> nx, nd, nz;
        Pack<T, 1> nB[kAhead ? BPT : 1], nC[kAhead ? BPT : 1];   // as loaded: converting would wait for the load
        auto bc = [&](const T* p, long long stride, long long tile, int e) {   // element e of this thread's share
            const int k = e * kThreads + tid, row = k / NP, n = k % NP;
            return row < TT && tile + row < t1 && n < a.N ? load_pack<1>(p + (tile + row) * stride + n) : zero_pack<T, 1>();
        };
        auto fetch = [&](long long tile) {
            const long long t = tile + srow;
            const int n = t < t1 ? scn : 0;
            nx = load8<T, ALIGNED>(xp + t * a.xs, n);
            nd = load8<T, ALIGNED>(dp + t * a.ds, n);
            if (!SUMMARY) nz = a.z ? load8<T, ALIGNED>(zp + t * a.zs, n) : zero_pack<T, 8>();
            if constexpr (kAhead) {
#pragma unroll
                for (int e = 0; e < BPT; ++e) {
                    nB[e] = bc(Bp, a.bs, tile, e);
                    if (!SUMMARY) nC[e] = bc(Cp, a.cs, tile, e);
                }
            }
        };
        auto put = [](T* s_bc, int k, int which, const Pack<T, 1>& p) {   // element k of B (0) or C (1), as it is
            store_pack<T, 1>(s_bc + (k / 4 * NBC + which) * 4 + k % 4, p);
        };
        auto lay = [&](long long tile, float* buf) {   // the fetched tile into a buffer
            float *s_dt = buf, *s_u = s_dt + CH * TT;
            T* s_bc = reinterpret_cast<T*>(s_u + (SUMMARY ? 1 : 2) * CH * TT);
            if (stager) {
                float x[8], v[8];
                unpack<T, 8>(nx, x);
                unpack<T, 8>(nd, v);
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    F2 dt = add2(F2{v[i], v[i + 1]}, F2{bias[i], bias[i + 1]});
                    if (a.softplus) dt = softplus2(dt);
                    const F2 u = mul2(dt, F2{x[i], x[i + 1]});
                    s_dt[cell<TT>(sc0 + i, srow)] = dt.x;
                    s_dt[cell<TT>(sc0 + i + 1, srow)] = dt.y;
                    s_u[cell<TT>(sc0 + i, srow)] = u.x;
                    s_u[cell<TT>(sc0 + i + 1, srow)] = u.y;
                }
            }
#pragma unroll
            for (int e = 0; e < BPT; ++e) {
                if (e * kThreads + tid >= TT * NP) continue;
                if constexpr (kAhead) {
                    put(s_bc, e * kThreads + tid, 0, nB[e]);
                    if (!SUMMARY) put(s_bc, e * kThreads + tid, 1, nC[e]);
                } else {
                    put(s_bc, e * kThreads + tid, 0, bc(Bp, a.bs, tile, e));
                    if (!SUMMARY) put(s_bc, e * kThreads + tid, 1, bc(Cp, a.cs, tile, e));
                }
            }
        };
        auto emit = [&](long long tile, const float* buf, const Pack<T, 8>& cx, const Pack<T, 8>& cz) {
            if constexpr (!SUMMARY) {
                const float* s_y = buf + 2 * CH * TT;
                if (!r.ok || tile >= r.e) r = find_seq(a.cu, a.num_seqs, a.M, a.T, tile);
                if (!stager || tile + srow >= t1) return;
                if (r.ok && tile + srow < r.e ? false : !find_seq(a.cu, a.num_seqs, a.M, a.T, tile + srow).ok) return;
                float x[8], z[8], y[8];
                unpack<T, 8>(cx, x);
                unpack<T, 8>(cz, z);
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    F2 o = fma2(F2{dsk[i], dsk[i + 1]}, F2{x[i], x[i + 1]},
                                F2{s_y[cell<TT>(sc0 + i, srow)], s_y[cell<TT>(sc0 + i + 1, srow)]});
                    if (a.z) {
                        const F2 zz{z[i], z[i + 1]};
                        o = mul2(o, mul2(zz, sigmoid2(zz)));
                    }
                    y[i] = o.x;
                    y[i + 1] = o.y;
                }
                store8<T, ALIGNED>(static_cast<T*>(a.out) + (tile + srow) * a.D + sd, y, scn);
            }
        };
        Pack<T, 8> cx = zero_pack<T, 8>(), cz = zero_pack<T, 8>();
        int b = 0;
        fetch(t0);
        for (long long tile = t0; tile < t1; tile += TT, b ^= 1) {
            lay(tile, sm + b * kBuf);   // the buffer's last scan ended before the last turn's emit
            bar_arrive<kFull>(b);
            const Pack<T, 8> px = cx, pz = cz;
            cx = nx;
            cz = nz;
            if (tile + TT < t1) fetch(tile + TT);
            if (tile > t0) {
                bar_sync<kDone>(b ^ 1);
                emit(tile - TT, sm + (b ^ 1) * kBuf, px, pz);
            }
        }
        if (t1 > t0) {
            bar_sync<kDone>(b ^ 1);
            emit(t0 + (t1 - t0 - 1) / TT * TT, sm + (b ^ 1) * kBuf, cx, cz);
        }
        return;
    }

    // ---- scan
    float A2[NS], h[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        const int n = s * NS + i;
        A2[i] = live && n < a.N ? a.A[(long long)d * a.N + n] * kLog2e : 0.f;
        h[i] = 0.f;
        if (!SUMMARY && !seg.whole && live && n < a.N)
            h[i] = hseg[(sg * a.D + d) * a.N + n];   // used unless a sequence starts at t0
    }
    float dtsum = 0.f;
    auto enter = [&](long long t) {   // row t is the first one, or the first behind r
        r = find_seq(a.cu, a.num_seqs, a.M, a.T, t);
        if (r.ok && r.b == t) {
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                const int n = s * NS + i;
                h[i] = a.h0 && live && n < a.N ? a.h0[((long long)r.q * a.D + d) * a.N + n] : 0.f;
            }
        }
    };
    auto finish = [&]() {   // the state is that of r's last row
        if constexpr (!SUMMARY) {
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                const int n = s * NS + i;
                if (a.hT != nullptr && live && n < a.N) a.hT[((long long)r.q * a.D + d) * a.N + n] = h[i];
            }
        }
    };
    int b = 0;
    for (long long tile = t0; tile < t1; tile += TT, b ^= 1) {
        float* buf = sm + b * kBuf;
        const float *s_dt = buf, *s_u = s_dt + CH * TT;
        const T* s_bc = reinterpret_cast<const T*>(s_u + (SUMMARY ? 1 : 2) * CH * TT) + s * NS * NBC;
        float* s_y = buf + 2 * CH * TT;
        using Q = Quads<T, !SUMMARY>;
        auto quads = [&](int i, Q* q) {   // this lane's B and C of row i
#pragma unroll
            for (int j = 0; j < NS / 4; ++j) q[j].load(s_bc + (i * NP + j * 4) * NBC);
        };
        auto row_step = [&](float dt, float u, const Q* q) {   // one row; the lane's share of y
            F2 acc{0.f, 0.f};
#pragma unroll
            for (int j = 0; j < NS; j += 4) {
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const F2 e = ex2(mul2(both(dt), F2{A2[j + 2 * m], A2[j + 2 * m + 1]}));
                    const F2 hn = fma2(e, F2{h[j + 2 * m], h[j + 2 * m + 1]}, mul2(both(u), q[j / 4].get(0, m)));
                    h[j + 2 * m] = hn.x;
                    h[j + 2 * m + 1] = hn.y;
                    if constexpr (!SUMMARY) acc = fma2(hn, q[j / 4].get(1, m), acc);
                }
            }
            if (SUMMARY) dtsum += dt;
            return acc.x + acc.y;
        };
        bar_sync<kFull>(b);
        const int rows = (int)(t1 - tile < TT ? t1 - tile : TT);
        if (!r.ok || tile >= r.e) enter(tile);
        if (rows == TT && r.ok && tile + TT <= r.e) {   // the tile lies in one sequence
            // four rows at a time, the next four's operands on their way from shared memory
            float4 nd = *reinterpret_cast<const float4*>(&s_dt[cell<TT>(ch, 0)]);
            float4 nu = *reinterpret_cast<const float4*>(&s_u[cell<TT>(ch, 0)]);
            Q nq[4][NS / 4];
#pragma unroll
            for (int k = 0; k < 4; ++k) quads(k, nq[k]);
#pragma unroll   // the whole tile: the scheduler mixes neighbouring rows (161 us for two turns together, 140 for all)
            for (int i = 0; i < TT; i += 4) {
                const float dts[4] = {nd.x, nd.y, nd.z, nd.w}, us[4] = {nu.x, nu.y, nu.z, nu.w};
                Q q[4][NS / 4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int j = 0; j < NS / 4; ++j) q[k][j] = nq[k][j];
                const int n = i + 4 < TT ? i + 4 : 0;   // behind the last four: the first again, unused
                nd = *reinterpret_cast<const float4*>(&s_dt[cell<TT>(ch, n)]);
                nu = *reinterpret_cast<const float4*>(&s_u[cell<TT>(ch, n)]);
#pragma unroll
                for (int k = 0; k < 4; ++k) quads(n + k, nq[k]);
                float y[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) y[k] = row_step(dts[k], us[k], q[k]);
                if constexpr (!SUMMARY) lane_sum4<S>(y[0], y[1], y[2], y[3], s, &s_y[cell<TT>(ch, i)]);
            }
            if (tile + TT == r.e) finish();
        } else {
            for (int i = 0; i < rows; ++i) {
                if (!r.ok || tile + i >= r.e) enter(tile + i);
                if (!r.ok) continue;   // a row of no sequence
                Q q[NS / 4];
                quads(i, q);
                float y = row_step(s_dt[cell<TT>(ch, i)], s_u[cell<TT>(ch, i)], q);
                if (!SUMMARY) {
#pragma unroll
                    for (int m = 1; m < S; m <<= 1) y += __shfl_xor_sync(0xffffffffu, y, m);
                    if (s == 0) s_y[cell<TT>(ch, i)] = y;
                }
                if (tile + i + 1 == r.e) finish();
            }
        }
        bar_arrive<kDone>(b);
    }
    if (SUMMARY && live) {
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            const int n = s * NS + i;
            if (n < a.N) hseg[(sg * a.D + d) * a.N + n] = h[i];
        }
        if (s == 0) dtseg[sg * a.D + d] = dtsum;
    }
}
template <typename T, int S, int NS, bool SUMMARY>
constexpr int scan_smem() {
    constexpr int CH = kThreads / S, TT = tile_rows<S>(), NP = S * NS;
    return 2 * ((int)sizeof(float) * (SUMMARY ? 2 : 3) * CH * TT + (int)sizeof(T) * (SUMMARY ? 1 : 2) * TT * NP);
}

// hseg[k] (the state that segment k alone ends with) -> the state that enters segment k.
__global__ void __launch_bounds__(128) ssm_join_kernel(SsmArgs a, Segments seg, float* hseg, const float* dtseg) {
    extern __shared__ uint8_t s_new[];
    for (long long k = threadIdx.x; k < seg.count; k += blockDim.x) {
        const long long t0 = k * seg.len, t1 = t0 + seg.len < a.M ? t0 + seg.len : a.M;
        s_new[k] = starts_inside(a, t0, t1);
    }
    __syncthreads();
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x, DN = (long long)a.D * a.N;
    if (i >= DN) return;
    const float A2 = a.A[i] * kLog2e;
    const long long d = i / a.N;
    float h = 0.f;
    constexpr int U = 8;   // segments whose values are loaded ahead of the chain
    for (long long k0 = 0; k0 < seg.count; k0 += U) {
        float own[U], dec[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool in = k0 + u < seg.count;
            own[u] = in ? hseg[(k0 + u) * DN + i] : 0.f;
            dec[u] = in ? dtseg[(k0 + u) * a.D + d] : 0.f;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (k0 + u >= seg.count) break;
            hseg[(k0 + u) * DN + i] = h;
            h = s_new[k0 + u] ? own[u] : fmaf(ex2(dec[u] * A2), h, own[u]);
        }
    }
}

// How the forward is laid out: lanes per channel, states per lane, segments.
struct Plan {
    int S, NS;
    Segments seg;
};
int lanes_for(int N, int NS) {
    int S = 1;
    while (S * NS < N) S *= 2;
    return S;
}
int states_for(int N, bool wide) { return wide || N > 32 ? 8 : 4; }
// Eight states per lane take a fifth fewer instructions per state than four (fewer sums over
// lanes, row operands read once for more states), but half as many CTAs: they are used where
// those still fill the SMs (two CTAs each), or where the rows are cut, which gives as many CTAs
// as are wanted.  One segment per sequence of a dense batch (all rows of a packed one) as soon as
// four states per lane give three CTAs on five SMs: cutting costs a second set of exponentials
// (2048 rows, 4096 channels, 16 states: 87 us whole, 123 us cut).
// 4 x 2048 rows, 2048 channels, 16 states: 161 us whole with four states per lane, 205 us with
// eight (128 CTAs); 32768 packed rows, 1024 channels: 442 us cut with eight, 489 us with four
// (before the tile was unrolled whole: now 140 us and 420 us).
Plan plan(long long B, long long T, int D, int N, int G, bool varlen) {
    const long long M = B * T, whole = varlen ? 1 : B;
    auto make = [&](bool wide) {
        Plan p;
        p.NS = states_for(N, wide);
        p.S = lanes_for(N, p.NS);
        p.seg = Segments{varlen ? M : T, whole, true};
        return p;
    };
    auto blocks = [&](const Plan& p) { return channel_blocks(D, G, kThreads / p.S); };
    Plan p = make(true);
    if (blocks(p) * whole >= 2 * kSMs) return p;
    const Plan narrow = make(false);
    if (blocks(narrow) * whole >= kSMs * 3 / 5) return narrow;
    long long count = 2LL * kSMs / blocks(p);   // what is resident at once, and no more
    const long long most = M / 128;             // about 128 rows each at least
    if (count > most) count = most;
    if (count > 1024) count = 1024;
    if (count <= 2 * whole) return narrow;      // twice the CTAs would only pay for twice the work
    const int tile = p.S >= 4 ? 32 : 8 * p.S;
    p.seg.len = ((M + count - 1) / count + tile - 1) / tile * tile;
    p.seg.count = (M + p.seg.len - 1) / p.seg.len;
    p.seg.whole = false;
    return p;
}

template <typename T, int S, int NS, bool ALIGNED>
cudaError_t fwd_go(const SsmArgs& a, const Segments& p, cudaStream_t s) {
    const long long blocks = channel_blocks(a.D, a.G, kThreads / S);
    // sequences without rows (packed, or T = 0) are served behind the segments
    const long long extra = a.cu != nullptr || a.T == 0 ? (a.num_seqs < 64 ? a.num_seqs : 64) : 0;
    if (blocks * (p.count + extra) > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    if (p.count + extra == 0) return cudaSuccess;
    const int nblk = (int)blocks;
    float* hseg = reinterpret_cast<float*>(a.ws);
    float* dtseg = hseg + p.count * a.D * a.N;
    cudaError_t e;
    if (!p.whole) {
        auto k = ssm_scan_kernel<T, S, NS, ALIGNED, true>;
        constexpr int sm1 = scan_smem<T, S, NS, true>();
        if ((e = allow_smem(k, sm1)) != cudaSuccess) return e;
        k<<<(unsigned)(blocks * p.count), 2 * kThreads, sm1, s>>>(a, p, nblk, hseg, dtseg);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        const long long dn = (long long)a.D * a.N;
        ssm_join_kernel<<<(unsigned)((dn + 127) / 128), 128, (size_t)p.count, s>>>(a, p, hseg, dtseg);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    auto k = ssm_scan_kernel<T, S, NS, ALIGNED, false>;
    constexpr int sm2 = scan_smem<T, S, NS, false>();
    if ((e = allow_smem(k, sm2)) != cudaSuccess) return e;
    k<<<(unsigned)(blocks * (p.count + extra)), 2 * kThreads, sm2, s>>>(a, p, nblk, hseg, dtseg);
    return cudaGetLastError();
}

template <typename T, bool ALIGNED>
cudaError_t fwd_n(const SsmArgs& a, const Plan& p, cudaStream_t s) {
    if (p.NS == 4) {
        switch (p.S) {
            case 1: return fwd_go<T, 1, 4, ALIGNED>(a, p.seg, s);
            case 2: return fwd_go<T, 2, 4, ALIGNED>(a, p.seg, s);
            case 4: return fwd_go<T, 4, 4, ALIGNED>(a, p.seg, s);
            default: return fwd_go<T, 8, 4, ALIGNED>(a, p.seg, s);
        }
    }
    switch (p.S) {
        case 1: return fwd_go<T, 1, 8, ALIGNED>(a, p.seg, s);
        case 2: return fwd_go<T, 2, 8, ALIGNED>(a, p.seg, s);
        case 4: return fwd_go<T, 4, 8, ALIGNED>(a, p.seg, s);
        case 8: return fwd_go<T, 8, 8, ALIGNED>(a, p.seg, s);
        default: return fwd_go<T, 16, 8, ALIGNED>(a, p.seg, s);
    }
}

template <typename T>
cudaError_t fwd_t(const SsmArgs& a, cudaStream_t s) {
    const int el = sizeof(T);
    const Plan p = plan(a.T > 0 ? a.M / a.T : 0, a.T, a.D, a.N, a.G, a.cu != nullptr);
    const bool al = (a.D / a.G) % 8 == 0 && vec_ok(a.x, a.xs * el, 16) && vec_ok(a.delta, a.ds * el, 16) &&
                    vec_ok(a.z, a.zs * el, 16) && vec_ok(a.out, (long long)a.D * el, 16);
    return al ? fwd_n<T, true>(a, p, s) : fwd_n<T, false>(a, p, s);
}

}  // namespace
}  // namespace ssm

}  // namespace kda
