// kda_conv.cu -- short causal depthwise convolution with optional SiLU: forward over
// rows, one-row step on a state of the last W - 1 inputs, gradients.
//
//   pre[t, d] = bias[d] + sum_j w[d, j] x[t - (W-1) + j, d],   out = pre sigmoid(pre)
//   dpre = d_out sigmoid(pre) (1 + pre (1 - sigmoid(pre)))
//   dx[s, d] = sum_j w[d, j] dpre[s + (W-1) - j, d],  dw[d, j] = sum_t dpre[t] x[t-(W-1)+j]
//
// Few operations per byte: HBM bounds every kernel here, with SiLU's exponential and reciprocal
// next (two per element at 16 per cycle and SM).  Every thread owns four channels and walks a
// run of rows with the window of earlier inputs in registers, so that each input is read once,
// plus W - 1 rows in front of each run.  The rows ahead are copied asynchronously into slots of
// shared memory that only this thread reads: enough bytes are under way without holding
// registers.  bf16: forward of 65536 x 4096, 4 taps, 209 us, 5.1 TB/s (its bound of three CTAs per SM
// spills 36 bytes, fp32 88); gradient of 8192 x 6144 74 us, 4.1 TB/s (16 warps per SM, which its 126
// registers leave, issue in half of their slots); a step of 256 x 4096 4 us in a captured graph.
//
// The tap count W is a template parameter: the window holds the W - 1 rows in front of the
// newest and no others (an unused tap of zero would make NaN of an infinity outside the window).
// Taps are aligned at the newest input: tap W - 1 is row t.
#include "kda_block.cuh"

namespace kda {
namespace {

template <int W, int VEC>
__device__ __forceinline__ void load_taps(const float* w, const float* bias, long long d0, float (*wr)[VEC], float* br) {
    if (W == 4 && (reinterpret_cast<uintptr_t>(w) & 15) == 0) {   // one 16-byte load per channel
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const float4 f = __ldg(reinterpret_cast<const float4*>(w) + d0 + v);
            const float t[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
            for (int j = 0; j < W; ++j) wr[j][v] = t[j & 3];
        }
    } else {
#pragma unroll
        for (int v = 0; v < VEC; ++v)
#pragma unroll
            for (int j = 0; j < W; ++j) wr[j][v] = __ldg(w + (d0 + v) * W + j);
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) br[v] = bias ? __ldg(bias + d0 + v) : 0.f;
}

// Inputs t - (W-1) .. t - 1 of the sequence r (from its state in front of row r.b).
template <typename T, int VEC, int W>
__device__ __forceinline__ void load_window(const ConvArgs& a, const SeqRange& r, long long t, long long d0,
                                            float (*win)[VEC]) {
    const T* x = static_cast<const T*>(a.x) + d0;
    const T* st = static_cast<const T*>(a.state0);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const long long p = t - (W - 1) + j;
        Pack<T, VEC> row = zero_pack<T, VEC>();
        if (p >= r.b) {
            row = load_pack<VEC>(x + p * a.xs);
        } else if (st != nullptr) {
            row = load_pack<VEC>(st + ((long long)r.q * (W - 1) + (W - 1) + (p - r.b)) * a.D + d0);
        }
        unpack<T, VEC>(row, win[j]);
    }
}

// The W rows in front of and at row t, in fp32 (unpacked once when a row enters).
template <int VEC, int W>
__device__ __forceinline__ void conv_pre(const float (*win)[VEC], const float* cur, const float (*wr)[VEC], const float* br,
                                         float* pre) {
#pragma unroll
    for (int v = 0; v < VEC; ++v) pre[v] = br[v];
#pragma unroll
    for (int j = 0; j < W; ++j) fma_n<VEC>(wr[j], j < W - 1 ? win[j < W - 1 ? j : 0] : cur, pre);
}
template <int VEC, int W>
__device__ __forceinline__ void shift_in(float (*win)[VEC], const float* cur) {
#pragma unroll
    for (int j = 0; j + 1 < W - 1; ++j)
#pragma unroll
        for (int v = 0; v < VEC; ++v) win[j][v] = win[j + 1][v];
#pragma unroll
    for (int v = 0; v < VEC; ++v) win[W - 2][v] = cur[v];
}

constexpr int kU = 4;       // rows worked on together
constexpr int kAhead = 4;   // groups of kU rows in the ring, one of them being worked on
template <typename T, int VEC>
constexpr int fwd_ring() { return VEC > 1 ? kAhead * kU * 256 * VEC * (int)sizeof(T) : 0; }

template <typename T, int VEC, int W, bool SILU>
__global__ void __launch_bounds__(256, W <= 4 ? 3 : 1) conv_fwd_kernel(ConvArgs a, long long run, long long nruns) {
    constexpr bool kFast = sizeof(T) == 2;
    extern __shared__ __align__(16) uint8_t ring_mem[];   // [kAhead][kU][thread]
    T* ring = reinterpret_cast<T*>(ring_mem);
    const int nvec = a.D / VEC;
    const long long idx = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    const long long d0 = (idx % nvec) * VEC;
    const long long who = idx / nvec;
    const T* x = static_cast<const T*>(a.x) + d0;
    if (who >= nruns) {   // behind the runs: the final state of one sequence
        const long long q = who - nruns;
        long long b, e;
        if (q >= a.num_seqs || !check_seq(a.cu, (int)q, a.M, a.T, a.dev_status, b, e) || a.stateT == nullptr) return;
        const T* st = static_cast<const T*>(a.state0);
        T* fin = static_cast<T*>(a.stateT);
        for (int j = 0; j < W - 1; ++j) {
            const long long p = e - (W - 1) + j;
            Pack<T, VEC> v = zero_pack<T, VEC>();
            if (p >= b) v = load_pack<VEC>(x + p * a.xs);
            else if (st != nullptr) v = load_pack<VEC>(st + (q * (W - 1) + (W - 1) + (p - b)) * a.D + d0);
            store_pack<T, VEC>(fin + (q * (W - 1) + j) * a.D + d0, v);
        }
        return;
    }
    float wr[W][VEC], br[VEC];
    load_taps<W, VEC>(a.w, a.bias, d0, wr, br);
    T* out = static_cast<T*>(a.out) + d0;
    float win[W - 1][VEC];

    long long t = who * run;
    const long long t1 = t + run < a.M ? t + run : a.M;
    auto emit = [&](long long row, const Pack<T, VEC>& raw) {
        float cur[VEC], pre[VEC];
        unpack<T, VEC>(raw, cur);
        conv_pre<VEC, W>(win, cur, wr, br, pre);
        if (SILU) silu_n<VEC, kFast>(pre);
        store_f32<T, VEC>(out + row * a.D, pre);
        shift_in<VEC, W>(win, cur);
    };
    while (t < t1) {
        const SeqRange r = find_seq(a.cu, a.num_seqs, a.M, a.T, t);
        if (!r.ok) { ++t; continue; }
        const long long stop = t1 < r.e ? t1 : r.e;
        load_window<T, VEC, W>(a, r, t, d0, win);
        const int quads = (int)((stop - t) / kU);
        const T* px = x + t * a.xs;
        if constexpr (VEC > 1) {   // kAhead - 1 groups of four rows under way
            int at = 0;
            auto ahead = [&](int q, int slot) {
                if (q < quads) {
#pragma unroll
                    for (int u = 0; u < kU; ++u)
                        copy_async<VEC * sizeof(T)>(&ring[((slot * kU + u) * 256 + threadIdx.x) * VEC], px + ((long long)q * kU + u) * a.xs);
                }
                copy_commit();
            };
#pragma unroll
            for (int k = 0; k < kAhead - 1; ++k) ahead(k, k);
#pragma unroll 1
            for (int q = 0; q < quads; ++q, t += kU) {
                copy_wait<kAhead - 2>();
                Pack<T, VEC> cur[kU];
#pragma unroll
                for (int u = 0; u < kU; ++u) cur[u] = lds_pack<T, VEC>(&ring[((at * kU + u) * 256 + threadIdx.x) * VEC]);
                ahead(q + kAhead - 1, at == 0 ? kAhead - 1 : at - 1);   // into the slot that the last turn read
                at = at == kAhead - 1 ? 0 : at + 1;
#pragma unroll
                for (int u = 0; u < kU; ++u) emit(t + u, cur[u]);
            }
            copy_wait<0>();
        } else {
            for (int q = 0; q < quads; ++q, t += kU) {
                Pack<T, VEC> cur[kU];
#pragma unroll
                for (int u = 0; u < kU; ++u) cur[u] = load_pack<VEC>(x + (t + u) * a.xs);
#pragma unroll
                for (int u = 0; u < kU; ++u) emit(t + u, cur[u]);
            }
        }
        for (; t < stop; ++t) emit(t, load_pack<VEC>(x + t * a.xs));
    }
}

// One row: a thread takes its channels of kSeqs sequences, whose loads are under way together and
// share one read of the taps (64 bytes per thread, as much as a sequence's state and input).  The
// state is stored in place, and out may be x: plain loads of both.
constexpr int kSeqs = 4;

template <typename T, int VEC, int W, bool SILU>
__global__ void __launch_bounds__(256) conv_step_kernel(ConvArgs a) {
    const int nvec = a.D / VEC;
    const long long idx = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    const long long n0 = idx / nvec * kSeqs, d0 = (idx % nvec) * VEC;
    if (n0 >= a.num_seqs) return;
    const long long ss = (long long)(W - 1) * a.D;   // a sequence's state
    T* st = static_cast<T*>(a.stateT) + n0 * ss + d0;
    const T* x = static_cast<const T*>(a.x) + n0 * a.xs + d0;
    T* out = static_cast<T*>(a.out) + n0 * a.D + d0;
    Pack<T, VEC> win[kSeqs][W];
#pragma unroll
    for (int q = 0; q < kSeqs; ++q) {
        const bool on = n0 + q < a.num_seqs;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            win[q][j] = on ? load_pack<VEC, false>(st + q * ss + (long long)j * a.D) : zero_pack<T, VEC>();
        }
        win[q][W - 1] = on ? load_pack<VEC, false>(x + q * a.xs) : zero_pack<T, VEC>();
    }
    float wr[W][VEC], br[VEC];
    load_taps<W, VEC>(a.w, a.bias, d0, wr, br);
#pragma unroll
    for (int q = 0; q < kSeqs; ++q) {
        if (n0 + q >= a.num_seqs) break;
        float pre[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) pre[v] = br[v];
#pragma unroll
        for (int j = 0; j < W; ++j) {
            float f[VEC];
            unpack<T, VEC>(win[q][j], f);
            fma_n<VEC>(wr[j], f, pre);
        }
        if (SILU) silu_n<VEC, sizeof(T) == 2>(pre);
        store_f32<T, VEC>(out + q * a.D, pre);
#pragma unroll
        for (int j = 1; j < W; ++j) store_pack<T, VEC>(st + q * ss + (long long)(j - 1) * a.D, win[q][j]);   // the state moves up by one row
    }
}

// Backward.  A CTA owns 32 * VEC channels; its eight warps walk runs of rows and keep
// their share of dw and db in registers, which are added over the warps at the end and
// written as one partial sum per CTA.  A run needs dpre of up to W - 1 rows behind it:
// those are computed again (they belong to the next run's dw).
constexpr int kBwdWarps = 8;
constexpr int kBwdAhead = 3;

template <typename T, typename TG, int VEC, int W, bool SILU>
__global__ void __launch_bounds__(32 * kBwdWarps) conv_bwd_kernel(ConvArgs a, long long run, long long nruns, int K) {
    constexpr bool kFast = sizeof(T) == 2;
    constexpr int NT = 32 * kBwdWarps;
    extern __shared__ __align__(16) float red[];   // the ring of rows; at the end [kBwdWarps][W + 1][VEC][32]
    T* ring_x = reinterpret_cast<T*>(red);
    TG* ring_g = reinterpret_cast<TG*>(ring_x + kBwdAhead * kU * NT * VEC);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long d0 = ((long long)blockIdx.x * 32 + lane) * VEC;
    const bool live = d0 < a.D;
    const T* x = static_cast<const T*>(a.x) + d0;
    const TG* dy = static_cast<const TG*>(a.d_out) + d0;
    T* dx = static_cast<T*>(a.dx) + d0;
    float dw[W][VEC] = {}, db[VEC] = {};
    if (live) {
        float wr[W][VEC], br[VEC];
        load_taps<W, VEC>(a.w, a.bias, d0, wr, br);
        const T* dfin = static_cast<const T*>(a.d_stateT);
        T* dst = static_cast<T*>(a.dstate0);
        for (long long rr = (long long)blockIdx.y * kBwdWarps + warp; rr < nruns; rr += (long long)K * kBwdWarps) {
            long long p0 = rr * run;
            const long long rend = p0 + run < a.M ? p0 + run : a.M;
            while (p0 < rend) {
                const SeqRange r = find_seq(a.cu, a.num_seqs, a.M, a.T, p0);
                if (!r.ok) { ++p0; continue; }
                const long long p1 = rend < r.e ? rend : r.e;
                float win[W - 1][VEC];
                load_window<T, VEC, W>(a, r, p0, d0, win);
                float dp[W][VEC] = {};   // dp[j] = dpre[t - j]
                // row t enters; row s = t - (W-1) has all of its gradients and leaves.  `edge`: s may lie
                // in front of the piece (the state's gradient, or another run's row) or be one of the
                // last W - 1 rows, which the final state holds.
                auto leave = [&](long long t, bool edge) {
                    const long long s = t - (W - 1);
                    T* to = dx + s * a.D;
                    float g[VEC] = {};
                    if (edge) {
                        if (s < p0) {
                            if (p0 != r.b || dst == nullptr) return;
                            to = dst + ((long long)r.q * (W - 1) + (W - 1) + (s - r.b)) * a.D + d0;
                        }
                        const long long k = s - r.e + (W - 1);   // the row is the final state's k-th
                        if (dfin != nullptr && k >= 0)
                            unpack<T, VEC>(load_pack<VEC>(dfin + ((long long)r.q * (W - 1) + k) * a.D + d0), g);
                    }
#pragma unroll
                    for (int j = 0; j < W; ++j) fma_n<VEC>(wr[j], dp[j], g);
                    store_f32<T, VEC>(to, g);
                };
                auto enter = [&](const Pack<T, VEC>& cur, const Pack<TG, VEC>& gcur, bool mine) {
                    float cf[VEC], g[VEC];
                    unpack<T, VEC>(cur, cf);
                    unpack<TG, VEC>(gcur, g);
                    if (SILU) {
                        float pre[VEC], sg[VEC];
                        conv_pre<VEC, W>(win, cf, wr, br, pre);
                        sigmoid_n<VEC, kFast>(pre, sg);
                        if constexpr (VEC > 1) {
#pragma unroll
                            for (int v = 0; v < VEC; v += 2) {
                                const F2 q{sg[v], sg[v + 1]}, p{pre[v], pre[v + 1]};
                                const F2 o = mul2(mul2(F2{g[v], g[v + 1]}, q), fma2(p, fma2(q, both(-1.0f), both(1.0f)), both(1.0f)));
                                g[v] = o.x;
                                g[v + 1] = o.y;
                            }
                        } else {
                            g[0] *= sg[0] * fmaf(pre[0], 1.0f - sg[0], 1.0f);
                        }
                    }
#pragma unroll
                    for (int j = W - 1; j > 0; --j)
#pragma unroll
                        for (int v = 0; v < VEC; ++v) dp[j][v] = dp[j - 1][v];
#pragma unroll
                    for (int v = 0; v < VEC; ++v) dp[0][v] = g[v];
                    if (mine) {
#pragma unroll
                        for (int v = 0; v < VEC; ++v) db[v] += g[v];
#pragma unroll
                        for (int j = 0; j < W; ++j) fma_n<VEC>(g, j < W - 1 ? win[j < W - 1 ? j : 0] : cf, dw[j]);
                    }
                    shift_in<VEC, W>(win, cf);
                };
                long long t = p0;
                const int quads = (int)((p1 - p0) / kU);
                Pack<T, VEC> cx[kU];
                Pack<TG, VEC> cg[kU];
                auto ahead = [&](int q, int slot) {   // four rows of x and d_out into the ring
                    if constexpr (VEC > 1) {
                        if (q < quads) {
#pragma unroll
                            for (int u = 0; u < kU; ++u) {
                                const long long at = p0 + (long long)q * kU + u;
                                copy_async<VEC * sizeof(T)>(&ring_x[((slot * kU + u) * NT + threadIdx.x) * VEC], x + at * a.xs);
                                copy_async<VEC * sizeof(TG)>(&ring_g[((slot * kU + u) * NT + threadIdx.x) * VEC], dy + at * a.D);
                            }
                        }
                        copy_commit();
                    }
                };
#pragma unroll
                for (int k = 0; k < kBwdAhead - 1; ++k) ahead(k, k);
                int slot = 0;
#pragma unroll 1
                for (int q = 0; q < quads; ++q, t += kU) {
                    if constexpr (VEC > 1) copy_wait<kBwdAhead - 2>();
#pragma unroll
                    for (int u = 0; u < kU; ++u) {
                        if constexpr (VEC > 1) {
                            cx[u] = lds_pack<T, VEC>(&ring_x[((slot * kU + u) * NT + threadIdx.x) * VEC]);
                            cg[u] = lds_pack<TG, VEC>(&ring_g[((slot * kU + u) * NT + threadIdx.x) * VEC]);
                        } else {
                            cx[u] = load_pack<VEC>(x + (t + u) * a.xs);
                            cg[u] = load_pack<VEC>(dy + (t + u) * a.D);
                        }
                    }
                    ahead(q + kBwdAhead - 1, slot == 0 ? kBwdAhead - 1 : slot - 1);
                    slot = slot == kBwdAhead - 1 ? 0 : slot + 1;
                    if (q * kU >= W - 1) {   // inside: s is a row of the piece, W or more in front of the end
#pragma unroll
                        for (int u = 0; u < kU; ++u) {
                            enter(cx[u], cg[u], true);
                            leave(t + u, false);
                        }
                    } else {
#pragma unroll
                        for (int u = 0; u < kU; ++u) {
                            enter(cx[u], cg[u], true);
                            leave(t + u, true);
                        }
                    }
                }
                if constexpr (VEC > 1) copy_wait<0>();
                for (; t < p1; ++t) {
                    enter(load_pack<VEC>(x + t * a.xs), load_pack<VEC>(dy + t * a.D), true);
                    leave(t, true);
                }
                for (; t < p1 + W - 1; ++t) {   // behind the piece: another run's rows, or past the sequence's end
                    if (t < r.e) {
                        enter(load_pack<VEC>(x + t * a.xs), load_pack<VEC>(dy + t * a.D), false);
                    } else {
#pragma unroll
                        for (int j = W - 1; j > 0; --j)
#pragma unroll
                            for (int v = 0; v < VEC; ++v) dp[j][v] = dp[j - 1][v];
#pragma unroll
                        for (int v = 0; v < VEC; ++v) dp[0][v] = 0.f;
                    }
                    leave(t, true);
                }
                p0 = p1;
            }
        }
        // Sequences without rows hand their final state's gradient through; bounds are checked.
        for (long long q = (long long)blockIdx.y * kBwdWarps + warp; q < a.num_seqs; q += (long long)K * kBwdWarps) {
            long long b, e;
            if (!check_seq(a.cu, (int)q, a.M, a.T, a.dev_status, b, e) || b != e || dst == nullptr) continue;
            for (int j = 0; j < W - 1; ++j) {
                Pack<T, VEC> v = zero_pack<T, VEC>();
                if (dfin != nullptr) v = load_pack<VEC>(dfin + (q * (W - 1) + j) * a.D + d0);
                store_pack<T, VEC>(dst + (q * (W - 1) + j) * a.D + d0, v);
            }
        }
    }
    __syncthreads();   // every thread is done with its ring
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
#pragma unroll
        for (int j = 0; j < W; ++j) red[((warp * (W + 1) + j) * VEC + v) * 32 + lane] = dw[j][v];
        red[((warp * (W + 1) + W) * VEC + v) * 32 + lane] = db[v];
    }
    __syncthreads();
    // part[blockIdx.y]: [D][W] of dw, then [D] of db
    float* part = a.part + (long long)blockIdx.y * a.D * (W + 1);
    for (int i = threadIdx.x; i < (W + 1) * VEC * 32; i += blockDim.x) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kBwdWarps; ++w) s += red[w * (W + 1) * VEC * 32 + i];
        const int j = i / (VEC * 32), v = (i / 32) % VEC, l = i & 31;
        const long long d = ((long long)blockIdx.x * 32 + l) * VEC + v;
        if (d >= a.D) continue;
        if (j == W) part[(long long)a.D * W + d] = s;
        else part[d * W + j] = s;
    }
}

// Rows per thread of the forward: one run for each thread that is resident at once (three CTAs
// per SM), so that the ring is filled once and the W - 1 rows in front of a run are few; at
// least eight rows, however few that leaves to run.
long long fwd_run(long long M, long long nvec) {
    const long long run = (M * nvec + kSMs * 768LL - 1) / (kSMs * 768LL);
    return run < 8 ? 8 : run;
}

struct BwdPlan {
    int K;
    long long run, nruns;
};
// One run of consecutive rows per warp, as many CTAs as are resident at once (two per SM) but no more
// than one per 128 rows: the rows divide evenly and the W - 1 rows behind a run, computed twice, are
// few.  (Below 128 rows in all the one CTA's runs are shorter, down to a row.)
BwdPlan bwd_plan(long long M, int D, int vec) {
    BwdPlan p;
    const long long nblk = (D + 32LL * vec - 1) / (32LL * vec);
    long long K = 2 * kSMs / nblk;
    const long long most = (M + 16LL * kBwdWarps - 1) / (16LL * kBwdWarps);
    if (K > most) K = most;
    p.K = (int)(K < 1 ? 1 : K);
    p.run = (M + (long long)p.K * kBwdWarps - 1) / ((long long)p.K * kBwdWarps);
    if (p.run < 1) p.run = 1;
    p.nruns = (M + p.run - 1) / p.run;
    return p;
}

template <typename T, int VEC, bool SILU>
cudaError_t fwd_w(const ConvArgs& a, cudaStream_t s) {
    const long long nvec = a.D / VEC;
    const long long run = fwd_run(a.M, nvec);
    const long long nruns = (a.M + run - 1) / run;
    const long long grid = (nvec * (nruns + a.num_seqs) + 255) / 256;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    constexpr int smem = fwd_ring<T, VEC>();
    auto k = a.W == 2   ? conv_fwd_kernel<T, VEC, 2, SILU>
             : a.W == 3 ? conv_fwd_kernel<T, VEC, 3, SILU>
             : a.W == 4 ? conv_fwd_kernel<T, VEC, 4, SILU>
             : a.W == 5 ? conv_fwd_kernel<T, VEC, 5, SILU>
             : a.W == 6 ? conv_fwd_kernel<T, VEC, 6, SILU>
             : a.W == 7 ? conv_fwd_kernel<T, VEC, 7, SILU>
                        : conv_fwd_kernel<T, VEC, 8, SILU>;
    cudaError_t e;
    if ((e = allow_smem(k, smem)) != cudaSuccess) return e;
    k<<<(unsigned)grid, 256, smem, s>>>(a, run, nruns);
    return cudaGetLastError();
}
template <typename T, int VEC, bool SILU>
cudaError_t step_w(const ConvArgs& a, cudaStream_t s) {
    const long long grid = ((long long)(a.D / VEC) * ((a.num_seqs + kSeqs - 1) / kSeqs) + 255) / 256;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    switch (a.W) {
        case 2: conv_step_kernel<T, VEC, 2, SILU><<<(unsigned)grid, 256, 0, s>>>(a); break;
        case 3: conv_step_kernel<T, VEC, 3, SILU><<<(unsigned)grid, 256, 0, s>>>(a); break;
        case 4: conv_step_kernel<T, VEC, 4, SILU><<<(unsigned)grid, 256, 0, s>>>(a); break;
        case 5: conv_step_kernel<T, VEC, 5, SILU><<<(unsigned)grid, 256, 0, s>>>(a); break;
        case 6: conv_step_kernel<T, VEC, 6, SILU><<<(unsigned)grid, 256, 0, s>>>(a); break;
        case 7: conv_step_kernel<T, VEC, 7, SILU><<<(unsigned)grid, 256, 0, s>>>(a); break;
        default: conv_step_kernel<T, VEC, 8, SILU><<<(unsigned)grid, 256, 0, s>>>(a); break;
    }
    return cudaGetLastError();
}
template <typename T, typename TG, int VEC, int W, bool SILU>
cudaError_t bwd_one(const ConvArgs& a, cudaStream_t s) {
    const BwdPlan p = bwd_plan(a.M, a.D, VEC);
    const dim3 grid((unsigned)((a.D + 32LL * VEC - 1) / (32 * VEC)), (unsigned)p.K);
    constexpr int sums = (int)sizeof(float) * kBwdWarps * (W + 1) * VEC * 32;
    constexpr int ring = VEC > 1 ? kBwdAhead * kU * 32 * kBwdWarps * VEC * (int)(sizeof(T) + sizeof(TG)) : 0;
    constexpr int smem = sums > ring ? sums : ring;
    auto k = conv_bwd_kernel<T, TG, VEC, W, SILU>;
    cudaError_t e = allow_smem(k, smem);
    if (e != cudaSuccess) return e;
    k<<<grid, 32 * kBwdWarps, smem, s>>>(a, p.run, p.nruns, p.K);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_colsum(a.part, p.K, (long long)a.D * a.W, a.dw, a.D, a.db, 0, nullptr, s);
}
template <typename T, typename TG, int VEC, bool SILU>
cudaError_t bwd_w(const ConvArgs& a, cudaStream_t s) {
    switch (a.W) {
        case 2: return bwd_one<T, TG, VEC, 2, SILU>(a, s);
        case 3: return bwd_one<T, TG, VEC, 3, SILU>(a, s);
        case 4: return bwd_one<T, TG, VEC, 4, SILU>(a, s);
        case 5: return bwd_one<T, TG, VEC, 5, SILU>(a, s);
        case 6: return bwd_one<T, TG, VEC, 6, SILU>(a, s);
        case 7: return bwd_one<T, TG, VEC, 7, SILU>(a, s);
        default: return bwd_one<T, TG, VEC, 8, SILU>(a, s);
    }
}
template <typename T, typename TG, int VEC>
cudaError_t bwd_act(const ConvArgs& a, bool silu, cudaStream_t s) {
    return silu ? bwd_w<T, TG, VEC, true>(a, s) : bwd_w<T, TG, VEC, false>(a, s);
}

// Accesses of `vec` elements need every row of every tensor to start on such a boundary.
bool rows_ok(const ConvArgs& a, int el, int vec) {
    const int by = el * vec;
    const long long row = (long long)a.D * el;
    return a.D % vec == 0 && vec_ok(a.x, a.xs * el, by) && vec_ok(a.out, row, by) && vec_ok(a.state0, row, by) &&
           vec_ok(a.stateT, row, by) && vec_ok(a.dx, row, by) && vec_ok(a.dstate0, row, by) &&
           vec_ok(a.d_stateT, row, by);
}

// Four channels per thread in either type: with eight, the window, the taps and the rows need
// 128 registers, and too few warps remain to cover the loads.
template <typename T>
cudaError_t fwd_t(const ConvArgs& a, bool silu, cudaStream_t s) {
    constexpr int V = 4;
    if (rows_ok(a, sizeof(T), V)) return silu ? fwd_w<T, V, true>(a, s) : fwd_w<T, V, false>(a, s);
    return silu ? fwd_w<T, 1, true>(a, s) : fwd_w<T, 1, false>(a, s);
}
template <typename T>
cudaError_t step_t(const ConvArgs& a, bool silu, cudaStream_t s) {
    constexpr int V = 4;
    if (rows_ok(a, sizeof(T), V)) return silu ? step_w<T, V, true>(a, s) : step_w<T, V, false>(a, s);
    return silu ? step_w<T, 1, true>(a, s) : step_w<T, 1, false>(a, s);
}

}  // namespace

cudaError_t launch_conv_fwd(const ConvArgs& a, bool bf16, bool silu, cudaStream_t s) {
    return bf16 ? fwd_t<__nv_bfloat16>(a, silu, s) : fwd_t<float>(a, silu, s);
}

cudaError_t launch_conv_step(const ConvArgs& a, bool bf16, bool silu, cudaStream_t s) {
    return bf16 ? step_t<__nv_bfloat16>(a, silu, s) : step_t<float>(a, silu, s);
}

size_t conv_bwd_workspace_bytes(long long M, int D, int W) {
    const int k4 = bwd_plan(M, D, 4).K, k1 = bwd_plan(M, D, 1).K;
    return sizeof(float) * (size_t)(k4 > k1 ? k4 : k1) * D * (W + 1);
}

cudaError_t launch_conv_bwd(const ConvArgs& a, bool bf16, bool grad_bf16, bool silu, cudaStream_t s) {
    const int el = bf16 ? 2 : 4, gel = grad_bf16 ? 2 : 4;
    const bool vec = rows_ok(a, el, 4) && vec_ok(a.d_out, (long long)a.D * gel, 4 * gel);
    if (!bf16) return vec ? bwd_act<float, float, 4>(a, silu, s) : bwd_act<float, float, 1>(a, silu, s);
    if (grad_bf16)
        return vec ? bwd_act<__nv_bfloat16, __nv_bfloat16, 4>(a, silu, s)
                   : bwd_act<__nv_bfloat16, __nv_bfloat16, 1>(a, silu, s);
    return vec ? bwd_act<__nv_bfloat16, float, 4>(a, silu, s) : bwd_act<__nv_bfloat16, float, 1>(a, silu, s);
}

}  // namespace kda
