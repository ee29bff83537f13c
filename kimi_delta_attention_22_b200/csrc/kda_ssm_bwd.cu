// kda_ssm_bwd.cu -- gradients of the selective state space scan.
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
// The rows are cut into segments of L, aligned to the row index.
//   1. summary: every segment alone, scanned once from zero, gives its last state, the
//      gradient that its rows send to the state in front of it (sum_t (prod a) C dy, the
//      running product taken along, so no second exponential), and the sum of dt.
//   2. join: along the segments, forward for the incoming states, backward for the
//      incoming state gradients (the decay over a segment is e^{A sum dt}).
//   3. gradients, all segments in parallel: a forward scan keeps the state in front of
//      every SUB rows; then, from the last SUB rows back, their states and decays are
//      computed again into registers and walked in reverse.
//   4. sums: of dB and dC over the channel blocks, of dA, dDskip and the bias over segments.
// Three sets of exponentials and about 21 fp32 operations per row, channel and state: the
// fp32 and special-function units bound it, not the bytes.
//
// Lanes as in the forward: S lanes of a channel, NS states each, 128 / S channels of a CTA.
// dB and dC sum over a warp's channels by halving exchanges: of 2 NS values, every lane of
// a channel set ends with its own few sums.
#include "kda_ssm.cuh"

namespace kda {
namespace ssm {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

template <int S>
constexpr int seg_rows() { return S >= 4 ? 64 : 32; }

// First / last rows of sequences and rows of any sequence, one bit per row of the segment.
struct Events {
    uint32_t first[2], last[2], in[2];
};
__device__ __forceinline__ bool bit(const uint32_t* m, int i) { return m[i >> 5] >> (i & 31) & 1; }

template <int L>
__device__ __forceinline__ void find_events(const SsmArgs& a, long long t0, Events* ev) {
    const int i = threadIdx.x;
    if (i < L) {
        SeqRange r{0, 0, 0, false};
        if (t0 + i < a.M) r = find_seq(a.cu, a.num_seqs, a.M, a.T, t0 + i);
        const uint32_t f = __ballot_sync(0xffffffffu, r.ok && r.b == t0 + i);
        const uint32_t l = __ballot_sync(0xffffffffu, r.ok && r.e == t0 + i + 1);
        const uint32_t in = __ballot_sync(0xffffffffu, r.ok);
        if ((i & 31) == 0) {
            ev->first[i >> 5] = f;
            ev->last[i >> 5] = l;
            ev->in[i >> 5] = in;
        }
    }
}

// dt, x (or dt x) and dy of the segment into shared memory [channel][row]; zeros in rows
// that no sequence covers, which then neither decay nor add anything.
template <typename T, int CH, int L, int LD, bool ALIGNED, bool TIMES>
__device__ __forceinline__ void stage(const SsmArgs& a, const ChannelBlock& cb, long long t0, const Events& ev, float* s_dt,
                                      float* s_x, float* s_dy) {
    constexpr int VPR = CH / 8, RPP = kThreads / VPR;   // rows per pass
    const int c0 = (threadIdx.x % VPR) * 8;
    const int cn = max(0, min(8, cb.n - c0)), d = cb.d0 + c0;
    float bias[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) bias[i] = i < cn && a.delta_bias ? a.delta_bias[d + i] : 0.f;
#pragma unroll
    for (int row0 = 0; row0 < L; row0 += RPP) {
        const int row = row0 + threadIdx.x / VPR;
        if (row >= L) break;
        const long long t = t0 + row;
        const bool in = bit(ev.in, row);
        const int n = in ? cn : 0;
        float x[8], v[8], g[8];
        unpack<T, 8>(load8<T, ALIGNED>(static_cast<const T*>(a.x) + t * a.xs + d, n), x);
        unpack<T, 8>(load8<T, ALIGNED>(static_cast<const T*>(a.delta) + t * a.ds + d, n), v);
        unpack<T, 8>(load8<T, ALIGNED>(static_cast<const T*>(a.d_out) + t * a.D + d, n), g);
        if (a.z != nullptr) {
            float z[8];
            unpack<T, 8>(load8<T, ALIGNED>(static_cast<const T*>(a.z) + t * a.zs + d, n), z);
#pragma unroll
            for (int i = 0; i < 8; ++i) g[i] *= z[i] * sigmoid<sizeof(T) == 2>(z[i]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[i] += bias[i];
            if (a.softplus) v[i] = softplus(v[i]);
            if (i >= n) v[i] = 0.f;
            s_dt[(c0 + i) * LD + row] = v[i];
            s_x[(c0 + i) * LD + row] = TIMES ? v[i] * x[i] : x[i];
            s_dy[(c0 + i) * LD + row] = g[i];
        }
    }
}

template <typename T, int L, int NP>
__device__ __forceinline__ void stage_bc(const SsmArgs& a, int g, long long t0, const Events& ev, float* s_B, float* s_C) {
    const T* Bp = static_cast<const T*>(a.Bm) + (long long)g * a.N;
    const T* Cp = static_cast<const T*>(a.Cm) + (long long)g * a.N;
#pragma unroll 8
    for (int k = threadIdx.x; k < L * NP; k += kThreads) {
        const int row = k / NP, n = k % NP;
        const bool on = n < a.N && bit(ev.in, row);
        s_B[k] = on ? to_f32<T>(Bp[(t0 + row) * a.bs + n]) : 0.f;
        s_C[k] = on ? to_f32<T>(Cp[(t0 + row) * a.cs + n]) : 0.f;
    }
}

// What the join needs to know of a segment.
constexpr uint8_t kStarts = 1;      // holds a sequence's first row (its last state is its own)
constexpr uint8_t kEnds = 2;        // the sequence of its first row ends in it
constexpr uint8_t kFirst = 4;       // its first row is a sequence's first row

template <typename T, int S, int NS, bool ALIGNED>
__global__ void __launch_bounds__(kThreads) ssm_bwd_summary_kernel(SsmArgs a, long long K, int nblk, float* hseg,
                                                                  float* rseg, float* dtseg, uint8_t* flags) {
    constexpr int CH = kThreads / S, L = seg_rows<S>(), LD = L + 4, NP = S * NS;
    extern __shared__ __align__(16) float sm[];
    float *s_dt = sm, *s_u = s_dt + CH * LD, *s_dy = s_u + CH * LD, *s_B = s_dy + CH * LD, *s_C = s_B + L * NP;
    __shared__ Events ev;
    const long long sg = blockIdx.x / nblk;
    const ChannelBlock cb = channel_block<CH>(blockIdx.x % nblk, a.D, a.G);
    const int tid = threadIdx.x, ch = tid / S, s = tid % S;
    const bool live = ch < cb.n;
    const int d = cb.d0 + (live ? ch : 0);
    if (sg >= K) {   // sequences without rows hand their state's gradient through
        for (long long q = sg - K; q < a.num_seqs; q += gridDim.x / nblk - K) {
            long long b, e;
            if (!check_seq(a.cu, (int)q, a.M, a.T, a.dev_status, b, e) || b != e || a.dh0 == nullptr || !live) continue;
            const long long at = (q * a.D + d) * a.N;
            for (int n = s * NS; n < s * NS + NS && n < a.N; ++n) a.dh0[at + n] = a.d_hT ? a.d_hT[at + n] : 0.f;
        }
        return;
    }
    const long long t0 = sg * L;
    find_events<L>(a, t0, &ev);
    __syncthreads();
    stage<T, CH, L, LD, ALIGNED, true>(a, cb, t0, ev, s_dt, s_u, s_dy);
    stage_bc<T, L, NP>(a, cb.g, t0, ev, s_B, s_C);
    float A2[NS], h[NS], p[NS], g[NS];
#pragma unroll
    for (int j = 0; j < NS; ++j) {
        const int n = s * NS + j;
        A2[j] = live && n < a.N ? a.A[(long long)d * a.N + n] * kLog2e : 0.f;
        h[j] = g[j] = 0.f;
        p[j] = 1.f;
    }
    float dtsum = 0.f;
    auto state_of = [&](const float* from, long long t, int j) {   // a state of the sequence of row t
        const int n = s * NS + j;
        if (from == nullptr || !live || n >= a.N) return 0.f;
        const SeqRange r = find_seq(a.cu, a.num_seqs, a.M, a.T, t);
        return from[((long long)r.q * a.D + d) * a.N + n];
    };
    __syncthreads();
#pragma unroll 2
    for (int i = 0; i < L; i += 4) {
        const float4 d4 = *reinterpret_cast<const float4*>(&s_dt[ch * LD + i]);
        const float4 u4 = *reinterpret_cast<const float4*>(&s_u[ch * LD + i]);
        const float4 g4 = *reinterpret_cast<const float4*>(&s_dy[ch * LD + i]);
        const float dts[4] = {d4.x, d4.y, d4.z, d4.w}, us[4] = {u4.x, u4.y, u4.z, u4.w}, gs[4] = {g4.x, g4.y, g4.z, g4.w};
        const uint32_t mf = ev.first[i >> 5] >> (i & 31), ml = ev.last[i >> 5] >> (i & 31);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (mf >> k & 1) {
#pragma unroll
                for (int j = 0; j < NS; ++j) {
                    h[j] = state_of(a.h0, t0 + i + k, j);
                    if (i + k > 0) p[j] = 0.f;   // rows behind the first sequence's end
                }
            }
#pragma unroll
            for (int j = 0; j < NS; ++j) {
                const float e = ex2(dts[k] * A2[j]);
                h[j] = fmaf(e, h[j], us[k] * s_B[(i + k) * NP + s * NS + j]);
                p[j] *= e;
                g[j] = fmaf(p[j], gs[k] * s_C[(i + k) * NP + s * NS + j], g[j]);
            }
            dtsum += dts[k];
            if (ml >> k & 1) {
#pragma unroll
                for (int j = 0; j < NS; ++j) {
                    if (a.d_hT != nullptr) g[j] = fmaf(p[j], state_of(a.d_hT, t0 + i + k, j), g[j]);
                    p[j] = 0.f;
                }
            }
        }
    }
    if (live) {
#pragma unroll
        for (int j = 0; j < NS; ++j) {
            const int n = s * NS + j;
            if (n < a.N) {
                hseg[(sg * a.D + d) * a.N + n] = h[j];
                rseg[(sg * a.D + d) * a.N + n] = g[j];
            }
        }
        if (s == 0) dtseg[sg * a.D + d] = dtsum;
    }
    if (blockIdx.x % nblk == 0 && tid == 0) {
        uint8_t f = 0;
        if (ev.first[0] | (L > 32 ? ev.first[1] : 0u)) f |= kStarts;
        if (ev.last[0] | (L > 32 ? ev.last[1] : 0u) | !(ev.in[0] & 1)) f |= kEnds;
        if ((ev.first[0] & 1) || !(ev.in[0] & 1)) f |= kFirst;
        flags[sg] = f;
    }
}

// y = 0: hseg[k] (segment k's own last state) -> the state in front of it.
// y = 1: rseg[k] (what its rows send to the state in front) -> the gradient of its last state.
__global__ void __launch_bounds__(128) ssm_bwd_join_kernel(SsmArgs a, long long K, float* hseg, float* rseg,
                                                           const float* dtseg, const uint8_t* flags) {
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x, DN = (long long)a.D * a.N;
    if (i >= DN) return;
    const float A2 = a.A[i] * kLog2e;
    const long long d = i / a.N;
    float c = 0.f;
    if (blockIdx.y == 0) {
#pragma unroll 8
        for (long long k = 0; k < K; ++k) {
            const float own = hseg[k * DN + i], dt = dtseg[k * a.D + d];
            const uint8_t f = flags[k];
            hseg[k * DN + i] = c;
            c = f & kStarts ? own : fmaf(ex2(dt * A2), c, own);
        }
    } else {
#pragma unroll 8
        for (long long k = K - 1; k >= 0; --k) {
            const float own = rseg[k * DN + i], dt = dtseg[k * a.D + d];
            const uint8_t f = flags[k];
            rseg[k * DN + i] = c;
            c = f & kFirst ? 0.f : f & kEnds ? own : fmaf(ex2(dt * A2), c, own);
        }
    }
}

template <int S, int NS, int SUB>
constexpr size_t grad_smem() {
    constexpr int CH = kThreads / S, L = seg_rows<S>(), LD = L + 4, NP = S * NS;
    return sizeof(float) * (6 * CH * LD + 2 * L * NP + (L / SUB) * NS * kThreads + 2 * kWarps * SUB * 2 * NP);
}

template <typename T, int S, int NS, int SUB, bool ALIGNED>
__global__ void __launch_bounds__(kThreads) ssm_bwd_grad_kernel(SsmArgs a, long long K, int nblk, const float* hseg,
                                                                const float* rseg, float* part, float* bcpart) {
    constexpr int CH = kThreads / S, L = seg_rows<S>(), LD = L + 4, NP = S * NS;
    constexpr int VPR = CH / 8, RPP = kThreads / VPR;
    constexpr int V = 2 * NS, CL = 32 / S, RV = V / CL > 0 ? V / CL : 1;   // sums per lane of dB, dC
    extern __shared__ __align__(16) float sm[];
    float *s_dt = sm, *s_x = s_dt + CH * LD, *s_dy = s_x + CH * LD;
    float *s_p = s_dy + CH * LD, *s_q = s_p + CH * LD, *s_y = s_q + CH * LD;
    float *s_B = s_y + CH * LD, *s_C = s_B + L * NP, *s_ck = s_C + L * NP, *s_red = s_ck + (L / SUB) * NS * kThreads;
    __shared__ Events ev;
    const long long sg = blockIdx.x / nblk;
    const int blk = blockIdx.x % nblk;
    const ChannelBlock cb = channel_block<CH>(blk, a.D, a.G);
    const int tid = threadIdx.x, ch = tid / S, s = tid % S, lane = tid & 31, warp = tid >> 5;
    const bool live = ch < cb.n;
    const int d = cb.d0 + (live ? ch : 0);
    const long long t0 = sg * L;
    find_events<L>(a, t0, &ev);
    __syncthreads();
    stage<T, CH, L, LD, ALIGNED, false>(a, cb, t0, ev, s_dt, s_x, s_dy);
    stage_bc<T, L, NP>(a, cb.g, t0, ev, s_B, s_C);

    float A2[NS], h[NS], dh[NS], dA[NS];
#pragma unroll
    for (int j = 0; j < NS; ++j) {
        const int n = s * NS + j;
        const bool on = live && n < a.N;
        A2[j] = on ? a.A[(long long)d * a.N + n] * kLog2e : 0.f;
        h[j] = on ? hseg[(sg * a.D + d) * a.N + n] : 0.f;
        dh[j] = on ? rseg[(sg * a.D + d) * a.N + n] : 0.f;
        dA[j] = 0.f;
    }
    auto state_of = [&](const float* from, int i, int j) {
        const int n = s * NS + j;
        if (from == nullptr || !live || n >= a.N) return 0.f;
        const SeqRange r = find_seq(a.cu, a.num_seqs, a.M, a.T, t0 + i);
        return from[((long long)r.q * a.D + d) * a.N + n];
    };
    __syncthreads();

    // forward: the state in front of every SUB rows
#pragma unroll 1
    for (int sb = 0; sb < L / SUB; ++sb) {
#pragma unroll
        for (int j = 0; j < NS; ++j) s_ck[(sb * NS + j) * kThreads + tid] = h[j];
#pragma unroll
        for (int i = 0; i < SUB; ++i) {
            const int r = sb * SUB + i;
            if (bit(ev.first, r)) {
#pragma unroll
                for (int j = 0; j < NS; ++j) h[j] = state_of(a.h0, r, j);
            }
            const float dt = s_dt[ch * LD + r], u = dt * s_x[ch * LD + r];
#pragma unroll
            for (int j = 0; j < NS; ++j) h[j] = fmaf(ex2(dt * A2[j]), h[j], u * s_B[r * NP + s * NS + j]);
        }
    }

    // which of a row's 2 NS sums this lane ends with, and whether it is the one to write them
    int off = 0;
    bool writer = true;
    {
        int cnt = V;
#pragma unroll
        for (int m = 16; m >= S; m >>= 1) {
            if (cnt > 1) {
                cnt /= 2;
                if (lane & m) off += cnt;
            } else if (lane & m) {
                writer = false;
            }
        }
    }

    const int rows = (int)(a.M - t0 < L ? a.M - t0 : L);
#pragma unroll 1
    for (int sb = L / SUB - 1; sb >= 0; --sb) {
        float ha[SUB][NS], ea[SUB][NS], hs[NS];
#pragma unroll
        for (int j = 0; j < NS; ++j) hs[j] = h[j] = s_ck[(sb * NS + j) * kThreads + tid];
#pragma unroll
        for (int i = 0; i < SUB; ++i) {
            const int r = sb * SUB + i;
            if (bit(ev.first, r)) {
#pragma unroll
                for (int j = 0; j < NS; ++j) h[j] = state_of(a.h0, r, j);
            }
            const float dt = s_dt[ch * LD + r], u = dt * s_x[ch * LD + r];
#pragma unroll
            for (int j = 0; j < NS; ++j) {
                ea[i][j] = ex2(dt * A2[j]);
                h[j] = fmaf(ea[i][j], h[j], u * s_B[r * NP + s * NS + j]);
                ha[i][j] = h[j];
            }
        }
        float* red = s_red + ((sb & 1) * kWarps + warp) * SUB * 2 * NP;
        float pv[4], qv[4], yv[4];
#pragma unroll
        for (int i = SUB - 1; i >= 0; --i) {
            const int r = sb * SUB + i;
            if (bit(ev.last, r)) {
#pragma unroll
                for (int j = 0; j < NS; ++j) dh[j] = state_of(a.d_hT, r, j);
            }
            const bool first = bit(ev.first, r);
            const float dt = s_dt[ch * LD + r], u = dt * s_x[ch * LD + r], dy = s_dy[ch * LD + r];
            float v[V], p = 0.f, q = 0.f, y = 0.f;
#pragma unroll
            for (int j = 0; j < NS; ++j) {
                const float B = s_B[r * NP + s * NS + j], C = s_C[r * NP + s * NS + j];
                float hp = i > 0 ? ha[i > 0 ? i - 1 : 0][j] : hs[j];
                if (first) hp = state_of(a.h0, r, j);
                dh[j] = fmaf(C, dy, dh[j]);
                y = fmaf(C, ha[i][j], y);
                v[j] = dh[j] * u;
                v[NS + j] = dy * ha[i][j];
                p = fmaf(dh[j], B, p);
                dh[j] *= ea[i][j];
                const float w = dh[j] * hp;
                dA[j] = fmaf(w, dt, dA[j]);
                q = fmaf(w, A2[j], q);
            }
            if (first) {
                const SeqRange sr = find_seq(a.cu, a.num_seqs, a.M, a.T, t0 + r);
#pragma unroll
                for (int j = 0; j < NS; ++j) {
                    const int n = s * NS + j;
                    if (a.dh0 != nullptr && live && n < a.N) a.dh0[((long long)sr.q * a.D + d) * a.N + n] = dh[j];
                    dh[j] = 0.f;
                }
            }
            // dB, dC over the warp's channels
            int cnt = V;
#pragma unroll
            for (int m = 16; m >= S; m >>= 1) {
                if (cnt > 1) {
                    cnt /= 2;
                    const bool up = lane & m;
#pragma unroll
                    for (int k = 0; k < cnt; ++k) {
                        const float keep = up ? v[k + cnt] : v[k], send = up ? v[k] : v[k + cnt];
                        v[k] = keep + __shfl_xor_sync(0xffffffffu, send, m);
                    }
                } else {
                    v[0] += __shfl_xor_sync(0xffffffffu, v[0], m);
                }
            }
            if (writer) {
#pragma unroll
                for (int k = 0; k < RV; ++k) {
                    const int o = off + k;   // 0..NS-1: dB, then dC
                    red[i * 2 * NP + (o < NS ? s * NS + o : NP + s * NS + o - NS)] = v[k];
                }
            }
            pv[i & 3] = p; qv[i & 3] = q; yv[i & 3] = y;
            if ((i & 3) == 0) {
                lane_sum4<S>(pv[0], pv[1], pv[2], pv[3], s, &s_p[ch * LD + r]);
                lane_sum4<S>(qv[0], qv[1], qv[2], qv[3], s, &s_q[ch * LD + r]);
                lane_sum4<S>(yv[0], yv[1], yv[2], yv[3], s, &s_y[ch * LD + r]);
            }
        }
        __syncthreads();
        for (int k = tid; k < SUB * 2 * NP; k += kThreads) {
            const int i = k / (2 * NP), w = k % (2 * NP) / NP, n = k % NP, r = sb * SUB + i;
            if (n >= a.N || r >= rows) continue;
            float t = 0.f;
#pragma unroll
            for (int x = 0; x < kWarps; ++x) t += s_red[((sb & 1) * kWarps + x) * SUB * 2 * NP + k];
            bcpart[(((long long)blk * a.M + t0 + r) * 2 + w) * a.N + n] = t;
        }
    }
    float* pseg = part + sg * ((long long)a.D * a.N + 2 * a.D);
    if (live) {
#pragma unroll
        for (int j = 0; j < NS; ++j)
            if (s * NS + j < a.N) pseg[(long long)d * a.N + s * NS + j] = dA[j];
    }
    __syncthreads();

    // rows and channels as they were staged: dx, ddelta, dz; dDskip and the bias' gradient
    const int c0 = (tid % VPR) * 8, cn = max(0, min(8, cb.n - c0)), dd = cb.d0 + c0;
    float sD[8] = {}, sb_[8] = {}, dsk[8], bias[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        dsk[i] = i < cn && a.Dskip ? a.Dskip[dd + i] : 0.f;
        bias[i] = i < cn && a.delta_bias ? a.delta_bias[dd + i] : 0.f;
    }
#pragma unroll 1
    for (int row = tid / VPR; row < L; row += RPP) {
        if (!bit(ev.in, row) || cn == 0) continue;
        const long long t = t0 + row;
        float v[8], dx[8], dv[8];
        unpack<T, 8>(load8<T, ALIGNED>(static_cast<const T*>(a.delta) + t * a.ds + dd, cn), v);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int at = (c0 + i) * LD + row;
            const float dt = s_dt[at], x = s_x[at], dy = s_dy[at], p = s_p[at];
            dx[i] = fmaf(p, dt, dsk[i] * dy);
            dv[i] = fmaf(p, x, s_q[at] * (1.0f / kLog2e));
            if (a.softplus) dv[i] *= sigmoid<false>(v[i] + bias[i]);
            sD[i] = fmaf(dy, x, sD[i]);
            sb_[i] += dv[i];
        }
        store8<T, ALIGNED>(static_cast<T*>(a.dx) + t * a.D + dd, dx, cn);
        store8<T, ALIGNED>(static_cast<T*>(a.ddelta) + t * a.D + dd, dv, cn);
        if (a.z != nullptr) {
            float z[8], g[8];
            unpack<T, 8>(load8<T, ALIGNED>(static_cast<const T*>(a.z) + t * a.zs + dd, cn), z);
            unpack<T, 8>(load8<T, ALIGNED>(static_cast<const T*>(a.d_out) + t * a.D + dd, cn), g);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int at = (c0 + i) * LD + row;
                const float sg1 = sigmoid<sizeof(T) == 2>(z[i]);
                g[i] *= fmaf(dsk[i], s_x[at], s_y[at]) * sg1 * fmaf(z[i], 1.0f - sg1, 1.0f);
            }
            store8<T, ALIGNED>(static_cast<T*>(a.dz) + t * a.D + dd, g, cn);
        }
    }
    __syncthreads();
    // over the rows: RPP partial sums per channel, in the staging area (2 RPP <= 2 L columns)
    float* s0 = sm;   // [2][RPP][CH]
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        s0[(tid / VPR) * CH + c0 + i] = sD[i];
        s0[(RPP + tid / VPR) * CH + c0 + i] = sb_[i];
    }
    __syncthreads();
    for (int k = tid; k < 2 * CH; k += kThreads) {
        const int w = k / CH, c = k % CH;
        if (c >= cb.n) continue;
        float t = 0.f;
        for (int r = 0; r < RPP; ++r) t += s0[(w * RPP + r) * CH + c];
        pseg[(long long)a.D * a.N + (long long)w * a.D + cb.d0 + c] = t;
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
#pragma unroll 8
    for (int b = 0; b < per; ++b) s += p[(long long)b * a.M * 2 * a.N];
    static_cast<T*>(w ? a.dC : a.dB)[(t * a.G + g) * a.N + n] = from_f32<T>(s);
}

struct Layout {
    long long K;      // segments
    int nblk, per;    // channel blocks in all, per group
    size_t hseg, rseg, dtseg, part, bcpart, flags, bytes;
};
int lanes_of(int N) { return N <= 4 ? 1 : N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : 16; }
Layout layout(long long M, int D, int N, int G) {
    Layout l;
    const int S = lanes_of(N), L = S >= 4 ? 64 : 32, CH = kThreads / S;
    l.K = (M + L - 1) / L;
    l.per = (D / G + CH - 1) / CH;
    l.nblk = l.per * G;
    size_t at = 0;
    auto take = [&](size_t n) { const size_t o = at; at += (n + 255) / 256 * 256; return o; };
    const size_t dn = (size_t)D * N;
    l.hseg = take(sizeof(float) * l.K * dn);
    l.rseg = take(sizeof(float) * l.K * dn);
    l.dtseg = take(sizeof(float) * l.K * D);
    l.part = take(sizeof(float) * (l.K > 0 ? l.K : 1) * (dn + 2 * D));
    l.bcpart = take(sizeof(float) * l.nblk * M * 2 * N);
    l.flags = take(l.K);
    l.bytes = at;
    return l;
}

template <typename T, int S, int NS, int SUB, bool ALIGNED>
cudaError_t go(const SsmArgs& a, cudaStream_t s) {
    const Layout l = layout(a.M, a.D, a.N, a.G);
    float* hseg = reinterpret_cast<float*>(a.ws + l.hseg);
    float* rseg = reinterpret_cast<float*>(a.ws + l.rseg);
    float* dtseg = reinterpret_cast<float*>(a.ws + l.dtseg);
    float* part = reinterpret_cast<float*>(a.ws + l.part);
    float* bcpart = reinterpret_cast<float*>(a.ws + l.bcpart);
    uint8_t* flags = a.ws + l.flags;
    const long long extra = a.cu != nullptr || a.T == 0 ? (a.num_seqs < 64 ? a.num_seqs : 64) : 0;
    const long long dn = (long long)a.D * a.N, bc = a.M * a.G * 2 * a.N;
    if (l.nblk * (l.K + extra) > 0x7fffffffLL || (bc + 255) / 256 > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    constexpr int CH = kThreads / S, L = seg_rows<S>(), LD = L + 4, NP = S * NS;
    constexpr size_t sm1 = sizeof(float) * (3 * CH * LD + 2 * L * NP), sm2 = grad_smem<S, NS, SUB>();
    cudaError_t e = cudaSuccess;
    if (l.K + extra > 0) {
        auto k1 = ssm_bwd_summary_kernel<T, S, NS, ALIGNED>;
        if ((e = cudaFuncSetAttribute(k1, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sm1)) != cudaSuccess) return e;
        k1<<<(unsigned)(l.nblk * (l.K + extra)), kThreads, sm1, s>>>(a, l.K, l.nblk, hseg, rseg, dtseg, flags);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    if (l.K > 0) {
        ssm_bwd_join_kernel<<<dim3((unsigned)((dn + 127) / 128), 2), 128, 0, s>>>(a, l.K, hseg, rseg, dtseg, flags);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        auto k3 = ssm_bwd_grad_kernel<T, S, NS, SUB, ALIGNED>;
        if ((e = cudaFuncSetAttribute(k3, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sm2)) != cudaSuccess) return e;
        k3<<<(unsigned)(l.nblk * l.K), kThreads, sm2, s>>>(a, l.K, l.nblk, hseg, rseg, part, bcpart);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        ssm_bwd_bc_kernel<T><<<(unsigned)((bc + 255) / 256), 256, 0, s>>>(a, l.per, bcpart);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    return launch_colsum(part, (int)l.K, dn, a.dA, a.D, a.dDskip, a.D, a.ddelta_bias, s);
}

template <typename T, bool ALIGNED>
cudaError_t go_n(const SsmArgs& a, cudaStream_t s) {
    if (a.N <= 4) return go<T, 1, 4, 8, ALIGNED>(a, s);
    if (a.N <= 8) return go<T, 2, 4, 8, ALIGNED>(a, s);
    if (a.N <= 16) return go<T, 4, 4, 8, ALIGNED>(a, s);
    if (a.N <= 32) return go<T, 8, 4, 8, ALIGNED>(a, s);
    if (a.N <= 64) return go<T, 16, 4, 8, ALIGNED>(a, s);
    return go<T, 16, 8, 4, ALIGNED>(a, s);
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

cudaError_t launch_ssm_bwd(const SsmArgs& a, bool bf16, cudaStream_t s) {
    return bf16 ? ssm::go_t<__nv_bfloat16>(a, s) : ssm::go_t<float>(a, s);
}

size_t ssm_bwd_workspace_bytes(long long B, long long T, int D, int N, int G) {
    return ssm::layout(B * T, D, N, G).bytes;
}

}  // namespace kda
