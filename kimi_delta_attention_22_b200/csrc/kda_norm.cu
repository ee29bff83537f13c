// kda_norm.cu -- layer norm over the last axis of x [rows, groups, D], forward and
// gradient, and the second stage of the parameter gradients' reductions.
//
//   xhat = (x - mean) rstd,   out = xhat w + b
//   gy = d_out w,  dx = rstd (gy - mean(gy) - xhat mean(gy xhat))
//   dw = sum_rows d_out xhat,  db = sum_rows d_out
//
// A handful of operations per element: HBM bounds both directions.  L lanes own one
// (row, group), each lane NC accesses of VEC elements (one access: 16 bytes, or one
// element where rows do not start on 16 bytes), so that the row is read once and stays in
// registers: the variance is the exact sum over (x - mean)^2, not a difference of moments.
// out may be x, and dx x or d_out: these are read by plain loads (or copies ahead, of other rows).
// The gradient's CTAs walk rows of one group with the parameter gradients of the lane's
// columns in registers, and write one partial sum each.  bf16, in a captured graph: gradient of
// 65536 x 4096 285 us, 5.7 TB/s (305 to 325 us as single calls, by card); per-head forward of
// 131072 x 128 14 to 15 us, 4.6 TB/s (a call takes 16.5 us, which is the host's time).
#include "kda_block.cuh"

namespace kda {
namespace {

// Sum of two values over the L lanes that share a row (L <= 32: lanes of a warp;
// else the whole CTA of L threads, through shared memory; buf is two such areas used in turn).
template <int L>
__device__ __forceinline__ float2 row_sum(float x, float y, float2* buf, int& turn, bool two = true) {
#pragma unroll
    for (int m = (L < 32 ? L : 32) / 2; m > 0; m >>= 1) {
        x += __shfl_xor_sync(0xffffffffu, x, m);
        if (two) y += __shfl_xor_sync(0xffffffffu, y, m);
    }
    if constexpr (L > 32) {
        constexpr int NW = L / 32;
        float2* b = buf + turn * NW;
        turn ^= 1;
        if ((threadIdx.x & 31) == 0) b[threadIdx.x >> 5] = make_float2(x, y);
        __syncthreads();
        x = y = 0.f;
        if constexpr (NW <= 8) {
#pragma unroll
            for (int i = 0; i < NW; ++i) {
                x += b[i].x;
                y += b[i].y;
            }
        } else {
            const int l = threadIdx.x & 31;
            if (l < NW) {
                x = b[l].x;
                y = b[l].y;
            }
#pragma unroll
            for (int m = 16; m > 0; m >>= 1) {
                x += __shfl_xor_sync(0xffffffffu, x, m);
                if (two) y += __shfl_xor_sync(0xffffffffu, y, m);
            }
        }
    }
    return make_float2(x, y);
}

template <int L>
constexpr int cta_threads() { return L > 256 ? L : 256; }
template <int L>
constexpr int cta_rows() { return L > 32 ? 1 : cta_threads<L>() / L; }
template <int L>
constexpr int block_threads() { return L > 32 ? L : 256; }

// Rows of one group that L lanes take together (short rows: the loads of four hide more
// latency, and their weights are read once).
template <int L, int NC>
constexpr int rows_per_item() { return L > 32 ? 1 : NC > 1 ? 2 : 4; }

__device__ __forceinline__ long long div_by(long long a, int b) {   // a >= 0; 32-bit where that is enough
    return a <= 0xffffffffLL ? (long long)((unsigned)a / (unsigned)b) : a / b;
}

// Whether access c of a lane lies in the row.  The layouts (norm_t) give a row of vector accesses,
// and every row of more than 32 lanes, more than half of the lanes' accesses, so only the upper
// half of them is ever compared; FULL: the row fills all of them.  The comparisons cost more
// than they look: each keeps the access apart as a branch of its own (65536 x 4096 gradient in a
// captured graph: 329 us with all, 285 us with none).
template <int VEC, int L, int NC, bool FULL>
__device__ __forceinline__ bool in_row(int c, int lane, int D) {
    if constexpr (FULL) return true;
    if ((VEC > 1 || L > 32) && c < NC / 2) return true;
    return (c * L + lane) * VEC < D;
}

// Parameters of an access' columns: fp32, at most 16 bytes at a time.
template <int VEC>
__device__ __forceinline__ void load_params(const float* p, float* o) {
    constexpr int PV = VEC > 4 ? 4 : VEC;
#pragma unroll
    for (int v = 0; v < VEC; v += PV) unpack<float, PV>(load_pack<PV>(p + v), o + v);
}
template <int VEC>
__device__ __forceinline__ F2 pair(const float* f, int v) { return F2{f[v], f[v + 1]}; }

// Two rows of 32 elements per lane would take 130 registers, which leaves one CTA of 256 threads per SM
// instead of two (bf16, 32768 x 1024: 39 us instead of 27).  The other layouts are not bounded (0): the
// compiler spends more registers under a bound of one or two CTAs (32768 x 4096: 132 us instead of 103).
template <int VEC, int L, int NC>
constexpr int fwd_ctas() { return L <= 32 && VEC * NC == 32 ? 2 : 0; }

template <typename T, int VEC, int L, int NC, bool FULL>
__global__ void __launch_bounds__(block_threads<L>(), fwd_ctas<VEC, L, NC>()) norm_fwd_kernel(NormArgs a) {
    constexpr int NI = rows_per_item<L, NC>();
    __shared__ float2 buf[L > 32 ? 2 * (L / 32) : 1];
    int turn = 0;
    const int lane = threadIdx.x % L, sub = threadIdx.x / L;
    const long long idx = (long long)blockIdx.x * cta_rows<L>() + sub, mb = div_by(idx, a.G);
    const int g = (int)(idx - mb * a.G);
    const long long row0 = mb * NI;
    const float inv = 1.0f / (float)a.D;
    const T* xg = static_cast<const T*>(a.x) + (long long)g * a.D;
    Pack<T, VEC> px[NI][NC];
#pragma unroll
    for (int r = 0; r < NI; ++r) {
        const bool live = row0 + r < a.rows;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int d = (c * L + lane) * VEC;
            px[r][c] = live && in_row<VEC, L, NC, FULL>(c, lane, a.D) ? load_pack<VEC, false>(xg + (row0 + r) * a.xs + d) : zero_pack<T, VEC>();
        }
    }
    float w[NC][VEC], b[NC][VEC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int d = (c * L + lane) * VEC;
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            w[c][v] = 1.f;
            b[c][v] = 0.f;
        }
        if (NI > 1 && in_row<VEC, L, NC, FULL>(c, lane, a.D)) {   // one row: read when they are needed instead
            if (a.w) load_params<VEC>(a.w + (long long)g * a.D + d, w[c]);
            if (a.b) load_params<VEC>(a.b + (long long)g * a.D + d, b[c]);
        }
    }
#pragma unroll
    for (int r = 0; r < NI; ++r) {
        float f[NC][VEC];
        float s = 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            unpack<T, VEC>(px[r][c], f[c]);
#pragma unroll
            for (int v = 0; v < VEC; ++v) s += f[c][v];
        }
        const float mean = row_sum<L>(s, 0.f, buf, turn, false).x * inv;
        F2 q{0.f, 0.f};
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            if (in_row<VEC, L, NC, FULL>(c, lane, a.D)) {
                if constexpr (VEC == 1) {
                    f[c][0] -= mean;
                    q.x = fmaf(f[c][0], f[c][0], q.x);
                } else {
#pragma unroll
                    for (int v = 0; v < VEC; v += 2) {
                        const F2 o = add2(pair<VEC>(f[c], v), both(-mean));
                        q = fma2(o, o, q);
                        f[c][v] = o.x;
                        f[c][v + 1] = o.y;
                    }
                }
            }
        }
        const float rstd = rsqrtf(row_sum<L>(q.x + q.y, 0.f, buf, turn, false).x * inv + a.eps);
        if (row0 + r >= a.rows) continue;   // no exchange is skipped: the next row's come first of all again
        const long long item = (row0 + r) * a.G + g;
        T* out = static_cast<T*>(a.out) + item * a.D;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int d = (c * L + lane) * VEC;
            if (!in_row<VEC, L, NC, FULL>(c, lane, a.D)) continue;
            if (NI == 1) {
                if (a.w) load_params<VEC>(a.w + (long long)g * a.D + d, w[c]);
                if (a.b) load_params<VEC>(a.b + (long long)g * a.D + d, b[c]);
            }
            if constexpr (VEC == 1) {
                f[c][0] = fmaf(f[c][0] * rstd, w[c][0], b[c][0]);
            } else {
#pragma unroll
                for (int v = 0; v < VEC; v += 2) {
                    const F2 o = fma2(mul2(pair<VEC>(f[c], v), both(rstd)), pair<VEC>(w[c], v), pair<VEC>(b[c], v));
                    f[c][v] = o.x;
                    f[c][v + 1] = o.y;
                }
            }
            store_f32<T, VEC>(out + d, f[c]);
        }
        if (lane == 0 && a.mean != nullptr) {
            a.mean[item] = mean;
            a.rstd[item] = rstd;
        }
    }
}

constexpr int kStages = 3;   // rows in the ring, one of them being worked on

// grid (K, G): CTA (k, g) walks rows k, k + K, .. (times the rows it holds at once) of group g.
// RING: x and d_out of the next rows are copied ahead (STG - 1 rows) into slots of shared memory
// that only the copying thread reads; without it a row is loaded in the turn that uses it.  A row is
// gone over twice in registers as it was loaded, once for its sums and the parameters'
// gradients, once for dx: unpacking again costs less than the registers of fp32 copies.
// Threads per SM that the registers are held to where two accesses of a lane leave the choice:
// three quarters of the warps hide a row's exchanges better than half of them with no spill
// (of two vector accesses with spills, of eight element accesses without).
template <int VEC, int L, int NC>
constexpr int bwd_threads() {
    if ((VEC == 1 && NC == 8) || (VEC == 8 && NC == 2 && L > 32 && L <= 256)) return 768;
    if (NC * VEC <= 8) return 1024;
    return block_threads<L>() > 512 ? block_threads<L>() : 512;
}

template <typename T, int VEC, int L, int NC, bool RING, bool FULL>
__global__ void __launch_bounds__(block_threads<L>(), bwd_threads<VEC, L, NC>() / block_threads<L>()) norm_bwd_kernel(NormArgs a, int K) {
    constexpr int R = cta_rows<L>(), NT = block_threads<L>(), STG = kStages;
    __shared__ float2 buf[L > 32 ? 2 * (L / 32) : 1];
    extern __shared__ __align__(16) uint4 ring[];   // [STG][2][NC][NT], then this thread's weights [NC][2][NT]
    int turn = 0;
    const int lane = threadIdx.x % L, sub = threadIdx.x / L;
    const int g = blockIdx.y;
    const long long step = (long long)K * R, gd = (long long)a.G * a.D;
    const float inv = 1.0f / (float)a.D;
    const T* xg = static_cast<const T*>(a.x) + (long long)g * a.D + lane * VEC;
    const T* yg = static_cast<const T*>(a.d_out) + (long long)g * a.D + lane * VEC;
    T* og = static_cast<T*>(a.dx) + (long long)g * a.D + lane * VEC;
    const float* wg = a.w + (long long)g * a.D + lane * VEC;
    float dw[NC][VEC] = {}, db[NC][VEC] = {};
    float4* s_w = reinterpret_cast<float4*>(ring + STG * 2 * NC * NT) + threadIdx.x;
    Pack<T, VEC> px[NC], pg[NC];
    auto in = [&](int c) { return in_row<VEC, L, NC, FULL>(c, lane, a.D); };
    auto weights = [&](int c, float* o) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) o[v] = 1.f;
        if (a.w != nullptr && in(c)) load_params<VEC>(wg + c * L * VEC, o);
    };
    if constexpr (RING) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            float o[VEC];
            weights(c, o);
#pragma unroll
            for (int v = 0; v < VEC; v += 4) s_w[(c * (VEC / 4) + v / 4) * NT] = make_float4(o[v], o[v + 1], o[v + 2], o[v + 3]);
        }
    }
    auto weights_again = [&](int c, float* o) {
        if constexpr (RING) {
#pragma unroll
            for (int v = 0; v < VEC; v += 4) {
                const float4 f = s_w[(c * (VEC / 4) + v / 4) * NT];
                o[v] = f.x; o[v + 1] = f.y; o[v + 2] = f.z; o[v + 3] = f.w;
            }
        } else {
            weights(c, o);
        }
    };
    // Every thread of the CTA makes the same number of turns (the sums meet in barriers).
    const long long first = (long long)blockIdx.x * R + sub;
    // running pointers: the row that is read (or copied ahead) next, the one that is written next
    const T *xn = xg + first * a.xs, *yn = yg + first * gd;
    T* on = og + first * gd;
    const float *mn = a.mean + first * a.G + g, *rn = a.rstd + first * a.G + g;
    long long left = first < a.rows ? (a.rows - first + step - 1) / step : 0;       // rows of this group of lanes
    long long ahead_left = left;
    auto ahead = [&](int st) {   // RING: the next row's copies (nothing behind the last row)
        if constexpr (RING) {
            if (ahead_left > 0) {
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    if (!in(c)) continue;
                    copy_async<16>(&ring[((st * 2 + 0) * NC + c) * NT + threadIdx.x], xn + c * L * VEC);
                    copy_async<16>(&ring[((st * 2 + 1) * NC + c) * NT + threadIdx.x], yn + c * L * VEC);
                }
                xn += step * a.xs;
                yn += step * gd;
                --ahead_left;
            }
            copy_commit();
        }
    };
    if constexpr (RING) {
#pragma unroll
        for (int k = 0; k < STG - 1; ++k) ahead(k);
    }
    float mean = left > 0 ? __ldg(mn) : 0.f, rstd = left > 0 ? __ldg(rn) : 0.f;
    int st = 0;
    for (long long base = (long long)blockIdx.x * R; base < a.rows; base += step, --left) {
        const bool live = left > 0;
        if constexpr (RING) copy_wait<STG - 2>();
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            px[c] = pg[c] = zero_pack<T, VEC>();
            if (!live || !in(c)) continue;
            if constexpr (RING) {
                px[c] = lds_pack<T, VEC>(&ring[((st * 2 + 0) * NC + c) * NT + threadIdx.x]);
                pg[c] = lds_pack<T, VEC>(&ring[((st * 2 + 1) * NC + c) * NT + threadIdx.x]);
            } else {
                px[c] = load_pack<VEC, false>(xn + c * L * VEC);
                pg[c] = load_pack<VEC, false>(yn + c * L * VEC);
            }
        }
        if constexpr (RING) {
            ahead(st == 0 ? STG - 1 : st - 1);   // into the slot that the last turn read
            st = st == STG - 1 ? 0 : st + 1;
        } else {
            xn += step * a.xs;
            yn += step * gd;
        }
        const float rs = rstd, mu = mean;
        mn += step * a.G;
        rn += step * a.G;
        if (left > 1) {
            mean = __ldg(mn);
            rstd = __ldg(rn);
        }
        F2 s1{0.f, 0.f}, s2{0.f, 0.f};
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            if (!in(c)) continue;
            float x[VEC], y[VEC], wr[VEC];
            unpack<T, VEC>(px[c], x);
            unpack<T, VEC>(pg[c], y);
            weights_again(c, wr);
            const float* w = wr;
            if constexpr (VEC == 1) {
                const float xh = (x[0] - mu) * rs, gw = y[0] * w[0];
                dw[c][0] = fmaf(y[0], xh, dw[c][0]);
                db[c][0] += y[0];
                s1.x += gw;
                s2.x = fmaf(gw, xh, s2.x);
            } else {
#pragma unroll
                for (int v = 0; v < VEC; v += 2) {
                    const F2 xh = mul2(add2(pair<VEC>(x, v), both(-mu)), both(rs)), gy = pair<VEC>(y, v);
                    const F2 nw = fma2(gy, xh, pair<VEC>(dw[c], v)), nb = add2(gy, pair<VEC>(db[c], v));
                    dw[c][v] = nw.x;
                    db[c][v] = nb.x;
                    dw[c][v + 1] = nw.y;
                    db[c][v + 1] = nb.y;
                    const F2 gw = mul2(gy, pair<VEC>(w, v));
                    s1 = add2(s1, gw);
                    s2 = fma2(gw, xh, s2);
                }
            }
        }
        const float2 t = row_sum<L>(s1.x + s1.y, s2.x + s2.y, buf, turn);
        if (live) {
            // rstd (gw - c1 - xhat c2) = gw rstd + ((x - mean) k2 + k1), k2 = -c2 rstd^2, k1 = -c1 rstd.  The
            // mean is taken from x first: x k2 + (k1 - mean k2) saves an addition and loses the digits that a
            // mean far above the deviation shares with x.
            const float k2 = -t.y * inv * rs * rs, k1 = -t.x * inv * rs;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                if (!in(c)) continue;
                float x[VEC], y[VEC], wr[VEC];
                unpack<T, VEC>(px[c], x);
                unpack<T, VEC>(pg[c], y);
                weights_again(c, wr);
                const float* w = wr;
                if constexpr (VEC == 1) {
                    x[0] = fmaf(y[0] * w[0], rs, fmaf(x[0] - mu, k2, k1));
                } else {
#pragma unroll
                    for (int v = 0; v < VEC; v += 2) {
                        const F2 gw = mul2(pair<VEC>(y, v), pair<VEC>(w, v));
                        const F2 o = fma2(gw, both(rs), fma2(add2(pair<VEC>(x, v), both(-mu)), both(k2), both(k1)));
                        x[v] = o.x;
                        x[v + 1] = o.y;
                    }
                }
                store_f32<T, VEC>(on + c * L * VEC, x);
            }
            on += step * gd;
        }
    }
    if (a.part == nullptr) return;
    // part[k]: dw [G][D], then db [G][D]
    float* pw = a.part + (long long)blockIdx.x * 2 * gd + (long long)g * a.D;
    float* pb = pw + gd;
    if constexpr (R == 1) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int d = (c * L + lane) * VEC;
#pragma unroll
            for (int v = 0; v < VEC; ++v)
                if (d < a.D) {
                    pw[d + v] = dw[c][v];
                    pb[d + v] = db[c][v];
                }
        }
    } else {
        __shared__ float red[R * L * 2];
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                __syncthreads();
                red[threadIdx.x] = dw[c][v];
                red[R * L + threadIdx.x] = db[c][v];
                __syncthreads();
                if (threadIdx.x < 2 * L) {
                    const int which = threadIdx.x / L, d = (c * L + lane) * VEC + v;
                    float s = 0.f;
                    for (int r = 0; r < R; ++r) s += red[which * R * L + r * L + lane];
                    if (d < a.D) (which ? pb : pw)[d] = s;
                }
            }
    }
}

// Sixteen interleaved partial sums per column, added in order.
constexpr int kSumRows = 16;
__global__ void __launch_bounds__(32 * kSumRows) colsum_kernel(const float* part, int K, long long cols, long long n0, float* out0,
                                                               long long n1, float* out1, long long n2, float* out2) {
    __shared__ float red[kSumRows][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const long long c = (long long)blockIdx.x * 32 + tx;
    float s = 0.f;
    if (c < cols) {
        const float* p = part + c;
#pragma unroll 8
        for (int k = ty; k < K; k += kSumRows) s += __ldg(p + (long long)k * cols);
    }
    red[ty][tx] = s;
    __syncthreads();
    if (ty != 0 || c >= cols) return;
#pragma unroll
    for (int i = 1; i < kSumRows; ++i) s += red[i][tx];
    if (c < n0) {
        if (out0) out0[c] = s;
    } else if (c < n0 + n1) {
        if (out1) out1[c - n0] = s;
    } else if (out2) {
        out2[c - n0 - n1] = s;
    }
}

// CTAs along the rows: as many as are resident at once (`sm_threads` per SM), at least four turns each.
int bwd_ctas(long long rows, int G, int rows_per_cta, int threads, int sm_threads) {
    long long K = ((long long)kSMs * (sm_threads > threads ? sm_threads / threads : 1) + G - 1) / G;
    const long long most = (rows + 4LL * rows_per_cta - 1) / (4LL * rows_per_cta);
    if (K > most) K = most;
    return (int)(K < 1 ? 1 : K);
}

template <typename T, int VEC, int L, int NC>
cudaError_t fwd_one(const NormArgs& a, cudaStream_t s) {
    constexpr int NI = rows_per_item<L, NC>();
    const long long items = (a.rows + NI - 1) / NI * a.G, grid = (items + cta_rows<L>() - 1) / cta_rows<L>();
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const bool full = VEC > 1 && a.D == L * NC * VEC;
    auto k = full ? norm_fwd_kernel<T, VEC, L, NC, (VEC > 1)> : norm_fwd_kernel<T, VEC, L, NC, false>;
    k<<<(unsigned)grid, block_threads<L>(), 0, s>>>(a);
    return cudaGetLastError();
}
template <int VEC, int L, int NC>
int layout_ctas(long long rows, int G) {
    return bwd_ctas(rows, G, cta_rows<L>(), block_threads<L>(), bwd_threads<VEC, L, NC>());
}
template <typename T, int VEC, int L, int NC>
cudaError_t bwd_one(const NormArgs& a, cudaStream_t s) {
    constexpr int bytes = NC * block_threads<L>() * (kStages * 32 + VEC * 4);
    constexpr bool RING = VEC > 1 && bytes <= 200 * 1024;
    constexpr int smem = RING ? bytes : 0;
    const int K = layout_ctas<VEC, L, NC>(a.rows, a.G);
    const bool full = VEC > 1 && a.D == L * NC * VEC;
    auto k = full ? norm_bwd_kernel<T, VEC, L, NC, RING, (VEC > 1)> : norm_bwd_kernel<T, VEC, L, NC, RING, false>;
    cudaError_t e;
    if ((e = allow_smem(k, smem)) != cudaSuccess) return e;
    k<<<dim3((unsigned)K, (unsigned)a.G), block_threads<L>(), smem, s>>>(a, K);
    e = cudaGetLastError();
    if (e != cudaSuccess || a.part == nullptr) return e;
    const long long gd = (long long)a.G * a.D;
    return launch_colsum(a.part, K, gd, a.dw, gd, a.db, 0, nullptr, s);
}

bool norm_vec(const NormArgs& a, int el) {
    const long long row = (long long)a.D * el;
    return a.D % (16 / el) == 0 && vec_ok(a.x, a.xs * el, 16) && vec_ok(a.x, row, 16) && vec_ok(a.out, row, 16) &&
           vec_ok(a.d_out, row, 16) && vec_ok(a.dx, row, 16) && vec_ok(a.w, 16, 16) && vec_ok(a.b, 16, 16);
}

// Lanes per row and accesses per lane: few lanes that hold the row in registers, so that
// short rows share a warp and no row waits for a barrier that it does not need.
// f(Layout<..>{}) is called for the layout of rows of D elements of EL bytes, with or without vector accesses.
template <int VEC_, int L_, int NC_>
struct Layout {
    static constexpr int VEC = VEC_, L = L_, NC = NC_;
};
template <int EL, bool BWD, typename F>
auto with_layout(bool vec, int D, F&& f) {
    constexpr int V = 16 / EL;
#define KDA_NORM(VEC, L, NC) return f(Layout<VEC, L, NC>{})
    if (vec) {
        const int n = D / V;   // accesses per row
        if (n <= 8) KDA_NORM(V, 8, 1);
        if (n <= 16) KDA_NORM(V, 8, 2);
        if (n <= 32) KDA_NORM(V, 32, 1);
        if (n <= 64) KDA_NORM(V, 32, 2);
        if constexpr (BWD) {
            // bf16 above 1024 columns: two accesses, as a row's sums and copies cost the same for each
            // lane (32768 x 4096: one 169 us, two 158, four 244).  fp32, with half the columns per
            // access, and short rows: one (32768 x 1024 bf16: 68 us with two, 58 with one; fp32 92 and 74)
            if (n <= 128) KDA_NORM(V, 128, 1);
            if constexpr (V == 4) {
                if (n <= 256) KDA_NORM(V, 256, 1);
                if (n <= 512) KDA_NORM(V, 512, 1);
            } else {
                if (n <= 256) KDA_NORM(V, 128, 2);
                if (n <= 512) KDA_NORM(V, 256, 2);
            }
            if (n <= 1024) KDA_NORM(V, 512, 2);
            if (n <= 2048) KDA_NORM(V, 512, 4);
        } else {
            // four accesses per lane: the loads of a row are under way together, and few warps meet in
            // its sums (bf16, two or one per lane: 32768 x 1024 42 us instead of 29, 32768 x 4096 119
            // instead of 105, 8192 x 16384 209 instead of 128; eight: 32768 x 2048 64 instead of 55)
            if (n <= 128) KDA_NORM(V, 32, 4);
            if (n <= 256) KDA_NORM(V, 64, 4);
            if (n <= 512) KDA_NORM(V, 128, 4);
            if (n <= 1024) KDA_NORM(V, 256, 4);
            if (n <= 2048) KDA_NORM(V, 512, 4);
        }
        if constexpr (V == 4) {
            if (n <= 4096) KDA_NORM(V, 1024, 4);
            KDA_NORM(V, 1024, 8);
        } else {
            KDA_NORM(V, 1024, 4);
        }
    }
    if (D <= 32) KDA_NORM(1, 8, 4);
    if (D <= 256) KDA_NORM(1, 32, 8);
    // Element accesses: CTAs of few warps with long runs per lane, several of them per SM (one CTA of
    // 1024 threads has nothing to do while its sums meet).  bf16, 8192 x 4095: forward 147 us with
    // 1024 lanes, 40 us with 256; gradient 184 and 97 us, of which half by its scalar arithmetic.
    if (D <= 512) KDA_NORM(1, 64, 8);
    if constexpr (BWD) {
        if (D <= 1024) KDA_NORM(1, 128, 8);
    } else {
        if (D <= 1024) KDA_NORM(1, 64, 16);
    }
    if (D <= 2048) KDA_NORM(1, 128, 16);
    if (D <= 4096) KDA_NORM(1, 256, 16);
    if (D <= 8192) KDA_NORM(1, 512, 16);
    if (D <= 16384) KDA_NORM(1, 1024, 16);
    KDA_NORM(1, 1024, 32);
#undef KDA_NORM
}

template <typename T, bool BWD>
cudaError_t norm_t(const NormArgs& a, cudaStream_t s) {
    return with_layout<sizeof(T), BWD>(norm_vec(a, sizeof(T)), a.D, [&](auto l) {
        using Lay = decltype(l);
        if constexpr (BWD) return bwd_one<T, Lay::VEC, Lay::L, Lay::NC>(a, s);
        else return fwd_one<T, Lay::VEC, Lay::L, Lay::NC>(a, s);
    });
}

// CTAs (partial sums) of the gradient's two possible layouts: the pointers' alignment decides between them.
template <int EL>
int most_ctas(long long rows, int G, int D) {
    const auto ctas = [&](auto l) { return layout_ctas<decltype(l)::VEC, decltype(l)::L, decltype(l)::NC>(rows, G); };
    const int one = with_layout<EL, true>(false, D, ctas);
    const int vec = D % (16 / EL) == 0 ? with_layout<EL, true>(true, D, ctas) : 0;
    return one > vec ? one : vec;
}

}  // namespace

cudaError_t launch_colsum(const float* part, int K, long long n0, float* out0, long long n1, float* out1, long long n2,
                          float* out2, cudaStream_t s) {
    const long long cols = n0 + n1 + n2;
    if (cols == 0) return cudaSuccess;
    colsum_kernel<<<(unsigned)((cols + 31) / 32), 32 * kSumRows, 0, s>>>(part, K, cols, n0, out0, n1, out1, n2, out2);
    return cudaGetLastError();
}

cudaError_t launch_norm_fwd(const NormArgs& a, bool bf16, cudaStream_t s) {
    return bf16 ? norm_t<__nv_bfloat16, false>(a, s) : norm_t<float, false>(a, s);
}
cudaError_t launch_norm_bwd(const NormArgs& a, bool bf16, cudaStream_t s) {
    return bf16 ? norm_t<__nv_bfloat16, true>(a, s) : norm_t<float, true>(a, s);
}

size_t norm_bwd_workspace_bytes(long long rows, int G, int D, bool bf16) {
    return sizeof(float) * 2 * (size_t)G * D * (bf16 ? most_ctas<2>(rows, G, D) : most_ctas<4>(rows, G, D));
}

}  // namespace kda
