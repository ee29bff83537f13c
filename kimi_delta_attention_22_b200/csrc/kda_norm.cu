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
// The gradient's CTAs walk rows of one group with the parameter gradients of the lane's
// columns in registers, and write one partial sum each.
#include "kda_block.cuh"

namespace kda {
namespace {

// Sum of two values over the L lanes that share a row (L <= 32: lanes of a warp;
// else the whole CTA of L threads, through shared memory; buf is two such areas used in turn).
template <int L>
__device__ __forceinline__ float2 row_sum(float x, float y, float2* buf, int& turn) {
#pragma unroll
    for (int m = (L < 32 ? L : 32) / 2; m > 0; m >>= 1) {
        x += __shfl_xor_sync(0xffffffffu, x, m);
        y += __shfl_xor_sync(0xffffffffu, y, m);
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
                y += __shfl_xor_sync(0xffffffffu, y, m);
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

// Rows in flight per group of lanes (short rows: the loads of two hide more latency).
template <int L>
constexpr int rows_per_group() { return L > 32 ? 1 : 2; }

__device__ __forceinline__ long long div_by(long long a, int b) {   // a >= 0; 32-bit where that is enough
    return a <= 0xffffffffLL ? (long long)((unsigned)a / (unsigned)b) : a / b;
}

template <typename T, int VEC, int L, int NC>
__global__ void __launch_bounds__(block_threads<L>()) norm_fwd_kernel(NormArgs a) {
    constexpr int NI = rows_per_group<L>();
    __shared__ float2 buf[L > 32 ? 2 * (L / 32) : 1];
    int turn = 0;
    const int lane = threadIdx.x % L, sub = threadIdx.x / L;
    const long long item0 = ((long long)blockIdx.x * cta_rows<L>() + sub) * NI, items = a.rows * a.G;
    const float inv = 1.0f / (float)a.D;
    Pack<T, VEC> px[NI][NC];
    int g[NI];
#pragma unroll
    for (int r = 0; r < NI; ++r) {
        const long long item = item0 + r < items ? item0 + r : 0, row = div_by(item, a.G);
        g[r] = (int)(item - row * a.G);
        const T* x = static_cast<const T*>(a.x) + row * a.xs + (long long)g[r] * a.D;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int d = (c * L + lane) * VEC;
            px[r][c] = d < a.D ? load_pack<VEC>(x + d) : zero_pack<T, VEC>();
        }
    }
#pragma unroll
    for (int r = 0; r < NI; ++r) {
        const long long item = item0 + r;
        float f[NC][VEC];
        float s = 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            unpack<T, VEC>(px[r][c], f[c]);
#pragma unroll
            for (int v = 0; v < VEC; ++v) s += f[c][v];
        }
        const float mean = row_sum<L>(s, 0.f, buf, turn).x * inv;
        s = 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            if ((c * L + lane) * VEC < a.D) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    f[c][v] -= mean;
                    s = fmaf(f[c][v], f[c][v], s);
                }
            }
        }
        const float rstd = rsqrtf(row_sum<L>(s, 0.f, buf, turn).x * inv + a.eps);
        if (item >= items) continue;   // no exchange is skipped: the next row's come first of all again
        T* out = static_cast<T*>(a.out) + item * a.D;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int d = (c * L + lane) * VEC;
            if (d >= a.D) continue;
            constexpr int PV = VEC > 4 ? 4 : VEC;   // parameters: fp32, at most 16 bytes at a time
#pragma unroll
            for (int v = 0; v < VEC; ++v) f[c][v] *= rstd;
#pragma unroll
            for (int v = 0; v < VEC; v += PV) {
                float t[PV];
                if (a.w) {
                    unpack<float, PV>(load_pack<PV>(a.w + (long long)g[r] * a.D + d + v), t);
#pragma unroll
                    for (int k = 0; k < PV; ++k) f[c][v + k] *= t[k];
                }
                if (a.b) {
                    unpack<float, PV>(load_pack<PV>(a.b + (long long)g[r] * a.D + d + v), t);
#pragma unroll
                    for (int k = 0; k < PV; ++k) f[c][v + k] += t[k];
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

__device__ __forceinline__ void copy16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}

// grid (K, G): CTA (k, g) walks rows k, k + K, .. (times the rows it holds at once) of group g.
// RING: x and d_out of the next rows are copied ahead (STG - 1 rows) into slots of shared memory
// that only the copying thread reads; without it the next row waits in registers.
template <typename T, int VEC, int L, int NC, bool RING>
__global__ void __launch_bounds__(block_threads<L>()) norm_bwd_kernel(NormArgs a, int K) {
    constexpr int R = cta_rows<L>(), NT = block_threads<L>(), STG = 4;
    __shared__ float2 buf[L > 32 ? 2 * (L / 32) : 1];
    extern __shared__ __align__(16) uint4 ring[];   // [STG][2][NC][NT]
    int turn = 0;
    const int lane = threadIdx.x % L, sub = threadIdx.x / L;
    const int g = blockIdx.y;
    const T* xg = static_cast<const T*>(a.x) + (long long)g * a.D;
    const T* yg = static_cast<const T*>(a.d_out) + (long long)g * a.D;
    const long long step = (long long)K * R, gd = (long long)a.G * a.D;
    const float inv = 1.0f / (float)a.D;
    float dw[NC][VEC] = {}, db[NC][VEC] = {};
    float w[RING ? 1 : NC][VEC];   // RING: read from the cache again for every row, the registers are worth more
    auto weight = [&](int c, float* o) {
        const int d = (c * L + lane) * VEC;
        constexpr int PV = VEC > 4 ? 4 : VEC;
#pragma unroll
        for (int v = 0; v < VEC; v += PV) {
            if (d < a.D && a.w) {
                unpack<float, PV>(load_pack<PV>(a.w + (long long)g * a.D + d + v), o + v);
            } else {
#pragma unroll
                for (int k = 0; k < PV; ++k) o[v + k] = d < a.D ? 1.f : 0.f;
            }
        }
    };
    if constexpr (!RING) {
#pragma unroll
        for (int c = 0; c < NC; ++c) weight(c, w[c]);
    }
    Pack<T, VEC> px[NC], pg[NC];
    float mean = 0.f, rstd = 0.f;
    auto ahead = [&](long long row, int st) {   // RING: a row's copies (nothing behind the last row)
        if constexpr (RING) {
            if (row < a.rows) {
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    const int d = (c * L + lane) * VEC;
                    if (d < a.D) {
                        copy16(&ring[((st * 2 + 0) * NC + c) * NT + threadIdx.x], xg + row * a.xs + d);
                        copy16(&ring[((st * 2 + 1) * NC + c) * NT + threadIdx.x], yg + row * gd + d);
                    }
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    };
    auto fetch = [&](long long row, int st) {   // row's x, d_out into registers
        const bool live = row < a.rows;
        if constexpr (RING) asm volatile("cp.async.wait_group %0;" ::"n"(STG - 2) : "memory");
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int d = (c * L + lane) * VEC;
            const bool in = live && d < a.D;
            px[c] = pg[c] = zero_pack<T, VEC>();
            if constexpr (RING) {
                if (in) {
                    const uint4 u = ring[((st * 2 + 0) * NC + c) * NT + threadIdx.x], v = ring[((st * 2 + 1) * NC + c) * NT + threadIdx.x];
                    px[c].w[0] = u.x; px[c].w[1] = u.y; px[c].w[2] = u.z; px[c].w[3] = u.w;
                    pg[c].w[0] = v.x; pg[c].w[1] = v.y; pg[c].w[2] = v.z; pg[c].w[3] = v.w;
                }
            } else if (in) {
                px[c] = load_pack<VEC>(xg + row * a.xs + d);
                pg[c] = load_pack<VEC>(yg + row * gd + d);
            }
        }
    };
    auto stats = [&](long long row) {
        const bool live = row < a.rows;
        mean = live ? __ldg(a.mean + row * a.G + g) : 0.f;
        rstd = live ? __ldg(a.rstd + row * a.G + g) : 0.f;
    };
    // Every thread of the CTA makes the same number of turns (the sums meet in barriers).
    const long long first = (long long)blockIdx.x * R;
    int st = 0;
    if constexpr (RING) {
#pragma unroll
        for (int k = 0; k < STG - 1; ++k) ahead(first + sub + k * step, k);
    } else {
        fetch(first + sub, 0);
    }
    stats(first + sub);
    for (long long base = first; base < a.rows; base += step) {
        const long long row = base + sub;
        if constexpr (RING) {
            fetch(row, st);
            ahead(row + (STG - 1) * step, (st + STG - 1) % STG);   // into the slot that the last turn read
            st = (st + 1) % STG;
        }
        float xh[NC][VEC], gy[NC][VEC];
        float s1 = 0.f, s2 = 0.f;
        const float rs = rstd, mu = mean;
        stats(row + step);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            unpack<T, VEC>(px[c], xh[c]);
            unpack<T, VEC>(pg[c], gy[c]);
            float wr[VEC];
            if constexpr (RING) weight(c, wr);
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                xh[c][v] = (xh[c][v] - mu) * rs;
                dw[c][v] = fmaf(gy[c][v], xh[c][v], dw[c][v]);
                db[c][v] += gy[c][v];
                gy[c][v] *= RING ? wr[v] : w[RING ? 0 : c][v];   // 0 behind the row's end
                s1 += gy[c][v];
                s2 = fmaf(gy[c][v], xh[c][v], s2);
            }
        }
        if constexpr (!RING) fetch(row + step, 0);   // under way while this row's sums meet
        const float2 t = row_sum<L>(s1, s2, buf, turn);
        const float c1 = t.x * inv, c2 = t.y * inv;
        if (row < a.rows) {
            T* dx = static_cast<T*>(a.dx) + (row * a.G + g) * a.D;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int d = (c * L + lane) * VEC;
                if (d >= a.D) continue;
                float o[VEC];
#pragma unroll
                for (int v = 0; v < VEC; ++v) o[v] = rs * (gy[c][v] - c1 - xh[c][v] * c2);
                store_f32<T, VEC>(dx + d, o);
            }
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

__global__ void __launch_bounds__(256) colsum_kernel(const float* part, int K, long long cols, long long n0, float* out0,
                                                     long long n1, float* out1, long long n2, float* out2) {
    __shared__ float red[8][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const long long c = (long long)blockIdx.x * 32 + tx;
    float s = 0.f;
    if (c < cols) {
        const float* p = part + c;
#pragma unroll 4
        for (int k = ty; k < K; k += 8) s += p[(long long)k * cols];
    }
    red[ty][tx] = s;
    __syncthreads();
    if (ty != 0 || c >= cols) return;
#pragma unroll
    for (int i = 1; i < 8; ++i) s += red[i][tx];
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
    const long long items = a.rows * a.G;
    constexpr int per = cta_rows<L>() * rows_per_group<L>();
    const long long grid = (items + per - 1) / per;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    norm_fwd_kernel<T, VEC, L, NC><<<(unsigned)grid, block_threads<L>(), 0, s>>>(a);
    return cudaGetLastError();
}
template <typename T, int VEC, int L, int NC>
cudaError_t bwd_one(const NormArgs& a, cudaStream_t s) {
    constexpr bool RING = VEC > 1 && NC * block_threads<L>() * 128 <= 128 * 1024;
    constexpr int smem = RING ? NC * block_threads<L>() * 128 : 0;   // 4 rows' x and d_out
    const int K = bwd_ctas(a.rows, a.G, cta_rows<L>(), block_threads<L>(), NC * VEC >= 16 ? 512 : 1024);
    auto k = norm_bwd_kernel<T, VEC, L, NC, RING>;
    cudaError_t e;
    if (smem > 0 && (e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
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

// Lanes per row and accesses per lane: the fewest lanes that hold the row in registers, so
// that short rows share a warp and no row waits for a barrier that it does not need.
template <typename T, bool BWD>
cudaError_t norm_t(const NormArgs& a, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
#define KDA_NORM(VEC, L, NC)                                \
    do {                                                    \
        if constexpr (BWD) return bwd_one<T, VEC, L, NC>(a, s); \
        else return fwd_one<T, VEC, L, NC>(a, s);           \
    } while (0)
    if (norm_vec(a, sizeof(T))) {
        const int n = a.D / V;   // accesses per row
        if (n <= 8) KDA_NORM(V, 8, 1);
        if (n <= 16) KDA_NORM(V, 16, 1);
        if (n <= 32) KDA_NORM(V, 32, 1);
        if (n <= 64) KDA_NORM(V, 32, 2);
        if (n <= 128) KDA_NORM(V, 128, 1);
        if (n <= 256) KDA_NORM(V, 256, 1);
        if (n <= 512) KDA_NORM(V, 256, 2);
        if (n <= 1024) KDA_NORM(V, 512, 2);
        if (n <= 2048) KDA_NORM(V, 1024, 2);
        if constexpr (V == 4) {
            if (n <= 4096) KDA_NORM(V, 1024, 4);
            KDA_NORM(V, 1024, 8);
        } else {
            KDA_NORM(V, 1024, 4);
        }
    }
    if (a.D <= 32) KDA_NORM(1, 8, 4);
    if (a.D <= 256) KDA_NORM(1, 32, 8);
    if (a.D <= 2048) KDA_NORM(1, 256, 8);
    if (a.D <= 8192) KDA_NORM(1, 1024, 8);
    KDA_NORM(1, 1024, 32);
#undef KDA_NORM
}

}  // namespace

cudaError_t launch_colsum(const float* part, int K, long long n0, float* out0, long long n1, float* out1, long long n2,
                          float* out2, cudaStream_t s) {
    const long long cols = n0 + n1 + n2;
    if (cols == 0) return cudaSuccess;
    colsum_kernel<<<(unsigned)((cols + 31) / 32), 256, 0, s>>>(part, K, cols, n0, out0, n1, out1, n2, out2);
    return cudaGetLastError();
}

cudaError_t launch_norm_fwd(const NormArgs& a, bool bf16, cudaStream_t s) {
    return bf16 ? norm_t<__nv_bfloat16, false>(a, s) : norm_t<float, false>(a, s);
}
cudaError_t launch_norm_bwd(const NormArgs& a, bool bf16, cudaStream_t s) {
    return bf16 ? norm_t<__nv_bfloat16, true>(a, s) : norm_t<float, true>(a, s);
}

// The partial sums of the most CTAs that any layout of the row would use.
size_t norm_bwd_workspace_bytes(long long rows, int G, int D) {
    return sizeof(float) * 2 * (size_t)G * D * bwd_ctas(rows, G, 1, 128, 1024);
}

}  // namespace kda
