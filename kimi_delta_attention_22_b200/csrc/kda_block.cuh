// kda_block.cuh -- launch interfaces and device helpers of the recurrent block's
// operators (short causal convolution, selective state space scan, layer norm).
#pragma once

#include "kda_internal.cuh"

namespace kda {

constexpr int kSMs = 148;   // B200

struct ConvArgs {
    const void* x;
    const float* w;
    const float* bias;
    const void* state0;
    const int32_t* cu;
    void* out;
    void* stateT;
    // backward
    const void* d_out;
    const void* d_stateT;
    void* dx;
    float* dw;
    float* db;
    void* dstate0;
    float* part;
    int32_t* dev_status;
    long long M, T;      // rows in all, rows per sequence (dense)
    long long xs;        // row stride of x
    int D, W, num_seqs;
};

cudaError_t launch_conv_fwd(const ConvArgs& a, bool bf16, bool silu, cudaStream_t s);
cudaError_t launch_conv_step(const ConvArgs& a, bool bf16, bool silu, cudaStream_t s);
cudaError_t launch_conv_bwd(const ConvArgs& a, bool bf16, bool grad_bf16, bool silu, cudaStream_t s);
size_t conv_bwd_workspace_bytes(long long M, int D, int W);

struct SsmArgs {
    const void* x;
    const void* delta;
    const float* A;
    const void* Bm;
    const void* Cm;
    const float* Dskip;
    const void* z;
    const float* delta_bias;
    const float* h0;
    const int32_t* cu;
    void* out;
    float* hT;
    // backward
    const void* d_out;
    const float* d_hT;
    void* dx;
    void* ddelta;
    float* dA;
    void* dB;
    void* dC;
    float* dDskip;
    void* dz;
    float* ddelta_bias;
    float* dh0;
    uint8_t* ws;
    int32_t* dev_status;
    long long M, T;      // rows in all, rows per sequence (dense)
    long long xs, ds, zs, bs, cs;   // row strides
    int D, N, G, num_seqs, softplus;
};

cudaError_t launch_ssm_fwd(const SsmArgs& a, bool bf16, cudaStream_t s);
size_t ssm_fwd_workspace_bytes(long long B, long long T, int D, int N, int G, bool varlen);
cudaError_t launch_ssm_step(const SsmArgs& a, bool bf16, cudaStream_t s);
cudaError_t launch_ssm_bwd(const SsmArgs& a, bool bf16, cudaStream_t s);
size_t ssm_bwd_workspace_bytes(long long B, long long T, int D, int N, int G);

struct NormArgs {
    const void* x;
    const float* w;
    const float* b;
    void* out;
    float* mean;
    float* rstd;
    const void* d_out;
    void* dx;
    float* dw;
    float* db;
    float* part;
    long long rows, xs;
    int G, D;
    float eps;
};

cudaError_t launch_norm_fwd(const NormArgs& a, bool bf16, cudaStream_t s);
cudaError_t launch_norm_bwd(const NormArgs& a, bool bf16, cudaStream_t s);
size_t norm_bwd_workspace_bytes(long long rows, int G, int D, bool bf16);

// out_i[c] = sum_k part[k][off_i + c], k in order within each of sixteen interleaved
// partial sums: the second stage of a parameter gradient's reduction over the rows.
cudaError_t launch_colsum(const float* part, int K, long long n0, float* out0, long long n1, float* out1,
                          long long n2, float* out2, cudaStream_t s);

// ------------------------------------------------------------------ device helpers

struct SeqRange {
    long long b, e;   // rows [b, e)
    int q;            // sequence
    bool ok;          // row t lies in a sequence whose bounds are consistent
};

// The sequence of row t (0 <= t < M).  Dense: t / T.  Packed: the last n with
// cu[n] <= t, which skips empty sequences; bounds that break the rules, the begin in front among
// them (a sequence that starts inside an earlier one), give ok = false, so that no address is
// ever formed from them.
__device__ __forceinline__ SeqRange find_seq(const int32_t* cu, int n, long long M, long long T, long long t) {
    SeqRange r;
    if (cu == nullptr) {
        r.q = t <= 0xffffffffLL ? (int)((unsigned)t / (unsigned)T) : (int)(t / T);   // t < M, T <= M
        r.b = (long long)r.q * T;
        r.e = r.b + T;
        r.ok = true;
        return r;
    }
    if (n <= 0) {   // a packed batch without sequences: cu has one entry
        r.q = 0;
        r.b = r.e = 0;
        r.ok = false;
        return r;
    }
    int lo = 0, hi = n;   // the last i in [0, n) with cu[i] <= t, or 0
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(cu + mid) <= t) lo = mid; else hi = mid;
    }
    r.q = lo;
    const int p = __ldg(cu + (lo > 0 ? lo - 1 : 0)), b = __ldg(cu + lo), e = __ldg(cu + lo + 1);
    r.b = b;
    r.e = e;
    r.ok = b >= 0 && p <= b && b <= t && t < e && e <= M && (lo > 0 || b == 0);
    return r;
}

// Bounds of sequence q with the same rules as find_seq; flags a broken one.
__device__ __forceinline__ bool check_seq(const int32_t* cu, int q, long long M, long long T, int32_t* dev_status,
                                          long long& b, long long& e) {
    if (cu == nullptr) {
        b = (long long)q * T;
        e = b + T;
        return true;
    }
    b = __ldg(cu + q);
    e = __ldg(cu + q + 1);
    const long long before = q > 0 ? __ldg(cu + q - 1) : b;
    if (b < 0 || b < before || e < b || e > M || (q == 0 && b != 0)) {
        if (dev_status) atomicOr(dev_status, KDA_DEV_BAD_SEQLENS);
        return false;
    }
    return true;
}

// VEC consecutive elements as one access (VEC * sizeof(T) = 16 or 8 bytes, or one element).
template <typename T, int VEC>
struct Pack {
    static constexpr int kWords = VEC * (int)sizeof(T) / 4 > 0 ? VEC * (int)sizeof(T) / 4 : 1;
    uint32_t w[kWords];
};
// READ_ONLY: the read-only path, for what no thread stores while the kernel runs.  A tensor that the
// kernel may store in place is read by plain loads, which stay in front of this thread's stores.
template <bool READ_ONLY, typename W>
__device__ __forceinline__ W load_word(const void* p) {
    const W* w = static_cast<const W*>(p);
    if constexpr (READ_ONLY) return __ldg(w);
    else return *w;
}
template <int VEC, bool READ_ONLY = true, typename T>
__device__ __forceinline__ Pack<T, VEC> load_pack(const T* p) {
    Pack<T, VEC> r;
    if constexpr (VEC * sizeof(T) == 16) {
        const uint4 v = load_word<READ_ONLY, uint4>(p);
        r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
    } else if constexpr (VEC * sizeof(T) == 8) {
        const uint2 v = load_word<READ_ONLY, uint2>(p);
        r.w[0] = v.x; r.w[1] = v.y;
    } else if constexpr (sizeof(T) == 2) {
        static_assert(VEC == 1, "one element");
        r.w[0] = load_word<READ_ONLY, unsigned short>(p);
    } else {
        static_assert(VEC == 1, "one element");
        r.w[0] = load_word<READ_ONLY, unsigned int>(p);
    }
    return r;
}
template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> zero_pack() {
    Pack<T, VEC> r;
#pragma unroll
    for (int i = 0; i < Pack<T, VEC>::kWords; ++i) r.w[i] = 0;
    return r;
}
template <typename T, int VEC>
__device__ __forceinline__ void unpack(const Pack<T, VEC>& p, float* f) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        if constexpr (sizeof(T) == 2) {   // bf16 is the upper half of an fp32
            f[i] = __uint_as_float((i & 1) ? (p.w[i / 2] & 0xffff0000u) : (p.w[i / 2] << 16));
        } else {
            f[i] = __uint_as_float(p.w[i]);
        }
    }
}
template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> pack(const float* f) {
    Pack<T, VEC> r;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) r.w[i] = __float_as_uint(f[i]);
    } else if constexpr (VEC == 1) {
        const __nv_bfloat16 h = __float2bfloat16_rn(f[0]);
        r.w[0] = *reinterpret_cast<const unsigned short*>(&h);
    } else {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            r.w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
    }
    return r;
}
template <typename T, int VEC>
__device__ __forceinline__ void store_pack(T* p, const Pack<T, VEC>& v) {
    if constexpr (VEC * sizeof(T) == 16) {
        *reinterpret_cast<uint4*>(p) = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
    } else if constexpr (VEC * sizeof(T) == 8) {
        *reinterpret_cast<uint2*>(p) = make_uint2(v.w[0], v.w[1]);
    } else if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<unsigned short*>(p) = (unsigned short)v.w[0];
    } else {
        *reinterpret_cast<unsigned int*>(p) = v.w[0];
    }
}
template <typename T, int VEC>
__device__ __forceinline__ void store_f32(T* p, const float* f) {
    store_pack<T, VEC>(p, pack<T, VEC>(f));
}

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// Two fp32 values in a register pair; one instruction works on both (the same roundings as
// two scalar ones, half the issue slots).
struct F2 {
    float x, y;
};
__device__ __forceinline__ unsigned long long f2_bits(F2 a) {
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
    return r;
}
__device__ __forceinline__ F2 f2_of(unsigned long long v) {
    F2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    unsigned long long r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(f2_bits(a)), "l"(f2_bits(b)));
    return f2_of(r);
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(f2_bits(a)), "l"(f2_bits(b)));
    return f2_of(r);
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(f2_bits(a)), "l"(f2_bits(b)), "l"(f2_bits(c)));
    return f2_of(r);
}
__device__ __forceinline__ F2 both(float v) { return F2{v, v}; }
__device__ __forceinline__ F2 ex2(F2 v) { return F2{ex2(v.x), ex2(v.y)}; }
__device__ __forceinline__ F2 rcp(F2 v) {
    F2 r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(v.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(v.y));
    return r;
}

// The functions of the step size and the gate work on pairs and take the hardware's exponential
// and reciprocal: each within a few units, |v| log2(e) more through the exponent's rounding.
__device__ __forceinline__ F2 sigmoid2(F2 v) { return rcp(add2(both(1.0f), ex2(mul2(v, both(-kLog2e))))); }

// a * b + c, a + b and a * b over VEC values, in pairs where there are pairs.
template <int VEC>
__device__ __forceinline__ void fma_n(const float* a, const float* b, float* c) {   // c += a * b
    if constexpr (VEC == 1) {
        c[0] = fmaf(a[0], b[0], c[0]);
    } else {
#pragma unroll
        for (int v = 0; v < VEC; v += 2) {
            const F2 o = fma2(F2{a[v], a[v + 1]}, F2{b[v], b[v + 1]}, F2{c[v], c[v + 1]});
            c[v] = o.x;
            c[v + 1] = o.y;
        }
    }
}

// 1 / (1 + e^-v).  FAST (bf16 outputs): the hardware exponential and quotient, within a few
// fp32 units, far below the output's rounding; otherwise the full-precision functions.
template <bool FAST>
__device__ __forceinline__ float sigmoid(float v) {
    if constexpr (FAST) return __fdividef(1.0f, 1.0f + __expf(-v));
    return 1.0f / (1.0f + expf(-v));
}

// v sigmoid(v) and its derivative sigmoid(v) (1 + v (1 - sigmoid(v))) over VEC values.
template <int VEC, bool FAST>
__device__ __forceinline__ void sigmoid_n(const float* v, float* s) {
    if constexpr (FAST && VEC > 1) {
#pragma unroll
        for (int i = 0; i < VEC; i += 2) {
            const F2 o = sigmoid2(F2{v[i], v[i + 1]});
            s[i] = o.x;
            s[i + 1] = o.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) s[i] = sigmoid<FAST>(v[i]);
    }
}
template <int VEC, bool FAST>
__device__ __forceinline__ void silu_n(float* v) {
    float s[VEC];
    sigmoid_n<VEC, FAST>(v, s);
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] *= s[i];
}

// Asynchronous copies into slots of shared memory that only the copying thread reads: rows are
// under way without holding registers, and no barrier is needed.
template <int BYTES>
__device__ __forceinline__ void copy_async(void* dst, const void* src) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory"); }
// A pack in shared memory.
template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> lds_pack(const void* p) {
    Pack<T, VEC> r;
    if constexpr (VEC * sizeof(T) == 16) {
        const uint4 v = *static_cast<const uint4*>(p);
        r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
    } else {
        static_assert(VEC * sizeof(T) == 8, "8 or 16 bytes");
        const uint2 v = *static_cast<const uint2*>(p);
        r.w[0] = v.x; r.w[1] = v.y;
    }
    return r;
}

// Dynamic shared memory beyond the 48 KB that a kernel may use unasked.
template <typename K>
inline cudaError_t allow_smem(K k, size_t bytes) {
    if (bytes <= 48 * 1024) return cudaSuccess;
    return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

// Whether every access of VEC * el bytes at p + k * stride_bytes is aligned.
inline bool vec_ok(const void* p, long long stride_bytes, int bytes) {
    return p == nullptr || ((reinterpret_cast<uintptr_t>(p) % (unsigned)bytes) == 0 && stride_bytes % bytes == 0);
}

}  // namespace kda
