// kda_ssm_step.cu -- one row of the selective scan on a state: h <- e^{dt A} h + dt x B,
// out = (C h + Dskip x) silu(z).
#include "kda_ssm.cuh"

namespace kda {
namespace ssm {
namespace {

// One row of every sequence: the fp32 state is read and written once, which bounds the step.
// S lanes per channel, NQ runs of four states per lane (one 16-byte access each where N is a
// multiple of 4); a thread takes the same channel of two sequences, all of their loads first.
template <typename T, int S, int NQ, bool VEC4>
__global__ void __launch_bounds__(256, 4) ssm_step_kernel(SsmArgs a) {
    constexpr int NB = 2;
    const unsigned i = blockIdx.x * 256u + threadIdx.x;
    const int s = (int)(i % S);
    const bool live = i / S < (unsigned)a.D;
    const int d = live ? (int)(i / S) : 0;
    const int g = a.G == 1 ? 0 : d / (a.D / a.G);
    const long long q0 = (long long)blockIdx.y * NB;
    float h[NB][NQ * 4], x[NB], v[NB], z[NB];
    Pack<T, 4> B[NB][NQ], C[NB][NQ];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const long long q = q0 + b;
        const bool on = live && q < a.num_seqs;
        const float* hp = a.hT + (q * a.D + d) * a.N;
        const T* Bp = static_cast<const T*>(a.Bm) + q * a.bs + (long long)g * a.N;
        const T* Cp = static_cast<const T*>(a.Cm) + q * a.cs + (long long)g * a.N;
#pragma unroll
        for (int k = 0; k < NQ; ++k) {
            const int n0 = (k * S + s) * 4;
            B[b][k] = C[b][k] = zero_pack<T, 4>();
            if (VEC4) {
                float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
                if (on && n0 < a.N) {
                    f = *reinterpret_cast<const float4*>(hp + n0);
                    B[b][k] = load_pack<4>(Bp + n0);
                    C[b][k] = load_pack<4>(Cp + n0);
                }
                h[b][4 * k] = f.x; h[b][4 * k + 1] = f.y; h[b][4 * k + 2] = f.z; h[b][4 * k + 3] = f.w;
            } else {
                float fb[4], fc[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bool in = on && n0 + j < a.N;
                    h[b][4 * k + j] = in ? hp[n0 + j] : 0.f;
                    fb[j] = in ? to_f32<T>(Bp[n0 + j]) : 0.f;
                    fc[j] = in ? to_f32<T>(Cp[n0 + j]) : 0.f;
                }
                B[b][k] = pack<T, 4>(fb);   // exact: they were of this type
                C[b][k] = pack<T, 4>(fc);
            }
        }
        x[b] = on ? to_f32<T>(static_cast<const T*>(a.x)[q * a.xs + d]) : 0.f;
        v[b] = on ? to_f32<T>(static_cast<const T*>(a.delta)[q * a.ds + d]) : 0.f;
        z[b] = on && a.z ? to_f32<T>(static_cast<const T*>(a.z)[q * a.zs + d]) : 0.f;
    }
    float A2[NQ * 4];
#pragma unroll
    for (int k = 0; k < NQ; ++k) {
        const int n0 = (k * S + s) * 4;
#pragma unroll
        for (int j = 0; j < 4; ++j) A2[4 * k + j] = 0.f;
        if (VEC4) {
            if (live && n0 < a.N) unpack<float, 4>(load_pack<4>(a.A + (long long)d * a.N + n0), A2 + 4 * k);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) A2[4 * k + j] = live && n0 + j < a.N ? a.A[(long long)d * a.N + n0 + j] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) A2[4 * k + j] *= kLog2e;
    }
    const float bias = a.delta_bias && live ? a.delta_bias[d] : 0.f;
    const float dsk = a.Dskip && live ? a.Dskip[d] : 0.f;
    F2 dt2{v[0] + bias, v[1] + bias};
    if (a.softplus) dt2 = softplus2(dt2);
    const F2 zz{z[0], z[1]}, gate = mul2(zz, sigmoid2(zz));
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const long long q = q0 + b;
        const bool on = live && q < a.num_seqs;
        const float dt = b ? dt2.y : dt2.x, u = dt * x[b];
        F2 acc{0.f, 0.f};
#pragma unroll
        for (int k = 0; k < NQ; ++k) {
            float fb[4], fc[4];
            unpack<T, 4>(B[b][k], fb);
            unpack<T, 4>(C[b][k], fc);
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
                const int n = 4 * k + j;
                const F2 e = ex2(mul2(both(dt), F2{A2[n], A2[n + 1]}));
                const F2 o = fma2(e, F2{h[b][n], h[b][n + 1]}, mul2(both(u), F2{fb[j], fb[j + 1]}));
                acc = fma2(o, F2{fc[j], fc[j + 1]}, acc);
                h[b][n] = o.x;
                h[b][n + 1] = o.y;
            }
        }
        float y = acc.x + acc.y;
#pragma unroll
        for (int m = 1; m < S; m <<= 1) y += __shfl_xor_sync(0xffffffffu, y, m);
        if (!on) continue;
        float* hp = a.hT + (q * a.D + d) * a.N;
#pragma unroll
        for (int k = 0; k < NQ; ++k) {
            const int n0 = (k * S + s) * 4;
            if (VEC4) {
                if (n0 < a.N)
                    *reinterpret_cast<float4*>(hp + n0) = make_float4(h[b][4 * k], h[b][4 * k + 1], h[b][4 * k + 2], h[b][4 * k + 3]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (n0 + j < a.N) hp[n0 + j] = h[b][4 * k + j];
            }
        }
        if (s == 0) {
            y = fmaf(dsk, x[b], y);
            if (a.z) y *= b ? gate.y : gate.x;
            static_cast<T*>(a.out)[q * a.D + d] = from_f32<T>(y);
        }
    }
}

template <typename T, int S, int NQ, bool VEC4>
cudaError_t step_go(const SsmArgs& a, cudaStream_t s) {
    const long long gx = ((long long)a.D * S + 255) / 256, gy = (a.num_seqs + 1) / 2;
    if ((long long)a.D * S > 0xffffff00LL || gy > 65535) return cudaErrorInvalidConfiguration;
    ssm_step_kernel<T, S, NQ, VEC4><<<dim3((unsigned)gx, (unsigned)gy), 256, 0, s>>>(a);
    return cudaGetLastError();
}
template <typename T, bool VEC4>
cudaError_t step_n(const SsmArgs& a, cudaStream_t s) {
    if (a.N <= 4) return step_go<T, 1, 1, VEC4>(a, s);
    if (a.N <= 8) return step_go<T, 1, 2, VEC4>(a, s);
    if (a.N <= 16) return step_go<T, 2, 2, VEC4>(a, s);
    if (a.N <= 32) return step_go<T, 4, 2, VEC4>(a, s);
    if (a.N <= 64) return step_go<T, 8, 2, VEC4>(a, s);
    return step_go<T, 16, 2, VEC4>(a, s);
}

}  // namespace
}  // namespace ssm

cudaError_t launch_ssm_step(const SsmArgs& a, bool bf16, cudaStream_t s) {
    const int b4 = bf16 ? 8 : 16, el = b4 / 4;   // four states at a time
    const bool v = a.N % 4 == 0 && vec_ok(a.hT, 16, 16) && vec_ok(a.A, 16, 16) && vec_ok(a.Bm, a.bs * el, b4) && vec_ok(a.Cm, a.cs * el, b4);
    if (bf16) return v ? ssm::step_n<__nv_bfloat16, true>(a, s) : ssm::step_n<__nv_bfloat16, false>(a, s);
    return v ? ssm::step_n<float, true>(a, s) : ssm::step_n<float, false>(a, s);
}

}  // namespace kda
