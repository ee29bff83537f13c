// kda_block_api.cu -- the C entry points of the recurrent block's operators: host-side
// validation and scratch.  As in kda_api.cu, every check runs before any launch and nothing
// synchronises; scratch without a caller workspace comes from the stream-ordered pool.
#include <initializer_list>
#include <stdint.h>

#include "kda_block.cuh"

namespace {

constexpr long long kMaxRows = 1LL << 31;   // row indexes are 64-bit; grids and partial sums bound the rows

kda_status_t status_of(cudaError_t e) {
    if (e == cudaSuccess) return KDA_OK;
    (void)cudaGetLastError();   // an allocation's or attribute's error stays behind otherwise, for the next launch to report
    return e == cudaErrorInvalidConfiguration ? KDA_ERR_UNSUPPORTED : KDA_ERR_CUDA;
}

bool aligned(const void* p, unsigned by) { return (reinterpret_cast<uintptr_t>(p) % by) == 0; }

bool dtype_ok(int t) { return t == KDA_F32 || t == KDA_BF16; }
unsigned el_of(int t) { return t == KDA_BF16 ? 2u : 4u; }

// B, T and num_seqs of a dense or packed batch.
bool batch_ok(int B, int T, int num_seqs, bool varlen) {
    if (B < 0 || T < 0 || num_seqs < 0) return false;
    return varlen ? B == 1 : num_seqs == B;
}

// Whether an output starts in an input's place.
bool in_place(std::initializer_list<const void*> outs, std::initializer_list<const void*> ins) {
    for (const void* o : outs)
        for (const void* i : ins)
            if (o != nullptr && o == i) return true;
    return false;
}
// Whether two outputs start at the same address.
bool one_place(std::initializer_list<const void*> outs) {
    for (const void* const* o = outs.begin(); o != outs.end(); ++o)
        for (const void* const* p = outs.begin(); p != o; ++p)
            if (*o != nullptr && *o == *p) return true;
    return false;
}
// As in_place for an output whose elements are stored by the thread that read the input's elements at
// the same index: in place is then right where consecutive rows of both lie `row` elements apart.
bool rows_shifted(const void* out, const void* in, long long rows, long long stride, long long row) {
    return out != nullptr && out == in && rows > 1 && stride != row;
}

kda_status_t check_workspace(const void* ws, size_t have, size_t need) {
    if (ws == nullptr) return KDA_OK;
    if (!aligned(ws, 256)) return KDA_ERR_MISALIGNED;
    return have < need ? KDA_ERR_INVALID_ARG : KDA_OK;
}

// Runs `go(scratch)` on the caller's workspace, or on `need` bytes of the stream-ordered pool.
template <typename F>
kda_status_t with_workspace(void* workspace, size_t need, cudaStream_t st, F&& go) {
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const bool pooled = ws == nullptr && need > 0;
    cudaError_t e = pooled ? cudaMallocAsync(reinterpret_cast<void**>(&ws), need, st) : cudaSuccess;
    if (e != cudaSuccess) return status_of(e);
    e = go(ws);
    if (pooled) {
        const cudaError_t f = cudaFreeAsync(ws, st);
        if (e == cudaSuccess) e = f;
    }
    return status_of(e);
}

kda_status_t conv_check(const kda_conv_shape_t* sh, bool varlen) {
    if (sh == nullptr) return KDA_ERR_INVALID_ARG;
    if (!batch_ok(sh->B, sh->T, sh->num_seqs, varlen) || sh->D <= 0 || sh->width < 1) return KDA_ERR_INVALID_ARG;
    if (!dtype_ok(sh->dtype) || (sh->activation != 0 && sh->activation != 1)) return KDA_ERR_INVALID_ARG;
    if (sh->x_stride != 0 && sh->x_stride < sh->D) return KDA_ERR_INVALID_ARG;
    if (!aligned(sh->dev_status, 4)) return KDA_ERR_MISALIGNED;
    if (sh->width < 2 || sh->width > 8 || (long long)sh->B * sh->T > kMaxRows) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

kda::ConvArgs conv_args(const kda_conv_shape_t* sh, const void* x, const float* w, const float* bias,
                        const void* state0, const int32_t* cu) {
    kda::ConvArgs a{};
    a.x = x; a.w = w; a.bias = bias; a.state0 = state0; a.cu = cu;
    a.dev_status = sh->dev_status;
    a.M = (long long)sh->B * sh->T;
    a.T = sh->T;
    a.xs = sh->x_stride != 0 ? sh->x_stride : sh->D;
    a.D = sh->D; a.W = sh->width; a.num_seqs = sh->num_seqs;
    return a;
}

kda_status_t ssm_check(const kda_ssm_shape_t* sh, bool varlen) {
    if (sh == nullptr) return KDA_ERR_INVALID_ARG;
    if (!batch_ok(sh->B, sh->T, sh->num_seqs, varlen) || sh->D <= 0 || sh->N <= 0 || sh->G <= 0 || sh->D % sh->G != 0)
        return KDA_ERR_INVALID_ARG;
    if (!dtype_ok(sh->dtype) || (sh->softplus != 0 && sh->softplus != 1)) return KDA_ERR_INVALID_ARG;
    const long long gn = (long long)sh->G * sh->N;
    const int64_t chan[] = {sh->x_stride, sh->delta_stride, sh->z_stride}, vec[] = {sh->b_stride, sh->c_stride};
    for (int64_t v : chan)
        if (v != 0 && v < sh->D) return KDA_ERR_INVALID_ARG;
    for (int64_t v : vec)
        if (v != 0 && v < gn) return KDA_ERR_INVALID_ARG;
    if (!aligned(sh->dev_status, 4)) return KDA_ERR_MISALIGNED;
    // (the gradient steps over D rows of at least four states with 32-bit strides: D N at 2^29 would overflow them)
    if (sh->N > 128 || (long long)sh->B * sh->T > kMaxRows || (long long)sh->D * sh->N >= (1LL << 29) || gn > 0x7fffffffLL)
        return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

kda::SsmArgs ssm_args(const kda_ssm_shape_t* sh, const void* x, const void* delta, const float* A, const void* Bm,
                      const void* Cm, const float* Dskip, const void* z, const float* delta_bias, const float* h0,
                      const int32_t* cu) {
    kda::SsmArgs a{};
    a.x = x; a.delta = delta; a.A = A; a.Bm = Bm; a.Cm = Cm; a.Dskip = Dskip; a.z = z; a.delta_bias = delta_bias;
    a.h0 = h0; a.cu = cu; a.dev_status = sh->dev_status;
    a.M = (long long)sh->B * sh->T;
    a.T = sh->T;
    const long long gn = (long long)sh->G * sh->N;
    a.xs = sh->x_stride != 0 ? sh->x_stride : sh->D;
    a.ds = sh->delta_stride != 0 ? sh->delta_stride : sh->D;
    a.zs = sh->z_stride != 0 ? sh->z_stride : sh->D;
    a.bs = sh->b_stride != 0 ? sh->b_stride : gn;
    a.cs = sh->c_stride != 0 ? sh->c_stride : gn;
    a.D = sh->D; a.N = sh->N; a.G = sh->G; a.num_seqs = sh->num_seqs; a.softplus = sh->softplus;
    return a;
}

bool ssm_pointers_aligned(const kda::SsmArgs& a, unsigned el) {
    return aligned(a.x, el) && aligned(a.delta, el) && aligned(a.Bm, el) && aligned(a.Cm, el) && aligned(a.z, el) &&
           aligned(a.A, 4) && aligned(a.Dskip, 4) && aligned(a.delta_bias, 4) && aligned(a.h0, 4) && aligned(a.cu, 4);
}

kda_status_t norm_check(const kda_norm_shape_t* sh) {
    if (sh == nullptr) return KDA_ERR_INVALID_ARG;
    if (sh->rows < 0 || sh->groups <= 0 || sh->D <= 0 || !dtype_ok(sh->dtype)) return KDA_ERR_INVALID_ARG;
    if (!(sh->eps >= 0.f)) return KDA_ERR_INVALID_ARG;
    if (sh->x_stride != 0 && sh->x_stride < (long long)sh->groups * sh->D) return KDA_ERR_INVALID_ARG;
    if (sh->D > 32768 || sh->groups > 65535 || sh->rows > kMaxRows) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

}  // namespace

extern "C" {

kda_status_t kda_conv_fwd(const kda_conv_shape_t* sh, const void* x, const float* weight, const float* bias,
                          const void* state0, const int32_t* cu_seqlens, void* out, void* stateT, void* stream) {
    const kda_status_t c = conv_check(sh, cu_seqlens != nullptr);
    if (c != KDA_OK) return c;
    kda::ConvArgs a = conv_args(sh, x, weight, bias, state0, cu_seqlens);
    a.out = out; a.stateT = stateT;
    if (!weight || (a.M > 0 && (!x || !out))) return KDA_ERR_INVALID_ARG;
    const unsigned el = el_of(sh->dtype);
    if (!aligned(x, el) || !aligned(weight, 4) || !aligned(bias, 4) || !aligned(state0, el) || !aligned(cu_seqlens, 4) ||
        !aligned(out, el) || !aligned(stateT, el))
        return KDA_ERR_MISALIGNED;
    if (in_place({stateT}, {state0}) || (a.M > 0 && (in_place({out, stateT}, {x, state0, weight, bias}) || one_place({out, stateT}))))
        return KDA_ERR_INVALID_ARG;
    if (sh->num_seqs == 0) return KDA_OK;
    return status_of(kda::launch_conv_fwd(a, sh->dtype == KDA_BF16, sh->activation == 1, static_cast<cudaStream_t>(stream)));
}

kda_status_t kda_conv_step(const kda_conv_shape_t* sh, const void* x, const float* weight, const float* bias,
                           void* state, void* out, void* stream) {
    const kda_status_t c = conv_check(sh, false);
    if (c != KDA_OK) return c;
    if (sh->T != 1) return KDA_ERR_INVALID_ARG;
    kda::ConvArgs a = conv_args(sh, x, weight, bias, nullptr, nullptr);
    a.out = out; a.stateT = state;
    if (!weight || (a.M > 0 && (!x || !out || !state))) return KDA_ERR_INVALID_ARG;
    const unsigned el = el_of(sh->dtype);
    if (!aligned(x, el) || !aligned(weight, 4) || !aligned(bias, 4) || !aligned(out, el) || !aligned(state, el))
        return KDA_ERR_MISALIGNED;
    if (a.M > 0 && (in_place({out}, {state, weight, bias}) || in_place({state}, {x, weight, bias}) ||
                    rows_shifted(out, x, a.M, a.xs, a.D)))
        return KDA_ERR_INVALID_ARG;
    if (sh->num_seqs == 0) return KDA_OK;
    return status_of(kda::launch_conv_step(a, sh->dtype == KDA_BF16, sh->activation == 1, static_cast<cudaStream_t>(stream)));
}

size_t kda_conv_bwd_workspace_size(const kda_conv_shape_t* sh) {
    if (sh == nullptr || sh->B < 0 || sh->T < 0 || sh->D <= 0 || sh->width < 2 || sh->width > 8) return 0;
    return kda::conv_bwd_workspace_bytes((long long)sh->B * sh->T, sh->D, sh->width);
}

kda_status_t kda_conv_bwd(const kda_conv_shape_t* sh, const void* x, const float* weight, const float* bias,
                          const void* state0, const int32_t* cu_seqlens, const void* d_out, const void* d_stateT,
                          void* dx, float* dweight, float* dbias, void* dstate0, void* workspace,
                          size_t workspace_bytes, void* stream) {
    kda_status_t c = conv_check(sh, cu_seqlens != nullptr);
    if (c != KDA_OK) return c;
    if (sh->grad_dtype != sh->dtype && sh->grad_dtype != KDA_F32) return KDA_ERR_INVALID_ARG;
    kda::ConvArgs a = conv_args(sh, x, weight, bias, state0, cu_seqlens);
    a.d_out = d_out; a.d_stateT = d_stateT;
    a.dx = dx; a.dw = dweight; a.db = dbias; a.dstate0 = dstate0;
    if (!weight || !dweight || (a.M > 0 && (!x || !d_out || !dx))) return KDA_ERR_INVALID_ARG;
    const unsigned el = el_of(sh->dtype);
    if (!aligned(x, el) || !aligned(weight, 4) || !aligned(bias, 4) || !aligned(state0, el) || !aligned(cu_seqlens, 4) ||
        !aligned(d_out, el_of(sh->grad_dtype)) || !aligned(d_stateT, el) || !aligned(dx, el) || !aligned(dweight, 4) ||
        !aligned(dbias, 4) || !aligned(dstate0, el))
        return KDA_ERR_MISALIGNED;
    const size_t need = kda_conv_bwd_workspace_size(sh);
    c = check_workspace(workspace, workspace_bytes, need);
    if (c != KDA_OK) return c;
    // runs read rows, states and their gradients that others store gradients over (those of the
    // parameters are stored behind the last read of anything)
    if (in_place({dstate0}, {state0, d_stateT}) ||
        (a.M > 0 && (in_place({dx, dstate0}, {x, d_out, state0, d_stateT, weight, bias}) || one_place({dx, dweight, dbias, dstate0}))))
        return KDA_ERR_INVALID_ARG;
    return with_workspace(workspace, need, static_cast<cudaStream_t>(stream), [&](uint8_t* ws) {
        a.part = reinterpret_cast<float*>(ws);
        return kda::launch_conv_bwd(a, sh->dtype == KDA_BF16, sh->grad_dtype == KDA_BF16, sh->activation == 1,
                                    static_cast<cudaStream_t>(stream));
    });
}

size_t kda_ssm_fwd_workspace_size(const kda_ssm_shape_t* sh, int varlen) {
    if (ssm_check(sh, varlen != 0) != KDA_OK) return 0;
    return kda::ssm_fwd_workspace_bytes(sh->B, sh->T, sh->D, sh->N, sh->G, varlen != 0);
}

kda_status_t kda_ssm_fwd(const kda_ssm_shape_t* sh, const void* x, const void* delta, const float* A, const void* Bm,
                         const void* Cm, const float* Dskip, const void* z, const float* delta_bias, const float* h0,
                         const int32_t* cu_seqlens, void* out, float* hT, void* workspace, size_t workspace_bytes,
                         void* stream) {
    kda_status_t c = ssm_check(sh, cu_seqlens != nullptr);
    if (c != KDA_OK) return c;
    kda::SsmArgs a = ssm_args(sh, x, delta, A, Bm, Cm, Dskip, z, delta_bias, h0, cu_seqlens);
    a.out = out; a.hT = hT;
    if (!A || (a.M > 0 && (!x || !delta || !Bm || !Cm || !out))) return KDA_ERR_INVALID_ARG;
    const unsigned el = el_of(sh->dtype);
    if (!ssm_pointers_aligned(a, el) || !aligned(out, el) || !aligned(hT, 4)) return KDA_ERR_MISALIGNED;
    const size_t need = kda_ssm_fwd_workspace_size(sh, cu_seqlens != nullptr);
    c = check_workspace(workspace, workspace_bytes, need);
    if (c != KDA_OK) return c;
    if (in_place({hT}, {h0}) || (a.M > 0 && (in_place({out, hT}, {x, delta, z, Bm, Cm, A, Dskip, delta_bias, h0}) || one_place({out, hT}))))
        return KDA_ERR_INVALID_ARG;
    if (sh->num_seqs == 0) return KDA_OK;
    return with_workspace(workspace, need, static_cast<cudaStream_t>(stream), [&](uint8_t* ws) {
        a.ws = ws;
        return kda::launch_ssm_fwd(a, sh->dtype == KDA_BF16, static_cast<cudaStream_t>(stream));
    });
}

kda_status_t kda_ssm_step(const kda_ssm_shape_t* sh, const void* x, const void* delta, const float* A, const void* Bm,
                          const void* Cm, const float* Dskip, const void* z, const float* delta_bias, float* h,
                          void* out, void* stream) {
    const kda_status_t c = ssm_check(sh, false);
    if (c != KDA_OK) return c;
    if (sh->T != 1) return KDA_ERR_INVALID_ARG;
    kda::SsmArgs a = ssm_args(sh, x, delta, A, Bm, Cm, Dskip, z, delta_bias, nullptr, nullptr);
    a.out = out; a.hT = h;
    if (!A || (a.M > 0 && (!x || !delta || !Bm || !Cm || !out || !h))) return KDA_ERR_INVALID_ARG;
    const unsigned el = el_of(sh->dtype);
    if (!ssm_pointers_aligned(a, el) || !aligned(out, el) || !aligned(h, 4)) return KDA_ERR_MISALIGNED;
    if (a.M > 0 && (in_place({out}, {Bm, Cm, A, Dskip, delta_bias, h}) || in_place({h}, {x, delta, z, Bm, Cm, A, Dskip, delta_bias}) ||
                    rows_shifted(out, x, a.M, a.xs, a.D) || rows_shifted(out, delta, a.M, a.ds, a.D) ||
                    rows_shifted(out, z, a.M, a.zs, a.D)))
        return KDA_ERR_INVALID_ARG;
    if (sh->num_seqs == 0) return KDA_OK;
    return status_of(kda::launch_ssm_step(a, sh->dtype == KDA_BF16, static_cast<cudaStream_t>(stream)));
}

size_t kda_ssm_bwd_workspace_size(const kda_ssm_shape_t* sh, int varlen) {
    if (ssm_check(sh, varlen != 0) != KDA_OK) return 0;
    return kda::ssm_bwd_workspace_bytes(sh->B, sh->T, sh->D, sh->N, sh->G);
}

kda_status_t kda_ssm_bwd(const kda_ssm_shape_t* sh, const void* x, const void* delta, const float* A, const void* Bm,
                         const void* Cm, const float* Dskip, const void* z, const float* delta_bias, const float* h0,
                         const int32_t* cu_seqlens, const void* d_out, const float* d_hT, void* dx, void* ddelta,
                         float* dA, void* dB, void* dC, float* dDskip, void* dz, float* ddelta_bias, float* dh0,
                         void* workspace, size_t workspace_bytes, void* stream) {
    kda_status_t c = ssm_check(sh, cu_seqlens != nullptr);
    if (c != KDA_OK) return c;
    kda::SsmArgs a = ssm_args(sh, x, delta, A, Bm, Cm, Dskip, z, delta_bias, h0, cu_seqlens);
    a.d_out = d_out; a.d_hT = d_hT; a.dx = dx; a.ddelta = ddelta; a.dA = dA; a.dB = dB; a.dC = dC;
    a.dDskip = dDskip; a.dz = dz; a.ddelta_bias = ddelta_bias; a.dh0 = dh0;
    if (!A || !dA || (a.M > 0 && (!x || !delta || !Bm || !Cm || !d_out || !dx || !ddelta || !dB || !dC)))
        return KDA_ERR_INVALID_ARG;
    // a gradient exactly where its input is given (rows may be absent altogether)
    if ((Dskip == nullptr) != (dDskip == nullptr) || (delta_bias == nullptr) != (ddelta_bias == nullptr) ||
        (a.M > 0 && (z == nullptr) != (dz == nullptr)))
        return KDA_ERR_INVALID_ARG;
    const unsigned el = el_of(sh->dtype);
    if (!ssm_pointers_aligned(a, el) || !aligned(d_out, el) || !aligned(d_hT, 4) || !aligned(dx, el) ||
        !aligned(ddelta, el) || !aligned(dA, 4) || !aligned(dB, el) || !aligned(dC, el) || !aligned(dDskip, 4) ||
        !aligned(dz, el) || !aligned(ddelta_bias, 4) || !aligned(dh0, 4))
        return KDA_ERR_MISALIGNED;
    const size_t need = kda_ssm_bwd_workspace_size(sh, cu_seqlens != nullptr);
    c = check_workspace(workspace, workspace_bytes, need);
    if (c != KDA_OK) return c;
    // segments read what others store gradients over; only h0 is read by the thread that stores dh0
    // (and the parameters' gradients are stored behind the last read of anything)
    if (in_place({dh0}, {d_hT}) ||
        (a.M > 0 && (in_place({dx, ddelta, dz, dB, dC}, {x, delta, z, Bm, Cm, A, Dskip, delta_bias, h0, d_out, d_hT}) ||
                     in_place({dh0}, {x, delta, z, Bm, Cm, A, Dskip, delta_bias, d_out}) ||
                     one_place({dx, ddelta, dA, dB, dC, dDskip, dz, ddelta_bias, dh0}))))
        return KDA_ERR_INVALID_ARG;
    return with_workspace(workspace, need, static_cast<cudaStream_t>(stream), [&](uint8_t* ws) {
        a.ws = ws;
        return kda::launch_ssm_bwd(a, sh->dtype == KDA_BF16, static_cast<cudaStream_t>(stream));
    });
}

kda_status_t kda_layer_norm_fwd(const kda_norm_shape_t* sh, const void* x, const float* weight, const float* bias,
                                void* out, float* mean, float* rstd, void* stream) {
    const kda_status_t c = norm_check(sh);
    if (c != KDA_OK) return c;
    if ((mean == nullptr) != (rstd == nullptr) && sh->rows > 0) return KDA_ERR_INVALID_ARG;
    if (sh->rows > 0 && (!x || !out)) return KDA_ERR_INVALID_ARG;
    const unsigned el = el_of(sh->dtype);
    if (!aligned(x, el) || !aligned(out, el) || !aligned(weight, 4) || !aligned(bias, 4) || !aligned(mean, 4) ||
        !aligned(rstd, 4))
        return KDA_ERR_MISALIGNED;
    if (sh->rows == 0) return KDA_OK;
    if (in_place({out, mean, rstd}, {weight, bias}) || in_place({mean, rstd}, {x}) || one_place({out, mean, rstd}))
        return KDA_ERR_INVALID_ARG;
    kda::NormArgs a{};
    a.x = x; a.w = weight; a.b = bias; a.out = out; a.mean = mean; a.rstd = rstd;
    a.rows = sh->rows; a.G = sh->groups; a.D = sh->D; a.eps = sh->eps;
    const long long row = (long long)sh->groups * sh->D;
    a.xs = sh->x_stride != 0 ? sh->x_stride : row;
    if (rows_shifted(out, x, a.rows, a.xs, row)) return KDA_ERR_INVALID_ARG;
    return status_of(kda::launch_norm_fwd(a, sh->dtype == KDA_BF16, static_cast<cudaStream_t>(stream)));
}

size_t kda_layer_norm_bwd_workspace_size(const kda_norm_shape_t* sh) {
    if (norm_check(sh) != KDA_OK) return 0;
    return kda::norm_bwd_workspace_bytes(sh->rows, sh->groups, sh->D, sh->dtype == KDA_BF16);
}

kda_status_t kda_layer_norm_bwd(const kda_norm_shape_t* sh, const void* d_out, const void* x, const float* weight,
                                const float* mean, const float* rstd, void* dx, float* dweight, float* dbias,
                                void* workspace, size_t workspace_bytes, void* stream) {
    kda_status_t c = norm_check(sh);
    if (c != KDA_OK) return c;
    if (sh->rows > 0 && (!d_out || !x || !mean || !rstd || !dx)) return KDA_ERR_INVALID_ARG;
    const unsigned el = el_of(sh->dtype);
    if (!aligned(d_out, el) || !aligned(x, el) || !aligned(dx, el) || !aligned(weight, 4) || !aligned(mean, 4) ||
        !aligned(rstd, 4) || !aligned(dweight, 4) || !aligned(dbias, 4))
        return KDA_ERR_MISALIGNED;
    const bool params = dweight != nullptr || dbias != nullptr;
    const size_t need = params ? kda_layer_norm_bwd_workspace_size(sh) : 0;
    c = check_workspace(workspace, workspace_bytes, need);
    if (c != KDA_OK) return c;
    if (sh->rows == 0 && !params) return KDA_OK;
    kda::NormArgs a{};
    a.d_out = d_out; a.x = x; a.w = weight; a.mean = const_cast<float*>(mean); a.rstd = const_cast<float*>(rstd);
    a.dx = dx; a.dw = dweight; a.db = dbias;
    a.rows = sh->rows; a.G = sh->groups; a.D = sh->D;
    const long long row = (long long)sh->groups * sh->D;
    a.xs = sh->x_stride != 0 ? sh->x_stride : row;
    if (a.rows > 0 && (in_place({dx}, {weight, mean, rstd}) || one_place({dx, dweight, dbias}) || rows_shifted(dx, x, a.rows, a.xs, row)))
        return KDA_ERR_INVALID_ARG;
    return with_workspace(need ? workspace : nullptr, need, static_cast<cudaStream_t>(stream), [&](uint8_t* ws) {
        a.part = reinterpret_cast<float*>(ws);
        return kda::launch_norm_bwd(a, sh->dtype == KDA_BF16, static_cast<cudaStream_t>(stream));
    });
}

}  // extern "C"
