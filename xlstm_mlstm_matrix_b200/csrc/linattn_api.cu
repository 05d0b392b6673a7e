// C ABI of the linear attention with a decay per head: argument validation.
// Declarations and the contract of every entry point: include/xlstm_layer.h.
#include <cmath>

#include "arg_checks.cuh"
#include "linattn.cuh"

namespace {

using namespace xlstm;

constexpr size_t kStatusBytes = 256;   // status block (16 B), padded

bool dims_ok(const xlstm_linattn_desc_t *d) {
    if (!d || d->B < 1 || d->H < 1 || d->T < 0) return false;
    if (d->d_qk < 16 || d->d_qk > 512 || d->d_qk % 16) return false;
    if (d->d_v < 16 || d->d_v > 512 || d->d_v % 16) return false;
    if (d->qkv_dtype != XLSTM_F32 && d->qkv_dtype != XLSTM_BF16) return false;
    if (!std::isfinite(d->scale)) return false;
    // launch grids, token and head indices are 32-bit
    const long long bh = (long long)d->B * d->H, tiles = ((long long)d->T + 63) / 64;
    return d->T <= (1 << 30) && bh * (tiles > 0 ? tiles : 1) <= (1 << 25);
}

size_t elem(const xlstm_linattn_desc_t *d) { return d->qkv_dtype == XLSTM_BF16 ? 2 : 4; }

LinAttnArgs pack(const xlstm_linattn_desc_t *d) {
    LinAttnArgs a{};
    a.B = d->B; a.H = d->H; a.T = d->T; a.dqk = d->d_qk; a.dv = d->d_v; a.dtype = d->qkv_dtype; a.scale = d->scale;
    return a;
}

// The state handed on unchanged (T = 0): zero where there was none.
xlstm_status_t pass_state(float *to, const float *from, size_t bytes, cudaStream_t s) {
    if (!to) return XLSTM_OK;
    const cudaError_t e = from ? cudaMemcpyAsync(to, from, bytes, cudaMemcpyDeviceToDevice, s)
                               : cudaMemsetAsync(to, 0, bytes, s);
    return e == cudaSuccess ? XLSTM_OK : XLSTM_ERR_CUDA;
}

xlstm_status_t check_workspace(void *ws, size_t have, size_t need) {
    if (!ws || have < need) return XLSTM_ERR_WORKSPACE;
    return (reinterpret_cast<uintptr_t>(ws) & 255u) ? XLSTM_ERR_INVALID_ARG : XLSTM_OK;
}

}  // namespace

extern "C" {

size_t xlstm_linattn_workspace_size(const xlstm_linattn_desc_t *desc) {
    return dims_ok(desc) ? kStatusBytes + linattn_workspace_bytes(pack(desc), false) : 0;
}

size_t xlstm_linattn_bwd_workspace_size(const xlstm_linattn_desc_t *desc) {
    return dims_ok(desc) ? kStatusBytes + linattn_workspace_bytes(pack(desc), true) : 0;
}

xlstm_status_t xlstm_linattn_fwd(const xlstm_linattn_desc_t *desc, const void *q, const void *k, const void *v,
                                 const float *log_decay, const int32_t *lens, const float *C_in, void *o,
                                 float *C_out, void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    if (!dims_ok(desc)) return XLSTM_ERR_INVALID_ARG;
    if (desc->T > 0 && (!q || !k || !v || !log_decay || !o)) return XLSTM_ERR_INVALID_ARG;
    for (const void *p : {q, k, v, (const void *)C_in, (const void *)o, (const void *)C_out})
        if (!aligned16(p)) return XLSTM_ERR_INVALID_ARG;
    if (!aligned4(log_decay) || !aligned4(lens)) return XLSTM_ERR_INVALID_ARG;
    const size_t BH = (size_t)desc->B * desc->H, T = (size_t)desc->T, e = elem(desc);
    const size_t sC = BH * desc->d_v * desc->d_qk * 4, need = xlstm_linattn_workspace_size(desc);
    const Range ins[] = {rg(q, BH * T * desc->d_qk * e), rg(k, BH * T * desc->d_qk * e), rg(v, BH * T * desc->d_v * e),
                         rg(log_decay, desc->H * sizeof(float)), rg(lens, desc->B * sizeof(int32_t)), rg(C_in, sC)};
    const Range outs[] = {rg(o, BH * T * desc->d_v * e), rg(C_out, sC), rg(workspace, need)};
    if (!outputs_disjoint(ins, outs)) return XLSTM_ERR_INVALID_ARG;
    const xlstm_status_t st = check_workspace(workspace, workspace_bytes, need);
    if (st != XLSTM_OK) return st;
    // the fp32 kernels have no wait that can fail, and clear the status block themselves
    if ((desc->T == 0 || desc->qkv_dtype == XLSTM_BF16) && cudaMemsetAsync(workspace, 0, 16, stream) != cudaSuccess)
        return XLSTM_ERR_CUDA;
    if (desc->T == 0) return pass_state(C_out, C_in, sC, stream);
    LinAttnArgs a = pack(desc);
    a.q = q; a.k = k; a.v = v; a.log_decay = log_decay; a.lens = lens; a.C0 = C_in; a.o = o; a.C1 = C_out;
    a.status = static_cast<int32_t *>(workspace);
    a.workspace = static_cast<char *>(workspace) + kStatusBytes;
    return launch_linattn_fwd(a, stream) == cudaSuccess ? XLSTM_OK : XLSTM_ERR_CUDA;
}

xlstm_status_t xlstm_linattn_step(const xlstm_linattn_desc_t *desc, const void *q, const void *k, const void *v,
                                  const float *log_decay, const float *C, void *o, float *C_new,
                                  cudaStream_t stream) {
    if (!desc) return XLSTM_ERR_INVALID_ARG;
    xlstm_linattn_desc_t d = *desc;
    d.T = 1;
    if (!dims_ok(&d)) return XLSTM_ERR_INVALID_ARG;
    for (const void *p : {q, k, v, (const void *)C, (const void *)o, (const void *)C_new})
        if (!p || !aligned16(p)) return XLSTM_ERR_INVALID_ARG;
    if (!log_decay || !aligned4(log_decay)) return XLSTM_ERR_INVALID_ARG;
    const size_t BH = (size_t)d.B * d.H, e = elem(&d), sC = BH * d.d_v * d.d_qk * 4;
    const Range ins[] = {rg(q, BH * d.d_qk * e), rg(k, BH * d.d_qk * e), rg(v, BH * d.d_v * e),
                         rg(log_decay, d.H * sizeof(float)), rg(C == C_new ? nullptr : C, sC)};
    const Range outs[] = {rg(o, BH * d.d_v * e), rg(C_new, sC)};
    if (!outputs_disjoint(ins, outs)) return XLSTM_ERR_INVALID_ARG;
    LinAttnArgs a = pack(&d);
    a.q = q; a.k = k; a.v = v; a.log_decay = log_decay; a.C0 = C; a.o = o; a.C1 = C_new;
    return launch_linattn_step(a, stream) == cudaSuccess ? XLSTM_OK : XLSTM_ERR_CUDA;
}

xlstm_status_t xlstm_linattn_bwd(const xlstm_linattn_desc_t *desc, const void *q, const void *k, const void *v,
                                 const float *log_decay, const int32_t *lens, const float *C_in, const void *do_,
                                 const float *dC_out, void *dq, void *dk, void *dv, float *dC_in, void *workspace,
                                 size_t workspace_bytes, cudaStream_t stream) {
    if (!dims_ok(desc)) return XLSTM_ERR_INVALID_ARG;
    if (desc->T > 0 && (!q || !k || !v || !log_decay || !do_ || !dq || !dk || !dv)) return XLSTM_ERR_INVALID_ARG;
    for (const void *p : {q, k, v, (const void *)C_in, do_, (const void *)dC_out, (const void *)dq, (const void *)dk,
                          (const void *)dv, (const void *)dC_in})
        if (!aligned16(p)) return XLSTM_ERR_INVALID_ARG;
    if (!aligned4(log_decay) || !aligned4(lens)) return XLSTM_ERR_INVALID_ARG;
    const size_t BH = (size_t)desc->B * desc->H, T = (size_t)desc->T, e = elem(desc);
    const size_t sC = BH * desc->d_v * desc->d_qk * 4, sk = BH * T * desc->d_qk * e, sv = BH * T * desc->d_v * e;
    const size_t need = xlstm_linattn_bwd_workspace_size(desc);
    const Range ins[] = {rg(q, sk), rg(k, sk), rg(v, sv), rg(log_decay, desc->H * sizeof(float)),
                         rg(lens, desc->B * sizeof(int32_t)), rg(C_in, sC), rg(do_, sv), rg(dC_out, sC)};
    const Range outs[] = {rg(dq, sk), rg(dk, sk), rg(dv, sv), rg(dC_in, sC), rg(workspace, need)};
    if (!outputs_disjoint(ins, outs)) return XLSTM_ERR_INVALID_ARG;
    const xlstm_status_t st = check_workspace(workspace, workspace_bytes, need);
    if (st != XLSTM_OK) return st;
    // the fp32 kernels have no wait that can fail, and clear the status block themselves
    if ((desc->T == 0 || desc->qkv_dtype == XLSTM_BF16) && cudaMemsetAsync(workspace, 0, 16, stream) != cudaSuccess)
        return XLSTM_ERR_CUDA;
    if (desc->T == 0) return pass_state(dC_in, dC_out, sC, stream);
    LinAttnArgs a = pack(desc);
    a.q = q; a.k = k; a.v = v; a.log_decay = log_decay; a.lens = lens; a.C0 = C_in;
    a.do_ = do_; a.dC1 = dC_out; a.dq = dq; a.dk = dk; a.dv_ = dv; a.dC0 = dC_in;
    a.status = static_cast<int32_t *>(workspace);
    a.workspace = static_cast<char *>(workspace) + kStatusBytes;
    return launch_linattn_bwd(a, stream) == cudaSuccess ? XLSTM_OK : XLSTM_ERR_CUDA;
}

}  // extern "C"
