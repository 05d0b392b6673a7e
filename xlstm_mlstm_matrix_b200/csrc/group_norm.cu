// Group norm with an activation, channels last (contract: include/xlstm_layer.h), and its gradients.
//
//   xh = (x - mean) rstd,  z = xh w + b,  y = z act(gate)  or  act(z)
//   dz = dy act(gate)  or  dy act'(z);   dgate = dy z act'(gate);   dw = sum dz xh,  db = sum dz
//   dx = rstd (dz w - mean(dz w) - xh mean(dz w xh))
//
// Bound by memory: every tensor is read or written once, with 16-byte accesses of bf16 (two of fp32).
// A group of D <= 512 channels sits in the registers of 2 to 32 lanes, so the statistics take two
// passes over registers (mean first, then the centred squares), not over memory, and the backward forms
// them again instead of reading saved ones.  A block owns one group of channels and a range of tokens:
// weight and bias are loaded once, and the backward's sums over tokens stay in registers until the
// range ends.  Their partial sums per block are added in a fixed order by a second kernel.
#include <cmath>

#include "arg_checks.cuh"
#include "common.cuh"
#include "../../include/xlstm_layer.h"

namespace xlstm {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kV = 8;   // channels of one access per lane

struct GroupNormP {
    int B, T, G, D, heads_major, act, tokens, tokens_per_block;
    float eps;
    const void *x;
    const float *weight, *bias;
    const void *gate, *dy;
    void *y;                    // forward: y; backward: dx
    void *dgate;
    float *part_w, *part_b;     // [blocks per group][G * D], null where not asked for
};

template <typename T>
__device__ __forceinline__ void load8(const T *p, float (&r)[kV]);
template <>
__device__ __forceinline__ void load8<float>(const float *p, float (&r)[kV]) {
    const float4 a = __ldcs(reinterpret_cast<const float4 *>(p)), b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
    r[0] = a.x; r[1] = a.y; r[2] = a.z; r[3] = a.w; r[4] = b.x; r[5] = b.y; r[6] = b.z; r[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16 *p, float (&r)[kV]) {
    const uint4 u = __ldcs(reinterpret_cast<const uint4 *>(p));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r[2 * i] = __uint_as_float(w[i] << 16);
        r[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void store8(float *p, const float (&r)[kV]) {
    __stcs(reinterpret_cast<float4 *>(p), make_float4(r[0], r[1], r[2], r[3]));
    __stcs(reinterpret_cast<float4 *>(p) + 1, make_float4(r[4], r[5], r[6], r[7]));
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&r)[kV]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(r[2 * i], r[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&v);
    }
    __stcs(reinterpret_cast<uint4 *>(p), make_uint4(w[0], w[1], w[2], w[3]));
}

// Sum over the LPR lanes that share a row.
template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// e^x through the hardware's base-2 exponential: a few units of 2^-23 at these arguments; x -> inf gives 0.
__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }
__device__ __forceinline__ float act_value(int act, float x) {
    return act == XLSTM_ACT_NONE ? x : act == XLSTM_ACT_SILU ? x * sigmoid(x) : sigmoid(x);
}
// act(x) and its derivative
__device__ __forceinline__ void act_both(int act, float x, float &f, float &df) {
    if (act == XLSTM_ACT_NONE) {
        f = x; df = 1.f;
        return;
    }
    const float p = sigmoid(x);
    if (act == XLSTM_ACT_SILU) {
        f = x * p; df = p * (1.f + x * (1.f - p));
    } else {
        f = p; df = p * (1.f - p);
    }
}

// LPR lanes per row, NV accesses of kV channels per lane.
template <int LPR, int NV>
struct Lane {
    int col[NV];
    bool in[NV];
    float w[NV][kV], b[NV][kV];
    __device__ __forceinline__ Lane(const GroupNormP &p, int g) {
        const int lcol = threadIdx.x % LPR;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            col[v] = kV * (lcol + v * LPR);
            in[v] = col[v] < p.D;
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                const int c = g * p.D + col[v] + i;
                w[v][i] = in[v] && p.weight ? __ldg(p.weight + c) : 1.f;
                b[v][i] = in[v] && p.bias ? __ldg(p.bias + c) : 0.f;
            }
        }
    }
};

__device__ __forceinline__ size_t x_offset(const GroupNormP &p, int token, int g) {
    if (!p.heads_major) return ((size_t)token * p.G + g) * p.D;
    const int b = token / p.T, t = token - b * p.T;
    return (((size_t)b * p.G + g) * p.T + t) * p.D;
}

// Centres the lane's values and returns the row's rstd.
template <int LPR, int NV>
__device__ __forceinline__ float centre(const GroupNormP &p, const Lane<LPR, NV> &ln, float (&x)[NV][kV]) {
    const float inv = 1.f / (float)p.D;
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < kV; ++i) s += x[v][i];   // 0 past D
    const float mu = row_sum<LPR>(s) * inv;
    float q = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            x[v][i] = ln.in[v] ? x[v][i] - mu : 0.f;
            q = fmaf(x[v][i], x[v][i], q);
        }
    return 1.f / sqrtf(fmaf(row_sum<LPR>(q), inv, p.eps));
}

template <typename Tx, typename Ty, int LPR, int NV>
__global__ void __launch_bounds__(kThreads) group_norm_kernel(GroupNormP p) {
    constexpr int RPW = 32 / LPR, U = NV == 1 ? 2 : 1;   // rows per warp and access, rows in flight
    const int g = blockIdx.x % p.G, base = (blockIdx.x / p.G) * p.tokens_per_block;
    const int end = min(p.tokens, base + p.tokens_per_block);
    const int warp = threadIdx.x / 32, sub = (threadIdx.x % 32) / LPR;
    const Lane<LPR, NV> ln(p, g);
    const Tx *x = static_cast<const Tx *>(p.x);
    const Ty *gate = static_cast<const Ty *>(p.gate);
    Ty *y = static_cast<Ty *>(p.y);
    for (int r0 = base + warp * RPW * U; r0 < end; r0 += kWarps * RPW * U) {
        float xv[U][NV][kV], gv[U][NV][kV];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int row = r0 + u * RPW + sub;
            const size_t xo = row < end ? x_offset(p, row, g) : 0, yo = ((size_t)row * p.G + g) * p.D;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
#pragma unroll
                for (int i = 0; i < kV; ++i) xv[u][v][i] = gv[u][v][i] = 0.f;
                if (row < end && ln.in[v]) {
                    load8(x + xo + ln.col[v], xv[u][v]);
                    if (gate) load8(gate + yo + ln.col[v], gv[u][v]);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int row = r0 + u * RPW + sub;
            const float rstd = centre(p, ln, xv[u]);
            const size_t yo = ((size_t)row * p.G + g) * p.D;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                float out[kV];
#pragma unroll
                for (int i = 0; i < kV; ++i) {
                    const float z = fmaf(xv[u][v][i] * rstd, ln.w[v][i], ln.b[v][i]);
                    out[i] = gate ? z * act_value(p.act, gv[u][v][i]) : act_value(p.act, z);
                }
                if (row < end && ln.in[v]) store8(y + yo + ln.col[v], out);
            }
        }
    }
}

template <typename Tx, typename Ty, int LPR, int NV>
__global__ void __launch_bounds__(kThreads) group_norm_bwd_kernel(GroupNormP p) {
    constexpr int RPW = 32 / LPR;
    __shared__ float red[kWarps][LPR * NV * kV];
    const int g = blockIdx.x % p.G, chunk = blockIdx.x / p.G, base = chunk * p.tokens_per_block;
    const int end = min(p.tokens, base + p.tokens_per_block);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, sub = lane / LPR;
    const Lane<LPR, NV> ln(p, g);
    const Tx *x = static_cast<const Tx *>(p.x);
    const Ty *gate = static_cast<const Ty *>(p.gate), *dy = static_cast<const Ty *>(p.dy);
    Tx *dx = static_cast<Tx *>(p.y);
    Ty *dgate = static_cast<Ty *>(p.dgate);
    const float inv = 1.f / (float)p.D;
    float sw[NV][kV] = {}, sb[NV][kV] = {};
    for (int r0 = base + warp * RPW; r0 < end; r0 += kWarps * RPW) {
        const int row = r0 + sub;
        const bool live = row < end;
        const size_t xo = live ? x_offset(p, row, g) : 0, yo = ((size_t)row * p.G + g) * p.D;
        float xv[NV][kV], gv[NV][kV], dv[NV][kV];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
#pragma unroll
            for (int i = 0; i < kV; ++i) xv[v][i] = gv[v][i] = dv[v][i] = 0.f;
            if (live && ln.in[v]) {
                load8(x + xo + ln.col[v], xv[v]);
                load8(dy + yo + ln.col[v], dv[v]);
                if (gate) load8(gate + yo + ln.col[v], gv[v]);
            }
        }
        const float rstd = centre(p, ln, xv);
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                const float xh = xv[v][i] * rstd, z = fmaf(xh, ln.w[v][i], ln.b[v][i]);
                float f, df, dz;
                if (gate) {
                    act_both(p.act, gv[v][i], f, df);
                    dz = dv[v][i] * f;
                    gv[v][i] = dv[v][i] * z * df;
                } else {
                    act_both(p.act, z, f, df);
                    dz = dv[v][i] * df;
                }
                sw[v][i] = fmaf(dz, xh, sw[v][i]);
                sb[v][i] += dz;
                dz *= ln.w[v][i];
                s1 += dz;
                s2 = fmaf(dz, xh, s2);
                dv[v][i] = dz;
                xv[v][i] = xh;
            }
            if (gate && live && ln.in[v]) store8(dgate + yo + ln.col[v], gv[v]);
        }
        s1 = row_sum<LPR>(s1) * inv;
        s2 = row_sum<LPR>(s2) * inv;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float out[kV];
#pragma unroll
            for (int i = 0; i < kV; ++i) out[i] = rstd * (dv[v][i] - s1 - xv[v][i] * s2);
            if (live && ln.in[v]) store8(dx + xo + ln.col[v], out);
        }
    }
    // this block's sums over its tokens: lanes of the same columns, then warps in order
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {
        float *part = pass ? p.part_b : p.part_w;
        if (!part) continue;
        __syncthreads();
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                float s = pass ? sb[v][i] : sw[v][i];
#pragma unroll
                for (int o = LPR; o < 32; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
                if (sub == 0) red[warp][(v * LPR + lane) * kV + i] = s;
            }
        __syncthreads();
        for (int c = threadIdx.x; c < p.D; c += kThreads) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) s += red[w][c];
            part[(size_t)chunk * p.G * p.D + g * p.D + c] = s;
        }
    }
}

// dweight and dbias: the blocks' partial sums, eight interleaved runs per channel, added in a fixed order.
__global__ void __launch_bounds__(kThreads) group_norm_sums_kernel(const float *part_w, const float *part_b, float *dw,
                                                                   float *db, int chunks, int C) {
    __shared__ float red[kWarps][32];
    const float *part = blockIdx.y ? part_b : part_w;
    float *out = blockIdx.y ? db : dw;
    if (!out) return;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, c = blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < C)
        for (int k = warp; k < chunks; k += kWarps) s += part[(size_t)k * C + c];
    red[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < C) {
#pragma unroll
        for (int w = 1; w < kWarps; ++w) s += red[w][lane];
        out[c] = s;
    }
}

int lanes_per_row(int D) {
    int l = 2;
    while (l < 32 && l * kV < D) l *= 2;
    return l;
}
// Tokens of one block: at least one pass of its warps, and about `target` blocks in all.
int tokens_per_block(int tokens, int G, int D, long long target) {
    const int pass = kWarps * (32 / lanes_per_row(D));
    const long long per = ((long long)tokens * G + target - 1) / target;
    return (int)((per + pass - 1) / pass * pass);
}
constexpr long long kFwdBlocks = 148 * 16;
constexpr long long kBwdBlocks = 148 * 4;   // also bounds the partial sums

int bwd_chunks(const xlstm_group_norm_desc_t *d) {
    const int tokens = d->B * d->T, tpb = tokens_per_block(tokens, d->G, d->D, kBwdBlocks);
    return (tokens + tpb - 1) / tpb;
}

template <typename Tx, typename Ty, bool kBwd>
void launch(const GroupNormP &p, unsigned blocks, cudaStream_t s) {
#define GROUP_NORM(LPR, NV)                                                             \
    if (kBwd) group_norm_bwd_kernel<Tx, Ty, LPR, NV><<<blocks, kThreads, 0, s>>>(p);    \
    else group_norm_kernel<Tx, Ty, LPR, NV><<<blocks, kThreads, 0, s>>>(p);
    if (p.D > 256) { GROUP_NORM(32, 2) return; }
    switch (lanes_per_row(p.D)) {
        case 2: GROUP_NORM(2, 1) break;
        case 4: GROUP_NORM(4, 1) break;
        case 8: GROUP_NORM(8, 1) break;
        case 16: GROUP_NORM(16, 1) break;
        default: GROUP_NORM(32, 1) break;
    }
#undef GROUP_NORM
}
template <bool kBwd>
cudaError_t launch_any(const xlstm_group_norm_desc_t *d, const GroupNormP &p, cudaStream_t s) {
    const unsigned blocks = (unsigned)((p.tokens + p.tokens_per_block - 1) / p.tokens_per_block) * p.G;
    const bool xb = d->x_dtype == XLSTM_BF16, yb = d->y_dtype == XLSTM_BF16;
    if (xb && yb) launch<__nv_bfloat16, __nv_bfloat16, kBwd>(p, blocks, s);
    else if (xb) launch<__nv_bfloat16, float, kBwd>(p, blocks, s);
    else if (yb) launch<float, __nv_bfloat16, kBwd>(p, blocks, s);
    else launch<float, float, kBwd>(p, blocks, s);
    return cudaGetLastError();
}

bool desc_ok(const xlstm_group_norm_desc_t *d) {
    if (!d || d->B < 1 || d->T < 0 || d->G < 1 || d->D < 16 || d->D > 512 || d->D % 16) return false;
    if (d->x_dtype != XLSTM_F32 && d->x_dtype != XLSTM_BF16) return false;
    if (d->y_dtype != XLSTM_F32 && d->y_dtype != XLSTM_BF16) return false;
    if (d->x_layout != XLSTM_HEADS_MAJOR && d->x_layout != XLSTM_CHANNELS_LAST) return false;
    if (d->act < XLSTM_ACT_NONE || d->act > XLSTM_ACT_SIGMOID) return false;
    if (!(d->eps > 0.f) || !std::isfinite(d->eps)) return false;
    const long long bt = (long long)d->B * (d->T > 0 ? d->T : 1);
    // token and channel indices are 32-bit
    return bt <= (1 << 30) && bt * d->G <= (1 << 30) && (long long)d->G * d->D <= (1 << 30);
}

GroupNormP pack(const xlstm_group_norm_desc_t *d, long long blocks) {
    GroupNormP p{};
    p.B = d->B; p.T = d->T; p.G = d->G; p.D = d->D; p.heads_major = d->x_layout == XLSTM_HEADS_MAJOR;
    p.act = d->act; p.eps = d->eps; p.tokens = d->B * d->T;
    p.tokens_per_block = tokens_per_block(p.tokens, d->G, d->D, blocks);
    return p;
}

}  // namespace
}  // namespace xlstm

using namespace xlstm;

extern "C" {

xlstm_status_t xlstm_group_norm(const xlstm_group_norm_desc_t *desc, const void *x, const float *weight,
                                const float *bias, const void *gate, void *y, cudaStream_t stream) {
    if (!desc_ok(desc)) return XLSTM_ERR_INVALID_ARG;
    if (desc->T > 0 && (!x || !y)) return XLSTM_ERR_INVALID_ARG;
    for (const void *q : {x, (const void *)weight, (const void *)bias, gate, (const void *)y})
        if (!aligned16(q)) return XLSTM_ERR_INVALID_ARG;
    const size_t n = (size_t)desc->B * desc->T * desc->G * desc->D, c = (size_t)desc->G * desc->D * sizeof(float);
    const size_t ex = desc->x_dtype == XLSTM_BF16 ? 2 : 4, ey = desc->y_dtype == XLSTM_BF16 ? 2 : 4;
    const Range ins[] = {rg(x, n * ex), rg(weight, c), rg(bias, c), rg(gate, n * ey)};
    const Range outs[] = {rg(y, n * ey)};
    if (!outputs_disjoint(ins, outs)) return XLSTM_ERR_INVALID_ARG;
    if (desc->T == 0) return XLSTM_OK;
    GroupNormP p = pack(desc, kFwdBlocks);
    p.x = x; p.weight = weight; p.bias = bias; p.gate = gate; p.y = y;
    return launch_any<false>(desc, p, stream) == cudaSuccess ? XLSTM_OK : XLSTM_ERR_CUDA;
}

size_t xlstm_group_norm_bwd_workspace_size(const xlstm_group_norm_desc_t *desc) {
    if (!desc_ok(desc)) return 0;
    const size_t bytes = desc->T ? 2 * (size_t)bwd_chunks(desc) * desc->G * desc->D * sizeof(float) : 0;
    return (bytes + 255) / 256 * 256 + 256;
}

xlstm_status_t xlstm_group_norm_bwd(const xlstm_group_norm_desc_t *desc, const void *x, const float *weight,
                                    const float *bias, const void *gate, const void *dy, void *dx, void *dgate,
                                    float *dweight, float *dbias, void *workspace, size_t workspace_bytes,
                                    cudaStream_t stream) {
    if (!desc_ok(desc)) return XLSTM_ERR_INVALID_ARG;
    if (desc->T > 0 && (!x || !dy || !dx || (gate == nullptr) != (dgate == nullptr))) return XLSTM_ERR_INVALID_ARG;
    for (const void *q : {x, (const void *)weight, (const void *)bias, gate, dy, (const void *)dx, (const void *)dgate,
                          (const void *)dweight, (const void *)dbias})
        if (!aligned16(q)) return XLSTM_ERR_INVALID_ARG;
    const bool sums = dweight || dbias;
    const size_t need = sums ? xlstm_group_norm_bwd_workspace_size(desc) : 0;
    const size_t n = (size_t)desc->B * desc->T * desc->G * desc->D, C = (size_t)desc->G * desc->D;
    const size_t ex = desc->x_dtype == XLSTM_BF16 ? 2 : 4, ey = desc->y_dtype == XLSTM_BF16 ? 2 : 4;
    const Range ins[] = {rg(x, n * ex), rg(weight, C * 4), rg(bias, C * 4), rg(gate, n * ey), rg(dy, n * ey)};
    const Range outs[] = {rg(dx, n * ex), rg(dgate, n * ey), rg(dweight, C * 4), rg(dbias, C * 4), rg(workspace, need)};
    if (!outputs_disjoint(ins, outs)) return XLSTM_ERR_INVALID_ARG;
    if (sums) {
        if (!workspace || workspace_bytes < need) return XLSTM_ERR_WORKSPACE;
        if (reinterpret_cast<uintptr_t>(workspace) & 255u) return XLSTM_ERR_INVALID_ARG;
    }
    if (desc->T == 0) {
        if (dweight && cudaMemsetAsync(dweight, 0, C * 4, stream) != cudaSuccess) return XLSTM_ERR_CUDA;
        if (dbias && cudaMemsetAsync(dbias, 0, C * 4, stream) != cudaSuccess) return XLSTM_ERR_CUDA;
        return XLSTM_OK;
    }
    GroupNormP p = pack(desc, kBwdBlocks);
    const int chunks = bwd_chunks(desc);
    p.x = x; p.weight = weight; p.bias = bias; p.gate = gate; p.dy = dy; p.y = dx; p.dgate = dgate;
    float *ws = static_cast<float *>(workspace);
    p.part_w = dweight ? ws : nullptr;
    p.part_b = dbias ? ws + (size_t)chunks * C : nullptr;
    if (launch_any<true>(desc, p, stream) != cudaSuccess) return XLSTM_ERR_CUDA;
    if (sums) {
        group_norm_sums_kernel<<<dim3((unsigned)((C + 31) / 32), 2), kThreads, 0, stream>>>(p.part_w, p.part_b, dweight,
                                                                                            dbias, chunks, (int)C);
        if (cudaGetLastError() != cudaSuccess) return XLSTM_ERR_CUDA;
    }
    return XLSTM_OK;
}

}  // extern "C"
