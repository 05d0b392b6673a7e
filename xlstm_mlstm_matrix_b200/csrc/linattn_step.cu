// One token of the linear attention with a decay per head: C' = l C + v k^T, o = scale C' q.
//
// Bound by the state's bytes: d_v x d_qk fp32 per head are read and written once (128 x 8 heads of 256 x 512: 172 to 184 us,
// 5.9 to 6.3 TB/s).  A block owns a range
// of rows of one head; the lanes of a warp cover whole rows with 16-byte accesses, all loads of a lane's
// rows issued before any is used.
#include "linattn.cuh"

namespace xlstm {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 2;   // rows a lane holds in flight

struct StepP {
    int H, dqk, dv, rows_per_block;
    float scale;
    const void *q, *k, *v;
    const float *log_decay, *C;
    void *o;
    float *C1;
};

__device__ __forceinline__ void put(float *p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

// NC: float4 columns per lane and row.
template <typename T, int NC>
__global__ void __launch_bounds__(kThreads) linattn_step_kernel(const __grid_constant__ StepP p) {
    wait_for_stream();
    const int G = p.dqk >> 2;                                        // float4s of a row
    const int LG = (G <= 32 && (G & (G - 1)) == 0) ? G : 32;         // lanes per row
    const int RW = 32 / LG;                                          // rows per warp and pass
    const int bh = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int lrow = lane / LG, lcol = lane % LG;
    const T *q = static_cast<const T *>(p.q) + (size_t)bh * p.dqk;
    const T *k = static_cast<const T *>(p.k) + (size_t)bh * p.dqk;
    const T *v = static_cast<const T *>(p.v) + (size_t)bh * p.dv;
    const float4 *C = reinterpret_cast<const float4 *>(p.C) + (size_t)bh * p.dv * G;
    float4 *C1 = reinterpret_cast<float4 *>(p.C1) + (size_t)bh * p.dv * G;
    T *o = static_cast<T *>(p.o) + (size_t)bh * p.dv;
    const float l = decay_pow(head_log_decay(p.log_decay, bh % p.H), 1);
    float4 qv[NC], kv[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int j = 4 * (lcol + c * LG);
        const bool in = j < p.dqk;
        qv[c] = in ? make_float4(to_f32(q[j]), to_f32(q[j + 1]), to_f32(q[j + 2]), to_f32(q[j + 3]))
                   : make_float4(0.f, 0.f, 0.f, 0.f);
        kv[c] = in ? make_float4(to_f32(k[j]), to_f32(k[j + 1]), to_f32(k[j + 2]), to_f32(k[j + 3]))
                   : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const int r_begin = blockIdx.y * p.rows_per_block, r_end = min(p.dv, r_begin + p.rows_per_block);
    for (int r0 = r_begin + warp * RW * kRows; r0 < r_end; r0 += (kThreads / 32) * RW * kRows) {
        float4 cv[kRows][NC];
        float vr[kRows], acc[kRows];
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            const int r = r0 + u * RW + lrow;
            vr[u] = r < r_end ? to_f32(v[r]) : 0.f;
            acc[u] = 0.f;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int j4 = lcol + c * LG;
                cv[u][c] = (r < r_end && j4 < G) ? __ldcs(C + (size_t)r * G + j4) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            const int r = r0 + u * RW + lrow;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int j4 = lcol + c * LG;
                float4 n;
                n.x = fmaf(l, cv[u][c].x, vr[u] * kv[c].x);
                n.y = fmaf(l, cv[u][c].y, vr[u] * kv[c].y);
                n.z = fmaf(l, cv[u][c].z, vr[u] * kv[c].z);
                n.w = fmaf(l, cv[u][c].w, vr[u] * kv[c].w);
                if (r < r_end && j4 < G) __stcs(C1 + (size_t)r * G + j4, n);
                acc[u] += n.x * qv[c].x + n.y * qv[c].y + n.z * qv[c].z + n.w * qv[c].w;
            }
        }
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            float s = acc[u];
            for (int d = LG >> 1; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
            const int r = r0 + u * RW + lrow;
            if (lcol == 0 && r < r_end) put(o + r, p.scale * s);
        }
    }
}

}  // namespace

cudaError_t launch_linattn_step(const LinAttnArgs &a, cudaStream_t s) {
    StepP p;
    p.H = a.H; p.dqk = a.dqk; p.dv = a.dv; p.scale = a.scale;
    p.q = a.q; p.k = a.k; p.v = a.v; p.log_decay = a.log_decay; p.C = a.C0; p.o = a.o; p.C1 = a.C1;
    // rows are independent, so a head splits over blocks, in place too: eight blocks per SM while a block
    // keeps 16 rows (64 x 8 heads of 128 x 128: 19.5 us; with two per SM 21.1, with 32 20.5)
    const long long BH = (long long)a.B * a.H, target = 8LL * sm_count();
    int split = 1;
    while (BH * split < target && a.dv / (split * 2) >= 16) split *= 2;
    p.rows_per_block = (a.dv + split - 1) / split;
    const dim3 grid((unsigned)BH, split);
    const int G = a.dqk / 4, LG = (G <= 32 && (G & (G - 1)) == 0) ? G : 32, nc = (G + LG - 1) / LG;
#define LINATTN_STEP(NCV)                                                            \
    if (nc == NCV)                                                                                             \
        return launch_early(a.dtype == XLSTM_BF16 ? linattn_step_kernel<__nv_bfloat16, NCV>                    \
                                                  : linattn_step_kernel<float, NCV>, grid, kThreads, 0, s, p);
    LINATTN_STEP(1) LINATTN_STEP(2) LINATTN_STEP(3) LINATTN_STEP(4)
#undef LINATTN_STEP
    return cudaErrorInvalidValue;
}

}  // namespace xlstm
