// Linear attention with a decay per head on fp32 CUDA cores: the state sums and the output
// tiles of fp32 inputs, and the chain over segments of both kernel families.
//
// Mathematics: linattn.cuh.  fp32 inputs promise fp32 results, which tensor-core products of
// fp32 operands reach only as three or more split products; these kernels hold every operand,
// product and sum in fp32 instead.
#include "linattn.cuh"

namespace xlstm {
namespace {

constexpr int kThreads = 256;
constexpr int kPad = 68;      // row pitch of the transposed 64-wide tiles (4-float aligned, spreads banks)
constexpr int kK = 32;        // inner-product columns staged at a time

__device__ __forceinline__ float4 load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ void store4(float *p, float4 x) { *reinterpret_cast<float4 *>(p) = x; }
__device__ __forceinline__ void store4(__nv_bfloat16 *p, float4 x) {
    __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
    *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<uint32_t *>(&a), *reinterpret_cast<uint32_t *>(&b));
}

// 64 rows x kK columns of a row-major matrix (nrows x ncols, rows `pitch` apart) into dst[column][row];
// zeros outside it.
__device__ __forceinline__ void stage_cols(float *dst, const float *src, size_t pitch, int nrows, int col0, int ncols) {
#pragma unroll
    for (int i = 0; i < 64 * kK / 4 / kThreads; ++i) {
        const int e = threadIdx.x + i * kThreads, r = e & 63, c = (e >> 6) * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < nrows && col0 + c < ncols) x = load4(src + (size_t)r * pitch + col0 + c);
        dst[(c + 0) * kPad + r] = x.x;
        dst[(c + 1) * kPad + r] = x.y;
        dst[(c + 2) * kPad + r] = x.z;
        dst[(c + 3) * kPad + r] = x.w;
    }
}
// kK rows x W columns into dst[row][column]; zeros outside.
template <int W>
__device__ __forceinline__ void stage_rows(float *dst, const float *src, size_t pitch, int nrows, int col0, int ncols) {
#pragma unroll
    for (int i = 0; i < kK * W / 4 / kThreads; ++i) {
        const int e = threadIdx.x + i * kThreads, r = e / (W / 4), c = (e % (W / 4)) * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < nrows && col0 + c < ncols) x = load4(src + (size_t)r * pitch + col0 + c);
        *reinterpret_cast<float4 *>(dst + r * W + c) = x;
    }
}

// acc[n][i][j] += sum_k a[k][4 ty + i] b[k][64 n + 4 tx + j]
template <int N>
__device__ __forceinline__ void tile_fma(float (&acc)[N][4][4], const float *a, int lda, const float *b, int ldb, int ty,
                                         int tx) {
#pragma unroll 4
    for (int k = 0; k < kK; ++k) {
        const float4 av = *reinterpret_cast<const float4 *>(a + k * lda + 4 * ty);
        const float ar[4] = {av.x, av.y, av.z, av.w};
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const float4 bv = *reinterpret_cast<const float4 *>(b + k * ldb + 64 * n + 4 * tx);
            const float br[4] = {bv.x, bv.y, bv.z, bv.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[n][i][j] = fmaf(ar[i], br[j], acc[n][i][j]);
        }
    }
}

// ---- U_n = sum_s w_s z_s y_s^T of one segment, 64 z rows x 64 N y columns per block ------------------
template <int N>
__global__ void __launch_bounds__(kThreads) sums_kernel(LinStateP p, int ztiles, int ytiles) {
    __shared__ __align__(16) float Zs[kK * 64];
    __shared__ __align__(16) float Ys[kK * 64 * N];
    __shared__ float ws[kK];
    int id = blockIdx.x;
    const int yt = id % ytiles; id /= ytiles;
    const int zt = id % ztiles; id /= ztiles;
    const int n = id % p.nseg, bh = id / p.nseg;
    const int len = seq_len(p.lens, bh / p.H, p.T), s0 = n * p.G, e = min(s0 + p.G, len);
    if (s0 >= len) return;
    const float ld = head_log_decay(p.log_decay, bh % p.H);
    const int tid = threadIdx.x, ty = tid / 16, tx = tid % 16;
    const int z0 = zt * 64, y0 = yt * 64 * N;
    const float *z = static_cast<const float *>(p.z) + (size_t)bh * p.T * p.dv;
    const float *y = static_cast<const float *>(p.y) + (size_t)bh * p.T * p.dqk;
    float acc[N][4][4] = {};
    for (int s = s0; s < e; s += kK) {
        const int rows = min(kK, e - s);
        __syncthreads();
        if (tid < kK)
            ws[tid] = tid < rows ? (p.rev ? p.scale * decay_pow(ld, s + tid - s0 + 1) : decay_pow(ld, e - 1 - s - tid))
                                 : 0.f;
        stage_rows<64>(Zs, z + (size_t)s * p.dv, p.dv, rows, z0, p.dv);
        stage_rows<64 * N>(Ys, y + (size_t)s * p.dqk, p.dqk, rows, y0, p.dqk);
        __syncthreads();
        for (int i = tid; i < kK * 64; i += kThreads) Zs[i] *= ws[i / 64];
        __syncthreads();
        tile_fma<N>(acc, Zs, 64, Ys, 64 * N, ty, tx);
    }
    float *U = p.sums + ((size_t)bh * p.nseg + n) * p.dv * p.dqk;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < N; ++c) {
            const int r = z0 + 4 * ty + i, col = y0 + 64 * c + 4 * tx;
            if (r < p.dv && col < p.dqk)
                store4(U + (size_t)r * p.dqk + col,
                       make_float4(acc[c][i][0], acc[c][i][1], acc[c][i][2], acc[c][i][3]));
        }
}

// ---- the chain over segments: states[n] = the state entering segment n; last = the state it ends in ----
// One thread carries four elements of a head's state through all segments; states may be the sums' own
// memory (each element is read before it is written).  The factor l^{e_n-s_n} is held as two floats: over a
// thousand segments one rounded factor would drift the oldest tokens' weight by a thousand of its roundings.
template <typename S>
__global__ void __launch_bounds__(kThreads) chain_kernel(LinStateP p, int per_head) {
    const int bh = blockIdx.x / per_head;
    const size_t area = (size_t)p.dv * p.dqk;
    const size_t el = ((size_t)(blockIdx.x % per_head) * kThreads + threadIdx.x) * 4;
    if (el >= area) return;
    const int len = seq_len(p.lens, bh / p.H, p.T), nseg = (len + p.G - 1) / p.G;
    const float ld = head_log_decay(p.log_decay, bh % p.H);
    const float *U = p.sums + (size_t)bh * p.nseg * area + el;
    S *out = static_cast<S *>(p.states) + (size_t)bh * p.nseg * area + el;
    float4 c = p.init ? load4(p.init + (size_t)bh * area + el) : make_float4(0.f, 0.f, 0.f, 0.f);
    const double full = exp((double)ld * p.G), tail = exp((double)ld * (len - (nseg - 1) * p.G));
    constexpr int kAhead = 8;   // sums in flight
    for (int i0 = 0; i0 < nseg; i0 += kAhead) {
        float4 u[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int n = p.rev ? nseg - 1 - (i0 + i) : i0 + i;
            u[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            // the last segment's sum only enters the final state
            if (i0 + i < nseg && (i0 + i + 1 < nseg || p.last)) u[i] = load4(U + (size_t)n * area);
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (i0 + i >= nseg) break;
            const int n = p.rev ? nseg - 1 - (i0 + i) : i0 + i;
            store4(out + (size_t)n * area, c);
            const double f = n == nseg - 1 ? tail : full;
            const float hi = (float)f, lo = (float)(f - (double)hi);
            c.x = fmaf(c.x, hi, fmaf(c.x, lo, u[i].x));
            c.y = fmaf(c.y, hi, fmaf(c.y, lo, u[i].y));
            c.z = fmaf(c.z, hi, fmaf(c.z, lo, u[i].z));
            c.w = fmaf(c.w, hi, fmaf(c.w, lo, u[i].w));
        }
    }
    if (p.last) store4(p.last + (size_t)bh * area + el, c);
}

// ---- output tiles: 64 tokens x 64 N columns per block ---------------------------------------------------
template <int N>
__global__ void __launch_bounds__(kThreads) tile_kernel(LinTileP p, int ttiles, int ztiles) {
    extern __shared__ __align__(16) float sm[];
    float *Xs = sm;                    // [kK][kPad]
    float *Ys = Xs + kK * kPad;        // [kK][kPad]
    float *Ps = Ys + kK * kPad;        // [64][kPad]: weighted scores, token s by token t
    float *Zs = Ps + 64 * kPad;        // [kK][64 N]
    float *pw = Zs + kK * 64 * N;      // l^0 .. l^G
    int id = blockIdx.x;
    const int zt = id % ztiles; id /= ztiles;
    const int tt = id % ttiles, bh = id / ttiles;
    const int len = seq_len(p.lens, bh / p.H, p.T), t0 = tt * 64, z0 = zt * 64 * N;
    const int tid = threadIdx.x, ty = tid / 16, tx = tid % 16;
    float *out = static_cast<float *>(p.out) + (size_t)bh * p.T * p.dz;
    float acc[N][4][4] = {};
    if (t0 < len) {
        const float ld = head_log_decay(p.log_decay, bh % p.H);
        const int n = t0 / p.G, s0 = n * p.G, e = min(s0 + p.G, len);
        for (int i = tid; i <= p.G; i += kThreads) pw[i] = decay_pow(ld, i);
        const float *x = static_cast<const float *>(p.x) + ((size_t)bh * p.T + t0) * p.dx;
        const float *y = static_cast<const float *>(p.y) + (size_t)bh * p.T * p.dx;
        const float *z = static_cast<const float *>(p.z) + (size_t)bh * p.T * p.dz;
        const int xrows = min(64, len - t0);
        __syncthreads();
        // the entering state's part
        const bool entry = p.rev ? (e < len || p.has_init) : (n > 0 || p.has_init);
        if (entry) {
            const float *M = static_cast<const float *>(p.states) + ((size_t)bh * p.nseg + n) * p.dx * p.dz;
            for (int k0 = 0; k0 < p.dx; k0 += kK) {
                __syncthreads();
                stage_cols(Xs, x, p.dx, xrows, k0, p.dx);
                if (p.state_t) {
                    stage_rows<64 * N>(Zs, M + (size_t)k0 * p.dz, p.dz, min(kK, p.dx - k0), z0, p.dz);
                    __syncthreads();
                    tile_fma<N>(acc, Xs, kPad, Zs, 64 * N, ty, tx);
                } else {
                    // [dz][dx]: 64 state rows at a time through the transposed tile
#pragma unroll
                    for (int c = 0; c < N; ++c) {
                        if (c) __syncthreads();
                        const int r0 = z0 + 64 * c;
                        stage_cols(Ys, M + (size_t)r0 * p.dx, p.dx, p.dz - r0, k0, p.dx);
                        __syncthreads();
                        float part[1][4][4];
#pragma unroll
                        for (int i = 0; i < 16; ++i) part[0][i / 4][i % 4] = acc[c][i / 4][i % 4];
                        tile_fma<1>(part, Xs, kPad, Ys, kPad, ty, tx);
#pragma unroll
                        for (int i = 0; i < 16; ++i) acc[c][i / 4][i % 4] = part[0][i / 4][i % 4];
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = t0 + 4 * ty + i;
                const float rho = t < len ? (p.rev ? pw[e - 1 - t] : p.scale * pw[t - s0 + 1]) : 0.f;
#pragma unroll
                for (int c = 0; c < N; ++c)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[c][i][j] *= rho;
            }
        }
        // the segment's own tokens on the causal (or, reversed, the later) side
        const int first = p.rev ? t0 : s0, stop = p.rev ? e : min(t0 + 64, e);
        for (int b0 = first; b0 < stop; b0 += 64) {
            const int yrows = min(64, e - b0);
            float sc[1][4][4] = {};
            for (int k0 = 0; k0 < p.dx; k0 += kK) {
                __syncthreads();
                stage_cols(Xs, x, p.dx, xrows, k0, p.dx);
                stage_cols(Ys, y + (size_t)b0 * p.dx, p.dx, yrows, k0, p.dx);
                __syncthreads();
                tile_fma<1>(sc, Xs, kPad, Ys, kPad, ty, tx);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int t = t0 + 4 * ty + i, s = b0 + 4 * tx + j, far = p.rev ? s - t : t - s;
                    Ps[(4 * tx + j) * kPad + 4 * ty + i] =
                        (far >= 0 && s < e && t < e) ? p.scale * pw[far] * sc[0][i][j] : 0.f;
                }
            for (int k0 = 0; k0 < 64; k0 += kK) {
                __syncthreads();
                stage_rows<64 * N>(Zs, z + (size_t)(b0 + k0) * p.dz, p.dz, yrows - k0, z0, p.dz);
                __syncthreads();
                tile_fma<N>(acc, Ps + k0 * kPad, kPad, Zs, 64 * N, ty, tx);
            }
        }
    }
    // rows at or past the sequence's end hold zeros
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = t0 + 4 * ty + i;
        if (t >= p.T) continue;
#pragma unroll
        for (int c = 0; c < N; ++c) {
            const int col = z0 + 64 * c + 4 * tx;
            if (col < p.dz)
                store4(out + (size_t)t * p.dz + col,
                       t < len ? make_float4(acc[c][i][0], acc[c][i][1], acc[c][i][2], acc[c][i][3])
                               : make_float4(0.f, 0.f, 0.f, 0.f));
        }
    }
}

int wide(int d) { return d > 128 ? 4 : d > 64 ? 2 : 1; }

template <int N>
cudaError_t tile_n(const LinTileP &p, cudaStream_t s) {
    const int tt = (p.T + 63) / 64, zt = (p.dz + 64 * N - 1) / (64 * N);
    const size_t smem = sizeof(float) * (2 * kK * kPad + 64 * kPad + kK * 64 * N + p.G + 1);
    cudaError_t e = cudaFuncSetAttribute(tile_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    tile_kernel<N><<<(unsigned)((size_t)p.B * p.H * tt * zt), kThreads, smem, s>>>(p, tt, zt);
    return cudaGetLastError();
}

}  // namespace

cudaError_t linattn_sums_simt(const LinStateP &p, cudaStream_t s) {
    const int N = wide(p.dqk), zt = (p.dv + 63) / 64, yt = (p.dqk + 64 * N - 1) / (64 * N);
    const unsigned blocks = (unsigned)((size_t)p.B * p.H * p.nseg * zt * yt);
    if (N == 1) sums_kernel<1><<<blocks, kThreads, 0, s>>>(p, zt, yt);
    else if (N == 2) sums_kernel<2><<<blocks, kThreads, 0, s>>>(p, zt, yt);
    else sums_kernel<4><<<blocks, kThreads, 0, s>>>(p, zt, yt);
    return cudaGetLastError();
}

cudaError_t linattn_tile_simt(const LinTileP &p, cudaStream_t s) {
    const int N = wide(p.dz);
    return N == 1 ? tile_n<1>(p, s) : N == 2 ? tile_n<2>(p, s) : tile_n<4>(p, s);
}

cudaError_t linattn_chain(const LinStateP &p, bool bf16, cudaStream_t s) {
    const int per_head = (int)(((size_t)p.dv * p.dqk / 4 + kThreads - 1) / kThreads);
    const unsigned blocks = (unsigned)((size_t)p.B * p.H * per_head);
    if (bf16) chain_kernel<__nv_bfloat16><<<blocks, kThreads, 0, s>>>(p, per_head);
    else chain_kernel<float><<<blocks, kThreads, 0, s>>>(p, per_head);
    return cudaGetLastError();
}

}  // namespace xlstm
