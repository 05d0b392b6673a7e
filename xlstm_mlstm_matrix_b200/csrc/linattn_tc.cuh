// Device pieces of the tensor-core linear attention beside sm100.cuh and tc_common.cuh.
#pragma once
#include "tc_common.cuh"

namespace xlstm {
namespace {

// Stores a 3-D tile from 128-byte-swizzled shared memory; what lies past the tensor's extents is dropped.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap *m, const void *src, int x, int y, int z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(m)),
                 "r"(smem_u32(src)), "r"(x), "r"(y), "r"(z)
                 : "memory");
}
// Waits until this thread's stores have read their shared memory.
__device__ __forceinline__ void tma_store_wait() {
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}

// One warp brings R rows x 64 columns of a row-major bf16 matrix (ncols wide, from column col0) into a
// swizzled box, zeros at and past row `rows` and past the last column: for the tile a sequence ends in,
// where a TMA copy would bring what lies behind its end.
template <int R>
__device__ __noinline__ void load_box_rows(uint8_t *box, const __nv_bfloat16 *src, int ncols, int rows, int col0,
                                           int lane) {
#pragma unroll 1
    for (int e0 = 0; e0 < R * 8; e0 += 256) {
        uint4 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int e = e0 + 32 * i + lane, r = e >> 3, col = col0 + 8 * (e & 7);
            v[i] = make_uint4(0, 0, 0, 0);
            if (r < rows && col < ncols) v[i] = __ldg(reinterpret_cast<const uint4 *>(src + (size_t)r * ncols + col));
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int e = e0 + 32 * i + lane;
            *reinterpret_cast<uint4 *>(box + sw128_offset(e >> 3, e & 7)) = v[i];
        }
    }
}

// w times eight bf16 values as a pair of bf16: hi = round(w v), lo = round(w v - hi).
__device__ __forceinline__ void split_scaled(const uint4 &u, float w, uint4 &hi, uint4 &lo) {
    const uint32_t in[4] = {u.x, u.y, u.z, u.w};
    uint32_t h[4], l[4];
    const float2 w2 = make_float2(w, w);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = __fmul2_rn(bf16x2_to_float2(in[i]), w2);
        h[i] = pack_bf16x2(x.x, x.y);
        const float2 f = bf16x2_to_float2(h[i]);
        l[i] = pack_bf16x2(x.x - f.x, x.y - f.y);
    }
    hi = make_uint4(h[0], h[1], h[2], h[3]);
    lo = make_uint4(l[0], l[1], l[2], l[3]);
}

}  // namespace
}  // namespace xlstm
