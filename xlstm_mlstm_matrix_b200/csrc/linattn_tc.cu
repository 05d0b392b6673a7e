// Linear attention with a decay per head on the tensor cores (bf16 inputs): segment sums and output tiles.
//
// Mathematics: linattn.cuh.  Both kernels are products fed by TMA into 128-byte-swizzled shared memory,
// issued as tcgen05.mma by one thread, accumulated in tensor memory in fp32.
//
// sums_tc_kernel: U_n = sum_s w_s z_s y_s^T, 128 z rows x NX y columns per block, 64 tokens a stage.  The
//   weighted rows w_s z_s enter as a pair of bf16 (high and rest): the final state leaves in fp32, and one
//   bf16 copy of each term would leave 2^-8 of it; the pair leaves 2^-16.
// tile_tc_kernel: 128 tokens x NZ output columns per block.  X (the block's own rows) stays in shared memory;
//   Y, Z and the entering state pass through a ring of 16 KB units.  Per 128 tokens of the segment the
//   scores X Y^T land in tensor memory, eight warps weight them with powers of the decay and write them back
//   as one bf16 copy (each rounding is relative to its own term), and the product with Z accumulates on top
//   of the state's part.  The state's part is scaled by rho_t in tensor memory while the scores are formed.
//   Two blocks share an SM, so that one's products run while the other waits for its weights.
#include "linattn.cuh"
#include "linattn_tc.cuh"
#include "tma_host.cuh"

namespace xlstm {
namespace {

// Codes of the bounded waits in the status block.
enum : int {
    kWhereSumEmpty = 201, kWhereSumFull = 202, kWhereSumScaled = 203, kWhereSumDone = 204,
    kWhereTileEmpty = 211, kWhereTileX = 212, kWhereTileFull = 213, kWhereTileScores = 214, kWhereTileWeights = 215,
    kWhereTileEntry = 216, kWhereTileProduct = 217, kWhereTileDone = 218,
};

constexpr int kThreads = 320;       // TMA warp, MMA warp, eight warps of arithmetic
constexpr int kMath = 8;            // arithmetic warps
constexpr int kUnit = 16384;        // bytes of one ring unit

// ---- segment sums ------------------------------------------------------------------------------------
template <int NX>
struct SumCfg {
    static constexpr int STAGES = 2;
    static constexpr int Y_BYTES = NX * 128;
    static constexpr int STAGE = 2 * kUnit + Y_BYTES;          // high part, rest, y
    static constexpr int OFF_BAR = STAGES * STAGE;
    static constexpr int B_FULL = 0, B_EMPTY = STAGES, B_SCALED = 2 * STAGES, B_DONE = 3 * STAGES;
    static constexpr int OFF_MISC = OFF_BAR + 8 * (3 * STAGES + 1);
    static constexpr int BYTES = OFF_MISC + 16;
};

template <int NX>
__global__ void __launch_bounds__(kThreads, 2)
    sums_tc_kernel(const __grid_constant__ CUtensorMap tmz, const __grid_constant__ CUtensorMap tmy, const LinStateP p,
                   const int ztiles, const int ytiles, int32_t *status) {
    using C = SumCfg<NX>;
    extern __shared__ __align__(1024) uint8_t sm[];
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + C::OFF_BAR);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + C::OFF_MISC);
    Shared sh{reinterpret_cast<volatile int *>(sm + C::OFF_MISC + 4), status};
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int id = blockIdx.x;
    const int y0 = id % ytiles * NX; id /= ytiles;
    const int z0 = id % ztiles * 128; id /= ztiles;
    const int n = id % p.nseg, bh = id / p.nseg;
    const int len = seq_len(p.lens, bh / p.H, p.T), s0 = n * p.G, e = min(s0 + p.G, len);
    // the sum of the chain's last segment only enters the final state
    if (s0 >= len || (!p.last && (p.rev ? n == 0 : e == len))) return;
    const int steps = (e - s0 + 63) / 64;

    if (tid == 0) {
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(&bar[C::B_FULL + i], 1);
            mbar_init(&bar[C::B_EMPTY + i], 1);
            mbar_init(&bar[C::B_SCALED + i], kMath);
        }
        mbar_init(&bar[C::B_DONE], 1);
        *sh.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, NX);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = *tmem_slot;

    if (warp == 0) {
        // ===================== loads =====================
        int c = 0;
        for (; c < steps; ++c) {
            const int st = c % C::STAGES, t = s0 + 64 * c;
            if (c >= C::STAGES && !waitw(sh, &bar[C::B_EMPTY + st], (c / C::STAGES - 1) & 1, kWhereSumEmpty)) break;
            uint8_t *Zs = sm + st * C::STAGE, *Ys = Zs + 2 * kUnit;
            if (p.lens && t + 64 > len) {
                const int rows = len - t;
                for (int b = 0; b < 2; ++b)
                    load_box_rows<64>(Zs + 8192 * b, static_cast<const __nv_bfloat16 *>(p.z) + ((size_t)bh * p.T + t) * p.dv,
                                      p.dv, rows, z0 + 64 * b, lane);
                for (int b = 0; b < NX / 64; ++b)
                    load_box_rows<64>(Ys + 8192 * b, static_cast<const __nv_bfloat16 *>(p.y) + ((size_t)bh * p.T + t) * p.dqk,
                                      p.dqk, rows, y0 + 64 * b, lane);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[C::B_FULL + st]);
            } else if (lane == 0) {
                mbar_arrive_expect_tx(&bar[C::B_FULL + st], kUnit + C::Y_BYTES);
                for (int b = 0; b < 2; ++b) tma_load_3d(Zs + 8192 * b, &tmz, &bar[C::B_FULL + st], z0 + 64 * b, t, bh);
                for (int b = 0; b < NX / 64; ++b)
                    tma_load_3d(Ys + 8192 * b, &tmy, &bar[C::B_FULL + st], y0 + 64 * b, t, bh);
            }
            __syncwarp();
        }
        // every copy issued lands before shared memory is released
        if (lane == 0)
            for (int st = 0; st < C::STAGES; ++st)
                if (c > st) drain_wait(&bar[C::B_FULL + st], ((c - 1 - st) / C::STAGES) & 1);
    } else if (warp == 1) {
        // ===================== products =====================
        if (lane == 0) {
            constexpr uint32_t id_u = make_idesc(128, NX, kFmtBF16, kFmtBF16, 1, 1);
            for (int c = 0; c < steps; ++c) {
                const int st = c % C::STAGES;
                if (!wait1(sh, &bar[C::B_SCALED + st], (c / C::STAGES) & 1, kWhereSumScaled)) break;
                tc_fence_after();
                const uint32_t base = smem_u32(sm + st * C::STAGE);
                const uint64_t hi = smem_desc_sw128(base, 8192, 1024), lo = smem_desc_sw128(base + kUnit, 8192, 1024);
                const uint64_t y = smem_desc_sw128(base + 2 * kUnit, 8192, 1024);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) {
                    const uint32_t k = ks * 2048 >> 4;
                    mma_f16_ss(tm, hi + k, y + k, id_u, c > 0 || ks > 0);
                    mma_f16_ss(tm, lo + k, y + k, id_u, 1);
                }
                tc_commit(&bar[C::B_EMPTY + st]);
            }
            tc_commit(&bar[C::B_DONE]);     // also with nothing in flight: the read-out waits for it
            drain_wait(&bar[C::B_DONE], 0);
        }
    } else {
        // ===================== weights, read-out =====================
        const int t256 = tid - 64;
        const float ld = head_log_decay(p.log_decay, bh % p.H);
        bool alive = true;
        for (int c = 0; c < steps; ++c) {
            const int st = c % C::STAGES;
            if (!waitw(sh, &bar[C::B_FULL + st], (c / C::STAGES) & 1, kWhereSumFull)) {
                alive = false;
                break;
            }
            uint8_t *Zs = sm + st * C::STAGE;
            // 16-byte chunks t256 + 256 i: token (t256 / 8) of the lower half, or 32 further
            float w[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int s = s0 + 64 * c + t256 / 8 + 32 * i;
                w[i] = s < e ? (p.rev ? p.scale * decay_pow(ld, s - s0 + 1) : decay_pow(ld, e - 1 - s)) : 0.f;
            }
            uint4 u[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) u[i] = *reinterpret_cast<const uint4 *>(Zs + 16 * (t256 + 256 * i));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint4 hi, lo;
                split_scaled(u[i], w[i & 1], hi, lo);
                *reinterpret_cast<uint4 *>(Zs + 16 * (t256 + 256 * i)) = hi;
                *reinterpret_cast<uint4 *>(Zs + kUnit + 16 * (t256 + 256 * i)) = lo;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[C::B_SCALED + st]);
        }
        alive = alive && waitw(sh, &bar[C::B_DONE], 0, kWhereSumDone) && !*sh.abort_flag;
        if (__all_sync(0xffffffffu, alive)) {
            tc_fence_after();
            const int quarter = warp & 3, half = (warp - 2) >> 2, r = z0 + 32 * quarter + lane;
            float *U = p.sums + ((size_t)bh * p.nseg + n) * p.dv * p.dqk + (size_t)r * p.dqk;
            constexpr int CH = NX / 2;     // columns of this warp
#pragma unroll 1
            for (int c = 0; c < CH; c += 32) {
                float x[32];
                tmem_ld32(tm + ((uint32_t)(32 * quarter) << 16) + half * CH + c, x);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    const int col = y0 + half * CH + c + i;
                    if (r < p.dv && col < p.dqk)
                        *reinterpret_cast<float4 *>(U + col) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
                }
            }
            tc_fence_before();
        }
    }
    __syncthreads();
    __syncwarp();
    if (warp == 1) tmem_dealloc(tm, NX);
}

// ---- output tiles ---------------------------------------------------------------------------------------
struct TileBars {   // indices into the barrier array
    static constexpr int X = 0, SCORES = 8, WEIGHTS = 9, PRODUCT = 10, ENTRY = 11, DONE = 12, RING = 13;   // RING: full, empty per stage
};
constexpr int kMaxStages = 7;
constexpr int kTileTail = 132 * 4 + (TileBars::RING + 2 * kMaxStages) * 8 + 16;   // table, barriers, slots

template <int NZ>
__global__ void __launch_bounds__(kThreads, 2)
    tile_tc_kernel(const __grid_constant__ CUtensorMap tmx, const __grid_constant__ CUtensorMap tmy,
                   const __grid_constant__ CUtensorMap tmz, const __grid_constant__ CUtensorMap tms,
                   const __grid_constant__ CUtensorMap tmo, const LinTileP p, const int ttiles, const int ztiles,
                   const int nkx, const int stages, int32_t *status) {
    extern __shared__ __align__(1024) uint8_t sm[];
    uint8_t *ring = sm + nkx * kUnit;
    float *tab = reinterpret_cast<float *>(ring + stages * kUnit);
    uint64_t *bar = reinterpret_cast<uint64_t *>(tab + 132);
    uint64_t *full = bar + TileBars::RING, *empty = full + stages;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(empty + stages);
    Shared sh{reinterpret_cast<volatile int *>(tmem_slot + 1), status};
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int id = blockIdx.x;
    const int z0 = id % ztiles * NZ; id /= ztiles;
    const int t0 = id % ttiles * 128, bh = id / ttiles;
    const int len = seq_len(p.lens, bh / p.H, p.T);
    if (t0 >= len) {   // behind the sequence: zeros
        __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out) + ((size_t)bh * p.T + t0) * p.dz;
        for (int i = tid; i < 128 * (NZ / 8); i += kThreads) {
            const int r = i / (NZ / 8), c = z0 + i % (NZ / 8) * 8;
            if (t0 + r < p.T && c < p.dz) *reinterpret_cast<uint4 *>(out + (size_t)r * p.dz + c) = make_uint4(0, 0, 0, 0);
        }
        return;
    }
    const int n = t0 / p.G, s0 = n * p.G, e = min(s0 + p.G, len);
    const float ld = head_log_decay(p.log_decay, bh % p.H);
    const bool entry = p.rev ? (e < len || p.has_init) : (n > 0 || p.has_init);
    // 128-token score tiles on this tile's past (future) side, its own first
    const int nj = p.rev ? (e - t0 + 127) / 128 : (t0 - s0) / 128 + 1;
    const int dir = p.rev ? 128 : -128;

    if (tid == 0) {
        for (int i = 0; i < nkx; ++i) mbar_init(&bar[TileBars::X + i], 1);
        mbar_init(&bar[TileBars::SCORES], 1);
        mbar_init(&bar[TileBars::WEIGHTS], kMath);
        mbar_init(&bar[TileBars::PRODUCT], 1);
        mbar_init(&bar[TileBars::ENTRY], 1);
        mbar_init(&bar[TileBars::DONE], 1);
        for (int i = 0; i < stages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        *sh.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, 256);
        tmem_relinquish();
    }
    // column c of a score tile at distance d tiles carries l^(128 (d - 1)) times tab[c] times the row's power
    for (int i = tid; i <= 128; i += kThreads) tab[i] = decay_pow(ld, p.rev ? i : 128 - i);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = *tmem_slot, tm_s = tm + 128;

    if (warp == 0) {
        // ===================== loads =====================
        int u = 0, xs = 0;  // ring units and chunks of X issued
        auto slot_free = [&](int st) {
            return u < stages || waitw(sh, &empty[st], (u / stages - 1) & 1, kWhereTileEmpty);
        };
        auto y_tile = [&](int j, bool with_x) {
            for (int c = 0; c < nkx; ++c) {
                if (with_x) {
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&bar[TileBars::X + c], kUnit);
                        tma_load_3d(sm + c * kUnit, &tmx, &bar[TileBars::X + c], 64 * c, t0, bh);
                    }
                    ++xs;
                }
                const int st = u % stages;
                if (!slot_free(st)) return false;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&full[st], kUnit);
                    tma_load_3d(ring + st * kUnit, &tmy, &full[st], 64 * c, t0 + j * dir, bh);
                }
                ++u;
            }
            return true;
        };
        auto entry_state = [&]() {
            const int slot = bh * p.nseg + n;
            for (int c = 0; c < nkx; ++c) {
                const int st = u % stages;
                if (!slot_free(st)) return false;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&full[st], NZ * 128);
                    if (p.state_t)
                        for (int b = 0; b < NZ / 64; ++b)
                            tma_load_3d(ring + st * kUnit + 8192 * b, &tms, &full[st], z0 + 64 * b, 64 * c, slot);
                    else
                        tma_load_3d(ring + st * kUnit, &tms, &full[st], 64 * c, z0, slot);
                }
                ++u;
            }
            return true;
        };
        auto z_tile = [&](int j) {
            constexpr int R = NZ == 128 ? 64 : 128;     // tokens of a unit
            for (int h = 0; h < 128 / R; ++h) {
                const int st = u % stages, t = t0 + j * dir + R * h;
                if (!slot_free(st)) return false;
                if (p.lens && t + R > len) {
                    // the tile the sequence ends in: rows behind its end read as zeros, whatever is there
                    for (int b = 0; b < NZ / 64; ++b)
                        load_box_rows<R>(ring + st * kUnit + 8192 * b,
                                         static_cast<const __nv_bfloat16 *>(p.z) + ((size_t)bh * p.T + t) * p.dz, p.dz,
                                         len - t, z0 + 64 * b, lane);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&full[st]);
                } else if (lane == 0) {
                    mbar_arrive_expect_tx(&full[st], kUnit);
                    for (int b = 0; b < NZ / 64; ++b)
                        tma_load_3d(ring + st * kUnit + 8192 * b, &tmz, &full[st], z0 + 64 * b, t, bh);
                }
                ++u;
            }
            return true;
        };
        bool go = y_tile(0, true);
        if (go && entry) go = entry_state();
        if (go) go = z_tile(0);
        for (int j = 1; go && j < nj; ++j) go = y_tile(j, false) && z_tile(j);
        __syncwarp();
        if (lane == 0) {
            // every copy issued lands before shared memory is released
            for (int st = 0; st < stages; ++st)
                if (u > st) drain_wait(&full[st], ((u - 1 - st) / stages) & 1);
            for (int c = 0; c < xs; ++c) drain_wait(&bar[TileBars::X + c], 0);
        }
    } else if (warp == 1) {
        // ===================== products =====================
        if (lane == 0) {
            constexpr uint32_t id_s = make_idesc(128, 128, kFmtBF16, kFmtBF16, 0, 0);
            constexpr uint32_t id_pz = make_idesc(128, NZ, kFmtBF16, kFmtBF16, 0, 1);
            const uint32_t id_e = make_idesc(128, NZ, kFmtBF16, kFmtBF16, 0, p.state_t);
            const uint64_t x = smem_desc_sw128(smem_u32(sm), 16, 1024);
            int u = 0;
            bool go = true;
            auto unit = [&](uint32_t &addr) {      // waits for the next ring unit
                const int st = u % stages;
                if (!wait1(sh, &full[st], (u / stages) & 1, kWhereTileFull)) return false;
                tc_fence_after();
                addr = smem_u32(ring + st * kUnit);
                return true;
            };
            auto release = [&]() { tc_commit(&empty[u++ % stages]); };
            for (int j = 0; go && j < nj; ++j) {
                // the weighted scores of the tile before share the columns
                if (j > 0 && !wait1(sh, &bar[TileBars::PRODUCT], (j - 1) & 1, kWhereTileProduct)) { go = false; break; }
                for (int c = 0; go && c < nkx; ++c) {
                    uint32_t a;
                    go = (j > 0 || wait1(sh, &bar[TileBars::X + c], 0, kWhereTileX)) && unit(a);
                    if (!go) break;
                    const uint64_t y = smem_desc_sw128(a, 16, 1024);
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        mma_f16_ss(tm_s, x + (uint32_t)((c * kUnit + 32 * ks) >> 4), y + 2 * ks, id_s, c > 0 || ks > 0);
                    release();
                }
                if (!go) break;
                tc_commit(&bar[TileBars::SCORES]);
                if (j == 0 && entry) {
                    for (int c = 0; go && c < nkx; ++c) {
                        uint32_t a;
                        if (!(go = unit(a))) break;
                        const uint64_t s = p.state_t ? smem_desc_sw128(a, 8192, 1024) : smem_desc_sw128(a, 16, 1024);
                        const uint32_t step = p.state_t ? 2048 >> 4 : 2;
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            mma_f16_ss(tm, x + (uint32_t)((c * kUnit + 32 * ks) >> 4), s + ks * step, id_e, c > 0 || ks > 0);
                        release();
                    }
                    if (!go) break;
                    tc_commit(&bar[TileBars::ENTRY]);
                }
                if (!(go = wait1(sh, &bar[TileBars::WEIGHTS], j & 1, kWhereTileWeights))) break;
                tc_fence_after();
                constexpr int R = NZ == 128 ? 64 : 128;
#pragma unroll
                for (int h = 0; h < 128 / R; ++h) {
                    uint32_t a;
                    if (!(go = unit(a))) break;
                    const uint64_t z = smem_desc_sw128(a, 8192, 1024);
#pragma unroll
                    for (int ks = 0; ks < R / 16; ++ks) {
                        const int k = h * (R / 16) + ks;     // 16 tokens: 8 packed columns, 64 apart per half tile
                        mma_f16_ts(tm, tm_s + 64 * (k / 4) + 8 * (k % 4), z + (uint32_t)(ks * 2048 >> 4), id_pz,
                                   entry || j > 0 || k > 0);
                    }
                    release();
                }
                if (go) tc_commit(&bar[TileBars::PRODUCT]);
            }
            tc_commit(&bar[TileBars::DONE]);
            drain_wait(&bar[TileBars::DONE], 0);
        }
    } else {
        // ===================== weights, read-out =====================
        const int quarter = warp & 3, half = (warp - 2) >> 2, r = 32 * quarter + lane, t = t0 + r;
        const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
        bool alive = true;
        for (int j = 0; j < nj; ++j) {
            if (!waitw(sh, &bar[TileBars::SCORES], j & 1, kWhereTileScores)) {
                alive = false;
                break;
            }
            tc_fence_after();
            const int cols = p.rev ? min(128, e - (t0 + 128 * j)) : 128;     // live columns
            // what the row contributes: scale times its power of the decay
            const float f = j == 0 ? p.scale
                                   : p.scale * decay_pow(ld, 128 * (j - 1) + (p.rev ? 128 - r : r));
            const int lo = j == 0 && p.rev ? r : 0, hi = j == 0 && !p.rev ? r + 1 : cols;
#pragma unroll
            for (int c0 = 0; c0 < 64; c0 += 32) {
                float x[32];
                tmem_ld32(tm_s + lanes + 64 * half + c0, x);
                tmem_wait_ld();
                const int c1 = 64 * half + c0;
                if (j > 0 && cols == 128) {
                    const float2 f2 = make_float2(f, f);
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        const float4 w = *reinterpret_cast<const float4 *>(tab + c1 + i);
                        const float2 a = __fmul2_rn(__fmul2_rn(make_float2(x[i], x[i + 1]), f2), make_float2(w.x, w.y));
                        const float2 b = __fmul2_rn(__fmul2_rn(make_float2(x[i + 2], x[i + 3]), f2), make_float2(w.z, w.w));
                        x[i] = a.x; x[i + 1] = a.y; x[i + 2] = b.x; x[i + 3] = b.y;
                    }
                } else {
                    // masked columns are selected away, not multiplied: their scores may be anything
                    const int off = j > 0 ? 0 : p.rev ? -r : 128 - r;
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const int c = c1 + i;
                        const float w = tab[min(max(c + off, 0), 128)];
                        x[i] = c >= lo && c < hi ? x[i] * f * w : 0.f;
                    }
                }
                uint32_t pk[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) pk[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
                tmem_st16(tm_s + lanes + 64 * half + c0 / 2, pk);
            }
            if (j == 0 && entry) {
                if (!waitw(sh, &bar[TileBars::ENTRY], 0, kWhereTileEntry)) {
                    alive = false;
                    break;
                }
                tc_fence_after();
                const float rho = p.rev ? decay_pow(ld, max(e - 1 - t, 0)) : p.scale * decay_pow(ld, t - s0 + 1);
#pragma unroll
                for (int c0 = 0; c0 < NZ / 2; c0 += 32) {
                    float x[32];
                    tmem_ld32(tm + lanes + half * (NZ / 2) + c0, x);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) x[i] *= rho;
                    tmem_st32(tm + lanes + half * (NZ / 2) + c0, x);
                }
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[TileBars::WEIGHTS]);
        }
        alive = alive && waitw(sh, &bar[TileBars::DONE], 0, kWhereTileDone) && !*sh.abort_flag;
        const bool ok = __all_sync(0xffffffffu, alive);
        // every load and product is done: the ring's first units stage the output for the TMA store
        if (ok) {
            tc_fence_after();
#pragma unroll
            for (int c0 = 0; c0 < NZ / 2; c0 += 32) {
                float x[32];
                tmem_ld32(tm + lanes + half * (NZ / 2) + c0, x);
                tmem_wait_ld();
                const int col = half * (NZ / 2) + c0;
                uint8_t *box = ring + (col / 64) * kUnit;
#pragma unroll
                for (int i = 0; i < 32; i += 8) {
                    uint4 v = make_uint4(pack_bf16x2(x[i], x[i + 1]), pack_bf16x2(x[i + 2], x[i + 3]),
                                         pack_bf16x2(x[i + 4], x[i + 5]), pack_bf16x2(x[i + 6], x[i + 7]));
                    if (t >= len) v = make_uint4(0, 0, 0, 0);
                    *reinterpret_cast<uint4 *>(box + sw128_offset(r, (col % 64 + i) / 8)) = v;
                }
            }
            tc_fence_before();
            fence_proxy_async_smem();
        }
        named_barrier(1, 32 * kMath);
        if (tid == 64 && ok) {
            for (int b = 0; b < NZ / 64; ++b)
                if (z0 + 64 * b < p.dz) tma_store_3d(&tmo, ring + b * kUnit, z0 + 64 * b, t0, bh);
            tma_store_wait();
        }
    }
    __syncthreads();
    __syncwarp();
    if (warp == 1) tmem_dealloc(tm, 256);
}

// ---- launches -----------------------------------------------------------------------------------------------
template <int NX>
cudaError_t sums_nx(const LinStateP &p, int32_t *status, cudaStream_t s) {
    using C = SumCfg<NX>;
    const uint64_t BH = (uint64_t)p.B * p.H;
    CUtensorMap tmz, tmy;
    if (!make_tmap_3d_bf16(&tmz, p.z, p.dv, p.T, BH, 64, 64) || !make_tmap_3d_bf16(&tmy, p.y, p.dqk, p.T, BH, 64, 64))
        return cudaErrorInvalidValue;
    const int zt = (p.dv + 127) / 128, yt = (p.dqk + NX - 1) / NX;
    cudaError_t e = cudaFuncSetAttribute(sums_tc_kernel<NX>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::BYTES);
    if (e != cudaSuccess) return e;
    sums_tc_kernel<NX><<<(unsigned)(BH * p.nseg * zt * yt), kThreads, C::BYTES, s>>>(tmz, tmy, p, zt, yt, status);
    return cudaGetLastError();
}

template <int NZ>
cudaError_t tile_nz(const LinTileP &p, int32_t *status, cudaStream_t s) {
    const uint64_t BH = (uint64_t)p.B * p.H;
    const int nkx = (p.dx + 63) / 64, tt = (p.T + 127) / 128, zt = (p.dz + NZ - 1) / NZ;
    // two blocks per SM where the block's own rows leave room for three units
    const int room = nkx <= 4 ? 7 : 14, stages = room - nkx < kMaxStages ? room - nkx : kMaxStages;
    CUtensorMap tmx, tmy, tmz, tms, tmo;
    constexpr int R = NZ == 128 ? 64 : 128;
    const bool ok =
        make_tmap_3d_bf16(&tmx, p.x, p.dx, p.T, BH, 64, 128) && make_tmap_3d_bf16(&tmy, p.y, p.dx, p.T, BH, 64, 128) &&
        make_tmap_3d_bf16(&tmz, p.z, p.dz, p.T, BH, 64, R) && make_tmap_3d_bf16(&tmo, p.out, p.dz, p.T, BH, 64, 128) &&
        (p.state_t ? make_tmap_3d_bf16(&tms, p.states, p.dz, p.dx, BH * p.nseg, 64, 64)
                   : make_tmap_3d_bf16(&tms, p.states, p.dx, p.dz, BH * p.nseg, 64, NZ));
    if (!ok) return cudaErrorInvalidValue;
    const int smem = (nkx + stages) * kUnit + kTileTail;
    cudaError_t e = cudaFuncSetAttribute(tile_tc_kernel<NZ>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    tile_tc_kernel<NZ><<<(unsigned)(BH * tt * zt), kThreads, smem, s>>>(tmx, tmy, tmz, tms, tmo, p, tt, zt, nkx, stages,
                                                                        status);
    return cudaGetLastError();
}

}  // namespace

cudaError_t linattn_sums_tc(const LinStateP &p, int32_t *status, cudaStream_t s) {
    return p.dqk > 64 ? sums_nx<128>(p, status, s) : sums_nx<64>(p, status, s);
}
cudaError_t linattn_tile_tc(const LinTileP &p, int32_t *status, cudaStream_t s) {
    return p.dz > 64 ? tile_nz<128>(p, status, s) : tile_nz<64>(p, status, s);
}

}  // namespace xlstm
