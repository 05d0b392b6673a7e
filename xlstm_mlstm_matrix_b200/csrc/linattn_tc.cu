// Linear attention with a decay per head on the tensor cores (bf16 inputs): segment sums and output tiles.
//
// Mathematics: linattn.cuh.  Both kernels are products fed by TMA into 128-byte-swizzled shared memory,
// issued as tcgen05.mma by one thread, accumulated in tensor memory in fp32.
//
// state_tc_kernel: U_n = sum_s w_s z_s y_s^T, 128 z rows x NX y columns per block, 32 tokens a stage, chained over
//   the segments where there are blocks enough.  The weighted rows w_s z_s enter as three bf16 parts: the final state
//   leaves in fp32, one part would leave 2^-8 of each term and two 2^-16.
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
    kWhereSumEmpty = 201, kWhereSumFull = 202, kWhereSumScaled = 203, kWhereSumDone = 204, kWhereSumTaken = 205, kWhereSumParts = 206,
    kWhereTileEmpty = 211, kWhereTileX = 212, kWhereTileFull = 213, kWhereTileScores = 214, kWhereTileWeights = 215,
    kWhereTileEntry = 216, kWhereTileProduct = 217, kWhereTileDone = 218,
};

constexpr int kThreads = 320;       // TMA warp, MMA warp, eight warps of arithmetic
constexpr int kMath = 8;            // arithmetic warps
constexpr int kUnit = 16384;        // bytes of one ring unit

// ---- entering states -----------------------------------------------------------------------------------
// SEQ: a block carries one 128 x NX tile of a head's state through all segments and stores it at each segment's
// entry; the state lives in the fold warps' registers in fp32, the sum of the next segment grows in the other half of
// tensor memory meanwhile.  Sums start from zero in every segment: the tensor core's accumulation truncates, and over a
// whole sequence in one accumulator that would bias the state by one step of 2^-24 per 16 tokens.
// SUM (too few tiles to fill the GPU): blocks take single segments and store their sums for the chain kernel.
constexpr int kStep = 32;                // tokens of one stage
constexpr int kPart = 128 * kStep * 2;   // one part of the weighted rows: 8 KB

template <int NX, bool SEQ>
struct StateCfg {
    // NX = 256: the state and the sum fill tensor memory, and the products wait while a sum is folded in.  NX <= 128: the
    // state lives in registers, and two sums take turns.
    static constexpr bool IN_TMEM = NX == 256;
    static constexpr int ACCS = IN_TMEM ? 1 : 2;
    // Loads run this many stages ahead (about 2000 cycles of latency against 400 to 800 of products a stage).
    static constexpr int STAGES = IN_TMEM ? 4 : 6, PARTS = IN_TMEM || !(SEQ || NX == 64) ? 2 : 3;
    static constexpr int Y_BYTES = NX * kStep * 2;
    static constexpr int STAGE = kPart + Y_BYTES;               // z and y as they come
    static constexpr int OFF_PARTS = STAGES * STAGE, PARTS_BYTES = 3 * kPart;
    static constexpr int OFF_OUT = OFF_PARTS + PARTS * PARTS_BYTES;
    static constexpr int OUT = 128 * NX * (SEQ ? 2 : 4);        // what a store leaves from
    static constexpr int OFF_BAR = OFF_OUT + OUT;
    static constexpr int B_FULL = 0, B_EMPTY = STAGES, B_SCALED = 2 * STAGES, B_ACC = 3 * STAGES, B_TAKEN = B_ACC + 2,
                         B_LAST = B_TAKEN + 2;
    static constexpr int OFF_MISC = OFF_BAR + 8 * (B_LAST + 1);
    static constexpr int BYTES = OFF_MISC + 16;
    static constexpr int STATE = NX;                            // state's first column (IN_TMEM)
    static constexpr int COLS = 2 * NX;
};
constexpr int kStateThreads = 640;       // TMA, MMA, two idle warps; two groups of four warps of weights; eight fold warps
constexpr int kFold = 384;               // first thread of the fold warps

// One tile's walk over its segments, the same in every role.
struct StateWalk {
    int bh, z0, y0, len, nseg, nm;       // segments of the sequence, and those whose sum is formed
    int first;                           // SUM: the block's only segment
};
template <int NX, bool SEQ>
__device__ __forceinline__ StateWalk state_walk(const LinStateP &p, int item, int ztiles, int ytiles) {
    StateWalk w;
    w.y0 = item % ytiles * NX; item /= ytiles;
    w.z0 = item % ztiles * 128; item /= ztiles;
    w.first = 0;
    if (!SEQ) { w.first = item % p.nseg; item /= p.nseg; }
    w.bh = item;
    w.len = seq_len(p.lens, item / p.H, p.T);
    w.nseg = (w.len + p.G - 1) / p.G;
    // the sum of the chain's last segment only enters the final state
    if (SEQ) w.nm = p.last ? w.nseg : w.nseg - 1;
    else w.nm = w.first < w.nseg && (p.last || w.first != (p.rev ? 0 : w.nseg - 1)) ? 1 : 0;
    return w;
}
// The k-th segment in chain order.
template <bool SEQ>
__device__ __forceinline__ int segment_of(const LinStateP &p, const StateWalk &w, int k) {
    return !SEQ ? w.first : p.rev ? w.nseg - 1 - k : k;
}

template <int NX, bool SEQ>
__global__ void __launch_bounds__(kStateThreads, 1)
    state_tc_kernel(const __grid_constant__ CUtensorMap tmz, const __grid_constant__ CUtensorMap tmy,
                    const __grid_constant__ CUtensorMap tmo, const __grid_constant__ LinStateP p, const int items,
                    const int ztiles, const int ytiles, int32_t *status) {
    using C = StateCfg<NX, SEQ>;
    extern __shared__ __align__(1024) uint8_t sm[];
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + C::OFF_BAR);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + C::OFF_MISC);
    Shared sh{reinterpret_cast<volatile int *>(sm + C::OFF_MISC + 4), status};
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(&bar[C::B_FULL + i], 1);
            mbar_init(&bar[C::B_EMPTY + i], 1);
            mbar_init(&bar[C::B_SCALED + i], 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar[C::B_ACC + i], 1);
            mbar_init(&bar[C::B_TAKEN + i], 8);
        }
        mbar_init(&bar[C::B_LAST], 1);
        *sh.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, C::COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = *tmem_slot;

    if (warp < 4) {
        if (warp == 0) {
            // ===================== loads =====================
            int c = 0;          // stages issued
            bool go = true;
            for (int item = blockIdx.x; go && item < items; item += gridDim.x) {
                const StateWalk w = state_walk<NX, SEQ>(p, item, ztiles, ytiles);
                for (int k = 0; go && k < w.nm; ++k) {
                    const int s0 = segment_of<SEQ>(p, w, k) * p.G, e = min(s0 + p.G, w.len);
                    for (int t = s0; t < e; t += kStep, ++c) {
                        const int st = c % C::STAGES;
                        if (c >= C::STAGES && !waitw(sh, &bar[C::B_EMPTY + st], (c / C::STAGES - 1) & 1, kWhereSumEmpty)) {
                            go = false;
                            break;
                        }
                        uint8_t *Zs = sm + st * C::STAGE, *Ys = Zs + kPart;
                        if (p.lens && t + kStep > w.len) {
                            for (int b = 0; b < 2; ++b)
                                load_box_rows<kStep>(Zs + 4096 * b,
                                                     static_cast<const __nv_bfloat16 *>(p.z) + ((size_t)w.bh * p.T + t) * p.dv,
                                                     p.dv, w.len - t, w.z0 + 64 * b, lane);
                            for (int b = 0; b < NX / 64; ++b)
                                load_box_rows<kStep>(Ys + 4096 * b,
                                                     static_cast<const __nv_bfloat16 *>(p.y) + ((size_t)w.bh * p.T + t) * p.dqk,
                                                     p.dqk, w.len - t, w.y0 + 64 * b, lane);
                            fence_proxy_async_smem();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&bar[C::B_FULL + st]);
                        } else if (lane == 0) {
                            mbar_arrive_expect_tx(&bar[C::B_FULL + st], kPart + C::Y_BYTES);
                            for (int b = 0; b < 2; ++b)
                                tma_load_3d(Zs + 4096 * b, &tmz, &bar[C::B_FULL + st], w.z0 + 64 * b, t, w.bh);
                            for (int b = 0; b < NX / 64; ++b)
                                tma_load_3d(Ys + 4096 * b, &tmy, &bar[C::B_FULL + st], w.y0 + 64 * b, t, w.bh);
                        }
                        __syncwarp();
                    }
                }
            }
            // every copy issued lands before shared memory is released
            if (lane == 0)
                for (int st = 0; st < C::STAGES; ++st)
                    if (c > st) drain_wait(&bar[C::B_FULL + st], ((c - 1 - st) / C::STAGES) & 1);
        } else if (warp == 1 && lane == 0) {
            // ===================== products =====================
            constexpr uint32_t id_u = make_idesc(128, NX, kFmtBF16, kFmtBF16, 1, 1);
            int c = 0, g = 0;   // stages consumed, segments summed
            bool go = true;
            for (int item = blockIdx.x; go && item < items; item += gridDim.x) {
                const StateWalk w = state_walk<NX, SEQ>(p, item, ztiles, ytiles);
                for (int k = 0; go && k < w.nm; ++k, ++g) {
                    const int s0 = segment_of<SEQ>(p, w, k) * p.G, e = min(s0 + p.G, w.len);
                    const uint32_t acc = tm + g % C::ACCS * NX;
                    if (g >= C::ACCS && !wait1(sh, &bar[C::B_TAKEN + g % C::ACCS], (g / C::ACCS - 1) & 1, kWhereSumTaken)) {
                        go = false;
                        break;
                    }
                    for (int t = s0; t < e; t += kStep, ++c) {
                        const int st = c % C::STAGES;
                        if (!wait1(sh, &bar[C::B_SCALED + st], (c / C::STAGES) & 1, kWhereSumScaled)) {
                            go = false;
                            break;
                        }
                        tc_fence_after();
                        const uint64_t z = smem_desc_sw128(smem_u32(sm + C::OFF_PARTS + c % C::PARTS * C::PARTS_BYTES), 4096, 1024);
                        const uint64_t y = smem_desc_sw128(smem_u32(sm + st * C::STAGE + kPart), 4096, 1024);
#pragma unroll
                        for (int ks = 0; ks < kStep / 16; ++ks)
#pragma unroll
                            for (int part = 0; part < 3; ++part)
                                mma_f16_ss(acc, z + (uint32_t)((part * kPart + ks * 2048) >> 4), y + (uint32_t)(ks * 2048 >> 4),
                                           id_u, t > s0 || ks > 0 || part > 0);
                        tc_commit(&bar[C::B_EMPTY + st]);
                    }
                    if (go) tc_commit(&bar[C::B_ACC + g % C::ACCS]);
                }
            }
            tc_commit(&bar[C::B_LAST]);     // nothing in flight when tensor memory is freed
            drain_wait(&bar[C::B_LAST], 0);
        }
    } else if (warp < 12) {
        // ===================== weights =====================
        // the two groups take every other stage
        const int t128 = tid & 127, group = (warp - 4) >> 2;
        int c = 0;
        bool go = true;
        for (int item = blockIdx.x; go && item < items; item += gridDim.x) {
            const StateWalk w = state_walk<NX, SEQ>(p, item, ztiles, ytiles);
            const float ld = head_log_decay(p.log_decay, w.bh % p.H);
            for (int k = 0; go && k < w.nm; ++k) {
                const int s0 = segment_of<SEQ>(p, w, k) * p.G, e = min(s0 + p.G, w.len);
                for (int t = s0; t < e; t += kStep, ++c) {
                    const int st = c % C::STAGES;
                    if ((c & 1) != group) continue;
                    // 16-byte chunks t128 + 128 i: token t128 / 8 of the upper half, or 16 further
                    float wt[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int s = t + t128 / 8 + 16 * i;
                        wt[i] = s < e ? (p.rev ? p.scale * decay_pow(ld, s - s0 + 1) : decay_pow(ld, e - 1 - s)) : 0.f;
                    }
                    if (!waitw(sh, &bar[C::B_FULL + st], (c / C::STAGES) & 1, kWhereSumFull)) {
                        go = false;
                        break;
                    }
                    const uint8_t *Zs = sm + st * C::STAGE;
                    uint8_t *parts = sm + C::OFF_PARTS + c % C::PARTS * C::PARTS_BYTES;
                    uint4 u[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) u[i] = *reinterpret_cast<const uint4 *>(Zs + 16 * (t128 + 128 * i));
                    // the products of the stage PARTS ago have read the parts' place
                    if (c >= C::PARTS && !waitw(sh, &bar[C::B_EMPTY + (c - C::PARTS) % C::STAGES],
                                                ((c - C::PARTS) / C::STAGES) & 1, kWhereSumParts)) {
                        go = false;
                        break;
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint4 part[3];
                        split_scaled(u[i], wt[i & 1], part);
#pragma unroll
                        for (int q = 0; q < 3; ++q)
                            *reinterpret_cast<uint4 *>(parts + q * kPart + 16 * (t128 + 128 * i)) = part[q];
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar[C::B_SCALED + st]);
                }
            }
        }
    } else {
        // ===================== fold =====================
        const int quarter = warp & 3, half = (warp - 12) >> 2, r = 32 * quarter + lane;
        constexpr int CH = NX / 2;      // columns of this thread
        const uint32_t own_tm = tm + ((uint32_t)(32 * quarter) << 16) + half * CH;
        uint8_t *out = sm + C::OFF_OUT;
        int g = 0;
        bool go = true, staged = false;
        // The thread that stores waits for its last store before the block writes the staging memory again.
        auto staging_free = [&]() {
            if (staged && tid == kFold) tma_store_wait();
            staged = true;
            named_barrier(1, 256);
        };
        auto store = [&](int slot, int z0, int y0) {
            fence_proxy_async_smem();
            named_barrier(1, 256);
            constexpr int W = SEQ ? 64 : 32;    // columns of a box
            if (tid == kFold) {
                for (int b = 0; b < NX / W; ++b)
                    if (y0 + W * b < p.dqk) tma_store_3d(&tmo, out + b * 16384, y0 + W * b, z0, slot);
                tma_store_commit();
            }
        };
        for (int item = blockIdx.x; go && item < items; item += gridDim.x) {
            const StateWalk w = state_walk<NX, SEQ>(p, item, ztiles, ytiles);
            if (SEQ) {
                const float ld = head_log_decay(p.log_decay, w.bh % p.H);
                const float4 f = decay_factors(ld, p.G, w.len - (w.nseg - 1) * p.G);
                const size_t own = ((size_t)w.bh * p.dv + w.z0 + r) * p.dqk + w.y0 + half * CH;   // this thread's columns
                const bool row = w.z0 + r < p.dv;
                const auto inside = [&](int i) { return row && w.y0 + half * CH + i < p.dqk; };
                // the state, 32 columns at a time: registers, or this thread's lane of tensor memory
                constexpr int KEPT = C::IN_TMEM ? 1 : CH / 32;
                float x[KEPT][32];
#pragma unroll
                for (int c0 = 0; c0 < CH; c0 += 32) {
                    float(&v)[32] = x[c0 / 32 % KEPT];
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        float4 u = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (p.init && inside(c0 + i)) u = *reinterpret_cast<const float4 *>(p.init + own + c0 + i);
                        v[i] = u.x; v[i + 1] = u.y; v[i + 2] = u.z; v[i + 3] = u.w;
                    }
                    if (C::IN_TMEM) tmem_st32(own_tm + C::STATE + c0, v);
                }
                if (C::IN_TMEM) tmem_wait_st();
                for (int k = 0; go && k < w.nseg; ++k) {
                    const int n = segment_of<SEQ>(p, w, k);
                    if (k > 0 || p.init) {      // the state entering segment n
                        staging_free();
#pragma unroll
                        for (int c0 = 0; c0 < CH; c0 += 32) {
                            float(&v)[32] = x[c0 / 32 % KEPT];
                            if (C::IN_TMEM) {
                                tmem_ld32(own_tm + C::STATE + c0, v);
                                tmem_wait_ld();
                            }
#pragma unroll
                            for (int i = 0; i < 32; i += 8) {
                                const int col = half * CH + c0 + i;
                                *reinterpret_cast<uint4 *>(out + (col / 64) * 16384 + sw128_offset(r, (col % 64) / 8)) =
                                    make_uint4(pack_bf16x2(v[i], v[i + 1]), pack_bf16x2(v[i + 2], v[i + 3]),
                                               pack_bf16x2(v[i + 4], v[i + 5]), pack_bf16x2(v[i + 6], v[i + 7]));
                            }
                        }
                        store(w.bh * p.nseg + n, w.z0, w.y0);
                    }
                    if (k >= w.nm) break;
                    if (!waitw(sh, &bar[C::B_ACC + g % C::ACCS], (g / C::ACCS) & 1, kWhereSumDone)) {
                        go = false;
                        break;
                    }
                    tc_fence_after();
                    const float hi = n == w.nseg - 1 ? f.z : f.x, lo = n == w.nseg - 1 ? f.w : f.y;
#pragma unroll
                    for (int c0 = 0; c0 < CH; c0 += 32) {
                        float(&v)[32] = x[c0 / 32 % KEPT];
                        if (C::IN_TMEM) tmem_ld32(own_tm + C::STATE + c0, v);
#pragma unroll
                        for (int c1 = 0; c1 < 32; c1 += 16) {
                            float u[16];
                            tmem_ld16(own_tm + g % C::ACCS * NX + c0 + c1, u);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 16; ++i) v[c1 + i] = fmaf(v[c1 + i], hi, fmaf(v[c1 + i], lo, u[i]));
                        }
                        if (C::IN_TMEM) tmem_st32(own_tm + C::STATE + c0, v);
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar[C::B_TAKEN + g % C::ACCS]);
                    if (C::IN_TMEM) tmem_wait_st();
                    ++g;
                }
                if (go && p.last) {
#pragma unroll
                    for (int c0 = 0; c0 < CH; c0 += 32) {
                        float(&v)[32] = x[c0 / 32 % KEPT];
                        if (C::IN_TMEM) {
                            tmem_ld32(own_tm + C::STATE + c0, v);
                            tmem_wait_ld();
                        }
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            if (inside(c0 + i))
                                *reinterpret_cast<float4 *>(p.last + own + c0 + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                    }
                }
            } else if (w.nm) {
                if (!waitw(sh, &bar[C::B_ACC + g % C::ACCS], (g / C::ACCS) & 1, kWhereSumDone)) {
                    go = false;
                    break;
                }
                tc_fence_after();
                staging_free();
#pragma unroll
                for (int c0 = 0; c0 < CH; c0 += 32) {
                    float u[32];
                    tmem_ld32(own_tm + g % C::ACCS * NX + c0, u);
                    tmem_wait_ld();
                    uint8_t *box = out + ((half * CH + c0) / 32) * 16384;
#pragma unroll
                    for (int i = 0; i < 32; i += 4)
                        *reinterpret_cast<float4 *>(box + sw128_offset(r, i / 4)) = make_float4(u[i], u[i + 1], u[i + 2], u[i + 3]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[C::B_TAKEN + g % C::ACCS]);
                ++g;
                store(w.bh * p.nseg + w.first, w.z0, w.y0);
            }
        }
        if (tid == kFold) tma_store_wait();
    }
    __syncthreads();
    __syncwarp();
    if (warp == 1) tmem_dealloc(tm, C::COLS);
}

// ---- output tiles ---------------------------------------------------------------------------------------
struct TileBars {   // indices into the barrier array
    static constexpr int X = 0, SCORES = 8, WEIGHTS = 9, PRODUCT = 10, ENTRY = 11, DONE = 12, RING = 13;   // RING: full, empty per stage
};
constexpr int kMaxStages = 7;
constexpr int kTab = 32 + 132 + 32;     // powers of the decay, room for masked columns on both sides
constexpr int kTileTail = kTab * 4 + (TileBars::RING + 2 * kMaxStages) * 8 + 16;   // table, barriers, slots
static_assert(7 * kUnit + kTileTail <= 113 * 1024, "two blocks share an SM");

template <int NZ>
__global__ void __launch_bounds__(kThreads, 2)
    tile_tc_kernel(const __grid_constant__ CUtensorMap tmx, const __grid_constant__ CUtensorMap tmy,
                   const __grid_constant__ CUtensorMap tmz, const __grid_constant__ CUtensorMap tms,
                   const __grid_constant__ CUtensorMap tmo, const LinTileP p, const int ttiles, const int ztiles,
                   const int nkx, const int stages, int32_t *status) {
    extern __shared__ __align__(1024) uint8_t sm[];
    uint8_t *ring = sm + nkx * kUnit;
    float *tab = reinterpret_cast<float *>(ring + stages * kUnit) + 32;
    uint64_t *bar = reinterpret_cast<uint64_t *>(tab + kTab - 32);
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
        // the first loads need no one else: they are on their way while the block sets itself up
        for (int c = 0; c < nkx; ++c) {
            mbar_arrive_expect_tx(&bar[TileBars::X + c], kUnit);
            tma_load_3d(sm + c * kUnit, &tmx, &bar[TileBars::X + c], 64 * c, t0, bh);
            if (c < stages) {
                mbar_arrive_expect_tx(&full[c], kUnit);
                tma_load_3d(ring + c * kUnit, &tmy, &full[c], 64 * c, t0, bh);
            }
        }
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, 256);
        tmem_relinquish();
    }
    // column c of a score tile at distance d tiles carries l^(128 (d - 1)) times tab[c] times the row's power
    for (int i = tid - 32; i < kTab - 32; i += kThreads)
        tab[i] = i >= 0 && i <= 128 ? decay_pow(ld, p.rev ? i : 128 - i) : 0.f;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = *tmem_slot, tm_s = tm + 128;

    if (warp == 0) {
        // ===================== loads =====================
        int u = min(nkx, stages);   // ring units issued
        auto slot_free = [&](int st) {
            return u < stages || waitw(sh, &empty[st], (u / stages - 1) & 1, kWhereTileEmpty);
        };
        auto y_tile = [&](int j) {
            for (int c = j ? 0 : u; c < nkx; ++c) {
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
        bool go = y_tile(0);
        if (go && entry) go = entry_state();
        if (go) go = z_tile(0);
        for (int j = 1; go && j < nj; ++j) go = y_tile(j) && z_tile(j);
        __syncwarp();
        if (lane == 0) {
            // every copy issued lands before shared memory is released
            for (int st = 0; st < stages; ++st)
                if (u > st) drain_wait(&full[st], ((u - 1 - st) / stages) & 1);
            for (int c = 0; c < nkx; ++c) drain_wait(&bar[TileBars::X + c], 0);
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
            // Blocks of 32 columns against this warp's 32 rows.  Where all columns are on the past (future) side, a
            // weight is the row's power times the column's; on the diagonal it is looked up by distance; masked
            // scores are selected away, not multiplied, for they may be anything.
#pragma unroll 1
            for (int b = 0; b < 2; ++b) {
                const int cb = 2 * half + b, c1 = 32 * cb, d = j > 0 ? 1 : p.rev ? cb - quarter : quarter - cb;
                const uint32_t from = tm_s + lanes + c1, to = tm_s + lanes + 64 * half + 16 * b;
                uint32_t pk[16];
                if (d < 0) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) pk[i] = 0;
                    tmem_st16(to, pk);
                    continue;
                }
                float x[32];
                tmem_ld32(from, x);
                float f = p.scale;
                if (j > 0) f *= decay_pow(ld, 128 * (j - 1) + (p.rev ? 128 - r : r));
                else if (d > 0) f *= decay_pow(ld, p.rev ? c1 - r : r - c1 - 32);
                tmem_wait_ld();
                if (d > 0 && c1 + 32 <= cols) {
                    const float4 *w4 = reinterpret_cast<const float4 *>(tab + (j > 0 ? c1 : p.rev ? 0 : 96));
                    const float2 f2 = make_float2(f, f);
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        const float4 w = w4[i / 4];
                        const float2 a = __fmul2_rn(__fmul2_rn(make_float2(x[i], x[i + 1]), f2), make_float2(w.x, w.y));
                        const float2 e2 = __fmul2_rn(__fmul2_rn(make_float2(x[i + 2], x[i + 3]), f2), make_float2(w.z, w.w));
                        pk[i / 2] = pack_bf16x2(a.x, a.y);
                        pk[i / 2 + 1] = pack_bf16x2(e2.x, e2.y);
                    }
                } else {
                    // the diagonal block, or one that the sequence ends in: columns lo .. hi - 1 are live
                    const float *w = tab + (d > 0 ? (j > 0 ? c1 : p.rev ? 0 : 96) : p.rev ? -lane : 128 - lane);
                    const int lo = d == 0 && p.rev ? lane : 0, hi = min(d == 0 && !p.rev ? lane + 1 : 32, cols - c1);
#pragma unroll
                    for (int i = 0; i < 32; ++i) x[i] = i >= lo && i < hi ? x[i] * f * w[i] : 0.f;
#pragma unroll
                    for (int i = 0; i < 16; ++i) pk[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
                }
                tmem_st16(to, pk);
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
            tma_store_commit();
            tma_store_wait();
        }
    }
    __syncthreads();
    __syncwarp();
    if (warp == 1) tmem_dealloc(tm, 256);
}

// ---- launches -----------------------------------------------------------------------------------------------
template <int NX, bool SEQ>
cudaError_t state_nx(const LinStateP &p, int32_t *status, cudaStream_t s) {
    using C = StateCfg<NX, SEQ>;
    const uint64_t BH = (uint64_t)p.B * p.H;
    CUtensorMap tmz, tmy, tmo;
    if (!make_tmap_3d_bf16(&tmz, p.z, p.dv, p.T, BH, 64, kStep) || !make_tmap_3d_bf16(&tmy, p.y, p.dqk, p.T, BH, 64, kStep) ||
        !(SEQ ? make_tmap_3d_bf16(&tmo, p.states, p.dqk, p.dv, BH * p.nseg, 64, 128)
              : make_tmap_3d_f32(&tmo, p.sums, p.dqk, p.dv, BH * p.nseg, 128)))
        return cudaErrorInvalidValue;
    auto *const kernel = state_tc_kernel<NX, SEQ>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::BYTES);
    if (e != cudaSuccess) return e;
    const int zt = (p.dv + 127) / 128, yt = (p.dqk + NX - 1) / NX;
    const size_t items = BH * zt * yt * (SEQ ? 1 : p.nseg);
    const unsigned grid = items < (size_t)sm_count() ? (unsigned)items : (unsigned)sm_count();
    kernel<<<grid, kStateThreads, C::BYTES, s>>>(tmz, tmy, tmo, p, (int)items, zt, yt, status);
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

bool linattn_states_seq(const LinStateP &p) {
    const int nx = p.dqk > 128 ? 256 : p.dqk > 64 ? 128 : 64;
    return p.nseg == 1 || (size_t)p.B * p.H * ((p.dv + 127) / 128) * ((p.dqk + nx - 1) / nx) >= 96;
}
cudaError_t linattn_states_tc(const LinStateP &p, int32_t *status, cudaStream_t s) {
    if (linattn_states_seq(p))
        return p.dqk > 128 ? state_nx<256, true>(p, status, s) : p.dqk > 64 ? state_nx<128, true>(p, status, s)
                                                                           : state_nx<64, true>(p, status, s);
    return p.dqk > 64 ? state_nx<128, false>(p, status, s) : state_nx<64, false>(p, status, s);
}
cudaError_t linattn_tile_tc(const LinTileP &p, int32_t *status, cudaStream_t s) {
    return p.dz > 64 ? tile_nz<128>(p, status, s) : tile_nz<64>(p, status, s);
}

}  // namespace xlstm
