// The MX4 1x1 convolution on the tensor cores: out[M, N] = act(x[M, K] w[N, K]^T
// + bias + r), tcgen05.mma kind::mxf4 with one e8m0 scale per 32 elements.
//
// Persistent CTAs, one per SM; a tile is 128 rows (pixels) x kBN channels, or
// 256 x 256 for a pair of CTAs that share each MMA (each holds half of the rows
// and half of the channels' weights).
//   warp 0      loads K steps of 256: x and w rows of 128 bytes (TMA, 128-byte
//               swizzle) and their scale tiles (512 bytes per 128 rows x 128 K,
//               stored in the order TMEM wants them) into a ring of stages;
//   warp 1      (of rank 0) copies the scales to TMEM (tcgen05.cp) and issues the
//               MMAs, four K = 64 steps a stage.  The scale columns belong to the
//               ring stage and are free exactly when it is.  Of rank 1: passes its
//               epilogue's hand-backs on to rank 0 (an arrival that releases at
//               cluster scope costs 700 cycles in the epilogue's way);
//   warps 4-..  epilogue: groups of eight warps, two per TMEM lane quarter, the
//               groups and the accumulators taking the tiles in turn, so that it
//               runs beside the next tiles' MMAs.  Results (and shortcut values
//               before them) pass through boxes of 128 rows x 128 bytes, a stream
//               of boxes for each group and side;
//   warp 2      loads the shortcut into free boxes (TMA); warp 3 and the last warp
//               store the finished ones of a side each: issuing a tensor copy
//               costs a thread several hundred cycles, which the epilogue warps
//               do not have.
// One CTA: two groups and three accumulators.  A warp's way through a box (TMEM,
// arithmetic, shared memory) is one long chain of latencies, and so is the way
// from a drained accumulator to the next one that is full; two groups keep two
// tiles in the first, the third accumulator hides the second.
// Pair: one group (its K loop is long enough to hide the epilogue behind).  TMEM
// has 512 columns, and the scales need theirs: two accumulators of 256 share
// 128, which are drained first, and the next tile's MMAs start when they are in
// registers.
// 16384 x 4096 x 4096 (pair): 121 us, 4.5 PFLOP/s.  The K loop runs at 6.1 PFLOP/s, bound
// by L2 (a stage of 35 KB per SM in 0.40 us is 12.9 TB/s over the chip; the tensor pipe
// alone would take 0.31), and every tile adds 1.4 us of hand-over; in a long run the
// power cap takes it to 142.  200704 x 128 x 512 with a shortcut (one CTA): 79 us, 5.4
// TB/s; without one 44 us, 5.0 TB/s: bound by memory.
// Every wait is bounded: on a timeout the CTA raises an abort flag, records a
// status bit, lets its copies and MMAs land and leaves.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cstring>

#include "x1cb_float.cuh"
#include "x1cb_internal.h"
#include "x1cb_plan.h"
#include "x1cb_ptx.cuh"

namespace x1cb {
namespace {

constexpr int kGroupWarps = 8;
constexpr int kMaxEpiWarps = 16;
constexpr int kStageK = 256;           // elements: 128 bytes of codes a row
constexpr int kRowsBytes = 128 * 128;  // codes of 128 rows in a stage
constexpr int kSfBytes = 1024;         // scales of 128 rows in a stage
constexpr int kTmem = 512;
constexpr int kIoBox = 128 * 128;      // a box: 128 rows x 128 bytes
constexpr int kMaxIo = 2;              // boxes per stream
constexpr uint64_t kDrainNs = 200000000ull;

struct MxArgs {
    const float *bias;
    const void *r;
    void *out;
    unsigned int *status;
    uint64_t wait_ns;
    long long M;
    int K, N, act, inject;
    int stages, k_steps, kt;  // ring depth; K steps of 256; scale tiles per row block
    int tiles, n_tiles;
    int io;                   // boxes per stream (TMA epilogue)
};

template <int BN, bool kPair> struct Shape {
    static constexpr int kBlocks = (BN + 127) / 128;  // scale blocks of the channels
    static constexpr int kWRows = kPair ? BN / 2 : BN;
    static constexpr int kW = kWRows * 128;           // weight codes of a stage
    static constexpr int kStage = kRowsBytes + kW + kSfBytes * (1 + kBlocks);
    static constexpr int kSfCols = 8 + kBlocks * 8;   // TMEM columns a stage's scales take
    static constexpr int kSharedCols = kPair ? 128 : 0;
    static constexpr int kSecond = BN - kSharedCols;  // from an accumulator to the next
    static constexpr int kAccs = kPair ? 2 : 3;
    static constexpr int kSfBase = (kAccs - 1) * kSecond + BN;
    static constexpr int kSfStages = (kTmem - kSfBase) / kSfCols;  // most ring stages
    static constexpr int kGroups = kPair ? 1 : 2;     // epilogue groups
    static constexpr int kEpiWarps = kGroups * kGroupWarps;
    static constexpr int kThreads = 32 * (5 + kEpiWarps);
};

// Tail of the dynamic shared memory behind the ring and the epilogue's boxes.
constexpr int kPatch = 32 * 33 * 4;  // an epilogue warp's transposing patch (plain epilogue)
struct Tail {
    alignas(16) float bias[kMaxEpiWarps][64];  // read four at a time
    unsigned long long bars[2 * 8 + 2 * 3 + 4];
    // by stream and slot: shortcut loaded, box written, box free again
    unsigned long long r_full[4][kMaxIo], ready[4][kMaxIo], free_box[4][kMaxIo];
    uint32_t tmem;
    int abort_flag;
};

// The tiles of a CTA (or of one of its epilogue groups): every `step`-th of the
// n_tiles x m_tiles, channels first.
struct Tiles {
    int t, end, step, mt, nt, n_tiles, step_m, step_n;

    __device__ __forceinline__ Tiles(const MxArgs &a, int first, int step_)
        : t(first), end(a.tiles), step(step_), mt(first / a.n_tiles), nt(first - mt * a.n_tiles),
          n_tiles(a.n_tiles), step_m(step_ / a.n_tiles), step_n(step_ - step_m * a.n_tiles)
    {
    }
    __device__ __forceinline__ bool done() const { return t >= end; }
    __device__ __forceinline__ void next()
    {
        t += step;
        mt += step_m;
        nt += step_n;
        if (nt >= n_tiles) {
            nt -= n_tiles;
            ++mt;
        }
    }
};

// The boxes of 128 rows x 128 bytes of a tile, in the order in which they are
// worked on: from the columns that the accumulators share on (accumulator 0
// shares its last columns with the first of accumulator 1).  Box j belongs to
// side j & 1 of its group.
template <typename T, int BN, bool kPair> struct Boxes {
    static constexpr int kCols = 128 / sizeof(T);
    static constexpr int kPer = BN / kCols;
    static __device__ __forceinline__ int col(int acc, int j)
    {
        return (acc ? j : kPer - 1 - j) * kCols;
    }
};

// Slot and phase of a stream's boxes.
struct Slot {
    int d = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int io)
    {
        if (++d == io) {
            d = 0;
            phase ^= 1u;
        }
    }
};

// Accumulator of a tile and the parity of its use.
template <int kAccs> struct Turn {
    int acc;
    uint32_t phase = 0;
    __device__ __forceinline__ explicit Turn(int first) : acc(first) {}
    __device__ __forceinline__ void next(int tiles)
    {
        acc += tiles;
        if (acc >= kAccs) {
            acc -= kAccs;
            phase ^= 1u;
        }
    }
};

// A load whose result stays as it came, in whole registers, until it is used: the
// parts of a 4-byte or the value of a 2-byte Vec would be taken out at once, each
// load waiting for the one before (200000 x 64 x 250 with a shortcut: 154 us, 66 so).
template <int BYTES> struct Late {
    using type = typename Raw<BYTES>::type;
    static __device__ __forceinline__ type load(const void *p)
    {
        return __ldg(static_cast<const type *>(p));
    }
};
template <> struct Late<2> {
    using type = uint32_t;
    static __device__ __forceinline__ type load(const void *p)
    {
        uint32_t v;
        asm volatile("ld.global.nc.u16 %0, [%1];" : "=r"(v) : "l"(p));
        return v;
    }
};

// kIo: outputs (and the shortcut) move as 128 x 128-byte boxes by TMA, which
// needs rows of a multiple of 16 bytes; otherwise the plain epilogue transposes
// through shared memory and stores element by element.
template <typename T, int BN, bool kPair, bool kIo>
__global__ void __launch_bounds__(Shape<BN, kPair>::kThreads, 1)
    conv_mx4_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                    const __grid_constant__ CUtensorMap tmXs,
                    const __grid_constant__ CUtensorMap tmWs,
                    const __grid_constant__ CUtensorMap tmR, const __grid_constant__ CUtensorMap tmO,
                    const MxArgs a)
{
    using S = Shape<BN, kPair>;
    extern __shared__ uint8_t raw[];
    // (aligned by an offset: a pointer made from an integer would lose its
    // address space, and every access through it become a generic one)
    uint8_t *smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    const uint32_t sbase = smem_u32(smem);
    // the epilogue's boxes first: they keep the 1024-byte alignment of the swizzle
    const int epi_bytes = kIo ? 2 * S::kGroups * a.io * kIoBox : S::kEpiWarps * kPatch;
    const uint32_t ring = sbase + ((epi_bytes + 1023) & ~1023);
    Tail *tail = reinterpret_cast<Tail *>(smem + (ring - sbase) + a.stages * S::kStage);
    const uint32_t bars = smem_u32(tail->bars);
    const auto full = [&](int s) { return bars + 8u * s; };
    const auto empty = [&](int s) { return bars + 8u * (a.stages + s); };
    const auto acc_full = [&](int b) { return bars + 8u * (2 * a.stages + b); };
    const auto acc_empty = [&](int b) { return bars + 8u * (2 * a.stages + 3 + b); };
    const uint32_t mma_done = bars + 8u * (2 * a.stages + 6), never = mma_done + 8u;
    const uint32_t exit_bar = never + 8u, shared_free = never + 16u;
    volatile int *abort_flag = &tail->abort_flag;
    const WaitCtl ctl{abort_flag, a.status, a.inject == 1 ? 4 * a.wait_ns : a.wait_ns};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = kPair ? cluster_ctarank() : 0u;
    const int unit = kPair ? blockIdx.x >> 1 : blockIdx.x;
    const int units = kPair ? gridDim.x >> 1 : gridDim.x;

    if (threadIdx.x == 0) {
        *abort_flag = 0;
        for (int s = 0; s < a.stages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        // drained by the group's warps; of a pair, rank 1's count as one at rank 0
        const int drains = kGroupWarps + (kPair && rank == 0 ? 1 : 0);
        for (int b = 0; b < S::kAccs; ++b) {
            mbar_init(acc_full(b), 1);
            mbar_init(acc_empty(b), drains);
        }
        mbar_init(shared_free, drains);
        for (int q = 0; q < 4; ++q)
            for (int d = 0; d < kMaxIo; ++d) {
                mbar_init(smem_u32(&tail->r_full[q][d]), 1);
                mbar_init(smem_u32(&tail->ready[q][d]), 4);  // a warp per lane quarter
                mbar_init(smem_u32(&tail->free_box[q][d]), 1);
            }
        mbar_init(mma_done, 1);
        mbar_init(never, 1);
        mbar_init(exit_bar, 1);
        fence_mbar_init();
        tma_prefetch_desc(&tmX);
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmXs);
        tma_prefetch_desc(&tmWs);
        if (kIo)
            tma_prefetch_desc(&tmO);
    }
    if (warp == 1) {
        if (kPair) {
            tmem_alloc_pair(smem_u32(&tail->tmem), kTmem);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(smem_u32(&tail->tmem), kTmem);
            tmem_relinquish();
        }
        tc_fence_before();
    }
    __syncthreads();
    if (kPair)  // both CTAs' barriers and TMEM exist before traffic crosses
        cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, tail->tmem, 0);
    griddep_wait();  // from here on global memory is touched

    if (warp == 0) {
        int s = 0, issued = 0;
        uint32_t ph = 0;
        bool ok = lane == 0;
        for (Tiles t(a, unit, units); ok && !t.done(); t.next()) {
            const int n0 = t.nt * BN;
            const int xblk = kPair ? 2 * t.mt + static_cast<int>(rank) : t.mt;
            for (int k = 0; k < a.k_steps; ++k) {
                if (!mbar_wait(empty(s), ph ^ 1u, ctl, kDevTimeoutProducer)) {
                    ok = false;
                    break;
                }
                const uint32_t st = ring + s * S::kStage, sf = st + kRowsBytes + S::kW;
                if constexpr (kPair) {
                    // both CTAs' loads complete on rank 0's barrier
                    if (rank == 0)
                        mbar_arrive_expect_tx(full(s), 2 * S::kStage);
                    const uint32_t bar = mapa_shared(full(s), 0);
                    tma2_load_2d(st, &tmX, bar, k * 128, xblk * 128);
                    tma2_load_2d(st + kRowsBytes, &tmW, bar, k * 128,
                                 n0 + static_cast<int>(rank) * S::kWRows);
                    tma2_load_3d(sf, &tmXs, bar, 0, 2 * k, xblk);
                    tma2_load_3d(sf + kSfBytes, &tmWs, bar, 0, 2 * k, n0 / 128);
                } else {
                    mbar_arrive_expect_tx(full(s), S::kStage);
                    tma_load_2d(st, &tmX, full(s), k * 128, xblk * 128);
                    tma_load_2d(st + kRowsBytes, &tmW, full(s), k * 128, n0);
                    tma_load_3d(sf, &tmXs, full(s), 0, 2 * k, xblk);
                    tma_load_3d(sf + kSfBytes, &tmWs, full(s), 0, 2 * k, n0 / 128);
                }
                ++issued;
                if (++s == a.stages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        // Let every copy still in flight land (after a failed wait elsewhere nobody
        // else waited for the last ones).  Of a pair, rank 0 waits for both and the
        // exit handshake holds rank 1 until then.
        if (rank == 0 && lane == 0)
            for (int i = max(0, issued - a.stages); i < issued; ++i)
                if (!mbar_drain(full(i % a.stages), (i / a.stages) & 1, kDrainNs))
                    atomicOr(a.status, kDevDrainFailed);
        __syncwarp();
    } else if (warp == 1 && rank == 0) {
        bool ok = true;
        if (a.inject == 1) {
            const WaitCtl planted{abort_flag, a.status, a.wait_ns};
            ok = __all_sync(0xffffffffu, mbar_wait(never, 0, planted, kDevTimeoutMma));
        }
        const auto wait = [&](uint32_t bar, uint32_t parity) {
            return __all_sync(0xffffffffu, kPair ? mbar_wait_cl(bar, parity, ctl, kDevTimeoutMma)
                                                 : mbar_wait(bar, parity, ctl, kDevTimeoutMma));
        };
        const auto commit = [&](uint32_t bar) {
            if (kPair)
                mma_commit_pair(bar);
            else
                mma_commit(bar);
        };
        int s = 0, i = 0;
        uint32_t ph = 0;
        Turn<S::kAccs> turn(0);
        for (Tiles t(a, unit, units); ok && !t.done(); t.next(), turn.next(1), ++i) {
            // The accumulator is free: its own last tile is drained, and the tile
            // before this one has left the shared columns.
            if (!wait(acc_empty(turn.acc), turn.phase ^ 1u) ||
                (kPair && i > 0 && !wait(shared_free, (i - 1) & 1)))
                break;
            tc_fence_after();
            const uint32_t d = tmem + turn.acc * S::kSecond;
            for (int k = 0; k < a.k_steps; ++k) {
                if (!wait(full(s), ph)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t st = ring + s * S::kStage, sf = st + kRowsBytes + S::kW;
                const uint32_t sfa = tmem + S::kSfBase + s * S::kSfCols, sfw = sfa + 8;
                const uint64_t ad = smem_desc_sw128(st), bd = smem_desc_sw128(st + kRowsBytes);
                constexpr uint32_t kM = kPair ? 256 : 128;
                const int left = (a.K - k * kStageK + 63) / 64;  // K = 64 steps
                if (left >= 4) {
                    mma_mx4_stage<kPair, S::kBlocks, 4>(d, ad, bd, idesc_mx4(kM, BN, 0),
                                                        idesc_mx4(kM, BN, 2), sfa, sfw, 0u,
                                                        smem_desc_scales(sf), k > 0);
                } else if (left == 2) {
                    mma_mx4_stage<kPair, S::kBlocks, 2>(d, ad, bd, idesc_mx4(kM, BN, 0),
                                                        idesc_mx4(kM, BN, 2), sfa, sfw, 0u,
                                                        smem_desc_scales(sf), k > 0);
                } else {
                    for (int j = 0; j < (left + 1) / 2; ++j) {
                        tmem_cp_scales<kPair>(sfa + 4 * j, smem_desc_scales(sf + 512 * j));
#pragma unroll
                        for (int b = 0; b < S::kBlocks; ++b)
                            tmem_cp_scales<kPair>(
                                sfw + S::kBlocks * 4 * j + 4 * b,
                                smem_desc_scales(sf + kSfBytes * (1 + b) + 512 * j));
                    }
                    for (int j = 0; j < left; ++j)
                        mma_mx4<kPair>(d, ad + 2 * j, bd + 2 * j, idesc_mx4(kM, BN, (j & 1) * 2),
                                       sfa + 4 * (j >> 1), sfw + S::kBlocks * 4 * (j >> 1),
                                       k > 0 || j > 0);
                }
                commit(empty(s));
                if (++s == a.stages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            if (!ok)
                break;
            commit(acc_full(turn.acc));
        }
        // No MMA may still read shared memory or write TMEM behind this point.
        commit(mma_done);
        if (lane == 0 && !mbar_drain(mma_done, 0, kDrainNs))
            atomicOr(a.status, kDevDrainFailed);
        __syncwarp();
    } else if (kPair && warp == 1) {
        // ---- rank 1: its epilogue's hand-backs, passed on in tile order -------------
        if (lane == 0) {
            Turn<S::kAccs> turn(0);
            int i = 0;
            for (Tiles t(a, unit, units); !t.done(); t.next(), turn.next(1), ++i) {
                if (!mbar_wait(shared_free, i & 1, ctl, kDevTimeoutMma))
                    break;
                mbar_arrive_cluster(mapa_shared(shared_free, 0));
                if (!mbar_wait(acc_empty(turn.acc), turn.phase, ctl, kDevTimeoutMma))
                    break;
                mbar_arrive_cluster(mapa_shared(acc_empty(turn.acc), 0));
            }
        }
        __syncwarp();
    } else if (kIo && warp == 2) {
        // ---- shortcut loads, boxes in tile order ------------------------------------
        using B = Boxes<T, BN, kPair>;
        if (lane == 0 && a.r) {
            Slot slot[S::kGroups][2];
            int group = 0;
            bool ok = true;
            Turn<S::kAccs> turn(0);
            for (Tiles t(a, unit, units); ok && !t.done(); t.next(), turn.next(1)) {
                const int row = t.mt * (kPair ? 256 : 128) + static_cast<int>(rank) * 128;
#pragma unroll
                for (int j = 0; j < B::kPer; ++j) {
                    Slot &sl = S::kGroups == 2 && group ? slot[S::kGroups - 1][j & 1] : slot[0][j & 1];
                    const int q = group * 2 + (j & 1);
                    const int ch = t.nt * BN + B::col(turn.acc, j);
                    const uint32_t bar = smem_u32(&tail->r_full[q][sl.d]);
                    if (!mbar_wait(smem_u32(&tail->free_box[q][sl.d]), sl.phase ^ 1u, ctl,
                                   kDevTimeoutProducer)) {
                        ok = false;
                        break;
                    }
                    if (row < a.M && ch < a.N) {
                        mbar_arrive_expect_tx(bar, kIoBox);
                        tma_load_2d(sbase + (q * a.io + sl.d) * kIoBox, &tmR, bar, ch, row);
                    } else {
                        mbar_arrive(bar);
                    }
                    sl.next(a.io);
                }
                group ^= S::kGroups - 1;
            }
            // Shortcut boxes in flight land before the CTA leaves: the last load of
            // slot d was in the stream's current phase if d lies before its next slot.
#pragma unroll
            for (int q = 0; q < 2 * S::kGroups; ++q) {
                const Slot &sl = slot[q / 2][q & 1];
                for (int d = 0; d < a.io; ++d)
                    if (!mbar_drain(smem_u32(&tail->r_full[q][d]),
                                    d < sl.d ? sl.phase : sl.phase ^ 1u, kDrainNs))
                        atomicOr(a.status, kDevDrainFailed);
            }
        }
        __syncwarp();
    } else if (warp == 3 || warp == 4 + S::kEpiWarps) {
        // ---- stores of one side's boxes, in tile order ------------------------------
        using B = Boxes<T, BN, kPair>;
        const int side = warp == 3 ? 0 : 1;
        if (kIo && lane == 0 && side < B::kPer) {
            Slot slot[S::kGroups];
            int group = 0;
            bool ok = true;
            Turn<S::kAccs> turn(0);
            for (Tiles t(a, unit, units); ok && !t.done(); t.next(), turn.next(1)) {
                const int row = t.mt * (kPair ? 256 : 128) + static_cast<int>(rank) * 128;
                Slot &sl = S::kGroups == 2 && group ? slot[S::kGroups - 1] : slot[0];
                const int q = group * 2 + side;
                for (int j = side; j < B::kPer; j += 2) {
                    const int ch = t.nt * BN + B::col(turn.acc, j);
                    if (!mbar_wait(smem_u32(&tail->ready[q][sl.d]), sl.phase, ctl,
                                   kDevTimeoutProducer)) {
                        ok = false;
                        break;
                    }
                    if (row < a.M && ch < a.N) {
                        tma_store_2d(&tmO, sbase + (q * a.io + sl.d) * kIoBox, ch, row);
                        bulk_commit();
                        bulk_wait_read<0>();
                    }
                    mbar_arrive(smem_u32(&tail->free_box[q][sl.d]));
                    sl.next(a.io);
                }
                group ^= S::kGroups - 1;
            }
            bulk_wait_all();
        }
        __syncwarp();
    } else if (warp >= 4) {
        const int e = warp - 4, quarter = e & 3, side = (e >> 2) & 1, group = e >> 3;
        const uint32_t lanes_at = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        const int row_off = static_cast<int>(rank) * 128 + quarter * 32;
        const auto release = [&](uint32_t bar) {  // after the warp's reads of the accumulator
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar);
        };
        Turn<S::kAccs> turn(group);
        const auto wait_acc = [&]() {
            const bool ok = __all_sync(0xffffffffu, mbar_wait(acc_full(turn.acc), turn.phase, ctl,
                                                              kDevTimeoutEpilogue));
            tc_fence_after();
            return ok;
        };
        if constexpr (kIo) {
            using B = Boxes<T, BN, kPair>;
            const int q = group * 2 + side;  // the stream
            float *bias = tail->bias[e];
            Slot slot;
            // a box's bias is loaded one box ahead, two channels a lane
            float b0 = 0.f, b1 = 0.f;
            const auto load_bias = [&](int c) {
                if (a.bias) {
                    c += lane;
                    b0 = c < a.N ? __ldg(a.bias + c) : 0.f;
                    if (B::kCols == 64)
                        b1 = c + 32 < a.N ? __ldg(a.bias + c + 32) : 0.f;
                }
            };
            Tiles t(a, unit + group * units, S::kGroups * units);
            if (!t.done())
                load_bias(t.nt * BN + B::col(turn.acc, side));
            bool ok = true;
            while (ok && !t.done()) {
                if (!wait_acc())
                    break;
                const int acc = turn.acc, n0 = t.nt * BN;
                t.next();
                turn.next(S::kGroups);
                const int n0_next = t.done() ? 0 : t.nt * BN;
                for (int j = side; j < B::kPer; j += 2) {
                    // The box is free, or holds the shortcut.
                    const uint32_t bar = smem_u32(a.r ? &tail->r_full[q][slot.d]
                                                      : &tail->free_box[q][slot.d]);
                    if (!__all_sync(0xffffffffu,
                                    mbar_wait(bar, a.r ? slot.phase : slot.phase ^ 1u, ctl,
                                              kDevTimeoutEpilogue))) {
                        ok = false;
                        break;
                    }
                    // Pair: the box's columns are read at once, and the accumulator (or
                    // its shared part) handed back before the arithmetic.  One CTA with
                    // two groups has the registers for 32 columns at a time.
                    const uint32_t at_acc = lanes_at + acc * S::kSecond + B::col(acc, j);
                    uint32_t v[kPair ? B::kCols / 32 : 1][32];
                    if constexpr (kPair) {
#pragma unroll
                        for (int h = 0; h < B::kCols / 32; ++h)
                            tmem_ld_32x32b_x32(at_acc + 32 * h, v[h]);
                    }
                    bias[lane] = b0;
                    if (B::kCols == 64)
                        bias[32 + lane] = b1;
                    const bool last = j + 2 >= B::kPer;
                    load_bias(last ? n0_next + B::col(turn.acc, side) : n0 + B::col(acc, j + 2));
                    if constexpr (kPair) {
#pragma unroll
                        for (int h = 0; h < B::kCols / 32; ++h)
                            tmem_ld_wait(v[h]);
                        constexpr int kShared = S::kSharedCols / B::kCols;
                        if (j < kShared && j + 2 >= kShared)
                            release(shared_free);
                        if (last)
                            release(acc_empty(acc));
                    }
                    __syncwarp();
                    uint8_t *mine = smem + (q * a.io + slot.d) * kIoBox + (quarter * 32 + lane) * 128;
#pragma unroll
                    for (int h = 0; h < B::kCols / 32; ++h) {
                        if constexpr (!kPair)
                            tmem_ld_32x32b_x32_sync(at_acc + 32 * h, v[0]);
                        const uint32_t(&w)[32] = v[kPair ? h : 0];
                        // 16 bytes (kV elements) at a time
                        constexpr int kV = 16 / sizeof(T);
#pragma unroll
                        for (int c = 0; c < 32; c += kV) {
                            uint8_t *at = mine + ((((32 * h + c) / kV) ^ (lane & 7)) * 16);
                            F2 f[kV / 2];
#pragma unroll
                            for (int i = 0; i < kV; i += 4) {
                                const float4 b =
                                    *reinterpret_cast<const float4 *>(bias + 32 * h + c + i);
                                f[i / 2] = add2(f2(__uint_as_float(w[c + i]),
                                                   __uint_as_float(w[c + i + 1])),
                                                f2(b.x, b.y));
                                f[i / 2 + 1] = add2(f2(__uint_as_float(w[c + i + 2]),
                                                       __uint_as_float(w[c + i + 3])),
                                                    f2(b.z, b.w));
                            }
                            if (a.r) {
                                const Vec<T, kV> rv = *reinterpret_cast<const Vec<T, kV> *>(at);
                                F2 g[kV / 2];
                                unpack<T, kV>(rv, g);
#pragma unroll
                                for (int i = 0; i < kV / 2; ++i)
                                    f[i] = add2(f[i], g[i]);
                            }
                            store_vec<T, kV>(reinterpret_cast<T *>(at), finish<T, kV>(f, a.act));
                        }
                    }
                    if (!kPair && last)
                        release(acc_empty(acc));
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(smem_u32(&tail->ready[q][slot.d]));
                    slot.next(a.io);
                }
                // a side without boxes still answers for its share of the barriers
                // (only a 64-channel tile of one CTA: no shared columns)
                if (side >= B::kPer)
                    release(acc_empty(acc));
            }
        } else {
            // Parts of 64 columns, 32 for each side: accumulator -> patch -> rows, in
            // turns of 8 V rows in which a lane takes V neighbouring columns of
            // every V-th row.  The shortcut of a turn is loaded while the one before it
            // is worked on (140800 x 96 x 52 with one: 79.8 us without that, 27.0 so),
            // the bias of a part likewise.  The turns are a loop of few instructions:
            // unrolled, fetching them took longer than the work.
            const auto plain = [&](auto vec) {
                constexpr int V = decltype(vec)::value, kParts = BN / 64, kRows = 8;
                constexpr int kTurn = kRows * V;  // rows a turn
                float *patch = reinterpret_cast<float *>(smem) + e * (kPatch / 4);
                const int lr = lane / (32 / V), lc = lane % (32 / V) * V;
                const size_t step = static_cast<size_t>(V) * a.N;
                struct Part {
                    size_t at;  // the lane's first element
                    int rows;   // rows from there on, counted in steps of V
                    float bias[V];
                };
                const auto part_at = [&](const Tiles &t, int acc, int part) {
                    Part p;
                    // (accumulator 0 shares its last columns with the next tile's first)
                    const int c = t.nt * BN + (acc ? part : kParts - 1 - part) * 64 + side * 32 + lc;
                    const long long row =
                        static_cast<long long>(t.mt) * (kPair ? 256 : 128) + row_off + lr;
                    p.rows = t.done() || c >= a.N
                                 ? 0
                                 : static_cast<int>(max(0ll, min(32ll - lr, a.M - row)));
                    p.at = static_cast<size_t>(row) * a.N + c;
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        p.bias[i] = a.bias && p.rows > 0 ? __ldg(a.bias + c + i) : 0.f;
                    return p;
                };
                using L = Late<sizeof(T) * V>;
                typename L::type rv[kRows];
                const auto load_r = [&](size_t at, int rows) {
                    if (a.r) {
                        const T *r = static_cast<const T *>(a.r) + at;
#pragma unroll
                        for (int i = 0; i < kRows; ++i)
                            if (i * V < rows)
                                rv[i] = L::load(r + i * step);
                    }
                };
                Tiles t(a, unit + group * units, S::kGroups * units);
                Part next = part_at(t, turn.acc, 0);
                load_r(next.at, next.rows);
                while (!t.done() && wait_acc()) {
                    const int acc = turn.acc;
                    const Tiles now = t;
                    t.next();
                    turn.next(S::kGroups);
#pragma unroll 1
                    for (int part = 0; part < kParts; ++part) {
                        const int c0 = (acc ? part : kParts - 1 - part) * 64 + side * 32;
                        const bool last = part == kParts - 1, any = now.nt * BN + c0 < a.N;
                        if (any) {
                            uint32_t v[32];
                            tmem_ld_32x32b_x32_sync(lanes_at + acc * S::kSecond + c0, v);
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                patch[lane * 33 + i] = __uint_as_float(v[i]);
                        }
                        if (kPair && part == S::kSharedCols / 64 - 1)
                            release(shared_free);
                        if (last)
                            release(acc_empty(acc));
                        const Part p = next;
                        next = part_at(last ? t : now, last ? turn.acc : acc, last ? 0 : part + 1);
                        __syncwarp();
                        size_t at = p.at;
                        const float *from = patch + lr * 33 + lc;
                        for (int row = any ? 0 : 32; row < 32; row += kTurn) {
                            float y[kTurn];
#pragma unroll
                            for (int i = 0; i < kTurn; ++i)
                                y[i] = from[i / V * V * 33 + i % V] + p.bias[i % V];
                            if (a.r) {
#pragma unroll
                                for (int i = 0; i < kRows; ++i) {
                                    F2 f[1];
                                    unpack<T, V>(*reinterpret_cast<const Vec<T, V> *>(&rv[i]), f);
                                    y[i * V] += un2(f[0]).x;
                                    if (V == 2)
                                        y[i * V + V - 1] += un2(f[0]).y;
                                }
                                const bool more = row + kTurn < 32;
                                load_r(more ? at + kRows * step : next.at,
                                       more ? p.rows - row - kTurn : next.rows);
                            }
                            activate(y, a.act);
                            T *to = static_cast<T *>(a.out) + at;
#pragma unroll
                            for (int i = 0; i < kRows; ++i) {
                                if (row + i * V < p.rows) {
                                    Vec<T, V> w;
#pragma unroll
                                    for (int k = 0; k < V; ++k)
                                        w.e[k] = from_f<T>(y[i * V + k]);
                                    store_vec<T, V>(to + i * step, w);
                                }
                            }
                            at += kRows * step;
                            from += kTurn * 33;
                        }
                        if (!any)
                            load_r(next.at, next.rows);
                        __syncwarp();
                    }
                }
            };
            if (a.N % 2 == 0)
                plain(std::integral_constant<int, 2>{});
            else
                plain(std::integral_constant<int, 1>{});
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (kPair) {
        if (threadIdx.x == 0 && !leave_pair(exit_bar, rank, ctl, kDrainNs))
            atomicOr(a.status, kDevDrainFailed);
        __syncthreads();
    }
    if (warp == 1) {
        tc_fence_after();
        if (kPair)
            tmem_dealloc_pair(tmem, kTmem);
        else
            tmem_dealloc(tmem, kTmem);
    }
}

CUtensorMapDataType map_type(int dtype)
{
    return dtype == X1CB_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
           : dtype == X1CB_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
}

// Shared memory of a launch: boxes per stream, ring stages, bytes.
struct Memory {
    int io, stages, bytes;
};
template <typename S, bool kIo> constexpr Memory memory(bool r, int k_steps)
{
    constexpr bool kPair = S::kGroups == 1;
    Memory m{};
    // A second box per stream where the epilogue is the longer part, at the cost of
    // ring stages.  Pair, one box against two: 16384 x 1024 x 4096 55.5 and 49.5, x 2048
    // 73.8 and 77.0; 50176 x 2048 x 256 with a shortcut 28.7 and 27.9.  One CTA, with a
    // shortcut: 200704 x 128 x 512 86.7 and 80.0, x 512 91.0 and 95.7.
    m.io = kPair ? (k_steps >= (r ? 12 : 8) ? 1 : 2) : r && k_steps == 1 ? 2 : 1;
    const int epi = ((kIo ? 2 * S::kGroups * m.io * kIoBox : S::kEpiWarps * kPatch) + 1023) & ~1023;
    const int fixed = 1024 + epi + static_cast<int>(sizeof(Tail));
    m.stages = std::min({(kSmemLimit - fixed) / S::kStage, S::kSfStages, 8});
    // The plain epilogue's loads need L1: 200000 x 64 x 250 with a shortcut 66.0 us
    // with all of the shared memory taken by the ring, 61.5 with half of it.
    if (!kIo && r)
        m.stages = std::min(m.stages, std::max(2, (110 * 1024 - fixed) / S::kStage));
    m.bytes = std::max(fixed + m.stages * S::kStage, kSmemAlone);
    return m;
}

// Every launch keeps its SM to itself, whatever its registers: clusters that wait
// for one another's TMEM columns could never end (tcgen05.alloc has no limit).
template <typename S, bool kIo> constexpr bool alone()
{
    for (int k = 1; k <= 16; ++k)
        for (int r = 0; r < 2; ++r) {
            const Memory m = memory<S, kIo>(r != 0, k);
            if (m.bytes < kSmemAlone || m.bytes > kSmemLimit || m.stages < 2)
                return false;
        }
    return true;
}
template <int BN, bool kPair> constexpr bool both_alone()
{
    return alone<Shape<BN, kPair>, true>() && alone<Shape<BN, kPair>, false>();
}
static_assert(both_alone<64, false>() && both_alone<128, false>() && both_alone<256, true>(),
              "a kernel that holds TMEM would share its SM");

template <typename T, int BN, bool kPair, bool kIo>
int run(const Mx4Call &c, int sms, cudaStream_t s)
{
    using S = Shape<BN, kPair>;
    constexpr int kTileM = kPair ? 256 : 128;
    MxArgs a{};
    unsigned int *forms = nullptr;
    if (int e = device_words(&a.status, &forms))
        return e;
    a.bias = c.bias;
    a.r = c.r;
    a.out = c.out;
    a.wait_ns = wait_limit_ns();
    a.M = c.M;
    a.K = c.K;
    a.N = c.N;
    a.act = c.act;
    a.inject = debug_inject();
    a.k_steps = (c.K + kStageK - 1) / kStageK;
    a.kt = (c.K + 127) / 128;
    a.n_tiles = (c.N + BN - 1) / BN;
    const long long tiles = (c.M + kTileM - 1) / kTileM * a.n_tiles;
    if (tiles > 0x7fffffffLL - sms)
        return X1CB_ERR_SHAPE;
    a.tiles = static_cast<int>(tiles);
    const Memory mem = memory<S, kIo>(c.r != nullptr, a.k_steps);
    a.io = mem.io;
    a.stages = mem.stages;

    CUtensorMap tmX, tmW, tmXs, tmWs, tmR, tmO;
    const uint64_t str[1] = {static_cast<uint64_t>(c.K) / 2};
    const uint64_t dx[2] = {str[0], static_cast<uint64_t>(c.M)};
    const uint64_t dw[2] = {str[0], static_cast<uint64_t>(c.N)};
    const uint32_t bx[2] = {128, 128}, bw[2] = {128, static_cast<uint32_t>(S::kWRows)};
    if (int e = encode_map(&tmX, c.x, 2, dx, str, bx, CU_TENSOR_MAP_SWIZZLE_128B))
        return e;
    if (int e = encode_map(&tmW, c.w, 2, dw, str, bw, CU_TENSOR_MAP_SWIZZLE_128B))
        return e;
    // scales: tiles of 128 words, kt of them per block of 128 rows
    const uint64_t sstr[2] = {512, static_cast<uint64_t>(a.kt) * 512};
    const uint64_t dxs[3] = {128, static_cast<uint64_t>(a.kt), static_cast<uint64_t>((c.M + 127) / 128)};
    const uint64_t dws[3] = {128, static_cast<uint64_t>(a.kt), static_cast<uint64_t>((c.N + 127) / 128)};
    const uint32_t bxs[3] = {128, 2, 1}, bws[3] = {128, 2, S::kBlocks};
    if (int e = encode_map(&tmXs, c.xs, 3, dxs, sstr, bxs, CU_TENSOR_MAP_SWIZZLE_NONE,
                           CU_TENSOR_MAP_DATA_TYPE_UINT32))
        return e;
    if (int e = encode_map(&tmWs, c.ws, 3, dws, sstr, bws, CU_TENSOR_MAP_SWIZZLE_NONE,
                           CU_TENSOR_MAP_DATA_TYPE_UINT32))
        return e;
    tmR = tmO = tmX;  // unused without kIo
    if (kIo) {
        const uint64_t ostr[1] = {static_cast<uint64_t>(c.N) * sizeof(T)};
        const uint64_t d[2] = {static_cast<uint64_t>(c.N), static_cast<uint64_t>(c.M)};
        const uint32_t b[2] = {128 / sizeof(T), 128};
        if (int e = encode_map(&tmO, c.out, 2, d, ostr, b, CU_TENSOR_MAP_SWIZZLE_128B,
                               map_type(c.dtype)))
            return e;
        if (c.r)
            if (int e = encode_map(&tmR, c.r, 2, d, ostr, b, CU_TENSOR_MAP_SWIZZLE_128B,
                                   map_type(c.dtype)))
                return e;
    }
    static std::atomic<bool> opted[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
        return X1CB_ERR_CUDA;
    const auto kern = conv_mx4_kernel<T, BN, kPair, kIo>;
    if (!opted[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit) !=
            cudaSuccess)
            return X1CB_ERR_CUDA;
        opted[dev].store(true, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3(static_cast<unsigned>(kPair ? 2 * std::min<long long>(tiles, sms / 2)
                                                   : std::min<long long>(tiles, sms)),
                       1, 1);
    cfg.blockDim = dim3(S::kThreads, 1, 1);
    cfg.dynamicSmemBytes = mem.bytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = kPair ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, tmX, tmW, tmXs, tmWs, tmR, tmO, a) == cudaSuccess
               ? X1CB_OK
               : X1CB_ERR_CUDA;
}

template <typename T> int run_tile(const Mx4Call &c, int sms, cudaStream_t s)
{
    const bool io = static_cast<size_t>(c.N) * sizeof(T) % 16 == 0;
    // Tiles of 64 channels against 128: 200000 x 256 x 64 13.3 and 14.8 us.
    if (c.N <= 64)
        return io ? run<T, 64, false, true>(c, sms, s) : run<T, 64, false, false>(c, sms, s);
    const long long pairs = (c.M + 255) / 256 * ((c.N + 255) / 256);
    // Pairs need a K loop that hides their hand-over, and at K = 1024 tiles enough that
    // the last round counts for little: 128 x 128 against pairs, 16384 x 512 x 4096 38.8
    // and 42.1 us, x 1024 57.5 and 49.9, x 2048 99.5 and 77.0; 5000 x 1024 x 2048 (160
    // tiles) 13.8 and 14.7, 9472 x 4096 x 512 (74) 17.7 and 15.6.
    if (pairs >= (c.K >= 2048 ? sms / 2 : 3 * (sms / 2)) && c.K >= 1024)
        return io ? run<T, 256, true, true>(c, sms, s) : run<T, 256, true, false>(c, sms, s);
    return io ? run<T, 128, false, true>(c, sms, s) : run<T, 128, false, false>(c, sms, s);
}

}  // namespace

int launch_conv_mx4_tiles(const Mx4Call &c, cudaStream_t s)
{
    int sms = 0;
    if (int e = current_sms(sms))
        return e;
    return c.dtype == X1CB_F32    ? run_tile<float>(c, sms, s)
           : c.dtype == X1CB_BF16 ? run_tile<__nv_bfloat16>(c, sms, s)
                                  : run_tile<__half>(c, sms, s);
}

}  // namespace x1cb
