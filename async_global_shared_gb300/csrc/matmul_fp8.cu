// c = a * b^T of e4m3 matrices with a scale for each block of 128 along k:
//     c[i, j] = sum over blocks kb of sa[i, kb] sb[j, kb] * P_kb[i, j],
//     P_kb[i, j] = sum over the block's 128 k of a[i, k] b[j, k].
// The scales differ from row to row and from block to block, so P_kb cannot
// stay in the tensor core's accumulator: each block's products go to an
// accumulator of their own in tensor memory, and consumer threads read it,
// multiply it by the two scales and add it to sums in registers while the
// tensor core works on the next blocks. sa sb is one factor, which has to be a
// float by itself. Orders that keep scales past 2^64 or below 2^-63 in range
// take another operation a value, and looking for such scales alone costs the
// consumers 4 to 13 % (8192^3 412 us, 449 with a second loop for blocks that
// have them; 4096 x 8192 x 16384 702 and 775).
//
// Below, P is the operand whose rows are the accumulator's rows (128 a CTA)
// and Q the one whose rows are its columns (BN a tile). Three forms:
//  - a pair of CTAs (CG = 2) shares 256 x 256 tiles: each loads half of either
//    operand, so a tile's operands cross the L2 once for two SMs; a persistent
//    grid walks the tiles;
//  - one CTA a 128 x 128 tile, where there are too few tiles of the former;
//  - SWAP: at most 32 rows of a. The weight b takes the P side, so that its rows fill
//    the 128 accumulator rows, and a's rows are the narrow side.
// The last two split k over the CTAs of a cluster where tiles are few: each
// sums its share, and the shares are added through distributed shared memory
// in rank order.
//
// What bounds it. One token times 8192 x 8192: the weight's bytes, 14.9 us = 4.5
// TB/s, of which 5 are the launch, the first loads and the reduction (8 tokens
// times 28672 x 8192: 39 us = 6.0 TB/s). 128 x 128 tiles: the consumers'
// instructions, 66 % of the issue slots over a CTA's life, beside 512 cycles a
// block of shared memory, 59 % (333 x 4104 x 5000: 18.6 us, a quarter of it
// launch, first loads and exit). 8192^3 in pairs: 440 us = 2.5
// PFLOP/s, 410 before the power limit lowers the clocks (596 with one CTA a
// 128 x 128 tile): the consumers, whose loads, sums and hand-over of a block
// take about 850 cycles beside 512 of matrix instructions. Scales by column on
// top: two operations a value, and the column scales' loads (4096 x 8192 x
// 16384: 701 us = 1.57 PFLOP/s; 599 without the loads; with c in 32 bits, as
// here, 56 bytes of spills a thread).
//
// Roles in a CTA, each a warp: the producer streams the operands' 128-byte
// wide boxes through a ring of shared-memory stages (tensor maps, 128-byte
// swizzle, rows and columns past the matrix arrive as zeros); one or two threads
// issue the matrix instructions; a warp brings the scales of
// the next blocks to shared memory; consumer warps own 32 rows each, one row
// a thread and up to 128 columns.
#include <algorithm>
#include <atomic>

#include "device_common.cuh"
#include "fp8_common.cuh"
#include "internal.h"
#include "tcgen05.cuh"

namespace ap {
namespace {

constexpr int kTile = 128;  // rows a CTA, and bytes of k in one stage (one scale block)
constexpr int kMmaK = 32;   // k of one matrix instruction
constexpr int kMaxSplit = 8;
constexpr int kScaleRun = 8;    // blocks of k whose scales are brought at once (one 32-byte sector of a row)
constexpr int kScaleSlots = 2;  // such runs in shared memory
constexpr int64_t kMaxTiles = int64_t(1) << 27;  // tile numbers plus a grid, times a cluster, stay in 32 bits

struct MatmulParams {
    const float* p_scales;
    const float* q_scales;
    void* c;
    int64_t np, nq, ldc;  // rows of P and of Q
    int p_shift;          // log2 of the rows of P that share a scale
    int32_t nkb;          // blocks of k
    int32_t tiles_p, tiles_q;
    int split;            // CTAs of a cluster that share a tile's k
    bool vec_c;           // rows of c start on 16-byte boundaries
    uint32_t tx_extra;    // fault injection: bytes every stage waits for in vain
    uint64_t timeout_ns;
    uint32_t* status;
};

template <int BN, int CG, int STAGES, bool PER_COL, bool SWAP>
struct Form {
    static constexpr int kGroups = BN < 128 ? 1 : 2;  // consumer groups, side by side along the columns
    static constexpr int kCols = BN / kGroups;           // columns of a group
    static constexpr int kMmaGroups = BN > 128 ? 2 : 1;  // matrix instructions side by side
    static constexpr int kMmaCols = BN / kMmaGroups;     // columns of one
    static constexpr int kConsumerWarps = 4 * kGroups;
    static constexpr int kThreads = 32 * (kConsumerWarps + 4);
    // The widest form: 384 threads of 168 registers at launch (64512), shared
    // out anew: 128 sums and the loads under way need more than 168.
    static constexpr int kOtherRegs = PER_COL ? 56 : 72, kConsumerRegs = PER_COL ? 224 : 216;
    static_assert(BN <= 128 || 128 * kOtherRegs + 256 * kConsumerRegs <= 384 * 168, "registers of the launch");
    static constexpr int kQBox = kMmaCols / CG;  // rows of Q this CTA loads for one instruction
    static constexpr uint32_t kPBytes = kTile * kTile, kQBytes = kQBox * kTile;
    static constexpr uint32_t kStageBytes = kPBytes + kMmaGroups * kQBytes;
    // Accumulators: the products of kRun blocks of k side by side are handed
    // over at once (a hand-over costs hundreds of cycles whatever its size),
    // in two buffers. The widest form fills tensor memory with one block each.
    static constexpr int kRun = CG == 2 ? 1 : 2;
    static constexpr int kBuffers = CG == 2 ? 512 / BN : 2;
    static constexpr uint32_t kTmemCols = kBuffers * kRun * BN;
    // CTAs an SM: the narrow forms wait more than they compute
    static constexpr int kCtas = SWAP ? 2 : 1;
    // c leaves through shared memory: a consumer warp's 32 rows of 128 bytes
    static constexpr uint32_t kStagingBytes = SWAP ? 0 : 32 * 128 * kConsumerWarps;
    static constexpr size_t kRingBytes = size_t(STAGES) * kStageBytes;
    static constexpr size_t kSmem = kRingBytes + kStagingBytes + 1024;
    // a split tile's shares: rows of BN floats, padded so that the 32 rows a
    // warp writes fall on different banks; or columns of 128 floats
    static constexpr int kSharePitch = BN + 4;
    static constexpr size_t kShareBytes = size_t(kTile) * kSharePitch * 4;
};

// Scales of a run of blocks, [slot][block][row or column]; the pitch puts the
// eight blocks of four rows that a copy writes at once on different banks.
template <typename F, int STAGES, bool PER_COL>
struct __align__(16) Shared {
    float row_scales[kScaleSlots][kScaleRun][kTile + 4];
    float col_scales[kScaleSlots][kScaleRun][PER_COL ? F::kGroups * F::kCols + 4 : 4];  // or one a group
    uint64_t full[STAGES], empty[STAGES];
    uint64_t acc_full[F::kBuffers][F::kMmaGroups], acc_empty[F::kBuffers][F::kMmaGroups];
    uint64_t scales_full[kScaleSlots], scales_empty[kScaleSlots];
    uint32_t tmem;
    int abort;
};

// Tile t of the walk: bands of 8 tiles along P, Q outermost within a band, so
// the CTAs of one moment share operand rows in the L2.
__device__ __forceinline__ void tile_at(const MatmulParams& P, int32_t t, int32_t* tp, int32_t* tq) {
    constexpr int kBand = 8;
    const int32_t per_band = kBand * P.tiles_q;
    const int32_t first = t / per_band * kBand;
    const int32_t high = P.tiles_p - first < kBand ? P.tiles_p - first : kBand;
    const int32_t r = t % per_band;
    *tp = first + r % high;
    *tq = r / high;
}

// Four values as the C type at p (aligned for a vector store).
template <typename C>
__device__ __forceinline__ void store4(C* p, float4 v) {
    if constexpr (sizeof(C) == 4)
        *reinterpret_cast<float4*>(p) = v;
    else
        *reinterpret_cast<uint2*>(p) = make_uint2(pack2<C>(v.x, v.y), pack2<C>(v.z, v.w));
}

__device__ __forceinline__ uint4 as_words(float a, float b, float c, float d) {
    return make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d));
}

template <typename C>
__device__ __forceinline__ C ld_shared(uint32_t addr) {
    C v;
    if constexpr (sizeof(C) == 4) {
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
    } else {
        uint16_t w;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(w) : "r"(addr));
        v = *reinterpret_cast<C*>(&w);
    }
    return v;
}
__device__ __forceinline__ void st_shared(uint32_t addr, float v) {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void st_shared4(uint32_t addr, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

template <typename C, int BN, int CG, int STAGES, bool PER_COL, bool SWAP>
__global__ void __launch_bounds__(Form<BN, CG, STAGES, PER_COL, SWAP>::kThreads, Form<BN, CG, STAGES, PER_COL, SWAP>::kCtas)
    matmul_fp8_kernel(const __grid_constant__ CUtensorMap map_p, const __grid_constant__ CUtensorMap map_q,
                      const __grid_constant__ CUtensorMap map_c, const __grid_constant__ MatmulParams P) {
    using F = Form<BN, CG, STAGES, PER_COL, SWAP>;
    constexpr int kCols = F::kCols;
    extern __shared__ unsigned char smem_raw[];
    __shared__ Shared<F, STAGES, PER_COL> sh;
    const uint32_t ring = (ptx::smem_addr(smem_raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int* abort_flag = &sh.abort;
    const uint32_t rank = CG == 2 || P.split > 1 ? ptx::cluster_ctarank() : 0;
    const int part = CG == 2 ? 0 : static_cast<int>(rank);  // share of k
    const int32_t kb0 = static_cast<uint32_t>(P.nkb * part) / P.split;  // nkb < 2^24, part < 8
    const int32_t kb1 = static_cast<uint32_t>(P.nkb * (part + 1)) / P.split;
    const int32_t tiles = P.tiles_p * P.tiles_q;  // at most kMaxTiles
    const int32_t per_tile = CG == 2 ? 2 : P.split;  // CTAs of a cluster
    const int32_t first_tile = static_cast<int32_t>(blockIdx.x) / per_tile;
    const int32_t tile_step = static_cast<int32_t>(gridDim.x) / per_tile;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            ptx::mbar_init(ptx::smem_addr(&sh.full[s]), 1);
            ptx::mbar_init(ptx::smem_addr(&sh.empty[s]), F::kMmaGroups);
        }
        for (int g = 0; g < F::kMmaGroups; ++g) {
            for (int s = 0; s < F::kBuffers; ++s) {
                ptx::mbar_init(ptx::smem_addr(&sh.acc_full[s][g]), 1);
                ptx::mbar_init(ptx::smem_addr(&sh.acc_empty[s][g]), CG * F::kConsumerWarps / F::kMmaGroups);
            }
        }
        for (int s = 0; s < kScaleSlots; ++s) {
            ptx::mbar_init(ptx::smem_addr(&sh.scales_full[s]), 32);
            ptx::mbar_init(ptx::smem_addr(&sh.scales_empty[s]), F::kConsumerWarps);
        }
        sh.abort = 0;
        ptx::fence_mbar_init();
    }
    if (threadIdx.x == 32) {
        ptx::prefetch_tensormap(&map_p);
        ptx::prefetch_tensormap(&map_q);
    }
    if (warp == F::kConsumerWarps + 1) ptx::tmem_alloc<CG>(ptx::smem_addr(&sh.tmem), F::kTmemCols);
    ptx::tcgen05_fence_before();
    __syncthreads();
    if (CG == 2) ptx::cluster_sync();  // the other CTA's barriers are ready too
    ptx::tcgen05_fence_after();
    const uint32_t tmem = sh.tmem;
    // Only now that this grid has its tensor memory: a next grid that took some
    // first and then waited for this one would keep it from starting.
    ptx::let_next_grid_start();
    ptx::wait_previous_grid();  // nothing above touches global memory

    // A wait that gives up ends its role; the CTA's abort flag ends the
    // others. The first probes go without wait_phase's clock reads.
    auto wait_at = [&](uint32_t bar, uint32_t parity, uint32_t site) {
        for (int i = 0; i < 64; ++i)
            if (ptx::mbar_try_wait(bar, parity)) return true;
        const int w = wait_phase<false>(bar, parity, P.timeout_ns, abort_flag);
        if (w == WAIT_TIMEOUT) raise_timeout(P.status, site, abort_flag);
        return w == WAIT_OK;
    };
    auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t site) { return wait_at(ptx::smem_addr(bar), parity, site); };

    // For a whole warp: one lane asks, since 32 lanes' probes of a barrier are
    // served one after another and hold up every other barrier of the SM.
    auto warp_wait = [&](uint64_t* bar, uint32_t parity, uint32_t site) {
        bool ok = true;
        if (lane == 0) ok = wait(bar, parity, site);
        return __shfl_sync(0xffffffffu, static_cast<int>(ok), 0) != 0;
    };

    if (warp >= F::kConsumerWarps) {
        if (BN > 128) ptx::regs_less<F::kOtherRegs>();
        if (warp == F::kConsumerWarps) {
            if (ptx::elect_one()) {  // producer
                uint32_t it = 0;
                bool ready = true, ok = true;
                for (int32_t t = first_tile; t < tiles && ok; t += tile_step) {
                    int32_t tp, tq;
                    tile_at(P, t, &tp, &tq);
                    const int32_t p0 = (tp * CG + (CG == 2 ? static_cast<int32_t>(rank) : 0)) * kTile;
                    const int32_t q0 = tq * BN + (CG == 2 ? static_cast<int32_t>(rank) * F::kQBox : 0);
                    for (int32_t kb = kb0; kb < kb1; ++kb, ++it) {
                        const uint32_t s = it % STAGES;
                        if (!ready && !wait(&sh.empty[s], (it / STAGES - 1) & 1, SITE_MM_PRODUCER_EMPTY)) {
                            ok = false;
                            break;
                        }
                        uint32_t bar = ptx::smem_addr(&sh.full[s]);
                        // a pair's stage is complete when both CTAs' boxes
                        // have landed; the even CTA's barrier counts them all
                        if (rank == 0 || CG == 1) ptx::mbar_arrive_expect_tx(bar, CG * F::kStageBytes + P.tx_extra);
                        if (CG == 2) bar = ptx::mapa(bar, 0);
                        const uint32_t dst = ring + s * F::kStageBytes;
                        ptx::operand_g2s<CG>(dst, &map_p, kb * kTile, p0, bar);
#pragma unroll
                        for (int g = 0; g < F::kMmaGroups; ++g)
                            ptx::operand_g2s<CG>(dst + F::kPBytes + g * F::kQBytes, &map_q, kb * kTile, q0 + g * F::kMmaCols, bar);
                        const uint32_t next = it + 1;
                        ready = next < STAGES || ptx::mbar_test(ptx::smem_addr(&sh.empty[next % STAGES]), (next / STAGES - 1) & 1);
                    }
                }
                // Nothing may still be landing in this CTA's shared memory or
                // arriving on its barriers when it leaves: a stage is released
                // after its boxes have landed and been read.
                for (uint32_t i = it > STAGES ? it - STAGES : 0; i < it; ++i)
                    if (!drain_wait<false>(ptx::smem_addr(&sh.empty[i % STAGES]), (i / STAGES) & 1, P.timeout_ns, P.status,
                                           SITE_MM_DRAIN, abort_flag))
                        break;
            }
        } else if (warp - F::kConsumerWarps - 1 < F::kMmaGroups) {
            // Matrix instructions, a warp for each of those side by side: a block's accumulator and
            // stage barriers cost one thread more than the instructions take.
            const int g = warp - F::kConsumerWarps - 1;
            if ((CG == 1 || rank == 0) && ptx::elect_one()) {
                constexpr uint32_t idesc = ptx::e4m3_instr_desc(CG * kTile, F::kMmaCols);
                uint32_t it = 0, step = 0;
                bool ok = true;
                for (int32_t t = first_tile; t < tiles && ok; t += tile_step) {
                    for (int32_t kb = kb0; kb < kb1 && ok; ++step) {
                        const uint32_t buf = step % F::kBuffers, turn = step / F::kBuffers;
                        // both barriers are asked at once: an answer takes
                        // over 150 cycles
                        bool full = ptx::mbar_test(ptx::smem_addr(&sh.full[it % STAGES]), (it / STAGES) & 1);
                        if (turn > 0 && !wait(&sh.acc_empty[buf][g], (turn - 1) & 1, SITE_MM_MMA_ACC)) {
                            ok = false;
                            break;
                        }
#pragma unroll 1
                        for (int j = 0; j < F::kRun && kb < kb1; ++j, ++kb, ++it) {
                            const uint32_t s = it % STAGES;
                            if (!full && !wait(&sh.full[s], (it / STAGES) & 1, SITE_MM_MMA_FULL)) {
                                ok = false;
                                break;
                            }
                            if (j + 1 < F::kRun)
                                full = ptx::mbar_test(ptx::smem_addr(&sh.full[(it + 1) % STAGES]), ((it + 1) / STAGES) & 1);
                            ptx::tcgen05_fence_after();
                            const uint64_t dp = ptx::operand_desc(ring + s * F::kStageBytes);
                            const uint64_t dq = ptx::operand_desc(ring + s * F::kStageBytes + F::kPBytes + g * F::kQBytes);
#pragma unroll
                            for (int k = 0; k < kTile / kMmaK; ++k)
                                ptx::mma_e4m3<CG>(tmem + (buf * F::kRun + j) * BN + g * F::kMmaCols,
                                                  dp + k * (kMmaK >> 4), dq + k * (kMmaK >> 4), idesc, k > 0);
                            ptx::mma_commit<CG>(ptx::smem_addr(&sh.empty[s]));
                        }
                        if (ok) ptx::mma_commit<CG>(ptx::smem_addr(&sh.acc_full[buf][g]));
                    }
                }
            }
        } else if (warp == F::kConsumerWarps + 3) {
            // Scales, by 4-byte asynchronous copies: lane l brings block l % 8
            // of every fourth row, so that a copy touches four rows (a sector
            // or two each) whatever their alignment, and all of a run are in
            // flight at once.
            const int e = lane & 7, r4 = lane >> 3;
            uint32_t run = 0;
            bool ok = true;
            for (int32_t t = first_tile; t < tiles && ok; t += tile_step) {
                int32_t tp, tq;
                tile_at(P, t, &tp, &tq);
                const int64_t p0 = (static_cast<int64_t>(tp) * CG + (CG == 2 ? rank : 0)) * kTile;
                const int64_t q0 = static_cast<int64_t>(tq) * BN;
                for (int32_t kb = kb0; kb < kb1; kb += kScaleRun, ++run) {
                    const uint32_t slot = run % kScaleSlots;
                    ok = run < kScaleSlots || warp_wait(&sh.scales_empty[slot], (run / kScaleSlots - 1) & 1, SITE_MM_SCALES_EMPTY);
                    if (!ok) break;
                    const int32_t at = kb + e < kb1 ? kb + e : kb;  // past the end: any valid block
#pragma unroll 4
                    for (int i = 0; i < kTile; i += 4) {
                        const int64_t row = p0 + i + r4;
                        ptx::cp_async_ca4(ptx::smem_addr(&sh.row_scales[slot][e][i + r4]),
                                          P.p_scales + ((row < P.np ? row : P.np - 1) >> P.p_shift) * P.nkb + at);
                    }
                    if (PER_COL) {
#pragma unroll 4
                        for (int i = 0; i < BN; i += 4) {
                            const int64_t col = q0 + i + r4;
                            ptx::cp_async_ca4(ptx::smem_addr(&sh.col_scales[slot][e][PER_COL ? i + r4 : 0]),
                                              P.q_scales + (col < P.nq ? col : P.nq - 1) * P.nkb + at);
                        }
                    } else if (r4 < F::kGroups) {
                        const int64_t col = q0 + r4 * kCols;
                        ptx::cp_async_ca4(ptx::smem_addr(&sh.col_scales[slot][e][r4]),
                                          P.q_scales + (col < P.nq ? col : P.nq - 1) / kTile * P.nkb + at);
                    }
                    ptx::cp_async_mbar_arrive_noinc(ptx::smem_addr(&sh.scales_full[slot]));
                }
            }
            ptx::cp_async_wait_all();
        }
    } else {  // consumers
        if (BN > 128) ptx::regs_more<F::kConsumerRegs>();
        constexpr int kLoad = 16;  // columns of one load from tensor memory
        constexpr int kLoads = kCols / kLoad;
        const int group = warp / 4, quad = warp % 4;
        const int source = group * F::kMmaGroups / F::kGroups;  // the matrix instructions whose columns these are
        const int my_row = 32 * quad + lane;  // accumulator row of this thread, in the CTA's 128
        const uint32_t staging = ring + static_cast<uint32_t>(F::kRingBytes) + 32 * 128 * warp;
        // Where the walk over blocks stands, kept as offsets and parities that
        // step with it: the index arithmetic of a block would otherwise be a
        // quarter of its instructions.
        static_assert(kScaleSlots == 2, "two in turn");
        constexpr uint32_t kBarStep = 8 * F::kMmaGroups;  // from a buffer's barrier to the next
        const uint32_t full_bars = ptx::smem_addr(&sh.acc_full[0][source]), empty_bars = ptx::smem_addr(&sh.acc_empty[0][source]);
        const uint32_t free_bars = CG == 2 ? ptx::mapa(empty_bars, 0) : empty_bars;
        const uint32_t lanes = tmem + group * kCols + (static_cast<uint32_t>(32 * quad) << 16);
        const float* const row_scale = &sh.row_scales[0][0][my_row];
        const float* const col_scale = &sh.col_scales[0][0][PER_COL ? group * kCols : group];
        constexpr int kRowPitch = sizeof(sh.row_scales[0][0]) / 4, kColPitch = sizeof(sh.col_scales[0][0]) / 4;
        uint32_t buf = 0, phase = 0;   // accumulator, and its barrier's parity
        uint32_t spot = 0, scale_phase = 0;  // block's scales, kScaleRun a slot, and the slots' parity
        bool ok = true;
        for (int32_t t = first_tile; t < tiles; t += tile_step) {
            int32_t tp, tq;
            tile_at(P, t, &tp, &tq);
            float acc[kCols];
#pragma unroll
            for (int j = 0; j < kCols; ++j) acc[j] = 0.0f;
            // A warp takes the blocks one after another, so what it waits for
            // is taken off that path: the next accumulator's barrier is asked
            // before this one's sums, a load from tensor memory is under way
            // while the sums of the one before are taken, and nothing on the
            // path branches by lane. (A load carried over to the next block
            // costs a move a register; starting each block afresh is faster.)
            ok = ok && warp_wait(&sh.scales_full[spot / kScaleRun], scale_phase, SITE_MM_SCALES_FULL);
            ok = ok && warp_wait(&sh.acc_full[buf][source], phase, SITE_MM_CONSUMER_ACC);
            int j = 0;  // block of the accumulator
            for (int32_t left = kb1 - kb0; left > 0 && ok; --left) {
                const bool over = F::kRun == 1 || j == F::kRun - 1 || left == 1;  // the accumulator's last block
                const uint32_t at = lanes + (buf * F::kRun + j) * BN;
                const uint32_t next_buf = (buf + 1) % F::kBuffers, next_phase = phase ^ (next_buf == 0 ? 1u : 0u);
                float v[2][kLoad];
                ptx::tcgen05_fence_after();
                ptx::tmem_ld(at, v[0]);
                bool ready = false;
                float scale = row_scale[spot * kRowPitch];
                const float* const cols_at = col_scale + spot * kColPitch;
                if (!PER_COL) scale *= *cols_at;
#pragma unroll
                for (int g = 0; g < kLoads; ++g) {
                    ptx::tmem_wait_ld();
                    if (g + 1 < kLoads) {
                        ptx::tmem_ld(at + kLoad * (g + 1), v[(g + 1) % 2]);
                    } else if (over) {
                        // all of the accumulator is in registers: it is free
                        // before the last sums are taken
                        ptx::tcgen05_fence_before();
                        __syncwarp();
                        ptx::mbar_arrive_if<CG == 2>(lane == 0, free_bars + buf * kBarStep);
                        ready = ptx::mbar_test(full_bars + next_buf * kBarStep, next_phase);
                    }
#pragma unroll
                    for (int i = 0; i < kLoad; i += 4) {
                        const int col = kLoad * g + i;
                        float4 cs = make_float4(scale, scale, scale, scale);
                        if (PER_COL) {
                            cs = *reinterpret_cast<const float4*>(cols_at + col);
                            cs.x *= scale, cs.y *= scale, cs.z *= scale, cs.w *= scale;
                        }
                        acc[col] = ptx::fma_ordered(v[g % 2][i], cs.x, acc[col]);
                        acc[col + 1] = ptx::fma_ordered(v[g % 2][i + 1], cs.y, acc[col + 1]);
                        acc[col + 2] = ptx::fma_ordered(v[g % 2][i + 2], cs.z, acc[col + 2]);
                        acc[col + 3] = ptx::fma_ordered(v[g % 2][i + 3], cs.w, acc[col + 3]);
                    }
                }
                if (over) {
                    if (left > 1) {
                        if (!ready) ready = wait_at(full_bars + next_buf * kBarStep, next_phase, SITE_MM_CONSUMER_ACC);
                        ok = __all_sync(0xffffffffu, ready);
                    }
                    phase = next_phase;
                    buf = next_buf;
                }
                if (F::kRun > 1) j = over ? 0 : j + 1;
                ++spot;
                if (spot % kScaleRun == 0 || left == 1) {  // this run's scales have been read
                    const uint32_t slot = (spot - 1) / kScaleRun;
                    __syncwarp();
                    ptx::mbar_arrive_if<false>(lane == 0, ptx::smem_addr(&sh.scales_empty[slot]));
                    spot = (slot ^ 1) * kScaleRun;
                    scale_phase ^= slot;
                    if (left > 1 && ok)
                        ok = __all_sync(0xffffffffu, wait_at(ptx::smem_addr(&sh.scales_full[slot ^ 1]), scale_phase,
                                                             SITE_MM_SCALES_FULL));
                }
            }
            const int64_t row = (static_cast<int64_t>(tp) * CG + (CG == 2 ? rank : 0)) * kTile + my_row;
            const int64_t q0 = static_cast<int64_t>(tq) * BN + group * kCols;  // this group's first column
            if (CG == 1 && P.split > 1) {
                // this CTA's share, into the ring (every stage has been read:
                // the last accumulator is complete)
#pragma unroll
                for (int j = 0; j < kCols; j += 4) {
                    const int col = group * kCols + j;
                    if (SWAP) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (q0 + col + i < P.nq) st_shared(ring + 4 * ((col + i) * kTile + my_row), acc[j + i]);
                    } else {
                        st_shared4(ring + 4 * (my_row * F::kSharePitch + col), as_words(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]));
                    }
                }
            } else if (!SWAP) {
                // 32 rows x 128 bytes at a time through the warp's staging:
                // 16-byte units at the places the tensor map's swizzle gives
                // them, so a warp's writes meet no bank twice. They leave by a
                // bulk copy, or, where rows of c do not start on 16-byte
                // boundaries, a row after another by runs of single elements
                // (1764 x 2305 x 1141 to bf16: 15.4 us, 54.6 with a row a
                // thread)
                constexpr int kPiece = 128 / sizeof(C), kUnit = 16 / sizeof(C);
                if (ok) {
#pragma unroll
                    for (int piece = 0; piece < (SWAP ? 0 : kCols / kPiece); ++piece) {
                        if (lane == 0) ptx::bulk_wait_read<0>();  // the previous piece has left
                        __syncwarp();
#pragma unroll
                        for (int u = 0; u < 8; ++u) {
                            const int j = piece * kPiece + u * kUnit;
                            uint4 w;
                            if constexpr (sizeof(C) == 4)
                                w = as_words(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
                            else
                                w = make_uint4(pack2<C>(acc[j], acc[j + 1]), pack2<C>(acc[j + 2], acc[j + 3]),
                                               pack2<C>(acc[j + 4], acc[j + 5]), pack2<C>(acc[j + 6], acc[j + 7]));
                            st_shared4(staging + 128 * lane + 16 * (u ^ (lane & 7)), w);
                        }
                        const int64_t row0 = row - lane, col0 = q0 + piece * kPiece;
                        if (P.vec_c) {
                            ptx::fence_proxy_async_smem();
                            __syncwarp();
                            if (lane == 0 && row0 < P.np && col0 < P.nq) {
                                ptx::tensor_s2g_2d(&map_c, static_cast<int32_t>(col0), static_cast<int32_t>(row0), staging);
                                ptx::bulk_commit();
                            }
                        } else {
                            __syncwarp();
                            const int rows = static_cast<int>(P.np - row0 < 32 ? P.np - row0 : 32);  // may be negative
                            const int cols = static_cast<int>(P.nq - col0 < kPiece ? P.nq - col0 : kPiece);
                            C* out = static_cast<C*>(P.c) + (row0 * P.ldc + col0);
#pragma unroll 2
                            for (int i = 0; i < rows; ++i, out += P.ldc) {
#pragma unroll
                                for (int e = lane; e < kPiece; e += 32) {
                                    const int at = e * static_cast<int>(sizeof(C));
                                    const C v = ld_shared<C>(staging + 128 * i + ((at & ~15) ^ (16 * (i & 7))) + (at & 15));
                                    if (e < cols) out[e] = v;
                                }
                            }
                        }
                    }
                }
            } else if (ok && row < P.np) {  // the threads of a warp write 32 neighbours of one row of c
                C* out = static_cast<C*>(P.c) + q0 * P.ldc + row;
#pragma unroll
                for (int j = 0; j < kCols; ++j)
                    if (j < P.nq - q0) out[j * P.ldc] = from_f32<C>(acc[j]);
            }
        }
        if (!SWAP && lane == 0) ptx::bulk_wait_all();
    }
    __syncwarp();  // the one-thread roles' idle lanes wait here
    ptx::tcgen05_fence_before();
    __syncthreads();
    ptx::tcgen05_fence_after();
    if (CG == 2) ptx::cluster_sync();  // neither CTA's memory goes while the other may still use or signal it
    if (warp == F::kConsumerWarps + 1) ptx::tmem_dealloc<CG>(tmem, F::kTmemCols);
    if (CG == 1 && P.split > 1) {
        ptx::cluster_sync();  // every share is written
        if (warp < F::kConsumerWarps && !*abort_flag) {
            int32_t tp, tq;
            tile_at(P, first_tile, &tp, &tq);
            const int64_t p0 = static_cast<int64_t>(tp) * kTile, q0 = static_cast<int64_t>(tq) * BN;
            const int cols = static_cast<int>(P.nq - q0 < BN ? P.nq - q0 : BN);
            const int rows = static_cast<int>(P.np - p0 < kTile ? P.np - p0 : kTile);
            if (SWAP) {  // a thread a value, neighbours of one row of c side by side
                const int all = cols * kTile;
                for (int i = all * part / P.split + threadIdx.x; i < all * (part + 1) / P.split; i += 32 * F::kConsumerWarps) {
                    float w[kMaxSplit];
#pragma unroll
                    for (int r = 0; r < kMaxSplit; ++r) w[r] = r < P.split ? ptx::cluster_ld(ptx::mapa(ring + 4 * i, r)) : 0.0f;
                    float v = w[0];
#pragma unroll
                    for (int r = 1; r < kMaxSplit; ++r) v += w[r];
                    const int row = i % kTile, c = i / kTile;
                    if (row < rows) static_cast<C*>(P.c)[(q0 + c) * P.ldc + p0 + row] = from_f32<C>(v);
                }
            } else {  // four values a thread, 16 or 32 neighbouring threads a row
                constexpr int kQuads = BN / 4;
                const int all = rows * kQuads;
                for (int i = all * part / P.split + threadIdx.x; i < all * (part + 1) / P.split; i += 32 * F::kConsumerWarps) {
                    const int row = i / kQuads, c = i % kQuads * 4;
                    float4 v = make_float4(0, 0, 0, 0);
#pragma unroll
                    for (int r = 0; r < kMaxSplit; ++r) {
                        if (r >= P.split) break;
                        const float4 w = ptx::cluster_ld4(ptx::mapa(ring + 4 * (row * F::kSharePitch + c), r));
                        v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
                    }
                    C* out = static_cast<C*>(P.c) + (p0 + row) * P.ldc + q0 + c;
                    if (P.vec_c && c + 4 <= cols) {
                        store4(out, v);
                    } else {
                        const float u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (c + e < cols) out[e] = from_f32<C>(u[e]);
                    }
                }
            }
        }
        __syncwarp();         // lanes' loops above differ in length, and the barrier takes whole warps
        ptx::cluster_sync();  // every share has been read
    }
}

// A matrix of rows x cols elements as boxes of 128 bytes by box_rows rows, in
// the swizzle of that width.
bool box_map(CUtensorMap* map, CUtensorMapDataType type, const void* p, int64_t size, int64_t rows, int64_t cols, int64_t ld,
             uint32_t box_rows) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld * size)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(128 / size), box_rows};
    const cuuint32_t estr[2] = {1, 1};
    auto encode = tensor_map_encoder();
    return encode != nullptr &&
           encode(map, type, 2, const_cast<void*>(p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Launch configuration of a form's grid in clusters.
struct Launch {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[2];
    Launch(int64_t grid, int threads, size_t smem, int cluster, cudaStream_t stream) {
        cfg.gridDim = dim3(static_cast<unsigned>(grid));
        cfg.blockDim = dim3(static_cast<unsigned>(threads));
        cfg.dynamicSmemBytes = smem;
        cfg.stream = stream;
        attr[0] = early_start();
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = cluster > 1 ? 2 : 1;
    }
};

// CTAs of a cluster that share a tile's k: as many (up to 8, each with at
// least two blocks of k) as leave every tile's cluster resident at once. The
// SMs of a GPC bound that: one-CTA-an-SM clusters of 4 and 6 leave 144 and 138
// of the 152 SMs usable, 7 and 8 only 105 and 120. (128 x 2048 x 8192, 16
// tiles: 24.4 us unsplit, 14.5 split 6, 20.3 split 8 in two waves.)
// The occupancy call counts one CTA an SM for kernels that use tensor memory;
// `ctas` is what their tensor memory, registers and shared memory allow.
template <typename K>
int split_for(K kernel, int threads, size_t smem, int ctas, std::atomic<int> (&resident)[kMaxSplit + 1], int64_t tiles,
              int64_t nkb) {
    for (int split = static_cast<int>(std::min<int64_t>(kMaxSplit, nkb / 2)); split > 1; --split) {
        int n = resident[split].load();
        if (n == 0) {
            Launch l(split, threads, smem, split, nullptr);
            int per_sm = 0;
            if (cudaOccupancyMaxActiveClusters(&n, kernel, &l.cfg) != cudaSuccess ||
                cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, smem) != cudaSuccess || per_sm < 1)
                n = 0;
            else if (per_sm < ctas)
                n = n * ctas / per_sm;
            n += 1;  // 0: not asked yet
            resident[split] = n;
        }
        if (tiles <= n - 1) return split;
    }
    return 1;
}

template <typename C, int BN, int CG, int STAGES, bool PER_COL, bool SWAP>
ap_status launch_form(const DeviceInfo& di, MatmulParams P, const MatmulArgs& a, cudaStream_t stream) {
    using F = Form<BN, CG, STAGES, PER_COL, SWAP>;
    static_assert(F::kCtas * (F::kSmem + sizeof(Shared<F, STAGES, PER_COL>) + 1024) <= kSmemPerSM, "shared memory of an SM");
    static_assert(F::kCtas * F::kTmemCols <= 512, "tensor memory of an SM");
    static_assert(F::kTmemCols >= 32 && (F::kTmemCols & (F::kTmemCols - 1)) == 0, "columns that can be allocated");
    static_assert(((F::kBuffers - 1) * F::kRun + F::kRun - 1) * BN + (F::kMmaGroups - 1) * F::kMmaCols + F::kMmaCols <= F::kTmemCols,
                  "the last accumulator's last columns are allocated");
    static_assert(F::kMmaCols % 16 == 0 && F::kMmaCols <= 256 && F::kCols % 16 == 0, "columns of an instruction, of a load");
    static_assert(F::kPBytes % 1024 == 0 && F::kQBytes % 1024 == 0 && F::kStageBytes % 1024 == 0, "operands start on swizzle atoms");
    static_assert(F::kQBox <= 256 && F::kQBox * CG * F::kMmaGroups == BN, "boxes cover the tile's columns");
    static_assert(1023 + F::kRingBytes + F::kStagingBytes <= F::kSmem, "ring and staging from the first 1024-byte boundary on");
    static_assert(CG == 2 || (SWAP ? size_t(BN) * kTile * 4 : F::kShareBytes) <= F::kRingBytes, "a share fits in the ring");
    static_assert(F::kShareBytes >= ((kTile - 1) * size_t(F::kSharePitch) + BN) * 4, "a share's last value");
    static_assert(sizeof(Shared<F, STAGES, PER_COL>::col_scales[0][0]) % 16 == 0 &&
                      sizeof(Shared<F, STAGES, PER_COL>::col_scales[0][0]) >= 4 * size_t(PER_COL ? F::kGroups * F::kCols : F::kGroups),
                  "a block's column scales, in whole 16-byte loads");
    P.np = SWAP ? a.n : a.m;
    P.nq = SWAP ? a.m : a.n;
    P.p_scales = SWAP ? a.b_scales : a.a_scales;
    P.q_scales = SWAP ? a.a_scales : a.b_scales;
    P.p_shift = SWAP && a.b_block_rows != 1 ? 7 : 0;
    const int64_t tiles_p = (P.np + CG * kTile - 1) / (CG * kTile), tiles_q = (P.nq + BN - 1) / BN;
    const int64_t tiles = tiles_p * tiles_q;
    if (tiles > kMaxTiles) return AP_ERR_SHAPE;
    P.tiles_p = static_cast<int32_t>(tiles_p);
    P.tiles_q = static_cast<int32_t>(tiles_q);
    auto kernel = matmul_fp8_kernel<C, BN, CG, STAGES, PER_COL, SWAP>;
    static std::atomic<int> configured[64];  // attribute set on this device (setting twice is harmless)
    static std::atomic<int> resident[64][kMaxSplit + 1];
    if (di.device < 0 || di.device >= 64) return AP_ERR_CUDA;
    if (!configured[di.device].load()) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(F::kSmem)) !=
            cudaSuccess)
            return AP_ERR_CUDA;
        configured[di.device] = 1;
    }
    P.split = CG == 2 ? 1 : split_for(kernel, F::kThreads, F::kSmem, F::kCtas, resident[di.device], tiles, P.nkb);
    CUtensorMap mp, mq, mc{};
    constexpr auto codes = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    if (!box_map(&mp, codes, SWAP ? a.b : a.a, 1, P.np, a.k, SWAP ? a.ldb : a.lda, kTile) ||
        !box_map(&mq, codes, SWAP ? a.a : a.b, 1, P.nq, a.k, SWAP ? a.lda : a.ldb, F::kQBox))
        return AP_ERR_CUDA;
    if (!SWAP && P.split == 1 && P.vec_c &&
        !box_map(&mc, sizeof(C) == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16, a.c, sizeof(C), a.m,
                 a.n, a.ldc, 32))
        return AP_ERR_CUDA;
    const int cluster = CG == 2 ? 2 : P.split;
    int64_t grid = tiles * cluster;
    if (P.split == 1) grid = std::min<int64_t>(grid, di.sms * F::kCtas / cluster * cluster);
    record_launch(PATH_MATMUL, grid, BN, static_cast<int64_t>(F::kSmem), STAGES,
                  (SWAP ? 1 : 0) | (CG == 2 ? 2 : 0) | P.split << 4);
    Launch l(grid, F::kThreads, F::kSmem, cluster, stream);
    return cudaLaunchKernelEx(&l.cfg, kernel, mp, mq, mc, P) == cudaSuccess ? AP_OK : AP_ERR_CUDA;
}

template <typename C>
ap_status launch_mm(const DeviceInfo& di, const MatmulParams& P, const MatmulArgs& a, cudaStream_t stream) {
    const bool rows = a.b_block_rows == 1;
    // Few rows: the weight on the accumulator's rows, a's rows padded to 16 or
    // 32 (times 8192 x 8192: one row 14.9 us, 15.4 padded to 32; 32 rows 17.0,
    // 48 in the 128 x 128 form 18.7).
    if (a.m <= 16) return launch_form<C, 16, 1, 5, true, true>(di, P, a, stream);
    if (a.m <= 32) return launch_form<C, 32, 1, 4, true, true>(di, P, a, stream);
    // Pairs from half the SMs' worth of their tiles on (8192^3: 440 us against
    // 596 one CTA a tile; 1024 x 2560 x 4096, 40 pairs: 19.0 against 25.5; the
    // other way 333 x 4104 x 5000, 34 pairs: 18.6 against 22.5), but not for
    // rows that one CTA's tile holds (64 x 16384 x 8192: 28.3 us against 33.8 in
    // pairs).
    const int64_t pairs = (a.m + 2 * kTile - 1) / (2 * kTile) * ((a.n + 255) / 256);
    if (a.m > kTile && pairs >= di.sms / 4)
        return rows ? launch_form<C, 256, 2, 5, true, false>(di, P, a, stream)
                    : launch_form<C, 256, 2, 5, false, false>(di, P, a, stream);
    return rows ? launch_form<C, 128, 1, 5, true, false>(di, P, a, stream)
                : launch_form<C, 128, 1, 5, false, false>(di, P, a, stream);
}

}  // namespace

ap_status launch_matmul_fp8(const DeviceInfo& di, const Options& o, const MatmulArgs& a, cudaStream_t stream) {
    const int64_t size = a.c_type == AP_F32 ? 4 : 2;
    if (a.k == 0) {  // all zeros
        const size_t pitch = static_cast<size_t>(a.ldc * size), width = static_cast<size_t>(a.n * size);
        if (pitch <= INT32_MAX)  // the largest pitch that a 2-D call takes
            return cudaMemset2DAsync(a.c, pitch, 0, width, static_cast<size_t>(a.m), stream) == cudaSuccess ? AP_OK : AP_ERR_CUDA;
        for (int64_t i = 0; i < a.m; ++i)
            if (cudaMemsetAsync(static_cast<char*>(a.c) + i * pitch, 0, width, stream) != cudaSuccess) return AP_ERR_CUDA;
        return AP_OK;
    }
    MatmulParams P{};
    P.c = a.c;
    P.ldc = a.ldc;
    P.nkb = static_cast<int32_t>((a.k + kTile - 1) / kTile);
    P.vec_c = rows_aligned(a.c, a.ldc, size, 16);
    P.tx_extra = static_cast<uint32_t>(o.tx_extra);
    P.timeout_ns = static_cast<uint64_t>(o.timeout_ns);
    P.status = di.status;
    switch (a.c_type) {
        case AP_BF16: return launch_mm<__nv_bfloat16>(di, P, a, stream);
        case AP_F16: return launch_mm<__half>(di, P, a, stream);
        default: return launch_mm<float>(di, P, a, stream);
    }
}

}  // namespace ap
