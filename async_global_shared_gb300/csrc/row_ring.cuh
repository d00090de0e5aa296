// Shared by the norm and its gradient: sums over a row, and the ring that
// streams whole rows of several matrices through shared memory.
#pragma once

#include <algorithm>
#include <atomic>

#include "device_common.cuh"
#include "fp8_common.cuh"
#include "internal.h"

namespace ap {
namespace {

// Sum over the threads that hold one row: a warp, or the whole CTA (every
// warp adds the warps' sums in the same order, so all threads get one value).
template <bool WARP>
__device__ __forceinline__ float row_sum(float v, float* scratch) {
    v = warp_sum(v);
    if (WARP) return v;
    const int warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    v = (threadIdx.x & 31) < warps ? scratch[threadIdx.x & 31] : 0.0f;
    return warp_sum(v);
}

// How a warp's 256 columns of a row lie in its threads, eight elements each.
// Whole rows (every matrix's rows on 16-byte boundaries, a multiple of eight
// columns): lane l has columns 8 l .. 8 l + 7 and moves them 16 bytes at a
// time. SPREAD, for all others: columns l, l + 32, ..., so that a warp's access
// to single elements still is one run of memory. (8287 x 166 floats: gradient
// 37 us with eight neighbours a thread and plain accesses.)
template <bool SPREAD>
__device__ __forceinline__ int first_column(int thread) {
    return SPREAD ? 8 * (thread & ~31) + (thread & 31) : 8 * thread;
}

// A thread's eight elements of a row's chunk at p, zeros past the row's end:
// `left` columns from p's on, p's own among them.
template <bool SPREAD, typename T>
__device__ __forceinline__ void take(const T* p, int left, float (&v)[8]) {
    if (!SPREAD && left > 0) {
        load8(p).unpack(v);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = SPREAD && 32 * i < left ? to_f32(p[32 * i]) : 0.0f;
}
template <bool SPREAD, typename T>
__device__ __forceinline__ void put(T* p, int left, const float (&v)[8]) {
    if (!SPREAD) {
        if (left > 0) store8(p, v);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (32 * i < left) p[32 * i] = from_f32<T>(v[i]);
}
template <bool SPREAD, typename T>
__device__ __forceinline__ void take_weight(const void* w, bool same, int col, int left, float (&v)[8]) {
    if (same)
        take<SPREAD>(static_cast<const T*>(w) + col, left, v);
    else
        take<SPREAD>(static_cast<const float*>(w) + col, left, v);
}

// ------------------------------------------------------------------ ring of rows
//
// Calls with many rows run a persistent CTA an SM: a producer thread streams
// whole rows of every input through a ring of shared-memory stages (one bulk
// copy a row and input, or one for all of a stage where rows follow each
// other without gaps), and 16 consumer warps take them from there. A row's
// sum makes every thread wait for every other once a row; with the next rows
// already on their way that wait costs no bandwidth.
//
// A row belongs to a team of warps, two to four chunks of eight elements a
// thread. A stage holds `turns` rows for each of `together` teams: one team
// where rows are large, so that a stage's place is filled again as soon as that
// team is done, all of them where rows are small, so that the producer has few
// stages to fill. Stage j of a CTA belongs to the teams' group j mod (teams /
// together) and holds the rows from (j * grid + CTA) * together * turns, turn
// m's row for the group's team t being m * together + t.
//
// A bulk copy moves whole 16-byte units. Rows that do not start or end on such
// a boundary bring the units they share with their neighbours whole and keep
// their place in a unit in shared memory; at the first and the last row, where
// a unit's other bytes may not be the matrix's, the producer moves the row's
// bytes of it itself.
constexpr int kRingWarps = 16;
constexpr int kRingThreads = 32 * (kRingWarps + 1);
constexpr int kMaxRingStages = 32;
constexpr int64_t kRingBytes = 200 * 1024;
constexpr int kMaxInputs = 3;

struct RowRing {
    const unsigned char* in[kMaxInputs];
    int64_t pitch[kMaxInputs];
    uint32_t bytes[kMaxInputs];   // of a row
    uint32_t apart[kMaxInputs];   // between a stage's rows
    uint32_t offset[kMaxInputs];  // of an input's rows in a stage
    const float* side;      // one float a row as well, or nullptr
    uint32_t side_offset;   // of their places in a stage
    uint32_t weight_offset; // of the weight in floats, past the stages
    uint32_t stage_bytes;
    uint32_t smem;          // all of it
    bool keep_weights, spread;
    int inputs, chunks, team_warps, teams, together, turns, stages;
    int64_t rows;
    uint32_t tx_extra;  // fault injection: bytes every stage waits for in vain
    int give_up;        // fault injection: the consumer warp, from 1, whose first wait gives up
    uint64_t timeout_ns;
    uint32_t* status;
};

struct RingBars {
    uint64_t full[kMaxRingStages], empty[kMaxRingStages];
    int abort;
};

__device__ __forceinline__ void ring_init(const RowRing& R, RingBars& b) {
    if (threadIdx.x == 0) {
        for (int s = 0; s < R.stages; ++s) {
            ptx::mbar_init(ptx::smem_addr(&b.full[s]), R.side != nullptr ? 33 : 1);
            ptx::mbar_init(ptx::smem_addr(&b.empty[s]), static_cast<uint32_t>(R.together * R.team_warps));
        }
        b.abort = 0;
        ptx::fence_mbar_init();
    }
    __syncthreads();
    ptx::wait_previous_grid();  // nothing before this touches global memory
}

__device__ __forceinline__ bool ring_wait(const RowRing& R, RingBars& b, uint64_t* bar, uint32_t parity, uint32_t site) {
    for (int i = 0; i < 64; ++i)
        if (ptx::mbar_try_wait(ptx::smem_addr(bar), parity)) return true;
    const int w = wait_phase<false>(ptx::smem_addr(bar), parity, R.timeout_ns, &b.abort);
    if (w == WAIT_TIMEOUT) raise_timeout(R.status, site, &b.abort);
    return w == WAIT_OK;
}

// A consumer warp's wait for stage s, one lane asking.
__device__ __forceinline__ bool stage_arrived(const RowRing& R, RingBars& b, int s, uint32_t round) {
    bool ok = true;
    if ((threadIdx.x & 31) == 0) {
        ok = R.give_up != static_cast<int>(threadIdx.x >> 5) + 1 && ring_wait(R, b, &b.full[s], round & 1, SITE_ROWS_CONSUMER);
        if (!ok) raise_timeout(R.status, SITE_ROWS_CONSUMER, &b.abort);
    }
    return __shfl_sync(0xffffffffu, static_cast<int>(ok), 0) != 0;
}

// Where a stage's row `slot` of input i lies in the input's part of the stage
// that starts with row `base`.
template <bool SPREAD>
__device__ __forceinline__ uint32_t row_place(const RowRing& R, int i, int64_t base, int slot) {
    const uint32_t at = slot * R.apart[i];
    if (!SPREAD) return at;
    const int64_t row = R.apart[i] == R.bytes[i] ? base : base + slot;
    return at + (static_cast<uint32_t>(reinterpret_cast<uintptr_t>(R.in[i]) + row * R.pitch[i]) & 15u);
}

// Brings bytes [from, to) of an input to dst, which has the place in a 16-byte
// unit that `from` has; [first, last) are the input's own bytes. What the
// barrier is to expect is told it here, its arrival is the caller's.
__device__ __forceinline__ void copy_units(uint32_t dst, const unsigned char* from, const unsigned char* to,
                                           const unsigned char* first, const unsigned char* last, uint32_t bar) {
    const auto down = [](const unsigned char* p) { return p - (reinterpret_cast<uintptr_t>(p) & 15); };
    const auto up = [&](const unsigned char* p) { return down(p + 15); };
    const auto by_hand = [&](const unsigned char* a, const unsigned char* b) {
        for (; a < b; a += 2)
            ptx::st_shared_u16(dst + static_cast<uint32_t>(a - from), *reinterpret_cast<const uint16_t*>(a));
    };
    const unsigned char* lo = down(from) >= first ? down(from) : up(from);
    const unsigned char* hi = up(to) <= last ? up(to) : down(to);
    if (lo >= hi) lo = hi = to;  // no whole unit
    by_hand(from, lo);
    if (hi > lo) {
        by_hand(hi, to);
        ptx::mbar_expect_tx(bar, static_cast<uint32_t>(hi - lo));
        ptx::bulk_g2s(dst + static_cast<uint32_t>(lo - from), lo, static_cast<uint32_t>(hi - lo), bar);
    }
}

// The producer warp: lane 0 issues the rows' copies, all lanes the side
// values' (4 bytes each, per-thread asynchronous copies on the same barrier).
__device__ __forceinline__ void ring_produce(const RowRing& R, RingBars& b, uint32_t smem) {
    const int lane = threadIdx.x & 31;
    const int64_t step = R.together * R.turns;
    uint32_t row_bytes = 0;
    for (int i = 0; i < R.inputs; ++i) row_bytes += R.bytes[i];
    int s = 0;
    uint32_t round = 0;
    int64_t issued = 0;
    for (int64_t row = blockIdx.x * step; row < R.rows; row += gridDim.x * step, ++issued) {
        bool ok = true;
        if (round > 0 && lane == 0) ok = ring_wait(R, b, &b.empty[s], (round - 1) & 1, SITE_ROWS_PRODUCER);
        if (!__shfl_sync(0xffffffffu, static_cast<int>(ok), 0)) break;
        const int n = static_cast<int>(R.rows - row < step ? R.rows - row : step);
        const uint32_t bar = ptx::smem_addr(&b.full[s]);
        const uint32_t stage = smem + s * R.stage_bytes;
        if (lane == 0 && R.spread) {
            for (int i = 0; i < R.inputs; ++i) {
                const unsigned char* src = R.in[i] + row * R.pitch[i];
                const unsigned char* last = R.in[i] + ((R.rows - 1) * R.pitch[i] + R.bytes[i]);
                const bool one = R.apart[i] == R.bytes[i];  // rows without gaps: one span
                for (int k = 0; k < (one ? 1 : n); ++k, src += R.pitch[i])
                    copy_units(stage + R.offset[i] + row_place<true>(R, i, row, k), src, src + (one ? n : 1) * R.bytes[i], R.in[i],
                               last, bar);
            }
            ptx::fence_proxy_async_smem();  // places filled by hand are copied over later
            ptx::mbar_arrive_expect_tx(bar, R.tx_extra);
        } else if (lane == 0) {
            ptx::mbar_arrive_expect_tx(bar, static_cast<uint32_t>(n) * row_bytes + R.tx_extra);
            for (int i = 0; i < R.inputs; ++i) {
                const uint32_t dst = stage + R.offset[i];
                const unsigned char* src = R.in[i] + row * R.pitch[i];
                if (R.pitch[i] == R.bytes[i]) {
                    ptx::bulk_g2s(dst, src, static_cast<uint32_t>(n) * R.bytes[i], bar);
                } else {
                    for (int k = 0; k < n; ++k)
                        ptx::bulk_g2s(dst + static_cast<uint32_t>(k) * R.bytes[i], src + k * R.pitch[i], R.bytes[i], bar);
                }
            }
        }
        __syncwarp();
        if (R.side != nullptr) {
            for (int k = lane; k < n; k += 32) ptx::cp_async_ca4(stage + R.side_offset + 4 * k, R.side + row + k);
            ptx::cp_async_mbar_arrive_noinc(bar);
        }
        if (++s == R.stages) s = 0, ++round;
    }
    ptx::cp_async_wait_all();
    // after an abort, copies may still be landing
    if (lane == 0 && *static_cast<volatile int*>(&b.abort)) {
        for (int64_t i = issued > R.stages ? issued - R.stages : 0; i < issued; ++i)
            if (!drain_wait<false>(ptx::smem_addr(&b.full[i % R.stages]), static_cast<uint32_t>(i / R.stages) & 1, R.timeout_ns,
                                   R.status, SITE_ROWS_DRAIN, &b.abort))
                break;
    }
}

// Sum over a team's warps, the same value in all its threads. `scratch` is the
// team's, one of two used in turn, so one barrier a sum is enough.
__device__ __forceinline__ float team_sum(float v, float* scratch, int team, int warps) {
    v = warp_sum(v);
    if (warps == 1) return v;
    const int lane = threadIdx.x & 31;
    if (lane == 0) scratch[(threadIdx.x >> 5) - team * warps] = v;
    ptx::named_barrier_sync(1 + team, 32 * warps);
    v = lane < warps ? scratch[lane] : 0.0f;
    return warp_sum(v);
}

// For a warp that gave up its wait for the stage whose first row of the team
// is `row`. Its team mates may have had their answer a moment before or after
// and count on it at the team's barriers, so it stays for the sums of all the
// rows that are left to them, stages `apart` rows apart; its part is NaN, and
// so is what they make of such a row.
__device__ __forceinline__ void attend_sums(const RowRing& R, float (*scratch)[kRingWarps], int team, int64_t row, int64_t apart,
                                            int turn) {
    if (R.team_warps == 1) return;
    for (; row < R.rows; row += apart)  // (the last stage's turns past the end have no sum)
        for (int m = 0; m < R.turns; ++m, turn ^= 1)
            if (row + m * R.together < R.rows)
                team_sum(__int_as_float(0x7fc00000), &scratch[turn][team * R.team_warps], team, R.team_warps);
}

// Fill in the plan for rows of `cols` elements; false where the ring does not
// take these rows (width). whole: the inputs' rows start on 16-byte boundaries
// and hold a multiple of eight columns.
bool plan_ring(const DeviceInfo& di, const Options& o, RowRing* R, int inputs, const void* const* in, const int64_t* ld,
               const int64_t* size, const float* side, int64_t rows, int64_t cols, bool whole) {
    if (cols > 256 * 4 * kRingWarps) return false;
    R->spread = !whole;
    R->side = side;
    R->tx_extra = static_cast<uint32_t>(o.tx_extra);
    R->give_up = static_cast<int>(o.give_up);
    R->timeout_ns = static_cast<uint64_t>(o.timeout_ns);
    R->status = di.status;
    R->inputs = inputs;
    R->rows = rows;
    int64_t row_bytes = 0;
    for (int i = 0; i < inputs; ++i) {
        R->in[i] = static_cast<const unsigned char*>(in[i]);
        R->pitch[i] = ld[i] * size[i];
        R->bytes[i] = static_cast<uint32_t>(cols * size[i]);
        R->apart[i] = whole || R->pitch[i] == R->bytes[i] ? R->bytes[i] : (R->bytes[i] + 31) / 16 * 16;
        row_bytes += cols * size[i];
    }
    // A thread's chunks of eight elements: what leaves fewest of the 16 warps
    // without a whole row (rows of 5000: ten busy with two chunks, 15 with
    // four). Of equals the norm takes the most chunks, so that several teams'
    // rows overlap (16384 x 4096: 72 us with four chunks, 81 with two), unless
    // rows are short; the gradient the fewest, whose weights and sums stay in
    // registers (16384 x 8192: 158 against 244 us). A plan whose stages do not
    // fit twice for every group of teams gives way to the next.
    const auto warps = [&](int64_t c) { return (cols + 256 * c - 1) / (256 * c); };
    const auto busy = [&](int64_t c) { return warps(c) > kRingWarps ? 0.0 : double(cols * (kRingWarps / warps(c))) / double(c); };
    int order[3] = {2, 3, 4};
    const bool most = side == nullptr && cols > 1024;
    std::stable_sort(order, order + 3, [&](int a, int b) { return busy(a) != busy(b) ? busy(a) > busy(b) : most && a > b; });
    for (int k = 0; k < 6; ++k) {
        const int c = order[k % 3];
        if (warps(c) > kRingWarps) continue;
        R->chunks = c;
        R->team_warps = static_cast<int>(warps(c));
        R->teams = kRingWarps / R->team_warps;
        R->together = side == nullptr && row_bytes >= 16 * 1024 ? 1 : R->teams;
        // stages of about 24 KiB, at most eight rows a team, fewer where that
        // would leave CTAs without one
        const int64_t group = row_bytes * R->together;
        R->turns = static_cast<int>(std::max<int64_t>(1, std::min({int64_t(8), 24 * 1024 / group, rows / (di.sms * R->teams)})));
        uint32_t at = 0;
        for (int i = 0; i < inputs; ++i) {
            R->offset[i] = at;
            at += R->apart[i] * static_cast<uint32_t>(R->together * R->turns);
            if (!whole) at = (at + 31) / 16 * 16;
        }
        R->side_offset = at;
        if (side != nullptr) at += static_cast<uint32_t>(4 * R->together * R->turns + 15) / 16 * 16;
        R->stage_bytes = at;
        // A place of the ring always belongs to the same group, whose waits
        // on its barrier then follow one another phase by phase: the stages
        // are a multiple of the groups.
        const int groups = R->teams / R->together;
        // Weights that two chunks do not hold in registers: in shared memory,
        // or, where no plan leaves room for them, read again from the L2
        // (32768 x 8192 with a 32-bit residual: 512 us, 431 with two chunks).
        const int64_t weights = c > 2 && k < 3 ? 4 * cols : 0;
        if (kRingBytes < weights || (c == 2 && k >= 3)) continue;
        R->keep_weights = weights > 0;
        R->stages = static_cast<int>(std::min<int64_t>(kMaxRingStages, (kRingBytes - weights) / at)) / groups * groups;
        R->weight_offset = static_cast<uint32_t>(R->stages) * at;
        R->smem = R->weight_offset + static_cast<uint32_t>(weights);
        if (R->stages >= 2 * groups) return true;
    }
    return false;
}

// CTAs of a ring kernel: one an SM, each with at least one stage of rows, and
// no more than the caller's cap (0: none).
int64_t ring_grid(const RowRing& R, int64_t sms, int64_t cap) {
    const int64_t step = R.together * R.turns;
    const int64_t grid = std::min(sms, (R.rows + step - 1) / step);
    return cap > 0 ? std::min(grid, cap) : grid;
}

// The weight in floats, by the 16 consumer warps.
template <typename T>
__device__ __forceinline__ void stage_weights(const void* w, bool same, int64_t cols, float* out) {
    for (int j = threadIdx.x; j < cols; j += 32 * kRingWarps)
        out[j] = same ? to_f32(static_cast<const T*>(w)[j]) : static_cast<const float*>(w)[j];
    ptx::named_barrier_sync(15, 32 * kRingWarps);
}

// Where a ring kernel's threads have their columns' weights: in registers (two
// chunks), in shared memory, or in the L2 where shared memory is full.
enum Weights { IN_REGISTERS, IN_SHARED, IN_L2 };

// Weights of a chunk that are not in registers.
template <typename T, Weights W, bool SPREAD, typename Params>
__device__ __forceinline__ void again_weight(const Params& P, const float* kept, int col, int left, float (&v)[8]) {
    if (W == IN_SHARED)
        take<SPREAD>(kept + col, left, v);
    else
        take_weight<SPREAD, T>(P.a.weight, P.a.weight_type == P.a.type, col, left, v);
}

constexpr int64_t kMaxGrid = int64_t(1) << 31;

// Launch of a persistent ring kernel of `grid` CTAs with its shared memory.
template <typename K, typename Params>
ap_status launch_ring_kernel(const DeviceInfo& di, K kernel, std::atomic<int> (&configured)[64], const Params& P,
                             const RowRing& ring, int64_t grid, int64_t path, cudaStream_t stream) {
    if (di.device < 0 || di.device >= 64) return AP_ERR_CUDA;
    if (!configured[di.device].load()) {  // attribute set on this device (setting twice is harmless)
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kRingBytes)) !=
            cudaSuccess)
            return AP_ERR_CUDA;
        configured[di.device] = 1;
    }
    const size_t smem = ring.smem;
    record_launch(path, grid, ring.together * ring.turns, static_cast<int64_t>(smem), ring.stages, 4 | (ring.spread ? 8 : 0));
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kRingThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr = early_start();
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, P, ring) == cudaSuccess ? AP_OK : AP_ERR_CUDA;
}

}  // namespace
}  // namespace ap
