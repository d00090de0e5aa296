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

template <typename T>
__device__ __forceinline__ void load_weight(const void* w, bool same, int64_t col, float (&v)[8]) {
    if (same)
        load8(static_cast<const T*>(w) + col).unpack(v);
    else
        load8(static_cast<const float*>(w) + col).unpack(v);
}
template <typename T>
__device__ __forceinline__ void load_weight(const void* w, bool same, bool vec, int64_t col, int64_t n, float (&v)[8]) {
    if (same)
        load8(static_cast<const T*>(w) + col, vec, n).unpack(v);
    else
        load8(static_cast<const float*>(w) + col, vec, n).unpack(v);
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
constexpr int kRingWarps = 16;
constexpr int kRingThreads = 32 * (kRingWarps + 1);
constexpr int kMaxRingStages = 32;
constexpr int64_t kRingBytes = 200 * 1024;
constexpr int kMaxInputs = 3;

struct RowRing {
    const unsigned char* in[kMaxInputs];
    int64_t pitch[kMaxInputs];
    uint32_t bytes[kMaxInputs];   // of a row
    uint32_t offset[kMaxInputs];  // of an input's rows in a stage
    const float* side;      // one float a row as well, or nullptr
    uint32_t side_offset;   // of their places in a stage
    uint32_t weight_offset; // of the weight in floats, past the stages
    uint32_t stage_bytes;
    uint32_t smem;          // all of it
    bool keep_weights;
    int inputs, chunks, team_warps, teams, together, turns, stages;
    int64_t rows;
    uint32_t tx_extra;  // fault injection: bytes every stage waits for in vain
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
        if (lane == 0) {
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

// Fill in the plan for rows of `cols` elements; false where the ring does not
// take these rows (alignment, width). The kernels then move whole chunks only;
// whether the outputs and the weight allow it is the caller's to check.
bool plan_ring(const DeviceInfo& di, const Options& o, RowRing* R, int inputs, const void* const* in, const int64_t* ld,
               const int64_t* size, const float* side, int64_t rows, int64_t cols) {
    if (cols % 8 != 0 || cols > 256 * 4 * kRingWarps) return false;
    R->side = side;
    R->tx_extra = static_cast<uint32_t>(o.tx_extra);
    R->timeout_ns = static_cast<uint64_t>(o.timeout_ns);
    R->status = di.status;
    R->inputs = inputs;
    R->rows = rows;
    int64_t row_bytes = 0;
    for (int i = 0; i < inputs; ++i) {
        if (!rows_aligned(in[i], ld[i], size[i], 16)) return false;
        R->in[i] = static_cast<const unsigned char*>(in[i]);
        R->pitch[i] = ld[i] * size[i];
        R->bytes[i] = static_cast<uint32_t>(cols * size[i]);
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
            at += R->bytes[i] * static_cast<uint32_t>(R->together * R->turns);
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

int64_t ring_grid(const RowRing& R, int64_t sms) {
    const int64_t step = R.together * R.turns;
    return std::min(sms, (R.rows + step - 1) / step);
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
template <typename T, Weights W, typename Params>
__device__ __forceinline__ void again_weight(const Params& P, const float* kept, int col, float (&v)[8]) {
    if (W == IN_SHARED)
        load8(kept + col).unpack(v);
    else
        load_weight<T>(P.a.weight, P.a.weight_type == P.a.type, col, v);
}

constexpr int64_t kMaxGrid = int64_t(1) << 31;

// Launch of a persistent ring kernel with its shared memory.
template <typename K, typename Params>
ap_status launch_ring_kernel(const DeviceInfo& di, K kernel, std::atomic<int> (&configured)[64], const Params& P,
                             const RowRing& ring, int64_t path, cudaStream_t stream) {
    if (di.device < 0 || di.device >= 64) return AP_ERR_CUDA;
    if (!configured[di.device].load()) {  // attribute set on this device (setting twice is harmless)
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kRingBytes)) !=
            cudaSuccess)
            return AP_ERR_CUDA;
        configured[di.device] = 1;
    }
    const int64_t grid = ring_grid(ring, di.sms);
    const size_t smem = ring.smem;
    record_launch(path, grid, ring.together * ring.turns, static_cast<int64_t>(smem), ring.stages, 4);
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
