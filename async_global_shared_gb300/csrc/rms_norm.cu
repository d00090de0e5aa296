// Root-mean-square norm with the residual's addition and an output in 16/32
// bits and / or e4m3. For a row of N values:
//     h = x + residual,  r = 1 / sqrt(sum(h^2) / N + eps),  y = (h r) w.
// h r is of the order of 1 whatever the row's and the weight's sizes; r w need
// not be a float.
// The sum comes before the first output, so a row is held in registers between
// the two and memory is passed over once. Memory bounds it: 32768 x 8192 bf16
// with a 32-bit residual, e4m3 out, 432 us = 6.85 TB/s; 16384 x 8192 with a bf16
// residual 151 us; 1237 x 5000 f16, both outputs, 9.2 us in a graph; one row of
// 4096 2.1. Rows off the 16-byte boundaries move element by element, where
// instructions bound it: 27513 x 3163 f16 with a 32-bit residual 223 us = 4.3
// TB/s.
#include "row_ring.cuh"

namespace ap {
namespace {

struct NormParams {
    NormArgs a;
    bool vec_x, vec_r, vec_y, vec_q, vec_w;  // 16-byte (codes: 8-byte) aligned rows (of rows too wide for registers)
    int64_t blocks;                          // scales of a row
};

// Zeros past the row's end, `left` columns from the thread's first one, for an
// infinite r (no eps, and squares that all vanish): 0 r would be NaN there, and
// a block's amax takes in what lies past the end. (Of whole rows a chunk lies
// in the row or past it: write_row looks.)
template <int C, bool SPREAD>
__device__ __forceinline__ void clear_past_end(float r, int64_t left, int64_t step, float (&y)[C][8]) {
    if (r <= 3.402823466e38f) return;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c * step + (SPREAD ? 32 * i : i) >= left) y[c][i] = 0.0f;
}

// What is written of a row's y, C chunks a thread `step` columns apart, the
// first at col. A block's 128 values lie in the 16 lanes of a half warp, its
// amax four shuffles away (SPREAD: four in each lane of the warp, five
// shuffles); the chunks' shuffles run side by side. RAGGED: the last chunk may
// be short and outputs may not be aligned.
template <typename T, int C, bool SPREAD, bool RAGGED = false>
__device__ __forceinline__ void write_row(const NormParams& P, int64_t row, int64_t col, int64_t step, const float (&y)[C][8]) {
    const NormArgs& a = P.a;
    const int64_t left = a.cols - col;
    if (a.y != nullptr) {
        T* out = static_cast<T*>(a.y) + (row * a.ldy + col);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (left <= c * step) continue;
            if (RAGGED)
                store8(out + c * step, P.vec_y, left - c * step, y[c]);
            else
                put<SPREAD>(out + c * step, static_cast<int>(left - c * step), y[c]);
        }
    }
    if (a.q != nullptr) {
        uint8_t* out = a.q + (row * a.ldq + col);
        constexpr int kPer = SPREAD ? 2 : 1;  // blocks that a thread has values of
        float m[C][kPer];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (SPREAD) {
                m[c][0] = amax3(amax3(y[c][0], y[c][1], y[c][2]), y[c][3], 0.0f);
                m[c][kPer - 1] = amax3(amax3(y[c][4], y[c][5], y[c][6]), y[c][7], 0.0f);
            } else {
                m[c][0] = RAGGED || c * step < left ? amax8(y[c]) : 0.0f;
            }
        }
#pragma unroll
        for (int o = SPREAD ? 16 : 8; o > 0; o >>= 1)
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int b = 0; b < kPer; ++b) m[c][b] = max_nan(m[c][b], __shfl_xor_sync(0xffffffffu, m[c][b], o));
        if (SPREAD) {
            const int lane = threadIdx.x & 31;
            float* scales = a.q_scales + (row * P.blocks + (col - lane) / kScaleBlock);
#pragma unroll
            for (int c = 0; c < C; ++c) {
                if (left <= c * step) continue;
                const Scale s0 = scale_of(m[c][0]), s1 = scale_of(m[c][kPer - 1]);
                float t[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) t[i] = y[c][i] * (i < 4 ? s0.inv : s1.inv);
                const uint2 w = codes8(t, 1.0f);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (c * step + 32 * i < left)
                        out[c * step + 32 * i] = static_cast<uint8_t>((i < 4 ? w.x >> (8 * i) : w.y >> (8 * (i - 4))) & 0xffu);
                if (lane == 0) {
                    scales[c * step / kScaleBlock] = s0.s;
                    if (left > c * step + kScaleBlock) scales[c * step / kScaleBlock + 1] = s1.s;
                }
            }
        } else {
            float* scales = a.q_scales + (row * P.blocks + col / kScaleBlock);
#pragma unroll
            for (int c = 0; c < C; ++c) {
                if (left <= c * step) continue;
                const Scale s = scale_of(m[c][0]);
                const uint2 w = codes8(y[c], s.inv);
                if (RAGGED)
                    store_codes(out + c * step, P.vec_q, left - c * step, w);
                else
                    *reinterpret_cast<uint2*>(out + c * step) = w;
                if ((threadIdx.x & 15) == 0) scales[c * step / kScaleBlock] = s.s;
            }
        }
    }
}

// One row a CTA (WARP: a warp), C chunks of eight elements a thread.
template <typename T, typename R, int C, bool WARP, bool SPREAD>
__global__ void __launch_bounds__(WARP ? 256 : 1024) rms_norm_kernel(const __grid_constant__ NormParams P) {
    __shared__ float scratch[32];
    ptx::let_next_grid_start();
    ptx::wait_previous_grid();
    const NormArgs& a = P.a;
    const int me = WARP ? threadIdx.x & 31 : threadIdx.x;  // in the row
    const int apart = 8 * (WARP ? 32 : blockDim.x);        // columns between a thread's chunks
    const int64_t row = WARP ? static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
    if (WARP && row >= a.rows) return;
    const int col = first_column<SPREAD>(me), left = static_cast<int>(a.cols) - col;
    const T* x = static_cast<const T*>(a.x) + (row * a.ldx + col);
    float h[C][8];
    float sum = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) take<SPREAD>(x + c * apart, left - c * apart, h[c]);
    if (a.residual != nullptr) {
        const R* r = static_cast<const R*>(a.residual) + (row * a.ldr + col);
        R* out = static_cast<R*>(a.residual_out) + (row * a.ldr + col);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float v[8];
            take<SPREAD>(r + c * apart, left - c * apart, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) h[c][i] += v[i];
            put<SPREAD>(out + c * apart, left - c * apart, h[c]);
        }
    }
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fmaf(h[c][i], h[c][i], sum);
    sum = row_sum<WARP>(sum, scratch);
    const float r = __frcp_rn(__fsqrt_rn(__fdiv_rn(sum, static_cast<float>(a.cols)) + a.eps));
    if (a.rstd != nullptr && me == 0) a.rstd[row] = r;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        float w[8];
        take_weight<SPREAD, T>(a.weight, a.weight_type == a.type, col + c * apart, left - c * apart, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[c][i] = h[c][i] * r * w[i];
    }
    if (SPREAD) clear_past_end<C, SPREAD>(r, left, apart, h);
    write_row<T, C, SPREAD>(P, row, col, apart, h);
}

// The ring's form: teams of warps, rows from shared memory, the weight in
// registers for the whole grid's life (four chunks: in shared memory). One row a
// CTA leaves the memory idle while the row's sum is on its way: 16384 x 8192
// took 235 us so, 151 with the ring.
template <typename T, typename R, int C, bool RES, Weights W, bool SPREAD>
__global__ void __launch_bounds__(kRingThreads, 1)
    rms_norm_ring_kernel(const __grid_constant__ NormParams P, const __grid_constant__ RowRing ring) {
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ RingBars bars;
    __shared__ float scratch[2][kRingWarps];
    constexpr bool kKeep = W == IN_REGISTERS;
    ptx::let_next_grid_start();
    ring_init(ring, bars);
    const NormArgs& a = P.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == kRingWarps) {
        ring_produce(ring, bars, ptx::smem_addr(smem));
        return;
    }
    float* weights = reinterpret_cast<float*>(smem + ring.weight_offset);
    if (W == IN_SHARED) stage_weights<T>(a.weight, a.weight_type == a.type, a.cols, weights);
    const int team = warp / ring.team_warps, width = 32 * ring.team_warps;
    if (team >= ring.teams) return;
    const int me = threadIdx.x - team * width;
    const int apart = 8 * width;  // columns between a thread's chunks
    const int col = first_column<SPREAD>(me), left = static_cast<int>(a.cols) - col;
    float w[kKeep ? C : 1][8];
    if (kKeep) {
#pragma unroll
        for (int c = 0; c < C; ++c)
            take_weight<SPREAD, T>(a.weight, a.weight_type == a.type, col + c * apart, left - c * apart, w[kKeep ? c : 0]);
    }
    const float inv = __frcp_rn(static_cast<float>(a.cols));
    const int64_t step = ring.together * ring.turns;
    const int groups = ring.teams / ring.together, group = team / ring.together, mate = team % ring.together;
    int s = group, turn = 0;
    uint32_t round = 0;
    while (s >= ring.stages) s -= ring.stages, ++round;
    for (int64_t base = (blockIdx.x + static_cast<int64_t>(gridDim.x) * group) * step; base < a.rows;
         base += gridDim.x * groups * step) {
        if (!stage_arrived(ring, bars, s, round)) {
            attend_sums(ring, scratch, team, base + mate, gridDim.x * groups * step, turn);
            break;
        }
        const unsigned char* stage = smem + s * ring.stage_bytes;
        for (int m = 0; m < ring.turns; ++m, turn ^= 1) {
            const int slot = m * ring.together + mate;
            const int64_t row = base + slot;
            const bool mine = row < a.rows;  // the same for the whole team
            float h[C][8];
            if (mine) {
                const T* x = reinterpret_cast<const T*>(stage + row_place<SPREAD>(ring, 0, base, slot)) + col;
                const R* res = RES ? reinterpret_cast<const R*>(stage + ring.offset[1] + row_place<SPREAD>(ring, 1, base, slot)) + col
                                   : nullptr;
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    take<SPREAD>(x + c * apart, left - c * apart, h[c]);
                    if (RES && left > c * apart) {
                        float v[8];
                        take<SPREAD>(res + c * apart, left - c * apart, v);
#pragma unroll
                        for (int i = 0; i < 8; ++i) h[c][i] += v[i];
                    }
                }
            }
            if (m == ring.turns - 1) {  // everything of the stage is in registers
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&bars.empty[s]));
            }
            if (!mine) continue;
            float sum = 0.0f;
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) sum = fmaf(h[c][i], h[c][i], sum);
            if (RES) {
                R* out = static_cast<R*>(a.residual_out) + (row * a.ldr + col);
#pragma unroll
                for (int c = 0; c < C; ++c) put<SPREAD>(out + c * apart, left - c * apart, h[c]);
            }
            sum = team_sum(sum, &scratch[turn][team * ring.team_warps], team, ring.team_warps);
            const float r = __frcp_rn(__fsqrt_rn(fmaf(sum, inv, a.eps)));
            if (a.rstd != nullptr && me == 0) a.rstd[row] = r;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                float again[8];
                if (!kKeep && left > c * apart) again_weight<T, W, SPREAD>(P, weights, col + c * apart, left - c * apart, again);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (kKeep || left > c * apart) h[c][i] = h[c][i] * r * (kKeep ? w[kKeep ? c : 0][i] : again[i]);
            }
            if (SPREAD) clear_past_end<C, SPREAD>(r, left, apart, h);
            write_row<T, C, SPREAD>(P, row, col, apart, h);
        }
        s += groups;
        while (s >= ring.stages) s -= ring.stages, ++round;
    }
}

// Rows too wide for registers: the row is read twice, the second time from
// the L2. All writes are in the second pass, so in-place calls still read
// every element before it is overwritten.
template <typename T, typename R>
__global__ void __launch_bounds__(1024) rms_norm_wide_kernel(const __grid_constant__ NormParams P) {
    __shared__ float scratch[32];
    ptx::let_next_grid_start();
    ptx::wait_previous_grid();
    const NormArgs& a = P.a;
    const int64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(a.x) + row * a.ldx;
    const R* res = a.residual != nullptr ? static_cast<const R*>(a.residual) + row * a.ldr : nullptr;
    auto load_h = [&](int64_t col, float(&h)[8]) {
        load8(x + col, P.vec_x, a.cols - col).unpack(h);
        if (res != nullptr) {
            float v[8];
            load8(res + col, P.vec_r, a.cols - col).unpack(v);
#pragma unroll
            for (int i = 0; i < 8; ++i) h[i] += v[i];
        }
    };
    const int64_t step = 8 * static_cast<int64_t>(blockDim.x);
    float sum = 0.0f;
    for (int64_t col = 8 * static_cast<int64_t>(threadIdx.x); col < a.cols; col += step) {
        float h[8];
        load_h(col, h);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fmaf(h[i], h[i], sum);
    }
    sum = row_sum<false>(sum, scratch);
    const float r = __frcp_rn(__fsqrt_rn(__fdiv_rn(sum, static_cast<float>(a.cols)) + a.eps));
    if (a.rstd != nullptr && threadIdx.x == 0) a.rstd[row] = r;
    // whole warps stay in the loop, for the shuffles of a block's amax
    for (int64_t base = 0; base < a.cols; base += step) {
        const int64_t col = base + 8 * static_cast<int64_t>(threadIdx.x);
        float h[1][8], w[8];
        load_h(col, h[0]);
        if (res != nullptr && col < a.cols)
            store8(static_cast<R*>(a.residual_out) + row * a.ldr + col, P.vec_r, a.cols - col, h[0]);
        if (a.weight_type == a.type)
            load8(static_cast<const T*>(a.weight) + col, P.vec_w, a.cols - col).unpack(w);
        else
            load8(static_cast<const float*>(a.weight) + col, P.vec_w, a.cols - col).unpack(w);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[0][i] = h[0][i] * r * w[i];
        clear_past_end<1, false>(r, a.cols - col, 0, h);
        write_row<T, 1, false, true>(P, row, col, 0, h);
    }
}

template <typename T, typename R, int C, bool WARP>
ap_status launch_norm_c(const NormParams& P, bool whole, cudaStream_t stream) {
    const int64_t chunks = (P.a.cols + 7) / 8;
    const int threads = WARP ? 256 : static_cast<int>(((chunks + C - 1) / C + 31) / 32 * 32);
    const int64_t grid = WARP ? (P.a.rows + 7) / 8 : P.a.rows;
    if (grid >= kMaxGrid) return AP_ERR_SHAPE;
    record_launch(PATH_NORM, grid, 8 * C, 0, 0, (WARP ? 1 : 0) | (whole ? 0 : 8));
    return whole ? launch_early(rms_norm_kernel<T, R, C, WARP, false>, grid, threads, stream, P)
                 : launch_early(rms_norm_kernel<T, R, C, WARP, true>, grid, threads, stream, P);
}

template <typename T, typename R, bool RES, bool SPREAD>
ap_status launch_norm_ring(const DeviceInfo& di, const NormParams& P, const RowRing& ring, int64_t grid, cudaStream_t stream) {
    static std::atomic<int> configured[5][64];
    if (ring.chunks == 2)
        return launch_ring_kernel(di, rms_norm_ring_kernel<T, R, 2, RES, IN_REGISTERS, SPREAD>, configured[0], P, ring, grid, PATH_NORM, stream);
    if (ring.chunks == 3)
        return ring.keep_weights
                   ? launch_ring_kernel(di, rms_norm_ring_kernel<T, R, 3, RES, IN_SHARED, SPREAD>, configured[1], P, ring, grid, PATH_NORM, stream)
                   : launch_ring_kernel(di, rms_norm_ring_kernel<T, R, 3, RES, IN_L2, SPREAD>, configured[2], P, ring, grid, PATH_NORM, stream);
    return ring.keep_weights
               ? launch_ring_kernel(di, rms_norm_ring_kernel<T, R, 4, RES, IN_SHARED, SPREAD>, configured[3], P, ring, grid, PATH_NORM, stream)
               : launch_ring_kernel(di, rms_norm_ring_kernel<T, R, 4, RES, IN_L2, SPREAD>, configured[4], P, ring, grid, PATH_NORM, stream);
}

// The ring's set-up is paid back from this many elements on (1216 x 4096: 8.2
// us against 8.8 without, 2432 x 4096: 13.7 against 16.9, 16384 x 4096: 72
// against 88); short rows are too much work for its one producer (16384 x 256:
// 9.6 us, 6.3 without).
constexpr int64_t kRingElements = int64_t(1) << 23, kRingColumns = 1024;

template <typename T, typename R>
ap_status launch_norm_t(const DeviceInfo& di, const Options& o, const NormArgs& a, cudaStream_t stream) {
    NormParams P;
    P.a = a;
    P.vec_x = rows_aligned(a.x, a.ldx, sizeof(T), 16);
    P.vec_r = rows_aligned(a.residual, a.ldr, sizeof(R), 16) && rows_aligned(a.residual_out, a.ldr, sizeof(R), 16);
    P.vec_y = rows_aligned(a.y, a.ldy, sizeof(T), 16);
    P.vec_q = rows_aligned(a.q, a.ldq, 1, 8);
    P.vec_w = reinterpret_cast<uintptr_t>(a.weight) % 16 == 0;
    P.blocks = (a.cols + kScaleBlock - 1) / kScaleBlock;
    RowRing ring;
    const void* const in[] = {a.x, a.residual};
    const int64_t ld[] = {a.ldx, a.ldr}, size[] = {sizeof(T), sizeof(R)};
    const bool res = a.residual != nullptr;
    const bool whole =
        a.cols % 8 == 0 && P.vec_x && (!res || P.vec_r) && P.vec_w && (a.y == nullptr || P.vec_y) && (a.q == nullptr || P.vec_q);
    const bool many = o.force_path == 1 || (o.force_path != 2 && a.cols > kRingColumns && a.rows >= kRingElements / a.cols);
    // One input alone leaves little to stream beside the work on a row, and a
    // CTA's one or two wide teams then wait on their sums with nothing else to
    // do (no residual, y in f16: 9728 x 12000 107 us against 95 in registers,
    // 9728 x 6000 55 against 49; with two teams of four chunks 9728 x 8192 63
    // against 71; with a residual 145 against 205 at 9728 x 12000). The same for
    // other types and outputs: 9728 x 12000 bf16 to e4m3 120 against 91, f32 to
    // e4m3 123 against 107, 9728 x 6000 62 and 51, 63 and 57, rows off the
    // boundaries (9728 x 6001 bf16 to e4m3) 80 and 72. f32 with y in f32, DRAM's
    // alone, is the same either way (161 and 160; 16384 columns 219 and 231).
    const auto idle = [&] { return o.force_path != 1 && !res && (ring.teams == 1 || (ring.teams == 2 && ring.chunks == 3)); };
    if (many && plan_ring(di, o, &ring, res ? 2 : 1, in, ld, size, nullptr, a.rows, a.cols, whole) && !idle()) {
        const int64_t grid = ring_grid(ring, di.sms, o.grid);
        if (whole)
            return res ? launch_norm_ring<T, R, true, false>(di, P, ring, grid, stream)
                       : launch_norm_ring<T, T, false, false>(di, P, ring, grid, stream);
        return res ? launch_norm_ring<T, R, true, true>(di, P, ring, grid, stream)
                   : launch_norm_ring<T, T, false, true>(di, P, ring, grid, stream);
    }
    if (a.cols <= 256) return launch_norm_c<T, R, 1, true>(P, whole, stream);
    if (a.cols <= 512) return launch_norm_c<T, R, 2, true>(P, whole, stream);
    if (a.cols <= 4096) return launch_norm_c<T, R, 1, false>(P, whole, stream);
    if (a.cols <= 8192) return launch_norm_c<T, R, 2, false>(P, whole, stream);
    if (a.cols <= 32768) return launch_norm_c<T, R, 4, false>(P, whole, stream);
    if (a.rows >= kMaxGrid) return AP_ERR_SHAPE;
    record_launch(PATH_NORM, a.rows, 0, 0, 0, 2);
    return launch_early(rms_norm_wide_kernel<T, R>, a.rows, 1024, stream, P);
}

}  // namespace

ap_status launch_rms_norm(const DeviceInfo& di, const Options& o, const NormArgs& a, cudaStream_t stream) {
    const bool same = a.residual == nullptr || a.residual_type == a.type;
    switch (a.type) {
        case AP_BF16:
            return same ? launch_norm_t<__nv_bfloat16, __nv_bfloat16>(di, o, a, stream)
                        : launch_norm_t<__nv_bfloat16, float>(di, o, a, stream);
        case AP_F16:
            return same ? launch_norm_t<__half, __half>(di, o, a, stream) : launch_norm_t<__half, float>(di, o, a, stream);
        default: return launch_norm_t<float, float>(di, o, a, stream);
    }
}

}  // namespace ap
