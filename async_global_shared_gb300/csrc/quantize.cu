// e4m3 codes and scales of a matrix, by row blocks or tiles, as it stands and
// / or transposed.
//
// Floor: every element is read once and each output's byte written once. The
// scale of a block needs its amax before the first code, so a tile of
// 128 x 128 elements stays in registers between the two; the transposed codes
// cross through shared memory, where a thread's eight rows of one column are
// one 8-byte unit. 16384 x 8192 bf16 both ways: 96 us = 5.7 TB/s; a float weight
// of 11003 x 4100 by tiles, both ways: 47 us = 5.7 TB/s; 64 x 16384 by rows: 6.4
// us, nearly all of it the call.
#include "device_common.cuh"
#include "fp8_common.cuh"
#include "internal.h"

namespace ap {
namespace {

struct QuantParams {
    QuantArgs a;
    bool vec_x, vec_q, vec_qt;
    int64_t blocks, blocks_t;  // scales of a row of q, of qt (tiles: of a row of tiles)
};

__device__ __forceinline__ float half_warp_max(float m) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}

// Row blocks only: a half warp a block, no exchange beyond its shuffles.
template <typename T>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const __grid_constant__ QuantParams P) {
    ptx::let_next_grid_start();
    ptx::wait_previous_grid();
    const QuantArgs& a = P.a;
    const int64_t block = static_cast<int64_t>(blockIdx.x) * 16 + threadIdx.x / 16;
    const int64_t row = block / P.blocks, bj = block % P.blocks;
    const int64_t col = bj * kScaleBlock + 8 * (threadIdx.x & 15);
    const int64_t n = row < a.rows ? a.cols - col : 0;
    float v[8];
    load8(static_cast<const T*>(a.x) + row * a.ldx + col, P.vec_x, n).unpack(v);
    const Scale s = scale_of(half_warp_max(amax8(v)));
    if (n > 0) store_codes(a.q + row * a.ldq + col, P.vec_q, n, codes8(v, s.inv));
    if (n > 0 && (threadIdx.x & 15) == 0) a.scales[block] = s.s;
}

// A 128 x 128 tile a CTA: thread t holds rows 8 (t / 16) .. + 7 of columns
// 8 (t % 16) .. + 7. What bounds the kernel beside memory is the number of
// instructions, so maxima are taken two 16-bit values at a time, eight rows'
// maxima cross 16 lanes in eight exchanges (each halves the rows a lane still
// carries, so a row's scale is computed by two lanes and not by 16), and both
// outputs' codes come from one unpacking. (Float by tiles: 34 % of the issue
// slots and 58 % of DRAM's peak; 98 registers leave two CTAs an SM, whose waits
// for their loads bound it.)
template <typename T, bool TILES>
__global__ void __launch_bounds__(256) quantize_tile_kernel(const __grid_constant__ QuantParams P) {
    using K = Peak<T>;
    using V = typename K::V;
    __shared__ float col_max[8][kScaleBlock];  // per warp, or [w][0]: the warp's amax (tiles)
    __shared__ __align__(16) uint2 turned[kScaleBlock][16];  // [column][8-row unit, exchanged by the column's chunk]
    ptx::let_next_grid_start();
    ptx::wait_previous_grid();
    const QuantArgs& a = P.a;
    const int lane = threadIdx.x & 31, chunk = threadIdx.x & 15, rows8 = threadIdx.x >> 4, warp = threadIdx.x >> 5;
    const int64_t tj = blockIdx.x % P.blocks, ti = blockIdx.x / P.blocks;
    const int64_t row0 = ti * kScaleBlock + 8 * rows8, col = tj * kScaleBlock + 8 * chunk;
    const int rows = static_cast<int>(a.rows - row0 < 8 ? a.rows - row0 : 8);  // of this thread that exist (may be negative)
    const int64_t cols = a.cols - col;
    Raw8<T> raw[8];
    const T* x = static_cast<const T*>(a.x) + (row0 * a.ldx + col);
#pragma unroll
    for (int p = 0; p < 8; ++p) raw[p] = load8(x + p * a.ldx, P.vec_x, p < rows ? cols : 0);

    float inv_row[8], inv_col[8];
    if (TILES) {
        V m = K::chunk(raw[0]);
#pragma unroll
        for (int p = 1; p < 8; ++p) m = K::max(m, K::chunk(raw[p]));
        float f = K::value(m);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) f = max_nan(f, __shfl_xor_sync(0xffffffffu, f, o));
        if (lane == 0) col_max[warp][0] = f;
        __syncthreads();
        f = col_max[0][0];
#pragma unroll
        for (int w = 1; w < 8; ++w) f = max_nan(f, col_max[w][0]);
        const Scale s = scale_of(f);
#pragma unroll
        for (int i = 0; i < 8; ++i) inv_row[i] = inv_col[i] = s.inv;
        if (threadIdx.x == 0) {
            if (a.q != nullptr) a.scales[ti * P.blocks + tj] = s.s;
            if (a.qt != nullptr) a.scales_t[tj * P.blocks_t + ti] = s.s;
        }
    } else {
        if (a.q != nullptr) {
            V m[8];
#pragma unroll
            for (int p = 0; p < 8; ++p) m[p] = K::chunk(raw[p]);
            // lane bits 3, 2, 1 choose the half of the rows a lane keeps
#pragma unroll
            for (int o = 8, n = 4; o > 1; o >>= 1, n >>= 1) {
                const bool high = (lane & o) != 0;
#pragma unroll
                for (int j = 0; j < n; ++j) {
                    const V mine = high ? m[n + j] : m[j], theirs = high ? m[j] : m[n + j];
                    m[j] = K::max(mine, __shfl_xor_sync(0xffffffffu, theirs, o));
                }
            }
            m[0] = K::max(m[0], __shfl_xor_sync(0xffffffffu, m[0], 1));
            const Scale s = scale_of(K::value(m[0]));  // of row (lane % 16) / 2
            const int p = chunk >> 1;
            if ((lane & 1) == 0 && p < rows) a.scales[(row0 + p) * P.blocks + tj] = s.s;
#pragma unroll
            for (int i = 0; i < 8; ++i) inv_row[i] = __shfl_sync(0xffffffffu, s.inv, (lane & 16) | (2 * i));
        }
        if (a.qt != nullptr) {
            V m[K::kWords];
#pragma unroll
            for (int i = 0; i < K::kWords; ++i) m[i] = K::word(raw[0], i);
#pragma unroll
            for (int p = 1; p < 8; ++p)
#pragma unroll
                for (int i = 0; i < K::kWords; ++i) m[i] = K::max(m[i], K::word(raw[p], i));
#pragma unroll
            for (int i = 0; i < K::kWords; ++i) m[i] = K::max(m[i], __shfl_xor_sync(0xffffffffu, m[i], 16));
            if ((lane & 16) == 0) {
#pragma unroll
                for (int i = 0; i < 8; ++i) col_max[warp][8 * chunk + i] = K::column(m, i);
            }
            __syncthreads();
            if (threadIdx.x < kScaleBlock) {
                float c = col_max[0][threadIdx.x];
#pragma unroll
                for (int w = 1; w < 8; ++w) c = max_nan(c, col_max[w][threadIdx.x]);
                const Scale s = scale_of(c);
                const int64_t j = tj * kScaleBlock + threadIdx.x;
                if (j < a.cols) a.scales_t[j * P.blocks_t + ti] = s.s;
                col_max[0][threadIdx.x] = s.inv;
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 8; ++i) inv_col[i] = col_max[0][8 * chunk + i];
        }
    }

    uint32_t lo[8], hi[8];  // codes of rows 0..3 and 4..7 of each of the thread's columns
    uint8_t* q = a.q + (row0 * a.ldq + col);
#pragma unroll
    for (int p = 0; p < 8; p += 2) {
        float v[8], u[8];
        raw[p].unpack(v);
        raw[p + 1].unpack(u);
        if (a.q != nullptr && cols > 0) {
            if (p < rows) store_codes(q + p * a.ldq, P.vec_q, cols, codes8(v, inv_row[p]));
            if (p + 1 < rows) store_codes(q + (p + 1) * a.ldq, P.vec_q, cols, codes8(u, inv_row[p + 1]));
        }
        if (a.qt != nullptr) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t two = e4m3x2(v[i] * inv_col[i], u[i] * inv_col[i]);
                if (p == 0) lo[i] = two;
                if (p == 2) lo[i] |= two << 16;
                if (p == 4) hi[i] = two;
                if (p == 6) hi[i] |= two << 16;
            }
        }
    }
    if (a.qt == nullptr) return;
    // unit rows8 of a column goes to place rows8 ^ chunk: the 16 lanes that
    // write one instruction's columns then cover all banks
#pragma unroll
    for (int i = 0; i < 8; ++i) turned[8 * chunk + i][rows8 ^ chunk] = make_uint2(lo[i], hi[i]);
    __syncthreads();
    // 16 lanes write a column's 128 codes
    const int64_t i0 = ti * kScaleBlock + 8 * chunk, j0 = tj * kScaleBlock + rows8;
    uint8_t* qt = a.qt + (j0 * a.ldqt + i0);
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const int c = 16 * p + rows8;
        if (j0 + 16 * p < a.cols && i0 < a.rows)
            store_codes(qt + 16 * p * a.ldqt, P.vec_qt, a.rows - i0, turned[c][chunk ^ (c >> 3)]);
    }
}

template <typename T>
ap_status launch_quant_t(const QuantArgs& a, cudaStream_t stream) {
    QuantParams P;
    P.a = a;
    P.vec_x = rows_aligned(a.x, a.ldx, sizeof(T), 16);
    P.vec_q = rows_aligned(a.q, a.ldq, 1, 8);
    P.vec_qt = rows_aligned(a.qt, a.ldqt, 1, 8);
    P.blocks = (a.cols + kScaleBlock - 1) / kScaleBlock;
    P.blocks_t = (a.rows + kScaleBlock - 1) / kScaleBlock;
    const bool rows_only = a.block_rows == 1 && a.qt == nullptr;
    const int64_t grid = rows_only ? (a.rows * P.blocks + 15) / 16 : P.blocks * P.blocks_t;
    if (grid >= (int64_t(1) << 31)) return AP_ERR_SHAPE;
    record_launch(PATH_QUANTIZE, grid, rows_only ? 8 : 64, 0, 0, 0);
    if (rows_only) return launch_early(quantize_rows_kernel<T>, grid, 256, stream, P);
    return a.block_rows == 1 ? launch_early(quantize_tile_kernel<T, false>, grid, 256, stream, P)
                             : launch_early(quantize_tile_kernel<T, true>, grid, 256, stream, P);
}

__global__ void __launch_bounds__(256) block_scale_kernel(const float* amax, float* scale, float* inv, int64_t n) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= n) return;
    const Scale s = scale_of(amax[i]);
    scale[i] = s.s;
    inv[i] = s.inv;
}

}  // namespace

ap_status launch_block_scale(const float* amax, float* scale, float* inv, int64_t n, cudaStream_t stream) {
    block_scale_kernel<<<static_cast<unsigned>((n + 255) / 256), 256, 0, stream>>>(amax, scale, inv, n);
    return cudaGetLastError() == cudaSuccess ? AP_OK : AP_ERR_CUDA;
}

ap_status launch_quantize(const DeviceInfo&, const QuantArgs& a, cudaStream_t stream) {
    switch (a.type) {
        case AP_BF16: return launch_quant_t<__nv_bfloat16>(a, stream);
        case AP_F16: return launch_quant_t<__half>(a, stream);
        default: return launch_quant_t<float>(a, stream);
    }
}

}  // namespace ap
