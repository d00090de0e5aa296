// e4m3 codes and scales of a matrix, by row blocks or tiles, as it stands and
// / or transposed.
//
// Floor: every element is read once and each output's byte written once. The
// scale of a block needs its amax before the first code, so a tile of
// 128 x 128 elements stays in registers between the two; the transposed codes
// cross through shared memory, where a thread's eight rows of one column are
// one 8-byte unit.
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
// 8 (t % 16) .. + 7.
template <typename T>
__global__ void __launch_bounds__(256) quantize_tile_kernel(const __grid_constant__ QuantParams P) {
    __shared__ float col_max[8][kScaleBlock];  // per warp, or [w][0]: the warp's amax (tiles)
    __shared__ __align__(16) uint2 turned[kScaleBlock][16];  // [column][8-row unit, exchanged by the column's chunk]
    ptx::let_next_grid_start();
    ptx::wait_previous_grid();
    const QuantArgs& a = P.a;
    const int chunk = threadIdx.x & 15, rows8 = threadIdx.x >> 4, warp = threadIdx.x >> 5;
    const int64_t tj = blockIdx.x % P.blocks, ti = blockIdx.x / P.blocks;
    const int64_t row0 = ti * kScaleBlock + 8 * rows8, col = tj * kScaleBlock + 8 * chunk;
    const bool tiles = a.block_rows != 1;
    Raw8<T> raw[8];
#pragma unroll
    for (int p = 0; p < 8; ++p)
        raw[p] = load8(static_cast<const T*>(a.x) + (row0 + p) * a.ldx + col, P.vec_x,
                       row0 + p < a.rows ? a.cols - col : 0);
    float inv_tile = 0.0f;
    float inv_col[8];
    if (tiles) {
        float m = 0.0f;
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            float v[8];
            raw[p].unpack(v);
            m = max_nan(m, amax8(v));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
        if ((threadIdx.x & 31) == 0) col_max[warp][0] = m;
        __syncthreads();
        m = col_max[0][0];
#pragma unroll
        for (int w = 1; w < 8; ++w) m = max_nan(m, col_max[w][0]);
        const Scale s = scale_of(m);
        inv_tile = s.inv;
        if (threadIdx.x == 0) {
            if (a.q != nullptr) a.scales[ti * P.blocks + tj] = s.s;
            if (a.qt != nullptr) a.scales_t[tj * P.blocks_t + ti] = s.s;
        }
    } else if (a.qt != nullptr) {
        float m[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            float v[8];
            raw[p].unpack(v);
#pragma unroll
            for (int i = 0; i < 8; ++i) m[i] = max_nan(m[i], fabsf(v[i]));
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            m[i] = max_nan(m[i], __shfl_xor_sync(0xffffffffu, m[i], 16));
            if ((threadIdx.x & 16) == 0) col_max[warp][8 * chunk + i] = m[i];
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
    if (a.q != nullptr) {
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            float v[8];
            raw[p].unpack(v);
            float inv = inv_tile;
            if (!tiles) {
                const Scale s = scale_of(half_warp_max(amax8(v)));
                inv = s.inv;
                if (chunk == 0 && row0 + p < a.rows) a.scales[(row0 + p) * P.blocks + tj] = s.s;
            }
            if (row0 + p < a.rows && col < a.cols)
                store_codes(a.q + (row0 + p) * a.ldq + col, P.vec_q, a.cols - col, codes8(v, inv));
        }
    }
    if (a.qt == nullptr) return;
    uint32_t lo[8], hi[8];  // codes of rows 0..3 and 4..7 of each of the thread's columns
#pragma unroll
    for (int p = 0; p < 8; p += 2) {
        float v[8], u[8];
        raw[p].unpack(v);
        raw[p + 1].unpack(u);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float inv = tiles ? inv_tile : inv_col[i];
            const uint32_t two = e4m3x2(v[i] * inv, u[i] * inv);
            if (p == 0) lo[i] = two;
            if (p == 2) lo[i] |= two << 16;
            if (p == 4) hi[i] = two;
            if (p == 6) hi[i] |= two << 16;
        }
    }
    // unit rows8 of a column goes to place rows8 ^ chunk: the 16 lanes that
    // write one instruction's columns then cover all banks
#pragma unroll
    for (int i = 0; i < 8; ++i) turned[8 * chunk + i][rows8 ^ chunk] = make_uint2(lo[i], hi[i]);
    __syncthreads();
    // 16 lanes write a column's 128 codes
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const int c = 16 * p + (threadIdx.x >> 4);
        const int64_t j = tj * kScaleBlock + c, i0 = ti * kScaleBlock + 8 * (threadIdx.x & 15);
        if (j < a.cols && i0 < a.rows)
            store_codes(a.qt + j * a.ldqt + i0, P.vec_qt, a.rows - i0, turned[c][(threadIdx.x & 15) ^ (c >> 3)]);
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
    return rows_only ? launch_early(quantize_rows_kernel<T>, grid, 256, stream, P)
                     : launch_early(quantize_tile_kernel<T>, grid, 256, stream, P);
}

}  // namespace

ap_status launch_quantize(const DeviceInfo&, const QuantArgs& a, cudaStream_t stream) {
    switch (a.type) {
        case AP_BF16: return launch_quant_t<__nv_bfloat16>(a, stream);
        case AP_F16: return launch_quant_t<__half>(a, stream);
        default: return launch_quant_t<float>(a, stream);
    }
}

}  // namespace ap
