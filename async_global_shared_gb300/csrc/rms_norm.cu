// Root-mean-square norm with the residual's addition and an output in 16/32
// bits and / or e4m3, and its gradient.
//
// Forward, for a row of N values:
//     h = x + residual,  r = 1 / sqrt(sum(h^2) / N + eps),  y = h r w.
// Backward, with n = h r and g = dy w: r depends on every h of the row,
// d r / d h_i = -r^3 h_i / N, so
//     dx = r (g - n mean(g n)) + dresidual,   dw_j = sum over rows of dy n.
// Both need one sum over the row before the first output, so a row is held
// in registers between the two and memory is passed over once.
#include <algorithm>

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

struct NormParams {
    NormArgs a;
    bool vec_x, vec_r, vec_y, vec_q, vec_w;  // 16-byte (codes: 8-byte) aligned rows
    int64_t blocks;                          // scales of a row
};

template <typename T>
__device__ __forceinline__ void load_weight(const void* w, bool same, bool vec, int64_t col, int64_t n, float (&v)[8]) {
    if (same)
        load8(static_cast<const T*>(w) + col, vec, n).unpack(v);
    else
        load8(static_cast<const float*>(w) + col, vec, n).unpack(v);
}

// y of one chunk and what is written of it. The 16 lanes of a half warp hold
// one block of 128, so its amax is four shuffles away.
template <typename T>
__device__ __forceinline__ void write_chunk(const NormParams& P, int64_t row, int64_t col, int64_t n, const float (&y)[8]) {
    const NormArgs& a = P.a;
    if (a.y != nullptr && n > 0) store8(static_cast<T*>(a.y) + row * a.ldy + col, P.vec_y, n, y);
    if (a.q != nullptr) {
        float m = amax8(y);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float s = scale_of(m);
        if (n > 0) {
            store_codes(a.q + row * a.ldq + col, P.vec_q, n, codes8(y, __frcp_rn(s)));
            if ((threadIdx.x & 15) == 0) a.q_scales[row * P.blocks + col / kScaleBlock] = s;
        }
    }
}

// One row a CTA (WARP: a warp), C chunks of eight elements a thread.
template <typename T, typename R, int C, bool WARP>
__global__ void __launch_bounds__(WARP ? 256 : 1024) rms_norm_kernel(const __grid_constant__ NormParams P) {
    __shared__ float scratch[32];
    const NormArgs& a = P.a;
    const int lane = WARP ? threadIdx.x & 31 : threadIdx.x;
    const int width = WARP ? 32 : blockDim.x;
    const int64_t row = WARP ? static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
    if (WARP && row >= a.rows) return;
    const T* x = static_cast<const T*>(a.x) + row * a.ldx;
    float h[C][8];
    float sum = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int64_t col = 8 * static_cast<int64_t>(c * width + lane);
        load8(x + col, P.vec_x, a.cols - col).unpack(h[c]);
    }
    if (a.residual != nullptr) {
        const R* r = static_cast<const R*>(a.residual) + row * a.ldr;
        R* out = static_cast<R*>(a.residual_out) + row * a.ldr;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int64_t col = 8 * static_cast<int64_t>(c * width + lane);
            float v[8];
            load8(r + col, P.vec_r, a.cols - col).unpack(v);
#pragma unroll
            for (int i = 0; i < 8; ++i) h[c][i] += v[i];
            if (col < a.cols) store8(out + col, P.vec_r, a.cols - col, h[c]);
        }
    }
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fmaf(h[c][i], h[c][i], sum);
    sum = row_sum<WARP>(sum, scratch);
    const float r = __frcp_rn(__fsqrt_rn(__fdiv_rn(sum, static_cast<float>(a.cols)) + a.eps));
    if (a.rstd != nullptr && lane == 0) a.rstd[row] = r;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int64_t col = 8 * static_cast<int64_t>(c * width + lane);
        float w[8];
        load_weight<T>(a.weight, a.weight_type == a.type, P.vec_w, col, a.cols - col, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] *= h[c][i] * r;
        write_chunk<T>(P, row, col, a.cols - col, w);
    }
}

// Rows too wide for registers: the row is read twice, the second time from
// the L2. All writes are in the second pass, so in-place calls still read
// every element before it is overwritten.
template <typename T, typename R>
__global__ void __launch_bounds__(1024) rms_norm_wide_kernel(const __grid_constant__ NormParams P) {
    __shared__ float scratch[32];
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
        float h[8], w[8];
        load_h(col, h);
        if (res != nullptr && col < a.cols)
            store8(static_cast<R*>(a.residual_out) + row * a.ldr + col, P.vec_r, a.cols - col, h);
        load_weight<T>(a.weight, a.weight_type == a.type, P.vec_w, col, a.cols - col, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] *= h[i] * r;
        write_chunk<T>(P, row, col, a.cols - col, w);
    }
}

constexpr int64_t kMaxGrid = int64_t(1) << 31;

ap_status launched() { return cudaGetLastError() == cudaSuccess ? AP_OK : AP_ERR_CUDA; }

template <typename T, typename R, int C, bool WARP>
ap_status launch_norm_c(const NormParams& P, cudaStream_t stream) {
    const int64_t chunks = (P.a.cols + 7) / 8;
    const int threads = WARP ? 256 : static_cast<int>(((chunks + C - 1) / C + 31) / 32 * 32);
    const int64_t grid = WARP ? (P.a.rows + 7) / 8 : P.a.rows;
    if (grid >= kMaxGrid) return AP_ERR_SHAPE;
    record_launch(PATH_NORM, grid, 8 * C, 0, 0, WARP ? 1 : 0);
    rms_norm_kernel<T, R, C, WARP><<<static_cast<unsigned>(grid), threads, 0, stream>>>(P);
    return launched();
}

template <typename T, typename R>
ap_status launch_norm_t(const DeviceInfo&, const NormArgs& a, cudaStream_t stream) {
    NormParams P;
    P.a = a;
    P.vec_x = rows_aligned(a.x, a.ldx, sizeof(T), 16);
    P.vec_r = rows_aligned(a.residual, a.ldr, sizeof(R), 16) && rows_aligned(a.residual_out, a.ldr, sizeof(R), 16);
    P.vec_y = rows_aligned(a.y, a.ldy, sizeof(T), 16);
    P.vec_q = rows_aligned(a.q, a.ldq, 1, 8);
    P.vec_w = reinterpret_cast<uintptr_t>(a.weight) % 16 == 0;
    P.blocks = (a.cols + kScaleBlock - 1) / kScaleBlock;
    if (a.cols <= 256) return launch_norm_c<T, R, 1, true>(P, stream);
    if (a.cols <= 512) return launch_norm_c<T, R, 2, true>(P, stream);
    if (a.cols <= 1024) return launch_norm_c<T, R, 4, true>(P, stream);
    if (a.cols <= 4096) return launch_norm_c<T, R, 1, false>(P, stream);
    if (a.cols <= 8192) return launch_norm_c<T, R, 2, false>(P, stream);
    if (a.cols <= 32768) return launch_norm_c<T, R, 4, false>(P, stream);
    if (a.rows >= kMaxGrid) return AP_ERR_SHAPE;
    record_launch(PATH_NORM, a.rows, 0, 0, 0, 2);
    rms_norm_wide_kernel<T, R><<<static_cast<unsigned>(a.rows), 1024, 0, stream>>>(P);
    return launched();
}

// ------------------------------------------------------------------ gradient

struct GradParams {
    NormGradArgs a;
    bool vec_dy, vec_h, vec_r, vec_dx, vec_w;
};

// CTA b takes rows b, b + grid, ...; a thread keeps its columns' share of
// dweight in registers and writes it to the CTA's row of the workspace at the
// end, so the sum's order depends on the sizes alone.
template <typename T, typename R, int C>
__global__ void __launch_bounds__(512) rms_norm_grad_kernel(const __grid_constant__ GradParams P) {
    __shared__ float scratch[2][32];
    const NormGradArgs& a = P.a;
    float dw[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[c][i] = 0.0f;
    const float inv = __frcp_rn(static_cast<float>(a.cols));
    int turn = 0;  // two scratch rows in turn: one barrier a row is enough
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
        const T* dy = static_cast<const T*>(a.dy) + row * a.lddy;
        const R* h = static_cast<const R*>(a.h) + row * a.ldh;
        const float r = a.rstd[row];
        float g[C][8], n[C][8];
        float sum = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int64_t col = 8 * static_cast<int64_t>(c * blockDim.x + threadIdx.x);
            float w[8];
            load8(dy + col, P.vec_dy, a.cols - col).unpack(g[c]);
            load8(h + col, P.vec_h, a.cols - col).unpack(n[c]);
            load_weight<T>(a.weight, a.weight_type == a.type, P.vec_w, col, a.cols - col, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                n[c][i] *= r;
                dw[c][i] = fmaf(g[c][i], n[c][i], dw[c][i]);
                g[c][i] *= w[i];
                sum = fmaf(g[c][i], n[c][i], sum);
            }
        }
        const float mean = row_sum<false>(sum, scratch[turn]) * inv;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int64_t col = 8 * static_cast<int64_t>(c * blockDim.x + threadIdx.x);
            if (col >= a.cols) continue;
#pragma unroll
            for (int i = 0; i < 8; ++i) g[c][i] = fmaf(-n[c][i], mean, g[c][i]);
            float d[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (a.dresidual != nullptr)
                load8(static_cast<const R*>(a.dresidual) + row * a.lddr + col, P.vec_r, a.cols - col).unpack(d);
#pragma unroll
            for (int i = 0; i < 8; ++i) g[c][i] = fmaf(r, g[c][i], d[i]);
            store8(static_cast<R*>(a.dx) + row * a.lddx + col, P.vec_dx, a.cols - col, g[c]);
        }
    }
    if (a.dweight == nullptr) return;
    float* part = a.workspace + static_cast<int64_t>(blockIdx.x) * a.cols;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int64_t col = 8 * static_cast<int64_t>(c * blockDim.x + threadIdx.x);
        if (col < a.cols) store8(part + col, a.cols % 4 == 0, a.cols - col, dw[c]);
    }
}

// Rows too wide for registers: two passes over each row, and the CTA's share
// of dweight is added up in its row of the workspace (every thread its own
// columns).
template <typename T, typename R>
__global__ void __launch_bounds__(1024) rms_norm_grad_wide_kernel(const __grid_constant__ GradParams P) {
    __shared__ float scratch[2][32];
    const NormGradArgs& a = P.a;
    const float inv = __frcp_rn(static_cast<float>(a.cols));
    int turn = 0;
    const bool same = a.weight_type == a.type;
    auto weight = [&](int64_t j) {
        return same ? to_f32(static_cast<const T*>(a.weight)[j]) : static_cast<const float*>(a.weight)[j];
    };
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
        const T* dy = static_cast<const T*>(a.dy) + row * a.lddy;
        const R* h = static_cast<const R*>(a.h) + row * a.ldh;
        const float r = a.rstd[row];
        float sum = 0.0f;
        for (int64_t j = threadIdx.x; j < a.cols; j += blockDim.x)
            sum = fmaf(to_f32(dy[j]) * weight(j), to_f32(h[j]) * r, sum);
        const float mean = row_sum<false>(sum, scratch[turn]) * inv;
        for (int64_t j = threadIdx.x; j < a.cols; j += blockDim.x) {
            const float d = to_f32(dy[j]), n = to_f32(h[j]) * r;
            const float more =
                a.dresidual != nullptr ? to_f32(static_cast<const R*>(a.dresidual)[row * a.lddr + j]) : 0.0f;
            static_cast<R*>(a.dx)[row * a.lddx + j] = from_f32<R>(fmaf(r, fmaf(-n, mean, d * weight(j)), more));
            if (a.dweight != nullptr) {
                float* part = a.workspace + static_cast<int64_t>(blockIdx.x) * a.cols + j;
                *part = row == blockIdx.x ? d * n : fmaf(d, n, *part);
            }
        }
    }
}

// dweight from the CTAs' shares: a CTA sums 32 columns, eight rows of
// partials at a time, and adds the eight sums in order.
__global__ void __launch_bounds__(256) sum_partials_kernel(const float* part, float* out, int64_t parts, int64_t cols) {
    __shared__ float sums[8][32];
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x % 32;
    const int y = threadIdx.x / 32;
    float v = 0.0f;
    if (col < cols)
        for (int64_t p = y; p < parts; p += 8) v += part[p * cols + col];
    sums[y][threadIdx.x % 32] = v;
    __syncthreads();
    if (y == 0 && col < cols) {
#pragma unroll
        for (int i = 1; i < 8; ++i) v += sums[i][threadIdx.x];
        out[col] = v;
    }
}

constexpr int64_t kGradSMs = 152;  // the partials' number is part of the interface (workspace size), so no device query

template <typename T, typename R, int C>
void run_grad(const GradParams& P, int64_t grid, cudaStream_t stream) {
    const int64_t chunks = (P.a.cols + 7) / 8;
    const int threads = static_cast<int>(((chunks + C - 1) / C + 31) / 32 * 32);
    record_launch(PATH_NORM_GRAD, grid, 8 * C, 0, 0, 0);
    rms_norm_grad_kernel<T, R, C><<<static_cast<unsigned>(grid), threads, 0, stream>>>(P);
}

template <typename T, typename R>
ap_status launch_grad_t(const NormGradArgs& a, cudaStream_t stream) {
    GradParams P;
    P.a = a;
    P.vec_dy = rows_aligned(a.dy, a.lddy, sizeof(T), 16);
    P.vec_h = rows_aligned(a.h, a.ldh, sizeof(R), 16);
    P.vec_r = rows_aligned(a.dresidual, a.lddr, sizeof(R), 16);
    P.vec_dx = rows_aligned(a.dx, a.lddx, sizeof(R), 16);
    P.vec_w = reinterpret_cast<uintptr_t>(a.weight) % 16 == 0;
    const int64_t grid = norm_grad_partials(a.rows, a.cols);
    if (grid > 0) {
        if (a.cols <= 4096) {
            run_grad<T, R, 1>(P, grid, stream);
        } else if (a.cols <= 8192) {
            run_grad<T, R, 2>(P, grid, stream);
        } else if (a.cols <= 16384) {
            run_grad<T, R, 4>(P, grid, stream);
        } else {
            record_launch(PATH_NORM_GRAD, grid, 0, 0, 0, 2);
            rms_norm_grad_wide_kernel<T, R><<<static_cast<unsigned>(grid), 1024, 0, stream>>>(P);
        }
        const ap_status st = launched();
        if (st != AP_OK) return st;
    }
    if (a.dweight == nullptr) return AP_OK;
    sum_partials_kernel<<<static_cast<unsigned>((a.cols + 31) / 32), 256, 0, stream>>>(a.workspace, a.dweight, grid,
                                                                                      a.cols);
    return launched();
}

}  // namespace

// CTAs of the gradient's kernel: as many as are resident at once (by their
// threads), each with at least one row.
int64_t norm_grad_partials(int64_t rows, int64_t cols) {
    const int64_t per_sm = cols <= 2048 ? 8 : (cols <= 4096 ? 4 : 2);
    return std::min(rows, kGradSMs * per_sm);
}

ap_status launch_rms_norm(const DeviceInfo& di, const NormArgs& a, cudaStream_t stream) {
    const bool same = a.residual == nullptr || a.residual_type == a.type;
    switch (a.type) {
        case AP_BF16:
            return same ? launch_norm_t<__nv_bfloat16, __nv_bfloat16>(di, a, stream)
                        : launch_norm_t<__nv_bfloat16, float>(di, a, stream);
        case AP_F16:
            return same ? launch_norm_t<__half, __half>(di, a, stream) : launch_norm_t<__half, float>(di, a, stream);
        default: return launch_norm_t<float, float>(di, a, stream);
    }
}

ap_status launch_rms_norm_backward(const DeviceInfo&, const NormGradArgs& a, cudaStream_t stream) {
    const bool same = a.residual_type == a.type;
    switch (a.type) {
        case AP_BF16:
            return same ? launch_grad_t<__nv_bfloat16, __nv_bfloat16>(a, stream)
                        : launch_grad_t<__nv_bfloat16, float>(a, stream);
        case AP_F16: return same ? launch_grad_t<__half, __half>(a, stream) : launch_grad_t<__half, float>(a, stream);
        default: return launch_grad_t<float, float>(a, stream);
    }
}

}  // namespace ap
