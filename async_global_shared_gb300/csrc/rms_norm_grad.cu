// Gradient of the root-mean-square norm. With n = h r and g = dy w: r depends on
// every h of the row, d r / d h_i = -r^3 h_i / N, so
//     dx = r (g - n mean(g n)) + dresidual,   dw_j = sum over rows of dy n.
// The mean comes before the first dx, so a row is held on the chip between the
// two and memory is passed over once. Memory bounds it: 16384 x 8192 bf16 with
// dresidual 161 us = 6.7 TB/s (415 with one row a CTA in registers); 777 x 2560
// f32 11.6 us, of which 4 are the two kernels' launches; 6062 x 2694 f16 and f32,
// rows off the 16-byte boundaries, 37 us = 4.4 TB/s.
#include "row_ring.cuh"

namespace ap {
namespace {

struct GradParams {
    NormGradArgs a;
};

// Few rows, or wider than the ring takes: CTA b takes rows b, b + grid, ...; a thread keeps its columns' share of
// dweight in registers and writes it to the CTA's row of the workspace at the
// end, so the sum's order depends on the sizes alone.
template <typename T, typename R, int C, bool SPREAD>
__global__ void __launch_bounds__(512) rms_norm_grad_kernel(const __grid_constant__ GradParams P) {
    __shared__ float scratch[2][32];
    ptx::let_next_grid_start();
    ptx::wait_previous_grid();
    const NormGradArgs& a = P.a;
    float dw[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[c][i] = 0.0f;
    const float inv = __frcp_rn(static_cast<float>(a.cols));
    const int first = first_column<SPREAD>(threadIdx.x), apart = 8 * blockDim.x, cols = static_cast<int>(a.cols);
    int turn = 0;  // two scratch rows in turn: one barrier a row is enough
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
        const T* dy = static_cast<const T*>(a.dy) + row * a.lddy;
        const R* h = static_cast<const R*>(a.h) + row * a.ldh;
        const float r = a.rstd[row];
        float g[C][8], n[C][8];
        float sum = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int col = first + c * apart;
            float w[8];
            take<SPREAD>(dy + col, cols - col, g[c]);
            take<SPREAD>(h + col, cols - col, n[c]);
            take_weight<SPREAD, T>(a.weight, a.weight_type == a.type, col, cols - col, w);
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
            const int col = first + c * apart;
            if (col >= cols) continue;
#pragma unroll
            for (int i = 0; i < 8; ++i) g[c][i] = fmaf(-n[c][i], mean, g[c][i]);
            float d[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (a.dresidual != nullptr) take<SPREAD>(static_cast<const R*>(a.dresidual) + row * a.lddr + col, cols - col, d);
#pragma unroll
            for (int i = 0; i < 8; ++i) g[c][i] = fmaf(r, g[c][i], d[i]);
            put<SPREAD>(static_cast<R*>(a.dx) + row * a.lddx + col, cols - col, g[c]);
        }
    }
    if (a.dweight == nullptr) return;
    float* part = a.workspace + static_cast<int64_t>(blockIdx.x) * a.cols;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int col = first + c * apart;
        put<SPREAD>(part + col, cols - col, dw[c]);
    }
}

// The ring's form: teams of warps, rows and their rstd from shared memory. A
// thread's columns are the same for every row, so it keeps their weights (four
// chunks: in shared memory) and their share of dweight in registers.
template <typename T, typename R, int C, bool RES, Weights W, bool SPREAD>
__global__ void __launch_bounds__(kRingThreads, 1)
    rms_norm_grad_ring_kernel(const __grid_constant__ GradParams P, const __grid_constant__ RowRing ring) {
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ RingBars bars;
    __shared__ float scratch[2][kRingWarps];
    constexpr bool kKeep = W == IN_REGISTERS;
    ptx::let_next_grid_start();
    ring_init(ring, bars);
    const NormGradArgs& a = P.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == kRingWarps) {
        ring_produce(ring, bars, ptx::smem_addr(smem));
        return;
    }
    const bool same = a.weight_type == a.type;
    float* weights = reinterpret_cast<float*>(smem + ring.weight_offset);
    if (W == IN_SHARED) stage_weights<T>(a.weight, same, a.cols, weights);
    const int team = warp / ring.team_warps, width = 32 * ring.team_warps;
    if (team >= ring.teams) return;
    const int me = threadIdx.x - team * width;
    const int first = first_column<SPREAD>(me), apart = 8 * width, cols = static_cast<int>(a.cols);
    float w[kKeep ? C : 1][8];
    if (kKeep) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int col = first + c * apart;
            if (col < cols) take_weight<SPREAD, T>(a.weight, same, col, cols - col, w[kKeep ? c : 0]);
        }
    }
    float dw[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[c][i] = 0.0f;
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
            if (mine) {
                // the row is read from shared memory again after its sum: that
                // is cheaper than the registers it would take
                const T* p = reinterpret_cast<const T*>(stage + row_place<SPREAD>(ring, 0, base, slot));
                const R* q = reinterpret_cast<const R*>(stage + ring.offset[1] + row_place<SPREAD>(ring, 1, base, slot));
                const float r = reinterpret_cast<const float*>(stage + ring.side_offset)[slot];
                float sum = 0.0f;
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const int col = first + c * apart;
                    if (col >= cols) continue;
                    float g[8], n[8], again[8];
                    take<SPREAD>(p + col, cols - col, g);
                    take<SPREAD>(q + col, cols - col, n);
                    if (!kKeep) again_weight<T, W, SPREAD>(P, weights, col, cols - col, again);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        n[i] *= r;
                        dw[c][i] = fmaf(g[i], n[i], dw[c][i]);
                        sum = fmaf(g[i] * (kKeep ? w[kKeep ? c : 0][i] : again[i]), n[i], sum);
                    }
                }
                const float mean = team_sum(sum, &scratch[turn][team * ring.team_warps], team, ring.team_warps) * inv;
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const int col = first + c * apart;
                    if (col >= cols) continue;
                    float g[8], n[8], d[8] = {0, 0, 0, 0, 0, 0, 0, 0}, again[8];
                    take<SPREAD>(p + col, cols - col, g);
                    take<SPREAD>(q + col, cols - col, n);
                    if (RES)
                        take<SPREAD>(reinterpret_cast<const R*>(stage + ring.offset[2] + row_place<SPREAD>(ring, 2, base, slot)) + col,
                                     cols - col, d);
                    if (!kKeep) again_weight<T, W, SPREAD>(P, weights, col, cols - col, again);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float gw = g[i] * (kKeep ? w[kKeep ? c : 0][i] : again[i]);
                        g[i] = fmaf(r, fmaf(-(n[i] * r), mean, gw), d[i]);
                    }
                    put<SPREAD>(static_cast<R*>(a.dx) + row * a.lddx + col, cols - col, g);
                }
            }
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&bars.empty[s]));
        s += groups;
        while (s >= ring.stages) s -= ring.stages, ++round;
    }
    if (a.dweight == nullptr) return;
    // the teams' shares, added in their order through the ring's memory (every
    // copy has landed and been read)
    float* part = a.workspace + static_cast<int64_t>(blockIdx.x) * a.cols;
    float* shares = reinterpret_cast<float*>(smem);
    if (ring.teams > 1) {
        const int all = ring.teams * width;
        ptx::named_barrier_sync(15, all);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int col = first + c * apart;
            put<SPREAD>(shares + team * cols + col, cols - col, dw[c]);
        }
        ptx::named_barrier_sync(15, all);
        for (int col = threadIdx.x; col < cols; col += all) {
            float v = shares[col];
            for (int t = 1; t < ring.teams; ++t) v += shares[t * cols + col];
            part[col] = v;
        }
    } else {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int col = first + c * apart;
            put<SPREAD>(part + col, cols - col, dw[c]);
        }
    }
}

// Rows too wide for registers: two passes over each row, and the CTA's share
// of dweight is added up in its row of the workspace (every thread its own
// columns).
template <typename T, typename R>
__global__ void __launch_bounds__(1024) rms_norm_grad_wide_kernel(const __grid_constant__ GradParams P) {
    __shared__ float scratch[2][32];
    ptx::let_next_grid_start();
    ptx::wait_previous_grid();
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
    ptx::let_next_grid_start();
    ptx::wait_previous_grid();
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

// The ring's set-up is not paid back where a CTA has two rows at most and they
// are few elements in all (304 x 1000: 11.5 us against 10.6 without, 608 x
// 1001: 11.8 against 10.6; the other way 1216 x 1001: 11.5 against 14.9, 304 x
// 11003: 15.6 against 23.5).
constexpr int64_t kFewElements = int64_t(1) << 20;
constexpr int64_t kGradSMs = 152;  // the partials' number is part of the interface (workspace size), so no device query

template <typename T, typename R, int C>
ap_status run_grad(const GradParams& P, bool whole, int64_t grid, cudaStream_t stream) {
    const int64_t chunks = (P.a.cols + 7) / 8;
    const int threads = static_cast<int>(((chunks + C - 1) / C + 31) / 32 * 32);
    record_launch(PATH_NORM_GRAD, grid, 8 * C, 0, 0, whole ? 0 : 8);
    return whole ? launch_early(rms_norm_grad_kernel<T, R, C, false>, grid, threads, stream, P)
                 : launch_early(rms_norm_grad_kernel<T, R, C, true>, grid, threads, stream, P);
}

template <typename T, typename R, bool RES, bool SPREAD>
ap_status launch_grad_ring(const DeviceInfo& di, const GradParams& P, const RowRing& ring, int64_t grid, cudaStream_t stream) {
    static std::atomic<int> configured[5][64];
    if (ring.chunks == 2)
        return launch_ring_kernel(di, rms_norm_grad_ring_kernel<T, R, 2, RES, IN_REGISTERS, SPREAD>, configured[0], P, ring, grid, PATH_NORM_GRAD, stream);
    if (ring.chunks == 3)
        return ring.keep_weights
                   ? launch_ring_kernel(di, rms_norm_grad_ring_kernel<T, R, 3, RES, IN_SHARED, SPREAD>, configured[1], P, ring, grid, PATH_NORM_GRAD, stream)
                   : launch_ring_kernel(di, rms_norm_grad_ring_kernel<T, R, 3, RES, IN_L2, SPREAD>, configured[2], P, ring, grid, PATH_NORM_GRAD, stream);
    return ring.keep_weights
               ? launch_ring_kernel(di, rms_norm_grad_ring_kernel<T, R, 4, RES, IN_SHARED, SPREAD>, configured[3], P, ring, grid, PATH_NORM_GRAD, stream)
               : launch_ring_kernel(di, rms_norm_grad_ring_kernel<T, R, 4, RES, IN_L2, SPREAD>, configured[4], P, ring, grid, PATH_NORM_GRAD, stream);
}

// Which kernel a call takes, and its CTAs: each writes one row of partial sums,
// so the sum over them takes the same number.
struct GradPlan {
    bool whole, rings;
    RowRing ring;
    int64_t grid;
};

template <typename T, typename R>
GradPlan plan_grad(const DeviceInfo& di, const Options& o, const NormGradArgs& a) {
    GradPlan g{};
    const void* const in[] = {a.dy, a.h, a.dresidual};
    const int64_t ld[] = {a.lddy, a.ldh, a.lddr}, size[] = {sizeof(T), sizeof(R), sizeof(R)};
    const bool res = a.dresidual != nullptr;
    g.whole = a.cols % 8 == 0 && rows_aligned(a.dy, a.lddy, sizeof(T), 16) && rows_aligned(a.h, a.ldh, sizeof(R), 16) &&
              (!res || rows_aligned(a.dresidual, a.lddr, sizeof(R), 16)) && rows_aligned(a.dx, a.lddx, sizeof(R), 16) &&
              reinterpret_cast<uintptr_t>(a.weight) % 16 == 0;
    g.grid = norm_grad_partials(a.rows, a.cols);
    const bool few = a.rows <= 4 * kGradSMs && a.rows <= kFewElements / a.cols;
    g.rings = a.rows > 0 && o.force_path != 2 && (o.force_path == 1 || !few) &&
              plan_ring(di, o, &g.ring, res ? 3 : 2, in, ld, size, a.rstd, a.rows, a.cols, g.whole);
    if (g.rings) g.grid = std::min(g.grid, ring_grid(g.ring, di.sms, o.grid));
    return g;
}

template <typename T, typename R>
ap_status launch_grad_t(const DeviceInfo& di, const Options& o, const NormGradArgs& a, cudaStream_t stream) {
    GradParams P;
    P.a = a;
    const GradPlan g = plan_grad<T, R>(di, o, a);
    const bool res = a.dresidual != nullptr;
    if (g.grid > 0) {
        ap_status st;
        if (g.rings) {
            if (g.whole)
                st = res ? launch_grad_ring<T, R, true, false>(di, P, g.ring, g.grid, stream)
                         : launch_grad_ring<T, R, false, false>(di, P, g.ring, g.grid, stream);
            else
                st = res ? launch_grad_ring<T, R, true, true>(di, P, g.ring, g.grid, stream)
                         : launch_grad_ring<T, R, false, true>(di, P, g.ring, g.grid, stream);
        } else if (a.cols <= 4096) {
            st = run_grad<T, R, 1>(P, g.whole, g.grid, stream);
        } else if (a.cols <= 8192) {
            st = run_grad<T, R, 2>(P, g.whole, g.grid, stream);
        } else if (a.cols <= 16384) {
            st = run_grad<T, R, 4>(P, g.whole, g.grid, stream);
        } else {
            record_launch(PATH_NORM_GRAD, g.grid, 0, 0, 0, 2);
            st = launch_early(rms_norm_grad_wide_kernel<T, R>, g.grid, 1024, stream, P);
        }
        if (st != AP_OK) return st;
    }
    if (a.dweight == nullptr) return AP_OK;
    return launch_early(sum_partials_kernel, (a.cols + 31) / 32, 256, stream, static_cast<const float*>(a.workspace),
                        a.dweight, g.grid, a.cols);
}

// f of the kernels' element types for these of the arguments.
template <typename F>
auto with_types(const NormGradArgs& a, F f) {
    const bool same = a.residual_type == a.type;
    switch (a.type) {
        case AP_BF16: return same ? f(__nv_bfloat16(), __nv_bfloat16()) : f(__nv_bfloat16(), 0.0f);
        case AP_F16: return same ? f(__half(), __half()) : f(__half(), 0.0f);
        default: return f(0.0f, 0.0f);
    }
}

}  // namespace

// CTAs of the gradient's kernels at most: the ring runs one an SM, the others
// two, each with at least one row.
int64_t norm_grad_partials(int64_t rows, int64_t) { return std::min(rows, kGradSMs * 2); }

ap_status launch_rms_norm_backward(const DeviceInfo& di, const Options& o, const NormGradArgs& a, cudaStream_t stream) {
    return with_types(a, [&](auto t, auto r) { return launch_grad_t<decltype(t), decltype(r)>(di, o, a, stream); });
}

int64_t norm_grad_ctas(const DeviceInfo& di, const Options& o, const NormGradArgs& a) {
    return with_types(a, [&](auto t, auto r) { return plan_grad<decltype(t), decltype(r)>(di, o, a).grid; });
}

}  // namespace ap
