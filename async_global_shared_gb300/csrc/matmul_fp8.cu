// c = a * b^T of e4m3 matrices with a scale for each block of 128 along k:
//     c[i, j] = sum over blocks kb of sa[i, kb] sb[j, kb] * P_kb[i, j],
//     P_kb[i, j] = sum over the block's 128 k of a[i, k] b[j, k].
// The scales differ from row to row and from block to block, so P_kb cannot
// stay in the tensor core's accumulator: each block's products go to their own
// accumulator in tensor memory, and consumer threads read it, multiply it by
// the two scales and add it to sums in registers while the tensor core works
// on the next block.
//
// One CTA computes a 128 x 128 tile. A producer thread streams the operands'
// 128 x 128-byte boxes through a ring of shared-memory stages (tensor maps,
// 128-byte swizzle, rows and columns past the matrix arrive as zeros); one
// thread issues the matrix instructions; four consumer warps own 32 rows each,
// one row a thread.
#include <atomic>

#include "device_common.cuh"
#include "fp8_common.cuh"
#include "internal.h"
#include "tcgen05.cuh"

namespace ap {
namespace {

constexpr int kTile = 128;               // rows of a, rows of b and bytes of k in one stage
constexpr int kMmaK = 32;                // k of one matrix instruction
constexpr int kStages = 6;
constexpr uint32_t kOperandBytes = kTile * kTile;
constexpr uint32_t kStageBytes = 2 * kOperandBytes;
constexpr int kConsumerWarps = 4;
constexpr int kThreads = 32 * (kConsumerWarps + 2);
constexpr uint32_t kTmemCols = 2 * kTile;  // two accumulators in turn

struct MatmulParams {
    const float* a_scales;
    const float* b_scales;
    void* c;
    int64_t m, n, ldc;
    int32_t nkb;      // blocks of k
    int32_t tiles_m;  // tiles along m
    bool vec_c;       // rows of c start on 16-byte boundaries
    uint32_t tx_extra;  // fault injection: bytes every stage waits for in vain
    uint64_t timeout_ns;
    uint32_t* status;
};

struct __align__(8) Shared {
    uint64_t full[kStages], empty[kStages];
    uint64_t acc_full[2], acc_empty[2];
    uint32_t tmem;
    int abort;
};

template <typename C, bool B_ROWS>
__global__ void __launch_bounds__(kThreads, 1)
    matmul_fp8_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                      const __grid_constant__ MatmulParams P) {
    extern __shared__ unsigned char smem_raw[];
    __shared__ Shared sh;
    __shared__ float col_scales[2][kTile];
    const uint32_t ring = (ptx::smem_addr(smem_raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t m0 = static_cast<int32_t>(blockIdx.x % P.tiles_m) * kTile;
    const int32_t n0 = static_cast<int32_t>(blockIdx.x / P.tiles_m) * kTile;
    volatile int* abort_flag = &sh.abort;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            ptx::mbar_init(ptx::smem_addr(&sh.full[s]), 1);
            ptx::mbar_init(ptx::smem_addr(&sh.empty[s]), 1);
        }
        for (int s = 0; s < 2; ++s) {
            ptx::mbar_init(ptx::smem_addr(&sh.acc_full[s]), 1);
            ptx::mbar_init(ptx::smem_addr(&sh.acc_empty[s]), kConsumerWarps);
        }
        sh.abort = 0;
        ptx::fence_mbar_init();
    }
    if (warp == kConsumerWarps) {
        ptx::tmem_alloc(ptx::smem_addr(&sh.tmem), kTmemCols);
        ptx::tmem_relinquish();
    }
    ptx::tcgen05_fence_before();
    __syncthreads();
    ptx::tcgen05_fence_after();
    const uint32_t tmem = sh.tmem;

    // A wait that gives up ends its role; the CTA's abort flag ends the others.
    auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t site) {
        const int w = wait_phase<false>(ptx::smem_addr(bar), parity, P.timeout_ns, abort_flag);
        if (w == WAIT_TIMEOUT) raise_timeout(P.status, site, abort_flag);
        return w == WAIT_OK;
    };

    if (warp == kConsumerWarps + 1) {
        if (lane == 0) {  // producer
            int issued = 0;
            for (; issued < P.nkb; ++issued) {
                const int s = issued % kStages;
                const uint32_t round = static_cast<uint32_t>(issued / kStages);
                if (round > 0 && !wait(&sh.empty[s], (round - 1) & 1, SITE_MM_PRODUCER_EMPTY)) break;
                const uint32_t bar = ptx::smem_addr(&sh.full[s]);
                ptx::mbar_arrive_expect_tx(bar, kStageBytes + P.tx_extra);
                ptx::tensor_g2s_2d(ring + s * kStageBytes, &map_a, issued * kTile, m0, bar);
                ptx::tensor_g2s_2d(ring + s * kStageBytes + kOperandBytes, &map_b, issued * kTile, n0, bar);
            }
            // nothing may still be landing in this CTA's shared memory or
            // arriving on its barriers when it leaves
            for (int i = issued > kStages ? issued - kStages : 0; i < issued; ++i) {
                const uint32_t parity = static_cast<uint32_t>(i / kStages) & 1;
                if (!drain_wait<false>(ptx::smem_addr(&sh.full[i % kStages]), parity, P.timeout_ns, P.status,
                                       SITE_MM_DRAIN, abort_flag) ||
                    !drain_wait<false>(ptx::smem_addr(&sh.empty[i % kStages]), parity, P.timeout_ns, P.status,
                                       SITE_MM_DRAIN, abort_flag))
                    break;
            }
        }
    } else if (warp == kConsumerWarps) {
        if (lane == 0) {  // matrix instructions
            constexpr uint32_t idesc = ptx::e4m3_instr_desc(kTile, kTile);
            for (int kb = 0; kb < P.nkb; ++kb) {
                const int s = kb % kStages, buf = kb & 1;
                const uint32_t turn = static_cast<uint32_t>(kb >> 1);
                if (turn > 0 && !wait(&sh.acc_empty[buf], (turn - 1) & 1, SITE_MM_MMA_ACC)) break;
                if (!wait(&sh.full[s], static_cast<uint32_t>(kb / kStages) & 1, SITE_MM_MMA_FULL)) break;
                ptx::tcgen05_fence_after();
                const uint64_t da = ptx::operand_desc(ring + s * kStageBytes);
                const uint64_t db = ptx::operand_desc(ring + s * kStageBytes + kOperandBytes);
#pragma unroll
                for (int k = 0; k < kTile / kMmaK; ++k)
                    ptx::mma_e4m3(tmem + buf * kTile, da + k * (kMmaK >> 4), db + k * (kMmaK >> 4), idesc, k > 0);
                ptx::mma_commit(ptx::smem_addr(&sh.empty[s]));
                ptx::mma_commit(ptx::smem_addr(&sh.acc_full[buf]));
            }
        }
    } else {  // consumers: thread = row m0 + 32 * warp + lane, all columns
        const int64_t row = m0 + 32 * warp + lane;
        const float* sa = P.a_scales + (row < P.m ? row : P.m - 1) * P.nkb;
        const int64_t my_col = n0 + 32 * warp + lane;  // B_ROWS: the column whose scales this thread fetches
        const float* sb = B_ROWS ? P.b_scales + (my_col < P.n ? my_col : P.n - 1) * P.nkb
                                 : P.b_scales + static_cast<int64_t>(n0 / kTile) * P.nkb;
        float acc[kTile];
#pragma unroll
        for (int j = 0; j < kTile; ++j) acc[j] = 0.0f;
        for (int kb = 0; kb < P.nkb; ++kb) {
            const int buf = kb & 1;
            float scale = sa[kb];
            if (B_ROWS) {
                col_scales[buf][32 * warp + lane] = sb[kb];
                ptx::named_barrier_sync(1, 32 * kConsumerWarps);
            } else {
                scale *= sb[kb];
            }
            // a lane that gave up must not leave its warp's collective loads
            const bool ok = wait(&sh.acc_full[buf], static_cast<uint32_t>(kb >> 1) & 1, SITE_MM_CONSUMER_ACC);
            if (!B_ROWS && !__all_sync(0xffffffffu, ok)) break;
            if (__all_sync(0xffffffffu, ok)) {
                ptx::tcgen05_fence_after();
                const uint32_t at = tmem + buf * kTile + (static_cast<uint32_t>(32 * warp) << 16);
                float v[2][16];
                ptx::tmem_ld16(at, v[0]);
#pragma unroll
                for (int g = 0; g < kTile / 16; ++g) {
                    ptx::tmem_wait_ld(v[g & 1]);
                    if (g + 1 < kTile / 16) ptx::tmem_ld16(at + 16 * (g + 1), v[(g + 1) & 1]);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int j = 16 * g + i;
                        acc[j] = fmaf(v[g & 1][i], B_ROWS ? scale * col_scales[buf][j] : scale, acc[j]);
                    }
                }
                ptx::tcgen05_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&sh.acc_empty[buf]));
            }
        }
        if (row < P.m && !*abort_flag) {
            C* out = static_cast<C*>(P.c) + row * P.ldc + n0;
#pragma unroll
            for (int j = 0; j < kTile; j += 8) {
                const int64_t left = P.n - n0 - j;
                if (left > 0) store8(out + j, P.vec_c, left, *reinterpret_cast<const float(*)[8]>(&acc[j]));
            }
        }
    }
    __syncwarp();  // the one-thread roles' idle lanes wait here
    ptx::tcgen05_fence_before();
    __syncthreads();
    ptx::tcgen05_fence_after();
    if (warp == kConsumerWarps) ptx::tmem_dealloc(tmem, kTmemCols);
}

// A rows x k byte matrix as boxes of 128 bytes by box_rows rows.
bool operand_map(CUtensorMap* map, const uint8_t* p, int64_t rows, int64_t k, int64_t ld, uint32_t box_rows) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(k), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(kTile), box_rows};
    const cuuint32_t estr[2] = {1, 1};
    auto encode = tensor_map_encoder();
    return encode != nullptr &&
           encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(p), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename C, bool B_ROWS>
ap_status launch_mm(const DeviceInfo& di, const MatmulParams& P, const CUtensorMap& ma, const CUtensorMap& mb,
                    int64_t grid, cudaStream_t stream) {
    constexpr size_t smem = kStages * kStageBytes + 1024;
    static std::atomic<int> configured[64];  // attribute set on this device (setting twice is harmless)
    if (di.device < 0 || di.device >= 64) return AP_ERR_CUDA;
    if (!configured[di.device].load()) {
        if (cudaFuncSetAttribute(matmul_fp8_kernel<C, B_ROWS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(smem)) != cudaSuccess)
            return AP_ERR_CUDA;
        configured[di.device] = 1;
    }
    record_launch(PATH_MATMUL, grid, kTile, static_cast<int64_t>(smem), kStages, B_ROWS ? 1 : 0);
    matmul_fp8_kernel<C, B_ROWS><<<static_cast<unsigned>(grid), kThreads, smem, stream>>>(ma, mb, P);
    return cudaGetLastError() == cudaSuccess ? AP_OK : AP_ERR_CUDA;
}

template <typename C>
ap_status launch_mm_c(const DeviceInfo& di, const MatmulParams& P, const CUtensorMap& ma, const CUtensorMap& mb,
                      int64_t grid, bool b_rows, cudaStream_t stream) {
    return b_rows ? launch_mm<C, true>(di, P, ma, mb, grid, stream) : launch_mm<C, false>(di, P, ma, mb, grid, stream);
}

}  // namespace

ap_status launch_matmul_fp8(const DeviceInfo& di, const Options& o, const MatmulArgs& a, cudaStream_t stream) {
    const int64_t size = a.c_type == AP_F32 ? 4 : 2;
    if (a.k == 0) {
        return cudaMemset2DAsync(a.c, static_cast<size_t>(a.ldc * size), 0, static_cast<size_t>(a.n * size),
                                 static_cast<size_t>(a.m), stream) == cudaSuccess
                   ? AP_OK
                   : AP_ERR_CUDA;
    }
    MatmulParams P;
    P.a_scales = a.a_scales;
    P.b_scales = a.b_scales;
    P.c = a.c;
    P.m = a.m;
    P.n = a.n;
    P.ldc = a.ldc;
    P.nkb = static_cast<int32_t>((a.k + kTile - 1) / kTile);
    P.tiles_m = static_cast<int32_t>((a.m + kTile - 1) / kTile);
    P.vec_c = rows_aligned(a.c, a.ldc, size, 16);
    P.tx_extra = static_cast<uint32_t>(o.tx_extra);
    P.timeout_ns = static_cast<uint64_t>(o.timeout_ns);
    P.status = di.status;
    const int64_t grid = P.tiles_m * ((a.n + kTile - 1) / kTile);
    if (grid >= (int64_t(1) << 31)) return AP_ERR_SHAPE;
    CUtensorMap ma, mb;
    if (!operand_map(&ma, a.a, a.m, a.k, a.lda, kTile) || !operand_map(&mb, a.b, a.n, a.k, a.ldb, kTile))
        return AP_ERR_CUDA;
    const bool b_rows = a.b_block_rows == 1;
    switch (a.c_type) {
        case AP_BF16: return launch_mm_c<__nv_bfloat16>(di, P, ma, mb, grid, b_rows, stream);
        case AP_F16: return launch_mm_c<__half>(di, P, ma, mb, grid, b_rows, stream);
        default: return launch_mm_c<float>(di, P, ma, mb, grid, b_rows, stream);
    }
}

}  // namespace ap
