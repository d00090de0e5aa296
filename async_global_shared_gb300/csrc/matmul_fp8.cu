// The 8-bit matrix product's forms and the rules that choose between them; the
// kernel is in matmul_fp8.cuh.
#include "matmul_fp8.cuh"

namespace ap {
namespace {

template <typename C, int BN, int CG, int STAGES, bool PER_COL, bool SWAP>
ap_status launch_form(const DeviceInfo& di, MatmulParams P, const MatmulArgs& a, cudaStream_t stream) {
    using F = Form<BN, CG, STAGES, PER_COL, SWAP>;
    static_assert(checked<BN, CG, STAGES, PER_COL, SWAP>());
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
    return cudaLaunchKernelEx(&l.cfg, kernel, mp, mq, mc, P, NoGate{}) == cudaSuccess ? AP_OK : AP_ERR_CUDA;
}

template <typename C>
ap_status launch_mm(const DeviceInfo& di, const MatmulParams& P, const MatmulArgs& a, cudaStream_t stream) {
    const bool rows = a.b_block_rows == 1;
    // Few rows: the weight on the accumulator's rows, a's rows padded to 16 or
    // 32 (times 8192 x 8192: one row 14.2 us, 15.4 padded to 32; 32 rows 16.2,
    // 48 in the 128 x 128 form 18.7).
    if (a.m <= 16) return launch_form<C, 16, 1, 4, true, true>(di, P, a, stream);
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
