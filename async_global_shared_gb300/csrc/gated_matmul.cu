// y = act(a Wg^T) * (a Wu^T) of 8-bit block-scaled matrices: the matrix product's
// kernel (matmul_fp8.cuh) with both weights' products in one accumulator, and
// the activation, the product and y's rounding to e4m3 where the sums are.
//
// What bounds it: one row of a times 16384 x 4096, the weights' bytes, 24.9 us = 5.4 TB/s, about 5
// of them start, fill and reduction. 8192 x 16384 x 4096 with both products and e4m3 out
// in pairs of CTAs: 975 to 1005 us = 2.2 PFLOP/s, the consumers' loads and sums as for the plain
// product (2.5), and about a tenth for the results' arithmetic and staging. 333 x 5000 x
// 4104, a CTA a tile: 26 to 27 us, 120 tiles on 152 SMs.
#include "matmul_fp8.cuh"

namespace ap {
namespace {

// No columns of a: every product is 0, and so is y.
template <typename C>
__global__ void __launch_bounds__(256) gated_zero_kernel(C* gate, C* up, C* y, uint8_t* q, float* q_scales, int64_t ldg, int64_t ldu,
                                                         int64_t ldy, int64_t ldq, int64_t m, int64_t n, int64_t blocks) {
    for (int64_t row = blockIdx.x; row < m; row += gridDim.x) {
        for (int64_t j = threadIdx.x; j < n; j += 256) {
            if (gate != nullptr) gate[row * ldg + j] = from_f32<C>(0.0f);
            if (up != nullptr) up[row * ldu + j] = from_f32<C>(0.0f);
            if (y != nullptr) y[row * ldy + j] = from_f32<C>(0.0f);
            if (q != nullptr) q[row * ldq + j] = 0;
            if (q != nullptr && j < blocks) q_scales[row * blocks + j] = kMinScale;
        }
    }
}

template <typename C, int BN, int CG, int STAGES, bool SWAP>
ap_status launch_form(const DeviceInfo& di, MatmulParams P, GateParams G, const GatedArgs& a, cudaStream_t stream) {
    using F = Form<BN, CG, STAGES, SWAP, SWAP, true>;
    static_assert(checked<BN, CG, STAGES, SWAP, SWAP, true>());
    P.np = SWAP ? a.n : a.m;
    P.nq = SWAP ? a.m : a.n;
    P.p_scales = SWAP ? a.gate_scales : a.a_scales;
    P.q_scales = SWAP ? a.a_scales : a.gate_scales;
    P.p_shift = 0;
    const int64_t tiles_p = (P.np + CG * kTile - 1) / (CG * kTile), tiles_q = (P.nq + F::kTileCols - 1) / F::kTileCols;
    const int64_t tiles = tiles_p * tiles_q;
    if (tiles > kMaxTiles) return AP_ERR_SHAPE;
    P.tiles_p = static_cast<int32_t>(tiles_p);
    P.tiles_q = static_cast<int32_t>(tiles_q);
    auto kernel = matmul_fp8_kernel<C, BN, CG, STAGES, SWAP, SWAP, true>;
    static std::atomic<int> configured[64];  // attribute set on this device (setting twice is harmless)
    static std::atomic<int> resident[64][kMaxSplit + 1];
    if (di.device < 0 || di.device >= 64) return AP_ERR_CUDA;
    if (!configured[di.device].load()) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(F::kSmem)) != cudaSuccess)
            return AP_ERR_CUDA;
        configured[di.device] = 1;
    }
    P.split = CG == 2 ? 1 : split_for(kernel, F::kThreads, F::kSmem, F::kCtas, resident[di.device], tiles, P.nkb);
    CUtensorMap mp, mq;
    constexpr auto codes = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    constexpr uint32_t box = SWAP ? kTile : F::kQBox;  // rows of a weight's box
    if (!box_map(SWAP ? &mp : &mq, codes, a.gate, 1, a.n, a.k, a.ldg, box) || !box_map(&G.up, codes, a.up, 1, a.n, a.k, a.ldu, box) ||
        !box_map(SWAP ? &mq : &mp, codes, a.a, 1, a.m, a.k, a.lda, SWAP ? F::kQBox : kTile))
        return AP_ERR_CUDA;
    if (CG == 2) {  // results by tensor maps, 32 rows of 128 bytes (codes: 64) a box
        constexpr auto type = sizeof(C) == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16;
        if ((G.gate_out != nullptr && G.vec_gate && !box_map(&G.out_gate, type, G.gate_out, sizeof(C), a.m, a.n, G.ldg, 32)) ||
            (G.up_out != nullptr && G.vec_up && !box_map(&G.out_up, type, G.up_out, sizeof(C), a.m, a.n, G.ldu, 32)) ||
            (G.y != nullptr && G.vec_y && !box_map(&G.out_y, type, G.y, sizeof(C), a.m, a.n, G.ldy, 32)) ||
            (G.q != nullptr && G.vec_q && !box_map(&G.out_q, codes, G.q, 1, a.m, a.n, G.ldq, 32, 64)))
            return AP_ERR_CUDA;
    }
    const int cluster = CG == 2 ? 2 : P.split;
    int64_t grid = tiles * cluster;  // one CTA or cluster a tile, whose sums end in the ring's place; pairs walk the tiles
    if (CG == 2) grid = std::min<int64_t>(grid, di.sms / 2 * 2);
    if (grid >= (int64_t(1) << 31)) return AP_ERR_SHAPE;
    record_launch(PATH_GATED_MATMUL, grid, BN, static_cast<int64_t>(F::kSmem), STAGES, (SWAP ? 1 : 0) | (CG == 2 ? 2 : 0) | P.split << 4);
    Launch l(grid, F::kThreads, F::kSmem, cluster, stream);
    return cudaLaunchKernelEx(&l.cfg, kernel, mp, mq, CUtensorMap{}, P, G) == cudaSuccess ? AP_OK : AP_ERR_CUDA;
}

template <typename C>
ap_status launch_t(const DeviceInfo& di, int64_t force, const MatmulParams& P, const GateParams& G, const GatedArgs& a, cudaStream_t stream) {
    if (a.k == 0) {
        const int64_t grid = std::min<int64_t>(a.m, 4 * di.sms);
        gated_zero_kernel<C><<<static_cast<unsigned>(grid), 256, 0, stream>>>(
            static_cast<C*>(G.gate_out), static_cast<C*>(G.up_out), static_cast<C*>(G.y), G.q, G.q_scales, G.ldg, G.ldu, G.ldy, G.ldq, a.m,
            a.n, G.blocks);
        return cudaGetLastError() == cudaSuccess ? AP_OK : AP_ERR_CUDA;
    }
    // As for the plain product: few rows of a on the narrow side, pairs from half
    // the SMs' worth of their tiles (256 rows by 128 columns of y) on, else a
    // CTA or cluster a tile of 128 x 128. A CTA by itself loads half again as
    // many bytes a stage, and its tile takes about 4 / 3 of the time of a pair's (2048
    // x 4096 x 4096: 84 us, 68 in pairs; with g, u and e4m3 98 and 72); but where the
    // rows' last 128 would be empty for a pair it may save a round of tiles (333 x 5000 x
    // 4104: 27 us in one round, 37 in the pairs' two; 384 x 16384 x 4096, three rounds
    // against four: 65 and 68 us, with e4m3 72 and 69).
    if (a.m <= 16) return launch_form<C, 16, 1, 5, true>(di, P, G, a, stream);
    if (a.m <= 32) return launch_form<C, 32, 1, 5, true>(di, P, G, a, stream);
    const int64_t pairs = (a.m + 2 * kTile - 1) / (2 * kTile) * ((a.n + kTile - 1) / kTile);
    const int64_t alone = (a.m + kTile - 1) / kTile * ((a.n + kTile - 1) / kTile);
    const int64_t rounds = (alone + di.sms - 1) / di.sms, pair_rounds = (pairs + di.sms / 2 - 1) / (di.sms / 2);
    const bool paired = a.m > kTile && pairs >= di.sms / 4 && 3 * pair_rounds <= 4 * rounds;
    if (force == 2 || (force != 1 && paired)) return launch_form<C, 256, 2, 5, false>(di, P, G, a, stream);
    return launch_form<C, 256, 1, 4, false>(di, P, G, a, stream);
}

}  // namespace

ap_status launch_gated_matmul(const DeviceInfo& di, const Options& o, const GatedArgs& a, cudaStream_t stream) {
    const int64_t size = a.type == AP_F32 ? 4 : 2;
    MatmulParams P{};
    P.nkb = static_cast<int32_t>((a.k + kTile - 1) / kTile);
    P.tx_extra = static_cast<uint32_t>(o.tx_extra);
    P.timeout_ns = static_cast<uint64_t>(o.timeout_ns);
    P.status = di.status;
    GateParams G{};
    G.up_scales = a.up_scales;
    G.gate_out = a.gate_out;
    G.up_out = a.up_out;
    G.y = a.y;
    G.q = a.q;
    G.q_scales = a.q_scales;
    G.ldg = a.ld_gate_out;
    G.ldu = a.ld_up_out;
    G.ldy = a.ldy;
    G.ldq = a.ldq;
    G.n = a.n;
    G.blocks = (a.n + kScaleBlock - 1) / kScaleBlock;
    G.vec_gate = rows_aligned(a.gate_out, a.ld_gate_out, size, 16);
    G.vec_up = rows_aligned(a.up_out, a.ld_up_out, size, 16);
    G.vec_y = rows_aligned(a.y, a.ldy, size, 16);
    G.vec_q = rows_aligned(a.q, a.ldq, 1, 16);
    G.act = gate_of(a.act);
    switch (a.type) {
        case AP_BF16: return launch_t<__nv_bfloat16>(di, o.force_path, P, G, a, stream);
        case AP_F16: return launch_t<__half>(di, o.force_path, P, G, a, stream);
        default: return launch_t<float>(di, o.force_path, P, G, a, stream);
    }
}

}  // namespace ap
