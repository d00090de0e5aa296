// The gradient of y = act(g) u: from dy (y's gradient), g and u
//     dg = dy u act'(g),  du = dy act(g),
// in the inputs' type, and in e4m3 as the products of a training step read
// them: [dg | du] side by side by row blocks, the same transposed, and
// h = act(g) u transposed, which the down projection's weight gradient needs
// and which the forward pass then need not keep.
//
// Floor: three inputs read once, each output written once (8192 x 16384 bf16 with
// all codes, silu: 221 us; it takes 358, 66 % of the issue slots busy with about 70
// instructions an element, and at the 128 registers of two CTAs an SM the 16-bit forms
// spill 60 to 84 bytes a thread; 1237 x 5000 fp16 with all outputs 14 and 34, two rounds
// of tiles; values alone, 4096 x 16384 bf16, 99 and 98). A block's scale
// needs its largest magnitude before the first code, and five kinds of codes
// (dg, du by rows; dg, du, h by columns) of a 128 x 128 tile are more than
// registers hold, so the tile's inputs stay in shared memory and the three
// values are computed twice, once for the maxima and once for the codes. The
// thread that computes a value is the one that copied it, so shared memory
// needs no barrier for them.
#include <algorithm>
#include <atomic>

#include "device_common.cuh"
#include "fp8_common.cuh"
#include "gate.cuh"
#include "internal.h"

namespace ap {
namespace {

struct GradParams {
    GatedGradArgs a;
    Gate gate;
    bool vec_dy, vec_g, vec_u, vec_dg, vec_du, vec_q, vec_qt, vec_ht;
    bool plain;                // all rows on the boundaries
    int64_t blocks, blocks_t;  // of a row, of a column
    int row_threads;           // values only: threads a row, a power of two
    int64_t row_ctas;          // values only: CTAs a row
};

// Two values that one instruction multiplies or adds.
struct Pair {
    uint64_t v;
    __device__ __forceinline__ Pair() {}
    __device__ __forceinline__ Pair(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b)); }
    __device__ __forceinline__ void get(float& a, float& b) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
};
__device__ __forceinline__ Pair operator*(Pair a, Pair b) {
    Pair r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ Pair operator+(Pair a, Pair b) {
    Pair r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
    Pair r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

// dg, du and h of two elements. With e = exp(-w(g)), s = 1 / (1 + e) (gate.cuh) and
// 1 - s = e s, without the cancellation (the limit keeps an infinite e out of a
// product with s = 0):
//     dg = dy s u (1 + g e s w'(g)),  du = dy s g,  h = g s u.
// Multiplications and additions take both elements at once (8192 x 16384, all codes:
// gelu 410 -> 376 us; silu, which has fewer, the same either way).
template <bool SILU>
__device__ __forceinline__ void gradient2(const Gate& p, const float (&dy)[8], const float (&g)[8], const float (&u)[8], int i, float (&dg)[8],
                                          float (&du)[8], float (&h)[8]) {
    const float low0 = max_nan(g[i], -128.0f), low1 = max_nan(g[i + 1], -128.0f);
    const Pair one(1.0f, 1.0f), low(low0, low1), near(min_nan(low0, 128.0f), min_nan(low1, 128.0f)), square = near * near;
    const Pair power = near * (SILU ? Pair(-p.e1, -p.e1) : fma2(square, Pair(-p.e3, -p.e3), Pair(-p.e1, -p.e1)));
    float e0, e1, s0, s1;
    power.get(e0, e1);
    e0 = exp2_approx(e0), e1 = exp2_approx(e1);
    (Pair(e0, e1) + one).get(s0, s1);
    const Pair s(rcp_approx(s0), rcp_approx(s1)), both(u[i], u[i + 1]);
    const Pair t = near * (Pair(fminf(e0, 1e38f), fminf(e1, 1e38f)) * s);
    const Pair rise = SILU ? t + one : fma2(t, fma2(square, Pair(p.c9, p.c9), Pair(p.c1, p.c1)), one);
    const Pair a = Pair(dy[i], dy[i + 1]) * s;
    (a * both * rise).get(dg[i], dg[i + 1]);
    (a * low).get(du[i], du[i + 1]);
    (low * s * both).get(h[i], h[i + 1]);
}

// Eight elements, the first n of them in memory, at an address of whole elements:
// 16-bit ones by 4-byte words, with the first and last alone where they lie in
// halves of words (5 loads or stores, not 8).
template <typename T>
__device__ __forceinline__ Raw8<T> load8_anywhere(const T* p, int64_t n) {
    if constexpr (sizeof(T) == 2) {
        if (n >= 8) {
            Raw8<T> r;
            const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
            if ((reinterpret_cast<uintptr_t>(p) & 2) == 0) {
                const uint32_t* w = reinterpret_cast<const uint32_t*>(p);
                r.w = make_uint4(w[0], w[1], w[2], w[3]);
            } else {
                const uint32_t* w = reinterpret_cast<const uint32_t*>(h + 1);
                const uint32_t first = h[0], a = w[0], b = w[1], c = w[2], last = h[7];
                r.w = make_uint4(first | a << 16, __funnelshift_r(a, b, 16), __funnelshift_r(b, c, 16), c >> 16 | last << 16);
            }
            return r;
        }
    }
    return load8(p, false, n);
}
template <typename T>
__device__ __forceinline__ void store8_anywhere(T* p, int64_t n, const float (&v)[8]) {
    if constexpr (sizeof(T) == 2) {
        if (n >= 8) {
            uint16_t* h = reinterpret_cast<uint16_t*>(p);
            if ((reinterpret_cast<uintptr_t>(p) & 2) == 0) {
#pragma unroll
                for (int i = 0; i < 4; ++i) reinterpret_cast<uint32_t*>(p)[i] = pack2<T>(v[2 * i], v[2 * i + 1]);
            } else {
                const uint32_t ends = pack2<T>(v[0], v[7]);
                h[0] = static_cast<uint16_t>(ends);
#pragma unroll
                for (int i = 0; i < 3; ++i) reinterpret_cast<uint32_t*>(h + 1)[i] = pack2<T>(v[2 * i + 1], v[2 * i + 2]);
                h[7] = static_cast<uint16_t>(ends >> 16);
            }
            return;
        }
    }
    store8(p, false, n, v);
}
template <typename T>
__device__ __forceinline__ Raw8<T> load8_maybe(const T* p, bool vec, int64_t n) {
    return vec ? load8(p, true, n) : load8_anywhere(p, n);
}
template <typename T>
__device__ __forceinline__ void store8_maybe(T* p, bool vec, int64_t n, const float (&v)[8]) {
    if (vec)
        store8(p, true, n, v);
    else
        store8_anywhere(p, n, v);
}

// dg and du in the inputs' type alone: eight neighbours a thread.
template <typename T, bool SILU>
__global__ void __launch_bounds__(256) gated_values_kernel(const __grid_constant__ GradParams P) {
    ptx::let_next_grid_start();
    ptx::wait_previous_grid();
    const GatedGradArgs& a = P.a;
    const int rows = 256 / P.row_threads;
    const int64_t row = static_cast<int64_t>(blockIdx.x) / P.row_ctas * rows + threadIdx.x / P.row_threads;
    const int64_t col = 8 * (static_cast<int64_t>(blockIdx.x) % P.row_ctas * 256 + threadIdx.x % P.row_threads);
    const int64_t n = a.cols - col;
    if (row >= a.rows || n <= 0) return;
    float dy[8], g[8], u[8];
    const Raw8<T> r0 = load8_maybe(static_cast<const T*>(a.dy) + row * a.lddy + col, P.vec_dy, n);
    const Raw8<T> r1 = load8_maybe(static_cast<const T*>(a.g) + row * a.ldg + col, P.vec_g, n);
    const Raw8<T> r2 = load8_maybe(static_cast<const T*>(a.u) + row * a.ldu + col, P.vec_u, n);
    r0.unpack(dy);
    r1.unpack(g);
    r2.unpack(u);
    float h[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2) gradient2<SILU>(P.gate, dy, g, u, i, g, u, h);
    if (a.dgate != nullptr) store8_maybe(static_cast<T*>(a.dgate) + row * a.lddg + col, P.vec_dg, n, g);
    if (a.dup != nullptr) store8_maybe(static_cast<T*>(a.dup) + row * a.lddu + col, P.vec_du, n, u);
}

// A thread's eight rows of an input in shared memory: unit p of thread t at
// [p][t], 16 bytes a unit (float: two).
template <typename T>
struct Kept {
    static constexpr int kUnits = sizeof(T) / 2;
    static constexpr uint32_t kBytes = 8 * 256 * 16 * kUnits;  // of an input's tile
    // An input's eight rows, n (or no) elements each: by asynchronous copies
    // where rows start on 16-byte boundaries, else all loads before the first store.
    static __device__ __forceinline__ void fetch(uint32_t at, const T* src, int64_t ld, const T* valid, bool vec, int rows, int64_t cols) {
        if (vec) {
#pragma unroll
            for (int p = 0; p < 8; ++p) {
                const int64_t n = p < rows ? cols : 0;
#pragma unroll
                for (int i = 0; i < kUnits; ++i) {
                    const int64_t left = (n - i * (8 / kUnits)) * static_cast<int64_t>(sizeof(T));
                    ptx::cp_async_cg16(at + ((p * kUnits + i) * 256 + threadIdx.x) * 16, left > 0 ? src + p * ld + i * (8 / kUnits) : valid,
                                       left >= 16 ? 16u : (left > 0 ? static_cast<uint32_t>(left) : 0u));
                }
            }
        } else {
            Raw8<T> r[8];
#pragma unroll
            for (int p = 0; p < 8; ++p) r[p] = load8_anywhere(src + p * ld, p < rows ? cols : 0);
#pragma unroll
            for (int p = 0; p < 8; ++p) {
                const uint4* w = reinterpret_cast<const uint4*>(&r[p]);
#pragma unroll
                for (int i = 0; i < kUnits; ++i)
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + ((p * kUnits + i) * 256 + threadIdx.x) * 16),
                                 "r"(w[i].x), "r"(w[i].y), "r"(w[i].z), "r"(w[i].w)
                                 : "memory");
            }
        }
    }
    static __device__ __forceinline__ void get(uint32_t at, int p, float (&v)[8]) {
        Raw8<T> r;
        uint4* w = reinterpret_cast<uint4*>(&r);
#pragma unroll
        for (int i = 0; i < kUnits; ++i)
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[i].x), "=r"(w[i].y), "=r"(w[i].z), "=r"(w[i].w)
                         : "r"(at + ((p * kUnits + i) * 256 + threadIdx.x) * 16)
                         : "memory");
        r.unpack(v);
    }
};

// The first n (may be negative) of eight codes, zeros after them: past a matrix's
// last column also in a block whose 1 / s is NaN.
__device__ __forceinline__ uint2 first_codes(uint2 w, int64_t n) {
    if (n >= 8) return w;
    const uint64_t keep = n > 0 ? ~uint64_t(0) >> (64 - 8 * n) : 0;
    return make_uint2(w.x & static_cast<uint32_t>(keep), w.y & static_cast<uint32_t>(keep >> 32));
}

constexpr int kTurned = kScaleBlock * 16 * 8;  // bytes of a tile's transposed codes

struct TileShared {
    float row_inv[kScaleBlock][2];     // 1 / s of a row's blocks of dg and du
    float col_max[3][4][kScaleBlock];  // [dg, du, h][warp, two in turn]; then the columns' 1 / s in [.][0]
};

// A 128 x 128 tile a CTA: thread t holds rows 8 (t / 16) .. + 7 of columns
// 8 (t % 16) .. + 7. WHOLE: every row and column exists, and every row starts on
// a 16-byte boundary (codes: 8). CODES: all codes are asked for and no values, as
// by a training step (8192 x 16384, at the time: 348 us, 379 with the questions left in).
template <typename T, bool SILU, bool WHOLE, bool CODES>
__device__ __forceinline__ void tile_grad(const GradParams& P, unsigned char* smem_raw, TileShared& sh) {
    using K = Kept<T>;
    auto& col_max = sh.col_max;
    const uint32_t at_dy = ptx::smem_addr(smem_raw), at_g = at_dy + K::kBytes, at_u = at_g + K::kBytes;
    const GatedGradArgs& a = P.a;
    const int lane = threadIdx.x & 31, chunk = threadIdx.x & 15, rows8 = threadIdx.x >> 4, warp = threadIdx.x >> 5;
    const int64_t tj = blockIdx.x % P.blocks, ti = blockIdx.x / P.blocks;
    const int64_t row0 = ti * kScaleBlock + 8 * rows8, col = tj * kScaleBlock + 8 * chunk;
    // rows of this thread that exist (may be negative), and columns
    const int rows = WHOLE ? 8 : static_cast<int>(a.rows - row0 < 8 ? a.rows - row0 : 8);
    const int64_t cols = WHOLE ? 8 : a.cols - col;
    const bool by_rows = CODES || a.q != nullptr, by_cols = CODES || a.qt != nullptr, h_cols = CODES || a.ht != nullptr;
    const int64_t half = P.blocks * kScaleBlock;  // du's first column beside dg
    {
        const T* dy = static_cast<const T*>(a.dy) + (row0 * a.lddy + col);
        const T* g = static_cast<const T*>(a.g) + (row0 * a.ldg + col);
        const T* u = static_cast<const T*>(a.u) + (row0 * a.ldu + col);
        K::fetch(at_dy, dy, a.lddy, static_cast<const T*>(a.dy), WHOLE || P.vec_dy, rows, cols);
        K::fetch(at_g, g, a.ldg, static_cast<const T*>(a.g), WHOLE || P.vec_g, rows, cols);
        K::fetch(at_u, u, a.ldu, static_cast<const T*>(a.u), WHOLE || P.vec_u, rows, cols);
        ptx::cp_async_commit();
        ptx::cp_async_wait_all();
    }

    // The loops over a thread's rows stay loops: unrolled, their instructions
    // outgrow the cache and two thirds of the time goes into fetching them.
    float max_g[8], max_u[8], max_h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) max_g[i] = max_u[i] = max_h[i] = 0.0f;
#pragma unroll 1
    for (int p = 0; p < 8; p += 2) {
        float peak[4];  // of dg in two rows, of du in two rows
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float dg[8], du[8], h[8];
            K::get(at_dy, p + r, dg);
            K::get(at_g, p + r, du);
            K::get(at_u, p + r, h);
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                gradient2<SILU>(P.gate, dg, du, h, i, dg, du, h);
#pragma unroll
                for (int k = i; k < i + 2; ++k) {
                    max_g[k] = max_nan(max_g[k], fabsf(dg[k]));
                    max_u[k] = max_nan(max_u[k], fabsf(du[k]));
                    max_h[k] = max_nan(max_h[k], fabsf(h[k]));
                }
            }
            if (!CODES && (WHOLE || (p + r < rows && cols > 0))) {
                if (a.dgate != nullptr) store8_maybe(static_cast<T*>(a.dgate) + (row0 + p + r) * a.lddg + col, WHOLE || P.vec_dg, cols, dg);
                if (a.dup != nullptr) store8_maybe(static_cast<T*>(a.dup) + (row0 + p + r) * a.lddu + col, WHOLE || P.vec_du, cols, du);
            }
            peak[r] = amax8(dg);
            peak[2 + r] = amax8(du);
        }
        if (by_rows) {
            // Four maxima over 16 lanes in five exchanges: the first two halve
            // what a lane carries, so that it ends with one and takes one scale.
            const bool up = (lane & 8) != 0, odd = (lane & 4) != 0;
            const float m0 = max_nan(up ? peak[2] : peak[0], __shfl_xor_sync(0xffffffffu, up ? peak[0] : peak[2], 8));
            const float m1 = max_nan(up ? peak[3] : peak[1], __shfl_xor_sync(0xffffffffu, up ? peak[1] : peak[3], 8));
            float m = max_nan(odd ? m1 : m0, __shfl_xor_sync(0xffffffffu, odd ? m0 : m1, 4));
            m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 2));
            m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 1));
            const Scale s = scale_of(m);
            const int r = p + (odd ? 1 : 0);
            if ((lane & 3) == 0) {
                sh.row_inv[8 * rows8 + r][up ? 1 : 0] = s.inv;
                if (r < rows) a.scales[(row0 + r) * 2 * P.blocks + (up ? P.blocks : 0) + tj] = s.s;
            }
        }
    }
    if (by_cols || h_cols) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            max_g[i] = max_nan(max_g[i], __shfl_xor_sync(0xffffffffu, max_g[i], 16));
            max_u[i] = max_nan(max_u[i], __shfl_xor_sync(0xffffffffu, max_u[i], 16));
            max_h[i] = max_nan(max_h[i], __shfl_xor_sync(0xffffffffu, max_h[i], 16));
        }
        for (int turn = 0; turn < 2; ++turn) {  // warps 4 to 7, then 0 to 3 beside them
            if ((lane & 16) == 0 && warp / 4 != turn) {
                float* m = &col_max[0][warp & 3][8 * chunk];
                constexpr int kNext = 4 * kScaleBlock;  // to the next of dg, du, h
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    m[i] = turn ? max_nan(m[i], max_g[i]) : max_g[i];
                    m[kNext + i] = turn ? max_nan(m[kNext + i], max_u[i]) : max_u[i];
                    m[2 * kNext + i] = turn ? max_nan(m[2 * kNext + i], max_h[i]) : max_h[i];
                }
            }
            __syncthreads();
        }
        for (int e = threadIdx.x; e < 3 * kScaleBlock; e += 256) {
            const int what = e / kScaleBlock, c = e % kScaleBlock;
            float m = col_max[what][0][c];
#pragma unroll
            for (int w = 1; w < 4; ++w) m = max_nan(m, col_max[what][w][c]);
            const Scale s = scale_of(m);
            const int64_t j = tj * kScaleBlock + c;
            if (what == 0 && by_cols) a.scales_t[j * P.blocks_t + ti] = s.s;
            if (what == 1 && by_cols && (WHOLE || j < a.cols)) a.scales_t[(half + j) * P.blocks_t + ti] = s.s;
            if (what == 2 && h_cols && (WHOLE || j < a.cols)) a.ht_scales[j * P.blocks_t + ti] = s.s;
            col_max[what][0][c] = s.inv;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            max_g[i] = col_max[0][0][8 * chunk + i];
            max_u[i] = col_max[1][0][8 * chunk + i];
            max_h[i] = col_max[2][0][8 * chunk + i];
        }
    } else {
        if (!by_rows) return;
        __syncwarp();  // row_inv is a warp's own
    }

    uint32_t lo[3][8], hi[3][8];  // codes of rows 0..3 and 4..7 of each of the thread's columns, shifted in two rows at a time
#pragma unroll
    for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) lo[k][i] = hi[k][i] = 0;
#pragma unroll 1
    for (int p = 0; p < 8; p += 2) {
        float dg[2][8], du[2][8], h[2][8];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            K::get(at_dy, p + r, dg[r]);
            K::get(at_g, p + r, du[r]);
            K::get(at_u, p + r, h[r]);
#pragma unroll
            for (int i = 0; i < 8; i += 2) gradient2<SILU>(P.gate, dg[r], du[r], h[r], i, dg[r], du[r], h[r]);
            if (by_rows && p + r < rows) {
                const float2 inv = *reinterpret_cast<const float2*>(sh.row_inv[8 * rows8 + p + r]);
                uint8_t* q = a.q + (row0 + p + r) * a.ldq + col;
                uint2 w = codes8(dg[r], inv.x);
                if (!WHOLE) w = first_codes(w, cols);
                store_codes(q, WHOLE || P.vec_q, 8, w);  // up to du's first column: zeros past dg's last
                if (cols > 0) store_codes(q + half, WHOLE || P.vec_q, cols, codes8(du[r], inv.y));
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t w[3] = {e4m3x2(dg[0][i] * max_g[i], dg[1][i] * max_g[i]), e4m3x2(du[0][i] * max_u[i], du[1][i] * max_u[i]),
                                   e4m3x2(h[0][i] * max_h[i], h[1][i] * max_h[i])};
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                lo[k][i] = __funnelshift_r(lo[k][i], hi[k][i], 16);
                hi[k][i] = __byte_perm(hi[k][i], w[k], 0x5432);
            }
        }
    }
    if (!by_cols && !h_cols) return;
    __syncthreads();  // the inputs have been read: their place takes the codes on their way
    uint2(*turned)[16] = reinterpret_cast<uint2(*)[16]>(smem_raw);
    // unit rows8 of a column goes to place rows8 ^ chunk: the 16 lanes that
    // write one instruction's columns then cover all banks
#pragma unroll
    for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) turned[k * kScaleBlock + 8 * chunk + i][rows8 ^ chunk] = make_uint2(lo[k][i], hi[k][i]);
    __syncthreads();
    // 16 lanes write a column's 128 codes
    const int64_t i0 = ti * kScaleBlock + 8 * chunk, j0 = tj * kScaleBlock + rows8, n = WHOLE ? 8 : a.rows - i0;
    if (n <= 0) return;
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const int c = 16 * p + rows8;
        const int64_t j = j0 + 16 * p;
        const bool in = WHOLE || j < a.cols;
        if (by_cols) {
            uint8_t* qt = a.qt + j * a.ldqt + i0;
            store_codes(qt, WHOLE || P.vec_qt, n, turned[c][chunk ^ (c >> 3)]);
            if (in) store_codes(qt + half * a.ldqt, WHOLE || P.vec_qt, n, turned[kScaleBlock + c][chunk ^ (c >> 3)]);
        }
        if (h_cols && in) store_codes(a.ht + j * a.ldht + i0, WHOLE || P.vec_ht, n, turned[2 * kScaleBlock + c][chunk ^ (c >> 3)]);
    }
}

template <typename T, bool SILU>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 2 : 1) gated_grad_kernel(const __grid_constant__ GradParams P) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    __shared__ __align__(16) TileShared sh;
    ptx::let_next_grid_start();
    ptx::wait_previous_grid();
    const int64_t tj = blockIdx.x % P.blocks, ti = blockIdx.x / P.blocks;
    const GatedGradArgs& a = P.a;
    if (!P.plain || (ti + 1) * kScaleBlock > a.rows || (tj + 1) * kScaleBlock > a.cols)
        tile_grad<T, SILU, false, false>(P, smem_raw, sh);
    else if (a.q != nullptr && a.qt != nullptr && a.ht != nullptr && a.dgate == nullptr && a.dup == nullptr)
        tile_grad<T, SILU, true, true>(P, smem_raw, sh);
    else
        tile_grad<T, SILU, true, false>(P, smem_raw, sh);
}

template <typename T, bool SILU>
ap_status launch_t(const DeviceInfo& di, const GatedGradArgs& a, cudaStream_t stream) {
    GradParams P;
    P.a = a;
    P.gate = gate_of(a.act);
    P.vec_dy = rows_aligned(a.dy, a.lddy, sizeof(T), 16);
    P.vec_g = rows_aligned(a.g, a.ldg, sizeof(T), 16);
    P.vec_u = rows_aligned(a.u, a.ldu, sizeof(T), 16);
    P.vec_dg = rows_aligned(a.dgate, a.lddg, sizeof(T), 16);
    P.vec_du = rows_aligned(a.dup, a.lddu, sizeof(T), 16);
    P.vec_q = rows_aligned(a.q, a.ldq, 1, 8);
    P.vec_qt = rows_aligned(a.qt, a.ldqt, 1, 8);
    P.vec_ht = rows_aligned(a.ht, a.ldht, 1, 8);
    P.plain = P.vec_dy && P.vec_g && P.vec_u && (a.dgate == nullptr || P.vec_dg) && (a.dup == nullptr || P.vec_du) &&
              (a.q == nullptr || P.vec_q) && (a.qt == nullptr || P.vec_qt) && (a.ht == nullptr || P.vec_ht);
    P.blocks = (a.cols + kScaleBlock - 1) / kScaleBlock;
    P.blocks_t = (a.rows + kScaleBlock - 1) / kScaleBlock;
    if (a.q == nullptr && a.qt == nullptr && a.ht == nullptr) {
        P.row_threads = 1;
        while (P.row_threads < 256 && 8 * static_cast<int64_t>(P.row_threads) < a.cols) P.row_threads *= 2;
        P.row_ctas = (a.cols + 8 * 256 - 1) / (8 * 256);
        const int64_t per_cta = 256 / P.row_threads;
        const int64_t grid = (a.rows + per_cta - 1) / per_cta * P.row_ctas;
        if (grid >= (int64_t(1) << 31)) return AP_ERR_SHAPE;
        record_launch(PATH_GATED_GRAD, grid, 8, 0, 0, 0);
        return launch_early(gated_values_kernel<T, SILU>, grid, 256, stream, P);
    }
    const int64_t grid = P.blocks * P.blocks_t;
    if (grid >= (int64_t(1) << 31)) return AP_ERR_SHAPE;
    constexpr size_t kSmem = 3 * Kept<T>::kBytes;
    static_assert(kSmem >= 3 * kTurned, "the codes fit in the inputs' place");
    static_assert((sizeof(T) == 2 ? 2 : 1) * (kSmem + sizeof(TileShared) + 1024) <= kSmemPerSM, "shared memory of an SM");
    auto kernel = gated_grad_kernel<T, SILU>;
    static std::atomic<int> configured[64];  // attribute set on this device (setting twice is harmless)
    if (di.device < 0 || di.device >= 64) return AP_ERR_CUDA;
    if (!configured[di.device].load()) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem)) != cudaSuccess)
            return AP_ERR_CUDA;
        configured[di.device] = 1;
    }
    record_launch(PATH_GATED_GRAD, grid, 64, static_cast<int64_t>(kSmem), 0, 1);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr = early_start();
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, P) == cudaSuccess ? AP_OK : AP_ERR_CUDA;
}

}  // namespace

ap_status launch_gated_grad(const DeviceInfo& di, const GatedGradArgs& a, cudaStream_t stream) {
    const bool silu = a.act == AP_ACT_SILU;
    switch (a.type) {
        case AP_BF16: return silu ? launch_t<__nv_bfloat16, true>(di, a, stream) : launch_t<__nv_bfloat16, false>(di, a, stream);
        case AP_F16: return silu ? launch_t<__half, true>(di, a, stream) : launch_t<__half, false>(di, a, stream);
        default: return silu ? launch_t<float, true>(di, a, stream) : launch_t<float, false>(di, a, stream);
    }
}

}  // namespace ap
