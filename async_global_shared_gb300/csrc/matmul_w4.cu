// c = x W^T for few rows of x and a weight of 4-bit codes with a scale (and
// zero point) for each group of 32, 64 or 128 columns; and the gated form
// y = act(x Wg^T) * (x Wu^T), which takes both weights' products side by side.
//     c[i, j] = sum over groups of scale[j, group] * sum x[i, k] (code[j, k] - zero[j, group])
//
// What bounds it: the codes, half a byte a weight, read once. Everything else
// is there to keep enough of them under way and to spend few instructions on a
// weight.
//  - A warp takes 16 rows of the weight (a row tile; of two weights, or two
//    tiles) and every so manieth block of 256 or 128 columns, and streams those codes
//    through a ring of shared memory of its own, by 16-byte asynchronous copies
//    (128 or 64 bytes a row and block): no barrier is needed before the end.
//  - A word of a row holds eight columns; shifts, masks and a subtraction bring columns i
//    and i + 4 at once into a pair of 16-bit numbers code - zero (see Codes).
//  - The products run on the warp's matrix instruction m16n8k16 with the
//    weight's rows on its 16 rows and the rows of x on its 8 columns, so up to
//    8 rows of x cost what one costs. (The tensor memory's instructions take the
//    weight from tensor memory or shared memory, so the widened codes, four times the
//    bytes that arrive, would be written there first. For 8 rows of x that is more
//    work; for many, whose weight would be widened once, it would be less: not built.)
//    Columns may be taken in any order as long as both operands agree: x is staged
//    with every eight of its values in the order 0 4 1 5 2 6 3 7, which is how the
//    codes come out of a word.
//  - A group's products are summed by themselves and then scaled, in 32 bits.
//  - x is staged for a stretch of blocks at a time.
//  - The warps of a CTA share the staged x. Where that leaves few CTAs a cluster
//    shares k, and adds its shares through distributed shared memory in rank
//    order.
// It measured (the codes at the rate of a copy would take 5.1, 10.2 and 11 us): one row
// times 8192 x 8192 13.0 us, gated times 16384 x 4096 20.9, 32 rows times 8192 x 16384
// 59.7. What bounds it then are instructions, 385 for 256 columns of 16 rows with all that
// is around them (the first case), about 176 of them the widening (11 for a word's eight
// codes; 9 in fp16); with two CTAs of eight warps an SM the issue slots are 43 % busy, and
// waits on the ring, the matrix instructions and one another take the rest. More than 32
// rows: 8192 x 8192 times 128 rows 89 us, 2048 rows 1220, 193 and 225 TFLOP/s.
#include <algorithm>
#include <atomic>

#include "device_common.cuh"
#include "fp8_common.cuh"
#include "gate.cuh"
#include "internal.h"
#include "tcgen05.cuh"

namespace ap {
namespace {

constexpr int kWarps = 8;
constexpr int kRows = 16;  // of a row tile
constexpr int kMaxSplit = 8;

struct W4Params {
    const void* x;
    const uint8_t* codes[2];
    const void* scales[2];
    const uint8_t* zeros[2];
    void* c;
    int64_t ldx, ldw[2], ldc;
    int64_t m, n, k;
    int64_t groups;   // of a row
    int group_steps;  // 32-column steps of a group: 1, 2 or 4
    int tiles_log;    // log2 of the warps of a CTA with rows of their own, 0 to 3; the others share their columns
    int split;        // CTAs of a cluster that share k
    int stretch;      // blocks staged at a time
    bool vec_x;
    ap_dtype c_type;
    Gate gate;
};

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t how) { return __byte_perm(a, b, how); }

__device__ __forceinline__ float lds4(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ void sts4(uint32_t addr, float v) { asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory"); }

// (w & mask) | power
__device__ __forceinline__ uint32_t code_of(uint32_t w, uint32_t mask, uint32_t power) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "r"(mask), "r"(power));
    return r;
}

// A word's eight codes as 16-bit numbers code - zero, pairs of columns (0, 4), (1, 5),
// (2, 6), (3, 7), exact for every code and zero point: a mask puts a code on the lowest
// mantissa bits of a power of two (128 in bf16, 1024 in fp16), and the power and the
// zero point are taken off in one operation for two codes. (A form whose products are of
// x and 16 + code and which takes 16 + zero times the group's sum of x off the group's
// sum saves that operation, but its sums lose what the correction cancels: a large x
// where code = zero, all x of one sign, an infinity. It measured 12.6, 20.4 and 63.8 us
// for the three above: it has to take and keep the sums of x. In 32 bits c is now off by
// 3e-8 to 7e-8 of its root mean square, 8 x 2048 x 4096 with x around 0, 1 or 16 standard
// deviations off it; the plain products in 32 bits by 3e-8 to 4e-7.)
template <typename T>
struct Codes;
template <>
struct Codes<__nv_bfloat16> {
    // bf16 has every whole number up to 256: of a zero point above 128 the first 128
    // are taken off with the power, the rest by a second subtraction (32 x 8192 x 16384,
    // zero points of 200: 62.0 us, 59.8 of 8).
    struct Zero {
        uint32_t first, rest;  // 128 + the first, twice; the rest
    };
    static constexpr uint32_t kPower = 0x43004300u;  // 128
    static __device__ __forceinline__ bool large(uint32_t zero) { return zero > 128; }
    static __device__ __forceinline__ uint32_t sub(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ Zero zero_of(uint32_t zero) {
        const uint32_t low = min(zero, 128u);
        return Zero{(0x4300u + low) * 0x10001u, zero - low};
    }
    static __device__ __forceinline__ void widen(uint32_t w, uint32_t mask, uint32_t power, const Zero& z, bool large, uint32_t (&p)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = sub(code_of(w >> (4 * i), mask, power), z.first);
        if (large) {
            const uint32_t rest = sub((0x4300u + z.rest) * 0x10001u, kPower);
#pragma unroll
            for (int i = 0; i < 4; ++i) p[i] = sub(p[i], rest);
        }
    }
    // d += (first: =) a * b
    static __device__ __forceinline__ void mma(float (&d)[4], bool first, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                               uint32_t b1) {
        if (first)
            asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
                : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
        else
            asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    }
};
template <>
struct Codes<__half> {
    // Codes on bits 0 to 3 as 1024 + code, those on bits 4 to 7 as 1024 + 16 code, a
    // sixteenth of which less 64 + zero is one fused operation; every number is whole
    // and below 2048.
    struct Zero {
        uint32_t first, second;  // 1024 + zero, -(64 + zero)
    };
    static constexpr uint32_t kPower = 0x64006400u;  // 1024
    static __device__ __forceinline__ bool large(uint32_t) { return false; }
    static __device__ __forceinline__ uint32_t sub(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ Zero zero_of(uint32_t zero) {
        const uint32_t first = (0x6400u + zero) * 0x10001u;
        return Zero{first, sub(0x63806380u, first)};  // 960 - (1024 + zero)
    }
    static __device__ __forceinline__ void widen(uint32_t w, uint32_t mask, uint32_t power, const Zero& z, bool, uint32_t (&p)[4]) {
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            const uint32_t v = w >> (4 * i);
            p[i] = sub(code_of(v, mask, power), z.first);
            asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(p[i + 1]) : "r"(code_of(v, mask << 4, power)), "r"(0x2C002C00u), "r"(z.second));
        }
    }
    // d += (first: =) a * b
    static __device__ __forceinline__ void mma(float (&d)[4], bool first, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                               uint32_t b1) {
        if (first)
            asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
                : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
        else
            asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    }
};

// Weights side by side, 8-row tiles of x, and what they take of shared memory.
template <int NT, bool GATED, int STEPS>
struct Form {
    // A warp's strands of 16 rows, which share what it loads of x: the same rows
    // of two weights (gated), or for more than 8 rows of x two row tiles of one
    // (32 x 8192 x 16384: 60 us, 72 with one at the time; the other way 1 x 8192 x 8192 12.6, 13.4
    // with two, whose ring is shorter).
    static constexpr int kStrands = GATED || NT > 1 ? 2 : 1;
    static constexpr int kOutputs = GATED ? 2 : 1;                        // sums a result takes
    static constexpr int kWarpRows = kRows * kStrands / kOutputs;         // weight rows of a warp
    // Columns of a step of the ring: 256 (128 bytes a row) have half as many
    // instructions around them as 128; but with more rows of x the staged x
    // takes the room.
    static constexpr int kBlock = NT == 1 ? 256 : 128;
    static constexpr int kSteps = kBlock / 32;         // of 32 columns: one word of a row a lane
    static constexpr int kPitch = kBlock / 2 + 16;     // of a row in the ring: eight rows' words on different banks
    static constexpr int kTileBytes = kRows * kPitch;
    static constexpr int kUnits = kBlock / 32;         // 16-byte units of a row, and lanes that copy it
    static constexpr int kTurns = kRows * kUnits / 32; // copies a lane and weight
    static constexpr int kCtas = NT == 4 || (GATED && STEPS == 1) ? 1 : 2;  // an SM: what their registers allow
    static constexpr int kStages = NT == 1 && kCtas == 2 && kStrands == 2 ? 2 : 4;
    static constexpr int64_t kSmemMost = kCtas == 1 ? kSmemOptinGB300 : kSmemPerSM / 2 - 1024;
    static constexpr int kRingBytes = kWarps * kStages * kStrands * kTileBytes;
    static constexpr int kXRows = 8 * NT;
    // shares of a CTA's sums: [part][output][x row][weight row]
    static constexpr int kShareBytes = kWarps * kStrands * kRows * kXRows * 4;
};

template <typename T, int NT, bool GATED, int STEPS>
__global__ void __launch_bounds__(32 * kWarps, (Form<NT, GATED, STEPS>::kCtas)) matmul_w4_kernel(const __grid_constant__ W4Params P) {
    using F = Form<NT, GATED, STEPS>;
    using H = Codes<T>;
    constexpr int kW = F::kStrands, kBlock = F::kBlock, kSteps = F::kSteps, kPitch = F::kPitch, kTileBytes = F::kTileBytes;
    constexpr int kGroups = kSteps / STEPS;  // of a block; STEPS 32-column steps each
    extern __shared__ __align__(16) unsigned char smem_raw[];
    const uint32_t smem = ptx::smem_addr(smem_raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int tiles = 1 << P.tiles_log;
    const int tile = warp & (tiles - 1), part = warp >> P.tiles_log, parts = kWarps >> P.tiles_log;
    const uint32_t rank = P.split > 1 ? ptx::cluster_ctarank() : 0, split = static_cast<uint32_t>(P.split);
    const int64_t row0 = static_cast<int64_t>(blockIdx.x / split * tiles) * F::kWarpRows;  // the CTA's first weight row
    const int64_t m0 = static_cast<int64_t>(blockIdx.y) * F::kXRows;
    const int xrows = static_cast<int>(P.m - m0 < F::kXRows ? P.m - m0 : F::kXRows);
    const uint32_t nb = static_cast<uint32_t>((P.k + kBlock - 1) / kBlock);  // below 2^24
    int b0 = 0, b1 = static_cast<int>(nb);
    if (P.split > 1) {
        b0 = static_cast<int>(nb * rank / split);
        b1 = static_cast<int>(nb * (rank + 1) / split);
    }
    const uint32_t ring = smem + static_cast<uint32_t>(warp * F::kStages * kW * kTileBytes);
    const uint32_t xs = smem + F::kRingBytes;  // x, 16-byte units in the order above
    const int stretch = P.stretch;
    const uint32_t xpitch = static_cast<uint32_t>(stretch) * (2 * kBlock) + 64;
    const int srows = tiles * F::kWarpRows;  // weight rows of the CTA
    auto row_of = [&](int w, int r) { return row0 + tile * F::kWarpRows + (GATED ? 0 : w * kRows) + r; };  // of a strand

    ptx::let_next_grid_start();
    ptx::wait_previous_grid();

    // The ring's copies of a block: a few units of 16 bytes a lane and weight, 8
    // (or 4) lanes a row. Only a row's last block may be cut short.
    const int64_t row_bytes = (P.k + 1) / 2;
    const int whole = static_cast<int>(row_bytes / (kBlock / 2));  // blocks with all their bytes
    constexpr int kUnits = F::kUnits, kTurns = F::kTurns, kApart = 32 / kUnits;  // rows between a lane's copies
    const int my_row = lane / kUnits, my_unit = lane % kUnits;
    const uint8_t* from[kW][kTurns];
#pragma unroll
    for (int w = 0; w < kW; ++w)
#pragma unroll
        for (int h = 0; h < kTurns; ++h) {
            const int64_t j = row_of(w, kApart * h + my_row);
            from[w][h] = P.codes[GATED ? w : 0] + (j < P.n ? j : P.n - 1) * P.ldw[GATED ? w : 0] + 16 * my_unit;
        }
    const uint32_t to = ring + my_row * kPitch + 16 * my_unit;
    auto fetch = [&](int b, uint32_t slot) {  // slot: its offset in the ring
        const uint32_t at = static_cast<uint32_t>(b) * (kBlock / 2);  // below 2^30
        if (b < whole) {
#pragma unroll
            for (int w = 0; w < kW; ++w)
#pragma unroll
                for (int h = 0; h < kTurns; ++h) ptx::cp_async_cg16(to + slot + w * kTileBytes + kApart * h * kPitch, from[w][h] + at, 16);
        } else {
            const int left = static_cast<int>(row_bytes - at) - 16 * my_unit;  // below 128, may be negative
            const uint32_t n = left >= 16 ? 16 : (left > 0 ? left : 0);
#pragma unroll
            for (int w = 0; w < kW; ++w)
#pragma unroll
                for (int h = 0; h < kTurns; ++h)
                    ptx::cp_async_cg16(to + slot + w * kTileBytes + kApart * h * kPitch, n ? from[w][h] + at : P.codes[0], n);
        }
    };
    // Scales and zero points of rows g and g + 8.
    const T* scales_at[kW][2];
    const uint8_t* zeros_at[kW][2];
#pragma unroll
    for (int w = 0; w < kW; ++w)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t j = row_of(w, 8 * h + g), at = (j < P.n ? j : P.n - 1) * P.groups;
            scales_at[w][h] = static_cast<const T*>(P.scales[GATED ? w : 0]) + at;
            zeros_at[w][h] = P.zeros[GATED ? w : 0] + at;
        }
    // x of the blocks from s0 on, by copies that fill with zeros past k, or
    // where rows do not start on 16-byte boundaries by single elements.
    const T* x = static_cast<const T*>(P.x) + m0 * P.ldx;
    auto stage_x = [&](int s0, int units) {
        const int64_t col0 = static_cast<int64_t>(s0) * kBlock;
        // a warp a row (with one row: all warps), 32 units at a time
        const bool one = xrows == 1;
#pragma unroll 1
        for (int r = one ? 0 : warp; r < xrows; r += kWarps) {
            const T* const src = x + r * P.ldx + col0;
            const uint32_t dst = xs + r * xpitch;
#pragma unroll 1
            for (int c = one ? threadIdx.x : lane; c < units; c += one ? 32 * kWarps : 32) {
                const int64_t n = P.k - col0 - 8 * c;
                if (P.vec_x)
                    ptx::cp_async_cg16(dst + 16 * c, n > 0 ? src + 8 * c : x, n >= 8 ? 16u : (n > 0 ? 2u * static_cast<uint32_t>(n) : 0u));
                else
                    *reinterpret_cast<uint4*>(smem_raw + (dst - smem) + 16 * c) = load8(src + 8 * c, false, n).w;
            }
        }
    };
    constexpr uint32_t kSlot = kW * kTileBytes, kEnd = F::kStages * kSlot;
    if (b0 < b1) stage_x(b0, (min(b0 + stretch, b1) - b0) * (kBlock / 8));
    ptx::cp_async_commit();
    int next = b0 + part;  // the next block to fetch
    uint32_t put = 0, take = 0;
#pragma unroll
    for (int s = 0; s < F::kStages - 1; ++s) {
        if (next < b1) fetch(next, put);
        ptx::cp_async_commit();
        next += parts;
        put += kSlot;
    }

    float acc[kW][NT][4];
#pragma unroll
    for (int w = 0; w < kW; ++w)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[w][j][i] = 0.0f;

    uint32_t mask = 0x000F000Fu, power = H::kPower;  // in registers
    asm volatile("" : "+r"(mask), "+r"(power));
    // Where this lane reads, as pointers: their constant parts become offsets
    // of the loads. Of rows of x past the last one the last (the results are dropped).
    const unsigned char* const words_at = smem_raw + (ring - smem) + g * kPitch + 4 * t;
    const unsigned char* x_at[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) x_at[j] = smem_raw + (xs - smem) + min(8 * j + g, xrows - 1) * xpitch + 16 * t;

    // Those of a block's groups, fetched for the next block as soon as this
    // one's are used.
    const int groups = static_cast<int>(P.groups);
    T scale[kW][2][kGroups];
    uint32_t zero[kW][2][kGroups];
    auto fetch_scales = [&](int w, int b) {
        const int64_t first = static_cast<int64_t>(b) * kGroups;
        const int left = groups - b * kGroups;  // groups past the last: nothing times 0
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const T* s = scales_at[w][h] + first;
#pragma unroll
            for (int q = 0; q < kGroups; ++q)
                scale[w][h][q] = q == 0 || q < left ? s[q] : from_f32<T>(0.0f);
        }
        if (P.zeros[0] != nullptr) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint8_t* z = zeros_at[w][h] + first;
#pragma unroll
                for (int q = 0; q < kGroups; ++q)
                    if (q == 0 || q < left) zero[w][h][q] = z[q];
            }
        }
    };
#pragma unroll
    for (int w = 0; w < kW; ++w)
#pragma unroll
        for (int i = 0; i < 2 * kGroups; ++i) {
            scale[w][i / kGroups][i % kGroups] = from_f32<T>(0.0f);
            zero[w][i / kGroups][i % kGroups] = 8;
        }
    int b = b0 + part;
    if (b < b1) {
#pragma unroll
        for (int w = 0; w < kW; ++w) fetch_scales(w, b);
    }
    for (int s0 = b0; s0 < b1; s0 += stretch) {
        const int s1 = min(s0 + stretch, b1);
        if (s0 > b0) __syncthreads();
        // x as it stands, then each thread puts its own units in order
        const int units = (s1 - s0) * (kBlock / 8);  // of a row
        if (s0 > b0) {
            stage_x(s0, units);
            ptx::cp_async_commit();
            ptx::cp_async_wait_all();
        } else {
            ptx::cp_async_wait_group<F::kStages - 1>();  // all but the ring's
        }
        const bool one = xrows == 1;
#pragma unroll 1
        for (int r = one ? 0 : warp; r < xrows; r += kWarps) {
            uint4* const row = reinterpret_cast<uint4*>(smem_raw + (xs - smem) + r * xpitch);
#pragma unroll 1
            for (int c = one ? threadIdx.x : lane; c < units; c += one ? 32 * kWarps : 32) {
                const uint4 w = row[c];
                row[c] = make_uint4(prmt(w.x, w.z, 0x5410), prmt(w.x, w.z, 0x7632), prmt(w.y, w.w, 0x5410), prmt(w.y, w.w, 0x7632));
            }
        }
        __syncthreads();
        for (; b < s1; b += parts) {
            ptx::cp_async_wait_group<F::kStages - 2>();
            __syncwarp();
            if (next < b1) fetch(next, put);
            ptx::cp_async_commit();
            next += parts;
            put = put + kSlot == kEnd ? 0 : put + kSlot;
            const unsigned char* const words = words_at + take;
            take = take + kSlot == kEnd ? 0 : take + kSlot;
            const uint32_t local = static_cast<uint32_t>(b - s0);
            const unsigned char* xb[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j) xb[j] = x_at[j] + local * (2 * kBlock);
            bool large = false;  // a zero point of the warp's rows that takes the second subtraction
            if (P.zeros[0] != nullptr) {
#pragma unroll
                for (int w = 0; w < kW; ++w)
#pragma unroll
                    for (int i = 0; i < 2 * kGroups; ++i) large |= H::large(zero[w][i / kGroups][i % kGroups]);
                large = __any_sync(0xffffffffu, large);
            }
#pragma unroll
            for (int q = 0; q < kGroups; ++q) {
                float sum[kW][NT][4];
                typename H::Zero zeros[kW][2];
#pragma unroll
                for (int w = 0; w < kW; ++w)
#pragma unroll
                    for (int h = 0; h < 2; ++h) zeros[w][h] = H::zero_of(zero[w][h][q]);
#pragma unroll
                for (int i = 0; i < STEPS; ++i) {
                    const int step = q * STEPS + i;
                    uint4 xv[NT];
#pragma unroll
                    for (int j = 0; j < NT; ++j) xv[j] = *reinterpret_cast<const uint4*>(xb[j] + 64 * step);
#pragma unroll
                    for (int w = 0; w < kW; ++w) {
                        uint32_t lo[4], hi[4];
                        H::widen(*reinterpret_cast<const uint32_t*>(words + w * kTileBytes + 16 * step), mask, power, zeros[w][0], large, lo);
                        H::widen(*reinterpret_cast<const uint32_t*>(words + w * kTileBytes + 8 * kPitch + 16 * step), mask, power, zeros[w][1],
                                 large, hi);
#pragma unroll
                        for (int j = 0; j < NT; ++j) {
                            H::mma(sum[w][j], i == 0, lo[0], hi[0], lo[1], hi[1], xv[j].x, xv[j].y);
                            H::mma(sum[w][j], false, lo[2], hi[2], lo[3], hi[3], xv[j].z, xv[j].w);
                        }
                    }
                }
#pragma unroll
                for (int w = 0; w < kW; ++w) {
                    const float ls = to_f32(scale[w][0][q]), hs = to_f32(scale[w][1][q]);
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        acc[w][j][0] = fmaf(ls, sum[w][j][0], acc[w][j][0]);
                        acc[w][j][1] = fmaf(ls, sum[w][j][1], acc[w][j][1]);
                        acc[w][j][2] = fmaf(hs, sum[w][j][2], acc[w][j][2]);
                        acc[w][j][3] = fmaf(hs, sum[w][j][3], acc[w][j][3]);
                    }
                }
            }
            if (b + parts < b1) {
#pragma unroll
                for (int w = 0; w < kW; ++w) fetch_scales(w, b + parts);
            }
        }
    }
    ptx::cp_async_wait_all();
    __syncthreads();

    // Shares, in the place of ring and stages: [part][output][x row][weight row of the CTA].
    constexpr int kOut = F::kOutputs;
    const uint32_t part_bytes = static_cast<uint32_t>(kOut * F::kXRows * srows) * 4;
#pragma unroll
    for (int w = 0; w < kW; ++w)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int xr = 8 * j + 2 * t + (i & 1), wr = tile * F::kWarpRows + (GATED ? 0 : w * kRows) + g + 8 * (i >> 1);
                sts4(smem + part * part_bytes + 4u * static_cast<uint32_t>(((GATED ? w : 0) * F::kXRows + xr) * srows + wr), acc[w][j][i]);
            }
    __syncthreads();
    const int outputs = xrows * srows, srows_log = P.tiles_log + (F::kWarpRows == kRows ? 4 : 5);
    auto parts_sum = [&](int w, int e) {
        float v = 0.0f;
#pragma unroll 1
        for (int p = 0; p < parts; ++p)
            v += lds4(smem + p * part_bytes + 4u * static_cast<uint32_t>(w * F::kXRows * srows + e));
        return v;
    };
    if (P.split > 1) {  // the CTA's own parts into the first, then the ranks' shares
#pragma unroll 1
        for (int e = threadIdx.x; e < outputs; e += 32 * kWarps)
#pragma unroll
            for (int w = 0; w < kOut; ++w) sts4(smem + 4u * static_cast<uint32_t>(w * F::kXRows * srows + e), parts_sum(w, e));
        __syncwarp();
        ptx::cluster_sync();
    }
    int e = threadIdx.x, e1 = outputs;
    if (P.split > 1) {
        e += static_cast<int>(outputs * rank / split);
        e1 = static_cast<int>(outputs * (rank + 1) / split);
    }
#pragma unroll 1
    for (; e < e1; e += 32 * kWarps) {
        float v[kOut];
#pragma unroll
        for (int w = 0; w < kOut; ++w) {
            if (P.split == 1) {
                v[w] = parts_sum(w, e);
            } else {
                float u[kMaxSplit];
#pragma unroll
                for (int r = 0; r < kMaxSplit; ++r)
                    u[r] = r < P.split ? ptx::cluster_ld(ptx::mapa(smem + 4u * static_cast<uint32_t>(w * F::kXRows * srows + e), r)) : 0.0f;
                v[w] = u[0];
#pragma unroll
                for (int r = 1; r < kMaxSplit; ++r) v[w] += u[r];
            }
        }
        const float y = GATED ? gate_value(P.gate, v[0]) * v[kOut - 1] : v[0];
        const int64_t j = row0 + (e & (srows - 1)), at = (m0 + (e >> srows_log)) * P.ldc + j;
        if (j < P.n) {
            if (P.c_type == AP_F32)
                static_cast<float*>(P.c)[at] = y;
            else
                static_cast<T*>(P.c)[at] = from_f32<T>(y);
        }
    }
    if (P.split > 1) {
        __syncwarp();         // lanes' loops above differ in length
        ptx::cluster_sync();  // every share has been read
    }
}

// Stretch and shared memory. A stretch has at least one block.
template <int NT, bool GATED, int STEPS>
bool plan_smem(W4Params& P, int64_t xrows, int64_t* bytes) {
    using F = Form<NT, GATED, STEPS>;
    const int64_t per_block = xrows * 2 * F::kBlock;
    const int64_t fixed = F::kRingBytes + xrows * 64;
    const int64_t nb = (P.k + F::kBlock - 1) / F::kBlock, mine = std::max<int64_t>(1, (nb + P.split - 1) / P.split);
    const int64_t fits = std::max<int64_t>(1, (F::kSmemMost - fixed) / per_block);
    // stretches of about the same length
    const int64_t stretches = (mine + fits - 1) / fits;
    P.stretch = static_cast<int>((mine + stretches - 1) / stretches);
    *bytes = std::max<int64_t>(fixed + P.stretch * per_block, F::kShareBytes);
    return *bytes <= kSmemOptinGB300;
}

template <typename T, int NT, bool GATED, int STEPS>
ap_status launch_form(const DeviceInfo& di, W4Params P, cudaStream_t stream) {
    using F = Form<NT, GATED, STEPS>;
    const int64_t row_tiles = (P.n + F::kWarpRows - 1) / F::kWarpRows, nb = (P.k + F::kBlock - 1) / F::kBlock;
    const int64_t chunks = (P.m + F::kXRows - 1) / F::kXRows;  // of x rows
    const int64_t xrows = std::min<int64_t>(P.m, F::kXRows);
    // Warps with rows of their own: all eight, which share the staged x, unless k in
    // eight shares then leaves SMs without a CTA; and k in so many shares as keep
    // all CTAs resident, each with two steps of the ring at least. (At the time: 1 x 4096 x
    // 16384: one and all of k a CTA 15.6 us, eight and an eighth 12.8; 1 x 8192 x
    // 8192: two 13.3, eight and a quarter 12.8; 32 x 8192 x 16384: four and a half
    // 81, eight and a quarter 64; the other way 1 x 1024 x 4096: eight 4.5, two 3.9.)
    const int64_t resident = F::kCtas * di.sms;
    auto ctas_of = [&](int log) { return (row_tiles + (1 << log) - 1) >> log; };
    int log = 3;
    while (log > 0 && ctas_of(log) * chunks * kMaxSplit < di.sms) --log;
    P.tiles_log = log;
    const int64_t ctas = ctas_of(log);
    P.split = 1;
    while (P.split < kMaxSplit && ctas * chunks * P.split * 2 <= resident && nb >= 2 * P.split * (kWarps >> log)) P.split *= 2;
    int64_t smem = 0;
    if (!plan_smem<NT, GATED, STEPS>(P, xrows, &smem)) return AP_ERR_SMEM;
    const int64_t grid = ctas * P.split;
    if (grid >= (int64_t(1) << 31) || chunks > 65535) return AP_ERR_SHAPE;
    auto kernel = matmul_w4_kernel<T, NT, GATED, STEPS>;
    static std::atomic<int> configured[64];  // attribute set on this device (setting twice is harmless)
    if (di.device < 0 || di.device >= 64) return AP_ERR_CUDA;
    if (!configured[di.device].load()) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmemOptinGB300)) !=
            cudaSuccess)
            return AP_ERR_CUDA;
        configured[di.device] = 1;
    }
    record_launch(PATH_MATMUL_W4, grid, 1 << log, smem, F::kStages, (GATED ? 1 : 0) | NT << 1 | P.split << 4);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), static_cast<unsigned>(chunks));
    cfg.blockDim = dim3(32 * kWarps);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0] = early_start();
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(P.split);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = P.split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, P) == cudaSuccess ? AP_OK : AP_ERR_CUDA;
}

template <typename T, int NT, bool GATED>
ap_status launch_group(const DeviceInfo& di, const W4Params& P, cudaStream_t stream) {
    switch (P.group_steps) {
        case 1: return launch_form<T, NT, GATED, 1>(di, P, stream);
        case 2: return launch_form<T, NT, GATED, 2>(di, P, stream);
        default: return launch_form<T, NT, GATED, 4>(di, P, stream);
    }
}

template <typename T, bool GATED>
ap_status launch_t(const DeviceInfo& di, const W4Params& P, cudaStream_t stream) {
    if (P.m <= 8) return launch_group<T, 1, GATED>(di, P, stream);
    if (P.m <= 16) return launch_group<T, 2, GATED>(di, P, stream);
    return launch_group<T, 4, GATED>(di, P, stream);
}

}  // namespace

ap_status launch_matmul_w4(const DeviceInfo& di, const MatmulW4Args& a, cudaStream_t stream) {
    W4Params P{};
    P.x = a.x;
    P.ldx = a.ldx;
    for (int w = 0; w < 2; ++w) {
        P.codes[w] = a.codes[w];
        P.scales[w] = a.scales[w];
        P.zeros[w] = a.zeros[w];
        P.ldw[w] = a.ldw[w];
    }
    P.c = a.c;
    P.ldc = a.ldc;
    P.m = a.m, P.n = a.n, P.k = a.k;
    P.groups = (a.k + a.group - 1) / a.group;
    P.group_steps = a.group / 32;
    P.vec_x = rows_aligned(a.x, a.ldx, 2, 16);
    P.c_type = a.c_type;
    P.gate = gate_of(a.act);
    if (a.type == AP_BF16)
        return a.gated ? launch_t<__nv_bfloat16, true>(di, P, stream) : launch_t<__nv_bfloat16, false>(di, P, stream);
    return a.gated ? launch_t<__half, true>(di, P, stream) : launch_t<__half, false>(di, P, stream);
}

}  // namespace ap
