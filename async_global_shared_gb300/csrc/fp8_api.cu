// C-ABI entry points of the 8-bit block-scaled operators: every check of the
// arguments is made here, before any CUDA call.
#include "internal.h"

using namespace ap;

namespace {

constexpr int64_t kMaxElems = int64_t(1) << 40;  // keeps every byte offset far from overflow
constexpr int64_t kMaxDim = (int64_t(1) << 31) - 512;  // coordinates of a tile stay in 31 bits

bool valid_type(ap_dtype t) { return t == AP_F32 || t == AP_BF16 || t == AP_F16; }
int64_t size_of(ap_dtype t) { return t == AP_F32 ? 4 : 2; }

// A rows x cols matrix of `size`-byte elements.
struct Matrix {
    const void* p;
    int64_t rows, cols, ld, size;
    uintptr_t at() const { return reinterpret_cast<uintptr_t>(p); }
    int64_t span() const { return ((rows - 1) * ld + cols) * size; }
};

bool valid_ld(int64_t rows, int64_t cols, int64_t ld) { return ld >= cols && ld <= kMaxElems / (rows > 0 ? rows : 1); }

bool aligned(const Matrix& a) { return a.at() % static_cast<uintptr_t>(a.size) == 0; }

// Whether two matrices share a byte. Rows of the same pitch that interleave
// without touching (column slices of one wider matrix) do not.
bool overlap(const Matrix& a, const Matrix& b) {
    if (a.p == nullptr || b.p == nullptr) return false;
    if (a.at() >= b.at() + static_cast<uintptr_t>(b.span()) || b.at() >= a.at() + static_cast<uintptr_t>(a.span()))
        return false;
    const int64_t pitch = a.ld * a.size;
    if (pitch != b.ld * b.size || a.rows == 1 || b.rows == 1) return true;
    const int64_t wa = a.cols * a.size, wb = b.cols * b.size;
    // offset of b's rows from a's within the pitch
    const int64_t d = a.at() <= b.at() ? static_cast<int64_t>((b.at() - a.at()) % static_cast<uintptr_t>(pitch))
                                       : (pitch - static_cast<int64_t>((a.at() - b.at()) % static_cast<uintptr_t>(pitch))) % pitch;
    return d < wa || d + wb > pitch;
}

bool same_place(const Matrix& a, const Matrix& b) { return a.p == b.p && a.ld == b.ld && a.size == b.size; }

int64_t blocks(int64_t n) { return (n + 127) / 128; }

Matrix floats(const void* p, int64_t rows, int64_t cols) { return Matrix{p, rows, cols, cols, 4}; }

}  // namespace

extern "C" {

ap_status ap_rms_norm(const void* x, int64_t ldx, ap_dtype type, const void* residual, void* residual_out, int64_t ldr,
                      ap_dtype residual_type, const void* weight, ap_dtype weight_type, float eps, int64_t rows,
                      int64_t cols, void* y, int64_t ldy, uint8_t* q, int64_t ldq, float* q_scales, float* rstd,
                      cudaStream_t stream) {
    if (!valid_type(type) || !valid_type(weight_type) || (weight_type != type && weight_type != AP_F32)) return AP_ERR_ARG;
    if (residual != nullptr && (!valid_type(residual_type) || (residual_type != type && residual_type != AP_F32)))
        return AP_ERR_ARG;
    if (!(eps >= 0.0f)) return AP_ERR_ARG;
    if (rows < 0 || cols < 0) return AP_ERR_SHAPE;
    if (rows == 0 || cols == 0) return AP_OK;
    if (cols > kMaxElems / rows || !valid_ld(rows, cols, ldx)) return AP_ERR_SHAPE;
    if (x == nullptr || weight == nullptr || (y == nullptr && q == nullptr)) return AP_ERR_NULL;
    if ((residual == nullptr) != (residual_out == nullptr) || (q == nullptr) != (q_scales == nullptr)) return AP_ERR_NULL;
    if ((residual != nullptr && !valid_ld(rows, cols, ldr)) || (y != nullptr && !valid_ld(rows, cols, ldy)) ||
        (q != nullptr && !valid_ld(rows, cols, ldq)))
        return AP_ERR_SHAPE;
    const int64_t rs = residual != nullptr ? size_of(residual_type) : 4;
    const Matrix in[] = {{x, rows, cols, ldx, size_of(type)},
                         {residual, rows, cols, ldr, rs},
                         {weight, 1, cols, cols, size_of(weight_type)}};
    const Matrix out[] = {{residual_out, rows, cols, ldr, rs},
                          {y, rows, cols, ldy, size_of(type)},
                          {q, rows, cols, ldq, 1},
                          floats(q_scales, rows, blocks(cols)),
                          floats(rstd, rows, 1)};
    for (const Matrix& i : in)
        if (i.p != nullptr && !aligned(i)) return AP_ERR_ALIGN;
    for (const Matrix& o : out)
        if (o.p != nullptr && !aligned(o)) return AP_ERR_ALIGN;
    for (int o = 0; o < 5; ++o) {
        for (int i = 0; i < 3; ++i) {
            const bool in_place = ((o == 0 && i == 1) || (o == 1 && i == 0)) && same_place(out[o], in[i]);
            if (!in_place && overlap(out[o], in[i])) return AP_ERR_ALIAS;
        }
        for (int p = 0; p < o; ++p)
            if (overlap(out[o], out[p])) return AP_ERR_ALIAS;
    }
    DeviceInfo di;
    const ap_status st = current_device(&di);
    if (st != AP_OK) return st;
    NormArgs a{x, residual, residual_out, weight, y, q, q_scales, rstd, rows, cols, ldx, ldr, ldy, ldq, type, residual_type,
               weight_type, eps};
    return launch_rms_norm(di, options(), a, stream);
}

int64_t ap_rms_norm_backward_workspace(int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 0 || (rows > 0 && cols > kMaxElems / rows)) return -1;
    return norm_grad_partials(rows, cols) * cols * 4;
}

ap_status ap_rms_norm_backward(const void* dy, int64_t lddy, ap_dtype type, const void* h, int64_t ldh,
                               ap_dtype residual_type, const void* weight, ap_dtype weight_type, const float* rstd,
                               const void* dresidual, int64_t lddr, int64_t rows, int64_t cols, void* dx, int64_t lddx,
                               float* dweight, void* workspace, cudaStream_t stream) {
    if (!valid_type(type) || !valid_type(weight_type) || (weight_type != type && weight_type != AP_F32)) return AP_ERR_ARG;
    if (!valid_type(residual_type) || (residual_type != type && residual_type != AP_F32)) return AP_ERR_ARG;
    if (rows < 0 || cols < 0) return AP_ERR_SHAPE;
    if (cols == 0 || (rows == 0 && dweight == nullptr)) return AP_OK;
    if (cols > kMaxElems / (rows > 0 ? rows : 1)) return AP_ERR_SHAPE;
    if (rows > 0) {
        if (!valid_ld(rows, cols, lddy) || !valid_ld(rows, cols, ldh) || !valid_ld(rows, cols, lddx)) return AP_ERR_SHAPE;
        if (dy == nullptr || h == nullptr || weight == nullptr || rstd == nullptr || dx == nullptr) return AP_ERR_NULL;
        if (dresidual != nullptr && !valid_ld(rows, cols, lddr)) return AP_ERR_SHAPE;
        if (dweight != nullptr && workspace == nullptr) return AP_ERR_NULL;
    } else {
        dy = h = weight = dresidual = nullptr;
        rstd = nullptr;
        dx = nullptr;
        workspace = nullptr;
    }
    const int64_t rs = size_of(residual_type);
    const int64_t partials = norm_grad_partials(rows, cols);
    const Matrix in[] = {{dy, rows, cols, lddy, size_of(type)},
                         {h, rows, cols, ldh, rs},
                         {dresidual, rows, cols, lddr, rs},
                         {weight, 1, cols, cols, size_of(weight_type)},
                         floats(rstd, rows, 1)};
    const Matrix out[] = {{dx, rows, cols, lddx, rs}, floats(dweight, 1, cols),
                          floats(dweight != nullptr ? workspace : nullptr, partials, cols)};
    for (const Matrix& i : in)
        if (i.p != nullptr && !aligned(i)) return AP_ERR_ALIGN;
    for (const Matrix& o : out)
        if (o.p != nullptr && !aligned(o)) return AP_ERR_ALIGN;
    if (out[2].p != nullptr && out[2].at() % 16 != 0) return AP_ERR_ALIGN;
    for (int o = 0; o < 3; ++o) {
        for (int i = 0; i < 5; ++i) {
            const bool in_place = o == 0 && i < 3 && same_place(out[o], in[i]);
            if (!in_place && overlap(out[o], in[i])) return AP_ERR_ALIAS;
        }
        for (int p = 0; p < o; ++p)
            if (overlap(out[o], out[p])) return AP_ERR_ALIAS;
    }
    DeviceInfo di;
    const ap_status st = current_device(&di);
    if (st != AP_OK) return st;
    NormGradArgs a{dy, h, weight, rstd, dresidual, dx, dweight, static_cast<float*>(workspace), rows, cols, lddy, ldh,
                   lddr, lddx, type, residual_type, weight_type};
    return launch_rms_norm_backward(di, options(), a, stream);
}

int64_t ap_debug_norm_grad_ctas(int64_t rows, int64_t cols, int type, int residual_type, int dresidual, int sms) {
    const ap_dtype t = static_cast<ap_dtype>(type), rt = static_cast<ap_dtype>(residual_type);
    if (!valid_type(t) || (rt != t && rt != AP_F32) || rows < 0 || cols < 1 || cols > kMaxElems / (rows > 0 ? rows : 1) || sms < 1)
        return -1;
    DeviceInfo di{};
    di.sms = sms;
    NormGradArgs a{};  // planned, not launched: addresses stand for aligned ones
    a.rows = rows;
    a.cols = a.lddy = a.ldh = a.lddr = a.lddx = cols;
    a.type = t;
    a.residual_type = rt;
    a.weight_type = AP_F32;
    a.rstd = reinterpret_cast<const float*>(256);
    a.dresidual = dresidual ? a.rstd : nullptr;
    return norm_grad_ctas(di, options(), a);
}

ap_status ap_quantize(const void* x, int64_t ldx, ap_dtype type, int64_t rows, int64_t cols, int block_rows, uint8_t* q,
                      int64_t ldq, float* scales, uint8_t* qt, int64_t ldqt, float* scales_t, cudaStream_t stream) {
    if (!valid_type(type) || (block_rows != 1 && block_rows != 128)) return AP_ERR_ARG;
    if (rows < 0 || cols < 0) return AP_ERR_SHAPE;
    if (rows == 0 || cols == 0) return AP_OK;
    if (cols > kMaxElems / rows || !valid_ld(rows, cols, ldx)) return AP_ERR_SHAPE;
    if (x == nullptr || (q == nullptr && qt == nullptr)) return AP_ERR_NULL;
    if ((q == nullptr) != (scales == nullptr) || (qt == nullptr) != (scales_t == nullptr)) return AP_ERR_NULL;
    if ((q != nullptr && !valid_ld(rows, cols, ldq)) || (qt != nullptr && !valid_ld(cols, rows, ldqt))) return AP_ERR_SHAPE;
    const bool tiles = block_rows == 128;
    const Matrix in{x, rows, cols, ldx, size_of(type)};
    const Matrix out[] = {{q, rows, cols, ldq, 1},
                          {qt, cols, rows, ldqt, 1},
                          floats(scales, tiles ? blocks(rows) : rows, blocks(cols)),
                          floats(scales_t, tiles ? blocks(cols) : cols, blocks(rows))};
    if (!aligned(in)) return AP_ERR_ALIGN;
    for (int o = 0; o < 4; ++o) {
        if (out[o].p != nullptr && !aligned(out[o])) return AP_ERR_ALIGN;
        if (overlap(out[o], in)) return AP_ERR_ALIAS;
        for (int p = 0; p < o; ++p)
            if (overlap(out[o], out[p])) return AP_ERR_ALIAS;
    }
    DeviceInfo di;
    const ap_status st = current_device(&di);
    if (st != AP_OK) return st;
    QuantArgs a{x, q, scales, qt, scales_t, rows, cols, ldx, ldq, ldqt, type, block_rows};
    return launch_quantize(di, a, stream);
}

ap_status ap_debug_block_scale(const float* amax, float* scale, float* inv, int64_t n, cudaStream_t stream) {
    if (n < 0 || n > (int64_t(1) << 30)) return AP_ERR_SHAPE;
    if (n == 0) return AP_OK;
    if (amax == nullptr || scale == nullptr || inv == nullptr) return AP_ERR_NULL;
    const Matrix all[] = {floats(amax, 1, n), floats(scale, 1, n), floats(inv, 1, n)};
    for (int i = 0; i < 3; ++i) {
        if (!aligned(all[i])) return AP_ERR_ALIGN;
        for (int j = 0; j < i; ++j)
            if (overlap(all[i], all[j])) return AP_ERR_ALIAS;
    }
    DeviceInfo di;
    const ap_status st = current_device(&di);
    if (st != AP_OK) return st;
    return launch_block_scale(amax, scale, inv, n, stream);
}

ap_status ap_matmul_fp8(const uint8_t* a, int64_t lda, const float* a_scales, const uint8_t* b, int64_t ldb,
                        const float* b_scales, int b_block_rows, void* c, int64_t ldc, ap_dtype c_type, int64_t m,
                        int64_t n, int64_t k, cudaStream_t stream) {
    if (!valid_type(c_type) || (b_block_rows != 1 && b_block_rows != 128)) return AP_ERR_ARG;
    if (m < 0 || n < 0 || k < 0 || m > kMaxDim || n > kMaxDim || k > kMaxDim) return AP_ERR_SHAPE;
    if (m == 0 || n == 0) return AP_OK;
    if (n > kMaxElems / m || !valid_ld(m, n, ldc)) return AP_ERR_SHAPE;
    if (c == nullptr) return AP_ERR_NULL;
    const Matrix out{c, m, n, ldc, size_of(c_type)};
    if (!aligned(out)) return AP_ERR_ALIGN;
    if (k > 0) {
        if (k > kMaxElems / m || k > kMaxElems / n || !valid_ld(m, k, lda) || !valid_ld(n, k, ldb)) return AP_ERR_SHAPE;
        if (a == nullptr || b == nullptr || a_scales == nullptr || b_scales == nullptr) return AP_ERR_NULL;
        const Matrix in[] = {{a, m, k, lda, 1},
                             {b, n, k, ldb, 1},
                             floats(a_scales, m, blocks(k)),
                             floats(b_scales, b_block_rows == 1 ? n : blocks(n), blocks(k))};
        for (int i = 0; i < 2; ++i)  // tensor maps: base and row pitch
            if (in[i].at() % 16 != 0 || in[i].ld % 16 != 0) return AP_ERR_ALIGN;
        for (const Matrix& i : in) {
            if (!aligned(i)) return AP_ERR_ALIGN;
            if (overlap(out, i)) return AP_ERR_ALIAS;
        }
    }
    DeviceInfo di;
    const ap_status st = current_device(&di);
    if (st != AP_OK) return st;
    MatmulArgs args{a, b, a_scales, b_scales, c, m, n, k, lda, ldb, ldc, c_type, b_block_rows};
    return launch_matmul_fp8(di, options(), args, stream);
}

}  // extern "C"
