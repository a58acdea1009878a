// api_mx.cpp -- argument checks of the microscaled-tensor entry points, and of
// the norm and the experts' operators around them.  See include/expzip.h for the
// contract.
#include <cmath>
#include <cstdint>

#include "ez_internal.h"

namespace {

constexpr uint64_t kMaxDim = 1ull << 31, kMaxValues = 1ull << 40;

bool al(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool known(uint32_t f) { return f >= EZ_MX_E2M1 && f <= EZ_MX_E5M2; }
bool size_ok(uint64_t rows, uint64_t cols)
{
    return rows <= kMaxDim && cols <= kMaxDim && (!rows || cols <= kMaxValues / rows);
}
bool form_ok(const void* codes, const void* scales) { return codes && scales && al(codes, 16) && al(scales, 16); }
// a row-major matrix of `bytes`-wide elements
bool matrix_ok(const void* p, uint64_t rows, uint64_t cols, uint64_t ld, uintptr_t bytes)
{
    return p && al(p, bytes) && (rows <= 1 || (ld >= cols && ld <= kMaxValues / rows));
}
constexpr uint64_t kMaxNorm = 16384, kMaxExperts = 1024, kMaxRows = (1ull << 31) - 1;
// The tokens' kernels (k_moe.cu) count columns in 32 bits with a sign and go some hundred
// past the last one.
constexpr uint64_t kMaxTokenCols = (1ull << 31) - 1024;
// Rows of a routing; false for sizes that have none.
bool routing_rows(uint64_t tokens, uint64_t choices, uint64_t experts, uint64_t* rows)
{
    if (tokens > kMaxDim || choices > kMaxDim) return false;
    const uint64_t pairs = tokens * choices, some = pairs < experts ? pairs : experts;
    *rows = (pairs + 127 * some) / 128 * 128;
    return *rows <= kMaxRows;
}
// The sizes of a routing's way back: rows, tokens and their choices.
bool back_ok(uint64_t rows, uint64_t tokens, uint64_t choices, uint64_t cols)
{
    return size_ok(rows, cols) && size_ok(tokens, cols) && rows <= kMaxRows && tokens <= kMaxRows &&
           choices <= kMaxRows && tokens * choices <= kMaxRows;
}
ez_status cuda_status(cudaError_t e) { return e == cudaSuccess ? EZ_OK : EZ_ERR_CUDA; }
cudaStream_t st(void* stream) { return static_cast<cudaStream_t>(stream); }

}  // namespace

extern "C" {

ez_status ez_mx_sizes(uint32_t format, uint64_t rows, uint64_t cols, uint64_t* code_bytes, uint64_t* scale_bytes)
{
    if (!known(format) || !size_ok(rows, cols)) return EZ_ERR_ARG;
    const uint64_t nb = (cols + 31) / 32;
    if (code_bytes) *code_bytes = rows * nb * (format == EZ_MX_E2M1 ? 16 : 32);
    if (scale_bytes) *scale_bytes = (rows + 127) / 128 * ((nb + 3) / 4) * 512;
    return EZ_OK;
}

ez_status ez_mx_quantize(const uint16_t* d_x, uint64_t rows, uint64_t cols, uint64_t ldx, uint32_t row_format,
                         uint8_t* d_row_codes, uint8_t* d_row_scales, uint32_t col_format, uint8_t* d_col_codes,
                         uint8_t* d_col_scales, void* stream)
{
    if ((row_format && !known(row_format)) || (col_format && !known(col_format)) || !(row_format || col_format) ||
        !size_ok(rows, cols))
        return EZ_ERR_ARG;
    if (!rows || !cols) return EZ_OK;
    if (!matrix_ok(d_x, rows, cols, ldx, 2) || (row_format && !form_ok(d_row_codes, d_row_scales)) ||
        (col_format && !form_ok(d_col_codes, d_col_scales)))
        return EZ_ERR_ARG;
    return cuda_status(ezk::launch_mx_quantize(d_x, rows, cols, ldx, (int)row_format, d_row_codes, d_row_scales,
                                               (int)col_format, d_col_codes, d_col_scales, st(stream)));
}

ez_status ez_mx_dequantize(uint32_t format, const uint8_t* d_codes, const uint8_t* d_scales, uint64_t rows,
                           uint64_t cols, uint16_t* d_out, uint64_t ldo, void* stream)
{
    if (!known(format) || !size_ok(rows, cols)) return EZ_ERR_ARG;
    if (!rows || !cols) return EZ_OK;
    if (!form_ok(d_codes, d_scales) || !matrix_ok(d_out, rows, cols, ldo, 2)) return EZ_ERR_ARG;
    return cuda_status(ezk::launch_mx_dequantize((int)format, d_codes, d_scales, rows, cols, d_out, ldo, st(stream)));
}

ez_status ez_mx_matmul(uint32_t a_format, const uint8_t* d_a_codes, const uint8_t* d_a_scales, uint64_t M,
                       uint32_t b_format, const uint8_t* d_b_codes, const uint8_t* d_b_scales, uint64_t N, uint64_t K,
                       const float* d_add, void* d_c, uint64_t ldc, int c_f32, uint32_t* d_status, void* stream)
{
    if (!known(a_format) || !known(b_format) || !size_ok(M, K) || !size_ok(N, K) || !size_ok(M, N))
        return EZ_ERR_ARG;
    if ((a_format == EZ_MX_E2M1) != (b_format == EZ_MX_E2M1)) return EZ_ERR_UNSUPPORTED;
    if ((c_f32 != 0 && c_f32 != 1) || (d_add && !c_f32) || !d_status || !al(d_status, 4)) return EZ_ERR_ARG;
    if (!M || !N) return EZ_OK;
    if (!matrix_ok(d_c, M, N, ldc, c_f32 ? 4 : 2) || (d_add && !al(d_add, 4))) return EZ_ERR_ARG;
    if (K && (!form_ok(d_a_codes, d_a_scales) || !form_ok(d_b_codes, d_b_scales))) return EZ_ERR_ARG;
    return cuda_status(ezk::launch_mx_matmul((int)a_format, d_a_codes, d_a_scales, M, (int)b_format, d_b_codes,
                                             d_b_scales, N, K, d_add, d_c, ldc, c_f32, d_status, st(stream)));
}

ez_status ez_mx_wait_limit(uint32_t polls)
{
    if (polls > 1u << 24) return EZ_ERR_ARG;
    ezk::set_mx_wait_limit(polls);
    return EZ_OK;
}

ez_status ez_mx_swiglu(uint32_t format, const uint16_t* d_gate, uint64_t ld_gate, const uint16_t* d_up, uint64_t ld_up,
                       uint64_t rows, uint64_t cols, uint8_t* d_gate_codes, uint8_t* d_gate_scales,
                       uint8_t* d_up_codes, uint8_t* d_up_scales, uint16_t* d_h, uint64_t ldh, void* stream)
{
    if (!known(format) || !size_ok(rows, cols)) return EZ_ERR_ARG;
    if (format == EZ_MX_E2M1) return EZ_ERR_UNSUPPORTED;
    if (!rows || !cols) return EZ_OK;
    if (!matrix_ok(d_gate, rows, cols, ld_gate, 2) || !matrix_ok(d_up, rows, cols, ld_up, 2) ||
        !matrix_ok(d_h, rows, cols, ldh, 2) || !form_ok(d_gate_codes, d_gate_scales) ||
        !form_ok(d_up_codes, d_up_scales))
        return EZ_ERR_ARG;
    return cuda_status(ezk::launch_mx_swiglu((int)format, d_gate, ld_gate, d_up, ld_up, rows, cols, d_gate_codes,
                                             d_gate_scales, d_up_codes, d_up_scales, d_h, ldh, st(stream)));
}

ez_status ez_mx_swiglu_backward(uint32_t format, const uint8_t* d_gate_codes, const uint8_t* d_gate_scales,
                                const uint8_t* d_up_codes, const uint8_t* d_up_scales, uint64_t rows, uint64_t cols,
                                const uint16_t* d_dh, uint64_t ld_dh, uint16_t* d_dgate, uint64_t ld_dgate,
                                uint16_t* d_dup, uint64_t ld_dup, uint16_t* d_h, uint64_t ldh, void* stream)
{
    if (!known(format) || !size_ok(rows, cols)) return EZ_ERR_ARG;
    if (format == EZ_MX_E2M1) return EZ_ERR_UNSUPPORTED;
    if (!rows || !cols) return EZ_OK;
    if (!form_ok(d_gate_codes, d_gate_scales) || !form_ok(d_up_codes, d_up_scales) ||
        !matrix_ok(d_dh, rows, cols, ld_dh, 2) || !matrix_ok(d_dgate, rows, cols, ld_dgate, 2) ||
        !matrix_ok(d_dup, rows, cols, ld_dup, 2) || (d_h && !matrix_ok(d_h, rows, cols, ldh, 2)))
        return EZ_ERR_ARG;
    return cuda_status(ezk::launch_mx_swiglu_backward((int)format, d_gate_codes, d_gate_scales, d_up_codes,
                                                      d_up_scales, rows, cols, d_dh, ld_dh, d_dgate, ld_dgate, d_dup,
                                                      ld_dup, d_h, ldh, st(stream)));
}

ez_status ez_mx_rms_norm(const uint16_t* d_x, uint64_t ldx, const uint16_t* d_residual, uint64_t ld_residual,
                         uint64_t rows, uint64_t cols, const uint16_t* d_weight, float eps, uint16_t* d_total,
                         uint64_t ld_total, float* d_rstd, float* d_rstd_low, uint16_t* d_y, uint64_t ldy,
                         uint32_t row_format, uint8_t* d_row_codes, uint8_t* d_row_scales, uint32_t col_format,
                         uint8_t* d_col_codes, uint8_t* d_col_scales, void* stream)
{
    if ((row_format && !known(row_format)) || (col_format && !known(col_format)) || !size_ok(rows, cols) ||
        !(eps >= 0.f) || !std::isfinite(eps) || !cols)
        return EZ_ERR_ARG;
    if (cols > kMaxNorm) return EZ_ERR_UNSUPPORTED;
    if (!rows) return EZ_OK;
    if (!(row_format || col_format || d_y) || !matrix_ok(d_x, rows, cols, ldx, 2) ||
        (d_residual && !matrix_ok(d_residual, rows, cols, ld_residual, 2)) ||
        !d_weight || !al(d_weight, 2) || (d_residual && !d_total) ||
        (d_total && !matrix_ok(d_total, rows, cols, ld_total, 2)) || !d_rstd || !al(d_rstd, 4) ||
        (col_format && !d_rstd_low) || !al(d_rstd_low, 4) || (d_y && !matrix_ok(d_y, rows, cols, ldy, 2)) ||
        (d_y && (d_y == d_total || (d_y == d_x && col_format && !d_total) ||
                 (rows > 1 && ((d_y == d_x && ldy != ldx) || (d_y == d_residual && ldy != ld_residual))))) ||
        (row_format && !form_ok(d_row_codes, d_row_scales)) ||
        (col_format && !form_ok(d_col_codes, d_col_scales)) || (d_total == d_x && rows > 1 && ld_total != ldx) ||
        (d_residual && d_total == d_residual && rows > 1 && ld_total != ld_residual))
        return EZ_ERR_ARG;
    return cuda_status(ezk::launch_mx_rms_norm(d_x, ldx, d_residual, ld_residual, rows, (uint32_t)cols, d_weight, eps,
                                               d_total, ld_total, d_rstd, d_rstd_low, d_y, ldy, (int)row_format, d_row_codes,
                                               d_row_scales, (int)col_format, d_col_codes, d_col_scales, st(stream)));
}

ez_status ez_mx_rms_norm_ws(uint64_t rows, uint64_t cols, uint64_t* ws_bytes)
{
    if (!size_ok(rows, cols) || !cols || !ws_bytes) return EZ_ERR_ARG;
    if (cols > kMaxNorm) return EZ_ERR_UNSUPPORTED;
    *ws_bytes = ezk::mx_rms_norm_ws(rows, cols);
    return EZ_OK;
}

ez_status ez_mx_rms_norm_backward(const uint16_t* d_dy, uint64_t ld_dy, const uint16_t* d_total, uint64_t ld_total,
                                  const float* d_rstd, const uint16_t* d_weight, const uint16_t* d_dtotal,
                                  uint64_t ld_dtotal, uint64_t rows, uint64_t cols, uint16_t* d_dx, uint64_t ld_dx,
                                  const float* d_add, float* d_dweight, void* d_ws, uint64_t ws_bytes, void* stream)
{
    if (!size_ok(rows, cols) || !cols || (d_add && !d_dweight) || !al(d_add, 4) || !al(d_dweight, 4)) return EZ_ERR_ARG;
    if (cols > kMaxNorm) return EZ_ERR_UNSUPPORTED;
    if (!rows && !d_dweight) return EZ_OK;
    if (rows && (!matrix_ok(d_dy, rows, cols, ld_dy, 2) || !matrix_ok(d_total, rows, cols, ld_total, 2) || !d_rstd ||
                 !al(d_rstd, 4) || !d_weight || !al(d_weight, 2) ||
                 (d_dtotal && !matrix_ok(d_dtotal, rows, cols, ld_dtotal, 2)) || !matrix_ok(d_dx, rows, cols, ld_dx, 2) ||
                 (d_dx == d_dy && rows > 1 && ld_dx != ld_dy) || (d_dx == d_dtotal && rows > 1 && ld_dx != ld_dtotal)))
        return EZ_ERR_ARG;
    const uint64_t need = d_dweight ? ezk::mx_rms_norm_ws(rows, cols) : 0;
    if (need && (!d_ws || !al(d_ws, 16))) return EZ_ERR_ARG;
    if (ws_bytes < need) return EZ_ERR_CAPACITY;
    return cuda_status(ezk::launch_mx_rms_norm_backward(d_dy, ld_dy, d_total, ld_total, d_rstd, d_weight, d_dtotal,
                                                        ld_dtotal, rows, (uint32_t)cols, d_dx, ld_dx, d_add, d_dweight,
                                                        static_cast<float*>(d_ws), st(stream)));
}

ez_status ez_moe_rows(uint64_t tokens, uint32_t choices, uint32_t experts, uint64_t* rows)
{
    if (!rows || !experts) return EZ_ERR_ARG;
    if (experts > kMaxExperts) return EZ_ERR_UNSUPPORTED;
    return routing_rows(tokens, choices, experts, rows) ? EZ_OK : EZ_ERR_ARG;
}

ez_status ez_moe_sort_ws(uint64_t tokens, uint32_t choices, uint32_t experts, uint64_t* ws_bytes)
{
    uint64_t rows;
    if (!ws_bytes) return EZ_ERR_ARG;
    const ez_status e = ez_moe_rows(tokens, choices, experts, &rows);
    if (e == EZ_OK) *ws_bytes = ezk::moe_sort_ws(tokens * choices, experts);
    return e;
}

ez_status ez_moe_sort(const void* d_ids, uint32_t id_bytes, uint64_t ld_ids, uint64_t tokens, uint32_t choices,
                      uint32_t experts, int32_t* d_counts, int32_t* d_offsets, int32_t* d_slots, int32_t* d_sources,
                      void* d_ws, uint64_t ws_bytes, void* stream)
{
    uint64_t rows;
    const ez_status e = ez_moe_rows(tokens, choices, experts, &rows);
    if (e != EZ_OK) return e;
    const uint64_t pairs = tokens * choices, need = ezk::moe_sort_ws(pairs, experts);
    if ((id_bytes != 4 && id_bytes != 8) || !d_counts || !al(d_counts, 4) || !d_offsets || !al(d_offsets, 4))
        return EZ_ERR_ARG;
    if (pairs && (!matrix_ok(d_ids, tokens, choices, ld_ids, id_bytes) || !d_slots || !al(d_slots, 4) || !d_sources ||
                  !al(d_sources, 4) || (need && (!d_ws || !al(d_ws, 4)))))
        return EZ_ERR_ARG;
    if (ws_bytes < need) return EZ_ERR_CAPACITY;
    return cuda_status(ezk::launch_moe_sort(d_ids, (int)id_bytes, ld_ids, tokens, choices, experts, rows, d_counts,
                                            d_offsets, d_slots, d_sources, d_ws, st(stream)));
}

ez_status ez_moe_dispatch(const uint16_t* d_x, uint64_t ldx, uint64_t tokens, uint64_t cols, const int32_t* d_offsets,
                          const int32_t* d_sources, const int32_t* d_slots, uint32_t choices, uint32_t experts,
                          const float* d_weights, uint32_t row_format, uint8_t* d_row_codes, uint8_t* d_row_scales,
                          uint32_t col_format, uint8_t* d_col_codes, uint8_t* d_col_scales, void* stream)
{
    uint64_t rows;
    const ez_status e = ez_moe_rows(tokens, choices, experts, &rows);
    if (e != EZ_OK) return e;
    if ((row_format && !known(row_format)) || (col_format && !known(col_format)) || !(row_format || col_format) ||
        !size_ok(rows, cols))
        return EZ_ERR_ARG;
    if (!rows || !cols) return EZ_OK;
    if (cols > kMaxTokenCols) return EZ_ERR_UNSUPPORTED;
    if (!matrix_ok(d_x, tokens, cols, ldx, 2) || !d_offsets || !al(d_offsets, 4) || !d_sources || !al(d_sources, 4) ||
        !d_slots || !al(d_slots, 4) || !al(d_weights, 4) || (row_format && !form_ok(d_row_codes, d_row_scales)) ||
        (col_format && !form_ok(d_col_codes, d_col_scales)))
        return EZ_ERR_ARG;
    return cuda_status(ezk::launch_moe_dispatch(d_x, ldx, (uint32_t)tokens, cols, d_offsets, d_sources, d_slots, choices,
                                                experts, rows, d_weights, (int)row_format, d_row_codes, d_row_scales,
                                                (int)col_format, d_col_codes, d_col_scales, st(stream)));
}

ez_status ez_moe_combine(const uint16_t* d_in, uint64_t ld_in, uint64_t rows, uint64_t cols, const int32_t* d_slots,
                         const float* d_weights, uint64_t tokens, uint32_t choices, uint16_t* d_y, uint64_t ldy,
                         void* stream)
{
    if (!back_ok(rows, tokens, choices, cols)) return EZ_ERR_ARG;
    if (!tokens || !cols) return EZ_OK;
    if (cols > kMaxTokenCols) return EZ_ERR_UNSUPPORTED;
    if ((rows && !matrix_ok(d_in, rows, cols, ld_in, 2)) || (choices && (!d_slots || !al(d_slots, 4))) ||
        !al(d_weights, 4) || !matrix_ok(d_y, tokens, cols, ldy, 2) || d_y == d_in)
        return EZ_ERR_ARG;
    return cuda_status(ezk::launch_moe_combine(d_in, ld_in, rows, (uint32_t)cols, d_slots, d_weights, (uint32_t)tokens,
                                               choices, d_y, ldy, st(stream)));
}

ez_status ez_moe_weight_gradient(const uint16_t* d_dy, uint64_t ld_dy, const uint16_t* d_in, uint64_t ld_in,
                                 uint64_t rows, uint64_t cols, const int32_t* d_slots, uint64_t tokens,
                                 uint32_t choices, float* d_dweights, void* stream)
{
    if (!back_ok(rows, tokens, choices, cols)) return EZ_ERR_ARG;
    if (!tokens || !choices) return EZ_OK;
    if (cols > kMaxTokenCols) return EZ_ERR_UNSUPPORTED;
    if ((cols && !matrix_ok(d_dy, tokens, cols, ld_dy, 2)) || (rows && cols && !matrix_ok(d_in, rows, cols, ld_in, 2)) ||
        !d_slots || !al(d_slots, 4) || !d_dweights || !al(d_dweights, 4))
        return EZ_ERR_ARG;
    return cuda_status(ezk::launch_moe_weight_gradient(d_dy, ld_dy, d_in, ld_in, rows, (uint32_t)cols, d_slots,
                                                       (uint32_t)tokens, choices, d_dweights, st(stream)));
}

ez_status ez_moe_matmul(uint32_t a_format, const uint8_t* d_a_codes, const uint8_t* d_a_scales, uint64_t rows,
                        uint32_t b_format, const uint8_t* d_b_codes, const uint8_t* d_b_scales, uint32_t experts,
                        uint64_t N, uint64_t K, const int32_t* d_counts, const int32_t* d_offsets, uint64_t pairs,
                        void* d_c, uint64_t ldc, int c_f32, uint32_t* d_status, void* stream)
{
    if (!known(a_format) || !known(b_format) || !experts || !size_ok(rows, K) || N > kMaxDim ||
        !size_ok(experts * N, K) || !size_ok(rows, N) || rows % 128 || rows > kMaxRows || !K ||
        (c_f32 != 0 && c_f32 != 1) || !d_status || !al(d_status, 4))
        return EZ_ERR_ARG;
    if ((a_format == EZ_MX_E2M1) != (b_format == EZ_MX_E2M1) || experts > kMaxExperts) return EZ_ERR_UNSUPPORTED;
    if (!rows || !N || !pairs) return EZ_OK;
    if (!matrix_ok(d_c, rows, N, ldc, c_f32 ? 4 : 2) || !form_ok(d_a_codes, d_a_scales) ||
        !form_ok(d_b_codes, d_b_scales) || !d_counts || !al(d_counts, 4) || !d_offsets || !al(d_offsets, 4))
        return EZ_ERR_ARG;
    return cuda_status(ezk::launch_moe_matmul((int)a_format, d_a_codes, d_a_scales, rows, (int)b_format, d_b_codes,
                                              d_b_scales, experts, N, K, d_counts, d_offsets,
                                              pairs < rows ? pairs : rows, d_c, ldc, c_f32, d_status, st(stream)));
}

ez_status ez_moe_gradient(uint32_t a_format, const uint8_t* d_a_codes, const uint8_t* d_a_scales, uint64_t N,
                          uint32_t b_format, const uint8_t* d_b_codes, const uint8_t* d_b_scales, uint64_t K,
                          uint64_t rows, uint32_t experts, const int32_t* d_offsets, const float* d_add, float* d_c,
                          uint64_t ldc, uint32_t* d_status, void* stream)
{
    if (!known(a_format) || !known(b_format) || !experts || !size_ok(N, rows) || !size_ok(K, rows) || N > kMaxDim ||
        !size_ok(experts * N, K) || rows % 128 || rows > kMaxRows || !d_status || !al(d_status, 4))
        return EZ_ERR_ARG;
    if (a_format == EZ_MX_E2M1 || b_format == EZ_MX_E2M1 || experts > kMaxExperts) return EZ_ERR_UNSUPPORTED;
    if (!N || !K) return EZ_OK;
    if (!matrix_ok(d_c, experts * N, K, ldc, 4) || !al(d_add, 4) || !d_offsets || !al(d_offsets, 4)) return EZ_ERR_ARG;
    if (rows && (!form_ok(d_a_codes, d_a_scales) || !form_ok(d_b_codes, d_b_scales))) return EZ_ERR_ARG;
    return cuda_status(ezk::launch_moe_gradient((int)a_format, d_a_codes, d_a_scales, N, (int)b_format, d_b_codes,
                                                d_b_scales, K, rows, experts, d_offsets, d_add, d_c, ldc, d_status,
                                                st(stream)));
}

}  // extern "C"
