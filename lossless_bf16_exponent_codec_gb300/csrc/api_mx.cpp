// api_mx.cpp -- argument checks of the microscaled-tensor entry points.  See
// include/expzip.h for the contract.
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

}  // extern "C"
