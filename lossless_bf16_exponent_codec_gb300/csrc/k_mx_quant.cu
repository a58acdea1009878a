// k_mx_quant.cu -- microscaled quantisation of a BF16 matrix and its inverse.
#include "ez_internal.h"
#include "ez_mx.cuh"

namespace ezk {
using namespace ezmx;

// One tile of 128 x 128 values: read once, encoded along its rows (row form)
// and, from shared memory, along its columns (column form: the transpose).
template <int ROW, int COL>
__global__ void __launch_bounds__(kThreadsMx) k_mx_quantize(Rows x, uint64_t rows, uint64_t cols, Form row,
                                                            Form col)
{
    __shared__ uint4 s_tile[COL ? kTileRows * 16 : 1];
    __shared__ uint4 s_row[32], s_col[32];
    const uint32_t t = threadIdx.x, seg = t & 15u;
    const uint64_t col_tiles = ez::cdiv(cols, kTileCols), row_tiles = ez::cdiv(rows, kTileRows);
    const uint64_t rt = blockIdx.x / col_tiles, ct = blockIdx.x - rt * col_tiles;
    const uint64_t c = ct * kTileCols + 8 * seg;

    uint4 v[kRowIters];
#pragma unroll
    for (int i = 0; i < kRowIters; ++i) {
        const uint64_t r = rt * kTileRows + (t >> 4) + kRowStep * i;
        v[i] = load8(x, r, c, r < rows ? cols : 0);
    }
#pragma unroll
    for (int i = 0; i < kRowIters; ++i) {
        const uint32_t lr = (t >> 4) + kRowStep * i;
        const uint64_t r = rt * kTileRows + lr;
        if constexpr (COL != 0) s_tile[lr * 16 + seg] = v[i];
        if constexpr (ROW != 0) {
            uint32_t code[2];
            const uint32_t s = quantise_quad<ROW>(v[i], code);
            const bool in = r < rows && c / kBlock * kBlock < cols;
            if ((t & 3u) == 0) reinterpret_cast<uint8_t*>(s_row)[scale_at(lr, seg >> 2)] = in ? (uint8_t)s : 0;
            if (in) {
                uint8_t* p = row.codes + r * code_pitch<ROW>(cols) + c * Fmt<ROW>::kBits / 8;
                if constexpr (Fmt<ROW>::kBits == 4)
                    *reinterpret_cast<uint32_t*>(p) = code[0];
                else
                    *reinterpret_cast<uint2*>(p) = make_uint2(code[0], code[1]);
            }
        }
    }
    __syncthreads();
    if constexpr (COL != 0) {
        // thread: columns 2 cp, 2 cp + 1 of the block of rows 32 rb ..; one
        // word per row, a warp's 32 words in a row of shared memory
        const uint32_t cp = t & 63u, rb = t >> 6;
        const uint32_t* tile = reinterpret_cast<const uint32_t*>(s_tile) + rb * 32 * 64 + cp;
        uint32_t w[32], m = 0u;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            w[i] = tile[i * 64];
            m = mag_max(m, w[i]);
        }
        const uint64_t r0 = rt * kTileRows + rb * 32;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t s = scale_byte<COL>(h ? m >> 16 : m & 0xFFFFu);
            const uint64_t cc = ct * kTileCols + 2 * cp + h;
            const bool in = cc < cols && r0 < rows;
            reinterpret_cast<uint8_t*>(s_col)[scale_at(2 * cp + h, rb)] = in ? (uint8_t)s : 0;
            const float inv = inv_scale(s);
            constexpr int kWords = Fmt<COL>::kBits;   // 32 values
            uint32_t code[kWords];
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                float f[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t u = w[8 * g + i];
                    f[i] = s == 255u ? 0.f : (h ? hi_f(u) : lo_f(u)) * inv;
                }
                encode8<COL>(f, code + g * (kWords / 4));
            }
            if (in) {
                uint4* p = reinterpret_cast<uint4*>(col.codes + cc * code_pitch<COL>(rows) +
                                                    r0 * Fmt<COL>::kBits / 8);
#pragma unroll
                for (int i = 0; i < kWords / 4; ++i)
                    p[i] = make_uint4(code[4 * i], code[4 * i + 1], code[4 * i + 2], code[4 * i + 3]);
            }
        }
        __syncthreads();
    }
    if (t < 32) {
        if constexpr (ROW != 0) reinterpret_cast<uint4*>(row.scales)[(rt * col_tiles + ct) * 32 + t] = s_row[t];
        if constexpr (COL != 0) reinterpret_cast<uint4*>(col.scales)[(ct * row_tiles + rt) * 32 + t] = s_col[t];
    }
}

template <int FMT>
__global__ void __launch_bounds__(kThreadsMx) k_mx_dequantize(Form in, uint64_t rows, uint64_t cols,
                                                              uint16_t* out, uint64_t ldo)
{
    __shared__ uint4 s_scale[32];
    const uint32_t t = threadIdx.x, seg = t & 15u;
    const uint64_t col_tiles = ez::cdiv(cols, kTileCols);
    const uint64_t rt = blockIdx.x / col_tiles, ct = blockIdx.x - rt * col_tiles;
    const uint64_t c = ct * kTileCols + 8 * seg;
    uint2 code[kRowIters];
#pragma unroll
    for (int i = 0; i < kRowIters; ++i) {
        const uint64_t r = rt * kTileRows + (t >> 4) + kRowStep * i;
        code[i] = make_uint2(0u, 0u);
        if (r < rows && c < cols) {
            const uint8_t* p = in.codes + r * code_pitch<FMT>(cols) + c * Fmt<FMT>::kBits / 8;
            if constexpr (Fmt<FMT>::kBits == 4)
                code[i].x = __ldg(reinterpret_cast<const uint32_t*>(p));
            else
                code[i] = __ldg(reinterpret_cast<const uint2*>(p));
        }
    }
    if (t < 32) s_scale[t] = ez::ld_v4_nc(in.scales + (blockIdx.x * 32ull + t) * 16);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kRowIters; ++i) {
        const uint32_t lr = (t >> 4) + kRowStep * i;
        const uint64_t r = rt * kTileRows + lr;
        const float s = scale_value(reinterpret_cast<const uint8_t*>(s_scale)[scale_at(lr, seg >> 2)]);
        const uint32_t w[2] = {code[i].x, code[i].y};
        float v[8];
        decode8<FMT>(w, v);
        store8(out + r * ldo, seg, c, r < rows ? cols : 0,
               make_uint4(bf16x2(v[0] * s, v[1] * s), bf16x2(v[2] * s, v[3] * s), bf16x2(v[4] * s, v[5] * s),
                          bf16x2(v[6] * s, v[7] * s)));
    }
}

namespace {

template <int ROW, int COL>
cudaError_t go(const Rows& x, uint64_t rows, uint64_t cols, Form row, Form col, cudaStream_t s)
{
    const unsigned grid = (unsigned)(ez::cdiv(rows, kTileRows) * ez::cdiv(cols, kTileCols));
    k_mx_quantize<ROW, COL><<<grid, kThreadsMx, 0, s>>>(x, rows, cols, row, col);
    return cudaGetLastError();
}

template <int ROW>
cudaError_t go_col(int col_fmt, const Rows& x, uint64_t rows, uint64_t cols, Form row, Form col, cudaStream_t s)
{
    switch (col_fmt) {
        case EZ_MX_E2M1: return go<ROW, EZ_MX_E2M1>(x, rows, cols, row, col, s);
        case EZ_MX_E4M3: return go<ROW, EZ_MX_E4M3>(x, rows, cols, row, col, s);
        case EZ_MX_E5M2: return go<ROW, EZ_MX_E5M2>(x, rows, cols, row, col, s);
    }
    if constexpr (ROW != 0) return go<ROW, 0>(x, rows, cols, row, col, s);
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_mx_quantize(const uint16_t* x, uint64_t rows, uint64_t cols, uint64_t ldx, int row_fmt,
                               uint8_t* row_codes, uint8_t* row_scales, int col_fmt, uint8_t* col_codes,
                               uint8_t* col_scales, cudaStream_t s)
{
    if (!rows || !cols) return cudaSuccess;
    const Rows v = make_rows(x, rows, cols, ldx);
    const Form row{row_codes, row_scales}, col{col_codes, col_scales};
    switch (row_fmt) {
        case EZ_MX_E2M1: return go_col<EZ_MX_E2M1>(col_fmt, v, rows, cols, row, col, s);
        case EZ_MX_E4M3: return go_col<EZ_MX_E4M3>(col_fmt, v, rows, cols, row, col, s);
        case EZ_MX_E5M2: return go_col<EZ_MX_E5M2>(col_fmt, v, rows, cols, row, col, s);
    }
    return go_col<0>(col_fmt, v, rows, cols, row, col, s);
}

cudaError_t launch_mx_dequantize(int fmt, const uint8_t* codes, const uint8_t* scales, uint64_t rows,
                                 uint64_t cols, uint16_t* out, uint64_t ldo, cudaStream_t s)
{
    if (!rows || !cols) return cudaSuccess;
    const unsigned grid = (unsigned)(ez::cdiv(rows, kTileRows) * ez::cdiv(cols, kTileCols));
    const Form in{const_cast<uint8_t*>(codes), const_cast<uint8_t*>(scales)};
    switch (fmt) {
        case EZ_MX_E2M1: k_mx_dequantize<EZ_MX_E2M1><<<grid, kThreadsMx, 0, s>>>(in, rows, cols, out, ldo); break;
        case EZ_MX_E4M3: k_mx_dequantize<EZ_MX_E4M3><<<grid, kThreadsMx, 0, s>>>(in, rows, cols, out, ldo); break;
        default: k_mx_dequantize<EZ_MX_E5M2><<<grid, kThreadsMx, 0, s>>>(in, rows, cols, out, ldo); break;
    }
    return cudaGetLastError();
}

}  // namespace ezk
