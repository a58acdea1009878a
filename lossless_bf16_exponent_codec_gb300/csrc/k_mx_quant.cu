// k_mx_quant.cu -- microscaled quantisation of a BF16 matrix and its inverse.
//
// Bound by memory at size: 16384 x 8192 values to 4-bit rows take 53 us (6.4
// TB/s, 0.96 of the measured copy rate), to 8-bit columns 65 (6.3), to both from
// one read 83 (5.8: the column pass through shared memory adds instructions, 2.4
// per cycle), and back from 4 bits 50 (6.8) and from 8 bits 59 (6.9).  Rows that do
// not start on 16 bytes cost a second load and a shift: 125 us for 16383 x 8191 to
// both forms, 59 back from 4 bits.  Small matrices are bound by latency
// (1 x 5120: 1.6 us a kernel).
#include "ez_internal.h"
#include "ez_mx.cuh"

namespace ezk {
using namespace ezmx;

// ROWS x 128 values: read once, encoded along the rows (row form) and, from
// shared memory, along the columns (column form: the transpose).
template <int ROW, int COL, int ROWS, bool FAST>
__device__ __forceinline__ void quantise_piece(const Rows& x, uint64_t rows, uint64_t cols, Form row, uint64_t r0,
                                               uint64_t c0, uint4* s_tile, uint8_t* s_row)
{
    const uint32_t t = threadIdx.x, seg = t & 15u;
    const uint64_t c = c0 + 8 * seg;
    constexpr int kIters = ROWS / kRowStep;
    uint4 v[kIters];
    constexpr int kFlight = FAST ? kIters : 2;
#pragma unroll
    for (int i0 = 0; i0 < kIters; i0 += kFlight) {
        Load8<FAST> in[kFlight];
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
            const uint64_t r = r0 + (t >> 4) + kRowStep * (i0 + i);
            in[i].start(x, r, c, r < rows ? cols : 0);
        }
#pragma unroll
        for (int i = 0; i < kFlight; ++i) v[i0 + i] = in[i].finish();
    }
    if constexpr (COL != 0) {
#pragma unroll
        for (int i = 0; i < kIters; ++i) s_tile[((t >> 4) + kRowStep * i) * 16 + seg] = v[i];
    }
    if constexpr (ROW != 0) {
        const bool block_in = FAST || c / kBlock * kBlock < cols;
        const uint64_t pitch = code_pitch<ROW>(cols);
        uint8_t* p = row.codes + (r0 + (t >> 4)) * pitch + c * Fmt<ROW>::kBits / 8;
#pragma unroll
        for (int i = 0; i < kIters; ++i) {
            const uint32_t lr = (t >> 4) + kRowStep * i;
            uint32_t code[2];
            const uint32_t s = quantise_quad<ROW>(v[i], code);
            const bool in = FAST || (block_in && r0 + lr < rows);
            if ((t & 3u) == 0) s_row[lr * 4 + (seg >> 2)] = in ? (uint8_t)s : 0;
            if (in) {
                if constexpr (Fmt<ROW>::kBits == 4)
                    *reinterpret_cast<uint32_t*>(p) = code[0];
                else
                    *reinterpret_cast<uint2*>(p) = make_uint2(code[0], code[1]);
            }
            p += kRowStep * pitch;
        }
    }
}

template <int ROW, int COL, int ROWS>
__global__ void __launch_bounds__(kThreadsMx, 4) k_mx_quantize(Rows x, uint64_t rows, uint64_t cols,
                                                               uint32_t col_tiles, int lines, Form row, Form col)
{
    __shared__ uint4 s_tile[COL ? ROWS * 16 : 1];
    __shared__ alignas(16) uint8_t s_row[ROWS * 4], s_col[128 * (ROWS / 32)];
    ez::grid_dep_launch();
    const uint32_t t = threadIdx.x;
    const uint32_t piece = blockIdx.x / col_tiles, ct = blockIdx.x - piece * col_tiles;
    const uint64_t r0 = (uint64_t)piece * ROWS, c0 = (uint64_t)ct * kTileCols;
    ez::grid_dep_wait();
    if (lines && r0 + ROWS <= rows && c0 + kTileCols <= cols)
        quantise_piece<ROW, COL, ROWS, true>(x, rows, cols, row, r0, c0, s_tile, s_row);
    else
        quantise_piece<ROW, COL, ROWS, false>(x, rows, cols, row, r0, c0, s_tile, s_row);
    __syncthreads();
    if constexpr (COL != 0) {
        // a thread: kCols neighbouring columns of a block of 32 rows; a row of
        // shared memory is read without conflicts by the lanes of a warp
        constexpr uint32_t kUnits = 128 * (ROWS / 32);
        constexpr int kCols = kUnits == 2 * kThreadsMx ? 2 : 1;
        const uint32_t u = t % (128 / kCols), rb = t / (128 / kCols);
        if (rb < ROWS / 32) {
            uint32_t w[32], m = 0u;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                if constexpr (kCols == 2)
                    w[i] = reinterpret_cast<const uint32_t*>(s_tile)[(rb * 32 + i) * 64 + u];
                else
                    w[i] = reinterpret_cast<const uint16_t*>(s_tile)[(rb * 32 + i) * 128 + u];
                m = mag_max(m, w[i]);
            }
            const uint64_t rblock = r0 + rb * 32;
            const uint32_t s0 = scale_byte<COL>(m & 0x7FFFu), s1 = scale_byte<COL>((m >> 16) & 0x7FFFu);
            uint32_t inv = (inv_scale(s0) & 0xFFFFu) | (inv_scale(s1) & 0xFFFF0000u);
            if (s0 == 255u || s1 == 255u) {
                const uint32_t keep = (s0 == 255u ? 0u : 0xFFFFu) | (s1 == 255u ? 0u : 0xFFFF0000u);
                inv &= keep;
#pragma unroll
                for (int i = 0; i < 32; ++i) w[i] &= keep;
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) w[i] = mul2(w[i], inv);
#pragma unroll
            for (int h = 0; h < kCols; ++h) {
                const uint64_t cc = c0 + kCols * u + h;
                const bool in = cc < cols && rblock < rows;
                s_col[(kCols * u + h) * (ROWS / 32) + rb] = in ? (uint8_t)(h ? s1 : s0) : 0;
                constexpr int kWords = Fmt<COL>::kBits;   // 32 codes
                uint32_t code[kWords];
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    float f[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[i] = h ? hi_f(w[8 * g + i]) : lo_f(w[8 * g + i]);
                    encode8<COL>(f, code + g * (kWords / 4));
                }
                if (in) {
                    uint8_t* p = col.codes + cc * code_pitch<COL>(rows) + rblock * Fmt<COL>::kBits / 8;
                    if (kWords == 8 && (reinterpret_cast<uintptr_t>(col.codes) & 31u) == 0) {
                        st_v8(p, code);          // one whole sector
                    } else {
#pragma unroll
                        for (int i = 0; i < kWords / 4; ++i)
                            reinterpret_cast<uint4*>(p)[i] =
                                make_uint4(code[4 * i], code[4 * i + 1], code[4 * i + 2], code[4 * i + 3]);
                    }
                }
            }
        }
        __syncthreads();
    }
    const uint64_t rt = r0 / kTileRows;
    const uint32_t lr = (uint32_t)(r0 % kTileRows);
    if constexpr (ROW != 0)
        if (t < ROWS)
            *scale_word(row.scales, rt * col_tiles + ct, lr + t) = reinterpret_cast<const uint32_t*>(s_row)[t];
    if constexpr (COL != 0)
        if (t < 128) {
            // the column form's tiles: its rows are the columns here
            const uint64_t tile = (uint64_t)ct * ez::cdiv(rows, kTileRows) + rt;
            uint32_t* p = scale_word(col.scales, tile, t);
            if constexpr (ROWS == 128)
                *p = reinterpret_cast<const uint32_t*>(s_col)[t];
            else if constexpr (ROWS == 64)
                reinterpret_cast<uint16_t*>(p)[lr / 64] = reinterpret_cast<const uint16_t*>(s_col)[t];
            else
                reinterpret_cast<uint8_t*>(p)[lr / 32] = s_col[t];
        }
}

// Eight consecutive codes that start at code `from` (0..7) of two neighbouring
// groups of eight.
template <int FMT>
__device__ __forceinline__ void shift_codes(const uint2& a, const uint2& b, uint32_t from, uint32_t* out)
{
    if constexpr (Fmt<FMT>::kBits == 4) {
        out[0] = __funnelshift_r(a.x, b.x, 4 * from);
    } else {
        const bool half = from & 4u;
        const uint32_t x = half ? a.y : a.x, y = half ? b.x : a.y, z = half ? b.y : b.x, s = 8 * (from & 3u);
        out[0] = __funnelshift_r(x, y, s);
        out[1] = __funnelshift_r(y, z, s);
    }
}

// A thread writes 16 aligned bytes of a row, so its first value is the row's
// misalignment before a multiple of 8 (LINES: rows on 16 bytes, none): it decodes
// codes of two neighbouring groups of eight, under the scales of one block or two.
// All its rows are 16 apart, 32 times the row stride in bytes, and so misaligned
// alike.
template <int FMT, int ROWS, bool LINES>
__global__ void __launch_bounds__(kThreadsMx) k_mx_dequantize(Form in, uint64_t rows, uint64_t cols,
                                                              uint32_t col_tiles, uint16_t* out, uint64_t ldo)
{
    __shared__ uint32_t s_scale[ROWS * 2 + 1];          // per row: 4 blocks before the tile, the tile's 4
    ez::grid_dep_launch();
    constexpr int kIters = ROWS / kRowStep, kGroup = Fmt<FMT>::kBits;            // bytes of a group
    const uint32_t t = threadIdx.x;
    const uint32_t piece = blockIdx.x / col_tiles, ct = blockIdx.x - piece * col_tiles;
    const uint64_t r0 = (uint64_t)piece * ROWS, c0 = (uint64_t)ct * kTileCols, row = r0 + (t >> 4);
    const uint64_t pitch = code_pitch<FMT>(cols);
    uint16_t* p = out + row * ldo + c0;
    // first value, and its group, from the tile's first column on; columns there
    const int c = 8 * (int)(t & 15u) - (LINES ? 0 : (int)(reinterpret_cast<uintptr_t>(p) & 15u) / 2);
    const int g = c >> 3, n = (int)min((int64_t)256, (int64_t)cols - (int64_t)c0);
    const int groups = (n + kBlock - 1) / kBlock * (kBlock / 8);
    const bool has_a = (ct || g >= 0) && g < groups, has_b = !LINES && g + 1 < groups && n > 0;
    const int left = row < rows ? (int)min((uint64_t)ROWS, rows - row) : 0;      // rows from this one on
    const uint8_t* src = in.codes + row * pitch + (int64_t)(ct * 16ull) * kGroup + g * kGroup;
    auto load = [](const uint8_t* at) {
        if constexpr (kGroup == 4)
            return make_uint2(__ldg(reinterpret_cast<const uint32_t*>(at)), 0u);
        else
            return __ldg(reinterpret_cast<const uint2*>(at));
    };
    ez::grid_dep_wait();
    uint2 a[kIters], b[LINES ? 1 : kIters];
#pragma unroll
    for (int i = 0; i < kIters; ++i, src += kRowStep * pitch) {
        const bool in_rows = i * kRowStep < left;
        a[i] = in_rows && has_a ? load(src) : make_uint2(0u, 0u);
        if constexpr (!LINES) b[i] = in_rows && has_b ? load(src + kGroup) : make_uint2(0u, 0u);
    }
    if (t < ROWS) {
        const uint64_t tiles = ez::cdiv(cols, kTileCols), tile = r0 / kTileRows * tiles + ct;
        const uint32_t lr = (uint32_t)(r0 % kTileRows) + t;
        s_scale[2 * t + 1] = ct < tiles ? *scale_word(in.scales, tile, lr) : 0u;
        if constexpr (!LINES) s_scale[2 * t] = ct ? *scale_word(in.scales, tile - 1, lr) : 0u;
    }
    __syncthreads();
    const uint8_t* sc = reinterpret_cast<const uint8_t*>(s_scale) + (t >> 4) * 8 + 4 + (c >> 5);
    const int same = 32 - (c & 31);                     // values of the first block
    const bool whole = (ct || c >= 0) && c + 8 <= n;
#pragma unroll
    for (int i = 0; i < kIters; ++i, p += kRowStep * ldo, sc += kRowStep * 8) {
        if (i * kRowStep >= left) break;
        uint32_t w[2] = {a[i].x, a[i].y};
        if constexpr (!LINES) shift_codes<FMT>(a[i], b[i], (uint32_t)c & 7u, w);
        float v[8];
        decode8<FMT>(w, v);
        const float s = scale_value(sc[0]);
        if constexpr (LINES) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] *= s;
        } else {
            const float s2 = scale_value(sc[1]);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] *= e < same ? s : s2;
        }
        const uint4 y = make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]), bf16x2(v[6], v[7]));
        if (whole) {
            *reinterpret_cast<uint4*>(p + c) = y;
        } else {
            const uint32_t x[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if ((ct || c + e >= 0) && c + e < n) p[c + e] = (uint16_t)(x[e / 2] >> (16 * (e & 1)));
        }
    }
}

namespace {

// A CTA on whole scale tiles (128 rows) moves most bytes per instruction; with
// too few tiles to put four such CTAs on every SM a CTA takes a piece of one:
// 777 x 2730 values to both 8-bit forms take 3.8 us in pieces of 32 rows, 5.1 in
// 64, 6.7 in 128; 2001 x 4109 to both 4-bit forms 9.6, 9.2 and 10.2.  Back from
// one form: 777 x 2730 in 8 bits 3.0, 3.7 and 4.0; 2001 x 4109 in 4 bits 5.5, 5.05
// and 6.3; 16383 x 8191 in 4 bits 68, 64 and 59.
uint64_t tiles_per_sm(uint64_t rows, uint64_t cols)
{
    const uint32_t sms = sm_count();
    return ez::cdiv(rows, kTileRows) * ez::cdiv(cols, kTileCols) / (sms ? sms : 1);
}

template <int ROW, int COL, int ROWS>
cudaError_t go_rows(const Rows& x, uint64_t rows, uint64_t cols, Form row, Form col, cudaStream_t s)
{
    const uint64_t col_tiles = ez::cdiv(cols, kTileCols);
    // whole scale tiles: every piece of the last one is there to clear its bytes
    const uint64_t pieces = ez::cdiv(rows, kTileRows) * (kTileRows / ROWS);
    return ez::launch_dependent(k_mx_quantize<ROW, COL, ROWS>, (unsigned)(pieces * col_tiles), kThreadsMx, 0, s, x,
                                rows, cols, (uint32_t)col_tiles, (int)lined(x.p, rows, x.ld), row, col);
}

template <int ROW, int COL>
cudaError_t go(const Rows& x, uint64_t rows, uint64_t cols, Form row, Form col, cudaStream_t s)
{
    const uint64_t per_sm = tiles_per_sm(rows, cols);
    if (per_sm >= 4) return go_rows<ROW, COL, 128>(x, rows, cols, row, col, s);
    if constexpr (COL != 0)
        if (per_sm >= 2) return go_rows<ROW, COL, 64>(x, rows, cols, row, col, s);
    return go_rows<ROW, COL, 32>(x, rows, cols, row, col, s);
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

template <int FMT, int ROWS>
cudaError_t back_rows(Form in, uint64_t rows, uint64_t cols, uint16_t* out, uint64_t ldo, cudaStream_t s)
{
    const bool lines = lined(out, rows, ldo);
    const uint64_t col_tiles = ez::cdiv(lines ? cols : cols + 7, kTileCols), pieces = ez::cdiv(rows, ROWS);
    return ez::launch_dependent(lines ? k_mx_dequantize<FMT, ROWS, true> : k_mx_dequantize<FMT, ROWS, false>,
                                (unsigned)(pieces * col_tiles), kThreadsMx, 0, s, in, rows, cols,
                                (uint32_t)col_tiles, out, ldo);
}

template <int FMT>
cudaError_t back(Form in, uint64_t rows, uint64_t cols, uint16_t* out, uint64_t ldo, cudaStream_t s)
{
    const uint64_t per_sm = tiles_per_sm(rows, cols);
    if (per_sm >= 4) return back_rows<FMT, 128>(in, rows, cols, out, ldo, s);
    if (per_sm >= 2) return back_rows<FMT, 64>(in, rows, cols, out, ldo, s);
    return back_rows<FMT, 32>(in, rows, cols, out, ldo, s);
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
    const Form in{const_cast<uint8_t*>(codes), const_cast<uint8_t*>(scales)};
    switch (fmt) {
        case EZ_MX_E2M1: return back<EZ_MX_E2M1>(in, rows, cols, out, ldo, s);
        case EZ_MX_E4M3: return back<EZ_MX_E4M3>(in, rows, cols, out, ldo, s);
    }
    return back<EZ_MX_E5M2>(in, rows, cols, out, ldo, s);
}

}  // namespace ezk
