// ez_mx_piece.cuh -- quantisation of a piece of a scale tile (ROWS x 128
// values), shared by the kernels that make microscaled forms: of a matrix, of
// its rows in another order, of normalised rows.
//
// A source says where the values come from:
//   start<FAST>(in, r, c)       start the loads of the eight values at (r, c)
//   finish<FAST>(in, r, lr, c)  their BF16 words, lr = r - r0
// FAST: the piece lies inside the matrix, whose rows are lined.
#pragma once

#include "ez_mx.cuh"

namespace ezmx {

struct MatrixSource {
    const Rows& x;
    uint64_t rows, cols;
    template <bool FAST>
    __device__ __forceinline__ void start(Load8<FAST>& in, uint64_t r, uint64_t c) const
    {
        in.start(x, r, c, r < rows ? cols : 0);
    }
    template <bool FAST>
    __device__ __forceinline__ uint4 finish(const Load8<FAST>& in, uint64_t, uint32_t, uint64_t) const
    {
        return in.finish();
    }
};

template <int COL, int ROWS>
struct PieceShared {
    uint4 tile[COL ? ROWS * 16 : 1];
    alignas(16) uint8_t row[ROWS * 4], col[128 * (ROWS / 32)];
};

// The piece at (r0, c0): read, encoded along the rows (row form) and left in
// shared memory for column_codes.
template <int ROW, int COL, int ROWS, bool FAST, class Source>
__device__ __forceinline__ void quantise_piece(const Source& src, uint64_t rows, uint64_t cols, Form row, uint64_t r0,
                                               uint64_t c0, PieceShared<COL, ROWS>& s)
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
        for (int i = 0; i < kFlight; ++i) src.template start<FAST>(in[i], r0 + (t >> 4) + kRowStep * (i0 + i), c);
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
            const uint32_t lr = (t >> 4) + kRowStep * (i0 + i);
            v[i0 + i] = src.template finish<FAST>(in[i], r0 + lr, lr, c);
        }
    }
    if constexpr (COL != 0) {
#pragma unroll
        for (int i = 0; i < kIters; ++i) s.tile[((t >> 4) + kRowStep * i) * 16 + seg] = v[i];
    }
    if constexpr (ROW != 0) {
        const bool block_in = FAST || c / kBlock * kBlock < cols;
        const uint64_t pitch = code_pitch<ROW>(cols);
        uint8_t* p = row.codes + (r0 + (t >> 4)) * pitch + c * Fmt<ROW>::kBits / 8;
#pragma unroll
        for (int i = 0; i < kIters; ++i) {
            const uint32_t lr = (t >> 4) + kRowStep * i;
            uint32_t code[2];
            const uint32_t sc = quantise_quad<ROW>(v[i], code);
            const bool in = FAST || (block_in && r0 + lr < rows);
            if ((t & 3u) == 0) s.row[lr * 4 + (seg >> 2)] = in ? (uint8_t)sc : 0;
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

// After a barrier: the piece's columns, encoded in blocks of 32 rows into the
// column form [cols, rows].  A thread: kCols neighbouring columns of a block of
// 32 rows; a row of shared memory is read without conflicts by the lanes of a
// warp.
template <int COL, int ROWS>
__device__ __forceinline__ void column_codes(uint64_t rows, uint64_t cols, Form col, uint64_t r0, uint64_t c0,
                                             PieceShared<COL, ROWS>& s)
{
    const uint32_t t = threadIdx.x;
    constexpr uint32_t kUnits = 128 * (ROWS / 32);
    constexpr int kCols = kUnits == 2 * kThreadsMx ? 2 : 1;
    const uint32_t u = t % (128 / kCols), rb = t / (128 / kCols);
    if (rb >= ROWS / 32) return;
    uint32_t w[32], m = 0u;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        if constexpr (kCols == 2)
            w[i] = reinterpret_cast<const uint32_t*>(s.tile)[(rb * 32 + i) * 64 + u];
        else
            w[i] = reinterpret_cast<const uint16_t*>(s.tile)[(rb * 32 + i) * 128 + u];
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
        s.col[(kCols * u + h) * (ROWS / 32) + rb] = in ? (uint8_t)(h ? s1 : s0) : 0;
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

// After a barrier: the piece's scale bytes, zeros outside the matrix.
template <int ROW, int COL, int ROWS>
__device__ __forceinline__ void store_scales(uint64_t rows, uint32_t col_tiles, uint32_t ct, Form row, Form col,
                                             uint64_t r0, const PieceShared<COL, ROWS>& s)
{
    const uint32_t t = threadIdx.x;
    const uint64_t rt = r0 / kTileRows;
    const uint32_t lr = (uint32_t)(r0 % kTileRows);
    if constexpr (ROW != 0)
        if (t < ROWS)
            *scale_word(row.scales, rt * col_tiles + ct, lr + t) = reinterpret_cast<const uint32_t*>(s.row)[t];
    if constexpr (COL != 0)
        if (t < 128) {
            // the column form's tiles: its rows are the columns here
            const uint64_t tile = (uint64_t)ct * ez::cdiv(rows, kTileRows) + rt;
            uint32_t* p = scale_word(col.scales, tile, t);
            if constexpr (ROWS == 128)
                *p = reinterpret_cast<const uint32_t*>(s.col)[t];
            else if constexpr (ROWS == 64)
                reinterpret_cast<uint16_t*>(p)[lr / 64] = reinterpret_cast<const uint16_t*>(s.col)[t];
            else
                reinterpret_cast<uint8_t*>(p)[lr / 32] = s.col[t];
        }
}

// Pieces of a scale tile: 128 rows per CTA where there are four tiles per SM, 64
// from two on where columns are encoded too, else 32 (k_mx_quant.cu has the times).
inline uint64_t tiles_per_sm(uint64_t rows, uint64_t cols)
{
    const uint32_t sms = sm_count();
    return ez::cdiv(rows, kTileRows) * ez::cdiv(cols, kTileCols) / (sms ? sms : 1);
}

}  // namespace ezmx
