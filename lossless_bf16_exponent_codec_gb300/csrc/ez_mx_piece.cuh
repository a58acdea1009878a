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
    uint4 tile[COL ? ROWS * 16 : 1];        // granule g of row r at tile_at(r, g)
    alignas(16) uint8_t row[COL ? 16 : ROWS * 4], col[128 * (ROWS / 32)];
};
// Lanes meet all banks with eight consecutive granules of a row, with granule j of the
// four blocks of two rows, and with the words of two granules in four blocks of 32 rows.
__device__ __forceinline__ uint32_t tile_at(uint32_t r, uint32_t g)
{
    return r * 16 + (g ^ (g >> 3) ^ (((r >> 5) ^ (r & 1u)) & 3u) << 1);
}

// The piece at (r0, c0), read.  Without a column form it is encoded along the rows on the
// spot, 8 values to a lane; with one it goes to shared memory, for row_codes and
// column_codes.
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
        for (int i = 0; i < kIters; ++i) s.tile[tile_at((t >> 4) + kRowStep * i, seg)] = v[i];
    } else {
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

// After a barrier: the piece's rows, encoded into the row form with their scale bytes, a
// block of 32 values by each lane.  Against 8 values to a lane and a block to four, whose
// scale each of them works out, that is a tenth of the instructions less.  Steps, 131072
// tokens' rows of 2048 to 4-bit rows and 8-bit columns, and 16384 x 8192: 192 and 83 us,
// with this 184 and 81, with products of halves 181, with whole lines of column codes 167
// and 77, with the clearing of poisoned blocks behind a vote 166 and 75.
template <int ROW, int COL, int ROWS>
__device__ __forceinline__ void row_codes(uint64_t rows, uint64_t cols, uint32_t col_tiles, uint32_t ct, Form row, uint64_t r0,
                                          uint64_t c0, const PieceShared<COL, ROWS>& s)
{
    constexpr uint32_t kStep = kThreadsMx / 4;
    const uint64_t pitch = code_pitch<ROW>(cols);
    const uint32_t b = threadIdx.x % 4;
    const bool block_in = c0 + b * kBlock < cols;
    uint8_t* to = row.codes + (r0 + threadIdx.x / 4) * pitch + (c0 + b * kBlock) * Fmt<ROW>::kBits / 8;
#pragma unroll
    for (uint32_t lr = threadIdx.x / 4; lr < ROWS; lr += kStep, to += kStep * pitch) {
        const uint32_t at = tile_at(lr, 4 * b);
        uint32_t y[16], m = 0u;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint4 v = s.tile[at ^ j];                 // tile_at(lr, 4 * b + j)
            y[4 * j] = v.x;
            y[4 * j + 1] = v.y;
            y[4 * j + 2] = v.z;
            y[4 * j + 3] = v.w;
            m = mag_max(mag_max(m, v.x), mag_max(mag_max(v.y, v.z), v.w));
        }
        const bool in = block_in && r0 + lr < rows;
        uint32_t sc = scale_byte<ROW>(mag_max(m, m >> 16) & 0x7FFFu), code[Fmt<ROW>::kBits];
        encode_block<ROW>(y, sc, code);
        if (in) store_codes32<ROW>(code, to);
        sc = in ? sc << (8 * b) : 0u;
        sc |= __shfl_xor_sync(ez::kFull, sc, 1);
        sc |= __shfl_xor_sync(ez::kFull, sc, 2);
        if (b == 0)
            *scale_word(row.scales, r0 / kTileRows * col_tiles + ct, (uint32_t)(r0 % kTileRows) + lr) = sc;
    }
}

// After a barrier: the piece's columns, encoded in blocks of 32 rows into the
// column form [cols, rows].  A thread: kCols neighbouring columns of a block of
// 32 rows; the blocks of a column go to neighbouring lanes, which store a whole line of
// 128 8-bit codes together.
template <int COL, int ROWS>
__device__ __forceinline__ void column_codes(uint64_t rows, uint64_t cols, Form col, uint64_t r0, uint64_t c0,
                                             PieceShared<COL, ROWS>& s)
{
    const uint32_t t = threadIdx.x;
    constexpr uint32_t kUnits = 128 * (ROWS / 32);
    constexpr int kCols = kUnits == 2 * kThreadsMx ? 2 : 1;
    const uint32_t u = t / (ROWS / 32), rb = t % (ROWS / 32);
    if (u >= 128 / kCols) return;
    constexpr uint32_t kPer = 8 / kCols;                  // of them to a granule
    const uint32_t even = tile_at(rb * 32, u / kPer) * kPer + u % kPer;
    const uint32_t odd = tile_at(rb * 32 + 1, u / kPer) * kPer + u % kPer;
    uint32_t w[32], most[4] = {};
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const uint32_t at = (i & ~1) * 16 * kPer + (i & 1 ? odd : even);
        if constexpr (kCols == 2)
            w[i] = reinterpret_cast<const uint32_t*>(s.tile)[at];
        else
            w[i] = reinterpret_cast<const uint16_t*>(s.tile)[at];
        most[i % 4] = mag_max(most[i % 4], w[i]);
    }
    const uint32_t m = mag_max(mag_max(most[0], most[1]), mag_max(most[2], most[3]));
    const uint64_t rblock = r0 + rb * 32;
    const uint32_t s0 = scale_byte<COL>(m & 0x7FFFu), s1 = scale_byte<COL>((m >> 16) & 0x7FFFu);
    uint32_t inv = (inv_scale(s0) & 0xFFFFu) | (inv_scale(s1) & 0xFFFF0000u);
    if (__any_sync(ez::kFull, s0 == 255u || s1 == 255u)) {
        const uint32_t keep = (s0 == 255u ? 0u : 0xFFFFu) | (s1 == 255u ? 0u : 0xFFFF0000u);
        inv &= keep;
#pragma unroll
        for (int i = 0; i < 32; ++i) w[i] &= keep;
    }
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
            for (int i = 0; i < 8; ++i) {
                float lo, hi;
                products(w[8 * g + i], inv, lo, hi);
                f[i] = h ? hi : lo;
            }
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

// After a barrier: the piece's scale bytes, zeros outside the matrix (the rows' only without
// a column form: else row_codes has stored them).
template <int ROW, int COL, int ROWS>
__device__ __forceinline__ void store_scales(uint64_t rows, uint32_t col_tiles, uint32_t ct, Form row, Form col,
                                             uint64_t r0, const PieceShared<COL, ROWS>& s)
{
    const uint32_t t = threadIdx.x;
    const uint64_t rt = r0 / kTileRows;
    const uint32_t lr = (uint32_t)(r0 % kTileRows);
    if constexpr (ROW != 0 && COL == 0)
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

// All of the above: a piece from its source to its forms.
template <int ROW, int COL, int ROWS, class Source>
__device__ __forceinline__ void encode_piece(const Source& src, bool fast, uint64_t rows, uint64_t cols, uint32_t col_tiles,
                                             uint32_t ct, Form row, Form col, uint64_t r0, PieceShared<COL, ROWS>& s)
{
    const uint64_t c0 = (uint64_t)ct * kTileCols;
    if (fast)
        quantise_piece<ROW, COL, ROWS, true>(src, rows, cols, row, r0, c0, s);
    else
        quantise_piece<ROW, COL, ROWS, false>(src, rows, cols, row, r0, c0, s);
    __syncthreads();
    if constexpr (COL != 0) {
        if constexpr (ROW != 0) row_codes<ROW, COL, ROWS>(rows, cols, col_tiles, ct, row, r0, c0, s);
        column_codes<COL, ROWS>(rows, cols, col, r0, c0, s);
        __syncthreads();
    }
    store_scales<ROW, COL, ROWS>(rows, col_tiles, ct, row, col, r0, s);
}

// Pieces of a scale tile: 128 rows per CTA where there are four tiles per SM, 64
// from two on where columns are encoded too, else 32 (k_mx_quant.cu has the times).
inline uint64_t tiles_per_sm(uint64_t rows, uint64_t cols)
{
    const uint32_t sms = sm_count();
    return ez::cdiv(rows, kTileRows) * ez::cdiv(cols, kTileCols) / (sms ? sms : 1);
}

}  // namespace ezmx
