// k_mx_norm.cu -- the residual's addition and a root-mean-square norm in front of
// a microscaled product, and its backward pass.
//
//   total = bf16(x + residual)           (x itself without a residual)
//   rstd  = 1 / sqrt(mean(total^2) + eps)
//   y     = bf16(total rstd weight), in BF16 and/or as the forms that quantisation
//           of y would give
// Back, with n = total rstd, g = dy weight and c = mean(g n) over a row:
//   dx = rstd (g - n c) + dtotal,        dweight = sum of dy n over the rows.
//
// Squares of BF16 values are exact in FP32; a thread adds up at most 32 of them
// before the sums of a row's threads meet in a tree.
#include "ez_internal.h"
#include "ez_mx_piece.cuh"

namespace ezk {
using namespace ezmx;

namespace {

struct NormArgs {
    Rows x, residual, weight;       // residual.p is null without one
    uint64_t rows;
    uint32_t cols, col_tiles;
    float eps;
    uint16_t *total, *y;            // null: not wanted
    uint64_t ldt, ldy;
    float* rstd;
    Form row;
};

// Sum over the TPR threads of a row, the same bits in all of them; every thread
// of the CTA calls it.  `part` holds a float per warp; two sums in turn use two.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* part)
{
#pragma unroll
    for (int m = 16; m; m >>= 1) v += __shfl_xor_sync(ez::kFull, v, m);
    if constexpr (TPR > 32) {
        constexpr int kWarps = TPR / 32;
        const uint32_t warp = threadIdx.x / 32;
        if (threadIdx.x % 32 == 0) part[warp] = v;
        __syncthreads();
        const float* p = part + warp / kWarps * kWarps;
        float s[kWarps];
#pragma unroll
        for (int i = 0; i < kWarps; ++i) s[i] = p[i];
#pragma unroll
        for (int m = kWarps / 2; m; m >>= 1)
#pragma unroll
            for (int i = 0; i < m; ++i) s[i] += s[i + m];
        v = s[0];
    }
    return v;
}

template <int TPR> constexpr int kThreadsOf = TPR > 256 ? TPR : 256;

}  // namespace

// TPR threads to a row, V groups of eight values to a thread (group v of thread t
// at column 8 (v TPR + t)); total, rstd, y and the row form, all in one read.
template <int TPR, int V, bool LINED, int ROW>
__global__ void __launch_bounds__(kThreadsOf<TPR>) k_rms_rows(const NormArgs a)
{
    constexpr int kRows = kThreadsOf<TPR> / TPR;
    __shared__ float s_part[kThreadsOf<TPR> / 32];
    extern __shared__ uint4 s_stage[];                  // not LINED: kRows rows
    ez::grid_dep_launch();
    const uint32_t t = threadIdx.x % TPR, g = threadIdx.x / TPR;
    const uint64_t row = (uint64_t)blockIdx.x * kRows + g, cols = row < a.rows ? a.cols : 0;
    uint4* const stage = s_stage + g * (V * TPR);
    ez::grid_dep_wait();
    using Load = Load8<LINED, false>;
    uint4 v[V];
    {
        Load x[V], r[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint32_t c = 8 * (i * TPR + t);
            x[i] = r[i] = Load{};
            if (c < cols) {
                x[i].start(a.x, row, c, cols);
                if (a.residual.p) r[i].start(a.residual, row, c, cols);
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            v[i] = x[i].finish();
            if (a.residual.p) {
                float p[8], q[8];
                unpack8(v[i], p);
                unpack8(r[i].finish(), q);
#pragma unroll
                for (int j = 0; j < 8; ++j) p[j] += q[j];
                v[i] = pack8(p);
            }
        }
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float p[8];
        unpack8(v[i], p);
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = __fmaf_rn(p[j], p[j], ss);
        const uint32_t c = 8 * (i * TPR + t);
        if (a.total) {
            if constexpr (LINED) {
                if (c < cols) *reinterpret_cast<uint4*>(a.total + row * a.ldt + c) = v[i];
            } else {
                stage[i * TPR + t] = v[i];
            }
        }
    }
    ss = row_sum<TPR>(ss, s_part);
    const float rstd = 1.f / sqrtf(ss / (float)a.cols + a.eps);
    if (t == 0 && cols) a.rstd[row] = rstd;
    if (!LINED && a.total) {
        __syncthreads();
        if (cols) store_row<TPR>(stage, a.total + row * a.ldt, (uint32_t)cols, t);
        if (a.y) __syncthreads();
    }
    if (ROW == 0 && !a.y) return;
    const uint64_t pitch = ROW ? code_pitch<ROW ? ROW : EZ_MX_E2M1>(a.cols) : 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const uint32_t c = 8 * (i * TPR + t);
        Load8<LINED> wl{};
        if (c < cols) wl.start(a.weight, 0, c, cols);
        float p[8], w[8];
        unpack8(v[i], p);
        unpack8(wl.finish(), w);
#pragma unroll
        for (int j = 0; j < 8; ++j) p[j] = p[j] * rstd * w[j];
        const uint4 y = pack8(p);
        if (a.y) {
            if constexpr (LINED) {
                if (c < cols) *reinterpret_cast<uint4*>(a.y + row * a.ldy + c) = y;
            } else {
                stage[i * TPR + t] = y;
            }
        }
        if constexpr (ROW != 0) {
            const bool in = c / kBlock * kBlock < cols;
            uint32_t code[2];
            uint32_t sc = quantise_quad<ROW>(y, code);
            if (in) {
                uint8_t* at = a.row.codes + row * pitch + (uint64_t)c * Fmt<ROW>::kBits / 8;
                if constexpr (Fmt<ROW>::kBits == 4)
                    *reinterpret_cast<uint32_t*>(at) = code[0];
                else
                    *reinterpret_cast<uint2*>(at) = make_uint2(code[0], code[1]);
            }
            // the scale bytes of a tile's four blocks, 16 lanes, in one word
            sc = in ? sc << (threadIdx.x / 4 % 4 * 8) : 0u;
            sc |= __shfl_xor_sync(ez::kFull, sc, 4);
            sc |= __shfl_xor_sync(ez::kFull, sc, 8);
            if (threadIdx.x % 16 == 0 && c / kTileCols < a.col_tiles)
                *scale_word(a.row.scales, row / kTileRows * a.col_tiles + c / kTileCols, (uint32_t)(row % kTileRows)) = sc;
        }
    }
    if (!LINED && a.y) {
        __syncthreads();
        if (cols) store_row<TPR>(stage, a.y + row * a.ldy, (uint32_t)cols, t);
    }
}

// ---- forms from total and rstd ---------------------------------------------------

namespace {

struct NormSource {
    const Rows& total;
    uint64_t rows, cols;
    const float* rstd;              // of the piece's rows
    float w[8];
    uint16_t* y;
    uint64_t ldy;
    template <bool FAST>
    __device__ __forceinline__ void start(Load8<FAST>& in, uint64_t r, uint64_t c) const
    {
        in.start(total, r, c, r < rows ? cols : 0);
    }
    template <bool FAST>
    __device__ __forceinline__ uint4 finish(const Load8<FAST>& in, uint64_t r, uint32_t lr, uint64_t c) const
    {
        float p[8];
        unpack8(in.finish(), p);
#pragma unroll
        for (int j = 0; j < 8; ++j) p[j] = FAST || r < rows ? p[j] * rstd[lr] * w[j] : 0.f;     // and not -0
        const uint4 v = pack8(p);
        if (y) {
            uint16_t* at = y + r * ldy + c;
            if constexpr (FAST) {
                *reinterpret_cast<uint4*>(at) = v;
            } else if (r < rows) {
                const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (c + j < cols) at[j] = (uint16_t)(x[j / 2] >> (16 * (j & 1)));
            }
        }
        return v;
    }
};

}  // namespace

template <int ROW, int COL, int ROWS>
__global__ void __launch_bounds__(kThreadsMx, 3) k_rms_forms(Rows total, const float* rstd, Rows weight, uint64_t rows,
                                                             uint64_t cols, uint32_t col_tiles, int lines, Form row,
                                                             Form col, uint16_t* y, uint64_t ldy)
{
    __shared__ PieceShared<COL, ROWS> s;
    __shared__ float s_rstd[ROWS];
    ez::grid_dep_launch();
    const uint32_t piece = blockIdx.x / col_tiles, ct = blockIdx.x - piece * col_tiles, t = threadIdx.x;
    const uint64_t r0 = (uint64_t)piece * ROWS, c0 = (uint64_t)ct * kTileCols;
    ez::grid_dep_wait();
    if (t < ROWS) s_rstd[t] = r0 + t < rows ? rstd[r0 + t] : 0.f;
    NormSource src{total, rows, cols, s_rstd, {}, y, ldy};
    Load8<false> w;
    w.start(weight, 0, c0 + 8 * (t & 15u), cols);
    unpack8(w.finish(), src.w);
    __syncthreads();
    if (lines && r0 + ROWS <= rows && c0 + kTileCols <= cols)
        quantise_piece<ROW, COL, ROWS, true>(src, rows, cols, row, r0, c0, s);
    else
        quantise_piece<ROW, COL, ROWS, false>(src, rows, cols, row, r0, c0, s);
    __syncthreads();
    if constexpr (COL != 0) {
        column_codes<COL, ROWS>(rows, cols, col, r0, c0, s);
        __syncthreads();
    }
    store_scales<ROW, COL, ROWS>(rows, col_tiles, ct, row, col, r0, s);
}

// ---- backward ----------------------------------------------------------------------

namespace {

struct NormBackArgs {
    Rows dy, total, weight, dtotal;     // dtotal.p is null without one
    const float* rstd;
    uint64_t rows;
    uint32_t cols;
    uint16_t* dx;
    uint64_t ldx;
    float* partial;                     // [partial rows, cols], or null
};

}  // namespace

// A CTA takes every gridDim-th group of rows; a thread's columns are the same in
// all of them, so that the weight's gradient is summed in its registers.
template <int TPR, int V, bool LINED>
__global__ void __launch_bounds__(kThreadsOf<TPR>) k_rms_back(const NormBackArgs a)
{
    constexpr int kRows = kThreadsOf<TPR> / TPR;
    __shared__ float s_part[2][kThreadsOf<TPR> / 32];
    extern __shared__ uint4 s_stage[];
    ez::grid_dep_launch();
    const uint32_t t = threadIdx.x % TPR, g = threadIdx.x / TPR;
    uint4* const stage = s_stage + g * (V * TPR);
    ez::grid_dep_wait();
    float dw[V][8] = {};
    uint32_t turn = 0;
    for (uint64_t r0 = (uint64_t)blockIdx.x * kRows; r0 < a.rows; r0 += (uint64_t)gridDim.x * kRows, turn ^= 1u) {
        const uint64_t row = r0 + g, cols = row < a.rows ? a.cols : 0;
        using Load = Load8<LINED, false>;
        Load ld[V], lt[V], lg[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint32_t c = 8 * (i * TPR + t);
            ld[i] = lt[i] = lg[i] = Load{};
            if (c < cols) {
                ld[i].start(a.dy, row, c, cols);
                lt[i].start(a.total, row, c, cols);
                if (a.dtotal.p) lg[i].start(a.dtotal, row, c, cols);
            }
        }
        const float rstd = cols ? a.rstd[row] : 0.f;
        uint4 gv[V], nv[V];
        float along = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint32_t c = 8 * (i * TPR + t);
            Load8<LINED> lw{};
            if (c < cols) lw.start(a.weight, 0, c, cols);
            float d[8], n[8], w[8];
            gv[i] = ld[i].finish();
            nv[i] = lt[i].finish();
            unpack8(gv[i], d);
            unpack8(nv[i], n);
            unpack8(lw.finish(), w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float nj = n[j] * rstd;
                along = __fmaf_rn(d[j] * w[j], nj, along);
                dw[i][j] = __fmaf_rn(d[j], nj, dw[i][j]);
            }
        }
        along = row_sum<TPR>(along, s_part[turn]) / (float)a.cols;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint32_t c = 8 * (i * TPR + t);
            Load8<LINED> lw{};
            if (c < cols) lw.start(a.weight, 0, c, cols);
            float d[8], n[8], w[8], e[8];
            unpack8(gv[i], d);
            unpack8(nv[i], n);
            unpack8(lw.finish(), w);
            unpack8(lg[i].finish(), e);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float nj = n[j] * rstd;
                d[j] = __fmaf_rn(rstd, d[j] * w[j] - nj * along, a.dtotal.p ? e[j] : 0.f);
            }
            const uint4 y = pack8(d);
            if constexpr (LINED) {
                if (c < cols) *reinterpret_cast<uint4*>(a.dx + row * a.ldx + c) = y;
            } else {
                stage[i * TPR + t] = y;
            }
        }
        if constexpr (!LINED) {
            __syncthreads();
            if (cols) store_row<TPR>(stage, a.dx + row * a.ldx, (uint32_t)cols, t);
            __syncthreads();
        }
    }
    if (!a.partial) return;
    float* const out = a.partial + ((uint64_t)blockIdx.x * kRows + g) * a.cols;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t c = 8 * (i * TPR + t) + j;
            if (c < a.cols) out[c] = dw[i][j];
        }
}

// The weight's gradient: the partial sums of each column, in a fixed order.
__global__ void __launch_bounds__(256) k_rms_dweight(const float* partial, uint32_t parts, uint32_t cols,
                                                     const float* add, float* dweight)
{
    __shared__ float s_sum[8][33];
    ez::grid_dep_launch();
    const uint32_t lane = threadIdx.x % 32, slice = threadIdx.x / 32, c = blockIdx.x * 32 + lane;
    ez::grid_dep_wait();
    float v = 0.f;
    if (c < cols)
        for (uint32_t p = slice; p < parts; p += 8) v += partial[(uint64_t)p * cols + c];
    s_sum[slice][lane] = v;
    __syncthreads();
    if (slice == 0 && c < cols) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += s_sum[i][lane];
        dweight[c] = add ? s + add[c] : s;
    }
}

// ---- host -----------------------------------------------------------------------------

namespace {

constexpr uint32_t kBackCtas = 304;

// Threads to a row and groups to a thread for a number of columns.
template <template <int, int> class Go, typename... A>
cudaError_t by_width(uint32_t cols, const A&... args)
{
    if (cols <= 256) return Go<32, 1>::run(args...);
    if (cols <= 1024) return Go<128, 1>::run(args...);
    if (cols <= 2048) return Go<128, 2>::run(args...);
    if (cols <= 4096) return Go<256, 2>::run(args...);
    if (cols <= 8192) return Go<256, 4>::run(args...);
    return Go<512, 4>::run(args...);         // up to 16384
}

template <int TPR, int V>
struct GoRows {
    template <bool LINED, int ROW>
    static cudaError_t launch(const NormArgs& a, cudaStream_t s)
    {
        constexpr uint64_t kRows = kThreadsOf<TPR> / TPR;
        auto kernel = k_rms_rows<TPR, V, LINED, ROW>;
        const size_t smem = LINED ? 0 : kRows * V * TPR * 16;
        // with a row form: the scale bytes of the rows of the last tile too
        const uint64_t rows = ROW ? ez::rup(a.rows, kTileRows) : a.rows;
        return ez::launch_dependent(kernel, (unsigned)ez::cdiv(rows, kRows), kThreadsOf<TPR>, smem, s, a);
    }
    static cudaError_t run(const NormArgs& a, const int& fmt, const bool& lines, const cudaStream_t& s)
    {
        switch (fmt) {
            case EZ_MX_E2M1: return lines ? launch<true, EZ_MX_E2M1>(a, s) : launch<false, EZ_MX_E2M1>(a, s);
            case EZ_MX_E4M3: return lines ? launch<true, EZ_MX_E4M3>(a, s) : launch<false, EZ_MX_E4M3>(a, s);
            case EZ_MX_E5M2: return lines ? launch<true, EZ_MX_E5M2>(a, s) : launch<false, EZ_MX_E5M2>(a, s);
        }
        return lines ? launch<true, 0>(a, s) : launch<false, 0>(a, s);
    }
};

template <int TPR, int V>
struct GoBack {
    template <bool LINED>
    static cudaError_t launch(const NormBackArgs& a, uint32_t& parts, cudaStream_t s)
    {
        constexpr uint64_t kRows = kThreadsOf<TPR> / TPR;
        const unsigned grid = (unsigned)ez::umin64(ez::cdiv(a.rows, kRows), kBackCtas);
        parts = grid * (uint32_t)kRows;
        return ez::launch_dependent(k_rms_back<TPR, V, LINED>, grid, kThreadsOf<TPR>, LINED ? 0 : kRows * V * TPR * 16, s,
                                    a);
    }
    static cudaError_t run(const NormBackArgs& a, const bool& lines, uint32_t* const& parts, const cudaStream_t& s)
    {
        return lines ? launch<true>(a, *parts, s) : launch<false>(a, *parts, s);
    }
};

template <int ROW, int COL, int ROWS>
cudaError_t forms_rows(const Rows& total, const NormArgs& a, Form row, Form col, cudaStream_t s)
{
    const uint64_t pieces = ez::cdiv(a.rows, kTileRows) * (kTileRows / ROWS);
    const int lines = lined(total.p, a.rows, total.ld) && (!a.y || lined(a.y, a.rows, a.ldy));
    return ez::launch_dependent(k_rms_forms<ROW, COL, ROWS>, (unsigned)(pieces * a.col_tiles), kThreadsMx, 0, s, total,
                                (const float*)a.rstd, a.weight, a.rows, (uint64_t)a.cols, a.col_tiles, lines, row, col,
                                a.y, a.ldy);
}
template <int ROW, int COL>
cudaError_t forms(const Rows& total, const NormArgs& a, Form row, Form col, cudaStream_t s)
{
    const uint64_t per_sm = tiles_per_sm(a.rows, a.cols);
    if (per_sm >= 4) return forms_rows<ROW, COL, 128>(total, a, row, col, s);
    if (per_sm >= 2) return forms_rows<ROW, COL, 64>(total, a, row, col, s);
    return forms_rows<ROW, COL, 32>(total, a, row, col, s);
}
template <int ROW>
cudaError_t forms_col(int col_fmt, const Rows& total, const NormArgs& a, Form row, Form col, cudaStream_t s)
{
    switch (col_fmt) {
        case EZ_MX_E2M1: return forms<ROW, EZ_MX_E2M1>(total, a, row, col, s);
        case EZ_MX_E4M3: return forms<ROW, EZ_MX_E4M3>(total, a, row, col, s);
    }
    return forms<ROW, EZ_MX_E5M2>(total, a, row, col, s);
}

// Rows of partial sums: groups of rows in all CTAs.
uint64_t part_rows(uint64_t rows, uint64_t cols)
{
    const uint64_t per = cols <= 256 ? 8 : cols <= 2048 ? 2 : 1;
    return ez::umin64(ez::cdiv(rows, per), kBackCtas) * per;
}

}  // namespace

cudaError_t launch_mx_rms_norm(const uint16_t* x, uint64_t ldx, const uint16_t* residual, uint64_t ldr, uint64_t rows,
                               uint32_t cols, const uint16_t* weight, float eps, uint16_t* total, uint64_t ldt,
                               float* rstd, uint16_t* y, uint64_t ldy, int row_fmt, uint8_t* row_codes,
                               uint8_t* row_scales, int col_fmt, uint8_t* col_codes, uint8_t* col_scales,
                               cudaStream_t s)
{
    NormArgs a{};
    a.x = make_rows(x, rows, cols, ldx);
    if (residual) a.residual = make_rows(residual, rows, cols, ldr);
    a.weight = make_rows(weight, 1, cols, cols);
    a.rows = rows;
    a.cols = cols;
    a.col_tiles = (uint32_t)ez::cdiv(cols, kTileCols);
    a.eps = eps;
    a.total = total;
    a.ldt = ldt;
    a.rstd = rstd;
    a.y = y;
    a.ldy = ldy;
    const Form row{row_codes, row_scales}, col{col_codes, col_scales};
    a.row = row;
    const bool lines = cols % 8 == 0 && lined(x, rows, ldx) && (!residual || lined(residual, rows, ldr)) &&
                       lined(weight, 1, cols) && (!total || lined(total, rows, ldt)) && (!y || lined(y, rows, ldy));
    if (!col_fmt) return by_width<GoRows>(cols, a, row_fmt, lines, s);
    NormArgs first = a;
    first.y = nullptr;
    const cudaError_t e = by_width<GoRows>(cols, first, 0, lines, s);
    if (e != cudaSuccess) return e;
    const Rows sum = total ? make_rows(total, rows, cols, ldt) : a.x;
    switch (row_fmt) {
        case EZ_MX_E2M1: return forms_col<EZ_MX_E2M1>(col_fmt, sum, a, row, col, s);
        case EZ_MX_E4M3: return forms_col<EZ_MX_E4M3>(col_fmt, sum, a, row, col, s);
        case EZ_MX_E5M2: return forms_col<EZ_MX_E5M2>(col_fmt, sum, a, row, col, s);
    }
    return forms_col<0>(col_fmt, sum, a, row, col, s);
}

uint64_t mx_rms_norm_ws(uint64_t rows, uint64_t cols) { return part_rows(rows, cols) * cols * 4; }

cudaError_t launch_mx_rms_norm_backward(const uint16_t* dy, uint64_t lddy, const uint16_t* total, uint64_t ldt,
                                        const float* rstd, const uint16_t* weight, const uint16_t* dtotal,
                                        uint64_t lddt, uint64_t rows, uint32_t cols, uint16_t* dx, uint64_t ldx,
                                        const float* add, float* dweight, float* ws, cudaStream_t s)
{
    NormBackArgs a{};
    a.dy = make_rows(dy, rows, cols, lddy);
    a.total = make_rows(total, rows, cols, ldt);
    a.weight = make_rows(weight, 1, cols, cols);
    if (dtotal) a.dtotal = make_rows(dtotal, rows, cols, lddt);
    a.rstd = rstd;
    a.rows = rows;
    a.cols = cols;
    a.dx = dx;
    a.ldx = ldx;
    a.partial = dweight ? ws : nullptr;
    const bool lines = cols % 8 == 0 && lined(dy, rows, lddy) && lined(total, rows, ldt) && lined(weight, 1, cols) &&
                       (!dtotal || lined(dtotal, rows, lddt)) && lined(dx, rows, ldx);
    uint32_t parts = 0;
    if (rows) {
        const cudaError_t e = by_width<GoBack>(cols, a, lines, &parts, s);
        if (e != cudaSuccess) return e;
    }
    if (!dweight) return cudaSuccess;
    return ez::launch_dependent(k_rms_dweight, (unsigned)ez::cdiv(cols, 32), 256, 0, s, (const float*)ws, parts, cols,
                                add, dweight);
}

}  // namespace ezk
