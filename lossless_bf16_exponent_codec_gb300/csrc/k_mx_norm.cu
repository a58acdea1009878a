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
// Squares of BF16 values are exact in FP32, and up to 32 of them are added up there;
// from there on a row's sum is a pair of FP32 numbers, so that rstd is the FP32 number
// nearest to the exact one but for a few in a thousand rows.  total weight is exact, and
// its product with rstd is rounded to FP32 and to BF16: a y next to a border of BF16 is
// next to a border of a 4-bit code often enough, in 10^8 values, for a sum in plain FP32
// and another rounded product to give other codes than 64-bit arithmetic does.
#include "ez_internal.h"
#include "ez_mx.cuh"
#include "ez_tc.cuh"

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

// An unevaluated sum.
struct Two {
    float hi, lo;
};
__device__ __forceinline__ Two add2(const Two& a, const Two& b)
{
    const float s = a.hi + b.hi, t = s - a.hi;
    return {s, ((a.hi - (s - t)) + (b.hi - t)) + (a.lo + b.lo)};
}
// Eight squares.
__device__ __forceinline__ float squares(const uint4& v)
{
    float p[8], s = 0.f;
    unpack8(v, p);
#pragma unroll
    for (int j = 0; j < 8; ++j) s = __fmaf_rn(p[j], p[j], s);
    return s;
}
// Sum over a warp, the same bits in all lanes: a sum and its error do not depend on
// the order of the two.
__device__ __forceinline__ Two warp_sum(Two v)
{
#pragma unroll
    for (int m = 16; m; m >>= 1) {
        v = add2(v, Two{__shfl_xor_sync(ez::kFull, v.hi, m), __shfl_xor_sync(ez::kFull, v.lo, m)});
    }
    return v;
}

// 1 / sqrt(sum / cols + eps): a Newton step from rsqrtf with the mean and the
// residual in pairs.  0 and infinities stay what rsqrtf says.
__device__ __forceinline__ float inverse_root(const Two& sum, float cols, float eps)
{
    const float q = sum.hi / cols;
    const Two mean{q, (__fmaf_rn(-q, cols, sum.hi) + sum.lo) / cols};
    Two m = add2(mean, Two{eps, 0.f});
    const float h = isinf(q) ? q : m.hi + m.lo;     // an infinity's residual is NaN
    const float r = rsqrtf(h);
    if (!(r > 0.f) || isinf(r)) return r;
    m.lo += m.hi - h;
    const float a = r * h, a_lo = __fmaf_rn(r, h, -a);                      // r m
    const float e = __fmaf_rn(-a, r, 1.f) - __fmaf_rn(m.lo, r, a_lo) * r;   // 1 - r^2 m
    return __fmaf_rn(0.5f * r, __fmaf_rn(0.75f * e, e, e), r);
}
// total weight, exact, times rstd.
__device__ __forceinline__ uint4 normed(const uint4& total, const uint4& weight, float rstd)
{
    float p[8], w[8];
    unpack8(total, p);
    unpack8(weight, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) p[j] = p[j] * w[j] * rstd;
    return pack8(p);
}

// Sum over the TPR threads of a row, the same bits in all of them; every thread
// of the CTA calls it.  `part` holds a pair per warp.
template <int TPR>
__device__ __forceinline__ Two row_sum(Two v, Two* part)
{
    v = warp_sum(v);
    if constexpr (TPR > 32) {
        constexpr int kWarps = TPR / 32;
        const uint32_t warp = threadIdx.x / 32;
        if (threadIdx.x % 32 == 0) part[warp] = v;
        __syncthreads();
        const Two* p = part + warp / kWarps * kWarps;
        v = p[0];
#pragma unroll
        for (int i = 1; i < kWarps; ++i) v = add2(v, p[i]);
    }
    return v;
}
// The same in plain FP32; two sums in turn use two `part`s.
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

// The sum of a value pair and its residual, in BF16.
__device__ __forceinline__ uint4 add8(const uint4& x, const uint4& r)
{
    float p[8], q[8];
    unpack8(x, p);
    unpack8(r, q);
#pragma unroll
    for (int j = 0; j < 8; ++j) p[j] += q[j];
    return pack8(p);
}

// A quad's codes of eight y each from column c on, and the scale bytes of a tile's
// row in one word; called by whole warps.
template <int ROW>
__device__ __forceinline__ void store_codes(const Form& form, const uint4& y, uint64_t row, uint32_t c, uint64_t cols,
                                            uint64_t pitch, uint32_t col_tiles)
{
    const bool in = c / kBlock * kBlock < cols;
    uint32_t code[2];
    uint32_t sc = quantise_quad<ROW>(y, code);
    if (in) {
        uint8_t* at = form.codes + row * pitch + (uint64_t)c * Fmt<ROW>::kBits / 8;
        if constexpr (Fmt<ROW>::kBits == 4)
            *reinterpret_cast<uint32_t*>(at) = code[0];
        else
            *reinterpret_cast<uint2*>(at) = make_uint2(code[0], code[1]);
    }
    sc = in ? sc << (threadIdx.x / 4 % 4 * 8) : 0u;     // four blocks, 16 lanes
    sc |= __shfl_xor_sync(ez::kFull, sc, 4);
    sc |= __shfl_xor_sync(ez::kFull, sc, 8);
    if (threadIdx.x % 16 == 0 && c / kTileCols < col_tiles)
        *scale_word(form.scales, row / kTileRows * col_tiles + c / kTileCols, (uint32_t)(row % kTileRows)) = sc;
}

template <int TPR> constexpr int kThreadsOf = TPR > 256 ? TPR : 256;

}  // namespace

// TPR threads to a row, V groups of eight values to a thread (group v of thread t
// at column 8 (v TPR + t)); total, rstd, y and the row form, all in one read.
template <int TPR, int V, bool LINED, int ROW>
__global__ void __launch_bounds__(kThreadsOf<TPR>) k_rms_rows(const NormArgs a)
{
    constexpr int kRows = kThreadsOf<TPR> / TPR;
    __shared__ Two s_part[kThreadsOf<TPR> / 32];
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
            if (a.residual.p) v[i] = add8(v[i], r[i].finish());
        }
    }
    Two sum{0.f, 0.f};
#pragma unroll
    for (int i = 0; i < V; ++i) {
        sum = add2(sum, Two{squares(v[i]), 0.f});
        const uint32_t c = 8 * (i * TPR + t);
        if (a.total) {
            if constexpr (LINED) {
                if (c < cols) *reinterpret_cast<uint4*>(a.total + row * a.ldt + c) = v[i];
            } else {
                stage[i * TPR + t] = v[i];
            }
        }
    }
    const float rstd = inverse_root(row_sum<TPR>(sum, s_part), (float)a.cols, a.eps);
    if (t == 0 && cols) a.rstd[row] = rstd;
    if (!LINED && a.total) {
        __syncthreads();
        if (cols) store_row<TPR>([=](uint32_t i) { return stage[i]; }, a.total + row * a.ldt, (uint32_t)cols, t);
        if (a.y) __syncthreads();
    }
    if (ROW == 0 && !a.y) return;
    const uint64_t pitch = ROW ? code_pitch<ROW ? ROW : EZ_MX_E2M1>(a.cols) : 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const uint32_t c = 8 * (i * TPR + t);
        Load8<LINED> w{};
        if (c < cols) w.start(a.weight, 0, c, cols);
        const uint4 y = normed(v[i], w.finish(), rstd);
        if (a.y) {
            if constexpr (LINED) {
                if (c < cols) *reinterpret_cast<uint4*>(a.y + row * a.ldy + c) = y;
            } else {
                stage[i * TPR + t] = y;
            }
        }
        if constexpr (ROW != 0) store_codes<ROW>(a.row, y, row, c, cols, pitch, a.col_tiles);
    }
    if (!LINED && a.y) {
        __syncthreads();
        if (cols) store_row<TPR>([=](uint32_t i) { return stage[i]; }, a.y + row * a.ldy, (uint32_t)cols, t);
    }
}

// ---- with a column form ------------------------------------------------------------

namespace {

constexpr int kBandRows = 32, kBandThreads = 256;

// The codes of a block of 32 values (BF16 words) with scale byte s.
template <int ROW>
__device__ __forceinline__ void store_block(uint32_t* y, uint32_t s, uint8_t* to)
{
    constexpr int kWords = Fmt<ROW>::kBits;
    if (s == 255u)
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] = 0u;
    const uint32_t inv = s == 255u ? 0u : inv_scale(s);
    uint32_t code[kWords];
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        float f[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t v = mul2(y[4 * g + i], inv);
            f[2 * i] = lo_f(v);
            f[2 * i + 1] = hi_f(v);
        }
        encode8<ROW>(f, code + g * (kWords / 4));
    }
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i)
        reinterpret_cast<uint4*>(to)[i] = make_uint4(code[4 * i], code[4 * i + 1], code[4 * i + 2], code[4 * i + 3]);
}

// Blocks of 32 rows of columns c and c + 1 (the halves of w, magnitudes' maxima m)
// into the column form: codes, and the scale byte of each.
template <int COL>
__device__ __forceinline__ void column_pair(uint32_t* w, uint32_t m, uint32_t c, uint64_t cols, bool some, uint64_t rows,
                                            uint64_t r0, uint64_t row_tiles, const Form& col)
{
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
    for (int h = 0; h < 2; ++h) {
        const uint32_t cc = c + h;
        const bool in = cc < cols && some;
        const uint64_t tile = cc / kTileCols * row_tiles + r0 / kTileRows;
        reinterpret_cast<uint8_t*>(scale_word(col.scales, tile, cc % kTileCols))[r0 % kTileRows / 32] =
            in ? (uint8_t)(h ? s1 : s0) : 0;
        constexpr int kWords = Fmt<COL>::kBits;     // 32 codes
        uint32_t code[kWords];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = h ? hi_f(w[8 * g + i]) : lo_f(w[8 * g + i]);
            encode8<COL>(f, code + g * (kWords / 4));
        }
        if (!in) continue;
        uint8_t* p = col.codes + cc * code_pitch<COL>(rows) + r0 * Fmt<COL>::kBits / 8;
        if (kWords == 8 && (reinterpret_cast<uintptr_t>(col.codes) & 31u) == 0) {
            st_v8(p, code);          // one whole sector
        } else {
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i)
                reinterpret_cast<uint4*>(p)[i] = make_uint4(code[4 * i], code[4 * i + 1], code[4 * i + 2], code[4 * i + 3]);
        }
    }
}

}  // namespace

// 32 rows (a block of the column form) by a cluster of CTAs, each on `width` of
// the columns, which it keeps in shared memory: total is read once, the sums of
// the squares meet through distributed shared memory, y takes total's place there
// and is encoded along the rows on the way, a block of 32 values by each lane, and along
// the columns at the end.  A warp takes a row at a time, so that rows at any alignment
// are stored from shared memory by the warp that wrote them.
//
// Granule g of a row (8 values) lies at g ^ (g / 8 % 4): eight lanes then meet all banks
// both with consecutive granules and with every fourth one.
__device__ __forceinline__ uint32_t band_at(uint32_t g) { return g ^ (g >> 3 & 3u); }

// Phase 1 of a row: total in shared memory (and out), the sum of its squares.  FULL: all
// of the CTA's columns are there, in groups of 1024.
template <bool LINED, bool FULL>
__device__ __forceinline__ Two band_total(const NormArgs& a, uint64_t row, uint32_t c0, uint32_t cols, uint32_t pitch8, uint4* q)
{
    constexpr int kFlight = LINED ? 4 : 2;
    const uint32_t lane = threadIdx.x % 32;
    Two sum{0.f, 0.f};
    for (uint32_t g0 = lane; g0 < pitch8; g0 += 32 * kFlight) {
        Load8<LINED, false> x[kFlight], r[kFlight];
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
            const uint32_t c = 8 * (g0 + 32 * i);
            if constexpr (!FULL) x[i] = r[i] = Load8<LINED, false>{};
            if (FULL || c < cols) {
                x[i].start(a.x, row, c0 + c, a.cols);
                if (a.residual.p) r[i].start(a.residual, row, c0 + c, a.cols);
            }
        }
        float part = 0.f;
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
            const uint32_t g = g0 + 32 * i;
            if (!FULL && g >= pitch8) break;
            uint4 v = x[i].finish();
            if (a.residual.p) v = add8(v, r[i].finish());
            q[band_at(g)] = v;
            part += squares(v);
            if (LINED && a.total && (FULL || 8 * g < cols)) *reinterpret_cast<uint4*>(a.total + row * a.ldt + c0 + 8 * g) = v;
        }
        sum = add2(sum, Two{part, 0.f});
    }
    return sum;
}

template <int ROW, int COL, bool LINED>
__global__ void __launch_bounds__(kBandThreads, 3) k_rms_band(const NormArgs a, const Form col, uint32_t width)
{
    extern __shared__ uint4 s_band[];                   // kBandRows rows of width / 8
    __shared__ Two s_part[8][kBandRows];                // of each CTA of the cluster
    __shared__ float s_rstd[kBandRows];
    ez::grid_dep_launch();
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32, pitch8 = width / 8;
    uint32_t n;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
    const uint32_t rank = eztc::cluster_rank(), c0 = rank * width;
    const uint64_t r0 = (uint64_t)(blockIdx.x / n) * kBandRows;
    const uint32_t here = min(width, a.cols > c0 ? a.cols - c0 : 0u);      // columns of this CTA
    const bool full = LINED && here == width && width % 1024 == 0 && r0 + kBandRows <= a.rows;
    eztc::cluster_arrive();                             // this CTA runs: its memory may be written
    ez::grid_dep_wait();
    for (uint32_t lr = warp; lr < kBandRows; lr += kBandThreads / 32) {
        const uint64_t row = r0 + lr;
        const uint32_t cols = row < a.rows ? here : 0;
        uint4* const q = s_band + lr * pitch8;
        Two sum = full ? band_total<LINED, LINED>(a, row, c0, cols, pitch8, q)
                       : band_total<LINED, false>(a, row, c0, cols, pitch8, q);
        sum = warp_sum(sum);
        if (lane == 0) s_part[rank][lr] = sum;
        if (!LINED && a.total) {
            __syncwarp();
            store_row<32>([=](uint32_t g) { return q[band_at(g)]; }, a.total + row * a.ldt + c0, cols, lane);
        }
    }
    eztc::cluster_wait();
    __syncthreads();
    if (n > 1) {
        // every CTA's sums to all others
        for (uint32_t i = threadIdx.x; i < n * kBandRows; i += kBandThreads) {
            const uint32_t to = i / kBandRows, lr = i % kBandRows;
            if (to == rank) continue;
            const Two v = s_part[rank][lr];
            eztc::peer_store64(eztc::peer_addr(eztc::smem_u32(&s_part[rank][lr]), to),
                               (uint64_t)__float_as_uint(v.lo) << 32 | __float_as_uint(v.hi));
        }
        eztc::cluster_sync();
    }
    if (threadIdx.x < kBandRows) {
        Two sum = s_part[0][threadIdx.x];
        for (uint32_t i = 1; i < n; ++i) sum = add2(sum, s_part[i][threadIdx.x]);
        const float rstd = inverse_root(sum, (float)a.cols, a.eps);
        s_rstd[threadIdx.x] = rstd;
        if (rank == 0 && r0 + threadIdx.x < a.rows) a.rstd[r0 + threadIdx.x] = rstd;
    }
    __syncthreads();
    const uint64_t row_pitch = ROW ? code_pitch<ROW ? ROW : EZ_MX_E2M1>(a.cols) : 0;
    for (uint32_t b0 = 0; b0 < width; b0 += 1024) {     // a lane's block of 32 columns
        const uint32_t b = b0 + 32 * lane;
        const bool mine = b < width, in = b < here;
        uint4 w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            w[j] = make_uint4(0u, 0u, 0u, 0u);
            if (b + 8 * j < here) {
                Load8<false> l;
                l.start(a.weight, 0, c0 + b + 8 * j, a.cols);
                w[j] = l.finish();
            }
        }
        for (uint32_t lr = warp; lr < kBandRows; lr += kBandThreads / 32) {
            const uint64_t row = r0 + lr;
            uint4* const q = s_band + lr * pitch8;
            const float rstd = s_rstd[lr];
            const bool some = mine && row < a.rows;     // a row that is none stays zero, and not -0
            uint32_t y[16], m = 0u;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                if (some) v = normed(q[band_at(b / 8 + j)], w[j], rstd);
                if (mine) q[band_at(b / 8 + j)] = v;
                y[4 * j] = v.x;
                y[4 * j + 1] = v.y;
                y[4 * j + 2] = v.z;
                y[4 * j + 3] = v.w;
                m = mag_max(mag_max(m, v.x), mag_max(mag_max(v.y, v.z), v.w));
            }
            if constexpr (ROW != 0) {
                uint32_t s = 0;
                if (some && in) {
                    s = scale_byte<ROW>(mag_max(m, m >> 16) & 0x7FFFu);
                    store_block<ROW>(y, s, a.row.codes + row * row_pitch + (uint64_t)(c0 + b) * Fmt<ROW>::kBits / 8);
                }
                s <<= lane % 4 * 8;                     // a tile's four blocks in one word
                s |= __shfl_xor_sync(ez::kFull, s, 1);
                s |= __shfl_xor_sync(ez::kFull, s, 2);
                if (lane % 4 == 0 && mine && (c0 + b) / kTileCols < a.col_tiles)
                    *scale_word(a.row.scales, row / kTileRows * a.col_tiles + (c0 + b) / kTileCols,
                                (uint32_t)(row % kTileRows)) = s;
            }
        }
    }
    __syncthreads();
    if (a.y)
        for (uint32_t lr = warp; lr < kBandRows && r0 + lr < a.rows; lr += kBandThreads / 32) {
            const uint4* const q = s_band + lr * pitch8;
            store_row<32>([=](uint32_t g) { return q[band_at(g)]; }, a.y + (r0 + lr) * a.ldy + c0, here, lane);
        }
    // two neighbouring columns to a thread
    const uint64_t row_tiles = ez::cdiv(a.rows, kTileRows);
    const bool some = r0 < a.rows;                      // else only scale bytes of the last tile
    for (uint32_t u = threadIdx.x; u < width / 2; u += kBandThreads) {
        const uint32_t c = c0 + 2 * u, at = band_at(u / 4) * 4 + u % 4;
        if (c / kTileCols >= a.col_tiles) break;
        const uint32_t* const p = reinterpret_cast<const uint32_t*>(s_band) + at;
        uint32_t w[kBandRows], m = 0u;
#pragma unroll
        for (int i = 0; i < kBandRows; ++i) {
            w[i] = p[i * (width / 2)];
            m = mag_max(m, w[i]);
        }
        column_pair<COL>(w, m, c, a.cols, some, a.rows, r0, row_tiles, col);
    }
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
            if (cols) store_row<TPR>([=](uint32_t i) { return stage[i]; }, a.dx + row * a.ldx, (uint32_t)cols, t);
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
constexpr int kSlices = 32;
__global__ void __launch_bounds__(32 * kSlices) k_rms_dweight(const float* partial, uint32_t parts, uint32_t cols,
                                                              const float* add, float* dweight)
{
    __shared__ float s_sum[kSlices][33];
    ez::grid_dep_launch();
    const uint32_t lane = threadIdx.x % 32, slice = threadIdx.x / 32, c = blockIdx.x * 32 + lane;
    ez::grid_dep_wait();
    float v = 0.f;
    if (c < cols)
#pragma unroll 8
        for (uint32_t p = slice; p < parts; p += kSlices) v += partial[(uint64_t)p * cols + c];
    s_sum[slice][lane] = v;
    __syncthreads();
    if (slice == 0 && c < cols) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < kSlices; ++i) s += s_sum[i][lane];
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

// Columns of a CTA: 1024 (64 KB, three CTAs to an SM), or what a cluster of 8 needs.
template <int ROW, int COL, bool LINED>
cudaError_t band(const NormArgs& a, Form col, cudaStream_t s)
{
    const uint32_t most = a.cols <= 8192 ? 1024 : 2048, n = (uint32_t)ez::cdiv(a.cols, most);
    const uint32_t width = (uint32_t)ez::rup(ez::cdiv(a.cols, n), kTileCols);
    auto kernel = k_rms_band<ROW, COL, LINED>;
    static ez::PerDeviceAttr raised;
    const cudaError_t e = ez::max_dyn_smem_per_device(raised, kernel, kBandRows * 2048 * 2);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2] = {};
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = n;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    // every band of the last scale tile, to clear its bytes
    cfg.gridDim = dim3((unsigned)(ez::rup(a.rows, kTileRows) / kBandRows * n));
    cfg.blockDim = dim3(kBandThreads);
    cfg.dynamicSmemBytes = kBandRows * width * 2;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, a, col, width);
}
template <int ROW, int COL>
cudaError_t band(const NormArgs& a, bool lines, Form col, cudaStream_t s)
{
    return lines ? band<ROW, COL, true>(a, col, s) : band<ROW, COL, false>(a, col, s);
}
template <int ROW>
cudaError_t band(int col_fmt, const NormArgs& a, bool lines, Form col, cudaStream_t s)
{
    switch (col_fmt) {
        case EZ_MX_E2M1: return band<ROW, EZ_MX_E2M1>(a, lines, col, s);
        case EZ_MX_E4M3: return band<ROW, EZ_MX_E4M3>(a, lines, col, s);
    }
    return band<ROW, EZ_MX_E5M2>(a, lines, col, s);
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
    switch (row_fmt) {
        case EZ_MX_E2M1: return band<EZ_MX_E2M1>(col_fmt, a, lines, col, s);
        case EZ_MX_E4M3: return band<EZ_MX_E4M3>(col_fmt, a, lines, col, s);
        case EZ_MX_E5M2: return band<EZ_MX_E5M2>(col_fmt, a, lines, col, s);
    }
    return band<0>(col_fmt, a, lines, col, s);
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
    return ez::launch_dependent(k_rms_dweight, (unsigned)ez::cdiv(cols, 32), 32 * kSlices, 0, s, (const float*)ws, parts, cols,
                                add, dweight);
}

}  // namespace ezk
