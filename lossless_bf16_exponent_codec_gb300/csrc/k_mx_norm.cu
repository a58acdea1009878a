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
// Squares of BF16 values are exact in FP32 and so is total weight, as far as its range
// goes (include/expzip.h).  Sums and rstd are pairs of FP32 numbers, so that y is the exact
// number rounded to FP32 and then to BF16.
// In a tensor of 10^8 values a y next to a border of BF16 is next to a border of a 4-bit
// code often enough for less than that to give other codes than 64-bit arithmetic does.
//
// Bound by memory at size, measured on one GB300: 16384 x 8192 with a residual to 4-bit
// rows 134 us (877 MB, 6.6 TB/s), the column form after it 78 (403 MB, 5.2: its loads wait
// while a piece is encoded); the backward pass 172 (1.07 GB, 6.3).  One row of 2048 is a
// launch's time.  Products of BF16 halves in FP32 and sums in BF16 are one instruction
// each (with shifts and masks to FP32 words the rows took 154).
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
    float *rstd, *low;              // low: what rstd's rounding leaves, for the columns; or null
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
// Two FP32 numbers in a register pair, and packed arithmetic on them.
using Pair = unsigned long long;
__device__ __forceinline__ Pair pair(float a, float b)
{
    Pair r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void split(Pair v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ Pair products(uint32_t a, uint32_t b)
{
    float lo, hi;
    ezmx::products(a, b, lo, hi);
    return pair(lo, hi);
}
__device__ __forceinline__ uint32_t word_of(Pair v)
{
    float a, b;
    split(v, a, b);
    return bf16x2(a, b);
}
__device__ __forceinline__ Pair plus(Pair a, Pair b)
{
    Pair r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ Pair minus(Pair a, Pair b)
{
    Pair r;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ Pair times(Pair a, Pair b)
{
    Pair r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ Pair fused(Pair a, Pair b, Pair c)
{
    Pair r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// A thread's sum of squares, of even and odd values, with what its additions round off.
struct Squares {
    Pair s = 0, e = 0;
    __device__ __forceinline__ void add(const uint4& v)
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const Pair q = products(w[j], w[j]), t = plus(s, q), b = minus(t, s);
            e = plus(e, plus(minus(s, minus(t, b)), minus(q, b)));
            s = t;
        }
    }
    __device__ __forceinline__ Two sum() const
    {
        Two a, b;
        split(s, a.hi, b.hi);
        split(e, a.lo, b.lo);
        return add2(a, b);
    }
};
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

// 1 / sqrt(sum / cols + eps): a Newton step from rsqrtf with everything in pairs.  0 and
// infinities stay what rsqrtf says.
__device__ __forceinline__ Two inverse_root(const Two& sum, float cols, float eps)
{
    const float q = sum.hi / cols;
    const Two mean{q, (__fmaf_rn(-q, cols, sum.hi) + sum.lo) / cols};
    Two m = add2(mean, Two{eps, 0.f});
    const float h = isinf(q) ? q : m.hi + m.lo;     // an infinity's residual is NaN
    const float r = rsqrtf(h);
    if (!(r > 0.f) || isinf(r)) return {r, 0.f};
    m.lo += m.hi - h;
    const float a = r * h, a_lo = __fmaf_rn(r, h, -a);                      // r m
    const float e = __fmaf_rn(-a, r, 1.f) - __fmaf_rn(m.lo, r, a_lo) * r;   // 1 - r^2 m
    const float d = 0.5f * r * __fmaf_rn(0.75f * e, e, e), t = r + d;
    return {t, d - (t - r)};
}

// total weight rstd, eight values.
__device__ __forceinline__ uint4 normed(const uint4& total, const uint4& weight, const Two& rstd)
{
    uint32_t t[4] = {total.x, total.y, total.z, total.w};
    const uint32_t w[4] = {weight.x, weight.y, weight.z, weight.w};
    const Pair hi = pair(rstd.hi, rstd.hi), lo = pair(rstd.lo, rstd.lo);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const Pair p = products(t[j], w[j]);
        t[j] = word_of(fused(p, hi, times(p, lo)));
    }
    return make_uint4(t[0], t[1], t[2], t[3]);
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

// x + residual in BF16, eight values.
__device__ __forceinline__ uint4 add8(const uint4& x, const uint4& r)
{
    return make_uint4(sums(x.x, r.x), sums(x.y, r.y), sums(x.z, r.z), sums(x.w, r.w));
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

// How rows lie.  kLined: on 16 bytes, their lengths too.  kPhased: all matrices' rows at the
// same place between 16-byte boundaries (rows of odd lengths one behind the other): a
// thread takes the granules of that place, from up to 7 values before the row's first, so
// that nothing is shifted but the weight, and the codes.  kOther: through shared memory.
enum { kLined, kPhased, kOther };

}  // namespace

// TPR threads to a row, V groups of eight values to a thread (group v of thread t
// at column 8 (v TPR + t), less the row's place); total, rstd, y and the row form, all in
// one read.  Rows of other places stay in shared memory, where they are on their way out
// anyway, a group at a time.
template <int TPR, int V, int MODE, int ROW>
__global__ void __launch_bounds__(kThreadsOf<TPR>) k_rms_rows(const NormArgs a)
{
    constexpr int kRows = kThreadsOf<TPR> / TPR, kUnroll = MODE == kOther ? 1 : V;
    constexpr bool kStaged = MODE == kOther;
    __shared__ Two s_part[kThreadsOf<TPR> / 32];
    extern __shared__ uint4 s_stage[];                  // but for kLined: kRows rows, and a granule behind each
    ez::grid_dep_launch();
    const uint32_t t = threadIdx.x % TPR, g = threadIdx.x / TPR;
    const uint64_t row = (uint64_t)blockIdx.x * kRows + g;
    const int cols = row < a.rows ? (int)a.cols : 0;
    const int off = MODE == kPhased && cols ? (int)(reinterpret_cast<uintptr_t>(a.x.p + row * a.x.ld) & 15u) / 2 : 0;
    uint4* const stage = s_stage + g * (V * TPR + 1);
    ez::grid_dep_wait();
    uint4 v[kStaged ? 1 : V];
    Squares sum;
    if constexpr (kStaged) {
#pragma unroll 1
        for (int i = 0; i < V; ++i) {
            const int c = 8 * (int)(i * TPR + t);
            Load8<false, false> x{}, r{};
            if (c < cols) {
                x.start(a.x, row, c, cols);
                if (a.residual.p) r.start(a.residual, row, c, cols);
            }
            v[0] = x.finish();
            if (a.residual.p) v[0] = add8(v[0], r.finish());
            sum.add(v[0]);
            stage[i * TPR + t] = v[0];
        }
    } else {
        uint4 r[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = 8 * (int)(i * TPR + t) - off;
            v[i] = r[i] = make_uint4(0u, 0u, 0u, 0u);
            if (c >= cols) continue;
            if constexpr (MODE == kLined) {
                v[i] = load16<false>(a.x.p + row * a.x.ld + c);
                if (a.residual.p) r[i] = load16<false>(a.residual.p + row * a.residual.ld + c);
            } else {
                v[i] = load_granule<false>(a.x, row, c, cols);
                if (a.residual.p) r[i] = load_granule<false>(a.residual, row, c, cols);
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = 8 * (int)(i * TPR + t) - off;
            if (a.residual.p) v[i] = add8(v[i], r[i]);
            if constexpr (MODE == kPhased) v[i] = only_columns(v[i], c, cols);
            sum.add(v[i]);
            if (a.total && c < cols) {
                if constexpr (MODE == kLined)
                    *reinterpret_cast<uint4*>(a.total + row * a.ldt + c) = v[i];
                else
                    store_granule(a.total + row * a.ldt, v[i], c, cols);
            }
        }
    }
    const Two rstd = inverse_root(row_sum<TPR>(sum.sum(), s_part), (float)a.cols, a.eps);
    if (t == 0 && cols) {
        a.rstd[row] = rstd.hi;
        if (a.low) a.low[row] = rstd.lo;
    }
    if (kStaged && a.total) {
        __syncthreads();
        if (cols) store_row<TPR>([=](uint32_t i) { return stage[i]; }, a.total + row * a.ldt, (uint32_t)cols, t);
        __syncthreads();
    }
    if (ROW == 0 && !a.y) return;
    const uint64_t pitch = ROW ? code_pitch<ROW ? ROW : EZ_MX_E2M1>(a.cols) : 0;
#pragma unroll kUnroll
    for (int i = 0; i < V; ++i) {
        const int c = 8 * (int)(i * TPR + t) - off;
        uint4 y = make_uint4(0u, 0u, 0u, 0u);
        if (c < cols) {
            if constexpr (MODE == kLined) {
                y = normed(v[i], load16<true>(a.weight.p + c), rstd);
                if (a.y) *reinterpret_cast<uint4*>(a.y + row * a.ldy + c) = y;
            } else {
                Any8 w;
                w.start(a.weight, 0, c, cols);
                y = normed(kStaged ? stage[i * TPR + t] : v[kStaged ? 0 : i], w.finish(), rstd);
                if (MODE == kPhased && a.y) store_granule(a.y + row * a.ldy, y, c, cols);
            }
        }
        if constexpr (MODE != kLined) stage[i * TPR + t] = y;
        if constexpr (MODE != kPhased && ROW != 0) store_codes<ROW>(a.row, y, row, (uint32_t)c, cols, pitch, a.col_tiles);
    }
    if (kStaged && a.y) {
        __syncthreads();
        if (cols) store_row<TPR>([=](uint32_t i) { return stage[i]; }, a.y + row * a.ldy, (uint32_t)cols, t);
    }
    if constexpr (MODE == kPhased && ROW != 0) {
        if (t == 0) stage[V * TPR] = make_uint4(0u, 0u, 0u, 0u);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint32_t k = i * TPR + t;
            const uint4 lo = stage[k], hi = stage[k + 1];
            const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            store_codes<ROW>(a.row, shift16(w, 2 * off), row, 8 * k, cols, pitch, a.col_tiles);
        }
    }
}

// ---- column form -----------------------------------------------------------------

namespace {

struct NormSource {
    const Rows& total;
    uint64_t rows, cols;
    const Two* rstd;                // of the piece's rows
    uint4 weight;                   // of the thread's columns
    template <bool FAST>
    __device__ __forceinline__ void start(Load8<FAST>& in, uint64_t r, uint64_t c) const
    {
        in.start(total, r, c, r < rows ? cols : 0);
    }
    template <bool FAST>
    __device__ __forceinline__ uint4 finish(const Load8<FAST>& in, uint64_t r, uint32_t lr, uint64_t) const
    {
        // a row that is none stays zero, and not -0
        return FAST || r < rows ? normed(in.finish(), weight, rstd[lr]) : make_uint4(0u, 0u, 0u, 0u);
    }
};

}  // namespace

// From total and rstd, a piece of a scale tile per CTA.  Bands of 32 rows that a cluster of
// CTAs kept in shared memory until it had their sums (total read once; 64 KB, three CTAs
// to an SM) took 242 us with rows and columns of 16384 x 8192, when this kernel and the one
// above took 216: loads stood still while a band was encoded.
template <int COL, int ROWS>
__global__ void __launch_bounds__(kThreadsMx, ROWS == 128 ? 3 : 4)
    k_rms_columns(Rows total, const float* rstd, const float* low, Rows weight, uint64_t rows, uint64_t cols,
                  uint32_t col_tiles, int lines, Form col)
{
    __shared__ PieceShared<COL, ROWS> s;
    __shared__ Two s_rstd[ROWS];
    ez::grid_dep_launch();
    const uint32_t piece = blockIdx.x / col_tiles, ct = blockIdx.x - piece * col_tiles, t = threadIdx.x;
    const uint64_t r0 = (uint64_t)piece * ROWS, c0 = (uint64_t)ct * kTileCols;
    ez::grid_dep_wait();
    if (t < ROWS) s_rstd[t] = r0 + t < rows ? Two{rstd[r0 + t], low[r0 + t]} : Two{0.f, 0.f};
    Load8<false> w;
    w.start(weight, 0, c0 + 8 * (t & 15u), cols);
    const NormSource src{total, rows, cols, s_rstd, w.finish()};
    __syncthreads();
    encode_piece<0, COL, ROWS>(src, lines && r0 + ROWS <= rows && c0 + kTileCols <= cols, rows, cols, col_tiles, ct,
                                Form{}, col, r0, s);
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

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" :: "l"(p)); }

// A CTA takes every gridDim-th group of rows; a thread's columns are the same in all of
// them (phased rows too: what lies between a CTA's rows is a multiple of 8 rows), so
// that the weight's gradient is summed in its registers.
template <int TPR, int V, int MODE>
__global__ void __launch_bounds__(kThreadsOf<TPR>, TPR <= 256 ? 2 : 1) k_rms_back(const NormBackArgs a)
{
    constexpr int kRows = kThreadsOf<TPR> / TPR;
    __shared__ float s_part[2][kThreadsOf<TPR> / 32];
    extern __shared__ uint4 s_stage[];                  // kOther: kRows rows
    ez::grid_dep_launch();
    const uint32_t t = threadIdx.x % TPR, g = threadIdx.x / TPR;
    const uint64_t first = (uint64_t)blockIdx.x * kRows + g;
    const int off = MODE == kPhased ? (int)(reinterpret_cast<uintptr_t>(a.dy.p + first * a.dy.ld) & 15u) / 2 : 0;
    uint4* const stage = s_stage + g * (V * TPR);
    ez::grid_dep_wait();
    // the weight of a group: from registers where there are any left
    auto read_weight = [&](int i) {
        const int c = 8 * (int)(i * TPR + t) - off;
        if (c >= (int)a.cols) return make_uint4(0u, 0u, 0u, 0u);
        if constexpr (MODE == kLined) {
            return load16<true>(a.weight.p + c);
        } else {
            Any8 l;
            l.start(a.weight, 0, c, (int)a.cols);
            return l.finish();
        }
    };
    constexpr bool kHeld = V <= 3;
    uint4 held[kHeld ? V : 1] = {};
    if constexpr (kHeld)
#pragma unroll
        for (int i = 0; i < V; ++i) held[i] = read_weight(i);
    auto weight = [&](int i) { return kHeld ? held[kHeld ? i : 0] : read_weight(i); };
    auto load_row = [&](uint64_t row, uint4* gv, uint4* nv, uint4* ev, float& rstd) {
        const int cols = row < a.rows ? (int)a.cols : 0;
        auto load = [&](const Rows& x, int c) {
            if constexpr (MODE == kLined) {
                return load16<false>(x.p + row * x.ld + c);
            } else if constexpr (MODE == kPhased) {
                return load_granule<false>(x, row, c, cols);
            } else {
                Load8<false, false> l;
                l.start(x, row, c, cols);
                return l.finish();
            }
        };
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = 8 * (int)(i * TPR + t) - off;
            gv[i] = nv[i] = ev[i] = make_uint4(0u, 0u, 0u, 0u);
            if (c >= cols) continue;
            gv[i] = load(a.dy, c);
            nv[i] = load(a.total, c);
            if (a.dtotal.p) ev[i] = load(a.dtotal, c);
        }
        rstd = cols ? a.rstd[row] : 0.f;
    };
    // short rows: the next one's values are on their way while a row is worked on (1001 rows
    // of 2731: 14.8 -> 11.3 us; longer rows have no registers left for it)
    constexpr bool kAhead = MODE != kOther && V <= 2;
    uint4 g_next[kAhead ? V : 1], n_next[kAhead ? V : 1], e_next[kAhead ? V : 1];
    float r_next;
    if constexpr (kAhead) load_row(first, g_next, n_next, e_next, r_next);
    float dw[V][8] = {};
    uint32_t turn = 0;
    for (uint64_t r0 = (uint64_t)blockIdx.x * kRows; r0 < a.rows; r0 += (uint64_t)gridDim.x * kRows, turn ^= 1u) {
        const uint64_t row = r0 + g;
        const int cols = row < a.rows ? (int)a.cols : 0;
        // the row after this one comes to L2 meanwhile
        if (const uint64_t next = row + (uint64_t)gridDim.x * kRows; MODE != kLined && !kAhead && next < a.rows)
            for (uint32_t c = 64 * t; c < a.cols; c += 64 * TPR) {
                prefetch_l2(a.dy.p + next * a.dy.ld + c);
                prefetch_l2(a.total.p + next * a.total.ld + c);
                if (a.dtotal.p) prefetch_l2(a.dtotal.p + next * a.dtotal.ld + c);
            }
        uint4 gv[V], nv[V], ev[V];
        float rstd;
        if constexpr (kAhead) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                gv[i] = g_next[i];
                nv[i] = n_next[i];
                ev[i] = e_next[i];
            }
            rstd = r_next;
            load_row(row + (uint64_t)gridDim.x * kRows, g_next, n_next, e_next, r_next);
        } else {
            load_row(row, gv, nv, ev, rstd);
        }
        float along = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if constexpr (MODE == kPhased) {
                const int c = 8 * (int)(i * TPR + t) - off;
                gv[i] = only_columns(gv[i], c, cols);
                nv[i] = only_columns(nv[i], c, cols);
            }
            float d[8], n[8], g[8];
            unpack8(gv[i], d);
            unpack8(nv[i], n);
            products8(gv[i], weight(i), g);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float nj = n[j] * rstd;
                along = __fmaf_rn(g[j], nj, along);
                dw[i][j] = __fmaf_rn(d[j], nj, dw[i][j]);
            }
        }
        along = row_sum<TPR>(along, s_part[turn]) / (float)a.cols;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = 8 * (int)(i * TPR + t) - off;
            float d[8], n[8], g[8], e[8];
            unpack8(nv[i], n);
            products8(gv[i], weight(i), g);
            unpack8(ev[i], e);
#pragma unroll
            for (int j = 0; j < 8; ++j) d[j] = __fmaf_rn(rstd, g[j] - n[j] * rstd * along, e[j]);
            const uint4 y = pack8(d);
            if constexpr (MODE == kOther) {
                stage[i * TPR + t] = y;
            } else if (c < cols) {
                if constexpr (MODE == kLined)
                    *reinterpret_cast<uint4*>(a.dx + row * a.ldx + c) = y;
                else
                    store_granule(a.dx + row * a.ldx, y, c, cols);
            }
        }
        if constexpr (MODE == kOther) {
            __syncthreads();
            if (cols) store_row<TPR>([=](uint32_t i) { return stage[i]; }, a.dx + row * a.ldx, (uint32_t)cols, t);
            __syncthreads();
        }
    }
    if (!a.partial) return;
    float* const out = a.partial + first * a.cols;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = 8 * (int)(i * TPR + t) - off + j;
            if (c >= 0 && c < (int)a.cols) out[c] = dw[i][j];
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

constexpr uint32_t kBackCtas = 304;           // a multiple of 8

// Threads to a row and groups to a thread for a number of columns, and those that phased
// rows reach over (up to kMostCols).
constexpr uint32_t kMostCols = 16384;
template <template <int, int> class Go, typename... A>
cudaError_t by_width(uint32_t cols, const A&... args)
{
    if (cols <= 256) return Go<32, 1>::run(args...);
    if (cols <= 1024) return Go<128, 1>::run(args...);
    if (cols <= 2048) return Go<128, 2>::run(args...);
    if (cols <= 4096) return Go<256, 2>::run(args...);
    if (cols <= 6144) return Go<256, 3>::run(args...);
    if (cols <= 8192) return Go<256, 4>::run(args...);
    return Go<512, 4>::run(args...);
}

// The way of a matrix's rows between 16-byte boundaries.
struct Place {
    uintptr_t at, step;         // of the first row; from row to row
    Place(const void* p, uint64_t rows, uint64_t ld)
        : at(reinterpret_cast<uintptr_t>(p) & 15u), step(rows > 1 ? ld * 2 % 16 : 0)
    {
    }
    bool operator==(const Place& o) const { return at == o.at && step == o.step; }
};

template <int TPR, int V>
struct GoRows {
    template <int MODE, int ROW>
    static cudaError_t launch(const NormArgs& a, cudaStream_t s)
    {
        constexpr uint64_t kRows = kThreadsOf<TPR> / TPR;
        constexpr size_t kSmem = MODE == kLined ? 0 : kRows * (V * TPR + 1) * 16;
        static_assert(kSmem <= 48 * 1024, "what a launch may ask for without an attribute");
        // with a row form: the scale bytes of the rows of the last tile too
        const uint64_t rows = ROW ? ez::rup(a.rows, kTileRows) : a.rows;
        return ez::launch_dependent(k_rms_rows<TPR, V, MODE, ROW>, (unsigned)ez::cdiv(rows, kRows), kThreadsOf<TPR>,
                                    kSmem, s, a);
    }
    template <int MODE>
    static cudaError_t go(const NormArgs& a, int fmt, cudaStream_t s)
    {
        switch (fmt) {
            case EZ_MX_E2M1: return launch<MODE, EZ_MX_E2M1>(a, s);
            case EZ_MX_E4M3: return launch<MODE, EZ_MX_E4M3>(a, s);
            case EZ_MX_E5M2: return launch<MODE, EZ_MX_E5M2>(a, s);
        }
        return launch<MODE, 0>(a, s);
    }
    static cudaError_t run(const NormArgs& a, const int& fmt, const int& mode, const cudaStream_t& s)
    {
        return mode == kLined ? go<kLined>(a, fmt, s) : mode == kPhased ? go<kPhased>(a, fmt, s) : go<kOther>(a, fmt, s);
    }
};

template <int TPR, int V>
struct GoBack {
    template <int MODE>
    static cudaError_t launch(const NormBackArgs& a, uint32_t& parts, cudaStream_t s)
    {
        constexpr uint64_t kRows = kThreadsOf<TPR> / TPR;
        constexpr size_t kSmem = MODE == kOther ? kRows * V * TPR * 16 : 0;
        const unsigned grid = (unsigned)ez::umin64(ez::cdiv(a.rows, kRows), kBackCtas);
        parts = grid * (uint32_t)kRows;
        return ez::launch_dependent(k_rms_back<TPR, V, MODE>, grid, kThreadsOf<TPR>, kSmem, s, a);
    }
    static cudaError_t run(const NormBackArgs& a, const int& mode, uint32_t* const& parts, const cudaStream_t& s)
    {
        return mode == kLined    ? launch<kLined>(a, *parts, s)
               : mode == kPhased ? launch<kPhased>(a, *parts, s)
                                 : launch<kOther>(a, *parts, s);
    }
};

template <int COL, int ROWS>
cudaError_t columns_rows(const Rows& total, const NormArgs& a, Form col, cudaStream_t s)
{
    const uint64_t pieces = ez::cdiv(a.rows, kTileRows) * (kTileRows / ROWS);
    return ez::launch_dependent(k_rms_columns<COL, ROWS>, (unsigned)(pieces * a.col_tiles), kThreadsMx, 0, s, total,
                                (const float*)a.rstd, (const float*)a.low, a.weight, a.rows, (uint64_t)a.cols, a.col_tiles,
                                (int)lined(total.p, a.rows, total.ld), col);
}
template <int COL>
cudaError_t columns(const Rows& total, const NormArgs& a, Form col, cudaStream_t s)
{
    const uint64_t per_sm = tiles_per_sm(a.rows, a.cols);
    if (per_sm >= 4) return columns_rows<COL, 128>(total, a, col, s);
    if (per_sm >= 2) return columns_rows<COL, 64>(total, a, col, s);
    return columns_rows<COL, 32>(total, a, col, s);
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
                               float* rstd, float* low, uint16_t* y, uint64_t ldy, int row_fmt, uint8_t* row_codes,
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
    a.low = low;
    a.y = y;
    a.ldy = ldy;
    const Form row{row_codes, row_scales}, col{col_codes, col_scales};
    a.row = row;
    const bool lines = cols % 8 == 0 && lined(x, rows, ldx) && (!residual || lined(residual, rows, ldr)) &&
                       lined(weight, 1, cols) && (!total || lined(total, rows, ldt)) && (!y || lined(y, rows, ldy));
    const Place place(x, rows, ldx);
    const bool phased = (!residual || place == Place(residual, rows, ldr)) && (!total || place == Place(total, rows, ldt)) &&
                        (!y || place == Place(y, rows, ldy));
    const int mode = lines ? kLined : phased && cols + 7 <= kMostCols ? kPhased : kOther;
    const Rows sum = total ? make_rows(total, rows, cols, ldt) : a.x;
    const cudaError_t e = by_width<GoRows>(cols + (mode == kPhased ? 7 : 0), a, row_fmt, mode, s);
    if (e != cudaSuccess || !col_fmt) return e;
    if (col_fmt == EZ_MX_E2M1) return columns<EZ_MX_E2M1>(sum, a, col, s);
    return col_fmt == EZ_MX_E4M3 ? columns<EZ_MX_E4M3>(sum, a, col, s) : columns<EZ_MX_E5M2>(sum, a, col, s);
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
    const Place place(dy, rows, lddy);
    const bool phased = place == Place(total, rows, ldt) && (!dtotal || place == Place(dtotal, rows, lddt)) &&
                        place == Place(dx, rows, ldx);
    const int mode = lines ? kLined : phased && cols + 7 <= kMostCols ? kPhased : kOther;
    uint32_t parts = 0;
    if (rows) {
        const cudaError_t e = by_width<GoBack>(cols + (mode == kPhased ? 7 : 0), a, mode, &parts, s);
        if (e != cudaSuccess) return e;
    }
    if (!dweight) return cudaSuccess;
    return ez::launch_dependent(k_rms_dweight, (unsigned)ez::cdiv(cols, 32), 32 * kSlices, 0, s, (const float*)ws, parts, cols,
                                add, dweight);
}

}  // namespace ezk
