// ez_mx.cuh -- the microscaled (MX) tensor in device code: formats, scales,
// and the row loads and stores the MX kernels share.
//
// A block of 32 values shares the scale 2^k, k the smallest integer with
// amax <= F * 2^k (F the format's largest magnitude), clamped to [kmin, kmax];
// the scale byte is k + 127, and 255 marks a block with an infinity or NaN.
// x * 2^-k is exact in FP32 unless it falls under 2^-126, far below half of
// any format's smallest step, so the hardware conversion's round to nearest
// even is the only rounding and the codes are a function of x alone.
//
// Every MX kernel but the product works on tiles of 128 rows by 128 columns
// (one 512-byte scale tile): 256 threads, thread t on columns
// 8 * (t & 15) .. + 7 of rows (t >> 4) + 16 i, so a block's four threads are
// neighbouring lanes and a warp moves two runs of 256 bytes.
#pragma once

#include <cstdint>

#include "ez_common.cuh"

namespace ezmx {

constexpr int kTileRows = 128, kTileCols = 128, kBlock = 32;
constexpr int kThreadsMx = 256, kRowStep = 16, kRowIters = kTileRows / kRowStep;

template <int FMT> struct Fmt;
// kFrac: F's fraction bits as BF16 holds them; kExp: F = 1.frac * 2^kExp
template <> struct Fmt<EZ_MX_E2M1> {
    static constexpr int kFrac = 0x40, kExp = 2, kMin = -127, kMax = 125, kBits = 4;
};
template <> struct Fmt<EZ_MX_E4M3> {
    static constexpr int kFrac = 0x60, kExp = 8, kMin = -124, kMax = 119, kBits = 8;
};
template <> struct Fmt<EZ_MX_E5M2> {
    static constexpr int kFrac = 0x60, kExp = 15, kMin = -117, kMax = 112, kBits = 8;
};

// Scale byte of a block whose largest magnitude has the BF16 bits mag.  A
// subnormal amax gives an exponent under kmin, which the clamp sets.
template <int FMT>
__device__ __forceinline__ uint32_t scale_byte(uint32_t mag)
{
    using F = Fmt<FMT>;
    if (mag >= 0x7F80u) return 255u;
    const int k = (int)(mag >> 7) - 127 - F::kExp + ((int)(mag & 0x7Fu) > F::kFrac ? 1 : 0);
    return (uint32_t)(min(max(k, F::kMin), F::kMax) + 127);
}
// 2^-k of a scale byte below 255 (k <= 125, so the result is normal).
__device__ __forceinline__ float inv_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }
// 2^k of a scale byte; 255 gives NaN, 0 the subnormal 2^-127.
__device__ __forceinline__ float scale_value(uint32_t byte)
{
    return byte == 255u ? __uint_as_float(0x7FFFFFFFu)
                        : __uint_as_float(byte ? byte << 23 : 0x00400000u);
}

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t mag_max(uint32_t a, uint32_t w)
{
    return __vmaxu2(a, w & 0x7FFF7FFFu);
}

// Codes of 8 scaled values: one word (E2M1, value 0 in the low half byte) or
// two words in order.
template <int FMT>
__device__ __forceinline__ void encode8(const float* v, uint32_t* out)
{
    if constexpr (FMT == EZ_MX_E2M1) {
        asm("{\n\t.reg .b8 a, b, c, d;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
            "mov.b32 %0, {a, b, c, d};\n\t}"
            : "=r"(out[0])
            : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float* p = v + 4 * i;
            if constexpr (FMT == EZ_MX_E4M3)
                asm("{\n\t.reg .b16 a, b;\n\t"
                    "cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\t"
                    "cvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\t"
                    "mov.b32 %0, {a, b};\n\t}"
                    : "=r"(out[i]) : "f"(p[0]), "f"(p[1]), "f"(p[2]), "f"(p[3]));
            else
                asm("{\n\t.reg .b16 a, b;\n\t"
                    "cvt.rn.satfinite.e5m2x2.f32 a, %2, %1;\n\t"
                    "cvt.rn.satfinite.e5m2x2.f32 b, %4, %3;\n\t"
                    "mov.b32 %0, {a, b};\n\t}"
                    : "=r"(out[i]) : "f"(p[0]), "f"(p[1]), "f"(p[2]), "f"(p[3]));
        }
    }
}

__device__ __forceinline__ void half2_to_f(uint32_t h, float* v)
{
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(v[0]), "=f"(v[1]) : "r"(h));
}
// The 8 values of one (E2M1) or two code words, before scaling.
template <int FMT>
__device__ __forceinline__ void decode8(const uint32_t* in, float* v)
{
    uint32_t h[4];
    if constexpr (FMT == EZ_MX_E2M1) {
        asm("{\n\t.reg .b8 a, b, c, d;\n\t"
            "mov.b32 {a, b, c, d}, %4;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
            "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
            "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
            "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
            : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(in[0]));
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if constexpr (FMT == EZ_MX_E4M3)
                asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
                    "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
                    : "=r"(h[2 * i]), "=r"(h[2 * i + 1]) : "r"(in[i]));
            else
                asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
                    "cvt.rn.f16x2.e5m2x2 %0, a;\n\tcvt.rn.f16x2.e5m2x2 %1, b;\n\t}"
                    : "=r"(h[2 * i]), "=r"(h[2 * i + 1]) : "r"(in[i]));
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) half2_to_f(h[i], v + 2 * i);
}

// Byte of (row, block) inside a 512-byte scale tile of 128 rows x 4 blocks.
// The order is the one the tensor core's scale operand has in tensor memory:
// lane row % 32, column row / 32, byte block.
__device__ __forceinline__ uint32_t scale_at(uint32_t row, uint32_t block)
{
    return (row & 31u) * 16u + (row >> 5) * 4u + block;
}

// ---- rows of BF16 at any 2-byte alignment -------------------------------------
// The 16 bytes at byte `m` (even, under 16) of the 32 bytes w.
__device__ __forceinline__ uint4 shift16(const uint32_t* w, uint32_t m)
{
    uint32_t a[6], b[5];
#pragma unroll
    for (int i = 0; i < 6; ++i) a[i] = (m & 8u) ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) b[i] = (m & 4u) ? a[i + 1] : a[i];
    const uint32_t s = (m & 2u) * 8u;
    return make_uint4(__funnelshift_r(b[0], b[1], s), __funnelshift_r(b[1], b[2], s),
                      __funnelshift_r(b[2], b[3], s), __funnelshift_r(b[3], b[4], s));
}

// A matrix of BF16 [rows, ld] whose rows start at any 2-byte alignment; lo
// and hi bound its bytes.  `aligned` (rows on 16-byte boundaries) is the same
// for the whole grid.
struct Rows {
    const uint16_t* p;
    uint64_t ld;
    const uint8_t *lo, *hi;
    int aligned;
};
inline Rows make_rows(const uint16_t* p, uint64_t rows, uint64_t cols, uint64_t ld)
{
    Rows r;
    r.p = p;
    r.ld = ld;
    r.lo = reinterpret_cast<const uint8_t*>(p);
    r.hi = rows ? reinterpret_cast<const uint8_t*>(p + (rows - 1) * ld + cols) : r.lo;
    r.aligned = (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % 8 == 0;
    return r;
}

// Values [col, col + 8) of `row`, zeros from `cols` on.  Unaligned rows read
// the two 16-byte granules around them (whole granules only inside the
// matrix's own bytes, single values at its ends) and shift: two loads that
// share their lines instead of eight 2-byte ones.
__device__ __forceinline__ uint4 load8(const Rows& x, uint64_t row, uint64_t col, uint64_t cols)
{
    uint4 r = make_uint4(0u, 0u, 0u, 0u);
    if (col >= cols) return r;
    const uint16_t* p = x.p + row * x.ld + col;
    if (x.aligned && col + 8 <= cols) return ez::ld_v4_nc(p);
    const uint32_t m = (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15u);
    const uint8_t* g = reinterpret_cast<const uint8_t*>(p) - m;
    if (col + 8 <= cols && g >= x.lo && g + 32 <= x.hi) {
        const uint4 a = ez::ld_v4_nc(g), b = ez::ld_v4_nc(g + 16);
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        return shift16(w, m);
    }
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t l = col + 2 * i < cols ? p[2 * i] : 0u;
        const uint32_t h = col + 2 * i + 1 < cols ? p[2 * i + 1] : 0u;
        w[i] = l | (h << 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void store_some(uint16_t* p, const uint32_t* w, int from, int to)
{
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i >= from && i < to) p[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
}

// Store the 8 values v at [col, col + 8) of the row at `row_p`, those below
// `cols` only (0: no row).  Called by whole warps, 16 lanes to a row, lane
// `seg` of them on col = tile column + 8 seg.  An unaligned row is written in
// aligned granules: a lane joins the end of its left neighbour's values with
// the start of its own, and single values are stored only at the ends of the
// 128 columns.
__device__ __forceinline__ void store8(uint16_t* row_p, uint32_t seg, uint64_t col, uint64_t cols, uint4 v)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t both[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        both[i] = __shfl_up_sync(ez::kFull, w[i], 1, 16);
        both[4 + i] = w[i];
    }
    if (col >= cols) return;
    uint16_t* p = row_p + col;
    const uint32_t m = (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15u);
    const bool whole = col + 8 <= cols;
    const int nv = whole ? 8 : (int)(cols - col), head = 8 - (int)(m >> 1);
    if (m == 0u) {
        if (whole)
            *reinterpret_cast<uint4*>(p) = v;
        else
            store_some(p, w, 0, nv);
        return;
    }
    if (seg == 0u || !whole) {
        store_some(p, w, 0, min(head, nv));
        if (seg != 0u) store_some(p - 8, both, head, 8);
    } else {
        *reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(p) - m) = shift16(both, 16u - m);
    }
    // the values past the granule: the right neighbour's, unless there is none
    if (seg == 15u || col + 8 >= cols) store_some(p, w, head, nv);
}

// Quantise the row block a quad of lanes holds (8 values each, as BF16 words)
// and return its scale byte; codes go to out.  Called by whole warps.
template <int FMT>
__device__ __forceinline__ uint32_t quantise_quad(const uint4& x, uint32_t* out)
{
    uint32_t m = mag_max(mag_max(mag_max(mag_max(0u, x.x), x.y), x.z), x.w);
    m = __vmaxu2(m, __shfl_xor_sync(ez::kFull, m, 1));
    m = __vmaxu2(m, __shfl_xor_sync(ez::kFull, m, 2));
    const uint32_t s = scale_byte<FMT>(max(m & 0xFFFFu, m >> 16));
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    float v[8];
    const float inv = inv_scale(s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = s == 255u ? 0.f : lo_f(w[i]) * inv;
        v[2 * i + 1] = s == 255u ? 0.f : hi_f(w[i]) * inv;
    }
    encode8<FMT>(v, out);
    return s;
}

// One form of a microscaled matrix [rows, cols] in device memory.
struct Form {
    uint8_t* codes;
    uint8_t* scales;
};
template <int FMT>
__host__ __device__ __forceinline__ uint64_t code_pitch(uint64_t cols)
{
    return (cols + kBlock - 1) / kBlock * (kBlock * Fmt<FMT>::kBits / 8);
}

}  // namespace ezmx
