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
// Every MX kernel but the product works on pieces of a scale tile (128 rows by
// 128 columns): 256 threads, thread t on columns 8 * (t & 15) .. + 7 of rows
// (t >> 4) + 16 i, so a block's four threads are neighbouring lanes and a warp
// moves two runs of 256 bytes.  A CTA takes 128 rows, or fewer when there are
// too few tiles to fill the GPU.
#pragma once

#include <cstdint>

#include "ez_common.cuh"

namespace ezmx {

constexpr int kTileRows = 128, kTileCols = 128, kBlock = 32;
constexpr int kThreadsMx = 256, kRowStep = 16;

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
// 2^-k of a scale byte below 255, twice in BF16 (k <= 125, so it is normal).
__device__ __forceinline__ uint32_t inv_scale(uint32_t byte) { return ((254u - byte) << 7) * 0x00010001u; }
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
// Larger magnitude of each half, a NaN if there is one (signs are left over).
__device__ __forceinline__ uint32_t mag_max(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ void st_v8(void* p, const uint32_t* w)
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 :: "l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}
__device__ __forceinline__ void ld_v8(const float* p, float* v)
{
    asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "l"(p) : "memory");
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Codes of 8 scaled values: one word (E2M1, value 0 in the low half byte) or
// two words in order.  Scaling in BF16 is exact too (only the exponent moves).
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
// and hi bound its bytes.
struct Rows {
    const uint16_t* p;
    uint64_t ld;
    const uint8_t *lo, *hi;
};
inline Rows make_rows(const uint16_t* p, uint64_t rows, uint64_t cols, uint64_t ld)
{
    Rows r;
    r.p = p;
    r.ld = ld;
    r.lo = reinterpret_cast<const uint8_t*>(p);
    r.hi = rows ? reinterpret_cast<const uint8_t*>(p + (rows - 1) * ld + cols) : r.lo;
    return r;
}
// Whether every row is on a 16-byte boundary.
inline bool lined(const void* p, uint64_t rows, uint64_t ld)
{
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (rows <= 1 || ld % 8 == 0);
}

// Values [col, col + 8) of a row, zeros from `cols` on, in two steps so that
// the loads of several rows are in flight together.  FAST: the rows are lined
// and the values all there.  Else the two 16-byte granules around them are read
// (whole granules only inside the matrix's own bytes, single values at its
// ends) and shifted: two loads that share their lines instead of eight 2-byte
// ones.
template <bool FAST> struct Load8;
template <> struct Load8<true> {
    uint4 v;
    __device__ __forceinline__ void start(const Rows& x, uint64_t row, uint64_t col, uint64_t)
    {
        v = ez::ld_v4_nc(x.p + row * x.ld + col);
    }
    __device__ __forceinline__ uint4 finish() const { return v; }
};
template <> struct Load8<false> {
    uint4 a, b;
    const uint16_t* p;
    int some;            // values to read one by one (0: the granules hold them)
    __device__ __forceinline__ void start(const Rows& x, uint64_t row, uint64_t col, uint64_t cols)
    {
        p = x.p + row * x.ld + col;
        a = b = make_uint4(0u, 0u, 0u, 0u);
        some = 0;
        if (col >= cols) return;
        const uint32_t m = (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15u);
        const uint8_t* g = reinterpret_cast<const uint8_t*>(p) - m;
        if (col + 8 <= cols && g >= x.lo && g + (m ? 32 : 16) <= x.hi) {
            a = ez::ld_v4_nc(g);
            if (m) b = ez::ld_v4_nc(g + 16);
        } else {
            some = col + 8 <= cols ? 8 : (int)(cols - col);
        }
    }
    __device__ __forceinline__ uint4 finish() const
    {
        if (some) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t l = 2 * i < some ? p[2 * i] : 0u, h = 2 * i + 1 < some ? p[2 * i + 1] : 0u;
                w[i] = l | (h << 16);
            }
            return make_uint4(w[0], w[1], w[2], w[3]);
        }
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        return shift16(w, (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15u));
    }
};

// 32 rows of 128 values on their way to rows at any alignment (17 granules a
// row: 16 and a spare, which also spreads the rows over the banks).
struct Stage {
    uint4 row[32][17];
};
// Called by 256 threads (t: 0..255) after a barrier (users that alternate
// between two stages need no second one): rows [r0, r0 + 32) below `rows`
// and columns [c0, c0 + 128) below `cols` of `out`.  Whole aligned granules are
// stored as such; the values before the first and after the last one of a row
// (under 8 each) one by one, one per thread.
__device__ __forceinline__ void store_stage(const Stage& s, uint16_t* out, uint64_t ld, uint64_t r0, uint64_t rows,
                                            uint64_t c0, uint64_t cols, uint32_t t)
{
    const int n = (int)(cols - c0 < kTileCols ? cols - c0 : kTileCols);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t lr = (t >> 4) + 16 * i;
        if (r0 + lr >= rows) break;
        uint16_t* p = out + (r0 + lr) * ld + c0;
        const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15u) / 2;
        const int col = 8 * (int)(t & 15u) - (int)off;       // this granule's first value
        if (col < 0 || col + 8 > n) continue;
        const uint4* q = &s.row[lr][t & 15u];
        if (off == 0) {
            *reinterpret_cast<uint4*>(p + col) = *q;
        } else {
            const uint4 a = q[-1], b = q[0];
            const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
            *reinterpret_cast<uint4*>(p + col) = shift16(w, 16 - 2 * off);
        }
    }
    const uint32_t lr = t >> 3;
    if (r0 + lr >= rows) return;
    uint16_t* p = out + (r0 + lr) * ld + c0;
    const uint16_t* v = reinterpret_cast<const uint16_t*>(s.row[lr]);
    const int off = (int)((reinterpret_cast<uintptr_t>(p) & 15u) / 2), e = (int)(t & 7u);
    const int first = off ? min(8 - off, n) : 0;                 // values before the first granule
    // the granules stored above end at 8 * 16 - off; what is left to n is under 8 values
    const int last = max(first, min((n + off) / 8, 16) * 8 - off);
    if (e < first) p[e] = v[e];
    if (last + e < n) p[last + e] = v[last + e];
}

// Quantise the row block a quad of lanes holds (8 values each, as BF16 words)
// and return its scale byte; codes go to out.  Called by whole warps.
template <int FMT>
__device__ __forceinline__ uint32_t quantise_quad(const uint4& x, uint32_t* out)
{
    uint32_t m = mag_max(mag_max(x.x, x.y), mag_max(x.z, x.w));
    m = mag_max(m, __shfl_xor_sync(ez::kFull, m, 1));
    m = mag_max(m, __shfl_xor_sync(ez::kFull, m, 2));
    const uint32_t s = scale_byte<FMT>(mag_max(m, m >> 16) & 0x7FFFu);
    uint32_t w[4] = {x.x, x.y, x.z, x.w}, inv = inv_scale(s);
    if (__any_sync(ez::kFull, s == 255u) && s == 255u) w[0] = w[1] = w[2] = w[3] = inv = 0u;
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t y = mul2(w[i], inv);
        v[2 * i] = lo_f(y);
        v[2 * i + 1] = hi_f(y);
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
// The word of scale bytes (4 blocks) of a row of a 512-byte scale tile.  The
// order is the one the tensor core's scale operand has in tensor memory: lane
// row % 32, column row / 32, byte block.
__device__ __forceinline__ uint32_t* scale_word(uint8_t* scales, uint64_t tile, uint32_t row)
{
    return reinterpret_cast<uint32_t*>(scales + tile * 512 + (row & 31u) * 16u + (row >> 5) * 4u);
}

// SMs of the current device; 0 if it cannot be asked.
inline uint32_t sm_count()
{
    static std::atomic<int> known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    int n = known[dev].load(std::memory_order_relaxed);
    if (!n) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        known[dev].store(n, std::memory_order_relaxed);
    }
    return (uint32_t)n;
}

}  // namespace ezmx
