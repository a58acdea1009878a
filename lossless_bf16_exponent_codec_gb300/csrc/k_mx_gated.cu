// k_mx_gated.cu -- the gated unit h = silu(g) u that keeps g and u in 8 bits,
// and its backward pass from what was kept.
//
// With s = 1 / (1 + exp(-g)):  h = g s u,  du = dh g s,
// dg = dh u s (1 + g (1 - s)).  FP32 from exp to the one rounding of each result.
//
// Both passes read and write each byte once and are bound by memory: 8192 x
// 14336 values take 137 us forward (947 MB, 6.9 TB/s) and 174 back with h (1.18
// GB, 6.8 TB/s), the measured copy rate.  Two rows of every input are in flight
// per thread and four CTAs per SM (64 registers): eight rows and two CTAs took
// 199 and 243 us.
#include "ez_internal.h"
#include "ez_mx.cuh"

namespace ezk {
using namespace ezmx;

// As a quarter of the reciprocal of a quarter of 1 + exp(-g), which does not pass
// 2^126: a fast division by more than that gives zero, from g = -87.4 on, though s is
// still a number down to g = -88.7, where exp(-g) leaves FP32.
__device__ __forceinline__ float logistic(float g)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(__fmaf_rn(0.25f, __expf(-g), 0.25f)));
    return 0.25f * r;
}

template <int FMT, int ROWS, bool FAST>
__device__ __forceinline__ void swiglu_piece(const Rows& gate, const Rows& up, uint64_t rows, uint64_t cols,
                                             Form gate8, Form up8, uint16_t* h, uint64_t ldh, uint64_t r0,
                                             uint64_t c0, Stage* s_stage, uint8_t* s_gate, uint8_t* s_up)
{
    const uint32_t t = threadIdx.x, seg = t & 15u;
    const uint64_t c = c0 + 8 * seg, pitch = code_pitch<FMT>(cols);
    const bool block_in = FAST || c / kBlock * kBlock < cols;
#pragma unroll 1
    for (int i0 = 0; i0 < ROWS; i0 += 32) {       // 32 rows at a time, two of them per thread
        Stage& s_h = s_stage[i0 / 32 & 1];
        Load8<FAST> gin[2], uin[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint64_t r = r0 + i0 + (t >> 4) + kRowStep * i;
            gin[i].start(gate, r, c, r < rows ? cols : 0);
            uin[i].start(up, r, c, r < rows ? cols : 0);
        }
        const uint4 g[2] = {gin[0].finish(), gin[1].finish()}, u[2] = {uin[0].finish(), uin[1].finish()};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t lr = i0 + (t >> 4) + kRowStep * i;
            const uint64_t r = r0 + lr;
            const uint32_t gw[4] = {g[i].x, g[i].y, g[i].z, g[i].w}, uw[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
            uint32_t hw[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float g0 = lo_f(gw[j]), g1 = hi_f(gw[j]);
                hw[j] = bf16x2(g0 * logistic(g0) * lo_f(uw[j]), g1 * logistic(g1) * hi_f(uw[j]));
            }
            const uint4 y = make_uint4(hw[0], hw[1], hw[2], hw[3]);
            if constexpr (FAST)
                *reinterpret_cast<uint4*>(h + r * ldh + c) = y;
            else
                s_h.row[lr & 31u][seg] = y;
            uint32_t gc[2], uc[2];
            const uint32_t gs = quantise_quad<FMT>(g[i], gc), us = quantise_quad<FMT>(u[i], uc);
            const bool in = FAST || (block_in && r < rows);
            if ((t & 3u) == 0) {
                s_gate[lr * 4 + (seg >> 2)] = in ? (uint8_t)gs : 0;
                s_up[lr * 4 + (seg >> 2)] = in ? (uint8_t)us : 0;
            }
            if (in) {
                const uint64_t at = r * pitch + c;
                *reinterpret_cast<uint2*>(gate8.codes + at) = make_uint2(gc[0], gc[1]);
                *reinterpret_cast<uint2*>(up8.codes + at) = make_uint2(uc[0], uc[1]);
            }
        }
        if constexpr (!FAST) {
            __syncthreads();
            store_stage(s_h, h, ldh, r0 + i0, rows, c0, cols, t);
        }
    }
}

template <int FMT, int ROWS>
__global__ void __launch_bounds__(kThreadsMx, 4) k_mx_swiglu(Rows gate, Rows up, uint64_t rows, uint64_t cols,
                                                             uint32_t col_tiles, int lines, Form gate8, Form up8,
                                                             uint16_t* h, uint64_t ldh)
{
    __shared__ Stage s_h[ROWS > 32 ? 2 : 1];
    __shared__ alignas(16) uint8_t s_gate[ROWS * 4], s_up[ROWS * 4];
    ez::grid_dep_launch();
    const uint32_t t = threadIdx.x;
    const uint32_t piece = blockIdx.x / col_tiles, ct = blockIdx.x - piece * col_tiles;
    const uint64_t r0 = (uint64_t)piece * ROWS, c0 = (uint64_t)ct * kTileCols;
    ez::grid_dep_wait();
    if (lines && r0 + ROWS <= rows && c0 + kTileCols <= cols)
        swiglu_piece<FMT, ROWS, true>(gate, up, rows, cols, gate8, up8, h, ldh, r0, c0, s_h, s_gate, s_up);
    else
        swiglu_piece<FMT, ROWS, false>(gate, up, rows, cols, gate8, up8, h, ldh, r0, c0, s_h, s_gate, s_up);
    __syncthreads();
    const uint64_t tile = r0 / kTileRows * col_tiles + ct;
    const uint32_t lr = (uint32_t)(r0 % kTileRows);
    if (t < ROWS)
        *scale_word(gate8.scales, tile, lr + t) = reinterpret_cast<const uint32_t*>(s_gate)[t];
    else if (t < 2 * ROWS)
        *scale_word(up8.scales, tile, lr + t - ROWS) = reinterpret_cast<const uint32_t*>(s_up)[t - ROWS];
}

struct Grads {
    uint16_t *dgate, *dup, *h;
    uint64_t ldg, ldu, ldh;
};

template <int FMT, bool H, int ROWS, bool FAST>
__device__ __forceinline__ void swiglu_back_piece(Form gate8, Form up8, uint64_t rows, uint64_t cols, const Rows& dh,
                                                  const Grads& out, uint64_t r0, uint64_t c0, Stage* s_out,
                                                  const uint8_t* s_gate, const uint8_t* s_up)
{
    const uint32_t t = threadIdx.x, seg = t & 15u;
    const uint64_t c = c0 + 8 * seg, pitch = code_pitch<FMT>(cols);
    const bool block_in = FAST || c / kBlock * kBlock < cols;
#pragma unroll 1
    for (int i0 = 0; i0 < ROWS; i0 += 32) {
        uint2 gc[2], uc[2];
        Load8<FAST> din[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint64_t r = r0 + i0 + (t >> 4) + kRowStep * i;
            gc[i] = uc[i] = make_uint2(0u, 0u);
            if (FAST || (block_in && r < rows)) {
                const uint64_t at = r * pitch + c;
                gc[i] = __ldg(reinterpret_cast<const uint2*>(gate8.codes + at));
                uc[i] = __ldg(reinterpret_cast<const uint2*>(up8.codes + at));
            }
            din[i].start(dh, r, c, r < rows ? cols : 0);
        }
        const uint4 d[2] = {din[0].finish(), din[1].finish()};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t lr = i0 + (t >> 4) + kRowStep * i, at = lr * 4 + (seg >> 2);
            const uint64_t r = r0 + lr;
            const float gs = scale_value(s_gate[at]), us = scale_value(s_up[at]);
            const uint32_t gw[2] = {gc[i].x, gc[i].y}, uw[2] = {uc[i].x, uc[i].y};
            const uint32_t dw[4] = {d[i].x, d[i].y, d[i].z, d[i].w};
            float g[8], u[8], dg[8], du[8], hv[8];
            decode8<FMT>(gw, g);
            decode8<FMT>(uw, u);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float gj = g[j] * gs, uj = u[j] * us, dj = (j & 1) ? hi_f(dw[j >> 1]) : lo_f(dw[j >> 1]);
                const float p = logistic(gj), a = gj * p;
                dg[j] = dj * uj * p * (1.f + gj * (1.f - p));
                du[j] = dj * a;
                hv[j] = a * uj;
            }
            const uint4 y[3] = {make_uint4(bf16x2(dg[0], dg[1]), bf16x2(dg[2], dg[3]), bf16x2(dg[4], dg[5]),
                                           bf16x2(dg[6], dg[7])),
                                make_uint4(bf16x2(du[0], du[1]), bf16x2(du[2], du[3]), bf16x2(du[4], du[5]),
                                           bf16x2(du[6], du[7])),
                                make_uint4(bf16x2(hv[0], hv[1]), bf16x2(hv[2], hv[3]), bf16x2(hv[4], hv[5]),
                                           bf16x2(hv[6], hv[7]))};
            if constexpr (FAST) {
                *reinterpret_cast<uint4*>(out.dgate + r * out.ldg + c) = y[0];
                *reinterpret_cast<uint4*>(out.dup + r * out.ldu + c) = y[1];
                if constexpr (H) *reinterpret_cast<uint4*>(out.h + r * out.ldh + c) = y[2];
            } else {
#pragma unroll
                for (int k = 0; k < (H ? 3 : 2); ++k) s_out[k].row[lr & 31u][seg] = y[k];
            }
        }
        if constexpr (!FAST) {
            __syncthreads();
            store_stage(s_out[0], out.dgate, out.ldg, r0 + i0, rows, c0, cols, t);
            store_stage(s_out[1], out.dup, out.ldu, r0 + i0, rows, c0, cols, t);
            if constexpr (H) store_stage(s_out[2], out.h, out.ldh, r0 + i0, rows, c0, cols, t);
            __syncthreads();
        }
    }
}

template <int FMT, bool H, int ROWS>
__global__ void __launch_bounds__(kThreadsMx, 4) k_mx_swiglu_backward(Form gate8, Form up8, uint64_t rows,
                                                                      uint64_t cols, uint32_t col_tiles, int lines,
                                                                      Rows dh, Grads out)
{
    __shared__ Stage s_out[H ? 3 : 2];
    __shared__ uint32_t s_gate[ROWS], s_up[ROWS];
    ez::grid_dep_launch();
    const uint32_t t = threadIdx.x;
    const uint32_t piece = blockIdx.x / col_tiles, ct = blockIdx.x - piece * col_tiles;
    const uint64_t r0 = (uint64_t)piece * ROWS, c0 = (uint64_t)ct * kTileCols;
    const uint64_t tile = r0 / kTileRows * col_tiles + ct;
    const uint32_t lr = (uint32_t)(r0 % kTileRows);
    ez::grid_dep_wait();
    if (t < ROWS)
        s_gate[t] = *scale_word(gate8.scales, tile, lr + t);
    else if (t < 2 * ROWS)
        s_up[t - ROWS] = *scale_word(up8.scales, tile, lr + t - ROWS);
    __syncthreads();
    const uint8_t *gs = reinterpret_cast<const uint8_t*>(s_gate), *us = reinterpret_cast<const uint8_t*>(s_up);
    if (lines && r0 + ROWS <= rows && c0 + kTileCols <= cols)
        swiglu_back_piece<FMT, H, ROWS, true>(gate8, up8, rows, cols, dh, out, r0, c0, s_out, gs, us);
    else
        swiglu_back_piece<FMT, H, ROWS, false>(gate8, up8, rows, cols, dh, out, r0, c0, s_out, gs, us);
}

namespace {

// as in the quantisation: 128 rows per CTA, or 32 when that leaves SMs idle
bool many(uint64_t rows, uint64_t cols)
{
    return ez::cdiv(rows, kTileRows) * ez::cdiv(cols, kTileCols) >= 4ull * sm_count();
}

template <int FMT, int ROWS>
cudaError_t forward(const Rows& g, const Rows& u, uint64_t rows, uint64_t cols, Form g8, Form u8, uint16_t* h,
                    uint64_t ldh, cudaStream_t s)
{
    const uint64_t col_tiles = ez::cdiv(cols, kTileCols);
    // whole scale tiles: every piece of the last one is there to clear its bytes
    const uint64_t pieces = ez::cdiv(rows, kTileRows) * (kTileRows / ROWS);
    const int lines = lined(g.p, rows, g.ld) && lined(u.p, rows, u.ld) && lined(h, rows, ldh);
    return ez::launch_dependent(k_mx_swiglu<FMT, ROWS>, (unsigned)(pieces * col_tiles), kThreadsMx, 0, s, g, u, rows,
                                cols, (uint32_t)col_tiles, lines, g8, u8, h, ldh);
}

template <int FMT, bool H, int ROWS>
cudaError_t backward(Form g8, Form u8, uint64_t rows, uint64_t cols, const Rows& dh, const Grads& out, cudaStream_t s)
{
    const uint64_t col_tiles = ez::cdiv(cols, kTileCols), pieces = ez::cdiv(rows, ROWS);
    const int lines = lined(dh.p, rows, dh.ld) && lined(out.dgate, rows, out.ldg) &&
                      lined(out.dup, rows, out.ldu) && (!H || lined(out.h, rows, out.ldh));
    return ez::launch_dependent(k_mx_swiglu_backward<FMT, H, ROWS>, (unsigned)(pieces * col_tiles), kThreadsMx, 0, s,
                                g8, u8, rows, cols, (uint32_t)col_tiles, lines, dh, out);
}

template <int FMT>
cudaError_t backward(Form g8, Form u8, uint64_t rows, uint64_t cols, const Rows& dh, const Grads& out, cudaStream_t s)
{
    if (many(rows, cols))
        return out.h ? backward<FMT, true, 128>(g8, u8, rows, cols, dh, out, s)
                     : backward<FMT, false, 128>(g8, u8, rows, cols, dh, out, s);
    return out.h ? backward<FMT, true, 32>(g8, u8, rows, cols, dh, out, s)
                 : backward<FMT, false, 32>(g8, u8, rows, cols, dh, out, s);
}

}  // namespace

cudaError_t launch_mx_swiglu(int fmt, const uint16_t* gate, uint64_t ldg, const uint16_t* up, uint64_t ldu,
                             uint64_t rows, uint64_t cols, uint8_t* gate_codes, uint8_t* gate_scales,
                             uint8_t* up_codes, uint8_t* up_scales, uint16_t* h, uint64_t ldh, cudaStream_t s)
{
    if (!rows || !cols) return cudaSuccess;
    const Rows g = make_rows(gate, rows, cols, ldg), u = make_rows(up, rows, cols, ldu);
    const Form g8{gate_codes, gate_scales}, u8{up_codes, up_scales};
    if (fmt == EZ_MX_E4M3)
        return many(rows, cols) ? forward<EZ_MX_E4M3, 128>(g, u, rows, cols, g8, u8, h, ldh, s)
                                : forward<EZ_MX_E4M3, 32>(g, u, rows, cols, g8, u8, h, ldh, s);
    return many(rows, cols) ? forward<EZ_MX_E5M2, 128>(g, u, rows, cols, g8, u8, h, ldh, s)
                            : forward<EZ_MX_E5M2, 32>(g, u, rows, cols, g8, u8, h, ldh, s);
}

cudaError_t launch_mx_swiglu_backward(int fmt, const uint8_t* gate_codes, const uint8_t* gate_scales,
                                      const uint8_t* up_codes, const uint8_t* up_scales, uint64_t rows,
                                      uint64_t cols, const uint16_t* dh, uint64_t lddh, uint16_t* dgate,
                                      uint64_t ldg, uint16_t* dup, uint64_t ldu, uint16_t* h, uint64_t ldh,
                                      cudaStream_t s)
{
    if (!rows || !cols) return cudaSuccess;
    const Rows d = make_rows(dh, rows, cols, lddh);
    const Form g8{const_cast<uint8_t*>(gate_codes), const_cast<uint8_t*>(gate_scales)};
    const Form u8{const_cast<uint8_t*>(up_codes), const_cast<uint8_t*>(up_scales)};
    const Grads out{dgate, dup, h, ldg, ldu, ldh};
    return fmt == EZ_MX_E4M3 ? backward<EZ_MX_E4M3>(g8, u8, rows, cols, d, out, s)
                             : backward<EZ_MX_E5M2>(g8, u8, rows, cols, d, out, s);
}

}  // namespace ezk
