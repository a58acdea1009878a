// k_mx_gated.cu -- the gated unit h = silu(g) u that keeps g and u in 8 bits,
// and its backward pass from what was kept.
//
// With s = 1 / (1 + exp(-g)):  h = g s u,  du = dh g s,
// dg = dh u s (1 + g (1 - s)).
#include "ez_internal.h"
#include "ez_mx.cuh"

namespace ezk {
using namespace ezmx;

__device__ __forceinline__ float logistic(float g) { return __fdividef(1.f, 1.f + __expf(-g)); }

template <int FMT>
__global__ void __launch_bounds__(kThreadsMx) k_mx_swiglu(Rows gate, Rows up, uint64_t rows, uint64_t cols,
                                                          Form gate8, Form up8, uint16_t* h, uint64_t ldh)
{
    __shared__ uint4 s_gate[32], s_up[32];
    const uint32_t t = threadIdx.x, seg = t & 15u;
    const uint64_t col_tiles = ez::cdiv(cols, kTileCols);
    const uint64_t rt = blockIdx.x / col_tiles, ct = blockIdx.x - rt * col_tiles;
    const uint64_t c = ct * kTileCols + 8 * seg;
    constexpr int kStep = 4;      // rows in flight per thread
#pragma unroll
    for (int i0 = 0; i0 < kRowIters; i0 += kStep) {
        uint4 g[kStep], u[kStep];
#pragma unroll
        for (int i = 0; i < kStep; ++i) {
            const uint64_t r = rt * kTileRows + (t >> 4) + kRowStep * (i0 + i);
            g[i] = load8(gate, r, c, r < rows ? cols : 0);
            u[i] = load8(up, r, c, r < rows ? cols : 0);
        }
#pragma unroll
        for (int i = 0; i < kStep; ++i) {
            const uint32_t lr = (t >> 4) + kRowStep * (i0 + i);
            const uint64_t r = rt * kTileRows + lr;
            const uint32_t gw[4] = {g[i].x, g[i].y, g[i].z, g[i].w}, uw[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
            uint32_t hw[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float g0 = lo_f(gw[j]), g1 = hi_f(gw[j]);
                hw[j] = bf16x2(g0 * logistic(g0) * lo_f(uw[j]), g1 * logistic(g1) * hi_f(uw[j]));
            }
            store8(h + r * ldh, seg, c, r < rows ? cols : 0, make_uint4(hw[0], hw[1], hw[2], hw[3]));
            uint32_t gc[2], uc[2];
            const uint32_t gs = quantise_quad<FMT>(g[i], gc), us = quantise_quad<FMT>(u[i], uc);
            const bool in = r < rows && c / kBlock * kBlock < cols;
            if ((t & 3u) == 0) {
                reinterpret_cast<uint8_t*>(s_gate)[scale_at(lr, seg >> 2)] = in ? (uint8_t)gs : 0;
                reinterpret_cast<uint8_t*>(s_up)[scale_at(lr, seg >> 2)] = in ? (uint8_t)us : 0;
            }
            if (in) {
                const uint64_t at = r * code_pitch<FMT>(cols) + c;
                *reinterpret_cast<uint2*>(gate8.codes + at) = make_uint2(gc[0], gc[1]);
                *reinterpret_cast<uint2*>(up8.codes + at) = make_uint2(uc[0], uc[1]);
            }
        }
    }
    __syncthreads();
    if (t < 32)
        reinterpret_cast<uint4*>(gate8.scales)[blockIdx.x * 32ull + t] = s_gate[t];
    else if (t < 64)
        reinterpret_cast<uint4*>(up8.scales)[blockIdx.x * 32ull + t - 32] = s_up[t - 32];
}

template <int FMT, bool H>
__global__ void __launch_bounds__(kThreadsMx) k_mx_swiglu_backward(Form gate8, Form up8, uint64_t rows,
                                                                   uint64_t cols, Rows dh, uint16_t* dgate,
                                                                   uint64_t ldg, uint16_t* dup, uint64_t ldu,
                                                                   uint16_t* h, uint64_t ldh)
{
    __shared__ uint4 s_gate[32], s_up[32];
    const uint32_t t = threadIdx.x, seg = t & 15u;
    const uint64_t col_tiles = ez::cdiv(cols, kTileCols);
    const uint64_t rt = blockIdx.x / col_tiles, ct = blockIdx.x - rt * col_tiles;
    const uint64_t c = ct * kTileCols + 8 * seg;
    if (t < 32)
        s_gate[t] = ez::ld_v4_nc(gate8.scales + (blockIdx.x * 32ull + t) * 16);
    else if (t < 64)
        s_up[t - 32] = ez::ld_v4_nc(up8.scales + (blockIdx.x * 32ull + t - 32) * 16);
    __syncthreads();
    constexpr int kStep = 4;
#pragma unroll
    for (int i0 = 0; i0 < kRowIters; i0 += kStep) {
        uint2 gc[kStep], uc[kStep];
        uint4 d[kStep];
#pragma unroll
        for (int i = 0; i < kStep; ++i) {
            const uint64_t r = rt * kTileRows + (t >> 4) + kRowStep * (i0 + i);
            gc[i] = uc[i] = make_uint2(0u, 0u);
            if (r < rows && c < cols) {
                const uint64_t at = r * code_pitch<FMT>(cols) + c;
                gc[i] = __ldg(reinterpret_cast<const uint2*>(gate8.codes + at));
                uc[i] = __ldg(reinterpret_cast<const uint2*>(up8.codes + at));
            }
            d[i] = load8(dh, r, c, r < rows ? cols : 0);
        }
#pragma unroll
        for (int i = 0; i < kStep; ++i) {
            const uint32_t lr = (t >> 4) + kRowStep * (i0 + i);
            const uint64_t r = rt * kTileRows + lr;
            const uint32_t at = scale_at(lr, seg >> 2);
            const float gs = scale_value(reinterpret_cast<const uint8_t*>(s_gate)[at]);
            const float us = scale_value(reinterpret_cast<const uint8_t*>(s_up)[at]);
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
            const uint64_t n = r < rows ? cols : 0;
            store8(dgate + r * ldg, seg, c, n, make_uint4(bf16x2(dg[0], dg[1]), bf16x2(dg[2], dg[3]),
                                                          bf16x2(dg[4], dg[5]), bf16x2(dg[6], dg[7])));
            store8(dup + r * ldu, seg, c, n, make_uint4(bf16x2(du[0], du[1]), bf16x2(du[2], du[3]),
                                                        bf16x2(du[4], du[5]), bf16x2(du[6], du[7])));
            if constexpr (H)
                store8(h + r * ldh, seg, c, n, make_uint4(bf16x2(hv[0], hv[1]), bf16x2(hv[2], hv[3]),
                                                          bf16x2(hv[4], hv[5]), bf16x2(hv[6], hv[7])));
        }
    }
}

namespace {
unsigned tiles(uint64_t rows, uint64_t cols)
{
    return (unsigned)(ez::cdiv(rows, kTileRows) * ez::cdiv(cols, kTileCols));
}
}  // namespace

cudaError_t launch_mx_swiglu(int fmt, const uint16_t* gate, uint64_t ldg, const uint16_t* up, uint64_t ldu,
                             uint64_t rows, uint64_t cols, uint8_t* gate_codes, uint8_t* gate_scales,
                             uint8_t* up_codes, uint8_t* up_scales, uint16_t* h, uint64_t ldh, cudaStream_t s)
{
    if (!rows || !cols) return cudaSuccess;
    const Rows g = make_rows(gate, rows, cols, ldg), u = make_rows(up, rows, cols, ldu);
    const Form g8{gate_codes, gate_scales}, u8{up_codes, up_scales};
    const unsigned grid = tiles(rows, cols);
    if (fmt == EZ_MX_E4M3)
        k_mx_swiglu<EZ_MX_E4M3><<<grid, kThreadsMx, 0, s>>>(g, u, rows, cols, g8, u8, h, ldh);
    else
        k_mx_swiglu<EZ_MX_E5M2><<<grid, kThreadsMx, 0, s>>>(g, u, rows, cols, g8, u8, h, ldh);
    return cudaGetLastError();
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
    const unsigned grid = tiles(rows, cols);
    auto run = [&](auto kernel) {
        kernel<<<grid, kThreadsMx, 0, s>>>(g8, u8, rows, cols, d, dgate, ldg, dup, ldu, h, ldh);
        return cudaGetLastError();
    };
    if (fmt == EZ_MX_E4M3)
        return h ? run(k_mx_swiglu_backward<EZ_MX_E4M3, true>) : run(k_mx_swiglu_backward<EZ_MX_E4M3, false>);
    return h ? run(k_mx_swiglu_backward<EZ_MX_E5M2, true>) : run(k_mx_swiglu_backward<EZ_MX_E5M2, false>);
}

}  // namespace ezk
