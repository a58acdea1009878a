// k_mx_matmul.cu -- C = A B^T of two microscaled matrices: a plain tiled
// kernel, 64 x 64 results per CTA, both operands decoded to FP32 in shared
// memory, FP32 sums.
#include "ez_internal.h"
#include "ez_mx.cuh"

namespace ezk {
using namespace ezmx;

namespace {
constexpr int kT = 64;
}

template <int FMT>
__device__ __forceinline__ void load_block(float (*s)[kT + 4], Form f, uint64_t row0, uint64_t rows, uint64_t cols,
                                           uint64_t kb)
{
    // 64 rows x 32 values: thread t decodes 8 values of row t / 4
    const uint32_t t = threadIdx.x, lr = t >> 2, q = t & 3u;
    const uint64_t r = row0 + lr;
    float v[8] = {};
    if (r < rows) {
        const uint8_t* p = f.codes + r * code_pitch<FMT>(cols) + (kb * 32 + q * 8) * Fmt<FMT>::kBits / 8;
        uint32_t w[2] = {reinterpret_cast<const uint32_t*>(p)[0], 0u};
        if (Fmt<FMT>::kBits == 8) w[1] = reinterpret_cast<const uint32_t*>(p)[1];
        decode8<FMT>(w, v);
        const uint64_t kt = ez::cdiv(ez::cdiv(cols, 32), 4);
        const float sc = scale_value(f.scales[(r / 128 * kt + kb / 4) * 512 + scale_at(r & 127, kb & 3)]);
        for (int i = 0; i < 8; ++i) v[i] *= sc;
    }
    for (int i = 0; i < 8; ++i) s[q * 8 + i][lr] = v[i];
}

template <int FA, int FB>
__global__ void __launch_bounds__(256) k_mx_matmul(Form a, uint64_t M, Form b, uint64_t N, uint64_t K,
                                                   const float* add, void* c, uint64_t ldc, int f32)
{
    __shared__ float sa[32][kT + 4], sb[32][kT + 4];
    const uint32_t t = threadIdx.x, tx = t & 15u, ty = t >> 4;
    const uint64_t nt = ez::cdiv(N, kT), m0 = blockIdx.x / nt * kT, n0 = blockIdx.x % nt * kT;
    float acc[4][4] = {};
    for (uint64_t kb = 0; kb < ez::cdiv(K, 32); ++kb) {
        load_block<FA>(sa, a, m0, M, K, kb);
        load_block<FB>(sb, b, n0, N, K, kb);
        __syncthreads();
#pragma unroll 8
        for (int k = 0; k < 32; ++k)
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j) acc[i][j] += sa[k][ty * 4 + i] * sb[k][tx * 4 + j];
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const uint64_t m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
            if (m >= M || n >= N) continue;
            const uint64_t at = m * ldc + n;
            const float v = add ? acc[i][j] + add[at] : acc[i][j];
            if (f32)
                static_cast<float*>(c)[at] = v;
            else
                static_cast<uint16_t*>(c)[at] = (uint16_t)bf16x2(v, 0.f);
        }
}

cudaError_t launch_mx_matmul(int fa, const uint8_t* ac, const uint8_t* as, uint64_t M, int fb, const uint8_t* bc,
                             const uint8_t* bs, uint64_t N, uint64_t K, const float* add, void* c, uint64_t ldc,
                             int f32, uint32_t* status, cudaStream_t s)
{
    (void)status;
    if (!M || !N) return cudaSuccess;
    const Form a{const_cast<uint8_t*>(ac), const_cast<uint8_t*>(as)}, b{const_cast<uint8_t*>(bc), const_cast<uint8_t*>(bs)};
    const unsigned grid = (unsigned)(ez::cdiv(M, kT) * ez::cdiv(N, kT));
    auto run = [&](auto kernel) {
        kernel<<<grid, 256, 0, s>>>(a, M, b, N, K, add, c, ldc, f32);
        return cudaGetLastError();
    };
    if (fa == EZ_MX_E2M1) return run(k_mx_matmul<EZ_MX_E2M1, EZ_MX_E2M1>);
    if (fa == EZ_MX_E4M3)
        return fb == EZ_MX_E4M3 ? run(k_mx_matmul<EZ_MX_E4M3, EZ_MX_E4M3>) : run(k_mx_matmul<EZ_MX_E4M3, EZ_MX_E5M2>);
    return fb == EZ_MX_E4M3 ? run(k_mx_matmul<EZ_MX_E5M2, EZ_MX_E4M3>) : run(k_mx_matmul<EZ_MX_E5M2, EZ_MX_E5M2>);
}

}  // namespace ezk
