// k_mx_matmul.cu -- C = A B^T of two microscaled matrices on the tensor cores
// (tcgen05 block-scaled products).
//
// One operand, P, gives tiles of 128 rows (the tensor core's lanes), the
// other, Q, tiles of NT rows (its columns); a CTA computes D[p, q] = sum_k
// P[p, k] Q[q, k] in tensor memory.  Normally P = A and Q = B; swapped, P = B
// and Q = A, so that a few rows of A fill the narrow side of the product and
// lanes run along C's rows, which are then stored in whole lines at any
// alignment.
//
// Warp 0 loads (TMA): a stage is 128 bytes of codes of every row (256 E2M1 or
// 128 8-bit values) and its scale tiles; warp 1 copies the scales to tensor
// memory and issues the products; warps 2..5 take finished tiles out.  The
// scales are stored in the order tensor memory wants, 512 bytes for 128 rows x
// 128 values, so they go there by bulk copy without being touched.  Every
// stage has its own columns for them: a stage's scales are written only after
// its barrier says that the products that read the last ones are done.
//
// Values past K are codes 0 (the code rows end with the last block and TMA
// fills zeros) with scale bytes 0 inside the last scale tile; products past
// the last scale tile are not issued, because what tensor memory holds there
// could be the byte of a NaN.  Rows past the end only reach results that are
// not stored.
#include "ez_internal.h"
#include "ez_mx.cuh"
#include "ez_tc.cuh"

namespace ezk {
using namespace ezmx;
using namespace eztc;

namespace {

constexpr int kMmaThreads = 192;     // 6 warps
constexpr uint32_t kMaxStages = 8;

template <int BITS, int NT>
struct Shape {
    static constexpr int kAtoms = BITS == 4 ? 2 : 1;          // scale tiles per stage and 128 rows
    static constexpr int kQTiles = NT > 128 ? 2 : 1;
    static constexpr int kStages = NT > 128 ? 4 : NT > 64 ? 6 : 5;
    static constexpr int kAcc = NT > 128 ? 1 : 2;             // accumulators
    static constexpr uint32_t kP = 128 * 128, kQ = NT * 128;  // code bytes of a stage
    static constexpr uint32_t kScaleP = kAtoms * 512, kScaleQ = kQTiles * kAtoms * 512;
    static constexpr uint32_t kStage = kP + kQ;
    static constexpr uint32_t kSmem = kStages * (kStage + kScaleP + kScaleQ) + 1024;
    static constexpr uint32_t kScaleCols = (kScaleP + kScaleQ) / 128;   // tensor memory columns per stage
    static constexpr uint32_t kCols = kAcc * (NT < 32 ? 32 : NT) + kStages * kScaleCols;
    static constexpr uint32_t kAlloc = kCols <= 64 ? 64 : kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
    static_assert(kCols <= 512 && kStages <= (int)kMaxStages, "tensor memory");
};

struct MmaArgs {
    const uint8_t *p_scales, *q_scales;
    uint32_t p_rows, q_rows;
    uint32_t p_tiles, q_tiles;
    uint32_t stages, scale_tiles;   // along K
    uint32_t idesc;
    uint32_t f32;
    const float* add;
    void* c;
    uint64_t ldc;
    uint32_t* status;
};

// P tiles in groups of 16, Q tiles inside a group: the CTAs at work at one
// time share few distinct rows of either operand
__device__ __forceinline__ void tile_of(uint32_t t, const MmaArgs& a, uint32_t& tp, uint32_t& tq)
{
    const uint32_t per = 16 * a.q_tiles, g = t / per, in = t - g * per;
    const uint32_t rows = min(16u, a.p_tiles - g * 16);
    tq = in / rows;
    tp = g * 16 + in - tq * rows;
}

__device__ __forceinline__ void store_c(const MmaArgs& a, uint64_t at, float v)
{
    if (a.f32)
        static_cast<float*>(a.c)[at] = a.add ? v + a.add[at] : v;
    else
        static_cast<uint16_t*>(a.c)[at] = (uint16_t)bf16x2(v, 0.f);
}

__device__ __forceinline__ void st_v8(void* p, const uint32_t* w)
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 :: "l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

}  // namespace

template <int BITS, int NT, bool SWAP, bool SPLIT>
__global__ void __launch_bounds__(kMmaThreads) k_mx_matmul(const __grid_constant__ CUtensorMap p_map,
                                                           const __grid_constant__ CUtensorMap q_map,
                                                           const MmaArgs a)
{
    using S = Shape<BITS, NT>;
    extern __shared__ uint8_t s_raw[];
    __shared__ unsigned long long s_full[S::kStages], s_empty[S::kStages], s_done[2], s_free[2], s_drain;
    __shared__ uint32_t s_tmem, s_abort;
    const uint32_t base = (smem_u32(s_raw) + 1023u) & ~1023u;
    uint8_t* const raw = s_raw + (base - smem_u32(s_raw));
    constexpr uint32_t kScaleBase = S::kStages * S::kStage, kScaleStage = S::kScaleP + S::kScaleQ;
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kStages; ++i) {
            ez::mbar_init(&s_full[i], 1);
            ez::mbar_init(&s_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            ez::mbar_init(&s_done[i], 1);
            ez::mbar_init(&s_free[i], 4);
        }
        ez::mbar_init(&s_drain, 1);
        s_abort = 0;
        ez::mbar_fence_init();
        if (a.stages) {
            prefetch_map(&p_map);
            prefetch_map(&q_map);
        }
    }
    if (warp == 1) tmem_alloc(&s_tmem, S::kAlloc);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = s_tmem, scale_cols = tmem + S::kAcc * (NT < 32 ? 32 : NT);

    const uint32_t tiles = a.p_tiles * a.q_tiles;
    uint32_t t0 = blockIdx.x, step = gridDim.x, k0 = 0, k1 = a.stages, split = 1, rank = 0;
    if constexpr (SPLIT) {
        asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(split));
        rank = cluster_rank();
        t0 = blockIdx.x / split;
        step = tiles;                       // one tile
        k0 = (uint32_t)((uint64_t)a.stages * rank / split);
        k1 = (uint32_t)((uint64_t)a.stages * (rank + 1) / split);
    }
    auto gave_up = [&] {
        atomicExch(&s_abort, 1u);
        atomicOr(a.status, EZ_DSTAT_TIMEOUT);
    };

    if (warp == 0) {
        if (lane == 0) {
            uint32_t n = 0;                 // stages loaded
            bool ok = true;
            for (uint32_t t = t0; t < tiles && ok; t += step) {
                uint32_t tp, tq;
                tile_of(t, a, tp, tq);
                const bool second = S::kQTiles == 2 && tq * NT + 128 < a.q_rows;
                for (uint32_t k = k0; k < k1; ++k, ++n) {
                    const uint32_t s = n % S::kStages;
                    if (n >= S::kStages && !wait(&s_empty[s], (n / S::kStages - 1) & 1, &s_abort)) {
                        ok = false;
                        break;
                    }
                    const uint32_t atoms = min((uint32_t)S::kAtoms, a.scale_tiles - k * S::kAtoms);
                    ez::mbar_arrive_expect_tx(&s_full[s], S::kStage + atoms * 512 * (second ? 3 : 2));
                    const uint32_t st = base + s * S::kStage;
                    tma_2d(st, &p_map, k * 128, tp * 128, &s_full[s]);
                    tma_2d(st + S::kP, &q_map, k * 128, tq * NT, &s_full[s]);
                    uint8_t* sc = raw + kScaleBase + s * kScaleStage;
                    const uint64_t kt = (uint64_t)k * S::kAtoms;
                    ez::bulk_g2s(sc, a.p_scales + ((uint64_t)tp * a.scale_tiles + kt) * 512, atoms * 512, &s_full[s]);
                    const uint64_t qt = (uint64_t)tq * NT / 128;
                    ez::bulk_g2s(sc + S::kScaleP, a.q_scales + (qt * a.scale_tiles + kt) * 512, atoms * 512,
                                 &s_full[s]);
                    if (second)
                        ez::bulk_g2s(sc + S::kScaleP + S::kAtoms * 512,
                                     a.q_scales + ((qt + 1) * a.scale_tiles + kt) * 512, atoms * 512, &s_full[s]);
                }
            }
            if (!ok) {
                gave_up();
                // copies in flight end before shared memory goes away
                for (uint32_t i = n > S::kStages ? n - S::kStages : 0; i < n; ++i)
                    wait(&s_full[i % S::kStages], (i / S::kStages) & 1, nullptr);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            uint32_t n = 0, j = 0;          // stages and tiles
            bool ok = true;
            for (uint32_t t = t0; t < tiles && ok; t += step, ++j) {
                const uint32_t buf = j % S::kAcc, d = tmem + buf * (NT < 32 ? 32 : NT);
                if (j >= S::kAcc && !wait(&s_free[buf], (j / S::kAcc - 1) & 1, &s_abort)) {
                    ok = false;
                    break;
                }
                fence_after();
                for (uint32_t k = k0; k < k1; ++k, ++n) {
                    const uint32_t s = n % S::kStages;
                    if (!wait(&s_full[s], (n / S::kStages) & 1, &s_abort)) {
                        ok = false;
                        break;
                    }
                    fence_after();
                    const uint32_t atoms = min((uint32_t)S::kAtoms, a.scale_tiles - k * S::kAtoms);
                    const uint32_t sc = base + kScaleBase + s * kScaleStage;
                    const uint32_t tp = scale_cols + s * S::kScaleCols, tq = tp + S::kAtoms * 4;
                    for (uint32_t i = 0; i < atoms; ++i) {
                        copy_scales(tp + i * 4, desc_scales(sc + i * 512));
#pragma unroll
                        for (uint32_t h = 0; h < (uint32_t)S::kQTiles; ++h)
                            copy_scales(tq + (i * S::kQTiles + h) * 4,
                                        desc_scales(sc + S::kScaleP + (h * S::kAtoms + i) * 512));
                    }
                    const uint64_t dp = desc_rows(base + s * S::kStage), dq = desc_rows(base + s * S::kStage + S::kP);
#pragma unroll
                    for (uint32_t i = 0; i < 4; ++i) {
                        const uint32_t atom = BITS == 4 ? i / 2 : 0, id = BITS == 4 ? (i % 2) * 2 : i;
                        if (atom < atoms)
                            mma<BITS>(d, dp + 2 * i, dq + 2 * i, a.idesc | scale_ids(id), tp + atom * 4,
                                      tq + atom * 4 * S::kQTiles, (k > k0 || i > 0) ? 1u : 0u);
                    }
                    commit(&s_empty[s]);
                }
                if (ok && k1 > k0) commit(&s_done[buf]);
            }
            if (!ok) {
                gave_up();
                commit(&s_drain);
                wait(&s_drain, 0, nullptr);
            }
        }
    } else {
        const uint32_t quarter = warp % 4, row = quarter * 32 + lane;
        uint32_t j = 0;
        for (uint32_t t = t0; t < tiles; t += step, ++j) {
            uint32_t tp, tq;
            tile_of(t, a, tp, tq);
            const uint32_t buf = j % S::kAcc, d = tmem + buf * (NT < 32 ? 32 : NT) + (quarter << 21);
            const bool have = k1 > k0;
            // every lane takes part in the loads below: the vote makes the wait's outcome the warp's
            if (have && !__all_sync(ez::kFull, wait(&s_done[buf], (j / S::kAcc) & 1, &s_abort))) {
                if (lane == 0) gave_up();
                break;
            }
            fence_after();
            const uint64_t p = (uint64_t)tp * 128 + row;
            constexpr int kChunk = NT < 32 ? 16 : 32;
#pragma unroll 1
            for (uint32_t q0 = 0; q0 < NT; q0 += kChunk) {
                uint32_t r[kChunk];
                if (have) {
                    if constexpr (kChunk == 16)
                        tmem_load16(d + q0, r);
                    else
                        tmem_load32(d + q0, r);
                    tmem_wait_load();
                } else {
#pragma unroll
                    for (int i = 0; i < kChunk; ++i) r[i] = 0u;
                }
                if (q0 + kChunk == NT) {
                    fence_before();
                    __syncwarp();
                    if (lane == 0) ez::mbar_arrive(&s_free[buf]);
                }
                const uint64_t q = (uint64_t)tq * NT + q0;
                if constexpr (SPLIT) {
                    float* part = reinterpret_cast<float*>(raw);
#pragma unroll
                    for (int i = 0; i < kChunk; ++i) part[(q0 + i) * 128 + row] = __uint_as_float(r[i]);
                } else if (p < a.p_rows) {
                    if constexpr (SWAP) {
#pragma unroll
                        for (int i = 0; i < kChunk; ++i)
                            if (q + i < a.q_rows) store_c(a, (q + i) * a.ldc + p, __uint_as_float(r[i]));
                    } else if (q + kChunk <= a.q_rows) {
                        const uint64_t at = p * a.ldc + q;
                        if (a.f32) {
                            float* c = static_cast<float*>(a.c) + at;
                            if (a.add) {
                                const float4* e = reinterpret_cast<const float4*>(a.add + at);
#pragma unroll
                                for (int i = 0; i < kChunk / 4; ++i) {
                                    const float4 v = e[i];
                                    r[4 * i] = __float_as_uint(__uint_as_float(r[4 * i]) + v.x);
                                    r[4 * i + 1] = __float_as_uint(__uint_as_float(r[4 * i + 1]) + v.y);
                                    r[4 * i + 2] = __float_as_uint(__uint_as_float(r[4 * i + 2]) + v.z);
                                    r[4 * i + 3] = __float_as_uint(__uint_as_float(r[4 * i + 3]) + v.w);
                                }
                            }
#pragma unroll
                            for (int i = 0; i < kChunk / 8; ++i) st_v8(c + 8 * i, r + 8 * i);
                        } else {
                            uint32_t w[kChunk / 2];
#pragma unroll
                            for (int i = 0; i < kChunk / 2; ++i)
                                w[i] = bf16x2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
                            uint16_t* c = static_cast<uint16_t*>(a.c) + at;
#pragma unroll
                            for (int i = 0; i < kChunk / 16; ++i) st_v8(c + 16 * i, w + 8 * i);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < kChunk; ++i)
                            if (q + i < a.q_rows) store_c(a, p * a.ldc + q + i, __uint_as_float(r[i]));
                    }
                }
            }
        }
    }
    __syncwarp();
    if constexpr (SPLIT) {
        // the parts of all CTAs of the cluster, added in the order of their ranks
        cluster_sync();
        uint32_t tp, tq;
        tile_of(t0, a, tp, tq);
        const uint32_t n = min((uint32_t)NT, a.q_rows - tq * NT), rows = min(128u, a.p_rows - tp * 128);
        const uint32_t part = base;
        for (uint32_t i = rank * kMmaThreads + threadIdx.x; i < n * 128; i += split * kMmaThreads) {
            const uint32_t q = i / 128, row = i % 128;
            if (row >= rows) continue;
            float v = 0.f;
            for (uint32_t s = 0; s < split; ++s) v += peer_load(part + i * 4, s);
            store_c(a, ((uint64_t)tq * NT + q) * a.ldc + (uint64_t)tp * 128 + row, v);
        }
        cluster_sync();
    }
    fence_before();
    __syncthreads();
    if (warp == 1) {
        fence_after();
        tmem_free(tmem, S::kAlloc);
    }
}

namespace {

using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                            const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                            CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

Encode encoder()
{
    static const Encode fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) !=
                cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<Encode>(f);
    }();
    return fn;
}

// Code rows as a 2-D byte matrix read in boxes of 128 bytes x box_rows, zeros outside.
bool code_map(CUtensorMap* m, const uint8_t* codes, uint64_t rows, uint64_t pitch, uint32_t box_rows)
{
    const Encode fn = encoder();
    if (!fn) return false;
    const cuuint64_t dims[2] = {pitch, rows}, strides[1] = {pitch};
    const cuuint32_t box[2] = {128, box_rows}, one[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(codes), dims, strides, box, one,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

uint32_t type_of(int fmt) { return fmt == EZ_MX_E4M3 ? 0u : 1u; }   // E2M1 and E5M2 are 1 in their kinds

struct Operand {
    int fmt;
    const uint8_t *codes, *scales;
    uint64_t rows;
};

template <int BITS, int NT, bool SWAP, bool SPLIT>
cudaError_t go(const Operand& p, const Operand& q, uint64_t K, MmaArgs a, uint32_t sms, uint32_t split, cudaStream_t s)
{
    using S = Shape<BITS, NT>;
    CUtensorMap pm{}, qm{};
    const uint64_t nb = ez::cdiv(K, 32), pitch = nb * (BITS * 4);
    a.p_scales = p.scales;
    a.q_scales = q.scales;
    a.p_rows = (uint32_t)p.rows;
    a.q_rows = (uint32_t)q.rows;
    a.p_tiles = (uint32_t)ez::cdiv(p.rows, 128);
    a.q_tiles = (uint32_t)ez::cdiv(q.rows, NT);
    a.scale_tiles = (uint32_t)ez::cdiv(nb, 4);
    a.stages = (uint32_t)ez::cdiv(a.scale_tiles, S::kAtoms);
    a.idesc = instr_desc(type_of(p.fmt), type_of(q.fmt), 128, NT);
    if (K && (!code_map(&pm, p.codes, p.rows, pitch, 128) || !code_map(&qm, q.codes, q.rows, pitch, NT)))
        return cudaErrorUnknown;
    auto kernel = k_mx_matmul<BITS, NT, SWAP, SPLIT>;
    static const cudaError_t set =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (set != cudaSuccess) return set;
    const uint64_t tiles = (uint64_t)a.p_tiles * a.q_tiles;
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(kMmaThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr{};
    if (SPLIT) {
        cfg.gridDim = dim3((unsigned)(tiles * split));
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = split;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
    } else {
        cfg.gridDim = dim3((unsigned)ez::umin64(tiles, sms));
    }
    return cudaLaunchKernelEx(&cfg, kernel, pm, qm, a);
}

template <int BITS>
cudaError_t choose(const Operand& A, const Operand& B, uint64_t K, const MmaArgs& a, uint32_t sms, cudaStream_t s)
{
    // swapped: few rows of A, or rows of C that are not on 32-byte boundaries
    const uint64_t row_bytes = a.ldc * (a.f32 ? 4 : 2);
    const bool lined = ((reinterpret_cast<uintptr_t>(a.c) | reinterpret_cast<uintptr_t>(a.add) | row_bytes) & 31u) == 0;
    const uint64_t stages = ez::cdiv(ez::cdiv(K, 128), BITS == 4 ? 2 : 1);
    if (A.rows <= 128) {
        const uint64_t tiles = ez::cdiv(B.rows, 128);
        uint32_t split = 1;
        while (split < 8 && tiles * split * 2 <= 2 * sms && stages >= 4 * split) split *= 2;
        if (A.rows <= 16) return go<BITS, 16, true, true>(B, A, K, a, sms, split, s);
        if (A.rows <= 32) return go<BITS, 32, true, true>(B, A, K, a, sms, split, s);
        if (A.rows <= 64) return go<BITS, 64, true, true>(B, A, K, a, sms, split, s);
        return go<BITS, 128, true, true>(B, A, K, a, sms, split, s);
    }
    const bool wide = ez::cdiv(A.rows, 128) * ez::cdiv(B.rows, 256) >= sms;
    if (!lined) {
        return wide ? go<BITS, 256, true, false>(B, A, K, a, sms, 1, s) : go<BITS, 128, true, false>(B, A, K, a, sms, 1, s);
    }
    return wide ? go<BITS, 256, false, false>(A, B, K, a, sms, 1, s) : go<BITS, 128, false, false>(A, B, K, a, sms, 1, s);
}

}  // namespace

cudaError_t launch_mx_matmul(int fa, const uint8_t* ac, const uint8_t* as, uint64_t M, int fb, const uint8_t* bc,
                             const uint8_t* bs, uint64_t N, uint64_t K, const float* add, void* c, uint64_t ldc,
                             int f32, uint32_t* status, cudaStream_t s)
{
    if (!M || !N) return cudaSuccess;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const Operand A{fa, ac, as, M}, B{fb, bc, bs, N};
    MmaArgs a{};
    a.f32 = (uint32_t)f32;
    a.add = add;
    a.c = c;
    a.ldc = ldc;
    a.status = status;
    return fa == EZ_MX_E2M1 ? choose<4>(A, B, K, a, (uint32_t)sms, s) : choose<8>(A, B, K, a, (uint32_t)sms, s);
}

}  // namespace ezk
