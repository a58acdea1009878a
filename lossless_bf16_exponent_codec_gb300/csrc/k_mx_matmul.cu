// k_mx_matmul.cu -- C = A B^T of two microscaled matrices on the tensor cores
// (tcgen05 block-scaled products, FP32 sums in tensor memory).
//
// One operand, P, gives the rows of a tile (the tensor core's lanes), the
// other, Q, its columns: D[p, q] = sum_k P[p, k] Q[q, k].  Normally P = A and
// Q = B; swapped, P = B and Q = A, so that lanes run along C's rows, which are
// then stored in whole lines whatever their alignment, and a few rows of A
// make a narrow tile.  Two kernels: k_mx_split (tiles of 128 x up to 128, K cut
// over the CTAs of a cluster) for products with few tiles, k_mx_pair (tiles of
// 256 x up to 256 by pairs of CTAs, persistent) for the others.
//
// A stage of the load ring is 128 bytes of codes of every row (256 E2M1 or 128
// 8-bit values) and their scale tiles.  Scales are stored in the order tensor
// memory wants, 512 bytes for 128 rows x 128 values, so they go there by bulk
// copies without passing through registers.  One warp loads, one issues products
// (in a pair another copies the scales), the others take finished tiles out.
//
// Bounds, measured on one GB300: 8192 x 8192 x 8192 in 4 bits takes 151 us, 7.3
// PFLOP/s = 0.94 of four times the measured BF16 rate, tensor pipe 82% busy;
// what is left: 1200 of the 20800 cycles of a tile at its end, and stages whose
// 512 cycles of products take 600 beside their loads.  8192 x 4096 x 16384 in 8
// bits added to an FP32 matrix: 354 to 365 us, 3.0 to 3.1 PFLOP/s = 0.77 to 0.8 of
// twice the BF16 rate, bound by the FP32 matrix read and written, the ends of
// segments and, in a long run, the power limit.  One row times 8192 x 8192 in 4
// bits: 9.0 us, 4.0 TB/s with launch and the cluster's join in it.
//
// Values past K are codes 0 (the code rows end with the last block and TMA
// fills zeros) with scale bytes 0 inside the last scale tile; products past the
// last scale tile are not issued, because what tensor memory holds there could
// be the byte of a NaN.  Rows past the end only reach results that are not
// stored.
//
// Long sums: the tensor core cuts off what does not fit when it adds a product
// to an FP32 sum, so its error grows with the number of additions (3.4e-6 of
// the result after the 512 of K = 16384 in 8 bits).  When C is FP32 the sum is
// cut into segments of kSegment stages that are added in FP32 registers with
// correct rounding: 0.53e-6 then.  8192 x 4096 x 16384 takes 355 us with segments
// of 24 stages, 365 with 16 (0.35e-6, what FP32 arithmetic gives), 347 with 32
// (0.66e-6).  An addend joins such a sum in one addition.  For a C rounded to the 8 bits of BF16 a
// segment has kLongSegment stages, under a millisecond, so that no wait comes near
// its limit however long K is.
#include "ez_internal.h"
#include "ez_mx.cuh"
#include "ez_tc.cuh"

namespace ezk {
using namespace ezmx;
using namespace eztc;

namespace {

constexpr uint32_t kSegment = 24, kLongSegment = 1024;
constexpr uint32_t kPRows = 128, kPBytes = kPRows * 128;   // P rows of a CTA, code bytes of a stage
constexpr uint32_t kMaxSmem = 227 * 1024 - 1024;

struct MmaArgs {
    const uint8_t *p_scales, *q_scales;
    uint32_t p_rows, q_rows;
    uint32_t p_tiles, q_tiles;
    uint32_t nq;                    // Q rows of a tile
    uint32_t steps, scale_tiles;    // stages and scale tiles along K
    uint32_t segment;               // stages added up in tensor memory
    uint32_t ring;                  // stages in shared memory
    uint32_t cols;                  // tensor memory columns
    uint32_t slots;                 // scale slots in tensor memory
    uint32_t idesc;
    uint32_t f32, swap;
    uint32_t staged;                // C leaves by TMA (k_mx_pair)
    uint32_t limit;                 // polls of a wait before it gives up
    const float* add;
    void* c;
    uint64_t ldc;
    uint32_t* status;
};

// Tile t: P tiles in groups of `group`, Q tiles inside a group, so that the
// CTAs at work at one time share few distinct rows of either operand.
__device__ __forceinline__ void tile_of(uint32_t t, uint32_t group, const MmaArgs& a, uint32_t& tp, uint32_t& tq)
{
    const uint32_t per = group * a.q_tiles, g = t / per, in = t - g * per;
    const uint32_t rows = min(group, a.p_tiles - g * group);
    tq = in / rows;
    tp = g * group + in - tq * rows;
}

__device__ __forceinline__ void store_c(const MmaArgs& a, uint64_t at, float v)
{
    if (a.f32)
        static_cast<float*>(a.c)[at] = a.add ? v + a.add[at] : v;
    else
        static_cast<uint16_t*>(a.c)[at] = (uint16_t)bf16x2(v, 0.f);
}

// Position in a ring of stages: slot and the parity its barrier has next.
struct Ring {
    uint32_t slot = 0, parity = 0;
    __device__ __forceinline__ void next(uint32_t n)
    {
        if (++slot == n) {
            slot = 0;
            parity ^= 1u;
        }
    }
};

}  // namespace

// ---- few tiles: K over a cluster ---------------------------------------------------

constexpr int kSplitThreads = 192;
constexpr uint32_t kMaxRing = 12, kMaxSplit = 8, kPartPitch = kPRows + 4;

// Add the sums of the SPLIT CTAs of a cluster, in the order of their ranks, and
// store this CTA's part of the tile.  Eight loads are in flight per thread:
// one at a time, a tile of 128 x 128 spends 3 us on their latency.  Only what is
// added up is loaded, and a thread arrives at the cluster's last barrier (release)
// between its last loads and the stores they end in: a CTA that has seen all
// arrivals may end, with no read of its memory under way, and nobody waits for the
// last stores.  The release costs 0.1 to 0.5 us (128 x 4096 x 4096 in 4 bits 6.1 ->
// 6.6, one row times 8192 x 8192 8.9 -> 9.0); holding all sums in registers, so that
// no store comes before it, gained nothing.
template <int SPLIT>
__device__ __forceinline__ void join(const MmaArgs& a, uint32_t base, uint32_t rank, uint32_t tp, uint32_t tq)
{
    constexpr uint32_t kItems = 8 / SPLIT, kStep = SPLIT * kSplitThreads;
    const uint32_t n = min(a.nq, a.q_rows - tq * a.nq), rows = min(kPRows, a.p_rows - tp * kPRows);
    uint32_t peer[SPLIT];
#pragma unroll
    for (uint32_t s = 0; s < SPLIT; ++s) peer[s] = peer_addr(base, s);
    const uint32_t first = rank * kSplitThreads + threadIdx.x, items = n * (a.swap ? 32 : rows);
    bool told = SPLIT == 1;
    auto tell = [&](uint32_t i0) {
        if (!told && i0 + kItems * kStep >= items) {
            cluster_arrive();
            told = true;
        }
    };
    if (a.swap) {
        // four consecutive results of a row of C per thread
        for (uint32_t i0 = first; i0 < items; i0 += kItems * kStep) {
            float4 v[kItems][SPLIT];
#pragma unroll
            for (uint32_t u = 0; u < kItems; ++u) {
                const uint32_t i = i0 + u * kStep, r = i % 32 * 4, off = (i / 32 * kPartPitch + r) * 4;
                if (i >= items || r >= rows) continue;
#pragma unroll
                for (uint32_t s = 0; s < SPLIT; ++s) v[u][s] = peer_load4(peer[s] + off);
            }
            tell(i0);
#pragma unroll
            for (uint32_t u = 0; u < kItems; ++u) {
                const uint32_t i = i0 + u * kStep, q = i / 32, r = i % 32 * 4;
                if (i >= items || r >= rows) continue;
                float4 t = v[u][0];
#pragma unroll
                for (uint32_t s = 1; s < SPLIT; ++s)
                    t = make_float4(t.x + v[u][s].x, t.y + v[u][s].y, t.z + v[u][s].z, t.w + v[u][s].w);
                const uint64_t at = ((uint64_t)tq * a.nq + q) * a.ldc + (uint64_t)tp * kPRows + r;
                uint16_t* const c16 = static_cast<uint16_t*>(a.c) + at;
                float* const c32 = static_cast<float*>(a.c) + at;
                const float* const e = a.add ? a.add + at : nullptr;
                if (!a.f32 && r + 4 <= rows && (reinterpret_cast<uintptr_t>(c16) & 7u) == 0) {
                    *reinterpret_cast<uint2*>(c16) = make_uint2(bf16x2(t.x, t.y), bf16x2(t.z, t.w));
                } else if (a.f32 && r + 4 <= rows &&
                           ((reinterpret_cast<uintptr_t>(c32) | reinterpret_cast<uintptr_t>(e)) & 15u) == 0) {
                    const float4 d = e ? *reinterpret_cast<const float4*>(e) : make_float4(0.f, 0.f, 0.f, 0.f);
                    *reinterpret_cast<float4*>(c32) = make_float4(t.x + d.x, t.y + d.y, t.z + d.z, t.w + d.w);
                } else {
                    const float w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
                    for (uint32_t j = 0; j < 4; ++j)
                        if (r + j < rows) store_c(a, at + j, w[j]);
                }
            }
        }
    } else {
        for (uint32_t i0 = first; i0 < items; i0 += kItems * kStep) {
            float v[kItems][SPLIT];
#pragma unroll
            for (uint32_t u = 0; u < kItems; ++u) {
                const uint32_t i = i0 + u * kStep, r = i / n, off = ((i - r * n) * kPartPitch + r) * 4;
                if (i >= items) continue;
#pragma unroll
                for (uint32_t s = 0; s < SPLIT; ++s) v[u][s] = peer_load(peer[s] + off);
            }
            tell(i0);
#pragma unroll
            for (uint32_t u = 0; u < kItems; ++u) {
                const uint32_t i = i0 + u * kStep, r = i / n, q = i - r * n;
                if (i >= items) continue;
                float t = v[u][0];
#pragma unroll
                for (uint32_t s = 1; s < SPLIT; ++s) t += v[u][s];
                store_c(a, ((uint64_t)tp * kPRows + r) * a.ldc + (uint64_t)tq * a.nq + q, t);
            }
        }
    }
    if (!told) cluster_arrive();
}

// NT: most Q rows of a tile (a.nq <= NT of them are used).  The CTAs of a
// cluster take the same tile and consecutive parts of K; their sums meet in
// shared memory and are added in the order of the ranks, each CTA writing a
// part of the tile.
template <int BITS, int NT>
__global__ void __launch_bounds__(kSplitThreads) k_mx_split(const __grid_constant__ CUtensorMap p_map,
                                                            const __grid_constant__ CUtensorMap q_map,
                                                            const MmaArgs a)
{
    constexpr uint32_t kAtoms = BITS == 4 ? 2 : 1;       // scale tiles of a stage and 128 rows
    constexpr uint32_t kScaleStage = 2 * kAtoms * 512, kScaleCols = 2 * kAtoms * 4;
    extern __shared__ uint8_t s_raw[];
    __shared__ unsigned long long s_full[kMaxRing], s_empty[kMaxRing], s_done[2], s_free[2], s_drain;
    __shared__ uint32_t s_tmem, s_abort;
    const uint32_t base = (smem_u32(s_raw) + 1023u) & ~1023u;
    uint8_t* const raw = s_raw + (base - smem_u32(s_raw));
    const uint32_t stage_bytes = kPBytes + a.nq * 128, scale_base = a.ring * stage_bytes;
    const uint32_t warp = __shfl_sync(ez::kFull, threadIdx.x / 32, 0), lane = threadIdx.x % 32;

    uint32_t split, tp, tq;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(split));
    const uint32_t rank = cluster_rank();
    tile_of(blockIdx.x / split, 16, a, tp, tq);
    const uint32_t k0 = (uint32_t)((uint64_t)a.steps * rank / split);
    const uint32_t k1 = (uint32_t)((uint64_t)a.steps * (rank + 1) / split);

    ez::grid_dep_launch();
    const bool one = elect();
    const uint8_t* const p_scales = a.p_scales + (uint64_t)tp * a.scale_tiles * 512;
    const uint8_t* const q_scales = a.q_scales + (uint64_t)(tq * a.nq / 128) * a.scale_tiles * 512;
    auto load = [&](uint32_t k, uint32_t s) {
        const uint32_t bytes = min(kAtoms, a.scale_tiles - k * kAtoms) * 512;
        const uint32_t st = base + s * stage_bytes, x = k * 128;
        uint8_t* const sc = raw + scale_base + s * kScaleStage;
        const uint64_t kt = (uint64_t)k * (kAtoms * 512);
        if (one) {
            ez::mbar_arrive_expect_tx(&s_full[s], stage_bytes + 2 * bytes);
            tma_2d(st, &p_map, x, tp * kPRows, &s_full[s]);
            ez::bulk_g2s(sc, p_scales + kt, bytes, &s_full[s]);
            tma_2d(st + kPBytes, &q_map, x, tq * a.nq, &s_full[s]);
            ez::bulk_g2s(sc + kAtoms * 512, q_scales + kt, bytes, &s_full[s]);
        }
    };
    // the first loads need nobody else's set-up
    const uint32_t first = min(k1 - k0, a.ring);
    if (warp == 0) {
        if (one) {
            for (uint32_t i = 0; i < a.ring; ++i) {
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
            if (a.steps) {
                prefetch_map(&p_map);
                prefetch_map(&q_map);
            }
        }
        ez::grid_dep_wait();
        for (uint32_t i = 0; i < first; ++i) load(k0 + i, i);
    }
    __syncwarp();
    if (warp == 1) tmem_alloc<1>(&s_tmem, a.cols);
    fence_before();
    ez::grid_dep_wait();        // before C, which an earlier kernel may still read, is written
    __syncthreads();
    fence_after();
    const uint32_t tmem = s_tmem, scale_cols = tmem + (k1 - k0 > a.segment ? 2 : 1) * NT;

    auto gave_up = [&] {
        atomicExch(&s_abort, 1u);
        atomicOr(a.status, EZ_DSTAT_TIMEOUT);
    };
    float sum[NT];
    uint32_t issued = first;            // stages (warp 0)
    if (warp == 0) {
        Ring r;
        bool ok = true;
        for (uint32_t k = k0 + first; k < k1; ++k, ++issued) {
            if (!wait_warp(&s_empty[r.slot], r.parity, &s_abort, a.limit)) {
                ok = false;
                break;
            }
            load(k, r.slot);
            r.next(a.ring);
        }
        if (!ok && one) gave_up();
    } else if (warp == 1) {
        Ring r;
        bool ok = true;
        uint32_t seg = 0, ready = 0;
        for (uint32_t k = k0; k < k1 && ok; ++seg) {
            const uint32_t buf = seg & 1u, d = tmem + buf * NT, end = min(k + a.segment, k1);
            if (seg >= 2 && !wait_warp(&s_free[buf], (seg / 2 - 1) & 1, &s_abort, a.limit)) {
                ok = false;
                break;
            }
            for (uint32_t begin = k; k < end; ++k) {
                if (!__all_sync(ez::kFull, ready) && !wait_warp(&s_full[r.slot], r.parity, &s_abort, a.limit)) {
                    ok = false;
                    break;
                }
                fence_after();
                const uint32_t rs = r.slot;
                r.next(a.ring);
                ready = peek(&s_full[r.slot], r.parity);
                const uint32_t atoms = min(kAtoms, a.scale_tiles - k * kAtoms);
                const uint32_t cp = scale_cols + rs * kScaleCols, cq = cp + kAtoms * 4;
                const uint64_t ds = desc_scales(base + scale_base + rs * kScaleStage);
                const uint64_t dp = desc_rows(base + rs * stage_bytes);
                const uint64_t dq = desc_rows(base + rs * stage_bytes + kPBytes);
                if (one) {
#pragma unroll
                    for (uint32_t i = 0; i < kAtoms; ++i)
                        if (i < atoms) {
                            copy_scales<1>(cp + i * 4, ds + i * 32);
                            copy_scales<1>(cq + i * 4, ds + (kAtoms + i) * 32);
                        }
#pragma unroll
                    for (uint32_t i = 0; i < 4; ++i) {
                        const uint32_t atom = BITS == 4 ? i / 2 : 0, id = BITS == 4 ? (i % 2) * 2 : i;
                        if (atom < atoms)
                            mma<BITS, 1>(d, dp + 2 * i, dq + 2 * i, a.idesc | scale_ids(id), cp + atom * 4,
                                         cq + atom * 4, (k > begin || i > 0) ? 1u : 0u);
                    }
                    if (k + a.ring < k1) commit(&s_empty[rs]);     // nobody waits for the last ones
                    if (k + 1 == end) commit(&s_done[buf]);
                }
            }
        }
        if (!ok && one) gave_up();
    } else {
        const uint32_t quarter = warp % 4;
#pragma unroll
        for (int i = 0; i < NT; ++i) sum[i] = 0.f;
        uint32_t seg = 0;
        for (uint32_t k = k0; k < k1; k += a.segment, ++seg) {
            const uint32_t buf = seg & 1u, d = tmem + buf * NT + (quarter << 21);
            // every lane takes part in the loads: the vote makes the wait's outcome the warp's
            if (!__all_sync(ez::kFull, wait(&s_done[buf], (seg / 2) & 1, &s_abort, a.limit))) {
                if (lane == 0) gave_up();
                break;
            }
            fence_after();
#pragma unroll
            for (int q0 = 0; q0 < NT; q0 += 32) {
                if (q0 < a.nq) {
                    uint32_t r[32];
                    tmem_load32(d + q0, r);
                    tmem_wait_load(r);
#pragma unroll
                    for (int i = 0; i < 32; ++i) sum[q0 + i] += __uint_as_float(r[i]);
                }
            }
            fence_before();
            __syncwarp();
            if (lane == 0) ez::mbar_arrive(&s_free[buf]);
        }
        // all products are done: the stages' memory takes the sums
        float* part = reinterpret_cast<float*>(raw) + quarter * 32 + lane;
#pragma unroll
        for (int i = 0; i < NT; ++i)
            if (i < a.nq) part[i * kPartPitch] = sum[i];
    }
    __syncwarp();
    if (split > 1)
        cluster_sync();
    else
        __syncthreads();
    if (s_abort) {
        // Whoever gave up: the last copies and products end before the memory does
        // that they read and write, those of roles that got to their end too.
        if (warp == 0 && one)
            for (uint32_t i = issued > a.ring ? issued - a.ring : 0; i < issued; ++i)
                drain(&s_full[i % a.ring], (i / a.ring) & 1);
        if (warp == 1 && one) {
            commit(&s_drain);
            drain(&s_drain, 0);
        }
    }
    switch (split) {
        case 1: join<1>(a, base, rank, tp, tq); break;
        case 2: join<2>(a, base, rank, tp, tq); break;
        case 4: join<4>(a, base, rank, tp, tq); break;
        default: join<8>(a, base, rank, tp, tq); break;
    }
    __syncwarp();
    if (split > 1) cluster_wait();      // join() has arrived
    fence_before();
    __syncthreads();
    if (warp == 1) {
        fence_after();
        tmem_free<1>(tmem, a.cols);
    }
}

// ---- many tiles: pairs of CTAs ------------------------------------------------------

constexpr int kPairThreads = 384;            // warps 0 load, 1 products, 2 scales, 4..11 take tiles out
constexpr uint32_t kTmemCols = 512, kGroup = 16;
// slots of tensor memory for scales: a stage's are copied when the products of
// the stage that many before it are done
constexpr uint32_t kWideSlots = 4, kMaxSlots = 8;

// 32 rows of C by 128 columns on their way from the lanes (one column each) of
// 4 warps to rows at any alignment.  The rows lie in shared memory as they do in
// C modulo 16 bytes (their pitch there is C's, modulo a granule), so whole
// granules move without shifting: 2.6 us for a tile of 256 columns in BF16, where
// storing 192 straight from the lanes, 64 bytes at an odd address per instruction,
// took 3.9; 2048 x 8191 x 1024 into FP32 22 us, from the lanes 37.
template <typename T>
struct RowStage {
    static constexpr int kGranule = 16 / sizeof(T), kLanes = 128 / kGranule;     // values; threads to a row
    static constexpr uint32_t kBytes = 32 * (128 + 2 * kGranule - 1) * sizeof(T) + 16;
    T* mem;
    T* out;                 // first row and column of the piece in C
    uint64_t ld;
    uint32_t pitch, off;
    int n, left;            // columns and rows of C from there on
    __device__ __forceinline__ RowStage(const MmaArgs& a, uint8_t* m, uint64_t r0, uint32_t c0)
        : mem(reinterpret_cast<T*>(m)), out(static_cast<T*>(a.c) + r0 * a.ldc + c0), ld(a.ldc)
    {
        pitch = 128 + kGranule + (uint32_t)(ld % kGranule);
        off = (uint32_t)(reinterpret_cast<uintptr_t>(out) / sizeof(T) % kGranule);
        n = c0 < a.p_rows ? (int)min(128u, a.p_rows - c0) : 0;
        left = r0 < a.q_rows ? (int)min((uint64_t)128, a.q_rows - r0) : 0;
    }
    __device__ __forceinline__ void put(const float* v, uint32_t column) const
    {
        T* to = mem + off + column;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            if constexpr (sizeof(T) == 2)
                to[i * pitch] = (T)bf16x2(v[i], 0.f);
            else
                to[i * pitch] = v[i];
        }
    }
    __device__ __forceinline__ void store(uint32_t t) const      // t: 0..127
    {
#pragma unroll
        for (int i = 0; i < 32 * kLanes / 128; ++i) {
            const int r = (int)t / kLanes + 128 / kLanes * i;
            const uint32_t s = off + r * pitch;
            const int col = kGranule * ((int)t % kLanes) - (int)(s % kGranule);
            if (r < left && col >= 0 && col + kGranule <= n)
                *reinterpret_cast<uint4*>(out + r * ld + col) = *reinterpret_cast<const uint4*>(mem + s + col);
        }
#pragma unroll
        for (int i = 0; i < 32 * kGranule / 128; ++i) {          // values before the first granule, after the last
            const int r = (int)t / kGranule + 128 / kGranule * i, e = (int)t % kGranule;
            const uint32_t s = off + r * pitch;
            const int o = (int)(s % kGranule), first = o ? min(kGranule - o, n) : 0;
            const int last = max(first, (n + o) / kGranule * kGranule - o);
            T* const row = out + r * ld;
            if (r < left && e < first) row[e] = mem[s + e];
            if (r < left && last + e < n) row[last + e] = mem[s + last + e];
        }
    }
    __device__ __forceinline__ void next()                       // the 32 rows below
    {
        out += 32 * ld;
        off = (uint32_t)(reinterpret_cast<uintptr_t>(out) / sizeof(T) % kGranule);
        left -= 32;
    }
};

__device__ __forceinline__ void half_sync(uint32_t half) { asm volatile("bar.sync %0, 128;" :: "r"(1 + half) : "memory"); }
// The same, and whether `ok` holds for all 128 threads.
__device__ __forceinline__ bool half_vote(uint32_t half, bool ok)
{
    uint32_t all;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\t"
                 "barrier.cta.red.and.pred q, %1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(all) : "r"(1 + half), "r"((uint32_t)ok) : "memory");
    return all != 0;
}

// At the start of a pair CTA's shared memory, which is then used to its last byte.
struct PairBarriers {
    unsigned long long full[kMaxRing], empty[kMaxRing], slot[kMaxSlots], scales[kMaxSlots], done[2], free[2], early,
        drain[2];
    uint64_t issued[2];         // after a role gave up: each CTA's stages, in the even one
    uint32_t tmem, abort;
};
constexpr uint32_t kPairHead = 1024, kPairSmem = 227 * 1024;
static_assert(sizeof(PairBarriers) <= kPairHead, "shared memory");

// Results of a warp's 32 rows, 64 bytes each, on their way to C: written by rows
// in the swizzle of the map and stored by TMA.
constexpr uint32_t kOutBytes = 32 * 64;
__device__ __forceinline__ void store_piece(const CUtensorMap* map, uint32_t mem, uint32_t lane, const uint32_t* w,
                                            uint32_t x, uint32_t y)
{
    if (lane == 0) tma_store_wait_read();       // of the piece before
    __syncwarp();
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i)
        st_shared4(mem + lane * 64 + (i ^ (lane >> 1 & 3u)) * 16, w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    fence_async();
    __syncwarp();
    if (lane == 0) tma_store_2d(map, x, y, mem);
}

// A pair's tile is 256 P rows (128 in each CTA's tensor memory) by a.nq Q rows
// (64, 128, 192 or 256; each CTA loads half and the tensor cores read both
// halves).  The even CTA issues for both.  Two sums take turns in tensor
// memory; for 256 columns they do not both fit beside the scales and overlap in
// a few columns, which are taken out first, so that the next tile's products
// start while the rest of this one's columns are on their way out.
//
// LATE: an addend joins a sum of several segments on the way out, after the last of
// them, so that C is rounded to its size once (1: from the lanes, 2: swapped).  Else
// the sum starts from it, which is the same for one segment, and it is read while
// the products run (2048 x 8191 x 1024: 44 us, read last 48).  From the lanes it is
// read by whole sectors, between the stores: by 16 bytes a lane, which L1 cannot hold
// until the other 16 are asked for, the weight gradient took 374 us instead of 363.
template <int BITS, int LATE>
__global__ void __launch_bounds__(kPairThreads, 1) k_mx_pair(const __grid_constant__ CUtensorMap p_map,
                                                             const __grid_constant__ CUtensorMap q_map,
                                                             const __grid_constant__ CUtensorMap ps_map,
                                                             const __grid_constant__ CUtensorMap qs_map,
                                                             const __grid_constant__ CUtensorMap c_map,
                                                             const MmaArgs a)
{
    constexpr uint32_t kAtoms = BITS == 4 ? 2 : 1;
    constexpr uint32_t kScaleStage = 3 * kAtoms * 512, kScaleCols = 3 * kAtoms * 4;
    // columns in the overlap of two sums of 256, which are taken out first
    constexpr uint32_t kOverlap = kWideSlots * kScaleCols;
    static_assert(kOverlap <= 96, "the first three of a warp's four chunks");
    extern __shared__ __align__(1024) uint8_t s_pair[];
    PairBarriers& s = *reinterpret_cast<PairBarriers*>(s_pair);
    uint8_t* const raw = s_pair + kPairHead;
    const uint32_t base = smem_u32(raw);
    const uint32_t stage_bytes = kPBytes + a.nq * 64, scale_base = a.ring * stage_bytes;
    const uint32_t warp = __shfl_sync(ez::kFull, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    const uint32_t rank = cluster_rank();

    ez::grid_dep_launch();
    if (threadIdx.x == 0) {
        for (uint32_t i = 0; i < a.ring; ++i) {
            ez::mbar_init(&s.full[i], 1);
            ez::mbar_init(&s.empty[i], 1);
        }
        for (uint32_t i = 0; i < a.slots; ++i) {
            ez::mbar_init(&s.slot[i], 1);
            ez::mbar_init(&s.scales[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            ez::mbar_init(&s.done[i], 1);
            ez::mbar_init(&s.free[i], 16);      // 8 warps of both CTAs
            ez::mbar_init(&s.drain[i], 1);
        }
        ez::mbar_init(&s.early, 8);             // the 4 warps of the overlapping half, both CTAs
        s.abort = 0;
        ez::mbar_fence_init();
        prefetch_map(&p_map);
        prefetch_map(&q_map);
        prefetch_map(&ps_map);
        prefetch_map(&qs_map);
        if (a.staged) prefetch_map(&c_map);
    }
    __syncwarp();
    if (warp == 1) tmem_alloc<2>(&s.tmem, kTmemCols);
    fence_before();
    __syncthreads();
    cluster_sync();                             // the other CTA's barriers are ready too
    fence_after();
    ez::grid_dep_wait();
    const uint32_t sum_cols = kTmemCols - a.slots * kScaleCols;
    const uint32_t tmem = s.tmem, scale_cols = tmem + sum_cols;
    const uint32_t second = min(a.nq, sum_cols - a.nq);     // where the second sum starts
    const bool overlap = second < a.nq;
    const uint32_t tiles = a.p_tiles * a.q_tiles, t0 = blockIdx.x / 2, step = gridDim.x / 2;
    const uint64_t my_tiles = (tiles - t0 + step - 1) / step;
    // scale tiles of the Q rows: nq may start in the middle of one
    const uint32_t q_scale_tiles = a.nq > 128 ? 2 : 1;

    // Ends the roles of both CTAs, which thereby agree on it after the barrier that
    // all roles end in.
    auto gave_up = [&] {
        peer_store(peer_addr(smem_u32(&s.abort), 0), 1u);
        peer_store(peer_addr(smem_u32(&s.abort), 1), 1u);
        atomicOr(a.status, EZ_DSTAT_TIMEOUT);
        fence_cluster();
    };
    const bool one = elect();
    uint64_t issued = 0;                // stages (warp 0)
    const uint32_t half_stage = kPBytes + a.nq * 64 + (1 + q_scale_tiles) * kAtoms * 512;     // a CTA's bytes

    // registers: 384 threads x 168 at launch = 128 x 40 + 256 x 232
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (warp == 0) {
            Ring r;
            bool ok = true;
            const uint32_t bar0 = peer_addr(smem_u32(&s.full[0]), 0);
            for (uint32_t t = t0; t < tiles && ok; t += step) {
                uint32_t tp, tq;
                tile_of(t, kGroup, a, tp, tq);
                const uint32_t p = (tp * 2 + rank) * kPRows, q = tq * a.nq;
                for (uint32_t k = 0; k < a.steps; ++k, ++issued) {
                    if (issued >= a.ring && !wait_warp(&s.empty[r.slot], r.parity ^ 1u, &s.abort, a.limit)) {
                        ok = false;
                        break;
                    }
                    const uint32_t bar = bar0 + r.slot * 8;
                    const uint32_t st = base + r.slot * stage_bytes, sc = base + scale_base + r.slot * kScaleStage;
                    if (one) {
                        // both CTAs' loads complete on the even CTA's barrier
                        if (rank == 0) ez::mbar_arrive_expect_tx(&s.full[r.slot], 2 * half_stage);
                        tma_2d_pair(st, &p_map, k * 128, p, bar);
                        tma_2d_pair(st + kPBytes, &q_map, k * 128, q + rank * (a.nq / 2), bar);
                        tma_3d_pair(sc, &ps_map, 0, k * kAtoms, p / 128, bar);
                        tma_3d_pair(sc + kAtoms * 512, &qs_map, 0, k * kAtoms, q / 128, bar);
                    }
                    r.next(a.ring);
                }
            }
            if (!ok && one) gave_up();
        } else if (warp == 1 && rank == 0) {
            Ring r, sl;
            uint32_t j = 0;                 // segments
            uint64_t left = my_tiles * a.steps;     // stages
            uint32_t ready = 0;             // the next stage's barrier, seen in time
            bool ok = true;
            for (uint32_t t = t0; t < tiles && ok; t += step) {
                uint32_t tp, tq;
                tile_of(t, kGroup, a, tp, tq);
                const uint32_t q_off = tq * a.nq % 128 / 32;     // 0 or 2 columns
                for (uint32_t k = 0; k < a.steps && ok; ++j) {
                    const uint32_t buf = j & 1u, d = tmem + buf * second, end = min(k + a.segment, a.steps);
                    // The scales are in tensor memory (and so the codes beside them here)
                    // long before the columns of this sum are free.
                    if (!wait_warp(&s.scales[sl.slot], sl.parity, &s.abort, a.limit) ||
                        (j >= 2 && !wait_warp(&s.free[buf], (j / 2 - 1) & 1, &s.abort, a.limit)) ||
                        (j >= 1 && overlap && !wait_warp(&s.early, (j - 1) & 1, &s.abort, a.limit))) {
                        ok = false;
                        break;
                    }
                    ready = 1;
                    for (uint32_t begin = k; k < end; ++k) {
                        if (!__all_sync(ez::kFull, ready) && !wait_warp(&s.scales[sl.slot], sl.parity, &s.abort, a.limit)) {
                            ok = false;
                            break;
                        }
                        fence_after();
                        const uint32_t rs = r.slot, ss = sl.slot;
                        r.next(a.ring);
                        sl.next(a.slots);
                        ready = peek(&s.scales[sl.slot], sl.parity);
                        const uint32_t atoms = min(kAtoms, a.scale_tiles - k * kAtoms);
                        const uint32_t cp = scale_cols + ss * kScaleCols, cq = cp + kAtoms * 4 + q_off;
                        const uint64_t dp = desc_rows(base + rs * stage_bytes);
                        const uint64_t dq = desc_rows(base + rs * stage_bytes + kPBytes);
                        if (one) {
#pragma unroll
                            for (uint32_t i = 0; i < 4; ++i) {
                                const uint32_t atom = BITS == 4 ? i / 2 : 0, id = BITS == 4 ? (i % 2) * 2 : i;
                                if (atom < atoms)
                                    mma<BITS, 2>(d, dp + 2 * i, dq + 2 * i, a.idesc | scale_ids(id), cp + atom * 4,
                                                 cq + atom * 8, (k > begin || i > 0) ? 1u : 0u);
                            }
                            // nobody waits for the last ones of either
                            if (left > a.ring) commit_pair(&s.empty[rs], 3);
                            if (left > a.slots) commit_pair(&s.slot[ss], 1);
                            if (k + 1 == end) commit_pair(&s.done[buf], 3);
                        }
                        --left;
                    }
                }
            }
            if (!ok && one) gave_up();
        } else if (warp == 2 && rank == 0) {
            // scales go to tensor memory a few stages ahead of their products
            Ring r, sl{0, 1};               // a new barrier's previous phase counts as over
            uint32_t ready = 0;
            bool ok = true;
            for (uint32_t t = t0; t < tiles && ok; t += step) {
                for (uint32_t k = 0; k < a.steps; ++k) {
                    if (!__all_sync(ez::kFull, ready) &&
                        (!wait_warp(&s.slot[sl.slot], sl.parity, &s.abort, a.limit) ||
                         !wait_warp(&s.full[r.slot], r.parity, &s.abort, a.limit))) {
                        ok = false;
                        break;
                    }
                    fence_after();
                    const uint32_t rs = r.slot, ss = sl.slot;
                    r.next(a.ring);
                    sl.next(a.slots);
                    ready = peek(&s.slot[sl.slot], sl.parity) & peek(&s.full[r.slot], r.parity);
                    const uint32_t atoms = min(kAtoms, a.scale_tiles - k * kAtoms);
                    const uint32_t cp = scale_cols + ss * kScaleCols, cq = cp + kAtoms * 4;
                    const uint64_t ds = desc_scales(base + scale_base + rs * kScaleStage);
                    if (one) {
#pragma unroll
                        for (uint32_t i = 0; i < kAtoms; ++i)
                            if (i < atoms) {
                                copy_scales<2>(cp + i * 4, ds + i * 32);
                                copy_scales<2>(cq + i * 8, ds + (kAtoms + i) * 32);
                                if (q_scale_tiles == 2) copy_scales<2>(cq + i * 8 + 4, ds + (2 * kAtoms + i) * 32);
                            }
                        commit_pair(&s.scales[ss], 1);
                    }
                }
            }
            if (!ok && one) gave_up();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
        // warp: lanes of its quarter, half `half` of the columns
        const uint32_t quarter = warp % 4, half = (warp - 4) / 4, half_cols = a.nq / 2;
        const uint32_t free_bar[2] = {peer_addr(smem_u32(&s.free[0]), 0), peer_addr(smem_u32(&s.free[1]), 0)};
        const uint32_t early_bar = peer_addr(smem_u32(&s.early), 0);
        uint8_t* const stage_mem = raw + a.ring * (stage_bytes + kScaleStage);
        const uint32_t out_mem = base + a.ring * (stage_bytes + kScaleStage) + (warp - 4) * kOutBytes;
        float sum[128];
        uint32_t j = 0;
        // Segments: an arrival that nobody waits for could reach the even CTA's
        // memory after its end, so the last ones are left out.
        uint64_t left = my_tiles * ((a.steps + a.segment - 1) / a.segment);
        bool ok = true;
        for (uint32_t t = t0; t < tiles && ok; t += step) {
            uint32_t tp, tq;
            tile_of(t, kGroup, a, tp, tq);
            const uint64_t p = (uint64_t)(tp * 2 + rank) * kPRows + quarter * 32 + lane;
            const uint64_t q0 = (uint64_t)tq * a.nq + half * half_cols;
#pragma unroll
            for (int c = 0; c < 128; c += 32) {
                float* r = sum + c;
                if (!LATE && a.add && p < a.p_rows && c < half_cols) {
                    if (!a.swap && q0 + c + 32 <= a.q_rows) {
                        const float4* e = reinterpret_cast<const float4*>(a.add + p * a.ldc + q0 + c);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float4 v = e[i];
                            r[4 * i] = v.x;
                            r[4 * i + 1] = v.y;
                            r[4 * i + 2] = v.z;
                            r[4 * i + 3] = v.w;
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const uint64_t q = q0 + c + i;
                            r[i] = q < a.q_rows ? a.add[a.swap ? q * a.ldc + p : p * a.ldc + q] : 0.f;
                        }
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) r[i] = 0.f;
                }
            }
            for (uint32_t k = 0; k < a.steps; k += a.segment, ++j, --left) {
                const uint32_t buf = j & 1u, d = tmem + buf * second + (quarter << 21) + half * half_cols;
                if (!__all_sync(ez::kFull, wait(&s.done[buf], (j / 2) & 1, &s.abort, a.limit))) {
                    if (lane == 0) gave_up();
                    ok = false;
                    break;
                }
                fence_after();
                uint32_t x[2][32];
                auto load = [&](auto chunk, uint32_t* to) {
                    constexpr uint32_t c = decltype(chunk)::value * 32;
                    if (c < half_cols) tmem_load32(d + c, to);
                };
                auto add = [&](auto chunk, const uint32_t* from) {
                    constexpr uint32_t c = decltype(chunk)::value * 32;
                    if (c < half_cols)
#pragma unroll
                        for (int i = 0; i < 32; ++i) sum[c + i] += __uint_as_float(from[i]);
                };
                auto tell = [&](uint32_t bar) {
                    fence_before();
                    __syncwarp();
                    if (lane == 0) peer_arrive(bar);
                };
                // two chunks at a time; the first sum's last columns are the second's first
                auto take_all = [&](auto c0, auto c1, auto c2, auto c3, uint32_t early_half) {
                    load(c0, x[0]);
                    load(c1, x[1]);
                    tmem_wait_load(x[0]);
                    tmem_wait_load(x[1]);
                    if (kOverlap <= 64 && overlap && half == early_half && left > 1) tell(early_bar);
                    add(c0, x[0]);
                    load(c2, x[0]);
                    add(c1, x[1]);
                    if (kOverlap > 64) {
                        tmem_wait_load(x[0]);
                        if (overlap && half == early_half && left > 1) tell(early_bar);
                    }
                    load(c3, x[1]);
                    tmem_wait_load(x[0]);
                    tmem_wait_load(x[1]);
                    if (left > 2) tell(free_bar[buf]);
                    add(c2, x[0]);
                    add(c3, x[1]);
                };
                using C0 = std::integral_constant<int, 0>;
                using C1 = std::integral_constant<int, 1>;
                using C2 = std::integral_constant<int, 2>;
                using C3 = std::integral_constant<int, 3>;
                if (buf == 0)
                    take_all(C3{}, C2{}, C1{}, C0{}, 1);
                else
                    take_all(C0{}, C1{}, C2{}, C3{}, 0);
            }
            // Swapped, the four warps of a half store together: they do so, and go on,
            // only if none of them gave up, so that none waits for one that has left.
            const bool swapped = LATE == 2 || (LATE == 0 && a.swap);
            if (swapped) ok = half_vote(half, ok);      // and the stage is free
            if (!ok) break;
            if (swapped) {
                const float* e = LATE == 2 ? a.add + q0 * a.ldc + p : nullptr;
                const int n = p < a.p_rows && q0 < a.q_rows ? (int)min(half_cols, a.q_rows - (uint32_t)q0) : 0;
                auto by_rows = [&](auto st) {
#pragma unroll
                    for (int c = 0; c < 128; c += 32) {
                        if (c >= half_cols) break;
                        if constexpr (LATE == 2) {
                            float v[32];
#pragma unroll
                            for (int i = 0; i < 32; ++i, e += a.ldc) v[i] = c + i < n ? *e : 0.f;
#pragma unroll
                            for (int i = 0; i < 32; ++i) sum[c + i] += v[i];
                        }
                        if (c) half_sync(half);     // the stage is free
                        st.put(sum + c, quarter * 32 + lane);
                        half_sync(half);
                        st.store(threadIdx.x & 127u);
                        st.next();
                    }
                };
                const uint32_t p0 = (tp * 2 + rank) * kPRows;
                if (a.f32)
                    by_rows(RowStage<float>(a, stage_mem + half * RowStage<float>::kBytes, q0, p0));
                else
                    by_rows(RowStage<uint16_t>(a, stage_mem + half * RowStage<uint16_t>::kBytes, q0, p0));
                continue;
            }
            if (LATE || !a.staged) {
                if (p >= a.p_rows) continue;
#pragma unroll
                for (int c = 0; c < 128; c += 32) {
                    if (c >= half_cols) break;
                    const uint64_t q = q0 + c, at = p * a.ldc + q;
                    float* const r = sum + c;
                    uint32_t w[32];
                    if (LATE == 1 && q + 32 <= a.q_rows) {      // whole sectors
                        float v[32];
#pragma unroll
                        for (int i = 0; i < 32; i += 8) ld_v8(a.add + at + i, v + i);
#pragma unroll
                        for (int i = 0; i < 32; ++i) r[i] += v[i];
                    }
                    if (q + 32 > a.q_rows) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            if (q + i >= a.q_rows) continue;
                            if (a.f32)
                                static_cast<float*>(a.c)[at + i] = LATE == 1 ? r[i] + a.add[at + i] : r[i];
                            else
                                static_cast<uint16_t*>(a.c)[at + i] = (uint16_t)bf16x2(r[i], 0.f);
                        }
                    } else if (a.f32) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(r[i]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) st_v8(static_cast<float*>(a.c) + at + 8 * i, w + 8 * i);
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i) w[i] = bf16x2(r[2 * i], r[2 * i + 1]);
#pragma unroll
                        for (int i = 0; i < 2; ++i) st_v8(static_cast<uint16_t*>(a.c) + at + 16 * i, w + 8 * i);
                    }
                }
                continue;
            }
            const uint32_t row0 = (tp * 2 + rank) * kPRows + quarter * 32;
            const uint32_t columns = row0 >= a.p_rows || q0 >= a.q_rows ? 0 : min(half_cols, a.q_rows - (uint32_t)q0);
#pragma unroll
            for (int c = 0; c < 128; c += 32) {
                if (c >= columns) break;
                const float* r = sum + c;
                uint32_t w[16];
                if (a.f32) {
#pragma unroll
                    for (int h = 0; h < 32; h += 16) {
                        if (c + h >= columns) break;
#pragma unroll
                        for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(r[h + i]);
                        store_piece(&c_map, out_mem, lane, w, (uint32_t)q0 + c + h, row0);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) w[i] = bf16x2(r[2 * i], r[2 * i + 1]);
                    store_piece(&c_map, out_mem, lane, w, (uint32_t)q0 + c, row0);
                }
            }
        }
        if (a.staged && lane == 0) tma_store_wait();
    }
    __syncwarp();
    fence_before();
    cluster_sync_relaxed();     // neither CTA signals or reads the other any more
    if (s.abort) {
        // Whoever gave up: the last copies and products of both CTAs end before the
        // memory does that they read and write, those of roles that got to their end
        // too.  The even CTA's barriers count both CTAs' copies; one CTA may have
        // issued stages that the other has not.
        if (warp == 0 && one) peer_store64(peer_addr(smem_u32(&s.issued[rank]), 0), issued);
        cluster_sync();
        if (rank == 0 && warp == 0 && one) {
            const uint64_t n0 = s.issued[0], n1 = s.issued[1], n = n0 > n1 ? n0 : n1;
            for (uint64_t i = n > a.ring ? n - a.ring : 0; i < n; ++i) {
                unsigned long long* const bar = &s.full[i % a.ring];
                if (i >= n0)
                    ez::mbar_arrive_expect_tx(bar, half_stage);
                else if (i >= n1)
                    ez::mbar_complete_tx(bar, half_stage);
                drain(bar, (uint32_t)(i / a.ring) & 1);
            }
        }
        if ((warp == 1 || warp == 2) && one) {
            if (rank == 0) commit_pair(&s.drain[warp - 1], 3);
            drain(&s.drain[warp - 1], 0);
        }
        cluster_sync();
    }
    if (warp == 1) {
        fence_after();
        tmem_free<2>(tmem, kTmemCols);
    }
}

// ---- host -----------------------------------------------------------------------------

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
// Scale tiles (128 words) along K and along the rows, read `atoms` x `tiles` at a time.
bool scale_map(CUtensorMap* m, const uint8_t* scales, uint64_t row_tiles, uint64_t k_tiles, uint32_t atoms,
               uint32_t tiles)
{
    const Encode fn = encoder();
    if (!fn) return false;
    const cuuint64_t dims[3] = {128, k_tiles, row_tiles}, strides[2] = {512, 512 * k_tiles};
    const cuuint32_t box[3] = {128, atoms, tiles}, one[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<uint8_t*>(scales), dims, strides, box, one,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// C as k_mx_pair stores it: pieces of 32 rows and 64 bytes.
bool c_map(CUtensorMap* m, const MmaArgs& a)
{
    const Encode fn = encoder();
    if (!fn) return false;
    const uint32_t bytes = a.f32 ? 4 : 2;
    const cuuint64_t dims[2] = {a.q_rows, a.p_rows}, strides[1] = {a.ldc * bytes};
    const cuuint32_t box[2] = {64 / bytes, 32}, one[2] = {1, 1};
    return fn(m, a.f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.c, dims, strides, box,
              one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

uint32_t type_of(int fmt) { return fmt == EZ_MX_E4M3 ? 0u : 1u; }   // E2M1 and E5M2 are 1 in their kinds

struct Operand {
    int fmt;
    const uint8_t *codes, *scales;
    uint64_t rows;
};

std::atomic<uint32_t> wait_limit{ez::kSpinLimit};

// Launch attributes: the cluster size, and a start while the kernel before
// drains (both kernels wait for it before they touch memory).
struct Clusters {
    cudaLaunchAttribute attr[2] = {};
    explicit Clusters(uint32_t size)
    {
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = size;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
    }
};

// Clusters of `size` CTAs of k_mx_split (one to an SM) that fit the current
// device at once; asked once for each size.
uint32_t most_clusters(uint32_t size)
{
    static std::atomic<int> known[64][kMaxSplit + 1];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    int n = known[dev][size].load(std::memory_order_relaxed);
    if (!n) {
        static ez::PerDeviceAttr raised;
        auto kernel = k_mx_split<4, 32>;
        Clusters attrs(size);
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(size);
        cfg.blockDim = dim3(kSplitThreads);
        cfg.dynamicSmemBytes = kMaxSmem;
        cfg.attrs = attrs.attr;
        cfg.numAttrs = 1;
        if (ez::max_dyn_smem_per_device(raised, kernel, kMaxSmem) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess)
            return 0;
        if (n <= 0) n = -1;
        known[dev][size].store(n, std::memory_order_relaxed);
    }
    return n > 0 ? (uint32_t)n : 0;
}

template <int BITS>
void fill(MmaArgs& a, const Operand& p, const Operand& q, uint64_t K, uint32_t m, uint32_t nq)
{
    a.p_scales = p.scales;
    a.q_scales = q.scales;
    a.p_rows = (uint32_t)p.rows;
    a.q_rows = (uint32_t)q.rows;
    a.p_tiles = (uint32_t)ez::cdiv(p.rows, m);
    a.q_tiles = (uint32_t)ez::cdiv(q.rows, nq);
    a.nq = nq;
    a.scale_tiles = (uint32_t)ez::cdiv(K, 128);
    a.steps = (uint32_t)ez::cdiv(K, BITS == 4 ? 256 : 128);
    a.segment = a.f32 ? kSegment : kLongSegment;
    a.idesc = instr_desc(type_of(p.fmt), type_of(q.fmt), m, nq);
}

template <int BITS>
uint64_t pitch_of(uint64_t K) { return ez::cdiv(K, 32) * (BITS * 4); }

template <int BITS, int NT>
cudaError_t go_split(const Operand& p, const Operand& q, uint64_t K, MmaArgs a, uint32_t nq, uint32_t split,
                     uint32_t ring, cudaStream_t s)
{
    fill<BITS>(a, p, q, K, kPRows, nq);
    CUtensorMap pm{}, qm{};
    if (K && (!code_map(&pm, p.codes, p.rows, pitch_of<BITS>(K), kPRows) ||
              !code_map(&qm, q.codes, q.rows, pitch_of<BITS>(K), nq)))
        return cudaErrorUnknown;
    constexpr uint32_t kAtoms = BITS == 4 ? 2 : 1;
    a.ring = ring;
    const uint32_t sums = ez::cdiv(a.steps, split) > a.segment ? 2 : 1;
    const uint32_t cols = sums * NT + ring * kAtoms * 8;
    a.cols = cols <= 64 ? 64 : cols <= 128 ? 128 : cols <= 256 ? 256 : 512;
    const uint32_t stages = ring * (kPBytes + nq * 128 + 2 * kAtoms * 512), part = nq * kPartPitch * 4;
    auto kernel = k_mx_split<BITS, NT>;
    static ez::PerDeviceAttr raised;
    const cudaError_t e = ez::max_dyn_smem_per_device(raised, kernel, kMaxSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(a.p_tiles * a.q_tiles * split);
    cfg.blockDim = dim3(kSplitThreads);
    cfg.dynamicSmemBytes = (stages > part ? stages : part) + 1024;
    cfg.stream = s;
    Clusters attrs(split);
    cfg.attrs = attrs.attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, pm, qm, a);
}

template <int BITS, int LATE>
cudaError_t go_pair(const Operand& p, const Operand& q, uint64_t K, MmaArgs a, uint32_t nq, uint32_t sms,
                    cudaStream_t s)
{
    fill<BITS>(a, p, q, K, 256, nq);
    CUtensorMap pm{}, qm{}, psm{}, qsm{}, cm{};
    constexpr uint32_t kAtoms = BITS == 4 ? 2 : 1;
    if (!code_map(&pm, p.codes, p.rows, pitch_of<BITS>(K), kPRows) ||
        !code_map(&qm, q.codes, q.rows, pitch_of<BITS>(K), nq / 2) ||
        !scale_map(&psm, p.scales, ez::cdiv(p.rows, 128), a.scale_tiles, kAtoms, 1) ||
        !scale_map(&qsm, q.scales, ez::cdiv(q.rows, 128), a.scale_tiles, kAtoms, nq > 128 ? 2 : 1) ||
        (a.staged && !c_map(&cm, a)))
        return cudaErrorUnknown;
    auto kernel = k_mx_pair<BITS, LATE>;
    const uint32_t stage = kPBytes + nq * 64 + 3 * kAtoms * 512;
    const uint32_t out = a.staged ? 8 * kOutBytes
                         : a.swap ? 2 * (a.f32 ? RowStage<float>::kBytes : RowStage<uint16_t>::kBytes)
                                  : 0;
    const uint32_t ring = (kPairSmem - kPairHead - out) / stage;
    a.ring = ring > kMaxRing ? kMaxRing : ring;
    const uint32_t slots = (kTmemCols - 2 * nq) / (3 * kAtoms * 4);
    a.slots = nq == 256 ? kWideSlots : slots > kMaxSlots ? kMaxSlots : slots;
    static ez::PerDeviceAttr raised;
    const cudaError_t e = ez::max_dyn_smem_per_device(raised, kernel, kPairSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)ez::umin64((uint64_t)a.p_tiles * a.q_tiles, sms / 2) * 2);
    cfg.blockDim = dim3(kPairThreads);
    cfg.dynamicSmemBytes = kPairHead + a.ring * stage + out;
    cfg.stream = s;
    Clusters attrs(2);
    cfg.attrs = attrs.attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, pm, qm, psm, qsm, cm, a);
}

template <int BITS>
cudaError_t choose(const Operand& A, const Operand& B, uint64_t K, MmaArgs a, uint32_t sms, cudaStream_t s)
{
    const uint64_t steps = ez::cdiv(K, BITS == 4 ? 256 : 128);
    // Tiles of 128 x 128 over clusters, when there are few: K is cut in up to 8
    // parts of 2 stages at least, as far as the clusters are resident at once
    // (16 clusters of 8 are not: 512 x 512 x 8192 took 15.7 us with them, 10.3
    // with clusters of 4).  Up to 64 rows a pair's tile of 256 x 64 wastes what it
    // covers (48 x 10240 x 5120: 11.6 us, clusters 9.3); from there the estimate
    // below decides (100 x 4000 x 512: pairs 5.3 us, clusters 6.0).
    const bool narrow = A.rows <= 64 || B.rows <= 64;
    const bool swap = A.rows <= 128 || B.rows > 128;
    const Operand &SP = swap ? B : A, &SQ = swap ? A : B;
    const uint32_t snq = SQ.rows >= 128 ? 128 : (uint32_t)ez::cdiv(SQ.rows, 16) * 16;
    const uint64_t tiles = ez::cdiv(SP.rows, 128) * ez::cdiv(SQ.rows, snq);
    uint32_t split = 1;
    while (split < kMaxSplit && tiles * split * 2 <= sms && steps >= 4 * split && tiles <= most_clusters(2 * split))
        split *= 2;
    // Pairs take 4.5 us + 0.19 us a stage (one round), clusters 6.4 us + 0.23 us a
    // stage of their own, fitted to 160..1024 rows and columns, K = 512..8192.
    const bool few = tiles < sms && split > 1 && 640 + 23 * steps / split < 450 + 19 * steps;
    if (narrow || few || !K) {
        a.swap = swap;
        const uint32_t stage = kPBytes + snq * 128 + (BITS == 4 ? 2048 : 1024);
        uint32_t ring = (kMaxSmem - 1024) / stage;
        ring = ring > kMaxRing ? kMaxRing : ring;
        if (snq <= 32) return go_split<BITS, 32>(SP, SQ, K, a, snq, split, ring, s);
        if (snq <= 64) return go_split<BITS, 64>(SP, SQ, K, a, snq, split, ring, s);
        return go_split<BITS, 128>(SP, SQ, K, a, snq, split, ring, s);
    }
    // How C is written: by TMA, which needs rows that begin and end on 16 bytes; in
    // sectors from the lanes, which needs rows that begin on 32; else swapped, across
    // the lanes.
    const uint32_t bytes = a.f32 ? 4 : 2;
    const uint64_t begins = reinterpret_cast<uintptr_t>(a.c) | reinterpret_cast<uintptr_t>(a.add) | a.ldc * bytes;
    const bool by_tma = ((begins | B.rows * bytes) & 15u) == 0, by_lanes = (begins & 31u) == 0;
    // An addend that joins on the way out is read there by sectors too: without rows
    // on 32 bytes C goes the swapped way (4096 x 4100 x 8192 in 8 bits 115 us, started
    // from the addend and stored by TMA 103).
    const bool late = a.add && steps > kSegment;
    a.swap = !by_lanes && (late || !by_tma);
    const Operand &P = a.swap ? B : A, &Q = a.swap ? A : B;
    // rounds of tiles times a round's time, which is far from proportional to its
    // columns: 10.8, 8.4, 7.3 and 6.4 us for 256, 192, 128 and 64 at K = 8192 in 4 bits
    constexpr uint32_t kRound[4] = {64, 73, 84, 108};
    uint32_t nq = 256;
    uint64_t best = ~0ull;
    for (uint32_t n = 256; n >= 64; n -= 64) {
        const uint64_t tiles = ez::cdiv(P.rows, 256) * ez::cdiv(Q.rows, n);
        const uint64_t cost = ez::cdiv(tiles, sms / 2) * kRound[n / 64 - 1];
        if (cost < best) {
            best = cost;
            nq = n;
        }
    }
    // TMA stores are the shorter way out, but they stand in the way of the next
    // tile's loads: 4096 x 1024 x 4096 in one round takes 9.7 us with them, 10.2 from
    // the lanes; 8192 x 8192 x 1024 38 and 42; 2048 x 8192 x 2048 19.4 and 17.8.
    const bool one_round = ez::cdiv(P.rows, 256) * ez::cdiv(Q.rows, nq) <= sms / 2;
    a.staged = !late && by_tma && (!by_lanes || one_round || steps <= 6);
    if (late) return a.swap ? go_pair<BITS, 2>(P, Q, K, a, nq, sms, s) : go_pair<BITS, 1>(P, Q, K, a, nq, sms, s);
    return go_pair<BITS, 0>(P, Q, K, a, nq, sms, s);
}

}  // namespace

void set_mx_wait_limit(uint32_t polls) { wait_limit.store(polls, std::memory_order_relaxed); }

cudaError_t launch_mx_matmul(int fa, const uint8_t* ac, const uint8_t* as, uint64_t M, int fb, const uint8_t* bc,
                             const uint8_t* bs, uint64_t N, uint64_t K, const float* add, void* c, uint64_t ldc,
                             int f32, uint32_t* status, cudaStream_t s)
{
    if (!M || !N) return cudaSuccess;
    const uint32_t sms = sm_count();
    if (!sms) return cudaErrorInvalidDevice;
    const Operand A{fa, ac, as, M}, B{fb, bc, bs, N};
    MmaArgs a{};
    a.f32 = (uint32_t)f32;
    a.add = add;
    a.c = c;
    a.ldc = ldc;
    a.status = status;
    a.limit = wait_limit.load(std::memory_order_relaxed);
    return fa == EZ_MX_E2M1 ? choose<4>(A, B, K, a, sms, s) : choose<8>(A, B, K, a, sms, s);
}

}  // namespace ezk
