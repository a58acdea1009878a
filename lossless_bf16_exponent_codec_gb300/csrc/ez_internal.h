// ez_internal.h -- plan object and kernel launchers of libexpzip (host side).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "expzip.h"

struct ez_plan_s {
    uint64_t n;
    uint32_t W, B, codec;
    uint64_t L;              // shard length
    uint32_t tpc;            // tiles per shard
    uint64_t slot_bytes;     // worst-case payload per shard
    double K;                // 16383 / (14 ln 2)
    // workspace layout (byte offsets); [0, zero_bytes) is cleared per call
    uint64_t off_ctr, off_info, off_shard_stats, off_bins, off_state_a, off_state_b, off_seg, off_escbuf, off_plbuf;
    uint64_t zero_bytes, ws_bytes;
    uint32_t n_bins;
    uint32_t hist_window;    // EZ_FLAG_WINDOW_HIST: window from the histogram
    uint32_t hash_cache;     // EZ_FLAG_HASH_CACHE: sender cache of block hashes
    uint64_t hstride;        // sender-cache bytes per shard (hash mode: 16 per block)
};

namespace ezk {

// Per-shard record of the reuse split, written by the tile that holds the
// shard's last value: the values by which the shard's last block falls short
// of B when that block changed, else 0.  The shard's changed-block count is
// the tile scan's last inclusive prefix, so its EXP length is
// m = n_changed * B - tail (no atomics on a per-shard total: with one shard
// every tile of the split would add to the same two words).
struct ShardInfo {
    unsigned long long tail;
    unsigned int pad[14];
};

struct WsView {
    uint32_t* counters;            // 8 tile counters
    uint32_t* shard_ctr;           // W per-shard tile counters
    ShardInfo* info;               // W records
    ez_stats_t* shard_stats;       // W records (reuse+code3 without caller stats)
    unsigned long long* state_a;
    unsigned long long* state_b;
    void* bins;                    // StatsBins[n_bins]
    uint8_t* escbuf;               // W * L bytes of staged escapes (coded reuse) or NULL
    uint8_t* plbuf;                // 3 KB of staged planes per tile (coded reuse) or NULL
    unsigned long long* seg_a;     // scan-segment states, two arrays of W * segments
    unsigned long long* seg_b;
};

WsView ws_view(const ez_plan_s* p, void* ws);

// Scan segments per chunk of tpc tiles (k_scan.cu).
cudaError_t launch_accumulate_bf16(float* acc, const uint16_t* x, uint64_t n, int first, cudaStream_t s);
cudaError_t launch_zero(void* p, uint64_t bytes, cudaStream_t s);
uint64_t tile_scan_segments(uint64_t tpc);

// Inclusive prefixes, per chunk, of the per-tile counts in st[count * tpc].
cudaError_t launch_tile_scan(const ez_plan_s* p, unsigned long long* st, uint32_t count,
                             unsigned long long* seg_st, uint32_t* counter, uint32_t* abort,
                             uint32_t* dstatus, cudaStream_t s);
// The same for two state arrays of the same geometry (own segment states and
// counters) in one launch.
cudaError_t launch_tile_scan2(const ez_plan_s* p, unsigned long long* st0, unsigned long long* seg0,
                              uint32_t* counter0, unsigned long long* st1, unsigned long long* seg1,
                              uint32_t* counter1, uint32_t count, uint32_t* abort, uint32_t* dstatus,
                              cudaStream_t s);

cudaError_t launch_stats(const ez_plan_s* p, const uint16_t* x, uint64_t n, ez_stats_t* out,
                         const WsView& w, cudaStream_t s);

// Statistics of shards [first, first+count) of the plan (values at x + i*L),
// one record per shard.
cudaError_t launch_shard_stats(const ez_plan_s* p, const uint16_t* x, uint32_t first, uint32_t count,
                               ez_stats_t* out, const WsView& w, cudaStream_t s);

cudaError_t launch_code3_encode(const ez_plan_s* p, const uint16_t* x, uint32_t first,
                                uint32_t count, const ez_stats_t* st, uint8_t* out,
                                uint64_t* sizes, uint32_t* dstatus, const WsView& w,
                                cudaStream_t s);

cudaError_t launch_code3_decode(const ez_plan_s* p, const uint8_t* in, const uint64_t* offsets,
                                uint32_t first, uint32_t count, uint16_t* out,
                                uint32_t* dstatus, const WsView& w, cudaStream_t s,
                                float* acc = nullptr, int acc_first = 0);

cudaError_t launch_reuse_encode(const ez_plan_s* p, const uint16_t* x, uint32_t first,
                                uint32_t count, uint8_t* cache, int cold, uint8_t* out,
                                uint64_t* sizes, ez_stats_t* st, uint32_t* dstatus,
                                const WsView& w, cudaStream_t s);

// FP8 codecs (k_fp8.cu): worst-case chunk bytes of L values, and the kernels.
uint64_t fp8_slot_bytes(uint32_t codec, uint64_t L);
cudaError_t launch_fp8_stats(const ez_plan_s* p, const uint8_t* x, uint64_t n, ez_fp8_stats_t* out,
                             const WsView& w, cudaStream_t s);
cudaError_t launch_fp8_encode(const ez_plan_s* p, const uint8_t* x, uint32_t first, uint32_t count,
                              const ez_fp8_stats_t* st, uint8_t* out, uint64_t* sizes, uint32_t* dstatus,
                              const WsView& w, cudaStream_t s);
cudaError_t launch_fp8_decode(const ez_plan_s* p, const uint8_t* in, const uint64_t* offsets, uint32_t first,
                              uint32_t count, uint8_t* out, uint32_t* dstatus, cudaStream_t s);

cudaError_t launch_reuse_decode(const ez_plan_s* p, const uint8_t* in, const uint64_t* offsets,
                                uint64_t single_avail, uint32_t first, uint32_t count,
                                uint8_t* cache, uint16_t* out, uint32_t* dstatus,
                                const WsView& w, cudaStream_t s);

// Microscaled tensors (k_mx_quant.cu, k_mx_gated.cu, k_mx_matmul.cu); the
// formats are ez_mx_format values, 0 for a form that is not wanted.
cudaError_t launch_mx_quantize(const uint16_t* x, uint64_t rows, uint64_t cols, uint64_t ldx, int row_fmt,
                               uint8_t* row_codes, uint8_t* row_scales, int col_fmt, uint8_t* col_codes,
                               uint8_t* col_scales, cudaStream_t s);
cudaError_t launch_mx_dequantize(int fmt, const uint8_t* codes, const uint8_t* scales, uint64_t rows,
                                 uint64_t cols, uint16_t* out, uint64_t ldo, cudaStream_t s);
cudaError_t launch_mx_matmul(int fa, const uint8_t* ac, const uint8_t* as, uint64_t M, int fb, const uint8_t* bc,
                             const uint8_t* bs, uint64_t N, uint64_t K, const float* add, void* c, uint64_t ldc,
                             int f32, uint32_t* dstatus, cudaStream_t s);
void set_mx_wait_limit(uint32_t polls);
cudaError_t launch_mx_swiglu(int fmt, const uint16_t* gate, uint64_t ldg, const uint16_t* up, uint64_t ldu,
                             uint64_t rows, uint64_t cols, uint8_t* gate_codes, uint8_t* gate_scales,
                             uint8_t* up_codes, uint8_t* up_scales, uint16_t* h, uint64_t ldh, cudaStream_t s);
cudaError_t launch_mx_swiglu_backward(int fmt, const uint8_t* gate_codes, const uint8_t* gate_scales,
                                      const uint8_t* up_codes, const uint8_t* up_scales, uint64_t rows,
                                      uint64_t cols, const uint16_t* dh, uint64_t lddh, uint16_t* dgate,
                                      uint64_t ldg, uint16_t* dup, uint64_t ldu, uint16_t* h, uint64_t ldh,
                                      cudaStream_t s);

// Norm, routing and the experts' products (k_mx_norm.cu, k_moe.cu, k_mx_matmul.cu).
cudaError_t launch_mx_rms_norm(const uint16_t* x, uint64_t ldx, const uint16_t* residual, uint64_t ldr, uint64_t rows,
                               uint32_t cols, const uint16_t* weight, float eps, uint16_t* total, uint64_t ldt,
                               float* rstd, float* low, uint16_t* y, uint64_t ldy, int row_fmt, uint8_t* row_codes,
                               uint8_t* row_scales, int col_fmt, uint8_t* col_codes, uint8_t* col_scales,
                               cudaStream_t s);
uint64_t mx_rms_norm_ws(uint64_t rows, uint64_t cols);
cudaError_t launch_mx_rms_norm_backward(const uint16_t* dy, uint64_t lddy, const uint16_t* total, uint64_t ldt,
                                        const float* rstd, const uint16_t* weight, const uint16_t* dtotal,
                                        uint64_t lddt, uint64_t rows, uint32_t cols, uint16_t* dx, uint64_t ldx,
                                        const float* add, float* dweight, float* ws, cudaStream_t s);
uint64_t moe_sort_ws(uint64_t pairs, uint64_t experts);
cudaError_t launch_moe_sort(const void* ids, int id_bytes, uint64_t ld, uint64_t tokens, uint32_t choices,
                            uint32_t experts, uint64_t rows, int* counts, int* offsets, int* slots, int* sources,
                            void* ws, cudaStream_t s);
cudaError_t launch_moe_dispatch(const uint16_t* x, uint64_t ldx, uint32_t tokens, uint64_t cols, const int* offsets,
                                const int* sources, const int* slots, uint32_t choices, uint32_t experts,
                                uint64_t rows, const float* weights, int row_fmt, uint8_t* row_codes, uint8_t* row_scales,
                                int col_fmt, uint8_t* col_codes, uint8_t* col_scales, cudaStream_t s);
cudaError_t launch_moe_combine(const uint16_t* in, uint64_t ld, uint64_t rows, uint32_t cols, const int* slots,
                               const float* weights, uint32_t tokens, uint32_t choices, uint16_t* y, uint64_t ldy,
                               cudaStream_t s);
cudaError_t launch_moe_weight_gradient(const uint16_t* dy, uint64_t lddy, const uint16_t* in, uint64_t ld,
                                       uint64_t rows, uint32_t cols, const int* slots, uint32_t tokens,
                                       uint32_t choices, float* dweights, cudaStream_t s);
cudaError_t launch_moe_matmul(int fa, const uint8_t* ac, const uint8_t* as, uint64_t rows, int fb, const uint8_t* bc,
                              const uint8_t* bs, uint32_t experts, uint64_t N, uint64_t K, const int* counts,
                              const int* offsets, uint64_t pairs, void* c, uint64_t ldc, int f32, uint32_t* status,
                              cudaStream_t s);
cudaError_t launch_moe_gradient(int fa, const uint8_t* ac, const uint8_t* as, uint64_t N, int fb, const uint8_t* bc,
                                const uint8_t* bs, uint64_t K, uint64_t rows, uint32_t experts, const int* offsets,
                                const float* add, float* c, uint64_t ldc, uint32_t* status, cudaStream_t s);

}  // namespace ezk
