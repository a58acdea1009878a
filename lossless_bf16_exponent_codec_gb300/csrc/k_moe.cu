// k_moe.cu -- the way of tokens to their experts and back: (token, choice) pairs
// sorted by expert, the tokens' values gathered in that order into microscaled
// forms, and the weighted sum of what the experts return, with the gradients.
//
// Pair i = t k + j is the j-th choice of token t.  Expert e's rows are
// [offsets[e], offsets[e + 1]), multiples of 128 (whole scale tiles, so that each
// expert's part of a form is a form), the first counts[e] of them its pairs in
// ascending order; sources[row] is the pair there, -1 in the padding and behind
// the last expert; slots[i] is the row of pair i, -1 if its id names no expert.
//
// Measured on one GB300, 16384 tokens of 2048 values with 8 choices of 64 experts: the
// sort 14 us in two launches (bound by latency; one launch up to 4096 pairs, 8 us), to
// 4-bit rows and 8-bit columns 161 (the gather of 570 MB through L2, a token's row for
// each of its choices, and the codes' instructions, 2.7 a cycle: 8-bit columns alone 126;
// 4-bit rows alone, by tokens, 51, 4.0 TB/s of scattered rows), back 105 (604 MB, 5.8
// TB/s); the weights' gradients of 6 choices 90 (470 MB, 5.2).
#include "ez_internal.h"
#include "ez_mx_piece.cuh"

namespace ezk {
using namespace ezmx;

// ---- sort ----------------------------------------------------------------------------

namespace {

constexpr int kSortThreads = 512, kSortWarps = kSortThreads / 32;
// Up to kSortAlone pairs one CTA sorts them in one launch; beyond that a CTA takes a chunk,
// of kSortChunk pairs at least.  98304 pairs of 64 experts, both launches one after the
// other: chunks of 4096 25 us, of 2048 16, of 1024 14; 524288 of 256: 128 chunks 30 us, 256
// chunks, whose counts every CTA adds up, 34.
constexpr uint32_t kSortAlone = 4096, kSortChunk = 1024, kMaxChunks = 128;

struct SortArgs {
    const void* ids;
    uint64_t ld;                    // of ids
    uint32_t choices, experts, pairs, chunk, rows;
    uint32_t* hist;                 // [chunks, experts]; null for one chunk
    int *counts, *offsets, *slots, *sources;
};

// The expert of a pair, -1 for none.
template <typename Id>
__device__ __forceinline__ int expert_of(const SortArgs& a, uint32_t i)
{
    uint64_t at = i;
    if (a.ld != a.choices) {
        const uint32_t t = i / a.choices;
        at = t * a.ld + (i - t * a.choices);
    }
    const Id e = static_cast<const Id*>(a.ids)[at];
    return e >= 0 && e < (Id)a.experts ? (int)e : -1;
}

// Calls f(pair, expert, lanes of the warp with the same expert) over the pairs
// [begin, end) of a warp, 32 at a time.  The ids of 256 pairs are read together:
// one after the other, the way through 4096 pairs took 8 us.
template <typename Id, typename F>
__device__ __forceinline__ void each_pair(const SortArgs& a, uint32_t begin, uint32_t end, F f)
{
    constexpr int kBatch = 8;
    for (uint32_t i0 = begin + threadIdx.x % 32; __any_sync(ez::kFull, i0 < end); i0 += 32 * kBatch) {
        int e[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) e[b] = i0 + 32 * b < end ? expert_of<Id>(a, i0 + 32 * b) : -1;
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
            if (__any_sync(ez::kFull, i0 + 32 * b < end)) f(i0 + 32 * b, e[b], __match_any_sync(ez::kFull, e[b]));
    }
}

// Per-warp counts of a CTA's pairs: s_cnt [kSortWarps, experts], after a barrier.
template <typename Id>
__device__ __forceinline__ void count_pairs(const SortArgs& a, uint32_t begin, uint32_t end, uint32_t* s_cnt)
{
    for (uint32_t i = threadIdx.x; i < kSortWarps * a.experts; i += kSortThreads) s_cnt[i] = 0;
    __syncthreads();
    uint32_t* const mine = s_cnt + threadIdx.x / 32 * a.experts;
    each_pair<Id>(a, begin, end, [&](uint32_t, int e, uint32_t same) {
        if (e >= 0 && (int)(threadIdx.x % 32) == __ffs(same) - 1) mine[e] += __popc(same);
        __syncwarp();
    });
    __syncthreads();
}

// The part of a CTA's pairs that a warp takes: consecutive ones, in warp order.
__device__ __forceinline__ void part_of(const SortArgs& a, uint32_t& begin, uint32_t& end)
{
    const uint32_t c0 = blockIdx.x * a.chunk, c1 = min(a.pairs, c0 + a.chunk);
    const uint32_t per = (a.chunk / 32 + kSortWarps - 1) / kSortWarps * 32;
    begin = min(c1, c0 + threadIdx.x / 32 * per);
    end = min(c1, begin + per);
}

}  // namespace

template <typename Id>
__global__ void __launch_bounds__(kSortThreads) k_moe_count(const SortArgs a)
{
    extern __shared__ uint32_t s_cnt[];
    ez::grid_dep_launch();
    ez::grid_dep_wait();
    uint32_t begin, end;
    part_of(a, begin, end);
    count_pairs<Id>(a, begin, end, s_cnt);
    for (uint32_t e = threadIdx.x; e < a.experts; e += kSortThreads) {
        uint32_t n = 0;
        for (int w = 0; w < kSortWarps; ++w) n += s_cnt[w * a.experts + e];
        a.hist[(uint64_t)blockIdx.x * a.experts + e] = n;
    }
}

// Every CTA adds up the counts of all chunks itself and places its own pairs.
template <typename Id>
__global__ void __launch_bounds__(kSortThreads) k_moe_place(const SortArgs a)
{
    extern __shared__ uint32_t s_cnt[];
    uint32_t* const s_total = s_cnt + kSortWarps * a.experts;       // [experts]
    uint32_t* const s_offset = s_total + a.experts;                 // [experts + 1]
    __shared__ uint32_t s_warp[kSortWarps];
    ez::grid_dep_launch();
    ez::grid_dep_wait();
    const uint32_t t = threadIdx.x;
    uint32_t begin, end;
    part_of(a, begin, end);
    count_pairs<Id>(a, begin, end, s_cnt);
    // totals; the warps' counts become the pairs of each expert before the warp's
    for (uint32_t e = t; e < a.experts; e += kSortThreads) {
        uint32_t before = 0, total = 0;
        if (a.hist)
#pragma unroll 16
            for (uint32_t c = 0; c < gridDim.x; ++c) {
                const uint32_t n = a.hist[(uint64_t)c * a.experts + e];
                before += c < blockIdx.x ? n : 0;
                total += n;
            }
        uint32_t own = before;
        for (int w = 0; w < kSortWarps; ++w) {
            const uint32_t n = s_cnt[w * a.experts + e];
            s_cnt[w * a.experts + e] = own;
            own += n;
        }
        s_total[e] = a.hist ? total : own;
    }
    __syncthreads();
    // offsets: a scan of the totals, rounded up to tiles; a thread takes `per` experts
    const uint32_t per = (a.experts + kSortThreads - 1) / kSortThreads;
    uint32_t mine = 0;
    for (uint32_t e = t * per; e < min(a.experts, (t + 1) * per); ++e)
        mine += (s_total[e] + kTileRows - 1) / kTileRows * kTileRows;
    uint32_t upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const uint32_t v = __shfl_up_sync(ez::kFull, upto, d);
        if (t % 32 >= d) upto += v;
    }
    if (t % 32 == 31) s_warp[t / 32] = upto;
    __syncthreads();
    uint32_t at = upto - mine;
    at += __reduce_add_sync(ez::kFull, t % 32 < t / 32 ? s_warp[t % 32] : 0u);
    for (uint32_t e = t * per; e < min(a.experts, (t + 1) * per); ++e) {
        s_offset[e] = at;
        at += (s_total[e] + kTileRows - 1) / kTileRows * kTileRows;
        if (e + 1 == a.experts) s_offset[a.experts] = at;
    }
    __syncthreads();
    uint32_t* const rank = s_cnt + t / 32 * a.experts;
    each_pair<Id>(a, begin, end, [&](uint32_t i, int e, uint32_t same) {
        uint32_t row = 0;
        if (e >= 0) row = s_offset[e] + rank[e] + __popc(same & ((1u << (t % 32)) - 1u));
        __syncwarp();
        if (e >= 0 && (int)(t % 32) == __ffs(same) - 1) rank[e] += __popc(same);
        __syncwarp();
        if (i < end) a.slots[i] = e >= 0 ? (int)row : -1;
        if (e >= 0) a.sources[row] = (int)i;
    });
    // what no pair names: padding (an expert to a warp), the rows behind the last expert
    for (uint32_t e = blockIdx.x * kSortWarps + t / 32; e < a.experts; e += gridDim.x * kSortWarps) {
        const uint32_t from = s_offset[e] + s_total[e], to = s_offset[e + 1];
#pragma unroll
        for (uint32_t i = 0; i < kTileRows; i += 32)
            if (from + i + t % 32 < to) a.sources[from + i + t % 32] = -1;
    }
    for (uint32_t r = s_offset[a.experts] + blockIdx.x * kSortThreads + t; r < a.rows; r += gridDim.x * kSortThreads)
        a.sources[r] = -1;
    if (blockIdx.x == 0)
        for (uint32_t e = t; e <= a.experts; e += kSortThreads) {
            a.offsets[e] = (int)s_offset[e];
            if (e < a.experts) a.counts[e] = (int)s_total[e];
        }
}

// ---- dispatch ----------------------------------------------------------------------------

namespace {

struct TokenSource {
    const Rows& x;
    uint64_t cols;
    const int* token;               // of the piece's rows, -1: none
    const float* weight;            // theirs; null: 1
    uint64_t r0;
    template <bool FAST>
    __device__ __forceinline__ void start(Load8<FAST>& in, uint64_t r, uint64_t c) const
    {
        const int t = token[r - r0];
        in = Load8<FAST>{};
        if (t >= 0) in.start(x, (uint64_t)t, c, cols);
    }
    template <bool FAST>
    __device__ __forceinline__ uint4 finish(const Load8<FAST>& in, uint64_t, uint32_t lr, uint64_t c) const
    {
        if (!weight) return in.finish();
        // the padding's weight is one; what lies behind the row stays zero (and not -0)
        const float w = weight[lr];
        float v[8];
        unpack8(in.finish(), v);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = FAST || c + j < cols ? v[j] * w : 0.f;
        return pack8(v);
    }
};

struct Lined8 {
    uint4 v;
    __device__ __forceinline__ void start(const Rows& x, uint64_t row, int col, int) { v = ez::ld_v4_nc(x.p + row * x.ld + col); }
    __device__ __forceinline__ uint4 finish() const { return v; }
};

struct DispatchArgs {
    Rows x;
    uint32_t tokens, choices, experts, col_tiles;
    uint64_t rows, cols;
    const int *offsets, *sources, *slots;
    const float* weights;
    int lines;
    uint32_t token_ctas;            // k_moe_rows: CTAs of the tokens, before those of the padding
    Form row, col;
};

__device__ __forceinline__ int row_of(int slot, uint64_t rows)
{
    return slot >= 0 && (uint64_t)slot < rows ? slot : -1;
}

}  // namespace

// As the quantisation of the gathered matrix, a piece of a scale tile per CTA; the
// pieces behind the last expert are left as they were.
template <int ROW, int COL, int ROWS>
__global__ void __launch_bounds__(kThreadsMx, 4) k_moe_dispatch(const DispatchArgs a)
{
    __shared__ PieceShared<COL, ROWS> s;
    __shared__ int s_token[ROWS];
    __shared__ float s_weight[ROWS];
    ez::grid_dep_launch();
    const uint32_t t = threadIdx.x;
    const uint32_t piece = blockIdx.x / a.col_tiles, ct = blockIdx.x - piece * a.col_tiles;
    const uint64_t r0 = (uint64_t)piece * ROWS, c0 = (uint64_t)ct * kTileCols;
    ez::grid_dep_wait();
    const int i = t < ROWS ? a.sources[r0 + t] : -1, end = a.offsets[a.experts];     // both on their way at once
    if ((int64_t)r0 >= (int64_t)end) return;
    if (t < ROWS) {
        const bool some = i >= 0 && (uint32_t)i < a.tokens * a.choices;
        s_token[t] = some ? (int)((uint32_t)i / a.choices) : -1;
        s_weight[t] = some && a.weights ? a.weights[i] : 1.f;
    }
    __syncthreads();
    const TokenSource src{a.x, a.cols, s_token, a.weights ? s_weight : nullptr, r0};
    encode_piece<ROW, COL, ROWS>(src, a.lines && c0 + kTileCols <= a.cols, a.rows, a.cols, a.col_tiles, ct,
                                a.row, a.col, r0, s);
}

// The row form alone, of rows that are the tokens' own: each token is encoded once and its
// codes stored for all its choices, a block of 32 values by each lane, 1024 by a warp;
// the CTAs behind the tokens' clear the padding, 32 rows each.  16384 tokens of 2048
// values with 8 choices to 4 bits: 51 us; a token's row gathered and encoded for each of
// its choices, as above, took 124.  With a column form beside it the two launches would
// take 51 + 126 us against 161 for one.
template <int ROW, bool LINED>
__global__ void __launch_bounds__(kThreadsMx) k_moe_rows(const DispatchArgs a, uint32_t chunks)
{
    constexpr int kWords = Fmt<ROW>::kBits;
    ez::grid_dep_launch();
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint64_t pitch = code_pitch<ROW>(a.cols);
    ez::grid_dep_wait();
    if (blockIdx.x >= a.token_ctas) {
        const uint64_t r0 = (uint64_t)(blockIdx.x - a.token_ctas) * 32;
        if ((int64_t)r0 >= (int64_t)a.offsets[a.experts]) return;
        for (uint32_t lr = warp; lr < 32; lr += kThreadsMx / 32) {
            const uint64_t r = r0 + lr;
            const int i = a.sources[r];
            if (i >= 0 && (uint32_t)i < a.tokens * a.choices) continue;
            for (uint64_t c = 16 * lane; c < pitch; c += 16 * 32)
                *reinterpret_cast<uint4*>(a.row.codes + r * pitch + c) = make_uint4(0u, 0u, 0u, 0u);
            for (uint32_t ct = lane; ct < a.col_tiles; ct += 32) {
                const uint32_t blocks = min(4u, (uint32_t)ez::cdiv(a.cols, kBlock) - 4 * ct);
                *scale_word(a.row.scales, r / kTileRows * a.col_tiles + ct, (uint32_t)(r % kTileRows)) =
                    scale_byte<ROW>(0u) * (0x01010101u >> (32 - 8 * blocks));
            }
        }
        return;
    }
    const uint64_t item = (uint64_t)blockIdx.x * (kThreadsMx / 32) + warp, token = item / chunks;
    if (token >= a.tokens) return;
    const uint32_t b = (uint32_t)(item - token * chunks) * 1024 + 32 * lane;       // the block's first column
    uint32_t y[16], m = 0u;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        const uint32_t c = b + 8 * j;
        if (c < a.cols) {
            std::conditional_t<LINED, Lined8, Any8> in;
            in.start(a.x, token, (int)c, (int)a.cols);
            v = LINED ? in.finish() : only_columns(in.finish(), (int)c, (int)a.cols);
        }
        y[4 * j] = v.x;
        y[4 * j + 1] = v.y;
        y[4 * j + 2] = v.z;
        y[4 * j + 3] = v.w;
        m = mag_max(mag_max(m, v.x), mag_max(mag_max(v.y, v.z), v.w));
    }
    const bool in = b < a.cols;
    uint32_t s = in ? scale_byte<ROW>(mag_max(m, m >> 16) & 0x7FFFu) : 0u, code[kWords];
    encode_block<ROW>(y, s, code);
    s <<= lane % 4 * 8;                     // a tile's four blocks in one word
    s |= __shfl_xor_sync(ez::kFull, s, 1);
    s |= __shfl_xor_sync(ez::kFull, s, 2);
    for (uint32_t j = 0; j < a.choices; ++j) {
        const int r = row_of(__ldg(a.slots + token * a.choices + j), a.rows);
        if (r < 0) continue;
        if (in) store_codes32<ROW>(code, a.row.codes + (uint64_t)r * pitch + (uint64_t)b * Fmt<ROW>::kBits / 8);
        if (lane % 4 == 0 && b / kTileCols < a.col_tiles)
            *scale_word(a.row.scales, (uint64_t)r / kTileRows * a.col_tiles + b / kTileCols, (uint32_t)r % kTileRows) = s;
    }
}

// ---- combine -----------------------------------------------------------------------------

namespace {

struct CombineArgs {
    Rows in;                        // [rows, cols], the experts' order
    uint64_t rows;
    uint32_t tokens, choices, cols;
    const int* slots;
    const float* weights;           // null: ones
    uint16_t* y;
    uint64_t ldy;
};

constexpr int kCombineThreads = 256;

}  // namespace

// A thread: an aligned granule of a token's row of y, whatever its alignment (its
// first value is the row's misalignment before a multiple of 8), with the rows of
// eight choices (or four, of two granules each) in flight; the choices are added up
// in their order.  No thread waits for another: with a stage in shared memory for rows
// at odd alignments 1543 tokens of 6 choices and 2731 values took 31 us, so 21 with
// nothing in L2.
template <bool LINED>
__global__ void __launch_bounds__(kCombineThreads) k_moe_combine(const CombineArgs a, uint32_t granules, ez::FastDiv div)
{
    ez::grid_dep_launch();
    const uint32_t i = blockIdx.x * kCombineThreads + threadIdx.x, token = ez::fdiv(i, div), g = i - token * granules;
    ez::grid_dep_wait();
    if (token >= a.tokens) return;
    uint16_t* const y = a.y + token * a.ldy;
    const int c = 8 * (int)g - (LINED ? 0 : (int)(reinterpret_cast<uintptr_t>(y) & 15u) / 2);
    const int* const slots = a.slots + (uint64_t)token * a.choices;
    const float* const weights = a.weights + (uint64_t)token * a.choices;
    if (c >= (int)a.cols) return;
    constexpr uint32_t kFlightRows = LINED ? 8 : 4;
    float sum[8] = {};
    for (uint32_t j0 = 0; j0 < a.choices; j0 += kFlightRows) {
        std::conditional_t<LINED, Lined8, Any8> in[kFlightRows];
        int row[kFlightRows];
        float w[kFlightRows];
#pragma unroll
        for (uint32_t j = 0; j < kFlightRows; ++j) row[j] = j0 + j < a.choices ? row_of(slots[j0 + j], a.rows) : -1;
#pragma unroll
        for (uint32_t j = 0; j < kFlightRows; ++j) {
            w[j] = row[j] >= 0 && a.weights ? weights[j0 + j] : 1.f;
            if (row[j] >= 0) in[j].start(a.in, (uint64_t)row[j], c, (int)a.cols);
        }
#pragma unroll
        for (uint32_t j = 0; j < kFlightRows; ++j) {
            if (row[j] < 0) continue;
            float v[8];
            unpack8(in[j].finish(), v);
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[e] = __fmaf_rn(v[e], w[j], sum[e]);
        }
    }
    const uint4 v = pack8(sum);
    if (LINED || (c >= 0 && c + 8 <= (int)a.cols)) {
        *reinterpret_cast<uint4*>(y + c) = v;
    } else {                            // the ends of the row
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (c + e >= 0 && c + e < (int)a.cols) y[c + e] = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
    }
}

// The gradient of a weight: the token's dy times the row that it weighed, a warp
// to a token, eight choices (or four, of two granules each) at a time.
template <bool LINED>
__global__ void __launch_bounds__(kCombineThreads) k_moe_weight_gradient(const Rows dy, const CombineArgs a,
                                                                         float* dweights)
{
    constexpr uint32_t kChoices = LINED ? 8 : 4;
    ez::grid_dep_launch();
    const uint32_t lane = threadIdx.x % 32;
    const uint64_t token = (uint64_t)blockIdx.x * (kCombineThreads / 32) + threadIdx.x / 32;
    ez::grid_dep_wait();
    if (token >= a.tokens) return;
    using Load = std::conditional_t<LINED, Lined8, Any8>;
    for (uint32_t j0 = 0; j0 < a.choices; j0 += kChoices) {
        int row[kChoices];
        float sum[kChoices] = {}, more[kChoices] = {};
#pragma unroll
        for (uint32_t j = 0; j < kChoices; ++j)
            row[j] = j0 + j < a.choices ? row_of(a.slots[token * a.choices + j0 + j], a.rows) : -1;
        for (int c = 8 * (int)lane; c < (int)a.cols; c += 256) {
            Load d, in[kChoices];
            d.start(dy, token, c, (int)a.cols);
#pragma unroll
            for (uint32_t j = 0; j < kChoices; ++j)
                if (row[j] >= 0) in[j].start(a.in, (uint64_t)row[j], c, (int)a.cols);
            const uint4 g = LINED ? d.finish() : only_columns(d.finish(), c, (int)a.cols);
#pragma unroll
            for (uint32_t j = 0; j < kChoices; ++j) {
                if (row[j] < 0) continue;
                const uint4 v = LINED ? in[j].finish() : only_columns(in[j].finish(), c, (int)a.cols);
                sum[j] = add_products(v.x, g.x, sum[j]);
                more[j] = add_products(v.y, g.y, more[j]);
                sum[j] = add_products(v.z, g.z, sum[j]);
                more[j] = add_products(v.w, g.w, more[j]);
            }
        }
#pragma unroll
        for (uint32_t j = 0; j < kChoices; ++j) {
            sum[j] += more[j];
#pragma unroll
            for (int m = 16; m; m >>= 1) sum[j] += __shfl_xor_sync(ez::kFull, sum[j], m);
            if (lane == j && j0 + j < a.choices) dweights[token * a.choices + j0 + j] = sum[j];
        }
    }
}

// ---- host -----------------------------------------------------------------------------

namespace {

uint64_t chunk_of(uint64_t pairs)
{
    if (pairs <= kSortAlone) return kSortAlone;
    const uint64_t per = ez::rup(ez::cdiv(pairs, kMaxChunks), 32);
    return per > kSortChunk ? per : kSortChunk;
}

template <typename Id>
cudaError_t sort(SortArgs a, cudaStream_t s)
{
    const unsigned chunks = (unsigned)(a.pairs ? ez::cdiv(a.pairs, a.chunk) : 1);
    const size_t smem = ((kSortWarps + 2) * (size_t)a.experts + 1) * 4;
    static ez::PerDeviceAttr raised_count, raised_place;
    if (smem > 48 * 1024) {
        cudaError_t e = ez::max_dyn_smem_per_device(raised_place, k_moe_place<Id>, 96 * 1024);
        if (e == cudaSuccess) e = ez::max_dyn_smem_per_device(raised_count, k_moe_count<Id>, 96 * 1024);
        if (e != cudaSuccess) return e;
    }
    if (chunks == 1) {
        a.hist = nullptr;
    } else {
        const cudaError_t e = ez::launch_dependent(k_moe_count<Id>, chunks, kSortThreads, smem, s, a);
        if (e != cudaSuccess) return e;
    }
    return ez::launch_dependent(k_moe_place<Id>, chunks, kSortThreads, smem, s, a);
}

template <int ROW, int COL, int ROWS>
cudaError_t dispatch_rows(const DispatchArgs& a, cudaStream_t s)
{
    return ez::launch_dependent(k_moe_dispatch<ROW, COL, ROWS>, (unsigned)(a.rows / ROWS * a.col_tiles), kThreadsMx, 0,
                                s, a);
}
template <int ROW, int COL>
cudaError_t dispatch(const DispatchArgs& a, cudaStream_t s)
{
    const uint64_t per_sm = tiles_per_sm(a.rows, a.cols);
    if (per_sm >= 4) return dispatch_rows<ROW, COL, 128>(a, s);
    if constexpr (COL != 0)
        if (per_sm >= 2) return dispatch_rows<ROW, COL, 64>(a, s);
    return dispatch_rows<ROW, COL, 32>(a, s);
}
template <int ROW>
cudaError_t token_rows(DispatchArgs a, cudaStream_t s)
{
    const uint32_t chunks = (uint32_t)ez::cdiv(a.cols, 1024);
    a.token_ctas = (uint32_t)ez::cdiv((uint64_t)a.tokens * chunks, kThreadsMx / 32);
    const unsigned grid = a.token_ctas + (unsigned)(a.rows / 32);
    return a.lines && a.cols % 8 == 0 ? ez::launch_dependent(k_moe_rows<ROW, true>, grid, kThreadsMx, 0, s, a, chunks)
                                      : ez::launch_dependent(k_moe_rows<ROW, false>, grid, kThreadsMx, 0, s, a, chunks);
}
template <int ROW>
cudaError_t dispatch_col(int col_fmt, const DispatchArgs& a, cudaStream_t s)
{
    if constexpr (ROW != 0)
        if (!col_fmt && !a.weights) return token_rows<ROW>(a, s);
    switch (col_fmt) {
        case EZ_MX_E2M1: return dispatch<ROW, EZ_MX_E2M1>(a, s);
        case EZ_MX_E4M3: return dispatch<ROW, EZ_MX_E4M3>(a, s);
        case EZ_MX_E5M2: return dispatch<ROW, EZ_MX_E5M2>(a, s);
    }
    if constexpr (ROW != 0) return dispatch<ROW, 0>(a, s);
    return cudaErrorInvalidValue;
}

}  // namespace

uint64_t moe_sort_ws(uint64_t pairs, uint64_t experts)
{
    const uint64_t chunks = ez::cdiv(pairs, chunk_of(pairs));
    return chunks > 1 ? chunks * experts * 4 : 0;
}

cudaError_t launch_moe_sort(const void* ids, int id_bytes, uint64_t ld, uint64_t tokens, uint32_t choices,
                            uint32_t experts, uint64_t rows, int* counts, int* offsets, int* slots, int* sources,
                            void* ws, cudaStream_t s)
{
    SortArgs a{};
    a.ids = ids;
    a.ld = ld;
    a.choices = choices;
    a.experts = experts;
    a.pairs = (uint32_t)(tokens * choices);
    a.chunk = (uint32_t)chunk_of(a.pairs);
    a.rows = (uint32_t)rows;
    a.hist = static_cast<uint32_t*>(ws);
    a.counts = counts;
    a.offsets = offsets;
    a.slots = slots;
    a.sources = sources;
    return id_bytes == 8 ? sort<int64_t>(a, s) : sort<int32_t>(a, s);
}

cudaError_t launch_moe_dispatch(const uint16_t* x, uint64_t ldx, uint32_t tokens, uint64_t cols, const int* offsets,
                                const int* sources, const int* slots, uint32_t choices, uint32_t experts,
                                uint64_t rows, const float* weights, int row_fmt, uint8_t* row_codes, uint8_t* row_scales,
                                int col_fmt, uint8_t* col_codes, uint8_t* col_scales, cudaStream_t s)
{
    DispatchArgs a{};
    a.x = make_rows(x, tokens, cols, ldx);
    a.tokens = tokens;
    a.choices = choices;
    a.experts = experts;
    a.col_tiles = (uint32_t)ez::cdiv(cols, kTileCols);
    a.rows = rows;
    a.cols = cols;
    a.offsets = offsets;
    a.sources = sources;
    a.slots = slots;
    a.weights = weights;
    a.lines = lined(x, tokens, ldx);
    a.row = Form{row_codes, row_scales};
    a.col = Form{col_codes, col_scales};
    switch (row_fmt) {
        case EZ_MX_E2M1: return dispatch_col<EZ_MX_E2M1>(col_fmt, a, s);
        case EZ_MX_E4M3: return dispatch_col<EZ_MX_E4M3>(col_fmt, a, s);
        case EZ_MX_E5M2: return dispatch_col<EZ_MX_E5M2>(col_fmt, a, s);
    }
    return dispatch_col<0>(col_fmt, a, s);
}

cudaError_t launch_moe_combine(const uint16_t* in, uint64_t ld, uint64_t rows, uint32_t cols, const int* slots,
                               const float* weights, uint32_t tokens, uint32_t choices, uint16_t* y, uint64_t ldy,
                               cudaStream_t s)
{
    CombineArgs a{make_rows(in, rows, cols, ld), rows, tokens, choices, cols, slots, weights, y, ldy};
    const bool lines = cols % 8 == 0 && lined(in, rows, ld) && lined(y, tokens, ldy);
    const uint32_t granules = (uint32_t)ez::cdiv(lines ? cols : cols + 7ull, 8);
    // as many tokens at a time as 32 bits count granules of
    const uint64_t most = ez::cdiv((1ull << 31) - kCombineThreads, granules) - 1;
    for (uint64_t t = 0; t < tokens; t += most, a.slots += most * choices, a.y += most * ldy) {
        if (t) a.weights = weights ? weights + t * choices : nullptr;
        a.tokens = (uint32_t)ez::umin64(most, tokens - t);
        const cudaError_t e = ez::launch_dependent(lines ? k_moe_combine<true> : k_moe_combine<false>,
                                                   (unsigned)ez::cdiv((uint64_t)a.tokens * granules, kCombineThreads),
                                                   kCombineThreads, 0, s, a, granules, ez::make_fastdiv(granules));
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_moe_weight_gradient(const uint16_t* dy, uint64_t lddy, const uint16_t* in, uint64_t ld,
                                       uint64_t rows, uint32_t cols, const int* slots, uint32_t tokens,
                                       uint32_t choices, float* dweights, cudaStream_t s)
{
    CombineArgs a{make_rows(in, rows, cols, ld), rows, tokens, choices, cols, slots, nullptr, nullptr, 0};
    const Rows d = make_rows(dy, tokens, cols, lddy);
    const bool lines = cols % 8 == 0 && lined(in, rows, ld) && lined(dy, tokens, lddy);
    return ez::launch_dependent(lines ? k_moe_weight_gradient<true> : k_moe_weight_gradient<false>,
                                (unsigned)ez::cdiv(tokens, kCombineThreads / 32), kCombineThreads, 0, s, d, a,
                                dweights);
}

}  // namespace ezk
