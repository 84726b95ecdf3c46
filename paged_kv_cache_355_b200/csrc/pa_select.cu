// pa_select.cu -- choosing the blocks a query attends to: per-block key
// bounds, a block score from them, and the choice of the best blocks.
//
// bounds: for each block and kv head, per channel the smallest and the largest
//   key value over the block's tokens.
// score:  for each query row, kv head and block, the largest over the group's
//   query heads of  sum_d max(q_d * lo_d, q_d * hi_d), which no dot product of
//   q with a key of the block exceeds.
// select: the first and the last blocks of the row, then those of the largest
//   score; equal scores go to the lower block.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "pa.h"
#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_rows.cuh"

namespace pa {
namespace {

constexpr int kWarps = 4;

// ---------------------------------------------------------------------------
// key bounds
// ---------------------------------------------------------------------------
struct BoundsParams {
    const void* k_pool;
    void* key_bounds;
    const int32_t* block_tables;
    int max_blocks_per_seq;
    const int32_t* context_lens;
    const int32_t* query_start;  // NULL: one new token a sequence
    int max_query_len, batch, num_kv_heads, block_size;
    int64_t num_blocks;
    int max_touched;  // blocks that max_query_len new tokens can lie in
    int* err;
};

// One warp per (sequence, block with new tokens, kv head): it reads the rows
// of the block's tokens, 32 / (D / 8) rows at a time, keeps the running
// minimum and maximum of its 8 channels, and joins the rows' lanes by
// shuffles.  Bound by the read of the keys: one pass, D * 2 values written for
// block_size * D read.  The whole block is read again for every new token
// rather than its bounds updated, so that the call can be repeated and follows
// a copied or rewritten block.
template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) key_bounds_kernel(const BoundsParams p) {
    constexpr int kLanes = D / kChunk;
    constexpr int kRows = 32 / kLanes;
    griddep_wait();
    griddep_launch_dependents();
    const int64_t unit = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int64_t per_seq = (int64_t)p.max_touched * p.num_kv_heads;
    const int64_t b = unit / per_seq;
    if (b >= p.batch) return;
    const int64_t rem = unit - b * per_seq;
    const int i = (int)(rem / p.num_kv_heads);
    const int h = (int)(rem - (int64_t)i * p.num_kv_heads);
    const int lane = threadIdx.x & 31;
    const int sub = lane / kLanes, chunk = lane % kLanes;

    const int L = p.context_lens[b];
    int64_t n = L > 0 ? 1 : 0;
    if (p.query_start) n = (int64_t)p.query_start[b + 1] - p.query_start[b];
    if (L < 0 || n < 0 || n > L || n > p.max_query_len || L > (int64_t)p.max_blocks_per_seq * p.block_size) {
        if (rem == 0 && lane == 0) record_error(p.err, PA_ERR_BAD_BLOCK_ID);
        return;
    }
    if (n == 0) return;
    const int64_t j = (L - n) / p.block_size + i;
    if (j > (L - 1) / p.block_size) return;
    const int64_t blk = p.block_tables[b * p.max_blocks_per_seq + j];
    if (blk < 0 || blk >= p.num_blocks) {
        if (h == 0 && lane == 0) record_error(p.err, PA_ERR_BAD_BLOCK_ID);
        return;
    }
    const int64_t left = L - j * p.block_size;
    const int held = left < p.block_size ? (int)left : p.block_size;  // tokens of the block
    const T* src = static_cast<const T*>(p.k_pool) + ((blk * p.num_kv_heads + h) * p.block_size) * D + chunk * kChunk;

    float lo[kChunk], hi[kChunk];
#pragma unroll
    for (int e = 0; e < kChunk; ++e) {
        lo[e] = __int_as_float(0x7f800000);
        hi[e] = __int_as_float(0xff800000);
    }
#pragma unroll 4
    for (int t = sub; t < held; t += kRows) {
        Chunk<T> raw;
        raw.load(src + t * D);
        float x[kChunk];
        raw.to_f32(x);
#pragma unroll
        for (int e = 0; e < kChunk; ++e) {
            lo[e] = min_nan(lo[e], x[e]);
            hi[e] = max_nan(hi[e], x[e]);
        }
    }
#pragma unroll
    for (int m = kLanes; m < 32; m <<= 1) {
#pragma unroll
        for (int e = 0; e < kChunk; ++e) {
            lo[e] = min_nan(lo[e], __shfl_xor_sync(0xffffffffu, lo[e], m));
            hi[e] = max_nan(hi[e], __shfl_xor_sync(0xffffffffu, hi[e], m));
        }
    }
    if (sub == 0) {
        T* dst = static_cast<T*>(p.key_bounds) + ((blk * p.num_kv_heads + h) * 2) * D + chunk * kChunk;
        Chunk<T> out;
        out.from_f32(lo);
        out.store(dst);
        out.from_f32(hi);
        out.store(dst + D);
    }
}

// ---------------------------------------------------------------------------
// block scores
// ---------------------------------------------------------------------------
struct ScoreParams {
    const void *q, *key_bounds;
    const int32_t *block_tables, *seq_ids, *context_lens;
    int max_blocks_per_seq, batch, max_context_len, block_size;
    float* scores;
    int64_t score_stride;  // blocks of one (row, kv head) of scores
    int64_t num_rows;
    int num_q_heads, num_kv_heads;
    int64_t num_blocks;
    int tiles;  // CTAs along the blocks of one (row, kv head)
    int* err;
};

// The row's block table and its number of blocks; false (after recording the
// error once, by `recorder`) where the sequence or the length is bad.
__device__ __forceinline__ bool row_blocks(const int32_t* block_tables, const int32_t* seq_ids,
                                           const int32_t* context_lens, int64_t row, int batch, int max_blocks_per_seq,
                                           int64_t max_len, int block_size, bool recorder, int* err,
                                           const int32_t*& table, int& blocks) {
    const int64_t seq = seq_ids ? (int64_t)seq_ids[row] : row;
    const int L = context_lens[row];
    if (seq < 0 || seq >= batch || L < 0 || L > max_len) {
        if (recorder) record_error(err, PA_ERR_BAD_BLOCK_ID);
        return false;
    }
    table = block_tables + seq * max_blocks_per_seq;
    blocks = (int)(((int64_t)L + block_size - 1) / block_size);
    return true;
}

constexpr int kScoreBlocksPerWarp = 16;

// CUDA-core form: D / 8 lanes hold one block's two rows, 8 channels each.
template <typename T, int D, int G>
__global__ void __launch_bounds__(kWarps * 32) block_scores_kernel(const ScoreParams p) {
    constexpr int kLanes = D / kChunk;
    constexpr int kRows = 32 / kLanes;
    griddep_wait();
    griddep_launch_dependents();
    const int64_t unit = blockIdx.x / p.tiles;
    const int tile = (int)(blockIdx.x - unit * p.tiles);
    const int64_t row = unit / p.num_kv_heads;
    const int h = (int)(unit - row * p.num_kv_heads);
    const int lane = threadIdx.x & 31;
    const int sub = lane / kLanes, chunk = lane % kLanes;
    const int32_t* table;
    int blocks;
    if (!row_blocks(p.block_tables, p.seq_ids, p.context_lens, row, p.batch, p.max_blocks_per_seq, p.max_context_len,
                    p.block_size, tile == 0 && h == 0 && threadIdx.x == 0, p.err, table, blocks))
        return;
    const int first = (tile * kWarps + (threadIdx.x >> 5)) * kScoreBlocksPerWarp;
    if (first >= blocks) return;
    const int end = min(blocks, first + kScoreBlocksPerWarp);

    float q[G][kChunk];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        Chunk<T> raw;
        raw.load(static_cast<const T*>(p.q) + ((row * p.num_q_heads + h * G + g) * D) + chunk * kChunk);
        raw.to_f32(q[g]);
    }
    float* out = p.scores + unit * p.score_stride;
    for (int base = first; base < end; base += kRows) {
        const int j = base + sub;
        bool ok = j < end;
        int64_t blk = -1;
        if (ok) {
            blk = table[j];
            if (blk < 0 || blk >= p.num_blocks) {
                record_error(p.err, PA_ERR_BAD_BLOCK_ID);
                ok = false;
            }
        }
        float lo[kChunk] = {}, hi[kChunk] = {};
        if (ok) {
            const T* src = static_cast<const T*>(p.key_bounds) + ((blk * p.num_kv_heads + h) * 2) * D + chunk * kChunk;
            Chunk<T> raw;
            raw.load(src);
            raw.to_f32(lo);
            raw.load(src + D);
            raw.to_f32(hi);
        }
        float best = __int_as_float(0xff800000);
#pragma unroll
        for (int g = 0; g < G; ++g) {
            float sum = 0.f;
#pragma unroll
            for (int e = 0; e < kChunk; ++e) sum = fmaf(q[g][e], q[g][e] < 0.f ? lo[e] : hi[e], sum);
#pragma unroll
            for (int m = kLanes / 2; m; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
            best = max_nan(best, sum);
        }
        if (ok && chunk == 0) out[j] = best;
    }
}

// ---------------------------------------------------------------------------
// selection
// ---------------------------------------------------------------------------
struct SelectParams {
    const float* scores;
    int64_t score_stride;
    const int32_t* context_lens;
    int max_context_len, block_size;
    int32_t* selected;
    int max_selected, num_first, num_last;
    int64_t num_rows;
    int num_kv_heads;
    int* err;
};

// A score as an integer of the same order: NaN above +inf, -0 equal to +0,
// everything below kForced.
constexpr uint32_t kForced = 0xffffffffu;
__device__ __forceinline__ uint32_t score_key(float x) {
    if (x != x) return kForced - 1;
    const uint32_t u = __float_as_uint(x + 0.0f);  // -0 + 0 = +0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

constexpr int kSelectThreads = 256;
constexpr int kSelectWarps = kSelectThreads / 32;

// One CTA per (row, kv head).  The K-th largest key is found digit by digit
// (radix select: a histogram of 256 counts of the keys that still match the
// digits found so far), then the blocks above it and the lowest-numbered
// blocks equal to it are written in ascending order, their places from warp
// ballots.  Counts are integers, so the order of the atomics changes nothing.
__global__ void __launch_bounds__(kSelectThreads) select_blocks_kernel(const SelectParams p) {
    __shared__ int hist[256];
    __shared__ int warp_above[kSelectWarps], warp_equal[kSelectWarps];
    __shared__ uint32_t s_prefix;
    __shared__ int s_want;
    griddep_wait();
    griddep_launch_dependents();
    const int64_t unit = blockIdx.x;
    const int64_t row = unit / p.num_kv_heads;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int L = p.context_lens[row];
    int32_t* out = p.selected + unit * p.max_selected;
    int blocks = 0;
    if (L < 0 || L > p.max_context_len) {
        if (unit == row * p.num_kv_heads && tid == 0) record_error(p.err, PA_ERR_BAD_BLOCK_ID);
    } else {
        blocks = (int)(((int64_t)L + p.block_size - 1) / p.block_size);
    }
    const int K = p.max_selected;
    if (blocks <= K) {
        for (int i = tid; i < K; i += kSelectThreads) out[i] = i < blocks ? i : -1;
        return;
    }
    const float* scores = p.scores + unit * p.score_stride;
    const int last = blocks - p.num_last;
    auto key_of = [&](int j) { return j < p.num_first || j >= last ? kForced : score_key(scores[j]); };

    // the K-th largest key: `prefix` holds the digits found, `want` how many of
    // the keys that start with them are still to be taken
    uint32_t prefix = 0, mask = 0;
    int want = K;
    for (int shift = 24; shift >= 0; shift -= 8) {
        hist[tid] = 0;
        __syncthreads();
        for (int j = tid; j < blocks; j += kSelectThreads) {
            const uint32_t key = key_of(j);
            if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & 255], 1);
        }
        __syncthreads();
        if (tid == 0) {
            int left = want, d = 255;
            for (; d > 0 && hist[d] < left; --d) left -= hist[d];
            s_prefix = prefix | ((uint32_t)d << shift);
            s_want = left;
        }
        __syncthreads();
        prefix = s_prefix;
        want = s_want;
        mask |= 0xffu << shift;
    }

    // ascending output: `want` blocks equal to the threshold, and all above it
    int done_above = 0, done_equal = 0;
    for (int base = 0; base < blocks; base += kSelectThreads) {
        const int j = base + tid;
        const uint32_t key = j < blocks ? key_of(j) : 0;
        const bool above = j < blocks && key > prefix, equal = j < blocks && key == prefix;
        const unsigned ma = __ballot_sync(0xffffffffu, above), me = __ballot_sync(0xffffffffu, equal);
        if (lane == 0) {
            warp_above[warp] = __popc(ma);
            warp_equal[warp] = __popc(me);
        }
        __syncthreads();
        int a = done_above, e = done_equal;
#pragma unroll
        for (int w = 0; w < kSelectWarps; ++w) {
            if (w < warp) {
                a += warp_above[w];
                e += warp_equal[w];
            }
            done_above += warp_above[w];
            done_equal += warp_equal[w];
        }
        const unsigned below = (1u << lane) - 1u;
        a += __popc(ma & below);
        e += __popc(me & below);
        if (above || (equal && e < want)) out[a + min(e, want)] = j;
        __syncthreads();
    }
}

template <typename T, int D>
int launch_scores_d(const ScoreParams& p, cudaStream_t st) {
    const int64_t grid = p.num_rows * p.num_kv_heads * p.tiles;
    if (grid > 0x7fffffff) return PA_ERR_UNSUPPORTED;
    const dim3 g((unsigned)grid), b(kWarps * 32);
    switch (p.num_q_heads / p.num_kv_heads) {
        case 1: return launch_pdl(block_scores_kernel<T, D, 1>, g, b, 0, st, p);
        case 2: return launch_pdl(block_scores_kernel<T, D, 2>, g, b, 0, st, p);
        case 4: return launch_pdl(block_scores_kernel<T, D, 4>, g, b, 0, st, p);
        case 8: return launch_pdl(block_scores_kernel<T, D, 8>, g, b, 0, st, p);
        case 16: return launch_pdl(block_scores_kernel<T, D, 16>, g, b, 0, st, p);
    }
    return PA_ERR_UNSUPPORTED;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" int pa_update_key_bounds(const void* k_pool, void* key_bounds, const int32_t* block_tables,
                                    int max_blocks_per_seq, const int32_t* context_lens, const int32_t* query_start,
                                    int max_query_len, int batch, int num_kv_heads, int head_dim, int block_size,
                                    int64_t num_blocks, int dtype, void* stream) {
    PA_NVTX_RANGE("pa_update_key_bounds");
    if (batch < 0 || max_blocks_per_seq < 0 || max_query_len < 0 || num_kv_heads <= 0 || head_dim <= 0 ||
        block_size <= 0 || num_blocks < 0 || !valid_dtype(dtype) || (!query_start && max_query_len < 1))
        return PA_ERR_INVALID_ARG;
    if (!supported_head_dim(head_dim) || !supported_block_size(block_size)) return PA_ERR_UNSUPPORTED;
    if (batch == 0 || max_query_len == 0) return PA_OK;
    if (!k_pool || !key_bounds || !block_tables || !context_lens || !aligned16(k_pool) || !aligned16(key_bounds))
        return PA_ERR_INVALID_ARG;
    BoundsParams p = {};
    p.k_pool = k_pool;
    p.key_bounds = key_bounds;
    p.block_tables = block_tables;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.context_lens = context_lens;
    p.query_start = query_start;
    p.max_query_len = query_start ? max_query_len : 1;
    p.batch = batch;
    p.num_kv_heads = num_kv_heads;
    p.block_size = block_size;
    p.num_blocks = num_blocks;
    // n tokens that end anywhere lie in at most (n - 2) / bs + 2 blocks
    p.max_touched = (int)(((int64_t)p.max_query_len + block_size - 2) / block_size) + 1;
    if (p.max_touched > max_blocks_per_seq) p.max_touched = max_blocks_per_seq > 0 ? max_blocks_per_seq : 1;
    const int64_t units = (int64_t)batch * p.max_touched * num_kv_heads;
    const int64_t blocks = (units + kWarps - 1) / kWarps;
    if (blocks > 0x7fffffff) return PA_ERR_UNSUPPORTED;
    p.err = error_word_ptr();
    if (!p.err) return PA_ERR_CUDA;
    const dim3 g((unsigned)blocks), b(kWarps * 32);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dtype == PA_BF16)
        return head_dim == 128 ? launch_pdl(key_bounds_kernel<__nv_bfloat16, 128>, g, b, 0, st, p)
                               : launch_pdl(key_bounds_kernel<__nv_bfloat16, 64>, g, b, 0, st, p);
    return head_dim == 128 ? launch_pdl(key_bounds_kernel<float, 128>, g, b, 0, st, p)
                           : launch_pdl(key_bounds_kernel<float, 64>, g, b, 0, st, p);
}

extern "C" int pa_block_scores(const void* q, const void* key_bounds, const int32_t* block_tables,
                               int max_blocks_per_seq, const int32_t* seq_ids, const int32_t* context_lens,
                               int max_context_len, int block_size, float* scores, int64_t score_stride,
                               int64_t num_rows, int batch, int num_q_heads, int num_kv_heads, int head_dim,
                               int64_t num_blocks, int dtype, void* stream) {
    PA_NVTX_RANGE("pa_block_scores");
    if (num_rows < 0 || batch < 0 || max_blocks_per_seq < 0 || max_context_len < 0 || num_q_heads <= 0 ||
        num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || num_blocks < 0 || !valid_dtype(dtype) ||
        num_q_heads % num_kv_heads != 0)
        return PA_ERR_INVALID_ARG;
    if (!supported_head_dim(head_dim) || !supported_block_size(block_size) ||
        !supported_group(num_q_heads / num_kv_heads, dtype))
        return PA_ERR_UNSUPPORTED;
    const int64_t tiles_of = ((int64_t)max_context_len + block_size - 1) / block_size;
    if (max_context_len > (int64_t)max_blocks_per_seq * block_size || score_stride < tiles_of ||
        (!seq_ids && num_rows > batch))
        return PA_ERR_INVALID_ARG;
    if (num_rows == 0 || max_context_len == 0) return PA_OK;
    if (!q || !key_bounds || !block_tables || !context_lens || !scores || !aligned16(q) || !aligned16(key_bounds) ||
        !aligned16(scores))
        return PA_ERR_INVALID_ARG;
    ScoreParams p = {};
    p.q = q;
    p.key_bounds = key_bounds;
    p.block_tables = block_tables;
    p.seq_ids = seq_ids;
    p.context_lens = context_lens;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.batch = batch;
    p.max_context_len = max_context_len;
    p.block_size = block_size;
    p.scores = scores;
    p.score_stride = score_stride;
    p.num_rows = num_rows;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.num_blocks = num_blocks;
    p.tiles = (int)((tiles_of + kWarps * kScoreBlocksPerWarp - 1) / (kWarps * kScoreBlocksPerWarp));
    p.err = error_word_ptr();
    if (!p.err) return PA_ERR_CUDA;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dtype == PA_BF16)
        return head_dim == 128 ? launch_scores_d<__nv_bfloat16, 128>(p, st) : launch_scores_d<__nv_bfloat16, 64>(p, st);
    return head_dim == 128 ? launch_scores_d<float, 128>(p, st) : launch_scores_d<float, 64>(p, st);
}

extern "C" int pa_select_blocks(const float* scores, int64_t score_stride, const int32_t* context_lens,
                                int max_context_len, int block_size, int32_t* selected, int max_selected,
                                int num_first, int num_last, int64_t num_rows, int num_kv_heads, void* stream) {
    PA_NVTX_RANGE("pa_select_blocks");
    if (num_rows < 0 || num_kv_heads <= 0 || max_context_len < 0 || block_size <= 0 || max_selected <= 0 ||
        num_first < 0 || num_last < 0 || (int64_t)num_first + num_last > max_selected)
        return PA_ERR_INVALID_ARG;
    if (!supported_block_size(block_size)) return PA_ERR_UNSUPPORTED;
    if (score_stride < ((int64_t)max_context_len + block_size - 1) / block_size) return PA_ERR_INVALID_ARG;
    if (num_rows == 0) return PA_OK;
    if (!scores || !context_lens || !selected || !aligned16(scores) || !aligned16(selected)) return PA_ERR_INVALID_ARG;
    const int64_t grid = num_rows * num_kv_heads;
    if (grid > 0x7fffffff) return PA_ERR_UNSUPPORTED;
    SelectParams p = {};
    p.scores = scores;
    p.score_stride = score_stride;
    p.context_lens = context_lens;
    p.max_context_len = max_context_len;
    p.block_size = block_size;
    p.selected = selected;
    p.max_selected = max_selected;
    p.num_first = num_first;
    p.num_last = num_last;
    p.num_rows = num_rows;
    p.num_kv_heads = num_kv_heads;
    p.err = error_word_ptr();
    if (!p.err) return PA_ERR_CUDA;
    return launch_pdl(select_blocks_kernel, dim3((unsigned)grid), dim3(kSelectThreads), 0,
                      static_cast<cudaStream_t>(stream), p);
}
