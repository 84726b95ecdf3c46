// pa_sparse.cu -- decode attention over a list of chosen blocks of each row
// and kv head, instead of over the whole context.
//
// For each row r and query head h of kv head g, over the tokens t < L of the
// blocks that selected[r][g] lists:
//   out[r][h] = sum_t softmax(scale * <q[r][h], K_t>)_t V_t.
// One pass with a running maximum and sum (log2 domain, fp32).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "pa.h"
#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_rows.cuh"

namespace pa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

struct SparseParams {
    const void *q, *k_pool, *v_pool;
    const int32_t *block_tables, *seq_ids, *context_lens, *selected;
    int max_blocks_per_seq, batch, max_selected, block_size;
    void* out;
    int out_bf16;
    float scale_log2;
    int64_t num_rows;
    int num_q_heads, num_kv_heads;
    int64_t num_blocks;
    int* err;
};

__device__ __forceinline__ void store_out(const SparseParams& p, int64_t at, float x) {
    if (p.out_bf16)
        static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16(x);
    else
        static_cast<float*>(p.out)[at] = x;
}

constexpr int kSimtWarps = 8;

// CUDA-core form.  One CTA per (row, kv head, G query heads); its warps take
// the listed blocks in turn.  D / 8 lanes hold one token's row; each such lane
// group keeps its own running maximum, sum and output, joined at the end.
template <typename T, int D, int G>
__global__ void __launch_bounds__(kSimtWarps * 32) sparse_simt_kernel(const SparseParams p, int head_slices) {
    constexpr int kLanes = D / kChunk;
    constexpr int kRows = 32 / kLanes;
    constexpr int kStates = kSimtWarps * kRows;
    __shared__ float s_m[kStates][G], s_l[kStates][G];
    __shared__ float s_o[kSimtWarps][G][D];
    griddep_wait();
    griddep_launch_dependents();
    const int64_t unit = blockIdx.x;
    const int64_t rg = unit / head_slices;  // (row, kv head)
    const int slice = (int)(unit - rg * head_slices);
    const int64_t row = rg / p.num_kv_heads;
    const int h = (int)(rg - row * p.num_kv_heads);
    const int head0 = h * (p.num_q_heads / p.num_kv_heads) + slice * G;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane / kLanes, chunk = lane % kLanes;

    const int64_t seq = p.seq_ids ? (int64_t)p.seq_ids[row] : row;
    const int L = p.context_lens[row];
    bool row_ok = seq >= 0 && seq < p.batch && L >= 0 && L <= (int64_t)p.max_blocks_per_seq * p.block_size;
    if (!row_ok && threadIdx.x == 0) record_error(p.err, PA_ERR_BAD_BLOCK_ID);
    const int32_t* table = p.block_tables + (row_ok ? seq : 0) * p.max_blocks_per_seq;
    const int32_t* list = p.selected + rg * p.max_selected;

    float q[G][kChunk], o[G][kChunk], m[G], l[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        Chunk<T> raw;
        raw.load(static_cast<const T*>(p.q) + (row * p.num_q_heads + head0 + g) * D + chunk * kChunk);
        raw.to_f32(q[g]);
        m[g] = __int_as_float(0xff800000);
        l[g] = 0.f;
#pragma unroll
        for (int e = 0; e < kChunk; ++e) {
            q[g][e] *= p.scale_log2;
            o[g][e] = 0.f;
        }
    }
    for (int i = warp; row_ok && i < p.max_selected; i += kSimtWarps) {
        const int j = list[i];
        if (j < 0) continue;
        int64_t blk = -1;
        if ((int64_t)j * p.block_size < L) blk = table[j];
        if (blk < 0 || blk >= p.num_blocks) {
            if (lane == 0) record_error(p.err, PA_ERR_BAD_BLOCK_ID);
            continue;
        }
        const int held = min(p.block_size, L - j * p.block_size);
        const int64_t base = ((blk * p.num_kv_heads + h) * p.block_size) * D + chunk * kChunk;
        for (int t0 = 0; t0 < held; t0 += kRows) {
            const int t = t0 + sub;
            const bool in = t < held;
            float k[kChunk] = {}, v[kChunk] = {};
            if (in) {
                Chunk<T> raw;
                raw.load(static_cast<const T*>(p.k_pool) + base + t * D);
                raw.to_f32(k);
                raw.load(static_cast<const T*>(p.v_pool) + base + t * D);
                raw.to_f32(v);
            }
#pragma unroll
            for (int g = 0; g < G; ++g) {
                float s = 0.f;
#pragma unroll
                for (int e = 0; e < kChunk; ++e) s = fmaf(q[g][e], k[e], s);
#pragma unroll
                for (int x = kLanes / 2; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
                if (!in) continue;
                const float top = fmaxf(m[g], s);
                const float base_m = top == __int_as_float(0xff800000) ? 0.f : top;
                const float keep = exp2f(m[g] - base_m), w = exp2f(s - base_m);
                m[g] = top;
                l[g] = l[g] * keep + w;
#pragma unroll
                for (int e = 0; e < kChunk; ++e) o[g][e] = fmaf(w, v[e], o[g][e] * keep);
            }
        }
    }
    // join the lane groups and warps
    const int state = warp * kRows + sub;
    if (chunk == 0) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
            s_m[state][g] = m[g];
            s_l[state][g] = l[g];
        }
    }
    __syncthreads();
#pragma unroll
    for (int g = 0; g < G; ++g) {
        float top = __int_as_float(0xff800000);
        for (int x = 0; x < kStates; ++x) top = fmaxf(top, s_m[x][g]);
        const float base_m = top == __int_as_float(0xff800000) ? 0.f : top;
        const float w = exp2f(m[g] - base_m);
#pragma unroll
        for (int e = 0; e < kChunk; ++e) {
            float x = o[g][e] * w;
#pragma unroll
            for (int y = kLanes; y < 32; y <<= 1) x += __shfl_xor_sync(0xffffffffu, x, y);
            if (sub == 0) s_o[warp][g][chunk * kChunk + e] = x;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < G * D; i += kSimtWarps * 32) {
        const int g = i / D, d = i - g * D;
        float top = __int_as_float(0xff800000);
        for (int x = 0; x < kStates; ++x) top = fmaxf(top, s_m[x][g]);
        const float base_m = top == __int_as_float(0xff800000) ? 0.f : top;
        float sum = 0.f, acc = 0.f;
        for (int x = 0; x < kStates; ++x) sum += s_l[x][g] * exp2f(s_m[x][g] - base_m);
#pragma unroll
        for (int x = 0; x < kSimtWarps; ++x) acc += s_o[x][g][d];
        // nothing attended: a zero row (a NaN sum stays NaN)
        store_out(p, (row * p.num_q_heads + head0 + g) * D + d, sum == 0.f ? 0.f : acc / sum);
    }
}

template <typename T, int D>
int launch_simt(const SparseParams& p, cudaStream_t st) {
    const int group = p.num_q_heads / p.num_kv_heads;
    const int slices = group > 8 ? group / 8 : 1;
    const int64_t grid = p.num_rows * p.num_kv_heads * slices;
    if (grid > 0x7fffffff) return PA_ERR_UNSUPPORTED;
    const dim3 g((unsigned)grid), b(kSimtWarps * 32);
    switch (group / slices) {
        case 1: return launch_pdl(sparse_simt_kernel<T, D, 1>, g, b, 0, st, p, slices);
        case 2: return launch_pdl(sparse_simt_kernel<T, D, 2>, g, b, 0, st, p, slices);
        case 4: return launch_pdl(sparse_simt_kernel<T, D, 4>, g, b, 0, st, p, slices);
        case 8: return launch_pdl(sparse_simt_kernel<T, D, 8>, g, b, 0, st, p, slices);
    }
    return PA_ERR_UNSUPPORTED;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" int pa_paged_attention_decode_sparse(const void* q, const void* k_pool, const void* v_pool,
                                                const int32_t* block_tables, int max_blocks_per_seq,
                                                const int32_t* seq_ids, const int32_t* context_lens,
                                                const int32_t* selected, int max_selected, float scale,
                                                int block_size, void* out, int out_dtype, int64_t num_rows,
                                                int batch, int num_q_heads, int num_kv_heads, int head_dim,
                                                int64_t num_blocks, int kv_dtype, void* stream) {
    PA_NVTX_RANGE("pa_paged_attention_decode_sparse");
    if (num_rows < 0 || batch < 0 || max_blocks_per_seq < 0 || max_selected <= 0 || num_q_heads <= 0 ||
        num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || num_blocks < 0 || !valid_dtype(kv_dtype) ||
        !valid_dtype(out_dtype) || num_q_heads % num_kv_heads != 0)
        return PA_ERR_INVALID_ARG;
    if (!supported_head_dim(head_dim) || !supported_block_size(block_size) ||
        !supported_group(num_q_heads / num_kv_heads, kv_dtype))
        return PA_ERR_UNSUPPORTED;
    if (!seq_ids && num_rows > batch) return PA_ERR_INVALID_ARG;
    if (num_rows == 0) return PA_OK;
    if (!q || !k_pool || !v_pool || !block_tables || !context_lens || !selected || !out || !aligned16(q) ||
        !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(out))
        return PA_ERR_INVALID_ARG;
    SparseParams p = {};
    p.q = q;
    p.k_pool = k_pool;
    p.v_pool = v_pool;
    p.block_tables = block_tables;
    p.seq_ids = seq_ids;
    p.context_lens = context_lens;
    p.selected = selected;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.batch = batch;
    p.max_selected = max_selected;
    p.block_size = block_size;
    p.out = out;
    p.out_bf16 = out_dtype == PA_BF16;
    p.scale_log2 = scale * kLog2e;
    p.num_rows = num_rows;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.num_blocks = num_blocks;
    p.err = error_word_ptr();
    if (!p.err) return PA_ERR_CUDA;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (kv_dtype == PA_BF16)
        return head_dim == 128 ? launch_simt<__nv_bfloat16, 128>(p, st) : launch_simt<__nv_bfloat16, 64>(p, st);
    return head_dim == 128 ? launch_simt<float, 128>(p, st) : launch_simt<float, 64>(p, st);
}
