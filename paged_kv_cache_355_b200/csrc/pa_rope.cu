// pa_rope.cu -- the cache write of rotary models: per-head RMS norms of q and
// k, the rotation of positions, and the write of k and v into their pool slots
// in one pass over the projection's output.
//
// For each head row x (q and k; v is copied):
//   y = x * rsqrt(mean(x^2) + eps) * w                     (when w is given)
//   (y1, y2) -> (y1 c - y2 s, y2 c + y1 s)                 for each pair p of
// the first rotary_dim elements, with c = table[pos][p], s = table[pos][R/2+p].
// All of it in fp32 from one load to one rounding at the store.
//
// Bound by memory: each q row is read and written once, each k and v row read
// once and written once; the arithmetic is about ten operations an element.
// A row of D elements lies in D / 8 lanes (16 bytes each in bf16), so a warp
// takes 2 (D 128) or 4 (D 64) heads at a time and the norm's sum and the far
// half of a pair come by shuffles, without shared memory.  One warp stays with
// one token, so that token's angles are loaded once for all of the warp's
// heads.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "pa.h"
#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_rows.cuh"

namespace pa {
namespace {

constexpr int kRopeWarps = 4;
constexpr int kUnroll = 4;  // head rows a lane has in flight

struct RopeParams {
    const void *query, *key, *value;
    int64_t q_stride, k_stride, v_stride;  // elements between tokens
    void *query_out, *k_pool, *v_pool;
    // slots: given, or derived from the block tables (decode form)
    const int64_t* slot_mapping;
    const int32_t* block_tables;
    int max_blocks_per_seq;
    const int32_t* context_lens;
    int64_t* slots_out;
    // positions [num_axes][num_tokens], or NULL (decode: context_lens - 1)
    const int32_t* positions;
    int num_axes;
    const int32_t* pair_axes;
    const float* cos_sin;
    int64_t max_position;
    int rotary_dim;
    const void *q_weight, *k_weight;
    float eps;
    int64_t num_tokens;
    int num_q_heads, num_kv_heads, block_size;
    int64_t num_blocks;
    int rows_per_warp;  // head rows (q, k and v counted) of one warp, a multiple of 32 / (D / 8)
    int slices;         // warps of one token
    int* err;
};

// c and s of this lane's 8 elements, for the halves form one pair an element,
// for the neighbours form one pair every two.  `chunk` is the lane's chunk of
// the row; chunks at or past rotary_dim / 8 are not rotated.  Returns false
// where a position or an axis is out of range (nothing is read there).
template <bool INTERLEAVED>
__device__ __forceinline__ bool load_angles(const RopeParams& p, int64_t token, int64_t text_pos, int chunk,
                                            float (&c)[kChunk], float (&s)[kChunk]) {
    const int half = p.rotary_dim / 2;
    constexpr int kPairs = INTERLEAVED ? kChunk / 2 : kChunk;
    if (chunk * kChunk >= p.rotary_dim) return true;
    const int e = chunk * kChunk;
    const int first = INTERLEAVED ? e / 2 : (e < half ? e : e - half);
    float cc[kPairs], ss[kPairs];
    if (p.pair_axes == nullptr) {
        const int64_t pos = p.positions ? (int64_t)p.positions[token] : text_pos;
        if (pos < 0 || pos >= p.max_position) return false;
        const float* row = p.cos_sin + pos * p.rotary_dim + first;
#pragma unroll
        for (int i = 0; i < kPairs; i += 4) {
            const float4 a = *reinterpret_cast<const float4*>(row + i);
            const float4 b = *reinterpret_cast<const float4*>(row + half + i);
            cc[i] = a.x; cc[i + 1] = a.y; cc[i + 2] = a.z; cc[i + 3] = a.w;
            ss[i] = b.x; ss[i + 1] = b.y; ss[i + 2] = b.z; ss[i + 3] = b.w;
        }
    } else {
        bool ok = true;
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
            const int axis = p.pair_axes[first + i];
            int64_t pos = -1;
            if (axis >= 0 && axis < p.num_axes) pos = p.positions[(int64_t)axis * p.num_tokens + token];
            if (pos < 0 || pos >= p.max_position) {
                ok = false;
                continue;
            }
            const float* row = p.cos_sin + pos * p.rotary_dim + first + i;
            cc[i] = row[0];
            ss[i] = row[half];
        }
        if (!ok) return false;
    }
    // the second element of a pair takes +s, the first -s
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
        if (INTERLEAVED) {
            c[i] = cc[i / 2];
            s[i] = (i & 1) ? ss[i / 2] : -ss[i / 2];
        } else {
            c[i] = cc[i];
            s[i] = e < half ? -ss[i] : ss[i];
        }
    }
    return true;
}

template <typename T, int D, bool INTERLEAVED, bool DECODE>
__global__ void __launch_bounds__(kRopeWarps * 32) rope_cache_kernel(const RopeParams p) {
    constexpr int kLanes = D / kChunk;    // lanes of one head row
    constexpr int kHeads = 32 / kLanes;   // head rows of a warp at a time
    griddep_wait();
    griddep_launch_dependents();
    const int64_t unit = (int64_t)blockIdx.x * kRopeWarps + (threadIdx.x >> 5);
    const int64_t token = unit / p.slices;
    if (token >= p.num_tokens) return;  // whole warps
    const int slice = (int)(unit - token * p.slices);
    const int lane = threadIdx.x & 31;
    const int sub = lane / kLanes, chunk = lane % kLanes;

    // where the token goes
    int64_t slot = -1;
    int64_t text_pos = -1;
    bool bad = false;
    if (DECODE) {
        const int L = p.context_lens[token];
        if (L > 0) {
            text_pos = L - 1;
            const int64_t j = text_pos / p.block_size;
            int64_t blk = -1;
            if (j < p.max_blocks_per_seq) blk = p.block_tables[token * p.max_blocks_per_seq + j];
            if (blk >= 0 && blk < p.num_blocks) slot = blk * p.block_size + text_pos % p.block_size;
        }
        bad = L != 0 && slot < 0;
    } else {
        slot = p.slot_mapping[token];
        bad = slot >= p.num_blocks * p.block_size;
    }
    float c[kChunk], s[kChunk];
    if (slot >= 0 && !bad) bad = !load_angles<INTERLEAVED>(p, token, text_pos, chunk, c, s);
    bad = __any_sync(0xffffffffu, bad);
    const bool write = slot >= 0 && !bad;
    if (slice == 0 && lane == 0) {
        if (bad) record_error(p.err, PA_ERR_BAD_BLOCK_ID);
        if (p.slots_out) p.slots_out[token] = write ? slot : -1;
    }
    if (!write) return;  // the same for every lane

    const bool turned = chunk * kChunk < p.rotary_dim;
    const int shift = p.rotary_dim / (2 * kChunk);  // chunks between the halves of a pair
    const int partner = !turned ? lane : (chunk < shift ? lane + shift : lane - shift);
    const int64_t blk = slot / p.block_size;
    const int off = (int)(slot - blk * p.block_size);
    const int Hq = p.num_q_heads, Hkv = p.num_kv_heads;
    const int total = Hq + 2 * Hkv;
    const int row_end = min(total, (slice + 1) * p.rows_per_warp);

    float wq[kChunk], wk[kChunk];
    if (p.q_weight) {
        Chunk<T> w;
        w.load(static_cast<const T*>(p.q_weight) + chunk * kChunk);
        w.to_f32(wq);
    }
    if (p.k_weight) {
        Chunk<T> w;
        w.load(static_cast<const T*>(p.k_weight) + chunk * kChunk);
        w.to_f32(wk);
    }
    const T* q_row = static_cast<const T*>(p.query) + token * p.q_stride + chunk * kChunk;
    const T* k_row = static_cast<const T*>(p.key) + token * p.k_stride + chunk * kChunk;
    const T* v_row = static_cast<const T*>(p.value) + token * p.v_stride + chunk * kChunk;
    T* q_dst = static_cast<T*>(p.query_out) + token * Hq * D + chunk * kChunk;
    const int64_t pool_row = ((blk * Hkv) * p.block_size + off) * D + chunk * kChunk;  // kv head 0
    T* k_dst = static_cast<T*>(p.k_pool) + pool_row;
    T* v_dst = static_cast<T*>(p.v_pool) + pool_row;
    const int64_t head_stride = (int64_t)p.block_size * D;  // between kv heads in the pool

    for (int base = slice * p.rows_per_warp; base < row_end; base += kHeads * kUnroll) {
        Chunk<T> raw[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int r = base + u * kHeads + sub;
            if (r < row_end) {
                const T* src = r < Hq ? q_row + (int64_t)r * D
                                      : (r < Hq + Hkv ? k_row + (int64_t)(r - Hq) * D
                                                      : v_row + (int64_t)(r - Hq - Hkv) * D);
                raw[u].load(src);
            } else {
                raw[u] = Chunk<T>{};
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int r = base + u * kHeads + sub;
            if (base + u * kHeads >= row_end) break;  // the same for every lane
            if (base + u * kHeads < Hq + Hkv) {       // at least one q or k row
                float x[kChunk];
                raw[u].to_f32(x);
                const bool is_q = r < Hq;
                if (is_q ? p.q_weight != nullptr : p.k_weight != nullptr) {
                    float sum = 0.f;
#pragma unroll
                    for (int i = 0; i < kChunk; ++i) sum = fmaf(x[i], x[i], sum);
                    // rows of one warp may differ in whether they have a norm,
                    // the lanes of one row do not
                    const unsigned row_mask = (kLanes == 32 ? 0xffffffffu : ((1u << kLanes) - 1u) << (sub * kLanes));
#pragma unroll
                    for (int m = kLanes / 2; m; m >>= 1) sum += __shfl_xor_sync(row_mask, sum, m);
                    const float inv = rsqrtf(sum * (1.0f / D) + p.eps);
#pragma unroll
                    for (int i = 0; i < kChunk; ++i) x[i] = x[i] * inv * (is_q ? wq[i] : wk[i]);
                }
                float y[kChunk];
#pragma unroll
                for (int i = 0; i < kChunk; ++i)
                    y[i] = INTERLEAVED ? x[i ^ 1] : __shfl_sync(0xffffffffu, x[i], partner);
                if (r < Hq + Hkv) {
                    if (turned) {
#pragma unroll
                        for (int i = 0; i < kChunk; ++i) x[i] = fmaf(x[i], c[i], y[i] * s[i]);
                    }
                    raw[u].from_f32(x);
                }
            }
            if (r < row_end) {
                T* dst = r < Hq ? q_dst + (int64_t)r * D
                                : (r < Hq + Hkv ? k_dst + (r - Hq) * head_stride : v_dst + (r - Hq - Hkv) * head_stride);
                raw[u].store(dst);
            }
        }
    }
}

template <typename T, int D, bool DECODE>
int launch_rope(RopeParams p, bool interleaved, cudaStream_t stream) {
    constexpr int kHeads = 32 / (D / kChunk);
    const int total = p.num_q_heads + 2 * p.num_kv_heads;
    // head rows of one warp: as few as one step of the warp while the grid is
    // short of 32 warps an SM, as many as 4 unrolled steps once it is not
    const int64_t steps = ((int64_t)total + kHeads - 1) / kHeads;
    int64_t per_warp = steps * p.num_tokens / ((int64_t)num_sms() * 32);
    if (per_warp < 1) per_warp = 1;
    if (per_warp > 4 * kUnroll) per_warp = 4 * kUnroll;
    p.rows_per_warp = (int)per_warp * kHeads;
    p.slices = (total + p.rows_per_warp - 1) / p.rows_per_warp;
    const int64_t blocks = (p.num_tokens * p.slices + kRopeWarps - 1) / kRopeWarps;
    if (blocks > 0x7fffffff) return PA_ERR_UNSUPPORTED;
    auto kernel = interleaved ? rope_cache_kernel<T, D, true, DECODE> : rope_cache_kernel<T, D, false, DECODE>;
    return launch_pdl(kernel, dim3((unsigned)blocks), dim3(kRopeWarps * 32), 0, stream, p);
}

// Checks that both entry points share, then the launch.
template <bool DECODE>
int rope_and_cache(RopeParams p, int interleaved, int head_dim, int dtype, void* stream) {
    if (p.num_tokens < 0 || p.num_q_heads <= 0 || p.num_kv_heads <= 0 || head_dim <= 0 || p.block_size <= 0 ||
        p.num_blocks < 0 || p.num_axes <= 0 || p.max_position < 0 || !valid_dtype(dtype) ||
        (interleaved != 0 && interleaved != 1) || !(p.eps >= 0.f))
        return PA_ERR_INVALID_ARG;
    if (!supported_head_dim(head_dim) || !supported_block_size(p.block_size)) return PA_ERR_UNSUPPORTED;
    if (p.rotary_dim < 16 || p.rotary_dim > head_dim || p.rotary_dim % 16 != 0) return PA_ERR_UNSUPPORTED;
    if (p.num_tokens == 0) return PA_OK;
    if (!p.query || !p.key || !p.value || !p.query_out || !p.k_pool || !p.v_pool || !p.cos_sin || p.max_position == 0)
        return PA_ERR_INVALID_ARG;
    if (DECODE ? (!p.block_tables || !p.context_lens || p.max_blocks_per_seq < 0) : (!p.slot_mapping || !p.positions))
        return PA_ERR_INVALID_ARG;
    if (p.num_axes > 1 && (!p.pair_axes || !p.positions)) return PA_ERR_INVALID_ARG;
    if (p.pair_axes && !p.positions) return PA_ERR_INVALID_ARG;
    const void* const arrays[] = {p.query, p.key, p.value, p.query_out, p.k_pool, p.v_pool, p.cos_sin, p.q_weight,
                                  p.k_weight};
    for (const void* a : arrays)
        if (!aligned16(a)) return PA_ERR_INVALID_ARG;
    const int64_t vec = (int64_t)(16 / dtype_bytes(dtype));
    if (p.q_stride < (int64_t)p.num_q_heads * head_dim || p.k_stride < (int64_t)p.num_kv_heads * head_dim ||
        p.v_stride < (int64_t)p.num_kv_heads * head_dim || p.q_stride % vec || p.k_stride % vec || p.v_stride % vec)
        return PA_ERR_INVALID_ARG;
    p.err = error_word_ptr();
    if (!p.err) return PA_ERR_CUDA;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dtype == PA_BF16)
        return head_dim == 128 ? launch_rope<__nv_bfloat16, 128, DECODE>(p, interleaved, st)
                               : launch_rope<__nv_bfloat16, 64, DECODE>(p, interleaved, st);
    return head_dim == 128 ? launch_rope<float, 128, DECODE>(p, interleaved, st)
                           : launch_rope<float, 64, DECODE>(p, interleaved, st);
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" int pa_rope_and_cache(const void* query, const void* key, const void* value, int64_t query_stride,
                                 int64_t key_stride, int64_t value_stride, void* query_out, void* k_pool,
                                 void* v_pool, const int64_t* slot_mapping, const int32_t* positions, int num_axes,
                                 const int32_t* pair_axes, const float* cos_sin, int64_t max_position,
                                 int rotary_dim, int interleaved, const void* q_weight, const void* k_weight,
                                 float eps, int64_t num_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                                 int block_size, int64_t num_blocks, int dtype, void* stream) {
    PA_NVTX_RANGE("pa_rope_and_cache");
    RopeParams p = {};
    p.query = query; p.key = key; p.value = value;
    p.q_stride = query_stride; p.k_stride = key_stride; p.v_stride = value_stride;
    p.query_out = query_out; p.k_pool = k_pool; p.v_pool = v_pool;
    p.slot_mapping = slot_mapping;
    p.positions = positions; p.num_axes = num_axes; p.pair_axes = pair_axes;
    p.cos_sin = cos_sin; p.max_position = max_position; p.rotary_dim = rotary_dim;
    p.q_weight = q_weight; p.k_weight = k_weight; p.eps = eps;
    p.num_tokens = num_tokens; p.num_q_heads = num_q_heads; p.num_kv_heads = num_kv_heads;
    p.block_size = block_size; p.num_blocks = num_blocks;
    return rope_and_cache<false>(p, interleaved, head_dim, dtype, stream);
}

extern "C" int pa_rope_and_cache_decode(const void* query, const void* key, const void* value, int64_t query_stride,
                                        int64_t key_stride, int64_t value_stride, void* query_out, void* k_pool,
                                        void* v_pool, const int32_t* block_tables, int max_blocks_per_seq,
                                        const int32_t* context_lens, const int32_t* positions, int num_axes,
                                        const int32_t* pair_axes, const float* cos_sin, int64_t max_position,
                                        int rotary_dim, int interleaved, const void* q_weight, const void* k_weight,
                                        float eps, int batch, int num_q_heads, int num_kv_heads, int head_dim,
                                        int block_size, int64_t num_blocks, int dtype, int64_t* slot_mapping,
                                        void* stream) {
    PA_NVTX_RANGE("pa_rope_and_cache_decode");
    RopeParams p = {};
    p.query = query; p.key = key; p.value = value;
    p.q_stride = query_stride; p.k_stride = key_stride; p.v_stride = value_stride;
    p.query_out = query_out; p.k_pool = k_pool; p.v_pool = v_pool;
    p.block_tables = block_tables; p.max_blocks_per_seq = max_blocks_per_seq; p.context_lens = context_lens;
    p.slots_out = slot_mapping;
    p.positions = positions; p.num_axes = num_axes; p.pair_axes = pair_axes;
    p.cos_sin = cos_sin; p.max_position = max_position; p.rotary_dim = rotary_dim;
    p.q_weight = q_weight; p.k_weight = k_weight; p.eps = eps;
    p.num_tokens = batch; p.num_q_heads = num_q_heads; p.num_kv_heads = num_kv_heads;
    p.block_size = block_size; p.num_blocks = num_blocks;
    return rope_and_cache<true>(p, interleaved, head_dim, dtype, stream);
}
