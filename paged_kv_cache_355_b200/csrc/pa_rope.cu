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
// A row of D elements lies in D / 8 lanes, so a warp takes 2 (D 128) or 4 (D 64)
// heads at a time and the norm's sum comes by shuffles.  One warp stays with
// one token (or a slice of its heads), whose angles it gathers once into shared
// memory, and keeps the rows after the ones it works on in flight.  A lane
// holds 8 elements, both elements of four pairs: 8 neighbours, or 4 of each half
// of the rotated part.
// Measured on one B200: 24,175 prompt tokens of 64 / 8 heads of 128, bf16, both
// norms, three axes (995 MB): 156 us, 6.4 TB/s, 0.97 of a copy; 4,582 tokens of
// 32 / 32 heads, half rotated, neighbours (226 MB): 37.2 us, 6.1 TB/s; a decode
// step of 256 sequences, 32 / 8 heads (6.4 MB): 3.2 us, two dependent loads and
// the launch.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "pa.h"
#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_rows.cuh"

namespace pa {
namespace {


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
    int batch;    // steps loaded together, of q, of k or of v; a step is 32 / (D / 8) head rows
    int batches;  // of one warp
    int slices;   // warps of one token
    int* err;
};

// Steps loaded together: 16 registers.
template <typename T>
constexpr int kMostSteps = sizeof(T) == 2 ? 4 : 2;

// One warp is one CTA, so that all that depends on its token and step alone is
// the same for the whole CTA and stays off the lanes.
template <typename T, int D, bool NEIGHBOURS, bool WHOLE, bool DECODE>  // WHOLE: rotary_dim is D
__global__ void __launch_bounds__(32, 24) rope_cache_kernel(const RopeParams p) {
    constexpr int kLanes = D / kChunk;              // lanes of one head row
    constexpr int kHeads = 32 / kLanes;             // head rows of a step
    constexpr int kAhead = kMostSteps<T>;
    __shared__ __align__(16) float cs[2][D / 2];    // the token's cosines and sines
    griddep_wait();
    griddep_launch_dependents();
    const int64_t token = blockIdx.x / p.slices;
    const int slice = (int)(blockIdx.x - token * p.slices);
    const int lane = threadIdx.x;
    const int sub = lane / kLanes, x = lane % kLanes;
    // the lane's elements: 4 from `own` and 4 from own + other, of the two halves
    // of the rotated part or of what is past it, so that the lanes' accesses lie
    // side by side; 8 together where neighbours pair
    const bool turned = WHOLE || x * kChunk < p.rotary_dim;
    const int own = NEIGHBOURS ? x * 8 : turned ? x * 4 : p.rotary_dim / 2 + x * 4;
    const int other = NEIGHBOURS ? 4 : WHOLE ? D / 2 : turned ? p.rotary_dim / 2 : (D - p.rotary_dim) / 2;

    const int Hq = p.num_q_heads, Hkv = p.num_kv_heads;
    const int batch_heads = p.batch * kHeads;
    const int q_batches = (Hq + batch_heads - 1) / batch_heads, kv_batches = (Hkv + batch_heads - 1) / batch_heads;
    const int v_first = q_batches + kv_batches;
    const int first = slice * p.batches, end = min(first + p.batches, v_first + kv_batches);
    const T* q_src = static_cast<const T*>(p.query) + token * p.q_stride;
    const T* k_src = static_cast<const T*>(p.key) + token * p.k_stride;
    const T* v_src = static_cast<const T*>(p.value) + token * p.v_stride;
    const int src_lane = sub * D + own;
    Chunk<T> rows[kAhead];
    auto load = [&](Chunk<T>(&to)[kAhead], int b) {
        const bool is_q = b < q_batches, is_v = b >= v_first;
        const int head = (is_q ? b : is_v ? b - v_first : b - q_batches) * batch_heads;
        const int limit = min(is_q ? Hq : Hkv, head + batch_heads) - sub;
        const T* src = (is_q ? q_src : is_v ? v_src : k_src) + (int64_t)head * D + src_lane;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            to[u] = Chunk<T>{};
            if (head + u * kHeads < limit) {
                if (NEIGHBOURS)
                    to[u].load(src + u * kHeads * D);
                else
                    to[u].load(src + u * kHeads * D, src + u * kHeads * D + other);
            }
        }
    };
    load(rows, first);  // beside the look-up of where they go

    // where the token goes: looked up here, looked at after the angles, so that
    // the two chains of loads run side by side
    const int shift = block_shift(p.block_size);
    int64_t text_pos = -1, place;  // the slot, or the block table's entry
    if (DECODE) {
        text_pos = (int64_t)p.context_lens[token] - 1;
        const int64_t j = text_pos >> shift;
        place = text_pos >= 0 && j < p.max_blocks_per_seq ? p.block_tables[token * p.max_blocks_per_seq + j] : -1;
    } else {
        place = p.slot_mapping[token];
    }
    // the token's angles, a pair or two a lane; a bad position or axis reads nothing
    const int half = p.rotary_dim / 2;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < D / 2; i += 32) {
        const int pair = i + lane;
        if (pair >= half) break;
        const int axis = p.pair_axes ? p.pair_axes[pair] : 0;
        int64_t pos = text_pos;
        if (p.positions) pos = axis >= 0 && axis < p.num_axes ? (int64_t)p.positions[(int64_t)axis * p.num_tokens + token] : -1;
        if (pos >= 0 && pos < p.max_position) {
            cs[0][pair] = p.cos_sin[pos * p.rotary_dim + pair];
            cs[1][pair] = p.cos_sin[pos * p.rotary_dim + half + pair];
        } else {
            bad = true;
        }
    }
    int64_t slot = -1;
    if (DECODE) {
        if (place >= 0 && place < p.num_blocks) slot = (place << shift) + (text_pos & (p.block_size - 1));
        bad = text_pos != -1 && (bad || slot < 0);  // a length of 0 is an empty sequence
    } else {
        slot = place;
        bad = slot >= 0 && (bad || slot >= p.num_blocks << shift);  // a negative slot is padding
    }
    bad = __any_sync(0xffffffffu, bad);
    const bool write = slot >= 0 && !bad;
    if (slice == 0 && lane == 0) {
        if (bad) record_error(p.err, PA_ERR_BAD_BLOCK_ID);
        if (p.slots_out) p.slots_out[token] = write ? slot : -1;
    }
    if (!write) return;  // the same for every lane
    __syncwarp();        // the angles are in

    // coefficients of the lane's four pairs, weights multiplied in:
    // (y1, y2) -> (y1 f[0] - y2 f[1], y2 f[2] + y1 f[3])
    float f[4][4];
    auto coefficients = [&](const void* weight) {
        float w[kChunk];
        if (weight) {
            Chunk<T> c;
            c.load(static_cast<const T*>(weight) + own, static_cast<const T*>(weight) + own + other);
            c.to_f32(w);
        } else {
#pragma unroll
            for (int i = 0; i < kChunk; ++i) w[i] = 1.f;
        }
        const float4 a = turned ? *reinterpret_cast<const float4*>(&cs[0][x * 4]) : make_float4(1.f, 1.f, 1.f, 1.f);
        const float4 b = turned ? *reinterpret_cast<const float4*>(&cs[1][x * 4]) : make_float4(0.f, 0.f, 0.f, 0.f);
        const float c[4] = {a.x, a.y, a.z, a.w}, s[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float w1 = w[NEIGHBOURS ? 2 * i : i], w2 = w[NEIGHBOURS ? 2 * i + 1 : i + 4];
            f[0][i] = w1 * c[i];
            f[1][i] = w2 * s[i];
            f[2][i] = w2 * c[i];
            f[3][i] = w1 * s[i];
        }
    };
    const int64_t blk = slot >> shift;
    const int off = (int)slot & (p.block_size - 1);
    T* q_dst = static_cast<T*>(p.query_out) + token * Hq * D;
    const int64_t pool_row = ((blk * Hkv) * p.block_size + off) * D;  // kv head 0
    T* k_dst = static_cast<T*>(p.k_pool) + pool_row;
    T* v_dst = static_cast<T*>(p.v_pool) + pool_row;
    const int64_t head_stride = (int64_t)p.block_size * D;  // between kv heads in the pool
    const int64_t pool_lane = sub * head_stride + own;

    for (int b = first; b < end; ++b) {
        Chunk<T> next[kAhead];
        if (b + 1 < end) load(next, b + 1);
        const bool is_q = b < q_batches, is_v = b >= v_first;
        const int head = (is_q ? b : is_v ? b - v_first : b - q_batches) * batch_heads;
        const int limit = min(is_q ? Hq : Hkv, head + batch_heads);
        const void* weight = is_q ? p.q_weight : p.k_weight;
        if (b == first || b == q_batches) coefficients(weight);
        T* dst = is_q ? q_dst + (int64_t)head * D + src_lane : (is_v ? v_dst : k_dst) + head * head_stride + pool_lane;
        const int64_t dst_step = is_q ? kHeads * D : kHeads * head_stride;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (head + u * kHeads >= limit) break;  // the same for every lane
            if (!is_v) {
                float y[kChunk];
                rows[u].to_f32(y);
                if (weight) {
                    float sum = 0.f;
#pragma unroll
                    for (int i = 0; i < kChunk; ++i) sum = fmaf(y[i], y[i], sum);
#pragma unroll
                    for (int m = kLanes / 2; m; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
                    const float inv = rsqrtf(sum * (1.0f / D) + p.eps);
#pragma unroll
                    for (int i = 0; i < kChunk; ++i) y[i] *= inv;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int a = NEIGHBOURS ? 2 * i : i, b = NEIGHBOURS ? 2 * i + 1 : i + 4;
                    const float y1 = y[a], y2 = y[b];
                    if (turned) {
                        y[a] = fmaf(y1, f[0][i], -(y2 * f[1][i]));
                        y[b] = fmaf(y2, f[2][i], y1 * f[3][i]);
                    } else {  // not by a sine of 0: the other element may be infinite
                        y[a] = y1 * f[0][i];
                        y[b] = y2 * f[2][i];
                    }
                }
                rows[u].from_f32(y);
            }
            if (head + u * kHeads + sub < limit) {
                if (NEIGHBOURS)
                    rows[u].store(dst);
                else
                    rows[u].store(dst, dst + other);
            }
            dst += dst_step;
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) rows[u] = next[u];
    }
}

template <typename T, int D, bool DECODE>
int launch_rope(RopeParams p, bool interleaved, cudaStream_t stream) {
    constexpr int kHeads = 32 / (D / kChunk);
    const int64_t steps = (p.num_q_heads + kHeads - 1) / kHeads + 2 * ((p.num_kv_heads + kHeads - 1) / kHeads);
    // Steps of one warp.  A token's look-ups are paid once a warp, so few tokens
    // share out their heads (4 tokens of 12 heads: 1.85 us with one step a warp,
    // 2.1 with all three), but not beyond one load of several steps where that
    // fills the SMs (256 tokens of 24 steps: 6.7 us with one, 3.2 with four);
    // many take a whole token a warp (24k tokens of 40 steps: 169 us with 16
    // steps, 156 with 40) as long as that leaves 64 warps an SM to even out
    // (4.6k tokens of 48 steps: 37.2 us with the 16 that this gives, 40.8 with 48).
    const int64_t all = steps * p.num_tokens, sms = num_sms();
    int64_t per_warp = all / (sms * 64);
    if (per_warp < 4 && all >= sms * 32) per_warp = 4;
    if (per_warp < 16 && p.num_tokens * ((steps + 15) / 16) >= sms * 28) per_warp = 16;
    per_warp = std::max((int64_t)1, std::min(per_warp, steps));
    p.batch = (int)std::min(per_warp, (int64_t)kMostSteps<T>);
    const int batch_heads = p.batch * kHeads;
    const int64_t batches = (p.num_q_heads + batch_heads - 1) / batch_heads + 2 * ((p.num_kv_heads + batch_heads - 1) / batch_heads);
    p.slices = (int)((batches * p.batch + per_warp - 1) / per_warp);
    p.batches = (int)((batches + p.slices - 1) / p.slices);  // evened out
    p.slices = (int)((batches + p.batches - 1) / p.batches);
    const int64_t blocks = p.num_tokens * p.slices;
    if (blocks > 0x7fffffff) return PA_ERR_UNSUPPORTED;
    const bool whole = p.rotary_dim == D;
    auto kernel = interleaved ? (whole ? rope_cache_kernel<T, D, true, true, DECODE> : rope_cache_kernel<T, D, true, false, DECODE>)
                              : (whole ? rope_cache_kernel<T, D, false, true, DECODE> : rope_cache_kernel<T, D, false, false, DECODE>);
    return launch_pdl(kernel, dim3((unsigned)blocks), dim3(32), 0, stream, p);
}

// Checks that both entry points share, then the launch.
template <bool DECODE>
int rope_and_cache(RopeParams p, int interleaved, int head_dim, int dtype, void* stream) {
    if (p.num_tokens < 0 || p.num_q_heads <= 0 || p.num_kv_heads <= 0 || head_dim <= 0 || p.block_size <= 0 ||
        p.num_blocks < 0 || p.num_axes <= 0 || p.max_position < 0 || !valid_dtype(dtype) ||
        (interleaved != 0 && interleaved != 1) || !(p.eps >= 0.f))
        return PA_ERR_INVALID_ARG;
    if (!supported_head_dim(head_dim) || !supported_block_size(p.block_size) || p.num_tokens > 0x7fffffff)
        return PA_ERR_UNSUPPORTED;
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
