// Declarations shared by the rotary, paged-cache and attention sources (not part of the C-ABI).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <memory>

#include "bitlin_internal.cuh"

namespace bitlin_impl {

// A frequency as a fixed-point fraction of a turn per position, 2^-64 turns,
// so that position * frequency modulo one turn is an exact wrapping product.
// The pair's axis lies in the low bits, which leaves the frequency to 2^-62
// turns: 2^-31 of a turn at the largest position.
using Turn = uint64_t;
constexpr int kAxisBits = 3;
constexpr Turn kAxisMask = (1u << kAxisBits) - 1;

struct KvBatch {
    const int32_t* q_offsets;  // [seqs + 1]
    const int32_t* kv_lens;    // [seqs]
    const int32_t* table;      // [seqs] rows of table_pages entries
    long long table_stride;
    int table_pages;
    int seqs;
};

// One call of the rotation kernel: rows of q to `out`, and for an append the
// rows of k (rotated) and v (copied) to the pools.
struct TurnParams {
    const void* src[3];       // q, k, v
    long long src_token[3], src_head[3];
    void* out;                // q's destination
    long long out_token, out_head;
    void* pool[2];            // k, v
    long long page_stride, slot_stride, head_stride;
    KvBatch batch;
    const Turn* turns;        // [rotary / 2], nullptr: no rotation
    int axes;
    const int32_t* pos;       // [axes][tokens], nullptr: the token's place
    int* index_error;         // set: a place outside the table or a page outside the pool
    int pages, page_size;
    int tokens, heads, kv_heads, dim, rotary;
    int adjacent, inverse;
    int append;               // 0: q alone
    int units;                // threads per row, set by the launcher
    int q_groups, kv_groups;  // blocks along y: q, k, v, set by the launcher
};

// Index of the sequence that owns token row `t` (t < q_offsets[seqs]), found
// by the whole warp: each round every lane probes one boundary of the range,
// so up to 32 sequences take one round and up to 1024 two.  Returns the
// largest s with q_offsets[s] <= t, or seqs when t is past the last row.
__device__ __forceinline__ int warp_sequence_of(const KvBatch& b, int t)
{
    const int lane = threadIdx.x & 31;
    int lo = 0, n = b.seqs + 1;  // the answer lies in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 31) >> 5;
        const int i = lo + lane * step;
        const bool le = lane * step < n && b.q_offsets[i] <= t;
        const unsigned votes = __ballot_sync(0xffffffffu, le);
        const int last = votes ? 31 - __clz(votes) : 0;
        const int end = lo + n;
        lo += last * step;
        n = min(step, end - lo);
    }
    return lo;
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// A call of the rotation kernel with a norm of each head before it, and the
// append to a cache in 4 bits (t.pool then holds codes, strides in bytes).
struct NormTurnParams {
    TurnParams t;
    const float* weight[2];   // q's, k's; nullptr: no norm
    double eps;
    uint8_t* scales[2];       // k's, v's (4-bit cache)
    long long scale_page, scale_slot, scale_head;
    // set by the launcher
    int team;                 // lanes to a row
    int kv_heads_per_team;    // heads of k (or v) that a team takes one after the other
    float inverse_dim, eps_f;
};

// The gradient of a norm and rotation (dx in x's type).
struct NormGradParams {
    const void *dy, *x;
    void* dx;
    long long dy_token, dy_head, x_token, x_head, dx_token, dx_head;
    const float* weight;
    double eps;
    const Turn* turns;
    const int32_t* pos;
    float* partial;           // [blocks][dim]
    float* dweight;           // [dim]
    int tokens, heads, dim, rotary, axes, adjacent;
    // set by the launcher
    int team, blocks;
    float inverse_dim, eps_f;
};

// One call of the attention kernel.
struct AttendParams {
    const void* v_pool;        // for the rare values that are put back (see attend.cu)
    long long page_stride, slot_stride, head_stride;
    KvBatch batch;
    void* out;
    long long out_token, out_head;
    float* lse;                // [tokens][heads] or nullptr
    float* ws_o;               // [2 * CTAs][128][padded dim]: unnormalised parts of outputs
    float* ws_ml;              // [2 * CTAs][128][2]: their rows' log2 maxima and sums
    int* tickets;              // [CTAs], zero between calls
    int* timed_out;            // set: a bounded wait gave up, and the tickets may not be zero
    int* index_error;
    long long wait_budget_ns;
    int pages, page_size, page_shift;  // page_shift: log2 of a power of two, else -1
    int tokens, heads, kv_heads, group, dim, causal;
    int tile_tokens, q_box;    // tokens of a 128-row tile, and of one copy of its queries
    int few;                   // tiles of up to 8 rows, the weights' digits in lanes of their own
    int item_extra;            // key tiles that an item's begin and end cost
    int box_k, box_v;          // slots of a page per TMA copy
    int stall_test;
    float scale;
};

// A paged cache in 4 bits (strides in bytes).
struct QuantPools {
    const uint8_t* codes[2];   // k, v
    const uint8_t* scales[2];
    long long page_stride, slot_stride, head_stride;
    long long scale_page, scale_slot, scale_head;
    int pages, page_size, kv_heads, dim;
};

// Rows of the batch's new tokens read back from it.
struct QuantReadParams {
    QuantPools pool;
    KvBatch batch;
    void* out[2];
    long long out_token[2], out_head[2];
    int* index_error;
    int tokens;
};

// The batch's pages as 16-bit ones.
struct QuantUnpackParams {
    QuantPools pool;
    KvBatch batch;
    void* out[2];
    long long page_stride, slot_stride, head_stride;
    int* index_error;
};

// Attention over it.
struct QuantAttendParams {
    QuantPools pool;
    KvBatch batch;
    const void* q;
    long long q_token, q_head;
    void* out;
    long long out_token, out_head;
    float* lse;
    float* ws_o;
    float* ws_ml;
    int* tickets;
    int* index_error;
    int tokens, heads, group, causal;
    int bf16;                  // the type of q and of a 16-bit output
    uint32_t magic;            // two float16 1024s (see quant.cuh)
    int group_inverse;         // 2^16 / group, rounded up: divides numbers below 256
    // the pools' strides in units of the largest power of two that divides them
    uint32_t unit, page_units, slot_units, head_units;
    uint32_t scale_unit, scale_page_units, scale_slot_units, scale_head_units;
    int page_shift;            // log2 of a page size that is a power of two, else -1
    float scale;
};

// Attention's workspace.  Nothing in it outlives a call but zero tickets, so
// handles whose calls run one after the other can share one.
struct KvWorkspace {
    unsigned char* data = nullptr;  // tickets, timed_out; then maxima and sums; then outputs
    size_t bytes = 0;
    KvWorkspace() = default;
    KvWorkspace(const KvWorkspace&) = delete;
    ~KvWorkspace() { cudaFree(data); }
};

struct KvWorkspaceParts {
    size_t timed_out, ml, o, bytes;  // the tickets lie at 0
};

}  // namespace bitlin_impl

struct bitlin_rope {
    int device = 0;
    int rotary = 0, axes = 0, adjacent = 0;
    bitlin_impl::Turn* turns = nullptr;
    int last_cuda_error = 0;
};

struct bitlin_kv {
    int device = 0;
    int num_sms = 0;
    void* k = nullptr;
    void* v = nullptr;
    int pages = 0, page_size = 0, kv_heads = 0, dim = 0, dtype = 0;
    long long page_stride = 0, slot_stride = 0, head_stride = 0;
    int last_cuda_error = 0;
    bitlin_status sticky = BITLIN_OK;
    int* index_error = nullptr;
    long long wait_budget_ns = 0;
    int stall_test = 0;
    alignas(64) unsigned char tmap_k[128];  // TMA descriptors of the pools (CUtensorMaps)
    alignas(64) unsigned char tmap_v[128];
    std::shared_ptr<bitlin_impl::KvWorkspace> workspace;
};

struct bitlin_kvq {
    int device = 0;
    int num_sms = 0;
    int dtype = 0;
    bitlin_impl::QuantPools pool = {};
    uint32_t unit = 0, scale_unit = 0;  // powers of two that divide the pools' strides
    int last_cuda_error = 0;
    int* index_error = nullptr;
    std::shared_ptr<bitlin_impl::KvWorkspace> workspace;
    // of the 16-bit cache that the last call went through, and whether a wait of such a call ran out
    std::weak_ptr<bitlin_impl::KvWorkspace> through;
    bool through_timed_out = false;
};

// bitlin_kv_attend whose pages outside the pool are reported to `index_error`.
bitlin_status bitlin_kv_attend_reporting(bitlin_kv_t kv, const bitlin_kv_batch* batch, int tokens, const bitlin_rows* q, int heads,
                                         float scale, int causal, const bitlin_rows* out, float* lse, int* index_error,
                                         bitlin_stream_t stream);
// Whether a bounded wait of a 16-bit cache's calls ran out in this workspace (the calls are through).
cudaError_t bitlin_kv_timed_out(const bitlin_impl::KvWorkspace& w, int num_sms, int* timed_out);

// Launchers (return a cudaError_t).
cudaError_t bitlin_launch_norm_turn(const bitlin_impl::NormTurnParams& p, int src_dtype, int dst_dtype, bool quant, cudaStream_t s);
int bitlin_norm_grad_blocks(int tokens, int heads);
cudaError_t bitlin_launch_norm_grad(const bitlin_impl::NormGradParams& p, int dy_dtype, int x_dtype, cudaStream_t s);
cudaError_t bitlin_launch_quant_read(const bitlin_impl::QuantReadParams& p, int dst_dtype, cudaStream_t s);
cudaError_t bitlin_launch_quant_unpack(const bitlin_impl::QuantUnpackParams& p, int dst_dtype, int num_sms, cudaStream_t s);
cudaError_t bitlin_launch_quant_attend(const bitlin_impl::QuantAttendParams& p, int out_dtype, int num_sms, cudaStream_t s);
cudaError_t bitlin_quant_attend_load(int dim);
bitlin_impl::KvWorkspaceParts bitlin_quant_attend_workspace(int num_sms);
cudaError_t bitlin_launch_turn(const bitlin_impl::TurnParams& p, int src_dtype, int dst_dtype, cudaStream_t s);
cudaError_t bitlin_launch_attend(const bitlin_impl::AttendParams& p, int dtype, int out_dtype, const void* tmap_q,
                                 const void* tmap_k, const void* tmap_v, int num_sms, cudaStream_t s);
// Tokens of a row tile, and of one TMA copy of its queries; whether its rows are few.
void bitlin_attend_rows(int tokens, int seqs, int group, int out_dtype, int* tile_tokens, int* q_box, int* few_rows);
// What an item of attention's work costs beside its key tiles, in key tiles.
int bitlin_attend_item_extra(int dim);
// Slots per TMA copy of the key and value pools.
void bitlin_attend_boxes(int dim, int page_size, int* box_k, int* box_v);
// The attention workspace's parts.
bitlin_impl::KvWorkspaceParts bitlin_attend_workspace(int dim, int num_sms);
// Load a cache's attention kernels and set their shared memory, so that no call has to.
cudaError_t bitlin_attend_load(int dim, int dtype);
