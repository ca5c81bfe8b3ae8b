// Attention of a batch's new tokens over their sequences in the paged cache.
//
// out = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m), s_j = scale * q . k_j,
// in one pass over the keys with the running maximum m and sum.  One warp per
// (token, query head): lane l holds elements l, l + 32, ... of q and of the
// output, and a key's score is a sum across the warp.
#include "kv_internal.cuh"
#include "ptx.cuh"

using namespace bitlin_impl;

namespace {

constexpr int kWarps = 8;

template <typename T, typename TO>
__global__ void __launch_bounds__(32 * kWarps) bitlin_attend_rows(const AttendParams p)
{
    ptx::griddep_wait();
    const int lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (row >= (long long)p.tokens * p.heads) return;
    const int t = (int)(row / p.heads), h = (int)(row - (long long)t * p.heads);
    const int seq = warp_sequence_of(p.batch, t);
    if (seq >= p.batch.seqs) return;
    int len = p.batch.kv_lens[seq];
    const long long held = (long long)p.batch.table_pages * p.page_size;
    if (len > held) {
        p.dev_error[kKvErrIndex] = 1;
        len = (int)held;
    }
    const int place = p.batch.kv_lens[seq] - (p.batch.q_offsets[seq + 1] - t);
    const int end = p.causal ? min(len, place + 1) : len;
    const int kh = h / (p.heads / p.kv_heads);

    const T* q = static_cast<const T*>(p.q) + t * p.q_token + h * p.q_head;
    float qv[8], acc[8], m = -INFINITY, sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        qv[i] = lane + 32 * i < p.dim ? to_f32(q[lane + 32 * i]) * p.scale : 0.f;
        acc[i] = 0.f;
    }
    for (int j = 0; j < end; ++j) {
        const int at = j / p.page_size;
        const int page = p.batch.table[seq * p.batch.table_stride + at];
        float kv[8], vv[8], s = 0.f;
        const bool in = page >= 0 && page < p.pages;
        if (!in) p.dev_error[kKvErrIndex] = 1;
        const long long base = page * p.page_stride + (j - at * p.page_size) * p.slot_stride + kh * p.head_stride;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool use = in && lane + 32 * i < p.dim;
            kv[i] = use ? to_f32(static_cast<const T*>(p.k_pool)[base + lane + 32 * i]) : 0.f;
            vv[i] = use ? to_f32(static_cast<const T*>(p.v_pool)[base + lane + 32 * i]) : 0.f;
            s += qv[i] * kv[i];
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        const float top = fmaxf(m, s), use = top == -INFINITY ? 0.f : top;
        const float keep = expf(m - use), w = expf(s - use);
        sum = sum * keep + w;
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = acc[i] * keep + w * vv[i];
        m = top;
    }
    TO* out = static_cast<TO*>(p.out) + t * p.out_token + h * p.out_head;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (lane + 32 * i < p.dim) out[lane + 32 * i] = from_f32<TO>(acc[i] * inv);
    if (p.lse && lane == 0) p.lse[row] = sum == 0.f ? -INFINITY : m + logf(sum);
}

template <typename T, typename TO>
cudaError_t launch(const AttendParams& p, cudaStream_t s)
{
    const long long rows = (long long)p.tokens * p.heads;
    bitlin_attend_rows<T, TO><<<(unsigned)((rows + kWarps - 1) / kWarps), 32 * kWarps, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t bitlin_launch_attend(const AttendParams& p, int dtype, int out_dtype, cudaStream_t s)
{
    if (dtype == BITLIN_BF16)
        return out_dtype == BITLIN_F32 ? launch<__nv_bfloat16, float>(p, s) : launch<__nv_bfloat16, __nv_bfloat16>(p, s);
    return out_dtype == BITLIN_F32 ? launch<__half, float>(p, s) : launch<__half, __half>(p, s);
}
