// Attention of a batch's new tokens over their sequences in a 4-bit cache.
//
// out = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m), s_j = scale * q . k_j, with
// k and v the values that the codes stand for (see quant.cuh).
//
// A block takes one query head of one token; its warps take keys in turn, each
// with a running maximum and sum, and are joined in shared memory.
#include <math.h>

#include "kv_internal.cuh"
#include "ptx.cuh"
#include "quant.cuh"

using namespace bitlin_impl;

namespace {

constexpr int kWarps = 4;

template <int D, typename T, typename TO>
__global__ void __launch_bounds__(32 * kWarps) bitlin_quant_attend(const QuantAttendParams p)
{
    constexpr int E = D / 32;  // elements of a lane
    __shared__ float sm[kWarps], sl[kWarps], so[kWarps][D];
    ptx::griddep_wait();
    const int t = blockIdx.x, h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int head = h / p.group;
    const int seq = warp_sequence_of(p.batch, t);
    if (seq >= p.batch.seqs) return;
    const int raw = min(max(p.batch.kv_lens[seq], 0), 1 << 30);
    const long long cap = (long long)p.batch.table_pages * p.pool.page_size;
    int len = raw < cap ? raw : (int)cap;
    if (len < raw) *p.index_error = 1;
    if (p.causal) len = min(len, max(raw - (p.batch.q_offsets[seq + 1] - t) + 1, 0));
    float q[E];
#pragma unroll
    for (int j = 0; j < E; ++j) q[j] = to_f32(static_cast<const T*>(p.q)[t * p.q_token + h * p.q_head + lane * E + j]);
    float m = -INFINITY, l = 0.f, o[E] = {};
    for (int key = warp; key < len; key += kWarps) {
        const int at = key / p.pool.page_size;
        const int page = p.batch.table[seq * p.batch.table_stride + at];
        const bool inside = page >= 0 && page < p.pool.pages;
        if (!inside) *p.index_error = 1;
        const long long slot = key - (long long)at * p.pool.page_size;
        float kv[2][E];
#pragma unroll
        for (int kind = 0; kind < 2; ++kind) {
            const uint8_t* codes = p.pool.codes[kind] + page * p.pool.page_stride + slot * p.pool.slot_stride + head * p.pool.head_stride;
            const uint8_t* scales = p.pool.scales[kind] + page * p.pool.scale_page + slot * p.pool.scale_slot + head * p.pool.scale_head;
            const float s = inside ? quant_scale(scales[lane / 8]) : 0.f;
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const int d = lane * E + j;
                kv[kind][j] = inside ? (float)((codes[d / 2] >> (4 * (d & 1)) & 15) - 8) * s : 0.f;
            }
        }
        float score = 0.f;
#pragma unroll
        for (int j = 0; j < E; ++j) score = fmaf(q[j], kv[0][j], score);
#pragma unroll
        for (int x = 16; x; x >>= 1) score += __shfl_xor_sync(0xffffffffu, score, x);
        score *= p.scale * 1.4426950408889634f;
        const float now = fmaxf(m, score), keep = m == -INFINITY ? 0.f : exp2f(m - now), w = exp2f(score - now);
        l = l * keep + w;
#pragma unroll
        for (int j = 0; j < E; ++j) o[j] = fmaf(w, kv[1][j], o[j] * keep);
        m = now;
    }
    if (lane == 0) {
        sm[warp] = m;
        sl[warp] = l;
    }
#pragma unroll
    for (int j = 0; j < E; ++j) so[warp][lane * E + j] = o[j];
    __syncthreads();
    float top = -INFINITY;
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm[w]);
    if (top == -INFINITY) top = 0.f;
    // (a sum of zero is that of no key; NaN scores leave the maximum alone and the sum NaN)
    auto part = [&](int w) { return sl[w] == 0.f ? 0.f : exp2f(sm[w] - top); };
    float total = 0.f;
    for (int w = 0; w < kWarps; ++w) total = fmaf(part(w), sl[w], total);
    for (int d = threadIdx.x; d < D; d += 32 * kWarps) {
        float x = 0.f;
        for (int w = 0; w < kWarps; ++w) x = fmaf(part(w), so[w][d], x);
        static_cast<TO*>(p.out)[t * p.out_token + h * p.out_head + d] = from_f32<TO>(total == 0.f ? 0.f : x / total);
    }
    if (p.lse && threadIdx.x == 0)
        p.lse[(long long)t * p.heads + h] = total == 0.f ? -INFINITY : 0.6931471805599453f * (top + log2f(total));
}

template <int D, typename T, typename TO>
cudaError_t launch(const QuantAttendParams& p, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.tokens, p.heads);
    cfg.blockDim = dim3(32 * kWarps);
    cfg.stream = s;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, bitlin_quant_attend<D, T, TO>, p);
}

template <typename T, typename TO>
cudaError_t pick(const QuantAttendParams& p, cudaStream_t s)
{
    return p.pool.dim == 64 ? launch<64, T, TO>(p, s) : p.pool.dim == 128 ? launch<128, T, TO>(p, s) : launch<256, T, TO>(p, s);
}

}  // namespace

KvWorkspaceParts bitlin_quant_attend_workspace(int, int)
{
    KvWorkspaceParts w = {};
    w.bytes = 256;
    return w;
}

cudaError_t bitlin_quant_attend_load(int, int) { return cudaSuccess; }

cudaError_t bitlin_launch_quant_attend(const QuantAttendParams& p, int dtype, int out_dtype, int, cudaStream_t s)
{
    if (dtype == BITLIN_BF16) return out_dtype == BITLIN_F32 ? pick<__nv_bfloat16, float>(p, s) : pick<__nv_bfloat16, __nv_bfloat16>(p, s);
    return out_dtype == BITLIN_F32 ? pick<__half, float>(p, s) : pick<__half, __half>(p, s);
}
