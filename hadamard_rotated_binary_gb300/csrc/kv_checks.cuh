// Argument checks and parameter set-up shared by the attention side's C-ABI sources.
#pragma once

#include <math.h>

#include "kv_internal.cuh"

namespace bitlin_impl {

inline bitlin_status status_of(cudaError_t e)
{
    // what is reported here is not left for a later call to find
    if (e != cudaSuccess) cudaGetLastError();
    return e == cudaSuccess ? BITLIN_OK : e == cudaErrorMemoryAllocation ? BITLIN_ENOMEM : BITLIN_ECUDA;
}

template <typename Handle>
bitlin_status from_cuda(Handle h, cudaError_t e)
{
    if (e != cudaSuccess) h->last_cuda_error = (int)e;
    return status_of(e);
}

// The current device, when it is one this library runs on.
inline bitlin_status current_device(int* dev)
{
    int major = 0, minor = 0;
    if (cudaGetDevice(dev) != cudaSuccess) return BITLIN_EDEVICE;
    cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, *dev);
    cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, *dev);
    return major == 10 && minor == 3 ? BITLIN_OK : BITLIN_EDEVICE;
}

inline bool on_device(int device)
{
    int dev = -1;
    return cudaGetDevice(&dev) == cudaSuccess && dev == device;
}

inline int type_size(int dtype) { return dtype == BITLIN_F32 ? 4 : 2; }

// A call of no tokens may have no memory.
inline bool rows_ok(const bitlin_rows* r, int tokens)
{
    return r && (r->data || tokens == 0) && (r->dtype == BITLIN_F32 || r->dtype == BITLIN_BF16 || r->dtype == BITLIN_F16) &&
           reinterpret_cast<uintptr_t>(r->data) % type_size(r->dtype) == 0;
}

// Rows that are moved 16 bytes at a time (TMA, vector stores).
inline bool rows_wide(const bitlin_rows* r)
{
    return reinterpret_cast<uintptr_t>(r->data) % 16 == 0 && r->token_stride > 0 && r->head_stride > 0 &&
           r->token_stride % 8 == 0 && r->head_stride % 8 == 0 && r->token_stride < (1LL << 38) &&
           r->head_stride < (1LL << 38);
}

inline bool sizes_ok(int tokens, int heads, int dim)
{
    return tokens >= 0 && heads >= 1 && heads <= 4096 && (unsigned long long)tokens * (unsigned)dim < (1ULL << 32);
}

inline bool batch_ok(const bitlin_kv_batch* b)
{
    return b && b->seqs >= 1 && b->q_offsets && b->kv_lens && b->table && b->table_pages >= 1 &&
           (b->seqs == 1 || b->table_stride >= b->table_pages);
}

inline KvBatch batch_of(const bitlin_kv_batch* b) { return {b->q_offsets, b->kv_lens, b->table, b->table_stride, b->table_pages, b->seqs}; }

inline void set_source(TurnParams& p, int i, const bitlin_rows* r)
{
    p.src[i] = r->data;
    p.src_token[i] = r->token_stride;
    p.src_head[i] = r->head_stride;
}

inline void set_rope(TurnParams& p, bitlin_rope_t r, const int32_t* pos)
{
    p.turns = r ? r->turns : nullptr;
    p.rotary = r ? r->rotary : 0;
    p.axes = r ? r->axes : 0;
    p.adjacent = r ? r->adjacent : 0;
    p.pos = pos;
}

inline void set_out(TurnParams& p, const bitlin_rows* r)
{
    p.out = r->data;
    p.out_token = r->token_stride;
    p.out_head = r->head_stride;
}

constexpr int kNormMaxDim = 256;  // of a head with a norm

inline bool weight_ok(const float* w) { return w && reinterpret_cast<uintptr_t>(w) % alignof(float) == 0; }
// At most 1e38: added to the mean of two squares or more whose sum f32 holds, it stays in f32's range.
inline bool eps_ok(double eps) { return eps >= 0 && eps <= 1e38; }
inline bool norms_ok(const bitlin_head_norms* n)
{
    return !n || ((!n->q || weight_ok(n->q)) && (!n->k || weight_ok(n->k)) && eps_ok(n->eps));
}

inline void set_norms(NormTurnParams& p, const bitlin_head_norms* n)
{
    if (!n) return;
    p.weight[0] = n->q;
    p.weight[1] = n->k;
    p.eps = n->eps;
}

// The arguments of an append to a cache of `dim` wide heads whose q comes in `dtype`.
inline bool append_ok(const bitlin_kv_batch* batch, int tokens, const bitlin_rows* k, const bitlin_rows* v, const bitlin_rows* q,
                      int heads, const bitlin_rows* q_out, int dim, int dtype, bitlin_rope_t rope)
{
    if (!batch_ok(batch) || !rows_ok(k, tokens) || !rows_ok(v, tokens) || k->dtype != v->dtype) return false;
    if (!sizes_ok(tokens, q ? heads : 1, dim) || (rope && rope->rotary > dim)) return false;
    return !q || (rows_ok(q, tokens) && rows_ok(q_out, tokens) && q->dtype == k->dtype && q_out->dtype == dtype);
}

inline void set_append(TurnParams& p, const bitlin_kv_batch* batch, int tokens, bitlin_rope_t rope, const int32_t* pos,
                       const bitlin_rows* k, const bitlin_rows* v, const bitlin_rows* q, int heads, const bitlin_rows* q_out)
{
    if (q) {
        set_source(p, 0, q);
        set_out(p, q_out);
    }
    set_source(p, 1, k);
    set_source(p, 2, v);
    set_rope(p, rope, pos);
    p.batch = batch_of(batch);
    p.tokens = tokens;
    p.heads = q ? heads : 0;
    p.append = 1;
}

}  // namespace bitlin_impl
