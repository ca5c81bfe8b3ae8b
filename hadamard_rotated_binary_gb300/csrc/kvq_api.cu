// C-ABI of the cache in 4 bits: handles, append, reading back, attention.
#include <cuda_runtime.h>

#include <memory>
#include <new>

#include "kv_checks.cuh"
#include "kv_internal.cuh"

using namespace bitlin_impl;

namespace {

// Rows (new tokens times query heads of a key head) that a sequence brings on average, from
// which on it pays to read its pages back to 16 bits first.  Measured, in us, 8 sequences of
// 2,000-6,000 keys, directly and through 16-bit pages: 128 dims, 64 rows 60 and 74, 128 rows
// 105 and 77; 256 dims, 72 rows 67 and 80, 144 rows 111 and 91; 64 dims, 64 rows 42 and 50,
// 128 rows 69 and 51.  An f32 output goes through them only where the caller says so: it is
// up to 3e-6 off there, 2.4 (f16) and 12 (bf16) times as far as f32 arithmetic, and closer than
// that directly.  The price of that: 344 us for 141 (24-72 tokens a sequence on 210-1,050 keys, 24 heads of
// 256), 9.2 ms for 1.6 (2,048 tokens over 32,768 keys); few key heads over long contexts gain
// (82 us to 30).
constexpr long long kThroughRows = 80;

// The largest power of two that divides three strides.
uint32_t unit_of(long long page, long long slot, long long head)
{
    const long long all = page | slot | head;
    const long long low = all & -all;
    return low < (1 << 30) ? (uint32_t)low : 1u << 30;
}

// Whether every slot lies less than 2^32 units from the first.
bool reaches(const bitlin_kvq_pools* p, uint32_t unit, long long page, long long slot, long long head)
{
    const __int128 last = (__int128)(p->pages - 1) * page + (__int128)(p->page_size - 1) * slot + (__int128)(p->kv_heads - 1) * head;
    return last / unit < ((__int128)1 << 32);
}

bool pool_ok(const bitlin_kvq_pools* p)
{
    if (!p) return false;
    for (const void* x : {p->k, p->v})
        if (!x || reinterpret_cast<uintptr_t>(x) % 16) return false;
    for (const void* x : {p->k_scale, p->v_scale})
        if (!x || reinterpret_cast<uintptr_t>(x) % 4) return false;
    if (p->pages < 1 || p->page_size < 1 || p->page_size > 65536 || p->kv_heads < 1 || p->kv_heads > 4096) return false;
    if (p->head_dim != 64 && p->head_dim != 128 && p->head_dim != 256) return false;
    for (long long stride : {p->page_stride, p->slot_stride, p->head_stride})
        if (stride < 16 || stride % 16 || stride >= (1LL << 39)) return false;
    for (long long stride : {p->scale_page_stride, p->scale_slot_stride, p->scale_head_stride})
        if (stride < 4 || stride % 4 || stride >= (1LL << 39)) return false;
    return reaches(p, unit_of(p->page_stride, p->slot_stride, p->head_stride), p->page_stride, p->slot_stride, p->head_stride) &&
           reaches(p, unit_of(p->scale_page_stride, p->scale_slot_stride, p->scale_head_stride), p->scale_page_stride, p->scale_slot_stride,
                   p->scale_head_stride);
}

QuantPools pools_of(const bitlin_kvq_pools* p)
{
    QuantPools q = {};
    q.codes[0] = static_cast<uint8_t*>(p->k);
    q.codes[1] = static_cast<uint8_t*>(p->v);
    q.scales[0] = static_cast<uint8_t*>(p->k_scale);
    q.scales[1] = static_cast<uint8_t*>(p->v_scale);
    q.page_stride = p->page_stride;
    q.slot_stride = p->slot_stride;
    q.head_stride = p->head_stride;
    q.scale_page = p->scale_page_stride;
    q.scale_slot = p->scale_slot_stride;
    q.scale_head = p->scale_head_stride;
    q.pages = p->pages;
    q.page_size = p->page_size;
    q.kv_heads = p->kv_heads;
    q.dim = p->head_dim;
    return q;
}

// A workspace for the handle's calls, with zero tickets.
cudaError_t new_workspace(bitlin_kvq& h)
{
    const KvWorkspaceParts parts = bitlin_quant_attend_workspace(h.num_sms);
    std::shared_ptr<KvWorkspace> w;
    try {
        w = std::make_shared<KvWorkspace>();
    } catch (const std::bad_alloc&) {
        return cudaErrorMemoryAllocation;
    }
    cudaError_t e = cudaMalloc(&w->data, parts.bytes);
    if (e == cudaSuccess) e = cudaMemset(w->data, 0, parts.ml);
    if (e != cudaSuccess) return e;
    w->bytes = parts.bytes;
    h.workspace = std::move(w);
    return cudaSuccess;
}

// Whether `through` has room for every page of the cache.
bool passes(const bitlin_kvq& h, const bitlin_kv* through)
{
    return through->device == h.device && through->dtype == h.dtype && through->pages == h.pool.pages &&
           through->page_size == h.pool.page_size && through->kv_heads == h.pool.kv_heads && through->dim == h.pool.dim;
}

}  // namespace

extern "C" {

bitlin_status bitlin_kvq_create(bitlin_kvq_t* out, const bitlin_kvq_pools* pools, int dtype)
{
    if (!out) return BITLIN_EINVAL;
    *out = nullptr;
    if (!pool_ok(pools) || (dtype != BITLIN_BF16 && dtype != BITLIN_F16)) return BITLIN_EINVAL;
    int dev = 0;
    bitlin_status st = current_device(&dev);
    if (st != BITLIN_OK) return st;
    std::unique_ptr<bitlin_kvq> h(new (std::nothrow) bitlin_kvq());
    if (!h) return BITLIN_ENOMEM;
    h->device = dev;
    h->dtype = dtype;
    h->pool = pools_of(pools);
    h->unit = unit_of(pools->page_stride, pools->slot_stride, pools->head_stride);
    h->scale_unit = unit_of(pools->scale_page_stride, pools->scale_slot_stride, pools->scale_head_stride);
    cudaError_t e = cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = bitlin_quant_attend_load(h->pool.dim);
    if (e == cudaSuccess) e = cudaMalloc(&h->index_error, sizeof(int));
    if (e == cudaSuccess) e = cudaMemset(h->index_error, 0, sizeof(int));
    if (e == cudaSuccess) e = new_workspace(*h);
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e != cudaSuccess) {
        cudaFree(h->index_error);
        return status_of(e);
    }
    *out = h.release();
    return BITLIN_OK;
}

bitlin_status bitlin_kvq_share(bitlin_kvq_t kvq, bitlin_kvq_t with)
{
    if (!kvq || !with || kvq->device != with->device) return BITLIN_EINVAL;
    // the handle's own workspace may be freed here: not under its calls
    const cudaError_t e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return from_cuda(kvq, e);
    kvq->workspace = with->workspace;
    return BITLIN_OK;
}

bitlin_status bitlin_kvq_append(bitlin_kvq_t kvq, const bitlin_kv_batch* batch, int tokens, bitlin_rope_t rope,
                                const int32_t* pos, const bitlin_rows* k, const bitlin_rows* v,
                                const bitlin_rows* q, int heads, const bitlin_rows* q_out,
                                const bitlin_head_norms* norms, bitlin_stream_t stream)
{
    if (!kvq || !append_ok(batch, tokens, k, v, q, heads, q_out, kvq->pool.dim, kvq->dtype, rope) || !norms_ok(norms)) return BITLIN_EINVAL;
    if (!on_device(kvq->device) || (rope && rope->device != kvq->device)) return BITLIN_EINVAL;
    if (tokens == 0) return BITLIN_OK;
    NormTurnParams n = {};
    TurnParams& p = n.t;
    set_append(p, batch, tokens, rope, pos, k, v, q, heads, q_out);
    for (int i = 0; i < 2; ++i) {
        p.pool[i] = const_cast<uint8_t*>(kvq->pool.codes[i]);
        n.scales[i] = const_cast<uint8_t*>(kvq->pool.scales[i]);
    }
    p.page_stride = kvq->pool.page_stride;
    p.slot_stride = kvq->pool.slot_stride;
    p.head_stride = kvq->pool.head_stride;
    n.scale_page = kvq->pool.scale_page;
    n.scale_slot = kvq->pool.scale_slot;
    n.scale_head = kvq->pool.scale_head;
    p.index_error = kvq->index_error;
    p.pages = kvq->pool.pages;
    p.page_size = kvq->pool.page_size;
    p.kv_heads = kvq->pool.kv_heads;
    p.dim = kvq->pool.dim;
    set_norms(n, norms);
    return from_cuda(kvq, bitlin_launch_norm_turn(n, k->dtype, kvq->dtype, true, reinterpret_cast<cudaStream_t>(stream)));
}

bitlin_status bitlin_kvq_read(bitlin_kvq_t kvq, const bitlin_kv_batch* batch, int tokens, const bitlin_rows* k,
                              const bitlin_rows* v, bitlin_stream_t stream)
{
    if (!kvq || !batch_ok(batch) || !rows_ok(k, tokens) || !rows_ok(v, tokens) || k->dtype != v->dtype) return BITLIN_EINVAL;
    if (!sizes_ok(tokens, kvq->pool.kv_heads, kvq->pool.dim) || !on_device(kvq->device)) return BITLIN_EINVAL;
    if (tokens == 0) return BITLIN_OK;
    QuantReadParams p = {};
    p.pool = kvq->pool;
    p.batch = batch_of(batch);
    const bitlin_rows* rows[2] = {k, v};
    for (int i = 0; i < 2; ++i) {
        p.out[i] = rows[i]->data;
        p.out_token[i] = rows[i]->token_stride;
        p.out_head[i] = rows[i]->head_stride;
    }
    p.index_error = kvq->index_error;
    p.tokens = tokens;
    return from_cuda(kvq, bitlin_launch_quant_read(p, k->dtype, reinterpret_cast<cudaStream_t>(stream)));
}

bitlin_status bitlin_kvq_attend(bitlin_kvq_t kvq, const bitlin_kv_batch* batch, int tokens, const bitlin_rows* q,
                                int heads, float scale, int causal, const bitlin_rows* out, float* lse,
                                bitlin_kv_t through, int f32_through, bitlin_stream_t stream)
{
    if (!kvq || !batch_ok(batch) || !rows_ok(q, tokens) || !rows_ok(out, tokens) || q->dtype != kvq->dtype) return BITLIN_EINVAL;
    if (out->dtype != kvq->dtype && out->dtype != BITLIN_F32) return BITLIN_EINVAL;
    if (!rows_wide(q) || !rows_wide(out) || !isfinite(scale) || (causal != 0 && causal != 1) ||
        (f32_through != 0 && f32_through != 1))
        return BITLIN_EINVAL;
    if (!sizes_ok(tokens, heads, kvq->pool.dim) || heads % kvq->pool.kv_heads || heads / kvq->pool.kv_heads > 128) return BITLIN_EINVAL;
    if (!on_device(kvq->device) || (through && !passes(*kvq, through))) return BITLIN_EINVAL;
    if (through && through->sticky != BITLIN_OK) return through->sticky;
    if (tokens == 0) return BITLIN_OK;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const long long rows = (long long)tokens * (heads / kvq->pool.kv_heads);
    if (through && (f32_through || out->dtype != BITLIN_F32) && rows > kThroughRows * (long long)batch->seqs) {
        if (kvq->through.lock() != through->workspace) {
            kvq->through = through->workspace;
            kvq->through_timed_out = false;
        } else if (kvq->through_timed_out) {
            return BITLIN_ETIMEOUT;
        }
        QuantUnpackParams u = {};
        u.pool = kvq->pool;
        u.batch = batch_of(batch);
        u.out[0] = through->k;
        u.out[1] = through->v;
        u.page_stride = through->page_stride;
        u.slot_stride = through->slot_stride;
        u.head_stride = through->head_stride;
        u.index_error = kvq->index_error;
        const cudaError_t e = bitlin_launch_quant_unpack(u, kvq->dtype, kvq->num_sms, s);
        if (e != cudaSuccess) return from_cuda(kvq, e);
        const bitlin_status st = bitlin_kv_attend_reporting(through, batch, tokens, q, heads, scale, causal, out, lse, kvq->index_error, stream);
        if (st == BITLIN_ECUDA || st == BITLIN_ENOMEM) kvq->last_cuda_error = through->last_cuda_error;
        return st;
    }
    const KvWorkspaceParts parts = bitlin_quant_attend_workspace(kvq->num_sms);
    unsigned char* workspace = kvq->workspace->data;
    QuantAttendParams p = {};
    p.pool = kvq->pool;
    p.batch = batch_of(batch);
    p.q = q->data;
    p.q_token = q->token_stride;
    p.q_head = q->head_stride;
    p.out = out->data;
    p.out_token = out->token_stride;
    p.out_head = out->head_stride;
    p.lse = lse;
    p.ws_o = reinterpret_cast<float*>(workspace + parts.o);
    p.ws_ml = reinterpret_cast<float*>(workspace + parts.ml);
    p.tickets = reinterpret_cast<int*>(workspace);
    p.index_error = kvq->index_error;
    p.tokens = tokens;
    p.heads = heads;
    p.group = heads / kvq->pool.kv_heads;
    p.causal = causal;
    p.scale = scale;
    p.bf16 = kvq->dtype == BITLIN_BF16;
    p.magic = 0x64006400u;
    p.group_inverse = (65536 + p.group - 1) / p.group;
    p.unit = kvq->unit;
    p.page_units = (uint32_t)(kvq->pool.page_stride / kvq->unit);
    p.slot_units = (uint32_t)(kvq->pool.slot_stride / kvq->unit);
    p.head_units = (uint32_t)(kvq->pool.head_stride / kvq->unit);
    p.scale_unit = kvq->scale_unit;
    p.scale_page_units = (uint32_t)(kvq->pool.scale_page / kvq->scale_unit);
    p.scale_slot_units = (uint32_t)(kvq->pool.scale_slot / kvq->scale_unit);
    p.scale_head_units = (uint32_t)(kvq->pool.scale_head / kvq->scale_unit);
    const int size = kvq->pool.page_size;
    p.page_shift = size & (size - 1) ? -1 : __builtin_ctz((unsigned)size);
    return from_cuda(kvq, bitlin_launch_quant_attend(p, out->dtype, kvq->num_sms, s));
}

bitlin_status bitlin_kvq_get_error(bitlin_kvq_t kvq)
{
    if (!kvq) return BITLIN_EINVAL;
    cudaError_t e = cudaDeviceSynchronize();
    int index_error = 0, timed_out = 0;
    const std::shared_ptr<KvWorkspace> through = kvq->through.lock();
    if (e == cudaSuccess && through) e = bitlin_kv_timed_out(*through, kvq->num_sms, &timed_out);
    if (e == cudaSuccess) e = cudaMemcpy(&index_error, kvq->index_error, sizeof(int), cudaMemcpyDeviceToHost);
    if (e != cudaSuccess) return from_cuda(kvq, e);
    if (timed_out) kvq->through_timed_out = true;
    if (kvq->through_timed_out) return BITLIN_ETIMEOUT;
    if (!index_error) return BITLIN_OK;
    e = cudaMemset(kvq->index_error, 0, sizeof(int));
    // before a later call, on whatever stream, can set it again
    if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);
    return e == cudaSuccess ? BITLIN_EINDEX : from_cuda(kvq, e);
}

int bitlin_kvq_cuda_error(bitlin_kvq_t kvq) { return kvq ? kvq->last_cuda_error : 0; }

bitlin_status bitlin_kvq_destroy(bitlin_kvq_t kvq)
{
    if (!kvq) return BITLIN_OK;
    cudaError_t e = cudaDeviceSynchronize();
    cudaFree(kvq->index_error);
    delete kvq;
    return e == cudaSuccess ? BITLIN_OK : BITLIN_ECUDA;
}

}  // extern "C"
