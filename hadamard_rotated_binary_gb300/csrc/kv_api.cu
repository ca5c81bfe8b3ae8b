// C-ABI of the attention side: rotary handles, paged-cache handles, argument checks.
#include <cuda_runtime.h>

#include <math.h>
#include <stdlib.h>

#include <memory>
#include <new>

#include "kv_internal.cuh"
#include "tensormap.cuh"

using namespace bitlin_impl;

namespace {

constexpr long long kDefaultWaitBudgetNs = 2000000000LL;  // 2 s per bounded wait

bitlin_status status_of(cudaError_t e)
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
bitlin_status current_device(int* dev)
{
    int major = 0, minor = 0;
    if (cudaGetDevice(dev) != cudaSuccess) return BITLIN_EDEVICE;
    cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, *dev);
    cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, *dev);
    return major == 10 && minor == 3 ? BITLIN_OK : BITLIN_EDEVICE;
}

bool on_device(int device)
{
    int dev = -1;
    return cudaGetDevice(&dev) == cudaSuccess && dev == device;
}

int type_size(int dtype) { return dtype == BITLIN_F32 ? 4 : 2; }

// A call of no tokens may have no memory.
bool rows_ok(const bitlin_rows* r, int tokens)
{
    return r && (r->data || tokens == 0) && (r->dtype == BITLIN_F32 || r->dtype == BITLIN_BF16 || r->dtype == BITLIN_F16) &&
           reinterpret_cast<uintptr_t>(r->data) % type_size(r->dtype) == 0;
}

// Rows that are moved 16 bytes at a time (TMA, vector stores).
bool rows_wide(const bitlin_rows* r)
{
    return reinterpret_cast<uintptr_t>(r->data) % 16 == 0 && r->token_stride > 0 && r->head_stride > 0 &&
           r->token_stride % 8 == 0 && r->head_stride % 8 == 0 && r->token_stride < (1LL << 38) &&
           r->head_stride < (1LL << 38);
}

bool sizes_ok(int tokens, int heads, int dim)
{
    return tokens >= 0 && heads >= 1 && heads <= 4096 && (unsigned long long)tokens * (unsigned)dim < (1ULL << 32);
}

bool batch_ok(const bitlin_kv_batch* b)
{
    return b && b->seqs >= 1 && b->q_offsets && b->kv_lens && b->table && b->table_pages >= 1 &&
           (b->seqs == 1 || b->table_stride >= b->table_pages);
}

KvBatch batch_of(const bitlin_kv_batch* b) { return {b->q_offsets, b->kv_lens, b->table, b->table_stride, b->table_pages, b->seqs}; }

void set_source(TurnParams& p, int i, const bitlin_rows* r)
{
    p.src[i] = r->data;
    p.src_token[i] = r->token_stride;
    p.src_head[i] = r->head_stride;
}

void set_rope(TurnParams& p, bitlin_rope_t r, const int32_t* pos)
{
    p.turns = r ? r->turns : nullptr;
    p.rotary = r ? r->rotary : 0;
    p.axes = r ? r->axes : 0;
    p.adjacent = r ? r->adjacent : 0;
    p.pos = pos;
}

void set_out(TurnParams& p, const bitlin_rows* r)
{
    p.out = r->data;
    p.out_token = r->token_stride;
    p.out_head = r->head_stride;
}

// f / (2 pi) modulo one turn, to one unit of 2^-64: the 24-bit significand of f
// times 1 / (2 pi) to 192 bits (pi by Machin's formula), enough for f32's largest
// exponent.
Turn turns_per_place(float f)
{
    const uint64_t inverse[3] = {0x28be60db9391054aULL, 0x7f09d5f47d4d3770ULL, 0x36d8a5664f10e410ULL};
    int exponent = 0;
    const uint64_t significand = (uint64_t)ldexpf(frexpf(fabsf(f), &exponent), 24);
    exponent -= 24;
    uint64_t product[4];  // from the lowest word; its unit is 2^(exponent - 192)
    uint64_t carry = 0;
    for (int i = 0; i < 3; ++i) {
        const unsigned __int128 x = (unsigned __int128)significand * inverse[2 - i] + carry;
        product[i] = (uint64_t)x;
        carry = (uint64_t)(x >> 64);
    }
    product[3] = carry;
    const int shift = 128 - exponent;  // product >> shift is in 2^-64; at least 24
    auto word = [&](int i) { return i < 4 ? product[i] : 0; };
    const int at = shift / 64, by = shift % 64;
    const uint64_t turns = by ? word(at) >> by | word(at + 1) << (64 - by) : word(at);
    const uint64_t half = word((shift - 1) / 64) >> (shift - 1) % 64 & 1;
    return f < 0 ? 0 - (turns + half) : turns + half;
}

// A tensor of 16-bit elements copied in boxes of 64 elements x `rows` (two of
// its dimensions), 128-byte swizzle, zeros outside.  dims and strides (bytes)
// from the innermost, whose stride is one element.
cudaError_t encode(unsigned char* tmap, int dtype, int rank, const void* data, const cuuint64_t* dims,
                   const cuuint64_t* strides, const cuuint32_t* box)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = bitlin_tensormap_encode_fn();
    if (!enc) return cudaErrorNotSupported;
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    const CUresult r = enc(reinterpret_cast<CUtensorMap*>(tmap),
                           dtype == BITLIN_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rank,
                           const_cast<void*>(data), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// A pool seen as [page][head][slot][dim], copied `box` slots of one head at a time.
cudaError_t encode_pool(const bitlin_kv& h, void* pool, int box, unsigned char* tmap)
{
    const cuuint64_t dims[4] = {(cuuint64_t)h.dim, (cuuint64_t)h.page_size, (cuuint64_t)h.kv_heads, (cuuint64_t)h.pages};
    const cuuint64_t strides[3] = {(cuuint64_t)h.slot_stride * 2, (cuuint64_t)h.head_stride * 2, (cuuint64_t)h.page_stride * 2};
    const cuuint32_t boxes[4] = {64, (cuuint32_t)box, 1, 1};
    return encode(tmap, h.dtype, 4, pool, dims, strides, boxes);
}

// Queries seen as [token][head][dim], copied a group's heads of `box` tokens at a time.
cudaError_t encode_queries(const bitlin_kv& h, const bitlin_rows& q, int tokens, int heads, int box, unsigned char* tmap)
{
    const cuuint64_t dims[3] = {(cuuint64_t)h.dim, (cuuint64_t)heads, (cuuint64_t)tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)q.head_stride * 2, (cuuint64_t)q.token_stride * 2};
    const cuuint32_t boxes[3] = {64, (cuuint32_t)(heads / h.kv_heads), (cuuint32_t)box};
    return encode(tmap, h.dtype, 3, q.data, dims, strides, boxes);
}

// A workspace for the handle's calls, with zero tickets.
cudaError_t new_workspace(bitlin_kv& h)
{
    const KvWorkspaceParts parts = bitlin_attend_workspace(h.dim, h.num_sms);
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

}  // namespace

extern "C" {

bitlin_status bitlin_rope_create(bitlin_rope_t* out, int rotary_dim, int axes, const float* inv_freq,
                                 const int32_t* axis, int pairing)
{
    if (!out) return BITLIN_EINVAL;
    *out = nullptr;
    if (!inv_freq || rotary_dim < 2 || rotary_dim % 2 || rotary_dim > 65536 || axes < 1 || axes > 8) return BITLIN_EINVAL;
    if (pairing != BITLIN_PAIRS_HALF && pairing != BITLIN_PAIRS_ADJACENT) return BITLIN_EINVAL;
    const int pairs = rotary_dim / 2;
    for (int i = 0; i < pairs; ++i)
        if (!isfinite(inv_freq[i]) || (axis && (axis[i] < 0 || axis[i] >= axes))) return BITLIN_EINVAL;
    int dev = 0;
    bitlin_status st = current_device(&dev);
    if (st != BITLIN_OK) return st;

    std::unique_ptr<Turn[]> turns(new (std::nothrow) Turn[pairs]);
    std::unique_ptr<bitlin_rope> r(new (std::nothrow) bitlin_rope());
    if (!turns || !r) return BITLIN_ENOMEM;
    for (int i = 0; i < pairs; ++i)
        turns[i] = ((turns_per_place(inv_freq[i]) + (kAxisMask + 1) / 2) & ~kAxisMask) | (Turn)(axis ? axis[i] : 0);
    r->device = dev;
    r->rotary = rotary_dim;
    r->axes = axes;
    r->adjacent = pairing == BITLIN_PAIRS_ADJACENT;
    cudaError_t e = cudaMalloc(&r->turns, pairs * sizeof(Turn));
    if (e == cudaSuccess) e = cudaMemcpy(r->turns, turns.get(), pairs * sizeof(Turn), cudaMemcpyHostToDevice);
    // A copy from pageable memory may return before it has landed, and streams that
    // do not block with the default one would not wait for it.
    if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);
    if (e != cudaSuccess) {
        cudaFree(r->turns);
        return status_of(e);
    }
    *out = r.release();
    return BITLIN_OK;
}

bitlin_status bitlin_rope_apply(bitlin_rope_t r, const bitlin_rows* x, int tokens, int heads, int head_dim,
                                const int32_t* pos, const bitlin_rows* out, int inverse, bitlin_stream_t stream)
{
    if (!r || !rows_ok(x, tokens) || !rows_ok(out, tokens) || (!pos && tokens) || !sizes_ok(tokens, heads, head_dim)) return BITLIN_EINVAL;
    if (head_dim < r->rotary || (inverse != 0 && inverse != 1) || !on_device(r->device)) return BITLIN_EINVAL;
    if (tokens == 0) return BITLIN_OK;
    TurnParams p = {};
    set_source(p, 0, x);
    set_out(p, out);
    set_rope(p, r, pos);
    p.tokens = tokens;
    p.heads = heads;
    p.dim = head_dim;
    p.inverse = inverse;
    return from_cuda(r, bitlin_launch_turn(p, x->dtype, out->dtype, reinterpret_cast<cudaStream_t>(stream)));
}

int bitlin_rope_cuda_error(bitlin_rope_t r) { return r ? r->last_cuda_error : 0; }

bitlin_status bitlin_rope_destroy(bitlin_rope_t r)
{
    if (!r) return BITLIN_OK;
    cudaError_t e = cudaDeviceSynchronize();
    cudaFree(r->turns);
    delete r;
    return e == cudaSuccess ? BITLIN_OK : BITLIN_ECUDA;
}

bitlin_status bitlin_kv_create(bitlin_kv_t* out, void* k, void* v, int pages, int page_size, int kv_heads,
                               int head_dim, int dtype, long long page_stride, long long slot_stride,
                               long long head_stride)
{
    if (!out) return BITLIN_EINVAL;
    *out = nullptr;
    if (!k || !v || reinterpret_cast<uintptr_t>(k) % 16 || reinterpret_cast<uintptr_t>(v) % 16) return BITLIN_EINVAL;
    if (pages < 1 || page_size < 8 || page_size % 8 || page_size > 65536 || kv_heads < 1 || kv_heads > 4096)
        return BITLIN_EINVAL;
    if (head_dim < 8 || head_dim % 8 || head_dim > 256 || (dtype != BITLIN_BF16 && dtype != BITLIN_F16))
        return BITLIN_EINVAL;
    for (long long stride : {page_stride, slot_stride, head_stride})
        if (stride < 8 || stride % 8 || stride >= (1LL << 39)) return BITLIN_EINVAL;
    int dev = 0;
    bitlin_status st = current_device(&dev);
    if (st != BITLIN_OK) return st;
    std::unique_ptr<bitlin_kv> h(new (std::nothrow) bitlin_kv());
    if (!h) return BITLIN_ENOMEM;
    h->device = dev;
    h->k = k;
    h->v = v;
    h->pages = pages;
    h->page_size = page_size;
    h->kv_heads = kv_heads;
    h->dim = head_dim;
    h->dtype = dtype;
    h->page_stride = page_stride;
    h->slot_stride = slot_stride;
    h->head_stride = head_stride;
    h->wait_budget_ns = kDefaultWaitBudgetNs;
    if (const char* env = getenv("BITLIN_WAIT_BUDGET_NS")) {
        const long long ns = atoll(env);
        if (ns > 0) h->wait_budget_ns = ns;
    }
    int box_k = 0, box_v = 0;
    bitlin_attend_boxes(head_dim, page_size, &box_k, &box_v);
    cudaError_t e = cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = encode_pool(*h, k, box_k, h->tmap_k);
    if (e == cudaSuccess) e = encode_pool(*h, v, box_v, h->tmap_v);
    if (e == cudaSuccess) e = bitlin_attend_load(head_dim, dtype);
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

bitlin_status bitlin_kv_share(bitlin_kv_t kv, bitlin_kv_t with)
{
    if (!kv || !with || kv->device != with->device) return BITLIN_EINVAL;
    if (with->workspace->bytes < bitlin_attend_workspace(kv->dim, kv->num_sms).bytes) return BITLIN_EINVAL;
    // the handle's own workspace may be freed here: not under its calls
    const cudaError_t e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return from_cuda(kv, e);
    kv->workspace = with->workspace;
    return BITLIN_OK;
}

bitlin_status bitlin_kv_append(bitlin_kv_t kv, const bitlin_kv_batch* batch, int tokens, bitlin_rope_t rope,
                               const int32_t* pos, const bitlin_rows* k, const bitlin_rows* v,
                               const bitlin_rows* q, int heads, const bitlin_rows* q_out, bitlin_stream_t stream)
{
    if (!kv || !batch_ok(batch) || !rows_ok(k, tokens) || !rows_ok(v, tokens) || k->dtype != v->dtype) return BITLIN_EINVAL;
    if (!sizes_ok(tokens, q ? heads : 1, kv->dim) || (rope && rope->rotary > kv->dim)) return BITLIN_EINVAL;
    if (q && (!rows_ok(q, tokens) || !rows_ok(q_out, tokens) || q->dtype != k->dtype || q_out->dtype != kv->dtype)) return BITLIN_EINVAL;
    if (!on_device(kv->device) || (rope && rope->device != kv->device)) return BITLIN_EINVAL;
    if (kv->sticky != BITLIN_OK) return kv->sticky;
    if (tokens == 0) return BITLIN_OK;
    TurnParams p = {};
    if (q) {
        set_source(p, 0, q);
        set_out(p, q_out);
    }
    set_source(p, 1, k);
    set_source(p, 2, v);
    set_rope(p, rope, pos);
    p.pool[0] = kv->k;
    p.pool[1] = kv->v;
    p.page_stride = kv->page_stride;
    p.slot_stride = kv->slot_stride;
    p.head_stride = kv->head_stride;
    p.batch = batch_of(batch);
    p.index_error = kv->index_error;
    p.pages = kv->pages;
    p.page_size = kv->page_size;
    p.tokens = tokens;
    p.heads = q ? heads : 0;
    p.kv_heads = kv->kv_heads;
    p.dim = kv->dim;
    p.append = 1;
    return from_cuda(kv, bitlin_launch_turn(p, k->dtype, kv->dtype, reinterpret_cast<cudaStream_t>(stream)));
}

bitlin_status bitlin_kv_attend(bitlin_kv_t kv, const bitlin_kv_batch* batch, int tokens, const bitlin_rows* q,
                               int heads, float scale, int causal, const bitlin_rows* out, float* lse,
                               bitlin_stream_t stream)
{
    if (!kv || !batch_ok(batch) || !rows_ok(q, tokens) || !rows_ok(out, tokens) || q->dtype != kv->dtype) return BITLIN_EINVAL;
    if (out->dtype != kv->dtype && out->dtype != BITLIN_F32) return BITLIN_EINVAL;
    if (!rows_wide(q) || !rows_wide(out) || !isfinite(scale) || (causal != 0 && causal != 1)) return BITLIN_EINVAL;
    if (!sizes_ok(tokens, heads, kv->dim) || heads % kv->kv_heads || heads / kv->kv_heads > 128) return BITLIN_EINVAL;
    if (!on_device(kv->device)) return BITLIN_EINVAL;
    if (kv->sticky != BITLIN_OK) return kv->sticky;
    if (tokens == 0) return BITLIN_OK;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const KvWorkspaceParts parts = bitlin_attend_workspace(kv->dim, kv->num_sms);
    unsigned char* workspace = kv->workspace->data;
    AttendParams p = {};
    p.v_pool = kv->v;
    p.page_stride = kv->page_stride;
    p.slot_stride = kv->slot_stride;
    p.head_stride = kv->head_stride;
    p.batch = batch_of(batch);
    p.out = out->data;
    p.out_token = out->token_stride;
    p.out_head = out->head_stride;
    p.lse = lse;
    p.ws_o = reinterpret_cast<float*>(workspace + parts.o);
    p.ws_ml = reinterpret_cast<float*>(workspace + parts.ml);
    p.tickets = reinterpret_cast<int*>(workspace);
    p.timed_out = reinterpret_cast<int*>(workspace + parts.timed_out);
    p.index_error = kv->index_error;
    p.wait_budget_ns = kv->wait_budget_ns;
    p.pages = kv->pages;
    p.page_size = kv->page_size;
    p.page_shift = kv->page_size & (kv->page_size - 1) ? -1 : __builtin_ctz((unsigned)kv->page_size);
    p.tokens = tokens;
    p.heads = heads;
    p.kv_heads = kv->kv_heads;
    p.group = heads / kv->kv_heads;
    p.dim = kv->dim;
    p.causal = causal;
    bitlin_attend_rows(tokens, batch->seqs, p.group, out->dtype, &p.tile_tokens, &p.q_box, &p.few);
    p.item_extra = bitlin_attend_item_extra(kv->dim);
    bitlin_attend_boxes(kv->dim, kv->page_size, &p.box_k, &p.box_v);
    p.stall_test = kv->stall_test;
    p.scale = scale;
    alignas(64) unsigned char tmap_q[128];
    const cudaError_t e = encode_queries(*kv, *q, tokens, heads, p.q_box, tmap_q);
    if (e != cudaSuccess) return from_cuda(kv, e);
    return from_cuda(kv, bitlin_launch_attend(p, kv->dtype, out->dtype, tmap_q, kv->tmap_k, kv->tmap_v, kv->num_sms, st));
}

bitlin_status bitlin_kv_set_wait_budget(bitlin_kv_t kv, long long ns)
{
    if (!kv || ns <= 0) return BITLIN_EINVAL;
    kv->wait_budget_ns = ns;
    return BITLIN_OK;
}

bitlin_status bitlin_kv_test_stall(bitlin_kv_t kv, int on)
{
    if (!kv) return BITLIN_EINVAL;
    kv->stall_test = on ? 1 : 0;
    return BITLIN_OK;
}

bitlin_status bitlin_kv_get_error(bitlin_kv_t kv)
{
    if (!kv) return BITLIN_EINVAL;
    cudaError_t e = cudaDeviceSynchronize();
    int timed_out = 0, index_error = 0;
    const KvWorkspaceParts parts = bitlin_attend_workspace(kv->dim, kv->num_sms);
    if (e == cudaSuccess) e = cudaMemcpy(&timed_out, kv->workspace->data + parts.timed_out, sizeof(int), cudaMemcpyDeviceToHost);
    if (e == cudaSuccess) e = cudaMemcpy(&index_error, kv->index_error, sizeof(int), cudaMemcpyDeviceToHost);
    if (e != cudaSuccess) return from_cuda(kv, e);
    if (timed_out) kv->sticky = BITLIN_ETIMEOUT;
    if (kv->sticky != BITLIN_OK || !index_error) return kv->sticky;
    e = cudaMemset(kv->index_error, 0, sizeof(int));
    // before a later call, on whatever stream, can set it again
    if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);
    return e == cudaSuccess ? BITLIN_EINDEX : from_cuda(kv, e);
}

int bitlin_kv_cuda_error(bitlin_kv_t kv) { return kv ? kv->last_cuda_error : 0; }

bitlin_status bitlin_kv_destroy(bitlin_kv_t kv)
{
    if (!kv) return BITLIN_OK;
    cudaError_t e = cudaDeviceSynchronize();
    cudaFree(kv->index_error);
    delete kv;
    return e == cudaSuccess ? BITLIN_OK : BITLIN_ECUDA;
}

}  // extern "C"
