// Rows of a 4-bit cache read back, and its pages as 16-bit ones.
//
// A value is (nibble - 8) * scale, exact in every output type (see quant.cuh).
// Bound: HBM, the writes of the 16-bit values above all.  A thread takes 8
// elements (a 32-bit word) of a head; a warp's words are consecutive.  Values are
// made two by two in f16 (by integer to float conversions the pages of a 32,768
// token context took 130 us, so 25).  Measured: 8,191 tokens of 8 heads of 128, k and v,
// read back to f16 in 7.8 us (5.5 TB/s; four heads to a thread 9.6, two 13.7).
#include "kv_internal.cuh"
#include "ptx.cuh"
#include "quant.cuh"

using namespace bitlin_impl;

namespace {

constexpr int kThreads = 128;
constexpr int kHeadsPerThread = 8;
constexpr int kUnpackThreads = 256;

// A word's eight values, two by two, as f16.
__device__ __forceinline__ void eight_halves(uint32_t word, uint32_t scale_byte, uint32_t (&v)[4])
{
    const QuantScale2 s = quant_scale2(scale_byte * 0x00010001u);
    const uint32_t magic = 0x64006400u;
    const __half2 a = quant_low(word, s, magic), b = quant_high(word, s, magic);  // elements 0 and 4, 1 and 5
    const __half2 c = quant_low(word >> 8, s, magic), d = quant_high(word >> 8, s, magic);
    auto bits = [](const __half2& x) { return *reinterpret_cast<const uint32_t*>(&x); };
    v[0] = __byte_perm(bits(a), bits(b), 0x5410);
    v[1] = __byte_perm(bits(c), bits(d), 0x5410);
    v[2] = __byte_perm(bits(a), bits(b), 0x7632);
    v[3] = __byte_perm(bits(c), bits(d), 0x7632);
}

// Two f16 values as two of T.
template <typename T>
__device__ __forceinline__ uint32_t two_of(uint32_t h)
{
    return h;
}
template <>
__device__ __forceinline__ uint32_t two_of<__nv_bfloat16>(uint32_t h)
{
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    const __nv_bfloat162 v = __floats2bfloat162_rn(f.x, f.y);
    return *reinterpret_cast<const uint32_t*>(&v);
}

template <typename T>
__device__ __forceinline__ void store8(T* dst, uint32_t word, uint32_t scale_byte, bool wide)
{
    uint32_t h[4];
    eight_halves(word, scale_byte, h);
    alignas(16) T v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (sizeof(T) == 4 || !wide) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
            v[2 * j] = from_f32<T>(f.x);
            v[2 * j + 1] = from_f32<T>(f.y);
        } else {
            reinterpret_cast<uint32_t*>(v)[j] = two_of<T>(h[j]);
        }
    }
    if (wide) {
#pragma unroll
        for (int j = 0; j < (int)sizeof(T) / 2; ++j) reinterpret_cast<uint4*>(dst)[j] = reinterpret_cast<const uint4*>(v)[j];
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) dst[j] = v[j];
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) bitlin_quant_read(const QuantReadParams p, int wide)
{
    ptx::griddep_wait();
    const int units = p.pool.dim / 8;
    const uint32_t idx = blockIdx.x * (uint32_t)kThreads + threadIdx.x;
    const uint32_t token = idx / (uint32_t)units;
    const int u = (int)(idx - token * (uint32_t)units);
    const int t = (int)min(token, (uint32_t)(p.tokens - 1));
    const int warp_first = (int)min((idx - (threadIdx.x & 31)) / (uint32_t)units, (uint32_t)(p.tokens - 1));
    int seq = warp_sequence_of(p.batch, warp_first);
    while (seq < p.batch.seqs && p.batch.q_offsets[seq + 1] <= t) ++seq;
    if (token >= (uint32_t)p.tokens || seq >= p.batch.seqs) return;
    const int place = p.batch.kv_lens[seq] - (p.batch.q_offsets[seq + 1] - t);
    const int at = place / p.pool.page_size;
    int page = -1;
    if (place >= 0 && at < p.batch.table_pages) page = p.batch.table[seq * p.batch.table_stride + at];
    const int groups = (p.pool.kv_heads + kHeadsPerThread - 1) / kHeadsPerThread;
    const int kind = blockIdx.y >= groups, h0 = (blockIdx.y - kind * groups) * kHeadsPerThread;
    const bool inside = page >= 0 && page < p.pool.pages;
    if (!inside) *p.index_error = 1;
    const long long slot = place - (long long)at * p.pool.page_size;
    const uint8_t* codes = p.pool.codes[kind] + page * p.pool.page_stride + slot * p.pool.slot_stride + 4 * u;
    const uint8_t* scales = p.pool.scales[kind] + page * p.pool.scale_page + slot * p.pool.scale_slot + 8 * u / (p.pool.dim / 4);
    T* out = static_cast<T*>(p.out[kind]) + t * p.out_token[kind] + 8 * u;
    uint32_t word[kHeadsPerThread], scale[kHeadsPerThread];
#pragma unroll
    for (int i = 0; i < kHeadsPerThread; ++i) {
        word[i] = scale[i] = 0;
        if (inside && h0 + i < p.pool.kv_heads) {
            word[i] = *reinterpret_cast<const uint32_t*>(codes + (h0 + i) * p.pool.head_stride);
            scale[i] = scales[(h0 + i) * p.pool.scale_head];
        }
    }
#pragma unroll
    for (int i = 0; i < kHeadsPerThread; ++i)
        if (h0 + i < p.pool.kv_heads) store8<T>(out + (h0 + i) * p.out_head[kind], word[i], scale[i], wide);
}

// Block (x, y): every gridDim.x-th page of every gridDim.y-th sequence.  A warp takes the slots of one head
// of K or of V, a word to a lane: 32 / (D / 8) slots at a time, eight times in flight.
template <typename T>
__global__ void __launch_bounds__(kUnpackThreads) bitlin_quant_unpack(const QuantUnpackParams p)
{
    constexpr int kBatch = 8;
    ptx::griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int units = p.pool.dim / 8, u = lane & (units - 1), slots = 32 / units, mine = lane / units;
    const int group = 8 * (8 * u / (p.pool.dim / 4));  // the group's byte in a head's scales, in bits
    for (int seq = blockIdx.y; seq < p.batch.seqs; seq += gridDim.y) {
        if (p.batch.q_offsets[seq + 1] <= p.batch.q_offsets[seq]) continue;  // nothing asks for it
        const int len = min(max(p.batch.kv_lens[seq], 0), 1 << 30);
        const int want = (int)(((long long)len + p.pool.page_size - 1) / p.pool.page_size);
        const int pages = min(want, p.batch.table_pages);
        if (pages < want) *p.index_error = 1;
        for (int at = blockIdx.x; at < pages; at += gridDim.x) {
            const int page = p.batch.table[seq * p.batch.table_stride + at];
            if (page < 0 || page >= p.pool.pages) {  // attention reads it as zeros
                *p.index_error = 1;
                continue;
            }
            const int held = min(p.pool.page_size, len - at * p.pool.page_size);
            for (int i = warp; i < 2 * p.pool.kv_heads; i += kUnpackThreads / 32) {
                const int kind = i & 1, head = i >> 1;
                const uint8_t* codes = p.pool.codes[kind] + page * p.pool.page_stride + head * p.pool.head_stride + 4 * u;
                const uint8_t* scales = p.pool.scales[kind] + page * p.pool.scale_page + head * p.pool.scale_head;
                T* out = static_cast<T*>(p.out[kind]) + page * p.page_stride + head * p.head_stride + 8 * u;
                for (int first = mine; first < held; first += slots * kBatch) {
                    uint32_t word[kBatch], scale[kBatch];
#pragma unroll
                    for (int j = 0; j < kBatch; ++j) {
                        const int slot = first + j * slots;
                        if (slot < held) {
                            word[j] = *reinterpret_cast<const uint32_t*>(codes + slot * p.pool.slot_stride);
                            scale[j] = *reinterpret_cast<const uint32_t*>(scales + slot * p.pool.scale_slot);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < kBatch; ++j) {
                        const int slot = first + j * slots;
                        if (slot < held) store8<T>(out + slot * p.slot_stride, word[j], scale[j] >> group & 0xff, true);
                    }
                }
            }
        }
    }
}

cudaLaunchConfig_t config(dim3 grid, cudaStream_t s, cudaLaunchAttribute* attr)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr->val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

template <typename T>
cudaError_t read(const QuantReadParams& p, cudaStream_t s)
{
    bool wide = true;
    for (int i = 0; i < 2; ++i) {
        const int n = 16 / sizeof(T);
        wide = wide && reinterpret_cast<uintptr_t>(p.out[i]) % 16 == 0 && p.out_token[i] % n == 0 && p.out_head[i] % n == 0;
    }
    const uint64_t threads = (uint64_t)p.tokens * (p.pool.dim / 8);
    const int groups = (p.pool.kv_heads + kHeadsPerThread - 1) / kHeadsPerThread;
    cudaLaunchAttribute attr = {};
    const cudaLaunchConfig_t cfg = config(dim3((unsigned)((threads + kThreads - 1) / kThreads), 2 * groups), s, &attr);
    return cudaLaunchKernelEx(&cfg, bitlin_quant_read<T>, p, (int)wide);
}

}  // namespace

cudaError_t bitlin_launch_quant_read(const QuantReadParams& p, int dst_dtype, cudaStream_t s)
{
    switch (dst_dtype) {
    case BITLIN_F32: return read<float>(p, s);
    case BITLIN_BF16: return read<__nv_bfloat16>(p, s);
    default: return read<__half>(p, s);
    }
}

cudaError_t bitlin_launch_quant_unpack(const QuantUnpackParams& p, int dst_dtype, int num_sms, cudaStream_t s)
{
    // blocks for sixteen to an SM, or for a page each
    const int want = (16 * num_sms + p.batch.seqs - 1) / p.batch.seqs;
    cudaLaunchAttribute attr = {};
    cudaLaunchConfig_t cfg = config(dim3(want < p.batch.table_pages ? want : p.batch.table_pages, p.batch.seqs < 65535 ? p.batch.seqs : 65535), s, &attr);
    cfg.blockDim = dim3(kUnpackThreads);
    return dst_dtype == BITLIN_BF16 ? cudaLaunchKernelEx(&cfg, bitlin_quant_unpack<__nv_bfloat16>, p)
                                    : cudaLaunchKernelEx(&cfg, bitlin_quant_unpack<__half>, p);
}
