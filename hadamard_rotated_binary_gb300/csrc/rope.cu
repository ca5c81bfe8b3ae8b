// Rotary positions with several axes, and the append of rotated keys and
// plain values to the paged cache.
//
// Mathematics: pair i of a head turns by t = pos[axis[i]] * inv_freq[i],
// (a, b) -> (a cos t - b sin t, b cos t + a sin t).  A frequency is held as a
// 64-bit fixed-point fraction of a turn, so pos * frequency modulo one turn is
// one wrapping integer product at every int32 position; its top 32 bits are the
// angle to 2^-32 of a turn (and 2^-31 at most from the frequency's rounding),
// already within half a turn of zero, and 24 of them enter the sine: 1e-7 at
// most.  There the hardware's sine and cosine are good to 2^-21, enough for a
// 16-bit output (2^-9 and 2^-12); an f32 output takes sincospi.
//
// Bound: HBM (each element is read once and written once).  A thread owns one
// "unit" of a head: two chunks of VEC consecutive elements, half the rotated
// (or the passed-through) part apart, which are the two sides of VEC pairs
// (pairs half R apart) or hold VEC/2 pairs each (adjacent pairs).  It takes
// its unit of kHeadsPerThread heads of one token, so the angles are computed
// once for them and all their loads are in flight together; a warp's chunks
// are consecutive, so loads and stores coalesce.  Where sizes, strides or
// alignment do not allow chunks, VEC = 1 takes one pair per thread.
//
// Measured (GB300, inputs changing from call to call): a video clip's 16,128 x
// 16 x 80 bf16 16.2 us (5.1 TB/s), the gradient of 4,097 x 24 x 256 f32 32.3 us
// (6.2 TB/s), prompts of 8,191 tokens appended with their queries (48 heads of
// 128) 40.3 us (5.5 TB/s); one token's queries 1.9 us in a graph.  The variants
// were compared on graph replays of one clip, whose 83 MB L2 partly holds: 12.9
// us as it is, two heads a thread 15.0 (the angles are computed twice as often),
// blocks of 256 13.5, chunks of 8 16-bit elements 13.5, sincospi for a 16-bit
// output and a 16-byte table entry 15.6.
#include "kv_internal.cuh"
#include "ptx.cuh"

using namespace bitlin_impl;

namespace {

constexpr int kThreads = 128;
constexpr int kHeadsPerThread = 4;

template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Chunk {
    T v[VEC];
};

template <typename TI, typename TO, int VEC>
__global__ void __launch_bounds__(kThreads) bitlin_turn(const TurnParams p)
{
    ptx::griddep_wait();
    const uint32_t idx = blockIdx.x * (uint32_t)kThreads + threadIdx.x;
    const uint32_t token = idx / (uint32_t)p.units;
    const int u = (int)(idx - token * (uint32_t)p.units);
    const int t = (int)min(token, (uint32_t)(p.tokens - 1));

    // which tensor: q, k or v, and which heads of it
    int kind = 0, group = blockIdx.y;
    if (group >= p.q_groups) {
        group -= p.q_groups;
        kind = 1;
        if (group >= p.kv_groups) {
            group -= p.kv_groups;
            kind = 2;
        }
    }
    const int heads = kind == 0 ? p.heads : p.kv_heads;
    const int h0 = group * kHeadsPerThread;

    // the token's place in its sequence (all lanes take part in the search)
    int place = 0;
    bool padding = false;
    int seq = 0;
    if (p.append) {
        const int warp_first = (int)min((idx - (threadIdx.x & 31)) / (uint32_t)p.units, (uint32_t)(p.tokens - 1));
        seq = warp_sequence_of(p.batch, warp_first);
        while (seq < p.batch.seqs && p.batch.q_offsets[seq + 1] <= t) ++seq;
        padding = seq >= p.batch.seqs;
        if (!padding) place = p.batch.kv_lens[seq] - (p.batch.q_offsets[seq + 1] - t);
    }
    if (token >= (uint32_t)p.tokens || padding) return;

    // where the row goes
    TO* dst;
    long long dst_head;
    if (kind == 0) {
        dst = static_cast<TO*>(p.out) + t * p.out_token;
        dst_head = p.out_head;
    } else {
        const int at = place / p.page_size;
        int page = -1;
        if (place >= 0 && at < p.batch.table_pages) page = p.batch.table[seq * p.batch.table_stride + at];
        if (page < 0 || page >= p.pages) {
            *p.index_error = 1;
            return;
        }
        dst = static_cast<TO*>(p.pool[kind - 1]) + page * p.page_stride + (place - at * p.page_size) * p.slot_stride;
        dst_head = p.head_stride;
    }
    const TI* src = static_cast<const TI*>(p.src[kind]) + t * p.src_token[kind];
    const long long src_head = p.src_head[kind];

    // the unit's two chunks
    const int rotated = p.rotary / 2 / VEC;  // units that rotate
    const bool turning = p.turns != nullptr && kind != 2 && u < rotated;
    int lo, hi;
    if (VEC > 1) {
        lo = u < rotated ? u * VEC : p.rotary + (u - rotated) * VEC;
        hi = lo + (u < rotated ? p.rotary : p.dim - p.rotary) / 2;
    } else if (u < rotated) {
        lo = p.adjacent ? 2 * u : u;
        hi = p.adjacent ? lo + 1 : u + p.rotary / 2;
    } else {
        lo = p.rotary + 2 * (u - rotated);
        hi = lo + 1;
    }
    const bool has_hi = VEC > 1 || hi < p.dim;

    float cs[VEC], sn[VEC];
    if (turning) {
        // the token's positions on up to four axes (a fifth to eighth is read where it is used)
        int at4[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) at4[x] = p.pos && x < p.axes ? p.pos[(long long)x * p.tokens + t] : place;
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            // adjacent pairs: chunk lo holds pairs lo/2.., chunk hi pairs hi/2..
            int f = lo + j;
            if (p.adjacent) f = VEC == 1 ? u : j < VEC / 2 ? lo / 2 + j : hi / 2 + j - VEC / 2;
            const Turn w = p.turns[f];
            const int axis = (int)(w & kAxisMask);
            int at = axis & 2 ? (axis & 1 ? at4[3] : at4[2]) : (axis & 1 ? at4[1] : at4[0]);
            if (axis >= 4 && p.pos) at = p.pos[(long long)axis * p.tokens + t];
            const int32_t frac = (int32_t)(((uint64_t)(long long)at * (w & ~kAxisMask)) >> 32);
            if (sizeof(TO) == 2) {
                const float angle = (float)frac * 1.4629180792671596e-9f;  // 2^-32 of a turn, in radians
                sn[j] = __sinf(angle);
                cs[j] = __cosf(angle);
            } else {
                sincospif((float)frac * 4.656612873077393e-10f /* 2^-31: half turns */, &sn[j], &cs[j]);
            }
            if (p.inverse) sn[j] = -sn[j];
        }
    }

    Chunk<TI, VEC> a[kHeadsPerThread], b[kHeadsPerThread];
#pragma unroll
    for (int i = 0; i < kHeadsPerThread; ++i) {
        if (h0 + i < heads) {
            const TI* row = src + (h0 + i) * src_head;
            a[i] = *reinterpret_cast<const Chunk<TI, VEC>*>(row + lo);
            if (has_hi) b[i] = *reinterpret_cast<const Chunk<TI, VEC>*>(row + hi);
        }
    }
#pragma unroll
    for (int i = 0; i < kHeadsPerThread; ++i) {
        if (h0 + i >= heads) break;
        float x[VEC], y[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            x[j] = to_f32(a[i].v[j]);
            y[j] = has_hi ? to_f32(b[i].v[j]) : 0.f;
        }
        if (turning) {
            if (VEC > 1 && p.adjacent) {
#pragma unroll
                for (int j = 0; j < VEC / 2; ++j) {
                    const float c0 = cs[j], s0 = sn[j], c1 = cs[VEC / 2 + j], s1 = sn[VEC / 2 + j];
                    const float x0 = x[2 * j], x1 = x[2 * j + 1], y0 = y[2 * j], y1 = y[2 * j + 1];
                    x[2 * j] = x0 * c0 - x1 * s0;
                    x[2 * j + 1] = x1 * c0 + x0 * s0;
                    y[2 * j] = y0 * c1 - y1 * s1;
                    y[2 * j + 1] = y1 * c1 + y0 * s1;
                }
            } else {
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const float x0 = x[j];
                    x[j] = x0 * cs[j] - y[j] * sn[j];
                    y[j] = y[j] * cs[j] + x0 * sn[j];
                }
            }
        }
        Chunk<TO, VEC> c, d;
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            c.v[j] = from_f32<TO>(x[j]);
            d.v[j] = from_f32<TO>(y[j]);
        }
        TO* row = dst + (h0 + i) * dst_head;
        *reinterpret_cast<Chunk<TO, VEC>*>(row + lo) = c;
        if (has_hi) *reinterpret_cast<Chunk<TO, VEC>*>(row + hi) = d;
    }
}

template <typename TI, typename TO, int VEC>
cudaError_t launch_turn(TurnParams& p, cudaStream_t s)
{
    p.units = VEC > 1 ? p.dim / (2 * VEC) : (p.dim + 1) / 2;
    p.q_groups = (p.heads + kHeadsPerThread - 1) / kHeadsPerThread;
    p.kv_groups = p.append ? (p.kv_heads + kHeadsPerThread - 1) / kHeadsPerThread : 0;
    const uint64_t threads = (uint64_t)p.tokens * p.units;
    const dim3 grid((unsigned)((threads + kThreads - 1) / kThreads), p.q_groups + 2 * p.kv_groups);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, bitlin_turn<TI, TO, VEC>, p);
}

// Whether rows of this tensor can be read or written in chunks of VEC elements.
bool chunked(const void* data, long long token, long long head, int size, int vec)
{
    return reinterpret_cast<uintptr_t>(data) % (uintptr_t)(size * vec) == 0 && token % vec == 0 && head % vec == 0;
}

// Whether all rows of a call divide into chunks of `vec` elements.
template <typename TI, typename TO>
bool divides(const TurnParams& p, int vec)
{
    bool ok = p.rotary % (2 * vec) == 0 && (p.dim - p.rotary) % (2 * vec) == 0;
    if (p.heads) {
        ok = ok && chunked(p.src[0], p.src_token[0], p.src_head[0], sizeof(TI), vec);
        ok = ok && chunked(p.out, p.out_token, p.out_head, sizeof(TO), vec);
    }
    if (p.append)
        for (int i = 1; i < 3; ++i) ok = ok && chunked(p.src[i], p.src_token[i], p.src_head[i], sizeof(TI), vec);
    return ok;
}

template <typename TI, typename TO>
cudaError_t pick_turn(const TurnParams& p, cudaStream_t s)
{
    TurnParams q = p;
    if (divides<TI, TO>(p, 4)) return launch_turn<TI, TO, 4>(q, s);
    if (divides<TI, TO>(p, 2)) return launch_turn<TI, TO, 2>(q, s);
    return launch_turn<TI, TO, 1>(q, s);
}

template <typename TI>
cudaError_t pick_out(const TurnParams& p, int dst_dtype, cudaStream_t s)
{
    switch (dst_dtype) {
    case BITLIN_F32: return pick_turn<TI, float>(p, s);
    case BITLIN_BF16: return pick_turn<TI, __nv_bfloat16>(p, s);
    default: return pick_turn<TI, __half>(p, s);
    }
}

}  // namespace

cudaError_t bitlin_launch_turn(const TurnParams& p, int src_dtype, int dst_dtype, cudaStream_t s)
{
    switch (src_dtype) {
    case BITLIN_F32: return pick_out<float>(p, dst_dtype, s);
    case BITLIN_BF16: return pick_out<__nv_bfloat16>(p, dst_dtype, s);
    default: return pick_out<__half>(p, dst_dtype, s);
    }
}
