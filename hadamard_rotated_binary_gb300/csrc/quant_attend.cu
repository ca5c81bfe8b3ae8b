// Attention of a batch's new tokens over their sequences in a 4-bit cache, one
// pass over the keys.
//
// out = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m), s_j = scale * q . k_j, with
// k and v the values that the codes stand for (see quant.cuh), a running maximum
// m and sum per row; exp(x) = 2^(x log2 e).
//
// A row is one query head of one token; the heads / kv_heads query heads that read
// a key head share a tile of 8, 16 or 24 rows (tokens outermost), so a single token of
// a grouped model reads each key once.
//
// Codes become f16 in registers, where they are the A operand of 16 x 8 x 16
// products: keys (for Q K^T) or dimensions (for P V) are the 16 rows of A and the
// queries the 8 columns of B.  A single token's few rows would leave most of a
// tensor-memory tile empty, and values that shared memory held in 16 bits would
// have to be written and read there at four times the codes' bytes; from registers
// the codes cross shared memory once.  Nibbles are taken from a word by masks (the
// order of a product's inner dimension is free: queries lie in the same order), and
// one fused multiply-add makes two values of them.  In P V the inner dimension is
// the keys: words of two keys are joined halfword by halfword first.
//
// Work: an item is (sequence, key head, tile of rows) and costs its steps of keys (a
// tile of 32 for each warp of a CTA) and some more.  All items lie end to end on one
// line, which is cut into equal parts, one for each of the CTAs that run at once; so a
// long context splits over all SMs and ragged batches balance, with no length known on
// the host.  In a CTA's part of an item the warps take tiles in turn, each with its own
// ring of copies in flight, maximum, sum and output, and meet only at its end.  A CTA that
// has only a part of an item leaves its unnormalised output with the rows' references
// and sums in the workspace; the last of the item's CTAs to be through joins the parts
// in their order (results do not depend on which one is last).
//
// Weights are relative to 2^7 of the running reference, which follows a row's
// maximum only when that grows by more than 2^8: f16 holds them up to 2^15, and what
// its smallest step loses is 2^-32 of the largest weight.  They are rounded to f16 for
// a 16-bit output and split in two f16 digits (22 bits) for an f32 one.  The products'
// additions truncate (3.4e-8 of an output per addition of positive values, measured), so
// an f32 output is added outside them, rounded: off by 1e-7 to 8e-7 of its norm from
// 2,000 to 131,072 keys an item, where f32 arithmetic in torch is by 1e-7 to 1.1e-6, for
// 5 us in 76 (64 tokens over 100-8,000 keys).
//
// Bound: HBM, and the issue of the codes' conversion beside it (at 256 dims some 1,200
// instructions of a warp for 32 keys, 620 of them masks, shifts, permutations and
// fused multiply-adds of the codes).  The loop over the keys moves 5.7 TB/s at 256 dims;
// an item's begin takes 2 us and its end 1.5, which the other CTA on the SM covers in
// part, a call's begin 4 us and its last join 4.  Measured (GB300, inputs changing from
// call to call): one token over 131,072 keys, 138 MB, 45 us (f32 out); 64 over 100-8,000
// keys, 274 MB, 70 us (3.9 TB/s; f32 out 80), with 8 heads of 128 dims (282 MB) 75 and of 64
// (149 MB) 52; one over 777 keys 11 us; 16 x 5 drafted tokens over 1,000-6,000 keys, 128 dims,
// 43 us, 256 dims 53; single tokens over 262,000 keys in all 68 us as 64 sequences, 78 as 256,
// 133 as 1,000 and 379 as 4,000 (more ends of items, and each CTA goes through all sequences to
// find its part; how much each takes was not measured).
#include <math.h>

#include "kv_internal.cuh"
#include "ptx.cuh"
#include "quant.cuh"

using namespace bitlin_impl;

namespace {

constexpr int kMaxLen = 1 << 30;
constexpr int KT = 32;            // keys of a tile
constexpr float kShift = 7.f;     // log2 of the largest weight when its reference is set
constexpr float kLazy = 8.f;      // log2 of the growth that another reference waits for

template <int D, int NT>
struct Cfg {
    // Warps of a CTA and CTAs on an SM, so that a thread has nearly the registers it needs: what
    // spills (bytes stored) is 156 at 256 dims and 16 rows, 52 at 256 dims, 8 rows and an f32 output,
    // 28 at most elsewhere.
    static constexpr int kOutputs = D / 32 * NT * 8;       // a thread's part of the output, in registers
    static constexpr int kBlocks = kOutputs > 64 ? 1 : 2;
    static constexpr int kWarps = kOutputs == 48 || kOutputs == 64 ? 6 : 8;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kRows = 8 * NT;
    static constexpr int kRow = D / 2;                     // bytes of a head's codes
    static constexpr int kCodes = KT * kRow;
    static constexpr int kSlot = kCodes + KT * 4;          // a tile's K or V, and its scales
    static constexpr int kLead = D == 256 ? 1 : 2;  // tiles that copies run ahead
    static constexpr int kSlots = 2 * kLead + 1;
    static constexpr int kRing = kSlots * kSlot;
    static constexpr int kQ = NT * (D / 32) * 512;
    static constexpr int kStep = kWarps * KT;              // keys of a step
    // Steps that an item's begin and end cost.  Measured, in us, 64 tokens over 100-8,000 keys, at 1/2/3:
    // 256 dims 69.0/69.4/70.6, 128 dims 81.0/73.7/74.7, 64 dims 62.1/54.6/52.0.
    static constexpr int kExtra = D == 256 ? 1 : D == 128 ? 2 : 3;
    // Eight rows of every warp, over the rings: float2s, with a gap after each lane's dimensions and rows
    // so far apart that the stores of 16 lanes (4 lanes' dimensions of 4 rows) meet no bank twice.
    static constexpr int kMergeRow = D / 2 + 8 + 10;
    static constexpr int kMerge = kWarps * 8 * kMergeRow * 8;
    static constexpr int kBytes = (kWarps * kRing > kMerge ? kWarps * kRing : kMerge) + kQ;
    static constexpr int kPart = kRows * D;                // floats of a part's output in the workspace
};

struct Seq {
    int row0, tokens;  // its token rows
    int place0;        // place of the first
    int len;           // keys held
    int tiles, steps;  // tiles of rows, steps of keys
};

template <class C>
__device__ __forceinline__ Seq load_seq(const QuantAttendParams& p, int s)
{
    Seq q;
    const int lo = p.batch.q_offsets[s], hi = p.batch.q_offsets[s + 1];
    const int raw = min(max(p.batch.kv_lens[s], 0), kMaxLen);
    const long long cap = (long long)p.batch.table_pages * p.pool.page_size;
    q.row0 = min(max(lo, 0), p.tokens);
    q.tokens = min(max(hi, q.row0), p.tokens) - q.row0;
    q.place0 = raw - (min(max(hi, 0), kMaxLen) - q.row0);
    q.len = raw < cap ? raw : (int)cap;
    if (q.len < raw && q.tokens) *p.index_error = 1;
    q.tiles = (int)(((long long)q.tokens * p.group + C::kRows - 1) / C::kRows);
    q.steps = max(1, (q.len + C::kStep - 1) / C::kStep);
    return q;
}

// What a CTA has of the line, and the item that it works on; in shared memory, so that
// the loop over the keys does not hold it in registers.
struct Work {
    long long per, extra;  // length of a CTA's part; the first `extra` CTAs have one more
    long long left;        // of this CTA's part
    long long line;        // where the item begins on the line
    Seq w;
    int seq, item, cost, from, to;
    int head, row0, rows;
    int j0, j1;            // steps of the part
    int end, lim_first;    // keys that the item's last row sees, and its first
    bool some, whole;      // whether there is a part, and whether it is all of the item
};

// x / n for n > 0; the sizes at hand nearly always fit 32 bits.
__device__ __forceinline__ long long divide(long long x, long long n)
{
    return ((x | n) >> 32) == 0 ? (long long)((uint32_t)x / (uint32_t)n) : x / n;
}

// The CTA whose part of the line holds x.
__device__ __forceinline__ int cta_of(const Work& s, long long x)
{
    const long long longer = s.extra * (s.per + 1);
    return (int)(x < longer ? divide(x, s.per + 1) : s.extra + divide(x - longer, s.per));
}

// Keys that a row of the item sees.
__device__ __forceinline__ int limit(const QuantAttendParams& p, const Work& k, int row)
{
    return p.causal ? min(max(k.w.place0 + (k.row0 + row) / p.group + 1, 0), k.w.len) : k.w.len;
}

// Cost of all items of a sequence (0 past the last one).
template <class C>
__device__ __forceinline__ long long seq_cost(const QuantAttendParams& p, int s)
{
    if (s >= p.batch.seqs) return 0;
    const Seq q = load_seq<C>(p, s);
    return (long long)q.tiles * p.pool.kv_heads * (q.steps + C::kExtra);
}

// One warp: where this CTA's part of the line begins.
template <class C>
__device__ void locate(const QuantAttendParams& p, Work* out)
{
    const int lane = threadIdx.x & 31, ctas = (int)gridDim.x, me = (int)blockIdx.x;
    long long total = 0, mine = 0;
    for (int base = 0; base < p.batch.seqs; base += 32) total += mine = seq_cost<C>(p, base + lane);
#pragma unroll
    for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    const long long per = divide(total, ctas), extra = total - per * ctas;
    const long long begin = per * me + min((long long)me, extra), left = per + (me < extra);
    long long before = 0, skip = 0;
    int seq = p.batch.seqs;
    for (int base = 0; base < p.batch.seqs && left > 0; base += 32) {
        if (p.batch.seqs > 32) mine = seq_cost<C>(p, base + lane);
        long long upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += u;
        }
        const unsigned past = __ballot_sync(0xffffffffu, before + upto > begin);
        if (past) {
            const int l = __ffs(past) - 1;
            seq = base + l;
            skip = begin - (before + __shfl_sync(0xffffffffu, upto - mine, l));
            break;
        }
        before += __shfl_sync(0xffffffffu, upto, 31);
    }
    if (lane != 0) return;
    Work k = {};
    k.per = per;
    k.extra = extra;
    k.left = left;
    k.seq = seq;
    if (left > 0) {
        k.w = load_seq<C>(p, seq);
        k.cost = k.w.steps + C::kExtra;
        k.item = (int)divide(skip, k.cost);
        k.from = (int)(skip - (long long)k.item * k.cost);
        k.line = begin - k.from;
    }
    k.item -= 1;  // what next_item moves on from
    k.line -= k.cost;
    *out = k;
}

// One thread: the next item of this CTA's part, if there is one.
template <class C>
__device__ void next_item(const QuantAttendParams& p, Work* out)
{
    Work k = *out;
    k.some = false;
    while (k.left > 0 && !k.some) {
        k.item += 1;
        k.line += k.cost;
        while (k.item >= k.w.tiles * p.pool.kv_heads) {  // the next sequence with rows
            k.item = 0;
            k.w = load_seq<C>(p, ++k.seq);
            k.cost = k.w.steps + C::kExtra;
        }
        k.to = (int)min((long long)k.cost, k.from + k.left);
        k.left -= k.to - k.from;
        k.j0 = max(k.from - C::kExtra, 0);
        k.j1 = k.to - C::kExtra;
        k.from = 0;
        k.some = k.j1 > k.j0;  // (else its begin alone: nothing to do)
    }
    if (k.some) {
        k.whole = k.j0 == 0 && k.j1 == k.w.steps;
        k.head = k.item / k.w.tiles;
        k.row0 = (k.item - k.head * k.w.tiles) * C::kRows;
        k.rows = min(C::kRows, k.w.tokens * p.group - k.row0);
        k.end = limit(p, k, k.rows - 1);
        k.lim_first = limit(p, k, 0);
    }
    *out = k;
}

// A 16-bit value of the call's type, and two of them.
__device__ __forceinline__ float half_word(uint16_t x, int bf16)
{
    return bf16 ? __uint_as_float((uint32_t)x << 16) : __half2float(__ushort_as_half(x));
}
__device__ __forceinline__ uint32_t half_words(float x, float y, int bf16)
{
    if (bf16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
    const __half2 v = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// Bytes from the start of a warp's K (or V) tile to 16-byte chunk x of a key's
// codes, placed so that the lanes' reads meet no bank twice: 8 lanes read 2 keys'
// quarters of K, or of V eighths of 4 keys that are two apart.
template <int D>
__device__ __forceinline__ int k_at(int key, int x)
{
    return key * (D / 2) + ((D == 256 ? x ^ (key & 1) : x) << 4);
}
template <int D>
__device__ __forceinline__ int v_at(int key, int x)
{
    const int at = key * (D / 2) + (x << 4);
    const int turn = D == 64 ? (key & 4) >> 1 : key & 6;
    return at ^ (turn << 4);
}

// The CTA that does the item's first step, and the one that does its last.
__device__ __forceinline__ int first_cta(const Work& k) { return cta_of(k, k.line + k.cost - k.w.steps); }
__device__ __forceinline__ int last_cta(const Work& k) { return cta_of(k, k.line + k.cost - 1); }
// Where part k of an item that begins at CTA `from` lies in the workspace: the first
// in its CTA's second slot, the others in their first.
__device__ __forceinline__ long long part_slot(int from, int k) { return 2LL * (from + k) + (k == 0 ? 1 : 0); }

// Parts of an item that a CTA reads at once, of `all`: so many groups of so many.
__device__ __forceinline__ int group_of(int all) { return all <= 16 ? all : 8 * ((int)(sqrtf((float)all) * 0.125f) + 1); }

// An item of which a CTA has a part.
struct Shared {
    int first, last;  // its CTAs; first = -1: there is none
    int token, head, row0, rows;
};

__device__ __forceinline__ float weight(float2 x, float ref) { return x.y == 0.f ? 0.f : ptx::ex2(x.x - ref); }  // (a sum of zero: no key)

// The token row and the head of a row of a tile.
struct Place {
    long long token;
    int head;
};
__device__ __forceinline__ Place place_of(const QuantAttendParams& p, int first_token, int head, int at)
{
    const int token = at / p.group;
    return {first_token + token, head * p.group + at - token * p.group};
}

// Four elements of a row's output from element d on.
template <int DIGITS>
__device__ __forceinline__ void write_four(const QuantAttendParams& p, Place at, int d, float4 x)
{
    const long long to = at.token * p.out_token + at.head * p.out_head + d;
    if (DIGITS > 1) *reinterpret_cast<float4*>(static_cast<float*>(p.out) + to) = x;
    else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + to) = make_uint2(half_words(x.x, x.y, p.bf16), half_words(x.z, x.w, p.bf16));
}
__device__ __forceinline__ void write_lse(const QuantAttendParams& p, Place at, float2 ml)
{
    p.lse[at.token * p.heads + at.head] = ml.y == 0.f ? -INFINITY : 0.6931471805599453f * (ml.x + log2f(ml.y));
}

template <int D, int NT, int DIGITS>
__global__ void __launch_bounds__(Cfg<D, NT>::kThreads, Cfg<D, NT>::kBlocks) bitlin_quant_attend(const __grid_constant__ QuantAttendParams p)
{
    using C = Cfg<D, NT>;
    constexpr int SUBS = KT / 16, KW = D / 32, VW = D / 64, MT = D / 16;
    constexpr int CPR = D / 32, COPIES = KT * CPR / 32;  // 16-byte chunks of a key, and copies of a lane
    extern __shared__ __align__(128) unsigned char smem[];
    constexpr int kWarps = C::kWarps;
    __shared__ Work work;
    __shared__ float factor[C::kRows];
    __shared__ float2 warp_ml[kWarps][C::kRows];  // references and sums of the warps
    __shared__ float warp_weight[kWarps][C::kRows];
    __shared__ float2 row_ml[C::kRows];           // and of all of them
    __shared__ Shared shared[2];                  // the items that began in an earlier CTA, and go on in the next
    __shared__ int joins[2], count_of[2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    unsigned char* my_ring = smem + warp * C::kRing;
    uint4* qf = reinterpret_cast<uint4*>(smem + (C::kBytes - C::kQ));
    const uint32_t my_ring_s = ptx::smem_u32(my_ring);

    ptx::griddep_wait();
    if (warp == 0) locate<C>(p, &work);
    if (threadIdx.x < 2) shared[threadIdx.x].first = -1;
    // Where this lane's copies of a tile go: chunk x of keys row, row + 32 / CPR, ...
    const int copy_row = lane / CPR, copy_x = lane & (CPR - 1);
    const uint32_t k_to = k_at<D>(copy_row, copy_x), v_to = v_at<D>(copy_row, copy_x);
    const uint32_t magic = p.magic;

    for (;;) {
        if (threadIdx.x == 0) next_item<C>(p, &work);
        __syncthreads();  // (and the ring and the queries of the item before are through)
        if (!work.some) break;
        const int head = work.head, end = work.end, lim_first = work.lim_first;
        const int first = (work.j0 * kWarps + warp) * KT;  // this warp's first key
        const int stop = min(end, work.j1 * C::kStep);
        const int n = stop > first ? (stop - first + C::kStep - 1) / C::kStep : 0;  // and its tiles

        // this warp's queries are on their way first: eight elements to a lane
        constexpr int LPR = D / 8, RPS = 32 / LPR, SETS = C::kRows / RPS, QS = (SETS + kWarps - 1) / kWarps;  // lanes of a row, rows of a set, sets, of a warp
        const int q_row = lane / LPR, q_unit = lane & (LPR - 1);
        uint4 raw[QS];
        {
            const int token0 = work.row0 / p.group, in_group = work.row0 - token0 * p.group;
            const uint16_t* from = static_cast<const uint16_t*>(p.q) + (long long)(work.w.row0 + token0) * p.q_token + head * p.group * p.q_head + 8 * q_unit;
#pragma unroll
            for (int j = 0; j < QS; ++j) {
                const int q = (warp + j * kWarps) * RPS + q_row, at = in_group + q, token = (at * p.group_inverse) >> 16;
                raw[j] = make_uint4(0, 0, 0, 0);
                if (q < work.rows) raw[j] = *reinterpret_cast<const uint4*>(from + token * p.q_token + (at - token * p.group) * p.q_head);
            }
        }

        // ---- copies: K and V of a tile one after the other through the ring.  A lane looks up one key;
        // where its codes and scale lie, in units of the pools' strides, goes round by shuffles.  Keys that
        // are not there get scales of zero and whatever codes lie at the pool's begin: values of zero.
        const int32_t* table = p.batch.table + work.seq * p.batch.table_stride;
        auto page_of = [&](int i) {  // the table's entry for this lane's key of tile i
            const int key = first + i * C::kStep + lane;
            return i < n && key < end ? __ldg(table + (p.page_shift >= 0 ? key >> p.page_shift : key / p.pool.page_size)) : -1;
        };
        uint32_t at = 0, scale_at = 0;  // of this lane's key of the tile in issue
        bool held = false;
        auto aim = [&](int i, int page) {
            const int key = first + i * C::kStep + lane;
            held = page >= 0 && page < p.pool.pages;
            if (!held && i < n && key < end) *p.index_error = 1;
            const int slot = p.page_shift >= 0 ? key & (p.pool.page_size - 1) : key % p.pool.page_size;
            at = held ? page * p.page_units + slot * p.slot_units + head * p.head_units : 0;
            scale_at = held ? page * p.scale_page_units + slot * p.scale_slot_units + head * p.scale_head_units : 0;
        };
        auto issue = [&](int i, int kind, int slot) {
            if (i < n) {
                const uint32_t to = my_ring_s + slot * C::kSlot, dst = to + (kind ? v_to : k_to), turned = kind && D == 256 ? dst ^ 64 : dst;
                const uint8_t* from = p.pool.codes[kind] + 16 * copy_x;
#pragma unroll
                for (int j = 0; j < COPIES; ++j)  // (v_at turns by bits 1 and 2 of the key, of which D == 256 changes one here)
                    ptx::cp_async16((j & 1 ? turned : dst) + j * (32 / CPR) * C::kRow,
                                    from + (uint64_t)__shfl_sync(0xffffffffu, at, copy_row + j * (32 / CPR)) * p.unit);
                ptx::cp_async4(to + C::kCodes + 4 * lane, p.pool.scales[kind] + (uint64_t)scale_at * p.scale_unit, held ? 4 : 0);
            }
            ptx::cp_async_commit();
        };
        int next_page;
        {
            int pages[C::kLead];
#pragma unroll
            for (int i = 0; i < C::kLead; ++i) pages[i] = page_of(i);
            next_page = page_of(C::kLead);
#pragma unroll
            for (int i = 0; i < C::kLead; ++i) {
                aim(i, pages[i]);
                issue(i, 0, 2 * i);
                issue(i, 1, 2 * i + 1);
            }
        }

        // ---- queries: a power of two brings a row's largest magnitude to 2^14 .. 2^15
#pragma unroll
        for (int j = 0; j < QS; ++j) {
            if (warp + j * kWarps >= SETS) break;
            const uint32_t words[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
            float x[8];
            int top = 0;  // magnitudes compare as integers; zero, infinity and NaN are left as they are
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[e] = half_word(words[e / 2] >> 16 * (e & 1), p.bf16);
                top = max(top, __float_as_int(fabsf(x[e])));
            }
            if (LPR == 32) {
                top = __reduce_max_sync(0xffffffffu, top);
            } else {
#pragma unroll
                for (int o = LPR / 2; o; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
            }
            const int by = top > 0 && top < 0x7f800000 ? min(14 + 127 - (top >> 23), 120) : 0;
            // a negative scale goes to the queries: products and scores then grow together
            const float up = copysignf(__int_as_float((127 + by) << 23), p.scale);
            const int q = (warp + j * kWarps) * RPS + q_row;
            if (q_unit == 0) factor[q] = fmaxf(fabsf(p.scale) * 1.4426950408889634f * __int_as_float((127 - by) << 23), 1e-36f);
            auto two = [&](int e) {
                const __half2 h = __floats2half2_rn(x[e] * up, x[e + 4] * up);
                return *reinterpret_cast<const uint32_t*>(&h);
            };
            qf[(q / 8 * KW + q_unit % (LPR / 4)) * 32 + (q & 7) * 4 + q_unit / (LPR / 4)] = make_uint4(two(0), two(1), two(2), two(3));
        }
        __syncthreads();

        // ---- this warp's tiles of the part
        float acc[MT][NT][4] = {};
        float base[NT][2], sum[NT][2] = {}, sl2[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                base[t][k] = -3e38f;  // far below any score: the first one is a growth
                sl2[t][k] = factor[8 * t + 2 * c + k];
            }
        auto u = [](const __half2& v) { return *reinterpret_cast<const uint32_t*>(&v); };
        int slot = 0;                        // of this tile's K
        int fill = 2 * C::kLead;             // of the next copies
        auto next = [](int x) { return x + 1 == C::kSlots ? 0 : x + 1; };
        for (int i = 0; i < n; ++i) {
            const int key0 = first + i * C::kStep;
            __syncwarp();  // (all lanes are through with the slot that is filled next)
            aim(i + C::kLead, next_page);
            issue(i + C::kLead, 0, fill);
            fill = next(fill);
            next_page = page_of(i + C::kLead + 1);
            ptx::cp_async_wait<C::kSlots - 1>();
            __syncwarp();

            // S = K Q^T, keys down, queries across
            float s[SUBS][NT][4];
            {
                const unsigned char* stage = my_ring + slot * C::kSlot;
                const uint32_t* scales = reinterpret_cast<const uint32_t*>(stage + C::kCodes) + r;
#pragma unroll
                for (int b = 0; b < SUBS; ++b, stage += 16 * C::kRow, scales += 16) {
                    float x0[NT][4] = {}, x1[NT][4] = {};  // two, so that a product does not wait for the one before
                    QuantScale2 q2[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) q2[k] = quant_scale2(__byte_perm(scales[8 * k], 0, 0x4040 + 0x0101 * c));
                    constexpr int H = KW < 4 ? KW : 4;  // words at a time
#pragma unroll
                    for (int h = 0; h < KW / H; ++h) {
                        uint32_t word[2][H];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            if (KW == 2) {
                                const uint2 x = *reinterpret_cast<const uint2*>(stage + (8 * k + r) * C::kRow + 8 * c);
                                word[k][0] = x.x;
                                word[k][1] = x.y;
                            } else {
                                const uint4 x = *reinterpret_cast<const uint4*>(stage + k_at<D>(8 * k + r, c * (KW / 4) + h));
                                word[k][0] = x.x;
                                word[k][1] = x.y;
                                word[k][H - 2] = x.z;
                                word[k][H - 1] = x.w;
                            }
                        }
#pragma unroll
                        for (int x = 0; x < H; ++x) {
                            __half2 a[2][4];
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                a[k][0] = quant_low(word[k][x], q2[k], magic);
                                a[k][1] = quant_high(word[k][x], q2[k], magic);
                                a[k][2] = quant_low(word[k][x] >> 8, q2[k], magic);
                                a[k][3] = quant_high(word[k][x] >> 8, q2[k], magic);
                            }
#pragma unroll
                            for (int t = 0; t < NT; ++t) {
                                const uint4 q = qf[(t * KW + h * H + x) * 32 + lane];
                                ptx::mma_f16(x0[t], u(a[0][0]), u(a[1][0]), u(a[0][1]), u(a[1][1]), q.x, q.y);
                                ptx::mma_f16(x1[t], u(a[0][2]), u(a[1][2]), u(a[0][3]), u(a[1][3]), q.z, q.w);
                            }
                        }
                    }
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float x = x0[t][k] + x1[t][k];
                            if (b == 0) s[0][t][k] = x;
                            else s[1][t][k] = x;
                        }
                }
            }

            // weights
            bool ask = false;
            if (key0 + KT > lim_first) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int lim = min(limit(p, work, 8 * t + 2 * c + k), end) - key0 - r;
#pragma unroll
                        for (int b = 0; b < SUBS; ++b) {
                            if (16 * b >= lim) s[b][t][k] = -INFINITY;
                            if (16 * b + 8 >= lim) s[b][t][k + 2] = -INFINITY;
                        }
                    }
            }
            float top[NT][2];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    top[t][k] = fmaxf(s[0][t][k], s[0][t][k + 2]);
#pragma unroll
                    for (int b = 1; b < SUBS; ++b) top[t][k] = fmaxf(top[t][k], fmaxf(s[b][t][k], s[b][t][k + 2]));
                    top[t][k] *= sl2[t][k];
                    ask |= top[t][k] > base[t][k] + (kShift + kLazy);
                }
            if (__any_sync(0xffffffffu, ask)) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) top[t][k] = fmaxf(top[t][k], __shfl_xor_sync(0xffffffffu, top[t][k], o));
                        if (top[t][k] > base[t][k] + (kShift + kLazy)) {  // the row's own growth alone: rows do not change one another
                            const float keep = ptx::ex2(base[t][k] - (top[t][k] - kShift));
                            base[t][k] = top[t][k] - kShift;
                            sum[t][k] *= keep;
#pragma unroll
                            for (int d = 0; d < MT; ++d) {
                                acc[d][t][k] *= keep;
                                acc[d][t][k + 2] *= keep;
                            }
                        }
                    }
            }
            uint32_t pf[SUBS][NT][DIGITS][2];
#pragma unroll
            for (int b = 0; b < SUBS; ++b)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float x = ptx::ex2(fmaf(s[b][t][2 * k], sl2[t][0], -base[t][0])), y = ptx::ex2(fmaf(s[b][t][2 * k + 1], sl2[t][1], -base[t][1]));
                        sum[t][0] += x;
                        sum[t][1] += y;
                        const __half2 hi = __floats2half2_rn(x, y);
                        pf[b][t][0][k] = ptx::transposed(u(hi));
                        if (DIGITS > 1) {
                            const float2 f = __half22float2(hi);
                            pf[b][t][DIGITS - 1][k] = ptx::transposed(u(__floats2half2_rn(x - f.x, y - f.y)));
                        }
                    }

            slot = next(slot);  // V
            __syncwarp();       // (all lanes are through with K)
            issue(i + C::kLead, 1, fill);
            fill = next(fill);
            ptx::cp_async_wait<C::kSlots - 1>();
            __syncwarp();

            // O += V^T P^T, dimensions down, queries across
            const unsigned char* stage = my_ring + slot * C::kSlot;
            const uint32_t* scales = reinterpret_cast<const uint32_t*>(stage + C::kCodes) + 2 * c;
            slot = next(slot);
#pragma unroll
            for (int b = 0; b < SUBS; ++b, stage += 16 * C::kRow, scales += 16) {
                QuantScale2 q2[2];
                uint32_t word[2][2][VW], pb[NT][DIGITS][2];
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int g = 0; g < DIGITS; ++g)
#pragma unroll
                        for (int k = 0; k < 2; ++k) pb[t][g][k] = b ? pf[1][t][g][k] : pf[0][t][g][k];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int key = 8 * k + 2 * c;
                    const uint2 two = *reinterpret_cast<const uint2*>(scales + 8 * k);
                    const uint32_t g = r >> 1;
                    q2[k] = quant_scale2(__byte_perm(two.x, two.y, g | (g + 4) << 8) & 0x00ff00ffu);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        if (VW == 1) {
                            word[k][e][0] = *reinterpret_cast<const uint32_t*>(stage + v_at<D>(key + e, r >> 2) + (r & 3) * 4);
                        } else if (VW == 2) {
                            const uint2 x = *reinterpret_cast<const uint2*>(stage + v_at<D>(key + e, r >> 1) + (r & 1) * 8);
                            word[k][e][0] = x.x;
                            word[k][e][1] = x.y;
                        } else {
                            const uint4 x = *reinterpret_cast<const uint4*>(stage + v_at<D>(key + e, r));
                            word[k][e][0] = x.x;
                            word[k][e][1] = x.y;
                            word[k][e][VW - 2] = x.z;
                            word[k][e][VW - 1] = x.w;
                        }
                    }
                }
#pragma unroll
                for (int x = 0; x < VW; ++x) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {  // four dimensions of the word's eight, for two keys each
                        __half2 a[2][4];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const uint32_t both = __byte_perm(word[k][0][x], word[k][1][x], h ? 0x7632 : 0x5410);
                            a[k][0] = quant_low(both, q2[k], magic);
                            a[k][1] = quant_high(both, q2[k], magic);
                            a[k][2] = quant_low(both >> 8, q2[k], magic);
                            a[k][3] = quant_high(both >> 8, q2[k], magic);
                        }
#pragma unroll
                        for (int d = 0; d < 2; ++d)
#pragma unroll
                            for (int t = 0; t < NT; ++t) {
                                float(&o)[4] = acc[4 * x + 2 * h + d][t];
                                if (DIGITS == 1) {
                                    ptx::mma_f16(o, u(a[0][2 * d]), u(a[0][2 * d + 1]), u(a[1][2 * d]), u(a[1][2 * d + 1]), pb[t][0][0], pb[t][0][1]);
                                } else {
                                    // (the products' additions truncate: these are rounded)
                                    float part[4] = {};
#pragma unroll
                                    for (int g = 0; g < DIGITS; ++g)
                                        ptx::mma_f16(part, u(a[0][2 * d]), u(a[0][2 * d + 1]), u(a[1][2 * d]), u(a[1][2 * d + 1]), pb[t][g][0], pb[t][g][1]);
#pragma unroll
                                    for (int k = 0; k < 4; ++k) o[k] += part[k];
                                }
                            }
                    }
                }
            }
        }
        ptx::cp_async_wait<0>();

        // ---- the warps' parts joined, eight rows at a time
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float x = sum[t][k];
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
                if (r == 0) warp_ml[warp][8 * t + 2 * c + k] = make_float2(base[t][k], x);
            }
        __syncthreads();  // the rings are through

        // (row q of eight, dimensions 2 i and 2 i + 1) of a warp's output in shared memory
        auto merge_at = [&](int who, int q, int i) {
            return reinterpret_cast<float2*>(smem) + (who * 8 + q) * C::kMergeRow + i + i / MT;
        };
        // after the last barrier below thread 0 may be at the next item, whose state takes this one's
        // place: what the joining needs of it is read here
        const int rows = work.rows, first_token = work.w.row0, tile_row0 = work.row0;
        const bool whole = work.whole;
        for (int row = warp; row < rows; row += kWarps) {
            const float2 x = lane < kWarps ? warp_ml[lane][row] : make_float2(0.f, 0.f);
            float ref = x.y == 0.f ? -INFINITY : x.x;
#pragma unroll
            for (int o = 4; o; o >>= 1) ref = fmaxf(ref, __shfl_xor_sync(0xffffffffu, ref, o));
            if (ref == -INFINITY) ref = 0.f;
            const float f = weight(x, ref);
            float total = f * x.y;
#pragma unroll
            for (int o = 4; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
            if (lane < kWarps) warp_weight[lane][row] = f;
            if (lane == 0) row_ml[row] = make_float2(ref, total);
        }
        const int from = first_cta(work);
        const long long slot_of_part = part_slot(from, (int)blockIdx.x - from);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if (8 * t >= rows) break;
            if (t) __syncthreads();
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) merge_at(warp, 2 * c + e, r * MT)[i] = make_float2(acc[i][t][e], acc[i][t][e + 2]);
            __syncthreads();
            // a warp takes a row, a lane four of its elements at a time
            for (int q = warp; q < 8 && 8 * t + q < rows; q += kWarps) {
                const int row = 8 * t + q;
                const float2 ml = row_ml[row];
                const float scale = !whole ? 1.f : ml.y == 0.f ? 0.f : 1.f / ml.y;
                const Place place = place_of(p, first_token, head, tile_row0 + row);
#pragma unroll
                for (int e = 0; e < (D + 127) / 128; ++e) {
                    const int d = 4 * (lane + 32 * e);
                    if (d >= D) break;
                    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int k = 0; k < kWarps; ++k) {
                        const float2* v = merge_at(k, q, d / 2);
                        const float2 x = v[0], y = v[1];
                        const float f = warp_weight[k][row];
                        o = make_float4(fmaf(f, x.x, o.x), fmaf(f, x.y, o.y), fmaf(f, y.x, o.z), fmaf(f, y.y, o.w));
                    }
                    o = make_float4(o.x * scale, o.y * scale, o.z * scale, o.w * scale);
                    if (whole) write_four<DIGITS>(p, place, d, o);
                    else __stcg(reinterpret_cast<float4*>(p.ws_o + slot_of_part * C::kPart + row * D + d), o);
                }
                if (lane == 0) {
                    if (!whole) __stcg(reinterpret_cast<float2*>(p.ws_ml) + slot_of_part * C::kRows + row, ml);
                    else if (p.lse) write_lse(p, place, ml);
                }
            }
        }
        if (!whole && threadIdx.x == 0) shared[from == (int)blockIdx.x] = {from, last_cta(work), first_token, head, tile_row0, rows};
    }

    // ---- items that CTAs share: the last one to come joins the parts.  Many parts are joined
    // in groups first, by the last CTA of each group, so that no CTA reads them all.
    constexpr int V = D == 256 ? 2 : 1;  // 16 bytes of a lane and part
    constexpr int kBatch = 8;            // parts in flight
    const bool busy = D >= 128 || lane < 16;
    bool alive[2] = {shared[0].first >= 0, shared[1].first >= 0};
#pragma unroll 1
    for (int level = 0; level < 2; ++level) {
        __syncthreads();
        if (threadIdx.x < 2) {
            const Shared item = shared[threadIdx.x];
            int mode = alive[threadIdx.x] ? 1 : 0;  // 0: no more to do, 1: goes on to the next level, 2: joins
            if (mode) {
                const int all = item.last - item.first + 1, group = group_of(all), groups = (all + group - 1) / group;
                const int first = level ? 0 : ((int)blockIdx.x - item.first) / group * group;
                const int count = !level ? min(group, all - first) : groups > 1 ? groups : all;
                if (level ? count > 1 : groups > 1 && count > 1) {
                    // (carries what the other threads wrote before they met, and brings
                    // what the other CTAs' threads wrote before theirs).  A group of several
                    // begins at a CTA that lies inside the item, an item at its own first.
                    int* ticket = p.tickets + level * (int)gridDim.x + item.first + first;
                    mode = ptx::atom_add_acq_rel(ticket, 1) == count - 1 ? 2 : 0;
                    if (mode) *ticket = 0;
                }
                count_of[threadIdx.x] = count;
            }
            joins[threadIdx.x] = mode;
        }
        __syncthreads();
#pragma unroll 1
        for (int which = 0; which < 2; ++which) {
            alive[which] = joins[which] != 0;
            if (joins[which] != 2) continue;
            const Shared item = shared[which];
            const int group = group_of(item.last - item.first + 1), count = count_of[which];
            const int first = level ? 0 : ((int)blockIdx.x - item.first) / group * group;
            const int each = level && item.last - item.first + 1 > group ? group : 1;  // how far the parts are apart
            auto slot_of = [&](int k) { return part_slot(item.first, first + k * each); };
#pragma unroll 1
            for (int row = warp; row < item.rows; row += kWarps) {
                float4 v[kBatch][V], o[V] = {};
                auto load = [&](int k) {
#pragma unroll
                    for (int j = 0; j < kBatch; ++j)
#pragma unroll
                        for (int e = 0; e < V; ++e)
                            if (k + j < count && busy) v[j][e] = __ldcg(reinterpret_cast<const float4*>(p.ws_o + slot_of(k + j) * C::kPart + row * D) + lane + 32 * e);
                };
                load(0);
                float2 x = make_float2(0.f, 0.f);
                if (lane < count) x = __ldcg(reinterpret_cast<const float2*>(p.ws_ml) + slot_of(lane) * C::kRows + row);
                float ref = x.y == 0.f ? -INFINITY : x.x;
#pragma unroll
                for (int s = 16; s; s >>= 1) ref = fmaxf(ref, __shfl_xor_sync(0xffffffffu, ref, s));
                if (ref == -INFINITY) ref = 0.f;
                const float f = weight(x, ref);
                float total = f * x.y;
#pragma unroll
                for (int s = 16; s; s >>= 1) total += __shfl_xor_sync(0xffffffffu, total, s);
#pragma unroll 1
                for (int k = 0; k < count; k += kBatch) {
                    if (k) load(k);
#pragma unroll
                    for (int j = 0; j < kBatch; ++j) {
                        const float g = __shfl_sync(0xffffffffu, f, (k + j) & 31);
                        if (k + j < count && busy) {
#pragma unroll
                            for (int e = 0; e < V; ++e)
                                o[e] = make_float4(fmaf(g, v[j][e].x, o[e].x), fmaf(g, v[j][e].y, o[e].y), fmaf(g, v[j][e].z, o[e].z),
                                                   fmaf(g, v[j][e].w, o[e].w));
                        }
                    }
                }
                const float scale = !level ? 1.f : total == 0.f ? 0.f : 1.f / total;
                const Place place = place_of(p, item.token, item.head, item.row0 + row);
                __syncwarp();
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float4 y = make_float4(o[e].x * scale, o[e].y * scale, o[e].z * scale, o[e].w * scale);
                    if (!busy) continue;
                    if (level) write_four<DIGITS>(p, place, 4 * (lane + 32 * e), y);
                    else __stcg(reinterpret_cast<float4*>(p.ws_o + slot_of(0) * C::kPart + row * D) + lane + 32 * e, y);
                }
                if (lane == 0) {
                    if (!level) __stcg(reinterpret_cast<float2*>(p.ws_ml) + slot_of(0) * C::kRows + row, make_float2(ref, total));
                    else if (p.lse) write_lse(p, place, make_float2(ref, total));
                }
            }
        }
    }
}

template <int D, int NT, int DIGITS>
cudaError_t load()
{
    static PerDeviceOnce once;
    int dev = 0;
    return once.run(&dev, [](int) {
        return cudaFuncSetAttribute(bitlin_quant_attend<D, NT, DIGITS>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D, NT>::kBytes);
    });
}

template <int D, int NT, int DIGITS>
cudaError_t launch(const QuantAttendParams& p, int num_sms, cudaStream_t s)
{
    const cudaError_t e = load<D, NT, DIGITS>();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(num_sms * Cfg<D, NT>::kBlocks);
    cfg.blockDim = dim3(Cfg<D, NT>::kThreads);
    cfg.dynamicSmemBytes = Cfg<D, NT>::kBytes;
    cfg.stream = s;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, bitlin_quant_attend<D, NT, DIGITS>, p);
}

// Tiles of 8 rows: by a sequence's rows on average, as far as the host knows them, up to
// what leaves a thread's part of the output in registers.  Measured, in us, 16 sequences
// of 1,000-6,000 keys with 5 tokens of 4 heads to a key head, 128 dims: 16 rows 51.3, 24 43.2.
template <int D, int DIGITS>
cudaError_t pick_rows(const QuantAttendParams& p, int num_sms, cudaStream_t s)
{
    constexpr int kMost = D == 256 ? 2 : 3;
    const long long rows = (long long)p.tokens * p.group, seqs = p.batch.seqs;
    if (rows <= 8 * seqs) return launch<D, 1, DIGITS>(p, num_sms, s);
    if (kMost == 2 || rows <= 16 * seqs) return launch<D, 2, DIGITS>(p, num_sms, s);
    return launch<D, kMost, DIGITS>(p, num_sms, s);
}

template <int DIGITS>
cudaError_t pick_dim(const QuantAttendParams& p, int num_sms, cudaStream_t s)
{
    switch (p.pool.dim) {
    case 64: return pick_rows<64, DIGITS>(p, num_sms, s);
    case 128: return pick_rows<128, DIGITS>(p, num_sms, s);
    default: return pick_rows<256, DIGITS>(p, num_sms, s);
    }
}

template <int D, int NT>
cudaError_t load_digits()
{
    const cudaError_t e = load<D, NT, 1>();
    return e == cudaSuccess ? load<D, NT, 2>() : e;
}

template <int D, int MOST>
cudaError_t load_all()
{
    cudaError_t e = load_digits<D, 1>();
    if (e == cudaSuccess) e = load_digits<D, 2>();
    if (e == cudaSuccess && MOST > 2) e = load_digits<D, MOST>();
    return e;
}

// The largest of all kernels' parts, two of a CTA, per SM.
template <int D, int NT>
constexpr size_t most_floats(size_t other)
{
    const size_t mine = (size_t)2 * Cfg<D, NT>::kBlocks * Cfg<D, NT>::kPart;
    return mine > other ? mine : other;
}
constexpr size_t kPartFloats =
    most_floats<64, 1>(most_floats<64, 2>(most_floats<64, 3>(most_floats<128, 1>(most_floats<128, 2>(most_floats<128, 3>(most_floats<256, 1>(most_floats<256, 2>(0))))))));
constexpr int kMostBlocks = 2, kMostRows = 24;

}  // namespace

// Tickets, zero between calls; then references and sums; then outputs.
KvWorkspaceParts bitlin_quant_attend_workspace(int num_sms)
{
    const size_t ctas = (size_t)kMostBlocks * num_sms;
    KvWorkspaceParts w;
    w.timed_out = 2 * ctas * sizeof(int);  // (no kernel here waits)
    w.ml = (w.timed_out + sizeof(int) + 255) / 256 * 256;
    w.o = (w.ml + 2 * ctas * kMostRows * 2 * sizeof(float) + 255) / 256 * 256;
    w.bytes = w.o + (size_t)num_sms * kPartFloats * sizeof(float);
    return w;
}

cudaError_t bitlin_quant_attend_load(int dim)
{
    return dim == 64 ? load_all<64, 3>() : dim == 128 ? load_all<128, 3>() : load_all<256, 2>();
}

cudaError_t bitlin_launch_quant_attend(const QuantAttendParams& p, int out_dtype, int num_sms, cudaStream_t s)
{
    return out_dtype == BITLIN_F32 ? pick_dim<2>(p, num_sms, s) : pick_dim<1>(p, num_sms, s);
}
