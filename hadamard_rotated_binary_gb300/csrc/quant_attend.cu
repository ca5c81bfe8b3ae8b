// Attention of a batch's new tokens over their sequences in a 4-bit cache, one
// pass over the keys.
//
// out = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m), s_j = scale * q . k_j, with
// k and v the values that the codes stand for (see quant.cuh), a running maximum
// m and sum per row; exp(x) = 2^(x log2 e).
//
// A row is one query head of one token; the heads / kv_heads query heads that read
// a key head share a tile of 8 or 16 rows (tokens outermost), so a single token of
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
// Work: an item is (sequence, key head, tile of rows) and costs its steps of keys
// and one more.  All items lie end to end on one line, which is cut into equal parts,
// one for each of the CTAs that run at once; so a long context splits over all SMs
// and ragged batches balance, with no length known on the host.  In a CTA's part of
// an item the eight warps take tiles of 16 or 32 keys in turn, each with its own ring
// of copies in flight, maximum, sum and output, and meet only at its end.  A CTA that
// has only a part of an item leaves its unnormalised output with the rows' references
// and sums in the workspace; the last of the item's CTAs to do so joins the parts
// in their order (results do not depend on which one is last).
//
// Weights are relative to 2^7 of the running reference, which follows a row's
// maximum only when that grows by more than 2^8: f16 holds them up to 2^15, and what
// its smallest step loses is 2^-32 of the largest weight.  They are rounded to f16 for
// a 16-bit output and split in two f16 digits (22 bits) for an f32 one.
#include <math.h>

#include "kv_internal.cuh"
#include "ptx.cuh"
#include "quant.cuh"

using namespace bitlin_impl;

namespace {

constexpr int kMaxLen = 1 << 30;
constexpr int kItemExtra = 1;     // steps that an item's begin and end cost
constexpr float kShift = 7.f;     // log2 of the largest weight when its reference is set
constexpr float kLazy = 8.f;      // log2 of the growth that another reference waits for
constexpr int kSlotFloats = 4096; // of a part's output in the workspace: rows x dim
constexpr int kSlotRows = 64;
constexpr int kJoin = 8;          // groups of parts come in multiples of this many
constexpr int kBatch = 4;         // parts in flight while they are joined

template <int D, int NT>
struct Cfg {
    // Warps of a CTA, so that two CTAs on an SM leave a thread the registers it needs.
    static constexpr int kWarps = D == 64 ? 8 : D == 256 && NT == 2 ? 8 : 6;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int KT = 32;                          // keys of a warp's tile
    static constexpr int kStep = kWarps * KT;              // keys of a CTA's step
    static constexpr int kRows = 8 * NT;
    static constexpr int kRow = D / 2;                     // bytes of a head's codes
    static constexpr int kCodes = KT * kRow;
    static constexpr int kSlot = kCodes + KT * 4;          // a tile's K or V, and its scales
    static constexpr int kLead = D == 256 ? 1 : 2;         // tiles that copies run ahead
    static constexpr int kSlots = 2 * kLead + 1;
    static constexpr int kRing = kWarps * kSlots * kSlot;
    static constexpr int kQ = NT * (D / 32) * 512;
    static constexpr int kMerge = kWarps * 8 * D * 4;      // eight rows of every warp, over the ring
    static constexpr int kBytes = (kRing > kMerge ? kRing : kMerge) + kQ;
    static constexpr int kBlocks = D == 256 && NT == 2 ? 1 : 2;  // CTAs on an SM
    static_assert(kRows * D <= kSlotFloats && kRows <= kSlotRows, "workspace");
};

struct Seq {
    int row0, tokens;  // its token rows
    int place0;        // place of the first
    int len;           // keys held
    int tiles, steps;  // row tiles, steps of keys
};

template <int STEP, int ROWS>
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
    q.tiles = (int)(((long long)q.tokens * p.group + ROWS - 1) / ROWS);
    q.steps = max(1, (q.len + STEP - 1) / STEP);
    return q;
}

// Where this CTA's part of the line begins and how long it is.
struct Start {
    long long per;    // length of a part; the first `extra` CTAs have one more
    long long extra;
    long long begin, length;
    long long skip;   // from the beginning of sequence `seq` to the part
    int seq;
};

__device__ __forceinline__ int cta_of(const Start& s, long long x)
{
    const long long longer = s.extra * (s.per + 1);
    return (int)(x < longer ? x / (s.per + 1) : s.extra + (x - longer) / s.per);
}

// One warp.
template <int STEP, int ROWS>
__device__ void locate(const QuantAttendParams& p, Start* out)
{
    const int lane = threadIdx.x & 31, grid = (int)gridDim.x, me = (int)blockIdx.x;
    auto cost = [&](int s) -> long long {
        if (s >= p.batch.seqs) return 0;
        const Seq q = load_seq<STEP, ROWS>(p, s);
        return (long long)q.tiles * p.pool.kv_heads * (q.steps + kItemExtra);
    };
    long long total = 0;
    for (int base = 0; base < p.batch.seqs; base += 32) total += cost(base + lane);
#pragma unroll
    for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    Start s;
    s.per = total / grid;
    s.extra = total - s.per * grid;
    s.begin = s.per * me + min((long long)me, s.extra);
    s.length = s.per + (me < s.extra);
    s.skip = 0;
    s.seq = p.batch.seqs;
    long long before = 0;
    for (int base = 0; base < p.batch.seqs && s.length > 0; base += 32) {
        const long long mine = cost(base + lane);
        long long upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += u;
        }
        const unsigned past = __ballot_sync(0xffffffffu, before + upto > s.begin);
        if (past) {
            const int l = __ffs(past) - 1;
            s.seq = base + l;
            s.skip = s.begin - (before + __shfl_sync(0xffffffffu, upto - mine, l));
            break;
        }
        before += __shfl_sync(0xffffffffu, upto, 31);
    }
    if (lane == 0) *out = s;
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

template <int D, int NT, int DIGITS>
__global__ void __launch_bounds__(Cfg<D, NT>::kThreads, Cfg<D, NT>::kBlocks) bitlin_quant_attend(const QuantAttendParams p)
{
    using C = Cfg<D, NT>;
    constexpr int kWarps = C::kWarps, kThreads = C::kThreads;
    constexpr int KT = C::KT, SUBS = KT / 16, KW = D / 32, VW = D / 64, MT = D / 16;
    constexpr int CPR = D / 32, COPIES = KT * CPR / 32;  // 16-byte chunks of a key, and copies of a lane
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ Start start;
    __shared__ float factor[C::kRows];
    __shared__ float2 warp_ml[kWarps][C::kRows];  // references and sums of the warps
    __shared__ float warp_weight[kWarps][C::kRows];
    __shared__ float2 row_ml[C::kRows];           // and of all of them
    __shared__ int last;
    unsigned char* ring = smem;
    uint4* qf = reinterpret_cast<uint4*>(smem + (C::kBytes - C::kQ));
    float* merge = reinterpret_cast<float*>(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;

    ptx::griddep_wait();
    if (warp == 0) locate<C::kStep, C::kRows>(p, &start);
    __syncthreads();
    long long left = start.length, skip = start.skip;
    if (left <= 0) return;
    long long line = start.begin - start.skip;  // where the current item begins
    int seq = start.seq;
    Seq w = load_seq<C::kStep, C::kRows>(p, seq);
    int cost = w.steps + kItemExtra;
    int item = (int)(skip / cost);
    line += (long long)item * cost;
    int from_step = (int)(skip - (long long)item * cost);
    unsigned char* my_ring = ring + warp * C::kSlots * C::kSlot;
    const uint32_t my_ring_s = ptx::smem_u32(my_ring);
    // Where this lane's copies of a tile go: chunk x of keys row, row + 32 / CPR, ...
    const int copy_row = lane / CPR, copy_x = lane & (CPR - 1);
    const uint32_t k_to = k_at<D>(copy_row, copy_x), v_to = v_at<D>(copy_row, copy_x);
    const bool one_page = p.pool.page_size % KT == 0;  // a tile lies in one page
    const long long copy_stride = (32 / CPR) * p.pool.slot_stride;
    const uint32_t magic = p.magic;
    auto page_index = [&](int key) { return p.page_shift >= 0 ? key >> p.page_shift : key / p.pool.page_size; };

    for (; left > 0; from_step = 0, line += cost, ++item) {
        while (item >= w.tiles * p.pool.kv_heads) {  // the next sequence with rows
            item = 0;
            w = load_seq<C::kStep, C::kRows>(p, ++seq);
            cost = w.steps + kItemExtra;
        }
        const int to_step = (int)min((long long)cost, from_step + left);
        left -= to_step - from_step;
        const int j0 = max(from_step - kItemExtra, 0), j1 = to_step - kItemExtra;
        if (j1 <= j0) continue;  // its begin alone: nothing to do
        const bool whole = j0 == 0 && j1 == w.steps;
        const int head = item / w.tiles, row0 = (item - head * w.tiles) * C::kRows;
        const int rows = min(C::kRows, w.tokens * p.group - row0);
        auto limit = [&](int row) {  // keys that a row sees
            return p.causal ? min(max(w.place0 + (row0 + row) / p.group + 1, 0), w.len) : w.len;
        };
        const int end = limit(rows - 1), lim_first = limit(0);
        const int first = (j0 * kWarps + warp) * KT;  // this warp's first key
        const int stop = min(end, j1 * C::kStep);
        const int n = stop > first ? (stop - first + C::kStep - 1) / C::kStep : 0;  // and its tiles

        __syncthreads();  // (the ring and the queries of the item before are through)

        // ---- copies: K and V of a tile one after the other through the ring
        const int32_t* table = p.batch.table + seq * p.batch.table_stride;
        const long long lane_at = head * p.pool.head_stride + (one_page ? copy_row * p.pool.slot_stride + 16 * copy_x : 0);
        const long long lane_scale = head * p.pool.scale_head + (one_page ? lane * p.pool.scale_slot : 0);
        auto page_of = [&](int i) {  // the table's entry for this lane's key of tile i
            const int key = first + i * C::kStep + (one_page ? 0 : lane);
            return i < n && key < end ? __ldg(table + page_index(key)) : -2;
        };
        // Of the tile in issue: its first key's codes and scales (this lane's part of them) or, where
        // a tile may span pages, this lane's key's; -1: zeros.
        long long at = 0, scale_at = 0;
        auto aim = [&](int i, int page) {
            const int key = first + i * C::kStep + (one_page ? 0 : lane);
            const bool inside = page >= 0 && page < p.pool.pages;
            if (page != -2 && !inside) *p.index_error = 1;
            const int slot = p.page_shift >= 0 ? key & (p.pool.page_size - 1) : key % p.pool.page_size;
            at = page * p.pool.page_stride + slot * p.pool.slot_stride + lane_at;
            scale_at = page * p.pool.scale_page + slot * p.pool.scale_slot + lane_scale;
            if (!inside) at = scale_at = -1;
        };
        auto issue = [&](int i, int kind, int slot) {
            if (i < n) {
                const uint32_t to = my_ring_s + slot * C::kSlot, dst = to + (kind ? v_to : k_to), turned = kind && D == 256 ? dst ^ 64 : dst;
                const int held = end - (first + i * C::kStep);  // keys of the tile
                // (v_at turns by bits 1 and 2 of the key, of which D == 256 changes one here)
                auto to_of = [&](int j) { return (j & 1 ? turned : dst) + j * (32 / CPR) * C::kRow; };
                if (one_page) {
                    const uint8_t* from = p.pool.codes[kind] + (at < 0 ? 0 : at);
                    const int rows_held = at < 0 ? 0 : held;
#pragma unroll
                    for (int j = 0; j < COPIES; ++j) {
                        const bool mine = copy_row + j * (32 / CPR) < rows_held;
                        ptx::cp_async16(to_of(j), mine ? from : p.pool.codes[kind], mine ? 16 : 0);
                        from += copy_stride;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < COPIES; ++j) {
                        const long long off = __shfl_sync(0xffffffffu, at, copy_row + j * (32 / CPR));
                        ptx::cp_async16(to_of(j), p.pool.codes[kind] + (off < 0 ? 0 : off + 16 * copy_x), off < 0 ? 0 : 16);
                    }
                }
                const bool mine = scale_at >= 0 && lane < held;
                ptx::cp_async4(to + C::kCodes + 4 * lane, p.pool.scales[kind] + (mine ? scale_at : 0), mine ? 4 : 0);
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
        for (int q = warp; q < C::kRows; q += kWarps) {
            constexpr int E = D / 32;
            float x[E], top = 0.f;
            const int row = row0 + q, token = row / p.group;
            const uint16_t* from = static_cast<const uint16_t*>(p.q) + (long long)(w.row0 + token) * p.q_token +
                                   (head * p.group + row - token * p.group) * p.q_head;
#pragma unroll
            for (int j = 0; j < E; ++j) {
                x[j] = q < rows ? half_word(from[lane * E + j], p.bf16) : 0.f;
                top = fmaxf(top, fabsf(x[j]));
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            int by = 0;
            if (top > 0.f && top < INFINITY) {
                frexpf(top, &by);
                by = min(15 - by, 120);
            }
            const float up = ldexpf(1.f, by);
            if (lane == 0) factor[q] = p.scale * 1.4426950408889634f * ldexpf(1.f, -by);
            __half* to = reinterpret_cast<__half*>(qf + (q / 8) * KW * 32);
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const int d = lane * E + j, quarter = d / (D / 4), in = d - quarter * (D / 4), i = in & 7;
                to[((in >> 3) * 32 + (q & 7) * 4 + quarter) * 8 + (i < 4 ? 2 * i : 2 * i - 7)] = __float2half_rn(x[j] * up);
            }
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
            float s[SUBS][NT][4] = {};
            {
                const unsigned char* stage = my_ring + slot * C::kSlot;
                const uint32_t* scales = reinterpret_cast<const uint32_t*>(stage + C::kCodes);
#pragma unroll
                for (int b = 0; b < SUBS; ++b) {
                    QuantScale2 q2[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) q2[k] = quant_scale2(__byte_perm(scales[16 * b + 8 * k + r], 0, 0x4040 + 0x0101 * c));
                    constexpr int H = KW < 4 ? KW : 4;  // words at a time
#pragma unroll
                    for (int h = 0; h < KW / H; ++h) {
                        uint32_t word[2][H];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const int key = 16 * b + 8 * k + r;
                            if (KW == 2) {
                                const uint2 x = *reinterpret_cast<const uint2*>(stage + key * C::kRow + 8 * c);
                                word[k][0] = x.x;
                                word[k][1] = x.y;
                            } else {
                                const uint4 x = *reinterpret_cast<const uint4*>(stage + k_at<D>(key, c * (KW / 4) + h));
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
                                ptx::mma_f16(s[b][t], u(a[0][0]), u(a[1][0]), u(a[0][1]), u(a[1][1]), q.x, q.y);
                                ptx::mma_f16(s[b][t], u(a[0][2]), u(a[1][2]), u(a[0][3]), u(a[1][3]), q.z, q.w);
                            }
                        }
                    }
                }
            }

            // weights
            bool ask = false;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int b = 0; b < SUBS; ++b) s[b][t][k] *= sl2[t][k & 1];
            if (key0 + KT > lim_first) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int lim = min(limit(8 * t + 2 * c + k), end) - key0 - r;
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
                        const float x = ptx::ex2(s[b][t][2 * k] - base[t][0]), y = ptx::ex2(s[b][t][2 * k + 1] - base[t][1]);
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
            const uint32_t* scales = reinterpret_cast<const uint32_t*>(stage + C::kCodes);
            slot = next(slot);
#pragma unroll
            for (int b = 0; b < SUBS; ++b) {
                QuantScale2 q2[2];
                uint32_t word[2][2][VW];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int key = 16 * b + 8 * k + 2 * c;
                    const uint2 two = *reinterpret_cast<const uint2*>(scales + key);
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
                            for (int t = 0; t < NT; ++t)
#pragma unroll
                                for (int g = 0; g < DIGITS; ++g)
                                    ptx::mma_f16(acc[4 * x + 2 * h + d][t], u(a[0][2 * d]), u(a[0][2 * d + 1]), u(a[1][2 * d]), u(a[1][2 * d + 1]),
                                                 pf[b][t][g][0], pf[b][t][g][1]);
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
            return reinterpret_cast<float2*>(merge) + (who * 8 + q) * (D / 2) + (i ^ ((i / MT ^ (q >> 1 << 2)) & (MT - 1)));
        };
        const int from = cta_of(start, line + kItemExtra), parts = cta_of(start, line + kItemExtra + w.steps - 1) - from + 1;
        float2* ws_ml = reinterpret_cast<float2*>(p.ws_ml);
        // the first part lies in its CTA's second slot, the others in their first
        auto slot_of = [&](int k) { return 2LL * (from + k) + (k == 0 ? 1 : 0); };
        const long long my_slot = slot_of((int)blockIdx.x - from);
        auto weight = [](float2 x, float ref) { return x.y == 0.f ? 0.f : ptx::ex2(x.x - ref); };  // (a sum of zero: no key)
        auto write_lse = [&](int row, float2 ml) {
            const int at = row0 + row, token = at / p.group;
            p.lse[(long long)(w.row0 + token) * p.heads + head * p.group + at - token * p.group] =
                ml.y == 0.f ? -INFINITY : 0.6931471805599453f * (ml.x + log2f(ml.y));
        };
        auto out_at = [&](int row) {
            const int at = row0 + row, token = at / p.group;
            return (long long)(w.row0 + token) * p.out_token + (head * p.group + at - token * p.group) * p.out_head;
        };
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
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if (8 * t >= rows) break;
            if (t) __syncthreads();
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int k = 0; k < 2; ++k) *merge_at(warp, 2 * c + k, r * MT + i) = make_float2(acc[i][t][k], acc[i][t][k + 2]);
            __syncthreads();
            for (int at = threadIdx.x; at < 8 * (D / 2); at += kThreads) {
                const int q = at / (D / 2), i = at - q * (D / 2), row = 8 * t + q;
                if (row >= rows) break;
                float2 o = make_float2(0.f, 0.f);
#pragma unroll
                for (int k = 0; k < kWarps; ++k) {
                    const float2 v = *merge_at(k, q, i);
                    const float f = warp_weight[k][row];
                    o.x = fmaf(f, v.x, o.x);
                    o.y = fmaf(f, v.y, o.y);
                }
                const float2 ml = row_ml[row];
                if (whole) {
                    const float inv = ml.y == 0.f ? 0.f : 1.f / ml.y;
                    const long long to = out_at(row) + 2 * i;
                    if (DIGITS > 1) *reinterpret_cast<float2*>(static_cast<float*>(p.out) + to) = make_float2(o.x * inv, o.y * inv);
                    else *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + to) = half_words(o.x * inv, o.y * inv, p.bf16);
                    if (p.lse && i == 0) write_lse(row, ml);
                } else {
                    __stcg(reinterpret_cast<float2*>(p.ws_o + my_slot * kSlotFloats + row * D) + i, o);
                    if (i == 0) __stcg(ws_ml + my_slot * kSlotRows + row, ml);
                }
            }
        }
        if (whole) continue;

        // ---- a part of an item: the last CTA to arrive joins them.  Many parts are joined
        // in groups first, by the last CTA of each group, so that no CTA reads them all.
        const int group = parts <= 2 * kJoin ? parts : (int)(sqrtf((float)parts) / kJoin + 1.f) * kJoin;
        const int groups = (parts + group - 1) / group, mine = ((int)blockIdx.x - from) / group;
        for (int level = groups > 1 ? 0 : 1; level < 2; ++level) {
            const int head_part = level ? 0 : mine * group;                                  // the first of those that are joined here,
            const int count = level ? groups : min(group, parts - head_part), each = level && groups > 1 ? group : 1;  // how many, how far apart
            const int joined = level && groups == 1 ? parts : count;
            if (joined > 1) {
                __syncthreads();
                if (threadIdx.x == 0) {
                    // (carries what the other threads wrote before they met, and brings
                    // what the other CTAs' threads wrote before theirs).  A group of several
                    // begins at a CTA that lies inside this item, an item at its own first.
                    int* ticket = p.tickets + level * (int)gridDim.x + from + head_part;
                    last = ptx::atom_add_acq_rel(ticket, 1) == joined - 1;
                    if (last) *ticket = 0;
                }
                __syncthreads();
                if (!last) break;
                for (int row = warp; row < rows; row += kWarps) {
                    constexpr int V = D == 256 ? 2 : 1;  // 16 bytes of a lane and part
                    const bool busy = D >= 128 || lane < 16;
                    const int k0 = lane;
                    float2 x = make_float2(0.f, 0.f);
                    if (k0 < joined) x = __ldcg(ws_ml + slot_of(head_part + k0 * each) * kSlotRows + row);
                    float ref = x.y == 0.f ? -INFINITY : x.x;
#pragma unroll
                    for (int o = 16; o; o >>= 1) ref = fmaxf(ref, __shfl_xor_sync(0xffffffffu, ref, o));
                    if (ref == -INFINITY) ref = 0.f;
                    const float f = weight(x, ref);
                    float total = f * x.y;
#pragma unroll
                    for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
                    float4 o[V] = {};
                    for (int k = 0; k < joined; k += kBatch) {
                        float4 v[kBatch][V];
#pragma unroll
                        for (int j = 0; j < kBatch; ++j)
#pragma unroll
                            for (int e = 0; e < V; ++e)
                                if (k + j < joined && busy)
                                    v[j][e] = __ldcg(reinterpret_cast<const float4*>(p.ws_o + slot_of(head_part + (k + j) * each) * kSlotFloats + row * D) + lane + 32 * e);
#pragma unroll
                        for (int j = 0; j < kBatch; ++j) {
                            const float g = __shfl_sync(0xffffffffu, f, (k + j) & 31);
                            if (k + j < joined && busy) {
#pragma unroll
                                for (int e = 0; e < V; ++e)
                                    o[e] = make_float4(fmaf(g, v[j][e].x, o[e].x), fmaf(g, v[j][e].y, o[e].y), fmaf(g, v[j][e].z, o[e].z),
                                                       fmaf(g, v[j][e].w, o[e].w));
                            }
                        }
                    }
                    if (level == 0) {
                        float* to = p.ws_o + slot_of(head_part) * kSlotFloats + row * D;
                        __syncwarp();
#pragma unroll
                        for (int e = 0; e < V; ++e)
                            if (busy) __stcg(reinterpret_cast<float4*>(to) + lane + 32 * e, o[e]);
                        if (lane == 0) __stcg(ws_ml + slot_of(head_part) * kSlotRows + row, make_float2(ref, total));
                    } else {
                        const float inv = total == 0.f ? 0.f : 1.f / total;
                        const long long to = out_at(row) + 4 * lane;
#pragma unroll
                        for (int e = 0; e < V; ++e) {
                            const float4 y = make_float4(o[e].x * inv, o[e].y * inv, o[e].z * inv, o[e].w * inv);
                            if (!busy) continue;
                            if (DIGITS > 1) *reinterpret_cast<float4*>(static_cast<float*>(p.out) + to + 128 * e) = y;
                            else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + to + 128 * e) =
                                make_uint2(half_words(y.x, y.y, p.bf16), half_words(y.z, y.w, p.bf16));
                        }
                        if (p.lse && lane == 0) write_lse(row, make_float2(ref, total));
                    }
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

template <int NT, int DIGITS>
cudaError_t pick_dim(const QuantAttendParams& p, int num_sms, cudaStream_t s)
{
    switch (p.pool.dim) {
    case 64: return launch<64, NT, DIGITS>(p, num_sms, s);
    case 128: return launch<128, NT, DIGITS>(p, num_sms, s);
    default: return launch<256, NT, DIGITS>(p, num_sms, s);
    }
}

template <int DIGITS>
cudaError_t pick_rows(const QuantAttendParams& p, int num_sms, cudaStream_t s)
{
    // A sequence's rows on average, as far as the host knows them.
    const bool few = (long long)p.tokens * p.group <= 8LL * p.batch.seqs;
    return few ? pick_dim<1, DIGITS>(p, num_sms, s) : pick_dim<2, DIGITS>(p, num_sms, s);
}

template <int D>
cudaError_t load_all()
{
    cudaError_t e = load<D, 1, 1>();
    if (e == cudaSuccess) e = load<D, 2, 1>();
    if (e == cudaSuccess) e = load<D, 1, 2>();
    if (e == cudaSuccess) e = load<D, 2, 2>();
    return e;
}

constexpr int kMostBlocks = 2;  // CTAs on an SM

}  // namespace

KvWorkspaceParts bitlin_quant_attend_workspace(int num_sms)
{
    const size_t slots = (size_t)2 * kMostBlocks * num_sms;
    KvWorkspaceParts w;
    w.timed_out = 2 * kMostBlocks * num_sms * sizeof(int);  // (no kernel here waits)
    w.ml = (w.timed_out + sizeof(int) + 255) / 256 * 256;
    w.o = w.ml + slots * kSlotRows * 2 * sizeof(float);
    w.bytes = w.o + slots * kSlotFloats * sizeof(float);
    return w;
}

cudaError_t bitlin_quant_attend_load(int dim)
{
    return dim == 64 ? load_all<64>() : dim == 128 ? load_all<128>() : load_all<256>();
}

cudaError_t bitlin_launch_quant_attend(const QuantAttendParams& p, int out_dtype, int num_sms, cudaStream_t s)
{
    return out_dtype == BITLIN_F32 ? pick_rows<2>(p, num_sms, s) : pick_rows<1>(p, num_sms, s);
}
