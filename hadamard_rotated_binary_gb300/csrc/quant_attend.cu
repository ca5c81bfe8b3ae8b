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

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxLen = 1 << 30;
constexpr int kItemExtra = 1;     // steps that an item's begin and end cost
constexpr float kShift = 7.f;     // log2 of the largest weight when its reference is set
constexpr float kLazy = 8.f;      // log2 of the growth that another reference waits for
constexpr int kSlotFloats = 4096; // of a part's output in the workspace: rows x dim
constexpr int kSlotRows = 64;

template <int D, int NT>
struct Cfg {
    static constexpr int KT = D == 256 ? 16 : 32;          // keys of a warp's tile
    static constexpr int kStep = kWarps * KT;              // keys of a CTA's step
    static constexpr int kRows = 8 * NT;
    static constexpr int kRow = D / 2;                     // bytes of a head's codes
    static constexpr int kCodes = KT * kRow;
    static constexpr int kStage = 2 * kCodes + 2 * KT * 4;  // K, V, their scales
    static constexpr int kStages = 3;
    static constexpr int kRing = kWarps * kStages * kStage;
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

template <int D, int NT, typename T, bool F32OUT>
__global__ void __launch_bounds__(kThreads, Cfg<D, NT>::kBlocks) bitlin_quant_attend(const QuantAttendParams p)
{
    using C = Cfg<D, NT>;
    constexpr int KT = C::KT, SUBS = KT / 16, KW = D / 32, VW = D / 64, MT = D / 16;
    constexpr int DIGITS = F32OUT ? 2 : 1;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ Start start;
    __shared__ float factor[C::kRows];
    __shared__ float2 warp_ml[kWarps][C::kRows];  // references and sums of the warps
    __shared__ float joined_ref[8], joined_sum[8];
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
    unsigned char* my_ring = ring + warp * C::kStages * C::kStage;
    const uint32_t my_ring_s = ptx::smem_u32(my_ring);

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

        // ---- queries: a power of two brings a row's largest magnitude to 2^14 .. 2^15
        __syncthreads();  // (the ring and the queries of the item before are through)
        for (int n = warp; n < C::kRows; n += kWarps) {
            constexpr int E = D / 32;
            float x[E], top = 0.f;
            const int row = row0 + n, token = row / p.group;
            const T* q = static_cast<const T*>(p.q) + (long long)(w.row0 + token) * p.q_token + (head * p.group + row - token * p.group) * p.q_head;
#pragma unroll
            for (int j = 0; j < E; ++j) {
                x[j] = n < rows ? to_f32(q[lane * E + j]) : 0.f;
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
            if (lane == 0) factor[n] = p.scale * 1.4426950408889634f * ldexpf(1.f, -by);
            __half* to = reinterpret_cast<__half*>(qf + (n / 8) * KW * 32);
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const int d = lane * E + j, quarter = d / (D / 4), at = d - quarter * (D / 4), i = at & 7;
                to[((at >> 3) * 32 + (n & 7) * 4 + quarter) * 8 + (i < 4 ? 2 * i : 2 * i - 7)] = __float2half_rn(x[j] * up);
            }
        }
        __syncthreads();

        // ---- this warp's tiles of the part
        const int first = (j0 * kWarps + warp) * KT;
        const int stop = min(end, j1 * C::kStep);
        const int n = stop > first ? (stop - first + C::kStep - 1) / C::kStep : 0;
        float sl2[NT][2];
        int lim[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int row = 8 * t + 2 * c + k;
                sl2[t][k] = factor[row];
                lim[t][k] = row < rows ? limit(row) : end;
            }
        const int32_t* table = p.batch.table + seq * p.batch.table_stride;
        const int my_key = lane & (KT - 1);
        auto page_of = [&](int i) {  // the table's entry for this lane's key of tile i
            const int key = first + i * C::kStep + my_key;
            return i < n && key < end ? __ldg(table + key / p.pool.page_size) : -2;
        };
        auto issue = [&](int i, int page) {
            if (i < n) {
                const int key = first + i * C::kStep + my_key;
                const bool inside = page >= 0 && page < p.pool.pages;
                if (page != -2 && !inside) *p.index_error = 1;
                const int slot = key % p.pool.page_size;
                const long long at = inside ? page * p.pool.page_stride + slot * p.pool.slot_stride + head * p.pool.head_stride : -1;
                const long long scale_at = inside ? page * p.pool.scale_page + slot * p.pool.scale_slot + head * p.pool.scale_head : 0;
                const uint32_t stage = my_ring_s + (i % C::kStages) * C::kStage;
                constexpr int CPR = D / 32;  // 16-byte chunks of a key
                const int x = lane & (CPR - 1);
#pragma unroll
                for (int j = 0; j < KT * CPR / 32; ++j) {
                    const int row = lane / CPR + j * (32 / CPR);
                    const long long from = __shfl_sync(0xffffffffu, at, row);
                    const int valid = from >= 0 ? 16 : 0;
                    const long long off = valid ? from + 16 * x : 0;
                    ptx::cp_async16(stage + k_at<D>(row, x), p.pool.codes[0] + off, valid);
                    ptx::cp_async16(stage + C::kCodes + v_at<D>(row, x), p.pool.codes[1] + off, valid);
                }
                if (lane < KT) {
                    ptx::cp_async4(stage + 2 * C::kCodes + 4 * lane, p.pool.scales[0] + scale_at, inside ? 4 : 0);
                    ptx::cp_async4(stage + 2 * C::kCodes + 4 * (KT + lane), p.pool.scales[1] + scale_at, inside ? 4 : 0);
                }
            }
            ptx::cp_async_commit();
        };
        {
            int pages[C::kStages - 1];
#pragma unroll
            for (int i = 0; i < C::kStages - 1; ++i) pages[i] = page_of(i);
#pragma unroll
            for (int i = 0; i < C::kStages - 1; ++i) issue(i, pages[i]);
        }
        int next_page = page_of(C::kStages - 1);

        float acc[MT][NT][4] = {};
        float m[NT][2], base[NT][2] = {}, sum[NT][2] = {};
#pragma unroll
        for (int t = 0; t < NT; ++t) m[t][0] = m[t][1] = -INFINITY;

        for (int i = 0; i < n; ++i) {
            __syncwarp();  // (all lanes are through with the stage that is filled next)
            issue(i + C::kStages - 1, next_page);
            next_page = page_of(i + C::kStages);
            ptx::cp_async_wait<C::kStages - 1>();
            __syncwarp();
            const unsigned char* stage = my_ring + (i % C::kStages) * C::kStage;
            const uint32_t* k_scale = reinterpret_cast<const uint32_t*>(stage + 2 * C::kCodes);
            const uint32_t* v_scale = k_scale + KT;
            const int key0 = first + i * C::kStep;

            // S = K Q^T, keys down, queries across
            float s[SUBS][NT][4] = {};
#pragma unroll
            for (int b = 0; b < SUBS; ++b) {
                QuantScale2 q2[2];
                uint32_t word[2][KW];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int key = 16 * b + 8 * k + r;
                    q2[k] = quant_scale2((k_scale[key] >> (8 * c) & 0xff) * 0x00010001u);
                    if (KW == 2) {
                        const uint2 x = *reinterpret_cast<const uint2*>(stage + key * C::kRow + 8 * c);
                        word[k][0] = x.x;
                        word[k][1] = x.y;
                    } else {
#pragma unroll
                        for (int h = 0; h < KW / 4; ++h) {
                            const uint4 x = *reinterpret_cast<const uint4*>(stage + k_at<D>(key, c * (KW / 4) + h));
                            word[k][4 * h] = x.x;
                            word[k][4 * h + 1] = x.y;
                            word[k][4 * h + 2] = x.z;
                            word[k][4 * h + 3] = x.w;
                        }
                    }
                }
#pragma unroll
                for (int x = 0; x < KW; ++x) {
                    __half2 a[2][4];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        a[k][0] = quant_low(word[k][x], q2[k]);
                        a[k][1] = quant_high(word[k][x], q2[k]);
                        a[k][2] = quant_low(word[k][x] >> 8, q2[k]);
                        a[k][3] = quant_high(word[k][x] >> 8, q2[k]);
                    }
                    auto u = [](const __half2& v) { return *reinterpret_cast<const uint32_t*>(&v); };
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        const uint4 q = qf[(t * KW + x) * 32 + lane];
                        ptx::mma_f16(s[b][t], u(a[0][0]), u(a[1][0]), u(a[0][1]), u(a[1][1]), q.x, q.y);
                        ptx::mma_f16(s[b][t], u(a[0][2]), u(a[1][2]), u(a[0][3]), u(a[1][3]), q.z, q.w);
                    }
                }
            }

            // weights
            bool ask = false;
#pragma unroll
            for (int b = 0; b < SUBS; ++b)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int k = 0; k < 4; ++k) s[b][t][k] *= sl2[t][k & 1];
            if (key0 + KT > lim_first) {
#pragma unroll
                for (int b = 0; b < SUBS; ++b)
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (key0 + 16 * b + 8 * (k >> 1) + r >= lim[t][k & 1]) s[b][t][k] = -INFINITY;
            }
#pragma unroll
            for (int b = 0; b < SUBS; ++b)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int k = 0; k < 4; ++k) ask |= s[b][t][k] > m[t][k & 1] + kLazy;
            if (__any_sync(0xffffffffu, ask)) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float top = -INFINITY;
#pragma unroll
                        for (int b = 0; b < SUBS; ++b) top = fmaxf(top, fmaxf(s[b][t][k], s[b][t][k + 2]));
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                        if (top > m[t][k] + kLazy) {  // the row's own growth alone: rows do not change one another
                            const float keep = m[t][k] == -INFINITY ? 0.f : ptx::ex2(m[t][k] - top);
                            m[t][k] = top;
                            base[t][k] = top - kShift;
                            sum[t][k] *= keep;
#pragma unroll
                            for (int i = 0; i < MT; ++i) {
                                acc[i][t][k] *= keep;
                                acc[i][t][k + 2] *= keep;
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
                        pf[b][t][0][k] = ptx::transposed(*reinterpret_cast<const uint32_t*>(&hi));
                        if (DIGITS > 1) {
                            const float2 f = __half22float2(hi);
                            const __half2 lo = __floats2half2_rn(x - f.x, y - f.y);
                            pf[b][t][DIGITS - 1][k] = ptx::transposed(*reinterpret_cast<const uint32_t*>(&lo));
                        }
                    }

            // O += V^T P^T, dimensions down, queries across
#pragma unroll
            for (int b = 0; b < SUBS; ++b) {
                QuantScale2 q2[2];
                uint32_t word[2][2][VW];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int key = 16 * b + 8 * k + 2 * c;
                    const uint32_t by = 8 * (r >> 1);
                    q2[k] = quant_scale2((v_scale[key] >> by & 0xff) | (v_scale[key + 1] >> by & 0xff) << 16);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const unsigned char* codes = stage + C::kCodes;
                        if (VW == 1) {
                            word[k][e][0] = *reinterpret_cast<const uint32_t*>(codes + v_at<D>(key + e, r >> 2) + (r & 3) * 4);
                        } else if (VW == 2) {
                            const uint2 x = *reinterpret_cast<const uint2*>(codes + v_at<D>(key + e, r >> 1) + (r & 1) * 8);
                            word[k][e][0] = x.x;
                            word[k][e][1] = x.y;
                        } else {
                            const uint4 x = *reinterpret_cast<const uint4*>(codes + v_at<D>(key + e, r));
                            word[k][e][0] = x.x;
                            word[k][e][1] = x.y;
                            word[k][e][VW - 2] = x.z;
                            word[k][e][VW - 1] = x.w;
                        }
                    }
                }
#pragma unroll
                for (int x = 0; x < VW; ++x) {
                    __half2 a[2][8];  // the word's eight dimensions, for two keys each
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t both = __byte_perm(word[k][0][x], word[k][1][x], h ? 0x7632 : 0x5410);
                            a[k][4 * h] = quant_low(both, q2[k]);
                            a[k][4 * h + 1] = quant_high(both, q2[k]);
                            a[k][4 * h + 2] = quant_low(both >> 8, q2[k]);
                            a[k][4 * h + 3] = quant_high(both >> 8, q2[k]);
                        }
                    }
                    auto u = [](const __half2& v) { return *reinterpret_cast<const uint32_t*>(&v); };
#pragma unroll
                    for (int d = 0; d < 4; ++d)
#pragma unroll
                        for (int t = 0; t < NT; ++t)
#pragma unroll
                            for (int g = 0; g < DIGITS; ++g)
                                ptx::mma_f16(acc[4 * x + d][t], u(a[0][2 * d]), u(a[0][2 * d + 1]), u(a[1][2 * d]), u(a[1][2 * d + 1]),
                                             pf[b][t][g][0], pf[b][t][g][1]);
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

        // (row q of eight, dimensions 2 i and 2 i + 1) of a warp's or part's output in shared memory
        auto merge_at = [&](int who, int q, int i) {
            const int lane_r = i / MT;
            return reinterpret_cast<float2*>(merge) + (who * 8 + q) * (D / 2) + (i ^ ((lane_r ^ (q >> 1 << 2)) & (MT - 1)));
        };
        const int from = cta_of(start, line + kItemExtra), to = cta_of(start, line + kItemExtra + w.steps - 1), parts = to - from + 1;
        const long long slot = 2LL * blockIdx.x + ((int)blockIdx.x == from ? 1 : 0);
        float2* ws_ml = reinterpret_cast<float2*>(p.ws_ml);
        auto weight = [](float2 x, float ref) { return x.y == 0.f ? 0.f : ptx::ex2(x.x - ref); };
        auto write_out = [&](int row, int i, float2 v) {
            const int at = row0 + row, token = at / p.group;
            const long long o = (long long)(w.row0 + token) * p.out_token + (head * p.group + at - token * p.group) * p.out_head + 2 * i;
            if (F32OUT) {
                *reinterpret_cast<float2*>(static_cast<float*>(p.out) + o) = v;
            } else {
                T* out = static_cast<T*>(p.out) + o;
                out[0] = from_f32<T>(v.x);
                out[1] = from_f32<T>(v.y);
            }
        };
        auto write_lse = [&](int row, float ref, float total) {
            const int at = row0 + row, token = at / p.group;
            p.lse[(long long)(w.row0 + token) * p.heads + head * p.group + at - token * p.group] =
                total == 0.f ? -INFINITY : 0.6931471805599453f * (ref + log2f(total));
        };
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
                float ref = -INFINITY, total = 0.f;
#pragma unroll
                for (int k = 0; k < kWarps; ++k)
                    if (warp_ml[k][row].y != 0.f) ref = fmaxf(ref, warp_ml[k][row].x);
                if (ref == -INFINITY) ref = 0.f;
                float2 o = make_float2(0.f, 0.f);
#pragma unroll
                for (int k = 0; k < kWarps; ++k) {
                    const float2 x = warp_ml[k][row];
                    const float f = weight(x, ref);
                    const float2 v = *merge_at(k, q, i);
                    total = fmaf(f, x.y, total);
                    o.x = fmaf(f, v.x, o.x);
                    o.y = fmaf(f, v.y, o.y);
                }
                if (whole) {
                    const float inv = total == 0.f ? 0.f : 1.f / total;
                    write_out(row, i, make_float2(o.x * inv, o.y * inv));
                    if (p.lse && i == 0) write_lse(row, ref, total);
                } else {
                    __stcg(reinterpret_cast<float2*>(p.ws_o + slot * kSlotFloats + row * D) + i, o);
                    if (i == 0) __stcg(ws_ml + slot * kSlotRows + row, make_float2(ref, total));
                }
            }
        }
        if (whole) continue;

        // ---- a part of an item: the last CTA to arrive joins them
        __syncthreads();
        if (threadIdx.x == 0) {
            // (carries what the other threads wrote before they met, and brings
            // what the other CTAs' threads wrote before theirs)
            last = ptx::atom_add_acq_rel(&p.tickets[from], 1) == parts - 1;
            if (last) p.tickets[from] = 0;
        }
        __syncthreads();
        if (!last) continue;
        // the first part lies in its CTA's second slot, the others in their first
        auto slot_of = [&](int k) { return 2LL * (from + k) + (k == 0 ? 1 : 0); };
        for (int t = 0; t < NT; ++t) {
            if (8 * t >= rows) break;
            if (t) __syncthreads();
            const int mine = 8 * t + warp;  // a warp finds a row's reference and sum
            if (mine < rows) {
                float ref = -INFINITY, total = 0.f;
                for (int k = lane; k < parts; k += 32) {
                    const float2 x = __ldcg(ws_ml + slot_of(k) * kSlotRows + mine);
                    if (x.y != 0.f) ref = fmaxf(ref, x.x);
                }
#pragma unroll
                for (int o = 16; o; o >>= 1) ref = fmaxf(ref, __shfl_xor_sync(0xffffffffu, ref, o));
                if (ref == -INFINITY) ref = 0.f;
                for (int k = lane; k < parts; k += 32) {
                    const float2 x = __ldcg(ws_ml + slot_of(k) * kSlotRows + mine);
                    total = fmaf(weight(x, ref), x.y, total);
                }
#pragma unroll
                for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
                if (lane == 0) {
                    joined_ref[warp] = ref;
                    joined_sum[warp] = total;
                    if (p.lse) write_lse(mine, ref, total);
                }
            }
            __syncthreads();
            // a warp adds every eighth part, then the warps' sums are added
            constexpr int PER = D / 64;  // float2 of a lane and row
            float2 o[8][PER] = {};
            for (int k = warp; k < parts; k += kWarps) {
                float2 x[8][PER];
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    if (8 * t + q < rows) {
#pragma unroll
                        for (int e = 0; e < PER; ++e)
                            x[q][e] = __ldcg(reinterpret_cast<const float2*>(p.ws_o + slot_of(k) * kSlotFloats + (8 * t + q) * D) + lane + 32 * e);
                    }
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    if (8 * t + q < rows) {
                        const float f = weight(__ldcg(ws_ml + slot_of(k) * kSlotRows + 8 * t + q), joined_ref[q]);
#pragma unroll
                        for (int e = 0; e < PER; ++e) {
                            o[q][e].x = fmaf(f, x[q][e].x, o[q][e].x);
                            o[q][e].y = fmaf(f, x[q][e].y, o[q][e].y);
                        }
                    }
            }
#pragma unroll
            for (int q = 0; q < 8; ++q)
#pragma unroll
                for (int e = 0; e < PER; ++e) *merge_at(warp, q, lane + 32 * e) = o[q][e];
            __syncthreads();
            for (int at = threadIdx.x; at < 8 * (D / 2); at += kThreads) {
                const int q = at / (D / 2), i = at - q * (D / 2), row = 8 * t + q;
                if (row >= rows) break;
                float2 v = make_float2(0.f, 0.f);
#pragma unroll
                for (int k = 0; k < kWarps; ++k) {
                    const float2 x = *merge_at(k, q, i);
                    v.x += x.x;
                    v.y += x.y;
                }
                const float inv = joined_sum[q] == 0.f ? 0.f : 1.f / joined_sum[q];
                write_out(row, i, make_float2(v.x * inv, v.y * inv));
            }
        }
    }
}

template <int D, int NT, typename T, bool F32OUT>
cudaError_t load()
{
    static PerDeviceOnce once;
    int dev = 0;
    return once.run(&dev, [](int) {
        return cudaFuncSetAttribute(bitlin_quant_attend<D, NT, T, F32OUT>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D, NT>::kBytes);
    });
}

template <int D, int NT, typename T, bool F32OUT>
cudaError_t launch(const QuantAttendParams& p, int num_sms, cudaStream_t s)
{
    const cudaError_t e = load<D, NT, T, F32OUT>();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(num_sms * Cfg<D, NT>::kBlocks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Cfg<D, NT>::kBytes;
    cfg.stream = s;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, bitlin_quant_attend<D, NT, T, F32OUT>, p);
}

template <int NT, typename T, bool F32OUT>
cudaError_t pick_dim(const QuantAttendParams& p, int num_sms, cudaStream_t s)
{
    switch (p.pool.dim) {
    case 64: return launch<64, NT, T, F32OUT>(p, num_sms, s);
    case 128: return launch<128, NT, T, F32OUT>(p, num_sms, s);
    default: return launch<256, NT, T, F32OUT>(p, num_sms, s);
    }
}

template <typename T, bool F32OUT>
cudaError_t pick_rows(const QuantAttendParams& p, int num_sms, cudaStream_t s)
{
    // A sequence's rows on average, as far as the host knows them.
    const bool few = (long long)p.tokens * p.group <= 8LL * p.batch.seqs;
    return few ? pick_dim<1, T, F32OUT>(p, num_sms, s) : pick_dim<2, T, F32OUT>(p, num_sms, s);
}

template <int D, typename T>
cudaError_t load_all()
{
    cudaError_t e = load<D, 1, T, false>();
    if (e == cudaSuccess) e = load<D, 2, T, false>();
    if (e == cudaSuccess) e = load<D, 1, T, true>();
    if (e == cudaSuccess) e = load<D, 2, T, true>();
    return e;
}

template <typename T>
cudaError_t load_dim(int dim)
{
    return dim == 64 ? load_all<64, T>() : dim == 128 ? load_all<128, T>() : load_all<256, T>();
}

constexpr int kMostBlocks = 2;  // CTAs on an SM

}  // namespace

KvWorkspaceParts bitlin_quant_attend_workspace(int num_sms)
{
    const size_t slots = (size_t)2 * kMostBlocks * num_sms;
    KvWorkspaceParts w;
    w.timed_out = kMostBlocks * num_sms * sizeof(int);  // (no kernel here waits)
    w.ml = (w.timed_out + sizeof(int) + 255) / 256 * 256;
    w.o = w.ml + slots * kSlotRows * 2 * sizeof(float);
    w.bytes = w.o + slots * kSlotFloats * sizeof(float);
    return w;
}

cudaError_t bitlin_quant_attend_load(int dim, int dtype)
{
    return dtype == BITLIN_BF16 ? load_dim<__nv_bfloat16>(dim) : load_dim<__half>(dim);
}

cudaError_t bitlin_launch_quant_attend(const QuantAttendParams& p, int dtype, int out_dtype, int num_sms, cudaStream_t s)
{
    if (dtype == BITLIN_BF16)
        return out_dtype == BITLIN_F32 ? pick_rows<__nv_bfloat16, true>(p, num_sms, s) : pick_rows<__nv_bfloat16, false>(p, num_sms, s);
    return out_dtype == BITLIN_F32 ? pick_rows<__half, true>(p, num_sms, s) : pick_rows<__half, false>(p, num_sms, s);
}
