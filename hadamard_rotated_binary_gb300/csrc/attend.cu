// Attention of a batch's new tokens over their sequences in the paged cache,
// on the tensor cores, one pass over the keys.
//
// out = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m), s_j = scale * q . k_j,
// with a running maximum m and sum per row; exp(x) = 2^(x log2 e).
//
// Tile: 128 rows of S = Q K^T in tensor memory (one lane per row), 128 keys.
// A row is one query head of one token; the heads / kv_heads query heads that
// read a key head share its rows (tokens outermost), so a single token of a
// grouped model still reads each key once.
//
// Work: an item is (sequence, key head, tile of rows) and costs its visible
// key tiles and a few more for its begin and end.  All items lie end to end on
// one line of tiles, sequences outermost, then key heads.  Where the items cost about the same, the CTAs
// first take whole items in rounds, neighbours side by side: the CTAs on one
// key head then read the same keys at the same time and L2 serves all but the
// first.  (2,048 tokens over 32,768 keys, 134 MB of K and V: equal parts of the
// line alone read 4.8 GB from HBM.)  What is left of the line, or all of it, is
// cut into equal parts, so a long context splits over all SMs and ragged
// batches balance, with no length known on the host.  A CTA that has only a
// part of an item leaves its unnormalised output with the row's maximum and
// sum in the workspace; the last of the item's CTAs to do so joins the parts in
// their order (results do not depend on which one is last).
//
// Roles of the 16 warps:
//   0-7   softmax, two warps to 32 rows (each takes half of the columns): S from
//         tensor memory, running maximum and sum, the weights P back over S as
//         the A operand of P V; the item's epilogue;
//   8-11  TMA: K and V pages through one ring of 16 KB chunks, in the order the
//         MMAs use them (K0, K1, V0, K2, V1, ...; up to 128 dims one K further
//         ahead); a chunk is 128 keys x 64 dims
//         of K or 8192 / DP keys x DP dims of V, page by page.  One warp's copies
//         run one after the other at about 40 B a clock, whatever their boxes
//         (measured: 31 B with 64-slot boxes, 62 from two warps, 91 from four,
//         where L2 is the limit), and the tensor cores eat 64 B a clock at DP =
//         256: four warps take the chunks in turn;
//   12    MMA issue: S tiles take turns in two buffers (three up to 128 dims), so
//         Q K^T of the next tile runs while the softmax works on this one;
//   13    Q of the next item (TMA: the group's heads of its tokens, row by row).
// The output stays in tensor memory; it is rescaled only when a row's maximum
// grows by more than 2^8 (until then the weights are relative to the older
// maximum, which f32 sums and the 16-bit weights' exponents hold).  The tensor
// cores' f32 additions truncate (measured: 2.1e-8 of the output lost per
// addition), so every kDrain tiles it is added, rounded to nearest, to an f32
// copy in the workspace and starts again from zero.
//
// The reference is rounded to f32 before it is subtracted, so the largest weight
// may be off from 1 by half a step of it, in numerator and sum alike: nothing is
// lost until that overflows the weights' type (a reference past 2^26 in an f16
// cache, 2^30 in bf16).  Subtracting the maximum first would be exact, for an
// instruction more per pair of scores.
//
// A 16-bit output's weights are rounded to the cache's type, which the tensor
// cores multiply; their sum is that of the unrounded ones (lse needs it).  The
// output is off by 2.1e-3 to 2.3e-3 of its norm in bf16 and 2.9e-4 in f16, its own
// rounding included (alone 1.65e-3 and 2.1e-4).  Dividing by the sum of the rounded
// ones instead gives 2.0e-3 to 2.1e-3 and 2.7e-4 and takes prompts 379 us for 362,
// a chunk 1,208 for 1,178, drafts 53.5 for 51.3: not kept.
// An f32 output's weights are several digits of that type, and what the tensor
// cores' additions lose between drains matters as much.
//   Many rows: two digits, one after the other into the same accumulator (16 bits of
//   a weight in bf16, 22 in f16).
//   Up to 8 rows (single tokens of up to 8 query heads to a key head): the queries
//   lie in the tile once for each digit, eight lanes apart, and each copy's lanes
//   hold one digit of the weights: three in bf16 (all 24 bits), two in f16, with
//   accumulators of their own, half the additions into each, and no product more.
//   The epilogue adds the digits' outputs across the lanes.
// Off by, of the output's norm (two digits in one accumulator -> this; f32
// arithmetic): bf16 over 777 keys 1.5e-6 -> 0.8e-6 (0.6e-6), 131,072 4.2e-6 -> 2.2e-6
// (1.0e-6), 64 tokens over 100-8,000 3.1e-6 -> 1.4e-6 (0.4e-6); f16 1.1e-6 -> 1.0e-6,
// 3.4e-6 -> 2.4e-6 and 2.5e-6 -> 1.75e-6.  Times: bf16 777 keys 14.0 -> 14.2 us,
// 131,072 102-111 -> 103-116 (103.3 and 101.9 where most lie), 64 tokens at
// 256/128/64 dims 194/191/166 -> 200/196/163; f16 194/191/175 -> 196/194/162.  Two
// digits in lanes of their own in bf16 leave 1.4e-6, 3.3e-6 and 2.6e-6.
// Many rows have no idle lanes.  There a third digit in shared memory, for want of
// tensor memory, with drains every 4 tiles, and drains every 4 tiles alone, were
// measured and not kept: one token over 131,072 keys 3.9e-6 -> 2.4e-6 for 100 -> 109
// us; f32 chunks 4.1e-6 -> 3.2e-6 for 449 -> 516 us.  (Keys and values in bf16 are
// themselves rounded to 2e-3.)
//
// Bound: single tokens by HBM (one over 131,072 keys, 537 MB, 103 to 116 us
// with inputs changing from call to call: 4.6 to 5.2 TB/s; 64 over 100-8,000 keys
// each, 1.06 GB, 167 to 171 us: 6.2 to 6.3 TB/s) or, where keys are few, by the latency of one pass
// through the stages (777 keys 14.2 us); many tokens by the feeding of
// K and V to one CTA's MMAs (2,048 over 32,768 keys 1.19 ms, 1.34 PFLOP/s; 4
// prompts of 700-4,096 tokens 362 us).  With the softmax reduced to its
// handshakes the prompts take 343 us and the chunk 1,045: it is not the limit.
#include <cuda.h>
#include <math.h>

#include "kv_internal.cuh"
#include "ptx.cuh"

using namespace bitlin_impl;

namespace {

constexpr int kRows = 128;        // rows of a tile (UMMA M)
constexpr int kKeys = 128;        // keys of a tile
constexpr int kThreads = 512;
constexpr int kSoftmax = 256;     // threads of the softmax warps
constexpr int kTmaWarp = 8, kTmaWarps = 4, kMmaWarp = 12, kQWarp = 13;
// Registers a thread: launched with 128, the two softmax warpgroups take what
// the other two give (2 * 184 + 2 * 72 = 4 * 128).
constexpr int kManyRegs = 184, kFewRegs = 72;
constexpr int kChunkBytes = 16384;
constexpr int kTmemCols = 512;
constexpr float kLazy = 8.f;      // log2 of the growth that a rescale waits for
constexpr int kMaxLen = 1 << 30;
// Tiles that accumulate in tensor memory before the output is drained: 16
// additions a tile for an f32 output (2.7e-6 lost at 8 tiles), 8 for a 16-bit
// one (4e-5, a hundredth of bf16's rounding).
template <bool F32OUT>
constexpr int kDrain = F32OUT ? 8 : 256;
// Rows of a tile whose weights' digits lie in lanes of their own, and those digits:
// 24 bits of a weight in bf16, 22 in f16.
constexpr int kFewRows = 8;
template <typename T>
constexpr int kFewDigits = 3;
template <>
constexpr int kFewDigits<__half> = 2;

template <int DP>
struct Cfg {
    static constexpr int NC = DP / 64;                    // chunks of a K (and of a V) tile
    static constexpr int KV = 8192 / DP;                  // keys of a V chunk
    static constexpr int kQBytes = kRows * DP * 2;
    static constexpr int kStages = (224 * 1024 - kQBytes) / kChunkBytes > 12 ? 12 : (224 * 1024 - kQBytes) / kChunkBytes;
    // Tensor memory: the output, then NB buffers of S, which run AHEAD tiles in
    // front of the output's products.  Three buffers where they fit keep a tile
    // of scores waiting for either softmax group.
    static constexpr int NB = DP == 256 ? 2 : 3, AHEAD = NB - 1;
    static constexpr int kOCol = 0, kSCol = kTmemCols - NB * kKeys;
    static_assert(kSCol >= DP, "tensor memory");
};

// A sequence's rows and keys, with every index brought into range.
struct Seq {
    int row0, rows;   // token rows of the call
    int place0;       // place of the first
    int len;          // keys held
    int tiles;        // row tiles
};

constexpr int kRounds = 64;       // rounds of whole items at most

struct Item {
    int seq, head, qt;
};

// What a CTA has to do: `rounds` whole items, then a part of the line's rest.
struct Start {
    int rounds;
    int ctas;          // CTAs that have a part of the rest
    long long per;     // its length; the first `extra` CTAs have one more
    int extra;
    Item item;         // where the part begins
    int skip;          // its cost that belongs to earlier CTAs
    long long line;    // where it begins on the rest of the line
    Seq q;             // its sequence
    Item round[kRounds];
};

template <int DP>
struct __align__(8) Shared {
    uint64_t full[Cfg<DP>::kStages], empty[Cfg<DP>::kStages];
    uint64_t q_full, q_empty;
    uint64_t s_full[Cfg<DP>::NB], p_ready[Cfg<DP>::NB], pv_done[Cfg<DP>::NB];
    uint64_t o_free;
    uint64_t pair[4];  // the two softmax warps of 32 rows meet (a bounded wait, unlike a named barrier)
    uint64_t join;     // all softmax warps meet
    uint64_t never, drain;
    Start start;
    uint32_t tmem_base;
    int last;         // this CTA joins the item's parts
    int bad;          // 1 + the part whose values held an infinity or a NaN
    int grown[4];            // 1 + the last tile that asked for another reference
    float half[2][kRows];    // what a row's two halves tell each other: maxima, sums
    int abort;
};

template <int DP>
constexpr int smem_bytes()
{
    constexpr int bytes = Cfg<DP>::kQBytes + Cfg<DP>::kStages * kChunkBytes + (int)sizeof(Shared<DP>);
    static_assert(bytes <= 227 * 1024, "shared memory of an SM");
    return bytes;
}

// ---- the line of tiles ------------------------------------------------------

__device__ __forceinline__ Seq load_seq(const AttendParams& p, int s)
{
    Seq q;
    const int lo = p.batch.q_offsets[s], hi = p.batch.q_offsets[s + 1];
    const int raw = min(max(p.batch.kv_lens[s], 0), kMaxLen);
    const long long cap = (long long)p.batch.table_pages * p.page_size;
    q.row0 = min(max(lo, 0), p.tokens);
    q.rows = min(max(hi, q.row0), p.tokens) - q.row0;
    q.place0 = raw - (min(max(hi, 0), kMaxLen) - q.row0);
    q.len = raw < cap ? raw : (int)cap;
    q.tiles = (q.rows + p.tile_tokens - 1) / p.tile_tokens;
    if (q.len < raw) *p.index_error = 1;
    return q;
}

// Keys that the last row of row tile qt sees.
__device__ __forceinline__ int item_end(const AttendParams& p, int rows, int place0, int len, int qt)
{
    if (!p.causal) return len;
    return min(max(place0 + min(rows, (qt + 1) * p.tile_tokens), 0), len);
}

// Key tiles of an item; one that sees no key still takes a tile (it writes zeros).
__device__ __forceinline__ int item_tiles(int end) { return max(1, (end + kKeys - 1) / kKeys); }

// What an item costs, in key tiles: those and its begin and end (queries, the
// search for the first reference, the output).  On the line the begin and end
// come first: a cut there leaves the item whole.
__device__ __forceinline__ int item_cost(const AttendParams& p, int rows, int place0, int len, int qt)
{
    return item_tiles(item_end(p, rows, place0, len, qt)) + p.item_extra;
}

template <typename T>
__device__ __forceinline__ T warp_scan(T v)  // inclusive
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T u = __shfl_up_sync(0xffffffffu, v, o);
        if ((int)(threadIdx.x & 31) >= o) v += u;
    }
    return v;
}

// Cost of one key head of sequence base + lane (0 past the last sequence).
// Sequences of several row tiles are summed by the whole warp, one after the other.
__device__ __forceinline__ long long seq_cost(const AttendParams& p, int base, Seq& q)
{
    const int lane = threadIdx.x & 31;
    q = {};
    if (base + lane < p.batch.seqs) q = load_seq(p, base + lane);
    long long sum = q.tiles == 1 ? item_cost(p, q.rows, q.place0, q.len, 0) : 0;
    unsigned many = __ballot_sync(0xffffffffu, q.tiles > 1);
    while (many) {
        const int l = __ffs(many) - 1;
        many &= many - 1;
        const int rows = __shfl_sync(0xffffffffu, q.rows, l), place0 = __shfl_sync(0xffffffffu, q.place0, l);
        const int len = __shfl_sync(0xffffffffu, q.len, l), tiles = __shfl_sync(0xffffffffu, q.tiles, l);
        long long part = 0;
        for (int qt = lane; qt < tiles; qt += 32) part += item_cost(p, rows, place0, len, qt);
#pragma unroll
        for (int o = 16; o; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
        if (lane == l) sum = part;
    }
    return sum;
}

// x / n for n > 0; the sizes at hand nearly always fit 32 bits.
__device__ __forceinline__ long long divide(long long x, long long n)
{
    return ((x | n) >> 32) == 0 ? (long long)((uint32_t)x / (uint32_t)n) : x / n;
}
// The CTA whose part of the line holds x.
__device__ __forceinline__ int cta_of(const Start& s, long long x)
{
    const long long longer = s.extra * (s.per + 1);
    return x < longer ? (int)divide(x, s.per + 1) : s.extra + (int)divide(x - longer, s.per);
}

// One warp: what this CTA has to do.
__device__ void locate(const AttendParams& p, Start* out)
{
    const int lane = threadIdx.x & 31, grid = (int)gridDim.x, me = (int)blockIdx.x;
    Seq q;
    long long total = 0, items = 0, one = 0;
    int least = 0x7fffffff, most = 0;
    for (int base = 0; base < p.batch.seqs; base += 32) {
        one = seq_cost(p, base, q);
        long long n = one * p.kv_heads;
        int count = q.tiles;
        if (count) {
            least = min(least, item_cost(p, q.rows, q.place0, q.len, 0));
            most = max(most, item_cost(p, q.rows, q.place0, q.len, q.tiles - 1));
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            n += __shfl_xor_sync(0xffffffffu, n, o);
            count += __shfl_xor_sync(0xffffffffu, count, o);
        }
        total += n;
        items += (long long)count * p.kv_heads;
    }
    least = __reduce_min_sync(0xffffffffu, least);
    most = __reduce_max_sync(0xffffffffu, most);
    // Rounds of whole items when they cost about the same, within an eighth.
    // Measured, in us, without rounds and with: 128 single tokens of 8 key heads
    // over keys within 3 % of 4,000 330 and 324, within 10 % 320 and 313, within 20 %
    // 305 and 301, within 40 % the same, within 80 % 213 and 226; 2,048 tokens over
    // 32,768 keys, costs within 7 % (128 dims) 937 and 928, over 16,384, within 14 %,
    // 458 and 468, over 8,192 227 and 239, over 4,096 112 and 124.
    const int rounds = items >= grid && most - least <= least / 8 ? (int)min(divide(items, grid), (long long)kRounds) : 0;

    // Cost of row tiles 0 .. qt-1 of a sequence.
    auto cost_before = [&](const Seq& u, int qt) {
        long long n = 0;
        for (int i = lane; i < qt; i += 32) n += item_cost(p, u.rows, u.place0, u.len, i);
#pragma unroll
        for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
        return n;
    };
    auto lane_seq = [&](int l) {
        Seq u;
        u.row0 = __shfl_sync(0xffffffffu, q.row0, l);
        u.rows = __shfl_sync(0xffffffffu, q.rows, l);
        u.place0 = __shfl_sync(0xffffffffu, q.place0, l);
        u.len = __shfl_sync(0xffffffffu, q.len, l);
        u.tiles = __shfl_sync(0xffffffffu, q.tiles, l);
        return u;
    };
    // The rounds' items, and the tiles on the line before the first item after them.
    long long line0 = 0;
    if (rounds) {
        long long items_before = 0, tiles_upto = 0;
        line0 = total;
        int k = 0;
        for (int base = 0; base < p.batch.seqs && k <= rounds; base += 32) {
            if (p.batch.seqs > 32) one = seq_cost(p, base, q);
            const long long upto = items_before + warp_scan((long long)q.tiles * p.kv_heads);
            const long long tiles = tiles_upto + warp_scan(one * p.kv_heads);
            for (; k <= rounds; ++k) {
                const long long x = k < rounds ? me + (long long)k * grid : (long long)rounds * grid;
                const unsigned past = __ballot_sync(0xffffffffu, upto > x);
                if (!past) break;
                const int l = __ffs(past) - 1;
                const Seq u = lane_seq(l);
                const int off = (int)(x - __shfl_sync(0xffffffffu, upto - (long long)q.tiles * p.kv_heads, l));
                const int head = off / u.tiles, qt = off - head * u.tiles;
                if (k < rounds) {
                    if (lane == 0) out->round[k] = {base + l, head, qt};
                } else {
                    const long long per = __shfl_sync(0xffffffffu, one, l);
                    line0 = __shfl_sync(0xffffffffu, tiles, l) - per * (p.kv_heads - head) + cost_before(u, qt);
                }
            }
            items_before = __shfl_sync(0xffffffffu, upto, 31);
            tiles_upto = __shfl_sync(0xffffffffu, tiles, 31);
        }
    }

    // The rest of the line, in equal parts.
    const long long rest = total - line0;
    const int ctas = rest < (long long)grid ? (int)rest : grid;
    Item item = {};
    int skip = 0, extra = 0;
    long long per_cta = 0, line = 0;
    Seq mine = {};
    if (me < ctas) {
        per_cta = divide(rest, ctas);
        extra = (int)(rest - per_cta * ctas);
        const long long x = line0 + per_cta * me + min(me, extra);
        long long before = 0;
        for (int base = 0; base < p.batch.seqs; base += 32) {
            if (p.batch.seqs > 32) one = seq_cost(p, base, q);
            const long long all = one * p.kv_heads;
            const long long upto = before + warp_scan(all);
            const unsigned past = __ballot_sync(0xffffffffu, upto > x);
            if (past) {
                const int l = __ffs(past) - 1;
                const long long per = __shfl_sync(0xffffffffu, one, l);
                long long off = x - __shfl_sync(0xffffffffu, upto - all, l);
                mine = lane_seq(l);
                item.seq = base + l;
                item.head = (int)divide(off, per);
                off -= item.head * per;
                for (int qb = 0; qb < mine.tiles; qb += 32) {
                    const int n = qb + lane < mine.tiles ? item_cost(p, mine.rows, mine.place0, mine.len, qb + lane) : 0;
                    const long long to = warp_scan((long long)n);
                    const unsigned hit = __ballot_sync(0xffffffffu, to > off);
                    if (hit) {
                        const int h = __ffs(hit) - 1;
                        item.qt = qb + h;
                        skip = (int)(off - __shfl_sync(0xffffffffu, to - n, h));
                        line = x - line0 - skip;
                        break;
                    }
                    off -= __shfl_sync(0xffffffffu, to, 31);
                }
                break;
            }
            before = __shfl_sync(0xffffffffu, upto, 31);
        }
    }
    if (lane == 0) {
        out->rounds = rounds;
        out->ctas = ctas;
        out->per = per_cta;
        out->extra = extra;
        out->item = item;
        out->skip = skip;
        out->line = line;
        out->q = mine;
    }
}

// A CTA's items and parts of items, one after the other; every role walks them alike.
struct Walk {
    const AttendParams& p;
    const Start& start;
    int round;            // whole items taken
    long long left;       // length of the part of the line still to come
    long long line;       // where the item begins on the line's rest
    int from;             // its cost that belongs to earlier CTAs
    int seq, head, qt;
    Seq q;
    int end;              // keys the item's last row sees
    int tiles, j0, j1;    // the item's key tiles, and this part of them

    __device__ Walk(const AttendParams& params, const Start& s) : p(params), start(s), round(0), left(0), line(0), from(0), seq(-1)
    {
        if (start.rounds) take_round();
        else take_rest();
    }
    __device__ bool valid() const { return round < start.rounds || left > 0; }
    __device__ bool in_rest() const { return round >= start.rounds; }
    __device__ void set()
    {
        end = item_end(p, q.rows, q.place0, q.len, qt);
        tiles = item_tiles(end);
        j0 = 0;
        j1 = tiles;
        if (in_rest()) {
            j0 = max(0, from - p.item_extra);
            j1 = (int)max(0LL, min((long long)tiles, from + left - p.item_extra));
        }
    }
    __device__ void take_round()
    {
        const Item it = start.round[round];
        if (it.seq != seq) q = load_seq(p, it.seq);
        seq = it.seq;
        head = it.head;
        qt = it.qt;
        set();
    }
    __device__ void take_rest()
    {
        if ((int)blockIdx.x >= start.ctas) return;
        left = start.per + ((int)blockIdx.x < start.extra ? 1 : 0);
        line = start.line;
        from = start.skip;
        seq = start.item.seq;
        head = start.item.head;
        qt = start.item.qt;
        q = start.q;
        set();
        if (j0 >= j1) step();  // a part of an item's begin alone
    }
    __device__ void next()
    {
        if (round < start.rounds) {
            if (++round < start.rounds) take_round();
            else take_rest();
        } else {
            step();
        }
    }
    // The next item of the part of the line that has a tile in it.
    __device__ void step()
    {
        do {
            const int cost = tiles + p.item_extra;
            left -= cost - from;
            line += cost;
            from = 0;
            if (left <= 0) return;
            if (++qt == q.tiles) {
                qt = 0;
                if (++head == p.kv_heads) {
                    head = 0;
                    q.tiles = 0;
                    while (q.tiles == 0 && seq + 1 < p.batch.seqs) q = load_seq(p, ++seq);
                    if (q.tiles == 0) {  // the lengths changed under the call
                        left = 0;
                        return;
                    }
                }
            }
            set();
            if (j1 == 0) left = 0;  // the part ends in this item's begin
        } while (left > 0 && j0 >= j1);
    }
    // tokens of the row tile
    __device__ int tokens() const { return min(p.tile_tokens, q.rows - qt * p.tile_tokens); }
};

// Waits for a barrier's phase like ptx::mbar_wait_bounded, in fewer
// instructions: this kernel's loops are bound by instruction fetch where they
// grow (see the softmax).
__device__ __forceinline__ bool wait(uint64_t* bar, int phase, volatile int* abort, long long budget)
{
    if (ptx::mbar_try_wait(bar, (uint32_t)phase & 1u)) return true;
    const uint64_t t0 = ptx::globaltimer();
    do {
        if (ptx::mbar_try_wait(bar, (uint32_t)phase & 1u)) return true;
        if (*abort) return false;
    } while ((long long)(ptx::globaltimer() - t0) <= budget);
    *abort = 1;
    return false;
}

// A whole warp waits; true when every lane saw the phase complete.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, int phase, volatile int* abort, long long budget)
{
    return __all_sync(0xffffffffu, wait(bar, phase, abort, budget));
}

// Page of a sequence and slot in it that hold key `key`.
__device__ __forceinline__ int page_at(const AttendParams& p, int key)
{
    return p.page_shift >= 0 ? key >> p.page_shift : key / p.page_size;
}
__device__ __forceinline__ int slot_at(const AttendParams& p, int key)
{
    return p.page_shift >= 0 ? key & (p.page_size - 1) : key % p.page_size;
}

// ---- weights ----------------------------------------------------------------

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b)
{
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t v);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t v)
{
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t v)
{
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

// The digits of a weight are runs of its significand: what it is up to a run's end
// less what it is up to its begin, which masks give.  (Digits rounded one after the
// other took 200 us for 196 on 64 tokens of 128 dims, 178 for 162 at 64 dims.)
template <typename T>
__device__ __forceinline__ uint32_t first_digits(int n)  // mask of the first n
{
    return n == 0 ? 0u : n >= kFewDigits<T> ? 0xFFFFFFFFu : kFewDigits<T> == 2 ? 0xFFFFE000u : n == 1 ? 0xFFFF0000u : 0xFFFFFF00u;
}
__device__ __forceinline__ float run(float x, uint32_t mask) { return __uint_as_float(__float_as_uint(x) & mask); }

// Exponent bits of a 16-bit element: all ones is an infinity or a NaN.
template <typename T>
constexpr uint32_t kExpBits = 0x7F80u;
template <>
constexpr uint32_t kExpBits<__half> = 0x7C00u;

// f16 weights are held 2^6 larger, which keeps 2^-31 of the largest one above
// their smallest step; with kLazy they stay below 2^14.  bf16 has f32's range.
template <typename T>
constexpr float kShift = 0.f;
template <>
constexpr float kShift<__half> = 6.f;

// Zero the infinities and NaNs of a word of two elements; whether there were any.
template <typename T>
__device__ __forceinline__ bool clean(uint32_t& w)
{
    constexpr uint32_t e = kExpBits<T>;
    const bool lo = (w & e) == e, hi = ((w >> 16) & e) == e;
    if (lo) w &= 0xFFFF0000u;
    if (hi) w &= 0x0000FFFFu;
    return lo || hi;
}

// ---- the kernel -------------------------------------------------------------

// F32OUT: the output is f32 and each weight is two digits of T, hi = T(w) and
// lo = T(w - hi), multiplied into the same accumulator one after the other.  FEW
// (F32OUT, tiles of up to 8 rows): each weight is kFewDigits digits, digit d of row
// r in lane 8 d + r, with an accumulator of its own.
template <int DP, typename T, bool F32OUT, bool FEW>
__global__ void __launch_bounds__(kThreads, 1)
    bitlin_attend(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                  const __grid_constant__ AttendParams p)
{
    using C = Cfg<DP>;
    constexpr int NC = C::NC, NS = C::kStages, KV = C::KV;
    constexpr bool kBf16 = sizeof(T) == 2 && kExpBits<T> == 0x7F80u;

    extern __shared__ __align__(1024) unsigned char smem[];  // (the swizzle's atoms are 1024 bytes)
    unsigned char* tile_q = smem;                // [NC][128 rows][64], 128-byte swizzle
    unsigned char* ring = smem + C::kQBytes;     // [NS][16 KB]
    auto* sh = reinterpret_cast<Shared<DP>*>(ring + NS * kChunkBytes);
    volatile int* abort = &sh->abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long budget = p.wait_budget_ns;

    if (warp == kTmaWarp && lane < NS) {
        ptx::mbar_init(&sh->full[lane], 1);
        ptx::mbar_init(&sh->empty[lane], 1);
        ptx::mbar_fence_init();
        ptx::fence_proxy_async_smem();
    }
    if (warp == kTmaWarp + 1) {
        if (lane < C::NB) {
            ptx::mbar_init(&sh->s_full[lane], 1);
            ptx::mbar_init(&sh->p_ready[lane], kSoftmax);
            ptx::mbar_init(&sh->pv_done[lane], 1);
        } else if (lane >= 4 && lane < 8) {
            ptx::mbar_init(&sh->pair[lane - 4], 2);
            if (lane == 4) sh->abort = sh->bad = 0;
        } else if (lane == 8) {
            ptx::mbar_init(&sh->q_full, 1);
            ptx::mbar_init(&sh->q_empty, 1);
            ptx::mbar_init(&sh->o_free, kSoftmax);
        } else if (lane == 9) {
            ptx::mbar_init(&sh->join, kSoftmax);
            ptx::mbar_init(&sh->never, 1);
            ptx::mbar_init(&sh->drain, 1);
        } else if (lane >= 10 && lane < 14) {
            sh->grown[lane - 10] = 0;
        }
        ptx::mbar_fence_init();
        ptx::fence_proxy_async_smem();
    }
    if (warp == kTmaWarp + 2 && lane == 0) {
        ptx::prefetch_tmap(&tmap_q);
        ptx::prefetch_tmap(&tmap_k);
        ptx::prefetch_tmap(&tmap_v);
    }
    if (warp == kMmaWarp) {
        ptx::tmem_alloc(&sh->tmem_base, kTmemCols);
        ptx::tmem_relinquish();
    }
    ptx::griddep_wait();
    if (warp == 0) locate(p, &sh->start);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    ptx::griddep_launch_dependents();
    const uint32_t tmem = sh->tmem_base;
    const Start& start = sh->start;

    if (warp >= kTmaWarp && warp < kTmaWarp + kTmaWarps) {
        ptx::give_registers<kFewRegs>();
        Walk w(p, start);
        const int mine = warp - kTmaWarp;
        int stage = 0;
        uint32_t phase = 0;
        int issued = 0;
        bool ok = true;
        // Lane l holds the page of keys 8l .. 8l+7 of a tile.  Entries are read two
        // tiles ahead and looked at only when their tile is copied: looking at
        // them at once put the table's latency into every tile (35 B a clock
        // instead of the 70 that the copies alone reach).
        auto entry = [&](int j) {
            const int key = j * kKeys + 8 * lane;
            return lane < kKeys / 8 && j < w.j1 && key < w.end ? p.batch.table[w.seq * p.batch.table_stride + page_at(p, key)] : 0;
        };
        auto checked = [&](int page) {
            if (page >= 0 && page < p.pages) return page;
            *p.index_error = 1;
            return -1;  // outside the pool: the copy fills zeros
        };
        auto next_stage = [&]() {
            ++issued;
            if (++stage == NS) {
                stage = 0;
                phase ^= 1u;
            }
        };
        for (; w.valid() && ok; w.next()) {
            int next[2] = {entry(w.j0), entry(w.j0 + 1)}, page_v[C::AHEAD];
            for (int j = w.j0; j < w.j1 + C::AHEAD && ok; ++j) {
                const int page_k = checked(next[0]);
                next[0] = next[1];
                next[1] = entry(j + 2);
                if (j < w.j1) {
                    // K tile j: NC chunks of 128 keys x 64 dims
                    const int keys = min(kKeys, w.end - j * kKeys);
                    const int boxes = keys > 0 ? (keys + p.box_k - 1) / p.box_k : 0;
                    const int at = min(lane * p.box_k, kKeys - 8);
                    const int page = __shfl_sync(0xffffffffu, page_k, at >> 3);
                    const int slot = slot_at(p, j * kKeys + at);
#pragma unroll 1
                    for (int c = 0; c < NC; ++c, next_stage()) {
                        if ((issued & (kTmaWarps - 1)) != mine) continue;
                        ok = warp_wait(&sh->empty[stage], phase ^ 1u, abort, budget);
                        if (!ok) break;
                        unsigned char* dst = ring + stage * kChunkBytes;
                        if (lane == 0) {
                            if (boxes) ptx::mbar_arrive_expect_tx(&sh->full[stage], boxes * p.box_k * 128);
                            else ptx::mbar_arrive(&sh->full[stage]);
                        }
                        __syncwarp();
                        if (lane < boxes)
                            ptx::tma_load_4d(dst + lane * p.box_k * 128, &tmap_k, 64 * c, slot, w.head, page,
                                             &sh->full[stage]);
                    }
                }
                if (j >= w.j0 + C::AHEAD && ok) {
                    // V tile j - AHEAD: NC chunks of KV keys x DP dims, as [dims / 64][KV][64]
                    const int box = lane / NC, dims = lane % NC;
#pragma unroll 1
                    for (int c = 0; c < NC; ++c, next_stage()) {
                        if ((issued & (kTmaWarps - 1)) != mine) continue;
                        const int key = (j - C::AHEAD) * kKeys + c * KV;
                        const int keys = min(KV, w.end - key);
                        const int boxes = keys > 0 ? (keys + p.box_v - 1) / p.box_v : 0;
                        const int at = min(c * KV + box * p.box_v, kKeys - 8);
                        const int page = __shfl_sync(0xffffffffu, page_v[C::AHEAD - 1], at >> 3);
                        const int slot = slot_at(p, (j - C::AHEAD) * kKeys + at);
                        ok = warp_wait(&sh->empty[stage], phase ^ 1u, abort, budget);
                        if (!ok) break;
                        unsigned char* dst = ring + stage * kChunkBytes;
                        if (lane == 0) {
                            if (boxes) ptx::mbar_arrive_expect_tx(&sh->full[stage], boxes * p.box_v * 128 * NC);
                            else ptx::mbar_arrive(&sh->full[stage]);
                        }
                        __syncwarp();
                        if (box < boxes)
                            ptx::tma_load_4d(dst + dims * (KV * 128) + box * p.box_v * 128, &tmap_v, 64 * dims, slot,
                                             w.head, page, &sh->full[stage]);
                    }
                }
#pragma unroll
                for (int a = C::AHEAD - 1; a > 0; --a) page_v[a] = page_v[a - 1];
                page_v[0] = page_k;
            }
        }
        // Every copy issued here must land before the CTA may exit.
        for (int i = issued > NS ? issued - NS : 0; i < issued; ++i) {
            if ((i & (kTmaWarps - 1)) != mine) continue;
            volatile int no_abort = 0;
            ptx::mbar_wait_bounded(&sh->full[i % NS], (uint32_t)(i / NS) & 1u, &no_abort, budget);
        }
    } else if (warp == kMmaWarp) {
        ptx::give_registers<kFewRegs>();
        Walk w(p, start);
        constexpr uint32_t idesc_s = ptx::idesc_f32(kRows, kKeys, kBf16, false);
        constexpr uint32_t idesc_o = ptx::idesc_f32(kRows, DP, kBf16, true);
        const uint64_t desc_q = ptx::smem_desc_sw128(ptx::smem_u32(tile_q));
        const uint64_t desc_k = ptx::smem_desc_sw128(ptx::smem_u32(ring));
        const uint64_t desc_v = ptx::smem_desc_sw128_mn(ptx::smem_u32(ring), KV * 128);
        int stage = 0;
        uint32_t phase = 0;
        int gt = 0;       // tiles so far, over all parts: S buffer t % NB of tile t
        int part = 0;
        bool ok = true, any = false;
        auto next_stage = [&]() {
            if (++stage == NS) {
                stage = 0;
                phase ^= 1u;
            }
        };
        for (; w.valid() && ok; w.next(), ++part) {
            const int n = w.j1 - w.j0;
            ok = warp_wait(&sh->q_full, part, abort, budget);
            // step i: S(i) = Q K(i)^T, then O += P(i - AHEAD) V(i - AHEAD)
            for (int i = 0; i < n + C::AHEAD && ok; ++i) {
                if (i < n) {
                    const int t = gt + i, b = t % C::NB;
                    // the buffer's previous weights have been multiplied
                    if (t >= C::NB) ok = warp_wait(&sh->pv_done[b], t / C::NB - 1, abort, budget);
                    for (int c = 0; c < NC && ok; ++c) {
                        ok = warp_wait(&sh->full[stage], phase, abort, budget);
                        if (!ok) break;
                        ptx::tc_fence_after();
                        if (ptx::elect_one()) {
                            const uint32_t d = tmem + C::kSCol + b * kKeys;
                            const uint64_t a = desc_q + (uint64_t)((c * kChunkBytes) >> 4);
                            const uint64_t k = desc_k + (uint64_t)((stage * kChunkBytes) >> 4);
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                ptx::mma_bf16(d, a + 2 * kk, k + 2 * kk, idesc_s, c > 0 || kk > 0 ? 1u : 0u);
                            ptx::mma_commit(&sh->empty[stage]);
                            if (c == NC - 1) {
                                ptx::mma_commit(&sh->s_full[b]);
                                if (i == n - 1) ptx::mma_commit(&sh->q_empty);
                            }
                        }
                        __syncwarp();
                        any = true;
                        next_stage();
                    }
                }
                if (i >= C::AHEAD && ok) {
                    const int iv = i - C::AHEAD, t = gt + iv, b = t % C::NB;
                    const bool fresh = iv % kDrain<F32OUT> == 0;  // the output starts from zero
                    if (iv == 0 && part > 0) ok = warp_wait(&sh->o_free, part - 1, abort, budget);
                    ok = ok && warp_wait(&sh->p_ready[b], t / C::NB, abort, budget);
                    for (int c = 0; c < NC && ok; ++c) {
                        ok = warp_wait(&sh->full[stage], phase, abort, budget);
                        if (!ok) break;
                        ptx::tc_fence_after();
                        if (ptx::elect_one()) {
                            const uint32_t pcol = tmem + C::kSCol + b * kKeys;
                            const uint64_t v = desc_v + (uint64_t)((stage * kChunkBytes) >> 4);
#pragma unroll
                            for (int kk = 0; kk < KV / 16; ++kk) {
                                // 16 keys are 8 columns; the weights of 32 keys lie in their scores' columns
                                const int key = c * KV + 16 * kk;
                                const uint32_t col = pcol + (key & ~31) + ((key & 31) >> 1);
                                ptx::mma_bf16_ts(tmem + C::kOCol, col, v + (uint64_t)(kk * 2048 >> 4), idesc_o,
                                                 !fresh || c > 0 || kk > 0 ? 1u : 0u);
                                if (F32OUT && !FEW)
                                    ptx::mma_bf16_ts(tmem + C::kOCol, col + 16, v + (uint64_t)(kk * 2048 >> 4), idesc_o, 1u);
                            }
                            ptx::mma_commit(&sh->empty[stage]);
                            if (c == NC - 1) ptx::mma_commit(&sh->pv_done[b]);
                        }
                        __syncwarp();
                        next_stage();
                    }
                }
            }
            gt += n;
        }
        // Wait for every MMA issued here before tensor memory is released.
        if (any) {
            if (ptx::elect_one()) ptx::mma_commit(&sh->drain);
            __syncwarp();
            volatile int no_abort = 0;
            ptx::mbar_wait_bounded(&sh->drain, 0u, &no_abort, budget);
        }
    } else if (warp >= kQWarp) {
        ptx::give_registers<kFewRegs>();
        if (warp == kQWarp) {
            Walk w(p, start);
            int part = 0;
            bool ok = true;
            for (; w.valid() && ok; w.next(), ++part) {
                if (part > 0) ok = warp_wait(&sh->q_empty, part - 1, abort, budget);
                if (!ok) break;
                // Boxes of q_box tokens x the group's heads x 64 dims; dims past the
                // head's are zeros (K's are, and a zero times what lies there must stay zero).
                // FEW: the tile's one box, once for each digit.
                const int boxes = FEW ? kFewDigits<T> : (w.tokens() + p.q_box - 1) / p.q_box;
                const int bytes = p.q_box * p.group * 128, apart = FEW ? kFewRows * 128 : bytes;
                if (lane == 0) ptx::mbar_arrive_expect_tx(&sh->q_full, boxes * bytes * NC);
                __syncwarp();
                for (int k = lane; k < boxes * NC; k += 32) {
                    const int c = k % NC, box = k / NC;
                    ptx::tma_load_3d(tile_q + c * kChunkBytes + box * apart, &tmap_q, 64 * c, w.head * p.group,
                                     w.q.row0 + w.qt * p.tile_tokens + (FEW ? 0 : box * p.q_box), &sh->q_full);
                }
            }
            // The last copies must land before the CTA may exit.
            if (part > 0) {
                volatile int no_abort = 0;
                ptx::mbar_wait_bounded(&sh->q_full, (uint32_t)(part - 1) & 1u, &no_abort, budget);
            }
        }
    } else {
        // ---- softmax and epilogue: thread = row and half of the columns.
        // A tile's weights are taken relative to the row's reference of the tile
        // before.  No maximum is looked for as long as their sum stays below
        // 2^kLazy, which bounds each of them: a pass over the scores less than a
        // running maximum needs.  Where a sum passes it (and in the first tile)
        // the two warps of the row find the maximum, rescale and start over.
        ptx::take_registers<kManyRegs>();
        Walk w(p, start);
        constexpr int HALF = DP / 2;             // output columns of a thread
        constexpr int G = kDrain<F32OUT>, NB = C::NB;
        const int side = warp >> 2, quad = warp & 3;
        const int r = threadIdx.x & (kRows - 1);
        const uint32_t lane_base = (uint32_t)(32 * quad) << 16;
        // log2 units; a scale of 0 becomes one that no score can make count, so
        // that a masked score (-inf) times it still is -inf
        const float sl2 = fmaxf(fabsf(p.scale) * 1.4426950408889634f, 1e-37f);
        const bool negative = p.scale < 0.f;
        const float sign = negative ? -1.f : 1.f, mul = sign * sl2;
        const float limit = exp2f(kLazy + kShift<T>);
        const int digit = FEW ? r / kFewRows : 0, my_row = FEW ? r % kFewRows : r;
        const int my_token = my_row / p.group, my_head = my_row - my_token * p.group;
        const uint32_t digit_to = first_digits<T>(digit + 1), digit_from = first_digits<T>(digit);
        int gt = 0, consumed = 0;                // tiles and ring chunks before this part
        int part = 0, joined = 0, paired = 0;    // parts before this one, meetings so far
        bool ok = true;
        // the two warps of these rows meet
        auto meet = [&]() {
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&sh->pair[quad]);
            ok = warp_wait(&sh->pair[quad], paired++, abort, budget);
        };
        for (; w.valid() && ok; w.next(), ++part) {
            const int n = w.j1 - w.j0;
            const int tokens = w.tokens();
            const bool valid = my_token < tokens && (!FEW || digit < kFewDigits<T>);
            const bool active = 32 * quad < tokens * p.group;     // the warp has a valid row
            const int first = w.q.place0 + w.qt * p.tile_tokens;  // place of the first token
            const int lim_first = p.causal ? min(max(first + 1, 0), w.q.len) : w.q.len;
            const int lim = !valid ? w.end : p.causal ? min(max(first + my_token + 1, 0), w.q.len) : w.q.len;
            float m = -INFINITY, base = -kShift<T>;  // reference, and what is subtracted from scaled scores
            float sum = 0.f;                         // weights of this half
            bool bad = false;
            // this thread's part of the workspace: f32 output drained so far, at reference ws_base
            const long long slot = 2LL * blockIdx.x + (w.j0 == 0 ? 1 : 0);
            // Up to 32 rows lie one after the other; more lie four columns of all rows
            // after the other, so that a warp's accesses are consecutive.
            const bool by_row = tokens * p.group <= 32;
            const int ws_col = by_row ? 1 : kRows, ws_row = by_row ? DP / 4 : 1;
            float4* ws_o = reinterpret_cast<float4*>(p.ws_o) + slot * (DP / 4) * kRows + side * (HALF / 4) * ws_col + r * ws_row;
            float ws_base = -INFINITY;
            // What drained output counts at the present reference: 0 where there was none
            // yet, since the first one may lie far below what stands for none.
            auto drained_by = [&]() { return ptx::ex2(ws_base - base); };
            // before it writes what its partner may still read of the part before
            if (active && part > 0) meet();
            if (!ok) break;
            const uint32_t out_col = tmem + lane_base + C::kOCol + side * HALF;
            for (int i = 0; i < n && ok; ++i) {
                const int t = gt + i, b = t % NB;
                uint64_t* wbar = p.stall_test && t == 0 ? &sh->never : &sh->s_full[b];
                ok = warp_wait(wbar, t / NB, abort, budget);
                if (!ok) break;
                ptx::tc_fence_after();
                const int key0 = (w.j0 + i) * kKeys;
                const bool edge = key0 + kKeys > lim_first;  // some row does not see the whole tile
                const bool fresh = i > 0 && i % G == 0;      // the output goes to the workspace first
                if (fresh) {
                    ok = warp_wait(&sh->pv_done[(t - 1) % NB], (t - 1) / NB, abort, budget);
                    if (!ok) break;
                    ptx::tc_fence_after();
                    if (active) {
                        const float f = drained_by();
#pragma unroll 1
                        for (int c = 0; c < HALF; c += 16) {
                            float o[16];
                            ptx::tmem_ld16(out_col + c, o);
                            ptx::tmem_wait_ld();
                            ptx::tmem_landed(o);
                            if (valid) {
#pragma unroll
                                for (int k = 0; k < 16; k += 4) {
                                    float4* to = ws_o + (c + k) / 4 * ws_col;
                                    float4 x = make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
                                    if (i > G && f == 1.f) {
                                        ptx::red_add4(to, x);
                                        continue;
                                    }
                                    if (i > G) {
                                        const float4 y = __ldcg(to);
                                        x = make_float4(fmaf(y.x, f, x.x), fmaf(y.y, f, x.y), fmaf(y.z, f, x.z), fmaf(y.w, f, x.w));
                                    }
                                    __stcg(to, x);
                                }
                            }
                            __syncwarp();
                        }
                        // (a row without a reference so far has drained nothing but zeros or NaNs)
                        ws_base = m == -INFINITY ? -INFINITY : base;
                    }
                }
                if (active) {
                    const uint32_t taddr = tmem + lane_base + C::kSCol + b * kKeys + 64 * side;
                    if (edge) {
                        // Scores that the row does not see, in place: what every tile
                        // runs below stays free of masks (and small: this kernel's code
                        // is larger than the instruction caches, and each way that is
                        // not the usual one costs a fetch).
                        const int see = lim - key0 - 64 * side;  // of these 64 keys, those that the row sees
#pragma unroll 1
                        for (int c = 0; c < 64; c += 16) {
                            float x[16];
                            uint32_t u[16];
                            ptx::tmem_ld16(taddr + c, x);
                            ptx::tmem_wait_ld();
                            ptx::tmem_landed(x);
#pragma unroll
                            for (int k = 0; k < 16; ++k) u[k] = __float_as_uint(c + k < see ? x[k] : -INFINITY * sign);
                            ptx::tmem_st16(taddr + c, u);
                        }
                        ptx::tmem_wait_st();
                    }
                    bool search = i == 0, settled = false;
                    float add = 0.f;
                    uint32_t hi[32], lo[32];
#pragma unroll 1
                    for (;;) {
                        float s[2][32];
                        ptx::tmem_ld32(taddr, s[0]);
                        ptx::tmem_ld32(taddr + 32, s[1]);
                        ptx::tmem_wait_ld();
                        ptx::tmem_landed(s[0]);
                        ptx::tmem_landed(s[1]);
                        if (!search) {
                            float2 add0 = make_float2(0.f, 0.f), add1 = make_float2(0.f, 0.f);
#pragma unroll
                            for (int k = 0; k < 64; k += 2) {
                                const float2 x = __ffma2_rn(make_float2(s[k >> 5][k & 31], s[k >> 5][(k & 31) + 1]),
                                                            make_float2(mul, mul), make_float2(-base, -base));
                                const float2 e = make_float2(ptx::ex2(x.x), ptx::ex2(x.y));
                                if (k & 2) add1 = __fadd2_rn(add1, e);
                                else add0 = __fadd2_rn(add0, e);
                                if (FEW) {
                                    hi[k / 2] = pack2<T>(run(e.x, digit_to) - run(e.x, digit_from),
                                                         run(e.y, digit_to) - run(e.y, digit_from));
                                    continue;
                                }
                                hi[k / 2] = pack2<T>(e.x, e.y);
                                if (F32OUT) {
                                    const float2 f = unpack2<T>(hi[k / 2]);
                                    lo[k / 2] = pack2<T>(e.x - f.x, e.y - f.y);
                                }
                            }
                            add0 = __fadd2_rn(add0, add1);
                            add = add0.x + add0.y;
                            if (settled) break;
                            // (a row without a reference so far needs one whatever its sum)
                            const bool ask = __any_sync(0xffffffffu, valid && (m == -INFINITY || add > limit));
                            if (ask && lane == 0) sh->grown[quad] = t + 1;
                            meet();
                            if (!ok || *(volatile int*)&sh->grown[quad] != t + 1) break;
                            search = true;
                            continue;
                        }
                        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int k = 0; k < 64; ++k) top[k & 3] = fmaxf(top[k & 3], s[k >> 5][k & 31] * sign);
                        const float mine = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                        sh->half[side][r] = mine;
                        meet();
                        if (!ok) break;
                        const float now = fmaxf(m, fmaxf(mine, *(volatile float*)&sh->half[side ^ 1][r]));
                        const float to = now > m ? now * sl2 - kShift<T> : base;
                        const float keep = m == -INFINITY ? 0.f : ptx::ex2(base - to);
                        if (now > m) sum *= keep;
                        m = now;
                        if (i > 0 && !fresh) {
                            ok = warp_wait(&sh->pv_done[(t - 1) % NB], (t - 1) / NB, abort, budget);
                            if (!ok) break;
                            ptx::tc_fence_after();
#pragma unroll 1
                            for (int c = 0; c < HALF; c += 16) {
                                float o[16];
                                uint32_t u[16];
                                ptx::tmem_ld16(out_col + c, o);
                                ptx::tmem_wait_ld();
                                ptx::tmem_landed(o);
#pragma unroll
                                for (int k = 0; k < 16; ++k) u[k] = __float_as_uint(o[k] * keep);
                                ptx::tmem_st16(out_col + c, u);
                            }
                        }
                        base = to;
                        search = false;
                        settled = true;
                    }
                    if (!ok) break;
                    sum += add;
                    // the weights of 32 keys over their scores: hi in the first 16 columns, lo in the others
#pragma unroll
                    for (int c = 0; c < 32; c += 16) {
                        uint32_t x[16];
#pragma unroll
                        for (int k = 0; k < 16; ++k) x[k] = hi[c + k];
                        ptx::tmem_st16(taddr + 2 * c, x);
                        if (F32OUT && !FEW) {
#pragma unroll
                            for (int k = 0; k < 16; ++k) x[k] = lo[c + k];
                            ptx::tmem_st16(taddr + 2 * c + 16, x);
                        }
                    }
                }
                if (edge) {
                    // Values that some row does not see: those past the item's last
                    // key become zeros (a weight of zero times what a free slot
                    // holds must be zero), infinities and NaNs between the first
                    // row's and the last row's last key too; the epilogue gives
                    // them back to the rows that see them.
                    const int lo = max(lim_first - key0, 0), hi = w.end - key0;
                    const int v0 = consumed + NC * min(2 * i + C::AHEAD + 1, n + i);
                    // A stage's parity answers for its last two chunks alone.  This tile's
                    // scores say that its K has landed; where the ring is shorter than from
                    // there to its V (256 dims: 12 chunks in 10 stages), the chunk before in
                    // the stage is one of the V before, which the MMAs have then to be
                    // through with.  (In a part's last tile no K lies between.)
                    if ((2 * C::AHEAD + 1) * NC > NS && i > 0 && i + 1 < n) {
                        ok = warp_wait(&sh->pv_done[(t - 1) % NB], (t - 1) / NB, abort, budget);
                        if (!ok) break;
                    }
#pragma unroll 1
                    for (int c = lo / KV; c < NC && ok; ++c) {
                        const int st = (v0 + c) % NS;
                        ok = warp_wait(&sh->full[st], (v0 + c) / NS, abort, budget);
                        if (!ok) break;
                        const int u = threadIdx.x;  // row u / 8, its 16 bytes u % 8
                        for (int row = max(lo - c * KV, 0) + (u >> 3); row < KV; row += kSoftmax / 8) {
                            uint4* at = reinterpret_cast<uint4*>(ring + st * kChunkBytes + row * 128 + (u & 7) * 16);
#pragma unroll
                            for (int d = 0; d < NC; ++d, at += KV * 8) {
                                if (c * KV + row >= hi) {
                                    *at = make_uint4(0, 0, 0, 0);
                                } else {
                                    uint4 x = *at;
                                    bool any = clean<T>(x.x);
                                    any |= clean<T>(x.y);
                                    any |= clean<T>(x.z);
                                    any |= clean<T>(x.w);
                                    if (any) {
                                        *at = x;
                                        bad = true;
                                    }
                                }
                            }
                        }
                    }
                    if (!ok) break;
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                }
                ptx::tmem_wait_st();
                ptx::tc_fence_before();
                ptx::mbar_arrive(&sh->p_ready[b]);
            }
            if (!ok) break;
            gt += n;
            consumed += 2 * NC * n;
            // The row's sum: all softmax warps meet once a part.
            if (active) {
                meet();  // (the partner has read the maxima)
                if (!ok) break;
                sh->half[side][r] = sum;
            }
            if (bad) sh->bad = part + 1;
            ptx::mbar_arrive(&sh->join);
            ok = warp_wait(&sh->join, joined++, abort, budget);
            if (!ok) break;
            sum = *(volatile float*)&sh->half[0][r] + *(volatile float*)&sh->half[1][r];
            // was there an infinity or a NaN among the values of this part?  (a later part's mark only costs a look)
            const bool edges = p.causal && w.j1 * kKeys > lim_first && lim_first < w.end;
            bad = edges && *(volatile int*)&sh->bad >= part + 1;

            // ---- epilogue
            const bool whole = w.j0 == 0 && w.j1 == w.tiles;
            ok = warp_wait(&sh->pv_done[(gt - 1) % C::NB], (gt - 1) / C::NB, abort, budget);
            if (!ok) break;
            ptx::tc_fence_after();
            const long long token = w.q.row0 + w.qt * p.tile_tokens + my_token;
            const int head = w.head * p.group + my_head;
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            if (active) {
                const bool drained = n > G && valid;
                const float f = drained_by();
                float4 x[4] = {};
                if (drained) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) x[k] = __ldcg(ws_o + k * ws_col);
                }
#pragma unroll 1
                for (int c = 0; c < HALF; c += 16) {
                    float o[16];
                    const int dim0 = side * HALF + c;
                    ptx::tmem_ld16(out_col + c, o);
                    ptx::tmem_wait_ld();
                    ptx::tmem_landed(o);
                    if (drained) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            o[4 * k] = fmaf(x[k].x, f, o[4 * k]);
                            o[4 * k + 1] = fmaf(x[k].y, f, o[4 * k + 1]);
                            o[4 * k + 2] = fmaf(x[k].z, f, o[4 * k + 2]);
                            o[4 * k + 3] = fmaf(x[k].w, f, o[4 * k + 3]);
                            if (c + 16 < HALF) x[k] = __ldcg(ws_o + ((c + 16) / 4 + k) * ws_col);
                        }
                    }
                    if (FEW) {
                        // the digits' products, smallest first
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const float second = __shfl_down_sync(0xffffffffu, o[k], kFewRows);
                            const float third = kFewDigits<T> > 2 ? __shfl_down_sync(0xffffffffu, o[k], 2 * kFewRows) : 0.f;
                            o[k] += second + third;
                        }
                    }
                    if (bad && valid) {
#pragma unroll 1
                        for (int key = max(lim_first, w.j0 * kKeys); key < min(lim, w.j1 * kKeys); ++key) {
                            const int page = p.batch.table[w.seq * p.batch.table_stride + page_at(p, key)];
                            if (page < 0 || page >= p.pages) continue;
                            const T* v = static_cast<const T*>(p.v_pool) + page * p.page_stride +
                                         slot_at(p, key) * p.slot_stride + w.head * p.head_stride;
#pragma unroll
                            for (int k = 0; k < 16; ++k) {
                                const float x = dim0 + k < p.dim ? to_f32(v[dim0 + k]) : 0.f;
                                if (!isfinite(x)) o[k] += x;
                            }
                        }
                    }
                    if (valid && digit == 0) {
                        if (!whole) {
#pragma unroll
                            for (int k = 0; k < 16; k += 4)
                                __stcg(ws_o + (c + k) / 4 * ws_col, make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]));
                        } else {
                            // eight elements at a time: 32 bytes of an f32 row, 16 of a 16-bit one
                            const long long at = token * p.out_token + head * p.out_head + dim0;
#pragma unroll
                            for (int k = 0; k < 16; k += 8) {
                                if (dim0 + k >= p.dim) break;
                                if (F32OUT) {
                                    float* out = static_cast<float*>(p.out) + at + k;
#pragma unroll
                                    for (int j = 0; j < 8; j += 4)
                                        *reinterpret_cast<float4*>(out + j) = make_float4(o[k + j] * inv, o[k + j + 1] * inv,
                                                                                          o[k + j + 2] * inv, o[k + j + 3] * inv);
                                } else {
                                    *reinterpret_cast<uint4*>(static_cast<T*>(p.out) + at + k) =
                                        make_uint4(pack2<T>(o[k] * inv, o[k + 1] * inv), pack2<T>(o[k + 2] * inv, o[k + 3] * inv),
                                                   pack2<T>(o[k + 4] * inv, o[k + 5] * inv), pack2<T>(o[k + 6] * inv, o[k + 7] * inv));
                                }
                            }
                        }
                    }
                    __syncwarp();
                }
            }
            ptx::tc_fence_before();
            ptx::mbar_arrive(&sh->o_free);
            if (whole) {
                if (valid && side == 0 && digit == 0 && p.lse)
                    p.lse[token * p.heads + head] = sum == 0.f ? -INFINITY : 0.6931471805599453f * (base + log2f(sum));
                continue;
            }

            // ---- a part of an item: the last one to arrive joins them
            if (valid && side == 0 && digit == 0)
                __stcg(reinterpret_cast<float2*>(p.ws_ml) + slot * kRows + r, make_float2(sum == 0.f ? -INFINITY : base, sum));
            const int from = cta_of(start, w.line + p.item_extra);
            const int to = cta_of(start, w.line + p.item_extra + w.tiles - 1);
            const int parts = to - from + 1;
            ptx::mbar_arrive(&sh->join);
            ok = warp_wait(&sh->join, joined++, abort, budget);
            if (!ok) break;
            if (threadIdx.x == 0) {
                // (carries what the other threads wrote before they met, and brings
                // what the other CTAs' threads wrote before theirs)
                sh->last = ptx::atom_add_acq_rel(&p.tickets[from], 1) == parts - 1;
                if (sh->last) p.tickets[from] = 0;
            }
            ptx::mbar_arrive(&sh->join);
            ok = warp_wait(&sh->join, joined++, abort, budget);
            if (!ok) break;
            if (*(volatile int*)&sh->last) {
                const int rows = tokens * p.group;
                const long long tok0 = w.q.row0 + w.qt * p.tile_tokens;
                // the first part lies in its CTA's second slot, the others in their first
                auto slot_of = [&](int k) { return 2LL * (from + k) + (k == 0 ? 1 : 0); };
                float2* ml = reinterpret_cast<float2*>(p.ws_ml);
                const float4* parts_o = reinterpret_cast<const float4*>(p.ws_o);
                auto weight = [&](float2 x, float ref) { return x.y == 0.f ? 0.f : ptx::ex2(x.x - ref); };
                auto write_lse = [&](int row, float ref, float total) {
                    const int tk = row / p.group;
                    p.lse[(tok0 + tk) * p.heads + w.head * p.group + row - tk * p.group] =
                        total == 0.f ? -INFINITY : 0.6931471805599453f * (ref + log2f(total));
                };
                // A part without a key holds zeros; one whose weight underflows against
                // another's is added all the same, so that a NaN or an infinity in it
                // reaches the output wherever the item was cut.
                auto add = [&](float4& acc, float x, float4 o) {
                    acc = make_float4(fmaf(x, o.x, acc.x), fmaf(x, o.y, acc.y), fmaf(x, o.z, acc.z), fmaf(x, o.w, acc.w));
                };
                auto write_out = [&](int row, int c, float4 v) {
                    if (4 * c >= p.dim) return;
                    const int tk = row / p.group;
                    const long long at = (tok0 + tk) * p.out_token + (w.head * p.group + row - tk * p.group) * p.out_head + 4 * c;
                    if (F32OUT) *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = v;
                    else *reinterpret_cast<uint2*>(static_cast<T*>(p.out) + at) = make_uint2(pack2<T>(v.x, v.y), pack2<T>(v.z, v.w));
                };
                const float2 none = make_float2(-INFINITY, 0.f);
                if (!by_row) {
                    // Many rows: a lane takes a row and an eighth of its columns.
                    constexpr int kCols = DP / 32;
                    for (int u = threadIdx.x; u < 8 * kRows; u += kSoftmax) {
                        const int row = u & (kRows - 1), c0 = (u / kRows) * kCols;
                        if (row >= rows) continue;
                        float top = -INFINITY, total = 0.f;
#pragma unroll 4
                        for (int k = 0; k < parts; ++k) top = fmaxf(top, __ldcg(ml + slot_of(k) * kRows + row).x);
                        const float ref = top == -INFINITY ? 0.f : top;
                        float4 acc[kCols] = {};
                        for (int k = 0; k < parts; ++k) {
                            const float2 x = __ldcg(ml + slot_of(k) * kRows + row);
                            float4 o[kCols];
#pragma unroll
                            for (int c = 0; c < kCols; ++c) o[c] = __ldcg(parts_o + (slot_of(k) * (DP / 4) + c0 + c) * kRows + row);
                            const float f = weight(x, ref);
                            total += f * x.y;
#pragma unroll
                            for (int c = 0; c < kCols; ++c) add(acc[c], f, o[c]);
                        }
                        const float scale = total == 0.f ? 0.f : 1.f / total;
#pragma unroll
                        for (int c = 0; c < kCols; ++c)
                            write_out(row, c0 + c, make_float4(acc[c].x * scale, acc[c].y * scale, acc[c].z * scale, acc[c].w * scale));
                        if (p.lse && c0 == 0) write_lse(row, ref, total);
                    }
                } else {
                    // A few rows of many parts (single tokens over a long context): a
                    // warp takes a row, its lanes first the parts, then the columns.
                    for (int row = warp; row < rows; row += kSoftmax / 32) {
                        const float2 x0 = lane < parts ? __ldcg(ml + slot_of(lane) * kRows + row) : none;
                        float top = x0.x;
                        for (int k = lane + 32; k < parts; k += 32) top = fmaxf(top, __ldcg(ml + slot_of(k) * kRows + row).x);
#pragma unroll
                        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                        const float ref = top == -INFINITY ? 0.f : top;
                        constexpr int V = DP <= 128 ? 1 : DP / 128;  // float4 columns of a lane
                        constexpr int kBatch = 8 / V;                // parts in flight
                        float total = 0.f;
                        float4 acc[V] = {};
                        for (int k0 = 0; k0 < parts; k0 += 32) {
                            const float2 x = k0 == 0 ? x0 : k0 + lane < parts ? __ldcg(ml + slot_of(k0 + lane) * kRows + row) : none;
                            const float mine = weight(x, ref);
                            total += mine * x.y;
                            for (int k = 0; k < min(32, parts - k0); k += kBatch) {
                                float4 o[kBatch][V];
#pragma unroll
                                for (int j = 0; j < kBatch; ++j)
#pragma unroll
                                    for (int v = 0; v < V; ++v)
                                        if (k0 + k + j < parts && lane + 32 * v < DP / 4)
                                            o[j][v] = __ldcg(parts_o + (slot_of(k0 + k + j) * kRows + row) * (DP / 4) + lane + 32 * v);
#pragma unroll
                                for (int j = 0; j < kBatch; ++j) {
                                    const float f = __shfl_sync(0xffffffffu, mine, k + j);
#pragma unroll
                                    for (int v = 0; v < V; ++v)
                                        if (k0 + k + j < parts && lane + 32 * v < DP / 4) add(acc[v], f, o[j][v]);
                                }
                            }
                        }
#pragma unroll
                        for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
                        const float scale = total == 0.f ? 0.f : 1.f / total;
#pragma unroll
                        for (int v = 0; v < V; ++v)
                            if (lane + 32 * v < DP / 4)
                                write_out(row, lane + 32 * v, make_float4(acc[v].x * scale, acc[v].y * scale, acc[v].z * scale, acc[v].w * scale));
                        if (p.lse && lane == 0) write_lse(row, ref, total);
                    }
                }
            }
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (threadIdx.x == 0 && sh->abort) *p.timed_out = 1;
    if (warp == kMmaWarp) ptx::tmem_dealloc(tmem, kTmemCols);
}

template <int DP, typename T, bool F32OUT, bool FEW>
cudaError_t load()
{
    static PerDeviceOnce once;
    int dev = 0;
    return once.run(&dev, [](int) {
        return cudaFuncSetAttribute(bitlin_attend<DP, T, F32OUT, FEW>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<DP>());
    });
}

template <int DP, typename T, bool F32OUT, bool FEW>
cudaError_t launch(const AttendParams& p, const void* tmap_q, const void* tmap_k, const void* tmap_v, int num_sms, cudaStream_t s)
{
    const cudaError_t e = load<DP, T, F32OUT, FEW>();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(num_sms);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem_bytes<DP>();
    cfg.stream = s;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, bitlin_attend<DP, T, F32OUT, FEW>, *static_cast<const CUtensorMap*>(tmap_q),
                              *static_cast<const CUtensorMap*>(tmap_k), *static_cast<const CUtensorMap*>(tmap_v), p);
}

template <typename T, bool F32OUT, bool FEW>
cudaError_t pick_dim(const AttendParams& p, const void* tmap_q, const void* tmap_k, const void* tmap_v, int num_sms,
                     cudaStream_t s)
{
    if (p.dim <= 64) return launch<64, T, F32OUT, FEW>(p, tmap_q, tmap_k, tmap_v, num_sms, s);
    if (p.dim <= 128) return launch<128, T, F32OUT, FEW>(p, tmap_q, tmap_k, tmap_v, num_sms, s);
    return launch<256, T, F32OUT, FEW>(p, tmap_q, tmap_k, tmap_v, num_sms, s);
}

template <typename T>
cudaError_t pick_output(const AttendParams& p, int out_dtype, const void* tmap_q, const void* tmap_k, const void* tmap_v,
                        int num_sms, cudaStream_t s)
{
    if (out_dtype != BITLIN_F32) return pick_dim<T, false, false>(p, tmap_q, tmap_k, tmap_v, num_sms, s);
    return p.few ? pick_dim<T, true, true>(p, tmap_q, tmap_k, tmap_v, num_sms, s)
                 : pick_dim<T, true, false>(p, tmap_q, tmap_k, tmap_v, num_sms, s);
}

template <int DP, typename T>
cudaError_t load_outputs()
{
    cudaError_t e = load<DP, T, false, false>();
    if (e == cudaSuccess) e = load<DP, T, true, false>();
    if (e == cudaSuccess) e = load<DP, T, true, true>();
    return e;
}

template <typename T>
cudaError_t load_dim(int dim)
{
    return dim <= 64 ? load_outputs<64, T>() : dim <= 128 ? load_outputs<128, T>() : load_outputs<256, T>();
}

int gcd(int a, int b) { return b ? gcd(b, a % b) : a; }

}  // namespace

void bitlin_attend_boxes(int dim, int page_size, int* box_k, int* box_v)
{
    const int padded = dim <= 64 ? 64 : dim <= 128 ? 128 : 256;
    *box_k = gcd(page_size, kKeys);
    *box_v = gcd(page_size, 8192 / padded);
}

// Measured, in us, at 0/1/2/3/4/6: 4 prompts of 700-4,096 tokens at 64 dims
// 335/290/257/232/233/245, at 128 414/355/315/284/262/277, at 256
// 487/399/357/321/328/345; 4 chunks of 512 tokens over 4,096 keys at 256 dims
// 183 at 2, 182 at 3, 188 at 4; a prompt of 4,000 beside 15 single tokens at 256
// dims 239 at 2, 206 at 3, 210 at 4.  64 single tokens at 64/128/256 dims 168/191/167
// without, 134/187/166 at 3, 135/186/166 at 4.  One long chunk or one token: no
// difference past the spread.
int bitlin_attend_item_extra(int dim) { return dim > 128 ? 3 : 4; }

KvWorkspaceParts bitlin_attend_workspace(int dim, int num_sms)
{
    const size_t padded = dim <= 64 ? 64 : dim <= 128 ? 128 : 256;
    const size_t rows = (size_t)2 * num_sms * kRows;
    KvWorkspaceParts w;
    w.timed_out = num_sms * sizeof(int);
    w.ml = (w.timed_out + sizeof(int) + 255) / 256 * 256;
    w.o = w.ml + rows * 2 * sizeof(float);
    w.bytes = w.o + rows * padded * sizeof(float);
    return w;
}

void bitlin_attend_rows(int tokens, int seqs, int group, int out_dtype, int* tile_tokens, int* q_box, int* few_rows)
{
    // An f32 output of a few rows a sequence: room for every digit in the tile.  The
    // lengths lie on the device: as many tokens as sequences are taken for one each
    // (another spread of them takes more tiles, each of which reads its keys).
    *few_rows = out_dtype == BITLIN_F32 && group <= kFewRows && (tokens == seqs || tokens <= kFewRows / group);
    if (*few_rows) {
        *tile_tokens = *q_box = kFewRows / group;
        return;
    }
    // A tile's rows in one box where sequences bring many tokens; where they
    // bring few, boxes of the fewest tokens whose rows keep the swizzle's atoms
    // of eight, so that single tokens do not fetch their neighbours' rows.  The
    // boxes can cost the tile rows (21 tokens of 6 heads become 20).  Measured, in
    // us, one box and boxes, at 256 dims, 6 heads to a key head: prompts of 700-4,096
    // tokens 359 and 364, 2,048 tokens over 32,768 keys 1,170 and 1,219; 15 single
    // tokens beside a prompt of 4,000, which the average below takes for many, 239
    // and 231; 64 single tokens 165.3 and 165.0.  At 64 and 128 dims all within 0.5 %.
    *tile_tokens = kRows / group;
    *q_box = *tile_tokens;
    const int few = 8 / gcd(group, 8);
    if (few < *tile_tokens && tokens / seqs < *tile_tokens) {
        *q_box = few;
        *tile_tokens -= *tile_tokens % few;
    }
}

cudaError_t bitlin_attend_load(int dim, int dtype)
{
    return dtype == BITLIN_BF16 ? load_dim<__nv_bfloat16>(dim) : load_dim<__half>(dim);
}

cudaError_t bitlin_launch_attend(const AttendParams& p, int dtype, int out_dtype, const void* tmap_q,
                                 const void* tmap_k, const void* tmap_v, int num_sms, cudaStream_t s)
{
    return dtype == BITLIN_BF16 ? pick_output<__nv_bfloat16>(p, out_dtype, tmap_q, tmap_k, tmap_v, num_sms, s)
                                : pick_output<__half>(p, out_dtype, tmap_q, tmap_k, tmap_v, num_sms, s);
}
