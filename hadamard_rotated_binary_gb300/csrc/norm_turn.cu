// A norm of each head with its rotation in the same pass, the append of such
// rows to a paged cache in 16 or 4 bits, and the gradient.
//
// Mathematics: n = x / sqrt(mean(x^2) + eps), y = R (w * n) with R the rotation
// of pairs by their positions (see rope.cu).  Backwards, with g = R^T dy and
// h = w * g: dx = r (h - n mean(h n)), r = 1 / sqrt(mean(x^2) + eps), and
// dw = sum over rows of g * n.
//
// Bound: HBM; each element is read once and written once.  A team of 8 to 32
// lanes holds a row: a lane owns two chunks of four elements, half the rotated
// (or the passed-through) part apart, so pairs stay in a thread; the sum of
// squares is five shuffles at most.  A team takes four heads of a token: the
// angles are computed once for them and their loads are in flight together, from
// before the token's place is looked up (loads after it: 36.6 us for 31.5 below).
// Where sizes, strides or alignment do not allow chunks, a lane takes up to four
// pairs of single elements: 2.5 times as long (8,192 x 16 x 80 bf16, 16 or 80 of 80
// rotated 14.2 us, 20 of 80 35.7).
//
// In 4 bits the codes are those of the exact real-valued row, whatever the order
// of the kernel's sums: a row is computed in 32 bits with a bound on its error
// (24 units of 2^-24 of |a| + |b|: sum of squares 9 / 2, rsqrt 4, products 2,
// angle, sine and cosine 4, rotation 2), and an element (or a group's scale)
// that lies within it of a border between two codes is computed again in 64 bits,
// one row in 500 to 900 of normal ones (counted with these bounds); so is a row whose squares
// leave the range of 32 bits.  Rows
// that neither a norm nor a rotation touches are exact.
// There a lane ends with eight consecutive elements (pairs half the rotated part
// apart go through shared memory), and a team takes several heads one after the
// other where there are tokens enough: what comes before a row, and its place,
// costs more than the row.
//
// Measured (GB300, inputs changing from call to call; four and eight heads to a team,
// two, in brackets): queries of 8,191 tokens, 32 heads of 128, bf16, 27.7 us (4.9 TB/s;
// 41, 38, before 16-bit chunks were taken apart by words); 4,097 x 24 x 256 f32 33.0 us
// (6.1 TB/s), its gradient 50 us (6.0 TB/s; two heads at a time 53, blocks of 128 whose
// sums are 608 rows to join 51); prompts of 8,191 tokens to 4 bits with their queries
// and read back 77 us, issue at 80 % of its rate, with 72 registers of a thread (64 the
// same, 96 eight to eleven more; with single elements 72 to 84 bytes of a thread spill).
// One token's queries 2.1 us in a graph.
#include "kv_internal.cuh"
#include "ptx.cuh"
#include "quant.cuh"

using namespace bitlin_impl;

namespace {

constexpr int kThreads = 128;
constexpr int kHeadsPerTeam = 4;
constexpr int kMaxDim = 256;
constexpr int kGradHeads = 4;     // heads that a team of the gradient takes
constexpr int kGradThreads = 256; // two blocks on an SM, the sums of each a row to join
constexpr float kRowError = 24.f * 5.9604645e-8f;

template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Chunk {
    T v[VEC];
};

// A chunk's elements, 16-bit ones two by two.
template <typename T, int VEC>
__device__ __forceinline__ void unpack(const Chunk<T, VEC>& c, float (&x)[VEC])
{
#pragma unroll
    for (int j = 0; j < VEC; ++j) x[j] = to_f32(c.v[j]);
}
template <>
__device__ __forceinline__ void unpack(const Chunk<__nv_bfloat16, 4>& c, float (&x)[4])
{
    const uint2 w = *reinterpret_cast<const uint2*>(&c);
    x[0] = __uint_as_float(w.x << 16);
    x[1] = __uint_as_float(w.x & 0xffff0000u);
    x[2] = __uint_as_float(w.y << 16);
    x[3] = __uint_as_float(w.y & 0xffff0000u);
}
template <>
__device__ __forceinline__ void unpack(const Chunk<__half, 4>& c, float (&x)[4])
{
    const uint2 w = *reinterpret_cast<const uint2*>(&c);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&w.x)), b = __half22float2(*reinterpret_cast<const __half2*>(&w.y));
    x[0] = a.x;
    x[1] = a.y;
    x[2] = b.x;
    x[3] = b.y;
}
template <typename T, int VEC>
__device__ __forceinline__ Chunk<T, VEC> pack(const float (&x)[VEC])
{
    Chunk<T, VEC> c;
#pragma unroll
    for (int j = 0; j < VEC; ++j) c.v[j] = from_f32<T>(x[j]);
    return c;
}
template <>
__device__ __forceinline__ Chunk<__nv_bfloat16, 4> pack(const float (&x)[4])
{
    const __nv_bfloat162 w[2] = {__floats2bfloat162_rn(x[0], x[1]), __floats2bfloat162_rn(x[2], x[3])};
    return *reinterpret_cast<const Chunk<__nv_bfloat16, 4>*>(w);
}
template <>
__device__ __forceinline__ Chunk<__half, 4> pack(const float (&x)[4])
{
    const __half2 w[2] = {__floats2half2_rn(x[0], x[1]), __floats2half2_rn(x[2], x[3])};
    return *reinterpret_cast<const Chunk<__half, 4>*>(w);
}

__device__ __forceinline__ float team_sum(float v, int team)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const float other = __shfl_xor_sync(0xffffffffu, v, o);
        v += o < team ? other : 0.f;
    }
    return v;
}

__device__ __forceinline__ double team_sum(double v, int team)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        if (o < team) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Where unit u of a row has its two chunks of VEC elements.
template <int VEC>
struct Unit {
    int lo, hi;
    bool held, has_hi, turns;  // in the row at all; its second chunk; inside the rotated part
};

template <int VEC>
__device__ __forceinline__ Unit<VEC> unit_of(int u, int dim, int rotary, int adjacent)
{
    Unit<VEC> x;
    const int rotated = rotary / 2 / VEC;
    x.turns = u < rotated;
    if (VEC > 1) {
        x.lo = x.turns ? u * VEC : rotary + (u - rotated) * VEC;
        x.hi = x.lo + (x.turns ? rotary : dim - rotary) / 2;
        x.held = u < dim / (2 * VEC);
        x.has_hi = x.held;
    } else {
        x.lo = x.turns ? (adjacent ? 2 * u : u) : rotary + 2 * (u - rotated);
        x.hi = x.turns && !adjacent ? x.lo + rotary / 2 : x.lo + 1;
        x.held = x.lo < dim;
        x.has_hi = x.hi < dim;
    }
    return x;
}

// Pair of the unit's element j.
template <int VEC>
__device__ __forceinline__ int pair_of(const Unit<VEC>& x, int u, int j, int adjacent)
{
    if (!adjacent) return x.lo + j;
    return VEC == 1 ? u : j < VEC / 2 ? x.lo / 2 + j : x.hi / 2 + j - VEC / 2;
}

// The angle of a pair as a fraction of a turn in 2^-64, signed.
__device__ __forceinline__ long long fraction(Turn w, const int32_t* pos, int tokens, int t, int place)
{
    const int axis = (int)(w & kAxisMask);
    const long long at = pos ? pos[(long long)axis * tokens + t] : place;
    return (long long)((uint64_t)at * (w & ~kAxisMask));
}

template <int VEC>
__device__ __forceinline__ void rotate(float (&x)[VEC], float (&y)[VEC], const float (&cs)[VEC], const float (&sn)[VEC], int adjacent)
{
    if (VEC > 1 && adjacent) {
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) {
            const int k = VEC / 2 + j, e = 2 * j < VEC ? 2 * j : 0, f = e + 1 < VEC ? e + 1 : 0;
            const float x0 = x[e], x1 = x[f], y0 = y[e], y1 = y[f];
            x[e] = x0 * cs[j] - x1 * sn[j];
            x[f] = x1 * cs[j] + x0 * sn[j];
            y[e] = y0 * cs[k] - y1 * sn[k];
            y[f] = y1 * cs[k] + y0 * sn[k];
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

// Elements of |a| + |b| of each output of a pair.
template <int VEC>
__device__ __forceinline__ void sizes(const float (&x)[VEC], const float (&y)[VEC], float (&ex)[VEC], float (&ey)[VEC], bool turning, int adjacent)
{
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        if (!turning) {
            ex[j] = fabsf(x[j]);
            ey[j] = fabsf(y[j]);
        } else if (VEC > 1 && adjacent) {
            ex[j] = fabsf(x[j]) + fabsf(x[j ^ 1]);
            ey[j] = fabsf(y[j]) + fabsf(y[j ^ 1]);
        } else {
            ex[j] = ey[j] = fabsf(x[j]) + fabsf(y[j]);
        }
    }
}

// One row's value of element d in 64 bits.
template <typename TI>
struct Exact {
    const TI* row;
    const float* weight;
    const Turn* turns;  // nullptr: not rotated
    const int32_t* pos;
    double r;
    int tokens, t, place, rotary, adjacent;

    __device__ double normed(int d) const
    {
        const double x = (double)to_f32(row[d]);
        return weight ? x * r * (double)weight[d] : x;
    }
    __device__ double operator()(int d) const
    {
        double v;
        if (!turns || d >= rotary) {
            v = normed(d);
        } else {
            const int half = rotary / 2;
            const int f = adjacent ? d >> 1 : d < half ? d : d - half;
            const bool first = adjacent ? !(d & 1) : d < half;
            const int other = adjacent ? d ^ 1 : first ? d + half : d - half;
            double sn, cs;
            sincospi((double)fraction(turns[f], pos, tokens, t, place) * 0x1p-63, &sn, &cs);
            v = normed(d) * cs + (first ? -sn : sn) * normed(other);
        }
        return v == v ? v : 0.0;  // a NaN is stored as zero
    }
};

// Codes of a lane's 8 elements d0.. and their group's scale in 64 bits: of the elements in
// `doubt` alone, or, where the scale itself is in doubt (`which`, the same for all lanes of a
// group), of all.  The whole warp takes part.
struct Codes {
    uint32_t word, scale;
};
template <typename TI>
__device__ __noinline__ Codes codes_again(Codes c, Exact<TI> e, uint32_t doubt, bool which, bool active, int d0, int dim, int team, double eps)
{
    const int width = dim / 32;
    double sum = 0;
    if (active)
        for (int j = 0; j < 8; ++j) {
            const double v = (double)to_f32(e.row[d0 + j]);
            sum += v * v;
        }
    sum = team_sum(sum, team);
    e.r = 1.0 / sqrt(sum / dim + eps);
    double top = 0;
    if (which) {
#pragma unroll 1
        for (int j = 0; j < 8; ++j) top = fmax(top, fabs(e(d0 + j)));
    }
#pragma unroll
    for (int o = 4; o; o >>= 1)
        if (o < width) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (which) {
        c.scale = quant_scale_code(top);
        doubt = c.scale ? 0xffu : 0u;
        if (!c.scale) c.word = 0x88888888u;
    }
    const double s = (double)quant_scale(c.scale);
    for (int j = 0; doubt; ++j, doubt >>= 1) {
        if (!(doubt & 1)) continue;
        const double code = fmin(fmax(rint(e(d0 + j) / s), -7.0), 7.0);
        c.word = (c.word & ~(0xfu << (4 * j))) | (uint32_t)((int)code + 8) << (4 * j);
    }
    __syncwarp();
    return c;
}

// Store a row's 8 elements d0.. of each lane u < D / 8 in 4 bits.  x: the values, size: |a| + |b|
// of each, kRowError of which it may be off (EXACT: nothing; `far`: anything).  All lanes of the
// warp take part.
//
// x / s comes from a product and one correction by its rest (Newton's iteration, as for
// 1 / s), which for 16-bit values lies on the right side of every border (and on the
// border itself where x / s does); an f32 value's rest x - c s, which is exact, decides.
// Adding 1.5 2^23 + 8 rounds to the nearest (ties to even) and leaves code + 8 in the low
// bits.
template <typename TI, bool EXACT, typename Again>
__device__ __forceinline__ void store_codes(float (&x)[8], const float (&size)[8], bool far, bool active, int u, int dim, int team, Again again,
                                            double eps, uint8_t* codes, uint8_t* scales)
{
    constexpr float kRound = 12582912.f + 8.f;
    const int d0 = 8 * u, width = dim / 32;  // lanes of a group: 2, 4 or 8
    float amax = 0.f, emax = 0.f, finite = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        finite = fmaf(x[j], 0.f, finite);
        amax = fmaxf(amax, fabsf(x[j]));
        if (!EXACT) emax = fmaxf(emax, size[j]);
    }
    if (finite != 0.f) {  // (an infinity or a NaN, which is stored as zero)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (x[j] != x[j]) x[j] = 0.f;
    }
#pragma unroll
    for (int o = 4; o; o >>= 1) {
        const int lane = o < width ? o : 0;  // (0: its own)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, lane));
        if (!EXACT) emax = fmaxf(emax, __shfl_xor_sync(0xffffffffu, emax, lane));
    }
    Codes c;
    c.scale = quant_scale_code(amax);
    const float s = quant_scale(c.scale), half = 0.5f * s, limit = 7.25f * s;
    float inv = ptx::rcp(s);  // 1 / s, corrected once
    inv = s > 0.f ? fmaf(fmaf(-s, inv, 1.f), inv, inv) : 0.f;
    float near = 0.f;  // the largest distance from a code, with its error
    uint32_t bits = 0;
#pragma unroll
    for (int j = 7; j >= 0; --j) {
        x[j] = fminf(fmaxf(x[j], -limit), limit);  // (the same code, 7 or -7)
        float q = x[j] * inv;
        q = fmaf(fmaf(-q, s, x[j]), inv, q) + kRound;
        if (!EXACT || sizeof(TI) == 4) {
            const float rest = fabsf(fmaf(kRound - q, s, x[j]));
            near = fmaxf(near, EXACT ? rest : fmaf(size[j], kRowError, rest));
        }
        bits = bits * 16 + __float_as_uint(q);
    }
    // (the sum of the 1.5 2^23s, which the low bits of each stand above)
    constexpr uint32_t kBias = 0x4b400000u * 0x11111111u;
    c.word = bits - kBias;
    if (EXACT && sizeof(TI) == 4) {
        // an f32 value nearer to a border than its quotient's rounding: decided by its rest
        if (near >= half && s > 0.f) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float code = (float)((int)(c.word >> (4 * j) & 15) - 8);
                const float rest = fmaf(-code, s, x[j]);
                if (fabsf(rest) > half || (fabsf(rest) == half && ((int)code & 1))) code += rest > 0.f ? 1.f : -1.f;
                c.word = (c.word & ~(0xfu << (4 * j))) | (uint32_t)((int)code + 8) << (4 * j);
            }
        }
    }
    if (!EXACT) {
        // Does a border lie within an element's error, or between two scales within the largest's?
        emax *= kRowError;
        const float above = 3.5f * (s + quant_scale(c.scale + 1)), below = c.scale ? 3.5f * (s + quant_scale(c.scale - 1)) : -1.f;
        // (an infinite largest with an infinite error, where root times weight overflows, tells nothing either)
        const bool which = active && (far || (amax + emax >= above && c.scale < kQuantTopScale) || !(amax - emax > below));
        if (__any_sync(0xffffffffu, active && (which || (near >= half && s > 0.f)))) {
            uint32_t doubt = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float rest = fmaf(-(float)((int)(c.word >> (4 * j) & 15) - 8), s, x[j]);
                if (fmaf(size[j], kRowError, fabsf(rest)) >= half) doubt |= 1u << j;
            }
            if (!active || s == 0.f) doubt = 0;
            c = codes_again<TI>(c, again(), doubt, which, active, d0, dim, team, eps);
        }
    }
    if (active) {
        *reinterpret_cast<uint32_t*>(codes + d0 / 2) = c.word;
        if ((u & (width - 1)) == 0) scales[u / width] = (uint8_t)c.scale;
    }
}

// Where a token's row of k or v goes: its place in its sequence, its page and slot.
struct Home {
    int place, page, slot;
    bool active;  // false: padding, or no place in the pool
};
// All lanes of a warp take part, with ascending tokens.
__device__ __forceinline__ Home home_of(const TurnParams& p, int t, bool active, bool pages)
{
    Home r = {0, 0, 0, active};
    if (!p.append) return r;
    if (!pages && p.pos) {  // a row of q needs no place: is it padding?
        r.active = active && t < p.batch.q_offsets[p.batch.seqs];
        return r;
    }
    const int first = __shfl_sync(0xffffffffu, t, 0);
    int seq = warp_sequence_of(p.batch, first);
    while (seq < p.batch.seqs && p.batch.q_offsets[seq + 1] <= t) ++seq;
    if (seq >= p.batch.seqs) {
        r.active = false;
        return r;
    }
    r.place = p.batch.kv_lens[seq] - (p.batch.q_offsets[seq + 1] - t);
    if (!pages || !active) return r;
    const int at = r.place / p.page_size;
    r.page = -1;
    if (r.place >= 0 && at < p.batch.table_pages) r.page = p.batch.table[seq * p.batch.table_stride + at];
    r.slot = r.place - at * p.page_size;
    if (r.page < 0 || r.page >= p.pages) {
        *p.index_error = 1;
        r.active = false;
    }
    return r;
}

// The k or v rows of heads h0 .. h1 - 1 of a token to a 4-bit cache: a lane ends with eight
// consecutive elements of a row.  It starts with them too, unless pairs lie half the rotated
// part apart: those are rotated in two chunks and go through shared memory.
template <typename TI, int VEC>
__device__ __forceinline__ void quant_rows(const NormTurnParams& np, int kind, int h0, int h1, int t, bool token, float* values, float* errors)
{
    constexpr int NU = VEC == 1 ? 4 : 1;
    const TurnParams& p = np.t;
    const int u0 = threadIdx.x & (np.team - 1);
    const float* weight = kind == 2 ? nullptr : np.weight[1];
    const bool rotating = p.turns != nullptr && kind != 2;
    const bool apart = VEC == 1 || (rotating && !p.adjacent);
    const bool exact = !weight && !rotating;

    Unit<VEC> unit[NU];
#pragma unroll
    for (int i = 0; i < NU; ++i) {
        const int u = u0 + 32 * i;
        unit[i] = unit_of<VEC>(u, p.dim, p.rotary, p.adjacent);
        if (!apart) {
            unit[i].lo = 8 * u;
            unit[i].hi = 8 * u + 4;
            unit[i].turns = 8 * u < p.rotary;
        }
        unit[i].turns = unit[i].turns && rotating;
        unit[i].held = unit[i].held && token;
        unit[i].has_hi = unit[i].has_hi && token;
    }
    Chunk<TI, VEC> a[NU] = {}, b[NU] = {};
    const long long src_head = p.src_head[kind], code_head = p.head_stride, scale_head = np.scale_head;
    const TI* row = static_cast<const TI*>(p.src[kind]) + t * p.src_token[kind] + h0 * src_head;
    auto load = [&]() {
#pragma unroll
        for (int i = 0; i < NU; ++i) {
            if (unit[i].held) a[i] = *reinterpret_cast<const Chunk<TI, VEC>*>(row + unit[i].lo);
            if (unit[i].has_hi) b[i] = *reinterpret_cast<const Chunk<TI, VEC>*>(row + unit[i].hi);
        }
        row += src_head;
    };
    load();
    float cs[NU][VEC], sn[NU][VEC], wx[NU][VEC], wy[NU][VEC];
#pragma unroll
    for (int i = 0; i < NU; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            wx[i][j] = weight && unit[i].held ? weight[unit[i].lo + j] : 1.f;
            wy[i][j] = weight && unit[i].has_hi ? weight[unit[i].hi + j] : 1.f;
        }

    const Home home = home_of(p, t, token, true);
    if (__ballot_sync(0xffffffffu, home.active) == 0) return;
    const int place = home.place;
    const bool mine = home.active && u0 < p.dim / 8;
    uint8_t* codes = static_cast<uint8_t*>(p.pool[kind - 1]) + home.page * p.page_stride + home.slot * p.slot_stride + h0 * code_head;
    uint8_t* scales = np.scales[kind - 1] + home.page * np.scale_page + home.slot * np.scale_slot + h0 * scale_head;
#pragma unroll
    for (int i = 0; i < NU; ++i) {
        const int u = u0 + 32 * i;
        if (unit[i].held && unit[i].turns) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const int f = pair_of<VEC>(unit[i], u, j, p.adjacent);
                const int32_t frac = (int32_t)(fraction(p.turns[f], p.pos, p.tokens, t, place) >> 32);
                sincospif((float)frac * 4.656612873077393e-10f /* 2^-31: half turns */, &sn[i][j], &cs[i][j]);
            }
        }
    }
#pragma unroll 1
    for (int h = h0; h < h1; ++h, codes += code_head, scales += scale_head) {
        alignas(16) float x[NU][VEC], y[NU][VEC], ex[NU][VEC], ey[NU][VEC];
#pragma unroll
        for (int i = 0; i < NU; ++i) {
            unpack(a[i], x[i]);
            unpack(b[i], y[i]);
        }
        if (h + 1 < h1) load();
        bool far = false;  // the squares leave what 32 bits hold well
        if (weight) {
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < NU; ++i) {
                float part = 0.f;
#pragma unroll
                for (int j = 0; j < VEC; ++j) part += fmaf(x[i][j], x[i][j], y[i][j] * y[i][j]);
                sum += part;
            }
            sum = team_sum(sum, np.team);
            const float mean = fmaf(sum, np.inverse_dim, np.eps_f), r = rsqrtf(mean);
            far = !(sum <= 3e38f && mean >= 1e-30f);
#pragma unroll
            for (int i = 0; i < NU; ++i)
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    x[i][j] *= r * wx[i][j];
                    y[i][j] *= r * wy[i][j];
                }
        }
#pragma unroll
        for (int i = 0; i < NU; ++i) {
            sizes<VEC>(x[i], y[i], ex[i], ey[i], unit[i].turns, p.adjacent);
            if (unit[i].turns) rotate<VEC>(x[i], y[i], cs[i], sn[i], p.adjacent);
        }
        alignas(16) float v[8] = {}, e[8] = {};
        if (!apart) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[j] = x[0][j % VEC];
                v[4 + j] = y[0][j % VEC];
                e[j] = ex[0][j % VEC];
                e[4 + j] = ey[0][j % VEC];
            }
        } else {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < NU; ++i) {
                if (unit[i].held) {
                    *reinterpret_cast<Chunk<float, VEC>*>(values + unit[i].lo) = *reinterpret_cast<const Chunk<float, VEC>*>(x[i]);
                    *reinterpret_cast<Chunk<float, VEC>*>(errors + unit[i].lo) = *reinterpret_cast<const Chunk<float, VEC>*>(ex[i]);
                }
                if (unit[i].has_hi) {
                    *reinterpret_cast<Chunk<float, VEC>*>(values + unit[i].hi) = *reinterpret_cast<const Chunk<float, VEC>*>(y[i]);
                    *reinterpret_cast<Chunk<float, VEC>*>(errors + unit[i].hi) = *reinterpret_cast<const Chunk<float, VEC>*>(ey[i]);
                }
            }
            __syncwarp();
            if (mine) {
#pragma unroll
                for (int j = 0; j < 8; j += 4) {
                    *reinterpret_cast<float4*>(v + j) = *reinterpret_cast<const float4*>(values + 8 * u0 + j);
                    *reinterpret_cast<float4*>(e + j) = *reinterpret_cast<const float4*>(errors + 8 * u0 + j);
                }
            }
        }
        auto again = [&]() {
            const TI* mine = static_cast<const TI*>(p.src[kind]) + t * p.src_token[kind] + h * src_head;
            return Exact<TI>{mine, weight, rotating ? p.turns : nullptr, p.pos, 0.0, p.tokens, t, place, p.rotary, p.adjacent};
        };
        if (exact) store_codes<TI, true>(v, e, false, mine, u0, p.dim, np.team, again, np.eps, codes, scales);
        else store_codes<TI, false>(v, e, far, mine, u0, p.dim, np.team, again, np.eps, codes, scales);
    }
}

template <typename TI, typename TO, int VEC, bool QUANT>
__global__ void __launch_bounds__(kThreads, QUANT ? 7 : 1) bitlin_norm_turn(const NormTurnParams np)
{
    constexpr int NU = VEC == 1 ? 4 : 1;  // units of a lane
    __shared__ __align__(16) float buffer[QUANT ? kThreads / 32 : 1][2][QUANT ? kMaxDim : 4];
    ptx::griddep_wait();
    const TurnParams& p = np.t;
    const int lane = threadIdx.x & 31, u0 = lane & (np.team - 1);
    const uint32_t idx = blockIdx.x * (uint32_t)(kThreads / np.team) + threadIdx.x / (uint32_t)np.team;  // the team's token
    const int t = (int)min(idx, (uint32_t)(p.tokens - 1));
    const bool token = idx < (uint32_t)p.tokens;

    // k, v or q, and which heads of it (the blocks that take longest come first)
    int kind = 1, group = blockIdx.y;
    if (group >= p.kv_groups) {
        group -= p.kv_groups;
        kind = 2;
        if (group >= p.kv_groups) {
            group -= p.kv_groups;
            kind = 0;
        }
    }
    const int heads = kind == 0 ? p.heads : p.kv_heads;
    const int h0 = group * (QUANT && kind ? np.kv_heads_per_team : kHeadsPerTeam);
    if (QUANT && kind) {
        float* row = buffer[threadIdx.x >> 5][0] + lane / np.team * p.dim;
        quant_rows<TI, VEC>(np, kind, h0, min(h0 + np.kv_heads_per_team, heads), t, token, row, row + kMaxDim);
        return;
    }
    const TI* src = static_cast<const TI*>(p.src[kind]) + t * p.src_token[kind];
    const long long src_head = p.src_head[kind];
    const float* weight = kind == 2 ? nullptr : np.weight[kind];
    const bool rotating = p.turns != nullptr && kind != 2;

    Unit<VEC> unit[NU];
#pragma unroll
    for (int i = 0; i < NU; ++i) {
        unit[i] = unit_of<VEC>(u0 + 32 * i, p.dim, p.rotary, p.adjacent);
        unit[i].turns = unit[i].turns && rotating;
    }
    Chunk<TI, VEC> a[kHeadsPerTeam][NU] = {}, b[kHeadsPerTeam][NU] = {};
#pragma unroll
    for (int h = 0; h < kHeadsPerTeam; ++h) {
        if (h0 + h < heads && token) {
            const TI* row = src + (h0 + h) * src_head;
#pragma unroll
            for (int i = 0; i < NU; ++i) {
                if (unit[i].held) a[h][i] = *reinterpret_cast<const Chunk<TI, VEC>*>(row + unit[i].lo);
                if (unit[i].has_hi) b[h][i] = *reinterpret_cast<const Chunk<TI, VEC>*>(row + unit[i].hi);
            }
        }
    }

    const Home home = home_of(p, t, token, kind != 0);
    const bool active = home.active;
    const int place = home.place;
    TO* dst = kind == 0 ? static_cast<TO*>(p.out) + t * p.out_token
                        : static_cast<TO*>(p.pool[kind - 1]) + home.page * p.page_stride + home.slot * p.slot_stride;
    const long long dst_head = kind == 0 ? p.out_head : p.head_stride;
    if (__ballot_sync(0xffffffffu, active) == 0) return;

    float cs[NU][VEC], sn[NU][VEC], wx[NU][VEC], wy[NU][VEC];
#pragma unroll
    for (int i = 0; i < NU; ++i) {
        const int u = u0 + 32 * i;
        const bool mine = active && unit[i].held;
        if (mine && unit[i].turns) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const int f = pair_of<VEC>(unit[i], u, j, p.adjacent);
                const int32_t frac = (int32_t)(fraction(p.turns[f], p.pos, p.tokens, t, place) >> 32);
                if (sizeof(TO) == 2) {
                    const float angle = (float)frac * 1.4629180792671596e-9f;  // 2^-32 of a turn, in radians
                    sn[i][j] = __sinf(angle);
                    cs[i][j] = __cosf(angle);
                } else {
                    sincospif((float)frac * 4.656612873077393e-10f /* 2^-31: half turns */, &sn[i][j], &cs[i][j]);
                }
            }
        }
        if (weight) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                wx[i][j] = mine ? weight[unit[i].lo + j] : 0.f;
                wy[i][j] = mine && unit[i].has_hi ? weight[unit[i].hi + j] : 0.f;
            }
        }
    }

    float r[kHeadsPerTeam];
    if (weight) {
#pragma unroll
        for (int h = 0; h < kHeadsPerTeam; ++h) {
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < NU; ++i) {
                float x[VEC], y[VEC], part = 0.f;
                unpack(a[h][i], x);
                unpack(b[h][i], y);
#pragma unroll
                for (int j = 0; j < VEC; ++j) part += fmaf(x[j], x[j], y[j] * y[j]);
                sum += part;
            }
            r[h] = sum;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            if (o < np.team) {
#pragma unroll
                for (int h = 0; h < kHeadsPerTeam; ++h) r[h] += __shfl_xor_sync(0xffffffffu, r[h], o);
            }
        }
#pragma unroll
        for (int h = 0; h < kHeadsPerTeam; ++h) r[h] = rsqrtf(fmaf(r[h], np.inverse_dim, np.eps_f));
    }
    if (!active) return;
    dst += h0 * dst_head;
#pragma unroll
    for (int h = 0; h < kHeadsPerTeam; ++h, dst += dst_head) {
        if (h0 + h >= heads) break;
#pragma unroll
        for (int i = 0; i < NU; ++i) {
            float x[VEC], y[VEC];
            unpack(a[h][i], x);
            unpack(b[h][i], y);
            if (weight) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    x[j] = x[j] * r[h] * wx[i][j];  // (root times weight may overflow where this does not)
                    y[j] = y[j] * r[h] * wy[i][j];
                }
            }
            if (unit[i].turns) rotate<VEC>(x, y, cs[i], sn[i], p.adjacent);
            if (unit[i].held) *reinterpret_cast<Chunk<TO, VEC>*>(dst + unit[i].lo) = pack<TO, VEC>(x);
            if (unit[i].has_hi) *reinterpret_cast<Chunk<TO, VEC>*>(dst + unit[i].hi) = pack<TO, VEC>(y);
        }
    }
}

// ---- the gradient -------------------------------------------------------------

template <typename TY, typename TX, int VEC>
__global__ void __launch_bounds__(kGradThreads, 2) bitlin_norm_grad(const NormGradParams p)
{
    constexpr int NU = VEC == 1 ? 4 : 1;
    constexpr int kHeads = kGradHeads;
    __shared__ float sums[8 * kGradThreads];  // a row for each team
    ptx::griddep_wait();
    const int lane = threadIdx.x & 31, u0 = lane & (p.team - 1);
    const int teams = kGradThreads / p.team, me = threadIdx.x / p.team;
    const int groups = (p.heads + kHeads - 1) / kHeads;
    const long long items = (long long)p.tokens * groups;

    Unit<VEC> unit[NU];
    float wx[NU][VEC], wy[NU][VEC], dwx[NU][VEC] = {}, dwy[NU][VEC] = {};
#pragma unroll
    for (int i = 0; i < NU; ++i) {
        unit[i] = unit_of<VEC>(u0 + 32 * i, p.dim, p.rotary, p.adjacent);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            wx[i][j] = unit[i].held ? p.weight[unit[i].lo + j] : 0.f;
            wy[i][j] = unit[i].has_hi ? p.weight[unit[i].hi + j] : 0.f;
        }
    }
    for (long long base = (long long)blockIdx.x * teams; base < items; base += (long long)gridDim.x * teams) {
        const bool active = base + me < items;
        const long long item = active ? base + me : items - 1;
        const int t = (int)(item / groups), h0 = (int)(item - (long long)t * groups) * kHeads;
        Chunk<TX, VEC> a[kHeads][NU] = {}, b[kHeads][NU] = {};
        Chunk<TY, VEC> ga[kHeads][NU] = {}, gb[kHeads][NU] = {};
#pragma unroll
        for (int h = 0; h < kHeads; ++h) {
            if (h0 + h >= p.heads || !active) continue;
            const TX* x = static_cast<const TX*>(p.x) + t * p.x_token + (h0 + h) * p.x_head;
            const TY* dy = static_cast<const TY*>(p.dy) + t * p.dy_token + (h0 + h) * p.dy_head;
#pragma unroll
            for (int i = 0; i < NU; ++i) {
                if (unit[i].held) {
                    a[h][i] = *reinterpret_cast<const Chunk<TX, VEC>*>(x + unit[i].lo);
                    ga[h][i] = *reinterpret_cast<const Chunk<TY, VEC>*>(dy + unit[i].lo);
                }
                if (unit[i].has_hi) {
                    b[h][i] = *reinterpret_cast<const Chunk<TX, VEC>*>(x + unit[i].hi);
                    gb[h][i] = *reinterpret_cast<const Chunk<TY, VEC>*>(dy + unit[i].hi);
                }
            }
        }
        float cs[NU][VEC], sn[NU][VEC];
#pragma unroll
        for (int i = 0; i < NU; ++i) {
            if (!unit[i].held || !unit[i].turns) continue;
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const int f = pair_of<VEC>(unit[i], u0 + 32 * i, j, p.adjacent);
                const int32_t frac = (int32_t)(fraction(p.turns[f], p.pos, p.tokens, t, 0) >> 32);
                sincospif((float)frac * 4.656612873077393e-10f, &sn[i][j], &cs[i][j]);
                sn[i][j] = -sn[i][j];  // back
            }
        }
#pragma unroll
        for (int h = 0; h < kHeads; ++h) {
            float x[NU][VEC], y[NU][VEC], gx[NU][VEC], gy[NU][VEC];
            float squares = 0.f, products = 0.f;
#pragma unroll
            for (int i = 0; i < NU; ++i) {
                unpack(a[h][i], x[i]);
                unpack(b[h][i], y[i]);
                unpack(ga[h][i], gx[i]);
                unpack(gb[h][i], gy[i]);
                if (unit[i].held && unit[i].turns) rotate<VEC>(gx[i], gy[i], cs[i], sn[i], p.adjacent);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    squares += fmaf(x[i][j], x[i][j], y[i][j] * y[i][j]);
                    products += fmaf(gx[i][j] * wx[i][j], x[i][j], gy[i][j] * wy[i][j] * y[i][j]);
                }
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                if (o < p.team) {
                    squares += __shfl_xor_sync(0xffffffffu, squares, o);
                    products += __shfl_xor_sync(0xffffffffu, products, o);
                }
            }
            const float r = rsqrtf(fmaf(squares, p.inverse_dim, p.eps_f));
            const float mean = products * p.inverse_dim * r * r;  // mean(h n) r: n = x r
            if (h0 + h >= p.heads || !active) continue;
            TX* dx = static_cast<TX*>(p.dx) + t * p.dx_token + (h0 + h) * p.dx_head;
#pragma unroll
            for (int i = 0; i < NU; ++i) {
                float c[VEC], d[VEC];
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    dwx[i][j] = fmaf(gx[i][j], x[i][j] * r, dwx[i][j]);
                    dwy[i][j] = fmaf(gy[i][j], y[i][j] * r, dwy[i][j]);
                    c[j] = r * (gx[i][j] * wx[i][j] - x[i][j] * mean);
                    d[j] = r * (gy[i][j] * wy[i][j] - y[i][j] * mean);
                }
                if (unit[i].held) *reinterpret_cast<Chunk<TX, VEC>*>(dx + unit[i].lo) = pack<TX, VEC>(c);
                if (unit[i].has_hi) *reinterpret_cast<Chunk<TX, VEC>*>(dx + unit[i].hi) = pack<TX, VEC>(d);
            }
        }
    }
    // the block's sum, teams in their order
#pragma unroll
    for (int i = 0; i < NU; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            if (unit[i].held) sums[me * p.dim + unit[i].lo + j] = dwx[i][j];
            if (unit[i].has_hi) sums[me * p.dim + unit[i].hi + j] = dwy[i][j];
        }
    __syncthreads();
    for (int d = threadIdx.x; d < p.dim; d += kGradThreads) {
        float sum = 0.f;
        for (int k = 0; k < teams; ++k) sum += sums[k * p.dim + d];
        p.partial[(long long)blockIdx.x * p.dim + d] = sum;
    }
}

// The blocks' sums joined in a fixed order: 32 elements to a block, 32 rows at a time.
__global__ void __launch_bounds__(1024) bitlin_norm_grad_join(const float* partial, float* dweight, int blocks, int dim)
{
    __shared__ float sums[32][33];
    ptx::griddep_wait();
    const int lane = threadIdx.x & 31, row = threadIdx.x >> 5, d = blockIdx.x * 32 + lane;
    float sum = 0.f;
    if (d < dim) {
#pragma unroll 8
        for (int k = row; k < blocks; k += 32) sum += partial[(long long)k * dim + d];
    }
    sums[row][lane] = sum;
    __syncthreads();
    if (row == 0 && d < dim) {
        sum = 0.f;
#pragma unroll
        for (int k = 0; k < 32; ++k) sum += sums[k][lane];
        dweight[d] = sum;
    }
}

// ---- launches -------------------------------------------------------------------

cudaLaunchConfig_t config(dim3 grid, int threads, cudaStream_t s, cudaLaunchAttribute* attr)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr->val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

// Lanes to a row of `dim` elements: a power of two of them, eight elements each.
int team_of(int dim, int vec)
{
    if (vec == 1) return 32;
    int team = 8;
    while (team * 8 < dim) team *= 2;
    return team;
}

template <typename TI, typename TO, int VEC, bool QUANT>
cudaError_t launch(NormTurnParams& p, cudaStream_t s)
{
    p.team = team_of(p.t.dim, VEC);
    p.inverse_dim = 1.f / p.t.dim;
    p.eps_f = (float)p.eps;
    p.t.q_groups = (p.t.heads + kHeadsPerTeam - 1) / kHeadsPerTeam;
    // k and v to 4 bits: a team takes as many heads of a token as leave 24 warps to an SM
    const long long rows = 2LL * p.t.tokens * p.t.kv_heads * p.team / 32, most = rows / (24 * 152);
    p.kv_heads_per_team = !QUANT ? kHeadsPerTeam : most < 1 ? 1 : most < p.t.kv_heads ? (int)most : p.t.kv_heads;
    p.t.kv_groups = p.t.append ? (p.t.kv_heads + p.kv_heads_per_team - 1) / p.kv_heads_per_team : 0;
    const int teams = kThreads / p.team;
    cudaLaunchAttribute attr = {};
    const cudaLaunchConfig_t cfg =
        config(dim3((unsigned)(((long long)p.t.tokens + teams - 1) / teams), p.t.q_groups + 2 * p.t.kv_groups), kThreads, s, &attr);
    return cudaLaunchKernelEx(&cfg, bitlin_norm_turn<TI, TO, VEC, QUANT>, p);
}

// Whether rows of this tensor can be read or written four elements at a time.
bool chunked(const void* data, long long token, long long head, int size)
{
    return reinterpret_cast<uintptr_t>(data) % (uintptr_t)(size * 4) == 0 && token % 4 == 0 && head % 4 == 0;
}

template <typename TI, typename TO, bool QUANT>
cudaError_t pick(const NormTurnParams& np, cudaStream_t s)
{
    NormTurnParams p = np;
    const TurnParams& t = p.t;
    bool wide = t.rotary % 8 == 0 && (t.dim - t.rotary) % 8 == 0;
    if (t.heads)
        wide = wide && chunked(t.src[0], t.src_token[0], t.src_head[0], sizeof(TI)) && chunked(t.out, t.out_token, t.out_head, sizeof(TO));
    if (t.append)
        for (int i = 1; i < 3; ++i) wide = wide && chunked(t.src[i], t.src_token[i], t.src_head[i], sizeof(TI));
    return wide ? launch<TI, TO, 4, QUANT>(p, s) : launch<TI, TO, 1, QUANT>(p, s);
}

template <typename TI>
cudaError_t pick_out(const NormTurnParams& p, int dst_dtype, bool quant, cudaStream_t s)
{
    if (quant) return dst_dtype == BITLIN_BF16 ? pick<TI, __nv_bfloat16, true>(p, s) : pick<TI, __half, true>(p, s);
    switch (dst_dtype) {
    case BITLIN_F32: return pick<TI, float, false>(p, s);
    case BITLIN_BF16: return pick<TI, __nv_bfloat16, false>(p, s);
    default: return pick<TI, __half, false>(p, s);
    }
}

template <typename TY, typename TX>
cudaError_t grad(const NormGradParams& np, cudaStream_t s)
{
    NormGradParams p = np;
    const bool wide = p.rotary % 8 == 0 && (p.dim - p.rotary) % 8 == 0 && chunked(p.dy, p.dy_token, p.dy_head, sizeof(TY)) &&
                      chunked(p.x, p.x_token, p.x_head, sizeof(TX)) && chunked(p.dx, p.dx_token, p.dx_head, sizeof(TX));
    p.team = team_of(p.dim, wide ? 4 : 1);
    p.inverse_dim = 1.f / p.dim;
    p.eps_f = (float)p.eps;
    p.blocks = bitlin_norm_grad_blocks(p.tokens, p.heads);
    cudaLaunchAttribute attr = {};
    cudaLaunchConfig_t cfg = config(dim3(p.blocks), kGradThreads, s, &attr);
    cudaError_t e = wide ? cudaLaunchKernelEx(&cfg, bitlin_norm_grad<TY, TX, 4>, p) : cudaLaunchKernelEx(&cfg, bitlin_norm_grad<TY, TX, 1>, p);
    if (e != cudaSuccess) return e;
    cfg = config(dim3((p.dim + 31) / 32), 1024, s, &attr);
    return cudaLaunchKernelEx(&cfg, bitlin_norm_grad_join, (const float*)p.partial, p.dweight, p.blocks, p.dim);
}

template <typename TY>
cudaError_t grad_x(const NormGradParams& p, int x_dtype, cudaStream_t s)
{
    switch (x_dtype) {
    case BITLIN_F32: return grad<TY, float>(p, s);
    case BITLIN_BF16: return grad<TY, __nv_bfloat16>(p, s);
    default: return grad<TY, __half>(p, s);
    }
}

}  // namespace

cudaError_t bitlin_launch_norm_turn(const NormTurnParams& p, int src_dtype, int dst_dtype, bool quant, cudaStream_t s)
{
    switch (src_dtype) {
    case BITLIN_F32: return pick_out<float>(p, dst_dtype, quant, s);
    case BITLIN_BF16: return pick_out<__nv_bfloat16>(p, dst_dtype, quant, s);
    default: return pick_out<__half>(p, dst_dtype, quant, s);
    }
}

int bitlin_norm_grad_blocks(int tokens, int heads)
{
    // two to each of 152 SMs, or as many as there are tokens and heads for
    const long long items = (long long)tokens * ((heads + kGradHeads - 1) / kGradHeads);
    const long long blocks = (items + kGradThreads / 32 - 1) / (kGradThreads / 32);
    return (int)(blocks < 304 ? blocks : 304);
}

cudaError_t bitlin_launch_norm_grad(const NormGradParams& p, int dy_dtype, int x_dtype, cudaStream_t s)
{
    switch (dy_dtype) {
    case BITLIN_F32: return grad_x<float>(p, x_dtype, s);
    case BITLIN_BF16: return grad_x<__nv_bfloat16>(p, x_dtype, s);
    default: return grad_x<__half>(p, x_dtype, s);
    }
}
