// w4a16_norm_rope.cu -- norms of queries and keys per head, rotary positions, and keys and values
// written into a paged cache, of 16 bits or held in 4.
//
// For every head of q and k, with weights w (no weights: y = x):
//     y = x rsqrt(mean x^2 + eps) w,
// then pair i < rot_dim / 2 is turned by its position's angle, (y1, y2) -> (y1 c - y2 s, y2 c + y1 s), as
// w4a16_rope_append does.  All in fp32; q, and k and v of the 16-bit cache, are rounded once.  In the
// 4-bit cache a group of values is coded, keys from norm and rotation in two fp32 parts:
//     b = r(min),  s = r((max - min) / 15),  code = (x - b) / s to the nearest integer, ties to even, in 0..15
// (r: to the cache's 16-bit type), which stands for code s + b.
//
// Bound by memory: each value is read once and written once.  A head belongs to D / 16 neighbouring threads of 16
// values (eight pairs) each, which meet in shuffles for the sum of squares and for the groups' smallest and largest
// values; a warp works on 32 / that many heads of one kind, with the next ones' values on their way, and a block on a
// token.  Arithmetic goes two values to an instruction, as instructions are what the 4-bit kernel is bound by.
// 6007 tokens of 32 / 8 heads of 128, bf16, 16-bit cache: 29.5 us, 5.1 TB/s of reads and writes; 8191 tokens with three
// axes into 4 bits (groups of 64, with k_out and v_out): 52 us, 4.1 TB/s (that kernel spills 104 bytes at its 96 registers); one token 3.2 us of latencies.
//
// Codes are those of exact arithmetic: a value next to the border of two codes, or a base or step next to the border of
// two 16-bit numbers, would fall on either side in fp32 (measured: four codes in 10^7, and a base or step in 10^4 groups).
// So keys that are to be coded are computed in two fp32 parts throughout, from the sum of squares to the remainder of the
// division, whose last roundings leave 2^-25 of a step: three codes in 10^8, and no base or step (of 10^7 groups).
#include <type_traits>

#include "w4a16_kv4.cuh"

namespace w4 {
namespace ops {

constexpr int NORM_MAX_AXES = 4;
constexpr int NORM_WARPS = 4;   // of a block of the any-size kernel
constexpr int NORM_MOST = 512;  // threads of a block where tokens are few
constexpr int NORM_PER_SM = 16; // warps that an SM holds

struct NormParams {
    const uint16_t *q, *k, *v;
    const uint16_t *q_norm, *k_norm;
    uint16_t *q_out, *k_cache, *v_cache; // 16-bit cache
    uint8_t *cache;                      // 4-bit cache
    uint16_t *k_out, *v_out;
    const float *table;
    const int32_t *positions;
    const long long *slots;
    int *status;
    long long page_stride, token_stride, head_stride; // elements; 4 bits: bytes, unused, bytes of a record
    long long total_slots;
    Kv4Record rec;
    float eps, per_dim; // per_dim: 1 / dim
    int ldq, ldk, ldv, ldqo, ldko, ldvo, ld_pos;
    int tokens, heads, kv, dim, rot, axes, max_pos, page;
    int cut[NORM_MAX_AXES]; // pair i belongs to the first axis a with i < cut[a]
    int adjacent, cuts; // cuts: some section ends inside eight pairs
    int copies16; // everything can be copied 16 bytes at a time
};

enum { KIND_Q = 0, KIND_K = 1, KIND_V = 2 };

__device__ __forceinline__ void report(const NormParams &p, int bit)
{
    if (p.status)
        atomicOr(p.status, bit);
}

__device__ __forceinline__ int axis_of(const NormParams &p, int pair)
{
    int axis = 0;
#pragma unroll
    for (int a = 0; a < NORM_MAX_AXES - 1; ++a)
        axis += (a < p.axes - 1 && pair >= p.cut[a]) ? 1 : 0;
    return axis;
}

__device__ __forceinline__ int checked_position(const NormParams &p, int pos)
{
    if (pos < 0 || pos >= p.max_pos) {
        report(p, W4A16_DEV_POSITION);
        return -1;
    }
    return pos;
}

// The page and the token in it of a slot; false for a negative slot (not cached) or, after reporting it,
// one past the cache.
__device__ __forceinline__ bool page_of(const NormParams &p, long long slot, long long &pg, int &token)
{
    if (slot < 0)
        return false;
    if (slot >= p.total_slots) {
        report(p, W4A16_DEV_SLOT);
        return false;
    }
    pg = p.total_slots < (1LL << 31) ? (long long)((uint32_t)slot / (uint32_t)p.page) : slot / p.page;
    token = (int)(slot - pg * p.page);
    return true;
}

__device__ __forceinline__ const uint16_t *head_src(const NormParams &p, int kind, int token, int h)
{
    const uint16_t *base = kind == KIND_Q ? p.q : kind == KIND_K ? p.k : p.v;
    const int ld = kind == KIND_Q ? p.ldq : kind == KIND_K ? p.ldk : p.ldv;
    return base + (long long)token * ld + (long long)h * p.dim;
}

// The rotation of the any-size kernel.  It serves sizes without 16-byte copies, and heads that are too wide for the 16-byte
// kernel here but not for w4a16_rope_append's; the two kernels of that round different products of a pair's second value,
// and so does this one.
__device__ __forceinline__ float turned_first(float a, float b, float c, float s)
{
    return fmaf(a, c, -(b * s));
}

__device__ __forceinline__ float turned_second(float a, float b, float c, float s, bool copies16)
{
    return copies16 ? fmaf(b, c, a * s) : fmaf(a, s, b * c);
}

// The smaller and the larger of two values, NaN where one is.
__device__ __forceinline__ float min_nan(float a, float b)
{
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// A value in two parts, hi + lo, the second below half a unit of the first (or a few of them).
struct Two {
    float hi, lo;
};

// a + b exactly.
__device__ __forceinline__ Two two_sum(float a, float b)
{
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}

__device__ __forceinline__ void two_sum(float2 a, float2 b, float2 &s, float2 &off)
{
    s = add(a, b);
    const float2 t = sub(s, a);
    off = add(sub(a, sub(s, t)), sub(b, t));
}

// x / 15, correctly rounded (for results that are not subnormal).
__device__ __forceinline__ float fifteenth(float x)
{
    const float q = x * (1.f / 15.f);
    return fmaf(fmaf(-q, 15.f, x), 1.f / 15.f, q);
}

// How a group of values is coded: the step and base as stored, and what coding needs of them.
struct Step {
    uint32_t stored;       // step, base (16 bits each)
    float s, b;            // as numbers; both NaN where the group has no finite range
    float size, from, inv; // for coding: step and base, 0 where there are none, and 1 / step (to a unit) or 0
};

// lo: the smallest value, step: (largest - smallest) / 15.
template <bool BF>
__device__ __forceinline__ Step step_of(float lo, float step)
{
    Step st;
    uint32_t sb = from_float<BF>(step), bb = from_float<BF>(lo);
    if (BF && (sb & 0x7F80) == 0)
        sb = 0; // a subnormal bf16 step has no inverse in fp32
    st.s = to_float<BF>((uint16_t)sb);
    st.b = to_float<BF>((uint16_t)bb);
    const bool fine = fabsf(st.s) < INFINITY && fabsf(st.b) < INFINITY; // false for NaN too
    st.size = fine ? st.s : 0.f;
    st.from = fine ? st.b : 0.f;
    float inv;
    asm("rcp.approx.f32 %0, %1;" : "=f"(inv) : "f"(st.size));
    inv = fmaf(fmaf(-st.size, inv, 1.f), inv, inv);
    st.inv = st.size > 0.f ? inv : 0.f;
    if (!fine) {
        st.s = st.b = NAN;
        sb = bb = 0x7FFF; // NaN in both types
    }
    st.stored = sb | bb << 16;
    return st;
}

// Adding this rounds a number below 2^22 to the nearest integer, ties to even, into the lowest bits.
constexpr float ROUND = 12582912.f;
constexpr uint32_t ROUND_BITS = 0x4B400000u;

// Eight times ROUND_BITS, shifted by 0, 4, .. 28 bits: what a word of codes on ROUND has too much.
constexpr uint32_t ROUND_WORD = ROUND_BITS * 0x11111111u;

// Two codes (as numbers on ROUND) of values 2 i and 2 i + 1, cut to 0..15 and put into a word, which starts as
// -ROUND_WORD; the numbers they stand for.  FROM_0: the codes are not negative.
template <bool FROM_0>
__device__ __forceinline__ float2 put(float2 t, int i, const Step &st, uint32_t &word)
{
    t.x = fminf(FROM_0 ? t.x : fmaxf(t.x, ROUND), ROUND + 15.f);
    t.y = fminf(FROM_0 ? t.y : fmaxf(t.y, ROUND), ROUND + 15.f);
    word += __float_as_uint(t.x) << (8 * i);
    word += __float_as_uint(t.y) << (8 * i + 4);
    return fma(add(t, both(-ROUND)), both(st.s), both(st.b));
}

// Eight 16-bit values coded into a word, and replaced by what the codes stand for.  d = x - b is exact where
// its digits fit, and the quotient correctly rounded (a Newton step on d / s, whose remainder is exact): values on the
// middle between two codes, which 16-bit numbers do hit, are seen as such and go to the even one.  The base is the
// smallest value itself.
__device__ __forceinline__ uint32_t code_values(float2 *x, const Step &st)
{
    uint32_t word = 0u - ROUND_WORD;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 d = add(x[i], both(-st.from));
        const float2 q = mul(d, both(st.inv));
        const float2 exact = fma(fma(q, both(-st.size), d), both(st.inv), q);
        x[i] = put<true>(add(exact, both(ROUND)), i, st, word);
    }
    return word;
}

// Eight keys r z in two parts, coded; x: what the codes stand for.  The first guess at a code is off by one at most;
// of the remainder r z - (b + q s) fp32 keeps 24 bits however small it is, and its quotient by s, correctly rounded as
// above, corrects the guess with ties to even.
__device__ __forceinline__ uint32_t code_keys(const float2 *z, const float2 *z_lo, const Two &r, float2 *x, const Step &st)
{
    uint32_t word = 0u - ROUND_WORD;
    const float2 scale = both(r.hi * st.inv), start = both(-st.from * st.inv);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 t = add(fma(z[i], scale, start), both(ROUND));
        const float2 minus = fma(add(t, both(-ROUND)), both(-st.size), both(-st.from)); // -(b + q s)
        const float2 rest =
            fma(both(r.hi), z_lo[i], fma(both(r.lo), z[i], fma(both(r.hi), z[i], minus)));
        const float2 q = mul(rest, both(st.inv));
        const float2 exact = fma(fma(q, both(-st.size), rest), both(st.inv), q);
        x[i] = put<false>(add(t, exact), i, st, word);
    }
    return word;
}

// Codes of values 0 2 4 6 ... of sixteen in a row and of 1 3 5 7 ... -> their two words in order.
__device__ __forceinline__ void interleave(uint32_t &even, uint32_t &odd)
{
    auto spread = [](uint32_t v) { // four codes to the low halves of four bytes
        v = (v | v << 8) & 0x00FF00FFu;
        return (v | v << 4) & 0x0F0F0F0Fu;
    };
    const uint32_t first = spread(even & 0xFFFFu) | spread(odd & 0xFFFFu) << 4;
    odd = spread(even >> 16) | spread(odd >> 16) << 4;
    even = first;
}

// Sixteen 16-bit values as they lie -> first members of eight pairs, second members, where pairs lie side by side;
// and back.
__device__ __forceinline__ void apart(uint4 &a, uint4 &b)
{
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    a = make_uint4(__byte_perm(w[0], w[1], 0x5410), __byte_perm(w[2], w[3], 0x5410), __byte_perm(w[4], w[5], 0x5410),
                   __byte_perm(w[6], w[7], 0x5410));
    b = make_uint4(__byte_perm(w[0], w[1], 0x7632), __byte_perm(w[2], w[3], 0x7632), __byte_perm(w[4], w[5], 0x7632),
                   __byte_perm(w[6], w[7], 0x7632));
}

__device__ __forceinline__ void together(uint4 &a, uint4 &b)
{
    const uint32_t f[4] = {a.x, a.y, a.z, a.w}, s[4] = {b.x, b.y, b.z, b.w};
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[2 * i] = __byte_perm(f[i], s[i], 0x5410);
        w[2 * i + 1] = __byte_perm(f[i], s[i], 0x7632);
    }
    a = make_uint4(w[0], w[1], w[2], w[3]);
    b = make_uint4(w[4], w[5], w[6], w[7]);
}

template <bool BF>
__device__ __forceinline__ void unpack16(const uint4 &a, const uint4 &b, float2 (&x)[8])
{
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        x[i] = BF ? make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u)) : unpack2<BF>(w[i]);
}

template <bool BF>
__device__ __forceinline__ uint4 pack8(const float2 *x)
{
    return make_uint4(pack2<BF>(x[0].x, x[0].y), pack2<BF>(x[1].x, x[1].y), pack2<BF>(x[2].x, x[2].y),
                      pack2<BF>(x[3].x, x[3].y));
}

__device__ __forceinline__ float min3(float a, float b, float c) // NaN where one is
{
    float r;
    asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// The cosines and sines of eight pairs from 8 j on, by their token's positions; false where one is out of range.
__device__ __forceinline__ bool angles(const NormParams &p, int token, int j, int pos, float2 (&c2)[4], float2 (&s2)[4])
{
    const int half = p.rot / 2;
    pos = checked_position(p, pos);
    const float *entry = p.table + (long long)max(pos, 0) * p.rot + 8 * j;
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        const float4 c = *reinterpret_cast<const float4 *>(entry + 2 * i);
        const float4 s = *reinterpret_cast<const float4 *>(entry + half + 2 * i);
        c2[i] = make_float2(c.x, c.y);
        c2[i + 1] = make_float2(c.z, c.w);
        s2[i] = make_float2(s.x, s.y);
        s2[i + 1] = make_float2(s.z, s.w);
    }
    bool known = pos >= 0;
    if (p.cuts) {
        // The pairs from a further section's start on take that axis's entries.
        const int last = axis_of(p, 8 * j + 7);
#pragma unroll 1
        for (int a = axis_of(p, 8 * j) + 1; a <= last; ++a) {
            const int from = p.cut[a - 1] - 8 * j;
            if (p.cut[a] == p.cut[a - 1])
                continue;
            const int pa = checked_position(p, p.positions[(long long)a * p.ld_pos + token]);
            known &= pa >= 0;
            const float *other = p.table + (long long)max(pa, 0) * p.rot + 8 * j;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i >= from) {
                    (i & 1 ? c2[i / 2].y : c2[i / 2].x) = other[i];
                    (i & 1 ? s2[i / 2].y : s2[i / 2].x) = other[half + i];
                }
        }
    }
    return known;
}

// Whether a number that may be off by `off` could round to another 16-bit number.
template <bool BF>
__device__ __forceinline__ bool in_doubt(float x, float off)
{
    return from_float<BF>(x - off) != from_float<BF>(x + off);
}

// What a token's heads share in a thread (chunk j of a head).
struct TokenOf {
    float2 c[4], s[4]; // the angles of its eight pairs
    long long pg;      // its place in the cache
    int token, in_page, j;
    bool live, known;  // it has a place; its positions are in range
    bool held, turns;  // the thread has values; ... pairs
};

template <int LANES>
__device__ __forceinline__ float sum_lanes(float x)
{
#pragma unroll
    for (int d = 1; d < LANES; d <<= 1)
        x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}

// Stores sixteen values as the head holds them.
template <bool BF>
__device__ __forceinline__ void store16(uint16_t *dst, int apart_by, bool beside, const float2 (&x)[8])
{
    uint4 a = pack8<BF>(x), b = pack8<BF>(x + 4);
    if (beside)
        together(a, b);
    *reinterpret_cast<uint4 *>(dst) = a;
    *reinterpret_cast<uint4 *>(dst + apart_by) = b;
}

// One head of q, or of k for the 16-bit cache: dst null: not written.
template <bool BF, int LANES>
__device__ __forceinline__ void plain_head(const NormParams &p, const TokenOf &t, uint4 x0, uint4 x1, const uint16_t *norm,
                                           uint16_t *dst)
{
    const bool beside = t.turns && p.adjacent;
    const int at0 = t.turns && !beside ? 8 * t.j : 16 * t.j, apart_by = t.turns && !beside ? p.rot / 2 : 8;
    if (beside)
        apart(x0, x1);
    float2 x[8];
    unpack16<BF>(x0, x1, x);
    if (norm) {
        uint4 w0 = make_uint4(0, 0, 0, 0), w1 = w0;
        if (t.held) {
            w0 = *reinterpret_cast<const uint4 *>(norm + at0);
            w1 = *reinterpret_cast<const uint4 *>(norm + at0 + apart_by);
        }
        if (beside)
            apart(w0, w1);
        float2 sum = mul(x[0], x[0]), w[8];
#pragma unroll
        for (int i = 1; i < 8; ++i)
            sum = fma(x[i], x[i], sum);
        unpack16<BF>(w0, w1, w);
        const float2 r = both(rsqrtf(fmaf(sum_lanes<LANES>(sum.x + sum.y), p.per_dim, p.eps)));
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = mul(mul(x[i], r), w[i]);
    }
    if (t.turns) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 a = x[i], b = x[4 + i];
            x[i] = fma(a, t.c[i], mul(b, make_float2(-t.s[i].x, -t.s[i].y)));
            x[4 + i] = fma(b, t.c[i], mul(a, t.s[i]));
        }
    }
    if (dst && t.held && t.known)
        store16<BF>(dst + at0, apart_by, beside, x);
}

// The smallest and the largest value of the groups to which a thread's two halves belong.
template <int GROUPS, int LANES>
__device__ __forceinline__ void extremes(const float2 (&x)[8], bool held, int g0, int g1, float (&lo)[2], float (&hi)[2])
{
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const float2 *v = x + 4 * e;
        lo[e] = min3(min3(v[0].x, v[0].y, v[1].x), min3(v[1].y, v[2].x, v[2].y), min_nan(v[3].x, v[3].y));
        hi[e] = max3(max3(v[0].x, v[0].y, v[1].x), max3(v[1].y, v[2].x, v[2].y), max_nan(v[3].x, v[3].y));
    }
    const float lo0 = lo[0], lo1 = lo[1], hi0 = hi[0], hi1 = hi[1];
#pragma unroll
    for (int q = 0; q < GROUPS; ++q) {
        float l = held && g0 == q ? lo0 : INFINITY, m = held && g0 == q ? hi0 : -INFINITY;
        if (held && g1 == q) {
            l = min_nan(l, lo1);
            m = max_nan(m, hi1);
        }
#pragma unroll
        for (int d = 1; d < LANES; d <<= 1) {
            l = min_nan(l, __shfl_xor_sync(0xffffffffu, l, d));
            m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, d));
        }
        if (q == 0 || g0 == q) {
            lo[0] = l;
            hi[0] = m;
        }
        if (q == 0 || g1 == q) {
            lo[1] = l;
            hi[1] = m;
        }
    }
}

// One head of k or v into the 4-bit cache; dst: where what it stands for goes, or null.
template <bool BF, int GROUPS, int LANES, bool KEY>
__device__ __forceinline__ void coded_head(const NormParams &p, const TokenOf &t, uint4 x0, uint4 x1, bool valid, int h,
                                           uint16_t *dst)
{
    const bool turns = KEY && t.turns, beside = turns && p.adjacent;
    const int at0 = turns && !beside ? 8 * t.j : 16 * t.j, apart_by = turns && !beside ? p.rot / 2 : 8, at1 = at0 + apart_by;
    if (beside)
        apart(x0, x1);
    float2 x[8];
    unpack16<BF>(x0, x1, x);
    // Groups are whole blocks of 64 values, and each half of a thread's lies in one of them.
    const int size = p.dim / GROUPS; // powers of two
    const int shift = GROUPS == 1 ? 31 : 31 - __clz(size), g0 = at0 >> shift, g1 = at1 >> shift;
    uint32_t word0, word1;
    Step st0, st1;
    float lo[2], hi[2];
    if (!KEY) {
        extremes<GROUPS, LANES>(x, t.held, g0, g1, lo, hi);
        st0 = step_of<BF>(lo[0], fifteenth(hi[0] - lo[0]));
        st1 = GROUPS == 1 ? st0 : step_of<BF>(lo[1], fifteenth(hi[1] - lo[1]));
        word0 = code_values(x, st0);
        word1 = code_values(x + 4, st1);
    } else {
        // Keys in two parts: r z with z = the turned x w (x w is exact).
        Two r = {1.f, 0.f};
        if (p.k_norm) {
            uint4 w0 = make_uint4(0, 0, 0, 0), w1 = w0;
            if (t.held) {
                w0 = *reinterpret_cast<const uint4 *>(p.k_norm + at0);
                w1 = *reinterpret_cast<const uint4 *>(p.k_norm + at1);
            }
            if (beside)
                apart(w0, w1);
            float2 sum = mul(x[0], x[0]), off = both(0.f); // (the squares are exact)
#pragma unroll
            for (int i = 1; i < 8; ++i) {
                float2 e;
                two_sum(sum, mul(x[i], x[i]), sum, e);
                off = add(off, e);
            }
            Two total = two_sum(sum.x, sum.y);
            total.lo += off.x + off.y;
#pragma unroll
            for (int d = 1; d < LANES; d <<= 1) {
                const float o = __shfl_xor_sync(0xffffffffu, total.hi, d), ol = __shfl_xor_sync(0xffffffffu, total.lo, d);
                const Two e = two_sum(total.hi, o);
                total = {e.hi, (total.lo + ol) + e.lo};
            }
            Two a = two_sum(total.hi * p.per_dim, p.eps); // (dim is a power of two)
            a.lo += total.lo * p.per_dim;
            r.hi = rsqrtf(a.hi);
            const float sq = __fmul_rn(r.hi, r.hi), sq_lo = fmaf(r.hi, r.hi, -sq);
            const float rest = fmaf(-a.lo, sq, fmaf(-a.hi, sq_lo, fmaf(-a.hi, sq, 1.f))); // 1 - a r^2
            r.lo = 0.5f * r.hi * rest;
            if (!(fabsf(r.lo) < r.hi))
                r.lo = 0.f; // sums of zero or infinity
            float2 w[8];
            unpack16<BF>(w0, w1, w);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                x[i] = mul(x[i], w[i]);
        }
        float2 z_lo[8]; // (x: the first parts)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            z_lo[i] = both(0.f);
        if (turns) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 a = x[i], b = x[4 + i], c = t.c[i], s = t.s[i];
                const float2 ns = make_float2(-s.x, -s.y), nc = make_float2(-c.x, -c.y);
                const float2 ac = mul(a, c), bs = mul(b, ns), bc = mul(b, c), as = mul(a, s);
                // The products' remainders, with the sign turned.
                const float2 ac_off = fma(a, nc, ac), bs_off = fma(b, s, bs), bc_off = fma(b, nc, bc), as_off = fma(a, ns, as);
                float2 e;
                two_sum(ac, bs, x[i], e);
                z_lo[i] = sub(e, add(ac_off, bs_off));
                two_sum(bc, as, x[4 + i], e);
                z_lo[4 + i] = sub(e, add(bc_off, as_off));
            }
        }
        extremes<GROUPS, LANES>(x, t.held, g0, g1, lo, hi); // r is positive: the extreme z are the extreme keys'
        // Base and step in fp32 are off by below 2^-21 of the larger extreme, and an eighth of that: mostly that does
        // not matter to their 16-bit numbers.
        float low[2], step[2];
        bool doubt = false;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float off = fmaxf(fabsf(lo[e]), fabsf(hi[e])) * r.hi * 0x1p-21f;
            low[e] = r.hi * lo[e];
            step[e] = r.hi * fifteenth(hi[e] - lo[e]);
            if (e < GROUPS)
                doubt |= in_doubt<BF>(low[e], off) || in_doubt<BF>(step[e], 0.125f * off);
        }
        if (__any_sync(0xffffffffu, doubt)) {
#pragma unroll 1
            for (int q = 0; q < GROUPS; ++q) {
                float l = INFINITY, m = -INFINITY; // the extremes' second parts, from whoever holds these
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (t.held && (e ? g1 : g0) == q)
#pragma unroll
                        for (int i = 4 * e; i < 4 * e + 4; ++i) {
                            l = fminf(l, fminf(x[i].x == lo[e] ? z_lo[i].x : INFINITY, x[i].y == lo[e] ? z_lo[i].y : INFINITY));
                            m = fmaxf(m, fmaxf(x[i].x == hi[e] ? z_lo[i].x : -INFINITY, x[i].y == hi[e] ? z_lo[i].y : -INFINITY));
                        }
#pragma unroll
                for (int d = 1; d < LANES; d <<= 1) {
                    l = fminf(l, __shfl_xor_sync(0xffffffffu, l, d));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if ((e ? g1 : g0) != q)
                        continue;
                    // The smallest key and the range over 15, each rounded once to fp32.
                    const float first = __fmul_rn(r.hi, lo[e]);
                    low[e] = first + fmaf(r.hi, l, fmaf(r.lo, lo[e], fmaf(r.hi, lo[e], -first)));
                    Two range = two_sum(hi[e], -lo[e]);
                    range.lo += m - l;
                    const float width = __fmul_rn(r.hi, range.hi);
                    const float rest = fmaf(r.hi, range.lo, fmaf(r.lo, range.hi, fmaf(r.hi, range.hi, -width)));
                    const float part = fifteenth(width);
                    step[e] = part + (fmaf(-part, 15.f, width) + rest) * (1.f / 15.f);
                }
            }
        }
        st0 = step_of<BF>(low[0], step[0]);
        st1 = GROUPS == 1 ? st0 : step_of<BF>(low[1], step[1]);
        float2 out[8];
        word0 = code_keys(x, z_lo, r, out, st0);
        word1 = code_keys(x + 4, z_lo + 4, r, out + 4, st1);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = out[i];
        if (beside)
            interleave(word0, word1);
    }
    if (!valid || !t.held || (KEY && !t.known))
        return;
    if (t.live) {
        uint8_t *row = p.cache + t.pg * p.page_stride + h * p.head_stride;
        uint32_t *codes = reinterpret_cast<uint32_t *>(row + (KEY ? 0 : p.rec.values)) + (long long)t.in_page * (p.dim / 8);
        const int blocks = p.dim / 64;
        codes[KEY ? kv4_key_place(at0 / 8, blocks) : kv4_value_place(at0 / 8, blocks)] = word0;
        codes[KEY ? kv4_key_place(at1 / 8, blocks) : kv4_value_place(at1 / 8, blocks)] = word1;
        // Whoever has a group's first value stores its step and base.
        uint32_t *params =
            reinterpret_cast<uint32_t *>(row + (KEY ? p.rec.key_params : p.rec.value_params)) + (long long)t.in_page * GROUPS;
        if ((at0 & (size - 1)) == 0)
            params[g0] = st0.stored;
        if ((at1 & (size - 1)) == 0)
            params[g1] = st1.stored;
    }
    if (dst)
        store16<BF>(dst + at0, apart_by, beside, x);
}

// 16-byte path: a block per token, of a warp where there are many (what belongs to a token is then looked up once for
// all of its heads: 6007 tokens of 32 / 8 heads of 128 take 29.5 us, 2 more with two warps a block and 7 with four), of as
// many as it has items where all of these run at once (FEW).  Thread j of a head's LANES: chunk j < rot / 16 of q and k is eight pairs, any
// other 16 values in a row; threads past dim / 16, and past a kind's heads, only take part in the shuffles.  A warp
// takes items of 32 / LANES heads of one kind, q_items of q, then kv_items of k, then as many of v.  GROUPS: groups of
// a row in the 4-bit cache, 0: the 16-bit cache.
template <bool BF, int GROUPS, int LANES, bool FEW>
__global__ void __launch_bounds__(FEW ? NORM_MOST : 32, FEW ? 1 : GROUPS ? (LANES == 16 ? 14 : 18) : 20)
    norm_rope_kernel(const NormParams p, int q_items, int kv_items)
{
    pdl_wait();
    pdl_launch_dependents();
    constexpr int AT_ONCE = 32 / LANES;
    const int lane = threadIdx.x & 31, mine = lane / LANES, warps = FEW ? blockDim.x >> 5 : 1;
    TokenOf t;
    t.token = blockIdx.x;
    t.j = lane % LANES;
    t.held = 16 * t.j < p.dim;
    t.turns = t.j < p.rot / 16;
    t.known = true;
    t.live = false;
    t.pg = 0;
    t.in_page = 0;
    int pos = 0;
    long long slot = -1;
    if (t.turns)
        pos = p.positions[(long long)axis_of(p, 8 * t.j) * p.ld_pos + t.token];
    if (p.kv > 0)
        slot = p.slots[t.token];

    const uint32_t lanes = (LANES == 32 ? 0xffffffffu : (1u << LANES % 32) - 1) << (lane - t.j);
    bool all_known = true;

    // All items of a kind that are this warp's, with the next one's values on their way.
    auto each = [&](auto kind_c, int item, int of_kind, const uint16_t *src, int ld, int heads, auto before, auto work) {
        constexpr int KIND = decltype(kind_c)::value;
        const bool halves = KIND != KIND_V && t.turns && !p.adjacent;
        const int apart_by = halves ? p.rot / 2 : 8, step = warps * AT_ONCE;
        int h = item * AT_ONCE + mine;
        src += (long long)t.token * ld + (long long)h * p.dim + (halves ? 8 : 16) * t.j;
        uint4 n0 = make_uint4(0, 0, 0, 0), n1 = n0;
        auto fetch = [&](int head) {
            if (t.held && head < heads) { // (past the heads: whatever was loaded last)
                n0 = *reinterpret_cast<const uint4 *>(src);
                n1 = *reinterpret_cast<const uint4 *>(src + apart_by);
                src += (long long)step * p.dim;
            }
        };
        fetch(h);
        before();
        for (; item < of_kind; item += warps, h += step) {
            const uint4 x0 = n0, x1 = n1;
            fetch(h + step);
            work(x0, x1, h);
        }
    };
    // What waits for the token's position and slot, behind the first loads of values.
    auto look_up = [&]() {
        if (t.turns)
            t.known = angles(p, t.token, t.j, pos, t.c, t.s);
        t.live = p.kv > 0 && page_of(p, slot, t.pg, t.in_page);
        all_known = (__ballot_sync(0xffffffffu, t.known) & lanes) == lanes; // what a coded key needs
    };
    const int warp = FEW ? threadIdx.x >> 5 : 0;
    each(std::integral_constant<int, KIND_Q>(), warp, q_items, p.q, p.ldq, p.heads, look_up, [&](uint4 x0, uint4 x1, int h) {
        uint16_t *dst = p.q_out + (long long)t.token * p.ldqo + (long long)h * p.dim;
        plain_head<BF, LANES>(p, t, x0, x1, p.q_norm, h < p.heads ? dst : nullptr);
    });
    // (a warp's turn: the kinds follow one another)
    const int first_k = (warp + warps - q_items % warps) % warps, first_v = (first_k + warps - kv_items % warps) % warps;
    auto nothing = [] {};
    const long long row = t.pg * p.page_stride + t.in_page * p.token_stride;
    if constexpr (GROUPS == 0) {
        each(std::integral_constant<int, KIND_K>(), first_k, kv_items, p.k, p.ldk, p.kv, nothing, [&](uint4 x0, uint4 x1, int h) {
            uint16_t *dst = p.k_cache + row + h * p.head_stride;
            plain_head<BF, LANES>(p, t, x0, x1, p.k_norm, h < p.kv && t.live ? dst : nullptr);
        });
        each(std::integral_constant<int, KIND_V>(), first_v, kv_items, p.v, p.ldv, p.kv, nothing, [&](uint4 x0, uint4 x1, int h) {
            if (h < p.kv && t.live && t.held) { // copied as it is
                uint16_t *dst = p.v_cache + row + h * p.head_stride + 16 * t.j;
                *reinterpret_cast<uint4 *>(dst) = x0;
                *reinterpret_cast<uint4 *>(dst + 8) = x1;
            }
        });
    } else {
        t.known = all_known;
        each(std::integral_constant<int, KIND_K>(), first_k, kv_items, p.k, p.ldk, p.kv, nothing, [&](uint4 x0, uint4 x1, int h) {
            uint16_t *dst = p.k_out ? p.k_out + (long long)t.token * p.ldko + (long long)h * p.dim : nullptr;
            coded_head<BF, GROUPS, LANES, true>(p, t, x0, x1, h < p.kv, h, dst);
        });
        each(std::integral_constant<int, KIND_V>(), first_v, kv_items, p.v, p.ldv, p.kv, nothing, [&](uint4 x0, uint4 x1, int h) {
            uint16_t *dst = p.v_out ? p.v_out + (long long)t.token * p.ldvo + (long long)h * p.dim : nullptr;
            coded_head<BF, GROUPS, LANES, false>(p, t, x0, x1, h < p.kv, h, dst);
        });
    }
}

// 16-bit cache, any even rot, any dim, any strides: a warp per token and head, a pair (or two values) per lane in
// 2-byte accesses.  Bound by their number.
template <bool BF>
__global__ void __launch_bounds__(32 * NORM_WARPS) norm_rope_any_kernel(const NormParams p, int q_heads, int all)
{
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const long long total = (long long)p.tokens * all;
    for (long long n = (long long)blockIdx.x * NORM_WARPS + (threadIdx.x >> 5); n < total;
         n += (long long)gridDim.x * NORM_WARPS) {
        const int token = (int)(n / all);
        int h = (int)(n - (long long)token * all);
        const int kind = h < q_heads ? KIND_Q : h < q_heads + p.kv ? KIND_K : KIND_V;
        h -= kind == KIND_Q ? 0 : kind == KIND_K ? q_heads : q_heads + p.kv;
        const uint16_t *src = head_src(p, kind, token, h);
        uint16_t *dst;
        if (kind == KIND_Q) {
            dst = p.q_out + (long long)token * p.ldqo + (long long)h * p.dim;
        } else {
            long long pg;
            int in_page;
            if (!page_of(p, p.slots[token], pg, in_page)) {
                if (kind == KIND_K) // its positions are looked at all the same
                    for (int i = lane; i < p.rot / 2; i += 32)
                        checked_position(p, p.positions[(long long)axis_of(p, i) * p.ld_pos + token]);
                continue;
            }
            dst = (kind == KIND_K ? p.k_cache : p.v_cache) + pg * p.page_stride + in_page * p.token_stride +
                  h * p.head_stride;
        }
        const uint16_t *norm = kind == KIND_Q ? p.q_norm : kind == KIND_K ? p.k_norm : nullptr;
        float r = 1.f;
        if (norm) {
            float sum = 0.f;
            for (int i = lane; i < p.dim; i += 32) {
                const float x = to_float<BF>(src[i]);
                sum = fmaf(x, x, sum);
            }
#pragma unroll
            for (int d = 1; d < 32; d <<= 1)
                sum += __shfl_xor_sync(0xffffffffu, sum, d);
            r = rsqrtf(fmaf(sum, p.per_dim, p.eps));
        }
        const int half = p.rot / 2, items = half + (p.dim - p.rot + 1) / 2;
        for (int i = lane; i < items; i += 32) {
            const bool turn = i < half;
            const int a = !turn ? p.rot + 2 * (i - half) : p.adjacent ? 2 * i : i;
            const int b = !turn || p.adjacent ? a + 1 : half + i;
            const bool two = b < p.dim;
            uint16_t ra = src[a], rb = two ? src[b] : 0;
            if (kind != KIND_V && (norm || turn)) {
                float x = to_float<BF>(ra), y = to_float<BF>(rb);
                if (norm) {
                    x = x * r * to_float<BF>(norm[a]);
                    y = two ? y * r * to_float<BF>(norm[b]) : 0.f;
                }
                if (turn) {
                    const int pos = checked_position(p, p.positions[(long long)axis_of(p, i) * p.ld_pos + token]);
                    if (pos < 0)
                        continue;
                    const float c = p.table[(long long)pos * p.rot + i], s = p.table[(long long)pos * p.rot + half + i];
                    const float z = turned_first(x, y, c, s);
                    y = turned_second(x, y, c, s, p.copies16);
                    x = z;
                }
                ra = from_float<BF>(x);
                rb = from_float<BF>(y);
            }
            dst[a] = ra;
            if (two)
                dst[b] = rb;
        }
    }
}

namespace {

// The arguments that both entries have, checked in the order of w4a16_rope_append's.
int check_common(const NormParams &p, const int32_t *sections, int n_pages)
{
    if (p.tokens < 0 || p.heads < 0 || p.kv < 0 || p.heads + (long long)p.kv <= 0 || p.dim <= 0 || p.rot < 0 ||
        p.rot % 2 != 0 || p.rot > p.dim || (p.kv > 0 && (p.page <= 0 || n_pages <= 0)) || !(p.eps >= 0.f) ||
        p.eps == INFINITY)
        return status_of(STAGE_ARG, W4A16_ARG_SHAPE);
    if (p.rot > 0) {
        if (p.max_pos <= 0 || p.axes <= 0 || p.axes > NORM_MAX_AXES)
            return status_of(STAGE_ARG, W4A16_ARG_SHAPE);
        if (!sections)
            return status_of(STAGE_ARG, W4A16_ARG_NULL);
    } else if (p.axes != 0) {
        return status_of(STAGE_ARG, W4A16_ARG_SHAPE);
    }
    long long sum = 0;
    for (int a = 0; a < p.axes; ++a) {
        if (sections[a] < 0)
            return status_of(STAGE_ARG, W4A16_ARG_SHAPE);
        sum += sections[a];
    }
    return sum == p.rot / 2 ? 0 : status_of(STAGE_ARG, W4A16_ARG_SHAPE);
}

// What calls without heads of a kind, or without rotation, would use is not looked at, its alignment included.
void drop_absent(NormParams &p)
{
    if (p.heads == 0)
        p.q = nullptr, p.q_out = nullptr, p.q_norm = nullptr;
    if (p.kv == 0) {
        p.k = p.v = p.k_norm = nullptr;
        p.k_cache = p.v_cache = p.k_out = p.v_out = nullptr;
        p.cache = nullptr;
        p.slots = nullptr;
    }
    if (p.rot == 0)
        p.table = nullptr, p.positions = nullptr;
}

int check_buffers(const NormParams &p)
{
    if ((p.rot > 0 && (!p.table || !p.positions)) || (p.heads > 0 && (!p.q || !p.q_out)) ||
        (p.kv > 0 && (!p.k || !p.v || !p.slots)))
        return status_of(STAGE_ARG, W4A16_ARG_NULL);
    const long long qw = (long long)p.heads * p.dim, kw = (long long)p.kv * p.dim;
    if (qw > 0x7FFFFFFFLL || kw > 0x7FFFFFFFLL || (long long)p.heads + 2LL * p.kv > (1 << 20))
        return status_of(STAGE_ARG, W4A16_ARG_OVERFLOW);
    if (p.ldq < qw || p.ldqo < qw || p.ldk < kw || p.ldv < kw || (p.k_out && p.ldko < kw) || (p.v_out && p.ldvo < kw) ||
        (p.rot > 0 && p.ld_pos < p.tokens))
        return status_of(STAGE_ARG, W4A16_ARG_SHAPE);
    if (!aligned(p.q, 2) || !aligned(p.k, 2) || !aligned(p.v, 2) || !aligned(p.q_out, 2) || !aligned(p.q_norm, 2) ||
        !aligned(p.k_norm, 2) || !aligned(p.table, 4) || !aligned(p.positions, 4) || !aligned(p.slots, 8) ||
        !aligned(p.status, 4))
        return status_of(STAGE_ARG, W4A16_ARG_ALIGN);
    return 0;
}

// Whether q, k, v and what both entries write in 16 bits can be copied 16 bytes at a time.
bool wide(const NormParams &p)
{
    const long long any = (p.heads ? (long long)(p.ldq | p.ldqo) : 0) | (p.kv ? p.ldk | p.ldv : 0);
    return p.dim % 16 == 0 && p.rot % 16 == 0 && any % 8 == 0 && aligned(p.q, 16) && aligned(p.k, 16) &&
           aligned(p.v, 16) && aligned(p.q_out, 16) && aligned(p.q_norm, 16) && aligned(p.k_norm, 16) &&
           aligned(p.table, 16);
}

template <bool BF, int GROUPS, int LANES>
int launch_lanes(const NormParams &p, cudaStream_t stream)
{
    int num_sms = 0;
    const cudaError_t err = sm_count(&num_sms);
    if (err != cudaSuccess)
        return status_of(STAGE_RESOURCE, err);
    constexpr int AT_ONCE = 32 / LANES; // heads of a warp
    const int q_items = (p.heads + AT_ONCE - 1) / AT_ONCE, kv_items = (p.kv + AT_ONCE - 1) / AT_ONCE;
    const int items = q_items + 2 * kv_items;
    // A warp per item while the GPU has room for all of them: a call of few tokens is as long as its longest warp.
    if ((long long)p.tokens * items <= (long long)num_sms * NORM_PER_SM) {
        const int warps = items < NORM_MOST / 32 ? items : NORM_MOST / 32;
        return launch_status(launch_pdl(norm_rope_kernel<BF, GROUPS, LANES, true>, dim3((unsigned)p.tokens),
                                        dim3(32 * warps), 0, stream, p, q_items, kv_items));
    }
    return launch_status(launch_pdl(norm_rope_kernel<BF, GROUPS, LANES, false>, dim3((unsigned)p.tokens), dim3(32), 0,
                                    stream, p, q_items, kv_items));
}

template <int GROUPS, int LANES>
int launch_type(bool bf, const NormParams &p, cudaStream_t stream)
{
    return bf ? launch_lanes<true, GROUPS, LANES>(p, stream) : launch_lanes<false, GROUPS, LANES>(p, stream);
}

NormParams params(const void *q, int ldq, const void *k, int ldk, const void *v, int ldv, const void *q_norm,
                  const void *k_norm, float eps, void *q_out, int ldqo, const float *cos_sin, int max_pos,
                  const int32_t *positions, int ld_pos, const long long *slots, int32_t *status, int n_tokens,
                  int n_heads, int n_kv_heads, int head_dim, int rot_dim, int n_axes, int page_size, int n_pages,
                  unsigned flags)
{
    NormParams p = {};
    p.q = static_cast<const uint16_t *>(q);
    p.k = static_cast<const uint16_t *>(k);
    p.v = static_cast<const uint16_t *>(v);
    p.q_norm = static_cast<const uint16_t *>(q_norm);
    p.k_norm = static_cast<const uint16_t *>(k_norm);
    p.q_out = static_cast<uint16_t *>(q_out);
    p.table = cos_sin;
    p.positions = positions;
    p.slots = slots;
    p.status = status;
    p.total_slots = (long long)n_pages * page_size;
    p.eps = eps;
    p.per_dim = head_dim > 0 ? 1.f / (float)head_dim : 0.f;
    p.ldq = ldq;
    p.ldk = ldk;
    p.ldv = ldv;
    p.ldqo = ldqo;
    p.ld_pos = ld_pos;
    p.tokens = n_tokens;
    p.heads = n_heads;
    p.kv = n_kv_heads;
    p.dim = head_dim;
    p.rot = rot_dim;
    p.axes = n_axes;
    p.max_pos = max_pos;
    p.page = page_size;
    p.adjacent = (flags & W4A16_FLAG_ROPE_ADJACENT) ? 1 : 0;
    return p;
}

void set_cuts(NormParams &p, const int32_t *sections)
{
    int cut = 0;
    for (int a = 0; a < NORM_MAX_AXES; ++a) {
        if (a < p.axes)
            cut += sections[a];
        p.cut[a] = cut;
    }
    p.cuts = 0;
    for (int a = 0; a < p.axes - 1; ++a)
        p.cuts |= p.cut[a] % 8 != 0;
}

} // namespace
} // namespace ops
} // namespace w4

using namespace w4;
using namespace w4::ops;

extern "C" int w4a16_norm_rope_append(const void *q, int ldq, const void *k, int ldk, const void *v, int ldv,
                                      const void *q_norm, const void *k_norm, float eps, void *q_out, int ldqo,
                                      void *k_cache, void *v_cache, long long kv_page_stride,
                                      long long kv_token_stride, long long kv_head_stride, const float *cos_sin,
                                      int max_pos, const int32_t *positions, int ld_pos, const long long *slots,
                                      int32_t *status, int n_tokens, int n_heads, int n_kv_heads, int head_dim,
                                      int rot_dim, const int32_t *sections, int n_axes, int page_size, int n_pages,
                                      unsigned flags, cudaStream_t stream)
{
    if (flags & ~(W4A16_FLAG_BF16 | W4A16_FLAG_ROPE_ADJACENT))
        return status_of(STAGE_ARG, W4A16_ARG_FLAGS);
    NormParams p = params(q, ldq, k, ldk, v, ldv, q_norm, k_norm, eps, q_out, ldqo, cos_sin, max_pos, positions,
                          ld_pos, slots, status, n_tokens, n_heads, n_kv_heads, head_dim, rot_dim, n_axes, page_size,
                          n_pages, flags);
    int st = check_common(p, sections, n_pages);
    if (st)
        return st;
    if (n_tokens == 0)
        return 0;
    p.k_cache = static_cast<uint16_t *>(k_cache);
    p.v_cache = static_cast<uint16_t *>(v_cache);
    drop_absent(p);
    if (n_kv_heads > 0 && (!k_cache || !v_cache))
        return status_of(STAGE_ARG, W4A16_ARG_NULL);
    st = check_buffers(p);
    if (st)
        return st;
    if (n_kv_heads > 0 && (kv_page_stride < 0 || kv_token_stride < 0 || kv_head_stride < 0))
        return status_of(STAGE_ARG, W4A16_ARG_SHAPE);
    if (!aligned(p.k_cache, 2) || !aligned(p.v_cache, 2))
        return status_of(STAGE_ARG, W4A16_ARG_ALIGN);
    p.page_stride = kv_page_stride;
    p.token_stride = kv_token_stride;
    p.head_stride = kv_head_stride;
    set_cuts(p, sections);
    const bool bf = (flags & W4A16_FLAG_BF16) != 0;
    const long long strides = n_kv_heads ? kv_page_stride | kv_token_stride | kv_head_stride : 0;
    p.copies16 = wide(p) && strides % 8 == 0 && aligned(p.k_cache, 16) && aligned(p.v_cache, 16);
    if (p.copies16 && head_dim <= 512)
        return head_dim <= 64    ? launch_type<0, 4>(bf, p, stream)
               : head_dim <= 128 ? launch_type<0, 8>(bf, p, stream)
               : head_dim <= 256 ? launch_type<0, 16>(bf, p, stream)
                                 : launch_type<0, 32>(bf, p, stream);
    int num_sms = 0;
    const cudaError_t err = sm_count(&num_sms);
    if (err != cudaSuccess)
        return status_of(STAGE_RESOURCE, err);
    const int all = n_heads + 2 * n_kv_heads;
    const long long want = ((long long)n_tokens * all + NORM_WARPS - 1) / NORM_WARPS, most = 16LL * num_sms;
    const dim3 grid((unsigned)(want < most ? want : most)), block(32 * NORM_WARPS);
    return launch_status(bf ? launch_pdl(norm_rope_any_kernel<true>, grid, block, 0, stream, p, n_heads, all)
                            : launch_pdl(norm_rope_any_kernel<false>, grid, block, 0, stream, p, n_heads, all));
}

extern "C" size_t w4a16_kv4_record_bytes(int page_size, int head_dim, int group_size)
{
    const int groups = kv4_dim(head_dim) ? kv4_groups(head_dim, group_size) : 0;
    if (page_size <= 0 || page_size > W4A16_KV4_MAX_PAGE || groups == 0)
        return 0;
    return (size_t)kv4_record_bytes(page_size, head_dim, groups);
}

extern "C" int w4a16_kv4_append(const void *q, int ldq, const void *k, int ldk, const void *v, int ldv,
                                const void *q_norm, const void *k_norm, float eps, void *q_out, int ldqo, void *cache,
                                long long page_stride, void *k_out, int ldko, void *v_out, int ldvo,
                                const float *cos_sin, int max_pos, const int32_t *positions, int ld_pos,
                                const long long *slots, int32_t *status, int n_tokens, int n_heads, int n_kv_heads,
                                int head_dim, int rot_dim, const int32_t *sections, int n_axes, int page_size,
                                int n_pages, int group_size, unsigned flags, cudaStream_t stream)
{
    if (flags & ~(W4A16_FLAG_BF16 | W4A16_FLAG_ROPE_ADJACENT))
        return status_of(STAGE_ARG, W4A16_ARG_FLAGS);
    NormParams p = params(q, ldq, k, ldk, v, ldv, q_norm, k_norm, eps, q_out, ldqo, cos_sin, max_pos, positions,
                          ld_pos, slots, status, n_tokens, n_heads, n_kv_heads, head_dim, rot_dim, n_axes, page_size,
                          n_pages, flags);
    int st = check_common(p, sections, n_pages);
    if (st)
        return st;
    if (n_kv_heads <= 0)
        return status_of(STAGE_ARG, W4A16_ARG_SHAPE);
    if (!kv4_dim(head_dim) || rot_dim % 16 != 0 || page_size > W4A16_KV4_MAX_PAGE)
        return status_of(STAGE_UNSUPPORTED, W4A16_ARG_SHAPE);
    const int groups = kv4_groups(head_dim, group_size);
    if (groups == 0)
        return status_of(STAGE_ARG, W4A16_ARG_GROUP);
    if (n_tokens == 0)
        return 0;
    p.cache = static_cast<uint8_t *>(cache);
    p.k_out = static_cast<uint16_t *>(k_out);
    p.v_out = static_cast<uint16_t *>(v_out);
    p.ldko = ldko;
    p.ldvo = ldvo;
    drop_absent(p);
    if (!cache)
        return status_of(STAGE_ARG, W4A16_ARG_NULL);
    st = check_buffers(p);
    if (st)
        return st;
    p.rec = kv4_record(page_size, head_dim, groups);
    if (page_stride < n_kv_heads * p.rec.bytes)
        return status_of(STAGE_ARG, W4A16_ARG_SHAPE);
    if (!wide(p) || page_stride % 16 != 0 || !aligned(cache, 16) || !aligned(k_out, 16) || !aligned(v_out, 16) ||
        (k_out && ldko % 8 != 0) || (v_out && ldvo % 8 != 0))
        return status_of(STAGE_ARG, W4A16_ARG_ALIGN);
    p.page_stride = page_stride;
    p.head_stride = p.rec.bytes;
    set_cuts(p, sections);
    const bool bf = (flags & W4A16_FLAG_BF16) != 0;
    if (head_dim == 64)
        return launch_type<1, 4>(bf, p, stream);
    if (head_dim == 128)
        return groups == 1 ? launch_type<1, 8>(bf, p, stream) : launch_type<2, 8>(bf, p, stream);
    return groups == 1   ? launch_type<1, 16>(bf, p, stream)
           : groups == 2 ? launch_type<2, 16>(bf, p, stream)
                         : launch_type<4, 16>(bf, p, stream);
}
