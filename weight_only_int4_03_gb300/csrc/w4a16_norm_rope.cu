// w4a16_norm_rope.cu -- norms of queries and keys per head, rotary positions, and keys and values
// written into a paged cache, of 16 bits or held in 4.
//
// For every head of q and k, with weights w (no weights: y = x):
//     y = x rsqrt(mean x^2 + eps) w,
// then pair i < rot_dim / 2 is turned by its position's angle, (y1, y2) -> (y1 c - y2 s, y2 c + y1 s), as
// w4a16_rope_append does.  All in fp32; q, and k and v of the 16-bit cache, are rounded once.  In the
// 4-bit cache a group of values is coded from the fp32 results:
//     b = r(min),  s = r((max - min) / 15),  code = (x - b) / s to the nearest integer, ties to even, in 0..15
// (r: to the cache's 16-bit type), which stands for code s + b.
//
// Bound by memory: each value is read once and written once.  A thread holds 16 values of a head
// (eight pairs) of NORM_HEADS heads of one kind (q, k or v), so that the weights stay in registers and a
// position's cosines and sines serve all of them; the D / 16 threads of a head lie in one warp and
// meet in shuffles for the sum of squares and for the groups' smallest and largest values.  Threads walk over
// tokens with the next token's values on their way.
#include "w4a16_kv4.cuh"

namespace w4 {
namespace ops {

constexpr int NORM_MAX_AXES = 4;
constexpr int NORM_HEADS = 2;
constexpr int NORM_THREADS = 128; // threads a block is filled up to
constexpr int NORM_PER_SM = 512;  // threads per SM that a launch asks for and the registers allow
constexpr int NORM_WARPS = 4;     // any-size kernel: warps of a block

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
    float eps;
    int ldq, ldk, ldv, ldqo, ldko, ldvo, ld_pos;
    int tokens, heads, kv, dim, rot, axes, max_pos, page;
    int cut[NORM_MAX_AXES]; // pair i belongs to the first axis a with i < cut[a]
    int adjacent;
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

// The rotation, in the same roundings wherever it is used.
__device__ __forceinline__ float turned_first(float a, float b, float c, float s)
{
    return fmaf(a, c, -(b * s));
}

__device__ __forceinline__ float turned_second(float a, float b, float c, float s)
{
    return fmaf(b, c, a * s);
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

// How a group of values is coded: the step and base as stored, and what coding needs of them.
struct Step {
    uint32_t stored;   // step, base (16 bits each)
    float s, b;        // as numbers; both NaN where the group has no finite range
    float from, inv, half;
};

template <bool BF>
__device__ __forceinline__ Step step_of(float lo, float hi)
{
    Step st;
    uint16_t sb = from_float<BF>((hi - lo) / 15.f), bb = from_float<BF>(lo);
    if (BF && (sb & 0x7F80) == 0)
        sb = 0; // a subnormal bf16 step has no inverse in fp32
    st.s = to_float<BF>(sb);
    st.b = to_float<BF>(bb);
    const bool fine = fabsf(st.s) < INFINITY && fabsf(st.b) < INFINITY; // false for NaN too
    st.from = fine ? st.b : 0.f;
    st.inv = fine && st.s > 0.f ? 1.f / st.s : 0.f;
    st.half = fine && st.s > 0.f ? 0.5f * st.s : INFINITY;
    if (!fine) {
        st.s = st.b = NAN;
        sb = bb = 0x7FFF; // NaN in both types
    }
    st.stored = (uint32_t)sb | (uint32_t)bb << 16;
    return st;
}

// The code of x: (x - b) / s to the nearest integer, ties to even.  The product with 1 / s is off by a few
// 2^-24, which decides wrongly only next to the middle between two codes: there the exact rest
// d - q s says which it is (values of the 16-bit types do lie on the middle).
__device__ __forceinline__ uint32_t code_of(float x, const Step &st)
{
    const float d = x - st.from;
    float q = rintf(d * st.inv);
    const float r = fmaf(-q, st.s, d);
    if (fabsf(r) >= st.half) {
        const bool odd = ((int)q & 1) != 0;
        if (r > st.half || (r == st.half && odd))
            q += 1.f;
        else if (r < -st.half || (r == -st.half && odd))
            q -= 1.f;
    }
    return (uint32_t)(int)fminf(fmaxf(q, 0.f), 15.f);
}

// Eight values at 8 * word of a row: coded into its word, and replaced by what the codes stand for.
__device__ __forceinline__ uint32_t code_eight(float *x, const Step &st)
{
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t c = code_of(x[i], st);
        word |= c << (4 * i);
        x[i] = fmaf((float)c, st.s, st.b);
    }
    return word;
}

template <bool BF>
__device__ __forceinline__ void unpack8(const uint4 &v, float *x)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2<BF>(w[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

template <bool BF>
__device__ __forceinline__ uint4 pack8(const float *x)
{
    return make_uint4(pack2<BF>(x[0], x[1]), pack2<BF>(x[2], x[3]), pack2<BF>(x[4], x[5]), pack2<BF>(x[6], x[7]));
}

// 16-byte path.  Item (kind, head group, chunk j) of a thread: chunk j < rot / 16 of q and k is eight pairs, any
// other 16 values in a row.  `lanes` threads, a power of two, belong to a head; those past dim / 16 only take part
// in the shuffles.  GROUPS: groups of a row in the 4-bit cache, 0: the 16-bit cache.  CUTS: some section ends
// inside a chunk.
template <bool BF, int GROUPS, bool CUTS>
__global__ void __launch_bounds__(256, NORM_PER_SM / 256)
    norm_rope_kernel(const NormParams p, int lanes, int q_groups, int kv_groups)
{
    pdl_wait();
    pdl_launch_dependents();
    const int item = blockIdx.y * blockDim.x + threadIdx.x;
    const int stride = gridDim.x * blockDim.y;
    int token = blockIdx.x * blockDim.y + threadIdx.y;
    int g = item / lanes;
    const int j = item - g * lanes;
    if (g >= q_groups + 2 * kv_groups || token >= p.tokens)
        return; // whole groups of lanes
    const uint32_t lane_id = (threadIdx.y * blockDim.x + threadIdx.x) & 31;
    const uint32_t mask = (lanes == 32 ? 0xffffffffu : (1u << lanes) - 1) << (lane_id & ~(uint32_t)(lanes - 1));
    const int kind = g < q_groups ? KIND_Q : g < q_groups + kv_groups ? KIND_K : KIND_V;
    g -= kind == KIND_Q ? 0 : kind == KIND_K ? q_groups : q_groups + kv_groups;
    const int h0 = g * NORM_HEADS, heads = kind == KIND_Q ? p.heads : p.kv;
    const int half = p.rot / 2;
    const bool held = 16 * j < p.dim;                       // this thread has values
    const bool pairs = kind != KIND_V && j < p.rot / 16;
    const bool halves = pairs && !p.adjacent;
    const int at0 = halves ? 8 * j : 16 * j, at1 = halves ? half + 8 * j : 16 * j + 8;
    const bool cached = kind != KIND_Q;
    const int axis0 = pairs ? axis_of(p, 8 * j) : 0, axis1 = CUTS && pairs ? axis_of(p, 8 * j + 7) : axis0;
    const int32_t *positions = p.positions + (long long)axis0 * p.ld_pos;
    const uint16_t *norm = kind == KIND_Q ? p.q_norm : kind == KIND_K ? p.k_norm : nullptr;
    uint4 w0 = make_uint4(0, 0, 0, 0), w1 = w0;
    if (norm && held) {
        w0 = *reinterpret_cast<const uint4 *>(norm + at0);
        w1 = *reinterpret_cast<const uint4 *>(norm + at1);
    }

    int next_pos = 0;
    long long next_slot = -1;
    uint4 n0[NORM_HEADS], n1[NORM_HEADS];
#pragma unroll
    for (int n = 0; n < NORM_HEADS; ++n)
        n0[n] = n1[n] = make_uint4(0, 0, 0, 0);
    auto fetch = [&](int t) {
#pragma unroll
        for (int n = 0; n < NORM_HEADS; ++n)
            if (held && h0 + n < heads) {
                const uint16_t *src = head_src(p, kind, t, h0 + n);
                n0[n] = *reinterpret_cast<const uint4 *>(src + at0);
                n1[n] = *reinterpret_cast<const uint4 *>(src + at1);
            }
        if (pairs)
            next_pos = positions[t];
        if (cached)
            next_slot = p.slots[t];
    };
    fetch(token);
    for (;;) {
        uint4 x0[NORM_HEADS], x1[NORM_HEADS];
#pragma unroll
        for (int n = 0; n < NORM_HEADS; ++n) {
            x0[n] = n0[n];
            x1[n] = n1[n];
        }
        const int t = token, pos = pairs ? checked_position(p, next_pos) : 0;
        long long pg = 0;
        int in_page = 0;
        const bool live = cached && page_of(p, next_slot, pg, in_page);
        bool known = pos >= 0;
        float c[8], s[8];
        if (pairs && known) {
            const float *entry = p.table + (long long)pos * p.rot + 8 * j;
#pragma unroll
            for (int i = 0; i < 8; i += 4) {
                *reinterpret_cast<float4 *>(c + i) = *reinterpret_cast<const float4 *>(entry + i);
                *reinterpret_cast<float4 *>(s + i) = *reinterpret_cast<const float4 *>(entry + half + i);
            }
            if (CUTS) {
                // The pairs from a further section's start on take that axis's entries.
#pragma unroll 1
                for (int a = axis0 + 1; a <= axis1; ++a) {
                    const int from = p.cut[a - 1] - 8 * j;
                    if (p.cut[a] == p.cut[a - 1])
                        continue;
                    const int pa = checked_position(p, p.positions[(long long)a * p.ld_pos + t]);
                    known &= pa >= 0;
                    const float *other = p.table + (long long)max(pa, 0) * p.rot + 8 * j;
#pragma unroll
                    for (int i = 0; i < 8; i += 4) {
                        const float4 c4 = *reinterpret_cast<const float4 *>(other + i);
                        const float4 s4 = *reinterpret_cast<const float4 *>(other + half + i);
                        const float cc[4] = {c4.x, c4.y, c4.z, c4.w}, ss[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            if (i + q >= from) {
                                c[i + q] = cc[q];
                                s[i + q] = ss[q];
                            }
                    }
                }
            }
        }
        const bool more = p.tokens - token > stride; // (the sum may pass 31 bits)
        if (more) {
            token += stride;
            fetch(token);
        }
        // A key in 4 bits needs all of its positions, as its groups are coded together.
        const bool whole = GROUPS > 0 && kind == KIND_K ? __all_sync(mask, known) != 0 : known;
#pragma unroll
        for (int n = 0; n < NORM_HEADS; ++n) {
            const int h = h0 + n;
            if (h >= heads)
                break; // whole groups of lanes
            if (GROUPS == 0 && kind == KIND_V) { // copied as it is
                if (live && held) {
                    uint16_t *dst = p.v_cache + pg * p.page_stride + in_page * p.token_stride + h * p.head_stride;
                    *reinterpret_cast<uint4 *>(dst + at0) = x0[n];
                    *reinterpret_cast<uint4 *>(dst + at1) = x1[n];
                }
                continue;
            }
            float x[16];
            unpack8<BF>(x0[n], x);
            unpack8<BF>(x1[n], x + 8);
            if (norm) {
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    sum = fmaf(x[i], x[i], sum);
                for (int d = 1; d < lanes; d <<= 1)
                    sum += __shfl_xor_sync(mask, sum, d);
                const float r = rsqrtf(sum / (float)p.dim + p.eps);
                float w[16];
                unpack8<BF>(w0, w);
                unpack8<BF>(w1, w + 8);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    x[i] = x[i] * r * w[i];
            }
            if (pairs && whole) {
                if (p.adjacent) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float a = x[2 * i], b = x[2 * i + 1];
                        x[2 * i] = turned_first(a, b, c[i], s[i]);
                        x[2 * i + 1] = turned_second(a, b, c[i], s[i]);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float a = x[i], b = x[8 + i];
                        x[i] = turned_first(a, b, c[i], s[i]);
                        x[8 + i] = turned_second(a, b, c[i], s[i]);
                    }
                }
            }
            uint16_t *dst = nullptr; // 16-bit results
            if (kind == KIND_Q)
                dst = p.q_out + (long long)t * p.ldqo + (long long)h * p.dim;
            else if (GROUPS == 0)
                dst = live ? p.k_cache + pg * p.page_stride + in_page * p.token_stride + h * p.head_stride : nullptr;
            else if (kind == KIND_K)
                dst = p.k_out ? p.k_out + (long long)t * p.ldko + (long long)h * p.dim : nullptr;
            else
                dst = p.v_out ? p.v_out + (long long)t * p.ldvo + (long long)h * p.dim : nullptr;
            if (GROUPS > 0 && kind != KIND_Q) {
                constexpr int N = GROUPS > 0 ? GROUPS : 1;
                // Groups are whole blocks of 64 values, and each half of a thread's values lies in one of them.
                const int size = p.dim / N, g0 = at0 / size, g1 = at1 / size;
                float lo[2] = {x[0], x[8]}, hi[2] = {x[0], x[8]};
#pragma unroll
                for (int i = 1; i < 8; ++i)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        lo[e] = min_nan(lo[e], x[8 * e + i]);
                        hi[e] = max_nan(hi[e], x[8 * e + i]);
                    }
                Step st0, st1;
                uint32_t stored = 0;
#pragma unroll
                for (int q = 0; q < N; ++q) {
                    float l = INFINITY, m = -INFINITY;
                    if (held && g0 == q) {
                        l = lo[0];
                        m = hi[0];
                    }
                    if (held && g1 == q) {
                        l = min_nan(l, lo[1]);
                        m = max_nan(m, hi[1]);
                    }
                    for (int d = 1; d < lanes; d <<= 1) {
                        l = min_nan(l, __shfl_xor_sync(mask, l, d));
                        m = max_nan(m, __shfl_xor_sync(mask, m, d));
                    }
                    const Step st = step_of<BF>(l, m);
                    if (q == 0 || g0 == q)
                        st0 = st;
                    if (q == 0 || g1 == q)
                        st1 = st;
                    if (j == q)
                        stored = st.stored;
                }
                const uint32_t word0 = code_eight(x, st0), word1 = code_eight(x + 8, st1);
                if (live && held && whole) {
                    uint8_t *row = p.cache + pg * p.page_stride + h * p.head_stride;
                    uint32_t *codes = reinterpret_cast<uint32_t *>(row + (kind == KIND_V ? p.rec.values : 0)) +
                                      (long long)in_page * (p.dim / 8);
                    const int blocks = p.dim / 64;
                    const int a0 = kind == KIND_K ? kv4_key_place(at0 / 8, blocks) : kv4_value_place(at0 / 8, blocks);
                    const int a1 = kind == KIND_K ? kv4_key_place(at1 / 8, blocks) : kv4_value_place(at1 / 8, blocks);
                    codes[a0] = word0;
                    codes[a1] = word1;
                    if (j < N)
                        reinterpret_cast<uint32_t *>(row + (kind == KIND_K ? p.rec.key_params : p.rec.value_params))
                            [(long long)in_page * N + j] = stored;
                }
            }
            if (dst && held && whole) {
                *reinterpret_cast<uint4 *>(dst + at0) = pack8<BF>(x);
                *reinterpret_cast<uint4 *>(dst + at1) = pack8<BF>(x + 8);
            }
        }
        if (!more)
            return;
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
            if (!page_of(p, p.slots[token], pg, in_page))
                continue;
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
            r = rsqrtf(sum / (float)p.dim + p.eps);
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
                    y = turned_second(x, y, c, s);
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
    return p.dim % 16 == 0 && p.rot % 16 == 0 && p.dim <= 512 && any % 8 == 0 && aligned(p.q, 16) && aligned(p.k, 16) &&
           aligned(p.v, 16) && aligned(p.q_out, 16) && aligned(p.q_norm, 16) && aligned(p.k_norm, 16) &&
           aligned(p.table, 16);
}

template <bool BF, int GROUPS>
int launch_wide(const NormParams &p, cudaStream_t stream)
{
    int lanes = 1;
    while (16 * lanes < p.dim)
        lanes *= 2;
    const int q_groups = (p.heads + NORM_HEADS - 1) / NORM_HEADS, kv_groups = (p.kv + NORM_HEADS - 1) / NORM_HEADS;
    const long long items = (long long)lanes * (q_groups + 2LL * kv_groups);
    // Blocks of whole tokens up to NORM_THREADS; wider tokens take blocks of their own side by side.
    const int bx = items < 256 ? (int)items : 256;
    const long long side = (items + bx - 1) / bx;
    if (side > 65535)
        return status_of(STAGE_ARG, W4A16_ARG_OVERFLOW);
    int by = NORM_THREADS / bx;
    by = by < 1 ? 1 : by > p.tokens ? p.tokens : by;
    int num_sms = 0;
    const cudaError_t err = sm_count(&num_sms);
    if (err != cudaSuccess)
        return status_of(STAGE_RESOURCE, err);
    const long long groups = (p.tokens + (long long)by - 1) / by;
    long long blocks = (long long)num_sms * (NORM_PER_SM / (bx * by)) / side;
    blocks = blocks < 1 ? 1 : blocks > groups ? groups : blocks;
    bool cuts = false;
    for (int a = 0; a < p.axes - 1; ++a)
        cuts |= p.cut[a] % 8 != 0;
    const auto kernel = cuts ? norm_rope_kernel<BF, GROUPS, true> : norm_rope_kernel<BF, GROUPS, false>;
    return launch_status(launch_pdl(kernel, dim3((unsigned)blocks, (unsigned)side), dim3(bx, by), 0, stream, p, lanes,
                                    q_groups, kv_groups));
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
    if (wide(p) && strides % 8 == 0 && aligned(p.k_cache, 16) && aligned(p.v_cache, 16))
        return bf ? launch_wide<true, 0>(p, stream) : launch_wide<false, 0>(p, stream);
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
    if (flags & W4A16_FLAG_BF16)
        return groups == 1   ? launch_wide<true, 1>(p, stream)
               : groups == 2 ? launch_wide<true, 2>(p, stream)
                             : launch_wide<true, 4>(p, stream);
    return groups == 1   ? launch_wide<false, 1>(p, stream)
           : groups == 2 ? launch_wide<false, 2>(p, stream)
                         : launch_wide<false, 4>(p, stream);
}
