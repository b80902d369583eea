// w4a16_kv4_attention.cu -- attention of one new token per sequence over a paged cache held in 4 bits.
//
// For sequence b, query head h of KV head c, over the positions i in [first, len), with the codes k, v in
// 0..15 and the steps s and bases a of the groups of values (w4a16_kv4.cuh):
//     x_i = scale sum_groups (s_i (q . k_i) + a_i sum q),   p_i = e^(x_i - max x),   l = sum p_i,
//     out = sum_i ((p_i s_i) (v_i - 8) + p_i (a_i + 8 s_i)) / l,   lse = max x + log l.
// So neither side is turned back into 16-bit values: codes go into the products as they are, steps and bases
// are applied in fp32 to sums and to p.  That values are v - 8 keeps the sums over a long axis near zero.
//
// Bound by memory in principle, by instructions in fact: a position of a KV head of 128 is 136 bytes,
// which at the copy rate leaves an SM 6 cycles for it.  What the design does about it:
//   - A code is the fp16 number q 2^-24 (or q 2^-20, four bits higher) as soon as the others are masked
//     off, so that a pair of keys costs one instruction and a shift for every second.  Values q 2^-20 meet queries a
//     sixteenth as large, and outputs of their own factor.  That holds for fp16 alone, so queries are
//     scaled to fp16 by a power of two per head (the largest to 2^13 or more, half of them to a sixteenth of that: off by at
//     most 2^-34 of the largest), whatever the cache's type.
//   - Values are taken two bits higher, q 2^-22 and q 2^-18, which costs a shift more: the tensor core aligns products by
//     their operands' exponents, a subnormal operand's being that of 2^-14, and cuts off what lies below the sum's 24 bits
//     or so from there.  For the same reason p s and its remainder have sums of their own, which only add exact products.
//     (With codes at 2^-24 and one chain for both, 36 % of the fp16 outputs over 131071 positions were not the formula's
//     rounded, all off in one direction; 1.5 % now.  That took 123 us instead of 129 for the 48 sequences below.)
//   - Positions are the rows of the score product (S^T = K Q^T) and value dims those of the value product
//     (O^T = V^T P^T), so that eight heads fill an m16n8k16.  P^T is the scores' fragment transposed by
//     movmatrix.  p s goes in as fp16, times a power of two that keeps it below 2^15, and the 16-bit remainder: 2^-22 of
//     itself down to 2^-16 of the largest step's, and 2^-38 of that below.  (Without the remainder, in bf16, the two long
//     cases below took 38 and 106 us; 2^-11 shows where outputs nearly cancel.)
//   - The maximum is lazy: it moves only when a score passes it by a factor of 4, and a step of 32 positions
//     asks for that by one vote; sums of p and of p a are kept per lane until the end.
//   - A value product starts from -8 sum p s (an MMA against constants makes it) and is added to the outputs in
//     fp32 every step: the MMA cuts sums off, which over many positions of one sign would show.
//   - The words of a row lie in the order of the lanes, so that a lane's share of a row is one load; keys are
//     copied to places that only the copying lane reads.  Where pages hold multiples of 16 positions, a page is
//     looked up once for 16 of them, and masks are applied only in steps that have something to mask.
// bf16, 128 wide: 48 sequences of 2048 to 32768 positions, 64 / 8 heads, 129 us, 4.6 TB/s of codes and parameters (the
// 16-bit cache's bytes would take 327 us at the copy rate); one of 131071 with 40 / 8 heads and groups of 64 45.5 us, 3.3
// TB/s, of which about 10 us pass before the first rows and in the join; fp16, 24 sequences of 5 to 9000 with a window of
// 2048, 12 / 12 heads of 64: 14.3 us, of which most is the start and the join; one of 41 positions: 4.4 us of latencies.
// Per 16 positions of 128 values: 8 score MMAs, 16 value MMAs and two for the start of each group, 96 conversions of codes.
// Eight warps per SM are what the registers allow: issue slots 52 % busy, ALU 48 %, MMA pipe 38 % in the 48 sequences.
// Heads of 256 spill (up to 140 bytes) and take eight heads at a time: a KV head of 16 is read twice.
// The work is split as in the 16-bit cache's attention (w4a16_split.cuh).
#include <type_traits>

#include "w4a16_kv4.cuh"
#include "w4a16_split.cuh"

namespace w4 {
namespace ops {

constexpr float KV4_UP = 8192.f;                       // what p s / reference is multiplied by for the value product
constexpr float KV4_LAZY = 2.f;                        // by how much (log2) a score may pass the maximum

struct Kv4AttParams {
    const uint16_t *q;
    const uint8_t *cache;
    uint16_t *out;
    float *lse;
    const int32_t *table;
    SplitParams split;
    long long page_stride;
    Kv4Record rec;
    int ldq, ldo, ld_table;
    int heads, group, tiles;
    int page, n_pages;
    uint32_t page_magic, page_shift; // position / page = umulhi(position, magic) >> shift; magic 0: page 1
    float scale_log2;
};

template <int D, int G, int NT>
struct Kv4Geom {
    static constexpr int BLOCKS = D / 64;
    static constexpr int ROW = D / 2;                  // bytes of a row of codes
    static constexpr int LANE = ROW / 4;               // a lane's bytes of a key row
    static constexpr int KEYS = 16 * ROW;              // a sub-step's keys, and as many bytes of values
    static constexpr int PARAMS = 16 * 4 * G;          // a sub-step's steps and bases of one side
    static constexpr int SUB = 2 * KEYS + 2 * PARAMS;
    // Sub-steps of 16 positions that a warp takes at once: what a step costs by itself (pages, the vote, adding up the
    // outputs) is shared by them.  Four at once, for 128 wide heads of one group, gain nothing in long rows (128.9 and 129.5
    // us for the 48 sequences) and lose in short ones (41 positions: 5.5 and 4.4 us); groups of 64 spill with four.
    static constexpr int SUBS = 2;
    static constexpr int STEP = 16 * SUBS;
    static constexpr int UNIT = SPLIT_WARPS * STEP;    // positions per work unit: a step of each warp
    static constexpr int STAGE = SUBS * SUB;
    static constexpr int STAGES = D == 256 ? 2 : 3; // (shared memory for two blocks at least)
    static constexpr int CTAS = D * NT > 64 ? 2 : 3;   // blocks per SM
    static_assert(CTAS <= SPLIT_MAX_CTAS, "a counter per block");
    static constexpr int ROW_COST = 4;                 // of a row by itself, in units
    static constexpr int HEADS = 8 * NT;
    static constexpr int SMEM = SPLIT_WARPS * STAGES * STAGE > SPLIT_WARPS * HEADS * D * 4 ? SPLIT_WARPS * STAGES * STAGE
                                                                                          : SPLIT_WARPS * HEADS * D * 4;
};

__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a)
{
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

// D = A * B + C, apart from D.
__device__ __forceinline__ void mma16816_from(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1, const float (&c)[4])
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

// N bytes from global to shared memory, or N zero bytes when `live` is false.
template <int N>
__device__ __forceinline__ void cp_async(uint32_t dst, const void *src, bool live)
{
    if (N == 16)
        cp_async16(dst, src, live);
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(live ? N : 0)
                     : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}

__device__ __forceinline__ uint2 lds64(uint32_t a)
{
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}

__device__ __forceinline__ uint32_t lds32(uint32_t a)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}

template <int WORDS>
__device__ __forceinline__ void lds_words(uint32_t a, uint32_t *w)
{
    if (WORDS == 1) {
        w[0] = lds32(a);
    } else if (WORDS == 2) {
        const uint2 v = lds64(a);
        w[0] = v.x;
        w[1] = v.y;
    } else {
        const uint4 v = lds128(a);
        w[0] = v.x;
        w[1] = v.y;
        w[2] = v.z;
        w[3] = v.w;
    }
}

// Where the 16-byte chunk `chunk` of value row `row` of a sub-step lies: spread so that the four rows which a load
// of all lanes touches lie in different banks.
template <int D>
__device__ __forceinline__ int value_chunk(int row, int chunk)
{
    return D == 64 ? chunk : D == 128 ? chunk ^ (row & 2) : chunk ^ (2 * (row & 3));
}

// WHOLE: pages hold multiples of 16 positions, so that a sub-step lies in one of them.
template <int D, int G, int NT, bool BF, bool WHOLE>
__global__ void __launch_bounds__(SPLIT_THREADS, Kv4Geom<D, G, NT>::CTAS) kv4_attention_kernel(const Kv4AttParams p)
{
    using M = Kv4Geom<D, G, NT>;
    constexpr int BLOCKS = M::BLOCKS, TILES = 4 * BLOCKS; // 16-wide tiles of the output dims
    constexpr int PER = BLOCKS / G;                       // blocks of 64 per group
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ SplitShared shared;
    __shared__ float stat[SPLIT_WARPS][M::HEADS][2];

    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31; // (warp: the same in all lanes)
    const int g = lane >> 2, t = lane & 3;
    const int row_of = (g >> 1) + 4 * (g & 1); // the position of the eight that is row g of the score product
    pdl_wait();
    pdl_launch_dependents();

    Split<M::UNIT, M::ROW_COST, true> split(p.split, shared);
    // Sequences without a position: zeros and -inf.
    for (int b = blockIdx.x; b < p.split.batch; b += gridDim.x) {
        if (!split.empty(b))
            continue;
        for (int i = tid; i < p.heads * D / 8; i += SPLIT_THREADS)
            *reinterpret_cast<uint4 *>(p.out + (long long)b * p.ldo + 8 * i) = make_uint4(0, 0, 0, 0);
        if (p.lse)
            for (int h = tid; h < p.heads; h += SPLIT_THREADS)
                p.lse[(long long)b * p.heads + h] = -INFINITY;
    }
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * (M::STAGES * M::STAGE);

    SplitSegment seg;
    while (split.next(seg)) {
        const int b = seg.b, c = seg.row / p.tiles, h0 = (seg.row - c * p.tiles) * M::HEADS;
        const int nh = min(M::HEADS, p.group - h0); // heads of this tile
        const int first = seg.first, len = seg.len, steps = seg.unit1 - seg.unit0;
        const int pos0 = seg.start + seg.unit0 * M::UNIT + warp * M::STEP; // this warp's first position

        // --- copies ---------------------------------------------------------------------------
        // A lane looks after positions row_of + 8 i, i < 2 SUBS, of a step.  Pages are looked up one step before they are used:
        // those of the sub-steps, or of each lane's positions.
        constexpr int SUBS = M::SUBS, LOOK = WHOLE ? SUBS : 2 * SUBS;
        const int32_t *tab = p.table + (long long)b * p.ld_table;
        const uint8_t *head = p.cache + c * p.rec.bytes;
        int next_page[LOOK], next_token[LOOK];
        auto look_up = [&](int step) {
#pragma unroll
            for (int i = 0; i < LOOK; ++i) {
                const int pos = pos0 + step * M::UNIT + (WHOLE ? 16 * i : row_of + 8 * i);
                const bool in = step < steps && pos < len && (WHOLE ? pos + 16 > first : pos >= first);
                const int at = p.page_magic ? (int)(__umulhi((uint32_t)pos, p.page_magic) >> p.page_shift) : pos;
                next_page[i] = in ? tab[at] : -1;
                next_token[i] = pos - at * p.page;
            }
        };
        // What is live of the steps in flight, the newest in the lowest bits: this lane's positions, and above them whether
        // all of the step is.
        uint32_t flight = 0;
        auto issue = [&](int step, int stage) {
            flight <<= 2 * SUBS + 1;
            if (step >= steps)
                return;
            const int pos = pos0 + step * M::UNIT;
            const uint32_t st = ring + stage * M::STAGE;
            constexpr int HALVES = D / 128; // 16-byte chunks of a lane in a row
            bool fine = WHOLE && pos >= first && pos + M::STEP <= len;
#pragma unroll
            for (int u = 0; u < (WHOLE ? SUBS : 0); ++u)
                fine = fine && (uint32_t)next_page[u] < (uint32_t)p.n_pages;
            if (fine) {
                flight |= (2u << 2 * SUBS) - 1;
#pragma unroll
                for (int u = 0; u < SUBS; ++u) {
                    const uint8_t *rec = head + (long long)next_page[u % LOOK] * p.page_stride;
                    const int token = next_token[u % LOOK] + row_of;
                    const uint8_t *keys = rec + (long long)token * M::ROW + (D == 64 ? 8 : 16) * t, *values = keys + p.rec.values;
                    const uint32_t sub = st + u * M::SUB;
                    const uint32_t key_to = sub + lane * (D == 64 ? 8 : 16), value_to = sub + M::KEYS + row_of * M::ROW;
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        if (D == 64) {
                            cp_async<8>(key_to + r * 256, keys + r * 8 * M::ROW, true);
                            cp_async<8>(value_to + r * 8 * M::ROW + t * 8, values + r * 8 * M::ROW, true);
                        } else {
#pragma unroll
                            for (int h = 0; h < HALVES; ++h) {
                                cp_async<16>(key_to + (r * HALVES + h) * 512, keys + r * 8 * M::ROW + h * 64, true);
                                cp_async<16>(value_to + r * 8 * M::ROW + value_chunk<D>(row_of, t + 4 * h) * 16,
                                             values + r * 8 * M::ROW + h * 64, true);
                            }
                        }
                    }
                    // Steps and bases: a lane copies those of one of its two positions of a sub-step, of one side.
                    const int row = token + 8 * (t & 1);
                    cp_async<4 * G>(sub + 2 * M::KEYS + (t >> 1) * M::PARAMS + (row_of + 8 * (t & 1)) * (4 * G),
                                    rec + (t >> 1 ? p.rec.value_params : p.rec.key_params) + (long long)row * (4 * G), true);
                }
                return;
            }
            const uint8_t *rec[2 * SUBS];
            uint32_t bits = 0;
            int token[2 * SUBS];
#pragma unroll
            for (int i = 0; i < 2 * SUBS; ++i) {
                const int at = pos + row_of + 8 * i, page = next_page[WHOLE ? i / 2 : i];
                const bool in = at >= first && at < len, ok = in && page >= 0 && page < p.n_pages;
                if (in && !ok)
                    atomicOr(p.split.status, W4A16_DEV_PAGE);
                rec[i] = head + (ok ? (long long)page * p.page_stride : 0);
                token[i] = ok ? next_token[WHOLE ? i / 2 : i] + (WHOLE ? row_of + 8 * (i & 1) : 0) : 0;
                bits |= (ok ? 1u : 0u) << i;
            }
            flight |= bits;
#pragma unroll
            for (int i = 0; i < 2 * SUBS; ++i) {
                const int r = i & 1, row = row_of + 8 * r;
                const uint32_t sub = st + (i >> 1) * M::SUB;
                const bool ok = (bits >> i) & 1u;
                const uint8_t *keys = rec[i] + (long long)token[i] * M::ROW, *values = keys + p.rec.values;
                if (D == 64) {
                    cp_async<8>(sub + r * 256 + lane * 8, keys + t * 8, ok);
                    cp_async<8>(sub + M::KEYS + row * M::ROW + t * 8, values + t * 8, ok);
                } else {
#pragma unroll
                    for (int h = 0; h < HALVES; ++h) {
                        const int ch = t + 4 * h;
                        cp_async<16>(sub + (r * HALVES + h) * 512 + lane * 16, keys + ch * 16, ok);
                        cp_async<16>(sub + M::KEYS + row * M::ROW + value_chunk<D>(row, ch) * 16, values + ch * 16, ok);
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < SUBS; ++u) {
                const int i = 2 * u + (t & 1);
                const bool ok = (bits >> i) & 1u;
                const uint8_t *src = (t & 1 ? rec[2 * u + 1] : rec[2 * u]) + (t >> 1 ? p.rec.value_params : p.rec.key_params) +
                                     (long long)(t & 1 ? token[2 * u + 1] : token[2 * u]) * (4 * G);
                cp_async<4 * G>(st + u * M::SUB + 2 * M::KEYS + (t >> 1) * M::PARAMS + (row_of + 8 * (t & 1)) * (4 * G), src, ok);
            }
        };

        look_up(0);
        // --- queries: B fragments of the score product ------------------------------------------
        uint32_t qf[NT][BLOCKS][2][4]; // [word of a block]: values 0 4, 2 6; a sixteenth of 1 5, 3 7
        float2 fac[NT], qs[NT][G];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const bool in = nt * 8 + g < nh;
            const uint16_t *qp = p.q + (long long)b * p.ldq + (long long)(c * p.group + h0 + (in ? nt * 8 + g : 0)) * D + 16 * t;
            uint4 raw[BLOCKS][2];
            float top = 0.f, sum[G];
#pragma unroll
            for (int k = 0; k < BLOCKS; ++k) {
                if (k % PER == 0)
                    sum[k / PER] = 0.f;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    raw[k][i] = in ? *reinterpret_cast<const uint4 *>(qp + 64 * k + 8 * i) : make_uint4(0, 0, 0, 0);
                    const uint32_t w[4] = {raw[k][i].x, raw[k][i].y, raw[k][i].z, raw[k][i].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 f = unpack2<BF>(w[e]);
                        top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
                        sum[k / PER] += f.x + f.y;
                    }
                }
            }
#pragma unroll
            for (int d = 1; d < 4; d <<= 1) {
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
#pragma unroll
                for (int e = 0; e < G; ++e)
                    sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], d);
            }
            const int up = min(max(13 - ((int)(__float_as_uint(top) >> 23) - 127), -100), 100);
            const float f0 = __uint_as_float((uint32_t)(up + 127) << 23), f1 = 0.0625f * f0;
#pragma unroll
            for (int k = 0; k < BLOCKS; ++k)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float2 v01 = unpack2<BF>(raw[k][i].x), v23 = unpack2<BF>(raw[k][i].y),
                                 v45 = unpack2<BF>(raw[k][i].z), v67 = unpack2<BF>(raw[k][i].w);
                    qf[nt][k][i][0] = pack2<false>(v01.x * f0, v45.x * f0);
                    qf[nt][k][i][1] = pack2<false>(v23.x * f0, v67.x * f0);
                    qf[nt][k][i][2] = pack2<false>(v01.y * f1, v45.y * f1);
                    qf[nt][k][i][3] = pack2<false>(v23.y * f1, v67.y * f1);
                }
            // This lane's columns are heads 2 t and 2 t + 1: their factor and sums.
            const float mine = p.scale_log2 * __uint_as_float((uint32_t)(24 - up + 127) << 23);
            const auto columns = [&](float v) {
                return make_float2(__shfl_sync(0xffffffffu, v, 8 * t), __shfl_sync(0xffffffffu, v, 8 * t + 4));
            };
            fac[nt] = columns(mine);
#pragma unroll
            for (int q = 0; q < G; ++q)
                qs[nt][q] = columns(p.scale_log2 * sum[q]);
        }
#pragma unroll
        for (int s = 0; s < M::STAGES - 1; ++s) {
            issue(s, s);
            cp_async_commit();
            look_up(s + 1);
        }

        // --- the running softmax ----------------------------------------------------------------
        // Pairs: heads 2 t and 2 t + 1.
        float2 o[NT][TILES][2], m[NT], l[NT], base[NT][G];
        float ref = 0.f, up = 0.f; // the power of two above every value step so far, and KV4_UP over it
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int n = 0; n < TILES; ++n)
                o[nt][n][0] = o[nt][n][1] = both(0.f);
            m[nt] = both(-3.402823466e38f); // not -inf: nothing live yet then gives p = 0
            l[nt] = both(0.f);
#pragma unroll
            for (int q = 0; q < G; ++q)
                base[nt][q] = both(0.f);
        }
        int stage = 0;
        for (int step = 0; step < steps; ++step) {
            cp_async_wait<M::STAGES - 2>();
            __syncwarp(); // every lane's copies of this stage have landed; the next one is free
            const uint32_t live = flight >> ((2 * SUBS + 1) * (M::STAGES - 2));
            {
                int ns = stage + M::STAGES - 1;
                ns = ns >= M::STAGES ? ns - M::STAGES : ns;
                issue(step + M::STAGES - 1, ns);
                cp_async_commit();
                look_up(step + M::STAGES);
            }
            const uint32_t st = ring + stage * M::STAGE;

            // Scores x[sub-step][tile][row] of positions row_of + 16 u (+ 8).
            float2 x[SUBS][NT][2];
            float vs[SUBS][2][G], va[SUBS][2][G];
#pragma unroll
            for (int u = 0; u < SUBS; ++u) {
                const uint32_t sub = st + u * M::SUB;
                uint32_t kw[2][BLOCKS * 2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    if (D == 64) {
                        lds_words<2>(sub + r * 256 + lane * 8, kw[r]);
                    } else {
#pragma unroll
                        for (int h = 0; h < D / 128; ++h)
                            lds_words<4>(sub + (r * (D / 128) + h) * 512 + lane * 16, kw[r] + 4 * h);
                    }
                }
                float ks[2][G], ka[2][G];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    uint32_t w[G];
                    lds_words<G>(sub + 2 * M::KEYS + (row_of + 8 * r) * (4 * G), w);
#pragma unroll
                    for (int q = 0; q < G; ++q) {
                        const float2 f = unpack2<BF>(w[q]);
                        ks[r][q] = f.x;
                        ka[r][q] = f.y;
                    }
                    lds_words<G>(sub + 2 * M::KEYS + M::PARAMS + (row_of + 8 * r) * (4 * G), w);
#pragma unroll
                    for (int q = 0; q < G; ++q) {
                        const float2 f = unpack2<BF>(w[q]);
                        vs[u][r][q] = f.x;
                        va[u][r][q] = fmaf(8.f, f.x, f.y);
                    }
                }
#pragma unroll
                for (int q = 0; q < G; ++q) {
                    float acc[NT][4], acc2[NT][4]; // two chains of sums
#pragma unroll
                    for (int k = 0; k < PER; ++k)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int blk = q * PER + k;
                            const uint32_t w0 = kw[0][2 * blk + i], w1 = kw[1][2 * blk + i], v0 = w0 >> 8, v1 = w1 >> 8;
                            const uint32_t lo = 0x000f000fu, hi = 0x00f000f0u;
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                const uint32_t *f = qf[nt][blk][i];
                                if (k == 0 && i == 0) {
                                    mma16816_zero<false>(acc[nt], w0 & lo, w1 & lo, v0 & lo, v1 & lo, f[0], f[1]);
                                    mma16816_zero<false>(acc2[nt], w0 & hi, w1 & hi, v0 & hi, v1 & hi, f[2], f[3]);
                                } else {
                                    mma16816<false>(acc[nt], w0 & lo, w1 & lo, v0 & lo, v1 & lo, f[0], f[1]);
                                    mma16816<false>(acc2[nt], w0 & hi, w1 & hi, v0 & hi, v1 & hi, f[2], f[3]);
                                }
                            }
                        }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const float2 sum = mul(add(make_float2(acc[nt][2 * r], acc[nt][2 * r + 1]),
                                                       make_float2(acc2[nt][2 * r], acc2[nt][2 * r + 1])),
                                                   both(ks[r][q]));
                            const float2 y = fma(sum, fac[nt], mul(both(ka[r][q]), qs[nt][q]));
                            x[u][nt][r] = q == 0 ? y : add(x[u][nt][r], y);
                        }
                }
            }
            if (!((live >> 2 * SUBS) & 1u)) {
#pragma unroll
                for (int u = 0; u < SUBS; ++u)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int r = 0; r < 2; ++r)
                            if (!((live >> (2 * u + r)) & 1u))
                                x[u][nt][r] = both(-INFINITY);
            }

            // Does a maximum or the reference of the value steps have to move?  (A NaN does not move anything.)
            float step_top = ref;
#pragma unroll
            for (int u = 0; u < SUBS; ++u)
#pragma unroll
                for (int q = 0; q < G; ++q)
                    step_top = fmaxf(step_top, fmaxf(fabsf(vs[u][0][q]), fabsf(vs[u][1][q])));
            bool moves = step_top > ref;
            float2 top[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                top[nt] = both(-INFINITY);
#pragma unroll
                for (int u = 0; u < SUBS; ++u) {
                    top[nt].x = fmaxf(top[nt].x, fmaxf(x[u][nt][0].x, x[u][nt][1].x));
                    top[nt].y = fmaxf(top[nt].y, fmaxf(x[u][nt][0].y, x[u][nt][1].y));
                }
                const float2 over = sub(top[nt], m[nt]);
                moves |= over.x > KV4_LAZY || over.y > KV4_LAZY;
            }
            if (__any_sync(0xffffffffu, moves)) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1)
                    step_top = fmaxf(step_top, __shfl_xor_sync(0xffffffffu, step_top, d));
                float turn = 1.f;
                if (step_top > ref) {
                    // The next power of two (2^-100 at least, whose inverse fp32 holds with room).
                    const float to = fmaxf(__uint_as_float(((__float_as_uint(step_top) >> 23) + 1) << 23), 7.888609052e-31f);
                    turn = ref / to;
                    ref = to;
                    up = KV4_UP / to;
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) {
                        top[nt].x = fmaxf(top[nt].x, __shfl_xor_sync(0xffffffffu, top[nt].x, d));
                        top[nt].y = fmaxf(top[nt].y, __shfl_xor_sync(0xffffffffu, top[nt].y, d));
                    }
                    const float2 to = make_float2(fmaxf(m[nt].x, top[nt].x), fmaxf(m[nt].y, top[nt].y));
                    const float2 f = make_float2(ex2(m[nt].x - to.x), ex2(m[nt].y - to.y)), fo = mul(f, both(turn));
                    m[nt] = to;
                    l[nt] = mul(l[nt], f);
#pragma unroll
                    for (int q = 0; q < G; ++q)
                        base[nt][q] = mul(base[nt][q], f);
#pragma unroll
                    for (int n = 0; n < TILES; ++n) {
                        o[nt][n][0] = mul(o[nt][n][0], fo);
                        o[nt][n][1] = mul(o[nt][n][1], fo);
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < SUBS; ++u)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const float2 y = sub(x[u][nt][r], m[nt]);
                        const float2 pe = make_float2(ex2(y.x), ex2(y.y));
                        x[u][nt][r] = pe;
                        l[nt] = add(l[nt], pe);
#pragma unroll
                        for (int q = 0; q < G; ++q)
                            base[nt][q] = fma(pe, both(va[u][r][q]), base[nt][q]);
                    }

            // The value product, group by group.
            uint32_t vw[SUBS][4][BLOCKS]; // words of positions t, t + 4, t + 8, t + 12 of a sub-step
#pragma unroll
            for (int u = 0; u < SUBS; ++u)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int row = t + 4 * e;
                    const uint32_t a = st + u * M::SUB + M::KEYS + row * M::ROW;
                    if (D == 64)
                        lds_words<1>(a + g * 4, vw[u][e]);
                    else if (D == 128)
                        lds_words<2>(a + value_chunk<D>(row, g >> 1) * 16 + (g & 1) * 8, vw[u][e]);
                    else
                        lds_words<4>(a + value_chunk<D>(row, g) * 16, vw[u][e]);
                }
#pragma unroll
            for (int q = 0; q < G; ++q) {
                // p s in two parts, and -8 sum p s of each, as the codes' rows are scaled.
                uint32_t ps[2][SUBS][NT][2];
                float start[2][NT][4];
#pragma unroll
                for (int u = 0; u < SUBS; ++u)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const float2 a = mul(x[u][nt][r], both(vs[u][r][q] * up));
                            const uint32_t first = pack2<false>(a.x, a.y);
                            const float2 rest = sub(a, unpack2<false>(first));
                            ps[0][u][nt][r] = transpose8x8(first);
                            ps[1][u][nt][r] = transpose8x8(pack2<false>(rest.x, rest.y));
                        }
                        constexpr uint32_t E = 0x80208020u, S = 0x82008200u; // -8 2^-22 and -8 2^-18, twice
#pragma unroll
                        for (int part = 0; part < 2; ++part)
                            if (u == 0)
                                mma16816_zero<false>(start[part][nt], E, S, E, S, ps[part][u][nt][0], ps[part][u][nt][1]);
                            else
                                mma16816<false>(start[part][nt], E, S, E, S, ps[part][u][nt][0], ps[part][u][nt][1]);
                    }
#pragma unroll
                for (int k = 0; k < PER; ++k) {
                    const int blk = q * PER + k;
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t w01[SUBS], w23[SUBS]; // codes 4 half .. 4 half + 3 of two positions each
#pragma unroll
                        for (int u = 0; u < SUBS; ++u) {
                            w01[u] = __byte_perm(vw[u][0][blk], vw[u][1][blk], half ? 0x7632 : 0x5410);
                            w23[u] = __byte_perm(vw[u][2][blk], vw[u][3][blk], half ? 0x7632 : 0x5410);
                        }
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const uint32_t ml = 0x003c003cu, mh = 0x03c003c0u;
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                float d[2][4]; // of either part
#pragma unroll
                                for (int u = 0; u < SUBS; ++u) {
                                    const uint32_t a = j ? w01[u] >> 6 : w01[u] << 2, e = j ? w23[u] >> 6 : w23[u] << 2;
#pragma unroll
                                    for (int part = 0; part < 2; ++part) {
                                        const uint32_t(&w)[2] = ps[part][u][nt];
                                        if (u == 0)
                                            mma16816_from(d[part], a & ml, a & mh, e & ml, e & mh, w[0], w[1], start[part][nt]);
                                        else
                                            mma16816<false>(d[part], a & ml, a & mh, e & ml, e & mh, w[0], w[1]);
                                    }
                                }
                                float2(&acc)[2] = o[nt][4 * blk + 2 * half + j];
#pragma unroll
                                for (int r = 0; r < 2; ++r)
                                    acc[r] = add(acc[r], add(make_float2(d[0][2 * r], d[0][2 * r + 1]),
                                                             make_float2(d[1][2 * r], d[1][2 * r + 1])));
                            }
                        }
                    }
                }
            }
            stage = stage + 1 == M::STAGES ? 0 : stage + 1;
        }
        cp_async_wait<0>();

        // --- the warps' results meet in shared memory (the ring is free) -----------------------
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) {
                const auto lanes = [&](float2 v) {
                    return add(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, d), __shfl_xor_sync(0xffffffffu, v.y, d)));
                };
                l[nt] = lanes(l[nt]);
#pragma unroll
                for (int q = 0; q < G; ++q)
                    base[nt][q] = lanes(base[nt][q]);
            }
        __syncthreads();
        float *acc = reinterpret_cast<float *>(smem); // [warp][head][D]
        constexpr float EVEN = 4194304.f / KV4_UP, ODD = 262144.f / KV4_UP; // (times ref: beyond fp32 where steps are large)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const auto of = [e](float2 v) { return e ? v.y : v.x; };
                float *mine = acc + (warp * M::HEADS + nt * 8 + 2 * t + e) * D + 8 * g;
#pragma unroll
                for (int n = 0; n < TILES; n += 2) { // values 2 n % 8 .. + 3 of block n / 4
                    const float a = of(base[nt][n / 4 / PER]);
                    const float4 v = make_float4(fmaf(of(o[nt][n][0]) * EVEN, ref, a), fmaf(of(o[nt][n][1]) * ODD, ref, a),
                                                 fmaf(of(o[nt][n + 1][0]) * EVEN, ref, a), fmaf(of(o[nt][n + 1][1]) * ODD, ref, a));
                    *reinterpret_cast<float4 *>(mine + 64 * (n / 4) + 2 * (n % 4)) = v;
                }
                if (g == 0) {
                    stat[warp][nt * 8 + 2 * t + e][0] = of(m[nt]);
                    stat[warp][nt * 8 + 2 * t + e][1] = of(l[nt]);
                }
            }
        __syncthreads();
        uint16_t *out = p.out + (long long)b * p.ldo + (long long)(c * p.group + h0) * D;
        float *lse = p.lse ? p.lse + (long long)b * p.heads + c * p.group + h0 : nullptr;
        split.template finish<D, M::HEADS, BF>(seg, acc, &stat[0][0][0], nh, out, lse);
    }
}

namespace {

using Kv4Kernel = void (*)(Kv4AttParams);

template <int D, int G, int NT>
cudaError_t kv4_kernel(bool bf, bool whole, Kv4Kernel &kernel, int &smem)
{
    static const Kv4Kernel kernels[4] = {kv4_attention_kernel<D, G, NT, false, false>, kv4_attention_kernel<D, G, NT, false, true>,
                                         kv4_attention_kernel<D, G, NT, true, false>, kv4_attention_kernel<D, G, NT, true, true>};
    const int v = 2 * bf + whole;
    kernel = kernels[v];
    smem = Kv4Geom<D, G, NT>::SMEM;
    return allow_smem<Kv4Geom<D, G, NT>, 4>(reinterpret_cast<const void *>(kernel), v, smem);
}

// Query heads of a tile, and blocks per SM.
int kv4_heads(int head_dim, int group)
{
    return head_dim < 256 && group > 8 ? 16 : 8;
}

int kv4_ctas(int head_dim, int heads)
{
    return head_dim == 64    ? heads == 8 ? Kv4Geom<64, 1, 1>::CTAS : Kv4Geom<64, 1, 2>::CTAS
           : head_dim == 128 ? heads == 8 ? Kv4Geom<128, 1, 1>::CTAS : Kv4Geom<128, 1, 2>::CTAS
                             : Kv4Geom<256, 1, 1>::CTAS;
}
SplitLayout kv4_layout(int head_dim, int heads, int num_sms)
{
    return split_layout((long long)num_sms * SPLIT_MAX_CTAS, (long long)num_sms * kv4_ctas(head_dim, heads),
                        heads * (head_dim + 2));
}

int kv4_check_sizes(int batch, int n_heads, int n_kv_heads, int head_dim)
{
    if (batch < 0 || n_heads <= 0 || n_kv_heads <= 0 || head_dim <= 0 || n_heads % n_kv_heads != 0)
        return status_of(STAGE_ARG, W4A16_ARG_SHAPE);
    if (!kv4_dim(head_dim) || batch > SPLIT_MAX_BATCH)
        return status_of(STAGE_UNSUPPORTED, W4A16_ARG_SHAPE);
    if ((long long)n_heads * head_dim > 0x3FFFFFFFLL || (long long)batch * n_heads > 0x7FFFFFFFLL)
        return status_of(STAGE_ARG, W4A16_ARG_OVERFLOW);
    return 0;
}

} // namespace
} // namespace ops
} // namespace w4

using namespace w4;
using namespace w4::ops;

extern "C" size_t w4a16_kv4_attention_workspace_size(int batch, int n_heads, int n_kv_heads, int head_dim, int num_sms)
{
    if (kv4_check_sizes(batch, n_heads, n_kv_heads, head_dim) != 0)
        return 0;
    if (num_sms <= 0 && sm_count(&num_sms) != cudaSuccess)
        return 0;
    return (size_t)kv4_layout(head_dim, kv4_heads(head_dim, n_heads / n_kv_heads), num_sms).total;
}

extern "C" int w4a16_kv4_attention(const void *q, int ldq, const void *cache, long long page_stride, void *out, int ldo,
                                   float *lse, const int32_t *block_table, int ld_table, const int32_t *seq_lens,
                                   void *workspace, size_t workspace_bytes, int batch, int n_heads, int n_kv_heads,
                                   int head_dim, int page_size, int n_pages, int max_pages, int group_size, int window,
                                   float scale, unsigned flags, cudaStream_t stream)
{
    if (flags & ~W4A16_FLAG_BF16)
        return status_of(STAGE_ARG, W4A16_ARG_FLAGS);
    int st = kv4_check_sizes(batch, n_heads, n_kv_heads, head_dim);
    if (st)
        return st;
    if (page_size <= 0 || n_pages <= 0 || max_pages <= 0 || window < 0)
        return status_of(STAGE_ARG, W4A16_ARG_SHAPE);
    if (page_size > W4A16_KV4_MAX_PAGE)
        return status_of(STAGE_UNSUPPORTED, W4A16_ARG_SHAPE);
    const int groups = kv4_groups(head_dim, group_size);
    if (groups == 0)
        return status_of(STAGE_ARG, W4A16_ARG_GROUP);
    if (batch == 0)
        return 0;
    if (!q || !cache || !out || !block_table || !seq_lens || !workspace)
        return status_of(STAGE_ARG, W4A16_ARG_NULL);
    Kv4AttParams p;
    p.rec = kv4_record(page_size, head_dim, groups);
    if (ldq < n_heads * head_dim || ldo < n_heads * head_dim || ld_table < max_pages ||
        page_stride < n_kv_heads * p.rec.bytes)
        return status_of(STAGE_ARG, W4A16_ARG_SHAPE);
    if (ldq % 8 != 0 || ldo % 8 != 0 || page_stride % 16 != 0 || !aligned(q, 16) || !aligned(cache, 16) ||
        !aligned(out, 16) || !aligned(lse, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
        !aligned(workspace, 256))
        return status_of(STAGE_ARG, W4A16_ARG_ALIGN);
    // Positions and units are counted in 32 bits (offsets into the cache in 64): a sequence holds
    // at most max_pages pages.
    const long long max_len = (long long)max_pages * page_size;
    constexpr int UNIT = Kv4Geom<64, 1, 1>::UNIT; // the smallest
    if (max_len > 0x7FFFFFFFLL - 64 * UNIT || ((max_len + UNIT - 1) / UNIT + 8) * batch > 0x7FFFFFFFLL)
        return status_of(STAGE_ARG, W4A16_ARG_OVERFLOW);

    int num_sms = 0;
    cudaError_t err = sm_count(&num_sms);
    if (err != cudaSuccess)
        return status_of(STAGE_RESOURCE, err);
    const int group = n_heads / n_kv_heads, heads = kv4_heads(head_dim, group);
    const SplitLayout lay = kv4_layout(head_dim, heads, num_sms);
    if (workspace_bytes < (size_t)lay.total)
        return status_of(STAGE_ARG, W4A16_ARG_WORKSPACE);
    p.q = static_cast<const uint16_t *>(q);
    p.cache = static_cast<const uint8_t *>(cache);
    p.out = static_cast<uint16_t *>(out);
    p.lse = lse;
    p.table = block_table;
    p.page_stride = page_stride;
    p.ldq = ldq;
    p.ldo = ldo;
    p.ld_table = ld_table;
    p.heads = n_heads;
    p.group = group;
    p.tiles = (group + heads - 1) / heads;
    p.page = page_size;
    p.n_pages = n_pages;
    p.scale_log2 = scale * 1.4426950408889634f;
    split_params(p.split, lay, workspace, seq_lens, batch, n_kv_heads * p.tiles, (int)max_len, window);
    // n / page for n < 2^31: with 2^(s - 1) < page <= 2^s, floor(n ceil(2^(31 + s) / page) / 2^(31 + s)).
    int s = 0;
    while ((1 << s) < page_size)
        ++s;
    p.page_magic = page_size == 1 ? 0 : (uint32_t)(((1ULL << (31 + s)) + page_size - 1) / page_size);
    p.page_shift = page_size == 1 ? 0 : s - 1;

    const bool bf = (flags & W4A16_FLAG_BF16) != 0, whole = page_size % 16 == 0;
    Kv4Kernel kernel;
    int smem;
    if (head_dim == 64)
        err = heads == 8 ? kv4_kernel<64, 1, 1>(bf, whole, kernel, smem) : kv4_kernel<64, 1, 2>(bf, whole, kernel, smem);
    else if (head_dim == 128 && heads == 8)
        err = groups == 1 ? kv4_kernel<128, 1, 1>(bf, whole, kernel, smem) : kv4_kernel<128, 2, 1>(bf, whole, kernel, smem);
    else if (head_dim == 128)
        err = groups == 1 ? kv4_kernel<128, 1, 2>(bf, whole, kernel, smem) : kv4_kernel<128, 2, 2>(bf, whole, kernel, smem);
    else
        err = groups == 1   ? kv4_kernel<256, 1, 1>(bf, whole, kernel, smem)
              : groups == 2 ? kv4_kernel<256, 2, 1>(bf, whole, kernel, smem)
                            : kv4_kernel<256, 4, 1>(bf, whole, kernel, smem);
    if (err != cudaSuccess)
        return status_of(STAGE_RESOURCE, err);
    const int grid = num_sms * kv4_ctas(head_dim, heads);
    return launch_status(launch_pdl(kernel, dim3(grid), dim3(SPLIT_THREADS), (size_t)smem, stream, p));
}
