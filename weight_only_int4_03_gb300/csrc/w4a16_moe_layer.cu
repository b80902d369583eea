// w4a16_moe_layer.cu -- a whole expert layer for a few tokens with 4-bit weights.
//
// For token t with input row x_t:
//     l_e = router[e] . x_t,   P = softmax(l),   the top_k experts e_1 .. e_k of largest l (ties: the
//     lowest index), weights w_j = P[e_j] (divided by their sum with W4A16_FLAG_MOE_RENORM),
//     y_t = residual_t + sum_j w_j Wd_{e_j}^T h_j,   h_j = act(Wg_{e_j}^T x_t) * (Wu_{e_j}^T x_t),
// with W = (q - z) s per group of rows.  Four launches, each starting while the one before drains:
//   route    router product, softmax, top-k, and the pairs (token, j) grouped by expert;
//   gate-up  h for every pair;
//   down     the pairs' outputs in fp32;
//   combine  the weighted sum over a token's experts in the order of j, and the residual.
// (Summing in the down launch, by the last team to finish a range of columns, took a fence and an
// atomic per unit and left T x 64 outputs to one team: 73 us against 51 us for 52 tokens on 8
// experts of 5120 x 1024.)
//
// Bound by memory: each chosen expert's codes are read once for all of its tokens.  What would bound
// it otherwise is the conversion of the codes, so the weights go into the MMA (m16n8k16, weights as
// its 16 rows, tokens as its 8 columns) with as few instructions as they allow:
//   fp16   a code in the low bits of an fp16 is the subnormal q 2^-24, and one nibble up 16 q 2^-24;
//          the MMA takes both exactly, so a mask is the whole conversion.  The two kinds go into
//          separate accumulators, joined as lo + hi / 16.
//   bf16   a code or-ed into the fraction of 128.0 is 128 + q.
// The zero point (and the 128) is then taken off the sums, sum (q - z) a = sum q a - z sum a, with
// sum a from one more MMA whose weights are all ones, shared by the block's columns.  Every sum of a
// step (a block, where a group is an odd number of them) starts from zero and is scaled in fp32; (q - z) s is
// never rounded.  In bf16 about five bits of a step's sum cancel with the 128, and the MMA cuts off instead of
// rounding: 2^-15 of a column's root mean square, far below y's 2^-9.
// h goes through the second product as a 16-bit value plus a 16-bit remainder, two columns of the down
// MMA, whose eight columns are mostly empty for a few tokens.  bf16's parts keep 2^-17 of any h (a third
// would take another MMA); fp16's keep 2^-23 of it, or an absolute 2^-25 where that is more.  fp16's parts
// end at 2 x 65504: what a value has beyond that is put down in fp32, its pair is marked beside its weight,
// and the combine launch adds it to the pair's outputs in fp32 (a search through the pair's h, in calls that
// have such values alone; the marks cost the other calls 0.1 us).
//
// A unit of work is 64 columns of one expert over all of K (down: or a part of it), done by a team of 1 to 8 warps that take
// its 128-row steps in turn.  A warp streams its steps through its own ring of cp.async stages, which
// runs on into its next unit, so no block-wide barrier sits between a copy and its use and the ring
// stays full across units.  Activations lie in the MMA's fragment order and come through the same ring, each lane's
// own fragments by its own copies (read from L1/L2 a block ahead they cost a wait per block: one token 46.2
// us against 44.9, 16 tokens 159 us against 155); columns that no token uses are not copied.
//
// Measured, the four launches together: one token, 8 experts of 4096 x 14336, two each, fp16: 44.8 us, 4.1
// TB/s of weights (the copies themselves run at 5.4 to 6.0 TB/s; routing and the first copies take
// 10 us); 16 tokens: 155 us, 4.8 TB/s; 64 tokens, bf16: 369 us, bound by the MMAs and the conversion, which run
// 1.43 (gate-up) and 2.43 times (down) over the codes, as a pass holds 16 and 8 of an expert's pairs;
// 7 tokens on 128 experts of 2048 x 768, eight each, bf16: 37.6 us; one token on 1024 x 1792: 12.8 us of
// latencies.
#include <math.h>

#include <type_traits>

#include "w4a16_ops.cuh"

namespace w4 {
namespace ops {

constexpr int MOE_MAX_TOKENS = 64;
constexpr int MOE_MAX_EXPERTS = 512;
constexpr int MOE_MAX_TOP = 16;
constexpr int MOE_MAX_PAIRS = MOE_MAX_TOKENS * MOE_MAX_TOP;
constexpr int MOE_WARPS = 8; // of a routing block
constexpr int MOE_THREADS = MOE_WARPS * 32;
constexpr int MOE_CHUNK = 4;   // tokens per routing block
// The counters of a workspace lie at its start, each at a place that no size of a call moves: a call of
// other sizes finds zeros where one before it has arrived and left, and draws from its own.
constexpr int MOE_ALL_CHUNKS = MOE_MAX_TOKENS / MOE_CHUNK; // arrivals of a chunk's blocks, then of the chunks
constexpr int MOE_TICKETS = MOE_ALL_CHUNKS + 1;            // units drawn by the two products
constexpr int MOE_COUNTERS = MOE_TICKETS + 2;
constexpr int MOE_ONE_LEVEL = MOE_WARPS; // tokens whose softmax and top-k one block does
// Pairs per expert up to which a down tile holds both parts of four pairs side by side (7 tokens on 128
// experts, 1.2 pairs each: 44.8 us against 46.4 us one after the other; 16 tokens on 8, four each: 175 us
// against 167 us).
constexpr double MOE_SIDE_MEAN = 3.0;
// Bytes of the tables that a product keeps in shared memory, at most.
constexpr int MOE_TABLES_MOST = (MOE_MAX_EXPERTS / 32 + 1) * 512 + MOE_MAX_PAIRS * 4;
constexpr int MOE_ROWS = 128;  // weight rows per step (two 64-row blocks)
constexpr float CODE_UNIT = 5.9604644775390625e-8f; // 2^-24: the fp16 value of the bits 1

// Element of a 64-row block in the order the MMA's lanes read it: lane t of a quad takes, for
// i = 0, 1, the eight values of 16-byte chunk 4 i + t, which are rows 32 (t & 1) + 8 p +
// 4 (t >> 1) + 2 i + {0, 1}, p = 0, 2, 1, 3 -- the rows of word 2 (t >> 1) + i of half t & 1, those of
// one nibble position (p even, p odd) side by side as the MMA wants its register pairs.
__host__ __device__ __forceinline__ int frag_index(int row)
{
    const int h = (row >> 5) & 1, p = (row >> 3) & 3, j = (row >> 1) & 3, e = row & 1;
    const int q = ((p & 1) << 1) | (p >> 1);
    return ((j & 1) * 4 + h + 2 * (j >> 1)) * 8 + 2 * q + e;
}

// Row of a 64-row block at place `at` of that order.
__host__ __device__ __forceinline__ int frag_row(int at)
{
    const int c = at >> 3, q = (at >> 1) & 3, p = ((q & 1) << 1) | (q >> 1);
    return (c & 1) * 32 + p * 8 + ((c >> 1) & 1) * 4 + (c >> 2) * 2 + (at & 1);
}

// Routing tables in the workspace.
struct MoeTables {
    // The active experts in increasing order: (first gate-up unit, first down unit, expert | pairs <<
    // 16, first pair in `sorted`).  From the end of the list to the end of its last 32 entries, at
    // least once: the totals of both kinds of units.
    int4 *experts;
    int chunks;      // 32-entry chunks of the list
    int *sorted;     // [pairs] pair ids t * top_k + j by expert, in increasing order within one
    int *token;      // [pairs] their tokens t
    int *ids;        // [pairs]
    // [pairs] weights, each with a mark's bits beside it: 0, or for a pair with values of h beyond fp16's parts
    // OVER | place in `sorted` << 9 | expert.
    float2 *weights;
};
constexpr int OVER = 1 << 20;
static_assert(MOE_MAX_EXPERTS <= 512 && MOE_MAX_PAIRS <= 1024, "a mark holds an expert and a place");

struct RouteParams {
    const uint16_t *x, *router;
    uint16_t *xf; // [tokens][hidden] in fragment order
    float *logits;
    int *topk_ids;
    float *topk_weights;
    int *counters; // [MOE_COUNTERS]; the tickets are zeroed for the products that follow
    MoeTables tab;
    int ldx, tokens, hidden, experts, top, renorm;
    int up_cols, down_cols; // units per expert and pass
    int up_shift, down_shift; // log2 of the pairs per pass
};

// A score as an unsigned number of the same order; a NaN counts as the lowest, so that top_k distinct
// experts come out whatever x holds.  0 is below every key.
__device__ __forceinline__ uint32_t score_key(float l)
{
    if (l != l)
        return 1u;
    const uint32_t bits = __float_as_uint(l == 0.f ? 0.f : l); // -0 and 0 are equal
    return bits & 0x80000000u ? ~bits : bits | 0x80000000u;    // -inf is 0x007FFFFF
}

__device__ __forceinline__ float key_score(uint32_t key)
{
    return key == 1u ? NAN : __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

// The top_k experts of one token by a warp, PER scores a lane: lane j gets the j-th one and its
// weight.
template <int PER>
__device__ __forceinline__ void choose_experts(const float *scores, int experts, int top_k, int renorm,
                                               int lane, int &at_out, float &w_out)
{
    float l[PER];
    uint32_t key[PER], most = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i)
        l[i] = i * 32 + lane < experts ? __ldcg(scores + i * 32 + lane) : -INFINITY;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        key[i] = i * 32 + lane < experts ? score_key(l[i]) : 0u;
        most = max(most, key[i]);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    const float top = most == 1u ? -INFINITY : key_score(most);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i)
        sum += i * 32 + lane < experts ? expf(l[i] - top) : 0.f;
#pragma unroll
    for (int d = 16; d; d >>= 1)
        sum += __shfl_xor_sync(0xffffffffu, sum, d);
    uint32_t mine = 0;
    at_out = 0;
    for (int j = 0; j < top_k; ++j) {
        uint32_t best = key[0];
        int at = lane;
#pragma unroll
        for (int i = 1; i < PER; ++i)
            if (key[i] > best) {
                best = key[i];
                at = i * 32 + lane;
            }
        most = __reduce_max_sync(0xffffffffu, best);
        at = (int)__reduce_min_sync(0xffffffffu, best == most ? (uint32_t)at : 0xffffffffu);
#pragma unroll
        for (int i = 0; i < PER; ++i)
            key[i] = at == i * 32 + lane ? 0u : key[i];
        if (lane == j) {
            mine = most;
            at_out = at;
        }
    }
    const float w = lane < top_k ? expf(key_score(mine) - top) / sum : 0.f;
    float chosen = w;
#pragma unroll
    for (int d = 16; d; d >>= 1)
        chosen += __shfl_xor_sync(0xffffffffu, chosen, d);
    w_out = renorm ? w / chosen : w;
}

// A block per expert and four tokens; the last of four tokens' blocks (up to MOE_ONE_LEVEL tokens: of
// all) takes their softmax and top-k, the last of those groups the pairs by expert.  Bound by latency, a
// chain of loads, one or two counters and scans: 4 us for one token and 8 experts, 7 us for 7 tokens and 128.  (One block for all experts of a small
// router did without a counter but read its rows one after the other: 61 us a layer instead of 50.)
template <bool BF>
__global__ void __launch_bounds__(MOE_THREADS) moe_layer_route_kernel(const RouteParams p)
{
    __shared__ int is_last;
    __shared__ float partial[MOE_WARPS][MOE_CHUNK];
    __shared__ __align__(16) int ids[MOE_MAX_PAIRS];
    __shared__ int rank[MOE_MAX_PAIRS];
    __shared__ int count[MOE_MAX_EXPERTS], off_of[MOE_MAX_EXPERTS];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_wait();
    pdl_launch_dependents();
    const int t0 = blockIdx.y * MOE_CHUNK, nt = min(MOE_CHUNK, p.tokens - t0);
    const bool one_level = p.tokens <= MOE_ONE_LEVEL;
    {
        // This block's share of the tokens' rows in fragment order.
        const int chunks = p.hidden / 8;
        for (int i = blockIdx.x * MOE_THREADS + tid; i < nt * chunks; i += gridDim.x * MOE_THREADS) {
            const int tt = i / chunks, c = i - tt * chunks;
            const int q = c & 7, t = q & 3, w = q >> 2;
            const uint16_t *src = p.x + (long long)(t0 + tt) * p.ldx + (c >> 3) * 64 + 32 * (t & 1) + 4 * (t >> 1) + 2 * w;
            uint4 v;
            v.x = *reinterpret_cast<const uint32_t *>(src);
            v.y = *reinterpret_cast<const uint32_t *>(src + 16);
            v.z = *reinterpret_cast<const uint32_t *>(src + 8);
            v.w = *reinterpret_cast<const uint32_t *>(src + 24);
            *reinterpret_cast<uint4 *>(p.xf + (long long)(t0 + tt) * p.hidden + c * 8) = v;
        }
    }
    // Scores: a block shares expert blockIdx.x's row; the scores meet in global memory, where the
    // chunk's last block picks them up.
    {
        float acc[MOE_CHUNK] = {0.f, 0.f, 0.f, 0.f};
        const uint16_t *r = p.router + (long long)blockIdx.x * p.hidden;
#pragma unroll 2
        for (int k = tid * 8; k < p.hidden; k += MOE_THREADS * 8) {
            const uint4 wv = *reinterpret_cast<const uint4 *>(r + k);
            const uint32_t ww[4] = {wv.x, wv.y, wv.z, wv.w};
            uint4 xv[MOE_CHUNK];
#pragma unroll
            for (int tt = 0; tt < MOE_CHUNK; ++tt)
                xv[tt] = tt < nt ? *reinterpret_cast<const uint4 *>(p.x + (long long)(t0 + tt) * p.ldx + k)
                                 : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int tt = 0; tt < MOE_CHUNK; ++tt) {
                const uint32_t xx[4] = {xv[tt].x, xv[tt].y, xv[tt].z, xv[tt].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 a = unpack2<BF>(ww[i]), b = unpack2<BF>(xx[i]);
                    acc[tt] = fmaf(a.x, b.x, acc[tt]);
                    acc[tt] = fmaf(a.y, b.y, acc[tt]);
                }
            }
        }
#pragma unroll
        for (int tt = 0; tt < MOE_CHUNK; ++tt) {
            float v = acc[tt];
#pragma unroll
            for (int d = 16; d; d >>= 1)
                v += __shfl_xor_sync(0xffffffffu, v, d);
            if (lane == 0)
                partial[warp][tt] = v;
        }
    }
    __syncthreads();
    if (warp == 0) {
        // The arriving thread's warp is the one that stored: a warp barrier orders it.
        if (lane < nt) {
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < MOE_WARPS; ++w)
                v += partial[w][lane];
            __stcg(p.logits + (long long)(t0 + lane) * p.experts + blockIdx.x, v);
        }
        __syncwarp();
        if (lane == 0) {
            int *counter = p.counters + (one_level ? 0 : blockIdx.y);
            const int last = arrive_counter(counter) == (int)(one_level ? gridDim.x * gridDim.y : gridDim.x) - 1;
            if (last)
                *counter = 0;
            is_last = last;
        }
    }
    __syncthreads();
    if (!is_last)
        return;

    // --- softmax and top-k of this chunk (or of all tokens), a warp per token -----------------
    const int pairs = p.tokens * p.top;
    const int tok = (one_level ? 0 : t0) + warp;
    if (tok < (one_level ? p.tokens : t0 + nt)) {
        int at;
        float w;
        const float *l = p.logits + (long long)tok * p.experts;
        if (p.experts <= 32)
            choose_experts<1>(l, p.experts, p.top, p.renorm, lane, at, w);
        else if (p.experts <= 128)
            choose_experts<4>(l, p.experts, p.top, p.renorm, lane, at, w);
        else
            choose_experts<MOE_MAX_EXPERTS / 32>(l, p.experts, p.top, p.renorm, lane, at, w);
        if (lane < p.top) {
            const int pair = tok * p.top + lane;
            p.tab.weights[pair] = make_float2(w, 0.f);
            if (one_level)
                ids[pair] = at;
            else
                __stcg(p.tab.ids + pair, at);
            if (p.topk_ids)
                p.topk_ids[pair] = at;
            if (p.topk_weights)
                p.topk_weights[pair] = w;
        }
    }
    __syncthreads();
    if (!one_level) {
        if (tid == 0) {
            const int last = arrive_counter(p.counters + MOE_ALL_CHUNKS) == (int)gridDim.y - 1;
            if (last)
                p.counters[MOE_ALL_CHUNKS] = 0;
            is_last = last;
        }
        __syncthreads();
        if (!is_last)
            return;
        for (int i = tid; i < pairs; i += MOE_THREADS)
            ids[i] = __ldcg(p.tab.ids + i);
        __syncthreads();
    }

    // --- pairs by expert ----------------------------------------------------------------------
    if (pairs <= 32) { // by one warp, a pair per lane
        if (warp == 0) {
            const bool in = lane < pairs;
            const int x = in ? ids[lane] : MOE_MAX_EXPERTS;
            const uint32_t same = __match_any_sync(0xffffffffu, x);
            const int n = __popc(same), before = __popc(same & ((1u << lane) - 1u));
            const bool leader = in && before == 0;
            const uint32_t passes = !leader ? 0u : (uint32_t)((n + (1 << p.up_shift) - 1) >> p.up_shift) |
                                                   (uint32_t)((n + (1 << p.down_shift) - 1) >> p.down_shift) << 16;
            int at = 0, order = 0; // pairs and experts before this lane's expert
            uint32_t sum = 0, total = 0;
            for (int j = 0; j < pairs; ++j) {
                const int xj = __shfl_sync(0xffffffffu, x, j);
                const uint32_t pj = __shfl_sync(0xffffffffu, passes, j);
                total += pj;
                if (xj < x) {
                    ++at;
                    order += pj != 0;
                    sum += pj;
                }
            }
            if (leader)
                p.tab.experts[order] = make_int4((int)(sum & 0xFFFF) * p.up_cols, (int)(sum >> 16) * p.down_cols,
                                                 x | n << 16, at);
            for (int i = __popc(__ballot_sync(0xffffffffu, leader)) + lane; i < p.tab.chunks * 32; i += 32)
                p.tab.experts[i] = make_int4((int)(total & 0xFFFF) * p.up_cols, (int)(total >> 16) * p.down_cols, 0, pairs);
            if (in) {
                p.tab.sorted[at + before] = lane;
                p.tab.token[at + before] = lane / p.top;
            }
            if (lane < 2)
                p.counters[MOE_TICKETS + lane] = 0;
        }
        return;
    }
    // More pairs (7 tokens on 60 experts, two each: 25.7 us with this way, one level less and the way
    // above: 24.2 us).  A pair's place among its expert's is the number of equal ids before it.
    for (int x = tid; x < p.experts; x += MOE_THREADS)
        count[x] = 0;
    for (int i = pairs + tid; i < (pairs + 3) / 4 * 4; i += MOE_THREADS)
        ids[i] = -1;
    __syncthreads();
    for (int i = tid; i < pairs; i += MOE_THREADS) {
        const int x = ids[i];
        int before = 0;
#pragma unroll 4
        for (int q = 0; q * 4 < i; ++q) {
            const int4 v = reinterpret_cast<const int4 *>(ids)[q];
            before += (v.x == x && q * 4 < i) + (v.y == x && q * 4 + 1 < i) + (v.z == x && q * 4 + 2 < i) +
                      (v.w == x && q * 4 + 3 < i);
        }
        rank[i] = before;
        atomicAdd(&count[x], 1);
    }
    __syncthreads();
    if (warp == 0) {
        // Running sums in 16-bit halves: active experts and pairs; gate-up and down passes.  None
        // passes 1024.
        uint32_t list = 0, passes = 0;
        for (int base = 0; base < p.experts; base += 32) {
            const int x = base + lane, n = x < p.experts ? count[x] : 0;
            const uint32_t a = n > 0 ? 1u | (uint32_t)n << 16 : 0u;
            const uint32_t b = (uint32_t)((n + (1 << p.up_shift) - 1) >> p.up_shift) |
                               (uint32_t)((n + (1 << p.down_shift) - 1) >> p.down_shift) << 16;
            uint32_t s = a, u = b;
#pragma unroll
            for (int q = 1; q < 32; q <<= 1) {
                const uint32_t s2 = __shfl_up_sync(0xffffffffu, s, q), u2 = __shfl_up_sync(0xffffffffu, u, q);
                if (lane >= q) {
                    s += s2;
                    u += u2;
                }
            }
            const uint32_t s0 = list + s - a, u0 = passes + u - b; // before this expert
            if (n > 0)
                p.tab.experts[s0 & 0xFFFF] = make_int4((int)(u0 & 0xFFFF) * p.up_cols, (int)(u0 >> 16) * p.down_cols,
                                                       x | n << 16, (int)(s0 >> 16));
            if (x < p.experts)
                off_of[x] = (int)(s0 >> 16);
            list += __shfl_sync(0xffffffffu, s, 31);
            passes += __shfl_sync(0xffffffffu, u, 31);
        }
        if (lane < 2)
            p.counters[MOE_TICKETS + lane] = 0;
        for (int i = (int)(list & 0xFFFF) + lane; i < p.tab.chunks * 32; i += 32)
            p.tab.experts[i] = make_int4((int)(passes & 0xFFFF) * p.up_cols, (int)(passes >> 16) * p.down_cols, 0,
                                         (int)(list >> 16));
    }
    __syncthreads();
    for (int i = tid; i < pairs; i += MOE_THREADS) {
        const int at = off_of[ids[i]] + rank[i];
        p.tab.sorted[at] = i;
        p.tab.token[at] = i / p.top;
    }
}

struct MoeGemm {
    const int32_t *w;        // packed tiles of every expert
    const uint16_t *s, *z;   // [E][G][N]; z null: 8
    const uint16_t *act;     // activation rows in fragment order, K values each
    uint16_t *h;             // gate-up: the pairs' h, two rows (value, remainder) per pair
    float *excess;           // gate-up, fp16: [pairs][inter] what h has beyond both, where its remainder is +-65504
    float *part;             // down: [pairs][splits][N] fp32
    int *ticket;             // units drawn beyond each team's first two
    int *status;
    MoeTables tab;
    long long expert_words, expert_groups;
    int k, n, steps;         // steps: 128-row steps of K
    int kblocks;             // 64-row blocks of K
    uint32_t group_magic;    // group of block n: umulhi(n, group_magic), or n when 0
    int per_block;           // groups of an odd number of blocks: scale every block's sums
    int col_units;           // units per expert, pass and split (at least 2)
    uint32_t col_magic;      // n / col_units = umulhi(n, col_magic)
    int splits;              // down: parts of K with units and partial outputs of their own
    int team;                // warps per team
    int pairs;
    int inter, glu;
};

// x, or fp16's largest finite value in its place; and whether an fp16 is that.
__device__ __forceinline__ float within(float x)
{
    return fabsf(x) > 65504.f ? copysignf(65504.f, x) : x;
}

__device__ __forceinline__ bool is_most(uint32_t bits)
{
    return (bits & 0x7FFFu) == 0x7BFFu;
}

// Gated activations as g sigmoid(x): x = g for silu, 2 sqrt(2/pi) (g + 0.044715 g^3) for gelu_tanh
// (1 + tanh t = 2 sigmoid(2 t)).
__device__ __forceinline__ float gate_act(float g, int kind)
{
    float x = g;
    if (kind != 1)
        x = 2.0f * 0.7978845608028654f * (g + 0.044715f * g * g * g);
    return g / (1.0f + expf(-x));
}

// (x & mask) | base in one instruction (the compiler spends two where both are constants).
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t mask, uint32_t base)
{
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(x), "r"(mask), "r"(base));
    return r;
}

__device__ __forceinline__ void team_sync(int team_id, int threads)
{
    if (threads == 32)
        __syncwarp();
    else
        asm volatile("bar.sync %0, %1;" ::"r"(team_id + 1), "r"(threads) : "memory");
}

// What a launch computes: the gated products; the down products with a pair's value and remainder
// in two columns of the MMA (up to four pairs a tile, in one MMA); or with both in one column, one
// after the other (up to eight pairs a tile, in two MMAs on the same weights).
enum MoeMode { GATE_UP = 0, DOWN_SIDE = 1, DOWN_TWICE = 2 };

__host__ __device__ constexpr int pairs_per_pass(int nt, int mode)
{
    return (mode == DOWN_SIDE ? 4 : 8) * nt;
}

// One unit of a team: an expert, a pass over its pairs, a range of columns and of 128-row steps.
struct Unit {
    int expert, col, first, cols; // first pair (in `sorted`), pairs of this pass
    int split, step0, step1;
};

// Unit u (the same in every lane): its expert is the last of the list whose first unit is at or
// before u, looked up by the warp's lanes together.
template <int NT, int MODE>
__device__ __forceinline__ Unit find_unit(const MoeGemm &p, const int4 *list, int u, int lane)
{
    int start = 0, id = 0, off = 0;
    for (int c = 0; c < p.tab.chunks; ++c) {
        const int4 e = list[c * 32 + lane];
        const int first = MODE != GATE_UP ? e.y : e.x;
        const uint32_t before = __ballot_sync(0xffffffffu, first <= u);
        if (before == 0)
            break;
        const int src = 31 - __clz(before);
        start = __shfl_sync(0xffffffffu, first, src);
        id = __shfl_sync(0xffffffffu, e.z, src);
        off = __shfl_sync(0xffffffffu, e.w, src);
        if (before != 0xffffffffu)
            break;
    }
    constexpr int PASS = pairs_per_pass(NT, MODE);
    const int local = u - start, part = (int)__umulhi((uint32_t)local, p.col_magic);
    Unit r;
    r.expert = id & 0xFFFF;
    r.col = local - part * p.col_units;
    int pass = part;
    r.split = 0;
    r.step0 = 0;
    r.step1 = p.steps;
    if (MODE != GATE_UP && p.splits > 1) {
        pass = part / p.splits;
        r.split = part - pass * p.splits;
        r.step0 = r.split * p.steps / p.splits;
        r.step1 = (r.split + 1) * p.steps / p.splits;
    }
    r.first = off + pass * PASS;
    r.cols = min(PASS, (id >> 16) - pass * PASS);
    return r;
}

// Sizes of a kernel variant.  NT: 8-column tiles of the MMA's token side; MT: 16-column tiles of
// weights (each activation fragment serves MT products).  A stage is one 64-row block.
template <int NT>
struct MoeGeom {
    static constexpr int MT = 4;
    static constexpr int WARPS = NT == 1 ? 8 : 4;
    static constexpr int CTAS = NT == 1 ? 2 : 3; // blocks per SM
    static constexpr int COLS = 16 * MT;
    static constexpr int SZ = COLS * 2;        // bytes of one scale (or zero) row
    static constexpr int WEIGHTS = 2048 + 2 * SZ; // codes, scales, zeros
    static constexpr int ACT = 1024;              // a tile's activations of a block (one part of them)
    static constexpr int STAGES = 3; // two in flight: at most one step, so at most into the next unit
    static constexpr int stage(int mode) { return WEIGHTS + ACT * (mode == DOWN_TWICE ? 2 : NT); }
    static constexpr int smem(int mode) { return WARPS * STAGES * stage(mode); }
};

template <int NT, bool BF, int MODE>
__global__ void __launch_bounds__(MoeGeom<NT>::WARPS * 32, MoeGeom<NT>::CTAS) moe_layer_gemm_kernel(const MoeGemm p)
{
    using G = MoeGeom<NT>;
    constexpr bool DOWN = MODE != GATE_UP;
    constexpr int PARTS = MODE == DOWN_TWICE ? 2 : 1; // activation rows per column
    constexpr int MT = G::MT, COLS = G::COLS, STAGES = G::STAGES;
    constexpr int STAGE = G::stage(MODE), RING = STAGES * STAGE;
    // fp16 with one token tile: the two nibble positions keep accumulators of their own, which saves
    // two shifts a word; with two tiles the registers go to the tiles.
    constexpr bool DUAL = !BF && NT == 1;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int drawn[G::WARPS][2];
    __shared__ int spot[G::WARPS]; // where a warp's sums of the unit lie, in floats
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;
    const int teams = G::WARPS / p.team, team = warp / p.team, member = warp - team * p.team;
    const int team_threads = p.team * 32, team_tid = member * 32 + lane;
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * RING;
    const uint8_t *ring_p = smem + warp * RING;
    // Down: the routing tables are those of the launch before the previous one, which had waited for
    // everything older and was complete before the previous one read them; so the first copies of the
    // weights, which only they decide, go out while the gate-up launch drains.  The tables are read
    // past L1, which may hold lines of an earlier call.
    if (!DOWN) {
        pdl_wait();
        pdl_launch_dependents();
    }
    // The list of experts and the tokens of the pairs go to shared memory at once: a look-up in L2 for
    // each unit, and another for its tokens, would hold up the first products by a microsecond (one
    // token on 8 experts of 1024 x 1792: 13.9 us without this, 13.2 us with it).
    int4 *list = reinterpret_cast<int4 *>(smem + G::smem(MODE));
    int *token = reinterpret_cast<int *>(list + p.tab.chunks * 32);
    for (int i = tid; i < p.tab.chunks * 32; i += G::WARPS * 32)
        list[i] = __ldcg(p.tab.experts + i);
    if (!DOWN)
        for (int i = tid; i < p.pairs; i += G::WARPS * 32)
            token[i] = __ldcg(p.tab.token + i);
    __syncthreads();
    const int4 total = list[p.tab.chunks * 32 - 1];
    const int units = DOWN ? total.y : total.x;
    // Consecutive units go to different blocks, so that a part round still reaches every SM.
    const int stride = gridDim.x * teams;
    const int u0 = team * gridDim.x + blockIdx.x;
    if (u0 >= units) {
        // The whole team leaves; the other teams of the block have barriers of their own.
        if (DOWN)
            pdl_wait();
        return;
    }

    // --- the copying side: (unit, block) runs ahead of the computing side ----------------------
    // A member takes the 128-row steps member, member + team, ..., two stages each.
    int iu = u0, ik = -1, ib = 0, ib_end = 0;
    const int32_t *i_w = nullptr; // this lane's piece of block 0, half 0 of the unit's columns
    const uint16_t *i_s = nullptr; // lanes 0-7: chunk `lane` of the expert's scale row 0; 8-15: zeros
    // This lane's chunk of its activation row's block 0 in each tile.  Columns past the last are not copied:
    // what the stage holds there goes into sums that nobody reads.
    const uint16_t *i_a[NT];
    int i_rows = 0; // columns in use on the token side
    const bool sz_zero = lane >= 8;
    const bool sz_mine = lane < (p.z ? 16 : 8);
    // The team's k-th unit: the first two follow from its number, the others are drawn from a common
    // counter two units ahead, so that teams that got on faster do more.
    const bool more = units > 2 * stride;
    if (more && p.team * p.splits > p.steps) {
        // A member without a step would run ahead of the drawn units; the plan never comes to this.
        if (team_tid == 0)
            atomicOr(p.status, W4A16_DEV_SCHEDULE);
        if (DOWN)
            pdl_wait();
        return;
    }
    auto unit_at = [&](int k) { return k == 0 ? u0 : k == 1 ? u0 + stride : more ? drawn[team][k & 1] : units; };
    auto enter = [&]() {
        Unit un;
        do { // a member may lack a step only where no unit is drawn (the plan sees to that)
            iu = unit_at(++ik);
            if (iu >= units)
                return;
            un = find_unit<NT, MODE>(p, list, iu, lane);
            ib = 2 * (un.step0 + member);
            ib_end = 2 * un.step1;
        } while (ib >= ib_end);
        const int n0 = un.col * COLS;
        i_w = p.w + un.expert * p.expert_words + (long long)(n0 >> 7) * p.kblocks * 1024 + (n0 & 127) * 4 + lane * 4;
        i_s = (sz_zero ? p.z : p.s) + un.expert * p.expert_groups * p.n + n0 + (lane & 7) * 8;
        i_rows = MODE == DOWN_SIDE ? 2 * un.cols : un.cols;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int c = min(n * 8 + g, i_rows - 1);
            const int row = MODE == GATE_UP     ? token[un.first + c]
                            : MODE == DOWN_SIDE ? 2 * un.first + c
                                                : 2 * (un.first + c);
            i_a[n] = p.act + (long long)row * p.k + t * 8;
        }
    };
    // The columns of a half 1 are stored with bit 2 flipped, so that the fragment reads below fall on
    // different banks.
    const uint32_t dst0 = ring + lane * 16, dst1 = ring + (lane ^ 4) * 16;
    auto copy_weights = [&](int stage) {
        const int32_t *w = i_w + (long long)ib * 1024;
        const uint32_t d0 = dst0 + stage * STAGE, d1 = dst1 + stage * STAGE;
        cp_async16_at<0, 0>(d0, w); // 64 columns of half 0, then of half 1
        cp_async16_at<512, 512>(d0, w);
        cp_async16_at<1024, 2048>(d1, w);
        cp_async16_at<1536, 2560>(d1, w);
        if (sz_mine) {
            const int grp = p.group_magic ? (int)__umulhi((uint32_t)ib, p.group_magic) : ib;
            cp_async16_at<2048, 0>(d0, i_s + (long long)grp * p.n);
        }
    };
    // The lane's own fragments: chunks t and 4 + t of its rows.
    auto copy_activations = [&](int stage, int block) {
        const uint32_t d = dst0 + stage * STAGE + G::WEIGHTS;
        const uint16_t *a = i_a[0] + block * 64;
        if (g < i_rows) {
            cp_async16_at<0, 0>(d, a);
            cp_async16_at<512, 64>(d, a);
            if (MODE == DOWN_TWICE) { // the remainder's row follows the value's
                cp_async16_at<G::ACT, 0>(d, a + p.k);
                cp_async16_at<G::ACT + 512, 64>(d, a + p.k);
            }
        }
        if (NT == 2 && 8 + g < i_rows) {
            a = i_a[NT - 1] + block * 64;
            cp_async16_at<G::ACT, 0>(d, a);
            cp_async16_at<G::ACT + 512, 64>(d, a);
        }
    };
    auto advance = [&]() {
        ++ib;
        if (!(ib & 1))
            ib += 2 * (p.team - 1);
    };
    auto issue = [&](int stage) {
        if (iu < units && ib >= ib_end)
            enter();
        if (iu < units) {
            copy_weights(stage);
            copy_activations(stage, ib);
            advance();
        }
        cp_async_commit();
    };
    // The first step, two stages: its weights, and once they are there its activations.
    static_assert(STAGES == 3, "the copies ahead are one step's");
    enter();
    {
        const int block = ib;
        const bool any = iu < units;
        if (any) {
            copy_weights(0);
            advance();
            copy_weights(1);
            advance();
        }
        if (DOWN) {
            pdl_wait();
            pdl_launch_dependents();
        }
        if (any)
            copy_activations(0, block);
        cp_async_commit();
        if (any)
            copy_activations(1, block + 1);
        cp_async_commit();
    }

    uint32_t nibble = 0x000F000Fu, base128 = 0x43004300u; // in registers, not known to the compiler
    asm volatile("" : "+r"(nibble), "+r"(base128));
    // Half t & 1, column g (bit 2 flipped in half 1), words 2 (t >> 1) and the next.
    const int w_lane = (t & 1) * (COLS * 16) + (g ^ ((t & 1) << 2)) * 16 + (t >> 1) * 8;
    int stage = 0;
    for (int k = 0;; ++k) {
        const int u = unit_at(k);
        if (u >= units)
            break;
        int ticket = 0;
        if (team_tid == 0)
            ticket = more ? atomicAdd(p.ticket, 1) : 0;
        const Unit un = find_unit<NT, MODE>(p, list, u, lane);
        const int rows = MODE == DOWN_SIDE ? 2 * un.cols : un.cols; // columns in use on the token side
        float out[MT][NT][4];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    out[m][n][i] = 0.f;

        // The member's steps for ND token tiles.
        auto sweep = [&](auto nd) {
            constexpr int ND = decltype(nd)::value;
            const int first = un.step0 + member;
            for (int step = first; step < un.step1; step += p.team) {
                float lo[MT][ND][4], hi[DUAL ? MT : 1][ND][4], sa[ND][4];
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    cp_async_wait<STAGES - 2>();
                    __syncwarp(); // every lane's copies have landed, and the stage before is free
                    issue(stage == 0 ? STAGES - 1 : stage - 1);
                    const uint8_t *st = ring_p + stage * STAGE;
                    stage = stage + 1 == STAGES ? 0 : stage + 1;
                    uint2 w[MT][2]; // column g, g + 8 of each tile: words 2 (t >> 1), + 1 of half t & 1
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            w[m][c] = *reinterpret_cast<const uint2 *>(st + w_lane + (m * 16 + c * 8) * 16);
                    constexpr uint32_t ONES = BF ? 0x3F803F80u : 0x3C003C00u;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint4 bv[PARTS][ND];
#pragma unroll
                        for (int r = 0; r < PARTS; ++r)
#pragma unroll
                            for (int n = 0; n < ND; ++n)
                                bv[r][n] = *reinterpret_cast<const uint4 *>(st + G::WEIGHTS + (r + n) * G::ACT + i * 512 + lane * 16);
#pragma unroll
                        for (int r = 0; r < PARTS; ++r)
#pragma unroll
                            for (int n = 0; n < ND; ++n) {
                                if (b == 0 && i == 0 && r == 0)
                                    mma16816_zero<BF>(sa[n], ONES, ONES, ONES, ONES, bv[r][n].x, bv[r][n].y);
                                else
                                    mma16816<BF>(sa[n], ONES, ONES, ONES, ONES, bv[r][n].x, bv[r][n].y);
                            }
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            const uint32_t x = i ? w[m][0].y : w[m][0].x, y = i ? w[m][1].y : w[m][1].x;
                            constexpr uint32_t L = 0x000F000Fu, H = 0x00F000F0u;
                            uint32_t a0, a1, a2, a3, c0, c1, c2, c3;
                            if (BF) {
                                a0 = and_or(x, nibble, base128);
                                a1 = and_or(y, nibble, base128);
                                a2 = and_or(x >> 8, nibble, base128);
                                a3 = and_or(y >> 8, nibble, base128);
                                c0 = and_or(x >> 4, nibble, base128);
                                c1 = and_or(y >> 4, nibble, base128);
                                c2 = and_or(x >> 12, nibble, base128);
                                c3 = and_or(y >> 12, nibble, base128);
                            } else {
                                const uint32_t x8 = x >> 8, y8 = y >> 8;
                                a0 = x & L;
                                a1 = y & L;
                                a2 = x8 & L;
                                a3 = y8 & L;
                                if (DUAL) {
                                    c0 = x & H;
                                    c1 = y & H;
                                    c2 = x8 & H;
                                    c3 = y8 & H;
                                } else {
                                    c0 = (x >> 4) & L;
                                    c1 = (y >> 4) & L;
                                    c2 = (x >> 12) & L;
                                    c3 = (y >> 12) & L;
                                }
                            }
                            // MMAs on one accumulator are kept apart: each waits for the one before.
#pragma unroll
                            for (int r = 0; r < PARTS; ++r) {
#pragma unroll
                                for (int n = 0; n < ND; ++n) {
                                    const uint4 v = bv[r][n];
                                    if (b == 0 && i == 0 && r == 0)
                                        mma16816_zero<BF>(lo[m][n], a0, a1, a2, a3, v.x, v.y);
                                    else
                                        mma16816<BF>(lo[m][n], a0, a1, a2, a3, v.x, v.y);
                                }
#pragma unroll
                                for (int n = 0; n < ND; ++n) {
                                    const uint4 v = bv[r][n];
                                    if (!DUAL)
                                        mma16816<BF>(lo[m][n], c0, c1, c2, c3, v.z, v.w);
                                    else if (b == 0 && i == 0 && r == 0)
                                        mma16816_zero<BF>(hi[m % (DUAL ? MT : 1)][n], c0, c1, c2, c3, v.z, v.w);
                                    else
                                        mma16816<BF>(hi[m % (DUAL ? MT : 1)][n], c0, c1, c2, c3, v.z, v.w);
                                }
                            }
                        }
#pragma unroll
                        for (int r = 0; r < PARTS; ++r)
#pragma unroll
                            for (int n = 0; n < ND; ++n)
                                mma16816<BF>(sa[n], ONES, ONES, ONES, ONES, bv[r][n].z, bv[r][n].w);
                    }
                    // End of a group (or of a step, whose two blocks then share one): scale the sums.
                    const uint8_t *sz = st + 2048;
                    auto flush = [&](auto zeros, bool again) {
#pragma unroll
                        for (int m = 0; m < MT; ++m)
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                const int col = m * 16 + c * 8 + g;
                                const float sc = to_float<BF>(*reinterpret_cast<const uint16_t *>(sz + col * 2));
                                float z = 8.f;
                                if (decltype(zeros)::value)
                                    z = to_float<BF>(*reinterpret_cast<const uint16_t *>(sz + G::SZ + col * 2));
                                z = BF ? z + 128.f : z * CODE_UNIT;
#pragma unroll
                                for (int n = 0; n < ND; ++n)
#pragma unroll
                                    for (int e = 0; e < 2; ++e) {
                                        const int i = 2 * c + e;
                                        float q = lo[m][n][i];
                                        if (DUAL)
                                            q = fmaf(hi[m % (DUAL ? MT : 1)][n][i], 0.0625f, q);
                                        q = fmaf(-z, sa[n][e], q);
                                        out[m][n][i] = fmaf(sc, q, out[m][n][i]);
                                        if (again) {
                                            lo[m][n][i] = 0.f;
                                            if (DUAL)
                                                hi[m % (DUAL ? MT : 1)][n][i] = 0.f;
                                        }
                                    }
                            }
                        if (again) {
#pragma unroll
                            for (int n = 0; n < ND; ++n)
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    sa[n][i] = 0.f;
                        }
                    };
                    if (b == 1 || p.per_block) {
                        if (p.z)
                            flush(std::true_type(), b == 0);
                        else
                            flush(std::false_type(), b == 0);
                    }
                }
            }
        };
        if (NT == 1 || rows <= 8)
            sweep(std::integral_constant<int, 1>());
        else
            sweep(std::integral_constant<int, NT>());

        // --- the team's warps join their sums (fixed order), in their free stages ---------------
        const int free_stage = stage == 0 ? STAGES - 1 : stage - 1;
        float *red = reinterpret_cast<float *>(smem + warp * RING + free_stage * STAGE); // [sum][lane]
        static_assert(MT * NT * (MODE == DOWN_SIDE ? 2 : 4) * 128 <= STAGE, "the sums fit a stage");
        __syncwarp(); // every lane has read the stage
        if (lane == 0)
            spot[warp] = (warp * RING + free_stage * STAGE) / 4;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if (MODE == DOWN_SIDE) { // columns 2 t and 2 t + 1 are a pair's value and remainder
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        red[((m * NT + n) * 2 + c) * 32 + lane] = out[m][n][2 * c] + out[m][n][2 * c + 1];
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        red[((m * NT + n) * 4 + i) * 32 + lane] = out[m][n][i];
                }
            }
        team_sync(team, team_threads);
        if (team_tid == 0)
            drawn[team][k & 1] = 2 * stride + ticket; // unit k + 2, known to the team after the next barrier
        const float *sums = reinterpret_cast<const float *>(smem);
        auto joined = [&](int v, int ln) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < G::WARPS; ++w)
                if (w < p.team)
                    s += sums[spot[team * p.team + w] + v * 32 + ln];
            return BF ? s : s * (1.f / CODE_UNIT);
        };
        if (!DOWN) {
            // Item: feature f of the unit's COLS / 2, pair pr.  Its gate sum is column f % 8 (+ 8) of
            // tile 2 (f / 16), its up sum of the next tile.
            for (int x = team_tid; x < un.cols * (COLS / 2); x += team_threads) {
                const int f = x % (COLS / 2), pr = x / (COLS / 2);
                const int ln = (f & 7) * 4 + ((pr >> 1) & 3), v = ((f >> 4) * 2 * NT + (pr >> 3)) * 4 + ((f >> 3) & 1) * 2 + (pr & 1);
                const float gate = joined(v, ln), up = joined(v + NT * 4, ln);
                const float hv = gate_act(gate, p.glu) * up;
                // fp16: the value part stops at the largest finite value and the remainder goes on
                // from there, as far again (a NaN stays one).
                const uint16_t hb = from_float<BF>(BF ? hv : within(hv));
                const float rest = hv - to_float<BF>(hb);
                const uint16_t lb = from_float<BF>(BF ? rest : within(rest));
                const int row = un.col * (COLS / 2) + f, place = un.first + pr;
                uint16_t *dst = p.h + (long long)(2 * place) * p.inter + (row & ~63) + frag_index(row & 63);
                dst[0] = hb;
                dst[p.inter] = lb;
                if (!BF && is_most(lb)) {
                    p.excess[(long long)place * p.inter + row] = rest - to_float<BF>(lb);
                    p.tab.weights[__ldcg(p.tab.sorted + place)].y = __int_as_float(OVER | place << 9 | un.expert);
                }
            }
        } else {
            // Item: column c of the unit, pair pr.
            for (int x = team_tid; x < un.cols * COLS; x += team_threads) {
                const int c = x % COLS, pr = x / COLS;
                const int half = (c >> 3) & 1;
                const int ln = (c & 7) * 4 + (MODE == DOWN_SIDE ? pr & 3 : (pr >> 1) & 3);
                const int v = MODE == DOWN_SIDE ? ((c >> 4) * NT + (pr >> 2)) * 2 + half
                                                : ((c >> 4) * NT + (pr >> 3)) * 4 + half * 2 + (pr & 1);
                const int pair = p.tab.sorted[un.first + pr];
                __stcg(p.part + ((long long)pair * p.splits + un.split) * p.n + un.col * COLS + c, joined(v, ln));
            }
        }
        team_sync(team, team_threads); // the stages are free
    }
    cp_async_wait<0>();
}

struct CombineParams {
    const float *part; // [pairs][splits][hidden]
    const float2 *weights;
    const uint16_t *residual;
    uint16_t *y;
    int tokens, top, splits, hidden, ldy, ldr;
    // The down product's operands, for values of h beyond fp16's parts.
    const uint16_t *h;
    const float *excess;
    const int32_t *w;
    const uint16_t *s, *z;
    long long expert_words, expert_groups;
    int k, group_rows;
};

// The outputs of columns col to col + 3 that the values of a marked pair's h beyond both their parts have:
// sum over such rows of excess (q - z) s, in the order of h's places.
__device__ __forceinline__ float4 excess_outputs(const CombineParams &p, int mark, int col)
{
    const int expert = mark & 511, place = (mark >> 9) & 1023;
    const uint4 *rest = reinterpret_cast<const uint4 *>(p.h + (2LL * place + 1) * p.k);
    const float *excess = p.excess + (long long)place * p.k;
    const int32_t *tiles = p.w + expert * p.expert_words + (long long)(col >> 7) * (p.k / 64) * 1024 + (col & 127) * 4;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    for (int c = 0; c < p.k / 8; ++c) {
        const uint4 v = __ldcg(rest + c);
        const uint32_t parts[4] = {v.x, v.y, v.z, v.w};
        for (int i = 0; i < 8; ++i) {
            if (!is_most(parts[i >> 1] >> (16 * (i & 1))))
                continue;
            const int r = frag_row((c & 7) * 8 + i), row = (c >> 3) * 64 + r;
            const float x = __ldcg(excess + row);
            const int32_t *words = tiles + (c >> 3) * 1024 + (r >> 5) * 512 + ((r >> 1) & 3);
            const int shift = 4 * ((r >> 3) & 3) + 16 * (r & 1);
            const long long at = (expert * p.expert_groups + row / p.group_rows) * p.hidden + col;
            for (int j = 0; j < 4; ++j) {
                const float q = (float)((words[4 * j] >> shift) & 15), z = p.z ? to_float<false>(p.z[at + j]) : 8.f;
                sum[j] = fmaf(x, (q - z) * to_float<false>(p.s[at + j]), sum[j]);
            }
        }
    }
    return make_float4(sum[0], sum[1], sum[2], sum[3]);
}

// y_t = residual_t + sum_j w_j (sum over the splits), in the order of j: a thread per quad of
// columns of a token.  The residual is older than the layer's first launch, so it is fetched (past
// L1, which may hold a line of an earlier call) before the down product is waited for.
template <bool BF>
__global__ void __launch_bounds__(128) moe_layer_combine_kernel(const CombineParams p)
{
    const int col = (blockIdx.x * 128 + threadIdx.x) * 4, tok = blockIdx.y;
    const bool in = col < p.hidden;
    uint2 rv = make_uint2(0, 0);
    if (in && p.residual)
        rv = __ldcg(reinterpret_cast<const uint2 *>(p.residual + (long long)tok * p.ldr + col));
    pdl_wait();
    pdl_launch_dependents();
    if (!in)
        return;
    const float4 *src = reinterpret_cast<const float4 *>(p.part + (long long)tok * p.top * p.splits * p.hidden + col);
    const float2 *wts = p.weights + tok * p.top;
    const int parts = p.top * p.splits;
    int marked = 0;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int q0 = 0; q0 < parts; q0 += 8) {
        float4 v[8];
        float2 wt[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const bool live = q0 + q < parts;
            v[q] = live ? __ldcg(src + (long long)(q0 + q) * (p.hidden / 4)) : make_float4(0.f, 0.f, 0.f, 0.f);
            wt[q] = live ? __ldcg(wts + (p.splits == 1 ? q0 + q : (q0 + q) / p.splits)) : make_float2(0.f, 0.f);
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            a.x = fmaf(wt[q].x, v[q].x, a.x);
            a.y = fmaf(wt[q].x, v[q].y, a.y);
            a.z = fmaf(wt[q].x, v[q].z, a.z);
            a.w = fmaf(wt[q].x, v[q].w, a.w);
            marked |= __float_as_int(wt[q].y);
        }
    }
    if (!BF && marked) {
        for (int j = 0; j < p.top; ++j) {
            const float2 wt = __ldcg(wts + j);
            if (__float_as_int(wt.y) == 0)
                continue;
            const float4 e = excess_outputs(p, __float_as_int(wt.y), col);
            a.x = fmaf(wt.x, e.x, a.x);
            a.y = fmaf(wt.x, e.y, a.y);
            a.z = fmaf(wt.x, e.z, a.z);
            a.w = fmaf(wt.x, e.w, a.w);
        }
    }
    const float2 r0 = unpack2<BF>(rv.x), r1 = unpack2<BF>(rv.y);
    uint2 o;
    o.x = pack2<BF>(a.x + r0.x, a.y + r0.y);
    o.y = pack2<BF>(a.z + r1.x, a.w + r1.y);
    *reinterpret_cast<uint2 *>(p.y + (long long)tok * p.ldy + col) = o;
}

namespace {

struct MoeLayout {
    long long counters, logits, tables, xf, h, part, excess, total;
    MoeTables tab;
};

// Parts of K that the partial outputs have room for.
int max_splits(int pairs)
{
    return pairs >= 128 ? 1 : pairs >= 64 ? 2 : pairs >= 32 ? 4 : 8;
}

// Rows of partial outputs that a workspace has room for: what these pairs need in as many parts, and
// what any fewer pairs need, so that a workspace for the most tokens serves fewer.
long long part_rows(int pairs)
{
    return pairs < 32 ? 8LL * pairs : pairs < 256 ? 256 : pairs;
}

MoeLayout moe_layout(char *ws, int tokens, int hidden, int inter, int experts, int top)
{
    MoeLayout l;
    const int pairs = tokens * top;
    l.counters = HEADER_BYTES;
    l.logits = round_up(l.counters + 4LL * MOE_COUNTERS, 256);
    l.tables = round_up(l.logits + 4LL * tokens * experts, 256);
    long long at = l.tables;
    auto take = [&](long long n) {
        char *r = ws + at;
        at += 4 * n;
        return r;
    };
    l.tab.chunks = ((experts < pairs ? experts : pairs) + 32) / 32;
    l.tab.experts = reinterpret_cast<int4 *>(take(4LL * 32 * l.tab.chunks));
    l.tab.weights = reinterpret_cast<float2 *>(take(2LL * pairs));
    l.tab.sorted = reinterpret_cast<int *>(take(pairs));
    l.tab.token = reinterpret_cast<int *>(take(pairs));
    l.tab.ids = reinterpret_cast<int *>(take(pairs));
    l.xf = round_up(at, 256);
    l.h = round_up(l.xf + 2LL * tokens * hidden, 256);
    l.part = round_up(l.h + 4LL * pairs * inter, 256);
    l.excess = round_up(l.part + 4LL * part_rows(pairs) * hidden, 256);
    l.total = round_up(l.excess + 4LL * pairs * inter, 256);
    return l;
}

int check_layer_sizes(int tokens, int hidden, int inter, int experts, int top)
{
    if (tokens < 0 || hidden <= 0 || inter <= 0)
        return status_of(STAGE_ARG, W4A16_ARG_SHAPE);
    if (experts <= 0 || top <= 0 || top > experts)
        return status_of(STAGE_ARG, W4A16_ARG_SCHEDULE);
    if (tokens > MOE_MAX_TOKENS || hidden % 256 != 0 || inter % 128 != 0)
        return status_of(STAGE_UNSUPPORTED, W4A16_ARG_SHAPE);
    if (experts > MOE_MAX_EXPERTS || top > MOE_MAX_TOP)
        return status_of(STAGE_UNSUPPORTED, W4A16_ARG_SCHEDULE);
    if ((long long)experts * hidden * inter / 4 > (1LL << 40) || hidden > (1 << 16) || inter > (1 << 16))
        return status_of(STAGE_ARG, W4A16_ARG_OVERFLOW);
    return 0;
}

using GemmKernel = void (*)(MoeGemm);
struct MoeFamily;

// The geometry of a variant, by its number of tiles.
struct MoeShape {
    int cols, warps, ctas, smem[3];
};

template <int NT>
MoeShape shape()
{
    using G = MoeGeom<NT>;
    return {G::COLS, G::WARPS, G::CTAS, {G::smem(GATE_UP), G::smem(DOWN_SIDE), G::smem(DOWN_TWICE)}};
}

MoeShape shape_of(int nt)
{
    return nt == 1 ? shape<1>() : shape<2>();
}

// 8-column tiles of the gate-up MMA's token side, by the pairs that an expert has on average and at
// most: one or two.  An expert with more pairs takes further passes over its weights, which then come
// from L2.  Two tiles leave room for twelve warps per SM instead of sixteen and pay from about eight
// pairs on (64 tokens on 8 experts of 4096 x 14336, two each: 390 us against 427 us with one tile);
// the down product, whose tile takes two MMAs, stays at one (390 us against 429 us with two).
int token_tiles(double mean, int most)
{
    return most <= 8 || mean <= 8.5 ? 1 : 2;
}

// Warps per team and parts of K of a product whose `units` units (expert, pass, columns; at most
// `most`) have `steps` steps each: the pair with the least time on the busiest warp, counting the end of a unit
// (joining the team's sums, storing) as two steps.
struct MoeSplit {
    int team, splits;
};

MoeSplit pick_split(double units, int most, int steps, const MoeShape &s, int num_sms, int max_splits)
{
    MoeSplit best = {1, 1};
    double least = -1;
    for (int team = s.warps; team >= 1; team /= 2)
        for (int splits = 1; splits <= max_splits && splits <= steps; ++splits) {
            const int teams = num_sms * s.ctas * (s.warps / team);
            if (team * splits > steps && (long long)most * splits > 2LL * teams)
                continue; // where units are drawn every member has a step of each
            const double even = units * splits / teams; // drawn units even out, but for the last
            const double rounds = even > 4.0 ? even + 1.0 : ceil(even - 0.001);
            const int part = (steps + splits - 1) / splits;
            const double cost = rounds * ((part + team - 1) / team + 2);
            if (least < 0 || cost < least) {
                least = cost;
                best = {team, splits};
            }
        }
    return best;
}

// What a call's experts come to, were each token's choice uniform: the number of them that have
// `pass` or fewer pairs counted once, up to twice that twice, and so on (an expert has n pairs with
// the binomial probability).
double expected_passes(int tokens, int experts, int top, int pass)
{
    const double q = (double)top / experts;
    if (q >= 1.0)
        return (double)experts * ((tokens + pass - 1) / pass);
    double chance = 1.0, sum = 0.0; // of n pairs
    for (int t = 0; t < tokens; ++t)
        chance *= 1.0 - q;
    for (int n = 1; n <= tokens; ++n) {
        chance *= q / (1.0 - q) * (tokens - n + 1) / n;
        sum += chance * ((n + pass - 1) / pass);
    }
    return experts * sum;
}

struct MoePlan {
    int nt_up, mode_down;
    MoeSplit up, down;
};

MoePlan moe_plan(int tokens, int hidden, int inter, int experts, int top, int num_sms)
{
    MoePlan p;
    const double active = expected_passes(tokens, experts, top, tokens), mean = tokens * (double)top / active;
    p.nt_up = token_tiles(mean, tokens);
    p.mode_down = tokens <= 4 || mean <= MOE_SIDE_MEAN ? DOWN_SIDE : DOWN_TWICE;
    const MoeShape up = shape_of(p.nt_up), down = shape_of(1);
    const int pairs = tokens * top, up_cols = 2 * inter / up.cols, down_cols = hidden / down.cols;
    p.up = pick_split(expected_passes(tokens, experts, top, pairs_per_pass(p.nt_up, GATE_UP)) * up_cols, pairs * up_cols,
                      hidden / MOE_ROWS, up, num_sms, 1);
    p.down = pick_split(expected_passes(tokens, experts, top, pairs_per_pass(1, p.mode_down)) * down_cols, pairs * down_cols,
                        inter / MOE_ROWS, down, num_sms, max_splits(pairs));
    return p;
}

cudaError_t launch_moe_gemm(MoeGemm &p, int nt, MoeSplit split, bool bf, int mode, int num_sms,
                            cudaStream_t stream)
{
    // [type][gate-up with two tiles, then the modes with one]
    static const GemmKernel kernels[2][4] = {
        {moe_layer_gemm_kernel<2, false, GATE_UP>, moe_layer_gemm_kernel<1, false, GATE_UP>,
         moe_layer_gemm_kernel<1, false, DOWN_SIDE>, moe_layer_gemm_kernel<1, false, DOWN_TWICE>},
        {moe_layer_gemm_kernel<2, true, GATE_UP>, moe_layer_gemm_kernel<1, true, GATE_UP>,
         moe_layer_gemm_kernel<1, true, DOWN_SIDE>, moe_layer_gemm_kernel<1, true, DOWN_TWICE>}};
    const int which = nt == 2 ? 0 : 1 + mode;
    const GemmKernel kernel = kernels[bf ? 1 : 0][which];
    const MoeShape s = shape_of(nt);
    const int smem = s.smem[mode];
    const int v = (bf ? 4 : 0) + which;
    cudaError_t err = allow_smem<MoeFamily, 8>(reinterpret_cast<const void *>(kernel), v, smem + MOE_TABLES_MOST);
    if (err != cudaSuccess)
        return err;
    p.team = split.team;
    p.splits = split.splits;
    p.col_units = p.n / s.cols;
    // Exact while n col_units < 2^32: an expert's unit numbers are below 16 passes x 8 splits x
    // col_units, and col_units is at most 2^11.
    p.col_magic = (uint32_t)((1ull << 32) / p.col_units + 1);
    const int tables = p.tab.chunks * 32 * (int)sizeof(int4) + (mode == GATE_UP ? p.pairs * 4 : 0);
    return launch_pdl(kernel, dim3(num_sms * s.ctas), dim3(s.warps * 32), (size_t)(smem + tables), stream, p);
}

} // namespace
} // namespace ops
} // namespace w4

using namespace w4;
using namespace w4::ops;

extern "C" size_t w4a16_moe_layer_workspace_size(int n_tokens, int hidden, int inter, int n_experts, int top_k)
{
    if (check_layer_sizes(n_tokens, hidden, inter, n_experts, top_k) != 0)
        return 0;
    return (size_t)moe_layout(nullptr, n_tokens > 0 ? n_tokens : 1, hidden, inter, n_experts, top_k).total;
}

extern "C" int w4a16_moe_layer(const void *x, int ldx, const void *router, const int32_t *gate_up,
                               const void *gate_up_scales, const void *gate_up_zeros, const int32_t *down,
                               const void *down_scales, const void *down_zeros, const void *residual, int ldr,
                               void *y, int ldy, int32_t *topk_ids, float *topk_weights, void *workspace,
                               size_t workspace_bytes, int n_tokens, int hidden, int inter, int n_experts,
                               int top_k, int group_size, int weight_type, unsigned flags, cudaStream_t stream)
{
    if (weight_type != W4A16_TYPE_U4 && weight_type != W4A16_TYPE_U4B8)
        return status_of(STAGE_ARG, W4A16_ARG_TYPE);
    const unsigned known = W4A16_FLAG_BF16 | W4A16_FLAG_IS_K_FULL | W4A16_FLAG_HAS_ZP | W4A16_FLAG_SWIGLU |
                           W4A16_FLAG_GEGLU | W4A16_FLAG_MOE_RENORM;
    const bool has_zp = (flags & W4A16_FLAG_HAS_ZP) != 0;
    const bool sw = (flags & W4A16_FLAG_SWIGLU) != 0, ge = (flags & W4A16_FLAG_GEGLU) != 0;
    if ((flags & ~known) || sw == ge || has_zp != (weight_type == W4A16_TYPE_U4) ||
        has_zp != (gate_up_zeros != nullptr) || has_zp != (down_zeros != nullptr))
        return status_of(STAGE_ARG, W4A16_ARG_FLAGS);
    int st = check_layer_sizes(n_tokens, hidden, inter, n_experts, top_k);
    if (st)
        return st;
    if (group_size != -1 &&
        (group_size <= 0 || group_size % 64 != 0 || hidden % group_size != 0 || inter % group_size != 0))
        return status_of(STAGE_ARG, W4A16_ARG_GROUP);
    if (n_tokens == 0)
        return 0;
    if (!x || !router || !gate_up || !gate_up_scales || !down || !down_scales || !y || !workspace)
        return status_of(STAGE_ARG, W4A16_ARG_NULL);
    if (ldx < hidden || ldy < hidden || (residual && ldr < hidden))
        return status_of(STAGE_ARG, W4A16_ARG_SHAPE);
    if (ldx % 8 != 0 || ldy % 8 != 0 || (residual && ldr % 8 != 0) || !aligned(x, 16) || !aligned(router, 16) ||
        !aligned(gate_up, 16) || !aligned(gate_up_scales, 16) || !aligned(gate_up_zeros, 16) ||
        !aligned(down, 16) || !aligned(down_scales, 16) || !aligned(down_zeros, 16) || !aligned(residual, 16) ||
        !aligned(y, 16) || !aligned(topk_ids, 4) || !aligned(topk_weights, 4) || !aligned(workspace, 256))
        return status_of(STAGE_ARG, W4A16_ARG_ALIGN);
    char *ws = static_cast<char *>(workspace);
    const MoeLayout lay = moe_layout(ws, n_tokens, hidden, inter, n_experts, top_k);
    if (workspace_bytes < (size_t)lay.total)
        return status_of(STAGE_ARG, W4A16_ARG_WORKSPACE);
    int num_sms = 0;
    cudaError_t err = sm_count(&num_sms);
    if (err != cudaSuccess)
        return status_of(STAGE_RESOURCE, err);

    const bool bf = (flags & W4A16_FLAG_BF16) != 0;
    const int chunks = (n_tokens + MOE_CHUNK - 1) / MOE_CHUNK;
    const MoePlan plan = moe_plan(n_tokens, hidden, inter, n_experts, top_k, num_sms);
    int *counters = reinterpret_cast<int *>(ws + lay.counters);
    RouteParams r;
    r.x = static_cast<const uint16_t *>(x);
    r.router = static_cast<const uint16_t *>(router);
    r.xf = reinterpret_cast<uint16_t *>(ws + lay.xf);
    r.logits = reinterpret_cast<float *>(ws + lay.logits);
    r.topk_ids = topk_ids;
    r.topk_weights = topk_weights;
    r.counters = counters;
    r.tab = lay.tab;
    r.ldx = ldx;
    r.tokens = n_tokens;
    r.hidden = hidden;
    r.experts = n_experts;
    r.top = top_k;
    r.renorm = (flags & W4A16_FLAG_MOE_RENORM) ? 1 : 0;
    r.up_cols = 2 * inter / shape_of(plan.nt_up).cols;
    r.down_cols = hidden / shape_of(1).cols * plan.down.splits;
    r.up_shift = plan.nt_up == 1 ? 3 : 4;
    r.down_shift = plan.mode_down == DOWN_SIDE ? 2 : 3;
    const dim3 grid(n_experts, chunks);
    err = bf ? launch_pdl(moe_layer_route_kernel<true>, grid, dim3(MOE_THREADS), 0, stream, r)
             : launch_pdl(moe_layer_route_kernel<false>, grid, dim3(MOE_THREADS), 0, stream, r);
    if (err != cudaSuccess)
        return status_of(STAGE_LAUNCH, err);

    MoeGemm m;
    m.w = gate_up;
    m.s = static_cast<const uint16_t *>(gate_up_scales);
    m.z = static_cast<const uint16_t *>(gate_up_zeros);
    m.act = r.xf;
    m.h = reinterpret_cast<uint16_t *>(ws + lay.h);
    m.part = reinterpret_cast<float *>(ws + lay.part);
    m.excess = reinterpret_cast<float *>(ws + lay.excess);
    m.ticket = counters + MOE_TICKETS;
    m.status = reinterpret_cast<int *>(ws);
    m.tab = lay.tab;
    m.pairs = n_tokens * top_k;
    m.k = hidden;
    m.n = 2 * inter;
    m.inter = inter;
    m.glu = sw ? 1 : 2;
    auto sizes = [&]() {
        m.expert_words = (long long)m.k * m.n / 8;
        m.steps = m.k / MOE_ROWS;
        m.kblocks = m.k / 64;
        // n / blocks = umulhi(n, 2^32 / blocks + 1) while n blocks < 2^32 (both are below 2^15).
        const int blocks = group_size == -1 ? m.kblocks : group_size / 64;
        m.group_magic = blocks == 1 ? 0u : (uint32_t)((1ull << 32) / blocks + 1);
        m.per_block = blocks % 2;
        m.expert_groups = m.kblocks / blocks;
    };
    sizes();
    err = launch_moe_gemm(m, plan.nt_up, plan.up, bf, GATE_UP, num_sms, stream);
    if (err != cudaSuccess)
        return status_of(STAGE_LAUNCH, err);
    m.w = down;
    m.s = static_cast<const uint16_t *>(down_scales);
    m.z = static_cast<const uint16_t *>(down_zeros);
    m.act = m.h;
    m.ticket += 1;
    m.k = inter;
    m.n = hidden;
    sizes();
    err = launch_moe_gemm(m, 1, plan.down, bf, plan.mode_down, num_sms, stream);
    if (err != cudaSuccess)
        return status_of(STAGE_LAUNCH, err);
    CombineParams c;
    c.part = m.part;
    c.weights = lay.tab.weights;
    c.residual = static_cast<const uint16_t *>(residual);
    c.y = static_cast<uint16_t *>(y);
    c.tokens = n_tokens;
    c.top = top_k;
    c.splits = plan.down.splits;
    c.hidden = hidden;
    c.ldy = ldy;
    c.ldr = ldr;
    c.h = m.h;
    c.excess = m.excess;
    c.w = m.w;
    c.s = m.s;
    c.z = m.z;
    c.expert_words = m.expert_words;
    c.expert_groups = m.expert_groups;
    c.k = inter;
    c.group_rows = group_size == -1 ? inter : group_size;
    const dim3 cgrid((hidden / 4 + 127) / 128, n_tokens);
    return launch_status(bf ? launch_pdl(moe_layer_combine_kernel<true>, cgrid, dim3(128), 0, stream, c)
                            : launch_pdl(moe_layer_combine_kernel<false>, cgrid, dim3(128), 0, stream, c));
}
