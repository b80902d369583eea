// w4a16_attention.cu -- attention of one new token per sequence over a paged key-value cache.
//
// For sequence b, query head h of KV head c = h / (n_heads / n_kv_heads), over the positions
// i in [first, len) (first = 0, or len - window with a sliding window):
//     x_i = scale q . k_i,   m = max x_i,   p_i = e^(x_i - m),   l = sum p_i,
//     out = sum p_i v_i / l,   lse = m + log l;     no position: out = 0, lse = -inf.
//
// Bound by memory: every live key and value row is read once, 4 head_dim bytes for 4 group
// head_dim flops, far below the tensor rate.  So the design is about keeping copies in flight on
// every SM whatever the lengths are:
//   - The work is cut into units of 64 positions of one row (sequence, KV head, head tile), numbered
//     in that order with a few numbers skipped before each row for what a row costs by itself, and
//     block c of G takes the numbers [c U / G, (c + 1) U / G).  Lengths are read on the device, so no
//     host copy of them is needed, ragged batches balance to one unit, and one long sequence spreads
//     over the whole GPU.
//   - A warp runs its own 16 positions of each unit: its own ring of cp.async stages, its own
//     running maximum, sum and output, so the inner loop has no block-wide barrier.  The rows of a
//     page may lie anywhere, so a row is copied by its own 16-byte copies; the page number of the
//     next step's rows is fetched one step ahead of the copies that need it.
//   - Keys and values go through mma.sync m16n8k16 with the group's query heads as the rows, which
//     is far from the tensor limit even with one head in sixteen rows.
//   - The four warps' results meet in shared memory; a row covered by several blocks is joined by
//     the last of them to arrive, in block order (bit-identical repeats).  One block reads 32 KiB of
//     partial results at a time, so more than 16 parts are joined in two levels, sixteen at a time by as many
//     blocks: 131072 positions of one KV head of 8 x 128 took 55 us with one level and take 25.
// Softmax runs in fp32 in base 2.  p is not rounded to 16 bits for the value product: it goes in as
// a 16-bit part and the 16-bit remainder (p - hi is exact in fp32).  bf16 keeps 2^-17 of any p so, the
// two parts' sixteen bits; a third part would take a further MMA.  fp16's parts hold 22 bits but end at
// 2^-25, so p goes in times 2^15 (exact, and p <= 1 stays in range), which keeps 2^-23 of p down to 2^-17
// and an absolute 2^-40 below: a long tail under one dominant position counts in the output as it does in l
// (without the factor, p below 2^-25 was in l alone).  With at most eight heads per KV head the remainder
// takes the upper eight rows of the same MMA, which are empty then; with more it costs a second MMA.
#include <type_traits>

#include "w4a16_ops.cuh"

namespace w4 {
namespace ops {

constexpr int ATT_WARPS = 4;
constexpr int ATT_THREADS = ATT_WARPS * 32;
constexpr int ATT_STEP = 16;                    // positions per warp and step
constexpr int ATT_UNIT = ATT_WARPS * ATT_STEP;  // positions per work unit
constexpr int ATT_ROWS = 16;                    // query heads per head tile
constexpr int ATT_MAX_BATCH = 4096;
constexpr float LN2 = 0.6931471805599453f;
constexpr int ATT_FAN = 16;                     // parts of a row joined at once
constexpr int ATT_SLOTS = 3;                    // partials of a block: first row, last row, joined group

struct AttParams {
    const uint16_t *q, *k, *v;
    uint16_t *out;
    float *lse;
    const int32_t *table, *lens;
    int *status, *counters, *group_counters;
    float *partials;
    long long page_stride, token_stride, head_stride;
    int ldq, ldo, ld_table;
    int batch, heads, kv, group, tiles; // tiles: head tiles of a KV head's group
    int page, n_pages, max_len, window;
    float scale_log2; // scale * log2(e)
};

// Positions [first, len) of sequence b; a length outside [0, max_len] is reported and clamped.
__device__ __forceinline__ void live_range(const AttParams &p, int b, int &first, int &len)
{
    len = p.lens[b];
    if (len < 0 || len > p.max_len) {
        atomicOr(p.status, W4A16_DEV_LENGTH);
        len = len < 0 ? 0 : p.max_len;
    }
    first = p.window > 0 && len > p.window ? len - p.window : 0;
}

// a / b for 0 <= a < 2^31 b: in 32 bits where both fit (64-bit division is a long sequence).
__device__ __forceinline__ int quotient(long long a, long long b, bool small)
{
    return small ? (int)((uint32_t)a / (uint32_t)b) : (int)(a / b);
}

template <int D>
struct AttGeom {
    static constexpr int ROW = D * 2;                  // bytes of a key or value row
    static constexpr int CHUNKS = D / 8;               // 16-byte chunks of a row
    static constexpr int STAGES = 3;
    static constexpr int CTAS = D == 64 ? 3 : D == 128 ? 2 : 1; // blocks per SM
    // What a row costs beside its units, in units: its queries, the start and the end of its copies
    // and the joining of the warps take about as long as copying 128 KiB.
    static constexpr int ROW_COST = D == 64 ? 8 : 4;
    static constexpr int STAGE = 2 * ATT_STEP * ROW;   // keys, then values
    static constexpr int WARP = STAGES * STAGE;
    static constexpr int SMEM = ATT_WARPS * WARP;
    static constexpr int SLOT = ATT_ROWS * (D + 2);    // floats of a partial: rows, then (m, l)
};

// PACK: at most eight heads in a tile.
// bf16, 128 wide: 32 sequences of 2048 to 32768 positions, 64 / 8 heads, 235 us, 6.55 TB/s of keys and
// values; one of 131071 with 40 / 8 heads 86.3 us, 6.22 TB/s (3 us pass before the first rows, 8 us
// from the last to the end of the join of 38 parts a row).  fp16, 24 sequences of 5 to 9000 with a
// window of 2048, 12 / 12 heads of 64: 17.6 us, of which half is the start and the join; one of 37
// positions: 4.0 us of latencies.
template <int D, bool BF, bool PACK>
__global__ void __launch_bounds__(ATT_THREADS, AttGeom<D>::CTAS)
    paged_attention_kernel(const AttParams p)
{
    using G = AttGeom<D>;
    constexpr int KS = D / 16; // k steps of the score product
    constexpr int NT = D / 8;  // 8-wide output tiles
    // What p is multiplied by for the value product, and its inverse for the outputs.
    constexpr float UP = BF ? 1.f : 32768.f, DOWN = 1.f / UP;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int prefix[ATT_MAX_BATCH + 1]; // numbers of one (KV head, head tile) before sequence b
    __shared__ int warp_sum[ATT_WARPS];
    __shared__ uint32_t live_mask[ATT_WARPS][G::STAGES];
    __shared__ float stat[ATT_WARPS][ATT_ROWS][2];
    __shared__ int is_last;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;
    pdl_wait();
    pdl_launch_dependents();

    // --- the schedule: units before each sequence ---------------------------------------------
    int run = 0;
    for (int base = 0; base < p.batch; base += ATT_THREADS) {
        const int b = base + tid;
        int n = 0;
        if (b < p.batch) {
            int first, len;
            live_range(p, b, first, len);
            n = (len - first + ATT_UNIT - 1) / ATT_UNIT;
            n += n > 0 ? G::ROW_COST : 0;
        }
        int incl = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d)
                incl += o;
        }
        if (lane == 31)
            warp_sum[warp] = incl;
        __syncthreads();
        int before = run;
#pragma unroll
        for (int w = 0; w < ATT_WARPS; ++w) {
            if (w < warp)
                before += warp_sum[w];
            run += warp_sum[w];
        }
        if (b < p.batch)
            prefix[b] = before + incl - n;
        __syncthreads();
    }
    if (tid == 0)
        prefix[p.batch] = run;
    __syncthreads();
    const int rows_per_seq = p.kv * p.tiles;
    const long long units = (long long)run * rows_per_seq;
    const int grid = (int)min((long long)gridDim.x, units);

    // Sequences without a position: zeros and -inf.
    for (int b = blockIdx.x; b < p.batch; b += gridDim.x) {
        if (prefix[b + 1] != prefix[b])
            continue;
        for (int i = tid; i < p.heads * D / 8; i += ATT_THREADS)
            *reinterpret_cast<uint4 *>(p.out + (long long)b * p.ldo + 8 * i) = make_uint4(0, 0, 0, 0);
        if (p.lse)
            for (int h = tid; h < p.heads; h += ATT_THREADS)
                p.lse[(long long)b * p.heads + h] = -INFINITY;
    }
    if ((int)blockIdx.x >= grid)
        return;

    const bool small = units * (grid + 1LL) < (1LL << 32);
    auto begin_of = [&](int c) {
        return small ? (long long)((uint32_t)(c * (uint32_t)units) / (uint32_t)grid) : c * units / grid;
    };
    auto owner_of = [&](long long number) { return quotient((number + 1) * grid - 1, units, small); };
    const long long u_begin = begin_of(blockIdx.x), u_end = begin_of(blockIdx.x + 1);
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * G::WARP;

    for (long long u = u_begin; u < u_end;) {
        // --- the row of this segment and its positions ----------------------------------------
        int lo = 0, hi = p.batch - 1; // last b with prefix[b] * rows_per_seq <= u
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if ((long long)prefix[mid] * rows_per_seq <= u)
                lo = mid;
            else
                hi = mid - 1;
        }
        const int b = lo, span = prefix[b + 1] - prefix[b], seq_units = span - G::ROW_COST;
        const long long rem = u - (long long)prefix[b] * rows_per_seq;
        const int row = quotient(rem, span, small);         // (KV head, head tile)
        const long long row_u0 = u - (rem - (long long)row * span) + G::ROW_COST; // of unit 0
        const int unit0 = (int)max(0LL, u - row_u0);
        const int unit1 = (int)min((long long)seq_units, u_end - row_u0);
        u = row_u0 + seq_units; // the row after this one
        if (unit1 <= unit0)
            break; // the range ends before the row's first unit
        const int c = row / p.tiles, h0 = (row - c * p.tiles) * ATT_ROWS;
        const int nh = min(ATT_ROWS, p.group - h0); // heads of this tile
        int first, len;
        live_range(p, b, first, len);
        const int steps = unit1 - unit0;
        const int pos0 = first + unit0 * ATT_UNIT + warp * ATT_STEP; // this warp's first position

        float o[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o[n][i] = 0.f;
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

        // --- copies ---------------------------------------------------------------------------
        // Lane r < 16 looks after row r of a step: page number fetched one step early, then the
        // row's element offset, handed to the copying lanes by shuffles.
        const int32_t *tab = p.table + (long long)b * p.ld_table;
        const long long head_off = (long long)c * p.head_stride;
        auto fetch_page = [&](int step) -> int {
            const int pos = pos0 + step * ATT_UNIT + (lane & 15);
            return step < steps && pos < len ? tab[pos / p.page] : -1;
        };
        auto issue = [&](int step, int stage, int pg) {
            const int pos = pos0 + step * ATT_UNIT + (lane & 15);
            const bool in = step < steps && pos < len;
            bool ok = in && pg >= 0 && pg < p.n_pages;
            if (in && !ok)
                atomicOr(p.status, W4A16_DEV_PAGE);
            const long long off =
                ok ? head_off + (long long)pg * p.page_stride + (long long)(pos % p.page) * p.token_stride : 0;
            const uint32_t mask = __ballot_sync(0xffffffffu, ok) & 0xffffu;
            if (lane == 0)
                live_mask[warp][stage] = mask;
            constexpr int ROWS_AT_ONCE = 32 / G::CHUNKS > 0 ? 32 / G::CHUNKS : 1;
            const int ch = lane % G::CHUNKS, sub = lane / G::CHUNKS;
            const uint32_t kst = ring + stage * G::STAGE, vst = kst + ATT_STEP * G::ROW;
#pragma unroll
            for (int r0 = 0; r0 < ATT_STEP; r0 += ROWS_AT_ONCE) {
                const int r = r0 + sub;
                const long long ro = __shfl_sync(0xffffffffu, off, r);
                const bool live = (mask >> r) & 1u;
                const uint32_t dst = r * G::ROW + ((ch ^ (r & 7)) << 4);
                cp_async16(kst + dst, p.k + ro + ch * 8, live);
                cp_async16(vst + dst, p.v + ro + ch * 8, live);
            }
        };
        int pages[G::STAGES];
#pragma unroll
        for (int s = 0; s < G::STAGES; ++s)
            pages[s] = fetch_page(s);

        // --- queries: A fragments of the score product ----------------------------------------
        uint32_t qa[KS][PACK ? 2 : 4];
        {
            const uint16_t *qp = p.q + (long long)b * p.ldq + (long long)(c * p.group + h0) * D;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const uint16_t *r0 = qp + (long long)g * D + ks * 16 + 2 * t;
                qa[ks][0] = g < nh ? *reinterpret_cast<const uint32_t *>(r0) : 0u;
                qa[ks][1] = g < nh ? *reinterpret_cast<const uint32_t *>(r0 + 8) : 0u;
                if (!PACK) {
                    const uint16_t *r1 = r0 + 8 * D;
                    qa[ks][2] = g + 8 < nh ? *reinterpret_cast<const uint32_t *>(r1) : 0u;
                    qa[ks][3] = g + 8 < nh ? *reinterpret_cast<const uint32_t *>(r1 + 8) : 0u;
                }
            }
        }

#pragma unroll
        for (int s = 0; s < G::STAGES - 1; ++s) {
            issue(s, s, pages[s]);
            cp_async_commit();
        }
        int next_page = pages[G::STAGES - 1];

        // --- the running softmax --------------------------------------------------------------
        int stage = 0;
        for (int step = 0; step < steps; ++step) {
            cp_async_wait<G::STAGES - 2>();
            __syncwarp(); // every lane's copies of this stage have landed; the next one is free
            {
                const int pg = next_page;
                next_page = fetch_page(step + G::STAGES);
                int ns = stage + G::STAGES - 1;
                ns = ns >= G::STAGES ? ns - G::STAGES : ns;
                issue(step + G::STAGES - 1, ns, pg);
                cp_async_commit();
            }
            const uint32_t kst = ring + stage * G::STAGE, vst = kst + ATT_STEP * G::ROW;
            const uint32_t mask = live_mask[warp][stage];
            float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
            {
                // The MMA cuts its sums off instead of rounding them, which over head_dim costs the scores (and lse)
                // up to a bit and a half: so two MMAs at a time, added in fp32 (lse of one position of 128: a
                // relative error of 7.9e-8 instead of 1.8e-7, at the same speed).  With PACK and 256
                // wide heads the registers do not suffice (47 sequences of 40 / 8 heads: 52 us instead of 45), and the
                // sum stays whole.
                constexpr int CHAIN = D == 256 && PACK ? KS : 2;
                float t0[4], t1[4];
                // Matrices: (positions 0-7, chunk 2 ks), (0-7, 2 ks + 1), (8-15, 2 ks), (8-15, 2 ks + 1).
                const int r = (lane & 7) + ((lane >> 4) << 3), cc = (lane >> 3) & 1;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    uint32_t kb[4];
                    ldsm_x4(kst + r * G::ROW + (((2 * ks + cc) ^ (r & 7)) << 4), kb);
                    const uint32_t a1 = PACK ? 0u : qa[ks][PACK ? 0 : 2], a3 = PACK ? 0u : qa[ks][PACK ? 0 : 3];
                    if (ks % CHAIN == 0) {
                        mma16816_zero<BF>(t0, qa[ks][0], a1, qa[ks][1], a3, kb[0], kb[1]);
                        mma16816_zero<BF>(t1, qa[ks][0], a1, qa[ks][1], a3, kb[2], kb[3]);
                    } else {
                        mma16816<BF>(t0, qa[ks][0], a1, qa[ks][1], a3, kb[0], kb[1]);
                        mma16816<BF>(t1, qa[ks][0], a1, qa[ks][1], a3, kb[2], kb[3]);
                    }
                    if (ks % CHAIN == CHAIN - 1) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            s0[i] += t0[i];
                            s1[i] += t1[i];
                        }
                    }
                }
            }
            // Values (row g: [0], [1]; row g + 8: [2], [3]) of positions 2 t, 2 t + 1 and 8 on.
            const uint32_t mk = mask >> (2 * t);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s0[i] = (mk >> (i & 1)) & 1u ? s0[i] * p.scale_log2 : -INFINITY;
                s1[i] = (mk >> (8 + (i & 1))) & 1u ? s1[i] * p.scale_log2 : -INFINITY;
            }
            uint32_t hi0, hi1, lo0, lo1; // p of row g, positions 2 t and 8 + 2 t: 16-bit part, remainder
            uint32_t hj0 = 0, hj1 = 0, lj0 = 0, lj1 = 0;
            float f0, f1 = 1.f;
            auto soften = [&](float &m, float &l, float a, float b2, float c2, float d2, float &f,
                              uint32_t &h_lo, uint32_t &h_hi, uint32_t &r_lo, uint32_t &r_hi) {
                float top = fmaxf(fmaxf(a, b2), fmaxf(c2, d2));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const float mn = fmaxf(m, top);
                const float base = mn == -INFINITY ? 0.f : mn; // nothing live yet: every p is 0
                f = exp2f(m - base);
                m = mn;
                const float pa = exp2f(a - base), pb = exp2f(b2 - base), pc = exp2f(c2 - base),
                            pd = exp2f(d2 - base);
                l = l * f + ((pa + pb) + (pc + pd));
                const float sa = pa * UP, sb = pb * UP, sc = pc * UP, sd = pd * UP;
                h_lo = pack2<BF>(sa, sb);
                h_hi = pack2<BF>(sc, sd);
                const float2 ra = unpack2<BF>(h_lo), rc = unpack2<BF>(h_hi);
                r_lo = pack2<BF>(sa - ra.x, sb - ra.y);
                r_hi = pack2<BF>(sc - rc.x, sd - rc.y);
            };
            soften(m0, l0, s0[0], s0[1], s1[0], s1[1], f0, hi0, hi1, lo0, lo1);
            if (!PACK)
                soften(m1, l1, s0[2], s0[3], s1[2], s1[3], f1, hj0, hj1, lj0, lj1);
            else
                f1 = f0;
            if (__any_sync(0xffffffffu, f0 != 1.f || f1 != 1.f)) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    o[n][0] *= f0;
                    o[n][1] *= f0;
                    o[n][2] *= f1;
                    o[n][3] *= f1;
                }
            }
            {
                // Matrices: (positions 0-7, chunk j), (8-15, j), (0-7, j + 1), (8-15, j + 1).
                const int r = (lane & 7) + (((lane >> 3) & 1) << 3), cc = lane >> 4;
#pragma unroll
                for (int n = 0; n < NT; n += 2) {
                    uint32_t vb[4];
                    ldsm_x4_trans(vst + r * G::ROW + (((n + cc) ^ (r & 7)) << 4), vb);
                    if (PACK) {
                        mma16816<BF>(o[n], hi0, lo0, hi1, lo1, vb[0], vb[1]);
                        mma16816<BF>(o[n + 1], hi0, lo0, hi1, lo1, vb[2], vb[3]);
                    } else {
                        mma16816<BF>(o[n], hi0, hj0, hi1, hj1, vb[0], vb[1]);
                        mma16816<BF>(o[n + 1], hi0, hj0, hi1, hj1, vb[2], vb[3]);
                        mma16816<BF>(o[n], lo0, lj0, lo1, lj1, vb[0], vb[1]);
                        mma16816<BF>(o[n + 1], lo0, lj0, lo1, lj1, vb[2], vb[3]);
                    }
                }
            }
            stage = stage + 1 == G::STAGES ? 0 : stage + 1;
        }
        cp_async_wait<0>();

        // --- the warps' results meet in shared memory (the ring is free) ----------------------
        l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
        l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
        __syncthreads();
        float *acc = reinterpret_cast<float *>(smem); // [warp][row][D]
        constexpr int R = PACK ? 8 : 16;
        {
            float *mine = acc + warp * R * D;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float a = PACK ? o[n][0] + o[n][2] : o[n][0], bb = PACK ? o[n][1] + o[n][3] : o[n][1];
                *reinterpret_cast<float2 *>(mine + g * D + n * 8 + 2 * t) = make_float2(a, bb);
                if (!PACK)
                    *reinterpret_cast<float2 *>(mine + (g + 8) * D + n * 8 + 2 * t) =
                        make_float2(o[n][2], o[n][3]);
            }
            if (t == 0) {
                stat[warp][g][0] = m0;
                stat[warp][g][1] = l0;
                if (!PACK) {
                    stat[warp][g + 8][0] = m1;
                    stat[warp][g + 8][1] = l1;
                }
            }
        }
        __syncthreads();
        const bool whole = steps == seq_units;
        const int slot = u_begin >= row_u0 ? 0 : 1; // a block shares at most its first and its last row
        float *part = p.partials + ((long long)blockIdx.x * ATT_SLOTS + slot) * G::SLOT;
        uint16_t *out = p.out + (long long)b * p.ldo + (long long)(c * p.group + h0) * D;
        const long long lse_at = (long long)b * p.heads + c * p.group + h0;
        for (int i = tid; i < nh * (D / 4); i += ATT_THREADS) {
            const int h = i / (D / 4), d = (i - h * (D / 4)) * 4;
            float mx = -INFINITY;
#pragma unroll
            for (int w = 0; w < ATT_WARPS; ++w)
                mx = fmaxf(mx, stat[w][h][0]);
            const float base = mx == -INFINITY ? 0.f : mx;
            float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
            float l = 0.f;
#pragma unroll
            for (int w = 0; w < ATT_WARPS; ++w) {
                const float f = exp2f(stat[w][h][0] - base);
                const float4 x = *reinterpret_cast<const float4 *>(acc + (w * R + h) * D + d);
                l += f * stat[w][h][1];
                sum.x += f * x.x;
                sum.y += f * x.y;
                sum.z += f * x.z;
                sum.w += f * x.w;
            }
            if (whole) {
                const float r = l == 0.f ? 0.f : DOWN / l;
                uint2 w2;
                w2.x = pack2<BF>(sum.x * r, sum.y * r);
                w2.y = pack2<BF>(sum.z * r, sum.w * r);
                *reinterpret_cast<uint2 *>(out + (long long)h * D + d) = w2;
                if (d == 0 && p.lse)
                    p.lse[lse_at + h] = l == 0.f ? -INFINITY : fmaf(base, LN2, logf(l));
            } else {
                __stcg(reinterpret_cast<float4 *>(part + h * D + d), sum);
                if (d == 0)
                    __stcg(reinterpret_cast<float2 *>(part + ATT_ROWS * D + 2 * h), make_float2(mx, l));
            }
        }
        if (!whole) {
            // The parts of a row are those of the blocks c_lo to c_hi, the owners of its first and its
            // last unit.  The last block to arrive joins them; where there are more than ATT_FAN, the
            // last of every ATT_FAN of them joins those first, so that many blocks share the reading.
            // A row's counter is that of its first block, in which no other row of several parts starts;
            // a group's likewise (a group of one part, which could share its block with the next row's
            // first, does not count).
            const int c_lo = owner_of(row_u0), c_hi = owner_of(row_u0 + seq_units - 1);
            const int lo_slot = begin_of(c_lo) >= row_u0 ? 0 : 1, parts = c_hi - c_lo + 1;
            const int group0 = ((int)blockIdx.x - c_lo) / ATT_FAN * ATT_FAN; // this block's group
            bool last_level = parts <= ATT_FAN;
            if (!last_level && group0 + 1 == parts)
                last_level = true; // a group of one part is read as it is
            for (;;) {
                // Joined here: a row's parts, a group of them, or a row's groups.
                const bool groups = last_level && parts > ATT_FAN;
                const int n = groups       ? (parts + ATT_FAN - 1) / ATT_FAN
                              : last_level ? parts
                                           : min(ATT_FAN, parts - group0);
                const int from = c_lo + (last_level ? 0 : group0);
                __syncthreads();
                if (tid == 0) {
                    int *counter = last_level ? p.counters + c_lo : p.group_counters + from;
                    const int last = arrive_counter(counter) == n - 1;
                    if (last)
                        *counter = 0;
                    is_last = last;
                }
                __syncthreads();
                if (!is_last)
                    break;
                // A thread sums ITEMS quads of outputs over the parts in block order, the loads of AT
                // parts in flight at once (sixteen loads in all: few parts of 16 heads of 256 take 11.2 us
                // instead of 13.2 with one quad at a time), rescaling as the maximum moves.
                auto join = [&](auto items_c, auto at_c) {
                    constexpr int ITEMS = decltype(items_c)::value, AT = decltype(at_c)::value;
                    const int quads = nh * (D / 4);
                    for (int i0 = tid; i0 < quads; i0 += ITEMS * ATT_THREADS) {
                        float m[ITEMS], l[ITEMS];
                        float4 sum[ITEMS];
#pragma unroll
                        for (int k = 0; k < ITEMS; ++k) {
                            m[k] = -INFINITY;
                            l[k] = 0.f;
                            sum[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                        }
                        for (int q0 = 0; q0 < n; q0 += AT) {
                            float2 ml[ITEMS][AT];
                            float4 x[ITEMS][AT];
#pragma unroll
                            for (int q = 0; q < AT; ++q) {
                                const int at = groups ? (q0 + q) * ATT_FAN : q0 + q;
                                const int which = groups && at + 1 < parts ? ATT_SLOTS - 1 : from + at == c_lo ? lo_slot : 0;
                                const float *pp = p.partials + ((long long)(from + at) * ATT_SLOTS + which) * G::SLOT;
#pragma unroll
                                for (int k = 0; k < ITEMS; ++k) {
                                    const int i = i0 + k * ATT_THREADS;
                                    const bool in = q0 + q < n && i < quads;
                                    ml[k][q] = in ? __ldcg(reinterpret_cast<const float2 *>(pp + ATT_ROWS * D) + i / (D / 4))
                                                  : make_float2(-INFINITY, 0.f);
                                    x[k][q] = in ? __ldcg(reinterpret_cast<const float4 *>(pp) + i)
                                                 : make_float4(0.f, 0.f, 0.f, 0.f);
                                }
                            }
#pragma unroll
                            for (int k = 0; k < ITEMS; ++k) {
                                float mn = m[k];
#pragma unroll
                                for (int q = 0; q < AT; ++q)
                                    mn = fmaxf(mn, ml[k][q].x);
                                const float base = mn == -INFINITY ? 0.f : mn, f0 = exp2f(m[k] - base);
                                m[k] = mn;
                                l[k] *= f0;
                                sum[k].x *= f0;
                                sum[k].y *= f0;
                                sum[k].z *= f0;
                                sum[k].w *= f0;
#pragma unroll
                                for (int q = 0; q < AT; ++q) {
                                    const float f = exp2f(ml[k][q].x - base);
                                    l[k] = fmaf(f, ml[k][q].y, l[k]);
                                    sum[k].x = fmaf(f, x[k][q].x, sum[k].x);
                                    sum[k].y = fmaf(f, x[k][q].y, sum[k].y);
                                    sum[k].z = fmaf(f, x[k][q].z, sum[k].z);
                                    sum[k].w = fmaf(f, x[k][q].w, sum[k].w);
                                }
                            }
                        }
#pragma unroll
                        for (int k = 0; k < ITEMS; ++k) {
                            const int i = i0 + k * ATT_THREADS;
                            if (i >= quads)
                                continue;
                            const bool first_quad = i % (D / 4) == 0;
                            if (last_level) {
                                const float r = l[k] == 0.f ? 0.f : DOWN / l[k];
                                uint2 w2;
                                w2.x = pack2<BF>(sum[k].x * r, sum[k].y * r);
                                w2.y = pack2<BF>(sum[k].z * r, sum[k].w * r);
                                *reinterpret_cast<uint2 *>(out + 4LL * i) = w2;
                                if (p.lse && first_quad)
                                    p.lse[lse_at + i / (D / 4)] =
                                        l[k] == 0.f ? -INFINITY : fmaf(m[k], LN2, logf(l[k]));
                            } else {
                                float *to = p.partials + ((long long)from * ATT_SLOTS + ATT_SLOTS - 1) * G::SLOT;
                                __stcg(reinterpret_cast<float4 *>(to) + i, sum[k]);
                                if (first_quad)
                                    __stcg(reinterpret_cast<float2 *>(to + ATT_ROWS * D) + i / (D / 4),
                                           make_float2(m[k], l[k]));
                            }
                        }
                    }
                };
                using std::integral_constant;
                if (n <= 4)
                    join(integral_constant<int, 4>(), integral_constant<int, 4>());
                else if (n <= 8)
                    join(integral_constant<int, 2>(), integral_constant<int, 8>());
                else
                    join(integral_constant<int, 1>(), integral_constant<int, 16>());
                if (last_level)
                    break;
                last_level = true;
            }
        }
        if (u < u_end)
            __syncthreads(); // the ring and the statistics are read before the next segment fills them
    }
}

namespace {

using AttKernel = void (*)(AttParams);

// The kernel of a call, allowed its shared memory on the current device (once per device).
template <int D>
cudaError_t att_kernel(bool bf, bool pack, AttKernel &kernel, int &smem)
{
    static const AttKernel kernels[4] = {
        paged_attention_kernel<D, false, false>, paged_attention_kernel<D, false, true>,
        paged_attention_kernel<D, true, false>, paged_attention_kernel<D, true, true>};
    const int v = (bf ? 2 : 0) + (pack ? 1 : 0);
    kernel = kernels[v];
    smem = AttGeom<D>::SMEM;
    return allow_smem<AttGeom<D>, 4>(reinterpret_cast<const void *>(kernel), v, smem);
}

int att_grid(int num_sms, int head_dim)
{
    return num_sms * (head_dim == 64 ? AttGeom<64>::CTAS : head_dim == 128 ? AttGeom<128>::CTAS : AttGeom<256>::CTAS);
}

// A workspace: status, the counters, the partials.  The counters' places are the same for calls of all
// sizes on a device (a counter per block of the largest grid), so that no call's partials lie where
// another one's counters have to be zero.
struct AttLayout {
    long long group_counters, counters, partials, total;
};

AttLayout att_layout(int head_dim, int num_sms)
{
    AttLayout l;
    const long long blocks = att_grid(num_sms, 64);
    static_assert(AttGeom<64>::CTAS >= AttGeom<128>::CTAS && AttGeom<64>::CTAS >= AttGeom<256>::CTAS, "the largest grid");
    l.group_counters = HEADER_BYTES;
    l.counters = l.group_counters + 4 * blocks;
    l.partials = round_up(l.counters + 4 * blocks, 256);
    l.total = l.partials + (long long)att_grid(num_sms, head_dim) * ATT_SLOTS * ATT_ROWS * (head_dim + 2) * 4;
    return l;
}

// Sizes that do not depend on a buffer; 0 or a status.
int check_sizes(int batch, int n_heads, int n_kv_heads, int head_dim)
{
    if (batch < 0 || n_heads <= 0 || n_kv_heads <= 0 || head_dim <= 0 || n_heads % n_kv_heads != 0)
        return status_of(STAGE_ARG, W4A16_ARG_SHAPE);
    if ((head_dim != 64 && head_dim != 128 && head_dim != 256) || batch > ATT_MAX_BATCH)
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

extern "C" size_t w4a16_paged_attention_workspace_size(int batch, int n_heads, int n_kv_heads, int head_dim,
                                                       int num_sms)
{
    if (check_sizes(batch, n_heads, n_kv_heads, head_dim) != 0)
        return 0;
    if (num_sms <= 0 && sm_count(&num_sms) != cudaSuccess)
        return 0;
    return (size_t)att_layout(head_dim, num_sms).total;
}

extern "C" int w4a16_paged_attention(const void *q, int ldq, const void *k_cache, const void *v_cache,
                                     long long kv_page_stride, long long kv_token_stride,
                                     long long kv_head_stride, void *out, int ldo, float *lse,
                                     const int32_t *block_table, int ld_table, const int32_t *seq_lens,
                                     void *workspace, size_t workspace_bytes, int batch, int n_heads,
                                     int n_kv_heads, int head_dim, int page_size, int n_pages,
                                     int max_pages, int window, float scale, unsigned flags,
                                     cudaStream_t stream)
{
    if (flags & ~W4A16_FLAG_BF16)
        return status_of(STAGE_ARG, W4A16_ARG_FLAGS);
    int st = check_sizes(batch, n_heads, n_kv_heads, head_dim);
    if (st)
        return st;
    if (page_size <= 0 || n_pages <= 0 || max_pages <= 0 || window < 0)
        return status_of(STAGE_ARG, W4A16_ARG_SHAPE);
    if (batch == 0)
        return 0;
    if (!q || !k_cache || !v_cache || !out || !block_table || !seq_lens || !workspace)
        return status_of(STAGE_ARG, W4A16_ARG_NULL);
    if (ldq < n_heads * head_dim || ldo < n_heads * head_dim || ld_table < max_pages ||
        kv_page_stride < 0 || kv_token_stride < 0 || kv_head_stride < 0)
        return status_of(STAGE_ARG, W4A16_ARG_SHAPE);
    if (ldq % 8 != 0 || ldo % 8 != 0 || kv_page_stride % 8 != 0 || kv_token_stride % 8 != 0 ||
        kv_head_stride % 8 != 0 || !aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        !aligned(out, 16) || !aligned(lse, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
        !aligned(workspace, 256))
        return status_of(STAGE_ARG, W4A16_ARG_ALIGN);
    // Positions and units are counted in 32 bits (offsets into the cache in 64): a sequence holds
    // at most max_pages pages.
    const long long max_len = (long long)max_pages * page_size;
    if (max_len > 0x7FFFFFFFLL - 64 * ATT_UNIT ||
        ((max_len + ATT_UNIT - 1) / ATT_UNIT + 8) * batch > 0x7FFFFFFFLL)
        return status_of(STAGE_ARG, W4A16_ARG_OVERFLOW);

    int num_sms = 0;
    cudaError_t err = sm_count(&num_sms);
    if (err != cudaSuccess)
        return status_of(STAGE_RESOURCE, err);
    const int group = n_heads / n_kv_heads, tiles = (group + ATT_ROWS - 1) / ATT_ROWS;
    const int grid = att_grid(num_sms, head_dim);
    const AttLayout lay = att_layout(head_dim, num_sms);
    if (workspace_bytes < (size_t)lay.total)
        return status_of(STAGE_ARG, W4A16_ARG_WORKSPACE);
    char *ws = static_cast<char *>(workspace);
    AttParams p;
    p.q = static_cast<const uint16_t *>(q);
    p.k = static_cast<const uint16_t *>(k_cache);
    p.v = static_cast<const uint16_t *>(v_cache);
    p.out = static_cast<uint16_t *>(out);
    p.lse = lse;
    p.table = block_table;
    p.lens = seq_lens;
    p.status = reinterpret_cast<int *>(ws);
    p.counters = reinterpret_cast<int *>(ws + lay.counters);
    p.group_counters = reinterpret_cast<int *>(ws + lay.group_counters);
    p.partials = reinterpret_cast<float *>(ws + lay.partials);
    p.page_stride = kv_page_stride;
    p.token_stride = kv_token_stride;
    p.head_stride = kv_head_stride;
    p.ldq = ldq;
    p.ldo = ldo;
    p.ld_table = ld_table;
    p.batch = batch;
    p.heads = n_heads;
    p.kv = n_kv_heads;
    p.group = group;
    p.tiles = tiles;
    p.page = page_size;
    p.n_pages = n_pages;
    p.max_len = (int)max_len;
    p.window = window;
    p.scale_log2 = scale * 1.4426950408889634f;
    const bool bf = (flags & W4A16_FLAG_BF16) != 0, pack = group <= 8;
    AttKernel kernel;
    int smem;
    err = head_dim == 64    ? att_kernel<64>(bf, pack, kernel, smem)
          : head_dim == 128 ? att_kernel<128>(bf, pack, kernel, smem)
                            : att_kernel<256>(bf, pack, kernel, smem);
    if (err != cudaSuccess)
        return status_of(STAGE_RESOURCE, err);
    return launch_status(launch_pdl(kernel, dim3(grid), dim3(ATT_THREADS), (size_t)smem, stream, p));
}
