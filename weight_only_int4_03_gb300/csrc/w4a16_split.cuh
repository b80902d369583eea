// w4a16_split.cuh -- how attention over sequences of any lengths is split over the GPU, and joined.
//
// A row is a sequence with some of its heads.  Its positions are cut into units, all rows' units are numbered in
// order with COST numbers skipped before each row for what a row costs by itself, and block c of G takes the
// numbers [c U / G, (c + 1) U / G).  Lengths are read on the device; ragged batches balance to one unit, and one
// long sequence spreads over all blocks.  A block's warps leave their results (outputs, maximum, sum) in shared
// memory; a row covered by several blocks is joined by the last of them to arrive, in block order, so that repeats
// are bit-identical.  More than SPLIT_FAN parts are joined in two levels, SPLIT_FAN at a time by as many blocks.
#pragma once

#include <type_traits>

#include "w4a16_ops.cuh"

namespace w4 {
namespace ops {

constexpr int SPLIT_WARPS = 4;
constexpr int SPLIT_THREADS = SPLIT_WARPS * 32;
constexpr int SPLIT_MAX_BATCH = 4096;
constexpr int SPLIT_MAX_CTAS = 3; // blocks per SM of any kernel that is split like this
constexpr int SPLIT_FAN = 16;  // parts of a row joined at once
constexpr int SPLIT_SLOTS = 3; // partials of a block: first row, last row, joined group
constexpr float SPLIT_LN2 = 0.6931471805599453f;

struct SplitParams {
    const int32_t *lens;
    int *status, *counters, *group_counters;
    float *partials;
    int batch, rows_per_seq, max_len, window;
    int slot; // floats of a partial: [heads][dim], then (maximum, sum) of each head
};

struct SplitShared {
    int prefix[SPLIT_MAX_BATCH + 1]; // numbers of one of a sequence's rows, before sequence b
    int warp_sum[SPLIT_WARPS];
    int is_last;
};

// Units [unit0, unit1) of row `row` of sequence b, whose positions are [first, len).
struct SplitSegment {
    long long row_u0; // number of the row's unit 0
    int b, row, first, len;
    int start; // of unit 0: first, or the multiple of a unit before it
    int unit0, unit1, units;
    bool more; // another segment of this block may follow
};

// A workspace: status, the counters, the partials.  The counters' places are the same for calls of all sizes and
// both kinds of cache on a device (a counter per block of the largest grid), so that no call's partials lie where another one's counters
// have to be zero.
struct SplitLayout {
    long long group_counters, counters, partials, total;
    int slot;
};

inline SplitLayout split_layout(long long most_blocks, long long blocks, int slot)
{
    SplitLayout l;
    l.group_counters = HEADER_BYTES;
    l.counters = l.group_counters + 4 * most_blocks;
    l.partials = round_up(l.counters + 4 * most_blocks, 256);
    l.total = l.partials + blocks * SPLIT_SLOTS * slot * 4;
    l.slot = slot;
    return l;
}

inline void split_params(SplitParams &p, const SplitLayout &lay, void *workspace, const int32_t *lens, int batch,
                         int rows_per_seq, int max_len, int window)
{
    char *ws = static_cast<char *>(workspace);
    p.lens = lens;
    p.status = reinterpret_cast<int *>(ws);
    p.counters = reinterpret_cast<int *>(ws + lay.counters);
    p.group_counters = reinterpret_cast<int *>(ws + lay.group_counters);
    p.partials = reinterpret_cast<float *>(ws + lay.partials);
    p.batch = batch;
    p.rows_per_seq = rows_per_seq;
    p.max_len = max_len;
    p.window = window;
    p.slot = lay.slot;
}

// a / b for 0 <= a < 2^31 b: in 32 bits where both fit (64-bit division is a long sequence).
__device__ __forceinline__ int split_quotient(long long a, long long b, bool small)
{
    return small ? (int)((uint32_t)a / (uint32_t)b) : (int)(a / b);
}

// ALIGNED: units begin at multiples of their size in the sequence, so that the first may hold positions before `first`.
template <int UNIT, int COST, bool ALIGNED>
struct Split {
    const SplitParams &p;
    SplitShared &s;
    long long total, u, u_begin, u_end;
    int grid;
    bool small;

    // Positions [first, len) of sequence b; a length outside [0, max_len] is reported and clamped.
    __device__ __forceinline__ void live_range(int b, int &first, int &len) const
    {
        len = p.lens[b];
        if (len < 0 || len > p.max_len) {
            atomicOr(p.status, W4A16_DEV_LENGTH);
            len = len < 0 ? 0 : p.max_len;
        }
        first = p.window > 0 && len > p.window ? len - p.window : 0;
    }

    static __device__ __forceinline__ int start_of(int first) { return ALIGNED ? first / UNIT * UNIT : first; }

    __device__ __forceinline__ long long begin_of(int c) const
    {
        return small ? (long long)((uint32_t)(c * (uint32_t)total) / (uint32_t)grid) : c * total / grid;
    }

    __device__ __forceinline__ int owner_of(long long number) const
    {
        return split_quotient((number + 1) * grid - 1, total, small);
    }

    __device__ __forceinline__ bool empty(int b) const { return s.prefix[b + 1] == s.prefix[b]; }

    // Numbers the units; all threads of the block take part.
    __device__ __forceinline__ Split(const SplitParams &params, SplitShared &shared) : p(params), s(shared)
    {
        const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
        int run = 0;
        for (int base = 0; base < p.batch; base += SPLIT_THREADS) {
            const int b = base + tid;
            int n = 0;
            if (b < p.batch) {
                int first, len;
                live_range(b, first, len);
                n = (len - start_of(first) + UNIT - 1) / UNIT;
                n += n > 0 ? COST : 0;
            }
            int incl = n;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, incl, d);
                if (lane >= d)
                    incl += o;
            }
            if (lane == 31)
                s.warp_sum[warp] = incl;
            __syncthreads();
            int before = run;
#pragma unroll
            for (int w = 0; w < SPLIT_WARPS; ++w) {
                if (w < warp)
                    before += s.warp_sum[w];
                run += s.warp_sum[w];
            }
            if (b < p.batch)
                s.prefix[b] = before + incl - n;
            __syncthreads();
        }
        if (tid == 0)
            s.prefix[p.batch] = run;
        __syncthreads();
        total = (long long)run * p.rows_per_seq;
        grid = (int)min((long long)gridDim.x, total);
        small = total * (grid + 1LL) < (1LL << 32);
        u_begin = u_end = 0;
        if ((int)blockIdx.x < grid) {
            u_begin = begin_of(blockIdx.x);
            u_end = begin_of(blockIdx.x + 1);
        }
        u = u_begin;
    }

    // The block's next segment; false when it has none left.
    __device__ __forceinline__ bool next(SplitSegment &seg)
    {
        if (u >= u_end)
            return false;
        int lo = 0, hi = p.batch - 1; // last b with prefix[b] * rows_per_seq <= u
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if ((long long)s.prefix[mid] * p.rows_per_seq <= u)
                lo = mid;
            else
                hi = mid - 1;
        }
        seg.b = lo;
        const int span = s.prefix[lo + 1] - s.prefix[lo];
        seg.units = span - COST;
        const long long rem = u - (long long)s.prefix[lo] * p.rows_per_seq;
        seg.row = split_quotient(rem, span, small);
        seg.row_u0 = u - (rem - (long long)seg.row * span) + COST;
        seg.unit0 = (int)max(0LL, u - seg.row_u0);
        seg.unit1 = (int)min((long long)seg.units, u_end - seg.row_u0);
        u = seg.row_u0 + seg.units; // the row after this one
        seg.more = u < u_end;
        if (seg.unit1 <= seg.unit0)
            return false; // the range ends before the row's first unit
        live_range(lo, seg.first, seg.len);
        seg.start = start_of(seg.first);
        return true;
    }

    // Joins the warps' results and writes a row that is whole, or joins its parts if this block is the last to
    // arrive.  acc: shared [warp][HEADS][D] of sum p v, stat: shared [warp][HEADS] of (log2 maximum, sum p), filled and
    // synchronised; the first nh heads count.  `down` multiplies the outputs.  Ends synchronised when a segment may follow.
    template <int D, int HEADS, bool BF>
    __device__ __forceinline__ void finish(const SplitSegment &seg, const float *acc, const float *stat, int nh,
                                           uint16_t *out, float *lse, float down = 1.f)
    {
        const int tid = threadIdx.x;
        const bool whole = seg.unit1 - seg.unit0 == seg.units;
        const int slot = u_begin >= seg.row_u0 ? 0 : 1; // a block shares at most its first and its last row
        float *part = p.partials + ((long long)blockIdx.x * SPLIT_SLOTS + slot) * p.slot;
        for (int i = tid; i < nh * (D / 4); i += SPLIT_THREADS) {
            const int h = i / (D / 4), d = (i - h * (D / 4)) * 4;
            float mx = -INFINITY;
#pragma unroll
            for (int w = 0; w < SPLIT_WARPS; ++w)
                mx = fmaxf(mx, stat[(w * HEADS + h) * 2]);
            const float base = mx == -INFINITY ? 0.f : mx;
            float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
            float l = 0.f;
#pragma unroll
            for (int w = 0; w < SPLIT_WARPS; ++w) {
                const float f = exp2f(stat[(w * HEADS + h) * 2] - base);
                const float4 x = *reinterpret_cast<const float4 *>(acc + (w * HEADS + h) * D + d);
                l += f * stat[(w * HEADS + h) * 2 + 1];
                sum.x += f * x.x;
                sum.y += f * x.y;
                sum.z += f * x.z;
                sum.w += f * x.w;
            }
            if (whole) {
                const float r = l == 0.f ? 0.f : down / l;
                uint2 w2;
                w2.x = pack2<BF>(sum.x * r, sum.y * r);
                w2.y = pack2<BF>(sum.z * r, sum.w * r);
                *reinterpret_cast<uint2 *>(out + (long long)h * D + d) = w2;
                if (d == 0 && lse)
                    lse[h] = l == 0.f ? -INFINITY : fmaf(base, SPLIT_LN2, logf(l));
            } else {
                __stcg(reinterpret_cast<float4 *>(part + h * D + d), sum);
                if (d == 0)
                    __stcg(reinterpret_cast<float2 *>(part + HEADS * D + 2 * h), make_float2(mx, l));
            }
        }
        if (!whole)
            join<D, HEADS, BF>(seg, nh, out, lse, down);
        if (seg.more)
            __syncthreads(); // the shared results are read before the next segment fills their place
    }

    // The parts of a row are those of the blocks c_lo to c_hi, the owners of its first and its last unit.  The last
    // block to arrive joins them; where there are more than SPLIT_FAN, the last of every SPLIT_FAN of them joins
    // those first, so that many blocks share the reading.  A row's counter is that of its first block, in which no
    // other row of several parts starts; a group's likewise (a group of one part, which could share its block with
    // the next row's first, does not count).
    template <int D, int HEADS, bool BF>
    __device__ __forceinline__ void join(const SplitSegment &seg, int nh, uint16_t *out, float *lse, float down)
    {
        const int tid = threadIdx.x;
        const int c_lo = owner_of(seg.row_u0), c_hi = owner_of(seg.row_u0 + seg.units - 1);
        const int lo_slot = begin_of(c_lo) >= seg.row_u0 ? 0 : 1, parts = c_hi - c_lo + 1;
        const int group0 = ((int)blockIdx.x - c_lo) / SPLIT_FAN * SPLIT_FAN; // this block's group
        bool last_level = parts <= SPLIT_FAN;
        if (!last_level && group0 + 1 == parts)
            last_level = true; // a group of one part is read as it is
        for (;;) {
            // Joined here: a row's parts, a group of them, or a row's groups.
            const bool groups = last_level && parts > SPLIT_FAN;
            const int n = groups       ? (parts + SPLIT_FAN - 1) / SPLIT_FAN
                          : last_level ? parts
                                       : min(SPLIT_FAN, parts - group0);
            const int from = c_lo + (last_level ? 0 : group0);
            __syncthreads();
            if (tid == 0) {
                int *counter = last_level ? p.counters + c_lo : p.group_counters + from;
                const int last = arrive_counter(counter) == n - 1;
                if (last)
                    *counter = 0;
                s.is_last = last;
            }
            __syncthreads();
            if (!s.is_last)
                break;
            // A thread sums ITEMS quads of outputs over the parts in block order, the loads of AT parts in flight at
            // once (sixteen loads in all), rescaling as the maximum moves.
            auto sum_parts = [&](auto items_c, auto at_c) {
                constexpr int ITEMS = decltype(items_c)::value, AT = decltype(at_c)::value;
                const int quads = nh * (D / 4);
                for (int i0 = tid; i0 < quads; i0 += ITEMS * SPLIT_THREADS) {
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
                            const int at = groups ? (q0 + q) * SPLIT_FAN : q0 + q;
                            const int which = groups && at + 1 < parts ? SPLIT_SLOTS - 1 : from + at == c_lo ? lo_slot : 0;
                            const float *pp = p.partials + ((long long)(from + at) * SPLIT_SLOTS + which) * p.slot;
#pragma unroll
                            for (int k = 0; k < ITEMS; ++k) {
                                const int i = i0 + k * SPLIT_THREADS;
                                const bool in = q0 + q < n && i < quads;
                                ml[k][q] = in ? __ldcg(reinterpret_cast<const float2 *>(pp + HEADS * D) + i / (D / 4))
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
                        const int i = i0 + k * SPLIT_THREADS;
                        if (i >= quads)
                            continue;
                        const bool first_quad = i % (D / 4) == 0;
                        if (last_level) {
                            const float r = l[k] == 0.f ? 0.f : down / l[k];
                            uint2 w2;
                            w2.x = pack2<BF>(sum[k].x * r, sum[k].y * r);
                            w2.y = pack2<BF>(sum[k].z * r, sum[k].w * r);
                            *reinterpret_cast<uint2 *>(out + 4LL * i) = w2;
                            if (lse && first_quad)
                                lse[i / (D / 4)] = l[k] == 0.f ? -INFINITY : fmaf(m[k], SPLIT_LN2, logf(l[k]));
                        } else {
                            float *to = p.partials + ((long long)from * SPLIT_SLOTS + SPLIT_SLOTS - 1) * p.slot;
                            __stcg(reinterpret_cast<float4 *>(to) + i, sum[k]);
                            if (first_quad)
                                __stcg(reinterpret_cast<float2 *>(to + HEADS * D) + i / (D / 4), make_float2(m[k], l[k]));
                        }
                    }
                }
            };
            using std::integral_constant;
            if (n <= 4)
                sum_parts(integral_constant<int, 4>(), integral_constant<int, 4>());
            else if (n <= 8)
                sum_parts(integral_constant<int, 2>(), integral_constant<int, 8>());
            else
                sum_parts(integral_constant<int, 1>(), integral_constant<int, 16>());
            if (last_level)
                break;
            last_level = true;
        }
    }
};

} // namespace ops
} // namespace w4
