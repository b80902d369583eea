// w4a16_rope.cu -- rotary positions on q and k, and k and v written into a paged cache.
//
// For token t and pair i of the rotated part of a head (i < rot_dim / 2), with the axis a that the
// sections give to pair i and (c, s) = table[positions[a][t]][i], [rot_dim / 2 + i]:
//     (x1, x2) -> (x1 c - x2 s, x2 c + x1 s),
// where (x1, x2) are values i and rot_dim / 2 + i of the head, or 2 i and 2 i + 1 (adjacent pairs).
// The rest of a head is copied.  Two fp32 products and one fp32 sum per value, rounded once.
//
// Bound by memory: each value of q, k and v is read once and written once, with one row of the
// table per token and axis.  A thread looks after eight pairs of ROPE_HEADS heads: it keeps their
// cosines and sines in registers for both heads and walks over tokens, with the next token's values,
// position and slot on their way while it works on one, so that only the table's load waits for
// another (the position's).
#include "w4a16_ops.cuh"

namespace w4 {
namespace ops {

constexpr int ROPE_MAX_AXES = 4;
constexpr int ROPE_HEADS = 2;     // heads per thread (16-byte path)
constexpr int ROPE_THREADS = 128; // threads a block is filled up to
constexpr int ROPE_PER_SM = 768;  // threads per SM that a launch asks for and the registers allow

struct RopeParams {
    const uint16_t *q, *k, *v;
    uint16_t *q_out, *k_cache, *v_cache;
    const float *table;       // [max_pos][rot]: cosines, then sines
    const int32_t *positions; // [axes][ld_pos]
    const long long *slots;   // [tokens]
    int *status;
    long long page_stride, token_stride, head_stride, total_slots;
    int ldq, ldk, ldv, ldqo, ld_pos;
    int tokens, heads, kv, dim, rot, axes, max_pos, page;
    int cut[ROPE_MAX_AXES]; // pair i belongs to the first axis a with i < cut[a]
    int adjacent;
};

__device__ __forceinline__ void report(const RopeParams &p, int bit)
{
    if (p.status)
        atomicOr(p.status, bit);
}

__device__ __forceinline__ int axis_of(const RopeParams &p, int pair)
{
    int axis = 0;
#pragma unroll
    for (int a = 0; a < ROPE_MAX_AXES - 1; ++a)
        axis += (a < p.axes - 1 && pair >= p.cut[a]) ? 1 : 0;
    return axis;
}

// A position inside the table, or -1 after reporting it.
__device__ __forceinline__ int checked_position(const RopeParams &p, int pos)
{
    if (pos < 0 || pos >= p.max_pos) {
        report(p, W4A16_DEV_POSITION);
        return -1;
    }
    return pos;
}

__device__ __forceinline__ int position_of(const RopeParams &p, int token, int pair)
{
    return checked_position(p, p.positions[(long long)axis_of(p, pair) * p.ld_pos + token]);
}

// Element offset of a slot's cache row (head 0), or -1: a negative slot (not cached) or, after
// reporting it, one past the cache.
__device__ __forceinline__ long long cache_row(const RopeParams &p, long long slot)
{
    if (slot < 0)
        return -1;
    if (slot >= p.total_slots) {
        report(p, W4A16_DEV_SLOT);
        return -1;
    }
    const long long pg = p.total_slots < (1LL << 31) ? (long long)((uint32_t)slot / (uint32_t)p.page) : slot / p.page;
    return pg * p.page_stride + (slot - pg * p.page) * p.token_stride;
}

// Head h of the joint list (q heads, k heads, v heads): where it is read.
__device__ __forceinline__ const uint16_t *head_src(const RopeParams &p, int token, int h)
{
    if (h < p.heads)
        return p.q + (long long)token * p.ldq + (long long)h * p.dim;
    const int c = h - p.heads;
    return c < p.kv ? p.k + (long long)token * p.ldk + (long long)c * p.dim
                    : p.v + (long long)token * p.ldv + (long long)(c - p.kv) * p.dim;
}

// ... and where it is written (null: nowhere).
__device__ __forceinline__ uint16_t *head_dst(const RopeParams &p, int token, int h, long long row)
{
    if (h < p.heads)
        return p.q_out + (long long)token * p.ldqo + (long long)h * p.dim;
    const int c = h - p.heads;
    if (row < 0)
        return nullptr;
    return c < p.kv ? p.k_cache + row + c * p.head_stride : p.v_cache + row + (c - p.kv) * p.head_stride;
}

// 16-byte path: rows, strides and cache 16-byte aligned, dim and rot multiples of 16.  Item (chunk
// j, head group g) of a thread: chunk j < rot / 16 is eight pairs, a later one 16 values that are
// copied.  CUTS: some section ends inside a chunk (as a branch for
// every call it took 97 registers instead of 74, before the values were fetched ahead, and 43.9 us instead
// of 38.6 for the case below).
// 8191 tokens of 32 / 8 heads of 128 with three axes, bf16: 34.8 us, 5.9 TB/s of reads and writes
// (one head per thread 46 us, no values fetched ahead 39 us); one token: 2.0 us.
template <bool BF, bool CUTS>
__global__ void __launch_bounds__(256, ROPE_PER_SM / 256) rope_vec_kernel(const RopeParams p, int chunks, int items)
{
    pdl_wait();
    pdl_launch_dependents();
    const int item = blockIdx.y * blockDim.x + threadIdx.x;
    const int stride = gridDim.x * blockDim.y;
    int token = blockIdx.x * blockDim.y + threadIdx.y;
    if (item >= items || token >= p.tokens)
        return;
    const int all = p.heads + 2 * p.kv, half = p.rot / 2;
    const int g = item / chunks, j = item - g * chunks, h0 = g * ROPE_HEADS;
    // Values of the two 16-byte pieces: pairs (i, half + i), or 16 values in a row.
    const bool pairs = j < p.rot / 16 && h0 < all - p.kv;
    const bool halves = j < p.rot / 16 && !p.adjacent;
    const int at0 = halves ? 8 * j : 16 * j, at1 = halves ? half + 8 * j : 16 * j + 8;
    const bool cached = p.kv > 0 && h0 + ROPE_HEADS > p.heads;
    const int32_t *positions = p.positions + (long long)axis_of(p, 8 * j) * p.ld_pos;
    const int axis0 = axis_of(p, 8 * j), axis1 = CUTS && pairs ? axis_of(p, 8 * j + 7) : axis0;

    int next_pos = 0;
    long long next_slot = -1;
    uint4 n0[ROPE_HEADS], n1[ROPE_HEADS];
    auto fetch = [&](int t) {
#pragma unroll
        for (int n = 0; n < ROPE_HEADS; ++n)
            if (h0 + n < all) {
                const uint16_t *src = head_src(p, t, h0 + n);
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
        uint4 x0[ROPE_HEADS], x1[ROPE_HEADS];
#pragma unroll
        for (int n = 0; n < ROPE_HEADS; ++n) {
            x0[n] = n0[n];
            x1[n] = n1[n];
        }
        const int t = token, pos = pairs ? checked_position(p, next_pos) : 0;
        const long long row = cached ? cache_row(p, next_slot) : -1;
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
#pragma unroll
        for (int n = 0; n < ROPE_HEADS; ++n) {
            const int h = h0 + n;
            const bool turn = pairs && h < all - p.kv;
            uint16_t *dst = h < all && (known || !turn) ? head_dst(p, t, h, row) : nullptr;
            if (!dst)
                continue;
            if (turn) {
                uint32_t *w0 = reinterpret_cast<uint32_t *>(&x0[n]);
                uint32_t *w1 = reinterpret_cast<uint32_t *>(&x1[n]);
                if (p.adjacent) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 a = unpack2<BF>(w0[i]), b = unpack2<BF>(w1[i]);
                        w0[i] = pack2<BF>(a.x * c[i] - a.y * s[i], a.y * c[i] + a.x * s[i]);
                        w1[i] = pack2<BF>(b.x * c[4 + i] - b.y * s[4 + i], b.y * c[4 + i] + b.x * s[4 + i]);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 a = unpack2<BF>(w0[i]), b = unpack2<BF>(w1[i]);
                        const float c0 = c[2 * i], c1 = c[2 * i + 1], s0 = s[2 * i], s1 = s[2 * i + 1];
                        w0[i] = pack2<BF>(a.x * c0 - b.x * s0, a.y * c1 - b.y * s1);
                        w1[i] = pack2<BF>(b.x * c0 + a.x * s0, b.y * c1 + a.y * s1);
                    }
                }
            }
            *reinterpret_cast<uint4 *>(dst + at0) = x0[n];
            *reinterpret_cast<uint4 *>(dst + at1) = x1[n];
        }
        if (!more)
            return;
    }
}

// Any even rot, any dim, any strides: one pair (or two copied values) per thread and head, in 2-byte
// accesses.  Bound by their number.
template <bool BF>
__global__ void __launch_bounds__(256) rope_any_kernel(const RopeParams p)
{
    pdl_wait();
    pdl_launch_dependents();
    const int token = blockIdx.x;
    const int all = p.heads + 2 * p.kv, half = p.rot / 2;
    const int rest = p.dim - p.rot, items = half + (rest + 1) / 2;
    const long long row = p.kv > 0 ? cache_row(p, p.slots[token]) : -1;
    for (long long n = threadIdx.x; n < (long long)items * all; n += blockDim.x) {
        const int h = (int)(n / items), i = (int)(n - (long long)h * items);
        const uint16_t *src = head_src(p, token, h);
        uint16_t *dst = head_dst(p, token, h, row);
        const bool turn = h < all - p.kv;
        int pos = 0;
        if (turn && i < half)
            pos = position_of(p, token, i);
        if (!dst || pos < 0)
            continue;
        if (i < half) {
            const int a = p.adjacent ? 2 * i : i, b = p.adjacent ? 2 * i + 1 : half + i;
            uint16_t ra = src[a], rb = src[b];
            if (turn) {
                const float c = p.table[(long long)pos * p.rot + i], s = p.table[(long long)pos * p.rot + half + i];
                const float x = to_float<BF>(ra), y = to_float<BF>(rb);
                ra = from_float<BF>(x * c - y * s);
                rb = from_float<BF>(y * c + x * s);
            }
            dst[a] = ra;
            dst[b] = rb;
        } else {
            const int a = p.rot + 2 * (i - half);
            dst[a] = src[a];
            if (a + 1 < p.dim)
                dst[a + 1] = src[a + 1];
        }
    }
}

} // namespace ops
} // namespace w4

using namespace w4;
using namespace w4::ops;

extern "C" int w4a16_rope_append(const void *q, int ldq, const void *k, int ldk, const void *v, int ldv,
                                 void *q_out, int ldqo, void *k_cache, void *v_cache,
                                 long long kv_page_stride, long long kv_token_stride,
                                 long long kv_head_stride, const float *cos_sin, int max_pos,
                                 const int32_t *positions, int ld_pos, const long long *slots,
                                 int32_t *status, int n_tokens, int n_heads, int n_kv_heads,
                                 int head_dim, int rot_dim, const int32_t *sections, int n_axes,
                                 int page_size, int n_pages, unsigned flags, cudaStream_t stream)
{
    if (flags & ~(W4A16_FLAG_BF16 | W4A16_FLAG_ROPE_ADJACENT))
        return status_of(STAGE_ARG, W4A16_ARG_FLAGS);
    if (n_tokens < 0 || n_heads < 0 || n_kv_heads < 0 || n_heads + (long long)n_kv_heads <= 0 ||
        head_dim <= 0 || rot_dim <= 0 || rot_dim % 2 != 0 || rot_dim > head_dim || max_pos <= 0 ||
        n_axes <= 0 || n_axes > ROPE_MAX_AXES || (n_kv_heads > 0 && (page_size <= 0 || n_pages <= 0)))
        return status_of(STAGE_ARG, W4A16_ARG_SHAPE);
    if (!sections)
        return status_of(STAGE_ARG, W4A16_ARG_NULL);
    long long sum = 0;
    for (int a = 0; a < n_axes; ++a) {
        if (sections[a] < 0)
            return status_of(STAGE_ARG, W4A16_ARG_SHAPE);
        sum += sections[a];
    }
    if (sum != rot_dim / 2)
        return status_of(STAGE_ARG, W4A16_ARG_SHAPE);
    if (n_tokens == 0)
        return 0;
    if (!cos_sin || !positions || (n_heads > 0 && (!q || !q_out)) ||
        (n_kv_heads > 0 && (!k || !v || !k_cache || !v_cache || !slots)))
        return status_of(STAGE_ARG, W4A16_ARG_NULL);
    if (n_heads == 0) // what absent heads would use is not looked at, its alignment included
        q = nullptr, q_out = nullptr;
    if (n_kv_heads == 0)
        k = nullptr, v = nullptr, k_cache = nullptr, v_cache = nullptr, slots = nullptr;
    const long long qw = (long long)n_heads * head_dim, kw = (long long)n_kv_heads * head_dim;
    if (qw > 0x7FFFFFFFLL || kw > 0x7FFFFFFFLL || (long long)n_heads + 2LL * n_kv_heads > (1 << 20))
        return status_of(STAGE_ARG, W4A16_ARG_OVERFLOW);
    if (ldq < qw || ldqo < qw || ldk < kw || ldv < kw || ld_pos < n_tokens ||
        (n_kv_heads > 0 && (kv_page_stride < 0 || kv_token_stride < 0 || kv_head_stride < 0)))
        return status_of(STAGE_ARG, W4A16_ARG_SHAPE);
    if (!aligned(q, 2) || !aligned(k, 2) || !aligned(v, 2) || !aligned(q_out, 2) || !aligned(k_cache, 2) ||
        !aligned(v_cache, 2) || !aligned(cos_sin, 4) || !aligned(positions, 4) || !aligned(slots, 8) ||
        !aligned(status, 4))
        return status_of(STAGE_ARG, W4A16_ARG_ALIGN);

    RopeParams p;
    p.q = static_cast<const uint16_t *>(q);
    p.k = static_cast<const uint16_t *>(k);
    p.v = static_cast<const uint16_t *>(v);
    p.q_out = static_cast<uint16_t *>(q_out);
    p.k_cache = static_cast<uint16_t *>(k_cache);
    p.v_cache = static_cast<uint16_t *>(v_cache);
    p.table = cos_sin;
    p.positions = positions;
    p.slots = slots;
    p.status = status;
    p.page_stride = kv_page_stride;
    p.token_stride = kv_token_stride;
    p.head_stride = kv_head_stride;
    p.total_slots = (long long)n_pages * page_size;
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
    int cut = 0;
    for (int a = 0; a < ROPE_MAX_AXES; ++a) {
        if (a < n_axes)
            cut += sections[a];
        p.cut[a] = cut;
    }
    const bool bf = (flags & W4A16_FLAG_BF16) != 0;
    const long long any = (n_heads ? (long long)(ldq | ldqo) : 0) |
                          (n_kv_heads ? (ldk | ldv | kv_page_stride | kv_token_stride | kv_head_stride) : 0);
    const bool vec = head_dim % 16 == 0 && rot_dim % 16 == 0 && any % 8 == 0 && aligned(q, 16) &&
                     aligned(k, 16) && aligned(v, 16) && aligned(q_out, 16) && aligned(k_cache, 16) &&
                     aligned(v_cache, 16) && aligned(cos_sin, 16);
    if (vec) {
        const int all = n_heads + 2 * n_kv_heads;
        const int chunks = head_dim / 16;
        const long long items = (long long)chunks * ((all + ROPE_HEADS - 1) / ROPE_HEADS);
        // Blocks of whole tokens up to ROPE_THREADS; wider tokens take blocks of their own side by side.
        const int bx = items < 256 ? (int)items : 256;
        const long long side = (items + bx - 1) / bx;
        if (side > 65535)
            return status_of(STAGE_ARG, W4A16_ARG_OVERFLOW);
        int by = ROPE_THREADS / bx;
        by = by < 1 ? 1 : by > n_tokens ? n_tokens : by;
        int num_sms = 0;
        const cudaError_t err = sm_count(&num_sms);
        if (err != cudaSuccess)
            return status_of(STAGE_RESOURCE, err);
        const long long groups = (n_tokens + (long long)by - 1) / by;
        long long blocks = (long long)num_sms * (ROPE_PER_SM / (bx * by)) / side;
        blocks = blocks < 1 ? 1 : blocks > groups ? groups : blocks;
        const dim3 grid((unsigned)blocks, (unsigned)side), block(bx, by);
        bool cuts = false;
        for (int a = 0; a < n_axes - 1; ++a)
            cuts |= p.cut[a] % 8 != 0;
        const auto kernel = bf ? (cuts ? rope_vec_kernel<true, true> : rope_vec_kernel<true, false>)
                               : (cuts ? rope_vec_kernel<false, true> : rope_vec_kernel<false, false>);
        return launch_status(launch_pdl(kernel, grid, block, 0, stream, p, chunks, (int)items));
    }
    const dim3 grid((unsigned)n_tokens), block(256);
    return launch_status(bf ? launch_pdl(rope_any_kernel<true>, grid, block, 0, stream, p)
                            : launch_pdl(rope_any_kernel<false>, grid, block, 0, stream, p));
}
