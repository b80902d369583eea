// w4a16_sample.cu -- the next token of each row of logits by temperature, top-k, top-p and min-p.
//
// With P_i = e^((l_i - max l) / T), tokens ordered by (logit falling, index rising):
//     top-k keeps the first k; top-p, of these, the shortest beginning whose sum reaches top_p times their sum;
//     min-p, of these, those with P_i >= min_p;
//     token = the first index i at which the sum of the kept P_j, j <= i, exceeds u times the sum of all kept.
// The kept tokens are those above a threshold logit and, of those at it, the first r by index.
//
// Where sums decide (which token's share holds u, where top-p ends), rounding would show: P is therefore a 64-bit
// integer, a multiple of 2^-43 good to 2^-30 of itself, and all sums are exact, in whatever order they are
// taken.  So results do not depend on the split, and atomics do no harm.  P comes from a table of 2^(-j/256) and a
// polynomial for the rest (the table-driven exponential of Tang, 1989); (l - max) / T is kept in two fp32 parts.
//
// A cluster of up to eight blocks holds a row: the logits are read from memory once, as 16-bit keys in their order, and
// stay in shared memory.  The threshold is found by the keys' high bytes and then the low bytes of one of them (256-bin
// histograms of counts and sums); blocks read one another's bins.  With top_k up to 128 only keys not below the k-th
// largest of the threads' largest ones can matter, which are few: they are gathered into one block, which decides.
// Where neither top-k nor top-p nor min-p limits a row there is no histogram.  Last, each warp sums its own range of
// indices, and the warp whose range holds u walks it; below the threshold no P is computed.
//
// What bounds it: for few rows the chain of cluster barriers, for many the instructions: 62 per logit where nothing limits a
// row (about thirty of them for its P, the rest for keys, votes and sums), 47 per logit where nine tenths are masked.
// Measured (device): one row of 32000 7.5 us; 48 x 131071 with all kinds of limits 42 (a row with top-p alone takes
// about 22 by itself: a P and the histogram's atomics for each logit); 32 x 256000 without limits 31.5; 256 x 100003
// nine tenths masked 84, 7 us of which the reading would take.  64-bit atomics in the histogram instead of three of 32
// bits: 96 for the second; 256 or 1024 threads: slower.
#include <cooperative_groups.h>

#include "w4a16_ops.cuh"

namespace w4 {
namespace ops {

namespace cg = cooperative_groups;

constexpr int SAMPLE_THREADS = 512;
constexpr int SAMPLE_WARPS = SAMPLE_THREADS / 32;
constexpr int SAMPLE_CLUSTER = 8;      // blocks of a row, at most
constexpr int SAMPLE_SLICE = 65536;    // logits of a block, at most: 128 KiB of keys
constexpr int SAMPLE_BITS = 43;        // P = 1 is 2^43: 2^19 tokens sum below 2^62
constexpr int SAMPLE_COPIES = 4;       // of a histogram, against lanes that meet at a bin
constexpr int SAMPLE_TABLE = 256;
constexpr int SAMPLE_SPARSE = 4;       // of eight logits, up to which a warp takes them one by one
constexpr int SAMPLE_FEW = 128;        // top_k up to which the tokens in question are gathered in one block
constexpr int SAMPLE_LIST = 1024;      // of these, at most
constexpr float SAMPLE_ROUND = 12582912.f; // rounds what is added to it to integers (ties to even), in its lowest bits
constexpr uint32_t SAMPLE_ROUND_BITS = 0x4B400000u;
constexpr float SAMPLE_HOTTEST = 0x1p100f;  // temperature, at most
constexpr float SAMPLE_COLDEST = 0x1p-126f; // what temperatures below count as (log2(e) / T is then still in fp32)

// 2^31 2^(-j/256).
__device__ const uint32_t SAMPLE_EXP[SAMPLE_TABLE] = {
    2147483648u, 2141676973u, 2135885998u, 2130110682u, 2124350982u, 2118606857u, 2112878262u, 2107165158u,
    2101467502u, 2095785251u, 2090118366u, 2084466803u, 2078830522u, 2073209480u, 2067603638u, 2062012954u,
    2056437387u, 2050876895u, 2045331439u, 2039800978u, 2034285470u, 2028784876u, 2023299156u, 2017828268u,
    2012372174u, 2006930832u, 2001504204u, 1996092249u, 1990694927u, 1985312200u, 1979944027u, 1974590370u,
    1969251188u, 1963926443u, 1958616096u, 1953320108u, 1948038440u, 1942771053u, 1937517909u, 1932278970u,
    1927054196u, 1921843549u, 1916646992u, 1911464486u, 1906295993u, 1901141476u, 1896000896u, 1890874216u,
    1885761398u, 1880662405u, 1875577199u, 1870505744u, 1865448001u, 1860403934u, 1855373507u, 1850356681u,
    1845353420u, 1840363688u, 1835387448u, 1830424663u, 1825475297u, 1820539314u, 1815616678u, 1810707353u,
    1805811301u, 1800928489u, 1796058879u, 1791202437u, 1786359126u, 1781528911u, 1776711757u, 1771907628u,
    1767116489u, 1762338305u, 1757573041u, 1752820662u, 1748081133u, 1743354420u, 1738640488u, 1733939301u,
    1729250827u, 1724575029u, 1719911875u, 1715261330u, 1710623359u, 1705997930u, 1701385007u, 1696784557u,
    1692196547u, 1687620943u, 1683057710u, 1678506817u, 1673968228u, 1669441912u, 1664927835u, 1660425963u,
    1655936265u, 1651458706u, 1646993254u, 1642539877u, 1638098541u, 1633669214u, 1629251865u, 1624846459u,
    1620452965u, 1616071351u, 1611701585u, 1607343634u, 1602997467u, 1598663052u, 1594340357u, 1590029350u,
    1585730000u, 1581442275u, 1577166143u, 1572901575u, 1568648537u, 1564406999u, 1560176931u, 1555958300u,
    1551751076u, 1547555228u, 1543370725u, 1539197537u, 1535035634u, 1530884983u, 1526745556u, 1522617322u,
    1518500250u, 1514394310u, 1510299473u, 1506215708u, 1502142985u, 1498081275u, 1494030547u, 1489990772u,
    1485961921u, 1481943963u, 1477936870u, 1473940611u, 1469955159u, 1465980482u, 1462016553u, 1458063343u,
    1454120821u, 1450188960u, 1446267730u, 1442357104u, 1438457051u, 1434567544u, 1430688553u, 1426820052u,
    1422962010u, 1419114401u, 1415277195u, 1411450365u, 1407633882u, 1403827719u, 1400031848u, 1396246240u,
    1392470869u, 1388705706u, 1384950723u, 1381205894u, 1377471191u, 1373746586u, 1370032052u, 1366327563u,
    1362633090u, 1358948606u, 1355274085u, 1351609500u, 1347954824u, 1344310030u, 1340675091u, 1337049980u,
    1333434672u, 1329829140u, 1326233356u, 1322647296u, 1319070932u, 1315504238u, 1311947188u, 1308399756u,
    1304861917u, 1301333643u, 1297814910u, 1294305692u, 1290805962u, 1287315695u, 1283834865u, 1280363448u,
    1276901417u, 1273448747u, 1270005413u, 1266571390u, 1263146652u, 1259731174u, 1256324931u, 1252927899u,
    1249540052u, 1246161366u, 1242791816u, 1239431376u, 1236080024u, 1232737732u, 1229404479u, 1226080238u,
    1222764986u, 1219458698u, 1216161350u, 1212872918u, 1209593378u, 1206322705u, 1203060876u, 1199807867u,
    1196563654u, 1193328213u, 1190101520u, 1186883552u, 1183674286u, 1180473697u, 1177281762u, 1174098458u,
    1170923762u, 1167757650u, 1164600099u, 1161451085u, 1158310587u, 1155178580u, 1152055042u, 1148939949u,
    1145833280u, 1142735011u, 1139645120u, 1136563583u, 1133490379u, 1130425485u, 1127368878u, 1124320536u,
    1121280436u, 1118248556u, 1115224875u, 1112209370u, 1109202018u, 1106202798u, 1103211687u, 1100228665u,
    1097253708u, 1094286796u, 1091327906u, 1088377016u, 1085434106u, 1082499153u, 1079572136u, 1076653033u,
};

struct SampleParams {
    const uint16_t *logits;
    const float *uniform, *temperature, *top_p, *min_p;
    const int32_t *top_k;
    int32_t *tokens, *status;
    float *logprobs;
    long long ld;
    int vocab, slice;
    int wide; // rows can be read 16 bytes at a time
};

struct SampleShared {
    uint2 exp[SAMPLE_TABLE]; // 2^31 2^(-j/256) as an integer (less SAMPLE_ROUND_BITS) and as a number
    uint32_t count[256 * SAMPLE_COPIES], low[256 * SAMPLE_COPIES], high[256 * SAMPLE_COPIES];
    // This block's bins, read by the cluster's other blocks; two sets in turn, so that a set is written again only
    // after a barrier which all of its readers have reached.
    unsigned long long bin_sum[2][256];
    uint32_t bin_count[2][256];
    unsigned long long all_sum[256]; // of all blocks: the last histogram that asked for them
    uint32_t all_count[256];
    // Written by every block of the cluster.
    uint32_t top[SAMPLE_CLUSTER], bound[SAMPLE_CLUSTER], listed_by[SAMPLE_CLUSTER];
    unsigned long long above[SAMPLE_CLUSTER];
    uint32_t ties[SAMPLE_CLUSTER];
    // Of this block's warps.
    uint32_t warp_top[SAMPLE_WARPS];
    unsigned long long warp_above[SAMPLE_WARPS];
    uint32_t warp_ties[SAMPLE_WARPS];
    // A search's result, and its sums by warp.
    unsigned long long found_above, found_other, total, total_other;
    unsigned long long of_warp[8], other_of_warp[8];
    // Tokens in question, key << 32 | ~index, so that the better one is larger: of this block, then (block 0) of all; the
    // kept ones of these, and their P.
    unsigned long long list[SAMPLE_LIST], gathered[SAMPLE_LIST], kept[SAMPLE_FEW], kept_share[SAMPLE_FEW];
    uint32_t listed, place, n_gathered, n_kept; // (n_gathered: block 0's)
    uint32_t found;
};

// 0xFFFF for each half whose highest bit is set.
__device__ __forceinline__ uint32_t signs(uint32_t w)
{
    uint32_t r;
    asm("prmt.b32 %0, %1, 0, 0xBB99;" : "=r"(r) : "r"(w));
    return r;
}

// 16-bit numbers as integers in the same order, two at a time; -0 counts as 0.
__device__ __forceinline__ uint32_t keys_of(uint32_t w)
{
    const uint32_t size = w & 0x7FFF7FFFu;
    w = size | (w & (size + 0x7FFF7FFFu) & 0x80008000u); // no sign without a size
    return w ^ (signs(w) | 0x80008000u);
}

// Whether one of eight numbers is a NaN; and these as -inf.
template <bool BF>
__device__ __forceinline__ bool has_nan(const uint4 &w)
{
    constexpr uint32_t ABOVE = BF ? 0x007F007Fu : 0x03FF03FFu; // what takes the size of a NaN to the sign's place
    const uint32_t any = ((w.x & 0x7FFF7FFFu) + ABOVE) | ((w.y & 0x7FFF7FFFu) + ABOVE) | ((w.z & 0x7FFF7FFFu) + ABOVE) |
                         ((w.w & 0x7FFF7FFFu) + ABOVE);
    return (any & 0x80008000u) != 0;
}

template <bool BF>
__device__ __forceinline__ uint32_t without_nan(uint32_t w)
{
    const uint32_t nan = signs((w & 0x7FFF7FFFu) + (BF ? 0x007F007Fu : 0x03FF03FFu));
    return (w & ~nan) | ((BF ? 0xFF80FF80u : 0xFC00FC00u) & nan);
}

// Two keys' numbers.
template <bool BF>
__device__ __forceinline__ float2 numbers_of(uint32_t keys)
{
    const uint32_t w = keys ^ (~signs(keys) | 0x80008000u);
    return BF ? make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)) : unpack2<BF>(w);
}

template <bool BF>
__device__ __forceinline__ constexpr uint32_t lowest_key() // of -inf
{
    return BF ? 0x007Fu : 0x03FFu;
}

// Eight keys of -inf: what lies past a slice.
template <bool BF>
__device__ __forceinline__ uint4 no_keys()
{
    constexpr uint32_t TWO = lowest_key<BF>() * 0x10001u;
    return make_uint4(TWO, TWO, TWO, TWO);
}

// P of logits, in units of 2^-43.
template <bool BF>
struct Share {
    float top, c_hi, c_lo; // the largest logit (finite); log2(e) / T in two parts
    const uint2 *exp;

    // 2^-y, y = n + j / 256 + a rest: kk holds n and j, z the rest times ln 2 (at most ln 2 / 512), fine: y < 44.5.
    __device__ __forceinline__ unsigned long long scaled(float kk, float z, bool fine) const
    {
        const uint32_t k = __float_as_uint(kk) - SAMPLE_ROUND_BITS;
        const uint2 e = exp[k & (SAMPLE_TABLE - 1)];
        const float q = z * fmaf(z, fmaf(z, -1.f / 6.f, 0.5f), -1.f); // e^-z - 1, to z^4 / 24 < 2^-42
        const uint32_t v = e.x + __float_as_uint(fmaf(__uint_as_float(e.y), q, SAMPLE_ROUND)); // 2^31 2^(n - y)
        const uint32_t n = k / SAMPLE_TABLE;
        // v 2^(12 - n): by a product, which where that is a shift to the right lies 32 bits higher, to be rounded.
        const bool small = n > 12;
        const unsigned long long r = (unsigned long long)v * (1u << ((12 - n) & 31)) + (small ? 0x80000000u : 0u);
        return !fine ? 0 : small ? r >> 32 : r;
    }

    __device__ __forceinline__ void operator()(uint32_t keys, unsigned long long &first, unsigned long long &second) const
    {
        const float2 l = numbers_of<BF>(keys), t = both(top);
        // d + rest is the difference, exactly, whichever of the two is the larger one in size.
        const float2 d = sub(t, l), minus = sub(d, t), rest = sub(sub(t, sub(d, minus)), add(l, minus));
        const float2 y = mul(d, both(c_hi));
        const float2 y_lo = add(fma(d, both(c_hi), make_float2(-y.x, -y.y)), fma(d, both(c_lo), mul(rest, both(c_hi))));
        const float2 kk = fma(y, both((float)SAMPLE_TABLE), both(SAMPLE_ROUND)), k = add(kk, both(-SAMPLE_ROUND));
        const float2 z = mul(add(fma(k, both(-1.f / SAMPLE_TABLE), y), y_lo), both(0.6931471805599453f));
        first = scaled(kk.x, z.x, y.x < 44.5f);
        second = scaled(kk.y, z.y, y.y < 44.5f);
    }

    __device__ __forceinline__ unsigned long long operator()(uint32_t key) const
    {
        unsigned long long p, ignored;
        (*this)(key * 0x10001u, p, ignored);
        return p;
    }
};

// A number in [0, 1) as a multiple of 2^-64, cut off (0 for those below 0).
__device__ __forceinline__ unsigned long long fraction(float x)
{
    const uint32_t bits = __float_as_uint(x);
    const int e = (int)(bits >> 23);
    const unsigned long long m = (bits & 0x7FFFFFu) | 0x800000u; // x = m 2^(e - 150)
    return !(x > 0.f) || e <= 86 - 24 ? 0 : e >= 86 ? m << min(e - 86, 40) : m >> (86 - e);
}

// log(part / all), near 1 by what is missing.
__device__ __forceinline__ float log_share(unsigned long long part, unsigned long long all)
{
    return part > all / 2 ? log1pf(-((float)(all - part) / (float)all)) : logf((float)part / (float)all);
}

// Adds `sum` to a bin's 64-bit sum of two 32-bit halves: the high one and the carry, when the low one was `old`; or all.
__device__ __forceinline__ void add_carry(uint32_t *high, unsigned long long sum, uint32_t old)
{
    const uint32_t carry = (uint32_t)(sum >> 32) + (old + (uint32_t)sum < old ? 1u : 0u);
    if (carry)
        atomicAdd(high, carry);
}

__device__ __forceinline__ void add_sum(uint32_t *low, uint32_t *high, unsigned long long sum)
{
    add_carry(high, sum, atomicAdd(low, (uint32_t)sum));
}

// Which of eight keys are at least `least`, a bit each.
__device__ __forceinline__ uint32_t at_least(const uint32_t (&w)[4], uint32_t least)
{
    uint32_t which = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        which |= (w[e] << 16 >= least << 16 ? 1u : 0u) << (2 * e) | (w[e] >= least << 16 ? 2u : 0u) << (2 * e);
    return which;
}

// Key e of eight, e not known before.
__device__ __forceinline__ uint32_t pick(const uint32_t (&w)[4], int e)
{
    const uint32_t pair = e & 4 ? (e & 2 ? w[3] : w[2]) : (e & 2 ? w[1] : w[0]);
    return e & 1 ? pair >> 16 : pair & 0xFFFFu;
}

// Whether some lane's eight keys are all at least `least`, or more than SAMPLE_SPARSE of them; if not, `which` of them are.
// All lanes of a warp take part.
__device__ __forceinline__ bool dense(const uint4 &k, uint32_t least, uint32_t &which)
{
    const uint32_t m = __vminu2(__vminu2(k.x, k.y), __vminu2(k.z, k.w));
    which = 0;
    if (__any_sync(0xffffffffu, min(m & 0xFFFFu, m >> 16) >= least))
        return true;
    const uint32_t w[4] = {k.x, k.y, k.z, k.w};
    which = at_least(w, least);
    return __any_sync(0xffffffffu, __popc(which) > SAMPLE_SPARSE);
}

// The largest of eight keys.
__device__ __forceinline__ uint32_t largest(const uint4 &k)
{
    const uint32_t m = __vmaxu2(__vmaxu2(k.x, k.y), __vmaxu2(k.z, k.w));
    return max(m & 0xFFFFu, m >> 16);
}

// The highest bin which, with `before` and the bins above it, has at least `want` of a measure: `weight` is that of bin
// 255 - thread.  Leaves the bin in found (256: there is not as much), what lies above it in found_above (with `before`),
// and the sum of `other` above it in found_other; total and total_other are those of all bins.
__device__ __noinline__ void find(SampleShared &s, unsigned long long weight, unsigned long long other,
                                  unsigned long long before, unsigned long long want)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    unsigned long long incl = weight, incl2 = other;
    if (tid < 256) {
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const unsigned long long o = __shfl_up_sync(0xffffffffu, incl, d), o2 = __shfl_up_sync(0xffffffffu, incl2, d);
            if (lane >= d) {
                incl += o;
                incl2 += o2;
            }
        }
        if (lane == 31) {
            s.of_warp[warp] = incl;
            s.other_of_warp[warp] = incl2;
        }
        if (tid == 0)
            s.found = 256;
    }
    __syncthreads();
    if (tid < 256) {
#pragma unroll
        for (int w = 0; w < 8; ++w)
            if (w < warp) {
                incl += s.of_warp[w];
                incl2 += s.other_of_warp[w];
            }
        if (tid == 255) {
            s.total = incl;
            s.total_other = incl2;
        }
        incl += before;
        if (incl >= want && incl - weight < want) {
            s.found = 255 - tid;
            s.found_above = incl - weight;
            s.found_other = incl2 - other;
        }
    }
    __syncthreads();
}

template <bool BF>
struct Sampler {
    SampleShared &s;
    const uint4 *keys; // the slice, eight keys at a time
    int vectors;       // of them
    cg::cluster_group cluster;
    Share<BF> share;

    int histograms;    // made so far

    __device__ __forceinline__ void clear(bool sums)
    {
        for (int i = threadIdx.x; i < 256 * SAMPLE_COPIES; i += SAMPLE_THREADS) {
            s.count[i] = 0;
            if (sums)
                s.low[i] = s.high[i] = 0;
        }
        __syncthreads();
    }

    // Merges the bins over copies and blocks into all_count and all_sum.
    __device__ __forceinline__ void merge(bool counts, bool sums)
    {
        const int tid = threadIdx.x, set = histograms++ & 1;
        __syncthreads();
        if (tid < 256) {
            uint32_t n = 0;
            unsigned long long sum = 0;
#pragma unroll
            for (int c = 0; c < SAMPLE_COPIES; ++c) {
                n += s.count[tid * SAMPLE_COPIES + c];
                if (sums)
                    sum += s.low[tid * SAMPLE_COPIES + c] + ((unsigned long long)s.high[tid * SAMPLE_COPIES + c] << 32);
            }
            s.bin_count[set][tid] = n;
            s.bin_sum[set][tid] = sum;
        }
        cluster.sync();
        if (tid < 256) {
            uint32_t n = 0;
            unsigned long long sum = 0;
            const unsigned blocks = cluster.num_blocks();
#pragma unroll
            for (unsigned r = 0; r < SAMPLE_CLUSTER; ++r)
                if (r < blocks) {
                    n += counts ? *cluster.map_shared_rank(&s.bin_count[set][tid], r) : 0;
                    sum += sums ? *cluster.map_shared_rank(&s.bin_sum[set][tid], r) : 0;
                }
            if (counts)
                s.all_count[tid] = n;
            if (sums)
                s.all_sum[tid] = sum;
        }
        __syncthreads();
    }

    // Histogram of the keys by high bytes: of counts, and of sums.
    __device__ __forceinline__ void coarse(bool counts, bool sums)
    {
        const int copy = threadIdx.x % SAMPLE_COPIES;
        constexpr uint32_t least = lowest_key<BF>() + 1;
        clear(sums);
        for (int first = threadIdx.x & ~31; first < vectors; first += SAMPLE_THREADS) { // (the same turns in all lanes)
            const int v = first + (threadIdx.x & 31);
            const uint4 k4 = v < vectors ? keys[v] : no_keys<BF>();
            const uint32_t w[4] = {k4.x, k4.y, k4.z, k4.w};
            uint32_t which;
            if (!dense(k4, least, which)) { // most are masked: the others one by one
                while (which) {
                    const uint32_t key = pick(w, __ffs(which) - 1), at = (key >> 8) * SAMPLE_COPIES + copy;
                    which &= which - 1;
                    if (counts)
                        atomicAdd(&s.count[at], 1u);
                    const unsigned long long x = sums ? share(key) : 0;
                    if (x)
                        add_sum(&s.low[at], &s.high[at], x);
                }
                continue;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t key[2] = {w[e] & 0xFFFFu, w[e] >> 16};
                const uint32_t at[2] = {(key[0] >> 8) * SAMPLE_COPIES + copy, (key[1] >> 8) * SAMPLE_COPIES + copy};
                if (counts) {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (key[i] >= least)
                            atomicAdd(&s.count[at[i]], 1u);
                }
                if (sums) { // both low halves before the carries, which wait for them
                    unsigned long long x[2];
                    uint32_t old[2] = {0, 0};
                    share(w[e], x[0], x[1]); // (0 for -inf)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if ((uint32_t)x[i])
                            old[i] = atomicAdd(&s.low[at[i]], (uint32_t)x[i]);
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        add_carry(&s.high[at[i]], x[i], old[i]);
                }
            }
        }
        merge(counts, sums);
    }

    // Histogram of the low bytes of the keys with high byte `byte`.
    __device__ __forceinline__ void fine(uint32_t byte)
    {
        const int copy = threadIdx.x % SAMPLE_COPIES;
        clear(false);
        for (int v = threadIdx.x; v < vectors; v += SAMPLE_THREADS) {
            const uint4 k4 = keys[v];
            if (largest(k4) >> 8 < byte)
                continue;
            const uint32_t w[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t key = (w[e >> 1] >> (16 * (e & 1))) & 0xFFFFu;
                if (key >> 8 == byte && key > lowest_key<BF>())
                    atomicAdd(&s.count[(key & 255) * SAMPLE_COPIES + copy], 1u);
            }
        }
        merge(true, false);
    }

    // find() over weigh(bin), with other(bin).
    template <class Weigh, class Other>
    __device__ __forceinline__ void search(unsigned long long before, unsigned long long want, Weigh weigh, Other other)
    {
        const int bin = 255 - (int)threadIdx.x;
        find(s, bin >= 0 ? weigh(bin) : 0, bin >= 0 ? other(bin) : 0, before, want);
    }

    // The token of a row of which top-k keeps a few, in block 0: `n` candidates lie in s.gathered, the kept ones among
    // them; their keys are from `low` to `high`.
    __device__ __forceinline__ void choose(int n, uint32_t low, uint32_t high, int top_k, float top_p, unsigned long long least,
                                           float u, int32_t *token, float *logprob)
    {
        const int tid = threadIdx.x;
        static_assert(SAMPLE_LIST == 2 * SAMPLE_THREADS && SAMPLE_FEW <= SAMPLE_THREADS, "two candidates a thread");
        const unsigned long long mine[2] = {tid < n ? s.gathered[tid] : 0,
                                            tid + SAMPLE_THREADS < n ? s.gathered[tid + SAMPLE_THREADS] : 0};
        const uint32_t key[2] = {(uint32_t)(mine[0] >> 32), (uint32_t)(mine[1] >> 32)};
        if (tid < SAMPLE_FEW)
            s.kept[tid] = s.kept_share[tid] = 0;
        if (tid == 0)
            s.n_kept = 0;
        // The top_k-th key or one with which as many are kept (0: all are), and how many of it are where not all are.
        uint32_t last = 0;
        int ties = 0;
        bool all_ties = true;
        __syncthreads();
        if (n > top_k) {
            auto count = [&](uint32_t at) { // of keys of at least `at`
                return __syncthreads_count(key[0] >= at) + (n > SAMPLE_THREADS ? __syncthreads_count(key[1] >= at) : 0);
            };
            uint32_t bit = low == high ? 0 : 1u << (31 - __clz(low ^ high)); // the first in which keys differ
            last = bit ? low & ~(2 * bit - 1) : low;
#pragma unroll 1
            for (all_ties = false; bit && !all_ties; bit >>= 1) {
                const int n_at = count(last | bit);
                if (n_at >= top_k)
                    last |= bit;
                all_ties = n_at == top_k; // (`last` then lies between the top_k-th key and the next one)
            }
            if (!all_ties)
                ties = top_k - count(last + 1);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            bool keep = mine[i] != 0 && key[i] >= last;
            if (keep && key[i] == last && !all_ties) {
                int better = 0; // ties of a lower index
                for (int j = 0; j < n; ++j) {
                    const unsigned long long o = s.gathered[j];
                    better += (uint32_t)(o >> 32) == last && o > mine[i];
                }
                keep = better < ties;
            }
            if (keep)
                s.kept[atomicAdd(&s.n_kept, 1u)] = mine[i];
        }
        __syncthreads();
        // A thread each for the kept ones: the other warps leave.
        if (tid >= SAMPLE_FEW)
            return;
        const auto sync = [] { asm volatile("bar.sync 1, %0;" ::"n"(SAMPLE_FEW) : "memory"); };
        const int kept = (int)s.n_kept;
        const unsigned long long me = s.kept[tid], x = tid < kept ? share((uint32_t)(me >> 32)) : 0;
        bool stays = tid < kept && x >= least;
        if (top_p < 1.f) {
            s.kept_share[tid] = x;
            sync();
            unsigned long long before = 0, total = 0;
#pragma unroll 4
            for (int j = 0; j < kept; ++j) {
                const unsigned long long y = s.kept_share[j];
                total += y;
                before += s.kept[j] > me ? y : 0;
            }
            const unsigned long long part = fraction(top_p);
            const unsigned long long want = max(1ULL, __umul64hi(part, total) + (part * total != 0)); // rounded up
            stays = stays && before < want;
            sync();
        }
        s.kept_share[tid] = stays ? x : 0;
        sync();
        unsigned long long all = 0, until = 0; // of all that stay; of those up to this index
#pragma unroll 4
        for (int j = 0; j < kept; ++j) {
            const unsigned long long y = s.kept_share[j];
            all += y;
            until += (uint32_t)s.kept[j] >= (uint32_t)me ? y : 0;
        }
        const unsigned long long at = __umul64hi(fraction(u), all);
        if (stays && x > 0 && until - x <= at && at < until) {
            *token = (int)~(uint32_t)me;
            if (logprob)
                *logprob = log_share(x, all);
        }
    }
};

template <bool BF>
__global__ void __launch_bounds__(SAMPLE_THREADS, 2) sample_kernel(const SampleParams p)
{
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ SampleShared s;
    uint4 *keys = reinterpret_cast<uint4 *>(smem);
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), blocks = (int)cluster.num_blocks();
    const int row = blockIdx.x / blocks, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid < SAMPLE_TABLE) {
        const uint32_t e = SAMPLE_EXP[tid];
        s.exp[tid] = make_uint2(e - SAMPLE_ROUND_BITS, __float_as_uint((float)e));
    }
    pdl_wait();
    pdl_launch_dependents();

    // --- the row's settings ----------------------------------------------------------------------
    const float temperature = p.temperature ? p.temperature[row] : 1.f;
    const float top_p = p.top_p ? p.top_p[row] : 1.f, min_p = p.min_p ? p.min_p[row] : 0.f;
    const float u = p.uniform[row];
    int top_k = p.top_k ? p.top_k[row] : 0;
    const bool greedy = temperature == 0.f;
    if (greedy)
        top_k = 1;
    cluster.barrier_arrive(); // waited for before the first look at another block's memory

    // --- the slice, as keys, and the largest ----------------------------------------------------
    const int begin = rank * p.slice, size = max(0, min(p.slice, p.vocab - begin));
    const int vectors = (size + 7) / 8;
    const uint16_t *src = p.logits + row * p.ld + begin;
    uint32_t best = 0; // two keys
    for (int v = tid; v < vectors; v += SAMPLE_THREADS) {
        uint4 w;
        if (p.wide && 8 * v + 8 <= size) {
            w = *reinterpret_cast<const uint4 *>(src + 8 * v);
        } else {
            constexpr uint32_t NONE = BF ? 0xFF80u : 0xFC00u; // -inf
            uint32_t h[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                h[e] = 8 * v + e < size ? src[8 * v + e] : NONE;
            w = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
        }
        if (has_nan<BF>(w))
            w = make_uint4(without_nan<BF>(w.x), without_nan<BF>(w.y), without_nan<BF>(w.z), without_nan<BF>(w.w));
        w = make_uint4(keys_of(w.x), keys_of(w.y), keys_of(w.z), keys_of(w.w));
        keys[v] = w;
        best = __vmaxu2(best, __vmaxu2(__vmaxu2(w.x, w.y), __vmaxu2(w.z, w.w)));
    }
    const uint32_t mine_best = max(best & 0xFFFFu, best >> 16);
    best = mine_best;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        best = max(best, __shfl_xor_sync(0xffffffffu, best, d));
    if (lane == 0)
        s.warp_top[warp] = best;
    if (tid == 0)
        s.listed = s.n_gathered = 0;
    __syncthreads();
    cluster.barrier_wait();
    if (!(temperature >= 0.f && temperature <= SAMPLE_HOTTEST) || top_p != top_p || min_p != min_p ||
        (!greedy && !(u >= 0.f && u < 1.f))) { // the whole cluster leaves
        if (rank == 0 && tid == 0) {
            p.tokens[row] = -1;
            if (p.logprobs)
                p.logprobs[row] = NAN;
            if (p.status)
                atomicOr(p.status, W4A16_DEV_SETTING);
        }
        return;
    }
    // Where top-k keeps a few: the top_k-th largest of this block's threads' largest keys, or one that not many more of
    // these reach.  That many of the row's keys are not below it, so no smaller one is kept.
    const bool few = top_k > 0 && top_k <= SAMPLE_FEW;
    uint32_t bound = 0;
    if (few) {
#pragma unroll 1
        for (uint32_t bit = 1u << 15; bit; bit >>= 1) {
            const int n = __syncthreads_count(mine_best >= (bound | bit));
            if (n >= top_k)
                bound |= bit;
            if (n >= top_k && n <= top_k + top_k / 4 + 8)
                break;
        }
    }
    if (tid < blocks) {
        best = 0;
        for (int w = 0; w < SAMPLE_WARPS; ++w)
            best = max(best, s.warp_top[w]);
        *cluster.map_shared_rank(&s.top[rank], tid) = best;
        *cluster.map_shared_rank(&s.bound[rank], tid) = bound;
    }
    cluster.sync();
    best = 0;
    for (int r = 0; r < blocks; ++r) {
        best = max(best, s.top[r]);
        bound = max(bound, s.bound[r]);
    }
    if (best <= lowest_key<BF>()) { // nothing to choose from
        if (rank == 0 && tid == 0) {
            p.tokens[row] = -1;
            if (p.logprobs)
                p.logprobs[row] = -INFINITY;
        }
        return;
    }

    const bool infinite = best == (BF ? 0xFF80u : 0xFC00u);
    constexpr uint32_t ZERO = 0x8000u; // the key of 0
    Sampler<BF> f{s, keys, vectors, cluster, {}, 0};
    f.share.top = infinite ? 0.f : numbers_of<BF>(best).x;
    // log2(e) = LOG + LOG_LO over T.
    constexpr float LOG = 1.44269502162933349609375f, LOG_LO = 1.92596299112661747e-8f;
    const float t = greedy ? 1.f : fmaxf(temperature, SAMPLE_COLDEST), c = LOG / t;
    f.share.c_hi = c;
    f.share.c_lo = (fmaf(-c, t, LOG) + LOG_LO) / t;
    f.share.exp = s.exp;
    const unsigned long long part = fraction(min_p);
    const unsigned long long least =
        min_p >= 1.f ? 1ULL << SAMPLE_BITS
                     : (part >> (64 - SAMPLE_BITS)) + ((part & ((1ULL << (64 - SAMPLE_BITS)) - 1)) != 0); // rounded up

    // --- a few tokens: gathered and chosen from in block 0 ---------------------------------------
    if (few) {
        // (infinite logits share everything, as zeros)
        bound = infinite ? best : max(bound, lowest_key<BF>() + 1);
        for (int v = tid; v < vectors; v += SAMPLE_THREADS) {
            const uint4 k4 = keys[v];
            if (largest(k4) < bound)
                continue;
            const uint32_t w[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t key = (w[e >> 1] >> (16 * (e & 1))) & 0xFFFFu;
                if (key < bound)
                    continue;
                const uint32_t at = atomicAdd(&s.listed, 1u);
                if (at < SAMPLE_LIST)
                    s.list[at] = (unsigned long long)(infinite ? ZERO : key) << 32 | (uint32_t)~(begin + 8 * v + e);
            }
        }
        __syncthreads();
        if (tid < blocks)
            *cluster.map_shared_rank(&s.listed_by[rank], tid) = s.listed;
        if (tid == 0) // a place in block 0's list, in any order
            s.place = atomicAdd(cluster.map_shared_rank(&s.n_gathered, 0), s.listed);
        __syncthreads();
        unsigned long long *to = cluster.map_shared_rank(s.gathered, 0);
        for (uint32_t i = tid; i < s.listed && s.place + i < SAMPLE_LIST; i += SAMPLE_THREADS)
            to[s.place + i] = s.list[i];
        cluster.sync(); // the last of rows that are decided here
        uint32_t n = 0;
        for (int r = 0; r < blocks; ++r)
            n += s.listed_by[r]; // (at most the vocabulary in all)
        if (n <= SAMPLE_LIST) {
            if (rank == 0)
                f.choose((int)n, infinite ? ZERO : bound, infinite ? ZERO : best, top_k, top_p, least, u, p.tokens + row,
                         p.logprobs ? p.logprobs + row : nullptr);
            return;
        }
        // (too many are equal or nearly so)
    }
    if (infinite) { // zeros among nothing
        for (int v = tid; v < vectors; v += SAMPLE_THREADS) {
            uint4 w = keys[v];
            uint32_t *k = reinterpret_cast<uint32_t *>(&w);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t top = __vcmpeq2(k[e], best * 0x10001u);
                k[e] = (top & (ZERO * 0x10001u)) | (~top & lowest_key<BF>() * 0x10001u);
            }
            keys[v] = w;
        }
        best = ZERO;
        __syncthreads();
    }

    // --- the threshold: keys above it are kept, and the first `ties` of those at it --------------
    uint32_t threshold = 0, ties = 0; // no key is 0
    if (top_k == 1) {
        threshold = best;
        ties = 1;
    } else if (top_k > 0 || top_p < 1.f) {
        const bool by_sum = top_p < 1.f;
        const auto counts = [&s = s](int b) { return (unsigned long long)s.all_count[b]; };
        const auto sums = [&s = s](int b) { return s.all_sum[b]; };
        const auto none = [](int) { return 0ULL; };
        f.coarse(top_k > 0, by_sum);
        int bin = -1;                     // high byte of the keys that the counts at hand are of
        unsigned long long above_bin = 0; // sum of the keys above them
        unsigned long long total = 0;     // sum of what top-k keeps
        if (top_k > 0) {
            if (by_sum)
                f.search(0, (unsigned long long)top_k, counts, sums);
            else
                f.search(0, (unsigned long long)top_k, counts, none);
            total = s.total_other;
            if (s.found < 256) {
                bin = (int)s.found;
                above_bin = s.found_other;
                const unsigned long long count_above = s.found_above;
                f.fine((uint32_t)bin);
                f.search(count_above, (unsigned long long)top_k, counts, none);
                threshold = (uint32_t)bin << 8 | s.found;
                ties = (uint32_t)(top_k - s.found_above);
            }
        }
        if (by_sum) {
            const uint32_t last = threshold, last_ties = ties; // what top-k keeps ends here
            // Sum of the kept keys of high byte `at` with low byte b, by the counts at hand.
            int at = bin;
            const auto kept = [&](int b) {
                const uint32_t key = (uint32_t)at << 8 | (uint32_t)b;
                const uint32_t n = key > last ? s.all_count[b] : key == last ? last_ties : 0u;
                return n ? n * f.share(key) : 0ULL;
            };
            if (bin >= 0) {
                __syncthreads(); // found is read before the search that writes it again
                f.search(0, ~0ULL, kept, none); // (for its total)
                total = above_bin + s.total;
            } else if (top_k <= 0) {
                f.search(0, ~0ULL, sums, none); // (for its total)
                total = s.total;
            }
            const unsigned long long part = fraction(top_p);
            const unsigned long long want = max(1ULL, __umul64hi(part, total) + (part * total != 0)); // rounded up
            unsigned long long above = above_bin;
            __syncthreads();
            if (bin < 0 || above_bin >= want) { // it ends above the counts at hand
                f.search(0, want, [&](int b) { return b > bin ? s.all_sum[b] : 0ULL; }, none);
                at = (int)s.found;
                above = s.found_above;
                f.fine((uint32_t)at);
            }
            f.search(above, want, kept, none);
            threshold = (uint32_t)at << 8 | s.found;
            const unsigned long long x = f.share(threshold);
            const uint32_t n = (uint32_t)((want - s.found_above + x - 1) / x); // those whose sum before is below want
            ties = min(n, threshold == last ? last_ties : s.all_count[s.found]);
        }
    }

    // --- sums of the kept, by warp and block, in the order of the indices -----------------------
    const unsigned long long tie_share = threshold ? f.share(threshold) : 0;
    const bool ties_count = tie_share >= least && tie_share > 0;
    // A warp's range: whole steps of 32 vectors.
    const int steps = (vectors + 31) / 32, per_warp = (steps + SAMPLE_WARPS - 1) / SAMPLE_WARPS;
    const int from = warp * per_warp, to = min(steps, from + per_warp);
    const uint32_t lowest = max(threshold, lowest_key<BF>() + 1); // of what counts
    auto value = [&](uint32_t key) {
        if (key <= threshold || key < lowest)
            return 0ULL;
        const unsigned long long x = f.share(key);
        return x >= least ? x : 0ULL;
    };
    unsigned long long above = 0;
    uint32_t at_it = 0;
    for (int st = from; st < to; ++st) {
        const int v = st * 32 + lane;
        const uint4 k4 = v < vectors ? keys[v] : no_keys<BF>();
        const uint32_t w[4] = {k4.x, k4.y, k4.z, k4.w};
        uint32_t which;
        if (threshold)
            which = at_least(w, lowest);
        if (threshold || !dense(k4, lowest, which)) { // few count: one by one
            while (which) {
                const uint32_t key = pick(w, __ffs(which) - 1);
                which &= which - 1;
                above += value(key);
                at_it += key == threshold;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                unsigned long long x, y;
                f.share(w[e], x, y);
                if (least) {
                    x = x >= least ? x : 0;
                    y = y >= least ? y : 0;
                }
                above += x + y;
            }
        }
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        above += __shfl_xor_sync(0xffffffffu, above, d);
        at_it += __shfl_xor_sync(0xffffffffu, at_it, d);
    }
    if (lane == 0) {
        s.warp_above[warp] = above;
        s.warp_ties[warp] = at_it;
    }
    __syncthreads();
    if (tid < blocks) {
        unsigned long long a = 0;
        uint32_t n = 0;
        for (int w = 0; w < SAMPLE_WARPS; ++w) {
            a += s.warp_above[w];
            n += s.warp_ties[w];
        }
        *cluster.map_shared_rank(&s.above[rank], tid) = a;
        *cluster.map_shared_rank(&s.ties[rank], tid) = n;
    }
    cluster.sync(); // the last: from here no block looks at another's memory

    // --- the range that holds u, walked by its warp ----------------------------------------------
    auto kept_ties = [&](uint32_t before, uint32_t n) { // of n ties after `before` others
        return ties_count ? min(n, ties > before ? ties - before : 0u) : 0u;
    };
    unsigned long long all = 0, sum = 0; // of all kept; of those before this warp's range
    uint32_t seen = 0, ties_before = 0;
    for (int r = 0; r < blocks; ++r) {
        const unsigned long long x = s.above[r] + kept_ties(seen, s.ties[r]) * tie_share;
        if (r < rank)
            sum += x;
        if (r == rank)
            ties_before = seen;
        all += x;
        seen += s.ties[r];
    }
    for (int w = 0; w < warp; ++w) {
        sum += s.warp_above[w] + kept_ties(ties_before, s.warp_ties[w]) * tie_share;
        ties_before += s.warp_ties[w];
    }
    const unsigned long long want = greedy ? 0 : __umul64hi(fraction(u), all);
    const unsigned long long mine = s.warp_above[warp] + kept_ties(ties_before, s.warp_ties[warp]) * tie_share;
    if (!(sum <= want && want < sum + mine))
        return;
    for (int st = from; st < to; ++st) {
        const int v = st * 32 + lane;
        uint32_t key[8];
        uint32_t n = 0;
        unsigned long long x = 0;
        const uint4 k4 = v < vectors ? keys[v] : make_uint4(0, 0, 0, 0);
        const uint32_t w[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            key[e] = (w[e >> 1] >> (16 * (e & 1))) & 0xFFFFu;
            x += value(key[e]);
            n += key[e] == threshold && v < vectors;
        }
        uint32_t n_incl = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t o = __shfl_up_sync(0xffffffffu, n_incl, d);
            if (lane >= d)
                n_incl += o;
        }
        uint32_t before = ties_before + n_incl - n;
        x += kept_ties(before, n) * tie_share;
        unsigned long long incl = x;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const unsigned long long o = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d)
                incl += o;
        }
        const uint32_t has = __ballot_sync(0xffffffffu, sum + incl > want);
        if (has) {
            if (lane == __ffs(has) - 1) {
                unsigned long long at = sum + incl - x;
                bool done = false;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (!done) {
                        unsigned long long y = value(key[e]);
                        if (key[e] == threshold) {
                            y = kept_ties(before, 1) * tie_share;
                            ++before;
                        }
                        at += y;
                        if (at > want) {
                            done = true;
                            p.tokens[row] = begin + 8 * v + e;
                            if (p.logprobs)
                                p.logprobs[row] = log_share(y, all);
                        }
                    }
            }
            return;
        }
        sum += __shfl_sync(0xffffffffu, incl, 31);
        ties_before += __shfl_sync(0xffffffffu, n_incl, 31);
    }
}

namespace {

struct SampleFamily {};

} // namespace
} // namespace ops
} // namespace w4

using namespace w4;
using namespace w4::ops;

extern "C" int w4a16_sample(const void *logits, int ld, const float *uniform, const float *temperature,
                            const int32_t *top_k, const float *top_p, const float *min_p, int32_t *tokens,
                            float *logprobs, int32_t *status, int batch, int vocab, unsigned flags, cudaStream_t stream)
{
    if (flags & ~W4A16_FLAG_BF16)
        return status_of(STAGE_ARG, W4A16_ARG_FLAGS);
    if (batch < 0 || vocab <= 0 || ld < vocab)
        return status_of(STAGE_ARG, W4A16_ARG_SHAPE);
    if (vocab > SAMPLE_CLUSTER * SAMPLE_SLICE || batch > (1 << 24))
        return status_of(STAGE_UNSUPPORTED, W4A16_ARG_SHAPE);
    if (batch == 0)
        return 0;
    if (!logits || !uniform || !tokens)
        return status_of(STAGE_ARG, W4A16_ARG_NULL);
    if (!aligned(logits, 2) || !aligned(uniform, 4) || !aligned(temperature, 4) || !aligned(top_k, 4) ||
        !aligned(top_p, 4) || !aligned(min_p, 4) || !aligned(tokens, 4) || !aligned(logprobs, 4) || !aligned(status, 4))
        return status_of(STAGE_ARG, W4A16_ARG_ALIGN);
    int num_sms = 0;
    cudaError_t err = sm_count(&num_sms);
    if (err != cudaSuccess)
        return status_of(STAGE_RESOURCE, err);
    // Blocks of a row: up to three an SM in all, of which two run at once (rows differ in work: 48 mixed rows of 131071
    // took, one after the other, 43.6 us with eight blocks, 48.3 with the six that run in one go, 58 with four); no slices below 4096 logits (one
    // row of 32000 takes 7.5 us with 4096, 8.1 with 8192), nor above 32768 where eight blocks allow, so that two blocks fit
    // an SM's shared memory (256 masked rows of 100003: 85 us with four blocks, 109 with seven, 115 with two).
    const long long at_once = 3LL * num_sms / batch, useful = (vocab + 4095) / 4096, needed = (vocab + 32767) / 32768;
    long long blocks64 = at_once < useful ? at_once : useful;
    blocks64 = blocks64 < needed ? needed : blocks64;
    const int blocks = (int)(blocks64 < SAMPLE_CLUSTER ? blocks64 : SAMPLE_CLUSTER);
    SampleParams p;
    p.logits = static_cast<const uint16_t *>(logits);
    p.uniform = uniform;
    p.temperature = temperature;
    p.top_p = top_p;
    p.min_p = min_p;
    p.top_k = top_k;
    p.tokens = tokens;
    p.status = status;
    p.logprobs = logprobs;
    p.ld = ld;
    p.vocab = vocab;
    p.slice = (int)round_up((vocab + blocks - 1) / blocks, 8);
    p.wide = ld % 8 == 0 && aligned(logits, 16);
    const bool bf = (flags & W4A16_FLAG_BF16) != 0;
    const auto kernel = bf ? sample_kernel<true> : sample_kernel<false>;
    err = allow_smem<SampleFamily, 2>(reinterpret_cast<const void *>(kernel), bf, 2 * SAMPLE_SLICE);
    if (err != cudaSuccess)
        return status_of(STAGE_RESOURCE, err);
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3((unsigned)(batch * blocks));
    lc.blockDim = dim3(SAMPLE_THREADS);
    lc.dynamicSmemBytes = (size_t)p.slice * 2;
    lc.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = blocks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    lc.attrs = attr;
    lc.numAttrs = 2;
    return launch_status(cudaLaunchKernelEx(&lc, kernel, p));
}
