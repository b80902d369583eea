// w4a16_kv4.cuh -- the paged key-value cache held in 4 bits: where a value lies, and how it is coded.
//
// A page holds one record per KV head.  A record of P positions of D values in G groups is
//     key codes [P][D / 8] words | value codes [P][D / 8] words | key steps and bases [P][G] | the values' [P][G]
// filled up to a multiple of 16 bytes.  A word holds eight codes of values 8 w .. 8 w + 7, the lowest first; a
// step and a base are two 16-bit values side by side.  The words of a row lie in the order in which the
// attention's lanes read them, so that a lane's words of a row are one load:
//     keys:    word w = 8 b + 2 t + i (block b of 64 values, lane t < 4, i < 2) at place 16 (b / 2) + 4 t + 2 (b % 2) + i
//              (D = 64: at place w),
//     values:  word w = 8 b + g (lane g < 8) at place g D / 64 + b.
#pragma once

#include "w4a16_ops.cuh"

namespace w4 {
namespace ops {

// Groups of a row, or 0 for a group size that the cache does not take.
inline int kv4_groups(int head_dim, int group_size)
{
    if (group_size == -1)
        return 1;
    return group_size > 0 && group_size % 64 == 0 && head_dim % group_size == 0 ? head_dim / group_size : 0;
}

inline bool kv4_dim(int head_dim)
{
    return head_dim == 64 || head_dim == 128 || head_dim == 256;
}

inline long long kv4_record_bytes(int page, int head_dim, int groups)
{
    return round_up((long long)page * (head_dim + 8 * groups), 16);
}

// Byte offsets inside a record.
struct Kv4Record {
    int values, key_params, value_params;
    long long bytes;
};

inline Kv4Record kv4_record(int page, int head_dim, int groups)
{
    Kv4Record r;
    r.values = page * (head_dim / 2);
    r.key_params = page * head_dim;
    r.value_params = r.key_params + page * groups * 4;
    r.bytes = kv4_record_bytes(page, head_dim, groups);
    return r;
}

// Places of words inside a row (head_dim / 64 = BLOCKS).
__device__ __forceinline__ int kv4_key_place(int word, int blocks)
{
    const int b = word >> 3, t = (word >> 1) & 3, i = word & 1;
    return blocks == 1 ? word : 16 * (b >> 1) + 4 * t + 2 * (b & 1) + i;
}

__device__ __forceinline__ int kv4_value_place(int word, int blocks)
{
    return (word & 7) * blocks + (word >> 3);
}

} // namespace ops
} // namespace w4
