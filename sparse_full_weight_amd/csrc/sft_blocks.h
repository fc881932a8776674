// sft_blocks.h -- strided arrays as the host sees them, to tell whether they
// lie apart.  Shared by the row-wise calls; not part of the public ABI.
#pragma once

#include <cstdint>

#include "sft_internal.h"

namespace sft {

// A block is `run` bytes, repeated along up to three dimensions.
struct Block {
    struct Dim {
        int64_t n, dist;      // dist in bytes
    };
    const void *at;
    int64_t run;
    Dim d[3];
};

// Bytes from a block's first to behind its last (0 of an empty one), or -1 where they are 2^46 or more.
int64_t extent(const Block &b);
// No byte in both.  May say no of blocks that interleave in an unlike manner.
bool apart(const Block &a, const Block &b);
// No byte in a block twice (may say no of unlike distances).
bool apart_within(const Block &b);
inline bool same(const Block &a, const Block &b) {
    bool eq = a.at == b.at && a.run == b.run;
    for (int i = 0; i < 3; ++i) eq = eq && a.d[i].n == b.d[i].n && (a.d[i].n <= 1 || a.d[i].dist == b.d[i].dist);
    return eq;
}

inline int64_t type_bytes(int32_t type) { return type == SFT_F32 ? 4 : 2; }
inline bool aligned_to(const void *p, int64_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline Block rows_block(const void *p, int64_t n, int64_t dist, int64_t len, int64_t size) {
    return Block{p, len * size, {{n, dist * size}, {1, 0}, {1, 0}}};
}
inline Block flat_block(const void *p, int64_t bytes) { return Block{p, bytes, {{1, 0}, {1, 0}, {1, 0}}}; }

}  // namespace sft
