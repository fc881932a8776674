// sft_blocks.cpp -- whether strided arrays lie apart (host).
#include <algorithm>

#include "sft_blocks.h"

namespace sft {

namespace {

constexpr __int128 kMost = __int128(1) << 46;

// Bytes that the dimensions closer together than `below` span.
__int128 span(const Block &b, int64_t below) {
    __int128 e = b.run;
    for (const Block::Dim &d : b.d)
        if (d.n > 1 && d.dist < below) e += __int128(d.n - 1) * d.dist;
    return e;
}

bool empty(const Block &b) {
    return !b.at || b.run <= 0 || b.d[0].n <= 0 || b.d[1].n <= 0 || b.d[2].n <= 0;
}

// Whether every place of the block, seen modulo s, lies in one run of *inner bytes.
bool folds(const Block &b, int64_t s, int64_t *inner) {
    for (const Block::Dim &d : b.d)
        if (d.n > 1 && d.dist >= s && d.dist % s) return false;
    const __int128 e = span(b, s);
    *inner = static_cast<int64_t>(std::min<__int128>(e, INT64_MAX));
    return e <= s;
}

}  // namespace

int64_t extent(const Block &b) {
    if (empty(b)) return 0;
    const __int128 e = span(b, INT64_MAX);
    return e < kMost ? static_cast<int64_t>(e) : -1;
}

bool apart(const Block &a, const Block &b) {
    if (empty(a) || empty(b)) return true;
    const uint8_t *pa = static_cast<const uint8_t *>(a.at), *pb = static_cast<const uint8_t *>(b.at);
    if (pa + extent(a) <= pb || pb + extent(b) <= pa) return true;
    // side by side in every period of a distance that both repeat by
    const Block *both[] = {&a, &b};
    for (const Block *from : both)
        for (const Block::Dim &d : from->d) {
            if (d.n <= 1 || d.dist <= 0) continue;
            int64_t in_a, in_b;
            if (!folds(a, d.dist, &in_a) || !folds(b, d.dist, &in_b)) continue;
            const int64_t off = ((pb - pa) % d.dist + d.dist) % d.dist;
            if (off >= in_a && off + in_b <= d.dist) return true;
        }
    return false;
}

bool apart_within(const Block &b) {
    if (empty(b)) return true;
    for (const Block::Dim &d : b.d)
        if (d.n > 1 && (d.dist < span(b, d.dist))) return false;
    // of equal distances one would repeat the other's places
    for (int i = 0; i < 3; ++i)
        for (int j = 0; j < i; ++j)
            if (b.d[i].n > 1 && b.d[j].n > 1 && b.d[i].dist == b.d[j].dist) return false;
    return true;
}

}  // namespace sft
