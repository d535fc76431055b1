// Shared memory of the eviction's selection.  Host only, standard library only.
#pragma once

#include <algorithm>

namespace sgp {

struct EvictWords {
    int key, list;  // 4-byte words for keys, and for the kept positions (0: the list is in memory)
};

// Keys of up to 49,152 positions, and the list where it fits beside them.  It never holds more
// positions than the cache, whatever the budget, so that up to 8192 positions leave room for two
// CTAs to an SM.  fixed: bytes that the selection needs besides.
inline EvictWords evict_words(int cap, int budget, int fixed) {
    const int key = (std::min(cap, 49152) + 255) & ~255;
    const int list = (std::min({cap, budget, 65536}) + 255) & ~255;  // (65,536 of them never fit)
    const int room = (227 * 1024 - fixed) / 4 - key;
    return {key, list <= room ? list : 0};
}

}  // namespace sgp
