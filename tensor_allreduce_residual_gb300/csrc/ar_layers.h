// ar_layers.h -- the buffers in which one call moves tokens or pages: every
// layer's keys and values.  Plain C++, which the host tests compile.
#pragma once

#include <stdint.h>

namespace ar {

constexpr int kMaxLayers = 128;
struct Layers {
    char* buffer[2 * kMaxLayers];
};

// Lists k[0], v[0], k[1], v[1] .. in `to`, each buffer once, and returns how many there are.  Layers that share a cache name it
// several times; its tokens move once, as a second owner of the same bytes would move what the first has moved already.
inline int distinct_buffers(Layers* to, void* const* k, void* const* v, int layers)
{
    constexpr int kSlots = 1024;  // of a hash table, a quarter full at the most
    uint16_t slots[kSlots] = {};  // a buffer's number and 1; 0: free
    int count = 0;
    for (int i = 0; i < 2 * layers; ++i) {
        char* const p = static_cast<char*>(i & 1 ? v[i >> 1] : k[i >> 1]);
        unsigned at = static_cast<unsigned>(reinterpret_cast<uintptr_t>(p) * 0x9e3779b97f4a7c15ull >> 54);
        while (slots[at] != 0 && to->buffer[slots[at] - 1] != p)
            at = (at + 1) % kSlots;
        if (slots[at] == 0) {
            to->buffer[count++] = p;
            slots[at] = static_cast<uint16_t>(count);
        }
    }
    return count;
}

}  // namespace ar
