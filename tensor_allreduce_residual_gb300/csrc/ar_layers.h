// ar_layers.h -- the buffers in which one call moves tokens or pages: every
// layer's keys and values.  Plain C++, which the host tests compile.
#pragma once

#include <stdint.h>

namespace ar {

constexpr int kMaxLayers = 128;
struct Layers {
    char* even[kMaxLayers];  // buffers 0, 2, 4 ..: each layer's keys where none is named twice
    char* odd[kMaxLayers];
};

// Lists k[0], v[0], k[1], v[1] .. in `to`, each buffer once, and returns how many there are.  Layers that share a cache name it
// several times; its tokens move once, as a second owner of the same bytes would move what the first has moved already.
inline int distinct_buffers(Layers* to, void* const* k, void* const* v, int layers)
{
    void* slots[8 * kMaxLayers];  // a hash table, a quarter full at the most
    int bits = 3;
    while ((1 << bits) < 8 * layers)
        ++bits;
    const unsigned mask = (1u << bits) - 1;
    for (unsigned i = 0; i <= mask; ++i)
        slots[i] = nullptr;
    int count = 0;
    for (int i = 0; i < 2 * layers; ++i) {
        void* const p = i & 1 ? v[i >> 1] : k[i >> 1];
        unsigned at = static_cast<unsigned>(reinterpret_cast<uintptr_t>(p) * 0x9e3779b97f4a7c15ull >> (64 - bits));
        while (slots[at] != nullptr && slots[at] != p)
            at = (at + 1) & mask;
        if (slots[at] == nullptr) {
            slots[at] = p;
            (count & 1 ? to->odd : to->even)[count >> 1] = static_cast<char*>(p);
            ++count;
        }
    }
    return count;
}

}  // namespace ar
