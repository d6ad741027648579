// Index arithmetic of the attention kernels, in plain C++ that a host compiler takes too: its
// edges are checked there.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define MOE_HD __host__ __device__ __forceinline__
#else
#define MOE_HD inline
#endif

namespace moe {

// The chunk kernel's ring of code tiles.  Keys and values take turns (copy number `it` is even
// for keys, odd for values) and each is converted by a group of its own.  A wait by parity tells a
// phase only from the one before it, so a group has to see every phase of the barriers it waits on.  With
// one "full" barrier to a slot and an odd number of slots it would see every second one: the copy before its
// own, still in flight, would leave the barrier with the parity that it waits for.  So there are two to
// a slot, and each belongs to one group.  The copying warp waits for both groups' slots in order: one
// "free" barrier to a slot.
template <int SLOTS>
struct CodeRing {
    static constexpr uint32_t kFull = 2 * SLOTS;  // "full" barriers
    static MOE_HD uint32_t slot(uint32_t it) { return it % SLOTS; }
    static MOE_HD uint32_t full(uint32_t it) { return it % kFull; }
    static MOE_HD uint32_t full_parity(uint32_t it) { return (it / kFull) & 1; }
    static MOE_HD uint32_t free_parity(uint32_t it) { return ((it / SLOTS) & 1) ^ 1; }
};

// Whether a sequence's rows [tok0, t1) lie in the batch's T and its length in the page table.  (By comparisons
// only: the difference of two offsets that are anything may wrap to a number of tokens that looks sound.)
MOE_HD bool seq_ok(int tok0, int t1, int len, int T, int64_t max_len) {
    return tok0 >= 0 && t1 >= tok0 && t1 <= T && len >= 0 && len <= max_len;
}

// The first key that the token at `pos` sees through a window (0: all).  (No difference is taken before it is
// known to be a key: a window may be any number, a position may lie before the start.)
MOE_HD int first_key(int pos, int window) { return window && pos >= window ? pos - window + 1 : 0; }

// Tiles of `count` keys from `key` on against the keys [from, to), none of the three below 0.  A length may be up
// to 2^31 - 16, so the end of its last tile only fits 32 bits without a sign.
MOE_HD bool tile_inside(int key, int count, int from, int to) {
    return key >= from && (uint32_t)key + count <= (uint32_t)to;
}
MOE_HD bool tile_meets(int key, int count, int from, int to) {
    return key < to && (uint32_t)key + count > (uint32_t)from;
}
// Tiles of 2^log2 keys that hold the keys [0, to), to >= 0.
MOE_HD int tiles_until(int to, int log2) { return (int)(((uint32_t)to + (1u << log2) - 1) >> log2); }

}  // namespace moe
