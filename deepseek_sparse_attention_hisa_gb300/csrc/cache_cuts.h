// Spans of tiles and the rows that they cut: the arithmetic that the combine over a cache in pages
// (k_cache_tc.cu) and the join of its parts have in common. Plain C++, so that the host can check it.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define HISA_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define HISA_HOST_DEVICE inline
#endif

namespace hisa {

// A row whose tiles lie in the spans of several CTAs: entry `row` of the list of cuts if there are as few rows as
// CTAs, else the entry of the CTA that has its first tile.
struct Cut {
    int64_t row;                                        // -1: none
    int first, last;                                    // the CTAs that have its first and its last tile
    int place, pad[3];                                  // of the first CTA's sums
};

// The first tile of CTA c's span: c total / groups (a 64-bit division takes a few hundred cycles).
HISA_HOST_DEVICE int64_t span_start(int c, int64_t total, int groups) {
    if (total < (int64_t)1 << 24) return (uint32_t)c * (uint32_t)total / (uint32_t)groups;
    return c * total / groups;
}
// The CTA whose span holds tile `tile`.
HISA_HOST_DEVICE int span_of(int64_t tile, int64_t total, int groups) { return (int)(((tile + 1) * groups - 1) / total); }

// Whether an entry names a row and parts that there are. Every entry is cleared before a CTA can give up, so
// only what is no entry at all fails here; the join takes its addresses from it.
HISA_HOST_DEVICE bool cut_fits(const Cut &k, int64_t rows, int ctas) {
    return k.row >= 0 && k.row < rows && k.first >= 0 && k.first <= k.last && k.last < ctas && k.place >= 2 * k.first &&
           k.place <= 2 * k.first + 1;
}

}  // namespace hisa
