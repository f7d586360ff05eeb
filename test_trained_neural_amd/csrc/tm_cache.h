// The paged 8-bit cache's layout (include/tm_attention.h), shared by its
// kernels (tm_cache.hip) and the attention that reads it (tm_attend.hip).
#pragma once

#include "../../include/tm_attention.h"
#include "tm_device.h"

struct tm_cache {
    int H, d, n_pages, n_seqs, seq_pages;
    size_t off[4], bytes;   // meta, scales, keys, values
};

namespace tmk {

constexpr int PAGE = TM_CACHE_PAGE, BLOCK = TM_CACHE_BLOCK;
constexpr int CACHE_E_MIN = -110, CACHE_E_MAX = 119;

// A cache's blob as a kernel sees it.
struct CacheView {
    unsigned char* k;
    unsigned char* v;
    unsigned char* scales;
    int* status;
    int* lengths;
    int* refs;
    int* table;
    int H, d, n_pages, n_seqs, seq_pages;

    __device__ size_t head_at(int page, int h) const { return (size_t)page * H + h; }
    // tokens a sequence holds, whatever the blob says
    __device__ int length(int s) const { return min(max(lengths[s], 0), seq_pages * PAGE); }
    __device__ int page_at(int s, int i) const { return table[(size_t)s * seq_pages + i]; }
    __device__ bool page_ok(int page) const { return (unsigned)page < (unsigned)n_pages; }
};

inline CacheView cache_view(const tm_cache* c, void* blob) {
    char* b = static_cast<char*>(blob);
    int* meta = reinterpret_cast<int*>(b + c->off[0]);
    return CacheView{reinterpret_cast<unsigned char*>(b + c->off[2]), reinterpret_cast<unsigned char*>(b + c->off[3]),
                     reinterpret_cast<unsigned char*>(b + c->off[1]), meta, meta + 64, meta + 64 + c->n_seqs,
                     meta + 64 + c->n_seqs + c->n_pages, c->H, c->d, c->n_pages, c->n_seqs, c->seq_pages};
}

// e + 127 as stored -> 2^e
__device__ __forceinline__ float scale_of(unsigned char byte) { return __builtin_bit_cast(float, (unsigned)byte << 23); }

// Calls f(integral_constant<D>) for the head widths the cache takes.
template <class F> hipError_t for_head_dim(int d, F&& f) {
    switch (d) {
        case 32: return f(std::integral_constant<int, 32>{});
        case 64: return f(std::integral_constant<int, 64>{});
        case 96: return f(std::integral_constant<int, 96>{});
        case 128: return f(std::integral_constant<int, 128>{});
        case 160: return f(std::integral_constant<int, 160>{});
        case 192: return f(std::integral_constant<int, 192>{});
        case 224: return f(std::integral_constant<int, 224>{});
        case 256: return f(std::integral_constant<int, 256>{});
    }
    return hipErrorInvalidValue;
}

inline bool ptr_ok(const void* p, size_t a) { return p && (uintptr_t)p % a == 0; }

// Distances of a token array in elements: multiples of 8 (with 16-byte
// aligned rows), not negative, small enough for 64-bit offsets.
inline bool strides_ok(long batch, long token) {
    const long lim = 1L << 40;
    return batch >= 0 && token >= 0 && batch <= lim && token <= lim && batch % 8 == 0 && token % 8 == 0;
}

// Bytes of tm_cache_attend's workspace (tm_attend.hip).
size_t attend_workspace(const tm_cache* c, int batch, int n_tokens, int heads);

}  // namespace tmk
