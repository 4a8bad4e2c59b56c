// The paged 8-bit key/value cache: what its kernels and their callers share.
// Layouts and meaning are those of include/rlt.h (rlt_cache8, rlt_rope).
#pragma once

#include "kernels.cuh"

namespace rlt {

struct Cache8 {
    uint8_t* pages;           // e4m3 [n_pages][2][kv_heads][page][dh]
    float* scales;            // [n_pages][2][kv_heads]
    const int32_t* table;     // [rows][row_pages]
    int* status;              // sticky word, may be null
    // what it is set to: bad table entry; bad length or position; a bounded wait gave up
    int arg_code, cap_code, late_code;
    int n_pages, rows, row_pages, page, kv_heads, dh;
};

struct Rope8 {                // rot = 0: no rotation
    const float* cs;          // [positions][rot/2]
    const float* sn;
    int positions, rot, interleaved, origin;
};

// One tensor [rows][n][heads][dh], heads adjacent, pitches in elements.
template <typename T>
struct Tok8 {
    T* p;
    int64_t row, token;
};

// Tokens start[b] .. start[b]+counts[b]-1 of every row (counts null: n each).
template <typename T>
[[nodiscard]]
cudaError_t launch_cache8_append(const Cache8& c, Tok8<const T> k, Tok8<const T> v,
                                 const int32_t* start, const int32_t* counts, int n,
                                 const Rope8& rope, cudaStream_t st);

// q as a sum of S partial slabs (S = 1: q itself), of fp32; a row's prefix is
// lens[b] + lens_add.
template <typename TQ, typename TO>
[[nodiscard]]
cudaError_t launch_cache8_attend(const Cache8& c, Tok8<const TQ> q, int slabs, size_t slab,
                                 Tok8<TO> out, int heads, int n, const int32_t* lens,
                                 int lens_add, float scale, const Rope8& rope, cudaStream_t st);

// The same, for n * heads / kv_heads <= 4.
template <typename TQ, typename TO>
[[nodiscard]]
cudaError_t launch_cache8_decode(const Cache8& c, Tok8<const TQ> q, int slabs, size_t slab,
                                 Tok8<TO> out, int heads, int n, const int32_t* lens,
                                 int lens_add, float scale, const Rope8& rope, cudaStream_t st);

}  // namespace rlt
