// Reordering rows within groups, in place (include/rlt.h: rlt_rows_reorder,
// rlt_state_reorder): row i of a group takes the contents of row parents[i].
//
// A thread owns one column -- the same 16 (8, 4, 1) bytes of every row of one
// group -- and reads what every moved row will hold before it writes any of
// them, so any parents, cycles included, are served in place without scratch,
// barriers or a second pass.  Rows that stay are neither read (but as someone's
// parent) nor written.  Bound by HBM: distinct parents read, moved rows
// written; all loads of a thread are in flight together.  The column narrows
// as the group grows so that it stays in registers (16 rows x 16 bytes, 32 x 8,
// 64 x 4).
#include <algorithm>

#include "beam.cuh"

namespace rlt {
namespace {

constexpr int NT = 256;

struct Segs {
    ReorderSeg s[kMaxSegs];
    int64_t cols[kMaxSegs];         // columns of one plane (at the largest length)
    int64_t end[kMaxSegs];          // columns of a row up to and with the segment
    int n;
};

// rows a group may have, and the bytes of a column
template <typename V, int K>
__global__ void __launch_bounds__(NT)
k_reorder(const __grid_constant__ Segs segs, const int32_t* __restrict__ parents, int beams,
          unsigned blocks_per_group) {
    __shared__ int s_from[K];
    pdl_enter();
    const unsigned group = blockIdx.x / blocks_per_group, part = blockIdx.x % blocks_per_group;
    for (int i = threadIdx.x; i < K; i += NT) {
        int p = i < beams ? __ldg(parents + (size_t)group * beams + i) : -1;
        s_from[i] = p == i || p >= beams ? -1 : p;
    }
    __syncthreads();
    int64_t col = (int64_t)part * NT + threadIdx.x;
    if (col >= segs.end[segs.n - 1]) return;
    int si = 0;
    while (col >= segs.end[si]) ++si;
    if (si) col -= segs.end[si - 1];
    const ReorderSeg& sg = segs.s[si];
    const int64_t plane = col / segs.cols[si], x = col - plane * segs.cols[si];
    const size_t row0 = (size_t)group * beams;
    const int64_t first = sg.start / sg.page * sg.unit;
    if (sg.pos) {                   // a group's rows sit at one position
        const int64_t last = ((int64_t)__ldg(sg.pos + row0) + sg.page - 1) / sg.page * sg.unit;
        if (first + (x + 1) * (int64_t)sizeof(V) > last) return;
        if (sg.from && first + x * (int64_t)sizeof(V) < __ldg(sg.from + row0) * sg.unit) return;
    }
    uint8_t* base = sg.base + (int64_t)row0 * sg.row + plane * sg.plane + first +
                    x * (int64_t)sizeof(V);
    V v[K];
#pragma unroll
    for (int i = 0; i < K; ++i)
        if (s_from[i] >= 0) v[i] = *reinterpret_cast<const V*>(base + (int64_t)s_from[i] * sg.row);
#pragma unroll
    for (int i = 0; i < K; ++i)
        if (s_from[i] >= 0) *reinterpret_cast<V*>(base + (int64_t)i * sg.row) = v[i];
}

}  // namespace

cudaError_t launch_reorder(const ReorderSeg* segs, int n_segs, const int32_t* parents, int groups,
                           int beams, cudaStream_t st) {
    Segs a = {};
    uint64_t align = 16;            // what divides every address of every column
    for (int i = 0; i < n_segs; ++i) {
        const ReorderSeg& s = segs[i];
        const int64_t blocks = (s.len + s.page - 1) / s.page - s.start / s.page;
        if (blocks <= 0 || s.planes <= 0 || s.unit <= 0) continue;
        a.s[a.n++] = s;
        for (uint64_t x : {(uint64_t)(uintptr_t)s.base, (uint64_t)s.row, (uint64_t)s.unit,
                           s.planes > 1 ? (uint64_t)s.plane : 0})
            while (x % align) align /= 2;
    }
    if (!a.n || groups <= 0 || beams < 2) return cudaSuccess;
    int width = (int)align;
    width = std::min(width, beams <= 16 ? 16 : beams <= 32 ? 8 : 4);
    if (width < 4) width = 1;
    if (width == 8 && beams <= 16) width = 4;       // one kernel for what is not 16-aligned
    int64_t total = 0;
    for (int i = 0; i < a.n; ++i) {
        const ReorderSeg& s = a.s[i];
        a.cols[i] = ((s.len + s.page - 1) / s.page - s.start / s.page) * s.unit / width;
        total += a.cols[i] * s.planes;
        a.end[i] = total;
    }
    const int64_t per = (total + NT - 1) / NT;
    if (per * groups > 0x7fffffff) return cudaErrorInvalidConfiguration;
    const dim3 grid((unsigned)(per * groups));
    const unsigned b = (unsigned)per;
    cudaError_t e;
    if (width == 16) {
        e = beams <= 4    ? launch(k_reorder<uint4, 4>, grid, NT, 0, st, a, parents, beams, b)
            : beams <= 8  ? launch(k_reorder<uint4, 8>, grid, NT, 0, st, a, parents, beams, b)
                          : launch(k_reorder<uint4, 16>, grid, NT, 0, st, a, parents, beams, b);
    } else if (width == 8) {
        e = launch(k_reorder<uint2, 32>, grid, NT, 0, st, a, parents, beams, b);
    } else if (width == 4) {
        e = launch(k_reorder<uint32_t, 64>, grid, NT, 0, st, a, parents, beams, b);
    } else {
        e = launch(k_reorder<uint8_t, 64>, grid, NT, 0, st, a, parents, beams, b);
    }
    if (e == cudaSuccess) rlt_count_launch();
    return e;
}

}  // namespace rlt
