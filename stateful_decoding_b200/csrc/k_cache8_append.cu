// Appending keys and values to the paged 8-bit cache: rotate the keys, find
// each (page, head)'s largest magnitude, choose its power-of-two scale, round
// to e4m3 (include/rlt.h: rlt_cache8_append).
//
// One item is one (row, page touched, key or value head): the page's new
// tokens are read once into registers (every load of the item in flight
// before the first is used), rotated there, reduced to their largest
// magnitude, and written as bytes, so the bytes moved are the operands' and
// the result's alone.  The kernel is bound by HBM for prompts and by its
// launch for single tokens.  Scales are powers of two so that a page whose
// scale grows as tokens arrive is brought to the new one exactly (e4m3
// exponents shift), but for values that fall into the subnormal range.
//
// A thread holds units of 2V values of one token: dims a..a+V-1 and b..b+V-1
// where, in the half layout, b = a + rot/2 (the rotation partners), else
// b = a + V.  V = 8 (16-byte loads of bf16), or 4 where rot is no multiple
// of 16.  An item of m tokens has m * dh/2V such units, spread
// over T threads, NIT units each: one warp per item (four items per CTA) up to
// 128 units -- generated tokens and short blocks, where 256-thread items left
// most threads idle -- and 256 threads beyond.
#include <cuda_fp8.h>
#include <float.h>

#include <algorithm>

#include "cache8.cuh"

namespace rlt {
namespace {

constexpr int kLeastExp = -110, kMostExp = 120;

// V (8 or 4) values on 16 (8, for 4 of bf16) bytes
template <int V>
__device__ __forceinline__ void load(const float* p, float* x) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(p + i));
        x[i] = v.x; x[i + 1] = v.y; x[i + 2] = v.z; x[i + 3] = v.w;
    }
}
__device__ __forceinline__ void unpack2(uint32_t w, float* x) {
    x[0] = __uint_as_float(w << 16);
    x[1] = __uint_as_float(w & 0xffff0000u);
}
template <int V>
__device__ __forceinline__ void load(const bf16* p, float* x) {
    if constexpr (V == 8) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
        unpack2(v.x, x);
        unpack2(v.y, x + 2);
        unpack2(v.z, x + 4);
        unpack2(v.w, x + 6);
    } else {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
        unpack2(v.x, x);
        unpack2(v.y, x + 2);
    }
}

// smallest 2^e with amax <= 448 * 2^e = 1.75 * 2^(e+8), e in [least, most]
__device__ __forceinline__ float pow2_scale(float amax) {
    if (!(amax > 0.f)) return __uint_as_float((uint32_t)(kLeastExp + 127) << 23);
    const uint32_t u = __float_as_uint(amax);
    int e = (int)(u >> 23) - 127;                    // subnormal amax: e = -127, clamped below
    e -= (u & 0x7fffffu) <= 0x600000u ? 8 : 7;       // mantissa up to 1.75
    e = max(kLeastExp, min(kMostExp, e));
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t two) {
    const __half2_raw h =
        __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(two & 0xffffu), __NV_E4M3);
    return __half22float2(__half2(h));
}
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float f) {
    const float2 a = from_e4m3x2(w), b = from_e4m3x2(w >> 16);
    return to_e4m3x4(a.x * f, a.y * f, b.x * f, b.y * f);
}

template <int V>
__device__ __forceinline__ void to_bytes(uint8_t* p, const float* x, float f) {
    const uint32_t lo = to_e4m3x4(x[0] * f, x[1] * f, x[2] * f, x[3] * f);
    if constexpr (V == 8)
        *reinterpret_cast<uint2*>(p) =
            make_uint2(lo, to_e4m3x4(x[4] * f, x[5] * f, x[6] * f, x[7] * f));
    else
        *reinterpret_cast<uint32_t*>(p) = lo;
}

// where the two halves of unit u of a token sit, and its first angle (-1: unrotated)
struct Unit {
    int a, b, ang;
};
template <int V>
__device__ __forceinline__ Unit unit_of(int u, int rot, bool inter) {
    if (inter || 2 * V * u >= rot) return {2 * V * u, 2 * V * u + V, 2 * V * u < rot ? V * u : -1};
    return {V * u, V * u + rot / 2, V * u};
}

// T threads per item, NIT units a thread; kItems items per CTA
template <typename T_, int V, int T, int NIT>
__global__ void __launch_bounds__(T == 32 ? 128 : T)
k_cache8_append(Cache8 c, Tok8<const T_> k, Tok8<const T_> v, const int32_t* __restrict__ start,
                const int32_t* __restrict__ counts, int n, int page_log2, int row_blocks,
                int n_items, Rope8 rope) {
    constexpr int kItems = T == 32 ? 4 : 1;
    pdl_enter();
    const int sub = T == 32 ? (int)threadIdx.x >> 5 : 0, tid = (int)threadIdx.x - sub * T;
    const int item = (int)blockIdx.x * kItems + sub;
    if (item >= n_items) return;                     // whole warps (T = 32) or no thread
    const int kv = item & 1, h = (item >> 1) % c.kv_heads;
    const int rb = (item >> 1) / c.kv_heads, row = rb / row_blocks, j = rb % row_blocks;
    const int s0 = __ldg(start + row);
    const int cnt = counts ? __ldg(counts + row) : n;
    const bool first = tid == 0 && h == 0 && kv == 0;
    auto say = [&](int code) {
        if (first && c.status) atomicCAS(c.status, 0, code);
    };
    const int page = 1 << page_log2, cap = c.row_pages << page_log2;
    if (cnt < 0 || cnt > n || s0 < 0 || s0 > cap || cnt > cap - s0) {
        // the tokens within the capacity are still written when the counts are sane
        if (j == 0) say(c.cap_code);
        if (cnt < 0 || cnt > n || s0 < 0 || s0 >= cap) return;
    }
    const int end = min(cap, s0 + cnt);
    const int block = (s0 >> page_log2) + j;
    int lo = max(s0, block << page_log2);
    int hi = min(end, (block + 1) << page_log2);
    const Rope8 r = rope;
    if (r.rot) {                                     // positions without a row in the table
        const int plo = -r.origin, phi = r.positions - r.origin;
        if (lo < hi && (lo < plo || hi > phi)) say(c.cap_code);
        lo = max(lo, plo);
        hi = min(hi, phi);
    }
    if (lo >= hi) return;
    // (used only after the loads below: its latency overlaps theirs)
    const int pg = __ldg(c.table + (size_t)row * c.row_pages + block);
    const int dh = c.dh, upt_log2 = (dh == 128 ? 7 : 6) - (V == 8 ? 4 : 3);
    const int upt = 1 << upt_log2;                   // units per token
    const int units = (hi - lo) << upt_log2;
    const Tok8<const T_> src = kv ? v : k;
    const T_* base = src.p + (int64_t)row * src.row + (int64_t)(lo - s0) * src.token +
                     (int64_t)h * dh;
    const int rot = kv ? 0 : r.rot;
    const bool inter = r.interleaved != 0;

    float x[NIT][2 * V];
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < NIT; ++i) {
        const int w = tid + i * T;
        if (w < units) {
            const Unit un = unit_of<V>(w & (upt - 1), rot, inter);
            const T_* p = base + (int64_t)(w >> upt_log2) * src.token;
            load<V>(p + un.a, x[i]);
            load<V>(p + un.b, x[i] + V);
        }
    }
#pragma unroll
    for (int i = 0; i < NIT; ++i) {
        const int w = tid + i * T;
        if (w < units) {
            const Unit un = unit_of<V>(w & (upt - 1), rot, inter);
            if (un.ang >= 0) {
                const size_t at =
                    (size_t)(lo + (w >> upt_log2) + r.origin) * (rot >> 1) + (size_t)un.ang;
                float cs[V], sn[V];
                load<V>(r.cs + at, cs);
                load<V>(r.sn + at, sn);
#pragma unroll
                for (int q = 0; q < V; ++q) {
                    // pair q: (x[q], x[q+V]) in the half layout, (x[2q], x[2q+1]) interleaved
                    const float x1 = inter ? x[i][2 * q] : x[i][q];
                    const float x2 = inter ? x[i][2 * q + 1] : x[i][q + V];
                    // rounded one by one, not contracted: the bytes do not depend on
                    // how a compiler fuses the pair
                    const float y1 = __fsub_rn(__fmul_rn(x1, cs[q]), __fmul_rn(x2, sn[q]));
                    const float y2 = __fadd_rn(__fmul_rn(x2, cs[q]), __fmul_rn(x1, sn[q]));
                    if (inter) {
                        x[i][2 * q] = y1;
                        x[i][2 * q + 1] = y2;
                    } else {
                        x[i][q] = y1;
                        x[i][q + V] = y2;
                    }
                }
            }
#pragma unroll
            for (int q = 0; q < 2 * V; ++q) amax = fmaxf(amax, fabsf(x[i][q]));   // skips NaN
        }
    }
    if (pg < 0 || pg >= c.n_pages) {                 // the same for the whole item
        say(c.arg_code);
        return;
    }
    amax = warp_max(amax);
    if constexpr (T > 32) {
        __shared__ float s_max[T / 32];
        if ((tid & 31) == 0) s_max[tid >> 5] = amax;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < T / 32; ++i) amax = fmaxf(amax, s_max[i]);
    }
    amax = fminf(amax, FLT_MAX);                     // infinities as the largest finite value
    float* scale_at = c.scales + ((size_t)pg * 2 + kv) * c.kv_heads + h;
    uint8_t* bytes = c.pages + (((size_t)pg * 2 + kv) * c.kv_heads + h) * (size_t)(page * dh);
    const int slot0 = lo - block * page, kept = s0 - block * page;
    float scale = pow2_scale(amax);
    if (kept > 0) {                                  // the row's earlier tokens in this page
        const float old = __ldcg(scale_at);
        if constexpr (T > 32) __syncthreads();       // every thread has read it before it changes
        else __syncwarp();
        if (old > 0.f && old >= scale) {
            scale = old;
        } else if (old > 0.f) {
            const float f = old / scale;
            uint4* q = reinterpret_cast<uint4*>(bytes);
            for (int i = tid; i < kept * dh / 16; i += T) {
                uint4 w = q[i];
                w.x = rescale4(w.x, f);
                w.y = rescale4(w.y, f);
                w.z = rescale4(w.z, f);
                w.w = rescale4(w.w, f);
                q[i] = w;
            }
        }
    }
    if (tid == 0) *scale_at = scale;
    const float inv = 1.f / scale;                   // exact for powers of two
    uint8_t* dst = bytes + (size_t)slot0 * dh;
#pragma unroll
    for (int i = 0; i < NIT; ++i) {
        const int w = tid + i * T;
        if (w < units) {
            const Unit un = unit_of<V>(w & (upt - 1), rot, inter);
            uint8_t* p = dst + (w >> upt_log2) * dh;
            to_bytes<V>(p + un.a, x[i], inv);
            to_bytes<V>(p + un.b, x[i] + V, inv);
        }
    }
}

}  // namespace

template <typename T>
cudaError_t launch_cache8_append(const Cache8& c, Tok8<const T> k, Tok8<const T> v,
                                 const int32_t* start, const int32_t* counts, int n,
                                 const Rope8& rope, cudaStream_t st) {
    if (c.rows <= 0 || n <= 0) return cudaSuccess;
    // pages a row can touch: n tokens from any slot of the first one
    const int row_blocks = (int)std::min<int64_t>(c.row_pages, ((int64_t)n + c.page - 2) / c.page + 1);
    const int64_t items = (int64_t)c.rows * row_blocks * c.kv_heads * 2;
    if (items > 0x7fffffff) return cudaErrorInvalidConfiguration;
    int page_log2 = 4;
    while ((1 << page_log2) < c.page) ++page_log2;
    auto go = [&](auto kern, int threads, int per_cta) {
        cudaError_t e = launch(kern, (unsigned)((items + per_cta - 1) / per_cta), threads, 0, st, c,
                               k, v, start, counts, n, page_log2, row_blocks, (int)items, rope);
        if (e == cudaSuccess) rlt_count_launch();
        return e;
    };
    const bool wide = rope.rot % 16 == 0;            // else a unit of 16 would turn in part
    const int units = std::min(n, c.page) * (c.dh / (wide ? 16 : 8));
    if (wide) {
        if (units <= 64) return go(k_cache8_append<T, 8, 32, 2>, 128, 4);
        if (units <= 128) return go(k_cache8_append<T, 8, 32, 4>, 128, 4);
        if (units <= 512) return go(k_cache8_append<T, 8, 256, 2>, 256, 1);
        return go(k_cache8_append<T, 8, 256, 4>, 256, 1);
    }
    if (units <= 128) return go(k_cache8_append<T, 4, 32, 4>, 128, 4);
    if (units <= 1024) return go(k_cache8_append<T, 4, 256, 4>, 256, 1);
    return go(k_cache8_append<T, 4, 256, 8>, 256, 1);
}

template cudaError_t launch_cache8_append<float>(const Cache8&, Tok8<const float>,
                                                 Tok8<const float>, const int32_t*,
                                                 const int32_t*, int, const Rope8&, cudaStream_t);
template cudaError_t launch_cache8_append<bf16>(const Cache8&, Tok8<const bf16>, Tok8<const bf16>,
                                                const int32_t*, const int32_t*, int, const Rope8&,
                                                cudaStream_t);

}  // namespace rlt
