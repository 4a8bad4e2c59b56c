// Appending keys and values to the paged 8-bit cache: rotate the keys, find
// each (page, head)'s largest magnitude, choose its power-of-two scale, round
// to e4m3 (include/rlt.h: rlt_cache8_append).
//
// One item is one (row, page touched, head), keys and values: the page's new
// tokens are read once, the keys rotated, both reduced to their largest
// magnitude, and written as bytes, so the bytes moved are the operands' and
// the result's alone.  The kernel is bound by HBM for prompts and by its
// launch for single tokens.  Scales are powers of two so that a page whose
// scale grows as tokens arrive is brought to the new one exactly (e4m3
// exponents shift), but for values that fall into the subnormal range.
//
// A CTA takes one page of one row and walks over its heads, T threads to an
// item: while one item is worked on, the next one's values are on their way to
// shared memory by asynchronous copies, into slots that the copying thread
// alone reads back (no barrier but the one of the item's maxima).  The page's
// cosines and sines stay in registers for all heads.
//
// A thread holds 16 key values of one token, as 8/V units, and the same 16
// value values: key dims a..a+V-1 and b..b+V-1 where, in the half layout,
// b = a + rot/2 (the rotation partners), else b = a + V.  V = 8 (16-byte copies
// of bf16), or 4 where rot is no multiple of 16.  T is the power of two that
// holds a page: one warp per item for generated tokens, 512 threads for pages
// of 64 x 128.  (K and V as items of their own, one unit of 16 a thread: 313
// instructions a unit, most of them for addresses, and 3.6 TB/s.)
#include <cuda_fp8.h>

#include <algorithm>

#include "cache8.cuh"

namespace rlt {
namespace {

constexpr int kLeastExp = -110, kMostExp = 120;

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}

// two fp32 values in one register pair: one instruction for both, each rounded by itself
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(lo), "f"(hi));
    return p;
}
__device__ __forceinline__ void unpair(uint64_t p, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// V values of T_ in pieces of at most 16 bytes; piece p of a thread is `pitch` behind piece p - 1,
// so that neighbouring threads' pieces are neighbours
template <typename T_, int V>
struct Half {
    static constexpr int BYTES = V * sizeof(T_) < 16 ? V * (int)sizeof(T_) : 16;
    static constexpr int PIECES = V * (int)sizeof(T_) / BYTES;
    static __device__ __forceinline__ void fetch(uint32_t slot, int pitch, const T_* p) {
#pragma unroll
        for (int i = 0; i < PIECES; ++i)
            copy_async<BYTES>(slot + i * pitch, p + i * (BYTES / (int)sizeof(T_)));
    }
    // value e goes to x[e]; with EVEN, even ones to x and odd ones to y
    template <bool EVEN>
    static __device__ __forceinline__ void get(const uint8_t* slot, int pitch, float* x, float* y) {
        float f[V];
        if constexpr (sizeof(T_) == 4) {
#pragma unroll
            for (int i = 0; i < PIECES; ++i) {
                const float4 v = *reinterpret_cast<const float4*>(slot + i * pitch);
                f[4 * i] = v.x, f[4 * i + 1] = v.y, f[4 * i + 2] = v.z, f[4 * i + 3] = v.w;
            }
        } else {
            uint32_t w[V / 2];
            if constexpr (V == 8) {
                const uint4 v = *reinterpret_cast<const uint4*>(slot);
                w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
            } else {
                const uint2 v = *reinterpret_cast<const uint2*>(slot);
                w[0] = v.x, w[1] = v.y;
            }
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                f[2 * i] = __uint_as_float(w[i] << 16);
                f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        }
#pragma unroll
        for (int e = 0; e < V; ++e) {
            if (EVEN) (e & 1 ? y : x)[e / 2] = f[e];
            else x[e] = f[e];
        }
    }
};

__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
    uint32_t r;
    asm("{\n"
        ".reg .b16 l, h;\n"
        "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n"
        "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n"
        "mov.b32 %0, {l, h};\n"
        "}\n"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
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

// The scale of a page whose new tokens' largest magnitude has the bits `top`, and its reciprocal:
// the smallest 2^e, e in [least, most], with top <= 448 * 2^e = 1.75 * 2^(e+8).  Mantissas above
// 1.75 carry into the exponent; infinity comes out as the largest finite value does.
__device__ __forceinline__ float scale_of(uint32_t top, float& inv) {
    int field = (int)((top + 0x1fffffu) >> 23) - 8;
    field = max(kLeastExp + 127, min(kMostExp + 127, field));
    inv = __uint_as_float((uint32_t)(254 - field) << 23);
    return __uint_as_float((uint32_t)field << 23);
}

// T threads per item; a CTA's groups of T take every GROUPS-th head
template <typename T_, int V, int T>
struct Shape {
    static constexpr int THREADS = T < 256 ? 256 : T, GROUPS = THREADS / T, Q = 8 / V;
    static constexpr int KEYS = 16 * (int)sizeof(T_) * THREADS;     // of every thread; values as many
    static constexpr int STAGE = 2 * KEYS;
    static constexpr int STAGES = STAGE <= 65536 ? 2 : 1;
};

template <typename T_, int V, int T>
__global__ void __launch_bounds__(Shape<T_, V, T>::THREADS, 1024 / Shape<T_, V, T>::THREADS)
k_cache8_append(Cache8 c, Tok8<const T_> k, Tok8<const T_> v, const int32_t* __restrict__ start,
                const int32_t* __restrict__ counts, int n, int page_log2, int row_blocks, int parts,
                Rope8 rope) {
    using S = Shape<T_, V, T>;
    using H = Half<T_, V>;
    using H8 = Half<T_, 8>;
    constexpr int PITCH = H::BYTES * S::THREADS, HALF = V * (int)sizeof(T_) * S::THREADS, Q = S::Q;
    constexpr int PITCH8 = 16 * S::THREADS, HALF8 = 8 * (int)sizeof(T_) * S::THREADS;
    extern __shared__ __align__(16) uint8_t smem[];     // STAGES x (keys, values)
    __shared__ uint32_t s_top[2][2][S::THREADS / 32];
    pdl_enter();
    const int sub = (int)threadIdx.x / T, tid = (int)threadIdx.x % T;
    const int part = (int)blockIdx.x % parts, rb = (int)blockIdx.x / parts;
    const int row = rb / row_blocks, j = rb % row_blocks;
    const int s0 = __ldg(start + row);
    const int cnt = counts ? __ldg(counts + row) : n;
    const bool first = threadIdx.x == 0 && part == 0;
    auto say = [&](int code) {
        if (first && c.status) atomicCAS(c.status, 0, code);
    };
    const int cap = c.row_pages << page_log2;
    if (cnt < 0 || cnt > n || s0 < 0 || s0 > cap || cnt > cap - s0) {
        // the tokens within the capacity are still written when the counts are sane
        if (j == 0) say(c.cap_code);
        if (cnt < 0 || cnt > n || s0 < 0 || s0 >= cap) return;
    }
    const int end = min(cap, s0 + cnt);
    const int block = (s0 >> page_log2) + j;
    int lo = max(s0, block << page_log2);
    int hi = min(end, (block + 1) << page_log2);
    if (rope.rot) {                                  // positions without a row in the table
        const int plo = -rope.origin, phi = rope.positions - rope.origin;
        if (lo < hi && (lo < plo || hi > phi)) say(c.cap_code);
        lo = max(lo, plo);
        hi = min(hi, phi);
    }
    if (lo >= hi) return;
    const int pg = __ldg(c.table + (size_t)row * c.row_pages + block);

    // this thread's values: dims [16 u, 16 u + 16) of V, units Q u .. Q u + Q - 1 of K, of token
    // lo + tok
    const int dh = c.dh, log2_per = dh == 128 ? 3 : 2;
    const int u = tid & ((1 << log2_per) - 1), tok = tid >> log2_per;
    const bool here = tok < hi - lo;
    const bool halves = !rope.interleaved;
    int ka[Q], kb[Q];
    bool turns[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int w = Q * u + q;
        turns[q] = 2 * V * w < rope.rot;
        ka[q] = turns[q] && halves ? V * w : 2 * V * w;
        kb[q] = turns[q] && halves ? V * w + (rope.rot >> 1) : 2 * V * w + V;
    }
    const int per = (c.kv_heads + parts - 1) / parts;
    const int h_end = min(c.kv_heads, (part + 1) * per);
    int h = part * per + sub, hf = h;                // the head worked on, the head fetched
    const T_* kp = k.p + (int64_t)row * k.row + (int64_t)(lo - s0 + tok) * k.token + (int64_t)h * dh;
    const T_* vp = v.p + (int64_t)row * v.row + (int64_t)(lo - s0 + tok) * v.token + (int64_t)h * dh +
                   16 * u;
    const uint32_t smem_u = (uint32_t)__cvta_generic_to_shared(smem);
    const uint32_t kslot = smem_u + threadIdx.x * H::BYTES;
    const uint32_t vslot = smem_u + S::KEYS + threadIdx.x * 16;
    auto fetch = [&](int stage) {
        if (here && hf < h_end) {
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                H::fetch(kslot + stage + 2 * q * HALF, PITCH, kp + ka[q]);
                H::fetch(kslot + stage + (2 * q + 1) * HALF, PITCH, kp + kb[q]);
            }
            H8::fetch(vslot + stage, PITCH8, vp);
            H8::fetch(vslot + stage + HALF8, PITCH8, vp + 8);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        hf += S::GROUPS;
        kp += S::GROUPS * dh;
        vp += S::GROUPS * dh;
    };
    fetch(0);
    float cs[8], sn[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) cs[e] = 1.f, sn[e] = 0.f;
#pragma unroll
    for (int e = 0; e < 8; e += 4) {
        if (turns[e / V] && here) {
            const size_t from =
                (size_t)(lo + tok + rope.origin) * (rope.rot >> 1) + (size_t)(8 * u + e);
            const float4 a = __ldg(reinterpret_cast<const float4*>(rope.cs + from));
            const float4 b = __ldg(reinterpret_cast<const float4*>(rope.sn + from));
            cs[e] = a.x, cs[e + 1] = a.y, cs[e + 2] = a.z, cs[e + 3] = a.w;
            sn[e] = b.x, sn[e + 1] = b.y, sn[e + 2] = b.z, sn[e + 3] = b.w;
        }
    }
    if (pg < 0 || pg >= c.n_pages) {                 // the same for the whole CTA
        say(c.arg_code);
        asm volatile("cp.async.wait_all;" ::: "memory");
        return;
    }
    const int kept = s0 - (block << page_log2);      // tokens of the row that the page already holds
    const size_t head_bytes = (size_t)dh << page_log2, v_heads = c.kv_heads;
    const size_t head0 = (size_t)pg * 2 * c.kv_heads + h;
    float* scale_at = c.scales + head0;
    uint8_t* page_at = c.pages + head0 * head_bytes;
    const uint32_t in_page = (uint32_t)((lo - (block << page_log2) + tok) * dh);

    // the scale of a head's keys (or values): grown, never shrunk, where the page holds tokens
    auto settle = [&](uint32_t top, float old, float& inv, float* at, uint8_t* bytes) {
        float scale = scale_of(top, inv);
        if (kept > 0 && old > 0.f) {
            if (old >= scale) {
                scale = old;
                inv = 1.f / old;                     // (the caller's own need not be a power of two)
            } else {
                const float f = old / scale;
                uint4* q = reinterpret_cast<uint4*>(bytes);
                for (int e = tid; e < kept * dh / 16; e += T) {
                    uint4 w = q[e];
                    w.x = rescale4(w.x, f);
                    w.y = rescale4(w.y, f);
                    w.z = rescale4(w.z, f);
                    w.w = rescale4(w.w, f);
                    q[e] = w;
                }
            }
        }
        if (tid == 0) *at = scale;
    };
    int stage = 0;
    for (int it = 0; it < (per + S::GROUPS - 1) / S::GROUPS; ++it) {
        if constexpr (S::STAGES == 2) fetch(S::STAGE - stage);
        const bool live = h < h_end;                 // (a group past the end still meets the barrier)
        float old_k = 0.f, old_v = 0.f;
        if (live && kept > 0) old_k = __ldcg(scale_at), old_v = __ldcg(scale_at + v_heads);
        asm volatile("cp.async.wait_group %0;" ::"n"(S::STAGES - 1) : "memory");
        const uint8_t* ks = smem + stage + threadIdx.x * H::BYTES;
        const uint8_t* vs = smem + stage + S::KEYS + threadIdx.x * 16;
        // keys: rotation pairs (x[e], y[e]): neighbours in the interleaved layout, else the halves'
        float x[8], y[8];
        uint32_t top_k = 0, top_v = 0;
        if (live && here) {
            float m = 0.f, z[16];
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                if (halves) {
                    H::template get<false>(ks + 2 * q * HALF, PITCH, x + V * q, nullptr);
                    H::template get<false>(ks + (2 * q + 1) * HALF, PITCH, y + V * q, nullptr);
                } else {
                    H::template get<true>(ks + 2 * q * HALF, PITCH, x + V * q, y + V * q);
                    H::template get<true>(ks + (2 * q + 1) * HALF, PITCH, x + V * q + V / 2,
                                          y + V * q + V / 2);
                }
                if (turns[q]) {
#pragma unroll
                    for (int e = V * q; e < V * q + V; e += 2) {
                        // products and sums rounded one by one, not contracted: the bytes do
                        // not depend on how a compiler fuses the pair (packed sums it does fuse)
                        const uint64_t x1 = pair(x[e], x[e + 1]), x2 = pair(y[e], y[e + 1]);
                        const uint64_t c1 = pair(cs[e], cs[e + 1]), s1 = pair(sn[e], sn[e + 1]);
                        float a[2], b[2], c[2], d[2];
                        unpair(mul2(x1, c1), a[0], a[1]);
                        unpair(mul2(x2, s1), b[0], b[1]);
                        unpair(mul2(x2, c1), c[0], c[1]);
                        unpair(mul2(x1, s1), d[0], d[1]);
                        x[e] = __fsub_rn(a[0], b[0]), x[e + 1] = __fsub_rn(a[1], b[1]);
                        y[e] = __fadd_rn(c[0], d[0]), y[e + 1] = __fadd_rn(c[1], d[1]);
                    }
                }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) m = fmaxf(m, fmaxf(fabsf(x[e]), fabsf(y[e])));  // skips NaN
            top_k = __float_as_uint(m);              // magnitudes order as their bits
            m = 0.f;
            H8::template get<false>(vs, PITCH8, z, nullptr);
            H8::template get<false>(vs + HALF8, PITCH8, z + 8, nullptr);
#pragma unroll
            for (int e = 0; e < 16; ++e) m = fmaxf(m, fabsf(z[e]));
            top_v = __float_as_uint(m);
        }
        top_k = __reduce_max_sync(0xffffffffu, top_k);
        top_v = __reduce_max_sync(0xffffffffu, top_v);
        if constexpr (T > 32) {                      // two buffers: one barrier an item is enough
            const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
            auto& w = s_top[it & 1];
            if (lane == 0) w[0][warp] = top_k, w[1][warp] = top_v;
            __syncthreads();
            const int from = sub * (T / 32) + (lane & (T / 32 - 1));
            top_k = __reduce_max_sync(0xffffffffu, w[0][from]);
            top_v = __reduce_max_sync(0xffffffffu, w[1][from]);
        } else {
            __syncwarp();                            // every lane has read the old scales
        }
        if (live) {
            float inv;
            settle(top_k, old_k, inv, scale_at, page_at);
            if (here) {
                const uint64_t f = pair(inv, inv);
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    unpair(mul2(pair(x[e], x[e + 1]), f), x[e], x[e + 1]);
                    unpair(mul2(pair(y[e], y[e + 1]), f), y[e], y[e + 1]);
                }
                uint8_t* at = page_at + in_page;
                if (halves) {
                    w[0] = to_e4m3x4(x[0], x[1], x[2], x[3]);
                    w[1] = to_e4m3x4(x[4], x[5], x[6], x[7]);
                    w[2] = to_e4m3x4(y[0], y[1], y[2], y[3]);
                    w[3] = to_e4m3x4(y[4], y[5], y[6], y[7]);
                    if constexpr (V == 8) {
                        *reinterpret_cast<uint2*>(at + ka[0]) = make_uint2(w[0], w[1]);
                        *reinterpret_cast<uint2*>(at + kb[0]) = make_uint2(w[2], w[3]);
                    } else {
#pragma unroll
                        for (int q = 0; q < Q; ++q) {
                            *reinterpret_cast<uint32_t*>(at + ka[q]) = w[q];
                            *reinterpret_cast<uint32_t*>(at + kb[q]) = w[2 + q];
                        }
                    }
                } else {                             // units side by side
                    w[0] = to_e4m3x4(x[0], y[0], x[1], y[1]);
                    w[1] = to_e4m3x4(x[2], y[2], x[3], y[3]);
                    w[2] = to_e4m3x4(x[4], y[4], x[5], y[5]);
                    w[3] = to_e4m3x4(x[6], y[6], x[7], y[7]);
                    *reinterpret_cast<uint4*>(at + 16 * u) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            uint8_t* v_page = page_at + v_heads * head_bytes;
            settle(top_v, old_v, inv, scale_at + v_heads, v_page);
            if (here) {
                float z[16];
                H8::template get<false>(vs, PITCH8, z, nullptr);
                H8::template get<false>(vs + HALF8, PITCH8, z + 8, nullptr);
                const uint64_t f = pair(inv, inv);
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 16; e += 2) unpair(mul2(pair(z[e], z[e + 1]), f), z[e], z[e + 1]);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    w[e] = to_e4m3x4(z[4 * e], z[4 * e + 1], z[4 * e + 2], z[4 * e + 3]);
                *reinterpret_cast<uint4*>(v_page + in_page + 16 * u) =
                    make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        if constexpr (S::STAGES == 1) fetch(0);
        else stage = S::STAGE - stage;
        h += S::GROUPS;
        scale_at += S::GROUPS;
        page_at += S::GROUPS * head_bytes;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

}  // namespace

template <typename T>
cudaError_t launch_cache8_append(const Cache8& c, Tok8<const T> k, Tok8<const T> v,
                                 const int32_t* start, const int32_t* counts, int n,
                                 const Rope8& rope, cudaStream_t st) {
    if (c.rows <= 0 || n <= 0) return cudaSuccess;
    // pages a row can touch: n tokens from any slot of the first one
    const int row_blocks = (int)std::min<int64_t>(c.row_pages, ((int64_t)n + c.page - 2) / c.page + 1);
    const int64_t blocks = (int64_t)c.rows * row_blocks;
    int page_log2 = 4;
    while ((1 << page_log2) < c.page) ++page_log2;
    auto go = [&](auto kern, auto shape) {
        using S = decltype(shape);
        // parts that share a page's heads: enough CTAs to fill the SMs (1024 threads each) four
        // times over while a group keeps two items to overlap; for few pages one item a group
        const auto ceil_to = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
        const int64_t fill = 148 * (1024 / S::THREADS);
        int64_t parts = std::min<int64_t>(ceil_to(4 * fill, blocks),
                                          std::max(1, c.kv_heads / (2 * S::GROUPS)));
        if (blocks * parts < fill)
            parts = std::min<int64_t>(ceil_to(fill, blocks), ceil_to(c.kv_heads, S::GROUPS));
        if (blocks * parts > 0x7fffffff) return cudaErrorInvalidConfiguration;
        const size_t smem = S::STAGES * S::STAGE;
        if (!set_smem_once(reinterpret_cast<const void*>(kern), smem))
            return cudaErrorInvalidConfiguration;
        cudaError_t e = launch(kern, (unsigned)(blocks * parts), S::THREADS, smem, st, c, k, v, start,
                               counts, n, page_log2, row_blocks, (int)parts, rope);
        if (e == cudaSuccess) rlt_count_launch();
        return e;
    };
    const int units = std::min(n, c.page) * (c.dh / 16);    // threads of an item
#define RLT_RUN(V)                                                                       \
    (units <= 32    ? go(k_cache8_append<T, V, 32>, Shape<T, V, 32>{})                   \
     : units <= 64  ? go(k_cache8_append<T, V, 64>, Shape<T, V, 64>{})                   \
     : units <= 128 ? go(k_cache8_append<T, V, 128>, Shape<T, V, 128>{})                 \
     : units <= 256 ? go(k_cache8_append<T, V, 256>, Shape<T, V, 256>{})                 \
     : units <= 512 ? go(k_cache8_append<T, V, 512>, Shape<T, V, 512>{})                 \
                    : go(k_cache8_append<T, V, 1024>, Shape<T, V, 1024>{}))
    return rope.rot % 16 == 0 ? RLT_RUN(8) : RLT_RUN(4);    // else a unit of 16 would turn in part
#undef RLT_RUN
}

template cudaError_t launch_cache8_append<float>(const Cache8&, Tok8<const float>,
                                                 Tok8<const float>, const int32_t*,
                                                 const int32_t*, int, const Rope8&, cudaStream_t);
template cudaError_t launch_cache8_append<bf16>(const Cache8&, Tok8<const bf16>, Tok8<const bf16>,
                                                const int32_t*, const int32_t*, int, const Rope8&,
                                                cudaStream_t);

}  // namespace rlt
