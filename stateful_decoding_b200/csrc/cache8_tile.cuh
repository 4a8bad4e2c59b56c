// Pieces that the kernels of attention over the paged 8-bit cache share.
#pragma once

#include <cuda_fp16.h>
#include <math.h>

#include "cache8.cuh"
#include "tc_common.cuh"

namespace rlt {
namespace {

constexpr int kTile = 16;               // keys per step of a warp

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(valid ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// a positive scale as m * 2^e, m in [1, 2) (subnormal ones are 2^-64 times a normal one)
__device__ __forceinline__ void split_scale(float v, float& m, float& e) {
    const bool small = v < 0x1p-126f;
    const uint32_t u = __float_as_uint(small ? v * 0x1p64f : v);
    m = __uint_as_float((u & 0x7fffffu) | 0x3f800000u);
    e = (float)((int)((u >> 23) & 255u) - (small ? 191 : 127));
}
// four e4m3 bytes as two pairs of fp16 values, exactly (NaN stays NaN)
__device__ __forceinline__ void h2x2_of(uint32_t four, uint32_t& lo, uint32_t& hi) {
    asm("{\n"
        ".reg .b16 a, b;\n"
        "mov.b32 {a, b}, %2;\n"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n"
        "}\n"
        : "=r"(lo), "=r"(hi)
        : "r"(four));
}
// the transpose of an 8x8 matrix of fp16 held two to a lane
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_h2(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
// the bits below fp16's 11, times 2^11
__device__ __forceinline__ uint32_t rest_h2(float lo, float hi, uint32_t lead) {
    const float2 f = unpack_h2(lead);
    return pack_h2((lo - f.x) * 2048.f, (hi - f.y) * 2048.f);
}

template <typename TQ>
struct QIn {
    const TQ* p;
    int64_t row, token;
    int slabs;              // partial sums to add (1: q itself)
    size_t slab;
};
__device__ __forceinline__ void load4(const QIn<float>& q, size_t at, float (&x)[4]) {
    float4 v = __ldg(reinterpret_cast<const float4*>(q.p + at));
    for (int s = 1; s < q.slabs; ++s) {
        const float4 w = __ldg(reinterpret_cast<const float4*>(q.p + (size_t)s * q.slab + at));
        v.x += w.x; v.y += w.y; v.z += w.z; v.w += w.w;
    }
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
}
__device__ __forceinline__ void load4(const QIn<bf16>& q, size_t at, float (&x)[4]) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(q.p + at));
    x[0] = __uint_as_float(v.x << 16);
    x[1] = __uint_as_float(v.x & 0xffff0000u);
    x[2] = __uint_as_float(v.y << 16);
    x[3] = __uint_as_float(v.y & 0xffff0000u);
}

// Dims d..d+3 (d a multiple of 4) of a query, rotated at its position: loads and arithmetic apart,
// so that the loads' latency overlaps what stands between.
template <typename TQ>
struct Q4 {
    float x[4], y[4], c[4], s[4];           // the dims, their partners, cosines and sines
    __device__ __forceinline__ void load(const QIn<TQ>& q, size_t at, int d, const Rope8& r, int pos) {
        load4(q, at + d, x);
        if (d >= r.rot) return;
        const int half = r.rot >> 1;
        const size_t row = (size_t)pos * half;
        if (r.interleaved) {
            const float2 a = __ldg(reinterpret_cast<const float2*>(r.cs + row + d / 2));
            const float2 b = __ldg(reinterpret_cast<const float2*>(r.sn + row + d / 2));
            c[0] = a.x, c[1] = a.y, s[0] = b.x, s[1] = b.y;
        } else {
            const bool low = d < half;
            load4(q, at + (low ? d + half : d - half), y);
            const size_t from = row + (low ? d : d - half);
            const float4 a = __ldg(reinterpret_cast<const float4*>(r.cs + from));
            const float4 b = __ldg(reinterpret_cast<const float4*>(r.sn + from));
            c[0] = a.x, c[1] = a.y, c[2] = a.z, c[3] = a.w;
            s[0] = b.x, s[1] = b.y, s[2] = b.z, s[3] = b.w;
        }
    }
    __device__ __forceinline__ float4 turned(int d, const Rope8& r) {
        if (d < r.rot) {
            if (r.interleaved) {
                rope_pair(x[0], x[1], c[0], s[0], x[0], x[1]);
                rope_pair(x[2], x[3], c[1], s[1], x[2], x[3]);
            } else {
                const bool low = d < (r.rot >> 1);
                float unused;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (low) rope_pair(x[e], y[e], c[e], s[e], x[e], unused);
                    else rope_pair(y[e], x[e], c[e], s[e], unused, x[e]);
                }
            }
        }
        return make_float4(x[0], x[1], x[2], x[3]);
    }
};

// Where a lane's pieces of a 16-key tile go in shared memory (K rows, then V rows): key rows and
// 16-byte chunks are permuted on the way in so that every fragment load is one conflict-free wide
// load.  Lane (g, t) = (lane/4, lane%4) reads dims [t D/4, (t+1) D/4) of key rows g and g + 8,
// and dims [g D/8, (g+1) D/8) of values 4i + t; key row r holds key
// sigma(r) = (r & 8) + 4 (r & 1) + (r & 7) / 2, the order the weights' transpose wants.
template <int D>
struct TileCopy {
    static constexpr int CPR = D / 16, RS = 32 / CPR, NK = kTile / RS;  // chunks per row, rows per pass
    int cr;
    uint32_t k_off[2], v_off;
    __device__ __forceinline__ explicit TileCopy(int lane) {
        cr = lane / CPR;
        const int ch = lane % CPR;
        if constexpr (D == 128) {           // rows cr + 4k -> 2 cr + (k & 1) + 8 (k / 2)
            k_off[0] = (uint32_t)(2 * cr * D + ch * 16);
            k_off[1] = (uint32_t)((2 * cr + 1) * D + (ch ^ 1) * 16);
            v_off = (uint32_t)(kTile * D + cr * D + (ch ^ (cr << 1)) * 16);
        } else {                            // rows cr + 8k -> 2 (cr & 3) + cr / 4 + 8k
            k_off[0] = (uint32_t)((((cr & 3) << 1) | (cr >> 2)) * D + ch * 16);
            k_off[1] = k_off[0] + 8 * D;
            v_off = (uint32_t)(kTile * D + cr * D + (ch ^ (cr & 2)) * 16);
        }
    }
    // the lane's chunks of keys kg and values vg (its own chunk of the tile's first rows) to the
    // tile at `at`; keys from `left` on are zero-filled rather than read
    __device__ __forceinline__ void operator()(uint32_t at, const uint8_t* kg, const uint8_t* vg,
                                               int left, const uint8_t* any) const {
        const bool whole = left >= kTile;
#pragma unroll
        for (int k = 0; k < NK; ++k) {
            const uint32_t kd = D == 128 ? k_off[k & 1] + (k >> 1) * 8 * D : k_off[k];
            const bool ok = whole || cr + k * RS < left;
            cp16(at + kd, ok ? kg + k * 512 : any, ok);
            cp16(at + v_off + k * RS * D, ok ? vg + k * 512 : any, ok);
        }
    }
};

// the fragments of a tile at `st`: chunk h of key rows g, g + 8; values 4i + t
template <int D>
__device__ __forceinline__ void load_keys(const uint8_t* st, int g, int t, int h, uint4& x,
                                          uint4& y) {
    const int kc = D == 128 ? (2 * t + h) ^ (g & 1) : t;
    x = *reinterpret_cast<const uint4*>(st + g * D + kc * 16);
    y = *reinterpret_cast<const uint4*>(st + (g + 8) * D + kc * 16);
}
template <int D>
__device__ __forceinline__ void load_values(const uint8_t* st, int g, int t,
                                            uint32_t (&vv)[4][D / 32]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint8_t* vp = st + kTile * D + (4 * i + t) * D;
        if constexpr (D == 128) {
            const uint4 v4 = *reinterpret_cast<const uint4*>(vp + ((g ^ (2 * t)) << 4));
            vv[i][0] = v4.x, vv[i][1] = v4.y, vv[i][2] = v4.z, vv[i][3] = v4.w;
        } else {
            const uint2 v2 =
                *reinterpret_cast<const uint2*>(vp + (((g >> 1) ^ (t & 2)) << 4) + ((g & 1) << 3));
            vv[i][0] = v2.x, vv[i][1] = v2.y;
        }
    }
}
// A value seen by some queries only: a NaN in it would reach the others as 0 x NaN, so it enters
// the product as 0; returned are the tile's keys (bits) with one, whose weights become NaN.
template <int D>
__device__ __forceinline__ uint32_t clear_nan(uint32_t (&vv)[4][D / 32], int t) {
    uint32_t poison = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t hit = 0;
#pragma unroll
        for (int x = 0; x < D / 32; ++x) {
            const uint32_t z = ((vv[i][x] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
            hit |= z;
            vv[i][x] &= ~((z >> 7) * 0xffu);
        }
        if (hit) poison |= 1u << (4 * i + t);
    }
    return __reduce_or_sync(0xffffffffu, poison);
}

}  // namespace
}  // namespace rlt
