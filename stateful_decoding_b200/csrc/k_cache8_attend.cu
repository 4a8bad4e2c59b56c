// Attention over the paged 8-bit cache (include/rlt.h: rlt_cache8_attend).
//
// Mathematics.  With byte values x, key scales ks and value scales vs per
// (page, head), o = sum_j p_j vs_j x^v_j / sum_j p_j, p_j = 2^(s_j),
// s_j = scale log2(e) ks_j q.x^k_j.  The value scale is folded into the
// exponent: w_j = 2^(s_j + log2 vs_j - m) with m a running maximum of
// s + log2 vs, so that o = sum w_j x^v_j / sum (w_j / vs_j): bytes enter the
// two products as they are (e4m3 is exact in fp16), a 16-key tile needs two
// scalars per head, and w stays within fp16's range whatever the scales.
//
// Matrix form.  One warp takes 16 keys at a time through m16n8k16 fp16
// products with fp32 sums: a single decoded token fills one row of 16, but
// converting a byte pair to fp16 is one instruction where multiplying it in
// fp32 on the CUDA cores would take four, so the tensor cores carry the
// per-key work of an HBM stream.  The unused rows buy precision: up to 8
// query vectors per key head (SPLIT) occupy rows 0-7 with the leading 11 bits
// of q (of w), rows 8-15 with the next 11 bits times 2^11, and the two rows'
// sums are added in fp32.  More than 8 bf16 queries fill 16 rows with the
// leading bits alone: a bf16 q is exact there (each row is brought near 1 by
// a power of two first), w is rounded to fp16 (2^-11 relative at most, below
// the bf16 output's 2^-9 step); fp32 types always run SPLIT.
//
// The maximum is raised only when a score passes it by 2^8 (one warp vote per
// tile instead of a reduction); fp16 holds weights up to 2^16.
//
// Data path.  Tiles reach a per-warp ring in shared memory by 16-byte
// cp.async copies; keys past the prefix and keys in bad pages are zero-filled
// rather than read, so whatever bytes sit there never enter a product.  Key
// rows and 16-byte chunks are permuted on the way in (krow, kchunk, vchunk)
// so that every fragment load is one conflict-free wide load: lane (g, t) =
// (lane/4, lane%4) reads dims [t D/4, (t+1) D/4) of its key and of its query
// row, and dims [g D/8, (g+1) D/8) of values 4i+t.
//
// Split.  The prefix of a (row, key head) is cut into runs for 4 warps of
// ceil(keys / 1024) CTAs (at most 16), a function of that prefix alone.  The
// warps' partial results meet in shared memory, the CTAs' through the
// cluster's distributed shared memory, always in run order: no scratch, no
// atomics, and the same bits for a row whatever batch or capacity it sits in.
#include <cooperative_groups.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math.h>

#include <algorithm>

#include "cache8.cuh"
#include "tc_common.cuh"

namespace cg = cooperative_groups;

namespace rlt {
namespace {

constexpr int kWarps = 4;
constexpr int kTile = 16;               // keys per step of a warp
constexpr int kKeysPerCta = 1024;
constexpr int kMaxCtas = 16;            // CTAs per (row, key head, query tile): one cluster
constexpr float kLag = 8.f;             // how far (log2) a score may pass the maximum

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
// two e4m3 bytes (the low 16 bits) as two fp16 values, exactly
__device__ __forceinline__ uint32_t h2_of(uint32_t two) {
    const __half2_raw h =
        __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(two & 0xffffu), __NV_E4M3);
    return (uint32_t)h.x | ((uint32_t)h.y << 16);
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

// dims d..d+3 (d a multiple of 4) of the query at `at`, rotated at position pos
template <typename TQ>
__device__ __forceinline__ void load_q4(const QIn<TQ>& q, size_t at, int d, const Rope8& r, int pos,
                                        float (&x)[4]) {
    load4(q, at + d, x);
    if (d >= r.rot) return;
    const int half = r.rot >> 1;
    const float* cs = r.cs + (size_t)pos * half;
    const float* sn = r.sn + (size_t)pos * half;
    if (r.interleaved) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float c = __ldg(cs + d / 2 + e), s = __ldg(sn + d / 2 + e);
            rope_pair(x[2 * e], x[2 * e + 1], c, s, x[2 * e], x[2 * e + 1]);
        }
    } else {
        const bool low = d < half;
        const int a = low ? d : d - half;
        float y[4], unused;
        load4(q, at + (low ? d + half : d - half), y);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float c = __ldg(cs + a + e), s = __ldg(sn + a + e);
            if (low) rope_pair(x[e], y[e], c, s, x[e], unused);
            else rope_pair(y[e], x[e], c, s, unused, x[e]);
        }
    }
}

// where key row r of a tile and its 16-byte chunk c go in shared memory
template <int D>
__device__ __forceinline__ uint32_t k_at(int r, int c) {
    const int pr = (r & 8) | ((r & 3) << 1) | ((r >> 2) & 1);
    return (uint32_t)(pr * D + ((D == 128 ? c ^ (pr & 1) : c) << 4));
}
template <int D>
__device__ __forceinline__ uint32_t v_at(int r, int c) {
    return (uint32_t)(r * D + ((D == 128 ? c ^ ((r & 3) << 1) : c ^ (r & 2)) << 4));
}

template <int D> constexpr int stages() { return D == 64 ? 4 : 3; }
template <int D> constexpr int stage_bytes() { return 2 * kTile * D + 16; }
template <int D> constexpr int ring_bytes() { return kWarps * stages<D>() * stage_bytes<D>(); }

struct Tile8 {              // per-page scalars of a tile, beside it in the ring
    float ks, lv, inv;      // key scale, log2 of the value scale, 1 / value scale
};

template <int D, bool SPLIT, typename TQ, typename TO>
__global__ void __launch_bounds__(kWarps * 32)
k_cache8_attend(Cache8 c, int page_log2, QIn<TQ> q, Tok8<TO> out, int share, int n, int q_tiles,
                const int32_t* __restrict__ lens, int lens_add, float scale_log2e, Rope8 rope) {
    constexpr int MT = SPLIT ? 8 : 16;      // query vectors per tile
    constexpr int NST = stages<D>(), SB = stage_bytes<D>(), KI = D / 16, VJ = D / 8;
    extern __shared__ __align__(128) uint8_t smem[];
    pdl_enter();
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int unit = (int)(blockIdx.x / (unsigned)C);
    const int mt = unit % q_tiles, bh = unit / q_tiles;
    const int kvh = bh % c.kv_heads, row = bh / c.kv_heads;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int nq = n * share;

    const int cap = c.row_pages << page_log2;
    const int L0 = __ldg(lens + row) + lens_add;
    const int L = max(0, min(cap, L0));
    if ((L0 < 0 || L0 > cap) && threadIdx.x == 0 && kvh == 0 && mt == 0 && rank == 0 && c.status)
        atomicCAS(c.status, 0, c.cap_code);
    const int r0 = mt * MT, r_last = min(nq, r0 + MT) - 1;
    const int vis_max = max(0, L - n + r_last / share + 1);   // keys any query of the tile sees
    const int vis_min = L - n + r0 / share + 1;               // keys all of them see
    const int nC = min(C, min(kMaxCtas, max(1, (vis_max + kKeysPerCta - 1) / kKeysPerCta)));
    if (rank >= nC) return;
    const int subs = (vis_max + kTile - 1) / kTile, runs = nC * kWarps;
    const int per = (subs + runs - 1) / runs;
    const int s_begin = min(subs, (rank * kWarps + warp) * per), s_end = min(subs, s_begin + per);

    // ---------------------------------------------------------------- tiles
    uint8_t* ring = smem + warp * (NST * SB);
    const uint32_t ring_u = tc::smem_u32(ring);
    const size_t head_bytes = (size_t)D << page_log2;
    int b_base = s_begin;                   // first tile of the batch below
    int b_page = -1;                        // lane l: the page of tile b_base + l, and its scalars
    float b_ks = 0.f, b_lv = -INFINITY, b_inv = 0.f;
    auto load_batch = [&]() {
        b_page = -1;
        b_ks = 0.f, b_lv = -INFINITY, b_inv = 0.f;
        const int s = b_base + lane;
        if (s < s_end) {
            const int p = __ldg(c.table + (size_t)row * c.row_pages + ((s * kTile) >> page_log2));
            if (p >= 0 && p < c.n_pages) {
                const float* sc = c.scales + (size_t)p * 2 * c.kv_heads + kvh;
                b_page = p;
                b_ks = __ldg(sc);
                const float vs = __ldg(sc + c.kv_heads);
                b_lv = log2f(vs);
                b_inv = 1.f / vs;
            } else if (c.status) {
                atomicCAS(c.status, 0, c.arg_code);
            }
        }
    };
    auto issue = [&](int i) {               // tile s_begin + i into stage i % NST
        const int s = s_begin + i;
        if (s < s_end) {
            if (s - b_base == 32) {
                b_base += 32;
                load_batch();
            }
            const int src = s - b_base;
            const int p = __shfl_sync(0xffffffffu, b_page, src);
            const float ks = __shfl_sync(0xffffffffu, b_ks, src);
            const float lv = __shfl_sync(0xffffffffu, b_lv, src);
            const float inv = __shfl_sync(0xffffffffu, b_inv, src);
            const int slot = i % NST, k0 = s * kTile;
            if (lane == 0)
                *reinterpret_cast<float4*>(ring + slot * SB + 2 * kTile * D) =
                    make_float4(ks, lv, inv, 0.f);
            const uint8_t* kg = c.pages + ((size_t)max(p, 0) * 2 * c.kv_heads + kvh) * head_bytes +
                                (size_t)(k0 & ((1 << page_log2) - 1)) * D;
            const uint8_t* vg = kg + (size_t)c.kv_heads * head_bytes;
            const int left = p >= 0 ? vis_max - k0 : 0;
            const uint32_t at = ring_u + slot * SB;
#pragma unroll
            for (int x = lane; x < D; x += 32) {        // D chunks of 16 bytes each
                const int r = x / (D / 16), ch = x % (D / 16);
                const bool ok = r < left;
                cp16(at + k_at<D>(r, ch), ok ? kg + x * 16 : c.pages, ok);
                cp16(at + kTile * D + v_at<D>(r, ch), ok ? vg + x * 16 : c.pages, ok);
            }
        }
        cp_commit();
    };
    load_batch();
#pragma unroll
    for (int i = 0; i < NST - 1; ++i) issue(i);

    // ---------------------------------------------------------------- queries
    // rows g (and, 16 rows, g + 8): this lane's dims [t D/4, (t+1) D/4)
    uint32_t qf[KI][4];
    float rf[SPLIT ? 1 : 2];                // score factor of the row: 2^e scale log2(e)
    int vis[SPLIT ? 1 : 2];                 // keys it sees
#pragma unroll
    for (int w = 0; w < (SPLIT ? 1 : 2); ++w) {
        const int r = r0 + g + 8 * w;
        const int i = r / share, pos = L - n + i + rope.origin;
        float x[KI][4];
        float amax = 0.f;
        vis[w] = r < nq ? max(0, L - n + i + 1) : 0;
        if (vis[w] > 0 && rope.rot && (pos < 0 || pos >= rope.positions)) {
            if (c.status) atomicCAS(c.status, 0, c.cap_code);
            vis[w] = 0;
        }
#pragma unroll
        for (int k = 0; k < KI; ++k) {
            if (vis[w] > 0) {
                const size_t at = (size_t)((int64_t)row * q.row + (int64_t)i * q.token) +
                                  (size_t)(kvh * share + r % share) * D;
                load_q4(q, at, t * (D / 4) + 4 * k, rope, pos, x[k]);
            } else {
                x[k][0] = x[k][1] = x[k][2] = x[k][3] = 0.f;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) amax = fmaxf(amax, fabsf(x[k][e]));
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        // bring the row near 1 by a power of two (exact); 2^±100 bounds keep both factors finite
        int e2 = (int)(__float_as_uint(amax) >> 23) - 127;
        e2 = max(-100, min(100, e2));
        const float down = __uint_as_float((uint32_t)(127 - e2) << 23);
        rf[w] = __uint_as_float((uint32_t)(127 + e2) << 23) * scale_log2e;
#pragma unroll
        for (int k = 0; k < KI; ++k) {
#pragma unroll
            for (int e = 0; e < 4; ++e) x[k][e] *= down;
            const uint32_t h0 = pack_h2(x[k][0], x[k][1]), h1 = pack_h2(x[k][2], x[k][3]);
            if (SPLIT) {
                qf[k][0] = h0;
                qf[k][2] = h1;
                qf[k][1] = rest_h2(x[k][0], x[k][1], h0);
                qf[k][3] = rest_h2(x[k][2], x[k][3], h1);
            } else {
                qf[k][0 + w] = h0;
                qf[k][2 + w] = h1;
            }
        }
    }

    // a query without a rotation sees nothing: its row has to be masked from the first key on
    const bool dead = vis[0] < min(vis_min, r0 + g < nq ? vis_min : 0) ||
                      (!SPLIT && vis[SPLIT ? 0 : 1] < min(vis_min, r0 + g + 8 < nq ? vis_min : 0));
    const int mask_from = __any_sync(0xffffffffu, dead) ? 0 : vis_min;

    // ---------------------------------------------------------------- the run
    float m[SPLIT ? 1 : 2], l[SPLIT ? 1 : 2], O[VJ][4];
#pragma unroll
    for (int w = 0; w < (SPLIT ? 1 : 2); ++w) m[w] = -INFINITY, l[w] = 0.f;
#pragma unroll
    for (int j = 0; j < VJ; ++j) O[j][0] = O[j][1] = O[j][2] = O[j][3] = 0.f;

    for (int it = 0; s_begin + it < s_end; ++it) {
        cp_wait<NST - 2>();
        __syncwarp();                       // the tile is here; every lane has left the last one
        issue(it + NST - 1);
        const uint8_t* st = ring + (it % NST) * SB;
        const float4 meta = *reinterpret_cast<const float4*>(st + 2 * kTile * D);
        const int k0 = (s_begin + it) * kTile;

        float cf[2][4];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            cf[u][0] = cf[u][1] = cf[u][2] = cf[u][3] = 0.f;
            const int pr = 8 * u + g;       // the permuted row that holds this lane's key
#pragma unroll
            for (int h = 0; h < D / 64; ++h) {
                const int ch = D == 128 ? (2 * t + h) ^ (pr & 1) : t;
                const uint4 kk = *reinterpret_cast<const uint4*>(st + pr * D + ch * 16);
                mma_f16(cf[u], qf[4 * h + 0], h2_of(kk.x), h2_of(kk.x >> 16));
                mma_f16(cf[u], qf[4 * h + 1], h2_of(kk.y), h2_of(kk.y >> 16));
                mma_f16(cf[u], qf[4 * h + 2], h2_of(kk.z), h2_of(kk.z >> 16));
                mma_f16(cf[u], qf[4 * h + 3], h2_of(kk.w), h2_of(kk.w >> 16));
            }
        }
        // values 4i + t, dims [g D/8, (g+1) D/8)
        uint32_t vv[4][D / 32];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint8_t* vp = st + kTile * D + (4 * i + t) * D;
            if constexpr (D == 128) {
                const uint4 v4 = *reinterpret_cast<const uint4*>(vp + ((g ^ (2 * t)) << 4));
                vv[i][0] = v4.x, vv[i][1] = v4.y, vv[i][2] = v4.z, vv[i][3] = v4.w;
            } else {
                const uint2 v2 = *reinterpret_cast<const uint2*>(
                    vp + (((g >> 1) ^ (t & 2)) << 4) + ((g & 1) << 3));
                vv[i][0] = v2.x, vv[i][1] = v2.y;
            }
        }
        // scores of keys 4i + t (i = 2u + e), the value scale folded in
        float s[SPLIT ? 1 : 2][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int u = i >> 1, e = i & 1;
            if (SPLIT) {
                s[0][i] = fmaf(fmaf(cf[u][2 + e], 1.f / 2048.f, cf[u][e]), rf[0] * meta.x, meta.y);
            } else {
                s[0][i] = fmaf(cf[u][e], rf[0] * meta.x, meta.y);
                s[SPLIT ? 0 : 1][i] = fmaf(cf[u][2 + e], rf[SPLIT ? 0 : 1] * meta.x, meta.y);
            }
        }
        const bool bad = !(meta.y > -INFINITY);
        float poison[4] = {0.f, 0.f, 0.f, 0.f};
        if (bad || k0 + kTile > mask_from) {  // the prefix ends in this tile for some query
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int key = k0 + 4 * i + t;
#pragma unroll
                for (int w = 0; w < (SPLIT ? 1 : 2); ++w)
                    if (bad || key >= vis[w]) s[w][i] = -INFINITY;
            }
            // A value seen by some queries only: a NaN in it would reach the others as
            // 0 x NaN, so it enters the product as 0 and the weights of those that see it
            // become NaN.
            if (vis_min < vis_max) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t hit = 0;
#pragma unroll
                    for (int x = 0; x < D / 32; ++x) {
                        const uint32_t z = ((vv[i][x] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                        hit |= z;
                        vv[i][x] &= ~((z >> 7) * 0xffu);
                    }
                    const uint32_t any = __ballot_sync(0xffffffffu, hit != 0);
                    if (any & (0x11111111u << t)) poison[i] = NAN;
                }
            }
        }
        float mx[SPLIT ? 1 : 2];
        bool raise = false;
#pragma unroll
        for (int w = 0; w < (SPLIT ? 1 : 2); ++w) {
            mx[w] = fmaxf(fmaxf(s[w][0], s[w][1]), fmaxf(s[w][2], s[w][3]));
            raise |= mx[w] > m[w] + kLag;
        }
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
            for (int w = 0; w < (SPLIT ? 1 : 2); ++w) {
                mx[w] = fmaxf(mx[w], __shfl_xor_sync(0xffffffffu, mx[w], 1));
                mx[w] = fmaxf(mx[w], __shfl_xor_sync(0xffffffffu, mx[w], 2));
                const float mn = fmaxf(m[w], mx[w]);
                const float f = m[w] == mn ? 1.f : ex2(m[w] - mn);   // m = -inf: 0
                m[w] = mn;
                l[w] *= f;
#pragma unroll
                for (int j = 0; j < VJ; ++j) {
                    if (SPLIT) {
                        O[j][0] *= f, O[j][1] *= f, O[j][2] *= f, O[j][3] *= f;
                    } else {
                        O[j][2 * w] *= f, O[j][2 * w + 1] *= f;
                    }
                }
            }
        }
        uint32_t a[4];
#pragma unroll
        for (int w = 0; w < (SPLIT ? 1 : 2); ++w) {
            const float base = m[w] == -INFINITY ? 0.f : m[w];
            float p[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                p[i] = ex2(s[w][i] - base);
                if (poison[i] != 0.f && s[w][i] != -INFINITY) p[i] = NAN;
                l[w] = fmaf(p[i], meta.z, l[w]);
            }
            const uint32_t h0 = pack_h2(p[0], p[1]), h1 = pack_h2(p[2], p[3]);
            if (SPLIT) {
                a[0] = h0;
                a[1] = rest_h2(p[0], p[1], h0);
                a[2] = h1;
                a[3] = rest_h2(p[2], p[3], h1);
            } else {
                a[0 + w] = h0;
                a[2 + w] = h1;
            }
        }
#pragma unroll
        for (int x = 0; x < D / 32; ++x) {
            // bytes 4x .. 4x+3 of the four values, paired (key 0, key 1) and (key 2, key 3)
            const uint32_t p0 = __byte_perm(vv[0][x], vv[1][x], 0x5140);
            const uint32_t p1 = __byte_perm(vv[0][x], vv[1][x], 0x7362);
            const uint32_t r0_ = __byte_perm(vv[2][x], vv[3][x], 0x5140);
            const uint32_t r1_ = __byte_perm(vv[2][x], vv[3][x], 0x7362);
            mma_f16(O[4 * x + 0], a, h2_of(p0), h2_of(r0_));
            mma_f16(O[4 * x + 1], a, h2_of(p0 >> 16), h2_of(r0_ >> 16));
            mma_f16(O[4 * x + 2], a, h2_of(p1), h2_of(r1_));
            mma_f16(O[4 * x + 3], a, h2_of(p1 >> 16), h2_of(r1_ >> 16));
        }
    }
    cp_wait<0>();
#pragma unroll
    for (int w = 0; w < (SPLIT ? 1 : 2); ++w) {     // the four lanes of a row hold parts of its sum
        l[w] += __shfl_xor_sync(0xffffffffu, l[w], 1);
        l[w] += __shfl_xor_sync(0xffffffffu, l[w], 2);
    }

    // ---------------------------------------------------------------- join
    // shared memory: warps' O [4][MT][D], m and l [4][MT]; this CTA's O [MT][D], m, l [MT]
    __syncthreads();
    float* wO = reinterpret_cast<float*>(smem);
    float* wM = wO + kWarps * MT * D;
    float* wL = wM + kWarps * MT;
    float* cO = wL + kWarps * MT;
    float* cM = cO + MT * D;
    float* cL = cM + MT;
    static_assert((kWarps + 1) * (MT * D + 2 * MT) * 4 <= ring_bytes<D>(), "join fits the ring");
    {
        float* o = wO + (warp * MT + g) * D;
#pragma unroll
        for (int j = 0; j < VJ; ++j) {
            // columns 2t, 2t+1 of product j: dims (2t) D/8 + j and (2t+1) D/8 + j
            const int d0 = 2 * t * VJ + j, d1 = d0 + VJ;
            if (SPLIT) {
                o[d0] = fmaf(O[j][2], 1.f / 2048.f, O[j][0]);
                o[d1] = fmaf(O[j][3], 1.f / 2048.f, O[j][1]);
            } else {
                o[d0] = O[j][0];
                o[d1] = O[j][1];
                o[8 * D + d0] = O[j][2];
                o[8 * D + d1] = O[j][3];
            }
        }
        if (t == 0) {
#pragma unroll
            for (int w = 0; w < (SPLIT ? 1 : 2); ++w) {
                wM[warp * MT + g + 8 * w] = m[w];
                wL[warp * MT + g + 8 * w] = l[w];
            }
        }
    }
    __syncthreads();
    auto put = [&](int r, int d, float o, float lsum) {
        const int rr = r0 + r;
        if (rr < nq)
            out.p[(int64_t)row * out.row + (int64_t)(rr / share) * out.token +
                  (int64_t)(kvh * share + rr % share) * D + d] =
                from_f<TO>(lsum == 0.f ? 0.f : o / lsum);
    };
    const int live = min(MT, nq - r0);
    for (int x = threadIdx.x; x < live * D; x += kWarps * 32) {
        const int r = x / D, d = x % D;
        float M = wM[r];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) M = fmaxf(M, wM[w * MT + r]);
        float o = 0.f, ls = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float mw = wM[w * MT + r];
            const float f = mw == -INFINITY ? 0.f : ex2(mw - M);
            o = fmaf(f, wO[(w * MT + r) * D + d], o);
            ls = fmaf(f, wL[w * MT + r], ls);
        }
        if (nC == 1) {
            put(r, d, o, ls);
        } else {
            cO[x] = o;
            if (d == 0) cM[r] = M, cL[r] = ls;
        }
    }
    if (nC == 1) return;
    cluster.sync();                         // (CTAs without a run have exited)
    for (int x = rank * kWarps * 32 + (int)threadIdx.x; x < live * D; x += nC * kWarps * 32) {
        const int r = x / D, d = x % D;
        float M = -INFINITY;
        for (int k = 0; k < nC; ++k) M = fmaxf(M, *cluster.map_shared_rank(cM + r, k));
        float o = 0.f, ls = 0.f;
        for (int k = 0; k < nC; ++k) {
            const float mk = *cluster.map_shared_rank(cM + r, k);
            const float f = mk == -INFINITY ? 0.f : ex2(mk - M);
            o = fmaf(f, *cluster.map_shared_rank(cO + x, k), o);
            ls = fmaf(f, *cluster.map_shared_rank(cL + r, k), ls);
        }
        put(r, d, o, ls);
    }
    cluster.sync();                         // no CTA leaves while its memory is read
}

template <int D, bool SPLIT, typename TQ, typename TO>
cudaError_t run(const Cache8& c, const QIn<TQ>& q, const Tok8<TO>& out, int heads, int n,
                const int32_t* lens, int lens_add, float scale, const Rope8& rope,
                cudaStream_t st) {
    constexpr int MT = SPLIT ? 8 : 16;
    auto* kern = k_cache8_attend<D, SPLIT, TQ, TO>;
    const void* kp = reinterpret_cast<const void*>(kern);
    const int share = heads / c.kv_heads, q_tiles = (n * share + MT - 1) / MT;
    int page_log2 = 4;
    while ((1 << page_log2) < c.page) ++page_log2;
    const int64_t cap = (int64_t)c.row_pages * c.page;
    int C = 1;
    while (C < kMaxCtas && (int64_t)C * kKeysPerCta < cap) C *= 2;
    const int64_t ctas = (int64_t)c.rows * c.kv_heads * q_tiles * C;
    if (ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
    if (!set_smem_once(kp, ring_bytes<D>()) || (C > 8 && !set_wide_cluster_once(kp)))
        return cudaErrorInvalidConfiguration;
    set_carveout_once(kp);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.dynamicSmemBytes = ring_bytes<D>();
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)C;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 2 : 1;
    const float scale_log2e = (float)((double)scale * 1.4426950408889634);
    cudaError_t e = cudaLaunchKernelEx(&cfg, kern, c, page_log2, q, out, share, n, q_tiles, lens,
                                       lens_add, scale_log2e, rope);
    if (e == cudaSuccess) rlt_count_launch();
    return e;
}

}  // namespace

template <typename TQ, typename TO>
cudaError_t launch_cache8_attend(const Cache8& c, Tok8<const TQ> q, int slabs, size_t slab,
                                 Tok8<TO> out, int heads, int n, const int32_t* lens,
                                 int lens_add, float scale, const Rope8& rope, cudaStream_t st) {
    if (c.rows <= 0 || n <= 0) return cudaSuccess;
    const QIn<TQ> qi{q.p, q.row, q.token, slabs, slab};
    // 16-row tiles where the bf16 queries of a key head do not fit 8 rows
    constexpr bool both16 = std::is_same<TQ, bf16>::value && std::is_same<TO, bf16>::value;
    if constexpr (both16) {
        if ((int64_t)n * (heads / c.kv_heads) > 8)
            return c.dh == 64 ? run<64, false>(c, qi, out, heads, n, lens, lens_add, scale, rope, st)
                              : run<128, false>(c, qi, out, heads, n, lens, lens_add, scale, rope, st);
    }
    return c.dh == 64 ? run<64, true>(c, qi, out, heads, n, lens, lens_add, scale, rope, st)
                      : run<128, true>(c, qi, out, heads, n, lens, lens_add, scale, rope, st);
}

#define RLT_INST(TQ, TO)                                                                         \
    template cudaError_t launch_cache8_attend<TQ, TO>(const Cache8&, Tok8<const TQ>, int, size_t, \
                                                      Tok8<TO>, int, int, const int32_t*, int,   \
                                                      float, const Rope8&, cudaStream_t);
RLT_INST(float, float)
RLT_INST(bf16, bf16)
RLT_INST(float, bf16)
#undef RLT_INST

}  // namespace rlt
