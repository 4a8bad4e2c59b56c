// Attention over the paged 8-bit cache for up to 4 query vectors per key head:
// generated tokens (include/rlt.h: rlt_cache8_attend).
//
// Mathematics.  With byte values x, key scales ks and value scales vs per
// (page, head), o = sum_j p_j vs_j x^v_j / sum_j p_j, p_j = 2^(s_j),
// s_j = scale log2(e) ks_j q.x^k_j.  Bytes enter the two products as they are
// (e4m3 is exact in fp16).  A tile of 16 keys lies in one page, so its weights
// are brought to its own largest score, p_j = 2^(s_j - t) with t whole and
// s_j <= t (2^15 p_j in fp16), and its product sum_j p_j x^v_j joins the others in
// fp32 by the factor vs 2^(t - e), the sum of the p_j by 2^(t - a): e and a are
// whole numbers that rise with the largest t + log2 vs and the largest t.  Two
// exponents, so that value scales cost the weights nothing, however far apart: a
// page of zeros has the scale 2^-110, one with an infinity 2^120.  A tile is lost
// only where it is 2^-190 of the largest (in o) or 2^-126 (in l).
//
// Matrix form.  One warp takes 16 keys at a time through m16n8k16 fp16
// products with fp32 sums, keys (then value dims) as the 16 rows, queries as
// the 8 columns: converting a byte pair to fp16 is one instruction where
// multiplying it in fp32 on the CUDA cores would take four, so the tensor
// cores carry the per-key work of an HBM stream even for one query.  Columns
// 2i and 2i + 1 hold query i's (then weight i's) leading 11 bits and the next
// 11 bits times 2^11: a lane meets both sums of a score, and adds them in
// fp32.  The weights pass from the score product's layout to the value
// product's operand by an 8x8 transpose of the warp's registers (movmatrix).
//
// Split.  A prefix is cut into a power of two of runs, of 64 to 256 keys up to 65536 keys (256
// runs at most, longer then), and their sums are joined as the leaves of a binary tree:
// pairs, pairs of pairs, ..., whoever works on them.  So the bits of a row do
// not depend on the batch or capacity it sits in, while its runs go to as few
// warps as fill the machine (8 for long prefixes in batches) or as many as there
// are (a cluster of up to 16 CTAs for a single row).  A warp joins its own runs
// as they end, a CTA its warps' results in shared memory, the cluster its CTAs'
// through distributed shared memory: no scratch, no atomics.
//
// Bound by HBM for long batches: 64 rows x 16 heads x 4.3k keys x 128 (1.14 GB) take
// 204-216 us from one B200 to another, 5.3-5.6 TB/s, 0.82-0.87 of the copy rate; 16 warps
// an SM, about 350 instructions a 4 KB tile.  256 rows x 8 heads of at most 256 keys x 64
// take 21 us (floor 5.5): their warps start and end, four dependent loads deep, for a few
// tiles each.  One row of 131072 keys x 8 heads takes 86 us (floor 42): 16 CTAs a head are
// a cluster's limit, and they pack on half of the SMs.  (Products added in pairs by packed
// fp32 instructions: 220 and 91 us.)
#include <cooperative_groups.h>

#include <algorithm>

#include "cache8_tile.cuh"

namespace cg = cooperative_groups;

namespace rlt {
namespace {

constexpr int kQueries = 4;
constexpr int kMaxRuns = 256;
constexpr int kMaxCtas = 16;            // of a cluster
constexpr size_t kMostSmem = 227 * 1024;

template <int D> constexpr int stages() { return D == 64 ? 4 : 3; }
template <int D> constexpr int stage_bytes() { return 2 * kTile * D + 16; }
template <int D, int NW> constexpr int ring_bytes() { return NW * stages<D>() * stage_bytes<D>(); }

// runs of a prefix: a power of two, of 4 tiles at least, 8 from 64 tiles on, 16 from 512 on (a run's
// end costs about half a tile)
__host__ __device__ __forceinline__ int runs_of(int tiles) {
    const int most = tiles < 64 ? tiles / 4 : tiles < 512 ? tiles / 8 : tiles / 16;
    int r = 1;
    while (r < kMaxRuns && 2 * r <= most) r *= 2;
    return r;
}
constexpr float kNone = -3e38f;         // exponent of an empty sum
constexpr float kAhead = 64.f;          // a new largest tile's factor, log2,
constexpr float kMost = 72.f;           // and the factor from which on the exponent rises
// A tile's product is at most 2^28 (16 keys, weights of 2^15, bytes of 448), with its factor 2^101;
// 2^30 keys are 2^26 tiles: below fp32's 2^128.

constexpr float kWeight = 15.f;         // log2 of the weights' factor in fp16

// 2^x, subnormal results included
__device__ __forceinline__ float pow2(float x) {
    float y;
    asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// the largest of a warp's values (one instruction; three shuffles for 8 lanes each take longer: 256
// rows x 8 heads of 256 keys 21.2 us, 20.8 with this)
__device__ __forceinline__ float warp_max(float x) {
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(x) : "f"(x));
    return x;
}
// Sums over some keys: l of weights, in units of 2^a; o of weighted values (one a dim), in units of 2^e
struct Sum {
    float a, e, l;
};
// The sums of two neighbours in the tree, the left one's in x, its factor and the right one's
// out: o = fa * o_left + fb * o_right, everywhere rounded alike
__device__ __forceinline__ void join2(Sum& x, const Sum& y, float& fa, float& fb) {
    const float A = fmaxf(x.a, y.a), E = fmaxf(x.e, y.e);
    x.l = fmaf(ex2(x.a - A), x.l, ex2(y.a - A) * y.l);
    fa = pow2(x.e - E);
    fb = pow2(y.e - E);
    x.a = A;
    x.e = E;
}
// The tree over N values, the first `there` of them (a power of two): the root's in x[0], o[0]
template <int N>
__device__ __forceinline__ void join_tree(Sum (&x)[N], float (&o)[N], int there) {
#pragma unroll
    for (int s = 1; s < N; s *= 2)
#pragma unroll
        for (int k = 0; k < N; k += 2 * s) {
            if (k + s >= there) break;
            float fa, fb;
            join2(x[k], x[k + s], fa, fb);
            o[k] = fmaf(fa, o[k], fb * o[k + s]);
        }
}

// 8 warps: two CTAs an SM; 16: one
template <int D, int NW, typename TQ, typename TO>
__global__ void __launch_bounds__(NW * 32, NW == 16 ? 1 : 2)
k_cache8_decode(Cache8 c, int page_log2, QIn<TQ> q, Tok8<TO> out, int share, int n, int units,
                int unit_warps, int levels, const int32_t* __restrict__ lens, int lens_add,
                float scale_log2e, Rope8 rope) {
    constexpr int NST = stages<D>(), SB = stage_bytes<D>(), KI = D / 16, VJ = D / 16;
    extern __shared__ __align__(128) uint8_t smem[];
    pdl_enter();
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int nq = n * share;
    // unit (row, key head) of this warp, and the warp's place among the unit's
    const int here = warp / unit_warps, wi = warp - here * unit_warps;
    const int64_t unit = (int64_t)(blockIdx.x / (unsigned)C) * (NW / unit_warps) + here;
    const bool alive = unit < units;
    const int row = alive ? (int)unit / c.kv_heads : 0, kvh = alive ? (int)unit % c.kv_heads : 0;

    const int cap = c.row_pages << page_log2;
    const int L0 = __ldg(lens + row) + lens_add;
    const int L = max(0, min(cap, L0));
    if ((L0 < 0 || L0 > cap) && alive && lane == 0 && wi == 0 && kvh == 0 && rank == 0 && c.status)
        atomicCAS(c.status, 0, c.cap_code);
    const int keys = alive ? L : 0;                 // the last query sees all, the first:
    const int vis_min = L - n + 1;
    const int tiles = (keys + kTile - 1) / kTile, runs = runs_of(tiles);
    // `per` runs a warp, warps 0 .. busy - 1 of CTAs 0 .. ctas - 1: all powers of two
    const int per = max(1, runs / (C * unit_warps)), busy = min(unit_warps, runs / per);
    const int ctas = max(1, runs / (per * unit_warps));
    if (rank >= ctas) return;                       // (one unit per CTA then)
    auto start_of = [&](int r) { return (int)((int64_t)r * tiles / runs); };
    const int r_begin = (rank * unit_warps + wi) * per, r_end = wi < busy ? r_begin + per : r_begin;
    const int s_begin = wi < busy ? start_of(r_begin) : 0, s_end = wi < busy ? start_of(r_end) : 0;
    // Shared memory: the warps' tiles, then what a warp keeps of its unfinished subtrees, one level
    // each: O [query][D], then the queries' a, e and l (a multiple of 4 floats in all).  A warp's
    // result goes to its own tiles, when they are done with; in the unit's first warp's tiles also
    // the queries (a stage that is filled last) and the CTA's result.
    const int run_floats = nq * (D + 4);
    uint8_t* const ring = smem + warp * (NST * SB);
    uint8_t* const first = smem + here * unit_warps * (NST * SB);
    float* const stack = reinterpret_cast<float*>(smem + ring_bytes<D, NW>()) +
                         warp * levels * run_floats;
    float* const s_q = reinterpret_cast<float*>(first + (NST - 1) * SB);    // [query][D + 4]
    float* const g_o = reinterpret_cast<float*>(first + 4096);
    float* const scratch = reinterpret_cast<float*>(first + 4096 + 2560);
    static_assert(kQueries * (D + 4) * 4 <= SB && kQueries * (D + 4) * 4 <= 2560 &&
                  4096 + 2560 + 3 * 16 * kQueries * 4 <= NST * SB, "they fit");

    // ---------------------------------------------------------------- queries: on their way
    const int qx = wi * 32 + lane;          // dims 4 qx .. of the unit's queries; the rest below
    auto fetch_q = [&](int x, Q4<TQ>& v) {  // false: nothing to see
        const int r = x / (D / 4), d = (x % (D / 4)) * 4;
        const int i = r / share, pos = L - n + i + rope.origin;
        const bool seen = alive && L - n + i >= 0;
        const bool lost = seen && rope.rot && (pos < 0 || pos >= rope.positions);
        if (lost && d == 0 && c.status) atomicCAS(c.status, 0, c.cap_code);
        if (!seen || lost) return false;
        v.load(q, (size_t)((int64_t)row * q.row + (int64_t)i * q.token) +
                      (size_t)(kvh * share + r % share) * D, d, rope, pos);
        return true;
    };
    Q4<TQ> q4;
    const bool q4_in = qx < nq * (D / 4) && fetch_q(qx, q4);

    // ---------------------------------------------------------------- tiles
    const uint32_t ring_u = tc::smem_u32(ring);
    const size_t head_bytes = (size_t)D << page_log2;
    const size_t v_bytes = (size_t)c.kv_heads * head_bytes;
    const uint8_t* const pages = c.pages + (size_t)kvh * head_bytes + lane * 16;
    int b_base = s_begin;                   // first tile of the batch below
    int b_page = -1;                        // lane l: the page of tile b_base + l, and its scalars,
    float b_ks = 0.f, b_vm = 0.f, b_ve = -INFINITY;     // the value scale as b_vm * 2^b_ve
    auto load_batch = [&]() {
        b_page = -1;
        b_ks = 0.f, b_vm = 0.f, b_ve = -INFINITY;
        const int s = b_base + lane;
        if (s < s_end) {
            const int p = __ldg(c.table + (size_t)row * c.row_pages + ((s * kTile) >> page_log2));
            if (p >= 0 && p < c.n_pages) {
                const float* sc = c.scales + (size_t)p * 2 * c.kv_heads + kvh;
                b_page = p;
                b_ks = __ldg(sc);
                split_scale(__ldg(sc + c.kv_heads), b_vm, b_ve);
            } else if (c.status) {
                atomicCAS(c.status, 0, c.arg_code);
            }
        }
    };
    const TileCopy<D> copy(lane);
    int fs = s_begin, fslot = 0;            // the tile fetched next, and its stage
    auto fetch = [&]() {
        if (fs < s_end) {
            if (fs - b_base == 32) {
                b_base += 32;
                load_batch();
            }
            const int src = fs - b_base;
            const int p = __shfl_sync(0xffffffffu, b_page, src);
            const float ks = __shfl_sync(0xffffffffu, b_ks, src);
            const float vm = __shfl_sync(0xffffffffu, b_vm, src);
            const float ve = __shfl_sync(0xffffffffu, b_ve, src);
            if (lane == 0)
                *reinterpret_cast<float4*>(ring + fslot * SB + 2 * kTile * D) =
                    make_float4(ks, vm, ve, 0.f);
            const int k0 = fs * kTile;
            const uint8_t* kg = pages + (size_t)max(p, 0) * 2 * v_bytes +
                                (size_t)((k0 & ((1 << page_log2) - 1)) * D);
            copy(ring_u + fslot * SB, kg, kg + v_bytes, p >= 0 ? keys - k0 : 0, c.pages);
        }
        cp_commit();
        ++fs;
        fslot = fslot + 1 == NST ? 0 : fslot + 1;
    };
    load_batch();
#pragma unroll
    for (int i = 0; i < NST - 1; ++i) fetch();

    // ---------------------------------------------------------------- queries
    // rotated once per unit, then split into operands by every warp
    auto put_q = [&](int x, bool in, Q4<TQ>& v) {
        const int r = x / (D / 4), d = (x % (D / 4)) * 4;
        *reinterpret_cast<float4*>(s_q + r * (D + 4) + d) =
            in ? v.turned(d, rope) : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    if (qx < nq * (D / 4)) put_q(qx, q4_in, q4);
    for (int x = qx + unit_warps * 32; x < nq * (D / 4); x += unit_warps * 32) {
        const bool in = fetch_q(x, q4);
        put_q(x, in, q4);
    }
    __syncthreads();
    // column g: query g/2, this lane's dims [t D/4, (t+1) D/4) of it, leading or trailing bits
    uint32_t qf[KI][2];
    float rf = 0.f;                         // score factor of query t: 2^e scale log2(e)
    int vis = 0;                            // keys it sees
    {
        const int r = g >> 1;
        const float* sq = s_q + r * (D + 4) + t * (D / 4);
        float amax = 0.f;
        if (r < nq)
#pragma unroll
            for (int k = 0; k < KI; ++k) {
                const float4 x = *reinterpret_cast<const float4*>(sq + 4 * k);
                amax = fmaxf(fmaxf(amax, fmaxf(fabsf(x.x), fabsf(x.y))), fmaxf(fabsf(x.z), fabsf(x.w)));
            }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        // bring the query near 1 by a power of two (exact); 2^+-100 keeps both factors finite
        int e2 = (int)(__float_as_uint(amax) >> 23) - 127;
        e2 = max(-100, min(100, e2));
        const float down = __uint_as_float((uint32_t)(127 - e2) << 23);
        const float up = __uint_as_float((uint32_t)(127 + e2) << 23) * scale_log2e;
#pragma unroll
        for (int k = 0; k < KI; ++k) {
            qf[k][0] = qf[k][1] = 0u;
            if (r < nq) {
                const float4 x = *reinterpret_cast<const float4*>(sq + 4 * k);
                const float x0 = x.x * down, x1 = x.y * down, x2 = x.z * down, x3 = x.w * down;
                const uint32_t h0 = pack_h2(x0, x1), h1 = pack_h2(x2, x3);
                qf[k][0] = g & 1 ? rest_h2(x0, x1, h0) : h0;
                qf[k][1] = g & 1 ? rest_h2(x2, x3, h1) : h1;
            }
        }
        rf = __shfl_sync(0xffffffffu, up, 8 * t);
        const int i = t / share, pos = L - n + i + rope.origin;
        vis = t < nq ? max(0, L - n + i + 1) : 0;
        if (rope.rot && (pos < 0 || pos >= rope.positions)) vis = 0;
    }
    __syncthreads();                        // the stage that held the queries is filled from here on
    // a query without a rotation sees nothing: its column has to be masked from the first key on
    const int mask_from = __any_sync(0xffffffffu, t < nq && vis < vis_min) ? 0 : vis_min;

    // ---------------------------------------------------------------- the runs
    // of query t: this lane's part of the weights' sum, and dims 2j, 2j + 1 of its D/8
    Sum sum = {kNone, kNone, 0.f};
    float O[VJ][2];
#pragma unroll
    for (int j = 0; j < VJ; ++j) O[j][0] = O[j][1] = 0.f;
    const int key_lo = 4 * (g & 1) + (g >> 1);      // sigma(g): the key of row g; row g + 8: + 8
    int slot = 0, run = 0, run_end = start_of(r_begin + 1);     // (run: of this warp's)

    for (int s = s_begin; s < s_end; ++s) {
        cp_wait<NST - 2>();
        __syncwarp();                       // the tile is here; every lane has left the last one
        fetch();
        const uint8_t* st = ring + slot * SB;
        slot = slot + 1 == NST ? 0 : slot + 1;
        const float4 meta = *reinterpret_cast<const float4*>(st + 2 * kTile * D);
        const int k0 = s * kTile;

        float cf[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
            uint4 x, y;
            load_keys<D>(st, g, t, h, x, y);
            const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t a[4];
                h2x2_of(xs[k], a[0], a[2]);
                h2x2_of(ys[k], a[1], a[3]);
                mma_f16(cf, a, qf[4 * h + k][0], qf[4 * h + k][1]);
            }
        }
        uint32_t vv[4][D / 32];
        load_values<D>(st, g, t, vv);
        // scores of key rows g, g + 8 and query t
        const float f = rf * meta.x;
        float s0 = fmaf(cf[1], 1.f / 2048.f, cf[0]) * f;
        float s1 = fmaf(cf[3], 1.f / 2048.f, cf[2]) * f;
        const bool bad = !(meta.z > -INFINITY);
        uint32_t poison = 0;                // keys of the tile with a NaN among their values
        if (bad || k0 + kTile > mask_from) {    // the prefix ends in this tile for some query
            if (bad || k0 + key_lo >= vis) s0 = -INFINITY;
            if (bad || k0 + key_lo + 8 >= vis) s1 = -INFINITY;
            if (mask_from < keys) poison = clear_nan<D>(vv, t);
        }
        float top = fmaxf(s0, s1);          // of query t's 8 lanes
        if (nq == 1) {
            top = warp_max(t ? -INFINITY : top);
        } else if (nq == 2) {
            const float of0 = warp_max(t == 0 ? top : -INFINITY);
            const float of1 = warp_max(t == 1 ? top : -INFINITY);
            top = t ? of1 : of0;
        } else {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        }
        top = ceilf(top);                   // -inf: the query sees none of the tile
        const float tv = top + meta.z;
        const bool up_a = top > sum.a + kMost, up_e = tv > sum.e + kMost;
        if (__any_sync(0xffffffffu, up_a || up_e)) {
            const float an = up_a ? top : sum.a, en = up_e ? tv - kAhead : sum.e;
            sum.l *= ex2(sum.a - an);
            const float r = pow2(sum.e - en);
            sum.a = an, sum.e = en;
#pragma unroll
            for (int j = 0; j < VJ; ++j) O[j][0] *= r, O[j][1] *= r;
        }
        const float to_l = ex2(top - sum.a), to_o = meta.y * ex2(tv - sum.e);
        const float zero = top == -INFINITY ? 0.f : top;
        float p0 = ex2(s0 - zero), p1 = ex2(s1 - zero);
        if (poison) {
            if (s0 != -INFINITY && ((poison >> key_lo) & 1u)) p0 = NAN;
            if (s1 != -INFINITY && ((poison >> (key_lo + 8)) & 1u)) p1 = NAN;
        }
        sum.l = fmaf(p0 + p1, to_l, sum.l);
        p0 *= 32768.f, p1 *= 32768.f;       // (kWeight: most of fp16's range lies below 1)
        // the value product's operand: column 2t the leading bits, 2t + 1 the rest
        const float h0 = __half2float(__float2half_rn(p0)), h1 = __half2float(__float2half_rn(p1));
        const uint32_t b0 = transpose8(pack_h2(h0, (p0 - h0) * 2048.f));
        const uint32_t b1 = transpose8(pack_h2(h1, (p1 - h1) * 2048.f));
#pragma unroll
        for (int x = 0; x < D / 32; ++x) {
            // bytes of the four values paired (key 0, key 1) and (key 2, key 3): bytes 0, 1 and
            // 2, 3 of word x are dims 4x .. 4x+3 of this lane
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                uint32_t a[4];
                float of[4] = {0.f, 0.f, 0.f, 0.f};
                h2x2_of(__byte_perm(vv[0][x], vv[1][x], y ? 0x7362 : 0x5140), a[0], a[1]);
                h2x2_of(__byte_perm(vv[2][x], vv[3][x], y ? 0x7362 : 0x5140), a[2], a[3]);
                mma_f16(of, a, b0, b1);
                float(&to)[2] = O[2 * x + y];
                to[0] = fmaf(fmaf(of[1], 1.f / 2048.f, of[0]), to_o, to[0]);
                to[1] = fmaf(fmaf(of[3], 1.f / 2048.f, of[2]), to_o, to[1]);
            }
        }
        if (s + 1 == run_end) {             // the run's sums, and those of the subtrees it completes
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) sum.l += __shfl_xor_sync(0xffffffffu, sum.l, o);
            const int at = t * D + g * (D / 8);
            int level = 0;
            for (; (run >> level) & 1; ++level) {
                const float* const z = stack + level * run_floats;
                if (t < nq) {
                    Sum left = {z[nq * D + t], z[nq * (D + 1) + t], z[nq * (D + 2) + t]};
                    float fa, fb;
                    join2(left, sum, fa, fb);
                    sum = left;
#pragma unroll
                    for (int j = 0; j < VJ; ++j) {
                        const float2 o = *reinterpret_cast<const float2*>(z + at + 2 * j);
                        O[j][0] = fmaf(fa, o.x, fb * O[j][0]);
                        O[j][1] = fmaf(fa, o.y, fb * O[j][1]);
                    }
                }
            }
            const bool last = s + 1 == s_end;
            if (last) cp_wait<0>();         // (the ring: no copy is on its way,
            __syncwarp();                   //  none is read; and the stack has been read)
            float* const to = last ? reinterpret_cast<float*>(ring) : stack + level * run_floats;
            if (t < nq) {
#pragma unroll
                for (int j = 0; j < VJ; ++j)
                    *reinterpret_cast<float2*>(to + at + 2 * j) = make_float2(O[j][0], O[j][1]);
                if (g == 0)
                    to[nq * D + t] = sum.a, to[nq * (D + 1) + t] = sum.e, to[nq * (D + 2) + t] = sum.l;
            }
#pragma unroll
            for (int j = 0; j < VJ; ++j) O[j][0] = O[j][1] = 0.f;
            sum = {kNone, kNone, 0.f};
            ++run;
            run_end = start_of(r_begin + run + 1);
        }
    }
    if (tiles == 0 && wi == 0)              // no key: an empty sum
        for (int x = lane; x < run_floats; x += 32)
            reinterpret_cast<float*>(ring)[x] = x >= nq * D && x < nq * (D + 2) ? kNone : 0.f;
    cp_wait<0>();
    __syncthreads();

    // ---------------------------------------------------------------- join
    auto put = [&](int r, int d, float o, const Sum& x) {   // o / l * 2^(e - a - kWeight)
        const float by = x.e - x.a - kWeight, half = floorf(0.5f * by);
        out.p[(int64_t)row * out.row + (int64_t)(r / share) * out.token +
              (int64_t)(kvh * share + r % share) * D + d] =
            from_f<TO>(x.l == 0.f ? 0.f : o / x.l * pow2(half) * pow2(by - half));
    };
    auto sum_at = [&](const float* z, int r) {
        return Sum{z[nq * D + r], z[nq * (D + 1) + r], z[nq * (D + 2) + r]};
    };
    if (alive)
        for (int x = wi * 32 + lane; x < nq * D; x += unit_warps * 32) {
            const int r = x / D;
            Sum sm[NW];
            float o[NW];
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const float* const z = reinterpret_cast<const float*>(first + w * (NST * SB));
                sm[w] = {kNone, kNone, 0.f}, o[w] = 0.f;
                if (w < busy) sm[w] = sum_at(z, r), o[w] = z[x];
            }
            join_tree<NW>(sm, o, busy);
            if (ctas == 1) {
                put(r, x - r * D, o[0], sm[0]);
            } else {
                g_o[x] = o[0];
                if (x == r * D)
                    g_o[nq * D + r] = sm[0].a, g_o[nq * (D + 1) + r] = sm[0].e,
                    g_o[nq * (D + 2) + r] = sm[0].l;
            }
        }
    if (ctas == 1) return;
    cluster.sync();                                 // (CTAs without a run have exited)
    for (int x = threadIdx.x; x < ctas * 3 * nq; x += NW * 32) {
        const int k = x / (3 * nq), r = x - k * 3 * nq;
        scratch[x] = *cluster.map_shared_rank(g_o + nq * D + r, k);
    }
    __syncthreads();
    for (int x = rank * NW * 32 + (int)threadIdx.x; x < nq * D; x += ctas * NW * 32) {
        const int r = x / D;
        Sum sm[kMaxCtas];
        float o[kMaxCtas];
#pragma unroll
        for (int k = 0; k < kMaxCtas; ++k) {        // (the remote loads are all in flight at once)
            sm[k] = {kNone, kNone, 0.f}, o[k] = 0.f;
            if (k < ctas) {
                o[k] = *cluster.map_shared_rank(g_o + x, k);
                const float* const z = scratch + k * 3 * nq + r;
                sm[k] = {z[0], z[nq], z[2 * nq]};
            }
        }
        join_tree<kMaxCtas>(sm, o, ctas);
        put(r, x - r * D, o[0], sm[0]);
    }
    cluster.sync();                                 // no CTA leaves while its memory is read
}

template <int D, int NW, typename TQ, typename TO>
cudaError_t run(const Cache8& c, const QIn<TQ>& q, const Tok8<TO>& out, int share, int n,
                const int32_t* lens, int lens_add, float scale, const Rope8& rope, int64_t units,
                int C, int unit_warps, int levels, size_t smem, cudaStream_t st) {
    auto* kern = k_cache8_decode<D, NW, TQ, TO>;
    const void* kp = reinterpret_cast<const void*>(kern);
    int page_log2 = 4;
    while ((1 << page_log2) < c.page) ++page_log2;
    const int per_cta = NW / unit_warps;
    const int64_t ctas = (units + per_cta - 1) / per_cta * C;
    if (ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
    if (smem > kMostSmem || !set_smem_once(kp, kMostSmem) || (C > 8 && !set_wide_cluster_once(kp)))
        return cudaErrorInvalidConfiguration;
    set_carveout_once(kp);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(NW * 32);
    cfg.dynamicSmemBytes = smem;
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
    cudaError_t e = cudaLaunchKernelEx(&cfg, kern, c, page_log2, q, out, share, n, (int)units,
                                       unit_warps, levels, lens, lens_add, scale_log2e, rope);
    if (e == cudaSuccess) rlt_count_launch();
    return e;
}

template <int D, typename TQ, typename TO>
cudaError_t plan(const Cache8& c, const QIn<TQ>& q, const Tok8<TO>& out, int share, int n,
                 const int32_t* lens, int lens_add, float scale, const Rope8& rope,
                 cudaStream_t st) {
    const int64_t cap = (int64_t)c.row_pages * c.page, units = (int64_t)c.rows * c.kv_heads;
    if (units > 0x7fffffff) return cudaErrorInvalidConfiguration;
    const int nq = n * share, runs = runs_of((int)((cap + kTile - 1) / kTile));
    auto levels = [&](int w) {                      // of the tree in one of w warps
        int v = 0;
        while ((w << v) < runs) ++v;
        return v;
    };
    auto smem = [&](int w) {
        return (size_t)ring_bytes<D, 8>() + (size_t)8 * levels(w) * nq * (D + 4) * 4;
    };
    // Warps of a unit, by the capacity (lengths are on the device).  Short prefixes: as few as come near filling the machine, 12 an SM up to 512
    // keys, then 16 (a warp starts and ends in about four tiles' time: 256 rows x 8 heads x 64 of
    // 256 keys take 21 us with one warp, 25 with two; 128 rows x 16 heads x 128 of 1024 keys 100
    // and 96: two measurements, nothing between them).  Longer ones: 8 (48 rows x 16 heads of 2k to 8k keys: 234 us with four, 202
    // with 8), and more as long as all run at once (9 rows x 16 heads of 4.3k keys: 50 us with 32,
    // in two turns, 37 with 16).  More also where the subtrees leave no room for two CTAs an SM.
    int w = std::min(cap <= 1024 ? 1 : 8, runs);
    while (w < runs && w < 8 * kMaxCtas &&
           ((cap <= 1024 ? units * w < 148 * (cap <= 512 ? 12 : 16) : units * w * 2 <= 148 * 16) ||
            smem(w) > 113 * 1024))
        w *= 2;
    // CTAs of 16 warps, one an SM, for the few longest rows: of clusters of 16 such CTAs 7 run at
    // a time, of 8-warp ones, two an SM, 14 (131072 keys: 4 key heads take 53 us with 16 warps a
    // CTA, 8 take 103, and 98 with 8 warps)
    if (runs == 16 * kMaxCtas && units <= 7)
        return run<D, 16>(c, q, out, share, n, lens, lens_add, scale, rope, units, kMaxCtas, 16, 0,
                          ring_bytes<D, 16>(), st);
    return run<D, 8>(c, q, out, share, n, lens, lens_add, scale, rope, units, std::max(1, w / 8),
                     std::min(w, 8), levels(w), smem(w), st);
}

}  // namespace

template <typename TQ, typename TO>
cudaError_t launch_cache8_decode(const Cache8& c, Tok8<const TQ> q, int slabs, size_t slab,
                                 Tok8<TO> out, int heads, int n, const int32_t* lens,
                                 int lens_add, float scale, const Rope8& rope, cudaStream_t st) {
    const QIn<TQ> qi{q.p, q.row, q.token, slabs, slab};
    const int share = heads / c.kv_heads;
    return c.dh == 64 ? plan<64>(c, qi, out, share, n, lens, lens_add, scale, rope, st)
                      : plan<128>(c, qi, out, share, n, lens, lens_add, scale, rope, st);
}

#define RLT_INST(TQ, TO)                                                                         \
    template cudaError_t launch_cache8_decode<TQ, TO>(const Cache8&, Tok8<const TQ>, int, size_t, \
                                                      Tok8<TO>, int, int, const int32_t*, int,   \
                                                      float, const Rope8&, cudaStream_t);
RLT_INST(float, float)
RLT_INST(bf16, bf16)
RLT_INST(float, bf16)
#undef RLT_INST

}  // namespace rlt
