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
// products with fp32 sums, keys (then value dims) as the 16 rows, queries as
// the 8 columns: converting a byte pair to fp16 is one instruction where
// multiplying it in fp32 on the CUDA cores would take four, so the tensor
// cores carry the per-key work of an HBM stream even for one query.  (Queries
// as rows, tried first, need twice the products and twice the registers of
// the output: 618 instructions per 4 KB tile and 12 warps an SM, 2.5 TB/s on 64
// rows x 16 heads x 4.3k keys.)  Columns left over buy precision:
//   FOLD   up to 4 query vectors per key head: columns 0-3 hold the leading 11
//          bits of q (of w), columns 4-7 the next 11 bits times 2^11, and the two
//          sums are added in fp32;
//   SPLIT  up to 8, fp32 types: the same in two products;
//   PLAIN  8 or 16 bf16 queries, leading bits alone: a bf16 q is exact there
//          (each query is brought near 1 by a power of two first), w is rounded
//          to fp16 (2^-11 relative at most, below the bf16 output's 2^-9 step).
// The weights pass from the score product's layout to the value product's
// operand by an 8x8 transpose of the warp's registers (movmatrix).
//
// The maximum is raised only when a score passes it by 2^8 (one warp vote per
// tile instead of a reduction); fp16 holds weights up to 2^16.
//
// Data path.  Tiles reach a per-warp ring in shared memory by 16-byte
// cp.async copies; keys past the prefix and keys in bad pages are zero-filled
// rather than read, so whatever bytes sit there never enter a product.  Key
// rows and 16-byte chunks are permuted on the way in so that every fragment
// load is one conflict-free wide load: lane (g, t) = (lane/4, lane%4) reads
// dims [t D/4, (t+1) D/4) of key rows g and g + 8 and of query g, and dims
// [g D/8, (g+1) D/8) of values 4i + t; key row r holds key
// sigma(r) = (r & 8) + 4 (r & 1) + (r & 7) / 2, the order the transpose wants.
//
// Split.  The prefix of a (row, key head) is cut into runs for 4 warps of
// 2^j <= keys / 1024 CTAs (1 to 16), a function of that prefix alone.  The
// warps' partial results meet in shared memory, the CTAs' through the
// cluster's distributed shared memory, always in run order: no scratch, no
// atomics, and the same bits for a row whatever batch or capacity it sits in.
#include <cooperative_groups.h>

#include <algorithm>
#include "cache8_tile.cuh"

namespace cg = cooperative_groups;

namespace rlt {
namespace {

constexpr int kWarps = 4;
constexpr int kKeysPerCta = 1024;
constexpr int kMaxCtas = 16;            // CTAs per (row, key head, query tile): one cluster

template <int D> constexpr int stages() { return D == 64 ? 4 : 3; }
template <int D> constexpr int stage_bytes() { return 2 * kTile * D + 16; }
template <int D> constexpr int ring_bytes() { return kWarps * stages<D>() * stage_bytes<D>(); }

enum Mode { SPLIT, PLAIN };
constexpr int queries_of(int mode, int nb) { return mode == SPLIT ? 8 : 8 * nb; }

// CTAs that share a prefix of `keys` keys: a power of two, kKeysPerCta keys each at least
__host__ __device__ __forceinline__ int ctas_of(int64_t keys) {
    int c = 1;
    while (c < kMaxCtas && (int64_t)c * 2 * kKeysPerCta <= keys) c *= 2;
    return c;
}

// MODE and NB (products of 8 columns): SPLIT 2, PLAIN 1 or 2
template <int D, int MODE, int NB, typename TQ, typename TO>
__global__ void __launch_bounds__(kWarps * 32)
k_cache8_attend(Cache8 c, int page_log2, QIn<TQ> q, Tok8<TO> out, int share, int n, int q_tiles,
                const int32_t* __restrict__ lens, int lens_add, float scale_log2e, Rope8 rope) {
    constexpr int QT = queries_of(MODE, NB);    // query vectors per tile
    constexpr int NS = MODE == PLAIN ? NB : 1;  // column tiles of scores: queries 8 b + 2t + e
    constexpr int NST = stages<D>(), SB = stage_bytes<D>(), KI = D / 16, VJ = D / 16;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(16) float s_q[QT][D + 4];
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
    const int r0 = mt * QT, live = min(QT, nq - r0);
    const int vis_max = max(0, L - n + (r0 + live - 1) / share + 1);  // keys any query of the tile sees
    const int vis_min = L - n + r0 / share + 1;                      // keys all of them see
    const int nC = min(C, ctas_of(vis_max));
    if (rank >= nC) return;
    const int subs = (vis_max + kTile - 1) / kTile, runs = nC * kWarps;
    const int per = (subs + runs - 1) / runs;
    const int s_begin = min(subs, (rank * kWarps + warp) * per), s_end = min(subs, s_begin + per);

    // ---------------------------------------------------------------- tiles
    uint8_t* ring = smem + warp * (NST * SB);
    const uint32_t ring_u = tc::smem_u32(ring);
    const size_t head_bytes = (size_t)D << page_log2;
    const size_t v_bytes = (size_t)c.kv_heads * head_bytes;
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
    const TileCopy<D> copy(lane);
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
                                (size_t)(k0 & ((1 << page_log2) - 1)) * D + lane * 16;
            copy(ring_u + slot * SB, kg, kg + v_bytes, p >= 0 ? vis_max - k0 : 0, c.pages);
        }
        cp_commit();
    };
    load_batch();
#pragma unroll
    for (int i = 0; i < NST - 1; ++i) issue(i);

    // ---------------------------------------------------------------- queries
    // rotated once per CTA, then split into operands by every warp
    for (int x = threadIdx.x; x < QT * (D / 4); x += kWarps * 32) {
        const int r = x / (D / 4), d = (x % (D / 4)) * 4;
        float y[4] = {0.f, 0.f, 0.f, 0.f};
        if (r < live) {
            const int rr = r0 + r, i = rr / share, pos = L - n + i + rope.origin;
            const bool seen = L - n + i >= 0;
            const bool lost = seen && rope.rot && (pos < 0 || pos >= rope.positions);
            if (lost && d == 0 && c.status) atomicCAS(c.status, 0, c.cap_code);
            if (seen && !lost) {
                const size_t at = (size_t)((int64_t)row * q.row + (int64_t)i * q.token) +
                                  (size_t)(kvh * share + rr % share) * D;
                load_q4(q, at, d, rope, pos, y);
            }
        }
        *reinterpret_cast<float4*>(&s_q[r][d]) = make_float4(y[0], y[1], y[2], y[3]);
    }
    __syncthreads();
    // column g of product b: this lane's dims [t D/4, (t+1) D/4) of its query
    uint32_t qf[KI][NB][2];
    float rf[NS][2];                        // score factor of queries 2t, 2t+1: 2^e scale log2(e)
    int vis[NS][2];                         // keys they see
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        if (MODE == SPLIT && b == 1) break;
        const int r = 8 * b + g;
        const float* sq = &s_q[r][t * (D / 4)];
        float amax = 0.f;
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
            const float4 x = *reinterpret_cast<const float4*>(sq + 4 * k);
            const float x0 = x.x * down, x1 = x.y * down, x2 = x.z * down, x3 = x.w * down;
            const uint32_t h0 = pack_h2(x0, x1), h1 = pack_h2(x2, x3);
            qf[k][b][0] = h0;
            qf[k][b][1] = h1;
            if (MODE == SPLIT) {
                qf[k][NB - 1][0] = rest_h2(x0, x1, h0);
                qf[k][NB - 1][1] = rest_h2(x2, x3, h1);
            }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int col = 2 * t + e;
            rf[b][e] = __shfl_sync(0xffffffffu, up, 4 * col);
            const int rr = r0 + 8 * b + col, i = rr / share, pos = L - n + i + rope.origin;
            vis[b][e] = rr < nq ? max(0, L - n + i + 1) : 0;
            if (rope.rot && (pos < 0 || pos >= rope.positions)) vis[b][e] = 0;
        }
    }
    // a query without a rotation sees nothing: its column has to be masked from the first key on
    bool lost = false;
#pragma unroll
    for (int b = 0; b < NS; ++b)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int col = 2 * t + e;
            lost |= 8 * b + col < live && vis[b][e] < vis_min;
        }
    const int mask_from = __any_sync(0xffffffffu, lost) ? 0 : vis_min;

    // ---------------------------------------------------------------- the run
    float m[NS][2], l[NS][2], O[VJ][NB][4];
#pragma unroll
    for (int b = 0; b < NS; ++b) m[b][0] = m[b][1] = -INFINITY, l[b][0] = l[b][1] = 0.f;
#pragma unroll
    for (int j = 0; j < VJ; ++j)
#pragma unroll
        for (int b = 0; b < NB; ++b) O[j][b][0] = O[j][b][1] = O[j][b][2] = O[j][b][3] = 0.f;
    const int key_lo = 4 * (g & 1) + (g >> 1);      // sigma(g): the key of row g; row g + 8: + 8

    for (int it = 0; s_begin + it < s_end; ++it) {
        cp_wait<NST - 2>();
        __syncwarp();                       // the tile is here; every lane has left the last one
        issue(it + NST - 1);
        const uint8_t* st = ring + (it % NST) * SB;
        const float4 meta = *reinterpret_cast<const float4*>(st + 2 * kTile * D);
        const int k0 = (s_begin + it) * kTile;

        float cf[NB][4];
#pragma unroll
        for (int b = 0; b < NB; ++b) cf[b][0] = cf[b][1] = cf[b][2] = cf[b][3] = 0.f;
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
#pragma unroll
                for (int b = 0; b < NB; ++b)
                    mma_f16(cf[b], a, qf[4 * h + k][b][0], qf[4 * h + k][b][1]);
            }
        }
        uint32_t vv[4][D / 32];
        load_values<D>(st, g, t, vv);
        // scores [key rows g, g + 8][queries 2t, 2t + 1], the value scale folded in
        float s[NS][4];
        if (MODE == SPLIT) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                s[0][i] = fmaf(fmaf(cf[NB - 1][i], 1.f / 2048.f, cf[0][i]), rf[0][i & 1] * meta.x,
                               meta.y);
        } else {
#pragma unroll
            for (int b = 0; b < NS; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    s[b][i] = fmaf(cf[b][i], rf[b][i & 1] * meta.x, meta.y);
        }
        const bool bad = !(meta.y > -INFINITY);
        uint32_t poison = 0;                // keys of the tile with a NaN among their values
        if (bad || k0 + kTile > mask_from) {    // the prefix ends in this tile for some query
#pragma unroll
            for (int b = 0; b < NS; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (bad || k0 + key_lo + 8 * (i >> 1) >= vis[b][i & 1]) s[b][i] = -INFINITY;
            if (mask_from < vis_max) poison = clear_nan<D>(vv, t);
        }
        bool raise = false;
        float mx[NS][2];
#pragma unroll
        for (int b = 0; b < NS; ++b)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                mx[b][e] = fmaxf(s[b][e], s[b][2 + e]);
                raise |= mx[b][e] > m[b][e] + kLag;
            }
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
            for (int b = 0; b < NS; ++b)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1)
                        mx[b][e] = fmaxf(mx[b][e], __shfl_xor_sync(0xffffffffu, mx[b][e], o));
                    const float mn = fmaxf(m[b][e], mx[b][e]);
                    const float f = m[b][e] == mn ? 1.f : ex2(m[b][e] - mn);    // m = -inf: 0
                    m[b][e] = mn;
                    l[b][e] *= f;
#pragma unroll
                    for (int j = 0; j < VJ; ++j) {
                        O[j][b][e] *= f, O[j][b][2 + e] *= f;
                        if (MODE == SPLIT) O[j][NB - 1][e] *= f, O[j][NB - 1][2 + e] *= f;
                    }
                }
        }
        uint32_t pb[NB][2];                 // the value product's operand
#pragma unroll
        for (int b = 0; b < NS; ++b) {
            float p[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float mm = m[b][i & 1];
                p[i] = ex2(s[b][i] - (mm == -INFINITY ? 0.f : mm));
                if (poison && s[b][i] != -INFINITY && ((poison >> (key_lo + 8 * (i >> 1))) & 1u))
                    p[i] = NAN;
                l[b][i & 1] = fmaf(p[i], meta.z, l[b][i & 1]);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float p0 = p[2 * h], p1 = p[2 * h + 1];
                const uint32_t lead = pack_h2(p0, p1);
                pb[b][h] = transpose8(lead);
                if (MODE == SPLIT) pb[NB - 1][h] = transpose8(rest_h2(p0, p1, lead));
            }
        }
#pragma unroll
        for (int x = 0; x < D / 32; ++x) {
            // bytes of the four values paired (key 0, key 1) and (key 2, key 3): bytes 0, 1 and
            // 2, 3 of word x are dims 4x .. 4x+3 of this lane
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                uint32_t a[4];
                h2x2_of(__byte_perm(vv[0][x], vv[1][x], y ? 0x7362 : 0x5140), a[0], a[1]);
                h2x2_of(__byte_perm(vv[2][x], vv[3][x], y ? 0x7362 : 0x5140), a[2], a[3]);
#pragma unroll
                for (int b = 0; b < NB; ++b) mma_f16(O[2 * x + y][b], a, pb[b][0], pb[b][1]);
            }
        }
    }
    cp_wait<0>();
#pragma unroll
    for (int b = 0; b < NS; ++b)            // the eight lanes of a column hold parts of its sum
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int o = 4; o < 32; o <<= 1)
                l[b][e] += __shfl_xor_sync(0xffffffffu, l[b][e], o);

    // ---------------------------------------------------------------- join
    // shared memory: warps' O [4][QT][D], m and l [4][QT]; this CTA's O [QT][D], m, l [QT]
    __syncthreads();
    float* wO = reinterpret_cast<float*>(smem);
    float* wM = wO + kWarps * QT * D;
    float* wL = wM + kWarps * QT;
    float* cO = wL + kWarps * QT;
    float* cM = cO + QT * D;
    float* cL = cM + QT;
    static_assert((kWarps + 1) * (QT * D + 2 * QT) * 4 <= ring_bytes<D>(), "join fits the ring");
    if (MODE == SPLIT) {                    // leading and trailing parts
#pragma unroll
        for (int j = 0; j < VJ; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) O[j][0][i] = fmaf(O[j][NB - 1][i], 1.f / 2048.f, O[j][0][i]);
    }
#pragma unroll
    for (int b = 0; b < NS; ++b)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = 8 * b + 2 * t + e;
            if (r < live) {
                float* o = wO + (warp * QT + r) * D + g * (D / 8);
#pragma unroll
                for (int j = 0; j < VJ; ++j)
                    *reinterpret_cast<float2*>(o + 2 * j) = make_float2(O[j][b][e], O[j][b][2 + e]);
                if (g == 0) wM[warp * QT + r] = m[b][e], wL[warp * QT + r] = l[b][e];
            }
        }
    __syncthreads();
    auto put = [&](int r, int d, float o, float lsum) {
        const int rr = r0 + r;
        out.p[(int64_t)row * out.row + (int64_t)(rr / share) * out.token +
              (int64_t)(kvh * share + rr % share) * D + d] =
            from_f<TO>(lsum == 0.f ? 0.f : o / lsum);
    };
    for (int x = threadIdx.x; x < live * D; x += kWarps * 32) {
        const int r = x / D, d = x % D;
        float M = wM[r];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) M = fmaxf(M, wM[w * QT + r]);
        float o = 0.f, ls = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float mw = wM[w * QT + r];
            const float f = mw == -INFINITY ? 0.f : ex2(mw - M);
            o = fmaf(f, wO[(w * QT + r) * D + d], o);
            ls = fmaf(f, wL[w * QT + r], ls);
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

template <int D, int MODE, int NB, typename TQ, typename TO>
cudaError_t run(const Cache8& c, const QIn<TQ>& q, const Tok8<TO>& out, int heads, int n,
                const int32_t* lens, int lens_add, float scale, const Rope8& rope,
                cudaStream_t st) {
    constexpr int MT = queries_of(MODE, NB);
    auto* kern = k_cache8_attend<D, MODE, NB, TQ, TO>;
    const void* kp = reinterpret_cast<const void*>(kern);
    const int share = heads / c.kv_heads, q_tiles = (n * share + MT - 1) / MT;
    int page_log2 = 4;
    while ((1 << page_log2) < c.page) ++page_log2;
    const int64_t cap = (int64_t)c.row_pages * c.page;
    const int C = ctas_of(cap);
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
    const int64_t nq = (int64_t)n * (heads / c.kv_heads);
#define RLT_RUN(MODE, NB)                                                                       \
    (c.dh == 64 ? run<64, MODE, NB>(c, qi, out, heads, n, lens, lens_add, scale, rope, st)       \
                : run<128, MODE, NB>(c, qi, out, heads, n, lens, lens_add, scale, rope, st))
    if (nq <= 4)
        return launch_cache8_decode<TQ, TO>(c, q, slabs, slab, out, heads, n, lens, lens_add, scale,
                                            rope, st);
    if constexpr (std::is_same<TQ, bf16>::value && std::is_same<TO, bf16>::value)
        return nq <= 8 ? RLT_RUN(PLAIN, 1) : RLT_RUN(PLAIN, 2);
    else
        return RLT_RUN(SPLIT, 2);
#undef RLT_RUN
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
