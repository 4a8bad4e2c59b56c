// Attention over the paged 8-bit cache for 5 and more query vectors per key
// head: blocks of tokens, shared key heads (include/rlt.h: rlt_cache8_attend).
//
// Mathematics, as for fewer queries (k_cache8_decode.cu): bytes enter both
// products as they are, value scales join the weights, and the sum of the
// weights has an exponent of its own.  With a query's a (the largest score, when
// it last rose) and whole number d (the largest s + log2 vs then, less a):
// p_j = 2^(s_j - a), l = sum p_j, w_j = p_j vs_j 2^(7 - d),
// o = sum w_j x^v_j / l * 2^(d - 7).  One exponent for both would lose the
// weights of a page of zeros, whose scale is 2^-110.  Here a CTA
// takes 128 keys at a time through the fifth-generation tensor cores, keys as
// the rows of the first product and value dims as those of the second:
//   S [128 keys][N]  = K [128][D] . Q^T       (K and Q row by row)
//   O [128 dims][N] += V^T [D][128] . w       (V and w as they lie, key by key)
// Both accumulators live in tensor memory.  One CTA an SM, three kinds of
// warps, two tiles of everything in turn:
//   8 convert  16 keys each: e4m3 bytes become fp16 (exactly) on their way
//              from registers, where the next tile's bytes arrive (the one
//              after is on its way to L2), to swizzled shared memory; one layout
//              [dims/64][key][64 dims] serves K, read along the dims, and V,
//              read across them;
//   1 issues   the products: tile i + 1's first one before tile i's second;
//   8 weigh    (16 for 64 columns) a thread has one key and, by its set of four
//              warps, 8 or 16 of the columns: weights need no exchange between
//              lanes, and any number of queries keeps all lanes busy.
//
// PARTS = 2 (fp32 types): columns 2i and 2i + 1 hold query i's (weight i's)
// leading 11 bits and the next 11 bits times 2^11, added in fp32.  PARTS = 1
// (bf16 types): leading bits alone.  Each query is brought near 1 by a power
// of two first: a bf16 query is exact then, a rotated one is rounded to fp16
// (half a step 2^-11 at most), as weights are: below the bf16 output's 2^-8.
// fp16 holds 2^-14 to 2^16, so a weight keeps its bits down to 2^-20 of the
// query's largest; below, it is off by 2^-31 (two parts: 2^-42) of that.
//
// a and d are raised only when a score or a weight passes them by 2^8 (one
// barrier vote per tile); then the columns' maxima are found and O rescaled.
//
// 16 rows of 103 to 20011 keys x 4 key heads x 32 queries (165 MB) take 112-114 us against
// 26 of the bytes: a tile takes about 2300 cycles (its conversion, its two products and
// its weighing are some 1400 each and wait for one another), a CTA's start and end
// about 17000.  fp32 types: 165 us.  (Sixteen queries a warp through m16n8k16 products, every key converted
// by each warp: 174 us; one stage, two CTAs an SM: 121.)  One register budget serves all
// three kinds of warps: at head size 128 a thread spills 88 to 140 bytes at 32 columns (96
// registers) and 344 to 484 at 64 (72 registers).
//
// Split.  The prefix of a (row, key head) is cut into runs of 2048 keys, or 4
// longer ones (16 from 32768 keys on), for a CTA each, a function of that
// prefix alone; they join through the cluster's distributed shared memory in
// run order: no scratch, no atomics, and the same bits for a row whatever batch
// or capacity it sits in.  The grid is the capacity's, though: CTAs past a row's own
// take tensor memory, read its length and leave.
#include <cooperative_groups.h>

#include <algorithm>

#include "cache8_tile.cuh"

namespace cg = cooperative_groups;

namespace rlt {
namespace {

constexpr int kConvert = 8;             // warps that convert
// warps that weigh, four to a set of columns; one more issues (16 for 64 columns: 16 rows of 103 to
// 20011 keys x 4 key heads x 128 queries took 294 us, now 277, and 318 with 8; for 32 columns 135 and
// 122)
constexpr int weigh_warps(int N) { return N == 64 ? 16 : 8; }
constexpr int threads_of(int N) { return 32 * (weigh_warps(N) + kConvert + 1); }
constexpr int kKeys = 128;              // of a tile
constexpr int kKeysPerCta = 2048;
constexpr int64_t kLongKeys = 32768;    // from here on
constexpr int kMaxCtas = 16;            // of a prefix: a cluster's most
// Larger clusters wait for as many SMs of one group of SMs to be free at once: 16 rows of 20011 keys
// x 4 key heads take 135, 149, 165, 214 us with at most 2, 4, 6, 8.  Fewer CTAs serve a few rows
// worse: a row's own time grows (103 to 20011 keys: 133, 121, 118, 127 us).
constexpr int kFewCtas = 4;
constexpr float kLag = 8.f;             // how far (log2) a score may pass a, with its value scale a + d
constexpr float kUp = 7.f;              // weights are up to 2^(kLag + kUp), within fp16's 2^16
constexpr float kNone = -3e38f;         // below every finite score
constexpr uint32_t kAtom = kKeys * 128; // 64 dims of 128 keys in fp16

// CTAs that share a prefix of `keys` keys: of kKeysPerCta keys each, then of more
__host__ __device__ __forceinline__ int ctas_of(int64_t keys) {
    const int64_t c = (keys + kKeysPerCta - 1) / kKeysPerCta;
    const int most = keys >= kLongKeys ? kMaxCtas : kFewCtas;
    return c < 1 ? 1 : c > most ? most : (int)c;
}
// Instruction descriptor: fp16 A and B, fp32 accumulator, M = 128; mn: both operands are stored
// along M and N rather than K.
constexpr uint32_t idesc_f16(int N, bool mn) {
    return (1u << 4) | (mn ? 3u << 15 : 0u) | ((uint32_t)(N >> 3) << 17) | ((128u >> 4) << 24);
}
// Shared-memory descriptor, 128-byte swizzle, stored along M (or N): 64 of them by 8 of K make an
// atom; atoms follow each other along K every 1024 bytes (SBO), along M every kAtom (LBO).
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(kAtom >> 4) << 16) | (64ull << 32) |
           (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ void mma_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                           bool accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t at, float* v) {
    uint32_t r[8];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7])
        : "r"(at));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st8(uint32_t at, const float* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(at),
        "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
        "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
        "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7])));
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void fence_async_shared() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ uint32_t key_of(float x) {   // order-preserving
    const uint32_t u = __float_as_uint(x);
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float float_of(uint32_t k) {
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

// two fp32 values in one register pair: one instruction for both
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
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

template <int D, int N>
constexpr size_t smem_of() {
    return 1024 + (size_t)(D / 64) * (4 * kAtom + N * 128) + 2 * kAtom;
}

// N columns of PARTS a query
template <int D, int N, int PARTS, typename TQ, typename TO>
__global__ void __launch_bounds__(threads_of(N), 1)
k_cache8_attend(Cache8 c, int page_log2, QIn<TQ> q, Tok8<TO> out, int share, int n, int q_tiles,
                const int32_t* __restrict__ lens, int lens_add, float scale_log2e, Rope8 rope) {
    constexpr int QT = N / PARTS;               // query vectors of a tile
    constexpr int kWarps = weigh_warps(N), kWeigh = 32 * kWarps, kThreads = threads_of(N);
    constexpr int NC = 4 * N / kWarps, NQ = NC / PARTS;     // a weighing thread's columns, and queries
    static_assert(NC == 8 || NC == 16, "a load of scores");
    constexpr int NL = D / 32;                  // a thread's 16-byte loads of K (and of V) per tile
    constexpr uint32_t kCols = 4 * N;           // tensor memory: S twice, then O (of two tiles)
    extern __shared__ uint8_t raw[];
    // per query: score factor; a (0 before the first score); how far a score and log2 of its value
    // scale together may pass a (kLag + d; kNone before the first score); 2^(kUp - d); the last rise of
    // a, and what it leaves of l and of O
    __shared__ __align__(16) float s_rf[QT], s_m[QT], s_room[QT], s_g[QT], s_up[QT], s_f[QT], s_fo[QT];
    __shared__ __align__(16) int s_vis[QT];
    __shared__ int64_t s_out[QT];               // where its output goes
    // Of a tile's 16-key groups: ks, vs, log2 vs or the whole number above (-inf: no such keys); the
    // keys with a NaN value.  Four tiles': K of
    // tile i + 2 is converted while tile i may still be weighed (V of i + 2 is not).
    __shared__ float4 s_meta[4][kKeys / 16];
    __shared__ uint32_t s_poison[4][kKeys / 16];
    __shared__ float s_red[4][QT], s_red2[4][QT];
    __shared__ __align__(8) uint64_t s_k[2], s_v[2], s_s[2], s_w[2], s_o[2];   // K, V, S, w there; O done
    __shared__ __align__(8) uint64_t s_there[4];                              // a tile's s_meta
    __shared__ __align__(8) uint64_t s_end;             // all products issued, after a wait gave up
    __shared__ int s_abort;
    __shared__ uint32_t s_tmem;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // Before the next kernel of the stream may start: it could take the tensor memory that this
    // CTA needs and then wait for this grid.
    if (warp == 0) tc::tmem_alloc(&s_tmem, kCols);
    if (tid == 0) {
        for (int b = 0; b < 2; ++b) {
            tc::mbar_init(&s_k[b], kConvert);
            tc::mbar_init(&s_v[b], kConvert);
            tc::mbar_init(&s_s[b], 1);
            tc::mbar_init(&s_w[b], kWarps);
            tc::mbar_init(&s_o[b], 1);
        }
        for (int b = 0; b < 4; ++b) tc::mbar_init(&s_there[b], kConvert);
        tc::mbar_init(&s_end, 1);
        s_abort = 0;
        tc::fence_mbar_init();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = s_tmem;
    pdl_enter();
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int unit = (int)(blockIdx.x / (unsigned)C);
    const int mt = unit % q_tiles, bh = unit / q_tiles;
    const int kvh = bh % c.kv_heads, row = bh / c.kv_heads;
    const int nq = n * share;

    const int cap = c.row_pages << page_log2;
    const int L0 = __ldg(lens + row) + lens_add;
    const int L = max(0, min(cap, L0));
    auto say = [&](int code) {
        if (c.status) atomicCAS(c.status, 0, code);
    };
    if ((L0 < 0 || L0 > cap) && tid == 0 && kvh == 0 && mt == 0 && rank == 0) say(c.cap_code);
    const int r0 = mt * QT, live = min(QT, nq - r0);
    const int keys = max(0, L - n + (r0 + live - 1) / share + 1);   // any query of the tile sees
    const int vis_min = L - n + r0 / share + 1;                     // all of them see
    const int nC = min(C, ctas_of(keys));
    if (rank >= nC) {
        if (warp == 0) tc::tmem_dealloc(tmem, kCols);
        return;
    }
    const int tiles = (keys + kKeys - 1) / kKeys, per = (tiles + nC - 1) / nC;
    const int t_begin = min(tiles, rank * per), t_end = min(tiles, t_begin + per);

    uint8_t* const base = reinterpret_cast<uint8_t*>(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    constexpr uint32_t KV = (D / 64) * kAtom;
    uint8_t* const K16 = base;                              // 2 x [D/64][key][64 dims]
    uint8_t* const V16 = K16 + 2 * KV;
    uint8_t* const W16 = V16 + 2 * KV;                      // 2 x weights [key][64 columns]
    uint8_t* const Q16 = W16 + 2 * kAtom;                   // [D/64][column][64 dims]
    // a bounded wait; once one gave up all do
    auto wait_for = [&](uint64_t* bar, int use) {
        for (uint32_t polls = 0; polls < (1u << 22); ++polls) {
            if (tc::mbar_try(bar, (uint32_t)use & 1u)) return true;
            if (*(volatile int*)&s_abort) return false;
        }
        *(volatile int*)&s_abort = 1;
        return false;
    };
    auto wait = [&](uint64_t* bar, int i) { return wait_for(bar, i >> 1); };    // its use by tile i
    auto arrive = [&](uint64_t* bar) {                      // the warp's writes are done
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar);
    };

    // ---------------------------------------------------------------- the next tile's bytes
    // a converting warp copies 16 keys, which share a page: lane (r, ch) chunk ch (and ch + 4) of
    // key r, r + 8
    const size_t head_bytes = (size_t)D << page_log2;
    const size_t v_bytes = (size_t)c.kv_heads * head_bytes;
    const int lr = lane >> 2, lc = lane & 3;
    const int cw = warp - kWarps;               // which of them
    uint4 kb[NL], vb[NL];
    float ks = 0.f, vs = 0.f;                   // vs = 0: no such keys
    int page_1 = -1, page_2 = -1;               // of the tile loaded next, and of the one after
    int entry = -1;                             // the table's, for the tile after that
    auto entry_of = [&](int tile) {
        const int k0 = tile * kKeys + cw * 16;
        return tile < t_end && k0 < keys
                   ? __ldg(c.table + (size_t)row * c.row_pages + (k0 >> page_log2)) : -1;
    };
    auto page_of = [&](int tile, int p) {       // -1: past the prefix, or bad
        if (p >= 0 && p < c.n_pages) return p;
        if (lane == 0 && tile < t_end && tile * kKeys + cw * 16 < keys) say(c.arg_code);
        return -1;
    };
    auto bytes_of = [&](int tile, int page) {
        const int k0 = tile * kKeys + cw * 16;
        return c.pages + ((size_t)max(page, 0) * 2 * c.kv_heads + kvh) * head_bytes +
               (size_t)((k0 & ((1 << page_log2) - 1)) * D);
    };
    auto load_half = [&](int tile, bool values, uint4 (&b)[NL]) {
        const int k0 = tile * kKeys + cw * 16;
        const uint8_t* from = bytes_of(tile, page_1) + lr * D + lc * 16 + (values ? v_bytes : 0);
#pragma unroll
        for (int j = 0; j < NL; ++j) {
            const int r8 = D == 128 ? j >> 1 : j, off = r8 * 8 * D + (D == 128 ? (j & 1) * 64 : 0);
            const bool ok = page_1 >= 0 && k0 + lr + 8 * r8 < keys;
            b[j] = ok ? __ldg(reinterpret_cast<const uint4*>(from + off)) : make_uint4(0, 0, 0, 0);
        }
    };
    auto load_scales = [&]() {
        vs = 0.f;
        if (page_1 >= 0) {
            const float* sc = c.scales + (size_t)page_1 * 2 * c.kv_heads + kvh;
            ks = __ldg(sc);
            vs = __ldg(sc + c.kv_heads);
        }
    };
    auto ahead = [&](int tile) {                // 128 bytes a lane: K by the first half, then V
        const int at = (lane & 15) * 128;
        if (page_2 >= 0 && at < 16 * D) {
            const uint8_t* p = bytes_of(tile, page_2) + at + (lane < 16 ? 0 : v_bytes);
            asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
        }
    };
    const bool converts = warp >= kWarps && warp < kWarps + kConvert;
    if (converts) {
        const int e0 = entry_of(t_begin), e1 = entry_of(t_begin + 1);
        entry = entry_of(t_begin + 2);
        page_1 = page_of(t_begin, e0);
        load_scales();
        load_half(t_begin, false, kb);
        load_half(t_begin, true, vb);
        page_2 = page_of(t_begin + 1, e1);
        ahead(t_begin + 1);
    }

    // queries: D/4 lanes to each, four dims a lane; the first QB of a lane's QR on their way first
    constexpr int QR = QT * (D / 4) / kWeigh > 0 ? QT * (D / 4) / kWeigh : 1, QB = QR < 4 ? QR : 4;
    static_assert(QR * kWeigh >= QT * (D / 4), "all queries");
    const int qd = (tid % (D / 4)) * 4;
    auto q_of = [&](int j) { return j * (kWeigh / (D / 4)) + tid / (D / 4); };
    auto fetch_q = [&](int r, int i, Q4<TQ>& v) {       // (of token i) false: nothing to see
        if (r >= live) return false;
        const int rr = r0 + r, pos = L - n + i + rope.origin;
        if (L - n + i < 0) return false;
        if (rope.rot && (pos < 0 || pos >= rope.positions)) {
            if (qd == 0) say(c.cap_code);
            return false;
        }
        v.load(q, (size_t)((int64_t)row * q.row + (int64_t)i * q.token) +
                      (size_t)(kvh * share + rr - i * share) * D, qd, rope, pos);
        return true;
    };
    // ---------------------------------------------------------------- queries: fp16 columns
    auto put_q = [&](int r, int i, bool in, Q4<TQ>& v) {
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (in) x = v.turned(qd, rope);
        float amax = fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w)));
#pragma unroll
        for (int o = D / 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        if (r >= QT) return;                    // (D = 64, N = 16: half of the threads have none)
        // bring the query near 1 by a power of two (exact); 2^+-100 keeps both factors finite
        int e2 = (int)(__float_as_uint(amax) >> 23) - 127;
        e2 = max(-100, min(100, e2));
        const float down = __uint_as_float((uint32_t)(127 - e2) << 23);
        x.x *= down, x.y *= down, x.z *= down, x.w *= down;
        const uint32_t h0 = pack_h2(x.x, x.y), h1 = pack_h2(x.z, x.w);
#pragma unroll
        for (int z = 0; z < PARTS; ++z) {
            const int col = r * PARTS + z, ch = (qd & 63) >> 3;
            *reinterpret_cast<uint2*>(Q16 + (qd >> 6) * (N * 128) + col * 128 +
                                      ((ch ^ (col & 7)) << 4) + (qd & 4) * 2) =
                z ? make_uint2(rest_h2(x.x, x.y, h0), rest_h2(x.z, x.w, h1)) : make_uint2(h0, h1);
        }
        if (qd == 0) {
            const int pos = L - n + i + rope.origin;
            int vis = r < live ? max(0, L - n + i + 1) : 0;
            if (rope.rot && (pos < 0 || pos >= rope.positions)) vis = 0;
            s_rf[r] = __uint_as_float((uint32_t)(127 + e2) << 23) * scale_log2e;
            s_m[r] = 0.f;
            s_room[r] = kNone;
            s_g[r] = 1.f;
            s_vis[r] = vis;
            s_out[r] = (int64_t)row * out.row + (int64_t)i * out.token +
                       (int64_t)(kvh * share + (r0 + r - i * share)) * D;
        }
    };
    if (warp < kWarps) {
        Q4<TQ> q4[QB];
        bool in[QB];
        int of[QB];
#pragma unroll
        for (int j0 = 0; j0 < QR; j0 += QB) {
#pragma unroll
            for (int j = 0; j < QB; ++j) {
                of[j] = (r0 + q_of(j0 + j)) / share;
                in[j] = fetch_q(q_of(j0 + j), of[j], q4[j]);
            }
#pragma unroll
            for (int j = 0; j < QB; ++j) put_q(q_of(j0 + j), of[j], in[j], q4[j]);
        }
        fence_async_shared();
    }
    __syncthreads();
    // a query without a rotation sees nothing: its column has to be masked from the first key on
    int lost = 0;
    if (tid < live) lost = s_vis[tid] < vis_min;
    const int mask_from = __syncthreads_or(lost) ? 0 : vis_min;

    // ---------------------------------------------------------------- the run
    const int T = t_end - t_begin;
    const int part = warp >> 2, key = tid & 127;            // a weighing thread's columns, and key
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t S = tmem + lanes + part * NC, O = tmem + lanes + 2 * N + part * NC;
    float l[NQ], acc[PARTS == 2 ? NQ : 1];                  // (acc: PARTS = 2, below)
#pragma unroll
    for (int i = 0; i < NQ; ++i) l[i] = 0.f;
#pragma unroll
    for (int i = 0; i < (PARTS == 2 ? NQ : 1); ++i) acc[i] = 0.f;
    // PARTS = 2: a tile's O, leading and trailing parts, joins the others in fp32 registers (a
    // thread's dim and its queries): the tensor cores' own sum over a long prefix truncates
    auto add_tile = [&](int i) {
        if constexpr (PARTS == 2) {
#pragma unroll
            for (int j = 0; j < NC; j += 8) {
                float o[8];
                tmem_ld8(O + (i & 1) * N + j, o);
#pragma unroll
                for (int z = 0; z < 8; z += 2) acc[(j + z) / 2] += fmaf(o[z + 1], 1.f / 2048.f, o[z]);
            }
        }
    };
    if (converts) {
        auto convert = [&](uint8_t* to, const uint4 (&b)[NL]) {
#pragma unroll
            for (int j = 0; j < NL; ++j) {
                const int r = cw * 16 + lr + 8 * (D == 128 ? j >> 1 : j);
                uint8_t* at = to + (D == 128 ? (j & 1) * kAtom : 0) + r * 128;
                uint4 x, y;
                h2x2_of(b[j].x, x.x, x.y);
                h2x2_of(b[j].y, x.z, x.w);
                h2x2_of(b[j].z, y.x, y.y);
                h2x2_of(b[j].w, y.z, y.w);
                *reinterpret_cast<uint4*>(at + (((2 * lc) ^ (r & 7)) << 4)) = x;
                *reinterpret_cast<uint4*>(at + (((2 * lc + 1) ^ (r & 7)) << 4)) = y;
            }
        };
        for (int i = 0; i < T; ++i) {
            const int b = i & 1, tile = t_begin + i;
            if (i >= 2 && !wait(&s_s[b], i - 2)) break;     // tile i - 2's K is done with
            convert(K16 + b * KV, kb);
            uint32_t poison = 0;
            if ((tile + 1) * kKeys > mask_from && mask_from < keys) {
                // A value seen by some queries only: a NaN in it would reach the others as 0 x NaN,
                // so it enters the product as 0 and the weights of those that see it become NaN.
#pragma unroll
                for (int j = 0; j < NL; ++j) {
                    uint32_t* w = &vb[j].x;
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const uint32_t z = ((w[x] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                        if (z) poison |= 1u << (lr + 8 * (D == 128 ? j >> 1 : j));
                        w[x] &= ~((z >> 7) * 0xffu);
                    }
                }
                poison = __reduce_or_sync(0xffffffffu, poison);
            }
            if (lane == 0) {
                // log2 vs, rounded up
                const int up = (int)((__float_as_uint(vs) + 0x7fffffu) >> 23) - 127;
                s_meta[i & 3][cw] = vs > 0.f ? make_float4(ks, vs, (float)up, 0.f)
                                         : make_float4(0.f, 0.f, -INFINITY, 0.f);
                s_poison[i & 3][cw] = poison;
            }
            fence_async_shared();
            arrive(&s_k[b]);
            if (lane == 0) tc::mbar_arrive(&s_there[i & 3]);
            page_1 = page_2;
            load_half(tile + 1, false, kb);
            load_scales();
            if (i >= 2 && !wait(&s_o[b], i - 2)) break;     // and its V
            convert(V16 + b * KV, vb);
            fence_async_shared();
            arrive(&s_v[b]);
            load_half(tile + 1, true, vb);
            page_2 = page_of(tile + 2, entry);
            ahead(tile + 2);
            entry = entry_of(tile + 3);
        }
    } else if (warp == kWarps + kConvert) {
        if (lane == 0) {
            // descriptors count in 16 bytes: a step adds to them
            const uint64_t k16 = tc::sdesc_k_sw128(tc::smem_u32(K16)),
                           q16 = tc::sdesc_k_sw128(tc::smem_u32(Q16)),
                           v16 = sdesc_mn_sw128(tc::smem_u32(V16)),
                           w16 = sdesc_mn_sw128(tc::smem_u32(W16));
            auto scores = [&](int i) {
                const int b = i & 1;
                if (!wait(&s_k[b], i)) return false;
                tc::fence_after_sync();
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    mma_f16_ss(tmem + b * N,
                               k16 + ((b * KV + (k >> 2) * kAtom + (k & 3) * 32) >> 4),
                               q16 + (((k >> 2) * (N * 128) + (k & 3) * 32) >> 4),
                               idesc_f16(N, false), k > 0);
                tc::mma_commit(&s_s[b]);
                return true;
            };
            bool ok = T > 0 && scores(0);
            for (int i = 0; i < T && ok; ++i) {
                // (tile i - 1's weights are there: S of tile i + 1 may overwrite its scores)
                if (i + 1 < T) ok = scores(i + 1);
                const int b = i & 1;
                ok = ok && wait(&s_v[b], i) && wait(&s_w[b], i);
                if (!ok) break;
                tc::fence_after_sync();
#pragma unroll
                for (int k = 0; k < kKeys / 16; ++k)
                    mma_f16_ss(tmem + 2 * N + (PARTS == 2 ? b * N : 0), v16 + ((b * KV + k * 2048) >> 4),
                               w16 + ((b * kAtom + k * 2048) >> 4), idesc_f16(N, true),
                               k > 0 || (PARTS == 1 && i > 0));
                tc::mma_commit(&s_o[b]);
            }
        }
        __syncwarp();
    } else {
        auto vote = [&](bool x) {                           // any of the weighing threads
            uint32_t any;
            asm volatile(
                "{\n .reg .pred p, r;\n setp.ne.u32 p, %1, 0;\n"
                " barrier.cta.red.or.pred r, 1, %2, p;\n selp.u32 %0, 1, 0, r;\n}\n"
                : "=r"(any)
                : "r"((uint32_t)x), "n"(kWeigh)
                : "memory");
            __syncwarp();
            return any != 0;
        };
        for (int i = 0; i < T; ++i) {
            const int b = i & 1, k0 = (t_begin + i) * kKeys;
            const bool tail = k0 + kKeys > mask_from;       // the prefix ends here for some query
            bool ok = wait_for(&s_there[i & 3], i >> 2) && wait(&s_s[b], i);     // scalars; scores
            ok = ok && (i < 2 || wait(&s_o[b], i - 2));             // and w's place is free
            __syncwarp();
            tc::fence_after_sync();
            // scores of this thread's key, less the queries' a
            const float4 meta = s_meta[i & 3][key >> 4];
            float x[NQ];
            {
                float cf[NC];
                if constexpr (NC == 8) tmem_ld8(S + b * N, cf);
                else tc::tmem_ld16(S + b * N, cf);
#pragma unroll
                for (int j = 0; j < NQ; ++j)
                    x[j] = PARTS == 2 ? fmaf(cf[PARTS * j + PARTS - 1], 1.f / 2048.f, cf[PARTS * j])
                                      : cf[j];
            }
            bool raise = false;
#pragma unroll
            for (int j = 0; j < NQ; j += 4) {
                const int at = (part * NQ + j) / 4;
                const float4 rf = reinterpret_cast<const float4*>(s_rf)[at];
                const float4 mq = reinterpret_cast<const float4*>(s_m)[at];
                const float4 room = reinterpret_cast<const float4*>(s_room)[at];
                const uint64_t k2 = pair(meta.x, meta.x);
                unpair(fma2(pair(x[j], x[j + 1]), mul2(pair(rf.x, rf.y), k2), pair(-mq.x, -mq.y)),
                       x[j], x[j + 1]);
                unpair(fma2(pair(x[j + 2], x[j + 3]), mul2(pair(rf.z, rf.w), k2),
                            pair(-mq.z, -mq.w)),
                       x[j + 2], x[j + 3]);
                if (tail) {
                    const int4 vis = reinterpret_cast<const int4*>(s_vis)[at];
                    if (k0 + key >= vis.x) x[j] = -INFINITY;
                    if (k0 + key >= vis.y) x[j + 1] = -INFINITY;
                    if (k0 + key >= vis.z) x[j + 2] = -INFINITY;
                    if (k0 + key >= vis.w) x[j + 3] = -INFINITY;
                }
                raise |= x[j] > fminf(kLag, room.x - meta.z) ||
                         x[j + 1] > fminf(kLag, room.y - meta.z) ||
                         x[j + 2] > fminf(kLag, room.z - meta.z) ||
                         x[j + 3] > fminf(kLag, room.w - meta.z);
            }
            if (meta.z == -INFINITY) {                      // no such key: not even a NaN of it
                raise = false;
#pragma unroll
                for (int j = 0; j < NQ; ++j) x[j] = -INFINITY;
            }
            if (PARTS == 2 && i) {
                ok = ok && wait(&s_o[b ^ 1], i - 1);
                __syncwarp();
                tc::fence_after_sync();
                add_tile(i - 1);
            }
            ok = ok && *(volatile int*)&s_abort == 0;
            if (vote(raise || !ok)) {
                if (vote(!ok)) break;                       // all of them
#pragma unroll
                for (int j = 0; j < NQ; ++j) {
                    const float y = x[j] == x[j] ? x[j] : -INFINITY;
                    const float top = float_of(__reduce_max_sync(0xffffffffu, key_of(y)));
                    const float top2 = float_of(__reduce_max_sync(0xffffffffu, key_of(y + meta.z)));
                    if (lane == 0) s_red[warp & 3][part * NQ + j] = top, s_red2[warp & 3][part * NQ + j] = top2;
                }
                vote(false);
                if (tid < QT) {
                    const float top = fmaxf(fmaxf(s_red[0][tid], s_red[1][tid]),
                                            fmaxf(s_red[2][tid], s_red[3][tid]));
                    const float top2 = fmaxf(fmaxf(s_red2[0][tid], s_red2[1][tid]),
                                             fmaxf(s_red2[2][tid], s_red2[3][tid]));
                    if (top > kNone) {                      // (else no score, here or so far: as it was)
                        const bool none = s_room[tid] == kNone;     // sums of 0 so far
                        // (the largest score itself: a key that dwarfs the others weighs exactly 1)
                        const float up = none ? top : fmaxf(0.f, top);
                        const float left = s_room[tid] - kLag - up;         // d, were it to stay a + d
                        // -105: p 2^(kUp - d) stays finite; scales of zeros alone lie below
                        float d = fmaxf(-105.f, ceilf(top2 - up));
                        if (!none) d = fmaxf(d, ceilf(left));
                        s_up[tid] = up;
                        s_f[tid] = none ? 1.f : ex2(-up);
                        s_fo[tid] = none ? 1.f : ex2(left - d);
                        s_m[tid] += up;
                        s_room[tid] = kLag + d;
                        s_g[tid] = ex2(kUp - d);
                    } else {
                        s_up[tid] = 0.f;
                        s_f[tid] = s_fo[tid] = 1.f;
                    }
                }
                if (i) ok = wait(&s_o[b ^ 1], i - 1);       // the product before this has finished
                if (vote(!ok)) break;
                tc::fence_after_sync();
                // (the sums so far shrink: in registers, or in tensor memory)
#pragma unroll
                for (int j = 0; j < NQ; ++j) {
                    x[j] -= s_up[part * NQ + j];
                    l[j] *= s_f[part * NQ + j];
                    if (PARTS == 2) acc[PARTS == 2 ? j : 0] *= s_fo[part * NQ + j];
                }
                if (PARTS == 1 && i)
#pragma unroll
                    for (int j = 0; j < NC; j += 8) {
                        float o[8];
                        tmem_ld8(O + j, o);
#pragma unroll
                        for (int z = 0; z < 8; ++z) o[z] *= s_fo[part * NQ + j + z];
                        tmem_st8(O + j, o);
                    }
            }
            const bool poisoned =
                tail && mask_from < keys && ((s_poison[i & 3][key >> 4] >> (key & 15)) & 1u);
#pragma unroll
            for (int j = 0; j < NC; j += 8) {               // weights, 8 columns at a time
                uint32_t w[4];
#pragma unroll
                for (int z = 0; z < 8 / PARTS; z += 4) {
                    const float4 g = reinterpret_cast<const float4*>(s_g)[(part * NQ + j / PARTS + z) / 4];
                    float p[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int qi = j / PARTS + z + e;
                        p[e] = ex2(x[qi]);
                        if (poisoned && x[qi] != -INFINITY) p[e] = NAN;
                        l[qi] += p[e];
                    }
                    // (finite factors: a weight of 0 stays 0)
                    const uint64_t v2 = pair(meta.y, meta.y);
                    unpair(mul2(mul2(pair(p[0], p[1]), pair(g.x, g.y)), v2), p[0], p[1]);
                    unpair(mul2(mul2(pair(p[2], p[3]), pair(g.z, g.w)), v2), p[2], p[3]);
                    if (PARTS == 2) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float h = __half2float(__float2half_rn(p[e]));
                            w[e] = pack_h2(h, (p[e] - h) * 2048.f);
                        }
                    } else {
                        w[z / 2] = pack_h2(p[0], p[1]);
                        w[z / 2 + 1] = pack_h2(p[2], p[3]);
                    }
                }
                const int ch = (part * NC + j) >> 3;
                *reinterpret_cast<uint4*>(W16 + b * kAtom + key * 128 + ((ch ^ (key & 7)) << 4)) =
                    make_uint4(w[0], w[1], w[2], w[3]);
            }
            fence_async_shared();
            tc::fence_before_sync();
            arrive(&s_w[b]);
        }
        if (T > 0) {
            wait(&s_o[(T - 1) & 1], T - 1);
            __syncwarp();
            tc::fence_after_sync();
            add_tile(T - 1);
        }
    }
    __syncthreads();
    tc::fence_after_sync();
    if (s_abort) {                          // a bounded wait gave up
        if (tid == 0) say(c.late_code);
        if (tid == 32 * (kWarps + kConvert)) {      // products under way end before their memory goes
            tc::mma_commit(&s_end);
            tc::mbar_wait(&s_end, 0, 1u << 22);
        }
    }

    // ---------------------------------------------------------------- join
    // l over the 128 keys, then this CTA's O [query][D], m, l
    float* const c_o = reinterpret_cast<float*>(K16);
    float* const c_l = s_rf;                                // (the queries' factors are done with)
    if (warp < kWarps) {
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
            const float s = warp_sum(l[j]);
            if (lane == 0) s_red[warp & 3][part * NQ + j] = s;
        }
    }
    __syncthreads();
    float* const c_d = s_room;
    if (tid < QT) {
        c_l[tid] = (s_red[0][tid] + s_red[1][tid]) + (s_red[2][tid] + s_red[3][tid]);
        if (c_d[tid] == kNone) s_m[tid] = -INFINITY, c_d[tid] = 0.f;     // a run without a score
        else c_d[tid] -= kLag;
        const float by = c_d[tid] - kUp, half = floorf(0.5f * by);      // 2^by / l in two factors
        s_f[tid] = c_l[tid] == 0.f ? 0.f : ex2(half) / c_l[tid];
        s_fo[tid] = ex2(by - half);
    }
    __syncthreads();
    if (warp < kWarps) {
        const int dim = 32 * (warp & 3) + lane;
#pragma unroll
        for (int j = 0; j < NC; j += 8) {
            float o[8];
            if (PARTS == 1 && T > 0) {
                tmem_ld8(O + j, o);
            } else {
#pragma unroll
                for (int z = 0; z < 8; ++z) o[z] = 0.f;
            }
#pragma unroll
            for (int z = 0; z < 8; z += PARTS) {
                const int r = part * NQ + (j + z) / PARTS;
                const float v = PARTS == 2 ? acc[PARTS == 2 ? (j + z) / 2 : 0] : o[z];
                if (r < live && dim < D) {
                    if (nC == 1)
                        out.p[s_out[r] + dim] =
                            from_f<TO>(c_l[r] == 0.f ? 0.f : v * s_f[r] * s_fo[r]);
                    else c_o[r * D + dim] = v;
                }
            }
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 0) tc::tmem_dealloc(tmem, kCols);
    if (nC == 1) return;
    cluster.sync();                         // (CTAs without a run have exited)
    // Every CTA's sums as one, in CTA order, each by its factor; this CTA's share of the outputs.
    // Every remote load of a thread is in flight at once: one after another, 16 CTAs took 12 us.
    float* const j_a = reinterpret_cast<float*>(W16);       // [cta][query]: a, later O's factor
    float* const j_d = j_a + kMaxCtas * QT;
    float* const j_l = j_d + kMaxCtas * QT;
    float* const j_sum = j_l + kMaxCtas * QT;               // l of all, and 2^(a + d - kUp) in two
    float* const j_by = j_sum + QT;
    static_assert((3 * kMaxCtas + 2) * QT * 4 <= 2 * kAtom, "they fit");
    for (int x = tid; x < nC * live; x += kThreads) {
        const int k = x / live, r = x - k * live;
        j_a[x] = *cluster.map_shared_rank(s_m + r, k);
        j_d[x] = *cluster.map_shared_rank(c_d + r, k);
        j_l[x] = *cluster.map_shared_rank(c_l + r, k);
    }
    __syncthreads();
    for (int r = tid; r < live; r += kThreads) {
        float top = -INFINITY, a = -INFINITY, d = 0.f, most = -INFINITY, ls = 0.f;
        for (int k = 0; k < nC; ++k) {          // the largest a; a and d of the largest a + d
            const float ak = j_a[k * live + r], dk = j_d[k * live + r];
            top = fmaxf(top, ak);
            if (ak + dk > most) most = ak + dk, a = ak, d = dk;
        }
        for (int k = 0; k < nC; ++k) {
            const int x = k * live + r;
            const float ak = j_a[x];
            const bool none = ak == -INFINITY;
            ls = fmaf(none ? 0.f : ex2(ak - top), j_l[x], ls);
            j_a[x] = none ? 0.f : ex2((ak - a) + (j_d[x] - d));
        }
        j_sum[r] = ls;
        j_by[r] = (a - top) + (d - kUp);
    }
    __syncthreads();
    for (int x = rank * kThreads + tid; x < live * D; x += nC * kThreads) {
        const int r = x / D;
        float v[kMaxCtas];
#pragma unroll
        for (int k = 0; k < kMaxCtas; ++k) v[k] = k < nC ? *cluster.map_shared_rank(c_o + x, k) : 0.f;
        float o = 0.f;
#pragma unroll
        for (int k = 0; k < kMaxCtas; ++k)
            if (k < nC) o = fmaf(j_a[k * live + r], v[k], o);
        const float by = j_by[r], half = floorf(0.5f * by);
        out.p[s_out[r] + x - r * D] =
            from_f<TO>(j_sum[r] == 0.f ? 0.f : o / j_sum[r] * ex2(half) * ex2(by - half));
    }
    cluster.sync();                         // no CTA leaves while its memory is read
}

template <int D, int N, int PARTS, typename TQ, typename TO>
cudaError_t run(const Cache8& c, const QIn<TQ>& q, const Tok8<TO>& out, int heads, int n,
                const int32_t* lens, int lens_add, float scale, const Rope8& rope,
                cudaStream_t st) {
    auto* kern = k_cache8_attend<D, N, PARTS, TQ, TO>;
    const void* kp = reinterpret_cast<const void*>(kern);
    const int share = heads / c.kv_heads, q_tiles = (n * share + N / PARTS - 1) / (N / PARTS);
    int page_log2 = 4;
    while ((1 << page_log2) < c.page) ++page_log2;
    const int64_t cap = (int64_t)c.row_pages * c.page;
    const int C = ctas_of(cap);
    const int64_t ctas = (int64_t)c.rows * c.kv_heads * q_tiles * C;
    if (ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
    constexpr size_t smem = smem_of<D, N>();
    if (!set_smem_once(kp, smem) || (C > 8 && !set_wide_cluster_once(kp)))
        return cudaErrorInvalidConfiguration;
    set_carveout_once(kp);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(threads_of(N));
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
    if (nq <= 4)
        return launch_cache8_decode<TQ, TO>(c, q, slabs, slab, out, heads, n, lens, lens_add, scale,
                                            rope, st);
    constexpr int P = std::is_same<TQ, bf16>::value && std::is_same<TO, bf16>::value ? 1 : 2;
#define RLT_RUN(N)                                                                                \
    (c.dh == 64 ? run<64, N, P>(c, qi, out, heads, n, lens, lens_add, scale, rope, st)            \
                : run<128, N, P>(c, qi, out, heads, n, lens, lens_add, scale, rope, st))
    const int64_t cols = nq * P;
    return cols <= 16 ? RLT_RUN(16) : cols <= 32 ? RLT_RUN(32) : RLT_RUN(64);
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
