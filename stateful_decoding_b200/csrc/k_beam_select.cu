// Beam search's selection (include/rlt.h: rlt_beam_select): of all
// continuations c(b, v) = score_b + log softmax(x_b / T)_v of a group's beams,
// the k largest.
//
// Within a beam the order of c is the order of x, so a beam's own k best
// logits (and its log-sum) are all that the group has to compare.  The work is
// one read of the logits, bound by HBM for batches of searches: a unit is one
// beam, or a slice of one where a group has fewer than 8 beams, and a cluster
// of up to 8 CTAs (16 for a few searches) holds a group's units.
//
//   scan    each of 256 threads reads 16-byte chunks tid, tid + 256, ... of its
//           unit, four in flight while four are worked on, and keeps the
//           largest logit it saw, and sum 2^((x - m) log2(e)/T) against its own
//           running maximum m (rescaled when m rises, four chunks at a time).
//   cut     the k-th largest of the maxima of 64 groups of four threads
//           bounds the k-th best logit from below: the k best of the unit lie
//           among the threads whose maximum reaches it.  Those threads' chunks
//           alone are read again (from L2) and their logits >= the cut
//           collected and ranked by counting: about k of them for small k; for k
//           near 64 the cut is the least of the groups' maxima, and the buffer's
//           1024 places may not do.  Then, as with ties, the k best are drawn one
//           by one by scanning the unit k times.
//   join    the units write their sorted lists into the first CTA's shared
//           memory and leave; it forms c in fp64 and ranks the candidates, by
//           counting up to 256 of them, else by one warp's merge.
//
// 128 searches x 5 beams x 100003 bf16 (128 MB, floor 20 us) take 49.5 us: 640 CTAs of 256
// threads, four to an SM, in clusters of 5 do not all run at once (592 places, fewer for clusters),
// so the last searches run alone; and a CTA's serial part (cut, second read, join) is long beside a
// scan of 13 steps.
//
// The exponent (x - m) log2(e)/T takes log2(e)/T in two parts and threads' sums
// are added in fp64: the error of the log-sum is that of single exponentials
// averaged over the vocabulary (about 1e-8), so beams compare as in exact
// arithmetic down to that distance.
#include <cooperative_groups.h>
#include <float.h>
#include <math.h>

#include <algorithm>

#include "beam.cuh"

namespace cg = cooperative_groups;

namespace rlt {
namespace {

constexpr int NT = 256, NW = NT / 32;
constexpr int NB = 4;                   // chunks per step of a thread
constexpr int kCand = 1024;             // candidates a unit may collect
constexpr int kSliceMin = 4096;         // logits of a slice at least
constexpr int kMostUnits = kMaxBeams;   // of a group

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// order-preserving key of a float (no NaN; the zeros, which compare equal, have one), and back
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float float_of(uint32_t key) {
    return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xffffffffu));
}

// two fp32 values in one register pair: one instruction for both
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(lo), "f"(hi));
    return p;
}
__device__ __forceinline__ float2 unpair(uint64_t p) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(p));
    return f;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
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

// 16 bytes of logits; clean: NaN becomes -inf; top: the largest; get: elements 2i, 2i + 1
template <typename T> struct Chunk;
template <> struct Chunk<float> {
    static constexpr int N = 4;
    static constexpr uint32_t kNone = 0xff800000u;      // -inf in every element
    static __device__ __forceinline__ void clean(uint4& v) {
        uint32_t* w = &v.x;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(fmaxf(__uint_as_float(w[i]), -INFINITY));
    }
    static __device__ __forceinline__ float top(const uint4& v) {
        return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)),
                     fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
    }
    static __device__ __forceinline__ float2 get(const uint4& v, int i) {
        return i ? make_float2(__uint_as_float(v.z), __uint_as_float(v.w))
                 : make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
    }
};
template <> struct Chunk<bf16> {
    static constexpr int N = 8;
    static constexpr uint32_t kNone = 0xff80ff80u;
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
        uint32_t d;
        asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        return d;
    }
    static __device__ __forceinline__ void clean(uint4& v) {
        v.x = max2(v.x, kNone);
        v.y = max2(v.y, kNone);
        v.z = max2(v.z, kNone);
        v.w = max2(v.w, kNone);
    }
    static __device__ __forceinline__ float top(const uint4& v) {
        const uint32_t m = max2(max2(v.x, v.y), max2(v.z, v.w));
        return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
    }
    static __device__ __forceinline__ float2 get(const uint4& v, int i) {
        const uint32_t w = i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
};

// The logits [lo, hi) of one row as 16-byte chunks on 16-byte boundaries; the
// first and last may be partial, and are then read element by element.
template <typename T>
struct Span {
    static constexpr int N = Chunk<T>::N;
    const T* row;           // element 0 of the row
    int lo, hi, first;      // first: element index of chunk 0's start (<= lo)
    int chunks, whole0, whole1;     // chunks [whole0, whole1) are whole
    __device__ Span(const T* r, int lo_, int hi_) : row(r), lo(lo_), hi(hi_) {
        const uintptr_t a = reinterpret_cast<uintptr_t>(r + lo);
        first = lo - (int)((a & 15) / sizeof(T));
        chunks = hi > lo ? (hi - first + N - 1) / N : 0;
        whole0 = first < lo ? 1 : 0;
        whole1 = chunks - (first + chunks * N > hi ? 1 : 0);
    }
    // chunk ci where whole, else nothing but -inf
    __device__ __forceinline__ uint4 fetch(int ci) const {
        constexpr uint32_t z = Chunk<T>::kNone;
        uint4 v = make_uint4(z, z, z, z);
        if (ci >= whole0 && ci < whole1)
            v = __ldg(reinterpret_cast<const uint4*>(row + first + (int64_t)ci * N));
        return v;
    }
    // any chunk; elements outside [lo, hi) and NaN come out as -inf
    __device__ __forceinline__ void load(int ci, float (&x)[N]) const {
        if (ci >= whole0 && ci < whole1) {
            uint4 v = fetch(ci);
            Chunk<T>::clean(v);
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                const float2 f = Chunk<T>::get(v, i);
                x[2 * i] = f.x, x[2 * i + 1] = f.y;
            }
        } else {
            const int e0 = first + ci * N;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                x[i] = -INFINITY;
                if (e0 + i >= lo && e0 + i < hi) x[i] = fmaxf(to_f(row[e0 + i]), -INFINITY);
            }
        }
    }
};

struct Entry {
    float x;
    int v;
};
__device__ __forceinline__ bool before(float x, int v, float y, int w) {
    return x > y || (x == y && v < w);
}

struct Unit {
    float m;                // largest logit (of the slice)
    int count;              // entries of its list
    double sum;             // sum of 2^((x - m) log2(e)/T)
};

template <typename T>
__global__ void __launch_bounds__(NT, 4)
k_beam_select(const T* __restrict__ logits, const float* __restrict__ scores,
              const uint8_t* __restrict__ finished, int eos, float temperature, int beams,
              int vocab, int slices, int k, int32_t* __restrict__ parents,
              int32_t* __restrict__ tokens, float* __restrict__ new_scores,
              uint8_t* __restrict__ new_finished) {
    constexpr int N = Chunk<T>::N, GROUPS = NT / 4;
    extern __shared__ __align__(16) uint8_t dyn[];      // candidates; in rank 0 the units' lists
    __shared__ Unit s_unit[kMostUnits];                 // rank 0: every unit's
    __shared__ uint32_t s_key[GROUPS];
    __shared__ float s_best[NW];
    __shared__ double s_sum[NW];
    __shared__ float s_m[NW];
    __shared__ int s_at[NW];
    __shared__ int s_n;
    __shared__ uint32_t s_cut;
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    pdl_enter();
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int group = (int)(blockIdx.x / (unsigned)C);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int units = beams * slices;                   // C <= units
    Entry* cand = reinterpret_cast<Entry*>(dyn);
    Entry* all = cand + kCand;                          // rank 0: [units][k]
    Unit* to_unit = cluster.map_shared_rank(s_unit, 0);
    Entry* to_list = cluster.map_shared_rank(all, 0);

    const double c64 = 1.4426950408889634 / (double)temperature;
    // both parts positive, so that -inf x either stays -inf
    const float c_hi = __double2float_rd(c64), c_lo = fmaxf((float)(c64 - (double)c_hi), FLT_MIN);
    auto e2 = [&](float d) { return ex2(fmaf(d, c_hi, d * c_lo)); };
    const uint64_t hi2 = pair(c_hi, c_hi), lo2 = pair(c_lo, c_lo);
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");    // every CTA runs: rank 0 takes writes

    for (int u = rank; u < units; u += C) {
        const int b = u / slices, sl = u % slices;
        const float score = __ldg(scores + (size_t)group * beams + b);
        const bool fin = finished && __ldg(finished + (size_t)group * beams + b);
        const bool sane = fabsf(score) < INFINITY;
        if (fin || !sane) {                             // nothing to read
            if (tid == 0) {
                to_unit[u] = {0.f, fin && sl == 0 && sane ? 1 : 0, 1.0};
                to_list[u * k] = {0.f, eos};
            }
            continue;
        }
        const int len = (vocab + slices - 1) / slices;
        const Span<T> span(logits + ((size_t)group * beams + b) * vocab, min(vocab, sl * len),
                           min(vocab, (sl + 1) * len));
        // ------------------------------------------------------------ scan
        float m = -INFINITY;
        uint64_t s2 = pair(0.f, 0.f);
        auto rise = [&](float top) {
            if (top > m) {
                const float f = m > -INFINITY ? e2(m - top) : 0.f;
                s2 = mul2(s2, pair(f, f));
                m = top;
            }
        };
        const int steps = (span.chunks + NB * NT - 1) / (NB * NT);
        uint4 next[NB];
#pragma unroll
        for (int q = 0; q < NB; ++q) next[q] = span.fetch(tid + q * NT);
        for (int i = 0; i < steps; ++i) {
            uint4 v[NB];
#pragma unroll
            for (int q = 0; q < NB; ++q) {
                v[q] = next[q];
                next[q] = span.fetch(tid + ((i + 1) * NB + q) * NT);
            }
            float top = -INFINITY;
#pragma unroll
            for (int q = 0; q < NB; ++q) {
                Chunk<T>::clean(v[q]);
                top = fmaxf(top, Chunk<T>::top(v[q]));
            }
            rise(top);
            if (m > -INFINITY) {
                const uint64_t m2 = pair(-m, -m);
                uint64_t t2 = pair(0.f, 0.f);
#pragma unroll
                for (int q = 0; q < NB; ++q)
#pragma unroll
                    for (int x = 0; x < N / 2; ++x) {
                        const float2 f = Chunk<T>::get(v[q], x);
                        const uint64_t d = add2(pair(f.x, f.y), m2);
                        const float2 e = unpair(fma2(d, hi2, mul2(d, lo2)));
                        t2 = add2(t2, pair(ex2(e.x), ex2(e.y)));
                    }
                s2 = add2(s2, t2);
            }
        }
        const float2 halves = unpair(s2);
        float s = halves.x + halves.y;
        for (int end = 0; end < 2; ++end) {             // the partial chunks at the ends
            const int ci = end ? span.whole1 : 0;
            const bool part = end ? ci < span.chunks && !(ci == 0 && span.whole0) : span.whole0 == 1;
            if (part && span.chunks > 0 && ci % NT == tid) {
                float x[N];
                span.load(ci, x);
                for (int q = 0; q < N; ++q) {
                    if (x[q] > m) {
                        s = m > -INFINITY ? s * e2(m - x[q]) : 0.f;
                        m = x[q];
                    }
                    if (m > -INFINITY) s += e2(x[q] - m);
                }
            }
        }
        // ------------------------------------------------------------ the warps' maxima and sums
        const uint32_t key = key_of(m);
        const float wm = float_of(__reduce_max_sync(0xffffffffu, key));
        double ds = m > -INFINITY ? (double)(s * e2(m - wm)) : 0.0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ds += __shfl_xor_sync(0xffffffffu, ds, o);
        if (lane == 0) s_m[warp] = wm, s_sum[warp] = ds;
        uint32_t gk = max(key, __shfl_xor_sync(0xffffffffu, key, 1));
        gk = max(gk, __shfl_xor_sync(0xffffffffu, gk, 2));
        if ((lane & 3) == 0) s_key[tid >> 2] = gk;
        if (tid == 0) s_n = 0;
        __syncthreads();
        // ------------------------------------------------------------ cut
        if (warp == 0) {                                // the k-th largest of the groups' maxima
            uint32_t mine[GROUPS / 32], cut = 0;
#pragma unroll
            for (int i = 0; i < GROUPS / 32; ++i) mine[i] = s_key[lane + 32 * i];
            for (int i = 0; i < k; ++i) {
                uint32_t best = mine[0];
#pragma unroll
                for (int j = 1; j < GROUPS / 32; ++j) best = max(best, mine[j]);
                cut = __reduce_max_sync(0xffffffffu, best);
                const uint32_t who = __ballot_sync(0xffffffffu, best == cut);
                if (lane == __ffs(who) - 1) {           // one of them is taken
                    bool gone = false;
#pragma unroll
                    for (int j = 0; j < GROUPS / 32; ++j)
                        if (!gone && mine[j] == cut) mine[j] = 0, gone = true;
                }
            }
            if (lane == 0) s_cut = cut;
        } else if (warp == 1) {
            const float pm = lane < NW ? s_m[lane] : -INFINITY;
            const float M = float_of(__reduce_max_sync(0xffffffffu, key_of(pm)));
            double sum = lane < NW && pm > -INFINITY ? s_sum[lane] * (double)e2(pm - M) : 0.0;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (lane == 0) to_unit[u].m = M, to_unit[u].sum = sum;
        }
        __syncthreads();
        const uint32_t cut = s_cut;
        for (uint32_t left = __ballot_sync(0xffffffffu, key >= cut && m > -INFINITY); left;
             left &= left - 1) {
            const int who = warp * 32 + __ffs(left) - 1;
            for (int c0 = who + lane * NT; c0 < span.chunks; c0 += 32 * NT) {
                float x[N];
                span.load(c0, x);
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (x[i] > -INFINITY && key_of(x[i]) >= cut) {
                        const int at = atomicAdd(&s_n, 1);
                        if (at < kCand) cand[at] = {x[i], span.first + c0 * N + i};
                    }
            }
        }
        __syncthreads();
        const int n = s_n;
        if (n <= kCand) {
            for (int i = tid; i < n; i += NT) {
                const Entry me = cand[i];
                int place = 0;
                for (int j = 0; j < n; ++j) place += before(cand[j].x, cand[j].v, me.x, me.v);
                if (place < k) to_list[u * k + place] = me;
            }
            if (tid == 0) to_unit[u].count = min(n, k);
        } else {
            // more ties at the cut than the buffer holds: one by one
            float px = INFINITY;
            int pv = -1;
            for (int i = 0; i < k; ++i) {
                float bx = -INFINITY;
                int bv = 0x7fffffff;
                for (int c0 = tid; c0 < span.chunks; c0 += NT) {
                    float x[N];
                    span.load(c0, x);
#pragma unroll
                    for (int q = 0; q < N; ++q) {
                        const int v = span.first + c0 * N + q;
                        if (before(px, pv, x[q], v) && before(x[q], v, bx, bv)) bx = x[q], bv = v;
                    }
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    const float ox = __shfl_xor_sync(0xffffffffu, bx, o);
                    const int ov = __shfl_xor_sync(0xffffffffu, bv, o);
                    if (before(ox, ov, bx, bv)) bx = ox, bv = ov;
                }
                __syncthreads();                        // the last round's winners are read
                if (lane == 0) s_best[warp] = bx, s_at[warp] = bv;
                __syncthreads();
                bx = s_best[0], bv = s_at[0];
                for (int w = 1; w < NW; ++w)
                    if (before(s_best[w], s_at[w], bx, bv)) bx = s_best[w], bv = s_at[w];
                if (tid == 0) to_list[u * k + i] = {bx, bv};
                px = bx, pv = bv;
            }
            if (tid == 0) to_unit[u].count = k;         // n > kCand >= k: all are finite
        }
        __syncthreads();                                // cand, s_key, s_n serve the next unit
    }
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    if (rank) return;                                   // their lists are in rank 0
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    // ------------------------------------------------------------ join
    __shared__ double s_base[kMaxBeams], s_top[kMaxBeams];
    __shared__ bool s_open[kMaxBeams], s_fin[kMaxBeams];
    if (tid < beams) {                                  // c = base + (x - top) / T
        const int b = tid;
        double base = (double)__ldg(scores + (size_t)group * beams + b), top = 0.0;
        const bool fin = finished && __ldg(finished + (size_t)group * beams + b);
        bool open = true;
        if (!fin) {
            float M = -INFINITY;
            for (int i = 0; i < slices; ++i) M = fmaxf(M, s_unit[b * slices + i].m);
            double sum = 0.0;
            for (int i = 0; i < slices; ++i) {
                const Unit& w = s_unit[b * slices + i];
                if (w.m > -INFINITY)
                    sum += w.m == M ? w.sum
                                    : w.sum * exp(((double)w.m - (double)M) / (double)temperature);
            }
            top = (double)M;
            base -= log(sum);
            open = fabsf(M) < INFINITY;                 // +inf logits, or none above -inf: closed
        }
        s_base[b] = base, s_top[b] = top, s_open[b] = open, s_fin[b] = fin;
    }
    __syncthreads();
    auto score_of = [&](int u, const Entry& e) {
        const int b = u / slices;
        return s_base[b] + (s_fin[b] ? 0.0 : ((double)e.x - s_top[b]) / (double)temperature);
    };
    auto put = [&](int place, double c, int flat, bool none) {
        const size_t to = (size_t)group * k + place;
        const int b = none ? 0 : flat / vocab, v = none ? 0 : flat % vocab;
        parents[to] = b;
        tokens[to] = v;
        new_scores[to] = none ? -INFINITY : (float)c;
        if (new_finished) new_finished[to] = !none && (s_fin[b] || v == eos);
    };
    const int total = units * k;
    if (total <= NT) {
        __shared__ double s_c[NT];
        __shared__ int s_flat[NT];
        double c = -INFINITY;
        int flat = 0x7fffffff;
        if (tid < total) {
            const int u = tid / k;
            if (s_open[u / slices] && tid % k < s_unit[u].count) {
                const Entry e = all[tid];
                c = score_of(u, e);
                flat = (u / slices) * vocab + e.v;
            }
            s_c[tid] = c;
            s_flat[tid] = flat;
        }
        const int valid = __syncthreads_count(c > -INFINITY);
        if (c > -INFINITY) {
            int place = 0;
            for (int j = 0; j < total; ++j)
                place += s_c[j] > c || (s_c[j] == c && s_flat[j] < flat);
            if (place < k) put(place, c, flat, false);
        }
        if (tid >= valid && tid < k) put(tid, 0.0, 0, true);
        return;
    }
    if (warp == 0) {
        // lane l merges lists l and l + 32
        double head[2];
        int at[2] = {0, 0}, flat[2];
        auto load = [&](int q) {
            const int u = lane + 32 * q;
            head[q] = -INFINITY;
            flat[q] = 0x7fffffff;
            if (u < units && s_open[u / slices] && at[q] < s_unit[u].count) {
                const Entry e = all[u * k + at[q]];
                head[q] = score_of(u, e);
                flat[q] = (u / slices) * vocab + e.v;
            }
        };
        load(0);
        load(1);
        for (int i = 0; i < k; ++i) {
            const int q = head[1] > head[0] || (head[1] == head[0] && flat[1] < flat[0]);
            double best = head[q];
            int bf = flat[q];
            const int own = bf;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const double ob = __shfl_xor_sync(0xffffffffu, best, o);
                const int of = __shfl_xor_sync(0xffffffffu, bf, o);
                if (ob > best || (ob == best && of < bf)) best = ob, bf = of;
            }
            const bool none = !(best > -INFINITY);
            if (lane == 0) put(i, best, bf, none);
            if (!none && own == bf) {                   // one lane alone holds that candidate
                ++at[q];
                load(q);
            }
        }
    }
}

}  // namespace

template <typename T>
cudaError_t launch_beam_select(const T* logits, const float* scores, const uint8_t* finished,
                               int eos, float temperature, int groups, int beams, int vocab,
                               int k, int32_t* parents, int32_t* tokens, float* new_scores,
                               uint8_t* new_finished, cudaStream_t st) {
    if (groups <= 0) return cudaSuccess;
    // slices and CTAs by beams and vocabulary alone: a group's bits do not depend on the batch
    int slices = 1;
    while (slices * 2 * beams <= 8 && vocab / (slices * 2) >= kSliceMin) slices *= 2;
    const int units = beams * slices;
    // CTAs of a group: as few as finish in as many turns as 8 would take (fewer idle at the end);
    // up to 16 where so few searches run that each may spread over more of the machine
    int most = 8;
    auto* kern = k_beam_select<T>;
    const void* kp = reinterpret_cast<const void*>(kern);
    if (units > 8 && groups <= 8 && set_wide_cluster_once(kp)) most = 16;
    const int turns = (units + most - 1) / most, C = (units + turns - 1) / turns;
    const int64_t ctas = (int64_t)groups * C;
    if (ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
    const size_t smem = sizeof(Entry) * (size_t)(kCand + units * k);
    if (!set_smem_once(kp, sizeof(Entry) * (kCand + kMaxBeams * kMaxBeams)))
        return cudaErrorInvalidConfiguration;
    set_carveout_once(kp);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(NT);
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
    cudaError_t e = cudaLaunchKernelEx(&cfg, kern, logits, scores, finished, eos, temperature,
                                       beams, vocab, slices, k, parents, tokens, new_scores,
                                       new_finished);
    if (e == cudaSuccess) rlt_count_launch();
    return e;
}

template cudaError_t launch_beam_select<float>(const float*, const float*, const uint8_t*, int,
                                               float, int, int, int, int, int32_t*, int32_t*,
                                               float*, uint8_t*, cudaStream_t);
template cudaError_t launch_beam_select<bf16>(const bf16*, const float*, const uint8_t*, int,
                                              float, int, int, int, int, int32_t*, int32_t*,
                                              float*, uint8_t*, cudaStream_t);

}  // namespace rlt
