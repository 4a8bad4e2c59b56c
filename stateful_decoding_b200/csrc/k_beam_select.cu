// Beam search's selection (include/rlt.h: rlt_beam_select): of all
// continuations c(b, v) = score_b + log softmax(x_b / T)_v of a group's beams,
// the k largest.
//
// Within a beam the order of c is the order of x, so a beam's own k best
// logits (and its log-sum) are all that the group has to compare.  The work is
// one read of the logits, bound by HBM: a unit is one beam, or a slice of one
// where a group has fewer than 8 beams, and a cluster of up to 8 CTAs holds a
// group's units.
//
//   scan    each thread reads 16-byte chunks tid, tid + 512, ... of its unit
//           and keeps the largest logit it saw, and sum 2^((x - m) log2(e)/T)
//           against its own running maximum m (rescaled when m rises).
//   cut     the k-th largest of the threads' maxima bounds the k-th best logit
//           from below: the k best of the unit lie among the few threads whose
//           maximum reaches it.  Those threads' chunks alone are read again
//           (from L2) and their logits >= the cut collected: about k of them,
//           ranked by counting.  When ties leave more than the buffer holds,
//           the k best are drawn one by one by scanning the unit k times.
//   join    the units' sorted lists meet in the cluster's first CTA; one warp
//           merges them with c in fp64.
//
// The exponent (x - m) log2(e)/T takes log2(e)/T in two parts and threads' sums
// are added in fp64: the error of the log-sum is that of single exponentials
// averaged over the vocabulary (about 1e-8), so beams compare as in exact
// arithmetic down to that distance.
#include <cooperative_groups.h>
#include <math.h>

#include <algorithm>

#include "beam.cuh"

namespace cg = cooperative_groups;

namespace rlt {
namespace {

constexpr int NT = 512, NW = NT / 32;
constexpr int kCand = 1024;             // candidates a unit may collect
constexpr int kMaxUnits = 8;            // units of one CTA: beams <= 64 over 8 CTAs
constexpr int kSliceMin = 4096;         // logits of a slice at least

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// order-preserving key of a float (no NaN)
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t u = __float_as_uint(x);
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

template <typename T> struct Chunk;
template <> struct Chunk<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void load(const float* p, float (&x)[4]) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(p));
        x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
    }
};
template <> struct Chunk<bf16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void load(const bf16* p, float (&x)[8]) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};

// The logits [lo, hi) of one row as 16-byte chunks on 16-byte boundaries; the
// first and last may be partial, and are then read element by element.
template <typename T>
struct Span {
    static constexpr int N = Chunk<T>::N;
    const T* row;           // element 0 of the row
    int lo, hi, first;      // first: element index of chunk 0's start (<= lo)
    int chunks;
    __device__ Span(const T* r, int lo_, int hi_) : row(r), lo(lo_), hi(hi_) {
        const uintptr_t a = reinterpret_cast<uintptr_t>(r + lo);
        first = lo - (int)((a & 15) / sizeof(T));
        chunks = hi > lo ? (hi - first + N - 1) / N : 0;
    }
    // chunk ci; elements outside [lo, hi) and NaN come out as -inf
    __device__ __forceinline__ void load(int ci, float (&x)[N]) const {
        const int e0 = first + ci * N;
        if (e0 >= lo && e0 + N <= hi) {
            Chunk<T>::load(row + e0, x);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                x[i] = -INFINITY;
                if (e0 + i >= lo && e0 + i < hi) x[i] = to_f(row[e0 + i]);
            }
        }
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = fmaxf(x[i], -INFINITY);   // NaN: -inf
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
__global__ void __launch_bounds__(NT, 2)
k_beam_select(const T* __restrict__ logits, const float* __restrict__ scores,
              const uint8_t* __restrict__ finished, int eos, float temperature, int beams,
              int vocab, int slices, int k, int32_t* __restrict__ parents,
              int32_t* __restrict__ tokens, float* __restrict__ new_scores,
              uint8_t* __restrict__ new_finished) {
    constexpr int N = Chunk<T>::N;
    extern __shared__ __align__(16) uint8_t dyn[];      // candidates, then the join's lists
    __shared__ Entry s_list[kMaxUnits][kMaxBeams];
    __shared__ Unit s_unit[kMaxUnits];
    __shared__ float s_best[NT];
    __shared__ int s_pick[NT];
    __shared__ double s_sum[NW];
    __shared__ float s_m[NW];
    __shared__ int s_at[NW];
    __shared__ int s_n, s_picks;
    pdl_enter();
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int group = (int)(blockIdx.x / (unsigned)C);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int units = beams * slices;
    if (rank >= units) return;                          // never rank 0
    Entry* cand = reinterpret_cast<Entry*>(dyn);

    const double c64 = 1.4426950408889634 / (double)temperature;
    const float c_hi = (float)c64, c_lo = (float)(c64 - (double)c_hi);
    auto e2 = [&](float d) {                            // (the bound keeps 0 x inf out)
        d = fmaxf(d, -1e16f);
        return ex2(fmaf(d, c_hi, d * c_lo));
    };

    int mine = 0;
    for (int u = rank; u < units; u += C, ++mine) {
        const int b = u / slices, sl = u % slices;
        const float score = __ldg(scores + (size_t)group * beams + b);
        const bool fin = finished && __ldg(finished + (size_t)group * beams + b);
        const bool sane = fabsf(score) < INFINITY;
        if (fin || !sane) {                             // nothing to read
            if (tid == 0) {
                s_unit[mine] = {0.f, fin && sl == 0 && sane ? 1 : 0, 1.0};
                s_list[mine][0] = {0.f, eos};
            }
            continue;
        }
        const int len = (vocab + slices - 1) / slices;
        const Span<T> span(logits + ((size_t)group * beams + b) * vocab, min(vocab, sl * len),
                           min(vocab, (sl + 1) * len));
        // ------------------------------------------------------------ scan
        float m = -INFINITY, s = 0.f;
        auto take = [&](const float (&x)[N]) {
            float cm = x[0];
#pragma unroll
            for (int i = 1; i < N; ++i) cm = fmaxf(cm, x[i]);
            if (cm > m) {
                s *= e2(m - cm);                        // m = -inf: 0 x 0
                m = cm;
            }
            if (m > -INFINITY) {
                float t = 0.f;
#pragma unroll
                for (int i = 0; i < N; ++i) t += e2(x[i] - m);
                s += t;
            }
        };
        int ci = tid;
        for (; ci + 3 * NT < span.chunks; ci += 4 * NT) {   // four loads in flight
            float x[4][N];
#pragma unroll
            for (int q = 0; q < 4; ++q) span.load(ci + q * NT, x[q]);
#pragma unroll
            for (int q = 0; q < 4; ++q) take(x[q]);
        }
        for (; ci < span.chunks; ci += NT) {
            float x[N];
            span.load(ci, x);
            take(x);
        }
        // ------------------------------------------------------------ the unit's maximum and sum
        const float wm = warp_max(m);
        if (lane == 0) s_m[warp] = wm;
        if (tid == 0) s_n = 0, s_picks = 0;
        __syncthreads();
        float M = s_m[0];
#pragma unroll
        for (int i = 1; i < NW; ++i) M = fmaxf(M, s_m[i]);
        double ds = m > -INFINITY ? (double)(s * e2(m - M)) : 0.0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ds += __shfl_xor_sync(0xffffffffu, ds, o);
        if (lane == 0) s_sum[warp] = ds;
        const bool dead = !(M > -INFINITY) || M == INFINITY;
        // ------------------------------------------------------------ cut
        // the k-th largest of the threads' maxima, found bit by bit on their keys
        const uint32_t key = key_of(m);
        uint32_t cut = 0;
        if (!dead)
            for (int bit = 31; bit >= 0; --bit) {
                const uint32_t at = cut | (1u << bit);
                if (__syncthreads_count(key >= at) >= k) cut = at;
            }
        __syncthreads();                                // s_sum is there too
        if (tid == 0) {
            double sum = 0.0;
            for (int i = 0; i < NW; ++i) sum += s_sum[i];
            s_unit[mine] = {M, 0, sum};
        }
        if (dead) {
            __syncthreads();
            continue;
        }
        if (key >= cut && m > -INFINITY) s_pick[atomicAdd(&s_picks, 1)] = tid;
        __syncthreads();
        const int picks = s_picks;
        for (int p = warp; p < picks; p += NW) {
            const int who = s_pick[p];
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
                if (place < k) s_list[mine][place] = me;
            }
            if (tid == 0) s_unit[mine].count = min(n, k);
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
                if (tid == 0) s_list[mine][i] = {bx, bv};
                px = bx, pv = bv;
            }
            if (tid == 0) s_unit[mine].count = k;       // n > kCand >= k: all are finite
        }
        __syncthreads();
    }
    __syncthreads();
    if (min(C, units) > 1) cluster.sync();              // (ranks without a unit have exited)
    if (rank == 0) {
        // ------------------------------------------------------------ join
        Entry* all = reinterpret_cast<Entry*>(dyn);     // [units][k]
        __shared__ Unit s_all[kMaxBeams];
        for (int u = tid; u < units; u += NT) s_all[u] = *cluster.map_shared_rank(&s_unit[u / C], u % C);
        __syncthreads();
        for (int i = tid; i < units * k; i += NT) {
            const int u = i / k, j = i % k;
            if (j < s_all[u].count) all[i] = *cluster.map_shared_rank(&s_list[u / C][j], u % C);
        }
        __syncthreads();
        if (warp == 0) {
            // lane l merges lists l and l + 32
            double base[2] = {0.0, 0.0}, head[2];       // c = base + (x - M) / T
            double top[2] = {0.0, 0.0};
            int at[2] = {0, 0}, flat[2];
            bool fin[2] = {false, false};
            auto load = [&](int q) {
                const int u = lane + 32 * q;
                head[q] = -INFINITY;
                flat[q] = 0x7fffffff;
                if (u < units && at[q] < s_all[u].count) {
                    const Entry e = all[u * k + at[q]];
                    head[q] = base[q] + (fin[q] ? 0.0 : ((double)e.x - top[q]) / (double)temperature);
                    flat[q] = (u / slices) * vocab + e.v;
                }
            };
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int u = lane + 32 * q;
                if (u < units) {
                    const int b = u / slices;
                    base[q] = (double)__ldg(scores + (size_t)group * beams + b);
                    fin[q] = finished && __ldg(finished + (size_t)group * beams + b);
                    if (!fin[q]) {
                        float M = -INFINITY;
                        for (int i = 0; i < slices; ++i) M = fmaxf(M, s_all[b * slices + i].m);
                        double sum = 0.0;
                        for (int i = 0; i < slices; ++i) {
                            const Unit& w = s_all[b * slices + i];
                            if (w.m > -INFINITY)
                                sum += w.sum * exp(((double)w.m - (double)M) / (double)temperature);
                        }
                        top[q] = (double)M;
                        base[q] -= log(sum);
                        // +inf logits, or none above -inf: no candidate of this beam
                        if (!(fabsf(M) < INFINITY)) at[q] = k;
                    }
                }
                load(q);
            }
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
                if (lane == 0) {
                    const size_t to = (size_t)group * k + i;
                    const int b = none ? 0 : bf / vocab, v = none ? 0 : bf % vocab;
                    parents[to] = b;
                    tokens[to] = v;
                    new_scores[to] = none ? -INFINITY : (float)best;
                    if (new_finished)
                        new_finished[to] =
                            !none && ((finished && finished[(size_t)group * beams + b]) || v == eos);
                }
                if (!none && own == bf) {               // one lane alone holds that candidate
                    ++at[q];
                    load(q);
                }
            }
        }
    }
    if (min(C, units) > 1) cluster.sync();              // no CTA leaves while its lists are read
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
    int C = 1;
    while (C < 8 && C < units) C *= 2;
    const int64_t ctas = (int64_t)groups * C;
    if (ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
    auto* kern = k_beam_select<T>;
    const size_t smem = sizeof(Entry) * (size_t)std::max(kCand, units * k);
    const void* kp = reinterpret_cast<const void*>(kern);
    if (!set_smem_once(kp, sizeof(Entry) * kMaxBeams * kMaxBeams))
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
