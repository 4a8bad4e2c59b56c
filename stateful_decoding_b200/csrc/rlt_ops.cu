// C ABI of the operators that work on the caller's buffers alone (no model or
// state): the paged 8-bit cache, beam selection, row reordering.  Everything
// is checked here, on the host, before a launch; what only the device can see
// (lengths, table entries, parents) the kernels check.
#include <nvtx3/nvToolsExt.h>

#include <cmath>

#include "../../include/rlt.h"
#include "beam.cuh"
#include "cache8.cuh"

namespace {

struct NvtxRange {
    explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
    NvtxRange(const NvtxRange&) = delete;
    NvtxRange& operator=(const NvtxRange&) = delete;
};

// the device that holds p, or -1 (host memory, or no such address)
int device_of(const void* p) {
    cudaPointerAttributes a;
    if (!p || cudaPointerGetAttributes(&a, p) != cudaSuccess) {
        cudaGetLastError();
        return -1;
    }
    return a.type == cudaMemoryTypeDevice || a.type == cudaMemoryTypeManaged ? a.device : -1;
}

// Makes a device current for the call and puts the caller's back.
struct OnDevice {
    int before = -1;
    bool ok = false;
    explicit OnDevice(int dev) {
        if (cudaGetDevice(&before) != cudaSuccess) {
            cudaGetLastError();
            before = -1;
            return;
        }
        ok = before == dev || cudaSetDevice(dev) == cudaSuccess;
        if (before == dev) before = -1;
        if (!ok) cudaGetLastError();
    }
    ~OnDevice() {
        if (before >= 0) cudaSetDevice(before);
    }
};

int rc_of(cudaError_t e) {
    if (e == cudaSuccess) return RLT_OK;
    cudaGetLastError();
    return e == cudaErrorInvalidConfiguration     ? RLT_E_UNSUPPORTED
           : e == cudaErrorInvalidResourceHandle ? RLT_E_ARG      // a stream of another device
                                                 : RLT_E_DEVICE;
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }
// a pitch in elements whose bytes are a multiple of 16, large enough not to overlap
bool pitch_ok(int64_t pitch, int64_t least, int64_t count, size_t elt) {
    return count <= 1 || (pitch >= least && pitch < ((int64_t)1 << 48) && pitch % (16 / (int64_t)elt) == 0);
}

constexpr int64_t kMostTokens = (int64_t)1 << 30;

// sizes, pointers and alignment of a cache; its device in *dev
int check_cache(const rlt_cache8* c, int* dev) {
    if (!c) return RLT_E_ARG;
    if (c->rows < 0 || c->row_pages < 1 || c->n_pages < 1 || c->kv_heads < 1 || c->page < 1 ||
        c->dh < 1)
        return RLT_E_ARG;
    if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128) return RLT_E_UNSUPPORTED;
    if (c->dh != 64 && c->dh != 128) return RLT_E_UNSUPPORTED;
    if ((int64_t)c->row_pages * c->page > kMostTokens || c->kv_heads > (1 << 20)) return RLT_E_UNSUPPORTED;
    const bool some = c->rows > 0;              // (a table of no rows may have no address)
    if (!c->pages || !c->scales || (some && !c->table) || !aligned16(c->pages) ||
        ((uintptr_t)c->scales & 3) || ((uintptr_t)c->table & 3) || ((uintptr_t)c->status & 3))
        return RLT_E_ARG;
    *dev = device_of(c->pages);
    if (*dev < 0 || device_of(c->scales) != *dev || (some && device_of(c->table) != *dev) ||
        (c->status && device_of(c->status) != *dev))
        return RLT_E_ARG;
    return RLT_OK;
}

int check_rope(const rlt_rope* r, int dh, int dev) {
    if (!r) return RLT_OK;
    if (r->rot < 0 || r->rot > dh || r->rot % 8 || r->positions < 1 || r->origin < -kMostTokens / 2 ||
        r->origin > kMostTokens / 2)
        return RLT_E_ARG;
    if (!r->cos || !r->sin || !aligned16(r->cos) || !aligned16(r->sin) ||
        device_of(r->cos) != dev || device_of(r->sin) != dev)
        return RLT_E_ARG;
    return RLT_OK;
}

rlt::Cache8 cache_of(const rlt_cache8* c) {
    return {(uint8_t*)c->pages, c->scales, c->table, c->status, RLT_E_ARG, RLT_E_CAPACITY, RLT_E_TIMEOUT,
            c->n_pages, c->rows, c->row_pages, c->page, c->kv_heads, c->dh};
}
rlt::Rope8 rope_of(const rlt_rope* r) {
    if (!r) return {nullptr, nullptr, 0, 0, 0, 0};
    return {r->cos, r->sin, r->positions, r->rot, r->interleaved, r->origin};
}

}  // namespace

extern "C" int rlt_cache8_append(const rlt_cache8* cache, int dtype, const void* k, int64_t k_row,
                                 int64_t k_token, const void* v, int64_t v_row, int64_t v_token,
                                 const int32_t* start, const int32_t* counts, int n,
                                 const rlt_rope* rope, void* stream) {
    NvtxRange nvtx("rlt_cache8_append");
    int dev = -1;
    if (int rc = check_cache(cache, &dev)) return rc;
    if (dtype != RLT_DTYPE_F32 && dtype != RLT_DTYPE_BF16) return RLT_E_ARG;
    if (n < 0 || n > kMostTokens) return RLT_E_ARG;
    if (int rc = check_rope(rope, cache->dh, dev)) return rc;
    if (cache->rows == 0 || n == 0) return RLT_OK;
    const size_t elt = dtype == RLT_DTYPE_BF16 ? 2 : 4;
    const int64_t wide = (int64_t)cache->kv_heads * cache->dh;
    if (!aligned16(k) || !aligned16(v) || !pitch_ok(k_token, wide, n, elt) ||
        !pitch_ok(v_token, wide, n, elt) || !pitch_ok(k_row, wide, cache->rows, elt) ||
        !pitch_ok(v_row, wide, cache->rows, elt) || ((uintptr_t)start & 3) ||
        ((uintptr_t)counts & 3))
        return RLT_E_ARG;
    if (device_of(k) != dev || device_of(v) != dev || device_of(start) != dev ||
        (counts && device_of(counts) != dev))
        return RLT_E_ARG;
    OnDevice on(dev);
    if (!on.ok) return RLT_E_DEVICE;
    const cudaStream_t st = (cudaStream_t)stream;
    const rlt::Cache8 c = cache_of(cache);
    const rlt::Rope8 r = rope_of(rope);
    if (dtype == RLT_DTYPE_BF16)
        return rc_of(rlt::launch_cache8_append<rlt::bf16>(
            c, {(const rlt::bf16*)k, k_row, k_token}, {(const rlt::bf16*)v, v_row, v_token}, start,
            counts, n, r, st));
    return rc_of(rlt::launch_cache8_append<float>(c, {(const float*)k, k_row, k_token},
                                                  {(const float*)v, v_row, v_token}, start, counts,
                                                  n, r, st));
}

extern "C" int rlt_cache8_attend(const rlt_cache8* cache, int dtype, const void* q, int64_t q_row,
                                 int64_t q_token, void* out, int64_t out_row, int64_t out_token,
                                 int heads, int n, const int32_t* lens, float scale,
                                 const rlt_rope* rope, void* stream) {
    NvtxRange nvtx("rlt_cache8_attend");
    int dev = -1;
    if (int rc = check_cache(cache, &dev)) return rc;
    if (dtype != RLT_DTYPE_F32 && dtype != RLT_DTYPE_BF16) return RLT_E_ARG;
    if (n < 0 || n > kMostTokens || heads < 1 || heads % cache->kv_heads || !std::isfinite(scale))
        return RLT_E_ARG;
    if ((int64_t)n * (heads / cache->kv_heads) > kMostTokens) return RLT_E_UNSUPPORTED;
    if (int rc = check_rope(rope, cache->dh, dev)) return rc;
    if (cache->rows == 0 || n == 0) return RLT_OK;
    const size_t elt = dtype == RLT_DTYPE_BF16 ? 2 : 4;
    const int64_t wide = (int64_t)heads * cache->dh;
    if (!aligned16(q) || !aligned16(out) || !pitch_ok(q_token, wide, n, elt) ||
        !pitch_ok(out_token, wide, n, elt) || !pitch_ok(q_row, wide, cache->rows, elt) ||
        !pitch_ok(out_row, wide, cache->rows, elt) || ((uintptr_t)lens & 3))
        return RLT_E_ARG;
    if (device_of(q) != dev || device_of(out) != dev || device_of(lens) != dev) return RLT_E_ARG;
    OnDevice on(dev);
    if (!on.ok) return RLT_E_DEVICE;
    const cudaStream_t st = (cudaStream_t)stream;
    const rlt::Cache8 c = cache_of(cache);
    const rlt::Rope8 r = rope_of(rope);
    if (dtype == RLT_DTYPE_BF16)
        return rc_of(rlt::launch_cache8_attend<rlt::bf16, rlt::bf16>(
            c, {(const rlt::bf16*)q, q_row, q_token}, 1, 0, {(rlt::bf16*)out, out_row, out_token},
            heads, n, lens, 0, scale, r, st));
    return rc_of(rlt::launch_cache8_attend<float, float>(c, {(const float*)q, q_row, q_token}, 1, 0,
                                                         {(float*)out, out_row, out_token}, heads,
                                                         n, lens, 0, scale, r, st));
}

extern "C" int rlt_beam_select(int dtype, const void* logits, const float* scores,
                               const uint8_t* finished, int eos, float temperature, int groups,
                               int beams, int vocab, int k, int32_t* parents, int32_t* tokens,
                               float* new_scores, uint8_t* new_finished, void* stream) {
    NvtxRange nvtx("rlt_beam_select");
    if (dtype != RLT_DTYPE_F32 && dtype != RLT_DTYPE_BF16) return RLT_E_ARG;
    if (groups < 0 || beams < 1 || beams > rlt::kMaxBeams || k < 1 || k > rlt::kMaxBeams ||
        vocab < 1 || vocab >= (1 << 24) || (int64_t)k > (int64_t)beams * vocab)
        return RLT_E_ARG;
    if (!(temperature >= 0x1p-20f && temperature <= 0x1p20f)) return RLT_E_ARG;
    if (finished && (eos < 0 || eos >= vocab)) return RLT_E_ARG;
    if (groups == 0) return RLT_OK;
    const size_t elt = dtype == RLT_DTYPE_BF16 ? 2 : 4;
    if ((uintptr_t)logits % elt || ((uintptr_t)scores & 3) || ((uintptr_t)parents & 3) ||
        ((uintptr_t)tokens & 3) || ((uintptr_t)new_scores & 3))
        return RLT_E_ARG;
    const int dev = device_of(logits);
    if (dev < 0 || device_of(scores) != dev || device_of(parents) != dev ||
        device_of(tokens) != dev || device_of(new_scores) != dev ||
        (finished && device_of(finished) != dev) ||
        (new_finished && device_of(new_finished) != dev))
        return RLT_E_ARG;
    OnDevice on(dev);
    if (!on.ok) return RLT_E_DEVICE;
    const cudaStream_t st = (cudaStream_t)stream;
    if (dtype == RLT_DTYPE_BF16)
        return rc_of(rlt::launch_beam_select<rlt::bf16>(
            (const rlt::bf16*)logits, scores, finished, eos, temperature, groups, beams, vocab, k,
            parents, tokens, new_scores, new_finished, st));
    return rc_of(rlt::launch_beam_select<float>((const float*)logits, scores, finished, eos,
                                                temperature, groups, beams, vocab, k, parents,
                                                tokens, new_scores, new_finished, st));
}

extern "C" int rlt_rows_reorder(void* rows, const int32_t* parents, int groups, int beams,
                                int64_t row_stride, int planes, int64_t plane_stride,
                                int64_t offset, int64_t bytes, void* stream) {
    NvtxRange nvtx("rlt_rows_reorder");
    if (groups < 0 || beams < 1 || beams > rlt::kMaxBeams || planes < 0 || offset < 0 || bytes < 0)
        return RLT_E_ARG;
    if (groups == 0 || planes == 0 || bytes == 0) return RLT_OK;
    // rows of planes, or planes of rows: either way no byte belongs to two
    const int64_t n_rows = (int64_t)groups * beams, most = (int64_t)1 << 48;
    if (row_stride < 0 || plane_stride < 0 || row_stride > most || plane_stride > most ||
        bytes > most || offset > most)
        return RLT_E_ARG;
    using i128 = __int128;
    const bool rows_outside = (i128)row_stride >= (i128)(planes - 1) * plane_stride + bytes &&
                              (planes == 1 || plane_stride >= bytes);
    const bool planes_outside = (i128)plane_stride >= (i128)(n_rows - 1) * row_stride + bytes &&
                                row_stride >= bytes;
    if (n_rows > 1 && !rows_outside && !(planes > 1 && planes_outside)) return RLT_E_ARG;
    if ((uintptr_t)parents & 3) return RLT_E_ARG;
    const int dev = device_of(rows);
    if (dev < 0 || device_of(parents) != dev) return RLT_E_ARG;
    OnDevice on(dev);
    if (!on.ok) return RLT_E_DEVICE;
    rlt::ReorderSeg s = {(uint8_t*)rows + offset, row_stride, plane_stride, bytes, nullptr, 0, 1,
                         planes, 1};
    return rc_of(rlt::launch_reorder(&s, 1, parents, groups, beams, (cudaStream_t)stream));
}
