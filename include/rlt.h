/*
 * rlt.h -- C ABI of the RLT transition engine (librlt.so, sm_100a).
 *
 * The Recurrent Looped Transformer carries a full decoder state
 * H_t = (s_t, C^D_t) -- the last decoder output and one sliding-window
 * key/value cache per decoder layer -- across every token, prompt and
 * response alike, and reads a prefix-restricted memory built by a causal
 * encoder (jiphyeonjeon.kr review "Recurrent Looped Transformer", §2-§3;
 * greeksharifa.github.io "Recurrent Looped Transformer 요약 설명", §2.1-§2.7).
 * This library runs that transition for a batch of independent sequences
 * ("rows") on one GPU.
 *
 * Conventions shared by every call
 * --------------------------------
 * - Return value: RLT_OK (0) on success, a negative RLT_E_* code otherwise.
 *   Nothing traps; device-side failures (a bounded wait that gave up) set a
 *   sticky per-state error word that rlt_state_check() reports.
 * - Streams: `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *   stream).  Calls are stream-ordered and asynchronous unless stated.
 * - Ownership: models and states are library-owned and freed by their
 *   destroy call.  Caller buffers (tokens, logits, ids) stay caller-owned; the
 *   library never frees or retains them past the call's stream work.
 * - Host or device pointers: every caller buffer may be host memory (pageable
 *   or pinned) or device memory of the state's device; the library checks with
 *   cudaPointerGetAttributes and stages host buffers through its own device
 *   copies on `stream`.  Host outputs are valid after `stream` synchronises.
 * - Rows are independent: row r's results do not depend on the batch size or
 *   on other rows' tokens, bit for bit (greeksharifa App. C.1, batching
 *   independent sequences).
 * - Positions are 1-based; BOS is position 1 (greeksharifa App. I).
 * - Threads: one model or state must not be used by two host threads at
 *   once; different states may run on different threads and streams.  A
 *   bounded wait that gives up inside the GEMMs or the bulk-copy attention
 *   kernels records it in a device-wide word (other kernels use the state's
 *   own), which the first rlt_state_check on that device to run afterwards
 *   reports and clears.
 */
#ifndef RLT_H
#define RLT_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define RLT_OK             0
#define RLT_E_ARG         -1  /* bad argument (null pointer, size, row index)            */
#define RLT_E_OOM         -2  /* device or host allocation failed                         */
#define RLT_E_CAPACITY    -3  /* a row's position would exceed the state's max_len        */
#define RLT_E_ORDER       -4  /* transition without an encoded token (pos_dec >= pos_enc) */
#define RLT_E_BLOB        -5  /* weight blob: bad magic, version, manifest or checksum    */
#define RLT_E_DEVICE      -6  /* a CUDA call failed (no device, launch error, fault)      */
#define RLT_E_TIMEOUT     -7  /* a bounded device wait gave up                            */
#define RLT_E_UNSUPPORTED -8  /* configuration this build does not run                    */
#define RLT_E_SNAPSHOT    -9  /* snapshot: bad magic, version or size, or other weights   */

#define RLT_DTYPE_F32  0
#define RLT_DTYPE_BF16 1

typedef struct rlt_model rlt_model;  /* weights on one device + config              */
typedef struct rlt_state rlt_state;  /* s, R, C^D rings, C^E, memory, e, positions   */

/* Model hyper-parameters as stored in the blob header. */
typedef struct rlt_config {
    int32_t vocab, d, heads, n_enc, n_dec, ffn, window, groups, chunk, variant, tied, dtype;
    double alpha, eps, rope_base;
} rlt_config;

/* Load a weight blob (host memory, copied; the caller may free it on return)
 * onto `device`.  Blob = 256-byte header (magic "RLTB", version 1, the
 * rlt_config fields, seed, tensor count, payload size, checksum) followed by
 * named tensor records in the fixed manifest order of the config.  Errors:
 * RLT_E_BLOB (bad magic/version/manifest/checksum), RLT_E_UNSUPPORTED (head
 * size other than 16, 32, 64, 128, or width d above 2048), RLT_E_DEVICE,
 * RLT_E_OOM.  Models on several devices may share a process: every call
 * makes its model's device current, and kernel attributes are set per
 * device. */
int rlt_create(const void* blob, size_t nbytes, int device, rlt_model** out);
void rlt_destroy(rlt_model* model);
int rlt_model_config(const rlt_model* model, rlt_config* out);

/* Allocate the per-row state for `batch` rows of up to `max_len` positions:
 * encoder cache C^E [L_E][2][h][max_len][d_h], memory M [G][2][h][max_len][d_h],
 * window rings C^D [L_D][2][h][W-1][d_h] (all in the model dtype), e_t
 * [max_len][d] fp32, s and R [d] fp32 -- the storage bound of the paper's
 * eq. 3.3 (jiphyeonjeon review §4.2) -- plus scratch for one call.  The
 * state starts reset (H_0).  Library-owned.  RLT_E_ARG for batch or max_len
 * <= 0; RLT_E_OOM when an allocation fails, or before allocating when
 * batch x (max_len + W + B_c + 16) x (3d + 2f' + vocab) x 4 x (2(L_E + L_D + G)
 * + 8), f' = f rounded up to 64 -- a bound on every buffer's bytes -- exceeds
 * 2^60. */
int rlt_state_create(rlt_model* model, int batch, int max_len, rlt_state** out);
void rlt_state_destroy(rlt_state* state);

/* rlt_state_create with flags (0: the same).  RLT_STATE_MEM8: the memory M is
 * held in 8 bits, a paged cache as below (pages of 64 positions, one scale per
 * page, head and K or V): about half the bytes of bf16 to hold and to stream
 * through every transition's cross-attention.  Keys and values go to it from
 * the fp32 products, rotated first, rounded once.  Everything else is held as
 * before.  Such a state's results differ from a plain one's by the rounding of
 * M, and in the last bits with how a prompt is split over rlt_encode calls (a
 * page whose scale grows rounds its smallest values again).  RLT_E_UNSUPPORTED
 * for a head size other than 64 and 128; rlt_state_save and rlt_state_load
 * return RLT_E_UNSUPPORTED (a snapshot carries M in the model dtype).
 * RLT_E_ARG for an unknown flag. */
#define RLT_STATE_MEM8 1u
int rlt_state_create_with(rlt_model* model, int batch, int max_len, uint32_t flags,
                          rlt_state** out);

/* Bytes of the per-row state proper (eq. 3.3 terms) and of everything the
 * state allocated on the device (state + scratch). */
int rlt_state_bytes(const rlt_state* state, size_t* per_row_state, size_t* total_device);

/* H_0 = (s_star, empty) for `n` rows listed in host array `rows` (NULL = all
 * rows): s = R = s_star, caches emptied, positions 0 (jiphyeonjeon review §3.1;
 * per-document reset, §6.1). */
int rlt_state_reset(rlt_state* state, const int32_t* rows, int n, void* stream);

/* Encode `n` tokens per row (tokens: int32 [batch][n], host or device) at
 * positions pos_enc+1..pos_enc+n: appends e_t, C^E and the memory entries
 * k^g_t = RoPE_t(W^g_K RMSNorm_E(e_t)), v^g_t = W^g_V RMSNorm_E(e_t)
 * (jiphyeonjeon review §2, eq. 2.1-2.2).  Splitting a prompt over several
 * calls gives the same result as one call (§3.2).  RLT_E_CAPACITY if a row
 * would pass max_len; RLT_E_ARG if a token id is outside [0, vocab) when the
 * tokens are on the host. */
int rlt_encode(rlt_state* state, const int32_t* tokens, int n, void* stream);

/* One transition per row at t = pos_dec+1: u_t = Merge(e_t, s_{t-1})
 * (RLT-2: the register R; RLT-0: u_t = e_t), then L_D decoder blocks
 * (window self-attention over C^D, cross-attention to M_{<=t}, FFN), giving
 * H_t (greeksharifa §2.3-§2.5; jiphyeonjeon review §3).  RLT_E_ORDER if a row
 * has no encoded token at t. */
int rlt_step(rlt_state* state, void* stream);

/* T transitions per row, the recurrent prefill (jiphyeonjeon review §3.2;
 * greeksharifa App. F.1).  RLT-1 runs T sequential steps; RLT-2 runs the
 * positions of each chunk together (ceil(T/B) sequential passes when rows
 * start chunk-aligned, greeksharifa App. I.2); RLT-0 runs blocks of positions
 * together.  Same results as T calls of rlt_step. */
int rlt_prefill(rlt_state* state, int T, void* stream);

/* Readout of every row's current s_t: logits = W_out RMSNorm_out(s_t)
 * (greeksharifa §2.3).  Each output may be NULL.  logits: fp32 [batch][vocab];
 * argmax: int32 [batch], lowest index among equal maxima; sampled: int32
 * [batch], first index i with sum_{j<=i} softmax(logits/temperature)_j > u,
 * u = the SplitMix64 uniform of (rng_seed, row, rng_step):
 *   key = mix64(rng_seed ^ mix64((row+1)*G)), u = top53(mix64(key + (rng_step+1)*G))
 * with G = 0x9E3779B97F4A7C15 and mix64 the SplitMix64 finaliser.  No top-k/p
 * truncation (jiphyeonjeon review §6.2).  temperature > 0.  Each output may
 * be device or host memory; device outputs are written in stream order, host
 * outputs are valid on return (the call then synchronises `stream`). */
int rlt_readout(rlt_state* state, float* logits, int32_t* argmax, int32_t* sampled,
                uint64_t rng_seed, uint64_t rng_step, float temperature, void* stream);

/* Replay: log-probabilities of given tokens under the current weights, each
 * read from the state that precedes it, then the token is consumed
 * (jiphyeonjeon review §6.2, eq. 5.3-5.5: log pi(y|c) = sum_i log p(y_i | c,
 * y_<i); greeksharifa App. D.3, F.4).  tokens: int32 [batch][n], host or
 * device, appended to every row as by rlt_encode; then for j = 0..n-1
 *   logprobs[b][j] = log softmax(logits_b / temperature)[tokens[b][j]],
 * logits_b = W_out RMSNorm_out(s) of row b before token j is consumed (for
 * a reset row and j = 0, the readout of s_star), followed by one transition.
 * temperature = 1 is the model's own distribution; the sampler's temperature
 * gives the distribution rlt_readout samples from (same max and summation,
 * so exp(logprob) is the sampling probability up to rounding).  Afterwards
 * every row has consumed the n tokens: the same state as rlt_encode +
 * rlt_prefill(n).  A replay from the sequence start resets the rows first;
 * the prompt's terms come out beside the response's and the caller keeps the
 * ones it needs.  logprobs: fp32 [batch][n], host or device (host: valid on
 * return; the call then synchronises `stream`).  One readout and one
 * transition per position (no graph replay).  The first call allocates
 * 8 * batch * max_len bytes of scratch in the state.  Errors: RLT_E_ARG (null
 * pointers, n < 0, temperature <= 0, a host token outside [0, vocab)),
 * RLT_E_ORDER (a row has encoded tokens not yet consumed), RLT_E_CAPACITY;
 * a device token outside [0, vocab) gives NaN and RLT_E_ARG from
 * rlt_state_check. */
int rlt_replay_logprobs(rlt_state* state, const int32_t* tokens, int n, float* logprobs,
                        float temperature, void* stream);

/* Packed documents: several independent documents one after another in each
 * row.  tokens: int32 [batch][n], host or device; doc_start: uint8
 * [batch][n], HOST memory, nonzero where a document starts.  Before token j
 * of row b with doc_start[b][j] != 0 the row restarts from H_0 (as
 * rlt_state_reset: s = R = s_star, positions 0, so token j is position 1 of
 * its document): the recurrent output, window rings, encoder cache and
 * positions are per document, and no attention crosses a document start
 * (jiphyeonjeon review §6.1; greeksharifa App. F).  Every token is encoded
 * and consumed (one transition each); a row without a start at column 0
 * continues its current document.  Row b then holds the state of its last
 * document as if that document alone had been encoded and prefilled in a
 * fresh row: bit for bit for RLT-1 and RLT-0; for RLT-2 within the rounding
 * of the two schedules (a lone prefill runs each chunk's positions as one
 * block, the packed run meets chunks cut at document starts).  The columns are cut where any row starts a
 * document, and each piece is one rlt_encode + rlt_prefill for all rows, so
 * rows sit at different positions.  Synchronises `stream` at every cut.
 * Errors, checked before anything runs: RLT_E_ARG (null pointers, n < 0,
 * doc_start in device memory, a host token outside [0, vocab)), RLT_E_ORDER (a row has encoded tokens not
 * yet consumed), RLT_E_CAPACITY (a document would pass max_len); later,
 * RLT_E_DEVICE if a CUDA call fails (the rows then hold the pieces before
 * it). */
int rlt_prefill_packed(rlt_state* state, const int32_t* tokens, const uint8_t* doc_start, int n,
                       void* stream);

/* Readout of caller-supplied state vectors that allocates nothing (no
 * counterpart in the method: a serving convenience for callers that hold a
 * model but no state, and may not allocate device memory).  s_rows: device
 * fp32 [rows][d]; row r is read out exactly as rlt_readout reads out row r of
 * a state whose s_t equals it (same logits, argmax and sampled id for the
 * same rng_seed, rng_step, temperature).  Outputs as in rlt_readout: each may
 * be NULL, device or host memory; host outputs are valid on return (the call
 * then synchronises `stream`, which also ends its use of the scratch).
 * Scratch: a file-scope device array of RLT_READOUT_ROWS_SCRATCH_BYTES (16 MiB)
 * per device.  A call needs rows*d*(2 for bf16, 4 for fp32) bytes, plus
 * rows*vocab*4 when `logits` is not a device pointer, plus rows*8, each rounded
 * up to 256; a call needing more returns RLT_E_ARG and launches nothing (e.g.
 * vocab 32000, d 2048, bf16, host logits: at most 127 rows).  Nothing in the scratch
 * has to start at zero.  The first call on a device looks the array's address
 * up (cudaGetSymbolAddress), which may load the module: make that first call
 * before any stream capture on the device begins.  All calls on one device
 * share the one array: calls in flight at the same time (other streams, other
 * threads) race on it; order them on one stream.
 * RLT_E_ARG also for a null model or s_rows, s_rows not in device memory,
 * rows < 0, temperature <= 0.  rows == 0 does nothing. */
#define RLT_READOUT_ROWS_SCRATCH_BYTES (16u << 20)
int rlt_readout_rows(const rlt_model* model, const float* s_rows, int rows, float* logits,
                     int32_t* argmax, int32_t* sampled, uint64_t rng_seed, uint64_t rng_step,
                     float temperature, void* stream);

/* Host copies of the per-row positions (arrays of `batch` int32; either may
 * be NULL).  pos_enc = tokens encoded, pos_dec = transitions applied. */
int rlt_state_positions(const rlt_state* state, int32_t* pos_enc, int32_t* pos_dec);

/* Copy one state component to `dst` (host or device), `nbytes` exactly its
 * size (query with dst = NULL: *nbytes_out receives the size).  Components:
 * RLT_PART_S / _R: fp32 [batch][d]; _E: fp32 [batch][max_len][d];
 * _MEM: model dtype [batch][G][2][h][max_len][d_h]; _RING: model dtype
 * [batch][L_D][2][h][W-1][d_h]; _ENC: model dtype [batch][L_E][2][h][max_len][d_h].
 * In a RLT_STATE_MEM8 state _MEM is e4m3 [G][batch * P][2][h][64][d_h], P =
 * ceil(max_len / 64), row b's positions 64 j + 1 .. in page b P + j, and
 * _MEM_SCALES fp32 [G][batch * P][2][h] (RLT_E_UNSUPPORTED in other states).
 * Synchronises `stream` when dst is host memory. */
#define RLT_PART_S    0
#define RLT_PART_R    1
#define RLT_PART_E    2
#define RLT_PART_MEM  3
#define RLT_PART_RING 4
#define RLT_PART_ENC  5
#define RLT_PART_MEM_SCALES 6
int rlt_state_read(rlt_state* state, int part, void* dst, size_t nbytes, size_t* nbytes_out,
                   void* stream);

/* Exact prefix snapshot of one row: everything the row needs to continue
 * exactly as if it had never stopped -- the encoder cache C^E and memory M of
 * every encoded position, s_t (and the RLT-2 register R), the window rings
 * C^D, the encoder outputs e_t of positions not yet transitioned, pos_enc,
 * pos_dec, and the identity of the weights and config (jiphyeonjeon review
 * §6.5, multi-turn serving; greeksharifa App. E, App. H).  A row restored
 * into any state of the same model -- another row, batch size, max_len,
 * process -- continues with the same results as the row it was taken from
 * (rows are independent, see above).  New tokens (a tool's output, a user
 * turn) are appended with rlt_encode and consumed with rlt_prefill, as on the
 * original row.  The sampler keeps no state: a sampled continuation repeats
 * with the same rng_seed and rng_step.
 *
 * Snapshot bytes (little-endian), independent of batch and max_len:
 *   [0,4) "RLTS"  [4,8) u32 version 1  [8,16) u64 checksum of the weight
 *   blob's payload  [16,20) i32 pos_enc  [20,24) i32 pos_dec  [24,72) the 12
 *   int32 fields of rlt_config in declaration order  [72,96) alpha, eps,
 *   rope_base as f64  [96,128) zero;
 *   then, with P = pos_enc, h heads, d_h = d/h, G' = G if L_D > 0 else 0:
 *   s fp32 [d]; R fp32 [d]; e fp32 [P][d]; C^E [L_E][2][h][P][d_h] and
 *   M [G'][2][h][P][d_h] in the model dtype; C^D [L_D][2][h][W-1][d_h] in
 *   the model dtype (ring slot of position t: (t-1) mod (W-1)).
 * Size = 128 + 8d + 4Pd + (2 h L_E + 2 h G') P d_h e + 2 h L_D (W-1) d_h e,
 * e = 2 (bf16) or 4 (fp32).
 *
 * rlt_state_save: writes row `row`'s snapshot to `dst` (host or device),
 * `nbytes` exactly its size (query with dst = NULL: *nbytes_out receives it).
 * Ordered after the work already queued on `stream`; synchronises `stream`.
 * RLT_E_ARG for a null state, a row outside [0, batch) or a wrong nbytes.
 *
 * rlt_state_load: replaces row `row` with the snapshot at `src` (host or
 * device, `nbytes` its size); other rows are untouched.  Synchronises
 * `stream`; `src` may be freed on return.  Errors, checked before anything is
 * written: RLT_E_ARG (null state or src, bad row), RLT_E_SNAPSHOT (bad magic,
 * version or reserved bytes, nbytes not the size the header implies, or a
 * checksum or config other than the state's model), RLT_E_CAPACITY (pos_enc
 * above the state's max_len).  RLT_E_DEVICE if a copy fails: the row's
 * contents are then undefined until it is reset or loaded again.
 *
 * rlt_snapshot_info: checks a snapshot in HOST memory without a device and
 * returns its config and positions (each output may be NULL); errors as
 * rlt_state_load's format checks (RLT_E_ARG for a null snapshot). */
#define RLT_SNAPSHOT_HEADER_BYTES 128
int rlt_state_save(rlt_state* state, int row, void* dst, size_t nbytes, size_t* nbytes_out,
                   void* stream);
int rlt_state_load(rlt_state* state, int row, const void* src, size_t nbytes, void* stream);
int rlt_snapshot_info(const void* snap, size_t nbytes, rlt_config* cfg, int32_t* pos_enc,
                      int32_t* pos_dec);

/* Synchronise `stream` and report the state's sticky device error word
 * (RLT_OK, RLT_E_TIMEOUT, ...), clearing it. */
int rlt_state_check(rlt_state* state, void* stream);

/* Failure-detection self-test (no counterpart in the method).  Enqueues on
 * `stream` one small kernel whose single wait nothing will ever satisfy --
 * kind 0: an mbarrier in shared memory that no thread arrives on; kind 1: a
 * word in global memory that no thread sets -- bounded by `polls` polls
 * through the same helpers as the library's own waits.  When the wait gives
 * up the kernel records a timeout in the state's error word and returns, so
 * the next rlt_state_check reports RLT_E_TIMEOUT (and clears it) and the
 * context stays usable; the state's contents are not touched.  No copy is in
 * flight and no tensor memory is held when it gives up.  A poll of kind 0
 * lasts as long as the hardware's try-wait suspends (a system-dependent
 * limit); a poll of kind 1 sleeps about 256 ns.  RLT_E_ARG for a null state,
 * another kind, or polls outside [1, 2^24]. */
int rlt_selftest_wait(rlt_state* state, int kind, uint32_t polls, void* stream);

/* Build flags of the loaded library.  RLT_BUILD_DEBUG: built with RLT_DEBUG=1
 * (librlt_debug.so): the kernels validate every row's position counters
 * before each encoder and transition block (0 <= pos_dec, pos_dec + n <=
 * pos_enc <= max_len; pos_enc + n <= max_len when encoding), check ring
 * slots and key indices where the decode attention forms them, and token
 * ids as every build does; a violation is recorded in the state's error
 * word -- rlt_state_check then returns RLT_E_ORDER, RLT_E_CAPACITY or
 * RLT_E_ARG -- and the access it guards is skipped.  Nothing traps. */
#define RLT_BUILD_DEBUG 1u
uint32_t rlt_build_flags(void);

/* Debug builds only: overwrite the DEVICE position counters of one row,
 * leaving the host's copy unchanged -- a stand-in for a corrupted or stale
 * device state, for testing the checks above.  Synchronises `stream`.
 * Returns RLT_E_UNSUPPORTED in other builds; RLT_E_ARG for a null state or a
 * row outside [0, batch).  A counter past max_len makes the next encode write
 * past the row's buffers: only a transition or a readout may follow. */
int rlt_debug_set_positions(rlt_state* state, int row, int32_t pos_enc, int32_t pos_dec,
                            void* stream);

/* ---------------------------------------------------------------------------
 * Paged 8-bit key/value cache (no counterpart in the method: serving memory
 * for long prefixes and large batches).
 *
 * Keys and values are e4m3 bytes (1 sign, 4 exponent, 3 mantissa bits; largest
 * 448) in pages of `page` tokens; every (page, head) has one fp32 scale for its
 * keys and one for its values, and a byte x stands for x * scale:
 *   pages  e4m3 [n_pages][2][kv_heads][page][dh]   (index 0: K, 1: V)
 *   scales fp32 [n_pages][2][kv_heads]             (positive and finite)
 *   table  int32 [rows][row_pages]                 token j of row b sits in page
 *          table[b][j / page], slot j % page.
 * All buffers are caller-owned device memory, `pages` aligned to 16 bytes; the
 * struct itself is host memory, read during the call only.  page is 16, 32, 64
 * or 128; dh is 64 or 128; n_pages times the bytes of a page may pass 2^32.
 * status (device int32, may be NULL) is a sticky word the kernels set to the
 * first problem they meet, which they step around: RLT_E_ARG, a table entry
 * outside [0, n_pages) (append: the tokens of that block are not written;
 * attend: its keys are not seen); RLT_E_CAPACITY, a length below 0 or above
 * row_pages * page, or a position without a row in the rotation table (append:
 * those tokens are not written; attend: a length is cut to the capacity, a
 * query without a rotation gives 0); RLT_E_TIMEOUT, a bounded wait inside
 * attend gave up (its output is then undefined).  The caller zeroes it.
 * Table entries of blocks past a row's length are not read.  Pages may be
 * shared between rows for reading; a page that two rows of one append write, or
 * one row twice, is undefined.  Attention is laid out for the table's width, since lengths are
 * on the device: 64 rows of 480 keys, 4 key heads x 8 queries of 128, take 31 us in
 * a table of 512 positions, 66 below 32768 and 195 from there on (one query a
 * key head, 16 of them: 43, 53, and 84 at 131072), so pass one no wider than the
 * rows need.
 *
 * These calls, rlt_beam_select and rlt_rows_reorder take no model or state.
 * They allocate nothing, use no scratch, keep nothing from call to call, read
 * lengths and tables on the device (so a captured call may be replayed with
 * new ones) and return with the calling thread's current device unchanged.
 * They run on the device that holds `pages` (the logits; the rows); every
 * buffer must be on that device and `stream` belong to it, else RLT_E_ARG.
 * RLT_E_ARG also for null or misaligned pointers, sizes below 1 (a call for
 * 0 rows or tokens does nothing), a type other than the two named;
 * RLT_E_UNSUPPORTED for a page or head size other than those above. */
typedef struct rlt_cache8 {
    void* pages;
    float* scales;
    const int32_t* table;
    int32_t* status;
    int32_t n_pages, rows, row_pages, page, kv_heads, dh;
} rlt_cache8;

/* Rotary positions: cos and sin (device fp32 [positions][rot/2], aligned to 16
 * bytes) of the angles of positions 0, 1, ...; the first `rot` dimensions of
 * each head (a multiple of 8, at most dh) are rotated in pairs, (j, j + rot/2)
 * or, with interleaved != 0, (2j, 2j+1):
 *   (x1, x2) -> (x1 c - x2 s, x2 c + x1 s).
 * Token j of a row has position j + origin (origin 1: this library's 1-based
 * positions).  Scalings for long contexts are the table's. */
typedef struct rlt_rope {
    const float* cos;
    const float* sin;
    int32_t positions, rot, interleaved, origin;
} rlt_rope;

/* Append: row b's tokens i < counts[b] (counts NULL: all n; a count outside
 * [0, n] is RLT_E_CAPACITY in status, and the row is left as it was) become
 * tokens start[b] + i of the cache, their keys rotated first when rope is not
 * NULL.  k, v: `dtype` (RLT_DTYPE_F32 or _BF16) [rows][n][kv_heads][dh] with
 * row and token pitches in elements, heads adjacent; pitches and addresses
 * multiples of 16 bytes.  start, counts: device int32 [rows].
 * The scale of a (page, head) is the smallest power of two, at least 2^-110,
 * that brings the largest magnitude of the tokens written to at most 448; a
 * page that already holds tokens of the row (start[b] inside it) keeps the
 * larger of its scale and the new one, its bytes brought to it (exactly, but
 * for magnitudes below 2^-6 of a scale, which round again).  Values are
 * rounded to nearest even after the rotation, whose products and sums are
 * rounded in fp32 one by one.  NaN stays NaN; infinities become +-448 scales
 * and count as the largest finite value. */
int rlt_cache8_append(const rlt_cache8* cache, int dtype, const void* k, int64_t k_row,
                      int64_t k_token, const void* v, int64_t v_row, int64_t v_token,
                      const int32_t* start, const int32_t* counts, int n, const rlt_rope* rope,
                      void* stream);

/* Attention of n queries per row over the row's first lens[b] tokens: query i
 * (the block's i-th newest-to-be: token lens[b] - n + i of the row) sees the
 * tokens 0 .. lens[b] - n + i; one that sees none gives 0.  heads is a
 * multiple of kv_heads, query head h reads key head h / (heads / kv_heads).
 *   out = softmax(scale * q . k) v, q rotated at its token's position when
 * rope is not NULL.  q, out: `dtype` [rows][n][heads][dh] with row and token
 * pitches in elements, heads adjacent, 16-byte multiples as above; out must not
 * overlap q.  lens: device int32 [rows].  Scores, the softmax and the sums are
 * fp32, and the value scales of a prefix may lie any distance apart (blocks of
 * zeros, 2^-110, among them).  With up to 4 query vectors per key head
 * (n * heads / kv_heads) a rotated query enters the score product and the
 * probabilities the value product with 22 significant bits (fewer below 2^-29
 * of the largest among 16 neighbouring keys).  With more, they do with 22 (fp32
 * types) or 11 (bf16 types), and a probability times its value scale below
 * 2^-20 of the query's largest is off by up to 2^-42 (bf16 types: 2^-31) of
 * that: beside values that much larger, in any dimension, a query's other
 * values lose bits, and beside an appended infinity they are lost.  A row's
 * result does not depend on the other rows, on `rows` or on row_pages, bit for
 * bit.  NaN in a value makes at least that dimension of the queries that see
 * it NaN, and of no others. */
int rlt_cache8_attend(const rlt_cache8* cache, int dtype, const void* q, int64_t q_row,
                      int64_t q_token, void* out, int64_t out_row, int64_t out_token, int heads,
                      int n, const int32_t* lens, float scale, const rlt_rope* rope,
                      void* stream);

/* Beam search's selection.  For every group (search) of `beams` rows of
 * logits (`dtype` fp32 or bf16, [groups][beams][vocab], dense, no alignment
 * beyond the element's) the candidates are, per beam b and token v,
 *   c(b, v) = scores[b] + log softmax(logits_b / temperature)[v],
 * and for a beam with finished[b] != 0 (uint8, NULL: none) the single candidate
 * (b, eos) with score scores[b].  The k largest go out in descending order,
 * equal ones by ascending b * vocab + v: parents (the beam within the group),
 * tokens, new_scores [groups][k]; new_finished (uint8, may be NULL) is 1 where
 * the parent was finished or the token is eos (eos < 0: no token is).  Scores
 * are formed and compared in fp64 and rounded once, but for the softmax's sum,
 * whose exponentials are single ones: c is off by about 1e-8, at most 2^-21, alike
 * for all candidates of a beam, so beams that close may change places.  Zero
 * logits of either sign are equal.  A logit of -inf or NaN is
 * no candidate, nor is anything of a beam whose score is not finite (its
 * logits are not read: the empty beams of a search's first token) or that has
 * a +inf logit; when fewer than k candidates are left, the remaining outputs
 * are parent 0, token 0, score -inf, not finished.  Outputs may not overlap
 * inputs.  1 <= beams, k <= 64, vocab < 2^24, k <= beams * vocab; temperature
 * in [2^-20, 2^20]; finished needs 0 <= eos < vocab. */
int rlt_beam_select(int dtype, const void* logits, const float* scores, const uint8_t* finished,
                    int eos, float temperature, int groups, int beams, int vocab, int k,
                    int32_t* parents, int32_t* tokens, float* new_scores, uint8_t* new_finished,
                    void* stream);

/* Reorders the rows of one buffer within groups of `beams` (1 .. 64), in
 * place: row g*beams + i takes the contents that row g*beams + parents[g][i]
 * had before the call, in bytes [offset, offset + bytes) of each of its
 * `planes` planes (plane_stride apart; rows row_stride apart).  parents:
 * device int32 [groups][beams]; an index outside [0, beams) leaves its row as
 * it was.  Any alignment; 16-byte multiples everywhere run fastest. */
int rlt_rows_reorder(void* rows, const int32_t* parents, int groups, int beams, int64_t row_stride,
                     int planes, int64_t plane_stride, int64_t offset, int64_t bytes,
                     void* stream);

/* Beam search over the rows of a state: rows g*beams .. g*beams + beams - 1 are
 * the beams of search g (beams divides batch, at most 64; RLT_E_ARG) and stand
 * at equal positions (else RLT_E_ORDER).
 *
 * rlt_state_reorder: row g*beams + i takes up all that row g*beams +
 * parents[g*beams + i] needs to continue (s, R, the window rings, C^E, M, the
 * e_t not yet consumed), all rows at once, in place.  The rows of a search
 * hold the same C^E and M at positions 1 .. shared (a common prompt; 0: none
 * promised), which are not moved.  parents: int32 [batch], host or device; on
 * the host an entry outside [0, beams) is RLT_E_ARG, on the device it leaves
 * its row as it was (RLT_E_ARG off 4 bytes, or on another device than the
 * model's).  e_t of consumed positions stay where they are. */
int rlt_state_reorder(rlt_state* state, const int32_t* parents, int beams, int shared,
                      void* stream);

/* One step of beam search: the readout of every row, rlt_beam_select with k =
 * beams over logits / temperature, rlt_state_reorder by the chosen parents,
 * then the chosen tokens are encoded and consumed (one transition).  scores
 * (fp32 [batch], log-probabilities so far) and finished (uint8 [batch], may be
 * NULL: no beam ends) are read and replaced; parents (within the search) and
 * tokens (int32 [batch]) receive what was chosen: the caller keeps them, step
 * by step, to read the sequences back.  A finished beam goes on with eos at an
 * unchanged score.  A search starts with all rows past the prompt, scores 0
 * for its first row and -infinity for the others.  All four arrays are memory
 * of the model's device, aligned to their elements (else RLT_E_ARG).  The first call allocates 5 * batch bytes in the state.  RLT_E_ORDER
 * when a row has encoded tokens not yet consumed, RLT_E_CAPACITY at max_len;
 * argument limits as rlt_beam_select's. */
int rlt_beam_step(rlt_state* state, float* scores, uint8_t* finished, int eos, float temperature,
                  int beams, int shared, int32_t* parents, int32_t* tokens, void* stream);

/* Number of kernels this library has launched in this process. */
uint64_t rlt_kernel_launches(void);

/* Live kernel timing for measurement.  While enabled (on != 0), the library
 * brackets every launch of the classes below with CUDA events recorded on the
 * launching stream and counts the algorithmic bytes each launch must move
 * (keys/values read, cache entries written, activations in and out; weights
 * excluded).  rlt_profile_query synchronises `stream`, sums the elapsed times
 * of the class since the last enable, and reports launches, total ms and
 * bytes.  Enabling resets the counters.  on = 1: transition blocks replayed
 * as CUDA graphs are timed as whole blocks (RLT_PROF_STEP) only; on = 2: they
 * replay a twin graph with event nodes around each attention launch (those
 * launches then lose their overlap with the kernel before them) and each
 * replay is followed by a stream synchronisation: for measurement only. */
#define RLT_PROF_XATTN 0  /* decoder cross-attention over M_{<=t}        */
#define RLT_PROF_SWA   1  /* decoder window attention over C^D           */
#define RLT_PROF_STEP  2  /* one whole transition block (merge .. s_t)   */
#define RLT_PROF_ENC   3  /* one whole encoder block (embed .. memory)   */
#define RLT_PROF_ENC1  4  /* the same, for a one-position call (a new   */
                          /* token during generation)                   */
#define RLT_PROF_NCLS  5
/* cls + RLT_PROF_NCLS * (l + 1) queries the window or cross-attention
 * launches of decoder layer l alone (0 <= l < L_D). */
int rlt_profile_enable(rlt_state* state, int on);
int rlt_profile_query(rlt_state* state, int cls, uint64_t* launches, double* total_ms,
                      double* bytes, void* stream);

/* Static description of a return code. */
const char* rlt_strerror(int code);

#ifdef __cplusplus
}
#endif
#endif /* RLT_H */
