/*
 * fadkv.h -- C ABI of the FAD-KV per-token KV encoding library (sm_103a).
 *
 * What it computes comes from "FAD-KV: Adaptive Dictionary KV Caching for
 * Efficient Reasoning Decoding" (thelatestinai.com/papers/2610.37921):
 *   - abstract: each token's key or value head-vector is represented as a
 *     sparse combination of dictionary atoms; a screening-based sparse coder
 *     makes a one-shot Top-n selection of a small candidate pool and then
 *     refines coefficients; a fixed-size adaptation reuses inactive atoms
 *     instead of growing the dictionary;
 *   - Fig. 2 caption: if the reconstruction error of an incoming vector is
 *     high, an inactive atom is replaced by a context-relevant atom, keeping
 *     the dictionary size fixed throughout decoding;
 *   - Table 5: ridge parameter 1e-4 + 0.20 diag(G), thresholds 0.50 (key) /
 *     0.70 (value), N = 4096 / 8192, s = 8 / 16, n = 256 / 512.
 * Conventions the pages leave open, fixed by this library:
 *   - the s atoms are chosen greedily inside the pool: at step k the atom of
 *     the pool (not yet chosen) with the largest |<d_j, e_k>| is added, the
 *     coefficients are refit by the ridge solve, e_{k+1} = x - D_S c;
 *   - every tie (Top-n cut, greedy choice) goes to the lower atom index;
 *   - replacement order: the m-th flagged vector of a call (ascending vector
 *     index, relres > delta strictly) takes the m-th inactive atom (ascending
 *     atom index, usage == 0 after the call's usage increments);
 *   - the replacement atom is the normalised ridge residual e/||e||; the
 *     vector gets it as an extra term with coefficient ||e||.
 *
 * Memory and threading model
 *   - Every array argument is a DEVICE pointer unless stated otherwise.  The
 *     caller owns all device memory (dictionary, usage counts, workspace,
 *     inputs, outputs); the library never allocates or frees device memory.
 *   - A handle covers G = num_dicts independent dictionaries of the same
 *     shape, stored back to back, so one call encodes a whole decode step
 *     (all layers, keys and values) in one launch per kernel.
 *     Layouts (row-major, dictionary-major):
 *       atoms     [G][N][d]   binary16 or binary32 (params.dtype)
 *       usage     [G][N]      int32
 *       x         [G][V][d]   same type as atoms
 *       idx       [G][V][s]   int32, pick order; -1 for a non-finite input
 *       coef      [G][V][s]   float32
 *       relres    [G][V]      float32, ||x - D_S c|| / ||x||  (0 if x = 0)
 *       repl_id   [G][V]      int32, replacement atom or -1
 *       repl_coef [G][V]      float32
 *       xhat      [G][V][d]   float32
 *   - All calls are asynchronous on the given CUDA stream (a cudaStream_t
 *     passed as void*; NULL = legacy default stream).  A handle is not
 *     thread-safe: issue its calls from one thread, in stream order.
 *   - Every encode batch must be passed to fadkv_adapt before the next
 *     encode or adapt on the same handle (otherwise the usage counts would
 *     miss that batch and an atom in use could be overwritten).  The host
 *     enforces this and returns FADKV_ERR_SEQUENCE.
 *
 * Errors
 *   - Functions return a fadkv_status; nothing is thrown across the ABI.
 *   - Argument errors are detected on the host before any launch, and leave
 *     the handle's state unchanged.
 *   - Conditions found on the device (non-finite input, a refit matrix that
 *     is not positive definite) set bits in the per-dictionary device status
 *     word, read back by fadkv_dict_stats after a stream sync.
 */
#ifndef FADKV_H
#define FADKV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define FADKV_ABI_VERSION 1
#define FADKV_MAX_DICTS 256   /* dictionaries per handle */
#define FADKV_MAX_S 32        /* largest sparsity s */
#define FADKV_MAX_POOL 1024   /* largest pool size n */

typedef enum {
    FADKV_OK = 0,
    FADKV_ERR_INVALID_ARG = 1,   /* null pointer, bad size, misaligned pointer */
    FADKV_ERR_UNSUPPORTED = 2,   /* shape outside what the kernels implement */
    FADKV_ERR_SEQUENCE = 3,      /* encode/adapt called out of order */
    FADKV_ERR_CUDA = 4,          /* a CUDA runtime call or launch failed */
    FADKV_ERR_WORKSPACE = 5      /* workspace too small */
} fadkv_status;

/* FADKV_BF16 is taken by the paged-cache calls only; dictionaries and codes
   are binary16 or binary32. */
typedef enum { FADKV_F16 = 0, FADKV_F32 = 1, FADKV_BF16 = 2 } fadkv_dtype;

/* Device status word bits (per dictionary, see fadkv_dict_stats). */
#define FADKV_DEV_NONFINITE_INPUT 0x1   /* an input held a NaN or infinity */
#define FADKV_DEV_NOT_SPD 0x2           /* a refit matrix lost positive definiteness */
#define FADKV_DEV_TIMEOUT 0x4           /* a kernel gave up waiting on its own pipeline */

typedef struct {
    int32_t num_dicts;   /* G, 1 .. FADKV_MAX_DICTS */
    int32_t N;           /* atoms per dictionary, multiple of 64 */
    int32_t d;           /* head dimension: 64 or 128 */
    int32_t n;           /* Top-n pool size, s <= n <= min(N, FADKV_MAX_POOL) */
    int32_t s;           /* atoms per vector, 1 .. FADKV_MAX_S */
    float lambda_abs;    /* ridge, absolute part (Table 5: 1e-4) */
    float lambda_rel;    /* ridge, part relative to diag(G) (Table 5: 0.20) */
    int32_t dtype;       /* fadkv_dtype of atoms and inputs */
    int32_t max_batch;   /* largest V (vectors per dictionary) of one call */
} fadkv_params;

typedef struct fadkv_dict_s* fadkv_dict;

/* Version of this ABI (FADKV_ABI_VERSION of the built library). */
int32_t fadkv_abi_version(void);

/* Human-readable name of a status code (static string). */
const char* fadkv_status_string(fadkv_status status);

/* Message of the last CUDA error seen by a call on this host thread
   (static thread-local buffer; "" if none). */
const char* fadkv_last_error(void);

/* Bytes of device workspace a handle with these parameters needs.
   Host-only; writes *bytes.  Errors: INVALID_ARG, UNSUPPORTED. */
fadkv_status fadkv_workspace_bytes(const fadkv_params* params, size_t* bytes);

/* Create a handle over caller-owned device memory.
     atoms      [G][N][d] dictionary (mutated by fadkv_adapt), 16-byte aligned
     usage      [G][N] usage counts (mutated by fadkv_adapt); an atom is
                inactive while its count is 0; a negative count marks a
                free slot, a row that holds no atom yet (keep its row zero:
                screening still reads it, and a zero row scores 0), which
                only fadkv_adapt_append fills
     delta      HOST array [G] of adaptation thresholds (Table 5: 0.50 for a
                key dictionary, 0.70 for a value dictionary); copied
     workspace  device buffer of at least fadkv_workspace_bytes bytes,
                256-byte aligned, ZERO-FILLED before this call (it holds the
                per-dictionary counters); owned by the caller, used by the
                handle until fadkv_dict_destroy
   Host-only: makes no CUDA call.  Errors: INVALID_ARG, UNSUPPORTED,
   WORKSPACE. */
fadkv_status fadkv_dict_create(const fadkv_params* params, void* atoms, int32_t* usage,
                               const float* delta, void* workspace, size_t workspace_bytes,
                               fadkv_dict* out);

/* Rebuild the handle's Gram matrices from the atoms as they stand.  For
   binary16 dictionaries screened on the tensor cores (N a multiple of 128,
   n <= 512, s <= 16) the greedy coder reads the inner products of the atoms
   from a Gram matrix per dictionary kept in the workspace (G * N * N * 4
   bytes of fadkv_workspace_bytes).  It is built by the first fadkv_encode
   and kept up to date by fadkv_adapt / fadkv_adapt_append, which rewrite its
   rows and columns of the atoms they write.  A caller that changes atoms in
   any other way (its own copies, fadkv_adapt_noalloc on the same buffer)
   calls this before the next fadkv_encode.  Asynchronous on `stream`; a
   no-op for handles without Gram matrices.  Errors: INVALID_ARG, CUDA. */
fadkv_status fadkv_dict_refresh(fadkv_dict dict, void* stream);

/* Free the host-side handle.  Device memory stays with the caller.
   The caller must make sure no work of this handle is still running. */
fadkv_status fadkv_dict_destroy(fadkv_dict dict);

/* Encode V vectors per dictionary (abstract; Fig. 2 caption: screening-based
   sparse coding).  For every x: scores r = D x; pool P = the n atoms with the
   largest |r_j| (ties to the lower j); s greedy picks inside P with the ridge
   refit (G + diag(lambda_abs + lambda_rel G_ii)) c = D_S x after each pick;
   relres = ||x - D_S c|| / ||x||.
     x [G][V][d]; outputs idx [G][V][s], coef [G][V][s], relres [G][V].
   0 <= V <= max_batch.  Every vector is encoded against the dictionary as it
   stands at the start of the call.  A vector holding a NaN or infinity gets
   idx = -1, coef = 0, relres = NaN and sets FADKV_DEV_NONFINITE_INPUT.
   Errors: INVALID_ARG, SEQUENCE (previous encode not adapted yet), CUDA. */
fadkv_status fadkv_encode(fadkv_dict dict, const void* x, int32_t V, int32_t* idx, float* coef,
                          float* relres, void* stream);

/* PL encode: the cheaper coder of the "PL (ours)" rows of Tables 1-4 (Table 4:
   Cost 0.13 of OMP, against 0.19 for the greedy coder).  The pages name it
   without spelling it out; this library reads it as screening plus a single
   ridge fit, the reading that cost supports: for every x, scores r = D x;
   S = the s atoms with the largest |r_j| (ties to the lower j); one solve
   (G + diag(lambda_abs + lambda_rel G_ii)) c = D_S x with G = D_S D_S^T;
   relres = ||x - D_S c|| / ||x|| (0 if x = 0).
     x [G][V][d]; outputs idx [G][V][s] in ASCENDING atom order (not a pick
     order), coef [G][V][s] aligned with idx, relres [G][V].
   Arguments, ordering and errors as for fadkv_encode: the batch counts as
   an encode and must be passed to fadkv_adapt (which works the same on
   either coder's output) before the next encode; a non-finite x gets
   idx = -1, coef = 0, relres = NaN.  The handle's n is not used.
   Errors: INVALID_ARG, SEQUENCE, CUDA. */
fadkv_status fadkv_encode_pl(fadkv_dict dict, const void* x, int32_t V, int32_t* idx, float* coef,
                             float* relres, void* stream);

/* Fixed-size adaptation of the batch just encoded (abstract; Fig. 2 caption).
   usage[idx] += 1 for every selected atom; then the m-th vector with
   relres > delta[g] (ascending v) takes the m-th atom with usage == 0
   (ascending id): that atom becomes e/||e|| with e = x - D_S c (rounded to
   the dictionary type), its usage becomes 1, repl_id[v] = its id and
   repl_coef[v] = ||e||.  Other vectors get repl_id = -1, repl_coef = 0.
   Flagged vectors left without an inactive atom keep their s-term code and
   are counted as overflow.  The dictionary keeps N atoms; free slots
   (usage < 0) are never taken.
   Arguments are the same x, V, idx, coef, relres as the encode call.
   Errors: INVALID_ARG, SEQUENCE (no encode pending, or a different V), CUDA. */
fadkv_status fadkv_adapt(fadkv_dict dict, const void* x, int32_t V, const int32_t* idx,
                         const float* coef, const float* relres, int32_t* repl_id,
                         float* repl_coef, void* stream);

/* Append-only growth: the strategy the pages contrast FAD-KV with (abstract:
   naive append-only updates grow the dictionary during generation; Fig. 2
   caption: FAD-KV replaces an inactive atom instead of appending a new one),
   for side-by-side runs.  The same as fadkv_adapt except for the rows the
   flagged vectors take: the m-th flagged vector (ascending v, relres >
   delta[g]) takes the m-th FREE SLOT (usage < 0, ascending id) instead of an
   inactive atom, so the dictionary grows by one atom per flagged vector
   into the capacity the caller reserved, and no atom, inactive or not, is
   ever rewritten.  Flagged vectors beyond the free slots are counted as
   overflow; "atoms replaced" in fadkv_dict_stats counts appended atoms.
   The dictionary's size is the number of rows with usage >= 0.  Arguments,
   sequence contract and errors as for fadkv_adapt. */
fadkv_status fadkv_adapt_append(fadkv_dict dict, const void* x, int32_t V, const int32_t* idx,
                                const float* coef, const float* relres, int32_t* repl_id,
                                float* repl_coef, void* stream);

/* Fixed-size adaptation without a handle and without caller scratch.  The
   pages have no counterpart to this call: it runs the same adaptation as
   fadkv_adapt (same kernel, same results) for callers that cannot give the
   library any device memory of its own, e.g. a plain C runtime with a fixed
   memory plan and no allocator, or a decode loop that must not call
   cudaMalloc / cudaFree since either can synchronise the whole device.
     params     shape and dtype (max_batch is not used; V is limited by the
                scratch instead); the same checks as fadkv_workspace_bytes
     atoms      [G][N][d] dictionary, 16-byte aligned (mutated)
     usage      [G][N] int32 usage counts (mutated)
     delta      HOST array [G] of thresholds, each >= 0
     x, V, idx, coef, relres, repl_id, repl_coef: as for fadkv_adapt
     stream     cudaStream_t as void*; NULL = legacy default stream
   Scratch: one statically sized device array inside the library (4 MiB per
   device) holds the inactive-atom list, the flagged-vector list and the
   counters.  A call needs 256-rounded 4*G*N + 4*G*V bytes plus 64*G; more
   than 4 MiB returns FADKV_ERR_WORKSPACE with the sizes in
   fadkv_last_error(), before any CUDA call.  Nothing in the scratch has to
   start at zero, and the library allocates and frees nothing.
   The first call on a device looks up the scratch's address there
   (cudaGetSymbolAddress, with that device current) and keeps it for the CUDA
   context current at the time; a call made in another context of that device
   (a non-primary context made current, or the primary context re-created
   after cudaDeviceReset) looks it up again.  A caller that records its calls
   under stream capture should make one call on each device, in the context
   it captures in, before capture begins.  All calls on one device share the
   one scratch array:
   calls that may run concurrently (different streams or host threads) race,
   so issue them in order on one stream.  There is no sequence check and no
   per-dictionary statistics: the caller keeps encode/adapt order itself.
   Errors: INVALID_ARG, UNSUPPORTED, WORKSPACE, CUDA. */
fadkv_status fadkv_adapt_noalloc(const fadkv_params* params, void* atoms, int32_t* usage,
                                 const float* delta, const void* x, int32_t V, const int32_t* idx,
                                 const float* coef, const float* relres, int32_t* repl_id,
                                 float* repl_coef, void* stream);

/* Sparse reconstruction (abstract: a sparse combination of atoms):
   xhat_v = sum_k coef[v][k] d_{idx[v][k]} + repl_coef[v] d_{repl_id[v]}.
   repl_id / repl_coef may both be NULL (no replacement terms); entries with
   idx or repl_id = -1 are skipped.  Valid for any code produced earlier by
   encode + adapt: atoms in use are never overwritten.
   Errors: INVALID_ARG, CUDA. */
fadkv_status fadkv_reconstruct(fadkv_dict dict, int32_t V, const int32_t* idx, const float* coef,
                               const int32_t* repl_id, const float* repl_coef, float* xhat,
                               void* stream);

/* Per-dictionary counters, copied to HOST memory host_out[G][FADKV_STATS_FIELDS];
   synchronises the stream.  Fields, in order: vectors encoded (adapted),
   atoms replaced, flagged vectors, overflow (flagged without an inactive
   atom), non-finite inputs, Top-n slow-path uses, device status word, 0.
   Errors: INVALID_ARG, CUDA. */
#define FADKV_STATS_FIELDS 8
fadkv_status fadkv_dict_stats(fadkv_dict dict, int64_t* host_out, void* stream);

/* Test hook: the Top-n pool of each x without changing any state.
   pool [G][V][n] int32, the pool's atom ids in no particular order (-1 for
   a non-finite input); pool_r (may be NULL) [G][V][n] float32 |r| of those
   atoms, in the same order.  Errors: INVALID_ARG, CUDA. */
fadkv_status fadkv_debug_pool(fadkv_dict dict, const void* x, int32_t V, int32_t* pool,
                              float* pool_r, void* stream);

/* Test hook: screening scores [G][V][N] float32 of each x, from the same
   screening kernel encode uses (tensor cores for binary16 dictionaries).
   No state changes.  V must not exceed the handle's internal pass size
   (at least min(max_batch, 128)).  Errors: INVALID_ARG, CUDA. */
fadkv_status fadkv_debug_scores(fadkv_dict dict, const void* x, int32_t V, float* scores, void* stream);

/* Test hook: the wall-clock limit, in nanoseconds, of the waits inside the
   tensor-core screening pipeline of this handle (0 = the default, 200 ms).
   A wait that runs out sets FADKV_DEV_TIMEOUT in the status word and the
   kernel stops early: that pass's candidates are then incomplete (codes stay
   valid atom ids, but are not the exact encode).  The kernel still waits for
   every copy and MMA it issued, with the default limit, before it returns.
   Host-only.  Errors: INVALID_ARG. */
fadkv_status fadkv_debug_wait_limit(fadkv_dict dict, uint64_t limit_ns);

/* Test hook: launches one thread that waits, with a limit of limit_ns
   (1 .. 10^10), on a barrier nothing ever arrives on, so the wait runs out
   and sets FADKV_DEV_TIMEOUT in dictionary 0's status word (read it with
   fadkv_dict_stats).  Nothing else is touched.  Asynchronous on `stream`.
   Errors: INVALID_ARG, CUDA. */
fadkv_status fadkv_debug_wait_probe(fadkv_dict dict, uint64_t limit_ns, void* stream);

/* ---------------------------------------------------------------------------
   The compressed KV store and decode attention over it.  Handle-free: both
   calls work on caller-owned buffers only.

   What the cache keeps instead of K and V is the codes (Table 4: the
   per-sequence KV memory of the dictionary methods against full KV).  The
   pages give no storage format; this library packs every nonzero into one
   32-bit word:
     bits 31..13  the coefficient rounded to 11 significant bits (round to
                  nearest, ties to even) in the layout of binary32's top 19
                  bits (sign, 8-bit exponent, 10 fraction bits); magnitudes
                  below 2^-126 are stored as 0;
     bits 12..0   the atom id (so N <= 8192).
   A token's code is s + 1 words: its s terms, then its replacement term
   from the adaptation (word 0 when it has none).  A skipped term (id -1, a
   zero or non-finite coefficient) is word 0: coefficient 0, atom 0.
   --------------------------------------------------------------------------- */
#define FADKV_PACK_ID_BITS 13

/* Store one step's codes in the per-sequence caches.
     G dictionaries, each with V = B * H vectors ordered v = b * H + h
     (sequence b, KV head h); idx / coef [G][V][s] and repl_id / repl_coef
     [G][V] (both NULL: no replacement words) as fadkv_encode / fadkv_adapt
     wrote them; pos [B] device int32: the token position of this step in
     each sequence's cache; cache [G][B][H][Tmax][s+1] uint32, written at
     [g][b][h][pos[b]][0..s] only (positions outside [0, Tmax) are skipped).
   All pointers are device pointers, 4-byte aligned.  Asynchronous on
   `stream`.  Errors: INVALID_ARG, UNSUPPORTED (N > 8192, s > FADKV_MAX_S),
   CUDA. */
fadkv_status fadkv_store_codes(int32_t G, int32_t B, int32_t H, int32_t s, int32_t N, const int32_t* idx,
                               const float* coef, const int32_t* repl_id, const float* repl_coef,
                               const int32_t* pos, uint32_t* cache, int32_t Tmax, void* stream);

typedef struct {
    int32_t layers;     /* L */
    int32_t B;          /* sequences */
    int32_t Hq;         /* query heads (a multiple of Hkv) */
    int32_t Hkv;        /* KV heads; query head h reads KV head h / (Hq / Hkv) */
    int32_t d;          /* head dimension: 64 or 128 */
    int32_t N;          /* atoms per dictionary, <= 8192 */
    int32_t s;          /* terms per code (s + 1 words per token) */
    int32_t Tmax;       /* cache capacity in tokens */
    int32_t dtype;      /* fadkv_dtype of the dictionaries */
    float scale;        /* score scale, 1/sqrt(d) for standard attention */
    int64_t dict_stride;   /* elements from layer l's key (value) dictionary to layer l+1's; a multiple of 8 */
    int64_t cache_stride;  /* words from layer l's key (value) cache to layer l+1's */
} fadkv_attn_params;

/* Decode attention over the compressed store, for every layer, sequence and
   query head in one call (three kernel launches for binary16 dictionaries,
   one for binary32):
     out[l][b][h] = sum_t p_t v_t,  p = softmax_t(scale <q[l][b][h], k_t>),
   over the tokens t < lengths[b] of KV head h / (Hq / Hkv) of sequence b,
   where k_t and v_t are the sparse combinations their packed codes name:
   k_t = sum_i c_ti dict_k[j_ti].  Neither K nor V is rebuilt: with
   u = dict_k q the scores are s + 1 gathers from u per token, and the output
   is dict_v^T w with w the attention-weighted sum of the value codes.
     dict_k, dict_v  device, layer l's [N][d] dictionaries at + l*dict_stride
                     (with one handle's atoms [2L][N][d], keys at even g:
                     dict_k = atoms, dict_v = atoms + N*d, dict_stride = 2*N*d),
                     16-byte aligned
     cache_k, cache_v device, layer l's [B][Hkv][Tmax][s+1] packed codes at
                     + l*cache_stride (fadkv_store_codes with G = 2L: cache_k
                     = cache, cache_v = cache + B*Hkv*Tmax*(s+1), cache_stride
                     = 2*B*Hkv*Tmax*(s+1))
     lengths         device [B] int32, clamped to [0, Tmax]; an empty
                     sequence gives 0
     q, out          device [L][B][Hq][d] float32 (q 16-byte aligned: its rows
                     are read as vectors)
     workspace       device, >= fadkv_attend_workspace_bytes bytes, 256-byte
                     aligned, caller-owned (contents need no initialisation)
   With binary16 dictionaries the two dictionary products run as per-layer
   tensor-core GEMMs over all sequences and heads (q and w enter as two
   binary16 terms each, about 22 significant bits; FP32 sums); the token
   pass is FP32.  Binary32 dictionaries: FP32 throughout.  Asynchronous on
   `stream`.  Errors: INVALID_ARG, UNSUPPORTED, WORKSPACE, CUDA. */
fadkv_status fadkv_attend(const fadkv_attn_params* params, const void* dict_k, const void* dict_v,
                          const uint32_t* cache_k, const uint32_t* cache_v, const int32_t* lengths,
                          const float* q, float* out, void* workspace, size_t workspace_bytes,
                          void* stream);

/* Device workspace fadkv_attend needs for these parameters (host-only;
   writes *bytes).  Binary16 dictionaries: the per-layer products U = scale
   Q D_K^T and the token pass's weights W, 8 * layers * B * Hq *
   round_up(N, 16) bytes and a little more; binary32 dictionaries: 0 (the
   workspace may then be NULL).  Errors: INVALID_ARG, UNSUPPORTED. */
fadkv_status fadkv_attend_workspace_bytes(const fadkv_attn_params* params, size_t* bytes);

/* ---------------------------------------------------------------------------
   The paged cache of full key/value vectors: what a decode loop keeps of the
   vectors that are not coded (a prompt before its encode, the recent window
   and the first tokens, or the whole cache in a full-KV run).  Attention over
   pages and over codes are separate answers: fadkv_attend takes no range of
   tokens and returns no log-sum-exp, so a window here and the codes of the
   other tokens do not join into one softmax.  Handle-free:
   every call works on caller-owned buffers only, asynchronously on `stream`,
   and can be captured into a CUDA graph.

   A pool holds num_pages pages of page_size tokens (a power of two, 8 ..
   1024) for every key/value head; keys and values are two pools of one
   layout.  Element (page, head, token in page, i) of a pool is at
     page * page_stride + head * head_stride + token * token_stride + i
   (strides in elements, multiples of 8; the pools 16-byte aligned).  Row b
   of the block table [B][max_pages] int32 lists the pages of request b in
   token order.  The slot of a token is page * page_size + token in page.
   --------------------------------------------------------------------------- */
#define FADKV_MAX_REQUESTS 12288   /* largest B of the paged-cache calls */

typedef struct {
    int32_t B;            /* requests, 0 .. FADKV_MAX_REQUESTS */
    int32_t page_size;    /* tokens per page */
    int32_t num_pages;    /* pages of a pool; num_pages * page_size < 2^31 */
    int32_t max_pages;    /* block-table entries per request */
    int32_t max_tokens;   /* rows of positions and slots */
} fadkv_page_params;

/* Plan of one step: gives the new tokens of every request their pages,
   positions and slots, and takes back the pages of requests that ended.
     add         [B] int32: new tokens of each request in this step; 0: none;
                 negative: the request ends
     lengths     [B] int32: tokens each request has cached (clamped to
                 [0, max_pages * page_size])
     block_table [B][max_pages] int32, in/out: entries of pages taken now are
                 written, all others left as they are
     free_pages  [num_pages] int32, in/out: the free pages are its first
                 free_count entries
     free_count  [1] int32 (clamped to [0, num_pages])
     lengths_out [B] int32, free_count_out [1] int32: their values after the
                 step; may be lengths and free_count themselves.  Kept apart,
                 the call can be repeated on the same inputs.
     starts      [B+1] int32: the requests' first rows among the step's tokens
                 (exclusive prefix sum of max(add, 0), saturated at 2^31 - 1)
     positions, slots  [max_tokens] int32: of every new token, request by
                 request; -1 for the rows past starts[B] and for requests
                 that are refused
     refused     [1] int32: requests refused in this step
   Order: first the ceil(lengths / page_size) pages of each ended request go
   to the end of the free list (ascending request, then page; what would pass
   num_pages is dropped), lengths_out = 0.  Then requests are served in
   ascending order; page m taken in this step is entry F - 1 - m of the free
   list, F its length after the returns.  A request is refused, and keeps its
   length, when its tokens would pass max_pages * page_size, when its rows
   would pass max_tokens, or when its pages and those that the requests
   before it asked for are more than F.
   All pointers are device pointers, 4-byte aligned.
   Errors: INVALID_ARG, UNSUPPORTED, CUDA. */
fadkv_status fadkv_page_plan(const fadkv_page_params* params, const int32_t* add, const int32_t* lengths,
                             int32_t* block_table, int32_t* free_pages, const int32_t* free_count,
                             int32_t* lengths_out, int32_t* free_count_out, int32_t* starts,
                             int32_t* positions, int32_t* slots, int32_t* refused, void* stream);

/* Rotation of positions.  Pair i of the rotated part (its first rotary_dim
   elements) turns by position * f_i, f_i = base^(-2 i / rotary_dim) before
   scaling for long contexts:
     FADKV_ROPE_PLAIN    f_i
     FADKV_ROPE_LINEAR   f_i / factor
     FADKV_ROPE_STRETCH  f_i of the base base * factor^(rotary_dim / (rotary_dim - 2))
     FADKV_ROPE_PARTS    with r = original * f_i / (2 pi) turns over the original
                         length and g = clamp((r - slow) / (fast - slow), 0, 1):
                         f_i * (g + (1 - g) / factor)
                         (linear in r; a checkpoint whose ramp is linear in the
                         pair's number i is another rotation)
   The rotated part is multiplied by amplitude (1 for none). */
#define FADKV_ROPE_MAX_PAIRS 64
typedef enum {
    FADKV_ROPE_PLAIN = 0,
    FADKV_ROPE_LINEAR = 1,
    FADKV_ROPE_STRETCH = 2,
    FADKV_ROPE_PARTS = 3
} fadkv_rope_scaling;

typedef struct {
    int32_t d;            /* head dimension: 64 or 128 */
    int32_t rotary_dim;   /* rotated elements: 0 (none) or a multiple of 16, <= d */
    int32_t interleaved;  /* pairs (2i, 2i+1) if set, (i, i + rotary_dim/2) if not */
    int32_t scaling;      /* fadkv_rope_scaling */
    double base;          /* > 1 */
    double factor;        /* >= 1 (LINEAR, STRETCH, PARTS) */
    double original;      /* > 0, trained length (PARTS) */
    double slow, fast;    /* slow < fast (PARTS) */
    double amplitude;     /* finite in 32 bits */
} fadkv_rope_params;

/* The rotation as the kernel reads it: a plain host struct, filled by
   fadkv_rope_init and kept by the caller. */
typedef struct {
    int32_t d, rotary_dim, interleaved;
    float amplitude;
    uint64_t turns[FADKV_ROPE_MAX_PAIRS];   /* f_i / (2 pi) in units of 2^-64 turns a position */
} fadkv_rope;

/* Host-only.  Errors: INVALID_ARG, UNSUPPORTED. */
fadkv_status fadkv_rope_init(const fadkv_rope_params* params, fadkv_rope* out);

typedef struct {
    int32_t T;            /* rows (new tokens of the step) */
    int32_t Hq, Hkv;      /* query and key/value heads */
    int32_t d;            /* head dimension: 64 or 128 */
    int32_t dtype;        /* of q, k, v and the norms' weights */
    int32_t q_dtype;      /* of q_out */
    int32_t kv_dtype;     /* of k_out and the pools */
    int32_t page_size, num_pages;
    float eps;            /* of the norms */
    int64_t q_stride, k_stride, v_stride;   /* elements from one token to the next, multiples of 8 */
    int64_t page_stride, head_stride, token_stride;   /* of the pools */
} fadkv_qk_params;

/* Norm, rotation and append of one step's keys, queries and values, in one
   pass.  Every query and key head-vector x becomes
     rotate(x / sqrt(mean(x^2) + eps) * w)
   in 32 bits, rounded once on storing; a null w leaves the norm out.
     q, k, v     rows of Hq (Hkv) heads of d elements, heads back to back, rows
                 q_stride (k_stride, v_stride) apart (three parts of one
                 projection's output, say); 16-byte aligned
     wq, wk      [d] or null
     positions   [T] int32; a row with a negative position is empty: its
                 q_out and k_out are 0 and nothing of it enters the pools
     slots       [T] int32: where row t's key and value go in the pools; slots
                 outside [0, num_pages * page_size) are skipped.  A slot may
                 appear once at most.  Null: nothing is appended.
     q_out       [T][Hq][d], e.g. binary32 for fadkv_attend
     k_out       [T][Hkv][d] or null: the keys as fadkv_encode takes them
                 (v = t * Hkv + h) with kv_dtype the dictionary's type
     k_pages, v_pages  pools (null with null slots)
   16-byte aligned throughout (positions, slots 4).  rope->d must equal d.
   Outputs and pools do not overlap the inputs.
   Errors: INVALID_ARG, UNSUPPORTED, CUDA. */
fadkv_status fadkv_qk_norm_rope(const fadkv_qk_params* params, const fadkv_rope* rope, const void* q,
                                const void* k, const void* v, const void* wq, const void* wk,
                                const int32_t* positions, const int32_t* slots, void* q_out, void* k_out,
                                void* k_pages, void* v_pages, void* stream);

typedef struct {
    int32_t B;            /* requests, 0 .. FADKV_MAX_REQUESTS */
    int32_t T;            /* query rows of all requests */
    int32_t Hq;           /* query heads (a multiple of Hkv); head h reads KV head h / (Hq / Hkv) */
    int32_t Hkv;
    int32_t d;            /* head dimension: 64 or 128 */
    int32_t dtype;        /* of q, the pools and out: FADKV_F16 or FADKV_BF16 */
    int32_t page_size, num_pages, max_pages;
    int32_t window;       /* a query sees its last `window` tokens, itself among them; 0: all */
    int32_t sinks;        /* first tokens that stay visible beside the window */
    float scale;          /* score scale, 1/sqrt(d) for standard attention */
    int64_t q_stride, out_stride;   /* elements from one row of q (out) to the next; heads back to back */
    int64_t page_stride, head_stride, token_stride;   /* of the pools */
} fadkv_paged_params;

/* Attention of one new token per request over the paged cache (T = B, row b is
   request b's; a step in which some requests bring none goes through
   fadkv_paged_prefill):
     out[b][h] = sum_j p_j v_j,  p = softmax_j(scale <q[b][h], k_j>),
     lse[b][h] = log sum_j exp(scale <q[b][h], k_j>),
   over the tokens j < lengths[b] that the query at position lengths[b] - 1
   sees: all, or with a window those with j > position - window or j < sinks.
   Tokens on pages outside [0, num_pages) are not seen.  A query that sees
   nothing gets out = 0 and lse = -inf.
     lengths     [B] int32, the new token included, clamped to
                 [0, max_pages * page_size]
     q           rows of Hq heads, 16-byte aligned; out likewise
     lse         [T][Hq] float32, or null
     workspace   >= fadkv_paged_attend_workspace_bytes bytes, 256-byte aligned,
                 ZERO-FILLED before its first use (each call leaves it fit for
                 the next, whatever that call's parameters; one workspace, of
                 the larger size, may serve fadkv_paged_prefill too); not to be
                 shared by calls that may run concurrently
   Scores, softmax and sums in 32 bits; the probabilities enter the product
   with the values as two 16-bit terms each (22 bits with binary16 pools, where
   one below 2^-40 of the largest is lost; 16 bits with bfloat16).  A seen value
   that is infinite makes that element of the heads that read it infinite or
   NaN (the two terms may differ in sign, or one be 0), a NaN makes it NaN; a
   score that is NaN or +inf makes the head's row and lse NaN.  Nothing else is
   touched by them.
   Errors: INVALID_ARG, UNSUPPORTED, WORKSPACE, CUDA. */
fadkv_status fadkv_paged_attend(const fadkv_paged_params* params, const void* k_pages, const void* v_pages,
                                const int32_t* block_table, const int32_t* lengths, const void* q, void* out,
                                float* lse, void* workspace, size_t workspace_bytes, void* stream);

/* The same after a plan: positions [T] as fadkv_page_plan writes them (or
   null: none refused).  A request whose row has a negative position was
   refused in this step; its lengths entry is that of the tokens before, which
   the row does not follow.  It sees nothing (out = 0, lse = -inf). */
fadkv_status fadkv_paged_attend_planned(const fadkv_paged_params* params, const void* k_pages, const void* v_pages,
                                        const int32_t* block_table, const int32_t* lengths,
                                        const int32_t* positions, const void* q, void* out, float* lse,
                                        void* workspace, size_t workspace_bytes, void* stream);

/* Device workspace fadkv_paged_attend needs (host-only; writes *bytes).
   Errors: INVALID_ARG, UNSUPPORTED. */
fadkv_status fadkv_paged_attend_workspace_bytes(const fadkv_paged_params* params, size_t* bytes);

/* The same attention for several new tokens per request (a prompt, or a chunk
   of it on top of cached tokens): rows starts[b] .. starts[b+1]-1 of q are
   the last tokens of request b, row i of its n at position lengths[b] - n + i.
   Keys and values of the new tokens are in the pools already.
     starts      [B+1] int32 as fadkv_page_plan writes them: 0, ascending; rows
                 at and past T are left out.  Rows of q past starts[B] are not
                 read and their out and lse not written.
   Rows whose position lengths[b] - n + i is negative see nothing (out = 0,
   lse = -inf).  The rows of a request that a plan refused are not its last
   tokens: use fadkv_paged_prefill_planned, or give it a length of 0.  What the
   pools hold where no row sees it is never used; a value that is not finite
   and that one row sees may reach other rows of its request.  The
   probabilities enter the product with the values in the type of the pools,
   rounded once; with binary16 one below 2^-32 of the largest may be lost.
   workspace   >= fadkv_paged_prefill_workspace_bytes bytes, 256-byte aligned,
               ZERO-FILLED before its first use.  Its first 8 bytes are a
               status word: FADKV_DEV_TIMEOUT is set in it if a kernel gave
               up waiting on its own pipeline (that call's out is then not
               complete).  No call clears it: fadkv_paged_status reads it
   Other arguments and errors as for fadkv_paged_attend. */
fadkv_status fadkv_paged_prefill(const fadkv_paged_params* params, const void* k_pages, const void* v_pages,
                                 const int32_t* block_table, const int32_t* lengths, const int32_t* starts,
                                 const void* q, void* out, float* lse, void* workspace,
                                 size_t workspace_bytes, void* stream);

/* The same after a plan: positions [T] as fadkv_page_plan writes them (or
   null: none refused).  A request whose first row has a negative position was
   refused in this step: its rows see nothing (out = 0, lse = -inf). */
fadkv_status fadkv_paged_prefill_planned(const fadkv_paged_params* params, const void* k_pages, const void* v_pages,
                                         const int32_t* block_table, const int32_t* lengths, const int32_t* starts,
                                         const int32_t* positions, const void* q, void* out, float* lse,
                                         void* workspace, size_t workspace_bytes, void* stream);

/* The status word of a workspace of fadkv_paged_prefill, copied to HOST memory
   *host_out and, if clear is set, zeroed; synchronises the stream.  A kernel
   that gave up has waited for every copy and product that it issued and left
   the workspace fit for the next call.
   Errors: INVALID_ARG, CUDA. */
fadkv_status fadkv_paged_status(void* workspace, uint64_t* host_out, int32_t clear, void* stream);

/* Test hook: the wall-clock limit, in nanoseconds, of the waits inside the
   pipeline of the fadkv_paged_prefill calls made from now on, in the whole
   process (0 = the default, 200 ms).  Host-only. */
fadkv_status fadkv_debug_paged_wait_limit(uint64_t limit_ns);

fadkv_status fadkv_paged_prefill_workspace_bytes(const fadkv_paged_params* params, size_t* bytes);

/* Kernel classes reported by fadkv_profile_read. */
#define FADKV_PROFILE_KERNELS 8
#define FADKV_K_SCREEN 0       /* screening (tensor cores + candidate filter, or FP32 scores) */
#define FADKV_K_TOPN 1         /* Top-n: the selection from the screening records and the exact
                                  pool fixup, or the radix Top-n over FP32 scores (binary32) */
#define FADKV_K_GREEDY 2       /* in-pool greedy selection + ridge refit (the PL fit for
                                  fadkv_encode_pl) */
#define FADKV_K_ADAPT 3        /* fixed-size adaptation */
#define FADKV_K_RECONSTRUCT 4  /* sparse reconstruction */
#define FADKV_K_GRAM 5         /* the dictionaries' Gram matrices: the build at the first encode
                                  (or fadkv_dict_refresh) and the update after each adaptation */

/* Tracing.  The library always counts its kernel launches per class.  With
   profiling enabled it also brackets every launch with a pair of CUDA events
   recorded on the launch stream and accumulates the device time between
   them.  Not for use inside CUDA-graph capture.  Errors: INVALID_ARG. */
fadkv_status fadkv_profile_enable(fadkv_dict dict, int32_t enable);

/* The kernel classes that profiling brackets with events: bit k of
   class_mask stands for class k (FADKV_K_*); all classes by default.  Launch
   counts are kept for every class regardless.  Bracketing fewer launches
   leaves the others back to back on the stream, so a timed step is
   perturbed less.  Errors: INVALID_ARG. */
fadkv_status fadkv_profile_select(fadkv_dict dict, uint32_t class_mask);

/* Launch counts and device milliseconds per kernel class since the last
   reset, written to HOST arrays launches[FADKV_PROFILE_KERNELS] and
   ms[FADKV_PROFILE_KERNELS] (either may be NULL).  Waits for the recorded
   events.  reset != 0 clears the accumulators afterwards.
   Errors: INVALID_ARG, CUDA. */
fadkv_status fadkv_profile_read(fadkv_dict dict, int64_t* launches, double* ms, int32_t reset);

#ifdef __cplusplus
}
#endif

#endif /* FADKV_H */
