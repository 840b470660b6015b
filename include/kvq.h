/*
 * kvq.h - C ABI of a GPU-resident quantised KV cache for one attention layer
 * holding B sequences: K stored q8_0 and V stored q5_1 (or both stored FP8
 * E4M3, one byte per element), with quantised append,
 * truncate-based rollback and split-K flash-decode attention (GQA fan-out,
 * learned sinks, sliding window over a rebased ring, T >= 1 causal rows).
 *
 * The operations follow these passages:
 *   memra-engine "Struct KvLayer": the quantised per-layer cache (type
 *     description: q8_0 K at 34 B / 32 elements, q5_1 V at 24 B / 32 elements,
 *     [token, kv_head, dim] element order, head_dim % 32 == 0), the device
 *     mirrors len_d (append slot before the append, t_kv after it) and base_d
 *     (physical row of logical row 0 for the windowed ring view:
 *     lstart = max(0, len - window), physical = row - base), fn physical_rows.
 *   memra-engine "Struct Cache": fn new (allocate by geometry and max context),
 *     fn rollback item C.1 (len = snapshot_len + accept_len, truncate, no copy).
 *   memra-engine "Module cache": trait KvDev (every device op is ordered on the
 *     caller's stream), fn kv_blk_bytes, fn cache_bytes_per_token,
 *     fn swa_ring_rows (the ring keeps at most 31 masked rows before the live
 *     window), fn cache_ring_row_cap.
 *   cortiq-engine "Struct LayerKvCache": attention semantics of
 *     fn attend_group / fn attend_group_upto (scale 1/sqrt(head_dim), window
 *     start `first`, causal `upto = s0 + i + 1`, sink logits joining max and
 *     denominator without a value) and fn o1_views (head h reads group h/hpk).
 *
 * Ownership.  The caller allocates and owns every device buffer (the two byte
 * planes, the counters and the workspace, sized by kvq_required_bytes) and
 * every stream.  The library owns only the host handle returned by kvq_alloc.
 * It never allocates device memory, never frees caller memory and never
 * synchronises a stream except in kvq_read_device_error.  All device work is
 * enqueued on the stream passed to the call (NULL = the legacy default
 * stream); the caller keeps its buffers alive until that work completes.
 *
 * Errors.  Every call validates its arguments against the host mirror of the
 * lengths before it enqueues anything.  On error it enqueues nothing, leaves
 * the cache unchanged and returns a status; kvq_last_error() then gives a
 * one-line message (thread-local).  KVQ_ECUDA reports a failed launch; the
 * cache state is then undefined.  Kernels never trap: a kernel that finds a
 * device counter out of range, or whose bounded wait runs out, writes a
 * nonzero code to the device error word and skips its work; read it with
 * kvq_read_device_error.
 *
 * Graph capture.  kvq_append, kvq_decode and kvq_truncate read the lengths and
 * the ring base on the device, so a captured append+decode step replays
 * correctly as the lengths grow.  After replaying a captured chain of appends
 * call kvq_note_replayed so the host mirror follows; after one that contains
 * kvq_truncate_device (its accepted counts read on the device), call
 * kvq_sync_len instead.  A ring rebase is decided
 * on the host inside kvq_append: capture at most kvq_ring_headroom() appends.
 */
#ifndef KVQ_H
#define KVQ_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum kvq_status {
    KVQ_OK = 0,
    KVQ_EINVAL = 1,        /* bad argument or geometry                       */
    KVQ_ERANGE = 2,        /* length/capacity out of range                   */
    KVQ_ECUDA = 3,         /* a CUDA runtime call failed                     */
    KVQ_EUNSUPPORTED = 4   /* valid request this build does not implement    */
} kvq_status;

typedef enum kvq_dtype { KVQ_F32 = 0, KVQ_BF16 = 1 } kvq_dtype;

/* Block formats (memra-engine "Module cache", fn kv_blk_bytes):
 *   KVQ_Q8_0: fp16 d = amax/127 (round to nearest even), then 32 int8 codes
 *             round-half-away-from-zero(x/d) clamped to [-127,127]    34 B
 *   KVQ_Q5_1: fp16 d = (max-min)/31, fp16 m = min, u32 qh (bit i = bit 4 of
 *             code i), 16 bytes qs (byte j = code j low nibble | code j+16
 *             low nibble << 4); codes round-half-away((x-m)/d) in [0,31]
 *             against the stored m and d                                24 B
 *   KVQ_FP8_E4M3: one byte per element, no scale (memra-engine "Module
 *             cache", items gkv_on and kv_fp8_on: K/V held in e4m3).
 *             Read as OCP FP8 E4M3: sign, 4 exponent bits with bias 7, 3
 *             fraction bits, no infinities, largest finite 448; round to
 *             nearest, ties to even, magnitudes above 448 saturate to 448.
 *             A 32-element block is 32 bytes.
 * All multi-byte fields are little-endian.  Inputs must be finite. */
typedef enum kvq_fmt { KVQ_Q8_0 = 0, KVQ_Q5_1 = 1, KVQ_FP8_E4M3 = 2 } kvq_fmt;

typedef struct kvq_config {
    int n_seq;        /* B: sequences held by this layer cache (1..4096)           */
    int n_kv_heads;   /* Hkv                                                       */
    int head_dim;     /* D: multiple of 32, at most 512                            */
    int max_q_heads;  /* largest Hq a decode may pass (a multiple of Hkv)          */
    int max_t;        /* largest T of one append or decode call (1..512)           */
    int max_rows;     /* physical rows per sequence.  Flat cache: the logical      */
                      /* capacity.  Ring: 0 selects window + 30 + max_t.           */
    int window;       /* 0: full attention; > 0: each query row sees at most the   */
                      /* last `window` rows up to and including its own row        */
    int ring;         /* 1: SWA ring addressing, physical = row - base (needs      */
                      /* window > 0); 0: flat rows [0, max_rows)                   */
    kvq_fmt k_fmt;    /* KVQ_Q8_0 with v_fmt KVQ_Q5_1, or KVQ_FP8_E4M3 with        */
    kvq_fmt v_fmt;    /* v_fmt KVQ_FP8_E4M3; no other pairs                        */
} kvq_config;

/* Device bytes the caller provides (each buffer 16-byte aligned), and the
 * geometry they hold ("Module cache", fn cache_bytes_per_token and
 * fn swa_ring_rows):
 *   k_plane   [n_seq][rows][k_row_bytes], k_row_bytes = kb*34,
 *             kb = n_kv_heads*head_dim/32, plus 128 bytes of padding (the
 *             generic decode's tile copies may pass the last row), rounded up
 *             to a multiple of 256 bytes
 *   v_plane   [n_seq][rows][v_row_bytes], v_row_bytes = kb*24 (padded and
 *             rounded likewise).  With FP8 E4M3 both rows are kb*32 bytes.
 *   counters  len_d[n_seq], base_d[n_seq], error word, the append's
 *             completion counter, the ring rebase's barrier words (int32)
 *   workspace decode partials, the split plan and the ring-rebase scratch
 *   rows      physical rows per sequence: max_rows for a flat cache, and for
 *             a ring max_rows or, when it is 0, window + 30 + max_t        */
typedef struct kvq_sizes {
    size_t k_plane, v_plane, counters, workspace;
    int rows, k_row_bytes, v_row_bytes;
} kvq_sizes;

typedef struct kvq_cache kvq_cache;

/* Sizes of the four device buffers for a configuration and the rows they
 * hold (fn new of "Struct Cache" allocates by geometry and maximum context;
 * the byte counts per row are fn cache_bytes_per_token's for one layer).
 * Pure host call: KVQ_EINVAL / KVQ_EUNSUPPORTED for a bad configuration. */
kvq_status kvq_required_bytes(const kvq_config* cfg, kvq_sizes* out);

/* Build a cache over caller buffers (fn new of "Struct Cache").  Validates the
 * geometry (head_dim % 32 == 0, formats q8_0/q5_1 or e4m3/e4m3, ring needs
 * window > 0),
 * checks 16-byte alignment, and enqueues on `stream` the zeroing of the
 * counters (len = 0, base = 0, error = 0).  Byte planes are not cleared:
 * rows at or beyond a sequence's length are never read.  `*out` receives a
 * host handle to release with kvq_free.  stream: a cudaStream_t or NULL. */
kvq_status kvq_alloc(const kvq_config* cfg, void* k_plane, void* v_plane,
                     void* counters, void* workspace, void* stream,
                     kvq_cache** out);

/* Release the host handle (device buffers stay the caller's).  NULL is a
 * no-op.  No passage: the pages' cache owns its memory, this one only a
 * host handle. */
void kvq_free(kvq_cache* cache);

/* Quantised append ("Struct KvLayer": append_kv_quantized_dc[w] writes at the
 * slot len_d, inc_seqlen then adds T).  k, v: device [n][T][Hkv][D] of dtype
 * (f32 or bf16), n = n_ids, or n_seq when seq_ids is NULL.  Row t of entry i
 * is quantised into row len+t of sequence seq_ids[i] (or i).  seq_ids is a
 * HOST array of distinct indices; n_ids <= n_seq.  Flat caches return
 * KVQ_ERANGE when len + T > max_rows.  Ring caches first rebase a sequence
 * whose live rows would overflow the ring: logical rows [new_base, len) with
 * new_base = max(0, len + 1 - window) rounded down to a multiple of 32 move to
 * physical row 0 and base becomes new_base (fn swa_ring_rows: at most 31
 * masked rows precede the live window).  The move is one cooperative launch
 * through shared memory when the rows are 16-byte multiples and the live
 * bytes fit the SMs' shared memory, else two copies through the workspace.
 * Host lengths advance by T. */
kvq_status kvq_append(kvq_cache* cache, const void* k, const void* v,
                      kvq_dtype dtype, int T, const int* seq_ids, int n_ids,
                      void* stream);

/* Decode attention over the quantised rows ("Struct LayerKvCache",
 * fn attend_group_upto).  q: device [n_seq][T][n_q_heads][D] (f32 or bf16);
 * its T rows are the last T rows appended to each sequence: row t sits at
 * position s0 + t, s0 = len - T, and sees logical rows [lstart_t, s0 + t + 1)
 * with lstart_t = max(0, s0 + t + 1 - window) when window > 0, else 0.
 * Head h reads KV group h / (n_q_heads / Hkv).  Scores are scale * <q, k_hat>
 * (scale <= 0 selects 1/sqrt(D)); sinks (device [n_q_heads] f32, or NULL) are
 * unscaled logits joining the max and the denominator with no value.
 * out: device f32 [n_seq][T][n_q_heads][D].  Every sequence needs len >= T.
 * Two launches: a split kernel writes partial softmax records (running max,
 * denominator, unnormalised output) and a merge kernel combines them with the
 * sinks.  The split kernel is the stream-K kernel (its CTAs, at most one per
 * SM, each take an equal share of all sequences' visible rows in 32-row
 * tiles) or the generic kernel over (sequence, row chunk) work items; see
 * kvq_set_decode_path. */
kvq_status kvq_decode(kvq_cache* cache, const void* q, kvq_dtype dtype, int T,
                      int n_q_heads, const float* sinks, float scale,
                      float* out, void* stream);

/* Bytes of the no-alloc decode scratch (a fixed device array in the library). */
#define KVQ_NOALLOC_SCRATCH_BYTES (16u << 20)

/* kvq_decode without the cache's workspace: the described design has no
 * counterpart of this call; it lets a caller decode without providing
 * partial-result memory.  Same arguments, semantics and results as
 * kvq_decode (the same kernels run on the same split plan), but the split
 * partials and the plan live in a file-scope device array of
 * KVQ_NOALLOC_SCRATCH_BYTES (16 MiB) inside the library: the call allocates
 * nothing.  The decode needs R records of (head_dim + 2) * 4 bytes.  On the
 * stream-K kernel R = (G + nqs * n_seq) * 4 * Hkv * QPS, where G <= 256 is
 * the CTA count (one per SM at most), u = ceil(hpk * T / 4) four-query units per KV head (hpk =
 * n_q_heads / Hkv), QPS = max(1, min(u, 16 / Hkv)) and nqs = ceil(u / QPS):
 * 64 sequences with 8 KV heads, 32 Q heads and T = 1 need about 3.6 MB on 152
 * SMs.  On the generic kernel R = n_seq * ceil(max visible rows / split rows)
 * * n_q_heads * T, plus a plan of n_seq + 1 ints.  A call that needs more
 * returns KVQ_ERANGE (nothing launched) and says how much.  Nothing in the
 * array has to start at zero: every byte read was written earlier in the
 * same call.  The array's address is resolved (cudaGetSymbolAddress, with the
 * device current) on the first call on a device and again whenever the
 * calling thread's current CUDA context differs from the one it was resolved
 * in: make the first call in each context before any stream capture.  All
 * calls share the one array per device, so two calls whose
 * kernels may overlap (other streams, other threads, other caches) race:
 * order them on one stream or synchronise between them. */
kvq_status kvq_decode_noalloc(kvq_cache* cache, const void* q, kvq_dtype dtype, int T,
                              int n_q_heads, const float* sinks, float scale,
                              float* out, void* stream);

/* Rollback ("Struct Cache", fn rollback, item C.1): set each sequence's
 * length to new_len[b] (a HOST array of n_seq values, usually
 * snapshot_len + accept_len), no data moves.  Needs new_len[b] <= len (the
 * lower end while a kvq_truncate_device is pending); a ring
 * sequence also needs max(0, new_len + 1 - window) >= base (rewinds never
 * move the base), else KVQ_ERANGE. */
kvq_status kvq_truncate(kvq_cache* cache, const int* new_len, void* stream);

/* Rollback with the accepted counts on the device ("Struct Cache", fn
 * rollback, item C.1, len = snapshot_len + accept_len, with snapshot_len =
 * len - T for the T draft rows just appended and verified; "Struct KvLayer",
 * field base_d: rewinds move len_d only).  accept_d: DEVICE int32 [n_seq],
 * read when the kernel runs, so a captured graph replays with whatever it
 * holds then.  For each sequence, len_d -= T - accept_d[b]: the first
 * accept_d[b] of the last T rows stay.  The kernel checks 0 <= accept <= T,
 * T <= len_d and, for a ring, max(0, new_len + 1 - window) >= base; a
 * sequence that fails keeps its length and the device error word becomes 1.
 * The host does not wait, so its mirror then knows each length only within
 * [len - T, len]: appends check capacity against the upper end, a ring
 * append that would rebase returns KVQ_ERANGE, decodes need T <= the lower
 * end, and kvq_truncate takes only new_len <= the lower end (which makes the
 * length exact again), until kvq_sync_len reads the lengths back.  The host
 * refuses (KVQ_ERANGE, nothing enqueued) when a sequence may hold fewer than
 * T rows or, for a ring, when accepting nothing would drop rows below base.
 * After replaying a graph that contains this call, call kvq_sync_len before
 * any other call on the cache (kvq_note_replayed cannot know the counts). */
kvq_status kvq_truncate_device(kvq_cache* cache, const int* accept_d, int T, void* stream);

/* Verification of drafted tokens: the accepted counts that
 * kvq_truncate_device takes, and each sequence's next token, from the
 * probabilities of a T-row step (the last token, then up to T - 1 drafts) and
 * random numbers of the caller's.  No passage: the pages take accepted counts
 * as given ("Struct Cache", fn rollback, item C.1).
 *
 * target: device [n_seq][T][vocab] of dtype (f32 or bf16): row t is the
 * target's distribution behind row t of the step.  draft: device
 * [n_seq][T - 1][vocab] of the same type: row t is what tokens[t] was drawn
 * from; NULL: the drafts were not drawn (each has probability 1).  Sequences
 * and rows lie target_seq / target_row (draft_seq / draft_row) elements apart,
 * any number >= 0, a row's elements side by side.  tokens: device int32
 * [n_seq][T - 1]; one outside [0, vocab) is no draft: the sequence's drafts end
 * there (its step may hold fewer than T - 1).  uniform: device f32 [n_seq][T] in [0, 1).
 * A probability that is not above 0 (NaN too) counts as 0, one above 1 as 1, in
 * the test of a draft as in the draw.
 *
 * Draft t stands while uniform[t] * q_t(tokens[t]) < p_t(tokens[t]) (the exact
 * products) and all before it stand.  With a the number that do:
 *   accept[b] = a + 1: the rows of the step that stay;
 *   next[b]: drawn from row a of target.  Weights are max(P_i - Q_i, 0) where
 *     draft a fell (P_i itself where those are all 0), else P_i, with P, Q the
 *     probabilities in whole units of 2^-52, rounded down.  The token is the
 *     first whose running sum passes floor(S * floor(uniform[T-1] * 2^31) /
 *     2^31), S the weights' sum: whole numbers throughout, the same token on
 *     every run.  -1 where all weights are 0.  (A row's probabilities sum to
 *     less than 4096, or the token is any, or -1.)
 *   lens[b] -= T - accept[b], where lens (device int32 [n_seq], or NULL) counts
 *     the step's rows, as a paged cache's lengths do.
 * One kernel; nothing is read of a row that is not needed.  T in [1, 512] (T =
 * 1: a draw from row 0), vocab up to 2^24, n_seq up to 65536. */
typedef struct kvq_verify_args {
    const void* target;
    const void* draft;
    const int* tokens;
    const float* uniform;
    kvq_dtype dtype;
    int n_seq, T, vocab;
    long long target_seq, target_row, draft_seq, draft_row;
    int* accept;          /* device int32 [n_seq]                            */
    int* next;            /* device int32 [n_seq]                            */
    int* lens;            /* device int32 [n_seq], read and written, or NULL */
} kvq_verify_args;
kvq_status kvq_verify(const kvq_verify_args* a, void* stream);

/* Synchronise `stream` and read the device lengths into the host mirror,
 * making it exact (after kvq_truncate_device).  KVQ_ERANGE if a device length
 * lies outside its sequence's resident rows (the mirror is then unchanged). */
kvq_status kvq_sync_len(kvq_cache* cache, void* stream);

/* Host mirror of the lengths and ring bases (HOST arrays of n_seq ints;
 * either pointer may be NULL): the host side of the len_d / base_d pair of
 * "Struct KvLayer".  After kvq_truncate_device and before kvq_sync_len the
 * lengths are upper bounds. */
kvq_status kvq_get_len(const kvq_cache* cache, int* len_host, int* base_host);

/* Advance the host mirror after `steps` replays of a captured graph that
 * appended T rows to every sequence per step. */
kvq_status kvq_note_replayed(kvq_cache* cache, int steps, int T);

/* Appends of T rows (to every sequence) that can run before a ring rebase is
 * due, i.e. how many steps a captured graph may replay. Flat caches: rows
 * left before max_rows, divided by T.  While a kvq_truncate_device is
 * pending it counts from the upper ends of the lengths (a safe undercount). */
kvq_status kvq_ring_headroom(const kvq_cache* cache, int T, int* steps);

/* fn physical_rows of "Struct KvLayer": map logical rows [start, end) of
 * sequence seq to physical rows; KVQ_ERANGE if any row is not resident. */
kvq_status kvq_physical_rows(const kvq_cache* cache, int seq, int start,
                             int end, int* phys_start, int* phys_end);

/* Synchronise `stream`, read the device error word into *err (0 = none;
 * 1 = a kernel saw a length or base out of range; 2 = a bounded wait ran
 * out) and clear it. */
kvq_status kvq_read_device_error(kvq_cache* cache, int* err, void* stream);

/* Choose the decode kernel: path 0 = automatic (the stream-K kernel whenever
 * it allows the cache and the call, else the generic split kernel),
 * 1 = generic, 2 = stream-K (KVQ_EUNSUPPORTED at decode time if it does not
 * allow them).  The stream-K kernel needs K and V token rows that are
 * 16-byte multiples (q8_0/q5_1: n_kv_heads * head_dim a multiple of 256;
 * E4M3: of 16) and at most 2048 bytes, head_dim 64, 128 or 256,
 * n_kv_heads <= 16, n_seq <= 1024 and its tiles within shared memory.
 * query_bits (0 = 16, or 16, or 24): on q8_0 K the stream-K kernel quantises
 * each pre-scaled query element per 32-element block to this many bits
 * against the block's largest magnitude and multiplies it with the int8 K
 * codes in integer dot products; 16 bits adds an error below 1e-4 to the
 * attention output on unit-variance data, 24 bits is at the level of fp32
 * rounding and costs half again as many dot products.  With E4M3 K the
 * queries stay f32 and query_bits does not apply. */
kvq_status kvq_set_decode_path(kvq_cache* cache, int path, int query_bits);

/* Score soft-capping for later decodes ("Struct LayerKvCache": the softcap
 * argument of fn attend_group / attend_group_upto, which the pages name
 * without defining; read as the usual logit soft-capping).  softcap > 0 maps
 * every scaled score s = scale * <q, k_hat> to softcap * tanh(s / softcap)
 * before the softmax; sink logits are not capped.  0 (the default) turns it
 * off.  Both decode kernels apply it.  KVQ_EINVAL for a negative or
 * non-finite value. */
kvq_status kvq_set_softcap(kvq_cache* cache, float softcap);

/* Row slices per 32-row tile on the stream-K kernel: 0 = automatic (two,
 * one warp per half tile, when 2 x (KV heads x four-query groups of a slice)
 * <= 16 and the CTAs have more than 16 tiles each; else one), 1, or 2 (taken
 * only where the geometry allows two; else one).  Results are the same up to
 * fp32 rounding; the choice moves speed only.  No passage: a tuning knob of
 * this implementation.  KVQ_EINVAL for another value. */
kvq_status kvq_set_row_slices(kvq_cache* cache, int slices);

/* Override the generic kernel's split size in rows (a multiple of 8, >= 64;
 * 0 = auto).  The stream-K kernel ignores it: its CTAs split the rows
 * evenly. */
kvq_status kvq_set_split_rows(kvq_cache* cache, int rows);

/* ------------------------------------------------------------------------
 * Paged cache.  No passage: the pages describe rows of one sequence side by
 * side; these calls hold the same block formats in pages that tables share
 * out, for a server whose sequences grow, share prefixes and come and go.
 *
 * The caller owns the page pool, the tables and the lengths.  A sequence is a
 * row of page numbers (its table) and a length; logical row r lies in page
 * table[r / page_rows].  Tables (int32 [n_seq][max_pages]), lengths (int32
 * [n_seq]) and every other index array are DEVICE arrays, read when the
 * kernels run, so a captured graph follows what they then hold.  A length
 * counts the rows including those the call itself appends or whose queries it
 * takes: an append of T rows writes logical rows [len - T, len), and the T
 * query rows of a decode sit at positions len - T .. len - 1.  Rollback is a
 * smaller length.  Nothing but the named rows is written.
 *
 * Layout.  Pool: [n_pages][n_kv_heads][page_rows / 16] cells; a cell holds 16
 * rows of one KV head in the order in which tensor-core fragments take them.
 * NB = head_dim / 32; row t of a cell: h = t / 8, j = (t % 8) / 2, s = t % 2;
 * element e: b = e / 32, g = (e % 32) / 4, r = e % 4, c = (e % 32) / 8;
 * n = h * NB + b, lane = 4 g + j.  Byte offsets in a cell:
 *   K code      (b/2)*1024 + t*64 + c*16 + (b%2)*8 + e%8
 *               (q8_0: the int8 code + 128; E4M3: the byte)
 *   q8_0 d      512 NB + (j*NB + b)*8 + (2h + s)*2                     fp16
 *   q5_1 codes  u16 at 544 NB + (n/4)*512 + lane*16 + (n%4)*4 + s*2: bits
 *               5r..5r+4 the code of r = 0, 1, 2, bit 15 bit 4 of r = 3; bits
 *               0..3 of r = 3 in nibble n%2 of byte
 *               800 NB + (n/4)*128 + lane*4 + s*2 + (n%4)/2
 *   q5_1 d, m   864 NB + (j*NB + b)*16 + (2h + s)*2, and + 8           fp16
 *   E4M3 V      512 NB + (n/2)*512 + lane*16 + (n%2)*8 + r*2 + s
 * A cell is 928 NB bytes (58 per 32 elements, as in the flat cache) or 1024 NB.
 *
 * Errors.  A page number outside the pool, a length below 0 or above max_pages *
 * page_rows, or one below the rows that an append brings (an entry that only
 * pads a batch is given none, by `starts`) sets the device error word to 1:
 * appends skip the row, decodes take a bad page's rows as masked and a bad
 * sequence as empty.  Rows that a length counts and no append wrote may be any
 * bytes: outputs of the queries that see them are undefined, unless they were
 * filled in another way with finite scales and values.  A query row
 * that sees no row (a sequence of length 0, a position below 0) gives zeros,
 * with or without a sink; one that is not finite, or whose score of a row is
 * above f32's range, gives NaN where it sees a row, and leaves all others as they
 * are (a score below f32's range is one of no weight).  Calls on one cache share its workspace: order them
 * on one stream (captured graphs that share a cache included).  A workspace
 * belongs to one cache: its counters are zero between that cache's calls. */
typedef struct kvq_paged_config {
    int n_pages;         /* pages in the pool                                     */
    int page_rows;       /* rows per page: 16, 32, 64, 128 or 256                 */
    int n_kv_heads;      /* Hkv: 1..128                                           */
    int head_dim;        /* D: 64, 128 or 256                                     */
    int max_q_heads;     /* largest Hq (a multiple of Hkv, at most 128 x Hkv)     */
    int max_seqs;        /* most sequences one call takes (1..1024)               */
    int max_pages;       /* entries of a sequence's table; max_pages * page_rows  */
                         /* at most 2^24                                          */
    int max_t;           /* largest T of a decode (1..64); appends have no limit  */
    kvq_fmt k_fmt;       /* KVQ_Q8_0 with KVQ_Q5_1, or KVQ_FP8_E4M3 twice         */
    kvq_fmt v_fmt;
    int bounds;          /* 1: appends keep key bounds per page (kvq_paged_select) */
    int rope_dim;        /* leading elements of a head that the append rotates: 0 */
                         /* or a multiple of 16 up to head_dim                    */
    int rope_interleaved;/* 0: pairs (i, i + rope_dim/2); 1: pairs (2i, 2i+1)     */
    double rope_base;    /* angle of pair i at position p: p * base^(-2i/rope_dim) */
} kvq_paged_config;

/* Device bytes the caller provides (each 16-byte aligned): pool, bounds (0
 * without cfg.bounds), workspace (the error word, decode partials, 8 bytes a
 * sequence, row and query head for kvq_paged_decode_scored, page scores).  Pool bytes need no initial value. */
typedef struct kvq_paged_sizes {
    size_t pool, bounds, workspace;
    size_t page_bytes, cell_bytes;
} kvq_paged_sizes;

typedef struct kvq_paged kvq_paged;

kvq_status kvq_paged_required_bytes(const kvq_paged_config* cfg, kvq_paged_sizes* out);

/* Build a paged cache over caller buffers and enqueue on `stream` the clearing
 * of the workspace's error word and counters.  rope_freq: HOST array of rope_dim / 2
 * radians per position that replaces base^(-2i/rope_dim) (scaled or stretched
 * rotations), or NULL; copied.  bounds may be NULL without cfg.bounds. */
kvq_status kvq_paged_alloc(const kvq_paged_config* cfg, void* pool, void* bounds, void* workspace,
                           const double* rope_freq, void* stream, kvq_paged** out);
void kvq_paged_free(kvq_paged* cache);

/* Append with the rotation applied on the way.  k, v: device [rows][Hkv][D]
 * of dtype, consecutive rows k_stride / v_stride elements apart (a multiple of
 * 8; Hkv * D when dense; a fused projection's slices are taken as they lie).
 * Without `starts` entry i of n has T rows, rows = n * T.  With `starts`
 * (device int32 [n + 1], non-decreasing) entry i has rows starts[i] ..
 * starts[i+1] - 1 of the `rows` there are; rows outside [starts[0], starts[n])
 * are neither read nor written.  Keys are rotated by their position in fp32
 * (angles kept to 2^-24 of a turn) and quantised from fp32; values only
 * quantised.  q (or NULL): device [rows][Hq][D] of dtype, q_stride apart,
 * rotated likewise into q_out, dense [rows][Hq][D]; q_out may be q when q is
 * dense.  With cfg.bounds the bounds of the pages that got rows are renewed
 * from all rows below the length.  A page that gets rows belongs to one entry.
 * Stored rows are finite: a q8_0 key stays within +-8319008 (127 x 65504), a
 * q5_1 block's ends within +-65280, E4M3 within +-448, what lies beyond (an
 * infinity too) is stored as that end.  A NaN is stored as zero, in q5_1 as its
 * block's least value (a block of NaN as zeros). */
kvq_status kvq_paged_append(kvq_paged* cache, const void* k, long long k_stride, const void* v, long long v_stride,
                            const void* q, long long q_stride, void* q_out, int n_q_heads, kvq_dtype dtype,
                            const int* tables, const int* lens, int n_seq, int T, const int* starts, int rows,
                            void* stream);

/* The append with each row's position given instead of its index in the
 * sequence: after an eviction (kvq_paged_compact) a row's index is no longer
 * its position, and rows of pictures and video have a position on each of
 * several axes (time, height, width).  positions: device int32 [rows][n_axes],
 * each in [0, 2^24); pair i of a head turns by positions[row][axis of pair i]
 * times its frequency.  A row with a position outside sets the error word and
 * is skipped, its query too.  Angles are worked out to nearly the last bits of
 * f32 at any position (kvq_paged_append's to 2^-24 of a turn: the two may differ
 * in a code here and there).  Rows are placed, and everything else is done, as by
 * kvq_paged_append.  Needs rope_dim > 0. */
kvq_status kvq_paged_append_at(kvq_paged* cache, const void* k, long long k_stride, const void* v, long long v_stride,
                               const void* q, long long q_stride, void* q_out, int n_q_heads, kvq_dtype dtype,
                               const int* tables, const int* lens, int n_seq, int T, const int* starts, int rows,
                               const int* positions, void* stream);

/* The axis of each rotated pair for later kvq_paged_append_at calls: a HOST
 * array of rope_dim / 2 numbers in [0, n_axes), copied; n_axes in [1, 4].  A
 * cache starts with one axis.  Enqueues nothing. */
kvq_status kvq_paged_set_axes(kvq_paged* cache, const int* axis, int n_axes);

/* Rows back as values: entry i's last T rows (or its rows by `starts`, as in
 * the append) into k_out, v_out, dense [rows][Hkv][D] of dtype, rounded once.
 * A row below 0 or in a bad page gives zeros (the latter sets the error
 * word). */
kvq_status kvq_paged_read(kvq_paged* cache, void* k_out, void* v_out, kvq_dtype dtype, const int* tables,
                          const int* lens, int n_seq, int T, const int* starts, int rows, void* stream);

/* Arguments that the decodes share.  q: device dense [n_seq][T][Hq][D] of
 * dtype; out the same shape and type (bf16 queries give bf16 outputs).  Row t
 * sees logical rows [max(0, p + 1 - window), p + 1), p = len - T + t (window
 * 0: all).  scale <= 0 selects 1/sqrt(D); softcap > 0 caps scaled scores to
 * softcap * tanh(s / softcap) (either, where positive, within 1e-30 .. 1e30);
 * sinks: device f32 [Hq] or NULL, logits (finite, or -inf: none) that join max
 * and denominator without a value.  out may be q. */
typedef struct kvq_paged_query {
    const void* q;
    void* out;
    kvq_dtype dtype;
    int n_seq, T, n_q_heads;
    const int* tables;
    const int* lens;
    const float* sinks;
    float scale, softcap;
    int window;
} kvq_paged_query;

/* Decode attention over the pages.  f32 queries keep f32 accuracy (factors
 * split in two or three parts); bf16 queries round probabilities and values
 * to fp16 inside, and so the keys of a shared prefix, scaled by a power of two
 * for each 32 rows (a key below 2^-28 of the largest of them keeps fewer than
 * fp16's 11 bits); a shared prefix's partial outputs are kept as fp16 scaled by
 * a power of two for each query; sums are f32 throughout. */
kvq_status kvq_paged_decode(kvq_paged* cache, const kvq_paged_query* a, void* stream);

/* The same result for a batch in which groups of sequences share a prefix,
 * whose rows are read once a group instead of once a sequence.  Group i is
 * sequences group_start[i] .. group_start[i+1] - 1 (device int32
 * [n_groups + 1], non-decreasing, inside [0, n_seq]); their first
 * prefix_len[i] rows are the same and are taken from the first member's table
 * (the prefix may end inside a page).  Sequences outside the groups have no
 * shared rows.  n_groups <= n_seq. */
kvq_status kvq_paged_decode_shared(kvq_paged* cache, const kvq_paged_query* a, const int* group_start,
                                   const int* prefix_len, int n_groups, void* stream);

/* Key bounds.  For each page, KV head and 32-element block over the rows below
 * the length: the smallest and largest dequantised key of each element, as
 * codes floor(min / ds) and ceil(max / ds) within +-127 of ds = max|key| *
 * (1/127) (f32 operations; zero codes when ds is 0).  Buffer: int8
 * [n_pages][Hkv][NB][2][32] (min, max), then f32 ds [n_pages][Hkv][NB].  Appends do this themselves; the call
 * is for pages filled in another way: it renews those that hold the last T
 * rows of each entry (or its rows by `starts`). */
kvq_status kvq_paged_bounds(kvq_paged* cache, const int* tables, const int* lens, int n_seq, int T, const int* starts,
                            int rows, void* stream);

/* Choose pages by their bounds.  For each sequence, query row t and KV head:
 * the query is coded per block (dq = amax * (1/127), c = rint(x * ((1/amax) *
 * 127)), f32 operations), and a page scores max over the KV head's queries of
 * sum over blocks, in order, of (dq ds) * sum_i (c_i > 0 ? c_i max_i : c_i min_i), in f32: an upper bound
 * of the coded query's products with the page's keys, and the same on every
 * run.  Pages: device int32 [n_seq][T][Hkv][keep] receives, ascending, the
 * first n_first and last n_last pages of those with a visible row and then the
 * best scored, ties to the lower index, -1 behind the last.  Uses q, dtype,
 * n_seq, T, n_q_heads, tables and lens of `a`.  Needs n_first, n_last >= 0,
 * n_first + n_last <= keep, n_seq * T <= 2048. */
kvq_status kvq_paged_select(kvq_paged* cache, const kvq_paged_query* a, int* pages, int keep, int n_first, int n_last,
                            void* stream);

/* Decode attention over the listed pages only: entries are indexes into the
 * sequence's table as kvq_paged_select gives them; negative ones are skipped,
 * a repeated one counts as often as it stands there.  window must be 0;
 * n_seq * T <= 2048. */
kvq_status kvq_paged_decode_sparse(kvq_paged* cache, const kvq_paged_query* a, const int* pages, int keep,
                                   void* stream);

/* Row scores: an f32 for each row and KV head of the pool, device
 * [n_pages][Hkv][page_rows], 16-byte aligned, kept until the cache is freed or
 * another buffer (or NULL: none) takes its place.  With a buffer set, appends
 * set the scores of the rows they write to 0, kvq_paged_decode_scored adds
 * attention weights and kvq_paged_compact moves scores with their rows.  The
 * contents are the caller's to read or write.  Enqueues nothing. */
kvq_status kvq_paged_set_scores(kvq_paged* cache, float* scores);

/* kvq_paged_decode, and the weights that its queries gave to each row added to
 * the row scores: for every row r below a sequence's length and every KV head,
 *   score = decay * score + sum over the T query rows and the head's queries of
 *           exp(s_r) / (sum over the rows seen of exp(s) + exp(sink)),
 * s the scaled (and capped) score, 0 for rows that a query does not see.
 * decay in [0, 1]; 0 does not read the old scores.  A query that is not finite
 * (its output is NaN) adds nothing.  Sums are f32 in a fixed order: two runs
 * give the same bits.  The pages of one call's sequences are their own: a page
 * in two tables of the call is written by both.  Rows of bad pages are left
 * out.  out must not overlap q.  Needs a buffer (kvq_paged_set_scores).
 * All T rows' queries count when the call runs: the weights of drafts that a
 * verification lets fall afterwards stay in the scores of the rows they saw. */
kvq_status kvq_paged_decode_scored(kvq_paged* cache, const kvq_paged_query* a, float decay, void* stream);

/* Room for a scored decode's scores: device f32 [n_pages][Hkv][page_rows][queries],
 * 16-byte aligned, queries in [1, 8], kept until another (or NULL: none) takes its
 * place.  With it, calls of at most `queries` queries a KV head (n_q_heads / Hkv * T)
 * whose scores, 8 bytes a row and query written and read, are fewer than the keys'
 * bytes keep them in the first pass, where the second pass else works them out
 * again from the keys: the same weights, and the less extra time the fewer the
 * queries (of 1 a third of it, of 8 of head_dim 64 all of it).  What it holds
 * lives within a call: caches with as many rows of all KV heads, whose calls are in one
 * stream's order, may have one together.  Enqueues nothing. */
kvq_status kvq_paged_set_score_scratch(kvq_paged* cache, float* scratch, int queries);

/* Choose the rows that stay.  rows: device int32 [n_seq][Hkv][keep] receives for
 * each sequence and KV head, ascending, the first n_first and last n_last rows
 * below the length and the best scored of the others, ties to the lower index
 * (a NaN score is the lowest); all rows where the length is at most keep; -1
 * behind the last.  Each KV head chooses for itself.  Needs n_first, n_last >= 0 and n_first + n_last
 * <= keep, keep in [1, 2^24], and a score buffer.  A bad length or page sets the
 * error word: no rows of that sequence, a score below all others for rows of that page. */
kvq_status kvq_paged_select_rows(kvq_paged* cache, const int* tables, const int* lens, int n_seq, int keep,
                                 int n_first, int n_last, int* rows, void* stream);

/* Move the listed rows together: entry i of rows[b][h] (int32 [n_seq][Hkv][keep]
 * as kvq_paged_select_rows gives them: the first min(lens[b], keep) entries are
 * rows of the sequence, strictly ascending) becomes row i of KV head h, bit for
 * bit, with its score where a buffer is set; with cfg.bounds the pages' key
 * bounds are renewed.  lens_out[b] = min(lens[b], keep) (lens_out may be lens).
 * The keys stay turned by the positions they were appended with: append the
 * next rows with kvq_paged_append_at.  (Of a bad length lens_out is that length.)
 *   tables_out NULL: in place, into the sequence's own pages; what lies behind
 *     the new length is then free.  A page belongs to one sequence.
 *   tables_out (device int32 [n_seq][max_pages]): into other pages (of a sequence that
 *     shares its first pages with others, say), none of which is in `tables`.
 * Of a sequence in error (a bad length, an entry out of range or order, a bad
 * page) the rows concerned are not moved and the error word is set; the others
 * are. */
kvq_status kvq_paged_compact(kvq_paged* cache, const int* tables, const int* lens, int n_seq, const int* rows,
                             int keep, const int* tables_out, int* lens_out, void* stream);

/* Synchronise `stream`, read the device error word into *err (0 = none, 1 = a
 * page number or length out of range, 2 = a bounded wait ran out), clear it. */
kvq_status kvq_paged_read_error(kvq_paged* cache, int* err, void* stream);

/* Bytes per 32-element block of a format: 34 (q8_0), 24 (q5_1) or 32
 * (FP8 E4M3); -1 if unknown ("Module cache", fn kv_blk_bytes). */
int kvq_block_bytes(kvq_fmt fmt);

/* Context-linear bytes one token occupies in this layer cache, K plus V
 * ("Module cache", fn cache_bytes_per_token, for a single layer); 0 on bad
 * input. */
size_t kvq_bytes_per_token(const kvq_config* cfg);

/* Message of the last failed call on this thread ("" if none).  No passage:
 * error reporting of this C interface. */
const char* kvq_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* KVQ_H */
