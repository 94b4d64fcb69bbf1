/*
 * libgradcomp — per-step gradient compression for data-parallel training on
 * AMD Instinct MI355X (gfx950).
 *
 * The operations follow these pages:
 *   [AdaComp] "AdaComp: Adaptive Residual Gradient Compression for
 *             Data-Parallel Distributed Training" (Chen et al.), the review's
 *             "Proposed method" list and Abstract.
 *   [DGC]     "Deep Gradient Compression: Reducing the Communication Bandwidth
 *             for Distributed Training" (Lin et al.), §3.1–§3.3, §5, §6 and
 *             Appendices A–D.
 *   [DCD]     "Communication Compression for Decentralized Training"
 *             (Tang et al.), DCD-PSGD steps 1–3, the signal-to-noise
 *             parameter alpha of the compression operator, and ECD-PSGD's
 *             extrapolation and estimate (Eqs. 3 and 4).
 *   [SlimDP]  "Slim-DP: A Light Communication Data Parallelism for DNN",
 *             §3 (core and explorer selection, significance, key caching)
 *             and the experimental setup (Quant-DP baseline: random
 *             quantization with buckets of 512).
 *   The embedding's lookup and gradient and the orthogonalised matrix update
 *   (Newton-Schulz products, as the Muon optimiser applies them), the layers'
 *   products, the top logits and the distillation loss come from no page: they
 *   are given by their formulas at each call.
 *
 * Conventions shared by every call
 * --------------------------------
 *  - Every buffer argument typed as a pointer to float / uint32_t / uint8_t /
 *    uint64_t / void is a DEVICE pointer owned by the caller.  Structs and
 *    arrays documented as "host" are read during the call and not retained.
 *  - A learner's model is one flat fp32 buffer of n_total elements.  Each
 *    layer tensor is a segment of it (gc_segment).  State buffers (AdaComp
 *    residual R, DGC momentum U and accumulator V) use the same flat layout.
 *  - Argument errors are detected on the host before anything is enqueued; on
 *    error no device buffer has been touched.  Errors are returned as negative
 *    gc_status codes; gc_last_error() gives a thread-local message.
 *  - Hot calls enqueue kernels on `stream` and return without synchronising.
 *    Counts and messages land in device memory.
 *  - Hot calls never allocate device memory, with one exception: the first
 *    call that uses a plan on a device uploads the plan's tables to that
 *    device (one hipMalloc + one synchronous copy per plan and device).
 *  - Results are bitwise deterministic: every floating-point operation is a
 *    single correctly rounded IEEE operation in a fixed order (no FMA
 *    contraction), and every reduction that feeds a decision uses a fixed
 *    pairwise tree (see gc_dgc_step and gc_adacomp_compress).
 *  - Non-finite inputs have defined results.  A NaN never counts toward a
 *    maximum (an AdaComp bin's, a DCD bucket's), is never selected by
 *    AdaComp (it stays in the residual) and quantizes to level 0 in DCD.
 *    +-Inf are magnitudes above every finite one: an Inf is its bin's
 *    maximum, and a DCD bucket whose maximum is Inf sends only level 0.  DGC
 *    ranks by the magnitude bits, where a NaN ranks above +Inf.  Every other
 *    step is the IEEE operation as written; NaNs that arithmetic makes carry
 *    no guaranteed sign or payload.
 *  - Input, state and output buffers must not alias each other (except
 *    x_out == x in gc_dcd_compress).
 *  - Calls on different streams are independent as long as they use
 *    different workspaces and outputs.
 */
#ifndef GRADCOMP_H
#define GRADCOMP_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------ status */
typedef int gc_status;
#define GC_OK          0
#define GC_EINVAL     -1   /* malformed argument (null pointer, bad range)   */
#define GC_ECAPACITY  -2   /* output or workspace capacity too small         */
#define GC_ERANGE     -3   /* size outside the supported range (n >= 2^32)   */
#define GC_EHIP       -4   /* a HIP runtime call failed                      */
#define GC_ENOTSUP    -5   /* valid but unsupported parameter combination    */

/* Thread-local text of the last error raised on this thread ("" if none). */
const char *gc_last_error(void);
/* Library version string, e.g. "libgradcomp 0.1.0". */
const char *gc_version(void);

/* ------------------------------------------------------------------ layout */
/*
 * One layer tensor inside the flat buffer (host struct).
 * Both methods act on each layer on its own: [AdaComp] applies the scheme
 * layer by layer; [DGC] §3.1 thresholds each gradient tensor.
 *   offset  : index of the segment's first element in the flat buffer.
 *   length  : number of elements n_s (>= 1).
 *   bin_len : AdaComp bin length L_T (>= 1, <= GC_MAX_BIN_LEN); bins restart
 *             at the segment start and the last bin may be partial.
 *   k       : DGC top-k count (1 <= k <= length).  gc_topk_count() gives the
 *             0.1%-density value ceil(n_s/1000) used by [DGC] §3.3/§4.
 */
typedef struct gc_segment {
    uint64_t offset;
    uint32_t length;
    uint32_t bin_len;
    uint32_t k;
    uint32_t reserved;   /* must be 0 */
} gc_segment;

#define GC_MAX_BIN_LEN   4096u
#define GC_MAX_MESSAGES  64
/* Longest segment, 2^32 - 2^18: a packed block of n_s elements holds up to
 * n_s + n_s / 32767 + 1 codes (an AdaComp message that sends every element,
 * plus its escapes), and that count travels as the block's u32 E. */
#define GC_MAX_SEGMENT_LEN 0xFFFC0000u

/* Opaque, immutable plan: validated segment table + device tables. */
typedef struct gc_plan gc_plan;

/*
 * Validate a segment table and build a plan.  Host only: touches no device.
 *   segs[nseg] (host) must be ascending by offset, non-overlapping, and lie in
 *   [0, n_total); n_total must be < 2^32 (indices are u32).  Gaps between
 *   segments are allowed and are never read or written.
 * Returns GC_EINVAL (bad table), GC_ERANGE (n_total >= 2^32), GC_ENOTSUP
 * (bin_len > GC_MAX_BIN_LEN or length > GC_MAX_SEGMENT_LEN).  *out is set
 * only on GC_OK.
 */
gc_status gc_plan_create(const gc_segment *segs, int nseg, uint64_t n_total,
                         gc_plan **out);
void      gc_plan_destroy(gc_plan *plan);
/* Put the plan's tables on the current device now: one hipMalloc and one
 * synchronous copy, once per plan and device (a hot call does the same on
 * its first use there).  For callers that capture a plan's first calls in a
 * HIP graph, or allocate nothing inside their hot loop.  Returns GC_OK once
 * the tables are there, GC_EINVAL for a NULL plan, GC_EHIP on a HIP error. */
gc_status gc_plan_upload(const gc_plan *plan);
int       gc_plan_num_segments(const gc_plan *plan);
uint64_t  gc_plan_num_elements(const gc_plan *plan);
/* Sum over segments of k (the DGC message size). */
uint64_t  gc_plan_total_k(const gc_plan *plan);
/* Sum over segments of ceil(length/bin_len) (AdaComp bin count). */
uint64_t  gc_plan_total_bins(const gc_plan *plan);
/* ceil(n / 1000), the per-tensor count at 99.9% sparsity. */
uint32_t  gc_topk_count(uint32_t n);

#define GC_OP_DGC      1
#define GC_OP_ADACOMP  2
#define GC_OP_PACK     3
#define GC_OP_DECODE   4
#define GC_OP_UNPACK   5
/* Device workspace bytes a hot call with this plan needs (0 if none). */
size_t gc_plan_workspace_bytes(const gc_plan *plan, int op);

/* ----------------------------------------------------------------- message */
/*
 * Sparse message (host struct whose members are device pointers).
 *   idx[cap]        : flat element indices, ascending within the message
 *                     (segments in plan order, ascending inside a segment).
 *   val[cap]        : value to add at idx — V_i for DGC, +-scale_s for AdaComp.
 *   seg_off[nseg+1] : entries of segment s are [seg_off[s], seg_off[s+1]);
 *                     seg_off[nseg] is the message's entry count.
 *   seg_scale[nseg] : AdaComp layer scale per segment (unused by DGC; may be
 *                     NULL there).
 *   cap             : capacity of idx/val in entries.
 */
typedef struct gc_sparse {
    uint32_t *idx;
    float    *val;
    uint32_t *seg_off;
    float    *seg_scale;
    uint64_t  cap;
} gc_sparse;

/* --------------------------------------------------------------- AdaComp */
/*
 * One AdaComp step for one learner ([AdaComp] "Proposed method", Abstract):
 *   a1  G_i = fl32(R_i + dW_i)                                (residual + new gradient)
 *   a2  g_max(b) = max_{i in b} |G_i|   over bins of bin_len  (exact; max is order-free)
 *   a3  sel_i  <=>  g_max(b) > 0  and  fl32(scale_factor * |G_i|) >= g_max(b)
 *       (the bin's own max always qualifies when scale_factor >= 1; 2.0 is the
 *        empirical factor the page gives)
 *   a4  scale_s = fl32( PSUM64(g_max over the segment's bins) / nbins_s )
 *       (mean of the bin maxima across the whole layer)
 *   a5  q_i = copysign(scale_s, G_i) if selected, else 0;  R_i <- fl32(G_i - q_i)
 *   a6  out: per segment, ascending idx with val = q_i; out->seg_scale[s] = scale_s.
 * PSUM64(x_0..x_{m-1}) converts each term to double, pads with +0.0 to the
 * next power of two and adds as a perfect binary tree in index order.
 *
 * Residual storage.  A learner's residual is the pair (R, state):
 *   state == NULL : R holds the exact residual before and after the call.
 *   state != NULL : deferred mode.  `state` is a caller-owned, 256-byte
 *     aligned device buffer of at least gc_adacomp_state_bytes(plan) bytes,
 *     zero-filled before the learner's first step and used with this plan
 *     only.  After a call, R holds G and the state records which entries the
 *     call sent and the layer scales; the residual of such an entry is
 *     fl32(R_i - copysign(scale_s, R_i)) (step a5, exactly), which the next
 *     call applies before a1.  R and dW then cross HBM once per step instead
 *     of twice.  Messages are identical in both modes; gc_adacomp_residual()
 *     gives the exact residual of (R, state).
 *   dW  [n_total] in,  R [n_total] in/out,
 *   out : cap >= gc_adacomp_message_cap(plan), the sum of the segment
 *         lengths (the worst case: every element sent).
 *   ws  : at least gc_plan_workspace_bytes(plan, GC_OP_ADACOMP) bytes.
 * Errors: GC_EINVAL (null pointer, scale_factor not finite or < 1, state
 *         not 256-byte aligned), GC_ECAPACITY (out->cap below
 *         gc_adacomp_message_cap, ws or state too small).
 */
gc_status gc_adacomp_compress(const gc_plan *plan, const float *dW, float *R, void *state,
                              size_t state_bytes, float scale_factor, gc_sparse *out,
                              void *ws, size_t ws_bytes, hipStream_t stream);

/*
 * The same step with the reading of the adaptive threshold chosen.  The
 * AdaComp page ("Proposed method") builds the threshold from a scale factor
 * (empirically 2x) that picks entries near the bin's max, without fixing what
 * the factor multiplies; both readings are offered, and neither is pinned by
 * the page:
 *   GC_ADACOMP_RULE_RESIDUAL (gc_adacomp_compress): step a3 above;
 *   GC_ADACOMP_RULE_GRADIENT: the factor weighs the new gradient instead,
 *     a3' H_i = fl32(G_i + fl32((scale_factor - 1) * dW_i))
 *              (for the factor 2, fl32(G_i + dW_i), i.e. R + 2 dW rounded
 *               from G)
 *         sel_i <=> g_max(b) > 0 and (|H_i| >= g_max(b) or |G_i| = g_max(b))
 *         (every entry at the bin's max is sent, as under the default).
 *   Steps a1, a2, a4-a6 and both residual modes are unchanged; an entry with
 *   G_i = +-0 that H sends gets copysign(scale_s, G_i).
 * opt: scale_factor finite and >= 1; rule one of the two; reserved zero.
 * Arguments, layouts and the other errors as gc_adacomp_compress.
 * Errors: GC_EINVAL also for a null opt, an unknown rule or nonzero
 *         reserved fields.
 */
#define GC_ADACOMP_RULE_RESIDUAL 0
#define GC_ADACOMP_RULE_GRADIENT 1
typedef struct gc_adacomp_options {
    float    scale_factor;  /* >= 1; 2.0 in the pages  */
    int      rule;          /* GC_ADACOMP_RULE_*       */
    uint32_t reserved[2];   /* must be 0               */
} gc_adacomp_options;
gc_status gc_adacomp_compress_ex(const gc_plan *plan, const float *dW, float *R, void *state,
                                 size_t state_bytes, const gc_adacomp_options *opt, gc_sparse *out,
                                 void *ws, size_t ws_bytes, hipStream_t stream);

/* Bytes of one learner's deferred-residual state for this plan (0 if plan
 * is NULL). */
size_t gc_adacomp_state_bytes(const gc_plan *plan);

/* Slots an AdaComp message needs for this plan: the sum of the segment
 * lengths (0 if plan is NULL).  Gaps between segments need none. */
uint64_t gc_adacomp_message_cap(const gc_plan *plan);

/* R_out[n_total] <- the exact residual held by (R, state): elements outside
 * every segment are copied, in-segment elements sent in the last deferred
 * step get fl32(R_i - copysign(scale_s, R_i)).  state == NULL copies R.
 * R_out must not overlap R; R and state are not modified.
 * Errors: GC_EINVAL (null R or R_out, overlap, misaligned state),
 *         GC_ECAPACITY (state smaller than gc_adacomp_state_bytes). */
gc_status gc_adacomp_residual(const gc_plan *plan, const float *R, const void *state,
                              size_t state_bytes, float *R_out, hipStream_t stream);

/* ------------------------------------------------------------------- DGC */
/*
 * One DGC step for one learner, vanilla momentum ([DGC] §3.1–§3.3, App. C, D):
 *   a7  local clipping (App. C), only if thr_G > 0:
 *         thr = fl32(thr_G / sqrt(num_nodes))            (in double)
 *         S_s = PSUM64(G_i^2 over the segment)            (squares exact in double)
 *         c_s = fl32(thr / sqrt(S_s)) if sqrt(S_s) > thr else 1
 *       G'_i = fl32(c_s * G_i)
 *   a8  momentum correction (§3.2):  U_i <- fl32(fl32(momentum*U_i) + G'_i)
 *                                    V_i <- fl32(V_i + U_i)
 *   a9  exact top-k (§3.1, §5): key_i = bits(V_i) & 0x7FFFFFFF; the k_s entries
 *       first in the order (key descending, index ascending) are sent.
 *   a10 momentum factor masking (§3.3): at sent indices V_i <- +0, U_i <- +0.
 *   out: per segment exactly k_s entries, ascending idx, val = V_i before masking.
 *   G [n_total] in;  U, V [n_total] in/out;  out->cap >= gc_plan_total_k(plan).
 *   0 <= momentum < 1;  num_nodes >= 1;  thr_G <= 0 disables clipping.
 * Errors: GC_EINVAL, GC_ECAPACITY (out->cap or ws too small).
 */
gc_status gc_dgc_step(const gc_plan *plan, const float *G, float *U, float *V,
                      float momentum, float thr_G, int num_nodes,
                      gc_sparse *out, void *ws, size_t ws_bytes,
                      hipStream_t stream);

/*
 * DGC step with the momentum kind and the selection mode chosen.
 * gc_dgc_step(plan, G, U, V, m, thr_G, N, ...) is this call with
 * {m, thr_G, N, GC_MOMENTUM_VANILLA, GC_SELECT_EXACT}.
 *
 * Momentum correction ([DGC] §3.2, App. B, App. D):
 *   GC_MOMENTUM_VANILLA  (Alg. 3)  U_i <- fl32(fl32(m*U_i) + G'_i);  V_i <- fl32(V_i + U_i)
 *   GC_MOMENTUM_NESTEROV (Alg. 4)  U_i <- fl32(fl32(m*U_i) + G'_i);
 *                                  V_i <- fl32(V_i + fl32(fl32(m*U_i) + G'_i))  (updated U_i)
 *   Nesterov SGD steps along m*U + G with U <- m*U + G; momentum correction
 *   accumulates that step direction in V instead of applying it.  Clipping
 *   (a7) and masking (a10) are as in gc_dgc_step.
 *
 * Selection ([DGC] §3.1, §5, §6):
 *   GC_SELECT_EXACT    exactly k_s entries per segment, as in gc_dgc_step.
 *   GC_SELECT_SAMPLED  the threshold is estimated from a sample and, when it
 *     lets through far more entries than k_s, the exact top-k is taken among
 *     those (hierarchical selection).  Per segment of n entries:
 *       sample: window w = 0, 1, ... covers entries [32*P*w, 32*P*(w+1)) of
 *         the segment; its block is the 32 entries starting at
 *         32*P*w + 32*((w * 2654435769 mod 2^32) mod P), those at or past n
 *         excluded (P = sample_period: 1/P of the entries; the page samples
 *         0.1% to 1%, P = 1000 to 100).  S = number of sampled entries.
 *       estimate: thr = the r-th largest key among the sampled entries'
 *         keys (of V after a8), r = ceil(S * k_s / n).
 *       C = #{ i : key_i >= thr }.  If C <= min(n, over * k_s), those C
 *         entries are sent; otherwise the exact top k_s (as GC_SELECT_EXACT).
 *     Segments' entries are laid end to end: seg_off[s+1] - seg_off[s] is
 *     the segment's count.  The call's cost grows with S (small P is slow).
 *   out->cap >= gc_dgc_message_cap(plan, opt).
 * Errors: as gc_dgc_step; GC_EINVAL also for an unknown momentum_kind or
 *         select, sample_period outside [1, GC_MAX_SAMPLE_PERIOD] or over < 1
 *         in sampled mode, reserved != 0.
 */
#define GC_MAX_SAMPLE_PERIOD  (1u << 26)
#define GC_MOMENTUM_VANILLA   0
#define GC_MOMENTUM_NESTEROV  1
#define GC_SELECT_EXACT       0
#define GC_SELECT_SAMPLED     1
typedef struct gc_dgc_options {
    float    momentum;       /* 0 <= m < 1                                   */
    float    thr_G;          /* clip threshold of the whole job; <= 0: none  */
    int      num_nodes;      /* N >= 1                                       */
    int      momentum_kind;  /* GC_MOMENTUM_*                                */
    int      select;         /* GC_SELECT_*                                  */
    uint32_t sample_period;  /* GC_SELECT_SAMPLED: 1 <= P <= GC_MAX_SAMPLE_PERIOD */
    uint32_t over;           /* GC_SELECT_SAMPLED: budget factor >= 1        */
    uint32_t reserved;       /* must be 0                                    */
    uint32_t density_num;    /* per-call density (warm-up): with             */
    uint32_t density_den;    /* density_den > 0, k_s = clamp(ceil(n_s *     */
                             /* density_num / density_den), 1, n_s) in place */
                             /* of the plan's k; 0 < num <= den; exact only  */
} gc_dgc_options;

/* Entries a message needs for these options: sum of k_s (exact), or sum of
 * min(n_s, over * k_s) (sampled).  0 if plan is NULL. */
uint64_t  gc_dgc_message_cap(const gc_plan *plan, const gc_dgc_options *opt);
gc_status gc_dgc_step_ex(const gc_plan *plan, const float *G, float *U, float *V,
                         const gc_dgc_options *opt, gc_sparse *out, void *ws,
                         size_t ws_bytes, hipStream_t stream);

/* ------------------------------------------------------------------ pack */
/*
 * Byte-exact run-length encoding of a message ([DGC] §3.1: 32-bit values and
 * 16-bit zero-run lengths).  Little-endian; every block 4-byte aligned.
 *   stream header : u32 'GCP2', u32 kind, u32 nseg, u32 0
 *   block table   : per segment u64 offset of its block from the stream
 *                   start, u32 E, u32 entries of the segment
 *   then the blocks in segment order, the first at 16 + 16 nseg:
 *   DGC block     : u32 'DGC1', u32 n_s, u32 E, u32 entries of the segment,
 *                   u16 run[E] (+ one u16 0 if E is odd), f32 val[E],
 *                   checkpoints
 *   AdaComp block : u32 'ADC1', u32 n_s, u32 E, f32 scale_s,
 *                   u16 code[E] (+ one u16 0 if E is odd), checkpoints;
 *                   code = sign << 15 | run  (sign 1 = negative)
 *   checkpoints   : for c = 0 .. ceil(E / 4096) - 1, u32 entries and u32
 *                   reader position p (as gc_unpack defines it) before code
 *                   4096 c
 * The table and the checkpoints let a receiver read blocks and tiles of
 * 4096 codes independently.
 * A run counts the unsent elements since the previous entry of the segment
 * (from the segment start for the first).  A run >= MAX is split: emit an
 * escape (run MAX; DGC value +0.0f), subtract MAX, repeat.  MAX is 65535 for
 * DGC and 32767 for AdaComp; E counts entries plus escapes.
 *   in       : a message produced for this plan (device counts are read;
 *              a segment's entries are taken up to its length).
 *   out      : device byte buffer of out_cap >= gc_pack_bound(plan, kind),
 *              which holds any AdaComp message and any DGC message of the
 *              plan's k per segment.  A DGC message with more entries per
 *              segment (a per-call density, or the sampled selection's
 *              budget) may need up to gc_dgc_pack_bound(plan, opt) bytes.
 *   out_bytes: device u64, receives the stream length.  When it exceeds
 *              out_cap the stream did not fit: out does not hold it (no
 *              byte past out_cap is written), and the message needs a
 *              buffer of at least *out_bytes bytes (the sizes above always
 *              suffice).
 * Errors: GC_EINVAL (bad kind / null), GC_ECAPACITY (out_cap or ws too small).
 */
#define GC_KIND_DGC      1
#define GC_KIND_ADACOMP  2
uint64_t  gc_pack_bound(const gc_plan *plan, int kind);
/* Stream bytes a DGC message of these selection options needs at most: the
 * bound above with k_s replaced by the call's entries per segment (a
 * per-call density's ceil(n_s num / den), or min(n_s, over k_s) sampled).
 * opt NULL: gc_pack_bound(plan, GC_KIND_DGC).  0 if plan is NULL. */
uint64_t  gc_dgc_pack_bound(const gc_plan *plan, const gc_dgc_options *opt);
gc_status gc_pack(const gc_plan *plan, int kind, const gc_sparse *in,
                  uint8_t *out, uint64_t out_cap, uint64_t *out_bytes,
                  void *ws, size_t ws_bytes, hipStream_t stream);

/*
 * The receiver's inverse of gc_pack: a stream (as gc_pack wrote it, for this
 * plan and kind) read back into a message for gc_decompress_accumulate.  Per
 * segment, codes are read in order from position p = 0: a code whose run is
 * MAX (DGC 0xFFFF; AdaComp 0x7FFF, sign bit ignored) advances p by MAX;
 * any other code puts an entry at segment position p + run, with val = the
 * code's f32 value (DGC) or +-scale_s by the sign bit (AdaComp), then sets
 * p to that position + 1.
 *   in       : device stream of in_bytes bytes (4-byte aligned, >= 16).
 *   out      : idx/val (ascending per segment), seg_off[nseg+1] and, for
 *              AdaComp, seg_scale[nseg].  Entries at or past out->cap are
 *              not written (seg_off is clamped to cap).
 *   status   : device u32, set to 0 for a stream that fits the plan, else a
 *              bitmask: 1 bad stream header (or too short for its table),
 *              2 a block table entry or block header that disagrees with the
 *              plan, the stream's bytes or the blocks before it (or
 *              trailing bytes): the whole stream is then read as empty,
 *              4 an entry outside its segment (not written), 8 more entries
 *              than out->cap, 16 a tile whose entries or positions disagree
 *              with the next checkpoint or the block's entry count.
 *              Whatever the stream, every write stays inside the message,
 *              inside the range seg_off gives its segment, and inside the
 *              segment's elements.
 *   ws       : gc_plan_workspace_bytes(plan, GC_OP_UNPACK) bytes.
 * One workgroup checks the table and headers; then every tile of 4096 codes
 * is read from its checkpoint, independently of the others.
 * Errors: GC_EINVAL (bad kind, null pointers, misaligned or short stream),
 *         GC_ECAPACITY (ws).
 */
gc_status gc_unpack(const gc_plan *plan, int kind, const uint8_t *in, uint64_t in_bytes,
                    gc_sparse *out, uint32_t *status, void *ws, size_t ws_bytes,
                    hipStream_t stream);

/* ---------------------------------------------------------------- decode */
/*
 * Decompress-and-aggregate K messages into a dense update ([DGC] App. A: the
 * nodes' gradients are summed; [AdaComp]: the learners' compressed gradients
 * are averaged).  For every element i of the plan's segments:
 *   S_i = +0.0f, then S_i = fl32(S_i + v_{k,i}) for k = 0..K-1 in array order
 *         over the messages that hold i;
 *   r_i = fl32(S_i / K) (GC_AVG) or S_i (GC_SUM);
 *   dense_i = r_i (accumulate == 0) or fl32(dense_i + r_i) (accumulate != 0).
 *   msgs (host array of K <= GC_MAX_MESSAGES): messages for this plan with
 *   indices inside segments and ascending.  dense [n_total] out (in/out if
 *   accumulate).  Elements in gaps between segments are not touched.
 * Errors: GC_EINVAL (K out of range, bad mode, null), GC_ECAPACITY (ws).
 */
#define GC_SUM  0
#define GC_AVG  1
gc_status gc_decompress_accumulate(const gc_plan *plan, const gc_sparse *msgs,
                                   int K, float *dense, int mode,
                                   int accumulate, void *ws, size_t ws_bytes,
                                   hipStream_t stream);

/*
 * For callers that cannot allocate device memory: code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc.  The same
 * operation and results as gc_decompress_accumulate, with no workspace
 * argument: the index pass's table (K * (chunks + 1) u32, where chunks is
 * the plan's count of 4096-element tiles) lives in a fixed 8 MiB device
 * array inside the library.  Each GPU holds its own copy until the process
 * ends.  The call allocates nothing: it looks the array's address up once per
 * device (hipGetSymbolAddress) and requires the plan's tables to be on the
 * current device already (gc_plan_upload, outside the caller's hot loop).
 * Every call on one GPU shares that GPU's array, so calls that overlap on one
 * GPU (other streams, other threads) race and give undefined results; calls
 * in one stream are ordered and safe.  Nothing in the array needs to start at
 * any value: each call writes every entry it reads.
 * gc_decompress_noalloc_max_chunks(K) is the largest plan chunk count the
 * array holds for K messages (2,097,152 / K - 1; 0 for K out of range).
 * Errors: as gc_decompress_accumulate, plus GC_ECAPACITY when the plan has
 *         more chunks than that (checked on the host) and GC_EINVAL when the
 *         plan was not uploaded to the current device.
 */
uint64_t  gc_decompress_noalloc_max_chunks(int K);
gc_status gc_decompress_accumulate_noalloc(const gc_plan *plan, const gc_sparse *msgs,
                                           int K, float *dense, int mode,
                                           int accumulate, hipStream_t stream);

/* ------------------------------------------------------------------- DCD */
/*
 * Compressed model difference with random quantization ([DCD] DCD-PSGD step 2;
 * [SlimDP] Quant-DP: buckets of 512; 8-bit and 4-bit precisions).
 *   z_i = fl32(x_half_i - x_i); buckets of `bucket` elements over [0, n).
 *   s_b = max |z_i| in bucket b -> scales[b].
 *   L = 2^(bits-1) - 1.  If s_b == 0 every code is 0 and C_i = 0.  Otherwise
 *     inv = fl32(L / s_b); y = min(L, fl32(|z_i| * inv)); l0 = floor(y);
 *     f = y - l0; r = word (i mod 4) of Philox4x32-10(key = (seed lo, seed hi),
 *     counter = (lo(i/4), hi(i/4), lo(step), hi(step))); u = (r >> 8) * 2^-24;
 *     l = l0 + (u < f); C_i = +-fl32(l * fl32(s_b / L)) with the sign of z_i.
 *   code_i = l == 0 ? 0 : (sign << (bits-1)) | l.  4-bit codes are packed two
 *   per byte, even index in the low nibble; 8-bit codes one per byte.
 *   x_out_i = fl32(x_i + C_i)  (x_out may equal x: step 2's local update).
 *   scales [ceil(n/bucket)], codes [ceil(n*bits/8)] out.
 *   codes must be 4-byte aligned.
 * Errors: GC_EINVAL (bits not 4 or 8, bucket 0, null, misaligned codes),
 *         GC_ENOTSUP (bucket not a power of two in [4, 4096]),
 *         GC_ERANGE (n > 2^32 - 8192).
 */
gc_status gc_dcd_compress(const float *x, const float *x_half, float *x_out,
                          uint64_t n, int bits, uint32_t bucket, uint64_t seed,
                          uint64_t step, float *scales, uint8_t *codes,
                          hipStream_t stream);

/*
 * DCD-PSGD step 3 ([DCD] step 3): a neighbour's replica advances by the
 * received compressed difference, x_hat_i <- fl32(x_hat_i + C_i), with C_i
 * decoded from the stream gc_dcd_compress wrote:
 *   code_i = codes[i] (8 bits) or nibble i%2 of codes[i/2] (4 bits, even i in
 *   the low nibble); level = code & L, L = 2^(bits-1) - 1; sign = bit bits-1;
 *   C_i = level == 0 ? 0 : +-fl32(level * fl32(scales[i/bucket] / L)).
 * Applied to a copy of x_t this reproduces gc_dcd_compress's x_out bit for
 * bit, so every replica stays equal to its node's model.
 *   scales [ceil(n/bucket)], codes [ceil(n*bits/8)] in (codes 4-byte aligned);
 *   x_hat [n] in/out.
 * Errors: GC_EINVAL (null, bits not 4 or 8, bucket 0, misaligned codes),
 *         GC_ENOTSUP (bucket not a power of two in [4, 4096]),
 *         GC_ERANGE (n > 2^32 - 8192).
 */
gc_status gc_dcd_decode(const float *scales, const uint8_t *codes, uint64_t n, int bits,
                        uint32_t bucket, float *x_hat, hipStream_t stream);

/*
 * DCD-PSGD step 1 ([DCD] step 1): the weighted average of the replicas (the
 * node's own model among them) and a stochastic gradient step:
 *   S_i = +0, then S_i = fl32(S_i + fl32(weights[j] * replicas[j][i])) for
 *         j = 0..K-1 in array order;
 *   x_half_i = fl32(S_i - fl32(lr * grad_i)).
 *   replicas (host array of K device pointers, 1 <= K <= GC_MAX_REPLICAS),
 *   weights (host array of K: row i of the mixing matrix W), grad [n] in,
 *   x_half [n] out (must not alias grad or a replica).
 * Errors: GC_EINVAL (null, K out of range, aliasing), GC_ERANGE (n > 2^32 - 8192).
 */
#define GC_MAX_REPLICAS 16
gc_status gc_dcd_mix(const float *const *replicas, const float *weights, int K,
                     const float *grad, float lr, float *x_half, uint64_t n,
                     hipStream_t stream);

/*
 * ECD-PSGD sender ([DCD] ECD-PSGD, Eq. 3): the extrapolated value
 *   z_i = fl32(fl32(a * x_prev_i) + fl32(b * x_i)),  a = fl32(1 - t/2), b = fl32(t/2)
 * (coefficients formed in double), quantized exactly as gc_dcd_compress
 * quantizes z (same code layout and scales) with Philox step = t.
 *   x_prev = x_{t-1}, x = x_t [n] in; t >= 1; scales, codes out.
 * Errors: as gc_dcd_decode; GC_EINVAL also for t = 0.
 */
gc_status gc_ecd_compress(const float *x_prev, const float *x, uint64_t n, uint64_t t,
                          int bits, uint32_t bucket, uint64_t seed, float *scales,
                          uint8_t *codes, hipStream_t stream);

/*
 * ECD-PSGD receiver ([DCD] ECD-PSGD, Eq. 4): the estimate of a neighbour's
 * model, x_tilde_i <- fl32(fl32(c1 * x_tilde_i) + fl32(c2 * C_i)) with
 * c1 = fl32(1 - 2/t), c2 = fl32(2/t) (formed in double), C_i decoded as in
 * gc_dcd_decode.  t >= 1.
 * Errors: as gc_dcd_decode; GC_EINVAL also for t = 0.
 */
gc_status gc_ecd_update(const float *scales, const uint8_t *codes, uint64_t n, int bits,
                        uint32_t bucket, uint64_t t, float *x_tilde, hipStream_t stream);

/* ---------------------------------------------------------------- Slim-DP */
/*
 * Slim-DP's communication set ([SlimDP] §3: a core of significant parameters
 * chosen by the server, plus an explorer of random parameters from outside
 * the core chosen by each worker at every communication).
 *
 * Core:  S_i = fl32(|w_i| + fl32(c * |g_i|)), c > 0 (the page combines the
 *   magnitudes of the parameter and of its gradient as a weighted sum with a
 *   positive coefficient; its equation is not printed).  Per segment, the k_s
 *   entries first in the order (S descending, index ascending) form the core
 *   (k_s from `plan`, e.g. ceil(beta * n_s)).
 *     core      : ascending idx, val = S_i; exactly sum(k_s) entries.
 *     core_mask : gc_slimdp_mask_words(plan) u32 words out: per segment a run
 *                 of ceil(n_s/32) words, bit j%32 of word j/32 set iff entry j
 *                 of the segment is in the core.
 * Explorer: per segment, the m_s non-core entries first in the order (key
 *   descending, index ascending), key_j = r >> 1 | 1 with r = word j%4 of
 *   Philox4x32-10(counter (j/4, s, lo(step), hi(step)), key (lo(seed),
 *   hi(seed))) for entry j of segment s; core entries never qualify.  A
 *   uniformly random set of m_s non-core entries, resampled with `step`.
 *     plan      : the same segments as core_plan with k_s = m_s, and
 *                 m_s + (core k_s) <= n_s.
 *     out       : ascending idx, val = delta_i; exactly sum(m_s) entries.
 * Core values: the core's keys are cached on both sides ([SlimDP] key caching
 *   filter), so a push sends only values: values[j] = delta[core->idx[j]]
 *   for j < gc_plan_total_k(core_plan) (core as gc_slimdp_core wrote it;
 *   indices at or past n_total are clamped to the last element).
 * Workspaces: gc_plan_workspace_bytes(plan, GC_OP_DGC).
 * Errors: GC_EINVAL (null, c not positive and finite, plans that differ in
 *         segments, core + explorer above a segment), GC_ECAPACITY.
 */
uint64_t  gc_slimdp_mask_words(const gc_plan *plan);
gc_status gc_slimdp_core(const gc_plan *plan, const float *w, const float *g, float c,
                         gc_sparse *core, uint32_t *core_mask, void *ws, size_t ws_bytes,
                         hipStream_t stream);
gc_status gc_slimdp_explore(const gc_plan *plan, const gc_plan *core_plan, const float *delta,
                            const uint32_t *core_mask, uint64_t seed, uint64_t step,
                            gc_sparse *out, void *ws, size_t ws_bytes, hipStream_t stream);
gc_status gc_slimdp_core_values(const gc_plan *core_plan, const gc_sparse *core,
                                const float *delta, float *values, hipStream_t stream);

/* ------------------------------------------------------------- embedding */
/*
 * The embedding of a flat model buffer: segment `seg` of the plan read as
 * `rows` x cols, row-major, cols = length / rows (rows must divide the
 * length).  A batch is n_tokens token ids (int32 or int64) and one dense row
 * per token, y or dy: cols elements of fp32, bf16 or fp16, `stride` elements
 * from one row to the next (stride >= cols; the elements between are neither
 * read nor written).  An id outside [0, rows) is padding: its row of y is
 * +0, and its row of dy is not read and counts for nothing.
 */
#define GC_F32   0
#define GC_BF16  1
#define GC_F16   2
#define GC_TOKENS_I32  0
#define GC_TOKENS_I64  1

/*
 * y_i = fl32(scale * w[t_i]), rounded to nearest (ties to even) once more
 * for bf16 and fp16.
 *   w [n_total] in, tokens [n_tokens] in, y out.  scale finite.
 * n_tokens == 0 enqueues nothing.  Needs neither workspace nor the plan's
 * tables on the device.
 * Errors: GC_EINVAL (null, seg or rows that do not fit the plan, unknown
 *         types, stride < cols, misaligned buffers, scale not finite),
 *         GC_ERANGE (n_tokens >= 2^28, n_tokens * stride > 2^48,
 *         n_tokens * cols > 2^35, or more than a launch's 2^32 threads).
 */
gc_status gc_embed_lookup(const gc_plan *plan, int seg, uint32_t rows, const float *w,
                          const void *tokens, int token_type, uint64_t n_tokens, float scale,
                          void *y, int y_type, uint64_t y_stride, hipStream_t stream);

/*
 * The gradient of the lookup.  For every row r with at least one token,
 *   S_r = sum in fp32 of dy_i over the positions i with t_i = r;
 *   accumulate == 0: g[r] = fl32(scale * S_r), every other row +0;
 *   accumulate != 0: g[r] = fl32(g[r] + fl32(scale * S_r)), no other row is
 *                    touched.
 * The order of a sum is fixed by the tokens alone: positions are ordered by
 * (row, position) and cut into blocks of 16; a row's positions of one block
 * are added in order from +0.  A row that lies in more than one block has
 * block sums s_0, s_1, ...; the sums Z_w of s_w, s_{w+16}, s_{w+32}, ...
 * (each in order from +0) are formed and added in the order Z_0, Z_1, ...,
 * Z_15.
 *   g  [n_total] out (in/out if accumulate); only the segment is touched.
 *   ws : gc_embed_workspace_bytes(plan, seg, rows, n_tokens) bytes (0 on an
 *        argument error).  n_tokens == 0 needs none (ws may be NULL).
 * Errors: as gc_embed_lookup; GC_ECAPACITY (ws too small).
 */
size_t    gc_embed_workspace_bytes(const gc_plan *plan, int seg, uint32_t rows, uint64_t n_tokens);
gc_status gc_embed_grad(const gc_plan *plan, int seg, uint32_t rows, const void *dy, int dy_type,
                        uint64_t dy_stride, const void *tokens, int token_type, uint64_t n_tokens,
                        float scale, float *g, int accumulate, void *ws, size_t ws_bytes,
                        hipStream_t stream);

/*
 * The same gradient as a message for gc_pack or gc_decompress_accumulate:
 * the rows that have tokens, ascending, all their columns, idx the flat
 * indices and val = fl32(scale * S_r).  seg_off is 0 up to seg and the entry
 * count behind it (the plan's other segments are empty); seg_scale is not
 * written.  Entries past the count are left as they were.
 *   out->cap >= gc_embed_message_cap(...) = min(n_tokens, rows) * cols.
 * A DGC stream of such a message needs up to gc_dgc_pack_bound with a density
 * of 1/1.
 * Errors: as gc_embed_grad; GC_ECAPACITY also for out->cap.
 */
uint64_t  gc_embed_message_cap(const gc_plan *plan, int seg, uint32_t rows, uint64_t n_tokens);
gc_status gc_embed_message(const gc_plan *plan, int seg, uint32_t rows, const void *dy, int dy_type,
                           uint64_t dy_stride, const void *tokens, int token_type,
                           uint64_t n_tokens, float scale, gc_sparse *out, void *ws,
                           size_t ws_bytes, hipStream_t stream);

/* ----------------------------------------------------- matrix updates */
/*
 * Segments of a plan that are weight matrices, for updates that treat a
 * matrix as a whole (Muon).  Opaque and immutable; it keeps nothing of the
 * gc_plan.
 *   rows[nseg] (host): the rows R of segment s, row-major, with C = length /
 *   R columns; 0 for a segment that is no matrix, which the calls below
 *   neither read nor write.
 * Host only: touches no device.  The tables go to a device as a gc_plan's do
 * (first use, or gc_matrix_plan_upload: one hipMalloc and one synchronous
 * copy per device).
 * Errors: GC_EINVAL (null, rows that do not divide a length, no matrix),
 *         GC_ENOTSUP (more than GC_MAX_MATRIX_DIM rows or columns),
 *         GC_ERANGE (more than 2^24 tiles of 64 x 64 or matrices).
 */
#define GC_MAX_MATRIX_DIM  (1u << 20)
typedef struct gc_matrix_plan gc_matrix_plan;
gc_status gc_matrix_plan_create(const gc_plan *plan, const uint32_t *rows, gc_matrix_plan **out);
void      gc_matrix_plan_destroy(gc_matrix_plan *mplan);
gc_status gc_matrix_plan_upload(const gc_matrix_plan *mplan);
/*
 * Device workspace bytes of gc_orthogonalize and gc_muon_step (0 for NULL):
 * 16 an element of the matrices, their rows and columns rounded up to 128
 * (8 where no matrix has more than 128 on its smaller side), 8 to 12 an element
 * of their m x m products, and the parts of products that are cut.  Calls that
 * run one after the other can share one workspace.
 */
size_t    gc_matrix_plan_workspace_bytes(const gc_matrix_plan *mplan);

/*
 * Every matrix D (R x C) of the plan, orthogonalised by Newton-Schulz
 * products:
 *   X_0 = D / (||D||_F + eps)   (the norm in double; X = D^T where R > C)
 *   X_{k+1} = a_k X_k + (b_k A + c_k A^2) X_k,  A = X_k X_k^T,
 *   k = 0 .. steps - 1, (a_k, b_k, c_k) = coef[k];   O = X_steps (transposed
 *   back).
 * Each step maps every singular value s of X to a s + b s^3 + c s^5 and
 * keeps the singular vectors.  With (3.4445, -4.7750, 2.0315) five steps
 * bring all but the smallest to between about 0.7 and 1.2.
 * Products are formed from operands of 22 bits with fp32 sums.  Measured on
 * random matrices against 64 bits, five of these steps end 0.2 to 1.4 times as
 * far off as with fp32 products (0.6e-6 to 3e-6 of the result); one or two
 * steps, or gentle coefficients such as (1.5, -0.5, 0), up to 5 times as far, at
 * 5e-7 of the result or less.  Where one or a few singular values make up the
 * matrix, theirs are single chains of roundings: about 2^-19 of a step's terms
 * at most, times the slopes of the later steps.  (Entries of X_0 below 2^-18,
 * where ||D|| is far below eps, keep an absolute 2^-40 instead.)  Unlike the
 * other calls' results it is no fixed sequence of IEEE operations, but the same
 * call on the same device gives the same bits.
 * D = 0 gives O = +-0.  A matrix with a NaN or Inf becomes NaN altogether and
 * leaves the others alone.
 *   D [n_total] in, O [n_total] out; O may be D, or must not overlap it.
 *   ws : gc_matrix_plan_workspace_bytes bytes.
 * Errors: GC_EINVAL (null, steps, eps negative or not finite, reserved not 0,
 *         coefficients that are not finite, or with which singular values
 *         of at most 1 at the start may pass 8 before the last step (1e12
 *         after it), those of a I + b A + c A^2 2^14, or all fall below 1e-12,
 *         where a step may be off by 2^-19 of the sizes of its terms;
 *         overlapping buffers), GC_ECAPACITY (ws).
 */
#define GC_MAX_ORTH_STEPS  16
typedef struct gc_orth_options {
    int      steps;                        /* 1 .. GC_MAX_ORTH_STEPS */
    float    eps;                          /* >= 0                   */
    float    coef[GC_MAX_ORTH_STEPS][3];   /* a, b, c of each step   */
    uint32_t reserved[2];                  /* must be 0              */
} gc_orth_options;
gc_status gc_orthogonalize(const gc_matrix_plan *mplan, const float *D, float *O,
                           const gc_orth_options *opt, void *ws, size_t ws_bytes,
                           hipStream_t stream);

/*
 * One Muon step on every matrix of the plan, from the gradient that
 * gc_decompress_accumulate (or the learner itself) left in G:
 *   U <- fl32(fl32(m*U) + G)
 *   D  = U (GC_MOMENTUM_VANILLA) or fl32(fl32(m*U) + G), U the new one
 *        (GC_MOMENTUM_NESTEROV)
 *   O  = D orthogonalised as above
 *   W <- fl32(fl32(d*W) - fl32(l*O)),  d = fl32(1 - lr * weight_decay),
 *        l = fl32(lr * s)  (formed in double)
 *   s = 1 (GC_MUON_SCALE_NONE), sqrt(max(1, R / C)) (GC_MUON_SCALE_SHAPE) or
 *       0.2 sqrt(max(R, C)) (GC_MUON_SCALE_RMS).
 * Where momentum correction already ran in DGC's V, m = 0 leaves it at that
 * (U then holds G).
 *   G [n_total] in, U, W [n_total] in/out; none overlaps another.
 * Errors: as gc_orthogonalize; GC_EINVAL also for momentum outside [0, 1), lr
 *         or weight_decay not finite, weight_decay < 0, an unknown
 *         momentum_kind or scale.
 */
#define GC_MUON_SCALE_NONE   0
#define GC_MUON_SCALE_SHAPE  1
#define GC_MUON_SCALE_RMS    2
typedef struct gc_muon_options {
    gc_orth_options orth;
    float    momentum;       /* 0 <= m < 1        */
    float    lr;
    float    weight_decay;   /* >= 0              */
    int      momentum_kind;  /* GC_MOMENTUM_*     */
    int      scale;          /* GC_MUON_SCALE_*   */
    uint32_t reserved;       /* must be 0         */
} gc_muon_options;
gc_status gc_muon_step(const gc_matrix_plan *mplan, const float *G, float *U, float *W,
                       const gc_muon_options *opt, void *ws, size_t ws_bytes, hipStream_t stream);

/* ------------------------------------------------------- layer products */
/*
 * A layer of the model: segment `seg` of the plan is its weight matrix W, rows
 * x cols, row-major (cols = length / rows), segment `bias_seg` its bias b of
 * `rows` elements (-1: none).  A batch is n_tokens rows of activations; every
 * such array has elements of `type` and its own stride, in elements, from one
 * row to the next (at least the row's length; the elements between are neither
 * read nor written).  w is the flat model in that type: the fp32 buffer itself,
 * or a copy of it in bf16 or fp16 with the same offsets.
 * Sums are fp32, over exact products for bf16 and fp16 (in their rounding a
 * subnormal operand counts as the smallest normal one).  For fp32 a product is
 * off by 2^-21 of itself at most, of either sign and by less than 2^-24 on
 * average (three bf16 parts an operand, six products of them), and what an
 * operand has below 2^-133 is dropped; short batches of forward and grad_input
 * may go by fp32 products instead.  Each output is rounded once.  The order of
 * a sum is fixed by the sizes and alignments, so the same call gives the same
 * bits.  NaN and Inf go where the formulas take them, but for an Inf in an fp32
 * operand, whose sums are NaN or that Inf; no row or column reaches another's
 * results.
 *
 * Activations: act(z) is z (GC_ACT_NONE), max(z, 0) (RELU; NaN stays),
 * z Phi(z) (GELU; Phi the normal distribution), z s(2 u) with
 * u = sqrt(2 / pi) (z + 0.044715 z^3) (GELU_TANH; s(v) = 1 / (1 + exp(-v))),
 * z s(z) (SILU).  RELU's slope at 0 is 0.  They are formed in fp32 before the
 * one rounding: for fp32 within (20 + 4 a) 2^-23 of themselves, a = z^2 / 2,
 * |2 u| or |z| the exponent they take, for bf16 and fp16 within 2^-14; a slope
 * within that part of its two terms' sizes.  What lies below 2^-119 may come out
 * as 0.
 */
#define GC_ACT_NONE       0
#define GC_ACT_RELU       1
#define GC_ACT_GELU       2
#define GC_ACT_GELU_TANH  3
#define GC_ACT_SILU       4
typedef struct gc_linear {
    int      seg;
    uint32_t rows;          /* outputs; must divide the segment's length        */
    int      bias_seg;      /* a segment of `rows` elements, or -1: no bias     */
    int      type;          /* GC_F32, GC_BF16 or GC_F16                        */
    uint32_t reserved[2];   /* must be 0                                        */
} gc_linear;

/* Device workspace bytes of the three calls below for any batch of up to
 * n_tokens rows (0 on an argument error): the parts of sums that are cut, at most
 * 33 MiB.  Calls that run one after the other can share one. */
size_t gc_linear_workspace_bytes(const gc_plan *plan, const gc_linear *layer, uint64_t n_tokens);

/*
 * z = x W^T + b;  y = act(z) + r.
 *   w [n_total] in; x [n_tokens][cols] in; y [n_tokens][rows] out.
 *   r [n_tokens][rows] in, or NULL: nothing is added.  r may be y (with its stride).
 *   z [n_tokens][rows] out, or NULL: z (rounded to the type; y is formed
 *     before that rounding), which gc_act_grad and gc_linear_grad_input take.
 * n_tokens == 0 enqueues nothing.
 * Errors: GC_EINVAL (null, seg, rows or bias_seg that do not fit the plan,
 *         unknown type or act, reserved not 0, a stride below its row, buffers
 *         not aligned to their elements, an output that is another buffer of
 *         the call), GC_ERANGE (n_tokens >= 2^28, n_tokens * max(rows, cols) >
 *         2^35, n_tokens * a stride > 2^48, more workgroups than a launch has),
 *         GC_ECAPACITY (ws).
 */
gc_status gc_linear_forward(const gc_plan *plan, const gc_linear *layer, const void *w, const void *x,
                            uint64_t x_stride, uint64_t n_tokens, int act, const void *r, uint64_t r_stride,
                            void *z, uint64_t z_stride, void *y, uint64_t y_stride, void *ws, size_t ws_bytes,
                            hipStream_t stream);

/*
 * dz = dy act'(z), the first step of the way back where no other call's
 * epilogue does it; n_rows x cols elements of `type`.  dz may be dy or z (with
 * its stride).
 * Errors: GC_EINVAL (null, unknown type or act, strides, misaligned buffers),
 *         GC_ERANGE (as above).
 */
gc_status gc_act_grad(const void *dy, uint64_t dy_stride, const void *z, uint64_t z_stride, int act, int type,
                      uint64_t n_rows, uint64_t cols, void *dz, uint64_t dz_stride, hipStream_t stream);

/*
 * The gradient of the layer's input, and of what the layer before it
 * activated: g = dz W + a;  dx = g;  dzx = g act'(z), where x = act(z) (+ a
 * residual) and a is the gradient that reaches x another way.
 *   dz [n_tokens][rows] in; w as above.
 *   a [n_tokens][cols] in, or NULL.  a may be dx or dzx (with its stride).
 *   dx, dzx [n_tokens][cols] out; either may be NULL, not both.  dzx is formed
 *     from g before its rounding to dx.
 *   z [n_tokens][cols] in; needed with dzx unless act is GC_ACT_NONE.
 * Errors: as gc_linear_forward.
 */
gc_status gc_linear_grad_input(const gc_plan *plan, const gc_linear *layer, const void *w, const void *dz,
                               uint64_t dz_stride, uint64_t n_tokens, const void *a, uint64_t a_stride, int act,
                               const void *z, uint64_t z_stride, void *dx, uint64_t dx_stride, void *dzx,
                               uint64_t dzx_stride, void *ws, size_t ws_bytes, hipStream_t stream);

/*
 * The gradient of the layer's weights, in the flat gradient that the
 * compression calls and gc_muon_step take: segment seg of g becomes dz^T x
 * and segment bias_seg (if any) the sum of dz's rows (accumulate == 0), or
 * fl32(g + that) (accumulate != 0).  Always fp32.
 *   dz [n_tokens][rows], x [n_tokens][cols] in; g [n_total] out (in/out).
 * n_tokens == 0 clears the segments, or with accumulate enqueues nothing.
 * Errors: as gc_linear_forward.
 */
gc_status gc_linear_grad_weight(const gc_plan *plan, const gc_linear *layer, const void *dz, uint64_t dz_stride,
                                const void *x, uint64_t x_stride, uint64_t n_tokens, float *g, int accumulate,
                                void *ws, size_t ws_bytes, hipStream_t stream);

/* ---------------------------------------------------------- distillation */
/*
 * Logits: n_rows rows of `vocab` elements of `type`, `stride` elements apart.
 * A logit of -Inf is a masked column.
 */
#define GC_MAX_VOCAB       (1u << 20)
#define GC_MAX_TOP_LOGITS  1024

/*
 * The top logits of every row, as a teacher sends them: the k entries first in
 * the order (value descending, index ascending) among the logits that are
 * neither NaN nor -Inf (+0 equals -0; exact, ties included).
 *   idx [n_rows][k] out: int32 columns; -1 behind a row's last entry.
 *   val [n_rows][k] out: the logits in fp32 (exact); -Inf there.
 *   lse [n_rows] out, or NULL: log sum_j exp(z_j / temperature) over the whole
 *     row (-Inf where every column is masked, NaN where one is NaN or +Inf).
 * n_rows == 0 enqueues nothing.
 * Errors: GC_EINVAL (null, unknown type, k = 0, stride < vocab, vocab = 0,
 *         temperature not positive, or it or log2(e) / temperature not finite
 *         in fp32, misaligned buffers), GC_ENOTSUP
 *         (vocab > GC_MAX_VOCAB, k > GC_MAX_TOP_LOGITS), GC_ERANGE (n_rows >=
 *         2^22, n_rows * stride > 2^48).
 */
gc_status gc_top_logits(const void *logits, int type, uint64_t stride, uint64_t n_rows, uint32_t vocab,
                        uint32_t k, float temperature, int32_t *idx, float *val, float *lse,
                        hipStream_t stream);

/*
 * The loss of a student's rows z against a teacher's top logits t_k at columns
 * c_k, and its gradient.  T = temperature, p = softmax(z / T).
 *   GC_DISTILL_TOP : q_k = exp(t_k / T) / sum of those (renormalised), q_r = 0
 *   GC_DISTILL_REST: q_k = exp(t_k / T - t_lse), q_r = max(0, 1 - sum_k q_k),
 *                    the mass of all columns that no entry names (p_r in the
 *                    student); where those are all masked, q_r = 0
 *   KL = sum_k q_k (log q_k - log p_{c_k}) + q_r (log q_r - log p_r)
 *        (a term with q = 0 is 0)
 *   loss = weight (kd_weight T^2 KL + ce_weight (log sum exp(z) - z_label))
 *   dlogits = grad_scale d loss / d z
 * An entry whose column lies outside [0, vocab), or whose t_k is -Inf, is no
 * entry; without any, or with kd_weight 0, there is no KL term.  Without a
 * label in [0, vocab), or with ce_weight 0, there is no label's term.  A row with
 * neither, or with weight 0, has loss 0 and a gradient of +0, whatever its logits
 * are.  A column that several entries name takes each of them.  In a row that
 * counts, a NaN or +Inf, or every column masked, makes the loss and the gradient
 * NaN; a masked column's gradient is +-0 unless the teacher or the label names
 * it, and if it does the loss is +Inf.
 *   idx [n_rows][idx_stride]: k int32 or int64 (idx_type GC_TOKENS_*); t
 *   [n_rows][t_stride]: k values of t_type; t_lse [n_rows] fp32 for
 *   GC_DISTILL_REST (gc_top_logits writes it, for the same T); labels [n_rows]
 *   of idx_type, or NULL; weights [n_rows] fp32, or NULL: 1.
 *   loss [n_rows] fp32 out.
 *   dlogits [n_rows][dstride] of `type` out, or NULL: the loss alone.  dlogits
 *     may be logits (with its stride).
 * k == 0 leaves the labels' term alone.  n_rows == 0 enqueues nothing.
 * Sums are fp32 (over the teacher's entries in double) in an order that the
 * sizes fix; their logarithms, within 2^-24, are combined in double.
 * Errors: as gc_top_logits; GC_EINVAL also for unknown types, a mode,
 *         kd_weight, ce_weight or grad_scale not finite, t_lse missing,
 *         reserved not 0.
 */
#define GC_DISTILL_TOP   0
#define GC_DISTILL_REST  1
typedef struct gc_distill_options {
    float    temperature;   /* > 0                */
    float    kd_weight;
    float    ce_weight;
    float    grad_scale;
    int      mode;          /* GC_DISTILL_*       */
    uint32_t reserved[3];   /* must be 0          */
} gc_distill_options;
gc_status gc_distill_loss(const void *logits, int type, uint64_t stride, uint64_t n_rows, uint32_t vocab,
                          const void *idx, int idx_type, uint64_t idx_stride, const void *t, int t_type,
                          uint64_t t_stride, uint32_t k, const float *t_lse, const void *labels,
                          const float *weights, const gc_distill_options *opt, float *loss, void *dlogits,
                          uint64_t dstride, hipStream_t stream);

/* ----------------------------------------------------------- measurement */
/*
 * Kernel timing for measurement tools (off by default).  While enabled, each
 * launch of a selected kernel is bracketed by a pair of HIP events recorded
 * on the caller's stream; nothing else changes.
 *   kernels : comma-separated kernel names ("dgc_update,ada_apply"), "*" for
 *             all, NULL or "" to disable.  Names: dgc_norm, dgc_prep,
 *             dgc_sample, dgc_bound, dgc_ssample, dgc_squant, dgc_update,
 *             dgc_select, dgc_stage, dgc_refine, dgc_sbase, dgc_count,
 *             dgc_scan, dgc_emit, ada_max, ada_binsum, ada_scale, ada_offsets,
 *             ada_apply, ada_fold, ada_emit, ada_residual,
 *             pack_tiles, pack_count, pack_layout, pack_write, unpack_walk,
 *             unpack_count, unpack_scan, unpack_write, decode_index,
 *             decode, dcd, dcd_decode, dcd_mix, ecd_compress, ecd_update,
 *             slimdp_values, stream_probe (Slim-DP selection reuses the
 *             dgc_* names), embed_lookup, embed_rank, embed_merge,
 *             embed_heads, embed_rows, embed_sum, embed_join, embed_small,
 *             embed_empty,
 *             orth_norm, orth_scale, orth_split, orth_gram, orth_poly,
 *             orth_pair, orth_apply, orth_join, orth_slab, orth_small,
 *             linear_product, linear_few, linear_join, act_grad, top_logits, distill.
 * gc_timing_take waits for the recorded events of one kernel and returns the
 * summed duration in milliseconds and the number of launches, then forgets
 * them.  Host-thread safe; not for use while a stream is being captured.
 */
gc_status gc_timing_enable(const char *kernels);
gc_status gc_timing_take(const char *kernel, double *total_ms, uint64_t *launches);

/*
 * A streaming reference for measurement tools, not part of any method:
 * d[i] = a[i] + b[i] and e[i] = c[i] + d[i] (fp32) for i < n, that is three
 * reads and two writes per element, the HBM traffic of the DGC update, in
 * the same chunk tiling, lane layout and cache hints as the dense kernels
 * and with none of their other work.  Timed beside dgc_update it gives the
 * bandwidth that access pattern reaches on the device.
 *   a, b, c : device, n floats each, read.   d, e : device, n floats each,
 *             written; they must not overlap each other or the inputs.
 *   n       : below 2^32; 0 enqueues nothing.
 * All pointers 4-byte aligned.  Errors (GC_EINVAL null or misaligned
 * pointer, GC_ERANGE n) are detected before anything is enqueued.
 * Asynchronous on `stream`.
 */
gc_status gc_stream_probe(const float *a, const float *b, const float *c, float *d, float *e, uint64_t n,
                          hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* GRADCOMP_H */
