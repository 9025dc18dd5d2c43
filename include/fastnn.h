/*
 * fastnn.h -- C ABI of the B200 (sm_100a) reciprocal nearest-neighbour
 * matcher for dense per-pixel descriptor maps (MASt3R's matching step).
 *
 * What is computed
 *   Similarity of two descriptors is their dot product; the nearest
 *   neighbour of a query in a database is argmax_k <q, db_k>, the LOWEST k
 *   among equal scores ("MASt3R dissection", section 3 Napkin Formula: the
 *   inference-time reciprocal set is written with argmax of dot products).
 *   A reciprocal match is a pair (i, j) with NN(D1[i], D2) = j and
 *   NN(D2[j], D1) = i ("MASt3R dissection", section 1 architecture diagram
 *   and section 3).
 *   Pointmaps (dtype FASTNN_F32_L2): rows are 3D points and the nearest
 *   neighbour is the nearest point, argmin_k |q - db_k|^2, lowest k on ties
 *   ("DUSt3R / MASt3R explained", the paragraph on recovering the cameras:
 *   pixels match when their predicted 3D points are nearest neighbours in
 *   the shared frame). The same reciprocal and fast schemes apply.
 *
 * Conventions shared by every entry point
 *   - Every data pointer is a DEVICE pointer owned by the caller. The library
 *     allocates no memory: scratch lives in a caller-provided workspace whose
 *     size comes from fastnn_workspace_size(). Workspace and descriptor
 *     pointers must be 256-byte aligned.
 *   - Descriptor maps are row-major [rows][d] (an image is [H][W][d], pixel
 *     index p = y * W + x); batches are [batch][rows][d].
 *   - dtype FASTNN_I8: int8 descriptors, int32 scores (exact).
 *     dtype FASTNN_BF16 / FASTNN_F16: bfloat16 / IEEE half descriptors (raw
 *     16-bit patterns), float32 scores (fp32 accumulation of exact products).
 *     1 <= d <= 64 for all three (d <= 32 runs one 32-element K step).
 *     dtype FASTNN_F32_L2: float32 points, 1 <= d <= 3 (DUSt3R pointmaps
 *     have d = 3); scores are float32 SQUARED DISTANCES (lower is nearer).
 *     Inputs must be finite. The squared distance of a point is computed in
 *     fp64 from the coordinate differences, (dx^2 + dy^2) + dz^2 with one
 *     rounding per operation, and rounded to fp32; the nearest point is the
 *     lowest index among those whose fp32 value is the smallest. (The
 *     kernels scan with fp32 scores 2<q, p> - |p|^2 and re-rank every point
 *     their rounding error could place first.)
 *   - Every call is asynchronous on `stream` (a cudaStream_t; NULL is the
 *     legacy default stream). The host blocks only in fastnn_device_status().
 *   - Return value: FASTNN_OK, or a negative fastnn_status describing an
 *     argument or launch error detected on the host; nothing has been
 *     enqueued when an argument error is returned. Errors found on the
 *     device (a bounded wait that ran out) are recorded in the workspace and
 *     read with fastnn_device_status().
 *   - Calls that share a workspace must be ordered (same stream or events);
 *     overlapping calls on one workspace race.
 */
#ifndef FASTNN_H_
#define FASTNN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st *fastnn_stream_t; /* same type as cudaStream_t */

typedef enum {
    FASTNN_OK = 0,
    FASTNN_ERR_INVALID = -1,     /* bad pointer, size, alignment or argument */
    FASTNN_ERR_UNSUPPORTED = -2, /* d (1..64; 1..3 for pointmaps) or dtype not taken */
    FASTNN_ERR_CAPACITY = -3,    /* output capacity or workspace too small */
    FASTNN_ERR_CUDA = -4,        /* a CUDA runtime call or launch failed */
    FASTNN_ERR_TIMEOUT = -5      /* a device-side bounded wait ran out */
} fastnn_status;

typedef enum {
    FASTNN_I8 = 0,     /* int8 descriptors, dot product, int32 scores */
    FASTNN_BF16 = 1,   /* bfloat16 descriptors, dot product, float32 scores */
    FASTNN_F16 = 2,    /* IEEE half descriptors, dot product, float32 scores */
    FASTNN_F32_L2 = 3  /* float32 3D points, Euclidean distance, float32 squared distances */
} fastnn_dtype;

typedef enum {
    FASTNN_OP_NN = 0,
    FASTNN_OP_RECIPROCAL = 1,
    FASTNN_OP_MUTUAL_DENSE = 2,
    FASTNN_OP_MUTUAL_FROM_NN = 3,
    FASTNN_OP_RECIPROCAL_MASKED = 4,
    FASTNN_OP_MUTUAL_DENSE_MASKED = 5,
    FASTNN_OP_IMAGE_ROWS = 6
} fastnn_op;

/*
 * Workspace bytes one call needs.
 *   FASTNN_OP_NN:           n1 = nq, n2 = ndb (batch and max_queries unused)
 *   FASTNN_OP_RECIPROCAL:   n1 = H1*W1, n2 = H2*W2, max_queries = number of
 *                           grid seeds per pair, batch = pairs
 *   FASTNN_OP_MUTUAL_DENSE: n1, n2 = pixel counts (batch, max_queries unused)
 *   FASTNN_OP_MUTUAL_FROM_NN: n1 = local image-1 rows, n2 = image-2 rows
 *                           (d must still be valid for dtype; unused)
 *   FASTNN_OP_RECIPROCAL_MASKED, FASTNN_OP_MUTUAL_DENSE_MASKED: as the
 *                           unmasked ops
 *   FASTNN_OP_IMAGE_ROWS:   n1 = entries of nn12, n2 = image-2 rows (d must
 *                           still be valid for dtype; unused)
 * Returns 0 for arguments no call would accept.
 */
size_t fastnn_workspace_size(int op, int64_t n1, int64_t n2, int d, int dtype,
                             int batch, int64_t max_queries);

/*
 * fastnn_nn -- nearest neighbour of every query row in a database.
 *   For i < nq: out_idx[i] = argmax_k <q[i], db[k]> (lowest k on ties),
 *   out_score[i] = that score (int32 for FASTNN_I8, float for the float
 *   types; out_score may be NULL). For FASTNN_F32_L2, out_idx[i] is the
 *   nearest point and out_score[i] its squared distance. This is the primitive of both matching schemes
 *   ("MASt3R dissection", section 3, argmax of dot products).
 *   q: [nq][d], db: [ndb][d]; nq >= 0, ndb >= 1; nq == 0 is a no-op.
 */
int fastnn_nn(const void *q, int64_t nq, const void *db, int64_t ndb, int d,
              int dtype, int32_t *out_idx, void *out_score, void *workspace,
              size_t workspace_bytes, fastnn_stream_t stream);

/*
 * fastnn_reciprocal -- MASt3R fast reciprocal matching ("DUSt3R / MASt3R
 * explained", the paragraph on fast reciprocal matching: seeds on a sparse
 * grid of image 1 are mapped to their best match in image 2 and back; pixels
 * that map onto themselves are kept; the others walk on).
 *   Seeds: pixels (x, y) of image 1 with x, y multiples of `subsample`
 *   (origin 0), S = ceil(H1/subsample) * ceil(W1/subsample) per pair.
 *   Round t = 1..max_iter while the frontier is non-empty: for u in the
 *   frontier, v = NN(D1[u], D2), u' = NN(D2[v], D1); u' == u keeps (u, v);
 *   otherwise u' joins the next frontier unless it was already in any
 *   frontier of this call (a pruning that leaves the kept set unchanged: the
 *   walk from a pixel is deterministic, and its first visit is the furthest
 *   ahead). Walks still open after max_iter rounds are dropped.
 *   desc1: [batch][H1][W1][d], desc2: [batch][H2][W2][d]; pairs independent.
 *   out_pairs: [batch][capacity][2] int32 (u, v) pixel indices in order of
 *   discovery (round, then frontier position); out_score: [batch][capacity]
 *   (int32 or float) or NULL; out_count: [batch] int32 pairs written per
 *   pair; out_iters: [batch] int32 rounds run with a non-empty frontier, or
 *   NULL; out_frontier: [batch][max_iter] int32 frontier size of each round
 *   (0 for rounds not run), or NULL. capacity must be >= S (at most one pair
 *   per seed), else
 *   FASTNN_ERR_CAPACITY. 1 <= subsample, 1 <= max_iter <= 255, S < 2^24.
 */
int fastnn_reciprocal(const void *desc1, int H1, int W1, const void *desc2,
                      int H2, int W2, int d, int dtype, int subsample,
                      int max_iter, int batch, int32_t *out_pairs,
                      void *out_score, int64_t capacity, int32_t *out_count,
                      int32_t *out_iters, int32_t *out_frontier,
                      void *workspace, size_t workspace_bytes,
                      fastnn_stream_t stream);

/*
 * fastnn_mutual_dense -- every mutual nearest-neighbour pair of two maps,
 * the brute-force reciprocal set ("MASt3R dissection", section 1 and section
 * 3; "DUSt3R / MASt3R explained" calls it the naive every-pixel-against-
 * every-pixel comparison that the fast scheme avoids).
 *   desc1: [n1][d], desc2: [n2][d]. Output pairs (i, j) in ascending i into
 *   out_pairs [capacity][2] int32 and out_score [capacity] (or NULL);
 *   *out_count (device int32) = number of pairs. capacity must be
 *   >= min(n1, n2), else FASTNN_ERR_CAPACITY.
 *   Work: NN12 for every row of desc1, then NN21 only for the rows of desc2
 *   that are some row's NN12 (no other row can be in a mutual pair).
 */
int fastnn_mutual_dense(const void *desc1, int64_t n1, const void *desc2,
                        int64_t n2, int d, int dtype, int32_t *out_pairs,
                        void *out_score, int64_t capacity, int32_t *out_count,
                        void *workspace, size_t workspace_bytes,
                        fastnn_stream_t stream);

/*
 * fastnn_mutual_from_nn -- the mutual test of the reciprocal set ("MASt3R
 * dissection", section 1 and section 3) applied to nearest-neighbour indices
 * that were computed elsewhere, for a row shard of image 1: local row i (global
 * row i0 + i) with partner j = nn12[i] is kept iff nn21[j] == i0 + i. This is
 * the last step of the dense mutual set when image 1's rows are split across
 * GPUs and nn21 (all n2 image-2 rows, global image-1 indices) was gathered.
 *   nn12: [n1] int32 in [0, n2); score12: [n1] int32/float or NULL;
 *   nn21: [n2] int32 in [0, n1_total), or -1 for a row with no partner (a row
 *   outside the image of NN12, see fastnn_image_rows). Output (i0 + i, j) in
 *   ascending i into
 *   out_pairs [capacity][2], scores into out_score (or NULL), *out_count =
 *   pairs. capacity >= min(n1, n2). n1 == 0 writes *out_count = 0.
 */
int fastnn_mutual_from_nn(const int32_t *nn12, const void *score12, int64_t n1,
                          int64_t i0, const int32_t *nn21, int64_t n2,
                          int64_t n1_total, int dtype, int32_t *out_pairs,
                          void *out_score, int64_t capacity, int32_t *out_count,
                          void *workspace, size_t workspace_bytes,
                          fastnn_stream_t stream);

/*
 * fastnn_image_rows -- the image-2 rows that can be in a mutual pair: a pair
 * (i, j) of the reciprocal set ("MASt3R dissection", section 1 and section 3)
 * has j = NN12(i), so only the rows some image-1 row matches need their own
 * nearest neighbour in image 1. Writes the distinct values of nn12 that lie
 * in [0, n2), in ascending order, to out_rows[0 .. *out_count) (device int32);
 * out_rows must hold min(n1, n2) entries. When image 1's rows are split
 * across GPUs, the gathered NN12 of all of them gives every rank the same
 * list, whose rows are then split for the backward pass.
 *   nn12: [n1] int32 (may be NULL when n1 == 0; values outside [0, n2) are
 *   ignored). Workspace: FASTNN_OP_IMAGE_ROWS.
 */
int fastnn_image_rows(const int32_t *nn12, int64_t n1, int64_t n2,
                      int32_t *out_rows, int32_t *out_count, void *workspace,
                      size_t workspace_bytes, fastnn_stream_t stream);

/*
 * fastnn_set_wait_timeout_ns -- limit of the kernels' bounded waits for the
 * calls that follow (process-wide; 0 restores the default of 2 s). Every wait
 * inside the kernels (a pipeline stage, an accumulator, a grid barrier) gives
 * up after this long: the kernel then stops issuing work, drains what it has
 * in flight (those waits always use the 2 s default), frees its tensor
 * memory and returns, and fastnn_device_status() reports FASTNN_ERR_TIMEOUT;
 * the outputs of that call are undefined, the context stays usable. Meant
 * for supervision and for testing that failure path (a limit far below a
 * call's duration makes its waits run out); the pages have no counterpart.
 */
void fastnn_set_wait_timeout_ns(uint64_t ns);

/*
 * Confidence-masked matching. The network predicts a confidence beside every
 * per-pixel output ("DUSt3R / MASt3R explained", the pointmap paragraph), and
 * the remedy for pixels whose geometry cannot be trusted is to mask them or
 * reject their low-confidence matches ("MASt3R dissection", section 5).
 * Here a pixel takes part iff conf >= conf_threshold: it is a candidate in
 * its image's database and, if on the seed grid, a seed; other pixels are
 * neither. Without a confidence map (NULL) every pixel of that image takes
 * part. Reported indices are pixel indices of the full maps; everything else
 * (tie rule, order of the output, scores, capacities, errors) is that of the
 * unmasked call. The kept pixels are compacted on the device, in pixel order,
 * before matching; confidences must not be NaN for pixels meant to be kept.
 *   conf1: [batch][H1][W1] float32 or NULL; conf2: [batch][H2][W2] or NULL.
 *   Workspace: FASTNN_OP_RECIPROCAL_MASKED (or _MUTUAL_DENSE_MASKED) sizes.
 *   capacity >= S (fast) / min(n1, n2) (dense) as for the unmasked calls;
 *   out_frontier counts kept seeds in round 1. A pair whose image 2 keeps no
 *   pixel runs one round and keeps nothing.
 */
int fastnn_reciprocal_masked(const void *desc1, const float *conf1, int H1,
                             int W1, const void *desc2, const float *conf2,
                             int H2, int W2, int d, int dtype,
                             float conf_threshold, int subsample, int max_iter,
                             int batch, int32_t *out_pairs, void *out_score,
                             int64_t capacity, int32_t *out_count,
                             int32_t *out_iters, int32_t *out_frontier,
                             void *workspace, size_t workspace_bytes,
                             fastnn_stream_t stream);

int fastnn_mutual_dense_masked(const void *desc1, const float *conf1, int64_t n1,
                               const void *desc2, const float *conf2,
                               int64_t n2, int d, int dtype,
                               float conf_threshold, int32_t *out_pairs,
                               void *out_score, int64_t capacity,
                               int32_t *out_count, void *workspace,
                               size_t workspace_bytes, fastnn_stream_t stream);

/*
 * fastnn_reciprocal_noalloc -- fastnn_reciprocal for callers that cannot
 * allocate device memory (a plugin inside an application that owns every
 * allocation, a real-time loop that must not take cudaMalloc's implicit
 * synchronisation, a fixed pre-reserved memory budget). The pages describe no
 * such entry point: it is a property of this library, with no counterpart in
 * the method.
 *   Arguments and results are those of fastnn_reciprocal without the
 *   workspace: the scratch is a static device array of
 *   FASTNN_NOALLOC_SCRATCH_BYTES (32 MiB) that every GPU loading this library
 *   holds until the process exits. Calls whose workspace would exceed it
 *   (fastnn_workspace_size) return FASTNN_ERR_CAPACITY and enqueue nothing;
 *   one 512x384 pair with int8 or bf16 descriptors fits.
 *   The first call on a device looks up the array's device address
 *   (cudaGetSymbolAddress) with that device current; make that first call
 *   before any stream capture. The call allocates nothing.
 *   All calls share the one array and it keeps the last call's contents (the
 *   call clears what must start at zero). Calls that overlap on the GPU (on
 *   different streams, or from several host threads without ordering) race on
 *   it. Argument errors are returned before anything is enqueued, with the
 *   statuses fastnn_reciprocal gives; a device-side bounded wait that ran out
 *   is read with fastnn_noalloc_device_status().
 */
#define FASTNN_NOALLOC_SCRATCH_BYTES (32u << 20)

int fastnn_reciprocal_noalloc(const void *desc1, int H1, int W1, const void *desc2,
                              int H2, int W2, int d, int dtype, int subsample,
                              int max_iter, int batch, int32_t *out_pairs,
                              void *out_score, int64_t capacity,
                              int32_t *out_count, int32_t *out_iters,
                              int32_t *out_frontier, fastnn_stream_t stream);

/*
 * fastnn_noalloc_device_status -- synchronise `stream` and read the device
 * status word that the last fastnn_reciprocal_noalloc call on the CURRENT
 * device left in the static scratch array: FASTNN_OK, or FASTNN_ERR_TIMEOUT
 * when one of that call's bounded waits ran out (its outputs are then
 * invalid). Blocks the host. If no allocation-free call has run on this
 * device yet, the first use looks up the array's address (as the first
 * allocation-free call does). Like the array itself, this has no counterpart
 * in the pages.
 */
int fastnn_noalloc_device_status(fastnn_stream_t stream);

/*
 * The token store: soft matching of one image's tokens (descriptors, patch
 * features) with those of the earlier images of its stream.
 *
 * fastnn_nn answers a query with the one database row of the largest dot
 * product. The calls below keep the rows of many images in a paged store and
 * answer a query with the softmax-weighted mean of the stored values under
 * the same dot products:
 *   out[t, h] = sum_p w_p value[p],  w_p = exp(scale <q[t, h], key[p]> - lse)
 * over the positions p of the token's own sequence (stream) that it sees.
 *
 * fastnn_store describes the store and one ragged batch of new tokens. Page
 * ids are physical; position p of sequence s lives in row p % page of page
 * page_table[s][p / page]. Tokens cu[s] .. cu[s + 1] - 1 of the batch belong
 * to sequence s. Query heads share key heads in equal groups: head h of q
 * reads key head h / (heads_q / heads). All index arrays are device int32;
 * they are read on the device only, so a captured graph follows their
 * contents. dtype is FASTNN_BF16 or FASTNN_F16 for keys, values, means,
 * queries and outputs alike. k_pages, v_pages and k_mean are contiguous and
 * 16-byte aligned. The current device is the one that holds them all. A batch
 * has at most 2^30 tokens, max_new (where n > 0) is 1 .. n.
 *
 * What the index arrays may hold (checked on the device, never read out of
 * range): a page id outside [0, n_pages) is a hole, whose positions do not
 * exist; positions past table_width * page do not exist; of a sequence with
 * more than max_new new tokens only the first max_new are taken; tokens at or
 * past cu[n_seqs] are left as they are, in the outputs too.
 */
typedef struct {
    void *k_pages;             /* [n_pages][heads][page][d] keys */
    void *v_pages;             /* [n_pages][heads][page][dv] values */
    void *k_mean;              /* [n_pages][heads][d] mean key of each page, or NULL */
    const int32_t *page_table; /* [n_seqs][table_width] physical page ids */
    const int32_t *lens;       /* [n_seqs] positions held (each call says when) */
    const int32_t *cu;         /* [n_seqs + 1] first new token of each sequence */
    int64_t n_pages;           /* >= 1 */
    int n_seqs;                /* 1 .. 65534 */
    int table_width;           /* >= 1; table_width * page < 2^31 - 256 */
    int page;                  /* positions in a page: 16, 32, 64 or 128 */
    int heads;                 /* key / value heads, 1 .. 1024 */
    int d;                     /* key elements: a multiple of 8, 8 .. 128 */
    int dv;                    /* value elements: a multiple of 8, 8 .. 128 */
    int dtype;                 /* FASTNN_BF16 or FASTNN_F16 */
} fastnn_store;

/* How the pairs that turn together lie in the rotated elements of one axis:
 * element j with j + half, or 2j with 2j + 1. */
typedef enum {
    FASTNN_ROTARY_HALF = 0,
    FASTNN_ROTARY_INTERLEAVED = 1
} fastnn_rotary_layout;

/*
 * A position rotation. The first `rot` elements of a row are cut into `axes`
 * equal parts, one for each position axis (a pixel has two); pair j of part a
 * turns by the angle pos[token][a] * freq[j] (radians, formed in fp64, so that
 * far positions keep their angle) and is multiplied by `scale`; the elements
 * after `rot` stay. Scaled positions (for axes longer than those seen in
 * training) are a matter of the freq table, and `scale` is the amplitude that
 * some of them carry.
 */
typedef struct {
    const int32_t *pos;  /* [tokens][axes] */
    const double *freq;  /* [rot / (2 * axes)] radians per position */
    int axes;            /* 1 or 2 */
    int rot;             /* a multiple of 2 * axes, at most d; 0 = no rotation */
    int layout;          /* fastnn_rotary_layout */
    float scale;         /* finite */
} fastnn_rotation;

/*
 * fastnn_rotary -- rotate the rows of x [n][heads][d] into out (same shape).
 *   inverse != 0 turns by the negative angles (times the same scale): the
 *   transposed map, which carries a gradient of out back to x.
 *   Tokens are x_stride (out_stride) elements apart, heads d elements.
 *   out may be x itself (same pointer and stride), else they must not
 *   overlap. Computed in fp32 and rounded once. 1 <= d <= 1024, any alignment
 *   (16-byte aligned rows are read widest). n == 0 is a no-op.
 */
int fastnn_rotary(const void *x, int64_t x_stride, int64_t n, int heads, int d,
                  int dtype, const fastnn_rotation *rotation, int inverse,
                  void *out, int64_t out_stride, fastnn_stream_t stream);

/*
 * fastnn_store_append -- put new keys and values into the store.
 *   store->lens are the positions held BEFORE the call: token i of sequence s
 *   becomes position lens[s] + i. k [n][heads][d] (token stride k_stride) is
 *   rotated on the way (rotation may be NULL), computed in fp32 and rounded
 *   once; v [n][heads][dv] (v_stride) is copied.
 *   If store->k_mean is given, the mean of every page that receives a token is
 *   written anew: the mean over the keys the page then holds, as stored,
 *   summed in fp32 and rounded once. Untouched pages keep theirs.
 *   The caller advances lens. Pages that receive tokens must not be shared by
 *   two sequences of the batch. k and v rows 16-byte aligned.
 *   A new token that has no place (a hole, or a position past the table) is
 *   not stored; fastnn_device_status() then reports FASTNN_ERR_INVALID, as it
 *   does for a sequence with a negative length or more than max_new tokens.
 *   workspace: FASTNN_STORE_APPEND_WORKSPACE bytes for that report, or NULL
 *   (nothing is reported). n == 0 is a no-op.
 */
#define FASTNN_STORE_APPEND_WORKSPACE 256
int fastnn_store_append(const fastnn_store *store, const void *k, int64_t k_stride,
                        const void *v, int64_t v_stride, int64_t n, int max_new,
                        const fastnn_rotation *rotation, void *workspace,
                        size_t workspace_bytes, fastnn_stream_t stream);

/*
 * fastnn_attend -- attention of the batch's tokens over their sequences.
 *   store->lens are the positions held INCLUDING the batch's tokens (append
 *   first). Token i of the n_s new tokens of sequence s sees positions below
 *   lens[s] (causal == 0) or below lens[s] - n_s + i + 1 (causal != 0).
 *   q [n][heads_q][d], token stride q_stride, rows 16-byte aligned; heads_q a
 *   multiple of store->heads; max_new * heads_q / heads < 2^31 - 16. out
 *   [n][heads_q][dv] contiguous; lse (or NULL)
 *   [n][heads_q] float32, the natural logarithm of the sum of the
 *   exponentials. A token that sees nothing gets out = 0, lse = -infinity.
 *   Products and sums in fp32; the weights of the second product are rounded
 *   to dtype (half a step: relative 2^-8 for bf16, 2^-11 for half), and out is
 *   rounded once. For values of mixed sign the two roundings are of one size:
 *   the error of out is then about sqrt(2) times that of one rounding.
 *   Keys and values at positions that some token of the call sees must be
 *   finite; what lies behind lens in a page is never used. NaN in a row of q
 *   makes that row of out and lse NaN (where it sees anything), and no other.
 *   pages (or NULL): [n][heads][select] logical page numbers (position / page),
 *   as fastnn_select_pages writes them: the token then sees only the positions
 *   of the pages listed for its key head. Entries outside its sequence's pages
 *   are skipped; a page that is listed twice counts twice.
 *   workspace: fastnn_attend_workspace_size() with the same arguments (256-byte
 *   aligned); where that is 256, for the status word alone, it may be NULL.
 *   n == 0 is a no-op.
 */
size_t fastnn_attend_workspace_size(const fastnn_store *store, int64_t n, int heads_q,
                                    int max_new, int select);
int fastnn_attend(const fastnn_store *store, const void *q, int64_t q_stride, int64_t n,
                  int heads_q, int max_new, int causal, float scale, const int32_t *pages,
                  int select, void *out, float *lse, void *workspace,
                  size_t workspace_bytes, fastnn_stream_t stream);

/*
 * fastnn_select_pages -- the pages worth a query's attention, by a cheap score.
 *   For each token t and key head g: the score of a page is the sum over the
 *   query heads of the group of <q[t, h], k_mean[page]>; the token's first
 *   keep_first and last keep_last visible pages are taken whatever their
 *   score, the best others fill up to `select`. out_pages [n][heads][select]
 *   int32: their logical numbers in ascending order, -1 behind the last.
 *   Visible lengths are those of fastnn_attend (lens including the batch);
 *   holes are never taken. The order of the scores is that of their fp64
 *   values; among equal ones the lowest page is first; a NaN score is last.
 *   Under causal, keep_last >= 1 keeps the mean of the page that holds the
 *   token's own future out of the choice, so 1 <= keep_last; keep_first +
 *   keep_last <= select <= 256. store->v_pages and k_pages are not read (may
 *   be NULL); dv is not used but must be valid.
 *   workspace: fastnn_select_workspace_size() bytes, 256-byte aligned; may be
 *   NULL where that is 256.
 */
size_t fastnn_select_workspace_size(const fastnn_store *store, int64_t n, int heads_q,
                                    int max_new);
int fastnn_select_pages(const fastnn_store *store, const void *q, int64_t q_stride,
                        int64_t n, int heads_q, int max_new, int causal, int keep_first,
                        int keep_last, int select, int32_t *out_pages, void *workspace,
                        size_t workspace_bytes, fastnn_stream_t stream);

/*
 * fastnn_device_status -- synchronise `stream` and read the device status
 * word of the last call that used `workspace`: FASTNN_OK, or
 * FASTNN_ERR_TIMEOUT when a kernel's bounded wait ran out (its outputs are
 * then invalid), FASTNN_ERR_INVALID when fastnn_store_append met index arrays
 * that leave a new token without a place. Blocks the host.
 */
int fastnn_device_status(const void *workspace, fastnn_stream_t stream);

/*
 * Benchmark instrumentation (not needed for matching). After
 * fastnn_kernel_timer_enable(capacity > 0), each of the next `capacity`
 * launches of the selected kinds (fastnn_kernel_timer_select below; by
 * default the nearest-neighbour and matching kernels) is bracketed by two
 * CUDA events recorded on the launching stream (events are created here, once,
 * not per call). fastnn_kernel_timer_read() waits for the recorded events,
 * returns the number of timed launches and their summed device time in
 * milliseconds, and starts a new count. fastnn_kernel_timer_enable(0)
 * destroys the events. Process-wide state: not for concurrent use from
 * several host threads.
 */
int fastnn_kernel_timer_enable(int capacity);
int fastnn_kernel_timer_read(int *launches, double *total_ms);

/*
 * fastnn_kernel_timer_select -- which launches the timer above brackets, as a
 * bit mask (each bracket covers the kernels one call of that kind launches):
 *   FASTNN_TIME_MATCHING (1, the default): the tensor-core and pointmap
 *     nearest-neighbour kernels and the persistent matching kernels;
 *   FASTNN_TIME_REPACK (2): the repack of each descriptor map;
 *   FASTNN_TIME_MUTUAL (4): the dense mutual test and ordered emit (count,
 *     scan, emit), and the list of image-2 rows the dense backward pass runs on;
 *   FASTNN_TIME_MASK (8): the confidence-mask compaction of each map.
 * kinds <= 0 leaves the selection as it is. Returns the previous selection.
 * Benchmark instrumentation: process-wide, like the timer itself.
 */
#define FASTNN_TIME_MATCHING 1
#define FASTNN_TIME_REPACK 2
#define FASTNN_TIME_MUTUAL 4
#define FASTNN_TIME_MASK 8
int fastnn_kernel_timer_select(int kinds);

/* Text of the last CUDA runtime error this library saw on the calling host
 * thread (the cause behind a FASTNN_ERR_CUDA return); a static string. */
const char *fastnn_last_cuda_error(void);

/* Human-readable name of a fastnn_status value (static string). */
const char *fastnn_status_str(int status);

#ifdef __cplusplus
}
#endif

#endif /* FASTNN_H_ */
