/*
 * lapmix -- the operators that stand beside the attention of lapnys.h in a
 * model: a gated linear recurrence (a linear-time causal token mixer) and the
 * root-mean-square norm with the residual's addition, each forward, backward
 * and for single tokens.  Part of liblapnys.so; status codes, storage types
 * (LAPNYS_F32, LAPNYS_BF16) and lapnys_status_string are those of lapnys.h.
 *
 * Recurrence, for every batch b, head h and channel c on its own:
 *
 *   h_t = f_t h_{t-1} + i_t x_t,   y_t = h_t,   t = 0 .. N-1,  h_{-1} = h0
 *   f = sigmoid(g), or with LAPMIX_GATE_LOG f = exp(min(g, 0))
 *   i = 1, or with LAPMIX_COUPLED i = 1 - f
 *
 * A gate of -infinity is f = 0: the token starts anew (documents packed one
 * behind the other).  Backward, of sum(dy * y) + sum(dhN * hN):
 *
 *   dh_t = dy_t + f_{t+1} dh_{t+1}   (dh_{N-1} = dy_{N-1} + dhN)
 *   dx = i dh,  dh0 = f_0 dh_0,  df = dh h_{t-1}  (LAPMIX_COUPLED: dh (h_{t-1} - x))
 *   dg = df f (1 - f), or with LAPMIX_GATE_LOG df f where g <= 0 and 0 elsewhere
 *
 * Norm, for every token's row of C = H * d columns (column h * d + c is
 * channel c of head h):
 *
 *   s = x + r                      rounded once to r's type (without r: x alone)
 *   y = s / sqrt(mean(s^2) + eps) * w      of s as it is stored
 *   e4m3: scale = max|y| / 448 over each group of columns, y / scale rounded
 *
 * Backward, of sum(dy * y) + sum(ds * s), with u = s / sqrt(mean(s^2) + eps):
 *
 *   dr = (w dy - u mean(w dy u)) / sqrt(mean(s^2) + eps) + ds,  dx = dr,
 *   dw = the sum over the rows of dy u
 *
 * Layouts.  Tensors of the recurrence, and the norm's x and dx, are
 * [B, H, N, d] with channels contiguous and a stride in elements for batches,
 * heads and tokens each, so [B, N, H, d] memory and slices of a projection's
 * output need no copy; strides of all zero mean dense C order.  Strides are
 * at least 0; elements of a tensor that is written may not coincide, inputs
 * may repeat (stride 0).  r, s, y, dy, ds and dr of the norm are dense
 * [B, N, C].  Base addresses need the alignment of an element; the kernels are
 * fastest where d and the strides are multiples of 4 elements (for the norm of
 * 8) and bases of 16 bytes.
 *
 * Precision: inputs widen exactly to float32; gates, states, products, norms
 * and their sums are float32; each output is rounded once, to nearest even.
 * Results do not depend on how work is scheduled: two calls on the same
 * inputs give the same bits.
 *
 * Ownership, streams and errors are those of lapnys.h: pointers belong to the
 * caller, work is enqueued on `stream` without synchronising, on a validation
 * error nothing is enqueued.  Every call can be captured into a graph.
 */
#ifndef LAPMIX_H_
#define LAPMIX_H_

#include "lapnys.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Storage of the norm's y only: 8-bit floats of 4 exponent and 3 fraction
 * bits without infinities (OCP e4m3), with float32 scales. */
enum { LAPMIX_E4M3 = 2 };

/* Recurrence flags (see above). */
enum { LAPMIX_GATE_LOG = 1u, LAPMIX_COUPLED = 2u };

/* The forward can keep the state before every LAPMIX_SCAN_TILE-th token for
 * the backward pass. */
#define LAPMIX_SCAN_TILE 128

typedef struct {
  int32_t B, H, N, d;   /* batches, heads, tokens (up to 2^30), channels
                           (B * H * d up to 2^28; beyond: LAPNYS_ERR_UNSUPPORTED) */
  int32_t dtype;        /* lapnys_dtype of x, g, y, dy, dx and dg */
  uint32_t flags;       /* LAPMIX_GATE_LOG | LAPMIX_COUPLED, or 0 */
  int64_t x_stride[3];  /* of x and dx: batch, head, token, in elements */
  int64_t g_stride[3];  /* of g and dg */
  int64_t y_stride[3];  /* of y and dy */
} lapmix_scan_params;

typedef struct {
  int32_t B, H, N, d;   /* B * N rows of H * d columns */
  int32_t x_dtype;      /* lapnys_dtype of x and dx */
  int32_t r_dtype;      /* lapnys_dtype of r, s, ds and dr */
  int32_t y_dtype;      /* lapnys_dtype of y and dy, or LAPMIX_E4M3 */
  int32_t group;        /* LAPMIX_E4M3: columns to a scale, a power of two
                           from 16 to 512 that divides H * d, 0 = the row */
  float eps;            /* > 0 */
  int32_t reserved;     /* 0 */
  int64_t x_stride[3];  /* of x and dx: batch, head, token, in elements */
} lapmix_norm_params;

/* Device workspace (bytes, possibly 0) of the recurrence's forward and
 * backward calls: host-only arithmetic, *bytes is written only on success.
 * Workspaces follow lapnys_forward_ws's rules: 256-byte aligned, contents on
 * entry do not matter, calls that share one must be ordered (two graphs that
 * are replayed at once need one each). */
int lapmix_scan_workspace_size(const lapmix_scan_params* p, size_t* bytes);

/* Bytes of the states that the forward keeps for the backward:
 * float32 [B, H, ceil(N / LAPMIX_SCAN_TILE), d]. */
int lapmix_scan_states_size(const lapmix_scan_params* p, size_t* bytes);

/* Forward.  h0: float32 [B, H, d], or NULL for zeros.  lengths: int32 [B] on
 * the device, or NULL; sequence b has its first lengths[b] tokens (values
 * outside 0 .. N count as the nearer end), later x and g are not read, later
 * y are written as 0.  hN: float32 [B, H, d], the state after the last token
 * (h0 for an empty sequence), or NULL; it may be h0 itself.  states: see
 * lapmix_scan_states_size, or NULL.  Outputs overlap neither each other, the
 * inputs nor ws (but hN may be h0). */
int lapmix_scan_forward_ws(const void* x, const void* g, const float* h0, const int32_t* lengths, void* y,
                           float* hN, float* states, const lapmix_scan_params* p, void* ws, size_t ws_bytes,
                           hipStream_t stream);

/* Backward.  states: what the forward wrote for the same x, g, h0 and
 * lengths.  dy: [B, H, N, d] in y's layout, read where there are tokens.
 * dhN: float32 [B, H, d] or NULL for zeros.  dx, dg: in the layouts of x and
 * g, 0 behind a sequence's end.  dh0: float32 [B, H, d] or NULL; it may be
 * dhN itself.  Overlaps as in the forward (dx and dg may be the two parts of
 * one interleaved buffer). */
int lapmix_scan_backward_ws(const void* x, const void* g, const float* states, const int32_t* lengths,
                            const void* dy, const float* dhN, void* dx, void* dg, float* dh0,
                            const lapmix_scan_params* p, void* ws, size_t ws_bytes, hipStream_t stream);

/* One token for every sequence of a batch (p->N = 1), on states in slots:
 * y = h_out[slot] = f h_in[slot] + i x.  h_in, h_out: float32
 * [n_slots, H, d], which may be the same pool.  slots: int32 [B] on the
 * device, or NULL for slot b of sequence b (then n_slots >= B).  A sequence
 * whose slot lies outside 0 .. n_slots-1 (a padded place of the batch) is
 * passed over: its y and all states stay as they were.  Each slot may be
 * named once in a call; a slot that is not named keeps its states. */
int lapmix_scan_step(const void* x, const void* g, const int32_t* slots, const float* h_in, float* h_out,
                     int32_t n_slots, void* y, const lapmix_scan_params* p, hipStream_t stream);

/* Forward of the norm.  r: [B, N, C] or NULL.  w: float32 [C].  s: [B, N, C]
 * of r_dtype, or NULL if it is not needed; it may be r itself.  y: [B, N, C].
 * scale: float32 [B, N, C / group] for LAPMIX_E4M3, else NULL.  A group whose
 * largest |y| lies below 2^-100 takes the scale 2^-100 / 448.  A group
 * narrower than the row needs d and x_stride to be multiples of 8 elements, and
 * bases of 16 bytes (y: 8), else LAPNYS_ERR_UNSUPPORTED.  Rows have up to 16384 columns
 * (wider ones: LAPNYS_ERR_UNSUPPORTED). */
int lapmix_norm_forward(const void* x, const void* r, const float* w, void* s, void* y, float* scale,
                        const lapmix_norm_params* p, hipStream_t stream);

/* Device workspace (bytes) of lapmix_norm_backward_ws. */
int lapmix_norm_workspace_size(const lapmix_norm_params* p, size_t* bytes);

/* Backward of the norm (y_dtype LAPNYS_F32 or LAPNYS_BF16: the type of dy).
 * s: what the forward stored.  ds: [B, N, C] of r_dtype, the gradient that
 * reaches the stream from behind, or NULL for zeros.  Outputs, each of which
 * may be NULL but not all: dr [B, N, C] of r_dtype (may be ds itself), dx
 * [B, H, N, d] in x's layout and type (the same values), dw float32 [C]. */
int lapmix_norm_backward_ws(const void* dy, const void* s, const float* w, const void* ds, void* dr, void* dx,
                            float* dw, const lapmix_norm_params* p, void* ws, size_t ws_bytes,
                            hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LAPMIX_H_ */
