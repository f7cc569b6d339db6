/*
 * gmm_experts.h - C ABI of libgmm: local experts behind the mixture's soft
 * assignment, and the optimiser step that trains them, on one GB300.
 *
 * A fitted mixture answers with each point's top-m components and their
 * responsibilities (gmm_assign_topm: ids, gamma).  Used as the gate of a
 * mixture of local experts (a localised gating network: Xu, Jordan and
 * Hinton, "An alternative model for mixtures of experts", 1995), a point's
 * row goes to its components, each component multiplies its rows by its own
 * weights, and the answers come back summed with gamma:
 *
 *   gmm_route            ids -> rows of the components in order, and back
 *   gmm_spread           rows to their components (and the gradient of gmm_collect)
 *   gmm_expert_product   Y[r] = W_k A[r] for the rows r of component k
 *   gmm_collect          out[n] = sum_t gamma[n,t] Z[slot[n,t]] (and the
 *                        gradient of gmm_spread)
 *   gmm_expert_product_dx, _dw   gradients of the product
 *   gmm_adamw_step       one AdamW step over many tensors at once
 *
 * Conventions are those of gmm.h: device pointers unless named *_host, no
 * device memory allocated by the library, asynchronous on `stream`, argument
 * errors returned before anything is queued.  Arrays are dense and
 * row-major; element types of rows and weights are gmm_dtype values, sums
 * are held in 32 bits and rounded once.  Results are bitwise reproducible.
 * Every array is aligned to its element type (GMM_ERR_INVALID_ARG if not).
 * N and R may be 0.
 */
#ifndef GMM_EXPERTS_H
#define GMM_EXPERTS_H

#include "gmm.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * gmm_route - the entries (n, t) of a top-m table in the order of their
 * components.  Entry e = n*m + t belongs to component ids[e]; an id outside
 * [0, K) leaves the entry out.  Component k's rows are offsets[k] ..
 * offsets[k+1]-1, its entries in ascending order of e.
 * ids:      N*m int32.
 * offsets:  K+1 int64 (written).
 * entry:    N*m int32 (written): the entry of each row; -1 past offsets[K].
 * slot:     N*m int32 (written): the row of each entry; -1 if left out.
 * ws:       gmm_route_ws_bytes(N, m, K) bytes.
 * 1 <= m <= 8, 1 <= K <= 65536, N*m <= 2^31 - 1.
 */
size_t gmm_route_ws_bytes(int64_t N, int m, int K);
gmm_status gmm_route(const int32_t* ids, int64_t N, int m, int K, int64_t* offsets,
                     int32_t* entry, int32_t* slot, void* ws, size_t ws_bytes, void* stream);

/*
 * gmm_spread - each point's row to its entries' rows:
 *   Y[slot[n,t]] = gamma[n,t] X[n]      (gamma NULL: 1)
 * and the rows from offsets[K] to R-1 are zero.  With Z (R rows) and dgamma:
 *   dgamma[n,t] = <X[n], Z[slot[n,t]]>, 0 where the entry is left out,
 * so that with X = d out this is the gradient of gmm_collect, and with
 * gamma NULL the forward dispatch.
 * X: N*D; slot: N*m (a slot outside [0, R) counts as left out); offsets:
 * K+1; gamma: N*m float or NULL; Z: R*D and dgamma: N*m float (written),
 * both or neither; Y: R*D (written; may not overlap X or Z).
 * D >= 1, 1 <= m <= 8; R <= 2^31 - 1.
 */
gmm_status gmm_spread(const void* X, gmm_dtype xdtype, int64_t N, int D, int m, int K, int64_t R,
                      const int32_t* slot, const int64_t* offsets, const float* gamma,
                      const void* Z, void* Y, float* dgamma, void* stream);

/*
 * gmm_collect - each point's answer from its entries' rows:
 *   out[n] = sum_t gamma[n,t] Z[slot[n,t]]      (gamma NULL: 1)
 * in the order of t; a point with every entry left out gets zeros.  With
 * gamma NULL this is the gradient of the forward dispatch.
 * Z: R*D; slot: N*m (outside [0, R): left out); gamma: N*m float or NULL;
 * out: N*D (written).
 */
gmm_status gmm_collect(const void* Z, gmm_dtype xdtype, int64_t N, int D, int m, int64_t R,
                       const int32_t* slot, const float* gamma, void* out, void* stream);

/*
 * The experts' products.  Component k owns the rows offsets[k] ..
 * offsets[k+1]-1 of A, Y, dA, dY and the matrix W[k] (d_out x d_in):
 *   gmm_expert_product      Y[r]  = W_k A[r]
 *   gmm_expert_product_dx   dA[r] = W_k^T dY[r]
 *   gmm_expert_product_dw   dW_k  = sum over the rows r of k of dY[r] A[r]^T
 * Rows from offsets[K] to R-1 of Y and dA are written as zeros; dW of a
 * component without rows is zero.  offsets must ascend from 0 to at most R
 * (gmm_route's do).
 * A, dA: R*d_in; Y, dY: R*d_out; W: K*d_out*d_in; all of type xdtype; dW:
 * K*d_out*d_in of type wdtype, xdtype or GMM_F32.
 * 16-bit rows of a multiple of 16 bytes at 16-byte aligned addresses use the
 * tensor cores; other sizes and GMM_F32 use CUDA cores in fp32.
 * ws: gmm_expert_ws_bytes(R, d_in, d_out, K, xdtype) bytes, 256-byte
 *     aligned, of one call at a time (calls that overlap need one each).  Its
 *     first 256 bytes are the status word's: zero them once, before the first
 *     call.  gmm_last_device_status(ws, stream) then reports the first wait
 *     that gave up in any of the calls since; no call resets the word.
 * d_in, d_out >= 1 with d_in*d_out <= 2^31 - 1, 1 <= K <= 65536, R <= 2^31 - 1.
 * More than 65535 blocks of 64 columns on CUDA cores, or 2^31 - 1 tiles on the
 * tensor cores, are GMM_ERR_UNSUPPORTED.
 */
size_t gmm_expert_ws_bytes(int64_t R, int d_in, int d_out, int K, gmm_dtype xdtype);
gmm_status gmm_expert_product(const void* A, gmm_dtype xdtype, int64_t R, int d_in, int d_out,
                              int K, const int64_t* offsets, const void* W, void* Y, void* ws,
                              size_t ws_bytes, void* stream);
gmm_status gmm_expert_product_dx(const void* dY, gmm_dtype xdtype, int64_t R, int d_in, int d_out,
                                 int K, const int64_t* offsets, const void* W, void* dA, void* ws,
                                 size_t ws_bytes, void* stream);
gmm_status gmm_expert_product_dw(const void* dY, const void* A, gmm_dtype xdtype, int64_t R,
                                 int d_in, int d_out, int K, const int64_t* offsets, void* dW,
                                 gmm_dtype wdtype, void* ws, size_t ws_bytes, void* stream);

/*
 * gmm_adamw_step - one step of Adam with decoupled weight decay (Kingma and
 * Ba 2015; Loshchilov and Hutter 2019) over `count` tensors, no two of their
 * arrays with memory in common.  In fp32, each operation rounded once and in
 * this order (with 8-bit moments the update m / (...) may differ by 2^-21 of
 * itself; the moments do not):
 *   g = grad_scale grad
 *   m = beta1 m + (1 - beta1) g;   v = beta2 v + (1 - beta2) g^2
 *   p = (1 - lr weight_decay) p
 *       - (lr / (1 - beta1^step)) m / (sqrt(v) / sqrt(1 - beta2^step) + eps)
 * param is read and written (rounded to its type); with `master` (fp32) the
 * parameter is held there and param receives its rounding.
 * state_bits 32: m and v are float arrays.
 * state_bits 8: blocks of 256 elements (the last one shorter) share a scale;
 *   m is held as c|c| S, c int8, S = m_scale = max|m| / 127^2, and sqrt(v)
 *   as c^2 S, c uint8, S = v_scale = max sqrt(v) / 255^2: the root of
 *   value / S is rounded, so small values keep their relative precision, and
 *   a positive v keeps a code above zero.  A block whose largest value is
 *   below 1e-30 is held as zeros.  The step uses the new m and v before they
 *   are rounded.  m_scale, v_scale: ceil(n / 256) floats.
 * rounding (8 bits): how that root is rounded.
 *   GMM_ROUND_NEAREST (0): to the nearest code.  What a step changes by less
 *   than half a code stays as it is, so these are no averages over more than a
 *   few steps: with beta2 = 0.999 v does not fall but with its block's largest,
 *   rises only from gradients of several times its root, and m of an element
 *   whose gradients end stays at up to 81 S with beta1 = 0.9.
 *   GMM_ROUND_SEEDED (1): to one of the two codes around it, at random, so
 *   that m and v (above its smallest code) are held without bias and move at
 *   their own rate: the rounding to train with.  The random numbers depend on
 *   the step, the tensor's place in the list and the element alone (Philox4x32
 *   with ten rounds; counter: element / 8, its high word, the tensor, 0 for m
 *   or 1 for v; key: the step; 16 bits an element), so results repeat.
 * skip: optional device int32; when it is not 0 the call changes nothing
 *   (the caller's check for non-finite gradients; without it a non-finite
 *   gradient goes into the parameter and the moments as the formula says, and
 *   in 8 bits, where a moment that is not finite has no code, every value of
 *   that moment in its block becomes NaN).
 * tensors_host: host array, read before the call returns.
 * opts->step and both corrections made from it are fixed by the call: a call
 * captured in a graph takes the same step at every replay.  For graphs there
 * is gmm_adamw_step_counted.
 * Arrays need the alignment of their element type only; 16-byte aligned
 * ones (8-byte for 8-bit moments) are faster.
 */
typedef struct {
  void* param;
  const void* grad;
  float* master;       /* NULL: none */
  void* m;
  void* v;
  float* m_scale;      /* state_bits 8 only */
  float* v_scale;
  int64_t n;
  gmm_dtype param_dtype;
  gmm_dtype grad_dtype;
} gmm_adamw_tensor;

#define GMM_ROUND_NEAREST 0
#define GMM_ROUND_SEEDED 1

/* Zero all of it before the fields are set. */
typedef struct {
  double lr, beta1, beta2, eps, weight_decay, grad_scale;
  int64_t step;        /* 1 at the first step */
  int state_bits;      /* 32 or 8 */
  int rounding;        /* of 8-bit moments: GMM_ROUND_NEAREST or _SEEDED */
  const int32_t* skip; /* NULL: never */
} gmm_adamw_opts;

gmm_status gmm_adamw_step(const gmm_adamw_tensor* tensors_host, int count,
                          const gmm_adamw_opts* opts, void* stream);

/*
 * gmm_adamw_step_counted - the same step, counted on the device: `steps`
 * (device, 8-byte aligned) holds the steps taken so far, this one is number
 * *steps + 1, and the call adds one to it after its last launch, also where
 * `skip` leaves everything else as it was.  opts->step is not read.
 */
gmm_status gmm_adamw_step_counted(const gmm_adamw_tensor* tensors_host, int count,
                                  const gmm_adamw_opts* opts, int64_t* steps, void* stream);

/* The moments in fp32, whatever holds them (for checkpoints and inspection):
 * m_out_host[i], v_out_host[i] are device pointers to n floats each, written.
 * The two pointer arrays are host arrays, read before the call returns. */
gmm_status gmm_adamw_moments(const gmm_adamw_tensor* tensors_host, int count, int state_bits,
                             float* const* m_out_host, float* const* v_out_host, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GMM_EXPERTS_H */
