/*
 * gmm_gate.h - C ABI of libgmm: a learned gate for the local experts of
 * gmm_experts.h, on one GB300.
 *
 * The fitted mixture answers with a point's top-m components and their
 * responsibilities (gmm_assign_topm).  A gate that is trained with the experts
 * answers the same from logits L (a row of K for each point, from whatever
 * network; gmm_expert_product with one component makes them from rows and a
 * matrix), p[n,k] = exp(L[n,k]) / sum_j exp(L[n,j]) in the place of the
 * responsibilities:
 *
 *   gmm_gate         the m largest components of a row and their share of p;
 *                    with them, what keeps all components in use: entries and
 *                    mass of each, and the balance loss
 *   gmm_gate_grad    the gradient of the logits
 *   gmm_distill      how far p is from a teacher's top entries (the mixture's
 *                    own, or a larger model's top logits), and its gradient
 *   gmm_layer_norm, gmm_layer_norm_grad   the rows that enter such a layer,
 *                    normalised, and the gradients of rows and weights
 *
 * Conventions are those of gmm.h and gmm_experts.h: device pointers, no device
 * memory allocated by the library, asynchronous on `stream`, argument errors
 * returned before anything is queued; arrays dense, row-major, aligned to
 * their element type (GMM_ERR_INVALID_ARG if not), outputs apart from inputs
 * and from one another.  Logits and rows are of a gmm_dtype; sums are held in
 * 32 bits or more and rounded once; a share below 2^-126 may be 0.  Results are
 * bitwise reproducible.  N may be 0.
 */
#ifndef GMM_GATE_H
#define GMM_GATE_H

#include "gmm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GMM_GATE_NORMALISED 1 /* the m shares of a row sum to one */

/*
 * gmm_gate - a row's m largest logits.
 * L:      N*K.  A logit of -inf is a component that is not there: it has no
 *         share and is never among the m.
 * live:   N bytes or NULL; a row whose byte is 0 (padding) is left out and not
 *         read.  So is a row whose logits are all -inf: ids -1, gamma 0, lse
 *         -inf, and it counts nowhere below.
 * ids:    N*m int32 (written): components by falling logit, ties to the lower
 *         one; -1 where the row has fewer than m.
 * gamma:  N*m float (written): p at ids, or with GMM_GATE_NORMALISED p at ids
 *         over the sum of the row's kept p; 0 where the id is -1.
 * lse:    N float (written) or NULL: log sum_k exp(L[n,k]).
 * A NaN counts as larger than every number; it makes gamma, lse and mass of
 * its row NaN, and so does +inf.
 * The balance outputs, all or none (NULL):
 * counts: K int64 (written): the entries of each component.
 * mass:   K float (written): mass_k = sum over the rows of p[n,k].
 * share:  K float (written): K counts_k / (sum_j counts_j * rows), `rows` those
 *         that count; 0 where none does.
 * loss:   1 float (written): sum_k share_k mass_k: K sum_k f_k P_k with the
 *         fractions f of the entries and the rows' mean P of p (Fedus, Zoph
 *         and Shazeer 2022); 1 where either is even.
 * ws:     gmm_gate_ws_bytes(N, K, m) bytes, 256-byte aligned, of one call at a
 *         time (calls that overlap need one each); NULL without the balance
 *         outputs.
 * 1 <= K <= 65536, 1 <= m <= 8, N*m <= 2^31 - 1.
 */
size_t gmm_gate_ws_bytes(int64_t N, int K, int m);
gmm_status gmm_gate(const void* L, gmm_dtype xdtype, int64_t N, int K, int m, int flags,
                    const uint8_t* live, int32_t* ids, float* gamma, float* lse, int64_t* counts,
                    float* mass, float* share, float* loss, void* ws, size_t ws_bytes,
                    void* stream);

/*
 * gmm_gate_grad - the gradient of the logits,
 *   dL[n] = (d gamma[n] / d L[n]) dgamma[n] + coef d loss / d L[n]
 * with ids and share held fixed:
 *   v_t = gamma_t dgamma_t, S = sum_t v_t;  normalised: v_t -= gamma_t S, S = 0
 *   dL[n,k] = p[n,k] (coef (share_k - sum_j share_j p[n,j]) - S)
 *             + sum over the t with ids[n,t] = k of v_t
 * and zeros in rows that are left out.
 * L, live, ids, gamma: as gmm_gate had and gave them (an id outside [0, K)
 * counts as -1; an id may stand twice).
 * dgamma: N*m float or NULL (0; ids and gamma may then be NULL too).
 * share:  gmm_gate's or NULL (no balance loss; coef is not read).
 * dL:     N*K of L's type (written).
 */
gmm_status gmm_gate_grad(const void* L, gmm_dtype xdtype, int64_t N, int K, int m, int flags,
                         const uint8_t* live, const int32_t* ids, const float* gamma,
                         const float* dgamma, const float* share, double coef, void* dL,
                         void* stream);

#define GMM_TEACHER_LOGITS 0
#define GMM_TEACHER_GAMMA 1
#define GMM_DISTILL_ADD 1

/*
 * gmm_distill - from a teacher's top entries: with the student's
 * p_n = softmax(L[n] / T) and the teacher's q_n over its entries alone,
 *   row_n = w_n T^2 sum_t q[n,t] (log q[n,t] - log p_n[ids[n,t]])
 *   loss  = scale sum_n row_n
 *   dL[n,k] = scale w_n T (p_n[k] - sum over the t with ids[n,t] = k of q[n,t])
 * (Hinton, Vinyals and Dean 2015).
 * L:       N*K, the student's logits; -inf has p = 0.
 * ids:     N*m int32, values: N*m float, the teacher's entries; an id outside
 *          [0, K) is none.  kind GMM_TEACHER_LOGITS: q = softmax(values / T);
 *          GMM_TEACHER_GAMMA: q in proportion to values^(1/T), values >= 0
 *          (gmm_assign_topm's ids and gamma).  An entry of share 0 (a logit
 *          of -inf, a gamma of 0) is none.
 * weights: N float or NULL (1).  A row of weight 0, whose logits are not read,
 *          or without an entry is left out: its row_n and dL are 0 (added: dL is
 *          as it was).
 * A row whose logits are all -inf has row_n = inf and p = 0; one that has -inf, or
 * a number 2^128 below its largest, at an entry has row_n = inf.  A large T leaves
 * row_n the difference of logarithms in 32 bits, T^2 times their rounding.
 * rows:    N float (written).
 * loss:    1 float (written).
 * dL:      N*K of L's type (written), or NULL: no gradient.  With
 *          GMM_DISTILL_ADD in flags the gradient is added to what dL holds
 *          (gmm_gate_grad's), in 32 bits, rounded once.
 * ws:      gmm_distill_ws_bytes() bytes, 256-byte aligned, of one call at a
 *          time.
 * T > 0, T and log2 e / T finite in fp32, 1 <= K <= 2^18, 1 <= m <= 64, N*m <= 2^31 - 1.
 */
size_t gmm_distill_ws_bytes(void);
gmm_status gmm_distill(const void* L, gmm_dtype xdtype, int64_t N, int K, int m, int kind, int flags,
                       double temperature, double scale, const int32_t* ids, const float* values,
                       const float* weights, float* rows, float* loss, void* dL, void* ws,
                       size_t ws_bytes, void* stream);

/*
 * gmm_layer_norm - each row about its mean, over its standard deviation:
 *   h[n] = (X[n] - mean) / sqrt(var + eps),  Y[n] = weight h[n] + bias
 * with mean and var = mean of squares about it over the row (Ba, Kiros and
 * Hinton 2016); var is taken about the mean, not as a difference of squares.
 * Sums are fp32: the elements' and the squared deviations' over a row have to be
 * below 2^128 (deviations up to 2^64 / sqrt(D), 10^17 at D = 32768).
 * X: N*D; weight, bias: D of wdtype (xdtype or GMM_F32), or NULL (1, 0); Y: N*D
 * of xdtype (written).  eps >= 0; 1 <= D <= 32768; N <= 2^31 - 1.
 *
 * gmm_layer_norm_grad - with g = weight dY (the statistics are taken again
 * from X, so nothing is kept between the calls):
 *   dX[n] = (g - mean(g) - h mean(g h)) / sqrt(var + eps)
 *   dweight = sum_n dY[n] h[n],  dbias = sum_n dY[n]
 * dX: N*D of xdtype (written) or NULL; dweight, dbias: D of wdtype (written),
 * both or neither; ws: gmm_layer_norm_ws_bytes(D) bytes, 256-byte aligned, of
 * one call at a time; NULL without dweight and dbias.
 */
gmm_status gmm_layer_norm(const void* X, gmm_dtype xdtype, int64_t N, int D, double eps,
                          const void* weight, const void* bias, gmm_dtype wdtype, void* Y,
                          void* stream);
size_t gmm_layer_norm_ws_bytes(int D);
gmm_status gmm_layer_norm_grad(const void* dY, const void* X, gmm_dtype xdtype, int64_t N, int D,
                               double eps, const void* weight, gmm_dtype wdtype, void* dX,
                               void* dweight, void* dbias, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GMM_GATE_H */
