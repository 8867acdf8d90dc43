/*
 * zr_packed.h — the training operators of zr.h with their arguments in one
 * array of 64-bit words, for bindings of interpreted languages, where handing
 * over a dozen arguments and arrays costs more than the call itself.
 *
 * Words are read in the order given for each entry point.  A tensor takes
 * 2 + 2 * ndim words: data address, ndim, sizes, element strides.  `S` is a
 * double's bit pattern; pointers and integers are one word each.  Every check,
 * result and status is that of the zr.h function of the same name; ndim
 * outside 0..8 in any tensor is ZR_ERR_RANK and nothing after it is read.
 * Entry points with `need`: with workspace 0 the call stores the workspace's
 * size in *need and launches nothing; with one that is too small it returns
 * ZR_ERR_WORKSPACE and stores the size too (not if it is merely misaligned).
 */
#ifndef ZR_PACKED_H_
#define ZR_PACKED_H_

#include "zr.h"

#ifdef __cplusplus
extern "C" {
#endif

/* S eps, dtype, stream, mean, rstd, x, gamma, beta, y (data and strides count; its sizes are x's). */
int zr_packed_layer_norm_fwd(const int64_t* words);
/* S unused, dtype, stream, mean, rstd, grad_gamma, grad_beta, workspace, workspace bytes,
 * grad_out, x, gamma, grad_x. */
int zr_packed_layer_norm_bwd(const int64_t* words, int64_t* need);
/* S p, dtype, stream, seed, offset, device_offset, x, residual, out. */
int zr_packed_dropout_fwd(const int64_t* words);
/* S p, dtype, stream, seed, offset, device_offset, grad_out, grad_x. */
int zr_packed_dropout_bwd(const int64_t* words);
/* S unused, dtype, stream, label_type, ignore_index, reduction, loss, lse, workspace,
 * workspace bytes, x, w, labels. */
int zr_packed_linear_xent_fwd(const int64_t* words, int64_t* need);
/* S unused, dtype, stream, label_type, ignore_index, reduction, grad_loss, lse, grad_x, grad_w,
 * workspace, workspace bytes, x, w, labels. */
int zr_packed_linear_xent_bwd(const int64_t* words, int64_t* need);

#ifdef __cplusplus
}
#endif

#endif /* ZR_PACKED_H_ */
