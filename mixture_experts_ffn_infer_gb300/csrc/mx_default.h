// What the torch binding uses for microscaled calls that are given no workspace.  Their device errors go to a word
// that the library keeps, one per device, zero at first: like a caller's own it accumulates (atomically, so on any
// number of streams) until moe_get_error reads it.
#ifndef MX_DEFAULT_H
#define MX_DEFAULT_H

#include "moe_mx.h"

#ifdef __cplusplus
extern "C" {
#endif

/* MOE_MX_PRODUCT_WORKSPACE bytes on the current device, or NULL where CUDA does not give their address. */
void *moe_mx_default_workspace(void);

/* moe_mx_layer_forward with its errors in moe_mx_default_workspace's word; the workspace's own is not used. */
moe_status moe_mx_layer_forward_default(const moe_mx_weights *gate_up, const moe_mx_weights *down, int32_t top_k,
                                        int64_t n_tokens, const void *x, const void *residual, const void *gain,
                                        float eps, const int32_t *topk_ids, const float *topk_weight,
                                        const float *x_global, const float *h_global, void *sum, void *out,
                                        int32_t out_is_fp32, void *workspace, size_t workspace_bytes,
                                        cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MX_DEFAULT_H */
