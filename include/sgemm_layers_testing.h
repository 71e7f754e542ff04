/*
 * libsgemm -- TEST-ONLY interface of the operators in sgemm_layers.h.
 *
 * Nothing here is part of the product interface: these are device-free forms of
 * choices that a call makes, so that tests can show which kernel a size reaches.
 */
#ifndef SGEMM_LAYERS_TESTING_H
#define SGEMM_LAYERS_TESTING_H

#ifdef __cplusplus
extern "C" {
#endif

/*
 * How sgemm_fp4 shares out an M x N x K product on a GPU with `sms` SMs:
 * *tokens = the tokens of a tile (16 to 128 on one SM, 256 on a pair of SMs; 1: the
 * kernel of one token, which has no tiles) and *parts = the blocks of a cluster that
 * divide a tile's K (1: none).  Launches nothing and makes no CUDA call.
 * SGEMM_ERR_INVALID_ARG for a NULL output, a size below 1 or above what sgemm_fp4
 * takes, or sms < 2.
 */
int sgemm_fp4_plan_model(int M, int N, int K, int sms, int *tokens, int *parts);

#ifdef __cplusplus
}
#endif

#endif /* SGEMM_LAYERS_TESTING_H */
