/*
 * hq_test.h -- test-only entry points of libhq (failure detection without a GPU fault).
 *
 * The encoder places each item (a block of 128 tile rows of one tile column) by a decoupled
 * look-back over the items before it, and the e4m3 product passes blocks between its warps; every
 * wait in them is bounded.  The entry points here make one item withhold its offset, or one block its
 * tensor-core work, so that the bounded waits for it run out: the kernel then records HQ_ERR_TIMEOUT
 * in the workspace status word, finishes, and the CUDA context stays usable.  They exist to test
 * that path; the method has no counterpart.  These entry points are built only into the test library libhq_test.so (sources compiled with HQ_TEST_HOOKS); the
 * product library libhq.so neither exports them nor carries the hook in its kernels.
 */
#ifndef HQ_TEST_H
#define HQ_TEST_H

#include "hq.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * As hq_encode, except that item `silent_item` (>= 1; items are numbered tile column by tile
 * column, ceil(rows / 128) per column at n = 64 or 128, ceil(rows / 64) at n = 256) never
 * publishes its word offset.  Expect HQ_ERR_TIMEOUT from hq_status_read and a code that is not
 * usable; the call takes about as long as the look-back limit (about a second).  HQ_ERR_ARG for
 * silent_item < 1 and for everything hq_encode rejects; HQ_ERR_UNSUPPORTED for lattices other than
 * E8 (only the E8 kernels of the test library carry the hook).
 */
hq_status_t hq_test_encode_silent_item(const void* x, hq_dtype_t dtype, int64_t rows, int64_t cols,
                                       const hq_params_t* p, hq_code_t* out, void* ws, size_t ws_bytes,
                                       int64_t silent_item, void* stream);

/*
 * As hq_gemm_fp8, except that every thread block withholds the tensor-core work of its block of K
 * `silent_block` (counted from its first) and of all after it, so that the waits for them run out (about a
 * second each).  Expect HQ_ERR_TIMEOUT from hq_status_read where a thread block has that many, and a product
 * that is not usable.  log (device, zeroed by the caller, 3 * 4096 words): for each thread block that waits for
 * operands, how many boxes it asked for, how many of the last of them, as many as its ring has stages,
 * it saw land before it left, and whether it saw its tensor-core work end.  Of a pair of thread blocks the
 * even one waits for both; here it asks for two boxes less than the odd one, as if its wait had run out first.
 */
hq_status_t hq_test_gemm_fp8_silent_block(const uint8_t* A, int64_t lda, const float* sa, int64_t M, const uint8_t* W,
                                          int64_t ldw, const float* sw, int64_t N, int64_t K, void* Y, hq_dtype_t ydtype,
                                          void* ws, size_t ws_bytes, int32_t silent_block, uint32_t* log, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* HQ_TEST_H */
