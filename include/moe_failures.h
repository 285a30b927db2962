/*
 * fp8_moe — failures that the library's kernels recorded, whichever workspace they were recorded in.
 * The pages describing the method have no counterpart to this header.
 *
 * A bounded wait that expires, and caller data that a kernel finds out of range, go to the status word of
 * the call's workspace (moe.h). That word is lost with a workspace that nobody keeps: those which the
 * Python modules take for one call. Each device therefore also keeps the first failure of any call since
 * it was last cleared. Nothing is written, and nothing costs time, where nothing fails.
 */
#ifndef FP8_MOE_FAILURES_H
#define FP8_MOE_FAILURES_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Reads the current device's kept failure into out[0] (MOE_OK or a MOE_ERR_DEVICE_* code), out[1] (its
 * where-code) and out[2] (its detail), after waiting for `stream`; if `clear` is non-zero and there is
 * one, it is forgotten. Work on other streams that has not finished may fail later. Not to be called
 * while a stream is captured. Returns MOE_OK, MOE_ERR_INVALID_ARG (out is NULL) or MOE_ERR_CUDA. */
int moe_device_failure(int32_t clear, int32_t out[3], void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8_MOE_FAILURES_H */
