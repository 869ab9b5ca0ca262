/*
 * moe_paged_test.h - failure-detection test hook of the calls in moe_paged.h.
 */
#ifndef MOE_PAGED_TEST_H_
#define MOE_PAGED_TEST_H_

#include "moe_paged.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Makes waits of the attention kernels run out. tile >= 0: each CTA's producer stops before its tile of that number (with
 * one token per sequence: before the first piece that begins there or later), as if a wait of its own had run out; -1 (the
 * default): never. What waits for the tiles that never come gives up after its limit of one to two seconds (waits for whole
 * pieces: longer for tables of 2^25 keys and more) and records a nonzero status in the workspace status word; every role
 * then leaves after at most two waits of its own, copies and products under way are waited for, and the kernel returns
 * (outputs undefined; the GPU and the context stay usable). Zero the workspace before its next use. Process-wide; affects
 * only later calls. Returns MOE_ERR_INVALID_ARG for other values.
 */
moe_status_t moe_test_paged_give_up(int tile);

#ifdef __cplusplus
}
#endif

#endif /* MOE_PAGED_TEST_H_ */
