// rcs_internal.h -- calls shared between the library's own source files; not
// part of the C ABI.
#ifndef RCS_INTERNAL_H
#define RCS_INTERNAL_H

#include <hip/hip_runtime_api.h>

#include <atomic>
#include <cstdint>

// Drops the events ckpt_pack_async keeps for a snapshot buffer of device dev
// (call before freeing the buffer; no copy out of it may still be pending).
void rcs_snapshot_forget(int dev, const void *snapshot);

// The C ABI's check that p is memory of the current device, and the bounds of
// the allocation it lies in (both null where the runtime reports none).
int rcs_device_allocation(const void *p, const char **lo, const char **hi);

// The check of a norm destination (a status code).
int rcs_check_norm_out(const double *p, int dev);

// The (current device, stream) workspace of the norm kernels: the partial
// sums, the clip record, and the flag that a norm has been computed there.
int rcs_norm_buffers(hipStream_t stream, double **partials, void **record,
                     std::atomic<bool> **has_norm);

#endif
