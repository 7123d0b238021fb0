// rcs_internal.h -- calls shared between the library's own source files; not
// part of the C ABI.
#ifndef RCS_INTERNAL_H
#define RCS_INTERNAL_H

#include <cstdint>

// Drops the events ckpt_pack_async keeps for a snapshot buffer of device dev
// (call before freeing the buffer; no copy out of it may still be pending).
void rcs_snapshot_forget(int dev, const void *snapshot);

// RCS_OK if p is device (or managed) memory of the current device, with the bounds of
// its allocation (null if the runtime reports none); RCS_EINVAL otherwise.
int rcs_device_allocation(const void *p, const char **lo, const char **hi);
// Whether [a, a + a_bytes) and [b, b + b_bytes) share a byte.
bool rcs_overlaps(const void *a, int64_t a_bytes, const void *b, int64_t b_bytes);

#endif
