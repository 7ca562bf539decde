// sgr_internal.h -- what the library's translation units share: per-device
// lookups defined in sgr_api.cu and the attention operators' device set-up
// defined in sgr_kv.cu.  Not part of the public interface.
#pragma once

namespace sgr {

constexpr int kMaxDevices = 64;

// Device error word of `dev` (allocates nothing).  Returns an sgr_status.
int device_error_word(int dev, unsigned** word);

// Kernel attributes of the attention operators on `dev`; idempotent,
// allocates nothing, called by sgr_init() and by their first call.  Returns
// an sgr_status.
int kv_init_device(int dev);

}  // namespace sgr
