// host.h -- host-side services shared by the API sources: device facts, the
// per-stream workspace, launch checks and the pass-1 profiling events.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

namespace kmi {

// Compute units of the current device; also prepares its memory pool once.
int device_setup(int *cus);

// KEOPS_OK, or KEOPS_ERR_HIP when a launch since the last check failed.
int check_launch();

bool overlaps(const void *a, int64_t abytes, const void *b, int64_t bbytes);

// KEOPS_OPT_PROFILE: an event pair around one launch (index, or -1 when off).
int prof_begin(hipStream_t st);
void prof_end(int idx, hipStream_t st);

struct WsEntry;

// A device buffer of the workspace cache (one per device, stream and slot), held for
// the duration of one call.
class Workspace {
 public:
  Workspace() = default;
  Workspace(const Workspace &) = delete;
  Workspace &operator=(const Workspace &) = delete;
  ~Workspace() { release(); }

  // A device buffer of at least `bytes` for work enqueued on `st` (null for 0 bytes).
  // Returns KEOPS_OK or KEOPS_ERR_ALLOC (nothing enqueued).
  int acquire(hipStream_t st, int slot, size_t bytes);

  char *ptr() const { return ptr_; }

 private:
  void release();

  char *ptr_ = nullptr;
  hipStream_t st_ = nullptr;
  WsEntry *entry_ = nullptr;
  bool owned_ = false;
};

}  // namespace kmi
