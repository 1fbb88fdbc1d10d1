// gdn_host.h -- host-side helpers shared by the C ABI's translation units:
// status reporting, the device's compute-unit count, alignment checks and the
// optional per-kernel timing.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdn.h"

namespace gdn_host {

// Sets the thread's gdn_last_error text and returns s.
gdn_status fail(gdn_status s, const char* fmt, ...);
gdn_status hip_fail(hipError_t e, const char* what);

// Compute units of the current device, cached per device.
int cu_count();

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline size_t align_up(size_t x) { return (x + 255) & ~size_t(255); }

template <class T>
T* at(void* base, size_t off) { return reinterpret_cast<T*>(static_cast<char*>(base) + off); }

// One launch's timing events (null while timing is off).
struct ProfRec { const char* name; hipEvent_t a, b; bool on, ok_a; };
ProfRec prof_begin(const char* name, hipStream_t s);
void prof_end(ProfRec& r, hipStream_t s);

// Launch through f() on stream s, bracketed by events when timing is enabled.
template <class F>
hipError_t timed(const char* name, hipStream_t s, F f) {
  ProfRec r = prof_begin(name, s);
  const hipError_t e = f();
  prof_end(r, s);
  return e;
}

}  // namespace gdn_host
