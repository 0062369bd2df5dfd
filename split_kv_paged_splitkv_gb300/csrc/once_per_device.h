// What a kernel needs set once on every device that runs it.
#pragma once

#include <atomic>
#include <cstdint>

namespace splitkv {

// set() where it has not succeeded on `device` before; what it returns, or `ok`.  `done` is the
// kernel's own, a bit per device: an attribute belongs to a device, and a failure is not
// kept.  (Devices from 64 on, of which there is no bit, are set every time.)
template <class Error, class Set>
Error once_per_device(std::atomic<uint64_t>& done, int device, Error ok, Set&& set) {
  const uint64_t bit = device < 64 ? uint64_t(1) << device : 0;
  if (done.load(std::memory_order_relaxed) & bit) return ok;
  const Error e = set();
  if (e == ok) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

}  // namespace splitkv
