// device_kind.h -- a device's SM count and whether it is the one that the kernels are built for.
// Neither changes, so the answer is kept; an answer that could not be had is not.
#pragma once

#include <atomic>

namespace msa {

enum class DeviceAttr { kSmCount, kMajor, kMinor };

// The SM count of an sm_103 device, -1 for any other device, 0 where a query failed.
// query(attr, &value) asks the device and says whether it answered.
template <typename Query>
int sm_count_of(std::atomic<int>* kept, Query query) {
  int sms = kept->load(std::memory_order_relaxed);
  if (sms != 0) return sms;
  int major = 0, minor = 0;
  if (!query(DeviceAttr::kSmCount, &sms) || !query(DeviceAttr::kMajor, &major) || !query(DeviceAttr::kMinor, &minor))
    return 0;
  if (major != 10 || minor != 3) sms = -1;
  kept->store(sms, std::memory_order_relaxed);
  return sms;
}

}  // namespace msa
