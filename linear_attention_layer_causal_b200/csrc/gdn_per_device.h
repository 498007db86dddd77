// gdn_per_device.h -- a value that is asked of the runtime once per device.
#pragma once

#include <atomic>
#include <mutex>

#include <driver_types.h>

namespace gdn {

// get() runs `query(&value)` on the first call for a device and keeps what it
// found.  A query that fails is returned to the call that met it and asked again
// by the next one.  Calls from several threads are safe.
template <class V, int kDevices = 64> class PerDevice {
    std::atomic<bool> ready_[kDevices] = {};
    V value_[kDevices] = {};
    std::mutex lock_;

  public:
    template <class Query> cudaError_t get(int device, Query query, const V **value) {
        if (device < 0 || device >= kDevices)
            return cudaErrorInvalidDevice;
        if (!ready_[device].load(std::memory_order_acquire)) {
            std::lock_guard<std::mutex> hold(lock_);
            if (!ready_[device].load(std::memory_order_relaxed)) {
                V found = {};
                const cudaError_t e = query(&found);
                if (e != cudaSuccess)
                    return e;
                value_[device] = found;
                ready_[device].store(true, std::memory_order_release);
            }
        }
        *value = &value_[device];
        return cudaSuccess;
    }
};

} // namespace gdn
