// per_device.cuh -- what the host asks of a device once and keeps: one value
// for each device ordinal, not for the process. Host code only; no CUDA
// header, so that it can be tested without a GPU.
#pragma once

#include <atomic>
#include <mutex>

namespace ep {

template <typename T, int kDevices = 64>
class PerDevice {
  public:
    // The value of `device`: `query(T*)`'s, asked until it succeeds once (its
    // result, 0 for success, is passed on). A failure is not kept. Devices past
    // kDevices are asked each time.
    template <typename Query>
    auto get(int device, T* value, Query query) -> decltype(query(value)) {
        using Error = decltype(query(value));
        if (device < 0 || device >= kDevices) return query(value);
        Entry& e = entries_[device];
        if (e.known.load(std::memory_order_acquire)) {
            *value = e.value;
            return Error{};
        }
        const std::lock_guard<std::mutex> lock(mutex_);
        if (!e.known.load(std::memory_order_relaxed)) {
            T found{};
            const Error err = query(&found);
            if (err != Error{}) return err;
            e.value = found;
            e.known.store(true, std::memory_order_release);
        }
        *value = e.value;
        return Error{};
    }

  private:
    struct Entry {
        std::atomic<bool> known{false};
        T value{};
    };
    Entry entries_[kDevices];
    std::mutex mutex_;
};

}  // namespace ep
