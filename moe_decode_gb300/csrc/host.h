// Host-side state and helpers shared by the C ABI's translation units.
#pragma once
#include <cstddef>
#include <cstdint>

namespace moe {

struct Options {
    int grid_ctas = 0;
    long long timeout_ns = 1000000000LL;
    unsigned long long* trace = nullptr;
    bool hold_back = false;
};
extern Options g_opt;
extern thread_local int g_last_launches;

struct DeviceInfo {
    int sms = 0;
    int smem_optin = 0;
    bool coop = false;
};
constexpr int kMaxDevices = 64;
// Properties of the current device (MOE_OK or MOE_ENODEVICE).
int device_info(DeviceInfo* out);

inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace moe
