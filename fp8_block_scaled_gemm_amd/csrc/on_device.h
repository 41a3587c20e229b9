// The current GPU for the length of a call.
#pragma once

#include <hip/hip_runtime_api.h>

#include <stdexcept>
#include <string>

// The library launches on the current device.  Where the tensors' GPU cannot be
// made current nothing may be launched: it would go to another one's context.
struct OnDevice {
    int before = -1;
    explicit OnDevice(int index) {
        int now = -1;
        if (hipGetDevice(&now) != hipSuccess) throw std::runtime_error("the current GPU is not known");
        if (now == index) return;
        if (hipSetDevice(index) != hipSuccess)
            throw std::runtime_error("GPU " + std::to_string(index) + " cannot be made the current one");
        before = now;
    }
    OnDevice(const OnDevice&) = delete;
    OnDevice& operator=(const OnDevice&) = delete;
    ~OnDevice() {
        if (before >= 0) (void)hipSetDevice(before);
    }
};
