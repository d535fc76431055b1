// Set-up that a kernel needs once on every device.  Host only, standard library only.
#pragma once

#include <mutex>
#include <set>
#include <utility>

namespace sgp {

class OncePerDevice {
public:
    // Runs setup() (0: success) unless it has succeeded for this device and kernel; its status.
    template <typename F>
    int run(int device, const void* kernel, F setup) {
        std::lock_guard<std::mutex> lk(mu_);
        const std::pair<int, const void*> key(device, kernel);
        if (done_.count(key)) return 0;
        const int e = setup();
        if (e == 0) done_.insert(key);
        return e;
    }

private:
    std::mutex mu_;
    std::set<std::pair<int, const void*>> done_;
};

}  // namespace sgp
