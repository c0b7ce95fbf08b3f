// device_memo.h -- what the driver was asked once, remembered for each device.
#pragma once

#include <atomic>

namespace w4a8 {

// Answers (whole numbers, 0 or more) to KEYS questions for each of DEVICES devices.  Parts of one model
// need not agree: how many clusters fit depends on a part's own processors.  A question that failed (a
// negative answer) is asked again by the next call.  Any threads may ask at the same time.
template <int DEVICES, int KEYS>
class DeviceMemo {
    std::atomic<int> known_[DEVICES][KEYS] = {};  // the answer + 1; 0: not known

   public:
    // `ask()` for a device and key that no earlier call has answered.  Outside the table: asked every time.
    template <typename Ask>
    int get(int device, int key, Ask&& ask) {
        if (device < 0 || device >= DEVICES || key < 0 || key >= KEYS) return ask();
        std::atomic<int>& known = known_[device][key];
        const int n = known.load(std::memory_order_relaxed);
        if (n > 0) return n - 1;
        const int answer = ask();
        if (answer >= 0) known.store(answer + 1, std::memory_order_relaxed);
        return answer;
    }
};

}  // namespace w4a8
