// Checks of csrc/device_memo.h; prints "ok".
#include "../w4a8_block_quantized_gb300/csrc/device_memo.h"

#include <cstdio>

static int asked = 0;
static int answer(int n) { return ++asked, n; }
#define CHECK(x) \
    if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; }

int main() {
    static w4a8::DeviceMemo<4, 3> memo;
    auto get = [](int dev, int key, int n) { return memo.get(dev, key, [n] { return answer(n); }); };
    CHECK(get(0, 1, 18) == 18 && asked == 1);
    CHECK(get(0, 1, 99) == 18 && asked == 1);  // remembered
    CHECK(get(1, 1, 17) == 17 && asked == 2);  // another device has its own
    CHECK(get(0, 2, 5) == 5 && asked == 3);    // as has another question
    CHECK(get(0, 1, 99) == 18 && get(1, 1, 99) == 17 && asked == 3);
    CHECK(get(2, 0, -2) == -2 && get(2, 0, 7) == 7 && asked == 5);  // a failure is not remembered
    CHECK(get(3, 0, 0) == 0 && get(3, 0, 4) == 0 && asked == 6);    // "none" is an answer
    CHECK(get(4, 0, 3) == 3 && get(4, 0, 2) == 2 && get(-1, 0, 1) == 1 && get(0, 3, 6) == 6 && asked == 10);
    std::puts("ok");
    return 0;
}
