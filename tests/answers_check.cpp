// Host checks of csrc/answers.h (built and run by test_answers_host.py).
#include "answers.h"

#include <cstdio>

static SsdAnswers<3> answers;
static int asked = 0;

static int get(int device, int key, int value) {
    return answers.get(device, key, [&]() {
        ++asked;
        return value;
    });
}
#define CHECK(c) \
    if (!(c)) return std::printf("failed: %s (line %d)\n", #c, __LINE__), 1

int main() {
    // a failure is handed back and not kept: the next call asks again
    CHECK(get(0, 1, -1) == -1 && asked == 1);
    CHECK(get(0, 1, 76) == 76 && asked == 2);
    CHECK(get(0, 1, 5) == 76 && asked == 2);
    // another device and another question have answers of their own
    CHECK(get(1, 1, 66) == 66 && asked == 3);
    CHECK(get(0, 2, 0) == 0 && asked == 4);
    CHECK(get(0, 2, 9) == 0 && asked == 4);
    CHECK(get(1, 1, 5) == 66 && get(0, 1, 5) == 76 && asked == 4);
    // a device past the table, or none, is asked every time
    CHECK(get(-1, 0, 3) == 3 && get(-1, 0, 4) == 4 && get(kSsdMaxDevices, 0, 7) == 7 && asked == 7);
    return 0;
}
