// Host-side checks of the attention-layer calls' own arithmetic (the same source the
// kernels use, compiled for the CPU).  One check a run, by name; 0: it holds.
#include <cstdio>
#include <cstring>
#include <random>

#include "attention_internal.h"

namespace {

std::mt19937_64 rng(7);

int pick(int lo, int hi) { return lo + (int)(rng() % (uint64_t)(hi - lo + 1)); }

#define HOLDS(x)                                                                 \
    do {                                                                         \
        if (!(x)) {                                                              \
            printf("line %d: %s\n", __LINE__, #x);                               \
            return 1;                                                            \
        }                                                                        \
    } while (0)

// A block's first unit in a list as long as the limits allow.
int check_places()
{
    const auto holds = [](long long in, int n) {
        const arf::UnitPlace p = arf::unit_place(in, n);
        return p.unit >= 0 && p.unit < n && p.item >= 0 && (long long)p.item * n + p.unit == in;
    };
    // 2^30 tokens are 2^24 units (and one for the end) for each of 128 heads
    const int n = (1 << 24) + 1;
    for (int head = 0; head < 128; ++head)
        for (int unit : {0, 1, n / 2, n - 1})
            HOLDS(holds((long long)head * n + unit, n));
    for (int trial = 0; trial < 1000000; ++trial) {
        const int per = pick(1, 1 << pick(1, 26));
        const long long in = (long long)pick(0, 1 << pick(1, 30)) * per + pick(0, per - 1);
        HOLDS(holds(in, per));
    }
    for (long long in : {0ll, (1ll << 31) - 1, 1ll << 31, (1ll << 32) - 1, 1ll << 32, (1ll << 40) + 7})
        HOLDS(holds(in, 1 << 26));
    return 0;
}

}  // namespace

int main(int argc, char** argv)
{
    const struct { const char* name; int (*run)(); } checks[] = {{"places", check_places}};
    for (const auto& c : checks)
        if (argc > 1 && strcmp(argv[1], c.name) == 0)
            return c.run();
    printf("no such check\n");
    return 2;
}
