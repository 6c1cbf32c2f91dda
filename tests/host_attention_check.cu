// Host-side checks of the attention-layer calls' own arithmetic (the same source the
// kernels use, compiled for the CPU).  One check a run, by name; 0: it holds (or was printed).
#include <cmath>
#include <cstdio>
#include <cstring>
#include <random>
#include <vector>

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

// Equal shares of a list of items: steps and ends of items (two steps' time each) of the busiest block
// against the mean.
int check_shares()
{
    for (int trial = 0; trial < 200; ++trial) {
        std::vector<int> items;
        const int kind = trial % 4, n = pick(20, 600);
        for (int i = 0; i < n; ++i)
            items.push_back(kind == 0 ? pick(1, 4) : kind == 1 ? (n - i + 7) / 8 : kind == 2 ? pick(0, 200)
                                                                                  : i ? 1 : 500);
        long long total = 0;
        for (int x : items)
            total += arf::share_of(x);
        const int blocks = total < 152 ? (int)total : 152;
        std::vector<double> busy(blocks);
        double all = 0;
        long long at = 0;
        for (int x : items) {
            for (int step = 0; step < x; ++step) {
                // the last block whose share begins at this step or before it
                const int b = (int)(((at + step + 1) * blocks - 1) / total);
                busy[b] += 1;
                if (step + 1 == x)
                    busy[b] += 2;
            }
            all += x ? x + 2 : 0;
            at += arf::share_of(x);
        }
        double most = 0;
        for (double b : busy)
            most = b > most ? b : most;
        // a share's whole units, and the end of an item that it has the last step of
        HOLDS(most <= all / blocks + 3);
    }
    return 0;
}

// Angles for the test to look at: position, bits of the frequency, bits of half_turns.
int print_turns()
{
    const auto line = [](int position, float f) {
        const float t = arf::half_turns(position, arf::turns_of(f));
        uint32_t a, b;
        memcpy(&a, &f, 4);
        memcpy(&b, &t, 4);
        printf("%d %u %u\n", position, a, b);
    };
    const int ends[] = {0, 1, -1, 4095, 4096, (1 << 24) - 1, (1 << 24) + 1, INT32_MAX, INT32_MIN, -70000};
    const float fs[] = {0.0f, 1.0f, -1.0f, 1e-4f, 2e-7f, 0.99999994f, 1.9999999f, 3.1415927f, 1000.5f,
                        1e-30f, 1e-42f};
    for (int p : ends)
        for (float f : fs)
            line(p, f);
    for (int i = 0; i < 20000; ++i) {
        const int bits = pick(1, 32);
        const int position = (int)(uint32_t)(rng() >> (64 - bits));
        const float u = (float)(rng() >> 40) * 0x1p-24f;
        line(i & 1 ? -position : position, i % 3 ? powf(10.0f, -7.0f * u) : powf(2.0f, 10.0f * u));
    }
    return 0;
}

}  // namespace

int main(int argc, char** argv)
{
    const struct { const char* name; int (*run)(); } checks[] = {{"places", check_places}, {"shares", check_shares},
                                                          {"turns", print_turns}};
    for (const auto& c : checks)
        if (argc > 1 && strcmp(argv[1], c.name) == 0)
            return c.run();
    printf("no such check\n");
    return 2;
}
