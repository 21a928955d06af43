// Host check of the key/value cache's index arithmetic (kv_internal.h): for
// whatever q_start, kv_len and sizes hold, rows stay within the packed
// tensors, tokens within the table, and a block's keys within the sequence.
#include <cstdio>
#include <cstdlib>
#include <random>

#include "kv_internal.h"

using namespace li8;

#define CHECK(x)                                              \
    do {                                                      \
        if (!(x)) {                                           \
            std::printf("failed: %s (case %d)\n", #x, i);     \
            return 1;                                         \
        }                                                     \
    } while (0)

int main()
{
    std::mt19937 rng(7);
    const int odd[] = {0, 1, -1, 2, 15, 16, 17, 63, 64, 65, 1000, INT32_MAX, INT32_MIN, INT32_MAX - 1, 1 << 30};
    auto any = [&]() {
        return rng() % 3 ? (int)(rng() % 200) - 20 : odd[rng() % (sizeof(odd) / sizeof(odd[0]))];
    };
    for (int i = 0; i < 2000000; i++) {
        const int tokens = abs(any() % 4096), max_q = abs(any() % 4096), max_kv = (int)(rng() % 5000);
        const KvSeq q = kv_sequence(any(), any(), any(), tokens, max_q, max_kv);
        CHECK(q.q0 >= 0 && q.n >= 0 && q.q0 + q.n <= tokens && q.n <= max_q);
        CHECK(q.len >= 0 && q.len <= max_kv);
        CHECK((int64_t)q.begin + q.n <= q.len);           // stored positions stay below len
        if (q.n == 0)
            continue;
        const int a = (int)(rng() % q.n), b = a + (int)(rng() % (q.n - a));
        const int window = rng() % 2 ? 0 : (rng() % 4 ? 1 + (int)(rng() % 300) : INT32_MAX);
        const bool causal = rng() % 2;
        const KvSpan s = kv_span(q.begin + a, q.begin + b, q.len, causal, window);
        CHECK(s.lo >= 0 && s.lo <= s.hi && s.base >= 0 && s.base <= s.lo && s.lo - s.base < 32);
        CHECK(s.hi <= q.len || s.hi == s.lo);             // (an empty span may lie past the end)
        // every key that some row sees is inside
        for (int r = a; r <= b; r++) {
            const int64_t p = (int64_t)q.begin + r;
            int64_t hi = q.len, lo = 0;
            if (causal && p + 1 < hi)
                hi = p + 1;
            if (window > 0 && p - window + 1 > 0)
                lo = p - window + 1;
            CHECK(lo >= hi || (lo >= s.lo && hi <= s.hi));
        }
        if (window > 0)   // what the plan reckons with
            CHECK((int64_t)s.hi - s.base <= (int64_t)window + (causal ? b - a : (int64_t)q.len - q.begin) + 31 ||
                  s.hi == s.lo);
    }
    std::printf("ok\n");
    return 0;
}
