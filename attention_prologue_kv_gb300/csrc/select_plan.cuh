// How kv_cache_select spreads a sequence: plain arithmetic, on the host and in its tests.
#pragma once

#include <stdint.h>

namespace kvr {

constexpr int SEL_THREADS = 1024;
constexpr int64_t SEL_ROOM = 49152;              // ranks that a CTA's shared memory takes
constexpr int SEL_SHARED = -1, SEL_AGAIN = 0;    // forms without keys in registers

struct SelectForm {
    int ctas;       // of a sequence, a cluster
    int64_t each;   // keys of a CTA at most
    int form;       // keys of a thread in registers, SEL_SHARED or SEL_AGAIN
};

// CTAs of a sequence: as many as registers need, and up to 8 while the SMs are not filled and a CTA has 4096 keys or more. (Of
// one sequence of 131000 keys 8 take 17 us and 16 took 20 to 24, whose counts every CTA reads; of 200000 keys 8, with ranks in
// shared memory, 26.8 and 16 20.9. 131000 keys with ranks in shared memory: 22.) most: 16 where the device has room for such
// clusters, else 8, the portable size.
inline SelectForm select_form(int64_t weight_len, int64_t n, int sms, int most) {
    int ctas = 1;
    while (ctas < most && (weight_len > int64_t(ctas) * SEL_THREADS * 16 ||
                           (ctas < 8 && weight_len >= int64_t(ctas) * 4096 && n * ctas * 2 <= sms)))
        ctas *= 2;
    const int64_t each = (weight_len + ctas - 1) / ctas;
    int form = each <= SEL_ROOM ? SEL_SHARED : SEL_AGAIN;
    for (int v = 16; v >= 1; v /= 2)
        if (each <= int64_t(SEL_THREADS) * v) form = v;
    return {ctas, each, form};
}

}  // namespace kvr
