// The division by a fixed divisor that the gradient operators' kernels use (fast_div in
// grad_launch.h): the quotient formed from its constants, against the processor's, for
// every small divisor, the largest ones, powers of two and their neighbours, at numerators
// around multiples of the divisor up to 2^62 - 1.
#include <cstdint>
#include <cstdio>
#include <cstdlib>

#include "grad_launch.h"

namespace {

// as the kernels do it: the high word of (4 n) * m, shifted
uint64_t quotient(uint64_t n, const zs::FastDiv &f) {
    return static_cast<uint64_t>((static_cast<unsigned __int128>(n << 2) * f.m) >> 64) >> f.s;
}

void check(uint64_t n, uint32_t d, const zs::FastDiv &f) {
    if (n >= 1ull << 62) return;
    if (quotient(n, f) != n / d) {
        std::printf("wrong: %llu / %u\n", static_cast<unsigned long long>(n), d);
        std::exit(1);
    }
}

uint64_t state = 88172645463325252ull;
uint64_t next() {
    state ^= state << 13;
    state ^= state >> 7;
    return state ^= state << 17;
}

void divisor(uint32_t d) {
    const zs::FastDiv f = zs::fast_div(d);
    const uint64_t top = (1ull << 62) - 1;
    for (uint64_t n : {uint64_t{0}, uint64_t{1}, uint64_t{d} - 1, uint64_t{d}, uint64_t{d} + 1, top,
                       top - 1, top / d * d, top / d * d - 1})
        check(n, d, f);
    for (int i = 0; i < 40; ++i) {
        const uint64_t q = next() % (top / d + 1);
        check(q * d, d, f);
        if (q > 0) check(q * d - 1, d, f);
        check(next() >> 2, d, f);
    }
}

}  // namespace

int main() {
    for (uint32_t d = 1; d < 20000; ++d) divisor(d);
    for (uint32_t b = 1; b < 32; ++b)
        for (int64_t o = -2; o <= 2; ++o) {
            const int64_t d = (int64_t{1} << b) + o;
            if (d >= 1 && d <= 0x7fffffff) divisor(static_cast<uint32_t>(d));
        }
    for (uint32_t d = 0x7fffffffu; d > 0x7fffffffu - 2000; --d) divisor(d);
    std::printf("ok\n");
    return 0;
}
