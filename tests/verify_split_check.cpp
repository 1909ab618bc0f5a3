// CPU check of a draft verification's CTAs a request (verify_split.cuh): powers of two within
// every limit, one more step of which would pass one of them; and never more than fit.
#include <cstdio>
#include <initializer_list>

#include "verify_split.cuh"

using namespace swiglu;

#define CHECK(x)                                                        \
    do {                                                                \
        if (!(x)) {                                                     \
            std::printf("%s: %lld requests of %lld, %d SMs, %d fit: %d\n", #x, (long long)requests, \
                        (long long)vocab, sms, fits, ctas);             \
            return 1;                                                   \
        }                                                               \
    } while (0)

int main() {
    const int64_t all_requests[] = {1, 2, 3, 9, 10, 38, 76, 77, 152, 153, 1000, int64_t(1) << 26};
    const int64_t vocabs[] = {1, 100, 4095, 4096, 8191, 32000, 128000, 1 << 20};
    for (const int64_t requests : all_requests)
        for (const int64_t vocab : vocabs)
            for (const int sms : {1, 8, 132, 152})
                for (const int fits : {1, 2, 3, 4, 7, 8, 15, 16, 32}) {
                    const int ctas = verify_ctas(requests, vocab, sms, fits);
                    CHECK(ctas >= 1 && (ctas & (ctas - 1)) == 0);
                    CHECK(ctas <= fits && ctas <= 16);
                    CHECK(ctas == 1 || ctas * requests <= 2 * sms);
                    CHECK(ctas == 1 || ctas * 2048 <= vocab);
                    const int twice = 2 * ctas;
                    CHECK(twice > fits || twice > 16 || twice * requests > 2 * sms ||
                          twice * int64_t(2048) > vocab);
                }
    std::puts("ok");
    return 0;
}
