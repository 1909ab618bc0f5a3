// How a draft verification is shared out (plain arithmetic, checked on the CPU).
#pragma once

#include <cstdint>

namespace swiglu {

constexpr int kVerifyThreads = 512;
constexpr int kVerifyMaxCluster = 16;    // CTAs a request

// CTAs a request, of one cluster: about two an SM over all requests, none with less than a load
// a lane (one request of 152000 values: 8.5 us with 16; 64 requests of 128000 17.6 with 4), and
// no more than `fits`, the largest cluster of which the device can run one at all.
inline int verify_ctas(int64_t requests, int64_t vocab, int sms, int fits) {
    const int most = fits < kVerifyMaxCluster ? fits : kVerifyMaxCluster;
    int ctas = 1;
    while (2 * ctas <= most && 2 * ctas * requests <= 2 * static_cast<int64_t>(sms) &&
           2 * ctas * int64_t(kVerifyThreads) * 4 <= vocab)
        ctas *= 2;
    return ctas;
}

}  // namespace swiglu
