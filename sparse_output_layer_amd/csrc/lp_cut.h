// lp_cut.h -- how a row of logits is cut into chunks for the log-probability
// kernels (logprob.hip).  Plain C++, so that it can be checked on the host.
#pragma once
#include <stdint.h>

namespace haste {

constexpr int kLpThreads = 256;
constexpr int kLpBatch = 4;      // vectors of a batch

// Rows in vectors of 16 bytes, aligned in memory (a row that starts inside one
// shares it with what is before).
struct Cut {
    int nc[2];        // chunks of the parts (head, tail)
    int per[2];       // vectors a chunk
    int nb;           // batches of kLpBatch vectors a thread: which kernel, 1, 2, 4 or 8
    int64_t items;    // B * (nc[0] + nc[1])
    constexpr int chunks() const { return nc[0] + nc[1]; }
    // what a workgroup of the kernel with nb batches goes over
    constexpr int most() const { return nb * kLpBatch * kLpThreads; }
    constexpr bool covered() const {
        return (nb == 1 || nb == 2 || nb == 4 || nb == 8) && per[0] <= most() && per[1] <= most();
    }
};

inline Cut cut_rows(int B, int64_t H, int64_t L, bool bf) {
    const int V = bf ? 8 : 4;
    const int64_t n[2] = {H, L};
    int64_t vec[2];
    for (int p = 0; p < 2; ++p) vec[p] = n[p] ? (n[p] + 2 * V - 2) / V : 0;   // from any start
    Cut c{};
    auto set = [&](int nb) {
        c.nb = nb;
        const int64_t most = c.most();
        for (int p = 0; p < 2; ++p) {
            c.nc[p] = (int)((vec[p] + most - 1) / most);
            c.per[p] = c.nc[p] ? (int)((vec[p] + c.nc[p] - 1) / c.nc[p]) : 0;
        }
        c.items = (int64_t)B * c.chunks();
    };
    // A single chunk (one launch) where it can be: 64 x 30000 bf16 9.8 us against
    // 12.3 in chunks, 4096 x 30000 61 to 66 against 61 to 63.  Else the largest
    // chunks that still give every CU two workgroups: from 2048 workgroups on 16 x
    // 2M takes 28 us instead of 21.5, from 128 on 4 x 2M 15.6 instead of 14.4; 512 x
    // 50000, then one chunk a row, 13.9 instead of 20.2 in two, 4096 x 50000 72
    // instead of 92 (K = 5: 16 and 24, 79 and 116).
    const bool one = (H == 0 || L == 0) && vec[0] + vec[1] <= 4 * kLpBatch * kLpThreads;
    int nb = one ? 1 : 8;
    set(nb);
    if (one)
        while (c.chunks() > 1) set(nb *= 2);
    else
        while (nb > 1 && c.items < 512) set(nb /= 2);
    return c;
}

}  // namespace haste
