// The segments of a sequence of linear attention, on the host: each begins where the one before ends, from 0 to the last token.
#include <cstdint>
#include <cstdio>

#include "linear.h"

int main() {
    const int tokens[] = {0, 1, 63, 64, 65, 640, 10007, 1 << 30, INT32_MAX - 200, INT32_MAX - 64}, segs[] = {1, 2, 3, 7, 19, 76, 152, 304};
    for (int n : tokens)
        for (int n_seg : segs) {
            const int chunks = (n + gdn::C - 1) / gdn::C, per_seg = (chunks + n_seg - 1) / n_seg;
            int at = 0;
            for (int part = 0; part < n_seg; ++part) {
                const gdn::LinearPart p = gdn::linear_part(n, chunks, per_seg, part);
                if (p.from != at || p.to < p.from || p.to > n || (p.to < n && p.to % gdn::C)) {
                    std::printf("%d tokens, segment %d of %d: %d .. %d behind %d\n", n, part, n_seg, p.from, p.to, at);
                    return 1;
                }
                at = p.to;
            }
            if (at != n) {
                std::printf("%d tokens in %d segments end at %d\n", n, n_seg, at);
                return 1;
            }
        }
    return 0;
}
