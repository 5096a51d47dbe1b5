// The tall tiles that the cross entropy takes for n rows (fragments_for): every
// row is in one tile, every tile has 5 to 8 fragments and rows of its own, and
// there are no more of them than a launch has workgroups for.  Prints "<n>
// failures".
#include <stdio.h>

#include "../../consumer_gemm_chain_amd/csrc/train_launch.h"

int main() {
    int failures = 0;
    const uint32_t columns[] = {1, 20, 196, 500}, cus[] = {0, 256};
    for (int n = 1; n <= (1 << 24); n += n < 6000 ? 1 : n / 7)
        for (uint32_t c : columns)
            for (uint32_t u : cus) {
                const mlpc::Fragments f = mlpc::fragments_for(n, c, u);
                const bool height = f.base >= 5 && f.base + (f.extra > 0) <= 8 && f.extra >= 0 && f.extra < f.tiles;
                const long last = 32L * ((long)(f.tiles - 1) * f.base + f.extra);       // first row of the last tile
                const bool rows = last < n && last + 32L * f.base >= n;
                const bool count = f.tiles <= (n + 159) / 160 && f.tiles >= (n + 255) / 256;
                if (!height || !rows || !count || !(f.cost > 0.f) || !(f.cost <= f.whole)) {
                    if (++failures < 10) printf("n %d: %d tiles of %d, %d longer, %g of %g\n", n, f.tiles, f.base, f.extra, f.cost, f.whole);
                }
            }
    if (mlpc::fragments_for(0, 1, 256).tiles != 0) ++failures;
    printf("%d failures\n", failures);
    return failures != 0;
}
