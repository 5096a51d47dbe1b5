// The tall tiles of a call whose rows are all left out (fragments_for of no
// rows): none, of no height, at no cost, whatever the columns and CUs.  Prints
// "<n> failures".
#include <stdio.h>

#include "../../consumer_gemm_chain_amd/csrc/train_launch.h"

int main() {
    int failures = 0;
    const uint32_t columns[] = {1, 20, 196, 500}, cus[] = {0, 1, 256};
    for (uint32_t c : columns)
        for (uint32_t u : cus) {
            const mlpc::Fragments f = mlpc::fragments_for(0, c, u);
            if (f.tiles != 0 || f.base != 0 || f.extra != 0 || f.cost != 0.f || f.whole != 0.f) {
                ++failures;
                printf("%u columns, %u CUs: %d tiles of %d, %d longer, %g of %g\n", c, u, f.tiles, f.base, f.extra, f.cost, f.whole);
            }
        }
    printf("%d failures\n", failures);
    return failures != 0;
}
