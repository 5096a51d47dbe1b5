// Calls entry points of the library that fail, with a message longer than a
// string keeps in place, while operator new throws: no exception may cross the
// C interface.  Prints "<n> failures" and exits 0 on success.
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <new>

#include "../../include/mlp_block.h"

static bool full = false;

void* operator new(size_t n) {
    if (full) throw std::bad_alloc();
    void* p = malloc(n ? n : 1);
    if (!p) abort();
    return p;
}
void operator delete(void* p) noexcept { free(p); }
void operator delete(void* p, size_t) noexcept { free(p); }

static int failures = 0;

template <class F>
static void fails(const char* what, F call, const char* needle) {
    bool threw = false;
    full = true;
    try {
        call();
    } catch (...) {
        threw = true;
    }
    full = false;
    if (threw || !strstr(mlp_chain_last_error(), needle)) {
        ++failures;
        printf("%s: %s\n", what, threw ? "an exception" : mlp_chain_last_error());
    }
}

int main() {
    int64_t plan[9];
    fails("norm create", [] { mlp_norm_create((int64_t)1 << 40, 0, 1e-5f, 1); }, "H must be in 1..");
    fails("linear create", [] { mlp_linear_create(4, 60, 64, 0, 0, 1); }, "multiples of 8");
    fails("linear plan", [&] { mlp_linear_plan(4, 64, 64, 0, 9, 256, plan, 9); }, "unknown pass 9");
    fails("forced plan", [] { mlp_linear_debug_set_plan(nullptr, 0, 0, 1); }, "NULL handle");
    printf("%d failures\n", failures);
    return failures != 0;
}
