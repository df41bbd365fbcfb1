// Test-only shim: the plan of row moves (csrc/rows_plan.cu), compiled here as plain C++.
#include <string.h>

#include "rows.h"

// Steps as pairs (src, dst) and the chains' first steps; returns the number of chains, or -1.
extern "C" int kda_test_rows_plan(const int *dst, const int *src, int n, int in_place, int *steps, int *first)
{
    kda::rows::Plan p;
    if (!kda::rows::plan(dst, src, n, in_place != 0, &p)) return -1;
    for (size_t i = 0; i < p.steps.size(); ++i) {
        steps[2 * i] = p.steps[i].src;
        steps[2 * i + 1] = p.steps[i].dst;
    }
    for (size_t i = 0; i < p.first.size(); ++i) first[i] = p.first[i];
    return (int)p.first.size() - 1;
}
