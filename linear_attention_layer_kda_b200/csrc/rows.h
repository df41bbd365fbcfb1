// rows.h -- host-only planning of row moves (rows_plan.cu; kept
// apart so that it can be checked without a GPU).
#pragma once

#include <vector>

namespace kda {
namespace rows {

// Steps of a plan, in the order in which each thread makes them for its own bytes of the rows.
constexpr int kZero = -1;   // source: zeros
constexpr int kSaved = -2;  // source: what the chain's last save kept
constexpr int kSave = -3;   // destination: keep the source row's bytes for later

struct Step { int src, dst; };
struct Plan {
    std::vector<Step> steps;
    std::vector<int> first;  // first step of every chain, and the end; chains touch different rows
};

// dst[i] <- the old src[i] for all i at once (src[i] = -1: zeros).  in_place: both name rows of the
// same pool.  Destinations must be distinct.  Returns false if they are not.
bool plan(const int *dst, const int *src, int n, bool in_place, Plan *out);

}  // namespace rows
}  // namespace kda
