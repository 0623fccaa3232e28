// vq_mx4_groups.h -- how many groups the mixture-of-experts layer's kernels cut
// a call's pairs into (plain C++).
#pragma once

namespace vqmi {

// The most groups of up to `group` pairs, each of one expert, that `pairs` pairs
// (token and slot) over `experts` experts make: at most min(pairs, experts)
// experts are chosen, and each leaves at most one group that is not full.
constexpr int mx4_moe_max_groups(int pairs, int experts, int group) {
  const int chosen = pairs < experts ? pairs : experts;
  return (pairs + (group - 1) * chosen) / group;
}

}  // namespace vqmi
