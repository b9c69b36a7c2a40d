// kv4_join.h -- where the partials of a cut unit of few-row attention lie (kv4_decode.cu), on host and device.
#pragma once

#include <cstdint>

namespace bitnet {

// Runs first .. last hold a unit; a block makes `warps` runs, `warps` apart. A block whose runs all lie
// inside the unit joined its warps' parts and left one partial, with its first run; the others left one each.
struct Kv4Join {
  int first, last, in0, in1;  // runs in0 .. in1 - 1 are those of whole blocks
  int head, blocks, count;    // partials of single runs before them, of whole blocks, and in all
  int warps;

  // The k-th partial's run.
  constexpr int run(int k) const {
    return k < head || blocks == 0 ? first + k : k < head + blocks ? in0 + (k - head) * warps : in1 + (k - head - blocks);
  }
};

// Of bounds as they were read from the workspace: no partials (count 0) where one run holds the unit, which it
// has finished, and where they cannot be a unit's of a call of n_runs runs. That is so where a wait ran
// out before they were written: whatever they are, no partial outside the workspace is looked at.
constexpr Kv4Join kv4_join(int first, int last, int n_runs, int warps) {
  Kv4Join j{first, last, 0, 0, 0, 0, 0, warps};
  if (first < 0 || first >= last || last >= n_runs) return j;
  j.in0 = first / warps * warps + warps;
  j.in1 = last / warps * warps;
  j.head = j.in0 - first;
  j.blocks = j.in0 < j.in1 ? (j.in1 - j.in0) / warps : 0;
  j.count = j.in0 < j.in1 ? j.head + j.blocks + last - j.in1 + 1 : last - first + 1;
  return j;
}

}  // namespace bitnet
