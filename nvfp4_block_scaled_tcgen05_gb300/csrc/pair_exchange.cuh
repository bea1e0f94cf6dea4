// Exchanges between the two epilogue warps e and e ^ 2 of PAIRED_ROWS tiles, numbered
// n = 0, 1, .. from the kernel's start: each warp writes half(n) of its own box, arrives at
// the pair's mbarrier, waits for it and reads the same half of the other's box.
//
// The barrier takes an arrival of both, so it cannot be more than one phase ahead of a lane
// that still waits (with a barrier per warp, at which the other one arrives, the other may
// arrive for n + 1 before the last lane has seen phase n, and that lane's parity test then
// fails for good).  A half is written again at n + 2: the writer has then waited for n + 1,
// at which the other arrived behind its reads of n.
#pragma once

namespace gb300 {

struct PairExchange {
  static constexpr int kArrivals = 2;  // that complete a phase
  static constexpr int bar(int e) { return e & 1; }  // the warp pair's mbarrier
  static constexpr unsigned parity(unsigned n) { return n & 1u; }
  static constexpr unsigned half(unsigned n) { return n & 1u; }
};

}  // namespace gb300
