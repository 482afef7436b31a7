// attn_parts.hpp -- how many workgroups share an attention call's line of work,
// and which of them a block of the grid is.  Plain arithmetic, for any compiler.
#pragma once

namespace gdn {

// Workgroups that take part, of n_wg: a grain of the line's length for each, and a
// whole number of them per key head, so that with sequences of one length, or a
// single one, no part holds the end of one head and the start of the next.  Where
// there are not that many, fewer take part, if at most `idle` are left without work
// by that (what each kernel gains and loses stands beside its number).
constexpr int attn_active(long long total, int n_wg, long long grain, int heads, int idle) {
  int active = total >= n_wg * grain
                   ? n_wg
                   : static_cast<int>((static_cast<double>(total) + grain - 1) / grain);
  if (heads <= n_wg) {
    const int up = (active + heads - 1) / heads * heads;
    if (up <= n_wg)
      active = up;
    else if (n_wg % heads <= idle)
      active = n_wg / heads * heads;
  }
  return active;
}

// Blocks are dealt out to the XCDs in turn.  Neighbours on the line share a head's
// keys: each XCD gets neighbours, for its L2, and each as many as the next (to
// within one), whatever part of the grid is active.  Blocks without work keep their
// own number, which is active or above.
constexpr int attn_spread(int block, int active, int xcds) {
  const int per = active / xcds, more = active % xcds;  // the first `more` have one more
  const int xcd = block % xcds, nth = block / xcds;
  if (nth >= per + (xcd < more ? 1 : 0)) return block;
  return xcd * per + (xcd < more ? xcd : more) + nth;
}

}  // namespace gdn
