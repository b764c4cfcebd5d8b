// How the launch of the head norm and rotation deals out its work (host; the tests compile it alone).
#pragma once

#include <stdint.h>

namespace ttl {

constexpr int kHeadWarps = 8;        // of a block
constexpr int kHeadMostSms = 152;    // of the card; the backward pass's workspace has a row for each block on as many

// Lanes that share a head of d columns, 16 each: a power of two.
inline int head_lanes(int d) {
  int l = 1;
  while (l * 16 < d) l *= 2;
  return l;
}

struct HeadDeal {
  int64_t groups;                    // of the tokens that a warp works on together
  int64_t warps;                     // that share the pairs of a group and a head evenly
  unsigned blocks;
};

// The shares are even, so the blocks are no more than the device holds at once, `resident` on each of its `sms`: one that
// waited for a place would run its whole share behind the others.
inline HeadDeal head_deal(int64_t T, int64_t heads, int d, int resident, int sms) {
  const int tokens = 32 / head_lanes(d);
  HeadDeal r;
  r.groups = (T + tokens - 1) / tokens;
  const int64_t pairs = r.groups * heads;
  const int64_t most = static_cast<int64_t>(resident) * (sms < kHeadMostSms ? sms : kHeadMostSms) * kHeadWarps;
  r.warps = pairs < most ? pairs : most;
  r.blocks = static_cast<unsigned>((r.warps + kHeadWarps - 1) / kHeadWarps);
  return r;
}

}  // namespace ttl
