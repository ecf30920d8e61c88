// What an occupancy query's answer means for launches of clusters (host, plain C++).
#pragma once

#include <algorithm>
#include <cstdint>

namespace moe {

// Clusters of `size` CTAs that run at once, of a query's answer `n` (`ok`: it had one) on `sms` SMs.  Pairs, which every form
// comes back to, are taken to fit where the query does not say so; larger clusters are not, and none fit: -1.
inline int clusters_that_fit(bool ok, int n, int sms, int size) {
  const int most = sms / size;
  if (ok && n > 0 && most > 0) return std::min(n, most);
  return size == 2 ? most : -1;
}

// How many pairs share a tile's contraction: as many of four or two as leave all tiles running at once, else one.
// `fit(pairs)`: how many clusters of so many pairs do.
template <class Fit>
int pairs_per_tile(int64_t tiles, Fit fit) {
  for (const int pairs : {4, 2})
    if (tiles <= fit(pairs)) return pairs;
  return 1;
}

}  // namespace moe
