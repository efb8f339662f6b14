// The row tiles of a grouped product: rows offsets[g] .. offsets[g + 1] - 1 belong to group g, and no tile crosses a
// group's end. P is the kernel's parameters: offsets (null: one group of all rows), M and G.
#pragma once
#include "moe_device.h"
#include "moe_internal.h"

namespace moe {

// LDS prefix sums of the groups' tile counts
struct Groups {
  int tile0[kMaxExperts + 1];
  int row0[kMaxExperts + 1];   // clamped offsets
};

template <class P>
__device__ __forceinline__ int clamped_offset(const P& p, int g) { return min(max(p.offsets[g], 0), (int)p.M); }

// fills s and returns the number of M-tiles of BM rows
template <int BM, class P>
__device__ __forceinline__ int group_tiles(const P& p, Groups& s) {
  if (!p.offsets) return (int)((p.M + BM - 1) / BM);
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x, per = (p.G + 63) >> 6, g0 = lane * per;
    int t = 0;
    for (int i = 0; i < per; ++i)
      if (g0 + i < p.G) t += (max(clamped_offset(p, g0 + i + 1) - clamped_offset(p, g0 + i), 0) + BM - 1) / BM;
    int inc = t;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(inc, d);
      if (lane >= d) inc += o;
    }
    int at = inc - t;
    for (int i = 0; i < per; ++i) {
      const int g = g0 + i;
      if (g >= p.G) break;
      const int a = clamped_offset(p, g), b = max(clamped_offset(p, g + 1), a);
      s.tile0[g] = at;
      s.row0[g] = a;
      at += (b - a + BM - 1) / BM;
    }
    if (lane == 63) {
      s.tile0[p.G] = inc;
      s.row0[p.G] = clamped_offset(p, p.G);
    }
  }
  __syncthreads();
  return s.tile0[p.G];
}

// M-tile mt: its group g, first row r0 and the group's last row + 1
template <int BM, class P>
__device__ __forceinline__ void find_tile(const P& p, const Groups& s, int mt, int& g, int& r0, int& end) {
  g = 0;
  r0 = mt * BM;
  end = (int)p.M;
  if (!p.offsets) return;
  int lo = 0, hi = p.G;   // the last group whose first tile is not past mt
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s.tile0[mid] <= mt) lo = mid;
    else hi = mid;
  }
  g = __builtin_amdgcn_readfirstlane(lo);
  r0 = __builtin_amdgcn_readfirstlane(s.row0[g] + (mt - s.tile0[g]) * BM);
  end = __builtin_amdgcn_readfirstlane(max(s.row0[g + 1], s.row0[g]));
}

}  // namespace moe
