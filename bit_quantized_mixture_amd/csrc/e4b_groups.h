// Row tiles of grouped rows, found by each wave from the groups' offsets: shared by the adapter kernels
// and the products of MXFP4 rows.
#pragma once

#include "e4b_device.h"

namespace e4b {

struct RowTile {
  int adapter;     // -1: none
  int64_t row0;
  int rows;        // 1 .. bm; 0: no such tile
};

// Inclusive sum over the wave's lanes in six steps of the vector unit: shifts by 1, 2, 4 and 8 in
// each row of 16 lanes, then a row's last lane onto the next row, and lane 31 onto the upper half.
__device__ __forceinline__ int wave_scan(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);
  return x;
}

// Rows lo .. hi of group g, clamped to the S rows there are and to ascending order.
__device__ __forceinline__ void group_rows(const int32_t* __restrict__ offsets, int g, int S, int* lo, int* hi) {
  const int a = offsets[g], b = offsets[g + 1];
  *lo = a < 0 ? 0 : (a > S ? S : a);
  *hi = b < *lo ? *lo : (b > S ? S : b);
}

__device__ __forceinline__ int adapter_of(const int32_t* __restrict__ ids, int group, int n) {
  const int a = ids ? ids[group] : group;
  return a >= 0 && a < n ? a : -1;
}

// Tile `tile` of the list that cuts every group into pieces of 1 << bm_log2 rows, found by each
// wave from the offsets, 64 groups a step (their adapters are read beside them: one latency, not two).
__device__ __forceinline__ RowTile find_tile(const int32_t* __restrict__ offsets, const int32_t* __restrict__ ids,
                                             int n_adapters, int G, int S, int bm_log2, uint32_t tile) {
  const int lane = threadIdx.x & (kWave - 1);
  int base = 0;
  for (int g0 = 0; g0 < G; g0 += kWave) {
    int lo = 0, hi = 0, a = -1;
    if (g0 + lane < G) {
      group_rows(offsets, g0 + lane, S, &lo, &hi);
      a = adapter_of(ids, g0 + lane, n_adapters);
    }
    const int n = int((int64_t(hi) - lo + (1 << bm_log2) - 1) >> bm_log2);
    const int ni = wave_scan(n);
    const int total = __builtin_amdgcn_readlane(ni, kWave - 1);
    if (int(tile) - base < total) {
      const int l = __ffsll((unsigned long long)__ballot(int(tile) - base < ni)) - 1;
      const int at = int(tile) - base - (__builtin_amdgcn_readlane(ni, l) - __builtin_amdgcn_readlane(n, l));
      if (at < 0 || at >= __builtin_amdgcn_readlane(n, l)) break;  // sums of offsets that descend can wrap
      const int row0 = __builtin_amdgcn_readlane(lo, l) + (at << bm_log2);
      const int left = __builtin_amdgcn_readlane(hi, l) - row0;
      return RowTile{__builtin_amdgcn_readlane(a, l), row0, left < (1 << bm_log2) ? left : (1 << bm_log2)};
    }
    base += total;
  }
  return RowTile{-1, 0, 0};
}

}  // namespace e4b
