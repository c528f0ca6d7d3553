// Token rows to expert order and back: the gather in front of the grouped products, the weighted
// combine behind them, and their gradients, as calls of their own (grouped-nf4-gemm 0.25.0
// project description, opening section: the combine among the glue kernels).  With slot
// s = t*k + j, sorted_slots[p] = s the slot of row p, and inv[s] = p:
//   permute           rows[p] = x[s / k]
//   combine           out[t] = sum_j w[t, j] * rows[inv[s]]     (w = 1: permute's gradient)
//   combine backward  g_rows[inv[s]] = w[t, j] * g_out[t],  g_w[t, j] = <g_out[t], rows[inv[s]]>
// Every kernel is bound by memory: a team of lanes (a power of two, a wave for rows of 512
// columns and more) walks one row with 16-byte accesses, sums are float32 in a fixed order.
#include "e4b_internal.h"
#include "e4b_rows.h"

namespace e4b {

namespace {

constexpr int kThreads = 256;
// Up to this many slots a kernel that needs inv finds its tokens' rows by reading sorted_slots
// itself (16 KB from the L2 cache for each workgroup, all loads in flight); beyond, one small launch
// or two write inv to the workspace.  Combine of float32 rows of 2048, us itself and behind a launch:
// 1024 slots 4.4 and 7.5, 4096 slots 9.2 and 10.0, 6400 slots 18.9 and 15.5.
constexpr int64_t kScanSlots = 4096;

__global__ void __launch_bounds__(kThreads) fill_inv_kernel(int32_t* __restrict__ inv, int64_t S) {
  const int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  if (i < S) inv[i] = -1;
}

// The highest row wins where a slot is named twice, so the result does not depend on the order.
__global__ void __launch_bounds__(kThreads) scatter_inv_kernel(const int32_t* __restrict__ slots, int64_t S,
                                                               int32_t* __restrict__ inv) {
  const int64_t p = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  if (p >= S) return;
  const int32_t s = slots[p];
  if (s >= 0 && s < S) atomicMax(inv + s, int32_t(p));
}

// inv in one launch: a workgroup has kRange slots in LDS and reads all of sorted_slots for them.  Up
// to kRangeSlots slots (256 KB to read, from the L2 cache) one such launch takes about as long as
// either of the two above (the gradient of 7862 small tokens 19.9 us with two, 17.4 with one; at
// 131072 slots it is 6 us longer than the two).
constexpr int kRange = 2048, kRangeThreads = 1024;
constexpr int64_t kRangeSlots = 65536;

__global__ void __launch_bounds__(kRangeThreads) range_inv_kernel(const int32_t* __restrict__ slots, int S,
                                                                  int32_t* __restrict__ inv) {
  __shared__ int32_t found[kRange];
  const int s0 = int(blockIdx.x) * kRange, n = S - s0 < kRange ? S - s0 : kRange;
  for (int i = threadIdx.x; i < kRange; i += kRangeThreads) found[i] = -1;
  __syncthreads();
  const int n4 = S >> 2;
#pragma unroll 4
  for (int q = threadIdx.x; q < n4; q += kRangeThreads) {
    const u32x4 v = reinterpret_cast<const u32x4*>(slots)[q];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t d = v[j] - uint32_t(s0);
      if (d < uint32_t(n)) atomicMax(found + d, 4 * q + j);
    }
  }
  for (int p = 4 * n4 + threadIdx.x; p < S; p += kRangeThreads) {
    const uint32_t d = uint32_t(slots[p]) - uint32_t(s0);
    if (d < uint32_t(n)) atomicMax(found + d, p);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kRangeThreads) inv[s0 + i] = found[i];
}

// Rows of the slots s0 .. s0 + n - 1 into found[0 .. n - 1] (LDS), -1 where no row names the slot.
__device__ __forceinline__ void scan_slots(const int32_t* __restrict__ slots, int S, int64_t s0, int n,
                                           int32_t* found) {
  for (int i = threadIdx.x; i < n; i += kThreads) found[i] = -1;
  __syncthreads();
  const int n4 = S >> 2;
#pragma unroll 4
  for (int q = threadIdx.x; q < n4; q += kThreads) {
    const u32x4 v = reinterpret_cast<const u32x4*>(slots)[q];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t d = int64_t(int32_t(v[j])) - s0;
      if (d >= 0 && d < n) atomicMax(found + d, 4 * q + j);
    }
  }
  for (int p = 4 * n4 + threadIdx.x; p < S; p += kThreads) {
    const int64_t d = int64_t(slots[p]) - s0;
    if (d >= 0 && d < n) atomicMax(found + d, p);
  }
  __syncthreads();
}

// rows[p] = x[slots[p] / k]; `halves` 2-byte units a row, moved as they are.  A slot outside
// [0, S) leaves a row of zeros.  67 MB of rows take 21 us.
__global__ void __launch_bounds__(kThreads) permute_kernel(const uint16_t* __restrict__ x,
                                                           const int32_t* __restrict__ slots, int64_t S,
                                                           int64_t halves, int k, int team_log2,
                                                           uint16_t* __restrict__ rows) {
  const int team = 1 << team_log2;
  int64_t p = (int64_t(blockIdx.x) * kThreads + threadIdx.x) >> team_log2;
  if (p >= S) return;
  const int lane = threadIdx.x & (team - 1);
  const int32_t s = slots[p];
  const bool named = s >= 0 && s < S;
  const uint16_t* src = x + int64_t(named ? s / k : 0) * halves;
  uint16_t* dst = rows + p * halves;
  const int64_t n8 = halves >> 3;
  constexpr int kUnroll = 4;
  int64_t c = lane;
  for (; c + (kUnroll - 1) * team < n8; c += kUnroll * team) {
    u32x4 v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) v[u] = *reinterpret_cast<const u32x4_any*>(src + 8 * (c + u * team));
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      *reinterpret_cast<u32x4_any*>(dst + 8 * (c + u * team)) = named ? v[u] : u32x4{0, 0, 0, 0};
  }
  for (; c < n8; c += team) {
    const u32x4 v = *reinterpret_cast<const u32x4_any*>(src + 8 * c);
    *reinterpret_cast<u32x4_any*>(dst + 8 * c) = named ? v : u32x4{0, 0, 0, 0};
  }
  for (int64_t h = 8 * n8 + lane; h < halves; h += team) dst[h] = named ? src[h] : uint16_t(0);
}

// The same in token order: a team item is up to 512 columns of one token, read once and written to
// the k rows of its slots.  The gather above reads each x row k times (from the memory-side cache,
// beside the stream of rows): 1.07 GB of rows took 310 us against 233 a call here, with stores that are
// not kept in the caches; 225 of them in this kernel, 5.4 TB/s.  Behind the items, workgroups look for
// rows that inv does not lead to (a slot out of range: zeros; a slot that a higher row names too) and
// write them by themselves.
__global__ void __launch_bounds__(kThreads) permute_scatter_kernel(const uint16_t* __restrict__ x,
                                                                   const int32_t* __restrict__ slots,
                                                                   const int32_t* __restrict__ inv, int64_t T,
                                                                   int64_t halves, int k, int team_log2,
                                                                   int64_t chunks, int64_t item_blocks,
                                                                   uint16_t* __restrict__ rows) {
  const int64_t S = T * k;
  if (blockIdx.x >= item_blocks) {
    __shared__ int32_t left[kThreads];
    __shared__ int32_t n_left;
    if (threadIdx.x == 0) n_left = 0;
    __syncthreads();
    const int64_t p = (int64_t(blockIdx.x) - item_blocks) * kThreads + threadIdx.x;
    if (p < S) {
      const int32_t s = slots[p];
      if (s < 0 || s >= S || inv[s] != p) left[atomicAdd(&n_left, 1)] = int32_t(p);
    }
    __syncthreads();
    for (int i = 0; i < n_left; ++i) {
      const int64_t r = left[i];
      const int32_t s = slots[r];
      const bool named = s >= 0 && s < S;
      for (int64_t h = threadIdx.x; h < halves; h += kThreads)
        rows[r * halves + h] = named ? x[(s / k) * halves + h] : uint16_t(0);
    }
    return;
  }
  const int team = 1 << team_log2;
  const int64_t item = (int64_t(blockIdx.x) * kThreads + threadIdx.x) >> team_log2;
  if (item >= T * chunks) return;
  const int64_t t = item / chunks;
  const int64_t c = ((item - t * chunks) * team + (threadIdx.x & (team - 1))) * 8;
  if (c >= halves) return;
  const uint16_t* src = x + t * halves + c;
  if (c + 8 <= halves) {
    const u32x4 v = *reinterpret_cast<const u32x4_any*>(src);
    for (int j = 0; j < k; ++j) {
      const int64_t p = inv[t * k + j];
      if (p >= 0 && p < S) __builtin_nontemporal_store(v, reinterpret_cast<u32x4_any*>(rows + p * halves + c));
    }
  } else {
    for (int j = 0; j < k; ++j) {
      const int64_t p = inv[t * k + j];
      if (p >= 0 && p < S)
        for (int64_t h = 0; c + h < halves; ++h) rows[p * halves + c + h] = src[h];
    }
  }
}

// One team item: V columns a lane of one token.  The loads of eight rows go out before the first
// is used.  131072 float32 rows of 4096 (2.28 GB) take 364 us, 6.3 TB/s; 12297 bf16 rows of 2880 into
// float32 (118 MB) 24 us, 4.9 TB/s; one token's eight rows of 2048 3.5 us, a chain of latencies.
template <int RDT, int ODT, int V, bool SCAN, bool ONCE>
__global__ void __launch_bounds__(kThreads) combine_rows_kernel(const row_elem<RDT>* __restrict__ rows,
                                                                const float* __restrict__ w,
                                                                const int32_t* __restrict__ inv_or_slots,
                                                                int64_t T, int64_t H, int k, int team_log2,
                                                                int64_t chunks,
                                                                row_elem<ODT>* __restrict__ out) {
  __shared__ int32_t found[SCAN ? kScanSlots : 1];
  const int team = 1 << team_log2;
  const int64_t S = T * k;
  const int64_t items = T * chunks;  // chunk c of token t: item t * chunks + c
  const int64_t first = (int64_t(blockIdx.x) * kThreads) >> team_log2;
  int64_t item = first + (int(threadIdx.x) >> team_log2);
  const int64_t t0 = first / chunks;
  if (SCAN) {
    int64_t last = first + (kThreads >> team_log2) - 1;
    if (last >= items) last = items - 1;
    scan_slots(inv_or_slots, int(S), t0 * k, int((last / chunks - t0 + 1) * k), found);
  }
  if (item >= items) return;
  int64_t t = item / chunks;
  if (team == kWave) t = (int64_t(__builtin_amdgcn_readfirstlane(int(t >> 32))) << 32) |
                         uint32_t(__builtin_amdgcn_readfirstlane(int(t)));
  const int64_t c = ((item - t * chunks) * team + (threadIdx.x & (team - 1))) * V;
  if (c >= H) return;
  const bool full = c + V <= H;
  float acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.f;
  constexpr int kRowsAhead = 8;
  for (int j0 = 0; j0 < k; j0 += kRowsAhead) {
    float v[kRowsAhead][V];
    float wj[kRowsAhead];
#pragma unroll
    for (int u = 0; u < kRowsAhead; ++u) {
      const int j = j0 + u;
      int64_t p = -1;
      if (j < k) p = SCAN ? found[(t - t0) * k + j] : inv_or_slots[t * k + j];
      wj[u] = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) v[u][i] = 0.f;
      if (p >= 0 && p < S) {  // a slot without a row adds nothing
        wj[u] = w ? w[t * k + j] : 1.f;
        const row_elem<RDT>* r = rows + p * H + c;
        if (full) {
          if constexpr (ONCE) load_once<V>(r, v[u]);
          else load_vec<V>(r, v[u]);
        } else {
#pragma unroll
          for (int i = 0; i < V; ++i)
            if (c + i < H) v[u][i] = load1(r + i);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kRowsAhead; ++u)
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] = fmaf(wj[u], v[u][i], acc[i]);
  }
  row_elem<ODT>* o = out + t * H + c;
  if (full) {
    store_vec<V>(o, acc);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (c + i < H) store1(o + i, acc[i]);
  }
}

// A team for each slot s = t*k + j: reads g_out[t] (the k teams of a token share it in the
// caches), writes its row's gradient, and sums the weight's gradient over the row.  8192 float32 rows
// of 2880 with bf16 gradients (153 MB) take 32 us, 4.8 TB/s.
template <int GDT, int RDT, int DDT, bool SCAN, bool GW, bool ONCE>
__global__ void __launch_bounds__(kThreads) combine_backward_kernel(
    const row_elem<GDT>* __restrict__ g_out, const row_elem<RDT>* __restrict__ rows,
    const float* __restrict__ w, const int32_t* __restrict__ inv_or_slots, int64_t S, int64_t H, int k,
    int team_log2, row_elem<DDT>* __restrict__ g_rows, float* __restrict__ g_w) {
  __shared__ int32_t found[SCAN ? kThreads : 1];
  const int team = 1 << team_log2;
  const int64_t s0 = (int64_t(blockIdx.x) * kThreads) >> team_log2;
  if (SCAN) scan_slots(inv_or_slots, int(S), s0, kThreads >> team_log2, found);
  const int64_t s = s0 + (int(threadIdx.x) >> team_log2);
  const int lane = threadIdx.x & (team - 1);
  float sum = 0.f;
  int64_t p = -1;
  if (s < S) p = SCAN ? found[s - s0] : inv_or_slots[s];
  if (p >= 0 && p < S) {
    const float ws = w[s];
    const row_elem<GDT>* g = g_out + (s / k) * H;
    const row_elem<RDT>* r = GW ? rows + p * H : nullptr;
    row_elem<DDT>* d = g_rows + p * H;
    const int64_t n8 = H >> 3;
#pragma unroll 2
    for (int64_t c = lane; c < n8; c += team) {
      float gv[8], rv[8];
      load_vec<8>(g + 8 * c, gv);
      if (GW) {
        if constexpr (ONCE) load_once<8>(r + 8 * c, rv);
        else load_vec<8>(r + 8 * c, rv);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fmaf(gv[i], rv[i], sum);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) gv[i] *= ws;
      store_vec<8>(d + 8 * c, gv);
    }
    for (int64_t h = 8 * n8 + lane; h < H; h += team) {
      const float gv = load1(g + h);
      if (GW) sum = fmaf(gv, load1(r + h), sum);
      store1(d + h, gv * ws);
    }
  }
  if (GW) {
    for (int m = 1; m < team; m <<= 1) sum += __shfl_xor(sum, m, kWave);
    if (s < S && lane == 0) g_w[s] = sum;  // 0 for a slot without a row
  }
}

// Lanes a row of n vectors is given: the power of two that covers it, a wave at most.
int team_log2_of(int64_t n) {
  int l = 0;
  while (l < 6 && (int64_t(1) << l) < n) ++l;
  return l;
}

unsigned blocks_of(int64_t items, int team_log2) {
  const int64_t per = kThreads >> team_log2;
  return unsigned((items + per - 1) / per);
}

hipError_t launch_inv(const int32_t* slots, int64_t S, int32_t* inv, hipStream_t stream) {
  if (S <= kRangeSlots) {
    hipLaunchKernelGGL(range_inv_kernel, dim3(unsigned((S + kRange - 1) / kRange)), dim3(kRangeThreads), 0, stream,
                       slots, int(S), inv);
    return hipGetLastError();
  }
  const unsigned grid = unsigned((S + kThreads - 1) / kThreads);
  hipLaunchKernelGGL(fill_inv_kernel, dim3(grid), dim3(kThreads), 0, stream, inv, S);
  hipLaunchKernelGGL(scatter_inv_kernel, dim3(grid), dim3(kThreads), 0, stream, slots, S, inv);
  return hipGetLastError();
}

// Whether rows of so many bytes are read past the caches: what the memory-side cache (256 MB) cannot
// have kept (2.1 GB: 405 us through it, 372 past it), and not what it may still have from the call
// that wrote it (combine and its gradient over 71 and 94 MB: 27 and 32 us through it, 35 and 35 past).
bool past_cache(int64_t bytes) { return bytes > (int64_t(256) << 20); }

template <int RDT, int ODT, int V>
void combine_types(const CombineLaunch& L, bool scan, hipStream_t stream) {
  const int64_t n = (L.H + V - 1) / V;
  const int tl = team_log2_of(n);
  const int64_t chunks = (n + (1 << tl) - 1) >> tl;
  const unsigned grid = blocks_of(L.T * chunks, tl);
  const auto* rows = static_cast<const row_elem<RDT>*>(L.rows);
  auto* out = static_cast<row_elem<ODT>*>(L.out);
  if (scan)
    hipLaunchKernelGGL((combine_rows_kernel<RDT, ODT, V, true, false>), dim3(grid), dim3(kThreads), 0, stream, rows,
                       L.w, L.slots, L.T, L.H, L.k, tl, chunks, out);
  else if (past_cache(L.T * L.k * L.H * int64_t(sizeof(row_elem<RDT>))))
    hipLaunchKernelGGL((combine_rows_kernel<RDT, ODT, V, false, true>), dim3(grid), dim3(kThreads), 0, stream, rows,
                       L.w, L.inv, L.T, L.H, L.k, tl, chunks, out);
  else
    hipLaunchKernelGGL((combine_rows_kernel<RDT, ODT, V, false, false>), dim3(grid), dim3(kThreads), 0, stream, rows,
                       L.w, L.inv, L.T, L.H, L.k, tl, chunks, out);
}

template <int GDT, int RDT, int DDT, bool GW>
void backward_types(const CombineBackwardLaunch& L, bool scan, hipStream_t stream) {
  const int64_t S = L.T * L.k;
  const int tl = team_log2_of((L.H + 7) / 8);
  const unsigned grid = blocks_of(S, tl);
  const auto* g = static_cast<const row_elem<GDT>*>(L.g_out);
  const auto* rows = static_cast<const row_elem<RDT>*>(L.rows);
  auto* d = static_cast<row_elem<DDT>*>(L.g_rows);
  if (scan)
    hipLaunchKernelGGL((combine_backward_kernel<GDT, RDT, DDT, true, GW, false>), dim3(grid), dim3(kThreads), 0, stream,
                       g, rows, L.w, L.slots, S, L.H, L.k, tl, d, L.g_w);
  else if (GW && past_cache(S * L.H * int64_t(sizeof(row_elem<RDT>))))
    hipLaunchKernelGGL((combine_backward_kernel<GDT, RDT, DDT, false, GW, GW>), dim3(grid), dim3(kThreads), 0, stream,
                       g, rows, L.w, L.inv, S, L.H, L.k, tl, d, L.g_w);
  else
    hipLaunchKernelGGL((combine_backward_kernel<GDT, RDT, DDT, false, GW, false>), dim3(grid), dim3(kThreads), 0,
                       stream, g, rows, L.w, L.inv, S, L.H, L.k, tl, d, L.g_w);
}

template <int GDT, int DDT>
void backward_rows(const CombineBackwardLaunch& L, bool scan, hipStream_t stream) {
  if (!L.g_w)
    backward_types<GDT, 0, DDT, false>(L, scan, stream);
  else if (L.rows_dtype == 0)
    backward_types<GDT, 0, DDT, true>(L, scan, stream);
  else
    backward_types<GDT, 1, DDT, true>(L, scan, stream);
}

}  // namespace

int64_t combine_inv_slots(int64_t S) { return S > kScanSlots ? S : 0; }

// Work items of the largest grid each launcher starts for the sizes (the caller checks them against
// a launch's limit; the slots' inverse has T * k at most).
int64_t permute_items(int64_t T, int64_t H, int k, int elem_halves) {
  const int64_t n = (H * elem_halves + 7) / 8, S = T * k;
  const int tl = team_log2_of(n);
  const int64_t per = kThreads >> tl, chunks = (n + (1 << tl) - 1) >> tl;
  if (permute_inv_slots(T, H, k, elem_halves) == 0) return (S + per - 1) / per * kThreads;
  return ((T * chunks + per - 1) / per + (S + kThreads - 1) / kThreads) * kThreads;
}
int64_t combine_items(int64_t T, int64_t H, int rows_dtype) {
  const int V = rows_dtype == 0 ? 8 : 4;
  const int64_t n = (H + V - 1) / V;
  const int tl = team_log2_of(n);
  const int64_t per = kThreads >> tl;
  return (T * ((n + (1 << tl) - 1) >> tl) + per - 1) / per * kThreads;
}
int64_t combine_backward_items(int64_t T, int64_t H, int k) {
  const int64_t per = kThreads >> team_log2_of((H + 7) / 8);
  return (T * k + per - 1) / per * kThreads;
}

// Token order from 128 MB of rows on, where what it saves (a fifth to a quarter of the time) is more
// than the two launches that invert the slots; 67 MB: 21 us gathered, 15 and about 5 in token order.
int64_t permute_inv_slots(int64_t T, int64_t H, int k, int elem_halves) {
  return k > 1 && T * k * H * 2 * elem_halves >= (int64_t(128) << 20) ? T * k : 0;
}

hipError_t launch_permute(const void* x, int elem_halves, int64_t T, int64_t H, int k, const int32_t* slots,
                          void* rows, int32_t* inv, hipStream_t stream) {
  const int64_t halves = H * elem_halves, S = T * k;
  const int tl = team_log2_of((halves + 7) / 8);
  if (permute_inv_slots(T, H, k, elem_halves)) {
    if (hipError_t e = launch_inv(slots, S, inv, stream); e != hipSuccess) return e;
    const int64_t chunks = ((halves + 7) / 8 + (1 << tl) - 1) >> tl, items = blocks_of(T * chunks, tl);
    hipLaunchKernelGGL(permute_scatter_kernel, dim3(unsigned(items + (S + kThreads - 1) / kThreads)), dim3(kThreads),
                       0, stream, static_cast<const uint16_t*>(x), slots, inv, T, halves, k, tl, chunks, items,
                       static_cast<uint16_t*>(rows));
    return hipGetLastError();
  }
  hipLaunchKernelGGL(permute_kernel, dim3(blocks_of(S, tl)), dim3(kThreads), 0, stream,
                     static_cast<const uint16_t*>(x), slots, S, halves, k, tl, static_cast<uint16_t*>(rows));
  return hipGetLastError();
}

hipError_t launch_combine(const CombineLaunch& L, hipStream_t stream) {
  const int64_t S = L.T * L.k;
  const bool scan = combine_inv_slots(S) == 0;
  if (!scan)
    if (hipError_t e = launch_inv(L.slots, S, L.inv, stream); e != hipSuccess) return e;
  if (L.rows_dtype == 0) {
    if (L.out_dtype == 0) combine_types<0, 0, 8>(L, scan, stream);
    else combine_types<0, 1, 8>(L, scan, stream);
  } else {
    if (L.out_dtype == 0) combine_types<1, 0, 4>(L, scan, stream);
    else combine_types<1, 1, 4>(L, scan, stream);
  }
  return hipGetLastError();
}

hipError_t launch_combine_backward(const CombineBackwardLaunch& L, hipStream_t stream) {
  const int64_t S = L.T * L.k;
  const bool scan = combine_inv_slots(S) == 0;
  if (!scan)
    if (hipError_t e = launch_inv(L.slots, S, L.inv, stream); e != hipSuccess) return e;
  if (L.g_dtype == 0) {
    if (L.g_rows_dtype == 0) backward_rows<0, 0>(L, scan, stream);
    else backward_rows<0, 1>(L, scan, stream);
  } else {
    if (L.g_rows_dtype == 0) backward_rows<1, 0>(L, scan, stream);
    else backward_rows<1, 1>(L, scan, stream);
  }
  return hipGetLastError();
}

}  // namespace e4b
