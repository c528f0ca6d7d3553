// The gated activation between the two products on rows, its gradient, and rows kept in 8 bits
// for the backward pass:
//   checkpoint  per 32 columns of a row: X = floor(log2 amax), one more where the largest would round
//               to 128 steps; q = rint(v 2^(6 - X)) in [-127, 127]; kept as int8 and the byte X + 127
//   restore     v' = q 2^(X - 6): a bf16 value exactly (7 bits and a sign), off by half a step at most
//   glu         h = G s(G) U, or with Gc = min(G, 7), Uc = clip(U, -7, 7): Gc s(1.702 Gc) (Uc + 1)
//   its gradient  dG = g U s (1 + G (1 - s)), dU = g G s; clamped: dG = [G <= 7] g (Uc + 1) s
//               (1 + 1.702 Gc (1 - s)), dU = [|U| <= 7] g Gc s
// Twenty operations for an element of 3 to 14 bytes: memory bounds all four.  A lane has 8 columns,
// or 4 of float32 rows, and neighbouring lanes neighbouring ones, so every access is whole lines; what is read once and
// written once goes past the caches.  A block's largest meets over 4 or 8 lanes of the vector unit: no LDS.
#include <type_traits>

#include "e4b_internal.h"
#include "e4b_rows.h"

namespace e4b {

namespace {

constexpr int kThreads = 256;

// Elements of a lane: what 16 bytes of a float32 row hold, else 8.
template <int DT> constexpr int lane_elems = DT == 1 ? 4 : 8;

// The largest of a value over the LANES neighbouring lanes that share a block of 32 (4 or 8).
template <int LANES>
__device__ __forceinline__ uint32_t block_max(uint32_t m) {
  m = max(m, uint32_t(__builtin_amdgcn_update_dpp(0, int(m), 0xB1, 0xf, 0xf, false)));   // lane ^ 1
  m = max(m, uint32_t(__builtin_amdgcn_update_dpp(0, int(m), 0x4E, 0xf, 0xf, false)));   // lane ^ 2
  if (LANES == 8) m = max(m, uint32_t(__builtin_amdgcn_update_dpp(0, int(m), 0x141, 0xf, 0xf, false)));  // 7 - lane
  return m;
}

// The exponent byte X + 127 of a block whose largest magnitude has these bits; 255 where it holds a NaN
// or an infinity.  The largest mantissas round to 128 steps: adding half a step there carries into the
// exponent (below 2^-126 the step is the subnormals', 2^16 of their units).  At the top, where that
// would be 2^128, the block stays at 2^127 and its largest saturate.
__device__ __forceinline__ uint32_t block_exponent(uint32_t amax) {
  if (amax >= 0x7F800000u) return 255u;
  if (amax < 0x00800000u) return amax >= 0x007F8000u ? 1u : 0u;
  const uint32_t e = (amax + 0x00010000u) >> 23;
  return e < 255u ? e : 254u;
}

// V values as int8 (in words, the first in the low byte).  Adding 1.5 * 2^23 rounds to the nearest even
// whole number and leaves it, in two's complement, in the low bits.
template <int V>
__device__ __forceinline__ void quantize8(const float (&v)[V], uint32_t byte, uint32_t (&q)[V / 4]) {
  const int up = 133 - int(byte);
#pragma unroll
  for (int w = 0; w < V / 4; ++w) {
    uint32_t b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float s = __builtin_amdgcn_fmed3f(__builtin_amdgcn_ldexpf(v[4 * w + j], up), -127.f, 127.f);
      b[j] = __float_as_uint(s + 12582912.f);
    }
    const uint32_t lo = perm(b[1], b[0], 0x0C0C0400u), hi = perm(b[3], b[2], 0x0C0C0400u);
    q[w] = byte == 255u ? 0u : perm(hi, lo, 0x05040100u);
  }
}

template <int V>
__device__ __forceinline__ uint32_t amax_bits(const float (&v)[V]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  return m;
}

// Stores V values' codes and, by the block's first lane, its byte.  `off` counts elements.
template <int V>
__device__ __forceinline__ void checkpoint(const float (&v)[V], int64_t off, int8_t* __restrict__ codes,
                                           uint8_t* __restrict__ scales) {
  const uint32_t byte = block_exponent(block_max<32 / V>(amax_bits(v)));
  uint32_t q[V / 4];
  quantize8(v, byte, q);
  if constexpr (V == 8) __builtin_nontemporal_store(u32x2{q[0], q[1]}, reinterpret_cast<u32x2*>(codes + off));
  else __builtin_nontemporal_store(q[0], reinterpret_cast<uint32_t*>(codes + off));
  if ((off & 31) == 0) scales[off >> 5] = uint8_t(byte);
}

// Rows as they come: bf16 or float32, or 8 bits with their exponent bytes (DT 2).
struct RowsIn {
  const void* rows;
  const uint8_t* scales;
};
template <int DT, int V>
__device__ __forceinline__ void load_in(const RowsIn& p, int64_t off, float (&v)[V]) {
  if constexpr (DT == 2) {
    static_assert(V == 8, "");
    const u32x2 q = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(static_cast<const int8_t*>(p.rows) + off));
    const float s = scale8(p.scales[off >> 5]);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = float(int(int8_t(q[i >> 2] >> (8 * (i & 3))))) * s;
  } else {
    load_once<V>(static_cast<const row_elem<DT>*>(p.rows) + off, v);
  }
}

// 131072 rows of 4096 bf16: 271 us (6.0 TB/s).
struct KeepArgs {
  RowsIn in;
  int8_t* codes;
  uint8_t* scales;
  int64_t items;          // of lane_elems elements each
};
template <int DT>
__global__ void __launch_bounds__(kThreads) checkpoint_kernel(KeepArgs p) {
  constexpr int V = lane_elems<DT>;
  const int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= p.items) return;  // a block's lanes all go or all stay
  float v[V];
  load_in<DT, V>(p.in, V * i, v);
  checkpoint<V>(v, V * i, p.codes, p.scales);
}

// The same rows back: 261 us (6.2 TB/s).
struct RestoreArgs {
  RowsIn in;
  void* out;
  int64_t items;
};
template <int ODT>
__global__ void __launch_bounds__(kThreads) restore_kernel(RestoreArgs p) {
  const int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= p.items) return;
  float v[8];
  load_in<2, 8>(p.in, 8 * i, v);
  store_vec<8>(static_cast<row_elem<ODT>*>(p.out) + 8 * i, v);
}

// Gate and up of V pairs.  `off`: the gates' first element, the ups stand I further on; interleaved, the
// first pair's, and the 2 V elements are one run.
struct GluArgs {
  RowsIn in;
  const void* g;          // the gradient of h (backward)
  void* out;              // h, or the gradient of the rows
  int8_t* codes;          // nullable: the rows' checkpoint (forward)
  uint8_t* scales;
  int64_t I;
  uint32_t items, per;    // of the call, of a row
};

// s(t) and 1 - s(t), the logistic function, from e^-|t|, which cannot overflow: below -87.3 it is 0 as e is.
// NaN stays NaN.
__device__ __forceinline__ void logistic(float t, float* s, float* rest) {
  const float e = __expf(-fabsf(t)), near = __builtin_amdgcn_rcpf(1.f + e), far = e * near;
  *s = t < 0.f ? far : near;
  *rest = t < 0.f ? near : far;
}
// The clamped form's t.  Far below, where s(t) is 0, t stays finite, so that t s(t) is 0 too, for a gate of -inf as
// well (the gate itself times s(t) is NaN there, as the formula has it).
__device__ __forceinline__ float steep(float gc) { return gc < -128.f ? -128.f : 1.702f * gc; }

template <bool CLAMPED>
__device__ __forceinline__ float glu(float g, float u) {
  float s, rest;
  if (!CLAMPED) {
    logistic(g, &s, &rest);
    return g * s * u;
  }
  const float gc = g > 7.f ? 7.f : g, uc = u > 7.f ? 7.f : (u < -7.f ? -7.f : u);  // NaN stays NaN
  logistic(steep(gc), &s, &rest);
  return gc * s * (uc + 1.f);
}
// The factor of the gate's gradient is taken first: it lies in [-0.1, 1.1] for every finite gate.  For an infinite one it
// is NaN in the silu form; in the clamped form 0.
template <bool CLAMPED>
__device__ __forceinline__ void glu_grad(float g, float gate, float up, float* d_gate, float* d_up) {
  float s, rest;
  if (!CLAMPED) {
    logistic(gate, &s, &rest);
    *d_gate = (s + gate * s * rest) * up * g;
    *d_up = gate * s * g;
    return;
  }
  const float gc = gate > 7.f ? 7.f : gate, uc = up > 7.f ? 7.f : (up < -7.f ? -7.f : up);
  const float t = steep(gc);
  logistic(t, &s, &rest);
  *d_gate = gate > 7.f ? 0.f : (s + t * s * rest) * (uc + 1.f) * g;
  *d_up = up > 7.f || up < -7.f ? 0.f : gc * s * g;
}

// 8192 rows of 2 x 14336 float32 to bf16, with their checkpoint: 228 us (6.2 TB/s); without it the rows would be read
// again for it (a second launch, 0.94 GB more).
// An item is V elements of gates and V of ups (halves), or V elements of pairs (interleaved).  Its h
// has V or V / 2 columns.
template <int DT, int ODT, bool CLAMPED, bool INTER, bool KEEP>
__global__ void __launch_bounds__(kThreads) glu_kernel(GluArgs p) {
  constexpr int V = lane_elems<DT>, H = INTER ? V / 2 : V;
  const uint32_t i = blockIdx.x * uint32_t(kThreads) + threadIdx.x;
  if (i >= p.items) return;
  row_elem<ODT>* out = static_cast<row_elem<ODT>*>(p.out) + int64_t(H) * i;
  float a[V], h[H];
  if constexpr (INTER) {
    load_in<DT, V>(p.in, int64_t(V) * i, a);
    if (KEEP) checkpoint<V>(a, int64_t(V) * i, p.codes, p.scales);
#pragma unroll
    for (int j = 0; j < H; ++j) h[j] = glu<CLAMPED>(a[2 * j], a[2 * j + 1]);
  } else {
    const int64_t off = int64_t(V) * i + int64_t(i / p.per) * p.I;
    float b[V];
    load_in<DT, V>(p.in, off, a);
    load_in<DT, V>(p.in, off + p.I, b);
    if (KEEP) {
      checkpoint<V>(a, off, p.codes, p.scales);
      checkpoint<V>(b, off + p.I, p.codes, p.scales);
    }
#pragma unroll
    for (int j = 0; j < H; ++j) h[j] = glu<CLAMPED>(a[j], b[j]);
  }
  store_short<H>(out, h);
}

// The same rows from their checkpoint, g float32, to bf16: 192 us (6.2 TB/s); 8191 rows of 2880 pairs 36 us (6.5 TB/s).
template <int DT, int GDT, int ODT, bool CLAMPED, bool INTER>
__global__ void __launch_bounds__(kThreads) glu_backward_kernel(GluArgs p) {
  constexpr int V = lane_elems<DT>, H = INTER ? V / 2 : V;
  const uint32_t i = blockIdx.x * uint32_t(kThreads) + threadIdx.x;
  if (i >= p.items) return;
  row_elem<ODT>* out = static_cast<row_elem<ODT>*>(p.out);
  float g[H];
  load_short<H>(static_cast<const row_elem<GDT>*>(p.g) + int64_t(H) * i, g);
  float a[V];
  if constexpr (INTER) {
    float d[V];
    load_in<DT, V>(p.in, int64_t(V) * i, a);
#pragma unroll
    for (int j = 0; j < H; ++j) glu_grad<CLAMPED>(g[j], a[2 * j], a[2 * j + 1], &d[2 * j], &d[2 * j + 1]);
    store_vec<V>(out + int64_t(V) * i, d);
  } else {
    const int64_t off = int64_t(V) * i + int64_t(i / p.per) * p.I;
    float b[V], da[V], db[V];
    load_in<DT, V>(p.in, off, a);
    load_in<DT, V>(p.in, off + p.I, b);
#pragma unroll
    for (int j = 0; j < V; ++j) glu_grad<CLAMPED>(g[j], a[j], b[j], &da[j], &db[j]);
    store_vec<V>(out + off, da);
    store_vec<V>(out + off + p.I, db);
  }
}

template <int DT, int ODT, bool CLAMPED, bool INTER>
void glu_keep(const GluArgs& a, unsigned grid, hipStream_t s) {
  if constexpr (DT != 2) {
    if (a.codes) {
      hipLaunchKernelGGL((glu_kernel<DT, ODT, CLAMPED, INTER, true>), dim3(grid), dim3(kThreads), 0, s, a);
      return;
    }
  }
  hipLaunchKernelGGL((glu_kernel<DT, ODT, CLAMPED, INTER, false>), dim3(grid), dim3(kThreads), 0, s, a);
}
template <int DT, int ODT, bool CLAMPED, bool INTER>
void glu_grad_of(const GluArgs& a, int g_dtype, unsigned grid, hipStream_t s) {
  if (g_dtype == 0) hipLaunchKernelGGL((glu_backward_kernel<DT, 0, ODT, CLAMPED, INTER>), dim3(grid), dim3(kThreads), 0, s, a);
  else hipLaunchKernelGGL((glu_backward_kernel<DT, 1, ODT, CLAMPED, INTER>), dim3(grid), dim3(kThreads), 0, s, a);
}
template <int DT, int ODT>
void glu_forms(const GluLaunch& L, const GluArgs& a, unsigned grid, hipStream_t s) {
  const auto go = [&](auto clamped, auto inter) {
    if (L.g) glu_grad_of<DT, ODT, clamped.value, inter.value>(a, L.g_dtype, grid, s);
    else glu_keep<DT, ODT, clamped.value, inter.value>(a, grid, s);
  };
  using T = std::true_type;
  using F = std::false_type;
  if (L.clamped) L.interleaved ? go(T{}, T{}) : go(T{}, F{});
  else L.interleaved ? go(F{}, T{}) : go(F{}, F{});
}
template <int DT>
void glu_out(const GluLaunch& L, const GluArgs& a, unsigned grid, hipStream_t s) {
  if (L.out_dtype == 0) glu_forms<DT, 0>(L, a, grid, s);
  else glu_forms<DT, 1>(L, a, grid, s);
}

int64_t blocks_of(int64_t items) { return (items + kThreads - 1) / kThreads; }
int elems_of(int dtype) { return dtype == 1 ? 4 : 8; }

}  // namespace

int64_t rows8_items(int64_t S, int64_t C, int dtype) { return blocks_of(S * C / elems_of(dtype)) * kThreads; }
int64_t glu_items(int64_t S, int64_t I, int rows_dtype, bool interleaved) {
  return blocks_of(S * I * (interleaved ? 2 : 1) / elems_of(rows_dtype)) * kThreads;
}

hipError_t launch_checkpoint(const void* x, int dtype, int64_t n, int8_t* codes, uint8_t* scales, hipStream_t stream) {
  if (n == 0) return hipSuccess;
  const KeepArgs a{{x, nullptr}, codes, scales, n / elems_of(dtype)};
  const dim3 grid(unsigned(blocks_of(a.items)));
  if (dtype == 0) hipLaunchKernelGGL((checkpoint_kernel<0>), grid, dim3(kThreads), 0, stream, a);
  else hipLaunchKernelGGL((checkpoint_kernel<1>), grid, dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_restore(const int8_t* codes, const uint8_t* scales, int64_t n, void* out, int out_dtype,
                          hipStream_t stream) {
  if (n == 0) return hipSuccess;
  const RestoreArgs a{{codes, scales}, out, n / 8};
  const dim3 grid(unsigned(blocks_of(a.items)));
  if (out_dtype == 0) hipLaunchKernelGGL((restore_kernel<0>), grid, dim3(kThreads), 0, stream, a);
  else hipLaunchKernelGGL((restore_kernel<1>), grid, dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_glu(const GluLaunch& L, hipStream_t stream) {
  const int64_t n = L.S * L.I * (L.interleaved ? 2 : 1) / elems_of(L.rows_dtype);
  if (n == 0) return hipSuccess;
  const GluArgs a{{L.rows, L.row_scales}, L.g, L.out, L.codes, L.scales, L.I, uint32_t(n),
                  uint32_t(L.I / elems_of(L.rows_dtype))};
  const unsigned grid = unsigned(blocks_of(n));
  if (L.rows_dtype == 0) glu_out<0>(L, a, grid, stream);
  else if (L.rows_dtype == 1) glu_out<1>(L, a, grid, stream);
  else glu_out<2>(L, a, grid, stream);
  return hipGetLastError();
}

}  // namespace e4b
