// Rows in MXFP4 (e2m1 codes, an e8m0 byte for each 32) and their grouped product with an MXFP4 stack:
//   quantise  rows p = x[slots[p] / k] (or x[p]): X = floor(log2 amax) - 2, code = e2m1(v 2^-X)
//   product   out[p, n] = bias[e, n] + sum_b 2^(xs[p, b] + ws[e, n, b] - 254) sum_j xq[p, b, j] wq[e, n, b, j]
// The block-scaled matrix instruction takes both operands' codes and bytes as they are: products of
// e2m1 values are exact, sums are float32.
#include "e4b_groups.h"
#include "e4b_internal.h"
#include "e4b_rows.h"

namespace e4b {

namespace {

constexpr int kThreads = 256;

struct QuantArgs {
  const void* x;
  const int32_t* slots;   // nullable
  uint8_t* blocks;
  uint8_t* scales;
  int64_t K, rows;        // rows: T * k
  uint32_t items, per;    // of 8 elements each: of the call, of a row
  int k;
};

// Eight elements a lane, four lanes a block.  Bound: memory.
template <int DT>
__global__ void __launch_bounds__(kThreads) quantize_kernel(QuantArgs p) {
  const uint32_t i = blockIdx.x * uint32_t(kThreads) + threadIdx.x;
  if (i >= p.items) return;
  const uint32_t row = i / p.per;
  int64_t src = row;
  bool none = false;
  if (p.slots) {
    const int32_t s = p.slots[row];
    none = s < 0 || s >= p.rows;
    src = none ? 0 : s / p.k;
  }
  float v[8];
  load_vec<8>(static_cast<const row_elem<DT>*>(p.x) + src * p.K + 8 * int64_t(i - row * p.per), v);
  uint32_t amax = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (none) v[j] = 0.f;
    amax = max(amax, __float_as_uint(v[j]) & 0x7FFFFFFFu);
  }
  amax = max(amax, uint32_t(__builtin_amdgcn_update_dpp(0, int(amax), 0xB1, 0xf, 0xf, false)));
  amax = max(amax, uint32_t(__builtin_amdgcn_update_dpp(0, int(amax), 0x4E, 0xf, 0xf, false)));
  const uint32_t e = amax >> 23;                       // floor(log2) + 127, 0 for subnormals and zero
  const uint32_t byte = e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
  uint32_t word = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float m = __builtin_amdgcn_ldexpf(fabsf(v[j]), 127 - int(byte));
    const uint32_t code = uint32_t(m > 0.25f) + (m >= 0.75f) + (m > 1.25f) + (m >= 1.75f) + (m > 2.5f) + (m >= 3.5f) + (m > 5.f);
    word |= (code | (__float_as_uint(v[j]) >> 28 & 8u)) << (4 * j);
  }
  reinterpret_cast<uint32_t*>(p.blocks)[i] = word;
  if ((i & 3) == 0) p.scales[i >> 2] = uint8_t(byte);
}

struct GemmArgs {
  const uint8_t* x;       // [S, K/32, 16]
  const uint8_t* xs;      // [S, K/32]
  const uint8_t* w;       // [E, N, K/32, 16]
  const uint8_t* ws;      // [E, N, K/32]
  const float* bias;      // nullable [E, N]
  const int32_t* offsets;
  void* out;              // [S, N]
  int64_t N, K;
  int S, E;
  uint32_t col_tiles;
};

typedef int v8i __attribute__((ext_vector_type(8)));
__device__ __forceinline__ v8i operand4(u32x4 a) { return v8i{int(a[0]), int(a[1]), int(a[2]), int(a[3]), 0, 0, 0, 0}; }

// A wave has 32 rows of an expert by 32 columns.  Operands of the 32x32x64 instruction: lane l holds block
// l / 32 of row or column l % 32 and its byte.
template <int ODT>
__global__ void __launch_bounds__(kThreads) gemm_kernel(GemmArgs p) {
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x >> 6;
  const int c = lane & 31, half = lane >> 5;
  const uint32_t tile = blockIdx.x / p.col_tiles;
  const RowTile t = find_tile(p.offsets, nullptr, p.E, p.E, p.S, 5, tile);
  if (t.rows == 0) return;
  const int64_t col = int64_t(blockIdx.x - tile * p.col_tiles) * 128 + 32 * wave + c;
  const int64_t n = col < p.N ? col : p.N - 1, blocks = p.K / 32;
  const int64_t xrow = t.row0 + (c < t.rows ? c : t.rows - 1), wrow = int64_t(t.adapter) * p.N + n;
  const uint8_t *xq = p.x + xrow * blocks * 16, *wq = p.w + wrow * blocks * 16;
  const uint8_t *xs = p.xs + xrow * blocks, *ws = p.ws + wrow * blocks;
  f32x16 acc = {};
  for (int64_t b = 0; b < blocks; b += 2) {
    const bool in = b + half < blocks;  // a block past the last: its bytes 0 on both sides, 2^-254 times something finite
    const int64_t at = in ? b + half : b;
    const u32x4 xa = *reinterpret_cast<const u32x4*>(xq + 16 * at), wb = *reinterpret_cast<const u32x4*>(wq + 16 * at);
    const int sa = in ? xs[at] : 0, sb = in ? ws[at] : 0;
    acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand4(xa), operand4(wb), acc, 4, 4, 0, sa, 0, sb);
  }
  if (col >= p.N) return;
  const float bias = p.bias ? p.bias[int64_t(t.adapter) * p.N + col] : 0.f;
  row_elem<ODT>* out = static_cast<row_elem<ODT>*>(p.out) + t.row0 * p.N + col;
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int row = 8 * (r >> 2) + 4 * half + (r & 3);
    if (row < t.rows) store1(out + row * p.N, acc[r] + bias);
  }
}

int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t row_tiles(const MxGemmLaunch& L) {
  const int64_t used = L.E < L.S ? L.E : L.S;
  return (L.S + used * 31) >> 5;
}

}  // namespace

int64_t quantize_mxfp4_items(int64_t S, int64_t K) { return div_up(S * K / 8, kThreads) * kThreads; }
int64_t mxfp4_gemm_items(const MxGemmLaunch& L) { return row_tiles(L) * div_up(L.N, 128) * kThreads; }

hipError_t launch_quantize_mxfp4(const void* x, int dtype, int64_t T, int64_t K, int k, const int32_t* slots,
                                 uint8_t* blocks, uint8_t* scales, hipStream_t stream) {
  if (T == 0) return hipSuccess;
  const int64_t S = T * k;
  const QuantArgs a{x, slots, blocks, scales, K, S, uint32_t(S * K / 8), uint32_t(K / 8), k};
  const dim3 grid(unsigned(div_up(a.items, kThreads)));
  if (dtype == 0) hipLaunchKernelGGL((quantize_kernel<0>), grid, dim3(kThreads), 0, stream, a);
  else hipLaunchKernelGGL((quantize_kernel<1>), grid, dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_mxfp4_gemm(const MxGemmLaunch& L, hipStream_t stream) {
  if (L.S == 0) return hipSuccess;
  const GemmArgs a{L.x, L.xs, L.w, L.ws, L.bias, L.offsets, L.out, L.N, L.K, int(L.S), int(L.E), uint32_t(div_up(L.N, 128))};
  const dim3 grid(unsigned(row_tiles(L) * a.col_tiles));
  if (L.out_dtype == 0) hipLaunchKernelGGL((gemm_kernel<0>), grid, dim3(kThreads), 0, stream, a);
  else hipLaunchKernelGGL((gemm_kernel<1>), grid, dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace e4b
