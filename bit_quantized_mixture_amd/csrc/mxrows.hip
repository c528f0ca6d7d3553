// Rows in MXFP4 (e2m1 codes, an e8m0 byte for each 32) and their grouped product with an MXFP4 stack:
//   quantise  rows p = x[slots[p] / k] (or x[p]): X = floor(log2 amax) - 2, code = e2m1(v 2^-X)
//   product   out[p, n] = bias[e, n] + sum_b 2^(xs[p, b] + ws[e, n, b] - 254) sum_j xq[p, b, j] wq[e, n, b, j]
// The block-scaled matrix instruction takes both operands' codes and bytes as they are: products of
// e2m1 values are exact, sums are float32.
#include <type_traits>

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

// A wave's tile in a launch that cuts every expert's rows into pieces of 1 << bm_log2 and its columns into
// `cols`: the row tiles of an expert stand in bands of up to kBand, a band's column after column, so that
// neighbours share both operands.  The workgroups are dealt to the XCDs in contiguous stretches of that
// list (workgroup b runs on XCD b % 8), each with an L2 cache of its own.
struct GemmTile {
  int expert;
  int64_t row0;
  int rows;        // 0: no such tile
  uint32_t col;
};
constexpr int kBand = 4;

__device__ __forceinline__ GemmTile find_gemm_tile(const int32_t* __restrict__ offsets, int E, int S, int bm_log2,
                                                   uint32_t cols, uint32_t block) {
  const int lane = threadIdx.x & (kWave - 1), bm = 1 << bm_log2;
  const auto tiles_at = [&](int g0, int* lo, int* hi) {
    *lo = *hi = 0;
    if (g0 + lane < E) group_rows(offsets, g0 + lane, S, lo, hi);
    return int((int64_t(*hi) - *lo + bm - 1) >> bm_log2);
  };
  int lo, hi, n = tiles_at(0, &lo, &hi), ni = wave_scan(n);
  uint64_t all = uint32_t(__builtin_amdgcn_readlane(ni, kWave - 1));
  for (int g0 = kWave; g0 < E; g0 += kWave) {
    int l, h;
    all += uint32_t(__builtin_amdgcn_readlane(wave_scan(tiles_at(g0, &l, &h)), kWave - 1));
  }
  const uint64_t total = all * cols;
  if (block >= total) return GemmTile{0, 0, 0, 0};
  const uint32_t xcd = block & 7u, per = uint32_t(total >> 3), rest = uint32_t(total & 7u);
  const uint32_t at = xcd * per + (xcd < rest ? xcd : rest) + (block >> 3);
  const uint32_t row_tile = at / cols;
  uint32_t base = 0;
  for (int g0 = 0; g0 < E; g0 += kWave) {
    if (g0 > 0) {
      n = tiles_at(g0, &lo, &hi);
      ni = wave_scan(n);
    }
    const uint32_t sum = uint32_t(__builtin_amdgcn_readlane(ni, kWave - 1));
    if (row_tile - base < sum) {
      const int l = __ffsll((unsigned long long)__ballot(row_tile - base < uint32_t(ni))) - 1;
      const uint32_t m = uint32_t(__builtin_amdgcn_readlane(n, l));
      const uint32_t first = base + uint32_t(__builtin_amdgcn_readlane(ni, l)) - m;
      const uint32_t within = at - first * cols, band = within / (kBand * cols);
      if (m == 0 || band * kBand >= m) break;  // sums of offsets that descend can wrap
      const uint32_t rows_of_band = m - band * kBand < kBand ? m - band * kBand : kBand;
      const uint32_t in_band = within - band * kBand * cols, col = in_band / rows_of_band;
      if (col >= cols) break;
      const uint32_t t = band * kBand + (in_band - col * rows_of_band);
      const int row0 = __builtin_amdgcn_readlane(lo, l) + int(t << bm_log2), left = __builtin_amdgcn_readlane(hi, l) - row0;
      return GemmTile{g0 + l, row0, left < bm ? left : bm, col};
    }
    base += sum;
  }
  return GemmTile{0, 0, 0, 0};
}

__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t res, uint32_t voff, uint32_t soff, void* lds_wave_base) {
#if defined(__HIP_DEVICE_COMPILE__)
  typedef __attribute__((address_space(3))) void lds_void;
  __builtin_amdgcn_raw_ptr_buffer_load_lds(res, (lds_void*)lds_wave_base, 16, int(voff), int(soff), 0, 0);
#endif
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t uniform_rsrc(const void* base, uint32_t bytes) {
  const uint64_t b = reinterpret_cast<uint64_t>(base);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(uint32_t(b)), hi = __builtin_amdgcn_readfirstlane(uint32_t(b >> 32));
  return buffer_rsrc(reinterpret_cast<const void*>(uint64_t(lo) | (uint64_t(hi) << 32)),
                     __builtin_amdgcn_readfirstlane(bytes));
}

typedef u32x4 u32x4_byte __attribute__((aligned(1)));

// 16 exponent bytes of a row from block `first` on, zeros behind its last (nb in all).  A row of bytes starts
// anywhere; no byte outside it is read: the last ones come with those before them, and are moved down.
__device__ __forceinline__ u32x4 load_bytes16(const uint8_t* __restrict__ row, int first, int nb) {
  return *reinterpret_cast<const u32x4_byte*>(row + (first + 16 <= nb ? first : nb - 16));
}
__device__ __forceinline__ u32x4 bytes_from(u32x4 v, int first, int nb) {
  const int down = first + 16 <= nb ? 0 : first + 16 - nb;
  if (down & 8) v = u32x4{v[2], v[3], 0u, 0u};
  if (down & 4) v = u32x4{v[1], v[2], v[3], 0u};
  const uint32_t by = uint32_t(down & 3);
  return u32x4{__builtin_amdgcn_alignbyte(v[1], v[0], by), __builtin_amdgcn_alignbyte(v[2], v[1], by),
               __builtin_amdgcn_alignbyte(v[3], v[2], by), __builtin_amdgcn_alignbyte(0u, v[3], by)};
}
// The same for a row of fewer than 16.
__device__ __forceinline__ u32x4 load_few_bytes(const uint8_t* __restrict__ row, int nb) {
  u32x4 v = {};
#pragma unroll
  for (int j = 0; j < 15; ++j)
    if (j < nb) v[j >> 2] |= uint32_t(row[j]) << (8 * (j & 3));
  return v;
}

// The tile form.  A workgroup has BM rows of an expert by BN columns, its WR by WC waves RB by CB blocks of
// 32 by 32 each.  K goes in chunks of 8 blocks (128 bytes of a row), copied straight into LDS, one chunk
// ahead: a copy instruction has 8 whole rows' pieces, a row's 16-byte piece p at place p ^ ((row >> 1) & 7),
// so that the 16 rows of a read spread over all banks.  Step s of a chunk takes blocks 2 s and 2 s + 1, a
// lane half one each.  Exponent bytes come for 16 blocks at a time through registers, sorted so that a
// lane's four of a chunk are one word, whose byte s the instruction picks.  What stands behind the last
// block is another block of the row under bytes of 0: 2^-254 times something finite.  Fragments are read one step ahead
// of their products, over the chunk's barrier too.
template <int ODT, int RB, int CB, int WR, int WC>
__global__ void __launch_bounds__(WR * WC * kWave) tile_kernel(GemmArgs p) {
  constexpr int kT = WR * WC * kWave, kW = WR * WC;
  constexpr int BM = 32 * RB * WR, BN = 32 * CB * WC, kRows = BM + BN;
  constexpr int kBmLog2 = BM == 256 ? 8 : (BM == 128 ? 7 : (BM == 64 ? 6 : 5));
  constexpr int kUnits = kRows / 8 / kW;           // copies of a wave and chunk
  constexpr int kTurns = (kRows + kT - 1) / kT;    // rows of bytes a thread has (some past the last)
  constexpr int kStage = kRows * 128, kBytes = kTurns * kT * 16;
  static_assert((kRows / 8) % kW == 0 && BM % 16 == 0, "copies");
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * kStage + 2 * kBytes];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 31, half = lane >> 5;
  const GemmTile t = find_gemm_tile(p.offsets, p.E, p.S, kBmLog2, p.col_tiles, blockIdx.x);
  if (t.rows == 0) return;
  const int nb = int(p.K >> 5), chunks = (nb + 7) >> 3;
  const uint32_t rowb = uint32_t(nb) * 16u;
  const int64_t n0 = int64_t(t.col) * BN;
  const int cols = p.N - n0 < BN ? int(p.N - n0) : BN;
  const int64_t wrow0 = int64_t(t.expert) * p.N + n0;
  const __amdgpu_buffer_rsrc_t xres = uniform_rsrc(p.x + t.row0 * rowb, uint32_t(t.rows) * rowb);
  const __amdgpu_buffer_rsrc_t wres = uniform_rsrc(p.w + wrow0 * rowb, uint32_t(cols) * rowb);

  // copies: unit u has rows 8 u .. of x (then of w), lane l place l % 8 of row l / 8
  uint32_t src[kUnits];
  const auto piece_of = [&](int unit) { return (lane & 7) ^ ((4 * unit + (lane >> 4)) & 7); };
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int unit = wave * kUnits + i, r = 8 * unit + (lane >> 3);
    const int last = (r < BM ? t.rows : cols) - 1, own = r < BM ? r : r - BM;
    src[i] = uint32_t(own < last ? own : last) * rowb + 16u * piece_of(unit);
  }
  // A copy of a chunk that does not exist reads one place again, into a stage that nothing reads.
  const auto copy_unit = [&](int chunk, int i) {
    const int left = nb - 8 * chunk;  // blocks of the row from here on
    const int unit = wave * kUnits + i, past = left < 8 ? piece_of(unit) - (left - 1) : 0;
    const uint32_t at = left > 0 ? src[i] - (past > 0 ? 16u * past : 0u) : 0u;
    dma16(8 * unit < BM ? xres : wres, at, left > 0 ? 128u * chunk : 0u, lds + (chunk & 1) * kStage + 1024 * unit);
  };
  const uint8_t* srow[kTurns];
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    const int r = tid + i * kT, last = (r < BM ? t.rows : cols) - 1, own = r < BM ? r : r - BM;
    srow[i] = (r < BM ? p.xs + t.row0 * nb : p.ws + wrow0 * nb) + int64_t(own < last ? own : last) * nb;
  }
  u32x4 sreg[kTurns];
  const auto load_scales = [&](int window) {  // past the last window: the last again, unused
    const int first = 16 * window < nb ? 16 * window : (nb - 1) & ~15;
#pragma unroll
    for (int i = 0; i < kTurns; ++i) sreg[i] = load_bytes16(srow[i], first, nb);
  };
  const auto put = [&](int window, int i, u32x4 v) {
    *reinterpret_cast<u32x4*>(lds + 2 * kStage + (window & 1) * kBytes + 16 * (tid + i * kT)) =
        u32x4{perm(v[1], v[0], 0x06040200u), perm(v[1], v[0], 0x07050301u), perm(v[3], v[2], 0x06040200u),
              perm(v[3], v[2], 0x07050301u)};
  };
  const auto put_scales = [&](int window) {
#pragma unroll
    for (int i = 0; i < kTurns; ++i) put(window, i, bytes_from(sreg[i], 16 * window, nb));
  };

  const int row_a = 32 * RB * (wave / WC), row_b = BM + 32 * CB * (wave % WC);
  struct Frags {
    u32x4 a[RB], b[CB];
  };
  struct Bytes {
    uint32_t a[RB], b[CB];
  };
  const auto frag = [&](const uint8_t* stage, int row, int s) {
    return *reinterpret_cast<const u32x4*>(stage + 128 * row + 16 * ((2 * s + half) ^ ((row >> 1) & 7)));
  };
  // Part i of RB of a step's fragments, and of a chunk's bytes.
  const auto read = [&](int chunk, int s, Frags& f, int i) {
    const uint8_t* stage = lds + (chunk & 1) * kStage;
    f.a[i] = frag(stage, row_a + 32 * i + c, s);
#pragma unroll
    for (int j = i * CB / RB; j < (i + 1) * CB / RB; ++j) f.b[j] = frag(stage, row_b + 32 * j + c, s);
  };
  const auto read_bytes = [&](int chunk, Bytes& f, int i) {
    const uint8_t* from = lds + 2 * kStage + ((chunk >> 1) & 1) * kBytes + 8 * (chunk & 1) + 4 * half;
    f.a[i] = *reinterpret_cast<const uint32_t*>(from + 16 * (row_a + 32 * i + c));
#pragma unroll
    for (int j = i * CB / RB; j < (i + 1) * CB / RB; ++j)
      f.b[j] = *reinterpret_cast<const uint32_t*>(from + 16 * (row_b + 32 * j + c));
  };
  f32x16 acc[RB][CB] = {};
  // The products of a step; `beside(i)` issues reads and copies before row i's, to run under them.
  const auto multiply = [&](auto step, const Frags& f, const Bytes& by, auto&& beside) {
    constexpr int s = decltype(step)::value;
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      beside(i);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < CB; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand4(f.a[i]), operand4(f.b[j]), acc[i][j], 4, 4, s,
                                                                    int(by.a[i]), s, int(by.b[j]));
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  using S0 = std::integral_constant<int, 0>;
  using S1 = std::integral_constant<int, 1>;
  using S2 = std::integral_constant<int, 2>;
  using S3 = std::integral_constant<int, 3>;
  constexpr int kPer = (kUnits + 2 * RB - 1) / (2 * RB);  // copies beside a row, over two steps
  const auto copies = [&](int chunk, int part) {
#pragma unroll
    for (int u = part * kPer; u < (part + 1) * kPer; ++u)
      if (u < kUnits) copy_unit(chunk, u);
  };
  const auto sync = [&] {  // a chunk has landed, and everyone is done with the stage of the one before
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(0));
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  };
  const auto nothing = [](int) {};

#pragma unroll
  for (int u = 0; u < kUnits; ++u) copy_unit(0, u);
  if (nb >= 16) {
    load_scales(0);
    put_scales(0);
    load_scales(1);
  } else {
#pragma unroll
    for (int i = 0; i < kTurns; ++i) put(0, i, load_few_bytes(srow[i], nb));
  }
  Frags f0, f1;
  Bytes even, odd;
  sync();
#pragma unroll
  for (int i = 0; i < RB; ++i) {
    read(0, 0, f0, i);
    read_bytes(0, even, i);
    if (chunks > 1) copies(1, i);
  }
  // A chunk that is not the last, up to its last step, under which the next one's first fragments are read.  No
  // branch inside: the compiler moves products over one.
  const auto body = [&](auto is_odd, auto copy_on, int k, const Bytes& by, Bytes& next) {
    multiply(S0{}, f0, by, [&](int i) {
      read(k, 1, f1, i);
      copies(k + 1, RB + i);
    });
    multiply(S1{}, f1, by, [&](int i) { read(k, 2, f0, i); });
    multiply(S2{}, f0, by, [&](int i) {
      read(k, 3, f1, i);
      if (decltype(is_odd)::value && i == 0) put_scales((k + 1) >> 1);
    });
    sync();
    multiply(S3{}, f1, by, [&](int i) {
      read(k + 1, 0, f0, i);
      read_bytes(k + 1, next, i);
      if (decltype(copy_on)::value) copies(k + 2, i);
      if (decltype(is_odd)::value && i == 0) load_scales((k + 3) >> 1);  // two chunks until it is put
    });
  };
  using Yes = std::true_type;
  using No = std::false_type;
  int k = 0;
  for (; k + 2 < chunks; k += 2) {
    body(No{}, Yes{}, k, even, odd);
    body(Yes{}, Yes{}, k + 1, odd, even);
  }
  if (k + 1 < chunks) {
    body(No{}, No{}, k, even, odd);
    even = odd;
    ++k;
  }
  const int steps = (nb - 8 * k + 1) >> 1;  // of the last chunk
  multiply(S0{}, f0, even, [&](int i) { read(k, 1, f1, i); });
  if (steps > 1) multiply(S1{}, f1, even, [&](int i) { read(k, 2, f0, i); });
  if (steps > 2) multiply(S2{}, f0, even, [&](int i) { read(k, 3, f1, i); });
  if (steps > 3) multiply(S3{}, f1, even, nothing);
  __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(0));  // no copy is left when the LDS is given back

  // out: element r of a block is row 8 (r / 4) + 4 half + r % 4, column c
  typedef row_elem<ODT> out_t;
  constexpr int kSize = sizeof(out_t);
#pragma unroll
  for (int i = 0; i < RB; ++i) {
    const int first = row_a + 32 * i, rows = t.rows - first < 32 ? t.rows - first : 32;
    if (rows <= 0) break;
    const uint32_t pitch = uint32_t(p.N) * kSize;
    const __amdgpu_buffer_rsrc_t ores =
        uniform_rsrc(static_cast<out_t*>(p.out) + (t.row0 + first) * p.N + n0, uint32_t(rows - 1) * pitch + uint32_t(cols) * kSize);
#pragma unroll
    for (int j = 0; j < CB; ++j) {
      const int col = row_b - BM + 32 * j + c;
      const bool in = col < cols;
      const float bias = p.bias && in ? p.bias[wrow0 + col] : 0.f;
      const uint32_t off = in ? uint32_t(4 * half) * pitch + uint32_t(col) * kSize : 0x80000000u;
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const uint32_t row = (8 * (r >> 2) + (r & 3)) * pitch;
        const float v = acc[i][j][r] + bias;
        if constexpr (ODT == 0) __builtin_amdgcn_raw_buffer_store_b16(bf16_rne(v), ores, off + row, 0, 0);
        else __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), ores, off + row, 0, 0);
      }
    }
  }
}

int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Rows and columns of a tile, by the mean number of an expert's rows.
struct TileForm {
  int bm, bn, threads;
};
TileForm tile_form(const MxGemmLaunch& L) {
  const int64_t mean = L.S / L.E;
  if (mean >= 192) return {256, 256, 256};
  if (mean >= 96) return {128, 128, 256};
  if (mean >= 48) return {64, 128, 256};
  return {32, 128, 256};
}
int64_t row_tiles(const MxGemmLaunch& L, int bm) {
  const int64_t used = L.E < L.S ? L.E : L.S;
  return (L.S + used * (bm - 1)) / bm;
}
int64_t gemm_blocks(const MxGemmLaunch& L) {
  const TileForm f = tile_form(L);
  return row_tiles(L, f.bm) * div_up(L.N, f.bn);
}
template <int RB, int CB, int WR, int WC>
void tile(const MxGemmLaunch& L, const GemmArgs& a, unsigned grid, hipStream_t s) {
  if (L.out_dtype == 0) hipLaunchKernelGGL((tile_kernel<0, RB, CB, WR, WC>), dim3(grid), dim3(WR * WC * kWave), 0, s, a);
  else hipLaunchKernelGGL((tile_kernel<1, RB, CB, WR, WC>), dim3(grid), dim3(WR * WC * kWave), 0, s, a);
}

}  // namespace

int64_t quantize_mxfp4_items(int64_t S, int64_t K) { return div_up(S * K / 8, kThreads) * kThreads; }
int64_t mxfp4_gemm_items(const MxGemmLaunch& L) { return gemm_blocks(L) * tile_form(L).threads; }

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
  const TileForm f = tile_form(L);
  const GemmArgs a{L.x, L.xs, L.w, L.ws, L.bias, L.offsets, L.out, L.N, L.K, int(L.S), int(L.E), uint32_t(div_up(L.N, f.bn))};
  const unsigned grid = unsigned(gemm_blocks(L));
  if (f.bm == 256) tile<4, 4, 2, 2>(L, a, grid, stream);
  else if (f.bm == 128) tile<2, 2, 2, 2>(L, a, grid, stream);
  else if (f.bm == 64) tile<2, 1, 1, 4>(L, a, grid, stream);
  else tile<1, 1, 1, 4>(L, a, grid, stream);
  return hipGetLastError();
}

}  // namespace e4b
