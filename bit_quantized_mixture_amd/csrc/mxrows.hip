// Rows in MXFP4 (e2m1 codes, an e8m0 byte for each 32) and their grouped product with an MXFP4 stack:
//   quantise  rows p = x[slots[p] / k] (or x[p]): X = floor(log2 amax) - 2, code = e2m1(v 2^-X)
//   product   out[p, n] = bias[e, n] + sum_b 2^(xs[p, b] + ws[e, n, b] - 254) sum_j xq[p, b, j] wq[e, n, b, j]
// The block-scaled matrix instruction takes both operands' codes and bytes as they are: products of
// e2m1 values are exact, sums are float32.
#include <type_traits>

#include "e4b_groups.h"
#include "e4b_internal.h"
#include "e4b_mx_forms.h"
#include "e4b_rows.h"

namespace e4b {

namespace {

constexpr int kThreads = 256;

struct QuantArgs {
  const void* x;
  const int32_t* slots;   // nullable
  uint8_t* blocks;
  uint8_t* scales;
  int64_t K;
  uint32_t rows;          // T * k
  uint32_t per, pieces;   // of a row: elements by eights, pieces of 64 * kQuantTurns of those
  uint32_t together;      // rows of a wave, where they are shorter than a piece
  uint32_t waves;
  int k;
};
constexpr int kQuantTurns = 4;

// Eight values divided by 2^(byte - 127) as e2m1 codes, the first in the low nibble: the conversion
// instruction rounds to nearest even and saturates at 6, as the format has it (checked for every bf16 value).
__device__ __forceinline__ uint32_t e2m1_of8(const float (&v)[8], uint32_t byte) {
  uint32_t word = 0;
#if defined(__HIP_DEVICE_COMPILE__)
  const float scale = e8m0_to_f32(byte);
  word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, v[0], v[1], scale, 0);
  word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, v[2], v[3], scale, 1);
  word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, v[4], v[5], scale, 2);
  word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, v[6], v[7], scale, 3);
#endif
  return word;
}

// A wave has a piece of one row, or (SHORT) several rows, a lane eight elements a turn, four lanes a block.
// Bound: memory; 8192 rows of 2880 gathered from 2048 tokens 11 us, 8192 of 14336 as they are 43 us (7 TB/s).
template <int DT, bool SHORT>
__global__ void __launch_bounds__(kThreads) quantize_kernel(QuantArgs p) {
  const int lane = threadIdx.x & (kWave - 1);
  const uint32_t task = blockIdx.x * uint32_t(kThreads / kWave) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (task >= p.waves) return;
  const uint32_t group = task / p.pieces, first = (task - group * p.pieces) * (kWave * kQuantTurns);
  uint32_t row[kQuantTurns], at[kQuantTurns];
  float v[kQuantTurns][8];
  bool none[kQuantTurns];
#pragma unroll
  for (int j = 0; j < kQuantTurns; ++j) {
    at[j] = first + kWave * j + lane;
    row[j] = group * p.together;
    if (SHORT) {
      const uint32_t r = at[j] / p.per;
      at[j] = r < p.together ? at[j] - r * p.per : p.per;
      row[j] += r;
      if (row[j] >= p.rows) at[j] = p.per;
    }
    none[j] = false;
    if (at[j] < p.per) {
      int64_t src = row[j];
      if (p.slots) {
        const int32_t s = p.slots[row[j]];
        none[j] = s < 0 || uint32_t(s) >= p.rows;
        src = none[j] ? 0 : s / p.k;
      }
      load_vec<8>(static_cast<const row_elem<DT>*>(p.x) + src * p.K + 8 * int64_t(at[j]), v[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < kQuantTurns; ++j) {
    if (at[j] >= p.per) return;  // a block's lanes all go or all stay, and none has a later turn
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (none[j]) v[j][i] = 0.f;
      amax = max(amax, __float_as_uint(v[j][i]) & 0x7FFFFFFFu);
    }
    amax = max(amax, uint32_t(__builtin_amdgcn_update_dpp(0, int(amax), 0xB1, 0xf, 0xf, false)));
    amax = max(amax, uint32_t(__builtin_amdgcn_update_dpp(0, int(amax), 0x4E, 0xf, 0xf, false)));
    const uint32_t e = amax >> 23;                       // floor(log2) + 127, 0 for subnormals and zero
    const uint32_t byte = e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
    const int64_t out = int64_t(row[j]) * p.per + at[j];
    __builtin_nontemporal_store(e2m1_of8(v[j], byte), reinterpret_cast<uint32_t*>(p.blocks) + out);
    if ((at[j] & 3) == 0) p.scales[out >> 2] = uint8_t(byte);
  }
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
  bool two_lists;
};

typedef int v8i __attribute__((ext_vector_type(8)));
__device__ __forceinline__ v8i operand4(u32x4 a) { return v8i{int(a[0]), int(a[1]), int(a[2]), int(a[3]), 0, 0, 0, 0}; }

// The tiles of a launch: every expert's rows cut into pieces of 1 << bm_log2 and its columns into `cols`.  The
// row tiles of an expert stand in bands of up to kBand, a band's column after column, so that neighbours
// share both operands.  In the larger forms, where a launch is few rounds of tiles, last pieces of half the rows
// and fewer are a list of their own behind all others, so that it ends with short tiles (8192 rows of 32 experts at
// [5760, 2880], at most 6 tiles a CU, 165 us in one list, 148 so; 4096 of 8 at [4096, 14336], 2, 185 and 155; 16384
// of 32, 8, 249 and 241; but 8192 of 8 at [28672, 4096], 17, 558 and 563: their columns are fetched twice; where the
// limit lies is measured at mx_two_lists).  The
// XCDs, each with an L2 cache of its own, have contiguous stretches of either list, and the workgroups of an XCD
// (workgroup b runs on XCD b % 8) take its stretches in turn.
struct GemmTile {
  int expert;
  int64_t row0;
  int rows;        // 0: no such tile
  uint32_t col;
};
constexpr int kBand = 8;

__device__ __forceinline__ GemmTile find_gemm_tile(const int32_t* __restrict__ offsets, int E, int S, int bm_log2,
                                                   uint32_t cols, bool two_lists, uint32_t block) {
  const int lane = threadIdx.x & (kWave - 1), bm = 1 << bm_log2;
  // Tiles of an expert's rows, and whether a short one follows.
  const auto tiles_at = [&](int g0, int* lo, int* hi, int* rest) {
    *lo = *hi = 0;
    if (g0 + lane < E) group_rows(offsets, g0 + lane, S, lo, hi);
    const int n = *hi - *lo, left = n & (bm - 1);
    *rest = two_lists && left > 0 && left <= bm / 2;
    return (n >> bm_log2) + (left > (two_lists ? bm / 2 : 0));
  };
  int lo, hi, rest, n = tiles_at(0, &lo, &hi, &rest), ni = wave_scan(n), ri = two_lists ? wave_scan(rest) : 0;
  uint64_t whole = uint32_t(__builtin_amdgcn_readlane(ni, kWave - 1)), shorts = uint32_t(__builtin_amdgcn_readlane(ri, kWave - 1));
  for (int g0 = kWave; g0 < E; g0 += kWave) {
    int l, h, r;
    whole += uint32_t(__builtin_amdgcn_readlane(wave_scan(tiles_at(g0, &l, &h, &r)), kWave - 1));
    if (two_lists) shorts += uint32_t(__builtin_amdgcn_readlane(wave_scan(r), kWave - 1));
  }
  const uint32_t xcd = block & 7u;
  uint32_t id = block >> 3;
  // an XCD's stretch of a list of `all`
  const auto take = [&](uint64_t all) {
    const uint32_t per = uint32_t(all >> 3), over = uint32_t(all & 7u), mine = per + (xcd < over);
    if (id >= mine) {
      id -= mine;
      return false;
    }
    id += xcd * per + (xcd < over ? xcd : over);
    return true;
  };
  bool is_short = false;
  if (!take(whole * cols)) {
    if (!take(shorts * cols)) return GemmTile{0, 0, 0, 0};
    is_short = true;
  }
  const uint32_t row_tile = id / cols;
  uint32_t base = 0;
  for (int g0 = 0; g0 < E; g0 += kWave) {
    if (g0 > 0) {
      n = tiles_at(g0, &lo, &hi, &rest);
      ni = wave_scan(n);
      if (two_lists) ri = wave_scan(rest);
    }
    const int count = is_short ? rest : n, ci = is_short ? ri : ni;
    const uint32_t sum = uint32_t(__builtin_amdgcn_readlane(ci, kWave - 1));
    if (row_tile - base < sum) {
      const int k = __ffsll((unsigned long long)__ballot(row_tile - base < uint32_t(ci))) - 1;
      const uint32_t m = uint32_t(__builtin_amdgcn_readlane(count, k));
      const uint32_t first = base + uint32_t(__builtin_amdgcn_readlane(ci, k)) - m;
      const uint32_t within = id - first * cols, band = within / (kBand * cols);
      if (m == 0 || band * kBand >= m) break;  // sums of offsets that descend can wrap
      const uint32_t high = m - band * kBand < kBand ? m - band * kBand : kBand;
      const uint32_t in_band = within - band * kBand * cols, col = in_band / high;
      if (col >= cols) break;
      const uint32_t t = band * kBand + (in_band - col * high) + (is_short ? uint32_t(__builtin_amdgcn_readlane(n, k)) : 0u);
      const int row0 = __builtin_amdgcn_readlane(lo, k) + int(t << bm_log2), left = __builtin_amdgcn_readlane(hi, k) - row0;
      return GemmTile{g0 + k, row0, left < bm ? left : bm, col};
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
__device__ __forceinline__ u32x4 load_bytes16(const uint8_t* __restrict__ rows, uint32_t row, int first, int nb) {
  return *reinterpret_cast<const u32x4_byte*>(rows + (row + uint32_t(first + 16 <= nb ? first : nb - 16)));
}
__device__ __forceinline__ u32x4 bytes_from(u32x4 v, int first, int nb) {
  const int down = first + 16 <= nb ? 0 : first + 16 - nb;
  if (down & 8) v = u32x4{v[2], v[3], 0u, 0u};
  if (down & 4) v = u32x4{v[1], v[2], v[3], 0u};
  const uint32_t by = uint32_t(down & 3);
  v = u32x4{__builtin_amdgcn_alignbyte(v[1], v[0], by), __builtin_amdgcn_alignbyte(v[2], v[1], by),
            __builtin_amdgcn_alignbyte(v[3], v[2], by), __builtin_amdgcn_alignbyte(0u, v[3], by)};
  return down < 16 ? v : u32x4{0u, 0u, 0u, 0u};
}
// The same for a row of fewer than 16.
__device__ __forceinline__ u32x4 load_few_bytes(const uint8_t* __restrict__ row, int nb) {
  u32x4 v = {};
#pragma unroll
  for (int j = 0; j < 15; ++j)
    if (j < nb) v[j >> 2] |= uint32_t(row[j]) << (8 * (j & 3));
  return v;
}

// Rows are stored past the caches (the instruction's non-temporal bit), which keeps the L2 caches for the
// operands: 2048 tokens of the 32-expert layer's gate_up rows 169 us kept, 153 so; 8168 rows of 64 experts at
// [4096, 1536] 74 and 62.
constexpr int kPastCaches = 2;

// Keeps the products of a row of blocks where they are written: without it the compiler gathers a loop's
// products behind all its reads.  There is no instruction in it, so nothing reads the sums here.
template <int N>
__device__ __forceinline__ void hold(f32x16 (&v)[N]) {
#if defined(__HIP_DEVICE_COMPILE__)
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+a"(v[i]));
#endif
}

// The tile form.  A workgroup has up to 32 RB WR rows of an expert by 32 CB WC columns; its WR by WC waves have
// every WR-th block of 32 rows and 32 CB columns each.  A tile of fewer rows runs the form for as many blocks as
// it has: what is left of an expert's rows behind whole tiles costs little more than its columns' bytes.
// K goes in chunks of 8 blocks (128 bytes of a row), copied straight into a ring of stages in LDS: a copy
// instruction has 8 whole rows' pieces, and a row's 16-byte piece p is at place p ^ ((row >> 1) & 7), so that the
// 16 rows of a read spread over all banks.  Step s of a chunk takes blocks 2 s and 2 s + 1, a lane half one
// each.  Exponent bytes come through registers for a window of 16 blocks at a time, sorted so that a lane's eight
// of a window are two words, whose bytes the instruction picks.  Fragments are read a step ahead of their
// products, over the chunk's barrier too.
// Bound: for few rows memory (512 rows of 128 experts at [1536, 2048] 35 us, 6.1 TB/s); for whole tiles the L2
// caches' requests (a workgroup reads 64 KB for 256 matrix instructions) and the clock under the matrix unit's
// power, and at K = 2880 the start and end of a tile, 15000 of 60000 cycles (8192 rows of 8 experts at [28672, 4096] 540 us,
// 3.6 PFLOP/s; of 32 at [5760, 2880] 148 us, 1.8; of one at [8192, 8192] 254 us, 4.3; the unit alone, from registers, 6.3
// on random codes).  Two stages of 128-byte rows fill the LDS at 256 x 256; chunks of
// half that with four stages, and 128 x 256 with two workgroups a CU, were slower (762 us against 660 of that
// state), so was a grid of one workgroup a CU that went through its tiles (660 against 552).
template <int ODT, int RB, int CB, int WR, int WC, int RING>
__global__ void __launch_bounds__(WR * WC * kWave, 2) tile_kernel(GemmArgs p) {
  constexpr int kW = WR * WC, kT = kW * kWave, CH = 8;
  constexpr int BM = 32 * RB * WR, BN = 32 * CB * WC, kRowBytes = 16 * CH, kEvery = 8 * kW;
  constexpr int kBmLog2 = BM == 256 ? 8 : (BM == 128 ? 7 : 6);
  constexpr int kRing = RING * (BM + BN) * kRowBytes;
  constexpr int kTurnRows = kT / 2, kTurns = (BM + BN + kTurnRows - 1) / kTurnRows;  // rows of bytes, two lanes each
  constexpr int kHalf = kTurns * kTurnRows * 16;   // a window's bytes in LDS
  static_assert(BM % kEvery == 0 && BN % kEvery == 0 && kEvery % 32 == 0, "copies");
  __shared__ __attribute__((aligned(16))) uint8_t lds[kRing + 2 * kHalf];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 31, half = lane >> 5;
  const GemmTile t = find_gemm_tile(p.offsets, p.E, p.S, kBmLog2, p.col_tiles, BM >= 128 && p.two_lists, blockIdx.x);
  if (t.rows == 0) return;
  const int nb = int(p.K >> 5), windows = (nb + 15) >> 4;
  const uint32_t rowb = uint32_t(nb) * 16u;
  const int64_t n0 = int64_t(t.col) * BN;
  const int cols = p.N - n0 < BN ? int(p.N - n0) : BN;
  const int64_t wrow0 = int64_t(t.expert) * p.N + n0;
  const __amdgpu_buffer_rsrc_t xres = uniform_rsrc(p.x + t.row0 * rowb, uint32_t(t.rows) * rowb);
  const __amdgpu_buffer_rsrc_t wres = uniform_rsrc(p.w + wrow0 * rowb, uint32_t(cols) * rowb);

  // copies: unit u has LDS rows 8 u .. (w's, then x's), lane l place l % 8 of row l / 8; a wave takes every kW-th
  // unit, so that a lane's units are whole numbers of rows apart.  A wave's 32 CB columns are dealt out to its
  // blocks in turn, so that a lane ends with CB neighbouring columns.
  const auto col_of = [](int r) { return (r & ~(32 * CB - 1)) + CB * (r & 31) + ((r >> 5) & (CB - 1)); };
  const int own_row = 8 * wave + (lane >> 3);
  const uint32_t own = 16u * ((lane & 7) ^ ((own_row >> 1) & 7));
  const uint32_t x_own = uint32_t(own_row) * rowb + own, w_own = uint32_t(col_of(own_row)) * rowb + own;
  constexpr int kUnitsW = BN / kEvery;
  // Copy i of a chunk into the stage at `stage`.  The buffers end with the tile's rows: nothing is fetched for what
  // stands behind them, nor for a chunk that does not exist (a row's blocks behind its last are the next
  // row's, under bytes of 0: 2^-254 times something finite).
  const auto copy_unit = [&](int chunk, int stage, int i) {
    const uint32_t from = chunk * CH < nb ? uint32_t(kRowBytes * chunk) : 0x80000000u;
    const uint32_t rows = i < kUnitsW ? col_of(i * kEvery) : (i - kUnitsW) * kEvery;
    dma16(i < kUnitsW ? wres : xres, (i < kUnitsW ? w_own : x_own) + (from + rows * rowb), 0u,
          lds + stage + 1024 * (i * kW + wave));
  };
  // Exponent bytes come for two windows at a time, a lane for each row and window.
  const uint8_t* sbase[kTurns];  // the same for a wave: its rows are all of w or all of x
  uint32_t soff[kTurns];
  u32x4 sreg[kTurns];
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    const int r = (tid >> 1) + i * kTurnRows < BM + BN ? (tid >> 1) + i * kTurnRows : 0;
    const bool of_w = __builtin_amdgcn_readfirstlane(r) < BN;
    const int last = (of_w ? cols : t.rows) - 1, row = of_w ? col_of(r) : r - BN;
    sbase[i] = of_w ? p.ws + wrow0 * nb : p.xs + t.row0 * nb;
    soff[i] = uint32_t(row < last ? row : last) * uint32_t(nb);
  }
  const auto load_scales = [&](int pair) {  // past the last window: the last again, unused
    const int first = 32 * pair + 16 * (tid & 1);
#pragma unroll
    for (int i = 0; i < kTurns; ++i) sreg[i] = load_bytes16(sbase[i], soff[i], first, nb);
  };
  const auto put = [&](int i, u32x4 v) {  // even blocks' bytes, then odd blocks'
    *reinterpret_cast<u32x4*>(lds + kRing + kHalf * (tid & 1) + 16 * ((tid >> 1) + i * kTurnRows)) =
        u32x4{perm(v[1], v[0], 0x06040200u), perm(v[3], v[2], 0x06040200u), perm(v[1], v[0], 0x07050301u),
              perm(v[3], v[2], 0x07050301u)};
  };
  const auto put_scales = [&](int pair) {
#pragma unroll
    for (int i = 0; i < kTurns; ++i) put(i, bytes_from(sreg[i], 32 * pair + 16 * (tid & 1), nb));
  };

  const int wave_row = wave / WC, wave_col = wave % WC;
  // (2 s + half) ^ swap = (half ^ swap) ^ 2 s, and a row's place is a multiple of 128.
  const uint32_t place = kRowBytes * c + 16u * (half ^ ((c >> 1) & 7));
  const uint32_t b_place = place + 32 * CB * kRowBytes * wave_col, a_place = place + (BN + 32 * wave_row) * kRowBytes;

  // The sums of R blocks for each wave, and their way out.
  const auto run = [&](auto blocks_of) {
    constexpr int R = decltype(blocks_of)::value;
    constexpr int kStage = (BN + 32 * WR * R) * kRowBytes, ST = kRing / kStage, kUnits = kUnitsW + 32 * WR * R / kEvery;
    struct Frags {
      u32x4 a[R], b[CB];
    };
    f32x16 acc[R][CB];
    Frags f0, f1;
    uint32_t bytes_a[2][R], bytes_b[2][CB];
    // Part i of R of a step's fragments, and of half a window's bytes.  Rows 32 apart have their pieces alike.
    const auto read = [&](int stage, int s, Frags& f, int i) {
      const uint8_t* from = lds + stage;
      f.a[i] = *reinterpret_cast<const u32x4*>(from + (a_place ^ (32u * s)) + 32 * WR * kRowBytes * i);
#pragma unroll
      for (int j = i * CB / R; j < (i + 1) * CB / R; ++j)
        f.b[j] = *reinterpret_cast<const u32x4*>(from + (b_place ^ (32u * s)) + 32 * kRowBytes * j);
    };
    const auto read_bytes = [&](int odd, int word, int i) {
      const uint8_t* from = lds + kRing + kHalf * odd + 8 * half + 4 * word + 16 * c;
      bytes_a[word][i] = *reinterpret_cast<const uint32_t*>(from + 16 * (BN + 32 * wave_row) + 512 * WR * i);
#pragma unroll
      for (int j = i * CB / R; j < (i + 1) * CB / R; ++j)
        bytes_b[word][j] = *reinterpret_cast<const uint32_t*>(from + 512 * CB * wave_col + 512 * j);
    };
    // The products of step `T` of a window; `beside(i)` issues reads and copies before row i's, to run under them.
    const auto multiply = [&](auto T, const Frags& f, auto&& beside) {
      constexpr int s = decltype(T)::value & 3, word = decltype(T)::value >> 2;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        beside(i);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < CB; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand4(f.a[i]), operand4(f.b[j]), acc[i][j], 4, 4, s,
                                                                      int(bytes_a[word][i]), s, int(bytes_b[word][j]));
        hold<CB>(acc[i]);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    constexpr int kPer = (kUnits + 2 * R - 1) / (2 * R);  // copies beside a row, over two steps
    const auto copies = [&](int chunk, int stage, int part) {
#pragma unroll
      for (int u = part * kPer; u < (part + 1) * kPer; ++u)
        if (u < kUnits) copy_unit(chunk, stage, u);
    };
    // All copies but the last `behind` have landed, and everyone is done with the stage before.
    const auto sync = [&](auto behind) {
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(decltype(behind)::value));
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_sched_barrier(0);
    };
    // Stages go round with the chunks: the one that the current chunk is in, and the n-th after it.
    int at = 0;
    const auto after = [](int stage, int n) {
      const int to = stage + n * kStage;
      return to >= ST * kStage ? to - ST * kStage : to;
    };
    // Step `T` of a window.  With MORE windows behind it, nothing in it is a branch: the compiler moves
    // products over one.
    const auto step = [&](auto T, auto more, int odd, int window) {
      constexpr int kT8 = decltype(T)::value, s = kT8 & 3, kChunk = kT8 >> 2;
      constexpr bool kMore = decltype(more)::value;
      const int chunk = 2 * window + kChunk;
      Frags& f = kT8 & 1 ? f1 : f0;
      Frags& g = kT8 & 1 ? f0 : f1;
      // the last chunk that is copied before this one ends: of the last window no more than it has
      constexpr int kCopied = kMore || kChunk + ST - 1 < 2 ? kChunk + ST - 1 : 1;
      if constexpr (s == 3) {
        constexpr bool kLast = !kMore && kT8 == 7;
        if (!kLast) sync(std::integral_constant<int, kCopied - kChunk - 1 < 0 ? 0 : (kCopied - kChunk - 1) * kUnits>{});
        const int here = at;
        at = after(at, 1);
        multiply(T, f, [&](int i) {
          if (!kLast) read(at, 0, g, i);
          if (kMore && kT8 == 7) read_bytes(odd ^ 1, 0, i);
          if (kMore || kChunk + ST < 2) copies(chunk + ST, here, i);
        });
      } else {
        multiply(T, f, [&](int i) {
          read(at, s + 1, g, i);
          if (kT8 == 0) read_bytes(odd, 1, i);
          if (s == 0 && (kMore || kChunk + ST - 1 < 2)) copies(chunk + ST - 1, after(at, ST - 1), R + i);
          if (kMore && kT8 == 4 && i == 0 && odd) {
            put_scales((window + 1) >> 1);
            load_scales((window + 3) >> 1);
          }
        });
      }
    };
    using Yes = std::true_type;
    using No = std::false_type;
    // The first window's bytes are asked for before the copies (loads come back in order), the next one's after.
    if (nb >= 16) load_scales(0);
#pragma unroll
    for (int k = 0; k < ST - 1; ++k)
#pragma unroll
      for (int u = 0; u < kUnits; ++u) copy_unit(k, k * kStage, u);
    if (nb >= 16) {
      put_scales(0);
    } else {
#pragma unroll
      for (int i = 0; i < kTurns; ++i) put(i, load_few_bytes(sbase[i] + soff[i], tid & 1 ? 0 : nb));
    }
    sync(std::integral_constant<int, 0>{});
    if (nb >= 16) load_scales(1);
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
      for (int j = 0; j < CB; ++j) acc[i][j] = f32x16{};
      read(0, 0, f0, i);
      read_bytes(0, 0, i);
      copies(ST - 1, (ST - 1) * kStage, i);
    }
    const auto window = [&](int odd, int w) {
      step(std::integral_constant<int, 0>{}, Yes{}, odd, w);
      step(std::integral_constant<int, 1>{}, Yes{}, odd, w);
      step(std::integral_constant<int, 2>{}, Yes{}, odd, w);
      step(std::integral_constant<int, 3>{}, Yes{}, odd, w);
      step(std::integral_constant<int, 4>{}, Yes{}, odd, w);
      step(std::integral_constant<int, 5>{}, Yes{}, odd, w);
      step(std::integral_constant<int, 6>{}, Yes{}, odd, w);
      step(std::integral_constant<int, 7>{}, Yes{}, odd, w);
    };
    int w = 0;
    for (; w + 2 < windows; w += 2) {
      window(0, w);
      window(1, w + 1);
    }
    if (w + 1 < windows) window(0, w++);
    const int steps = (nb - 16 * w + 1) >> 1, odd = w & 1;  // 1 .. 8 of the last window
    step(std::integral_constant<int, 0>{}, No{}, odd, w);
    if (steps > 1) step(std::integral_constant<int, 1>{}, No{}, odd, w);
    if (steps > 2) step(std::integral_constant<int, 2>{}, No{}, odd, w);
    if (steps > 3) step(std::integral_constant<int, 3>{}, No{}, odd, w);
    if (steps > 4) step(std::integral_constant<int, 4>{}, No{}, odd, w);
    if (steps > 5) step(std::integral_constant<int, 5>{}, No{}, odd, w);
    if (steps > 6) step(std::integral_constant<int, 6>{}, No{}, odd, w);
    if (steps > 7) step(std::integral_constant<int, 7>{}, No{}, odd, w);
    __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(0));  // no copy is left when the LDS is given back

    // out: element r of a block is row 8 (r / 4) + 4 half + r % 4; a lane's columns are CB c ..
    typedef row_elem<ODT> out_t;
    constexpr int kSize = sizeof(out_t);
    // the lane's number anew: kept over the loop it would be a register too many
    const int l = int(__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u)));
    const int lane_col = CB * (32 * wave_col + (l & 31));
    float bias[CB];
#pragma unroll
    for (int j = 0; j < CB; ++j) bias[j] = p.bias && lane_col + j < cols ? p.bias[wrow0 + lane_col + j] : 0.f;
    const uint32_t pitch = uint32_t(p.N) * kSize;
    const auto store = [&](auto together) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int first = 32 * (WR * i + wave_row), rows = t.rows - first < 32 ? t.rows - first : 32;
        if (rows <= 0) break;
        const __amdgpu_buffer_rsrc_t ores = uniform_rsrc(static_cast<out_t*>(p.out) + (t.row0 + first) * p.N + n0,
                                                         uint32_t(rows - 1) * pitch + uint32_t(cols) * kSize);
        uint32_t to[CB];
#pragma unroll
        for (int j = 0; j < CB; ++j)
          to[j] = lane_col + j < cols ? uint32_t(4 * (l >> 5)) * pitch + uint32_t(lane_col + j) * kSize : 0x80000000u;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const uint32_t row = uint32_t(8 * (r >> 2) + (r & 3)) * pitch;
          if constexpr (decltype(together)::value) {
            static_assert(CB == 2, "columns of a lane");
            const float v0 = acc[i][0][r] + bias[0], v1 = acc[i][1][r] + bias[1];
            if constexpr (ODT == 0) __builtin_amdgcn_raw_buffer_store_b32(bf16_rne2(v0, v1), ores, to[0] + row, 0, kPastCaches);
            else __builtin_amdgcn_raw_buffer_store_b64(u32x2{__float_as_uint(v0), __float_as_uint(v1)}, ores, to[0] + row, 0, kPastCaches);
          } else {
#pragma unroll
            for (int j = 0; j < CB; ++j) {
              const float v = acc[i][j][r] + bias[j];
              if constexpr (ODT == 0) __builtin_amdgcn_raw_buffer_store_b16(bf16_rne(v), ores, to[j] + row, 0, kPastCaches);
              else __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), ores, to[j] + row, 0, kPastCaches);
            }
          }
          if ((r & 3) == 3) __builtin_amdgcn_sched_barrier(0);  // a few sums in registers at a time
        }
      }
    };
    if (CB == 2 && p.N % CB == 0) store(std::integral_constant<bool, CB == 2>{});  // rows begin at the pair's alignment
    else store(std::false_type{});
  };
  const int blocks = (t.rows + 32 * WR - 1) / (32 * WR);
  if (RB > 2 && blocks > 2) run(std::integral_constant<int, RB>{});
  else if (RB > 1 && blocks > 1) run(std::integral_constant<int, RB < 2 ? RB : 2>{});
  else run(std::integral_constant<int, 1>{});
}

// The form of few tiles, where the tile form would leave CUs without one.  A workgroup has up to 16 RB rows of an
// expert by 16 CB columns; its WK waves take chunks of 16 blocks in turn, straight from memory into the
// instruction's registers, and their sums meet in LDS in a fixed order.  Step s of a chunk takes blocks 4 s to
// 4 s + 3, sixteen lanes each: half a line of a row, so w's lines are kept for the next step (past the caches 29.4 us
// for two experts' row at [28672, 4096], 27.9 so).  Bound: the latency of a chunk's loads and the join, and for many
// rows the rows of x that every column tile reads anew.  Two chunks under way where registers allow it (one row
// at [4096, 14336] 10.0 us, one chunk 13.7; for 2 x 2 blocks two take the second workgroup of a CU its registers, for 4 x 4 there is no room).
template <int ODT, int WK, int RB, int CB>
__global__ void __launch_bounds__(WK * kWave, RB * CB == 1 ? 4 : 2) few_kernel(GemmArgs p) {
  constexpr int BM = 16 * RB, BN = 16 * CB, kBmLog2 = RB == 1 ? 4 : (RB == 2 ? 5 : 6), CH = 16;
  __shared__ f32x4 part[WK][RB][CB][kWave];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 15, q = lane >> 4;
  const GemmTile t = find_gemm_tile(p.offsets, p.E, p.S, kBmLog2, p.col_tiles, false, blockIdx.x);
  if (t.rows == 0) return;
  const int nb = int(p.K >> 5), chunks = (nb + CH - 1) / CH;
  const uint32_t rowb = uint32_t(nb) * 16u;
  const int64_t n0 = int64_t(t.col) * BN;
  const int cols = p.N - n0 < BN ? int(p.N - n0) : BN;
  const int64_t wrow0 = int64_t(t.expert) * p.N + n0;
  const __amdgpu_buffer_rsrc_t xres = uniform_rsrc(p.x + t.row0 * rowb, uint32_t(t.rows) * rowb);
  const __amdgpu_buffer_rsrc_t wres = uniform_rsrc(p.w + wrow0 * rowb, uint32_t(cols) * rowb);
  const uint8_t *wsb = p.ws + wrow0 * nb, *xsb = p.xs + t.row0 * nb;
  const uint32_t own = uint32_t(c) * rowb + 16u * q;
  // Rows behind the last have no codes (the buffers end) and the last one's bytes, which nothing reads outside.
  uint32_t w_bytes[CB], x_bytes[RB];
#pragma unroll
  for (int j = 0; j < CB; ++j) w_bytes[j] = uint32_t(16 * j + c < cols ? 16 * j + c : cols - 1) * uint32_t(nb);
#pragma unroll
  for (int i = 0; i < RB; ++i) x_bytes[i] = uint32_t(16 * i + c < t.rows ? 16 * i + c : t.rows - 1) * uint32_t(nb);

  struct Chunk {
    u32x4 w[CB][4], x[RB][4], ws[CB], xs[RB];
  };
  const auto load_codes = [&](int chunk, Chunk& k) {
    const uint32_t at = own + uint32_t(16 * CH * chunk);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
#pragma unroll
      for (int j = 0; j < CB; ++j)
        k.w[j][s] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(wres, at + 64u * s + 16u * j * rowb, 0, 0));
#pragma unroll
      for (int i = 0; i < RB; ++i)
        k.x[i][s] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(xres, at + 64u * s + 16u * i * rowb, 0, 0));
    }
  };
  const auto load = [&](int chunk, Chunk& k) {
#pragma unroll
    for (int j = 0; j < CB; ++j) k.ws[j] = load_bytes16(wsb, w_bytes[j], CH * chunk, nb);
#pragma unroll
    for (int i = 0; i < RB; ++i) k.xs[i] = load_bytes16(xsb, x_bytes[i], CH * chunk, nb);
    load_codes(chunk, k);
  };
  f32x4 acc[RB][CB];
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < CB; ++j) acc[i][j] = f32x4{};
  const uint32_t low = 0x0C0C0400u + 0x0101u * q, high = 0x04000C0Cu + 0x01010000u * q;  // byte q of each word
  const auto bytes_of = [&](u32x4 v) {
    return int(perm(v[1], v[0], low) | perm(v[3], v[2], high));
  };
  const auto multiply = [&](const Chunk& k) {
    int wb[CB], xb[RB];
#pragma unroll
    for (int j = 0; j < CB; ++j) wb[j] = bytes_of(k.ws[j]);
#pragma unroll
    for (int i = 0; i < RB; ++i) xb[i] = bytes_of(k.xs[i]);
    const auto step = [&](auto S) {
      constexpr int s = decltype(S)::value;
#pragma unroll
      for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < CB; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand4(k.x[i][s]), operand4(k.w[j][s]), acc[i][j], 4, 4,
                                                                       s, xb[i], s, wb[j]);
    };
    step(std::integral_constant<int, 0>{});
    step(std::integral_constant<int, 1>{});
    step(std::integral_constant<int, 2>{});
    step(std::integral_constant<int, 3>{});
  };
  const auto use = [&](int chunk, Chunk& k) {
#pragma unroll
    for (int j = 0; j < CB; ++j) k.ws[j] = bytes_from(k.ws[j], CH * chunk, nb);
#pragma unroll
    for (int i = 0; i < RB; ++i) k.xs[i] = bytes_from(k.xs[i], CH * chunk, nb);
    multiply(k);
  };
  if (nb >= 16) {
    int at = wave;
    if constexpr (RB * CB == 1) {
      // A chunk is loaded before the last is used.  The loop goes on only where both are there: the compiler waits
      // for every load behind a branch that may or may not have had some.
      Chunk k0, k1;
      if (at < chunks) load(at, k0);
      while (at < chunks) {
        if (at + WK >= chunks) {
          use(at, k0);
          break;
        }
        load(at + WK, k1);
        use(at, k0);
        at += WK;
        if (at + WK >= chunks) {
          use(at, k1);
          break;
        }
        load(at + WK, k0);
        use(at, k1);
        at += WK;
      }
    } else {
      for (; at < chunks; at += WK) {
        Chunk k;
        load(at, k);
        use(at, k);
      }
    }
  } else if (wave == 0) {
    Chunk k;
    load_codes(0, k);
#pragma unroll
    for (int j = 0; j < CB; ++j) k.ws[j] = load_few_bytes(wsb + w_bytes[j], nb);
#pragma unroll
    for (int i = 0; i < RB; ++i) k.xs[i] = load_few_bytes(xsb + x_bytes[i], nb);
    multiply(k);
  }
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < CB; ++j) part[wave][i][j][lane] = acc[i][j];
  __syncthreads();
  // element r of lane l is row 4 (l / 16) + r, column l % 16
  for (int o = tid; o < BM * BN; o += WK * kWave) {
    const int col = o & (BN - 1), row = o / BN, from = 16 * ((row & 15) >> 2) + (col & 15);
    if (row >= t.rows || col >= cols) continue;
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < WK; ++w) sum += reinterpret_cast<const float*>(&part[w][row >> 4][col >> 4][from])[row & 3];
    if (p.bias) sum += p.bias[wrow0 + col];
    row_elem<ODT>* to = static_cast<row_elem<ODT>*>(p.out) + (t.row0 + row) * p.N + n0 + col;
    if constexpr (ODT == 0) *to = bf16_rne(sum);
    else *to = sum;
  }
}

template <int RB, int CB, int WR, int WC, int RING>
void tile(const MxGemmLaunch& L, const GemmArgs& a, unsigned grid, hipStream_t s) {
  if (L.out_dtype == 0) hipLaunchKernelGGL((tile_kernel<0, RB, CB, WR, WC, RING>), dim3(grid), dim3(WR * WC * kWave), 0, s, a);
  else hipLaunchKernelGGL((tile_kernel<1, RB, CB, WR, WC, RING>), dim3(grid), dim3(WR * WC * kWave), 0, s, a);
}

template <int RB, int CB>
void few(const MxGemmLaunch& L, const GemmArgs& a, unsigned grid, hipStream_t s) {
  if (L.out_dtype == 0) hipLaunchKernelGGL((few_kernel<0, 4, RB, CB>), dim3(grid), dim3(4 * kWave), 0, s, a);
  else hipLaunchKernelGGL((few_kernel<1, 4, RB, CB>), dim3(grid), dim3(4 * kWave), 0, s, a);
}

}  // namespace

// A wave for every piece of a row, or for several rows.
struct QuantShape {
  int64_t per, pieces, together, waves;
};
QuantShape quant_shape(int64_t S, int64_t K) {
  QuantShape q{K / 8, mx_div_up(K / 8, kWave * kQuantTurns), 1, 0};
  if (q.per <= kWave * kQuantTurns / 2) q.together = kWave * kQuantTurns / q.per;
  q.waves = mx_div_up(S, q.together) * q.pieces;
  return q;
}
int64_t quantize_mxfp4_items(int64_t S, int64_t K) { return mx_div_up(quant_shape(S, K).waves * kWave, kThreads) * kThreads; }
int64_t mxfp4_gemm_items(const MxGemmLaunch& L) {
  const MxTileForm f = mx_tile_form(L.E, L.N, L.S, cu_count());
  return mx_gemm_blocks(f, L.E, L.N, L.S) * f.threads;
}

hipError_t launch_quantize_mxfp4(const void* x, int dtype, int64_t T, int64_t K, int k, const int32_t* slots,
                                 uint8_t* blocks, uint8_t* scales, hipStream_t stream) {
  if (T == 0) return hipSuccess;
  const int64_t S = T * k;
  const QuantShape q = quant_shape(S, K);
  const QuantArgs a{x, slots, blocks, scales, K, uint32_t(S), uint32_t(q.per), uint32_t(q.pieces), uint32_t(q.together),
                    uint32_t(q.waves), k};
  const dim3 grid(unsigned(mx_div_up(q.waves * kWave, kThreads)));
  const auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, stream, a); };
  if (q.together > 1) dtype == 0 ? go(quantize_kernel<0, true>) : go(quantize_kernel<1, true>);
  else dtype == 0 ? go(quantize_kernel<0, false>) : go(quantize_kernel<1, false>);
  return hipGetLastError();
}

hipError_t launch_mxfp4_gemm(const MxGemmLaunch& L, hipStream_t stream) {
  if (L.S == 0) return hipSuccess;
  const MxTileForm f = mx_tile_form(L.E, L.N, L.S, cu_count());
  const int64_t blocks = mx_gemm_blocks(f, L.E, L.N, L.S);
  const GemmArgs a{L.x, L.xs, L.w, L.ws, L.bias, L.offsets, L.out, L.N, L.K, int(L.S), int(L.E), uint32_t(mx_div_up(L.N, f.bn)),
                   mx_two_lists(blocks, cu_count())};
  const unsigned grid = unsigned(blocks);
  if (f.bm == 256) tile<4, 2, 2, 4, 2>(L, a, grid, stream);
  else if (f.bm == 128) tile<2, 2, 2, 2, 2>(L, a, grid, stream);
  else if (f.bm == 64 && f.bn == 128) tile<2, 1, 1, 4, 3>(L, a, grid, stream);
  else if (f.bm == 64) few<4, 4>(L, a, grid, stream);
  else if (f.bm == 32) few<2, 2>(L, a, grid, stream);
  else few<1, 1>(L, a, grid, stream);
  return hipGetLastError();
}

}  // namespace e4b
