// Low-rank adapters on grouped rows, beside a projection that others compute, and their
// gradients.  Rows are grouped (by expert: the router's offsets; by request: the batch's), a group
// g uses adapter a = group_adapter[g] (or g itself):
//   forward    z = x A_a^T,  out = y + s_a z B_a^T
//   backward   u = s_a g B_a,  gx = gx0 + u A_a,  gA_a = sum_p u_p^T x_p,  gB_a = s_a sum_p g_p^T z_p
// with A_a [r, K], B_a [N, r] bf16, r = 8 .. 128.  About 2r / b flop for each byte moved (b the
// bytes of an element read and written): by its bytes and operations alone memory bounds every rank
// taken here, so the kernels are three streaming passes with the matrix unit beside them (the gradients
// above rank 32 are not that near: z and u there cost as much as g, at one workgroup a CU):
//   shrink   [rows, C] x [r, C]^T -> [rows, r]     (z from x and A)
//   expand   [rows, r] x [C, r]^T added to [rows, C]   (out from z and B; gx from u and A^T)
//   grad     [rows, r]^T x [rows, C] -> [r, C]     (gA from u and x; gB from z and g, with u in the same pass)
// Products of bf16 values go through the bf16 matrix instruction exactly, with float32 sums.  z
// and u are float32 all the way: in expand each is cut into three bf16 parts (8 + 8 + 8 bits of
// its 24-bit significand: no rounding) that stand behind one another in the contraction, and so in
// grad.
#include "e4b_internal.h"
#include "e4b_rows.h"

namespace e4b {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;

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

// Loads and stores go through buffers that end with the tile's rows or the adapter's matrix: a
// lane's offset is fixed for the tile, the step's offset is scalar, and what lies past the end
// reads as zero and is not written, with no test (64-bit addresses and tests by lane cost the small
// tiles a tenth: 17.4 us against 15.6 for 64 decoded tokens).
__device__ __forceinline__ u32x4 buf_load(__amdgpu_buffer_rsrc_t r, uint32_t lane_off, uint32_t off) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, lane_off, off, 0));
}
__device__ __forceinline__ bf16x8 buf_load8(__amdgpu_buffer_rsrc_t r, uint32_t lane_off, uint32_t off) {
  return __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(r, lane_off, off, 0));
}
// A buffer whose base and size are the same in every lane; said so, they stay in scalar registers
// (else each access becomes a loop over the lanes' values).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t wave_rsrc(const void* base, uint32_t bytes) {
  const uint64_t b = reinterpret_cast<uint64_t>(base);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(uint32_t(b)), hi = __builtin_amdgcn_readfirstlane(uint32_t(b >> 32));
  return buffer_rsrc(reinterpret_cast<const void*>(uint64_t(lo) | (uint64_t(hi) << 32)),
                     __builtin_amdgcn_readfirstlane(bytes));
}
// Stores of rows go past the caches (the instruction's non-temporal bit): more is written than they
// hold, and kept there it slowed the kernels that followed (8-expert down projection 113 us, 99 so: the
// call again and again, with no reader of the rows in between).
constexpr int kPastCaches = 2;
constexpr uint32_t kNowhere = 0x80000000u;  // past the end of every buffer (of 2^31 bytes at most)

// 16 bytes a lane.  A store of more than 64 bits reads its registers some cycles after it is issued,
// and the compiler keeps their next values away for as long, except where the offset is in a scalar
// register: there nothing stood between such a store and the next write of its first register, and
// with other work on the CU some rows came out with that value in them.  So the whole offset is the
// lane's (past-the-end lanes still are: kNowhere and a tile's offsets stay under 2^32).
__device__ __forceinline__ void store_wide(u32x4 v, __amdgpu_buffer_rsrc_t r, uint32_t lane_off) {
  __builtin_amdgcn_raw_buffer_store_b128(v, r, lane_off, 0, kPastCaches);
}

// Sums of one wave over its units of 64 columns (128 bytes of each row): acc[b][k] gets rows 16b ..
// of the tile by ranks 16k .. .  The wave takes its share of the units first .. end - 1 one after the
// other (the waves' units in turn read 10 % slower).  A unit comes in whole lines (8 lanes a row; a
// matrix operand read straight from memory has neighbouring lanes in different rows, and costs the
// load path three times as long) through registers into the wave's own LDS, the next AHEAD units'
// loads in flight.  The 16-byte pieces of a row are exchanged by the row so that reads of 16 rows
// spread over all banks.  The adapter is the matrix instruction's first operand, so a lane ends with
// 4 ranks of one row.
constexpr int kUnitBytes = 2048;  // 16 rows of a unit
template <int RB, int RT, int AHEAD>
__device__ __forceinline__ void shrink_sums(uint8_t* lds, const uint16_t* __restrict__ m, const uint16_t* __restrict__ w,
                                            uint32_t C, int r, int rows, int first, int end, int waves,
                                            f32x4 (&acc)[RB][RT]) {
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t c = lane & 15, q = lane >> 4, lrow = lane >> 3, lpiece = lane & 7;
  const __amdgpu_buffer_rsrc_t mres = wave_rsrc(m, uint32_t(rows) * C * 2u);
  const __amdgpu_buffer_rsrc_t wres = wave_rsrc(w, uint32_t(r) * C * 2u);
  const uint32_t lane_off = lrow * C * 2u + 16u * lpiece, step = 16u * C;  // bytes of 8 rows
  constexpr int kM = 2 * RB, kLoads = 2 * (RB + RT);
  uint8_t* own = lds + wave * (RB + RT) * kUnitBytes;
  const int share = (end - first + waves - 1) / waves, from = first + wave * share;
  const int to = from + share < end ? from + share : end;
  auto load = [&](int s, u32x4 (&v)[kLoads]) {  // past the share and the columns: zeros; past the rows of m and w too
    const uint32_t off = s < to && 64u * s + 8u * lpiece < C ? lane_off : kNowhere;
#pragma unroll
    for (int j = 0; j < kLoads; ++j)
      v[j] = j < kM ? buf_load(mres, off, 128u * s + j * step) : buf_load(wres, off, 128u * s + (j - kM) * step);
  };
  auto multiply = [&](const u32x4 (&v)[kLoads], auto&& next) {
#pragma unroll
    for (int j = 0; j < kLoads; ++j)
      *reinterpret_cast<u32x4*>(own + 1024 * j + 128 * lrow + 16 * (lpiece ^ ((lrow >> 1) | (4 * (j & 1))))) = v[j];
    next();
    bf16x8 f[2][RB + RT];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int b = 0; b < RB + RT; ++b)
        f[u][b] = *reinterpret_cast<const bf16x8*>(own + kUnitBytes * b + 128 * c + 16 * ((4 * u + q) ^ (c >> 1)));
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int k = 0; k < RT; ++k)
          acc[b][k] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f[u][RB + k], f[u][b], acc[b][k], 0, 0, 0);
  };
  u32x4 v[AHEAD][kLoads];
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) load(from + i, v[i]);
  for (int s = from; s < to; s += AHEAD) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (i == 0 || s + i < to)
        multiply(v[i], [&] {
          if (s + i + AHEAD < to) load(s + i + AHEAD, v[i]);
        });
  }
}

template <int RB, int RT>
__device__ __forceinline__ void zero_sums(f32x4 (&acc)[RB][RT]) {
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int k = 0; k < RT; ++k) acc[b][k] = f32x4{0.f, 0.f, 0.f, 0.f};
}

struct ShrinkArgs {
  const uint16_t* m;      // [S, C]
  const uint16_t* w;      // [n, r, C]
  const float* scale;     // nullable: 1
  const int32_t* offsets;
  const int32_t* ids;     // nullable: group = adapter
  float* z;               // [ksplit, S, r]
  int64_t C;
  int S, G, n, r, bm_log2;
  uint32_t ksplit;
  int per;                // units of a piece
};

// A workgroup: up to 16 * RB rows of a group and one piece of the columns; its waves'
// sums meet in LDS.  Bound: HBM, by x: 8192 rows of 14336 at rank 16 (239 MB) take 47 us, 5.0 TB/s.
// 5003 rows of 2880 at rank 64 (29 MB) take 11 us, most of it the round of latencies of a workgroup
// that has three units a wave.
template <int RB, int RT>
__global__ void __launch_bounds__(kThreads) shrink_kernel(ShrinkArgs p) {
  // the waves' units, and after them the waves' sums
  constexpr int kUnits = kWaves * (RB + RT) * kUnitBytes, kSums = kWaves * RB * RT * kWave * 16;
  __shared__ __attribute__((aligned(16))) uint8_t lds[kUnits > kSums ? kUnits : kSums];
  f32x4 (*part)[RB * RT][kWave] = reinterpret_cast<f32x4 (*)[RB * RT][kWave]>(lds);
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x >> 6;
  const int c = lane & 15, q = lane >> 4;
  const uint32_t tile = blockIdx.x / p.ksplit;
  const int ks = int(blockIdx.x - tile * p.ksplit);
  const RowTile t = find_tile(p.offsets, p.ids, p.n, p.G, p.S, p.bm_log2, tile);
  if (t.rows == 0) return;
  const int a = t.adapter;
  f32x4 acc[RB][RT];
  zero_sums(acc);
  if (a >= 0) {
    const int units = int((p.C + 63) >> 6);
    const int end = (ks + 1) * p.per < units ? (ks + 1) * p.per : units;
    shrink_sums<RB, RT, 1>(lds, p.m + t.row0 * p.C, p.w + int64_t(a) * p.r * p.C, uint32_t(p.C), p.r, t.rows,
                           ks * p.per, end, kWaves, acc);
  }
  __syncthreads();
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int k = 0; k < RT; ++k) part[wave][b * RT + k][lane] = acc[b][k];
  const float sc = a >= 0 && p.scale ? p.scale[a] : 1.f;
  __syncthreads();
  float* z = p.z + int64_t(ks) * p.S * p.r;
#pragma unroll
  for (int i0 = 0; i0 < RB * RT; i0 += kWaves) {
    const int i = i0 + wave;
    if (i >= RB * RT) break;
    f32x4 v = part[0][i][lane];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) v += part[w][i][lane];
    const int row = 16 * (i / RT) + c, rank = 16 * (i % RT) + 4 * q;
    if (row < t.rows && rank < p.r) *reinterpret_cast<f32x4*>(z + (t.row0 + row) * p.r + rank) = v * sc;
  }
}

// The three parts of v, v = hi + mid + lo exactly, each the 8 leading bits of what is left.  An
// infinity or NaN stands in the first part alone.
struct Parts {
  uint32_t hi, mid, lo;  // bf16 in the upper half
};
__device__ __forceinline__ Parts split3(float v) {
  const uint32_t b = __float_as_uint(v);
  const bool finite = (b & 0x7F800000u) != 0x7F800000u;
  const float r1 = v - __uint_as_float(b & 0xFFFF0000u);
  const uint32_t b1 = __float_as_uint(r1);
  const float r2 = r1 - __uint_as_float(b1 & 0xFFFF0000u);
  Parts p;
  p.hi = finite ? b : b | ((b & 0x007FFFFFu) ? 0x00400000u : 0u);
  p.mid = finite ? b1 : 0u;
  p.lo = finite ? __float_as_uint(r2) : 0u;
  return p;
}
// The upper halves of two words as one (first in the low half).
__device__ __forceinline__ uint32_t hi2(uint32_t first, uint32_t second) { return perm(second, first, 0x07060302u); }

// Geometry of the second product at RP ranks (r rounded up to a power of two) and out type ODT: the
// row's z stands as hi | mid | lo parts of RP ranks behind one another in the contraction, the
// matrix instruction's first operand.  A wave takes 64 columns at a time, four matrix tiles with the
// columns dealt out in turn (tile h has columns 4c + h), so that a lane holds 4 consecutive columns
// and 16 neighbouring lanes a row's 64: the rows are read and written in whole lines.  (With a lane
// in a row of its own, as the instruction's other orientation has it, each access cost the load path
// about 45 cycles instead of 16: gx of the 32-expert layer 55 us.)
template <int RP, int ODT>
struct Expand {
  static constexpr int kSteps = (3 * RP + 31) / 32;      // 32-deep matrix steps over the three parts
  static constexpr int kFrags = RP >= 32 ? RP / 32 : 1;  // distinct adapter fragments among them
  static constexpr int kStride = 32 * kSteps + 8;        // LDS row in bf16 (16 rows hit distinct banks)
  static constexpr int kH = 4, kCols = 64;
  typedef row_elem<ODT> out_t;

  // Ranks rank .. rank + 3 of one row into the LDS row zr.
  static __device__ __forceinline__ void put(uint16_t* zr, int rank, f32x4 v) {
    Parts s[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j] = split3(v[j]);
    *reinterpret_cast<u32x2*>(zr + rank) = u32x2{hi2(s[0].hi, s[1].hi), hi2(s[2].hi, s[3].hi)};
    *reinterpret_cast<u32x2*>(zr + RP + rank) = u32x2{hi2(s[0].mid, s[1].mid), hi2(s[2].mid, s[3].mid)};
    *reinterpret_cast<u32x2*>(zr + 2 * RP + rank) = u32x2{hi2(s[0].lo, s[1].lo), hi2(s[2].lo, s[3].lo)};
    if (3 * RP + rank < 32 * kSteps) *reinterpret_cast<u32x2*>(zr + 3 * RP + rank) = u32x2{0u, 0u};
  }

  // What a step reads: 4 columns of 4 rows of each row block, and the adapter's fragments.
  typedef uint32_t vec __attribute__((ext_vector_type(ODT == 0 ? 2 : 4)));
  template <int RB>
  struct Step {
    vec y[RB][4];
    bf16x8 w[kH][kFrags];
  };
  static constexpr uint32_t kSize = sizeof(out_t);

  // The rows of a tile (row 0 at base and out) and the adapter's [C, r].
  template <int RB>
  struct Rows {
    __amdgpu_buffer_rsrc_t base, out, w;
    uint32_t C, r, row_off, w_off[kFrags];
    int rows;
    bool adapter;

    __device__ __forceinline__ Rows(const out_t* base_, out_t* out_, const uint16_t* w_, uint32_t C_, int r_, int rows_,
                                    bool adapter_)
        : base(wave_rsrc(base_, base_ ? uint32_t(rows_) * C_ * kSize : 0u)),  // no base: all of it reads as zero
          out(wave_rsrc(out_, uint32_t(rows_) * C_ * kSize)),
          w(wave_rsrc(w_, C_ * uint32_t(r_) * 2u)), C(C_), r(uint32_t(r_)), rows(rows_), adapter(adapter_) {
      const uint32_t lane = threadIdx.x & (kWave - 1), c = lane & 15, q = lane >> 4;
      row_off = (4 * q * C + 4 * c) * kSize;
#pragma unroll
      for (int f = 0; f < kFrags; ++f) {
        const uint32_t rank = (32u * f + 8u * q) % RP;  // ranks past r meet zeros of z
        w_off[f] = (4 * c * r + (rank < r ? rank : 0u)) * 2u;
      }
    }

    // The lane's offset in step s: past every row where its columns are past the last.
    __device__ __forceinline__ uint32_t lane_off(uint32_t s) const {
      return kCols * s + 4 * (threadIdx.x & 15) < C ? row_off : kNowhere;
    }

    __device__ __forceinline__ void load(uint32_t s, Step<RB>& t) const {
      const uint32_t off = lane_off(s);
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (RB == 1 && e >= rows) continue;  // no lane has such a row (decoded tokens)
          const uint32_t at = (kCols * s + (16 * b + e) * C) * kSize;
          if constexpr (ODT == 0) t.y[b][e] = __builtin_bit_cast(vec, __builtin_amdgcn_raw_buffer_load_b64(base, off, at, 0));
          else t.y[b][e] = buf_load(base, off, at);
        }
      if (adapter) {
#pragma unroll
        for (int h = 0; h < kH; ++h)
#pragma unroll
          for (int f = 0; f < kFrags; ++f) t.w[h][f] = buf_load8(w, w_off[f], (kCols * s + h) * r * 2u);
      }
    }

    __device__ __forceinline__ void finish(uint32_t s, const Step<RB>& t, const bf16x8 (&zf)[RB][kSteps]) const {
      const uint32_t off = lane_off(s);
#pragma unroll
      for (int b = 0; b < RB; ++b) {
        f32x4 d[kH];
        if (adapter) {
#pragma unroll
          for (int h = 0; h < kH; ++h) d[h] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int k = 0; k < kSteps; ++k)
#pragma unroll
            for (int h = 0; h < kH; ++h)
              d[h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(zf[b][k], t.w[h][k % kFrags], d[h], 0, 0, 0);
        } else {  // y + -0 is y, whichever zero y is
#pragma unroll
          for (int h = 0; h < kH; ++h) d[h] = f32x4{-0.f, -0.f, -0.f, -0.f};
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (RB == 1 && e >= rows) continue;
          const uint32_t at = (kCols * s + (16 * b + e) * C) * kSize;
          const vec y = t.y[b][e];
          if constexpr (ODT == 1) {
            u32x4 o;
#pragma unroll
            for (int h = 0; h < 4; ++h) o[h] = __float_as_uint(__uint_as_float(y[h]) + d[h][e]);
            store_wide(o, out, off + at);
          } else {
            u32x2 o;
#pragma unroll
            for (int h = 0; h < 2; ++h)
              o[h] = bf16_rne2(__uint_as_float(y[h] << 16) + d[2 * h][e],
                               __uint_as_float(y[h] & 0xFFFF0000u) + d[2 * h + 1][e]);
            __builtin_amdgcn_raw_buffer_store_b64(o, out, off, at, kPastCaches);
          }
        }
      }
    }
  };

  template <int RB>
  static __device__ __forceinline__ void fragments(const uint16_t* zs, bf16x8 (&zf)[RB][kSteps]) {
    const int lane = threadIdx.x & (kWave - 1), c = lane & 15, q = lane >> 4;
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int k = 0; k < kSteps; ++k)
        zf[b][k] = *reinterpret_cast<const bf16x8*>(zs + (16 * b + c) * kStride + 32 * k + 8 * q);
  }

  // Steps whose loads a wave has in flight together.
  static constexpr int ahead(int rb) { return rb == 1 && RP <= 32 ? 2 : 1; }
};

struct ExpandArgs {
  const float* z;         // [ksplit, S, r]: the sum over ksplit is taken here
  const uint16_t* w;      // [n, C, r]
  const float* scale;     // nullable: 1
  const int32_t* offsets;
  const int32_t* ids;
  const void* base;       // nullable [S, C]
  void* out;              // [S, C]
  float* z_out;           // nullable [S, r]: the summed z
  int64_t C;
  int S, G, n, r, bm_log2, ksplit;
  uint32_t chunks;
  int per;                // column steps of a chunk
};

// A workgroup: up to 16 * RB rows of a group and one piece of the columns.  Bound: HBM, by the rows
// read and written: 8192 rows of 4096 float32 at rank 16 (270 MB) take 50 us, 5.4 TB/s; 5003 bf16 rows
// of 2880 at rank 64 (60 MB) 21 us, where the z of a tile and its three parts (made by each workgroup
// before its first product) are a third.
template <int RB, int RP, int ODT>
__global__ void __launch_bounds__(kThreads) expand_kernel(ExpandArgs p) {
  typedef Expand<RP, ODT> X;
  __shared__ __attribute__((aligned(16))) uint16_t zs[16 * RB * X::kStride];
  const uint32_t tile = blockIdx.x / p.chunks;
  const int chunk = int(blockIdx.x - tile * p.chunks);
  const RowTile t = find_tile(p.offsets, p.ids, p.n, p.G, p.S, p.bm_log2, tile);
  if (t.rows == 0) return;
  const int a = t.adapter;
  const bool z_out = p.z_out && chunk == 0;
  if (a < 0 && p.base == p.out && !z_out) return;  // these rows stay as they are

  const float sc = a >= 0 && p.scale ? p.scale[a] : 1.f;
  for (int i = threadIdx.x; i < 16 * RB * (RP / 4); i += kThreads) {  // 4 ranks of a row
    const int row = i / (RP / 4), rank = 4 * (i % (RP / 4));
    f32x4 v = f32x4{0.f, 0.f, 0.f, 0.f};
    if (row < t.rows && rank < p.r) {
      const int64_t at = (t.row0 + row) * p.r + rank;
      if (a >= 0) {
        const int64_t piece = int64_t(p.S) * p.r;
        for (int k0 = 0; k0 < p.ksplit; k0 += 4) {  // the pieces, four loads in flight (the last repeated)
          f32x4 o[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            o[k] = *reinterpret_cast<const f32x4*>(p.z + (k0 + k < p.ksplit ? k0 + k : p.ksplit - 1) * piece + at);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (k0 + k < p.ksplit) v += o[k];
        }
      }
      if (z_out) *reinterpret_cast<f32x4*>(p.z_out + at) = v;
    }
    X::put(zs + row * X::kStride, rank, v * sc);
  }
  __syncthreads();
  if (a < 0 && p.base == p.out) return;
  bf16x8 zf[RB][X::kSteps];
  X::template fragments<RB>(zs, zf);
  const int steps = int((p.C + X::kCols - 1) / X::kCols);
  const int end = (chunk + 1) * p.per < steps ? (chunk + 1) * p.per : steps;
  const typename X::out_t* base = static_cast<const typename X::out_t*>(p.base);
  const typename X::template Rows<RB> rows(base ? base + t.row0 * p.C : nullptr,
                                           static_cast<typename X::out_t*>(p.out) + t.row0 * p.C,
                                           p.w + int64_t(a < 0 ? 0 : a) * p.C * p.r, uint32_t(p.C), p.r, t.rows, a >= 0);
  constexpr int kAhead = X::ahead(RB);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int s = chunk * p.per + wave; s < end; s += kAhead * kWaves) {
    typename X::template Step<RB> st[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (i == 0 || s + i * kWaves < end) rows.load(s + i * kWaves, st[i]);
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (i == 0 || s + i * kWaves < end) rows.finish(s + i * kWaves, st[i], zf);
  }
}

struct FusedArgs {
  const uint16_t* x;      // [S, K]
  const uint16_t* a;      // [n, r, K]
  const uint16_t* b;      // [n, N, r]
  const float* scale;
  const int32_t* offsets;
  const int32_t* ids;
  const void* y;
  void* out;
  float* z;               // nullable
  int64_t K, N;
  int S, G, n, r;
  uint32_t chunks;
  int per;
};

// Waves of the one-launch form: 16, 8 where their units would not fit LDS.
constexpr int fused_waves(int rp) { return rp <= 32 ? 16 : 8; }

// Both products in one launch for tiles of at most 16 rows (decoded tokens): every workgroup of a
// tile computes the tile's z for itself, from all of x and the adapter's A, instead of waiting for
// another launch to do it.  A tile's workgroups have neighbouring ids and run on different XCDs, so
// each reads x and A through an L2 cache of its own: 64 tokens of 48 adapters fetch 50 MB from beyond
// them, where the inputs are at most 32 MB.
// Bound: that, and the chain of latencies (offsets, x and A, the waves' sums, B and y).  The kernel
// alone, traced: one token at [14336, 4096] and rank 16 7.9 us, 64 of 48 adapters (36 MB read and
// written) 14.1 us, 512 rows of 128 adapters at [1536, 2048] (23 MB) 9.8 us.
template <int RP, int ODT>
__global__ void __launch_bounds__(fused_waves(RP) * kWave) fused_kernel(FusedArgs p) {
  typedef Expand<RP, ODT> X;
  constexpr int RT = (RP + 15) / 16, kFusedWaves = fused_waves(RP);
  constexpr int kUnits = kFusedWaves * (1 + RT) * kUnitBytes, kSums = kFusedWaves * RT * kWave * 16;
  __shared__ __attribute__((aligned(16))) uint8_t lds[kUnits > kSums ? kUnits : kSums];
  f32x4 (*part)[RT][kWave] = reinterpret_cast<f32x4 (*)[RT][kWave]>(lds);
  __shared__ __attribute__((aligned(16))) uint16_t zs[16 * X::kStride];
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t tile = blockIdx.x / p.chunks;
  const int chunk = int(blockIdx.x - tile * p.chunks);
  const RowTile t = find_tile(p.offsets, p.ids, p.n, p.G, p.S, 4, tile);
  if (t.rows == 0) return;
  const int a = t.adapter;
  const bool z_out = p.z && chunk == 0;
  if (a < 0 && p.y == p.out && !z_out) return;
  const float sc = a >= 0 && p.scale ? p.scale[a] : 1.f;
  const int steps = int((p.N + X::kCols - 1) / X::kCols);
  const int end = (chunk + 1) * p.per < steps ? (chunk + 1) * p.per : steps;
  const typename X::out_t* y = static_cast<const typename X::out_t*>(p.y);
  const typename X::template Rows<1> rows(y ? y + t.row0 * p.N : nullptr,
                                          static_cast<typename X::out_t*>(p.out) + t.row0 * p.N,
                                          p.b + int64_t(a < 0 ? 0 : a) * p.N * p.r, uint32_t(p.N), p.r, t.rows, a >= 0);
  int s = chunk * p.per + wave;
  // The first step's loads go out before z is computed (two steps' made 64 tokens no faster, 15.3 us
  // and 15.4, and one token slower, 10.0 us and 8.0).
  typename X::template Step<1> st;
  if (s < end) rows.load(s, st);
  f32x4 acc[1][RT];
  zero_sums(acc);
  if (a >= 0) {
    shrink_sums<1, RT, RT <= 2 ? 2 : 1>(lds, p.x + t.row0 * p.K, p.a + int64_t(a) * p.r * p.K, uint32_t(p.K), p.r,
                                        t.rows, 0, int((p.K + 63) >> 6), kFusedWaves, acc);
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < RT; ++k) part[wave][k][lane] = acc[0][k];
  __syncthreads();
  if (wave < RT) {
    f32x4 v = part[0][wave][lane];
#pragma unroll
    for (int w = 1; w < kFusedWaves; ++w) v += part[w][wave][lane];
    const int row = lane & 15, rank = 16 * wave + 4 * (lane >> 4);
    if (rank >= p.r) v = f32x4{0.f, 0.f, 0.f, 0.f};  // repeated ranks
    if (z_out && row < t.rows && rank < p.r) *reinterpret_cast<f32x4*>(p.z + (t.row0 + row) * p.r + rank) = v;
    if (rank < RP) X::put(zs + row * X::kStride, rank, v * sc);
  }
  __syncthreads();
  if (a < 0 && p.y == p.out) return;
  bf16x8 zf[1][X::kSteps];
  X::template fragments<1>(zs, zf);
  while (s < end) {
    rows.finish(s, st, zf);
    s += kFusedWaves;
    if (s < end) rows.load(s, st);
  }
}

// A tile of the gradient pass: group g's rows cut evenly into ceil(rows / most) pieces of a multiple
// of 64 rows (the last ones may hold fewer, or none).
struct GradTile {
  int adapter, row0, rows;
  int kept;        // index among the tiles that write parts; -1: the group's only tile
  bool valid;
};

__device__ __forceinline__ int grad_tiles(int rows, int most) {
  return int((uint32_t(rows) + uint32_t(most) - 1u) / uint32_t(most));
}

// As find_tile.  `single`: a group of one tile is not counted among the kept ones.
__device__ __forceinline__ GradTile find_grad_tile(const int32_t* __restrict__ offsets, const int32_t* __restrict__ ids,
                                                   int n_adapters, int G, int S, int most, uint32_t tile,
                                                   bool single) {
  const int lane = threadIdx.x & (kWave - 1);
  int base = 0, kbase = 0;
  for (int g0 = 0; g0 < G; g0 += kWave) {
    int lo = 0, hi = 0, a = -1;
    if (g0 + lane < G) {
      group_rows(offsets, g0 + lane, S, &lo, &hi);
      a = adapter_of(ids, g0 + lane, n_adapters);
    }
    const int n = grad_tiles(hi - lo, most);
    const int k = single && n == 1 ? 0 : n;
    const int ni = wave_scan(n), ki = wave_scan(k);
    const int total = __builtin_amdgcn_readlane(ni, kWave - 1);
    if (int(tile) - base < total) {
      const int l = __ffsll((unsigned long long)__ballot(int(tile) - base < ni)) - 1;
      const int nl = __builtin_amdgcn_readlane(n, l), lol = __builtin_amdgcn_readlane(lo, l);
      const int rows = __builtin_amdgcn_readlane(hi, l) - lol;
      const int at = int(tile) - base - (__builtin_amdgcn_readlane(ni, l) - nl);
      if (at < 0 || at >= nl) break;  // as above
      const int per = (grad_tiles(rows, nl) + 63) & ~63;
      const int64_t first = int64_t(at) * per;
      GradTile t;
      t.adapter = __builtin_amdgcn_readlane(a, l);
      t.rows = int(rows - first < 0 ? 0 : (rows - first < per ? rows - first : per));
      t.row0 = lol + (t.rows > 0 ? int(first) : 0);
      t.kept = single && nl == 1 ? -1 : kbase + __builtin_amdgcn_readlane(ki - k, l) + at;
      t.valid = true;
      return t;
    }
    base += total;
    kbase += __builtin_amdgcn_readlane(ki, kWave - 1);
  }
  return GradTile{-1, 0, 0, 0, false};
}

struct GradArgs {
  const float* v;         // [S, r]: z or u (read for grad)
  const uint16_t* m;      // [S, C]: g or x
  const uint16_t* w;      // [n, C, r]: B, for u
  const float* scale;     // nullable: 1; of grad and of u
  const int32_t* offsets;
  const int32_t* ids;
  float* grad;            // nullable [n, r, C], or [n, C, r] (BYCOL)
  float* parts;           // [parts_cap][r, C] (or [C, r])
  float* upart;           // nullable [chunks, S, r]: scale * m B, summed over a chunk's columns
  int64_t parts_cap;      // parts there is room for (offsets that are not ascending ask for more)
  uint32_t C;
  int S, G, n, r, most;
  uint32_t chunks;
};

constexpr int kGradRows = 64, kGradCols = 256;  // a block in LDS: 64 rows of 512 bytes

// LDS byte of the 16-byte piece `piece` of row `row` of a block.  Rows are 512 bytes; the 32-byte
// units of a row and the halves of a unit are exchanged by the row so that the 16-byte reads of 16
// rows and the transposing reads (4 rows by 32 bytes for each 16 lanes) spread over all 64 banks.
__device__ __forceinline__ uint32_t block_at(int row, int piece) {
  const uint32_t f = (row & 3) | ((row >> 1) & 4), h = (row >> 2) & 1;
  return 512u * row + ((uint32_t(piece >> 1) ^ f) * 32u) + ((uint32_t(piece & 1) ^ h) * 16u);
}

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

// Transposing LDS read: the 16 lanes of a group give the addresses of 4 rows by 16 columns (lane i:
// row i / 4, columns 4 (i % 4) .. + 3); lane i gets column i of the 4 rows.
__device__ __forceinline__ s16x4 lds_read_tr(const uint8_t* at) {
#if defined(__HIP_DEVICE_COMPILE__)
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)at);
#else
  return s16x4{};
#endif
}

// One pass over m for both products it enters: grad = v^T m over the tile's rows, and (with UP)
// u = m B over a chunk's columns.  A workgroup takes the rows of one tile and 256 * NSUB columns, in
// blocks of 64 rows by 256 columns that come in whole lines through registers (the next block's
// loads in flight) into LDS.  grad: a wave has 64 of the block's columns; the contraction runs over
// the rows, so m is read transposed, and v stands in LDS transposed in its three parts.  u: a wave
// has 16 of the block's rows and all its columns; B stands in LDS transposed.
// Bound: HBM in long groups: g of 8192 rows of 28672 at rank 16 (470 MB) takes 117 us, 4.0 TB/s (4.2
// with u's partial sums).  32 groups of 128 .. 384 rows of 2880 at rank 32 (47 MB) take 25 us: one
// round of workgroups that ends with the longest group, four or five blocks one after the other.
// One pass instead of two reads m once: 8192 rows of 28672 took 387 us for all gradients with a pass
// each for u and grad (and float32 matrix instructions), 191 so.
template <int RT, int NSUB, bool UP, bool BYCOL>
__global__ void __launch_bounds__(kThreads) grad_kernel(GradArgs p) {
  constexpr int kVStride = kGradRows + 8;               // v^T row in bf16
  constexpr int kWCols = kGradCols * NSUB, kWStride = kWCols + 8;
  constexpr uint32_t kBlock = kGradRows * kGradCols * 2;
  constexpr uint32_t kV = 3 * 16 * RT * kVStride * 2;
  __shared__ __attribute__((aligned(16))) uint8_t lds[kBlock + kV + (UP ? 16 * RT * kWStride * 2 : 0)];
  uint16_t* vt = reinterpret_cast<uint16_t*>(lds + kBlock);          // [3][16 RT][kVStride]
  uint16_t* wt = reinterpret_cast<uint16_t*>(lds + kBlock + kV);     // [16 RT][kWStride]
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 15, q = lane >> 4;
  const uint32_t tile = blockIdx.x / p.chunks;
  const int chunk = int(blockIdx.x - tile * p.chunks);
  const GradTile t = find_grad_tile(p.offsets, p.ids, p.n, p.G, p.S, p.most, tile, p.ids == nullptr);
  if (!t.valid) return;
  const int a = t.adapter;
  if (a < 0) return;
  const uint32_t col0 = uint32_t(chunk) * kWCols;
  const bool grad = p.grad != nullptr;
  const float sc = p.scale ? p.scale[a] : 1.f;

  f32x4 acc[NSUB][4][RT];
#pragma unroll
  for (int s = 0; s < NSUB; ++s) zero_sums(acc[s]);

  // The block's loads: thread i of row i / 32 takes piece i % 32 of every 8th row.  Offsets are
  // taken from the block's first row, so they stay small however long the tile is.
  const int prow = tid >> 5, piece = tid & 31;
  auto load_block = [&](int row, int sub, u32x4 (&v)[8]) {
    const uint16_t* at = p.m + (int64_t(t.row0) + row) * p.C;
    const int left = t.rows - row;
    const __amdgpu_buffer_rsrc_t res =
        wave_rsrc(at, left > 0 ? uint32_t(left < kGradRows ? left : kGradRows) * p.C * 2u : 0u);
    const uint32_t col = col0 + kGradCols * sub + 8 * piece;
#pragma unroll
    for (int j = 0; j < 8; ++j)  // read once, past the caches (gate_up gradients 199 us kept, 190 so)
      v[j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                           res, col < p.C ? (prow * p.C + col) * 2u : kNowhere, 16u * j * p.C,
                                           kPastCaches));
  };
  // v of a block: two rows of one rank a thread and turn.
  constexpr int kVTurns = kGradRows / 2 * 16 * RT / kThreads;
  auto load_v = [&](int row, float (&v)[kVTurns][2]) {
    const int left = t.rows - row;
    const __amdgpu_buffer_rsrc_t res =
        wave_rsrc(p.v + (int64_t(t.row0) + row) * p.r, grad && left > 0 ? uint32_t(left < kGradRows ? left : kGradRows) * p.r * 4u : 0u);
#pragma unroll
    for (int j = 0; j < kVTurns; ++j) {
      const int i = tid + j * kThreads, rank = i % (16 * RT), pair = i / (16 * RT);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        v[j][h] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
            res, rank < p.r ? uint32_t(((2 * pair + h) * p.r + rank) * 4) : kNowhere, 0, 0));
    }
  };

  // Fragments of a block.  m transposed: columns 64 wave + 16 ct + c, rows 32 ks + 8 q .. + 7.
  auto m_columns = [&](int ks, int ct) {
    s16x8 mt;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r4 = 32 * ks + 8 * q + 4 * h + (c >> 2), u = 4 * wave + ct;
      const s16x4 x = lds_read_tr(lds + block_at(r4, 2 * u + ((c >> 1) & 1)) + 8 * (c & 1));
#pragma unroll
      for (int j = 0; j < 4; ++j) mt[4 * h + j] = x[j];
    }
    return __builtin_bit_cast(bf16x8, mt);
  };
  auto v_ranks = [&](int ks, int k, int h) {
    return *reinterpret_cast<const bf16x8*>(vt + (16 * RT * h + 16 * k + c) * kVStride + 32 * ks + 8 * q);
  };
  auto m_rows = [&](int s) {
    return *reinterpret_cast<const bf16x8*>(lds + block_at(16 * wave + c, 4 * s + q));
  };
  auto w_ranks = [&](int sub, int s, int k) {
    return *reinterpret_cast<const bf16x8*>(wt + (16 * k + c) * kWStride + kGradCols * sub + 32 * s + 8 * q);
  };
  constexpr int kUSteps = RT <= 2 ? 4 : (RT == 4 ? 2 : 1);  // steps of u whose fragments are read together

  u32x4 mv[8];
  float vv[kVTurns][2];
  load_v(0, vv);
  load_block(0, 0, mv);
  if (UP) {  // B^T of the chunk: 8 ranks of a column a thread and turn
    const int per = p.r >> 3;
    for (int i = tid; i < kWCols * per; i += kThreads) {
      const int n = i / per, k = 8 * (i - n * per);
      u32x4 b = u32x4{0u, 0u, 0u, 0u};
      if (col0 + n < p.C) b = *reinterpret_cast<const u32x4*>(p.w + (int64_t(a) * p.C + col0 + n) * p.r + k);
#pragma unroll
      for (int j = 0; j < 8; ++j) wt[(k + j) * kWStride + n] = uint16_t(j & 1 ? b[j >> 1] >> 16 : b[j >> 1] & 0xFFFFu);
    }
  }

  f32x4 us[RT];
#pragma unroll
  for (int k = 0; k < RT; ++k) us[k] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int row = 0; row < t.rows; row += kGradRows) {
#pragma unroll
    for (int sub = 0; sub < NSUB; ++sub) {
      __syncthreads();  // the last block has been read
#pragma unroll
      for (int j = 0; j < 8; ++j) *reinterpret_cast<u32x4*>(lds + block_at(prow + 8 * j, piece)) = mv[j];
      if (sub == 0 && grad) {
#pragma unroll
        for (int j = 0; j < kVTurns; ++j) {
          const int e = tid + j * kThreads, rank = e % (16 * RT), pair = e / (16 * RT);
          const Parts x = split3(vv[j][0]), y = split3(vv[j][1]);
          uint32_t* at = reinterpret_cast<uint32_t*>(vt + rank * kVStride) + pair;
          at[0] = hi2(x.hi, y.hi);
          at[16 * RT * kVStride / 2] = hi2(x.mid, y.mid);
          at[2 * (16 * RT * kVStride / 2)] = hi2(x.lo, y.lo);
        }
      }
      __syncthreads();
      if (sub + 1 < NSUB) {
        load_block(row, sub + 1, mv);
      } else {  // past the tile: zeros, unused
        load_v(row + kGradRows, vv);
        load_block(row + kGradRows, 0, mv);
      }
      // Fragments are read from LDS a group ahead of the products that use them: two waves a SIMD do
      // not hide the reads' latency (read where used, a block took twice as long).
      bf16x8 um[kUSteps], uw[kUSteps][RT];
      auto read_u = [&](int s0) {
#pragma unroll
        for (int s = 0; s < kUSteps; ++s) {
          um[s] = m_rows(s0 + s);
#pragma unroll
          for (int k = 0; k < RT; ++k) uw[s][k] = w_ranks(sub, s0 + s, k);
        }
      };
      if (grad) {
        bf16x8 mf[2][4];
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
          for (int ct = 0; ct < 4; ++ct) mf[ks][ct] = m_columns(ks, ct);
        bf16x8 vf[3], vn[3];
#pragma unroll
        for (int h = 0; h < 3; ++h) vf[h] = v_ranks(0, 0, h);
#pragma unroll
        for (int g = 0; g < 2 * RT; ++g) {  // (ks, rank tile) in turn, the next one's v in flight
          const int ks = g / RT, k = g % RT;
          if (g + 1 < 2 * RT) {
#pragma unroll
            for (int h = 0; h < 3; ++h) vn[h] = v_ranks((g + 1) / RT, (g + 1) % RT, h);
          } else if (UP) {
            read_u(0);
          }
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int h = 0; h < 3; ++h)
#pragma unroll
            for (int ct = 0; ct < 4; ++ct)
              acc[sub][ct][k] = BYCOL ? __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf[h], mf[ks][ct], acc[sub][ct][k], 0, 0, 0)
                                      : __builtin_amdgcn_mfma_f32_16x16x32_bf16(mf[ks][ct], vf[h], acc[sub][ct][k], 0, 0, 0);
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int h = 0; h < 3; ++h) vf[h] = vn[h];
        }
      } else if (UP) {
        read_u(0);
      }
      if (UP) {
#pragma unroll
        for (int s0 = 0; s0 < kGradCols / 32; s0 += kUSteps) {
          bf16x8 m0[kUSteps], w0[kUSteps][RT];
#pragma unroll
          for (int s = 0; s < kUSteps; ++s) {
            m0[s] = um[s];
#pragma unroll
            for (int k = 0; k < RT; ++k) w0[s][k] = uw[s][k];
          }
          if (s0 + kUSteps < kGradCols / 32) read_u(s0 + kUSteps);
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int s = 0; s < kUSteps; ++s)
#pragma unroll
            for (int k = 0; k < RT; ++k) us[k] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w0[s][k], m0[s], us[k], 0, 0, 0);
          __builtin_amdgcn_sched_barrier(0);
        }
        if (sub == NSUB - 1) {
          const int at = row + 16 * wave + c;
#pragma unroll
          for (int k = 0; k < RT; ++k) {
            const int rank = 16 * k + 4 * q;
            if (at < t.rows && rank < p.r)
              *reinterpret_cast<f32x4*>(p.upart + (int64_t(chunk) * p.S + t.row0 + at) * p.r + rank) = us[k] * sc;
            us[k] = f32x4{0.f, 0.f, 0.f, 0.f};
          }
        }
      }
    }
  }
  if (!grad || t.kept >= p.parts_cap) return;
  float* dst = t.kept < 0 ? p.grad + int64_t(a) * p.r * p.C : p.parts + int64_t(t.kept) * p.r * p.C;
#pragma unroll
  for (int sub = 0; sub < NSUB; ++sub)
#pragma unroll
    for (int ct = 0; ct < 4; ++ct)
#pragma unroll
      for (int k = 0; k < RT; ++k) {
        const uint32_t cc = col0 + kGradCols * sub + 64 * wave + 16 * ct;
        if (BYCOL) {
          const int rank = 16 * k + 4 * q;
          if (cc + c < p.C && rank < p.r)
            *reinterpret_cast<f32x4*>(dst + int64_t(cc + c) * p.r + rank) = acc[sub][ct][k] * sc;
        } else {
          const int rank = 16 * k + c;
          if (cc + 4 * q < p.C && rank < p.r)
            *reinterpret_cast<f32x4*>(dst + int64_t(rank) * p.C + cc + 4 * q) = acc[sub][ct][k] * sc;
        }
      }
}

// One gradient's parts.
struct ReducePart {
  const float* parts;     // [parts_cap, len]
  float* grad;            // [n, len]
  int64_t len, parts_cap;
  int most;
  uint32_t chunks;        // workgroups an adapter has
};
struct ReduceArgs {
  ReducePart of[2];
  uint32_t first;         // workgroups of of[0]
  const int32_t* offsets;
  const int32_t* ids;
  int S, G, n;
};
constexpr int kReduceTurns = 8, kReduceLen = 4 * kThreads * kReduceTurns;

// grad[a] = the sum of the parts of a's groups in order (0 without rows); a group of one tile
// under ids == NULL has written its adapter's gradient itself.  Bound: the launch behind the passes'
// writes; both gradients in one launch take 5.5 us at 8 adapters of rank 16, [28672, 4096].
__global__ void __launch_bounds__(kThreads) grad_reduce_kernel(ReduceArgs p) {
  const int lane = threadIdx.x & (kWave - 1);
  const bool second = blockIdx.x >= p.first;
  const ReducePart& t = p.of[second ? 1 : 0];
  const uint32_t block = second ? blockIdx.x - p.first : blockIdx.x;
  const int a = int(block / t.chunks);
  const int64_t e0 = int64_t(block - a * t.chunks) * kReduceLen + 4 * threadIdx.x;
  const bool single = p.ids == nullptr;
  f32x4 sum[kReduceTurns];
#pragma unroll
  for (int j = 0; j < kReduceTurns; ++j) sum[j] = f32x4{0.f, 0.f, 0.f, 0.f};
  int kbase = 0;
  for (int g0 = 0; g0 < p.G; g0 += kWave) {
    int lo = 0, hi = 0, id = -1;
    if (g0 + lane < p.G) {
      group_rows(p.offsets, g0 + lane, p.S, &lo, &hi);
      id = adapter_of(p.ids, g0 + lane, p.n);
    }
    const int n = grad_tiles(hi - lo, t.most);
    const int k = single && n == 1 ? 0 : n;
    const int ki = wave_scan(k);
    if (single && a >= g0 && a < g0 + kWave && __builtin_amdgcn_readlane(n, a - g0) == 1) return;
    uint64_t mine = __ballot(id == a && k > 0);
    while (mine) {
      const int l = __ffsll((unsigned long long)mine) - 1;
      mine &= mine - 1;
      const int64_t first = kbase + __builtin_amdgcn_readlane(ki - k, l);
      int64_t cnt = first < 0 ? 0 : __builtin_amdgcn_readlane(k, l);
      if (cnt > t.parts_cap - first) cnt = t.parts_cap - first;
      for (int64_t i = 0; i < cnt; ++i) {
        const float* src = t.parts + (first + i) * t.len;
        f32x4 v[kReduceTurns];
#pragma unroll
        for (int j = 0; j < kReduceTurns; ++j) {
          const int64_t e = e0 + 4 * kThreads * j;
          v[j] = *reinterpret_cast<const f32x4*>(src + (e < t.len ? e : 0));
        }
#pragma unroll
        for (int j = 0; j < kReduceTurns; ++j) sum[j] += v[j];
      }
    }
    kbase += __builtin_amdgcn_readlane(ki, kWave - 1);
  }
#pragma unroll
  for (int j = 0; j < kReduceTurns; ++j) {
    const int64_t e = e0 + 4 * kThreads * j;
    if (e < t.len) *reinterpret_cast<f32x4*>(t.grad + int64_t(a) * t.len + e) = sum[j];
  }
}

// Between the gradient pass and what uses u: u[p] = the sum of its chunks in a fixed order (16 lanes
// have 4 ranks each, the wave's four groups of 16 a quarter of the chunks each; rows of no adapter
// hold garbage here and there, and nothing reads them), and A^T [n, K, r] for the expand (a thread
// has 8 ranks of 8 columns).  Bound: the launch and one round of loads behind the pass's writes: 8 us
// for 56 chunks of 8192 rows at rank 16 (29 MB), 9 for 12 chunks at rank 32 and 6 MB of A.
struct BetweenArgs {
  const float* upart;     // [chunks, S, r]
  float* u;               // [S, r]
  const uint16_t* a;      // [n, r, K]
  uint16_t* at;           // nullable [n, K, r]
  int64_t len;            // S * r
  uint32_t u_blocks;
  int n, r, chunks, K;
};
__device__ __forceinline__ void sum_u(const BetweenArgs& p, int64_t wave) {
  const int lane = threadIdx.x & (kWave - 1);
  const int64_t e = 4 * (16 * wave + (lane & 15)), at = e < p.len ? e : 0;
  f32x4 sum = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int k0 = lane >> 4; k0 < p.chunks; k0 += 32) {  // eight loads in flight (past the last: the last again)
    f32x4 o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      o[j] = *reinterpret_cast<const f32x4*>(p.upart + (k0 + 4 * j < p.chunks ? k0 + 4 * j : p.chunks - 1) * p.len + at);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (k0 + 4 * j < p.chunks) sum += o[j];
  }
#pragma unroll
  for (int m = 16; m < kWave; m <<= 1)
#pragma unroll
    for (int j = 0; j < 4; ++j) sum[j] += __shfl_xor(sum[j], m, kWave);
  if (lane < 16 && e < p.len) *reinterpret_cast<f32x4*>(p.u + e) = sum;
}
__global__ void __launch_bounds__(kThreads) between_kernel(BetweenArgs p) {
  if (blockIdx.x < p.u_blocks) {
    sum_u(p, int64_t(blockIdx.x) * kWaves + (threadIdx.x >> 6));
    return;
  }
  const int64_t i = int64_t(blockIdx.x - p.u_blocks) * kThreads + threadIdx.x;
  const int cols = p.K >> 3, ranks = p.r >> 3;
  if (i >= int64_t(p.n) * ranks * cols) return;
  const int64_t col = i % cols, j = i / cols, rank = j % ranks, a = j / ranks;
  const uint16_t* src = p.a + ((a * p.r + 8 * rank) * p.K + 8 * col);
  u32x4 v[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = *reinterpret_cast<const u32x4*>(src + int64_t(k) * p.K);
  uint16_t* dst = p.at + ((a * p.K + 8 * col) * p.r + 8 * rank);
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    u32x4 o;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      o[k] = perm(v[2 * k + 1][c >> 1], v[2 * k][c >> 1], c & 1 ? 0x07060302u : 0x05040100u);
    *reinterpret_cast<u32x4*>(dst + int64_t(c) * p.r) = o;
  }
}

int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Row tiles of 1 << bm_log2 rows that G groups of S rows can need.
int64_t tiles_bound(int64_t S, int64_t G, int bm_log2) {
  const int64_t used = G < S ? G : S;
  return (S + used * ((int64_t(1) << bm_log2) - 1)) >> bm_log2;
}

int log2_up(int64_t v) {
  int l = 0;
  while ((int64_t(1) << l) < v) ++l;
  return l;
}

// Rows of a shrink or expand tile: 16 where groups average no more (decoded tokens), else 64, or
// 32 at ranks over 64, whose parts fill the registers.  64 groups at [2048, 2048], rank 64, us with
// 16-row and with 64-row tiles: 14 rows a group 16.4 and 19.6, 20 rows 22.7 and 21.4; 32 groups at
// [4096, 4096], rank 16: 14 rows 11.7 and 12.4, 20 rows 13.9 and 13.4, 32 rows 17.6 and 15.1.
int row_tile_log2(int64_t S, int64_t G, int r) { return S <= 16 * G ? 4 : (r > 64 ? 5 : 6); }

// Rows of a shrink tile: 32 from rank 33 on, where the sums and fragments of 64 rows leave room for
// one workgroup a CU.
int shrink_tile_log2(const LoraGroups& q) {
  const int l = row_tile_log2(q.S, q.G, q.r);
  return q.r > 32 && l > 5 ? 5 : l;
}

// Pieces the columns of a shrink are cut into: as many workgroups as are resident together up to rank
// 64 (three on every CU; 24 prompts of rank 64: 31 us a call, 37 with a third more), no piece under 512
// columns (two units for each wave).  Above rank 64 two are resident, and three are still wanted: with
// 768 and with 512, us a call at rank 128, 24 prompts at [2880, 2880] 55 and 59, 2048 rows of 8 experts
// at [4096, 4096] 39 and 46, but 8192 rows at [4096, 14336] 157 and 148.
int shrink_pieces(const LoraGroups& q, int64_t C) {
  const int64_t tiles = tiles_bound(q.S, q.G, shrink_tile_log2(q));
  const int64_t want = 768 / (tiles > 0 ? tiles : 1), most = C / 512;
  const int64_t k = want < most ? want : most;
  return int(k < 1 ? 1 : (k > 16 ? 16 : k));
}

// Column blocks of 256 a workgroup of the gradient pass takes: with u more, so that u's partial
// sums (r float32 for each row and workgroup) stay few beside m; as many as the registers hold.
int grad_subs(int r, bool up) { return up && r <= 16 ? 2 : 1; }

// Rows of a gradient tile at most: as many tiles as give every CU two workgroups (a tile costs a
// float32 write and read of its [r, C] sums).  Up to rank 32 that is one resident round.  Above, a CU
// holds one workgroup and it is two; with 512 and with 256 workgroups, us a call at ranks 64 and 128, 32
// experts at [2880, 2880] 128 / 285 and 131 / 286, 8 experts at [14336, 4096] 235 / 585 and 225 / 567,
// half of 16384 rows in one of 64 groups at rank 64 257 and 271.  Gradients of 32 experts at [2880, 2880] and of 8 at
// [28672, 4096]: 96 and 191 us; with half as many tiles again 111 and 198, with three quarters as many
// 95 and 193.  Each group's rest is about half a tile, and is taken off the tiles that are wanted, but
// no more than half of them: where many groups share the rows, one that has most of them still has to
// be cut (16384 rows in 128 groups at [2048, 2048], rank 32: 126 us, and with half the rows in one group
// 138; 499 where the groups' rests took all and that group was a single tile).
int grad_rows(const LoraGroups& q, int64_t C, bool up) {
  const int64_t chunks = div_up(C, kGradCols * grad_subs(q.r, up));
  const int64_t used = q.G < q.S ? q.G : q.S;
  const int64_t round = 512 / chunks;
  int64_t tiles = round - (used < round ? used / 2 : round / 2);
  if (tiles < 1) tiles = 1;
  int64_t most = (div_up(q.S, tiles) + 63) / 64 * 64;
  return int(most < 128 ? 128 : (most > (1 << 20) ? 1 << 20 : most));
}
int64_t grad_tiles_bound(const LoraGroups& q, int most) {
  const int64_t used = q.G < q.S ? q.G : q.S;
  return (q.S + used * (most - 1)) / most;
}

// Tiles that write parts: all where adapters are shared by groups; without ids only those of
// groups of several tiles, at most two for each `most` rows.  With ids that is a float32 [r, C] for every
// group that has rows, written and read again, whether its adapter has other groups or not: 8192 rows in
// 1024 groups at rank 64, [14336, 4096], ask for 5 GB.
int64_t parts_bound(const LoraGroups& q, int most) {
  const int64_t all = grad_tiles_bound(q, most), kept = 2 * q.S / most;
  return q.ids || all < kept ? all : kept;
}

// 32-row tiles are for ranks over 32, 64-row tiles for the others.
template <int RB>
void shrink_rb(const ShrinkArgs& a, dim3 grid, hipStream_t s) {
  if constexpr (RB != 2) {
    if (a.r <= 16) hipLaunchKernelGGL((shrink_kernel<RB, 1>), grid, dim3(kThreads), 0, s, a);
    else if (a.r <= 32) hipLaunchKernelGGL((shrink_kernel<RB, 2>), grid, dim3(kThreads), 0, s, a);
  }
  if constexpr (RB != 4) {
    if (a.r > 64) hipLaunchKernelGGL((shrink_kernel<RB, 8>), grid, dim3(kThreads), 0, s, a);
    else if (a.r > 32) hipLaunchKernelGGL((shrink_kernel<RB, 4>), grid, dim3(kThreads), 0, s, a);
  }
}

hipError_t shrink(const LoraGroups& q, const uint16_t* m, const uint16_t* w, const float* scale, int64_t C, float* z,
                  int pieces, hipStream_t s) {
  const int bm = shrink_tile_log2(q);
  ShrinkArgs a{m, w, scale, q.offsets, q.ids, z, C, int(q.S), int(q.G), int(q.n), q.r, bm, uint32_t(pieces), 0};
  a.per = int(div_up(div_up(C, 64), pieces));
  const dim3 grid(unsigned(tiles_bound(q.S, q.G, bm) * pieces));
  if (grid.x == 0) return hipSuccess;
  if (a.bm_log2 == 4) shrink_rb<1>(a, grid, s);
  else if (a.bm_log2 == 5) shrink_rb<2>(a, grid, s);
  else shrink_rb<4>(a, grid, s);
  return hipGetLastError();
}

// 32-row tiles are for ranks over 64, 64-row tiles for the others.
template <int RB, int ODT>
void expand_rb(const ExpandArgs& a, dim3 grid, hipStream_t s) {
  if constexpr (RB != 2) {
    if (a.r <= 8) hipLaunchKernelGGL((expand_kernel<RB, 8, ODT>), grid, dim3(kThreads), 0, s, a);
    else if (a.r <= 16) hipLaunchKernelGGL((expand_kernel<RB, 16, ODT>), grid, dim3(kThreads), 0, s, a);
    else if (a.r <= 32) hipLaunchKernelGGL((expand_kernel<RB, 32, ODT>), grid, dim3(kThreads), 0, s, a);
    else if (a.r <= 64) hipLaunchKernelGGL((expand_kernel<RB, 64, ODT>), grid, dim3(kThreads), 0, s, a);
  }
  if constexpr (RB != 4)
    if (a.r > 64) hipLaunchKernelGGL((expand_kernel<RB, 128, ODT>), grid, dim3(kThreads), 0, s, a);
}

template <int ODT>
void expand_dt(const ExpandArgs& a, dim3 grid, hipStream_t s) {
  if (a.bm_log2 == 4) expand_rb<1, ODT>(a, grid, s);
  else if (a.bm_log2 == 5) expand_rb<2, ODT>(a, grid, s);
  else expand_rb<4, ODT>(a, grid, s);
}

// Pieces the columns of an expand are cut into, by the workgroups wanted, a step for each wave at
// least.  From rank 33 on the parts of a tile's z are worth keeping for as many columns as one
// resident round leaves (rank 64, 24 prompts: 21 us, 26 with twice the workgroups or more); below,
// ten workgroups a CU, most of a step or two a wave, keep the memory busy to the end (gx of the
// 32-expert layer: 39 us, 42 with four, 52 with less than two).
int expand_chunks(int64_t tiles, int64_t C, int waves, int wanted) {
  const int64_t most = div_up(div_up(C, 64), waves), want = wanted / (tiles > 0 ? tiles : 1);
  return int(want < 1 ? 1 : (want < most ? want : most));
}

int expand_wanted(int r) { return r > 32 ? 512 : 2560; }
constexpr int kFusedWanted = 256;

hipError_t expand(const LoraGroups& q, const float* z, int pieces, const uint16_t* w, const float* scale, int64_t C,
                  const void* base, void* out, int odt, float* z_out, hipStream_t s) {
  const int bm = row_tile_log2(q.S, q.G, q.r);
  const int64_t tiles = tiles_bound(q.S, q.G, bm);
  const int chunks = expand_chunks(tiles, C, kWaves, expand_wanted(q.r));
  ExpandArgs a{z, w, scale, q.offsets, q.ids, base, out, z_out, C, int(q.S), int(q.G), int(q.n), q.r, bm, pieces,
               uint32_t(chunks), int(div_up(div_up(C, 64), chunks))};
  const dim3 grid(unsigned(tiles * chunks));
  if (grid.x == 0) return hipSuccess;
  if (odt == 0) expand_dt<0>(a, grid, s);
  else expand_dt<1>(a, grid, s);
  return hipGetLastError();
}

template <bool UP, bool BYCOL>
void grad_rt(const GradArgs& a, unsigned grid, hipStream_t s) {
  if (a.r <= 16) hipLaunchKernelGGL((grad_kernel<1, UP ? 2 : 1, UP, BYCOL>), dim3(grid), dim3(kThreads), 0, s, a);
  else if (a.r <= 32) hipLaunchKernelGGL((grad_kernel<2, 1, UP, BYCOL>), dim3(grid), dim3(kThreads), 0, s, a);
  else if (a.r <= 64) hipLaunchKernelGGL((grad_kernel<4, 1, UP, BYCOL>), dim3(grid), dim3(kThreads), 0, s, a);
  else hipLaunchKernelGGL((grad_kernel<8, 1, UP, BYCOL>), dim3(grid), dim3(kThreads), 0, s, a);
}

// The gradient pass over m: grad (nullable) from v, and with upart also u.
hipError_t grad_pass(const LoraGroups& q, const float* v, const uint16_t* m, const uint16_t* w, const float* scale,
                     int64_t C, bool by_column, float* grad, float* parts, float* upart, hipStream_t s) {
  const bool up = upart != nullptr;
  GradArgs a{};
  a.v = v;
  a.m = m;
  a.w = w;
  a.scale = scale;
  a.offsets = q.offsets;
  a.ids = q.ids;
  a.grad = grad;
  a.parts = parts;
  a.upart = upart;
  a.C = uint32_t(C);
  a.S = int(q.S);
  a.G = int(q.G);
  a.n = int(q.n);
  a.r = q.r;
  a.most = grad_rows(q, C, up);
  a.parts_cap = parts_bound(q, a.most);
  a.chunks = uint32_t(div_up(C, kGradCols * grad_subs(q.r, up)));
  const unsigned grid = unsigned(grad_tiles_bound(q, a.most) * a.chunks);
  if (grid) {
    if (up) grad_rt<true, true>(a, grid, s);
    else if (by_column) grad_rt<false, true>(a, grid, s);
    else grad_rt<false, false>(a, grid, s);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Adds the sums over grad's parts to a reduce launch.
void reduce_of(const LoraGroups& q, int64_t C, bool up, float* grad, const float* parts, ReducePart* t) {
  t->parts = parts;
  t->grad = grad;
  t->len = q.r * C;
  t->most = grad_rows(q, C, up);
  t->parts_cap = parts_bound(q, t->most);
  t->chunks = uint32_t(div_up(t->len, kReduceLen));
}

// Workgroups of the launch between the passes: those that sum u, and those that transpose A.
int64_t between_u_blocks(const LoraGroups& q) { return div_up(q.S * (q.r / 4), 16 * kWaves); }
int64_t between_at_blocks(const LoraGroups& q) { return div_up(q.n * (q.r / 8) * (q.K / 8), kThreads); }

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

// Workspace of a backward call.
struct BackwardLayout {
  size_t u, upart, at, parts_a, parts_b, total;
};
BackwardLayout backward_layout(const LoraBackwardLaunch& L) {
  const LoraGroups& q = L.q;
  BackwardLayout w{};
  const bool need_u = L.gx || L.ga;
  size_t off = 0;
  w.u = off;
  if (need_u) off += align256(size_t(q.S) * q.r * 4);
  w.upart = off;
  if (need_u) off += align256(size_t(div_up(q.N, kGradCols * grad_subs(q.r, true))) * q.S * q.r * 4);
  w.at = off;
  if (L.gx) off += align256(size_t(q.n) * q.r * q.K * 2);
  w.parts_a = off;
  if (L.ga) off += align256(size_t(parts_bound(q, grad_rows(q, q.K, false))) * q.r * q.K * 4);
  w.parts_b = off;
  if (L.gb) off += align256(size_t(parts_bound(q, grad_rows(q, q.N, need_u))) * q.r * q.N * 4);
  w.total = off;
  return w;
}

}  // namespace

// Whether the forward call runs as one launch: tiles of at most 16 rows, and an A that every workgroup
// of a tile reads in a few microseconds, about what the second launch would cost.  us in one launch
// and in two: 64 tokens of 48 adapters at r K = 65536 14.8 and 20.7, at 131072 20.7 and 24.1, at 262144
// 22.6 and 15.9 (one token: 7.5 and 6.9, where a second launch costs the host 3; 12.5 and 8.2).
bool lora_fused(const LoraGroups& q) {
  return row_tile_log2(q.S, q.G, q.r) == 4 && q.r <= 64 && int64_t(q.r) * q.K <= (1 << 17);
}

size_t lora_ws_bytes(const LoraLaunch& L) {
  const LoraGroups& q = L.q;
  if (lora_fused(q)) return 0;
  return align256(size_t(shrink_pieces(q, q.K)) * q.S * q.r * 4);
}

size_t lora_backward_ws_bytes(const LoraBackwardLaunch& L) { return backward_layout(L).total; }

// Work items of the largest grid a call starts.
int64_t expand_blocks(const LoraGroups& q, int64_t C) {
  const int64_t tiles = tiles_bound(q.S, q.G, row_tile_log2(q.S, q.G, q.r));
  return tiles * expand_chunks(tiles, C, kWaves, expand_wanted(q.r));
}
int64_t lora_items(const LoraLaunch& L) {
  const LoraGroups& q = L.q;
  if (lora_fused(q)) {
    const int64_t tiles = tiles_bound(q.S, q.G, 4);
    return tiles * expand_chunks(tiles, q.N, fused_waves(q.r), kFusedWanted) * fused_waves(q.r) * kWave;
  }
  const int64_t shrink = tiles_bound(q.S, q.G, shrink_tile_log2(q)) * shrink_pieces(q, q.K);
  const int64_t expand = expand_blocks(q, q.N);
  return (shrink > expand ? shrink : expand) * kThreads;
}
int64_t lora_backward_items(const LoraBackwardLaunch& L) {
  const LoraGroups& q = L.q;
  const bool need_u = L.gx || L.ga;
  const auto pass = [&](int64_t C, bool up) {
    return grad_tiles_bound(q, grad_rows(q, C, up)) * div_up(C, kGradCols * grad_subs(q.r, up));
  };
  const auto sums = [&](int64_t C) { return q.n * div_up(q.r * C, kReduceLen); };
  const int64_t blocks[] = {pass(q.N, need_u), L.ga ? pass(q.K, false) : 0, L.gx ? expand_blocks(q, q.K) : 0,
                            need_u ? between_u_blocks(q) + (L.gx ? between_at_blocks(q) : 0) : 0,
                            (L.gb ? sums(q.N) : 0) + (L.ga ? sums(q.K) : 0)};
  int64_t most = 0;
  for (int64_t v : blocks) most = v > most ? v : most;
  return most * kThreads;
}

template <int ODT>
void fused_dt(const FusedArgs& a, dim3 grid, hipStream_t s) {
  if (a.r <= 8) hipLaunchKernelGGL((fused_kernel<8, ODT>), grid, dim3(fused_waves(8) * kWave), 0, s, a);
  else if (a.r <= 16) hipLaunchKernelGGL((fused_kernel<16, ODT>), grid, dim3(fused_waves(16) * kWave), 0, s, a);
  else if (a.r <= 32) hipLaunchKernelGGL((fused_kernel<32, ODT>), grid, dim3(fused_waves(32) * kWave), 0, s, a);
  else hipLaunchKernelGGL((fused_kernel<64, ODT>), grid, dim3(fused_waves(64) * kWave), 0, s, a);
}

hipError_t launch_lora(const LoraLaunch& L, hipStream_t stream) {
  const LoraGroups& q = L.q;
  if (lora_fused(q)) {
    const int64_t tiles = tiles_bound(q.S, q.G, 4);
    const int chunks = expand_chunks(tiles, q.N, fused_waves(q.r), kFusedWanted);
    FusedArgs a{L.x, L.a, L.b, L.scale, q.offsets, q.ids, L.y, L.out, L.z, q.K, q.N, int(q.S), int(q.G), int(q.n),
                q.r, uint32_t(chunks), int(div_up(div_up(q.N, 64), chunks))};
    const dim3 grid(unsigned(tiles * chunks));
    if (L.out_dtype == 0) fused_dt<0>(a, grid, stream);
    else fused_dt<1>(a, grid, stream);
    return hipGetLastError();
  }
  const int pieces = shrink_pieces(q, q.K);
  float* z = pieces == 1 && L.z ? L.z : reinterpret_cast<float*>(L.ws);
  if (hipError_t e = shrink(q, L.x, L.a, nullptr, q.K, z, pieces, stream); e != hipSuccess) return e;
  return expand(q, z, pieces, L.b, L.scale, q.N, L.y, L.out, L.out_dtype, pieces > 1 ? L.z : nullptr, stream);
}

hipError_t launch_lora_backward(const LoraBackwardLaunch& L, hipStream_t stream) {
  const LoraGroups& q = L.q;
  const BackwardLayout w = backward_layout(L);
  char* ws = reinterpret_cast<char*>(L.ws);
  float* u = reinterpret_cast<float*>(ws + w.u);
  float* parts_a = reinterpret_cast<float*>(ws + w.parts_a);
  float* parts_b = reinterpret_cast<float*>(ws + w.parts_b);
  const bool need_u = L.gx || L.ga;  // as the layout has it
  hipError_t e = hipSuccess;
  if (q.S > 0) {
    float* upart = need_u ? reinterpret_cast<float*>(ws + w.upart) : nullptr;
    if ((e = grad_pass(q, L.z, L.g, L.b, L.scale, q.N, true, L.gb, parts_b, upart, stream)) != hipSuccess) return e;
    if (need_u) {
      uint16_t* at = L.gx ? reinterpret_cast<uint16_t*>(ws + w.at) : nullptr;
      const int64_t u_blocks = between_u_blocks(q);
      const int64_t t_blocks = at ? between_at_blocks(q) : 0;
      BetweenArgs a{upart, u, L.a, at, q.S * q.r, uint32_t(u_blocks), int(q.n), q.r,
                    int(div_up(q.N, kGradCols * grad_subs(q.r, true))), int(q.K)};
      hipLaunchKernelGGL(between_kernel, dim3(unsigned(u_blocks + t_blocks)), dim3(kThreads), 0, stream, a);
      if ((e = hipGetLastError()) != hipSuccess) return e;
      if (L.gx) {
        e = expand(q, u, 1, at, nullptr, q.K, L.gx_base, L.gx, L.gx_dtype, nullptr, stream);
        if (e != hipSuccess) return e;
      }
      if (L.ga) {
        e = grad_pass(q, u, L.x, nullptr, nullptr, q.K, false, L.ga, parts_a, nullptr, stream);
        if (e != hipSuccess) return e;
      }
    }
  }
  if (!L.ga && !L.gb) return e;
  ReduceArgs d{};
  d.offsets = q.offsets;
  d.ids = q.ids;
  d.S = int(q.S);
  d.G = int(q.G);
  d.n = int(q.n);
  int64_t blocks = 0;
  if (L.gb) {
    reduce_of(q, q.N, need_u, L.gb, parts_b, &d.of[0]);
    blocks = q.n * d.of[0].chunks;
  }
  d.first = uint32_t(blocks);
  if (L.ga) {
    reduce_of(q, q.K, false, L.ga, parts_a, &d.of[1]);
    blocks += q.n * d.of[1].chunks;
  }
  hipLaunchKernelGGL(grad_reduce_kernel, dim3(unsigned(blocks)), dim3(kThreads), 0, stream, d);
  return hipGetLastError();
}

}  // namespace e4b
