// Low-rank adapters on grouped rows, beside a projection that others compute, and their
// gradients.  Rows are grouped (by expert: the router's offsets; by request: the batch's), a group
// g uses adapter a = group_adapter[g] (or g itself):
//   forward    z = x A_a^T,  out = y + s_a z B_a^T
//   backward   u = s_a g B_a,  gx = gx0 + u A_a,  gA_a = sum_p u_p^T x_p,  gB_a = s_a sum_p g_p^T z_p
// with A_a [r, K], B_a [N, r] bf16, r = 8 .. 128.  About 2r / b flop for each byte moved (b the
// bytes of an element read and written): bound by memory at every rank taken here, so the kernels
// are three streaming passes with the matrix unit beside them:
//   shrink   [rows, C] x [r, C]^T -> [rows, r]     (z from x and A; u from g and B^T)
//   expand   [rows, r] x [C, r]^T added to [rows, C]   (out from z and B; gx from u and A^T)
//   wgrad    [rows, r]^T x [rows, C] -> [r, C]     (gA from u and x; gB from z and g)
// Products of bf16 values go through the bf16 matrix instruction exactly, with float32 sums.  z
// and u are float32 all the way: in expand each is cut into three bf16 parts (8 + 8 + 8 bits of
// its 24-bit significand: no rounding) that stand behind one another in the contraction, in wgrad
// they enter the float32 matrix instruction.
#include "e4b_internal.h"
#include "e4b_rows.h"

namespace e4b {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;

struct RowTile {
  int group;
  int64_t row0;
  int rows;        // 1 .. bm; 0: no such tile
  int64_t kept;    // index among the tiles of groups with more than one (find_tile's `single` false)
};

// Tile `tile` of the list that cuts every group into pieces of 1 << bm_log2 rows, found by each
// wave from the offsets (64 groups a step).  Offsets are clamped to [0, S] and to ascending order,
// so a tile never reaches a row outside the matrices.
__device__ __forceinline__ RowTile find_tile(const int32_t* __restrict__ offsets, int G, int64_t S, int bm_log2,
                                             int64_t tile, bool single) {
  const int lane = threadIdx.x & (kWave - 1);
  int64_t base = 0, kbase = 0;
  for (int g0 = 0; g0 < G; g0 += kWave) {
    const int g = g0 + lane;
    int64_t lo = 0, hi = 0;
    if (g < G) {
      lo = offsets[g];
      hi = offsets[g + 1];
      lo = lo < 0 ? 0 : (lo > S ? S : lo);
      hi = hi < lo ? lo : (hi > S ? S : hi);
    }
    const int n = int((hi - lo + (int64_t(1) << bm_log2) - 1) >> bm_log2);
    const int k = single && n == 1 ? 0 : n;
    int ni = n, ki = k;  // inclusive sums over the wave
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const int a = __shfl_up(ni, d, kWave), b = __shfl_up(ki, d, kWave);
      if (lane >= d) {
        ni += a;
        ki += b;
      }
    }
    const int total = __shfl(ni, kWave - 1, kWave);
    if (tile < base + total) {
      const uint64_t hit = __ballot(tile < base + ni);
      const int l = __ffsll((unsigned long long)hit) - 1;
      const int64_t at = tile - (base + __shfl(ni - n, l, kWave));
      RowTile t;
      t.group = g0 + l;
      t.row0 = __shfl(int(lo), l, kWave) + (at << bm_log2);
      const int64_t left = __shfl(int(hi), l, kWave) - t.row0;
      t.rows = int(left < (int64_t(1) << bm_log2) ? left : (int64_t(1) << bm_log2));
      t.kept = kbase + __shfl(ki - k, l, kWave) + at;
      if (single && __shfl(n, l, kWave) == 1) t.kept = -1;
      return t;
    }
    base += total;
    kbase += __shfl(ki, kWave - 1, kWave);
  }
  return RowTile{0, 0, 0, 0};
}

__device__ __forceinline__ int adapter_of(const int32_t* __restrict__ ids, int group, int n) {
  const int a = ids ? ids[group] : group;
  return a >= 0 && a < n ? a : -1;
}

__device__ __forceinline__ bf16x8 load8(const uint16_t* p) { return *reinterpret_cast<const bf16x8*>(p); }

struct ShrinkArgs {
  const uint16_t* m;      // [S, C]
  const uint16_t* w;      // [n, r, C]
  const float* scale;     // nullable: 1
  const int32_t* offsets;
  const int32_t* ids;     // nullable: group = adapter
  float* z;               // [ksplit, S, r]
  int64_t S, C;
  int G, n, r, bm_log2, ksplit;
};

// A workgroup: up to 16 * RB rows of a group, one of ksplit pieces of the columns; its waves take
// 32-column steps in turn (256 contiguous bytes of each row together) and their sums meet in LDS.
// The adapter is the matrix instruction's first operand, so a lane ends with 4 ranks of one row.
template <int RB, int RT>
__global__ void __launch_bounds__(kThreads) shrink_kernel(ShrinkArgs p) {
  __shared__ f32x4 part[kWaves][RB * RT][kWave];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x >> 6;
  const int c = lane & 15, q = lane >> 4;
  const int ks = int(blockIdx.x) % p.ksplit;
  const RowTile t = find_tile(p.offsets, p.G, p.S, p.bm_log2, int64_t(blockIdx.x) / p.ksplit, false);
  if (t.rows == 0) return;
  const int a = adapter_of(p.ids, t.group, p.n);
  f32x4 acc[RB][RT];
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int k = 0; k < RT; ++k) acc[b][k] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (a >= 0) {
    const uint16_t* mp[RB];
    const uint16_t* wp[RT];
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      const int row = 16 * b + c < t.rows ? 16 * b + c : t.rows - 1;  // a row past the tile repeats its last
      mp[b] = p.m + (t.row0 + row) * p.C + 8 * q;
    }
#pragma unroll
    for (int k = 0; k < RT; ++k) {
      const int i = 16 * k + c < p.r ? 16 * k + c : p.r - 1;          // ranks past r are not stored
      wp[k] = p.w + (int64_t(a) * p.r + i) * p.C + 8 * q;
    }
    const int64_t steps = (p.C + 31) >> 5, full = p.C >> 5;
    const int64_t per = (steps + p.ksplit - 1) / p.ksplit;
    const int64_t end = (ks + 1) * per < steps ? (ks + 1) * per : steps;
    const int64_t fend = end < full ? end : full;
    constexpr int U = RB * RT <= 4 ? 4 : 2;
    int64_t s = ks * per + wave;
    for (; s + (U - 1) * kWaves < fend; s += U * kWaves) {
      bf16x8 mv[U][RB], wv[U][RT];
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int b = 0; b < RB; ++b) mv[u][b] = load8(mp[b] + 32 * (s + u * kWaves));
#pragma unroll
        for (int k = 0; k < RT; ++k) wv[u][k] = load8(wp[k] + 32 * (s + u * kWaves));
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int b = 0; b < RB; ++b)
#pragma unroll
          for (int k = 0; k < RT; ++k)
            acc[b][k] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv[u][k], mv[u][b], acc[b][k], 0, 0, 0);
    }
    for (; s < end; s += kWaves) {
      const bool in = 32 * s + 8 * q < p.C;  // the last step may hold fewer than 32 columns
      const int64_t at = in ? 32 * s : 0;
      bf16x8 wv[RT];
#pragma unroll
      for (int k = 0; k < RT; ++k) wv[k] = in ? load8(wp[k] + at) : bf16x8{};
#pragma unroll
      for (int b = 0; b < RB; ++b) {
        const bf16x8 mv = in ? load8(mp[b] + at) : bf16x8{};
#pragma unroll
        for (int k = 0; k < RT; ++k)
          acc[b][k] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv[k], mv, acc[b][k], 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int k = 0; k < RT; ++k) part[wave][b * RT + k][lane] = acc[b][k];
  __syncthreads();
  const float sc = a >= 0 && p.scale ? p.scale[a] : 1.f;
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

struct ExpandArgs {
  const float* z;         // [ksplit, S, r]: the sum over ksplit is taken here
  const uint16_t* w;      // [n, C, r]
  const float* scale;     // nullable: 1
  const int32_t* offsets;
  const int32_t* ids;
  const void* base;       // nullable [S, C]
  void* out;              // [S, C]
  float* z_out;           // nullable [S, r]: the summed z
  int64_t S, C;
  int G, n, r, bm_log2, ksplit, chunks;
};

// v = hi + mid + lo exactly: each part the 8 leading bits of what is left.  An infinity or NaN
// stands in the first part alone.
__device__ __forceinline__ void split3(float v, uint16_t (&h)[3]) {
  const uint32_t b = __float_as_uint(v);
  h[0] = uint16_t(b >> 16);
  if ((b & 0x7F800000u) == 0x7F800000u) {
    if ((b & 0x007FFFFFu) != 0) h[0] |= 0x40;
    h[1] = h[2] = 0;
    return;
  }
  const float r1 = v - __uint_as_float(b & 0xFFFF0000u);
  const uint32_t b1 = __float_as_uint(r1);
  h[1] = uint16_t(b1 >> 16);
  h[2] = uint16_t(__float_as_uint(r1 - __uint_as_float(b1 & 0xFFFF0000u)) >> 16);
}

// A workgroup: up to 16 * RB rows of a group and one of `chunks` pieces of the columns.  The rows'
// z stands in registers as hi | mid | lo parts of RP (r rounded up to a power of two) ranks each;
// waves take 32 columns at a time: two matrix tiles whose rows are dealt out so that a lane holds
// 8 consecutive columns of one row.
template <int RB, int RP, int ODT>
__global__ void __launch_bounds__(kThreads) expand_kernel(ExpandArgs p) {
  constexpr int kSteps = (3 * RP + 31) / 32;           // 32-deep matrix steps over the three parts
  constexpr int kFrags = RP >= 32 ? RP / 32 : 1;       // distinct adapter fragments among them
  constexpr int kStride = 32 * kSteps + 8;             // LDS row in bf16 (16 rows hit distinct banks)
  __shared__ __attribute__((aligned(16))) uint16_t zs[16 * RB * kStride];
  typedef row_elem<ODT> out_t;
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x >> 6;
  const int c = lane & 15, q = lane >> 4;
  const int chunk = int(blockIdx.x) % p.chunks;
  const RowTile t = find_tile(p.offsets, p.G, p.S, p.bm_log2, int64_t(blockIdx.x) / p.chunks, false);
  if (t.rows == 0) return;
  const int a = adapter_of(p.ids, t.group, p.n);
  if (a < 0 && p.base == p.out && !(p.z_out && chunk == 0)) return;  // these rows stay as they are

  const float sc = a >= 0 && p.scale ? p.scale[a] : 1.f;
  for (int i = threadIdx.x; i < 16 * RB * 4 * kSteps; i += kThreads) {
    const int row = i / (4 * kSteps), ch = i % (4 * kSteps);  // 8 positions of the contraction
    const int part = 8 * ch / RP, rank = 8 * ch % RP;
    uint16_t h[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (part < 3 && row < t.rows && rank < p.r && a >= 0) {
      const float* zp = p.z + (t.row0 + row) * p.r + rank;
      float v[8];
      load_vec<8>(zp, v);
      for (int k = 1; k < p.ksplit; ++k) {
        float o[8];
        load_vec<8>(zp + int64_t(k) * p.S * p.r, o);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += o[j];
      }
      if (p.z_out && chunk == 0 && part == 0) store_vec<8>(p.z_out + (t.row0 + row) * p.r + rank, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint16_t s[3];
        split3(v[j] * sc, s);
        h[j] = s[part];
      }
    } else if (p.z_out && chunk == 0 && part == 0 && row < t.rows && rank < p.r) {
      const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      store_vec<8>(p.z_out + (t.row0 + row) * p.r + rank, zero);
    }
    u32x4 d;
#pragma unroll
    for (int j = 0; j < 4; ++j) d[j] = uint32_t(h[2 * j]) | (uint32_t(h[2 * j + 1]) << 16);
    *reinterpret_cast<u32x4*>(zs + row * kStride + 8 * ch) = d;
  }
  __syncthreads();
  if (a < 0 && p.base == p.out) return;
  bf16x8 zf[RB][kSteps];
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int k = 0; k < kSteps; ++k)
      zf[b][k] = *reinterpret_cast<const bf16x8*>(zs + (16 * b + c) * kStride + 32 * k + 8 * q);

  const int64_t steps = (p.C + 31) >> 5, per = (steps + p.chunks - 1) / p.chunks;
  const int64_t end = (chunk + 1) * per < steps ? (chunk + 1) * per : steps;
  const out_t* base = static_cast<const out_t*>(p.base);
  out_t* out = static_cast<out_t*>(p.out);
  for (int64_t s = chunk * per + wave; s < end; s += kWaves) {
    const int64_t col = 32 * s + 8 * q;
    const bool in = col < p.C;
    float y[RB][8];
#pragma unroll
    for (int b = 0; b < RB; ++b) {
#pragma unroll
      for (int j = 0; j < 8; ++j) y[b][j] = 0.f;
      if (base && in && 16 * b + c < t.rows) load_vec<8>(base + (t.row0 + 16 * b + c) * p.C + col, y[b]);
    }
    if (a >= 0) {
      bf16x8 wf[2][kFrags];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        int64_t n = 32 * s + 8 * (c >> 2) + 4 * h + (c & 3);
        n = n < p.C ? n : p.C - 1;                    // columns past C are not stored
#pragma unroll
        for (int f = 0; f < kFrags; ++f) {
          const int rank = (32 * f + 8 * q) % RP;     // ranks past r meet zeros of z: no garbage there
          wf[h][f] = rank < p.r ? load8(p.w + (int64_t(a) * p.C + n) * p.r + rank) : bf16x8{};
        }
      }
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          f32x4 d = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int k = 0; k < kSteps; ++k)
            d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[h][k % kFrags], zf[b][k], d, 0, 0, 0);
#pragma unroll
          for (int j = 0; j < 4; ++j) y[b][4 * h + j] += d[j];
        }
    }
#pragma unroll
    for (int b = 0; b < RB; ++b)
      if (in && 16 * b + c < t.rows) store_vec<8>(out + (t.row0 + 16 * b + c) * p.C + col, y[b]);
  }
}

struct WgradArgs {
  const float* v;         // [S, r]
  const uint16_t* m;      // [S, C]
  const float* scale;     // nullable: 1
  const int32_t* offsets;
  const int32_t* ids;
  float* grad;            // [n, r, C], or [n, C, r] (by_column)
  float* parts;           // [tiles, r, C] (or [tiles, C, r])
  int64_t S, C, parts_cap;  // parts there is room for (offsets that are not ascending ask for more)
  int G, n, r, bm_log2, chunks, by_column;
};

constexpr int kWgradCols = 128 * kWaves;

// A workgroup: the rows of one tile and 512 columns, a wave 128 of them (8 a lane, 16 bytes of a
// row) by up to 16 * RT ranks.  Four rows feed one float32 matrix instruction for each of a lane's
// 8 columns, no transposition: the instruction's column index is the lane, and its 8 tiles are the
// lanes' 8 columns.
template <int RT>
__global__ void __launch_bounds__(kThreads) wgrad_kernel(WgradArgs p) {
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x >> 6;
  const int c = lane & 15, q = lane >> 4;
  const int chunk = int(blockIdx.x) % p.chunks;
  const int rank0 = 16 * RT * int(blockIdx.y);
  const bool single = p.ids == nullptr;
  const RowTile t = find_tile(p.offsets, p.G, p.S, p.bm_log2, int64_t(blockIdx.x) / p.chunks, single);
  if (t.rows == 0) return;
  const int a = adapter_of(p.ids, t.group, p.n);
  if (a < 0) return;
  const int64_t col = int64_t(chunk) * kWgradCols + 128 * wave + 8 * c;
  const bool in = col < p.C;
  const uint16_t* mp = p.m + t.row0 * p.C + (in ? col : 0);
  const float* vp = p.v + t.row0 * p.r;
  f32x4 acc[RT][8];
#pragma unroll
  for (int k = 0; k < RT; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[k][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto fma_rows = [&](const u32x4& mv, const float (&vv)[RT]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float mf = __uint_as_float(j & 1 ? mv[j >> 1] & 0xFFFF0000u : mv[j >> 1] << 16);
#pragma unroll
      for (int k = 0; k < RT; ++k) acc[k][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(vv[k], mf, acc[k][j], 0, 0, 0);
    }
  };
  constexpr int U = RT <= 2 ? 8 : 4;
  int row = q;
  for (; row - q + 4 * U <= t.rows; row += 4 * U) {
    u32x4 mv[U];
    float vv[U][RT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      mv[u] = *reinterpret_cast<const u32x4*>(mp + int64_t(row + 4 * u) * p.C);
#pragma unroll
      for (int k = 0; k < RT; ++k) {
        const int i = rank0 + 16 * k + c;
        vv[u][k] = vp[int64_t(row + 4 * u) * p.r + (i < p.r ? i : 0)];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) fma_rows(mv[u], vv[u]);
  }
  for (; row - q < t.rows; row += 4) {  // rows past the tile enter as zeros
    u32x4 mv = u32x4{0, 0, 0, 0};
    float vv[RT];
#pragma unroll
    for (int k = 0; k < RT; ++k) vv[k] = 0.f;
    if (row < t.rows) {
      mv = *reinterpret_cast<const u32x4*>(mp + int64_t(row) * p.C);
#pragma unroll
      for (int k = 0; k < RT; ++k) {
        const int i = rank0 + 16 * k + c;
        vv[k] = vp[int64_t(row) * p.r + (i < p.r ? i : 0)];
      }
    }
    fma_rows(mv, vv);
  }
  if (!in || t.kept >= p.parts_cap) return;
  const float sc = p.scale ? p.scale[a] : 1.f;
  float* dst = t.kept < 0 ? p.grad + int64_t(a) * p.r * p.C : p.parts + t.kept * p.r * p.C;
#pragma unroll
  for (int k = 0; k < RT; ++k) {
    const int i = rank0 + 16 * k + 4 * q;
    if (i >= p.r) continue;
    if (p.by_column) {
#pragma unroll
      for (int j = 0; j < 8; ++j) *reinterpret_cast<f32x4*>(dst + (col + j) * p.r + i) = acc[k][j] * sc;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float* d = dst + int64_t(i + e) * p.C + col;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<f32x4*>(d + 4 * h) =
              f32x4{acc[k][4 * h][e], acc[k][4 * h + 1][e], acc[k][4 * h + 2][e], acc[k][4 * h + 3][e]} * sc;
      }
    }
  }
}

struct ReduceArgs {
  const float* parts;     // [tiles, len]
  const int32_t* offsets;
  const int32_t* ids;
  float* grad;            // [n, len]
  int64_t S, len, parts_cap;
  int G, n, bm_log2, chunks;
};

// grad[a] = the sum of the parts of a's groups in order (0 without rows); a group of one tile
// under ids == NULL has written its adapter's gradient itself.
__global__ void __launch_bounds__(kThreads) wgrad_reduce_kernel(ReduceArgs p) {
  const int lane = threadIdx.x & (kWave - 1);
  const int a = int(int64_t(blockIdx.x) / p.chunks);
  const int64_t e = (int64_t(int(blockIdx.x) % p.chunks) * kThreads + threadIdx.x) * 4;
  const bool single = p.ids == nullptr;
  f32x4 sum = f32x4{0.f, 0.f, 0.f, 0.f};
  int64_t kbase = 0;
  for (int g0 = 0; g0 < p.G; g0 += kWave) {
    const int g = g0 + lane;
    int64_t lo = 0, hi = 0;
    int id = -1;
    if (g < p.G) {
      lo = p.offsets[g];
      hi = p.offsets[g + 1];
      lo = lo < 0 ? 0 : (lo > p.S ? p.S : lo);
      hi = hi < lo ? lo : (hi > p.S ? p.S : hi);
      id = adapter_of(p.ids, g, p.n);
    }
    const int n = int((hi - lo + (int64_t(1) << p.bm_log2) - 1) >> p.bm_log2);
    const int k = single && n == 1 ? 0 : n;
    int ki = k;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const int b = __shfl_up(ki, d, kWave);
      if (lane >= d) ki += b;
    }
    if (single && a >= g0 && a < g0 + kWave && __shfl(n, a - g0, kWave) == 1) return;
    uint64_t mine = __ballot(id == a && k > 0);
    while (mine) {
      const int l = __ffsll((unsigned long long)mine) - 1;
      mine &= mine - 1;
      const int cnt = __shfl(k, l, kWave);
      const int64_t first = kbase + __shfl(ki - k, l, kWave);
      if (e < p.len)
        for (int i = 0; i < cnt && first + i < p.parts_cap; ++i)
          sum += *reinterpret_cast<const f32x4*>(p.parts + (first + i) * p.len + e);
    }
    kbase += __shfl(ki, kWave - 1, kWave);
  }
  if (e < p.len) *reinterpret_cast<f32x4*>(p.grad + int64_t(a) * p.len + e) = sum;
}

// [n, R, C] -> [n, C, R] bf16, 64 x 64 tiles through LDS.
__global__ void __launch_bounds__(kThreads) transpose_kernel(const uint16_t* __restrict__ src, int R, int C,
                                                             int tiles_r, int tiles_c, uint16_t* __restrict__ dst) {
  __shared__ uint16_t t[64][66];
  const int tc = int(blockIdx.x) % tiles_c, tr = int(blockIdx.x) / tiles_c % tiles_r;
  const int64_t at = int64_t(int(blockIdx.x) / tiles_c / tiles_r) * R * C;
  for (int i = threadIdx.x; i < 64 * 64; i += kThreads) {
    const int r = 64 * tr + i / 64, c = 64 * tc + i % 64;
    if (r < R && c < C) t[i / 64][i % 64] = src[at + int64_t(r) * C + c];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 64 * 64; i += kThreads) {
    const int c = 64 * tc + i / 64, r = 64 * tr + i % 64;
    if (r < R && c < C) dst[at + int64_t(c) * R + r] = t[i % 64][i / 64];
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
// 32 at ranks over 64, whose parts fill the registers.
int row_tile_log2(int64_t S, int64_t G, int r) { return S <= 16 * G ? 4 : (r > 64 ? 5 : 6); }

// Pieces the columns of a shrink are cut into: enough workgroups for two on every CU, no piece
// under 512 columns (four 32-column steps a wave).
int shrink_pieces(int64_t tiles, int64_t C) {
  const int64_t want = div_up(512, tiles > 0 ? tiles : 1), most = C / 512;
  const int64_t k = want < most ? want : most;
  return int(k < 1 ? 1 : (k > 16 ? 16 : k));
}

// Rows of a wgrad tile: as many as leave four workgroups a CU, 64 at least (a tile costs one
// float32 write and read of its [r, C] sums).
int wgrad_tile_log2(int64_t S, int64_t C) {
  const int64_t chunks = div_up(C, kWgradCols);
  const int l = log2_up(div_up(S * chunks, 1024));
  return l < 6 ? 6 : (l > 20 ? 20 : l);
}

// Tiles that write parts: all where adapters are shared by groups; without ids only those of
// groups of several tiles, at most two for each full tile of rows.
int64_t parts_bound(int64_t S, int64_t G, int bm_log2, bool ids) {
  const int64_t all = tiles_bound(S, G, bm_log2), kept = (2 * S) >> bm_log2;
  return ids || all < kept ? all : kept;
}

template <int RB>
void shrink_rb(const ShrinkArgs& a, unsigned grid, hipStream_t s) {
  if (a.r <= 16) hipLaunchKernelGGL((shrink_kernel<RB, 1>), dim3(grid), dim3(kThreads), 0, s, a);
  else if (a.r <= 32) hipLaunchKernelGGL((shrink_kernel<RB, 2>), dim3(grid), dim3(kThreads), 0, s, a);
  else if (a.r <= 64) hipLaunchKernelGGL((shrink_kernel<RB, 4>), dim3(grid), dim3(kThreads), 0, s, a);
  else if constexpr (RB <= 2) hipLaunchKernelGGL((shrink_kernel<RB, 8>), dim3(grid), dim3(kThreads), 0, s, a);
}

hipError_t shrink(const ShrinkArgs& a, int64_t tiles, hipStream_t s) {
  const unsigned grid = unsigned(tiles * a.ksplit);
  if (grid == 0) return hipSuccess;
  if (a.bm_log2 == 4) shrink_rb<1>(a, grid, s);
  else if (a.bm_log2 == 5) shrink_rb<2>(a, grid, s);
  else shrink_rb<4>(a, grid, s);
  return hipGetLastError();
}

template <int RB, int ODT>
void expand_rb(const ExpandArgs& a, unsigned grid, hipStream_t s) {
  if (a.r <= 8) hipLaunchKernelGGL((expand_kernel<RB, 8, ODT>), dim3(grid), dim3(kThreads), 0, s, a);
  else if (a.r <= 16) hipLaunchKernelGGL((expand_kernel<RB, 16, ODT>), dim3(grid), dim3(kThreads), 0, s, a);
  else if (a.r <= 32) hipLaunchKernelGGL((expand_kernel<RB, 32, ODT>), dim3(grid), dim3(kThreads), 0, s, a);
  else if (a.r <= 64) hipLaunchKernelGGL((expand_kernel<RB, 64, ODT>), dim3(grid), dim3(kThreads), 0, s, a);
  else if constexpr (RB <= 2) hipLaunchKernelGGL((expand_kernel<RB, 128, ODT>), dim3(grid), dim3(kThreads), 0, s, a);
}

template <int ODT>
void expand_dt(const ExpandArgs& a, unsigned grid, hipStream_t s) {
  if (a.bm_log2 == 4) expand_rb<1, ODT>(a, grid, s);
  else if (a.bm_log2 == 5) expand_rb<2, ODT>(a, grid, s);
  else expand_rb<4, ODT>(a, grid, s);
}

int expand_chunks(int64_t tiles, int64_t C) {
  const int64_t most = div_up(div_up(C, 32), kWaves), want = div_up(1024, tiles > 0 ? tiles : 1);
  return int(want < most ? want : most);
}

hipError_t expand(const ExpandArgs& a, int odt, int64_t tiles, hipStream_t s) {
  const unsigned grid = unsigned(tiles * a.chunks);
  if (grid == 0) return hipSuccess;
  if (odt == 0) expand_dt<0>(a, grid, s);
  else expand_dt<1>(a, grid, s);
  return hipGetLastError();
}

hipError_t transpose(const uint16_t* src, int64_t n, int64_t R, int64_t C, uint16_t* dst, hipStream_t s) {
  const int64_t tr = div_up(R, 64), tc = div_up(C, 64);
  hipLaunchKernelGGL(transpose_kernel, dim3(unsigned(n * tr * tc)), dim3(kThreads), 0, s, src, int(R), int(C),
                     int(tr), int(tc), dst);
  return hipGetLastError();
}

hipError_t wgrad(const LoraGroups& q, const float* v, const uint16_t* m, const float* scale, int64_t C, bool by_column,
                 float* grad, float* parts, hipStream_t s) {
  WgradArgs a{};
  a.v = v;
  a.m = m;
  a.scale = scale;
  a.offsets = q.offsets;
  a.ids = q.ids;
  a.grad = grad;
  a.parts = parts;
  a.S = q.S;
  a.C = C;
  a.G = int(q.G);
  a.n = int(q.n);
  a.r = q.r;
  a.bm_log2 = wgrad_tile_log2(q.S, C);
  a.chunks = int(div_up(C, kWgradCols));
  a.by_column = by_column ? 1 : 0;
  a.parts_cap = parts_bound(q.S, q.G, a.bm_log2, q.ids != nullptr);
  const unsigned grid = unsigned(tiles_bound(q.S, q.G, a.bm_log2) * a.chunks);
  if (grid == 0) ;  // no rows: the sums below are over nothing
  else if (q.r <= 16) hipLaunchKernelGGL(wgrad_kernel<1>, dim3(grid), dim3(kThreads), 0, s, a);
  else if (q.r <= 32) hipLaunchKernelGGL(wgrad_kernel<2>, dim3(grid), dim3(kThreads), 0, s, a);
  else hipLaunchKernelGGL(wgrad_kernel<4>, dim3(grid, q.r > 64 ? 2 : 1), dim3(kThreads), 0, s, a);
  if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  ReduceArgs d{};
  d.parts = parts;
  d.offsets = q.offsets;
  d.ids = q.ids;
  d.grad = grad;
  d.S = q.S;
  d.len = q.r * C;
  d.parts_cap = a.parts_cap;
  d.G = a.G;
  d.n = a.n;
  d.bm_log2 = a.bm_log2;
  d.chunks = int(div_up(d.len, 4 * kThreads));
  hipLaunchKernelGGL(wgrad_reduce_kernel, dim3(unsigned(q.n * d.chunks)), dim3(kThreads), 0, s, d);
  return hipGetLastError();
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

// Workspace of a backward call.
struct BackwardLayout {
  int pieces;
  size_t u, upart, bt, at, parts, total;
};
BackwardLayout backward_layout(const LoraBackwardLaunch& L) {
  const LoraGroups& q = L.q;
  BackwardLayout w{};
  const int64_t tiles = tiles_bound(q.S, q.G, row_tile_log2(q.S, q.G, q.r));
  const bool need_u = L.gx || L.ga;
  // the pieces of u are summed where gx is expanded from them
  w.pieces = L.gx ? shrink_pieces(tiles, q.N) : 1;
  size_t off = 0;
  w.u = off;
  if (need_u) off += align256(size_t(q.S) * q.r * 4);
  w.upart = off;
  if (w.pieces > 1) off += align256(size_t(w.pieces) * q.S * q.r * 4);
  w.bt = off;
  if (need_u) off += align256(size_t(q.n) * q.r * q.N * 2);
  w.at = off;
  if (L.gx) off += align256(size_t(q.n) * q.r * q.K * 2);
  w.parts = off;
  size_t pa = 0, pb = 0;  // one after the other in the same place
  if (L.ga) pa = size_t(parts_bound(q.S, q.G, wgrad_tile_log2(q.S, q.K), q.ids != nullptr)) * q.r * q.K * 4;
  if (L.gb) pb = size_t(parts_bound(q.S, q.G, wgrad_tile_log2(q.S, q.N), q.ids != nullptr)) * q.r * q.N * 4;
  off += align256(pa > pb ? pa : pb);
  w.total = off;
  return w;
}

}  // namespace

size_t lora_ws_bytes(const LoraLaunch& L) {
  const LoraGroups& q = L.q;
  const int64_t tiles = tiles_bound(q.S, q.G, row_tile_log2(q.S, q.G, q.r));
  return align256(size_t(shrink_pieces(tiles, q.K)) * q.S * q.r * 4);
}

size_t lora_backward_ws_bytes(const LoraBackwardLaunch& L) { return backward_layout(L).total; }

// Workgroups of the largest grid a call with these sizes starts.
int64_t lora_blocks(const LoraGroups& q) {
  const int64_t C = q.K > q.N ? q.K : q.N, c = q.K > q.N ? q.N : q.K;
  const int64_t tiles = tiles_bound(q.S, q.G, row_tile_log2(q.S, q.G, q.r));
  int64_t most = tiles * 16;
  const int64_t of[] = {tiles * div_up(C, 128), tiles_bound(q.S, q.G, wgrad_tile_log2(q.S, c)) * div_up(C, kWgradCols),
                        q.n * div_up(int64_t(q.r) * C, 4 * kThreads), q.n * div_up(q.r, 64) * div_up(C, 64)};
  for (int64_t v : of) most = v > most ? v : most;
  return most;
}

hipError_t launch_lora(const LoraLaunch& L, hipStream_t stream) {
  const LoraGroups& q = L.q;
  const int bm = row_tile_log2(q.S, q.G, q.r);
  const int64_t tiles = tiles_bound(q.S, q.G, bm);
  const int pieces = shrink_pieces(tiles, q.K);
  float* z = pieces == 1 && L.z ? L.z : reinterpret_cast<float*>(L.ws);
  ShrinkArgs a{L.x, L.a, nullptr, q.offsets, q.ids, z, q.S, q.K, int(q.G), int(q.n), q.r, bm, pieces};
  if (hipError_t e = shrink(a, tiles, stream); e != hipSuccess) return e;
  ExpandArgs b{z, L.b, L.scale, q.offsets, q.ids, L.y, L.out, pieces > 1 ? L.z : nullptr, q.S, q.N,
               int(q.G), int(q.n), q.r, bm, pieces, expand_chunks(tiles, q.N)};
  return expand(b, L.out_dtype, tiles, stream);
}

hipError_t launch_lora_backward(const LoraBackwardLaunch& L, hipStream_t stream) {
  const LoraGroups& q = L.q;
  const BackwardLayout w = backward_layout(L);
  char* ws = reinterpret_cast<char*>(L.ws);
  const int bm = row_tile_log2(q.S, q.G, q.r);
  const int64_t tiles = tiles_bound(q.S, q.G, bm);
  float* u = reinterpret_cast<float*>(ws + w.u);
  float* parts = reinterpret_cast<float*>(ws + w.parts);
  hipError_t e = hipSuccess;
  if ((L.gx || L.ga) && q.S > 0) {
    uint16_t* bt = reinterpret_cast<uint16_t*>(ws + w.bt);
    if ((e = transpose(L.b, q.n, q.N, q.r, bt, stream)) != hipSuccess) return e;
    float* to = w.pieces > 1 ? reinterpret_cast<float*>(ws + w.upart) : u;
    ShrinkArgs a{L.g, bt, L.scale, q.offsets, q.ids, to, q.S, q.N, int(q.G), int(q.n), q.r, bm, w.pieces};
    if ((e = shrink(a, tiles, stream)) != hipSuccess) return e;
    if (L.gx) {
      uint16_t* at = reinterpret_cast<uint16_t*>(ws + w.at);
      if ((e = transpose(L.a, q.n, q.r, q.K, at, stream)) != hipSuccess) return e;
      ExpandArgs b{to, at, nullptr, q.offsets, q.ids, L.gx_base, L.gx, w.pieces > 1 ? u : nullptr, q.S, q.K,
                   int(q.G), int(q.n), q.r, bm, w.pieces, expand_chunks(tiles, q.K)};
      if ((e = expand(b, L.gx_dtype, tiles, stream)) != hipSuccess) return e;
    }
  }
  if (L.ga && (e = wgrad(q, u, L.x, nullptr, q.K, false, L.ga, parts, stream)) != hipSuccess) return e;
  if (L.gb && (e = wgrad(q, L.z, L.g, L.scale, q.N, true, L.gb, parts, stream)) != hipSuccess) return e;
  return e;
}

}  // namespace e4b
