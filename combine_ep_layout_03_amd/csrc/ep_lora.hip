// Low-rank adapters over the expert-major segments, and their gradients:
//     out[r] = base[r] + s_e (x[r] A_e^T) B_e^T
//     dx[r]  = base[r] + s_e (g[r] B_e) A_e
//     dA_e   = s_e sum_r v_r x[r]^T,  dB_e = s_e sum_r g[r] u_r^T
// with u_r = A_e x[r] and v_r = B_e^T g[r], held in fp32 in the workspace.
//
// Three kernels on v_mfma_f32_16x16x32_bf16 (lane l holds operand row l % 16,
// elements (l / 16) * 8 .. + 7 of the contraction, and of the result column
// l % 16, rows (l / 16) * 4 .. + 3):
//   shrink   u or v: a tile of rows against all R rows of A_e (or columns of
//            B_e), the long contraction split over the waves and blocks
//   expand   out or dx: a tile of rows by 128 columns per wave, contraction R
//   weights  dA and dB: 128 columns per wave against all of R, contraction
//            over a chunk of an expert's rows
// u and v enter the second product as two bf16 parts, high and low: 16
// significand bits, so the result is as good as its own bf16 rounding allows
// (one bf16 part alone would add an error of the size of that rounding).
//
// A matrix whose contraction index is not contiguous in memory is transposed
// in registers: a lane loads 8 rows of 8 columns and forms, with 32 byte
// permutes, the 8 operands that hold one column each; operand row rho of
// product m then stands for column 8 perm(rho) + m.  That also leaves each
// lane with 8 neighbouring columns of the result.
#include "ep_layer.h"

namespace ep {

namespace {

constexpr int kCols = 128;  // columns of one wave
constexpr int kRowsStaged = 64;  // rows of u or v staged at a time by the weight gradients
constexpr int kRowPitch = kRowsStaged + 8;

__device__ __forceinline__ f32x4_t mfma(u32x4 a, u32x4 b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                 __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

__device__ __forceinline__ u32x4 load16(const uint16_t* p) { return *reinterpret_cast<const u32x4*>(p); }

// f as bf16 parts hi + lo.  Where hi is infinite lo is 0, not inf - inf.
__device__ __forceinline__ void split(float f, uint16_t& hi, uint16_t& lo) {
  hi = bf16_of(f);
  const float h = bf16_to_f32(hi);
  lo = fabsf(h) < __builtin_inff() ? bf16_of(f - h) : 0;
}

// Column m of the 8 x 8 block held as rows v[0..7] of 8 columns.
template <int M>
__device__ __forceinline__ u32x4 column(const u32x4 (&v)[8]) {
  constexpr uint32_t kSel = (M & 1) ? 0x07060302u : 0x05040100u;
  u32x4 r;
#pragma unroll
  for (int p = 0; p < 4; ++p) r[p] = __builtin_amdgcn_perm(v[2 * p + 1][M / 2], v[2 * p][M / 2], kSel);
  return r;
}
__device__ __forceinline__ void columns(const u32x4 (&v)[8], u32x4 (&c)[8]) {
  c[0] = column<0>(v);
  c[1] = column<1>(v);
  c[2] = column<2>(v);
  c[3] = column<3>(v);
  c[4] = column<4>(v);
  c[5] = column<5>(v);
  c[6] = column<6>(v);
  c[7] = column<7>(v);
}

// Block of 8 columns that operand row rho stands for.  Result rows 4 q + i of
// quarter q then are blocks 4 i + q: the four quarters' stores of one i are
// neighbours.
__device__ __forceinline__ int perm(int rho) { return (rho & 3) * 4 + (rho >> 2); }

// Tile `tile` of the experts' rows cut into tiles of 2^shift rows, experts in
// order.  Every lane of the wave calls it with the same arguments.
struct Tile {
  int e;      // expert, -1: no such tile
  int im;     // tile within the expert
  int count;  // the expert's rows
  int slot;   // tiles of experts with several tiles, before this expert
};
__device__ __forceinline__ Tile find_tile(const int32_t* counts, int E, int shift, int tile) {
  const int lane = threadIdx.x & (kWave - 1);
  const int per = (E + kWave - 1) / kWave;  // at most 16
  int c[16];
  int sum = 0, many = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int e = lane * per + i;
    c[i] = i < per && e < E ? counts[e] : 0;
    const int n = (c[i] + (1 << shift) - 1) >> shift;
    sum += n;
    many += n > 1 ? n : 0;
  }
  int incl = sum, incl_many = many;
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) {
    const int a = __shfl_up(incl, off, kWave);
    const int b = __shfl_up(incl_many, off, kWave);
    if (lane >= off) {
      incl += a;
      incl_many += b;
    }
  }
  const uint64_t after = ballot(incl > tile);
  Tile t = {-1, 0, 0, 0};
  if (after == 0) return t;
  const int L = static_cast<int>(__builtin_ctzll(after));
  int left = tile - readlane(incl - sum, L);
  int slot = readlane(incl_many - many, L);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int ci = readlane(c[i], L);
    const int n = (ci + (1 << shift) - 1) >> shift;
    if (t.e < 0) {
      if (left < n) {
        t = {L * per + i, left, ci, slot};
      } else {
        left -= n;
        slot += n > 1 ? n : 0;
      }
    }
  }
  return t;
}

// ------------------------------------------------------------------- shrink
struct ShrinkArgs {
  const uint16_t* in;  // bf16 rows of C elements, row stride ld
  int64_t ld;
  const int32_t* map;
  const uint16_t* w;  // [E, R, C], or (KMAJOR) [E, C, R]
  int C, R, E;
  float* part;     // [S, rows, R]
  int64_t stride;  // rows * R
  int S;
  const int32_t* counts;
  const int32_t* offsets;
  int32_t* status;
  uint32_t generation;
};

// Block: one row tile (16 MT rows) and one split of the contraction, whose
// 64-wide pieces the 4 waves take in turn.
template <int RT, int MT, bool KMAJOR>
__global__ __launch_bounds__(kBlock) void k_lora_shrink(ShrinkArgs a) {
  constexpr int kShift = MT == 1 ? 4 : MT == 2 ? 5 : 6;
  constexpr int kPitch = RT * 16 + 4;
  __shared__ float red[MT * 16 * kPitch];
  if (!layout_current(a.status, a.generation)) return;
  const Tile t = find_tile(a.counts, a.E, kShift, static_cast<int>(blockIdx.x));
  if (t.e < 0) return;  // the whole block
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
  const int l16 = lane & 15, q = lane >> 4;
  const int row0 = a.offsets[t.e] + (t.im << kShift);
  const int nrows = min(16 * MT, t.count - (t.im << kShift));

  const uint16_t* xr[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int r = row0 + min(m * 16 + l16, nrows - 1);  // rows past the tile repeat its last
    xr[m] = a.in + static_cast<int64_t>(a.map ? a.map[r] : r) * a.ld;
  }
  const uint16_t* w = a.w + static_cast<int64_t>(t.e) * a.R * a.C;
  f32x4_t acc[MT][RT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < RT; ++j) acc[m][j] = f32x4_t{};

  const int pieces = (a.C + 63) / 64;
  const int s = static_cast<int>(blockIdx.y);
  const int p0 = static_cast<int>(static_cast<int64_t>(pieces) * s / a.S);
  const int p1 = static_cast<int>(static_cast<int64_t>(pieces) * (s + 1) / a.S);
  for (int p = p0 + wave; p < p1; p += kWavesPerBlock) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = p * 64 + h * 32 + q * 8;
      const bool ok = k < a.C;  // C is a multiple of 8
      u32x4 xv[MT], wv[RT];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        xv[m] = u32x4{0u, 0u, 0u, 0u};
        if (ok) xv[m] = load16(xr[m] + k);
      }
#pragma unroll
      for (int j = 0; j < RT; ++j) {
        const int jr = min(j * 16 + l16, a.R - 1);  // columns past R repeat the last, and are dropped
        wv[j] = u32x4{0u, 0u, 0u, 0u};
        if (ok) {
          if (KMAJOR) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint16_t* wp = w + static_cast<int64_t>(k + 2 * i) * a.R + jr;
              wv[j][i] = static_cast<uint32_t>(wp[0]) | (static_cast<uint32_t>(wp[a.R]) << 16);
            }
          } else {
            wv[j] = load16(w + static_cast<int64_t>(jr) * a.C + k);
          }
        }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < RT; ++j) acc[m][j] = mfma(wv[j], xv[m], acc[m][j]);
    }
  }
  // the waves' sums, added in wave order
  for (int n = 0; n < kWavesPerBlock; ++n) {
    if (wave == n) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < RT; ++j) {
          f32x4_t* d = reinterpret_cast<f32x4_t*>(red + (m * 16 + l16) * kPitch + j * 16 + q * 4);
          *d = n == 0 ? acc[m][j] : *d + acc[m][j];
        }
    }
    __syncthreads();
  }
  float* out = a.part + s * a.stride + static_cast<int64_t>(row0) * a.R;
  for (int i = threadIdx.x; i < nrows * a.R; i += kBlock) out[i] = red[(i / a.R) * kPitch + i % a.R];
}

// ------------------------------------------------------------------- expand
struct ExpandArgs {
  const float* part;  // [S, rows, R]
  int64_t stride;
  int S;
  const uint16_t* w;  // [E, N, R], or (JMAJOR) [E, R, N]
  const float* scales;
  const uint16_t* base;
  int64_t ldbase;
  uint16_t* out;
  int64_t ldout;
  const int32_t* map;
  const int32_t* slot;
  int64_t T;
  int N, R, E;
  const int32_t* counts;
  const int32_t* offsets;
  int32_t* status;
  uint32_t generation;
};

// Rows of out that belong to no selection (token rows only): base's row, or
// zeros.  32 tokens per block.
__device__ __forceinline__ void copy_unselected(const ExpandArgs& a, int64_t t0, int wave, int lane) {
  if (a.base == a.out) return;
  for (int i = 0; i < 8; ++i) {
    const int64_t t = t0 + wave * 8 + i;
    if (t >= a.T || a.slot[t] >= 0) continue;
    for (int n = lane * 8; n < a.N; n += kWave * 8) {
      u32x4 v = {0u, 0u, 0u, 0u};
      if (a.base) v = load16(a.base + t * a.ldbase + n);
      *reinterpret_cast<u32x4*>(a.out + t * a.ldout + n) = v;
    }
  }
}

// Block: one row tile by 512 columns.  PACK: R <= 16, the high parts in the
// first half of one contraction step and the low parts in the second.
template <int KS, int MT, bool PACK, bool JMAJOR>
__global__ __launch_bounds__(kBlock) void k_lora_expand(ExpandArgs a) {
  constexpr int kShift = MT == 1 ? 4 : MT == 2 ? 5 : 6;
  if (!layout_current(a.status, a.generation)) return;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
  const int ncb = (a.N + 4 * kCols - 1) / (4 * kCols);
  if (static_cast<int>(blockIdx.y) == ncb) {  // the layer of rows of no selection
    for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * 32; t0 < a.T; t0 += static_cast<int64_t>(gridDim.x) * 32)
      copy_unselected(a, t0, wave, lane);
    return;
  }
  const Tile t = find_tile(a.counts, a.E, kShift, static_cast<int>(blockIdx.x));
  if (t.e < 0) return;
  const int n0 = (static_cast<int>(blockIdx.y) * 4 + wave) * kCols;
  if (n0 >= a.N) return;
  const int l16 = lane & 15, q = lane >> 4;
  const int row0 = a.offsets[t.e] + (t.im << kShift);
  const int nrows = min(16 * MT, t.count - (t.im << kShift));
  const float scale = a.scales ? a.scales[t.e] : 1.0f;

  // operands of the rows: 8 of u's elements as high and low parts
  u32x4 hi[MT][KS], lo[MT][KS];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int r = row0 + min(m * 16 + l16, nrows - 1);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const int j = PACK ? (q & 1) * 8 : ks * 32 + q * 8;
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = 0.0f;
      if (j < a.R) {
        for (int s = 0; s < a.S; ++s) {
          const f32x4_t* p = reinterpret_cast<const f32x4_t*>(a.part + s * a.stride + static_cast<int64_t>(r) * a.R + j);
          const f32x4_t p0 = p[0], p1 = p[1];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            f[i] += p0[i];
            f[4 + i] += p1[i];
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint16_t h0, l0, h1, l1;
        split(f[2 * i], h0, l0);
        split(f[2 * i + 1], h1, l1);
        const uint32_t hh = h0 | (static_cast<uint32_t>(h1) << 16);
        const uint32_t ll = l0 | (static_cast<uint32_t>(l1) << 16);
        hi[m][ks][i] = PACK && q >= 2 ? ll : hh;
        lo[m][ks][i] = ll;
      }
    }
  }

  const uint16_t* w = a.w + static_cast<int64_t>(t.e) * a.R * a.N;
  const int blk = n0 + perm(l16) * 8;  // first of this operand row's 8 columns
  f32x4_t acc[MT][8];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int c = 0; c < 8; ++c) acc[m][c] = f32x4_t{};
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) {
    const int j = PACK ? (q & 1) * 8 : ks * 32 + q * 8;
    u32x4 wv[8];
    const bool ok = j < a.R && blk < a.N;
    if (JMAJOR) {
      u32x4 v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = u32x4{0u, 0u, 0u, 0u};
        if (ok) v[i] = load16(w + static_cast<int64_t>(j + i) * a.N + blk);
      }
      columns(v, wv);
    } else {
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        wv[c] = u32x4{0u, 0u, 0u, 0u};
        if (ok) wv[c] = load16(w + static_cast<int64_t>(blk + c) * a.R + j);
      }
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) {
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        acc[m][c] = mfma(wv[c], hi[m][ks], acc[m][c]);
        if (!PACK) acc[m][c] = mfma(wv[c], lo[m][ks], acc[m][c]);
      }
    }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int rl = m * 16 + l16;
    if (rl >= nrows) continue;
    const int r = row0 + rl;
    const int64_t orow = a.map ? a.map[r] : r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = n0 + (i * 4 + q) * 8;
      if (n >= a.N) continue;
      u32x4 bv = {0u, 0u, 0u, 0u};
      if (a.base) bv = load16(a.base + orow * a.ldbase + n);
      u32x4 o;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        o[c] = bf16x2_of(__builtin_fmaf(scale, acc[m][2 * c][i], bf16_lo(bv[c])),
                         __builtin_fmaf(scale, acc[m][2 * c + 1][i], bf16_hi(bv[c])));
      *reinterpret_cast<u32x4*>(a.out + orow * a.ldout + n) = o;
    }
  }
}

// --------------------------------------------------------- weight gradients
struct WeightGradArgs {
  // [0]: dA from x and v, [1]: dB from g and u
  const uint16_t* in[2];  // bf16 rows
  int64_t ld[2];
  const int32_t* map[2];
  int C[2];            // columns: H, N
  const float* part[2];  // v, u: [S, rows, R]
  int S[2];
  int64_t stride;
  uint16_t* out[2];  // dA [E, R, H], dB [E, N, R]
  float* slots;
  int64_t slot_size;  // R * (H + N)
  const float* scales;
  int R, E, shift;
  const int32_t* counts;
  const int32_t* offsets;
  int32_t* status;
  uint32_t generation;
};

// Block: one chunk of an expert's rows, 512 columns of x (or g), 16 JT of the
// R.  The columns are the row operand for dA, whose rows are R's, and the
// column operand for dB, whose rows are the columns: each lane ends with
// neighbouring elements of the result.
template <int JT, int B>
__device__ __forceinline__ void weight_grad(const WeightGradArgs& a, const Tile& t, int cb, int jg,
                                            uint16_t (*s_hi)[kRowPitch], uint16_t (*s_lo)[kRowPitch]) {
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
  const int l16 = lane & 15, q = lane >> 4;
  const int C = a.C[B], R = a.R;
  const int c0 = (cb * 4 + wave) * kCols;
  const int col = c0 + perm(l16) * 8;
  const int j0 = jg * JT * 16;
  const int first = t.im << a.shift;
  const int row0 = a.offsets[t.e] + first;
  const int nrows = min(1 << a.shift, t.count - first);

  f32x4_t acc[8][JT];
#pragma unroll
  for (int c = 0; c < 8; ++c)
#pragma unroll
    for (int j = 0; j < JT; ++j) acc[c][j] = f32x4_t{};

  for (int r0 = 0; r0 < nrows; r0 += kRowsStaged) {
    __syncthreads();  // the rows staged before are used up
    for (int i = threadIdx.x; i < kRowsStaged * JT * 16; i += kBlock) {
      const int r = i / (JT * 16), j = i % (JT * 16);
      float f = 0.0f;
      if (r0 + r < nrows && j0 + j < R) {
        const float* p = a.part[B] + static_cast<int64_t>(row0 + r0 + r) * R + j0 + j;
        for (int s = 0; s < a.S[B]; ++s) f += p[s * a.stride];
      }
      uint16_t h, l;
      split(f, h, l);
      s_hi[j][r] = h;
      s_lo[j][r] = l;
    }
    __syncthreads();
#pragma unroll
    for (int ks = 0; ks < kRowsStaged / 32; ++ks) {
      const int rq = r0 + ks * 32 + q * 8;
      u32x4 v[8], cv[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = u32x4{0u, 0u, 0u, 0u};
        if (rq + i < nrows && col < C) {
          const int r = row0 + rq + i;
          const int64_t xr = a.map[B] ? a.map[B][r] : r;
          v[i] = load16(a.in[B] + xr * a.ld[B] + col);
        }
      }
      columns(v, cv);
#pragma unroll
      for (int j = 0; j < JT; ++j) {
        const u32x4 h = *reinterpret_cast<const u32x4*>(&s_hi[j * 16 + l16][ks * 32 + q * 8]);
        const u32x4 l = *reinterpret_cast<const u32x4*>(&s_lo[j * 16 + l16][ks * 32 + q * 8]);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          if (B == 0) {
            acc[c][j] = mfma(cv[c], h, acc[c][j]);
            acc[c][j] = mfma(cv[c], l, acc[c][j]);
          } else {
            acc[c][j] = mfma(h, cv[c], acc[c][j]);
            acc[c][j] = mfma(l, cv[c], acc[c][j]);
          }
        }
      }
    }
  }

  const bool whole = t.count <= (1 << a.shift);
  const float scale = whole && a.scales ? a.scales[t.e] : 1.0f;
  uint16_t* out = a.out[B] + static_cast<int64_t>(t.e) * R * C;
  float* slot = whole ? nullptr
                      : a.slots + static_cast<int64_t>(t.slot + t.im) * a.slot_size +
                            (B == 0 ? 0 : static_cast<int64_t>(R) * a.C[0]);
#pragma unroll
  for (int j = 0; j < JT; ++j) {
    if (B == 0) {
      // rows 4 q + i: columns c0 + (4 i + q) 8 + c; column l16: row j of dA
      const int jr = j0 + j * 16 + l16;
      if (jr >= R) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = c0 + (i * 4 + q) * 8;
        if (n >= C) continue;
        const int64_t at = static_cast<int64_t>(jr) * C + n;
        if (whole) {
          u32x4 o;
#pragma unroll
          for (int c = 0; c < 4; ++c) o[c] = bf16x2_of(scale * acc[2 * c][j][i], scale * acc[2 * c + 1][j][i]);
          *reinterpret_cast<u32x4*>(out + at) = o;
        } else {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            f32x4_t o;
#pragma unroll
            for (int d = 0; d < 4; ++d) o[d] = acc[4 * c + d][j][i];
            *reinterpret_cast<f32x4_t*>(slot + at + 4 * c) = o;
          }
        }
      }
    } else {
      // rows 4 q + i: R's j0 + 16 j + 4 q + i; column l16: columns col + c
      const int jr = j0 + j * 16 + q * 4;
      if (jr >= R || col >= C) continue;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const int64_t at = static_cast<int64_t>(col + c) * R + jr;
        if (whole) {
          u32x2 o;
          o[0] = bf16x2_of(scale * acc[c][j][0], scale * acc[c][j][1]);
          o[1] = bf16x2_of(scale * acc[c][j][2], scale * acc[c][j][3]);
          *reinterpret_cast<u32x2*>(out + at) = o;
        } else {
          *reinterpret_cast<f32x4_t*>(slot + at) = acc[c][j];
        }
      }
    }
  }
}

template <int JT>
__global__ __launch_bounds__(kBlock) void k_lora_weight_grad(WeightGradArgs a) {
  __shared__ __align__(16) uint16_t s_hi[JT * 16][kRowPitch];
  __shared__ __align__(16) uint16_t s_lo[JT * 16][kRowPitch];
  if (!layout_current(a.status, a.generation)) return;
  const Tile t = find_tile(a.counts, a.E, a.shift, static_cast<int>(blockIdx.x));
  if (t.e < 0) return;
  const int nca = (a.C[0] + 4 * kCols - 1) / (4 * kCols);
  const int cb = static_cast<int>(blockIdx.y);
  if (cb < nca) weight_grad<JT, 0>(a, t, cb, static_cast<int>(blockIdx.z), s_hi, s_lo);
  else weight_grad<JT, 1>(a, t, cb - nca, static_cast<int>(blockIdx.z), s_hi, s_lo);
}

// Experts of several chunks: their partial gradients added in chunk order,
// scaled and rounded once.  Experts without rows: zeros.  Block (e, part).
__global__ __launch_bounds__(kBlock) void k_lora_join(WeightGradArgs a) {
  if (!layout_current(a.status, a.generation)) return;
  const int e = static_cast<int>(blockIdx.x);
  const int n = (a.counts[e] + (1 << a.shift) - 1) >> a.shift;
  if (n == 1) return;
  int64_t first = 0;
  if (n > 1) {
    // tiles of experts with several tiles before this one
    __shared__ int s_many[kWavesPerBlock];
    int many = 0;
    for (int i = threadIdx.x; i < e; i += kBlock) {
      const int c = (a.counts[i] + (1 << a.shift) - 1) >> a.shift;
      many += c > 1 ? c : 0;
    }
#pragma unroll
    for (int off = kWave / 2; off > 0; off >>= 1) many += __shfl_xor(many, off, kWave);
    if ((threadIdx.x & (kWave - 1)) == 0) s_many[threadIdx.x / kWave] = many;
    __syncthreads();
    for (int w = 0; w < kWavesPerBlock; ++w) first += s_many[w];
  }
  const float scale = a.scales ? a.scales[e] : 1.0f;
  const int64_t size_a = static_cast<int64_t>(a.R) * a.C[0];
  const int64_t size_b = static_cast<int64_t>(a.R) * a.C[1];
  const int64_t quads = a.slot_size / 4;  // R is a multiple of 8
  for (int64_t i = static_cast<int64_t>(blockIdx.y) * kBlock + threadIdx.x; i < quads;
       i += static_cast<int64_t>(gridDim.y) * kBlock) {
    f32x4_t sum = f32x4_t{};
    for (int c = 0; c < n; ++c)
      sum += *reinterpret_cast<const f32x4_t*>(a.slots + (first + c) * a.slot_size + 4 * i);
    u32x2 o;
    o[0] = bf16x2_of(scale * sum[0], scale * sum[1]);
    o[1] = bf16x2_of(scale * sum[2], scale * sum[3]);
    if (n == 0) o = u32x2{0u, 0u};
    uint16_t* out = 4 * i < size_a ? a.out[0] + e * size_a + 4 * i : a.out[1] + e * size_b + (4 * i - size_a);
    *reinterpret_cast<u32x2*>(out) = o;
  }
}

// ------------------------------------------------------------------ launches
template <bool KMAJOR>
hipError_t shrink(const ShrinkArgs& a, const LoraGeom& g, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(g.max_tiles), static_cast<unsigned>(a.S));
  const int rt = (a.R + 15) / 16;
  auto go = [&](auto k1, auto k2, auto k4) {
    if (g.row_tiles == 1) k1<<<grid, kBlock, 0, s>>>(a);
    else if (g.row_tiles == 2) k2<<<grid, kBlock, 0, s>>>(a);
    else k4<<<grid, kBlock, 0, s>>>(a);
    return hipGetLastError();
  };
  if (rt <= 1) return go(k_lora_shrink<1, 1, KMAJOR>, k_lora_shrink<1, 2, KMAJOR>, k_lora_shrink<1, 4, KMAJOR>);
  if (rt <= 2) return go(k_lora_shrink<2, 1, KMAJOR>, k_lora_shrink<2, 2, KMAJOR>, k_lora_shrink<2, 4, KMAJOR>);
  if (rt <= 4) return go(k_lora_shrink<4, 1, KMAJOR>, k_lora_shrink<4, 2, KMAJOR>, k_lora_shrink<4, 4, KMAJOR>);
  return go(k_lora_shrink<8, 1, KMAJOR>, k_lora_shrink<8, 2, KMAJOR>, k_lora_shrink<8, 4, KMAJOR>);
}

template <bool JMAJOR>
hipError_t expand(const ExpandArgs& a, const LoraGeom& g, hipStream_t s) {
  const unsigned ncb = static_cast<unsigned>((a.N + 4 * kCols - 1) / (4 * kCols));
  const dim3 grid(static_cast<unsigned>(g.max_tiles), ncb + (a.map && a.base != a.out ? 1u : 0u));
  auto go = [&](auto k1, auto k2, auto k4) {
    if (g.row_tiles == 1) k1<<<grid, kBlock, 0, s>>>(a);
    else if (g.row_tiles == 2) k2<<<grid, kBlock, 0, s>>>(a);
    else k4<<<grid, kBlock, 0, s>>>(a);
    return hipGetLastError();
  };
  if (a.R <= 16)
    return go(k_lora_expand<1, 1, true, JMAJOR>, k_lora_expand<1, 2, true, JMAJOR>, k_lora_expand<1, 4, true, JMAJOR>);
  if (a.R <= 32)
    return go(k_lora_expand<1, 1, false, JMAJOR>, k_lora_expand<1, 2, false, JMAJOR>, k_lora_expand<1, 4, false, JMAJOR>);
  if (a.R <= 64)
    return go(k_lora_expand<2, 1, false, JMAJOR>, k_lora_expand<2, 2, false, JMAJOR>, k_lora_expand<2, 4, false, JMAJOR>);
  return go(k_lora_expand<4, 1, false, JMAJOR>, k_lora_expand<4, 2, false, JMAJOR>, k_lora_expand<4, 4, false, JMAJOR>);
}

int64_t up16(int64_t n) { return (n + 15) / 16 * 16; }

ShrinkArgs shrink_args(const LoraArgs& a, const LoraGeom& g) {
  ShrinkArgs s = {};
  s.R = a.R;
  s.E = a.E;
  s.stride = g.rows * a.R;
  s.counts = a.counts;
  s.offsets = a.offsets;
  s.status = a.status;
  s.generation = a.generation;
  return s;
}

ExpandArgs expand_args(const LoraArgs& a, const LoraGeom& g) {
  ExpandArgs x = {};
  x.stride = g.rows * a.R;
  x.scales = a.scales;
  x.base = a.base;
  x.ldbase = a.ldbase;
  x.out = a.out;
  x.ldout = a.ldout;
  x.map = a.omap;
  x.slot = a.slot;
  x.T = a.T;
  x.R = a.R;
  x.E = a.E;
  x.counts = a.counts;
  x.offsets = a.offsets;
  x.status = a.status;
  x.generation = a.generation;
  return x;
}

}  // namespace

LoraGeom lora_geom(int64_t rows, int E, int H, int N, int R, bool backward) {
  LoraGeom g = {};
  g.rows = rows;
  const int64_t used = rows < E ? rows : E;  // experts with rows, at most
  const int64_t avg = rows / E;
  g.row_tiles = avg >= 64 ? 4 : avg >= 32 ? 2 : 1;
  g.max_tiles = rows / (16 * g.row_tiles) + used;
  // enough blocks for every CU twice, of at least 256 of the contraction
  auto splits = [&](int C) {
    int64_t s = 512 / (g.max_tiles > 0 ? g.max_tiles : 1);
    const int64_t most = C / 256 > 0 ? C / 256 : 1;
    if (s > most) s = most;
    return static_cast<int>(s < 1 ? 1 : s > 16 ? 16 : s);
  };
  g.split_x = splits(H);
  g.u_bytes = static_cast<size_t>(up16(g.split_x * rows * R * 4));
  if (backward) {
    g.split_g = splits(N);
    g.v_bytes = static_cast<size_t>(up16(g.split_g * rows * R * 4));
    g.chunk_shift = 6;
    while ((static_cast<int64_t>(32) << g.chunk_shift) < rows) ++g.chunk_shift;
    g.max_chunks = (rows >> g.chunk_shift) + used;
    // an expert of several chunks has more than one chunk of rows, so its
    // chunks are fewer than twice its rows over the chunk size
    g.slots = 2 * (rows >> g.chunk_shift);
    g.slot_bytes = static_cast<size_t>(g.slots) * R * (static_cast<size_t>(H) + N) * 4;
  }
  return g;
}

hipError_t launch_lora(const LoraArgs& a, const LoraGeom& g, hipStream_t s) {
  ShrinkArgs sh = shrink_args(a, g);
  sh.in = a.x;
  sh.ld = a.ldx;
  sh.map = a.xmap;
  sh.w = a.a;
  sh.C = a.H;
  sh.part = a.u;
  sh.S = g.split_x;
  hipError_t err = shrink<false>(sh, g, s);
  if (err != hipSuccess) return err;
  ExpandArgs ex = expand_args(a, g);
  ex.part = a.u;
  ex.S = g.split_x;
  ex.w = a.b;
  ex.N = a.N;
  return expand<false>(ex, g, s);
}

namespace {

// u, v and from v the rows' gradients.
hipError_t row_gradients(const LoraArgs& a, const LoraGeom& g, hipStream_t s) {
  ShrinkArgs sh = shrink_args(a, g);
  sh.in = a.x;
  sh.ld = a.ldx;
  sh.map = a.xmap;
  sh.w = a.a;
  sh.C = a.H;
  sh.part = a.u;
  sh.S = g.split_x;
  hipError_t err = shrink<false>(sh, g, s);
  if (err != hipSuccess) return err;
  sh.in = a.go;
  sh.ld = a.ldgo;
  sh.map = a.omap;
  sh.w = a.b;
  sh.C = a.N;
  sh.part = a.v;
  sh.S = g.split_g;
  err = shrink<true>(sh, g, s);
  if (err != hipSuccess) return err;
  ExpandArgs ex = expand_args(a, g);
  ex.part = a.v;
  ex.S = g.split_g;
  ex.w = a.a;
  ex.N = a.H;
  return expand<true>(ex, g, s);
}

}  // namespace

hipError_t launch_lora_backward(const LoraArgs& a, const LoraGeom& g, hipStream_t s) {
  if (g.rows > 0) {
    const hipError_t err = row_gradients(a, g, s);
    if (err != hipSuccess) return err;
  }
  WeightGradArgs w = {};
  w.in[0] = a.x;
  w.ld[0] = a.ldx;
  w.map[0] = a.xmap;
  w.C[0] = a.H;
  w.part[0] = a.v;
  w.S[0] = g.split_g;
  w.out[0] = a.ga;
  w.in[1] = a.go;
  w.ld[1] = a.ldgo;
  w.map[1] = a.omap;
  w.C[1] = a.N;
  w.part[1] = a.u;
  w.S[1] = g.split_x;
  w.out[1] = a.gb;
  w.stride = g.rows * a.R;
  w.slots = a.slots;
  w.slot_size = static_cast<int64_t>(a.R) * (static_cast<int64_t>(a.H) + a.N);
  w.scales = a.scales;
  w.R = a.R;
  w.E = a.E;
  w.shift = g.chunk_shift;
  w.counts = a.counts;
  w.offsets = a.offsets;
  w.status = a.status;
  w.generation = a.generation;
  const int per = 4 * kCols;
  const unsigned cb = static_cast<unsigned>((a.H + per - 1) / per + (a.N + per - 1) / per);
  const unsigned chunks = static_cast<unsigned>(g.max_chunks);
  if (chunks > 0) {
    if (a.R <= 16) k_lora_weight_grad<1><<<dim3(chunks, cb, 1), kBlock, 0, s>>>(w);
    else if (a.R <= 32) k_lora_weight_grad<2><<<dim3(chunks, cb, 1), kBlock, 0, s>>>(w);
    else k_lora_weight_grad<4><<<dim3(chunks, cb, a.R <= 64 ? 1 : 2), kBlock, 0, s>>>(w);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  int64_t parts = w.slot_size / 4 / kBlock / 4;  // 4 quads per thread
  parts = parts < 1 ? 1 : parts > 256 ? 256 : parts;
  k_lora_join<<<dim3(static_cast<unsigned>(a.E), static_cast<unsigned>(parts)), kBlock, 0, s>>>(w);
  return hipGetLastError();
}

}  // namespace ep
