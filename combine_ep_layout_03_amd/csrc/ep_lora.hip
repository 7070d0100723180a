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
// u and v enter the second product as three bf16 parts of 8 significand bits
// each, which together are the fp32 value: nothing is rounded between the two
// products.  (With two parts, 16 bits, up to 0.2% of the results were rounded
// the other way; the third costs 72 us instead of 69 in the weight gradients of
// 16,384 rows x 4096 -> 2048, rank 32, 179 instead of 162 at rank 128, and
// nothing that shows elsewhere.)
//
// A matrix whose contraction index is not contiguous in memory is transposed
// in registers: a lane loads 8 rows of 8 columns and forms, with 32 byte
// permutes, the 8 operands that hold one column each; operand column l of
// product c then stands for column 8 l + c.  That also leaves each lane with 8
// neighbouring columns of the result, and 16 lanes with 256 contiguous bytes.
//
// Loads and stores keep neighbouring lanes on neighbouring 16 bytes: a load
// whose neighbouring lanes lie in different rows costs the L1 one access per
// lane instead of one per 64 bytes, and measured 1.5 to 2 times slower.
//
// Measured (a plain copy: 4.98 TB/s):
//     16,384 rows, 4096 -> 2048, rank 32, 64 experts, in expert order
//       forward   shrink 32 us (x 134 MB), expand 36 us (base and out 134 MB)
//       backward  shrink 55 us (x and g 201 MB), gradients 75 us (x and g again,
//                 and dx, 134 MB), join 5 us
//     the same at rank 128: backward shrink 148 us, gradients 190 us, join 9 us
//     8111 tokens, 7168 -> 2048, rank 64, 10% without an adapter
//       forward   shrink 27 us (x 105 MB), expand 19 us (base and out 66 MB);
//                 rank 128: 49 and 29 us
//     61 tokens, 4096 -> 4096, rank 16, 48 adapters: 5.7 + 5.5 us; 509 tokens,
//       rank 8, backward: 7.2 + 9.9 + 4.0 us.  Launch, tile search and three
//       dependent loads are most of these.
// At their peak rate the matrix units need a tenth of a kernel's time up to rank
// 32 and a fifth at rank 128: memory's latency and rate bound the long ones,
// above rank 64 the L2's too, as a block keeps few rows of each matrix it reads.
#include <type_traits>

#include "ep_layer.h"

namespace ep {

namespace {

constexpr int kCols = 128;  // columns of one wave
constexpr int kXcds = 8;
constexpr int kMaxSplits = 4;  // splits of a contraction over blocks

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ f32x4_t mfma(u32x4 a, u32x4 b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                 __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

__device__ __forceinline__ u32x4 load16(const uint16_t* p) { return *reinterpret_cast<const u32x4*>(p); }
// STREAM: non-temporal, for the only read of rows that the caches could not keep.
template <bool STREAM>
__device__ __forceinline__ u32x4 load_row16(const uint16_t* p) {
  return STREAM ? __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p)) : load16(p);
}

// LDS that one wave alone uses is accessed in order: only the compiler has to
// keep the order.
__device__ __forceinline__ void wave_lds_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// f as the sum of three bf16 parts, each the leading 8 significand bits of what
// the ones before leave: exact, but for bits below bf16's smallest denormal,
// 2^-133.  The parts have f's sign or are zero, so no sum of them overflows
// that f does not, and the largest fp32 stays finite.  Every part of an
// infinity or NaN is that infinity or a NaN.
constexpr int kParts = 3;
__device__ __forceinline__ void split(float f, uint16_t (&part)[kParts]) {
  const uint32_t b = __float_as_uint(f);
  const float r = f - __uint_as_float(b & 0xffff0000u);
  const uint32_t c = __float_as_uint(r);
  const float last = r - __uint_as_float(c & 0xffff0000u);
  const bool finite = (b & 0x7f800000u) != 0x7f800000u;
  // what a NaN's upper half has lost must not make it an infinity
  part[0] = static_cast<uint16_t>(f == f ? b >> 16 : 0x7fc0u);
  part[1] = finite ? static_cast<uint16_t>(c >> 16) : part[0];
  part[2] = finite ? static_cast<uint16_t>(__float_as_uint(last) >> 16) : part[0];
}

// Where the other factor is infinite, a part of zero makes NaN of what the formula
// has infinite: there the second and third part of a value that is not 0 are
// replaced, if zero, by the smallest denormal with its sign (the matrix
// instructions take denormals as they are).  To be called by the whole block,
// after a barrier and before another, for the first `count` elements of each
// part in LDS.
__device__ __forceinline__ void fill_parts(uint16_t* s_part, int part_size, int count) {
  for (int i = threadIdx.x; i < count; i += static_cast<int>(blockDim.x)) {
    const uint16_t first = s_part[i];
#pragma unroll
    for (int d = 1; d < kParts; ++d) {
      uint16_t& p = s_part[d * part_size + i];
      if ((first & 0x7fff) != 0 && (p & 0x7fff) == 0) p = (first & 0x8000) | 1;
    }
  }
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

// Tile `index` of the experts' rows, cut into tiles of 2^shift rows in expert
// order.  BY_XCD: blocks go round-robin over the 8 XCDs, so index b stands for
// tile (b % 8) * ceil(tiles / 8) + b / 8, and neighbouring tiles, which share an
// expert's matrix, meet in one L2.  Every lane calls it with the same arguments.
struct Tile {
  int e;      // expert, -1: no such tile
  int row0;   // first row
  int nrows;  // rows of the tile
  int slot;   // where an expert of several tiles keeps this tile's partial
              // result: the number of such experts' tiles before; -1 for an expert of one tile
};
__device__ __forceinline__ int wave_inclusive_scan(int v) {
  // within rows of 16 lanes, then row 0's total to row 1 and row 2's to row 3,
  // then the lower half's to the upper
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true);  // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true);  // row_shr:2
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true);  // row_shr:4
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, true);  // row_shr:8
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // row_bcast:15
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // row_bcast:31
  return v;
}
template <bool BY_XCD>
__device__ __forceinline__ Tile find_tile(const int32_t* counts, const int32_t* offsets, int E, int shift,
                                          int index) {
  const int lane = threadIdx.x & (kWave - 1);
  const int per = (E + kWave - 1) / kWave;  // experts per lane, at most 16
  auto tiles_of = [&](int c) { return (c + (1 << shift) - 1) >> shift; };
  int count = 0, sum = 0, many = 0;
  for (int i = 0; i < per; ++i) {
    const int e = lane * per + i;
    count = e < E ? counts[e] : 0;
    const int n = tiles_of(count);
    sum += n;
    many += n > 1 ? n : 0;
  }
  int incl = wave_inclusive_scan(sum), incl_many = wave_inclusive_scan(many);
  Tile t = {-1, 0, 0, -1};
  int tile = index;
  if (BY_XCD) {
    const int per_xcd = (readlane(incl, kWave - 1) + kXcds - 1) / kXcds;
    if (index / kXcds >= per_xcd) return t;
    tile = (index % kXcds) * per_xcd + index / kXcds;
  }
  uint64_t after = ballot(incl > tile);
  if (after == 0) return t;
  int L = static_cast<int>(__builtin_ctzll(after));
  int left = tile - readlane(incl - sum, L);
  int slot = readlane(incl_many - many, L);
  int e = L;
  if (per > 1) {  // the expert among the lane's
    const int first = L * per;
    count = lane < per && first + lane < E ? counts[first + lane] : 0;
    const int n = tiles_of(count);
    incl = wave_inclusive_scan(n);
    incl_many = wave_inclusive_scan(n > 1 ? n : 0);
    after = ballot(incl > left);
    L = static_cast<int>(__builtin_ctzll(after));
    slot += readlane(incl_many - (n > 1 ? n : 0), L);
    left -= readlane(incl - n, L);
    e = first + L;
  }
  count = readlane(count, L);
  t.e = e;
  t.row0 = offsets[e] + (left << shift);
  t.nrows = min(1 << shift, count - (left << shift));
  t.slot = count > (1 << shift) ? slot + left : -1;
  return t;
}

// A tile as the first kernel left it in the workspace for the later ones.
__device__ __forceinline__ Tile stored_tile(const int32_t* tiles, int block) {
  const int32_t* p = tiles + 4 * static_cast<int64_t>(block);
  return {__builtin_amdgcn_readfirstlane(p[0]), __builtin_amdgcn_readfirstlane(p[1]),
          __builtin_amdgcn_readfirstlane(p[2]), __builtin_amdgcn_readfirstlane(p[3])};
}
__device__ __forceinline__ void store_tile(int32_t* tiles, int block, const Tile& t) {
  int32_t* p = tiles + 4 * static_cast<int64_t>(block);
  p[0] = t.e;
  p[1] = t.row0;
  p[2] = t.nrows;
  p[3] = t.slot;
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
  bool streamed;  // the rows are not read again and too many for the caches
  // tiles of the kernels to come, written by two waves of split 0's blocks
  int32_t* expand_tiles;  // num_expand == 0: none
  int num_expand, expand_shift;
  int32_t* chunks;  // num_chunks == 0: none
  int num_chunks, chunk_shift;
  const int32_t* counts;
  const int32_t* offsets;
  int32_t* status;
  uint32_t generation;
};


// Block: one row tile (16 MT rows) and one split of the contraction, whose
// 64-wide pieces the NW waves take in turn, the next piece's loads in flight
// while one is multiplied.  The waves' sums are added in wave order.  Four
// waves a block: several blocks share a CU, and one's start and end hide
// behind another's loads; eight for tiles of 16 rows, which are few (61 rows x
// 4096, rank 16: 4.9 us against 5.4 with four).  Two pieces of x in flight
// instead of one: 34 us against 31 at 8111 rows x 7168, rank 64 (the registers
// cost a resident block).
template <int RT, int MT, int NW, bool KMAJOR>
struct ShrinkLds {
  // one wave's sums
  static constexpr int kPitch = RT * 16 + 4;
  static constexpr int kRed = MT * 16 * kPitch;
  // k-major: 32 KiB of the matrix as 8 x 8 blocks, transposed: RT * 16 rows of
  // kStage (and 8, so that rows start on different banks)
  static constexpr int kBlocks = 256;
  static constexpr int kStage = kBlocks * 64 / (RT * 16);
  static constexpr int kWBytes = KMAJOR ? RT * 16 * (kStage + 8) * 2 : 0;
  static constexpr int kXBytes = NW * (KMAJOR ? MT : MT + RT) * 2048;
  static constexpr int kBytes = NW * kRed * 4 > kWBytes + kXBytes ? NW * kRed * 4 : kWBytes + kXBytes;
};

template <int RT, int MT, int NW, bool KMAJOR, bool STREAM>
__device__ __forceinline__ void shrink(const ShrinkArgs& a, char* s_mem) {
  using Lds = ShrinkLds<RT, MT, NW, KMAJOR>;
  constexpr int kShift = MT == 1 ? 4 : MT == 2 ? 5 : 6;
  constexpr int kPitch = Lds::kPitch, kRed = Lds::kRed, kStage = Lds::kStage, kWBytes = Lds::kWBytes;
  if (!layout_current(a.status, a.generation)) return;
  if (static_cast<int>(blockIdx.y) >= a.S) return;
  const int block = static_cast<int>(blockIdx.x);
  const Tile t = find_tile<true>(a.counts, a.offsets, a.E, kShift, block);
  static_assert(NW > 2, "waves 1 and 2 write the tables");
  if (blockIdx.y == 0) {
    const int w = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
    auto table = [&](int32_t* out, int n, int shift) {
      for (int b = block; b < n; b += static_cast<int>(gridDim.x)) {
        const Tile c = find_tile<false>(a.counts, a.offsets, a.E, shift, b);
        if ((threadIdx.x & (kWave - 1)) == 0) store_tile(out, b, c);
      }
    };
    if (w == 1) table(a.expand_tiles, a.num_expand, a.expand_shift);
    if (w == 2) table(a.chunks, a.num_chunks, a.chunk_shift);
  }
  if (t.e < 0) return;  // the whole block
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
  const int l16 = lane & 15, q = lane >> 4;

  // A wave's 64-wide piece of its rows passes through LDS: loaded 8 rows of a
  // whole 128-byte line per instruction, read as operands.  16-byte unit u of
  // row r lies at r * 8 + (u ^ ((r >> 1) & 7)), which keeps the reads of 16 rows
  // at one u on distinct banks.
  const int l8 = lane >> 3, unit = lane & 7;
  const uint16_t* xr[2 * MT];
#pragma unroll
  for (int n = 0; n < 2 * MT; ++n) {
    const int r = t.row0 + min(n * 8 + l8, t.nrows - 1);  // rows past the tile repeat its last
    xr[n] = a.in + static_cast<int64_t>(a.map ? a.map[r] : r) * a.ld + unit * 8;
  }
  const uint16_t* w = a.w + static_cast<int64_t>(t.e) * a.R * a.C;
  u32x4* s_x = reinterpret_cast<u32x4*>(s_mem + kWBytes) + wave * (KMAJOR ? MT : MT + RT) * 128;
  u32x4* s_wt = s_x + MT * 128;
  auto put = [&](u32x4* to, int n, u32x4 v) __attribute__((always_inline)) {
    to[(n * 8 + l8) * 8 + (unit ^ ((n * 4 + (lane >> 4)) & 7))] = v;
  };
  auto get = [&](const u32x4* from, int m, int h) __attribute__((always_inline)) {
    return from[(m * 16 + l16) * 8 + ((h * 4 + q) ^ ((l16 >> 1) & 7))];
  };
  f32x4_t acc[MT][RT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < RT; ++j) acc[m][j] = f32x4_t{};

  const int pieces = (a.C + 63) / 64;
  const int s = static_cast<int>(blockIdx.y);
  const int p0 = static_cast<int>(static_cast<int64_t>(pieces) * s / a.S);
  const int p1 = static_cast<int>(static_cast<int64_t>(pieces) * (s + 1) / a.S);

  // Elements past C (a multiple of 8) are zeros, in both operands: loaded from
  // the last 8, replaced when they are put into LDS.
  auto place = [&](int p) __attribute__((always_inline)) { return min(p * 64, a.C - 8 - unit * 8); };
  auto past = [&](int p) __attribute__((always_inline)) { return p * 64 + unit * 8 >= a.C; };
  auto load_x = [&](int p, u32x4 (&x)[2 * MT]) __attribute__((always_inline)) {
#pragma unroll
    for (int n = 0; n < 2 * MT; ++n) x[n] = load_row16<STREAM>(xr[n] + place(p));
  };
  auto put_x = [&](int p, u32x4 (&x)[2 * MT]) __attribute__((always_inline)) {
#pragma unroll
    for (int n = 0; n < 2 * MT; ++n) put(s_x, n, past(p) ? u32x4{0u, 0u, 0u, 0u} : x[n]);
  };
  if constexpr (!KMAJOR) {
    const uint16_t* wr = w + static_cast<int64_t>(l8) * a.C + unit * 8;
    auto load_w = [&](int p, u32x4 (&v)[2 * RT]) __attribute__((always_inline)) {
#pragma unroll
      for (int n = 0; n < 2 * RT; ++n)  // rows past R (a multiple of 8) repeat the last 8, and are dropped
        v[n] = load16(wr + static_cast<int64_t>(min(n * 8, a.R - 8)) * a.C + place(p));
    };
    u32x4 x[2 * MT], v[2 * RT];
    int p = p0 + wave;
    if (p < p1) {
      load_x(p, x);
      load_w(p, v);
    }
    while (p < p1) {
      wave_lds_sync();  // the last piece's operands are read
      put_x(p, x);
#pragma unroll
      for (int n = 0; n < 2 * RT; ++n) put(s_wt, n, past(p) ? u32x4{0u, 0u, 0u, 0u} : v[n]);
      wave_lds_sync();
      p += NW;
      if (p < p1) {
        load_x(p, x);
        load_w(p, v);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        u32x4 wv[RT];
#pragma unroll
        for (int j = 0; j < RT; ++j) wv[j] = get(s_wt, j, h);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const u32x4 xv = get(s_x, m, h);
#pragma unroll
          for (int j = 0; j < RT; ++j) acc[m][j] = mfma(wv[j], xv, acc[m][j]);
        }
      }
    }
  } else {
    uint16_t* s_w = reinterpret_cast<uint16_t*>(s_mem);
    constexpr int kWPitch = kStage + 8;
    const int k_end = min(p1 * 64, a.C);
    for (int k0 = p0 * 64; k0 < k_end; k0 += kStage) {
      u32x4 x[2 * MT];
      int k = k0 + wave * 64;
      const int q1 = min(k0 + kStage, k_end);
      if (k < q1) load_x(k / 64, x);
      // 8 x 8 blocks (8 k, 8 of R) transposed in registers, k contiguous in LDS
      if (k0 > p0 * 64) __syncthreads();
      for (int b = threadIdx.x; b < Lds::kBlocks; b += NW * kWave) {
        const int jb = b % (RT * 2), kb = b / (RT * 2);
        const int kk = k0 + kb * 8;
        u32x4 v[8], c[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[i] = u32x4{0u, 0u, 0u, 0u};
          if (kk < k_end && jb * 8 < a.R) v[i] = load16(w + static_cast<int64_t>(kk + i) * a.R + jb * 8);
        }
        columns(v, c);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *reinterpret_cast<u32x4*>(s_w + (jb * 8 + i) * kWPitch + kb * 8) = c[i];
      }
      __syncthreads();
      for (; k < q1; k += NW * 64) {
        wave_lds_sync();
        put_x(k / 64, x);
        wave_lds_sync();
        if (k + NW * 64 < q1) load_x(k / 64 + NW, x);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          u32x4 v[RT];
#pragma unroll
          for (int j = 0; j < RT; ++j)
            v[j] = *reinterpret_cast<const u32x4*>(s_w + (j * 16 + l16) * kWPitch + k - k0 + h * 32 + q * 8);
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const u32x4 xv = get(s_x, m, h);
#pragma unroll
            for (int j = 0; j < RT; ++j) acc[m][j] = mfma(v[j], xv, acc[m][j]);
          }
        }
      }
    }
  }
  __syncthreads();  // the operands' LDS is reused
  float* red = reinterpret_cast<float*>(s_mem);
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < RT; ++j)
      *reinterpret_cast<f32x4_t*>(red + wave * kRed + (m * 16 + l16) * kPitch + j * 16 + q * 4) = acc[m][j];
  __syncthreads();
  float* out = a.part + s * a.stride + static_cast<int64_t>(t.row0) * a.R;
  const int quads = a.R / 4;
  for (int i = threadIdx.x; i < t.nrows * quads; i += NW * kWave) {
    const float* p = red + (i / quads) * kPitch + i % quads * 4;
    f32x4_t f = *reinterpret_cast<const f32x4_t*>(p);
#pragma unroll
    for (int n = 1; n < NW; ++n) f += *reinterpret_cast<const f32x4_t*>(p + n * kRed);
    *reinterpret_cast<f32x4_t*>(out + 4 * i) = f;
  }
}

template <int RT, int MT, int NW>
__global__ __launch_bounds__(NW* kWave) void k_lora_shrink(ShrinkArgs a) {
  __shared__ __align__(16) char s_mem[ShrinkLds<RT, MT, NW, false>::kBytes];
  if (a.streamed) shrink<RT, MT, NW, false, true>(a, s_mem);
  else shrink<RT, MT, NW, false, false>(a, s_mem);
}

// u and v of the backward pass in one launch: 509 rows x 4096, rank 8: 7.1 us
// against 6.0 and 5.5 us in two; 16,384 rows x 4096 -> 2048, rank 32: 55 us
// against 40 and 23 us.
template <int RT, int MT, int NW>
__global__ __launch_bounds__(NW* kWave) void k_lora_shrink_both(ShrinkArgs u, ShrinkArgs v) {
  constexpr int kU = ShrinkLds<RT, MT, NW, false>::kBytes, kV = ShrinkLds<RT, MT, NW, true>::kBytes;
  __shared__ __align__(16) char s_mem[kU > kV ? kU : kV];
  if (blockIdx.z == 0) shrink<RT, MT, NW, false, false>(u, s_mem);
  else shrink<RT, MT, NW, true, false>(v, s_mem);
}

// ------------------------------------------------------------------- expand
struct ExpandArgs {
  const float* part;  // [S, rows, R]
  int64_t stride;
  int S;  // 1, 2 or 4
  const uint16_t* w;  // [E, N, R], or (JMAJOR) [E, R, N]
  const float* scales;
  const uint16_t* base;
  int64_t ldbase;
  uint16_t* out;
  int64_t ldout;
  const int32_t* map;
  const int32_t* slot;
  int64_t T;
  int N, R;
  const int32_t* tiles;
  int64_t num_tiles;
  int32_t* status;
  uint32_t generation;
};

// Rows of out that belong to no selection (token rows only): base's row, or
// zeros.  A block takes 8 tokens from t0, then from t0 + step, ...; requests
// without an adapter are runs of tokens, so a wave takes no more than two at a
// time (with eight, 10% of 8111 tokens x 2048 took 36 us, the rest of the kernel 26).
constexpr int kCopyTokens = 8;
__device__ __forceinline__ void copy_unselected(const ExpandArgs& a, int64_t t0, int64_t step) {
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
  constexpr int kEach = kCopyTokens / kWavesPerBlock;
  for (; t0 < a.T; t0 += step) {
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int64_t t = t0 + wave * kEach + i;
      if (t >= a.T || a.slot[t] >= 0) continue;
      for (int n0 = lane * 8; n0 < a.N; n0 += 4 * kWave * 8) {
        u32x4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          v[k] = u32x4{0u, 0u, 0u, 0u};
          const int n = n0 + k * kWave * 8;
          if (a.base && n < a.N) v[k] = load16(a.base + t * a.ldbase + n);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int n = n0 + k * kWave * 8;
          if (n < a.N) *reinterpret_cast<u32x4*>(a.out + t * a.ldout + n) = v[k];
        }
      }
    }
  }
}

// Quads (4 neighbouring elements) of u or v, the S splits added in order,
// passed on one by one: put(i, quad) for every i of the block's threads below
// `count`, where at(i) is the quad's place in a split, or null for zeros.  Four
// quads' loads are in flight together.
template <int S, typename At, typename Put>
__device__ __forceinline__ void joined_quads(int count, int64_t stride, At at, Put put) {
  constexpr int kBatch = 4;
  const int nt = static_cast<int>(blockDim.x);
  for (int i0 = threadIdx.x; i0 < count; i0 += kBatch * nt) {
    f32x4_t f[kBatch][S];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const float* p = i0 + b * nt < count ? at(i0 + b * nt) : nullptr;
#pragma unroll
      for (int s = 0; s < S; ++s) {
        f[b][s] = f32x4_t{};
        if (p) f[b][s] = *reinterpret_cast<const f32x4_t*>(p + s * stride);
      }
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (i0 + b * nt >= count) continue;
      f32x4_t sum = f[b][0];
#pragma unroll
      for (int s = 1; s < S; ++s) sum += f[b][s];
      put(i0 + b * nt, sum);
    }
  }
}
template <typename At, typename Put>
__device__ __forceinline__ void joined_quads(int S, int count, int64_t stride, At at, Put put) {
  if (S == 1) joined_quads<1>(count, stride, at, put);
  else if (S == 2) joined_quads<2>(count, stride, at, put);
  else joined_quads<4>(count, stride, at, put);
}
__device__ __forceinline__ void split4(f32x4_t f, u32x2 (&part)[kParts]) {
  uint16_t h[4][kParts];
#pragma unroll
  for (int i = 0; i < 4; ++i) split(f[i], h[i]);
#pragma unroll
  for (int d = 0; d < kParts; ++d)
#pragma unroll
    for (int i = 0; i < 2; ++i) part[d][i] = h[2 * i][d] | (static_cast<uint32_t>(h[2 * i + 1][d]) << 16);
}

// Rows of a result tile at most, as much of u as LDS holds comfortably.
__host__ __device__ constexpr int expand_rows(int KS) { return KS <= 2 ? 128 : 64; }

// Block: one tile of rows by 512 columns.  u's rows are put into LDS, as their
// bf16 parts; a wave holds its 128 columns of the matrix in registers and
// takes the tile's rows 16 at a time, the next 32 rows' base in flight.  The
// loop over whole groups has no condition inside: memory operations complete in
// order, and with a load or store that may be skipped the compiler waits for
// all of them instead of counting.
template <int KS>
struct ExpandLds {
  static constexpr int kPitch = KS * 32 + 8;
  static constexpr int kStaged = expand_rows(KS);
  static constexpr int kPart = kStaged * kPitch;  // elements of one part
  static constexpr int kBytes = kParts * kPart * 2 + kStaged * 4 + kWavesPerBlock * 4;
};

template <int KS, bool JMAJOR>
__device__ __forceinline__ void expand(const ExpandArgs& a, int64_t index, int col_block, char* s_mem) {
  using Lds = ExpandLds<KS>;
  constexpr int kPitch = Lds::kPitch, kStaged = Lds::kStaged;
  uint16_t* const s_u = reinterpret_cast<uint16_t*>(s_mem);
  int* const s_row = reinterpret_cast<int*>(s_mem + kParts * Lds::kPart * 2);
  int* const s_infinite = s_row + kStaged;  // per wave: is an element of its columns?
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
  const Tile t = stored_tile(a.tiles, static_cast<int>(index));
  if (t.e < 0) return;
  const int n0 = (col_block * 4 + wave) * kCols;
  const int l16 = lane & 15, q = lane >> 4;
  const float scale = a.scales ? a.scales[t.e] : 1.0f;
  const uint16_t* w = a.w + static_cast<int64_t>(t.e) * a.R * a.N;

  // the rows' places in base and out; rows past the tile repeat its last
  for (int r = threadIdx.x; r < kStaged; r += kBlock) {
    const int at = t.row0 + min(r, t.nrows - 1);
    s_row[r] = a.map ? a.map[at] : at;
  }
  // Columns n .. n + 7 of this lane.  Lanes past N work on the last 8 columns
  // and store nothing; R's elements past R are zeros.
  const bool whole = n0 + kCols <= a.N;
  const bool inside = n0 + l16 * 8 < a.N;
  const int n = inside ? n0 + l16 * 8 : a.N - 8;
  u32x4 wv[KS][8];
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) {
    const int j = ks * 32 + q * 8;
    u32x4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = u32x4{0u, 0u, 0u, 0u};
      if (j < a.R) v[i] = JMAJOR ? load16(w + static_cast<int64_t>(j + i) * a.N + n)
                                 : load16(w + static_cast<int64_t>(n + i) * a.R + j);
    }
    if (JMAJOR) {
      columns(v, wv[ks]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) wv[ks][i] = v[i];
    }
  }
  u16x2 largest = {};  // magnitudes of its bits; infinities and NaN are 0x7f80 and more
#pragma unroll
  for (int ks = 0; ks < KS; ++ks)
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        largest = __builtin_elementwise_max(largest, __builtin_bit_cast(u16x2, wv[ks][i][c] & 0x7fff7fffu));
  const bool infinite = ballot(largest[0] >= 0x7f80 || largest[1] >= 0x7f80) != 0;
  if (lane == 0) s_infinite[wave] = infinite;
  constexpr int kQuads = KS * 8;  // of a row, the ones past R zeros
  const int groups = (t.nrows + 15) / 16;
  joined_quads(
      a.S, groups * 16 * kQuads, a.stride,
      [&](int i) -> const float* {
        const int r = i / kQuads, j = i % kQuads * 4;
        if (r >= t.nrows || j >= a.R) return nullptr;
        return a.part + static_cast<int64_t>(t.row0 + r) * a.R + j;
      },
      [&](int i, f32x4_t f) {
        const int r = i / kQuads, j = i % kQuads * 4;
        u32x2 part[kParts];
        split4(f, part);
#pragma unroll
        for (int d = 0; d < kParts; ++d)
          *reinterpret_cast<u32x2*>(s_u + d * Lds::kPart + r * kPitch + j) = part[d];
      });
  __syncthreads();
  if (s_infinite[0] | s_infinite[1] | s_infinite[2] | s_infinite[3]) {  // the whole block
    fill_parts(s_u, Lds::kPart, groups * 16 * kPitch);
    __syncthreads();
  }
  if (n0 >= a.N) return;

  // this lane's rows 4 q + i of group m
  auto rows = [&](int m, int64_t (&row)[4]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) row[i] = s_row[m * 16 + q * 4 + i];
  };
  auto load_base = [&](const int64_t (&row)[4], u32x4 (&b)[4]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = load16(a.base + row[i] * a.ldbase + n);
  };
  auto result = [&](int m, const u32x4 (&base)[4], u32x4 (&o)[4]) __attribute__((always_inline)) {
    f32x4_t acc[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) acc[c] = f32x4_t{};
#pragma unroll
    for (int d = 0; d < kParts; ++d) {
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const int at = (m * 16 + l16) * kPitch + ks * 32 + q * 8;
        const u32x4 u = *reinterpret_cast<const u32x4*>(s_u + d * Lds::kPart + at);
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[c] = mfma(u, wv[ks][c], acc[c]);
      }
      // the parts one after the other: read together they cost registers, and with
      // KS == 2 some are spilled (8111 x 2048, rank 64: 22.1 us against 19.0)
      if (KS == 2) __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        o[i][c] = bf16x2_of(__builtin_fmaf(scale, acc[2 * c][i], bf16_lo(base[i][c])),
                            __builtin_fmaf(scale, acc[2 * c + 1][i], bf16_hi(base[i][c])));
  };
  // whole groups, two at a time
  const int pairs = whole ? t.nrows / 32 : 0;
  auto whole_groups = [&](auto with_base) __attribute__((always_inline)) {
    int64_t row[2][4];
    u32x4 base[2][4] = {};
#pragma unroll
    for (int d = 0; d < 2; ++d) {
      rows(d, row[d]);
      if (with_base.value) load_base(row[d], base[d]);
    }
    auto pair = [&](int p) __attribute__((always_inline)) {
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        u32x4 o[4];
        result(2 * p + d, base[d], o);
        int64_t next[4];
        rows(min(2 * p + d + 2, kStaged / 16 - 1), next);  // past the tile: its last row
        if (with_base.value) load_base(next, base[d]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          __builtin_nontemporal_store(o[i], reinterpret_cast<u32x4*>(a.out + row[d][i] * a.ldout + n));
          row[d][i] = next[i];
        }
      }
    };
    // the first apart: at the loop's head as many operations then are open on
    // entry as on return
    pair(0);
    for (int p = 1; p < pairs; ++p) pair(p);
  };
  if (pairs > 0) {
    if (a.base) whole_groups(std::integral_constant<bool, true>());
    else whole_groups(std::integral_constant<bool, false>());
  }
  for (int m = 2 * pairs; m < groups; ++m) {
    int64_t row[4];
    u32x4 base[4] = {}, o[4];
    rows(m, row);
    if (a.base) load_base(row, base);
    result(m, base, o);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (inside && m * 16 + q * 4 + i < t.nrows) *reinterpret_cast<u32x4*>(a.out + row[i] * a.ldout + n) = o[i];
  }
}

// Block `block` of `blocks`: the columns of a tile fastest, and after the tiles
// the rows of no selection.  (As further columns of the tiles the copies were on
// the same XCDs throughout wherever all columns together were a multiple of 8.)
template <int KS, bool JMAJOR>
__device__ __forceinline__ void expand_block(const ExpandArgs& a, unsigned block, unsigned blocks, char* s_mem) {
  const unsigned ncb = static_cast<unsigned>((a.N + 4 * kCols - 1) / (4 * kCols));
  const unsigned tiles = static_cast<unsigned>(a.num_tiles) * ncb;
  if (block < tiles) {
    expand<KS, JMAJOR>(a, block / ncb, static_cast<int>(block % ncb), s_mem);
  } else {
    copy_unselected(a, static_cast<int64_t>(block - tiles) * kCopyTokens,
                    static_cast<int64_t>(blocks - tiles) * kCopyTokens);
  }
}

template <int KS>
__global__ __launch_bounds__(kBlock) __attribute__((amdgpu_waves_per_eu(KS == 1 ? 3 : 2))) void k_lora_expand(
    ExpandArgs a) {
  __shared__ __align__(16) char s_mem[ExpandLds<KS>::kBytes];
  if (!layout_current(a.status, a.generation)) return;
  expand_block<KS, false>(a, blockIdx.x, gridDim.x, s_mem);
}

// --------------------------------------------------------- weight gradients
struct WeightGradArgs {
  // [0]: dA from x and v, [1]: dB from g and u
  const uint16_t* in[2];  // bf16 rows
  int64_t ld[2];
  const int32_t* map[2];
  int C[2];            // columns: H, N
  const float* part[2];  // v, u: [S, rows, R]
  int S[2];              // 1, 2 or 4
  int64_t stride;
  uint16_t* out[2];  // dA [E, R, H], dB [E, N, R]
  float* slots;
  int64_t slot_size;  // R * (H + N)
  const float* scales;
  int R, E, shift;
  bool streamed[2];
  const int32_t* chunks;
  const int32_t* counts;
  int32_t* status;
  uint32_t generation;
};

// Rows of u or v that a block holds in LDS at a time: 24 KiB as three bf16 parts.
__host__ __device__ constexpr int staged_rows(int JT) { return 256 / JT; }

// Block: one chunk of an expert's rows, 128 NW columns of x (or g), 16 JT of the
// R.  A wave takes 32 rows by 128 columns per step, one or two steps in flight, loaded
// without a condition (see k_lora_expand).  A lane ends with R's 4 q + i (i < 4)
// of each 16 and 8 neighbouring columns.
template <int JT, int NW, int B, bool STREAM>
__device__ __forceinline__ void weight_grad(const WeightGradArgs& a, const Tile& t, int cb, int jg, uint16_t* s_part,
                                            int* s_nan, int* s_row) {
  constexpr int kStaged = staged_rows(JT);
  constexpr int kPitch = kStaged + 8;
  constexpr int kPart = JT * 16 * kPitch;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
  const int l16 = lane & 15, q = lane >> 4;
  const int C = a.C[B], R = a.R;
  const int c0 = (cb * NW + wave) * kCols;
  const int col = c0 + l16 * 8;
  const int j0 = jg * JT * 16;

  // the rows' places; lanes past C work on its last 8 columns and store nothing
  for (int r = threadIdx.x; r < t.nrows; r += NW * kWave) s_row[r] = a.map[B] ? a.map[B][t.row0 + r] : t.row0 + r;
  __syncthreads();
  const uint16_t* in = a.in[B] + min(col, C - 8);
  auto load_step = [&](int r, u32x4 (&v)[8]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = load_row16<STREAM>(in + s_row[min(r + q * 8 + i, t.nrows - 1)] * a.ld[B]);
  };
  constexpr int kAhead = JT <= 2 ? 2 : 1;  // steps in flight, as registers allow
  f32x4_t acc[8][JT];
  // Infinities among the rows are found by what they do: where a result is NaN
  // the block starts again, with no part of zero.
  for (bool fill = false;; fill = true) {
#pragma unroll
    for (int c = 0; c < 8; ++c)
#pragma unroll
      for (int j = 0; j < JT; ++j) acc[c][j] = f32x4_t{};
    u32x4 v[kAhead][8];
#pragma unroll
    for (int d = 0; d < kAhead; ++d) load_step(32 * d, v[d]);
    for (int r0 = 0; r0 < t.nrows; r0 += kStaged) {
      if (r0 > 0) __syncthreads();  // the rows staged before are used up
      const int staged = min(kStaged, (t.nrows - r0 + 63) / 64 * 64);
      joined_quads(
          a.S[B], staged * JT * 4, a.stride,
          [&](int i) -> const float* {
            const int r = i / (JT * 4), j = j0 + i % (JT * 4) * 4;
            if (r0 + r >= t.nrows || j >= R) return nullptr;
            return a.part[B] + static_cast<int64_t>(t.row0 + r0 + r) * R + j;
          },
          [&](int i, f32x4_t f) {
            const int r = i / (JT * 4), j = i % (JT * 4) * 4;
#pragma unroll
            for (int d = 0; d < 4; ++d) {
              uint16_t part[kParts];
              split(f[d], part);
#pragma unroll
              for (int n = 0; n < kParts; ++n) s_part[n * kPart + (j + d) * kPitch + r] = part[n];
            }
          });
      __syncthreads();
      if (fill) {
        fill_parts(s_part, kPart, kPart);
        __syncthreads();
      }
      for (int r = 0; r < staged; r += 32 * kAhead) {
#pragma unroll
        for (int d = 0; d < kAhead; ++d) {
          const int at_row = r0 + r + d * 32;
          if (at_row + 32 > t.nrows) {  // rows past the chunk are zeros in both operands
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (at_row + q * 8 + i >= t.nrows) v[d][i] = u32x4{0u, 0u, 0u, 0u};
          }
          u32x4 cv[8];
          columns(v[d], cv);
          load_step(at_row + 32 * kAhead, v[d]);
#pragma unroll
          for (int j = 0; j < JT; ++j) {
            const int at = (j * 16 + l16) * kPitch + r + d * 32 + q * 8;
#pragma unroll
            for (int n = 0; n < kParts; ++n) {
              const u32x4 p = *reinterpret_cast<const u32x4*>(s_part + n * kPart + at);
#pragma unroll
              for (int c = 0; c < 8; ++c) acc[c][j] = mfma(p, cv[c], acc[c][j]);
            }
          }
        }
      }
    }
    if (fill) break;
    float sum = 0.0f;
#pragma unroll
    for (int c = 0; c < 8; ++c)
#pragma unroll
      for (int j = 0; j < JT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) sum += acc[c][j][i];
    const bool nan = ballot(sum != sum) != 0;
    if (lane == 0) s_nan[wave] = nan;
    __syncthreads();  // and the rows staged last are used up
    int again = 0;
#pragma unroll
    for (int i = 0; i < NW; ++i) again |= s_nan[i];
    if (again == 0) break;  // the whole block
  }

  const bool whole = t.slot < 0;
  const float scale = whole && a.scales ? a.scales[t.e] : 1.0f;
  uint16_t* out = a.out[B] + static_cast<int64_t>(t.e) * R * C;
  float* slot = whole ? nullptr
                      : a.slots + static_cast<int64_t>(t.slot) * a.slot_size +
                            (B == 0 ? 0 : static_cast<int64_t>(R) * a.C[0]);
#pragma unroll
  for (int j = 0; j < JT; ++j) {
    const int jr = j0 + j * 16 + q * 4;
    if (jr >= R || col >= C) continue;
    if (B == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t at = static_cast<int64_t>(jr + i) * C + col;
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

// dA, dB and dx in one launch: all need u and v and no more.  The first
// blocks take the weight gradients, the longer work, the others tiles of dx.
template <int KS, int JT>
__global__ __launch_bounds__(kBlock) __attribute__((amdgpu_waves_per_eu(2))) void k_lora_gradients(
    WeightGradArgs w, ExpandArgs x, unsigned weight_blocks) {
  constexpr int kParted = kParts * JT * 16 * (staged_rows(JT) + 8) * 2;
  constexpr int kW = kParted + kWavesPerBlock * 4, kX = ExpandLds<KS>::kBytes;
  __shared__ __align__(16) char s_mem[kW > kX ? kW : kX];
  extern __shared__ int s_row[];  // a chunk's rows
  if (!layout_current(w.status, w.generation)) return;
  if (blockIdx.x < weight_blocks) {
    constexpr int kPer = kWavesPerBlock * kCols;
    const int nca = (w.C[0] + kPer - 1) / kPer, ncb = (w.C[1] + kPer - 1) / kPer;
    const int jgs = (w.R + 16 * JT - 1) / (16 * JT);
    // columns fastest: blocks of a chunk read its rows together
    const int cols = nca + ncb;
    int at = static_cast<int>(blockIdx.x);
    const int cb = at % cols;
    at /= cols;
    const int jg = at % jgs;
    const Tile t = stored_tile(w.chunks, at / jgs);
    if (t.e < 0) return;
    uint16_t* const s_part = reinterpret_cast<uint16_t*>(s_mem);
    int* const s_nan = reinterpret_cast<int*>(s_mem + kParted);
    auto grad = [&](auto stream) __attribute__((always_inline)) {
      constexpr bool kStream = decltype(stream)::value;
      if (cb < nca) weight_grad<JT, kWavesPerBlock, 0, kStream>(w, t, cb, jg, s_part, s_nan, s_row);
      else weight_grad<JT, kWavesPerBlock, 1, kStream>(w, t, cb - nca, jg, s_part, s_nan, s_row);
    };
    // (KS == 4 is a rank above 64, whose rows are never streamed)
    if (KS < 4 && w.streamed[cb < nca ? 0 : 1]) grad(std::integral_constant<bool, KS < 4>());
    else grad(std::integral_constant<bool, false>());
  } else {
    expand_block<KS, true>(x, blockIdx.x - weight_blocks, gridDim.x - weight_blocks, s_mem);
  }
}

// Experts of several chunks: their partial gradients added in chunk order,
// scaled and rounded once.  Experts without rows: zeros.  Blocks (part of an
// expert's quads, of 4 elements; every 8th of these experts).
__global__ __launch_bounds__(kBlock) void k_lora_join(WeightGradArgs a) {
  __shared__ int s_e[1024], s_n[1024], s_first[1024];
  __shared__ int s_count;
  if (!layout_current(a.status, a.generation)) return;
  if (threadIdx.x < kWave) {
    const int lane = threadIdx.x;
    int count = 0, first = 0;  // experts to join; chunks of those with several
    for (int e0 = 0; e0 < a.E; e0 += kWave) {
      const int e = e0 + lane;
      const int n = e < a.E ? (a.counts[e] + (1 << a.shift) - 1) >> a.shift : 1;
      const uint64_t todo = ballot(n != 1);
      int incl = n > 1 ? n : 0;
#pragma unroll
      for (int off = 1; off < kWave; off <<= 1) {
        const int v = __shfl_up(incl, off, kWave);
        if (lane >= off) incl += v;
      }
      if (n != 1) {
        const int at = count + __popcll(todo & lanemask_lt());
        s_e[at] = e;
        s_n[at] = n;
        s_first[at] = first + incl - (n > 1 ? n : 0);
      }
      count += __popcll(todo);
      first += readlane(incl, kWave - 1);
    }
    if (lane == 0) s_count = count;
  }
  __syncthreads();
  const int64_t size_a = static_cast<int64_t>(a.R) * a.C[0];
  const int64_t size_b = static_cast<int64_t>(a.R) * a.C[1];
  const int64_t quads = a.slot_size / 4;  // R is a multiple of 8
  for (int k = static_cast<int>(blockIdx.y); k < s_count; k += static_cast<int>(gridDim.y)) {
    const int64_t e = s_e[k];
    const int n = s_n[k];
    const float scale = a.scales ? a.scales[e] : 1.0f;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x; i < quads;
         i += static_cast<int64_t>(gridDim.x) * kBlock) {
      f32x4_t sum = f32x4_t{};
      const float* p = a.slots + s_first[k] * a.slot_size + 4 * i;
#pragma unroll 8
      for (int c = 0; c < n; ++c) sum += *reinterpret_cast<const f32x4_t*>(p + c * a.slot_size);
      u32x2 o;
      o[0] = bf16x2_of(scale * sum[0], scale * sum[1]);
      o[1] = bf16x2_of(scale * sum[2], scale * sum[3]);
      if (n == 0) o = u32x2{0u, 0u};
      uint16_t* out = 4 * i < size_a ? a.out[0] + e * size_a + 4 * i : a.out[1] + e * size_b + (4 * i - size_a);
      *reinterpret_cast<u32x2*>(out) = o;
    }
  }
}

// ------------------------------------------------------------------ launches
template <int RT, int MT, int NW>
void shrink_mt(const ShrinkArgs& u, const ShrinkArgs* v, const LoraGeom& g, hipStream_t s) {
  const int splits = v && v->S > u.S ? v->S : u.S;
  const dim3 grid(static_cast<unsigned>(g.max_tiles), static_cast<unsigned>(splits), v ? 2 : 1);
  if (v) k_lora_shrink_both<RT, MT, NW><<<grid, NW * kWave, 0, s>>>(u, *v);
  else k_lora_shrink<RT, MT, NW><<<grid, NW * kWave, 0, s>>>(u);
}

template <int RT>
void shrink_rt(const ShrinkArgs& u, const ShrinkArgs* v, const LoraGeom& g, hipStream_t s) {
  constexpr int kMost = RT < 8 ? 4 : 2;  // registers
  if (g.row_tiles == 1) shrink_mt<RT, 1, 8>(u, v, g, s);
  else if (g.row_tiles == 2) shrink_mt<RT, 2, 4>(u, v, g, s);
  else shrink_mt<RT, kMost, 4>(u, v, g, s);
}

// u, and v where it is wanted
hipError_t launch_shrink(const ShrinkArgs& u, const ShrinkArgs* v, const LoraGeom& g, hipStream_t s) {
  if (u.R <= 16) shrink_rt<1>(u, v, g, s);
  else if (u.R <= 32) shrink_rt<2>(u, v, g, s);
  else if (u.R <= 64) shrink_rt<4>(u, v, g, s);
  else shrink_rt<8>(u, v, g, s);
  return hipGetLastError();
}

// Blocks of a result: its tiles', and those that write the rows of no selection
// where there may be any to write.
unsigned expand_blocks(const ExpandArgs& a) {
  int64_t n = a.num_tiles * ((a.N + 4 * kCols - 1) / (4 * kCols));
  if (a.map && a.base != a.out) {
    const int64_t copies = (a.T + kCopyTokens - 1) / kCopyTokens;
    n += copies < kLoraMaxCopyBlocks ? copies : kLoraMaxCopyBlocks;
  }
  return static_cast<unsigned>(n);
}

hipError_t launch_expand(const ExpandArgs& a, hipStream_t s) {
  const unsigned grid = expand_blocks(a);
  if (a.R <= 32) k_lora_expand<1><<<grid, kBlock, 0, s>>>(a);
  else if (a.R <= 64) k_lora_expand<2><<<grid, kBlock, 0, s>>>(a);
  else k_lora_expand<4><<<grid, kBlock, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_gradients(const WeightGradArgs& w, const ExpandArgs& x, const LoraGeom& g, hipStream_t s) {
  const unsigned wb = static_cast<unsigned>(lora_weight_blocks(g, w.C[0], w.C[1], w.R));
  const unsigned blocks = wb + expand_blocks(x);
  const size_t lds = sizeof(int) << g.chunk_shift;
  if (w.R <= 16) k_lora_gradients<1, 1><<<blocks, kBlock, lds, s>>>(w, x, wb);
  else if (w.R <= 32) k_lora_gradients<1, 2><<<blocks, kBlock, lds, s>>>(w, x, wb);
  else if (w.R <= 64) k_lora_gradients<2, 4><<<blocks, kBlock, lds, s>>>(w, x, wb);
  else k_lora_gradients<4, 4><<<blocks, kBlock, lds, s>>>(w, x, wb);
  return hipGetLastError();
}

int64_t up16(int64_t n) { return (n + 15) / 16 * 16; }

ShrinkArgs shrink_args(const LoraArgs& a, const LoraGeom& g) {
  ShrinkArgs s = {};
  s.R = a.R;
  s.E = a.E;
  s.stride = g.rows * a.R;
  s.expand_tiles = a.expand_tiles;
  s.num_expand = static_cast<int>(g.max_expand);
  s.expand_shift = g.expand_shift;
  s.counts = a.counts;
  s.offsets = a.offsets;
  s.status = a.status;
  s.generation = a.generation;
  return s;
}

// Are the rows of this many columns too large to be found in the caches (256 MB
// beside the memory, shared with all else) by whoever reads them next?  Read for
// the last time here, they then make room for what is: the shrink of 8111 x 7168
// takes 27 us against 32, of 8192 x 4096 (64 MB) 19 against 21, while a caller's
// second use of 2048 x 7168 (29 MB) would cost 18 against 14; the weight
// gradients of 16,384 x 4096 + 2048 and the shrink before the next call's 129 us
// against 133, of 2048 x 4096 + 4096 27.5 against 25.
bool large_rows(const LoraArgs& a, int64_t columns) {
  const int64_t rows = a.T * a.K;
  return rows * columns * 2 >= (64 << 20);
}

// Is a row of x read once by a kernel that reads all of them?  Not where its K
// selections gather it, each into the tile of another expert: streamed, 4096
// tokens x 4096, K = 4, rank 32 took 32 us against 26 (shrink), 8192 tokens x
// 7168, K = 8, rank 16 178 against 145, and their weight gradients (8192 x 4096
// + 2048, K = 4) 118 against 110.
bool x_read_once(const LoraArgs& a) { return !a.xmap || a.K == 1; }

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
  x.tiles = a.expand_tiles;
  x.num_tiles = g.max_expand;
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
  auto up8 = [](int64_t n) { return (n + kXcds - 1) / kXcds * kXcds; };
  // Tiles of 64 rows read an expert's matrix less often (8111 rows x 7168, rank
  // 64: 31 us against 46 with tiles of 16; tiles of 128 gain nothing more, 16,384
  // x 4096 takes 34 us against 32); smaller ones where its rows, or all rows, are
  // few, and above rank 64 for want of registers (rank 128: 16,384 x 4096 66 us
  // with 32 rows, 72 with 64).
  const int64_t wide = R <= 64 ? 4 : 2;
  int64_t tiles = avg >= 64 ? 4 : avg >= 32 ? 2 : 1;
  if (rows < 2048) tiles = 1;
  else if (rows < 4096 && tiles > 2) tiles = 2;
  g.row_tiles = static_cast<int>(tiles < wide ? tiles : wide);
  g.max_tiles = up8(rows / (16 * g.row_tiles) + used);
  // The contraction is split over blocks too, as far as a split keeps 512
  // elements, until there are four blocks per CU (61 rows x 4096: 4.9 us against
  // 7.2 without; 8111 x 7168: 32 against 43; 16,384 x 4096: 36 against 41 with two
  // per CU and 44 without), in the backward pass two (the weight gradients read
  // every split's part again: 16,384 x 4096, both kernels, 133 us against 140 with
  // four per CU and 135 with one).
  const int enough = backward ? 512 : 1024;
  auto splits = [&](int C) {
    int n = 1;
    while (n < kMaxSplits && g.max_tiles * n < enough && C >= 512 * n) n *= 2;
    return n;
  };
  // The result's tiles: the longest of which the rows alone, in one expert, fill
  // three quarters of the CUs (rank 64, 8111 x 2048: 19.0 us with 128 rows, 19.4
  // with 64, 22.5 with 32; 2048 x 2048: 8.6 with 32, 11.4 with 16; rank 16, 1024 x
  // 4096: 8.5 with 32, 9.1 with 16)
  const int64_t col_blocks = ((backward ? H : N) + 4 * kCols - 1) / (4 * kCols);
  g.expand_shift = R <= 64 ? 7 : 6;
  while (g.expand_shift > 4 && (rows >> g.expand_shift) * col_blocks < 192) --g.expand_shift;
  g.max_expand = up8((rows >> g.expand_shift) + used);
  g.expand_bytes = static_cast<size_t>(g.max_expand) * 16;
  g.split_x = splits(H);
  g.u_bytes = static_cast<size_t>(up16(g.split_x * rows * R * 4));
  if (backward) {
    g.split_g = splits(N);
    g.v_bytes = static_cast<size_t>(up16(g.split_g * rows * R * 4));
    // Chunks of an expert's rows, about 32 of all rows: more cost partial
    // gradients, fewer leave CUs idle (65,536 rows x 2048 -> 2048, rank 32, join
    // included, in four experts: 159 us; with 64 chunks 151, with 16 207; in 64
    // experts 150, 176 and 150.  16,384 x 4096 + 2048: 78, 88 and 78, and 80, 95
    // and 79.  509 rows: 13 us with chunks of 128 rows, 12 with 64, 15 with 256).  A chunk has
    // 4096 rows at most, as its list of rows lies in LDS (16 KiB, so that two
    // blocks fit a CU): above 131,072 rows there are more, one for 4096 rows, and
    // the partial gradients grow with the rows (524,288 rows, rank 64, 7168 ->
    // 2048: 256 of 2.4 MB).
    g.chunk_shift = 7;
    while (g.chunk_shift < 12 && (static_cast<int64_t>(32) << g.chunk_shift) < rows) ++g.chunk_shift;
    g.max_chunks = up8((rows >> g.chunk_shift) + used);
    g.chunk_bytes = static_cast<size_t>(g.max_chunks) * 16;
    // an expert of several chunks has more than one chunk of rows, so its
    // chunks are at most twice its rows over the chunk size
    g.slots = 2 * (rows >> g.chunk_shift);
    g.slot_bytes = static_cast<size_t>(g.slots) * R * (static_cast<size_t>(H) + N) * 4;
  }
  return g;
}

int64_t lora_weight_blocks(const LoraGeom& g, int H, int N, int R) {
  const int per = kWavesPerBlock * kCols;
  const int groups = R <= 64 ? 1 : 2;  // of R
  return g.max_chunks * groups * ((H + per - 1) / per + (N + per - 1) / per);
}

hipError_t launch_lora(const LoraArgs& a, const LoraGeom& g, hipStream_t s) {
  ShrinkArgs u = shrink_args(a, g);
  u.in = a.x;
  u.ld = a.ldx;
  u.map = a.xmap;
  u.w = a.a;
  u.C = a.H;
  u.part = a.u;
  u.S = g.split_x;
  u.streamed = x_read_once(a) && large_rows(a, a.H);
  const hipError_t err = launch_shrink(u, nullptr, g, s);
  if (err != hipSuccess) return err;
  ExpandArgs x = expand_args(a, g);
  x.part = a.u;
  x.S = g.split_x;
  x.w = a.b;
  x.N = a.N;
  return launch_expand(x, s);
}

hipError_t launch_lora_backward(const LoraArgs& a, const LoraGeom& g, hipStream_t s) {
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
  // above rank 64 two groups of blocks, one for each half of R, read the rows:
  // rank 128, 16,384 x 4096 + 2048, with the shrink 330 us streamed, 324 not
  w.streamed[1] = a.R <= 64 && large_rows(a, a.H + a.N);
  w.streamed[0] = w.streamed[1] && x_read_once(a);
  w.chunks = a.chunks;
  w.counts = a.counts;
  w.status = a.status;
  w.generation = a.generation;
  if (a.T > 0) {
    ShrinkArgs u = shrink_args(a, g);
    ShrinkArgs v = u;
    u.in = a.x;
    u.ld = a.ldx;
    u.map = a.xmap;
    u.w = a.a;
    u.C = a.H;
    u.part = a.u;
    u.S = g.split_x;
    u.chunks = a.chunks;
    u.num_chunks = static_cast<int>(g.max_chunks);
    u.chunk_shift = g.chunk_shift;
    v.in = a.go;
    v.ld = a.ldgo;
    v.map = a.omap;
    v.w = a.b;
    v.C = a.N;
    v.part = a.v;
    v.S = g.split_g;
    v.num_expand = 0;  // u's blocks write the tables
    hipError_t err = launch_shrink(u, &v, g, s);
    if (err != hipSuccess) return err;
    ExpandArgs x = expand_args(a, g);
    x.part = a.v;
    x.S = g.split_g;
    x.w = a.a;
    x.N = a.H;
    err = launch_gradients(w, x, g, s);
    if (err != hipSuccess) return err;
  }
  const int64_t parts = (w.slot_size / 4 + kBlock - 1) / kBlock;
  k_lora_join<<<dim3(static_cast<unsigned>(parts < 256 ? parts : 256), a.E < 8 ? a.E : 8), kBlock, 0, s>>>(w);
  return hipGetLastError();
}

}  // namespace ep
