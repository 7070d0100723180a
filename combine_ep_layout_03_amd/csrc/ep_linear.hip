// The experts' layers over the expert-major segments: product with bias,
// activation and residual in its epilogue, and the products of its gradient.
//
// With x the rows of expert e, w[e] its W x H weights and g the gradient of
// the values before the activation,
//     forward  z[r, n] = sum_h x[r, h] w[e, n, h] + bias[e, n]
//     grad_x   [r, h]  = sum_n g[r, n] w[e, n, h]
//     grad_w   [n, h]  = sum_r g[r, n] x[r, h]
// One kernel does all three.  A tile has rows (x's rows, g's rows, g's
// columns) and columns (w's rows, w's columns, x's columns); an operand whose
// contraction runs along memory is read from LDS by ds_read_b128, one whose
// contraction runs across rows of memory by the transposing
// ds_read_b64_tr_b16, which hands each lane four contraction steps of its
// column.
//
// A block has 8 waves in 2 (rows) x 4 (columns).  A wave owns MI sub-tiles of
// 32 rows, interleaved with the other row half's so that a tile of any height
// splits evenly, and 64 columns, as v_mfma_f32_32x32x16_bf16 accumulators.  The
// contraction runs 32 at a time through LDS rings of 3 or 4 stages that
// LDS-direct loads fill three steps ahead: waves 0-3 the row ring (64 wide,
// whole 128-byte lines, where rows run along memory), waves 4-7 the column
// ring.  XOR swizzles of the 16- or 32-byte pieces, made when a lane picks what
// it loads, keep the operand reads on distinct banks (conflicts: 2% of the LDS
// cycles).  A wave reads a half step's operands before it multiplies the other
// half's, with one barrier a step.
//
// What bounds it (65,536 rows x 7168 -> 2048 over 32 experts, 1.92 TFLOP): 1.81
// to 1.90 ms forward, 1010 to 1065 TFLOP/s; grad_x 1.88 to 1.98, grad_w 1.78 to
// 1.87.  The matrix units are busy half of the cycles at 1.96 GHz.  Without its
// loads the same kernel takes 1.41 ms, without its products 1.41, without loads
// and operand reads 1.22: loads and products overlap for three quarters of the
// time.  Measured and dropped: operands read and products issued in alternating
// phases of two barriers (1.99 ms); loads, or operand reads, issued between the
// products (1.96 to 2.00); a fifth stage, and a row ring of 32-wide stages (the
// same); blocks that stay on their CU and issue the next tile's loads before
// they store (weight gradients of 256 rows an expert 1.12 ms against 1.09: a
// wave's stores and loads retire in one order, so its loads wait for its
// stores).
#include "ep_expert.h"
#include "ep_linear_plan.h"

namespace ep {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 512;
constexpr int kBN = kTileCols;
constexpr int kBK = kTileStep;
constexpr int kXBK = 2 * kBK;  // stage of a row operand that runs along memory (whole lines)
constexpr int kRowGroup = 8;  // row tiles that share a run of column tiles

enum Kind { kForward, kGradX, kGradW };

// where lanes past the contraction's end load from
__device__ __align__(16) const uint32_t kZeros[4] = {0u, 0u, 0u, 0u};

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return static_cast<uint32_t>(
      reinterpret_cast<uintptr_t>((const __attribute__((address_space(3))) void*)p));
}

// a pointer that is the same in every lane, as the compiler may not know
__device__ __forceinline__ const char* scalar(const char* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<int>(v));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<int>(v >> 32));
  return reinterpret_cast<const char*>((static_cast<uint64_t>(hi) << 32) | lo);
}

// 16 bytes a lane from base + off to LDS at `to` + 16 lane, not tracked by the
// compiler: its wait counts cannot tell the stages of a ring apart, and would
// drain every load before each LDS read.  wait_vm below is what waits.
// The compiler does not count wait states for them: `base` must not come from a
// vector instruction (v_readfirstlane) fewer than 5 before, which is so as the
// code is built, by the scalar additions between, and held by a test of the
// assembly.  (An s_nop 4 behind `scalar`: 65,536 rows x 7168 -> 2048 1.85 ms
// against 1.87, the gathered gated layer of 64 experts 0.72 against 0.70; s_nop 3
// in each statement 1.91 and 0.70.)
// m0 is named as clobbered, so that no value of the compiler's is kept there
// (it warns that the register is one of its own, which it is).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void load_lds16(const char* base, uint32_t off, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               :
               : "s"(to), "v"(off), "s"(base)
               : "m0", "memory");
}
__device__ __forceinline__ void load_lds16(const char* p, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
               :
               : "s"(to), "v"(p)
               : "m0", "memory");
}
#pragma clang diagnostic pop

// wait until at most n vector-memory loads of this wave are outstanding
// (rounded down to a value listed); the other counters are left alone
__device__ __forceinline__ void wait_vm(int n) {
  if (n >= 10) __builtin_amdgcn_s_waitcnt(0xF70 | 10);
  else if (n >= 8) __builtin_amdgcn_s_waitcnt(0xF70 | 8);
  else if (n >= 4) __builtin_amdgcn_s_waitcnt(0xF70 | 4);
  else if (n >= 2) __builtin_amdgcn_s_waitcnt(0xF70 | 2);
  else __builtin_amdgcn_s_waitcnt(0xF70);
}

__device__ __forceinline__ void block_sync() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// ------------------------------------------------------------- activations
// 1 / (1 + exp(-z)): exp of a large -z is inf and the quotient 0
__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __expf(-z));
}
constexpr float kSqrtHalf = 0.70710678118654752f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kTanhScale = 0.79788456080286536f;  // sqrt(2 / pi)
constexpr float kTanhCubic = 0.044715f;

// The normal distribution function, erfc(-z / sqrt 2) / 2.  (1 + 2 x) exp(x^2)
// erfc(x) is smooth over all x >= 0 in s = (x - k) / (x + k) (Shepherd and
// Laframboise, Math. Comp. 36, 1981); the coefficients are a Chebyshev fit of
// degree 9 for k = 2.5 up to x = 12, where exp(-x^2) is below fp32 (relative
// error 6.5e-8).  In fp32 the result's relative error is 4e-7 down to z = -2
// and grows with the rounding of the exponential's argument to 8e-6 at -13, far
// below the bf16 half step of 3.9e-3 that the results end in.  A few dozen
// instructions without a branch; erfcf's two branches took 1262 spilled
// registers with 8 elements a lane.
__device__ __forceinline__ float normal_cdf(float z) {
  constexpr float kFit[10] = {1.26483822f, -0.122356892f, -0.0990232155f, 0.15763326f, -0.102984153f, 0.0327342302f, 0.00100810081f, -0.0042856955f, 0.000354380376f, 0.000468412938f};
  const float x = fminf(fabsf(z) * kSqrtHalf, 12.0f);
  const float s = (x - 2.5f) * __builtin_amdgcn_rcpf(x + 2.5f);
  float p = kFit[9];
#pragma unroll
  for (int i = 8; i >= 0; --i) p = __builtin_fmaf(p, s, kFit[i]);
  const float tail = 0.5f * p * __builtin_amdgcn_rcpf(1.0f + 2.0f * x) * __expf(-0.5f * z * z);
  return z < 0.0f ? tail : 1.0f - tail;
}

// N values become their activations
template <int N>
__device__ __forceinline__ void act_values(float* z, int act) {
  switch (act) {
    case kActRelu:
#pragma unroll
      for (int d = 0; d < N; ++d) z[d] = z[d] < 0.0f ? 0.0f : z[d];
      break;
    case kActSilu:
#pragma unroll
      for (int d = 0; d < N; ++d) z[d] *= sigmoid(z[d]);
      break;
    case kActGelu:
#pragma unroll
      for (int d = 0; d < N; ++d) {
        z[d] *= normal_cdf(z[d]);
        if (d & 1) __builtin_amdgcn_sched_barrier(0);  // two at a time, for want of registers
      }
      break;
    case kActGeluTanh:
#pragma unroll
      for (int d = 0; d < N; ++d) z[d] *= sigmoid(2.0f * kTanhScale * (z[d] + kTanhCubic * z[d] * z[d] * z[d]));
      break;
    default:
      break;
  }
}
// value and derivative
__device__ __forceinline__ void act_slope(float z, int act, float& value, float& slope) {
  switch (act) {
    case kActRelu:
      value = z < 0.0f ? 0.0f : z;
      slope = z > 0.0f ? 1.0f : 0.0f;
      break;
    case kActSilu: {
      const float p = sigmoid(z);
      value = z * p;
      slope = p + value * (1.0f - p);
      break;
    }
    case kActGelu: {
      const float cdf = normal_cdf(z);
      value = z * cdf;
      slope = cdf + z * kInvSqrt2Pi * __expf(-0.5f * z * z);
      break;
    }
    case kActGeluTanh: {
      const float p = sigmoid(2.0f * kTanhScale * (z + kTanhCubic * z * z * z));
      value = z * p;
      // far out p (1 - p) is 0 and z z may be inf: the term is 0
      const float d = p * (1.0f - p);
      slope = d == 0.0f ? p : p + 2.0f * z * d * kTanhScale * (1.0f + 3.0f * kTanhCubic * z * z);
      break;
    }
    default:
      value = z;
      slope = 1.0f;
  }
}

// -------------------------------------------------------- operand fragments
// One 16-wide half step's operands of a wave: row sub-tiles i and column
// sub-tiles t.
template <int MI>
struct Frags {
  bf16x8 col[2];
  bf16x8 row[MI];
};
typedef short i16x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ bf16x8 lds_read(uint32_t at) {
  return *reinterpret_cast<const __attribute__((address_space(3))) bf16x8*>(at);
}
// four contraction steps of this lane's column, and four more `rows4` bytes on
__device__ __forceinline__ bf16x8 lds_read_across(uint32_t at, uint32_t rows4) {
  typedef __attribute__((address_space(3))) i16x4* P;
  const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<P>(at));
  const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<P>(at + rows4));
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// ------------------------------------------------------------------- tiles
// A tile's place: expert, first row and rows, first column, contraction.
struct Tile {
  int e;
  int64_t row0;  // first expert-major row (grad_w: of the contraction)
  int nrows;     // valid tile rows
  int r0;        // grad_w: first of the W outputs
  int n0;        // first column (forward, gated: of the gate half)
  int k;         // contraction length
  int split;
};

// The tile of a block (blocks are dealt to the 8 XCDs round-robin): runs of `run` tiles, or of an eighth of all if that is less,
// are dealt to the XCDs in turn, so that tiles side by side share an L2.
__device__ __forceinline__ int tile_at(int block, int total, int run) {
  const int r = min(run, (total + kXcds - 1) / kXcds);
  const int i = block / kXcds;
  return (i / r * kXcds + block % kXcds) * r + i % r;
}

// Tile `local` of mt x nt: groups of kRowGroup row tiles, within a group
// column-major, so tiles that run side by side share rows and columns.
__device__ __forceinline__ void tile_of(int local, int mt, int nt, int& im, int& jn) {
  const int group = local / (kRowGroup * nt);
  const int rows = min(kRowGroup, mt - group * kRowGroup);
  const int at = local - group * kRowGroup * nt;
  im = group * kRowGroup + at % rows;
  jn = at / rows;
}

// Tiles of 128 rows run two blocks a CU (80 KiB of LDS and 128 registers
// each), one's prologue and epilogue under the other's products.
template <int MI>
constexpr int kBlocksPerCu = MI == 2 ? 2 : 1;

// bytes of the rings
template <Kind KIND, int MI>
constexpr int kRingBytes = KIND == kGradW ? (MI == 2 ? 3 : 4) * (kBK * 64 * MI * 2 + kBN * kBK * 2)
                                          : 2 * 64 * MI * kXBK * 2 + (MI == 2 ? 3 : 4) * kBN * kBK * 2;

// block `block` of a product, its rings at `lds`
template <Kind KIND, int MI, bool GATHER>
__device__ __forceinline__ void linear_block(const LinearArgs& a, const int block, char* const lds) {
  constexpr bool kRowAcross = KIND == kGradW;    // row operand's contraction runs across memory
  constexpr bool kColAcross = KIND != kForward;  // column operand's
  static_assert(!kRowAcross || MI == 2 || MI == 4, "heights of a row operand across memory");
  constexpr int kStages = MI == 2 ? 3 : 4;  // ring of 32-wide stages
  constexpr int kBM = 64 * MI;
  constexpr int kRowStages = kRowAcross ? kStages : 2;
  constexpr int kRowBytes = kRowAcross ? kBK * kBM * 2 : kBM * kXBK * 2;  // of a stage
  constexpr int kColBytes = kBN * kBK * 2;
  constexpr int kRing = kRowStages * kRowBytes + kStages * kColBytes;
  // the tile table lies in the ring until the first load, the epilogue's
  // slices after the last
  static_assert((1024 + 8) * 4 <= kRing && 8 * 4096 <= kRing, "table and slices fit");
  static_assert(kRing == kRingBytes<KIND, MI>, "rings as allocated");
  char* const sRow = lds;
  char* const sCol = lds + kRowStages * kRowBytes;
  int* const sTiles = reinterpret_cast<int*>(lds);

  const int tid = threadIdx.x;
  const int lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int wm = wave >> 2;   // row half: sub-tiles wm, wm + 2, ...
  const int wn = wave & 3;    // 64-column slab
  const int lr = lane & 31;   // operand row within a sub-tile
  const int lkv = lane >> 5;  // 8-wide part of a 16-step
  const bool gated = KIND == kForward && a.gated;
  const int cols = KIND == kForward ? a.N : a.H;  // columns of the output
  const int tile_cols = gated ? kBN / 2 : kBN;
  const int nt = (cols + tile_cols - 1) / tile_cols;

  // ---- tiles
  Tile T;
  int im, jn;
  if constexpr (KIND == kGradW) {
    const int mt = (a.W + kBM - 1) / kBM;
    const int total = a.E * a.splits * mt * nt;  // below 2^22
    const int run = a.even && *a.even == 0 ? kCusPerXcd : a.run;
    const int tile = tile_at(block, total, run);
    if (tile >= total) return;
    const int es = tile / (mt * nt);
    T.e = es / a.splits;
    // three words from memory, together: short contractions feel each latency
    int32_t stamp = a.status[kStatusGeneration];
    int cnt = a.counts[T.e], offset = a.offsets[T.e];
    asm volatile("" : "+s"(stamp), "+s"(cnt), "+s"(offset));
    cnt = __builtin_amdgcn_readfirstlane(cnt);
    offset = __builtin_amdgcn_readfirstlane(offset);
    if (!layout_current(a.status, stamp, a.generation)) return;
    tile_of(tile - es * mt * nt, mt, nt, im, jn);
    T.split = es - T.e * a.splits;
    const int per = ((cnt + a.splits - 1) / a.splits + kBK - 1) / kBK * kBK;
    const int first = min(cnt, per * T.split);
    T.row0 = offset + first;
    T.k = min(per, cnt - first);
    T.r0 = im * kBM;
    T.nrows = min(kBM, a.W - T.r0);
  } else {
    if (!layout_current(a.status, a.generation)) return;
    // row tiles of each expert times column tiles, then their exclusive
    // prefix (the same in every block)
    for (int e = tid; e < a.E; e += kThreads) sTiles[e] = (a.counts[e] + kBM - 1) / kBM * nt;
    __syncthreads();
    // values from LDS are the same in every lane: scalar from here on
    const int total = __builtin_amdgcn_readfirstlane(block_exclusive_scan<kThreads>(sTiles, a.E, sTiles + 1024));
    if (total == 0) return;
    const int tile = tile_at(block, total, a.run);
    if (tile >= total) return;
    // the last expert whose first tile is not past it (empty ones repeat the
    // prefix of the next)
    int lo = 0, hi = a.E - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (__builtin_amdgcn_readfirstlane(sTiles[mid]) <= tile) lo = mid;
      else hi = mid - 1;
    }
    T.e = lo;
    const int cnt = __builtin_amdgcn_readfirstlane(a.counts[lo]);
    const int mt = (cnt + kBM - 1) / kBM;
    tile_of(tile - __builtin_amdgcn_readfirstlane(sTiles[lo]), mt, nt, im, jn);
    // the rows split evenly over the tiles, in steps of 32: none is empty
    const int per = ((cnt + mt - 1) / mt + 31) / 32 * 32;
    T.row0 = __builtin_amdgcn_readfirstlane(a.offsets[lo]) + im * per;
    T.nrows = min(per, cnt - im * per);
    T.k = KIND == kForward ? a.H : a.W;
    T.r0 = T.split = 0;
    __syncthreads();  // the table is read before the ring's first load
  }
  T.n0 = jn * tile_cols;

  // ---- loads: waves 0-3 fill the row ring, waves 4-7 the column ring
  constexpr int kRowLoads = kRowBytes / 4096;  // per wave and stage, 1 KiB each
  constexpr int kColLoads = kColBytes / 4096;
  constexpr int kLoads = kRowLoads > kColLoads ? kRowLoads : kColLoads;
  const bool row_wave = wave < 4;
  const int64_t up_half = gated ? static_cast<int64_t>(a.N) * a.H * 2 : 0;
  int nk, nsx;  // 32-wide steps, 64-wide stages
  // Stage 0's addresses: a base that the wave shares and each lane's offset
  // of it (bytes; for gathered rows, that may lie anywhere, in 16 bytes).
  const char* base;
  uint32_t off[kLoads];
  auto place = [&]() __attribute__((always_inline)) {
    nk = (T.k + kBK - 1) / kBK;
    nsx = (nk + 1) / 2;
    int l = lane;  // opaque, so that its parts are formed here and not kept through the products
    asm volatile("" : "+v"(l));
#pragma unroll
    for (int q = 0; q < kLoads; ++q) {
      if (row_wave) {
        const int s = (wave * kRowLoads + (q < kRowLoads ? q : 0)) * 64 + l;
        if constexpr (kRowAcross) {
          constexpr int kShift = MI == 4 ? 5 : 4;  // 16-byte slots of a contraction row
          const int k = s >> kShift, p = s & ((1 << kShift) - 1);
          const int c = T.r0 + ((p >> 1) ^ ((k & 3) << 1)) * 16 + (p & 1) * 8;
          off[q] = static_cast<uint32_t>((k * a.ldg + (c < a.W ? c : 0)) * 2);
        } else {
          const int r = s >> 3;
          const int kv = (s & 7) ^ ((r >> 1) & 7);
          const int valid = r < T.nrows ? r : 0;
          if constexpr (KIND == kForward && GATHER)
            off[q] = static_cast<uint32_t>((a.xmap[T.row0 + valid] * a.ldx >> 3) + kv);
          else
            off[q] = static_cast<uint32_t>((valid * (KIND == kForward ? a.ldx : a.ldg) + kv * 8) * 2);
        }
      } else {
        const int s = ((wave - 4) * kColLoads + (q < kColLoads ? q : 0)) * 64 + l;
        if constexpr (kColAcross) {
          const int k = s >> 5, p = s & 31;
          const int c = T.n0 + ((p >> 1) ^ ((k & 3) << 1)) * 16 + (p & 1) * 8;
          const int col = c < a.H ? c : 0;
          if constexpr (KIND == kGradX) off[q] = static_cast<uint32_t>((static_cast<int64_t>(k) * a.H + col) * 2);
          else off[q] = static_cast<uint32_t>((GATHER ? col : k * a.ldx + col) * 2);
        } else {
          const int r = s >> 2;
          const int kv = (s & 3) ^ ((r >> 2) & 3);
          // tile column -> row of w; gated tiles take 32 gate and 32 up rows
          // a wave, and the base of the loads q = 2, 3 is the up half's
          const int n = gated ? (r >> 6) * 32 + (r & 31) : r;
          off[q] = static_cast<uint32_t>((static_cast<int64_t>(T.n0 + n < a.N ? n : 0) * a.H + kv * 8) * 2);
        }
      }
    }
    const uint16_t* from;
    if (row_wave) {
      if constexpr (KIND == kForward) from = GATHER ? a.x : a.x + T.row0 * a.ldx;
      else from = a.g + T.row0 * a.ldg;
    } else {
      if constexpr (KIND == kGradW) from = GATHER ? a.x : a.x + T.row0 * a.ldx;
      else from = a.w + (static_cast<int64_t>(T.e) * a.W + (KIND == kForward ? T.n0 : 0)) * a.H;
    }
    base = scalar(reinterpret_cast<const char*>(from));
  };
  auto issue_row = [&](int st) __attribute__((always_inline)) {
    const uint32_t to = lds_addr(sRow) + (st % kRowStages) * kRowBytes + wave * kRowLoads * 1024;
    constexpr int kWide = kRowAcross ? kBK : kXBK;
    constexpr bool kFar = KIND == kForward && GATHER;  // offsets of 16 bytes
    const char* const from = base + st * (kRowAcross ? kBK * a.ldg * 2 : kXBK * 2);
    if ((st + 1) * kWide <= T.k) {
#pragma unroll
      for (int q = 0; q < kRowLoads; ++q) {
        if constexpr (kFar) load_lds16(from + (static_cast<uint64_t>(off[q]) << 4), to + q * 1024);
        else load_lds16(from, off[q], to + q * 1024);
      }
    } else {
      int l = lane;  // opaque, so that nothing of the last stage is formed ahead and kept
      asm volatile("" : "+v"(l));
#pragma unroll 1
      for (int q = 0; q < kRowLoads; ++q) {
        uint32_t o = 0;
#pragma unroll
        for (int r = 0; r < kRowLoads; ++r) o = r == q ? off[r] : o;
        const int s = (wave * kRowLoads + q) * 64 + l;
        const int k = kRowAcross ? s >> (MI == 4 ? 5 : 4) : ((s & 7) ^ ((s >> 4) & 7)) * 8;
        const char* p = from + (kFar ? static_cast<uint64_t>(o) << 4 : o);
        load_lds16(st * kWide + k < T.k ? p : reinterpret_cast<const char*>(kZeros), to + q * 1024);
      }
    }
  };
  // grad_w on gathered rows: the tokens of this wave's 8 contraction rows of a
  // stage, in scalar registers, loaded a stage ahead.  (Scalar loads: a wait
  // for a vector load would wait for the LDS-direct loads before it.)
  int token[8];
  auto next_tokens = [&](int st) __attribute__((always_inline)) {
    if constexpr (KIND == kGradW && GATHER) {
      const auto* map = reinterpret_cast<const __attribute__((address_space(4))) int32_t*>(
          reinterpret_cast<uintptr_t>(a.xmap + T.row0));
#pragma unroll
      for (int j = 0; j < 8; ++j) token[j] = map[min(st * kBK + (wave - 4) * 8 + j, T.k - 1)];
    }
  };
  auto issue_col = [&](int st) __attribute__((always_inline)) {
    const uint32_t to = lds_addr(sCol) + (st % kStages) * kColBytes + (wave - 4) * kColLoads * 1024;
    constexpr bool kRowsApart = KIND == kGradW && GATHER;
    const char* const from =
        kRowsApart ? base : base + st * (KIND == kForward ? kBK * 2 : static_cast<int64_t>(kBK) * (KIND == kGradX ? a.H : a.ldx) * 2);
    int64_t row[kColLoads];
    if constexpr (kRowsApart) {
#pragma unroll
      for (int q = 0; q < kColLoads; ++q) {
        const int64_t lo = token[2 * q] * a.ldx * 2, hi = token[2 * q + 1] * a.ldx * 2;
        row[q] = lane < 32 ? lo : hi;
      }
      next_tokens(st + 1);
    }
    if ((st + 1) * kBK <= T.k) {
#pragma unroll
      for (int q = 0; q < kColLoads; ++q) {
        if constexpr (kRowsApart) load_lds16(from + off[q] + row[q], to + q * 1024);
        else load_lds16(from + (KIND == kForward && q >= 2 ? up_half : 0), off[q], to + q * 1024);
      }
    } else {
      int l = lane;
      asm volatile("" : "+v"(l));
#pragma unroll
      for (int q = 0; q < kColLoads; ++q) {
        const int s = ((wave - 4) * kColLoads + q) * 64 + l;
        const int k = kColAcross ? s >> 5 : ((s & 3) ^ ((s >> 4) & 3)) * 8;
        const char* p = from + off[q];
        if constexpr (kRowsApart) p += row[q];
        if constexpr (KIND == kForward) p += q >= 2 ? up_half : 0;
        load_lds16(st * kBK + k < T.k ? p : reinterpret_cast<const char*>(kZeros), to + q * 1024);
      }
    }
  };
  // This wave's loads of the stages that step kt reads have landed, as of the
  // middle of step kt - 1 (kt = 0: before the first).  32-wide stages up to kt
  // + kStages - 2 are issued by then (0: kStages - 1); of 64-wide row stages 0
  // and 1, and stage s + 1 in the middle of step 2 s - 1.
  auto wait_own = [&](int kt) __attribute__((always_inline)) {
    if (row_wave && !kRowAcross) {
      const int issued = min(nsx - 1, (kt & 1) ? (kt >> 1) + 1 : max(kt >> 1, 1));
      wait_vm(kRowLoads * (issued - (kt >> 1)));
    } else {
      wait_vm((row_wave ? kRowLoads : kColLoads) * min(kt == 0 ? kStages - 1 : kStages - 2, nk - 1 - kt));
    }
  };
  // in the middle of step kt, when every wave has read all of it: the stage
  // that takes its slot
  auto issue_next = [&](int kt) __attribute__((always_inline)) {
    if (row_wave && !kRowAcross) {
      if ((kt & 1) && (kt >> 1) + 2 < nsx) issue_row((kt >> 1) + 2);
    } else if (kt + kStages < nk) {
      if (row_wave) issue_row(kt + kStages);
      else issue_col(kt + kStages);
    }
  };

  // ---- products
  // operand addresses within a stage
  const int j16 = lane & 15, g2 = (lane >> 4) & 1;
  const uint32_t row_at =
      lds_addr(sRow) + (kRowAcross ? (lkv * 8 + (j16 >> 2)) * (kBM * 2) + ((wm * 2 + g2) ^ ((j16 >> 2) << 1)) * 32 + (j16 & 3) * 8
                                   : (wm * 32 + lr) * 128 + (lkv ^ ((lr >> 1) & 7)) * 16);
  const uint32_t col_at =
      lds_addr(sCol) + (kColAcross ? (lkv * 8 + (j16 >> 2)) * 512 + ((wn * 4 + g2) ^ ((j16 >> 2) << 1)) * 32 + (j16 & 3) * 8
                                   : (wn * 64 + lr) * 64 + (lkv ^ ((lr >> 2) & 3)) * 16);
  auto read_half = [&](int kt, int kk, Frags<MI>& f) __attribute__((always_inline)) {
    const uint32_t c = col_at + (kt % kStages) * kColBytes;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      if constexpr (kColAcross) f.col[t] = lds_read_across((c ^ (t * 64)) + kk * 8192, 2048);
      else f.col[t] = lds_read((c ^ (kk * 32)) + t * 2048);
    }
    if constexpr (kRowAcross) {
      const uint32_t r = row_at + (kt % kStages) * kRowBytes;
#pragma unroll
      for (int i = 0; i < MI; ++i)
        f.row[i] = lds_read_across((r ^ ((i & 1) * 128)) + (i >> 1) * 256 + kk * 16 * kBM * 2, 4 * kBM * 2);
    } else {
      const uint32_t r = (row_at + ((kt >> 1) % kRowStages) * kRowBytes) ^ ((kt & 1) * 64 + kk * 32);
#pragma unroll
      for (int i = 0; i < MI; ++i) f.row[i] = lds_read(r + i * 8192);
    }
  };
  f32x16 acc[MI][2];
  int live = 0;  // sub-tiles of this wave with a valid row (none if its columns lie past the end)
  // grad_w: column sums of g for the bias, sub-tile i = wn of the first
  // column tile's waves
  const bool want_bias = KIND == kGradW && a.gb != nullptr && T.n0 == 0;
  float bias_sum = 0.0f;
  int mine[MI];  // i == wn, in terms that the compiler cannot make an index (and scratch memory) of
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    mine[i] = __builtin_amdgcn_readfirstlane(i == wn);
    if constexpr (KIND == kGradW) asm volatile("" : "+s"(mine[i]));
  }
  auto mfma_half = [&](const Frags<MI>& f) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      if (i < live) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
          acc[i][t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.col[t], f.row[i], acc[i][t], 0, 0, 0);
      }
    }
    if constexpr (KIND == kGradW) {
      if (want_bias) {
#pragma unroll
        for (int i = 0; i < MI; ++i) {
          if (mine[i]) {
            const u32x4 v = __builtin_bit_cast(u32x4, f.row[i]);
#pragma unroll
            for (int d = 0; d < 4; ++d) bias_sum += bf16_lo(v[d]) + bf16_hi(v[d]);
          }
        }
      }
    }
  };

  // ---- epilogue.  Lane l of an accumulator holds row l % 32 and
  // the columns (j / 4) * 8 + (l / 32) * 4 + j % 4 of a sub-tile, j < 16.  Bias,
  // activation, gate (the up half lies in the same lanes) and residual are
  // applied there; then a wave turns the rounded 32 x 64 through its own slice
  // of LDS, so that stores are 16 bytes a lane and whole lines (32-byte pieces
  // of lines straight from the registers: 1168 against 1064 us for a weight
  // gradient of 2.1 GB).
  const uint32_t slice = lds_addr(lds) + wave * 4096;
  typedef __attribute__((address_space(3))) u32x2* Lds8;
  typedef __attribute__((address_space(3))) u32x4* Lds16;
  // 16-byte piece c of row r: rows 2 j and 2 j + 1 fill the banks, XOR keeps
  // 16 rows of a piece on distinct ones
  auto piece = [&](int r, int c) __attribute__((always_inline)) {
    return slice + r * 128 + ((c ^ ((r >> 1) & 7)) << 4);
  };
  auto settle = [&]() __attribute__((always_inline)) {  // this wave's LDS writes before its reads, and back
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  };
  auto finish = [&]() __attribute__((always_inline)) {
    const int col0 = T.n0 + wn * (gated ? 32 : 64);
    if constexpr (KIND == kGradW) {
      if (want_bias) {
        const float sum = bias_sum + __shfl_xor(bias_sum, 32, kWave);
        const int n = T.r0 + (2 * wn + wm) * 32 + lr;
        if (wn < MI && lkv == 0 && n < a.W) {
          if (a.splits == 1) a.gb[static_cast<int64_t>(T.e) * a.W + n] = bf16_of(sum);
          else
            a.part[static_cast<int64_t>(a.splits) * a.E * a.W * a.H +
                   (static_cast<int64_t>(T.split) * a.E + T.e) * a.W + n] = sum;
        }
      }
    }
    if constexpr (KIND != kForward) {
      if (KIND == kGradX || a.splits == 1) {
        // no arithmetic is left: up to four sub-tiles at once, each through a slice of its own
        uint16_t* const to = KIND == kGradX ? a.out + T.row0 * a.ldout
                                            : a.gw + (static_cast<int64_t>(T.e) * a.W + T.r0) * a.H;
        const int64_t ld = KIND == kGradX ? a.ldout : a.H;
        constexpr int kAtOnce = MI == 5 ? 4 : MI;
        static_assert(kAtOnce * 8 * 4096 <= kRing, "slices fit");
#pragma unroll
        for (int i0 = 0; i0 < MI; i0 += kAtOnce) {
          settle();
#pragma unroll
          for (int i = i0; i < MI && i < i0 + kAtOnce; ++i) {
            if (i >= live) continue;
#pragma unroll
            for (int g = 0; g < 8; ++g) {
              const f32x16& v = acc[i][g >> 2];
              const int d = (g & 3) * 4;
              *reinterpret_cast<Lds8>(piece(lr, g) + (i - i0) * 8 * 4096 + lkv * 8) =
                  u32x2{bf16x2_of(v[d], v[d + 1]), bf16x2_of(v[d + 2], v[d + 3])};
            }
          }
          settle();
#pragma unroll
          for (int i = i0; i < MI && i < i0 + kAtOnce; ++i) {
            if (i >= live) continue;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int r = j * 8 + (lane >> 3), c = lane & 7;
              const int row = (2 * i + wm) * 32 + r, n = col0 + c * 8;
              if (row < T.nrows && n < a.H)
                *reinterpret_cast<u32x4*>(to + row * ld + n) = *reinterpret_cast<Lds16>(piece(r, c) + (i - i0) * 8 * 4096);
            }
          }
        }
        return;
      }
    }
#pragma unroll 1  // one copy of the code
    for (int now = 0; now < live; ++now) {
      int l = lane;  // opaque: no address is formed ahead of the loop and kept through it
      asm volatile("" : "+v"(l));
      const int er = l & 31, eh = l >> 5;
      float z[32];  // columns t * 32 + ...
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        if (i != now) continue;
#pragma unroll
        for (int d = 0; d < 32; ++d) z[d] = acc[i][d >> 4][d & 15];
      }
      const int sub = (2 * now + wm) * 32;
      const int rows = min(32, T.nrows - sub);
      // rounds z's first `pieces` 16-byte pieces a row and stores them at to(row, piece)
      auto emit = [&](int pieces, auto to) __attribute__((always_inline)) {
        settle();
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          if (g >= pieces) break;
          *reinterpret_cast<Lds8>(piece(er, g) + eh * 8) =
              u32x2{bf16x2_of(z[4 * g], z[4 * g + 1]), bf16x2_of(z[4 * g + 2], z[4 * g + 3])};
        }
        settle();
        const int shift = pieces == 8 ? 3 : 2;
#pragma unroll 1
        for (int it = l; it < rows << shift; it += kWave) {
          const int r = it >> shift, c = it & (pieces - 1);
          uint16_t* const at = to(r, c);
          if (at) *reinterpret_cast<u32x4*>(at) = *reinterpret_cast<Lds16>(piece(r, c));
        }
      };
      if constexpr (KIND == kForward) {
        const int64_t row = T.row0 + sub;  // of the sub-tile's row 0
        // columns 4 g .. 4 g + 3 of this lane: n, or past the end (not loaded, not stored)
        auto column = [&](int g) { return col0 + (gated ? g & 3 : g) * 8 + eh * 4; };
        auto add4 = [&](int g, const uint16_t* from) __attribute__((always_inline)) {
          const u32x2 b = *reinterpret_cast<const u32x2*>(from);
          z[4 * g] += bf16_lo(b[0]);
          z[4 * g + 1] += bf16_hi(b[0]);
          z[4 * g + 2] += bf16_lo(b[1]);
          z[4 * g + 3] += bf16_hi(b[1]);
        };
        if (a.bias) {
          const uint16_t* bias = a.bias + static_cast<int64_t>(T.e) * a.W;
#pragma unroll
          for (int g = 0; g < 8; ++g) {
            const int n = column(g);
            if (n < a.N) add4(g, bias + (gated && g >= 4 ? a.N : 0) + n);
          }
        }
        if (a.pre)
          emit(8, [&](int r, int c) {
            const int n = col0 + (gated ? c & 3 : c) * 8;
            return n < a.N ? a.pre + (row + r) * a.ldpre + (gated && c >= 4 ? a.N : 0) + n : nullptr;
          });
#pragma unroll
        for (int d = 0; d < 32; d += 8) {
          if (gated && d >= 16) break;
          act_values<8>(z + d, a.act);
        }
        if (gated) {
#pragma unroll
          for (int d = 0; d < 16; ++d) z[d] *= z[16 + d];
        }
        if (a.res && er < rows) {
          const uint16_t* res = a.res + (row + er) * a.ldres;
#pragma unroll
          for (int g = 0; g < 8; ++g) {
            if (gated && g >= 4) break;
            const int n = column(g);
            if (n < a.N) add4(g, res + n);
          }
        }
        emit(gated ? 4 : 8, [&](int r, int c) {
          const int n = col0 + c * 8;
          return n < a.N ? a.out + (row + r) * a.ldout + n : nullptr;
        });
      } else if constexpr (KIND == kGradW) {  // a part of split rows
        if (er < rows) {
          float* const to =
              a.part + ((static_cast<int64_t>(T.split) * a.E + T.e) * a.W + T.r0 + sub + er) * static_cast<int64_t>(a.H);
#pragma unroll
          for (int g = 0; g < 8; ++g) {
            const int n = col0 + g * 8 + eh * 4;
            if (n < a.H) *reinterpret_cast<f32x4*>(to + n) = f32x4{z[4 * g], z[4 * g + 1], z[4 * g + 2], z[4 * g + 3]};
          }
        }
      }
    }
  };

  place();
  if (row_wave) {
    if constexpr (kRowAcross) {
      for (int kt = 0; kt < kStages && kt < nk; ++kt) issue_row(kt);
    } else {
      issue_row(0);
      if (nsx > 1) issue_row(1);
    }
  } else {
    if (nk > 0) next_tokens(0);
    for (int kt = 0; kt < kStages && kt < nk; ++kt) issue_col(kt);
  }
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    live += (2 * i + wm) * 32 < T.nrows ? 1 : 0;
#pragma unroll
    for (int t = 0; t < 2; ++t) acc[i][t] = f32x16{};
  }
  if (T.n0 + wn * (gated ? 32 : 64) >= cols) live = 0;
  // A wave reads one half step's operands while it multiplies the other's.
  // One barrier a step, in its middle: before it a wave has the step's last
  // operands in registers and its own loads of the next step in LDS, so after
  // it the next step may be read and this step's slots filled again.
  if (nk > 0) {
    Frags<MI> even, odd;
    wait_own(0);
    block_sync();
    read_half(0, 0, even);
    for (int kt = 0; kt < nk; ++kt) {
      read_half(kt, 1, odd);
      __builtin_amdgcn_sched_barrier(0);
      mfma_half(even);
      __builtin_amdgcn_sched_barrier(0);
      wait_own(kt + 1);
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      block_sync();
      if (kt + 1 < nk) {
        issue_next(kt);
        read_half(kt + 1, 0, even);
      }
      __builtin_amdgcn_sched_barrier(0);
      mfma_half(odd);
    }
  }
  // nobody reads the ring any more: every wave passed the last step's barrier
  finish();
}

template <Kind KIND, int MI, bool GATHER>
__global__ __launch_bounds__(kThreads, 2 * kBlocksPerCu<MI>) void k_linear(LinearArgs a) {
  __shared__ __align__(1024) char lds[kRingBytes<KIND, MI>];
  linear_block<KIND, MI, GATHER>(a, static_cast<int>(blockIdx.x), lds);
}

// Both gradients: the first `x_blocks` (a multiple of 8) are grad_x's.  Neither
// needs the other, and one's blocks fill the CUs that the other's leave.
template <int MX, int MW, bool GATHER>
__global__ __launch_bounds__(kThreads, 2 * kBlocksPerCu<MX>) void k_linear_grads(LinearArgs x, LinearArgs w, int x_blocks) {
  static_assert(kBlocksPerCu<MX> == kBlocksPerCu<MW>, "tiles of one occupancy");
  constexpr int kX = kRingBytes<kGradX, MX>, kW = kRingBytes<kGradW, MW>;
  __shared__ __align__(1024) char lds[kX > kW ? kX : kW];
  const int block = static_cast<int>(blockIdx.x);
  if (block < x_blocks) linear_block<kGradX, MX, false>(x, block, lds);
  else linear_block<kGradW, MW, GATHER>(w, block - x_blocks, lds);
}

// ---------------------------------------------------------------- few rows
// Forward where experts have a few rows each (a decoding step: the weights are
// read once and nothing else counts), or the whole problem is small.  A block
// takes 64 of an expert's columns (32 gate and 32 up with a gate) and 16 of
// its rows; its 8 waves take the 128-byte lines of the contraction in turn.
// Weights and rows go straight from memory into the operands of v_mfma_f32_16x16x32_bf16 (a
// load instruction takes 64 bytes of 16 weight rows), a line ahead of the
// product, so a wave keeps 8 KiB of weights in flight and waits for nobody;
// the waves' sums meet in LDS at the end, in their order.  16 tokens x 4096 ->
// 2 x 2048, top-4 of 64 experts: 244 us, 5.6 TB/s of weights (the tiles above:
// 260; two lines ahead 250, non-temporal weights 246, 32 rows a block 254); one
// expert of 16 rows, 4096 -> 4096: 21 us (56).
template <bool GATHER>
__global__ __launch_bounds__(kThreads, 4) void k_linear_few(LinearArgs a) {
  constexpr int kWaves = kThreads / kWave;
  constexpr int kRows = 16;
  __shared__ __align__(16) f32x4 s_sum[kWaves][4][kWave];
  static_assert((1024 + kWaves) * 4 <= sizeof(s_sum), "tile table fits");
  int* const sTiles = reinterpret_cast<int*>(s_sum);
  if (!layout_current(a.status, a.generation)) return;
  const int tid = threadIdx.x;
  const int lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int tile_cols = a.gated ? 32 : 64;
  const int nt = (a.N + tile_cols - 1) / tile_cols;

  for (int e = tid; e < a.E; e += kThreads) sTiles[e] = (a.counts[e] + kRows - 1) / kRows * nt;
  __syncthreads();
  const int total = __builtin_amdgcn_readfirstlane(block_exclusive_scan<kThreads>(sTiles, a.E, sTiles + 1024));
  if (total == 0) return;
  const int tile = tile_at(static_cast<int>(blockIdx.x), total, a.run);
  if (tile >= total) return;
  int lo = 0, hi = a.E - 1;  // the last expert whose first tile is not past it
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__builtin_amdgcn_readfirstlane(sTiles[mid]) <= tile) lo = mid;
    else hi = mid - 1;
  }
  const int e = lo;
  const int cnt = a.counts[e];
  const int mt = (cnt + kRows - 1) / kRows;
  const int local = tile - __builtin_amdgcn_readfirstlane(sTiles[e]);
  // row tiles of the same columns side by side: they share weights
  const int im = local % mt;
  const int n0 = local / mt * tile_cols;
  const int per = (cnt + mt - 1) / mt;
  const int64_t row0 = a.offsets[e] + im * per;
  const int nrows = min(per, cnt - im * per);
  __syncthreads();  // the table is read before the sums are written

  const int m = lane & 15, q = lane >> 4;
  const uint16_t* wp[4];
#pragma unroll
  for (int f = 0; f < 4; ++f) {
    const int c = n0 + (a.gated ? f & 1 : f) * 16 + m;
    const int64_t w = (c < a.N ? c : n0) + (a.gated && f >= 2 ? a.N : 0);
    wp[f] = a.w + (static_cast<int64_t>(e) * a.W + w) * a.H + q * 8;
  }
  const int64_t xr = row0 + (m < nrows ? m : 0);
  const uint16_t* const xp = a.x + (GATHER ? static_cast<int64_t>(a.xmap[xr]) : xr) * a.ldx + q * 8;
  f32x4 acc[4];
#pragma unroll
  for (int f = 0; f < 4; ++f) acc[f] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  struct Line {
    bf16x8 w[2][4], x[2];
  };
  auto load = [&](int line, Line& l) __attribute__((always_inline)) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = line * 64 + h * 32;
#pragma unroll
      for (int f = 0; f < 4; ++f) l.w[h][f] = *reinterpret_cast<const bf16x8*>(wp[f] + k);
      l.x[h] = *reinterpret_cast<const bf16x8*>(xp + k);
    }
  };
  auto multiply = [&](const Line& l) __attribute__((always_inline)) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int f = 0; f < 4; ++f)
        acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(l.w[h][f], l.x[h], acc[f], 0, 0, 0);
  };
  const int lines = a.H / 64;  // whole ones
  Line one, two;
  int at = wave;
  if (at < lines) load(at, one);
  while (at < lines) {
    if (at + kWaves < lines) load(at + kWaves, two);
    multiply(one);
    at += kWaves;
    if (at >= lines) break;
    if (at + kWaves < lines) load(at + kWaves, one);
    multiply(two);
    at += kWaves;
  }
  if (at == lines && a.H % 64) {  // the rest, by the wave whose turn it is; zeros past its end
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = lines * 64 + h * 32;
      const bool in = k + q * 8 < a.H;
#pragma unroll
      for (int f = 0; f < 4; ++f) one.w[h][f] = in ? *reinterpret_cast<const bf16x8*>(wp[f] + k) : bf16x8{};
      one.x[h] = in ? *reinterpret_cast<const bf16x8*>(xp + k) : bf16x8{};
    }
    multiply(one);
  }
#pragma unroll
  for (int f = 0; f < 4; ++f) s_sum[wave][f][lane] = acc[f];
  __syncthreads();

  // lane l of a sum holds row l % 16 and columns (l / 16) * 4 .. + 3
  const int f = wave, r = m, n = n0 + f * 16 + q * 4;
  if (f < (a.gated ? 2 : 4) && r < nrows && n < a.N) {
    f32x4 v = s_sum[0][f][lane];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) v += s_sum[w][f][lane];
    const int64_t row = row0 + r;
    auto load4 = [&](const uint16_t* p) __attribute__((always_inline)) {
      const u32x2 b = *reinterpret_cast<const u32x2*>(p);
      return f32x4{bf16_lo(b[0]), bf16_hi(b[0]), bf16_lo(b[1]), bf16_hi(b[1])};
    };
    auto store4 = [&](uint16_t* p, const f32x4& x) __attribute__((always_inline)) {
      *reinterpret_cast<u32x2*>(p) = u32x2{bf16x2_of(x[0], x[1]), bf16x2_of(x[2], x[3])};
    };
    const uint16_t* bias = a.bias ? a.bias + static_cast<int64_t>(e) * a.W : nullptr;
    if (bias) v += load4(bias + n);
    if (a.pre) store4(a.pre + row * a.ldpre + n, v);
    float z[4] = {v[0], v[1], v[2], v[3]};
    act_values<4>(z, a.act);
    v = f32x4{z[0], z[1], z[2], z[3]};
    if (a.gated) {
      f32x4 u = s_sum[0][2 + f][lane];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) u += s_sum[w][2 + f][lane];
      if (bias) u += load4(bias + a.N + n);
      if (a.pre) store4(a.pre + row * a.ldpre + a.N + n, u);
      v *= u;
    }
    if (a.res) v += load4(a.res + row * a.ldres + n);
    store4(a.out + row * a.ldout + n, v);
  }
}

// Do the experts have much the same rows (none over 3/2 of the mean)?
__global__ __launch_bounds__(kBlock) void k_linear_even(const int32_t* counts, int E, int32_t* even, int32_t* status,
                                                        uint32_t generation) {
  __shared__ int s_most[kWavesPerBlock], s_all[kWavesPerBlock];
  if (!layout_current(status, generation)) return;
  int most = 0, all = 0;
  for (int e = threadIdx.x; e < E; e += kBlock) {
    most = max(most, counts[e]);
    all += counts[e];
  }
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) {
    most = max(most, __shfl_xor(most, off, kWave));
    all += __shfl_xor(all, off, kWave);
  }
  if ((threadIdx.x & (kWave - 1)) == 0) {
    s_most[threadIdx.x / kWave] = most;
    s_all[threadIdx.x / kWave] = all;
  }
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int w = 1; w < kWavesPerBlock; ++w) {
    most = max(most, s_most[w]);
    all += s_all[w];
  }
  *even = 2ll * most * E <= 3ll * all;
}

// Weight gradients of split rows: the parts' sum, in their order.  8 elements
// a thread; the bias's parts follow the weights'.
__global__ __launch_bounds__(kBlock) void k_linear_join(const float* part, int splits, int64_t nw, int64_t nb,
                                                        uint16_t* gw, uint16_t* gb, int32_t* status,
                                                        uint32_t generation) {
  if (!layout_current(status, generation)) return;
  const int64_t at = (static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x) * 8;
  const bool weights = at < nw;
  if (!weights && (gb == nullptr || at - nw >= nb)) return;
  const float* p = weights ? part + at : part + splits * nw + (at - nw);
  const int64_t stride = weights ? nw : nb;
  float v[8] = {};
  for (int s = 0; s < splits; ++s) {
    const f32x4 lo = *reinterpret_cast<const f32x4*>(p + s * stride);
    const f32x4 hi = *reinterpret_cast<const f32x4*>(p + s * stride + 4);
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      v[d] += lo[d];
      v[d + 4] += hi[d];
    }
  }
  u32x4 b;
#pragma unroll
  for (int d = 0; d < 4; ++d) b[d] = bf16x2_of(v[2 * d], v[2 * d + 1]);
  *reinterpret_cast<u32x4*>(weights ? gw + at : gb + (at - nw)) = b;
}

// 8 columns a lane; a wave walks the columns of one row.  grad_pre is rounded to
// bf16 here, before the products that are formed from it: the matrix
// instructions take bf16, and the gradients are of the grad_pre that is
// returned.  It adds its error to that of the results' own rounding (2.4e-3 of
// their norm against 1.7e-3); keeping it as two bf16 parts would take each
// product twice.
__global__ __launch_bounds__(kBlock) void k_act_backward(ActBackwardArgs a) {
  if (!layout_current(a.status, a.generation)) return;
  const int lane = lane_id();
  const int64_t rows = a.offsets[a.E];
  for (int64_t r = global_wave(); r < rows; r += grid_waves()) {
    if (a.padded) {
      int lo = 0, hi = a.E - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.offsets[mid] <= r) lo = mid;
        else hi = mid - 1;
      }
      if (r - a.offsets[lo] >= a.counts[lo]) continue;
    }
    const uint16_t* go = a.go + r * a.ldgo;
    const uint16_t* pre = a.pre + r * a.ldpre;
    uint16_t* gpre = a.gpre + r * a.ldgpre;
    for (int n = lane * 8; n < a.N; n += kWave * 8) {
      const u32x4 g4 = *reinterpret_cast<const u32x4*>(go + n);
      const u32x4 z4 = *reinterpret_cast<const u32x4*>(pre + n);
      u32x4 u4 = {0u, 0u, 0u, 0u};
      if (a.gated) u4 = *reinterpret_cast<const u32x4*>(pre + a.N + n);
      u32x4 gate, up;
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const float g[2] = {bf16_lo(g4[d]), bf16_hi(g4[d])};
        const float z[2] = {bf16_lo(z4[d]), bf16_hi(z4[d])};
        const float u[2] = {bf16_lo(u4[d]), bf16_hi(u4[d])};
        float dz[2], du[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float value, slope;
          act_slope(z[h], a.act, value, slope);
          dz[h] = a.gated ? g[h] * u[h] * slope : g[h] * slope;
          du[h] = g[h] * value;
        }
        gate[d] = bf16x2_of(dz[0], dz[1]);
        up[d] = bf16x2_of(du[0], du[1]);
      }
      *reinterpret_cast<u32x4*>(gpre + n) = gate;
      if (a.gated) *reinterpret_cast<u32x4*>(gpre + a.N + n) = up;
    }
  }
}

template <Kind KIND, bool GATHER>
hipError_t launch_rows(const LinearArgs& a, const LinearPlan& plan, hipStream_t s) {
  LinearArgs b = a;
  b.run = plan.run;
  if (plan.mi == 2) k_linear<KIND, 2, GATHER><<<plan.blocks, kThreads, 0, s>>>(b);
  else if (plan.mi == 4) k_linear<KIND, 4, GATHER><<<plan.blocks, kThreads, 0, s>>>(b);
  else k_linear<KIND, 5, GATHER><<<plan.blocks, kThreads, 0, s>>>(b);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_linear(const LinearArgs& a, int64_t rows, hipStream_t s) {
  const LinearPlan plan = plan_forward(rows, a.E, a.N, a.gated);
  if (plan.mi != 0) return a.xmap ? launch_rows<kForward, true>(a, plan, s) : launch_rows<kForward, false>(a, plan, s);
  LinearArgs b = a;
  b.run = plan.run;
  if (a.xmap) k_linear_few<true><<<plan.blocks, kThreads, 0, s>>>(b);
  else k_linear_few<false><<<plan.blocks, kThreads, 0, s>>>(b);
  return hipGetLastError();
}

hipError_t launch_linear_grads(const LinearArgs* x, const LinearArgs* w, int64_t rows, hipStream_t s) {
  if (!x && !w) return hipSuccess;
  const LinearArgs& any = w ? *w : *x;
  const GradsPlan plan = plan_grads(rows, any.E, any.H, any.W, w ? w->splits : 1, x != nullptr, w != nullptr);
  if (!w) return launch_rows<kGradX, false>(*x, plan.x, s);
  const LinearArgs& a = *w;
  LinearArgs b = a;
  b.run = plan.w.run;
  b.even = nullptr;
  if (plan.by_expert) {
    b.even = reinterpret_cast<int32_t*>(a.part);  // no part of split rows lies there
    k_linear_even<<<1, kBlock, 0, s>>>(a.counts, a.E, b.even, a.status, a.generation);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (x && !plan.together) {
    const hipError_t e = launch_rows<kGradX, false>(*x, plan.x, s);
    if (e != hipSuccess) return e;
  }
  const unsigned blocks = plan.w.blocks;
  const bool half = plan.w.mi == 2;
  if (plan.together) {
    LinearArgs c = *x;
    c.run = plan.x.run;
    const int x_blocks = static_cast<int>(plan.x.blocks);
#define EP_GRADS(MX, MW)                                                                                     \
  if (a.xmap) k_linear_grads<MX, MW, true><<<plan.x.blocks + blocks, kThreads, 0, s>>>(c, b, x_blocks);       \
  else k_linear_grads<MX, MW, false><<<plan.x.blocks + blocks, kThreads, 0, s>>>(c, b, x_blocks);
    if (half) {
      EP_GRADS(2, 2)
    } else if (plan.x.mi == 4) {
      EP_GRADS(4, 4)
    } else {
      EP_GRADS(5, 4)
    }
#undef EP_GRADS
  } else if (half && a.xmap) k_linear<kGradW, 2, true><<<blocks, kThreads, 0, s>>>(b);
  else if (half) k_linear<kGradW, 2, false><<<blocks, kThreads, 0, s>>>(b);
  else if (a.xmap) k_linear<kGradW, 4, true><<<blocks, kThreads, 0, s>>>(b);
  else k_linear<kGradW, 4, false><<<blocks, kThreads, 0, s>>>(b);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  const int64_t nw = static_cast<int64_t>(a.E) * a.W * a.H, nb = static_cast<int64_t>(a.E) * a.W;
  k_linear_join<<<static_cast<unsigned>(ceil_div(nw + nb, 8 * kBlock)), kBlock, 0, s>>>(
      a.part, a.splits, nw, nb, a.gw, a.gb, a.status, a.generation);
  return hipGetLastError();
}

hipError_t launch_act_backward(const ActBackwardArgs& a, int64_t rows, hipStream_t s) {
  const int64_t blocks = ceil_div(rows, kWavesPerBlock);
  k_act_backward<<<static_cast<unsigned>(blocks < 8192 ? blocks : 8192), kBlock, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace ep
