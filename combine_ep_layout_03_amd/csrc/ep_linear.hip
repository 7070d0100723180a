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
// Tile and pipeline follow the grouped GEMM (ep_gemm.hip): 8 waves in 2 (rows)
// x 4 (columns), a wave owns MI sub-tiles of 32 rows and 64 columns in
// v_mfma_f32_32x32x16_bf16 accumulators, the contraction runs 32 at a time
// through LDS rings filled by LDS-direct loads, and the two waves of a SIMD
// take turns at reading operands and issuing matrix instructions.
#include "ep_expert.h"

namespace ep {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 512;
constexpr int kBN = 256;     // columns of a tile
constexpr int kBK = 32;      // contraction step
constexpr int kStages = 4;   // ring of 32-wide stages, three ahead
constexpr int kXBK = 2 * kBK;  // stage of a row operand that runs along memory (whole lines)
constexpr int kXcds = 8;
constexpr int kRowGroup = 8;  // row tiles that share a run of column tiles
constexpr int kOutPitch = 68;  // floats per row of a wave's epilogue slice

enum Kind { kForward, kGradX, kGradW };

// where lanes past the contraction's end load from
__device__ __align__(16) const uint32_t kZeros[4] = {0u, 0u, 0u, 0u};

__device__ __forceinline__ bf16x8 as_bf16x8(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return static_cast<uint32_t>(
      reinterpret_cast<uintptr_t>((const __attribute__((address_space(3))) void*)p));
}

__device__ __forceinline__ void load_lds16(const void* src, void* dst) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                   (__attribute__((address_space(3))) void*)dst, 16, 0, 0);
}

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

__device__ __forceinline__ float act_value(float z, int act) {
  switch (act) {
    case kActRelu: return z < 0.0f ? 0.0f : z;
    case kActSilu: return z * sigmoid(z);
    case kActGelu: return z * 0.5f * erfcf(-z * kSqrtHalf);
    case kActGeluTanh: return z * sigmoid(2.0f * kTanhScale * (z + kTanhCubic * z * z * z));
    default: return z;
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
      const float cdf = 0.5f * erfcf(-z * kSqrtHalf);
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
// One contraction step's operands of a wave: row sub-tiles i and column
// sub-tiles t, for the two 16-wide halves kk of the step.  The reads and the
// wait for them are one asm block, so no register is used before it is there.
template <int MI>
struct Frags {
  u32x4 col[2][2];
  u32x4 row[2][MI];
};
#define EP_RD(dst, at, off) "ds_read_b128 %[" dst "], %[" at "] offset:" off "\n\t"
#define EP_TR(dst, at, off) "ds_read_b64_tr_b16 %[" dst "], %[" at "] offset:" off "\n\t"
#define EP_COLS \
  EP_RD("w00", "c0", "0") EP_RD("w01", "c0", "2048") EP_RD("w10", "c1", "0") EP_RD("w11", "c1", "2048")
#define EP_COLS_OUT \
  [w00] "=&v"(f.col[0][0]), [w01] "=&v"(f.col[0][1]), [w10] "=&v"(f.col[1][0]), [w11] "=&v"(f.col[1][1])
#define EP_COLS_T                                                                                     \
  EP_TR("w000", "c0", "0") EP_TR("w001", "c0", "2048") EP_TR("w010", "c1", "0")                       \
  EP_TR("w011", "c1", "2048") EP_TR("w100", "c0", "8192") EP_TR("w101", "c0", "10240")                \
  EP_TR("w110", "c1", "8192") EP_TR("w111", "c1", "10240")
#define EP_COLS_T_OUT                                                                                 \
  [w000] "=&v"(c[0][0][0]), [w001] "=&v"(c[0][0][1]), [w010] "=&v"(c[0][1][0]),                       \
      [w011] "=&v"(c[0][1][1]), [w100] "=&v"(c[1][0][0]), [w101] "=&v"(c[1][0][1]),                   \
      [w110] "=&v"(c[1][1][0]), [w111] "=&v"(c[1][1][1])
#define EP_ROWS1 EP_RD("x00", "r0", "0") EP_RD("x10", "r1", "0")
#define EP_ROWS2 EP_ROWS1 EP_RD("x01", "r0", "8192") EP_RD("x11", "r1", "8192")
#define EP_ROWS4                                                                    \
  EP_ROWS2 EP_RD("x02", "r0", "16384") EP_RD("x12", "r1", "16384")                  \
  EP_RD("x03", "r0", "24576") EP_RD("x13", "r1", "24576")
#define EP_ROWS5 EP_ROWS4 EP_RD("x04", "r0", "32768") EP_RD("x14", "r1", "32768")
#define EP_ROWS1_OUT [x00] "=&v"(f.row[0][0]), [x10] "=&v"(f.row[1][0])
#define EP_ROWS2_OUT EP_ROWS1_OUT, [x01] "=&v"(f.row[0][1]), [x11] "=&v"(f.row[1][1])
#define EP_ROWS4_OUT                                                                       \
  EP_ROWS2_OUT, [x02] "=&v"(f.row[0][2]), [x12] "=&v"(f.row[1][2]), [x03] "=&v"(f.row[0][3]), \
      [x13] "=&v"(f.row[1][3])
#define EP_ROWS5_OUT EP_ROWS4_OUT, [x04] "=&v"(f.row[0][4]), [x14] "=&v"(f.row[1][4])
#define EP_IN [c0] "v"(c0), [c1] "v"(c1), [r0] "v"(r0), [r1] "v"(r1)
#define EP_WAIT "s_waitcnt lgkmcnt(0)"

// rows and columns along memory: r0, r1 and c0, c1 are the addresses of the
// two halves kk
template <int MI>
__device__ __forceinline__ void read_plain(Frags<MI>& f, uint32_t r0, uint32_t r1, uint32_t c0, uint32_t c1) {
  if constexpr (MI == 1) asm volatile(EP_COLS EP_ROWS1 EP_WAIT : EP_COLS_OUT, EP_ROWS1_OUT : EP_IN);
  if constexpr (MI == 2) asm volatile(EP_COLS EP_ROWS2 EP_WAIT : EP_COLS_OUT, EP_ROWS2_OUT : EP_IN);
  if constexpr (MI == 4) asm volatile(EP_COLS EP_ROWS4 EP_WAIT : EP_COLS_OUT, EP_ROWS4_OUT : EP_IN);
  if constexpr (MI == 5) asm volatile(EP_COLS EP_ROWS5 EP_WAIT : EP_COLS_OUT, EP_ROWS5_OUT : EP_IN);
}
// columns across memory: c0, c1 are the addresses of the two sub-tiles t
template <int MI>
__device__ __forceinline__ void read_cols_across(Frags<MI>& f, uint32_t r0, uint32_t r1, uint32_t c0, uint32_t c1) {
  u32x2 c[2][2][2];  // kk, t, contraction half
  if constexpr (MI == 1) asm volatile(EP_COLS_T EP_ROWS1 EP_WAIT : EP_COLS_T_OUT, EP_ROWS1_OUT : EP_IN);
  if constexpr (MI == 2) asm volatile(EP_COLS_T EP_ROWS2 EP_WAIT : EP_COLS_T_OUT, EP_ROWS2_OUT : EP_IN);
  if constexpr (MI == 4) asm volatile(EP_COLS_T EP_ROWS4 EP_WAIT : EP_COLS_T_OUT, EP_ROWS4_OUT : EP_IN);
  if constexpr (MI == 5) asm volatile(EP_COLS_T EP_ROWS5 EP_WAIT : EP_COLS_T_OUT, EP_ROWS5_OUT : EP_IN);
#pragma unroll
  for (int kk = 0; kk < 2; ++kk)
#pragma unroll
    for (int t = 0; t < 2; ++t) f.col[kk][t] = __builtin_shufflevector(c[kk][t][0], c[kk][t][1], 0, 1, 2, 3);
}
// both across memory: r0, r1 are the addresses of even and odd sub-tiles i
__device__ __forceinline__ void read_across(Frags<4>& f, uint32_t r0, uint32_t r1, uint32_t c0, uint32_t c1) {
  u32x2 c[2][2][2], x[2][4][2];
  asm volatile(EP_COLS_T                                                                              //
               EP_TR("x000", "r0", "0") EP_TR("x001", "r0", "2048") EP_TR("x010", "r1", "0")          //
               EP_TR("x011", "r1", "2048") EP_TR("x020", "r0", "256") EP_TR("x021", "r0", "2304")     //
               EP_TR("x030", "r1", "256") EP_TR("x031", "r1", "2304") EP_TR("x100", "r0", "8192")     //
               EP_TR("x101", "r0", "10240") EP_TR("x110", "r1", "8192") EP_TR("x111", "r1", "10240")  //
               EP_TR("x120", "r0", "8448") EP_TR("x121", "r0", "10496") EP_TR("x130", "r1", "8448")   //
               EP_TR("x131", "r1", "10496") EP_WAIT
               : EP_COLS_T_OUT, [x000] "=&v"(x[0][0][0]), [x001] "=&v"(x[0][0][1]),
                 [x010] "=&v"(x[0][1][0]), [x011] "=&v"(x[0][1][1]), [x020] "=&v"(x[0][2][0]),
                 [x021] "=&v"(x[0][2][1]), [x030] "=&v"(x[0][3][0]), [x031] "=&v"(x[0][3][1]),
                 [x100] "=&v"(x[1][0][0]), [x101] "=&v"(x[1][0][1]), [x110] "=&v"(x[1][1][0]),
                 [x111] "=&v"(x[1][1][1]), [x120] "=&v"(x[1][2][0]), [x121] "=&v"(x[1][2][1]),
                 [x130] "=&v"(x[1][3][0]), [x131] "=&v"(x[1][3][1])
               : EP_IN);
#pragma unroll
  for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
    for (int t = 0; t < 2; ++t) f.col[kk][t] = __builtin_shufflevector(c[kk][t][0], c[kk][t][1], 0, 1, 2, 3);
#pragma unroll
    for (int i = 0; i < 4; ++i) f.row[kk][i] = __builtin_shufflevector(x[kk][i][0], x[kk][i][1], 0, 1, 2, 3);
  }
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

// Number of the block in an order where each XCD takes a contiguous run
// (blocks are dealt to the 8 XCDs round-robin); false past `total`.
__device__ __forceinline__ bool xcd_run(int64_t total, int64_t& tile) {
  const int64_t per = (total + kXcds - 1) / kXcds;
  const int64_t seat = blockIdx.x / kXcds;
  if (seat >= per) return false;
  tile = static_cast<int64_t>(blockIdx.x % kXcds) * per + seat;
  return tile < total;
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

template <Kind KIND, int MI, bool GATHER>
__global__ __launch_bounds__(kThreads) void k_linear(LinearArgs a) {
  constexpr bool kRowAcross = KIND == kGradW;    // row operand's contraction runs across memory
  constexpr bool kColAcross = KIND != kForward;  // column operand's
  static_assert(!kRowAcross || MI == 4, "a row operand across memory is 256 wide");
  constexpr int kBM = 64 * MI;
  constexpr int kRowStages = kRowAcross ? kStages : 2;
  constexpr int kRowBytes = kRowAcross ? kBK * kBM * 2 : kBM * kXBK * 2;  // of a stage
  constexpr int kColBytes = kBN * kBK * 2;
  constexpr int kRing = kRowStages * kRowBytes + kStages * kColBytes;
  constexpr int kOut = 8 * 32 * kOutPitch * 4;
  static_assert((1024 + 16 + kThreads / kWave) * sizeof(int) <= kRing, "tile table fits");
  __shared__ __align__(1024) char lds[kRing > kOut ? kRing : kOut];
  char* const sRow = lds;
  char* const sCol = lds + kRowStages * kRowBytes;

  if (!layout_current(a.status, a.generation)) return;
  const int tid = threadIdx.x;
  const int lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);

  // ---- the block's tile
  Tile T;
  const int nt = KIND == kForward ? (a.N + (a.gated ? kBN / 2 : kBN) - 1) / (a.gated ? kBN / 2 : kBN)
                                  : (a.H + kBN - 1) / kBN;
  if constexpr (KIND == kGradW) {
    const int mt = (a.W + kBM - 1) / kBM;
    int64_t tile;
    if (!xcd_run(static_cast<int64_t>(a.E) * a.splits * mt * nt, tile)) return;
    const int es = static_cast<int>(tile / (mt * nt));
    int im, jn;
    tile_of(static_cast<int>(tile - static_cast<int64_t>(es) * mt * nt), mt, nt, im, jn);
    T.e = es / a.splits;
    T.split = es - T.e * a.splits;
    const int cnt = a.counts[T.e];
    const int per = ((cnt + a.splits - 1) / a.splits + kBK - 1) / kBK * kBK;
    const int first = min(cnt, per * T.split);
    T.row0 = a.offsets[T.e] + first;
    T.k = min(per, cnt - first);
    T.r0 = im * kBM;
    T.nrows = min(kBM, a.W - T.r0);
    T.n0 = jn * kBN;
  } else {
    // row tiles of each expert times column tiles, then their exclusive
    // prefix (the same in every block); the table lies in the ring until the
    // first load
    int* const sTiles = reinterpret_cast<int*>(lds);
    int* const sTmp = sTiles + 1024 + 8;
    for (int e = tid; e < a.E; e += kThreads) sTiles[e] = (a.counts[e] + kBM - 1) / kBM * nt;
    __syncthreads();
    const int total = block_exclusive_scan<kThreads>(sTiles, a.E, sTmp);
    int64_t tile;
    if (!xcd_run(total, tile)) return;
    // the last expert whose first tile is not past it (empty ones repeat the
    // prefix of the next)
    int lo = 0, hi = a.E - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (sTiles[mid] <= tile) lo = mid;
      else hi = mid - 1;
    }
    T.e = lo;
    const int cnt = a.counts[lo];
    const int mt = (cnt + kBM - 1) / kBM;
    int im, jn;
    tile_of(static_cast<int>(tile) - sTiles[lo], mt, nt, im, jn);
    // the rows split evenly over the tiles, in steps of 32: none is empty
    const int per = ((cnt + mt - 1) / mt + 31) / 32 * 32;
    T.row0 = a.offsets[lo] + im * per;
    T.nrows = min(per, cnt - im * per);
    T.n0 = jn * (KIND == kForward && a.gated ? kBN / 2 : kBN);
    T.k = KIND == kForward ? a.H : a.W;
    T.r0 = 0;
    T.split = 0;
    __syncthreads();  // the table is read before the ring's first load
  }

  // ---- loads: waves 0-3 fill the row ring, waves 4-7 the column ring
  constexpr int kRowLoads = kRowBytes / 4096;  // per wave and stage, 1 KiB each
  constexpr int kColLoads = kColBytes / 4096;
  constexpr int kLoads = kRowLoads > kColLoads ? kRowLoads : kColLoads;
  const bool row_wave = wave < 4;
  // Stage 0's addresses: a base that the wave shares and each lane's offset
  // of it (bytes; for gathered rows, that may lie anywhere, in 16 bytes).
  const char* base;
  uint32_t off[kLoads];
#pragma unroll
  for (int q = 0; q < kLoads; ++q) {
    if (row_wave) {
      const int s = (wave * kRowLoads + (q < kRowLoads ? q : 0)) * 64 + lane;
      if constexpr (kRowAcross) {
        const int k = s >> 5, p = s & 31;
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
      const int s = ((wave - 4) * kColLoads + (q < kColLoads ? q : 0)) * 64 + lane;
      if constexpr (kColAcross) {
        const int k = s >> 5, p = s & 31;
        const int c = T.n0 + ((p >> 1) ^ ((k & 3) << 1)) * 16 + (p & 1) * 8;
        const int col = c < a.H ? c : 0;
        if constexpr (KIND == kGradX) off[q] = static_cast<uint32_t>((static_cast<int64_t>(k) * a.H + col) * 2);
        else off[q] = static_cast<uint32_t>((GATHER ? col : k * a.ldx + col) * 2);
      } else {
        const int r = s >> 2;
        const int kv = (s & 3) ^ ((r >> 2) & 3);
        // tile column -> row of w; gated tiles take 32 gate and 32 up rows a
        // wave, and the base of the loads q = 2, 3 is the up half's
        const int n = a.gated ? (r >> 6) * 32 + (r & 31) : r;
        off[q] = static_cast<uint32_t>((static_cast<int64_t>(T.n0 + n < a.N ? n : 0) * a.H + kv * 8) * 2);
      }
    }
  }
  if (row_wave) {
    if constexpr (kRowAcross) base = reinterpret_cast<const char*>(a.g + T.row0 * a.ldg);
    else if constexpr (KIND == kGradX) base = reinterpret_cast<const char*>(a.g + T.row0 * a.ldg);
    else base = reinterpret_cast<const char*>(GATHER ? a.x : a.x + T.row0 * a.ldx);
  } else {
    if constexpr (KIND == kGradW) base = reinterpret_cast<const char*>(GATHER ? a.x : a.x + T.row0 * a.ldx);
    else if constexpr (KIND == kGradX) base = reinterpret_cast<const char*>(a.w + static_cast<int64_t>(T.e) * a.W * a.H);
    else base = reinterpret_cast<const char*>(a.w + (static_cast<int64_t>(T.e) * a.W + T.n0) * a.H);
  }
  const int64_t up_half = KIND == kForward && a.gated ? static_cast<int64_t>(a.N) * a.H * 2 : 0;
  const int nk = (T.k + kBK - 1) / kBK;
  const int nsx = (nk + 1) / 2;  // 64-wide stages

  auto issue_row = [&](int st) __attribute__((always_inline)) {
    char* const to = sRow + (st % kRowStages) * kRowBytes + wave * kRowLoads * 1024;
    constexpr int kWide = kRowAcross ? kBK : kXBK;
    const char* const from = base + st * (kRowAcross ? kBK * a.ldg * 2 : kXBK * 2);
    const bool whole = (st + 1) * kWide <= T.k;
    auto at = [&](int q) { return from + (KIND == kForward && GATHER ? static_cast<uint64_t>(off[q]) << 4 : off[q]); };
#pragma unroll
    for (int q = 0; q < kRowLoads; ++q) {
      const char* p = at(q);
      if (!whole) {
        const int s = (wave * kRowLoads + q) * 64 + lane;
        const int k = kRowAcross ? s >> 5 : ((s & 7) ^ ((s >> 4) & 7)) * 8;
        if (st * kWide + k >= T.k) p = reinterpret_cast<const char*>(kZeros);
      }
      load_lds16(p, to + q * 1024);
    }
  };
  // grad_w on gathered rows: token of this wave's 8 contraction rows of a
  // stage, one a lane, loaded a stage ahead
  int token = 0;
  auto next_token = [&](int st) __attribute__((always_inline)) {
    if constexpr (KIND == kGradW && GATHER) {
      const int k = st * kBK + (wave - 4) * 8 + (lane & 7);
      token = a.xmap[T.row0 + (k < T.k ? k : T.k - 1)];
    }
  };
  auto issue_col = [&](int st) __attribute__((always_inline)) {
    char* const to = sCol + (st % kStages) * kColBytes + (wave - 4) * kColLoads * 1024;
    const bool whole = (st + 1) * kBK <= T.k;
    constexpr bool kRowsApart = KIND == kGradW && GATHER;
    const char* const from =
        kRowsApart ? base : base + st * (KIND == kForward ? kBK * 2 : static_cast<int64_t>(kBK) * (KIND == kGradX ? a.H : a.ldx) * 2);
    int64_t row[kColLoads];
    if constexpr (kRowsApart) {
#pragma unroll
      for (int q = 0; q < kColLoads; ++q) {
        const int lo = __builtin_amdgcn_readlane(token, 2 * q);
        const int hi = __builtin_amdgcn_readlane(token, 2 * q + 1);
        row[q] = (lane < 32 ? lo : hi) * a.ldx * 2;
      }
      next_token(st + 1);
    }
    auto at = [&](int q) {
      if constexpr (kRowsApart) return from + off[q] + row[q];
      else return from + (KIND == kForward && q >= 2 ? up_half : 0) + off[q];
    };
    if (whole) {
#pragma unroll
      for (int q = 0; q < kColLoads; ++q) load_lds16(at(q), to + q * 1024);
    } else {
      int l = lane;
      asm volatile("" : "+v"(l));
#pragma unroll
      for (int q = 0; q < kColLoads; ++q) {
        const int s = ((wave - 4) * kColLoads + q) * 64 + l;
        const int k = kColAcross ? s >> 5 : ((s & 3) ^ ((s >> 4) & 3)) * 8;
        load_lds16(st * kBK + k < T.k ? at(q) : reinterpret_cast<const char*>(kZeros), to + q * 1024);
      }
    }
  };
  // this wave's loads of the stages that step kt reads have landed.  A
  // 64-wide row stage kt / 2: stages 0 and 1 are issued up front and stage
  // s + 1 at step 2 s (s >= 1).  A 32-wide stage kt: kt + 1 and kt + 2 are
  // younger.  (With gathered rows a token load may be younger too: then a
  // load or two more than needed is waited for.)
  auto wait_own = [&](int kt) __attribute__((always_inline)) {
    if (row_wave && !kRowAcross) {
      const int sx = kt >> 1;
      const int issued = min(nsx - 1, (kt & 1) ? sx + 1 : max(sx, 1));
      wait_vm(kRowLoads * (issued - sx));
    } else {
      wait_vm(4 * min(kStages - 2, nk - 1 - kt));
    }
  };
  // after step kt's first barrier: the stage whose slot was read last at step
  // kt - 1, by both halves before that barrier
  auto issue_next = [&](int kt) __attribute__((always_inline)) {
    if (row_wave && !kRowAcross) {
      if (!(kt & 1) && kt >= 2 && (kt >> 1) + 1 < nsx) issue_row((kt >> 1) + 1);
    } else if (kt + kStages - 1 < nk) {
      if (row_wave) issue_row(kt + kStages - 1);
      else issue_col(kt + kStages - 1);
    }
  };

  const int wm = wave >> 2;   // row half: sub-tiles wm, wm + 2, ...
  const int wn = wave & 3;    // 64-column slab
  const int lr = lane & 31;   // operand row within a sub-tile
  const int lkv = lane >> 5;  // 8-wide part of a 16-step
  // sub-tiles of this wave with a valid row (none if its columns lie past the end)
  int live = 0;
#pragma unroll
  for (int i = 0; i < MI; ++i) live += (2 * i + wm) * 32 < T.nrows ? 1 : 0;
  const int cols = KIND == kForward ? a.N : a.H;  // columns of the output
  const int col0 = T.n0 + wn * (KIND == kForward && a.gated ? 32 : 64);
  if (col0 >= cols) live = 0;

  f32x16 acc[MI][2];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int t = 0; t < 2; ++t) acc[i][t] = f32x16{};
  // grad_w: column sums of g for the bias, sub-tile i = wn of the first
  // column tile's waves
  float bias_sum = 0.0f;
  const bool want_bias = KIND == kGradW && a.gb != nullptr && T.n0 == 0;
  int mine[MI];  // i == wn, in terms that the compiler cannot make an index (and scratch memory) of
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    mine[i] = __builtin_amdgcn_readfirstlane(i == wn);
    if constexpr (KIND == kGradW) asm volatile("" : "+s"(mine[i]));
  }

  // operand addresses within a stage
  const int j16 = lane & 15, g2 = (lane >> 4) & 1;
  const uint32_t row_at =
      lds_addr(sRow) + (kRowAcross ? (lkv * 8 + (j16 >> 2)) * 512 + ((wm * 2 + g2) ^ ((j16 >> 2) << 1)) * 32 + (j16 & 3) * 8
                                   : (wm * 32 + lr) * 128 + (lkv ^ ((lr >> 1) & 7)) * 16);
  const uint32_t col_at =
      lds_addr(sCol) + (kColAcross ? (lkv * 8 + (j16 >> 2)) * 512 + ((wn * 4 + g2) ^ ((j16 >> 2) << 1)) * 32 + (j16 & 3) * 8
                                   : (wn * 64 + lr) * 64 + (lkv ^ ((lr >> 2) & 3)) * 16);
  Frags<MI> f;
  auto read_stage = [&](int kt) __attribute__((always_inline)) {
    const uint32_t c = col_at + (kt % kStages) * kColBytes;
    if constexpr (kRowAcross) {
      const uint32_t r = row_at + (kt % kStages) * kRowBytes;
      read_across(f, r, r ^ 128u, c, c ^ 64u);
    } else {
      const uint32_t r = (row_at + ((kt >> 1) % kRowStages) * kRowBytes) ^ ((kt & 1) << 6);
      if constexpr (kColAcross) read_cols_across<MI>(f, r, r ^ 32u, c, c ^ 64u);
      else read_plain<MI>(f, r, r ^ 32u, c, c ^ 32u);
    }
  };
  auto mfma_stage = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        if (i < live) {
#pragma unroll
          for (int t = 0; t < 2; ++t)
            acc[i][t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(f.col[kk][t]), as_bf16x8(f.row[kk][i]),
                                                                acc[i][t], 0, 0, 0);
        }
      }
    }
    if constexpr (KIND == kGradW) {
      if (want_bias) {
#pragma unroll
        for (int i = 0; i < MI; ++i) {
          if (mine[i]) {
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
              for (int d = 0; d < 4; ++d) bias_sum += bf16_lo(f.row[kk][i][d]) + bf16_hi(f.row[kk][i][d]);
          }
        }
      }
    }
  };

  // The two waves of a SIMD (one of each row half) run half a step apart: one
  // reads its operands while the other issues matrix instructions.  Both
  // loops pass the same barriers in the same order.
  if (row_wave) {
    if constexpr (kRowAcross) {
      for (int kt = 0; kt < kStages - 1 && kt < nk; ++kt) issue_row(kt);
    } else {
      issue_row(0);
      if (nsx > 1) issue_row(1);
    }
  } else {
    if (nk > 0) next_token(0);
    for (int kt = 0; kt < kStages - 1 && kt < nk; ++kt) issue_col(kt);
  }
  const bool work = live > 0 || want_bias;
  if (wm == 0) {
    for (int kt = 0; kt < nk; ++kt) {
      wait_own(kt);
      block_sync();
      issue_next(kt);
      if (work) read_stage(kt);
      block_sync();
      if (work) mfma_stage();
    }
  } else {
    for (int kt = 0; kt < nk; ++kt) {
      wait_own(kt);
      block_sync();
      issue_next(kt);
      if (kt > 0 && work) mfma_stage();
      block_sync();
      if (work) read_stage(kt);
    }
    if (nk > 0 && work) mfma_stage();
  }

  // ---- epilogue.  Lane l of D holds row l % 32 and the columns
  // (i / 4) * 8 + (l / 32) * 4 + i % 4 of each sub-tile.  A wave turns each
  // sub-tile through its own slice of LDS, so that 8 lanes hold a row's 64
  // columns, 8 each, and every store is 16 bytes of a whole line.
  __syncthreads();
  if constexpr (KIND == kGradW) {
    if (want_bias) {
      const float sum = bias_sum + __shfl_xor(bias_sum, 32, kWave);
      const int n = T.r0 + (2 * wn + wm) * 32 + lr;
      if (lkv == 0 && n < a.W) {
        if (a.splits == 1) a.gb[static_cast<int64_t>(T.e) * a.W + n] = bf16_of(sum);
        else
          a.part[static_cast<int64_t>(a.splits) * a.E * a.W * a.H +
                 (static_cast<int64_t>(T.split) * a.E + T.e) * a.W + n] = sum;
      }
    }
  }
  float* const slice = reinterpret_cast<float*>(lds) + wave * 32 * kOutPitch;
  auto settle = [&]() __attribute__((always_inline)) {  // this wave's LDS writes before its reads, and back
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  };
#pragma unroll 1  // one copy of the activations' code
  for (int now = 0; now < live; ++now) {
    const int sub = (2 * now + wm) * 32;
    settle();
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      if (i != now) continue;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const f32x4 v = {acc[i][t][4 * g], acc[i][t][4 * g + 1], acc[i][t][4 * g + 2], acc[i][t][4 * g + 3]};
          *reinterpret_cast<f32x4*>(slice + lr * kOutPitch + t * 32 + g * 8 + lkv * 4) = v;
        }
    }
    settle();
    const int rows = min(32, T.nrows - sub);
    const bool gated = KIND == kForward && a.gated;
    const int per_row = gated ? 4 : 8;  // lanes of a row
    for (int it = lane; it < 32 * per_row; it += kWave) {
      const int r = it / per_row, c = it % per_row * 8;
      const int n = col0 + c;
      if (r >= rows || n >= cols) continue;
      float v[8];
      *reinterpret_cast<f32x4*>(v) = *reinterpret_cast<const f32x4*>(slice + r * kOutPitch + c);
      *reinterpret_cast<f32x4*>(v + 4) = *reinterpret_cast<const f32x4*>(slice + r * kOutPitch + c + 4);
      auto store8 = [&](uint16_t* to, const float* x) __attribute__((always_inline)) {
        u32x4 b;
#pragma unroll
        for (int d = 0; d < 4; ++d) b[d] = bf16x2_of(x[2 * d], x[2 * d + 1]);
        *reinterpret_cast<u32x4*>(to) = b;
      };
      auto add8 = [&](float* x, const uint16_t* from) __attribute__((always_inline)) {
        const u32x4 b = *reinterpret_cast<const u32x4*>(from);
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          x[2 * d] += bf16_lo(b[d]);
          x[2 * d + 1] += bf16_hi(b[d]);
        }
      };
      if constexpr (KIND == kForward) {
        const int64_t row = T.row0 + sub + r;
        const uint16_t* bias = a.bias ? a.bias + static_cast<int64_t>(T.e) * a.W : nullptr;
        if (bias) add8(v, bias + n);
        if (a.pre) store8(a.pre + row * a.ldpre + n, v);
#pragma unroll
        for (int d = 0; d < 8; ++d) v[d] = act_value(v[d], a.act);
        if (gated) {
          float u[8];
          *reinterpret_cast<f32x4*>(u) = *reinterpret_cast<const f32x4*>(slice + r * kOutPitch + 32 + c);
          *reinterpret_cast<f32x4*>(u + 4) = *reinterpret_cast<const f32x4*>(slice + r * kOutPitch + 36 + c);
          if (bias) add8(u, bias + a.N + n);
          if (a.pre) store8(a.pre + row * a.ldpre + a.N + n, u);
#pragma unroll
          for (int d = 0; d < 8; ++d) v[d] *= u[d];
        }
        if (a.res) add8(v, a.res + row * a.ldres + n);
        store8(a.out + row * a.ldout + n, v);
      } else if constexpr (KIND == kGradX) {
        store8(a.out + (T.row0 + sub + r) * a.ldout + n, v);
      } else {
        const int64_t at = (static_cast<int64_t>(T.e) * a.W + T.r0 + sub + r) * a.H + n;
        if (a.splits == 1) {
          store8(a.gw + at, v);
        } else {
          float* to = a.part + static_cast<int64_t>(T.split) * a.E * a.W * a.H + at;
          *reinterpret_cast<f32x4*>(to) = *reinterpret_cast<const f32x4*>(v);
          *reinterpret_cast<f32x4*>(to + 4) = *reinterpret_cast<const f32x4*>(v + 4);
        }
      }
    }
  }
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

// 8 columns a lane; a wave walks the columns of one row.
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

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

unsigned xcd_grid(int64_t tiles) { return static_cast<unsigned>(ceil_div(tiles, kXcds) * kXcds); }

int64_t row_tiles(int64_t rows, int E, int bm) { return ceil_div(rows, bm) + (rows < E ? rows : E); }

template <Kind KIND, bool GATHER>
hipError_t launch_rows(const LinearArgs& a, int64_t rows, int64_t nt, hipStream_t s) {
  // tile height by the rows an expert has if all have the same
  const int64_t avg = rows / a.E;
  if (avg <= 64) k_linear<KIND, 1, GATHER><<<xcd_grid(row_tiles(rows, a.E, 64) * nt), kThreads, 0, s>>>(a);
  else if (avg <= 128) k_linear<KIND, 2, GATHER><<<xcd_grid(row_tiles(rows, a.E, 128) * nt), kThreads, 0, s>>>(a);
  else k_linear<KIND, 5, GATHER><<<xcd_grid(row_tiles(rows, a.E, 320) * nt), kThreads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

LinearGeom linear_geom(int64_t rows, int E, int H, int W) {
  LinearGeom g;
  g.rows = rows;
  const int64_t tiles = ceil_div(W, 256) * ceil_div(H, kBN) * E;
  // enough blocks for the chip, and 256 rows of an even share at least
  int64_t splits = tiles < 512 ? 512 / tiles : 1;
  const int64_t most = rows / E / 256;
  if (splits > most) splits = most;
  g.splits = static_cast<int>(splits > 1 ? splits : 1);
  g.part_bytes = g.splits > 1 ? (static_cast<size_t>(W) * H + W) * E * g.splits * 4 : 0;
  return g;
}

int64_t linear_max_tiles(int64_t rows, int E, int H, int W, int splits) {
  // columns of 128 (gated) or 256; rows of 64 at least
  const int64_t wide = ceil_div(W > H ? W : H, 128);
  const int64_t by_rows = row_tiles(rows, E, 64) * wide;
  const int64_t by_weights = ceil_div(W, 256) * ceil_div(H, kBN) * E * splits;
  return by_rows > by_weights ? by_rows : by_weights;
}

hipError_t launch_linear(const LinearArgs& a, int64_t rows, hipStream_t s) {
  const int64_t nt = ceil_div(a.N, a.gated ? kBN / 2 : kBN);
  return a.xmap ? launch_rows<kForward, true>(a, rows, nt, s) : launch_rows<kForward, false>(a, rows, nt, s);
}

hipError_t launch_linear_grad_x(const LinearArgs& a, int64_t rows, hipStream_t s) {
  return launch_rows<kGradX, false>(a, rows, ceil_div(a.H, kBN), s);
}

hipError_t launch_linear_grad_w(const LinearArgs& a, hipStream_t s) {
  const int64_t tiles = ceil_div(a.W, 256) * ceil_div(a.H, kBN) * a.E * a.splits;
  if (a.xmap) k_linear<kGradW, 4, true><<<xcd_grid(tiles), kThreads, 0, s>>>(a);
  else k_linear<kGradW, 4, false><<<xcd_grid(tiles), kThreads, 0, s>>>(a);
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
