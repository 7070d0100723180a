// The router's balance loss and its gradient.
//
// With p[t] a token's scores over their sum and, for each sequence b, n its
// tokens, c[e] its selections of expert e and m[e] the mean of p[t, e],
//     loss = coef / B sum_b E / (K n) sum_e c[e] m[e]
//     grad_logits[t, e] = p_e (f_e - sum_j f_j p_j) (* 1 - s_e for sigmoid),
//     f_e = grad_loss coef E c[e] / (B K n^2).
//
// The logits are read once (65,536 x 256 fp32: 67 MB).  Forward 20 us, bound by
// the latency of each element's exponential and quotient, and 10 us of the join;
// the gradient with a base is bound by memory, 45 us for 201 MB (47 without
// loading a row ahead).  A token has 16 lanes (64 above 256 experts), so a wave
// works on four tokens at once and a token's maximum and sum cost four lane
// moves within a row of 16.  A lane keeps the same experts for every token of
// its block, so the sums over tokens stay in registers until the block's tokens
// of a sequence are through, and the gradient's f does.  Sums go block by block
// into slots of the workspace and a second kernel adds the slots in their order:
// no floating-point atomics, equal inputs give equal bytes.
#include <float.h>

#include "ep_expert.h"

namespace ep {

namespace {

constexpr float kNegInf = -__builtin_inff();
constexpr int kJoinCols = 16;      // columns of a join block
constexpr int kJoinThreads = 512;  // 16 columns x 32 runs of slots

// v of the lane n further on in the row of 16
template <int N>
__device__ __forceinline__ float turned(float v) {
  return __uint_as_float(static_cast<uint32_t>(
      __builtin_amdgcn_update_dpp(0, static_cast<int>(__float_as_uint(v)), 0x120 + N, 0xF, 0xF, true)));
}
struct Add {
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
struct Larger {
  __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
// f over a token's LPT lanes, in every one of them
template <int LPT, typename F>
__device__ __forceinline__ float over_token(float v, F f) {
  v = f(v, turned<8>(v));
  v = f(v, turned<4>(v));
  v = f(v, turned<2>(v));
  v = f(v, turned<1>(v));
  if constexpr (LPT == 64) {
    v = f(v, __shfl_xor(v, 16, kWave));
    v = f(v, __shfl_xor(v, 32, kWave));
  }
  return v;
}

// NaN -> -inf (out), +inf -> the largest finite value
__device__ __forceinline__ float clean(float l) { return l != l ? kNegInf : fminf(l, FLT_MAX); }

// NE elements of a row for lane g of LPT: vectors of V, LPT * V apart;
// elements past E are `past`.
template <int LPT, int NE, int V>
__device__ __forceinline__ int element(int g, int i) {
  return (i / V) * (LPT * V) + g * V + i % V;
}
template <int LPT, int NE, int V>
__device__ __forceinline__ void load_row(const float* row, int g, int E, float past, float (&v)[NE]) {
#pragma unroll
  for (int i = 0; i < NE; i += V) {
    const int e = element<LPT, NE, V>(g, i);
    if constexpr (V == 4) {
      f32x4_t x = {past, past, past, past};
      if (e < E) x = *reinterpret_cast<const f32x4_t*>(row + e);
#pragma unroll
      for (int d = 0; d < 4; ++d) v[i + d] = x[d];
    } else {
      v[i] = e < E ? row[e] : past;
    }
  }
}
template <int LPT, int NE, int V>
__device__ __forceinline__ void load_row(const uint16_t* row, int g, int E, float past, float (&v)[NE]) {
#pragma unroll
  for (int i = 0; i < NE; i += V) {
    const int e = element<LPT, NE, V>(g, i);
    if constexpr (V == 4) {
      if (e < E) {
        const u32x2 x = *reinterpret_cast<const u32x2*>(row + e);
        v[i] = bf16_lo(x[0]);
        v[i + 1] = bf16_hi(x[0]);
        v[i + 2] = bf16_lo(x[1]);
        v[i + 3] = bf16_hi(x[1]);
      } else {
#pragma unroll
        for (int d = 0; d < 4; ++d) v[i + d] = past;
      }
    } else {
      v[i] = e < E ? bf16_to_f32(row[e]) : past;
    }
  }
}
template <int LPT, int NE, int V>
__device__ __forceinline__ void store_row(float* row, int g, int E, const float (&v)[NE]) {
#pragma unroll
  for (int i = 0; i < NE; i += V) {
    const int e = element<LPT, NE, V>(g, i);
    if (e >= E) continue;
    if constexpr (V == 4) *reinterpret_cast<f32x4_t*>(row + e) = f32x4_t{v[i], v[i + 1], v[i + 2], v[i + 3]};
    else row[e] = v[i];
  }
}
template <int LPT, int NE, int V>
__device__ __forceinline__ void store_row(uint16_t* row, int g, int E, const float (&v)[NE]) {
#pragma unroll
  for (int i = 0; i < NE; i += V) {
    const int e = element<LPT, NE, V>(g, i);
    if (e >= E) continue;
    if constexpr (V == 4) *reinterpret_cast<u32x2*>(row + e) = u32x2{bf16x2_of(v[i], v[i + 1]), bf16x2_of(v[i + 2], v[i + 3])};
    else row[e] = bf16_of(v[i]);
  }
}

// A token's logits l (cleaned here) become its shares p; `rest` = 1 - s.
// Sigmoid scores are formed relative to exp(min(top, 0)), so that a token
// whose scores all underflow still has shares.
template <int LPT, int NE>
__device__ __forceinline__ void shares(float (&l)[NE], bool sigmoid, float (&rest)[NE]) {
  float top = kNegInf;
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    l[i] = clean(l[i]);
    top = fmaxf(top, l[i]);
  }
  top = over_token<LPT>(top, Larger());
  if (top == kNegInf) top = 0.0f;  // every expert out
  const float below = fminf(top, 0.0f);
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const float x = l[i];
    if (sigmoid) {
      const float q = __expf(-fabsf(x));  // exp(-inf) = 0 for an expert that is out
      const float r = __builtin_amdgcn_rcpf(1.0f + q);
      rest[i] = x >= 0.0f ? q * r : r;
      // below = 0 but for tokens of negative logits alone
      l[i] = x >= 0.0f ? r : (below < 0.0f ? __expf(x - below) : q) * r;
    } else {
      rest[i] = 1.0f;
      l[i] = __expf(x - top);
    }
    sum += l[i];
  }
  sum = over_token<LPT>(sum, Add());
  const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
  for (int i = 0; i < NE; ++i) l[i] *= inv;
}

__device__ __forceinline__ int64_t offset_of(const BalanceArgs& a, int b) {
  if (!a.seq) return b == 0 ? 0 : a.T;
  const int64_t v = a.seq[b];
  return v < 0 ? 0 : v > a.T ? a.T : v;
}
// the first sequence that ends past token t (B: none), by 64 probes at a time
__device__ __forceinline__ int sequence_at(const BalanceArgs& a, int64_t t) {
  int lo = 0, n = a.B;  // it is one of lo .. lo + n
  while (n > 0) {
    const int step = (n + kWave - 1) / kWave;
    // lane l: does the last of the l-th `step` sequences end past t?
    const int last = lo + min((lane_id() + 1) * step, n) - 1;
    const uint64_t past = ballot(lane_id() * step < n && offset_of(a, last + 1) > t);
    if (past == 0) return lo + n;
    const int l = __builtin_ctzll(past);
    lo += l * step;
    if (step == 1) return lo;
    n = min(step, n - l * step) - 1;  // the last one is past t
  }
  return lo;
}

template <int LPT, int NE, int V, typename LT>
__global__ __launch_bounds__(kBlock) void k_balance(BalanceArgs a, int chunk) {
  constexpr int kPer = kWave / LPT;  // tokens of a wave at once
  constexpr int kEarly = 2;          // ids a thread: 64 tokens of top-8
  __shared__ float s_sum[kWavesPerBlock][LPT * NE];
  __shared__ int s_count[1024];
  __shared__ int s_tokens;
  const int tid = threadIdx.x;
  const int lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int g = lane & (LPT - 1);
  const LT* logits = static_cast<const LT*>(a.logits);
  if (blockIdx.x == 0 && tid == 0) *a.done = 0;  // for the join
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * chunk;
  const int64_t t1 = t0 + chunk < a.T ? t0 + chunk : a.T;
  for (int b = sequence_at(a, t0); b < a.B; ++b) {
    const int64_t first = offset_of(a, b);
    if (first >= t1) break;
    const int64_t lo = first > t0 ? first : t0;
    const int64_t end = offset_of(a, b + 1);
    const int64_t hi = end < t1 ? end : t1;
    if (hi <= lo) continue;
    for (int e = tid; e < a.E; e += kBlock) s_count[e] = 0;
    if (tid == 0) s_tokens = 0;
    __syncthreads();
    float acc[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) acc[i] = 0.0f;
    int live = 0;
    // a row is loaded while the one before is worked on
    float next[NE];
    bool next_live = false;
    auto fetch = [&](int64_t t) __attribute__((always_inline)) {
      next_live = t < hi && (!a.mask || a.mask[t]);
      if (t < hi) load_row<LPT, NE, V>(logits + t * a.E, g, a.E, kNegInf, next);
    };
    int64_t t = lo + wave * kPer + lane / LPT;
    fetch(t);
    // the first ids are on their way meanwhile (T K < 2^31)
    const uint32_t id_end = static_cast<uint32_t>(hi * a.K);
    uint32_t at = static_cast<uint32_t>(lo * a.K) + tid;
    int64_t early[kEarly];
#pragma unroll
    for (int j = 0; j < kEarly; ++j) early[j] = at + j * kBlock < id_end ? a.idx[at + j * kBlock] : -1;
    for (; t < hi; t += kWavesPerBlock * kPer) {
      float l[NE], rest[NE];
#pragma unroll
      for (int i = 0; i < NE; ++i) l[i] = next[i];
      const bool on = next_live;
      fetch(t + kWavesPerBlock * kPer);
      if (!on) continue;
      shares<LPT>(l, a.sigmoid, rest);
#pragma unroll
      for (int i = 0; i < NE; ++i) acc[i] += l[i];
      live += g == 0;
    }
    // the wave's tokens side by side, then the waves
    if constexpr (LPT == 16) {
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        acc[i] += __shfl_xor(acc[i], 16, kWave);
        acc[i] += __shfl_xor(acc[i], 32, kWave);
      }
    }
    if (lane < LPT) {
#pragma unroll
      for (int i = 0; i < NE; ++i) s_sum[wave][element<LPT, NE, V>(g, i)] = acc[i];
    }
    if (live) atomicAdd(&s_tokens, live);
    auto count = [&](uint32_t i, int64_t e) __attribute__((always_inline)) {
      if (e >= 0 && e < a.E && (!a.mask || a.mask[i / static_cast<uint32_t>(a.K)])) atomicAdd(&s_count[e], 1);
    };
#pragma unroll
    for (int j = 0; j < kEarly; ++j) count(at + j * kBlock, early[j]);
    for (at += kEarly * kBlock; at < id_end; at += kBlock) count(at, a.idx[at]);
    __syncthreads();
    const int64_t slot = blockIdx.x + static_cast<int64_t>(b);
    for (int e = tid; e < a.E; e += kBlock) {
      float v = s_sum[0][e];
#pragma unroll
      for (int w = 1; w < kWavesPerBlock; ++w) v += s_sum[w][e];
      a.part_sum[slot * a.E + e] = v;
      a.part_count[slot * a.E + e] = s_count[e];
    }
    if (tid == 0) a.part_tokens[slot] = s_tokens;
    __syncthreads();
  }
}

// A block's part of the loss, as a double, goes into two words of the workspace
// that no other block reads or writes: the block's first item is (b, 16 columns),
// and the first slot of sequence b (going by where b begins, if it is empty) has
// a sum and a count for the first of those columns, which only this item reads.
constexpr int kMaxJoins = 1024;
__device__ __forceinline__ int64_t part_at(const BalanceArgs& a, int chunk, int cols, int block) {
  const int b = block / cols;
  return (offset_of(a, b) / chunk + b) * a.E + block % cols * kJoinCols;
}

// Item (b, 16 columns): the slots of sequence b added up, 32 runs of slots
// side by side and then the runs, and the columns' part of the loss.  The block
// that finishes last adds the parts in their order.  Parts and ticket are
// read-modify-write atomics, which are carried out where all XCDs see them, and
// a block waits for its part's before it takes its ticket: no other memory has
// to be ordered between blocks.  (With fences, each of which writes back an L2,
// the ticket took 18 us for 256 blocks.)
__global__ __launch_bounds__(kJoinThreads) void k_balance_join(BalanceArgs a, int chunk, int cols) {
  constexpr int kRuns = kJoinThreads / kJoinCols;
  __shared__ float s_sum[kRuns][kJoinCols];
  __shared__ int s_count[kRuns][kJoinCols];
  __shared__ int s_tokens[kRuns];
  __shared__ double s_part[kJoinThreads / kWave];
  __shared__ bool s_last;
  const int tid = threadIdx.x;
  const int run = tid / kJoinCols, c = tid % kJoinCols;
  double part = 0.0;
  for (int item = blockIdx.x; item < a.B * cols; item += gridDim.x) {
    const int b = item / cols;
    const int e = item % cols * kJoinCols + c;
    const int64_t first = offset_of(a, b), end = offset_of(a, b + 1);
    float sum = 0.0f;
    int count = 0, tokens = 0;
    if (end > first) {
      const int64_t s0 = first / chunk + b, s1 = (end - 1) / chunk + b;
#pragma unroll 4
      for (int64_t s = s0 + run; s <= s1; s += kRuns) {
        if (e < a.E) {
          sum += a.part_sum[s * a.E + e];
          count += a.part_count[s * a.E + e];
        }
        tokens += a.part_tokens[s];
      }
    }
    s_sum[run][c] = sum;
    s_count[run][c] = count;
    if (c == 0) s_tokens[run] = tokens;
    __syncthreads();
    if (tid < kJoinCols) {
      sum = 0.0f;
      count = tokens = 0;
#pragma unroll 8
      for (int r = 0; r < kRuns; ++r) {
        sum += s_sum[r][c];
        count += s_count[r][c];
        tokens += s_tokens[r];
      }
      if (e < a.E) {
        const float mean = tokens > 0 ? sum / static_cast<float>(tokens) : 0.0f;
        a.mean[static_cast<int64_t>(b) * a.E + e] = mean;
        a.counts[static_cast<int64_t>(b) * a.E + e] = count;
        if (tokens > 0) part += static_cast<double>(count) * mean / tokens;
      }
      if (e == 0) a.tokens[b] = tokens;
    }
    __syncthreads();
  }
  if (tid < kJoinCols) {
#pragma unroll
    for (int off = 1; off < kJoinCols; off <<= 1) part += __shfl_xor(part, off, kJoinCols);
  }
  uint32_t* const high = reinterpret_cast<uint32_t*>(a.part_sum);
  uint32_t* const low = reinterpret_cast<uint32_t*>(a.part_count);
  if (tid == 0) {
    const uint64_t bits = static_cast<uint64_t>(__double_as_longlong(part));
    const int64_t at = part_at(a, chunk, cols, blockIdx.x);
    const uint32_t h = __hip_atomic_exchange(high + at, static_cast<uint32_t>(bits >> 32), __ATOMIC_RELAXED,
                                             __HIP_MEMORY_SCOPE_AGENT);
    const uint32_t l =
        __hip_atomic_exchange(low + at, static_cast<uint32_t>(bits), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    asm volatile("s_waitcnt vmcnt(0)" : : "v"(h), "v"(l) : "memory");  // both have returned
    s_last = __hip_atomic_fetch_add(a.done, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
  }
  __syncthreads();
  if (!s_last) return;
  part = 0.0;
  for (int i = tid; i < static_cast<int>(gridDim.x); i += kJoinThreads) {
    const int64_t at = part_at(a, chunk, cols, i);
    // (exchanges, since a load might find an older line in this XCD's L2)
    const uint64_t h = __hip_atomic_exchange(high + at, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const uint64_t l = __hip_atomic_exchange(low + at, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    part += __longlong_as_double(static_cast<long long>(h << 32 | l));
  }
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) part += __shfl_xor(part, off, kWave);
  if ((tid & (kWave - 1)) == 0) s_part[tid / kWave] = part;
  __syncthreads();
  if (tid != 0) return;
  for (int w = 1; w < kJoinThreads / kWave; ++w) part += s_part[w];
  a.loss[0] = static_cast<float>(part * a.E / (static_cast<double>(a.K) * a.B) * a.coef);
}

// no token: every output is 0
__global__ __launch_bounds__(kBlock) void k_balance_empty(BalanceArgs a) {
  const int64_t n = static_cast<int64_t>(a.B) * a.E;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * kBlock) {
    a.counts[i] = 0;
    a.mean[i] = 0.0f;
    if (i < a.B) a.tokens[i] = 0;
    if (i == 0) a.loss[0] = 0.0f;
  }
}

template <int LPT, int NE, int V, typename LT>
__global__ __launch_bounds__(kBlock) void k_balance_backward(BalanceArgs a, int chunk) {
  constexpr int kPer = kWave / LPT;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int g = lane & (LPT - 1);
  const LT* logits = static_cast<const LT*>(a.logits);
  const LT* base = static_cast<const LT*>(a.base);
  LT* out = static_cast<LT*>(a.glogits);
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * chunk;
  const int64_t t1 = t0 + chunk < a.T ? t0 + chunk : a.T;
  const float scale = a.gloss[0] * a.scale;
  int b = sequence_at(a, t0);
  for (int64_t lo = t0; lo < t1;) {
    // the run of tokens from lo that are of one sequence, or of none
    while (b < a.B && offset_of(a, b + 1) <= lo) ++b;
    const int64_t first = b < a.B ? offset_of(a, b) : t1;
    const bool inside = first <= lo;
    const int64_t end = inside ? offset_of(a, b + 1) : first;
    const int64_t hi = end < t1 ? end : t1;
    float f[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) f[i] = 0.0f;
    if (inside) {
      const float n = static_cast<float>(max(a.tokens[b], 1));
      const float per = scale / n / n;
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        const int e = element<LPT, NE, V>(g, i);
        if (e < a.E) f[i] = static_cast<float>(a.counts[static_cast<int64_t>(b) * a.E + e]) * per;
      }
    }
    // rows are loaded while the ones before are worked on
    float next[NE], next_base[NE];
    auto fetch = [&](int64_t t) __attribute__((always_inline)) {
      if (t >= hi) return;
      load_row<LPT, NE, V>(logits + t * a.E, g, a.E, kNegInf, next);
      if (base) load_row<LPT, NE, V>(base + t * a.E, g, a.E, 0.0f, next_base);
    };
    int64_t t = lo + wave * kPer + lane / LPT;
    fetch(t);
    for (; t < hi; t += kWavesPerBlock * kPer) {
      float d[NE], more[NE];
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        d[i] = next[i];
        more[i] = base ? next_base[i] : 0.0f;
      }
      const bool on = inside && (!a.mask || a.mask[t]);
      fetch(t + kWavesPerBlock * kPer);
      if (on) {
        float rest[NE];
        shares<LPT>(d, a.sigmoid, rest);
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < NE; ++i) dot += f[i] * d[i];
        dot = over_token<LPT>(dot, Add());
#pragma unroll
        for (int i = 0; i < NE; ++i) d[i] = d[i] * (f[i] - dot) * rest[i];
      } else {
#pragma unroll
        for (int i = 0; i < NE; ++i) d[i] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < NE; ++i) d[i] += more[i];
      store_row<LPT, NE, V>(out + t * a.E, g, a.E, d);
    }
    lo = hi;
  }
}

// Calls f(k) with the kernel instance for E experts and these pointers: 16
// lanes a token with 4 or 16 elements each, 64 lanes above 256 experts; rows
// as vectors of four where every row starts on one.
#define EP_BALANCE_PICK(KERNEL, LAUNCH)                                        \
  if (a.bf16) {                                                               \
    if (vec) {                                                                \
      if (a.E <= 64) LAUNCH((KERNEL<16, 4, 4, uint16_t>));                    \
      else if (a.E <= 256) LAUNCH((KERNEL<16, 16, 4, uint16_t>));             \
      else LAUNCH((KERNEL<64, 16, 4, uint16_t>));                             \
    } else {                                                                  \
      if (a.E <= 64) LAUNCH((KERNEL<16, 4, 1, uint16_t>));                    \
      else if (a.E <= 256) LAUNCH((KERNEL<16, 16, 1, uint16_t>));             \
      else LAUNCH((KERNEL<64, 16, 1, uint16_t>));                             \
    }                                                                         \
  } else {                                                                    \
    if (vec) {                                                                \
      if (a.E <= 64) LAUNCH((KERNEL<16, 4, 4, float>));                       \
      else if (a.E <= 256) LAUNCH((KERNEL<16, 16, 4, float>));                \
      else LAUNCH((KERNEL<64, 16, 4, float>));                                \
    } else {                                                                  \
      if (a.E <= 64) LAUNCH((KERNEL<16, 4, 1, float>));                       \
      else if (a.E <= 256) LAUNCH((KERNEL<16, 16, 1, float>));                \
      else LAUNCH((KERNEL<64, 16, 1, float>));                                \
    }                                                                         \
  }

bool on_vector(const void* p, bool bf16) {
  return (reinterpret_cast<uintptr_t>(p) & (bf16 ? 7 : 15)) == 0;
}

// tokens of a block: enough blocks for the chip, and few enough slots
int chunk_of(int64_t T) {
  int c = 16;
  while (T / c > 1024) c *= 2;
  return c;
}

}  // namespace

BalanceGeom balance_geom(int64_t T, int E, int B) {
  BalanceGeom g;
  g.chunk = chunk_of(T);
  g.chunks = (T + g.chunk - 1) / g.chunk;
  g.slots = g.chunks + B;
  g.cols = (E + kJoinCols - 1) / kJoinCols;
  auto up = [](size_t n) { return (n + 15) / 16 * 16; };
  g.sum_bytes = up(static_cast<size_t>(g.slots) * E * 4);
  g.count_bytes = up(static_cast<size_t>(g.slots) * E * 4);
  g.token_bytes = up(static_cast<size_t>(g.slots) * 4);
  const int64_t items = static_cast<int64_t>(B) * g.cols;
  g.joins = static_cast<int>(items < kMaxJoins ? items : kMaxJoins);
  return g;
}

hipError_t launch_balance(const BalanceArgs& a, const BalanceGeom& g, hipStream_t s) {
  if (a.T == 0) {
    const int64_t blocks = (static_cast<int64_t>(a.B) * a.E + kBlock - 1) / kBlock;
    k_balance_empty<<<static_cast<unsigned>(blocks < 1024 ? blocks : 1024), kBlock, 0, s>>>(a);
    return hipGetLastError();
  }
  const bool vec = a.E % 4 == 0 && on_vector(a.logits, a.bf16);
#define EP_LAUNCH(K) K<<<static_cast<unsigned>(g.chunks), kBlock, 0, s>>>(a, g.chunk)
  EP_BALANCE_PICK(k_balance, EP_LAUNCH)
#undef EP_LAUNCH
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  k_balance_join<<<static_cast<unsigned>(g.joins), kJoinThreads, 0, s>>>(a, g.chunk, g.cols);
  return hipGetLastError();
}

hipError_t launch_balance_backward(const BalanceArgs& a, hipStream_t s) {
  const bool vec = a.E % 4 == 0 && on_vector(a.logits, a.bf16) && on_vector(a.glogits, a.bf16) &&
                   on_vector(a.base, a.bf16);
  const int chunk = chunk_of(a.T);
#define EP_LAUNCH(K) K<<<static_cast<unsigned>((a.T + chunk - 1) / chunk), kBlock, 0, s>>>(a, chunk)
  EP_BALANCE_PICK(k_balance_backward, EP_LAUNCH)
#undef EP_LAUNCH
  return hipGetLastError();
}

}  // namespace ep
