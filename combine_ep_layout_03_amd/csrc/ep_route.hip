// Router: each token's K experts of largest selection value, and its weights.
//
// LPT lanes work on one token; lane g holds experts j * 4 * LPT + 4 g + c (c <
// 4), NV of them in registers.  With 16 lanes a wave takes four tokens and
// each step of a reduction runs for all four; with 64 a token has the
// shortest chain of steps (see route_e for the choice).
//
// A key is one 32-bit integer: the value in an order-preserving form, its low
// bits replaced by the complement of the expert's place among the lane's (of
// equal keys in two lanes the lower lane's goes first).  Each lane sorts its
// keys once; a round then is a maximum over the lanes' heads and a shift in
// the lane that held it.  For bf16 logits without a bias the low 16 bits are
// free for the whole index and nothing is lost.  Otherwise the rounds order the
// experts only up to a tolerance (the bits given up, and the error of scores
// computed with the hardware's exponential and reciprocal), so neighbours closer
// than it are put in order by their exact values: the fp32 logits, or score +
// bias in binary64.  That takes one binary64 score per candidate, for the
// candidates down to the first clear gap below the Kth.  Groups are treated
// alike.  Where even that leaves doubt (too many candidates, a group whose best
// two are in doubt) the token is done again, by fp32 logits in rounds on the
// logits themselves, else in binary64 throughout.
//
// A wave does one task and ends: in a loop over tasks the compiler keeps what
// does not change between them, some 400 instructions' results, and spills.
//
// Measured, 256 experts, top-8.  65,536 tokens, bf16 softmax: 20 us, 2 TB/s;
// the vector units issue for 16 of them (600 instructions a wave).  Sigmoid +
// bias, 4 of 8 groups: 8192 tokens 13.0 us, two waves per SIMD, of which the
// vector units issue for 5: the chain of dependent steps bounds it; 16 tokens 6.8
// us, that chain once.  fp32 softmax: 65,536 tokens 28 us, 33 where the logits
// hold bf16 values with their many ties, 66 where a token's are all equal (380
// before those had rounds of their own); the binary64 path, all scores equal:
// 740.
#include <float.h>

#include "ep_layer.h"

namespace ep {

namespace {

constexpr float kNegInf = -__builtin_inff();

__device__ __forceinline__ void lds_sync() {
  // LDS is private to the wave here and its accesses complete in order: only
  // the compiler has to keep them in order
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

template <typename LT>
__device__ __forceinline__ float raw_logit(const LT* p);
template <>
__device__ __forceinline__ float raw_logit<float>(const float* p) {
  return *p;
}
template <>
__device__ __forceinline__ float raw_logit<uint16_t>(const uint16_t* p) {
  return bf16_to_f32(*p);
}

// NaN -> -inf (cannot be chosen), +inf -> the largest finite value, -0 -> +0
__device__ __forceinline__ float clean_logit(float l) {
  return l != l ? kNegInf : fminf(l, FLT_MAX) + 0.0f;
}

// A chosen expert's score up to a factor common to its token's chosen ones,
// whose largest logit is top: exp(l - top), or sigmoid(l) / exp(min(top, 0)),
// neither of which underflows for the largest.
__device__ __forceinline__ float relative_score(float l, float top, bool sigmoid) {
  if (!sigmoid) return expf(l - top);
  return l < 0.0f ? expf(l - fminf(top, 0.0f)) / (1.0f + expf(l)) : 1.0f / (1.0f + expf(-l));
}

__device__ __forceinline__ float sigmoid32(float l) {
  const float e = expf(-fabsf(l));  // at most 1, so nothing overflows and small scores stay
  return (l < 0.0f ? e : 1.0f) / (1.0f + e);
}

// order-preserving map to unsigned integers
__device__ __forceinline__ uint32_t ordered(float f) {
  const uint32_t b = __float_as_uint(f);
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}

__device__ __forceinline__ int64_t wave_task() {
  return static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x;
}

// ------------------------------------------------- reductions over LPT lanes
// v from the lane N places round the row of 16
template <int N>
__device__ __forceinline__ uint32_t row_turn(uint32_t v) {
  return static_cast<uint32_t>(
      __builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x120 | N, 0xf, 0xf, true));
}
template <int N>
__device__ __forceinline__ uint32_t turn(uint32_t v) {
  if constexpr (N >= 16) return __shfl_xor(v, N, kWave);
  else return row_turn<N>(v);
}
template <int N>
__device__ __forceinline__ float turn(float v) {
  return __uint_as_float(turn<N>(__float_as_uint(v)));
}
template <int N>
__device__ __forceinline__ uint64_t turn(uint64_t v) {
  return (static_cast<uint64_t>(turn<N>(static_cast<uint32_t>(v >> 32))) << 32) |
         turn<N>(static_cast<uint32_t>(v));
}
template <int N>
__device__ __forceinline__ double turn(double v) {
  return __longlong_as_double(static_cast<long long>(turn<N>(static_cast<uint64_t>(__double_as_longlong(v)))));
}

struct Max {
  template <typename T>
  __device__ __forceinline__ T operator()(T a, T b) const {
    return a > b ? a : b;
  }
};
struct Min {
  template <typename T>
  __device__ __forceinline__ T operator()(T a, T b) const {
    return a < b ? a : b;
  }
};
struct Or {
  __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const { return a | b; }
};
struct Sum {
  template <typename T>
  __device__ __forceinline__ T operator()(T a, T b) const {
    return a + b;
  }
};
// f of v and the v of the other row of 16 (or half of 32): the swap leaves
// the even rows' values in one result and the odd rows' in the other
template <int N, typename F>
__device__ __forceinline__ uint32_t across(uint32_t v, F f) {
  if constexpr (N == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return f(static_cast<uint32_t>(r[0]), static_cast<uint32_t>(r[1]));
  } else {
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return f(static_cast<uint32_t>(r[0]), static_cast<uint32_t>(r[1]));
  }
}
template <int N, typename F>
__device__ __forceinline__ float across(float v, F f) {
  return __uint_as_float(across<N>(__float_as_uint(v), [&](uint32_t a, uint32_t b) {
    return __float_as_uint(f(__uint_as_float(a), __uint_as_float(b)));
  }));
}
template <int N, typename F>
__device__ __forceinline__ double across(double v, F f) {
  return f(v, turn<N>(v));
}
__device__ __forceinline__ uint32_t uniform(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(v)));
}
__device__ __forceinline__ float uniform(float v) { return __uint_as_float(uniform(__float_as_uint(v))); }
__device__ __forceinline__ double uniform(double v) { return v; }
// the reduction of v over the token's LPT lanes, in every one of them (in a
// scalar register where they are the whole wave, so branches on it are scalar)
template <int LPT, typename T, typename F>
__device__ __forceinline__ T over_token(T v, F f) {
  v = f(v, turn<8>(v));
  v = f(v, turn<4>(v));
  v = f(v, turn<2>(v));
  v = f(v, turn<1>(v));
  if constexpr (LPT >= 32) v = across<16>(v, f);
  if constexpr (LPT >= 64) v = uniform(across<32>(v, f));
  return v;
}
// v of the token's lane g
template <int LPT, typename T>
__device__ __forceinline__ T from_lane(T v, int g) {
  return __shfl(v, g, LPT);
}

// e / gsize for e < 1024: (e * m) >> 20 with m = ceil(2^20 / gsize) is exact,
// as e * (m * gsize - 2^20) <= 1023 * 1023 < 2^20
__device__ __forceinline__ int group_of(int e, uint32_t magic) {
  return static_cast<int>((static_cast<uint32_t>(e) * magic) >> 20);
}

// The open groups of one token as a bit mask, from the groups' values gv[G] in
// LDS: fewer than tg are better (larger, or equal with a lower index).  last and
// next: the smallest open and the largest closed value.
template <int LPT, typename F>
__device__ __forceinline__ uint64_t open_groups(const F* gv, int G, int tg, int g, F& last, F& next) {
  uint32_t lo = 0, hi = 0;
  last = __builtin_inf();
  next = -__builtin_inf();
  for (int q = g; q < G; q += LPT) {
    const F v = gv[q];
    int better = 0;
#pragma unroll 4
    for (int o = 0; o < G; ++o) {
      const F u = gv[o];
      better += (u > v || (u == v && o < q)) ? 1 : 0;
    }
    if (better < tg) {
      if (q < 32) lo |= 1u << q;
      else hi |= 1u << (q - 32);
      last = v < last ? v : last;
    } else {
      next = v > next ? v : next;
    }
  }
  lo = over_token<LPT>(lo, Or());
  if (G > 32) hi = over_token<LPT>(hi, Or());
  last = over_token<LPT>(last, Min());
  next = over_token<LPT>(next, Max());
  return (static_cast<uint64_t>(hi) << 32) | lo;
}

// ----------------------------------------------------------------- binary64
__device__ __forceinline__ double sigmoid64(double l) { return 1.0 / (1.0 + exp(-l)); }

// Scores of one token's cleaned logits in binary64.
struct Score64 {
  bool sigmoid;
  double lmax, sum;
  __device__ __forceinline__ double operator()(float l) const {
    return sigmoid ? sigmoid64(l) : exp(static_cast<double>(l) - lmax) / sum;
  }
};
template <int LPT, typename LT>
__device__ __forceinline__ Score64 score64(const RouteArgs& a, const LT* row, int g, float lmax) {
  Score64 s = {a.sigmoid, static_cast<double>(lmax), 1.0};
  if (!a.sigmoid) {
    double sum = 0.0;
    for (int e = g; e < a.E; e += LPT) {
      const float l = clean_logit(raw_logit(row + e));
      if (l > kNegInf) sum += exp(static_cast<double>(l) - s.lmax);
    }
    s.sum = over_token<LPT>(sum, Sum());
  }
  return s;
}

// The experts a token has chosen: s_idx[K] in LDS, -1 where there is none.
// The whole of it in binary64: val [E], gv [kMaxRouteGroups] in LDS.
template <int LPT, typename LT>
__device__ __forceinline__ void choose64(const RouteArgs& a, const LT* row, int g, float lmax,
                                         double* val, double* gv, int* s_idx) {
  const double none = -__builtin_inf();
  const int E = a.E;
  const Score64 score = score64<LPT>(a, row, g, lmax);
  uint64_t open = ~0ull;
  const uint32_t magic = a.G ? ((1u << 20) + a.gsize - 1) / a.gsize : 0u;
  if (a.G) {
    const bool by_logit = !a.bias && a.gtop == 1;
    for (int q = g; q < a.G; q += LPT) {
      double m1 = none, m2 = none;
      for (int e = q * a.gsize; e < (q + 1) * a.gsize; ++e) {
        const float l = clean_logit(raw_logit(row + e));
        double v = by_logit ? static_cast<double>(l) : score(l) + (a.bias ? static_cast<double>(a.bias[e]) : 0.0);
        if (l == kNegInf || v != v) v = none;
        m2 = v > m1 ? m1 : v > m2 ? v : m2;
        m1 = v > m1 ? v : m1;
      }
      gv[q] = (a.gtop == 2 && m2 > none) ? m1 + m2 : m1;
    }
    lds_sync();
    double last, next;
    open = open_groups<LPT>(gv, a.G, a.tg, g, last, next);
    lds_sync();
  }
  for (int e = g; e < E; e += LPT) {
    const float l = clean_logit(raw_logit(row + e));
    double v = a.bias ? score(l) + static_cast<double>(a.bias[e]) : static_cast<double>(l);
    if (l == kNegInf || v != v || (a.G && !((open >> group_of(e, magic)) & 1))) v = none;
    val[e] = v;
  }
  lds_sync();
  for (int k = 0; k < a.K; ++k) {
    double best = none;
    int at = INT32_MAX;
    for (int e = g; e < E; e += LPT) {
      const double v = val[e];
      if (v > best) {
        best = v;
        at = e;
      }
    }
    const double top = over_token<LPT>(best, Max());
    const uint32_t mine = (best == top && best > none) ? static_cast<uint32_t>(at) : UINT32_MAX;
    const uint32_t win = over_token<LPT>(mine, Min());
    const int e = win == UINT32_MAX ? -1 : static_cast<int>(win);
    if (e >= 0 && e % LPT == g) val[e] = none;
    if (g == 0) s_idx[k] = e;
    lds_sync();
  }
}

// ------------------------------------------------------------------ forward
constexpr float kLog2e = 1.44269504088896340736f;

// Batcher's odd-even merge sort, descending.
template <int N>
__device__ __forceinline__ void sort_descending(uint32_t (&k)[N]) {
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int q = p; q >= 1; q /= 2)
#pragma unroll
      for (int j = q % p; j <= N - 1 - q; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i)
          if (i + j + q < N && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
            const uint32_t x = k[i + j], y = k[i + j + q];
            k[i + j] = x > y ? x : y;
            k[i + j + q] = x > y ? y : x;
          }
}

// The N largest of k[0..M), descending.
template <int M, int N>
__device__ __forceinline__ void keep_largest(uint32_t (&k)[M], uint32_t (&out)[N]) {
  if constexpr (M == N) {
#pragma unroll
    for (int i = 0; i < N; ++i) out[i] = k[i];
    sort_descending(out);
  } else {
    static_assert(M == 2 * N, "two halves");
    uint32_t x[N], y[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      x[i] = k[i];
      y[i] = k[N + i];
    }
    sort_descending(x);
    sort_descending(y);
    // the larger of x[i] and y[N - 1 - i] are the N largest, a bitonic run
#pragma unroll
    for (int i = 0; i < N; ++i) out[i] = x[i] > y[N - 1 - i] ? x[i] : y[N - 1 - i];
#pragma unroll
    for (int d = N / 2; d >= 1; d /= 2)
#pragma unroll
      for (int i = 0; i < N; ++i)
        if ((i & d) == 0) {
          const uint32_t u = out[i], v = out[i + d];
          out[i] = u > v ? u : v;
          out[i + d] = u > v ? v : u;
        }
  }
}

__host__ __device__ constexpr int log2i(int n) { return n <= 1 ? 0 : 1 + log2i(n / 2); }

// What experts are compared by: bf16 logits (exact in a key), fp32 logits, or
// score + bias.
enum { kByBf16, kByFp32, kByScore };

// KEEP: keys a lane keeps sorted, NV or (K <= 8) half of 16.
template <int LPT, int NV, int KEEP, typename LT, int BY>
__global__ __launch_bounds__(kWave) __attribute__((amdgpu_waves_per_eu(4))) void k_route(
    RouteArgs a) {
  constexpr int kTok = kWave / LPT;             // tokens per wave
  constexpr int kCap = LPT * NV;                // experts a token's lanes hold
  constexpr int kCand = LPT >= 32 ? 64 : 48;    // candidates kept, more than K
  constexpr int kOut = LPT >= 32 ? 1 : 2;       // selections per lane
  constexpr int kLow = BY == kByBf16 ? 16 : log2i(NV);  // index bits of a key
  constexpr uint32_t kLowMask = (1u << kLow) - 1;
  constexpr int kPitch = kCap + 32 > 2 * kCand ? kCap + 32 : 2 * kCand;
  static_assert(kTok * kPitch >= 2 * kCap || kTok == 1, "choose64's values");
  __shared__ __align__(8) float s_val[kTok * kPitch > 2 * kCap ? kTok * kPitch : 2 * kCap];
  __shared__ double s_gv[kTok * kMaxRouteGroups];
  __shared__ uint32_t s_key[kTok][kCand];
  __shared__ int s_idx[kTok][kCand];
  const int lane = threadIdx.x;
  const int g = lane % LPT;
  const int tok = lane / LPT;
  const int E = a.E, K = a.K;
  const LT* all = static_cast<const LT*>(a.logits);
  float* valf = s_val + tok * kPitch;                     // one token's values
  double* cand = reinterpret_cast<double*>(valf);          // or its candidates'
  double* gv = s_gv + tok * kMaxRouteGroups;
  float* gvf = reinterpret_cast<float*>(gv);
  uint32_t* keys = s_key[tok];
  int* idxs = s_idx[tok];
  const uint32_t magic = a.G ? ((1u << 20) + a.gsize - 1) / a.gsize : 0u;
  const bool vec = E % 4 == 0 && (reinterpret_cast<uintptr_t>(all) & (4 * sizeof(LT) - 1)) == 0 &&
                   (reinterpret_cast<uintptr_t>(a.bias) & 15) == 0;
  const bool group_scores = a.G && (BY == kByScore || a.gtop == 2);
  const bool need_scores = BY == kByScore || group_scores;
  const bool need_sum = !a.sigmoid && (need_scores || !a.renorm);

  const int64_t t = wave_task() * kTok + tok;
  if (t >= a.T) return;  // whole groups of LPT lanes: the reductions stay within a token
  const LT* row = all + t * E;
  const bool masked = a.mask && a.mask[t] == 0;
  float lmax = kNegInf, lsum = 1.0f;
  int chosen[kOut];
#pragma unroll
  for (int i = 0; i < kOut; ++i) chosen[i] = -1;
  if (!masked) {
    float l[NV], bias[BY == kByScore ? NV : 1];
#pragma unroll
    for (int j = 0; j < NV / 4; ++j) {
      const int e0 = j * 4 * LPT + 4 * g;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        l[4 * j + c] = kNegInf;
        if constexpr (BY == kByScore) bias[4 * j + c] = 0.0f;
      }
      if (vec) {
        if (e0 < E) {
          if constexpr (BY == kByScore) {
            const f32x4_t v = *reinterpret_cast<const f32x4_t*>(a.bias + e0);
#pragma unroll
            for (int c = 0; c < 4; ++c) bias[4 * j + c] = v[c];
          }
          if constexpr (sizeof(LT) == 4) {
            const u32x4 v = *reinterpret_cast<const u32x4*>(row + e0);
#pragma unroll
            for (int c = 0; c < 4; ++c) l[4 * j + c] = __uint_as_float(v[c]);
          } else {
            const u32x2 v = *reinterpret_cast<const u32x2*>(row + e0);
            l[4 * j] = bf16_lo(v[0]);
            l[4 * j + 1] = bf16_hi(v[0]);
            l[4 * j + 2] = bf16_lo(v[1]);
            l[4 * j + 3] = bf16_hi(v[1]);
          }
        }
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (e0 + c < E) {
            l[4 * j + c] = raw_logit(row + e0 + c);
            if constexpr (BY == kByScore) bias[4 * j + c] = a.bias[e0 + c];
          }
      }
    }
    auto expert = [&](int i) { return (i / 4) * 4 * LPT + 4 * g + i % 4; };
    uint32_t all_keys[NV];
    auto make_key = [&](int i, float v) {
      uint32_t key = (ordered(v) & ~kLowMask) | (kLowMask - static_cast<uint32_t>(BY == kByBf16 ? expert(i) : i));
      asm("" : "+v"(key));  // a select, not a branch around the key's making
      return v > kNegInf ? key : 0u;
    };
    if constexpr (BY == kByBf16) {
      // NaN is left out by the comparison; +inf stays above the largest bf16
#pragma unroll
      for (int i = 0; i < NV; ++i) all_keys[i] = make_key(i, l[i] + 0.0f);
    }
    if (BY != kByBf16 || a.G || need_sum) {
#pragma unroll
      for (int i = 0; i < NV; ++i) l[i] = clean_logit(l[i]);
    }
    if constexpr (BY == kByFp32) {
#pragma unroll
      for (int i = 0; i < NV; ++i) all_keys[i] = make_key(i, l[i]);
    }

    if (need_sum) {
      float m = l[0];
#pragma unroll
      for (int i = 1; i < NV; ++i) m = fmaxf(m, l[i]);
      lmax = over_token<LPT>(m, Max());
    }
    // Scores for the comparisons, with the hardware's exponential and
    // reciprocal (1 ulp each).  An exponent x is off by at most 2.5 |x| 2^-24,
    // |x| <= 88 where the result counts, so a score's relative error is below
    // (2.5 * 88 + 30) 2^-24 < 2^-16; as exp(x) |x| <= 0.37 for x < 0, its
    // absolute error is below 7 * 2^-24 for the sigmoid, and for the softmax,
    // whose sum is off by the average of its terms, below 61 * 2^-24.
    float c[NV];
    float bmax = 0.0f;
    if (need_sum) {
      float s = 0.0f;
      if (lmax > kNegInf) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          // the weights that are not renormalised need the sum to fp32's accuracy
          c[i] = a.renorm ? __builtin_amdgcn_exp2f((l[i] - lmax) * kLog2e) : expf(l[i] - lmax);
          s += c[i];
        }
      }
      lsum = over_token<LPT>(s, Sum());
    }
    if (need_scores) {
      const float inv = __builtin_amdgcn_rcpf(lsum);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float v = a.sigmoid ? __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-l[i] * kLog2e)) : c[i] * inv;
        if constexpr (BY == kByScore) {
          if (fabsf(bias[i]) < __builtin_inff()) bmax = fmaxf(bmax, fabsf(bias[i]));
          v += bias[i];
        }
        c[i] = (l[i] == kNegInf || v != v) ? kNegInf : v;
      }
      if constexpr (BY == kByScore) bmax = over_token<LPT>(bmax, Max());
    }
    // bounds on the error of a value, score + bias, and of half a sum of two (half
    // of what two errors and the sum's rounding add up to)
    const float cap = a.sigmoid ? 0x1p-21f : 0x1p-18f;
    auto err = [&](float v) {
      return fminf(cap, 0x1p-16f * (fabsf(v) + bmax)) + 0x1p-22f * fabsf(v) + 1e-37f;
    };
    auto err2 = [&](float v) {
      return fminf(cap, 0x1p-16f * (fabsf(v) + bmax)) + (0x1p-22f * fabsf(v) + 0x1p-21f * bmax) + 1e-37f;
    };

    uint64_t open = ~0ull;
    bool doubt = false;
    if (a.G) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (expert(i) < E) valf[expert(i)] = group_scores ? c[i] : l[i];
      lds_sync();
      // P lanes read one group, each every Pth value from a start that
      // keeps the groups on different banks
      const int P = a.G * 4 <= LPT && a.gsize % 4 == 0 ? 4 : a.G * 2 <= LPT && a.gsize % 2 == 0 ? 2 : 1;
      const int sub = g % P;
      // a group's value; of two, half the sum: two finite biases' may overflow
      auto value = [&](float m1, float m2) {
        return a.gtop == 1 ? m1 : m2 > kNegInf ? 0.5f * m1 + 0.5f * m2 : 0.5f * m1;
      };
      for (int q = g / P; q < a.G; q += LPT / P) {
        float m1 = kNegInf, m2 = kNegInf;
        int at = (q * P) % a.gsize;
        at = at - at % P + sub;
#pragma unroll 4
        for (int n = 0; n < a.gsize; n += P) {
          const float v = valf[q * a.gsize + at];
          at += P;
          if (at >= a.gsize) at -= a.gsize;
          m2 = __builtin_amdgcn_fmed3f(m1, m2, v);  // m1 >= m2
          m1 = fmaxf(m1, v);
        }
        for (int off = 1; off < P; off <<= 1) {
          const float o1 = __shfl_xor(m1, off, kWave), o2 = __shfl_xor(m2, off, kWave);
          m2 = fmaxf(fminf(m1, o1), fmaxf(m2, o2));
          m1 = fmaxf(m1, o1);
        }
        if (sub == 0) gvf[q] = value(m1, m2);
      }
      lds_sync();
      float last, next;
      open = open_groups<LPT>(gvf, a.G, a.tg, g, last, next);
      lds_sync();
      if (group_scores && next > kNegInf && last - next <= err2(last) + err2(next)) {
        // the groups' values in binary64: each group's best one or two,
        // found by their fp32 values, if those leave no doubt
        const Score64 score = score64<LPT>(a, row, g, lmax);
        auto exact = [&](int e) {
          return score(clean_logit(raw_logit(row + e))) + (BY == kByScore ? static_cast<double>(a.bias[e]) : 0.0);
        };
        for (int q = g; q < a.G; q += LPT) {
          float m1 = kNegInf, m2 = kNegInf, m3 = kNegInf;
          int e1 = -1, e2 = -1;
          for (int n = 0; n < a.gsize; ++n) {
            const float v = valf[q * a.gsize + n];
            if (v > m1) {
              m3 = m2;
              m2 = m1;
              e2 = e1;
              m1 = v;
              e1 = q * a.gsize + n;
            } else if (v > m2) {
              m3 = m2;
              m2 = v;
              e2 = q * a.gsize + n;
            } else if (v > m3) {
              m3 = v;
            }
          }
          const float in = a.gtop == 2 ? m2 : m1, out = a.gtop == 2 ? m3 : m2;
          if (out > kNegInf && in - out <= err(in) + err(out)) doubt = true;
          double v = -__builtin_inf();
          if (e1 >= 0) v = exact(e1);
          if (a.gtop == 2 && e2 >= 0) v += exact(e2);
          gv[q] = v;
        }
        lds_sync();
        double last64, next64;
        open = open_groups<LPT>(gv, a.G, a.tg, g, last64, next64);
        doubt = over_token<LPT>(doubt ? 1u : 0u, Or()) != 0u;
        lds_sync();
      }
    }

    if constexpr (BY == kByScore) {
#pragma unroll
      for (int i = 0; i < NV; ++i) all_keys[i] = make_key(i, c[i]);
    }
    if (a.G) {
      if (a.gsize % 4 == 0) {  // four neighbours share a group
#pragma unroll
        for (int j = 0; j < NV / 4; ++j) {
          const bool shut = !((open >> group_of(expert(4 * j), magic)) & 1);
#pragma unroll
          for (int c = 0; c < 4; ++c) all_keys[4 * j + c] = shut ? 0u : all_keys[4 * j + c];
        }
      } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
          all_keys[i] = (open >> group_of(expert(i), magic)) & 1 ? all_keys[i] : 0u;
      }
    }
    const bool group_doubt = doubt;
    uint32_t key[KEEP];
    keep_largest(all_keys, key);
    auto close = [&](uint32_t x, uint32_t y) {
      const float u = unordered(x & ~kLowMask), v = unordered(y & ~kLowMask);
      float tol = 0x1p-22f * (1u << kLow) * fabsf(v) + 1e-37f;
      if (BY == kByScore) tol += err(u) + err(v);
      return !(u - v > tol);  // two of +inf, whose difference is NaN, are equal
    };
    const uint64_t before = lanemask_lt() & ~((1ull << (tok * LPT)) - 1);  // the token's lanes below this one
    auto drop_head = [&](bool mine) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < KEEP - 1; ++i) key[i] = mine ? key[i + 1] : key[i];
      key[KEEP - 1] = mine ? 0u : key[KEEP - 1];
    };
    int count = 0;  // candidates, in the same order in all of the token's lanes
    if constexpr (BY == kByBf16) {
      for (int k = 0; k < K; ++k) {
        const uint32_t m = over_token<LPT>(key[0], Max());
        drop_head(key[0] == m);
        const int e = m != 0u ? static_cast<int>(kLowMask - (m & kLowMask)) : -1;
#pragma unroll
        for (int i = 0; i < kOut; ++i) chosen[i] = k == g + i * LPT ? e : chosen[i];
      }
    } else {
      // candidates worth keeping: exact rounds by logits cost little more
      const int limit = BY == kByFp32 ? K + 4 : kCand;
      int taken = 0;  // of this lane's keys
      uint32_t prev = 0;
      for (int k = 0;; ++k) {
        const uint32_t m = over_token<LPT>(key[0], Max());
        if (k >= K) {  // beyond the Kth, down to the first clear gap
          if (prev == 0u || m == 0u || !close(prev, m)) break;
          if (count == limit) {
            doubt = true;
            break;
          }
        }
        bool mine = key[0] == m && m != 0u;
        mine = mine && (ballot(mine) & before) == 0;  // the lowest lane of equal keys
        if (mine) {
          keys[count] = m;
          idxs[count] = expert(static_cast<int>(kLowMask - (m & kLowMask)));
        }
        drop_head(mine);
        count += m != 0u ? 1 : 0;
        taken += mine ? 1 : 0;
        prev = m;
      }
      // a lane whose kept keys are used up may have had another
      if (KEEP < NV) doubt |= over_token<LPT>(taken == KEEP ? 1u : 0u, Or()) != 0u;
    }
    lds_sync();
    bool near = false;  // the candidates were put in order by their exact values: in keys
    if (BY != kByBf16 && !doubt) {
      for (int k = g; k < count - 1; k += LPT) near |= close(keys[k], keys[k + 1]);
      near = over_token<LPT>(near ? 1u : 0u, Or()) != 0u;
      if (near) {
        // the candidates' exact values, and each one's place among them
        Score64 score = {};
        if (BY == kByScore) score = score64<LPT>(a, row, g, lmax);
        for (int k = g; k < count; k += LPT) {
          const int e = idxs[k];
          const float x = clean_logit(raw_logit(row + e));
          cand[k] = BY == kByScore ? score(x) + static_cast<double>(a.bias[e]) : static_cast<double>(x);
        }
        lds_sync();
        for (int k = g; k < count; k += LPT) {
          const double v = cand[k];
          const int e = idxs[k];
          int place = 0;
#pragma unroll 4
          for (int j = 0; j < count; ++j) place += (cand[j] > v || (cand[j] == v && idxs[j] < e)) ? 1 : 0;
          keys[place] = static_cast<uint32_t>(e);
        }
        lds_sync();
      }
    }
    if (BY == kByFp32 && doubt && !group_doubt) {
      // a round after the other by the logits themselves (a row of equal ones)
      float v[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        v[i] = kNegInf;
        if (expert(i) < E && ((open >> (a.G ? group_of(expert(i), magic) : 0)) & 1))
          v[i] = clean_logit(raw_logit(row + expert(i)));
      }
      for (int k = 0; k < K; ++k) {
        float best = kNegInf;
        uint32_t at = UINT32_MAX;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          at = v[i] > best ? static_cast<uint32_t>(expert(i)) : at;
          best = fmaxf(best, v[i]);
        }
        const float most = over_token<LPT>(best, Max());
        const uint32_t win = over_token<LPT>(best == most ? at : UINT32_MAX, Min());
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] = static_cast<uint32_t>(expert(i)) == win ? kNegInf : v[i];
#pragma unroll
        for (int i = 0; i < kOut; ++i) chosen[i] = k == g + i * LPT ? static_cast<int>(win) : chosen[i];
      }
    } else if (doubt) {
      // one token after the other: its values take the whole array
      for (int d = 0; d < kTok; ++d)
        if (d == tok) choose64<LPT>(a, row, g, lmax, reinterpret_cast<double*>(s_val), gv, idxs);
#pragma unroll
      for (int i = 0; i < kOut; ++i)
        if (g + i * LPT < K) chosen[i] = idxs[g + i * LPT];
    } else if (BY != kByBf16) {
#pragma unroll
      for (int i = 0; i < kOut; ++i) {
        const int k = g + i * LPT;
        if (k < K && k < count) chosen[i] = near ? static_cast<int>(keys[k]) : idxs[k];
      }
    }
    lds_sync();
  }

  // weights of selections g and g + LPT
  float lc[kOut], w[kOut];
  float top = kNegInf;
#pragma unroll
  for (int i = 0; i < kOut; ++i) {
    lc[i] = chosen[i] >= 0 ? clean_logit(raw_logit(row + chosen[i])) : kNegInf;
    top = fmaxf(top, lc[i]);
  }
  if (a.renorm) {
    top = over_token<LPT>(top, Max());
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kOut; ++i) {
      w[i] = chosen[i] >= 0 ? relative_score(lc[i], top, a.sigmoid) : 0.0f;
      sum += w[i];
    }
    sum = over_token<LPT>(sum, Sum());
#pragma unroll
    for (int i = 0; i < kOut; ++i) w[i] = w[i] / sum * a.scale;
  } else {
#pragma unroll
    for (int i = 0; i < kOut; ++i)
      w[i] = (a.sigmoid ? sigmoid32(lc[i]) : expf(lc[i] - lmax) / lsum) * a.scale;
  }
#pragma unroll
  for (int i = 0; i < kOut; ++i) {
    const int k = g + i * LPT;
    if (k < K) {
      a.idx[t * K + k] = chosen[i];
      a.w[t * K + k] = chosen[i] >= 0 ? w[i] : 0.0f;
    }
  }
}

// ----------------------------------------------------------------- backward
// With p the scores, n_k = p_k / sum p of the selected, h_k = scale dw_k (0 where
// an expert is not selected):
//     softmax               dl_e = p_e (h_e - sum_j h_j p_j), every expert
//     softmax, renormalised dl_k = n_k (h_k - sum_j h_j n_j), the selected alone
//     sigmoid               dl_k = p_k (1 - p_k) h_k
//     sigmoid, renormalised dl_k = n_k (1 - p_k) (h_k - sum_j h_j n_j)
// Lane g of a token holds selections g and g + LPT; the gradient's row is put
// together in LDS and written whole.  65,536 tokens x 256, top-8, sigmoid
// renormalised, fp32: 19.6 us, 140 MB, much of it still in the memory-side cache;
// the vector units issue for half of that time.  4096 x 64, softmax: 5.2 us.  The
// dense gradient (softmax, not renormalised) passes over a row three times, an
// element a lane: 65,536 x 256 60 us in fp32, 42 in bf16, two to three times its
// bytes.
template <int LPT, typename LT>
__global__ __launch_bounds__(kWave) void k_route_backward(RouteArgs a, int cap) {
  extern __shared__ float s_row[];  // [64 / LPT][cap]
  constexpr int kTok = kWave / LPT;
  constexpr int kSlots = LPT >= 32 ? 1 : 2;
  const int lane = threadIdx.x;
  const int g = lane % LPT;
  const int tok = lane / LPT;
  const int E = a.E, K = a.K;
  float* d_row = s_row + tok * cap;
  const bool vec = E % 4 == 0 &&
                   ((reinterpret_cast<uintptr_t>(a.logits) | reinterpret_cast<uintptr_t>(a.glogits)) &
                    (4 * sizeof(LT) - 1)) == 0;
  const bool dense = !a.sigmoid && !a.renorm;
  const int64_t t = wave_task() * kTok + tok;
  if (t >= a.T) return;
  const LT* row = static_cast<const LT*>(a.logits) + t * E;
  LT* out = static_cast<LT*>(a.glogits) + t * E;

  for (int e = g; e < cap; e += LPT) d_row[e] = 0.0f;
  int idx[kSlots];
  float gw[kSlots], lc[kSlots], d[kSlots];
  float top = kNegInf;
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    const int k = g + i * LPT;
    idx[i] = -1;
    gw[i] = 0.0f;
    if (k < K) {
      const int64_t e = a.idx[t * K + k];
      if (e >= 0 && e < E) {
        idx[i] = static_cast<int>(e);
        gw[i] = a.gw[t * K + k] * a.scale;
      }
    }
    lc[i] = idx[i] >= 0 ? clean_logit(raw_logit(row + idx[i])) : kNegInf;
    top = fmaxf(top, lc[i]);
  }
  if (a.renorm) {
    top = over_token<LPT>(top, Max());
    float w[kSlots];
    float sum = 0.0f, dot = 0.0f;
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      w[i] = 0.0f;
      if (lc[i] > kNegInf) w[i] = relative_score(lc[i], top, a.sigmoid);
      sum += w[i];
    }
    sum = over_token<LPT>(sum, Sum());
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      w[i] = sum > 0.0f ? w[i] / sum : 0.0f;
      if (idx[i] >= 0) dot += w[i] * gw[i];
    }
    dot = over_token<LPT>(dot, Sum());
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      d[i] = w[i] * (gw[i] - dot);
      if (a.sigmoid) d[i] *= sigmoid32(-lc[i]);
    }
  } else if (a.sigmoid) {
#pragma unroll
    for (int i = 0; i < kSlots; ++i) d[i] = gw[i] * sigmoid32(-lc[i]) * sigmoid32(lc[i]);
  } else {
#pragma unroll
    for (int i = 0; i < kSlots; ++i) d[i] = gw[i];
  }
#pragma unroll
  for (int i = 0; i < kSlots; ++i)
    if (idx[i] < 0 || lc[i] == kNegInf) d[i] = 0.0f;
  // an expert named more than once: each of its selections carries the sum
  // of their terms in ascending k, so they write the same value
  float total[kSlots];
#pragma unroll
  for (int i = 0; i < kSlots; ++i) total[i] = 0.0f;
  for (int k = 0; k < K; ++k) {
    const int from = k % LPT;
    const bool second = kSlots > 1 && k >= LPT;
    const int ek = from_lane<LPT>(second ? idx[kSlots - 1] : idx[0], from);
    const float dk = from_lane<LPT>(second ? d[kSlots - 1] : d[0], from);
#pragma unroll
    for (int i = 0; i < kSlots; ++i) total[i] += ek == idx[i] ? dk : 0.0f;
  }
  lds_sync();
#pragma unroll
  for (int i = 0; i < kSlots; ++i)
    if (idx[i] >= 0) d_row[idx[i]] = total[i];
  lds_sync();

  float m = kNegInf, inv = 0.0f, dot = 0.0f;
  if (dense) {
    for (int e = g; e < E; e += LPT) m = fmaxf(m, clean_logit(raw_logit(row + e)));
    m = over_token<LPT>(m, Max());
    float s = 0.0f;
    if (m > kNegInf) {
      for (int e = g; e < E; e += LPT) {
        const float x = expf(clean_logit(raw_logit(row + e)) - m);
        s += x;
        dot += x * d_row[e];
      }
    }
    s = over_token<LPT>(s, Sum());
    dot = over_token<LPT>(dot, Sum());
    inv = s > 0.0f ? 1.0f / s : 0.0f;
    dot *= inv;
  }
  auto value = [&](int e) {
    const float dv = d_row[e];
    if (!dense) return dv;
    const float l = clean_logit(raw_logit(row + e));
    return l > kNegInf ? expf(l - m) * inv * (dv - dot) : 0.0f;
  };
  if (vec) {
    for (int e = 4 * g; e < E; e += 4 * LPT) {
      const float v0 = value(e), v1 = value(e + 1), v2 = value(e + 2), v3 = value(e + 3);
      if constexpr (sizeof(LT) == 4) {
        u32x4 v;
        v[0] = __float_as_uint(v0);
        v[1] = __float_as_uint(v1);
        v[2] = __float_as_uint(v2);
        v[3] = __float_as_uint(v3);
        *reinterpret_cast<u32x4*>(out + e) = v;
      } else {
        u32x2 v;
        v[0] = bf16x2_of(v0, v1);
        v[1] = bf16x2_of(v2, v3);
        *reinterpret_cast<u32x2*>(out + e) = v;
      }
    }
  } else {
    for (int e = g; e < E; e += LPT) {
      if constexpr (sizeof(LT) == 4) out[e] = value(e);
      else out[e] = bf16_of(value(e));
    }
  }
  lds_sync();
}

// Tokens up to which one wave takes one token: the chain of a round is shorter
// that way, the instructions of all tokens together more.  256 experts, sigmoid
// + bias, 4 of 8 groups: 15 tokens 6.8 us against 8.3 with 16 lanes a token,
// 2047: 8.3 against 10.1, 4095: 11.0 against 10.4, 8191: 16.2 against 12.0.
// bf16 softmax: 2046: 4.4 against 4.5, 4094: 5.8 against 4.7.
constexpr int64_t kSmallBatch = 2048;

// Blocks of one wave for `waves` wave tasks, in two dimensions: a dimension
// holds fewer than 2^32 threads.
dim3 route_grid(int64_t waves) {
  constexpr int64_t kMaxX = 1 << 22;
  if (waves <= kMaxX) return dim3(static_cast<unsigned>(waves));
  return dim3(static_cast<unsigned>(kMaxX), static_cast<unsigned>((waves + kMaxX - 1) / kMaxX));
}

template <int LPT, int NV, int KEEP, typename LT>
hipError_t route_k(const RouteArgs& a, hipStream_t s) {
  const dim3 grid = route_grid((a.T + kWave / LPT - 1) / (kWave / LPT));
  if (a.bias) k_route<LPT, NV, KEEP, LT, kByScore><<<grid, kWave, 0, s>>>(a);
  else if constexpr (sizeof(LT) == 2) k_route<LPT, NV, KEEP, LT, kByBf16><<<grid, kWave, 0, s>>>(a);
  else k_route<LPT, NV, KEEP, LT, kByFp32><<<grid, kWave, 0, s>>>(a);
  return hipGetLastError();
}

template <typename LT>
hipError_t route_e(const RouteArgs& a, hipStream_t s) {
  if (a.T <= kSmallBatch) {
    if (a.E <= 256) return route_k<64, 4, 4, LT>(a, s);
    if (a.E <= 512) return route_k<64, 8, 8, LT>(a, s);
    return route_k<64, 16, 16, LT>(a, s);
  }
  if (a.E <= 64) return route_k<16, 4, 4, LT>(a, s);
  if (a.E <= 128) return route_k<16, 8, 8, LT>(a, s);
  if (a.E <= 256) return a.K <= 8 ? route_k<16, 16, 8, LT>(a, s) : route_k<16, 16, 16, LT>(a, s);
  if (a.E <= 512) return a.K <= 8 ? route_k<32, 16, 8, LT>(a, s) : route_k<32, 16, 16, LT>(a, s);
  return route_k<64, 16, 16, LT>(a, s);
}

template <typename LT>
hipError_t backward_e(const RouteArgs& a, hipStream_t s) {
  const int cap = (a.E + 3) / 4 * 4;
  auto go = [&](auto kern, int lpt) {
    const int tok = kWave / lpt;
    const int64_t waves = (a.T + tok - 1) / tok;
    kern<<<route_grid(waves), kWave, static_cast<size_t>(tok) * cap * sizeof(float), s>>>(a, cap);
    return hipGetLastError();
  };
  if (a.E <= 256) return go(k_route_backward<16, LT>, 16);
  if (a.E <= 512) return go(k_route_backward<32, LT>, 32);
  return go(k_route_backward<64, LT>, 64);
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, hipStream_t s) {
  return a.bf16 ? route_e<uint16_t>(a, s) : route_e<float>(a, s);
}

hipError_t launch_route_backward(const RouteArgs& a, hipStream_t s) {
  return a.bf16 ? backward_e<uint16_t>(a, s) : backward_e<float>(a, s);
}

}  // namespace ep
