// Router: each token's K experts of largest selection value, and its weights.
//
// LPT lanes work on one token (16 up to 256 experts, 32 up to 512, 64 up to
// 1024), so a wave takes 64 / LPT tokens and the reductions of K rounds run
// for all of them at once; lane g of a token holds experts j * 4 * LPT + 4 g
// + c (c < 4), up to NV of them in registers.
//
// The K rounds find a maximum over keys (value, then lowest index, in one
// unsigned integer: 64 bits, or 32 for bf16 logits without a bias) and drop
// it.  Values that a rounding could order wrongly (scores plus a bias, sums
// of scores) are computed in fp32 with a bound on their error; a token whose
// neighbouring values lie within it, and are not the values of one and the
// same logit and bias, is done again in binary64.  That is about one token in
// a thousand, and gives the order of the binary64 values for all.
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

// order-preserving map to unsigned integers
__device__ __forceinline__ uint32_t ordered(float f) {
  const uint32_t b = __float_as_uint(f);
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
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
struct Sum {
  template <typename T>
  __device__ __forceinline__ T operator()(T a, T b) const {
    return a + b;
  }
};
// the reduction of v over the token's LPT lanes, in every one of them
template <int LPT, typename T, typename F>
__device__ __forceinline__ T over_token(T v, F f) {
  v = f(v, turn<8>(v));
  v = f(v, turn<4>(v));
  v = f(v, turn<2>(v));
  v = f(v, turn<1>(v));
  if constexpr (LPT >= 32) v = f(v, turn<16>(v));
  if constexpr (LPT >= 64) v = f(v, turn<32>(v));
  return v;
}
// v of the token's lane g
template <int LPT, typename T>
__device__ __forceinline__ T from_lane(T v, int g) {
  return __shfl(v, g, LPT);
}

// ------------------------------------------------------------------- groups
// The open groups of one token as a bit mask, from selection values val[E] in
// LDS (-inf: cannot be chosen).  `err(v)` bounds the error of a group's value;
// near is set where the last open and the first closed group are closer.
template <int LPT, typename F, typename Err>
__device__ __forceinline__ uint64_t open_groups(const F* val, const RouteArgs& a, int g, F* gv,
                                                Err err, bool& near) {
  const F none = -__builtin_inf();
  for (int q = g; q < a.G; q += LPT) {
    F m1 = none, m2 = none;
    int i = q % a.gsize;  // staggered starts keep the lanes on different LDS banks
    for (int n = 0; n < a.gsize; ++n) {
      const F v = val[q * a.gsize + i];
      if (v > m1) {
        m2 = m1;
        m1 = v;
      } else if (v > m2) {
        m2 = v;
      }
      if (++i == a.gsize) i = 0;
    }
    gv[q] = (a.gtop == 2 && m2 > none) ? m1 + m2 : m1;
  }
  lds_sync();
  uint32_t lo = 0, hi = 0;
  F last = __builtin_inf(), next = none;
  for (int q = g; q < a.G; q += LPT) {
    const F v = gv[q];
    int better = 0;
    for (int o = 0; o < a.G; ++o) {
      const F u = gv[o];
      better += (u > v || (u == v && o < q)) ? 1 : 0;
    }
    if (better < a.tg) {
      if (q < 32) lo |= 1u << q;
      else hi |= 1u << (q - 32);
      last = v < last ? v : last;
    } else {
      next = v > next ? v : next;
    }
  }
  lo = over_token<LPT>(lo, [](uint32_t x, uint32_t y) { return x | y; });
  hi = over_token<LPT>(hi, [](uint32_t x, uint32_t y) { return x | y; });
  last = over_token<LPT>(last, Min());
  next = over_token<LPT>(next, Max());
  // two infinities are equal values, and equal values go to the lowest index
  near = next > none && last - next <= err(last) + err(next);
  return (static_cast<uint64_t>(hi) << 32) | lo;
}

// e / gsize for e < 1024: (e * m) >> 20 with m = ceil(2^20 / gsize) is exact,
// as e * (m * gsize - 2^20) <= 1023 * 1023 < 2^20
__device__ __forceinline__ int group_of(int e, uint32_t magic) {
  return static_cast<int>((static_cast<uint32_t>(e) * magic) >> 20);
}

// --------------------------------------------------------- binary64, in LDS
__device__ __forceinline__ double sigmoid64(double l) { return 1.0 / (1.0 + exp(-l)); }

// The experts of selections g and g + LPT of a token, -1 where there is none.
struct Chosen {
  int lo = -1, hi = -1;
  template <int LPT>
  __device__ __forceinline__ void set(int k, int g, int e) {
    if (k == g) lo = e;
    if (LPT < 32 && k == g + LPT) hi = e;
  }
  __device__ __forceinline__ int operator[](int i) const { return i == 0 ? lo : hi; }
};

// One token again in binary64.  val [E], gv [kMaxRouteGroups] in LDS.
template <int LPT, typename LT>
__device__ __forceinline__ Chosen choose64(const RouteArgs& a, const LT* logits, int g, float lmax,
                                        double* val, double* gv) {
  const double none = -__builtin_inf();
  const int E = a.E;
  double sum = 0.0;
  if (!a.sigmoid) {
    for (int e = g; e < E; e += LPT) {
      const float l = clean_logit(raw_logit(logits + e));
      if (l > kNegInf) sum += exp(static_cast<double>(l) - static_cast<double>(lmax));
    }
    sum = over_token<LPT>(sum, Sum());
  }
  auto score = [&](float l) {
    return a.sigmoid ? sigmoid64(l) : exp(static_cast<double>(l) - static_cast<double>(lmax)) / sum;
  };
  uint64_t open = ~0ull;
  const uint32_t magic = a.G ? ((1u << 20) + a.gsize - 1) / a.gsize : 0u;
  if (a.G) {
    const bool by_logit = !a.bias && a.gtop == 1;
    for (int e = g; e < E; e += LPT) {
      const float l = clean_logit(raw_logit(logits + e));
      double v = by_logit ? static_cast<double>(l) : score(l) + (a.bias ? static_cast<double>(a.bias[e]) : 0.0);
      if (l == kNegInf || v != v) v = none;
      val[e] = v;
    }
    lds_sync();
    bool near;
    open = open_groups<LPT>(val, a, g, gv, [](double) { return 0.0; }, near);
    lds_sync();
  }
  for (int e = g; e < E; e += LPT) {
    const float l = clean_logit(raw_logit(logits + e));
    double v = a.bias ? score(l) + static_cast<double>(a.bias[e]) : static_cast<double>(l);
    if (l == kNegInf || v != v || (a.G && !((open >> group_of(e, magic)) & 1))) v = none;
    val[e] = v;
  }
  lds_sync();
  Chosen chosen;
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
    if (win == UINT32_MAX) break;
    if (static_cast<int>(win) % LPT == g) val[win] = none;
    lds_sync();
    chosen.template set<LPT>(k, g, static_cast<int>(win));
  }
  return chosen;
}

// ------------------------------------------------------------------ forward
// KEY32: bf16 logits without a bias, whose key fits 32 bits.
template <int LPT, int NV, typename LT, bool KEY32>
__global__ __launch_bounds__(kWave) void k_route(RouteArgs a, int64_t waves) {
  constexpr int kTok = kWave / LPT;  // tokens per wave
  constexpr int kCap = LPT * NV;     // experts a token's lanes hold
  __shared__ double s_val[kTok * kCap];
  __shared__ double s_gv[kTok * kMaxRouteGroups];
  const int lane = threadIdx.x;
  const int g = lane % LPT;
  const int tok = lane / LPT;
  const int E = a.E, K = a.K;
  const LT* all = static_cast<const LT*>(a.logits);
  float* valf = reinterpret_cast<float*>(s_val + tok * kCap);
  float* gvf = reinterpret_cast<float*>(s_gv + tok * kMaxRouteGroups);
  const uint32_t magic = a.G ? ((1u << 20) + a.gsize - 1) / a.gsize : 0u;
  const bool vec = E % 4 == 0 && (reinterpret_cast<uintptr_t>(all) & (4 * sizeof(LT) - 1)) == 0;
  const bool scored = a.bias != nullptr;  // experts compared by score + bias
  const bool need_scores = scored || (a.G && a.gtop == 2);
  const bool need_sum = !a.sigmoid && (need_scores || !a.renorm);

  for (int64_t wv = blockIdx.x; wv < waves; wv += gridDim.x) {
    const int64_t t = wv * kTok + tok;
    if (t >= a.T) continue;  // whole groups of LPT lanes: the reductions stay within a token
    const LT* row = all + t * E;
    Chosen chosen;
    const bool masked = a.mask && a.mask[t] == 0;
    float lmax = kNegInf, lsum = 1.0f;
    if (!masked) {
      float l[NV];
#pragma unroll
      for (int j = 0; j < NV / 4; ++j) {
        const int e0 = j * 4 * LPT + 4 * g;
        if (vec) {
          if (e0 < E) {
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
          } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) l[4 * j + c] = kNegInf;
          }
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c) l[4 * j + c] = e0 + c < E ? raw_logit(row + e0 + c) : kNegInf;
        }
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) l[i] = clean_logit(l[i]);
      auto expert = [&](int i) { return (i / 4) * 4 * LPT + 4 * g + i % 4; };

      if (need_sum) {
        float m = l[0];
#pragma unroll
        for (int i = 1; i < NV; ++i) m = fmaxf(m, l[i]);
        lmax = over_token<LPT>(m, Max());
        float s = 0.0f;
        if (lmax > kNegInf) {
#pragma unroll
          for (int i = 0; i < NV; ++i) s += expf(l[i] - lmax);
        }
        lsum = over_token<LPT>(s, Sum());
      }

      // selection values, and the bound on their error: a score's relative
      // error is below 2^-21 for the sigmoid (exponential, sum, quotient: 4
      // roundings) and 2^-17 for the softmax (the rounded exponent l - max,
      // up to 88, adds 88 * 2^-24); adding the bias is one more rounding
      float c[KEY32 ? 1 : NV];
      float bmax = 0.0f;
      if constexpr (!KEY32) {
#pragma unroll
        for (int i = 0; i < NV; ++i) c[i] = l[i];
      }
      const float rel = a.sigmoid ? 0x1p-21f : 0x1p-17f;
      bool near = false;
      uint64_t open = ~0ull;
      if (need_scores) {
        float score[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          float v = a.sigmoid ? 1.0f / (1.0f + expf(-l[i])) : expf(l[i] - lmax) / lsum;
          if (scored) {
            const float b = expert(i) < E ? a.bias[expert(i)] : 0.0f;
            if (fabsf(b) < __builtin_inff()) bmax = fmaxf(bmax, fabsf(b));
            v += b;
          }
          score[i] = (l[i] == kNegInf || v != v) ? kNegInf : v;
        }
        if (scored) {
          bmax = over_token<LPT>(bmax, Max());
          if constexpr (!KEY32) {
#pragma unroll
            for (int i = 0; i < NV; ++i) c[i] = score[i];
          }
        }
        if (a.G) {
#pragma unroll
          for (int i = 0; i < NV; ++i)
            if (expert(i) < E) valf[expert(i)] = score[i];
        }
      } else if (a.G) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (expert(i) < E) valf[expert(i)] = l[i];
      }
      auto err = [&](float v) {
        return rel * fminf(1.0f, fabsf(v) + bmax) + 0x1p-23f * fabsf(v) + 1e-37f;
      };
      if (a.G) {
        lds_sync();
        if (need_scores) {
          // a sum of two values: twice the bound, and the sum's rounding
          open = open_groups<LPT>(valf, a, g, gvf, [&](float v) {
            return 2.0f * (rel * fminf(1.0f, fabsf(v) + 2.0f * bmax) + 0x1p-22f * (fabsf(v) + bmax) + 1e-37f);
          }, near);
        } else {
          open = open_groups<LPT>(valf, a, g, gvf, [](float) { return 0.0f; }, near);
          near = false;  // logits are exact: equal groups go to the lowest index
        }
        lds_sync();
      }

      if (!near) {
        // keys: the ordered value above the complement of the index; 0 = none
        if constexpr (KEY32) {
          uint32_t key[NV];
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            const int e = expert(i);
            const bool ok = l[i] > kNegInf && (!a.G || ((open >> group_of(e, magic)) & 1));
            // only +inf, cleaned, reaches the largest finite fp32 here: it
            // stays above the largest bf16
            const uint32_t value = l[i] >= FLT_MAX ? 0xFF800000u : ordered(l[i]) & 0xFFFF0000u;
            key[i] = ok ? value | (0xFFFFu - static_cast<uint32_t>(e)) : 0u;
          }
          for (int k = 0; k < K; ++k) {
            uint32_t m = key[0];
#pragma unroll
            for (int i = 1; i < NV; ++i) m = m > key[i] ? m : key[i];
            m = over_token<LPT>(m, Max());
            if (m == 0u) break;
#pragma unroll
            for (int i = 0; i < NV; ++i) key[i] = key[i] == m ? 0u : key[i];
            chosen.template set<LPT>(k, g, static_cast<int>(0xFFFFu - (m & 0xFFFFu)));
          }
        } else {
          uint64_t key[NV];
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            const int e = expert(i);
            const bool ok = c[i] > kNegInf && (!a.G || ((open >> group_of(e, magic)) & 1));
            key[i] = ok ? (static_cast<uint64_t>(ordered(c[i])) << 32) | ~static_cast<uint32_t>(e) : 0ull;
          }
          float prev = 0.0f;
          int prev_e = -1;
          // one round more than K: the first expert left out must be clear of the last chosen
          for (int k = 0; k < K + (scored ? 1 : 0); ++k) {
            uint64_t m = key[0];
#pragma unroll
            for (int i = 1; i < NV; ++i) m = m > key[i] ? m : key[i];
            m = over_token<LPT>(m, Max());
            if (m == 0ull) break;
            const int e = static_cast<int>(~static_cast<uint32_t>(m));
            if (scored) {
              const float v = unordered(static_cast<uint32_t>(m >> 32));
              if (prev_e >= 0 && prev - v <= err(prev) + err(v)) {
                // values of one and the same logit and bias are equal in binary64 too
                const bool same = raw_logit(row + e) == raw_logit(row + prev_e) && a.bias[e] == a.bias[prev_e];
                if (!same) near = true;
              }
              prev = v;
              prev_e = e;
            }
            if (k == K || near) break;
#pragma unroll
            for (int i = 0; i < NV; ++i) key[i] = key[i] == m ? 0ull : key[i];
            chosen.template set<LPT>(k, g, e);
          }
        }
      }
      if (near) chosen = choose64<LPT>(a, row, g, lmax, s_val + tok * kCap, s_gv + tok * kMaxRouteGroups);
    }

    // weights of selections g and g + LPT
    constexpr int kSlots = LPT >= 32 ? 1 : 2;
    float lc[kSlots], w[kSlots];
    float top = kNegInf;
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      lc[i] = chosen[i] >= 0 ? clean_logit(raw_logit(row + chosen[i])) : kNegInf;
      top = fmaxf(top, lc[i]);
    }
    if (a.renorm) {
      // relative to the largest: softmax exp(l - top); sigmoid(l) =
      // exp(-log(1 + exp(-l)))
      top = over_token<LPT>(top, Max());
      const float ltop = fminf(top, 0.0f) - log1pf(expf(-fabsf(top)));
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < kSlots; ++i) {
        float e = 0.0f;
        if (chosen[i] >= 0) {
          e = a.sigmoid ? expf(fminf(lc[i], 0.0f) - log1pf(expf(-fabsf(lc[i]))) - ltop) : expf(lc[i] - top);
        }
        w[i] = e;
        sum += e;
      }
      sum = over_token<LPT>(sum, Sum());
#pragma unroll
      for (int i = 0; i < kSlots; ++i) w[i] = w[i] / sum * a.scale;
    } else {
#pragma unroll
      for (int i = 0; i < kSlots; ++i)
        w[i] = (a.sigmoid ? 1.0f / (1.0f + expf(-lc[i])) : expf(lc[i] - lmax) / lsum) * a.scale;
    }
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      const int k = g + i * LPT;
      if (k < K) {
        a.idx[t * K + k] = chosen[i];
        a.w[t * K + k] = chosen[i] >= 0 ? w[i] : 0.0f;
      }
    }
  }
}

// ----------------------------------------------------------------- backward
// Lane g of a token holds selections g and g + LPT; the gradient's row is put
// together in LDS and written whole.
template <int LPT, typename LT>
__global__ __launch_bounds__(kWave) void k_route_backward(RouteArgs a, int64_t waves, int cap) {
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
  for (int64_t wv = blockIdx.x; wv < waves; wv += gridDim.x) {
    const int64_t t = wv * kTok + tok;
    if (t >= a.T) continue;
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
      const float ltop = fminf(top, 0.0f) - log1pf(expf(-fabsf(top)));
      float w[kSlots];
      float sum = 0.0f, dot = 0.0f;
#pragma unroll
      for (int i = 0; i < kSlots; ++i) {
        w[i] = 0.0f;
        if (lc[i] > kNegInf)
          w[i] = a.sigmoid ? expf(fminf(lc[i], 0.0f) - log1pf(expf(-fabsf(lc[i]))) - ltop) : expf(lc[i] - top);
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
        if (a.sigmoid) d[i] *= 1.0f / (1.0f + expf(lc[i]));
      }
    } else if (a.sigmoid) {
#pragma unroll
      for (int i = 0; i < kSlots; ++i) d[i] = gw[i] / (1.0f + expf(lc[i])) * (1.0f / (1.0f + expf(-lc[i])));
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
}

// Blocks (one wave each) for `waves` wave tasks; the kernels walk them
// cyclically, so a capped grid still covers them.
unsigned route_blocks(int64_t waves) {
  constexpr int64_t kMaxBlocks = 1 << 22;
  return static_cast<unsigned>(waves < kMaxBlocks ? waves : kMaxBlocks);
}

template <int LPT, int NV, typename LT>
hipError_t route_k(const RouteArgs& a, hipStream_t s) {
  const int64_t waves = (a.T + kWave / LPT - 1) / (kWave / LPT);
  if constexpr (sizeof(LT) == 2) {
    if (!a.bias) {
      k_route<LPT, NV, LT, true><<<route_blocks(waves), kWave, 0, s>>>(a, waves);
      return hipGetLastError();
    }
  }
  k_route<LPT, NV, LT, false><<<route_blocks(waves), kWave, 0, s>>>(a, waves);
  return hipGetLastError();
}

template <typename LT>
hipError_t route_e(const RouteArgs& a, hipStream_t s) {
  if (a.E <= 64) return route_k<16, 4, LT>(a, s);
  if (a.E <= 128) return route_k<16, 8, LT>(a, s);
  if (a.E <= 256) return route_k<16, 16, LT>(a, s);
  if (a.E <= 512) return route_k<32, 16, LT>(a, s);
  return route_k<64, 16, LT>(a, s);
}

template <typename LT>
hipError_t backward_e(const RouteArgs& a, hipStream_t s) {
  const int cap = (a.E + 3) / 4 * 4;
  auto go = [&](auto kern, int lpt) {
    const int tok = kWave / lpt;
    const int64_t waves = (a.T + tok - 1) / tok;
    kern<<<route_blocks(waves), kWave, static_cast<size_t>(tok) * cap * sizeof(float), s>>>(a, waves, cap);
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
