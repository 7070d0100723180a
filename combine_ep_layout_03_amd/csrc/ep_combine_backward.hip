// Gradient of the combine: out[t] = sum_k w[t,k] y[slot[t,k]], so
//     grad_y[slot[t,k]] = w[t,k] grad_out[t],
//     grad_w[t,k]       = <grad_out[t], y[slot[t,k]]>.
// Reads grad_out and every selected y row once and writes every selected
// grad_y row once: HBM-bound.
//
// WPT waves share one token (a block is 4 waves, 4 / WPT tokens): wave c of a
// token takes the row's vectors c * 64 + lane, + WPT * 64, ...; it loads the
// grad_out vector once and with it the K rows' vectors, so K loads are in
// flight, adds to K dot products held in registers and stores K vectors.  The
// lanes' partial sums are added in a butterfly and the waves' partial sums
// in ascending order: a fixed order, no atomics.  8192 tokens x 7168, top-8 of
// 256 (2.0 GB): 405 us, 4.9 TB/s, where a plain copy reaches 4.98; 368 us where
// every token names the same 8 experts, so neighbouring tokens' rows are
// neighbours.  K = 9, 16 and 32: 445, 778 and 1517 us, the same rate.  Above K = 8
// the two buffer resources of each selection are more scalar registers than
// there are, and 200 (up to 16) or 500 (up to 32) are spilled to lanes of vector
// registers, once a token: memory still bounds the kernel.
#include "ep_layer.h"

namespace ep {

namespace {

template <int VE>
__device__ __forceinline__ float vget(const typename VecOf<2 * VE>::type& v, int e);
template <>
__device__ __forceinline__ float vget<8>(const u32x4& v, int e) {
  return (e & 1) ? bf16_hi(v[e >> 1]) : bf16_lo(v[e >> 1]);
}
template <>
__device__ __forceinline__ float vget<4>(const u32x2& v, int e) {
  return (e & 1) ? bf16_hi(v[e >> 1]) : bf16_lo(v[e >> 1]);
}
template <>
__device__ __forceinline__ float vget<2>(const uint32_t& v, int e) {
  return e ? bf16_hi(v) : bf16_lo(v);
}
template <>
__device__ __forceinline__ float vget<1>(const uint16_t& v, int) {
  return bf16_to_f32(v);
}

// the vector of bf16(w * v)
__device__ __forceinline__ u32x4 scaled(const u32x4& v, float w) {
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = bf16x2_of(w * bf16_lo(v[i]), w * bf16_hi(v[i]));
  return r;
}
__device__ __forceinline__ u32x2 scaled(const u32x2& v, float w) {
  u32x2 r;
#pragma unroll
  for (int i = 0; i < 2; ++i) r[i] = bf16x2_of(w * bf16_lo(v[i]), w * bf16_hi(v[i]));
  return r;
}
__device__ __forceinline__ uint32_t scaled(uint32_t v, float w) {
  return bf16x2_of(w * bf16_lo(v), w * bf16_hi(v));
}
__device__ __forceinline__ uint16_t scaled(uint16_t v, float w) { return bf16_of(w * bf16_to_f32(v)); }

// Non-temporal buffer stores of 16, 8, 4 and 2 bytes; past the resource's end
// they are dropped.
__device__ __forceinline__ void buffer_store_nt(__amdgpu_buffer_rsrc_t r, uint32_t off, u32x4 v) {
  __builtin_amdgcn_raw_buffer_store_b128(v, r, static_cast<int>(off), 0, 2);
}
__device__ __forceinline__ void buffer_store_nt(__amdgpu_buffer_rsrc_t r, uint32_t off, u32x2 v) {
  __builtin_amdgcn_raw_buffer_store_b64(v, r, static_cast<int>(off), 0, 2);
}
__device__ __forceinline__ void buffer_store_nt(__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t v) {
  __builtin_amdgcn_raw_buffer_store_b32(v, r, static_cast<int>(off), 0, 2);
}
__device__ __forceinline__ void buffer_store_nt(__amdgpu_buffer_rsrc_t r, uint32_t off, uint16_t v) {
  __builtin_amdgcn_raw_buffer_store_b16(v, r, static_cast<int>(off), 0, 2);
}

template <int KMAX, int VE, int WPT>
__global__ __launch_bounds__(kBlock) void k_combine_backward(CombineBackwardArgs a, int64_t groups) {
  using V = typename VecOf<2 * VE>::type;
  __shared__ float part[kWavesPerBlock][KMAX];
  if (!layout_current(a.status, a.generation)) return;  // the whole grid, before any barrier
  constexpr int kTokens = kWavesPerBlock / WPT;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
  const int c = wave % WPT;
  const int nvec = a.H / VE;
  const uint32_t row_bytes = static_cast<uint32_t>(nvec) * static_cast<uint32_t>(sizeof(V));
  for (int64_t grp = blockIdx.x; grp < groups; grp += gridDim.x) {
    const int64_t t = grp * kTokens + wave / WPT;
    const bool live = t < a.T;
    int s = -1;
    float wt = 0.0f;
    if (live && lane < a.K) {
      s = a.slot[t * a.K + lane];
      wt = a.w[t * a.K + lane];
      if (s >= 0 && static_cast<int64_t>(s) >= a.y_rows) {
        a.status[kStatusCombineOob] = 1;
        s = -1;
      }
    }
    // The token's rows as buffer resources with wave-uniform bases; a
    // selection without a row gets an empty one, whose loads return zeros
    // and whose stores are dropped.
    __amdgpu_buffer_rsrc_t in_row[KMAX], out_row[KMAX];
    float w[KMAX], dot[KMAX];
#pragma unroll
    for (int k = 0; k < KMAX; ++k) {
      const int row = readlane(s, k);
      const int64_t off = static_cast<int64_t>(row < 0 ? 0 : row) * row_bytes;
      in_row[k] = buffer_rsrc(static_cast<const char*>(a.y) + off, row < 0 ? 0u : row_bytes);
      out_row[k] = buffer_rsrc(static_cast<char*>(a.gy) + off, row < 0 ? 0u : row_bytes);
      w[k] = __int_as_float(readlane(__float_as_int(wt), k));
      dot[k] = 0.0f;
    }
    if (live) {
      const V* go = static_cast<const V*>(a.go) + t * nvec;
      for (int i = c * kWave + lane; i < nvec; i += WPT * kWave) {
        const uint32_t off = static_cast<uint32_t>(i) * static_cast<uint32_t>(sizeof(V));
        const V g = go[i];
        V in[KMAX];
#pragma unroll
        for (int k = 0; k < KMAX; ++k) in[k] = buffer_load_nt<V>(in_row[k], off);
#pragma unroll
        for (int k = 0; k < KMAX; ++k) {
          buffer_store_nt(out_row[k], off, scaled(g, w[k]));
#pragma unroll
          for (int e = 0; e < VE; ++e)
            dot[k] = __builtin_fmaf(vget<VE>(g, e), vget<VE>(in[k], e), dot[k]);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < KMAX; ++k) {
#pragma unroll
      for (int off = kWave / 2; off > 0; off >>= 1) dot[k] += __shfl_xor(dot[k], off, kWave);
    }
    if (lane == 0) {
#pragma unroll
      for (int k = 0; k < KMAX; ++k) part[wave][k] = dot[k];
    }
    __syncthreads();
    if (live && c == 0 && lane < a.K) {
      float sum = part[wave][lane];
#pragma unroll
      for (int i = 1; i < WPT; ++i) sum += part[wave + i][lane];
      a.gw[t * a.K + lane] = s >= 0 ? sum : 0.0f;
    }
    __syncthreads();  // the partial sums are read before the next tokens' are written
  }
}

template <int KMAX, int VE, int WPT>
hipError_t launch_t(const CombineBackwardArgs& a, hipStream_t s) {
  constexpr int64_t kTokens = kWavesPerBlock / WPT;
  constexpr int64_t kMaxBlocks = (1LL << 24) - 1;  // a grid holds fewer than 2^32 threads
  const int64_t groups = (a.T + kTokens - 1) / kTokens;
  k_combine_backward<KMAX, VE, WPT>
      <<<static_cast<unsigned>(groups < kMaxBlocks ? groups : kMaxBlocks), kBlock, 0, s>>>(a, groups);
  return hipGetLastError();
}

// One wave a token where the row has one vector per lane at most (8193 x 256,
// top-2: 6.5 us against 11.6 with four waves; 8191 x 512: 9.2 against 13.4),
// else four (8191 x 2048, top-8: 107 us against 117 with one; 126 tokens: 5.3
// against 8.1; 8192 x 7168: 405 against 401).
template <int KMAX, int VE>
hipError_t launch_w(const CombineBackwardArgs& a, hipStream_t s) {
  return a.H / VE <= kWave ? launch_t<KMAX, VE, 1>(a, s) : launch_t<KMAX, VE, 4>(a, s);
}

template <int KMAX>
hipError_t launch_v(const CombineBackwardArgs& a, int ve, hipStream_t s) {
  switch (ve) {
    case 8: return launch_w<KMAX, 8>(a, s);
    case 4: return launch_w<KMAX, 4>(a, s);
    case 2: return launch_w<KMAX, 2>(a, s);
    default: return launch_w<KMAX, 1>(a, s);
  }
}

}  // namespace

hipError_t launch_combine_backward(const CombineBackwardArgs& a, int vec_elems, hipStream_t s) {
  if (a.K <= 1) return launch_v<1>(a, vec_elems, s);
  if (a.K <= 2) return launch_v<2>(a, vec_elems, s);
  if (a.K <= 4) return launch_v<4>(a, vec_elems, s);
  if (a.K <= 8) return launch_v<8>(a, vec_elems, s);
  if (a.K <= 16) return launch_v<16>(a, vec_elems, s);
  return launch_v<32>(a, vec_elems, s);
}

}  // namespace ep
