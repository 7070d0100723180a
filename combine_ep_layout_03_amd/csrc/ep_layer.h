// Internal launch interface of the layer operators (ep_mi355x_layer.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "ep_device.h"
#include "ep_internal.h"

namespace ep {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

// fp32 -> bf16, round to nearest even by the hardware conversion, which keeps
// infinities and NaN (f32_to_bf16_bits is for finite sums).
__device__ __forceinline__ uint16_t bf16_of(float f) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f));
}
__device__ __forceinline__ uint32_t bf16x2_of(float lo, float hi) {
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  b2 v;
  v[0] = static_cast<__bf16>(lo);
  v[1] = static_cast<__bf16>(hi);
  return __builtin_bit_cast(uint32_t, v);
}

constexpr int kMaxRouteGroups = 64;  // EP_MAX_ROUTE_GROUPS

struct RouteArgs {
  const void* logits;  // [T, E], fp32 or bf16
  const float* bias;   // optional [E]
  const uint8_t* mask;  // optional [T], 0 = no selection
  int64_t* idx;        // [T, K]
  float* w;            // [T, K]
  const float* gw;     // backward: [T, K]
  void* glogits;       // backward: [T, E], the logits' type
  int64_t T;
  int E, K;
  int G;        // expert groups, 0 = none
  int gsize;    // E / G
  int tg;       // groups that stay open
  int gtop;     // 1 or 2
  bool sigmoid, renorm, bf16;
  float scale;
};
hipError_t launch_route(const RouteArgs& a, hipStream_t s);
hipError_t launch_route_backward(const RouteArgs& a, hipStream_t s);

// EP_STATUS_COMBINE_OOB
constexpr int kStatusCombineOob = 4;

struct CombineBackwardArgs {
  const void* go;   // bf16 [T, H]
  const void* y;    // bf16 [y_rows, H]
  void* gy;         // bf16 [y_rows, H]
  const float* w;   // [T, K]
  float* gw;        // [T, K]
  const int32_t* slot;
  int32_t* status;
  uint32_t generation;
  int64_t T, y_rows;
  int K, H;
};
// `vec_elems` in {8, 4, 2, 1} divides H and the base alignments (in bf16 elements).
hipError_t launch_combine_backward(const CombineBackwardArgs& a, int vec_elems, hipStream_t s);

// Low-rank adapters.  Launch geometry, from the sizes alone (how many rows
// each expert has is known on the device only).
struct LoraGeom {
  int64_t rows;       // expert-major rows at most, padding included
  int row_tiles;      // 16-row sub-tiles per row tile: 1, 2 or 4
  int64_t max_tiles;  // row tiles at most
  int expand_shift;    // log2 of the rows of a tile of the result
  int64_t max_expand;  // such tiles at most
  int split_x;        // splits of the contraction over H (u = A x)
  int split_g;        // splits of the contraction over N (v = B^T g; backward)
  int chunk_shift;    // log2 of the rows of a weight-gradient chunk
  int64_t max_chunks;  // weight-gradient chunks at most
  int64_t slots;       // partial gradients of experts with several chunks, at most
  // workspace parts, multiples of 16
  size_t expand_bytes, chunk_bytes, u_bytes, v_bytes, slot_bytes;
  size_t bytes() const { return expand_bytes + chunk_bytes + u_bytes + v_bytes + slot_bytes; }
};
// blocks that write the rows of no selection, at most
constexpr int64_t kLoraMaxCopyBlocks = 2048;
LoraGeom lora_geom(int64_t rows, int E, int H, int N, int R, bool backward);

struct LoraArgs {
  const uint16_t* x;  // bf16 rows, row stride ldx
  int64_t ldx;
  const int32_t* xmap;  // row of x for each expert-major row; null: itself
  const uint16_t* base;  // null: zeros
  int64_t ldbase;
  uint16_t* out;
  int64_t ldout;
  const int32_t* omap;  // row of base and out; null: itself
  const uint16_t* a;    // [E, R, H]
  const uint16_t* b;    // [E, N, R]
  const float* scales;  // [E], null: 1
  const int32_t* counts;
  const int32_t* offsets;
  const int32_t* slot;  // [T], to find the tokens of no row (omap only)
  int64_t T;
  int K, E, H, N, R;
  // backward: grad_out [.., N] with omap's rows, base and out are [.., H]
  const uint16_t* go;
  int64_t ldgo;
  uint16_t* ga;  // [E, R, H]
  uint16_t* gb;  // [E, N, R]
  int32_t* expand_tiles;  // workspace: 4 words per tile of the result
  int32_t* chunks;        // and per weight-gradient chunk
  float* u;      // split_x partial sums of [rows, R]
  float* v;      // split_g partial sums of [rows, R]
  float* slots;  // partial gradients
  int32_t* status;
  uint32_t generation;
};
// blocks of the weight gradients
int64_t lora_weight_blocks(const LoraGeom& g, int H, int N, int R);
hipError_t launch_lora(const LoraArgs& a, const LoraGeom& g, hipStream_t s);
hipError_t launch_lora_backward(const LoraArgs& a, const LoraGeom& g, hipStream_t s);

}  // namespace ep
