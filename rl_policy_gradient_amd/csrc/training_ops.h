// Launchers of the embedding, its gradient and the gradients' global norm.
// Each enqueues on `st` and returns the launch's hipError_t; every argument has
// been checked by the host (gradients_api.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace plp {

// One tensor of a norm's or a clipping's launch: `tiles` workgroups begin at
// the launch's workgroup `first`, and the last of them has `tail` elements.
struct GradEntry {
  void* p;
  uint32_t first;
  uint32_t tail_bf16;  // tail << 1 | whether bf16
};
// Tensors of one launch: the table goes by value in the kernel's arguments,
// which hold 4 KB.
constexpr int kGradMaxTensors = 240;
struct GradLaunch {
  GradEntry t[kGradMaxTensors];
  uint32_t count, groups;   // tensors, workgroups
  uint32_t tile_shift;      // elements of a whole tile, log2
  uint32_t first_tensor;    // of the whole list
  uint32_t first_tile;      // this launch's first workgroup among all launches'
};

// The sums of squares: one double a tile into part, the tile each tensor begins
// at into start.
hipError_t launch_grad_squares(const GradLaunch& a, double* part, uint32_t* start, hipStream_t st);
struct GradFinish {
  const double* part;
  const uint32_t* start;
  const float* grad_scale;  // or NULL
  float *norm, *scale, *norms;  // norms may be NULL
  double max_norm, eps;
  uint32_t tiles, count;
};
static_assert(sizeof(GradLaunch) + sizeof(GradFinish) <= 4096, "kernel arguments");
hipError_t launch_grad_finish(const GradFinish& a, hipStream_t st);
// Both in one launch of one workgroup, for lists of up to so many tiles.
constexpr int kGradSmallTiles = 128;
static_assert(kGradSmallTiles <= kGradMaxTensors, "a tensor has a tile: such a list goes in one launch");
hipError_t launch_grad_small(const GradLaunch& a, const GradFinish& f, hipStream_t st);
// g = round(g scale), unless scale is 1 or not finite.
hipError_t launch_grad_clip(const GradLaunch& a, const float* scale, hipStream_t st);

// y = round(scale weight[token]); zeros for a token outside [0, V).
struct EmbedFwd {
  const int64_t* tokens;
  const void* weight;
  void* y;
  int64_t N;
  int H, V, dtype;
  float scale;
};
hipError_t launch_embed_fwd(const EmbedFwd& a, hipStream_t st);

// grad_weight (+)= scale (sum of the rows of grad_y by token), the rows of a
// token in their order. How the work is cut goes by the sizes alone.
struct EmbedBwdPlan {
  bool radix;        // N above what is sorted by counting
  int passes, bits;  // radix passes and the bits of each
  int blocks;        // workgroups of a radix pass
  int64_t per;       // tokens of each
  int slices;        // column slices of a row
  int items;         // tokens of one range
  int64_t ranges;
  bool shared;       // whether ranges can share a row
};
EmbedBwdPlan embed_bwd_plan(int64_t N, int H, int V, int grad_y_dtype);
// Columns of a partial sum: whole vectors, so that none is cut at a row's end.
__host__ __device__ inline int part_width(int H) { return (H + 7) / 8 * 8; }
struct EmbedBwd {
  const int64_t* tokens;
  const void* grad_y;
  void* grad_weight;
  int64_t N;
  int H, V, grad_y_dtype, grad_weight_dtype, accumulate;
  float scale;
  // workspace
  uint32_t *key[2], *pos[2];    // [N] each; the second pair with radix passes only
  uint32_t* hist;               // [blocks][1 << bits], with radix passes only
  float *head, *tail;           // [ranges][part_width(H)] partial sums of rows that ranges share: of the range they
                                // end in, and of those before
  int32_t* tail_row;            // [ranges] the row that tail is of, or -1
  uint32_t* shared_rows;        // how many ranges have a head
  uint2* shared_list;           // [ranges] which, and the rows they are of
};
hipError_t launch_embed_bwd(const EmbedBwd& a, hipStream_t st);

}  // namespace plp
