// Launch interface of the norm and rotation of heads (heads.hip) and of dropout
// (dropout.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attention.h"

namespace dmuon {

constexpr int kRopeHalf = 128;   // most pairs of a head
constexpr int kRopeTokens = 16;  // most tokens of a step of a workgroup

struct RopeArgs {
  AttnView x[2];          // q and k
  AttnView dy[2];         // backward
  void* out[2];           // contiguous: y, or dx
  const void* w[2];       // both null: rotation alone
  void* dw[2];
  float* part;            // backward with weights: dim floats for each workgroup
  const void* positions;  // int64, (tokens, axes)
  int64_t tokens;
  int32_t heads[2];
  int32_t axes, dim, rot, interleaved, esize;
  int32_t parts[2];       // workgroups of q's and k's heads, tokens of a step: rope_cut
  int32_t step[2];
  float eps;
  double turn[kRopeHalf];  // turns of pair p per step of its position
  uint8_t axis[kRopeHalf];
};
void rope_cut(RopeArgs& a, bool bwd);
hipError_t launch_rope(const RopeArgs& a, bool bwd, hipStream_t st);

struct DropoutArgs {
  const void* x;
  const void* residual;  // nullable
  void* y;
  int64_t n;
  uint64_t seed, offset;
  const int64_t* state;  // device, nullable: seed and a number added to offset
  uint32_t cut;          // of 65536: a number below it drops its element
  float scale;
  int32_t esize;
};
hipError_t launch_dropout(const DropoutArgs& a, hipStream_t st);

}  // namespace dmuon
