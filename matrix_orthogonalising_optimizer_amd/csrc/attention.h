// Launch interface of the attention kernels (attention_*.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dmuon {

// Queries, keys and values as (token, head, element); strides in bytes, the
// elements of a head contiguous, every row of a head 16-byte aligned and
// `dim_in` elements (a multiple of 16 bytes, those past `dim` zero) long.
struct AttnView {
  const void* p;
  int64_t ts, hs;  // from token to token, from head to head
};
struct AttnArgs {
  AttnView q, k, v;
  AttnView dy, y;          // backward
  void* out;               // (tokens_q, heads, dim): y, or dq
  void* dk;                // (tokens_k, kv_heads, dim)
  void* dv;
  float* lse;              // (heads, tokens_q)
  float* stats;            // backward: lse log2 e, then the rows' sums of dy y, (kv_heads, tokens_q, group) each
  const int32_t* cu_q;     // sequences + 1 first rows each, or both null: equal lengths
  const int32_t* cu_k;
  int64_t tokens_q, tokens_k;
  int32_t sequences, heads, kv_heads, group;  // group = heads / kv_heads
  uint32_t group_magic;    // ceil(2^32 / group), 0 for 1: x / group by one multiplication
  int32_t dim, dim_in;
  int32_t causal;
  int32_t vec_out;         // results' rows are 16-byte aligned
  float scale;
  uint32_t slots;          // tiles of rows (or of keys), an upper bound
  uint32_t unit0;          // first unit of the launch
  int32_t wide;            // tiles of 256 rows (or keys) shared by eight waves, or of 128 by four
  int32_t parts;           // workgroups that share a tile's work; with more than one their results go to
  float* partial;          // (parts, tokens_q, heads, padded width), or (parts, dk and dv, tokens_k, kv_heads, ..)
  float2* partial_ml;      // forward, (parts, heads, tokens_q): the rows' references and sums
};

// ATTN_JOIN_..: the parts of the results.
enum AttnPass : int { ATTN_FWD = 0, ATTN_DQ = 1, ATTN_DKV = 2, ATTN_JOIN_FWD = 3, ATTN_JOIN_DQ = 4, ATTN_JOIN_KEYS = 5 };

// `padded`: the head width that the kernel is built for (attn_padded).
hipError_t launch_attn_bf16_64(AttnPass pass, const AttnArgs& a, int64_t grid, hipStream_t st);
hipError_t launch_attn_bf16_96(AttnPass pass, const AttnArgs& a, int64_t grid, hipStream_t st);
hipError_t launch_attn_bf16_128(AttnPass pass, const AttnArgs& a, int64_t grid, hipStream_t st);
hipError_t launch_attn_bf16_256(AttnPass pass, const AttnArgs& a, int64_t grid, hipStream_t st);
hipError_t launch_attn_f32_64(AttnPass pass, const AttnArgs& a, int64_t grid, hipStream_t st);
hipError_t launch_attn_f32_96(AttnPass pass, const AttnArgs& a, int64_t grid, hipStream_t st);
hipError_t launch_attn_f32_128(AttnPass pass, const AttnArgs& a, int64_t grid, hipStream_t st);

// Heads whose rows are not 16-byte aligned or whole 16-byte chunks, copied to
// (token, head, dim_in) with zeros past dim.
struct GatherArgs {
  const void* src[5];
  void* dst[5];
  int64_t ts[5], hs[5];  // elements
  int64_t tokens[5];
  int32_t heads[5];
  int32_t n, dim, dim_in, esize;
};
hipError_t launch_gather_heads(const GatherArgs& a, hipStream_t st);

}  // namespace dmuon
