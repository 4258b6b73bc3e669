// layer.h -- the attention-layer operators' launches, shared by their entry
// points (layer_api.cpp) and their kernels (rope.hip, attention.hip,
// lora.hip).  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>

#include "libconv.h"

namespace libconv {

// libconv_qk_norm_rope; strides in bytes.
struct RopeArgs {
  const char* in[3];        // q, k, v
  char* out[3];
  long long in_row[3], in_head[3], out_row[3], out_head[3];
  const void* weight[2];    // q, k; may be null
  const double* freqs;
  const int* positions;
  const int* slots;
  int T, heads[3];          // heads[2]: 0 without v
  int D, half;              // half: pairs that turn
  int pairs0, pairs01;      // pairs of axis 0, of axes 0 and 1
  int interleaved, out_rows;
  float eps;
  int steps, chunks;        // filled by the launch
  int step_k, step_v;       // first steps of the keys and of the values
};
libconv_status rope_launch(RopeArgs a, int dtype, hipStream_t stream);

// libconv_prefix_attention; strides in bytes.
struct AttnArgs {
  const char *q, *kp, *vp, *k, *v;
  const int* lengths;
  char* out;
  float* lse;
  long long q_b, q_r, q_h, kp_r, kp_h, vp_r, vp_h, k_b, k_r, k_h, v_b, v_r, v_h, o_b, o_r, o_h;
  int B, Sq, P, S, Hk, G, D;
  float scale;              // |scale| log2(e), never 0
  int flip;                 // -1: q changes sign (scale < 0), 1: q counts as 0 (scale 0)
  int causal;
  // plan
  int shared;               // prefix rows stacked over the entries, then joined
  int waves, prefix_waves;  // that split a workgroup's keys: 1 (none) or 4
  int splits, prefix_splits;
  int chunk;                // shared: own keys of a split (a multiple of 128)
  float* part;              // [slots][Hk][B*Sq*G][D] partial outputs
  float* part_lse;          // [slots][Hk][B*Sq*G], log2; null: written directly
};
// Fills the plan for `cus` compute units and returns the workspace bytes it
// takes; with a smaller workspace the plan has to be made with allowed = false.
long long attn_plan(AttnArgs* a, int dtype, int cus, bool allowed);
libconv_status attn_launch(AttnArgs a, int dtype, hipStream_t stream);

// libconv_lora_linear; strides in bytes.
struct LoraArgs {
  const char *x, *w, *a, *b;
  const void* bias;
  const float* scales;
  const int *starts, *adapters;
  char* y;
  int T, K, N, rank, n_adapters, n_requests;  // n_adapters 0: no low-rank term
  long long x_row, y_row;
  unsigned char* low;       // [T][low_width] low-rank values, 4 bytes each
  int* adapter_of;          // [T]
  int low_width;
  // not too many rows: sums of runs of the sum's axis [splits][T][N up to 64s],
  // the runs' bytes and the tile they are formed in; splits 0 otherwise
  float* part;
  int splits, run, tile;
  long long part_at;        // where `part` begins in the workspace
};
// Fills the plan, and returns the workspace bytes it takes.
long long lora_plan(LoraArgs* a, int dtype, int cus);
libconv_status lora_launch(LoraArgs a, int dtype, int cus, hipStream_t stream);

}  // namespace libconv
