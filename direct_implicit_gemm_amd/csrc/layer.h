// layer.h -- the attention-layer operators' launches, shared by their entry
// points (layer_api.cpp) and their kernels (rope.hip, attention.hip,
// lora.hip, kv_cache.hip, cache_attention.hip, linear.hip).  Not part of the public ABI.
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

// The cache in 8 bits; strides in bytes.
struct CacheView {
  char* codes[2];           // keys, values
  float* scale[2];          // [blocks][Hk]
  long long block[2], token[2], head[2];
  const int* lengths;
  const int* table;         // [B][width]
  int B, blocks, log_block, width, Hk, D;
};
// libconv_kv_cache_write (rows of k and v) and _read (entries' rows).
struct CacheCopyArgs {
  CacheView c;
  char* x[2];               // k, v
  long long entry[2], row[2], head[2];
  const int* starts;        // write
  int T;                    // rows of k and v, or (read) of an entry
};
libconv_status cache_write_launch(const CacheCopyArgs& a, int format, int dtype,
                                  hipStream_t stream);
libconv_status cache_read_launch(const CacheCopyArgs& a, int format, int dtype,
                                 hipStream_t stream);

// libconv_cache_attention; strides in bytes.
struct CacheAttnArgs {
  CacheView c;
  const char* q;
  char* out;
  float* lse;
  const int* starts;
  long long q_r, q_h, o_r, o_h;
  int T, max_rows, G;
  float scale;              // |scale| log2(e), never 0
  int flip;                 // -1: q changes sign (scale < 0), 1: q counts as 0 (scale 0)
  int causal;
  // plan
  int few_groups;           // workgroups that share the keys of entries of few rows;
                            // 0: one to an entry and key head
  int set;                  // rows of a key head of entries of more rows to a workgroup
  int sets;                 // of each entry; 0: side by side
  int units;                // sets in all, with their key heads
  int splits;               // and shares of their keys
  // partial results of the former [2 few_groups][32] and of the latter [splits][units]
  // [set] (rows of no entry take no room), normed: D outputs and the log2 of their sum,
  // each
  float *part, *part_lse, *many, *many_lse;
};
// Fills the plan for `cus` compute units and returns the workspace bytes it
// takes; with a smaller workspace the plan has to be made with allowed = false.
long long cache_attn_plan(CacheAttnArgs* a, int dtype, int cus, bool allowed);
// Puts the partial results into a workspace of that many bytes.
void cache_attn_place(CacheAttnArgs* a, char* workspace);
libconv_status cache_attn_launch(CacheAttnArgs a, int format, int dtype, hipStream_t stream);

// libconv_linear; strides in bytes.
struct LinearArgs {
  const char *x, *w;
  const void* bias;
  const char* residual;
  char* y;
  int T, K, N, act;
  long long x_row, r_row, y_row;
  // plan: sums of runs of the sum's axis [splits][T][N up to 64s], the runs' bytes
  float* part;
  int splits, run, tile;
  int stages;   // of tiles of 128
};
long long linear_plan(LinearArgs* a, int dtype, int cus, bool allowed);
libconv_status linear_launch(LinearArgs a, int dtype, hipStream_t stream);

}  // namespace libconv
