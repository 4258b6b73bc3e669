// lora.hip -- a projection shared by all rows with a low-rank adapter for
// each request beside it.
//
//   y[t] = W x[t] + bias + s_a B_a (A_a x[t])
//
// Two launches.  The first finds each row's adapter and forms the low-rank
// values s_a A_a x[t] in fp32 (for 32 rows: adapter by adapter, each lane
// keeping the result of its own row's; the sum's axis is split over the waves
// of a workgroup, so that nothing is left to add up).  The second is the
// projection; a workgroup starts its sums with the low-rank term of its tile,
// so y is written once.  The low-rank values of 16-bit types enter the matrix
// instructions as two bfloat16 numbers, high and low part (16 significant
// bits): one would round the low-rank term to 8 bits before the sum.  fp16
// adapters are split the same way (three products), because a low-rank value
// may be past fp16's range where y is not.
//
// The projection is formed transposed (outputs n on the rows of the matrix
// instructions, tokens on their columns), so that a lane holds 4 consecutive
// outputs of one token.  Both operands have their sums' axis dense: a stage
// is 128 bytes of it, copied straight into LDS, double-buffered.  Up to 64
// rows are bound by reading W once: a workgroup takes 16 outputs and its 8
// waves split the sum's axis, reading W and x straight into registers.
#include "device_common.h"
#include "layer.h"

namespace libconv {
namespace {

constexpr int kLowRows = 32;      // rows of a workgroup of the first launch
constexpr int kFewRows = 64;      // up to which W is read once, and bounds the call

__device__ __forceinline__ u32x4_t load16(__amdgpu_buffer_rsrc_t r, int off) {
  return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}

// Low-rank value r of a row, at the row's values.
template <int DT>
__device__ __forceinline__ void store_low(const LoraArgs& a, unsigned char* at, int r, float v) {
  if constexpr (DT == DT_F32) {
    reinterpret_cast<float*>(at)[r] = v;
  } else {
    const uint16_t hi = Elem<DT_BF16>::from_f32(v);
    const float rest = v - Elem<DT_BF16>::bits_to_f32(hi);
    reinterpret_cast<uint16_t*>(at)[r] = hi;
    reinterpret_cast<uint16_t*>(at)[a.low_width + r] = Elem<DT_BF16>::from_f32(rest);
  }
}

// The first launch.  Writes, for every row t, adapter_of[t] (-1: none) and,
// for rows that have one, width values from low + 4 width t on: fp32 ones, or
// (16-bit types) width high bfloat16 parts and then width low parts.  Values
// from the rank on are 0.  Grid: row tiles x shares of the adapters of a tile
// (with few rows there are as many adapters as rows, and few tiles) x 32 of
// the rank.
template <int DT, int NW>
__global__ __launch_bounds__(64 * NW) void low_kernel(const LoraArgs a) {
  constexpr int EB = Elem<DT>::bytes;
  constexpr int THREADS = 64 * NW;
  __shared__ int ad_of[kLowRows];
  __shared__ float red[NW][32][33];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int l32 = lane & 31, half = lane >> 5;
  const int row0 = blockIdx.x * kLowRows, r0 = blockIdx.z * 32;

  // threads take requests in turn and write the rows they have in the tile
  if (threadIdx.x < kLowRows) ad_of[threadIdx.x] = -1;
  lds_barrier();
  for (int r = threadIdx.x; r < a.n_requests; r += THREADS) {
    const int ad = a.adapters[r], s0 = a.starts[r], s1 = a.starts[r + 1];
    if (ad < 0 || ad >= a.n_adapters) continue;
    const int lo = s0 > row0 ? s0 : row0, hi = s1 < row0 + kLowRows ? s1 : row0 + kLowRows;
    for (int t = lo; t < hi; ++t) ad_of[t - row0] = ad;
  }
  lds_barrier();
  const bool row_ok = row0 + l32 < a.T;
  const int mine = row_ok ? ad_of[l32] : -1;
  if (blockIdx.y == 0 && blockIdx.z == 0 && wave == 0 && half == 0 && row_ok)
    a.adapter_of[row0 + l32] = mine;

  const int row_bytes = a.K * EB;
  const int steps = (row_bytes + 31) / 32;
  const int k0 = (int)((long long)steps * wave / NW);
  const int k1 = (int)((long long)steps * (wave + 1) / NW);
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.x + (long long)row0 * a.x_row, 0x7ffffff0u);
  const int x_off = l32 * (int)a.x_row, a_off = l32 * row_bytes;
  const bool rank_ok = r0 + l32 < a.rank;

  float16_t res = {};
  bool kept = false;   // this lane's row is this workgroup's to write
  uint64_t left = __ballot(mine >= 0);
  for (int turn = 0; left; ++turn) {
    const int ad = __builtin_amdgcn_readlane(mine, __builtin_ctzll(left));
    left &= ~__ballot(mine == ad);
    if (turn % gridDim.y != blockIdx.y) continue;
    const __amdgpu_buffer_rsrc_t ra =
        make_rsrc(a.a + ((long long)ad * a.rank + r0) * row_bytes, 0x7ffffff0u);
    float16_t acc = {};
    constexpr int U = 8;
    for (int k = k0; k < k1; k += U) {
      u32x4_t xf[U], af[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int off = (k + u) * 32 + half * 16;
        const bool in = k + u < k1 && off < row_bytes;
        xf[u] = load16(rx, guard_offset(in && row_ok, x_off + off));
        af[u] = load16(ra, guard_offset(in && rank_ok, a_off + off));
      }
      __builtin_amdgcn_sched_barrier(0);   // all of a batch's reads in flight together
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < Mma<DT>::KSUB; ++e) Mma<DT>::step(af[u], xf[u], acc, e);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) res[i] = mine == ad ? acc[i] : res[i];
    kept = kept || mine == ad;
  }
  const uint64_t rows = __ballot(kept);   // the same in all waves
  if (rows == 0) return;
#pragma unroll
  for (int i = 0; i < 16; ++i) red[wave][l32][(i & 3) + 8 * (i >> 2) + 4 * half] = res[i];
  lds_barrier();
  for (int i = threadIdx.x; i < 32 * 32; i += THREADS) {
    const int t = i >> 5, r = i & 31;
    if (!(rows >> t & 1)) continue;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) v += red[w][t][r];
    v *= a.scales[ad_of[t]];
    store_low<DT>(a, a.low + (long long)(row0 + t) * a.low_width * 4, r0 + r, v);
  }
}

// 16 bytes of row t's low-rank values (and of their low parts), 0 where the
// row is not one of adapter ad's.
template <int DT>
__device__ __forceinline__ void load_low(const LoraArgs& a, __amdgpu_buffer_rsrc_t rl, int t,
                                         bool ok, int off, u32x4_t* hi, u32x4_t* lo) {
  const int at = t * a.low_width * 4 + off;
  *hi = load16(rl, guard_offset(ok, at));
  if constexpr (DT == DT_F32) *lo = u32x4_t{0, 0, 0, 0};
  else *lo = load16(rl, guard_offset(ok, at + a.low_width * 2));
}

// 16 bytes of row n of adapter ad's B, from component r on; 0 past the rank.
template <int DT>
__device__ __forceinline__ u32x4_t load_b(const LoraArgs& a, __amdgpu_buffer_rsrc_t rb, int n,
                                          int r) {
  constexpr int EB = Elem<DT>::bytes, E = 16 / EB;
  const bool ok = n < a.N;
  const int at = (n * a.rank + r) * EB;
  if (a.rank % E == 0) return load16(rb, guard_offset(ok && r < a.rank, at));
  u32x4_t v = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const uint32_t x = Elem<DT>::load_bits(rb, guard_offset(ok && r + e < a.rank, at + e * EB));
    v[e * EB / 4] |= EB == 4 ? x : (x & 0xffffu) << (16 * (e & 1));
  }
  return v;
}

// 8 fp16 values as a high and a low bfloat16 part (8 + 8 bits hold all 11).
__device__ __forceinline__ void split_f16(const u32x4_t& v, u32x4_t* hi, u32x4_t* lo) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float x0 = Elem<DT_F16>::bits_to_f32(v[j] & 0xffffu);
    const float x1 = Elem<DT_F16>::bits_to_f32(v[j] >> 16);
    const uint32_t h0 = Elem<DT_BF16>::from_f32(x0), h1 = Elem<DT_BF16>::from_f32(x1);
    (*hi)[j] = h0 | (h1 << 16);
    const uint32_t l0 = Elem<DT_BF16>::from_f32(x0 - Elem<DT_BF16>::bits_to_f32(h0));
    const uint32_t l1 = Elem<DT_BF16>::from_f32(x1 - Elem<DT_BF16>::bits_to_f32(h1));
    (*lo)[j] = l0 | (l1 << 16);
  }
}

// The matrix instructions of a tile: 32 outputs x 32 tokens, 32 bytes of the
// sums' axis a step (Big), or 16 x 16 and 64 bytes.
template <int DT, bool Big> struct Step;
template <int DT> struct Step<DT, true> {
  using Acc = float16_t;
  __device__ static __forceinline__ void run(const u32x4_t& w, const u32x4_t& x, Acc& c) {
#pragma unroll
    for (int e = 0; e < Mma<DT>::KSUB; ++e) Mma<DT>::step(w, x, c, e);
  }
};
template <int DT> struct Step<DT, false> {
  using Acc = float4_t;
  __device__ static __forceinline__ void run(const u32x4_t& w, const u32x4_t& x, Acc& c) {
    if constexpr (DT == DT_F32) {
      const float4_t wf = __builtin_bit_cast(float4_t, w), xf = __builtin_bit_cast(float4_t, x);
#pragma unroll
      for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(wf[e], xf[e], c, 0, 0, 0);
    } else if constexpr (DT == DT_F16) {
      c = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, w),
                                                 __builtin_bit_cast(half8_t, x), c, 0, 0, 0);
    } else {
      c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, w),
                                                  __builtin_bit_cast(bf16x8_t, x), c, 0, 0, 0);
    }
  }
};

// One step of the low-rank term: bf holds B, hi and lo the low-rank values
// (for fp32, hi is the value itself).
template <int DT, bool Big>
__device__ __forceinline__ void low_step(const u32x4_t& bf, const u32x4_t& hi, const u32x4_t& lo,
                                         typename Step<DT, Big>::Acc& c) {
  if constexpr (DT == DT_F32) {
    Step<DT, Big>::run(bf, hi, c);
  } else if constexpr (DT == DT_BF16) {
    Step<DT, Big>::run(bf, hi, c);
    Step<DT, Big>::run(bf, lo, c);
  } else {
    u32x4_t bh, bl;
    split_f16(bf, &bh, &bl);
    Step<DT_BF16, Big>::run(bh, hi, c);
    Step<DT_BF16, Big>::run(bh, lo, c);
    Step<DT_BF16, Big>::run(bl, hi, c);
  }
}

// 4 consecutive outputs of a token.
template <int DT>
__device__ __forceinline__ void store4(const LoraArgs& a, int t, int n, const float* v) {
  constexpr int EB = Elem<DT>::bytes;
  float o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    o[j] = v[j];
    if (a.bias && n + j < a.N) {
      if constexpr (DT == DT_F32)
        o[j] += static_cast<const float*>(a.bias)[n + j];
      else
        o[j] += Elem<DT>::bits_to_f32(static_cast<const uint16_t*>(a.bias)[n + j]);
    }
  }
  char* at = a.y + t * a.y_row + (long long)n * EB;
  if (n + 4 <= a.N && (reinterpret_cast<uintptr_t>(at) & (4 * EB - 1)) == 0) {
    if constexpr (DT == DT_F32)
      *reinterpret_cast<float4_t*>(at) = float4_t{o[0], o[1], o[2], o[3]};
    else
      *reinterpret_cast<u32x2_t*>(at) =
          u32x2_t{(uint32_t)Elem<DT>::from_f32(o[0]) | ((uint32_t)Elem<DT>::from_f32(o[1]) << 16),
                  (uint32_t)Elem<DT>::from_f32(o[2]) | ((uint32_t)Elem<DT>::from_f32(o[3]) << 16)};
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (n + j < a.N) {
      if constexpr (DT == DT_F32) reinterpret_cast<float*>(at)[j] = o[j];
      else reinterpret_cast<uint16_t*>(at)[j] = Elem<DT>::from_f32(o[j]);
    }
}

// Position of the 16-byte chunk c of a 128-byte row in LDS: the 16 lanes that
// read one chunk of 16 rows at a time hit all banks.
__device__ __forceinline__ int chunk_at(int row, int c) { return c ^ ((row >> 1) & 7); }

// Many rows: BM tokens x BN outputs, WM x WN waves.
template <int DT, int BM, int BN, int WM, int WN, int NS>
__global__ __launch_bounds__(64 * WM * WN) void tile_kernel(const LoraArgs a, int tiles_m,
                                                            int tiles_n) {
  constexpr int EB = Elem<DT>::bytes;
  constexpr int THREADS = 64 * WM * WN;
  constexpr int MB = BM / WM / 32, NB = BN / WN / 32;   // 32 x 32 blocks of a wave
  constexpr int STAGE = (BM + BN) * 128;
  __shared__ __attribute__((aligned(1024))) unsigned char lds[NS * STAGE];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int l32 = lane & 31, half = lane >> 5;
  const int wm = wave % WM, wn = wave / WM;

  // workgroups of one XCD follow one another over a band of 4 tiles of
  // outputs, so that its L2 holds the x and W tiles they share
  const int n_tiles = tiles_m * tiles_n;
  const int per = n_tiles >> 3, more = n_tiles & 7, xcd = blockIdx.x & 7;
  const int id = xcd * per + (xcd < more ? xcd : more) + (blockIdx.x >> 3);
  constexpr int BAND = 4;
  const int band = id / (BAND * tiles_m), in_band = id - band * BAND * tiles_m;
  const int width_n = tiles_n - band * BAND < BAND ? tiles_n - band * BAND : BAND;
  const int m0 = in_band / width_n * BM;
  const int n0 = (band * BAND + in_band % width_n) * BN;

  float16_t acc[NB][MB];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < MB; ++j) acc[i][j] = float16_t{};

  // stages
  const int row_bytes = a.K * EB;
  const int stages = (row_bytes + 127) / 128;
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.x + (long long)m0 * a.x_row, 0x7ffffff0u);
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(a.w + (long long)n0 * row_bytes, 0x7ffffff0u);
  constexpr int CX = BM * 8 / THREADS, CW = BN * 8 / THREADS;   // copies a thread
  int x_off[CX], w_off[CW];   // of stage 0; past the end where the row is
  int x_chunk[CX], w_chunk[CW];
#pragma unroll
  for (int c = 0; c < CX; ++c) {
    const int unit = c * THREADS + threadIdx.x, row = unit >> 3;
    x_chunk[c] = chunk_at(row, unit & 7) * 16;
    x_off[c] = m0 + row < a.T ? row * (int)a.x_row + x_chunk[c] : kOobOffset;
  }
#pragma unroll
  for (int c = 0; c < CW; ++c) {
    const int unit = c * THREADS + threadIdx.x, row = unit >> 3;
    w_chunk[c] = chunk_at(row, unit & 7) * 16;
    w_off[c] = n0 + row < a.N ? row * row_bytes + w_chunk[c] : kOobOffset;
  }
#define LIBCONV_COPY_STAGE(st, at)                                                              \
  {                                                                                             \
    unsigned char* to = lds + (at) * STAGE;                                                     \
    const int k = (st) * 128;                                                                   \
    _Pragma("unroll") for (int c = 0; c < CX; ++c) copy16_to_lds(                               \
        rx, to + (c * THREADS + wave * 64) * 16,                                                \
        guard_offset(x_off[c] >= 0 && k + x_chunk[c] < row_bytes, x_off[c] + k));               \
    _Pragma("unroll") for (int c = 0; c < CW; ++c) copy16_to_lds(                               \
        rw, to + BM * 128 + (c * THREADS + wave * 64) * 16,                                     \
        guard_offset(w_off[c] >= 0 && k + w_chunk[c] < row_bytes, w_off[c] + k));               \
  }
  // NS - 1 stages are on their way at a time; those past the last read nothing
#pragma unroll
  for (int st = 0; st < NS - 1; ++st) LIBCONV_COPY_STAGE(st, st)

  if (a.n_adapters > 0) {
    constexpr int LB = DT == DT_F32 ? 4 : 2;   // bytes of a low-rank value
    const __amdgpu_buffer_rsrc_t rl =
        make_rsrc(a.low + (long long)m0 * a.low_width * 4, 0x7ffffff0u);
#pragma unroll
    for (int j = 0; j < MB; ++j) {
      const int t = (wm * MB + j) * 32 + l32;
      const int mine = m0 + t < a.T ? a.adapter_of[m0 + t] : -1;
      uint64_t left = __ballot(mine >= 0);
      while (left) {
        const int ad = __builtin_amdgcn_readlane(mine, __builtin_ctzll(left));
        left &= ~__ballot(mine == ad);
        const __amdgpu_buffer_rsrc_t rb =
            make_rsrc(a.b + (long long)ad * a.N * a.rank * EB, 0x7ffffff0u);
        const int steps = (a.rank * LB + 31) / 32;
        for (int s = 0; s < steps; s += 2) {   // two steps' reads together
          u32x4_t hi[2], lo[2], bf[2][NB];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int off = (s + u) * 32 + half * 16;
            load_low<DT>(a, rl, t, mine == ad && s + u < steps, off, &hi[u], &lo[u]);
#pragma unroll
            for (int i = 0; i < NB; ++i)
              bf[u][i] = load_b<DT>(a, rb, n0 + (wn * NB + i) * 32 + l32, off / LB);
          }
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < NB; ++i) low_step<DT, true>(bf[u][i], hi[u], lo[u], acc[i][j]);
        }
      }
    }
  }

  int at = 0, free = NS - 1;   // stages in use and to be filled
  for (int st = 0; st < stages; ++st) {
    wait_vmcnt<(NS - 2) * (CX + CW)>();
    lds_barrier();
    LIBCONV_COPY_STAGE(st + NS - 1, free)
    const unsigned char* xs = lds + at * STAGE;
    free = at;
    at = at + 1 < NS ? at + 1 : 0;
    const unsigned char* ws = xs + BM * 128;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      u32x4_t wf[NB], xf[MB];
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const int row = (wn * NB + i) * 32 + l32;
        wf[i] = *reinterpret_cast<const u32x4_t*>(ws + row * 128 + chunk_at(row, 2 * k + half) * 16);
      }
#pragma unroll
      for (int j = 0; j < MB; ++j) {
        const int row = (wm * MB + j) * 32 + l32;
        xf[j] = *reinterpret_cast<const u32x4_t*>(xs + row * 128 + chunk_at(row, 2 * k + half) * 16);
      }
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = 0; j < MB; ++j) Step<DT, true>::run(wf[i], xf[j], acc[i][j]);
    }
  }
#undef LIBCONV_COPY_STAGE

#pragma unroll
  for (int j = 0; j < MB; ++j) {
    const int t = m0 + (wm * MB + j) * 32 + l32;
    if (t >= a.T) continue;
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int n = n0 + (wn * NB + i) * 32 + 8 * r + 4 * half;
        const float v[4] = {acc[i][j][4 * r], acc[i][j][4 * r + 1], acc[i][j][4 * r + 2],
                            acc[i][j][4 * r + 3]};
        if (n < a.N) store4<DT>(a, t, n, v);
      }
  }
}

// Up to 16 * RB rows without adapters: 16 outputs a workgroup, the sum's axis
// split over 8 waves, joined in the order of the waves.
constexpr int kFewWaves = 8;
template <int DT, int RB>
__global__ __launch_bounds__(64 * kFewWaves, 2) void few_kernel(const LoraArgs a) {
  constexpr int EB = Elem<DT>::bytes;
  constexpr int THREADS = 64 * kFewWaves, ROWS = 16 * RB;
  __shared__ __attribute__((aligned(16))) float join[kFewWaves * ROWS * 20];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int l16 = lane & 15, quarter = lane >> 4;
  const int n0 = blockIdx.x * 16;

  const int row_bytes = a.K * EB;
  const int steps = (row_bytes + 63) / 64;
  const int k0 = steps * wave / kFewWaves, k1 = steps * (wave + 1) / kFewWaves;
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.x, 0x7ffffff0u);
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(a.w + (long long)n0 * row_bytes, 0x7ffffff0u);
  const bool n_ok = n0 + l16 < a.N;
  // W is what the call reads from memory: 16 steps of it are on their way at
  // a time, the first before anything else is waited for; x comes from L2, a
  // group of 4 steps ahead
  constexpr int U = 4, AHEAD = 4;
  const int groups = (k1 - k0 + U - 1) / U;
  u32x4_t wf[AHEAD][U], xf[2][U][RB];
  auto fetch_w = [&](int g, u32x4_t* w) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + g * U + u, off = k * 64 + quarter * 16;
      w[u] = load16(rw, guard_offset(n_ok && k < k1 && off < row_bytes, l16 * row_bytes + off));
    }
  };
  auto fetch_x = [&](int g, u32x4_t (*x)[RB]) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < RB; ++j) {
        const int k = k0 + g * U + u, off = k * 64 + quarter * 16;
        x[u][j] = load16(rx, guard_offset(k < k1 && off < row_bytes && j * 16 + l16 < a.T,
                                          (j * 16 + l16) * (int)a.x_row + off));
      }
  };
#pragma unroll
  for (int g = 0; g < AHEAD; ++g) fetch_w(g, wf[g]);
  fetch_x(0, xf[0]);

  __builtin_amdgcn_sched_barrier(0);

  float4_t acc[RB];
#pragma unroll
  for (int j = 0; j < RB; ++j) acc[j] = float4_t{0, 0, 0, 0};
  for (int g0 = 0; g0 < groups; g0 += AHEAD) {
#pragma unroll
    for (int v = 0; v < AHEAD; ++v) {
      if (g0 + v >= groups) break;
      fetch_x(g0 + v + 1, xf[(v + 1) & 1]);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < RB; ++j) Step<DT, false>::run(wf[v][u], xf[v & 1][u][j], acc[j]);
      __builtin_amdgcn_sched_barrier(0);
      if (g0 + AHEAD < groups) fetch_w(g0 + v + AHEAD, wf[v]);
    }
  }

  // [wave][token][output], 20 floats a token: writes and reads without conflicts
#pragma unroll
  for (int j = 0; j < RB; ++j)
    *reinterpret_cast<float4_t*>(join + ((wave * ROWS + j * 16 + l16) * 20 + quarter * 4)) = acc[j];
  lds_barrier();
  for (int i = threadIdx.x; i < ROWS * 4; i += THREADS) {
    const int t = i >> 2, q = i & 3;
    float v[4] = {0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < kFewWaves; ++w) {
      const float4_t p = *reinterpret_cast<const float4_t*>(join + ((w * ROWS + t) * 20 + q * 4));
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] += p[j];
    }
    if (t < a.T && n0 + q * 4 < a.N) store4<DT>(a, t, n0 + q * 4, v);
  }
}

// Up to 64 rows with adapters, in two launches: the shared product in runs of
// the sum's axis beside the low-rank values, then the sum of all.

// Low-rank values r0 .. r0 + 15 of row t (fp32) and the row's adapter: 16 bytes
// of x and of each row of A a lane, dense reads that are all on their way at
// once.
template <int DT>
__device__ __forceinline__ void low_row(const LoraArgs& a, int t, int r0, unsigned char* lds) {
  constexpr int E = 16 / Elem<DT>::bytes, R = 16, THREADS = 256;
  int* found = reinterpret_cast<int*>(lds);
  float* red = reinterpret_cast<float*>(lds + 16);   // [4][R]
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int row_bytes = a.K * Elem<DT>::bytes;
  if (threadIdx.x == 0) *found = -1;
  lds_barrier();
  for (int r = threadIdx.x; r < a.n_requests; r += THREADS) {
    const int ad = a.adapters[r], s0 = a.starts[r], s1 = a.starts[r + 1];
    if (s0 <= t && t < s1 && ad >= 0 && ad < a.n_adapters) *found = ad;
  }
  lds_barrier();
  const int ad = __builtin_amdgcn_readfirstlane(*found);
  if (r0 == 0 && threadIdx.x == 0) a.adapter_of[t] = ad;
  if (ad < 0) return;
  const float scale = a.scales[ad];
  const int ranks = a.rank - r0 < R ? a.rank - r0 : R;   // <= 0: padding, zeros
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.x + t * a.x_row, row_bytes);
  const __amdgpu_buffer_rsrc_t ra =
      make_rsrc(a.a + ((long long)ad * a.rank + (ranks > 0 ? r0 : 0)) * row_bytes,
                ranks > 0 ? (uint32_t)(ranks * row_bytes) : 0u);
  float sum[R] = {};
  for (int off = threadIdx.x * 16; off < row_bytes; off += THREADS * 16) {
    const u32x4_t xv = load16(rx, off);
    u32x4_t av[R];
#pragma unroll
    for (int r = 0; r < R; ++r) av[r] = load16(ra, r * row_bytes + off);
    __builtin_amdgcn_sched_barrier(0);
    float x[E];
    unpack<DT>(xv, x);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float w[E];
      unpack<DT>(av[r], w);
#pragma unroll
      for (int e = 0; e < E; ++e) sum[r] = fmaf(x[e], w[e], sum[r]);
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) sum[r] += __shfl_xor(sum[r], m);
  if (lane == 0)
#pragma unroll
    for (int r = 0; r < R; ++r) red[wave * R + r] = sum[r];
  lds_barrier();
  if (threadIdx.x < R) {
    const int r = threadIdx.x;
    const float v = red[r] + red[R + r] + red[2 * R + r] + red[3 * R + r];
    reinterpret_cast<float*>(a.low)[(long long)t * a.low_width + r0 + r] = v * scale;
  }
}

// Four waves take 16 outputs each and a run of the sum's axis: x arrives in
// LDS, W straight in registers (each of its values has one reader), all of a
// run on its way at once.  The first `low_jobs` workgroups take the low-rank
// values meanwhile.
constexpr int kRun = 1024;   // bytes of a run, at most
template <int DT, int RB>
__global__ __launch_bounds__(256, 2) void run_kernel(const LoraArgs a, int low_jobs) {
  constexpr int EB = Elem<DT>::bytes, ROWS = 16 * RB, STEPS = kRun / 64;
  __shared__ __attribute__((aligned(1024))) unsigned char lds[ROWS * kRun];
  if ((int)blockIdx.x < low_jobs) {
    low_row<DT>(a, (int)blockIdx.x % a.T, (int)blockIdx.x / a.T * 16, lds);
    return;
  }
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int l16 = lane & 15, quarter = lane >> 4;
  const int id = blockIdx.x - low_jobs;
  const int split = id % a.splits, n0 = id / a.splits * 64 + wave * 16;
  const int row_bytes = a.K * EB;
  const int c0 = split * a.run, c1 = c0 + a.run < row_bytes ? c0 + a.run : row_bytes;
  const int stages = (c1 - c0 + 127) / 128;
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.x, 0x7ffffff0u);
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(a.w + (long long)n0 * row_bytes, 0x7ffffff0u);
  // x: 128 bytes of all rows after 128 bytes of all rows
#pragma unroll
  for (int j = 0; j < ROWS * kRun / 16 / 256; ++j) {
    const int unit = j * 256 + threadIdx.x;
    const int row = unit / 8 % ROWS;
    const int off = c0 + unit / (ROWS * 8) * 128 + chunk_at(row, unit & 7) * 16;
    if (j * 256 < stages * ROWS * 8)
      copy16_to_lds(rx, lds + (j * 256 + wave * 64) * 16,
                    guard_offset(row < a.T && off < c1, row * (int)a.x_row + off));
  }
  u32x4_t wf[STEPS];
#pragma unroll
  for (int k = 0; k < STEPS; ++k) {
    const int off = c0 + k * 64 + quarter * 16;
    wf[k] = load16(rw, guard_offset(n0 + l16 < a.N && off < c1, l16 * row_bytes + off));
  }
  __builtin_amdgcn_sched_barrier(0);
  wait_vmcnt<STEPS>();
  lds_barrier();
  float4_t acc[RB];
#pragma unroll
  for (int j = 0; j < RB; ++j) acc[j] = float4_t{0, 0, 0, 0};
#pragma unroll
  for (int k = 0; k < STEPS; ++k) {
    if (k * 64 < c1 - c0) {
#pragma unroll
      for (int j = 0; j < RB; ++j) {
        const int row = j * 16 + l16;
        const u32x4_t xf = *reinterpret_cast<const u32x4_t*>(
            lds + (k / 2 * ROWS + row) * 128 + chunk_at(row, (k & 1) * 4 + quarter) * 16);
        Step<DT, false>::run(wf[k], xf, acc[j]);
      }
    }
  }
  const long long n_pad = (a.N + 63) / 64 * 64;
#pragma unroll
  for (int j = 0; j < RB; ++j) {
    const int t = j * 16 + l16;
    if (t < a.T)
      *reinterpret_cast<float4_t*>(a.part + ((long long)split * a.T + t) * n_pad + n0 +
                                   quarter * 4) = acc[j];
  }
}

// y of row blockIdx.y: the runs in their order, the bias, the low-rank term.
template <int DT>
__global__ __launch_bounds__(256) void sum_kernel(const LoraArgs a) {
  constexpr int EB = Elem<DT>::bytes, E = 16 / EB;
  const int n = blockIdx.x * 256 + threadIdx.x, t = blockIdx.y;
  if (n >= a.N) return;
  const int ad = __builtin_amdgcn_readfirstlane(a.adapter_of[t]);
  const long long n_pad = (a.N + 63) / 64 * 64;
  const float* part = a.part + t * n_pad + n;
  float v = 0.0f;
  for (int s = 0; s < a.splits; s += 8) {
    float p[8];
#pragma unroll
    for (int u = 0; u < 8; ++u)
      p[u] = s + u < a.splits ? part[(long long)(s + u) * a.T * n_pad] : 0.0f;
#pragma unroll
    for (int u = 0; u < 8; ++u) v += p[u];
  }
  if (a.bias) {
    if constexpr (DT == DT_F32) v += static_cast<const float*>(a.bias)[n];
    else v += Elem<DT>::bits_to_f32(static_cast<const uint16_t*>(a.bias)[n]);
  }
  if (ad >= 0) {
    const char* b = a.b + ((long long)ad * a.N + n) * a.rank * EB;
    const float* low = reinterpret_cast<const float*>(a.low) + (long long)t * a.low_width;
    if (a.rank % E == 0) {
      for (int r = 0; r < a.rank; r += E) {
        float w[E];
        unpack<DT>(*reinterpret_cast<const u32x4_t*>(b + r * EB), w);
#pragma unroll
        for (int e = 0; e < E; ++e) v = fmaf(low[r + e], w[e], v);
      }
    } else {
      for (int r = 0; r < a.rank; ++r) {
        float w;
        if constexpr (DT == DT_F32) w = reinterpret_cast<const float*>(b)[r];
        else w = Elem<DT>::bits_to_f32(reinterpret_cast<const uint16_t*>(b)[r]);
        v = fmaf(low[r], w, v);
      }
    }
  }
  char* y = a.y + t * a.y_row + (long long)n * EB;
  if constexpr (DT == DT_F32) *reinterpret_cast<float*>(y) = v;
  else *reinterpret_cast<uint16_t*>(y) = Elem<DT>::from_f32(v);
}

template <int DT>
void launch_runs(const LoraArgs& a, hipStream_t stream) {
  const int low_jobs = a.T * ((a.rank + 15) / 16);
  const dim3 grid((unsigned)(low_jobs + (a.N + 63) / 64 * a.splits)), threads(256);
  if (a.T <= 16)
    hipLaunchKernelGGL((run_kernel<DT, 1>), grid, threads, 0, stream, a, low_jobs);
  else if (a.T <= 32)
    hipLaunchKernelGGL((run_kernel<DT, 2>), grid, threads, 0, stream, a, low_jobs);
  else
    hipLaunchKernelGGL((run_kernel<DT, 4>), grid, threads, 0, stream, a, low_jobs);
  hipLaunchKernelGGL((sum_kernel<DT>), dim3((unsigned)((a.N + 255) / 256), (unsigned)a.T), threads,
                     0, stream, a);
}

template <int DT, int BM, int BN, int WM, int WN, int NS>
void launch_tile(const LoraArgs& a, hipStream_t stream) {
  const int tm = (a.T + BM - 1) / BM, tn = (a.N + BN - 1) / BN;
  hipLaunchKernelGGL((tile_kernel<DT, BM, BN, WM, WN, NS>), dim3((unsigned)(tm * tn)),
                     dim3(64 * WM * WN), 0, stream, a, tm, tn);
}

// Time of a launch in units of one 256 x 256 tile: rounds of workgroups over
// the compute units, each as long as its workgroups together on one unit.
double tile_cost(const LoraArgs& a, int cus, int bm, int bn, int per_cu, double speed) {
  const double tiles = (double)((a.T + bm - 1) / bm) * ((a.N + bn - 1) / bn);
  const double rounds = (double)(long long)((tiles + (double)cus * per_cu - 1) / (cus * per_cu));
  const double share = tiles < (double)cus * per_cu ? (tiles > cus ? tiles / cus : 1.0) : per_cu;
  return rounds * share * bm * bn / speed;
}

template <int DT>
void launch_dt(const LoraArgs& a, int cus, hipStream_t stream) {
  if (a.n_adapters > 0 && a.T <= kFewRows) {
    launch_runs<DT>(a, stream);
    return;
  }
  if (a.n_adapters > 0) {
    // with few row tiles, 16 waves to one and the tile's adapters dealt out
    const int tiles = (a.T + kLowRows - 1) / kLowRows;
    int shares = cus / tiles;
    const int most = a.n_adapters < kLowRows ? a.n_adapters : kLowRows;
    if (shares > most) shares = most;
    const dim3 grid((unsigned)tiles, (unsigned)(shares < 1 ? 1 : shares),
                    (unsigned)(a.low_width / 32));
    if (tiles < cus)
      hipLaunchKernelGGL((low_kernel<DT, 16>), grid, dim3(64 * 16), 0, stream, a);
    else
      hipLaunchKernelGGL((low_kernel<DT, 8>), grid, dim3(64 * 8), 0, stream, a);
  }
  if (a.T <= kFewRows) {
    const dim3 grid((unsigned)((a.N + 15) / 16)), threads(64 * kFewWaves);
    if (a.T <= 16) hipLaunchKernelGGL((few_kernel<DT, 1>), grid, threads, 0, stream, a);
    else if (a.T <= 32) hipLaunchKernelGGL((few_kernel<DT, 2>), grid, threads, 0, stream, a);
    else hipLaunchKernelGGL((few_kernel<DT, 4>), grid, threads, 0, stream, a);
    return;
  }
  const double c256 = tile_cost(a, cus, 256, 256, 1, 1.0);
  const double c128 = tile_cost(a, cus, 128, 128, 2, 0.75);
  const double c64 = tile_cost(a, cus, 64, 64, 4, 0.4);
  if (c256 <= c128 && c256 <= c64) launch_tile<DT, 256, 256, 4, 2, 2>(a, stream);
  else if (c128 <= c64) launch_tile<DT, 128, 128, 2, 2, 2>(a, stream);
  else launch_tile<DT, 64, 64, 2, 2, 4>(a, stream);
}

}  // namespace

long long lora_plan(LoraArgs* a, int dtype, int cus) {
  a->low_width = a->splits = a->run = 0;
  if (a->n_adapters == 0 || a->T == 0) return 0;
  a->low_width = (a->rank + 31) / 32 * 32;
  const long long low = (long long)a->T * (a->low_width + 1) * 4;
  a->part_at = (low + 255) / 256 * 256;
  if (a->T > kFewRows) return low;
  // runs of the sum's axis: two workgroups a compute unit if they have 256
  // bytes or more
  const int row_bytes = a->K * (dtype == LIBCONV_F32 ? 4 : 2);
  const int tiles = (a->N + 63) / 64;
  int runs = 2 * cus / tiles;
  if (runs > row_bytes / 256) runs = row_bytes / 256;
  if (runs < (row_bytes + kRun - 1) / kRun) runs = (row_bytes + kRun - 1) / kRun;
  a->run = ((row_bytes + runs - 1) / runs + 127) / 128 * 128;
  a->splits = (row_bytes + a->run - 1) / a->run;
  return a->part_at + (long long)a->splits * a->T * tiles * 64 * 4;
}

libconv_status lora_launch(LoraArgs a, int dtype, int cus, hipStream_t stream) {
  if (dtype == LIBCONV_F32) launch_dt<DT_F32>(a, cus, stream);
  else if (dtype == LIBCONV_F16) launch_dt<DT_F16>(a, cus, stream);
  else launch_dt<DT_BF16>(a, cus, stream);
  return hipGetLastError() == hipSuccess ? LIBCONV_OK : LIBCONV_ERR_LAUNCH;
}

}  // namespace libconv
