// lora.hip -- a projection shared by all rows with a low-rank adapter for
// each request beside it.
//
//   y[t] = W x[t] + bias + s_a B_a (A_a x[t])
//
// Two launches, in one of two ways.  Up to about 1000 rows: the first forms the
// product in fp32 (in runs of the sum's axis, if it has too few tiles to fill
// the GPU) and, beside it, the low-rank values s_a A_a x[t]; the second adds
// the runs, the bias and the low-rank term.  Many rows: the first finds each
// row's adapter and forms the low-rank values; the second is the projection,
// whose workgroups start their sums with the low-rank term of their tile, so y
// is written once.  There the low-rank values of 16-bit types enter the matrix
// instructions as two bfloat16 numbers, high and low part (16 significant
// bits): one would round the low-rank term to 8 bits before the sum.  fp16
// adapters are split the same way (three products), because a low-rank value
// may be past fp16's range where y is not.
//
// The projection is formed transposed (outputs n on the rows of the matrix
// instructions, tokens on their columns), so that a lane holds 4 consecutive
// outputs of one token.  Both operands have their sums' axis dense: a stage
// is 128 bytes of it, copied straight into LDS.  Up to 64 rows are bound by
// reading W once.
#include "device_common.h"
#include "layer.h"

namespace libconv {
namespace {

constexpr int kLowRows = 32;      // rows of a workgroup of the first launch
constexpr int kFewRows = 64;      // up to which W is read once, and bounds the call
constexpr int kLowGroup = 4;      // rows that share their reads of A, where more
// Workgroups of 256 lanes of a launch, which holds less than 2^32 lanes (a
// launch's low-rank workgroups come on top).
constexpr long long kMostGroups = (1 << 24) - 4096;

__device__ __forceinline__ u32x4_t load16(__amdgpu_buffer_rsrc_t r, int off) {
  return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}

// Low-rank value r of a row, at the row's values.  The high part is always
// finite: an infinity or a NaN is the low part beside a 0, because fp16 B's low
// part (mostly 0) is multiplied by the high part too, and 0 times an infinity
// would be a NaN.
template <int DT>
__device__ __forceinline__ void store_low(const LoraArgs& a, unsigned char* at, int r, float v) {
  if constexpr (DT == DT_F32) {
    reinterpret_cast<float*>(at)[r] = v;
  } else {
    const bool finite = __builtin_isfinite(v);
    uint16_t hi = Elem<DT_BF16>::from_f32(v);
    // (a value that would be rounded to an infinity keeps the largest number)
    if ((hi & 0x7f80u) == 0x7f80u) hi = finite ? hi - 1 : 0;
    const float rest = finite ? v - Elem<DT_BF16>::bits_to_f32(hi) : v;
    reinterpret_cast<uint16_t*>(at)[r] = hi;
    reinterpret_cast<uint16_t*>(at)[a.low_width + r] = Elem<DT_BF16>::from_f32(rest);
  }
}

// 32 rows of x times 32 rows of another operand: both arrive in LDS 256 bytes
// of the sums' axis at a time, NS - 1 such stages on their way; the four waves
// take 64 bytes of each, so acc holds a quarter of the sums.  off: of this
// thread's copies (rows 16 apart, two of x and two of the other; see
// offsets32).  Chunk c of row r is kept at c ^ (r & 15), so that 16 rows'
// reads of one chunk hit all banks.
constexpr int kStage32 = 64 * 256;
__device__ __forceinline__ int column32() {   // bytes of a thread's chunk in a row
  return ((threadIdx.x & 15) ^ (threadIdx.x >> 4)) * 16;
}
__device__ __forceinline__ void offsets32(int* off, int rows, int stride) {
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int row = c * 16 + (threadIdx.x >> 4);
    off[c] = row < rows ? row * stride + column32() : kOobOffset;
  }
}
template <int DT, int NS>
__device__ __forceinline__ void product32(__amdgpu_buffer_rsrc_t rx, __amdgpu_buffer_rsrc_t rw,
                                          const int* off, int row_bytes, unsigned char* lds,
                                          float16_t& acc) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int l32 = lane & 31, half = lane >> 5;
  const int stages = (row_bytes + 255) / 256, column = column32();
#define LIBCONV_COPY_STAGE(st, at)                                                              \
  {                                                                                             \
    const int k = (st) * 256;                                                                   \
    _Pragma("unroll") for (int c = 0; c < 4; ++c) copy16_to_lds(                                \
        c < 2 ? rx : rw, lds + (at) * kStage32 + (c * 256 + wave * 64) * 16,                    \
        guard_offset(off[c] >= 0 && k + column < row_bytes, off[c] + k));                       \
  }
  // past the last stage they read nothing
#pragma unroll
  for (int st = 0; st < NS - 1; ++st) LIBCONV_COPY_STAGE(st, st)
  for (int st = 0; st < stages; ++st) {
    wait_vmcnt<(NS - 2) * 4>();
    lds_barrier();
    LIBCONV_COPY_STAGE(st + NS - 1, (st + NS - 1) % NS)
    const unsigned char* xs = lds + st % NS * kStage32 + l32 * 256;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int at = ((wave * 4 + u * 2 + half) ^ (l32 & 15)) * 16;
      const u32x4_t xf = *reinterpret_cast<const u32x4_t*>(xs + at);
      const u32x4_t wf = *reinterpret_cast<const u32x4_t*>(xs + 32 * 256 + at);
#pragma unroll
      for (int e = 0; e < Mma<DT>::KSUB; ++e) Mma<DT>::step(wf, xf, acc, e);
    }
  }
#undef LIBCONV_COPY_STAGE
  wait_vmcnt<0>();
}

// The first launch.  Writes, for every row t, adapter_of[t] (-1: none) and,
// for rows that have one, width values from low + 4 width t on: fp32 ones, or
// (16-bit types) width high bfloat16 parts and then width low parts.  Values
// from the rank on are 0.  Grid: row tiles x shares of the adapters of a tile
// x 32 of the rank.  Bound by latency (a stage 0.28 us) and by what a compute
// unit reads of L2: 2167 rows of 1280, rank 64 in 8.6 us, 8192 rows of 4096, rank
// 32 in 24 us (67 MB of x; registers in place of LDS: 34 us).
template <int DT, int NS>
__global__ __launch_bounds__(256, NS <= 4 ? 2 : 1) void low_kernel(const LoraArgs a) {
  constexpr int EB = Elem<DT>::bytes, THREADS = 256;
  // (nothing beside the stages: with 64 KB and a little the workgroup would be
  // alone on its compute unit)
  __shared__ __attribute__((aligned(1024))) unsigned char lds[NS * kStage32];
  int* const ad_of = reinterpret_cast<int*>(lds);   // until the stages fill
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
  lds_barrier();
  if (blockIdx.y == 0 && blockIdx.z == 0 && wave == 0 && half == 0 && row_ok)
    a.adapter_of[row0 + l32] = mine;

  const int row_bytes = a.K * EB;
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.x + (long long)row0 * a.x_row, 0x7ffffff0u);
  int off[4];
  offsets32(off, a.T - row0, (int)a.x_row);
  offsets32(off + 2, a.rank - r0, row_bytes);

  float16_t res = {};
  bool kept = false;   // this lane's row is this workgroup's to write
  uint64_t left = __ballot(mine >= 0);
  for (int turn = 0; left; turn = turn + 1 < (int)gridDim.y ? turn + 1 : 0) {
    const int ad = __builtin_amdgcn_readlane(mine, __builtin_ctzll(left));
    left &= ~__ballot(mine == ad);
    if (turn != (int)blockIdx.y) continue;
    const float scale = a.scales[ad];
    const __amdgpu_buffer_rsrc_t ra =
        make_rsrc(a.a + ((long long)ad * a.rank + r0) * row_bytes, 0x7ffffff0u);
    if (kept) lds_barrier();   // the last adapter's stages are read
    float16_t acc = {};
    product32<DT, NS>(rx, ra, off, row_bytes, lds, acc);
#pragma unroll
    for (int i = 0; i < 16; ++i) res[i] = mine == ad ? acc[i] * scale : res[i];
    kept = true;
  }
  if (!kept) return;   // the same in all waves
  // rows of this workgroup's adapters
  uint64_t rows = 0;
  {
    uint64_t rest = __ballot(mine >= 0);
    for (int turn = 0; rest; turn = turn + 1 < (int)gridDim.y ? turn + 1 : 0) {
      const uint64_t same = __ballot(mine == __builtin_amdgcn_readlane(mine, __builtin_ctzll(rest)));
      rest &= ~same;
      if (turn == (int)blockIdx.y) rows |= same;
    }
  }
  float(*red)[32][33] = reinterpret_cast<float(*)[32][33]>(lds);
  lds_barrier();
#pragma unroll
  for (int i = 0; i < 16; ++i) red[wave][l32][(i & 3) + 8 * (i >> 2) + 4 * half] = res[i];
  lds_barrier();
  for (int i = threadIdx.x; i < 32 * 32; i += THREADS) {
    const int t = i >> 5, r = i & 31;
    // (past the rank, an infinity of x times the 0 that stands for A is no 0)
    if (rows >> t & 1)
      store_low<DT>(a, a.low + (long long)(row0 + t) * a.low_width * 4, r0 + r,
                    r0 + r < a.rank ? red[0][t][r] + red[1][t][r] + red[2][t][r] + red[3][t][r]
                                    : 0.0f);
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

// An infinity or a NaN of B is not for the matrix instructions.  Where tokens of
// several adapters share a block, the others' low-rank values are 0 for an
// adapter's step, and 0 times it would reach them; and of a low-rank value in two
// parts, the low one may be 0 or of the other sign.  drop_not_finite puts 1 with
// its sign in its place (no 0: the low-rank value may itself be an infinity), and
// add_not_finite adds what it gives its own tokens to the written outputs (which
// are not finite then, whatever else they are).
template <int DT>
__device__ __forceinline__ bool drop_not_finite(u32x4_t& v) {
  bool any = false;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t w = v[j];
    if constexpr (DT == DT_F32) {
      const bool bad = (w & 0x7f800000u) == 0x7f800000u;
      w = bad ? (w & 0x80000000u) | 0x3f800000u : w;
      any = any || bad;
    } else {
      constexpr uint32_t E = DT == DT_F16 ? 0x7c00u : 0x7f80u, ONE = DT == DT_F16 ? 0x3c00u : 0x3f80u;
      const bool low = (w & E) == E, high = (w & (E << 16)) == E << 16;
      w = low ? (w & 0xffff8000u) | ONE : w;
      w = high ? (w & 0x8000ffffu) | ONE << 16 : w;
      any = any || low || high;
    }
    v[j] = w;
  }
  return any;
}
// The largest magnitudes so far of a word's values, and whether they are not
// finite: fewer instructions than dropping, which is hardly ever needed.
template <int DT> __device__ __forceinline__ uint32_t largest(uint32_t so_far, uint32_t w) {
  if constexpr (DT == DT_F32) {
    w &= 0x7fffffffu;
    return so_far > w ? so_far : w;
  } else {
    typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(
                                            __builtin_bit_cast(u16x2_t, so_far),
                                            __builtin_bit_cast(u16x2_t, w & 0x7fff7fffu)));
  }
}
template <int DT> __device__ __forceinline__ bool not_finite(uint32_t top) {
  if constexpr (DT == DT_F32) return top >= 0x7f800000u;
  constexpr uint32_t E = DT == DT_F16 ? 0x7c00u : 0x7f80u;
  return (top & 0xffffu) >= E || (top >> 16) >= E;
}
// Output n of token t, written by this lane.
template <int DT>
__device__ __forceinline__ void add_not_finite(const LoraArgs& a, int t, int n) {
  constexpr int EB = Elem<DT>::bytes;
  const int ad = a.adapter_of[t];
  if (ad < 0) return;
  const char* b = a.b + ((long long)ad * a.N + n) * a.rank * EB;
  const unsigned char* low = a.low + (long long)t * a.low_width * 4;
  float extra = 0.0f;
  for (int r = 0; r < a.rank; ++r) {
    float w, v;
    if constexpr (DT == DT_F32) {
      w = reinterpret_cast<const float*>(b)[r];
      v = reinterpret_cast<const float*>(low)[r];
    } else {
      w = Elem<DT>::bits_to_f32(reinterpret_cast<const uint16_t*>(b)[r]);
      v = Elem<DT_BF16>::bits_to_f32(reinterpret_cast<const uint16_t*>(low)[r]) +
          Elem<DT_BF16>::bits_to_f32(reinterpret_cast<const uint16_t*>(low)[a.low_width + r]);
    }
    if (!__builtin_isfinite(w)) extra = fmaf(w, v, extra);
  }
  if (extra == 0.0f) return;
  char* y = a.y + t * a.y_row + (long long)n * EB;
  if constexpr (DT == DT_F32) {
    *reinterpret_cast<float*>(y) += extra;
  } else {
    uint16_t* h = reinterpret_cast<uint16_t*>(y);
    *h = Elem<DT>::from_f32(Elem<DT>::bits_to_f32(*h) + extra);
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

// Fewer rows, in two launches: the shared product in runs of the sum's axis
// beside the low-rank values, then the sum of all (sum_kernel).

// Sums of N values over the wave, N a power of 2: each step halves the values a
// lane keeps, so lane l ends with value l * N / 64.
template <int N, int M = 32>
__device__ __forceinline__ float wave_sum(float* v) {
  if constexpr (M == 0) {
    return v[0];
  } else if constexpr (N == 1) {
    v[0] += __shfl_xor(v[0], M);
  } else {
    const bool upper = (threadIdx.x & M) != 0;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const float keep = upper ? v[i + N / 2] : v[i], give = upper ? v[i] : v[i + N / 2];
      v[i] = keep + __shfl_xor(give, M);
    }
  }
  return wave_sum<(N > 1 ? N / 2 : 1), M / 2>(v);
}

// Low-rank values r0 .. r0 + 15 of RT rows from t0 on (fp32), and the rows'
// adapters: 16 bytes of x and of each row of A a lane, dense reads that are all
// on their way at once.  256 threads.  64 rows of 4096, rank 16, by themselves:
// 7 us (with 32 rows to a workgroup 16 us).
template <int DT, int RT>
__device__ __forceinline__ void low_rows(const LoraArgs& a, int t0, int r0, unsigned char* lds) {
  constexpr int E = 16 / Elem<DT>::bytes, R = 16, THREADS = 256;
  int* found = reinterpret_cast<int*>(lds);
  float* red = reinterpret_cast<float*>(lds + 64);   // [4][RT * R]
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int row_bytes = a.K * Elem<DT>::bytes;
  if (threadIdx.x < RT) found[threadIdx.x] = -1;
  lds_barrier();
  for (int r = threadIdx.x; r < a.n_requests; r += THREADS) {
    const int ad = a.adapters[r], s0 = a.starts[r], s1 = a.starts[r + 1];
    if (ad < 0 || ad >= a.n_adapters) continue;
#pragma unroll
    for (int i = 0; i < RT; ++i)
      if (s0 <= t0 + i && t0 + i < s1) found[i] = ad;
  }
  lds_barrier();
  int of[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
    of[i] = t0 + i < a.T ? __builtin_amdgcn_readfirstlane(found[i]) : -1;
  if (r0 == 0 && threadIdx.x < RT && t0 + (int)threadIdx.x < a.T)
    a.adapter_of[t0 + threadIdx.x] = found[threadIdx.x];
  const int ranks = a.rank - r0 < R ? a.rank - r0 : R;   // <= 0: padding, zeros
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.x + t0 * a.x_row, 0x7ffffff0u);
#pragma unroll
  for (int turn = 0; turn < RT; ++turn) {
    const int ad = of[turn];
    bool first = ad >= 0;   // of the rows with this adapter
#pragma unroll
    for (int i = 0; i < turn; ++i) first = first && of[i] != ad;
    if (!first) continue;
    const float scale = a.scales[ad];
    const __amdgpu_buffer_rsrc_t ra =
        make_rsrc(a.a + ((long long)ad * a.rank + (ranks > 0 ? r0 : 0)) * row_bytes,
                  ranks > 0 ? (uint32_t)(ranks * row_bytes) : 0u);
    float sum[RT * R] = {};
    for (int off = threadIdx.x * 16; off < row_bytes; off += THREADS * 16) {
      u32x4_t xv[RT], av[R];
#pragma unroll
      for (int i = 0; i < RT; ++i)
        xv[i] = load16(rx, guard_offset(of[i] == ad, i * (int)a.x_row + off));
#pragma unroll
      for (int r = 0; r < R; ++r) av[r] = load16(ra, r * row_bytes + off);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float w[E];
        unpack<DT>(av[r], w);
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          float x[E];
          unpack<DT>(xv[i], x);
#pragma unroll
          for (int e = 0; e < E; ++e) sum[i * R + r] = fmaf(x[e], w[e], sum[i * R + r]);
        }
      }
    }
    const float v = wave_sum<RT * R>(sum);
    constexpr int LANES = 64 / (RT * R);
    if (turn > 0) lds_barrier();   // the last sums are read
    if (lane % LANES == 0) red[wave * RT * R + lane / LANES] = v;
    lds_barrier();
    if (threadIdx.x < RT * R) {
      const int i = threadIdx.x;
      if (found[i / R] == ad)
        reinterpret_cast<float*>(a.low)[(long long)(t0 + i / R) * a.low_width + r0 + i % R] =
            (red[i] + red[RT * R + i] + red[2 * RT * R + i] + red[3 * RT * R + i]) * scale;
    }
  }
}

// Tile of the fp32 sums of run `split`, 4 consecutive outputs of a token.
__device__ __forceinline__ void store_part(const LoraArgs& a, int split, int t, int n, float4_t v) {
  const long long n_pad = (a.N + 63) / 64 * 64;
  if (t < a.T && n < n_pad)
    *reinterpret_cast<float4_t*>(a.part + ((long long)split * a.T + t) * n_pad + n) = v;
}

// BM tokens x BN outputs, WM x WN waves, NS stages in LDS or on their way.  Runs: the
// first `low_jobs` workgroups form low-rank values, the others the sums of a
// run of the sum's axis.  Bound by the matrix units in 256 x 256 tiles: 8192
// rows, 4096 -> 8192 in bf16 450-490 us with the low-rank term of rank 32, 437
// without it (1.27 PFLOP/s); in 128 x 128 tiles 2167 rows, 1280 -> 3840 in fp16
// 44 and 29 us.
template <int DT, int BM, int BN, int WM, int WN, int NS, bool Runs>
__global__ __launch_bounds__(64 * WM * WN, 2) void tile_kernel(const LoraArgs a, int tiles_m,
                                                            int tiles_n, int low_jobs) {
  constexpr int EB = Elem<DT>::bytes;
  constexpr int THREADS = 64 * WM * WN;
  constexpr int MB = BM / WM / 32, NB = BN / WN / 32;   // 32 x 32 blocks of a wave
  constexpr int STAGE = (BM + BN) * 128;
  __shared__ __attribute__((aligned(1024))) unsigned char lds[NS * STAGE];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int l32 = lane & 31, half = lane >> 5;
  const int wm = wave % WM, wn = wave / WM;

  int block = blockIdx.x, split = 0;
  if constexpr (Runs) {
    if (block < low_jobs) {
      const int groups = (a.T + kLowGroup - 1) / kLowGroup;
      low_rows<DT, kLowGroup>(a, block % groups * kLowGroup, block / groups * 16, lds);
      return;
    }
    block -= low_jobs;
    split = block / (tiles_m * tiles_n);
    block -= split * tiles_m * tiles_n;
  }
  // workgroups of one XCD follow one another over a band of 4 tiles of
  // outputs, so that its L2 holds the x and W tiles they share
  const int n_tiles = tiles_m * tiles_n;
  const int per = n_tiles >> 3, more = n_tiles & 7, xcd = block & 7;
  const int id = xcd * per + (xcd < more ? xcd : more) + (block >> 3);
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
  const int row = a.K * EB;   // bytes of a row of W
  const int begin = Runs ? split * a.run : 0;
  const int row_bytes = Runs && begin + a.run < row ? a.run : row - begin;   // of this run
  const int stages = (row_bytes + 127) / 128;
  // a thread copies one 16-byte chunk of rows PASS apart: its place in them is
  // the same, and the rows are told apart by a scalar offset.  Rows that do not
  // exist lie past the resource's end.
  constexpr int PASS = THREADS / 8;
  static_assert(PASS % 16 == 0, "one chunk for a thread's rows");
  const int rows_x = a.T - m0 < BM ? a.T - m0 : BM, rows_w = a.N - n0 < BN ? a.N - n0 : BN;
  const int x_row = (int)a.x_row;
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.x + (long long)m0 * a.x_row + begin,
                                              (uint32_t)((rows_x - 1) * x_row + row_bytes));
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(a.w + (long long)n0 * row + begin,
                                              (uint32_t)((rows_w - 1) * row + row_bytes));
  const int chunk = chunk_at(threadIdx.x >> 3, threadIdx.x & 7) * 16;
  const int x_off = (int)(threadIdx.x >> 3) * x_row + chunk;
  const int w_off = (int)(threadIdx.x >> 3) * row + chunk;
  constexpr int CX = BM / PASS, CW = BN / PASS;   // copies a thread
#define LIBCONV_COPY_STAGE(st, at)                                                              \
  {                                                                                             \
    unsigned char* to = lds + (at) * STAGE + wave * 1024;                                       \
    const int k = (st) * 128;                                                                   \
    const bool in = k + chunk < row_bytes;                                                      \
    const int xo = in ? x_off + k : kFarOffset, wo = in ? w_off + k : kFarOffset;               \
    _Pragma("unroll") for (int c = 0; c < CX; ++c)                                              \
        copy16_to_lds(rx, to + c * THREADS * 16, xo, c * PASS * x_row);                         \
    _Pragma("unroll") for (int c = 0; c < CW; ++c)                                              \
        copy16_to_lds(rw, to + BM * 128 + c * THREADS * 16, wo, c * PASS * row);                \
  }
  // NS stages are in LDS or on their way; those past the last read nothing
#pragma unroll
  for (int st = 0; st < NS; ++st) LIBCONV_COPY_STAGE(st, st)

  bool dropped = false;   // values of B that are not finite
  if (!Runs && a.n_adapters > 0) {
    constexpr int LB = DT == DT_F32 ? 4 : 2;   // bytes of a low-rank value
    const __amdgpu_buffer_rsrc_t rl =
        make_rsrc(a.low + (long long)m0 * a.low_width * 4, 0x7ffffff0u);
    constexpr int U = MB * NB <= 4 ? 4 : 2;   // steps whose reads are issued together
    int mine[MB];
    uint64_t left[MB];
#pragma unroll
    for (int j = 0; j < MB; ++j) {
      const int t = m0 + (wm * MB + j) * 32 + l32;
      mine[j] = t < a.T ? a.adapter_of[t] : -1;
    }
#pragma unroll
    for (int j = 0; j < MB; ++j) left[j] = __ballot(mine[j] >= 0);
    const int steps = (a.rank * LB + 31) / 32;
    for (;;) {   // the adapters of the wave's tokens
      int ad = -1;
#pragma unroll
      for (int j = 0; j < MB; ++j)
        if (ad < 0 && left[j]) ad = __builtin_amdgcn_readlane(mine[j], __builtin_ctzll(left[j]));
      if (ad < 0) break;
#pragma unroll
      for (int j = 0; j < MB; ++j) left[j] &= ~__ballot(mine[j] == ad);
      bool mixed = false;
#pragma unroll
      for (int j = 0; j < MB; ++j)
        mixed = mixed || __any(mine[j] != ad && m0 + (wm * MB + j) * 32 + l32 < a.T);
      const __amdgpu_buffer_rsrc_t rb =
          make_rsrc(a.b + (long long)ad * a.N * a.rank * EB, 0x7ffffff0u);
      for (int s = 0; s < steps; s += U) {
        u32x4_t hi[U][MB], lo[U][MB], bf[U][NB];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int off = (s + u) * 32 + half * 16;
#pragma unroll
          for (int j = 0; j < MB; ++j)
            load_low<DT>(a, rl, (wm * MB + j) * 32 + l32, mine[j] == ad && s + u < steps, off,
                         &hi[u][j], &lo[u][j]);
#pragma unroll
          for (int i = 0; i < NB; ++i)
            bf[u][i] = load_b<DT>(a, rb, n0 + (wn * NB + i) * 32 + l32, off / LB);
        }
        __builtin_amdgcn_sched_barrier(0);
        if (mixed || DT != DT_F32) {
          uint32_t top = 0;
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < NB; ++i)
#pragma unroll
              for (int j = 0; j < 4; ++j) top = largest<DT>(top, bf[u][i][j]);
          if (__any(not_finite<DT>(top))) {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
              for (int i = 0; i < NB; ++i) dropped |= drop_not_finite<DT>(bf[u][i]);
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (s + u < steps)
#pragma unroll
            for (int i = 0; i < NB; ++i)
#pragma unroll
              for (int j = 0; j < MB; ++j)
                low_step<DT, true>(bf[u][i], hi[u][j], lo[u][j], acc[i][j]);
      }
    }
  }

  // 32 bytes of the sums' axis a step, whose operands are read a step ahead:
  // those of a stage's first step before the last matrix instructions of the
  // stage before, which cover the barrier between
  u32x4_t wf[2][NB], xf[2][MB];
  auto read = [&](const unsigned char* xs, int k, u32x4_t* w, u32x4_t* x) {
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int r = (wn * NB + i) * 32 + l32;
      w[i] = *reinterpret_cast<const u32x4_t*>(xs + (BM + r) * 128 +
                                               chunk_at(r, 2 * k + half) * 16);
    }
#pragma unroll
    for (int j = 0; j < MB; ++j) {
      const int r = (wm * MB + j) * 32 + l32;
      x[j] = *reinterpret_cast<const u32x4_t*>(xs + r * 128 + chunk_at(r, 2 * k + half) * 16);
    }
  };
  wait_vmcnt<(NS - 1) * (CX + CW)>();
  lds_barrier();
  read(lds, 0, wf[0], xf[0]);
  int at = 0;   // the stage in use
  for (int st = 0; st < stages; ++st) {
    const unsigned char* xs = lds + at * STAGE;
    const int next = at + 1 < NS ? at + 1 : 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k < 3) {
        read(xs, k + 1, wf[(k + 1) & 1], xf[(k + 1) & 1]);
      } else {
        // nobody reads this stage any more, the next one has arrived
        wait_vmcnt<(NS - 2) * (CX + CW)>();
        lds_barrier();
        LIBCONV_COPY_STAGE(st + NS, at)
        read(lds + next * STAGE, 0, wf[0], xf[0]);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = 0; j < MB; ++j)
          Step<DT, true>::run(wf[k & 1][i], xf[k & 1][j], acc[i][j]);
    }
    at = next;
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
        if constexpr (Runs)
          store_part(a, split, t, n, float4_t{v[0], v[1], v[2], v[3]});
        else if (n < a.N)
          store4<DT>(a, t, n, v);
      }
  }
  if (!Runs && __any(dropped)) {
    for (int k = 0; k < 16 * NB * MB; ++k) {
      const int t = m0 + (wm * MB + k / (16 * NB)) * 32 + l32;
      const int n = n0 + (wn * NB + k / 16 % NB) * 32 + 8 * (k / 4 % 4) + 4 * half + k % 4;
      if (t < a.T && n < a.N) add_not_finite<DT>(a, t, n);
    }
  }
}

// 32 tokens x 32 outputs, the sums' axis split over the four waves: for fp32,
// whose matrix instructions are slow enough that larger tiles leave compute
// units idle.  128 rows, 2048 -> 2048: 15 us (64 x 64 tiles: 40).
template <int DT, bool Runs>
__global__ __launch_bounds__(256, 2) void small_kernel(const LoraArgs a, int low_jobs) {
  constexpr int EB = Elem<DT>::bytes, NS = 4;
  __shared__ __attribute__((aligned(1024))) unsigned char lds[NS * kStage32];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int l32 = lane & 31, half = lane >> 5;
  const int tiles_n = (a.N + 31) / 32;
  int block = blockIdx.x, split = 0;
  if constexpr (Runs) {
    if (block < low_jobs) {
      const int groups = (a.T + kLowGroup - 1) / kLowGroup;
      low_rows<DT, kLowGroup>(a, block % groups * kLowGroup, block / groups * 16, lds);
      return;
    }
    block -= low_jobs;
    const int tiles = tiles_n * ((a.T + 31) / 32);
    split = block / tiles;
    block -= split * tiles;
  }
  const int m0 = block / tiles_n * 32, n0 = block % tiles_n * 32;
  const int row = a.K * EB;   // bytes of a row of W
  const int begin = Runs ? split * a.run : 0;
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.x + (long long)m0 * a.x_row + begin, 0x7ffffff0u);
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(a.w + (long long)n0 * row + begin, 0x7ffffff0u);
  int off[4];
  offsets32(off, a.T - m0, (int)a.x_row);
  offsets32(off + 2, a.N - n0, row);
  float16_t acc = {};
  product32<DT, NS>(rx, rw, off, Runs && begin + a.run < row ? a.run : row - begin, lds, acc);
  int dropped = 0;   // whether values of B were not finite
  if (!Runs && a.n_adapters > 0) {
    constexpr int LB = DT == DT_F32 ? 4 : 2;
    const __amdgpu_buffer_rsrc_t rl =
        make_rsrc(a.low + (long long)m0 * a.low_width * 4, 0x7ffffff0u);
    const int mine = m0 + l32 < a.T ? a.adapter_of[m0 + l32] : -1;
    const int steps = (a.rank * LB + 31) / 32;
    uint64_t left = __ballot(mine >= 0);
    while (left) {
      const int ad = __builtin_amdgcn_readlane(mine, __builtin_ctzll(left));
      left &= ~__ballot(mine == ad);
      const __amdgpu_buffer_rsrc_t rb =
          make_rsrc(a.b + (long long)ad * a.N * a.rank * EB, 0x7ffffff0u);
      for (int s = wave; s < steps; s += 4) {   // the waves take steps in turn
        const int at = s * 32 + half * 16;
        u32x4_t hi, lo;
        load_low<DT>(a, rl, l32, mine == ad, at, &hi, &lo);
        u32x4_t bf = load_b<DT>(a, rb, n0 + l32, at / LB);
        if (__any(drop_not_finite<DT>(bf))) dropped = 1;
        low_step<DT, true>(bf, hi, lo, acc);
      }
    }
  }
  float(*red)[32][36] = reinterpret_cast<float(*)[32][36]>(lds);
  int* flags = reinterpret_cast<int*>(lds + 4 * 32 * 36 * 4);
  lds_barrier();
  if (lane == 0) flags[wave] = dropped;
#pragma unroll
  for (int r = 0; r < 4; ++r)
    *reinterpret_cast<float4_t*>(&red[wave][l32][8 * r + 4 * half]) =
        float4_t{acc[4 * r], acc[4 * r + 1], acc[4 * r + 2], acc[4 * r + 3]};
  lds_barrier();
  const int t = threadIdx.x >> 3, n = (threadIdx.x & 7) * 4;
  float v[4] = {0, 0, 0, 0};
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const float4_t p = *reinterpret_cast<const float4_t*>(&red[w][t][n]);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] += p[j];
  }
  if constexpr (Runs)
    store_part(a, split, m0 + t, n0 + n, float4_t{v[0], v[1], v[2], v[3]});
  else if (m0 + t < a.T && n0 + n < a.N) {
    store4<DT>(a, m0 + t, n0 + n, v);
    if (flags[0] | flags[1] | flags[2] | flags[3])
      for (int j = 0; j < 4; ++j)
        if (n0 + n + j < a.N) add_not_finite<DT>(a, m0 + t, n0 + n + j);
  }
}

// Up to 16 * RB rows without adapters: 16 outputs a workgroup, the sum's axis
// split over 8 waves, joined in the order of the waves.  Bound by reading W, and
// x again from L2: 4096 -> 4096 in bf16, 16 rows 9.8 us, 64 rows 22 us.
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

// Four waves take 16 outputs each and a run of the sum's axis: x arrives in
// LDS, W straight in registers (each of its values has one reader), all of a
// run on its way at once.  The first `low_jobs` workgroups take the low-rank
// values meanwhile.  64 rows, 4096 -> 4096, rank 16 in bf16: 12 us (42 MB, and x
// from L2 for each 64 outputs; one round of workgroups that load, wait, compute
// and store, so that nothing overlaps).
// Bytes of a run, at most: x of 64 rows then takes 48 KB, and three workgroups
// share a compute unit (4096 -> 4096, 64 rows 16.7 us with the sum; runs of 1024
// 17.4, of 512 17.8; a row of 4160 17.1, 19.6 and 18.8).
constexpr int kRun = 768;
template <int DT, int RB>
__global__ __launch_bounds__(256, 2) void run_kernel(const LoraArgs a, int low_jobs) {
  constexpr int EB = Elem<DT>::bytes, ROWS = 16 * RB, STEPS = kRun / 64;
  __shared__ __attribute__((aligned(1024))) unsigned char lds[ROWS * kRun];
  if ((int)blockIdx.x < low_jobs) {
    low_rows<DT, 1>(a, (int)blockIdx.x % a.T, (int)blockIdx.x / a.T * 16, lds);
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
#pragma unroll
  for (int j = 0; j < RB; ++j) store_part(a, split, j * 16 + l16, n0 + quarter * 4, acc[j]);
}

// y of TT rows from TT blockIdx.y on: the runs in their order, the bias, the
// low-rank term.  A thread an output; rows of one adapter share their reads of
// B.  64 rows, 4096 outputs, 8 runs: 4 us.
template <int DT, int TT>
__global__ __launch_bounds__(256) void sum_kernel(const LoraArgs a) {
  constexpr int EB = Elem<DT>::bytes, E = 16 / EB;
  const int n = blockIdx.x * 256 + threadIdx.x, t0 = blockIdx.y * TT;
  if (n >= a.N) return;
  const long long n_pad = (a.N + 63) / 64 * 64;
  const float* part = a.part + t0 * n_pad + n;
  const int rows = a.T - t0 < TT ? a.T - t0 : TT;
  int of[TT];
  float v[TT];
#pragma unroll
  for (int i = 0; i < TT; ++i) {
    of[i] = i < rows ? __builtin_amdgcn_readfirstlane(a.adapter_of[t0 + i]) : -1;
    v[i] = 0.0f;
  }
  constexpr int U = 8 / TT;
  for (int s = 0; s < a.splits; s += U) {
    float p[U][TT];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < TT; ++i)
        p[u][i] = s + u < a.splits && i < rows ? part[((long long)(s + u) * a.T + i) * n_pad] : 0.0f;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < TT; ++i) v[i] += p[u][i];
  }
  if (a.bias) {
    float bias;
    if constexpr (DT == DT_F32) bias = static_cast<const float*>(a.bias)[n];
    else bias = Elem<DT>::bits_to_f32(static_cast<const uint16_t*>(a.bias)[n]);
#pragma unroll
    for (int i = 0; i < TT; ++i) v[i] += bias;
  }
  const float* low = reinterpret_cast<const float*>(a.low) + (long long)t0 * a.low_width;
#pragma unroll
  for (int turn = 0; turn < TT; ++turn) {
    const int ad = of[turn];
    bool first = ad >= 0;   // of the rows with this adapter
#pragma unroll
    for (int i = 0; i < turn; ++i) first = first && of[i] != ad;
    if (!first) continue;
    const char* b = a.b + ((long long)ad * a.N + n) * a.rank * EB;
    if (a.rank % E == 0) {
      for (int r = 0; r < a.rank; r += E) {
        float w[E];
        unpack<DT>(*reinterpret_cast<const u32x4_t*>(b + r * EB), w);
#pragma unroll
        for (int i = turn; i < TT; ++i)
          if (of[i] == ad)
#pragma unroll
            for (int e = 0; e < E; ++e) v[i] = fmaf(low[i * a.low_width + r + e], w[e], v[i]);
      }
    } else {
      for (int r = 0; r < a.rank; ++r) {
        float w;
        if constexpr (DT == DT_F32) w = reinterpret_cast<const float*>(b)[r];
        else w = Elem<DT>::bits_to_f32(reinterpret_cast<const uint16_t*>(b)[r]);
#pragma unroll
        for (int i = turn; i < TT; ++i)
          if (of[i] == ad) v[i] = fmaf(low[i * a.low_width + r], w, v[i]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < TT; ++i) {
    if (i >= rows) continue;
    char* y = a.y + (t0 + i) * a.y_row + (long long)n * EB;
    if constexpr (DT == DT_F32) *reinterpret_cast<float*>(y) = v[i];
    else *reinterpret_cast<uint16_t*>(y) = Elem<DT>::from_f32(v[i]);
  }
}

template <int DT, int BM, int BN, int WM, int WN, int NS, bool Runs>
void launch_tile(const LoraArgs& a, int low_jobs, hipStream_t stream) {
  const int tm = (a.T + BM - 1) / BM, tn = (a.N + BN - 1) / BN;
  hipLaunchKernelGGL((tile_kernel<DT, BM, BN, WM, WN, NS, Runs>),
                     dim3((unsigned)(low_jobs + tm * tn * (Runs ? a.splits : 1))),
                     dim3(64 * WM * WN), 0, stream, a, tm, tn, low_jobs);
}

template <int DT>
void launch_runs(const LoraArgs& a, hipStream_t stream) {
  const int parts = (a.rank + 15) / 16;
  const dim3 threads(256);
  if (a.T <= kFewRows) {
    const int low_jobs = a.T * parts;
    const dim3 grid((unsigned)(low_jobs + (a.N + 63) / 64 * a.splits));
    if (a.T <= 16)
      hipLaunchKernelGGL((run_kernel<DT, 1>), grid, threads, 0, stream, a, low_jobs);
    else if (a.T <= 32)
      hipLaunchKernelGGL((run_kernel<DT, 2>), grid, threads, 0, stream, a, low_jobs);
    else
      hipLaunchKernelGGL((run_kernel<DT, 4>), grid, threads, 0, stream, a, low_jobs);
    hipLaunchKernelGGL((sum_kernel<DT, 1>), dim3((unsigned)((a.N + 255) / 256), (unsigned)a.T),
                       threads, 0, stream, a);
    return;
  }
  const int low_jobs = (a.T + kLowGroup - 1) / kLowGroup * parts;
  if (a.tile == 128) {
    launch_tile<DT, 128, 128, 2, 2, 2, true>(a, low_jobs, stream);
  } else if (a.tile == 64) {
    launch_tile<DT, 64, 64, 2, 2, 4, true>(a, low_jobs, stream);
  } else if constexpr (DT == DT_F32) {
    const int tiles = (a.T + 31) / 32 * ((a.N + 31) / 32);
    hipLaunchKernelGGL((small_kernel<DT, true>), dim3((unsigned)(low_jobs + tiles * a.splits)),
                       threads, 0, stream, a, low_jobs);
  }
  hipLaunchKernelGGL((sum_kernel<DT, 4>),
                     dim3((unsigned)((a.N + 255) / 256), (unsigned)((a.T + 3) / 4)), threads, 0,
                     stream, a);
}

// Time of a launch in units of one 256 x 256 tile: rounds of workgroups over
// the compute units, each as long as its workgroups together on one unit.
double tile_cost(const LoraArgs& a, int cus, int splits, int b, int per_cu, double speed) {
  const double tiles = (double)((a.T + b - 1) / b) * ((a.N + b - 1) / b) * splits;
  const double rounds = (double)(long long)((tiles + (double)cus * per_cu - 1) / (cus * per_cu));
  const double share = tiles < (double)cus * per_cu ? (tiles > cus ? tiles / cus : 1.0) : per_cu;
  return rounds * share * b * b / splits / speed;
}

// Side of the tiles the product is formed in.  fp32 is bound by the matrix
// instructions: what the fullest compute unit has to do.
int pick_tile(const LoraArgs& a, int eb, int cus, int splits) {
  if (eb == 4) {
    auto work = [&](long long b) {
      const long long tiles = ((a.T + b - 1) / b) * ((a.N + b - 1) / b) * splits;
      return (double)((tiles + cus - 1) / cus * b * b);
    };
    const double w128 = work(128) * 0.85, w64 = work(64) * 0.92;
    // (sizes are checked for tiles of 64; four times as many may be more than a
    // launch holds)
    const long long n32 = ((a.T + 31LL) / 32) * ((a.N + 31LL) / 32);
    const double w32 = n32 * splits < kMostGroups ? work(32) : 2.0 * (w128 + w64);
    return w128 <= w64 && w128 <= w32 ? 128 : w64 <= w32 ? 64 : 32;
  }
  const double c256 = tile_cost(a, cus, splits, 256, 1, 1.0);
  const double c128 = tile_cost(a, cus, splits, 128, 2, 0.75);
  const double c64 = tile_cost(a, cus, splits, 64, 4, 0.4);
  return c256 <= c128 && c256 <= c64 ? 256 : c128 <= c64 ? 128 : 64;
}

template <int DT>
void launch_dt(const LoraArgs& a, int cus, hipStream_t stream) {
  if (a.splits > 0) {
    launch_runs<DT>(a, stream);
    return;
  }
  if (a.n_adapters > 0) {
    // with few row tiles, the adapters of a tile are dealt out
    const int tiles = (a.T + kLowRows - 1) / kLowRows, parts = a.low_width / 32;
    int shares = 2 * cus / (tiles * parts);
    const int most = a.n_adapters < kLowRows ? a.n_adapters : kLowRows;
    if (shares > most) shares = most;
    if (shares < 1) shares = 1;
    const dim3 grid((unsigned)tiles, (unsigned)shares, (unsigned)parts);
    // alone on its compute unit, a workgroup has twice the stages on their way
    if (tiles * shares * parts > cus)
      hipLaunchKernelGGL((low_kernel<DT, 4>), grid, dim3(256), 0, stream, a);
    else
      hipLaunchKernelGGL((low_kernel<DT, 8>), grid, dim3(256), 0, stream, a);
  }
  // (workgroups of twice the lanes; more outputs are for the tiles below)
  if (a.T <= kFewRows && (a.N + 15) / 16 < kMostGroups / 2) {
    const dim3 grid((unsigned)((a.N + 15) / 16)), threads(64 * kFewWaves);
    if (a.T <= 16) hipLaunchKernelGGL((few_kernel<DT, 1>), grid, threads, 0, stream, a);
    else if (a.T <= 32) hipLaunchKernelGGL((few_kernel<DT, 2>), grid, threads, 0, stream, a);
    else hipLaunchKernelGGL((few_kernel<DT, 4>), grid, threads, 0, stream, a);
    return;
  }
  const int tile = pick_tile(a, DT == DT_F32 ? 4 : 2, cus, 1);
  if constexpr (DT == DT_F32) {
    if (tile == 128) launch_tile<DT, 128, 128, 2, 2, 2, false>(a, 0, stream);
    else if (tile == 64) launch_tile<DT, 64, 64, 2, 2, 4, false>(a, 0, stream);
    else
      hipLaunchKernelGGL((small_kernel<DT, false>),
                         dim3((unsigned)((a.T + 31) / 32 * ((a.N + 31) / 32))), dim3(256), 0,
                         stream, a, 0);
  } else {
    if (tile == 256) launch_tile<DT, 256, 256, 4, 2, 2, false>(a, 0, stream);
    else if (tile == 128) launch_tile<DT, 128, 128, 2, 2, 2, false>(a, 0, stream);
    else launch_tile<DT, 64, 64, 2, 2, 4, false>(a, 0, stream);
  }
}

}  // namespace

long long lora_plan(LoraArgs* a, int dtype, int cus) {
  a->low_width = a->splits = a->run = a->tile = 0;
  if (a->n_adapters == 0 || a->T == 0) return 0;
  a->low_width = (a->rank + 31) / 32 * 32;
  const long long low = (long long)a->T * (a->low_width + 1) * 4;
  a->part_at = (low + 255) / 256 * 256;
  const int eb = dtype == LIBCONV_F32 ? 4 : 2;
  const long long row_bytes = (long long)a->K * eb, n_pad = (a->N + 63) / 64 * 64;
  long long runs;
  if (a->T <= kFewRows) {
    // two workgroups a compute unit if they have 256 bytes or more
    runs = 2 * cus / (n_pad / 64);
    if (runs > row_bytes / 256) runs = row_bytes / 256;
    if (runs < (row_bytes + kRun - 1) / kRun) runs = (row_bytes + kRun - 1) / kRun;
  } else {
    // the low-rank values row by row read A again for each group of rows, the
    // sum reads and writes y again in fp32: for few rows only.  Measured
    // against low_kernel and tile_kernel one after the other, K and N 4096,
    // rank 16: 128 rows 20 us against 41, 512 rows 42 against 49, 1024 rows 60
    // against 68; K and N 640: 1000 rows 14.5 against 13.6
    const double again = (double)((a->T + kLowGroup - 1) / kLowGroup) *
                         ((a->rank + 15) / 16 * 16) * row_bytes;
    if (a->T > 1024 || again > 128e6) return low;
    a->tile = pick_tile(*a, eb, cus, 1);
    if (a->tile == 256) a->tile = 128;
    const long long tiles = ((a->T + a->tile - 1) / a->tile) * ((a->N + a->tile - 1) / a->tile);
    runs = cus / tiles;
    if (runs > row_bytes / 1024) runs = row_bytes / 1024;
    if (runs > 8) runs = 8;
    if (runs < 1) runs = 1;
  }
  a->run = (int)(((row_bytes + runs - 1) / runs + 255) / 256 * 256);
  a->splits = (int)((row_bytes + a->run - 1) / a->run);
  return a->part_at + a->splits * a->T * n_pad * 4;
}

libconv_status lora_launch(LoraArgs a, int dtype, int cus, hipStream_t stream) {
  if (dtype == LIBCONV_F32) launch_dt<DT_F32>(a, cus, stream);
  else if (dtype == LIBCONV_F16) launch_dt<DT_F16>(a, cus, stream);
  else launch_dt<DT_BF16>(a, cus, stream);
  return hipGetLastError() == hipSuccess ? LIBCONV_OK : LIBCONV_ERR_LAUNCH;
}

}  // namespace libconv
