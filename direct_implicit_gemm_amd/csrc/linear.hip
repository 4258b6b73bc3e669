// linear.hip -- a projection with bias, activation and residual.
//
//   y[t] = act(W x[t] + bias) + residual[t]
//
// The product is formed transposed (outputs n on the rows of the matrix
// instructions, tokens on their columns), so that a lane holds 4 consecutive
// outputs of one token.  Both operands have their sums' axis dense: a stage
// is 128 bytes of it, copied straight into LDS.
#include "device_common.h"
#include "layer.h"

#include <cmath>

namespace libconv {
namespace {

// The activation of a sum in fp32.  tanh GELU and SiLU: the exponentials and the
// quotient are the hardware's (about one step each), but an exponent u is off by
// half steps of itself, so that results of large negative sums are off by 6 |u|
// of fp32's half steps (less than a 16-bit output's step up to |u| = 80).
// GELU = v Phi(v): Phi(-a) = erfcx(a / sqrt 2) exp(-a^2 / 2) / 2, for its tail (1 + erf
// is 4 % off at v = -5 in fp32, and 0 from -5.6 on).
template <int DT, int ACT> __device__ __forceinline__ float activated(float v) {
  constexpr float kLog2e = 1.4426950408889634f;
  constexpr float kTwoC = 2.0f * 0.7978845608028654f;   // sqrt(2 / pi)
  if constexpr (ACT == LIBCONV_ACT_RELU) return v > 0.0f ? v : 0.0f;
  if constexpr (ACT == LIBCONV_ACT_GELU) {
    float c;   // Phi(-|v|)
    if constexpr (DT == DT_F32) {
      // (the square's rounding is made up for; from 64 on all is 0)
      const float a = fminf(__builtin_fabsf(v), 64.0f), s = a * a;
      const float e = expf(-0.5f * s);
      c = 0.5f * erfcxf(a * 0.70710678118654752f) * fmaf(-0.5f * fmaf(a, a, -s), e, e);
    } else {
      // erfcx(z) = t poly(t), t = 1 / (1 + 0.44 z): fitted for the least relative error,
      // 2^-17.5 for 0 <= z <= 10.3
      const float t = __builtin_amdgcn_rcpf(fmaf(__builtin_fabsf(v), 0.31112698f, 1.0f));
      c = fmaf(t, -0.146106108f, 0.350653872f);
      c = fmaf(t, c, 0.0407293994f);
      c = fmaf(t, c, 0.263587385f);
      c = fmaf(t, c, 0.242569234f);
      c = fmaf(t, c, 0.248561053f);
      c *= 0.5f * t * __builtin_amdgcn_exp2f(-0.5f * kLog2e * (v * v));
    }
    return v * (v > 0.0f ? 1.0f - c : c);
  }
  if constexpr (ACT == LIBCONV_ACT_GELU_TANH) {
    // (1 + tanh(u)) / 2 = 1 / (1 + exp(-2 u))
    const float u2 = v * fmaf(v * v, kTwoC * 0.044715f, kTwoC);
    return v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * u2));
  }
  if constexpr (ACT == LIBCONV_ACT_SILU)
    return v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * v));
  return v;
}
template <int DT, int ACT>
__device__ __forceinline__ void activate_by(float* v, const float* bias, const float* r) {
#pragma unroll
  for (int j = 0; j < 16 / Elem<DT>::bytes; ++j)
    v[j] = activated<DT, ACT>(v[j] + bias[j]) + r[j];
}
template <int DT>
__device__ __forceinline__ void activate(float* v, const float* bias, const float* r, int act) {
  if (act == LIBCONV_ACT_NONE) activate_by<DT, LIBCONV_ACT_NONE>(v, bias, r);
  else if (act == LIBCONV_ACT_RELU) activate_by<DT, LIBCONV_ACT_RELU>(v, bias, r);
  else if (act == LIBCONV_ACT_GELU) activate_by<DT, LIBCONV_ACT_GELU>(v, bias, r);
  else if (act == LIBCONV_ACT_GELU_TANH) activate_by<DT, LIBCONV_ACT_GELU_TANH>(v, bias, r);
  else activate_by<DT, LIBCONV_ACT_SILU>(v, bias, r);
}

template <int DT> __device__ __forceinline__ float load1(const void* p, long long i) {
  if constexpr (DT == DT_F32) return static_cast<const float*>(p)[i];
  else return Elem<DT>::bits_to_f32(static_cast<const uint16_t*>(p)[i]);
}

// 16 bytes of a token's outputs, from n on, with bias, activation and residual.
// Where they do not lie on 16-byte boundaries or reach past N, one by one.
template <int DT> struct Outputs {
  static constexpr int EB = Elem<DT>::bytes, E = 16 / EB;
  int n;
  bool whole, whole_r;
  float bias[E];

  __device__ __forceinline__ Outputs(const LinearArgs& a, int first) : n(first) {
    const unsigned at = (unsigned)n * EB;   // (modulo 16)
    whole = n + E <= a.N && (((unsigned)reinterpret_cast<uintptr_t>(a.y) + at) & 15) == 0 &&
            (a.y_row & 15) == 0;
    whole_r = a.residual && n + E <= a.N &&
              (((unsigned)reinterpret_cast<uintptr_t>(a.residual) + at) & 15) == 0 &&
              (a.r_row & 15) == 0;
#pragma unroll
    for (int j = 0; j < E; ++j)
      bias[j] = a.bias && n + j < a.N ? load1<DT>(a.bias, n + j) : 0.0f;
  }
  // What can be read ahead of a token's residual.
  __device__ __forceinline__ u32x4_t residual(const LinearArgs& a, int t) const {
    u32x4_t v = {0, 0, 0, 0};
    if (whole_r && t < a.T)
      v = *reinterpret_cast<const u32x4_t*>(a.residual + t * a.r_row + (long long)n * EB);
    return v;
  }
  __device__ __forceinline__ void finish(const LinearArgs& a, int t, float* v,
                                         const u32x4_t& ahead) const {
    if (t >= a.T || n >= a.N) return;
    float r[E];
    unpack<DT>(ahead, r);
    if (a.residual && !whole_r) {
#pragma unroll
      for (int j = 0; j < E; ++j)
        if (n + j < a.N) r[j] = load1<DT>(a.residual + t * a.r_row, n + j);
    }
    activate<DT>(v, bias, r, a.act);
    char* at = a.y + t * a.y_row + (long long)n * EB;
    const u32x4_t w = pack<DT>(v);
    if (whole) {
      store_out16(at, w);
      return;
    }
#pragma unroll
    for (int j = 0; j < E; ++j)
      if (n + j < a.N) {
        if constexpr (EB == 4) reinterpret_cast<uint32_t*>(at)[j] = w[j];
        else reinterpret_cast<uint16_t*>(at)[j] = (uint16_t)(w[j / 2] >> (16 * (j & 1)));
      }
  }
};

// Position of the 16-byte chunk c of a 128-byte row in LDS: the 16 lanes that
// read one chunk of 16 rows at a time hit all banks.
__device__ __forceinline__ int chunk_at(int row, int c) { return c ^ ((row >> 1) & 7); }

// BM tokens x BN outputs, WM x WN waves; stages of 128 bytes of the sums' axis, NS
// of them in LDS or on their way.  Runs: the sums of a run of the sum's axis.
// 256 x 256 with 8 waves of 128 x 64: each number from LDS meets as many others as the
// registers of 2 waves a SIMD hold sums.  8192 x 4096 x 8192 in bfloat16: 437 us (1.26
// PFLOP/s; the library's product 420, matrix instructions alone 311), with bias, tanh
// GELU and residual 459: the matrix units, at the clock that they leave (1.7 GHz).  4
// waves of 128 x 128: 445; stages of 64 bytes, 4 of them: 475; a stage's copies in one
// step 443, over four 455.  fp32, 4096 x 4096 x 4096: 148 TFLOP/s (the library 139).
template <int DT, int BM, int BN, int WM, int WN, int NS, int SPREAD, bool Runs>
__global__
__launch_bounds__(64 * WM * WN, WM * WN == 4 && NS * (BM + BN) > 640 ? 1 : 2)   // by their room
void tile_kernel(const LinearArgs a, int tiles_m, int tiles_n) {
  constexpr int SB = 128;
  constexpr int EB = Elem<DT>::bytes;
  constexpr int THREADS = 64 * WM * WN;
  constexpr int MB = BM / WM / 32, NB = BN / WN / 32;   // 32 x 32 blocks of a wave
  constexpr int STAGE = (BM + BN) * SB, CPR = SB / 16, STEPS = SB / 32;
  __shared__ __attribute__((aligned(1024))) unsigned char lds[NS * STAGE];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int l32 = lane & 31, half = lane >> 5;
  const int wm = wave % WM, wn = wave / WM;

  // workgroups of one XCD follow one another over a band of 4 tiles of
  // outputs, so that its L2 holds the x and W tiles they share
  const int n_tiles = tiles_m * tiles_n;
  const int split = Runs ? blockIdx.x / n_tiles : 0, block = blockIdx.x - split * n_tiles;
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

  const int row = a.K * EB;   // bytes of a row of W
  const int from = Runs ? split * a.run : 0;
  const int run = Runs && from + a.run < row ? a.run : row - from;   // of this run
  const int stages = (run + SB - 1) / SB;
  // a thread copies one 16-byte chunk of rows PASS apart: its place in them is
  // the same, and the rows are told apart by a scalar offset.  Rows that do not
  // exist lie past the resource's end.
  constexpr int PASS = THREADS / CPR;
  static_assert(PASS % 16 == 0, "one chunk for a thread's rows");
  const int rows_x = a.T - m0 < BM ? a.T - m0 : BM, rows_w = a.N - n0 < BN ? a.N - n0 : BN;
  const int x_row = (int)a.x_row;
  const __amdgpu_buffer_rsrc_t rx =
      make_rsrc(a.x + (long long)m0 * a.x_row + from, (uint32_t)((rows_x - 1) * x_row + run));
  const __amdgpu_buffer_rsrc_t rw =
      make_rsrc(a.w + (long long)n0 * row + from, (uint32_t)((rows_w - 1) * row + run));
  const int chunk = chunk_at(threadIdx.x / CPR, threadIdx.x % CPR) * 16;
  const int x_off = (int)(threadIdx.x / CPR) * x_row + chunk;
  const int w_off = (int)(threadIdx.x / CPR) * row + chunk;
  constexpr int CX = BM / PASS, CW = BN / PASS;   // copies a thread
  // 32 bytes of the sums' axis a step.  Its operands are read a step ahead, in the
  // order in which they are taken, and a stage's copies are spread over SPREAD
  // steps, the last of a stage (which frees its place) and those of the next: one
  // read or copy after a matrix instruction, which runs meanwhile.
  constexpr int MMA = NB * MB, READS = NB + MB, COPIES = CX + CW, PARTS = COPIES / SPREAD;
  static_assert(COPIES % SPREAD == 0, "the same number of copies a step");
  // bytes from the stage's first that a thread copies, past the end where the row
  // has ended
  auto begin_of = [&](int st) { return st * SB + chunk < run ? st * SB : kFarOffset; };
  // copy c (first x's, then W's) into stage `at`
  auto copy = [&](int begin, int at, int c) __attribute__((always_inline)) {
    unsigned char* to = lds + at * STAGE + wave * 1024 + c * THREADS * 16;
    if (c < CX) copy16_to_lds(rx, to, x_off + begin, c * PASS * x_row);
    else copy16_to_lds(rw, to, w_off + begin, (c - CX) * PASS * row);
  };
  u32x4_t wf[2][NB], xf[2][MB];
  // this lane's place in a block of 32 rows of x and of W, for each step (the same in
  // all blocks)
  int at_x[STEPS], at_w[STEPS];
#pragma unroll
  for (int k = 0; k < STEPS; ++k) {
    const int in = l32 * SB + chunk_at(l32, 2 * k + half) * 16;
    at_x[k] = in + wm * MB * 32 * SB;
    at_w[k] = in + (BM + wn * NB * 32) * SB;
  }
  auto read = [&](int at, int k, int n, u32x4_t* w, u32x4_t* x) __attribute__((always_inline)) {
    if (n >= 1 && n <= MB) {
      x[n - 1] =
          *reinterpret_cast<const u32x4_t*>(lds + at_x[k] + (at * STAGE + (n - 1) * 32 * SB));
    } else {
      const int i = n == 0 ? 0 : n - MB;
      w[i] = *reinterpret_cast<const u32x4_t*>(lds + at_w[k] + (at * STAGE + i * 32 * SB));
    }
  };
#pragma unroll
  for (int st = 0; st < NS; ++st)
#pragma unroll
    for (int c = 0; c < (st < NS - 1 ? COPIES : PARTS); ++c) copy(begin_of(st), st, c);
  wait_vmcnt<(NS - 2) * COPIES + PARTS>();
  lds_barrier();
#pragma unroll
  for (int n = 0; n < READS; ++n) read(0, 0, n, wf[0], xf[0]);
  // Stage st, which lies at place `at` (a constant where it is called, so that the
  // addresses are).
  auto stage = [&](int st, int at) __attribute__((always_inline)) {
    const int next = at + 1 < NS ? at + 1 : 0, before = at > 0 ? at - 1 : NS - 1;
    const int begin = begin_of(st + NS - 1), begin_next = begin_of(st + NS);
#pragma unroll
    for (int k = 0; k < STEPS; ++k) {
      const bool last = k == STEPS - 1;
      // matrix instructions before the barrier of a stage's last step
      constexpr int EARLY = MMA / 4;
      const int first = last ? EARLY : 0, left = MMA - first;
#pragma unroll
      for (int n = 0; n < MMA; ++n) {
        if (last && n == EARLY) {
          // nobody reads this stage any more, the next one has arrived
          __builtin_amdgcn_sched_barrier(0);
          wait_vmcnt<(NS - 2) * COPIES>();
          lds_barrier();
        }
#pragma unroll
        for (int e = 0; e < Mma<DT>::KSUB; ++e)
          Mma<DT>::step(wf[k & 1][n / MB], xf[k & 1][n % MB], acc[n / MB][n % MB], e);
        // this instruction's share of the reads and of the copies
        const int i = n - first;
        if (i >= 0) {
#pragma unroll
          for (int q = 0; q < READS; ++q)
            if (q * (left > READS ? 1 : left) / (left > READS ? 1 : READS) == i)
              read(last ? next : at, last ? 0 : k + 1, q, wf[(k + 1) & 1], xf[(k + 1) & 1]);
#pragma unroll
          for (int c = 0; c < PARTS; ++c)
            if ((2 * c + 1) * left / (2 * PARTS) == i) {
              if (last) copy(begin_next, at, c);
              else if (k + 1 < SPREAD) copy(begin, before, (k + 1) * PARTS + c);
            }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
  };
  int st = 0;
  for (; st + NS <= stages; st += NS) {
#pragma unroll
    for (int i = 0; i < NS; ++i) stage(st + i, i);
  }
#pragma unroll
  for (int i = 0; i < NS - 1; ++i)
    if (st + i < stages) stage(st + i, i);
  wait_vmcnt<0>();

  if constexpr (Runs) {
    const long long n_pad = (a.N + 63) / 64 * 64;
#pragma unroll
    for (int j = 0; j < MB; ++j) {
      const int t = m0 + (wm * MB + j) * 32 + l32;
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int n = n0 + (wn * NB + i) * 32 + 8 * r + 4 * half;
          if (t < a.T && n < n_pad)
            *reinterpret_cast<float4_t*>(a.part + ((long long)split * a.T + t) * n_pad + n) =
                float4_t{acc[i][j][4 * r], acc[i][j][4 * r + 1], acc[i][j][4 * r + 2],
                         acc[i][j][4 * r + 3]};
        }
    }
    return;
  }
  lds_barrier();   // the stages are read: each wave has a part of them for its sums
  // 32 tokens at a time, through LDS: a lane then has 16 bytes of a token's outputs,
  // and neighbouring lanes neighbouring ones.  The residual of the next 32 tokens
  // is on its way meanwhile.
  constexpr int E = 16 / EB, COLS = NB * 32, LPT = COLS / E, TPI = 64 / LPT;   // lanes of a token
  constexpr int PAD = COLS + 4, TURNS = 32 / TPI;   // floats of a token in LDS
  constexpr bool AHEAD = EB == 2;   // (fp32: twice the room, for a call that is far slower)
  constexpr int ROOM = 32 * PAD * 4 + (AHEAD ? TURNS * 1024 : 0);
  static_assert(Runs || ROOM * WM * WN <= NS * STAGE,
                "32 tokens' sums and residual fit a wave's part");
  float* const sums = reinterpret_cast<float*>(lds + wave * ROOM);
  u32x4_t* const ahead = reinterpret_cast<u32x4_t*>(lds + wave * ROOM + 32 * PAD * 4) + lane;
  const Outputs<DT> out(a, n0 + wn * COLS + lane % LPT * E);
  const int t_first = m0 + wm * MB * 32 + lane / LPT;
  u32x4_t res[TURNS];
  if constexpr (AHEAD) {
#pragma unroll
    for (int i = 0; i < TURNS; ++i) res[i] = out.residual(a, t_first + i * TPI);
  }
#pragma unroll
  for (int j = 0; j < MB; ++j) {
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        *reinterpret_cast<float4_t*>(sums + l32 * PAD + i * 32 + 8 * r + 4 * half) =
            float4_t{acc[i][j][4 * r], acc[i][j][4 * r + 1], acc[i][j][4 * r + 2],
                     acc[i][j][4 * r + 3]};
    if constexpr (AHEAD) {
#pragma unroll
      for (int i = 0; i < TURNS; ++i) ahead[i * 64] = res[i];
      if (j + 1 < MB) {
#pragma unroll
        for (int i = 0; i < TURNS; ++i) res[i] = out.residual(a, t_first + (j + 1) * 32 + i * TPI);
      }
    }
    lds_fence();
#pragma unroll 1
    for (int i = 0; i < TURNS; ++i) {
      const float* from = sums + (lane / LPT + i * TPI) * PAD + lane % LPT * E;
      float v[E];
#pragma unroll
      for (int e = 0; e < E; e += 4) {
        const float4_t f = *reinterpret_cast<const float4_t*>(from + e);
#pragma unroll
        for (int q = 0; q < 4; ++q) v[e + q] = f[q];
      }
      const int t = t_first + j * 32 + i * TPI;
      out.finish(a, t, v, AHEAD ? ahead[i * 64] : out.residual(a, t));
    }
    lds_fence();
  }
}

// y from the sums of its runs, in their order; a thread 16 bytes of a token.  Few rows
// are bound by the weights' way to the compute units, which takes them all: 64 rows of
// 4096 sums and outputs have 64 tiles, in 4 runs each (8.5 us, 38 MB at 4.4 TB/s) and
// the runs' sums 3.5 us later; twice the runs 14.1 us instead of 12.2.
template <int DT> __global__ __launch_bounds__(256) void sum_kernel(const LinearArgs a) {
  constexpr int E = 16 / Elem<DT>::bytes, U = 8;
  const int n = (blockIdx.x * 256 + threadIdx.x) * E, t = blockIdx.y;
  if (n >= a.N) return;
  const long long n_pad = (a.N + 63) / 64 * 64;
  const Outputs<DT> out(a, n);
  const u32x4_t res = out.residual(a, t);
  const float* part = a.part + t * n_pad + n;
  float v[E] = {};
  for (int s = 0; s < a.splits; s += U) {
    float4_t p[U][E / 4];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < E / 4; ++e) {
        p[u][e] = float4_t{0, 0, 0, 0};
        if (s + u < a.splits)
          p[u][e] = *reinterpret_cast<const float4_t*>(part + (long long)(s + u) * a.T * n_pad +
                                                       4 * e);
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] += p[u][e / 4][e % 4];
  }
  out.finish(a, t, v, res);
}

template <int DT, int BM, int BN, int WM, int WN, int NS, int SPREAD, bool Runs = false>
void launch_tile(const LinearArgs& a, hipStream_t stream) {
  const int tm = (a.T + BM - 1) / BM, tn = (a.N + BN - 1) / BN;
  hipLaunchKernelGGL((tile_kernel<DT, BM, BN, WM, WN, NS, SPREAD, Runs>),
                     dim3((unsigned)(tm * tn * (Runs ? a.splits : 1))), dim3(64 * WM * WN), 0,
                     stream, a, tm, tn);
}

template <int DT> void launch_dt(const LinearArgs& a, hipStream_t stream) {
  if (a.part) {
    launch_tile<DT, 64, 64, 2, 2, 4, 1, true>(a, stream);
    constexpr int E = 16 / Elem<DT>::bytes;
    hipLaunchKernelGGL((sum_kernel<DT>),
                       dim3((unsigned)((a.N + 256 * E - 1) / (256 * E)), (unsigned)a.T), dim3(256),
                       0, stream, a);
    return;
  }
  if constexpr (DT != DT_F32) {
    if (a.tile == 256) {
      launch_tile<DT, 256, 256, 2, 4, 2, 2>(a, stream);
      return;
    }
    if (a.tile == 128 && a.stages == 4) {
      launch_tile<DT, 128, 128, 2, 2, 4, 4>(a, stream);
      return;
    }
  }
  if (a.tile == 128) launch_tile<DT, 128, 128, 2, 2, 2, 4>(a, stream);
  else launch_tile<DT, 64, 64, 2, 2, 4, 1>(a, stream);
}

// Time that a launch's sums of one element take on the fullest compute unit, with the
// sums' axis in `runs` runs, in units of one element of 256 x 256 tiles on it.  `alone`:
// the speed where no unit has a second workgroup.  (Workgroups on one unit share its
// matrix units: how many its LDS holds at a time does not count.)
double fullest(const LinearArgs& a, int cus, int side, int runs, double speed, double alone) {
  const double tiles =
      (double)((a.T + side - 1) / side) * ((a.N + side - 1) / side) * runs;
  const double most = std::ceil(tiles / cus);
  return most * side * side / (most > 1.0 ? speed : alone);
}

}  // namespace

long long linear_plan(LinearArgs* a, int dtype, int cus, bool allowed) {
  a->splits = a->run = 0;
  const bool f32 = dtype == LIBCONV_F32;
  // 16 bits, from products with 4096 sums and 4096 outputs in bfloat16, by tiles of
  // 64 / 128 / 256 (us): 256 rows 18 / 26 / 74, 1000 rows 59 / 37 / 78, 2048 rows 134 / 73 / 89,
  // 4096 rows 257 / 161 / 132; 2167 rows of 1280, 3840 outputs 41 / 27 / 34.  fp32 is bound
  // by the matrix instructions, whatever the tile, and what is left idle decides: 625 rows
  // of 2728, 3884 outputs (610 and 155 tiles of 64 and 128) 132 / 167, 2837 of 1304, 279 outputs
  // 26 / 84, 3769 of 368, 4123 outputs (3835 and 990) 116 / 113.
  const double c256 = fullest(*a, cus, 256, 1, 1.0, 1.0),
               c128 = f32 ? fullest(*a, cus, 128, 1, 1.0, 1.0)
                          : fullest(*a, cus, 128, 1, 0.75, 0.75);
  const double s64 = f32 ? 0.94 : 0.4, alone64 = f32 ? 0.94 : 0.3;
  const double c64 = fullest(*a, cus, 64, 1, s64, alone64);
  a->tile = !f32 && c256 <= c128 && c256 <= c64 ? 256 : c128 <= c64 ? 128 : 64;
  // One workgroup a compute unit: its room goes into stages (1000 rows 48 -> 37 us;
  // fp32, bound by the matrix units, 296 -> 299).
  a->stages = !f32 && (long long)((a->T + 127) / 128) * ((a->N + 127) / 128) <= cus ? 4 : 2;
  if (!allowed || a->T == 0 || a->T > 65535) return 0;   // (a row of the sums' grid each)
  // Runs of the sums' axis, in tiles of 64, where the fullest unit is done sooner by more
  // than the runs' sums take.  Microseconds: a stage of 128 bytes of a 64 x 64 tile at speed
  // 1, three stages for a tile's start and end, `sum` for the second launch (16 bits: with
  // what a first load waits for), 6 bytes a picosecond for the partial sums.  Of 220
  // sizes of 1 to 8192 rows, 128 to 4096 sums, 64 to 14336 outputs in each type, times are
  // 1.4 % (fp32) and 0.7 % (bfloat16) over the best of all tiles and runs; as many runs as
  // have a compute unit each: 5.8 and 7.6 %.  136 rows of 3624, 3934 outputs in fp32 (186
  // tiles) 61 us, in runs 52; 1462 rows of 688, 188 outputs in bfloat16 6.0, in runs 8.0.
  const long long row = (long long)a->K * (f32 ? 4 : 2), n_pad = (a->N + 63) / 64 * 64;
  const int stages = (int)((row + 127) / 128);
  const double stage = (f32 ? 0.46 : 0.08) / (64 * 64), sum = f32 ? 2.0 : 4.0;
  const double worth = f32 ? 1.0 : 0.9;   // (16 bits: less is not sure)
  const double tile = a->tile == 256 ? c256 : a->tile == 128 ? c128 : c64;
  double best = tile * stage * (stages + 3);
  for (int runs = 2; runs <= 16 && runs * (f32 ? 2 : 4) <= stages; ++runs) {
    const int run = (stages + runs - 1) / runs;
    if ((stages + run - 1) / run != runs) continue;
    const double t = fullest(*a, cus, 64, runs, s64, alone64) * stage * (run + 3) + sum +
                     8.0 * runs * a->T * n_pad / 6e6;
    if (t >= worth * best) continue;
    best = t;
    a->splits = runs;
    a->run = run * 128;
  }
  if (a->splits == 0) return 0;
  a->tile = 64;
  return 4LL * a->splits * a->T * n_pad;
}

libconv_status linear_launch(LinearArgs a, int dtype, hipStream_t stream) {
  if (dtype == LIBCONV_F32) launch_dt<DT_F32>(a, stream);
  else if (dtype == LIBCONV_F16) launch_dt<DT_F16>(a, stream);
  else launch_dt<DT_BF16>(a, stream);
  return hipGetLastError() == hipSuccess ? LIBCONV_OK : LIBCONV_ERR_LAUNCH;
}

}  // namespace libconv
