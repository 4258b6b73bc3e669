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

namespace libconv {
namespace {

// The activation of a sum in fp32.  The exponentials and the quotient are the
// hardware's (about one step each); what is left is far below a 16-bit output's
// step, and a few steps of a 32-bit one.
__device__ __forceinline__ float activated(float v, int act) {
  constexpr float kLog2e = 1.4426950408889634f;
  if (act == LIBCONV_ACT_RELU) return v > 0.0f ? v : 0.0f;
  if (act == LIBCONV_ACT_GELU) return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
  if (act == LIBCONV_ACT_GELU_TANH) {
    // (1 + tanh(u)) / 2 = 1 / (1 + exp(-2 u))
    const float u2 = v * fmaf(v * v, 2.0f * 0.7978845608028654f * 0.044715f, 2.0f * 0.7978845608028654f);
    return v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * u2));
  }
  if (act == LIBCONV_ACT_SILU)
    return v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * v));
  return v;
}

template <int DT> __device__ __forceinline__ float load1(const void* p, long long i) {
  if constexpr (DT == DT_F32) return static_cast<const float*>(p)[i];
  else return Elem<DT>::bits_to_f32(static_cast<const uint16_t*>(p)[i]);
}

// 4 consecutive outputs of a token from their sums; those past N are not there.
template <int DT>
__device__ __forceinline__ void finish4(const LinearArgs& a, int t, int n, const float* v) {
  constexpr int EB = Elem<DT>::bytes;
  char* at = a.y + t * a.y_row + (long long)n * EB;
  const char* rt = a.residual ? a.residual + t * a.r_row + (long long)n * EB : nullptr;
  const bool whole = n + 4 <= a.N;
  float o[4], r[4] = {0, 0, 0, 0};
  if (rt) {
    if (whole && (reinterpret_cast<uintptr_t>(rt) & (4 * EB - 1)) == 0) {
      if constexpr (EB == 4) {
        const float4_t f = *reinterpret_cast<const float4_t*>(rt);
#pragma unroll
        for (int j = 0; j < 4; ++j) r[j] = f[j];
      } else {
        const u32x2_t w = *reinterpret_cast<const u32x2_t*>(rt);
#pragma unroll
        for (int j = 0; j < 4; ++j) r[j] = Elem<DT>::bits_to_f32((w[j / 2] >> (16 * (j & 1))) & 0xffffu);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (n + j < a.N) r[j] = load1<DT>(rt, j);
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float b = a.bias && n + j < a.N ? load1<DT>(a.bias, n + j) : 0.0f;
    o[j] = activated(v[j] + b, a.act) + r[j];
  }
  if (whole && (reinterpret_cast<uintptr_t>(at) & (4 * EB - 1)) == 0) {
    if constexpr (EB == 4)
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
      if constexpr (EB == 4) reinterpret_cast<float*>(at)[j] = o[j];
      else reinterpret_cast<uint16_t*>(at)[j] = Elem<DT>::from_f32(o[j]);
    }
}

// Position of the 16-byte chunk c of a 128-byte row in LDS: the 16 lanes that
// read one chunk of 16 rows at a time hit all banks.
__device__ __forceinline__ int chunk_at(int row, int c) { return c ^ ((row >> 1) & 7); }

// BM tokens x BN outputs, WM x WN waves, NS stages in LDS or on their way.
template <int DT, int BM, int BN, int WM, int WN, int NS>
__global__ __launch_bounds__(64 * WM * WN, 2) void tile_kernel(const LinearArgs a, int tiles_m,
                                                               int tiles_n) {
  constexpr int EB = Elem<DT>::bytes;
  constexpr int THREADS = 64 * WM * WN;
  constexpr int MB = BM / WM / 32, NB = BN / WN / 32;   // 32 x 32 blocks of a wave
  constexpr int STAGE = (BM + BN) * 128;
  __shared__ __attribute__((aligned(1024))) unsigned char lds[NS * STAGE];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int l32 = lane & 31, half = lane >> 5;
  const int wm = wave % WM, wn = wave / WM;
  const int m0 = blockIdx.x / tiles_n * BM, n0 = blockIdx.x % tiles_n * BN;

  float16_t acc[NB][MB];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < MB; ++j) acc[i][j] = float16_t{};

  const int row = a.K * EB;   // bytes of a row of W
  const int stages = (row + 127) / 128;
  constexpr int PASS = THREADS / 8;
  static_assert(PASS % 16 == 0, "one chunk for a thread's rows");
  const int rows_x = a.T - m0 < BM ? a.T - m0 : BM, rows_w = a.N - n0 < BN ? a.N - n0 : BN;
  const int x_row = (int)a.x_row;
  const __amdgpu_buffer_rsrc_t rx =
      make_rsrc(a.x + (long long)m0 * a.x_row, (uint32_t)((rows_x - 1) * x_row + row));
  const __amdgpu_buffer_rsrc_t rw =
      make_rsrc(a.w + (long long)n0 * row, (uint32_t)((rows_w - 1) * row + row));
  const int chunk = chunk_at(threadIdx.x >> 3, threadIdx.x & 7) * 16;
  const int x_off = (int)(threadIdx.x >> 3) * x_row + chunk;
  const int w_off = (int)(threadIdx.x >> 3) * row + chunk;
  constexpr int CX = BM / PASS, CW = BN / PASS;   // copies a thread
  auto copy_stage = [&](int st, int at) {
    unsigned char* to = lds + at * STAGE + wave * 1024;
    const int k = st * 128;
    const bool in = k + chunk < row;
    const int xo = in ? x_off + k : kFarOffset, wo = in ? w_off + k : kFarOffset;
#pragma unroll
    for (int c = 0; c < CX; ++c) copy16_to_lds(rx, to + c * THREADS * 16, xo, c * PASS * x_row);
#pragma unroll
    for (int c = 0; c < CW; ++c)
      copy16_to_lds(rw, to + BM * 128 + c * THREADS * 16, wo, c * PASS * row);
  };
#pragma unroll
  for (int st = 0; st < NS - 1; ++st) copy_stage(st, st);
  for (int st = 0; st < stages; ++st) {
    wait_vmcnt<(NS - 2) * (CX + CW)>();
    lds_barrier();   // this stage has arrived for all, nobody reads the one before
    copy_stage(st + NS - 1, (st + NS - 1) % NS);
    const unsigned char* xs = lds + st % NS * STAGE;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      u32x4_t wf[NB], xf[MB];
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const int r = (wn * NB + i) * 32 + l32;
        wf[i] = *reinterpret_cast<const u32x4_t*>(xs + (BM + r) * 128 +
                                                  chunk_at(r, 2 * k + half) * 16);
      }
#pragma unroll
      for (int j = 0; j < MB; ++j) {
        const int r = (wm * MB + j) * 32 + l32;
        xf[j] = *reinterpret_cast<const u32x4_t*>(xs + r * 128 + chunk_at(r, 2 * k + half) * 16);
      }
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = 0; j < MB; ++j)
#pragma unroll
          for (int e = 0; e < Mma<DT>::KSUB; ++e) Mma<DT>::step(wf[i], xf[j], acc[i][j], e);
    }
  }
  wait_vmcnt<0>();

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
        if (n < a.N) finish4<DT>(a, t, n, v);
      }
  }
}

template <int DT> void launch_dt(const LinearArgs& a, hipStream_t stream) {
  const int tm = (a.T + 63) / 64, tn = (a.N + 63) / 64;
  hipLaunchKernelGGL((tile_kernel<DT, 64, 64, 2, 2, 4>), dim3((unsigned)(tm * tn)), dim3(256), 0,
                     stream, a, tm, tn);
}

}  // namespace

long long linear_plan(LinearArgs* a, int, int, bool) {
  a->splits = a->run = a->tile = 0;
  return 0;
}

libconv_status linear_launch(LinearArgs a, int dtype, hipStream_t stream) {
  if (dtype == LIBCONV_F32) launch_dt<DT_F32>(a, stream);
  else if (dtype == LIBCONV_F16) launch_dt<DT_F16>(a, stream);
  else launch_dt<DT_BF16>(a, stream);
  return hipGetLastError() == hipSuccess ? LIBCONV_OK : LIBCONV_ERR_LAUNCH;
}

}  // namespace libconv
