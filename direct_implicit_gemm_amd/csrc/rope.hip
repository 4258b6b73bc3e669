// rope.hip -- norms of queries and keys for each head with the position
// rotation in the same pass, and the write of keys and values into a cache.
//
//   n = x / sqrt(mean(x^2) + eps) * weight
//   (a, b) -> (a cos t - b sin t, b cos t + a sin t),  t = position * freq
//
// Bound by memory: every value is read once and written once.  A wave takes
// one token and a run of its heads (queries, keys, values in a row).  LPH lanes
// hold one head, 32 bytes each: 16 bytes of the first and of the second half of
// what turns, so that both members of a pair are in one lane and nothing but
// the sum of squares crosses lanes.  The angles are the same for all heads of a
// token: the wave's lanes form cos and sin of one pair each, once, and the
// heads' lanes read theirs back from LDS.  Measured: 38400 tokens of 40 heads of
// 128 in bf16 (787 MB) 144 us, 5.46 TB/s (a lane with 16 bytes of a head and its
// partner's fetched from another lane: 246 us); 2053 tokens of 20 heads of 128
// in fp32 8.1 us, 5.2 TB/s; 8 tokens of 60 heads of 64 4.8 us, latency.
#include "device_common.h"
#include "layer.h"

namespace libconv {
namespace {

constexpr int kWaves = 4;
constexpr int kUnroll = 4;   // steps whose loads are issued together

template <int CTRL> __device__ __forceinline__ float add_dpp(float v) {
  return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(
                                           0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
// Sum over LPH neighbouring lanes, in every one of them.
template <int LPH> __device__ __forceinline__ float lanes_sum(float v) {
  v = add_dpp<0xb1>(v);                            // pairs
  v = add_dpp<0x4e>(v);                            // pairs of a quad
  if constexpr (LPH >= 8) v = add_dpp<0x141>(v);   // quads of 8 lanes (mirrored)
  if constexpr (LPH >= 16) v = add_dpp<0x140>(v);  // halves of 16 (mirrored)
  if constexpr (LPH >= 32) v += __shfl_xor(v, 16);
  return v;
}

template <int DT, int LPH, bool Interleaved>
__global__ __launch_bounds__(64 * kWaves) void rope_kernel(const RopeArgs a) {
  constexpr int E = 16 / Elem<DT>::bytes;   // elements of 16 bytes
  constexpr int HPW = 64 / LPH;             // heads a step
  __shared__ float2 table[kWaves][128];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const long long unit = (long long)blockIdx.x * kWaves + wave;
  const int token = (int)(unit / a.chunks);
  if (token >= a.T) return;   // whole waves; the kernel has no barrier
  const int chunk = (int)(unit % a.chunks);
  const int s0 = (int)((long long)a.steps * chunk / a.chunks);
  const int s1 = (int)((long long)a.steps * (chunk + 1) / a.chunks);

  // this lane's two chunks of 16 bytes: the same of both halves of what turns;
  // of what does not, and of interleaved pairs, also one of either half (a
  // step's lanes then read and write whole lines at a time: neighbouring chunks
  // a lane had 1.7 times the bytes written)
  const int sub = lane % LPH, group = lane / LPH, chunks = a.D / E;
  const int paired = Interleaved ? 0 : a.half / E;
  const int rest = (chunks - 2 * paired + 1) / 2;   // lanes past the paired ones
  const int c1 = sub < paired ? sub : paired + sub;
  const int c2 = c1 + (sub < paired ? paired : rest);
  const bool live1 = sub < paired + rest, live2 = live1 && c2 < chunks;
  const int row_out = a.slots ? a.slots[token] : token;
  const bool row_ok = !a.slots || (row_out >= 0 && row_out < a.out_rows);

  // where a step's heads lie: steps are counted through queries, keys, values
  u32x4_t raw[kUnroll][2];
  auto kind_of = [&](int s) { return s < a.step_k ? 0 : s < a.step_v ? 1 : 2; };
  auto head_of = [&](int s) {
    return (s - (s < a.step_k ? 0 : s < a.step_v ? a.step_k : a.step_v)) * HPW;
  };
  auto fetch = [&](int s, u32x4_t* v) {
    v[0] = v[1] = u32x4_t{0, 0, 0, 0};
    if (s >= s1) return;
    const int kind = kind_of(s), head = head_of(s);
    const char* at = a.in[kind] + token * a.in_row[kind] + head * a.in_head[kind];
    if (head + group >= a.heads[kind]) return;
    const long long in_group = group * a.in_head[kind];
    if (live1) v[0] = *reinterpret_cast<const u32x4_t*>(at + (in_group + c1 * 16));
    if (live2) v[1] = *reinterpret_cast<const u32x4_t*>(at + (in_group + c2 * 16));
  };
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) fetch(s0 + u, raw[u]);

  // one turn's cos and sin of each pair, in 64 bits up to the reduced angle:
  // a position of 10^6 at a frequency of 1 has lost 4 digits in fp32
  for (int p = lane; p < a.half; p += 64) {
    const int axis = p < a.pairs0 ? 0 : p < a.pairs01 ? 1 : 2;
    const double turn = (double)a.positions[(long long)axis * a.T + token] *
                        (a.freqs[p] * 0.15915494309189533577);   // 1 / (2 pi)
    float sn, cs;
    sincospif(2.0f * (float)(turn - __builtin_rint(turn)), &sn, &cs);
    table[wave][p] = make_float2(cs, sn);
  }
  lds_fence();

  // cos and sin of this lane's pairs; those of interleaved pairs of its first
  // chunk, then of its second
  float c[E], s[E];
  bool on[E];
#pragma unroll
  for (int j = 0; j < E; ++j) {
    const int pair = Interleaved ? (j < E / 2 ? c1 : c2) * (E / 2) + j % (E / 2) : sub * E + j;
    on[j] = pair < a.half;
    const float2 t = table[wave][on[j] ? pair : 0];
    c[j] = on[j] ? t.x : 1.0f;
    s[j] = on[j] ? t.y : 0.0f;
  }
  const bool all_turn = 2 * a.half == a.D;   // else what does not turn is selected

  const uint32_t one = DT == DT_F32 ? 0x3f800000u : DT == DT_F16 ? 0x3c003c00u : 0x3f803f80u;
  u32x4_t weight[2][2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    weight[k][0] = weight[k][1] = u32x4_t{one, one, one, one};
    if (a.weight[k]) {
      const char* w = static_cast<const char*>(a.weight[k]);
      if (live1) weight[k][0] = *reinterpret_cast<const u32x4_t*>(w + c1 * 16);
      if (live2) weight[k][1] = *reinterpret_cast<const u32x4_t*>(w + c2 * 16);
    }
  }
  const float inv_d = 1.0f / (float)a.D;

  auto finish = [&](int st, const u32x4_t* v) {
    const int kind = kind_of(st), head = head_of(st);
    u32x4_t res[2] = {v[0], v[1]};
    if (kind < 2) {
      float x[2][E], w[2][E];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        unpack<DT>(v[h], x[h]);
        unpack<DT>(kind == 0 ? weight[0][h] : weight[1][h], w[h]);
      }
      float sum = 0.0f;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < E; ++j) sum = fmaf(x[h][j], x[h][j], sum);
      const float mean = fmaf(lanes_sum<LPH>(sum), inv_d, a.eps);
      float rs = __builtin_amdgcn_rsqf(mean);   // within one step
      if (__any(mean < 0x1p-120f)) rs = 1.0f / sqrtf(mean);   // takes small numbers for 0
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < E; ++j) x[h][j] = x[h][j] * rs * w[h][j];
      // the members of pair j
      float o[2][E];
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const int h0 = Interleaved ? j / (E / 2) : 0, h1 = Interleaved ? h0 : 1;
        const int i0 = Interleaved ? 2 * (j % (E / 2)) : j, i1 = Interleaved ? i0 + 1 : j;
        const float p = x[h0][i0], q = x[h1][i1];
        o[h0][i0] = fmaf(p, c[j], -(q * s[j]));
        o[h1][i1] = fmaf(q, c[j], p * s[j]);
        if (!all_turn) {
          o[h0][i0] = on[j] ? o[h0][i0] : p;
          o[h1][i1] = on[j] ? o[h1][i1] : q;
        }
      }
      res[0] = pack<DT>(o[0]);
      res[1] = pack<DT>(o[1]);
    }
    if (head + group < a.heads[kind] && (kind == 0 || row_ok)) {
      const long long row = kind == 0 ? token : row_out;
      char* at = a.out[kind] + row * a.out_row[kind] + head * a.out_head[kind];
      const long long in_group = group * a.out_head[kind];
      if (live1) store_out16(at + (in_group + c1 * 16), res[0]);
      if (live2) store_out16(at + (in_group + c2 * 16), res[1]);
    }
  };
  for (int st = s0; st < s1; st += kUnroll) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (st + u < s1) finish(st + u, raw[u]);
      fetch(st + kUnroll + u, raw[u]);
    }
  }
}

template <int DT, int LPH>
void launch(RopeArgs& a, hipStream_t stream) {
  constexpr int HPW = 64 / LPH;
  auto steps = [](int heads) { return (heads + HPW - 1) / HPW; };
  a.step_k = steps(a.heads[0]);
  a.step_v = a.step_k + steps(a.heads[1]);
  a.steps = a.step_v + steps(a.heads[2]);
  // Few tokens: their heads are spread over waves; many: a wave keeps a
  // token, so that its angles are formed once.
  const long long want = 4096;
  long long chunks = (want + a.T - 1) / a.T;
  if (chunks > a.steps) chunks = a.steps;
  a.chunks = (int)chunks;
  const long long blocks = ((long long)a.T * chunks + kWaves - 1) / kWaves;
  const dim3 grid((unsigned)blocks), threads(64 * kWaves);
  if (a.interleaved)
    hipLaunchKernelGGL(HIP_KERNEL_NAME(rope_kernel<DT, LPH, true>), grid, threads, 0, stream, a);
  else
    hipLaunchKernelGGL(HIP_KERNEL_NAME(rope_kernel<DT, LPH, false>), grid, threads, 0, stream, a);
}

template <int DT>
void launch_dt(RopeArgs& a, hipStream_t stream) {
  const int lanes = (a.D * Elem<DT>::bytes + 31) / 32;
  if (lanes <= 4) launch<DT, 4>(a, stream);
  else if (lanes <= 8) launch<DT, 8>(a, stream);
  else if (lanes <= 16) launch<DT, 16>(a, stream);
  else launch<DT, 32>(a, stream);
}

}  // namespace

libconv_status rope_launch(RopeArgs a, int dtype, hipStream_t stream) {
  if (dtype == LIBCONV_F32) launch_dt<DT_F32>(a, stream);
  else if (dtype == LIBCONV_F16) launch_dt<DT_F16>(a, stream);
  else launch_dt<DT_BF16>(a, stream);
  return hipGetLastError() == hipSuccess ? LIBCONV_OK : LIBCONV_ERR_LAUNCH;
}

}  // namespace libconv
