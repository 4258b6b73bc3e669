// rope.hip -- norms of queries and keys for each head with the position
// rotation in the same pass, and the write of keys and values into a cache.
//
//   n = x / sqrt(mean(x^2) + eps) * weight
//   (a, b) -> (a cos t - b sin t, b cos t + a sin t),  t = position * freq
//
// Bound by memory: every value is read once and written once.  A wave takes
// one token and a run of its heads (queries, keys, values in a row): LPH
// lanes hold one head, 16 bytes each, so a step moves 64 / LPH heads with one
// load and one store a lane.  The angles are the same for all heads of a
// token: the wave's lanes form cos and sin of one pair each, once, and the
// heads read them back from LDS.
#include "device_common.h"
#include "layer.h"

namespace libconv {
namespace {

constexpr int kWaves = 4;
constexpr int kUnroll = 4;   // steps whose loads are issued together

template <int DT, int LPH>
__global__ __launch_bounds__(64 * kWaves) void rope_kernel(const RopeArgs a) {
  constexpr int E = 16 / Elem<DT>::bytes;   // elements a lane holds of a head
  constexpr int HPW = 64 / LPH;             // heads a step
  __shared__ float2 table[kWaves][128];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const long long unit = (long long)blockIdx.x * kWaves + wave;
  const int token = (int)(unit / a.chunks);
  if (token >= a.T) return;   // whole waves; the kernel has no barrier
  const int chunk = (int)(unit % a.chunks);
  const int s0 = (int)((long long)a.steps * chunk / a.chunks);
  const int s1 = (int)((long long)a.steps * (chunk + 1) / a.chunks);

  const int sub = lane % LPH, group = lane / LPH, e0 = sub * E;
  const bool live = e0 < a.D;
  const int row_out = a.slots ? a.slots[token] : token;
  const bool row_ok = !a.slots || (row_out >= 0 && row_out < a.out_rows);

  // where a step's head lies: heads are counted through queries, keys, values
  u32x4_t raw[kUnroll];
  auto kind_of = [&](int head) {
    return head < a.heads[0] ? 0 : head < a.heads[0] + a.heads[1] ? 1 : 2;
  };
  const int total = a.heads[0] + a.heads[1] + a.heads[2];
  auto fetch = [&](int s, u32x4_t& v) {
    const int head = s * HPW + group;
    v = u32x4_t{0, 0, 0, 0};
    if (s < s1 && head < total && live) {
      const int kind = kind_of(head);
      const int h = head - (kind > 0 ? a.heads[0] : 0) - (kind > 1 ? a.heads[1] : 0);
      const char* base = kind == 0 ? a.in[0] : kind == 1 ? a.in[1] : a.in[2];
      const long long row = kind == 0 ? a.in_row[0] : kind == 1 ? a.in_row[1] : a.in_row[2];
      const long long hs = kind == 0 ? a.in_head[0] : kind == 1 ? a.in_head[1] : a.in_head[2];
      v = *reinterpret_cast<const u32x4_t*>(base + token * row + h * hs + sub * 16);
    }
  };
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) fetch(s0 + u, raw[u]);

  // one turn's cos and sin of each pair, in 64 bits up to the reduced angle:
  // a position of 10^6 at a frequency of 1 has lost 4 digits in fp32
  for (int p = lane; p < a.half; p += 64) {
    const int axis = p < a.pairs0 ? 0 : p < a.pairs01 ? 1 : 2;
    const double turns = (double)a.positions[(long long)axis * a.T + token] *
                         (a.freqs[p] * 0.15915494309189533577);   // 1 / (2 pi)
    float sn, cs;
    sincospif(2.0f * (float)(turns - __builtin_rint(turns)), &sn, &cs);
    table[wave][p] = make_float2(cs, sn);
  }
  lds_fence();

  // this lane's factors: out_j = n_j c_j + n_partner(j) s_j
  float c[E], s[E];
  const int first = e0 < a.half ? e0 : e0 - a.half;   // half-split: pair of element 0
  const int partner = e0 < a.half ? sub + a.half / E : sub - a.half / E;
  const bool turned = live && e0 < 2 * a.half;
#pragma unroll
  for (int j = 0; j < E; ++j) {
    const int pair = a.interleaved ? (e0 + j) >> 1 : first + j;
    const bool on = a.interleaved ? pair < a.half : turned;
    const float2 t = table[wave][on ? pair : 0];
    const bool lower = a.interleaved ? (j & 1) == 0 : e0 < a.half;
    c[j] = on ? t.x : 1.0f;
    s[j] = on ? (lower ? -t.y : t.y) : 0.0f;
  }
  const int source = (turned && !a.interleaved ? partner : sub) + group * LPH;
  const int partner_e0 = (source - group * LPH) * E;

  // weights of this lane's elements and of its partner's
  const uint32_t one = DT == DT_F32 ? 0x3f800000u : DT == DT_F16 ? 0x3c003c00u : 0x3f803f80u;
  u32x4_t own_w[2], other_w[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    own_w[k] = other_w[k] = u32x4_t{one, one, one, one};
    if (a.weight[k] && live) {
      const char* w = static_cast<const char*>(a.weight[k]);
      own_w[k] = *reinterpret_cast<const u32x4_t*>(w + sub * 16);
      other_w[k] = *reinterpret_cast<const u32x4_t*>(w + partner_e0 * Elem<DT>::bytes);
    }
  }
  const float inv_d = 1.0f / (float)a.D;

  auto finish = [&](int st, const u32x4_t& v) {
    const int head = st * HPW + group;
    const int kind = kind_of(head);
    float x[E], o[E];
    unpack<DT>(v, x);
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < E; ++j) sum = fmaf(x[j], x[j], sum);
#pragma unroll
    for (int m = 1; m < LPH; m <<= 1) sum += __shfl_xor(sum, m);
    const float rs = 1.0f / sqrtf(fmaf(sum, inv_d, a.eps));
    float w[E], y[E], wy[E];
    unpack<DT>(kind == 0 ? own_w[0] : own_w[1], w);
    if (a.interleaved) {
#pragma unroll
      for (int j = 0; j < E; ++j) x[j] = x[j] * rs * w[j];
#pragma unroll
      for (int j = 0; j < E; ++j) o[j] = fmaf(x[j], c[j], x[j ^ 1] * s[j]);
    } else {
      u32x4_t r;
#pragma unroll
      for (int j = 0; j < 4; ++j) r[j] = (uint32_t)__shfl((int)v[j], source);
      unpack<DT>(r, y);
      unpack<DT>(kind == 0 ? other_w[0] : other_w[1], wy);
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const float n = x[j] * rs * w[j], p = y[j] * rs * wy[j];
        o[j] = fmaf(n, c[j], p * s[j]);
      }
    }
    const u32x4_t res = kind == 2 ? v : pack<DT>(o);
    if (st < s1 && head < total && live && (kind == 0 || row_ok)) {
      const int h = head - (kind > 0 ? a.heads[0] : 0) - (kind > 1 ? a.heads[1] : 0);
      char* base = kind == 0 ? a.out[0] : kind == 1 ? a.out[1] : a.out[2];
      const long long row = kind == 0 ? a.out_row[0] : kind == 1 ? a.out_row[1] : a.out_row[2];
      const long long hs = kind == 0 ? a.out_head[0] : kind == 1 ? a.out_head[1] : a.out_head[2];
      const long long at = kind == 0 ? token : row_out;
      *reinterpret_cast<u32x4_t*>(base + at * row + h * hs + sub * 16) = res;
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
  a.steps = (a.heads[0] + a.heads[1] + a.heads[2] + HPW - 1) / HPW;
  // Few tokens: their heads are spread over waves; many: a wave keeps a
  // token, so that its angles are formed once.
  const long long want = 4096;
  long long chunks = (want + a.T - 1) / a.T;
  if (chunks > a.steps) chunks = a.steps;
  a.chunks = (int)chunks;
  const long long blocks = ((long long)a.T * chunks + kWaves - 1) / kWaves;
  hipLaunchKernelGGL(HIP_KERNEL_NAME(rope_kernel<DT, LPH>), dim3((unsigned)blocks),
                     dim3(64 * kWaves), 0, stream, a);
}

template <int DT>
void launch_dt(RopeArgs& a, hipStream_t stream) {
  const int lanes = a.D * Elem<DT>::bytes / 16;
  if (lanes <= 8) launch<DT, 8>(a, stream);
  else if (lanes <= 16) launch<DT, 16>(a, stream);
  else if (lanes <= 32) launch<DT, 32>(a, stream);
  else launch<DT, 64>(a, stream);
}

}  // namespace

libconv_status rope_launch(RopeArgs a, int dtype, hipStream_t stream) {
  if (dtype == LIBCONV_F32) launch_dt<DT_F32>(a, stream);
  else if (dtype == LIBCONV_F16) launch_dt<DT_F16>(a, stream);
  else launch_dt<DT_BF16>(a, stream);
  return hipGetLastError() == hipSuccess ? LIBCONV_OK : LIBCONV_ERR_LAUNCH;
}

}  // namespace libconv
