// layer_api.cpp -- entry points of the attention-layer operators: argument
// checks (all before anything is enqueued), plans and launches.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>
#include <numeric>

#include "internal.h"
#include "layer.h"

namespace libconv {
namespace {

constexpr long long kMaxInt = 0x7fffffff;
// Strides are below 2^40 elements and extents below 2^31, so that sums of
// their products stay inside 64 bits.
constexpr long long kMaxStride = 1LL << 40;
// Tiles are addressed with 32-bit offsets from their first row: 256 rows.
constexpr long long kMaxRowBytes = (1LL << 23) - 16;
constexpr int kMaxRows = (1 << 26) - 64;   // of a launch with a wave to a row

bool good_dtype(int dt) { return dt == LIBCONV_F32 || dt == LIBCONV_F16 || dt == LIBCONV_BF16; }

// A strided operand of up to three axes over dense vectors of `dense` bytes.
struct View {
  const char* p = nullptr;
  long long n[3] = {1, 1, 1}, s[3] = {0, 0, 0};   // extents, strides in bytes
  long long dense = 0;
  bool empty() const { return n[0] == 0 || n[1] == 0 || n[2] == 0; }
  // Bytes from the first to past the last.
  long long span() const {
    return empty() ? 0
                   : (n[0] - 1) * s[0] + (n[1] - 1) * s[1] + (n[2] - 1) * s[2] + dense;
  }
  // Whether no two vectors share a byte: each axis, by growing stride, steps
  // past everything the axes before it cover.
  bool distinct() const {
    int o[3] = {0, 1, 2};
    for (int i = 0; i < 2; ++i)
      for (int j = 0; j < 2 - i; ++j)
        if (s[o[j]] > s[o[j + 1]]) { const int t = o[j]; o[j] = o[j + 1]; o[j + 1] = t; }
    long long cover = dense;
    for (int i = 0; i < 3; ++i) {
      if (n[o[i]] <= 1) continue;
      if (s[o[i]] < cover) return false;
      cover += (n[o[i]] - 1) * s[o[i]];
    }
    return true;
  }
  // What all rows (of axes 0 and 1) are multiples of apart; 0: one row.
  long long row_step() const { return std::gcd(s[0], s[1]); }
  // Bytes of one row's heads.
  long long in_row() const { return (n[2] - 1) * s[2] + dense; }
};

View view(const void* p, long long n0, long long s0, long long n1, long long s1, long long n2,
          long long s2, long long d, int eb) {
  View v;
  v.p = static_cast<const char*>(p);
  v.n[0] = n0; v.n[1] = n1; v.n[2] = n2;
  // an axis of one index has no stride
  v.s[0] = n0 > 1 ? s0 * eb : 0;
  v.s[1] = n1 > 1 ? s1 * eb : 0;
  v.s[2] = n2 > 1 ? s2 * eb : 0;
  v.dense = d * eb;
  return v;
}

bool aligned16(const View& v) {
  return v.empty() || (((uintptr_t)v.p | (uintptr_t)(v.s[0] | v.s[1] | v.s[2])) & 15) == 0;
}

bool ranges_meet(const void* a, long long abytes, const void* b, long long bbytes) {
  if (!a || !b || abytes <= 0 || bbytes <= 0) return false;
  const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
  return a0 < b0 + (uintptr_t)bbytes && b0 < a0 + (uintptr_t)abytes;
}

// Whether two operands may share a byte.  Slices of the rows of one buffer
// (queries, keys and values of a fused projection) lie in one another's range
// without meeting, where each has a part of its own of the step that all their
// rows are multiples of apart.
bool meet(const View& a, const View& b) {
  if (!ranges_meet(a.p, a.span(), b.p, b.span())) return false;
  const long long step = std::gcd(a.row_step(), b.row_step());
  if (step == 0) return true;
  long long d = (long long)((intptr_t)b.p - (intptr_t)a.p) % step;
  if (d < 0) d += step;
  return d < a.in_row() || d + b.in_row() > step;
}

bool good_strides(const long long* s, int n) {
  for (int i = 0; i < n; ++i)
    if (s[i] < 0 || s[i] >= kMaxStride) return false;
  return true;
}

// ---------------------------------------------------------------- attention
libconv_status attn_shape(int B, int Sq, int P, int S, int q_heads, int k_heads, int head_dim,
                          int dtype) {
  if (!good_dtype(dtype)) return LIBCONV_ERR_BAD_DTYPE;
  if (B < 0 || Sq < 0 || P < 0 || S < 0 || q_heads < 1 || k_heads < 1 || head_dim < 1 ||
      q_heads % k_heads != 0)
    return LIBCONV_ERR_BAD_SHAPE;
  if (head_dim > 128 || head_dim % 8 != 0) return LIBCONV_ERR_UNSUPPORTED;
  // rows and keys are counted in 31 bits, the lanes of a launch (256 to 32 rows
  // of a key head) in 32
  const double rows = (double)B * Sq * q_heads;
  const double groups = (double)B * k_heads * (((double)Sq * (q_heads / k_heads) + 31) / 32);
  if (rows > (double)(kMaxInt / 64) || groups > (double)((1 << 24) - 4096) ||
      (double)P + S > (double)(kMaxInt - 1024))
    return LIBCONV_ERR_TOO_LARGE;
  return LIBCONV_OK;
}

void attn_sizes(AttnArgs* a, int B, int Sq, int P, int S, int q_heads, int k_heads, int head_dim) {
  std::memset(a, 0, sizeof(*a));
  a->B = B; a->Sq = Sq; a->P = P; a->S = S;
  a->Hk = k_heads; a->G = q_heads / k_heads; a->D = head_dim;
}

// -------------------------------------------------------------------- lora
libconv_status lora_shape(int T, int K, int N, int rank, int n_adapters, int n_requests,
                          int dtype) {
  if (!good_dtype(dtype)) return LIBCONV_ERR_BAD_DTYPE;
  if (T < 0 || K < 1 || N < 1 || n_adapters < 0 || n_requests < 0) return LIBCONV_ERR_BAD_SHAPE;
  const bool low = n_adapters > 0 && n_requests > 0;
  if (low && rank < 1) return LIBCONV_ERR_BAD_SHAPE;
  if (K % 8 != 0 || (low && rank > 128)) return LIBCONV_ERR_UNSUPPORTED;
  const long long eb = dtype_bytes(dtype);
  // offsets inside a tile of W and of an adapter's B: 31 bits; the lanes of a
  // launch (256 to 32 rows, or to a tile of 64 x 64): 32
  if (K * eb > kMaxRowBytes || T > kMaxRows ||
      (low && (long long)N * rank * eb >= kMaxInt - 1024) ||
      ((double)T / 64 + 1) * ((double)N / 64 + 1) > (double)(1 << 24))
    return LIBCONV_ERR_TOO_LARGE;
  return LIBCONV_OK;
}

}  // namespace
}  // namespace libconv

using namespace libconv;

extern "C" {

libconv_status libconv_qk_norm_rope(const void* q, const void* k, const void* v, void* q_out,
                                    void* k_out, void* v_out, const void* q_weight,
                                    const void* k_weight, const double* freqs,
                                    const int* positions, const int* slots,
                                    const long long* strides, int T, int q_heads, int k_heads,
                                    int head_dim, int rot_dim, int pairs0, int pairs1, int pairs2,
                                    int interleaved, int out_rows, float eps, int dtype,
                                    void* stream) {
  if (!good_dtype(dtype)) return LIBCONV_ERR_BAD_DTYPE;
  if (T < 0 || q_heads < 1 || k_heads < 1 || head_dim < 1 || rot_dim < 0 || pairs0 < 0 ||
      pairs1 < 0 || pairs2 < 0 || out_rows < 0 || !(eps >= 0.0f) || std::isinf(eps))
    return LIBCONV_ERR_BAD_SHAPE;
  if ((long long)pairs0 + pairs1 + pairs2 != rot_dim / 2 || rot_dim % 2 != 0 ||
      rot_dim > head_dim)
    return LIBCONV_ERR_BAD_SHAPE;
  if (head_dim > 256 || head_dim % 8 != 0 || (!interleaved && rot_dim % 16 != 0))
    return LIBCONV_ERR_UNSUPPORTED;
  if ((long long)q_heads + 2LL * k_heads > (1 << 24) || T > kMaxRows)
    return LIBCONV_ERR_TOO_LARGE;
  if (!strides || !q || !k || !q_out || !k_out || (!v != !v_out)) return LIBCONV_ERR_NULL_POINTER;
  if (rot_dim > 0 && (!freqs || !positions)) return LIBCONV_ERR_NULL_POINTER;
  if (!good_strides(strides, 12)) return LIBCONV_ERR_BAD_SHAPE;
  const int eb = dtype_bytes(dtype);
  const void* in[3] = {q, k, v};
  void* out[3] = {q_out, k_out, v_out};
  View vi[3], vo[3];
  const int parts = v ? 3 : 2;
  for (int i = 0; i < parts; ++i) {
    const int h = i == 0 ? q_heads : k_heads;
    vi[i] = view(in[i], 1, 0, T, strides[2 * i], h, strides[2 * i + 1], head_dim, eb);
    vo[i] = view(out[i], 1, 0, i > 0 && slots ? out_rows : T, strides[6 + 2 * i], h,
                 strides[7 + 2 * i], head_dim, eb);
    if (!aligned16(vi[i]) || !aligned16(vo[i])) return LIBCONV_ERR_MISALIGNED;
  }
  if ((((uintptr_t)q_weight | (uintptr_t)k_weight) & 15) != 0 || ((uintptr_t)freqs & 7) != 0 ||
      (((uintptr_t)positions | (uintptr_t)slots) & 3) != 0)
    return LIBCONV_ERR_MISALIGNED;
  const long long wb = (long long)head_dim * eb;
  const long long fb = (long long)rot_dim / 2 * 8;
  const int axes = pairs2 > 0 ? 3 : pairs1 > 0 ? 2 : 1;
  for (int i = 0; i < parts; ++i) {
    if (!vo[i].distinct()) return LIBCONV_ERR_ALIAS;
    for (int j = 0; j < parts; ++j) {
      // a token's head is read whole before it is written, by the same lanes
      const bool in_place = i == j && !slots && in[i] == out[i] && vi[i].s[1] == vo[i].s[1] &&
                            vi[i].s[2] == vo[i].s[2];
      if (!in_place && meet(vo[i], vi[j])) return LIBCONV_ERR_ALIAS;
      if (i != j && meet(vo[i], vo[j])) return LIBCONV_ERR_ALIAS;
    }
    const long long n = vo[i].span();
    if (ranges_meet(out[i], n, q_weight, wb) || ranges_meet(out[i], n, k_weight, wb) ||
        ranges_meet(out[i], n, freqs, fb) ||
        ranges_meet(out[i], n, positions, (rot_dim > 0 ? 4LL : 0) * axes * T) ||
        ranges_meet(out[i], n, slots, 4LL * T))
      return LIBCONV_ERR_ALIAS;
  }
  if (T == 0) return LIBCONV_OK;
  int cus = 0;
  if (!current_device(&cus)) return LIBCONV_ERR_NO_DEVICE;
  RopeArgs a;
  std::memset(&a, 0, sizeof(a));
  for (int i = 0; i < parts; ++i) {
    a.in[i] = vi[i].p;
    a.out[i] = static_cast<char*>(out[i]);
    a.in_row[i] = vi[i].s[1];
    a.in_head[i] = vi[i].s[2];
    a.out_row[i] = vo[i].s[1];
    a.out_head[i] = vo[i].s[2];
    a.heads[i] = i == 0 ? q_heads : k_heads;
  }
  a.weight[0] = q_weight;
  a.weight[1] = k_weight;
  a.freqs = freqs;
  a.positions = positions;
  a.slots = slots;
  a.T = T;
  a.D = head_dim;
  a.half = rot_dim / 2;
  a.pairs0 = pairs0;
  a.pairs01 = pairs0 + pairs1;
  a.interleaved = interleaved != 0;
  a.out_rows = out_rows;
  a.eps = eps;
  return rope_launch(a, dtype, reinterpret_cast<hipStream_t>(stream));
}

long long libconv_prefix_attention_workspace(int B, int Sq, int P, int S, int q_heads,
                                             int k_heads, int head_dim, int dtype) {
  if (attn_shape(B, Sq, P, S, q_heads, k_heads, head_dim, dtype) != LIBCONV_OK) return -1;
  AttnArgs a;
  attn_sizes(&a, B, Sq, P, S, q_heads, k_heads, head_dim);
  return attn_plan(&a, dtype, kPlanCus, true);
}

libconv_status libconv_prefix_attention(const void* q, const void* k_prefix, const void* v_prefix,
                                        const void* k, const void* v, const int* lengths,
                                        void* out, float* lse, const long long* strides, int B,
                                        int Sq, int P, int S, int q_heads, int k_heads,
                                        int head_dim, float scale, int causal, int dtype,
                                        void* workspace, long long workspace_bytes,
                                        void* stream) {
  const libconv_status st = attn_shape(B, Sq, P, S, q_heads, k_heads, head_dim, dtype);
  if (st != LIBCONV_OK) return st;
  if (!std::isfinite(scale) || workspace_bytes < 0) return LIBCONV_ERR_BAD_SHAPE;
  if (!strides || !q || !out || (P > 0 && (!k_prefix || !v_prefix)) ||
      (S > 0 && (!k || !v)) || !lengths)
    return LIBCONV_ERR_NULL_POINTER;
  if (!good_strides(strides, 16)) return LIBCONV_ERR_BAD_SHAPE;
  const int eb = dtype_bytes(dtype);
  const long long D = head_dim;
  const View vq = view(q, B, strides[0], Sq, strides[1], q_heads, strides[2], D, eb);
  const View vkp = view(k_prefix, 1, 0, P, strides[3], k_heads, strides[4], D, eb);
  const View vvp = view(v_prefix, 1, 0, P, strides[5], k_heads, strides[6], D, eb);
  const View vk = view(k, B, strides[7], S, strides[8], k_heads, strides[9], D, eb);
  const View vv = view(v, B, strides[10], S, strides[11], k_heads, strides[12], D, eb);
  const View vo = view(out, B, strides[13], Sq, strides[14], q_heads, strides[15], D, eb);
  if (!aligned16(vq) || !aligned16(vkp) || !aligned16(vvp) || !aligned16(vk) || !aligned16(vv) ||
      !aligned16(vo) || (((uintptr_t)lengths | (uintptr_t)lse) & 3) != 0)
    return LIBCONV_ERR_MISALIGNED;
  if (vkp.s[1] > kMaxRowBytes || vvp.s[1] > kMaxRowBytes || vk.s[1] > kMaxRowBytes ||
      vv.s[1] > kMaxRowBytes)
    return LIBCONV_ERR_TOO_LARGE;
  const long long lse_bytes = (long long)B * q_heads * Sq * 4;
  if (!vo.distinct() || meet(vo, vq) || meet(vo, vkp) || meet(vo, vvp) || meet(vo, vk) ||
      meet(vo, vv) || ranges_meet(out, vo.span(), lengths, 4LL * B) ||
      ranges_meet(out, vo.span(), lse, lse_bytes))
    return LIBCONV_ERR_ALIAS;
  const View* inputs[5] = {&vq, &vkp, &vvp, &vk, &vv};
  for (const View* x : inputs)
    if (ranges_meet(lse, lse_bytes, x->p, x->span()) ||
        ranges_meet(workspace, workspace_bytes, x->p, x->span()))
      return LIBCONV_ERR_ALIAS;
  if (ranges_meet(lse, lse_bytes, lengths, 4LL * B)) return LIBCONV_ERR_ALIAS;
  if (workspace) {
    if (((uintptr_t)workspace & 255) != 0) return LIBCONV_ERR_MISALIGNED;
    if (ranges_meet(workspace, workspace_bytes, out, vo.span()) ||
        ranges_meet(workspace, workspace_bytes, lse, lse_bytes) ||
        ranges_meet(workspace, workspace_bytes, lengths, 4LL * B))
      return LIBCONV_ERR_ALIAS;
  }
  if (B == 0 || Sq == 0) return LIBCONV_OK;
  int cus = 0;
  if (!current_device(&cus)) return LIBCONV_ERR_NO_DEVICE;
  AttnArgs a;
  attn_sizes(&a, B, Sq, P, S, q_heads, k_heads, head_dim);
  a.q = vq.p; a.kp = vkp.p; a.vp = vvp.p; a.k = vk.p; a.v = vv.p;
  a.lengths = lengths;
  a.out = static_cast<char*>(out);
  a.lse = lse;
  a.q_b = vq.s[0]; a.q_r = vq.s[1]; a.q_h = vq.s[2];
  a.kp_r = vkp.s[1]; a.kp_h = vkp.s[2];
  a.vp_r = vvp.s[1]; a.vp_h = vvp.s[2];
  a.k_b = vk.s[0]; a.k_r = vk.s[1]; a.k_h = vk.s[2];
  a.v_b = vv.s[0]; a.v_r = vv.s[1]; a.v_h = vv.s[2];
  a.o_b = vo.s[0]; a.o_r = vo.s[1]; a.o_h = vo.s[2];
  a.scale = scale == 0.0f ? 1.0f : std::fabs(scale) * 1.4426950408889634f;
  a.flip = scale == 0.0f ? 1 : scale < 0.0f ? -1 : 0;
  a.causal = causal != 0;
  const long long need = attn_plan(&a, dtype, kPlanCus, true);
  if (need > 0) {
    if (workspace && workspace_bytes >= need) {
      const long long slots = a.splits + (a.shared ? a.prefix_splits : 0);
      a.part = static_cast<float*>(workspace);
      a.part_lse = a.part + slots * a.Hk * a.B * a.Sq * a.G * a.D;
    } else {
      attn_plan(&a, dtype, kPlanCus, false);
    }
  }
  return attn_launch(a, dtype, reinterpret_cast<hipStream_t>(stream));
}

long long libconv_lora_workspace(int T, int K, int N, int rank, int n_adapters, int n_requests,
                                 int dtype) {
  if (lora_shape(T, K, N, rank, n_adapters, n_requests, dtype) != LIBCONV_OK) return -1;
  LoraArgs a;
  std::memset(&a, 0, sizeof(a));
  a.T = T; a.K = K; a.N = N; a.rank = rank;
  a.n_adapters = n_requests > 0 ? n_adapters : 0;
  a.n_requests = n_requests;
  return lora_plan(&a, dtype, kPlanCus);
}

libconv_status libconv_lora_linear(const void* x, const void* w, const void* bias, const void* a,
                                   const void* b, const float* scales, const int* row_starts,
                                   const int* adapters, void* y, int T, int K, int N, int rank,
                                   int n_adapters, int n_requests, long long x_stride,
                                   long long y_stride, int dtype, void* workspace,
                                   long long workspace_bytes, void* stream) {
  const libconv_status st = lora_shape(T, K, N, rank, n_adapters, n_requests, dtype);
  if (st != LIBCONV_OK) return st;
  const bool low = n_adapters > 0 && n_requests > 0;
  if (!x || !w || !y || (low && (!a || !b || !scales || !row_starts || !adapters)))
    return LIBCONV_ERR_NULL_POINTER;
  const int eb = dtype_bytes(dtype);
  if (workspace_bytes < 0 || x_stride < 0 || y_stride < 0 || x_stride >= kMaxStride ||
      y_stride >= kMaxStride || (T > 1 && y_stride < N))
    return LIBCONV_ERR_BAD_SHAPE;
  const View vx = view(x, 1, 0, T, x_stride, 1, 0, K, eb);
  const View vy = view(y, 1, 0, T, y_stride, 1, 0, N, eb);
  if (vx.s[1] > kMaxRowBytes) return LIBCONV_ERR_TOO_LARGE;
  if (!aligned16(vx) || (((uintptr_t)w | (uintptr_t)(low ? a : nullptr) |
                          (uintptr_t)(low ? b : nullptr)) & 15) != 0 ||
      (((uintptr_t)y | (uintptr_t)bias) & (eb - 1)) != 0 ||
      (low && (((uintptr_t)scales | (uintptr_t)row_starts | (uintptr_t)adapters) & 3) != 0))
    return LIBCONV_ERR_MISALIGNED;
  const void* read[8] = {x, w, bias, low ? a : nullptr, low ? b : nullptr,
                         low ? scales : nullptr, low ? row_starts : nullptr,
                         low ? adapters : nullptr};
  const long long bytes[8] = {vx.span(), (long long)N * K * eb, (long long)N * eb,
                              (long long)n_adapters * rank * K * eb,
                              (long long)n_adapters * rank * N * eb, 4LL * n_adapters,
                              4LL * (n_requests + 1LL), 4LL * n_requests};
  const long long yb = T > 0 ? vy.span() : 0;
  if (T > 0 && meet(vy, vx)) return LIBCONV_ERR_ALIAS;
  for (int i = 0; i < 8; ++i)
    if ((i > 0 && ranges_meet(y, yb, read[i], bytes[i])) ||
        ranges_meet(workspace, workspace_bytes, read[i], bytes[i]))
      return LIBCONV_ERR_ALIAS;
  if (ranges_meet(workspace, workspace_bytes, y, yb)) return LIBCONV_ERR_ALIAS;
  if (((uintptr_t)workspace & 255) != 0) return LIBCONV_ERR_MISALIGNED;
  if (T == 0) return LIBCONV_OK;
  LoraArgs l;
  std::memset(&l, 0, sizeof(l));
  l.x = vx.p;
  l.w = static_cast<const char*>(w);
  l.bias = bias;
  l.a = static_cast<const char*>(a);
  l.b = static_cast<const char*>(b);
  l.scales = scales;
  l.starts = row_starts;
  l.adapters = adapters;
  l.y = static_cast<char*>(y);
  l.T = T; l.K = K; l.N = N; l.rank = rank;
  l.n_adapters = low ? n_adapters : 0;
  l.n_requests = n_requests;
  l.x_row = vx.s[1];
  l.y_row = vy.s[1];
  if (lora_plan(&l, dtype, kPlanCus) > (workspace ? workspace_bytes : 0))
    return LIBCONV_ERR_SCRATCH_TOO_SMALL;
  l.low = static_cast<unsigned char*>(workspace);
  l.adapter_of = reinterpret_cast<int*>(l.low + (long long)T * l.low_width * 4);
  l.part = reinterpret_cast<float*>(l.low + l.part_at);
  int cus = 0;
  if (!current_device(&cus)) return LIBCONV_ERR_NO_DEVICE;
  return lora_launch(l, dtype, cus, reinterpret_cast<hipStream_t>(stream));
}

}  // extern "C"
