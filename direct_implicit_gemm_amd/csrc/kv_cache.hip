// kv_cache.hip -- keys and values appended to a cache of 8-bit codes, and read
// back.
//
//   s = max(s so far, least 2^e with max |x| / 2^e <= largest code)
//   code = rne(x / s),  codes that were there: rne(code * old / s)
//   read back: code * s
//
// The unit of either is one head's keys or values of one block: a wave takes
// one, so that the largest magnitude is a reduction over its lanes.  Both are
// bound by memory: 12 entries of 3200 tokens, 20 heads of 128 in blocks of 64, written
// in 121 us and read in 128 (591 MB each, bfloat16 and E4M3: 4.9 and 4.6 TB/s, where a
// copy of 1 GiB reaches 5.1).  One token of each of 64 entries, 8 heads: 5 us, a launch.
#include "codes.h"
#include "layer.h"

namespace libconv {
namespace {

constexpr int kThreads = 256;
constexpr int kWindow = 256;   // rows that a workgroup of the write looks over, at most: a
                               // block's, so that no two begin a block of the same entry

// idx / chunks of a row for idx below 256 rows of 32 chunks.
struct RowOf {
  unsigned chunks, m;
  __device__ __forceinline__ explicit RowOf(int c) : chunks(c), m((1u << 18) / c + 1) {}
  __device__ __forceinline__ int row(int i) const { return (int)((unsigned)i * m >> 18); }
};

// The largest magnitudes so far, as bits: of a word's two 16-bit values side by
// side, or of its one.
template <int DT> __device__ __forceinline__ uint32_t larger(uint32_t top, uint32_t w) {
  if constexpr (DT == DT_F32) {
    w &= 0x7fffffffu;
    return w > top ? w : top;
  } else {
    typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(
        uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, top),
                                            __builtin_bit_cast(u16x2_t, w & 0x7fff7fffu)));
  }
}
// ... over the wave, as the bits of a float; infinities and NaN are larger than all
// others.
template <int DT> __device__ __forceinline__ uint32_t top_of_wave(uint32_t top) {
  if constexpr (DT != DT_F32) top = (top & 0xffffu) > (top >> 16) ? top & 0xffffu : top >> 16;
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) {
    const uint32_t other = (uint32_t)__shfl_xor((int)top, m);
    top = other > top ? other : top;
  }
  if constexpr (DT == DT_F32) return top;
  return __builtin_bit_cast(uint32_t, Elem<DT>::bits_to_f32(top));
}
// The word without its infinities and NaN.
template <int DT> __device__ __forceinline__ uint32_t finite_of(uint32_t w) {
  if constexpr (DT == DT_F32) {
    return (w & 0x7f800000u) == 0x7f800000u ? 0u : w;
  } else {
    constexpr uint32_t E = DT == DT_F16 ? 0x7c00u : 0x7f80u;
    if ((w & E) == E) w &= 0xffff0000u;
    if ((w & (E << 16)) == E << 16) w &= 0xffffu;
    return w;
  }
}

// The least power of two, 2^-126 or more, that brings a magnitude (as bits) down
// to the largest code: 127 = 1.984375 2^6, 448 = 1.75 2^8.
template <int CF> __device__ __forceinline__ float scale_for(uint32_t top) {
  constexpr bool I8 = CF == LIBCONV_CACHE_I8;
  int e = (int)(top >> 23) - (I8 ? 6 : 8) + ((top & 0x7fffffu) > (I8 ? 0x7e0000u : 0x600000u));
  e = e < 1 ? 1 : e;
  return __builtin_bit_cast(float, (uint32_t)e << 23);
}

// Whether products with it and quotients by it are exact, as those of the scales
// written here (powers of two, no denormal ones) are.
__device__ __forceinline__ bool divides(float s) {
  const uint32_t u = __builtin_bit_cast(uint32_t, s);
  return (u & 0x7fffffu) == 0 && u != 0;
}
// A number in fp32 from which its code is rounded as from itself: inexact ones get
// an odd last bit, and lie on no border between two codes.  (The quotients of other
// scales in fp32, and then rounded to codes: 45.5 / 7 = 6.5 became 7, and of the
// bfloat16 numbers 1 in 100 met another code by a scale of 0.3.)
__device__ __forceinline__ float round_to_odd(double q) {
  const float f = (float)q;
  uint32_t u = __builtin_bit_cast(uint32_t, f);
  if ((double)f != q) {
    if (__builtin_fabs((double)f) > __builtin_fabs(q)) --u;
    u |= 1u;
  }
  return __builtin_bit_cast(float, u);
}

// One head's keys or values of a block: `rows` rows from x on become the tokens
// from `held` on of the block at `codes`.  HELD reads of a lane stay in registers
// between the largest magnitude and the rounding, others are read again.  (Above:
// largest magnitudes of two 16-bit values at a time, no look for infinities where
// there are none, and all of a block's 16 KB in registers 168 -> 124 us.)
template <int DT, int CF, int HELD>
__device__ __forceinline__ void write_block(const char* x, long long x_row, char* codes,
                                            long long token, float* scale, int rows, int held,
                                            int D) {
  constexpr int EB = Elem<DT>::bytes, E = 16 / EB;
  const int lane = threadIdx.x & 63;
  const float old_as_is = held > 0 ? *scale : 0.0f;
  const int chunks = D / E, total = rows * chunks;
  const RowOf by(chunks);
  auto read = [&](int i) {
    const int row = by.row(i);
    return *reinterpret_cast<const u32x4_t*>(x + row * x_row + (i - row * chunks) * 16);
  };
  u32x4_t raw[HELD];
  uint32_t top = 0;
#pragma unroll
  for (int u = 0; u < HELD; ++u) {
    raw[u] = u32x4_t{0, 0, 0, 0};
    if (u * 64 + lane < total) raw[u] = read(u * 64 + lane);
  }
#pragma unroll
  for (int u = 0; u < HELD; ++u)
#pragma unroll
    for (int j = 0; j < 4; ++j) top = larger<DT>(top, raw[u][j]);
  for (int i = HELD * 64 + lane; i < total; i += 64) {
    const u32x4_t v = read(i);
#pragma unroll
    for (int j = 0; j < 4; ++j) top = larger<DT>(top, v[j]);
  }
  top = top_of_wave<DT>(top);
  const bool finite = top < 0x7f800000u;
  if (!finite) {   // once more, without them
    top = 0;
    for (int i = lane; i < total; i += 64) {
      const u32x4_t v = read(i);
#pragma unroll
      for (int j = 0; j < 4; ++j) top = larger<DT>(top, finite_of<DT>(v[j]));
    }
    top = top_of_wave<DT>(top);
  }
  // (a scale that is no positive number stands for codes of no value)
  const float old = old_as_is > 0.0f && __builtin_isfinite(old_as_is) ? old_as_is : 0.0f;
  const float s = fmaxf(scale_for<CF>(top), old), inv = 1.0f / s;
  auto write = [&](int i, const u32x4_t& v, bool exact) __attribute__((always_inline)) {
    const int row = by.row(i);
    float f[E];
    unpack<DT>(v, f);
#pragma unroll
    for (int j = 0; j < E; ++j)
      f[j] = exact ? f[j] * inv : round_to_odd((double)f[j] / (double)s);
    char* at = codes + (held + row) * token + (i - row * chunks) * E;
    u32x2_t w;
#pragma unroll
    for (int j = 0; j < E / 4; ++j)
      w[j] = finite && exact ? codes_within<CF>(f + 4 * j) : codes_of<CF>(f + 4 * j);
    if constexpr (EB == 4) *reinterpret_cast<uint32_t*>(at) = w[0];
    else *reinterpret_cast<u32x2_t*>(at) = w;
  };
  if (divides(s)) {
#pragma unroll
    for (int u = 0; u < HELD; ++u)
      if (u * 64 + lane < total) write(u * 64 + lane, raw[u], true);
    for (int i = HELD * 64 + lane; i < total; i += 64) write(i, read(i), true);
  } else {   // (a scale that others wrote; read again, for one copy of the division)
#pragma unroll 1
    for (int i = lane; i < total; i += 64) write(i, read(i), false);
  }
  if (held > 0 && s != old_as_is) {   // (s is a power of two then, and its quotients exact)
    const float down = old / s;
    const bool exact = divides(old);
    const int words = D / 4;
    for (int i = lane; i < held * words; i += 64) {
      const int row = i / words;
      uint32_t* at = reinterpret_cast<uint32_t*>(codes + row * token + (i - row * words) * 4);
      float f[4];
      code_values<CF>(*at, f);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        f[j] = exact ? f[j] * down : round_to_odd((double)f[j] * ((double)old * (double)inv));
      *at = codes_of<CF>(f);
    }
  }
  if (lane == 0 && s != old_as_is) *scale = s;
}

// A workgroup looks over a block's number of rows for those that are their entry's
// first in a block, and its waves take the blocks' heads, keys and values, in turn (with
// the gridDim.y workgroups of the same rows).  Windows of 16 rows, whatever the block's
// size: 520 us instead of 168.
template <int DT, int CF, int HELD>
__global__ __launch_bounds__(kThreads) void write_kernel(const CacheCopyArgs a) {
  __shared__ int count, first[kWindow], rows[kWindow], held[kWindow], block[kWindow];
  const CacheView& c = a.c;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int size = 1 << c.log_block;
  const int r0 = blockIdx.x << c.log_block, r1 = r0 + size < a.T ? r0 + size : a.T;
  if (threadIdx.x == 0) count = 0;
  lds_barrier();
  for (int b = threadIdx.x; b < c.B; b += kThreads) {
    int s0 = a.starts[b], s1 = a.starts[b + 1], n = c.lengths[b];
    s0 = s0 < 0 ? 0 : s0;
    s1 = s1 > a.T ? a.T : s1;
    if (s0 >= r1 || s1 <= r0 || s0 >= s1) continue;
    const long long most = (long long)c.width << c.log_block;
    n = n < 0 ? 0 : n > most ? (int)most : n;
    // row t is at position n - s1 + t; the first row that is written, and the
    // first of this window that begins a block
    const int begin = s1 - n > s0 ? s1 - n : s0;
    const int lo = begin > r0 ? begin : r0, hi = s1 < r1 ? s1 : r1;
    const int next = lo + ((s1 - n - lo) & (size - 1));
    for (int k = 0; k < 2; ++k) {
      const int t = k == 0 ? begin : next;
      if (t < lo || t >= hi || (k == 1 && t == begin)) continue;
      const int p = n - s1 + t, in = p & (size - 1);
      const int id = c.table[(long long)b * c.width + (p >> c.log_block)];
      if (id < 0 || id >= c.blocks) continue;
      const int at = atomicAdd(&count, 1);   // (their order changes nothing)
      if (at >= kWindow) continue;           // rows of several entries: not allowed
      first[at] = t;
      rows[at] = s1 - t < size - in ? s1 - t : size - in;
      held[at] = in;
      block[at] = id;
    }
  }
  lds_barrier();
  const int found = __builtin_amdgcn_readfirstlane(count < kWindow ? count : kWindow);
  for (int job = blockIdx.y * 4 + wave; job < found * 2 * c.Hk; job += 4 * gridDim.y) {
    const int f = job / (2 * c.Hk), of = job - f * 2 * c.Hk;
    const int kv = of >= c.Hk, h = of - kv * c.Hk;
    const int t = __builtin_amdgcn_readfirstlane(first[f]);
    const int id = __builtin_amdgcn_readfirstlane(block[f]);
    write_block<DT, CF, HELD>(a.x[kv] + t * a.row[kv] + h * a.head[kv], a.row[kv],
                              c.codes[kv] + id * c.block[kv] + h * c.head[kv], c.token[kv],
                              c.scale[kv] + (long long)id * c.Hk + h,
                              __builtin_amdgcn_readfirstlane(rows[f]),
                              __builtin_amdgcn_readfirstlane(held[f]), c.D);
  }
}

// A workgroup takes a block of an entry, its waves the heads, keys and values, in
// turn (with the gridDim.y workgroups of the same block).
template <int DT, int CF>
__global__ __launch_bounds__(kThreads) void read_kernel(const CacheCopyArgs a, int per_entry) {
  constexpr int EB = Elem<DT>::bytes, E = 16 / EB, U = 4;
  const CacheView& c = a.c;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int b = blockIdx.x / per_entry, i = blockIdx.x - b * per_entry;
  int n = c.lengths[b];
  n = n < a.T ? n : a.T;
  const int p0 = i << c.log_block;
  if (p0 >= n) return;
  const int id = c.table[(long long)b * c.width + i];
  if (id < 0 || id >= c.blocks) return;
  const int rows = n - p0 < (1 << c.log_block) ? n - p0 : 1 << c.log_block;
  const int chunks = c.D / E, total = rows * chunks;
  const RowOf by(chunks);
  for (int job = blockIdx.y * 4 + wave; job < 2 * c.Hk; job += 4 * gridDim.y) {
    const int kv = job >= c.Hk, h = job - kv * c.Hk;
    const char* codes = c.codes[kv] + id * c.block[kv] + h * c.head[kv];
    char* to = a.x[kv] + b * a.entry[kv] + p0 * a.row[kv] + h * a.head[kv];
    const float s = c.scale[kv][(long long)id * c.Hk + h];
    for (int at = lane; at < total; at += 64 * U) {
      u32x2_t w[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        w[u] = u32x2_t{0, 0};
        const int j = at + u * 64, row = by.row(j);
        const char* from = codes + row * c.token[kv] + (j - row * chunks) * E;
        if (j < total) {
          if constexpr (EB == 4) w[u][0] = *reinterpret_cast<const uint32_t*>(from);
          else w[u] = *reinterpret_cast<const u32x2_t*>(from);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int j = at + u * 64, row = by.row(j);
        if (j >= total) continue;
        float f[8];
        code_values<CF>(w[u][0], f);
        if constexpr (EB == 2) code_values<CF>(w[u][1], f + 4);
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] *= s;
        store_out16(to + row * a.row[kv] + (j - row * chunks) * 16, pack<DT>(f));
      }
    }
  }
}

// Workgroups of `x` that take turns at `jobs` waves' work each: enough for the
// GPU, if there is that much.
unsigned turns(long long x, long long jobs) {
  const long long want = (2048 + x - 1) / x, most = (jobs + 3) / 4;
  const long long y = want < most ? want : most;
  return (unsigned)(y < 1 ? 1 : y > 65535 ? 65535 : y);
}

template <class F> libconv_status by_type(int format, int dtype, F&& f) {
  if (format == LIBCONV_CACHE_I8) {
    if (dtype == LIBCONV_F32) f.template run<DT_F32, LIBCONV_CACHE_I8>();
    else if (dtype == LIBCONV_F16) f.template run<DT_F16, LIBCONV_CACHE_I8>();
    else f.template run<DT_BF16, LIBCONV_CACHE_I8>();
  } else {
    if (dtype == LIBCONV_F32) f.template run<DT_F32, LIBCONV_CACHE_E4M3>();
    else if (dtype == LIBCONV_F16) f.template run<DT_F16, LIBCONV_CACHE_E4M3>();
    else f.template run<DT_BF16, LIBCONV_CACHE_E4M3>();
  }
  return hipGetLastError() == hipSuccess ? LIBCONV_OK : LIBCONV_ERR_LAUNCH;
}

struct Write {
  const CacheCopyArgs& a;
  hipStream_t stream;
  template <int DT, int CF> void run() {
    const int size = 1 << a.c.log_block, x = (a.T + size - 1) / size;
    // rows of one entry: a block's heads; single tokens: those of each row
    const unsigned block = (2u * a.c.Hk + 3) / 4;
    const unsigned rows = turns(x, 2LL * a.c.Hk * (a.T < size ? a.T : size));
    const unsigned y = block > rows ? block : rows;
    const dim3 grid((unsigned)x, y > 65535 ? 65535 : y), threads(kThreads);
    // (registers for no more than a block has: blocks of 16 tokens leave most idle)
    if (size * a.c.D * Elem<DT>::bytes <= 8 * 1024)
      hipLaunchKernelGGL((write_kernel<DT, CF, 8>), grid, threads, 0, stream, a);
    else
      hipLaunchKernelGGL((write_kernel<DT, CF, 16>), grid, threads, 0, stream, a);
  }
};
struct Read {
  const CacheCopyArgs& a;
  hipStream_t stream;
  template <int DT, int CF> void run() {
    const int per = (int)(((long long)a.T + (1 << a.c.log_block) - 1) >> a.c.log_block);
    const long long x = (long long)per * a.c.B;
    hipLaunchKernelGGL((read_kernel<DT, CF>), dim3((unsigned)x, turns(x, 2LL * a.c.Hk)),
                       dim3(kThreads), 0, stream, a, per);
  }
};

}  // namespace

libconv_status cache_write_launch(const CacheCopyArgs& a, int format, int dtype,
                                  hipStream_t stream) {
  return by_type(format, dtype, Write{a, stream});
}
libconv_status cache_read_launch(const CacheCopyArgs& a, int format, int dtype,
                                 hipStream_t stream) {
  return by_type(format, dtype, Read{a, stream});
}

}  // namespace libconv
