// cache_attention.hip -- attention of a ragged batch over a cache of keys and
// values in 8-bit codes, in blocks with a scale for each head.
//
//   out = sum_j p_j s_v(j) c_v(j),  p = softmax_j(scale s_k(j) <q, c_k(j)>)
//
// One pass over the keys with the running maximum m and sum l of a softmax, as in
// attention.hip: S = K Q^T and O = V^T P transposed, keys and components on the
// rows of the matrix instructions and queries on their columns, so that a lane
// holds scores, maximum, sum and outputs of one query.  The codes enter the
// matrix instructions as 16-bit numbers, which hold them exactly; the scale of a
// block's keys multiplies their scores, that of its values their probabilities
// (16 consecutive keys always have one scale).
//
// Entries with up to 32 rows a key head (single tokens) are bound by memory: one
// set of 32 columns holds all their queries, so that codes are read once, and
// workgroups share the tiles of all heads.  Entries with more are bound by
// the matrix and vector units: 128 rows share codes that are widened once.
#include "codes.h"
#include "internal.h"
#include "layer.h"

namespace libconv {
namespace {

constexpr int kThreads = 256;
// Of few rows: waves that split a workgroup's keys, and keys of a tile, 32 for each.
constexpr int kFewWaves = 4, kFewThreads = 64 * kFewWaves, kTile = 32 * kFewWaves;
constexpr int kFewRows = 32;     // rows of a key head that one set of matrix columns holds

// Terms that q and the probabilities enter the matrix instructions as: bfloat16
// holds 8 bits, fp16's 11 and fp32's 24 take two and three.  (q in fp16 meets
// codes in fp16; the probabilities times their scale may be past its range.)  q is
// exact.  The probabilities are rounded to what the output holds, as in attention.hip:
// each is off by half a step of it, which a sum of many evens out (bfloat16: 0.0023 of
// the output in all, of which the output's own rounding is 0.0016).
template <int DT> struct Terms {
  static constexpr int Q = DT == DT_F32 ? 3 : 1, P = DT == DT_F32 ? 3 : DT == DT_F16 ? 2 : 1;
  static constexpr int KT = DT == DT_F16 ? DT_F16 : DT_BF16;   // type of the first product
};

// Two numbers as N bfloat16 terms: each the rest of the ones before, rounded.
// Infinite: they may be infinities, which then have no rest.
template <int N, bool Infinite = false>
__device__ __forceinline__ void split2(float a, float b, uint32_t* w) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    w[i] = pack2<DT_BF16>(a, b);
    if (i + 1 < N) {
      const float ha = __builtin_bit_cast(float, w[i] << 16);
      const float hb = __builtin_bit_cast(float, w[i] & 0xffff0000u);
      a = !Infinite || __builtin_isfinite(ha) ? a - ha : 0.0f;
      b = !Infinite || __builtin_isfinite(hb) ? b - hb : 0.0f;
    }
  }
}

template <int DP> struct Shape {
  static constexpr int RB = DP <= 64 ? 64 : 128;   // bytes of a row of codes in LDS
  static constexpr int CPR = RB / 16;              // 16-byte chunks of it
  static constexpr int KS = DP / 16;               // steps of the first product
  static constexpr int DB = DP / 32;               // blocks of 32 components
  static constexpr int PART = 32 * RB;             // a wave's keys (values) of a tile
  static constexpr int COPIES = PART / 1024;       // 16 bytes a lane each
  static constexpr int WAVE = 2 * 2 * PART + 256 + 1024;   // stages of keys and values, blocks,
                                                           // scales
  static constexpr int LDS = kFewWaves * WAVE;
};
// Chunk c of row r is kept at c ^ swizzle(r): 16 rows' reads of one chunk, and the
// 8 rows that 16 lanes read a chunk of, hit all banks.
template <int CPR> __device__ __forceinline__ int swizzle(int row) {
  return CPR == 8 ? (row >> 1) & 7 : (row >> 2) & 3;
}

// 8 codes of one column: the 16 lanes of a quarter wave name 8 bytes each of 8
// rows of 16.  (restrict: as for read_column)
__device__ __forceinline__ u32x2_t read_column8(const unsigned char* __restrict p) {
  typedef int i32x2_t __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                                         (__attribute__((address_space(3))) i32x2_t*)p));
}

// One 4-byte read a lane straight into LDS, lane l's at dst + 4 l.
__device__ __forceinline__ void copy4_to_lds(__amdgpu_buffer_rsrc_t r, unsigned char* dst,
                                             int off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)dst, 4, off,
                                           0, 0, 0);
}

// An entry: its rows and its keys.
struct Entry {
  int row0, n, rows;   // first row, rows, rows of a key head that are computed
  int len;
};
__device__ __forceinline__ Entry entry_of(const CacheAttnArgs& a, int b) {
  Entry e;
  int s0 = a.starts[b], s1 = a.starts[b + 1], len = a.c.lengths[b];
  s0 = s0 < 0 ? 0 : s0;
  s1 = s1 > a.T ? a.T : s1;
  const int most = a.c.width << a.c.log_block;
  e.row0 = s0;
  e.n = s1 > s0 ? s1 - s0 : 0;
  e.rows = (e.n < a.max_rows ? e.n : a.max_rows) * a.G;
  e.len = len < 0 ? 0 : len > most ? most : len;
  return e;
}

// Whether an entry's rows fit one set of columns.
__device__ __forceinline__ bool few(const Entry& e) { return e.rows > 0 && e.rows <= kFewRows; }
// Tiles of such an entry (one without keys still has an output to write).
__device__ __forceinline__ int few_tiles(const Entry& e) {
  const int t = (e.len + kTile - 1) / kTile;
  return few(e) ? (t > 0 ? t : 1) : 0;
}

// Sum over the lanes up to this one.
__device__ __forceinline__ long long lanes_before(long long v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const long long o = __shfl_up(v, d);
    v += lane >= d ? o : 0;
  }
  return v;
}
__device__ __forceinline__ long long of_lane(long long v, int lane) {
  const uint32_t lo = __builtin_amdgcn_readlane((int)v, lane);
  return ((long long)__builtin_amdgcn_readlane((int)(v >> 32), lane) << 32) | lo;
}

// The entries' work, `weight(entry)` each, side by side.  A lane looks at `chunk`
// entries one after another; whoever needs one of them has the lanes look at those
// of its chunk once more, 64 at a time.  (A workgroup that went through all entries
// 64 at a time: 1024 entries, 2 heads of 64 228 us instead of 186.)
template <class W> struct Entries {
  const CacheAttnArgs& a;
  W weight;
  int chunk;
  Entry mine;          // this lane's entry of those that were looked at last
  long long w, up_to;  // work of this lane's chunk, and of those up to it

  __device__ __forceinline__ Entries(const CacheAttnArgs& args, W f) : a(args), weight(f) {
    chunk = (a.c.B + 63) >> 6;
    w = 0;
    const int first = (int)(threadIdx.x & 63) * chunk;
    mine = Entry{0, 0, 0, 0};
#pragma unroll 4
    for (int i = 0; i < chunk; ++i)
      if (first + i < a.c.B) {
        mine = entry_of(a, first + i);
        w += weight(mine);
      }
    up_to = lanes_before(w);
  }
  __device__ __forceinline__ long long total() const { return of_lane(up_to, 63); }
  // The lanes' entries from b on, up to `end`, and their work.
  __device__ __forceinline__ int look(int b, int end) {
    b += threadIdx.x & 63;
    mine = Entry{0, 0, 0, 0};
    if (b < end) mine = entry_of(a, b);
    return b < end ? weight(mine) : 0;
  }
  // The entry that holds number x of the work, and where its own begins; b = B: none.
  struct Found {
    Entry e;
    int b, weight;
    long long first;
  };
  __device__ __forceinline__ Found entry(int l, int b, int weight, long long first) const {
    Found f;
    f.e.row0 = __builtin_amdgcn_readlane(mine.row0, l);
    f.e.n = __builtin_amdgcn_readlane(mine.n, l);
    f.e.rows = __builtin_amdgcn_readlane(mine.rows, l);
    f.e.len = __builtin_amdgcn_readlane(mine.len, l);
    f.b = b;
    f.weight = weight;
    f.first = first;
    return f;
  }
  __device__ __forceinline__ Found find(long long x) {
    const uint64_t past = __ballot(up_to > x);
    if (!past) return {Entry{0, 0, 0, 0}, a.c.B, 0, total()};
    const int l = __builtin_ctzll(past);
    long long sum = of_lane(up_to - w, l);
    if (chunk == 1) return entry(l, l, (int)of_lane(w, l), sum);
    const int end = (l + 1) * chunk < a.c.B ? (l + 1) * chunk : a.c.B;
    for (int first = l * chunk; first < end; first += 64) {
      const int v = look(first, end);
      const long long to = lanes_before(v);
      const uint64_t in = __ballot(sum + to > x);
      if (in) {
        const int i = __builtin_ctzll(in);
        const int weight = __builtin_amdgcn_readlane(v, i);
        return entry(i, first + i, weight, sum + of_lane(to, i) - weight);
      }
      sum += of_lane(to, 63);
    }
    return {Entry{0, 0, 0, 0}, a.c.B, 0, sum};   // (not reached)
  }
};

// How the few_groups workgroups share the tiles of all heads: each a run of `per`,
// where a head begins with kStart tiles' time of no keys (a workgroup reads queries and
// table and fills its stages meanwhile): tile t of a head that begins at u is at
// u + kStart + t.
constexpr int kStart = 2;   // (64 entries of 1 to 8192 keys and 8 heads of 128: 0 129 us, 2 117,
                            // 3 119, 5 120)
__device__ __forceinline__ int few_units(const Entry& e) {
  const int t = few_tiles(e);
  return t > 0 ? t + kStart : 0;
}
__device__ __forceinline__ long long share_of(long long total, int groups) {
  const long long per = (total + groups - 1) / groups;
  return per < 2 ? 2 : per;   // (fewer keys are not worth a partial result)
}

// Rows `row_tile` * 32 .. of key head hk of an entry over tiles t0 .. t1 - 1 of its
// keys, in order; slot: where the partial result goes (-1: to the output), in units of
// the rows that a workgroup takes.
struct Job {
  Entry e;
  int b, hk, row_tile, t0, t1;
  long long slot;
};

// One job of few rows.  Each wave of four takes 32 keys of a tile through LDS
// stages of its own (two tiles of keys and of values, copied by it without
// registers), with its own maximum and sum, and never waits for the others before
// they are joined at the end.  Codes are read from LDS as 8-bit columns and rows
// and widened in registers: what a wave does for its keys is about 550
// instructions (128 components), two workgroups a compute unit, which keeps up
// with memory: 64 entries of 8 heads with 4096 keys, 537 MB, take 107 us (5.0
// TB/s).  Where few workgroups have keys the instructions bound it: a tile of 128
// keys takes 1.4 us.  Eight waves: 1024 keys 17.1 -> 15.3 us, but 32 to 256 keys
// 6.6 -> 9.1, for another copy of the kernel; two waves: 1000 keys 12.4 -> 19.7.
template <int DT, int CF, int DP>
__device__ __forceinline__ void attend_few(const CacheAttnArgs& a, const Job& job,
                                           unsigned char* lds) {
  using Z = Shape<DP>;
  constexpr int RB = Z::RB, CPR = Z::CPR, KS = Z::KS, DB = Z::DB, COPIES = Z::COPIES;
  constexpr int NQ = Terms<DT>::Q, NP = Terms<DT>::P, KT = Terms<DT>::KT;
  constexpr int EB = Elem<DT>::bytes;
  const CacheView& c = a.c;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int l32 = lane & 31, half = lane >> 5;
  const int len = job.e.len, D = c.D, hk = job.hk;

  // this lane's query
  const int local = job.row_tile * 32 + l32;
  const bool row_ok = local < job.e.rows;
  const int row = row_ok ? local : 0, qi = row / a.G, qg = row - qi * a.G;
  const char* qp =
      a.q + (long long)(job.e.row0 + qi) * a.q_r + (long long)(hk * a.G + qg) * a.q_h;
  u32x4_t qf[NQ][KS];
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    const int el = ((s & ~1) + half) * 16 + (s & 1) * 8;
    u32x4_t raw[EB / 2];
#pragma unroll
    for (int i = 0; i < EB / 2; ++i) {
      raw[i] = u32x4_t{0, 0, 0, 0};
      if (row_ok && el < D) raw[i] = *reinterpret_cast<const u32x4_t*>(qp + el * EB + i * 16);
      if (a.flip) {
        const uint32_t sign = EB == 4 ? 0x80000000u : 0x80008000u;
        raw[i] = a.flip < 0 ? raw[i] ^ u32x4_t{sign, sign, sign, sign} : u32x4_t{0, 0, 0, 0};
      }
    }
    if constexpr (DT == DT_F32) {
      float f[8];
      unpack<DT_F32>(raw[0], f);
      unpack<DT_F32>(raw[1], f + 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t w[NQ];
        split2<NQ, true>(f[2 * j], f[2 * j + 1], w);
#pragma unroll
        for (int i = 0; i < NQ; ++i) qf[i][s][j] = w[i];
      }
    } else {
      qf[0][s] = raw[0];
    }
  }

  // The groups of 16 keys that this wave reads, 64 (32 tiles) at a time: lane L holds
  // where the codes of group L & 1 of tile first + L / 2 lie, and how many there
  // are; their scales are in LDS.  The blocks of the next 32 tiles, and then
  // their scales, arrive in LDS too: what arrives in a register would have to be
  // waited for with everything else that is on its way.
  unsigned char* const mine = lds + wave * Z::WAVE;
  int* const blocks_in = reinterpret_cast<int*>(mine + 4 * Z::PART);
  float* const scales_in = reinterpret_cast<float*>(mine + 4 * Z::PART + 256);   // [2][2][64]
  const int mask = (1 << c.log_block) - 1;
  struct Groups {
    int at[2][2];   // offset of the codes from the caches' first: low and high word
    int rows;       // 0: none
  };
  auto position = [&](int first) {
    return (first + (lane >> 1)) * kTile + wave * 32 + (lane & 1) * 16;
  };
  const int* const table = c.table + (long long)job.b * c.width;
  const int last = len - 1;   // (tiles are counted so that positions fit 31 bits)
  auto locate = [&](int first, int id) {
    Groups g;
    const int p = position(first), left = len - p;
    const bool any = p <= last && id >= 0 && id < c.blocks;
    g.rows = !any ? 0 : left < 16 ? left : 16;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const long long off = any ? id * c.block[kv] + (p & mask) * c.token[kv] : 0;
      g.at[kv][0] = (int)off;
      g.at[kv][1] = (int)(off >> 32);
    }
    return g;
  };
  // copies of 4 bytes a lane
  const __amdgpu_buffer_rsrc_t scale_rsrc[2] = {
      make_rsrc(c.scale[0], (uint32_t)c.blocks * (uint32_t)c.Hk * 4u),
      make_rsrc(c.scale[1], (uint32_t)c.blocks * (uint32_t)c.Hk * 4u)};
  auto fetch_scales = [&](int id, bool any, int to) {
#pragma unroll
    for (int kv = 0; kv < 2; ++kv)
      copy4_to_lds(scale_rsrc[kv], reinterpret_cast<unsigned char*>(scales_in + (to * 2 + kv) * 64),
                   any ? (id * c.Hk + hk) * 4 : kFarOffset);
  };
  const __amdgpu_buffer_rsrc_t table_rsrc = make_rsrc(table, (uint32_t)c.width * 4u);
  auto fetch_blocks = [&](int first) {
    const int p = position(first);
    copy4_to_lds(table_rsrc, reinterpret_cast<unsigned char*>(blocks_in),
                 p <= last ? (p >> c.log_block) * 4 : kFarOffset);
  };
  int at = job.t0;   // first tile of the batch in hand
  Groups now, next;
  {
    int id = -1;
    if (position(at) <= last) id = table[position(at) >> c.log_block];
    now = next = locate(at, id);
    fetch_scales(id, now.rows > 0, 0);
  }

  // copies: 16 bytes of a row a lane
  constexpr int PASS = 64 / CPR;   // rows of a copy
  const int row_in = lane / CPR;
  int off[2][2];                   // keys and values, of even and odd copies of a group
#pragma unroll
  for (int kv = 0; kv < 2; ++kv)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int chunk = (lane % CPR) ^ swizzle<CPR>(j * PASS + row_in);
      off[kv][j] = chunk * 16 < D ? row_in * (int)c.token[kv] + chunk * 16 : kFarOffset;
    }
  auto stage = [&](int t, int kv) { return mine + (((t - job.t0) & 1) * 2 + kv) * Z::PART; };
  auto copy = [&](int t, int kv) {
    const char* const codes = c.codes[kv] + hk * c.head[kv];
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const int in = ((t - at) * 2 + g) & 63;
      const bool ahead = t - at >= 32;
      const int rows = __builtin_amdgcn_readlane(ahead ? next.rows : now.rows, in);
      const uint32_t lo = __builtin_amdgcn_readlane(ahead ? next.at[kv][0] : now.at[kv][0], in);
      const int hi = __builtin_amdgcn_readlane(ahead ? next.at[kv][1] : now.at[kv][1], in);
      const bool any = t < job.t1 && rows > 0;
      const __amdgpu_buffer_rsrc_t r =
          make_rsrc(codes + (((long long)hi << 32) | lo),
                    any ? (uint32_t)((rows - 1) * (int)c.token[kv] + D) : 0u);
#pragma unroll
      for (int j = 0; j < 16 / PASS; ++j)
        copy16_to_lds(r, stage(t, kv) + (g * (16 / PASS) + j) * 1024, off[kv][j],
                      j * PASS * (int)c.token[kv]);
    }
  };
  copy(job.t0, 0);
  copy(job.t0, 1);
  copy(job.t0 + 1, 0);
  copy(job.t0 + 1, 1);
  // keys that this query sees, and that every query of the tile does
  const int first_row = job.row_tile * 32;
  const int lim = a.causal ? len - job.e.n + qi + 1 : len;
  const int lim_all = a.causal ? len - job.e.n + first_row / a.G + 1 : len;
  // the queries have arrived (they were asked for before the blocks): the loop's
  // first use would wait for them again and again
#pragma unroll
  for (int i = 0; i < NQ; ++i)
#pragma unroll
    for (int s = 0; s < KS; ++s) asm volatile("" : "+v"(qf[i][s]));

  float16_t acc[DB];
#pragma unroll
  for (int d = 0; d < DB; ++d) acc[d] = float16_t{};
  float m = kLowest, l = 0.0f;

  const int krow = l32 * RB, ksw = swizzle<CPR>(l32);
  const int vrow = (((lane & 15) >> 1) & 3) + 8 * ((lane & 15) >> 3) + 4 * half;

  int buffer = 0;   // of the scales
  for (int t = job.t0; t < job.t1; ++t) {
    if (t - at == 32) {
      at += 32;
      now = next;
      buffer ^= 1;
    }
    // (the waits of two tiles cover a copy that was issued before them)
    if (t - at == 8 && at + 32 < job.t1) fetch_blocks(at + 32);
    if (t - at == 12 && at + 32 < job.t1) {
      const int id = blocks_in[lane];
      next = locate(at + 32, id);
      fetch_scales(id, next.rows > 0, buffer ^ 1);
    }
    const int in = (t - at) * 2;

    wait_vmcnt<3 * COPIES>();
    lds_fence();
    const float* const of = scales_in + buffer * 128 + in;
    float f[2], add[2], fv[2];
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      f[g] = of[g] * a.scale;
      fv[g] = of[64 + g];
      add[g] = __builtin_amdgcn_readlane(now.rows, in + g) > 0 ? 0.0f : kNegInf;
    }
    float16_t s = {};
    const unsigned char* kt = stage(t, 0);
#pragma unroll
    for (int j = 0; j < KS / 2; ++j) {
      const u32x4_t w =
          *reinterpret_cast<const u32x4_t*>(kt + krow + (((2 * j + half) ^ ksw) * 16));
      const u32x4_t k0 = code_values16<CF, KT>(w[0], w[1]), k1 = code_values16<CF, KT>(w[2], w[3]);
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        Mma<KT>::step(k0, qf[i][2 * j], s, 0);
        Mma<KT>::step(k1, qf[i][2 * j + 1], s, 0);
      }
    }
    lds_fence();
    copy(t + 2, 0);

#pragma unroll
    for (int r = 0; r < 16; ++r) s[r] = fmaf(s[r], f[r >> 3], add[r >> 3]);
    const int p0 = t * kTile + wave * 32;
    if (p0 + 32 > lim_all) {
      const int lane_lim = lim - p0 - 4 * half;
#pragma unroll
      for (int r = 0; r < 16; ++r)
        s[r] = (r & 3) + 8 * (r >> 2) < lane_lim ? s[r] : kNegInf;
    }
    float top = s[0];
#pragma unroll
    for (int r = 1; r < 16; ++r) top = fmaxf(top, s[r]);
    top = swap_halves_max(top);
    // the maximum moves only when it falls behind by 2^SLACK: the sums are hardly ever
    // rescaled
    constexpr float SLACK = 8.0f;
    if (__any(top > m + SLACK)) {
      const float m_new = top > m + SLACK ? top : m, fall = __builtin_amdgcn_exp2f(m - m_new);
      m = m_new;
      l *= fall;
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[d][r] *= fall;
    }
    u32x4_t pf[NP][2];
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      s[r] = __builtin_amdgcn_exp2f(s[r] - m);
      l += s[r];
      s[r] *= fv[r >> 3];
    }
#pragma unroll
    for (int r = 0; r < 16; r += 2) {
      uint32_t w[NP];
      split2<NP>(s[r], s[r + 1], w);
#pragma unroll
      for (int i = 0; i < NP; ++i) pf[i][r >> 3][(r & 7) >> 1] = w[i];
    }

    wait_vmcnt<3 * COPIES>();
    lds_fence();
    const unsigned char* vt = stage(t, 1);
#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
      for (int d = 0; d < DB; ++d) {
        const int r = g * 16 + vrow, chunk = (2 * d + ((lane >> 4) & 1)) ^ swizzle<CPR>(r);
        const u32x2_t w = read_column8(vt + r * RB + chunk * 16 + (lane & 1) * 8);
        const u32x4_t vf = code_values16<CF, DT_BF16>(w[0], w[1]);
#pragma unroll
        for (int i = 0; i < NP; ++i) Mma<DT_BF16>::step(vf, pf[i][g], acc[d], 0);
      }
    lds_fence();
    copy(t + 2, 1);
  }
  wait_vmcnt<0>();

  // join the waves: each leaves maximum, sum and outputs (DP components, 32 rows
  // fastest) in LDS and sums 32 components of all
  l += __shfl_xor(l, 32);
  static_assert(kFewWaves * 32 * DP * 4 <= Z::LDS - 1024, "the join fits the stages");
  float* const tops = reinterpret_cast<float*>(lds + Z::LDS - 1024);   // [wave][32], then the sums
  constexpr int SUMS = kFewWaves * 32;
  lds_barrier();   // every wave is done with its stages, no copy is on its way
  float* const rooms = reinterpret_cast<float*>(lds);
  if (half == 0) {
    tops[wave * 32 + l32] = m;
    tops[SUMS + wave * 32 + l32] = l;
  }
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int r = 0; r < 16; ++r)
      rooms[(wave * DP + d * 32 + (r & 3) + 8 * (r >> 2) + 4 * half) * 32 + l32] = acc[d][r];
  lds_barrier();
  for (int d = wave; d < DB; d += kFewWaves) {
    float m_all = tops[l32];
#pragma unroll
    for (int w = 1; w < kFewWaves; ++w) m_all = fmaxf(m_all, tops[w * 32 + l32]);
    float o[16] = {};
    l = 0.0f;
#pragma unroll
    for (int w = 0; w < kFewWaves; ++w) {
      const float g = __builtin_amdgcn_exp2f(tops[w * 32 + l32] - m_all);
      l = fmaf(tops[SUMS + w * 32 + l32], g, l);
#pragma unroll
      for (int r = 0; r < 16; ++r)
        o[r] = fmaf(rooms[(w * DP + d * 32 + (r & 3) + 8 * (r >> 2) + 4 * half) * 32 + l32], g,
                    o[r]);
    }
    if (!row_ok) continue;
    const float inv = l > 0.0f ? 1.0f / l : l;   // 0 keys: 0; a NaN stays
    const float lse2 = l == 0.0f ? kNegInf : m_all + __builtin_amdgcn_logf(l);
    const long long slot = job.slot * kFewRows + local, t = job.e.row0 + qi;
    const int head = hk * a.G + qg;
    if (d == 0 && half == 0) {
      if (job.slot >= 0) a.part_lse[slot] = lse2;
      else if (a.lse) a.lse[t * (c.Hk * a.G) + head] = lse2 * kLn2;
    }
    char* const op = a.out + t * a.o_r + head * a.o_h;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int comp = d * 32 + 8 * r + 4 * half;
      if (comp >= D) continue;
      const float4_t v = {o[4 * r] * inv, o[4 * r + 1] * inv, o[4 * r + 2] * inv,
                          o[4 * r + 3] * inv};
      if (job.slot >= 0)
        *reinterpret_cast<float4_t*>(a.part + slot * D + comp) = v;
      else if constexpr (EB == 4)
        *reinterpret_cast<float4_t*>(op + comp * 4) = v;
      else
        *reinterpret_cast<u32x2_t*>(op + comp * 2) =
            u32x2_t{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3])};
    }
  }
  lds_barrier();   // the joined results are read
}

// Many rows: four waves of 32 rows share tiles of 64 keys, widened to 16 bits once
// for all of them (each wave widening the keys that it meets, as few rows do: 8 x
// 2048 rows behind 4096 tokens, 32 / 8 heads of 128, 1500 us; shared: 820, 1.0
// PFLOP/s in bfloat16; matrix units 45 % busy, vector units 55, LDS 45, a quarter of
// that with bank conflicts).  64 rows
// a wave: 1009 instead of 848 us, one workgroup of eight waves: 1300.  A wave
// reads the codes of 16 rows of keys and of values a tile ahead into registers,
// and widens them into LDS a tile (keys: two) before they are used.  A power of
// two is taken into the widened numbers, which hold the product exactly.
// `General`, where a block that the workgroup reads is not there or has a scale
// for which they do not: scores and probabilities are multiplied instead.
constexpr int kManyRows = 128;
template <int DP> struct Wide {
  static constexpr int RAW = DP <= 64 ? 64 : 128;   // bytes of a row of codes
  static constexpr int RB = 2 * RAW, CPR = RB / 16;  // of a row of 16-bit numbers
  static constexpr int BN = 64, TILE = BN * RB;
  static constexpr int LOADS = 16 * RAW / 1024;      // 16 bytes a lane, of 16 rows
  static constexpr int LDS = 4 * TILE;
};
template <int CPR> __device__ __forceinline__ int k_swizzle16(int row) {
  return CPR == 16 ? row & 15 : (row >> 1) & 7;
}
template <int CPR> __device__ __forceinline__ int v_swizzle16(int row) {
  // (the lowest bit for the writes, of every second chunk of two or four rows at a time)
  return CPR == 16 ? (row & 3) << 2 | (row & 1) : ((row >> 1) & 1) * 5;
}
// Whether the scale is a power of two and all its products with codes, which are
// multiples of 2^-9 up to 448, are numbers of the 16-bit type (bfloat16: no denormal
// ones, and far enough from its largest for sums of them).
template <int DT> __device__ __forceinline__ bool folds(float s) {
  const bool power = (__builtin_bit_cast(uint32_t, s) & 0x007fffffu) == 0;
  return power && (DT == DT_F16 ? s >= 0x1p-15f && s <= 0x1p7f : s >= 0x1p-117f && s <= 0x1p100f);
}

struct Keys {
  static constexpr bool value = true;
};
struct Values {
  static constexpr bool value = false;
};

template <int DT, int CF, int DP, bool General>
__device__ __forceinline__ void attend_many(const CacheAttnArgs& a, const Job& job,
                                            unsigned char* lds) {
  using Z = Wide<DP>;
  constexpr int EB = Elem<DT>::bytes, RAW = Z::RAW, RB = Z::RB, CPR = Z::CPR, BN = Z::BN;
  constexpr int KS = DP / 16, DB = DP / 32, LOADS = Z::LOADS;
  // fp16 probabilities meet fp16 values, as in attention.hip: multiplied by 2^LIFT, so
  // that those down to 2^-36 of the largest count.  (General: values as codes in
  // bfloat16 and probabilities times their scales, which may be past fp16's range.)
  constexpr bool HALF = DT == DT_F16 && !General;
  constexpr int NQ = Terms<DT>::Q, KT = Terms<DT>::KT;
  constexpr int NP = HALF ? 1 : Terms<DT>::P, VT = HALF ? DT_F16 : DT_BF16;
  constexpr float SLACK = HALF ? 4.0f : 8.0f;   // log2 of how far a maximum may fall behind
  constexpr float LIFT = HALF ? 15.0f - SLACK : 0.0f;
  const CacheView& c = a.c;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int l32 = lane & 31, half = lane >> 5;
  const int D = c.D, hk = job.hk, len = job.e.len, t0 = job.t0, t1 = job.t1, n = t1 - t0;
  const int mask = (1 << c.log_block) - 1;

  // this lane's query
  const int first = (job.row_tile * 4 + wave) * 32, local = first + l32;
  const bool row_ok = local < job.e.rows;
  const int row = row_ok ? local : 0, qi = row / a.G, head = hk * a.G + row - qi * a.G;
  const int lim = a.causal ? len - job.e.n + qi + 1 : len;
  // every row of the wave sees the keys below this
  const int all = a.causal ? len - job.e.n + (first < job.e.rows ? first / a.G : 0) + 1 : len;
  const int whole = __builtin_amdgcn_readfirstlane(all < 0 ? 0 : all & ~31);
  const char* qp = a.q + (long long)(job.e.row0 + qi) * a.q_r + (long long)head * a.q_h;
  u32x4_t qf[NQ][KS];
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    const int el = (2 * s + half) * 8;
    u32x4_t raw[EB / 2];
#pragma unroll
    for (int i = 0; i < EB / 2; ++i) {
      raw[i] = u32x4_t{0, 0, 0, 0};
      if (row_ok && el < D)
        raw[i] = *reinterpret_cast<const u32x4_t*>(qp + el * EB + i * 16);
      if (a.flip) {
        const uint32_t sign = EB == 4 ? 0x80000000u : 0x80008000u;
        raw[i] = a.flip < 0 ? raw[i] ^ u32x4_t{sign, sign, sign, sign} : u32x4_t{0, 0, 0, 0};
      }
    }
    if constexpr (DT == DT_F32) {
      float f[8];
      unpack<DT_F32>(raw[0], f);
      unpack<DT_F32>(raw[1], f + 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t w[NQ];
        split2<NQ, true>(f[2 * j], f[2 * j + 1], w);
#pragma unroll
        for (int i = 0; i < NQ; ++i) qf[i][s][j] = w[i];
      }
    } else {
      qf[0][s] = raw[0];
    }
  }

  // This wave's rows of a tile: 16 from wave * 16 on, of one block.  Lane L holds
  // where those of tile i = L (mod 64) lie and their scales; half of the lanes are
  // filled again when their tiles are done.
  int rows = 0, where[2][2];
  float scales[2];
  const int* const table = c.table + (long long)job.b * c.width;
  auto locate = [&](int i) {
    const int p = (t0 + i) * BN + wave * 16, left = len - p;
    int id = -1;
    if (left > 0) id = table[p >> c.log_block];
    const bool any = id >= 0 && id < c.blocks;
    rows = !any ? 0 : left < 16 ? left : 16;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const long long off = any ? id * c.block[kv] + (p & mask) * c.token[kv] : 0;
      where[kv][0] = (int)off;
      where[kv][1] = (int)(off >> 32);
      scales[kv] = any ? c.scale[kv][(long long)id * c.Hk + hk] : 1.0f;
    }
  };
  locate(lane);
  auto scale_of = [&](int i, int kv) {
    return __builtin_bit_cast(
        float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, scales[kv]), i & 63));
  };
  // Of the general form: scales and addend of group L & 3 of tile i = L / 4 (mod 16).
  float by_k = 0.0f, by_v = 0.0f, addend = 0.0f;
  auto look = [&](int i) {
    const int p = (t0 + i + (lane >> 2)) * BN + (lane & 3) * 16;
    int id = -1;
    if (p < len) id = table[p >> c.log_block];
    const bool any = id >= 0 && id < c.blocks;
    by_k = any ? c.scale[0][(long long)id * c.Hk + hk] : 1.0f;
    by_v = any ? c.scale[1][(long long)id * c.Hk + hk] : 1.0f;
    addend = any || p >= len ? 0.0f : kNegInf;
  };
  auto group = [&](float v, int i, int g) {
    return __builtin_bit_cast(
        float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), (i & 15) * 4 + g));
  };

  // tile i's codes: 16 bytes of a row a lane; rows past the end and components from D
  // on arrive as zeros
  constexpr int LPR = RAW / 16, PASS = 64 / LPR;
  const int row_in = lane / LPR, chunk_in = lane % LPR;
  int off[2];
#pragma unroll
  for (int kv = 0; kv < 2; ++kv)
    off[kv] = chunk_in * 16 < D ? row_in * (int)c.token[kv] + chunk_in * 16 : kFarOffset;
  struct Part {
    u32x4_t codes[LOADS];
  };
  auto fetch = [&](int i, int kv) __attribute__((always_inline)) {
    const int have = __builtin_amdgcn_readlane(rows, i & 63);
    const uint32_t lo = __builtin_amdgcn_readlane(where[kv][0], i & 63);
    const int hi = __builtin_amdgcn_readlane(where[kv][1], i & 63);
    const __amdgpu_buffer_rsrc_t r =
        make_rsrc(c.codes[kv] + hk * c.head[kv] + (((long long)hi << 32) | lo),
                  i < n && have > 0 ? (uint32_t)((have - 1) * (int)c.token[kv] + D) : 0u);
    Part x;
#pragma unroll
    for (int j = 0; j < LOADS; ++j)
      x.codes[j] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                                   r, off[kv], j * PASS * (int)c.token[kv], 0));
    return x;
  };
  // where a lane's 16 codes go, of even and odd chunks
  int to[2][LOADS][2];
#pragma unroll
  for (int kv = 0; kv < 2; ++kv)
#pragma unroll
    for (int j = 0; j < LOADS; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = wave * 16 + j * PASS + row_in;
        to[kv][j][e] = kv * 2 * Z::TILE + row * RB +
                       ((2 * chunk_in + e) ^
                        (kv == 0 ? k_swizzle16<CPR>(row) : v_swizzle16<CPR>(row))) * 16;
      }
  // Widens tile i's; odd: i & 1, a constant where it is called.
  auto widen = [&](const Part& x, int i, int odd, auto keys) __attribute__((always_inline)) {
    constexpr int kv = decltype(keys)::value ? 0 : 1;
    const float scale = scale_of(i, kv);
#pragma unroll
    for (int j = 0; j < LOADS; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t w0 = x.codes[j][2 * e], w1 = x.codes[j][2 * e + 1];
        *reinterpret_cast<u32x4_t*>(lds + to[kv][j][e] + odd * Z::TILE) =
            General ? code_values16<CF, (kv == 0 ? KT : VT)>(w0, w1)
                    : code_values16<CF, KT>(w0, w1, scale);
      }
  };

  float16_t acc[DB];
  float m = kLowest, l = 0.0f, fall = 1.0f;
#pragma unroll
  for (int d = 0; d < DB; ++d) acc[d] = float16_t{};
  // LDS offsets that do not change from tile to tile
  const int krow = l32 * RB, ksw = (half ^ k_swizzle16<CPR>(l32)) * 16;
  const int i16 = lane & 15, vrow = 4 * half + (i16 >> 2);
  const int vchunk = ((lane >> 4) & 1) * 2 + ((i16 & 3) >> 1);
  using Probabilities = u32x4_t[NP][2];

  auto score = [&](const unsigned char* kt, int b, float16_t& s) __attribute__((always_inline)) {
    s = float16_t{};
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const u32x4_t kf =
          *reinterpret_cast<const u32x4_t*>(kt + krow + b * 32 * RB + (ksw ^ (ks * 32)));
#pragma unroll
      for (int i = 0; i < NQ; ++i) Mma<KT>::step(kf, qf[i][ks], s, 0);
    }
  };
  // scores of block b of tile i as they count
  auto settle = [&](int i, int b, float16_t& s) __attribute__((always_inline)) {
    if constexpr (General) {
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const float by = group(by_k, i, 2 * b + g), add = group(addend, i, 2 * b + g);
#pragma unroll
        for (int r = 0; r < 8; ++r) s[8 * g + r] = fmaf(s[8 * g + r], by, add);
      }
    }
    const int key0 = (t0 + i) * BN + b * 32;
    if (key0 + 32 > whole) {
      const int lane_lim = lim - key0 - 4 * half;
#pragma unroll
      for (int r = 0; r < 16; ++r)
        s[r] = (r & 3) + 8 * (r >> 2) < lane_lim ? s[r] : kNegInf;
    }
  };
  // The maximum moves only when it falls behind by 2^SLACK: the sums are hardly
  // ever rescaled.
  auto move_up = [&](const float16_t& s) __attribute__((always_inline)) {
    float top = s[0];
#pragma unroll
    for (int r = 1; r < 16; ++r) top = fmaxf(top, s[r]);
    top = swap_halves_max(top) * a.scale;
    const float m_new = top > m + SLACK ? top : m;
    fall = __builtin_amdgcn_exp2f(m - m_new);
    m = m_new;
    l *= fall;
  };
  auto probabilities = [&](int i, int b, float16_t& s, Probabilities& p)
      __attribute__((always_inline)) {
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      s[r] = __builtin_amdgcn_exp2f(fmaf(s[r], a.scale, LIFT - m));
      l += s[r];
    }
    if constexpr (General) {
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const float by = group(by_v, i, 2 * b + g);
#pragma unroll
        for (int r = 0; r < 8; ++r) s[8 * g + r] *= by;
      }
    }
#pragma unroll
    for (int r = 0; r < 16; r += 2) {
      uint32_t w[NP];
      if constexpr (NP == 1) w[0] = pack2<VT>(s[r], s[r + 1]);
      else split2<NP>(s[r], s[r + 1], w);
#pragma unroll
      for (int j = 0; j < NP; ++j) p[j][r >> 3][(r & 7) >> 1] = w[j];
    }
  };
  auto add_values = [&](const unsigned char* vt, int b, const Probabilities& p)
      __attribute__((always_inline)) {
#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
      for (int d = 0; d < DB; ++d) {
        const int chunk = (d * 4 + vchunk) ^ v_swizzle16<CPR>(vrow);
        const unsigned char* from = vt + (b * 32 + g * 16 + vrow) * RB + chunk * 16 + (i16 & 1) * 8;
        const u32x2_t lo = read_column(from), hi = read_column(from + 8 * RB);
        const u32x4_t vf = {lo[0], lo[1], hi[0], hi[1]};
#pragma unroll
        for (int j = 0; j < NP; ++j) Mma<VT>::step(vf, p[j][g], acc[d], 0);
      }
  };
  // (p is formed up to here: its first use is past a branch, where the compiler
  // would take its computation, away from the matrix instructions)
  auto follow = [&](Probabilities& p) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < NP; ++j) asm volatile("" : "+v"(p[j][0]), "+v"(p[j][1]), "+v"(l));
    if (__any(fall != 1.0f)) {
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[d][r] *= fall;
    }
  };

  // Pipelined over blocks of 32 keys: while the vector units form a block's
  // probabilities, the matrix units form the scores of the next block and add the
  // values of the block before, in the same wave.  Keys are therefore a tile ahead
  // of values.
  unsigned char* const kt = lds;
  unsigned char* const vt = lds + 2 * Z::TILE;
  if (n > 0) {
    float16_t s0, s1;       // scores of two blocks
    Probabilities p0, p1;       // probabilities of two blocks
    Part xk = fetch(0, 0), xv = fetch(0, 1);
    {
      const Part x = fetch(1, 0);
      if (General) look(0);
      widen(xk, 0, 0, Keys{});
      widen(xv, 0, 0, Values{});
      widen(x, 1, 1, Keys{});
    }
    xk = fetch(2, 0);
    xv = fetch(1, 1);
    lds_barrier();
    score(kt, 0, s0);
    score(kt, 1, s1);
    settle(0, 0, s0);
    move_up(s0);                // nothing to rescale yet
    probabilities(0, 0, s0, p0);
    // Tile i's second block and tile i + 1's first.  odd is i & 1, a constant where it
    // is called, so that the places' addresses are.
    auto two_blocks = [&](int i, int odd) __attribute__((always_inline)) {
      const unsigned char* k1 = kt + (1 - odd) * Z::TILE;
      const unsigned char* v0 = vt + odd * Z::TILE;
      // (waited for here, not where they are used in every tile)
      if ((i & 31) == 16 && i > 32 && i + 16 < n) {
        if ((lane >> 5) == ((i >> 5) - 1 & 1)) locate((i & ~31) + 32 + (lane & 31));
        asm volatile("" : "+v"(scales[0]), "+v"(scales[1]));
      }
      // keys of tile i + 1 and values of tile i lie there for all, and nobody reads
      // keys of tile i and values of tile i - 1 any more
      lds_barrier();
      settle(i, 1, s1);
      move_up(s1);
      score(k1, 0, s0);
      // behind the first matrix instructions
      widen(xk, i + 2, odd, Keys{});
      widen(xv, i + 1, 1 - odd, Values{});
      xk = fetch(i + 3, 0);
      xv = fetch(i + 2, 1);
      probabilities(i, 1, s1, p1);
      add_values(v0, 0, p0);
      follow(p1);
      if (General && (i & 15) == 15) {
        look(i + 1);
        asm volatile("" : "+v"(by_k), "+v"(by_v), "+v"(addend));
      }
      settle(i + 1, 0, s0);
      move_up(s0);
      score(k1, 1, s1);
      probabilities(i + 1, 0, s0, p0);
      add_values(v0, 1, p1);
      follow(p0);
    };
    int i = 0;
    for (; i + 2 < n; i += 2) {
      two_blocks(i, 0);
      two_blocks(i + 1, 1);
    }
    if (i + 1 < n) two_blocks(i, 0);
    const unsigned char* v0 = vt + ((n - 1) & 1) * Z::TILE;
    lds_barrier();
    settle(n - 1, 1, s1);
    move_up(s1);
    probabilities(n - 1, 1, s1, p1);
    add_values(v0, 0, p0);
    follow(p1);
    add_values(v0, 1, p1);
  }

  const int heads = c.Hk * a.G;
  const float sum = l + __shfl_xor(l, 32);
  if (!row_ok) return;
  const float inv = sum > 0.0f ? 1.0f / sum : sum;   // 0 keys: 0; a NaN stays
  const float lse2 = sum == 0.0f ? kNegInf : m + (__builtin_amdgcn_logf(sum) - LIFT);
  const long long t = job.e.row0 + qi, at = job.slot * kManyRows + wave * 32 + l32;
  if (half == 0) {
    if (job.slot >= 0) a.many_lse[at] = lse2;
    else if (a.lse) a.lse[t * heads + head] = lse2 * kLn2;
  }
  char* const op = a.out + t * a.o_r + head * a.o_h;
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int comp = d * 32 + 8 * r + 4 * half;
      if (comp >= D) continue;
      const float4_t o = {acc[d][4 * r] * inv, acc[d][4 * r + 1] * inv,
                          acc[d][4 * r + 2] * inv, acc[d][4 * r + 3] * inv};
      if (job.slot >= 0)
        *reinterpret_cast<float4_t*>(a.many + at * D + comp) = o;
      else if constexpr (EB == 4)
        *reinterpret_cast<float4_t*>(op + comp * 4) = o;
      else
        *reinterpret_cast<u32x2_t*>(op + comp * 2) =
            u32x2_t{pack2<DT>(o[0], o[1]), pack2<DT>(o[2], o[3])};
    }
}

// The unit of number x of the sets of `size` rows of the entries with more than a
// few (with `all`, of any), and of a key head.  a.sets: of every entry, some of them
// empty; 0: as many as each has, side by side.
struct Unit {
  Entry e;
  int b, hk, set, keys;   // keys: those that its last row sees
};
__device__ __forceinline__ bool unit_of(const CacheAttnArgs& a, int number, int size, int all,
                                        Unit* u) {
  const int x = number / a.c.Hk;
  u->hk = number - x * a.c.Hk;
  if (a.sets > 0) {
    u->b = x / a.sets;
    if (u->b >= a.c.B) return false;
    u->e = entry_of(a, u->b);
    u->set = a.sets - 1 - (x - u->b * a.sets);   // causal: the longest first
    if ((!all && few(u->e)) || u->set * size >= u->e.rows) return false;
  } else {
    auto weight = [=](const Entry& e) { return all || !few(e) ? (e.rows + size - 1) / size : 0; };
    Entries<decltype(weight)> entries(a, weight);
    const auto f = entries.find(x);
    if (f.b >= a.c.B) return false;
    u->b = f.b;
    u->e = f.e;
    u->set = f.weight - 1 - (x - (int)f.first);
  }
  const int end = (u->set + 1) * size, last = (end < u->e.rows ? end : u->e.rows) - 1;
  const int keys = a.causal ? u->e.len - u->e.n + last / a.G + 1 : u->e.len;
  u->keys = keys > 0 ? keys : 0;
  return true;
}

// Entries of few rows: the tiles of all their key heads in a row, entry after
// entry, each workgroup a run of them of one length (so that entries of very
// different lengths fill the GPU to the end).  A head whose tiles lie in one run
// is written at once, of others the runs' parts are joined (join_few).  64 entries
// of 1 to 8192 keys and 8 heads of 128, 540 MB: 117 us, where one workgroup takes 95
// for the longest entry alone.
template <int DT, int CF, int DP>
__device__ __forceinline__ void few_run(const CacheAttnArgs& a, int group, unsigned char* lds) {
  Job job;
  job.row_tile = 0;
  if (a.few_groups == 0) {
    job.b = group / a.c.Hk;
    job.hk = group - job.b * a.c.Hk;
    job.e = entry_of(a, job.b);
    job.t0 = 0;
    job.t1 = few_tiles(job.e);
    job.slot = -1;
    if (job.t1 > 0) attend_few<DT, CF, DP>(a, job, lds);
    return;
  }
  auto weight = [](const Entry& e) { return few_units(e); };
  Entries<decltype(weight)> entries(a, weight);
  const int Hk = a.c.Hk;
  const long long total = entries.total() * Hk, per = share_of(total, a.few_groups);
  long long x = group * per;
  const long long begin = x, end = x + per < total ? x + per : total;
  while (x < end) {
    const auto f = entries.find(x / Hk);
    job.b = f.b;
    job.e = f.e;
    // the entry's heads one after another
    while (x < end && x < (f.first + f.weight) * Hk) {
      const int in = (int)(x - f.first * Hk);
      job.hk = in / f.weight;
      const int from = in - job.hk * f.weight;
      const int to = f.weight - from < end - x ? f.weight : from + (int)(end - x);
      job.t0 = from > kStart ? from - kStart : 0;
      job.t1 = to - kStart;
      job.slot = job.t0 == 0 && to == f.weight ? -1 : 2LL * group + (x == begin ? 0 : 1);
      if (job.t1 > job.t0) attend_few<DT, CF, DP>(a, job, lds);
      x += to - from;
    }
  }
}

// `units` workgroups of 32 rows of a key head, for calls that have few such sets and
// few keys, and behind them those of the entries of few rows.
template <int DT, int CF, int DP>
__global__ __launch_bounds__(kFewThreads, 2) void few_kernel(const CacheAttnArgs a, int units,
                                                             int all) {
  __shared__ __attribute__((aligned(1024))) unsigned char lds[Shape<DP>::LDS];
  if ((int)blockIdx.x >= units) {
    few_run<DT, CF, DP>(a, blockIdx.x - units, lds);
    return;
  }
  Unit u;
  if (!unit_of(a, blockIdx.x, 32, all, &u)) return;
  const Job job = {u.e, u.b, u.hk, u.set, 0, (u.keys + kTile - 1) / kTile, -1};
  attend_few<DT, CF, DP>(a, job, lds);
}

// Shares of a set's keys: up to a.splits, of kShare tiles at least.  (As many of every
// set: prompts of 600 rows with 2000 keys beside 20 single tokens 56 us, like this 41;
// 512 rows with 16384 keys beside 512 139 and 124.  4 or 8 tiles: the same within 3 %.)
constexpr int kShare = 6;
__device__ __forceinline__ int shares_of(const CacheAttnArgs& a, const Unit& u, int tile) {
  const int s = (u.keys + tile - 1) / tile / kShare;
  return s < 1 ? 1 : s > a.splits ? a.splits : s;
}

// `units` sets of 128 rows of a key head, the keys in up to a.splits shares, a workgroup
// each, and behind them the workgroups of the entries of few rows, which fill the
// GPU while the last sets end.
template <int DT, int CF, int DP>
__global__ __launch_bounds__(kThreads, 2) void many_kernel(const CacheAttnArgs a, int units,
                                                           int all) {
  using Z = Wide<DP>;
  __shared__ __attribute__((aligned(1024))) unsigned char
      lds[Z::LDS > Shape<DP>::LDS ? Z::LDS : Shape<DP>::LDS];
  if ((int)blockIdx.x >= units * a.splits) {
    few_run<DT, CF, DP>(a, blockIdx.x - units * a.splits, lds);
    return;
  }
  const int split = blockIdx.x / units, unit = blockIdx.x - split * units;
  Unit u;
  // (consecutive workgroups, which lie on different XCDs, are of different heads: an
  // XCD then reads few heads of every entry, however long each is.  With an XCD to
  // an entry the longest one held up the end.)
  if (!unit_of(a, unit, kManyRows, all, &u)) return;
  const CacheView& c = a.c;
  const int tiles = (u.keys + Z::BN - 1) / Z::BN, shares = shares_of(a, u, Z::BN);
  if (split >= shares) return;
  const Job job = {u.e,
                   u.b,
                   u.hk,
                   u.set,
                   (int)((long long)tiles * split / shares),
                   (int)((long long)tiles * (split + 1) / shares),
                   shares > 1 ? (long long)split * units + unit : -1};
  // whether all blocks are there, with scales that the widened numbers can take in
  bool plain = true;
  const int last = job.t1 * Z::BN < u.e.len ? job.t1 * Z::BN : u.e.len;
  const int b0 = (job.t0 * Z::BN) >> c.log_block;
  const int b1 = (last + (1 << c.log_block) - 1) >> c.log_block;
  for (int i = b0 + threadIdx.x; i < b1; i += kThreads) {
    const int id = c.table[(long long)u.b * c.width + i];
    if (id < 0 || id >= c.blocks) {
      plain = false;
    } else {
      const long long at = (long long)id * c.Hk + u.hk;
      plain = plain && folds<DT>(c.scale[0][at]) && folds<DT>(c.scale[1][at]);
    }
  }
  if (__syncthreads_and(plain)) attend_many<DT, CF, DP, false>(a, job, lds);
  else attend_many<DT, CF, DP, true>(a, job, lds);
}

// Adds U parts (their sums' log2 and normed outputs) to a maximum, a sum and outputs.
template <int U>
__device__ __forceinline__ void take_parts(const float* w, const float4_t* v, float* m, float* sum,
                                           float4_t* o) {
  float m_new = *m;
#pragma unroll
  for (int i = 0; i < U; ++i) m_new = fmaxf(m_new, w[i]);
  const float fall = __builtin_amdgcn_exp2f(*m - m_new);
  *m = m_new;
  *sum *= fall;
  *o *= fall;
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const float p = __builtin_amdgcn_exp2f(w[i] - m_new);
    *sum += p;
#pragma unroll
    for (int j = 0; j < 4; ++j) (*o)[j] = fmaf(p, v[i][j], (*o)[j]);
  }
}

// Joins the parts of a row of the key head in which run number g + 1 begins, if
// its first keys are of run g: out = sum_s 2^(lse_s - lse) o_s.  (Not a workgroup
// for each head's rows, of which there may be far more than runs.)  LPR lanes a
// part, 4 components a lane; the workgroup's sets of lanes take parts in turn and
// meet in LDS, in order.  (A workgroup takes every kRows-th row.)
constexpr int kRows = 4;
template <int DT, int LPR>
__device__ __forceinline__ void join_few(const CacheAttnArgs& a, int g, int part) {
  constexpr int SETS = kThreads / LPR;
  __shared__ float tops[SETS], sums[SETS];
  __shared__ float4_t outs[SETS][LPR];
  const int Hk = a.c.Hk, D = a.c.D;
  auto weight = [](const Entry& x) { return few_units(x); };
  Entries<decltype(weight)> entries(a, weight);
  const long long total = entries.total() * Hk, per = share_of(total, a.few_groups);
  const long long x = (g + 1) * per;
  if (x >= total) return;
  const auto f = entries.find(x / Hk);
  const Entry e = f.e;
  const int hk = (int)(x - f.first * Hk) / f.weight;
  const long long u0 = f.first * Hk + (long long)hk * f.weight;
  const int g0 = (int)((u0 + kStart) / per), g1 = (int)((u0 + f.weight - 1) / per);
  if (g0 != g || g1 == g) return;
  const int set = threadIdx.x / LPR, lane = threadIdx.x % LPR;
  const bool live = 4 * lane < D;
  for (int row = part; row < e.rows; row += kRows) {
    float m = kLowest, sum = 0.0f;
    float4_t o = {0.0f, 0.0f, 0.0f, 0.0f};
    constexpr int U = 4;   // parts that are on their way at a time
    for (int g = g0 + set; g <= g1; g += U * SETS) {
      float w[U];
      float4_t v[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int gi = g + i * SETS;
        // a run's first part is its slot 0
        const long long slot = (2LL * gi + (gi == g0 && u0 > g0 * per ? 1 : 0)) * kFewRows + row;
        w[i] = kNegInf;
        v[i] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
        if (gi <= g1) {
          w[i] = a.part_lse[slot];
          if (live) v[i] = *reinterpret_cast<const float4_t*>(a.part + slot * D + 4 * lane);
        }
      }
      take_parts<U>(w, v, &m, &sum, &o);
    }
    __syncthreads();   // the last row's are read
    if (lane == 0) {
      tops[set] = m;
      sums[set] = sum;
    }
    outs[set][lane] = o;
    __syncthreads();
    if (set > 0) continue;
    float m_all = m;
#pragma unroll
    for (int s = 1; s < SETS; ++s) m_all = fmaxf(m_all, tops[s]);
    sum = 0.0f;
    o = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int s = 0; s < SETS; ++s) {
      const float p = __builtin_amdgcn_exp2f(tops[s] - m_all);
      sum = fmaf(sums[s], p, sum);
      const float4_t v = outs[s][lane];
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = fmaf(p, v[j], o[j]);
    }
    const float inv = sum > 0.0f ? 1.0f / sum : sum;
    const int qi = row / a.G, head = hk * a.G + row - qi * a.G;
    const long long t = e.row0 + qi;
    if (a.lse && lane == 0)
      a.lse[t * (Hk * a.G) + head] =
          sum == 0.0f ? kNegInf : (m_all + __builtin_amdgcn_logf(sum)) * kLn2;
    if (!live) continue;
    char* op = a.out + t * a.o_r + head * a.o_h;
    if constexpr (DT == DT_F32)
      *reinterpret_cast<float4_t*>(op + 16 * lane) = o * inv;
    else
      *reinterpret_cast<u32x2_t*>(op + 8 * lane) =
          u32x2_t{pack2<DT>(o[0] * inv, o[1] * inv), pack2<DT>(o[2] * inv, o[3] * inv)};
  }
}

// Joins the splits of the rows of a set, the workgroup `part` of kParts of it: LPR
// lanes a row, 4 components a lane.
constexpr int kParts = 4;
template <int DT, int LPR>
__device__ __forceinline__ void join_many(const CacheAttnArgs& a, int units, int unit, int part,
                                          int all) {
  Unit u;
  if (!unit_of(a, unit, kManyRows, all, &u)) return;
  const int shares = shares_of(a, u, Wide<128>::BN);
  if (shares == 1) return;
  const int lane = threadIdx.x % LPR, D = a.c.D, heads = a.c.Hk * a.G;
  const bool live = 4 * lane < D;
  for (int r = threadIdx.x / LPR + part * (kThreads / LPR); r < kManyRows;
       r += kParts * (kThreads / LPR)) {
    const int row = u.set * kManyRows + r;
    if (row >= u.e.rows) return;
    const int qi = row / a.G, head = u.hk * a.G + row - qi * a.G;
    const long long t = u.e.row0 + qi, step = (long long)units * kManyRows;
    const long long at = (long long)unit * kManyRows + r;
    float m = kLowest, sum = 0.0f;
    float4_t o = {0.0f, 0.0f, 0.0f, 0.0f};
    constexpr int U = 4;
    for (int s = 0; s < shares; s += U) {
      float w[U];
      float4_t v[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        w[i] = kNegInf;
        v[i] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
        if (s + i < shares) {
          w[i] = a.many_lse[(s + i) * step + at];
          if (live)
            v[i] =
                *reinterpret_cast<const float4_t*>(a.many + ((s + i) * step + at) * D + 4 * lane);
        }
      }
      take_parts<U>(w, v, &m, &sum, &o);
    }
    const float inv = sum > 0.0f ? 1.0f / sum : sum;
    if (a.lse && lane == 0)
      a.lse[t * heads + head] = sum == 0.0f ? kNegInf : (m + __builtin_amdgcn_logf(sum)) * kLn2;
    if (!live) continue;
    char* op = a.out + t * a.o_r + head * a.o_h;
    if constexpr (DT == DT_F32)
      *reinterpret_cast<float4_t*>(op + 16 * lane) = o * inv;
    else
      *reinterpret_cast<u32x2_t*>(op + 8 * lane) =
          u32x2_t{pack2<DT>(o[0] * inv, o[1] * inv), pack2<DT>(o[2] * inv, o[3] * inv)};
  }
}

// What has parts: kParts workgroups for each of `units` sets, and behind them, for each
// run but the last of the few rows, `rows` of them, kRows if there are that many.
template <int DT, int LPR>
__global__ __launch_bounds__(kThreads) void join_kernel(const CacheAttnArgs a, int units, int rows,
                                                        int all) {
  const int x = blockIdx.x;
  if (x < units * kParts) {
    join_many<DT, LPR>(a, units, x / kParts, x & (kParts - 1), all);
  } else {
    const int y = x - units * kParts;
    join_few<DT, LPR>(a, y / rows, y % rows);
  }
}

// Sets of `size` rows of a key head that a batch may have: of each entry, or side by
// side, which takes a look at all entries' rows (64 at a time).
long long sets_of_each(const CacheAttnArgs& a, long long size) {
  return ((long long)a.max_rows * a.G + size - 1) / size;
}
long long row_sets(const CacheAttnArgs& a, long long size) {
  const long long each = sets_of_each(a, size) * a.c.B, all = (long long)a.T * a.G / size + a.c.B;
  return each < all ? each : all;
}

template <int DT, int CF, int DP>
void launch(const CacheAttnArgs& a, hipStream_t stream) {
  constexpr int LPR = DP <= 64 ? 16 : 32;
  const long long most = (long long)a.max_rows * a.G;
  // all entries have the most rows, or (rows of no entry) none does
  const int all = most > kFewRows && (long long)a.T == (long long)a.max_rows * a.c.B;
  const int groups = all || a.G > kFewRows ? 0 : a.few_groups > 0 ? a.few_groups : a.c.B * a.c.Hk;
  const int units = a.units;
  if (a.set == kManyRows)
    hipLaunchKernelGGL((many_kernel<DT, CF, DP>), dim3((unsigned)(units * a.splits + groups)),
                       dim3(kThreads), 0, stream, a, units, all);
  else
    hipLaunchKernelGGL((few_kernel<DT, CF, DP>), dim3((unsigned)(units + groups)),
                       dim3(kFewThreads), 0, stream, a, units, all);
  const int sets = a.splits > 1 ? units : 0, rows = most < kRows ? (int)most : kRows;
  const int runs = groups > 0 && a.few_groups > 0 ? a.few_groups - 1 : 0;
  if (sets + runs > 0)
    hipLaunchKernelGGL((join_kernel<DT, LPR>), dim3((unsigned)(sets * kParts + runs * rows)),
                       dim3(kThreads), 0, stream, a, sets, rows, all);
}

template <int DT, int CF> void launch_cf(const CacheAttnArgs& a, hipStream_t stream) {
  if (a.c.D <= 64) launch<DT, CF, 64>(a, stream);
  else if (a.c.D <= 96) launch<DT, CF, 96>(a, stream);
  else launch<DT, CF, 128>(a, stream);
}
template <int DT> void launch_dt(const CacheAttnArgs& a, int format, hipStream_t stream) {
  if (format == LIBCONV_CACHE_I8) launch_cf<DT, LIBCONV_CACHE_I8>(a, stream);
  else launch_cf<DT, LIBCONV_CACHE_E4M3>(a, stream);
}

}  // namespace

long long cache_attn_plan(CacheAttnArgs* a, int dtype, int cus, bool allowed) {
  a->few_groups = 0;
  a->splits = 1;
  a->set = 32;
  a->sets = 0;
  a->units = 0;
  if (a->T == 0 || a->c.B == 0) return 0;
  const long long keys = (long long)a->c.width << a->c.log_block;
  const bool many = (long long)a->max_rows * a->G > kFewRows;
  if (many) {
    // Sets of 128 rows, each with its keys in up to as many shares as make 4 workgroups
    // a compute unit: 9 entries of 517 rows in all behind up to 4096
    // keys, 4 heads of 80 in fp16: 67 us; 2 a unit 77, 3: 69, 6: 71.  Shares of 512 keys or
    // more, past 32 of them of 2048 (what they leave has to be joined): 16 rows of 4 heads of 128,
    // 131072 keys, bfloat16, 16 shares 194 us, 32: 112, 64: 84, 128: 100; 100 rows of 2 heads, 32768
    // keys 68, 60, 75 us.
    const long long n = row_sets(*a, kManyRows) * a->c.Hk;
    const long long of512 = keys / 512 < 32 ? keys / 512 : 32, of2048 = keys / 2048;
    long long s = 4LL * cus / n;
    if (s > (of512 > of2048 ? of512 : of2048)) s = of512 > of2048 ? of512 : of2048;
    if (s < 1 || !allowed) s = 1;
    // Where that is not one for every second unit, sets of 32 rows, a workgroup with all
    // keys of its set each: 2 entries of 130 rows and 8 heads of 64, 520 keys, fp32: 13 us, with
    // sets of 128 rows 25.  But only while there are few keys: 16 rows of 4 heads of 128,
    // sets of 32 / 128 rows, 1024 keys 17 / 22 us, 2048: 27 / 23, 8192: 87 / 28, 131072: 1289 / 84;
    // one token of 64 heads that share one, 1024: 16 / 21, 2048: 26 / 22, 131072: 1283 / 81.
    if (n * s >= cus / 2 || s >= 4) {
      a->set = kManyRows;
      a->splits = (int)s;
    }
    // Empty sets of an entry end at once, but each takes a workgroup; where only some
    // entries have many rows, sets side by side have each workgroup look over all
    // entries.  One prompt of 600 rows among others of 1 to 39, 2 heads of 64, side by
    // side / of each entry: 300 entries 29 / 39 us, 700 56 / 76, 2000 258 / 197.
    const long long each = sets_of_each(*a, a->set) * a->c.B;
    // (2^24 workgroups of 256 lanes are the most of a launch)
    if ((each + a->c.B) * a->c.Hk < (1 << 24) - 4096 &&
        (each <= 2 * row_sets(*a, a->set) || a->c.B > 1024))
      a->sets = (int)sets_of_each(*a, a->set);
  }
  // Few rows share their keys where the longest head alone may take longer than all
  // together.  Heads of 128, ragged entries, shared / alone: up to 1100 keys, 32
  // heads 15 / 18 us, 256 heads 24 / 19; up to 2048, 128 heads 22 / 28, 256 heads 31 / 30;
  // up to 8192, 32 heads 26 / 94, 512 heads 115 / 128, 1024 heads 228 / 250.  Heads of 64:
  // up to 2048 keys, 64 heads 16 / 19, 256 heads 27 / 20.
  if (allowed && a->G <= kFewRows && keys >= 1024 && keys >= 16LL * a->c.B * a->c.Hk)
    a->few_groups = 2 * cus;
  if (many)
    a->units = (int)((a->sets > 0 ? (long long)a->sets * a->c.B : row_sets(*a, a->set)) * a->c.Hk);
  const long long rows = a->splits > 1 ? (long long)a->units * kManyRows * a->splits : 0;
  return (2LL * a->few_groups * kFewRows + rows) * (a->c.D + 1) * 4;
}

void cache_attn_place(CacheAttnArgs* a, char* workspace) {
  const long long few = 2LL * a->few_groups * kFewRows;
  const long long rows = (long long)a->units * kManyRows * a->splits;
  a->part = reinterpret_cast<float*>(workspace);
  a->many = a->part + few * a->c.D;
  a->part_lse = a->many + (a->splits > 1 ? rows * a->c.D : 0);
  a->many_lse = a->part_lse + few;
}

libconv_status cache_attn_launch(CacheAttnArgs a, int format, int dtype, hipStream_t stream) {
  if (dtype == LIBCONV_F32) launch_dt<DT_F32>(a, format, stream);
  else if (dtype == LIBCONV_F16) launch_dt<DT_F16>(a, format, stream);
  else launch_dt<DT_BF16>(a, format, stream);
  return hipGetLastError() == hipSuccess ? LIBCONV_OK : LIBCONV_ERR_LAUNCH;
}

}  // namespace libconv
