// attention.hip -- attention of a batch over keys all entries share (the
// prefix) and each entry's own keys.
//
//   out = sum_j p_j v_j,  p = softmax_j(scale <q, k_j>)
//
// One pass over the keys with the running maximum m and sum l of a softmax:
// for a tile of keys S = K Q^T, m' = max(m, S), O = O 2^(m - m') + V^T 2^(S - m').
// The products are formed transposed (keys and head components on the rows of
// the matrix instructions, queries on their columns): a lane then holds
// scores, maximum, sum and outputs of one query only, so nothing but the
// maximum crosses lanes, and the scores of 4 consecutive keys a lane holds
// are what the second product wants from it if V's rows are read in the same
// order (the transposing LDS read gives 4 consecutive keys of one component).
//
// Rows: the queries of all heads that share a key head lie side by side (row
// = ((entry, query), head of the group)), 32 to a wave.  A workgroup of four
// waves holds 128, 64 or 32 rows; with fewer rows the waves share a row block
// and split the keys of a tile (WK), and join at the end through LDS.
#include "device_common.h"
#include "layer.h"

namespace libconv {
namespace {

constexpr int kThreads = 256;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -__builtin_inff();
constexpr float kLowest = -3.402823466e38f;   // the maximum of no keys: finite, so that no
                                              // difference of maxima is a NaN
constexpr float kSlack = 8.0f;   // log2 of how far a maximum may fall behind

template <int DT, int DP, int WK> struct Shape {
  static constexpr int EB = Elem<DT>::bytes;
  static constexpr int RB = (DP <= 64 ? 64 : 128) * EB;    // bytes of a row of K or V in LDS
  static constexpr int CPR = RB / 16;                      // 16-byte chunks of it
  static constexpr int KPW = EB == 4 ? 32 : WK == 1 ? 64 : 32;  // keys a wave takes of a tile
  static constexpr int BN = KPW * WK;                      // keys of a tile
  static constexpr int ROWS = 128 / WK;                    // rows of a workgroup
  static constexpr int TILE = BN * RB;
  static constexpr int LDS = 4 * TILE;                     // K and V, two stages
  static constexpr int WAVES = 2 * LDS <= 160 * 1024 ? 2 : 1;   // workgroups a compute unit, at least
};

typedef short s16x4_t __attribute__((ext_vector_type(4)));

// 16-byte chunk of a row of K (V) in LDS is kept at chunk ^ swizzle(row): the
// 16 lanes that read one chunk of 16 rows at a time then hit all banks (in
// rows of 512 bytes, twice: a copy covers 8 rows there, and a thread's chunk
// is the same for all of its copies; the fp32 product is far slower anyway).
template <int CPR> __device__ __forceinline__ int k_swizzle(int row) {
  return CPR == 32 ? row & 7 : CPR == 16 ? row & 15 : (row >> 1) & 7;
}
// V is read 64 contiguous bytes of each of 4 rows at a time (16-bit types), or
// 128 bytes of two rows 4 apart (fp32).
template <int EB, int CPR> __device__ __forceinline__ int v_swizzle(int row) {
  if constexpr (EB == 4) return ((row >> 2) & 1) << 3;
  return CPR >= 16 ? (row & 3) << 2 : ((row >> 1) & 1) << 2;
}

// The larger of v in this lane and in the lane 32 away.
__device__ __forceinline__ float swap_halves_max(float v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return fmaxf(__builtin_bit_cast(float, r[0]), __builtin_bit_cast(float, r[1]));
}

// 4 elements of one column of 16-bit elements: the 16 lanes of a quarter wave
// name 8 bytes each of 4 rows.  `p` is restrict so that the read has a scope of
// its own: without one, the compiler lets it wait for every copy to LDS that
// is on its way, those of the next tile among them.
__device__ __forceinline__ u32x2_t read_column(const unsigned char* __restrict p) {
  return __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                         (__attribute__((address_space(3))) s16x4_t*)p));
}

// Lane's 4 probabilities -> 2 words of the 16-bit type.
template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  const f32x2_t v = {a, b};
  if constexpr (DT == DT_F16) {
    typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, half2_t));
  } else {
    typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
  }
}

// A walk over a workgroup's tiles of K or of V: prefix, then own keys.
struct Cursor {
  const char* p;        // row 0 of the tile
  int stride;           // of its rows in bytes (below 2^24)
  int left;             // rows from there to the end of the run; <= 0 past the end
  int off;              // this lane's bytes of its first row, past any end without such
  const char* own_p;    // the own keys' first tile, where the run follows
  int own_stride, own_left, own_off;
};

// Copies a tile's rows into LDS, 16 bytes a lane, and moves on.  Rows past the
// run's end and components from D on arrive as zeros: they lie past the
// resource's end (rows that lie closer than their own length repeat bytes of
// valid rows instead, whose scores are masked).
template <int DT, int DP, int WK, bool V>
__device__ __forceinline__ void copy_tile(Cursor& c, unsigned char* lds, int row_bytes) {
  using Z = Shape<DT, DP, WK>;
  constexpr int PASS = kThreads / Z::CPR;   // rows of a copy of the workgroup
  const int rows = c.left < Z::BN ? c.left : Z::BN;
  const __amdgpu_buffer_rsrc_t r =
      make_rsrc(c.p, rows > 0 ? (uint32_t)((rows - 1) * c.stride + row_bytes) : 0u);
  unsigned char* to = lds + __builtin_amdgcn_readfirstlane(threadIdx.x & ~63) * 16;
#pragma unroll
  for (int j = 0; j < Z::BN / PASS; ++j)
    copy16_to_lds(r, to + j * kThreads * 16, c.off, j * PASS * c.stride);
  c.p += (long long)Z::BN * c.stride;
  c.left -= Z::BN;
  if (c.left <= 0) {   // the own keys; past them there is nothing
    c.p = c.own_p;
    c.stride = c.own_stride;
    c.left = c.own_left;
    c.off = c.own_off;
    c.own_left = 0;
  }
}

// What a workgroup computes: rows [row0, row0 + rows) of key head hk (rows are
// counted over the entries), prefix keys [0, P) and own keys of entry b, of
// whose tiles it takes share `split` of `splits`; slot: where its partial
// result goes (-1: straight to the output).
struct Job {
  int row0, rows, hk, b;
  bool prefix, own;
  int split, splits, slot;
};

template <int DT, int DP, int WK>
__device__ __forceinline__ void attend(const AttnArgs& a, const Job& job, unsigned char* lds) {
  using Z = Shape<DT, DP, WK>;
  constexpr int EB = Z::EB, RB = Z::RB, CPR = Z::CPR, KPW = Z::KPW, BN = Z::BN;
  constexpr int KS = DP * EB / 32;  // steps of the first product
  constexpr int NB = KPW / 32;      // blocks of 32 keys a wave
  constexpr int DB = DP / 32;       // blocks of 32 components
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int l32 = lane & 31, half = lane >> 5;
  const int wr = wave / WK, wk = wave % WK;   // row block, key share
  const int row_bytes = a.D * EB, d_chunks = row_bytes / 16;

  // this lane's query
  const int local = wr * 32 + l32;
  const bool row_ok = local < job.rows;
  const int row = job.row0 + (row_ok ? local : 0);
  const int per_entry = a.Sq * a.G;
  const int qb = row / per_entry, in_entry = row % per_entry;
  const int qi = in_entry / a.G, qg = in_entry % a.G;
  const char* qp = a.q + qb * a.q_b + qi * a.q_r + (long long)(job.hk * a.G + qg) * a.q_h;
  u32x4_t qf[KS];
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    const int chunk = 2 * s + half;
    qf[s] = u32x4_t{0, 0, 0, 0};
    if (row_ok && chunk < d_chunks) qf[s] = *reinterpret_cast<const u32x4_t*>(qp + chunk * 16);
    if (a.flip) {
      const uint32_t sign = EB == 4 ? 0x80000000u : 0x80008000u;
      qf[s] = a.flip < 0 ? qf[s] ^ u32x4_t{sign, sign, sign, sign} : u32x4_t{0, 0, 0, 0};
    }
  }

  // own keys of the entry, and how many of them this query sees
  int n_own = 0, lim = 0, lim_wave = 0, end_own = 0;
  if (job.own) {
    n_own = a.lengths[job.b];
    n_own = n_own < 0 ? 0 : n_own > a.S ? a.S : n_own;
    lim = lim_wave = end_own = n_own;
    if (a.causal) {
      const int first = (job.row0 + wr * 32) % per_entry;   // the wave's first row, as it may be
      const int last = (job.row0 + job.rows - 1) % per_entry;
      lim = n_own - a.Sq + qi + 1;
      lim_wave = n_own - a.Sq + first / a.G + 1;
      end_own = n_own - a.Sq + last / a.G + 1;
      if (end_own < 0) end_own = 0;
    }
  }
  const int tiles_p = job.prefix ? (a.P + BN - 1) / BN : 0;
  const int tiles = tiles_p + (end_own + BN - 1) / BN;
  const int t0 = (int)((long long)tiles * job.split / job.splits);
  const int t1 = (int)((long long)tiles * (job.split + 1) / job.splits);

  const char* kp = a.kp + job.hk * a.kp_h;
  const char* vp = a.vp + job.hk * a.vp_h;
  const char* ko = a.k + job.b * a.k_b + job.hk * a.k_h;
  const char* vo = a.v + job.b * a.v_b + job.hk * a.v_h;
  // a thread's rows of a copy lie a multiple of 16 (rows of 512 bytes: 8) apart: its
  // chunk of them is the same for all
  const int c_row = threadIdx.x / CPR, c_slot = threadIdx.x % CPR;
  auto cursor = [&](const char* p, long long stride, const char* o, long long own_stride,
                    int chunk) {
    Cursor c;
    c.own_p = o;
    c.own_stride = (int)own_stride;
    c.own_left = end_own;
    c.own_off = chunk < d_chunks ? c_row * (int)own_stride + chunk * 16 : kFarOffset;
    c.p = p + (long long)t0 * BN * stride;
    c.stride = (int)stride;
    c.left = a.P - t0 * BN;
    c.off = chunk < d_chunks ? c_row * (int)stride + chunk * 16 : kFarOffset;
    if (t0 >= tiles_p) {
      c.p = o + (long long)(t0 - tiles_p) * BN * own_stride;
      c.stride = (int)own_stride;
      c.left = end_own - (t0 - tiles_p) * BN;
      c.off = c.own_off;
      c.own_left = 0;
    }
    return c;
  };
  static_assert(kThreads / CPR % (CPR == 32 ? 8 : 16) == 0, "one swizzle for a thread's rows");
  Cursor ck = cursor(kp, a.kp_r, ko, a.k_r, c_slot ^ k_swizzle<CPR>(c_row));
  Cursor cv = cursor(vp, a.vp_r, vo, a.v_r, c_slot ^ v_swizzle<EB, CPR>(c_row));

  float16_t acc[DB];
#pragma unroll
  for (int d = 0; d < DB; ++d) acc[d] = float16_t{};
  float m = kLowest, l = 0.0f;   // maximum (times scale, log2) and sum of this lane's half

  // LDS offsets that do not change from tile to tile
  const int krow = (wk * KPW + l32) * RB;
  const int ksw = (half ^ k_swizzle<CPR>(l32)) * 16;
  const int i16 = lane & 15;
  const int vrow16 = 4 * half + (i16 >> 2);
  const int vchunk16 = ((lane >> 4) & 1) * 2 + ((i16 & 3) >> 1);

  // scores of a block of 32 keys of a tile, key on the rows, query on the columns
  auto score = [&](const unsigned char* kt, int b, float16_t& s) {
    s = float16_t{};
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const u32x4_t kf = *reinterpret_cast<const u32x4_t*>(kt + krow + b * 32 * RB +
                                                           (ksw ^ (ks * 32)));
#pragma unroll
      for (int e = 0; e < Mma<DT>::KSUB; ++e) Mma<DT>::step(kf, qf[ks], s, e);
    }
  };
  // keys past the end and keys the causal mask hides; key0: the block's first
  auto mask = [&](int t, int b, float16_t& s) {
    const bool own = t >= tiles_p;
    const int key0 = (own ? t - tiles_p : t) * BN + wk * KPW + b * 32;
    if (key0 + 32 > (own ? lim_wave : a.P)) {
      const int lane_lim = (own ? lim : a.P) - key0 - 4 * half;
#pragma unroll
      for (int r = 0; r < 16; ++r)
        s[r] = (r & 3) + 8 * (r >> 2) < lane_lim ? s[r] : kNegInf;
    }
  };
  auto top_of = [&](const float16_t& s) {
    float top = s[0];
#pragma unroll
    for (int r = 1; r < 16; ++r) top = fmaxf(top, s[r]);
    return swap_halves_max(top) * a.scale;
  };
  // probabilities times 2^(their maximum - m), added to the sum
  auto probabilities = [&](float16_t& s) {
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      s[r] = __builtin_amdgcn_exp2f(fmaf(s[r], a.scale, -m));
      l += s[r];
    }
  };
  auto rescale = [&](float f) {
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[d][r] *= f;
  };
  // 16 keys a step of the second product: this lane's are 4 half + {0..3, 8..11}
  auto pack = [&](const float16_t& s, u32x4_t* pf) {
    if constexpr (EB == 2) {
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) pf[c][e] = pack2<DT>(s[c * 8 + 2 * e], s[c * 8 + 2 * e + 1]);
    }
  };
  auto add_values = [&](const unsigned char* vt, int b, const u32x4_t* pf) {
    if constexpr (EB == 2) {
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int d = 0; d < DB; ++d) {
          const int chunk = (d * 4 + vchunk16) ^ v_swizzle<EB, CPR>(vrow16);
          const unsigned char* at =
              vt + (wk * KPW + b * 32 + c * 16 + vrow16) * RB + chunk * 16 + (i16 & 1) * 8;
          const u32x2_t lo = read_column(at), hi = read_column(at + 8 * RB);
          const u32x4_t vf = {lo[0], lo[1], hi[0], hi[1]};
          Mma<DT>::step(vf, pf[c], acc[d], 0);
        }
    }
  };

  if constexpr (EB == 2 && WK == 1) {
    // Pipelined over blocks of 32 keys: while the vector units form a block's
    // probabilities, the matrix units form the scores of the next block and
    // add the values of the block before, in the same wave.  K is therefore a
    // tile ahead of V.
    static_assert(NB == 2, "a tile is two blocks");
    unsigned char* const kt = lds;
    unsigned char* const vt = lds + 2 * Z::TILE;
    constexpr int COPIES = Z::BN * CPR / kThreads;   // of a tile, a thread
    const int n = t1 - t0;
    float16_t s0, s1;      // scores of two blocks
    u32x4_t p0[2], p1[2];  // probabilities of two blocks
    float f;               // what a block's maximum makes of the sums so far
    // The maximum moves only when it falls behind by 2^8, which fp16
    // probabilities bear too: the sums are hardly ever rescaled.
    auto move_up = [&](const float16_t& s) {
      const float top = top_of(s);
      const float m_new = top > m + kSlack ? top : m;
      f = __builtin_amdgcn_exp2f(m - m_new);
      m = m_new;
      l *= f;
    };
    // `p` is formed up to here (its first use is past a branch, where the
    // compiler would take its computation, away from the matrix instructions)
    auto follow = [&](u32x4_t* p) {
      asm volatile("" : "+v"(p[0]), "+v"(p[1]), "+v"(l));
      if (__any(f != 1.0f)) rescale(f);
    };
    if (n > 0) {
      copy_tile<DT, DP, WK, false>(ck, kt, row_bytes);
      copy_tile<DT, DP, WK, true>(cv, vt, row_bytes);
      copy_tile<DT, DP, WK, false>(ck, kt + Z::TILE, row_bytes);
      wait_vmcnt<2 * COPIES>();
      lds_barrier();
      score(kt, 0, s0);
      score(kt, 1, s1);
      mask(t0, 0, s0);
      move_up(s0);   // nothing to rescale yet
      probabilities(s0);
      pack(s0, p0);
      for (int i = 0; i < n - 1; ++i) {
        // K of tile i + 1 and V of tile i have arrived for this wave, after the
        // barrier for all, and nobody reads K of tile i and V of i - 1 any more
        const unsigned char* k1 = kt + ((i + 1) & 1) * Z::TILE;
        const unsigned char* v0 = vt + (i & 1) * Z::TILE;
        wait_vmcnt<0>();
        lds_barrier();
        copy_tile<DT, DP, WK, true>(cv, vt + ((i + 1) & 1) * Z::TILE, row_bytes);
        copy_tile<DT, DP, WK, false>(ck, kt + (i & 1) * Z::TILE, row_bytes);
        mask(t0 + i, 1, s1);
        move_up(s1);
        score(k1, 0, s0);
        probabilities(s1);
        pack(s1, p1);
        add_values(v0, 0, p0);
        follow(p1);
        mask(t0 + i + 1, 0, s0);
        move_up(s0);
        score(k1, 1, s1);
        probabilities(s0);
        pack(s0, p0);
        add_values(v0, 1, p1);
        follow(p0);
      }
      const unsigned char* v0 = vt + ((n - 1) & 1) * Z::TILE;
      wait_vmcnt<0>();
      lds_barrier();
      mask(t1 - 1, 1, s1);
      move_up(s1);
      probabilities(s1);
      pack(s1, p1);
      add_values(v0, 0, p0);
      follow(p1);
      add_values(v0, 1, p1);
    }
  } else {
    if (t0 < t1) {
      copy_tile<DT, DP, WK, false>(ck, lds, row_bytes);
      copy_tile<DT, DP, WK, true>(cv, lds + Z::TILE, row_bytes);
    }
    for (int t = t0; t < t1; ++t) {
      unsigned char* kt = lds + ((t - t0) & 1) * 2 * Z::TILE;
      unsigned char* vt = kt + Z::TILE;
      // this wave's copies have arrived; after the barrier everyone's have, and
      // nobody reads the other stage any more
      wait_vmcnt<0>();
      lds_barrier();
      if (t + 1 < t1) {
        unsigned char* next = lds + ((t + 1 - t0) & 1) * 2 * Z::TILE;
        copy_tile<DT, DP, WK, false>(ck, next, row_bytes);
        copy_tile<DT, DP, WK, true>(cv, next + Z::TILE, row_bytes);
      }
      static_assert(NB == 1, "32 keys a wave");
      float16_t s;
      score(kt, 0, s);
      mask(t, 0, s);
      const float top = top_of(s);
      if (__any(top > m)) {
        const float m_new = fmaxf(m, top);
        const float f = __builtin_amdgcn_exp2f(m - m_new);
        m = m_new;
        l *= f;
        rescale(f);
      }
      probabilities(s);
      if constexpr (EB == 4) {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int vr = wk * KPW + (r & 3) + 8 * (r >> 2) + 4 * half;
#pragma unroll
          for (int d = 0; d < DB; ++d) {
            const int chunk = (d * 8 + (l32 >> 2)) ^ v_swizzle<EB, CPR>(vr);
            const float vf = *reinterpret_cast<const float*>(vt + vr * RB + chunk * 16 +
                                                             (l32 & 3) * 4);
            acc[d] = __builtin_amdgcn_mfma_f32_32x32x2f32(vf, s[r], acc[d], 0, 0, 0);
          }
        }
      } else {
        u32x4_t pf[2];
        pack(s, pf);
        add_values(vt, 0, pf);
      }
    }
  }

  l += __shfl_xor(l, 32);
  if constexpr (WK > 1) {
    // join the waves that split this row block's keys: each leaves maximum,
    // sum and outputs (32 rows, DP components, rows fastest) in LDS
    constexpr int PER = 32 * (DP + 2) * 4;
    static_assert(4 / WK * (WK - 1) * PER <= Z::LDS, "the join fits the stages");
    lds_barrier();   // every wave is done with the stages (its copies have arrived)
    unsigned char* room = lds + wr * (WK - 1) * PER;   // of the row block's waves 1, 2, ..
    float* mine = reinterpret_cast<float*>(room + (wk - 1) * PER);
    if (wk > 0) {
      if (half == 0) {
        mine[l32] = m;
        mine[32 + l32] = l;
      }
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int comp = d * 32 + (r & 3) + 8 * (r >> 2) + 4 * half;
          mine[(2 + comp) * 32 + l32] = acc[d][r];
        }
    }
    lds_barrier();
    if (wk > 0) return;
    float m_all = m;
#pragma unroll
    for (int w = 1; w < WK; ++w)
      m_all = fmaxf(m_all, reinterpret_cast<const float*>(room + (w - 1) * PER)[l32]);
    const float f = __builtin_amdgcn_exp2f(m - m_all);
    l *= f;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[d][r] *= f;
#pragma unroll
    for (int w = 1; w < WK; ++w) {
      const float* o = reinterpret_cast<const float*>(room + (w - 1) * PER);
      const float g = __builtin_amdgcn_exp2f(o[l32] - m_all);
      l = fmaf(o[32 + l32], g, l);
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int comp = d * 32 + (r & 3) + 8 * (r >> 2) + 4 * half;
          acc[d][r] = fmaf(o[(2 + comp) * 32 + l32], g, acc[d][r]);
        }
    }
    m = m_all;
  }

  if (!row_ok) return;
  const float inv = l > 0.0f ? 1.0f / l : l;   // 0 keys: 0; a NaN stays
  const float lse2 = l == 0.0f ? kNegInf : m + __builtin_amdgcn_logf(l);
  if (job.slot >= 0) {
    const long long at = ((long long)job.slot * a.Hk + job.hk) * ((long long)a.B * per_entry) + row;
    if (half == 0) a.part_lse[at] = lse2;
    float* po = a.part + at * a.D;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int comp = d * 32 + 8 * r + 4 * half;
        if (comp < a.D)
          *reinterpret_cast<float4_t*>(po + comp) =
              float4_t{acc[d][4 * r] * inv, acc[d][4 * r + 1] * inv, acc[d][4 * r + 2] * inv,
                       acc[d][4 * r + 3] * inv};
      }
    return;
  }
  const int head = job.hk * a.G + qg;
  if (a.lse && half == 0) a.lse[((long long)qb * a.Hk * a.G + head) * a.Sq + qi] = lse2 * kLn2;
  char* op = a.out + qb * a.o_b + qi * a.o_r + head * a.o_h;
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int comp = d * 32 + 8 * r + 4 * half;
      if (comp >= a.D) continue;
      const float o0 = acc[d][4 * r] * inv, o1 = acc[d][4 * r + 1] * inv,
                  o2 = acc[d][4 * r + 2] * inv, o3 = acc[d][4 * r + 3] * inv;
      if constexpr (EB == 4)
        *reinterpret_cast<float4_t*>(op + comp * 4) = float4_t{o0, o1, o2, o3};
      else
        *reinterpret_cast<u32x2_t*>(op + comp * 2) = u32x2_t{pack2<DT>(o0, o1), pack2<DT>(o2, o3)};
    }
}

// Workgroups that read the same keys (one entry and key head) follow one
// another on one XCD, whose L2 then holds those keys: dispatch deals
// workgroups out to the 8 XCDs in turn.
__device__ __forceinline__ int xcd_order(int id, int n) {
  const int per = n >> 3, more = n & 7, x = id & 7;
  return x * per + (x < more ? x : more) + (id >> 3);
}

// Each entry's rows over its prefix and own keys.
template <int DT, int DP, int WK>
__global__ __launch_bounds__(kThreads, (Shape<DT, DP, WK>::WAVES)) void attn_kernel(const AttnArgs a) {
  using Z = Shape<DT, DP, WK>;
  __shared__ __attribute__((aligned(1024))) unsigned char lds[Z::LDS];
  const int per_entry = a.Sq * a.G;
  const int row_tiles = (per_entry + Z::ROWS - 1) / Z::ROWS;
  int id = xcd_order(blockIdx.x, gridDim.x);
  Job job;
  int tile = id % row_tiles;
  id /= row_tiles;
  tile = row_tiles - 1 - tile;   // causal: the longest rows first
  job.split = id % a.splits;
  id /= a.splits;
  job.hk = id % a.Hk;
  job.b = id / a.Hk;
  job.row0 = job.b * per_entry + tile * Z::ROWS;
  job.rows = per_entry - tile * Z::ROWS < Z::ROWS ? per_entry - tile * Z::ROWS : Z::ROWS;
  job.splits = a.splits;
  job.prefix = !a.shared;
  job.own = true;
  job.slot = a.part ? (a.shared ? a.prefix_splits : 0) + job.split : -1;
  attend<DT, DP, WK>(a, job, lds);
}

// Rows of all entries, side by side, over the prefix.
template <int DT, int DP, int WK>
__global__ __launch_bounds__(kThreads, (Shape<DT, DP, WK>::WAVES)) void attn_prefix_kernel(const AttnArgs a) {
  using Z = Shape<DT, DP, WK>;
  __shared__ __attribute__((aligned(1024))) unsigned char lds[Z::LDS];
  const int all = a.B * a.Sq * a.G;
  const int row_tiles = (all + Z::ROWS - 1) / Z::ROWS;
  int id = xcd_order(blockIdx.x, gridDim.x);
  Job job;
  const int tile = id % row_tiles;
  id /= row_tiles;
  job.split = id % a.prefix_splits;
  job.hk = id / a.prefix_splits;
  job.b = 0;
  job.row0 = tile * Z::ROWS;
  job.rows = all - job.row0 < Z::ROWS ? all - job.row0 : Z::ROWS;
  job.splits = a.prefix_splits;
  job.prefix = true;
  job.own = false;
  job.slot = job.split;
  attend<DT, DP, WK>(a, job, lds);
}

// Joins the partial results of one row: out = sum_s 2^(lse_s - lse) o_s, in
// the order of the slots.  A wave a row, two components a lane.
template <int DT>
__global__ __launch_bounds__(kThreads) void attn_join_kernel(const AttnArgs a, int slots) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const long long per = (long long)a.B * a.Sq * a.G, all = per * a.Hk;
  const long long at = (long long)blockIdx.x * 4 + wave;
  if (at >= all) return;
  const int hk = (int)(at / per), row = (int)(at % per);
  const int per_entry = a.Sq * a.G;
  const int b = row / per_entry, i = row % per_entry / a.G, g = row % a.G;
  float m = kNegInf;
  for (int s = lane; s < slots; s += 64) m = fmaxf(m, a.part_lse[s * all + at]);
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) m = fmaxf(m, __shfl_xor(m, x));
  const float base = m == kNegInf ? 0.0f : m;
  float sum = 0.0f, o0 = 0.0f, o1 = 0.0f;
  const bool live = 2 * lane < a.D;
  for (int s = 0; s < slots; ++s) {
    const float w = __builtin_amdgcn_exp2f(a.part_lse[s * all + at] - base);
    sum += w;
    if (live) {
      const float2 v = *reinterpret_cast<const float2*>(a.part + (s * all + at) * a.D + 2 * lane);
      o0 = fmaf(w, v.x, o0);
      o1 = fmaf(w, v.y, o1);
    }
  }
  const float inv = sum > 0.0f ? 1.0f / sum : sum;
  const int head = hk * a.G + g;
  if (a.lse && lane == 0)
    a.lse[((long long)b * a.Hk * a.G + head) * a.Sq + i] =
        sum == 0.0f ? kNegInf : (base + __builtin_amdgcn_logf(sum)) * kLn2;
  if (!live) return;
  char* op = a.out + b * a.o_b + i * a.o_r + head * a.o_h;
  if constexpr (DT == DT_F32)
    *reinterpret_cast<float2*>(op + 8 * lane) = make_float2(o0 * inv, o1 * inv);
  else
    *reinterpret_cast<uint32_t*>(op + 4 * lane) = pack2<DT>(o0 * inv, o1 * inv);
}

int key_waves(long long rows, int eb) {
  const int wk = rows <= 32 ? 4 : rows <= 64 ? 2 : 1;
  return eb == 4 && wk == 4 ? 2 : wk;   // fp32: four stages of 128 keys would not fit
}
int tile_keys(int wk, int eb) { return eb == 4 ? 32 * wk : wk == 4 ? 128 : 64; }

template <int DT, int DP>
void launch(const AttnArgs& a, hipStream_t stream) {
  const long long per_entry = (long long)a.Sq * a.G, all = a.B * per_entry;
  constexpr int EB = Elem<DT>::bytes;
  const int wk = key_waves(per_entry, EB), wp = key_waves(all, EB);
  const dim3 threads(kThreads);
  if (a.shared) {
    const long long tiles = (all + 128 / wp - 1) / (128 / wp);
    const dim3 grid((unsigned)(tiles * a.prefix_splits * a.Hk));
    if (wp == 1)
      hipLaunchKernelGGL((attn_prefix_kernel<DT, DP, 1>), grid, threads, 0, stream, a);
    else if (wp == 2)
      hipLaunchKernelGGL((attn_prefix_kernel<DT, DP, 2>), grid, threads, 0, stream, a);
    else if constexpr (EB == 2)
      hipLaunchKernelGGL((attn_prefix_kernel<DT, DP, 4>), grid, threads, 0, stream, a);
  }
  const long long tiles = (per_entry + 128 / wk - 1) / (128 / wk);
  const dim3 grid((unsigned)(tiles * a.splits * a.Hk * a.B));
  if (wk == 1)
    hipLaunchKernelGGL((attn_kernel<DT, DP, 1>), grid, threads, 0, stream, a);
  else if (wk == 2)
    hipLaunchKernelGGL((attn_kernel<DT, DP, 2>), grid, threads, 0, stream, a);
  else if constexpr (EB == 2)
    hipLaunchKernelGGL((attn_kernel<DT, DP, 4>), grid, threads, 0, stream, a);
  if (a.part)
    hipLaunchKernelGGL((attn_join_kernel<DT>), dim3((unsigned)((all * a.Hk + 3) / 4)), threads, 0,
                       stream, a, a.splits + (a.shared ? a.prefix_splits : 0));
}

template <int DT>
void launch_dt(const AttnArgs& a, hipStream_t stream) {
  if (a.D <= 64) launch<DT, 64>(a, stream);
  else if (a.D <= 96) launch<DT, 96>(a, stream);
  else launch<DT, 128>(a, stream);
}

}  // namespace

long long attn_plan(AttnArgs* a, int dtype, int cus, bool allowed) {
  const int eb = dtype == LIBCONV_F32 ? 4 : 2;
  const long long per_entry = (long long)a->Sq * a->G, all = a->B * per_entry;
  a->shared = 0;
  a->splits = a->prefix_splits = 1;
  if (!allowed || all == 0) return 0;
  // Workgroups wanted: two a compute unit.
  const long long want = 2LL * cus;
  // Splits so that `groups` workgroups become `want`, each with 256 keys or more.
  auto split = [&](long long groups, long long keys) {
    long long s = groups > 0 ? want / groups : 1;
    if (s > keys / 256) s = keys / 256;
    return (int)(s < 1 ? 1 : s > 64 ? 64 : s);
  };
  const int wk = key_waves(per_entry, eb);
  const long long groups = a->B * a->Hk * ((per_entry + 128 / wk - 1) / (128 / wk));
  // The prefix once for all entries: with few rows an entry, reading it for
  // each of them would be what the call spends its time on.
  if (a->B > 1 && per_entry <= 64 && a->P >= 128) {
    const int wp = key_waves(all, eb);
    a->shared = 1;
    a->prefix_splits = split(a->Hk * ((all + 128 / wp - 1) / (128 / wp)), a->P);
    a->splits = split(groups, a->S);
  } else {
    a->splits = split(groups, (long long)a->P + a->S);
  }
  const int slots = a->splits + (a->shared ? a->prefix_splits : 0);
  if (slots == 1) return 0;
  return slots * a->Hk * all * (a->D + 1LL) * 4;
}

libconv_status attn_launch(AttnArgs a, int dtype, hipStream_t stream) {
  if (dtype == LIBCONV_F32) launch_dt<DT_F32>(a, stream);
  else if (dtype == LIBCONV_F16) launch_dt<DT_F16>(a, stream);
  else launch_dt<DT_BF16>(a, stream);
  return hipGetLastError() == hipSuccess ? LIBCONV_OK : LIBCONV_ERR_LAUNCH;
}

}  // namespace libconv
