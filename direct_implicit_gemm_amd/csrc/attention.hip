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
// waves holds 128 rows that share their tiles of keys (WK = 1), or, with few
// rows, 32, and its waves take a quarter of each tile's keys (WK = 4): such a
// wave copies the keys it reads itself, waits for nobody until the four join
// through LDS at the end, and is bound by the keys it reads from memory.
//
// With many rows the matrix units bound it, and the vector units' exponentials
// nearly as much: 32 scores a lane of a 32 x 64 tile take about 380 cycles of
// 1024 that its products take, so both have to run at a time (see the loop).
// Measured: 12 entries of 3200 queries, 20 heads of 128, 3277 keys, bf16, 1.25
// ms (1.03 PFLOP/s; the loop with both products after one another 2.4 ms).
#include "device_common.h"
#include "internal.h"
#include "layer.h"

namespace libconv {
namespace {

constexpr int kThreads = 256;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -__builtin_inff();
constexpr float kLowest = -3.402823466e38f;   // the maximum of no keys: finite, so that no
                                              // difference of maxima is a NaN
// log2 of how far a maximum may fall behind (lazy), and of what the
// probabilities are multiplied by.  fp16 ends at 2^-24: probabilities below
// 2^-25 of the largest would vanish from the second product and still count in
// the sum, and those below 2^-14 lose bits.  Multiplied by 2^15, less the slack,
// the largest stays below 2^16, and 2^-36 (2^-40 where the maximum is exact) is
// what vanishes; the sum is multiplied alike, so the quotient needs no care.
// bfloat16 ends where fp32 does.
template <int DT> constexpr float slack() { return DT == DT_F16 ? 4.0f : 8.0f; }
template <int DT, bool Lazy> constexpr float lift() {
  return DT != DT_F16 ? 0.0f : Lazy ? 15.0f - slack<DT>() : 15.0f;
}

template <int DT, int DP, int WK> struct Shape {
  static_assert(WK == 1 || WK == 4, "rows or keys split over the four waves");
  static constexpr int EB = Elem<DT>::bytes;
  static constexpr int RB = (DP <= 64 ? 64 : 128) * EB;    // bytes of a row of K or V in LDS
  static constexpr int CPR = RB / 16;                      // 16-byte chunks of it
  static constexpr int KPW = EB == 4 || WK == 4 ? 32 : 64; // keys a wave takes of a tile
  static constexpr int BN = KPW * WK;                      // keys of a tile
  static constexpr int ROWS = 128 / WK;                    // rows of a workgroup
  static constexpr int TILE = BN * RB;
  static constexpr int LDS = (WK == 1 ? 4 : 2) * TILE;     // K and V; two stages where shared
};
// Workgroups that a compute unit's LDS holds, at most 2 counted.
constexpr int fit(int lds) { return 2 * lds <= 160 * 1024 ? 2 : 1; }

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
  // (through scalars: a bit cast of a vector's element takes element 0)
  const uint32_t lower = r[0], upper = r[1];
  return fmaxf(__builtin_bit_cast(float, lower), __builtin_bit_cast(float, upper));
}

// 4 elements of one column of 16-bit elements: the 16 lanes of a quarter wave
// name 8 bytes each of 4 rows.  `p` is restrict so that the read has a scope of
// its own: without one, the compiler lets it wait for every copy to LDS that
// is on its way, those of the next tile among them.
__device__ __forceinline__ u32x2_t read_column(const unsigned char* __restrict p) {
  return __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                         (__attribute__((address_space(3))) s16x4_t*)p));
}

// Probabilities are rounded to the 16-bit type for the second product (their sum
// is not): an error of that one rounding beside the output's own, 0.0022 to
// 0.0024 of the output in bf16 and 0.00029 in fp16 against 0.0017 and 0.00021 of
// a product in fp32.  Two terms a probability would hold 16 bits, for half again
// the matrix work of what the matrix units bound.
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

// A walk over the tiles of K or of V: prefix, then own keys.
struct Cursor {
  const char* p;        // this copy's first row of the tile
  int stride;           // of rows in bytes (below 2^24)
  int left;             // rows from there to the end of the run; <= 0 past it
  const char* own_p;    // the own keys' first tile, where the run follows
  int own_stride, own_left;
};
__device__ __forceinline__ void advance(Cursor& c, int keys, int skip) {
  // after the run the own keys, past them nothing (selects: a branch would
  // part the code it stands in)
  const char* const p = c.p + (unsigned)keys * (unsigned)c.stride;
  const int left = c.left - keys;
  const bool more = left + skip > 0;
  c.p = more ? p : c.own_p;
  c.stride = more ? c.stride : c.own_stride;
  c.left = more ? left : c.own_left;
  c.own_left = more ? c.own_left : -skip;
}

// Copies N * LANES / CPR rows into LDS, 16 bytes a lane, thread t of LANES.
// Rows past the run's end and components from D on arrive as zeros: they lie
// past the resource's end (rows that lie closer than their own length repeat
// bytes of valid rows instead, whose scores are masked).
template <int EB, int CPR, int LANES, int N, bool V>
__device__ __forceinline__ void copy_rows(const Cursor& c, unsigned char* lds, int t,
                                          int row_bytes) {
  constexpr int PASS = LANES / CPR;   // rows of a copy
  const int rows = c.left < N * PASS ? c.left : N * PASS;
  const int bytes = (rows - 1) * c.stride + row_bytes;
  const __amdgpu_buffer_rsrc_t r = make_rsrc(c.p, rows > 0 ? bytes : 0);
  const int row = t / CPR, slot = t % CPR;
  const int at = row * c.stride;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int in = row + j * PASS;
    const int chunk = slot ^ (V ? v_swizzle<EB, CPR>(in) : k_swizzle<CPR>(in));
    copy16_to_lds(r, lds + j * LANES * 16, chunk * 16 < row_bytes ? at + chunk * 16 : kFarOffset,
                  j * PASS * c.stride);
  }
}

// What a workgroup computes: rows [row0, row0 + rows) of key head hk (rows are
// counted over the entries), prefix keys [0, P) and own keys of entry b, of
// whose tiles it takes share `split` of `splits` (splits 0: those of run
// `split` of `chunk` keys, if any); slot: where its partial result goes (-1:
// straight to the output).
struct Job {
  int row0, rows, hk, b;
  bool prefix, own;
  int split, splits, chunk, slot;
};

template <int DT, int DP, int WK>
__device__ __forceinline__ void attend(const AttnArgs& a, const Job& job, unsigned char* lds) {
  using Z = Shape<DT, DP, WK>;
  constexpr int EB = Z::EB, RB = Z::RB, CPR = Z::CPR, KPW = Z::KPW, BN = Z::BN;
  constexpr int KS = DP * EB / 32;  // steps of the first product
  constexpr int NB = KPW / 32;      // blocks of 32 keys a wave
  constexpr int DB = DP / 32;       // blocks of 32 components
  constexpr float LIFT = lift<DT, EB == 2 && WK == 1>();
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
  int t0, t1;
  if (job.splits > 0) {
    t0 = (int)((long long)tiles * job.split / job.splits);
    t1 = (int)((long long)tiles * (job.split + 1) / job.splits);
  } else {
    // nothing to leave where the entry has no such keys: the join knows
    if ((long long)job.split * job.chunk >= n_own) return;
    t0 = job.split * (job.chunk / BN);
    t1 = t0 + job.chunk / BN;
    t1 = t1 < tiles ? t1 : tiles;
  }

  const char* kp = a.kp + job.hk * a.kp_h;
  const char* vp = a.vp + job.hk * a.vp_h;
  const char* ko = a.k + job.b * a.k_b + job.hk * a.k_h;
  const char* vo = a.v + job.b * a.v_b + job.hk * a.v_h;
  // this workgroup's or this wave's keys of tiles t0 .. t1 - 1; past them it
  // reads nothing
  const int end_p = t1 < tiles_p ? t1 * BN : a.P;
  const int last_own = t1 <= tiles_p ? 0 : (t1 - tiles_p) * BN < end_own ? (t1 - tiles_p) * BN
                                                                         : end_own;
  auto cursor = [&](const char* p, long long stride, const char* o, long long own_stride) {
    const int skip = wk * KPW;
    Cursor c;
    c.own_p = o + skip * own_stride;
    c.own_stride = (int)own_stride;
    c.own_left = last_own - skip;
    c.p = p + ((long long)t0 * BN + skip) * stride;
    c.stride = (int)stride;
    c.left = end_p - t0 * BN - skip;
    if (t0 >= tiles_p) {
      c.p = o + ((long long)(t0 - tiles_p) * BN + skip) * own_stride;
      c.stride = (int)own_stride;
      c.left = last_own - (t0 - tiles_p) * BN - skip;
      c.own_left = -skip;
    }
    return c;
  };
  Cursor ck = cursor(kp, a.kp_r, ko, a.k_r);
  Cursor cv = cursor(vp, a.vp_r, vo, a.v_r);
  // The part of a tile that comes next; lanes: those that copy it together.
  constexpr int LANES = WK == 1 ? kThreads : 64;
  constexpr int COPIES = KPW * CPR / LANES;
  const int lane_id = WK == 1 ? threadIdx.x : lane;
  const int wave_to = WK == 1 ? wave * 1024 : 0;
  auto copy_k = [&](unsigned char* to) {
    copy_rows<EB, CPR, LANES, COPIES, false>(ck, to + wave_to, lane_id, row_bytes);
    advance(ck, BN, wk * KPW);
  };
  auto copy_v = [&](unsigned char* to) {
    copy_rows<EB, CPR, LANES, COPIES, true>(cv, to + wave_to, lane_id, row_bytes);
    advance(cv, BN, wk * KPW);
  };

  float16_t acc[DB];
#pragma unroll
  for (int d = 0; d < DB; ++d) acc[d] = float16_t{};
  float m = kLowest, l = 0.0f;   // maximum (times scale, log2) and sum of this lane's half

  // LDS offsets that do not change from tile to tile
  const int krow = l32 * RB;
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
  // keys past the end and keys the causal mask hides: of blocks that begin
  // from whole_p on in the prefix and from whole_own on in the own keys
  const int whole_p = job.prefix ? a.P & ~31 : 0, whole_own = (lim_wave & ~31) + tiles_p * BN;
  auto mask = [&](int t, int b, float16_t& s) {
    const int key0 = t * BN + wk * KPW + b * 32;   // counted over both
    if (key0 >= whole_p && (key0 < tiles_p * BN || key0 >= whole_own)) {
      const int lane_lim = (t < tiles_p ? a.P : lim + tiles_p * BN) - key0 - 4 * half;
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
  // probabilities times 2^(LIFT + their maximum - m), added to the sum
  auto probabilities = [&](float16_t& s) {
    const float base = LIFT == 0.0f ? -m : LIFT - m;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      s[r] = __builtin_amdgcn_exp2f(fmaf(s[r], a.scale, base));
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
              vt + (b * 32 + c * 16 + vrow16) * RB + chunk * 16 + (i16 & 1) * 8;
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
    const int n = t1 - t0;
    float16_t s0, s1;      // scores of two blocks
    u32x4_t p0[2], p1[2];  // probabilities of two blocks
    float f;               // what a block's maximum makes of the sums so far
    // The maximum moves only when it falls behind by 2^slack: the sums are
    // hardly ever rescaled.
    auto move_up = [&](const float16_t& s) {
      const float top = top_of(s);
      const float m_new = top > m + slack<DT>() ? top : m;
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
      copy_k(kt);
      copy_v(vt);
      copy_k(kt + Z::TILE);
      wait_vmcnt<2 * COPIES>();
      lds_barrier();
      score(kt, 0, s0);
      score(kt, 1, s1);
      mask(t0, 0, s0);
      move_up(s0);   // nothing to rescale yet
      probabilities(s0);
      pack(s0, p0);
      // Two blocks: tile i's second and tile i + 1's first.  odd is i & 1, a
      // constant where it is called, so that the stages' addresses are.
      auto two_blocks = [&](int i, int odd) __attribute__((always_inline)) {
        // K of tile i + 1 and V of tile i have arrived for this wave, after the
        // barrier for all, and nobody reads K of tile i and V of i - 1 any more
        const unsigned char* k1 = kt + (1 - odd) * Z::TILE;
        const unsigned char* v0 = vt + odd * Z::TILE;
        wait_vmcnt<0>();
        lds_barrier();
        mask(t0 + i, 1, s1);
        move_up(s1);
        score(k1, 0, s0);
        // behind the first matrix instructions, which cover their scalar work
        copy_v(vt + (1 - odd) * Z::TILE);
        copy_k(kt + odd * Z::TILE);
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
      };
      int i = 0;
      for (; i + 2 < n; i += 2) {
        two_blocks(i, 0);
        two_blocks(i + 1, 1);
      }
      if (i + 1 < n) two_blocks(i, 0);
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
    static_assert(NB == 1, "32 keys a wave");
    float16_t s;
    auto softmax = [&](int t) {
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
    };
    auto add = [&](const unsigned char* vt) {
      if constexpr (EB == 4) {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int vr = (r & 3) + 8 * (r >> 2) + 4 * half;
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
    };
    if constexpr (WK == 1) {
      if (t0 < t1) {
        copy_k(lds);
        copy_v(lds + Z::TILE);
      }
      for (int t = t0; t < t1; ++t) {
        unsigned char* kt = lds + ((t - t0) & 1) * 2 * Z::TILE;
        // this wave's copies have arrived; after the barrier everyone's have, and
        // nobody reads the other stage any more
        wait_vmcnt<0>();
        lds_barrier();
        if (t + 1 < t1) {
          unsigned char* next = lds + ((t + 1 - t0) & 1) * 2 * Z::TILE;
          copy_k(next);
          copy_v(next + Z::TILE);
        }
        score(kt, 0, s);
        softmax(t);
        add(kt + Z::TILE);
      }
    } else {
      // a wave's own 32 keys of a tile, K and V one stage each: the next copy
      // to a stage starts when its reads are done (and past the last tile
      // reads nothing, so that the counts stay the same)
      unsigned char* const kt = lds + wave * (2 * 32 * RB);
      unsigned char* const vt = kt + 32 * RB;
      if (t0 < t1) {
        copy_k(kt);
        copy_v(vt);
      }
      for (int t = t0; t < t1; ++t) {
        wait_vmcnt<COPIES>();
        lds_fence();
        score(kt, 0, s);
        lds_fence();
        copy_k(kt);
        softmax(t);
        wait_vmcnt<COPIES>();
        lds_fence();
        add(vt);
        lds_fence();
        copy_v(vt);
      }
      wait_vmcnt<0>();
    }
  }

  l += __shfl_xor(l, 32);
  if constexpr (WK > 1) {
    // join the waves that split this row block's keys: each leaves maximum,
    // sum and outputs (32 rows, DP components, rows fastest) in LDS
    constexpr int PER = 32 * (DP + 2) * 4;
    static_assert((WK - 1) * PER <= Z::LDS, "the join fits the stages");
    lds_barrier();   // every wave is done with its stages, no copy is on its way
    unsigned char* room = lds;   // of the waves 1, 2, ..
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
  const float lse2 = l == 0.0f ? kNegInf : m + (__builtin_amdgcn_logf(l) - LIFT);
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

// Each entry's rows over its prefix and own keys.  130 queries of 2 entries, 8
// heads of 64 over 333 + 190 keys in fp32: 14 us, and 3 of the join (bound by
// the fp32 matrix instructions of 160 workgroups); one query of 4 entries, 20
// heads of 64 over 1000 keys in bf16: 10 us (80 workgroups, whose waves take 8
// tiles of keys one after another; eight waves instead of four: 10 us).
template <int DT, int DP, int WK>
__global__ __launch_bounds__(kThreads, fit((Shape<DT, DP, WK>::LDS))) void attn_kernel(
    const AttnArgs a) {
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
  job.chunk = 0;
  job.prefix = true;
  job.own = true;
  job.slot = a.part ? job.split : -1;
  attend<DT, DP, WK>(a, job, lds);
}

// The prefix once for all entries: the first `prefix_jobs` workgroups take the
// rows of all entries, side by side, over shares of the prefix (WP: how they
// split); the others take each entry's rows over runs of its own keys.  64
// entries of one query, 32 heads over 8 key heads of 128, 8192 shared and up to
// 2048 own keys in bf16 (303 MB): 67 us, 4.5 TB/s; in two launches, own keys
// not split, 25 + 86 us.
template <int DT, int DP, int WP>
__global__ __launch_bounds__(kThreads, fit((Shape<DT, DP, WP>::LDS > Shape<DT, DP, 4>::LDS
                                                ? Shape<DT, DP, WP>::LDS
                                                : Shape<DT, DP, 4>::LDS)))
void attn_shared_kernel(const AttnArgs a, int prefix_jobs) {
  using Z = Shape<DT, DP, WP>;
  using ZO = Shape<DT, DP, 4>;
  constexpr int LDS = Z::LDS > ZO::LDS ? Z::LDS : ZO::LDS;
  __shared__ __attribute__((aligned(1024))) unsigned char lds[LDS];
  const int per_entry = a.Sq * a.G;
  Job job;
  if ((int)blockIdx.x < prefix_jobs) {
    const int all = a.B * per_entry;
    const int row_tiles = (all + Z::ROWS - 1) / Z::ROWS;
    int id = xcd_order(blockIdx.x, prefix_jobs);
    const int tile = id % row_tiles;
    id /= row_tiles;
    job.split = id % a.prefix_splits;
    job.hk = id / a.prefix_splits;
    job.b = 0;
    job.row0 = tile * Z::ROWS;
    job.rows = all - job.row0 < Z::ROWS ? all - job.row0 : Z::ROWS;
    job.splits = a.prefix_splits;
    job.chunk = 0;
    job.prefix = true;
    job.own = false;
    job.slot = job.split;
    attend<DT, DP, WP>(a, job, lds);
  } else {
    const int row_tiles = (per_entry + ZO::ROWS - 1) / ZO::ROWS;
    int id = blockIdx.x - prefix_jobs;
    const int tile = id % row_tiles;
    id /= row_tiles;
    job.hk = id % a.Hk;
    id /= a.Hk;
    job.b = id % a.B;
    job.split = id / a.B;
    job.row0 = job.b * per_entry + tile * ZO::ROWS;
    job.rows = per_entry - tile * ZO::ROWS < ZO::ROWS ? per_entry - tile * ZO::ROWS : ZO::ROWS;
    job.splits = 0;
    job.chunk = a.chunk;
    job.prefix = false;
    job.own = true;
    job.slot = a.prefix_splits + job.split;
    attend<DT, DP, 4>(a, job, lds);
  }
}

// Joins the partial results of each row: out = sum_s 2^(lse_s - lse) o_s, in
// the order of the slots.  LPR lanes a row, 4 components a lane; one pass, 8
// slots' reads on their way at a time.  Bound by reading the partial results:
// 2048 rows of 128 in up to 16 slots 5 us, 24800 rows of 80 in two 8.5 us.
template <int DT, int LPR>
__global__ __launch_bounds__(kThreads) void attn_join_kernel(const AttnArgs a) {
  const int lane = threadIdx.x % LPR;
  const long long per = (long long)a.B * a.Sq * a.G, all = per * a.Hk;
  const long long at = (long long)blockIdx.x * (kThreads / LPR) + threadIdx.x / LPR;
  if (at >= all) return;
  const int hk = (int)(at / per), row = (int)(at % per);
  const int per_entry = a.Sq * a.G;
  const int b = row / per_entry, i = row % per_entry / a.G, g = row % a.G;
  int slots = a.splits;
  if (a.shared) {   // own keys: the slots that have any
    int n = a.lengths[b];
    n = n < 0 ? 0 : n > a.S ? a.S : n;
    slots = a.prefix_splits + (n + a.chunk - 1) / a.chunk;
  }
  const bool live = 4 * lane < a.D;
  const float* lse = a.part_lse + at;
  const float* part = a.part + at * a.D + (live ? 4 * lane : 0);
  float m = kLowest, sum = 0.0f;
  float4_t o = {0.0f, 0.0f, 0.0f, 0.0f};
  constexpr int U = 8;
  for (int s = 0; s < slots; s += U) {
    float w[U];
    float4_t v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      w[u] = kNegInf;
      v[u] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
      if (s + u < slots) {
        w[u] = lse[(s + u) * all];
        v[u] = *reinterpret_cast<const float4_t*>(part + (s + u) * all * a.D);
      }
    }
    float m_new = m;
#pragma unroll
    for (int u = 0; u < U; ++u) m_new = fmaxf(m_new, w[u]);
    const float f = __builtin_amdgcn_exp2f(m - m_new);
    m = m_new;
    sum *= f;
    o *= f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float p = __builtin_amdgcn_exp2f(w[u] - m);
      sum += p;
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = fmaf(p, v[u][j], o[j]);
    }
  }
  const float inv = sum > 0.0f ? 1.0f / sum : sum;
  const int head = hk * a.G + g;
  if (a.lse && lane == 0)
    a.lse[((long long)b * a.Hk * a.G + head) * a.Sq + i] =
        sum == 0.0f ? kNegInf : (m + __builtin_amdgcn_logf(sum)) * kLn2;
  if (!live) return;
  char* op = a.out + b * a.o_b + i * a.o_r + head * a.o_h;
  if constexpr (DT == DT_F32)
    *reinterpret_cast<float4_t*>(op + 16 * lane) = o * inv;
  else
    *reinterpret_cast<u32x2_t*>(op + 8 * lane) =
        u32x2_t{pack2<DT>(o[0] * inv, o[1] * inv), pack2<DT>(o[2] * inv, o[3] * inv)};
}

// How many of a workgroup's waves split its keys: all with up to 64 rows (the
// rows of `sets` row sets), and where workgroups of 128 rows would leave half
// the compute units idle.  Measured with heads of 128: 8 heads of 4 entries of
// 500 queries over 600 keys (128 workgroups of 128 rows) 17 us against 25, over
// 3000 keys 46 against 45; 8 entries (256) 29 against 32, 90 against 73.
int key_waves(long long rows, long long sets) {
  return rows <= 64 || (rows + 127) / 128 * sets <= kPlanCus / 2 ? 4 : 1;
}
long long row_tiles(long long rows, int waves) {
  const int r = 128 / waves;
  return (rows + r - 1) / r;
}

template <int DT, int DP>
void launch(const AttnArgs& a, hipStream_t stream) {
  const long long per_entry = (long long)a.Sq * a.G, all = a.B * per_entry;
  const dim3 threads(kThreads);
  if (a.shared) {
    const int prefix_jobs = (int)(row_tiles(all, a.prefix_waves) * a.prefix_splits * a.Hk);
    const long long own_jobs = row_tiles(per_entry, 4) * a.splits * a.Hk * a.B;
    const dim3 grid((unsigned)(prefix_jobs + own_jobs));
    if (a.prefix_waves == 1)
      hipLaunchKernelGGL((attn_shared_kernel<DT, DP, 1>), grid, threads, 0, stream, a,
                         prefix_jobs);
    else
      hipLaunchKernelGGL((attn_shared_kernel<DT, DP, 4>), grid, threads, 0, stream, a,
                         prefix_jobs);
  } else {
    const dim3 grid((unsigned)(row_tiles(per_entry, a.waves) * a.splits * a.Hk * a.B));
    if (a.waves == 1)
      hipLaunchKernelGGL((attn_kernel<DT, DP, 1>), grid, threads, 0, stream, a);
    else
      hipLaunchKernelGGL((attn_kernel<DT, DP, 4>), grid, threads, 0, stream, a);
  }
  if (a.part) {
    constexpr int LPR = DP <= 64 ? 16 : 32;
    const long long per = kThreads / LPR;
    hipLaunchKernelGGL((attn_join_kernel<DT, LPR>),
                       dim3((unsigned)((all * a.Hk + per - 1) / per)), threads, 0, stream, a);
  }
}

template <int DT>
void launch_dt(const AttnArgs& a, hipStream_t stream) {
  if (a.D <= 64) launch<DT, 64>(a, stream);
  else if (a.D <= 96) launch<DT, 96>(a, stream);
  else launch<DT, 128>(a, stream);
}

}  // namespace

long long attn_plan(AttnArgs* a, int dtype, int cus, bool allowed) {
  const long long per_entry = (long long)a->Sq * a->G, all = a->B * per_entry;
  a->shared = 0;
  a->splits = a->prefix_splits = 1;
  a->chunk = 0;
  a->waves = key_waves(per_entry, (long long)a->B * a->Hk);
  if (!allowed || all == 0) return 0;
  // Few keys: one launch, no workspace and nothing to join.  Measured, calls in
  // a row (in a graph), one launch against two: one query of 4 entries with 20
  // key heads of 64 in 16 bits, 520 keys 8.3 us (8.0) against 10.7 (9.7), 760
  // keys 9.2 (9.1) against 10.2 (9.2), 1000 keys 10.4 (10.4) against 9.7 (9.3),
  // which a workspace is not worth; 12 entries (240 workgroups), 760 keys 9.9
  // (10.0) against 10.5 (9.6), 1000 keys 11.9 (12.3) against 10.2 (9.6); heads
  // of 128, 552 keys 10.9 (10.6) against 13.2 (12.4), 1000 keys 14.2 (14.0)
  // against 12.6 (11.7); fp32 of 64, 440 keys 17.3 (17.1) against 18.4 (17.4),
  // 130 queries over 523 keys 17.4 (17.4) against 16.4 (15.6).
  const long long keys = a->P + (long long)a->S, sets = (long long)a->B * a->Hk;
  const long long key_bytes = a->D * (dtype == LIBCONV_F32 ? 4LL : 2LL);
  if (a->waves == 4 && (keys <= (dtype == LIBCONV_F32 ? 512 : 768) ||
                        (sets <= kPlanCus / 2 && keys * key_bytes <= 128 * 1024)))
    return 0;
  // Splits so that `groups` workgroups become `want`, each with `least` keys
  // or more.
  auto split = [&](long long want, long long groups, long long keys, long long least) {
    long long s = groups > 0 ? want / groups : 1;
    if (s > keys / least) s = keys / least;
    return (int)(s < 1 ? 1 : s > 64 ? 64 : s);
  };
  const long long groups = a->B * a->Hk * row_tiles(per_entry, a->waves);
  // The prefix once for all entries: with few rows an entry, reading it for
  // each of them would be what the call spends its time on.  With more than 64
  // there is little in it either way, and much to join (bf16, 4 query heads a
  // key head of 128, shared against not): 8 entries of 68 rows a key head over
  // 4096 + 256 keys 31.5 us and 35.2, 128 rows 40.7 and 40.2; 32 entries over
  // 2048 + 128, 68 rows 44.9 and 43.2, 128 rows 69 and 52.  (Its workgroups come
  // on top of the entries', whose number is bounded by what a launch holds: the
  // most entries read it each.)
  const long long prefix_groups = a->Hk * row_tiles(all, all <= 64 ? 4 : 1);
  if (a->B > 1 && per_entry <= 64 && a->P >= 128 && groups + prefix_groups < (1 << 24)) {
    a->shared = 1;
    // (a share of the prefix leaves a partial result of every row: few with
    // many rows)
    a->waves = 4;
    a->prefix_waves = all <= 64 ? 4 : 1;
    a->prefix_splits = split(2LL * cus, prefix_groups, a->P, 256);
    if (all > 64 && a->prefix_splits > 8) a->prefix_splits = 8;
    // own keys: runs of one length, so that long entries do not hold up the
    // end; about half of them will have keys
    const long long runs = split(8LL * cus, groups, a->S, 256);
    const long long chunk = ((a->S + runs - 1) / runs + 127) / 128 * 128;
    a->chunk = (int)(chunk < 128 ? 128 : chunk);
    a->splits = (a->S + a->chunk - 1) / a->chunk;
  } else {
    // twice as many gained nothing (24 800 rows of heads of 80: 48 us either way)
    a->splits = split(2LL * cus, groups, (long long)a->P + a->S, 256);
  }
  const int slots = a->splits + (a->shared ? a->prefix_splits : 0);
  if (!a->shared && slots == 1) return 0;
  return slots * a->Hk * all * (a->D + 1LL) * 4;
}

libconv_status attn_launch(AttnArgs a, int dtype, hipStream_t stream) {
  if (dtype == LIBCONV_F32) launch_dt<DT_F32>(a, stream);
  else if (dtype == LIBCONV_F16) launch_dt<DT_F16>(a, stream);
  else launch_dt<DT_BF16>(a, stream);
  return hipGetLastError() == hipSuccess ? LIBCONV_OK : LIBCONV_ERR_LAUNCH;
}

}  // namespace libconv
