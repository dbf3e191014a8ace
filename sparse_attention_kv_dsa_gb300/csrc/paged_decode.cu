// Attention of one new token per sequence over a paged key/value cache.
//
//   x_t = scale q . k_t, capped and biased;  out = sum_t e^(x_t) v_t / sum_t e^(x_t);
//   lse = log sum_t e^(x_t)   over the tokens t that the query sees.
//
// Bound: a seen key and value (4 d bytes a token and KV head in bf16) is read once for each
// group of 16 of its KV head's G query heads (8 in float32), 4 d operations a head: 16 operations
// a byte at most, so HBM up to G = 16 (8).  More heads read the cache ceil(G / 16) (ceil(G / 8))
// times, from L2 where the groups meet there.  16 sequences of 20K, one KV head of 128: bf16 68 us
// at G = 16, 86 at 32, 132 at 64, 213 at 128; float32 136 at 8, 222 at 16, 1484 at 128.  The
// many-token call with a row a sequence packs a KV head's heads and reads the cache once: bf16 68,
// 69, 70, 75 us, float32 310 to 64 heads and 581 at 128.
//
// Split.  The cache is dealt out in units: tiles of TILE tokens of one KV head and up to ROWS
// of its query heads, ordered by (sequence, KV head, tile).  A persistent grid computes from
// the device's own lengths how many units there are and gives each CTA a run of equal weight
// (a (sequence, head) weighs one unit besides its tiles: its queries, its joining), so that
// ragged batches, one long sequence and many short ones all spread evenly, and one captured
// graph serves any lengths.  A run may cross sequences; the loads run on across the
// border.  A (sequence, head) whose units lie in one CTA is finished there; otherwise each of
// its CTAs leaves a partial (o, m, l) -- at most two a CTA: the end of a run of units begun
// elsewhere (slot 0), and the start of one finished elsewhere (slot 1) -- and a second kernel
// joins them in order: sums of a fixed order, no atomics.
//
// Inside a CTA each warp takes its own share of every tile's tokens through its own ring of
// cp.async stages with its own running maximum, so that the main loop has no barrier; the four
// warps' states are joined where a (sequence, head) ends.
// bf16: S = Q K^T and O += P V on the warp-level tensor instruction (16 query heads as its M;
// G <= 16 leaves it idle rows, and still 16 operations a byte are an eighth of its rate).
// float32: on the FMA units, products and sums in float32: 8 tokens a warp, four lanes to a token
// for the scores, a lane to four values for the results.
//
// Measured on a GB300 (copy rate 6.78 TB/s): 16 sequences of 32K-48K tokens, 8 KV heads of 128
// (2.63 GB) 386 to 397 us, 6.6 to 6.8 TB/s; 96 of up to 4K, 8 KV heads of 64, cap and window (552 MB)
// 95 to 103 us, 5.4 to 5.8 TB/s; 4 float32 sequences (109 MB) 39 us; one of 8K (33.5 MB) 22 us, 17 a
// call in a captured graph.  The join alone takes 7 to 11 us with cold caches, where its warps wait
// for loads and for instructions (22 to 38 and 8 to 13 stalled warps an issue but for the 96
// sequences, 11 and 2): most of what the short calls spend beside their bytes.  Not kept: a join of 512 threads a row, and one in a rolled loop with a
// single load in flight (16 sequences 402 to 410 us); a third stage in place of the third CTA.
//
// A cache in 8 bits (WarpQ8): half the bytes, 32 operations a byte, and twice the tokens a second to
// work on: instructions bound it.  Units come by TMA where their tokens are all there (page boxes of 8
// tokens or more), so that a warp of 32 tokens spends some 640 instructions on 8 KB (its maxima are
// compared lane by lane, and joined only where one moves: 228 us where each unit joins them).  Measured: 16
// sequences of 32K-48K, 8 KV heads of 128 (1.32 GB) 223 to 226 us, 5.9 TB/s (306 us with cp.async, four warps a
// CTA and integer divisions in the look-ups); 96 of up to 4K, d = 64, cap and window (278 MB) 77 us, 3.6 TB/s,
// issue 53 % busy; one of 8K 15.7 us a call in a captured graph.  Not kept: 16 tokens a warp and eight warps (16 sequences
// 333 us), 64 tokens a warp at d = 64 (96 sequences 86 us).
//
// A few new tokens a sequence over codes (MULTI; up to 32 rows, (new token, query head of the group) pairs, a
// sequence on average, no document starts; sequences with more rows than `most` are another kernel's): the same split and loop with up to 32 rows to a unit,
// each with its own end.  The tensor-core kernel of the many-token call spends its single warps' turns
// there (16 sequences of 17K-20K with 4 new tokens each 287 us on 128-row tiles).  Here 205 us, 3.1 TB/s: eight
// warps of 255 registers an SM, latency (1.8 stalled warps an issue wait for the instruction before, issue
// 35 % busy, tensor 33 %).  Not kept: two warps with the scores of 16 tokens each and half of the values' results
// of both, twelve warps an SM (256 us, half more instructions); units of 16 rows (255 us); scores of the second 16
// tokens among the results of the first (294 us, spills).

#include "paged_map.cuh"

namespace echo {

constexpr int PD_MAX_ROWS = 16;
constexpr int PD_MAX_CTAS = 608;     // partial slots: two a CTA
constexpr int PD_MULTI_CTAS = 320;   // of a call of few tokens
// Tiles of a page table up to which a sequence is not split (e4m3): one launch less for the host (20 us a
// call, 24 with the join), and on the GPU 8 sequences of 300 8.5 us instead of 11.4, of 700 (4 tiles) 11.5 instead of
// 12.7, but of 1400 18.4 instead of 13.6.
constexpr int64_t PD_WHOLE_TILES = 4;
constexpr int PD_RING = 4;           // units whose look-ups are kept: one more than stages, or more

struct DecodeParams {
  echo_paged_kv_t C;
  echo_paged_scales_t X;             // of a cache in 8 bits
  FastDiv page;                      // by page_tokens
  const void *q;
  int64_t q_stride;
  const int32_t *seq_len;
  int B, Hq, G, HG;                  // query heads of a KV head, groups of ROWS of them
  const float *slopes;
  int window;
  const int32_t *first_tok, *prefix_len;
  ScoreForm f;
  void *out;
  float *lse;
  float *po, *pml;                   // partials [2 CTAs][rows][d], [2 CTAs][rows][2]
  int32_t *rec;                      // [CTAs][4]: the split (sequence, head group) that ends in the CTA
  int prows;                         // rows of a partial: min(G, ROWS)
  int nctas;
  int whole;                         // e4m3: every (sequence, KV head, group) is one CTA's, none is split
  // several new tokens a sequence (MULTI): rows q_start[b] .. of sequence b, of N; G FastDiv'ed
  const int32_t *q_start;
  int N, most;                       // sequences of more packed rows than `most` are left out, *some: there are any
  int32_t *some;
  FastDiv group;
};

struct E4m3 {                        // element of a cache in 8 bits
  uint8_t code;
};

// NT: tiles of 8 rows (query heads, MULTI: query heads of a few new tokens) of e4m3's products.
template <typename T, int D, int NT = 2, bool MULTI = false>
struct PdShape {
  static constexpr bool F32 = sizeof(T) == 4, BF = sizeof(T) == 2, Q8 = sizeof(T) == 1;
  using Act = std::conditional_t<F32, float, __nv_bfloat16>;   // of queries and results
  static constexpr int WARPS = !Q8 ? 4 : !MULTI ? (D == 128 ? 6 : 4) : NT == 4 ? (D == 128 ? 4 : 6) : D == 128 ? 6 : 8;
  static constexpr int THREADS = 32 * WARPS;
  static constexpr int MIN_WEIGHT = Q8 ? 2 : 3;         // least weight of a CTA's run (e4m3, one sequence of 8K: 3 is 17.2 us, 1 and 2 16.1)
  static constexpr int ROWS = F32 ? 8 : MULTI ? 8 * NT : 16;    // rows of a unit
  static constexpr int TW = F32 ? 8 : BF && D == 128 ? 16 : 32;       // tokens of a warp: 8 KB of keys and values
                                                        // (f32, d = 64, and e4m3: 4 KB)
  static constexpr int TILE = WARPS * TW;
  static constexpr int ROWB = D * (int)sizeof(T);       // bytes of a key (or value)
  static constexpr int ALIGN = Q8 ? 1024 : 128;         // of the stages: TMA's swizzle goes by the address
  static constexpr int QROWB = D * (int)sizeof(Act);    // bytes of a query
  static constexpr int QACC = ROWS * (F32 ? QROWB : Q8 ? D * 4 : QROWB + D * 4);   // of the query tile and the joined
                                                        // results, which lie in its place but for bf16
  static constexpr int HALF = TW * ROWB;                // a warp's keys of a tile
  // Stages of a warp's ring and CTAs an SM.  bf16 rows of 128 values stream best from two CTAs of
  // three stages (16 x 32K-48K tokens: 396 us, two stages 401); d = 64 and float32 have more
  // instructions a byte and want the warps of a third CTA (b96 capped 103 us, two CTAs 112; float32
  // 39 us, two CTAs 43).
  static constexpr int STAGES = BF && D == 128 ? 3 : 2;
  static constexpr int CTAS = (D == 128 && !F32) || MULTI ? 2 : Q8 ? 4 : 3;
  static constexpr bool NO_REGS = MULTI || (Q8 && NT == 2);   // no registers left for a warp's place in its run
};

// What sequence b's query sees, as tiles; a sequence that sees nothing has one tile of
// nothing, which writes its empty rows.
struct DecodeSpan {
  int len, first, pre, lo;
  TileSpan t;
  __device__ __forceinline__ int n() const { return t.nA + t.nB; }
};
// MULTI: of a sequence's new tokens, the rows [s0, s0 + n) of the packed arrays.
__device__ __forceinline__ int decode_rows(const DecodeParams &P, int b, int &s0) {
  s0 = min(max(P.q_start[b], 0), P.N);
  const int n = max(min(max(P.q_start[b + 1], 0), P.N) - s0, 0);
  return (int64_t)n * P.G <= P.most ? n : 0;
}
template <bool MULTI = false>
__device__ __forceinline__ DecodeSpan decode_span(const DecodeParams &P, int b, int tile, int rows = 1) {
  DecodeSpan s;
  s.len = paged_len(P.C, P.seq_len, b);
  s.first = P.first_tok ? max(P.first_tok[b], 0) : 0;
  s.pre = P.prefix_len ? min(P.prefix_len[b], s.len) : 0;
  s.lo = P.window ? max(s.first, MULTI ? s.len - rows + 1 - P.window : s.len - P.window) : s.first;
  s.t = tile_span(s.first, s.pre, s.lo, s.len, tile);
  if (s.n() == 0) s.t.nA = 1;
  return s;
}

// A unit of a warp's ring.
struct UnitInfo {
  int b, kvh, hg, t0, len;           // hg: group of ROWS of the KV head's query heads; t0: the warp's first token
  int c0;                            // CTA of (b, kvh, hg)'s first unit
  int flags;                         // 1 the run's first unit of them, 2 its last, 4 begun elsewhere, 8 goes on elsewhere
  uint32_t there;                    // tokens that are seen and there
};

// A warp's place in its run, what does not change from unit to unit: of the look-ups, and of the unit at hand.
// The same in every lane; kept in shared memory where registers are few (16 sequences of 32K-48K, 16 heads to
// a KV head 303 -> 292 us, MULTI's 16 x 4 drafted tokens 213 -> 211 us).
struct PdPlace {
  DecodeSpan cs;                     // current (sequence, head group)'s tiles
  int cb, cHG, cn, ckvh, chg;        // it, groups of its KV head, tiles
  uint32_t ws;                       // weight before it
  int s0, r0, nrows, h0;             // the unit's: first row of its sequence (MULTI) and of its own, rows, first head
  int minpos, maxlo, pre;            // MULTI: what every row of it sees
};

struct PdRow {                       // MULTI: of a row: its score's factor, its bias, its position (-1: it sees nothing), its lower end
  float fa, sl;
  int pos, lo;
};

template <typename T, int D, int NT, bool MULTI>
struct PdShared {
  using Sh = PdShape<T, D, NT, MULTI>;
  UnitInfo info[Sh::WARPS][PD_RING];
  uint32_t sum[Sh::WARPS], before;    // before: weight before sequence seq
  int seq;
  float m[Sh::WARPS][MULTI ? Sh::ROWS : PD_MAX_ROWS], l[Sh::WARPS][MULTI ? Sh::ROWS : PD_MAX_ROWS];
  PdRow row[MULTI ? Sh::ROWS : 1];
  PdPlace place[Sh::NO_REGS ? Sh::WARPS : 1];
  alignas(16) float p[Sh::F32 ? Sh::WARPS : 1][8][8];              // f32: weights [head][token]
  uint64_t full[Sh::Q8 ? Sh::WARPS : 1][Sh::STAGES];              // e4m3: a warp's stage is there
  // e4m3, of a stage's tokens: the upper halves of 2^(exponent of the key) and, in the lower half, of
  // 2^-(exponent of the value); that exponent
  float2 ex[Sh::Q8 ? Sh::WARPS : 1][Sh::STAGES][Sh::Q8 ? Sh::TW : 1];
};

template <typename T, int D, int NT, bool MULTI>
constexpr size_t pd_smem() {
  using Sh = PdShape<T, D, NT, MULTI>;
  return Sh::ALIGN + (size_t)Sh::WARPS * Sh::STAGES * 2 * Sh::HALF + Sh::QACC +
         sizeof(PdShared<T, D, NT, MULTI>);
}

__device__ __forceinline__ void pd_ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void pd_ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// c += a (16x16, row) * b (16x8, col), bf16 inputs, f32 accumulate
__device__ __forceinline__ void pd_mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void pd_cp_arrive(uint64_t *bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ uint32_t pd_pack(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}

// Byte offset of 16-byte chunk c of row r in a tile of ROWB-byte rows: chunks are permuted
// within 128 bytes by the row, so that eight rows read at one chunk lie in eight bank groups (rows
// of 64 bytes: two rows to 128 bytes, permuted within each).
template <int ROWB>
__device__ __forceinline__ uint32_t pd_at(int r, int c) {
  return (uint32_t)(r * ROWB + ((c ^ (ROWB == 64 ? (r >> 1) & 3 : r & 7)) << 4));
}

// One warp's attention state in bf16: 16 heads x D values as tensor-instruction accumulators
// (rows gid and gid + 8 of the lane).
// R8: at most 8 heads, and nothing is done for rows gid + 8.
template <int D, bool R8>
struct WarpBf {
  using T = __nv_bfloat16;
  static constexpr int TW = PdShape<T, D>::TW, ROWB = PdShape<T, D>::ROWB;
  float o[D / 8][4], m0, m1, l0, l1, sl0, sl1;
  uint32_t qa[D / 16][4];

  __device__ __forceinline__ void begin(const DecodeParams &P, const unsigned char *qt, int h0, int nrows, int lane) {
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    m0 = m1 = -INFINITY;
    l0 = l1 = sl0 = sl1 = 0.f;
    const int gid = lane >> 2, mi = lane >> 3, r = (mi & 1) * 8 + (lane & 7);
    if (P.slopes) {
      if (gid < nrows) sl0 = P.slopes[h0 + gid] * kPgLog2e;
      if (!R8 && gid + 8 < nrows) sl1 = P.slopes[h0 + gid + 8] * kPgLog2e;
    }
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) pd_ldsm_x4(smem_u32(qt) + pd_at<ROWB>(r, ks * 2 + (mi >> 1)), qa[ks]);
  }

  __device__ __forceinline__ void tile(const DecodeParams &P, const UnitInfo &I, const unsigned char *kt,
                                       const unsigned char *vt, const unsigned char *, float (*)[8], const float2 *, int,
                                       int lane) {
    const int mi = lane >> 3, tig = lane & 3;
    float s[TW / 8][4];
#pragma unroll
    for (int i = 0; i < TW / 8; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
      for (int g = 0; g < TW / 16; ++g) {
        uint32_t b[4];
        pd_ldsm_x4(smem_u32(kt) + pd_at<ROWB>(g * 16 + (mi >> 1) * 8 + (lane & 7), ks * 2 + (mi & 1)), b);
        pd_mma(s[2 * g], qa[ks], b[0], b[1]);
        pd_mma(s[2 * g + 1], qa[ks], b[2], b[3]);
      }
    float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
    for (int t = 0; t < TW / 8; ++t)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int r = t * 8 + 2 * tig + y;
        const float far = (float)(I.len - 1 - (I.t0 + r));
        const bool ok = (I.there >> r) & 1u;
        float a = score_log2(P.f, s[t][y]);
        if (P.slopes) a -= sl0 * far;
        s[t][y] = ok ? a : -INFINITY;
        mx0 = fmaxf(mx0, s[t][y]);
        if (!R8) {
          float c = score_log2(P.f, s[t][2 + y]);
          if (P.slopes) c -= sl1 * far;
          s[t][2 + y] = ok ? c : -INFINITY;
          mx1 = fmaxf(mx1, s[t][2 + y]);
        }
      }
#pragma unroll
    for (int y = 1; y <= 2; y <<= 1) {
      mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, y));
      if (!R8) mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, y));
    }
    // a row's maximum moves a few times in a long sequence: the results are rescaled only then
    if (__any_sync(0xffffffffu, mx0 > m0 || (!R8 && mx1 > m1))) {
      const float n0 = fmaxf(m0, mx0), n1 = R8 ? m1 : fmaxf(m1, mx1);
      const float c0 = n0 == -INFINITY ? 1.f : ex2(m0 - n0), c1 = R8 || n1 == -INFINITY ? 1.f : ex2(m1 - n1);
      m0 = n0;
      m1 = n1;
      l0 *= c0;
      l1 *= c1;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        o[i][0] *= c0;
        o[i][1] *= c0;
        if (!R8) {
          o[i][2] *= c1;
          o[i][3] *= c1;
        }
      }
    }
    const float z0 = m0 == -INFINITY ? 0.f : m0, z1 = m1 == -INFINITY ? 0.f : m1;
    // weights, rounded to bf16 for the product (by 2^-8 of each at most; the sums take the
    // unrounded ones)
#pragma unroll
    for (int g = 0; g < TW / 16; ++g) {
      uint32_t pa[4];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const float *x = s[2 * g + t];
        const float p0 = ex2(x[0] - z0), p1 = ex2(x[1] - z0);
        l0 += p0 + p1;
        pa[2 * t] = pd_pack(p0, p1);
        pa[2 * t + 1] = 0;
        if (!R8) {
          const float p2 = ex2(x[2] - z1), p3 = ex2(x[3] - z1);
          l1 += p2 + p3;
          pa[2 * t + 1] = pd_pack(p2, p3);
        }
      }
      const int r = g * 16 + (mi & 1) * 8 + (lane & 7);
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        uint32_t b[4];
        pd_ldsm_x4_t(smem_u32(vt) + pd_at<ROWB>(r, j * 2 + (mi >> 1)), b);
        pd_mma(o[2 * j], pa, b[0], b[1]);
        pd_mma(o[2 * j + 1], pa, b[2], b[3]);
      }
    }
  }

  __device__ __forceinline__ void stats(float *m, float *l, int, int lane) {
    float s0 = l0, s1 = l1;
#pragma unroll
    for (int y = 1; y <= 2; y <<= 1) {
      s0 += __shfl_xor_sync(0xffffffffu, s0, y);
      s1 += __shfl_xor_sync(0xffffffffu, s1, y);
    }
    if ((lane & 3) == 0) {
      m[lane >> 2] = m0;
      m[(lane >> 2) + 8] = m1;
      l[lane >> 2] = s0;
      l[(lane >> 2) + 8] = s1;
    }
  }

  // acc[row][value] (+)= f[row] * o
  __device__ __forceinline__ void add_to(float *acc, const float *M, bool set, int, int lane) {
    const int gid = lane >> 2, col = 2 * (lane & 3);
    const float f0 = M[gid] == -INFINITY ? 0.f : ex2(m0 - M[gid]), f1 = M[gid + 8] == -INFINITY ? 0.f : ex2(m1 - M[gid + 8]);
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      float2 *a = reinterpret_cast<float2 *>(acc + gid * D + i * 8 + col), *c = reinterpret_cast<float2 *>(acc + (gid + 8) * D + i * 8 + col);
      float2 x = make_float2(o[i][0] * f0, o[i][1] * f0), y = make_float2(o[i][2] * f1, o[i][3] * f1);
      if (!set) {
        const float2 u = *a;
        x.x += u.x; x.y += u.y;
      }
      *a = x;
      if (!R8) {
        if (!set) {
          const float2 v = *c;
          y.x += v.x; y.y += v.y;
        }
        *c = y;
      }
    }
  }
};

// One warp's attention state in float32: 8 heads, the lane's four values of each (d = 64: two
// lanes share a chunk of values, each with half of the tokens).
template <int D>
struct WarpF32 {
  static constexpr int KC = D / 4, ROWB = D * 4, LPC = 32 / KC;
  float o[8][4], m[8], l[8], sl[8];

  __device__ __forceinline__ void begin(const DecodeParams &P, const unsigned char *, int h0, int nrows, int) {
#pragma unroll
    for (int h = 0; h < 8; ++h) {
      o[h][0] = o[h][1] = o[h][2] = o[h][3] = 0.f;
      m[h] = -INFINITY;
      l[h] = 0.f;
      sl[h] = P.slopes && h < nrows ? P.slopes[h0 + h] * kPgLog2e : 0.f;
    }
  }

  __device__ __forceinline__ void tile(const DecodeParams &P, const UnitInfo &I, const unsigned char *kt,
                                       const unsigned char *vt, const unsigned char *qt, float (*pw)[8], const float2 *,
                                       int nrows, int lane) {
    const int tk = lane >> 2, qd = lane & 3;              // token, and which of its four lanes
    const bool ok = (I.there >> tk) & 1u;
    const float far = (float)(I.len - 1 - (I.t0 + tk));
    // the lane's chunks of its key: 4 (j ^ (tk & 1)) + qd, so that two rows differ in bank group
    float4 kv[KC / 4];
#pragma unroll
    for (int j = 0; j < KC / 4; ++j)
      kv[j] = *reinterpret_cast<const float4 *>(kt + pd_at<ROWB>(tk, 4 * (j ^ (tk & 1)) + qd));
#pragma unroll
    for (int h = 0; h < 8; ++h)
      if (h < nrows) {
        const float4 *q = reinterpret_cast<const float4 *>(qt + h * ROWB) + qd;
        float a = 0.f, b = 0.f;
#pragma unroll
        for (int j = 0; j < KC / 4; j += 2) {
          const float4 x = q[4 * (j ^ (tk & 1))], y = q[4 * ((j + 1) ^ (tk & 1))];
          a = fmaf(x.x, kv[j].x, fmaf(x.y, kv[j].y, fmaf(x.z, kv[j].z, fmaf(x.w, kv[j].w, a))));
          b = fmaf(y.x, kv[j + 1].x, fmaf(y.y, kv[j + 1].y, fmaf(y.z, kv[j + 1].z, fmaf(y.w, kv[j + 1].w, b))));
        }
        float s = a + b;
        s += __shfl_xor_sync(0xffffffffu, s, 1);
        s += __shfl_xor_sync(0xffffffffu, s, 2);
        s = score_log2(P.f, s) - sl[h] * far;
        s = ok ? s : -INFINITY;
        float mx = s;
#pragma unroll
        for (int y = 4; y < 32; y <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, y));
        if (mx > m[h]) {                                  // the same in every lane
          const float c = ex2(m[h] - mx);
          m[h] = mx;
          l[h] *= c;
#pragma unroll
          for (int e = 0; e < 4; ++e) o[h][e] *= c;
        }
        const float p = ex2(s - (m[h] == -INFINITY ? 0.f : m[h]));
        l[h] += p;
        if (qd == 0) pw[h][tk] = p;
      }
    __syncwarp();
    const int c = lane % KC, part = lane / KC;
    float4 vv[8 / LPC];
#pragma unroll
    for (int t = 0; t < 8 / LPC; ++t)
      vv[t] = *reinterpret_cast<const float4 *>(vt + pd_at<ROWB>(part * (8 / LPC) + t, c));
#pragma unroll
    for (int h = 0; h < 8; ++h)
      if (h < nrows) {
#pragma unroll
        for (int t = 0; t < 8 / LPC; t += 4) {
          const float4 p = *reinterpret_cast<const float4 *>(&pw[h][part * (8 / LPC) + t]);
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float w = u == 0 ? p.x : u == 1 ? p.y : u == 2 ? p.z : p.w;
            o[h][0] = fmaf(w, vv[t + u].x, o[h][0]);
            o[h][1] = fmaf(w, vv[t + u].y, o[h][1]);
            o[h][2] = fmaf(w, vv[t + u].z, o[h][2]);
            o[h][3] = fmaf(w, vv[t + u].w, o[h][3]);
          }
        }
      }
  }

  __device__ __forceinline__ void stats(float *ms, float *ls, int nrows, int lane) {
#pragma unroll
    for (int h = 0; h < 8; ++h)
      if (h < nrows) {
        float s = l[h];                                   // the four lanes of a token hold the same
#pragma unroll
        for (int y = 4; y < 32; y <<= 1) s += __shfl_xor_sync(0xffffffffu, s, y);
        if (lane == 0) {
          ms[h] = m[h];
          ls[h] = s;
        }
      }
  }

  __device__ __forceinline__ void add_to(float *acc, const float *M, bool set, int nrows, int lane) {
    const int c = lane % KC;
#pragma unroll
    for (int h = 0; h < 8; ++h)
      if (h < nrows) {
        const float f = M[h] == -INFINITY ? 0.f : ex2(m[h] - M[h]);
        float4 x = make_float4(o[h][0] * f, o[h][1] * f, o[h][2] * f, o[h][3] * f);
        if (LPC == 2) {
          x.x += __shfl_xor_sync(0xffffffffu, x.x, 16);
          x.y += __shfl_xor_sync(0xffffffffu, x.y, 16);
          x.z += __shfl_xor_sync(0xffffffffu, x.z, 16);
          x.w += __shfl_xor_sync(0xffffffffu, x.w, 16);
        }
        float4 *a = reinterpret_cast<float4 *>(acc + h * D) + c;
        if (!set) {
          const float4 u = *a;
          x.x += u.x; x.y += u.y; x.z += u.z; x.w += u.w;
        }
        __syncwarp();                                     // d = 64: both lanes of a chunk have read it
        *a = x;
      }
  }
};

// c += a (16x16, row) * b (16x8, col), float16 inputs, f32 accumulate
__device__ __forceinline__ void pd_mma_h(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pd_pack_h(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Transposes an 8 x 8 matrix of 16-bit values spread over the warp (row lane / 4, columns 2 (lane % 4), + 1).
__device__ __forceinline__ uint32_t pd_transpose(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// One warp's attention state over e4m3 codes.  Tokens are the M of the products (16 at a time) and
// query heads their N (8, or 8 twice): a group of 8 heads leaves nothing idle, and the codes, turned
// into float16 (exact, one instruction for two), are the A operand:
//   S^T = K Q^T: a lane takes 16 (d = 64) or 32 codes in a row of a token -- the order of the sum over
//     d is free, so that the query takes the same one -- without a shuffle;
//   O^T = V^T P^T: pairs of codes by the transposing matrix load, tokens and values put in order by one
//     byte permutation; P^T by the transposing move.
// A query is scaled to a largest value in [2^13, 2^14) by a power of two.  The exponents of keys
// multiply the scores; those of values, ve, are added to them: with y = x + ve,
//   o = sum 2^(y - z) code,  l = sum 2^(y - z) 2^-ve,
// z = 10 below a maximum of y that moves when it is passed by 5, so that weights stay below 2^15, and
// those of float16's lowest step, 2^-24, are 2^-34 of the largest.
// MULTI: rows are (new token, query head) pairs, each with an end of its own; their scaled queries lie in
// shared memory (pd_rows), four or two tiles of 8 rows behind one another for each step of the sum.
template <int D, int NT, bool MULTI>
struct WarpQ8 {
  static constexpr int ROWB = D, QROWB = 2 * D, KS = D / 16, CH = D / 64, MT = PdShape<E4m3, D>::TW / 16;
  float o[D / 16][NT][4], m[NT][2], l[NT][2], sl[MULTI ? 1 : NT][2], fa[MULTI ? 1 : NT][2];   // rows 8 nt + 2 (lane % 4), + 1
  uint32_t qb[MULTI ? 1 : NT][KS][2];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int j = 0; j < D / 16; ++j) o[j][nt][0] = o[j][nt][1] = o[j][nt][2] = o[j][nt][3] = 0.f;
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
    }
  }

  __device__ __forceinline__ void begin(const DecodeParams &P, const unsigned char *qt, int h0, int nrows, int lane) {
    const int gid = lane >> 2, tig = lane & 3;
    clear();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      // head 8 nt + gid, values 16 CH tig ..
      const uint4 *q = reinterpret_cast<const uint4 *>(qt + (8 * nt + gid) * QROWB + tig * 32 * CH);
      float x[16 * CH], mx = 0.f;
#pragma unroll
      for (int c = 0; c < 2 * CH; ++c) {
        const uint4 u = q[c];
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[8 * c + 2 * e] = __uint_as_float(w[e] << 16);
          x[8 * c + 2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
        }
      }
#pragma unroll
      for (int e = 0; e < 16 * CH; ++e) mx = fmaxf(mx, fabsf(x[e]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const int up = q8_query_exp(mx);
      const float f = exp2i(up);
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        qb[nt][ks][0] = pd_pack_h(x[4 * ks] * f, x[4 * ks + 1] * f);
        qb[nt][ks][1] = pd_pack_h(x[4 * ks + 2] * f, x[4 * ks + 3] * f);
      }
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int h = 8 * nt + 2 * tig + y;
        fa[nt][y] = P.f.a * exp2i(-__shfl_sync(0xffffffffu, up, 4 * (2 * tig + y)));
        sl[nt][y] = P.slopes && h < nrows ? P.slopes[h0 + h] * kPgLog2e : 0.f;
      }
    }
  }

  // MULTI: this warp's tile of 8 rows of a unit, row `base + gid` of the sequence's (token r / G, head r % G):
  // scaled to float16 into qf, [step][pair of tiles][lane][tile of the pair][2], and what else a row has.
  static __device__ __forceinline__ void rows_begin(const DecodeParams &P, unsigned char *qf, PdRow *row, int nt, int base, int nr,
                                                    int s0, int n, int len, int kvh, int lane) {
    const int gid = lane >> 2, tig = lane & 3, r = base + gid;
    const bool there = r < nr;
    const int tk = there ? div_by(P.group, r) : 0, hd = there ? kvh * P.G + r - tk * P.G : 0;
    const uint4 *q = reinterpret_cast<const uint4 *>((const __nv_bfloat16 *)P.q + (int64_t)(s0 + tk) * P.q_stride + (int64_t)hd * D) + tig * 2 * CH;
    uint32_t w[8 * CH];
#pragma unroll
    for (int c = 0; c < 2 * CH; ++c) {
      const uint4 u = there ? __ldg(q + c) : make_uint4(0, 0, 0, 0);
      w[4 * c] = u.x; w[4 * c + 1] = u.y; w[4 * c + 2] = u.z; w[4 * c + 3] = u.w;
    }
    float mx = 0.f;
#pragma unroll
    for (int e = 0; e < 8 * CH; ++e)
      mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(w[e] << 16)), fabsf(__uint_as_float(w[e] & 0xffff0000u))));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    const int up = q8_query_exp(mx);
    const float f = exp2i(up);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const uint32_t a = w[2 * ks], b = w[2 * ks + 1];
      *reinterpret_cast<uint2 *>(qf + (((ks * (NT / 2) + (nt >> 1)) * 32 + lane) * 2 + (nt & 1)) * 8) =
          make_uint2(pd_pack_h(__uint_as_float(a << 16) * f, __uint_as_float(a & 0xffff0000u) * f),
                     pd_pack_h(__uint_as_float(b << 16) * f, __uint_as_float(b & 0xffff0000u) * f));
    }
    if (tig == 0) {
      const int pos = there ? max(len - n + tk, -1) : -1;
      row[8 * nt + gid] = {P.f.a * exp2i(-up), P.slopes && there ? P.slopes[hd] * kPgLog2e : 0.f, pos,
                           pos < 0 ? 0x7fffffff : P.window ? max(pos - P.window + 1, 0) : 0};
    }
  }

  __device__ __forceinline__ void tile(const DecodeParams &P, const UnitInfo &I, const unsigned char *kt,
                                       const unsigned char *vt, const unsigned char *qf, float (*)[8], const float2 *ex,
                                       int, int lane, const PdRow *row = nullptr, bool seen = true, int pre = 0) {
    const int gid = lane >> 2, tig = lane & 3, mi = lane >> 3;
    float s[MT][NT][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) s[mt][nt][0] = s[mt][nt][1] = s[mt][nt][2] = s[mt][nt][3] = 0.f;
    if constexpr (MULTI) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        uint32_t k[MT][2][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int r = 0; r < 2; ++r)
            *reinterpret_cast<uint4 *>(&k[mt][r][0]) =
                *reinterpret_cast<const uint4 *>(kt + pd_at<ROWB>(mt * 16 + r * 8 + gid, tig * CH + c));
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          uint4 b[NT / 2];
#pragma unroll
          for (int np = 0; np < NT / 2; ++np) b[np] = reinterpret_cast<const uint4 *>(qf)[((4 * c + ks) * (NT / 2) + np) * 32 + lane];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            uint32_t a[4];
            q8_halves(k[mt][0][ks], a[0], a[2]);
            q8_halves(k[mt][1][ks], a[1], a[3]);
#pragma unroll
            for (int np = 0; np < NT / 2; ++np) {
              pd_mma_h(s[mt][2 * np], a, b[np].x, b[np].y);
              pd_mma_h(s[mt][2 * np + 1], a, b[np].z, b[np].w);
            }
          }
        }
      }
    }
#pragma unroll
    for (int mt = 0; mt < (MULTI ? 0 : MT); ++mt) {
      uint32_t k[2][4 * CH];
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int c = 0; c < CH; ++c)
          *reinterpret_cast<uint4 *>(&k[r][4 * c]) =
              *reinterpret_cast<const uint4 *>(kt + pd_at<ROWB>(mt * 16 + r * 8 + gid, tig * CH + c));
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        uint32_t a[4];
        q8_halves(k[0][ks], a[0], a[2]);
        q8_halves(k[1][ks], a[1], a[3]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) pd_mma_h(s[mt][nt], a, qb[MULTI ? 0 : nt][ks][0], qb[MULTI ? 0 : nt][ks][1]);
      }
    }
    float mx[NT][2], vx[MT][2], vf[MT][2];
    // score (mt, hf, nt, y): token 16 mt + 8 hf + gid, row 8 nt + 2 tig + y
    auto scores = [&](auto &&f) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int y = 0; y < 2; ++y) f(s[mt][nt][2 * hf + y], mt, hf, nt, y);
    };
    {
      float fr[NT][2], kf[MT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          fr[nt][y] = MULTI ? row[8 * nt + 2 * tig + y].fa : fa[MULTI ? 0 : nt][y];
          mx[nt][y] = -INFINITY;
        }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const float2 e = ex[mt * 16 + hf * 8 + gid];
          kf[mt][hf] = __uint_as_float(__float_as_uint(e.x) & 0xffff0000u);
          vx[mt][hf] = e.y;
          vf[mt][hf] = __uint_as_float(__float_as_uint(e.x) << 16);
        }
      // plain scores in two steps, and else what is between them
      if (!P.f.capped && !P.slopes && seen && I.there == 0xffffffffu) {
        scores([&](float &x, int mt, int hf, int nt, int y) { x = fmaf(x * kf[mt][hf], fr[nt][y], vx[mt][hf]); });
      } else {
        scores([&](float &x, int mt, int hf, int nt, int y) { x = x * kf[mt][hf] * fr[nt][y]; });
        if (P.f.capped) {                                 // the polynomial where every score of the warp is small enough
          float um = 0.f;
          scores([&](float &x, int, int, int, int) { um = fmaxf(um, fabsf(x)); });
          if (__all_sync(0xffffffffu, um * um <= kTanhW)) scores([&](float &x, int, int, int, int) { x = P.f.c * tanh_small(x); });
          else scores([&](float &x, int, int, int, int) { x = P.f.c * tanh_ex2(x); });
        }
        if constexpr (MULTI) {
          if (P.slopes || !seen)                          // the rows' own biases and ends
            scores([&](float &x, int mt, int hf, int nt, int y) {
              const PdRow w = row[8 * nt + 2 * tig + y];
              const int t = I.t0 + mt * 16 + hf * 8 + gid;
              x -= w.sl * fabsf((float)(w.pos - t));
              x = (t <= w.pos && t >= w.lo) || (t < pre && w.pos >= 0) ? x : -INFINITY;
            });
        } else if (P.slopes) {
          const float far = (float)(I.len - 1 - I.t0 - gid);
          scores([&](float &x, int mt, int hf, int nt, int y) { x -= sl[MULTI ? 0 : nt][y] * (far - (float)(mt * 16 + hf * 8)); });
        }
        if (I.there != 0xffffffffu)
          scores([&](float &x, int mt, int hf, int, int) { x = (I.there >> (mt * 16 + hf * 8 + gid)) & 1u ? x : -INFINITY; });
        scores([&](float &x, int mt, int hf, int, int) { x += vx[mt][hf]; });
      }
    }
    scores([&](float &x, int, int, int nt, int y) { mx[nt][y] = fmaxf(mx[nt][y], x); });
    bool up = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int y = 0; y < 2; ++y) up |= mx[nt][y] > m[nt][y] + 5.f;
    if (__any_sync(0xffffffffu, up)) {                    // a few times in a long sequence
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) mx[nt][y] = fmaxf(mx[nt][y], __shfl_xor_sync(0xffffffffu, mx[nt][y], x));
          const float n = mx[nt][y] > m[nt][y] + 5.f ? mx[nt][y] : m[nt][y];
          const float c = n == -INFINITY ? 1.f : ex2(m[nt][y] - n);
          m[nt][y] = n;
          l[nt][y] *= c;
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            o[j][nt][y] *= c;
            o[j][nt][2 + y] *= c;
          }
        }
    }
    uint32_t pb[MT][NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float z0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0] - 10.f, z1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1] - 10.f;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          // weights, rounded to float16 for the product (by 2^-11 of each at most; the sums take the
          // unrounded ones)
          const float p0 = ex2(s[mt][nt][2 * hf] - z0), p1 = ex2(s[mt][nt][2 * hf + 1] - z1);
          l[nt][0] = fmaf(p0, vf[mt][hf], l[nt][0]);
          l[nt][1] = fmaf(p1, vf[mt][hf], l[nt][1]);
          pb[mt][nt][hf] = pd_transpose(pd_pack_h(p0, p1));
        }
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int j = 0; j < D / 16; j += 2) {
        uint32_t b[4];
        pd_ldsm_x4_t(smem_u32(vt) + pd_at<ROWB>(mt * 16 + (mi & 1) * 8 + (lane & 7), j + (mi >> 1)), b);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t a[4];                                  // rows gid: value 16 (j + x) + 2 gid, rows gid + 8: the next one
          q8_halves(__byte_perm(b[2 * x], 0, 0x3120), a[0], a[1]);
          q8_halves(__byte_perm(b[2 * x + 1], 0, 0x3120), a[2], a[3]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) pd_mma_h(o[j + x][nt], a, pb[mt][nt][0], pb[mt][nt][1]);
        }
      }
  }

  __device__ __forceinline__ float zero(float x) const { return x == -INFINITY ? x : x - 10.f; }   // what o and l are relative to
  __device__ __forceinline__ void stats(float *ms, float *ls, int, int lane) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        float s = l[nt][y];
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        if (lane < 4) {
          ms[8 * nt + 2 * lane + y] = zero(m[nt][y]);
          ls[8 * nt + 2 * lane + y] = s;
        }
      }
  }

  __device__ __forceinline__ void add_to(float *acc, const float *M, bool set, int nrows, int lane) {
    const int gid = lane >> 2, tig = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int h = 8 * nt + 2 * tig + y;
        if (h >= nrows) continue;
        const float f = M[h] == -INFINITY ? 0.f : ex2(zero(m[nt][y]) - M[h]);
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          float2 *a = reinterpret_cast<float2 *>(acc + h * D + 16 * j + 2 * gid);
          float2 x = make_float2(o[j][nt][y] * f, o[j][nt][2 + y] * f);
          if (!set) {
            const float2 u = *a;
            x.x += u.x; x.y += u.y;
          }
          *a = x;
        }
      }
  }
};

// NT: bf16: 1 for at most 8 heads to a KV head.
template <typename T, int D, int NT, bool MULTI>
__global__ void __launch_bounds__(PdShape<T, D, NT, MULTI>::THREADS, PdShape<T, D, NT, MULTI>::CTAS)
    paged_decode_kernel(const __grid_constant__ DecodeParams P, const __grid_constant__ CUtensorMap kmap,
                        const __grid_constant__ CUtensorMap vmap, int box) {
  using Sh = PdShape<T, D, NT, MULTI>;
  using Act = typename Sh::Act;
  using State = std::conditional_t<Sh::Q8, WarpQ8<D, NT, MULTI>, std::conditional_t<Sh::BF, WarpBf<D, NT == 1>, WarpF32<D>>>;
  constexpr int PD_WARPS = Sh::WARPS, PD_THREADS = Sh::THREADS;
  constexpr int TILE = Sh::TILE, TW = Sh::TW, ST = Sh::STAGES, ROWB = Sh::ROWB, HALF = Sh::HALF, ROWS = Sh::ROWS;
  constexpr int QROWB = Sh::QROWB;
  constexpr int ACCS = Sh::Q8 && NT == 1 ? 2 : 1;        // sums of the warps' results: with 8 rows there is room for two
  constexpr int KC = ROWB / 16, QC = QROWB / 16;         // 16-byte chunks of a key, of a query
  extern __shared__ unsigned char pd_raw[];
  unsigned char *sm = pd_raw + ((0u - smem_u32(pd_raw)) & (Sh::ALIGN - 1));   // (an offset: it stays a pointer to shared memory)
  unsigned char *qs = sm + PD_WARPS * ST * 2 * HALF;     // the query tile
  float *acc = reinterpret_cast<float *>(qs + (Sh::BF ? ROWS * QROWB : 0));               // the warps' results, joined
  auto &S = *reinterpret_cast<PdShared<T, D, NT, MULTI> *>(qs + Sh::QACC);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const echo_paged_kv_t &C = P.C;
  // groups of ROWS rows of a KV head, and the rows of sequence b
  auto groups = [&](int rows) { return MULTI ? (int)(((int64_t)rows * P.G + ROWS - 1) / ROWS) : P.HG; };
  // weight of an item of `tiles` tiles, and how far a run that ends at u1 comes in one that begins at ws
  const bool whole_items = Sh::Q8 && P.whole;
  auto weight = [&](int tiles) { return whole_items ? 1u : (uint32_t)(tiles + 1); };
  auto run_end = [&](int tiles, uint32_t ws, uint32_t u1) {
    return whole_items ? (ws < u1 ? tiles : 0) : min(tiles, (int)(u1 - ws) - 1);
  };
  auto rows_of = [&](int b) {
    int s0;
    return MULTI ? decode_rows(P, b, s0) : 1;
  };
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- this CTA's run: a scan over the sequences, PD_THREADS at a time; with few sequences one
  // scan gives the total and finds the place.  Whether it is found is known from the barrier behind
  // the writes of S.seq and S.before, the same in every thread: nobody reads either ahead of it
  uint32_t total = 0, end = 0, n = 0, per = 0, u0 = 0, u1 = 0;
  bool found = false, bad = false, some = false;
  if (tid == 0) P.rec[blockIdx.x * 4] = 0;
  if (Sh::Q8) {
    if (tid == 0) {
      for (int i = 0; i < PD_WARPS * ST; ++i) mbar_init(&S.full[0][i], 32);
      fence_mbar_init();
    }
    if (tid == 32 && box) {
      tma_prefetch_desc(&kmap);
      tma_prefetch_desc(&vmap);
    }
  }
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    uint32_t at = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < P.B && !found; b0 += PD_THREADS) {
      if (pass == 0 || P.B > PD_THREADS) {
        const int rb = b0 + tid < P.B ? rows_of(b0 + tid) : 0;
        if (MULTI && b0 + tid < P.B) {
          const int s = min(P.q_start[b0 + tid], P.N), e = max(P.q_start[b0 + tid + 1], 0);
          bad |= s > e;
          some |= (int64_t)(min(e, P.N) - max(s, 0)) * P.G > P.most;
        }
        n = rb ? weight(decode_span<MULTI>(P, b0 + tid, TILE, rb).n()) * (uint32_t)(C.n_kv_heads * groups(rb)) : 0;
        uint32_t x = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        __syncthreads();
        if (lane == 31) S.sum[warp] = x;
        __syncthreads();
        end = at + x;
#pragma unroll
        for (int w = 0; w < PD_WARPS; ++w) {
          if (w < warp) end += S.sum[w];
          at += S.sum[w];
        }
      }
      if (pass == 1) {
        const bool mine = end - n <= u0 && u0 < end;
        if (mine) { S.seq = b0 + tid; S.before = end - n; }
        found = __syncthreads_or(mine);
      }
    }
    if (pass == 0) {
      if (MULTI) {
        const bool descends = __syncthreads_or(bad);
        some = __syncthreads_or(some) && !descends;
        if (blockIdx.x == 0 && tid == 0) *P.some = some;
        if (descends) {                                  // no work is done
          if (tid == 0) paged_fail(C.status, ECHO_ERR_INVALID_ARG);
          return;
        }
      }
      total = at;
      per = max((total + P.nctas - 1) / P.nctas, whole_items ? 1u : (uint32_t)Sh::MIN_WEIGHT);
      u0 = per * blockIdx.x;
      u1 = min(total, u0 + per);
      if (u0 >= total) return;
    }
  }
  if (!found) return;                                    // (lengths that another stream changes between the passes)

  // ---- cursor of the look-ups (the same in every thread): tile ci of its part [i0, ce) of the
  // current (sequence, head group), which begins at weight ws
  PdPlace in_registers;
  PdPlace &K = Sh::NO_REGS ? S.place[Sh::NO_REGS ? warp : 0] : in_registers;
  int ci, i0, ce, c0;                                    // c0: CTA of the current one's first unit
  {
    PdPlace k = {};
    k.cb = S.seq;
    const int rows = rows_of(k.cb);
    k.cHG = groups(rows);
    k.cs = decode_span<MULTI>(P, k.cb, TILE, rows);
    k.cn = k.cs.n();
    const int hh0 = (int)((u0 - S.before) / weight(k.cn));
    k.ckvh = hh0 / k.cHG;
    k.chg = hh0 - k.ckvh * k.cHG;
    k.ws = S.before + (uint32_t)hh0 * weight(k.cn);
    i0 = ci = max(0, (int)(u0 - k.ws) - 1);
    ce = run_end(k.cn, k.ws, u1);
    c0 = (int)((k.ws + 1) / per);
    K = k;
  }
  __syncwarp();
  int cu = 0;                                            // units looked up
  int32_t ent = -1;                                      // the last one's page-table entry of this lane's token
  int tok = -1, prow = 0;                                // that token, and its row of the page
  UnitInfo *ring = S.info[warp];
  auto look_up = [&]() {
    tok = -1;
    if (ci >= ce) return;                                // the run is over
    const int t0 = K.cs.t.tile(ci) * TILE + warp * TW;
    const int t = t0 + lane;
    if (lane < TW && t >= K.cs.first && t < K.cs.len && (t >= K.cs.lo || t < K.cs.pre)) {
      const int pg = div_by(P.page, t);
      tok = t;
      prow = t - pg * C.page_tokens;
      ent = __ldg(C.page_table + (int64_t)K.cb * C.max_pages + pg);
    }
    if (lane == 0) {
      UnitInfo &I = ring[cu % PD_RING];
      I.b = K.cb; I.kvh = K.ckvh; I.hg = K.chg; I.t0 = t0; I.len = K.cs.len;
      I.flags = (ci == i0 ? 1 : 0) | (ci + 1 == ce ? 2 : 0) | (i0 > 0 ? 4 : 0) | (ce < K.cn ? 8 : 0);
      I.c0 = c0;
    }
    ++cu;
    if (++ci == ce && ce == K.cn) {                      // on to the next (sequence, head group)
      PdPlace k = K;
      __syncwarp();                                      // every lane has it
      k.ws += weight(k.cn);
      if (++k.chg == k.cHG) k.chg = 0, ++k.ckvh;
      if (k.ckvh == C.n_kv_heads) {
        k.ckvh = 0;
        int rows;
        do {
          ++k.cb;
          rows = k.cb < P.B ? rows_of(k.cb) : 1;
        } while (MULTI && rows == 0);                    // sequences without rows weigh nothing
        if (k.cb < P.B) {
          k.cHG = groups(rows);
          k.cs = decode_span<MULTI>(P, k.cb, TILE, rows);
          k.cn = k.cs.n();
        } else {
          k.ws = u1;
        }
      }
      i0 = ci = 0;
      ce = run_end(k.cn, k.ws, u1);
      c0 = (int)((k.ws + 1) / per);
      K = k;
      __syncwarp();
    }
  };
  // turns unit x's entries into offsets and copies the warp's keys and values into its stage
  unsigned char *stages = sm + warp * ST * 2 * HALF;
  uint32_t pend = 0;                                     // e4m3: exponent bytes of the unit loaded last
  bool dead = false;                                     // a bounded wait gave up: reported, and nothing more is loaded
  int loaded = 0;
  auto load = [&](int x) {
    if (Sh::Q8 && x > 0 && x <= cu) {
      const int ve = q8_exp(pend >> 8);
      S.ex[Sh::Q8 ? warp : 0][(x - 1) % ST][lane] =
          make_float2(__uint_as_float(__float_as_uint(exp2i(q8_exp(pend & 255u))) | __float_as_uint(exp2i(-ve)) >> 16), (float)ve);
    }
    if (x < cu && !(Sh::Q8 && dead)) {
      loaded = x + 1;
      const bool page = tok >= 0 && ent >= 0 && ent < C.n_pages;
      if (tok >= 0 && !page) paged_fail(C.status, ECHO_ERR_PAGE);
      const uint32_t there = __ballot_sync(0xffffffffu, page);
      UnitInfo &I = ring[x % PD_RING];
      if (lane == 0) I.there = there;
      __syncwarp();
      const int kvh = I.kvh;
      unsigned char *kt = stages + (x % ST) * 2 * HALF, *vt = kt + HALF;
      uint64_t *full = &S.full[Sh::Q8 ? warp : 0][x % ST];
      if (Sh::Q8 && box && there == 0xffffffffu) {       // by TMA, box by box
        if (lane == 0) mbar_arrive_expect_tx(full, 2 * HALF);
        else mbar_arrive(full);
#pragma unroll 1
        for (int i = 0; i < TW; i += box) {
          const int e = __shfl_sync(0xffffffffu, ent, i), r = __shfl_sync(0xffffffffu, prow, i);
          if (pg_elect()) {
            pg_tma4(kt + i * ROWB, &kmap, full, 0, r, kvh, e);
            pg_tma4(vt + i * ROWB, &vmap, full, 0, r, kvh, e);
          }
        }
      } else {
        const int64_t row = page ? (int64_t)ent * C.page_stride + (int64_t)prow * C.row_stride : -1;
        const int64_t head = (int64_t)kvh * C.head_stride;
        const T *kb = (const T *)C.k + head, *vb = (const T *)C.v + head;
#pragma unroll
        for (int i = 0; i < TW * KC / 32; ++i) {
          const int r = (i * 32 + lane) / KC, c = (i * 32 + lane) % KC;
          const int64_t g = __shfl_sync(0xffffffffu, row, r);
          const int64_t off = (g >= 0 ? g : 0) + c * (16 / (int)sizeof(T));
          const uint32_t nbytes = g >= 0 ? 16u : 0u;
          cp_async_16(kt + pd_at<ROWB>(r, c), kb + off, nbytes);
          cp_async_16(vt + pd_at<ROWB>(r, c), vb + off, nbytes);
        }
        if (Sh::Q8) pd_cp_arrive(full);
      }
      if (Sh::Q8 && page) {
        const int64_t e = (int64_t)ent * P.X.page_stride + (int64_t)prow * P.X.row_stride + (int64_t)kvh * P.X.head_stride;
        pend = (uint32_t)__ldg(P.X.k + e) | ((uint32_t)__ldg(P.X.v + e) << 8);
      }
    }
    if (Sh::Q8) __syncwarp();
    else cp_async_commit();
  };
  for (int i = 0; i < ST - 1; ++i) {
    look_up();
    load(i);
  }
  look_up();

  State A;
  int &nrows = K.nrows, &h0 = K.h0, &s0 = K.s0, &r0 = K.r0, &minpos = K.minpos, &maxlo = K.maxlo, &pre = K.pre;
  // row r of the unit: its place in the results, in rows of D values
  auto out_row = [&](int b, int kvh, int r) {
    if (!MULTI) return (int64_t)b * P.Hq + h0 + r;
    const int tk = div_by(P.group, r0 + r);
    return (int64_t)(s0 + tk) * P.Hq + kvh * P.G + (r0 + r - tk * P.G);
  };
  for (int x = 0; x < cu; ++x) {                         // (the look-ups are ahead of it, or over)
    if (Sh::Q8) {
      if (!dead && !__all_sync(0xffffffffu, mbar_wait(&S.full[Sh::Q8 ? warp : 0][x % ST], (x / ST) & 1))) {
        paged_fail(C.status, ECHO_ERR_TIMEOUT);
        dead = true;
      }
      if (box && ring[x % PD_RING].there != 0xffffffffu) fence_proxy_async_smem();   // came by cp.async: TMA may take its place
    } else {
      cp_async_wait<ST - 2>();
    }
    __syncwarp();                                        // unit x is there, and unit x - 1's stage is free
    load(x + ST - 1);
    look_up();                                           // unit x + ST
    const UnitInfo &I = ring[x % PD_RING];
    if (I.flags & 1) {                                   // a new (sequence, head group): every warp is past the last one
      const int hg = I.hg;
      if (!Sh::BF) __syncthreads();                      // the last one's joined results lie in the query tile's place
      if constexpr (MULTI) {
        const int nq = decode_rows(P, I.b, s0);
        r0 = hg * ROWS;
        nrows = min(ROWS, nq * P.G - r0);
        pre = P.prefix_len ? min(P.prefix_len[I.b], I.len) : 0;
        if (tid == 0 && I.len < nq) paged_fail(C.status, ECHO_ERR_INVALID_ARG);
        if (warp < NT) State::rows_begin(P, qs, S.row, warp, r0 + 8 * warp, nq * P.G, s0, nq, I.len, I.kvh, lane);
        __syncthreads();
        minpos = __reduce_min_sync(0xffffffffu, lane < nrows ? S.row[lane].pos : 0x7fffffff);
        maxlo = __reduce_max_sync(0xffffffffu, lane < nrows ? S.row[lane].lo : 0);
        A.clear();
      } else {
        h0 = I.kvh * P.G + hg * ROWS;
        nrows = min(ROWS, P.G - hg * ROWS);
        const Act *q = (const Act *)P.q + (int64_t)I.b * P.q_stride + (int64_t)h0 * D;
        for (int i = tid; i < ROWS * QC; i += PD_THREADS) {
          const int r = i / QC, c = i % QC;
          uint4 v = make_uint4(0, 0, 0, 0);
          if (r < nrows) v = reinterpret_cast<const uint4 *>(q + (int64_t)r * D)[c];
          *reinterpret_cast<uint4 *>(qs + (Sh::BF ? pd_at<ROWB>(r, c) : r * QROWB + c * 16)) = v;
        }
        __syncthreads();
        A.begin(P, qs, h0, nrows, lane);
      }
    }
    const unsigned char *kt = stages + (x % ST) * 2 * HALF;
    if constexpr (MULTI) {
      const bool seen = (I.t0 + TW - 1 <= minpos && I.t0 >= maxlo) || (I.t0 + TW <= pre && minpos >= 0);
      A.tile(P, I, kt, kt + HALF, qs, nullptr, S.ex[warp][x % ST], nrows, lane, S.row, seen, pre);
    } else {
      A.tile(P, I, kt, kt + HALF, qs, S.p[Sh::F32 ? warp : 0], S.ex[Sh::Q8 ? warp : 0][x % ST], nrows, lane);
    }
    if (I.flags & 2) {                                   // the run's last unit of this (sequence, head group)
      A.stats(S.m[warp], S.l[warp], nrows, lane);
      __syncthreads();
      float *M = S.m[0];
      if (warp == 0 && lane < nrows) {                   // joined: (m, l) of warp 0's entries
        float mm = S.m[0][lane], ll = 0.f;
#pragma unroll
        for (int w = 1; w < PD_WARPS; ++w) mm = fmaxf(mm, S.m[w][lane]);
#pragma unroll
        for (int w = 0; w < PD_WARPS; ++w) ll += mm == -INFINITY ? 0.f : ex2(S.m[w][lane] - mm) * S.l[w][lane];
        S.m[0][lane] = mm;
        S.l[0][lane] = ll;
      }
      for (int w = 0; w < PD_WARPS; w += ACCS) {
        __syncthreads();
        if (warp / ACCS == w / ACCS) A.add_to(acc + (warp % ACCS) * 8 * D, M, w == 0, nrows, lane);
      }
      __syncthreads();
      const bool whole = !(I.flags & 12);
      const int64_t slot = 2 * blockIdx.x + ((I.flags & 4) ? 0 : 1);
      for (int i = tid; i < nrows * (D / 4); i += PD_THREADS) {
        const int r = i / (D / 4), c = i % (D / 4);
        float4 v = *reinterpret_cast<const float4 *>(acc + r * D + 4 * c);
        if (ACCS == 2) {
          const float4 u = *reinterpret_cast<const float4 *>(acc + (8 + r) * D + 4 * c);
          v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
        }
        if (whole) {
          const float L = S.l[0][r], inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
          v.x *= inv; v.y *= inv; v.z *= inv; v.w *= inv;
          Act *dst = (Act *)P.out + out_row(I.b, I.kvh, r) * D + 4 * c;
          if constexpr (!Sh::F32) *reinterpret_cast<uint2 *>(dst) = make_uint2(pd_pack(v.x, v.y), pd_pack(v.z, v.w));
          else *reinterpret_cast<float4 *>(dst) = v;
        } else {
          *reinterpret_cast<float4 *>(P.po + (slot * P.prows + r) * D + 4 * c) = v;
        }
      }
      if (tid < nrows) {
        const float mm = S.m[0][tid], L = S.l[0][tid];
        if (whole) P.lse[out_row(I.b, I.kvh, tid)] = L == 0.f ? -INFINITY : (mm + log2f(L)) * kPgLn2;
        else *reinterpret_cast<float2 *>(P.pml + (slot * P.prows + tid) * 2) = make_float2(mm, L);
      }
      if (tid == 0 && (I.flags & 12) == 4) {             // a split one ends here: to be joined
        int32_t *rec = P.rec + blockIdx.x * 4;
        rec[1] = I.c0;
        rec[2] = I.b;
        rec[3] = I.kvh * (MULTI ? groups(rows_of(I.b)) : P.HG) + I.hg;
        rec[0] = 1;
      }
    }
  }
  cp_async_wait_all();
  // after a wait that gave up, the copies in flight land before the CTA ends (bounded waits)
  for (int x = max(0, loaded - ST); Sh::Q8 && dead && x < loaded; ++x) mbar_wait(&S.full[Sh::Q8 ? warp : 0][x % ST], (x / ST) & 1);
}

// Joins the partials of the (sequence, head group) that ends in CTA blockIdx.x: slot 1 of its
// first CTA, then slot 0 of the following ones.  A block takes one row, a thread one value; the
// maxima first, then the weighted sums in the order of the CTAs.
template <typename T, int D, int NT, bool MULTI>
__global__ void __launch_bounds__(D) paged_decode_join_kernel(const __grid_constant__ DecodeParams P) {
  __shared__ float wt[PD_MAX_CTAS];
  __shared__ float red[2][D / 32];
  using Sh = PdShape<T, D, NT, MULTI>;
  constexpr int ROWS = Sh::ROWS;
  if (MULTI) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c1 = blockIdx.x, r = blockIdx.y, tid = threadIdx.x;
  const int4 rec = *reinterpret_cast<const int4 *>(P.rec + c1 * 4);
  if (rec.x == 0) return;
  int s0 = 0;
  const int c0 = rec.y, b = rec.z, hh = rec.w, NR = (MULTI ? decode_rows(P, b, s0) : 1) * P.G;
  const int HG = MULTI ? (NR + ROWS - 1) / ROWS : P.HG, kvh = hh / HG, r0 = (hh - kvh * HG) * ROWS;
  if (r >= min(ROWS, NR - r0)) return;
  const int np = c1 - c0 + 1;
  auto row = [&](int i) { return (int64_t)(2 * (c0 + i) + (i == 0 ? 1 : 0)) * P.prows + r; };
  float M = -INFINITY;
  for (int i = tid; i < np; i += D) M = fmaxf(M, P.pml[row(i) * 2]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if ((tid & 31) == 0) red[0][tid >> 5] = M;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < D / 32; ++w) M = fmaxf(M, red[0][w]);
  float L = 0.f;
  for (int i = tid; i < np; i += D) {
    const float2 ml = *reinterpret_cast<const float2 *>(P.pml + row(i) * 2);
    const float w = M == -INFINITY ? 0.f : ex2(ml.x - M);
    wt[i] = w;
    L += w * ml.y;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
  if ((tid & 31) == 0) red[1][tid >> 5] = L;
  __syncthreads();
  L = 0.f;
#pragma unroll
  for (int w = 0; w < D / 32; ++w) L += red[1][w];
  float v = 0.f;
#pragma unroll 8
  for (int i = 0; i < np; ++i) v = fmaf(wt[i], P.po[row(i) * D + tid], v);
  const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
  const int tk = MULTI ? div_by(P.group, r0 + r) : 0;
  const int64_t orow = (int64_t)(MULTI ? s0 + tk : b) * P.Hq + kvh * P.G + r0 + r - tk * P.G;
  if constexpr (Sh::F32) ((float *)P.out)[orow * D + tid] = v * inv;
  else ((__nv_bfloat16 *)P.out)[orow * D + tid] = __float2bfloat16_rn(v * inv);
  if (tid == 0) P.lse[orow] = L == 0.f ? -INFINITY : (M + log2f(L)) * kPgLn2;
}

template <typename T, int D, int NT, bool MULTI = false>
static echo_status_t launch_decode(DecodeParams &P, cudaStream_t st) {
  using Sh = PdShape<T, D, NT, MULTI>;
  constexpr size_t smem = pd_smem<T, D, NT, MULTI>();
  static_assert(Sh::CTAS * (smem + 1024) <= 228 * 1024, "the CTAs of an SM fit its shared memory");
  P.HG = (P.G + Sh::ROWS - 1) / Sh::ROWS;
  P.prows = (int)std::min<int64_t>(MULTI ? (int64_t)P.N * P.G : P.G, Sh::ROWS);
  P.nctas = std::min(sm_count() * Sh::CTAS, MULTI ? PD_MULTI_CTAS : PD_MAX_CTAS);
  // weights are counted in 32 bits: sequences x heads x tiles of the longest one
  const double groups = MULTI ? (double)P.N * P.G / Sh::ROWS + P.B : (double)P.B * P.HG;
  if (groups * P.C.n_kv_heads * ((double)P.C.max_pages * P.C.page_tokens / Sh::TILE + 4) > 2147483647.0)
    return ECHO_ERR_UNSUPPORTED;
  // what the page tables bound by a few tiles is not split, and there is nothing to join
  P.whole = Sh::Q8 && (int64_t)P.C.max_pages * P.C.page_tokens <= PD_WHOLE_TILES * Sh::TILE;
  ECHO_CUDA_OK((allow_smem<paged_decode_kernel<T, D, NT, MULTI>>(smem)));
  CUtensorMap kmap = {}, vmap = {};
  int box = 0;
  if (Sh::Q8) {
    // pages [page][head][row][code], boxes of `box` rows of a warp's tokens (8 or more, the period of the
    // swizzle); the stride of a dimension of one entry is never used: any that is valid will do
    const echo_paged_kv_t &C = P.C;
    box = std::min(C.page_tokens & -C.page_tokens, Sh::TW);
    const int64_t dims[4] = {D, C.page_tokens, C.n_kv_heads, C.n_pages};
    const int64_t sd[3] = {C.page_tokens > 1 ? C.row_stride : D, C.n_kv_heads > 1 ? C.head_stride : D,
                           C.n_pages > 1 ? C.page_stride : D};
    const int bx[4] = {D, box, 1, 1};
    const CUtensorMapSwizzle swz = D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
    if (box < 8 || !pg_map(&kmap, C.k, ECHO_E4M3, 4, dims, sd, bx, swz) || !pg_map(&vmap, C.v, ECHO_E4M3, 4, dims, sd, bx, swz)) box = 0;
  }
  paged_decode_kernel<T, D, NT, MULTI><<<P.nctas, Sh::THREADS, smem, st>>>(P, kmap, vmap, box);
  ECHO_LAUNCH_OK();
  if (P.whole) return ECHO_OK;
  ECHO_CUDA_OK(launch_after(paged_decode_join_kernel<T, D, NT, MULTI>, dim3(P.nctas, P.prows), dim3(D), 0, st, P));
  return ECHO_OK;
}

template <int D>
static echo_status_t launch_decode_d(DecodeParams &P, cudaStream_t st) {
  if (P.C.dtype == ECHO_F32) return launch_decode<float, D, 1>(P, st);
  if (P.C.dtype == ECHO_E4M3) return P.G <= 8 ? launch_decode<E4m3, D, 1>(P, st) : launch_decode<E4m3, D, 2>(P, st);
  return P.G <= 8 ? launch_decode<__nv_bfloat16, D, 1>(P, st) : launch_decode<__nv_bfloat16, D, 2>(P, st);
}

// Partials of a call of few tokens: two a CTA of up to 32 rows, in the many-token call's workspace.
static DecodeParams decode_params(const echo_paged_kv_t *cache, const echo_paged_scales_t *scales, const void *q, int64_t q_stride,
                                  const int32_t *seq_len, int32_t B, int32_t Hq, const echo_attn_scores_t *scores, void *out,
                                  float *lse, void *workspace) {
  DecodeParams P = {};
  P.C = *cache;
  if (scales) P.X = *scales;
  P.page = fast_div(cache->page_tokens);
  P.q = q; P.q_stride = q_stride; P.seq_len = seq_len;
  P.B = B; P.Hq = Hq; P.G = Hq / cache->n_kv_heads;
  P.slopes = scores->slopes; P.window = scores->window;
  P.first_tok = scores->first_tok; P.prefix_len = scores->prefix_len;
  P.f = score_form(scores);
  P.out = out; P.lse = lse;
  P.rec = reinterpret_cast<int32_t *>(workspace);
  P.po = reinterpret_cast<float *>(P.rec + 4 * PD_MAX_CTAS);
  return P;
}

static_assert(4 * PD_MULTI_CTAS <= kPgSomeAt, "the records of a call of few tokens lie ahead of the note");
bool few_tokens_q8(int64_t N, int64_t B, int64_t G, const echo_attn_scores_t *scores) { return !scores->first_tok && N * G <= 32 * B; }

echo_status_t launch_few_tokens_q8(const echo_paged_kv_t *cache, const echo_paged_scales_t *scales, const void *q, int64_t q_stride,
                                   const int32_t *q_start, const int32_t *seq_len, int32_t N, int32_t B, int32_t Hq,
                                   const echo_attn_scores_t *scores_of, int most, void *out, float *lse, void *workspace,
                                   cudaStream_t st) {
  DecodeParams P = decode_params(cache, scales, q, q_stride, seq_len, B, Hq, scores_of, out, lse, workspace);
  P.q_start = q_start;
  P.N = N;
  P.most = most;
  P.some = P.rec + kPgSomeAt;
  P.po = reinterpret_cast<float *>(P.rec + kPgRecords);
  P.group = fast_div(P.G);
  const bool two = (int64_t)N * P.G <= 16 * (int64_t)B;   // rows of a sequence that two tiles of 8 hold on average
  P.pml = P.po + (size_t)2 * PD_MULTI_CTAS * std::min<int64_t>((int64_t)N * P.G, two ? 16 : 32) * cache->head_dim;
  if (cache->head_dim == 128) return two ? launch_decode<E4m3, 128, 2, true>(P, st) : launch_decode<E4m3, 128, 4, true>(P, st);
  return two ? launch_decode<E4m3, 64, 2, true>(P, st) : launch_decode<E4m3, 64, 4, true>(P, st);
}

}  // namespace echo

using namespace echo;

extern "C" size_t echo_paged_decode_workspace_bytes(int32_t Hq, int32_t n_kv_heads, int32_t d) {
  if (Hq <= 0 || n_kv_heads <= 0 || d <= 0 || Hq % n_kv_heads) return 0;
  return (size_t)PD_MAX_CTAS * (2 * std::min(Hq / n_kv_heads, PD_MAX_ROWS) * (d + 2) + 4) * sizeof(float);
}

// scales: of a cache in 8 bits, and else NULL.
static echo_status_t attn_decode(const echo_paged_kv_t *cache, const echo_paged_scales_t *scales, const void *q,
                                 int64_t q_stride, const int32_t *seq_len, int32_t B, int32_t Hq,
                                 const echo_attn_scores_t *scores, void *out, float *lse, void *workspace,
                                 size_t workspace_bytes, cudaStream_t cs) {
  const echo_status_t st = paged_scores_check(scores);
  if (st != ECHO_OK) return st;
  if (!q || !seq_len || !out || !lse || B <= 0 || Hq <= 0) return ECHO_ERR_INVALID_ARG;
  if (Hq % cache->n_kv_heads || Hq / cache->n_kv_heads > 128) return ECHO_ERR_UNSUPPORTED;
  if (!workspace) return ECHO_ERR_INVALID_ARG;
  const int act = paged_act_type(cache->dtype);
  if (!paged_rows_ok(q, q_stride, act) || !paged_rows_ok(out, 0, act) ||
      (reinterpret_cast<uintptr_t>(workspace) & 15))
    return ECHO_ERR_INVALID_ARG;
  if (workspace_bytes < echo_paged_decode_workspace_bytes(Hq, cache->n_kv_heads, cache->head_dim))
    return ECHO_ERR_INVALID_ARG;
  DecodeParams P = decode_params(cache, scales, q, q_stride, seq_len, B, Hq, scores, out, lse, workspace);
  P.pml = P.po + (size_t)2 * PD_MAX_CTAS * std::min(P.G, PD_MAX_ROWS) * cache->head_dim;
  return cache->head_dim == 128 ? launch_decode_d<128>(P, cs) : launch_decode_d<64>(P, cs);
}

extern "C" echo_status_t echo_paged_attn_decode(const echo_paged_kv_t *cache, const void *q, int64_t q_stride,
                                                const int32_t *seq_len, int32_t B, int32_t Hq,
                                                const echo_attn_scores_t *scores, void *out, float *lse,
                                                void *workspace, size_t workspace_bytes, echo_stream_t stream) {
  const echo_status_t st = paged_check(cache);
  if (st != ECHO_OK) return st;
  return attn_decode(cache, nullptr, q, q_stride, seq_len, B, Hq, scores, out, lse, workspace, workspace_bytes,
                     (cudaStream_t)stream);
}

extern "C" echo_status_t echo_paged_attn_decode_q8(const echo_paged_kv_t *cache, const echo_paged_scales_t *scales,
                                                   const void *q, int64_t q_stride, const int32_t *seq_len, int32_t B,
                                                   int32_t Hq, const echo_attn_scores_t *scores_of, void *out,
                                                   float *lse, void *workspace, size_t workspace_bytes,
                                                   echo_stream_t stream) {
  echo_status_t st = paged_check(cache, true);
  if (st == ECHO_OK) st = paged_scales_check(scales);
  if (st != ECHO_OK) return st;
  return attn_decode(cache, scales, q, q_stride, seq_len, B, Hq, scores_of, out, lse, workspace, workspace_bytes,
                     (cudaStream_t)stream);
}
