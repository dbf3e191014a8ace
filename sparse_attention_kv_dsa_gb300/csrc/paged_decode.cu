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

#include "paged.cuh"

namespace echo {

constexpr int PD_THREADS = 128, PD_WARPS = 4;
constexpr int PD_MAX_ROWS = 16;
constexpr int PD_MAX_CTAS = 608;     // partial slots: two a CTA
constexpr int PD_MIN_WEIGHT = 3;     // least weight of a CTA's run
constexpr int PD_RING = 8;           // units whose look-ups are kept

struct DecodeParams {
  echo_paged_kv_t C;
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
};

template <typename T, int D>
struct PdShape {
  static constexpr bool BF = sizeof(T) == 2;
  static constexpr int ROWS = BF ? 16 : 8;              // query heads of a unit
  static constexpr int TW = BF ? (D == 128 ? 16 : 32) : 8;   // tokens of a warp: 8 KB of keys and values
                                                        // (f32, d = 64: 4 KB)
  static constexpr int TILE = PD_WARPS * TW;
  static constexpr int ROWB = D * (int)sizeof(T);       // bytes of a key (or value)
  static constexpr int HALF = TW * ROWB;                // a warp's keys of a tile
  // Stages of a warp's ring and CTAs an SM.  bf16 rows of 128 values stream best from two CTAs of
  // three stages (16 x 32K-48K tokens: 396 us, two stages 401); d = 64 and float32 have more
  // instructions a byte and want the warps of a third CTA (b96 capped 103 us, two CTAs 112; float32
  // 39 us, two CTAs 43).
  static constexpr int STAGES = BF && D == 128 ? 3 : 2;
  static constexpr int CTAS = BF && D == 128 ? 2 : 3;
};

// What sequence b's query sees, as tiles; a sequence that sees nothing has one tile of
// nothing, which writes its empty rows.
struct DecodeSpan {
  int len, first, pre, lo;
  TileSpan t;
  __device__ __forceinline__ int n() const { return t.nA + t.nB; }
};
__device__ __forceinline__ DecodeSpan decode_span(const DecodeParams &P, int b, int tile) {
  DecodeSpan s;
  s.len = paged_len(P.C, P.seq_len, b);
  s.first = P.first_tok ? max(P.first_tok[b], 0) : 0;
  s.pre = P.prefix_len ? min(P.prefix_len[b], s.len) : 0;
  s.lo = P.window ? max(s.first, s.len - P.window) : s.first;
  s.t = tile_span(s.first, s.pre, s.lo, s.len, tile);
  if (s.n() == 0) s.t.nA = 1;
  return s;
}

// A unit of a warp's ring.
struct UnitInfo {
  int b, hh, t0, len;                // t0: the warp's first token
  int c0;                            // CTA of (b, hh)'s first unit
  int flags;                         // 1 the run's first unit of (b, hh), 2 its last, 4 begun elsewhere, 8 goes on elsewhere
  uint32_t there;                    // tokens that are seen and there
};

template <typename T, int D>
struct PdShared {
  using Sh = PdShape<T, D>;
  UnitInfo info[PD_WARPS][PD_RING];
  uint32_t sum[PD_WARPS], before;    // before: weight before sequence seq
  int seq;
  float m[PD_WARPS][PD_MAX_ROWS], l[PD_WARPS][PD_MAX_ROWS];
  alignas(16) float p[Sh::BF ? 1 : PD_WARPS][8][8];               // f32: weights [head][token]
};

template <typename T, int D>
constexpr size_t pd_smem() {
  using Sh = PdShape<T, D>;
  return 128 + (size_t)PD_WARPS * Sh::STAGES * 2 * Sh::HALF + Sh::ROWS * Sh::ROWB + (Sh::BF ? Sh::ROWS * D * 4 : 0) +
         sizeof(PdShared<T, D>);
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
__device__ __forceinline__ uint32_t pd_pack(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}

// Byte offset of 16-byte chunk c of row r in a tile of ROWB-byte rows: chunks are permuted
// within 128 bytes by the row, so that eight rows read at one chunk lie in eight bank groups.
template <int ROWB>
__device__ __forceinline__ uint32_t pd_at(int r, int c) {
  return (uint32_t)(r * ROWB + ((c ^ (r & 7)) << 4));
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
                                       const unsigned char *vt, const unsigned char *, float (*)[8], int, int lane) {
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
                                       const unsigned char *vt, const unsigned char *qt, float (*pw)[8], int nrows, int lane) {
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

template <typename T, int D, bool R8>
__global__ void __launch_bounds__(PD_THREADS, PdShape<T, D>::CTAS) paged_decode_kernel(const __grid_constant__ DecodeParams P) {
  using Sh = PdShape<T, D>;
  using State = std::conditional_t<Sh::BF, WarpBf<D, R8>, WarpF32<D>>;
  constexpr int TILE = Sh::TILE, TW = Sh::TW, ST = Sh::STAGES, ROWB = Sh::ROWB, HALF = Sh::HALF, ROWS = Sh::ROWS;
  constexpr int KC = ROWB / 16;                          // 16-byte chunks of a key
  extern __shared__ unsigned char pd_raw[];
  unsigned char *sm = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(pd_raw) + 127) & ~uintptr_t(127));
  unsigned char *qs = sm + PD_WARPS * ST * 2 * HALF;     // the query tile
  float *acc = reinterpret_cast<float *>(qs + (Sh::BF ? ROWS * ROWB : 0));                // the warps' results, joined
  PdShared<T, D> &S = *reinterpret_cast<PdShared<T, D> *>(qs + ROWS * ROWB + (Sh::BF ? ROWS * D * 4 : 0));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const echo_paged_kv_t &C = P.C;
  const int HH = C.n_kv_heads * P.HG;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- this CTA's run: a scan over the sequences, PD_THREADS at a time; with few sequences one
  // scan gives the total and finds the place.  Whether it is found is known from the barrier behind
  // the writes of S.seq and S.before, the same in every thread: nobody reads either ahead of it
  uint32_t total = 0, end = 0, n = 0, per = 0, u0 = 0, u1 = 0;
  bool found = false;
  if (tid == 0) P.rec[blockIdx.x * 4] = 0;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    uint32_t at = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < P.B && !found; b0 += PD_THREADS) {
      if (pass == 0 || P.B > PD_THREADS) {
        n = b0 + tid < P.B ? (uint32_t)(decode_span(P, b0 + tid, TILE).n() + 1) * (uint32_t)HH : 0;
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
      total = at;
      per = max((total + P.nctas - 1) / P.nctas, (uint32_t)PD_MIN_WEIGHT);
      u0 = per * blockIdx.x;
      u1 = min(total, u0 + per);
      if (u0 >= total) return;
    }
  }
  if (!found) return;                                    // (lengths that another stream changes between the passes)

  // ---- cursor of the look-ups (the same in every thread): tile ci of its part [i0, ce) of the
  // current (sequence, head group), which begins at weight ws
  int cb = S.seq;
  DecodeSpan cs = decode_span(P, cb, TILE);
  int cn = cs.n(), chh = (int)((u0 - S.before) / (uint32_t)(cn + 1)), ci, i0, ce;
  uint32_t ws = S.before + (uint32_t)chh * (uint32_t)(cn + 1);
  i0 = ci = max(0, (int)(u0 - ws) - 1);
  ce = min(cn, (int)(u1 - ws) - 1);
  int cu = 0;                                            // units looked up
  int32_t ent = -1;                                      // the last one's page-table entry of this lane's token
  int tok = -1;
  UnitInfo *ring = S.info[warp];
  auto look_up = [&]() {
    tok = -1;
    if (ci >= ce) return;                                // the run is over
    const int t0 = cs.t.tile(ci) * TILE + warp * TW;
    const int t = t0 + lane;
    if (lane < TW && t >= cs.first && t < cs.len && (t >= cs.lo || t < cs.pre)) {
      tok = t;
      ent = __ldg(C.page_table + (int64_t)cb * C.max_pages + div_by(P.page, t));
    }
    if (lane == 0) {
      UnitInfo &I = ring[cu % PD_RING];
      I.b = cb; I.hh = chh; I.t0 = t0; I.len = cs.len;
      I.flags = (ci == i0 ? 1 : 0) | (ci + 1 == ce ? 2 : 0) | (i0 > 0 ? 4 : 0) | (ce < cn ? 8 : 0);
      I.c0 = (int)((ws + 1) / per);
    }
    ++cu;
    if (++ci == ce && ce == cn) {                        // on to the next (sequence, head group)
      ws += cn + 1;
      if (++chh == HH) {
        chh = 0;
        if (cb + 1 < P.B) {
          cs = decode_span(P, ++cb, TILE);
          cn = cs.n();
        } else {
          ws = u1;
        }
      }
      i0 = ci = 0;
      ce = min(cn, (int)(u1 - ws) - 1);
    }
  };
  // turns unit x's entries into offsets and copies the warp's keys and values into its stage
  unsigned char *stages = sm + warp * ST * 2 * HALF;
  auto load = [&](int x) {
    if (x < cu) {
      int64_t row = -1;
      if (tok >= 0) {
        if (ent < 0 || ent >= C.n_pages) paged_fail(C.status, ECHO_ERR_PAGE);
        else row = (int64_t)ent * C.page_stride + (int64_t)(tok - div_by(P.page, tok) * C.page_tokens) * C.row_stride;
      }
      const uint32_t there = __ballot_sync(0xffffffffu, row >= 0);
      UnitInfo &I = ring[x % PD_RING];
      if (lane == 0) I.there = there;
      __syncwarp();
      const int64_t head = (int64_t)(I.hh / P.HG) * C.head_stride;
      const T *kb = (const T *)C.k + head, *vb = (const T *)C.v + head;
      unsigned char *kt = stages + (x % ST) * 2 * HALF, *vt = kt + HALF;
#pragma unroll
      for (int i = 0; i < TW * KC / 32; ++i) {
        const int r = (i * 32 + lane) / KC, c = (i * 32 + lane) % KC;
        const int64_t g = __shfl_sync(0xffffffffu, row, r);
        const int64_t off = (g >= 0 ? g : 0) + c * (16 / (int)sizeof(T));
        const uint32_t nbytes = g >= 0 ? 16u : 0u;
        cp_async_16(kt + pd_at<ROWB>(r, c), kb + off, nbytes);
        cp_async_16(vt + pd_at<ROWB>(r, c), vb + off, nbytes);
      }
    }
    cp_async_commit();
  };
  for (int i = 0; i < ST - 1; ++i) {
    look_up();
    load(i);
  }
  look_up();

  State A;
  int nrows = 0, h0 = 0;
  for (int x = 0; x < cu; ++x) {                         // (the look-ups are ahead of it, or over)
    cp_async_wait<ST - 2>();
    __syncwarp();                                        // unit x is there, and unit x - 1's stage is free
    load(x + ST - 1);
    look_up();                                           // unit x + ST
    const UnitInfo &I = ring[x % PD_RING];
    if (I.flags & 1) {                                   // a new (sequence, head group): every warp is past the last one
      const int hg = I.hh % P.HG;
      h0 = (I.hh / P.HG) * P.G + hg * ROWS;
      nrows = min(ROWS, P.G - hg * ROWS);
      if (!Sh::BF) __syncthreads();                      // float32's joined results lie in the query tile's place
      const T *q = (const T *)P.q + (int64_t)I.b * P.q_stride + (int64_t)h0 * D;
      for (int i = tid; i < ROWS * KC; i += PD_THREADS) {
        const int r = i / KC, c = i % KC;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (r < nrows) v = reinterpret_cast<const uint4 *>(q + (int64_t)r * D)[c];
        *reinterpret_cast<uint4 *>(qs + (Sh::BF ? pd_at<ROWB>(r, c) : r * ROWB + c * 16)) = v;
      }
      __syncthreads();
      A.begin(P, qs, h0, nrows, lane);
    }
    const unsigned char *kt = stages + (x % ST) * 2 * HALF;
    A.tile(P, I, kt, kt + HALF, qs, S.p[Sh::BF ? 0 : warp], nrows, lane);
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
      for (int w = 0; w < PD_WARPS; ++w) {
        __syncthreads();
        if (warp == w) A.add_to(acc, M, w == 0, nrows, lane);
      }
      __syncthreads();
      const bool whole = !(I.flags & 12);
      const int64_t slot = 2 * blockIdx.x + ((I.flags & 4) ? 0 : 1);
      for (int i = tid; i < nrows * (D / 4); i += PD_THREADS) {
        const int r = i / (D / 4), c = i % (D / 4);
        float4 v = *reinterpret_cast<const float4 *>(acc + r * D + 4 * c);
        if (whole) {
          const float L = S.l[0][r], inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
          v.x *= inv; v.y *= inv; v.z *= inv; v.w *= inv;
          T *dst = (T *)P.out + ((int64_t)I.b * P.Hq + h0 + r) * D + 4 * c;
          if constexpr (Sh::BF) *reinterpret_cast<uint2 *>(dst) = make_uint2(pd_pack(v.x, v.y), pd_pack(v.z, v.w));
          else *reinterpret_cast<float4 *>(dst) = v;
        } else {
          *reinterpret_cast<float4 *>(P.po + (slot * P.prows + r) * D + 4 * c) = v;
        }
      }
      if (tid < nrows) {
        const float mm = S.m[0][tid], L = S.l[0][tid];
        if (whole) P.lse[(int64_t)I.b * P.Hq + h0 + tid] = L == 0.f ? -INFINITY : (mm + log2f(L)) * kPgLn2;
        else *reinterpret_cast<float2 *>(P.pml + (slot * P.prows + tid) * 2) = make_float2(mm, L);
      }
      if (tid == 0 && (I.flags & 12) == 4) {             // a split one ends here: to be joined
        int32_t *rec = P.rec + blockIdx.x * 4;
        rec[1] = I.c0;
        rec[2] = I.b;
        rec[3] = I.hh;
        rec[0] = 1;
      }
    }
  }
  cp_async_wait_all();
}

// Joins the partials of the (sequence, head group) that ends in CTA blockIdx.x: slot 1 of its
// first CTA, then slot 0 of the following ones.  A block takes one row, a thread one value; the
// maxima first, then the weighted sums in the order of the CTAs.
template <typename T, int D>
__global__ void __launch_bounds__(D) paged_decode_join_kernel(const __grid_constant__ DecodeParams P) {
  __shared__ float wt[PD_MAX_CTAS];
  __shared__ float red[2][D / 32];
  constexpr int ROWS = PdShape<T, D>::ROWS;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c1 = blockIdx.x, r = blockIdx.y, tid = threadIdx.x;
  const int4 rec = *reinterpret_cast<const int4 *>(P.rec + c1 * 4);
  if (rec.x == 0) return;
  const int c0 = rec.y, b = rec.z, hh = rec.w, hg = hh % P.HG;
  if (r >= min(ROWS, P.G - hg * ROWS)) return;
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
  const int64_t orow = (int64_t)b * P.Hq + (hh / P.HG) * P.G + hg * ROWS + r;
  if constexpr (sizeof(T) == 2) ((T *)P.out)[orow * D + tid] = __float2bfloat16_rn(v * inv);
  else ((T *)P.out)[orow * D + tid] = v * inv;
  if (tid == 0) P.lse[orow] = L == 0.f ? -INFINITY : (M + log2f(L)) * kPgLn2;
}

template <typename T, int D, bool R8>
static echo_status_t launch_decode(DecodeParams &P, cudaStream_t st) {
  using Sh = PdShape<T, D>;
  constexpr size_t smem = pd_smem<T, D>();
  static_assert(Sh::CTAS * (smem + 1024) <= 228 * 1024, "the CTAs of an SM fit its shared memory");
  P.HG = (P.G + Sh::ROWS - 1) / Sh::ROWS;
  P.prows = std::min(P.G, Sh::ROWS);
  P.nctas = std::min(sm_count() * Sh::CTAS, PD_MAX_CTAS);
  // weights are counted in 32 bits: sequences x heads x tiles of the longest one
  if ((double)P.B * P.C.n_kv_heads * P.HG * ((double)P.C.max_pages * P.C.page_tokens / Sh::TILE + 4) > 2147483647.0)
    return ECHO_ERR_UNSUPPORTED;
  ECHO_CUDA_OK((allow_smem<paged_decode_kernel<T, D, R8>>(smem)));
  paged_decode_kernel<T, D, R8><<<P.nctas, PD_THREADS, smem, st>>>(P);
  ECHO_LAUNCH_OK();
  ECHO_CUDA_OK(launch_after(paged_decode_join_kernel<T, D>, dim3(P.nctas, P.prows), dim3(D), st, P));
  return ECHO_OK;
}

template <int D>
static echo_status_t launch_decode_d(DecodeParams &P, cudaStream_t st) {
  if (P.C.dtype == ECHO_F32) return launch_decode<float, D, true>(P, st);
  return P.G <= 8 ? launch_decode<__nv_bfloat16, D, true>(P, st) : launch_decode<__nv_bfloat16, D, false>(P, st);
}

}  // namespace echo

using namespace echo;

extern "C" size_t echo_paged_decode_workspace_bytes(int32_t Hq, int32_t n_kv_heads, int32_t d) {
  if (Hq <= 0 || n_kv_heads <= 0 || d <= 0 || Hq % n_kv_heads) return 0;
  return (size_t)PD_MAX_CTAS * (2 * std::min(Hq / n_kv_heads, PD_MAX_ROWS) * (d + 2) + 4) * sizeof(float);
}

extern "C" echo_status_t echo_paged_attn_decode(const echo_paged_kv_t *cache, const void *q, int64_t q_stride,
                                                const int32_t *seq_len, int32_t B, int32_t Hq,
                                                const echo_attn_scores_t *scores, void *out, float *lse,
                                                void *workspace, size_t workspace_bytes, echo_stream_t stream) {
  echo_status_t st = paged_check(cache);
  if (st == ECHO_OK) st = paged_scores_check(scores);
  if (st != ECHO_OK) return st;
  if (!q || !seq_len || !out || !lse || B <= 0 || Hq <= 0) return ECHO_ERR_INVALID_ARG;
  if (Hq % cache->n_kv_heads || Hq / cache->n_kv_heads > 128) return ECHO_ERR_UNSUPPORTED;
  if (!workspace) return ECHO_ERR_INVALID_ARG;
  if (!paged_rows_ok(q, q_stride, cache->dtype) || !paged_rows_ok(out, 0, cache->dtype) ||
      (reinterpret_cast<uintptr_t>(workspace) & 15))
    return ECHO_ERR_INVALID_ARG;
  if (workspace_bytes < echo_paged_decode_workspace_bytes(Hq, cache->n_kv_heads, cache->head_dim))
    return ECHO_ERR_INVALID_ARG;
  DecodeParams P;
  P.C = *cache;
  P.page = fast_div(cache->page_tokens);
  P.q = q; P.q_stride = q_stride; P.seq_len = seq_len;
  P.B = B; P.Hq = Hq; P.G = Hq / cache->n_kv_heads;
  P.slopes = scores->slopes; P.window = scores->window;
  P.first_tok = scores->first_tok; P.prefix_len = scores->prefix_len;
  P.f = score_form(scores);
  P.out = out; P.lse = lse;
  P.rec = reinterpret_cast<int32_t *>(workspace);
  P.po = reinterpret_cast<float *>(P.rec + 4 * PD_MAX_CTAS);
  P.pml = P.po + (size_t)2 * PD_MAX_CTAS * std::min(P.G, PD_MAX_ROWS) * cache->head_dim;
  cudaStream_t cs = (cudaStream_t)stream;
  return cache->head_dim == 128 ? launch_decode_d<128>(P, cs) : launch_decode_d<64>(P, cs);
}
