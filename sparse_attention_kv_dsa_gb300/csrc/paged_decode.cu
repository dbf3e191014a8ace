// Attention of one new token per sequence over a paged key/value cache.
//
//   x_t = scale q . k_t, capped and biased;  out = sum_t e^(x_t) v_t / sum_t e^(x_t);
//   lse = log sum_t e^(x_t)   over the tokens t that the query sees.
//
// Bound: every seen key and value is read once (4 d bytes a token and KV head in bf16)
// for 4 G d operations, G query heads to a KV head: 16 operations a byte at most, so HBM.
//
// Split.  The cache is dealt out in units: 64-token tiles (32 in float32) of one KV head and
// up to 16 of its query heads, ordered by (sequence, KV head, tile).  A persistent grid
// computes from the device's own lengths how many units there are and gives each CTA an equal
// run of them, so that ragged batches, one long sequence and many short ones all spread
// evenly, and one captured graph serves any lengths.  A run may cross sequences; the loads
// run on across the border.  A (sequence, head) whose units lie in one CTA is finished
// there; otherwise each of its CTAs leaves a partial (o, m, l) -- at most two a CTA: the end
// of a run of units begun elsewhere (slot 0), and the start of one finished elsewhere (slot
// 1) -- and a second kernel joins them in order: sums of a fixed order, no atomics.

#include "paged.cuh"

namespace echo {

constexpr int PD_THREADS = 128;
constexpr int PD_ROWS = 16;          // query heads of a unit
constexpr int PD_MAX_CTAS = 608;     // partial slots: two a CTA
constexpr int PD_MIN_UNITS = 2;      // fewest units of a CTA's run
constexpr int PD_RING = 8;           // units whose look-ups are kept

struct DecodeParams {
  echo_paged_kv_t C;
  const void *q;
  int64_t q_stride;
  const int32_t *seq_len;
  int B, Hq, G, HG;                  // query heads of a KV head, groups of 16 of them
  const float *slopes;
  int window;
  const int32_t *first_tok, *prefix_len;
  ScoreForm f;
  void *out;
  float *lse;
  float *po, *pml;                   // partials [2 CTAs][rows][d], [2 CTAs][rows][2]
  int prows;                         // rows of a partial: min(G, 16)
  int nctas;
};

// What sequence b's query sees, as tiles.
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
  return s;
}

// Sum over the block (every thread gets it).
__device__ __forceinline__ long long block_sum(long long v, long long *warp) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) warp[threadIdx.x >> 5] = v;
  __syncthreads();
  long long s = 0;
#pragma unroll
  for (int w = 0; w < PD_THREADS / 32; ++w) s += warp[w];
  __syncthreads();
  return s;
}

// Units of a CTA's run.
__device__ __forceinline__ long long units_per_cta(long long total, int nctas) {
  return max((total + nctas - 1) / nctas, (long long)PD_MIN_UNITS);
}

// A unit of the ring: its tile's rows, and what it is.
struct UnitInfo {
  int b, hh, t0, flags;              // flags: 1 first unit of the run for (b, hh), 2 last, 4 begun elsewhere, 8 goes on elsewhere
  int len;
};

template <typename T, int TILE>
struct PdShared {
  int64_t row[PD_RING][TILE];        // offset of the token's row, -1: not seen
  UnitInfo info[PD_RING];
  long long warp[PD_THREADS / 32];
  int seq;
  long long before;
  float mx[4][PD_ROWS], ls[4][PD_ROWS];
};

template <typename T, int D>
struct PdShape {
  static constexpr int TILE = sizeof(T) == 2 ? 64 : 32;
  static constexpr int STAGES = 3;
  static constexpr int ROWB = D * (int)sizeof(T);       // bytes of a key (or value)
  static constexpr int HALF = TILE * ROWB;              // bytes of a tile's keys
  static constexpr int PBYTES = sizeof(T) == 2 ? PD_ROWS * TILE * 2 : PD_ROWS * TILE * 4;
  static constexpr size_t SMEM = 128 + (size_t)STAGES * 2 * HALF + 2 * PD_ROWS * ROWB + PBYTES + sizeof(PdShared<T, TILE>);
};

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

// Byte offset of 16-byte chunk c of row r in a tile of ROWB-byte rows: chunks are permuted
// within 128 bytes by the row, so that eight rows read at one chunk lie in eight bank groups.
template <int ROWB>
__device__ __forceinline__ uint32_t pd_at(int r, int c) {
  return (uint32_t)(r * ROWB + ((c ^ (r & 7)) << 4));
}

template <typename T>
__device__ __forceinline__ T pd_round(float x) {
  if constexpr (sizeof(T) == 2) return __float2bfloat16_rn(x);
  else return x;
}

template <typename T, int D>
__global__ void __launch_bounds__(PD_THREADS) paged_decode_kernel(const __grid_constant__ DecodeParams P) {
  using Sh = PdShape<T, D>;
  constexpr int TILE = Sh::TILE, ST = Sh::STAGES, ROWB = Sh::ROWB, HALF = Sh::HALF;
  constexpr int KC = ROWB / 16;                          // 16-byte chunks of a key
  constexpr bool BF = sizeof(T) == 2;
  extern __shared__ unsigned char pd_raw[];
  unsigned char *sm = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(pd_raw) + 127) & ~uintptr_t(127));
  unsigned char *qs = sm + ST * 2 * HALF;                // two query tiles (this segment's and the next one's)
  unsigned char *ps = qs + 2 * PD_ROWS * ROWB;           // probabilities of the tile
  PdShared<T, TILE> &S = *reinterpret_cast<PdShared<T, TILE> *>(ps + Sh::PBYTES);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const echo_paged_kv_t &C = P.C;
  const int HH = C.n_kv_heads * P.HG;

  // ---- this CTA's run of units
  long long mine = 0;
  for (int b = tid; b < P.B; b += PD_THREADS) mine += decode_span(P, b, TILE).n();
  const long long total = block_sum(mine, S.warp) * HH;
  const long long per = units_per_cta(total, P.nctas);
  const long long u0 = per * blockIdx.x, u1 = min(total, u0 + per);
  if (u0 >= u1) return;
  // the sequence of unit u0: a scan over the sequences, PD_THREADS at a time
  if (tid == 0) S.seq = -1;
  long long base = 0;
  for (int b0 = 0; b0 < P.B; b0 += PD_THREADS) {
    const int b = b0 + tid;
    long long n = b < P.B ? (long long)decode_span(P, b, TILE).n() * HH : 0;
    long long x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) S.warp[warp] = x;
    __syncthreads();
    long long pre = base;
    for (int w = 0; w < warp; ++w) pre += S.warp[w];
    const long long end = pre + x, start = end - n;
    if (start <= u0 && u0 < end) { S.seq = b; S.before = start; }
    for (int w = 0; w < PD_THREADS / 32; ++w) base += S.warp[w];
    __syncthreads();
    if (S.seq >= 0) break;
  }

  // ---- cursor of the look-ups (the same in every thread)
  int cb = S.seq, chh, ci;
  DecodeSpan cs = decode_span(P, cb, TILE);
  {
    const long long off = u0 - S.before;
    chh = (int)(off / cs.n());
    ci = (int)(off % cs.n());
  }
  const int nu = (int)(u1 - u0);                         // a run is at most 2^31 tokens of one head ... in tiles
  int cu = 0;                                            // units looked up
  // look up unit cu: thread r < TILE finds its token's row
  auto look_up = [&]() {
    if (cu >= nu) return;
    const int e = cu % PD_RING;
    const int t0 = cs.t.tile(ci) * TILE;
    if (tid < TILE) {
      const int t = t0 + tid;
      const bool seen = t >= cs.first && t < cs.len && (t >= cs.lo || t < cs.pre);
      S.row[e][tid] = seen ? paged_row(C, cb, t) : -1;
    }
    if (tid == PD_THREADS - 1) {
      UnitInfo I;
      I.b = cb; I.hh = chh; I.t0 = t0; I.len = cs.len;
      const bool lastu = ci + 1 == cs.n() || cu + 1 == nu;
      I.flags = ((ci == 0 || cu == 0) ? 1 : 0) | (lastu ? 2 : 0) | ((cu < ci) ? 4 : 0) |
                ((lastu && ci + 1 != cs.n()) ? 8 : 0);
      S.info[e] = I;
    }
    ++cu;
    if (++ci == cs.n()) {
      ci = 0;
      if (++chh == HH) {
        chh = 0;
        if (cu < nu) {
          do cs = decode_span(P, ++cb, TILE); while (cs.n() == 0 && cb < P.B - 1);
        }
      }
    }
  };
  // copy unit x's keys and values into its stage
  auto load = [&](int x) {
    if (x < nu) {
      const int e = x % PD_RING;
      const int kvh = S.info[e].hh / P.HG;
      const T *kb = (const T *)C.k + (int64_t)kvh * C.head_stride, *vb = (const T *)C.v + (int64_t)kvh * C.head_stride;
      unsigned char *kt = sm + (x % ST) * 2 * HALF, *vt = kt + HALF;
#pragma unroll 4
      for (int i = tid; i < TILE * KC; i += PD_THREADS) {
        const int r = i / KC, c = i % KC;
        const int64_t g = S.row[e][r];
        const int64_t off = (g >= 0 ? g : 0) + c * (16 / (int)sizeof(T));
        const uint32_t nbytes = g >= 0 ? 16u : 0u;
        cp_async_16(kt + pd_at<ROWB>(r, c), kb + off, nbytes);
        cp_async_16(vt + pd_at<ROWB>(r, c), vb + off, nbytes);
      }
    }
    cp_async_commit();
  };
  for (int i = 0; i < ST; ++i) look_up();
  __syncthreads();
  for (int i = 0; i < ST - 1; ++i) load(i);

  float o[BF ? D / 32 : 4][4];                           // bf16: n-tiles of D/4 values; f32: heads x 4 values
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;      // bf16: rows gid, gid + 8
  float mh[4], lh[4];                                    // f32: this warp's heads
  uint32_t qa[BF ? D / 16 : 1][4];
  const int gid = lane >> 2, tig = lane & 3;
  float sl0 = 0.f, sl1 = 0.f, slh[4] = {0.f, 0.f, 0.f, 0.f};
  int nrows = 0, h0 = 0, nseg = 0;

  for (int x = 0; x < nu; ++x) {
    const int e = x % PD_RING;
    const UnitInfo I = S.info[e];
    if (I.flags & 1) {                                   // a new (sequence, head group)
      const int kvh = I.hh / P.HG, hg = I.hh % P.HG;
      h0 = kvh * P.G + hg * PD_ROWS;
      nrows = min(PD_ROWS, P.G - hg * PD_ROWS);
      unsigned char *qt = qs + (nseg & 1) * PD_ROWS * ROWB;
      ++nseg;
      const T *q = (const T *)P.q + (int64_t)I.b * P.q_stride + (int64_t)h0 * D;
      for (int i = tid; i < PD_ROWS * KC; i += PD_THREADS) {
        const int r = i / KC, c = i % KC;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (r < nrows) v = reinterpret_cast<const uint4 *>(q + (int64_t)r * D)[c];
        *reinterpret_cast<uint4 *>(qt + pd_at<ROWB>(r, c)) = v;
      }
#pragma unroll
      for (int i = 0; i < (BF ? D / 32 : 4); ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
      m0 = m1 = -INFINITY;
      l0 = l1 = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) { mh[i] = -INFINITY; lh[i] = 0.f; }
      if (P.slopes) {
        if constexpr (BF) {
          sl0 = gid < nrows ? P.slopes[h0 + gid] * kPgLog2e : 0.f;
          sl1 = gid + 8 < nrows ? P.slopes[h0 + gid + 8] * kPgLog2e : 0.f;
        } else {
          for (int i = 0; i < 4; ++i) slh[i] = warp + 4 * i < nrows ? P.slopes[h0 + warp + 4 * i] * kPgLog2e : 0.f;
        }
      }
    }
    look_up();                                           // unit x + ST
    cp_async_wait<ST - 2>();
    __syncthreads();                                     // unit x is there; unit x - 1's stage is free
    load(x + ST - 1);
    const unsigned char *kt = sm + (x % ST) * 2 * HALF, *vt = kt + HALF;
    const unsigned char *qt = qs + ((nseg - 1) & 1) * PD_ROWS * ROWB;

    if constexpr (BF) {
      if (I.flags & 1) {
        const int mi = lane >> 3, r = (mi & 1) * 8 + (lane & 7);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) pd_ldsm_x4(smem_u32(qt) + pd_at<ROWB>(r, ks * 2 + (mi >> 1)), qa[ks]);
      }
      // scores of this warp's 16 tokens
      const int rw = warp * 16;
      float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      {
        const int mi = lane >> 3, r = rw + (mi >> 1) * 8 + (lane & 7);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          uint32_t b[4];
          pd_ldsm_x4(smem_u32(kt) + pd_at<ROWB>(r, ks * 2 + (mi & 1)), b);
          pd_mma(s[0], qa[ks], b[0], b[1]);
          pd_mma(s[1], qa[ks], b[2], b[3]);
        }
      }
      float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int r = rw + t * 8 + 2 * tig + y;
          const bool ok = S.row[e][r] >= 0;
          float a = score_log2(P.f, s[t][y]), c = score_log2(P.f, s[t][2 + y]);
          if (P.slopes) {
            const float far = (float)(I.len - 1 - (I.t0 + r));
            a -= sl0 * far;
            c -= sl1 * far;
          }
          s[t][y] = ok ? a : -INFINITY;
          s[t][2 + y] = ok ? c : -INFINITY;
          mx0 = fmaxf(mx0, s[t][y]);
          mx1 = fmaxf(mx1, s[t][2 + y]);
        }
#pragma unroll
      for (int y = 1; y <= 2; y <<= 1) {
        mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, y));
        mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, y));
      }
      if (tig == 0) {
        S.mx[warp][gid] = mx0;
        S.mx[warp][gid + 8] = mx1;
      }
      __syncthreads();
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        mx0 = fmaxf(mx0, S.mx[w][gid]);
        mx1 = fmaxf(mx1, S.mx[w][gid + 8]);
      }
      const float n0 = fmaxf(m0, mx0), n1 = fmaxf(m1, mx1);
      const float z0 = n0 == -INFINITY ? 0.f : n0, z1 = n1 == -INFINITY ? 0.f : n1;
      const float c0 = exp2f(m0 - z0), c1 = exp2f(m1 - z1);
      m0 = n0;
      m1 = n1;
      // probabilities in bf16 (half a step, 2^-9 of each; the sums take the unrounded ones)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const float p0 = exp2f(s[t][0] - z0), p1 = exp2f(s[t][1] - z0), p2 = exp2f(s[t][2] - z1), p3 = exp2f(s[t][3] - z1);
        if (t == 0) { l0 *= c0; l1 *= c1; }
        l0 += p0 + p1;
        l1 += p2 + p3;
        const int ch = (rw + t * 8) / 8;
        const __nv_bfloat162 a = __floats2bfloat162_rn(p0, p1), c = __floats2bfloat162_rn(p2, p3);
        *reinterpret_cast<__nv_bfloat162 *>(ps + pd_at<TILE * 2>(gid, ch) + 4 * tig) = a;
        *reinterpret_cast<__nv_bfloat162 *>(ps + pd_at<TILE * 2>(gid + 8, ch) + 4 * tig) = c;
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        o[i][0] *= c0;
        o[i][1] *= c0;
        o[i][2] *= c1;
        o[i][3] *= c1;
      }
      // o[:, this warp's D/4 values] += P (16 x 64) V
      {
        const int mi = lane >> 3;
#pragma unroll
        for (int ks = 0; ks < TILE / 16; ++ks) {
          uint32_t a[4];
          pd_ldsm_x4(smem_u32(ps) + pd_at<TILE * 2>((mi & 1) * 8 + (lane & 7), ks * 2 + (mi >> 1)), a);
          const int r = ks * 16 + (mi & 1) * 8 + (lane & 7);
#pragma unroll
          for (int j = 0; j < D / 64; ++j) {
            uint32_t b[4];
            pd_ldsm_x4_t(smem_u32(vt) + pd_at<ROWB>(r, warp * (D / 32) + j * 2 + (mi >> 1)), b);
            pd_mma(o[2 * j], a, b[0], b[1]);
            pd_mma(o[2 * j + 1], a, b[2], b[3]);
          }
        }
      }
      if (I.flags & 2) {                                 // the run's last unit of this (sequence, head group)
        float s0 = l0, s1 = l1;
#pragma unroll
        for (int y = 1; y <= 2; y <<= 1) {
          s0 += __shfl_xor_sync(0xffffffffu, s0, y);
          s1 += __shfl_xor_sync(0xffffffffu, s1, y);
        }
        if (tig == 0) {
          S.ls[warp][gid] = s0;
          S.ls[warp][gid + 8] = s1;
        }
        __syncthreads();
        const float L0 = S.ls[0][gid] + S.ls[1][gid] + S.ls[2][gid] + S.ls[3][gid];
        const float L1 = S.ls[0][gid + 8] + S.ls[1][gid + 8] + S.ls[2][gid + 8] + S.ls[3][gid + 8];
        const bool whole = !(I.flags & 12);
        const int slot = 2 * blockIdx.x + ((I.flags & 4) ? 0 : 1);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int r = gid + 8 * half;
          if (r >= nrows) continue;
          const float L = half ? L1 : L0, M = half ? m1 : m0;
          if (whole) {
            const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
            T *dst = (T *)P.out + ((int64_t)I.b * P.Hq + h0 + r) * D + warp * (D / 4) + 2 * tig;
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
              *reinterpret_cast<__nv_bfloat162 *>(dst + 8 * i) =
                  __floats2bfloat162_rn(o[i][2 * half] * inv, o[i][2 * half + 1] * inv);
            if (warp == 0 && tig == 0)
              P.lse[(int64_t)I.b * P.Hq + h0 + r] = L == 0.f ? -INFINITY : (M + log2f(L)) * kPgLn2;
          } else {
            float *dst = P.po + ((int64_t)slot * P.prows + r) * D + warp * (D / 4) + 2 * tig;
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
              *reinterpret_cast<float2 *>(dst + 8 * i) = make_float2(o[i][2 * half], o[i][2 * half + 1]);
            if (warp == 0 && tig == 0)
              *reinterpret_cast<float2 *>(P.pml + ((int64_t)slot * P.prows + r) * 2) = make_float2(M, L);
          }
        }
      }
    } else {
      // float32: warp w takes heads w, w + 4, ...; lane = token for the scores, then lane = a
      // 16-byte chunk of the values (D = 64: two lanes' halves of the tokens for each chunk)
      const float *pt = reinterpret_cast<const float *>(ps);
      const bool ok = S.row[e][lane] >= 0;
      float s[4] = {0.f, 0.f, 0.f, 0.f};
      const int nh = (nrows - warp + 3) / 4;             // heads of this warp
      if (nh > 0) {
        for (int c = 0; c < KC; ++c) {
          const float4 kv = *reinterpret_cast<const float4 *>(kt + pd_at<ROWB>(lane, c));
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (i < nh) {
              const int r = warp + 4 * i;
              const float4 qv = *reinterpret_cast<const float4 *>(qt + pd_at<ROWB>(r, c));
              s[i] = fmaf(qv.x, kv.x, fmaf(qv.y, kv.y, fmaf(qv.z, kv.z, fmaf(qv.w, kv.w, s[i]))));
            }
        }
        const float far = (float)(I.len - 1 - (I.t0 + lane));
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i < nh) {
            float a = score_log2(P.f, s[i]);
            if (P.slopes) a -= slh[i] * far;
            a = ok ? a : -INFINITY;
            float mx = a;
#pragma unroll
            for (int y = 16; y > 0; y >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, y));
            const float nm = fmaxf(mh[i], mx), z = nm == -INFINITY ? 0.f : nm;
            const float c = exp2f(mh[i] - z), p = exp2f(a - z);
            mh[i] = nm;
            lh[i] = lh[i] * c + p;
            reinterpret_cast<float *>(ps)[(warp + 4 * i) * TILE + lane] = p;
#pragma unroll
            for (int j = 0; j < 4; ++j) o[i][j] *= c;
          }
        __syncwarp();
        constexpr int LPT = 32 / KC;                     // lanes of a chunk: 1 (D = 128) or 2
        const int c = lane % KC, part = lane / KC;
        for (int r = part; r < TILE; r += LPT) {
          const float4 vv = *reinterpret_cast<const float4 *>(vt + pd_at<ROWB>(r, c));
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (i < nh) {
              const float p = pt[(warp + 4 * i) * TILE + r];
              o[i][0] = fmaf(p, vv.x, o[i][0]);
              o[i][1] = fmaf(p, vv.y, o[i][1]);
              o[i][2] = fmaf(p, vv.z, o[i][2]);
              o[i][3] = fmaf(p, vv.w, o[i][3]);
            }
        }
        if (I.flags & 2) {
          const bool whole = !(I.flags & 12);
          const int slot = 2 * blockIdx.x + ((I.flags & 4) ? 0 : 1);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (i < nh) {
              float L = lh[i];
#pragma unroll
              for (int y = 16; y > 0; y >>= 1) L += __shfl_xor_sync(0xffffffffu, L, y);
              float4 v = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
              if (LPT == 2) {
                v.x += __shfl_xor_sync(0xffffffffu, v.x, 16);
                v.y += __shfl_xor_sync(0xffffffffu, v.y, 16);
                v.z += __shfl_xor_sync(0xffffffffu, v.z, 16);
                v.w += __shfl_xor_sync(0xffffffffu, v.w, 16);
              }
              const int r = warp + 4 * i;
              if (whole) {
                const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
                if (part == 0)
                  *reinterpret_cast<float4 *>((float *)P.out + ((int64_t)I.b * P.Hq + h0 + r) * D + 4 * c) =
                      make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
                if (lane == 0)
                  P.lse[(int64_t)I.b * P.Hq + h0 + r] = L == 0.f ? -INFINITY : (mh[i] + log2f(L)) * kPgLn2;
              } else {
                if (part == 0) *reinterpret_cast<float4 *>(P.po + ((int64_t)slot * P.prows + r) * D + 4 * c) = v;
                if (lane == 0)
                  *reinterpret_cast<float2 *>(P.pml + ((int64_t)slot * P.prows + r) * 2) = make_float2(mh[i], L);
              }
            }
        }
      }
    }
  }
  cp_async_wait_all();
}

// Joins the partials of one (sequence, head group) in the order of their units, and gives a
// sequence that sees nothing its empty rows.  One CTA each; a warp takes every fourth row.
template <typename T, int D>
__global__ void __launch_bounds__(PD_THREADS) paged_decode_join_kernel(const __grid_constant__ DecodeParams P) {
  constexpr int TILE = PdShape<T, D>::TILE, VL = D / 32;
  __shared__ long long warp_sum[PD_THREADS / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int HH = P.C.n_kv_heads * P.HG, b = blockIdx.x / HH, hh = blockIdx.x % HH;
  long long all = 0, before = 0;
  int n = 0;
  for (int i = tid; i < P.B; i += PD_THREADS) {
    const int k = decode_span(P, i, TILE).n();
    all += k;
    if (i < b) before += k;
  }
  n = decode_span(P, b, TILE).n();
  const long long per = units_per_cta(block_sum(all, warp_sum) * HH, P.nctas);
  const long long s0 = block_sum(before, warp_sum) * HH + (long long)hh * n, s1 = s0 + n;
  const int hg = hh % P.HG, h0 = (hh / P.HG) * P.G + hg * PD_ROWS, nrows = min(PD_ROWS, P.G - hg * PD_ROWS);
  const long long c0 = n ? s0 / per : 0, c1 = n ? (s1 - 1) / per : 0;
  if (n && c0 == c1) return;                             // finished by its CTA
  for (int r = warp; r < nrows; r += PD_THREADS / 32) {
    float M = -INFINITY, L = 0.f, v[VL];
#pragma unroll
    for (int i = 0; i < VL; ++i) v[i] = 0.f;
    if (n) {
      for (long long c = c0; c <= c1; ++c) {
        const int64_t row = (2 * c + (c == c0 ? 1 : 0)) * P.prows + r;
        const float m = P.pml[row * 2], l = P.pml[row * 2 + 1];
        const float nm = fmaxf(M, m), z = nm == -INFINITY ? 0.f : nm;
        const float wa = exp2f(M - z), wb = exp2f(m - z);
        M = nm;
        L = L * wa + l * wb;
        const float *o = P.po + row * D + lane * VL;
#pragma unroll
        for (int i = 0; i < VL; ++i) v[i] = v[i] * wa + o[i] * wb;
      }
    }
    const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
    T *dst = (T *)P.out + ((int64_t)b * P.Hq + h0 + r) * D + lane * VL;
#pragma unroll
    for (int i = 0; i < VL; ++i) dst[i] = pd_round<T>(v[i] * inv);
    if (lane == 0) P.lse[(int64_t)b * P.Hq + h0 + r] = L == 0.f ? -INFINITY : (M + log2f(L)) * kPgLn2;
  }
}

template <typename T, int D>
static echo_status_t launch_decode(DecodeParams &P, cudaStream_t st) {
  using Sh = PdShape<T, D>;
  static_assert(Sh::SMEM <= 227 * 1024, "fits an SM");
  constexpr int occ = (int)std::min<size_t>(4, 227 * 1024 / (Sh::SMEM + 1024));
  P.nctas = std::min(sm_count() * occ, PD_MAX_CTAS);
  ECHO_CUDA_OK(cudaFuncSetAttribute(paged_decode_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Sh::SMEM));
  paged_decode_kernel<T, D><<<P.nctas, PD_THREADS, Sh::SMEM, st>>>(P);
  ECHO_LAUNCH_OK();
  paged_decode_join_kernel<T, D><<<P.B * P.C.n_kv_heads * P.HG, PD_THREADS, 0, st>>>(P);
  ECHO_LAUNCH_OK();
  return ECHO_OK;
}

}  // namespace echo

using namespace echo;

extern "C" size_t echo_paged_decode_workspace_bytes(int32_t Hq, int32_t n_kv_heads, int32_t d) {
  if (Hq <= 0 || n_kv_heads <= 0 || d <= 0 || Hq % n_kv_heads) return 0;
  return (size_t)2 * PD_MAX_CTAS * std::min(Hq / n_kv_heads, PD_ROWS) * (d + 2) * sizeof(float);
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
  P.q = q; P.q_stride = q_stride; P.seq_len = seq_len;
  P.B = B; P.Hq = Hq; P.G = Hq / cache->n_kv_heads; P.HG = (P.G + PD_ROWS - 1) / PD_ROWS;
  if ((int64_t)B * cache->n_kv_heads * P.HG > 0x7fffffff) return ECHO_ERR_UNSUPPORTED;
  P.slopes = scores->slopes; P.window = scores->window;
  P.first_tok = scores->first_tok; P.prefix_len = scores->prefix_len;
  P.f = score_form(scores);
  P.out = out; P.lse = lse;
  P.prows = std::min(P.G, PD_ROWS);
  P.po = reinterpret_cast<float *>(workspace);
  P.pml = P.po + (size_t)2 * PD_MAX_CTAS * P.prows * cache->head_dim;
  cudaStream_t cs = (cudaStream_t)stream;
  if (cache->dtype == ECHO_BF16)
    return cache->head_dim == 128 ? launch_decode<__nv_bfloat16, 128>(P, cs) : launch_decode<__nv_bfloat16, 64>(P, cs);
  return cache->head_dim == 128 ? launch_decode<float, 128>(P, cs) : launch_decode<float, 64>(P, cs);
}
