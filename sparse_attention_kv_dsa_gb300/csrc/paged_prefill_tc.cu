// Tensor-core form (bf16) of the many-token attention over a paged key/value cache.
//
// Bound: 4 d operations for each pair of query head and seen token on the tensor cores, and
// one power (with a cap: a tanh too) on the special-function units.
//
// A persistent CTA per SM.  The work is dealt out in units -- one 128-token tile of the cache
// for one row tile of 256 packed rows (token r / G, head r % G of the KV head's group) --
// ordered by (sequence, row tile, KV head, tile); every CTA takes a run of them of equal
// weight (a row tile begins with PF_ITEM_WEIGHT units' worth: its queries, its epilogue),
// found from the device's own lengths and masks, so that ragged prompts, the triangle of a causal
// mask and a few rows over a long cache all spread evenly.  A row tile whose units lie in
// several CTAs leaves partials (two slots a CTA) that a second kernel joins in order.
//
// Inside a CTA the 256 rows are two M = 128 tiles that share keys and values:
//   S_i = Q_i K^T  (tcgen05, K-major operands in 128-byte-swizzled shared memory)
//   P_i = 2^(x - m) by four warps, one row a thread, bf16 back into TMEM over S_i
//   O_i += P_i V   (A from TMEM, V as stored: MN-major)
// in the order PV_0(j) QK_0(j+1) PV_1(j) QK_1(j+1): the tensor cores work on one tile while
// the other's softmax runs.  A row tile of 128 rows at most (a few drafted tokens over a long
// cache) has no second tile to alternate with: its two halves of TMEM and of the softmax warps
// then take its tiles of the cache in turn, each with its own O, m and l, joined at the end.
// The running maximum m of a row is only moved when a tile's
// maximum passes it by 2^8 (the weights stay below 256, exact in the float32 sums), so O is
// rescaled in TMEM a few times in a long row and not with every tile.
// TMEM columns: S_0 0-127, S_1 128-255 (P_i in the first 64 of S_i), O_0 256.., O_1 384...
// Warps 0-3 and 4-7: softmax and epilogue of tile 0 and 1 (192 registers: a row's 128 scores
// stay in registers); warp 11: MMA issue; warp 9: the walk over the units and their page-table
// look-ups; warp 10: the queries; warps 12, 13: the keys; 14, 15: the values.  A tile of the
// cache whose 128 tokens are all seen by some row comes by TMA, in boxes of the largest power of two of rows
// that divides a page (8 or more, the period of the swizzle); the tiles at the ends of the
// seen range, and pages that no box fits, by cp.async row by row, unseen tokens as zeros.  Two
// warps share a tile, as the issue of its boxes takes time whatever their size: 16-row pages need 16
// of them.
//
// Measured on a GB300 (cuBLAS bf16 1.94 PFLOP/s): a prompt of 8192, 64 heads of 128 over 8,
// 0.90 to 0.92 ms, 1.2 PFLOP/s; 512 tokens over 32K, capped, 331 us, 0.82 PFLOP/s; 16 x 4 drafted
// tokens over 17K-20K, 204 to 208 us, 5.9 TB/s; 8 packed prompts with documents and distance bias,
// 51 us, 48 a call in a captured graph.  No unit is full in the prompt (tensor 51 %, issue 50 %,
// special functions 33 %, FMA 13 %) nor in the capped chunk (35, 46, 18, 25 %): a tile's product,
// softmax and product follow one another, and two tiles in turn do not fill the gaps.  In the packed
// prompts and the drafted tokens barriers of the plan (1.6 to 2.3 stalled warps an issue) and
// missing instructions (0.8 to 1.5) count too.  The layout of the code and of PtShared moves the
// prompt by percents: with the products unrolled for both tiles it took 1000 us (capped chunk 347).
// Handing P over in two parts gains 25 us of the prompt and 3 of the capped chunk.  Not kept: 32-column stores of P, scores read from
// TMEM twice in 32-column steps (1060 us rolled, 1131 unrolled; capped chunk 374 and 387), the
// second half of the scores loaded under the first one's maximum (953 us, capped chunk 350).

#include <atomic>
#include <cudaTypedefs.h>

#include "paged_prefill.cuh"

namespace echo {

constexpr int PT_THREADS = 512;      // four warpgroups of 128 registers: 192 + 192 + 88 + 40 after the split
constexpr int PT_ROWS = 256, PT_KEYS = 128;
constexpr int PT_ITEMS = 4;          // ring of row tiles in flight
constexpr int PT_UNITS = 4;          // ring of units looked up
constexpr int PT_VM = 8;             // ring of the tiles' token masks

template <int D>
struct PtShape {
  static constexpr int ATOMS = D / 64;
  static constexpr int QB = ATOMS * 128 * 128;         // bytes of a query tile (and of a key or value tile)
  static constexpr int SLOTS = D == 128 ? 4 : 6;
};

struct PtShared {
  uint64_t qfull[2], qempty[2], full[8], empty[8];
  uint64_t sfull[2], pfull[2], pmost[2], pvdone[2], oempty[2], mlfull;
  uint64_t ifull[PT_ITEMS], iempty[PT_ITEMS], ufull[PT_UNITS], uempty[PT_UNITS];
  float2 ml[128];                    // (m, l) of the second half of a row tile whose tiles alternate
  uint32_t tmem_base;
  int fail;
  uint32_t vm[PT_VM][4];             // tokens there, of unit x in entry x % PT_VM
  uint32_t vmtag[PT_VM];             // 2 (x + 1) + (all of them there)
  RowTile item[PT_ITEMS];
  int64_t row[PT_UNITS][PT_KEYS];           // of a unit's tokens: offset of the row (-1: not there), and page
  int32_t page[PT_UNITS][PT_KEYS];
  int kvh[PT_UNITS], t0[PT_UNITS], whole[PT_UNITS];       // of a unit: KV head (-1: no more units), first token, every token there
  PlanShared plan;
  uint64_t drain;                    // behind the rest: 8 bytes more ahead of the arrays cost a prompt 2 %
};

template <int D>
constexpr size_t pt_smem() {
  return 1024 + (size_t)(2 + PtShape<D>::SLOTS) * PtShape<D>::QB + sizeof(PtShared);
}

__device__ __forceinline__ void pt_cp_arrive(uint64_t *bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void pt_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
      "%14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void pt_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void pt_ld64(uint32_t taddr, uint32_t (&r)[64]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63]) : "r"(taddr) : "memory");
}
__device__ __forceinline__ void pt_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void pt_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// One lane of the warp, for the TMA and MMA instructions.  With it in place of `lane == 0`, rolled
// waits, and TMA loads by a warp each, the prompt of 8192 went from 2.64 to 1.63 ms.
__device__ __forceinline__ bool pt_elect() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
// Bounded wait for a phase (a second from the 64th poll on).  Rolled up (see above), and the global
// timer only read when the wait is long: that, two load warps a tile and a walk ahead of them took
// the prompt of 8192 from 1.25 to 1.06 ms.
__device__ __forceinline__ bool pt_wait1(uint64_t *bar, uint32_t parity) {
  uint64_t t0 = 0;
#pragma unroll 1
  for (uint32_t i = 1; !mbar_try_wait(bar, parity); ++i) {
    if ((i & 63u) == 0) {
      const uint64_t t = global_ns();
      if (t0 == 0) t0 = t;
      if (t - t0 > kWaitLimitNs) return false;
    }
  }
  return true;
}
// Bounded wait of a whole warp: the same answer in every lane, and the warp together again
// (the .aligned TMEM instructions want that).
__device__ __forceinline__ bool pt_wait(uint64_t *bar, uint32_t parity) {
  return __all_sync(0xffffffffu, pt_wait1(bar, parity));
}
__device__ __forceinline__ void pt_tma3(void *dst, const CUtensorMap *map, uint64_t *bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
__device__ __forceinline__ void pt_tma4(void *dst, const CUtensorMap *map, uint64_t *bar, int c0, int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}
__device__ __forceinline__ float pt_max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// Pairs of floats, one instruction for both.
__device__ __forceinline__ uint64_t pt_pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void pt_split(uint64_t p, float &a, float &b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
}
__device__ __forceinline__ uint64_t pt_fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.ftz.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t pt_mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.ftz.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t pt_add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.ftz.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ void pt_release(uint32_t *p, uint32_t v) {
  asm volatile("st.release.cta.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(p)), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t pt_acquire(const uint32_t *p) {
  uint32_t v;
  asm volatile("ld.acquire.cta.shared::cta.b32 %0, [%1];" : "=r"(v) : "r"(smem_u32(p)) : "memory");
  return v;
}
__device__ __forceinline__ void pt_store32(void *p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
// bits [a, b) of a word
__device__ __forceinline__ uint32_t pt_bits(int a, int b) {
  a = min(max(a, 0), 32);
  b = min(max(b, 0), 32);
  const uint32_t hi = b >= 32 ? 0xffffffffu : (1u << b) - 1u, lo = a >= 32 ? 0xffffffffu : (1u << a) - 1u;
  return hi & ~lo;
}

// After a wait that gave up: the products in flight end (a bounded wait again), before their TMEM
// is given back; the CTA's partials are not joined, and the call reports.
static __device__ __noinline__ void pt_failed(uint64_t *drain, int32_t *rec, int32_t *status) {
  const int warp = threadIdx.x >> 5;
  if (warp == 11) {
    if (pt_elect()) mma_commit(drain);
    pt_wait(drain, 0);
  }
  if (threadIdx.x == 0) {
    rec[0] = 0;
    paged_fail(status, ECHO_ERR_TIMEOUT);
  }
}

template <int D, int MOD, bool ALT>
__global__ void __launch_bounds__(PT_THREADS, 1) paged_prefill_tc_kernel(const __grid_constant__ PrefillParams P,
                                                                        const __grid_constant__ CUtensorMap kmap,
                                                                        const __grid_constant__ CUtensorMap vmap,
                                                                        const __grid_constant__ CUtensorMap qmap,
                                                                        int box, int qbox) {
  using Sh = PtShape<D>;
  constexpr int QB = Sh::QB, ATOMS = Sh::ATOMS, SLOTS = Sh::SLOTS;
  constexpr bool CAP = MOD & 1, BIAS = MOD & 2;
  extern __shared__ unsigned char pt_raw[];
  unsigned char *R = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(pt_raw) + 1023) & ~uintptr_t(1023));
  PtShared &S = *reinterpret_cast<PtShared *>(R + (2 + SLOTS) * QB);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const echo_paged_kv_t &C = P.C;
  const int G = P.G;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.qfull[i], 32);
      mbar_init(&S.qempty[i], 1);
      mbar_init(&S.sfull[i], 1);
      mbar_init(&S.pfull[i], 128);
      mbar_init(&S.pmost[i], 128);
      mbar_init(&S.pvdone[i], 1);
      mbar_init(&S.oempty[i], 128);
    }
    for (int i = 0; i < SLOTS; ++i) { mbar_init(&S.full[i], 64); mbar_init(&S.empty[i], 1); }
    for (int i = 0; i < PT_ITEMS; ++i) { mbar_init(&S.ifull[i], 1); mbar_init(&S.iempty[i], 10); }
    for (int i = 0; i < PT_UNITS; ++i) { mbar_init(&S.ufull[i], 1); mbar_init(&S.uempty[i], 4); }
    for (int i = 0; i < PT_VM; ++i) S.vmtag[i] = 0;
    mbar_init(&S.mlfull, 128);
    mbar_init(&S.drain, 1);
    S.fail = 0;
    fence_mbar_init();
  }
  if (warp == 11) {
    tmem_alloc(&S.tmem_base, 512);
    tmem_relinquish();
  }
  if (tid == 32) {                                        // the first loads' descriptors, on their way
    if (box) {
      tma_prefetch_desc(&kmap);
      tma_prefetch_desc(&vmap);
    }
    if (qbox) tma_prefetch_desc(&qmap);
  }

  const RunPlan pl = prefill_plan<PT_ROWS, PT_KEYS, PT_THREADS>(P, S.plan, reinterpret_cast<uint32_t *>(R));
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem_base;
  bool ok = true;

  if (warp >= 8) {
    if (warp >= 12) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
      // -------------------------------------------------------- keys, values --
      const int which = (warp - 12) >> 1, half = warp & 1;
      const CUtensorMap *map = which ? &vmap : &kmap;
      const int nbox = box ? PT_KEYS / box : 0, jb = nbox > 1 ? half * (nbox >> 1) : 0;
      const int je = nbox > 1 ? jb + (nbox >> 1) : (half ? 0 : nbox);      // this warp's boxes
      int issued = 0;
      for (int x = 0;; ++x) {
        const int e = x % PT_UNITS, g = 2 * x + which, sl = g % SLOTS;
        if (!pt_wait(&S.ufull[e], (x / PT_UNITS) & 1)) { ok = false; break; }
        const int kvh = S.kvh[e];
        if (kvh < 0) break;
        if (!pt_wait(&S.empty[sl], ((g / SLOTS) & 1) ^ 1)) { ok = false; break; }
        unsigned char *dst = R + (2 + sl) * QB;
        if (S.whole[e]) {
          if (lane == 0 && je > jb) mbar_arrive_expect_tx(&S.full[sl], (je - jb) * box * 128 * ATOMS);
          else mbar_arrive(&S.full[sl]);
          const int j = min(jb + lane, PT_KEYS / box - 1), tj = S.t0[e] + j * box;     // box jb + lane
          const int pg = S.page[e][j * box], rj = tj - div_by(P.page, tj) * C.page_tokens;
          __syncwarp();
#pragma unroll 2
          for (int q = jb; q < je; ++q) {
            const int pq = __shfl_sync(0xffffffffu, pg, q - jb), rq = __shfl_sync(0xffffffffu, rj, q - jb);
            if (pt_elect()) {
#pragma unroll
              for (int a = 0; a < ATOMS; ++a)
                pt_tma4(dst + a * 16384 + q * box * 128, map, &S.full[sl], a * 64, rq, kvh, pq);
            }
          }
          __syncwarp();
        } else {
          const int c = lane & 7;
          const __nv_bfloat16 *src = (const __nv_bfloat16 *)(which ? C.v : C.k) + (int64_t)kvh * C.head_stride + c * 8;
#pragma unroll 4
          for (int k = 0; k < 16; ++k) {
            const int r = half * 64 + (lane >> 3) + 4 * k;
            const int64_t o = S.row[e][r];
            const __nv_bfloat16 *p = src + (o >= 0 ? o : 0);
#pragma unroll
            for (int a = 0; a < ATOMS; ++a)
              cp_async_16(dst + a * 16384 + r * 128 + ((c ^ (r & 7)) << 4), p + a * 64, o >= 0 ? 16u : 0u);
          }
          pt_cp_arrive(&S.full[sl]);
          __syncwarp();
        }
        if (lane == 0) mbar_arrive(&S.uempty[e]);
        issued = g + 1;
      }
      cp_async_wait_all();
      // after a failed wait, the copies in flight land before the CTA ends (bounded waits)
      for (int g = max(which, issued + 1 - SLOTS); !ok && g < issued; g += 2)
        pt_wait(&S.full[g % SLOTS], (g / SLOTS) & 1);
    } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    // ------------------------------------------------------------ walk, queries --
    if (warp == 9) {
      RowTileWalk<PT_ROWS, PT_KEYS> W(P, S.plan, pl);
      const RowTile &I = W.I;
      int nitem = 0, i = I.i0;                            // i: tile of the unit looked up next
      auto hand_over = [&]() {                            // the row tile, to the other warps
        const int e = nitem % PT_ITEMS;
        ok = ok && pt_wait(&S.iempty[e], ((nitem / PT_ITEMS) & 1) ^ 1);
        if (ok && lane == 0) {
          S.item[e] = I;
          mbar_arrive(&S.ifull[e]);
        }
        ++nitem;
      };
      if (lane == 0) P.rec[blockIdx.x * 8] = 0;
      hand_over();
      for (int x = 0;; ++x) {
        if (x > 0 && i == I.i1) {
          W.next();
          i = I.i0;
          hand_over();
        }
        const bool more = I.i1 >= 0;
        const int e = x % PT_UNITS, v = x % PT_VM, t0 = more ? I.span.tile(i++) * PT_KEYS : 0;
        int32_t ent[4];
        uint32_t seen = 0, all = 0xffffffffu;             // seen, bit k: token t0 + lane + 32 k is seen by some row
        if (more) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int t = t0 + lane + 32 * k;
            const bool some = t < I.len && t >= I.first && ((t >= I.lo && t < I.hi) || t < I.pre);
            seen |= some ? 1u << k : 0u;
            ent[k] = some ? __ldg(C.page_table + (int64_t)I.b * C.max_pages + div_by(P.page, t)) : -1;
          }
          if (I.holes) {                                  // less what no row sees
            uint32_t own = 0;
#pragma unroll 1
            for (int k = 0; k < 4; ++k) {
              const int t = t0 + lane + 32 * k;
              own |= (seen_by_some(P, I, t0 + 32 * k) || t < I.pre) ? 1u << k : 0u;
            }
            seen &= own;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (!((seen >> k) & 1u)) ent[k] = -1;
          }
        }
        ok = ok && pt_wait(&S.uempty[e], ((x / PT_UNITS) & 1) ^ 1);
        if (!ok) break;                                   // the others give up at their own waits
        if (more) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const bool page = ent[k] >= 0 && ent[k] < C.n_pages;
            if (((seen >> k) & 1u) && !page) paged_fail(C.status, ECHO_ERR_PAGE);
            const uint32_t m = __ballot_sync(0xffffffffu, page);
            all &= m;
            if (lane == 0) S.vm[v][k] = m;
            S.page[e][lane + 32 * k] = ent[k];
          }
          if (!box || all != 0xffffffffu) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int t = t0 + lane + 32 * k;
              const bool page = ent[k] >= 0 && ent[k] < C.n_pages;
              S.row[e][lane + 32 * k] = page ? (int64_t)ent[k] * C.page_stride +
                                                   (int64_t)(t - div_by(P.page, t) * C.page_tokens) * C.row_stride
                                             : -1;
            }
          }
          if (lane == 0) {
            S.t0[e] = t0;
            S.whole[e] = box && all == 0xffffffffu;
            pt_release(&S.vmtag[v], 2u * (uint32_t)(x + 1) + (all == 0xffffffffu ? 1u : 0u));
          }
        }
        __syncwarp();
        if (lane == 0) {
          S.kvh[e] = more ? I.kvh : -1;
          mbar_arrive(&S.ufull[e]);
        }
        if (!more) break;
      }
    } else if (warp == 10) {
      int nq[2] = {0, 0}, nitem = 0;
      while (ok) {
        const int e = nitem % PT_ITEMS;
        if (!pt_wait(&S.ifull[e], (nitem / PT_ITEMS) & 1)) { ok = false; break; }
        ++nitem;
        const int s0 = S.item[e].s0, r0 = S.item[e].r0, nr = S.item[e].nr, kvh = S.item[e].kvh, i1 = S.item[e].i1;
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.iempty[e]);
        if (i1 < 0) break;
        for (int h = 0; h < (nr > 128 ? 2 : 1) && ok; ++h) {
          if (!pt_wait(&S.qempty[h], (nq[h] & 1) ^ 1)) { ok = false; break; }
          ++nq[h];
          unsigned char *dst = R + h * QB;
          if (qbox) {                                     // G divides 128: whole tokens
            if (lane == 0) mbar_arrive_expect_tx(&S.qfull[h], QB);
            else mbar_arrive(&S.qfull[h]);
            __syncwarp();
            if (pt_elect()) {
#pragma unroll
              for (int a = 0; a < ATOMS; ++a)
                pt_tma3(dst + a * 16384, &qmap, &S.qfull[h], a * 64, kvh * G, s0 + div_by(P.group, r0 + 128 * h));
            }
            __syncwarp();
          } else {
            const int c = lane & 7;
            const __nv_bfloat16 *q = (const __nv_bfloat16 *)P.q + (int64_t)s0 * P.q_stride + (int64_t)kvh * G * D + c * 8;
#pragma unroll 4
            for (int k = 0; k < 32; ++k) {
              const int r = (lane >> 3) + 4 * k, rt = h * 128 + r;
              const bool there = rt < nr;
              const int t = there ? div_by(P.group, r0 + rt) : 0, gh = there ? r0 + rt - t * G : 0;
              const __nv_bfloat16 *src = q + (int64_t)t * P.q_stride + gh * D;
#pragma unroll
              for (int a = 0; a < ATOMS; ++a)
                cp_async_16(dst + a * 16384 + r * 128 + ((c ^ (r & 7)) << 4), src + a * 64, there ? 16u : 0u);
            }
            pt_cp_arrive(&S.qfull[h]);
          }
        }
      }
      for (int h = 0; !ok && h < 2; ++h)
        if (nq[h]) pt_wait(&S.qfull[h], (nq[h] - 1) & 1);
    }
    if (warp == 10) cp_async_wait_all();
    if (warp == 11 && pt_elect()) {
    // ------------------------------------------------------------------ MMA --
      // One thread issues everything, and the tensor cores wait whenever it is late: what can be
      // waited for early (the keys of unit x + 1 and the values of x) is, before the weights of
      // x; a tile's PV(x) and QK(x + 1) then go out together.  A commit behind other commits
      // stalls until the products before it are done, so there is one a QK, and what else it
      // sets free -- K(x), V(x - 1), a row tile's queries -- the softmax warps hand back when
      // they wake up on it.
      constexpr uint32_t id_qk = instr_desc(FMT_BF16, FMT_BF16, 0, 0, 128, 128);
      constexpr uint32_t id_pv = instr_desc(FMT_BF16, FMT_BF16, 0, 1, 128, D);
      const uint32_t ring = smem_u32(R + 2 * QB);
      const uint64_t qd = smem_desc(smem_u32(R), 16, 1024, LAYOUT_SW128);
      const uint64_t kd = smem_desc(ring, 16, 1024, LAYOUT_SW128);
      const uint64_t vd = smem_desc(ring, 128 * 128, 1024, LAYOUT_SW128);
      // slots and phases: keys of the unit whose scores come next, values of unit x; phase bits
      // of the tiles' queries and weights, and of the O that an epilogue gives back
      uint32_t ks = 0, kph = 0, vs = 1, vph = 0, qph = 0, pph = 0, oph = 3;
      int nitem = 0;
      while (ok) {
        const int e = nitem % PT_ITEMS;                   // the next row tile
        if (!pt_wait1(&S.ifull[e], (nitem / PT_ITEMS) & 1)) { ok = false; break; }
        const int i1 = S.item[e].i1, n = i1 - S.item[e].i0;
        const bool two = S.item[e].nr > 128;
        mbar_arrive(&S.iempty[e]);
        ++nitem;
        if (i1 < 0) break;
        // Step j: the values of unit j, then the scores of unit j + lag into the S that they left;
        // of both tiles, or of the half whose turn it is.  One rolled body for the first scores,
        // the loop and the last values: what this thread runs has to stay in the instruction
        // cache beside the softmax.
        const int lag = ALT && !two && n >= 2 ? 2 : 1;
#pragma unroll 1
        for (int j = -lag; ok && j < n; ++j) {
          const bool more = j + lag < n;
          if (more) ok = pt_wait1(&S.full[ks], kph);
          if (j >= 0) ok = ok && pt_wait1(&S.full[vs], vph);
          fence_proxy_async_smem();                       // the loaders' cp.async writes, for the tensor cores
#pragma unroll 1
          for (int h = 0; ok && h <= (two ? 1 : 0); ++h) {
            const int t = lag == 2 ? j & 1 : h;
            const uint32_t bit = 1u << t, st = tmem + 128u * t;
            if (j >= 0) {
              ok = pt_wait1(&S.pmost[t], (pph >> t) & 1u); // weights of the first 96 tokens
              if (j < lag) {                              // the row tile's first values
                ok = ok && pt_wait1(&S.oempty[t], (oph >> t) & 1u);
                oph ^= bit;
              }
              if (!ok) break;
              tc_fence_after();
              const uint64_t bd = vd + (uint64_t)(vs * (QB >> 4));
#pragma unroll 4
              for (int k = 0; k < 3 * PT_KEYS / 64; ++k)
                pt_mma_ts(st + 256u, st + 8u * k, bd + 128 * k, id_pv, (j >= lag || k) ? 1u : 0u);
              ok = pt_wait1(&S.pfull[t], (pph >> t) & 1u);
              pph ^= bit;
              if (!ok) break;
              tc_fence_after();
#pragma unroll
              for (int k = 3 * PT_KEYS / 64; k < PT_KEYS / 16; ++k)
                pt_mma_ts(st + 256u, st + 8u * k, bd + 128 * k, id_pv, 1u);
            }
            if (more) {
              if (j < 0 && (lag == 1 || j == -2)) {
                ok = pt_wait1(&S.qfull[h], (qph >> h) & 1u);
                qph ^= 1u << h;
                if (!ok) break;
                fence_proxy_async_smem();
              }
              tc_fence_after();
              const uint64_t ad = qd + (uint64_t)(h * (QB >> 4)), bd = kd + (uint64_t)(ks * (QB >> 4));
#pragma unroll 4
              for (int k = 0; k < D / 16; ++k) {
                const uint32_t o = (uint32_t)((k >> 2) * 1024 + (k & 3) * 2);
                mma_f16(st, ad + o, bd + o, id_qk, k ? 1u : 0u);
              }
              mma_commit(&S.sfull[t]);
            } else {
              mma_commit(&S.pvdone[t]);                   // the epilogue's
            }
          }
          if (more) {
            ks += 2;
            if (ks >= SLOTS) { ks = 0; kph ^= 1; }
          }
          if (j >= 0) {
            vs += 2;
            if (vs >= SLOTS) { vs = 1; vph ^= 1; }
          }
        }
      }
    }
    }
  } else {
    // -------------------------------------------------------------- softmax --
    asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
    const int t = warp >> 2;
    const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t ts = trow + 128u * t, to = trow + 256u + 128u * t;
    const int wr = (warp & 3) * 32 + lane;                // row of the tile
    const float aa = fmaxf(P.f.a, 1e-37f);                // a scale of 0 keeps masked scores at -inf
    // units, row tiles, this half's units and its finished sums (with row tiles that alternate:
    // both halves'), such row tiles, and value tiles of the last row tile not handed back, so far
    int x = 0, nitem = 0, ns = 0, nd[2] = {0, 0}, nalt = 0, vrem = 0;
    while (ok) {
      const int e = nitem % PT_ITEMS;
      if (!pt_wait(&S.ifull[e], (nitem / PT_ITEMS) & 1)) { ok = false; break; }
      ++nitem;
      const RowTile &I = S.item[e];
      const int i0 = I.i0, i1 = I.i1;
      if (i1 < 0) break;
      const bool two = I.nr > 128, alt = ALT && !two && i1 - i0 >= 2;
      if (t == 1 && !two && !alt) {
        x += i1 - i0;
        if (ALT) {
          ++nd[0];
          vrem = 1;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.iempty[e]);
        continue;
      }
      const int r = (alt ? 0 : t * 128) + wr;             // row of the row tile
      const int len = I.len, n = I.n, nr = I.nr, r0 = I.r0, s0 = I.s0, kvh = I.kvh, elsewhere = I.elsewhere, c0 = I.c0;
      const TileSpan span = I.span;
      int pre = I.pre;
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.iempty[e]);
      const bool there = r < nr, some = r - lane < nr;
      const int tk = there ? div_by(P.group, r0 + r) : 0, hd = there ? kvh * G + (r0 + r) - tk * G : 0;
      int pos = len - n + tk, first = 0, lo = 0;
      if (!there || pos < 0) {
        first = lo = 0x7fffffff;
        pos = -1;
        pre = 0;
      } else {
        if (P.first_tok) first = max(__ldg(P.first_tok + s0 + tk), 0);
        lo = P.window ? max(first, pos - P.window + 1) : first;
      }
      float slope = 0.f;
      if (BIAS && P.slopes && there) slope = __ldg(P.slopes + hd) * kPgLog2e;
      // tiles that every row of the warp sees whole: by its window, and by its prefix
      const int wa = __reduce_max_sync(0xffffffffu, there ? (int)(((unsigned)lo + PT_KEYS - 1) / PT_KEYS) : 0);
      const int wb = __reduce_min_sync(0xffffffffu, there ? (pos + 1) / PT_KEYS : 0x7fffffff);
      const int pa = __reduce_max_sync(0xffffffffu, there ? (int)(((unsigned)first + PT_KEYS - 1) / PT_KEYS) : 0);
      const int pb = __reduce_min_sync(0xffffffffu, there ? pre / PT_KEYS : 0x7fffffff);
      float m = -INFINITY, l = 0.f;
      const int step = alt ? 2 : 1;
      int i = i0;
      if (alt) i += t, x += t;
      for (; i < i1; i += step, x += step, ++ns) {
        if (!pt_wait(&S.sfull[t], ns & 1)) { ok = false; break; }
        tc_fence_after();
        if ((warp & 3) == 0 && lane == 0) {                // every product up to this QK is done
          if (alt || t == (two ? 1 : 0)) {                 // (of two tiles' the second is issued last)
            mbar_arrive(&S.empty[(2 * x) % SLOTS]);
            if (!ALT) {
              if (x > 0) mbar_arrive(&S.empty[(2 * x - 1) % SLOTS]);
            } else if (i - step >= i0) {
              mbar_arrive(&S.empty[(2 * (x - step) + 1) % SLOTS]);
            } else if (i == i0) {
              for (int k = 1; k <= vrem; ++k) mbar_arrive(&S.empty[(2 * (x - k) + 1) % SLOTS]);
            }
          }
          if (i + 1 == i1) mbar_arrive(&S.qempty[alt ? 0 : t]);
        }
        if (some) {
          const int ti = span.tile(i), t0 = ti * PT_KEYS;
          float v[128];
          {
            uint32_t (*u)[64] = reinterpret_cast<uint32_t (*)[64]>(v);
#pragma unroll
            for (int k = 0; k < 2; ++k) pt_ld64(ts + 64 * k, u[k]);
          }
          // the tile's token mask: written before its keys were loaded, so it is there
          uint32_t tag = pt_acquire(&S.vmtag[x % PT_VM]);
          const bool whole = ((ti >= wa && ti < wb) || (ti >= pa && ti < pb)) && tag == 2u * (uint32_t)(x + 1) + 1u;
          tmem_wait_ld();
          if (CAP) {
            // u = s a, then tanh by its polynomial where every score of the warp is small enough
            // (seven operations of two scores each on the FMA units): the general form's power and
            // reciprocal go through the special-function units (without it the capped chunk took 456 us)
            const uint64_t a2 = pt_pair(P.f.a, P.f.a);
            float um = 0.f;
#pragma unroll
            for (int k = 0; k < 128; k += 2) {
              pt_split(pt_mul2(pt_pair(v[k], v[k + 1]), a2), v[k], v[k + 1]);
              um = pt_max3(um, fabsf(v[k]), fabsf(v[k + 1]));
            }
            if (__all_sync(0xffffffffu, um * um <= kTanhW)) {
              const uint64_t c5 = pt_pair(kTanh5, kTanh5), c4 = pt_pair(kTanh4, kTanh4), c3 = pt_pair(kTanh3, kTanh3),
                             c2 = pt_pair(kTanh2, kTanh2), c1 = pt_pair(kTanh1, kTanh1);
#pragma unroll
              for (int k = 0; k < 128; k += 2) {
                const uint64_t u = pt_pair(v[k], v[k + 1]), w = pt_mul2(u, u);
                uint64_t p = pt_fma2(w, c5, c4);
                p = pt_fma2(w, p, c3);
                p = pt_fma2(w, p, c2);
                p = pt_fma2(w, p, c1);
                pt_split(pt_fma2(pt_mul2(u, w), p, u), v[k], v[k + 1]);
              }
            } else {
#pragma unroll
              for (int k = 0; k < 128; ++k) v[k] = tanh_ex2(v[k]);
            }
          }
          if (BIAS) {
            const float mul = CAP ? P.f.c : P.f.a;
            if (pre == 0 || ti < wb) {
              // no token behind a row's position counts: |p - t| = (p - t0) - k
              const float d0 = -slope * (float)(pos - t0);
              const uint64_t m2 = pt_pair(mul, mul), s2 = pt_pair(slope, slope), d2 = pt_pair(d0, d0);
#pragma unroll
              for (int k = 0; k < 128; k += 2)
                pt_split(pt_fma2(pt_pair(v[k], v[k + 1]), m2, pt_fma2(s2, pt_pair((float)k, (float)(k + 1)), d2)), v[k], v[k + 1]);
            } else {
              const float d0 = (float)(pos - t0);
#pragma unroll
              for (int k = 0; k < 128; ++k) v[k] = fmaf(-slope, fabsf(d0 - (float)k), v[k] * mul);
            }
          }
          if (!whole) {                                   // the same in every lane
            for (uint32_t k = 0; (tag >> 1) != (uint32_t)(x + 1) && k < (1u << 20); ++k) tag = pt_acquire(&S.vmtag[x % PT_VM]);
            if ((tag >> 1) != (uint32_t)(x + 1)) S.fail = 1;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int w0 = t0 + 32 * k;
              const uint32_t w = (pt_bits(lo - w0, pos + 1 - w0) | pt_bits(first - w0, pre - w0)) & S.vm[x % PT_VM][k];
#pragma unroll
              for (int q = 0; q < 32; ++q) v[32 * k + q] = (w >> q) & 1u ? v[32 * k + q] : -INFINITY;
            }
          }
          float mx4[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
          for (int k = 4; k < 124; k += 8) {
#pragma unroll
            for (int q = 0; q < 4; ++q) mx4[q] = pt_max3(mx4[q], v[k + 2 * q], v[k + 2 * q + 1]);
          }
          mx4[0] = pt_max3(mx4[0], v[124], v[125]);
          mx4[1] = pt_max3(mx4[1], v[126], v[127]);
          float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
          const float sc = BIAS ? 1.f : CAP ? P.f.c : aa;
          mx *= sc;
          // move the maximum when it is passed by 2^8, or was none (PV of the tile before was
          // issued ahead of this tile's QK: it is done)
          const float nm = mx > m + 8.f ? mx : m;
          if (i < i0 + step) {
            m = mx;
          } else if (__any_sync(0xffffffffu, nm != m)) {
            const float corr = nm != m ? ex2(m - nm) : 1.f;
            m = nm;
            l *= corr;
#pragma unroll 1
            for (int k = 0; k < D; k += 16) {
              uint32_t o[16];
              pt_ld16(to + k, o);
              tmem_wait_ld();
#pragma unroll
              for (int q = 0; q < 16; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * corr);
              pt_st16(to + k, o);
            }
          }
          const float z = m == -INFINITY ? 0.f : m;
          // weights, rounded to bf16 for the product (by 2^-8 of each at most); the sum takes the
          // unrounded ones
          const uint64_t sc2 = pt_pair(sc, sc), z2 = pt_pair(-z, -z);
          uint64_t l2[4] = {0, 0, 0, 0};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t pk[16];
#pragma unroll
            for (int q = 0; q < 32; q += 2) {
              float a, c;
              pt_split(pt_fma2(pt_pair(v[32 * k + q], v[32 * k + q + 1]), sc2, z2), a, c);
              a = ex2(a);
              c = ex2(c);
              l2[(q >> 1) & 3] = pt_add2(l2[(q >> 1) & 3], pt_pair(a, c));
              const __nv_bfloat162 h = __floats2bfloat162_rn(a, c);
              pk[q >> 1] = *reinterpret_cast<const uint32_t *>(&h);
            }
            if (k == 3) {
              pt_wait_st();
              tc_fence_before();
              mbar_arrive(&S.pmost[t]);                    // three quarters: their product can start
            }
            pt_st16(ts + 16 * k, pk);
          }
          {
            float a, c;
            pt_split(pt_add2(pt_add2(l2[0], l2[1]), pt_add2(l2[2], l2[3])), a, c);
            l += a + c;
          }
          pt_wait_st();
        } else {
          mbar_arrive(&S.pmost[t]);
        }
        tc_fence_before();
        mbar_arrive(&S.pfull[t]);
      }
      if (!ok) break;
      // ---- epilogue
      if (alt) x -= i - i1;
      vrem = step;
      float f0 = 1.f, f1 = 0.f;
      if (alt) {
        // half 0 joins both: O_1 from its own lanes of TMEM, (m, l) through shared memory, which
        // half 0 has read by the time it gives O_1 up
        if (t == 1) {
          if (nd[1] && !pt_wait(&S.oempty[1], (nd[1] - 1) & 1)) { ok = false; break; }
          S.ml[wr] = make_float2(m, l);
          mbar_arrive(&S.mlfull);
        } else if (!pt_wait(&S.mlfull, nalt & 1) || !pt_wait(&S.pvdone[0], nd[0] & 1)) {
          ok = false;
          break;
        }
        if (!pt_wait(&S.pvdone[1], nd[1] & 1)) { ok = false; break; }
        ++nalt;
        ++nd[0];
        ++nd[1];
        if (t == 1) continue;
        const float2 o = S.ml[wr];
        const float nm = fmaxf(m, o.x), z = nm == -INFINITY ? 0.f : nm;
        f0 = ex2(m - z);
        f1 = ex2(o.x - z);
        m = nm;
        l = l * f0 + o.y * f1;
      } else {
        if (!pt_wait(&S.pvdone[t], nd[ALT ? t : 0] & 1)) { ok = false; break; }
        ++nd[0];
        if (ALT && two) ++nd[1];
      }
      tc_fence_after();
      const bool done = elsewhere == 0;
      const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
      const int64_t orow = (int64_t)(s0 + tk) * P.Hq + hd;
      const int64_t prow = (int64_t)(2 * blockIdx.x + ((elsewhere & 1) ? 0 : 1)) * P.prows + r;
      if (some) {
#pragma unroll 1
        for (int k = 0; k < D; k += 32) {
          uint32_t o[32];
          tmem_ld32(to + k, o);
          if (alt) {
            uint32_t o1[32];
            tmem_ld32(to + 128 + k, o1);
            tmem_wait_ld();
#pragma unroll
            for (int q = 0; q < 32; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * f0 + __uint_as_float(o1[q]) * f1);
          }
          tmem_wait_ld();
          if (there) {
            if (done) {
              __nv_bfloat16 *dst = (__nv_bfloat16 *)P.out + orow * D + k;
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                uint32_t w[8];
#pragma unroll
                for (int y = 0; y < 8; ++y) {
                  const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(o[16 * q + 2 * y]) * inv,
                                                                 __uint_as_float(o[16 * q + 2 * y + 1]) * inv);
                  w[y] = *reinterpret_cast<const uint32_t *>(&h);
                }
                if (P.wide) {                              // whole 32-byte sectors
                  pt_store32(dst + 16 * q, w);
                } else {
                  reinterpret_cast<uint4 *>(dst + 16 * q)[0] = make_uint4(w[0], w[1], w[2], w[3]);
                  reinterpret_cast<uint4 *>(dst + 16 * q)[1] = make_uint4(w[4], w[5], w[6], w[7]);
                }
              }
            } else {
              uint4 *dst = reinterpret_cast<uint4 *>(P.po + prow * D + k);
#pragma unroll
              for (int q = 0; q < 8; ++q) dst[q] = make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
            }
          }
        }
      }
      tc_fence_before();
      mbar_arrive(&S.oempty[t]);
      if (alt) mbar_arrive(&S.oempty[1]);
      if (there) {
        if (done) P.lse[orow] = l == 0.f ? -INFINITY : (m + log2f(l)) * kPgLn2;
        else *reinterpret_cast<float2 *>(P.pml + prow * 2) = make_float2(m, l);
      }
      if (r == 0 && elsewhere == 1) {                      // a split row tile ends here: to be joined
        join_record(P, c0, s0, r0, nr, kvh);
      }
    }
  }
  if (!ok) S.fail = 1;                                    // a bounded wait gave up
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (S.fail) pt_failed(&S.drain, P.rec + blockIdx.x * 8, C.status);
  if (warp == 11) tmem_dealloc(tmem, 512);
}

// A bf16 tensor of `nd` dimensions with 128-byte-swizzled boxes of 64 innermost values; strides
// in values, of all but the innermost dimension.  False where a stride is none that a tensor
// map takes (the loads then go row by row).
static bool bf16_map(CUtensorMap *m, const void *base, int nd, const int64_t *dims, const int64_t *strides, const int *box) {
  static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> fn{nullptr};
  PFN_cuTensorMapEncodeTiled_v12000 enc = fn.load(std::memory_order_acquire);
  if (!enc) {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult qr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &qr) != cudaSuccess ||
        qr != cudaDriverEntryPointSuccess)
      return false;
    enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    fn.store(enc, std::memory_order_release);
  }
  cuuint64_t ds[4], st[3];
  cuuint32_t bx[4], es[4] = {1, 1, 1, 1};
  for (int i = 0; i < nd; ++i) {
    ds[i] = (cuuint64_t)dims[i];
    bx[i] = (cuuint32_t)box[i];
    if (i + 1 < nd) {
      if (strides[i] <= 0 || strides[i] >= (1ll << 38)) return false;
      st[i] = (cuuint64_t)strides[i] * 2;
    }
  }
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)nd, const_cast<void *>(base), ds, st, bx, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int MOD, bool ALT>
static echo_status_t launch_tc(PrefillParams &P, cudaStream_t st) {
  static_assert(pt_smem<D>() <= 227 * 1024, "fits an SM");
  ECHO_CUDA_OK((allow_smem<paged_prefill_tc_kernel<D, MOD, ALT>>(pt_smem<D>())));
  int box = std::min(P.C.page_tokens & -P.C.page_tokens, PT_KEYS), qbox = 128 % P.G == 0 ? 128 / P.G : 0;
  CUtensorMap kmap = {}, vmap = {}, qmap = {};
  {
    // pages [page][head][row][value], boxes of `box` rows; the stride of a dimension of one
    // entry is never used: any that is valid will do
    const echo_paged_kv_t &C = P.C;
    const int64_t dims[4] = {D, C.page_tokens, C.n_kv_heads, C.n_pages};
    const int64_t st[3] = {C.page_tokens > 1 ? C.row_stride : D, C.n_kv_heads > 1 ? C.head_stride : D,
                           C.n_pages > 1 ? C.page_stride : D};
    const int bx[4] = {64, box, 1, 1};
    if (box < 8 || !bf16_map(&kmap, C.k, 4, dims, st, bx) || !bf16_map(&vmap, C.v, 4, dims, st, bx)) box = 0;
    // queries [token][head][value], boxes of 128 packed rows
    const int64_t qd[3] = {D, P.Hq, P.N}, qs[2] = {D, P.N > 1 ? P.q_stride : D};
    const int qb[3] = {64, P.G, qbox};
    if (qbox && !bf16_map(&qmap, P.q, 3, qd, qs, qb)) qbox = 0;
  }
  const int grid = std::min(sm_count(), PF_MAX_CTAS / 2);
  paged_prefill_tc_kernel<D, MOD, ALT><<<grid, PT_THREADS, pt_smem<D>(), st>>>(P, kmap, vmap, qmap, box, qbox);
  ECHO_LAUNCH_OK();
  ECHO_CUDA_OK(launch_after(paged_prefill_join_kernel<__nv_bfloat16, D>, dim3(grid, (P.prows + 3) / 4), dim3(128), st, P));
  return ECHO_OK;
}

template <int D>
static echo_status_t launch_mod(PrefillParams &P, cudaStream_t st) {
  // a negative scale goes with the bias: the plain form takes the largest raw product
  const int mod = (P.f.capped ? 1 : 0) | (P.slopes || P.f.a < 0.f ? 2 : 0);
  // Row tiles of one query tile alternate over the cache only in a kernel of their own: four
  // drafted tokens each of 16 sequences of 20K went from 227 to 207 us with it, a prompt of 8192
  // from 1000 to 1080 (its loop then spills).  Taken where a sequence's rows on average fit one
  // query tile; either kernel is right for any mixture.
  const bool alt = (int64_t)P.N * P.G <= 128 * (int64_t)P.B;
  switch (2 * mod + (alt ? 1 : 0)) {
    case 0: return launch_tc<D, 0, false>(P, st);
    case 1: return launch_tc<D, 0, true>(P, st);
    case 2: return launch_tc<D, 1, false>(P, st);
    case 3: return launch_tc<D, 1, true>(P, st);
    case 4: return launch_tc<D, 2, false>(P, st);
    case 5: return launch_tc<D, 2, true>(P, st);
    case 6: return launch_tc<D, 3, false>(P, st);
    default: return launch_tc<D, 3, true>(P, st);
  }
}

echo_status_t launch_prefill_tc(PrefillParams &P, cudaStream_t st) {
  return P.C.head_dim == 128 ? launch_mod<128>(P, st) : launch_mod<64>(P, st);
}

}  // namespace echo
