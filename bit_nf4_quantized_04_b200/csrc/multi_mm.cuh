// The many-adapter product for many tokens, over a base in 16 bits:
//
//   D[t, f] = sum_c X[t, c] W[f, c] + sum over the tile's adapters of E[t] . G[f]   (forward)
//   D[t, f] = sum_c X[t, c] W[c, f] + ...                                           (dX)
//
// with t a token (M of them), f an output feature, X = x or dY, W the bf16 base [N, K], and per
// adapter that a 256-token tile names E = its tokens' s u or s v (other rows zero) and G its B
// rows or A columns.
//
// k_gemm dequantizes inside its operand producer, so it converts each weight once per column
// tile: at 256 tokens a tile its converters' byte permutes and the shared memory traffic of one
// CTA's 128 x 256 tile (A 16 KB and B 32 KB written and read per 64 of the contraction, 768
// cycles of shared memory against 512 of tensor core) hold it at 0.55 of the bf16 peak. With
// many tokens it is cheaper to write bf16(W_hat) once (2.5 bytes per weight, from L2 or HBM) and
// to multiply by pairs of CTAs: cta_group::2 MMAs of 256 tokens x 256 features, each CTA holding
// half of either operand (32 KB written and read per step), two accumulators of 256 TMEM columns
// so that a tile's epilogue runs under the next tile's products.
//
// Roles (192 threads per CTA): warp 0 issues this CTA's TMA loads, which all report to the
// leading CTA's barriers; warp 1 of the leading CTA issues the MMAs for the pair and releases
// stages in both by multicast commits; warps 2-5 read their CTA's 128 accumulator rows, round to
// bf16 and store 32 x 64 pieces by TMA. The adapters' operands come as further ring positions of
// rp = 16, 32 or 64 columns, one per adapter of the tile's list, from copies that k_multi_stage
// padded to rp and freed of non-finite entries (whose products the epilogue adds to their own
// adapter's tokens, only if there are any: mm_fix).
//
// Bound by the tensor pipe (89 to 94 % busy over the kernel): 4096 tokens through 11008 x 4096 with 8
// adapters of r = 16, 225 to 245 us forward (1651 to 1514 TFLOP/s) and 241 to 258 us for dX (1536 to
// 1433) on two boxes, whose clocks under this load differ. What is left is the last
// wave of tiles; cutting it along the contraction with partial tiles through L2 lost (5120 x 5120,
// 1531 tokens: 113 us for the call instead of 105 at the time), so tiles stay whole.
#pragma once
#include "common.cuh"
#include "gemm.cuh"
#include "multi.cuh"

namespace qnf4 {

// ---------------------------------------------------------------------------
// CTA pairs
// ---------------------------------------------------------------------------
QNF4_DEV void tmem_alloc2(uint32_t* dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst_smem)),
               "r"(ncols)
               : "memory");
}
QNF4_DEV void tmem_relinquish2() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
QNF4_DEV void tmem_dealloc2(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
QNF4_DEV void mma2_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrive on the barrier at this offset in both CTAs once the MMAs issued so far are complete.
QNF4_DEV void mma2_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}
QNF4_DEV uint32_t map_to_cta(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
// Tile into this CTA's shared memory, completion on a barrier of either CTA of the pair.
QNF4_DEV void tma_load_2d_pair(void* dst, const CUtensorMap* map, uint32_t bar, int32_t x, int32_t y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
      : "memory");
}
QNF4_DEV void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// ---------------------------------------------------------------------------
// The 16-bit base and the adapters' operand
// ---------------------------------------------------------------------------
// W_hat as bf16 (each weight bf16(fp32(level * constant)), as the linear layers define it; no
// work for a 16-bit base), and the adapters' B [n, N, r] or A [n, r, K] copied with rows of rp
// (zeros past r) and non-finite entries replaced by zero; bad[CTA] says whether it met any. Bound by
// writing W; each packed byte is one lookup of two levels, two products and one conversion. Six CTAs per SM
// of at most 40 registers (11008 x 4096: 23 us; one code at a time from a level table 30 us).
struct StageArgs {
  const uint32_t* packed;  // null for a 16-bit base
  const uint8_t* code2;
  const float* scale2;
  const float* mean;
  int64_t n8;              // weights / 8
  uint16_t* W;
  const uint16_t* src;     // B [rows, r], or A [n, r, K]
  uint16_t* dst;           // [rows, rp], or [n, rp, K]
  int64_t rows, cols;      // rows: n N, or n; cols: 1, or K
  int r, rp;
  int* bad;                // [gridDim.x]
  float levels[16];
};

constexpr int kStageCopies = 8;  // of the pair table, one per lane mod 8

__global__ void __launch_bounds__(256, 6) k_multi_stage(const __grid_constant__ StageArgs g) {
  // entry b, copy j at b * 8 + j: the two levels a packed byte selects. A lane's copy fixes three
  // bits of the bank pair, so that two lanes of a half warp meet half the time and no more do.
  __shared__ float2 s_pair[256 * kStageCopies];
  const int tid = threadIdx.x, lane = tid & 31;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * 256 + tid, step = static_cast<int64_t>(gridDim.x) * 256;
  if (g.packed)
    for (int i = tid; i < 256 * kStageCopies; i += 256) {
      const int b = i / kStageCopies;
      s_pair[i] = make_float2(g.levels[b >> 4], g.levels[b & 15]);
    }
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  // adapters: 8 elements of a row of rp (B), or of a row of K (A)
  uint32_t bad = 0u;
  if (g.cols == 1) {
    const int per = g.rp / 8;
    for (int64_t i = t0; i < g.rows * per; i += step) {
      const int64_t row = i / per;
      const int j0 = static_cast<int>(i - row * per) * 8;
      const uint16_t* s = g.src + row * g.r + j0;
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if ((g.r & 7) == 0) {
        if (j0 < g.r) v = __ldg(reinterpret_cast<const uint4*>(s));
      } else {
        uint32_t e[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) e[k] = j0 + k < g.r ? s[k] : 0u;
        v = make_uint4(e[0] | (e[1] << 16), e[2] | (e[3] << 16), e[4] | (e[5] << 16), e[6] | (e[7] << 16));
      }
      bad |= bf16x2_nonfinite(v.x) | bf16x2_nonfinite(v.y) | bf16x2_nonfinite(v.z) | bf16x2_nonfinite(v.w);
      v = make_uint4(bf16x2_finite(v.x), bf16x2_finite(v.y), bf16x2_finite(v.z), bf16x2_finite(v.w));
      reinterpret_cast<uint4*>(g.dst)[i] = v;
    }
  } else {
    const int64_t per = g.cols / 8;
    for (int64_t i = t0; i < g.rows * g.rp * per; i += step) {
      const int64_t row = i / per, a = row / g.rp;
      const int j = static_cast<int>(row - a * g.rp);
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (j < g.r) v = __ldg(reinterpret_cast<const uint4*>(g.src + (a * g.r + j) * g.cols + (i - row * per) * 8));
      bad |= bf16x2_nonfinite(v.x) | bf16x2_nonfinite(v.y) | bf16x2_nonfinite(v.z) | bf16x2_nonfinite(v.w);
      v = make_uint4(bf16x2_finite(v.x), bf16x2_finite(v.y), bf16x2_finite(v.z), bf16x2_finite(v.w));
      reinterpret_cast<uint4*>(g.dst)[i] = v;
    }
  }
  const int any = __syncthreads_or(bad != 0u);
  if (tid == 0) g.bad[blockIdx.x] = any;
  if (!g.packed) return;
  const float mu = *g.mean;
  const float2* tab = s_pair + (lane & (kStageCopies - 1));
  const int64_t n1 = g.n8 >> 3;  // blocks
  // a warp takes 128 words (8 codes each): 16 blocks, whose constants lanes 0-15 make
  const int64_t wstep = static_cast<int64_t>(gridDim.x) * 8 * 128;
#pragma unroll 2
  for (int64_t w0 = (static_cast<int64_t>(blockIdx.x) * 8 + (tid >> 5)) * 128; w0 < g.n8; w0 += wstep) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = w0 + 32 * k + lane < g.n8 ? __ldg(g.packed + w0 + 32 * k + lane) : 0u;
    const int64_t b = (w0 >> 3) + (lane & 15);
    const float mine = b < n1 ? fmaf(e4m3_to_f32(__ldg(g.code2 + b)), __ldg(g.scale2 + (b >> 8)), mu) : 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float c = __shfl_sync(0xffffffffu, mine, 4 * k + (lane >> 3));
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 v = tab[__byte_perm(w[k], 0u, 0x4440u + j) * kStageCopies];
        o[j] = pack_bf16x2(v.x * c, v.y * c);
      }
      if (w0 + 32 * k + lane < g.n8) reinterpret_cast<uint4*>(g.W)[w0 + 32 * k + lane] = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

// ---------------------------------------------------------------------------
// The product
// ---------------------------------------------------------------------------
// A stage is 128 of the contraction: the one thread that issues the MMAs spends about 590 cycles
// on a stage of 64 (barrier test 120, four MMAs 270, commit 80, loop 100) that holds 512 cycles of
// tensor work, so that it, not the tensor cores, set the pace; eight MMAs per barrier reverse
// that. An odd last half is zero fill.
constexpr int kMmStages = 3;
constexpr uint32_t kMmHalf = 32768u;                  // per CTA: 128 x 64 of X, 128 x 64 of W
constexpr uint32_t kMmStage = 2u * kMmHalf;
constexpr uint32_t kMmOut = 4u * 2u * 4096u;          // per epilogue warp two 32 x 64 pieces
constexpr size_t kMmSmem = 1024 + kMmStages * kMmStage + kMmOut;
constexpr int kMmGroup = 8;  // token tiles that share a sweep over the features (L2 reuse)

struct MmArgs {
  CUtensorMap tmX;  // X [M, C]: boxes of 128 x 64
  CUtensorMap tmW;  // W [N, K]: boxes of 128 x 64 (forward), 64 x 64 (dX)
  CUtensorMap tmE;  // adapter products [tiles][dmax][256][rp]: boxes of 128 x rp
  CUtensorMap tmG;  // adapter rows [n N, rp]: 128 x rp; or [n rp, K]: rp x 64
  CUtensorMap tmO;  // out [M, F]: boxes of 32 x 64
  int64_t M, F;
  int nk;           // 128-wide steps of the contraction
  int tt, ft;       // tiles of 256 tokens, of 256 features
  int rp, dmax;
  const int* cnt;   // [tt] adapters of a tile
  const int* list;  // [tt][dmax]
  int64_t grows;    // rows of tmG per adapter: N, or rp
  // the non-finite entries: whether there are any, and where they and s u are
  const int* bad;   // [nbad] flags
  int nbad;
  const int* ids;
  const uint16_t* ext;  // B [n, N, r] (entry f js + j), or A [n, r, K] (entry j js + f)
  const uint16_t* exp;
  int64_t as, js;
  int r, n;
  int wait_ext;         // E, cnt and list come from the previous grid
  unsigned long long wait_ns;
};

// What the zeroed non-finite entries of its own adapter add to D[t, f] (see ext_fix).
template <bool MN>
__device__ __noinline__ float mm_fix(const MmArgs& g, int64_t t, int64_t f) {
  if (t >= g.M || f >= g.F) return 0.f;
  const int a = g.ids[t];
  if (static_cast<unsigned>(a) >= static_cast<unsigned>(g.n)) return 0.f;
  const int64_t tile = t >> 8;
  int slot = 0;
  while (slot < __ldcg(g.cnt + tile) && __ldcg(g.list + tile * g.dmax + slot) != a) ++slot;
  const uint16_t* u = g.exp + ((tile * g.dmax + slot) * 256 + (t & 255)) * g.rp;
  const uint16_t* e = g.ext + a * g.as;
  float s = 0.f;
  for (int j = 0; j < g.r; ++j) {
    const uint16_t b = MN ? e[j * g.js + f] : e[f * g.js + j];
    if ((b & 0x7F80u) == 0x7F80u)
      s += __uint_as_float(static_cast<uint32_t>(b) << 16) * __uint_as_float(static_cast<uint32_t>(__ldcg(u + j)) << 16);
  }
  return s;
}

QNF4_DEV void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

// MN: the base and the adapters' operand are read feature-major (dX).
template <bool MN>
__global__ void __launch_bounds__(kMultiThreads, 1) k_multi_mm(const __grid_constant__ MmArgs g) {
  extern __shared__ uint8_t msm_raw[];
  __shared__ __align__(8) uint64_t full[kMmStages], empty[kMmStages], acc_full[2], acc_free[2], fin_bar;
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  uint8_t* base = msm_raw + ((1024u - (smem_u32(msm_raw) & 1023u)) & 1023u);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  if (tid == 0) {
    for (int i = 0; i < kMmStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_free[i], 8);  // the epilogue warps of both CTAs
    }
    mbar_init(&fin_bar, 1);
    s_abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&g.tmX);
    tma_prefetch_desc(&g.tmW);
    tma_prefetch_desc(&g.tmE);
    tma_prefetch_desc(&g.tmG);
    tma_prefetch_desc(&g.tmO);
  }
  if (warp == 1) {
    tmem_alloc2(&s_tmem, 512);
    tmem_relinquish2();
    tc_fence_before();
  }
  __syncthreads();
  cluster_sync();  // the pair's barriers are initialised
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  // Not waited for here: the previous grid. It is the projections' (forward) or the gradients' (dX),
  // which let this one in only after their own wait, so whatever ran before them has completed: the
  // 16-bit base and the adapters' copies, and for dX the projections too. A pair so starts when its
  // two SMs are free, under the previous grid's last CTAs, and only the forward's adapter positions
  // wait for that grid. What earlier grids wrote is read from L2 (TMA, ld.cg). (5120 x 5120, 1531
  // tokens: 91 us instead of 95; backward of 4096 x 4096, 4096 tokens: 146 instead of 156.)
  griddep_launch_dependents();

  const int tiles = g.tt * g.ft;
  const int pair = blockIdx.x >> 1, npair = gridDim.x >> 1;
  auto tile_of = [&](int u, int& t, int& f) {
    const int span = kMmGroup * g.ft;
    const int grp = u / span, rem = u - grp * span;
    const int h = g.tt - grp * kMmGroup < kMmGroup ? g.tt - grp * kMmGroup : kMmGroup;
    f = rem / h;
    t = grp * kMmGroup + rem - f * h;
  };
  if (warp == 0) {
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (int u = pair; u < tiles && ok; u += npair) {
        int t, f;
        tile_of(u, t, f);
        const int32_t tok = t * 256 + static_cast<int>(rank) * 128, feat = f * 256 + static_cast<int>(rank) * 128;
        auto slot = [&]() -> bool {
          return it < kMmStages || wait_or_abort(&empty[it % kMmStages], static_cast<uint32_t>(it / kMmStages - 1) & 1u,
                                                 g.wait_ns, &s_abort, 101, true);
        };
        for (int i = 0; i < g.nk; ++i, ++it) {
          ok = slot();
          if (!ok) break;
          const int s = it % kMmStages;
          uint8_t* st = base + s * kMmStage;
          const uint32_t bar = map_to_cta(&full[s], 0);
          if (rank == 0) mbar_expect_tx(&full[s], 2u * kMmStage);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint8_t* sh = st + h * kMmHalf;
            const int32_t c = i * 128 + h * 64;
            tma_load_2d_pair(sh, &g.tmX, bar, c, tok);
            if (!MN) {
              tma_load_2d_pair(sh + 16384, &g.tmW, bar, c, feat);
            } else {
              tma_load_2d_pair(sh + 16384, &g.tmW, bar, feat, c);
              tma_load_2d_pair(sh + 24576, &g.tmW, bar, feat + 64, c);
            }
          }
        }
        if (!ok) break;
        if (g.wait_ext) griddep_wait();
        const int nx = __ldcg(g.cnt + t);
        for (int x = 0; x < nx; ++x, ++it) {
          ok = slot();
          if (!ok) break;
          const int s = it % kMmStages, a = __ldcg(g.list + static_cast<int64_t>(t) * g.dmax + x);
          uint8_t* st = base + s * kMmStage;
          const uint32_t bar = map_to_cta(&full[s], 0);
          const uint32_t bytes = 256u * static_cast<uint32_t>(g.rp);  // of either operand
          if (rank == 0) mbar_expect_tx(&full[s], 4u * bytes);
          tma_load_2d_pair(st, &g.tmE, bar, 0, (t * g.dmax + x) * 256 + static_cast<int>(rank) * 128);
          if (!MN) {
            tma_load_2d_pair(st + 16384, &g.tmG, bar, 0, static_cast<int32_t>(a * g.grows + feat));
          } else {
            tma_load_2d_pair(st + 16384, &g.tmG, bar, feat, static_cast<int32_t>(a * g.grows));
            tma_load_2d_pair(st + 16384 + bytes / 2, &g.tmG, bar, feat + 64, static_cast<int32_t>(a * g.grows));
          }
        }
      }
      // the copies that both CTAs issued land on the leading CTA's barriers
      if (rank == 0) drain_ring(full, it, kMmStages, g.wait_ns, 102);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0) {
      const uint32_t idesc = idesc_bf16(256, 256, 0u, MN ? 1u : 0u);
      const uint32_t lay = g.rp == 16 ? 6u : (g.rp == 32 ? 4u : 2u);  // 32-, 64-, 128-byte swizzle
      const uint32_t rowb = 2u * static_cast<uint32_t>(g.rp);
      const uint32_t smb = smem_u32(base);
      const uint64_t ad0 = smem_desc(smb, 16, 1024, kLayoutSW128);
      const uint64_t bd0 = MN ? smem_desc(smb + 16384, 8192, 1024, kLayoutSW128) : smem_desc(smb + 16384, 16, 1024, kLayoutSW128);
      const uint64_t ae0 = smem_desc(smb, 16, 8u * rowb, lay);
      const uint64_t be0 = MN ? smem_desc(smb + 16384, 64u * rowb, 1024, kLayoutSW128) : smem_desc(smb + 16384, 16, 8u * rowb, lay);
      RingPos p;
      int k = 0;
      bool ok = true;
      for (int u = pair; u < tiles && ok; u += npair, ++k) {
        int t, f;
        tile_of(u, t, f);
        if (k >= 2) ok = wait_or_abort(&acc_free[k & 1], static_cast<uint32_t>(k / 2 - 1) & 1u, g.wait_ns, &s_abort, 103);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + static_cast<uint32_t>(k & 1) * 256u;
        for (int i = 0; i < g.nk; ++i, p.next(kMmStages)) {
          ok = __all_sync(0xffffffffu, wait_or_abort(&full[p.s], p.ph, g.wait_ns, &s_abort, 104));
          if (!ok) break;
          tc_fence_after();
          const uint32_t so = static_cast<uint32_t>(p.s) * (kMmStage >> 4);
          const uint64_t ad = ad0 + so, bd = bd0 + so;
          if (lane == 0) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
              const uint32_t h = (kk >> 2) * (kMmHalf >> 4), k4 = kk & 3;
              mma2_ss(d, ad + h + 2u * k4, bd + h + (MN ? (2048u >> 4) : 2u) * k4, idesc, (i > 0 || kk > 0) ? 1u : 0u);
            }
            mma2_commit(&empty[p.s]);
          }
          __syncwarp();
        }
        if (ok) {
          if (g.wait_ext) griddep_wait();
          const int nx = __ldcg(g.cnt + t);
          for (int x = 0; x < nx; ++x, p.next(kMmStages)) {
            ok = __all_sync(0xffffffffu, wait_or_abort(&full[p.s], p.ph, g.wait_ns, &s_abort, 104));
            if (!ok) break;
            tc_fence_after();
            const uint32_t so = static_cast<uint32_t>(p.s) * (kMmStage >> 4);
            const uint64_t ad = ae0 + so, bd = be0 + so;
            if (lane == 0) {
              for (int kk = 0; kk < g.rp / 16; ++kk) mma2_ss(d, ad + 2u * kk, bd + (MN ? (2048u >> 4) : 2u) * kk, idesc, 1u);
              mma2_commit(&empty[p.s]);
            }
            __syncwarp();
          }
        }
        if (lane == 0) mma2_commit(&acc_full[k & 1]);
      }
      if (lane == 0) {
        mma2_commit(&fin_bar);
        drain_wait(&fin_bar, 0, g.wait_ns, 105);
      }
    }
    __syncwarp();
  } else {
    const int q = warp & 3;
    uint8_t* out = base + kMmStages * kMmStage + q * 8192;
    int met = 0;
    for (int i = lane; i < g.nbad; i += 32) met |= __ldcg(g.bad + i);
    const bool bad = __any_sync(0xffffffffu, met != 0);
    int k = 0, piece = 0;
    for (int u = pair; u < tiles; u += npair, ++k) {
      int t, f;
      tile_of(u, t, f);
      if (!__all_sync(0xffffffffu, wait_or_abort(&acc_full[k & 1], static_cast<uint32_t>(k / 2) & 1u, g.wait_ns, &s_abort, 106, true))) break;
      tc_fence_after();
      const uint32_t d = tmem + static_cast<uint32_t>(k & 1) * 256u + (static_cast<uint32_t>(q * 32) << 16);
      const int64_t tok0 = static_cast<int64_t>(t) * 256 + rank * 128 + q * 32;
      for (int c = 0; c < 4; ++c, ++piece) {
        uint32_t v0[32], v1[32];
        tmem_ld32(d + c * 64, v0);
        tmem_ld32(d + c * 64 + 32, v1);
        tmem_wait_ld();
        if (c == 3) {  // the accumulator is read
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(map_to_cta(&acc_free[k & 1], 0));
        }
        const int64_t f0 = static_cast<int64_t>(f) * 256 + c * 64;
        if (bad) {
          if (g.wait_ext) griddep_wait();
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            v0[j] = __float_as_uint(__uint_as_float(v0[j]) + mm_fix<MN>(g, tok0 + lane, f0 + j));
            v1[j] = __float_as_uint(__uint_as_float(v1[j]) + mm_fix<MN>(g, tok0 + lane, f0 + 32 + j));
          }
        }
        // the warp's piece before last has left this buffer
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
        __syncwarp();
        uint8_t* buf = out + (piece & 1) * 4096;
        uint32_t o[32];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          o[j] = pack_bf16x2(__uint_as_float(v0[2 * j]), __uint_as_float(v0[2 * j + 1]));
          o[16 + j] = pack_bf16x2(__uint_as_float(v1[2 * j]), __uint_as_float(v1[2 * j + 1]));
        }
        store_row_sw128(buf, lane, o);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
          if (tok0 < g.M && f0 < g.F) tma_store_2d(&g.tmO, buf, static_cast<int32_t>(f0), static_cast<int32_t>(tok0));
          bulk_commit();
        }
      }
    }
    if (lane == 0) bulk_wait0();
    __syncwarp();
    tc_fence_before();
  }
  griddep_wait();  // so that this grid's end is also the end of all before it
  __syncthreads();
  if (s_abort) {
    // the other CTA's copies report to the leading one, so after a give-up nobody can wait for
    // each of them: they have all landed long before this is over (1 ms)
    const long long t0 = wait_clock();
    while (wait_clock() - t0 < ns_cycles(1000000)) {
    }
  }
  cluster_sync();  // no CTA leaves while the other may still signal it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc2(tmem, 512);
  }
}

}  // namespace qnf4
