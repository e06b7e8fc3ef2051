// Many adapters over one frozen base: every token m names its adapter a = ids[m] (an id
// outside 0 .. n - 1: none), and
//
//   h[m]  = x[m] What^T + s[a] (x[m] A[a]^T) B[a]^T
//   dX[m] = dY[m] What + s[a] (dY[m] B[a]) A[a]
//   dA[a] = sum over the tokens of a of s[a] (dY[m] B[a])^T x[m]
//   dB[a] = sum over the tokens of a of dY[m]^T s[a] (x[m] A[a]^T)
//
// ("QLoRA: Efficient Finetuning of Quantized LLMs" (Heng's Blog), opening formula, for the
// adapters of many requests or of several trainings at once). The base product and the
// adapters' second product share one accumulator (the MULTI instances of k_gemm). The
// kernels here make what those read and the adapters' gradients:
//
//   k_multi_prep  (backward) tokens sorted by adapter, B transposed
//   k_multi_proj  u = s x A^T and v = s dY B of every token's own adapter
//   k_multi_grad  dA and dB, over the sorted tokens
//
// and, for many tokens, multi_mm.cuh has the product itself.
#pragma once
#include "common.cuh"
#include "gemm.cuh"

namespace qnf4 {

constexpr int kMultiMaxAdapters = 4096;
constexpr int kMultiThreads = 192;  // TMA warp, MMA warp, four epilogue warps
constexpr int kMultiMaxStages = 8;

// Wait for a phase regardless of the abort flag, within the drain's limit.
QNF4_DEV bool drain_wait(uint64_t* bar, uint32_t parity, unsigned long long wait_ns, unsigned int site) {
  const long long t0 = wait_clock();
  while (!mbar_try_wait_long(bar, parity)) {
    if (wait_clock() - t0 > ns_cycles(drain_ns(wait_ns))) {
      set_err(site);
      return false;
    }
  }
  return true;
}
// The last copy issued into each of the ring's slots has landed (within one drain's limit).
QNF4_DEV void drain_ring(uint64_t* full, int issued, int nst, unsigned long long wait_ns, unsigned int site) {
  const int slots = issued < nst ? issued : nst;
  for (int s = 0; s < slots; ++s) {
    const int j = s + nst * ((issued - 1 - s) / nst);
    if (!drain_wait(&full[s], static_cast<uint32_t>(j / nst) & 1u, wait_ns, site)) return;
  }
}

// A position in a ring of n slots: its slot and phase, advanced without a division (one on the
// MMA warp's path costs more than the step's MMAs). The MMA warps walk their loops with all lanes,
// so that everything but the instructions of the one elected lane is uniform and stays in uniform
// registers, where the MMAs want their descriptors.
struct RingPos {
  int s = 0;
  uint32_t ph = 0;
  QNF4_DEV void next(int n) {
    if (++s == n) {
      s = 0;
      ph ^= 1u;
    }
  }
};

// v as three bf16 parts that add up to it exactly (24 bits, 8 to a part), all of v's sign and none
// of them zero unless v is: an infinity they are multiplied with then gives three infinities of one
// sign, whose sum is what the product with v would be. (Rounding to nearest gives parts of either
// sign, and zeros where fewer parts are enough.) Infinities and NaNs are their own three parts.
// (Below 2^-125 the last part may vanish.)
QNF4_DEV void bf16_parts(float v, uint16_t (&h)[3]) {
  auto head = [](float x) { return __uint_as_float(__float_as_uint(x) & 0xFFFF0000u); };  // toward zero
  if (!isfinite(v)) {
    h[0] = h[1] = h[2] = f2bf(v);
    return;
  }
  float p0 = head(v), p1 = v - p0, p2;
  if (p1 == 0.f) {  // 8 bits: halves and quarters
    p0 = 0.5f * v;
    p1 = p2 = 0.25f * v;
  } else {
    const float rest = p1;
    p1 = head(rest);
    p2 = rest - p1;
    if (p2 == 0.f) p1 = p2 = 0.5f * rest;
  }
  const float p[3] = {p0, p1, p2};
#pragma unroll
  for (int k = 0; k < 3; ++k) h[k] = static_cast<uint16_t>(__float_as_uint(p[k]) >> 16);
}

// ---------------------------------------------------------------------------
// Projections onto the tokens' own adapters
// ---------------------------------------------------------------------------
// P[m][0 .. r) = scales[a] sum_c X[m, c] F[a][0 .. r)[c]. A CTA takes 128 tokens, a batch of the
// adapters that they name (its slots) and a slice of the contraction; X and the adapters' rows come
// by TMA (128-byte swizzle), one MMA of N = slots x r16 multiplies every token with every slot, and
// the epilogue keeps each token's own slot: with a few slots per tile the extra products cost nothing
// beside the stream of X, and rows of different tokens or adapters never mix. The slices of a
// contraction are the CTAs of a cluster: each leaves its tokens' sums in shared memory and adds up a
// share of the tokens over all of them, in rank order.
//
// Bound by reading X, and with few tokens by what a CTA spends beside its steps: 2 us to find the
// adapters, 1 us of cluster barrier, 1 us to add up, 2 us to store. Measured: 4096 tokens of 8
// adapters of r = 16, C = 4096, 18 us (1.9 TB/s, X from HBM); both projections of 8192 tokens of
// r = 64, C = 5120 and 13824, 86 us (3.6 TB/s). A ring twice as long at one CTA per SM was slower
// (2048 tokens, C = 4096: the whole forward 71 us instead of 65).
//
// The tensor cores' additions truncate: a bf16 sum of C products in one accumulator comes out
// short by 1.1e-9 C relative (measured: 9.1e-6 at C = 8192), which fp32 gradients would show.
// So two accumulators take turns, kFlushSteps steps each, and the epilogue warps add them up in
// registers with rounded fp32 additions while the other one fills.
//
// X does not depend on which adapters the tile names, so its first steps are on their way while
// the CTA finds them out; X and the adapters' rows therefore have rings of their own, from either
// end of one buffer, of as many steps as fit once the number of slots is known.
//
// Outputs: the main product's operand blocks (bf16 s u, zeros in the other slots; the rounding, at
// most 2^-8 of s u, is the one-adapter layer's too, and a second bf16 part would be rp more columns of
// the product for every adapter of a tile), the tile's list of adapters, and for the gradients the values in three bf16 parts that add up to the
// fp32 value (bf16_parts), transposed to [3 r16][sorted token].
constexpr int kFlushSteps = 4;
constexpr uint32_t kProjRing = 104u * 1024u;
constexpr uint32_t kProjSmem = 1024u + kProjRing;  // two CTAs per SM
// Slots x r16 of a batch. Up to 128 columns the two accumulators fit the CTA's half of TMEM; a
// wider batch (rare with many tokens: more than two adapters of rank 64 among 128 of them) uses one
// and waits for each flush, which costs less than streaming X again for a second batch.
constexpr int kProjMaxCols = 256;
static_assert(2u * (16384u + kProjMaxCols * 128u) <= kProjRing, "two steps");
static_assert(128u * 68u * 4u + 128u * 64u * 4u <= kProjRing, "the sums reuse the rings");

struct ProjArgs {
  CUtensorMap tmX[2], tmF[2];  // X [M, C] in boxes of xrows x 64, F [n r, C] in boxes of r16 x 64
  int nsteps[2];
  int swap;                    // the second job is the longer one: its CTAs come first
  uint16_t* exp[2];            // operand blocks [tiles][cmax][tn][width], or null
  uint16_t* pt[2];             // parts [3 r16][ldp], or null
  const int* ids;
  const float* scales;
  const int* pos;              // sorted position of each token
  int64_t M, ldp;
  int n, r, r16, per, tn, dmax, cmax;
  int width;                   // columns of an operand block: 64, or the padded rank (per = 1)
  int sb, nz;                  // slots per batch; CTA z takes the batches z, z + nz, ...
  int slices;                  // cluster size
  int xrows;                   // rows of X fetched per step: 128, or fewer tokens rounded up to 16
  uint32_t tmem_cols;
  int* cnt;                    // [tiles]
  int* list;                   // [tiles][dmax]
  unsigned* ctr;               // the main product's arrival counters, cleared here
  int nctr;
  unsigned long long wait_ns;
};

__global__ void __launch_bounds__(kMultiThreads, 2) k_multi_proj(const __grid_constant__ ProjArgs g) {
  extern __shared__ uint8_t psm_raw[];
  __shared__ __align__(8) uint64_t full[kMultiMaxStages], empty[kMultiMaxStages], acc_full[2], acc_free[2], fin_bar;
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  __shared__ uint32_t s_mask[kMultiMaxAdapters / 32], s_own[kMultiMaxAdapters / 32];
  __shared__ int s_pre[kMultiMaxAdapters / 32], s_opre[kMultiMaxAdapters / 32];
  __shared__ int s_total, s_ototal;
  __shared__ int s_slot[128], s_tslot[128], s_ad[16];
  __shared__ float s_scale[128];
  uint8_t* base = psm_raw + ((1024u - (smem_u32(psm_raw) & 1023u)) & 1023u);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = g.slices > 1 ? cluster_rank() : 0u;  // == blockIdx.x
  const int jz = blockIdx.z / g.nz, job = jz ^ g.swap, z = blockIdx.z - jz * g.nz;
  const int64_t row0 = static_cast<int64_t>(blockIdx.y) * 128;
  const int64_t tile = row0 / g.tn;
  const int words = (g.n + 31) >> 5;

  if (tid == 0) {
    for (int i = 0; i < kMultiMaxStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_free[i], 128);
    }
    mbar_init(&fin_bar, 1);
    s_abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&g.tmX[job]);
    tma_prefetch_desc(&g.tmF[job]);
  }
  if (warp == 1) {
    tmem_alloc(&s_tmem, g.tmem_cols);
    tmem_relinquish();
    tc_fence_before();
  }
  for (int i = tid; i < words; i += kMultiThreads) s_mask[i] = s_own[i] = 0u;
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  griddep_wait();
  griddep_launch_dependents();

  const int r16 = g.r16;
  const uint32_t xbytes = static_cast<uint32_t>(g.xrows) * 128u;
  // the slices take the steps in turn: a cluster's CTAs read neighbouring columns of the same rows
  // at about the same time, so a DRAM page opened for a row serves all of them
  const int k0 = static_cast<int>(rank);
  const int steps = g.nsteps[job] > k0 ? (g.nsteps[job] - k0 + g.slices - 1) / g.slices : 0;
  // X of the first steps of the CTA's first batch (there may be none: then they are waited for
  // at the end)
  const uint32_t fmost = static_cast<uint32_t>(g.sb * r16) * 128u;
  const int least = static_cast<int>(kProjRing / (xbytes + fmost)) < kMultiMaxStages
                        ? static_cast<int>(kProjRing / (xbytes + fmost)) : kMultiMaxStages;
  const int ahead = steps < least ? steps : least;
  if (warp == 0 && lane == 0) {
    for (int i = 0; i < ahead; ++i) {
      mbar_expect_more(&full[i], xbytes);
      tma_load_2d(base + i * xbytes, &g.tmX[job], &full[i], (k0 + i * g.slices) * 64, static_cast<int32_t>(row0));
    }
  }

  // the adapters of the column tile as a bit set, in which an adapter's rank is its place in the
  // main product's operand, and those of the CTA's own tokens, whose ranks are the slots here
  const int64_t tok0 = tile * g.tn;
  const int ntok = static_cast<int>(g.M - tok0 < g.tn ? g.M - tok0 : g.tn);
  for (int i = tid; i < ntok; i += kMultiThreads) {
    const uint32_t a = static_cast<uint32_t>(g.ids[tok0 + i]);
    if (a < static_cast<uint32_t>(g.n)) {
      atomicOr(&s_mask[a >> 5], 1u << (a & 31));
      if (static_cast<uint64_t>(tok0 + i - row0) < 128u) atomicOr(&s_own[a >> 5], 1u << (a & 31));
    }
  }
  if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0)
    for (int i = tid; i < g.nctr; i += kMultiThreads) g.ctr[i] = 0u;
  __syncthreads();
  if (warp == 0 || warp == 2) {
    const uint32_t* mask = warp == 0 ? s_mask : s_own;
    int* pre = warp == 0 ? s_pre : s_opre;
    int before = 0;
    for (int w0 = 0; w0 < words; w0 += 32) {
      const int c = w0 + lane < words ? __popc(mask[w0 + lane]) : 0;
      int inc = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      if (w0 + lane < words) pre[w0 + lane] = before + inc - c;
      before += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (lane == 0) (warp == 0 ? s_total : s_ototal) = before;
  }
  __syncthreads();
  const int ttotal = s_total, total = s_ototal;  // of the tile, of the CTA's tokens
  const bool lists = z == 0 && job == 0 && blockIdx.x == 0 && row0 == tok0;
  if (lists) {
    if (tid == 0) g.cnt[tile] = ttotal;
    for (int w = tid; w < words; w += kMultiThreads) {
      int s = s_pre[w];
      for (uint32_t m = s_mask[w]; m; m &= m - 1, ++s)
        if (in_bounds(s < g.dmax, 91)) g.list[tile * g.dmax + s] = w * 32 + __ffs(m) - 1;
    }
  }
  if (tid < 128) {
    const int64_t m = row0 + tid;
    const uint32_t a = m < g.M ? static_cast<uint32_t>(g.ids[m]) : 0xffffffffu;
    const bool live = a < static_cast<uint32_t>(g.n);
    const uint32_t below = (1u << (a & 31)) - 1u;
    s_slot[tid] = live ? s_opre[a >> 5] + __popc(s_own[a >> 5] & below) : -1;
    s_tslot[tid] = live ? s_pre[a >> 5] + __popc(s_mask[a >> 5] & below) : -1;
    s_scale[tid] = live ? g.scales[a] : 0.f;
  }

  // the rings are cut for this CTA's first batch, its largest
  const uint32_t fslot = static_cast<uint32_t>(r16) * 128u;
  const int nb0 = total - z * g.sb < g.sb ? total - z * g.sb : g.sb;
  const uint32_t fstage = static_cast<uint32_t>(nb0 > 0 ? nb0 : 1) * fslot;
  const int fit = static_cast<int>(kProjRing / (xbytes + fstage));
  const int nst = fit < kMultiMaxStages ? fit : kMultiMaxStages;
  uint8_t* fring = base + kProjRing - static_cast<uint32_t>(nst) * fstage;
  int it = 0;  // steps of earlier batches
  RingPos pos;               // this warp's place in the rings
  int issued = 0;            // steps whose copies warp 0 has issued
  uint32_t turn_n = 0;       // accumulator turns so far

  for (int first = z * g.sb; first < total; first += g.nz * g.sb) {  // alike in the whole cluster
    const int nb = total - first < g.sb ? total - first : g.sb;
    const bool two = 2 * nb * r16 <= static_cast<int>(g.tmem_cols);  // accumulators
    for (int w = tid; w < words; w += kMultiThreads) {
      int s = s_opre[w];
      for (uint32_t m = s_own[w]; m; m &= m - 1, ++s)
        if (s >= first && s < first + nb) s_ad[s - first] = w * 32 + __ffs(m) - 1;
    }
    __syncthreads();
    if (warp == 0) {
      if (!__shfl_sync(0xffffffffu, s_abort, 0)) {
        bool all = true;
        for (int i = it; i < it + steps && all; ++i, pos.next(nst)) {
          const int s = pos.s;
          if (i >= nst) {  // every lane waits, so all of them leave together
            all = __all_sync(0xffffffffu, wait_or_abort(&empty[s], pos.ph ^ 1u, g.wait_ns, &s_abort, 91, true));
            if (!all) break;
          }
          const int32_t c = (k0 + (i - it) * g.slices) * 64;
          const uint32_t fbytes = static_cast<uint32_t>(nb) * fslot;
          if (lane == 0) {
            if (i < ahead) {  // X is on its way
              mbar_expect_tx(&full[s], fbytes);
            } else {
              mbar_expect_tx(&full[s], xbytes + fbytes);
              tma_load_2d(base + s * xbytes, &g.tmX[job], &full[s], c, static_cast<int32_t>(row0));
            }
          }
          __syncwarp();
          if (lane < nb)
            tma_load_2d(fring + static_cast<uint32_t>(s) * fstage + lane * fslot, &g.tmF[job], &full[s], c, s_ad[lane] * g.r);
          ++issued;
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      if (!__shfl_sync(0xffffffffu, s_abort, 0)) {
        const uint32_t idesc = idesc_bf16(128, static_cast<uint32_t>(nb * r16), 0u, 0u);
        const uint64_t ad0 = smem_desc(smem_u32(base), 16, 1024, kLayoutSW128);
        const uint64_t bd0 = smem_desc(smem_u32(fring), 16, 1024, kLayoutSW128);
        bool ok = true;
        uint32_t b = turn_n;
        for (int i = 0; i < steps && ok; ++i, pos.next(nst)) {
          const int s = pos.s, turn = i % kFlushSteps;
          if (turn == 0 && two && b >= 2)
            ok = wait_or_abort(&acc_free[b & 1], (b / 2 - 1) & 1u, g.wait_ns, &s_abort, 90);
          if (turn == 0 && !two && b >= 1)
            ok = wait_or_abort(&acc_free[(b - 1) & 1], ((b - 1) / 2) & 1u, g.wait_ns, &s_abort, 90);
          ok = ok && wait_or_abort(&full[s], pos.ph, g.wait_ns, &s_abort, 93);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          // (rows past xrows are whatever lies there: their products are not read)
          const uint64_t ad = ad0 + ((static_cast<uint32_t>(s) * xbytes) >> 4);
          const uint64_t bd = bd0 + ((static_cast<uint32_t>(s) * fstage) >> 4);
          const uint32_t d = tmem + (two ? (b & 1u) * (g.tmem_cols / 2) : 0u);
          const bool last = turn == kFlushSteps - 1 || i == steps - 1;
          if (lane == 0) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) mma_ss(d, ad + 2u * kk, bd + 2u * kk, idesc, (turn > 0 || kk > 0) ? 1u : 0u);
            mma_commit(&empty[s]);
            if (last) mma_commit(&acc_full[b & 1]);
          }
          __syncwarp();
          b += last;
        }
      }
      __syncwarp();
    } else {
      // add up each token's own slot, then leave the sums in shared memory (the ring is idle
      // once the batch's MMAs are done)
      const int q = warp & 3, row = q * 32 + lane;
      const int mine = s_slot[row] - first;
      float sum[64];
#pragma unroll
      for (int c = 0; c < 64; ++c) sum[c] = 0.f;
      const int turns = (steps + kFlushSteps - 1) / kFlushSteps;
      bool ok = !__shfl_sync(0xffffffffu, s_abort, 0);
      for (int t = 0; t < turns && ok; ++t) {
        const uint32_t b = turn_n + t;
        ok = __all_sync(0xffffffffu, wait_or_abort(&acc_full[b & 1], (b / 2) & 1u, g.wait_ns, &s_abort, 94));
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + (two ? (b & 1u) * (g.tmem_cols / 2) : 0u) + (static_cast<uint32_t>(q * 32) << 16);
        for (int sl = 0; sl < nb; ++sl) {
          if (!__any_sync(0xffffffffu, mine == sl)) continue;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if (c * 16 < r16) {
              uint32_t v[16];
              tmem_ld16(d + sl * r16 + c * 16, v);
              tmem_wait_ld();
              if (mine == sl) {
#pragma unroll
                for (int j = 0; j < 16; ++j) sum[c * 16 + j] += __uint_as_float(v[j]);
              }
            }
          }
        }
        tc_fence_before();
        mbar_arrive(&acc_free[b & 1]);
      }
      if (ok) {
        float* part = reinterpret_cast<float*>(base) + row * (r16 + 4);  // 16-byte rows, no bank conflicts
#pragma unroll
        for (int c = 0; c < 64; c += 4)
          if (c < r16) *reinterpret_cast<float4*>(part + c) = make_float4(sum[c], sum[c + 1], sum[c + 2], sum[c + 3]);
      }
    }
    it += steps;
    turn_n += (steps + kFlushSteps - 1) / kFlushSteps;
    __syncthreads();
    if (g.slices > 1) cluster_sync();
    // this CTA's share of the tokens, summed over the slices
    const int share = 128 / g.slices, r0 = static_cast<int>(rank) * share;
    float* fin = reinterpret_cast<float*>(base + 128 * 68 * 4);
    const uint32_t part0 = smem_u32(base);
    const int q4 = r16 / 4;
    for (int i = tid; i < share * q4; i += kMultiThreads) {
      const int row = r0 + i / q4, j = 4 * (i % q4);
      const int mine = s_slot[row] - first;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (mine >= 0 && mine < nb) {
        const uint32_t at = part0 + static_cast<uint32_t>(row * (r16 + 4) + j) * 4u;
        float4 p[8];
#pragma unroll
        for (int c = 0; c < 8; ++c)
          if (c < g.slices) p[c] = ld_cluster_f4(at, static_cast<uint32_t>(c));
#pragma unroll
        for (int c = 0; c < 8; ++c)
          if (c < g.slices) {
            v.x += p[c].x;
            v.y += p[c].y;
            v.z += p[c].z;
            v.w += p[c].w;
          }
        const float sc = s_scale[row];
        v.x = j < g.r ? v.x * sc : 0.f;
        v.y = j + 1 < g.r ? v.y * sc : 0.f;
        v.z = j + 2 < g.r ? v.z * sc : 0.f;
        v.w = j + 3 < g.r ? v.w * sc : 0.f;
      }
      *reinterpret_cast<float4*>(fin + 4 * i) = v;
    }
    __syncthreads();
    if (g.slices > 1) cluster_arrive();  // this CTA has read the others' sums
    const bool ok = !s_abort;
    if (ok && g.exp[job]) {
      // the tokens of this batch, and with the first batch those without an adapter: their rows
      // of every block of the tile, zeros but in their own adapter's place
      const int nch = (ttotal + g.per - 1) / g.per;
      const int w8 = g.width / 8;
      for (int i = tid; i < share * nch * w8; i += kMultiThreads) {
        const int q8 = i % w8, row = i / w8 / nch, c = i / w8 - row * nch;
        const int64_t m = row0 + r0 + row;
        const int mine = s_slot[r0 + row] - first, ts = s_tslot[r0 + row];
        if (m >= g.M || !(ts < 0 ? first == 0 : mine >= 0 && mine < nb)) continue;
        const int p = 8 * q8 / r16, j = 8 * q8 - p * r16;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (p < g.per && ts == c * g.per + p) {
          const float* f = fin + row * r16 + j;
          v = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                         pack_bf16x2(f[6], f[7]));
        }
        *reinterpret_cast<uint4*>(g.exp[job] + (((tile * g.cmax + c) * g.tn + (m - tok0)) * g.width + 8 * q8)) = v;
      }
    }
    if (ok && g.pt[job]) {
      for (int i = tid; i < share * r16; i += kMultiThreads) {
        const int j = i / share, row = i - j * share;
        const int mine = s_slot[r0 + row] - first;
        if (mine < 0 || mine >= nb) continue;
        uint16_t h[3];
        bf16_parts(fin[row * r16 + j], h);
        int64_t at = j * g.ldp + g.pos[row0 + r0 + row];
#pragma unroll
        for (int k = 0; k < 3; ++k) {
          g.pt[job][at] = h[k];
          at += static_cast<int64_t>(r16) * g.ldp;
        }
      }
    }
    // the others have read this CTA's sums: the next batch's copies write there
    fence_proxy_async();
    if (g.slices > 1) cluster_wait();
    __syncthreads();
  }
  // Every copy and MMA of this CTA completes before it leaves (they have, unless it gave up or
  // had no batch: steps of X fetched ahead whose adapter rows were not are completed here).
  if (warp == 0 && lane == 0) {
    for (int i = issued; i < ahead; ++i) mbar_arrive(&full[i]);
    drain_ring(full, issued < ahead ? ahead : issued, nst, g.wait_ns, 92);
  }
  if (warp == 1 && lane == 0) {
    mma_commit(&fin_bar);
    drain_wait(&fin_bar, 0, g.wait_ns, 95);
  }
  if (total == 0 && ttotal > 0 && z == 0 && rank == 0 && g.exp[job]) {
    // none of these tokens has an adapter, but others of their tile do
    const int nch = (ttotal + g.per - 1) / g.per, w8 = g.width / 8;
    for (int i = tid; i < 128 * nch * w8; i += kMultiThreads) {
      const int q8 = i % w8, row = i / w8 / nch, c = i / w8 - row * nch;
      if (row0 + row < g.M)
        *reinterpret_cast<uint4*>(g.exp[job] + (((tile * g.cmax + c) * g.tn + (row0 + row - tok0)) * g.width + 8 * q8)) =
            make_uint4(0u, 0u, 0u, 0u);
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, g.tmem_cols);
  }
}

// ---------------------------------------------------------------------------
// Backward preparation
// ---------------------------------------------------------------------------
// CTA 0 sorts the tokens by adapter (stable, so equal calls sum in equal order; every warp takes a
// run of tokens and, where the table of all warps' positions fits, walks it without a barrier, else
// the warps take 32 tokens each in turn): adapter a's tokens take the positions off[a] .. off[a] +
// count, each adapter starting on a multiple of 64, with the adapter's last token repeated up to its
// end (k_multi_grad fetches those rows and clears them).
// It cuts every adapter's 64-token steps into slices of at most `lsteps` (one empty slice for
// an adapter without tokens), the work list of k_multi_grad. The other CTAs transpose B
// [n, N, r] into BT [n, r, N], clear the projections' parts and the counters. Bound by the latency
// of CTA 0's passes over the ids: 6 us for 4096 tokens of 4 adapters, 10 us for 8192 of 8 (one CTA
// keeps the sort free of a grid-wide barrier; by many tokens it runs under the stage kernel's end).
// Up to 4096 tokens only named adapters are transposed, at a pass over the ids for each 64 rows of each
// adapter: nothing for a few, but with 4096 adapters of r = 16 and N = 11008, 8 of them named by 64
// tokens, most of a backward call of 4.2 ms (writing dB's zeros takes 0.45).
struct GradSlice {
  int a, p0, steps;
  int count;   // slices of this adapter
  int index;   // this one among them
  int group;   // ordinal among the adapters of more than one slice, for counters
  int part0;   // first of the adapter's slices among those of such adapters, for partials
  int tail;    // tokens of the last step, the rest of whose 64 positions is padding
};

struct PrepArgs {
  const int* ids;
  int64_t M;
  int n, r, lsteps, slmax;
  int64_t ldp;
  int* pos;          // [M]
  int* perm;         // [ldp]
  GradSlice* slices; // [slmax]
  int* nslices;      // [1]
  const uint16_t* B;
  uint16_t* BT;
  int64_t N;
  uint4* clear;      // 16-byte words to clear
  int64_t nclear;
  int lazy;          // the previous grid's results are not read here: wait for it at the end
};

constexpr int kPrepThreads = 1024;
constexpr int kPrepTable = 256;  // adapters of the per-warp position table (34 KB)

__global__ void __launch_bounds__(kPrepThreads) k_multi_prep(const __grid_constant__ PrepArgs g) {
  extern __shared__ int prep_sm[];
  __shared__ int s_warp[4][32];
  __shared__ int s_sum[4];
  if (!g.lazy) griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (blockIdx.x == 0) {
    int* cnt = prep_sm;           // [n] counts
    int* off = prep_sm + g.n;     // [n] next position of each adapter
    for (int a = tid; a < g.n; a += kPrepThreads) cnt[a] = 0;
    if (tid < 4) s_sum[tid] = 0;
    __syncthreads();
    for (int64_t m = tid; m < g.M; m += kPrepThreads) {
      const uint32_t a = static_cast<uint32_t>(g.ids[m]);
      if (a < static_cast<uint32_t>(g.n)) atomicAdd(&cnt[a], 1);
    }
    __syncthreads();
    // exclusive sums over the adapters of: 64-token steps, slices, adapters of several
    // slices, and their slices
    for (int a0 = 0; a0 < g.n; a0 += kPrepThreads) {
      const int a = a0 + tid;
      const int c = a < g.n ? cnt[a] : 0;
      const int steps = (c + 63) >> 6;
      const int sl = a < g.n ? (steps ? (steps + g.lsteps - 1) / g.lsteps : 1) : 0;
      const int own[4] = {steps, sl, sl > 1 ? 1 : 0, sl > 1 ? sl : 0};
      int inc[4];
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        inc[v] = own[v];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int t = __shfl_up_sync(0xffffffffu, inc[v], o);
          if (lane >= o) inc[v] += t;
        }
        if (lane == 31) s_warp[v][warp] = inc[v];
      }
      __syncthreads();
      if (warp < 4) {
        const int own_w = s_warp[warp][lane];
        int w = own_w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int t = __shfl_up_sync(0xffffffffu, w, o);
          if (lane >= o) w += t;
        }
        const int before = s_sum[warp];
        __syncwarp();
        s_warp[warp][lane] = before + w - own_w;
        if (lane == 31) s_sum[warp] = before + w;
      }
      __syncthreads();
      int ex[4];
#pragma unroll
      for (int v = 0; v < 4; ++v) ex[v] = s_warp[v][warp] + inc[v] - own[v];
      if (a < g.n) {
        off[a] = ex[0] * 64;
        for (int i = 0; i < sl; ++i) {
          const int st = steps - i * g.lsteps;
          if (in_bounds(ex[1] + i < g.slmax, 92))
            g.slices[ex[1] + i] = GradSlice{a, (ex[0] + i * g.lsteps) * 64, st < g.lsteps ? st : g.lsteps, sl, i,
                                            ex[2], ex[3], i == sl - 1 && (c & 63) ? c & 63 : 64};
        }
      }
      __syncthreads();
    }
    if (tid == 0) *g.nslices = s_sum[1];
    if (g.n <= kPrepTable) {
      // a run of tokens per warp: its counts, then its first position in every adapter
      int* own = prep_sm + 2 * g.n;  // [32][n]
      for (int i = tid; i < 32 * g.n; i += kPrepThreads) own[i] = 0;
      const int64_t run = (((g.M + 31) / 32) + 31) / 32 * 32;
      const int64_t m0 = warp * run, m1 = m0 + run < g.M ? m0 + run : g.M;
      __syncthreads();
      for (int64_t m = m0 + lane; m < m1; m += 32) {
        const uint32_t id = static_cast<uint32_t>(g.ids[m]);
        if (id < static_cast<uint32_t>(g.n)) atomicAdd(&own[warp * g.n + id], 1);
      }
      __syncthreads();
      for (int a = tid; a < g.n; a += kPrepThreads) {
        int p = off[a];
        for (int w = 0; w < 32; ++w) {
          const int c = own[w * g.n + a];
          own[w * g.n + a] = p;
          p += c;
        }
        off[a] = p;
      }
      __syncthreads();
      for (int64_t mb = m0; mb < m1; mb += 32) {
        const int64_t m = mb + lane;
        const uint32_t id = m < m1 ? static_cast<uint32_t>(g.ids[m]) : 0xffffffffu;
        const bool live = id < static_cast<uint32_t>(g.n);
        const uint32_t same = __match_any_sync(0xffffffffu, live ? static_cast<int>(id) : -1);
        const int before = __popc(same & ((1u << lane) - 1u));
        int p = -1;
        if (live) {
          p = own[warp * g.n + id] + before;
          if (in_bounds(p < g.ldp, 93)) g.perm[p] = static_cast<int>(m);
        }
        if (m < m1) g.pos[m] = p;
        __syncwarp();
        if (live && before == 0) own[warp * g.n + id] += __popc(same);
        __syncwarp();
      }
    } else {
      for (int64_t m0 = 0; m0 < g.M; m0 += kPrepThreads) {
        const int64_t m = m0 + tid;
        const uint32_t id = m < g.M ? static_cast<uint32_t>(g.ids[m]) : 0xffffffffu;
        const bool live = id < static_cast<uint32_t>(g.n);
        const uint32_t same = __match_any_sync(0xffffffffu, live ? static_cast<int>(id) : -1);
        const int before = __popc(same & ((1u << lane) - 1u));
        const int64_t rest = g.M - m0;
        const int turns = static_cast<int>(rest < kPrepThreads ? (rest + 31) / 32 : 32);
        int p = -1;
        for (int w = 0; w < turns; ++w) {
          if (w == warp) {
            if (live) p = off[id] + before;
            __syncwarp();
            if (live && before == 0) off[id] += __popc(same);
          }
          __syncthreads();
        }
        if (live && in_bounds(p < g.ldp, 93)) g.perm[p] = static_cast<int>(m);
        if (m < g.M) g.pos[m] = p;
      }
    }
    // the rest of each adapter's last step: its last token again
    __threadfence_block();
    __syncthreads();
    for (int a = warp; a < g.n; a += kPrepThreads / 32) {
      const int c = cnt[a];
      if (c == 0) continue;
      const int end = off[a], stop = end - c + ((c + 63) & ~63);
      const int last = g.perm[end - 1];
      for (int p = end + lane; p < stop; p += 32)
        if (in_bounds(p < g.ldp, 94)) g.perm[p] = last;
    }
    if (g.lazy) griddep_wait();
    return;
  }
  const int64_t nt = (g.N + 63) / 64;
  uint16_t* sm = reinterpret_cast<uint16_t*>(prep_sm);  // [64][r + 1]
  for (int64_t u = blockIdx.x - 1; u < nt * g.n; u += gridDim.x - 1) {
    const int64_t a = u / nt, n0 = (u - a * nt) * 64;
    if (g.M <= 4 * kPrepThreads) {  // few tokens: is there one that names this adapter?
      bool named = false;
      for (int64_t m = tid; m < g.M; m += kPrepThreads) named |= g.ids[m] == static_cast<int>(a);
      if (!__syncthreads_or(named)) continue;
    }
    const int rows = static_cast<int>(g.N - n0 < 64 ? g.N - n0 : 64);
    const uint16_t* src = g.B + (a * g.N + n0) * g.r;
    for (int i = tid; i < rows * g.r; i += kPrepThreads) sm[(i / g.r) * (g.r + 1) + i % g.r] = src[i];
    __syncthreads();
    for (int i = tid; i < 64 * g.r; i += kPrepThreads) {
      const int j = i >> 6, c = i & 63;
      if (c < rows) g.BT[(a * g.r + j) * g.N + n0 + c] = sm[c * (g.r + 1) + j];
    }
    __syncthreads();
  }
  for (int64_t i = static_cast<int64_t>(blockIdx.x - 1) * kPrepThreads + tid; i < g.nclear;
       i += static_cast<int64_t>(gridDim.x - 1) * kPrepThreads)
    g.clear[i] = make_uint4(0u, 0u, 0u, 0u);
  if (g.lazy) griddep_wait();
}

// ---------------------------------------------------------------------------
// The adapters' gradients
// ---------------------------------------------------------------------------
// G[a][f][j] = sum over the sorted tokens p of adapter a of X[perm[p], f] P[p][j], with X = x
// and P = v for dA, X = dY and P = u for dB, both in one launch. A CTA takes 128 features and
// the slices blockIdx.y, blockIdx.y + gridDim.y, ... of the adapters' tokens, with the loads of the
// next slice on their way while one is written out (many adapters of a few tokens each make short
// slices, and a CTA for each spent its time on setting up); 64 tokens a step: the TMA warp gathers
// their rows (four rows per instruction, one instruction per lane) into an MN-major tile, or, where
// they follow one another as the tokens of a request or sample do, copies them in two boxes; the
// three parts of P come as a K-major tile of 3 r16 rows, and two MMAs multiply X with them: the first
// two parts into an accumulator each, the third, 2^-8 of the second, on top of the second's. As in
// the projections two pairs of accumulators take turns of kFlushSteps steps and are added up in registers.
// The work is bound by reading X once (it is often still in L2 from the projections); tokens
// of other adapters are never read, so neither their number nor their values matter. An
// adapter of several slices goes through fp32 partial tiles that the last of its CTAs to
// finish adds up in slice order. Measured: 4096 tokens of 8 adapters of r = 16, 4096 and 11008
// features, 36 us (3.6 TB/s); 8192 tokens of r = 64, 13824 and 5120 features, 79 us (3.9 TB/s).
struct MultiGradArgs {
  CUtensorMap tmX[2];  // x [M, K], dY [M, N]: boxes of 1 x 64, for gathers
  CUtensorMap tmR[2];  // the same in boxes of 64 x 64
  CUtensorMap tmP[2];  // parts of v, u: [3 r16][ldp] in boxes of 3 r16 x 64
  float* out[2];
  int64_t F[2];
  int64_t as[2], js[2], fs[2];  // element strides of out for adapter, row j, feature
  int ft[2];                    // feature tiles
  int r, r16;
  uint32_t ring_bytes, tmem_cols;
  const GradSlice* slices;
  const int* nslices;
  const int* perm;
  float* part;                  // [slices of several][ft tiles][r16][128]
  unsigned* ctr;                // [groups][ft tiles], zero on entry
  int64_t part_elems, ctr_elems;
  unsigned long long wait_ns;
};

__global__ void __launch_bounds__(kMultiThreads, 2) k_multi_grad(const __grid_constant__ MultiGradArgs g) {
  extern __shared__ uint8_t gsm_raw[];
  __shared__ __align__(8) uint64_t full[kMultiMaxStages], empty[kMultiMaxStages], acc_full[2], acc_free[2], fin_bar;
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  __shared__ volatile int s_last;
  uint8_t* base = gsm_raw + ((1024u - (smem_u32(gsm_raw) & 1023u)) & 1023u);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int job = static_cast<int>(blockIdx.x) < g.ft[0] ? 0 : 1;
  const int64_t f0 = static_cast<int64_t>(blockIdx.x - (job ? g.ft[0] : 0)) * 128;
  if (tid == 0) {
    for (int i = 0; i < kMultiMaxStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_free[i], 128);
    }
    mbar_init(&fin_bar, 1);
    s_abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&g.tmX[job]);
    tma_prefetch_desc(&g.tmR[job]);
    tma_prefetch_desc(&g.tmP[job]);
  }
  if (warp == 1) {
    tmem_alloc(&s_tmem, g.tmem_cols);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  griddep_wait();
  griddep_launch_dependents();
  const int nsl = *g.nslices;
  const int r16 = g.r16;
  const uint32_t stage = 16384u + static_cast<uint32_t>(3 * r16) * 128u;
  const int fit = static_cast<int>(g.ring_bytes / stage);
  const int nst = fit < kMultiMaxStages ? fit : kMultiMaxStages;
  if (warp == 0) {
    int issued = 0;
    bool all = true;
    RingPos p;  // (the phase of a slot's previous use is the opposite one)
    for (int y = blockIdx.y; y < nsl && all; y += gridDim.y) {
      const GradSlice sl = g.slices[y];
      for (int i = 0; i < sl.steps && all; ++i, p.next(nst)) {
        const int s = p.s;
        const int4 rows = *reinterpret_cast<const int4*>(g.perm + sl.p0 + i * 64 + (lane & 15) * 4);
        const int row0 = __shfl_sync(0xffffffffu, rows.x, 0), mine0 = row0 + (lane & 15) * 4;
        const bool run = __all_sync(0xffffffffu, rows.x == mine0 && rows.y == mine0 + 1 && rows.z == mine0 + 2 && rows.w == mine0 + 3);
        const bool ok = issued < nst || wait_or_abort(&empty[s], p.ph ^ 1u, g.wait_ns, &s_abort, 96, true);
        all = __all_sync(0xffffffffu, ok);
        if (!all) break;
        uint8_t* st = base + static_cast<uint32_t>(s) * stage;
        // features past the last one: their D rows are not stored, so nothing is fetched
        const bool both = f0 + 64 < g.F[job];
        if (lane == 0) {
          mbar_expect_tx(&full[s], both ? stage : stage - 8192u);
          tma_load_2d(st + 16384, &g.tmP[job], &full[s], sl.p0 + i * 64, 0);
        }
        __syncwarp();
        const int half = lane >> 4;
        if (run) {
          if ((lane & 15) == 0 && (half == 0 || both))
            tma_load_2d(st + half * 8192, &g.tmR[job], &full[s], static_cast<int32_t>(f0) + half * 64, row0);
        } else if (half == 0 || both)
          tma_gather4(st + half * 8192 + (lane & 15) * 512, &g.tmX[job], &full[s],
                      static_cast<int32_t>(f0) + half * 64, rows);
        ++issued;
      }
    }
    if (lane == 0) drain_ring(full, issued, nst, g.wait_ns, 97);
    __syncwarp();
  } else if (warp == 1) {
    const uint32_t idesc = idesc_bf16(128, static_cast<uint32_t>(r16), 1u, 0u);
    const uint32_t idesc2 = idesc_bf16(128, static_cast<uint32_t>(2 * r16), 1u, 0u);
    const uint32_t pstep = (static_cast<uint32_t>(r16) * 128u) >> 4;  // descriptor units per part
    const uint64_t ad0 = smem_desc(smem_u32(base), 8192, 1024, kLayoutSW128);
    const uint64_t bd0 = smem_desc(smem_u32(base) + 16384, 16, 1024, kLayoutSW128);
    bool ok = true;
    uint32_t b = 0;
    RingPos p;
    for (int y = blockIdx.y; y < nsl && ok; y += gridDim.y) {
      const int steps = g.slices[y].steps, tail = g.slices[y].tail;
      for (int i = 0; i < steps && ok; ++i, p.next(nst)) {
        const int s = p.s, turn = i % kFlushSteps;
        if (turn == 0 && b >= 2)
          ok = wait_or_abort(&acc_free[b & 1], (b / 2 - 1) & 1u, g.wait_ns, &s_abort, 89);
        ok = ok && wait_or_abort(&full[s], p.ph, g.wait_ns, &s_abort, 98);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (i == steps - 1 && tail < 64) {
          // the rows past the adapter's tokens: their P is zero, but zero times an infinity is NaN
          // (a row is 128 bytes of either half, whatever the swizzle)
          uint8_t* rest = base + static_cast<uint32_t>(s) * stage + static_cast<uint32_t>(tail) * 128u;
          for (int c = lane; c < (64 - tail) * 8; c += 32) {
            reinterpret_cast<uint4*>(rest)[c] = make_uint4(0u, 0u, 0u, 0u);
            reinterpret_cast<uint4*>(rest + 8192)[c] = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async();
          __syncwarp();
        }
        tc_fence_after();
        const uint32_t so = (static_cast<uint32_t>(s) * stage) >> 4;
        const uint64_t ad = ad0 + so, bd = bd0 + so;
        const uint32_t d = tmem + (b & 1u) * (g.tmem_cols / 2);
        const bool last = turn == kFlushSteps - 1 || i == steps - 1;
        if (lane == 0) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint64_t a = ad + (2048u >> 4) * kk;
            const uint32_t acc = (turn > 0 || kk > 0) ? 1u : 0u;
            mma_ss(d, a, bd + 2u * kk, idesc2, acc);
            mma_ss(d + r16, a, bd + 2 * pstep + 2u * kk, idesc, 1u);
          }
          mma_commit(&empty[s]);
          if (last) mma_commit(&acc_full[b & 1]);
        }
        __syncwarp();
        b += last;
      }
    }
    if (lane == 0) {
      mma_commit(&fin_bar);
      drain_wait(&fin_bar, 0, g.wait_ns, 100);
    }
    __syncwarp();
  } else {
    const int q = warp & 3, row = q * 32 + lane;
    const int64_t f = f0 + row;
    const int64_t js = g.js[job];
    const bool in = f < g.F[job];
    const int64_t tiles = g.ft[0] + g.ft[1];
    const int64_t tsz = static_cast<int64_t>(r16) * 128;
    uint32_t b = 0;
    for (int y = blockIdx.y; y < nsl; y += gridDim.y) {
      const GradSlice sl = g.slices[y];
      float sum[64];
#pragma unroll
      for (int c = 0; c < 64; ++c) sum[c] = 0.f;
      const int turns = (sl.steps + kFlushSteps - 1) / kFlushSteps;
      for (int k = 0; k < turns; ++k, ++b) {
        if (!__all_sync(0xffffffffu, wait_or_abort(&acc_full[b & 1], (b / 2) & 1u, g.wait_ns, &s_abort, 99))) break;
        tc_fence_after();
        const uint32_t d = tmem + (b & 1u) * (g.tmem_cols / 2) + (static_cast<uint32_t>(q * 32) << 16);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (c * 16 < r16) {
            uint32_t hi[16], lo[16];
            tmem_ld16(d + c * 16, hi);
            tmem_ld16(d + r16 + c * 16, lo);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j) sum[c * 16 + j] += __uint_as_float(hi[j]) + __uint_as_float(lo[j]);
          }
        }
        tc_fence_before();
        mbar_arrive(&acc_free[b & 1]);
      }
      // the four warps go on or give up together
      named_sync(1, 128);
      if (tid == 64) s_last = s_abort ? 0 : 1;
      named_sync(1, 128);
      const bool ok = s_last != 0;
      named_sync(1, 128);
      if (!ok) break;
      float* out = g.out[job] + sl.a * g.as[job] + f * g.fs[job];
      bool write = true;
      if (sl.count > 1) {
        const int64_t at = (sl.part0 + sl.index) * tiles + blockIdx.x;
        float* mine = g.part + at * tsz + row;
        if (in_bounds((at + 1) * tsz <= g.part_elems, 95)) {
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (c < r16) __stcg(mine + c * 128, sum[c]);
        }
        __threadfence();
        named_sync(1, 128);
        if (tid == 64) {
          const int64_t c = sl.group * tiles + blockIdx.x;
          s_last = in_bounds(c < g.ctr_elems, 96) && atomicAdd(g.ctr + c, 1u) == static_cast<unsigned>(sl.count - 1);
        }
        named_sync(1, 128);
        write = s_last != 0;
        if (write) {
          __threadfence();
          const float* all = g.part + (sl.part0 * tiles + blockIdx.x) * tsz + row;
#pragma unroll
          for (int c = 0; c < 64; ++c) sum[c] = 0.f;
          for (int k = 0; k < sl.count; ++k) {
#pragma unroll
            for (int c = 0; c < 64; ++c)
              if (c < r16) sum[c] += __ldcg(all + k * tiles * tsz + c * 128);
          }
        }
        named_sync(1, 128);  // s_last is free again
      }
      if (write && in) {
        if (js == 1 && (g.r & 3) == 0) {
#pragma unroll
          for (int c = 0; c < 64; c += 4)
            if (c < g.r) *reinterpret_cast<float4*>(out + c) = make_float4(sum[c], sum[c + 1], sum[c + 2], sum[c + 3]);
        } else {
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (c < g.r) out[c * js] = sum[c];
        }
      }
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, g.tmem_cols);
  }
}

}  // namespace qnf4
