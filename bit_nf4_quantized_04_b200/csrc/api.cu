// C ABI of libqnf4 (declared in include/qnf4.h): argument checks, workspace
// layout, tensor-map creation and kernel launches. All device code of the library
// is compiled in this one translation unit.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <cublas_v2.h>
#include <cusolverDn.h>
#include <dlfcn.h>
#include <nvtx3/nvToolsExt.h>

#include <algorithm>
#include <cmath>
#include <atomic>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <string>
#include <vector>

#include "../../include/qnf4.h"
#include "chanq.cuh"
#include "common.cuh"
#include "decode.cuh"
#include "gemm.cuh"
#include "grad.cuh"
#include "loftq.cuh"
#include "multi.cuh"
#include "multi_mm.cuh"
#include "quant.cuh"
#include "tables.h"

namespace qnf4 {
namespace {

thread_local std::string g_last = "";
unsigned long long g_wait_ns = 1000000000ull;

qnf4_status fail(qnf4_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_last = buf;
  return s;
}
qnf4_status ok() { return QNF4_OK; }

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

std::atomic<unsigned long long> g_launches{0};
thread_local cudaEvent_t g_ev_start = nullptr, g_ev_stop = nullptr;

// Check the last launch(es) and count `n` kernels of this library as launched.
// first failure of a cudaLaunchKernelEx launch since the last launched() check
thread_local cudaError_t g_launch_err = cudaSuccess;

qnf4_status launched(const char* what, int n = 1) {
  g_launches.fetch_add(static_cast<unsigned long long>(n), std::memory_order_relaxed);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) e = g_launch_err;
  g_launch_err = cudaSuccess;
  if (e != cudaSuccess) return fail(QNF4_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  return QNF4_OK;
}

// Launch as a programmatic dependent of the previous kernel in the stream: the kernel
// may start (and run its prologue) while that kernel finishes. Every kernel launched this way
// calls griddepcontrol.wait before it touches what the grid before it may still write or read,
// and at the latest before it ends (which of them read anything earlier: see k_gemm).
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                       Args... args) {
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
  if (e != cudaSuccess && g_launch_err == cudaSuccess) g_launch_err = e;
  return e;
}

int num_sms() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  static std::mutex mu;
  static std::vector<int> cache;
  std::lock_guard<std::mutex> lk(mu);
  if (static_cast<int>(cache.size()) <= dev) cache.resize(dev + 1, 0);
  if (cache[dev] == 0) {
    int v = 0;
    cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev);
    cache[dev] = v > 0 ? v : 148;
  }
  return cache[dev];
}

QuantTab make_tab() {
  const Nf4Tables& t = nf4_tables();
  QuantTab q;
  std::memcpy(q.thr, t.thr, sizeof(q.thr));
  std::memcpy(q.levels, t.levels, sizeof(q.levels));
  q.bin_h = t.bin_h;
  std::memcpy(q.bin_th, t.bin_th, sizeof(q.bin_th));
  return q;
}

int quant_grid_chunks(int64_t chunks) {
  // persistent: kQCtasPerSm streaming CTAs per SM, never more warps than chunks
  const int64_t ctas = (chunks + kQWorkers - 1) / kQWorkers;
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(ctas, num_sms() * kQCtasPerSm)));
}
int quant_grid(int64_t nblocks) { return quant_grid_chunks((nblocks + kQChunkBlocks - 1) / kQChunkBlocks); }

bool g_quant_smem_set[64] = {};

qnf4_status quant_smem_attr() {
  // the quantizer's code search needs the bin table (always found for the NF4 levels)
  if (nf4_tables().bin_h < 1 || nf4_tables().bin_h > kQMaxH)
    return fail(QNF4_ERR_ARG, "internal: no NF4 bin table the quantizer can hold");
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 64 && !g_quant_smem_set[dev]) {
    for (auto fn : {k_nf4_quant<true, true>, k_nf4_quant<true, false>, k_nf4_quant<false, true>,
                    k_nf4_quant<false, true, true>}) {
      const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 static_cast<int>(kQSmem));
      if (e != cudaSuccess) return fail(QNF4_ERR_CUDA, "smem attribute: %s", cudaGetErrorString(e));
    }
    g_quant_smem_set[dev] = true;
  }
  return QNF4_OK;
}

qnf4_status check_weight(const qnf4_weight* w) {
  if (!w) return fail(QNF4_ERR_ARG, "weight is NULL");
  if (w->block1 != 64 || w->block2 != 256)
    return fail(QNF4_ERR_ARG, "block1 must be 64 and block2 256 (got %d, %d)", w->block1, w->block2);
  if (w->N <= 0 || w->K <= 0) return fail(QNF4_ERR_SHAPE, "N and K must be positive");
  if (w->K % 64) return fail(QNF4_ERR_SHAPE, "K must be a multiple of 64 (got %lld)", (long long)w->K);
  if (!w->packed || !w->code2 || !w->scale2 || !w->mean) return fail(QNF4_ERR_ARG, "weight has a NULL buffer");
  if (!al16(w->packed) || !al16(w->code2) || !al16(w->scale2) || !al16(w->mean))
    return fail(QNF4_ERR_ALIGN, "weight buffers must be 16-byte aligned");
  return ok();
}


// ---------------------------------------------------------------------------
// tcgen05 GEMM planning: tile sizes, split-K and the workspace carve-up
// ---------------------------------------------------------------------------
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static EncodeFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeFn>(p);
  });
  return fn;
}

// 2-D tensor map over a row-major [outer, inner] matrix with row stride ld elements.
bool make_map(CUtensorMap* m, const void* ptr, bool u8, uint64_t inner, uint64_t outer,
              uint64_t ld, uint32_t box_in, uint32_t box_out, bool sw128) {
  std::memset(m, 0, sizeof(*m));
  EncodeFn fn = encode_fn();
  if (!fn) return false;
  const uint64_t es = u8 ? 1 : 2;
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {ld * es};
  cuuint32_t box[2] = {box_in, box_out};
  cuuint32_t estr[2] = {1, 1};
  const CUresult r = fn(m, u8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                        const_cast<void*>(ptr), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE,
                        sw128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// The same for bf16 with a swizzle of its own.
bool make_map_sw(CUtensorMap* m, const void* ptr, uint64_t inner, uint64_t outer, uint64_t ld, uint32_t box_in,
                 uint32_t box_out, CUtensorMapSwizzle sw) {
  std::memset(m, 0, sizeof(*m));
  EncodeFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {ld * 2};
  cuuint32_t box[2] = {box_in, box_out};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The quantizer's view of a weight: a [nblocks, 64] bf16 matrix, loaded in boxes of
// kQChunkBlocks rows with the 128-byte swizzle.
bool quant_map(CUtensorMap* m, const void* W, int64_t nblocks) {
  if (nblocks > INT32_MAX) return false;  // the row coordinate is a 32-bit integer
  return make_map(m, W, false, 64, static_cast<uint64_t>(nblocks), 64, 64, kQChunkBlocks, true);
}

// One weight as the only job of a quantize launch (false if its map cannot be made).
bool one_quant_job(QuantJobs* j, const void* W, int64_t nblocks, uint8_t* packed, float* absmax) {
  std::memset(j, 0, sizeof(*j));
  j->n = 1;
  j->nblocks[0] = nblocks;
  j->chunk0[0] = 0;
  j->chunk0[1] = (nblocks + kQChunkBlocks - 1) / kQChunkBlocks;
  j->packed[0] = reinterpret_cast<uint32_t*>(packed);
  j->absmax[0] = absmax;
  return quant_map(&j->map[0], W, nblocks);
}

// CTAs of a double-quantization launch over nb2 256-blocks, each a contiguous run.
int dq_grid(DqJobs* d, int64_t nb2) {
  const int64_t P = std::max<int64_t>(1, std::min<int64_t>((nb2 + 7) / 8, num_sms() * 4));
  d->per_cta = std::max<int64_t>(1, (nb2 + P - 1) / P);
  return static_cast<int>(std::max<int64_t>(1, (nb2 + d->per_cta - 1) / d->per_cta));
}

// One tensor as the only job of a double-quantization launch; returns the grid.
int one_dq_job(DqJobs* d, const float* c, int64_t nb1, const double* part, int npart, int64_t count,
               uint8_t* code2, float* scale2, float* mean, const double* sse_part, int nsse,
               double* sse_out) {
  std::memset(d, 0, sizeof(*d));
  d->n = 1;
  d->c[0] = c;
  d->nb1[0] = nb1;
  d->count[0] = count;
  d->part[0] = part;
  d->npart = npart;
  d->code2[0] = code2;
  d->scale2[0] = scale2;
  d->mean[0] = mean;
  d->sse_part[0] = sse_part;
  d->nsse = nsse;
  d->sse_out[0] = sse_out;
  d->b2_0[0] = 0;
  d->b2_0[1] = (nb1 + 255) / 256;
  return dq_grid(d, d->b2_0[1]);
}

// x [M, K] bf16 seen as [K/64][M][64]: box = 16 column blocks x rows x 64 columns
// (128-byte swizzle on the 128-byte rows).
bool make_map_xblocks(CUtensorMap* m, const void* x, uint64_t K, uint64_t M, uint32_t rows) {
  std::memset(m, 0, sizeof(*m));
  EncodeFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {64, M, K / 64};
  cuuint64_t strides[2] = {K * 2, 128};
  cuuint32_t box[3] = {64, rows, kDecSbBlocks};
  cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(x), dims, strides,
                        box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// packed [N, K/2] bytes seen as [N][K/256][128] (K a multiple of 256): box = rows x 4
// column groups x 128 bytes, each row's 512 bytes in order (128-byte swizzle).
bool make_map_wcols(CUtensorMap* m, const void* packed, uint64_t K, uint64_t N, uint32_t rows) {
  std::memset(m, 0, sizeof(*m));
  EncodeFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {128, K / 256, N};
  cuuint64_t strides[2] = {128, K / 2};
  cuuint32_t box[3] = {128, kDecGroups, rows};
  cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(packed), dims, strides,
                        box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

struct GemmPlan {
  int asrc = 0, tn = 16, has_ext = 0;
  int64_t rows = 0, cols = 0;
  int nsteps = 0, row_tiles = 0, col_tiles = 0, s1 = 1, s2 = 0;
  // work units: full_tiles whole tiles, then tail_tiles tiles cut into tail_splits
  // contraction slices of tail_sps steps; grid = persistent CTAs
  int full_tiles = 0, tail_tiles = 0, tail_splits = 1, tail_sps = 0, units = 0, grid = 1;
  int ctas_per_sm = 1;
  int nset = 1;  // converter warp sets (4 warps each)
  int lut = 0;   // NF4 dequantization through the shared-memory pair table
  int clus = 1;  // many adapters: the slices of a tile are the CTAs of a cluster (no partials)
  size_t smem = 0;
  size_t part_floats() const {
    return tail_splits > 1 && clus == 1 ? static_cast<size_t>(tail_tiles) * tail_splits * tn * 128 : 0;
  }
  int64_t tiles() const { return static_cast<int64_t>(row_tiles) * col_tiles; }
};

constexpr size_t kSmemLimit = 227 * 1024;

// Tiling (measured on the Llama shapes): three converter sets for wide tiles, one set
// and two CTAs per SM for thin tiles, a 7-deep TMEM A ring for thin tiles, and
// contraction slices of at least four steps.
constexpr int kNsetWide = 3;
constexpr int kNsetThin = 1;
constexpr int kCtasThin = 2;
constexpr int kS2ThinTmem = 7;
constexpr int kMinSplitSteps = 4;

int tn_for_tokens(int64_t M) {
  if (M <= 16) return 16;
  if (M <= 32) return 32;
  if (M <= 64) return 64;
  if (M <= 128) return 128;
  return 256;
}

GemmPlan plan_gemm(int asrc, int64_t rows, int64_t cols, int64_t contraction, int tn,
                   int has_ext, int nsm) {
  GemmPlan p;
  p.asrc = asrc;
  p.tn = tn;
  p.has_ext = has_ext;
  p.rows = rows;
  p.cols = cols;
  p.nsteps = static_cast<int>((contraction + kStep - 1) / kStep);
  p.row_tiles = static_cast<int>((rows + kRowsTile - 1) / kRowsTile);
  p.col_tiles = static_cast<int>((cols + tn - 1) / tn);
  // Thin N tiles (decode, rank-r GEMMs) are latency bound: give them two CTAs per SM
  // and a shallower dequant ring; wide tiles take the whole shared memory.
  const bool thin = tn <= 32;
  p.ctas_per_sm = thin ? kCtasThin : 1;
  // Wide tiles need several converter sets to keep the tensor core fed; thin tiles
  // run more CTAs per SM instead.
  p.nset = src_deq(asrc) ? (thin ? kNsetThin : kNsetWide) : 1;
  if (src_tmem_a(asrc)) {
    // TMEM A stages. Each is reusable only after the MMA that read it has completed,
    // so the ring depth bounds the steps in flight per MMA round trip: as deep as the
    // accumulator leaves room for (256 columns per CTA at two CTAs per SM, 512 at one).
    const int room = static_cast<int>(((p.ctas_per_sm == 2 ? 256u : 512u) - acc_cols(tn)) / 32u);
    p.s2 = std::min(room, thin ? kS2ThinTmem : 8);
    if (p.s2 > kMaxS2) p.s2 = kMaxS2;
  } else {
    p.s2 = src_deq(asrc) ? ((thin ? 2 : 4)) : 0;
  }
  // Thin NF4 tiles (decode) dequantize through the shared-memory pair table (32 copies):
  // their converters are bound by integer issue, which the table moves to the load and
  // fma pipes.
  const bool nf4 = asrc == A_NF4_K || asrc == A_NF4_MN;
  p.lut = (nf4 && thin) ? 32 : 0;
  // 1 KB to align the dynamic buffer, 1 KB for static shared data, per CTA
  const size_t budget = (p.ctas_per_sm == 2 ? (kSmemLimit / 2 - 2048) : kSmemLimit) - 2048;
  for (int pass = 0; pass < 2; ++pass) {
    const SmemPlan one = smem_plan(asrc, tn, 1, p.s2, has_ext, p.lut);
    const size_t fixed = one.total - one.slot1;
    p.s1 = static_cast<int>(std::min<size_t>(kMaxS1, (budget - fixed) / one.slot1));
    // the dequantized-A ring may not be deeper than the load ring (its stages are
    // released through the load ring's barriers)
    if (p.s2 > p.s1) p.s2 = p.s1;
  }
  p.smem = smem_plan(asrc, tn, p.s1, p.s2, has_ext, p.lut).total + 1024;
  // Persistent CTAs, one per slot, take the tiles in waves. The tiles of a last,
  // partial wave are cut into contraction slices so that wave is as full as it can
  // be: as many slices as the idle slots allow, at least four steps each (each slice
  // costs a partial tile and one more term in the last slice's reduction).
  const int64_t tiles = p.tiles();
  const int64_t slots = static_cast<int64_t>(nsm) * p.ctas_per_sm;
  p.full_tiles = static_cast<int>((tiles / slots) * slots);
  p.tail_tiles = static_cast<int>(tiles - p.full_tiles);
  int best = 1;
  if (p.tail_tiles > 0 && p.nsteps > 1) {
    const int max_splits = std::max(1, p.nsteps / kMinSplitSteps);
    best = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(max_splits, slots / p.tail_tiles)));
  }
  p.tail_sps = (p.nsteps + best - 1) / best;
  p.tail_splits = p.tail_sps > 0 ? (p.nsteps + p.tail_sps - 1) / p.tail_sps : 1;
  p.units = p.full_tiles + p.tail_tiles * p.tail_splits;
  p.grid = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(p.units, slots)));
  return p;
}

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Workspace of one linear-layer call (forward or backward).
struct LinPlan {
  int r16 = 16;
  int64_t ldm = 0, ldn = 0;
  GemmPlan u, v, main, da, db;
  size_t off_up = 0, off_ut = 0, off_vp = 0, off_vt = 0, off_bt = 0, off_part = 0, off_cnt = 0;
  size_t off_upart = 0, off_ucnt = 0;  // the u kernel's own split-K area (it may overlap the next)
  size_t total = 0;
};

LinPlan plan_linear(int main_src, int64_t N, int64_t K, int64_t M, int r, bool bwd, int nsm) {
  LinPlan L;
  L.r16 = ((r + 15) / 16) * 16;
  L.ldm = ((M + 7) / 8) * 8;
  L.ldn = ((N + 7) / 8) * 8;
  const int tnm = tn_for_tokens(M);
  size_t part = 0;
  int64_t cnt = 1;
  L.u = plan_gemm(A_DENSE_K, M, L.r16, K, L.r16, 0, nsm);
  if (!bwd) {
    L.main = plan_gemm(main_src, N, M, K, tnm, 1, nsm);
  } else {
    L.v = plan_gemm(A_DENSE_K, M, L.r16, N, L.r16, 0, nsm);
    L.main = plan_gemm(main_src, K, M, N, tnm, 1, nsm);
    L.da = plan_gemm(A_DENSE_MN, K, L.r16, M, L.r16, 0, nsm);
    L.db = plan_gemm(A_DENSE_MN, N, L.r16, M, L.r16, 0, nsm);
    for (const GemmPlan* g : {&L.v, &L.da, &L.db}) {
      part = std::max(part, g->part_floats());
      cnt = std::max(cnt, g->tiles());
    }
  }
  part = std::max(part, L.main.part_floats());
  cnt = std::max(cnt, L.main.tiles());
  size_t o = 0;
  L.off_up = o;
  o = align256(o + static_cast<size_t>(M) * 64 * 2);
  if (bwd) {
    L.off_ut = o;
    o = align256(o + static_cast<size_t>(L.r16) * L.ldm * 2);
    L.off_vp = o;
    o = align256(o + static_cast<size_t>(M) * 64 * 2);
    L.off_vt = o;
    o = align256(o + static_cast<size_t>(L.r16) * L.ldm * 2);
    L.off_bt = o;
    o = align256(o + static_cast<size_t>(L.r16) * L.ldn * 2);
  }
  L.off_upart = o;
  o = align256(o + L.u.part_floats() * sizeof(float));
  L.off_part = o;
  o = align256(o + part * sizeof(float));
  // counters last, so one memset clears both areas
  L.off_ucnt = o;
  o = align256(o + static_cast<size_t>(L.u.tiles()) * sizeof(unsigned int));
  L.off_cnt = o;
  o = align256(o + static_cast<size_t>(cnt) * sizeof(unsigned int));
  L.total = o;
  return L;
}

bool g_smem_set[2][6][4][3][64] = {};

template <int ASRC, int NSET, int MINB, bool MULTI = false>
qnf4_status launch_gemm(const GemmPlan& p, const CUtensorMap& a, const CUtensorMap& b,
                        const CUtensorMap& bx, const CUtensorMap& o, const CUtensorMap& t, GemmArgs g,
                        cudaStream_t s) {
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 64 && !g_smem_set[MULTI][ASRC][NSET][MINB][dev]) {
    const cudaError_t e = cudaFuncSetAttribute(k_gemm<ASRC, NSET, MINB, MULTI>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(kSmemLimit - 1024));
    if (e != cudaSuccess) return fail(QNF4_ERR_CUDA, "smem attribute: %s", cudaGetErrorString(e));
    g_smem_set[MULTI][ASRC][NSET][MINB][dev] = true;
  }
  if (p.s1 < 1 || p.s1 > kMaxS1 || p.s2 < 0 || p.s2 > kMaxS2 || p.s2 > p.s1 || p.tn < 16 || p.tn > 256 ||
      p.tn % 16 || tmem_cols(ASRC, p.tn, p.s2) > (p.ctas_per_sm == 2 ? 256u : 512u) ||
      (src_deq(ASRC) && NSET > p.s2))
    return fail(QNF4_ERR_ARG, "internal tiling out of range (s1 %d, s2 %d, tn %d)", p.s1, p.s2, p.tn);
  g.rows = p.rows;
  g.cols = p.cols;
  g.nsteps = p.nsteps;
  g.row_tiles = p.row_tiles;
  g.full_tiles = p.full_tiles;
  g.tail_tiles = p.tail_tiles;
  g.tail_splits = p.tail_splits;
  g.tail_sps = p.tail_sps;
  g.nunits = p.units;
  g.tn = p.tn;
  g.s1 = p.s1;
  g.s2 = p.s2;
  g.has_ext = p.has_ext;
  g.lut = p.lut;
  g.part_elems = static_cast<int64_t>(p.part_floats());
  g.cnt_elems = p.tail_tiles;
  g.wait_ns = g_wait_ns;
  g.clus = p.clus;
  if (!p.has_ext) g.stage = 0;  // the staging buffers live in the adapter tile
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  if (p.units < 1) return QNF4_OK;  // empty D: nothing to compute
  cfg.gridDim = dim3(p.grid, 1, 1);
  cfg.blockDim = dim3(gemm_threads(NSET), 1, 1);
  cfg.dynamicSmemBytes = p.smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(p.clus);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.clus > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, k_gemm<ASRC, NSET, MINB, MULTI>, a, b, bx, o, t, g);
  if (e != cudaSuccess) {
    g_launches.fetch_add(1, std::memory_order_relaxed);
    cudaGetLastError();
    return fail(QNF4_ERR_CUDA, "gemm launch: %s", cudaGetErrorString(e));
  }
  return launched("gemm");
}

// The instantiated (source, converter sets, CTAs per SM) combinations.
template <int ASRC>
qnf4_status launch_deq(const GemmPlan& p, const CUtensorMap& a, const CUtensorMap& b,
                       const CUtensorMap& bx, const CUtensorMap& o, const CUtensorMap& t,
                       const GemmArgs& g, cudaStream_t s) {
  const int key = p.nset * 10 + p.ctas_per_sm;
  switch (key) {
    case 11: return launch_gemm<ASRC, 1, 1>(p, a, b, bx, o, t, g, s);
    case 12: return launch_gemm<ASRC, 1, 2>(p, a, b, bx, o, t, g, s);
    case 21: return launch_gemm<ASRC, 2, 1>(p, a, b, bx, o, t, g, s);
    case 22: return launch_gemm<ASRC, 2, 2>(p, a, b, bx, o, t, g, s);
    case 31: return launch_gemm<ASRC, 3, 1>(p, a, b, bx, o, t, g, s);
    default: return fail(QNF4_ERR_ARG, "no kernel for %d converter sets x %d CTAs/SM", p.nset, p.ctas_per_sm);
  }
}

qnf4_status launch_any(const GemmPlan& p, const CUtensorMap& a, const CUtensorMap& b,
                       const CUtensorMap& bx, const CUtensorMap& o, const CUtensorMap& t,
                       const GemmArgs& g, cudaStream_t s) {
  switch (p.asrc) {
    case A_NF4_K: return launch_deq<A_NF4_K>(p, a, b, bx, o, t, g, s);
    case A_NF4_MN: return launch_deq<A_NF4_MN>(p, a, b, bx, o, t, g, s);
    case A_DENSE_K:
      return p.ctas_per_sm == 2 ? launch_gemm<A_DENSE_K, 1, 2>(p, a, b, bx, o, t, g, s)
                                : launch_gemm<A_DENSE_K, 1, 1>(p, a, b, bx, o, t, g, s);
    case A_DENSE_MN:
      return p.ctas_per_sm == 2 ? launch_gemm<A_DENSE_MN, 1, 2>(p, a, b, bx, o, t, g, s)
                                : launch_gemm<A_DENSE_MN, 1, 1>(p, a, b, bx, o, t, g, s);
    case A_CHANQ_MN: return launch_deq<A_CHANQ_MN>(p, a, b, bx, o, t, g, s);
    default: return launch_deq<A_CHANQ_K>(p, a, b, bx, o, t, g, s);
  }
}

// The many-adapter instances: wide tiles and thin ones of each source.
template <int ASRC>
qnf4_status launch_multi_src(const GemmPlan& p, const CUtensorMap& a, const CUtensorMap& b,
                             const CUtensorMap& bx, const CUtensorMap& o, const CUtensorMap& t,
                             const GemmArgs& g, cudaStream_t s) {
  constexpr int kWide = src_deq(ASRC) ? kNsetWide : 1;
  return p.ctas_per_sm == 2 ? launch_gemm<ASRC, 1, 2, true>(p, a, b, bx, o, t, g, s)
                            : launch_gemm<ASRC, kWide, 1, true>(p, a, b, bx, o, t, g, s);
}

qnf4_status launch_multi(const GemmPlan& p, const CUtensorMap& a, const CUtensorMap& b,
                         const CUtensorMap& bx, const CUtensorMap& o, const CUtensorMap& t,
                         const GemmArgs& g, cudaStream_t s) {
  switch (p.asrc) {
    case A_NF4_K: return launch_multi_src<A_NF4_K>(p, a, b, bx, o, t, g, s);
    case A_NF4_MN: return launch_multi_src<A_NF4_MN>(p, a, b, bx, o, t, g, s);
    case A_DENSE_K: return launch_multi_src<A_DENSE_K>(p, a, b, bx, o, t, g, s);
    case A_DENSE_MN: return launch_multi_src<A_DENSE_MN>(p, a, b, bx, o, t, g, s);
    default: return fail(QNF4_ERR_ARG, "no many-adapter kernel for source %d", p.asrc);
  }
}

GemmArgs base_args() {
  GemmArgs g;
  std::memset(&g, 0, sizeof(g));
  const Nf4Tables& t = nf4_tables();
  std::memcpy(g.levels, t.levels, sizeof(g.levels));
  // extents for the checked build's index tests: unbounded until a caller narrows them
  g.out_elems = g.out2_elems = g.part_elems = g.cnt_elems = g.cst_elems = INT64_MAX;
  return g;
}

// The frozen base of one linear layer, in one of its three storage forms.
struct BaseSrc {
  int kind = A_NF4_K;        // A_NF4_K (NF4), A_DENSE_K (bf16), A_CHANQ_K (per-channel)
  const qnf4_weight* w = nullptr;
  const void* Wd = nullptr;  // dense bf16 [N, K]
  const uint8_t* cq_packed = nullptr;
  const int64_t* cq_row_off = nullptr;
  const uint8_t* cq_bits = nullptr;
  const float* cq_map = nullptr;
  const int64_t* cq_map_off = nullptr;
  const float* cq_absmax = nullptr;
  // per-channel backward: the codes widened to the NF4 nibble layout [N, K/2] and the
  // rows' 16-entry tables [N, 16], made in the workspace by k_chanq_widen
  uint8_t* cq_wide = nullptr;
  float* cq_tab = nullptr;
  int64_t N = 0, K = 0;
};

// Output map of the staged epilogue: bf16 D with rows contiguous (ld elements between
// columns), stored in boxes of 128 rows x 8 columns. False when the layout does not allow
// it (row stride not a multiple of 16 bytes); the epilogue then stores element by element.
bool stage_map(CUtensorMap* m, void* out, int64_t rows, int64_t cols, int64_t ld) {
  std::memset(m, 0, sizeof(*m));
  if ((ld * 2) % 16 != 0 || !al16(out)) return false;
  return make_map(m, out, false, rows, cols, ld, 128, 8, false);
}

// Workspace after the backward's own: the widened codes [N, K/2] and the tables [N, 16].
size_t chanq_wide_bytes(int64_t N, int64_t K) {
  return align256(static_cast<size_t>(N) * static_cast<size_t>(K / 2)) +
         align256(static_cast<size_t>(N) * 16 * sizeof(float));
}

// 2-D fp32 tensor [outer, inner] (row stride ld elements), no swizzle.
bool make_map_f32(CUtensorMap* m, const void* ptr, uint64_t inner, uint64_t outer, uint64_t ld,
                  uint32_t box_in, uint32_t box_out) {
  std::memset(m, 0, sizeof(*m));
  EncodeFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {ld * 4};
  cuuint32_t box[2] = {box_in, box_out};
  cuuint32_t estr[2] = {1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<void*>(ptr), dims, strides,
                        box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

qnf4_status map_fail() { return fail(QNF4_ERR_CUDA, "cuTensorMapEncodeTiled unavailable or refused the layout"); }

// u = x A^T (contraction K), written as bf16(scale u) into up [M, 64] and, when ut is
// given, transposed into ut [r16, ldm].
qnf4_status run_u(const LinPlan& L, const void* x, const void* A, int64_t M, int64_t K, int r,
                  float scale, uint16_t* up, uint16_t* ut, float* part, unsigned* cnt, cudaStream_t s) {
  CUtensorMap ma, mb, none;
  std::memset(&none, 0, sizeof(none));
  if (!make_map(&ma, x, false, K, M, K, 64, 128, true)) return map_fail();
  if (!make_map(&mb, A, false, K, r, K, 64, L.r16, true)) return map_fail();
  GemmArgs g = base_args();
  g.epi = EPI_UV;
  g.out = up;
  g.out2 = ut;
  g.o2_ld = L.ldm;
  g.out_elems = M * 64;
  g.out2_elems = static_cast<int64_t>(L.r16) * L.ldm;
  g.scale = scale;
  g.part = part;
  g.counters = cnt;
  return launch_any(L.u, ma, mb, none, none, none, g, s);
}

// ---------------------------------------------------------------------------
// Decode-size forward (M <= 16 tokens): k_lora_u, then k_nf4_decode (see decode.cuh)
// ---------------------------------------------------------------------------
constexpr int64_t kDecodeMaxTokens = 16;

// Workspace of one decode-size layer: its adapter projection partials, 256-aligned.
size_t decode_ws_bytes(int64_t K, int64_t M, int r) {
  const int64_t ks = (K + kDecUChunk - 1) / kDecUChunk;
  return align256(static_cast<size_t>(ks) * r * M * sizeof(float));
}

bool g_dec_smem_set[2][2][64] = {};

template <int Q, bool MULTI>
cudaError_t launch_decode(const DecodeArgs& a, int P, cudaStream_t s) {
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 64 && !g_dec_smem_set[MULTI][Q - 1][dev]) {
    const cudaError_t e = cudaFuncSetAttribute(k_nf4_decode<Q, MULTI>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(kDecSmem));
    if (e != cudaSuccess) return e;
    g_dec_smem_set[MULTI][Q - 1][dev] = true;
  }
  return launch_pdl(k_nf4_decode<Q, MULTI>, dim3(P), dim3(kDecBlockThreads), kDecSmem, s, a, g_wait_ns);
}

// A buffer of a call, and lists of them: a many-adapter call's kernels (and the layers of a group)
// run into one another, so one that it writes may overlap no other.
struct Buf {
  const void* p = nullptr;
  size_t bytes = 0;
};
struct BufList {
  Buf v[64];
  int n = 0;
  void add(const void* p, int64_t elems, size_t size) { v[n++] = Buf{p, static_cast<size_t>(elems) * size}; }
};
qnf4_status check_apart(const BufList& written, const BufList& read) {
  auto meet = [](const Buf& a, const Buf& b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + b.bytes && y < x + a.bytes;
  };
  for (int i = 0; i < written.n; ++i) {
    for (int j = 0; j < i; ++j)
      if (meet(written.v[i], written.v[j])) return fail(QNF4_ERR_ARG, "an output or the workspace overlaps another one");
    for (int j = 0; j < read.n; ++j)
      if (meet(written.v[i], read.v[j])) return fail(QNF4_ERR_ARG, "an output or the workspace overlaps another argument");
  }
  return QNF4_OK;
}
void add_nf4(BufList* b, const qnf4_weight& w) {
  const int64_t nb = w.N * w.K / 64;
  b->add(w.packed, nb, 32);
  b->add(w.code2, nb, 1);
  b->add(w.scale2, (nb + 255) / 256, sizeof(float));
  b->add(w.mean, 1, sizeof(float));
}

// Decode-size forward of n independent layers in one launch pair (k_lora_u, then
// k_nf4_decode); the layers share M, r and scale, or with ids their many adapters (nad of
// them, with their scales; As and Bs are then stacks). Arguments are checked by the caller.
qnf4_status decode_group(int n, const qnf4_weight* w, const void* const* xs, int64_t M,
                         const void* const* As, const void* const* Bs, int r, float scale,
                         void* const* hs, void* ws, size_t ws_bytes, cudaStream_t s,
                         const int* ids = nullptr, int nad = 0, const float* scales = nullptr) {
  size_t need = 0;
  for (int l = 0; l < n; ++l) need += decode_ws_bytes(w[l].K, M, r);
  if (!ws || ws_bytes < need) return fail(QNF4_ERR_WORKSPACE, "workspace too small (%zu < %zu)", ws_bytes, need);
  // (the sums in it are read in fp32 words; many adapters keep the ABI's 16 bytes at every M)
  const uintptr_t unit = ids ? 16u : sizeof(float);
  if (reinterpret_cast<uintptr_t>(ws) % unit)
    return fail(QNF4_ERR_ALIGN, "the workspace must be %zu-byte aligned", static_cast<size_t>(unit));
  if (ids) {
    static_assert(7 * kDecMaxGroup + 2 <= 64, "the lists hold a group");
    BufList out, in;
    out.add(ws, static_cast<int64_t>(need), 1);
    in.add(ids, M, sizeof(int));
    in.add(scales, nad, sizeof(float));
    for (int l = 0; l < n; ++l) {
      out.add(hs[l], M * w[l].N, 2);
      in.add(xs[l], M * w[l].K, 2);
      in.add(As[l], nad * r * w[l].K, 2);
      in.add(Bs[l], nad * w[l].N * r, 2);
      add_nf4(&in, w[l]);
    }
    const qnf4_status st = check_apart(out, in);
    if (st != QNF4_OK) return st;
  }
  static thread_local DecodeArgs a;  // about 10 KB: kept off the stack
  std::memset(&a, 0, sizeof(a));
  a.n = n;
  a.M = static_cast<int>(M);
  a.r = r;
  a.scale = scale;
  a.ids = ids;
  a.nad = nad;
  a.scales = scales;
  std::memcpy(a.levels, nf4_tables().levels, sizeof(a.levels));
  size_t off = 0;
  int64_t units = 0, kmax = 0;
  double total = 0.0;  // work = units x K (bytes per unit are 8 K)
  for (int l = 0; l < n; ++l) {
    const int64_t N = w[l].N, K = w[l].K;
    DecLayer& L = a.L[l];
    L.N = N;
    L.K = K;
    L.nkb = static_cast<int>(K / 64);
    L.ks = static_cast<int>((K + kDecUChunk - 1) / kDecUChunk);
    L.w3d = K % 256 == 0 ? 1 : 0;
    L.unit0 = units;
    L.nb2 = (N * (K / 64) + 255) / 256;
    L.code2 = w[l].code2;
    L.scale2 = w[l].scale2;
    L.mean = w[l].mean;
    L.x = static_cast<const uint16_t*>(xs[l]);
    L.A = static_cast<const uint16_t*>(As[l]);
    L.Bm = static_cast<const uint16_t*>(Bs[l]);
    L.h = static_cast<uint16_t*>(hs[l]);
    L.upart = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + off);
    off += decode_ws_bytes(K, M, r);
    for (int i = 0; i < kDecMaxRb; ++i) {
      const uint32_t rows = 16u * (i + 1);
      const bool ok = L.w3d ? make_map_wcols(&a.wmap[l][i], w[l].packed, K, N, rows)
                            : make_map(&a.wmap[l][i], w[l].packed, true, K / 2, N, K / 2, 128, rows, true);
      if (!ok) return map_fail();
    }
    if (!make_map_xblocks(&a.xmap[l], xs[l], K, M, static_cast<uint32_t>(M))) return map_fail();
    const int64_t rbs = (N + 15) / 16;
    units += rbs;
    total += static_cast<double>(rbs) * static_cast<double>(K);
    kmax = std::max(kmax, K);
  }
  a.units = units;
  // CTA p takes the units from the first one whose start lies at or past p / P of the
  // total work (units x K), so every CTA streams about the same number of bytes
  const int P = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({num_sms(), units, kDecMaxCta})));
  {
    int p = 0;
    double cum = 0.0;
    int64_t u = 0;
    a.cta_unit[0] = 0;
    for (int l = 0; l < n; ++l) {
      const int64_t rbs = (w[l].N + 15) / 16;
      for (int64_t b = 0; b < rbs; ++b, ++u) {
        while (p + 1 < P && cum >= total * (p + 1) / P) a.cta_unit[++p] = u;
        cum += static_cast<double>(w[l].K);
      }
    }
    while (p < P) a.cta_unit[++p] = units;
  }
  if (g_ev_start) cudaEventRecord(g_ev_start, s);
  const int ksmax = static_cast<int>((kmax + kDecUChunk - 1) / kDecUChunk);
  cudaError_t e = ids ? launch_pdl(k_lora_u<true>, dim3(r, ksmax, n), dim3(128), 0, s, a)
                      : launch_pdl(k_lora_u<false>, dim3(r, ksmax, n), dim3(128), 0, s, a);
  if (e != cudaSuccess) return fail(QNF4_ERR_CUDA, "k_lora_u launch: %s", cudaGetErrorString(e));
  if (ids)
    e = M <= 8 ? launch_decode<1, true>(a, P, s) : launch_decode<2, true>(a, P, s);
  else
    e = M <= 8 ? launch_decode<1, false>(a, P, s) : launch_decode<2, false>(a, P, s);
  if (e != cudaSuccess) return fail(QNF4_ERR_CUDA, "k_nf4_decode launch: %s", cudaGetErrorString(e));
  if (g_ev_stop) cudaEventRecord(g_ev_stop, s);
  return launched("decode_fwd", 2);
}

qnf4_status decode_fwd(const qnf4_weight* w, const void* x, int64_t M, const void* A, const void* B,
                       int r, float scale, void* h, void* ws, size_t ws_bytes, cudaStream_t s) {
  return decode_group(1, w, &x, M, &A, &B, r, scale, &h, ws, ws_bytes, s);
}

qnf4_status linear_fwd(const BaseSrc& src, const void* x, int64_t M, const void* A, const void* B,
                       int r, float scale, void* h, void* ws, size_t ws_bytes, cudaStream_t s) {
  const int64_t N = src.N, K = src.K;
  const LinPlan L = plan_linear(src.kind, N, K, M, r, false, num_sms());
  if (!ws || ws_bytes < L.total) return fail(QNF4_ERR_WORKSPACE, "workspace too small (%zu < %zu)", ws_bytes, L.total);
  uint8_t* w8 = static_cast<uint8_t*>(ws);
  uint16_t* up = reinterpret_cast<uint16_t*>(w8 + L.off_up);
  float* part = reinterpret_cast<float*>(w8 + L.off_part);
  unsigned* cnt = reinterpret_cast<unsigned*>(w8 + L.off_cnt);
  if (cudaMemsetAsync(w8 + L.off_ucnt, 0, L.total - L.off_ucnt, s) != cudaSuccess)
    return launched("memset", 0);
  qnf4_status st = run_u(L, x, A, M, K, r, scale, up, nullptr,
                         reinterpret_cast<float*>(w8 + L.off_upart),
                         reinterpret_cast<unsigned*>(w8 + L.off_ucnt), s);
  if (st != QNF4_OK) return st;
  CUtensorMap ma, mb, mbx, none;
  std::memset(&none, 0, sizeof(none));
  std::memset(&ma, 0, sizeof(ma));
  const int tn = L.main.tn;
  if (src.kind == A_NF4_K) {
    if (!make_map(&ma, src.w->packed, true, K / 2, N, K / 2, 32, 128, false)) return map_fail();
  } else if (src.kind == A_DENSE_K) {
    if (!make_map(&ma, src.Wd, false, K, N, K, 64, 128, true)) return map_fail();
  }
  if (!make_map(&mb, x, false, K, M, K, 64, tn, true)) return map_fail();
  if (!make_map(&mbx, up, false, 64, M, 64, 64, tn, true)) return map_fail();
  GemmArgs g = base_args();
  g.ext_k16 = L.r16 / 16;
  g.ext_r = r;
  g.ext_a = static_cast<const uint16_t*>(B);
  g.ext_ld = r;
  g.wN = N;
  g.nbk = K / 64;
  if (src.kind == A_NF4_K) {
    g.code2 = src.w->code2;
    g.scale2 = src.w->scale2;
    g.mean = src.w->mean;
    g.packed = src.w->packed;
  } else if (src.kind == A_CHANQ_K) {
    g.cq_packed = src.cq_packed;
    g.cq_row_off = src.cq_row_off;
    g.cq_bits = src.cq_bits;
    g.cq_map = src.cq_map;
    g.cq_map_off = src.cq_map_off;
    g.cq_absmax = src.cq_absmax;
  }
  g.epi = EPI_BF16;
  g.out = h;
  g.o_rs = 1;
  g.o_cs = N;
  g.out_elems = M * N;
  if (src.kind == A_NF4_K) g.cst_elems = N * (K / 64);
  CUtensorMap mo;
  g.stage = stage_map(&mo, h, N, M, N) ? 1 : 0;
  g.part = part;
  g.counters = cnt;
  g.lazy_dep = 1;  // only the adapter chunk reads what the u kernel writes
  if (g_ev_start) cudaEventRecord(g_ev_start, s);
  st = launch_any(L.main, ma, mb, mbx, mo, none, g, s);
  if (g_ev_stop) cudaEventRecord(g_ev_stop, s);
  return st;
}

qnf4_status linear_bwd(const BaseSrc& src, const void* x, const void* dY, int64_t M, const void* A,
                       const void* B, int r, float scale, void* dX, float* dA, float* dB, void* ws,
                       size_t ws_bytes, cudaStream_t s) {
  const int64_t N = src.N, K = src.K;
  const int main_src =
      src.kind == A_NF4_K ? A_NF4_MN : (src.kind == A_CHANQ_K ? A_CHANQ_MN : A_DENSE_MN);
  const LinPlan L = plan_linear(main_src, N, K, M, r, true, num_sms());
  if (!ws || ws_bytes < L.total) return fail(QNF4_ERR_WORKSPACE, "workspace too small (%zu < %zu)", ws_bytes, L.total);
  uint8_t* w8 = static_cast<uint8_t*>(ws);
  uint16_t* ut = reinterpret_cast<uint16_t*>(w8 + L.off_ut);
  uint16_t* vp = reinterpret_cast<uint16_t*>(w8 + L.off_vp);
  uint16_t* vt = reinterpret_cast<uint16_t*>(w8 + L.off_vt);
  uint16_t* bt = reinterpret_cast<uint16_t*>(w8 + L.off_bt);
  float* part = reinterpret_cast<float*>(w8 + L.off_part);
  unsigned* cnt = reinterpret_cast<unsigned*>(w8 + L.off_cnt);
  if (cudaMemsetAsync(w8 + L.off_ucnt, 0, L.total - L.off_ucnt, s) != cudaSuccess)
    return launched("memset", 0);
  // B^T for v = dY B
  {
    const int grid = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>((N * r + 255) / 256, num_sms() * 4)));
    k_transpose_b<<<grid, 256, 0, s>>>(static_cast<const uint16_t*>(B), N, r, bt, L.ldn);
    qnf4_status st = launched("transpose_b");
    if (st != QNF4_OK) return st;
  }
  qnf4_status st = QNF4_OK;
  CUtensorMap none;
  std::memset(&none, 0, sizeof(none));
  // Order: v and u, then dA and dB while x and dY are still in L2 (both are
  // HBM-bound), then dX (tensor-bound).
  // v = dY B  ->  vp = bf16(scale v) [M, 64], vt = its transpose [r16, ldm]
  {
    CUtensorMap ma, mb;
    if (!make_map(&ma, dY, false, N, M, N, 64, 128, true)) return map_fail();
    if (!make_map(&mb, bt, false, N, r, L.ldn, 64, L.r16, true)) return map_fail();
    GemmArgs g = base_args();
    g.epi = EPI_UV;
    g.out = vp;
    g.out2 = vt;
    g.o2_ld = L.ldm;
    g.out_elems = M * 64;
    g.out2_elems = static_cast<int64_t>(L.r16) * L.ldm;
    g.scale = scale;
    g.part = part;
    g.counters = cnt;
    st = launch_any(L.v, ma, mb, none, none, none, g, s);
    if (st != QNF4_OK) return st;
  }
  // (scale u)^T for dB
  st = run_u(L, x, A, M, K, r, scale, nullptr, ut,
                         reinterpret_cast<float*>(w8 + L.off_upart),
                         reinterpret_cast<unsigned*>(w8 + L.off_ucnt), s);
  if (st != QNF4_OK) return st;
  // dA = (scale v)^T x  -> [r, K]
  {
    CUtensorMap ma, mb;
    if (!make_map(&ma, x, false, K, M, K, 64, 64, true)) return map_fail();
    if (!make_map(&mb, vt, false, M, L.r16, L.ldm, 64, L.r16, true)) return map_fail();
    GemmArgs g = base_args();
    g.epi = EPI_F32;
    g.out = dA;
    g.o_rs = 1;
    g.o_cs = K;
    g.out_cols = r;
    g.out_elems = static_cast<int64_t>(r) * K;
    g.scale = 1.f;
    g.part = part;
    g.counters = cnt;
    st = launch_any(L.da, ma, mb, none, none, none, g, s);
    if (st != QNF4_OK) return st;
  }
  // dB = dY^T (scale u)  -> [N, r]
  {
    CUtensorMap ma, mb;
    if (!make_map(&ma, dY, false, N, M, N, 64, 64, true)) return map_fail();
    if (!make_map(&mb, ut, false, M, L.r16, L.ldm, 64, L.r16, true)) return map_fail();
    GemmArgs g = base_args();
    g.epi = EPI_F32;
    g.out = dB;
    g.o_rs = r;
    g.o_cs = 1;
    g.out_cols = r;
    g.out_elems = N * r;
    g.scale = 1.f;
    g.part = part;
    g.counters = cnt;
    st = launch_any(L.db, ma, mb, none, none, none, g, s);
    if (st != QNF4_OK) return st;
  }
  // dX = dY W_hat + (scale v) A
  {
    CUtensorMap ma, mb, mbx, mt;
    std::memset(&mt, 0, sizeof(mt));
    const int tn = L.main.tn;
    if (main_src == A_NF4_MN) {
      if (!make_map(&ma, src.w->packed, true, K / 2, N, K / 2, 64, 64, false)) return map_fail();
    } else if (main_src == A_CHANQ_MN) {
      if (!make_map(&ma, src.cq_wide, true, K / 2, N, K / 2, 64, 64, false)) return map_fail();
      if (!make_map_f32(&mt, src.cq_tab, 16, N, 16, 16, 64)) return map_fail();
    } else {
      if (!make_map(&ma, src.Wd, false, K, N, K, 64, 64, true)) return map_fail();
    }
    if (!make_map(&mb, dY, false, N, M, N, 64, tn, true)) return map_fail();
    if (!make_map(&mbx, vp, false, 64, M, 64, 64, tn, true)) return map_fail();
    GemmArgs g = base_args();
    g.ext_k16 = L.r16 / 16;
    g.ext_r = r;
    g.ext_a = static_cast<const uint16_t*>(A);
    g.ext_ld = K;
    g.wN = N;
    g.nbk = K / 64;
    if (main_src == A_NF4_MN) {
      g.code2 = src.w->code2;
      g.scale2 = src.w->scale2;
      g.mean = src.w->mean;
    } else if (main_src == A_CHANQ_MN) {
      g.cq_absmax = src.cq_absmax;
    }
    g.epi = EPI_BF16;
    g.out = dX;
    g.o_rs = 1;
    g.o_cs = K;
    g.out_elems = M * K;
    if (main_src == A_NF4_MN || main_src == A_CHANQ_MN) g.cst_elems = N * (K / 64);
    CUtensorMap mo;
    g.stage = stage_map(&mo, dX, K, M, K) ? 1 : 0;
    g.part = part;
    g.counters = cnt;
    if (g_ev_start) cudaEventRecord(g_ev_start, s);
    st = launch_any(L.main, ma, mb, mbx, mo, mt, g, s);
    if (g_ev_stop) cudaEventRecord(g_ev_stop, s);
    if (st != QNF4_OK) return st;
  }
  return QNF4_OK;
}

qnf4_status check_linear_args(int64_t N, int64_t K, int64_t M, int r, bool bwd,
                              std::initializer_list<const void*> ptrs) {
  if (N <= 0 || K <= 0) return fail(QNF4_ERR_SHAPE, "N and K must be positive");
  if (K % 64) return fail(QNF4_ERR_SHAPE, "K must be a multiple of 64 (got %lld)", (long long)K);
  if (bwd && N % 8) return fail(QNF4_ERR_SHAPE, "the backward needs N to be a multiple of 8 (got %lld)", (long long)N);
  if (M < 0) return fail(QNF4_ERR_SHAPE, "M must be >= 0");
  if (M > (int64_t)INT32_MAX) return fail(QNF4_ERR_SHAPE, "M too large");
  if (r < 1 || r > 64) return fail(QNF4_ERR_ARG, "r must be in [1, 64] (got %d)", r);
  for (const void* p : ptrs) {
    if (!p) return fail(QNF4_ERR_ARG, "NULL buffer");
    if (!al16(p)) return fail(QNF4_ERR_ALIGN, "buffers must be 16-byte aligned");
  }
  return QNF4_OK;
}


// ---------------------------------------------------------------------------
// Workspace for the allocation-free forward (qnf4_qlora_linear_fwd_noalloc). A
// file-scope device array: every GPU that loads the library holds it until exit.
// 32 MiB covers the forward's split-K partial tiles at their largest (one 256-column
// tile slice per CTA slot: 148 x 256 x 128 fp32 on a B200, 19.4 MB), the adapter
// projection's partials and the bf16 (s u) rows (128 bytes per token) up to 65536
// tokens, for every N, K and r <= 64.
// ---------------------------------------------------------------------------
constexpr size_t kNoAllocScratchBytes = size_t(32) << 20;  // 32 MiB
static __device__ __align__(256) uint8_t g_noalloc_scratch[kNoAllocScratchBytes];

// Device address of the array on each device, looked up once per device with that
// device current (cudaGetSymbolAddress); later calls read the cached address without
// taking the lock. nullptr and a message on failure.
void* noalloc_scratch_ptr() {
  constexpr int kMaxDev = 64;
  static std::atomic<void*> cache[kMaxDev] = {};
  static std::mutex mu;
  int dev = 0;
  const cudaError_t ge = cudaGetDevice(&dev);
  if (ge != cudaSuccess) {
    fail(QNF4_ERR_CUDA, "cudaGetDevice: %s", cudaGetErrorString(ge));
    return nullptr;
  }
  if (dev < 0 || dev >= kMaxDev) {
    fail(QNF4_ERR_CUDA, "device %d out of range for the built-in scratch (at most %d devices)", dev, kMaxDev);
    return nullptr;
  }
  if (void* p = cache[dev].load(std::memory_order_acquire)) return p;
  std::lock_guard<std::mutex> lk(mu);
  if (void* p = cache[dev].load(std::memory_order_relaxed)) return p;
  void* p = nullptr;
  const cudaError_t e = cudaGetSymbolAddress(&p, g_noalloc_scratch);
  if (e != cudaSuccess) {
    fail(QNF4_ERR_CUDA, "scratch address: %s", cudaGetErrorString(e));
    return nullptr;
  }
  cache[dev].store(p, std::memory_order_release);
  return p;
}
// ---------------------------------------------------------------------------
// Dense linear algebra for the LoftQ initialisation's truncated SVD: cuBLAS (sgemm) and
// cuSOLVER (syevd), loaded at first use by soname (torch's copies when torch has loaded
// them, else the toolkit's), so the library still loads where they are absent.
// ---------------------------------------------------------------------------
struct LinAlgLib {
  bool ok = false;
  decltype(&cublasCreate_v2) blas_create = nullptr;
  decltype(&cublasSetStream_v2) blas_stream = nullptr;
  decltype(&cublasSgemm_v2) sgemm = nullptr;
  decltype(&cusolverDnCreate) sol_create = nullptr;
  decltype(&cusolverDnSetStream) sol_stream = nullptr;
  decltype(&cusolverDnSsyevd_bufferSize) syevd_size = nullptr;
  decltype(&cusolverDnSsyevd) syevd = nullptr;
};

const LinAlgLib& linalg_lib() {
  static const LinAlgLib lib = [] {
    LinAlgLib l;
    auto open = [](std::initializer_list<const char*> names) -> void* {
      for (const char* n : names)
        if (void* h = dlopen(n, RTLD_NOW | RTLD_GLOBAL)) return h;
      return nullptr;
    };
    void* hb = open({"libcublas.so.12", "/usr/local/cuda/lib64/libcublas.so.12", "libcublas.so"});
    void* hs = open({"libcusolver.so.11", "/usr/local/cuda/lib64/libcusolver.so.11", "libcusolver.so"});
    if (!hb || !hs) return l;
    l.blas_create = reinterpret_cast<decltype(l.blas_create)>(dlsym(hb, "cublasCreate_v2"));
    l.blas_stream = reinterpret_cast<decltype(l.blas_stream)>(dlsym(hb, "cublasSetStream_v2"));
    l.sgemm = reinterpret_cast<decltype(l.sgemm)>(dlsym(hb, "cublasSgemm_v2"));
    l.sol_create = reinterpret_cast<decltype(l.sol_create)>(dlsym(hs, "cusolverDnCreate"));
    l.sol_stream = reinterpret_cast<decltype(l.sol_stream)>(dlsym(hs, "cusolverDnSetStream"));
    l.syevd_size = reinterpret_cast<decltype(l.syevd_size)>(dlsym(hs, "cusolverDnSsyevd_bufferSize"));
    l.syevd = reinterpret_cast<decltype(l.syevd)>(dlsym(hs, "cusolverDnSsyevd"));
    l.ok = l.blas_create && l.blas_stream && l.sgemm && l.sol_create && l.sol_stream &&
           l.syevd_size && l.syevd;
    return l;
  }();
  return lib;
}

// One cuBLAS and one cuSOLVER handle per device, kept for the process.
bool linalg_handles(cublasHandle_t* hb, cusolverDnHandle_t* hs) {
  const LinAlgLib& L = linalg_lib();
  if (!L.ok) return false;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return false;
  static std::mutex mu;
  static cublasHandle_t b[64] = {};
  static cusolverDnHandle_t so[64] = {};
  std::lock_guard<std::mutex> lk(mu);
  if (!b[dev] && L.blas_create(&b[dev]) != CUBLAS_STATUS_SUCCESS) return false;
  if (!so[dev] && L.sol_create(&so[dev]) != CUSOLVER_STATUS_SUCCESS) return false;
  *hb = b[dev];
  *hs = so[dev];
  return true;
}

// Floats of syevd workspace for an m x m Gram matrix: the library's own query when a GPU
// and cuSOLVER are at hand, and never below the LAPACK bound 1 + 6m + 2m^2.
size_t loftq_lwork(int64_t m) {
  size_t need = 1 + 6 * static_cast<size_t>(m) + 2 * static_cast<size_t>(m) * static_cast<size_t>(m);
  cublasHandle_t hb;
  cusolverDnHandle_t hs;
  if (linalg_handles(&hb, &hs)) {
    int lw = 0;
    if (linalg_lib().syevd_size(hs, CUSOLVER_EIG_MODE_VECTOR, CUBLAS_FILL_MODE_LOWER, static_cast<int>(m),
                                nullptr, static_cast<int>(m), nullptr, &lw) == CUSOLVER_STATUS_SUCCESS)
      need = std::max(need, static_cast<size_t>(lw));
  }
  return need;
}

struct LoftqLayout {
  size_t tgt, q, absmax, dq, gram, eig, p, info, work, total;
  int64_t m;
  size_t lwork;
};

LoftqLayout loftq_layout(int64_t N, int64_t K, int r) {
  LoftqLayout l{};
  l.m = std::min(N, K);
  l.lwork = loftq_lwork(l.m);
  size_t o = 0;
  l.tgt = o;    o = align256(o + static_cast<size_t>(N) * K * 2);
  l.q = o;      o = align256(o + static_cast<size_t>(N) * K * 4);
  l.absmax = o; o = align256(o + static_cast<size_t>(N) * K / 64 * 4);
  l.dq = o;     o = align256(o + qnf4_workspace_size(QNF4_OP_DOUBLE_QUANT, 0, 0, 0, 0));
  l.gram = o;   o = align256(o + static_cast<size_t>(l.m) * l.m * 4);
  l.eig = o;    o = align256(o + static_cast<size_t>(l.m) * 4);
  l.p = o;      o = align256(o + static_cast<size_t>(l.m) * r * 4);
  l.info = o;   o = align256(o + 16);
  l.work = o;   o = align256(o + l.lwork * 4);
  l.total = o;
  return l;
}

// ---------------------------------------------------------------------------
// Many adapters over one base (see multi.cuh)
// ---------------------------------------------------------------------------

// Tiling of the projections: slots per CTA, their batches, contraction slices.
struct ProjPlan {
  int sb = 4, nz = 1, slices = 1;
  uint32_t tmem = 32;
};

struct MultiPlan {
  int r16 = 16, per = 4, tn = 16, tiles = 0, dmax = 1, cmax = 1;
  GemmPlan main;
  ProjPlan proj;
  // backward: sorted positions, steps per gradient slice, slices, tiles of features
  int64_t ldp = 0;
  int lsteps = 1, slmax = 1, ftiles = 0;
  int64_t part_elems = 0, ctr_elems = 0;
  size_t off_cnt = 0, off_list = 0, off_exp = 0, off_part = 0, off_ctr = 0;
  size_t off_pos = 0, off_perm = 0, off_slices = 0, off_nsl = 0, off_bt = 0;
  size_t off_pt = 0, off_gctr = 0, off_clear_end = 0, off_gpart = 0, total = 0;
  // many tokens: the product over a 16-bit base (multi_mm.cuh); rp = operand columns per adapter
  bool mm = false;
  int rp = 64;
  size_t off_w = 0, off_g = 0, off_bad = 0;
};

// Product for many tokens (multi_mm.cuh) or k_gemm's? The former costs writing the base in 16
// bits and tiles of 256 tokens; its output rows must be 16-byte aligned, and its copies of the
// adapters stay below the base's size. Measured, k_gemm against this, us, 8 adapters of r = 16 (tokens
// in runs; the whole call):
//   forward NF4   4096 x 4096   43 / 49 at 512 tokens, 49 / 52 at 767, 56 / 53 at 1024
//                 4096 x 11008  76 / 100, 101 / 104, 112 / 106     (N x K)
//                 11008 x 4096  92 / 83, 95 / 89, 131 / 104
//   forward bf16  4096 x 4096   40 / 42, 43 / 44, 49 / 45;  11008 x 4096  91 / 62, 86 / 68, 119 / 83
//   backward NF4  4096 x 4096   68 / 68, 83 / 71, 87 / 75;  11008 x 4096 122 / 137, 167 / 142, 173 / 144
// One threshold for all: it is right within a quarter over an NF4 base. It is not where the base is 16-bit
// and wide: from 257 tokens on (more tiles than SMs) k_gemm's cut last wave loses to this by up to a half
// (384 tokens: 90 / 61).
// The bound on the copies, over NF4 4096 x 4096, forward: 1024 adapters of r = 16, tokens in runs, 116 / 197
// at 1024 tokens, 322 / 390 at 4096; 256 of r = 64 266 / 219, 466 / 322, and 2500 / 1438 where each of 4096
// tokens draws its own. Right for r = 16, not for 64; backward the two are within a tenth.
constexpr int64_t kMmMinTokens = 768;
bool use_mm(int64_t N, int64_t K, int64_t M, int n, int rp, bool bwd) {
  return M >= kMmMinTokens && N % 8 == 0 && static_cast<int64_t>(n) * rp <= (bwd ? N : K) &&
         n * N <= INT32_MAX;  // rows of the copies are 32-bit coordinates
}
int stage_grid() { return num_sms() * 6; }

// At most two CTAs per SM, all at once (a CTA costs about 6 us beside its steps, so a second wave
// of shorter ones loses): first by slices of the contraction (at least two steps each), then,
// where few tokens name many adapters, by taking the batches of slots in parallel and making
// them smaller. With 1024 tokens and more the token tiles fill the SMs, and a tile rarely
// names more adapters than one batch holds, so its CTAs take the batches one after another.
// The backward's two projections (csteps, the longer, and csteps2) share a launch, the longer one's
// CTAs first; where those alone would outlast an even share of all the steps by a quarter, both are
// cut further and a second wave of shorter CTAs fills up (5120 x 13824, 8192 tokens: 86 us, 117 uncut).
ProjPlan plan_proj(int64_t M, int64_t csteps, int64_t csteps2, int dmax, int per, int r16, int nsm) {
  ProjPlan p;
  const int64_t tiles = (M + 127) / 128 * (csteps2 ? 2 : 1);
  const int slots = (dmax + per - 1) / per * per;
  const int sbmax = kProjMaxCols / r16 / per * per;
  p.sb = std::min(slots, sbmax);
  while (p.slices < 8 && tiles * 2 * p.slices <= 2 * nsm && csteps / (2 * p.slices) >= 2) p.slices *= 2;
  while (csteps2 && p.slices < 8 && csteps / (2 * p.slices) >= 16 &&
         csteps / p.slices * 2 * nsm > (M + 127) / 128 * (csteps + csteps2) * 5 / 4)
    p.slices *= 2;
  auto batches = [&] { return (slots + p.sb - 1) / p.sb; };
  while (p.sb > per && tiles * p.slices * batches() < nsm) p.sb = std::max(per, p.sb / 2 / per * per);
  p.nz = static_cast<int>(std::min<int64_t>(batches(), std::max<int64_t>(1, 2 * nsm / (tiles * p.slices))));
  while (p.tmem < 256 && p.tmem < static_cast<uint32_t>(2 * p.sb * r16)) p.tmem <<= 1;
  return p;
}

MultiPlan plan_multi(int main_src, int64_t N, int64_t K, int64_t M, int n, int r, bool bwd, int nsm) {
  MultiPlan P;
  P.r16 = ((r + 15) / 16) * 16;
  P.per = 64 / P.r16;
  P.rp = r <= 16 ? 16 : (r <= 32 ? 32 : 64);
  P.mm = use_mm(N, K, M, n, P.rp, bwd);
  if (P.mm) {
    P.tn = 256;
    P.tiles = static_cast<int>((M + 255) / 256);
    P.per = 1;
  } else {
    P.tn = tn_for_tokens(M);
    P.main = bwd ? plan_gemm(main_src, K, M, N, P.tn, 1, nsm) : plan_gemm(main_src, N, M, K, P.tn, 1, nsm);
    P.tiles = P.main.col_tiles;
    // Few tiles, all of them cut: the slices of each form a cluster (at most 8).
    GemmPlan& m = P.main;
    if (m.full_tiles == 0 && m.tail_splits > 1 && static_cast<size_t>(m.tn) * 512 + 1024 <= m.smem) {
      m.tail_sps = (m.nsteps + std::min(8, m.tail_splits) - 1) / std::min(8, m.tail_splits);
      m.tail_splits = (m.nsteps + m.tail_sps - 1) / m.tail_sps;
      m.units = m.grid = m.tail_tiles * m.tail_splits;
      m.clus = m.tail_splits;
    }
  }
  const int width = P.mm ? P.rp : 64;
  P.dmax = static_cast<int>(std::min<int64_t>({n, P.tn, M}));
  P.cmax = (P.dmax + P.per - 1) / P.per;
  P.proj = plan_proj(M, (bwd ? std::max(N, K) : K) / 64, bwd ? std::max<int64_t>(1, std::min(N, K) / 64) : 0, P.dmax, P.per, P.r16, nsm);
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = align256(o + bytes);
    return at;
  };
  P.off_cnt = take(static_cast<size_t>(P.tiles) * sizeof(int));
  P.off_list = take(static_cast<size_t>(P.tiles) * P.dmax * sizeof(int));
  P.off_exp = take(static_cast<size_t>(P.tiles) * P.cmax * P.tn * width * 2);
  if (P.mm) {
    const bool nf4 = main_src == A_NF4_K || main_src == A_NF4_MN;
    P.off_w = take(nf4 ? static_cast<size_t>(N) * K * 2 : 0);
    P.off_g = take(static_cast<size_t>(n) * P.rp * (bwd ? K : N) * 2);
    P.off_bad = take(static_cast<size_t>(stage_grid()) * sizeof(int));
  }
  P.off_part = take(P.main.part_floats() * sizeof(float));
  P.off_ctr = take(static_cast<size_t>(P.mm ? 0 : P.main.tiles()) * sizeof(unsigned));
  if (bwd) {
    P.ldp = (M + 63) / 64 * 64 + 64 * std::min<int64_t>(n, M);
    P.ftiles = static_cast<int>((K + 127) / 128 + (N + 127) / 128);
    // slices of 8 to 64 steps, twice as long as would make one wave of two CTAs per SM out of one
    // adapter: several adapters are that many slices to begin with
    P.lsteps = static_cast<int>(std::max<int64_t>(8, std::min<int64_t>(64, 2 * M * P.ftiles / (64 * 2 * nsm))));
    const int64_t several = M / (64 * P.lsteps);  // adapters of more than one slice, at most
    P.slmax = static_cast<int>(several + n);
    P.part_elems = 2 * several * P.ftiles * 128 * P.r16;
    P.ctr_elems = several * P.ftiles;
    P.off_pos = take(static_cast<size_t>(M) * sizeof(int));
    P.off_perm = take(static_cast<size_t>(P.ldp) * sizeof(int));
    P.off_slices = take(static_cast<size_t>(P.slmax) * sizeof(GradSlice));
    P.off_nsl = take(sizeof(int));
    P.off_bt = take(static_cast<size_t>(n) * r * N * 2);
    P.off_pt = take(static_cast<size_t>(6) * P.r16 * P.ldp * 2);
    P.off_gctr = take(static_cast<size_t>(P.ctr_elems) * sizeof(unsigned));
    P.off_clear_end = o;
    P.off_gpart = take(static_cast<size_t>(P.part_elems) * sizeof(float));
  }
  P.total = o;
  return P;
}

// The adapters of a many-adapter call.
struct Adapters {
  const int* ids = nullptr;
  const void* A = nullptr;
  const void* B = nullptr;
  const float* scales = nullptr;
  int n = 0, r = 0;
};

bool g_proj_smem_set[64] = {}, g_grad_smem_set[64] = {};

// Launch as launch_pdl does, in clusters of `cluster` CTAs along x, with the kernel's dynamic
// shared memory limit set once per device.
template <typename... KArgs, typename... Args>
cudaError_t launch_multi_kernel(void (*kern)(KArgs...), bool* set, dim3 grid, int threads, size_t smem,
                                int cluster, cudaStream_t s, const Args&... args) {
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 64 || !set[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    if (dev < 64) set[dev] = true;
  }
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
  if (e != cudaSuccess && g_launch_err == cudaSuccess) g_launch_err = e;
  return e;
}

// One projection of a launch: X [M, C] onto F [n r, C], with the outputs wanted.
struct ProjJob {
  const void* X;
  const void* F;
  int64_t C;
  uint16_t* exp;
  uint16_t* pt;
};

qnf4_status multi_proj(const MultiPlan& P, const Adapters& ad, int64_t M, const ProjJob* jobs, int njobs,
                       uint8_t* w8, cudaStream_t s) {
  static thread_local ProjArgs g;
  std::memset(&g, 0, sizeof(g));
  const int xrows = static_cast<int>(std::min<int64_t>(128, (M + 15) / 16 * 16));
  g.xrows = xrows;
  for (int i = 0; i < njobs; ++i) {
    const ProjJob& j = jobs[i];
    if (!make_map(&g.tmX[i], j.X, false, j.C, M, j.C, 64, static_cast<uint32_t>(xrows), true) ||
        !make_map(&g.tmF[i], j.F, false, j.C, static_cast<uint64_t>(ad.n) * ad.r, j.C, 64, P.r16, true))
      return map_fail();
    g.nsteps[i] = static_cast<int>((j.C + 63) / 64);
    g.exp[i] = j.exp;
    g.pt[i] = j.pt;
  }
  g.swap = njobs > 1 && jobs[1].C > jobs[0].C;
  g.ids = ad.ids;
  g.scales = ad.scales;
  g.pos = reinterpret_cast<const int*>(w8 + P.off_pos);
  g.M = M;
  g.ldp = P.ldp;
  g.n = ad.n;
  g.r = ad.r;
  g.r16 = P.r16;
  g.per = P.per;
  g.tn = P.tn;
  g.dmax = P.dmax;
  g.cmax = P.cmax;
  g.sb = P.proj.sb;
  g.nz = P.proj.nz;
  g.slices = P.proj.slices;
  g.tmem_cols = P.proj.tmem;
  g.cnt = reinterpret_cast<int*>(w8 + P.off_cnt);
  g.list = reinterpret_cast<int*>(w8 + P.off_list);
  g.ctr = reinterpret_cast<unsigned*>(w8 + P.off_ctr);
  g.nctr = P.mm ? 0 : static_cast<int>(P.main.tiles());
  g.width = P.mm ? P.rp : 64;
  g.wait_ns = g_wait_ns;
  launch_multi_kernel(k_multi_proj, g_proj_smem_set,
                      dim3(P.proj.slices, static_cast<unsigned>((M + 127) / 128), njobs * P.proj.nz), kMultiThreads,
                      kProjSmem, P.proj.slices, s, g);
  return launched("multi_proj");
}

// The base product with the adapters' second product: D = base x X^T + ext (see k_gemm).
qnf4_status multi_main(const BaseSrc& src, int main_src, const MultiPlan& P, const Adapters& ad, const void* X,
                       int64_t M, const void* ext, int64_t ext_ld, int64_t ext_as, void* out, uint8_t* w8,
                       cudaStream_t s) {
  const int64_t N = src.N, K = src.K;
  const bool mn = src_mn(main_src);
  const int64_t rows = mn ? K : N, con = mn ? N : K;
  CUtensorMap ma, mb, mbx, mo, none;
  std::memset(&none, 0, sizeof(none));
  bool ok = true;
  switch (main_src) {
    case A_NF4_K: ok = make_map(&ma, src.w->packed, true, K / 2, N, K / 2, 32, 128, false); break;
    case A_NF4_MN: ok = make_map(&ma, src.w->packed, true, K / 2, N, K / 2, 64, 64, false); break;
    case A_DENSE_K: ok = make_map(&ma, src.Wd, false, K, N, K, 64, 128, true); break;
    default: ok = make_map(&ma, src.Wd, false, K, N, K, 64, 64, true); break;
  }
  uint16_t* exp = reinterpret_cast<uint16_t*>(w8 + P.off_exp);
  if (!ok || !make_map(&mb, X, false, con, M, con, 64, P.tn, true) ||
      !make_map(&mbx, exp, false, 64, static_cast<uint64_t>(P.tiles) * P.cmax * P.tn, 64, 64, P.tn, true))
    return map_fail();
  GemmArgs g = base_args();
  g.ext_k16 = 4;
  g.ext_r = ad.r;
  g.ext_a = static_cast<const uint16_t*>(ext);
  g.ext_ld = ext_ld;
  g.ext_as = ext_as;
  g.mt_cnt = reinterpret_cast<const int*>(w8 + P.off_cnt);
  g.mt_list = reinterpret_cast<const int*>(w8 + P.off_list);
  g.mt_ids = ad.ids;
  g.mt_exp = exp;
  g.mt_dmax = P.dmax;
  g.mt_cmax = P.cmax;
  g.mt_per = P.per;
  g.mt_r16 = P.r16;
  g.wN = N;
  g.nbk = K / 64;
  if (src.w) {
    g.code2 = src.w->code2;
    g.scale2 = src.w->scale2;
    g.mean = src.w->mean;
    g.packed = src.w->packed;
    g.cst_elems = N * (K / 64);
  }
  g.epi = EPI_BF16;
  g.out = out;
  g.o_rs = 1;
  g.o_cs = rows;
  g.out_elems = M * rows;
  g.stage = stage_map(&mo, out, rows, M, rows) ? 1 : 0;
  g.part = reinterpret_cast<float*>(w8 + P.off_part);
  g.counters = reinterpret_cast<unsigned*>(w8 + P.off_ctr);
  g.lazy_dep = P.main.units == P.main.grid ? 1 : 0;  // one unit per CTA: the base need not wait
  if (g_ev_start) cudaEventRecord(g_ev_start, s);
  const qnf4_status st = launch_multi(P.main, ma, mb, mbx, mo, none, g, s);
  if (g_ev_stop) cudaEventRecord(g_ev_stop, s);
  return st;
}

// Many tokens: the base in 16 bits and the adapters' second operand (rows cols as in StageArgs).
qnf4_status multi_stage(const BaseSrc& src, const MultiPlan& P, const Adapters& ad, bool bwd, uint8_t* w8,
                        cudaStream_t s) {
  StageArgs g;
  std::memset(&g, 0, sizeof(g));
  if (src.w) {
    g.packed = reinterpret_cast<const uint32_t*>(src.w->packed);
    g.code2 = src.w->code2;
    g.scale2 = src.w->scale2;
    g.mean = src.w->mean;
    g.n8 = src.N * src.K / 8;
    g.W = reinterpret_cast<uint16_t*>(w8 + P.off_w);
  }
  g.src = static_cast<const uint16_t*>(bwd ? ad.A : ad.B);
  g.dst = reinterpret_cast<uint16_t*>(w8 + P.off_g);
  g.rows = bwd ? ad.n : static_cast<int64_t>(ad.n) * src.N;
  g.cols = bwd ? src.K : 1;
  g.r = ad.r;
  g.rp = P.rp;
  g.bad = reinterpret_cast<int*>(w8 + P.off_bad);
  std::memcpy(g.levels, nf4_tables().levels, sizeof(g.levels));
  launch_pdl(k_multi_stage, dim3(stage_grid()), dim3(256), 0, s, g);
  return launched("multi_stage");
}

// CTA pairs of k_multi_mm that the device holds at once (one CTA per SM).
template <bool MN>
int mm_pairs() {
  static std::mutex mu;
  static int cache[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  std::lock_guard<std::mutex> lk(mu);
  int& c = cache[dev < 64 ? dev : 0];
  if (c == 0) {
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3(num_sms() / 2 * 2);
    cfg.blockDim = dim3(kMultiThreads);
    cfg.dynamicSmemBytes = kMmSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int k = 0;
    if (cudaFuncSetAttribute(k_multi_mm<MN>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kMmSmem)) !=
            cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&k, k_multi_mm<MN>, &cfg) != cudaSuccess || k < 1) {
      cudaGetLastError();
      return 0;
    }
    c = k;
  }
  return c;
}

bool g_mm_smem_set[2][64] = {};

template <bool MN>
qnf4_status multi_mm(const BaseSrc& src, const MultiPlan& P, const Adapters& ad, const void* X, int64_t M, void* out,
                     uint8_t* w8, cudaStream_t s) {
  const int64_t N = src.N, K = src.K, F = MN ? K : N, C = MN ? N : K;
  const void* W = src.w ? static_cast<const void*>(w8 + P.off_w) : src.Wd;
  uint16_t* exp = reinterpret_cast<uint16_t*>(w8 + P.off_exp);
  uint16_t* ag = reinterpret_cast<uint16_t*>(w8 + P.off_g);
  static thread_local MmArgs g;
  std::memset(&g, 0, sizeof(g));
  const auto sw = P.rp == 16 ? CU_TENSOR_MAP_SWIZZLE_32B : (P.rp == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
  if (!make_map(&g.tmX, X, false, C, M, C, 64, 128, true) || !make_map(&g.tmW, W, false, K, N, K, 64, MN ? 64 : 128, true) ||
      !make_map_sw(&g.tmE, exp, P.rp, static_cast<uint64_t>(P.tiles) * P.dmax * 256, P.rp, P.rp, 128, sw) ||
      !(MN ? make_map(&g.tmG, ag, false, K, static_cast<uint64_t>(ad.n) * P.rp, K, 64, P.rp, true)
           : make_map_sw(&g.tmG, ag, P.rp, static_cast<uint64_t>(ad.n) * N, P.rp, P.rp, 128, sw)) ||
      !make_map(&g.tmO, out, false, F, M, F, 64, 32, true))
    return map_fail();
  g.M = M;
  g.F = F;
  g.nk = static_cast<int>((C + 127) / 128);
  g.tt = P.tiles;
  g.ft = static_cast<int>((F + 255) / 256);
  const int pairs = mm_pairs<MN>();
  if (pairs < 1) return fail(QNF4_ERR_CUDA, "no CTA pair of the many-token product fits this device");
  g.rp = P.rp;
  g.dmax = P.dmax;
  g.cnt = reinterpret_cast<const int*>(w8 + P.off_cnt);
  g.list = reinterpret_cast<const int*>(w8 + P.off_list);
  g.grows = MN ? P.rp : N;
  g.bad = reinterpret_cast<const int*>(w8 + P.off_bad);
  g.nbad = stage_grid();
  g.ids = ad.ids;
  g.ext = static_cast<const uint16_t*>(MN ? ad.A : ad.B);
  g.exp = exp;
  g.as = static_cast<int64_t>(ad.r) * (MN ? K : N);
  g.js = MN ? K : ad.r;
  g.r = ad.r;
  g.n = ad.n;
  g.wait_ext = MN ? 0 : 1;
  g.wait_ns = g_wait_ns;
  if (g_ev_start) cudaEventRecord(g_ev_start, s);
  launch_multi_kernel(k_multi_mm<MN>, g_mm_smem_set[MN], dim3(2 * std::min(pairs, g.tt * g.ft)), kMultiThreads, kMmSmem, 2, s, g);
  if (g_ev_stop) cudaEventRecord(g_ev_stop, s);
  return launched("multi_mm");
}

// What a many-adapter call reads, beside its X and dY.
void add_reads(BufList* b, const BaseSrc& src, const Adapters& ad, int64_t M) {
  b->add(ad.ids, M, sizeof(int));
  b->add(ad.scales, ad.n, sizeof(float));
  b->add(ad.A, ad.n * ad.r * src.K, 2);
  b->add(ad.B, ad.n * src.N * ad.r, 2);
  if (src.w)
    add_nf4(b, *src.w);
  else
    b->add(src.Wd, src.N * src.K, 2);
}

qnf4_status multi_fwd(const BaseSrc& src, const Adapters& ad, const void* x, int64_t M, void* h, void* ws,
                      size_t ws_bytes, cudaStream_t s) {
  const MultiPlan P = plan_multi(src.kind, src.N, src.K, M, ad.n, ad.r, false, num_sms());
  if (!ws || ws_bytes < P.total) return fail(QNF4_ERR_WORKSPACE, "workspace too small (%zu < %zu)", ws_bytes, P.total);
  if (!al16(ws)) return fail(QNF4_ERR_ALIGN, "the workspace must be 16-byte aligned");
  BufList out, in;
  out.add(ws, static_cast<int64_t>(P.total), 1);
  out.add(h, M * src.N, 2);
  in.add(x, M * src.K, 2);
  add_reads(&in, src, ad, M);
  qnf4_status st = check_apart(out, in);
  if (st != QNF4_OK) return st;
  uint8_t* w8 = static_cast<uint8_t*>(ws);
  const ProjJob job{x, ad.A, src.K, reinterpret_cast<uint16_t*>(w8 + P.off_exp), nullptr};
  if (P.mm) st = multi_stage(src, P, ad, false, w8, s);
  // (k_multi_mm relies on the projections' wait for the grid before them, see there)
  if (st == QNF4_OK) st = multi_proj(P, ad, M, &job, 1, w8, s);
  if (st != QNF4_OK) return st;
  if (P.mm) return multi_mm<false>(src, P, ad, x, M, h, w8, s);
  return multi_main(src, src.kind, P, ad, x, M, ad.B, ad.r, src.N * ad.r, h, w8, s);
}

constexpr uint32_t kGradRing = 104u * 1024u;  // with 2 CTAs per SM; at least three stages

qnf4_status multi_grad(const MultiPlan& P, const Adapters& ad, const void* x, const void* dY, int64_t M, int64_t N,
                       int64_t K, const uint16_t* ptv, const uint16_t* ptu, float* dA, float* dB, uint8_t* w8,
                       cudaStream_t s) {
  static thread_local MultiGradArgs g;
  std::memset(&g, 0, sizeof(g));
  const int64_t r = ad.r;
  if (!make_map(&g.tmX[0], x, false, K, M, K, 64, 1, true) || !make_map(&g.tmX[1], dY, false, N, M, N, 64, 1, true) ||
      !make_map(&g.tmR[0], x, false, K, M, K, 64, 64, true) || !make_map(&g.tmR[1], dY, false, N, M, N, 64, 64, true) ||
      !make_map(&g.tmP[0], ptv, false, P.ldp, 3 * P.r16, P.ldp, 64, 3 * P.r16, true) ||
      !make_map(&g.tmP[1], ptu, false, P.ldp, 3 * P.r16, P.ldp, 64, 3 * P.r16, true))
    return map_fail();
  g.out[0] = dA;
  g.F[0] = K;
  g.as[0] = r * K;
  g.js[0] = K;
  g.fs[0] = 1;
  g.ft[0] = static_cast<int>((K + 127) / 128);
  g.out[1] = dB;
  g.F[1] = N;
  g.as[1] = N * r;
  g.js[1] = 1;
  g.fs[1] = r;
  g.ft[1] = static_cast<int>((N + 127) / 128);
  g.r = ad.r;
  g.r16 = P.r16;
  g.ring_bytes = kGradRing;
  g.tmem_cols = 32;
  while (g.tmem_cols < static_cast<uint32_t>(4 * P.r16)) g.tmem_cols <<= 1;
  g.slices = reinterpret_cast<const GradSlice*>(w8 + P.off_slices);
  g.nslices = reinterpret_cast<const int*>(w8 + P.off_nsl);
  g.perm = reinterpret_cast<const int*>(w8 + P.off_perm);
  g.part = reinterpret_cast<float*>(w8 + P.off_gpart);
  g.ctr = reinterpret_cast<unsigned*>(w8 + P.off_gctr);
  g.part_elems = P.part_elems;
  g.ctr_elems = P.ctr_elems;
  g.wait_ns = g_wait_ns;
  // two CTAs per SM at once; with few slices one each
  const int64_t gy = std::max<int64_t>(1, std::min<int64_t>(P.slmax, 2 * num_sms() / P.ftiles));
  launch_multi_kernel(k_multi_grad, g_grad_smem_set, dim3(P.ftiles, static_cast<unsigned>(gy)), kMultiThreads, kGradRing + 1024, 1, s, g);
  return launched("multi_grad");
}

qnf4_status multi_bwd(const BaseSrc& src, const Adapters& ad, const void* x, const void* dY, int64_t M, void* dX,
                      float* dA, float* dB, void* ws, size_t ws_bytes, cudaStream_t s) {
  const int64_t N = src.N, K = src.K;
  const int main_src = src.kind == A_NF4_K ? A_NF4_MN : A_DENSE_MN;
  const MultiPlan P = plan_multi(main_src, N, K, M, ad.n, ad.r, true, num_sms());
  if (!ws || ws_bytes < P.total) return fail(QNF4_ERR_WORKSPACE, "workspace too small (%zu < %zu)", ws_bytes, P.total);
  if (!al16(ws)) return fail(QNF4_ERR_ALIGN, "the workspace must be 16-byte aligned");
  BufList out, in;
  out.add(ws, static_cast<int64_t>(P.total), 1);
  out.add(dX, M * K, 2);
  out.add(dA, ad.n * ad.r * K, sizeof(float));
  out.add(dB, ad.n * N * ad.r, sizeof(float));
  in.add(x, M * K, 2);
  in.add(dY, M * N, 2);
  add_reads(&in, src, ad, M);
  qnf4_status st = check_apart(out, in);
  if (st != QNF4_OK) return st;
  uint8_t* w8 = static_cast<uint8_t*>(ws);
  uint16_t* bt = reinterpret_cast<uint16_t*>(w8 + P.off_bt);
  uint16_t* ptv = reinterpret_cast<uint16_t*>(w8 + P.off_pt);
  uint16_t* ptu = ptv + 3 * P.r16 * P.ldp;
  const int r = ad.r;
  PrepArgs pr;
  std::memset(&pr, 0, sizeof(pr));
  pr.ids = ad.ids;
  pr.M = M;
  pr.n = ad.n;
  pr.r = r;
  pr.lsteps = P.lsteps;
  pr.slmax = P.slmax;
  pr.ldp = P.ldp;
  pr.pos = reinterpret_cast<int*>(w8 + P.off_pos);
  pr.perm = reinterpret_cast<int*>(w8 + P.off_perm);
  pr.slices = reinterpret_cast<GradSlice*>(w8 + P.off_slices);
  pr.nslices = reinterpret_cast<int*>(w8 + P.off_nsl);
  pr.B = static_cast<const uint16_t*>(ad.B);
  pr.BT = bt;
  pr.N = N;
  pr.clear = reinterpret_cast<uint4*>(w8 + P.off_pt);
  pr.nclear = static_cast<int64_t>(P.off_clear_end - P.off_pt) / 16;
  pr.lazy = P.mm;
  if (P.mm) st = multi_stage(src, P, ad, true, w8, s);
  if (st != QNF4_OK) return st;
  const int64_t blocks = std::max<int64_t>(ad.n * ((N + 63) / 64), 8);
  launch_pdl(k_multi_prep, dim3(1 + static_cast<unsigned>(std::min<int64_t>(blocks, num_sms()))), dim3(kPrepThreads),
             std::max<size_t>(static_cast<size_t>(ad.n) * (ad.n <= kPrepTable ? 136 : 8), 64u * (r + 1) * 2), s, pr);
  st = launched("multi_prep");
  if (st != QNF4_OK) return st;
  const ProjJob jobs[2] = {{dY, bt, N, reinterpret_cast<uint16_t*>(w8 + P.off_exp), ptv}, {x, ad.A, K, nullptr, ptu}};
  st = multi_proj(P, ad, M, jobs, 2, w8, s);
  if (st != QNF4_OK) return st;
  st = multi_grad(P, ad, x, dY, M, N, K, ptv, ptu, dA, dB, w8, s);
  if (st != QNF4_OK) return st;
  if (P.mm) return multi_mm<true>(src, P, ad, dY, M, dX, w8, s);
  return multi_main(src, main_src, P, ad, dY, M, ad.A, K, static_cast<int64_t>(r) * K, dX, w8, s);
}

qnf4_status check_multi_args(int64_t N, int64_t K, int64_t M, int n, int r, bool bwd,
                             std::initializer_list<const void*> ptrs) {
  const qnf4_status st = check_linear_args(N, K, M, r, bwd, ptrs);
  if (st != QNF4_OK) return st;
  if (n < 1 || n > kMultiMaxAdapters)
    return fail(QNF4_ERR_ARG, "the number of adapters must be in [1, %d] (got %d)", kMultiMaxAdapters, n);
  if (M > 65535 * 128) return fail(QNF4_ERR_SHAPE, "at most %d tokens (got %lld)", 65535 * 128, (long long)M);
  // rows of the tiles' operand blocks are 32-bit copy coordinates
  if ((M + 255) / 256 * std::min<int64_t>({n, 256, std::max<int64_t>(M, 1)}) * 256 > INT32_MAX)
    return fail(QNF4_ERR_SHAPE, "too many tokens for %d adapters (got %lld)", n, (long long)M);
  return QNF4_OK;
}

// ---------------------------------------------------------------------------
// Gradient norms and clipping over a list of tensors (see grad.cuh)
// ---------------------------------------------------------------------------
// Elements of a piece of this list.
int grad_piece_size(int32_t count, const int64_t* elems) {
  int64_t total = 0;
  for (int32_t t = 0; t < count; ++t) total += elems[t];
  return total <= kGradShortList ? kGradShortPiece : kGradPiece;
}

// Pieces of one adapter's part over the whole list.
int64_t grad_pieces(int32_t count, const int64_t* elems, int32_t n) {
  const int piece = grad_piece_size(count, elems);
  int64_t p = 0;
  for (int32_t t = 0; t < count; ++t) p += (elems[t] / n + piece - 1) / piece;
  return p;
}

size_t grad_ws_bytes(int32_t count, const int64_t* elems, int32_t n) {
  return align256(static_cast<size_t>(grad_pieces(count, elems, n)) * n * sizeof(double)) +
         align256(static_cast<size_t>(n) * sizeof(float));
}

// An output is its own gradient's buffer or overlaps no gradient, and no two outputs overlap: else
// one piece would read what another has already written.
qnf4_status check_grad_outputs(int32_t count, const void* const* g, const int32_t* dtype, const int64_t* elems,
                               void* const* out) {
  struct Span {
    uintptr_t at, end;
    int32_t t;
  };
  auto span = [&](const void* p, int32_t t) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    return Span{at, at + static_cast<uintptr_t>(elems[t]) * (dtype[t] == QNF4_OUT_BF16 ? 2 : 4), t};
  };
  std::vector<Span> v;
  v.reserve(static_cast<size_t>(count));
  for (int32_t t = 0; t < count; ++t)
    if (elems[t]) v.push_back(span(out[t], t));
  const auto before = [](const Span& a, const Span& b) { return a.at < b.at; };
  if (!std::is_sorted(v.begin(), v.end(), before)) std::sort(v.begin(), v.end(), before);
  for (size_t i = 1; i < v.size(); ++i)
    if (v[i].at < v[i - 1].end) return fail(QNF4_ERR_ARG, "outputs %d and %d overlap", v[i - 1].t, v[i].t);
  for (int32_t t = 0; t < count; ++t) {
    if (!elems[t] || out[t] == g[t]) continue;
    const Span in = span(g[t], t);
    auto it = std::lower_bound(v.begin(), v.end(), in, before);  // the outputs are disjoint: ends ascend too
    if ((it != v.end() && it->at < in.end) || (it != v.begin() && (it - 1)->end > in.at))
      return fail(QNF4_ERR_ARG, "an output overlaps gradient %d", t);
  }
  return QNF4_OK;
}

// The norms and the workspace lie apart from each other and from every gradient and output.
qnf4_status check_grad_apart(int32_t count, const void* const* g, const int32_t* dtype, const int64_t* elems,
                             int32_t n, void* const* out, const float* norm, const void* ws, size_t need) {
  const uintptr_t nb = reinterpret_cast<uintptr_t>(norm), ne = nb + static_cast<uintptr_t>(n) * sizeof(float);
  const uintptr_t wb = reinterpret_cast<uintptr_t>(ws), we = wb + need;
  if (nb < we && wb < ne) return fail(QNF4_ERR_ARG, "norm overlaps the workspace");
  for (int32_t t = 0; t < count; ++t) {
    const uintptr_t bytes = static_cast<uintptr_t>(elems[t]) * (dtype[t] == QNF4_OUT_BF16 ? 2 : 4);
    if (!bytes) continue;
    for (const void* p : {g[t], out ? static_cast<const void*>(out[t]) : g[t]}) {
      const uintptr_t at = reinterpret_cast<uintptr_t>(p), end = at + bytes;
      if ((at < ne && nb < end) || (at < we && wb < end))
        return fail(QNF4_ERR_ARG, "norm or the workspace overlaps tensor %d", t);
    }
  }
  return QNF4_OK;
}

qnf4_status check_grad_args(int32_t count, const void* const* g, const int32_t* dtype, const int64_t* elems,
                            int32_t n, void* const* out, const float* norm) {
  if (count < 0) return fail(QNF4_ERR_ARG, "count must be >= 0 (got %d)", count);
  if (n < 1) return fail(QNF4_ERR_ARG, "n must be positive (got %d)", n);
  if (count > 0 && (!g || !dtype || !elems)) return fail(QNF4_ERR_ARG, "NULL array");
  if (!norm) return fail(QNF4_ERR_ARG, "NULL norm");
  if (!al16(norm)) return fail(QNF4_ERR_ALIGN, "norm must be 16-byte aligned");
  for (int32_t t = 0; t < count; ++t) {
    if (dtype[t] != QNF4_OUT_F32 && dtype[t] != QNF4_OUT_BF16)
      return fail(QNF4_ERR_ARG, "tensor %d: dtype must be fp32 or bf16", t);
    if (elems[t] < 0 || elems[t] % n)
      return fail(QNF4_ERR_SHAPE, "tensor %d: %lld elements are not %d equal parts", t, (long long)elems[t], n);
    if (elems[t] == 0) continue;
    if (!g[t] || (out && !out[t])) return fail(QNF4_ERR_ARG, "tensor %d: NULL buffer", t);
    const uintptr_t es = dtype[t] == QNF4_OUT_BF16 ? 2 : 4;
    if (reinterpret_cast<uintptr_t>(g[t]) % es || (out && reinterpret_cast<uintptr_t>(out[t]) % es))
      return fail(QNF4_ERR_ALIGN, "tensor %d: not aligned to its element size", t);
  }
  return out ? check_grad_outputs(count, g, dtype, elems, out) : QNF4_OK;
}

// The launches' table of tensors [t0, t0 + count).
template <int CAP>
void grad_tab(GradTab<CAP>* tab, int32_t t0, int32_t count, const void* const* g, const int32_t* dtype,
              const int64_t* elems, int32_t n, void* const* out, int piece, int64_t base, int64_t pieces) {
  std::memset(tab->bf16, 0, sizeof(tab->bf16));
  tab->piece = piece;
  tab->count = count;
  tab->n = n;
  tab->base = base;
  tab->pieces = pieces;
  tab->piece0[0] = 0;
  for (int32_t i = 0; i < count; ++i) {
    const int32_t t = t0 + i;
    tab->in[i] = g[t];
    tab->out[i] = out ? out[t] : nullptr;
    tab->part[i] = elems[t] / n;
    tab->piece0[i + 1] = tab->piece0[i] + (tab->part[i] + piece - 1) / piece;
    if (dtype[t] == QNF4_OUT_BF16) tab->bf16[i >> 5] |= 1u << (i & 31);
  }
}

template <int CAP>
qnf4_status grad_norm_clip_in(int32_t count, const void* const* g, const int32_t* dtype, const int64_t* elems,
                           int32_t n, float max_norm, void* const* out, float* norm, void* ws,
                           size_t ws_bytes, cudaStream_t s) {
  const size_t need = grad_ws_bytes(count, elems, n);
  if (!ws || !al16(ws) || ws_bytes < need)
    return fail(QNF4_ERR_WORKSPACE, "workspace too small or not 16-byte aligned (%zu < %zu)", ws_bytes, need);
  const qnf4_status st = check_grad_apart(count, g, dtype, elems, n, out, norm, ws, need);
  if (st != QNF4_OK) return st;
  const int64_t pieces = grad_pieces(count, elems, n);
  double* sums = static_cast<double*>(ws);
  float* coef = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) +
                                         align256(static_cast<size_t>(pieces) * n * sizeof(double)));
  static thread_local GradTab<CAP> tab;  // up to 16 KB: kept off the stack
  int launches = 0;
  const int piece = grad_piece_size(count, elems);
  // (a list cut over several launches would have its norms added up in each)
  const bool few = grad_few(pieces, n) && count <= CAP;
  auto pass = [&](bool scale) {
    int64_t base = 0;
    for (int32_t t0 = 0; t0 < count; t0 += CAP) {
      grad_tab<CAP>(&tab, t0, std::min(CAP, count - t0), g, dtype, elems, n, out, piece, base, pieces);
      const int64_t per = tab.piece0[tab.count];
      base += per;
      if (per == 0) continue;
      const int64_t ctas = (per * n + kGradWarps - 1) / kGradWarps;
      const dim3 grid(static_cast<unsigned>(std::min<int64_t>(ctas, num_sms() * 8)));
      if (scale)
        launch_pdl(k_grad_scale<CAP>, grid, dim3(32 * kGradWarps), 0, s, tab,
                   few ? static_cast<const float*>(nullptr) : static_cast<const float*>(coef),
                   static_cast<const double*>(sums), max_norm, norm);
      else
        launch_pdl(k_grad_sq<CAP>, grid, dim3(32 * kGradWarps), 0, s, tab, sums);
      ++launches;
    }
  };
  pass(false);
  if (!out || !few || pieces == 0) {
    launch_pdl(k_grad_norm, dim3(static_cast<unsigned>(n)), dim3(512), 0, s, static_cast<const double*>(sums),
               pieces, max_norm, few ? 1 : 0, norm, out && !few ? coef : static_cast<float*>(nullptr));
    ++launches;
  }
  if (out) pass(true);
  return launched(out ? "clip_grad_norm" : "grad_norm", launches);
}

qnf4_status grad_norm_clip(int32_t count, const void* const* g, const int32_t* dtype, const int64_t* elems,
                           int32_t n, float max_norm, void* const* out, float* norm, void* ws,
                           size_t ws_bytes, cudaStream_t s) {
  return count <= kGradFewTensors
             ? grad_norm_clip_in<kGradFewTensors>(count, g, dtype, elems, n, max_norm, out, norm, ws, ws_bytes, s)
             : grad_norm_clip_in<kGradMaxTensors>(count, g, dtype, elems, n, max_norm, out, norm, ws, ws_bytes, s);
}

}  // namespace
}  // namespace qnf4

using namespace qnf4;

// NVTX range around each ABI call (named after the call), for timeline tools; a
// no-op unless a tool is attached to the process.
struct TraceRange {
  explicit TraceRange(const char* name) { nvtxRangePushA(name); }
  ~TraceRange() { nvtxRangePop(); }
  TraceRange(const TraceRange&) = delete;
  TraceRange& operator=(const TraceRange&) = delete;
};

extern "C" {

qnf4_status qnf4_nf4_codebook(float levels[16], float thresholds[15]) {
  const Nf4Tables& t = nf4_tables();
  if (levels) std::memcpy(levels, t.levels, 16 * sizeof(float));
  if (thresholds) std::memcpy(thresholds, t.thr, 15 * sizeof(float));
  return QNF4_OK;
}

const char* qnf4_last_error(void) { return g_last.c_str(); }

unsigned long long qnf4_launch_count(void) { return g_launches.load(std::memory_order_relaxed); }


qnf4_status qnf4_set_timing_events(void* start, void* stop) {
  if ((start == nullptr) != (stop == nullptr)) return fail(QNF4_ERR_ARG, "give both events or neither");
  g_ev_start = static_cast<cudaEvent_t>(start);
  g_ev_stop = static_cast<cudaEvent_t>(stop);
  return QNF4_OK;
}

qnf4_status qnf4_set_wait_timeout_ns(uint64_t ns) {
  if (ns == 0) return fail(QNF4_ERR_ARG, "timeout must be positive");
  g_wait_ns = ns;
  return QNF4_OK;
}

qnf4_status qnf4_check(void* stream) {
  TraceRange trace_("qnf4_check");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return fail(QNF4_ERR_CUDA, "stream: %s", cudaGetErrorString(e));
  unsigned int flag = 0;
  e = cudaMemcpyFromSymbol(&flag, g_qnf4_err, sizeof(flag));
  if (e != cudaSuccess) return fail(QNF4_ERR_CUDA, "error flag: %s", cudaGetErrorString(e));
  if (flag) {
    const unsigned int zero = 0;
    cudaMemcpyToSymbol(g_qnf4_err, &zero, sizeof(zero));
    if (flag == kErrEigensolve) return fail(QNF4_ERR_CUDA, "LoftQ eigensolve failed (cuSOLVER info != 0)");
    if (flag >= kErrBoundsBase)
      return fail(QNF4_ERR_BOUNDS, "a kernel index fell outside its buffer (site %u)", flag - kErrBoundsBase);
    return fail(QNF4_ERR_TIMEOUT, "a kernel wait gave up (site %u)", flag);
  }
  return QNF4_OK;
}

size_t qnf4_workspace_size(int32_t op, int64_t N, int64_t K, int64_t M, int32_t r) {
  switch (op) {
    case QNF4_OP_QUANTIZE: return kQuantMaxGrid * sizeof(double);
    case QNF4_OP_LAYER_STATS: return 2 * kQuantMaxGrid * sizeof(double);
    case QNF4_OP_QUANTIZE_WEIGHT: return 2 * kQuantMaxGrid * sizeof(double);
    case QNF4_OP_QUANTIZE_WEIGHT_GROUP: return 2 * kQMaxJobs * kQuantMaxGrid * sizeof(double);
    case QNF4_OP_LAYER_STATS_GROUP: return 2 * kQMaxJobs * kQuantMaxGrid * sizeof(double);
    case QNF4_OP_DOUBLE_QUANT: return kDqPartials * sizeof(double);
    case QNF4_OP_FWD: {
      const size_t t = plan_linear(A_NF4_K, N, K, M, r, false, num_sms()).total;
      return M <= kDecodeMaxTokens ? std::max(t, decode_ws_bytes(K, M, r)) : t;
    }
    case QNF4_OP_BWD: return plan_linear(A_NF4_MN, N, K, M, r, true, num_sms()).total;
    case QNF4_OP_CHANQ_FWD: return plan_linear(A_CHANQ_K, N, K, M, r, false, num_sms()).total;
    case QNF4_OP_LOFTQ: return loftq_layout(N, K, r).total;
    case QNF4_OP_CHANQ_BWD: {
      const size_t t = plan_linear(A_CHANQ_MN, N, K, M, r, true, num_sms()).total;
      return t + chanq_wide_bytes(N, K);
    }
    default: return 0;
  }
}

qnf4_status qnf4_nf4_quantize(const void* W, int64_t N, int64_t K, int32_t block1, uint8_t* packed,
                              float* absmax, double* sse, void* ws, size_t ws_bytes, void* stream) {
  TraceRange trace_("qnf4_nf4_quantize");
  if (block1 != 64) return fail(QNF4_ERR_ARG, "block1 must be 64");
  if (N < 0 || K <= 0) return fail(QNF4_ERR_SHAPE, "bad shape");
  if (K % 64) return fail(QNF4_ERR_SHAPE, "K must be a multiple of 64");
  if (!W || !packed || !absmax) return fail(QNF4_ERR_ARG, "NULL buffer");
  if (!al16(W) || !al16(packed) || !al16(absmax) || (sse && !al16(sse)))
    return fail(QNF4_ERR_ALIGN, "buffers must be 16-byte aligned");
  if (sse && (!ws || ws_bytes < qnf4_workspace_size(QNF4_OP_QUANTIZE, N, K, 0, 0)))
    return fail(QNF4_ERR_WORKSPACE, "workspace too small");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t nblocks = N * K / 64;
  if (nblocks == 0) {
    if (sse) cudaMemsetAsync(sse, 0, sizeof(double), s);
    return launched("quantize(empty)", 0);
  }
  qnf4_status st = quant_smem_attr();
  if (st != QNF4_OK) return st;
  const int grid = quant_grid(nblocks);
  static thread_local QuantJobs jobs;
  if (!one_quant_job(&jobs, W, nblocks, packed, absmax)) return map_fail();
  const QuantTab tab = make_tab();
  if (sse) {
    launch_pdl(k_nf4_quant<true, true>, dim3(grid), dim3(kQThreads), kQSmem, s, jobs,
               static_cast<double*>(ws), tab, g_wait_ns, 0.f, static_cast<double*>(nullptr),
               static_cast<double*>(nullptr));
    launch_pdl(k_sum_partials, dim3(1), dim3(256), 0, s, static_cast<const double*>(ws), grid, sse);
    return launched("nf4_quantize", 2);
  }
  launch_pdl(k_nf4_quant<true, false>, dim3(grid), dim3(kQThreads), kQSmem, s, jobs,
             static_cast<double*>(nullptr), tab, g_wait_ns, 0.f, static_cast<double*>(nullptr),
             static_cast<double*>(nullptr));
  return launched("nf4_quantize");
}

qnf4_status qnf4_quantize_weight(const void* W, int64_t N, int64_t K, uint8_t* packed, float* absmax,
                                 uint8_t* code2, float* scale2, float* mean, double* sse, void* ws,
                                 size_t ws_bytes, void* stream) {
  TraceRange trace_("qnf4_quantize_weight");
  if (N <= 0 || K <= 0) return fail(QNF4_ERR_SHAPE, "N and K must be positive");
  if (K % 64) return fail(QNF4_ERR_SHAPE, "K must be a multiple of 64");
  if (!W || !packed || !absmax || !code2 || !scale2 || !mean) return fail(QNF4_ERR_ARG, "NULL buffer");
  for (const void* p : {W, static_cast<const void*>(packed), static_cast<const void*>(absmax),
                        static_cast<const void*>(code2), static_cast<const void*>(scale2),
                        static_cast<const void*>(mean)})
    if (!al16(p)) return fail(QNF4_ERR_ALIGN, "buffers must be 16-byte aligned");
  if (sse && !al16(sse)) return fail(QNF4_ERR_ALIGN, "buffers must be 16-byte aligned");
  if (!ws || ws_bytes < qnf4_workspace_size(QNF4_OP_QUANTIZE_WEIGHT, N, K, 0, 0))
    return fail(QNF4_ERR_WORKSPACE, "workspace too small");
  qnf4_status st = quant_smem_attr();
  if (st != QNF4_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t nblocks = N * K / 64;
  const int grid = quant_grid(nblocks);
  static thread_local QuantJobs jobs;
  if (!one_quant_job(&jobs, W, nblocks, packed, absmax)) return map_fail();
  double* asum = static_cast<double*>(ws);
  double* ssep = asum + kQuantMaxGrid;
  const QuantTab tab = make_tab();
  if (sse) {
    launch_pdl(k_nf4_quant<true, true>, dim3(grid), dim3(kQThreads), kQSmem, s, jobs, ssep, tab,
               g_wait_ns, 0.f, static_cast<double*>(nullptr), asum);
  } else {
    launch_pdl(k_nf4_quant<true, false>, dim3(grid), dim3(kQThreads), kQSmem, s, jobs,
               static_cast<double*>(nullptr), tab, g_wait_ns, 0.f, static_cast<double*>(nullptr), asum);
  }
  static thread_local DqJobs dq;
  const int egrid = one_dq_job(&dq, absmax, nblocks, asum, grid, nblocks, code2, scale2, mean,
                               sse ? ssep : nullptr, grid, sse);
  launch_pdl(k_dq_encode, dim3(egrid), dim3(256), 0, s, dq);
  return launched("quantize_weight", 2);
}

qnf4_status qnf4_quantize_weight_group(int32_t n, const void* const* W, const int64_t* N,
                                       const int64_t* K, uint8_t* const* packed, float* const* absmax,
                                       uint8_t* const* code2, float* const* scale2, float* const* mean,
                                       double* const* sse, void* ws, size_t ws_bytes, void* stream) {
  TraceRange trace_("qnf4_quantize_weight_group");
  if (n < 1 || n > kQMaxJobs) return fail(QNF4_ERR_ARG, "n must be in [1, %d] (got %d)", kQMaxJobs, n);
  if (!W || !N || !K || !packed || !absmax || !code2 || !scale2 || !mean) return fail(QNF4_ERR_ARG, "NULL array");
  for (int l = 0; l < n; ++l) {
    if (N[l] <= 0 || K[l] <= 0) return fail(QNF4_ERR_SHAPE, "weight %d: N and K must be positive", l);
    if (K[l] % 64) return fail(QNF4_ERR_SHAPE, "weight %d: K must be a multiple of 64", l);
    if (!W[l] || !packed[l] || !absmax[l] || !code2[l] || !scale2[l] || !mean[l] || (sse && !sse[l]))
      return fail(QNF4_ERR_ARG, "weight %d: NULL buffer", l);
    for (const void* p : {W[l], static_cast<const void*>(packed[l]), static_cast<const void*>(absmax[l]),
                          static_cast<const void*>(code2[l]), static_cast<const void*>(scale2[l]),
                          static_cast<const void*>(mean[l]), static_cast<const void*>(sse ? sse[l] : nullptr)})
      if (p && !al16(p)) return fail(QNF4_ERR_ALIGN, "buffers must be 16-byte aligned");
  }
  if (!ws || ws_bytes < qnf4_workspace_size(QNF4_OP_QUANTIZE_WEIGHT_GROUP, 0, 0, 0, 0))
    return fail(QNF4_ERR_WORKSPACE, "workspace too small");
  qnf4_status st = quant_smem_attr();
  if (st != QNF4_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  static thread_local QuantJobs jobs;
  static thread_local DqJobs dq;
  std::memset(&jobs, 0, sizeof(jobs));
  std::memset(&dq, 0, sizeof(dq));
  jobs.n = dq.n = n;
  jobs.chunk0[0] = dq.b2_0[0] = 0;
  double* asum = static_cast<double*>(ws);
  double* ssep = asum + kQMaxJobs * kQuantMaxGrid;
  for (int l = 0; l < n; ++l) {
    const int64_t nb = N[l] * K[l] / 64;
    jobs.nblocks[l] = nb;
    jobs.chunk0[l + 1] = jobs.chunk0[l] + (nb + kQChunkBlocks - 1) / kQChunkBlocks;
    jobs.packed[l] = reinterpret_cast<uint32_t*>(packed[l]);
    jobs.absmax[l] = absmax[l];
    if (!quant_map(&jobs.map[l], W[l], nb)) return map_fail();
    dq.c[l] = absmax[l];
    dq.nb1[l] = nb;
    dq.count[l] = nb;
    dq.part[l] = asum + l * kQuantMaxGrid;
    dq.code2[l] = code2[l];
    dq.scale2[l] = scale2[l];
    dq.mean[l] = mean[l];
    dq.sse_part[l] = ssep + l * kQuantMaxGrid;
    dq.sse_out[l] = sse ? sse[l] : nullptr;
    dq.b2_0[l + 1] = dq.b2_0[l] + (nb + 255) / 256;
  }
  const int grid = quant_grid_chunks(jobs.chunk0[n]);
  dq.npart = dq.nsse = grid;
  const QuantTab tab = make_tab();
  if (sse) {
    launch_pdl(k_nf4_quant<true, true>, dim3(grid), dim3(kQThreads), kQSmem, s, jobs, ssep, tab,
               g_wait_ns, 0.f, static_cast<double*>(nullptr), asum);
  } else {
    launch_pdl(k_nf4_quant<true, false>, dim3(grid), dim3(kQThreads), kQSmem, s, jobs,
               static_cast<double*>(nullptr), tab, g_wait_ns, 0.f, static_cast<double*>(nullptr), asum);
  }
  const int egrid = std::max(dq_grid(&dq, dq.b2_0[n]), n);  // CTA l < n folds weight l's SSE
  launch_pdl(k_dq_encode, dim3(egrid), dim3(256), 0, s, dq);
  return launched("quantize_weight_group", 2);
}

qnf4_status qnf4_nf4_layer_stats_group(int32_t n, const void* const* W, const int64_t* N,
                                       const int64_t* K, float tau, double* const* sse,
                                       double* const* below, void* ws, size_t ws_bytes, void* stream) {
  TraceRange trace_("qnf4_nf4_layer_stats_group");
  if (n < 1 || n > kQMaxJobs) return fail(QNF4_ERR_ARG, "n must be in [1, %d] (got %d)", kQMaxJobs, n);
  if (!W || !N || !K || !sse) return fail(QNF4_ERR_ARG, "NULL array");
  if (below && (!(tau >= 0.f) || std::isinf(tau))) return fail(QNF4_ERR_ARG, "tau must be finite and >= 0");
  for (int l = 0; l < n; ++l) {
    if (N[l] <= 0 || K[l] <= 0) return fail(QNF4_ERR_SHAPE, "weight %d: N and K must be positive", l);
    if (K[l] % 64) return fail(QNF4_ERR_SHAPE, "weight %d: K must be a multiple of 64", l);
    if (!W[l] || !sse[l] || (below && !below[l])) return fail(QNF4_ERR_ARG, "weight %d: NULL buffer", l);
    if (!al16(W[l]) || !al16(sse[l]) || (below && !al16(below[l])))
      return fail(QNF4_ERR_ALIGN, "buffers must be 16-byte aligned");
  }
  if (!ws || ws_bytes < qnf4_workspace_size(QNF4_OP_LAYER_STATS_GROUP, 0, 0, 0, 0))
    return fail(QNF4_ERR_WORKSPACE, "workspace too small");
  qnf4_status st = quant_smem_attr();
  if (st != QNF4_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  static thread_local QuantJobs jobs;
  std::memset(&jobs, 0, sizeof(jobs));
  jobs.n = n;
  SumJobs sj;
  std::memset(&sj, 0, sizeof(sj));
  for (int l = 0; l < n; ++l) {
    const int64_t nb = N[l] * K[l] / 64;
    jobs.nblocks[l] = nb;
    jobs.chunk0[l + 1] = jobs.chunk0[l] + (nb + kQChunkBlocks - 1) / kQChunkBlocks;
    if (!quant_map(&jobs.map[l], W[l], nb)) return map_fail();
    sj.out[l] = sse[l];
  }
  const int grid = quant_grid_chunks(jobs.chunk0[n]);
  double* part = static_cast<double*>(ws);  // SSE partials, then the counts', per job
  const QuantTab tab = make_tab();
  if (below) {
    launch_pdl(k_nf4_quant<false, true, true>, dim3(grid), dim3(kQThreads), kQSmem, s, jobs, part, tab,
               g_wait_ns, tau, part + kQMaxJobs * kQuantMaxGrid, static_cast<double*>(nullptr));
  } else {
    launch_pdl(k_nf4_quant<false, true>, dim3(grid), dim3(kQThreads), kQSmem, s, jobs, part, tab,
               g_wait_ns, 0.f, static_cast<double*>(nullptr), static_cast<double*>(nullptr));
  }
  launch_pdl(k_sum_partials_jobs, dim3(n), dim3(256), 0, s, static_cast<const double*>(part), grid, sj);
  if (below) {
    SumJobs sj2;
    std::memset(&sj2, 0, sizeof(sj2));
    for (int l = 0; l < n; ++l) sj2.out[l] = below[l];
    launch_pdl(k_sum_partials_jobs, dim3(n), dim3(256), 0, s,
               static_cast<const double*>(part + kQMaxJobs * kQuantMaxGrid), grid, sj2);
  }
  return launched("nf4_layer_stats_group", below ? 3 : 2);
}

qnf4_status qnf4_nf4_recon_error(const void* W, int64_t N, int64_t K, int32_t block1, double* sse,
                                 void* ws, size_t ws_bytes, void* stream) {
  TraceRange trace_("qnf4_nf4_recon_error");
  if (block1 != 64) return fail(QNF4_ERR_ARG, "block1 must be 64");
  if (N < 0 || K <= 0) return fail(QNF4_ERR_SHAPE, "bad shape");
  if (K % 64) return fail(QNF4_ERR_SHAPE, "K must be a multiple of 64");
  if (!W || !sse) return fail(QNF4_ERR_ARG, "NULL buffer");
  if (!al16(W) || !al16(sse)) return fail(QNF4_ERR_ALIGN, "buffers must be 16-byte aligned");
  if (!ws || ws_bytes < qnf4_workspace_size(QNF4_OP_QUANTIZE, N, K, 0, 0))
    return fail(QNF4_ERR_WORKSPACE, "workspace too small");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t nblocks = N * K / 64;
  if (nblocks == 0) {
    cudaMemsetAsync(sse, 0, sizeof(double), s);
    return launched("recon_error(empty)", 0);
  }
  qnf4_status st = quant_smem_attr();
  if (st != QNF4_OK) return st;
  const int grid = quant_grid(nblocks);
  static thread_local QuantJobs jobs;
  if (!one_quant_job(&jobs, W, nblocks, nullptr, nullptr)) return map_fail();
  launch_pdl(k_nf4_quant<false, true>, dim3(grid), dim3(kQThreads), kQSmem, s, jobs,
             static_cast<double*>(ws), make_tab(), g_wait_ns, 0.f, static_cast<double*>(nullptr),
             static_cast<double*>(nullptr));
  launch_pdl(k_sum_partials, dim3(1), dim3(256), 0, s, static_cast<const double*>(ws), grid, sse);
  return launched("nf4_recon_error", 2);
}

qnf4_status qnf4_nf4_layer_stats(const void* W, int64_t N, int64_t K, float tau, double* sse,
                                 double* below, void* ws, size_t ws_bytes, void* stream) {
  TraceRange trace_("qnf4_nf4_layer_stats");
  if (N < 0 || K <= 0) return fail(QNF4_ERR_SHAPE, "bad shape");
  if (K % 64) return fail(QNF4_ERR_SHAPE, "K must be a multiple of 64");
  if (!W || !sse || !below) return fail(QNF4_ERR_ARG, "NULL buffer");
  if (!al16(W) || !al16(sse) || !al16(below)) return fail(QNF4_ERR_ALIGN, "buffers must be 16-byte aligned");
  if (!(tau >= 0.f) || std::isinf(tau)) return fail(QNF4_ERR_ARG, "tau must be finite and >= 0");
  if (!ws || ws_bytes < qnf4_workspace_size(QNF4_OP_LAYER_STATS, N, K, 0, 0))
    return fail(QNF4_ERR_WORKSPACE, "workspace too small");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t nblocks = N * K / 64;
  if (nblocks == 0) {
    cudaMemsetAsync(sse, 0, sizeof(double), s);
    cudaMemsetAsync(below, 0, sizeof(double), s);
    return launched("layer_stats(empty)", 0);
  }
  qnf4_status st = quant_smem_attr();
  if (st != QNF4_OK) return st;
  const int grid = quant_grid(nblocks);
  static thread_local QuantJobs jobs;
  if (!one_quant_job(&jobs, W, nblocks, nullptr, nullptr)) return map_fail();
  double* part = static_cast<double*>(ws);
  launch_pdl(k_nf4_quant<false, true, true>, dim3(grid), dim3(kQThreads), kQSmem, s, jobs, part,
             make_tab(), g_wait_ns, tau, part + kQuantMaxGrid, static_cast<double*>(nullptr));
  launch_pdl(k_sum_partials, dim3(1), dim3(256), 0, s, part, grid, sse);
  launch_pdl(k_sum_partials, dim3(1), dim3(256), 0, s, part + kQuantMaxGrid, grid, below);
  return launched("nf4_layer_stats", 3);
}

qnf4_status qnf4_double_quant(const float* absmax, int64_t nb1, int32_t block2, uint8_t* code2,
                              float* scale2, float* mean, void* ws, size_t ws_bytes, void* stream) {
  TraceRange trace_("qnf4_double_quant");
  if (block2 != 256) return fail(QNF4_ERR_ARG, "block2 must be 256");
  if (nb1 <= 0) return fail(QNF4_ERR_SHAPE, "nb1 must be positive");
  if (!absmax || !code2 || !scale2 || !mean) return fail(QNF4_ERR_ARG, "NULL buffer");
  if (!al16(absmax) || !al16(code2) || !al16(scale2) || !al16(mean))
    return fail(QNF4_ERR_ALIGN, "buffers must be 16-byte aligned");
  if (!ws || ws_bytes < qnf4_workspace_size(QNF4_OP_DOUBLE_QUANT, 0, 0, 0, 0))
    return fail(QNF4_ERR_WORKSPACE, "workspace too small");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  double* part = static_cast<double*>(ws);
  k_dq_partial<<<kDqPartials, 256, 0, s>>>(absmax, nb1, part);
  static thread_local DqJobs dq;
  const int grid = one_dq_job(&dq, absmax, nb1, part, kDqPartials, nb1, code2, scale2, mean, nullptr, 0, nullptr);
  launch_pdl(k_dq_encode, dim3(grid), dim3(256), 0, s, dq);
  return launched("double_quant", 2);
}

qnf4_status qnf4_dq_sum(const float* absmax, int64_t nb1, double* sum, void* ws, size_t ws_bytes,
                        void* stream) {
  TraceRange trace_("qnf4_dq_sum");
  if (nb1 <= 0) return fail(QNF4_ERR_SHAPE, "nb1 must be positive");
  if (!absmax || !sum) return fail(QNF4_ERR_ARG, "NULL buffer");
  if (!al16(absmax) || !al16(sum)) return fail(QNF4_ERR_ALIGN, "buffers must be 16-byte aligned");
  if (!ws || ws_bytes < qnf4_workspace_size(QNF4_OP_DOUBLE_QUANT, 0, 0, 0, 0))
    return fail(QNF4_ERR_WORKSPACE, "workspace too small");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  double* part = static_cast<double*>(ws);
  k_dq_partial<<<kDqPartials, 256, 0, s>>>(absmax, nb1, part);
  launch_pdl(k_sum_partials, dim3(1), dim3(256), 0, s, part, kDqPartials, sum);
  return launched("dq_sum", 2);
}

qnf4_status qnf4_double_quant_shard(const float* absmax, int64_t nb1, int32_t block2,
                                    const double* total_sum, int64_t total_count, uint8_t* code2,
                                    float* scale2, float* mean, void* stream) {
  TraceRange trace_("qnf4_double_quant_shard");
  if (block2 != 256) return fail(QNF4_ERR_ARG, "block2 must be 256");
  if (nb1 <= 0) return fail(QNF4_ERR_SHAPE, "nb1 must be positive");
  if (total_count < nb1) return fail(QNF4_ERR_SHAPE, "total_count must be >= nb1");
  if (!absmax || !total_sum || !code2 || !scale2 || !mean) return fail(QNF4_ERR_ARG, "NULL buffer");
  if (!al16(absmax) || !al16(total_sum) || !al16(code2) || !al16(scale2) || !al16(mean))
    return fail(QNF4_ERR_ALIGN, "buffers must be 16-byte aligned");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  static thread_local DqJobs dq;
  const int grid = one_dq_job(&dq, absmax, nb1, total_sum, 1, total_count, code2, scale2, mean, nullptr, 0, nullptr);
  launch_pdl(k_dq_encode, dim3(grid), dim3(256), 0, s, dq);
  return launched("dq_encode_shard");
}

qnf4_status qnf4_dequant(const qnf4_weight* w, void* out, int32_t out_dtype, void* stream) {
  TraceRange trace_("qnf4_dequant");
  qnf4_status st = check_weight(w);
  if (st != QNF4_OK) return st;
  if (!out) return fail(QNF4_ERR_ARG, "NULL output");
  if (!al16(out)) return fail(QNF4_ERR_ALIGN, "output must be 16-byte aligned");
  if (out_dtype != QNF4_OUT_F32 && out_dtype != QNF4_OUT_BF16)
    return fail(QNF4_ERR_ARG, "out_dtype must be QNF4_OUT_F32 or QNF4_OUT_BF16");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t n8 = w->N * w->K / 8;
  const int grid = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>((n8 + 255) / 256, num_sms() * 8)));
  const QuantTab tab = make_tab();
  const uint32_t* p = reinterpret_cast<const uint32_t*>(w->packed);
  if (out_dtype == QNF4_OUT_BF16)
    k_dequant<true><<<grid, 256, 0, s>>>(p, w->code2, w->scale2, w->mean, n8, out, tab);
  else
    k_dequant<false><<<grid, 256, 0, s>>>(p, w->code2, w->scale2, w->mean, n8, out, tab);
  return launched("dequant");
}

qnf4_status qnf4_rank_topk(const double* sse, const int64_t* n_params, int32_t n_layers, int32_t k,
                           int32_t* out) {
  if (!sse || !n_params || (!out && k > 0)) return fail(QNF4_ERR_ARG, "NULL host buffer");
  if (n_layers < 0 || k < 0 || k > n_layers) return fail(QNF4_ERR_ARG, "need 0 <= k <= n_layers");
  std::vector<int32_t> idx(n_layers);
  for (int32_t i = 0; i < n_layers; ++i) {
    if (n_params[i] <= 0) return fail(QNF4_ERR_ARG, "n_params must be positive");
    idx[i] = i;
  }
  // epsilon_i = sse_i / n_i, descending; ties to the lower index (stable)
  std::stable_sort(idx.begin(), idx.end(), [&](int32_t a, int32_t b) {
    return sse[a] / static_cast<double>(n_params[a]) > sse[b] / static_cast<double>(n_params[b]);
  });
  for (int32_t i = 0; i < k; ++i) out[i] = idx[i];
  return QNF4_OK;
}

qnf4_status qnf4_chanq_quantize(const void* W, int64_t N, int64_t K, const uint8_t* bits,
                                const float* thr, const int64_t* thr_off, uint8_t* packed,
                                const int64_t* row_off, float* absmax, void* stream) {
  TraceRange trace_("qnf4_chanq_quantize");
  if (N < 0 || K <= 0) return fail(QNF4_ERR_SHAPE, "bad shape");
  if (K % 64) return fail(QNF4_ERR_SHAPE, "K must be a multiple of 64");
  if (!W || !bits || !thr || !thr_off || !packed || !row_off || !absmax)
    return fail(QNF4_ERR_ARG, "NULL buffer");
  if (!al16(W) || !al16(bits) || !al16(thr) || !al16(thr_off) || !al16(packed) || !al16(row_off) ||
      !al16(absmax))
    return fail(QNF4_ERR_ALIGN, "buffers must be 16-byte aligned");
  if (N == 0) return QNF4_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int grid = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>((N + 7) / 8, num_sms() * 8)));
  k_chanq_quant<<<grid, 256, 0, s>>>(static_cast<const uint16_t*>(W), N, K, bits, thr, thr_off,
                                     packed, row_off, absmax);
  return launched("chanq_quantize");
}

qnf4_status qnf4_qlora_linear_fwd(const qnf4_weight* w, const void* x, int64_t M, const void* A,
                                  const void* B, int32_t r, float scale, void* h, void* ws,
                                  size_t ws_bytes, void* stream) {
  TraceRange trace_("qnf4_qlora_linear_fwd");
  qnf4_status st = check_weight(w);
  if (st != QNF4_OK) return st;
  st = check_linear_args(w->N, w->K, M, r, false, {x, A, B, h});
  if (st != QNF4_OK) return st;
  if (M == 0) return QNF4_OK;
  if (M <= kDecodeMaxTokens)
    return decode_fwd(w, x, M, A, B, r, scale, h, ws, ws_bytes, static_cast<cudaStream_t>(stream));
  BaseSrc src;
  src.kind = A_NF4_K;
  src.w = w;
  src.N = w->N;
  src.K = w->K;
  return linear_fwd(src, x, M, A, B, r, scale, h, ws, ws_bytes, static_cast<cudaStream_t>(stream));
}

qnf4_status qnf4_qlora_linear_fwd_group(int32_t n, const qnf4_weight* w, const void* const* x,
                                        int64_t M, const void* const* A, const void* const* B,
                                        int32_t r, float scale, void* const* h, void* ws,
                                        size_t ws_bytes, void* stream) {
  TraceRange trace_("qnf4_qlora_linear_fwd_group");
  if (n < 1 || n > kDecMaxGroup) return fail(QNF4_ERR_ARG, "n must be in [1, %d] (got %d)", kDecMaxGroup, n);
  if (!w || !x || !A || !B || !h) return fail(QNF4_ERR_ARG, "NULL array");
  if (M < 1 || M > kDecodeMaxTokens)
    return fail(QNF4_ERR_SHAPE, "the grouped forward takes 1 to %lld tokens (got %lld)",
                static_cast<long long>(kDecodeMaxTokens), static_cast<long long>(M));
  size_t need = 0;
  for (int l = 0; l < n; ++l) {
    qnf4_status st = check_weight(&w[l]);
    if (st != QNF4_OK) return st;
    st = check_linear_args(w[l].N, w[l].K, M, r, false, {x[l], A[l], B[l], h[l]});
    if (st != QNF4_OK) return st;
    need += decode_ws_bytes(w[l].K, M, r);
  }
  if (!ws || ws_bytes < need) return fail(QNF4_ERR_WORKSPACE, "workspace too small (%zu < %zu)", ws_bytes, need);
  return decode_group(n, w, x, M, A, B, r, scale, h, ws, ws_bytes, static_cast<cudaStream_t>(stream));
}

qnf4_status qnf4_qlora_linear_fwd_noalloc(const qnf4_weight* w, const void* x, int64_t M,
                                          const void* A, const void* B, int32_t r, float scale,
                                          void* h, void* stream) {
  TraceRange trace_("qnf4_qlora_linear_fwd_noalloc");
  qnf4_status st = check_weight(w);
  if (st != QNF4_OK) return st;
  st = check_linear_args(w->N, w->K, M, r, false, {x, A, B, h});
  if (st != QNF4_OK) return st;
  if (M == 0) return QNF4_OK;
  const size_t need = qnf4_workspace_size(QNF4_OP_FWD, w->N, w->K, M, r);
  if (need > kNoAllocScratchBytes)
    return fail(QNF4_ERR_WORKSPACE,
                "this shape needs %zu bytes of workspace; the built-in scratch holds %zu "
                "(use qnf4_qlora_linear_fwd with a caller-provided workspace)",
                need, kNoAllocScratchBytes);
  void* ws = noalloc_scratch_ptr();
  if (!ws) return QNF4_ERR_CUDA;
  return qnf4_qlora_linear_fwd(w, x, M, A, B, r, scale, h, ws, kNoAllocScratchBytes, stream);
}

qnf4_status qnf4_qlora_linear_bwd(const qnf4_weight* w, const void* x, const void* dY, int64_t M,
                                  const void* A, const void* B, int32_t r, float scale, void* dX,
                                  float* dA, float* dB, void* ws, size_t ws_bytes, void* stream) {
  TraceRange trace_("qnf4_qlora_linear_bwd");
  qnf4_status st = check_weight(w);
  if (st != QNF4_OK) return st;
  st = check_linear_args(w->N, w->K, M, r, true, {x, dY, A, B, dX, dA, dB});
  if (st != QNF4_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (M == 0) {
    cudaMemsetAsync(dA, 0, sizeof(float) * r * w->K, s);
    cudaMemsetAsync(dB, 0, sizeof(float) * r * w->N, s);
    return launched("bwd(M=0)", 0);
  }
  BaseSrc src;
  src.kind = A_NF4_K;
  src.w = w;
  src.N = w->N;
  src.K = w->K;
  return linear_bwd(src, x, dY, M, A, B, r, scale, dX, dA, dB, ws, ws_bytes, s);
}

qnf4_status qnf4_dense_linear_fwd(const void* W, int64_t N, int64_t K, const void* x, int64_t M,
                                  const void* A, const void* B, int32_t r, float scale, void* h,
                                  void* ws, size_t ws_bytes, void* stream) {
  TraceRange trace_("qnf4_dense_linear_fwd");
  qnf4_status st = check_linear_args(N, K, M, r, false, {W, x, A, B, h});
  if (st != QNF4_OK) return st;
  if (M == 0) return QNF4_OK;
  BaseSrc src;
  src.kind = A_DENSE_K;
  src.Wd = W;
  src.N = N;
  src.K = K;
  return linear_fwd(src, x, M, A, B, r, scale, h, ws, ws_bytes, static_cast<cudaStream_t>(stream));
}

qnf4_status qnf4_dense_linear_bwd(const void* W, int64_t N, int64_t K, const void* x, const void* dY,
                                  int64_t M, const void* A, const void* B, int32_t r, float scale,
                                  void* dX, float* dA, float* dB, void* ws, size_t ws_bytes,
                                  void* stream) {
  TraceRange trace_("qnf4_dense_linear_bwd");
  qnf4_status st = check_linear_args(N, K, M, r, true, {W, x, dY, A, B, dX, dA, dB});
  if (st != QNF4_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (M == 0) {
    cudaMemsetAsync(dA, 0, sizeof(float) * r * K, s);
    cudaMemsetAsync(dB, 0, sizeof(float) * r * N, s);
    return launched("bwd(M=0)", 0);
  }
  BaseSrc src;
  src.kind = A_DENSE_K;
  src.Wd = W;
  src.N = N;
  src.K = K;
  return linear_bwd(src, x, dY, M, A, B, r, scale, dX, dA, dB, ws, ws_bytes, s);
}

qnf4_status qnf4_chanq_linear_fwd(const uint8_t* packed, const int64_t* row_off, const uint8_t* bits,
                                  const float* map, const int64_t* map_off, const float* absmax,
                                  int64_t N, int64_t K, const void* x, int64_t M, const void* A,
                                  const void* B, int32_t r, float scale, void* h, void* ws,
                                  size_t ws_bytes, void* stream) {
  TraceRange trace_("qnf4_chanq_linear_fwd");
  qnf4_status st = check_linear_args(N, K, M, r, false, {packed, row_off, bits, map, map_off, absmax, x, A, B, h});
  if (st != QNF4_OK) return st;
  if (M == 0) return QNF4_OK;
  BaseSrc src;
  src.kind = A_CHANQ_K;
  src.cq_packed = packed;
  src.cq_row_off = row_off;
  src.cq_bits = bits;
  src.cq_map = map;
  src.cq_map_off = map_off;
  src.cq_absmax = absmax;
  src.N = N;
  src.K = K;
  return linear_fwd(src, x, M, A, B, r, scale, h, ws, ws_bytes, static_cast<cudaStream_t>(stream));
}

qnf4_status qnf4_chanq_learn(const void* W_bf16, int64_t N, int64_t K, int32_t bits,
                             const float* thr0, int32_t iters, float* map, float* thr,
                             double* err, int32_t* iters_done, void* stream) {
  TraceRange trace_("qnf4_chanq_learn");
  for (const void* p : {W_bf16, static_cast<const void*>(thr0), static_cast<const void*>(map),
                        static_cast<const void*>(thr), static_cast<const void*>(err)}) {
    if (!p) return fail(QNF4_ERR_ARG, "NULL buffer");
    if (!al16(p)) return fail(QNF4_ERR_ALIGN, "buffers must be 16-byte aligned");
  }
  if (bits != 1 && bits != 2 && bits != 4) return fail(QNF4_ERR_ARG, "bits must be 1, 2 or 4 (got %d)", bits);
  if (iters < 1) return fail(QNF4_ERR_ARG, "iters must be >= 1");
  if (N < 0 || K <= 0 || K % 64) return fail(QNF4_ERR_SHAPE, "K must be a positive multiple of 64");
  if (K > 32768) return fail(QNF4_ERR_SHAPE, "K at most 32768 (the row lives in shared memory)");
  if (N == 0) return QNF4_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const size_t smem = static_cast<size_t>(K) * 4 + static_cast<size_t>(K / 64) * 4;
  const int grid = static_cast<int>(std::min<int64_t>(N, static_cast<int64_t>(num_sms()) * 4));
  auto go = [&](auto kern) -> qnf4_status {
    if (smem > 48 * 1024 &&
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
      return fail(QNF4_ERR_CUDA, "shared memory attribute refused");
    kern<<<grid, kLearnThreads, smem, s>>>(static_cast<const uint16_t*>(W_bf16), N, K, thr0, iters, map,
                                           thr, err, iters_done);
    return launched("chanq_learn");
  };
  if (bits == 1) return go(k_chanq_learn<2>);
  if (bits == 2) return go(k_chanq_learn<4>);
  return go(k_chanq_learn<16>);
}

qnf4_status qnf4_loftq_nf4(const void* W_bf16, int64_t N, int64_t K, int32_t r, int32_t steps,
                           uint8_t* packed, uint8_t* code2, float* scale2, float* mean, float* A,
                           float* B, double* errs, void* ws, size_t ws_bytes, void* stream) {
  TraceRange trace_("qnf4_loftq_nf4");
  for (const void* p : {W_bf16, static_cast<const void*>(packed), static_cast<const void*>(code2),
                        static_cast<const void*>(scale2), static_cast<const void*>(mean),
                        static_cast<const void*>(A), static_cast<const void*>(B),
                        static_cast<const void*>(errs)}) {
    if (!p) return fail(QNF4_ERR_ARG, "NULL buffer");
    if (!al16(p)) return fail(QNF4_ERR_ALIGN, "buffers must be 16-byte aligned");
  }
  if (N <= 0 || K <= 0 || K % 64) return fail(QNF4_ERR_SHAPE, "N > 0 and K a positive multiple of 64");
  if (r < 1 || r > std::min(N, K)) return fail(QNF4_ERR_ARG, "r must be in [1, min(N, K)]");
  if (steps < 1) return fail(QNF4_ERR_ARG, "steps must be >= 1");
  if (std::min(N, K) > 16384) return fail(QNF4_ERR_SHAPE, "min(N, K) at most 16384 (the Gram matrix)");
  cublasHandle_t hb;
  cusolverDnHandle_t hs;
  if (!linalg_handles(&hb, &hs)) return fail(QNF4_ERR_CUDA, "cuBLAS / cuSOLVER unavailable");
  const LoftqLayout l = loftq_layout(N, K, r);
  if (!ws || ws_bytes < l.total) return fail(QNF4_ERR_WORKSPACE, "workspace too small (%zu < %zu)", ws_bytes, l.total);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const LinAlgLib& L = linalg_lib();
  if (L.blas_stream(hb, s) != CUBLAS_STATUS_SUCCESS || L.sol_stream(hs, s) != CUSOLVER_STATUS_SUCCESS)
    return fail(QNF4_ERR_CUDA, "cuBLAS / cuSOLVER stream");
  uint8_t* w8 = static_cast<uint8_t*>(ws);
  uint16_t* tgt = reinterpret_cast<uint16_t*>(w8 + l.tgt);
  float* Q = reinterpret_cast<float*>(w8 + l.q);
  float* absmax = reinterpret_cast<float*>(w8 + l.absmax);
  float* G = reinterpret_cast<float*>(w8 + l.gram);
  float* eig = reinterpret_cast<float*>(w8 + l.eig);
  float* P = reinterpret_cast<float*>(w8 + l.p);
  int* info = reinterpret_cast<int*>(w8 + l.info);
  float* work = reinterpret_cast<float*>(w8 + l.work);
  const int64_t m = l.m;
  const bool gram_k = N >= K;  // Gram R^T R (K x K) when N >= K, else R R^T (N x N)
  cudaMemsetAsync(A, 0, sizeof(float) * r * K, s);
  cudaMemsetAsync(B, 0, sizeof(float) * N * r, s);
  qnf4_weight wq{N, K, 64, 256, packed, code2, scale2, mean};
  const int grid = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>((N * K + 255) / 256, num_sms() * 8)));
  const float one = 1.f, zero = 0.f;
  for (int t = 0; t < steps; ++t) {
    k_loftq_target<<<grid, 256, 0, s>>>(static_cast<const uint16_t*>(W_bf16), B, A, N, K, r, tgt);
    qnf4_status st = launched("loftq_target");
    if (st != QNF4_OK) return st;
    st = qnf4_nf4_quantize(tgt, N, K, 64, packed, absmax, nullptr, nullptr, 0, stream);
    if (st != QNF4_OK) return st;
    st = qnf4_double_quant(absmax, N * K / 64, 256, code2, scale2, mean, w8 + l.dq,
                           qnf4_workspace_size(QNF4_OP_DOUBLE_QUANT, 0, 0, 0, 0), stream);
    if (st != QNF4_OK) return st;
    st = qnf4_dequant(&wq, Q, QNF4_OUT_F32, stream);
    if (st != QNF4_OK) return st;
    k_loftq_residual<<<grid, 256, 0, s>>>(static_cast<const uint16_t*>(W_bf16), Q, N * K);
    st = launched("loftq_residual");
    if (st != QNF4_OK) return st;
    // R row-major [N, K] is column-major K x N with leading dimension K
    const cublasStatus_t g1 =
        gram_k ? L.sgemm(hb, CUBLAS_OP_N, CUBLAS_OP_T, static_cast<int>(K), static_cast<int>(K),
                         static_cast<int>(N), &one, Q, static_cast<int>(K), Q, static_cast<int>(K), &zero, G,
                         static_cast<int>(K))
               : L.sgemm(hb, CUBLAS_OP_T, CUBLAS_OP_N, static_cast<int>(N), static_cast<int>(N),
                         static_cast<int>(K), &one, Q, static_cast<int>(K), Q, static_cast<int>(K), &zero, G,
                         static_cast<int>(N));
    if (g1 != CUBLAS_STATUS_SUCCESS) return fail(QNF4_ERR_CUDA, "cuBLAS sgemm (Gram) failed");
    if (L.syevd(hs, CUSOLVER_EIG_MODE_VECTOR, CUBLAS_FILL_MODE_LOWER, static_cast<int>(m), G,
                static_cast<int>(m), eig, work, static_cast<int>(l.lwork), info) != CUSOLVER_STATUS_SUCCESS)
      return fail(QNF4_ERR_CUDA, "cuSOLVER syevd failed");
    const int fg = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>((m * r + 255) / 256, num_sms() * 4)));
    // top-r eigenvectors: Gram on the K side gives V (A = rho V^T, B = R V / rho), on the
    // N side U (B = rho U, A^T = R^T U / rho)
    k_loftq_factor<<<fg, 256, 0, s>>>(G, eig, m, r, P, gram_k ? A : B, gram_k ? 0 : 1);
    st = launched("loftq_factor");
    if (st != QNF4_OK) return st;
    const cublasStatus_t g2 =
        gram_k ? L.sgemm(hb, CUBLAS_OP_T, CUBLAS_OP_N, r, static_cast<int>(N), static_cast<int>(K), &one, P,
                         static_cast<int>(K), Q, static_cast<int>(K), &zero, B, r)
               : L.sgemm(hb, CUBLAS_OP_N, CUBLAS_OP_N, static_cast<int>(K), r, static_cast<int>(N), &one, Q,
                         static_cast<int>(K), P, static_cast<int>(N), &zero, A, static_cast<int>(K));
    if (g2 != CUBLAS_STATUS_SUCCESS) return fail(QNF4_ERR_CUDA, "cuBLAS sgemm (factor) failed");
    k_loftq_err<<<1, 256, 0, s>>>(eig, m, r, info, errs + t);
    st = launched("loftq_err");
    if (st != QNF4_OK) return st;
  }
  return QNF4_OK;
}

qnf4_status qnf4_chanq_linear_bwd(const uint8_t* packed, const int64_t* row_off, const uint8_t* bits,
                                  const float* map, const int64_t* map_off, const float* absmax,
                                  int64_t N, int64_t K, const void* x, const void* dY, int64_t M,
                                  const void* A, const void* B, int32_t r, float scale, void* dX,
                                  float* dA, float* dB, void* ws, size_t ws_bytes, void* stream) {
  TraceRange trace_("qnf4_chanq_linear_bwd");
  qnf4_status st = check_linear_args(N, K, M, r, true,
                                     {packed, row_off, bits, map, map_off, absmax, x, dY, A, B, dX, dA, dB});
  if (st != QNF4_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (M == 0) {
    cudaMemsetAsync(dA, 0, sizeof(float) * r * K, s);
    cudaMemsetAsync(dB, 0, sizeof(float) * r * N, s);
    return launched("bwd(M=0)", 0);
  }
  const size_t own = plan_linear(A_CHANQ_MN, N, K, M, r, true, num_sms()).total;
  if (!ws || ws_bytes < own + chanq_wide_bytes(N, K))
    return fail(QNF4_ERR_WORKSPACE, "workspace too small (%zu < %zu)", ws_bytes, own + chanq_wide_bytes(N, K));
  BaseSrc src;
  src.kind = A_CHANQ_K;
  src.cq_packed = packed;
  src.cq_row_off = row_off;
  src.cq_bits = bits;
  src.cq_map = map;
  src.cq_map_off = map_off;
  src.cq_absmax = absmax;
  src.cq_wide = static_cast<uint8_t*>(ws) + own;
  src.cq_tab = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + own +
                                        align256(static_cast<size_t>(N) * static_cast<size_t>(K / 2)));
  src.N = N;
  src.K = K;
  {
    const int grid = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>((N + 7) / 8, num_sms() * 8)));
    k_chanq_widen<<<grid, 256, 0, s>>>(packed, row_off, bits, map, map_off, N, K, src.cq_wide, src.cq_tab);
    st = launched("chanq_widen");
    if (st != QNF4_OK) return st;
  }
  return linear_bwd(src, x, dY, M, A, B, r, scale, dX, dA, dB, ws, own, s);
}

size_t qnf4_multi_workspace_size(int32_t op, int64_t N, int64_t K, int64_t M, int32_t n, int32_t r) {
  if (N < 1 || K < 1 || M < 1 || n < 1 || r < 1 || r > 64) return 0;
  // the NF4 and bf16 sources' plans differ in their rings and so in their slices
  if (op == QNF4_OP_FWD)
    return std::max({plan_multi(A_NF4_K, N, K, M, n, r, false, num_sms()).total,
                     plan_multi(A_DENSE_K, N, K, M, n, r, false, num_sms()).total,
                     M <= kDecodeMaxTokens ? decode_ws_bytes(K, M, r) : 0});
  if (op == QNF4_OP_BWD)
    return std::max(plan_multi(A_NF4_MN, N, K, M, n, r, true, num_sms()).total,
                    plan_multi(A_DENSE_MN, N, K, M, n, r, true, num_sms()).total);
  return 0;
}

qnf4_status qnf4_qlora_linear_multi_fwd(const qnf4_weight* w, const void* x, int64_t M, const int32_t* ids,
                                        int32_t n, const void* A, const void* B, int32_t r, const float* scales,
                                        void* h, void* ws, size_t ws_bytes, void* stream) {
  TraceRange trace_("qnf4_qlora_linear_multi_fwd");
  qnf4_status st = check_weight(w);
  if (st != QNF4_OK) return st;
  st = check_multi_args(w->N, w->K, M, n, r, false, {x, ids, A, B, scales, h});
  if (st != QNF4_OK) return st;
  if (M == 0) return QNF4_OK;
  if (M <= kDecodeMaxTokens)
    return decode_group(1, w, &x, M, &A, &B, r, 0.f, &h, ws, ws_bytes, static_cast<cudaStream_t>(stream), ids, n,
                        scales);
  BaseSrc src;
  src.kind = A_NF4_K;
  src.w = w;
  src.N = w->N;
  src.K = w->K;
  return multi_fwd(src, Adapters{ids, A, B, scales, n, r}, x, M, h, ws, ws_bytes, static_cast<cudaStream_t>(stream));
}

qnf4_status qnf4_qlora_linear_multi_fwd_group(int32_t k, const qnf4_weight* w, const void* const* x, int64_t M,
                                              const int32_t* ids, int32_t n, const void* const* A,
                                              const void* const* B, int32_t r, const float* scales,
                                              void* const* h, void* ws, size_t ws_bytes, void* stream) {
  TraceRange trace_("qnf4_qlora_linear_multi_fwd_group");
  if (k < 1 || k > kDecMaxGroup) return fail(QNF4_ERR_ARG, "the layers must be in [1, %d] (got %d)", kDecMaxGroup, k);
  if (!w || !x || !A || !B || !h) return fail(QNF4_ERR_ARG, "NULL array");
  if (M < 1 || M > kDecodeMaxTokens)
    return fail(QNF4_ERR_SHAPE, "the grouped forward takes 1 to %lld tokens (got %lld)",
                static_cast<long long>(kDecodeMaxTokens), static_cast<long long>(M));
  for (int l = 0; l < k; ++l) {
    qnf4_status st = check_weight(&w[l]);
    if (st != QNF4_OK) return st;
    st = check_multi_args(w[l].N, w[l].K, M, n, r, false, {x[l], ids, A[l], B[l], scales, h[l]});
    if (st != QNF4_OK) return st;
  }
  return decode_group(k, w, x, M, A, B, r, 0.f, h, ws, ws_bytes, static_cast<cudaStream_t>(stream), ids, n, scales);
}

qnf4_status qnf4_dense_linear_multi_fwd(const void* W, int64_t N, int64_t K, const void* x, int64_t M,
                                        const int32_t* ids, int32_t n, const void* A, const void* B, int32_t r,
                                        const float* scales, void* h, void* ws, size_t ws_bytes, void* stream) {
  TraceRange trace_("qnf4_dense_linear_multi_fwd");
  qnf4_status st = check_multi_args(N, K, M, n, r, false, {W, x, ids, A, B, scales, h});
  if (st != QNF4_OK) return st;
  if (M == 0) return QNF4_OK;
  BaseSrc src;
  src.kind = A_DENSE_K;
  src.Wd = W;
  src.N = N;
  src.K = K;
  return multi_fwd(src, Adapters{ids, A, B, scales, n, r}, x, M, h, ws, ws_bytes, static_cast<cudaStream_t>(stream));
}

qnf4_status qnf4_qlora_linear_multi_bwd(const qnf4_weight* w, const void* x, const void* dY, int64_t M,
                                        const int32_t* ids, int32_t n, const void* A, const void* B, int32_t r,
                                        const float* scales, void* dX, float* dA, float* dB, void* ws,
                                        size_t ws_bytes, void* stream) {
  TraceRange trace_("qnf4_qlora_linear_multi_bwd");
  qnf4_status st = check_weight(w);
  if (st != QNF4_OK) return st;
  st = check_multi_args(w->N, w->K, M, n, r, true, {x, dY, ids, A, B, scales, dX, dA, dB});
  if (st != QNF4_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (M == 0) {
    cudaMemsetAsync(dA, 0, sizeof(float) * n * r * w->K, s);
    cudaMemsetAsync(dB, 0, sizeof(float) * n * r * w->N, s);
    return launched("multi_bwd(M=0)", 0);
  }
  BaseSrc src;
  src.kind = A_NF4_K;
  src.w = w;
  src.N = w->N;
  src.K = w->K;
  return multi_bwd(src, Adapters{ids, A, B, scales, n, r}, x, dY, M, dX, dA, dB, ws, ws_bytes, s);
}

qnf4_status qnf4_dense_linear_multi_bwd(const void* W, int64_t N, int64_t K, const void* x, const void* dY,
                                        int64_t M, const int32_t* ids, int32_t n, const void* A, const void* B,
                                        int32_t r, const float* scales, void* dX, float* dA, float* dB, void* ws,
                                        size_t ws_bytes, void* stream) {
  TraceRange trace_("qnf4_dense_linear_multi_bwd");
  qnf4_status st = check_multi_args(N, K, M, n, r, true, {W, x, dY, ids, A, B, scales, dX, dA, dB});
  if (st != QNF4_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (M == 0) {
    cudaMemsetAsync(dA, 0, sizeof(float) * n * r * K, s);
    cudaMemsetAsync(dB, 0, sizeof(float) * n * r * N, s);
    return launched("multi_bwd(M=0)", 0);
  }
  BaseSrc src;
  src.kind = A_DENSE_K;
  src.Wd = W;
  src.N = N;
  src.K = K;
  return multi_bwd(src, Adapters{ids, A, B, scales, n, r}, x, dY, M, dX, dA, dB, ws, ws_bytes, s);
}

size_t qnf4_grad_workspace_size(int32_t count, const int64_t* elems, int32_t n) {
  if (count < 0 || n < 1 || (count > 0 && !elems)) return 0;
  return grad_ws_bytes(count, elems, n);
}

qnf4_status qnf4_grad_norm(int32_t count, const void* const* g, const int32_t* dtype, const int64_t* elems,
                           int32_t n, float* norm, void* ws, size_t ws_bytes, void* stream) {
  TraceRange trace_("qnf4_grad_norm");
  qnf4_status st = check_grad_args(count, g, dtype, elems, n, nullptr, norm);
  if (st != QNF4_OK) return st;
  return grad_norm_clip(count, g, dtype, elems, n, 0.f, nullptr, norm, ws, ws_bytes,
                        static_cast<cudaStream_t>(stream));
}

qnf4_status qnf4_clip_grad_norm(int32_t count, const void* const* g, const int32_t* dtype, const int64_t* elems,
                                int32_t n, float max_norm, void* const* out, float* norm, void* ws,
                                size_t ws_bytes, void* stream) {
  TraceRange trace_("qnf4_clip_grad_norm");
  if (!(max_norm >= 0.f) || std::isinf(max_norm)) return fail(QNF4_ERR_ARG, "max_norm must be finite and >= 0");
  if (!out) return fail(QNF4_ERR_ARG, "NULL out");
  qnf4_status st = check_grad_args(count, g, dtype, elems, n, out, norm);
  if (st != QNF4_OK) return st;
  return grad_norm_clip(count, g, dtype, elems, n, max_norm, out, norm, ws, ws_bytes,
                        static_cast<cudaStream_t>(stream));
}

}  // extern "C"
