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
// kernels here make what those read and the adapters' gradients.
#pragma once
#include "common.cuh"

namespace qnf4 {

// The distinct adapters of each tile of tn tokens: list[tile][0 .. cnt) ascending.
__global__ void __launch_bounds__(256) k_multi_tiles(const int* __restrict__ ids, int64_t M, int n, int tn,
                                                     int dmax, int* __restrict__ cnt, int* __restrict__ list) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ int s_id[256];
  __shared__ int s_first[256];
  const int64_t m0 = static_cast<int64_t>(blockIdx.x) * tn;
  const int i = threadIdx.x;
  int id = -1;
  if (i < tn && m0 + i < M) {
    id = ids[m0 + i];
    if (static_cast<unsigned>(id) >= static_cast<unsigned>(n)) id = -1;
  }
  s_id[i] = id;
  __syncthreads();
  bool first = id >= 0;
  for (int p = 0; p < i && first; ++p) first = s_id[p] != id;
  s_first[i] = first;
  const int total = __syncthreads_count(first);
  if (first) {
    int rank = 0;
    for (int p = 0; p < 256; ++p) rank += s_first[p] && s_id[p] < id;
    if (in_bounds(rank < dmax, 91)) list[blockIdx.x * static_cast<int64_t>(dmax) + rank] = id;
  }
  if (i == 0) cnt[blockIdx.x] = total;
}

// A token's projection onto its adapter: p[m][j] = scale[a] sum_c X[m, c] F[a as + j js + c cs],
// written into the tile's blocks of the adapter product (bf16; zeros in the other slots) and,
// where p32 is given, as fp32 [M][r16]. One CTA per token.
__global__ void __launch_bounds__(128) k_multi_proj(const uint16_t* __restrict__ X, int64_t C,
                                                    const uint16_t* __restrict__ F, int64_t as, int64_t js,
                                                    int64_t cs, const int* __restrict__ ids,
                                                    const float* __restrict__ scales, int n, int r, int r16,
                                                    int tn, int dmax, int cmax, const int* __restrict__ cnt,
                                                    const int* __restrict__ list, uint16_t* __restrict__ exp,
                                                    float* __restrict__ p32) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ float s_p[64];
  const int64_t m = blockIdx.x;
  const int a = ids[m];
  const bool live = static_cast<unsigned>(a) < static_cast<unsigned>(n);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int j = warp; j < r16; j += 4) {
    float v = 0.f;
    if (live && j < r) {
      for (int64_t c = lane; c < C; c += 32)
        v = fmaf(__uint_as_float(static_cast<uint32_t>(X[m * C + c]) << 16),
                 __uint_as_float(static_cast<uint32_t>(F[a * as + j * js + c * cs]) << 16), v);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      v *= scales[a];
    }
    if (lane == 0) {
      s_p[j] = v;
      if (p32) p32[m * r16 + j] = v;
    }
  }
  __syncthreads();
  if (!exp) return;
  const int64_t t = m / tn;
  const int per = 64 / r16, slots = cnt[t];
  int slot = -1;
  for (int s = 0; s < slots; ++s)
    if (live && list[t * dmax + s] == a) slot = s;
  for (int i = threadIdx.x; i < (slots + per - 1) / per * 64; i += 128) {
    const int c = i / 64, p = (i % 64) / r16, j = (i % 64) % r16;
    const bool mine = slot >= 0 && p < per && slot == c * per + p;
    exp[((t * cmax + c) * tn + (m - t * tn)) * 64 + i % 64] =
        static_cast<uint16_t>(pack_bf16x2(mine ? s_p[j] : 0.f, 0.f));
  }
}

// out[a as + j js + f fs] = sum over the tokens of a of P[m][j] X[m, f]: a thread per feature f,
// sixteen rows j per block of the z axis.
__global__ void __launch_bounds__(128) k_multi_grad(const uint16_t* __restrict__ X, int64_t F, int64_t M,
                                                    const float* __restrict__ P, int r, int r16,
                                                    const int* __restrict__ ids, float* __restrict__ out,
                                                    int64_t as, int64_t js, int64_t fs) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t f = static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x;
  const int a = blockIdx.y, j0 = blockIdx.z * 16;
  float acc[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) acc[j] = 0.f;
  for (int64_t m = 0; m < M; ++m) {
    if (ids[m] != a || f >= F) continue;
    const float x = __uint_as_float(static_cast<uint32_t>(X[m * F + f]) << 16);
#pragma unroll
    for (int j = 0; j < 16; ++j) acc[j] = fmaf(P[m * r16 + j0 + j], x, acc[j]);
  }
  if (f < F) {
    for (int j = 0; j < 16; ++j)
      if (j0 + j < r) out[a * as + (j0 + j) * js + f * fs] = acc[j];
  }
}

}  // namespace qnf4
