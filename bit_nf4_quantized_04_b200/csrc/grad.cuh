// Gradient norms over many tensors, per adapter, and clipping by them.
//
//   norm[a] = sqrt( sum_t sum_{i in part a of tensor t} g_t[i]^2 ),   a = 0 .. n - 1
//   out_t[i] = g_t[i] * min(1, max_norm / (norm[a] + 1e-6))
//
// where every tensor is n equal contiguous parts (the gradients dA [n, r, K] and dB [n, N, r]
// of n adapters over one frozen base), n = 1 being the ordinary global norm. Adapters are
// independent models, so one whose gradient overflows must not scale the others'.
//
// The work is bound by memory: one read for the norm, one read and one write for the
// scaling. It is cut into pieces of kGradPiece elements of one part, one piece per warp, so
// tensors of every size share one list and a warp needs no barrier. A piece's squares are
// summed in float64 (fp32 squares overflow from 1.8e19 on and vanish below 1e-23; the
// float64 pipe has the rate to spare here) and the pieces' sums are added in a fixed order:
// the result does not depend on the schedule.
//
// Measured: 448 fp32 tensors of 40 M elements together, one norm: 99 us on the GPU for 481 MB (two
// reads and a write), 4.9 TB/s; 14 bf16 tensors of 2.5 M elements, four norms: 12 us, most of it the
// latency of two launches in a row.
#pragma once
#include "common.cuh"

namespace qnf4 {

// Tensors per launch: the table travels in the kernel's arguments (32 bytes a tensor), which a
// short list keeps short.
constexpr int kGradMaxTensors = 512;
constexpr int kGradFewTensors = 32;
constexpr int kGradWarps = 8;
// Elements of a piece: 4096, or 1024 where the whole list is short, so that there are more warps
// than SMs can hide latency with (14 bf16 gradients, 2.5 M elements: 610 warps against 2440).
constexpr int kGradPiece = 4096;
constexpr int kGradShortPiece = 1024;
constexpr int64_t kGradShortList = 1 << 23;  // elements

template <int CAP>
struct GradTab {
  const void* in[CAP];
  void* out[CAP];
  int64_t part[CAP];           // elements of one adapter's part
  int64_t piece0[CAP + 1];     // pieces per adapter before tensor t (in this launch)
  uint32_t bf16[CAP / 32];     // bit t: tensor t is bf16, else fp32
  int piece;                               // elements of a piece
  int count;                               // tensors in this launch
  int n;                                   // adapters
  int64_t base;                            // pieces per adapter in earlier launches
  int64_t pieces;                          // pieces per adapter in all launches
};

// Piece q of adapter a: tensor t and the elements [e0, e1) of its part.
struct GradPiece {
  int t;
  int64_t e0, e1;
};
template <int CAP>
QNF4_DEV GradPiece grad_piece(const GradTab<CAP>& g, int64_t q) {
  int lo = 0, hi = g.count - 1;  // last tensor with piece0 <= q (empty tensors hold no piece)
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (g.piece0[mid] <= q) lo = mid;
    else hi = mid - 1;
  }
  GradPiece p;
  p.t = lo;
  p.e0 = (q - g.piece0[lo]) * g.piece;
  p.e1 = p.e0 + g.piece < g.part[lo] ? p.e0 + g.piece : g.part[lo];
  return p;
}

template <int CAP>
QNF4_DEV bool grad_is_bf16(const GradTab<CAP>& g, int t) { return (g.bf16[t >> 5] >> (t & 31)) & 1u; }
QNF4_DEV float bf16_of(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
QNF4_DEV double sq_add(double s, float v) { return fma(static_cast<double>(v), static_cast<double>(v), s); }

// Elements before the first 16-byte boundary at or after p, at most n.
template <typename T>
QNF4_DEV int64_t head_elems(const T* p, int64_t n) {
  const int64_t h = ((16 - (reinterpret_cast<uintptr_t>(p) & 15u)) & 15u) / sizeof(T);
  return h < n ? h : n;
}

// part_sum[a * pieces + q] = the squares of piece q of adapter a
template <int CAP>
__global__ void __launch_bounds__(32 * kGradWarps) k_grad_sq(const __grid_constant__ GradTab<CAP> g,
                                                            double* __restrict__ part_sum) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t per = g.piece0[g.count];
  const int64_t total = per * g.n;
  for (int64_t w = static_cast<int64_t>(blockIdx.x) * kGradWarps + (threadIdx.x >> 5); w < total;
       w += static_cast<int64_t>(gridDim.x) * kGradWarps) {
    const int64_t a = w / per, q = w - a * per;
    const GradPiece p = grad_piece(g, q);
    const int64_t at = a * g.part[p.t] + p.e0, len = p.e1 - p.e0;
    double s0 = 0.0, s1 = 0.0;
    if (grad_is_bf16(g, p.t)) {
      const uint16_t* x = static_cast<const uint16_t*>(g.in[p.t]) + at;
      const int64_t h = head_elems(x, len), nv = (len - h) / 8;
      const uint4* xv = reinterpret_cast<const uint4*>(x + h);
      if (lane < h) s0 = sq_add(s0, bf16_of(x[lane]));
#pragma unroll 8
      for (int64_t i = lane; i < nv; i += 32) {
        const uint4 v = __ldg(xv + i);
        s0 = sq_add(sq_add(s0, bf16lo(v.x)), bf16hi(v.x));
        s1 = sq_add(sq_add(s1, bf16lo(v.y)), bf16hi(v.y));
        s0 = sq_add(sq_add(s0, bf16lo(v.z)), bf16hi(v.z));
        s1 = sq_add(sq_add(s1, bf16lo(v.w)), bf16hi(v.w));
      }
      const int64_t r = h + nv * 8 + lane;
      if (r < len) s1 = sq_add(s1, bf16_of(x[r]));
    } else {
      const float* x = static_cast<const float*>(g.in[p.t]) + at;
      const int64_t h = head_elems(x, len), nv = (len - h) / 4;
      const float4* xv = reinterpret_cast<const float4*>(x + h);
      if (lane < h) s0 = sq_add(s0, x[lane]);
#pragma unroll 8
      for (int64_t i = lane; i < nv; i += 32) {
        const float4 v = __ldg(xv + i);
        s0 = sq_add(sq_add(s0, v.x), v.y);
        s1 = sq_add(sq_add(s1, v.z), v.w);
      }
      const int64_t r = h + nv * 4 + lane;
      if (r < len) s1 = sq_add(s1, x[r]);
    }
    s0 += s1;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s0 += __shfl_xor_sync(0xffffffffu, s0, o);
    if (lane == 0 && in_bounds(g.base + q < g.pieces, 81)) part_sum[a * g.pieces + g.base + q] = s0;
  }
}

// The sum of an adapter's pieces by one warp, in a fixed order (all lanes return it).
QNF4_DEV double grad_warp_sum(const double* src, int64_t pieces) {
  double s = 0.0;
#pragma unroll 8
  for (int64_t i = threadIdx.x & 31; i < pieces; i += 32) s += __ldcg(src + i);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}
// min(1, max_norm / (norm + 1e-6)); a NaN norm gives a NaN factor
QNF4_DEV float grad_factor(float norm, float max_norm) {
  const float c = max_norm / (norm + 1e-6f);
  return c > 1.f ? 1.f : c;
}

// Lists of few pieces need no kernel of their own for the norms: every CTA of the scaling kernel
// adds them up itself.
constexpr int64_t kGradFewPieces = 4096;  // of all adapters together
constexpr int kGradFewAdapters = 64;
inline bool grad_few(int64_t pieces, int n) { return pieces * n <= kGradFewPieces && n <= kGradFewAdapters; }

// norm[a] and, for clipping, the factor coef[a]. One CTA per adapter, its pieces added in a fixed
// order (few pieces: in the order of the scaling kernel).
__global__ void __launch_bounds__(512) k_grad_norm(const double* __restrict__ part_sum, int64_t pieces,
                                                   float max_norm, int few, float* __restrict__ norm,
                                                   float* __restrict__ coef) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ double s_sum[16];
  const double* src = part_sum + blockIdx.x * pieces;
  if (few) {
    const double t = threadIdx.x < 32 ? grad_warp_sum(src, pieces) : 0.0;
    if (threadIdx.x == 0) norm[blockIdx.x] = static_cast<float>(sqrt(t));
    return;
  }
  double s = 0.0;
#pragma unroll 8
  for (int64_t i = threadIdx.x; i < pieces; i += 512) s += __ldcg(src + i);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    double t = 0.0;
    for (int i = 0; i < 16; ++i) t += s_sum[i];
    const float v = static_cast<float>(sqrt(t));
    norm[blockIdx.x] = v;
    if (coef) coef[blockIdx.x] = grad_factor(v, max_norm);
  }
}

// out = g * coef[a] (coef null: few pieces, added up here, and written to norm by CTA 0); where the
// output is the input, an adapter whose factor is 1 is left.
template <int CAP>
__global__ void __launch_bounds__(32 * kGradWarps) k_grad_scale(const __grid_constant__ GradTab<CAP> g,
                                                               const float* __restrict__ coef,
                                                               const double* __restrict__ part_sum,
                                                               float max_norm, float* __restrict__ norm) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ float s_coef[kGradFewAdapters];
  const int lane = threadIdx.x & 31;
  if (!coef) {
    for (int a = threadIdx.x >> 5; a < g.n; a += kGradWarps) {
      const float v = static_cast<float>(sqrt(grad_warp_sum(part_sum + a * g.pieces, g.pieces)));
      if (lane == 0) {
        s_coef[a] = grad_factor(v, max_norm);
        if (blockIdx.x == 0) norm[a] = v;
      }
    }
    __syncthreads();
  }
  const int64_t per = g.piece0[g.count];
  const int64_t total = per * g.n;
  for (int64_t w = static_cast<int64_t>(blockIdx.x) * kGradWarps + (threadIdx.x >> 5); w < total;
       w += static_cast<int64_t>(gridDim.x) * kGradWarps) {
    const int64_t a = w / per, q = w - a * per;
    const GradPiece p = grad_piece(g, q);
    const float c = coef ? __ldcg(coef + a) : s_coef[a];
    if (c == 1.f && g.out[p.t] == g.in[p.t]) continue;
    const int64_t at = a * g.part[p.t] + p.e0, len = p.e1 - p.e0;
    if (grad_is_bf16(g, p.t)) {
      const uint16_t* x = static_cast<const uint16_t*>(g.in[p.t]) + at;
      uint16_t* y = static_cast<uint16_t*>(g.out[p.t]) + at;
      const bool same = ((reinterpret_cast<uintptr_t>(x) ^ reinterpret_cast<uintptr_t>(y)) & 15u) == 0;
      const int64_t h = same ? head_elems(x, len) : 0, nv = same ? (len - h) / 8 : 0;
      const uint4* xv = reinterpret_cast<const uint4*>(x + h);
      uint4* yv = reinterpret_cast<uint4*>(y + h);
      auto one = [&](int64_t i) { y[i] = static_cast<uint16_t>(pack_bf16x2(bf16_of(x[i]) * c, 0.f)); };
      if (lane < h) one(lane);
#pragma unroll 8
      for (int64_t i = lane; i < nv; i += 32) {
        uint4 v = xv[i];
        v.x = pack_bf16x2(bf16lo(v.x) * c, bf16hi(v.x) * c);
        v.y = pack_bf16x2(bf16lo(v.y) * c, bf16hi(v.y) * c);
        v.z = pack_bf16x2(bf16lo(v.z) * c, bf16hi(v.z) * c);
        v.w = pack_bf16x2(bf16lo(v.w) * c, bf16hi(v.w) * c);
        yv[i] = v;
      }
      for (int64_t i = h + nv * 8 + lane; i < len; i += 32) one(i);
    } else {
      const float* x = static_cast<const float*>(g.in[p.t]) + at;
      float* y = static_cast<float*>(g.out[p.t]) + at;
      const bool same = ((reinterpret_cast<uintptr_t>(x) ^ reinterpret_cast<uintptr_t>(y)) & 15u) == 0;
      const int64_t h = same ? head_elems(x, len) : 0, nv = same ? (len - h) / 4 : 0;
      const float4* xv = reinterpret_cast<const float4*>(x + h);
      float4* yv = reinterpret_cast<float4*>(y + h);
      if (lane < h) y[lane] = x[lane] * c;
#pragma unroll 8
      for (int64_t i = lane; i < nv; i += 32) {
        float4 v = xv[i];
        v.x *= c;
        v.y *= c;
        v.z *= c;
        v.w *= c;
        yv[i] = v;
      }
      for (int64_t i = h + nv * 4 + lane; i < len; i += 32) y[i] = x[i] * c;
    }
  }
}

}  // namespace qnf4
