// Attention of one new token per sequence over its pages.
//
//   s_j = scale q . k_j  (then cap tanh(s_j / cap)),  out = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m)
//
// Simple form: one block per (sequence, query head); each warp walks every
// fourth key with a running maximum and sum, and the warps are joined at the end.
#include "kvpop_paged.cuh"

#include <cuda_fp8.h>

namespace kvpop {
namespace {

constexpr int kWarps = 4;

template <typename T, int D, bool E4M3>
__global__ void __launch_bounds__(kWarps * 32) attend_simple_kernel(const __grid_constant__ AttendArgs a) {
  constexpr int E = D / 32;
  __shared__ float sm_acc[kWarps][D], sm_m[kWarps], sm_l[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int hq = blockIdx.x, b = blockIdx.y, h = hq / a.G;
  int n = a.lens[b];
  const int64_t cap = static_cast<int64_t>(a.width) << a.pg.page_shift;
  if (n < 0 || n > cap) {
    if (threadIdx.x == 0) set_error(a.pg.err, DEVERR_BAD_INDEX);
    n = n < 0 ? 0 : static_cast<int>(cap);
  }
  const int lo = a.window > 0 && n > a.window ? n - a.window : 0;
  const int64_t qrow = static_cast<int64_t>(b) * a.Hq + hq;
  float q[E], acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = Elem<T>::to_f32(static_cast<const T*>(a.q)[qrow * D + lane * E + e]);
    acc[e] = 0.f;
  }
  float m = -INFINITY, sum = 0.f;
  bool any = false;
  for (int i = lo + warp; i < n; i += kWarps) {
    const int page = a.table[b * a.table_stride + (i >> a.pg.page_shift)];
    if (page < 0 || page >= a.pg.n_pages) {
      if (lane == 0) set_error(a.pg.err, DEVERR_BAD_INDEX);
      continue;
    }
    any = true;
    const int64_t krow = (((static_cast<int64_t>(page) * a.pg.Hkv + h) * 2) << a.pg.page_shift) +
                         (i & ((1 << a.pg.page_shift) - 1));
    const int64_t vrow = krow + (1 << a.pg.page_shift);
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      float kx;
      if (E4M3) kx = static_cast<float>(reinterpret_cast<const __nv_fp8_e4m3*>(a.pg.pages)[krow * D + lane * E + e]);
      else kx = Elem<T>::to_f32(reinterpret_cast<const T*>(a.pg.pages)[krow * D + lane * E + e]);
      s = fmaf(q[e], kx, s);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    s *= a.scale * (E4M3 ? a.pg.scales[krow] : 1.f);
    if (a.softcap > 0.f) s = a.softcap * tanhf(s / a.softcap);
    const float m1 = fmaxf(m, s);
    const float mu = m1 == -INFINITY ? 0.f : m1;
    const float c = expf(m - mu), p = expf(s - mu);
    const float pv = p * (E4M3 ? a.pg.scales[vrow] : 1.f);
    sum = sum * c + p;
    m = m1;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      float vx;
      if (E4M3) vx = static_cast<float>(reinterpret_cast<const __nv_fp8_e4m3*>(a.pg.pages)[vrow * D + lane * E + e]);
      else vx = Elem<T>::to_f32(reinterpret_cast<const T*>(a.pg.pages)[vrow * D + lane * E + e]);
      acc[e] = fmaf(pv, vx, acc[e] * c);
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) sm_acc[warp][lane * E + e] = acc[e];
  if (lane == 0) { sm_m[warp] = m; sm_l[warp] = sum; }
  any = __syncthreads_or(any);
  float M = -INFINITY;
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm_m[w]);
  const float Mu = M == -INFINITY ? 0.f : M;
  float L = 0.f;
  for (int w = 0; w < kWarps; ++w) L += sm_l[w] * expf(sm_m[w] - Mu);
  for (int e = threadIdx.x; e < D; e += kWarps * 32) {
    float o = 0.f;
    for (int w = 0; w < kWarps; ++w) o += sm_acc[w][e] * expf(sm_m[w] - Mu);
    static_cast<T*>(a.out)[qrow * D + e] = Elem<T>::from_f32(any ? o / L : 0.f);
  }
  if (threadIdx.x == 0 && a.lse) a.lse[qrow] = any ? Mu + logf(L) : -INFINITY;
}

template <typename T, int D, bool E4M3>
int attend_t(const AttendArgs& a, cudaStream_t st) {
  attend_simple_kernel<T, D, E4M3><<<dim3(a.Hq, a.batch), kWarps * 32, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace

int launch_attend(const AttendArgs& a, int dtype, int d, int num_sms, cudaStream_t st) {
  (void)num_sms;
  const bool e8 = a.pg.scales != nullptr;
  if (dtype == KVPOP_DTYPE_BF16) {
    if (d == 128) return e8 ? attend_t<__nv_bfloat16, 128, true>(a, st) : attend_t<__nv_bfloat16, 128, false>(a, st);
    if (d == 64) return e8 ? attend_t<__nv_bfloat16, 64, true>(a, st) : attend_t<__nv_bfloat16, 64, false>(a, st);
  } else if (!e8) {
    if (d == 128) return attend_t<float, 128, false>(a, st);
    if (d == 64) return attend_t<float, 64, false>(a, st);
  }
  return -2;
}

}  // namespace kvpop
