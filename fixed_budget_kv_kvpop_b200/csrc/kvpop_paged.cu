// Paged cache: norm and rotation of new tokens' heads, the write into pages
// (as they are, or e4m3 with one scale per row) and the read back.
//
// All are one pass over rows of d elements.  A row is held by d / 8 lanes with
// eight elements each, as two groups of four: element groups oa and ob.
#include "kvpop_paged.cuh"

#include <cuda_fp8.h>

namespace kvpop {
namespace {

constexpr float kPerStep = 1.f / 448.f;   // 448: the largest e4m3 value
constexpr int kThreads = 256;

// Four consecutive elements as fp32, and back with one rounding.
template <typename T> __device__ __forceinline__ void load4(const T* p, float* x);
template <> __device__ __forceinline__ void load4<float>(const float* p, float* x) {
  const float4 r = *reinterpret_cast<const float4*>(p);
  x[0] = r.x; x[1] = r.y; x[2] = r.z; x[3] = r.w;
}
template <> __device__ __forceinline__ void load4<__nv_bfloat16>(const __nv_bfloat16* p, float* x) {
  const uint2 r = *reinterpret_cast<const uint2*>(p);
  const float2 lo = bf2_to_f2(r.x), hi = bf2_to_f2(r.y);
  x[0] = lo.x; x[1] = lo.y; x[2] = hi.x; x[3] = hi.y;
}
template <typename T> __device__ __forceinline__ void store4(T* p, const float* x);
template <> __device__ __forceinline__ void store4<float>(float* p, const float* x) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
template <> __device__ __forceinline__ void store4<__nv_bfloat16>(__nv_bfloat16* p, const float* x) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
}

// Maximum that keeps a NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ uint32_t to_e4m3x4(const float* x) {
  const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[0], x[1]), __NV_SATFINITE, __NV_E4M3);
  const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[2], x[3]), __NV_SATFINITE, __NV_E4M3);
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// Cosine and sine of pos * inv_freq.  The angle is formed in fp64 as turns and
// reduced to half a turn either way there, so far positions lose nothing:
// at position 2^20 the fraction is off by about 2^20 * 2^-53 turns.
__device__ __forceinline__ void turn_of(int pos, double inv_freq, float scale, float& c, float& s) {
  const double t = static_cast<double>(pos) * (inv_freq * 0.15915494309189533577);
  sincospif(2.f * static_cast<float>(t - rint(t)), &s, &c);
  c *= scale;
  s *= scale;
}

template <typename T, int D, bool E4M3, int MODE>
__global__ void __launch_bounds__(kThreads) heads_kernel(const __grid_constant__ HeadsArgs a, int passes, int chunk) {
  constexpr int LPR = D / 8;          // lanes per row
  constexpr int RPW = 32 / LPR;       // rows per warp and pass
  const int lane = threadIdx.x & 31;
  const int l = lane % LPR, sub = lane / LPR;
  const int64_t n_items = static_cast<int64_t>(a.batch) * a.n_tokens * ((passes + chunk - 1) / chunk);
  const int nch = (passes + chunk - 1) / chunk;
  for (int64_t item = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32; item < n_items;
       item += static_cast<int64_t>(gridDim.x) * (kThreads / 32)) {
    const int64_t t = item / nch;
    const int p0 = static_cast<int>(item % nch) * chunk;
    const int p1 = min(passes, p0 + chunk);
    const int b = static_cast<int>(t / a.n_tokens), i = static_cast<int>(t % a.n_tokens);

    int64_t slot = -1;
    if (MODE != HEADS_DENSE) {
      const int s = a.slots[t];
      if (s >= 0) {
        if ((s >> a.pg.page_shift) < a.pg.n_pages) slot = s;
        else if (lane == 0) set_error(a.pg.err, DEVERR_BAD_INDEX);
      }
    }
    // this lane's two element groups of a turned row, and their four turns
    int oa = 4 * l, ob = D / 2 + 4 * l;
    float cs[4], sn[4];
    if (MODE != HEADS_APPEND) {
      const int rot = a.rope.rot;
      const int pos = a.pos[t];
      const bool inter = a.rope.interleaved != 0;
      if (!inter && rot < D) {
        const int j = l - rot / 8;
        oa = j < 0 ? 4 * l : rot + 4 * j;
        ob = j < 0 ? 4 * l + rot / 2 : rot + (D - rot) / 2 + 4 * j;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // pair index: (p, p + rot / 2), or (2p, 2p + 1)
        const int p = inter ? ((e < 2 ? oa : ob) / 2 + (e & 1)) : oa + e;
        const bool turned = inter ? p < rot / 2 : oa < rot / 2;
        cs[e] = 1.f; sn[e] = 0.f;
        if (turned) turn_of(pos, a.rope.inv_freq[p], a.rope.scale, cs[e], sn[e]);
      }
    }
    const int n_rows = (MODE == HEADS_APPEND ? 0 : a.Hq) + a.Hkv * (MODE == HEADS_DENSE ? 1 : 2);
    for (int p = p0; p < p1; ++p) {
      const int r = p * RPW + sub;
      const bool live = r < n_rows;
      // row kinds: queries, keys, values
      const int rq = MODE == HEADS_APPEND ? 0 : a.Hq;
      const int kind = r < rq ? 0 : r < rq + a.Hkv ? 1 : 2;
      const int h = kind == 0 ? r : kind == 1 ? r - rq : r - rq - a.Hkv;
      const RowsView& src = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
      const bool todo = live && (kind == 0 || MODE == HEADS_DENSE || slot >= 0);
      const bool turn = MODE != HEADS_APPEND && kind < 2;
      const int ea = turn ? oa : 4 * l, eb = turn ? ob : D / 2 + 4 * l;
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = 0.f;
      if (todo) {
        const T* row = reinterpret_cast<const T*>(src.p) + b * src.bs + i * src.ts + h * src.hs;
        load4<T>(row + ea, x);
        load4<T>(row + eb, x + 4);
      }
      if (MODE != HEADS_APPEND) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float* w = kind == 0 ? a.rope.q_weight : a.rope.k_weight;
        if (turn && w != nullptr && todo) {
          const float rn = rsqrtf(ss * (1.f / D) + a.rope.eps);
          float wv[8];
          load4<float>(w + ea, wv);
          load4<float>(w + eb, wv + 4);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = x[e] * rn * wv[e];
        }
        if (turn) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float& u = a.rope.interleaved ? x[2 * e] : x[e];
            float& v = a.rope.interleaved ? x[2 * e + 1] : x[e + 4];
            const float u0 = u, v0 = v;
            u = u0 * cs[e] - v0 * sn[e];
            v = v0 * cs[e] + u0 * sn[e];
          }
        }
      }
      if (kind == 0 || MODE == HEADS_DENSE) {
        const RowsView& dst = kind == 0 ? a.qo : a.ko;
        if (todo) {
          T* row = reinterpret_cast<T*>(dst.p) + b * dst.bs + i * dst.ts + h * dst.hs;
          store4<T>(row + ea, x);
          store4<T>(row + eb, x + 4);
        }
      }
      if (MODE != HEADS_DENSE) {
        const int64_t page = slot >> a.pg.page_shift;
        const int64_t prow = ((page * a.pg.Hkv + h) * 2 + (kind - 1)) << a.pg.page_shift;
        const int64_t at = prow + (slot & ((1 << a.pg.page_shift) - 1));
        if (E4M3) {
          float m = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) m = max_nan(m, fabsf(x[e]));
#pragma unroll
          for (int o = LPR / 2; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
          if (todo && kind > 0) {
            float scale = m * kPerStep;
            if (!(scale < __int_as_float(0x7f800000))) scale = __int_as_float(0x7fffffff);   // inf or NaN: the row reads back as NaN
            else if (scale < 1.17549435e-38f) scale = 0.f;                                   // held as zeros
            // a true division: quotients that fall on the middle between two held values are common (both
            // sides have few bits), and a product with the reciprocal would round those to either side
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = scale == 0.f ? 0.f : x[e] / scale;
            *reinterpret_cast<uint32_t*>(a.pg.pages + at * D + ea) = to_e4m3x4(x);
            *reinterpret_cast<uint32_t*>(a.pg.pages + at * D + eb) = to_e4m3x4(x + 4);
            if (l == 0) a.pg.scales[at] = scale;
          }
        } else if (todo && kind > 0) {
          T* row = reinterpret_cast<T*>(a.pg.pages) + at * D;
          store4<T>(row + ea, x);
          store4<T>(row + eb, x + 4);
        }
      }
    }
  }
}

// Four held elements as fp32.
template <typename T, bool E4M3>
__device__ __forceinline__ void held4(const PagedLayer& pg, int64_t row, int D, int e0, float scale, float* x) {
  if (E4M3) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(pg.pages + row * D + e0);
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> (16 * p)), __NV_E4M3);
      const float2 f = __half22float2(__half2(h));
      x[2 * p] = f.x * scale;
      x[2 * p + 1] = f.y * scale;
    }
  } else {
    load4<T>(reinterpret_cast<const T*>(pg.pages) + row * D + e0, x);
  }
}

constexpr int kGatherTokens = 64;

template <typename T, int D, bool E4M3>
__global__ void __launch_bounds__(kThreads) gather_kernel(const __grid_constant__ GatherArgs a) {
  constexpr int LPR = D / 8, RPW = 32 / LPR;
  const int lane = threadIdx.x & 31, l = lane % LPR;
  const int b = blockIdx.z, h = blockIdx.y >> 1, kv = blockIdx.y & 1;
  int n = a.lens[b];
  const int64_t cap = min(static_cast<int64_t>(a.n_tokens), static_cast<int64_t>(a.width) << a.pg.page_shift);
  if (n < 0 || n > cap) {
    if (threadIdx.x == 0 && blockIdx.x == 0) set_error(a.pg.err, DEVERR_BAD_INDEX);
    n = n < 0 ? 0 : static_cast<int>(cap);
  }
  const RowsView& dst = kv ? a.v : a.k;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kGatherTokens;
  for (int j = threadIdx.x / LPR; j < kGatherTokens; j += kThreads / LPR) {
    const int64_t i = t0 + j;
    if (i >= n) break;
    const int page = a.table[b * a.table_stride + (i >> a.pg.page_shift)];
    if (page < 0 || page >= a.pg.n_pages) {
      if (l == 0) set_error(a.pg.err, DEVERR_BAD_INDEX);
      continue;
    }
    const int64_t row = (((static_cast<int64_t>(page) * a.pg.Hkv + h) * 2 + kv) << a.pg.page_shift) +
                        (i & ((1 << a.pg.page_shift) - 1));
    const float scale = E4M3 ? a.pg.scales[row] : 1.f;
    float x[8];
    held4<T, E4M3>(a.pg, row, D, 8 * l, scale, x);
    held4<T, E4M3>(a.pg, row, D, 8 * l + 4, scale, x + 4);
    T* out = reinterpret_cast<T*>(dst.p) + b * dst.bs + i * dst.ts + h * dst.hs + 8 * l;
    store4<T>(out, x);
    store4<T>(out + 4, x + 4);
  }
  (void)RPW;
}

template <typename T, int D, bool E4M3>
int heads_t(const HeadsArgs& a, int mode, int num_sms, cudaStream_t st) {
  const int rows = (mode == HEADS_APPEND ? 0 : a.Hq) + a.Hkv * (mode == HEADS_DENSE ? 1 : 2);
  const int rpw = 32 / (D / 8);
  const int passes = (rows + rpw - 1) / rpw;
  const int64_t tokens = static_cast<int64_t>(a.batch) * a.n_tokens;
  const int chunk = tokens >= 4 * num_sms ? passes : 1;
  const int64_t warps = tokens * ((passes + chunk - 1) / chunk);
  int64_t grid = (warps + kThreads / 32 - 1) / (kThreads / 32);
  if (grid > 1 << 20) grid = 1 << 20;
  if (mode == HEADS_DENSE)
    heads_kernel<T, D, false, HEADS_DENSE><<<static_cast<unsigned>(grid), kThreads, 0, st>>>(a, passes, chunk);
  else if (mode == HEADS_APPEND)
    heads_kernel<T, D, E4M3, HEADS_APPEND><<<static_cast<unsigned>(grid), kThreads, 0, st>>>(a, passes, chunk);
  else
    heads_kernel<T, D, E4M3, HEADS_STEP><<<static_cast<unsigned>(grid), kThreads, 0, st>>>(a, passes, chunk);
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

template <typename T, int D, bool E4M3>
int gather_t(const GatherArgs& a, cudaStream_t st) {
  const dim3 grid((a.n_tokens + kGatherTokens - 1) / kGatherTokens, a.pg.Hkv * 2, a.batch);
  gather_kernel<T, D, E4M3><<<grid, kThreads, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace

int launch_heads(const HeadsArgs& a, int dtype, int d, int mode, int num_sms, cudaStream_t st) {
  const bool e8 = a.pg.scales != nullptr;
  if (dtype == KVPOP_DTYPE_BF16) {
    if (d == 128) return e8 ? heads_t<__nv_bfloat16, 128, true>(a, mode, num_sms, st)
                            : heads_t<__nv_bfloat16, 128, false>(a, mode, num_sms, st);
    if (d == 64) return e8 ? heads_t<__nv_bfloat16, 64, true>(a, mode, num_sms, st)
                           : heads_t<__nv_bfloat16, 64, false>(a, mode, num_sms, st);
  } else if (!e8) {
    if (d == 128) return heads_t<float, 128, false>(a, mode, num_sms, st);
    if (d == 64) return heads_t<float, 64, false>(a, mode, num_sms, st);
  }
  return -2;
}

int launch_gather(const GatherArgs& a, int dtype, int d, cudaStream_t st) {
  const bool e8 = a.pg.scales != nullptr;
  if (dtype == KVPOP_DTYPE_BF16) {
    if (d == 128) return e8 ? gather_t<__nv_bfloat16, 128, true>(a, st) : gather_t<__nv_bfloat16, 128, false>(a, st);
    if (d == 64) return e8 ? gather_t<__nv_bfloat16, 64, true>(a, st) : gather_t<__nv_bfloat16, 64, false>(a, st);
  } else if (!e8) {
    if (d == 128) return gather_t<float, 128, false>(a, st);
    if (d == 64) return gather_t<float, 64, false>(a, st);
  }
  return -2;
}

}  // namespace kvpop
