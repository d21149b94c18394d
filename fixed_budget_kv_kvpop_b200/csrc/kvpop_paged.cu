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
// The same held as they are loaded, for rows that wait their turn.
template <typename T> struct Raw4;
template <> struct Raw4<float> { float4 v; };
template <> struct Raw4<__nv_bfloat16> { uint2 v; };
__device__ __forceinline__ void unpack4(const Raw4<float>& r, float* x) {
  x[0] = r.v.x; x[1] = r.v.y; x[2] = r.v.z; x[3] = r.v.w;
}
__device__ __forceinline__ void unpack4(const Raw4<__nv_bfloat16>& r, float* x) {
  const float2 lo = bf2_to_f2(r.v.x), hi = bf2_to_f2(r.v.y);
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

// e4m3(x / scale) of eight elements.  The quotients have to be the rounded
// ones: bf16 rows often put them on the middle between two held values, and a
// product with the reciprocal would send those to either side.  With r the
// rounded reciprocal, q = x r is off by an ulp or so, and q + (x - q scale) r,
// the remainder being exact in one FMA, is the rounded quotient (Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor",
// 1990); compared with the division for every bf16 significand and 2^23 scales.
// Below 2^-90 the remainder could underflow: those rows divide.
__device__ __forceinline__ void quotients(float (&x)[8], float scale) {
  if (scale == 0.f) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = 0.f;
  } else if (scale < 8.0779357e-28f) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = x[e] / scale;
  } else {
    const float r = 1.f / scale;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float q = x[e] * r;
      x[e] = fmaf(fmaf(-q, scale, x[e]), r, q);
    }
  }
}

// Scale of a row whose largest magnitude is m.
__device__ __forceinline__ float scale_of(float m) {
  const float scale = m * kPerStep;
  if (!(scale < __int_as_float(0x7f800000))) return __int_as_float(0x7fffffff);   // inf or NaN: the row reads back as NaN
  return scale < 1.17549435e-38f ? 0.f : scale;                                   // subnormal: held as zeros
}

// Row `slot` of a page range: index of head h's key (kv = 0) or value row.
__device__ __forceinline__ int64_t page_row(const PagedLayer& pg, int64_t slot, int h, int kv) {
  return ((((slot >> pg.page_shift) * pg.Hkv + h) * 2 + kv) << pg.page_shift) + (slot & ((1 << pg.page_shift) - 1));
}

// Heads of new tokens: norm, rotation, and with HEADS_STEP the write into pages.
// Bound by HBM (every row is read and written once).  wpt warps share a token:
// its cosines and sines (fp64 angles) are formed once, by different lanes, and
// handed over in shared memory, while the rows' loads, up to U per lane, are
// already on their way.
template <typename T, int D, bool E4M3, int MODE>
__global__ void __launch_bounds__(kThreads, 3) heads_kernel(const __grid_constant__ HeadsArgs a, int passes, int wpt_shift) {
  constexpr int LPR = D / 8;          // lanes per row
  constexpr int RPW = 32 / LPR;       // rows per warp and pass
  constexpr int U = 4;
  __shared__ __align__(16) float2 turns[2][kThreads / 32][D / 2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int l = lane % LPR, sub = lane / LPR;
  const int wpt = 1 << wpt_shift;
  const int seat = warp >> wpt_shift, wt = warp & (wpt - 1), seats = (kThreads / 32) >> wpt_shift;
  const int tokens = a.batch * a.n_tokens;
  const int rot = a.rope.rot;
  const bool inter = a.rope.interleaved != 0;
  const int n_rows = a.Hq + a.Hkv * (MODE == HEADS_DENSE ? 1 : 2);
  // this lane's two element groups of a row, and their turns' places
  int oa = 4 * l, ob = D / 2 + 4 * l;
  if (!inter && rot < D) {
    const int j = l - rot / 8;
    oa = j < 0 ? 4 * l : rot + 4 * j;
    ob = j < 0 ? 4 * l + rot / 2 : rot + (D - rot) / 2 + 4 * j;
  }
  const int pa = inter ? oa / 2 : oa, pb = inter ? ob / 2 : oa + 2;   // pairs pa, pa + 1 and pb, pb + 1

  int buf = 0;
  for (int t0 = blockIdx.x * seats; t0 < tokens; t0 += gridDim.x * seats, buf ^= 1) {
    const int t = t0 + seat;
    const bool live = t < tokens;
    const int b = live ? t / a.n_tokens : 0, i = live ? t - b * a.n_tokens : 0;
    const T* qrow = reinterpret_cast<const T*>(a.q.p) + b * a.q.bs + i * a.q.ts;
    const T* krow = reinterpret_cast<const T*>(a.k.p) + b * a.k.bs + i * a.k.ts;
    const T* vrow = MODE == HEADS_DENSE ? nullptr : reinterpret_cast<const T*>(a.v.p) + b * a.v.bs + i * a.v.ts;
    bool turned = false;
    float4 ca, cb;
    int64_t slot = -1;
    for (int p0 = wt; p0 < passes || (p0 == wt); p0 += U * wpt) {
      Raw4<T> xa[U], xb[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = (p0 + u * wpt) * RPW + sub;
        if (live && r < n_rows) {
          const T* src = r < a.Hq ? qrow + r * a.q.hs
                                  : r < a.Hq + a.Hkv ? krow + (r - a.Hq) * a.k.hs : vrow + (r - a.Hq - a.Hkv) * a.v.hs;
          xa[u] = *reinterpret_cast<const Raw4<T>*>(src + oa);
          xb[u] = *reinterpret_cast<const Raw4<T>*>(src + ob);
        }
      }
      if (!turned) {
        turned = true;
        if (live) {
          const int pos = a.pos[t];
          for (int p = wt * 32 + lane; p < rot / 2; p += wpt * 32) {
            float2 cs;
            turn_of(pos, a.rope.inv_freq[p], a.rope.scale, cs.x, cs.y);
            turns[buf][seat][p] = cs;
          }
          if (MODE == HEADS_STEP) {
            const int s = a.slots[t];
            if (s >= 0) {
              if ((s >> a.pg.page_shift) < a.pg.n_pages) slot = s;
              else if (lane == 0) set_error(a.pg.err, DEVERR_BAD_INDEX);
            }
          }
        }
        __syncthreads();
        ca = pa < rot / 2 ? *reinterpret_cast<const float4*>(&turns[buf][seat][pa]) : make_float4(1.f, 0.f, 1.f, 0.f);
        cb = pb < rot / 2 ? *reinterpret_cast<const float4*>(&turns[buf][seat][pb]) : make_float4(1.f, 0.f, 1.f, 0.f);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = (p0 + u * wpt) * RPW + sub;
        if ((p0 + u * wpt) * RPW >= n_rows) break;
        const int kind = r < a.Hq ? 0 : r < a.Hq + a.Hkv ? 1 : 2;    // query, key, value
        const int h = kind == 0 ? r : kind == 1 ? r - a.Hq : r - a.Hq - a.Hkv;
        const bool on = live && r < n_rows;
        float y[8];
        float ss = 0.f;
        if (on) {
          unpack4(xa[u], y);
          unpack4(xb[u], y + 4);
        }
        if (on && kind < 2) {
#pragma unroll
          for (int e = 0; e < 8; ++e) ss = fmaf(y[e], y[e], ss);
        }
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (kind < 2 && on) {
          const float* w = kind == 0 ? a.rope.q_weight : a.rope.k_weight;
          if (w != nullptr) {
            const float rn = rsqrtf(ss * (1.f / D) + a.rope.eps);
            float wv[8];
            load4<float>(w + oa, wv);
            load4<float>(w + ob, wv + 4);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = y[e] * rn * wv[e];
          }
          auto turn = [](float& p, float& q, float c, float s) {
            const float p0 = p, q0 = q;
            p = p0 * c - q0 * s;
            q = q0 * c + p0 * s;
          };
          if (inter) {
            turn(y[0], y[1], ca.x, ca.y); turn(y[2], y[3], ca.z, ca.w);
            turn(y[4], y[5], cb.x, cb.y); turn(y[6], y[7], cb.z, cb.w);
          } else {
            turn(y[0], y[4], ca.x, ca.y); turn(y[1], y[5], ca.z, ca.w);
            turn(y[2], y[6], cb.x, cb.y); turn(y[3], y[7], cb.z, cb.w);
          }
        }
        if (on && (kind == 0 || MODE == HEADS_DENSE)) {
          const RowsView& dst = kind == 0 ? a.qo : a.ko;
          T* row = reinterpret_cast<T*>(dst.p) + b * dst.bs + i * dst.ts + h * dst.hs;
          store4<T>(row + oa, y);
          store4<T>(row + ob, y + 4);
        }
        if (MODE == HEADS_STEP) {
          const bool keep = on && kind > 0 && slot >= 0;
          const int64_t at = keep ? page_row(a.pg, slot, h, kind - 1) : 0;
          if (E4M3) {
            float m = 0.f;
            if (keep) {
#pragma unroll
              for (int e = 0; e < 8; ++e) m = max_nan(m, fabsf(y[e]));
            }
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
            if (keep) {
              const float scale = scale_of(m);
              quotients(y, scale);
              *reinterpret_cast<uint32_t*>(a.pg.pages + at * D + oa) = to_e4m3x4(y);
              *reinterpret_cast<uint32_t*>(a.pg.pages + at * D + ob) = to_e4m3x4(y + 4);
              if (l == 0) a.pg.scales[at] = scale;
            }
          } else if (keep) {
            T* row = reinterpret_cast<T*>(a.pg.pages) + at * D;
            store4<T>(row + oa, y);
            store4<T>(row + ob, y + 4);
          }
        }
      }
    }
  }
}

// Eight consecutive elements as they lie in memory.
template <typename T> struct Raw8;
template <> struct Raw8<float> { float4 a, b; };
template <> struct Raw8<__nv_bfloat16> { uint4 a; };
__device__ __forceinline__ void unpack8(const Raw8<__nv_bfloat16>& r, float* x) { unpack16(r.a, x, __nv_bfloat16()); }
__device__ __forceinline__ void unpack8(const Raw8<float>& r, float* x) {
  x[0] = r.a.x; x[1] = r.a.y; x[2] = r.a.z; x[3] = r.a.w;
  x[4] = r.b.x; x[5] = r.b.y; x[6] = r.b.z; x[7] = r.b.w;
}

// Keys and values of new tokens into pages.  Bound by HBM.  A warp takes `chunk`
// passes of one token, RPW rows each, with U rows per lane on their way at a time.
template <typename T, int D, bool E4M3>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ HeadsArgs a, int passes, int chunk) {
  constexpr int LPR = D / 8, RPW = 32 / LPR, U = 4;
  const int lane = threadIdx.x & 31, l = lane % LPR, sub = lane / LPR;
  const int nch = (passes + chunk - 1) / chunk;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32;
  const int64_t t = item / nch;
  if (t >= static_cast<int64_t>(a.batch) * a.n_tokens) return;
  const int p_beg = static_cast<int>(item - t * nch) * chunk, p_end = min(passes, p_beg + chunk);
  const int b = static_cast<int>(t / a.n_tokens), i = static_cast<int>(t - static_cast<int64_t>(b) * a.n_tokens);
  const T* krow = reinterpret_cast<const T*>(a.k.p) + b * a.k.bs + i * a.k.ts + 8 * l;
  const T* vrow = reinterpret_cast<const T*>(a.v.p) + b * a.v.bs + i * a.v.ts + 8 * l;
  const int s = a.slots[t];
  for (int p0 = p_beg; p0 < p_end; p0 += U) {
    Raw8<T> x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = (p0 + u) * RPW + sub;
      if (p0 + u < p_end && r < 2 * a.Hkv)
        x[u] = *reinterpret_cast<const Raw8<T>*>(r < a.Hkv ? krow + r * a.k.hs : vrow + (r - a.Hkv) * a.v.hs);
    }
    if (s < 0) return;
    if ((s >> a.pg.page_shift) >= a.pg.n_pages) {
      if (lane == 0) set_error(a.pg.err, DEVERR_BAD_INDEX);
      return;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (p0 + u >= p_end) break;
      const int r = (p0 + u) * RPW + sub;
      const bool on = r < 2 * a.Hkv;
      const int kv = r < a.Hkv ? 0 : 1;
      const int64_t at = on ? page_row(a.pg, s, r - kv * a.Hkv, kv) : 0;
      if constexpr (E4M3) {
        float y[8];
        float m = 0.f;
        if (on) {
          unpack8(x[u], y);
#pragma unroll
          for (int e = 0; e < 8; ++e) m = max_nan(m, fabsf(y[e]));
        }
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (on) {
          const float scale = scale_of(m);
          quotients(y, scale);
          *reinterpret_cast<uint2*>(a.pg.pages + at * D + 8 * l) = make_uint2(to_e4m3x4(y), to_e4m3x4(y + 4));
          if (l == 0) a.pg.scales[at] = scale;
        }
      } else if (on) {
        *reinterpret_cast<Raw8<T>*>(reinterpret_cast<T*>(a.pg.pages) + at * D + 8 * l) = x[u];
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
  if (mode == HEADS_APPEND) {
    const int chunk = tokens >= 4 * num_sms ? passes : 1;
    const int64_t warps = tokens * ((passes + chunk - 1) / chunk);
    const int64_t grid = (warps + kThreads / 32 - 1) / (kThreads / 32);
    append_kernel<T, D, E4M3><<<static_cast<unsigned>(grid), kThreads, 0, st>>>(a, passes, chunk);
    return cudaGetLastError() == cudaSuccess ? 0 : -1;
  }
  int shift = 0;      // warps per token: about three passes each
  while (shift < 3 && (passes >> shift) > 3) ++shift;
  const int seats = (kThreads / 32) >> shift;
  const int64_t grid = (tokens + seats - 1) / seats;
  if (mode == HEADS_DENSE)
    heads_kernel<T, D, false, HEADS_DENSE><<<static_cast<unsigned>(grid), kThreads, 0, st>>>(a, passes, shift);
  else
    heads_kernel<T, D, E4M3, HEADS_STEP><<<static_cast<unsigned>(grid), kThreads, 0, st>>>(a, passes, shift);
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
