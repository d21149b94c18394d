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

__device__ __forceinline__ uint32_t to_e4m3x4(const float* x) {
  const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[0], x[1]), __NV_SATFINITE, __NV_E4M3);
  const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[2], x[3]), __NV_SATFINITE, __NV_E4M3);
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// A frequency as the fraction of a turn per position, in units of 2^-64.
// Products with a position wrap at whole turns, so the angle of any int32
// position keeps all its bits (off by at most 2^-25 turns at 2^31, from the
// frequency's own 53 bits), and no fp64 instruction is left per token: their
// conversions ran at a sixteenth of the fp32 ones' rate and took 95% of the
// conversion pipe's time.
__device__ __forceinline__ uint64_t turn_step(double inv_freq) {
  const double t = inv_freq * 0.15915494309189533577;
  return __double2ull_rz((t - floor(t)) * 18446744073709551616.0);
}
__device__ __forceinline__ void turn_of(int pos, uint64_t step, float scale, float& c, float& s) {
  const uint64_t at = static_cast<uint64_t>(static_cast<int64_t>(pos)) * step;
  const float half_turns = static_cast<float>(static_cast<int32_t>(at >> 32)) * (1.f / 2147483648.f);
  sincospif(half_turns, &s, &c);
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
    const float2 r2 = make_float2(r, r), s2 = make_float2(-scale, -scale);
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const float2 v = make_float2(x[e], x[e + 1]);
      const float2 q = __fmul2_rn(v, r2);
      const float2 y = ffma2(ffma2(q, s2, v), r2, q);
      x[e] = y.x; x[e + 1] = y.y;
    }
  }
}

// Scale of a row whose largest magnitude is m.
__device__ __forceinline__ float scale_of(float m) {
  const float scale = m * kPerStep;
  if (!(scale < __int_as_float(0x7f800000))) return __int_as_float(0x7fffffff);   // inf or NaN: the row reads back as NaN
  return scale < 1.17549435e-38f ? 0.f : scale;                                   // subnormal: held as zeros
}

// Largest magnitude of eight elements as its bits: unsigned order is the order
// of magnitudes, with infinities and then NaN on top.
__device__ __forceinline__ uint32_t top_bits(const float (&x)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(x[e]) & 0x7fffffffu);
  return m;
}

// New tokens' heads.  HEADS_DENSE: queries and keys are normalised, turned and
// written; HEADS_STEP: the same, but keys, and the values as they are, go into pages.
//
// Bound by HBM: every row is read and written once.  What stood in the way was
// the number of instructions (265 a pass of two rows, 2.3 issued per cycle),
// so all that does not depend on the token is done once: a warp keeps the same
// heads for every token of its CTA (addresses, kinds), and the norm's weights
// are multiplied into the token's cosines and sines, once per token, in shared
// memory:  y = (x * wc + x_partner * ws) / rms.  The next token's rows are
// loaded before the present one's are worked on.
template <typename T, int D, bool E4M3, int MODE, bool INTER>
__global__ void __launch_bounds__(kThreads, 2) heads_kernel(const __grid_constant__ HeadsArgs a, int q_passes, int kv_passes, int wpt_shift) {
  constexpr int LPR = D / 8;          // lanes per row
  constexpr int RPW = 32 / LPR;       // rows per warp and pass
  constexpr int U = 4;                // rows of a lane on their way
  // [buffer][token of the CTA][query, key][wc, ws][element]
  __shared__ __align__(16) float table[2][kThreads / 32][2][2][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int l = lane % LPR, sub = lane / LPR;
  const int wpt = 1 << wpt_shift;     // warps per token
  const int seat = warp >> wpt_shift, wt = warp & (wpt - 1), seats = (kThreads / 32) >> wpt_shift;
  const int tokens = a.batch * a.n_tokens;
  const int rot = a.rope.rot;
  const int passes = q_passes + kv_passes * (MODE == HEADS_DENSE ? 1 : 2);
  const int groups = (passes + U * wpt - 1) / (U * wpt);
  // the lane's element groups [oa, oa + 4), [ob, ob + 4): partners are equal places of the two, or neighbours
  int oa = 4 * l, ob = D / 2 + 4 * l;
  if (!INTER && rot < D) {
    const int j = l - rot / 8;
    oa = j < 0 ? 4 * l : rot + 4 * j;
    ob = j < 0 ? 4 * l + rot / 2 : rot + (D - rot) / 2 + 4 * j;
  }
  const bool q_norm = a.rope.q_weight != nullptr, k_norm = a.rope.k_weight != nullptr;

  // rows of a group: kind 0 query, 1 key, 2 value, 3 none
  int kind[U], page_off[U];
  bool on[U];
  int64_t src_off[U], dst_off[U];
  auto setup = [&](int grp) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int p = (grp * U + u) * wpt + wt;
      kind[u] = p >= passes ? 3 : p < q_passes ? 0 : p < q_passes + kv_passes ? 1 : 2;
      const int h = (kind[u] == 0 ? p : kind[u] == 1 ? p - q_passes : p - q_passes - kv_passes) * RPW + sub;
      on[u] = kind[u] < 3 && h < (kind[u] == 0 ? a.Hq : a.Hkv);
      src_off[u] = h * (kind[u] == 0 ? a.q.hs : kind[u] == 1 ? a.k.hs : a.v.hs);
      dst_off[u] = h * (kind[u] == 0 ? a.qo.hs : a.ko.hs);
      page_off[u] = (h * 2 + kind[u] - 1) << a.pg.page_shift;
    }
  };
  Raw4<T> xa[U], xb[U];
  auto load = [&](int t) {
    const int b = t / a.n_tokens, i = t - b * a.n_tokens;
    const T* q = reinterpret_cast<const T*>(a.q.p) + b * a.q.bs + i * a.q.ts;
    const T* k = reinterpret_cast<const T*>(a.k.p) + b * a.k.bs + i * a.k.ts;
    const T* v = reinterpret_cast<const T*>(a.v.p) + b * a.v.bs + i * a.v.ts;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!on[u]) continue;
      const T* row = (kind[u] == 0 ? q : kind[u] == 1 ? k : v) + src_off[u];
      xa[u] = *reinterpret_cast<const Raw4<T>*>(row + oa);
      xb[u] = *reinterpret_cast<const Raw4<T>*>(row + ob);
    }
  };

  // pairs that this lane turns, for every token: wt * 32 + lane, and wpt * 32 on
  constexpr int kSlots = D / 64;
  auto first_of = [&](int p) { return INTER ? 2 * p : p < rot / 2 ? p : 2 * p; };
  auto second_of = [&](int p) { return INTER ? 2 * p + 1 : p < rot / 2 ? p + rot / 2 : 2 * p + 1; };
  uint64_t freq[kSlots];
#pragma unroll
  for (int x = 0; x < kSlots; ++x) {
    const int p = wt * 32 + lane + x * wpt * 32;
    freq[x] = p < rot / 2 ? turn_step(a.rope.inv_freq[p]) : 0;
  }

  int t = blockIdx.x * seats + seat;
  const int step = gridDim.x * seats;
  setup(0);
  int pos = 0, slot_next = -1;
  if (t < tokens) {
    load(t);
    pos = a.pos[t];
    if (MODE != HEADS_DENSE) slot_next = a.slots[t];
  }
  int buf = 0;
  for (int t0 = blockIdx.x * seats; t0 < tokens; t0 += step, t += step, buf ^= 1) {
    const bool live = t < tokens;
    float (&tab)[2][2][D] = table[buf][seat];
    if (live) {
#pragma unroll
      for (int x = 0; x < kSlots; ++x) {
        const int p = wt * 32 + lane + x * wpt * 32;
        if (p >= D / 2) break;
        const int ea = first_of(p), eb = second_of(p);
        float c = 1.f, s = 0.f;
        if (p < rot / 2) turn_of(pos, freq[x], a.rope.scale, c, s);
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const float* w = y == 0 ? a.rope.q_weight : a.rope.k_weight;
          const float wa = w ? w[ea] : 1.f, wb = w ? w[eb] : 1.f;
          tab[y][0][ea] = wa * c; tab[y][0][eb] = wb * c;
          tab[y][1][ea] = -(wb * s); tab[y][1][eb] = wa * s;
        }
      }
    }
    __syncthreads();
    const int slot = slot_next;
    bool keep = MODE != HEADS_DENSE && live && slot >= 0;
    if (keep && (slot >> a.pg.page_shift) >= a.pg.n_pages) {
      keep = false;
      if (lane == 0 && wt == 0) set_error(a.pg.err, DEVERR_BAD_INDEX);
    }
    const int64_t page_base = ((static_cast<int64_t>(slot >> a.pg.page_shift) * a.pg.Hkv * 2) << a.pg.page_shift) +
                              (slot & ((1 << a.pg.page_shift) - 1));
    const int b = t / a.n_tokens, i = t - b * a.n_tokens;
    T* const qo = reinterpret_cast<T*>(a.qo.p) + b * a.qo.bs + i * a.qo.ts;
    T* const ko = reinterpret_cast<T*>(a.ko.p) + b * a.ko.bs + i * a.ko.ts;

    for (int grp = 0; grp < groups; ++grp) {
      if (groups > 1) {
        setup(grp);
        if (live && grp > 0) load(t);
      }
      Raw4<T> ya[U], yb[U];
#pragma unroll
      for (int u = 0; u < U; ++u) { ya[u] = xa[u]; yb[u] = xb[u]; }
      if (grp == groups - 1) {       // the next token's first rows
        const int tn = t + step;
        if (tn < tokens) {
          if (groups == 1) load(tn);
          pos = a.pos[tn];
          if (MODE != HEADS_DENSE) slot_next = a.slots[tn];
        }
      }
      int held = -1;                 // kind whose factors are in wc, ws
      float wc[8], ws[8];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (kind[u] == 3) break;     // the same for the whole warp
        float y[8];
        if (on[u]) {
          unpack4(ya[u], y);
          unpack4(yb[u], y + 4);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = 0.f;
        }
        if (kind[u] < 2) {
          if (held != kind[u]) {
            held = kind[u];
            load4<float>(&tab[held][0][oa], wc);
            load4<float>(&tab[held][0][ob], wc + 4);
            load4<float>(&tab[held][1][oa], ws);
            load4<float>(&tab[held][1][ob], ws + 4);
          }
          float rn = 1.f;
          if (held == 0 ? q_norm : k_norm) {
            float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
              const float2 v = make_float2(y[e], y[e + 1]);
              s2 = ffma2(v, v, s2);
            }
            float ss = s2.x + s2.y;
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            rn = rsqrtf(fmaf(ss, 1.f / D, a.rope.eps));
          }
          float z[8];
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const float2 v = make_float2(y[e], y[e + 1]);
            const float2 w = INTER ? make_float2(y[e + 1], y[e]) : make_float2(y[e ^ 4], y[(e ^ 4) + 1]);
            float2 r = __fmul2_rn(w, make_float2(ws[e], ws[e + 1]));
            r = ffma2(v, make_float2(wc[e], wc[e + 1]), r);
            r = __fmul2_rn(r, make_float2(rn, rn));
            z[e] = r.x; z[e + 1] = r.y;
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = z[e];
        }
        if (kind[u] == 0 || MODE == HEADS_DENSE) {
          if (live && on[u]) {
            T* row = (kind[u] == 0 ? qo : ko) + dst_off[u];
            store4<T>(row + oa, y);
            store4<T>(row + ob, y + 4);
          }
          continue;
        }
        if constexpr (MODE != HEADS_DENSE) {
          const int64_t at = page_base + page_off[u];
          if constexpr (E4M3) {
            uint32_t m = top_bits(y);
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
            if (keep && on[u]) {
              const float scale = scale_of(__uint_as_float(m));
              quotients(y, scale);
              uint8_t* row = a.pg.pages + at * D;
              *reinterpret_cast<uint32_t*>(row + oa) = to_e4m3x4(y);
              *reinterpret_cast<uint32_t*>(row + ob) = to_e4m3x4(y + 4);
              if (l == 0) a.pg.scales[at] = scale;
            }
          } else if (keep && on[u]) {
            T* row = reinterpret_cast<T*>(a.pg.pages) + at * D;
            store4<T>(row + oa, y);
            store4<T>(row + ob, y + 4);
          }
        }
      }
    }
    if (groups > 1) {
      setup(0);
      if (t + step < tokens) load(t + step);
    }
  }
}

// Eight consecutive elements as they lie in memory.
template <typename T> struct Raw8;
template <> struct __align__(16) Raw8<float> { float4 a, b; };
template <> struct __align__(16) Raw8<__nv_bfloat16> { uint4 a; };

// Keys and values of new tokens into pages.  Bound by HBM.  A warp takes one
// token's keys or values (blockIdx.y: which, and which `chunk` of their
// passes), RPW rows a pass, U rows per lane on their way at a time.
template <typename T, int D, bool E4M3>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ HeadsArgs a, int passes, int chunk) {
  constexpr int LPR = D / 8, RPW = 32 / LPR, U = 4;
  const int lane = threadIdx.x & 31, l = lane % LPR, sub = lane / LPR;
  const int t = blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
  if (t >= a.batch * a.n_tokens) return;
  const int kv = blockIdx.y & 1, p_beg = (blockIdx.y >> 1) * chunk, p_end = min(passes, p_beg + chunk);
  const RowsView& src = kv ? a.v : a.k;
  const int b = a.batch == 1 ? 0 : t / a.n_tokens, i = t - b * a.n_tokens;
  int h = p_beg * RPW + sub;
  const T* row = reinterpret_cast<const T*>(src.p) + b * src.bs + i * src.ts + h * src.hs + 8 * l;
  const int64_t hop = RPW * src.hs;
  const int s = a.slots[t];
  const int64_t at0 = ((static_cast<int64_t>(s >> a.pg.page_shift) * a.pg.Hkv * 2 + kv) << a.pg.page_shift) +
                      (s & ((1 << a.pg.page_shift) - 1));
  for (int p0 = p_beg; p0 < p_end; p0 += U) {
    Raw8<T> x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (p0 + u < p_end && h + u * RPW < a.Hkv) x[u] = *reinterpret_cast<const Raw8<T>*>(row);
      row += hop;
    }
    if (s < 0) return;
    if ((s >> a.pg.page_shift) >= a.pg.n_pages) {
      if (lane == 0) set_error(a.pg.err, DEVERR_BAD_INDEX);
      return;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (p0 + u >= p_end) break;
      const bool on = h + u * RPW < a.Hkv;
      const int64_t at = at0 + (static_cast<int64_t>(2 * (h + u * RPW)) << a.pg.page_shift);
      if constexpr (E4M3) {
        // magnitudes in pairs: unsigned order of their bits, as top_bits
        const uint4 w = x[u].a;
        uint32_t m2 = __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu), __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu));
        if (!on) m2 = 0;
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) m2 = __vmaxu2(m2, __shfl_xor_sync(0xffffffffu, m2, o));
        if (on) {
          const float scale = scale_of(__uint_as_float(max(m2 & 0xffff0000u, m2 << 16)));
          float y[8];
          unpack16(w, y, __nv_bfloat16());
          quotients(y, scale);
          *reinterpret_cast<uint2*>(a.pg.pages + at * D + 8 * l) = make_uint2(to_e4m3x4(y), to_e4m3x4(y + 4));
          if (l == 0) a.pg.scales[at] = scale;
        }
      } else if (on) {
        *reinterpret_cast<Raw8<T>*>(reinterpret_cast<T*>(a.pg.pages) + at * D + 8 * l) = x[u];
      }
    }
    h += U * RPW;
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
int append_t(const HeadsArgs& a, int num_sms, cudaStream_t st) {
  constexpr int RPW = 32 / (D / 8), W = kThreads / 32;
  const int passes = (a.Hkv + RPW - 1) / RPW, tokens = a.batch * a.n_tokens;
  // few tokens: one pass per warp, the shortest way through
  const int chunk = static_cast<int64_t>(tokens) * passes < 16 * num_sms ? 1 : passes;
  const dim3 grid((tokens + W - 1) / W, 2 * ((passes + chunk - 1) / chunk));
  append_kernel<T, D, E4M3><<<grid, kThreads, 0, st>>>(a, passes, chunk);
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

template <typename T, int D, bool E4M3, int MODE>
int new_heads_t(const HeadsArgs& a, int num_sms, cudaStream_t st) {
  constexpr int RPW = 32 / (D / 8);
  const int q_passes = (a.Hq + RPW - 1) / RPW, kv_passes = (a.Hkv + RPW - 1) / RPW;
  const int passes = q_passes + kv_passes * (MODE == HEADS_DENSE ? 1 : 2);
  const int64_t tokens = static_cast<int64_t>(a.batch) * a.n_tokens;
  // Warps per token: with few tokens one pass each, for the shortest way
  // through; with many, up to four rows of a lane on their way at once.
  const int most = tokens * passes < 16 * num_sms ? 1 : 4;
  int shift = 0;
  while (shift < 3 && (passes >> shift) > most) ++shift;
  const int seats = (kThreads / 32) >> shift;
  int64_t grid = (tokens + seats - 1) / seats;
  if (grid > 2 * num_sms) grid = 2 * num_sms;      // two CTAs stay on each SM and walk the tokens
  const unsigned n = static_cast<unsigned>(grid);
  if (a.rope.interleaved) heads_kernel<T, D, E4M3, MODE, true><<<n, kThreads, 0, st>>>(a, q_passes, kv_passes, shift);
  else heads_kernel<T, D, E4M3, MODE, false><<<n, kThreads, 0, st>>>(a, q_passes, kv_passes, shift);
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

template <typename T, int D, bool E4M3>
int heads_t(const HeadsArgs& a, int mode, int num_sms, cudaStream_t st) {
  if (mode == HEADS_DENSE) return new_heads_t<T, D, false, HEADS_DENSE>(a, num_sms, st);
  if (mode == HEADS_APPEND) return append_t<T, D, E4M3>(a, num_sms, st);
  return new_heads_t<T, D, E4M3, HEADS_STEP>(a, num_sms, st);
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
