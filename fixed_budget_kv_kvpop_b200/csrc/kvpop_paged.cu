// Paged cache: norm and rotation of new tokens' heads, the write into pages
// (as they are, or e4m3 with one scale per row) and the read back.
//
// All are one pass over rows of d elements.
#include "kvpop_paged.cuh"

#include <atomic>
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

__device__ __forceinline__ uint32_t to_e4m3x4(const float* x) {
  const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[0], x[1]), __NV_SATFINITE, __NV_E4M3);
  const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[2], x[3]), __NV_SATFINITE, __NV_E4M3);
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// A frequency as the fraction of a turn per position, in units of 2^-64.
// Products with a position wrap at whole turns, so the angle of any int32
// position keeps all its bits: off by at most 2^-32 turns from the cut to 32
// bits, and at position 2^31 by 2^-23.6 turns more from the step's own rounding
// for frequencies up to 1 (an fp64 product position * frequency is off by up to
// 2^-24.6 turns there), in proportion below.  And no fp64 instruction is left per token: their
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

// e4m3(x / scale) of N elements.  The quotients have to be the rounded
// ones: bf16 rows often put them on the middle between two held values, and a
// product with the reciprocal would send those to either side.  With r the
// rounded reciprocal, q = x r is off by an ulp or so, and q + (x - q scale) r,
// the remainder being exact in one FMA, is the rounded quotient (Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor",
// 1990).  The tests compare held bytes for every pair of bf16 significands, and
// for fp32 rows under 25 factors.  Below 2^-90 the remainder could underflow:
// those rows divide.
template <int N>
__device__ __forceinline__ void quotients(float (&x)[N], float scale) {
  if (scale == 0.f) {
#pragma unroll
    for (int e = 0; e < N; ++e) x[e] = 0.f;
  } else if (scale < 8.0779357e-28f) {
#pragma unroll
    for (int e = 0; e < N; ++e) x[e] = x[e] / scale;
  } else {
    const float r = 1.f / scale;
    const float2 r2 = make_float2(r, r), s2 = make_float2(-scale, -scale);
#pragma unroll
    for (int e = 0; e < N; e += 2) {
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

// Largest magnitude of N elements as its bits: unsigned order is the order of
// magnitudes, with infinities and then NaN on top.
template <int N>
__device__ __forceinline__ uint32_t top_bits(const float (&x)[N]) {
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < N; ++e) m = max(m, __float_as_uint(x[e]) & 0x7fffffffu);
  return m;
}

// Eight consecutive elements as they lie in memory.
template <typename T> struct Raw8;
template <> struct __align__(16) Raw8<float> { float4 a, b; };
template <> struct __align__(16) Raw8<__nv_bfloat16> { uint4 a; };
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* x) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}
__device__ __forceinline__ void store8(float* p, const float* x) {
  store4<float>(p, x);
  store4<float>(p + 4, x + 4);
}

// Where a lane's 16 elements of a row lie: groups of eight, A and B, each as two
// groups of four.  Partners of a turn are the same places of A and B, or
// neighbours.  WIDE: each group of eight is consecutive and 16-byte aligned.
struct Places {
  int a0, a1, b0, b1;
};
template <typename T, int D, bool INTER>
__device__ __forceinline__ Places places_of(int l, int rot) {
  if (INTER || rot == D) return Places{8 * l, 8 * l + 4, D / 2 + 8 * l, D / 2 + 8 * l + 4};
  if (rot % 16 == 0) {
    const int i = 8 * l < rot / 2 ? 8 * l : rot + 16 * (l - rot / 16);
    const int j = 8 * l < rot / 2 ? i + rot / 2 : i + 8;
    return Places{i, i + 4, j, j + 4};
  }
  // quadruples 2l and 2l + 1 of pairs, each turned or not
  int at[2], to[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int q = 2 * l + x;
    at[x] = 4 * q < rot / 2 ? 4 * q : rot + 8 * (q - rot / 8);
    to[x] = 4 * q < rot / 2 ? at[x] + rot / 2 : at[x] + 4;
  }
  return Places{at[0], at[1], to[0], to[1]};
}
template <int N>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src) {
  if constexpr (N == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(dst), "l"(src) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" :: "r"(dst), "l"(src), "n"(N) : "memory");
}
// Starts the copy of a group of eight elements into this lane's 16-byte cells,
// which lie 512 bytes (a warp's worth) apart.
template <typename T, bool WIDE>
__device__ __forceinline__ void copy_group(uint32_t cell, const T* row, int i, int j) {
  if constexpr (sizeof(T) == 4) {
    cp_async<16>(cell, row + i);
    cp_async<16>(cell + 512, row + j);
  } else if constexpr (WIDE) {
    cp_async<16>(cell, row + i);
  } else {
    cp_async<8>(cell, row + i);
    cp_async<8>(cell + 8, row + j);
  }
}
template <typename T>
__device__ __forceinline__ void read_group(const uint8_t* cell, float* x) {
  if constexpr (sizeof(T) == 4) {
    load4<float>(reinterpret_cast<const float*>(cell), x);
    load4<float>(reinterpret_cast<const float*>(cell + 512), x + 4);
  } else {
    unpack16(*reinterpret_cast<const uint4*>(cell), x, __nv_bfloat16());
  }
}
template <typename T, bool WIDE>
__device__ __forceinline__ void store_group(T* row, int i, int j, const float* x) {
  if constexpr (WIDE) {
    store8(row + i, x);
  } else {
    store4<T>(row + i, x);
    store4<T>(row + j, x + 4);
  }
}
// Sixteen quotients as e4m3.
template <bool WIDE>
__device__ __forceinline__ void store_e4m3(uint8_t* row, const Places& at, const float* x) {
  if constexpr (WIDE) {
    *reinterpret_cast<uint2*>(row + at.a0) = make_uint2(to_e4m3x4(x), to_e4m3x4(x + 4));
    *reinterpret_cast<uint2*>(row + at.b0) = make_uint2(to_e4m3x4(x + 8), to_e4m3x4(x + 12));
  } else {
    *reinterpret_cast<uint32_t*>(row + at.a0) = to_e4m3x4(x);
    *reinterpret_cast<uint32_t*>(row + at.a1) = to_e4m3x4(x + 4);
    *reinterpret_cast<uint32_t*>(row + at.b0) = to_e4m3x4(x + 8);
    *reinterpret_cast<uint32_t*>(row + at.b1) = to_e4m3x4(x + 12);
  }
}

// New tokens' heads.  HEADS_DENSE: queries and keys are normalised, turned and
// written; HEADS_STEP: the same, but keys, and the values as they are, go into pages.
//
// Bound by HBM: every row is read and written once.  What stands in the way is
// the number of instructions and the bytes on their way.  So d / 16 lanes share
// a row (a sum of squares takes three exchanges for four rows), with many
// tokens one warp takes a whole token (position and turns once, no barrier),
// the norm's weights are multiplied into the token's cosines and sines, in
// shared memory:  y = (x * wc + x_partner * ws) / rms,  and rows come by
// asynchronous copies, DEPTH passes ahead across tokens, into cells that only
// the lane that asked for them reads, so that they need no registers and no
// barrier.  ALL: every element is turned (telling them apart takes 16 selects
// a pass: 8192 tokens of 40 heads 33.5 us without, 34.6 us with).
constexpr int kHeadsDepth = 3;      // 4096 tokens of 40 heads: 3 18.4 us, 4 18.2, 6 18.6, 8 19.0; 8192: 33.1, 33.4, 33.4, 34.3; 32768: 112, 122, 123, 121
template <typename T, int D, bool E4M3, int MODE, bool INTER, bool WIDE, bool ALL>
__global__ void __launch_bounds__(kThreads, 2) heads_kernel(const __grid_constant__ HeadsArgs a, int q_passes, int kv_passes, int wpt_shift) {
  constexpr int LPR = D / 16;         // lanes per row
  constexpr int RPW = 32 / LPR;       // rows per warp and pass
  constexpr int kSlots = D / 64;      // pairs of a lane, at most
  constexpr int PASS = 32 * 16 * sizeof(T);      // bytes of a pass
  constexpr int DEPTH = kHeadsDepth;
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int l = lane % LPR, sub = lane / LPR;
  const int wpt = 1 << wpt_shift;     // warps per token
  const int seat = warp >> wpt_shift, wt = warp & (wpt - 1), seats = (kThreads / 32) >> wpt_shift;
  const int tokens = a.batch * a.n_tokens;
  const int passes = q_passes + kv_passes * (MODE == HEADS_DENSE ? 1 : 2);
  const int rot = ALL ? D : a.rope.rot;
  const Places at_ = places_of<T, D, INTER>(l, rot);
  const bool turned[4] = {at_.a0 < rot, at_.a1 < rot, at_.b0 < rot, at_.b1 < rot};
  uint8_t* const ring = smem + warp * (DEPTH * PASS) + lane * 16;
  float* const tab = reinterpret_cast<float*>(smem + (kThreads / 32) * (DEPTH * PASS)) + seat * (4 * D);   // [query, key][wc, ws][element]

  const int step = gridDim.x * seats;
  auto batch_of = [&](int t) { return a.batch == 1 ? 0 : t / a.n_tokens; };

  // ---- copies: pass g of token pt, DEPTH passes ahead ----
  int pt = blockIdx.x * seats + seat, pg = wt, p_cell = 0;
  const T *pq = nullptr, *pk = nullptr, *pv = nullptr;
  auto open = [&]() {
    if (pt >= tokens) return;
    const int b = batch_of(pt), i = pt - b * a.n_tokens;
    pq = reinterpret_cast<const T*>(a.q.p) + b * a.q.bs + i * a.q.ts;
    pk = reinterpret_cast<const T*>(a.k.p) + b * a.k.bs + i * a.k.ts;
    if (MODE == HEADS_STEP) pv = reinterpret_cast<const T*>(a.v.p) + b * a.v.bs + i * a.v.ts;
  };
  auto ask = [&]() {
    if (pt < tokens && pg < passes) {
      const int kind = pg < q_passes ? 0 : pg < q_passes + kv_passes ? 1 : 2;
      const int h = (kind == 0 ? pg : kind == 1 ? pg - q_passes : pg - q_passes - kv_passes) * RPW + sub;
      if (h < (kind == 0 ? a.Hq : a.Hkv)) {
        const T* row = kind == 0 ? pq + h * a.q.hs : kind == 1 ? pk + h * a.k.hs : pv + h * a.v.hs;
        const uint32_t cell = smem_u32(ring) + p_cell * PASS;
        copy_group<T, WIDE>(cell, row, at_.a0, at_.a1);
        copy_group<T, WIDE>(cell + PASS / 2, row, at_.b0, at_.b1);
      }
      p_cell = p_cell + 1 == DEPTH ? 0 : p_cell + 1;
      pg += wpt;
      if (pg >= passes) {
        pg = wt;
        pt += step;
        open();
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  wait_for_prior_kernel();
  // positions and slots are read one token ahead, frequencies before the first copies are asked for
  int pos_next = 0, slot_next = -1;
  auto look = [&](int t) {
    if (t >= tokens) return;
    pos_next = a.pos[t];
    if (MODE == HEADS_STEP) slot_next = a.slots[t];
  };
  look(pt);
  // pairs that this lane turns, for every token: wt * 32 + lane, and wpt * 32 on
  double inv_freq[kSlots];
  uint64_t freq[kSlots];
#pragma unroll
  for (int x = 0; x < kSlots; ++x) {
    const int p = wt * 32 + lane + x * wpt * 32;
    inv_freq[x] = p < rot / 2 ? a.rope.inv_freq[p] : 0.0;
  }
  open();
#pragma unroll 1
  for (int x = 0; x < DEPTH; ++x) ask();
#pragma unroll
  for (int x = 0; x < kSlots; ++x) freq[x] = turn_step(inv_freq[x]);

  int cell = 0;
#pragma unroll 1
  for (int t0 = blockIdx.x * seats; t0 < tokens; t0 += step) {
    const int t = t0 + seat;
    const bool live = t < tokens;
    const int pos = pos_next, slot = slot_next;
    look(t + step);
    if (live) {
#pragma unroll
      for (int x = 0; x < kSlots; ++x) {
        const int p = wt * 32 + lane + x * wpt * 32;
        if (p >= D / 2) break;
        const int ea = INTER ? 2 * p : p < rot / 2 ? p : 2 * p;
        const int eb = INTER ? 2 * p + 1 : p < rot / 2 ? p + rot / 2 : 2 * p + 1;
        float c = 1.f, s = 0.f;
        if (p < rot / 2) turn_of(pos, freq[x], a.rope.scale, c, s);
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const float* w = y == 0 ? a.rope.q_weight : a.rope.k_weight;
          const float wa = w ? w[ea] : 1.f, wb = w ? w[eb] : 1.f;
          float* to = tab + 2 * y * D;
          to[ea] = wa * c; to[eb] = wb * c;
          to[D + ea] = -(wb * s); to[D + eb] = wa * s;
        }
      }
    }
    if (wpt_shift) __syncthreads();
    else __syncwarp();
    bool keep = MODE == HEADS_STEP && live && slot >= 0;
    if (keep && (slot >> a.pg.page_shift) >= a.pg.n_pages) {
      keep = false;
      if (lane == 0 && wt == 0) set_error(a.pg.err, DEVERR_BAD_INDEX);
    }
    const int64_t page_base = ((static_cast<int64_t>(slot >> a.pg.page_shift) * a.pg.Hkv * 2) << a.pg.page_shift) +
                              (slot & ((1 << a.pg.page_shift) - 1));
    if (live) {
      const int b = batch_of(t), i = t - b * a.n_tokens;
      T* const qo = reinterpret_cast<T*>(a.qo.p) + b * a.qo.bs + i * a.qo.ts;
      T* const ko = reinterpret_cast<T*>(a.ko.p) + b * a.ko.bs + i * a.ko.ts;
      int held = -1;                  // kind whose factors are in wc, ws
      float wc[16], ws[16];
#pragma unroll 1
      for (int g = wt; g < passes; g += wpt) {
        const int kind = g < q_passes ? 0 : g < q_passes + kv_passes ? 1 : 2;    // the same for the warp
        const int h = (kind == 0 ? g : kind == 1 ? g - q_passes : g - q_passes - kv_passes) * RPW + sub;
        const bool on = h < (kind == 0 ? a.Hq : a.Hkv);
        asm volatile("cp.async.wait_group %0;" :: "n"(DEPTH - 1) : "memory");
        float y[16];
        read_group<T>(ring + cell * PASS, y);
        read_group<T>(ring + cell * PASS + PASS / 2, y + 8);
        cell = cell + 1 == DEPTH ? 0 : cell + 1;
        if (kind < 2) {
          if (held != kind) {
            held = kind;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              float* w = x == 0 ? wc : ws;
              const float* from = tab + (2 * kind + x) * D;
              load4<float>(from + at_.a0, w);
              load4<float>(from + at_.a1, w + 4);
              load4<float>(from + at_.b0, w + 8);
              load4<float>(from + at_.b1, w + 12);
            }
          }
          float rn = 1.f;
          if ((kind == 0 ? a.rope.q_weight : a.rope.k_weight) != nullptr) {
            float2 s2 = make_float2(0.f, 0.f), s3 = s2;
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
              const float2 v = make_float2(y[e], y[e + 1]), w = make_float2(y[e + 2], y[e + 3]);
              s2 = ffma2(v, v, s2);
              s3 = ffma2(w, w, s3);
            }
            float ss = (s2.x + s2.y) + (s3.x + s3.y);
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            rn = rsqrtf(fmaf(ss, 1.f / D, a.rope.eps));
          }
          float z[16];
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            const float2 v = make_float2(y[e], y[e + 1]);
            const float2 w = INTER ? make_float2(y[e + 1], y[e]) : make_float2(y[e ^ 8], y[(e ^ 8) + 1]);
            float2 r = __fmul2_rn(w, make_float2(ws[e], ws[e + 1]));
            if (!ALL && !turned[e / 4]) r = make_float2(0.f, 0.f);      // not w * 0: w may be an infinity
            r = ffma2(v, make_float2(wc[e], wc[e + 1]), r);
            r = __fmul2_rn(r, make_float2(rn, rn));
            z[e] = r.x; z[e + 1] = r.y;
          }
#pragma unroll
          for (int e = 0; e < 16; ++e) y[e] = z[e];
        }
        if (MODE == HEADS_DENSE || kind == 0) {
          if (on) {
            T* row = kind == 0 ? qo + h * a.qo.hs : ko + h * a.ko.hs;
            store_group<T, WIDE>(row, at_.a0, at_.a1, y);
            store_group<T, WIDE>(row, at_.b0, at_.b1, y + 8);
          }
        } else {
          const int64_t at = page_base + (static_cast<int64_t>(h * 2 + kind - 1) << a.pg.page_shift);
          if constexpr (E4M3) {
            uint32_t m = on ? top_bits(y) : 0u;
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
            if (keep && on) {
              const float scale = scale_of(__uint_as_float(m));
              quotients(y, scale);
              store_e4m3<WIDE>(a.pg.pages + at * D, at_, y);
              if (l == 0) a.pg.scales[at] = scale;
            }
          } else if (keep && on) {
            T* row = reinterpret_cast<T*>(a.pg.pages) + at * D;
            store_group<T, WIDE>(row, at_.a0, at_.a1, y);
            store_group<T, WIDE>(row, at_.b0, at_.b1, y + 8);
          }
        }
        ask();
      }
    }
    // the table is written again for the next token
    if (t0 + step < tokens) {
      if (wpt_shift) __syncthreads();
      else __syncwarp();
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}
template <typename T, int D>
constexpr int heads_smem() { return (kThreads / 32) * (kHeadsDepth * 32 * 16 * static_cast<int>(sizeof(T)) + 4 * D * 4); }

// Keys and values of new tokens into pages.  Bound by HBM.  A warp takes one
// token's keys or values (blockIdx.y: which, and which `chunk` of their
// passes), RPW rows a pass, U passes on their way at a time.  Rows that are
// only copied take d / 8 lanes (16 bytes each in bf16), rows that are
// quantised d / 16, which halves the exchanges and reciprocals per row.  Five
// blocks per SM: 65536 tokens to 8 bits take 76.8 us, 80.6 with four, 77.7 with six.
template <typename T, int D, bool E4M3>
__global__ void __launch_bounds__(kThreads, 5) append_kernel(const __grid_constant__ HeadsArgs a, int passes, int chunk) {
  constexpr int LPR = E4M3 ? D / 16 : D / 8, RPW = 32 / LPR, U = E4M3 ? 2 : 4;
  wait_for_prior_kernel();
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
    Raw8<T> x[U], x2[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (p0 + u < p_end && h + u * RPW < a.Hkv) {
        x[u] = *reinterpret_cast<const Raw8<T>*>(row);
        if (E4M3) x2[u] = *reinterpret_cast<const Raw8<T>*>(row + D / 2);
      }
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
        const uint4 w = x[u].a, w2 = x2[u].a;
        constexpr uint32_t k = 0x7fff7fffu;
        uint32_t m2 = __vmaxu2(__vmaxu2(__vmaxu2(w.x & k, w.y & k), __vmaxu2(w.z & k, w.w & k)),
                               __vmaxu2(__vmaxu2(w2.x & k, w2.y & k), __vmaxu2(w2.z & k, w2.w & k)));
        if (!on) m2 = 0;
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) m2 = __vmaxu2(m2, __shfl_xor_sync(0xffffffffu, m2, o));
        if (on) {
          const float scale = scale_of(__uint_as_float(max(m2 & 0xffff0000u, m2 << 16)));
          float y[16];
          unpack16(w, y, __nv_bfloat16());
          unpack16(w2, y + 8, __nv_bfloat16());
          quotients(y, scale);
          uint8_t* held = a.pg.pages + at * D + 8 * l;
          *reinterpret_cast<uint2*>(held) = make_uint2(to_e4m3x4(y), to_e4m3x4(y + 4));
          *reinterpret_cast<uint2*>(held + D / 2) = make_uint2(to_e4m3x4(y + 8), to_e4m3x4(y + 12));
          if (l == 0) a.pg.scales[at] = scale;
        }
      } else if (on) {
        *reinterpret_cast<Raw8<T>*>(reinterpret_cast<T*>(a.pg.pages) + at * D + 8 * l) = x[u];
      }
    }
    h += U * RPW;
  }
}

// Rows of sequences back out of their pages.  Bound by HBM.  A block takes
// kGatherTokens tokens of one sequence and head, keys or values: they lie one
// after another in their pages.  A lane moves 16 bytes of held elements, and
// all rows of a lane are on their way before the first is converted.
constexpr int kGatherTokens = 64;

template <typename T, int D, bool E4M3>
__global__ void __launch_bounds__(kThreads) gather_kernel(const __grid_constant__ GatherArgs a) {
  constexpr int PER = 16 / (E4M3 ? 1 : static_cast<int>(sizeof(T)));    // elements per lane
  constexpr int LPR = D / PER, STEP = kThreads / LPR, U = (kGatherTokens + STEP - 1) / STEP;
  const int l = threadIdx.x % LPR;
  wait_for_prior_kernel();
  const int b = blockIdx.z, h = blockIdx.y >> 1, kv = blockIdx.y & 1;
  int n = a.lens[b];
  const int64_t cap = min(static_cast<int64_t>(a.n_tokens), static_cast<int64_t>(a.width) << a.pg.page_shift);
  if (n < 0 || n > cap) {
    if (threadIdx.x == 0 && blockIdx.x == 0) set_error(a.pg.err, DEVERR_BAD_INDEX);
    n = n < 0 ? 0 : static_cast<int>(cap);
  }
  const RowsView& dst = kv ? a.v : a.k;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kGatherTokens + threadIdx.x / LPR;
  uint4 held[U];
  float scale[U];
  bool on[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t i = t0 + u * STEP;
    on[u] = false;
    if (i >= n || u * STEP + static_cast<int>(threadIdx.x) / LPR >= kGatherTokens) continue;
    const int page = a.table[b * a.table_stride + (i >> a.pg.page_shift)];
    if (page < 0 || page >= a.pg.n_pages) {
      if (l == 0) set_error(a.pg.err, DEVERR_BAD_INDEX);
      continue;
    }
    on[u] = true;
    const int64_t row = (((static_cast<int64_t>(page) * a.pg.Hkv + h) * 2 + kv) << a.pg.page_shift) +
                        (i & ((1 << a.pg.page_shift) - 1));
    held[u] = *reinterpret_cast<const uint4*>(a.pg.pages + (row * LPR + l) * 16);
    if (E4M3) scale[u] = a.pg.scales[row];
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (!on[u]) continue;
    T* out = reinterpret_cast<T*>(dst.p) + b * dst.bs + (t0 + u * STEP) * dst.ts + h * dst.hs + PER * l;
    if constexpr (E4M3) {
      const uint32_t w[4] = {held[u].x, held[u].y, held[u].z, held[u].w};
      float x[16];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[i / 2] >> (16 * (i & 1))), __NV_E4M3);
        const float2 f = __half22float2(__half2(r));
        x[2 * i] = f.x * scale[u];
        x[2 * i + 1] = f.y * scale[u];
      }
      store8(out, x);
      store8(out + 8, x + 8);
    } else {
      *reinterpret_cast<uint4*>(out) = held[u];
    }
  }
}

template <typename T, int D, bool E4M3>
int append_t(const HeadsArgs& a, int num_sms, cudaStream_t st) {
  constexpr int RPW = 32 / (E4M3 ? D / 16 : D / 8), W = kThreads / 32;
  const int passes = (a.Hkv + RPW - 1) / RPW, tokens = a.batch * a.n_tokens;
  // few tokens: one pass per warp, the shortest way through
  const int chunk = static_cast<int64_t>(tokens) * passes < 16 * num_sms ? 1 : passes;
  const dim3 grid((tokens + W - 1) / W, 2 * ((passes + chunk - 1) / chunk));
  return launch_dependent(append_kernel<T, D, E4M3>, grid, kThreads, 0, st, a, passes, chunk);
}

template <typename T, int D, bool E4M3, int MODE>
int new_heads_t(const HeadsArgs& a, int num_sms, cudaStream_t st) {
  constexpr int RPW = 32 / (D / 16);
  const int q_passes = (a.Hq + RPW - 1) / RPW, kv_passes = (a.Hkv + RPW - 1) / RPW;
  const int passes = q_passes + kv_passes * (MODE == HEADS_DENSE ? 1 : 2);
  const int64_t tokens = static_cast<int64_t>(a.batch) * a.n_tokens;
  // Warps per token: as many as it takes to have 16 warps on each SM, up to one pass each.
  int shift = 0;
  while (shift < 3 && (passes >> shift) > 1 && (tokens << shift) < 16 * num_sms) ++shift;
  const int seats = (kThreads / 32) >> shift;
  int64_t grid = (tokens + seats - 1) / seats;
  if (grid > 2 * num_sms) grid = 2 * num_sms;      // two CTAs stay on each SM and walk the tokens
  const bool all = a.rope.rot == D;
  const int which = (a.rope.interleaved ? 0 : a.rope.rot % 16 == 0 ? 2 : 4) + (all ? 1 : 0);
  const auto kernel = which == 0   ? heads_kernel<T, D, E4M3, MODE, true, true, false>
                      : which == 1 ? heads_kernel<T, D, E4M3, MODE, true, true, true>
                      : which == 2 ? heads_kernel<T, D, E4M3, MODE, false, true, false>
                      : which == 3 ? heads_kernel<T, D, E4M3, MODE, false, true, true>
                                   : heads_kernel<T, D, E4M3, MODE, false, false, false>;
  constexpr int smem = heads_smem<T, D>();
  if (smem > 48 * 1024) {
    // once for each device (up to 64 of them) and variant
    static std::atomic<uint64_t> done[5];
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess) return -1;
    const uint64_t bit = UINT64_C(1) << (device & 63);
    if (device > 63 || !(done[which].load(std::memory_order_relaxed) & bit)) {
      if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return -1;
      done[which].fetch_or(bit, std::memory_order_relaxed);
    }
  }
  return launch_dependent(kernel, dim3(static_cast<unsigned>(grid)), kThreads, smem, st, a, q_passes, kv_passes, shift);
}

template <typename T, int D, bool E4M3>
int heads_t(const HeadsArgs& a, int mode, int num_sms, cudaStream_t st) {
  if (mode == HEADS_DENSE) return new_heads_t<T, D, false, HEADS_DENSE>(a, num_sms, st);
  if (mode == HEADS_APPEND) return append_t<T, D, E4M3>(a, num_sms, st);
  return new_heads_t<T, D, E4M3, HEADS_STEP>(a, num_sms, st);
}

template <typename T, int D, bool E4M3>
int gather_t(const GatherArgs& a, cudaStream_t st) {
  const dim3 grid((static_cast<unsigned>(a.n_tokens) + kGatherTokens - 1) / kGatherTokens, a.pg.Hkv * 2, a.batch);
  return launch_dependent(gather_kernel<T, D, E4M3>, grid, kThreads, 0, st, a);
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
