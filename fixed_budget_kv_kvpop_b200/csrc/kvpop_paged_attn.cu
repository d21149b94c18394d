// Attention of one new token per sequence over its pages, in one launch.
//
//   s_j = scale q . k_j  (then cap tanh(s_j / cap)),  out = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m)
//
// Work split.  The keys of a sequence are cut into blocks of KB.  CTAs work in
// groups of Hkv, one for each KV head, so that the heads of a page, which are
// neighbours in memory, are read at the same time.  The groups either take one
// part of one sequence each, all parts as even as they come, or, where that
// leaves the largest part well above the average, equal contiguous ranges of
// all sequences' blocks (32 sequences of 16384 to 32768 tokens in 8 bits: 331
// and 239 us; 16 of 8192 in fp32: 163 and 181 us).  Every CTA finds its range
// from the lengths on the device.  Where the page table is so narrow that even
// the longest sequences it can hold give no more parts of kMinShare blocks than
// there are groups, those are the parts, and nothing is searched for: short
// calls are a chain of latencies (117 tokens: 5.5 us so, 6.1 us searched).
// Many sequences of a few blocks each go, head by head, to single warps, which
// then meet nobody (512 of 60 tokens: 38 us so, 72 us with a CTA for each).
// Where a sequence lies in several ranges, each leaves a partial (accumulator,
// running maximum, sum), and the CTA that arrives last joins them in their
// order, so results do not depend on who is last.
// Inside a CTA each warp has a ring of stages of its own: it copies block after
// block into it by tensor copies (one instruction per 16 keys and values) and
// computes on the oldest, the next one or more being on their way.  Warps meet once per item, to join their sums.
#include "kvpop_paged.cuh"
#include "kvpop_paged_split.cuh"

#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cudaTypedefs.h>

namespace kvpop {
namespace {

constexpr int NW = 4;                    // warps per CTA
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// Weights are relative to a running maximum, kRaise (in powers of two) above the largest score when it was set: it
// moves when a score passes it, so that no weight passes 1 and few scores move it.
constexpr float kRaise = 8.f;

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ void tma_load_5d(void* dst, const CUtensorMap* map, int x, int y, int z, int k, int w,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];"
      :: "r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(k), "r"(w),
         "r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void mma_f16_16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
               "{%8, %9}, {%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two e4m3 bytes -> f16 pair, exactly.
__device__ __forceinline__ uint32_t e4m3_to_f16(uint32_t x) {
  uint32_t r;
  asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, lo;\n}" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t e4m3_to_f16_high(uint32_t x) {
  uint32_t r;
  asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, hi;\n}" : "=r"(r) : "r"(x));
  return r;
}
// (lo, hi) -> f16x2 word, round to nearest even; lo in the low half.
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Four e4m3 bytes -> bf16 pairs of bytes 0, 2 and of bytes 1, 3, exactly.
__device__ __forceinline__ void e4m3_to_bf16(uint32_t x, uint32_t& even, uint32_t& odd) {
  const uint32_t lo = e4m3_to_f16(x), hi = e4m3_to_f16_high(x);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  even = __byte_perm(__float_as_uint(a.x), __float_as_uint(b.x), 0x7632);   // four significant bits: the upper halves are all
  odd = __byte_perm(__float_as_uint(a.y), __float_as_uint(b.y), 0x7632);
}

// The lanes of a warp, for the split's arithmetic.  nb0: blocks of sequence `lane`.
template <typename Sum>
struct LaneWarp {
  using Lanes = int;
  struct Hit {
    int lane, own;
    int64_t sum;     // up to the lane, or (not found) of all
  };
  int nb0;
  template <typename F> __device__ __forceinline__ int lanes(F f) const { return f(static_cast<int>(threadIdx.x & 31)); }
  template <typename F> __device__ __forceinline__ int cached(F) const { return nb0; }
  template <typename F> __device__ __forceinline__ int each(int v, F f) const { return f(v); }
  __device__ __forceinline__ int few(int v) const { return __reduce_add_sync(0xffffffffu, v); }
  __device__ __forceinline__ int64_t sum(int v) const {
    if (sizeof(Sum) == 4) return __reduce_add_sync(0xffffffffu, static_cast<unsigned>(v));
    return (static_cast<int64_t>(few(v >> 16)) << 16) + few(v & 0xffff);
  }
  __device__ __forceinline__ int top(int v) const { return __reduce_max_sync(0xffffffffu, v); }
  __device__ __forceinline__ int some(int v) const { return __popc(__ballot_sync(0xffffffffu, v > 0)); }
  __device__ __forceinline__ bool find(int v, int64_t before, int64_t target, bool many, Hit& hit) const {
    const int lane = threadIdx.x & 31;
    Sum sum = v;
    if (many) {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const Sum u = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += u;
      }
    }
    const unsigned past = __ballot_sync(0xffffffffu, before + static_cast<int64_t>(sum) > target);
    hit.lane = past ? __ffs(past) - 1 : 31;
    hit.own = __shfl_sync(0xffffffffu, v, hit.lane);
    hit.sum = static_cast<int64_t>(__shfl_sync(0xffffffffu, sum, hit.lane));
    return past != 0;
  }
};

// The whole warp's next item, made by its first lane.
template <typename F>
__device__ __forceinline__ void put_item(Item* it, F make) {
  __syncwarp();                      // the old item has been read
  if ((threadIdx.x & 31) == 0) *it = make();
  __syncwarp();
}
// The item of a group where parts are fixed.
template <int KB>
__device__ __forceinline__ bool fixed_item(const Split& sp, Item* it, int grp, int h) {
  Item x;
  if (!fixed_part<KB>(sp, grp, h, x)) return false;
  put_item(it, [&] { return x; });
  return true;
}
// The warp's first or next item where warps take one sequence and head each (pos: which).
template <int KB>
__device__ __noinline__ bool solo_item(const Split* spp, Item* it, bool start) {
  const int warps = gridDim.x * NW;
  Item x;
  if (!solo_part<KB>(*spp, start ? static_cast<int>(blockIdx.x) * NW + static_cast<int>(threadIdx.x) / 32 : static_cast<int>(it->pos) + warps, warps, x))
    return false;
  put_item(it, [&] { return x; });
  return true;
}
// The CTA's first or next item; false at the end.  nb0: blocks of sequence `lane`.
template <int KB>
__device__ __noinline__ bool next_item(const Split* spp, Item* it, int nb0, bool start) {
  LaneWarp<BlockSum<KB>> w{nb0};
  return next_part<KB>(w, *spp, *it, start, blockIdx.x, gridDim.x, [&](auto make) { put_item(it, make); });
}

// An item that is a part of its sequence, kept until the parts are joined.
struct Part {
  int b, h, first, parts, second;    // as Item
};
// Shared memory of a CTA beside its rings, the accumulators to join and the weights.
template <int GP, int NST>
struct AttendShared {
  uint64_t bars[NW][NST];
  Split split[NW];
  Item items[NW][2];
  float ml[NW][GP][2];     // each warp's running maxima and sums
  int32_t any[NW];         // whether it saw a key
  Part open[2];
  int32_t last[2];
  int32_t live[NW][NST];   // pieces that were copied into a stage
};

// What a warp's ring holds.  A block is NSUB pieces of KEYS keys and values;
// a piece comes by one tensor copy (bf16, e4m3) or two plain ones (fp32).
template <typename T, int D, bool E4M3, int GP>
struct Geo {
  static constexpr bool F32 = sizeof(T) == 4;
  static constexpr int ES = E4M3 ? 1 : static_cast<int>(sizeof(T));
  static constexpr int KEYS = F32 && D == 128 ? 8 : 16;
  static constexpr int SUB = 2 * KEYS * D * ES;              // bytes of a piece
  static constexpr int STAGE = 8192;
  static constexpr int NSUB = STAGE / SUB;
  static constexpr int KB = KEYS * NSUB;                     // keys of a block (one stage)
  static constexpr int ROWB = D * ES < 128 ? D * ES : 128;   // bytes of a row in one box of a tensor copy
  static constexpr int HALVES = D * ES / ROWB;
  static constexpr int SCALE = E4M3 ? NSUB * 128 : 0;        // bytes of scales of a stage
  static constexpr int MERGE = NW * GP * D * 4;              // accumulators that the warps of a CTA join
  static constexpr int WEIGHTS = F32 ? NW * KEYS * 16 : 0;   // fp32: weights of a piece for four heads
  // CTAs per SM.  More warps hide the chain from a block's arrival to its sums,
  // up to where registers run out: with 2 and with 3 CTAs 64 x 8192 bf16 takes
  // 334 and 325 us, 32 x 32768 e4m3 284 and 240 us, 64 x 8192 fp32 of 64
  // elements 173 and 178 us, 16 x 8192 fp32 of 128 164 and 179 us.  (In runs of
  // a second the GPU holds its 1000 W by its clock, and most of that goes.)
  // Above four heads three fit by spilling or with one stage, and the two ways
  // are not far apart in either direction (8 heads: 64 x 8192 bf16 323 and
  // 314 us, 64 x 1000 bf16 49 and 52; 16 heads: 64 x 8192 bf16 328 and 346,
  // 16 x 8192 fp32 509 and 707) but for fp32 rows of 64 elements, where three
  // would pay (64 x 8192 of 8 heads 311 and 231 us, of 16 heads 639 and 439)
  static constexpr int CTAS = GP > 4 ? 2 : F32 ? (D == 64 ? 3 : 2) : 3;
  // Stages of a warp's ring: as many as fit, two at least, so that a copy is on its way while a warp computes
  // (32 x 32768 e4m3 with four heads, where two just fit: 240 us, 264 us with one).  1 KB of each CTA's share is the system's.
  static constexpr int smem(int nst) {
    return (NW * nst * (STAGE + SCALE) + MERGE + WEIGHTS + static_cast<int>(sizeof(AttendShared<GP, 1>)) + NW * (nst - 1) * 12 + 127) & ~127;
  }
  static constexpr int stages() {
    int n = 8;
    while (n > 0 && CTAS * (smem(n) + 1024) > 228 * 1024) --n;
    return n;
  }
  static constexpr int NST = stages();
  static constexpr int SMEM = smem(NST);
  using Shared = AttendShared<GP, NST>;
  static_assert(NST >= 2, "a warp needs two stages");
  static_assert(NW * NST * (STAGE + SCALE) + MERGE + WEIGHTS + static_cast<int>(sizeof(Shared)) <= SMEM, "shared memory of a CTA");
};

struct AttendScratch {
  float* acc;        // [2 kAttendRanges][G][D]
  float* ml;         // [2 kAttendRanges][G][4]: running maximum, sum, whether any key was seen
  int32_t* ticket;   // [units], zero between launches
};

__device__ __forceinline__ void write4(__nv_bfloat16* p, const float4& o, float L, bool any) {
  *reinterpret_cast<uint2*>(p) = any ? make_uint2(pack_bf16(o.x / L, o.y / L), pack_bf16(o.z / L, o.w / L)) : make_uint2(0u, 0u);
}
__device__ __forceinline__ void write4(float* p, const float4& o, float L, bool any) {
  *reinterpret_cast<float4*>(p) = any ? make_float4(o.x / L, o.y / L, o.z / L, o.w / L) : make_float4(0.f, 0.f, 0.f, 0.f);
}

// One warp's part of an item for bf16 and 8-bit rows: 16 keys a piece, on
// m16n8k16 matrix instructions.  S = Q K^T has the queries as rows (up to four
// heads fill rows 0..3 and again 4..7), and its accumulator fragment, as
// weights, is the B fragment of O^T += V^T P^T.  Weights go in as two bf16
// terms (16 bits): with up to four heads the repeated rows carry the low
// terms, so they cost nothing, else a second instruction does.  8-bit keys are
// widened to f16, exactly (queries then are f16 too, scaled by a power of two),
// 8-bit values to bf16: a key's scale multiplies its score, a value's scale
// its weight, and only bf16 holds every weight times every scale to the same
// 16 bits.  (Values and weights in f16 take fewer instructions, but need one
// reference for all weights of a warp, 2^31 below which a token is lost:
// 32 x 32768 took 257 us so and 267 us in bf16 when a warp had one stage.)
template <int D, bool E4M3, int GP>
struct MmaPieces {
  using Geometry = Geo<__nv_bfloat16, D, E4M3, GP>;
  using G_ = Geometry;
  using Elements = __nv_bfloat16;
  static constexpr int kD = D, kGP = GP;
  static constexpr int R = GP == 16 ? 2 : 1;      // query rows per lane
  static constexpr int KS = D / 16;               // 16-wide steps over the head
  static constexpr int PK = G_::NSUB > 1 && GP < 16 ? 2 : 1;
  uint32_t qf[KS][4];
  float qmul[R];
  float acc[R][KS][4];
  float m[R], l[R];
  uint32_t kx[2], vx[4];      // this lane's offsets into a piece, for its loads of keys and of values

  // Offset of 16-byte chunk c of row r in a piece's keys (or values): boxes of
  // 128-byte (64-byte) rows, whose chunks the copy has placed at c ^ (r & 7)
  // (c ^ (r >> 1 & 3)).
  static __device__ __forceinline__ uint32_t place(int r, int c) {
    if (G_::ROWB == 128) return (c >> 3) * (16 * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
    return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
  }

  __device__ __forceinline__ void open(const AttendArgs& a, int b, int h) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, G = a.G;
    const float qscale = a.scale * kLog2e;
    // chunks 4 apart (keys) and 2 apart (values) differ in bits that the rows'
    // swizzle leaves in place: the rest of a load's address is a constant
#pragma unroll
    for (int i = 0; i < 2; ++i) kx[i] = place(lane & 7, (4 * i + (lane >> 3)) & (G_::ROWB / 16 - 1));
#pragma unroll
    for (int i = 0; i < 4; ++i)
      vx[i] = E4M3 ? place((lane & 7) + (((lane >> 3) & 1) << 3), (2 * i + (lane >> 4)) & (G_::ROWB / 16 - 1))
                   : place((lane & 7) + ((lane >> 4) << 3), (2 * i + ((lane >> 3) & 1)) & (G_::ROWB / 16 - 1));
    // queries as A fragments: row g (and g + 8); up to four heads fill rows 0..3 and again 4..7
    {
      const __nv_bfloat16* qb = static_cast<const __nv_bfloat16*>(a.q) + (static_cast<int64_t>(b) * a.Hq + static_cast<int64_t>(h) * G) * D;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = GP == 4 ? (g & 3) : g + 8 * r;
        const bool on = r < R && row < G;
        const uint32_t* src = reinterpret_cast<const uint32_t*>(qb + static_cast<int64_t>(on ? row : 0) * D);
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          // bf16: elements 2t, 2t + 1 and 2t + 8, 2t + 9 of a step; 8 bits: 4t .. 4t + 3
          qf[k][r] = on ? src[k * 8 + (E4M3 ? 2 * t : t)] : 0u;
          qf[k][r + 2] = on ? src[k * 8 + (E4M3 ? 2 * t + 1 : t + 4)] : 0u;
        }
        if (r < R) qmul[r] = qscale;
        if (E4M3 && r < R) {
          // to f16, exactly: the row is scaled by a power of two that brings its largest magnitude to [2^13, 2^14)
          float top = 0.f;
#pragma unroll
          for (int k = 0; k < KS; ++k) {
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
              const float2 v = bf2_to_f2(qf[k][r + i]);
              top = fmaxf(top, fmaxf(fabsf(v.x), fabsf(v.y)));
            }
          }
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;
          e = top == 0.f || e > 127 ? 13 : e < -100 ? -100 : e;
          const float up = __uint_as_float(static_cast<uint32_t>(127 + 13 - e) << 23);
          qmul[r] = qscale * __uint_as_float(static_cast<uint32_t>(127 - 13 + e) << 23);
#pragma unroll
          for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
              const float2 v = bf2_to_f2(qf[k][r + i]);
              qf[k][r + i] = pack_f16(v.x * up, v.y * up);
            }
        }
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      m[r] = -INFINITY; l[r] = 0.f;
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[r][k][i] = 0.f;
    }
  }

  // PK pieces at a time: twice the keys in the same chain of steps.  have: which of them were copied.
  __device__ __forceinline__ void pieces(const AttendArgs& a, uint8_t* kbase, const uint8_t* scales, int key0, int lo, int n,
                                         unsigned have, float*, bool& cleared) {
    const int lane = threadIdx.x & 31, t = lane & 3;
    const uint32_t ks = smem_u32(kbase), vs = ks + G_::SUB / 2;
    const bool part = key0 < lo || key0 + 16 * PK > n || have != (1u << PK) - 1;
    auto attended = [&](int i) { return key0 + i >= lo && key0 + i < n && ((have >> (i >> 4)) & 1); };
    if (part) {
      // values of tokens that are not attended: whatever they hold, weight zero must give zero
#pragma unroll
      for (int p = 0; p < PK; ++p) {
        const int row = lane >> 1;
        if (attended(16 * p + row)) continue;
        constexpr int CH = G_::ROWB / 16;
#pragma unroll
        for (int hf = 0; hf < G_::HALVES; ++hf)
#pragma unroll
          for (int c = 0; c < CH / 2; ++c)
            *reinterpret_cast<uint4*>(kbase + p * G_::SUB + G_::SUB / 2 + hf * 16 * G_::ROWB + row * G_::ROWB + ((lane & 1) * (CH / 2) + c) * 16) =
                make_uint4(0, 0, 0, 0);
      }
      cleared = true;
      __syncwarp();
    }
    // ---- scores: rows are queries, columns eight keys for each nb; two chains of sums each for a single piece ----
    constexpr int NB = 2 * PK, CHAINS = PK == 1 ? 2 : 1;
    float s[NB][CHAINS][4];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int c = 0; c < CHAINS; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[nb][c][i] = 0.f;
    if constexpr (!E4M3) {
#pragma unroll
      for (int k = 0; k < KS / 2; ++k) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          uint32_t f[4];
          ldsm_x4(ks + (nb >> 1) * G_::SUB + kx[k & 1] + (k >> 1) * 2048 + (nb & 1) * (8 * G_::ROWB), f);
          mma_bf16_16816(s[nb][0], qf[2 * k], f[0], f[1]);
          mma_bf16_16816(s[nb][CHAINS - 1], qf[2 * k + 1], f[2], f[3]);
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < KS / 4; ++k) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          uint32_t f[4];
          ldsm_x4(ks + (nb >> 1) * G_::SUB + kx[k & 1] + (k >> 1) * 2048 + (nb & 1) * (8 * G_::ROWB), f);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            mma_f16_16816(s[nb][i & (CHAINS - 1)], qf[4 * k + i], e4m3_to_f16(f[i]), e4m3_to_f16_high(f[i]));
        }
      }
    }
    float2 kf[NB], vf[NB];
    if constexpr (E4M3) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const float2* sp = reinterpret_cast<const float2*>(scales + (nb >> 1) * 128) + (nb & 1) * 4 + t;
        kf[nb] = sp[0]; vf[nb] = sp[8];
        if (part) {     // scales of tokens that are not attended may be anything
          if (!attended(nb * 8 + 2 * t)) vf[nb].x = 0.f;
          if (!attended(nb * 8 + 2 * t + 1)) vf[nb].y = 0.f;
        }
      }
    }
    uint32_t ph[R][NB], pl[R][NB];     // weights as two terms
    float x[R][2 * NB];
    float top[R];
    bool raise = false;
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int i = 0; i < 2 * NB; ++i) {
        float y = s[i >> 1][0][2 * r + (i & 1)];
        if (CHAINS == 2) y += s[i >> 1][CHAINS - 1][2 * r + (i & 1)];
        // (the two factors first: the sum times a large key's scale alone may pass fp32)
        if constexpr (E4M3) x[r][i] = y * (((i & 1) ? kf[i >> 1].y : kf[i >> 1].x) * qmul[r]);
        else x[r][i] = y * qmul[r];
      }
      if (a.softcap > 0.f) {
#pragma unroll
        for (int i = 0; i < 2 * NB; ++i) x[r][i] = a.softcap * kLog2e * tanhf(x[r][i] * (kLn2 / a.softcap));
      }
      if (part) {
#pragma unroll
        for (int i = 0; i < 2 * NB; ++i)
          if (!attended((i >> 1) * 8 + 2 * t + (i & 1))) x[r][i] = -INFINITY;
      }
      top[r] = x[r][0];
#pragma unroll
      for (int i = 1; i < 2 * NB; ++i) top[r] = fmaxf(top[r], x[r][i]);
      raise |= top[r] > m[r];
    }
    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float y = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
        y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 2));
        const float m1 = fmaxf(m[r], y + kRaise);
        const float c = m[r] == -INFINITY ? 0.f : ex2(m[r] - m1);
        m[r] = m1;
        l[r] *= c;
        // accumulator columns 2t, 2t + 1 belong to rows 2t, 2t + 1
        const float c0 = __shfl_sync(0xffffffffu, c, 8 * t), c1 = __shfl_sync(0xffffffffu, c, 8 * t + 4);
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          acc[r][k][0] *= c0; acc[r][k][1] *= c1;
          acc[r][k][2] *= c0; acc[r][k][3] *= c1;
        }
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float mu = m[r] == -INFINITY ? 0.f : m[r];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        float p0 = ex2(x[r][2 * nb] - mu), p1 = ex2(x[r][2 * nb + 1] - mu);
        l[r] += p0 + p1;
        if constexpr (E4M3) {
          p0 *= vf[nb].x;
          p1 *= vf[nb].y;
        }
        const uint32_t hi = pack_bf16(p0, p1);
        const float2 hf = bf2_to_f2(hi);
        const uint32_t lo = pack_bf16(p0 - hf.x, p1 - hf.y);
        if (GP == 4) {
          ph[r][nb] = lane < 16 ? hi : lo;     // rows 4..7 repeat the heads: they carry the low terms
        } else {
          ph[r][nb] = hi;
          pl[r][nb] = lo;
        }
      }
    }
    // ---- accumulators += V^T P^T: rows are head elements, columns queries ----
#pragma unroll
    for (int p = 0; p < PK; ++p) {
      if constexpr (!E4M3) {
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          uint32_t f[4];
          ldsm_x4_t(vs + p * G_::SUB + vx[k & 3] + (k >> 2) * 2048, f);
#pragma unroll
          for (int r = 0; r < R; ++r) {
            mma_bf16_16816(acc[r][k], f, ph[r][2 * p], ph[r][2 * p + 1]);
            if (GP != 4) mma_bf16_16816(acc[r][k], f, pl[r][2 * p], pl[r][2 * p + 1]);
          }
        }
      } else {
#pragma unroll
        for (int k = 0; k < KS; k += 2) {
          uint32_t f[4];
          ldsm_x4_t(vs + p * G_::SUB + vx[k >> 1], f);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            // bytes: two keys' elements 2g, 2g + 1 -> the keys' pairs of element 2g (row g) and of 2g + 1 (row g + 8)
            uint32_t v[4];
            e4m3_to_bf16(f[2 * c], v[0], v[1]);
            e4m3_to_bf16(f[2 * c + 1], v[2], v[3]);
#pragma unroll
            for (int r = 0; r < R; ++r) {
              mma_bf16_16816(acc[r][k + c], v, ph[r][2 * p], ph[r][2 * p + 1]);
              if (GP != 4) mma_bf16_16816(acc[r][k + c], v, pl[r][2 * p], pl[r][2 * p + 1]);
            }
          }
        }
      }
    }
  }

  // Accumulators, running maxima and sums of this warp to shared memory.
  __device__ __forceinline__ void close(float* macc, float (*ml)[2], int warp, bool any) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      const int row = g + 8 * r;
      if (t == 0 && row < GP) {
        ml[row][0] = m[r]; ml[row][1] = l[r];
      }
      if (any) {
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          // element of head dimension that accumulator rows g and g + 8 hold
          const int e0 = k * 16 + (E4M3 ? 2 * g : g), e1 = E4M3 ? e0 + 1 : e0 + 8;
          if constexpr (GP == 4) {
            // columns 0..3 hold the high terms' sums, 4..7 the low terms': the lanes of a pair add up one row each
            const bool up = t & 2;
            const float s0 = __shfl_xor_sync(0xffffffffu, up ? acc[r][k][0] : acc[r][k][2], 2);
            const float s1 = __shfl_xor_sync(0xffffffffu, up ? acc[r][k][1] : acc[r][k][3], 2);
            float* o = macc + (warp * GP + 2 * (t & 1)) * D + (up ? e1 : e0);
            o[0] = (up ? acc[r][k][2] : acc[r][k][0]) + s0;
            o[D] = (up ? acc[r][k][3] : acc[r][k][1]) + s1;
          } else {
            float* o = macc + (warp * GP + 2 * t + 8 * r) * D;
            o[e0] = acc[r][k][0]; o[D + e0] = acc[r][k][1];
            o[e1] = acc[r][k][2]; o[D + e1] = acc[r][k][3];
          }
        }
      }
    }
  }
};

// The same for fp32 rows, on fp32 FMAs.  Eight lanes share a key (four keys at
// a time), each with D / 8 elements; four heads' dot products are reduced
// together, so that each pair of lanes ends with one head's score.  The
// weights of a piece go through shared memory, and each lane accumulates D / 32
// elements of four heads.  More than four heads: the next four after these,
// over the same keys, their queries read again.
template <int D, int GP>
struct FmaPieces {
  using Geometry = Geo<float, D, false, GP>;
  using G_ = Geometry;
  using Elements = float;
  static constexpr int kD = D, kGP = GP;
  static constexpr int NC = GP / 4;               // groups of four heads
  static constexpr int QV = D / 32, E = D / 32;   // float4s of a key's eighth; elements of a lane's accumulator
  static constexpr int KEYS = G_::KEYS, PK = 1;
  const float* qbase;
  int heads;
  float4 q[4][QV];                                // of the group in hand
  float acc[NC][4][E];
  float m[NC], l[NC];                             // of this lane's head of each group

  __device__ __forceinline__ void load_q(int c) {
    const int part = threadIdx.x & 7;
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
      for (int v = 0; v < QV; ++v)
        q[x][v] = 4 * c + x < heads ? *reinterpret_cast<const float4*>(qbase + static_cast<int64_t>(4 * c + x) * D + (part + 8 * v) * 4)
                                    : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __device__ __forceinline__ void open(const AttendArgs& a, int b, int h) {
    qbase = static_cast<const float*>(a.q) + (static_cast<int64_t>(b) * a.Hq + static_cast<int64_t>(h) * a.G) * D;
    heads = a.G;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      m[c] = -INFINITY; l[c] = 0.f;
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int e = 0; e < E; ++e) acc[c][x][e] = 0.f;
    }
    if (NC == 1) load_q(0);
  }

  __device__ __forceinline__ void pieces(const AttendArgs& a, uint8_t* kbase, const uint8_t*, int key0, int lo, int n, unsigned, float* wbuf, bool&) {
    const int lane = threadIdx.x & 31, part = lane & 7, kg = lane >> 3;
    const float4* keys = reinterpret_cast<const float4*>(kbase);
    const float* values = reinterpret_cast<const float*>(kbase + G_::SUB / 2);
    const int k_lo = max(lo - key0, 0), k_hi = min(n - key0, KEYS);    // attended keys of the piece
    const int head = ((part >> 2) & 1) * 2 + ((part >> 1) & 1);        // this lane's head of four
    const float qscale = a.scale * kLog2e;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      if (4 * c >= heads) break;
      if (NC > 1) load_q(c);
      float x[KEYS / 4];
      float top = -INFINITY;
#pragma unroll
      for (int p = 0; p < KEYS / 4; ++p) {
        const int key = 4 * p + kg;
        float2 s[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) s[y] = make_float2(0.f, 0.f);
#pragma unroll
        for (int v = 0; v < QV; ++v) {
          const float4 k = keys[key * (D / 4) + part + 8 * v];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            s[y] = ffma2(make_float2(k.x, k.y), make_float2(q[y][v].x, q[y][v].y), s[y]);
            s[y] = ffma2(make_float2(k.z, k.w), make_float2(q[y][v].z, q[y][v].w), s[y]);
          }
        }
        // four sums over eight lanes: each exchange halves the heads a lane still adds up
        float d[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) d[y] = s[y].x + s[y].y;
        const bool up4 = part & 4, up2 = part & 2;
        float e0 = (up4 ? d[2] : d[0]) + __shfl_xor_sync(0xffffffffu, up4 ? d[0] : d[2], 4);
        float e1 = (up4 ? d[3] : d[1]) + __shfl_xor_sync(0xffffffffu, up4 ? d[1] : d[3], 4);
        float f = (up2 ? e1 : e0) + __shfl_xor_sync(0xffffffffu, up2 ? e0 : e1, 2);
        f += __shfl_xor_sync(0xffffffffu, f, 1);
        f *= qscale;
        if (a.softcap > 0.f) f = a.softcap * kLog2e * tanhf(f * (kLn2 / a.softcap));
        x[p] = key >= k_lo && key < k_hi ? f : -INFINITY;
        top = fmaxf(top, x[p]);
      }
      if (__any_sync(0xffffffffu, top > m[c])) {
        float y = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
        y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 16));
        const float m1 = fmaxf(m[c], y + kRaise);
        const float f = m[c] == -INFINITY ? 0.f : ex2(m[c] - m1);
        m[c] = m1;
        l[c] *= f;
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          const float fz = __shfl_sync(0xffffffffu, f, (z >> 1) * 4 + (z & 1) * 2);
#pragma unroll
          for (int e = 0; e < E; ++e) acc[c][z][e] *= fz;
        }
      }
      const float mu = m[c] == -INFINITY ? 0.f : m[c];
      __syncwarp();                       // the weights before these have been read
#pragma unroll
      for (int p = 0; p < KEYS / 4; ++p) {
        const float w = ex2(x[p] - mu);
        l[c] += w;
        if (!(part & 1)) wbuf[(4 * p + kg) * 4 + head] = w;
      }
      __syncwarp();
      auto add = [&](int key) {
        const float4 w = *reinterpret_cast<const float4*>(wbuf + key * 4);
        const float wz[4] = {w.x, w.y, w.z, w.w};
        float v[E];
        if constexpr (E == 4) {
          const float4 r = *reinterpret_cast<const float4*>(values + key * D + lane * 4);
          v[0] = r.x; v[1] = r.y; v[2] = r.z; v[3] = r.w;
        } else {
          const float2 r = *reinterpret_cast<const float2*>(values + key * D + lane * 2);
          v[0] = r.x; v[1] = r.y;
        }
#pragma unroll
        for (int z = 0; z < 4; ++z)
#pragma unroll
          for (int e = 0; e < E; e += 2) {
            const float2 r = ffma2(make_float2(wz[z], wz[z]), make_float2(v[e], v[e + 1]), make_float2(acc[c][z][e], acc[c][z][e + 1]));
            acc[c][z][e] = r.x; acc[c][z][e + 1] = r.y;
          }
      };
      if (k_lo == 0 && k_hi == KEYS) {
#pragma unroll
        for (int key = 0; key < KEYS; ++key) add(key);
      } else {
        // values of tokens that are not attended are not touched: they may be anything
        for (int key = k_lo; key < k_hi; ++key) add(key);
      }
    }
  }

  __device__ __forceinline__ void close(float* macc, float (*ml)[2], int warp, bool any) {
    const int lane = threadIdx.x & 31, part = lane & 7;
    const int head = ((part >> 2) & 1) * 2 + ((part >> 1) & 1);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      float s = l[c];
      s += __shfl_xor_sync(0xffffffffu, s, 8);
      s += __shfl_xor_sync(0xffffffffu, s, 16);
      if (lane < 8 && !(part & 1)) {
        ml[4 * c + head][0] = m[c]; ml[4 * c + head][1] = s;
      }
      if (any) {
#pragma unroll
        for (int z = 0; z < 4; ++z)
#pragma unroll
          for (int e = 0; e < E; ++e) macc[(warp * GP + 4 * c + z) * D + lane * E + e] = acc[c][z][e];
      }
    }
  }
};

// The kernel after the split.  SOLO: warps take whole sequences and heads, and no two warps meet.
template <typename C, bool SOLO>
__device__ __forceinline__ void attend_items(const CUtensorMap& map, const AttendArgs& a, const AttendScratch& sc,
                                             typename C::Geometry::Shared& sh, int nb0, Span span0, uint8_t* smem) {
  using G_ = typename C::Geometry;
  using T = typename C::Elements;
  constexpr int D = C::kD, GP = C::kGP, KB = G_::KB, NSUB = G_::NSUB, NST = G_::NST;
  constexpr bool E4M3 = G_::SCALE > 0;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Split* const spp = &sh.split[warp];
  uint8_t* ring = smem + warp * NST * G_::STAGE;
  uint8_t* sring = smem + NW * NST * G_::STAGE + warp * NST * G_::SCALE;
  float* macc = reinterpret_cast<float*>(smem + NW * NST * (G_::STAGE + G_::SCALE));   // [NW][GP][D]
  float* wbuf = macc + NW * GP * D + warp * (G_::WEIGHTS / (4 * NW));
  uint64_t* bars = sh.bars[warp];
  int32_t* live = sh.live[warp];
  auto& items = sh.items;
  const int Hkv = a.pg.Hkv, G = a.G, n_cta = gridDim.x;
  // sequences without a token
  auto zeros = [&]() {
    for (int b = blockIdx.x; b < a.batch; b += n_cta) {
      if (span_of(*spp, a.lens[b]).n > 0) continue;
      for (int i = threadIdx.x; i < a.Hq * D; i += NW * 32)
        static_cast<T*>(a.out)[static_cast<int64_t>(b) * a.Hq * D + i] = Elem<T>::from_f32(0.f);
      if (a.lse)
        for (int i = threadIdx.x; i < a.Hq; i += NW * 32) a.lse[static_cast<int64_t>(b) * a.Hq + i] = -INFINITY;
    }
  };

  // ---- items: the one in hand, and the producer's, NST blocks ahead ----
  bool some;
  if constexpr (SOLO) {
    some = solo_item<KB>(spp, &items[warp][0], true);
  } else if (a.fixed > 0) {
    some = n_cta >= Hkv && fixed_item<KB>(*spp, &items[warp][0], blockIdx.x / Hkv, blockIdx.x % Hkv);
  } else if (spp->aligned && a.batch <= 32 && n_cta >= Hkv) {
    // what next_item does, from what the lanes already have
    const int grp = blockIdx.x / Hkv;
    const int own = parts_of(nb0, static_cast<int>(spp->share));
    int sum = own;
    if (a.batch > 1) {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += u;
      }
    }
    const unsigned past = __ballot_sync(0xffffffffu, sum > grp);
    some = past != 0 && grp < spp->groups;
    if (some && lane == __ffs(past) - 1) {
      const int part = grp - (sum - own), share = static_cast<int>(spp->share), j0 = span0.lo / KB;
      const int j = j0 + part * share, jend = min(j + share, j0 + nb0);
      items[warp][0] = Item{lane, static_cast<int>(blockIdx.x) - grp * Hkv, span0.lo, span0.n, j, jend, grp - part, own, 0, jend - j, 0};
    }
    __syncwarp();
  } else {
    some = next_item<KB>(spp, &items[warp][0], nb0, true);
  }
  if (!some) {            // the whole CTA, or (SOLO) this warp alone
    zeros();
    return;
  }
  if (lane == 0) items[warp][1] = items[warp][0];
  __syncwarp();
  const Item& w = items[warp][0];
  Item& p = items[warp][1];
  // first own block of an item: blocks go to the warps in turn
  constexpr int kStride = SOLO ? 1 : NW;
  auto first_own = [&](int j) { return SOLO ? j : j + ((warp - j) & (NW - 1)); };
  auto next = [&](Item* it) {
    if constexpr (SOLO) return solo_item<KB>(spp, it, false);
    else return next_item<KB>(spp, it, nb0, false);
  };
  bool dead = false;     // a wait ran out: nothing more is copied or computed
  bool p_more = true;
  int pj = first_own(p.j), p_end = p.jend, seq_p = 0, page_next = -1;
  bool page_want = false;
  auto settle = [&]() {  // moves p to an item that has a block for this warp
    while (p_more && pj >= p_end) {
      p_more = next(&p);
      pj = first_own(p.j);
      p_end = p.jend;
    }
  };
  auto load_page = [&]() {   // lane i: the page of piece i of the next block
    const int key = pj * KB + lane * G_::KEYS;
    page_want = p_more && lane < NSUB && key < p.n && key + G_::KEYS > p.lo;
    if (page_want) page_next = a.table[p.b * a.table_stride + (key >> a.pg.page_shift)];
  };
  auto issue = [&]() {
    if (!p_more || dead) return;
    const int st = seq_p % NST;
    const bool ok = page_want && page_next >= 0 && page_next < a.pg.n_pages;
    if (page_want && !ok) set_error(a.pg.err, DEVERR_BAD_INDEX);
    const unsigned m = __ballot_sync(0xffffffffu, ok);
    if (lane == 0) {
      live[st] = static_cast<int32_t>(m);
      mbar_arrive_expect_tx(&bars[st], __popc(m) * (G_::SUB + (E4M3 ? 128 : 0)));
    }
    __syncwarp();
    if (ok) {
      const int row = (pj * KB + lane * G_::KEYS) & ((1 << a.pg.page_shift) - 1);
      const int w5 = page_next * Hkv + p.h;
      if constexpr (G_::F32) {
        const float* from = reinterpret_cast<const float*>(a.pg.pages) + (((static_cast<int64_t>(w5) * 2) << a.pg.page_shift) + row) * D;
        bulk_g2s(ring + st * G_::STAGE + lane * G_::SUB, from, G_::SUB / 2, &bars[st]);
        bulk_g2s(ring + st * G_::STAGE + lane * G_::SUB + G_::SUB / 2, from + (static_cast<int64_t>(D) << a.pg.page_shift), G_::SUB / 2, &bars[st]);
      } else {
        tma_load_5d(ring + st * G_::STAGE + lane * G_::SUB, &map, 0, row, 0, 0, w5, &bars[st]);
      }
      if (E4M3) {
        const float* s0 = a.pg.scales + ((static_cast<int64_t>(w5) * 2) << a.pg.page_shift) + row;
        bulk_g2s(sring + st * G_::SCALE + lane * 128, s0, 64, &bars[st]);
        bulk_g2s(sring + st * G_::SCALE + lane * 128 + 64, s0 + (1 << a.pg.page_shift), 64, &bars[st]);
      }
    }
    ++seq_p;
    pj += kStride;
    settle();
    load_page();
  };
  settle();
  load_page();
  for (int s = 0; s < NST; ++s) issue();
  zeros();               // while the first copies are on their way

  // ---- items ----
  int n_open = 0;          // items that are parts of their sequence
  int seq_c = 0;
  for (bool more = true; more;) {
    C c;
    c.open(a, w.b, w.h);
    bool any = false;
    const int lo = w.lo, n = w.n, jend = w.jend;

    for (int j = first_own(w.j); j < jend; j += kStride) {
      const int st = seq_c % NST;
      if (!dead && !mbar_wait(&bars[st], (seq_c / NST) & 1)) {
        if (lane == 0) set_error(a.pg.err, DEVERR_TIMEOUT);
        dead = true;
      }
      dead = __any_sync(0xffffffffu, dead);
      bool cleared = false;
      const unsigned have = dead ? 0u : static_cast<unsigned>(live[st]);
#pragma unroll 1
      for (int sub = 0; sub < NSUB; sub += C::PK) {
        const unsigned in_hand = (have >> sub) & ((1u << C::PK) - 1);
        if (in_hand == 0) continue;
        any = true;
        c.pieces(a, ring + st * G_::STAGE + sub * G_::SUB, sring + st * G_::SCALE + sub * 128, j * KB + sub * G_::KEYS, lo, n, in_hand, wbuf, cleared);
      }
      if (cleared) fence_proxy_async_smem();   // those stores come before the next copy into the stage
      __syncwarp();
      if (!dead) {
        ++seq_c;
        issue();
      }
    }

    // ---- join the warps ----
    c.close(macc, sh.ml[warp], warp, any);
    if (lane == 0) sh.any[warp] = any;
    if constexpr (SOLO) __syncwarp();
    else __syncthreads();
    const bool complete = SOLO || w.parts == 1;
    const int64_t slot = complete ? 0 : slot_of(w, static_cast<int>(blockIdx.x) / Hkv - w.first, Hkv);
    const int64_t orow = static_cast<int64_t>(w.b) * a.Hq + static_cast<int64_t>(w.h) * G;
    for (int i = SOLO ? lane : threadIdx.x; i < G * (D / 4); i += SOLO ? 32 : NW * 32) {
      const int q = i / (D / 4), e = (i % (D / 4)) * 4;
      float M = -INFINITY, seen = 0.f;
#pragma unroll
      for (int x = 0; x < NW; ++x) {
        if (SOLO && x != warp) continue;
        M = fmaxf(M, sh.ml[x][q][0]);
        seen += sh.any[x];
      }
      const float mu = M == -INFINITY ? 0.f : M;
      float L = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int x = 0; x < NW; ++x) {
        if (SOLO && x != warp) continue;
        if (!sh.any[x]) continue;
        const float c = ex2(sh.ml[x][q][0] - mu);
        const float4 v = *reinterpret_cast<const float4*>(&macc[(x * GP + q) * D + e]);
        L = fmaf(c, sh.ml[x][q][1], L);
        o.x = fmaf(c, v.x, o.x); o.y = fmaf(c, v.y, o.y); o.z = fmaf(c, v.z, o.z); o.w = fmaf(c, v.w, o.w);
      }
      if (complete) {
        write4(static_cast<T*>(a.out) + (orow + q) * D + e, o, L, seen > 0.f);
        if (a.lse && e == 0) a.lse[orow + q] = seen > 0.f ? (mu + log2f(L)) * kLn2 : -INFINITY;
      } else {
        __stcg(reinterpret_cast<float4*>(sc.acc + (slot * G + q) * D + e), o);
        if (e == 0) __stcg(reinterpret_cast<float4*>(sc.ml + (slot * G + q) * 4), make_float4(M, L, seen, 0.f));
      }
    }
    if (!complete) {
      if (threadIdx.x == 0) sh.open[n_open] = Part{w.b, w.h, w.first, w.parts, w.second};
      ++n_open;
    }
    if constexpr (SOLO) __syncwarp();      // the join's buffers are free again
    else __syncthreads();
    more = next(&items[warp][0]);
  }
  // ---- sequences that lie in other ranges too (the range's first and last): join them if all parts are there ----
  // Left for the end, since each step waits for the one before at the far side of L2, 2 us and more while the
  // GPU reads at full speed.
  if (!SOLO && n_open > 0) {
    __threadfence();
    __syncthreads();
    if (threadIdx.x < n_open) {
      const Part& x = sh.open[threadIdx.x];
      sh.last[threadIdx.x] = atomicAdd(&sc.ticket[static_cast<int64_t>(x.b) * Hkv + x.h], 1) == x.parts - 1;
    }
    __syncthreads();
    for (int i_open = 0; i_open < n_open; ++i_open) {
      if (!sh.last[i_open]) continue;
      const Part& x = sh.open[i_open];
      const int64_t orow = static_cast<int64_t>(x.b) * a.Hq + static_cast<int64_t>(x.h) * G;
      __threadfence();
      if (threadIdx.x == 0) sc.ticket[static_cast<int64_t>(x.b) * Hkv + x.h] = 0;
      for (int i = threadIdx.x; i < G * (D / 4); i += NW * 32) {
        const int q = i / (D / 4), e = (i % (D / 4)) * 4;
        float M = -INFINITY, L = 0.f, seen = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        constexpr int PB = 8;          // partials on their way at a time
        for (int c0 = 0; c0 < x.parts; c0 += PB) {
          float4 ml[PB], v[PB];
#pragma unroll
          for (int c = 0; c < PB; ++c) {
            ml[c] = make_float4(-INFINITY, 0.f, 0.f, 0.f);
            if (c0 + c < x.parts) {
              const int64_t sl = slot_of(x, c0 + c, Hkv) * G + q;
              ml[c] = __ldcg(reinterpret_cast<const float4*>(sc.ml + sl * 4));
              v[c] = __ldcg(reinterpret_cast<const float4*>(sc.acc + sl * D + e));
            }
          }
          float M1 = M;
#pragma unroll
          for (int c = 0; c < PB; ++c) M1 = fmaxf(M1, ml[c].x);
          const float mu = M1 == -INFINITY ? 0.f : M1, ca = ex2(M - mu);
          M = M1;
          L *= ca; o.x *= ca; o.y *= ca; o.z *= ca; o.w *= ca;
#pragma unroll
          for (int c = 0; c < PB; ++c) {
            if (ml[c].z == 0.f) continue;      // no key in that part
            const float cb = ex2(ml[c].x - mu);
            seen += ml[c].z;
            L = fmaf(cb, ml[c].y, L);
            o.x = fmaf(cb, v[c].x, o.x); o.y = fmaf(cb, v[c].y, o.y);
            o.z = fmaf(cb, v[c].z, o.z); o.w = fmaf(cb, v[c].w, o.w);
          }
        }
        write4(static_cast<T*>(a.out) + (orow + q) * D + e, o, L, seen > 0.f);
        if (a.lse && e == 0) a.lse[orow + q] = seen > 0.f ? ((M == -INFINITY ? 0.f : M) + log2f(L)) * kLn2 : -INFINITY;
      }
    }
  }
  // copies that a dead warp leaves in flight: wait for them (bounded) before its shared memory goes
  if (dead)
    for (; seq_c < seq_p; ++seq_c) mbar_wait(&bars[seq_c % NST], (seq_c / NST) & 1);
}

template <typename C>
__global__ void __launch_bounds__(NW * 32, C::Geometry::CTAS)
attend_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ AttendArgs a, const AttendScratch sc) {
  using G_ = typename C::Geometry;
  constexpr int D = C::kD, GP = C::kGP, KB = G_::KB, NST = G_::NST;
  extern __shared__ __align__(1024) uint8_t smem_raw[];     // the copies' swizzle needs 1024
  uint8_t* smem = smem_raw;
  // Four heads of 128 fp32 elements: the compiler keeps more loads on their way where it does not see that they are
  // of shared memory (16 x 8192: 161 us, 176 us where it does; eight heads the other way, 286 and 266 us).
  if (G_::F32 && D == 128 && GP == 4) asm volatile("" : "+l"(smem));
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto& sh = *reinterpret_cast<typename G_::Shared*>(smem + NW * NST * (G_::STAGE + G_::SCALE) + NW * GP * D * 4 + G_::WEIGHTS);
  if (lane == 0) {
    if (!G_::F32) asm volatile("prefetch.tensormap [%0];" :: "l"(reinterpret_cast<uint64_t>(&map)) : "memory");
    for (int s = 0; s < NST; ++s) mbar_init(&sh.bars[warp][s], 1);
    mbar_fence_init();
  }
  __syncwarp();

  wait_for_prior_kernel();
  // ---- the split ----
  const int Hkv = a.pg.Hkv, n_cta = gridDim.x;
  Split sp;
  sp.lens = a.lens;
  sp.batch = a.batch; sp.Hkv = Hkv; sp.window = a.window; sp.fixed = a.fixed;
  sp.cap = static_cast<int>(min(static_cast<int64_t>(a.width) << a.pg.page_shift, kMostTokens));
  sp.groups = max(1, n_cta / Hkv);
  sp.total = 0; sp.share = kMinShare; sp.aligned = 0; sp.solo = 0;
  int nb0 = 0;             // blocks of sequence `lane`
  Span span0{0, 0};        // and its tokens
  if (a.fixed > 0) {
    if (warp == 0 && lane == 0 && blockIdx.x < a.batch) {
      const int given = a.lens[blockIdx.x];
      if (given != span_of(sp, given).n) set_error(a.pg.err, DEVERR_BAD_INDEX);
    }
  } else {
    bool bad_len = false;
    LaneWarp<BlockSum<KB>> w{0};
    split_work<KB>(w, sp, G_::F32, [&](int b, int nb, const Span& s, int given) {
      if (b < 32) {
        w.nb0 = nb0 = nb;
        span0 = s;
      }
      bad_len |= given != s.n;
    });
    if (bad_len && blockIdx.x == 0 && warp == 0) set_error(a.pg.err, DEVERR_BAD_INDEX);
  }
  if (lane == 0) sh.split[warp] = sp;
  __syncwarp();
  if (sp.solo) attend_items<C, true>(map, a, sc, sh, nb0, span0, smem);
  else attend_items<C, false>(map, a, sc, sh, nb0, span0, smem);
}

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  void* fn = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
      q != cudaDriverEntryPointSuccess)
    return nullptr;
  return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
}

// Calls f with the kernel of (dtype, d, 8 bits, heads per KV head) and its shared memory.
template <typename F>
int with_kernel(int dtype, int d, bool e8, int G, F f) {
#define KVPOP_ATTEND_F32(DD, PP) \
  if (d == DD && G <= PP) return f(attend_kernel<FmaPieces<DD, PP>>, FmaPieces<DD, PP>::Geometry::SMEM, FmaPieces<DD, PP>::Geometry::CTAS, \
                                           FmaPieces<DD, PP>::Geometry::KB);
  if (dtype == KVPOP_DTYPE_F32) {
    if (e8) return -2;
    KVPOP_ATTEND_F32(128, 4) KVPOP_ATTEND_F32(128, 8) KVPOP_ATTEND_F32(128, 16)
    KVPOP_ATTEND_F32(64, 4) KVPOP_ATTEND_F32(64, 8) KVPOP_ATTEND_F32(64, 16)
    return -2;
  }
#undef KVPOP_ATTEND_F32
#define KVPOP_ATTEND(DD, EE, PP) \
  if (d == DD && e8 == EE && G <= PP) return f(attend_kernel<MmaPieces<DD, EE, PP>>, MmaPieces<DD, EE, PP>::Geometry::SMEM, MmaPieces<DD, EE, PP>::Geometry::CTAS, \
                                                      MmaPieces<DD, EE, PP>::Geometry::KB);
  KVPOP_ATTEND(128, false, 4) KVPOP_ATTEND(128, false, 8) KVPOP_ATTEND(128, false, 16)
  KVPOP_ATTEND(128, true, 4) KVPOP_ATTEND(128, true, 8) KVPOP_ATTEND(128, true, 16)
  KVPOP_ATTEND(64, false, 4) KVPOP_ATTEND(64, false, 8) KVPOP_ATTEND(64, false, 16)
  KVPOP_ATTEND(64, true, 4) KVPOP_ATTEND(64, true, 8) KVPOP_ATTEND(64, true, 16)
#undef KVPOP_ATTEND
  return -2;
}

}  // namespace

size_t attend_scratch_bytes(int G, int d, int units) {
  return static_cast<size_t>(kAttendRanges) * 2 * G * (d + 4) * 4 + ((static_cast<size_t>(units) * 4 + 255) & ~static_cast<size_t>(255));
}

int make_attend_map(CUtensorMap* map, void* pages, int dtype, int d, bool e8, int page_size, int64_t page_heads) {
  if (dtype != KVPOP_DTYPE_BF16) return 0;     // fp32 rows are not read through a map
  const auto encode = tensor_map_encoder();
  if (encode == nullptr) return -1;
  const int es = e8 ? 1 : 2, row = d * es, part = row < 128 ? row : 128;
  const cuuint64_t dim[5] = {static_cast<cuuint64_t>(part / es), static_cast<cuuint64_t>(page_size),
                             static_cast<cuuint64_t>(row / part), 2, static_cast<cuuint64_t>(page_heads)};
  const cuuint64_t stride[4] = {static_cast<cuuint64_t>(row), static_cast<cuuint64_t>(part),
                                static_cast<cuuint64_t>(row) * page_size, static_cast<cuuint64_t>(row) * page_size * 2};
  const cuuint32_t box[5] = {static_cast<cuuint32_t>(part / es), 16, static_cast<cuuint32_t>(row / part), 2, 1};
  const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
  const CUresult r = encode(map, e8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, pages, dim,
                            stride, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            part == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? 0 : -1;
}

int prepare_attend(int dtype, int d, bool e8, int G) {
  return with_kernel(dtype, d, e8, G, [](auto kernel, int smem, int, int) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) == cudaSuccess ? 0 : -1;
  });
}

int launch_attend(const CUtensorMap& map, const AttendArgs& a, void* scratch, int dtype, int d, int num_sms,
                  cudaStream_t st) {
  const bool e8 = a.pg.scales != nullptr;
  AttendScratch sc;
  sc.acc = static_cast<float*>(scratch);
  sc.ml = sc.acc + static_cast<size_t>(kAttendRanges) * 2 * a.G * d;
  sc.ticket = reinterpret_cast<int32_t*>(sc.ml + static_cast<size_t>(kAttendRanges) * 2 * a.G * 4);
  return with_kernel(dtype, d, e8, a.G, [&](auto kernel, int smem, int ctas, int KB) {
    const Launch x = launch_of(ctas * num_sms < kAttendRanges ? ctas * num_sms : kAttendRanges,
                               static_cast<int64_t>(a.width) << a.pg.page_shift, KB, a.window, a.pg.Hkv, a.batch);
    AttendArgs b = a;
    b.fixed = x.fixed;
    return launch_dependent(kernel, dim3(x.grid), NW * 32, smem, st, map, b, sc);
  });
}

}  // namespace kvpop
