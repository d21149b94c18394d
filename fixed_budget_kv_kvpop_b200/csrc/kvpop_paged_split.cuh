// How the paged attention's work is split (kvpop_paged_attn.cu): arithmetic on
// lengths and blocks alone, for the kernel and, as plain C++, for the tests
// that check it.  What needs the 32 lanes of a warp goes through W, a warp (in
// the kernel) or a loop over lanes (in the tests):
//   W::Lanes               a value per lane
//   lanes(f)               f(lane) of each lane
//   each(v, f)             f of each lane's value
//   sum(v), top(v)         over the lanes
//   few(v)                 sum(v) where 32 bits hold it
//   some(v)                how many lanes are above 0
//   find(v, before, target, many, hit)   whether before + the sum of v passes target, and at which lane first; many: v
//                          may be above 0 past the first lane
//   cached(f)              lanes(f) of the first 32 sequences' blocks, which the caller may have
#pragma once
#include <cstdint>
#include <type_traits>

#ifdef __CUDACC__
#define KVPOP_HD __host__ __device__ __forceinline__
#else
#define KVPOP_HD inline
#endif

namespace kvpop {

constexpr int kMinShare = 8;             // blocks of a part at least (1 x 1024 tokens: 4 10.4 us, 8 9.3 us, 16 10.5 us, 32 12.9 us)
constexpr int64_t kMostTokens = INT64_C(1) << 30;   // of a sequence
// If there are more sequences than groups and none has more tokens than this, they go to single warps.  Few long ones
// would leave warps idle (8 groups of 4 heads, bf16: 64 x 200 20 us against 26, 64 x 300 26 against 28, 256 x 300 68
// against 67; e4m3 64 x 400 33 against 31), the sooner the more a warp has to compute (fp32 on the FMA units, 8 groups
// of 16 heads: 80 x 60 47 us against 53, 80 x 250 144 against 116).
constexpr int solo_tokens(bool f32) { return f32 ? 64 : 256; }
// Largest part that is taken for one part of one sequence per group, when equal
// ranges would have `even` blocks: ranges cost a second item and its join.
KVPOP_HD int64_t most_of(int64_t even) { return even + even / 5 + 16; }

template <typename T> KVPOP_HD T lesser(T a, T b) { return a < b ? a : b; }
template <typename T> KVPOP_HD T greater(T a, T b) { return a > b ? a : b; }

// a / b for a >= 0, b > 0: in 32 bits where they allow, a fraction of the 64-bit division's time.
KVPOP_HD int64_t quotient(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}
KVPOP_HD int parts_of(int blocks, int share) {
  return static_cast<int>(static_cast<uint32_t>(blocks + share - 1) / static_cast<uint32_t>(share));
}

// The sequences and how their work is split.  Kept in shared memory, one copy
// per warp: the function that finds items reads it from there, where an
// argument struct passed on by address costs a trip to global memory.
struct Split {
  const int32_t* lens;
  int64_t total;     // blocks of all sequences: at most 2^37
  int64_t share;     // blocks of a range
  int batch, Hkv, window;
  int fixed;         // > 0: parts of kMinShare blocks, this many groups of CTAs for each sequence
  int cap;           // tokens that a row of the page table can name
  int groups;        // groups of CTAs
  int aligned;       // one part of one sequence per group
  int solo;          // whole sequences of one head, each by a warp of its own
};

// Attended tokens [lo, n) of a sequence whose length is given as n; lengths outside the table are cut.
struct Span {
  int lo, n;
};
KVPOP_HD Span span_of(const Split& sp, int n) {
  n = n < 0 ? 0 : lesser(n, sp.cap);
  return Span{sp.window > 0 && n > sp.window ? n - sp.window : 0, n};
}
// A sum of blocks over 32 sequences.
template <int KB>
using BlockSum = std::conditional_t<32 * (kMostTokens / KB) <= UINT32_MAX, uint32_t, uint64_t>;
// Blocks of sequence b.
template <int KB>
KVPOP_HD int blocks_of(const Split& sp, int b) {
  const Span s = span_of(sp, sp.lens[b]);
  return (s.n + KB - 1) / KB - s.lo / KB;
}

// An item: blocks of one sequence and head.  Each warp keeps two in shared
// memory, the one it computes on and the one it copies for, so that they take
// no registers in the loops.
struct Item {
  int b, h;
  int lo, n;         // the sequence's attended tokens
  int j, jend;       // blocks [j, jend) of the item; block x holds tokens x KB .. x KB + KB - 1
  int first, parts;  // groups that hold a part of the sequence
  int second;        // 1: in the first of them it is not the range's first sequence
  int64_t left;      // blocks of the range from this item on
  int64_t pos;       // of the item's first block among all blocks (ranges)
};

// CTAs of a launch and how many groups of them each sequence has where parts
// are fixed: as many as fit the GPU (`most`), and no more than the longest
// sequences that the tables can name (`tokens`) would take.
struct Launch {
  int grid, fixed;
};
KVPOP_HD Launch launch_of(int64_t most, int64_t tokens, int KB, int window, int Hkv, int batch) {
  int64_t blocks = (tokens + KB - 1) / KB;
  if (window > 0 && window / KB + 2 < blocks) blocks = window / KB + 2;     // a window may begin and end inside a block
  const int64_t per = (blocks + kMinShare - 1) / kMinShare;
  const int64_t need = static_cast<int64_t>(Hkv) * batch * per;
  return Launch{static_cast<int>(need < 1 ? 1 : need < most ? need : most), need >= 1 && need <= most ? static_cast<int>(per) : 0};
}

// The split of sp's sequences where parts are not fixed.  see(b, blocks, span,
// length as given): called once for each sequence, on its lane.
template <int KB, typename W, typename F>
KVPOP_HD void split_work(W& w, Split& sp, bool f32, F see) {
  int64_t total = 0;
  int longest = 0, seqs = 0;
  for (int b0 = 0; b0 < sp.batch; b0 += 32) {
    const auto nb = w.lanes([&](int lane) {
      const int b = b0 + lane;
      if (b >= sp.batch) return 0;
      const int given = sp.lens[b];
      const Span s = span_of(sp, given);
      const int n = (s.n + KB - 1) / KB - s.lo / KB;
      see(b, n, s, given);
      return n;
    });
    total += w.sum(nb);
    longest = greater(longest, w.top(nb));
    seqs += w.some(nb);
  }
  sp.total = total;
  const int64_t even = quotient(total + sp.groups - 1, sp.groups);
  sp.share = greater(even, static_cast<int64_t>(kMinShare));
  if (longest * KB <= solo_tokens(f32) && seqs > sp.groups) {
    sp.solo = 1;
  } else if (seqs > 0 && seqs <= sp.groups) {
    // the smallest largest part with which there are no more parts than groups
    auto fits = [&](int s) {
      int items = 0;
      for (int b0 = 0; b0 < sp.batch; b0 += 32) {
        auto count = [&](int lane) { return b0 + lane < sp.batch ? blocks_of<KB>(sp, b0 + lane) : 0; };
        const auto nb = b0 == 0 ? w.cached(count) : w.lanes(count);
        items += w.few(w.each(nb, [&](int x) { return lesser(parts_of(x, s), sp.groups + 1); }));
      }
      return items <= sp.groups;
    };
    const int per = sp.groups / seqs;
    // (no more sequences than groups: no share above the longest)
    int lo = static_cast<int>(sp.share), hi = (longest + per - 1) / per;     // hi fits: no sequence has more than `per` parts
    if (hi <= lo || fits(lo)) {
      hi = lo;
    } else {
      while (hi - lo > 1 + lo / 32) {
        const int mid = lo + (hi - lo) / 2;
        if (fits(mid)) hi = mid;
        else lo = mid;
      }
    }
    if (hi <= most_of(sp.share)) {
      sp.aligned = 1;
      sp.share = hi;
    }
  }
}

// Where an item lies: block `skip` of sequence b (or, aligned, its part `skip` of `parts`), head h.
struct Place {
  int b, h, parts, skip;
  int64_t left, pos;
};

// The item of a group where parts are fixed: kMinShare blocks of one sequence.
template <int KB>
KVPOP_HD bool fixed_part(const Split& sp, int grp, int h, Item& x) {
  const int b = grp / sp.fixed, part = grp - b * sp.fixed;
  const Span s = span_of(sp, sp.lens[b]);
  const int j0 = s.lo / KB, nb = (s.n + KB - 1) / KB - j0;
  if (part * kMinShare >= nb) return false;
  const int j = j0 + part * kMinShare, jend = lesser(j + kMinShare, j0 + nb);
  x = Item{b, h, s.lo, s.n, j, jend, grp - part, parts_of(nb, kMinShare), 0, jend - j, 0};
  return true;
}

// Warp u's item, or the next one that has blocks, where warps take one sequence and head each.
template <int KB>
KVPOP_HD bool solo_part(const Split& sp, int u, int warps, Item& x) {
  const int units = sp.batch * sp.Hkv;
  int b = 0, nb = 0;
  for (;; u += warps) {
    if (u >= units) return false;
    b = u / sp.Hkv;
    nb = blocks_of<KB>(sp, b);
    if (nb > 0) break;
  }
  const Span s = span_of(sp, sp.lens[b]);
  const int j0 = s.lo / KB;
  x = Item{b, u - b * sp.Hkv, s.lo, s.n, j0, j0 + nb, 0, 1, 0, nb, u};
  return true;
}

// The item at a place.
template <int KB>
KVPOP_HD Item item_at(const Split& sp, const Place& p, int grp) {
  const Span s = span_of(sp, sp.lens[p.b]);
  const int j0 = s.lo / KB, nb = (s.n + KB - 1) / KB - j0;
  Item x;
  x.b = p.b; x.h = p.h; x.lo = s.lo; x.n = s.n; x.pos = p.pos;
  if (sp.aligned) {         // part `skip`
    const int share = static_cast<int>(sp.share);
    x.j = j0 + p.skip * share;
    x.jend = lesser(x.j + share, j0 + nb);
    x.left = x.jend - x.j;
    x.first = grp - p.skip; x.parts = p.parts; x.second = 0;
  } else {
    x.j = j0 + p.skip;
    x.jend = static_cast<int>(lesser(static_cast<int64_t>(j0 + nb), x.j + p.left));
    x.left = p.left;
    const int64_t beg = p.pos - p.skip;              // of the sequence
    x.first = static_cast<int>(quotient(beg, sp.share));
    x.parts = static_cast<int>(quotient(beg + nb - 1, sp.share)) - x.first + 1;
    x.second = beg != x.first * sp.share;
  }
  return x;
}

// CTA cta's first or next item (`it`: the one before); false at the end.  CTAs
// take one head, or with more heads than CTAs every n_cta-th.  put(f): takes
// the item that f() makes.
template <int KB, typename W, typename P>
KVPOP_HD bool next_part(W& w, const Split& sp, const Item& it, bool start, int cta, int n_cta, P put) {
  const bool many = sp.Hkv > n_cta;
  const int grp = many ? 0 : cta / sp.Hkv;
  if (!start && it.left > it.jend - it.j) {       // the range goes on in the next sequence that has blocks
    int b = it.b;
    do ++b; while (blocks_of<KB>(sp, b) == 0);
    const Place x{b, it.h, 1, 0, it.left - (it.jend - it.j), it.pos + (it.jend - it.j)};
    put([&] { return item_at<KB>(sp, x, grp); });
    return true;
  }
  const int h = start ? (many ? cta : cta - grp * sp.Hkv) : it.h + n_cta;
  if (h >= sp.Hkv || grp >= sp.groups) return false;
  if (sp.fixed > 0) {
    Item x;
    if (!fixed_part<KB>(sp, grp, h, x)) return false;
    put([&] { return x; });
    return true;
  }
  // the sequence in which the range begins
  const int64_t target = sp.aligned ? grp : grp * sp.share;
  int64_t before = 0;
  for (int b0 = 0;; b0 += 32) {
    if (b0 >= sp.batch) return false;
    auto count = [&](int lane) { return b0 + lane < sp.batch ? blocks_of<KB>(sp, b0 + lane) : 0; };
    auto own = b0 == 0 ? w.cached(count) : w.lanes(count);
    if (sp.aligned) own = w.each(own, [&](int nb) { return parts_of(nb, static_cast<int>(sp.share)); });
    typename W::Hit hit;
    if (w.find(own, before, target, sp.batch > 1, hit)) {
      const Place x{b0 + hit.lane, h, hit.own, static_cast<int>(target - before - (hit.sum - hit.own)),
                    lesser(sp.share, sp.total - target), target};
      put([&] { return item_at<KB>(sp, x, grp); });
      return true;
    }
    before += hit.sum;
  }
}

// Partials.  A range begins in one sequence and ends in another, so a group
// leaves at most two partials per head: that of its range's first sequence,
// and another.  Partial i of an item's sequence: by group, and whether its
// range begins with this sequence.
template <typename X>
KVPOP_HD int64_t slot_of(const X& x, int i, int Hkv) {
  return static_cast<int64_t>(2 * (x.first + i) + (i == 0 ? x.second : 0)) * Hkv + x.h;
}

}  // namespace kvpop
