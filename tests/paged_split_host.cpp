// The split of the paged attention's work (kvpop_paged_split.cuh), compiled as
// plain C++: every item of every CTA, with loops in the place of a warp's lanes.
#include <array>
#include <cstdint>

#include "kvpop_paged_split.cuh"

using namespace kvpop;

namespace {

template <typename Sum>
struct LoopWarp {
  using Lanes = std::array<int, 32>;
  struct Hit {
    int lane, own;
    int64_t sum;
  };
  template <typename F> Lanes lanes(F f) const {
    Lanes v;
    for (int i = 0; i < 32; ++i) v[i] = f(i);
    return v;
  }
  template <typename F> Lanes cached(F f) const { return lanes(f); }
  template <typename F> Lanes each(const Lanes& v, F f) const { return lanes([&](int i) { return f(v[i]); }); }
  int64_t sum(const Lanes& v) const {
    Sum s = 0;
    for (int x : v) s += x;
    return static_cast<int64_t>(s);
  }
  int few(const Lanes& v) const {
    int s = 0;
    for (int x : v) s += x;
    return s;
  }
  int top(const Lanes& v) const {
    int m = v[0];
    for (int x : v) m = x > m ? x : m;
    return m;
  }
  int some(const Lanes& v) const {
    int n = 0;
    for (int x : v) n += x > 0;
    return n;
  }
  bool find(const Lanes& v, int64_t before, int64_t target, bool, Hit& hit) const {
    Sum s = 0;
    for (int i = 0; i < 32; ++i) {
      s += v[i];
      hit = Hit{i, v[i], static_cast<int64_t>(s)};
      if (before + static_cast<int64_t>(s) > target) return true;
    }
    return false;
  }
};

// out: rows of ten numbers, (CTA, warp or -1, b, h, j, jend, first, parts, own partial's slot, 0-based number of the item).
template <int KB>
int64_t items(bool f32, const int32_t* lens, int batch, int Hkv, int window, int64_t tokens, int most, int warps_per_cta,
              int64_t* out, int64_t room, int64_t* how) {
  const Launch launch = launch_of(most, tokens, KB, window, Hkv, batch);
  Split sp{};
  sp.lens = lens;
  sp.batch = batch; sp.Hkv = Hkv; sp.window = window; sp.fixed = launch.fixed;
  sp.cap = static_cast<int>(lesser(tokens, kMostTokens));
  sp.groups = greater(1, launch.grid / Hkv);
  sp.share = kMinShare;
  LoopWarp<BlockSum<KB>> w;
  if (sp.fixed == 0) split_work<KB>(w, sp, f32, [](int, int, const Span&, int) {});
  const int64_t facts[] = {launch.grid, sp.fixed, sp.groups, sp.share, sp.total, sp.aligned, sp.solo};
  for (int i = 0; i < 7; ++i) how[i] = facts[i];
  int64_t n = 0;
  auto note = [&](int cta, int warp, const Item& x, int at) {
    if (n < room) {
      const int grp = Hkv > launch.grid ? 0 : cta / Hkv;
      const int64_t slot = x.parts > 1 ? slot_of(x, grp - x.first, Hkv) : -1;
      const int64_t row[] = {cta, warp, x.b, x.h, x.j, x.jend, x.first, x.parts, slot, at};
      for (int i = 0; i < 10; ++i) out[n * 10 + i] = row[i];
    }
    ++n;
  };
  Item x{};
  for (int cta = 0; cta < launch.grid; ++cta) {
    if (sp.solo) {
      for (int warp = 0; warp < warps_per_cta; ++warp) {
        const int all = launch.grid * warps_per_cta;
        int at = 0;
        for (int u = cta * warps_per_cta + warp; solo_part<KB>(sp, u, all, x); u = static_cast<int>(x.pos) + all) note(cta, warp, x, at++);
      }
    } else {
      auto put = [&](auto make) { x = make(); };
      int at = 0;
      for (bool start = true; next_part<KB>(w, sp, x, start, cta, launch.grid, put); start = false) note(cta, -1, x, at++);
    }
  }
  return n;
}

}  // namespace

extern "C" int64_t split_items(int KB, int f32, const int32_t* lens, int batch, int Hkv, int window, int64_t tokens, int most,
                               int warps_per_cta, int64_t* out, int64_t room, int64_t* how) {
  switch (KB) {
    case 8: return items<8>(f32, lens, batch, Hkv, window, tokens, most, warps_per_cta, out, room, how);
    case 16: return items<16>(f32, lens, batch, Hkv, window, tokens, most, warps_per_cta, out, room, how);
    case 32: return items<32>(f32, lens, batch, Hkv, window, tokens, most, warps_per_cta, out, room, how);
    case 64: return items<64>(f32, lens, batch, Hkv, window, tokens, most, warps_per_cta, out, room, how);
  }
  return -1;
}
// The slot of partial i of a sequence whose parts begin in group `first`.
extern "C" int64_t split_slot(int first, int second, int h, int i, int Hkv) {
  Item x{};
  x.first = first; x.second = second; x.h = h;
  return slot_of(x, i, Hkv);
}
