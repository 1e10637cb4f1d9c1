// Host-only check of the split-K W4A16 workspace (the layout functions of w4a16_kernel.cuh, which the
// library and the kernel use): for every shape, tickets and partial slots lie inside the required
// size; every split tile has tickets of its own; and for every pair of shapes no partial of one call
// covers a ticket of the other, so that calls of different shapes can share a workspace.
// Prints "ok" and exits 0, else prints the first failure.
#include <cstdio>
#include <set>
#include <vector>

#include "w4a16_kernel.cuh"

struct Shape {
  long long T, G;        // tiles, slices per tile
  int mpad, C;           // CTAs
};

struct Range {
  size_t lo, hi;
};

// Bytes that a call's tickets and partials take.
static bool ranges(const Shape& s, Range& tickets, Range& partials) {
  const long long U = s.T * s.G;
  const size_t slot = static_cast<size_t>(s.mpad) * 128 * 4;
  const size_t at = attn::w4_partials_offset(static_cast<int>(s.T * 128));
  tickets = {~size_t(0), 0};
  partials = {~size_t(0), 0};
  std::set<int> used;
  for (long long t = 0; t < s.T; ++t) {
    const int lo = attn::w4_cta_of(t * s.G, U, s.C), hi = attn::w4_cta_of(t * s.G + s.G - 1, U, s.C);
    if (lo == hi) continue;
    for (int q = 0; q < 4; ++q) {
      const int i = attn::w4_ticket(lo, q);
      if (i < 0 || !used.insert(i).second) return false;
      const size_t b = static_cast<size_t>(i) * 4;
      if (b < tickets.lo) tickets.lo = b;
      if (b + 4 > tickets.hi) tickets.hi = b + 4;
    }
    for (int c = lo; c <= hi; ++c) {
      const size_t k = 2 * static_cast<size_t>(c) + (attn::w4_unit0(c, U, s.C) / s.G == t ? 0 : 1);
      if (at + k * slot < partials.lo) partials.lo = at + k * slot;
      if (at + (k + 1) * slot > partials.hi) partials.hi = at + (k + 1) * slot;
    }
  }
  return true;
}

int main() {
  std::vector<Shape> shapes;
  const long long tiles[] = {1, 2, 3, 8, 9, 24, 32, 36, 48, 112, 148, 224, 296, 300, 448, 528, 897, 1002, 4000};
  const long long gs[] = {1, 3, 10, 17, 32, 64, 128};
  for (long long T : tiles)
    for (long long G : gs)
      for (int mpad : {16, 48, 128}) {
        const long long U = T * G;
        long long cap = U / 8;
        cap = cap < 1 ? 1 : (cap > attn::kW4MaxCtas ? attn::kW4MaxCtas : cap);
        for (int most : {2 * 148, 2 * 132, 40}) shapes.push_back({T, G, mpad, static_cast<int>(cap < most ? cap : most)});
      }
  size_t ticket_end = 0, partial_begin = ~size_t(0);
  for (const Shape& s : shapes) {
    Range t, p;
    const long long U = s.T * s.G;
    long long cap = U / 8;
    cap = cap < 1 ? 1 : (cap > attn::kW4MaxCtas ? attn::kW4MaxCtas : cap);
    const size_t need = attn::w4_workspace_bytes(static_cast<int>(s.T * 128), s.mpad, static_cast<int>(cap));
    if (!ranges(s, t, p) || t.hi > need || p.hi > need) {
      std::printf("FAIL T=%lld G=%lld mpad=%d C=%d: tickets end %zu, partials end %zu, size %zu\n", s.T, s.G, s.mpad, s.C,
                  t.hi, p.hi, need);
      return 1;
    }
    if (t.hi > ticket_end) ticket_end = t.hi;
    if (p.lo < partial_begin) partial_begin = p.lo;
  }
  // every pair: the lowest partial of any call lies behind the highest ticket of any other
  if (ticket_end > partial_begin || ticket_end > attn::kW4TicketBytes) {
    std::printf("FAIL tickets reach byte %zu, partials begin at %zu\n", ticket_end, partial_begin);
    return 1;
  }
  std::printf("ok %zu shapes, tickets below %zu, partials from %zu\n", shapes.size(), ticket_end, partial_begin);
  return 0;
}
