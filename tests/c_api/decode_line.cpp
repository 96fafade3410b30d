// The cut of the few-token layer's work into tickets, over many shapes: every unit is in one
// ticket, every piece of a cut tile has a partial-sum entry of its own inside the buffer,
// and there are no more tickets than the buffer is sized for unless no tile is cut.
#include <stdio.h>

#include <vector>

#include "decode_line.cuh"

using namespace moe::decode;

static int fail(const Line& l, int slots, int per_block, int least, const char* what) {
  printf("%s: slots %d nj %d kc %d per_block %d least %d: q %d tickets %d\n", what, slots, l.nj, l.kc, per_block, least,
         l.q, l.tickets);
  return 1;
}

static int check(int slots, int nj, int kc, int per_block, int least) {
  const Line l = make_line(slots, nj, kc, per_block, least);
  const int most = ticket_count((int64_t)slots * nj * kc, per_block);
  if (l.q < (least < kc ? least : kc)) return fail(l, slots, per_block, least, "a ticket is too short");
  if (l.tickets > most && l.q != kc) return fail(l, slots, per_block, least, "too many tickets");
  if (l.start(0) != 0 || l.start(l.tickets) != l.units || l.start(l.tickets - 1) >= l.units)
    return fail(l, slots, per_block, least, "the line's ends");
  if (l.units > 100000) return 0;
  std::vector<char> used(2 * (size_t)most, 0);
  int pos = 0;
  for (int t = 0; t < l.tickets; ++t) {
    const int end = l.start(t + 1);
    while (pos < end) {
      const Piece p = piece_at(l, pos, end);
      const int a = p.tile * kc;
      if (p.len <= 0 || a + p.k0 != pos || p.k0 + p.len > kc || l.ticket_of(pos) != t)
        return fail(l, slots, per_block, least, "a piece");
      if (p.len != kc) {
        const int e = l.entry(t, a);
        if (e < 0 || e >= 2 * most || used[e]) return fail(l, slots, per_block, least, "a piece's entry");
        // what adds the pieces up finds the first ticket's by its entry, the others' at 2 t
        if (t != l.ticket_of(a) && e != 2 * t) return fail(l, slots, per_block, least, "a later piece's entry");
        used[e] = 1;
      }
      pos += p.len;
    }
  }
  return pos == l.units ? 0 : fail(l, slots, per_block, least, "a unit is missing");
}

int main() {
  const int slots[] = {1, 2, 3, 4, 7, 16, 26, 61, 64, 130, 256}, nj[] = {1, 2, 3, 8, 10, 11, 16, 64, 112, 512};
  const int kc[] = {2, 4, 6, 10, 22, 32, 64, 112, 224, 1024}, per_block[] = {2, 4}, least[] = {4, 8, 13, 15, 32};
  int bad = 0;
  for (int s : slots)
    for (int j : nj)
      for (int k : kc)
        for (int p : per_block)
          for (int l : least) bad += check(s, j, k, p, l);
  printf("%d bad\n", bad);
  return bad != 0;
}
