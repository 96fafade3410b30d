// The few-token layer's work as a line of units cut into tickets (decode_umma.cu).
// Plain arithmetic, for the kernels, their host side and a compiler without CUDA.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define MOE_LINE_FN __host__ __device__ __forceinline__
#else
#define MOE_LINE_FN inline
#endif

namespace moe {
namespace decode {

constexpr int kBlocks = 148;                // of the expert kernels: one an SM
constexpr int kLongUnits = 16;

// A phase's line of units and its cut into tickets of q units.
struct Line {
  int nj, kc;      // tiles of a slot, units of a tile
  int units, q, tickets;
  MOE_LINE_FN int start(int t) const { return t * q < units ? t * q : units; }
  MOE_LINE_FN int ticket_of(int u) const { return u / q; }
  // Partial-sum entry of ticket t's piece of the tile that starts at unit a.
  MOE_LINE_FN int entry(int t, int a) const { return 2 * t + (t * q >= a ? 0 : 1); }
};
// One ticket a block, or `per_block` of them where that leaves two a block at least
// kLongUnits units each.  More tickets even out the blocks' ends, and cut tiles
// into more pieces: 2 a block for gate/up and 4 for down measured best (2 and 2: 208 us
// for 8 tokens 4096/64/4/2048, 200 with 2 and 4, 202 with 4 and 4; a line
// ending in shorter tickets gained nothing over that).
MOE_LINE_FN int ticket_count(int64_t units, int per_block) {
  return units >= (int64_t)kBlocks * 2 * kLongUnits ? per_block * kBlocks : kBlocks;
}
// A ticket shorter than `least` units, whose pieces' partial sums would cost more than their weights
// with many tokens, becomes `least` units long; where a tile is no longer than that, it becomes the
// tile, also if that is the shorter: nothing is cut then and nothing passes through partial sums
// (100 tokens 256/6/6/8192: 113 us, 123 with tickets of the blocks' equal shares; 128 tokens
// 128/8/8/8192: 148 and 154).  Only such a line, which has no piece to keep, has more
// tickets than ticket_count.
MOE_LINE_FN Line make_line(int slots, int nj, int kc, int per_block, int least) {
  Line l;
  l.nj = nj;
  l.kc = kc;
  l.units = slots * nj * kc;
  const int most = ticket_count(l.units, per_block);
  l.q = (l.units + most - 1) / most;
  if (l.q < least) l.q = least < kc ? least : kc;
  l.tickets = (l.units + l.q - 1) / l.q;
  return l;
}
// A ticket's next piece: units [pos, pos + len) of one tile.
struct Piece {
  int tile, k0, len;
};
MOE_LINE_FN Piece piece_at(const Line& l, int pos, int end) {
  Piece p;
  p.tile = pos / l.kc;
  p.k0 = pos - p.tile * l.kc;
  p.len = l.kc - p.k0 < end - pos ? l.kc - p.k0 : end - pos;
  return p;
}
}  // namespace decode
}  // namespace moe
