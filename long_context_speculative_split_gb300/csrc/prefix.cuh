// Work partition of the shared-prefix attention, used by the kernels that attend
// over the prefix and by the merge that joins their partial results.
//
// All R = B * T * G query rows of a KV head read the same prefix keys, so they
// form one matrix of R rows; a "pair" is (KV head, block of tile_rows of those
// rows).  The work of a pair is a run of steps along the keys, the steps of all
// pairs lie on one line, and CTA c of n takes the part [c * total / n,
// (c + 1) * total / n) of that line: every CTA gets the same number of steps
// whatever the number of pairs and keys, and a pair is cut at most where a CTA's
// part ends.  Each (CTA, pair) that has steps in common writes one partial
// result to slot c + pair: along the line either c or the pair grows from one
// partial to the next, so no two share a slot.  The prefix length is read on the
// device, so the partition is too.
#pragma once

#include <stdint.h>

#include "internal.h"

namespace mgd {

// Steps of the line for a prefix of plen keys.
struct PrefixLine {
  int nt;      // steps of a pair that uses its whole row block
  int last;    // steps of each head's last pair
  int head;    // steps of one head
  int total;   // of all heads
  int n;       // CTAs that take part
};

__host__ __device__ inline PrefixLine prefix_line(const PrefixGeom &g, int plen, int grid) {
  PrefixLine w;
  w.nt = (plen + g.key_tile - 1) / g.key_tile;
  w.last = g.last_half ? (w.nt + 1) / 2 : w.nt;
  w.head = (g.RT - 1) * w.nt + w.last;
  w.total = w.head * g.Hkv;
  w.n = grid < w.total ? grid : w.total;
  return w;
}
__host__ __device__ inline int prefix_cta_begin(const PrefixLine &w, int c) {
  return static_cast<int>(static_cast<int64_t>(c) * w.total / w.n);
}
// The CTA whose part holds step x.
__host__ __device__ inline int prefix_cta_of(const PrefixLine &w, int x) {
  const uint64_t a = (static_cast<uint64_t>(x) + 1) * w.n - 1;  // the quotient of 32-bit numbers is far cheaper
  return static_cast<int>(a >> 32 ? a / w.total : static_cast<uint32_t>(a) / static_cast<uint32_t>(w.total));
}
__host__ __device__ inline int prefix_pair_begin(const PrefixLine &w, int h, int rt) { return h * w.head + rt * w.nt; }
__host__ __device__ inline int prefix_pair_steps(const PrefixGeom &g, const PrefixLine &w, int rt) {
  return rt == g.RT - 1 ? w.last : w.nt;
}

}  // namespace mgd
