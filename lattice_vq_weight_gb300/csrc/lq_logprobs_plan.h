// How the rows of logits are divided among CTAs (lq_logprobs.cu).  Host code, apart from
// CUDA.  Internal to the library.
#pragma once

#include <cstdint>

namespace lq {
namespace score {

constexpr int kThreads = 512;                  // that compute, of a CTA
constexpr int kMaxCluster = 8;                 // CTAs that share a row
constexpr int kPieces = 4;                     // of a share
constexpr int kMostBytes = 208 * 1024;         // of a share in shared memory at once
constexpr int kFixed = 64 * 1024;              // what a row costs beside its elements, in elements of a CTA's

struct Division {
  int cluster;               // CTAs per row
  int64_t share;             // elements of a row per CTA
  int segment;               // of those in shared memory at once
  int per_piece;             // 16-byte chunks of a piece, whole batches: chunks one at a time take twice as long
  int chunks;                // of a segment, whose ends may be partial ones
};

struct Plan {
  Division d;
  int64_t clusters;          // to launch
};

// Elements of a share that are in shared memory at once, at most.
inline int64_t most_elements(int esize) { return (kMostBytes - 32) / esize; }

inline Division divide(int64_t vocab, int esize, int cluster) {
  Division d;
  const int64_t most = most_elements(esize);
  d.cluster = cluster;
  d.share = (vocab + cluster - 1) / cluster;
  d.segment = (int)(d.share < most ? d.share : most);
  d.chunks = (d.segment * esize + 15) / 16 + 1;
  const int unit = kThreads * (esize == 2 ? 2 : 4);
  d.per_piece = (d.chunks + kPieces - 1) / kPieces;
  if (d.per_piece > unit / 2) d.per_piece = (d.per_piece + unit - 1) / unit * unit;
  return d;
}

// CTAs per row: enough to hold it in shared memory (or all that a cluster can have), and of
// those the number that ends first, by the rows that a cluster takes one after the other.
// (96 rows of 32000: one CTA each 8.9 us, two 16.6; 33 of 50001: four each 8.7, eight 23.
// Three, 400 rows of 128256 in fp32: 100 us against four's 68.)  at_once(c): clusters of c
// CTAs that the device holds, one CTA per SM (two need more registers than there are), 0 if
// none; false if there is no such c.
template <typename AtOnce>
bool make_plan(int64_t rows, int64_t vocab, int esize, AtOnce at_once, Plan* plan) {
  int64_t least = INT64_MAX;
  for (int c = 1; c <= kMaxCluster && (c == 1 || vocab * esize / c >= 4096); c *= 2) {
    const Division d = divide(vocab, esize, c);
    if (c < kMaxCluster && d.share > d.segment) continue;
    const int64_t clusters = at_once(c);
    if (clusters <= 0) continue;
    const int64_t elements = (int64_t)d.per_piece * kPieces * (16 / esize);
    const int64_t cost = (rows + clusters - 1) / clusters * (elements + kFixed);
    if (cost < least) {
      least = cost;
      plan->d = d;
      plan->clusters = rows < clusters ? rows : clusters;   // each stays for row after row
    }
  }
  return least < INT64_MAX;
}

}  // namespace score
}  // namespace lq
