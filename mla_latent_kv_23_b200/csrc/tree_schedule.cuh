// Work of the tree attention: row blocks, chunks and segments.
//
// A sequence with n drafted tokens and n_h heads has n n_h query rows (flat
// row i = token i / n_h, head i % n_h), all against the same cached tokens.
// They are taken in blocks of 128 rows, the M dimension of the contractions:
// one block per token at 128 heads, eight tokens per block at 16 heads.  A
// block crosses every 64-token tile of its sequence; a chunk is a run of
// (sequence, block, tile) in that order, over the sequences that have work,
// given by where it and the next chunk start, and the part of a chunk inside one block is a segment.  A segment
// that covers a whole block writes u and lse, any other a partial result.
#pragma once

#include "mla.h"
#include "tree.h"

namespace mla {

// Sequence b as the kernels see it.  n = 0 where it has no drafted tokens, or
// where what the host cannot see is wrong (flag != 0): nothing is read or
// written out of range for it.
struct TreeSeq {
  int b;       // its place in the batch
  int row0;    // its first token of the packed rows
  int n;       // drafted tokens, the last n of its L cached ones
  int L;
  int blocks;  // row blocks
  int tiles;
  int flag;
};

__device__ __forceinline__ void tree_extent(TreeSeq& s, int n_h) {
  s.blocks = (s.n * n_h + kTreeRows - 1) / kTreeRows;
  s.tiles = (s.L - 1) / kTreeTile + 1;
}

__device__ __forceinline__ TreeSeq tree_seq(const int* __restrict__ cu_q,
                                            const int* __restrict__ seqlens, int b, int T, int n_h,
                                            long long max_len) {
  TreeSeq s;
  s.b = b;
  s.row0 = cu_q[b];
  const int end = cu_q[b + 1];
  s.L = seqlens[b];
  s.n = 0;
  s.flag = 0;
  // (with cu_q[b - 1] > cu_q[b] the rows may be the sequence's before it, too)
  if (s.row0 < 0 || end < s.row0 || end > T || end - s.row0 > kTreeMaxNodes ||
      (b > 0 && cu_q[b - 1] > s.row0))
    s.flag = MLA_DEVFLAG_BAD_TREE;
  else
    s.n = end - s.row0;
  s.blocks = s.tiles = 0;
  if (s.n > 0) {
    if (s.L < s.n || s.L > max_len)
      s.flag = MLA_DEVFLAG_BAD_SEQLEN;  // its rows get u = 0, lse = -inf
    else
      tree_extent(s, n_h);
  }
  return s;
}

struct TreeSegment {
  int g;       // row block
  int t0, t1;  // tiles
  int whole;   // covers every tile of the block
  int slot;    // partial slot where it does not
  int first;   // the block's first flat row
  int rows;    // the block's rows (<= 128)
  TreeSeq seq;
};

// The plan's list of the sequences that have work: token, count, length, place.
__device__ __forceinline__ TreeSeq tree_listed(int4 v, int n_h) {
  TreeSeq s;
  s.row0 = v.x;
  s.n = v.y;
  s.L = v.z;
  s.b = v.w;
  s.flag = 0;
  tree_extent(s, n_h);
  return s;
}

struct TreeWalk {
  const int4* seqs;
  int n_h, chunk;
  int k, g, t;     // next tile: place on the list, row block, tile
  int ke, ge, te;  // where the next chunk starts
  TreeSeq seq;     // of place k

  __device__ __forceinline__ void init(const int* rec, const int4* list, int heads, int chunk_id) {
    seqs = list;
    n_h = heads;
    chunk = chunk_id;
    const int4* r = reinterpret_cast<const int4*>(rec) + 2 * chunk_id;
    const int4 r0 = r[0], s0 = r[1], r1 = r[2];  // independent: one memory round trip
    k = r0.x;
    g = r0.y;
    t = r0.z;
    ke = r1.x;
    ge = r1.y;
    te = r1.z;
    seq = tree_listed(s0, n_h);
  }

  __device__ __forceinline__ bool next(TreeSegment& s) {
    while (true) {
      if (k > ke || (k == ke && (g > ge || (g == ge && t >= te)))) return false;
      if (g < seq.blocks) break;
      ++k;
      g = t = 0;
      // (the chunks end at the list's end, which has no entry)
      if (k < ke || te > 0 || ge > 0) seq = tree_listed(seqs[k], n_h);
    }
    s.g = g;
    s.t0 = t;
    s.t1 = (k == ke && g == ge) ? min(te, seq.tiles) : seq.tiles;
    s.whole = t == 0 && s.t1 == seq.tiles;
    s.slot = 2 * chunk + (t == 0 ? 1 : 0);
    s.first = seq.row0 * n_h + g * kTreeRows;
    s.rows = min(kTreeRows, seq.n * n_h - g * kTreeRows);
    s.seq = seq;
    ++g;
    t = 0;
    return true;
  }
};

}  // namespace mla
