// kv8_plan.h -- how the attention over the 8-bit paged KV cache is launched: the
// sizes of its workgroups' pieces and of the memory that they join in.  Plain
// C++ of the sizes alone, so that a host program can check the bounds.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

namespace nvfp4 {

struct Kv8Pool {
  uint8_t *k, *v;    // codes  [pages][heads][page * D]
  uint8_t *ks, *vs;  // scales [pages][heads]
  float *w;          // accumulated attention weight [pages][page], or null
  int pages, heads, shift;
};

struct Kv8Batch {
  const int *table;   // [seqs][cols] page of each block of tokens
  const int *lens;    // [seqs] tokens, the call's own with them
  const int *starts;  // [seqs + 1] first row of each sequence, or null: rows / seqs each
  int seqs, cols, rows, max_rows;
};

struct Kv8Rows {  // bf16 [rows][heads][dim], the last dimension contiguous
  const void *ptr;
  int64_t row_stride, head_stride;  // elements
};

// Attention of rows over the cache: out bf16 [rows][q_heads][dim], lse fp32
// [rows][q_heads].  `max_len` bounds the lengths (the grid's size only: a
// longer sequence is a caller's error that leaves its further tokens unseen).
struct Kv8Attn {
  Kv8Rows q;
  int q_heads, max_len;
  int window;   // 0: none
  float scale;
  void *out;
  float *lse;   // or null
};

struct Kv8Plan {
  int group;    // query heads per KV head
  bool few;     // the kernel that splits the tokens (few rows)
  int ct, spw, rounds;  // its 16-column tiles, a wave's 32-token steps at a time, and times
  int blocks;   // column blocks of a sequence
  int splits;   // parts of a sequence's tokens (few rows)
  bool dealt;   // equal runs of tiles for the workgroups (many rows)
  // the weights pass: tokens of a sequence (rounded up); columns whose scores
  // the attention leaves for it (0: it takes K again), parts of the columns
  int len_pad, score_cols, parts;
  int link_bits, link_blocks;  // of the lists of blocks (Kv8Links)
  size_t counter_bytes, part_floats, score_floats, link_words;
};
constexpr int kKv8MaxItems = 65536;  // arrival counters

constexpr int kKv8LinkBits = 11, kKv8Chains = 32;  // at most 2^11 workgroups of so many lists

constexpr int kDecodeWaves = 4;  // of a workgroup (few rows)
constexpr int kMaxSplits = 128;  // of a sequence's tokens
constexpr int kMaxSteps = 31;  // a wave's, two units a lane; lanes 62 and 63 name none
// waves a SIMD holds: what the accumulators (D * CT / 4 registers), Q and the codes leave room for
constexpr int decode_waves(int dim, int ct) { return dim * ct <= 64 ? 4 : dim * ct <= 128 ? 3 : 2; }
// many rows:
constexpr int kManyCols = 256;     // of an item
constexpr int kManyGroups = 256;   // one on each CU
constexpr int kManyItems = 384;    // most that are dealt
constexpr int kStart = 6;          // an item's start and end cost as much as so many tiles
constexpr int many_floats(int dim) { return kManyCols * dim + 4 * kManyCols; }  // of a part
// the weights:
constexpr int kWeightWaves = 8, kWeightTokens = 64 * kWeightWaves;  // of a workgroup

// Few rows: up to so many (row, head) columns of a KV head.  Beyond one
// workgroup's (16, 32 or 64 by head size) its blocks read the codes again,
// from the caches; at 128 columns of 8 sequences of 16000 tokens the two
// kernels take 64 and 62 us, at 66 50 and 60 us, at 105 of 13 short ones 21
// and 29 us (head size 256: at 120 86 and 80 us).
constexpr int kv8_few_cols(int dim) { return dim == 256 ? 64 : 128; }
constexpr int kWeightGroups = 512;  // of the second pass over K
// workgroups wanted: those that the CUs hold at a time (bound of a plan's: kDecodeGroups)
constexpr int kDecodeGroups = 768;
inline int decode_groups(int dim, int ct) { return std::min(256 * decode_waves(dim, ct), kDecodeGroups); }

// 16-column tiles of a workgroup: as many accumulators as leave two waves a SIMD
inline int few_tiles(int64_t cols, int dim) { return std::min(cols <= 16 ? 1 : cols <= 32 ? 2 : 4, 256 / dim); }

inline int64_t cols_of(const Kv8Batch &s, const Kv8Plan &pl) { return (int64_t)s.max_rows * pl.group; }

inline Kv8Plan kv8_plan(const Kv8Attn &a, const Kv8Pool &c, const Kv8Batch &s, int dim) {
  Kv8Plan pl = {};
  pl.group = a.q_heads / c.heads;
  const int64_t cols = cols_of(s, pl);
  pl.few = cols <= kv8_few_cols(dim);
  // (the same for every call, so that one of other sizes finds its words as they have to be)
  pl.counter_bytes = (size_t)(kKv8MaxItems + (kKv8Chains << kKv8LinkBits)) * 4;
  if (pl.few) {
    pl.ct = few_tiles(cols, dim);
    pl.blocks = (int)((cols + 16 * pl.ct - 1) / (16 * pl.ct));
    const int items = std::max(s.seqs * c.heads * pl.blocks, 1);
    const int64_t seen = a.window ? std::min<int64_t>(a.max_len, (int64_t)a.window + s.max_rows + 31) : a.max_len;
    const int steps = (int)((seen + 31) / 32) + (a.window ? 1 : 0);
    // Equal pieces of the longest sequence, as many as fill the CUs once, of at
    // most kMaxSteps steps a wave.  Two sequences of 131000 tokens, 8 KV heads:
    // 32 pieces each (a part of the CUs' places unused) 107 us, 46 pieces (all
    // of them) 95 us, 64 pieces 100 us; more cost more in the join.
    const int even = std::max((steps + 3) / 4, 1);  // steps of a wave if it were one piece
    // One workgroup joins an item's pieces, so where there are few items s
    // pieces cost steps / s + s of it: no more than in proportion to the root of
    // the steps, the fewer the larger a piece's sums (1 item, 130000 tokens: 64
    // pieces 26 us, 128 30 us; 8 items, 16000 tokens: 32 16 us, 96 20 us; 4 items
    // of 64 columns, 15879 tokens: 16 27 us, 108 63 us), and then as many for
    // each CU (32 items: 13 32 us, 8 25 us).
    int filled = (decode_groups(dim, pl.ct) + items - 1) / items;
    const int joined = std::max((int)(1.25 * std::sqrt(steps * 128.0 / (pl.ct * dim))), 1);
    if (joined < filled) filled = items * joined >= 256 ? items * joined / 256 * 256 / items : joined;
    int want = std::max(filled, (even + kMaxSteps - 1) / kMaxSteps);
    want = std::min(want, even);
    pl.spw = (even + want - 1) / want;
    auto pieces = [&](int spw) { return std::max((steps + 4 * spw - 1) / (4 * spw), 1); };
    const int most = items <= kKv8MaxItems ? kMaxSplits : 1;
    pl.rounds = (pieces(pl.spw) + most - 1) / most;
    pl.splits = (pieces(pl.spw) + pl.rounds - 1) / pl.rounds;
    if (pl.splits > 1)
      pl.part_floats = (size_t)items * pl.splits * 16 * pl.ct * (dim + 2);
  }
  if (!pl.few) {
    pl.blocks = (int)((cols + kManyCols - 1) / kManyCols);
    const int64_t items = std::max<int64_t>((int64_t)s.seqs * c.heads * pl.blocks, 1);
    const int64_t seen = a.window ? std::min<int64_t>(a.max_len, (int64_t)a.window + s.max_rows) : a.max_len;
    // Dealt where items are too few to even out over the CUs, and long enough
    // for parts to pay.  6 sequences of up to 900 rows and 9000 tokens (384
    // items) 308 us as items, 257 us dealt; a prompt of 8192 (1024 items) 518
    // and 613 us: its short items cost more starts than the idle CUs.
    pl.dealt = items <= kManyItems && seen >= 1024 && items * (a.max_len / 32 + 8) < (1 << 30);
    if (pl.dealt) pl.part_floats = 2 * kManyGroups * (size_t)many_floats(dim) + 2 * (size_t)items;
  }
  pl.len_pad = (a.max_len + kWeightTokens - 1) / kWeightTokens * kWeightTokens;
  pl.parts = 1;
  if (c.w) {
    pl.link_blocks = (int)(((int64_t)a.max_len + (1 << c.shift) - 1) >> c.shift);
    pl.link_words = 2 * (size_t)s.seqs * pl.link_blocks;
    while (pl.link_bits < kKv8LinkBits && 1 << pl.link_bits < c.pages) ++pl.link_bits;
    const size_t tokens = (size_t)s.seqs * c.heads * pl.len_pad;
    if (pl.few && cols <= 16 && cols * pl.len_pad < (1 << 29)) {
      pl.score_cols = (int)cols;
      pl.score_floats = tokens * (size_t)cols;
    } else {
      // two workgroups a CU where the columns allow it
      const int64_t groups = (int64_t)s.seqs * c.heads * (pl.len_pad / kWeightTokens);
      pl.parts = (int)std::max<int64_t>(std::min<int64_t>(kWeightGroups / std::max<int64_t>(groups, 1), cols / 256), 1);
      pl.score_floats = tokens * (size_t)pl.parts;
    }
  }
  return pl;
}

// Bytes of a workspace: the arrival counters, then the floats.
inline size_t kv8_align(size_t b) { return (b + 255) & ~(size_t)255; }
inline size_t kv8_workspace_bytes(const Kv8Plan &pl) {
  return kv8_align(pl.counter_bytes) + kv8_align(4 * (pl.part_floats + pl.score_floats + pl.link_words));
}

// Those of any call with these sequences or fewer, as many rows and tokens of
// each or fewer, and any window.  The pieces of a sequence do not only grow with
// its tokens (129 are taken in two rounds of 65, 128 in one) and a window may
// add a step, so each width of the columns is bounded by the most pieces it has.
inline size_t kv8_workspace_bound(const Kv8Attn &a, const Kv8Pool &c, const Kv8Batch &s, int dim) {
  const Kv8Plan pl = kv8_plan(a, c, s, dim);
  const size_t pairs = std::max((size_t)s.seqs * c.heads, (size_t)1);
  // steps of a wave if it were one piece (a window may take a step more)
  const size_t even = ((size_t)(a.max_len + 31) / 32 + 1 + 3) / 4;
  const size_t longest = std::min((even + kMaxSteps - 1) / kMaxSteps, (size_t)kMaxSplits);
  const int64_t few = std::max<int64_t>(std::min<int64_t>(cols_of(s, pl), kv8_few_cols(dim)), 1);
  size_t floats = 0;
  for (int64_t cols = 16; cols < few + 16; cols += 16) {
    const int ct = few_tiles(cols, dim);
    // (with more items than counters no sequence is split)
    const size_t items = std::min<size_t>(pairs * ((cols + 16 * ct - 1) / (16 * ct)), kKv8MaxItems);
    // as many as fill the CUs, or as many as the longest sequence's steps ask for
    const size_t pieces = std::min(std::max(decode_groups(dim, ct) + items, items * longest), items * kMaxSplits);
    floats = std::max(floats, pieces * 16 * ct * (dim + 2));
  }
  if (!pl.few) floats = std::max(floats, 2 * kManyGroups * (size_t)many_floats(dim) + 2 * kManyItems);
  // 16 columns' scores, or kWeightGroups parts of kWeightTokens
  if (c.w) floats += std::max(pairs * pl.len_pad * 16, (size_t)kWeightGroups * kWeightTokens) + pl.link_words;
  return kv8_align(pl.counter_bytes) + kv8_align(4 * floats);
}

}  // namespace nvfp4
