// Index arithmetic of chunk attention over pages, shared by the kernel and by host code: what a piece of work sees, and how the
// line of all work is cut.
#pragma once
#include <stdint.h>

#include "paged.h"

namespace adp {

constexpr int kChunkKeys = 64;       // positions of a block
// Blocks that a part of a piece has at least (8: 32 sequences of up to 8 tokens 131 us instead of 127, prompts and single tokens
// together 76 instead of 74), and that are worth a CTA of their own (8 rows over 2,000 and over 16,000 positions: 22.6 and 42.7 us; 16:
// 24.7 and 39.5; 24: 27.7 and 39.7; over e4m3 28.7 and 48.5; 33 and 47; 39 and 48).
constexpr int kChunkMinPart = 4;
constexpr int kChunkMinWork = 8;
constexpr int kNoWindow = 0x7FFFFFFF;

ADP_INLINE int32_t chunk_min(int32_t a, int32_t b) { return a < b ? a : b; }
ADP_INLINE int32_t chunk_max(int32_t a, int32_t b) { return a > b ? a : b; }

// The blocks that rows at positions first .. last see, as one line: those of the first `sinks` positions, then those from the
// window of the first row to the last row's own.
struct ChunkSpan {
  int32_t head;  // blocks of the sinks
  int32_t gap;   // blocks left out behind them
  int32_t n;     // blocks of the line
  int32_t low;   // the first position that is not seen as one of the first ones only
};
ADP_INLINE ChunkSpan chunk_span(int32_t first, int32_t last, int32_t window, int32_t sinks) {
  ChunkSpan s;
  s.low = chunk_max(0, chunk_max(first, 0) - window + 1);
  s.head = (chunk_min(sinks, s.low) + kChunkKeys - 1) / kChunkKeys;
  s.gap = chunk_max(0, s.low / kChunkKeys - s.head);
  s.n = last < 0 ? 0 : last / kChunkKeys + 1 - s.gap;
  return s;
}
// The block (by its position in the cache) that is number i of the line, and the number of a block behind the sinks'.
ADP_INLINE int32_t chunk_block(const ChunkSpan& s, int32_t i) { return i < s.head ? i : i + s.gap; }

// What starting and ending a piece of work costs, in blocks of it: where its rows fit one tile, whose blocks cost half as much, and
// whose results the tiles add up, twice as many (4 for both: 32 sequences of up to 8 tokens 130.5 us instead of 127; 8 for both: prompts and
// single tokens together 77.4 instead of 74).  A block itself counts as one for both: the line is cut by blocks, not by their time.
ADP_INLINE int32_t chunk_over(int32_t tokens, int32_t tile) { return tokens <= tile ? 8 : 4; }

// Where a cut that falls j units behind a piece's blocks' start (negative: in front) goes: whole blocks, and no part of less than
// kChunkMinPart.
ADP_INLINE int32_t chunk_cut(int32_t blocks, int64_t j) {
  if (j < kChunkMinPart) return 0;
  return blocks - j < kChunkMinPart ? blocks : (int32_t)j;
}

// CTAs that share work of `total` units in `items` pieces: one for every piece, and more where the pieces are long.
ADP_INLINE int32_t chunk_parts(int64_t total, int64_t items, int32_t ctas) {
  const int64_t by_work = total / kChunkMinWork, want = items > by_work ? items : by_work;
  return want < 1 ? 1 : want > ctas ? ctas : (int32_t)want;
}

}  // namespace adp
