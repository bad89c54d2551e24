// Index arithmetic of the paged KV cache operators, shared by the kernels and by host code: where a
// cached position lies, which sequence a packed row belongs to, and how the attention's work is split.
// Every value that reaches a kernel in device memory (lengths, page numbers, row offsets) is checked
// here before it becomes an address.
#pragma once
#include <stdint.h>

#if defined(__CUDACC__)
#define ADP_INLINE __host__ __device__ __forceinline__
#else
#define ADP_INLINE static inline
#endif

namespace adp {

constexpr int kPagedMaxSeqs = 8192;   // sequences of one attention call
constexpr int kPagedMaxPage = 1024;   // positions of a page
constexpr int kPagedWarps = 4;        // warps of an attention CTA, each with a share of the CTA's units

// Cached positions of a sequence: its length, within what its table row can name.
ADP_INLINE int32_t paged_length(int32_t len, int32_t table_width, int log2_page) {
  const int64_t cap = (int64_t)table_width << log2_page;
  return len < 0 ? 0 : (len > cap ? (int32_t)cap : len);
}

// Position of packed row i of a sequence whose rows end before row `next`: its last rows are its last
// positions.  Negative where it has fewer positions than rows.
ADP_INLINE int64_t paged_position(int32_t len, int32_t next, int32_t i) { return (int64_t)len - ((int64_t)next - i); }

// Whether packed row i is one of sequence b's rows [first, next) by its offsets: those of sequence 0 start at 0.
ADP_INLINE bool paged_holds(int32_t b, int32_t first, int32_t next, int32_t i) {
  return first <= i && i < next && (b == 0 ? first == 0 : first >= 0);
}

// The page of a position: an entry of the sequence's table row, or -1 where it has none or names no page.
ADP_INLINE int32_t paged_page(const int32_t* table_row, int32_t table_width, int32_t n_pages, int log2_page, int64_t pos) {
  if (pos < 0 || (pos >> log2_page) >= table_width) return -1;
  const int32_t p = table_row[pos >> log2_page];
  return p >= 0 && p < n_pages ? p : -1;
}

// The attention's work is a line of `total` units (a unit: some consecutive positions of one sequence for
// one KV head and tile of query heads), cut into `parts` even ranges: part i has [begin(i), begin(i + 1)).
ADP_INLINE int64_t split_begin(int64_t total, int32_t parts, int32_t i) { return total * i / parts; }
// The part that unit u falls into (total >= parts).
ADP_INLINE int32_t split_owner(int64_t total, int32_t parts, int64_t u) { return (int32_t)(((u + 1) * parts - 1) / total); }
// CTAs that share `total` units: one unit for each of their warps at least, as long as CTAs are left.
ADP_INLINE int32_t split_parts(int64_t total, int32_t ctas) {
  const int64_t want = (total + kPagedWarps - 1) / kPagedWarps;
  return want < 1 ? 1 : (want > ctas ? ctas : (int32_t)want);
}

// Heads that a warp takes of a row's line of `heads`, `step` of them at a time: the line is cut over several warps as long as the
// call's warps, for n_rows rows, are no more than the `held` that run at once.
ADP_INLINE int32_t row_part_heads(int32_t heads, int32_t step, int32_t n_rows, int32_t held) {
  const int32_t most = (heads + step - 1) / step, room = held / n_rows, parts = room < 1 ? 1 : room > most ? most : room;
  return (most + parts - 1) / parts * step;
}

// How long a wait inside packed attention may take: some wait for a whole piece of work, which sees up to n_k keys (13 ns a
// key, measured), and some for the search of the next one, which looks through up to n_seqs sequences (about 2 us for 32).
ADP_INLINE uint64_t packed_wait_ns(int32_t n_k, int32_t n_seqs) {
  return 1000000000ull + 100ull * (uint64_t)n_k + 1000ull * (uint64_t)n_seqs;
}

}  // namespace adp
