// k6_packed_tma.h -- tensor maps over packed token rows [tokens][heads][128] of
// 16-bit elements with a stride between tokens, and over pages of such rows:
// 64-dim panels in 128-byte swizzled rows, zero fill past the last token or page.
#pragma once

#include <cuda.h>

#include "k6_internal.h"

namespace k6 {

// box = 64 dims x box_heads x box_tokens; smem row = token * box_heads + head.
bool make_rows_map(CUtensorMap *m, const void *base, long tokens, int heads, long stride, int box_heads,
                   int box_tokens, const char **why);

// Pages of one head's keys.  A box is 2^g.box_log2 tokens: 64 dims of them, [pages][tokens]
// [heads][128], or (grouped; c.span wanted) both 64-dim panels as groups of 8
// tokens, each group's panels one behind the other.
bool make_pages_map(CUtensorMap *m, const PagedCache &c, const PagedGeom &g, bool grouped, const char **why);

// A query tile: the G heads of one key head of g.tpt tokens.
static inline bool packed_q_map(CUtensorMap *m, const void *q, const PackedGeom &g, long stride, const char **why) {
    return make_rows_map(m, q, g.Tq, g.H, stride, g.G, g.tpt, why);
}

// A tile of 128 keys of one head.
static inline bool packed_kv_map(CUtensorMap *m, const void *k, long tokens, int heads, long stride,
                                 const char **why) {
    return make_rows_map(m, k, tokens, heads, stride, 1, 128, why);
}

}  // namespace k6
