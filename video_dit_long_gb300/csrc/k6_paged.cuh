// k6_paged.cuh -- the plan of a batch of streams whose keys lie in pages: what
// the plan kernel writes and the append and attention kernels read.
//
// Stream s has the query tokens [cu_q[s], cu_q[s+1]) and k_lens[s] keys, the new
// tokens' own among them: query i of Lq sits at key position Lk - Lq + i, and key
// position p lies at token p % page of page table[s][p / page].  The mask is that
// of packed sequences (k6_packed.cuh).
//
// Streams of a group have their first `shared` tokens in common.  Where it saves
// work the tokens of the whole group form the rows of tiles over those keys,
// fetched out of the first stream's pages, up to a multiple of 128 that every
// query of the group sees; the streams' own tiles then begin there.  Each row has
// partials of both, joined like those of a split key range:
//   out = sum_c 2^(lse_c - lse) out_c,   lse = log2 sum_c 2^lse_c.
#pragma once

#include "k6_packed.cuh"

namespace k6 {

constexpr unsigned PAGED_MAGIC = 0x6b365047u;

struct PagedHeader : PackedHeader {
    int page, n_pages, max_pages, n_groups;
};
static_assert(sizeof(PagedHeader) <= PACKED_HEADER_BYTES, "plan header");

// The rows of one unit of tiles: a stream's own keys, or a group's shared ones.
struct __align__(16) PagedUnits {
    int q0, Lq;        // query tokens
    int Lk;            // keys, from the stream's first one (also where lo > 0)
    int lo;            // first key tile
    int row;           // row of the table
    int tiles;         // query tiles; 0: no work of its own
    int prefix;        // the group's first tile over shared keys, or -1: none
    int group_q0;      // first query token of the group
};

// The partials of a tile: n of them from row `row` on, `step` rows apart.
struct __align__(16) PagedParts {
    int row, n, step, unused;
};

// MERGE_ROWS rows, from r0 on, of a tile of one key head that have partials: the
// tile's own, and (prefix >= 0) those of the group's tiles over shared keys, from
// tile `prefix` on.  Where all of the rows belong to one of those tiles its
// partials stand here (prefix = -1): the join is a read less deep.
constexpr int MERGE_ROWS = 16;
struct __align__(16) PagedMerge {
    int tok0, n_tok_hk;
    int prefix, group_q0;
    int row, n, step;  // as in PagedParts, of the tile's row 0
    int r0;
    PagedParts shared; // of the tile's row 0; n = 0: none, or not here
};

struct PagedPlan {
    PagedHeader *head;
    int *count;           // [sms] items of each CTA (fwd and sched as in a PackedPlan)
    PackedItem *first;    // [sms] the first item of each CTA, beside the header, with the key head above its tokens
    PagedMerge *merge;    // [cap_merge, or one per SM where that is more]
    PagedParts *prefix;   // [Hkv][cap_prefix] partials of the tiles over shared keys
    PagedUnits *units;    // [n_seq + n_groups]
    PackedItem *fwd;      // krow0 is the row of the table
    int *sched;
    int *slot;            // [Tq] where a new token's key lies: page * page tokens + place, or -1: nowhere
};

// The plan's parts.  Those up to the first `sms` entries of merge lie in every plan
// on a GPU of that many SMs: see packed_plan_common_bytes.
static inline __host__ __device__ PagedPlan paged_plan_at(void *base, const PagedGeom &p) {
    PagedPlan r;
    char *b = static_cast<char *>(base);
    r.head = reinterpret_cast<PagedHeader *>(b);
    b += PACKED_HEADER_BYTES;
    r.count = reinterpret_cast<int *>(b);
    b += ((size_t)p.g.sms * sizeof(int) + 15) / 16 * 16;
    r.first = reinterpret_cast<PackedItem *>(b);
    b += (size_t)p.g.sms * sizeof(PackedItem);
    r.merge = reinterpret_cast<PagedMerge *>(b);
    b += (size_t)packed_merge_rows(p.g) * sizeof(PagedMerge);
    r.prefix = reinterpret_cast<PagedParts *>(b);
    b += (size_t)p.cap_prefix * p.g.Hkv * sizeof(PagedParts);
    r.units = reinterpret_cast<PagedUnits *>(b);
    b += ((size_t)p.g.n_seq + p.n_groups) * sizeof(PagedUnits);
    r.fwd = reinterpret_cast<PackedItem *>(b);
    b += (size_t)p.g.cap_fwd * sizeof(PackedItem);
    r.sched = reinterpret_cast<int *>(b);
    b += ((size_t)p.g.cap_sched * sizeof(int) + 15) / 16 * 16;
    r.slot = reinterpret_cast<int *>(b);
    return r;
}

// A tile of 128 keys comes in boxes of 2^box_log2 tokens of one page each (a box
// divides both): box i of tile kt of a stream of Lk keys is `tok` tokens into the
// page of the table's column `column`.  paged_boxes: how many of them hold keys.
static inline __host__ __device__ int paged_boxes(const PagedGeom &g, int Lk, int kt) {
    const int left = Lk - kt * 128;
    return ((left < 128 ? left : 128) + (1 << g.box_log2) - 1) >> g.box_log2;
}
static inline __host__ __device__ int paged_box(const PagedGeom &g, int kt, int i, int &column) {
    const int pos = kt * 128 + (i << g.box_log2);
    column = (int)((unsigned long long)(unsigned)pos * g.page_mul >> g.page_shift);
    return pos - column * g.page;
}
// The geometry's part of that.  page_mul = ceil(2^s / page) with 2^(s - 29) >= page: its excess over 2^s / page, below 1,
// times x / 2^s stays below 1 / page, so the quotient's integer part is right; page_mul < 2^30 + 1.
static inline void paged_set_page(PagedGeom &g, int page) {
    g.page = page;
    for (g.box_log2 = 7; page % (1 << g.box_log2); g.box_log2--) {}
    for (g.page_shift = 29; 1ll << (g.page_shift - 29) < page; g.page_shift++) {}
    g.page_mul = (unsigned)(((1ull << g.page_shift) + page - 1) / page);
}
// The page to copy from: one that the pool does not have becomes the first behind it, where a copy fills with zeros.
static inline __host__ __device__ int paged_page(const PagedGeom &g, int page) {
    return (unsigned)page < (unsigned)g.n_pages ? page : g.n_pages;
}
// The same in groups of 8 tokens, `span` of them from one page to the next: how many the pool has, and the one that a
// box begins at.
static inline __host__ __device__ int paged_groups(const PagedGeom &g, int span) {
    return (g.n_pages - 1) * span + g.page / 8;
}
static inline __host__ __device__ int paged_group(const PagedGeom &g, int span, int page, int tok) {
    return (unsigned)page < (unsigned)g.n_pages ? page * span + tok / 8 : paged_groups(g, span);
}

// Key position of the query token in row t of a stream of Lk keys whose rows end at `end` (t < end), or -1: the token lies
// before position 0, or Lk is no length that the table has room for.  Lk comes from the device: it may be any int, and
// neither the comparisons nor the difference leave an int's range.
static inline __host__ __device__ int paged_position(const PagedGeom &g, int t, int end, int Lk) {
    return 0 <= Lk && Lk <= g.g.Tk && end - t <= Lk ? Lk - (end - t) : -1;
}

// True if the plan was made for this batch and holds valid lists.
static inline __device__ bool paged_plan_ok(const PagedHeader &h, const PagedGeom &p) {
    return h.magic == PAGED_MAGIC && !h.bad && h.n_seq == p.g.n_seq && h.H == p.g.H && h.Hkv == p.g.Hkv &&
           h.block == p.g.block && h.Tq == p.g.Tq && h.page == p.page && h.n_pages == p.n_pages &&
           h.max_pages == p.max_pages && h.n_groups == p.n_groups;
}

}  // namespace k6
