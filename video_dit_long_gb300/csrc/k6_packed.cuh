// k6_packed.cuh -- the plan of a batch of packed sequences: what the plan kernel
// writes and the attention kernels read, and the mask they share.
//
// Mask.  Query token i (of Lq) of a sequence sits at key position
// i + Lk - Lq (the queries are the newest tokens) and sees the keys j < limit:
//   block == 0: limit = Lk;
//   block == F: limit = clip((floor((i + Lk - Lq) / F) + 1) F, 0, Lk),
// F = 1 causal, F > 1 causal by frames of F tokens.  The limit never falls with
// i, so a tile of query tokens needs the key tiles below its last token's
// limit, and key j is seen by the query tokens i >= floor(j / F) F - (Lk - Lq).
#pragma once

#include <cuda_runtime.h>

#include "k6_internal.h"

namespace k6 {

constexpr unsigned PACKED_MAGIC = 0x6b36504cu;

struct PackedHeader {
    unsigned magic;
    int n_seq, H, Hkv, block, Tq, Tk;  // what the plan was made for
    int n_fwd, n_merge, n_q, n_k;      // items in each list
    int stream;                        // forward items laid out per CTA (count[]), or one list for every key head
    int slot_step;                     // partials of a split tile lie this far apart
    int q_lo, q_hi, k_lo, k_hi;        // token rows that belong to a sequence
    int bad;                           // the offsets are not ascending within the tokens: no list is valid
};
constexpr size_t PACKED_HEADER_BYTES = 256;
static_assert(sizeof(PackedHeader) <= PACKED_HEADER_BYTES, "plan header");

// One tile of query tokens over key tiles [kt0, kt1) of its sequence.
struct __align__(16) PackedItem {
    int tok0;          // first token row of q
    int n_tok_hk;      // tokens (1 .. tpt) in the low 8 bits, and (forward, per CTA) the key head above them
    int krow0, Lk;     // the sequence's first row of k, and its keys
    int pos0;          // key position of token tok0
    int kt0, kt1;
    int slot;          // partial output, or -1: the item covers all of its tile's keys
};
// One tile of 128 keys over query tiles [qt0, qt1) of its sequence.
struct __align__(16) PackedKItem {
    int krow0, n_key;  // first row of k, keys (1 .. 128)
    int key0;          // position of the first key in its sequence
    int qrow0, Lq;     // the sequence's first row of q, and its queries
    int off;           // Lk - Lq
    int qt0, qt1;
};
// The n partials of a split tile of one key head, from slot0 on, slot_step apart.
struct __align__(16) PackedMerge {
    int tok0, n_tok_hk, slot0, n;
};

struct PackedPlan {
    PackedHeader *head;
    int *count;         // [sms]: forward items of each CTA
    PackedMerge *merge; // [packed_merge_rows]
    PackedItem *fwd;    // [sms][cap_rows] items of each CTA, or [cap_q + extra] for every key head, heaviest first
    int *sched;         // sorted list: [round][sms] the (key head * n_fwd + item) of each CTA, or -1
    PackedItem *q;      // [cap_q], unsplit (backward), heaviest first
    PackedKItem *k;     // [cap_k], heaviest first
};

// Split tiles a plan has room for: one per SM at least, whatever the batch.
static inline __host__ __device__ int packed_merge_rows(const PackedGeom &p) {
    return p.cap_merge > p.sms ? p.cap_merge : p.sms;
}

// The start of every plan on a GPU of `sms` SMs, of any batch: the header, the
// CTAs' counts and the first `sms` split tiles.  A kernel may read this much, and
// no more, before the header has told it that the plan is its batch's: the lists
// behind it lie where the batch's sizes put them, and a plan of a smaller batch
// ends before a larger one's.
static inline __host__ __device__ size_t packed_plan_common_bytes(int sms) {
    return PACKED_HEADER_BYTES + ((size_t)sms * sizeof(int) + 15) / 16 * 16 + (size_t)sms * sizeof(PackedMerge);
}

static inline __host__ __device__ PackedPlan packed_plan_at(void *base, const PackedGeom &p) {
    PackedPlan r;
    char *b = static_cast<char *>(base);
    r.head = reinterpret_cast<PackedHeader *>(b);
    b += PACKED_HEADER_BYTES;
    r.count = reinterpret_cast<int *>(b);
    b += ((size_t)p.sms * sizeof(int) + 15) / 16 * 16;
    r.merge = reinterpret_cast<PackedMerge *>(b);
    b += (size_t)packed_merge_rows(p) * sizeof(PackedMerge);
    r.fwd = reinterpret_cast<PackedItem *>(b);
    b += (size_t)p.cap_fwd * sizeof(PackedItem);
    r.sched = reinterpret_cast<int *>(b);
    b += ((size_t)p.cap_sched * sizeof(int) + 15) / 16 * 16;
    r.q = reinterpret_cast<PackedItem *>(b);
    b += (size_t)p.cap_q * sizeof(PackedItem);
    r.k = reinterpret_cast<PackedKItem *>(b);
    return r;
}

// True if the plan was made for this batch and holds valid lists.
static inline __device__ bool packed_plan_ok(const PackedHeader &h, const PackedGeom &p) {
    return h.magic == PACKED_MAGIC && !h.bad && h.n_seq == p.n_seq && h.H == p.H && h.Hkv == p.Hkv &&
           h.block == p.block && h.Tq == p.Tq && h.Tk == p.Tk;
}

// Keys that the token at key position `pos` sees (pos may be negative: none).
// The host keeps block and Lk below 2^30, so the product stays below 2^31.
static inline __device__ int packed_limit(int pos, int Lk, int block) {
    if (block == 0) return Lk;
    if (pos < 0) return 0;
    return min(Lk, (pos / block + 1) * block);
}

// The first query token that sees key `key`.
static inline __device__ int packed_first_query(int key, int off, int block) {
    if (block == 0) return 0;
    return max(0, key / block * block - off);
}

}  // namespace k6
