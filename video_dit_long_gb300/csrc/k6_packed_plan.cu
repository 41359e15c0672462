// k6_packed_plan.cu -- lays out the work of packed attention on the device, once
// per batch.  The offsets stay on the device, so a batch can be planned inside a
// captured graph; a layer stack reuses the plan.
//
// Three blocks, one list each: forward items, unsplit query tiles (backward dq)
// and key tiles (backward dk/dv).  Warps stride over sequences, lanes over a
// sequence's tiles.
//
// Forward, up to STREAM_MOST key tiles per SM: every unit (a query tile of one
// key head) costs its key tiles plus ITEM_COST; the units of the batch, end to
// end, are cut into one stretch per SM, so that all SMs finish together
// whatever the lengths: a stretch may begin or end inside a unit, whose
// partials are then joined.  A cut that would leave a piece of less than
// MIN_PIECE tiles moves to the unit's border.  Larger batches: one list of
// query tiles per key head, heaviest first (a counting sort by work), dealt out
// in rounds of one unit per SM, one head after another, so that CTAs running
// together share a head's K and V in L2; in each round the heaviest unit goes to
// the SM with the least work so far (25,920 tokens by frames, 24/8 heads: loads
// within 0.7 % of the mean; dealt out to and fro, 11 %).  Only units longer than
// the SMs' share are cut.  The other two lists are sorted alike; their items are
// blocks, which the hardware hands out.
//
// 6-38 us for a dozen sequences, once per batch, whatever the layers.  It grows
// with the units: the dealing takes 118 us for 25,920 tokens by frames, 24/8
// heads (33 rounds of the SMs' units) and 191 us for 52,360 tokens, 24/24 heads (65);
// 1,000 sequences of 5 tokens, 8 key heads, take 114 us cut into stretches, and
// 10,000, which are dealt out however short they are (526 rounds), 2.3 ms.
//
// The order inside a class of equal work, and so which SM runs an item and
// which slot holds a partial, may differ between runs; every item writes rows
// of its own and partials are joined in key order, so results do not.
//
// Streams over a cache of pages (k6_paged.cuh) are planned by the same code, from
// units of tiles that the kernel first makes of the streams and of the groups that
// share a prefix: 8-17 us for steps of up to 32 streams.
#include "k6_paged.cuh"

namespace k6 {

constexpr int MIN_PIECE = 4;       // key tiles of a piece at least
constexpr int ITEM_COST = 2;       // start and end of an item in key tiles: 1.6 us against 0.7 us a tile
constexpr int STREAM_MOST = 256;   // cost per SM up to which the batch is cut into one stretch per SM
constexpr int STREAM_SEQS = 1024;  // and sequences
// Over pages, where new tokens are few and joins are by rows: measured in a captured graph, us, pieces of 4 and of 2 at
// least, new tokens over shared prompts 18.1 and 17.3, two streams' next frame 67.8 and 66.8, a mixed step 35.5 and 34.9.
constexpr int PAGED_PIECE = 2;
// An item of few rows has tiles that wait for HBM, beside which its start costs less: 1 against 2 took 32 tokens over a
// shared prefix from 37.7 to 36.7 us, a mixed step from 34.0 to 33.5, 12 tokens over long caches from 48.3 to 48.6.
constexpr int FEW_ROWS = 64, FEW_ROWS_ITEM = 1;
constexpr int SHARE_LEAST = 8;     // key tiles that a shared prefix saves at least

PackedGeom packed_geom(const Geom &g, const k6attn_packed &b, int sms) {
    PackedGeom p;
    p.n_seq = b.n_seq;
    p.H = g.H, p.Hkv = b.kv_heads, p.G = g.H / b.kv_heads, p.block = b.mask_block;
    p.Tq = (int)b.q_tokens, p.Tk = (int)b.k_tokens;
    p.tpt = 128 / p.G;
    p.rows = p.tpt * p.G;
    // sum of ceil(L / n) <= floor(T / n) + sequences
    p.cap_q = p.Tq / p.tpt + p.n_seq;
    p.cap_k = p.Tk / 128 + p.n_seq;
    p.sms = sms;
    // both pieces of a cut have MIN_PIECE tiles: nothing to cut below twice that
    p.extra = p.Tk > (2 * MIN_PIECE - 1) * 128 ? (sms + p.Hkv - 1) / p.Hkv : 0;
    // one cut per SM at most; or, per key head, n < 2 tiles / chunk pieces of each unit longer than chunk
    p.cap_slots = p.extra ? 2 * (p.extra * p.Hkv > sms ? p.extra * p.Hkv : sms) : 0;
    p.cap_merge = p.cap_slots / 2;
    // a stretch of cost q, after its ends moved by MIN_PIECE + ITEM_COST at most, holds units of cost > ITEM_COST
    const long most = ((long)p.cap_q * p.Hkv * ((p.Tk + 127) / 128 + 1 + ITEM_COST) + sms - 1) / sms;
    p.cap_rows = (int)(most < STREAM_MOST ? most : STREAM_MOST) / (ITEM_COST + 1) + 8;
    const long list = (long)p.cap_q + p.extra, rows = (long)sms * p.cap_rows;
    p.cap_fwd = (int)(list > rows ? list : rows);
    // batches that surely are cut into stretches need no schedule
    p.cap_sched = most <= STREAM_MOST && p.n_seq <= STREAM_SEQS ? 0 : (list * p.Hkv + sms - 1) / sms * sms;
    return p;
}

PagedGeom paged_geom(const Geom &g, const k6attn_paged &b, int sms) {
    PagedGeom r;
    paged_set_page(r, b.page_tokens);
    r.n_pages = (int)b.n_pages, r.max_pages = b.max_pages, r.n_groups = b.n_groups;
    PackedGeom &p = r.g;
    p.n_seq = b.n_seq;
    p.H = g.H, p.Hkv = b.kv_heads, p.G = g.H / b.kv_heads, p.block = b.mask_block;
    p.Tq = (int)b.q_tokens, p.Tk = b.max_pages * b.page_tokens;
    p.tpt = 128 / p.G;
    p.rows = p.tpt * p.G;
    p.sms = sms;
    // a group is taken together only where that halves its query tiles: at most two of each stream's, half of that
    // over the shared keys
    r.cap_prefix = b.n_groups > 0 ? b.n_seq : 0;
    const long own = (long)p.Tq / p.tpt + b.n_seq, joined = b.n_groups > 0 ? (own < 2L * b.n_seq ? own : 2L * b.n_seq) : 0;
    p.cap_q = (int)own + r.cap_prefix;
    p.cap_k = 0;
    p.extra = p.Tk > (2 * PAGED_PIECE - 1) * 128 ? (sms + p.Hkv - 1) / p.Hkv : 0;
    p.cap_slots = p.extra ? 2 * (p.extra * p.Hkv > sms ? p.extra * p.Hkv : sms) : 0;
    // joins of MERGE_ROWS rows: of whole tiles that are cut, and of every row that a group may share
    const long joined_rows = joined * p.rows < (long)p.Tq * p.G ? joined * p.rows : (long)p.Tq * p.G;
    p.cap_merge = (int)((long)p.cap_slots / 2 * ((p.rows + MERGE_ROWS - 1) / MERGE_ROWS) +
                        (joined_rows / MERGE_ROWS + joined) * p.Hkv);
    const long rows = (long)p.Tq * p.H, own_rows = joined * p.Hkv * p.rows, prefix_rows = (long)r.cap_prefix * p.Hkv * p.rows;
    r.cap_part = (long)p.cap_slots * p.rows + (own_rows < rows ? own_rows : rows) + (prefix_rows < rows ? prefix_rows : rows);
    const long most = ((long)p.cap_q * p.Hkv * ((p.Tk + 127L) / 128 + 1 + ITEM_COST) + sms - 1) / sms;
    p.cap_rows = (int)(most < STREAM_MOST ? most : STREAM_MOST) / (FEW_ROWS_ITEM + 1) + 8;
    const long list = (long)p.cap_q + p.extra, all = (long)sms * p.cap_rows;
    p.cap_fwd = (int)(list > all ? list : all);
    p.cap_sched = most <= STREAM_MOST && p.n_seq + b.n_groups <= STREAM_SEQS ? 0 : (list * p.Hkv + sms - 1) / sms * sms;
    return r;
}

size_t paged_plan_bytes(const PagedGeom &p) {
    return reinterpret_cast<size_t>(paged_plan_at(nullptr, p).slot) + (size_t)p.g.Tq * sizeof(int);
}

size_t packed_plan_bytes(const PackedGeom &p) {
    const PackedPlan at = packed_plan_at(nullptr, p);
    return reinterpret_cast<size_t>(at.k) + (size_t)p.cap_k * sizeof(PackedKItem);
}

namespace {

constexpr int THREADS = 1024, WARPS = THREADS / 32, CLASSES = 256, MAX_SMS = 512;

enum List { FWD, QTILES, KTILES };

struct Seq {
    int q0, Lq, k0, Lk, tiles;
    int lo;            // first key tile
    bool parts;        // its rows are joined with others': partials, whether cut or not
    bool seen;         // every key is seen by every row, whatever the mask
    int prefix, group_q0;
};

// What the lists are made of.  Batch: packed sequences.
struct Batch {
    static constexpr int PIECE = MIN_PIECE;
    static constexpr bool CAPACITY = false;  // Tk is the batch's keys
    __device__ __forceinline__ static int item_cost(const PackedGeom &, const Seq &, int) { return ITEM_COST; }
    const int *cu_q, *cu_k;
    PackedPlan plan;
    int n;
    template <List LIST>
    __device__ __forceinline__ Seq sequence(const PackedGeom &p, int s) const {
        Seq r;
        r.q0 = cu_q[s], r.Lq = cu_q[s + 1] - r.q0;
        r.k0 = cu_k[s], r.Lk = cu_k[s + 1] - r.k0;
        r.tiles = LIST == KTILES ? (r.Lk + 127) / 128 : (r.Lq + p.tpt - 1) / p.tpt;
        r.lo = 0, r.parts = r.seen = false, r.prefix = r.group_q0 = -1;
        return r;
    }
    // Room for the n partials of a tile, of every key head from hk0 on up to hk1, and its joins: the first one's slot,
    // and how far the next piece's lies behind it.
    __device__ __forceinline__ int partials(const PackedGeom &p, int &slots, int &merges, const Seq &, int, int tok0,
                                            int n_tok, int hk0, int hk1, int n, int &step) const {
        const int heads = hk1 - hk0, slot = atomicAdd(&slots, n), m = atomicAdd(&merges, heads);
        for (int h = 0; h < heads; h++)
            if (m + h < p.cap_merge) plan.merge[m + h] = {tok0, n_tok | (hk0 + h) << 8, slot * heads + h, n};
        step = 1;
        return slot;
    }
    __device__ __forceinline__ bool full(const PackedGeom &p, int slots, int heads) const {
        return (long)slots * heads > p.cap_slots;
    }
};

// Pages: units of tiles; those behind the streams' own are over shared keys.  A slot is a row of the partials.
struct PagedBatch {
    static constexpr int PIECE = PAGED_PIECE;
    static constexpr bool CAPACITY = true;  // Tk is the most that a stream's table has room for
    __device__ __forceinline__ static int item_cost(const PackedGeom &p, const Seq &s, int t) {
        return min(p.tpt, s.Lq - t * p.tpt) * p.G <= FEW_ROWS ? FEW_ROWS_ITEM : ITEM_COST;
    }
    PagedPlan plan;
    int n, n_seq, cap_prefix;
    long cap_part;
    template <List LIST>
    __device__ __forceinline__ Seq sequence(const PackedGeom &, int s) const {
        const PagedUnits u = plan.units[s];
        Seq r;
        r.q0 = u.q0, r.Lq = u.Lq, r.k0 = u.row, r.Lk = u.Lk, r.tiles = u.tiles, r.lo = u.lo;
        r.parts = u.prefix >= 0, r.seen = s >= n_seq;
        r.prefix = u.prefix, r.group_q0 = u.group_q0;
        return r;
    }
    __device__ __forceinline__ int partials(const PackedGeom &p, int &slots, int &merges, const Seq &s, int t, int tok0,
                                            int n_tok, int hk0, int hk1, int n, int &step) const {
        const int rows = n_tok * p.G, heads = hk1 - hk0;
        step = rows * heads;
        const int slot = n > 0 ? atomicAdd(&slots, n * step) : 0;
        const int per_head = (rows + MERGE_ROWS - 1) / MERGE_ROWS;
        int m = s.seen ? 0 : atomicAdd(&merges, heads * per_head);
        for (int h = 0; h < heads; h++) {
            const int row = slot + h * rows;
            if (s.seen) plan.prefix[(long)(hk0 + h) * cap_prefix + s.prefix + t] = {row, n, step, 0};
            else
                for (int r0 = 0; r0 < rows; r0 += MERGE_ROWS, m++)
                    if (m < p.cap_merge) 
                        plan.merge[m] = {tok0, n_tok | (hk0 + h) << 8, s.prefix, s.group_q0, row, n, step, r0, {0, 0, 0, 0}};
        }
        return slot;
    }
    __device__ __forceinline__ bool full(const PackedGeom &, int slots, int) const { return slots > cap_part; }
};

// Key position of a tile's first token; beyond every key where all of them are seen.
__device__ __forceinline__ int first_pos(const PackedGeom &p, const Seq &s, int t) {
    return s.seen ? 1 << 29 : t * p.tpt + s.Lk - s.Lq;
}

// Tiles of the other side that tile t of the sequence meets: [lo, hi).
template <List LIST>
__device__ __forceinline__ void range(const PackedGeom &p, const Seq &s, int t, int &lo, int &hi) {
    if (LIST == KTILES) {
        lo = packed_first_query(t * 128, s.Lk - s.Lq, p.block) / p.tpt;
        hi = (s.Lq + p.tpt - 1) / p.tpt;
        if (lo > hi) lo = hi;
    } else {
        const int last = min((t + 1) * p.tpt, s.Lq) - 1;
        lo = s.lo;
        hi = s.seen ? s.Lk / 128 : (packed_limit(last + s.Lk - s.Lq, s.Lk, p.block) + 127) / 128;
        if (hi < lo) hi = lo;
    }
}

__device__ __forceinline__ int work_class(int work, int most) {
    return min(CLASSES - 1, (int)((long)work * CLASSES / (most + 1)));
}

struct Shared {
    int count[CLASSES];
    int at[CLASSES];
    int bad, total;
    unsigned long long work;
    int top;           // the largest unit's
    int slots, merges;
    // stretches: first unit and item count of each CTA; cost and tiles of the sequences before each one
    int first[MAX_SMS], items[MAX_SMS];
    int cost[STREAM_SEQS + 1], tiles[STREAM_SEQS + 1];
    int warp_sum[WARPS];
    // dealing out: each SM's load, a round's works, the ranks of both, and both by rank
    int load[MAX_SMS], work_of[MAX_SMS], rank[2][MAX_SMS], sm_at[MAX_SMS], unit_at[MAX_SMS];
};

// The schedule of n items for every key head (see the head of this file).
template <class Plan>
__device__ void deal(const PackedGeom &p, const Plan &plan, Shared &sh, int n) {
    const long units = (long)n * p.Hkv;
    // half the threads rank each side; as many as fit share one entry's comparisons
    const int side = threadIdx.x / (THREADS / 2), x = threadIdx.x % (THREADS / 2);
    const int shares = THREADS / 2 / p.sms, i = x % p.sms, share = x / p.sms;
    const bool one = side == 0 && x < p.sms;  // a thread for each SM
    if (one) sh.load[i] = 0;
    // the work of unit base + i, read a round ahead; item: its place among those of a key head
    int item = n > 0 ? i % n : 0;
    auto work = [&](long u) {
        if (!one || u >= units) return 0;
        const PackedItem &it = plan.fwd[item];
        const int w = it.kt1 - it.kt0 + ITEM_COST;
        for (item += p.sms; item >= n;) item -= n;
        return w;
    };
    int next = work(i);
    for (long base = 0; base < units; base += p.sms) {
        if (one) {
            sh.work_of[i] = next;
            sh.rank[0][i] = sh.rank[1][i] = 0;
        }
        next = work(base + p.sms + i);
        __syncthreads();
        if (share < shares) {
            const int j0 = (int)((long)p.sms * share / shares), j1 = (int)((long)p.sms * (share + 1) / shares);
            int rank = 0;
            if (side == 0) {  // the least loaded SM first
                const int mine = sh.load[i];
                for (int j = j0; j < j1; j++) rank += sh.load[j] < mine || (sh.load[j] == mine && j < i);
            } else {  // the heaviest unit first
                const int mine = sh.work_of[i];
                for (int j = j0; j < j1; j++) rank += sh.work_of[j] > mine || (sh.work_of[j] == mine && j < i);
            }
            atomicAdd(&sh.rank[side][i], rank);
        }
        __syncthreads();
        if (one) sh.sm_at[sh.rank[0][i]] = i, sh.unit_at[sh.rank[1][i]] = i;
        __syncthreads();
        if (one) {
            const int sm = sh.sm_at[i], u = sh.unit_at[i];
            plan.sched[base + sm] = base + u < units ? (int)(base + u) : -1;
            sh.load[sm] += sh.work_of[u];
        }
        __syncthreads();
    }
}

template <List LIST, class B>
__device__ void build(const PackedGeom &p, const B &b, Shared &sh) {
    const auto &plan = b.plan;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    // a warp to a sequence; with fewer sequences than warps all threads to each
    const bool few = b.n < WARPS;
    const int s0 = few ? 0 : warp, ds = few ? 1 : WARPS, t0 = few ? (int)threadIdx.x : lane, dt = few ? THREADS : 32;
    int most = LIST == KTILES ? (p.Tq + p.tpt - 1) / p.tpt : (p.Tk + 127) / 128;
    int chunk = 1 << 30;
    if (LIST == FWD && p.extra > 0) {
        // key tiles per item: the batch's work over the items aimed at
        unsigned long long w = 0;
        int top = 1;
        for (int s = s0; s < b.n; s += ds) {
            const Seq q = b.template sequence<LIST>(p, s);
            for (int t = t0; t < q.tiles; t += dt) {
                int lo, hi;
                range<LIST>(p, q, t, lo, hi);
                w += hi - lo;
                top = max(top, hi - lo);
            }
        }
        atomicAdd(&sh.work, w);
        atomicMax(&sh.top, top);
        __syncthreads();
        if (B::CAPACITY) most = sh.top;  // the classes then span what there is, not what there may be
        // extra * chunk >= work, so that the pieces beyond one per tile number at most extra
        const unsigned long long c = (sh.work + p.extra - 1) / p.extra;
        chunk = c < (1u << 30) ? max(2 * B::PIECE, (int)c) : 1 << 30;
    }
    for (int s = s0; s < b.n; s += ds) {
        const Seq q = b.template sequence<LIST>(p, s);
        for (int t = t0; t < q.tiles; t += dt) {
            int lo, hi;
            range<LIST>(p, q, t, lo, hi);
            const int n = max(1, (hi - lo + chunk - 1) / chunk);
            atomicAdd(&sh.count[work_class((hi - lo) / n, most)], n);
        }
    }
    __syncthreads();
    if (warp == 0) {  // exclusive sums from the heaviest class down: lane l holds classes 255 - 8l .. 248 - 8l
        int mine = 0;
        for (int i = 0; i < CLASSES / 32; i++) mine += sh.count[CLASSES - 1 - (lane * (CLASSES / 32) + i)];
        int upto = mine;
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
        int at = upto - mine;
        for (int i = 0; i < CLASSES / 32; i++) {
            const int c = CLASSES - 1 - (lane * (CLASSES / 32) + i);
            sh.at[c] = at;
            at += sh.count[c];
        }
        if (lane == 31) sh.total = at;
    }
    __syncthreads();
    if (LIST == FWD && sh.total > p.cap_q + p.extra) {  // the same for all threads
        if (threadIdx.x == 0) sh.bad = 1;
        return;
    }
    for (int s = s0; s < b.n; s += ds) {
        const Seq q = b.template sequence<LIST>(p, s);
        for (int t = t0; t < q.tiles; t += dt) {
            int lo, hi;
            range<LIST>(p, q, t, lo, hi);
            if constexpr (LIST == KTILES) {
                PackedKItem it;
                it.krow0 = q.k0 + t * 128;
                it.key0 = t * 128;
                it.n_key = min(128, q.Lk - t * 128);
                it.qrow0 = q.q0, it.Lq = q.Lq, it.off = q.Lk - q.Lq;
                it.qt0 = lo, it.qt1 = hi;
                plan.k[atomicAdd(&sh.at[work_class(hi - lo, most)], 1)] = it;
                continue;
            }
            const int n = max(1, (hi - lo + chunk - 1) / chunk);
            int i = atomicAdd(&sh.at[work_class((hi - lo) / n, most)], n);
            PackedItem it;
            it.tok0 = q.q0 + t * p.tpt;
            it.n_tok_hk = min(p.tpt, q.Lq - t * p.tpt);
            it.krow0 = q.k0, it.Lk = q.Lk;
            it.pos0 = first_pos(p, q, t);
            int slot = -1, step = 0;
            const bool parts = n > 1 || (q.parts && hi > lo);
            if (parts || q.parts)
                slot = b.partials(p, sh.slots, sh.merges, q, t, it.tok0, it.n_tok_hk, 0, p.Hkv, parts ? n : 0, step);
            for (int c = 0; c < n; c++, i++) {  // pieces of equal length, to within a tile
                it.kt0 = lo + (int)((long)(hi - lo) * c / n), it.kt1 = lo + (int)((long)(hi - lo) * (c + 1) / n);
                it.slot = parts ? slot + c * step : -1;
                if constexpr (LIST == FWD) plan.fwd[i] = it;
                else plan.q[i] = it;
            }
        }
    }
    __syncthreads();
    if (LIST == FWD) deal(p, plan, sh, sh.total);
    if (threadIdx.x == 0) {
        if (LIST == FWD) {
            plan.head->n_fwd = sh.total, plan.head->n_merge = sh.merges;
            plan.head->stream = 0, plan.head->slot_step = p.Hkv;
            if (b.full(p, sh.slots, p.Hkv) || sh.merges > p.cap_merge) sh.bad = 1;
        } else if (LIST == QTILES) {
            plan.head->n_q = sh.total;
        } else {
            plan.head->n_k = sh.total;
        }
    }
}

// The batch cut into one stretch per SM.  False (the same for all threads): too
// large, nothing was written.
template <class B>
__device__ bool build_stretches(const PackedGeom &p, const B &b, Shared &sh) {
    const auto &plan = b.plan;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (b.n > STREAM_SEQS) return false;
    // cost and tiles of each sequence, then of those before it
    unsigned long long all = 0;
    for (int s = warp; s < b.n; s += WARPS) {
        const Seq q = b.template sequence<FWD>(p, s);
        unsigned long long c = 0;
        for (int t = lane; t < q.tiles; t += 32) {
            int lo, hi;
            range<FWD>(p, q, t, lo, hi);
            c += max(hi - lo, 1) + b.item_cost(p, q, t);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
        all += c;
        if (lane == 0) {  // a sum beyond the limit below is never used
            sh.cost[s] = (int)(c < (1ull << 30) ? c : 1ull << 30);
            sh.tiles[s] = q.tiles;
        }
    }
    if (lane == 0) atomicAdd(&sh.work, all);
    __syncthreads();
    const unsigned long long total = sh.work * (unsigned long long)p.Hkv;
    __syncthreads();
    if (threadIdx.x == 0) sh.work = 0;  // the sorted list counts anew
    if (total > (unsigned long long)p.sms * STREAM_MOST) {
        __syncthreads();
        return false;
    }
    {  // exclusive sums over the sequences: one thread each (STREAM_SEQS threads)
        const int s = threadIdx.x;
        const int c = s < b.n ? sh.cost[s] : 0, n = s < b.n ? sh.tiles[s] : 0;
        for (int pass = 0; pass < 2; pass++) {
            const int mine = pass ? n : c;
            int upto = mine;
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += v;
            }
            if (lane == 31) sh.warp_sum[warp] = upto;
            __syncthreads();
            int before = 0;
            for (int w = 0; w < warp; w++) before += sh.warp_sum[w];
            (pass ? sh.tiles : sh.cost)[s] = before + upto - mine;
            if (s == THREADS - 1) (pass ? sh.tiles : sh.cost)[STREAM_SEQS] = before + upto;
            __syncthreads();
        }
    }
    const int head_cost = sh.cost[STREAM_SEQS], head_tiles = sh.tiles[STREAM_SEQS];  // of one key head
    const int Q = max(1, ((int)total + p.sms - 1) / p.sms);
    for (int c = threadIdx.x; c < p.sms; c += THREADS) sh.first[c] = 1 << 30, sh.items[c] = 0;
    __syncthreads();
    // pass 0: the unit that each stretch begins with; pass 1: the items
    for (int pass = 0; pass < 2; pass++) {
        for (int s = warp; s < b.n; s += WARPS) {
            const Seq q = b.template sequence<FWD>(p, s);
            int run = sh.cost[s];
            for (int t0 = 0; t0 < q.tiles; t0 += 32) {
                int tile_lo = 0, tile_work = 0, tile_cost = 0;
                if (t0 + lane < q.tiles) {
                    range<FWD>(p, q, t0 + lane, tile_lo, tile_work);
                    tile_work -= tile_lo;
                    tile_cost = max(tile_work, 1) + b.item_cost(p, q, t0 + lane);
                }
                int upto = tile_cost;
                for (int o = 1; o < 32; o <<= 1) {
                    const int v = __shfl_up_sync(0xffffffffu, upto, o);
                    if (lane >= o) upto += v;
                }
                const int tile_at = run + upto - tile_cost;
                run += __shfl_sync(0xffffffffu, upto, 31);
                // the units of these tiles and every key head, one a lane
                const int units = min(32, q.tiles - t0) * p.Hkv;
                for (int u0 = 0; u0 < units; u0 += 32) {
                    const int u = min(u0 + lane, units - 1), src = u / p.Hkv, hk = u - src * p.Hkv, t = t0 + src;
                    const int at = __shfl_sync(0xffffffffu, tile_at, src), cost = __shfl_sync(0xffffffffu, tile_cost, src);
                    const int lo = __shfl_sync(0xffffffffu, tile_lo, src), work = __shfl_sync(0xffffffffu, tile_work, src);
                    if (u0 + lane >= units) continue;
                    const int start = b.item_cost(p, q, t);
                    const int a = hk * head_cost + at, z = a + cost, unit = hk * head_tiles + sh.tiles[s] + t;
                    const int c0 = (a + Q - 1) / Q, c1 = min(p.sms, (z + Q - 1) / Q);  // borders in [a, z): [c0, c1)
                    // tile at which border c cuts the unit, moved to its ends where a piece would be too short (and
                    // to multiples of that least piece where the borders are closer)
                    auto cut = [&](int c) {
                        int x = max(0, c * Q - a - start);
                        if (Q < B::PIECE) x -= x % B::PIECE;
                        return x < B::PIECE ? 0 : work - x < B::PIECE ? work : x;
                    };
                    if (pass == 0) {
                        for (int c = c0; c < c1; c++) sh.first[c] = unit + (cut(c) >= max(work, 1) ? 1 : 0);
                        continue;
                    }
                    int n = 1;
                    for (int c = c0, from = 0; c < c1; c++) {
                        const int x = cut(c);
                        if (x > from && x < work) n++, from = x;
                    }
                    PackedItem it;
                    it.tok0 = q.q0 + t * p.tpt;
                    it.n_tok_hk = min(p.tpt, q.Lq - t * p.tpt) | hk << 8;
                    it.krow0 = q.k0, it.Lk = q.Lk;
                    it.pos0 = first_pos(p, q, t);
                    int slot = -1, step = 0;
                    const bool parts = n > 1 || (q.parts && work > 0);
                    if (parts || q.parts)
                        slot = b.partials(p, sh.slots, sh.merges, q, t, it.tok0, it.n_tok_hk & 255, hk, hk + 1,
                                          parts ? n : 0, step);
                    int from = 0, piece = 0, owner = min(p.sms - 1, a / Q);
                    for (int c = c0; c <= c1; c++) {
                        const int x = c < c1 ? cut(c) : work;
                        if (c < c1 && x >= work && work > 0) continue;  // begins with the next unit
                        if (c < c1 && x == from) {  // the stretch before it ends here
                            owner = c;
                            continue;
                        }
                        // the piece [from, x) belongs to `owner`; the border c begins the next one
                        const int k = unit - sh.first[owner];
                        it.kt0 = lo + from, it.kt1 = lo + x;
                        it.slot = parts ? slot + piece * step : -1;
                        if (k >= 0 && k < p.cap_rows) {
                            plan.fwd[(long)owner * p.cap_rows + k] = it;
                            atomicMax(&sh.items[owner], k + 1);
                        } else {
                            sh.bad = 1;
                        }
                        from = x, piece++, owner = c;
                    }
                }
            }
        }
        __syncthreads();
    }
    for (int c = threadIdx.x; c < p.sms; c += THREADS) plan.count[c] = sh.items[c];
    if (threadIdx.x == 0) {
        plan.head->n_fwd = 0, plan.head->n_merge = sh.merges;
        plan.head->stream = 1, plan.head->slot_step = 1;
        if (b.full(p, sh.slots, 1) || sh.merges > p.cap_merge) sh.bad = 1;
    }
    return true;
}

__global__ void __launch_bounds__(THREADS) packed_plan_kernel(const PackedGeom p, const int *__restrict__ cu_q,
                                                              const int *__restrict__ cu_k, void *base, int *err) {
    __shared__ Shared sh;
    const PackedPlan plan = packed_plan_at(base, p);
    if (threadIdx.x < CLASSES) sh.count[threadIdx.x] = 0;
    if (threadIdx.x == 0) {
        sh.work = 0;
        sh.top = 0;
        sh.slots = sh.merges = 0;
        sh.bad = cu_q[0] < 0 || cu_k[0] < 0 || cu_q[p.n_seq] > p.Tq || cu_k[p.n_seq] > p.Tk;
    }
    __syncthreads();
    for (int s = threadIdx.x; s < p.n_seq; s += THREADS)
        if (cu_q[s + 1] < cu_q[s] || cu_k[s + 1] < cu_k[s]) sh.bad = 1;
    __syncthreads();
    const bool bad = sh.bad;
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        PackedHeader *h = plan.head;
        h->magic = PACKED_MAGIC;
        h->n_seq = p.n_seq, h->H = p.H, h->Hkv = p.Hkv, h->block = p.block, h->Tq = p.Tq, h->Tk = p.Tk;
        h->q_lo = cu_q[0], h->q_hi = cu_q[p.n_seq], h->k_lo = cu_k[0], h->k_hi = cu_k[p.n_seq];
        h->bad = bad;
        if (bad) atomicCAS(err, DEV_OK, DEV_PLAN);
    }
    if (bad) return;
    const Batch b{cu_q, cu_k, plan, p.n_seq};
    if (blockIdx.x == 0) {
        if (!build_stretches(p, b, sh)) build<FWD>(p, b, sh);
        // work that found no room in the lists (their sizes are upper bounds, so there is none) makes the plan a bad
        // one: calls report it instead of leaving rows out
        __syncthreads();
        if (threadIdx.x == 0 && sh.bad) {
            plan.head->bad = 1;
            atomicCAS(err, DEV_OK, DEV_PLAN);
        }
    } else if (blockIdx.x == 1) build<QTILES>(p, b, sh);
    else build<KTILES>(p, b, sh);
}

// The units of a batch over pages: the streams' own keys, and a group's shared
// ones where taking its streams together at least halves its query tiles and saves
// SHARE_LEAST key tiles.
__device__ void paged_units(const PagedGeom &pg, const PagedPlan &plan, const int *cu_q, const int *k_lens,
                            const int *cu_groups, const int *shared, int *prefix_tiles) {
    const PackedGeom &p = pg.g;
    for (int s = threadIdx.x; s < p.n_seq; s += THREADS) {
        const int q0 = cu_q[s], Lq = cu_q[s + 1] - q0;
        plan.units[s] = {q0, Lq, k_lens[s], 0, s, (Lq + p.tpt - 1) / p.tpt, -1, 0};
    }
    __syncthreads();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    for (int g = warp; g < pg.n_groups; g += WARPS) {
        const int s0 = cu_groups[g], s1 = cu_groups[g + 1];
        int keys = shared[g], first = s1, tiles = 0;
        for (int s = s0 + lane; s < s1; s += 32) {
            const PagedUnits u = plan.units[s];
            if (u.Lq == 0) continue;
            keys = min(keys, packed_limit(u.Lk - u.Lq, u.Lk, p.block));  // what the stream's first query sees
            first = min(first, s);
            tiles += u.tiles;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            keys = min(keys, __shfl_xor_sync(0xffffffffu, keys, o));
            first = min(first, __shfl_xor_sync(0xffffffffu, first, o));
            tiles += __shfl_xor_sync(0xffffffffu, tiles, o);
        }
        const int q0 = cu_q[s0], Lq = cu_q[s1] - q0, together = (Lq + p.tpt - 1) / p.tpt, lo = keys / 128;
        bool use = lo > 0 && 2 * together <= tiles && (long)(tiles - together) * lo >= SHARE_LEAST;
        int at = 0;
        if (use && lane == 0) at = atomicAdd(prefix_tiles, together);
        at = __shfl_sync(0xffffffffu, at, 0);
        use = use && at + together <= pg.cap_prefix;
        if (lane == 0) plan.units[p.n_seq + g] = {q0, Lq, lo * 128, 0, first, use ? together : 0, at, q0};
        if (!use) continue;
        for (int s = s0 + lane; s < s1; s += 32) plan.units[s].lo = lo, plan.units[s].prefix = at, plan.units[s].group_q0 = q0;
    }
    __syncthreads();
}

// Block 0: the lists.  The others: where each new token's key lies.
__global__ void __launch_bounds__(THREADS) paged_plan_kernel(const PagedGeom pg, const int *__restrict__ cu_q,
                                                             const int *__restrict__ k_lens,
                                                             const int *__restrict__ table,
                                                             const int *__restrict__ cu_groups,
                                                             const int *__restrict__ shared, void *base, int *err) {
    const PackedGeom &p = pg.g;
    const PagedPlan plan = paged_plan_at(base, pg);
    if (blockIdx.x > 0) {
        for (int t = (blockIdx.x - 1) * THREADS + threadIdx.x; t < p.Tq; t += (gridDim.x - 1) * THREADS) {
            int s = 0, z = p.n_seq;  // the last stream that begins at t or before
            while (z - s > 1) {
                const int m = s + (z - s) / 2;
                if (cu_q[m] <= t) s = m;
                else z = m;
            }
            int slot = -1;
            const int end = cu_q[s + 1];
            const int pos = cu_q[s] <= t && t < end ? paged_position(pg, t, end, k_lens[s]) : -1;
            if (pos >= 0) {
                const int page = table[(long)s * pg.max_pages + pos / pg.page];
                if ((unsigned)page < (unsigned)pg.n_pages) slot = page * pg.page + pos % pg.page;
                else atomicCAS(err, DEV_OK, DEV_PLAN);
            }
            plan.slot[t] = slot;
        }
        return;
    }
    __shared__ Shared sh;
    __shared__ int prefix_tiles;
    if (threadIdx.x < CLASSES) sh.count[threadIdx.x] = 0;
    if (threadIdx.x == 0) {
        sh.work = 0;
        sh.top = 0;
        sh.slots = sh.merges = prefix_tiles = 0;
        sh.bad = cu_q[0] < 0 || cu_q[p.n_seq] > p.Tq;
        if (pg.n_groups > 0 && (cu_groups[0] < 0 || cu_groups[pg.n_groups] > p.n_seq)) sh.bad = 1;
    }
    __syncthreads();
    const int most = pg.n_pages > 0 ? p.Tk : 0;  // without pages there are no keys, and the calls have no map of them
    for (int s = threadIdx.x; s < p.n_seq; s += THREADS)
        if (cu_q[s + 1] < cu_q[s] || k_lens[s] < 0 || k_lens[s] > most) sh.bad = 1;
    for (int g = threadIdx.x; g < pg.n_groups; g += THREADS)
        if (cu_groups[g + 1] < cu_groups[g] || shared[g] < 0) sh.bad = 1;
    __syncthreads();
    const bool bad = sh.bad;
    if (threadIdx.x == 0) {
        PagedHeader *h = plan.head;
        h->magic = PAGED_MAGIC;
        h->n_seq = p.n_seq, h->H = p.H, h->Hkv = p.Hkv, h->block = p.block, h->Tq = p.Tq, h->Tk = p.Tk;
        h->q_lo = cu_q[0], h->q_hi = cu_q[p.n_seq], h->k_lo = h->k_hi = 0;
        h->n_q = h->n_k = 0;
        h->page = pg.page, h->n_pages = pg.n_pages, h->max_pages = pg.max_pages, h->n_groups = pg.n_groups;
        h->bad = bad;
        if (bad) atomicCAS(err, DEV_OK, DEV_PLAN);
    }
    if (bad) return;
    paged_units(pg, plan, cu_q, k_lens, cu_groups, shared, &prefix_tiles);
    const PagedBatch b{plan, p.n_seq + pg.n_groups, p.n_seq, pg.cap_prefix, pg.cap_part};
    const bool stretches = build_stretches(p, b, sh);
    if (!stretches) build<FWD>(p, b, sh);
    __syncthreads();
    if (threadIdx.x == 0 && sh.bad) {
        plan.head->bad = 1;
        atomicCAS(err, DEV_OK, DEV_PLAN);
    }
    for (int i = threadIdx.x; i < sh.merges && !sh.bad; i += THREADS) {
        PagedMerge &m = plan.merge[i];
        if (m.prefix < 0) continue;
        // the first and the last token of the rows, in the group's tiles
        const int n_tok = m.n_tok_hk & 255, at = m.tok0 - m.group_q0;
        const int a = (at + m.r0 / p.G) / p.tpt, z = (at + min(n_tok - 1, (m.r0 + MERGE_ROWS - 1) / p.G)) / p.tpt;
        if (a != z) continue;
        m.shared = plan.prefix[(long)(m.n_tok_hk >> 8) * pg.cap_prefix + m.prefix + a];
        m.shared.row += (at - a * p.tpt) * p.G;
        m.prefix = -1;
    }
    const int n = sh.total, per_sm = stretches ? 0 : (int)(((long)n * p.Hkv + p.sms - 1) / p.sms);
    for (int c = threadIdx.x; c < p.sms && !sh.bad; c += THREADS) {
        PackedItem it;
        it.kt0 = it.kt1 = it.n_tok_hk = 0;  // a CTA without one
        if (stretches) {
            if (plan.count[c] > 0) it = plan.fwd[(long)c * p.cap_rows];
        } else {
            const int u = per_sm > 0 ? plan.sched[c] : -1;
            if (u >= 0) it = plan.fwd[u % n], it.n_tok_hk |= u / n << 8;
        }
        plan.first[c] = it;
    }
}

}  // namespace

cudaError_t launch_paged_plan(const PagedGeom &p, const int *cu_q, const int *k_lens, const int *table,
                              const int *cu_groups, const int *shared, void *plan, int *err, cudaStream_t st) {
    const long blocks = ((long)p.g.Tq + THREADS - 1) / THREADS;
    paged_plan_kernel<<<(unsigned)(1 + (blocks < p.g.sms ? blocks : p.g.sms)), THREADS, 0, st>>>(
        p, cu_q, k_lens, table, cu_groups, shared, plan, err);
    return cudaGetLastError();
}

cudaError_t launch_packed_plan(const PackedGeom &p, const int *cu_q, const int *cu_k, void *plan, int *err,
                               cudaStream_t st) {
    packed_plan_kernel<<<3, THREADS, 0, st>>>(p, cu_q, cu_k, plan, err);
    return cudaGetLastError();
}

}  // namespace k6
