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
// 18-46 us for a dozen sequences, once per batch, whatever the layers.  It grows
// with the units: the dealing takes 131 us for 25,920 tokens by frames, 24/8
// heads (33 rounds of the SMs' units) and 203 us for 52,360 tokens, 24/24 heads (65);
// 1,000 sequences of 5 tokens, 8 key heads, take 351 us cut into stretches, and
// 10,000, which are dealt out however short they are (526 rounds), 2.4 ms.
//
// The order inside a class of equal work, and so which SM runs an item and
// which slot holds a partial, may differ between runs; every item writes rows
// of its own and partials are joined in key order, so results do not.
#include "k6_packed.cuh"

namespace k6 {

constexpr int MIN_PIECE = 4;       // key tiles of a piece at least
constexpr int ITEM_COST = 2;       // start and end of an item in key tiles: 1.6 us against 0.7 us a tile
constexpr int STREAM_MOST = 256;   // cost per SM up to which the batch is cut into one stretch per SM
constexpr int STREAM_SEQS = 1024;  // and sequences

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

size_t packed_plan_bytes(const PackedGeom &p) {
    const PackedPlan at = packed_plan_at(nullptr, p);
    return reinterpret_cast<size_t>(at.k) + (size_t)p.cap_k * sizeof(PackedKItem);
}

namespace {

constexpr int THREADS = 1024, WARPS = THREADS / 32, CLASSES = 256, MAX_SMS = 512;

enum List { FWD, QTILES, KTILES };

struct Seq {
    int q0, Lq, k0, Lk, tiles;
};

template <List LIST>
__device__ __forceinline__ Seq sequence(const PackedGeom &p, const int *cu_q, const int *cu_k, int s) {
    Seq r;
    r.q0 = cu_q[s], r.Lq = cu_q[s + 1] - r.q0;
    r.k0 = cu_k[s], r.Lk = cu_k[s + 1] - r.k0;
    r.tiles = LIST == KTILES ? (r.Lk + 127) / 128 : (r.Lq + p.tpt - 1) / p.tpt;
    return r;
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
        lo = 0;
        hi = (packed_limit(last + s.Lk - s.Lq, s.Lk, p.block) + 127) / 128;
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
    int slots, merges;
    // stretches: first unit and item count of each CTA; cost and tiles of the sequences before each one
    int first[MAX_SMS], items[MAX_SMS];
    int cost[STREAM_SEQS + 1], tiles[STREAM_SEQS + 1];
    int warp_sum[WARPS];
    // dealing out: each SM's load, a round's works, and both by rank
    int load[MAX_SMS], work_of[MAX_SMS], sm_at[MAX_SMS], unit_at[MAX_SMS];
};

// The schedule of n items for every key head (see the head of this file).
__device__ void deal(const PackedGeom &p, const PackedPlan &plan, Shared &sh, int n) {
    const long units = (long)n * p.Hkv;
    const int t = threadIdx.x, side = t / (THREADS / 2), i = t % (THREADS / 2);  // half the threads rank each side
    if (side == 0 && i < p.sms) sh.load[i] = 0;
    for (long base = 0; base < units; base += p.sms) {
        if (side == 0 && i < p.sms) {
            int w = 0;
            if (base + i < units) {
                const PackedItem &it = plan.fwd[(base + i) % n];
                w = it.kt1 - it.kt0 + ITEM_COST;
            }
            sh.work_of[i] = w;
        }
        __syncthreads();
        if (i < p.sms) {
            int rank = 0;
            if (side == 0) {  // the least loaded SM first
                const int mine = sh.load[i];
                for (int j = 0; j < p.sms; j++) rank += sh.load[j] < mine || (sh.load[j] == mine && j < i);
                sh.sm_at[rank] = i;
            } else {  // the heaviest unit first
                const int mine = sh.work_of[i];
                for (int j = 0; j < p.sms; j++) rank += sh.work_of[j] > mine || (sh.work_of[j] == mine && j < i);
                sh.unit_at[rank] = i;
            }
        }
        __syncthreads();
        if (side == 0 && i < p.sms) {
            const int sm = sh.sm_at[i], u = sh.unit_at[i];
            plan.sched[base + sm] = base + u < units ? (int)(base + u) : -1;
            sh.load[sm] += sh.work_of[u];
        }
        __syncthreads();
    }
}

template <List LIST>
__device__ void build(const PackedGeom &p, const int *cu_q, const int *cu_k, const PackedPlan &plan, Shared &sh) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int most = LIST == KTILES ? (p.Tq + p.tpt - 1) / p.tpt : (p.Tk + 127) / 128;
    int chunk = 1 << 30;
    if (LIST == FWD && p.extra > 0) {
        // key tiles per item: the batch's work over the items aimed at
        unsigned long long w = 0;
        for (int s = warp; s < p.n_seq; s += WARPS) {
            const Seq q = sequence<LIST>(p, cu_q, cu_k, s);
            for (int t = lane; t < q.tiles; t += 32) {
                int lo, hi;
                range<LIST>(p, q, t, lo, hi);
                w += hi - lo;
            }
        }
        atomicAdd(&sh.work, w);
        __syncthreads();
        // extra * chunk >= work, so that the pieces beyond one per tile number at most extra
        const unsigned long long c = (sh.work + p.extra - 1) / p.extra;
        chunk = c < (1u << 30) ? max(2 * MIN_PIECE, (int)c) : 1 << 30;
    }
    for (int s = warp; s < p.n_seq; s += WARPS) {
        const Seq q = sequence<LIST>(p, cu_q, cu_k, s);
        for (int t = lane; t < q.tiles; t += 32) {
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
    for (int s = warp; s < p.n_seq; s += WARPS) {
        const Seq q = sequence<LIST>(p, cu_q, cu_k, s);
        for (int t = lane; t < q.tiles; t += 32) {
            int lo, hi;
            range<LIST>(p, q, t, lo, hi);
            if (LIST == KTILES) {
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
            it.pos0 = t * p.tpt + q.Lk - q.Lq;
            int slot = -1;
            if (n > 1) {
                slot = atomicAdd(&sh.slots, n);
                const int m = atomicAdd(&sh.merges, p.Hkv);
                for (int hk = 0; hk < p.Hkv; hk++)
                    if (m + hk < p.cap_merge) plan.merge[m + hk] = {it.tok0, it.n_tok_hk | hk << 8, slot * p.Hkv + hk, n};
            }
            for (int c = 0; c < n; c++, i++) {  // pieces of equal length, to within a tile
                it.kt0 = (int)((long)hi * c / n), it.kt1 = (int)((long)hi * (c + 1) / n);
                it.slot = n > 1 ? slot + c : -1;
                (LIST == FWD ? plan.fwd : plan.q)[i] = it;
            }
        }
    }
    __syncthreads();
    if (LIST == FWD) deal(p, plan, sh, sh.total);
    if (threadIdx.x == 0) {
        if (LIST == FWD) {
            plan.head->n_fwd = sh.total, plan.head->n_merge = sh.merges;
            plan.head->stream = 0, plan.head->slot_step = p.Hkv;
            if ((long)sh.slots * p.Hkv > p.cap_slots || sh.merges > p.cap_merge) sh.bad = 1;
        } else if (LIST == QTILES) {
            plan.head->n_q = sh.total;
        } else {
            plan.head->n_k = sh.total;
        }
    }
}

// The batch cut into one stretch per SM.  False (the same for all threads): too
// large, nothing was written.
__device__ bool build_stretches(const PackedGeom &p, const int *cu_q, const int *cu_k, const PackedPlan &plan,
                                Shared &sh) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (p.n_seq > STREAM_SEQS) return false;
    // cost and tiles of each sequence, then of those before it
    unsigned long long all = 0;
    for (int s = warp; s < p.n_seq; s += WARPS) {
        const Seq q = sequence<FWD>(p, cu_q, cu_k, s);
        unsigned long long c = 0;
        for (int t = lane; t < q.tiles; t += 32) {
            int lo, hi;
            range<FWD>(p, q, t, lo, hi);
            c += max(hi, 1) + ITEM_COST;
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
        const int c = s < p.n_seq ? sh.cost[s] : 0, n = s < p.n_seq ? sh.tiles[s] : 0;
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
        for (int s = warp; s < p.n_seq; s += WARPS) {
            const Seq q = sequence<FWD>(p, cu_q, cu_k, s);
            int run = sh.cost[s];
            for (int t0 = 0; t0 < q.tiles; t0 += 32) {
                const int t = t0 + lane;
                int lo = 0, work = 0, cost = 0;
                if (t < q.tiles) {
                    range<FWD>(p, q, t, lo, work);
                    cost = max(work, 1) + ITEM_COST;
                }
                int upto = cost;
                for (int o = 1; o < 32; o <<= 1) {
                    const int v = __shfl_up_sync(0xffffffffu, upto, o);
                    if (lane >= o) upto += v;
                }
                const int at = run + upto - cost;
                run += __shfl_sync(0xffffffffu, upto, 31);
                if (t >= q.tiles) continue;
                for (int hk = 0; hk < p.Hkv; hk++) {
                    const int a = hk * head_cost + at, b = a + cost, unit = hk * head_tiles + sh.tiles[s] + t;
                    const int c0 = (a + Q - 1) / Q, c1 = min(p.sms, (b + Q - 1) / Q);  // borders in [a, b): [c0, c1)
                    // tile at which border c cuts the unit, moved to its ends where a piece would be too short (and
                    // to multiples of MIN_PIECE where the borders are closer than that)
                    auto cut = [&](int c) {
                        int x = max(0, c * Q - a - ITEM_COST);
                        if (Q < MIN_PIECE) x -= x % MIN_PIECE;
                        return x < MIN_PIECE ? 0 : work - x < MIN_PIECE ? work : x;
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
                    it.pos0 = t * p.tpt + q.Lk - q.Lq;
                    int slot = -1;
                    if (n > 1) {
                        slot = atomicAdd(&sh.slots, n);
                        const int m = atomicAdd(&sh.merges, 1);
                        if (m < p.cap_merge) plan.merge[m] = {it.tok0, it.n_tok_hk, slot, n};
                    }
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
                        it.kt0 = from, it.kt1 = x;
                        it.slot = n > 1 ? slot + piece : -1;
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
        if (sh.slots > p.cap_slots || sh.merges > p.cap_merge) sh.bad = 1;
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
    if (blockIdx.x == 0) {
        if (!build_stretches(p, cu_q, cu_k, plan, sh)) build<FWD>(p, cu_q, cu_k, plan, sh);
        // work that found no room in the lists (their sizes are upper bounds, so there is none) makes the plan a bad
        // one: calls report it instead of leaving rows out
        __syncthreads();
        if (threadIdx.x == 0 && sh.bad) {
            plan.head->bad = 1;
            atomicCAS(err, DEV_OK, DEV_PLAN);
        }
    } else if (blockIdx.x == 1) build<QTILES>(p, cu_q, cu_k, plan, sh);
    else build<KTILES>(p, cu_q, cu_k, plan, sh);
}

}  // namespace

cudaError_t launch_packed_plan(const PackedGeom &p, const int *cu_q, const int *cu_k, void *plan, int *err,
                               cudaStream_t st) {
    packed_plan_kernel<<<3, THREADS, 0, st>>>(p, cu_q, cu_k, plan, err);
    return cudaGetLastError();
}

}  // namespace k6
