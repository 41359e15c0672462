// k6_packed_plan.cu -- lays out the work of packed attention on the device, once
// per batch: lists of query tiles and key tiles from the sequences' offsets,
// heaviest first, with long key ranges of few query tiles split so that the
// GPU's SMs share them.  The offsets stay on the device, so a batch can be
// planned inside a captured graph; a layer stack reuses the plan.
//
// Three blocks, one list each: forward items (with splits), unsplit query
// tiles (backward dq) and key tiles (backward dk/dv).  Warps stride over
// sequences, lanes over a sequence's tiles; a counting sort by work in 256
// classes orders the items.  The order within a class, and so which SM runs an
// item and which slot holds a partial, may differ between runs; every item
// writes rows of its own and partials are joined in key order, so results do
// not.
#include "k6_packed.cuh"

namespace k6 {

// Key tiles below which a range is never split: a piece should outlast the
// start and the join of a work item.
constexpr int MIN_CHUNK = 4;
// Work items aimed at, per SM, when long ranges are split.
constexpr int ITEMS_PER_SM = 2;

PackedGeom packed_geom(const Geom &g, const k6attn_packed &b) {
    PackedGeom p;
    p.n_seq = b.n_seq;
    p.H = g.H, p.Hkv = b.kv_heads, p.G = g.H / b.kv_heads, p.block = b.mask_block;
    p.Tq = (int)b.q_tokens, p.Tk = (int)b.k_tokens;
    p.tpt = 128 / p.G;
    p.rows = p.tpt * p.G;
    // sum of ceil(L / n) <= floor(T / n) + sequences
    p.cap_q = p.Tq / p.tpt + p.n_seq;
    p.cap_k = p.Tk / 128 + p.n_seq;
    int dev = 0, sms = 152;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    // no sequence has more than MIN_CHUNK key tiles: nothing to split
    p.extra = p.Tk > MIN_CHUNK * 128 ? (ITEMS_PER_SM * sms + p.Hkv - 1) / p.Hkv : 0;
    p.cap_slots = 2 * p.extra;
    return p;
}

size_t packed_plan_bytes(const PackedGeom &p) {
    const PackedPlan at = packed_plan_at(nullptr, p);
    return reinterpret_cast<size_t>(at.merge) + (size_t)p.extra * sizeof(PackedMerge);
}

namespace {

constexpr int THREADS = 1024, WARPS = THREADS / 32, CLASSES = 256;

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
};

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
        chunk = c < (1u << 30) ? max(MIN_CHUNK, (int)c) : 1 << 30;
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
            it.n_tok = min(p.tpt, q.Lq - t * p.tpt);
            it.krow0 = q.k0, it.Lk = q.Lk;
            it.pos0 = t * p.tpt + q.Lk - q.Lq;
            int slot = -1;
            if (n > 1) {
                slot = atomicAdd(&sh.slots, n);
                plan.merge[atomicAdd(&sh.merges, 1)] = {it.tok0, it.n_tok, slot, n};
            }
            for (int c = 0; c < n; c++, i++) {  // pieces of equal length, to within a tile
                it.kt0 = (int)((long)hi * c / n), it.kt1 = (int)((long)hi * (c + 1) / n);
                it.slot = n > 1 ? slot + c : -1;
                (LIST == FWD ? plan.fwd : plan.q)[i] = it;
            }
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        if (LIST == FWD) {
            plan.head->n_fwd = sh.total, plan.head->n_merge = sh.merges, plan.head->n_slots = sh.slots;
            plan.head->chunk = chunk;
        } else if (LIST == QTILES) {
            plan.head->n_q = sh.total;
        } else {
            plan.head->n_k = sh.total;
        }
    }
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
    if (blockIdx.x == 0) build<FWD>(p, cu_q, cu_k, plan, sh);
    else if (blockIdx.x == 1) build<QTILES>(p, cu_q, cu_k, plan, sh);
    else build<KTILES>(p, cu_q, cu_k, plan, sh);
}

}  // namespace

cudaError_t launch_packed_plan(const PackedGeom &p, const int *cu_q, const int *cu_k, void *plan, int *err,
                               cudaStream_t st) {
    packed_plan_kernel<<<3, THREADS, 0, st>>>(p, cu_q, cu_k, plan, err);
    return cudaGetLastError();
}

}  // namespace k6
