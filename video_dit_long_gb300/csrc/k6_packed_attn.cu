// k6_packed_attn.cu -- attention over packed sequences with grouped key heads,
// on tcgen05 tensor cores: full, causal, or causal by frames, from one query
// token over a long cache to whole clips.
//
// For query token i of a sequence, query head h and its key head h / G,
//   o = sum_{j < L_i} softmax_j(q . k_j / sqrt(d)) v_j,   lse = log sum_{j < L_i} exp(q . k_j / sqrt(d)),
// L_i the mask's limit (k6_packed.cuh).  A row that sees no key gets o = 0 and
// lse = -inf.
//
// A tile of 128 query rows holds 128 / G tokens of ALL G query heads of one key
// head (one TMA box of tokens x heads), so K and V are read once per key head,
// and a single new token fills G rows of a tile instead of one.  A work item is
// one such tile over a range of 128-key tiles.  The CTAs are persistent (one a
// SM) and walk the items that the plan gives them (k6_packed_plan.cu).  A tile
// whose keys are cut into several items leaves partials (fp32 O normalised, lse
// in base 2) in the workspace, which packed_merge_kernel joins in key order.
//
// Roles in a CTA (512 threads), shared memory (Q tile, three K and three V tiles of
// 32 KB) and tensor memory (S 2 x 128 columns, P 2 x 64, O 128):
//   warp 8   TMA of the item's Q tile and its K tiles;   warp 11   of V tiles;
//   warp 9   S(n) = Q K_n^T;   warp 10   O += P(n) V_n, and the zeroing of the
//            rows of V behind the sequence's last key, where another
//            sequence's rows or unwritten memory lie: P is zero there, but
//            0 * NaN is not;
//   warps 0-7  two softmax groups on alternate tiles, one thread a row;
//   warps 12-15  the epilogue: joins the groups' row sums, takes O out of tensor
//            memory (handing it back before storing) and stores it.
// Items overlap: every role but the last runs on into the next item while the
// epilogue finishes one.  (With the epilogue in the softmax groups an item cost
// 3.4 us beyond its tiles: 1 warp a scheduler runs its serial code slowly.)
// All waits are bounded (DEV_TIMEOUT), as in the other kernels.
//
// Bounds and figures on one GB300.  Long clips: the tensor pipe under the power
// cap; 25,920 tokens causal by frames of 1,620, 24/8 heads, 2.98 ms = 1.47
// PFLOP/s, 77 % of a library product's burst (the pipe active 79 % of the time; a
// tile takes 1,370 cycles, its products 1,024).  New tokens over long caches: HBM;
// 12 streams of 1 to 52,360 keys, 24/4 heads, 51.7 us, 77 % of a copy's rate, of
// which the start and the join take 8 us.  Short prompts: the start and end of one
// item, 7.2 us a call in a captured graph (the binding's call takes 8 on the host).
#include <cuda.h>
#include <cuda_bf16.h>

#include "k6_device.cuh"
#include "k6_packed.cuh"
#include "k6_packed_tma.h"

namespace k6 {

namespace pf {
constexpr int D = 128, BM = 128, BN = 128;
constexpr int PANEL = BM * 64 * 2;
constexpr int TILE = 2 * PANEL;
// Three slots each for K and V, each kind with a producer warp of its own: K(n) takes K(n-3)'s slot as soon as
// S(n-3) is done, V(n) takes V(n-3)'s when P(n-3).V is.
constexpr int NSLOT = 3;
// S and P have tensor memory of their own, two buffers each: S(n) may be issued when the softmax has read S(n-2).
// (With P over S in three buffers S(n) waited for P(n-3).V, and the chain P(n) -> P(n).V -> S(n+3) -> softmax set
// a pace of 1,500 cycles a tile, half as much again as the products take.)
constexpr int NBUF = 2;
constexpr int P_PARTS = 2;
constexpr int KP = BN / P_PARTS;
constexpr int SMEM_Q = 0;
constexpr int SMEM_KV = TILE;
constexpr int SMEM_V = SMEM_KV + NSLOT * TILE;
constexpr int SMEM_BAR = SMEM_V + NSLOT * TILE;
// q_full, q_empty, k_full, k_empty, v_full, v_empty [slot], s_full, s_free [buffer], p_part [buffer][part], o_final,
// o_free, drain, posted, sums_free, pv_buf [buffer], m_ready [tile parity][warp]
constexpr int NBAR = 2 + 4 * NSLOT + 2 * NBUF + NBUF * P_PARTS + 5 + NBUF + 8;
constexpr int SMEM_XCH = (SMEM_BAR + NBAR * 8 + 8 + 15) & ~15;  // + TMEM address, abort flag
constexpr int SMEM_TOTAL = SMEM_XCH + (BM + 2 * 2 * BM) * 4;    // row max; (l, m) of each group
static_assert(SMEM_TOTAL <= 227 * 1024, "shared memory plan exceeds the per-CTA limit");
constexpr int THREADS = 512;
// Register split (launch: 512 x 128 = 65536): 2*128*176 + 128*64 + 128*96 = 65536.
constexpr int REGS_SOFTMAX = 176;
constexpr int REGS_CONTROL = 64;
constexpr int REGS_EPILOGUE = 96;
constexpr int TMEM_COLS = 512;
constexpr int P_COL = NBUF * BN;              // P buffers: 64 columns each
constexpr int O_COL = P_COL + NBUF * BN / 2;
constexpr float RESCALE_THRESHOLD = 8.0f;     // log2 units: O is rescaled when the max grows past 2^8
constexpr unsigned long long DRAIN_NS = 1000000000ull;
}  // namespace pf

struct PackedFwdParams {
    PackedGeom g;
    const void *plan;
    float scale_log2;                         // log2(e) / sqrt(d)
    __nv_bfloat16 *out;
    long out_stride;
    float *lse;                               // [H][Tq], or null
    float *part_o, *part_lse;                 // [partial][128][128], [partial][128]
    uint32_t idesc_qk;
    int wide;                                 // rows of out are 32-byte aligned
    unsigned long long wait_limit_ns;
    int *err;
};

namespace {

// exp2 of a difference from a maximum that may be -inf (nothing seen yet): 0 then.
__device__ __forceinline__ float ex2_from(float m, float m_new) { return m == -INFINITY ? 0.f : ex2(m - m_new); }

// The items of this CTA: its row of the plan's stretches, or its column of the
// schedule of (item, key head) pairs.
struct Walk {
    const PackedItem *list;
    const int *sched;   // null: list is this CTA's own
    uint32_t rounds, n_items;
    int slots;          // partials that one slot number stands for (1, or one for every key head)
    __device__ Walk(const PackedPlan &plan, const PackedGeom &g, bool ok) {
        list = plan.fwd;
        const int mine = plan.count[blockIdx.x];  // beside the header, in every plan: no wait between the two (the grid is g.sms)
        slots = plan.head->slot_step;
        n_items = (uint32_t)plan.head->n_fwd;
        if (plan.head->stream) {
            list += (long)blockIdx.x * g.cap_rows;
            sched = nullptr;
            rounds = (uint32_t)mine;
        } else {
            sched = plan.sched + blockIdx.x;
            rounds = (n_items * (uint32_t)g.Hkv + gridDim.x - 1) / gridDim.x;
        }
        if (!ok) rounds = 0;
    }
    __device__ bool at(uint32_t k, PackedItem &it, int &hk) const {
        uint32_t i = k;
        if (sched) {
            const int u = sched[(long)k * gridDim.x];
            if (u < 0) return false;
            hk = (int)((uint32_t)u / n_items);
            i = (uint32_t)u - (uint32_t)hk * n_items;
        }
        it = list[i];
        if (!sched) hk = it.n_tok_hk >> 8;
        return true;
    }
};

// 32 bytes in one store.
__device__ __forceinline__ void st_global_32(void *p, const uint32_t *v) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

__global__ void __launch_bounds__(pf::THREADS, 1)
    packed_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const PackedFwdParams p) {
    using namespace pf;
    extern __shared__ __align__(1024) uint8_t smem[];
    launch_next_kernel();
    if (smem_u32(smem) & 1023u) {  // the same for every thread: the CTA leaves before any barrier
        wait_previous_kernel();
        if (threadIdx.x == 0) atomicCAS(p.err, DEV_OK, DEV_LAYOUT);
        return;
    }
    // barriers and tensor memory are set up while the kernel before this one drains
    uint64_t *q_full = reinterpret_cast<uint64_t *>(smem + SMEM_BAR);
    uint64_t *q_empty = q_full + 1;
    uint64_t *k_full = q_empty + 1;
    uint64_t *k_empty = k_full + NSLOT;
    uint64_t *v_full = k_empty + NSLOT;
    uint64_t *v_empty = v_full + NSLOT;
    uint64_t *s_full = v_empty + NSLOT;
    uint64_t *s_free = s_full + NBUF;      // the softmax has read S (128 arrivals)
    uint64_t *p_part = s_free + NBUF;      // [buffer][part], 128 arrivals each
    uint64_t *o_final = p_part + NBUF * P_PARTS;
    uint64_t *o_free = o_final + 1;        // the epilogue has O in registers (128 arrivals)
    uint64_t *drain = o_free + 1;
    uint64_t *posted = drain + 1;          // both softmax groups posted an item's (l, m)
    uint64_t *sums_free = posted + 1;      // the epilogue has read them
    uint64_t *pv_buf = sums_free + 1;      // [buffer]: P.V of the P in that buffer done
    uint64_t *m_ready = pv_buf + NBUF;    // [tile parity][warp % 4]: row max after the tile published
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(m_ready + 8);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int i = 0; i < NSLOT; i++) {
            mbar_init(&k_full[i], 1);
            mbar_init(&k_empty[i], 1);
            mbar_init(&v_full[i], 1);
            mbar_init(&v_empty[i], 1);
        }
        for (int b = 0; b < NBUF; b++) {
            mbar_init(&s_full[b], 1);
            mbar_init(&s_free[b], BM);
            mbar_init(&pv_buf[b], 1);
        }
        for (int q = 0; q < NBUF * P_PARTS; q++) mbar_init(&p_part[q], BM);
        mbar_init(o_final, 1);
        mbar_init(o_free, BM);
        mbar_init(drain, 2);  // one commit per MMA issuer
        mbar_init(posted, 2 * BM);
        mbar_init(sums_free, BM);
        for (int q = 0; q < 8; q++) mbar_init(&m_ready[q], 32);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 9) {
        tmem_alloc(tmem_slot, TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    wait_previous_kernel();
    const PackedPlan plan = packed_plan_at(const_cast<void *>(p.plan), p.g);
    const bool plan_ok = packed_plan_ok(*plan.head, p.g);
    if (!plan_ok && threadIdx.x == 0) atomicCAS(p.err, DEV_OK, DEV_PLAN);
    const Walk walk(plan, p.g, plan_ok);  // nothing to walk under a plan that is not this batch's
    const WaitCtx w{p.wait_limit_ns, p.err, abort_flag};

    float *xm = reinterpret_cast<float *>(smem + SMEM_XCH);  // [row]: max after the latest tile
    float *xe = xm + BM;                                      // [group][row][l, m]

    if (warp >= 8 && warp < 12) {
        regs_decrease<REGS_CONTROL>();
        if (warp == 8 || warp == 11) {
            // ------------------------------------- TMA producers: K and Q (8), V (11)
            const bool leader = elect_one();
            const CUtensorMap *tm = warp == 8 ? &tm_k : &tm_v;
            uint64_t *full = warp == 8 ? k_full : v_full, *empty = warp == 8 ? k_empty : v_empty;
            uint8_t *ring = smem + (warp == 8 ? SMEM_KV : SMEM_V);
            if (leader) {
                prefetch_tmap(tm);
                if (warp == 8) prefetch_tmap(&tm_q);
            }
            uint32_t n = 0;       // tiles loaded
            uint32_t uc = 0;      // items with keys so far
            bool ok = true;
            for (uint32_t k = 0; k < walk.rounds && ok; k++) {
                PackedItem it;
                int hk;
                if (!walk.at(k, it, hk)) continue;
                const int T = it.kt1 - it.kt0;
                if (T <= 0) continue;
                for (int j = 0; j < T && ok; j++, n++) {
                    const uint32_t slot = n % NSLOT;
                    if (!(ok = mbar_wait_w(&empty[slot], ((n / NSLOT) & 1) ^ 1, w))) break;
                    if (leader) {
                        uint8_t *dst = ring + slot * TILE;
                        const int row = it.krow0 + (it.kt0 + j) * BN;
                        mbar_arrive_expect_tx(&full[slot], TILE);
                        tma_load_4d(dst, tm, &full[slot], 0, hk, row, 0);
                        tma_load_4d(dst + PANEL, tm, &full[slot], 64, hk, row, 0);
                    }
                    if (j == 0 && warp == 8) {  // Q once the last S of the item before has read its tile
                        if (!(ok = uc == 0 || mbar_wait_w(q_empty, (uc - 1) & 1, w))) {
                            n++;  // this tile's load was issued
                            break;
                        }
                        if (leader) {
                            mbar_arrive_expect_tx(q_full, (uint32_t)p.g.rows * 256u);
                            tma_load_4d(smem + SMEM_Q, &tm_q, q_full, 0, hk * p.g.G, it.tok0, 0);
                            tma_load_4d(smem + SMEM_Q + PANEL, &tm_q, q_full, 64, hk * p.g.G, it.tok0, 0);
                        }
                        uc++;
                    }
                }
            }
            // every copy issued lands before the CTA can exit
            if (uc > 0) mbar_drain(q_full, (uc - 1) & 1, DRAIN_NS);
            for (uint32_t i = n > NSLOT ? n - NSLOT : 0; i < n; i++)
                mbar_drain(&full[i % NSLOT], (i / NSLOT) & 1, DRAIN_NS);
        } else if (warp == 9 || warp == 10) {
            // ------------------------------------------------- MMA issuers
            const uint32_t idesc_pv = idesc_bf16_f32(BM, D, true);
            const uint64_t dq0 = smem_desc_sw128(smem_u32(smem + SMEM_Q), 16, 1024);     // Q / K: K-major
            const uint64_t dk0 = smem_desc_sw128(smem_u32(smem + SMEM_KV), 16, 1024);
            const uint64_t dv0 = smem_desc_sw128(smem_u32(smem + SMEM_V), PANEL, 1024);  // V: MN-major
            uint32_t tile = 0;    // key tiles of earlier items
            uint32_t uc = 0;
            bool ok = true;
            for (uint32_t k = 0; k < walk.rounds && ok; k++) {
                PackedItem it;
                int hk;
                if (!walk.at(k, it, hk)) continue;
                const int T = it.kt1 - it.kt0;
                if (T <= 0) continue;
                if (warp == 9) {
                    ok = mbar_wait_w(q_full, uc & 1, w);
                    for (int t = 0; t < T && ok; t++) {
                        const uint32_t n = tile + t, slot = n % NSLOT;
                        // S(n) takes the buffer of S(n-2), which the softmax has read
                        if (n >= NBUF && !(ok = mbar_wait_w(&s_free[n % NBUF], (n / NBUF - 1) & 1, w))) break;
                        if (!(ok = mbar_wait_w(&k_full[slot], (n / NSLOT) & 1, w))) break;
                        tc_fence_after();
                        const uint64_t kb = dk0 + ((uint64_t)(slot * TILE) >> 4);
#pragma unroll
                        for (int kk = 0; kk < D / 16; kk++) {
                            const uint64_t off = (uint64_t)((kk >> 2) * PANEL + (kk & 3) * 32) >> 4;
                            mma_ss_w(tmem + (n % NBUF) * BN, dq0 + off, kb + off, p.idesc_qk, kk > 0);
                        }
                        tc_commit_w(&s_full[n % NBUF]);  // K(n)'s slot is freed by the softmax, which sees S(n)
                    }
                    if (ok) tc_commit_w(q_empty);
                } else {
                    for (int j = 0; j < T && ok; j++) {
                        const uint32_t n = tile + j, slot = n % NSLOT;
                        if (!(ok = mbar_wait_w(&v_full[slot], (n / NSLOT) & 1, w))) break;
                        const int valid = it.Lk - (it.kt0 + j) * BN;
                        if (valid < BN) {  // rows behind the sequence's last key: zero (P is)
                            uint8_t *v = smem + SMEM_V + slot * TILE;
                            for (int c = valid * 8 + lane; c < BN * 8; c += 32) {
                                *reinterpret_cast<uint4 *>(v + c * 16) = make_uint4(0, 0, 0, 0);
                                *reinterpret_cast<uint4 *>(v + PANEL + c * 16) = make_uint4(0, 0, 0, 0);
                            }
                            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                            __syncwarp();
                        }
                        const uint64_t vb = dv0 + ((uint64_t)(slot * TILE) >> 4);
                        const uint32_t pb = tmem + P_COL + (n % NBUF) * (BN / 2);
                        for (int q = 0; q < P_PARTS && ok; q++) {
                            if (!(ok = mbar_wait_w(&p_part[(n % NBUF) * P_PARTS + q], (n / NBUF) & 1, w))) break;
                            // the first product of an item overwrites O: the epilogue before has read it
                            if (j == 0 && q == 0 && uc > 0 && !(ok = mbar_wait_w(o_free, (uc - 1) & 1, w))) break;
                            tc_fence_after();
#pragma unroll
                            for (int kk = q * (KP / 16); kk < (q + 1) * (KP / 16); kk++)
                                mma_ts_w(tmem + O_COL, pb + kk * 8, vb + ((uint64_t)(kk * 16 * 128) >> 4), idesc_pv,
                                         (j > 0 || kk > 0) ? 1u : 0u);
                        }
                        if (!ok) break;
                        tc_commit_w(&v_empty[slot]);
                        tc_commit_w(&pv_buf[n % NBUF]);
                        if (j + 1 == T) tc_commit_w(o_final);
                    }
                }
                tile += T;
                uc++;
            }
            // every MMA issued completes before tensor memory is freed (one commit per issuer)
            tc_commit_w(drain);
            mbar_drain(drain, 0, DRAIN_NS);
        }
        __syncwarp();
    } else if (warp >= 12) {
        regs_decrease<REGS_EPILOGUE>();
        // ------------------------------------ epilogue (thread = row = TMEM lane)
        const int wq = warp % 4;
        const int r = 32 * wq + lane;
        const int rtok = r / p.g.G, rhead = r - rtok * p.g.G;  // this row's token of a tile and head of a group
        const uint32_t tO = tmem + ((uint32_t)(32 * wq) << 16) + O_COL;
        uint32_t n_epi = 0;
        bool ok = true;
        for (uint32_t k = 0; k < walk.rounds && ok; k++) {
            PackedItem it;
            int hk;
            if (!walk.at(k, it, hk)) continue;
            const int n_tok = it.n_tok_hk & 255;
            const bool live = rtok < n_tok && r < p.g.rows;
            float *lse = p.lse ? p.lse + (long)(hk * p.g.G + rhead) * p.g.Tq + it.tok0 + rtok : nullptr;
            if (it.kt1 <= it.kt0) {  // no key is seen by any row of the tile
                if (live) {
                    __nv_bfloat16 *dst =
                        p.out + ((long)it.tok0 + rtok) * p.out_stride + (long)(hk * p.g.G + rhead) * D;
#pragma unroll
                    for (int c = 0; c < D; c += 8) *reinterpret_cast<uint4 *>(dst + c) = make_uint4(0, 0, 0, 0);
                    if (lse) *lse = -INFINITY;
                }
                continue;
            }
            if (!(ok = mbar_wait(posted, n_epi & 1, w))) break;
            const float l0 = xe[r * 2], m0 = xe[r * 2 + 1], l1 = xe[(BM + r) * 2], m1 = xe[(BM + r) * 2 + 1];
            mbar_arrive(sums_free);
            const float m_fin = fmaxf(m0, m1);  // the max O is expressed in
            const float l_tot = l0 * ex2_from(m0, m_fin) + l1 * ex2_from(m1, m_fin);
            const bool none = l_tot == 0.f;  // the row sees nothing
            const float inv = none ? 0.f : 1.f / l_tot;
            const float lse2 = none ? -INFINITY : m_fin + log2f(l_tot);
            if (!(ok = mbar_wait(o_final, n_epi & 1, w))) break;
            tc_fence_after();
            // each thread stores its row, a 32-byte sector at a time
            const bool part = it.slot >= 0;
            const long prow = ((long)it.slot * walk.slots + (walk.slots > 1 ? hk : 0)) * BM + r;
            if (part) {
                float *dst = p.part_o + prow * D;
#pragma unroll 1
                for (int cc = 0; cc < D / 32; cc++) {
                    uint32_t o[32];
                    tmem_ld32(tO + cc * 32, o);
                    tmem_ld_wait();
                    if (cc + 1 == D / 32) {  // O is out of tensor memory
                        tc_fence_before();
                        mbar_arrive(o_free);
                    }
#pragma unroll
                    for (int c = 0; c < 32; c++) o[c] = none ? 0u : __float_as_uint(__uint_as_float(o[c]) * inv);
                    if (live) {
#pragma unroll
                        for (int c = 0; c < 32; c += 8) st_global_32(dst + cc * 32 + c, &o[c]);
                    }
                    __syncwarp();
                }
            } else {
                uint32_t b[D / 2];  // the row as bf16
#pragma unroll
                for (int cc = 0; cc < D / 32; cc++) {
                    uint32_t o[32];
                    tmem_ld32(tO + cc * 32, o);
                    tmem_ld_wait();
#pragma unroll
                    for (int c = 0; c < 32; c += 2)
                        b[(cc * 32 + c) / 2] = none ? 0u
                                                    : pack_bf16x2(__uint_as_float(o[c]) * inv,
                                                                  __uint_as_float(o[c + 1]) * inv);
                }
                tc_fence_before();
                mbar_arrive(o_free);  // O is out of tensor memory
                if (live) {
                    __nv_bfloat16 *dst =
                        p.out + ((long)it.tok0 + rtok) * p.out_stride + (long)(hk * p.g.G + rhead) * D;
                    if (p.wide) {
#pragma unroll
                        for (int c = 0; c < D / 2; c += 8) st_global_32(dst + 2 * c, &b[c]);
                    } else {  // rows are 16-byte aligned only
#pragma unroll
                        for (int c = 0; c < D / 2; c += 4)
                            *reinterpret_cast<uint4 *>(dst + 2 * c) = make_uint4(b[c], b[c + 1], b[c + 2], b[c + 3]);
                    }
                }
            }
            if (live) {
                if (part) p.part_lse[prow] = lse2;
                else if (lse) *lse = lse2 * 0.69314718055994531f;
            }
            n_epi++;
        }
    } else {
        regs_increase<REGS_SOFTMAX>();
        // ------------------------------------ softmax (group hf)
        // Group hf takes the tiles n with n % 2 == hf, whole rows (thread = row =
        // TMEM lane).  The groups share the row's running max through shared
        // memory (m_ready); O is rescaled in tensor memory only when a tile's max
        // exceeds it by 2^8.  Each group keeps the row sum of its own tiles, in
        // the max it last saw, and posts it for the epilogue.
        const int hf = warp / 4, wq = warp % 4;
        const int r = threadIdx.x % BM;
        const int rtok = r / p.g.G;  // this row's token of a tile
        const uint32_t lane_base = tmem + ((uint32_t)(32 * wq) << 16);
        const uint32_t tO = lane_base + O_COL;
        const float sl2 = p.scale_log2;
        uint32_t tile = 0, n_item = 0;
        bool ok = true;
        for (uint32_t k = 0; k < walk.rounds && ok; k++) {
            PackedItem it;
            int hk;
            if (!walk.at(k, it, hk)) continue;
            const int T = it.kt1 - it.kt0;
            if (T <= 0) continue;
            const bool live = rtok < (it.n_tok_hk & 255) && r < p.g.rows;
            // keys this row sees; rows past the tile's tokens see what the sequence has (their results are dropped)
            const int lim = live ? packed_limit(it.pos0 + rtok, it.Lk, p.g.block) : it.Lk;
            float m_run = -INFINITY;  // the row max in force after the latest tile
            float m_own = -INFINITY;  // the max l_own is expressed in
            float l_own = 0.f;
            for (int j = 0; j < T; j++) {
                const uint32_t n = tile + j;
                if ((int)(n & 1) != hf) continue;
                const uint32_t tS = lane_base + (n % NBUF) * BN, tP = lane_base + P_COL + (n % NBUF) * (BN / 2);
                if (!mbar_wait(&s_full[n % NBUF], (n / NBUF) & 1, w)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (r == 0) mbar_arrive(&k_empty[n % NSLOT]);  // K(n) read
                if (n > 0) {  // the max after tile n-1, every phase waited for in turn
                    if (!mbar_wait(&m_ready[((n - 1) & 1) * 4 + wq], ((n - 1) >> 1) & 1, w)) {
                        ok = false;
                        break;
                    }
                    if (j > 0) m_run = xm[r];
                }
                uint32_t s[BN];
#pragma unroll
                for (int cc = 0; cc < BN / 32; cc++)
                    tmem_ld32(tS + cc * 32, *reinterpret_cast<uint32_t(*)[32]>(&s[cc * 32]));
                tmem_ld_wait();
                tc_fence_before();
                mbar_arrive(&s_free[n % NBUF]);  // S(n+2) may take the buffer
                const int rel = lim - (it.kt0 + j) * BN;  // columns below rel are seen
                if (__any_sync(0xffffffffu, rel < BN)) {
#pragma unroll
                    for (int k = 0; k < BN; k++)
                        if (k >= rel) s[k] = 0xff800000u;
                }
                float mc[4];
#pragma unroll
                for (int c4 = 0; c4 < 4; c4++) {
                    const uint32_t *x = &s[c4 * 32];
                    float m = fmax3(__uint_as_float(x[0]), __uint_as_float(x[1]), __uint_as_float(x[2]));
#pragma unroll
                    for (int k = 3; k < 31; k += 2) m = fmax3(m, __uint_as_float(x[k]), __uint_as_float(x[k + 1]));
                    mc[c4] = fmaxf(m, __uint_as_float(x[31]));
                }
                const float mt = fmaxf(fmaxf(mc[0], mc[1]), fmaxf(mc[2], mc[3])) * sl2;
                bool need = false, rescale = false;  // rescale: warp-uniform
                float alpha = 1.f;
                if (j == 0) m_run = mt;
                else need = mt > m_run + RESCALE_THRESHOLD;  // also from -inf: nothing seen before
                if (__any_sync(0xffffffffu, need)) {
                    rescale = true;
                    if (need) {
                        alpha = ex2_from(m_run, mt);
                        m_run = mt;
                    }
                }
                xm[r] = m_run;
                mbar_arrive(&m_ready[(n & 1) * 4 + wq]);
                if (m_own != m_run) {
                    l_own *= ex2_from(m_own, m_run);
                    m_own = m_run;
                }
                // p = 2^(s * scale*log2e - m); with nothing seen so far every s is -inf and p = 0
                const float m_use = m_run == -INFINITY ? 0.f : m_run;
                const uint64_t scale2 = f2(sl2, sl2), negm2 = f2(-m_use, -m_use);
                uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
                for (int q = 0; q < P_PARTS; q++) {
                    uint32_t pk[KP / 2];
#pragma unroll
                    for (int k = 0; k < KP; k += 2) {
                        const int kk = q * KP + k;
                        float a, b2;
                        f2_split(ffma2(f2(__uint_as_float(s[kk]), __uint_as_float(s[kk + 1])), scale2, negm2), a, b2);
                        const float p0 = ex2(a), p1 = ex2(b2);
                        // P in bf16, the type of V (one MMA takes one type): 2^-8 of each term, the
                        // row sum keeps fp32
                        pk[k / 2] = pack_bf16x2(p0, p1);
                        acc[(k / 2) & 3] = fadd2(acc[(k / 2) & 3], f2(p0, p1));
                    }
                    if (q == 0 && n >= NBUF) {  // P(n) takes the buffer of P(n-2)
                        if (!mbar_wait(&pv_buf[n % NBUF], (n / NBUF - 1) & 1, w)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                    }
                    tmem_st_cols<KP / 2>(tP + q * (KP / 2), pk);
                    if (q == 0 && rescale) {
                        // O holds P.V of tiles < n once P(n-1).V is done; rescale it before P(n).V
                        if (!mbar_wait(&pv_buf[(n - 1) % NBUF], ((n - 1) / NBUF) & 1, w)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
#pragma unroll
                        for (int cc = 0; cc < D / 32; cc++) {
                            uint32_t o[32];
                            tmem_ld32(tO + cc * 32, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int k = 0; k < 32; k++) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
                            tmem_st32(tO + cc * 32, o);
                        }
                    }
                    tmem_st_wait();
                    tc_fence_before();
                    mbar_arrive(&p_part[(n % NBUF) * P_PARTS + q]);
                }
                if (!ok) break;
                float a0, a1, b0, b1;
                f2_split(fadd2(acc[0], acc[1]), a0, a1);
                f2_split(fadd2(acc[2], acc[3]), b0, b1);
                l_own += (a0 + a1) + (b0 + b1);
            }
            if (!ok) break;
            // post the row sum of this group's tiles, once the epilogue has read the item before's
            if (n_item > 0 && !mbar_wait(sums_free, (n_item - 1) & 1, w)) {
                ok = false;
                break;
            }
            xe[(hf * BM + r) * 2] = l_own;
            xe[(hf * BM + r) * 2 + 1] = m_own;
            mbar_arrive(posted);
            n_item++;
            tile += T;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, TMEM_COLS);
    }
}

// Joins the partials of the split tiles: half a warp per row of a split tile,
// 32 bytes a lane,
//   lse = log2 sum_c 2^lse_c,   o = sum_c 2^(lse_c - lse) o_c.
// All rows fit the GPU at once, so that the kernel is two reads deep: the
// partial's place, then its data.
__global__ void __launch_bounds__(256) packed_merge_kernel(const PackedFwdParams p) {
    launch_next_kernel();
    wait_previous_kernel();
    const PackedPlan plan = packed_plan_at(const_cast<void *>(p.plan), p.g);
    const int lane = threadIdx.x & 15;
    const uint32_t x = (blockIdx.x * blockDim.x + threadIdx.x) >> 4;
    const uint32_t mi = x / (uint32_t)p.g.rows;
    const int r = (int)(x - mi * (uint32_t)p.g.rows);
    if (mi >= (uint32_t)p.g.cap_merge) return;
    // the first p.g.sms split tiles lie in every plan (packed_plan_common_bytes): read beside the header, with no wait
    // between the two; those behind them only once the header has shown that the plan is this batch's
    const bool early = mi < (uint32_t)p.g.sms;
    PackedMerge m;
    if (early) m = plan.merge[mi];
    const PackedHeader head = *plan.head;
    if (!packed_plan_ok(head, p.g) || mi >= (uint32_t)head.n_merge) return;  // the attention kernel reported a bad plan
    if (!early) m = plan.merge[mi];
    if (r / p.g.G >= (m.n_tok_hk & 255)) return;
    const long base = (long)m.slot0 * 128 + r, step = (long)head.slot_step * 128;
    constexpr int kU = 4;  // partials in flight
    float top = -INFINITY, sum = 0.f, acc[8];
#pragma unroll
    for (int e = 0; e < 8; e++) acc[e] = 0.f;
    for (int c = 0; c < m.n; c += kU) {
        float4 o[kU][2];
        float l[kU];
#pragma unroll
        for (int i = 0; i < kU; i++) {
            l[i] = -INFINITY, o[i][0] = o[i][1] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c + i < m.n) {
                const long row = base + (c + i) * step;
                l[i] = p.part_lse[row];
                o[i][0] = reinterpret_cast<const float4 *>(p.part_o + row * 128)[2 * lane];
                o[i][1] = reinterpret_cast<const float4 *>(p.part_o + row * 128)[2 * lane + 1];
            }
        }
        float m_new = top;
#pragma unroll
        for (int i = 0; i < kU; i++) m_new = fmaxf(m_new, l[i]);
        const float ref = m_new == -INFINITY ? 0.f : m_new;
        const float old = ex2(top - ref);  // 0 from -inf
        top = m_new;
        sum *= old;
#pragma unroll
        for (int e = 0; e < 8; e++) acc[e] *= old;
#pragma unroll
        for (int i = 0; i < kU; i++) {
            const float f = ex2(l[i] - ref);
            sum += f;
            const float v[8] = {o[i][0].x, o[i][0].y, o[i][0].z, o[i][0].w, o[i][1].x, o[i][1].y, o[i][1].z, o[i][1].w};
#pragma unroll
            for (int e = 0; e < 8; e++) acc[e] = fmaf(f, v[e], acc[e]);
        }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const long tok = (long)m.tok0 + r / p.g.G;
    const int head_q = (m.n_tok_hk >> 8) * p.g.G + r % p.g.G;
    *reinterpret_cast<uint4 *>(p.out + tok * p.out_stride + (long)head_q * 128 + lane * 8) =
        make_uint4(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv),
                   pack_bf16x2(acc[4] * inv, acc[5] * inv), pack_bf16x2(acc[6] * inv, acc[7] * inv));
    if (lane == 0 && p.lse)
        p.lse[(long)head_q * p.g.Tq + tok] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
}

}  // namespace

size_t packed_fwd_workspace(const PackedGeom &p) {
    const size_t rows = (size_t)p.cap_slots * 128;
    return rows ? round256(rows * 128 * 4) + round256(rows * 4) + 256 : 0;  // 256: see launch_packed_fwd
}

cudaError_t launch_packed_fwd(const PackedGeom &g, const PackedPtrs &t, void *out, long out_stride, float *lse,
                              void *ws, cudaStream_t st, const char **why) {
    if (g.Tq == 0) return cudaSuccess;
    CUtensorMap mq, mk, mv;
    // without key rows no tile has keys and the maps of k and v are never used
    if (!packed_q_map(&mq, t.q, g, t.q_stride, why) ||
        !packed_kv_map(&mk, g.Tk ? t.k : t.q, g.Tk ? g.Tk : g.Tq, g.Tk ? g.Hkv : 1, g.Tk ? t.k_stride : t.q_stride, why) ||
        !packed_kv_map(&mv, g.Tk ? t.v : t.q, g.Tk ? g.Tk : g.Tq, g.Tk ? g.Hkv : 1, g.Tk ? t.v_stride : t.q_stride, why))
        return cudaErrorInvalidValue;
    cudaError_t e = set_max_dynamic_smem((const void *)packed_fwd_kernel, pf::SMEM_TOTAL);
    if (e != cudaSuccess) return e;
    PackedFwdParams p;
    p.g = g;
    p.plan = t.plan;
    p.scale_log2 = (float)(1.4426950408889634 / sqrt(128.0));
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.out_stride = out_stride;
    p.lse = lse;
    const size_t rows = (size_t)g.cap_slots * 128;
    // partial rows are stored 32 bytes at a time; the caller's workspace may be 16-byte aligned only
    char *at = reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(ws) + 31) & ~(uintptr_t)31);
    p.part_o = reinterpret_cast<float *>(at);
    p.part_lse = reinterpret_cast<float *>(at + round256(rows * 128 * 4));
    // Q.K^T operands: bf16 (A/B format 1) or fp16 (format 0)
    p.idesc_qk = idesc_bf16_f32(128, 128, false);
    if (t.qk_f16) p.idesc_qk &= ~((7u << 7) | (7u << 10));
    p.wide = (reinterpret_cast<uintptr_t>(out) % 32 == 0 && out_stride * 2 % 32 == 0) ? 1 : 0;
    p.wait_limit_ns = t.wait_limit_ns;
    p.err = t.err;
    e = launch_after(packed_fwd_kernel, (unsigned)g.sms, pf::THREADS, pf::SMEM_TOTAL, st, mq, mk, mv, p);
    if (e != cudaSuccess || g.extra == 0) return e;
    return launch_after(packed_merge_kernel, (unsigned)(((long)g.cap_merge * g.rows + 15) / 16), 256, 0, st, p);
}

}  // namespace k6
