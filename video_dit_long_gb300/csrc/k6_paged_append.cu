// k6_paged_append.cu -- new tokens over a cache of pages: per-head QK-norm and
// rotation of queries and keys as k6_packed_norm.cu computes them, the keys and the
// values to the places in the pages that the plan gives their tokens.
//
// Bound by HBM: each row is read once and written once.  A head row is 16 lanes of
// one 16-byte vector; a warp takes a run of a token's heads of q, of k or of v, with
// several vectors a lane in flight, and computes its pairs' sin and cos once a run.
// The rest is instructions: the products of the rotation go two to an instruction
// (52,360 tokens of 24/8 heads 188 us without, 174 with), and stores that are not
// kept in the caches give the reads more of them (169 us, 6.3 TB/s, 93 % of a copy's).
// Eight tokens take 3.2 us, 2,669 of them (24/4 heads) 13.5: start, the plan's header and
// a second round of runs.
//
// Measured and not kept, us for 52,360 / 2,669 / 8 tokens (169 / 13.5 / 3.2 as it is): vectors x blocks 6 x 3 183 /
// 13.8 / 3.4, 4 x 3 184 / 13.5 / 3.2 (both before the stores), 3 x 5 and 2 x 5 232 / 20 (spills); k and v in one run 203 /
// 14.6 / 3.7; a block for four tokens with a table of sin and cos in shared memory 218 / 16.4 / 3.5; rows brought to and
// from shared memory by bulk copies, a ring for each warp, 180 / 14.9 / 3.4 at best (176 / 12.0 / 2.8 with the
// arithmetic taken out of a copy: the copies are no faster).
#include "k6_norm_rope.cuh"
#include "k6_paged.cuh"

namespace k6 {

namespace {

constexpr int BLOCKS_PER_SM = 4;  // of 256 threads
constexpr int VECS = 4;           // that a lane has in flight
constexpr int PASS = 2 * VECS;    // heads that a warp takes at a time
constexpr int WHOLE_FROM = 16;    // tokens an SM from which a warp takes all heads of a token
constexpr int ROW = 256;          // bytes

struct AppendArgs {
    PagedGeom g;
    const void *plan;
    const char *x[3];              // q, k, v; strides between tokens in bytes
    long x_stride[3];
    char *q_out;
    long q_out_stride;
    PagedCache cache[2];           // strides in bytes
    int heads[3], run[3], runs[3]; // heads (of q: 0 without queries), of a warp at a time; runs of a token
    const int *positions;
    const unsigned long long *turns;
    int seg1, seg2;
    const float *w[2];
    float eps;
    int *err;
};

template <typename TO, bool NORM>
__global__ void __launch_bounds__(256, BLOCKS_PER_SM) paged_append_kernel(const AppendArgs a) {
    using T = __nv_bfloat16;
    constexpr int D = 128, N = 8, NP = 4, LPH = 16;
    launch_next_kernel();
    wait_previous_kernel();
    const PagedPlan plan = paged_plan_at(const_cast<void *>(a.plan), a.g);
    const PagedHeader head = *plan.head;
    if (!paged_plan_ok(head, a.g)) {
        if (blockIdx.x == 0 && threadIdx.x == 0) atomicCAS(a.err, DEV_OK, DEV_PLAN);
        return;
    }
    const int lane = threadIdx.x & 31, sub = lane % LPH, grp = lane / LPH;
    // units: runs of q of the streams' tokens (the rows of others may hold anything), then of k, then of v
    const long tokens = head.q_hi - head.q_lo;
    const long units_q = tokens * a.runs[0], units_qk = units_q + tokens * a.runs[1], units = units_qk + tokens * a.runs[2];
    float top = 0.f;
    for (long u = (blockIdx.x * (long)blockDim.x + threadIdx.x) >> 5; u < units; u += ((long)gridDim.x * blockDim.x) >> 5) {
        const int kind = u < units_q ? 0 : u < units_qk ? 1 : 2;
        const unsigned v = (unsigned)(u - (kind == 0 ? 0 : kind == 1 ? units_q : units_qk));
        const unsigned t = a.runs[kind] == 1 ? v : v / (unsigned)a.runs[kind];
        const int h0 = (int)(v - t * a.runs[kind]) * a.run[kind], h1 = min(h0 + a.run[kind], a.heads[kind]);
        const long tok = (long)head.q_lo + t;
        const char *x0 = a.x[kind] + tok * a.x_stride[kind] + sub * 16;
        char *z0 = a.q_out + tok * a.q_out_stride + sub * 16;
        long step = ROW;
        if (kind > 0) {
            const int slot = plan.slot[tok];
            if (slot < 0) continue;  // more queries than keys, or a page that is not one (the plan reported it)
            const PagedCache &to = a.cache[kind - 1];
            const int page = slot / a.g.page, in = slot - page * a.g.page;
            z0 = static_cast<char *>(to.p) + (long)page * to.page + (long)in * to.token + sub * 16;
            step = to.head;
        }
        Turn<NP> turn;
        for (int hb = h0; hb < h1; hb += PASS) {
            uint4 raw[VECS];
#pragma unroll
            for (int i = 0; i < VECS; i++) {
                const int h = hb + grp + 2 * i;
                raw[i] = make_uint4(0, 0, 0, 0);
                if (h < h1) raw[i] = __ldcs(reinterpret_cast<const uint4 *>(x0 + (long)h * ROW));
            }
            if (kind == 2) {  // values as they are
#pragma unroll
                for (int i = 0; i < VECS; i++) {
                    const int h = hb + grp + 2 * i;
                    if (h < h1) __stcs(reinterpret_cast<uint4 *>(z0 + h * step), raw[i]);
                }
                continue;
            }
            if (hb == h0) {
                const int p3[3] = {a.positions[3 * tok], a.positions[3 * tok + 1], a.positions[3 * tok + 2]};
                float c[NP], s[NP], w[N];
                cos_sin_at<NP>(p3, a.turns, a.seg1, a.seg2, sub * NP, c, s);
#pragma unroll
                for (int k = 0; k < N; k++) w[k] = NORM ? a.w[kind][sub * N + k] : 1.f;
                turn.set(c, s, w);
            }
#pragma unroll
            for (int i = 0; i < VECS; i++) {
                float z[N];
                turned<T, D, NORM>(raw[i], turn, a.eps, z);
                const int h = hb + grp + 2 * i;
                if (h < h1) {
                    if constexpr (std::is_same<TO, __half>::value) {
#pragma unroll
                        for (int k = 0; k < NP; k++) top = max_abs(top, z[2 * k], z[2 * k + 1]);
                    }
                    __stcs(reinterpret_cast<uint4 *>(z0 + h * step), Row<TO>::pack(z));
                }
            }
        }
    }
    if constexpr (std::is_same<TO, __half>::value) {
        if (!(top < 65520.f)) atomicCAS(a.err, DEV_OK, DEV_RANGE);  // not a finite half
    }
}

}  // namespace

cudaError_t launch_paged_append(const Geom &g, const PagedGeom &p, const PagedAppend &t, k6attn_dtype out,
                                cudaStream_t st) {
    if (p.g.Tq == 0) return cudaSuccess;
    AppendArgs a = {};
    a.g = p, a.plan = t.plan;
    a.q_out = static_cast<char *>(t.q_out), a.q_out_stride = t.q_out_stride * 2;
    for (int c = 0; c < 2; c++) {
        a.cache[c] = {t.cache[c].p, t.cache[c].page * 2, t.cache[c].token * 2, t.cache[c].head * 2, 0};
        a.w[c] = t.w[c];
    }
    a.positions = t.positions, a.turns = t.turns;
    a.seg1 = g.axis_dim[0] / 2, a.seg2 = (g.axis_dim[0] + g.axis_dim[1]) / 2;
    a.eps = t.eps, a.err = t.err;
    long units = 0;
    for (int i = 0; i < 3; i++) {
        a.x[i] = static_cast<const char *>(t.x[i]), a.x_stride[i] = t.x_stride[i] * 2;
        a.heads[i] = i > 0 ? p.g.Hkv : t.x[0] ? g.H : 0;
        // see choose_runs of k6_packed_norm.cu
        const int whole = (a.heads[i] + PASS - 1) / PASS * PASS;
        a.run[i] = p.g.Tq >= WHOLE_FROM * p.g.sms && whole > 0 ? whole : PASS;
        a.runs[i] = (a.heads[i] + a.run[i] - 1) / a.run[i];
        units += (long)p.g.Tq * a.runs[i];
    }
    const long want = (units + 7) / 8, most = (long)p.g.sms * BLOCKS_PER_SM;
    auto launch = [&](auto kernel) {
        return launch_after(kernel, (unsigned)(want < most ? want : most), 256, 0, st, a);
    };
    const bool norm = t.w[1] != nullptr;
    if (out == K6ATTN_F16) return norm ? launch(paged_append_kernel<__half, true>) : launch(paged_append_kernel<__half, false>);
    return norm ? launch(paged_append_kernel<__nv_bfloat16, true>) : launch(paged_append_kernel<__nv_bfloat16, false>);
}

}  // namespace k6
