// k6_paged_append.cu -- new tokens over a cache of pages: per-head QK-norm and
// rotation of queries and keys as k6_packed_norm.cu computes them, the keys and the
// values to the places in the pages that the plan gives their tokens.
//
// Bound by HBM: each row is read once and written once.  A head row is 16 lanes of
// one 16-byte vector; a warp takes a run of a token's heads of q, of k or of v, with
// several vectors a lane in flight, and computes its pairs' sin and cos once a run.
// Steps of few tokens are cut into one stretch of passes (8 heads) a warp, so that
// all warps end together: whole runs dealt out in strides left 2,669 tokens with four
// passes on some warps for 2.7 on average (24/4 heads 13.5 -> 10.7 us).  The rest is
// instructions: the products of the rotation go two to an instruction
// (52,360 tokens of 24/8 heads 188 us without, 174 with), and stores that are not
// kept in the caches give the reads more of them (169 us, 6.3 TB/s, 93 % of a copy's).
// Eight tokens take 2.9 us, start and the plan's header.
//
// Measured and not kept, us for 52,360 / 2,669 / 8 tokens, in strides (169 / 13.5 / 3.2): vectors x blocks 6 x 3 183 /
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
// Tokens an SM from which warps stride over the tokens' heads, where there are key heads for whole passes; a stretch of passes
// a warp below that.  Measured in a captured graph, us, strides / stretches, 8 tokens, 2,669, 8,000, 52,360: 24/8 heads 4.5 /
// 2.9, 12.8 / 12.0, 28.3 / 28.1, 170.5 / 171.5; 24/24 heads 4.7 / 3.0, 18.3 / 18.1, 48.2 / 52.0, 303 / 318; 24/4 heads 4.4 / 2.8,
// 11.9 / 10.8, 25.3 / 24.8, 154.3 / 143.8.
constexpr int STRIDE_FROM = 40;
constexpr int ROW = 256;          // bytes

struct AppendArgs {
    PagedGeom g;
    const void *plan;
    const char *x[3];              // q, k, v; strides between tokens in bytes
    long x_stride[3];
    char *q_out;
    long q_out_stride;
    PagedCache cache[2];           // strides in bytes
    int heads[3];                  // of q: 0 without queries
    unsigned q_passes, passes;     // of a token
    const int *positions;
    const unsigned long long *turns;
    int seg1, seg2;
    const float *w[2];
    float eps;
    int *err;
};

// A warp's runs: heads [h0, h1) of q (kind 0), k (1) or v (2) of a token.  STRIDE: all heads of a token's q, of all
// tokens in the warps' strides, then of k, then of v.  Else the passes (PASS heads at most) of the tokens, a token's q, k
// and v one behind another, are cut into one stretch a warp.
template <bool STRIDE>
struct Runs {
    unsigned at, end, t, r;  // units or passes; the token and the pass in it
    __device__ Runs(const AppendArgs &a, unsigned tokens) {
        const unsigned warps = gridDim.x * (blockDim.x / 32), w = (blockIdx.x * blockDim.x + threadIdx.x) / 32;
        if (STRIDE) {
            at = w, end = (a.q_passes > 0 ? 3 : 2) * tokens;
        } else {
            const unsigned all = tokens * a.passes, per = all / warps, more = all - per * warps;
            at = w * per + min(w, more), end = at + per + (w < more ? 1 : 0);
            t = at / a.passes, r = at - t * a.passes;
        }
    }
    __device__ bool next(const AppendArgs &a, unsigned tokens, int &kind, unsigned &tok, int &h0, int &h1) {
        if (at >= end) return false;
        if (STRIDE) {
            const unsigned third = (at >= tokens ? 1 : 0) + (at >= 2 * tokens ? 1 : 0);
            kind = (int)third + (a.q_passes > 0 ? 0 : 1);
            tok = at - third * tokens;
            h0 = 0, h1 = a.heads[kind];
            at += gridDim.x * (blockDim.x / 32);
        } else {
            const unsigned qk = (a.q_passes + a.passes) / 2;  // k and v have as many
            kind = r < a.q_passes ? 0 : r < qk ? 1 : 2;
            const unsigned begin = kind == 0 ? 0 : kind == 1 ? a.q_passes : qk;
            const unsigned border = kind == 0 ? a.q_passes : kind == 1 ? qk : a.passes, n = min(border - r, end - at);
            tok = t;
            h0 = (int)(r - begin) * PASS, h1 = min(h0 + (int)n * PASS, a.heads[kind]);
            at += n, r += n;
            if (r == a.passes) r = 0, t++;
        }
        return true;
    }
};

template <typename TO, bool NORM, bool STRIDE>
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
    const unsigned tokens = (unsigned)(head.q_hi - head.q_lo);  // the streams': the rows of others may hold anything
    Runs<STRIDE> runs(a, tokens);
    float top = 0.f;
    int kind, h0, h1;
    for (unsigned t; runs.next(a, tokens, kind, t, h0, h1);) {
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
    for (int i = 0; i < 3; i++) {
        a.x[i] = static_cast<const char *>(t.x[i]), a.x_stride[i] = t.x_stride[i] * 2;
        a.heads[i] = i > 0 ? p.g.Hkv : t.x[0] ? g.H : 0;
        a.passes += (a.heads[i] + PASS - 1) / PASS;
        if (i == 0) a.q_passes = a.passes;
    }
    const bool stride = p.g.Tq >= STRIDE_FROM * p.g.sms && p.g.Hkv >= PASS;
    const long want = ((long)p.g.Tq * a.passes + 7) / 8, most = (long)p.g.sms * BLOCKS_PER_SM;
    auto launch = [&](auto kernel) {
        return launch_after(kernel, (unsigned)(want < most ? want : most), 256, 0, st, a);
    };
    const bool norm = t.w[1] != nullptr;
    auto pick = [&](auto type) {
        using TO = decltype(type);
        if (stride) return norm ? launch(paged_append_kernel<TO, true, true>) : launch(paged_append_kernel<TO, false, true>);
        return norm ? launch(paged_append_kernel<TO, true, false>) : launch(paged_append_kernel<TO, false, false>);
    };
    return out == K6ATTN_F16 ? pick(__half()) : pick(__nv_bfloat16());
}

}  // namespace k6
