// k6_packed_norm.cu -- per-head RMS norm of queries and keys and the rotation by
// (t, h, w) positions in one pass over packed token rows, and its gradient.
//
// For a token with positions p_a and a head row x of d values,
//   r = (mean(x^2) + eps)^(-1/2),   y = x r w   (y = x without weights),
//   (z_2i, z_2i+1) = (y_2i c_i - y_2i+1 s_i, y_2i s_i + y_2i+1 c_i),
// pair i of the segment of axis a turning by p_a theta^(-2i/d_a) ("Context
// Parallelism in vLLM Omni Neuron", "Self-Attention with Context Parallelism":
// QK-norm, then the rotary embedding).  Backward, with gz the gradient of z:
//   gy = R^T gz,   dw = sum over tokens and heads of gy x r,
//   g = gy w,   dx = r (g - x r mean(g x r)).
// Statistics, angles and sums are fp32 or wider; the one rounding is that of
// each output element to its type.
//
// Angles: the frequency of a pair is kept as a 64-bit fixed-point fraction of a
// turn, so position * frequency modulo 2^64 is the reduced angle with an error
// below |position| 2^-55 turns, at any 32-bit position, in integer arithmetic;
// its top 32 bits go to sincospi as a float, which costs up to 2^-26 of a turn
// (2^-23.4 in the angle, the size of sin and cos's own rounding) near half a turn.
// No per-token table is read: 12 bytes of positions serve all heads of a token.
//
// Bound by HBM: each element is read once and written once (backward: x and gz
// read, dx written).  A head row is 16 lanes (32 for 512-byte rows) of one
// 16-byte vector each, so its sum of squares is 4 (5) shuffles; a warp takes a
// run of a token's heads, computes its pairs' sin and cos once per run, and has
// several vectors a lane in flight.  52,360 tokens on one GB300: forward 24/8
// heads to fp16 145 us (5.9 TB/s, 87 % of a copy's), backward 24/24 heads 294 us
// (6.6 TB/s, 97 %).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "k6_device.cuh"
#include "k6_paged.cuh"

namespace k6 {

namespace {

// 16 bytes of a row as pairs (2k, 2k + 1) in fp32, and back.
template <typename T>
struct Row;
template <>
struct Row<__nv_bfloat16> {
    static constexpr int N = 8;
    __device__ static void unpack(const uint4 &u, uint64_t (&x)[4]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int k = 0; k < 4; k++) x[k] = f2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u));
    }
    __device__ static uint4 pack(const float (&x)[8]) {
        return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                          pack_bf16x2(x[6], x[7]));
    }
};
template <>
struct Row<__half> {
    __device__ static uint4 pack(const float (&x)[8]) {
        uint4 u;
        __half2 *b = reinterpret_cast<__half2 *>(&u);
#pragma unroll
        for (int k = 0; k < 4; k++) b[k] = __floats2half2_rn(x[2 * k], x[2 * k + 1]);
        return u;
    }
};
template <>
struct Row<float> {
    static constexpr int N = 4;
    __device__ static void unpack(const uint4 &u, uint64_t (&x)[2]) {
        x[0] = f2(__uint_as_float(u.x), __uint_as_float(u.y));
        x[1] = f2(__uint_as_float(u.z), __uint_as_float(u.w));
    }
    __device__ static uint4 pack(const float (&x)[4]) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
};

__device__ __forceinline__ uint64_t fmul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// The larger of m, |a| and |b|; NaN if one is.
__device__ __forceinline__ float max_abs(float m, float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(fabsf(a)), "f"(fabsf(b)));
    return r;
}

// Blocks of 256 threads resident on an SM: what the registers are bounded to, and the grid.
// Vectors that a lane has in flight (of x; in the backward pass of x and of gz each).  Measured at 52,360
// tokens, us: forward (24/8 heads) 4 vectors x 4 blocks 143, 6 x 3 143, 8 x 3 147, 3 x 5 205 (spills); 4 x 3
// with the next vectors loaded ahead 144.  Backward (24/24) 6 x 2 290, 4 x 2 309, 2 x 3 330, 8 x 2 325, and
// 2 x 2 with the next ones loaded ahead 390.
constexpr int FWD_BLOCKS_PER_SM = 4, BWD_BLOCKS_PER_SM = 2;
constexpr int FWD_VECS = 4, BWD_VECS = 6;

// Token rows of one tensor: `base`, and bytes from one token to the next.
struct Rows {
    char *base;
    long stride;
};

struct NormRopeArgs {
    long tokens;
    int heads[2];                  // query heads, key heads
    int run[2];                    // heads of a token that one warp takes at a time
    int runs[2];                   // runs of a token: ceil(heads / run)
    long units_q, units;           // runs over all tokens: of queries; and of keys behind them
    Rows x[2], z[2];               // [0] queries, [1] keys.  z: the output, or its gradient
    Rows dx[2];
    const int *positions;          // [tokens][3]
    const int *cu;                 // [n_seq + 1] offsets: only the tokens between the first and the last; or null
    int n_seq;
    const unsigned long long *turns;
    int seg1, seg2;                // first pair of the h and w axes
    const float *w[2];             // [d] each, or null: no norm
    float eps;
    float *part;                   // backward: [blocks][2][d] partial sums of the weights' gradients
    int *err;
};

// cos and sin of the NP pairs from pair0 on, at a token's positions.  The
// frequencies are re-read (L1) rather than kept: 2 NP registers less a lane.
// No load here takes the non-coherent path: a kernel that begins while the one
// before it ends may read what that one wrote.
template <int NP>
__device__ __forceinline__ void cos_sin(const NormRopeArgs &a, long tok, int pair0, float (&c)[NP], float (&s)[NP]) {
    const int p0 = a.positions[3 * tok], p1 = a.positions[3 * tok + 1], p2 = a.positions[3 * tok + 2];
#pragma unroll
    for (int k = 0; k < NP; k++) {
        const int p = pair0 + k < a.seg1 ? p0 : pair0 + k < a.seg2 ? p1 : p2;
        const unsigned long long turns = a.turns[pair0 + k];
        const int top = (int)(((unsigned long long)(long long)p * turns) >> 32);  // in [-1/2, 1/2) turns
        sincospif((float)top * 0x1p-31f, &s[k], &c[k]);
    }
}

// The tokens that belong to a sequence, [r[0], r[1]), where offsets say.  The whole block.
__device__ __forceinline__ void token_range(const NormRopeArgs &a, int (&r)[2]) {
    if (!a.cu) return;
    if (threadIdx.x == 0) r[0] = __ldg(a.cu), r[1] = __ldg(a.cu + a.n_seq);
    __syncthreads();
}

// Unit u: which tensor, token, first head and end.
struct Unit {
    int t, h0, h1;
    long tok;
};
__device__ __forceinline__ Unit unit_at(const NormRopeArgs &a, long u) {
    Unit r;
    r.t = u >= a.units_q;
    if (r.t) u -= a.units_q;
    r.tok = a.runs[r.t] == 1 ? u : u / a.runs[r.t];
    r.h0 = (int)(u - r.tok * a.runs[r.t]) * a.run[r.t];
    r.h1 = min(r.h0 + a.run[r.t], a.heads[r.t]);
    return r;
}

template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// What turns and weighs the NP pairs of a lane at a unit's token, p: a pair becomes
// z = r (x0 p0 - x1 p1, x0 p2 + x1 p3), the weights times cos and sin.
template <int NP, bool NORM>
__device__ __forceinline__ void turn_and_weigh(const NormRopeArgs &a, const Unit &un, int sub, float (&p)[NP][4]) {
    float c[NP], s[NP];
    cos_sin<NP>(a, un.tok, sub * NP, c, s);
#pragma unroll
    for (int k = 0; k < NP; k++) {
        float w0 = 1.f, w1 = 1.f;
        if constexpr (NORM) {
            w0 = a.w[un.t][sub * 2 * NP + 2 * k];
            w1 = a.w[un.t][sub * 2 * NP + 2 * k + 1];
        }
        p[k][0] = w0 * c[k], p[k][1] = w1 * s[k], p[k][2] = w0 * s[k], p[k][3] = w1 * c[k];
    }
}

// A lane's vector of a head row: normed by the row's lanes, weighed and turned.
template <typename T, int D, bool NORM, int NP>
__device__ __forceinline__ void turned(const uint4 &raw, const float (&p)[NP][4], float eps, float (&z)[2 * NP]) {
    uint64_t x[NP];
    Row<T>::unpack(raw, x);
    if constexpr (NORM) {
        uint64_t ss = fmul2(x[0], x[0]);
#pragma unroll
        for (int k = 1; k < NP; k++) ss = ffma2(x[k], x[k], ss);
        float s0, s1;
        f2_split(ss, s0, s1);
        const float r = rsqrtf(lanes_sum<D / (2 * NP)>(s0 + s1) * (1.f / D) + eps);
#pragma unroll
        for (int k = 0; k < NP; k++) x[k] = fmul2(x[k], f2(r, r));
    }
#pragma unroll
    for (int k = 0; k < NP; k++) {
        float x0, x1;
        f2_split(x[k], x0, x1);
        z[2 * k] = x0 * p[k][0] - x1 * p[k][1];
        z[2 * k + 1] = x0 * p[k][2] + x1 * p[k][3];
    }
}

// D = head dim, T = element type of the rows, TO = of the output.
template <typename T, typename TO, int D, bool NORM>
__global__ void __launch_bounds__(256, FWD_BLOCKS_PER_SM) packed_norm_rope_kernel(const NormRopeArgs a) {
    constexpr int N = Row<T>::N, NP = N / 2;
    constexpr int LPH = D / N;       // lanes of a head row
    constexpr int HPW = 32 / LPH;    // heads a warp handles side by side
    constexpr int kU = FWD_VECS;
    constexpr int ROW = D * sizeof(T);
    static_assert(sizeof(T) == sizeof(TO), "rows keep their element size");
    const int lane = threadIdx.x & 31, sub = lane % LPH, grp = lane / LPH;
    const long nwarps = ((long)gridDim.x * blockDim.x) >> 5;
    float top = 0.f;
    __shared__ int range[2];
    token_range(a, range);
    for (long u = (blockIdx.x * (long)blockDim.x + threadIdx.x) >> 5; u < a.units; u += nwarps) {
        const Unit un = unit_at(a, u);
        if (a.cu && (un.tok < range[0] || un.tok >= range[1])) continue;  // padding: whatever it holds
        const char *x0 = a.x[un.t].base + un.tok * a.x[un.t].stride + sub * 16;
        char *z0 = a.z[un.t].base + un.tok * a.z[un.t].stride + sub * 16;
        float p[NP][4];
        for (int hb = un.h0; hb < un.h1; hb += HPW * kU) {
            uint4 raw[kU];
#pragma unroll
            for (int i = 0; i < kU; i++) {
                const int h = hb + grp + i * HPW;
                raw[i] = make_uint4(0, 0, 0, 0);
                if (h < un.h1) raw[i] = __ldcs(reinterpret_cast<const uint4 *>(x0 + (long)h * ROW));
            }
            if (hb == un.h0) turn_and_weigh<NP, NORM>(a, un, sub, p);
#pragma unroll
            for (int i = 0; i < kU; i++) {
                float z[N];
                turned<T, D, NORM>(raw[i], p, a.eps, z);
                const int h = hb + grp + i * HPW;
                if (h < un.h1) {
                    if constexpr (std::is_same<TO, __half>::value) {
#pragma unroll
                        for (int k = 0; k < NP; k++) top = max_abs(top, z[2 * k], z[2 * k + 1]);
                    }
                    __stcs(reinterpret_cast<uint4 *>(z0 + (long)h * ROW), Row<TO>::pack(z));
                }
            }
        }
    }
    if constexpr (std::is_same<TO, __half>::value) {
        if (!(top < 65520.f)) atomicCAS(a.err, DEV_OK, DEV_RANGE);  // not a finite half
    }
}

// New tokens over a cache of pages: q as above; k as above, but to the place in the
// pages that the plan gives the token; v as it is, beside it.
struct AppendArgs {
    NormRopeArgs n;                // of q, k, v: x; z[0] the rotated queries
    PagedGeom g;
    const void *plan;
    int heads_v, run_v, runs_v;
    long units_qk;                 // runs of q and k; those of v behind them up to n.units
    Rows v;
    PagedCache cache[2];           // strides in bytes
};

// A token's place: byte offset of head 0 in cache c.
__device__ __forceinline__ long cache_at(const AppendArgs &a, int c, int slot) {
    const int page = slot / a.g.page, tok = slot - page * a.g.page;
    return (long)page * a.cache[c].page + (long)tok * a.cache[c].token;
}

template <typename TO, bool NORM>
__global__ void __launch_bounds__(256, FWD_BLOCKS_PER_SM) paged_append_kernel(const AppendArgs a) {
    using T = __nv_bfloat16;
    constexpr int D = 128, N = 8, NP = N / 2, LPH = D / N, HPW = 32 / LPH, kU = FWD_VECS, ROW = D * sizeof(T);
    launch_next_kernel();
    wait_previous_kernel();
    const PagedPlan plan = paged_plan_at(const_cast<void *>(a.plan), a.g);
    const PagedHeader head = *plan.head;
    if (!paged_plan_ok(head, a.g)) {
        if (blockIdx.x == 0 && threadIdx.x == 0) atomicCAS(a.n.err, DEV_OK, DEV_PLAN);
        return;
    }
    const int lane = threadIdx.x & 31, sub = lane % LPH, grp = lane / LPH;
    const long nwarps = ((long)gridDim.x * blockDim.x) >> 5;
    float top = 0.f;
    for (long u = (blockIdx.x * (long)blockDim.x + threadIdx.x) >> 5; u < a.n.units; u += nwarps) {
        Unit un;
        if (u < a.units_qk) {
            un = unit_at(a.n, u);
        } else {
            const long w = u - a.units_qk;
            un.t = 2;
            un.tok = a.runs_v == 1 ? w : w / a.runs_v;
            un.h0 = (int)(w - un.tok * a.runs_v) * a.run_v;
            un.h1 = min(un.h0 + a.run_v, a.heads_v);
        }
        if (un.tok < head.q_lo || un.tok >= head.q_hi) continue;  // padding: whatever it holds
        const Rows x = un.t == 2 ? a.v : a.n.x[un.t];
        const char *x0 = x.base + un.tok * x.stride + sub * 16;
        char *z0;
        long step = ROW;
        if (un.t == 0) {
            z0 = a.n.z[0].base + un.tok * a.n.z[0].stride + sub * 16;
        } else {
            const int slot = plan.slot[un.tok];
            if (slot < 0) continue;  // more queries than keys, or a page that is not one (the plan reported it)
            z0 = static_cast<char *>(a.cache[un.t - 1].p) + cache_at(a, un.t - 1, slot) + sub * 16;
            step = a.cache[un.t - 1].head;
        }
        if (un.t == 2) {
            for (int hb = un.h0; hb < un.h1; hb += HPW * kU) {
                uint4 raw[kU];
#pragma unroll
                for (int i = 0; i < kU; i++) {
                    const int h = hb + grp + i * HPW;
                    if (h < un.h1) raw[i] = __ldcs(reinterpret_cast<const uint4 *>(x0 + (long)h * ROW));
                }
#pragma unroll
                for (int i = 0; i < kU; i++) {
                    const int h = hb + grp + i * HPW;
                    if (h < un.h1) *reinterpret_cast<uint4 *>(z0 + h * step) = raw[i];
                }
            }
            continue;
        }
        float p[NP][4];
        for (int hb = un.h0; hb < un.h1; hb += HPW * kU) {
            uint4 raw[kU];
#pragma unroll
            for (int i = 0; i < kU; i++) {
                const int h = hb + grp + i * HPW;
                raw[i] = make_uint4(0, 0, 0, 0);
                if (h < un.h1) raw[i] = __ldcs(reinterpret_cast<const uint4 *>(x0 + (long)h * ROW));
            }
            if (hb == un.h0) turn_and_weigh<NP, NORM>(a.n, un, sub, p);
#pragma unroll
            for (int i = 0; i < kU; i++) {
                float z[N];
                turned<T, D, NORM>(raw[i], p, a.n.eps, z);
                const int h = hb + grp + i * HPW;
                if (h < un.h1) {
                    if constexpr (std::is_same<TO, __half>::value) {
#pragma unroll
                        for (int k = 0; k < NP; k++) top = max_abs(top, z[2 * k], z[2 * k + 1]);
                    }
                    *reinterpret_cast<uint4 *>(z0 + h * step) = Row<TO>::pack(z);
                }
            }
        }
    }
    if constexpr (std::is_same<TO, __half>::value) {
        if (!(top < 65520.f)) atomicCAS(a.n.err, DEV_OK, DEV_RANGE);  // not a finite half
    }
}

// The gradient: dx, and this block's partial sums of dw in a.part[block][2][D].
// A lane owns the same N dims of every head it meets, so dw is a running sum in
// its registers (first over the warp's units of queries, then over those of
// keys); lanes and warps of the block are joined through shared memory in a
// fixed order, and blocks by packed_norm_dw_kernel, so that the result does not
// depend on timing.
template <typename T, int D, bool NORM>
__global__ void __launch_bounds__(256, BWD_BLOCKS_PER_SM) packed_norm_rope_bwd_kernel(const NormRopeArgs a) {
    constexpr int N = Row<T>::N, NP = N / 2;
    constexpr int LPH = D / N, HPW = 32 / LPH;
    constexpr int kU = BWD_VECS;
    constexpr int ROW = D * sizeof(T);
    __shared__ float sum[8][2][D];
    const int lane = threadIdx.x & 31, sub = lane % LPH, grp = lane / LPH, warp = threadIdx.x >> 5;
    const long warp0 = (blockIdx.x * (long)blockDim.x + threadIdx.x) >> 5;
    const long nwarps = ((long)gridDim.x * blockDim.x) >> 5;
    uint64_t acc[NP];
#pragma unroll
    for (int k = 0; k < NP; k++) acc[k] = 0;
    auto flush = [&](int t) {
#pragma unroll
        for (int k = 0; k < NP; k++) {
            float v[2];
            f2_split(acc[k], v[0], v[1]);
#pragma unroll
            for (int e = 0; e < 2; e++) {
#pragma unroll
                for (int o = 16; o >= LPH; o >>= 1) v[e] += __shfl_xor_sync(0xffffffffu, v[e], o);
                if (grp == 0) sum[warp][t][sub * N + 2 * k + e] = v[e];
            }
            acc[k] = 0;
        }
    };
    int met = 0;  // the tensor that acc belongs to
    __shared__ int range[2];
    token_range(a, range);
    for (long u = warp0; u < a.units; u += nwarps) {
        const Unit un = unit_at(a, u);
        if (a.cu && (un.tok < range[0] || un.tok >= range[1])) continue;  // padding: whatever it holds
        const char *x0 = a.x[un.t].base + un.tok * a.x[un.t].stride + sub * 16;
        const char *z0 = a.z[un.t].base + un.tok * a.z[un.t].stride + sub * 16;
        char *d0 = a.dx[un.t].base + un.tok * a.dx[un.t].stride + sub * 16;
        float c[NP], s[NP];
        uint64_t w[NP];
        for (int hb = un.h0; hb < un.h1; hb += HPW * kU) {
            uint4 rx[kU], rg[kU];
#pragma unroll
            for (int i = 0; i < kU; i++) {
                const int h = hb + grp + i * HPW;
                rx[i] = rg[i] = make_uint4(0, 0, 0, 0);
                if (h < un.h1) {
                    rg[i] = __ldcs(reinterpret_cast<const uint4 *>(z0 + (long)h * ROW));
                    if constexpr (NORM) rx[i] = __ldcs(reinterpret_cast<const uint4 *>(x0 + (long)h * ROW));
                }
            }
            if (hb == un.h0) {
                if constexpr (NORM) {
                    if (un.t != met) flush(0);
#pragma unroll
                    for (int k = 0; k < NP; k++)
                        w[k] = f2(__ldg(a.w[un.t] + sub * N + 2 * k), __ldg(a.w[un.t] + sub * N + 2 * k + 1));
                }
                met = un.t;
                cos_sin<NP>(a, un.tok, sub * NP, c, s);
            }
#pragma unroll
            for (int i = 0; i < kU; i++) {
                const int h = hb + grp + i * HPW;
                const bool live = h < un.h1;
                uint64_t g[NP];
                Row<T>::unpack(rg[i], g);
#pragma unroll
                for (int k = 0; k < NP; k++) {  // the rotation turned back
                    float re, im;
                    f2_split(g[k], re, im);
                    g[k] = f2(re * c[k] + im * s[k], im * c[k] - re * s[k]);
                }
                if constexpr (NORM) {
                    uint64_t x[NP], gw[NP];
                    Row<T>::unpack(rx[i], x);
#pragma unroll
                    for (int k = 0; k < NP; k++) gw[k] = fmul2(g[k], w[k]);
                    uint64_t ss = fmul2(x[0], x[0]), gx = fmul2(gw[0], x[0]);
#pragma unroll
                    for (int k = 1; k < NP; k++) ss = ffma2(x[k], x[k], ss), gx = ffma2(gw[k], x[k], gx);
                    float s0, s1, g0, g1;
                    f2_split(ss, s0, s1);
                    f2_split(gx, g0, g1);
                    const float r = rsqrtf(lanes_sum<LPH>(s0 + s1) * (1.f / D) + a.eps);
                    const float m = lanes_sum<LPH>(g0 + g1) * (1.f / D) * r;  // mean of g x r
                    if (live) {  // a lane past the run holds zeros, whose r may be infinite
#pragma unroll
                        for (int k = 0; k < NP; k++) {
                            const uint64_t xh = fmul2(x[k], f2(r, r));
                            acc[k] = ffma2(g[k], xh, acc[k]);
                            g[k] = fmul2(ffma2(xh, f2(-m, -m), gw[k]), f2(r, r));
                        }
                    }
                }
                if (live) {
                    float d[N];
#pragma unroll
                    for (int k = 0; k < NP; k++) f2_split(g[k], d[2 * k], d[2 * k + 1]);
                    __stcs(reinterpret_cast<uint4 *>(d0 + (long)h * ROW), Row<T>::pack(d));
                }
            }
        }
    }
    if constexpr (NORM) {
        flush(met);
        // a warp that met one tensor only has nothing of the other
        const bool both = met == 1 && warp0 < a.units_q;
        if (!both)
            for (int i = lane; i < D; i += 32) sum[warp][met ^ 1][i] = 0.f;
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * D; i += 256) {
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < 8; w++) v += sum[w][i / D][i % D];
            a.part[(long)blockIdx.x * 2 * D + i] = v;
        }
    }
}

// dw[t][e] = sum over blocks of part[block][t][e], in a fixed order.  One block
// per 32 columns; a warp per slice of the blocks, its lanes the columns.
__global__ void __launch_bounds__(1024) packed_norm_dw_kernel(const float *part, int blocks, int D,
                                                              float *__restrict__ dq_w, float *__restrict__ dk_w) {
    wait_previous_kernel();
    __shared__ float sum[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;
    float v = 0.f;
#pragma unroll 8
    for (int b = warp; b < blocks; b += 32) v += part[(long)b * 2 * D + col];
    sum[warp][lane] = v;
    __syncthreads();
    if (warp == 0) {
        v = 0.f;
#pragma unroll
        for (int w = 0; w < 32; w++) v += sum[w][lane];
        if (col < D) dq_w[col] = v;
        else dk_w[col - D] = v;
    }
}

NormRopeArgs norm_args(const Geom &g, const PackedNormRope &p) {
    NormRopeArgs a = {};
    a.tokens = p.tokens;
    a.heads[0] = g.H, a.heads[1] = p.Hkv;
    for (int t = 0; t < 2; t++) {
        a.x[t] = {static_cast<char *>(const_cast<void *>(p.x[t])), p.x_stride[t] * g.elem};
        a.z[t] = {static_cast<char *>(p.z[t]), p.z_stride[t] * g.elem};
        a.dx[t] = {static_cast<char *>(p.dx[t]), p.dx_stride[t] * g.elem};
        a.w[t] = p.w[t];
    }
    a.positions = p.positions;
    a.cu = p.cu, a.n_seq = p.n_seq;
    a.turns = p.turns;
    a.seg1 = g.axis_dim[0] / 2;
    a.seg2 = (g.axis_dim[0] + g.axis_dim[1]) / 2;
    a.eps = p.eps;
    a.err = p.err;
    return a;
}

// A token's heads go to one warp when there are tokens enough to fill the GPU;
// with fewer, each warp takes one pass of `pass` heads, so that a few tokens
// still spread over the SMs (the sin and cos are then computed once per pass).
// Whole tokens against passes, us in a graph, 24/8 heads: 300 tokens forward 5.9
// and 3.5, 1,000 6.9 and 5.5, 2,432 9.6 and 9.6, 12,000 34.1 and 36.2; backward
// 300 8.6 and 7.1, 2,432 16.3 and 17.1, 12,000 55.0 and 57.6.
void choose_runs(NormRopeArgs &a, int pass, int sms) {
    for (int t = 0; t < 2; t++) {
        a.run[t] = a.tokens >= 16L * sms && a.heads[t] > 0 ? (a.heads[t] + pass - 1) / pass * pass : pass;
        a.runs[t] = (a.heads[t] + a.run[t] - 1) / a.run[t];
    }
    a.units_q = a.tokens * a.runs[0];
    a.units = a.units_q + a.tokens * a.runs[1];
}

// Blocks of 256 threads: at most `per_sm` a SM, at most one unit per warp.
long norm_blocks(const NormRopeArgs &a, int per_sm, int sms) {
    const long want = (a.units + 7) / 8, wave = (long)sms * per_sm;
    return want < wave ? want : wave;
}

}  // namespace

cudaError_t launch_paged_append(const Geom &g, const PagedGeom &p, const PagedAppend &t, k6attn_dtype out,
                                cudaStream_t st) {
    if (p.g.Tq == 0) return cudaSuccess;
    AppendArgs a = {};
    a.n.tokens = p.g.Tq;
    a.n.heads[0] = t.x[0] ? g.H : 0, a.n.heads[1] = p.g.Hkv, a.heads_v = p.g.Hkv;
    auto rows = [&](const void *x, long stride) { return Rows{static_cast<char *>(const_cast<void *>(x)), stride * 2}; };
    a.n.x[0] = rows(t.x[0], t.x_stride[0]), a.n.x[1] = rows(t.x[1], t.x_stride[1]), a.v = rows(t.x[2], t.x_stride[2]);
    a.n.z[0] = rows(t.q_out, t.q_out_stride);
    for (int c = 0; c < 2; c++)
        a.cache[c] = {t.cache[c].p, t.cache[c].page * 2, t.cache[c].token * 2, t.cache[c].head * 2, 0}, a.n.w[c] = t.w[c];
    a.n.positions = t.positions, a.n.turns = t.turns;
    a.n.seg1 = g.axis_dim[0] / 2, a.n.seg2 = (g.axis_dim[0] + g.axis_dim[1]) / 2;
    a.n.eps = t.eps, a.n.err = t.err;
    a.g = p, a.plan = t.plan;
    const int pass = FWD_VECS * 32 * 8 / 128;
    choose_runs(a.n, pass, p.g.sms);
    a.run_v = a.n.run[1], a.runs_v = a.n.runs[1];
    a.units_qk = a.n.units;
    a.n.units += a.n.tokens * a.runs_v;
    auto launch = [&](auto kernel) {
        return launch_after(kernel, (unsigned)norm_blocks(a.n, FWD_BLOCKS_PER_SM, p.g.sms), 256, 0, st, a);
    };
    const bool norm = t.w[0] || t.w[1];
    if (out == K6ATTN_F16) return norm ? launch(paged_append_kernel<__half, true>) : launch(paged_append_kernel<__half, false>);
    return norm ? launch(paged_append_kernel<__nv_bfloat16, true>) : launch(paged_append_kernel<__nv_bfloat16, false>);
}

size_t packed_norm_rope_bwd_workspace(const Geom &g, long tokens, int sms) {
    if (tokens <= 0) return 0;
    return (size_t)sms * BWD_BLOCKS_PER_SM * 2 * g.d * sizeof(float);
}

cudaError_t launch_packed_norm_rope(const Geom &g, const PackedNormRope &p, k6attn_dtype out, cudaStream_t st) {
    if (p.tokens == 0) return cudaSuccess;
    NormRopeArgs a = norm_args(g, p);
    const int sms = p.sms;
    auto launch = [&](auto kernel, int vec) {
        choose_runs(a, FWD_VECS * 32 * vec / g.d, sms);
        kernel<<<(unsigned)norm_blocks(a, FWD_BLOCKS_PER_SM, sms), 256, 0, st>>>(a);
    };
    const bool norm = p.w[0] != nullptr;
    if (g.dtype == K6ATTN_F32 && g.d == 128)
        norm ? launch(packed_norm_rope_kernel<float, float, 128, true>, 4)
             : launch(packed_norm_rope_kernel<float, float, 128, false>, 4);
    else if (g.dtype == K6ATTN_F32)
        norm ? launch(packed_norm_rope_kernel<float, float, 64, true>, 4)
             : launch(packed_norm_rope_kernel<float, float, 64, false>, 4);
    else if (out == K6ATTN_F16)
        norm ? launch(packed_norm_rope_kernel<__nv_bfloat16, __half, 128, true>, 8)
             : launch(packed_norm_rope_kernel<__nv_bfloat16, __half, 128, false>, 8);
    else
        norm ? launch(packed_norm_rope_kernel<__nv_bfloat16, __nv_bfloat16, 128, true>, 8)
             : launch(packed_norm_rope_kernel<__nv_bfloat16, __nv_bfloat16, 128, false>, 8);
    return cudaGetLastError();
}

cudaError_t launch_packed_norm_rope_bwd(const Geom &g, const PackedNormRope &p, float *dq_w, float *dk_w, void *ws,
                                        cudaStream_t st) {
    const bool norm = p.w[0] != nullptr;
    if (p.tokens == 0) {
        cudaError_t e = cudaSuccess;
        if (norm) e = cudaMemsetAsync(dq_w, 0, g.d * sizeof(float), st);
        if (norm && e == cudaSuccess) e = cudaMemsetAsync(dk_w, 0, g.d * sizeof(float), st);
        return e;
    }
    NormRopeArgs a = norm_args(g, p);
    a.part = static_cast<float *>(ws);
    const int sms = p.sms;
    long blocks = 0;
    auto launch = [&](auto kernel, int vec) {
        choose_runs(a, BWD_VECS * 32 * vec / g.d, sms);
        blocks = norm_blocks(a, BWD_BLOCKS_PER_SM, sms);
        kernel<<<(unsigned)blocks, 256, 0, st>>>(a);
    };
    if (g.dtype == K6ATTN_F32 && g.d == 128)
        norm ? launch(packed_norm_rope_bwd_kernel<float, 128, true>, 4)
             : launch(packed_norm_rope_bwd_kernel<float, 128, false>, 4);
    else if (g.dtype == K6ATTN_F32)
        norm ? launch(packed_norm_rope_bwd_kernel<float, 64, true>, 4)
             : launch(packed_norm_rope_bwd_kernel<float, 64, false>, 4);
    else
        norm ? launch(packed_norm_rope_bwd_kernel<__nv_bfloat16, 128, true>, 8)
             : launch(packed_norm_rope_bwd_kernel<__nv_bfloat16, 128, false>, 8);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !norm) return e;
    return launch_after(packed_norm_dw_kernel, 2 * g.d / 32, 1024, 0, st, a.part, (int)blocks, g.d, dq_w, dk_w);
}

}  // namespace k6
