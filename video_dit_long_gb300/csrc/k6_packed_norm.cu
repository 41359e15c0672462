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
// Angles: k6_norm_rope.cuh.
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

#include "k6_internal.h"
#include "k6_norm_rope.cuh"

namespace k6 {

namespace {

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

// cos and sin of the NP pairs from pair0 on, at a token's positions.
template <int NP>
__device__ __forceinline__ void cos_sin(const NormRopeArgs &a, long tok, int pair0, float (&c)[NP], float (&s)[NP]) {
    const int p[3] = {__ldg(a.positions + 3 * tok), __ldg(a.positions + 3 * tok + 1), __ldg(a.positions + 3 * tok + 2)};
    cos_sin_at<NP>(p, a.turns, a.seg1, a.seg2, pair0, c, s);
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
        Turn<NP> turn;
        for (int hb = un.h0; hb < un.h1; hb += HPW * kU) {
            uint4 raw[kU];
#pragma unroll
            for (int i = 0; i < kU; i++) {
                const int h = hb + grp + i * HPW;
                raw[i] = make_uint4(0, 0, 0, 0);
                if (h < un.h1) raw[i] = __ldcs(reinterpret_cast<const uint4 *>(x0 + (long)h * ROW));
            }
            if (hb == un.h0) {
                float c[NP], s[NP], w[N];
                cos_sin<NP>(a, un.tok, sub * NP, c, s);
#pragma unroll
                for (int k = 0; k < N; k++) w[k] = NORM ? __ldg(a.w[un.t] + sub * N + k) : 1.f;
                turn.set(c, s, w);
            }
#pragma unroll
            for (int i = 0; i < kU; i++) {
                float z[N];
                turned<T, D, NORM>(raw[i], turn, a.eps, z);
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
        a.run[t] = a.tokens >= 16L * sms ? (a.heads[t] + pass - 1) / pass * pass : pass;
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
