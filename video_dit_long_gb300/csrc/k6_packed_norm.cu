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
// its top 32 bits go to sincospi.  No per-token table is read: 12 bytes of
// positions serve all heads of a token.
//
// Bound by HBM: each element is read once and written once (backward: x and gz
// read, dx written).  A head row is 16 lanes (32 for 512-byte rows) of one
// 16-byte vector each, so its sum of squares is 4 (5) shuffles; a warp takes a
// run of a token's heads, kU vectors in flight per lane, and computes its
// pairs' sin and cos once per run.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "k6_device.cuh"
#include "k6_internal.h"

namespace k6 {

namespace {

template <typename T>
struct Row;
template <>
struct Row<__nv_bfloat16> {
    static constexpr int N = 8;
    __device__ static void unpack(const uint4 &u, float (&x)[8]) {
        const __nv_bfloat162 *b = reinterpret_cast<const __nv_bfloat162 *>(&u);
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const float2 f = __bfloat1622float2(b[k]);
            x[2 * k] = f.x, x[2 * k + 1] = f.y;
        }
    }
    __device__ static uint4 pack(const float (&x)[8]) {
        return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                          pack_bf16x2(x[6], x[7]));
    }
};
template <>
struct Row<__half> {
    static constexpr int N = 8;
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
    __device__ static void unpack(const uint4 &u, float (&x)[4]) {
        x[0] = __uint_as_float(u.x), x[1] = __uint_as_float(u.y), x[2] = __uint_as_float(u.z),
        x[3] = __uint_as_float(u.w);
    }
    __device__ static uint4 pack(const float (&x)[4]) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
};

// Token rows of one tensor: `base`, and bytes from one token to the next.
struct Rows {
    char *base;
    long stride;
};

struct NormRopeArgs {
    long tokens;
    int H, heads;                  // query heads; query and key heads together
    int run;                       // heads of a token that one warp takes at a time
    int runs;                      // runs of a token: ceil(heads / run)
    Rows x[2], z[2];               // [0] queries, [1] keys.  z: the output, or its gradient
    Rows dx[2];
    const int *positions;          // [tokens][3]
    const unsigned long long *turns;
    int seg1, seg2;                // first pair of the h and w axes
    const float *w[2];             // [d] each, or null: no norm
    float eps;
    float *part;                   // backward: [blocks][2][d] partial sums of the weights' gradients
    int *err;
};

// The angles of a lane's pairs.  turns and axis are fixed for the lane.
template <int NP>
struct Angles {
    unsigned long long turns[NP];
    int axis[NP];
    __device__ void init(const NormRopeArgs &a, int pair0) {
#pragma unroll
        for (int k = 0; k < NP; k++) {
            turns[k] = __ldg(a.turns + pair0 + k);
            axis[k] = pair0 + k < a.seg1 ? 0 : pair0 + k < a.seg2 ? 1 : 2;
        }
    }
    __device__ void cos_sin(const NormRopeArgs &a, long tok, float (&c)[NP], float (&s)[NP]) const {
        const int p0 = __ldg(a.positions + 3 * tok), p1 = __ldg(a.positions + 3 * tok + 1),
                  p2 = __ldg(a.positions + 3 * tok + 2);
#pragma unroll
        for (int k = 0; k < NP; k++) {
            const int p = axis[k] == 0 ? p0 : axis[k] == 1 ? p1 : p2;
            const int top = (int)(((unsigned long long)(long long)p * turns[k]) >> 32);  // in [-1/2, 1/2) turns
            sincospif((float)top * 0x1p-31f, &s[k], &c[k]);
        }
    }
};

template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// D = head dim, T = element type of the rows, TO = of the output.
template <typename T, typename TO, int D, bool NORM>
__global__ void __launch_bounds__(256) packed_norm_rope_kernel(const NormRopeArgs a) {
    constexpr int N = Row<T>::N, NP = N / 2;
    constexpr int LPH = D / N;       // lanes of a head row
    constexpr int HPW = 32 / LPH;    // heads a warp handles side by side
    constexpr int kU = 4;            // vectors in flight per lane
    static_assert(sizeof(T) == sizeof(TO), "rows keep their element size");
    const int lane = threadIdx.x & 31, sub = lane % LPH, grp = lane / LPH;
    const long warp0 = (blockIdx.x * (long)blockDim.x + threadIdx.x) >> 5;
    const long nwarps = ((long)gridDim.x * blockDim.x) >> 5;
    Angles<NP> ang;
    ang.init(a, sub * NP);
    float wq[N], wk[N];
    if constexpr (NORM) {
#pragma unroll
        for (int k = 0; k < N; k++) wq[k] = __ldg(a.w[0] + sub * N + k), wk[k] = __ldg(a.w[1] + sub * N + k);
    }
    bool bad = false;
    const long units = a.tokens * a.runs;
    for (long u = warp0; u < units; u += nwarps) {
        const long tok = a.runs == 1 ? u : u / a.runs;
        const int h0 = (int)(u - tok * a.runs) * a.run;
        const int h1 = min(h0 + a.run, a.heads);
        const char *xq = a.x[0].base + tok * a.x[0].stride + sub * 16, *xk = a.x[1].base + tok * a.x[1].stride + sub * 16;
        char *zq = a.z[0].base + tok * a.z[0].stride + sub * 16, *zk = a.z[1].base + tok * a.z[1].stride + sub * 16;
        float c[NP], s[NP];
        for (int hb = h0; hb < h1; hb += HPW * kU) {
            uint4 raw[kU];
#pragma unroll
            for (int i = 0; i < kU; i++) {
                const int hh = hb + i * HPW + grp;
                raw[i] = make_uint4(0, 0, 0, 0);
                if (hh < h1)
                    raw[i] = __ldcs(reinterpret_cast<const uint4 *>(hh < a.H ? xq + (long)hh * (D * sizeof(T))
                                                                             : xk + (long)(hh - a.H) * (D * sizeof(T))));
            }
            if (hb == h0) ang.cos_sin(a, tok, c, s);  // under the first loads
#pragma unroll
            for (int i = 0; i < kU; i++) {
                const int hh = hb + i * HPW + grp;
                float x[N];
                Row<T>::unpack(raw[i], x);
                if constexpr (NORM) {
                    float ss = 0.f;
#pragma unroll
                    for (int k = 0; k < N; k++) ss = fmaf(x[k], x[k], ss);
                    const float r = rsqrtf(lanes_sum<LPH>(ss) * (1.f / D) + a.eps);
                    const bool isq = hh < a.H;
#pragma unroll
                    for (int k = 0; k < N; k++) x[k] *= r * (isq ? wq[k] : wk[k]);
                }
#pragma unroll
                for (int k = 0; k < NP; k++) {
                    const float re = x[2 * k], im = x[2 * k + 1];
                    x[2 * k] = re * c[k] - im * s[k];
                    x[2 * k + 1] = re * s[k] + im * c[k];
                }
                if (hh < h1) {
                    if constexpr (std::is_same<TO, __half>::value) {
#pragma unroll
                        for (int k = 0; k < N; k++) bad |= !(fabsf(x[k]) < 65520.f);  // a finite half
                    }
                    *reinterpret_cast<uint4 *>(hh < a.H ? zq + (long)hh * (D * sizeof(T))
                                                        : zk + (long)(hh - a.H) * (D * sizeof(T))) = Row<TO>::pack(x);
                }
            }
        }
    }
    if (bad) atomicCAS(a.err, DEV_OK, DEV_RANGE);
}

// The gradient: dx, and this block's partial sums of dw in a.part[block][2][D].
// A lane owns the same N dims of every head it meets, so dw is a running sum in
// its registers; lanes and warps of the block are joined through shared memory
// in a fixed order, and blocks by packed_norm_dw_kernel, so that the result
// does not depend on timing.
template <typename T, int D, bool NORM>
__global__ void __launch_bounds__(256) packed_norm_rope_bwd_kernel(const NormRopeArgs a) {
    constexpr int N = Row<T>::N, NP = N / 2;
    constexpr int LPH = D / N, HPW = 32 / LPH;
    constexpr int kU = 2;
    const int lane = threadIdx.x & 31, sub = lane % LPH, grp = lane / LPH;
    const long warp0 = (blockIdx.x * (long)blockDim.x + threadIdx.x) >> 5;
    const long nwarps = ((long)gridDim.x * blockDim.x) >> 5;
    Angles<NP> ang;
    ang.init(a, sub * NP);
    float wq[N], wk[N], aq[N], ak[N];
#pragma unroll
    for (int k = 0; k < N; k++) {
        aq[k] = ak[k] = 0.f;
        if constexpr (NORM) wq[k] = __ldg(a.w[0] + sub * N + k), wk[k] = __ldg(a.w[1] + sub * N + k);
    }
    const long units = a.tokens * a.runs;
    for (long u = warp0; u < units; u += nwarps) {
        const long tok = a.runs == 1 ? u : u / a.runs;
        const int h0 = (int)(u - tok * a.runs) * a.run;
        const int h1 = min(h0 + a.run, a.heads);
        float c[NP], s[NP];
        for (int hb = h0; hb < h1; hb += HPW * kU) {
            uint4 rx[kU], rg[kU];
#pragma unroll
            for (int i = 0; i < kU; i++) {
                const int hh = hb + i * HPW + grp;
                const int t = hh < a.H ? 0 : 1;
                const long off = (long)(t ? hh - a.H : hh) * (D * sizeof(T)) + sub * 16;
                rx[i] = rg[i] = make_uint4(0, 0, 0, 0);
                if (hh < h1) {
                    rg[i] = __ldcs(reinterpret_cast<const uint4 *>(a.z[t].base + tok * a.z[t].stride + off));
                    if constexpr (NORM)
                        rx[i] = __ldcs(reinterpret_cast<const uint4 *>(a.x[t].base + tok * a.x[t].stride + off));
                }
            }
            if (hb == h0) ang.cos_sin(a, tok, c, s);
#pragma unroll
            for (int i = 0; i < kU; i++) {
                const int hh = hb + i * HPW + grp;
                const bool live = hh < h1, isq = hh < a.H;
                float g[N];
                Row<T>::unpack(rg[i], g);
#pragma unroll
                for (int k = 0; k < NP; k++) {  // the rotation turned back
                    const float re = g[2 * k], im = g[2 * k + 1];
                    g[2 * k] = re * c[k] + im * s[k];
                    g[2 * k + 1] = im * c[k] - re * s[k];
                }
                if constexpr (NORM) {
                    float x[N];
                    Row<T>::unpack(rx[i], x);
                    float ss = 0.f, gx = 0.f;
#pragma unroll
                    for (int k = 0; k < N; k++) {
                        ss = fmaf(x[k], x[k], ss);
                        gx = fmaf(g[k] * (isq ? wq[k] : wk[k]), x[k], gx);
                    }
                    const float r = rsqrtf(lanes_sum<LPH>(ss) * (1.f / D) + a.eps);
                    const float m = lanes_sum<LPH>(gx) * (1.f / D) * r;  // mean of g x r
                    if (live) {  // a lane past the run holds zeros, whose r may be infinite
#pragma unroll
                        for (int k = 0; k < N; k++) {
                            const float xh = x[k] * r;
                            if (isq) aq[k] = fmaf(g[k], xh, aq[k]);
                            else ak[k] = fmaf(g[k], xh, ak[k]);
                            g[k] = r * (g[k] * (isq ? wq[k] : wk[k]) - xh * m);
                        }
                    }
                }
                if (live) {
                    const int t = isq ? 0 : 1;
                    *reinterpret_cast<uint4 *>(a.dx[t].base + tok * a.dx[t].stride +
                                               (long)(t ? hh - a.H : hh) * (D * sizeof(T)) + sub * 16) =
                        Row<T>::pack(g);
                }
            }
        }
    }
    if constexpr (NORM) {
        __shared__ float sum[8][2][D];
        const int warp = threadIdx.x >> 5;
#pragma unroll
        for (int k = 0; k < N; k++) {
#pragma unroll
            for (int o = 16; o >= LPH; o >>= 1) {
                aq[k] += __shfl_xor_sync(0xffffffffu, aq[k], o);
                ak[k] += __shfl_xor_sync(0xffffffffu, ak[k], o);
            }
            if (grp == 0) sum[warp][0][sub * N + k] = aq[k], sum[warp][1][sub * N + k] = ak[k];
        }
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
__global__ void __launch_bounds__(1024) packed_norm_dw_kernel(const float *__restrict__ part, int blocks, int D,
                                                              float *__restrict__ dq_w, float *__restrict__ dk_w) {
    __shared__ float sum[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;
    float v = 0.f;
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
    a.H = g.H, a.heads = g.H + p.Hkv;
    for (int t = 0; t < 2; t++) {
        a.x[t] = {static_cast<char *>(const_cast<void *>(p.x[t])), p.x_stride[t] * g.elem};
        a.z[t] = {static_cast<char *>(p.z[t]), p.z_stride[t] * g.elem};
        a.dx[t] = {static_cast<char *>(p.dx[t]), p.dx_stride[t] * g.elem};
        a.w[t] = p.w[t];
    }
    a.positions = p.positions;
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
void choose_runs(NormRopeArgs &a, int pass, int sms) {
    a.run = a.tokens >= 16L * sms ? (a.heads + pass - 1) / pass * pass : pass;
    a.runs = (a.heads + a.run - 1) / a.run;
}

int sm_count() {
    int dev = 0, sms = 152;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms;
}

// Blocks of 256 threads: at most `per_sm` a SM, at most one unit per warp.
long norm_blocks(const NormRopeArgs &a, int per_sm, int sms) {
    const long want = (a.tokens * a.runs + 7) / 8, wave = (long)sms * per_sm;
    return want < wave ? want : wave;
}

constexpr int BWD_BLOCKS_PER_SM = 4;

}  // namespace

size_t packed_norm_rope_bwd_workspace(const Geom &g, long tokens) {
    if (tokens <= 0) return 0;
    return (size_t)sm_count() * BWD_BLOCKS_PER_SM * 2 * g.d * sizeof(float);
}

cudaError_t launch_packed_norm_rope(const Geom &g, const PackedNormRope &p, k6attn_dtype out, cudaStream_t st) {
    if (p.tokens == 0) return cudaSuccess;
    NormRopeArgs a = norm_args(g, p);
    const int sms = sm_count();
    auto launch = [&](auto kernel, int vec) {
        choose_runs(a, 4 * 32 * vec / g.d, sms);
        int per_sm = 1;
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, 256, 0);
        kernel<<<(unsigned)norm_blocks(a, per_sm > 0 ? per_sm : 1, sms), 256, 0, st>>>(a);
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
    const int sms = sm_count();
    long blocks = 0;
    auto launch = [&](auto kernel, int vec) {
        choose_runs(a, 2 * 32 * vec / g.d, sms);
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
    packed_norm_dw_kernel<<<2 * g.d / 32, 1024, 0, st>>>(a.part, (int)blocks, g.d, dq_w, dk_w);
    return cudaGetLastError();
}

}  // namespace k6
