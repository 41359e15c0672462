// k6_norm_rope.cuh -- what the kernels that norm and rotate head rows share: 16
// bytes of a row as fp32 pairs and back, a pair's angle, and a lane's part of a row.
//
// Angles: the frequency of a pair is kept as a 64-bit fixed-point fraction of a
// turn, so position * frequency modulo 2^64 is the reduced angle with an error
// below |position| 2^-55 turns, at any 32-bit position, in integer arithmetic;
// its top 32 bits go to sincospi as a float, which costs up to 2^-26 of a turn
// (2^-23.4 in the angle, the size of sin and cos's own rounding) near half a turn.
// No per-token table is read: 12 bytes of positions serve all heads of a token.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "k6_device.cuh"

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

// cos and sin of the NP pairs from pair0 on, at the positions p.  The frequencies
// are re-read (L1) rather than kept: 2 NP registers less a lane.
template <int NP>
__device__ __forceinline__ void cos_sin_at(const int (&p)[3], const unsigned long long *turns, int seg1, int seg2, int pair0,
                                           float (&c)[NP], float (&s)[NP]) {
#pragma unroll
    for (int k = 0; k < NP; k++) {
        const int at = pair0 + k < seg1 ? p[0] : pair0 + k < seg2 ? p[1] : p[2];
        const unsigned long long turn = __ldg(turns + pair0 + k);
        const int top = (int)(((unsigned long long)(long long)at * turn) >> 32);  // in [-1/2, 1/2) turns
        sincospif((float)top * 0x1p-31f, &s[k], &c[k]);
    }
}

template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// What turns and weighs a lane's NP pairs, two pairs to an operation: of pairs 2g and
// 2g + 1, w0 c, -w1 s, w0 s, w1 c.
template <int NP>
struct Turn {
    uint64_t p[NP / 2][4];
    // w: the lane's 2 NP weights
    __device__ __forceinline__ void set(const float (&c)[NP], const float (&s)[NP], const float (&w)[2 * NP]) {
        float e[NP][4];
#pragma unroll
        for (int k = 0; k < NP; k++) {
            const float w0 = w[2 * k], w1 = w[2 * k + 1];
            e[k][0] = w0 * c[k], e[k][1] = -(w1 * s[k]), e[k][2] = w0 * s[k], e[k][3] = w1 * c[k];
        }
#pragma unroll
        for (int g = 0; g < NP / 2; g++)
#pragma unroll
            for (int i = 0; i < 4; i++) p[g][i] = f2(e[2 * g][i], e[2 * g + 1][i]);
    }
};

// A lane's vector of a head row, normed by the row's lanes, weighed and turned.
template <typename T, int D, bool NORM, int NP>
__device__ __forceinline__ void turned(const uint4 &raw, const Turn<NP> &turn, float eps, float (&z)[2 * NP]) {
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
    for (int g = 0; g < NP / 2; g++) {
        float a0, a1, b0, b1;
        f2_split(x[2 * g], a0, a1);
        f2_split(x[2 * g + 1], b0, b1);
        const uint64_t x0 = f2(a0, b0), x1 = f2(a1, b1);
        f2_split(ffma2(x0, turn.p[g][0], fmul2(x1, turn.p[g][1])), z[4 * g], z[4 * g + 2]);
        f2_split(ffma2(x0, turn.p[g][2], fmul2(x1, turn.p[g][3])), z[4 * g + 1], z[4 * g + 3]);
    }
}

}  // namespace

}  // namespace k6
