// k6_packed_bwd.cu -- gradients of packed attention on tcgen05.
//
// Of out = softmax(S) V over the keys each row sees (k6_packed.cuh), S = Q K^T / sqrt(d):
//   D_i = sum_e dO_ie O_ie,   P = exp(S - lse),   dS = P o (dO V^T - D),
//   dV = P^T dO,   dQ = dS K / sqrt(d),   dK = dS^T Q / sqrt(d),
// dK and dV summed over the G query heads of a key head inside the accumulator:
// a tile of query rows holds 128 / G tokens of all G heads (one TMA box), so
// the sum over heads is part of the product over rows.  The two kinds of item
// follow the joint-sequence backward (one stationary 128-row tile per CTA, the
// other side streamed by TMA; warps 0-7 form P and dS, warp 8 copies, warp 9
// issues the MMAs), walking the plan's lists: query tiles over the key tiles
// below their limit (dq), key tiles over the query tiles that see them
// (dk, dv), heaviest first, in one grid.  Each output row is written by one CTA: no atomics,
// the same bits every run.
//
// Streamed tiles that reach past their sequence hold another sequence's rows
// (or unwritten memory, or NaN): the MMA warp zeroes those rows in shared
// memory before they enter a product over rows, since 0 * NaN is not 0.
//
// fp16 q/k: dS must have K's and Q's type, and gradients are often far below
// fp16's 2^-24.  |dS_ij| <= |dO_i| |v_j| + |D_i|, so each row of an accumulator is
// carried times a power of two of its own that brings this bound to 2^15, and the
// epilogue takes it out again (exact): a row of dQ takes |dO_i|, |D_i| and the
// largest |v_j| of its key tiles; a row of dK takes |v_j| and the largest |dO_i|
// and |D_i| of the queries that see its key.  So a small gradient keeps its bits
// beside large ones, and a sequence's gradients do not depend on the others.  The
// pre-pass leaves the logarithms of these norms by row, token and tile.  bf16 q/k
// need none.
//
// Seven products are executed for the five of the formulas (S and dP in both
// kinds of item), so that nothing is summed across CTAs.  25,920 tokens causal by
// frames of 1,620, 24/8 heads, on one GB300: 11.1 ms, 1.38 PFLOP/s executed, 80 %
// of a long product's; 3,152 + 1,081 + 257 + 77 + 1 tokens, 24/24 heads: 445 us,
// 5.5 us an item beyond its steps.  Items are never cut: few key heads (1,500
// tokens, 24/1 heads, 530 us) or few queries over many keys (8 over 52,360, 24/4
// heads, 595 us) leave most SMs idle.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "k6_device.cuh"
#include "k6_packed.cuh"
#include "k6_packed_tma.h"

namespace k6 {

namespace pb {
constexpr int D = 128, BM = 128;
constexpr int PANEL = BM * 64 * 2;
constexpr int TILE = 2 * PANEL;
constexpr int THREADS = 320;                // warps 0-7 rows, 8 TMA, 9 MMA + TMEM
constexpr int SMEM_DATA = 7 * TILE;
constexpr int SMEM_LD = SMEM_DATA + 256;    // barriers, TMEM slot and abort flag before it
constexpr int SMEM_ALLOC = SMEM_LD + 2 * 2 * BM * 4;  // lse and D of two tiles of query rows (dk/dv)
static_assert(SMEM_ALLOC <= 227 * 1024, "shared memory plan exceeds the per-CTA limit");
constexpr unsigned long long DRAIN_NS = 1000000000ull;
constexpr float LOG2E = 1.4426950408889634f;
}  // namespace pb

// log2 of norms, for the scale of dS (fp16 q/k; null pointers otherwise): -inf for
// zeros, for rows that see nothing (they have no say) and for rows that are not
// finite (which make their own results NaN, whatever the scale).
struct PackedTops {
    float *row;    // [Hkv][Tq * G]: |dO_i|
    float2 *tok;   // [Hkv][Tq]: the largest {|dO_i|, |D_i|} of a token's G rows
    float2 *tile;  // [Hkv][Tq]: the same of a query tile's rows, at its first token
    float *key;    // [Hkv][Tk]: |v_j|
    float *ktile;  // [Hkv][Tk]: the largest |v_j| of a key tile, at its first key
};

struct PackedBwdParams {
    PackedGeom g;
    const void *plan;
    float scale_log2, scale;                // log2(e)/sqrt(d), 1/sqrt(d)
    const float2 *LD;                       // [Hkv][Tq * G] {lse * log2(e), D}; lse = +inf for a row that sees nothing
    PackedTops tops;
    uint32_t dkv_blocks;                    // blocks of key tiles, ahead of those of query tiles
    __nv_bfloat16 *dq, *dk, *dv;
    long dq_stride, dk_stride, dv_stride;
    uint32_t idesc_qk, idesc_bf16, idesc_bf16_mn, idesc_ds_mn;
    int ds_f16;
    uint32_t inv_g;                         // ceil(2^16 / G): (row * inv_g) >> 16 == row / G for row < 128
    unsigned long long wait_limit_ns;
    int *err;
};

namespace {

__device__ __forceinline__ uint32_t pack_ds(float lo, float hi, bool f16) {
    if (f16) {
        __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<uint32_t *>(&h);
    }
    return pack_bf16x2(lo, hi);
}

__device__ __forceinline__ void tmem_ld16_here(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
// 2^x in program order, so the exps of a row pass run before the wait that follows them.
__device__ __forceinline__ float ex2_in_order(float x) {
    float y;
    asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void st_shared_16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}

// 2^e, -126 <= e <= 127.
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

// Four rows of 16 lanes each (half a warp) summed side by side: two steps leave
// lane `sub` with a part of row sub / 4, and the steps 2 and 1 of the sum to go.
__device__ __forceinline__ float fold(float lo, float hi, bool up, int o) {
    return (up ? hi : lo) + __shfl_xor_sync(0xffffffffu, up ? lo : hi, o);
}
__device__ __forceinline__ float fold_rows(const float (&x)[4], int sub) {
    return fold(fold(x[0], x[2], sub & 8, 8), fold(x[1], x[3], sub & 8, 8), sub & 4, 4);
}

// log2 of the squared 2-norms of four rows of 128 bf16 values, 8 in each lane
// (`x`) of half a warp: lane `sub` holds the sum `q` of row sub / 4's squares and
// gets its logarithm: -inf for zeros, inf or NaN where the row is not finite.
// Squares leave fp32's range long before bf16 values do: where one comes near its
// ends, the rows are summed again from scaled values.  A whole warp.
__device__ __forceinline__ float log2_squares(float q, const uint4 (&x)[4], int lane) {
    float log_q = log2f(q);
    if (__any_sync(0xffffffffu, !(q >= 0x1p-80f && q <= 0x1p120f))) {
        const int row = (lane & 15) >> 2, first = lane & 16;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float was = __shfl_sync(0xffffffffu, q, first + 4 * i);
            const int shift = was > 1.f ? -70 : 70;
            const float by = pow2(shift);
            const __nv_bfloat162 *v = reinterpret_cast<const __nv_bfloat162 *>(&x[i]);
            float sum = 0.f;
#pragma unroll
            for (int k = 0; k < 4; k++) {
                const float2 f = __bfloat1622float2(v[k]);
                sum = fmaf(f.x * by, f.x * by, fmaf(f.y * by, f.y * by, sum));
            }
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (row == i && !(q >= 0x1p-80f && q <= 0x1p120f)) log_q = log2f(sum) - 2.f * (float)shift;
        }
    }
    return log_q;
}

// The power of two 2^e that a row of dS is carried with: twice 2^top, the bound of
// its elements, times 2^e in (2^14, 2^15].  |e| <= 100: gradients of 2^-100 and
// 2^100 are far outside what else fp32 holds of them.
__device__ __forceinline__ int ds_exponent(float top) {
    return (int)fmaxf(-100.f, fminf(100.f, 14.f - ceilf(top)));  // 100 where all is zero
}

// Floats (no NaN) as integers of the same order, for atomicMax; its own inverse.
__device__ __forceinline__ int ordered(float x) {
    const int i = __float_as_int(x);
    return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float unordered(int i) { return __int_as_float(i ^ ((i >> 31) & 0x7fffffff)); }

// -------------------------------------------------------------- pre-pass

// LD of every query row of the sequences, and for fp16 q/k the tops.  A team of
// warps takes one query tile of a key head after another (128 rows at most), then
// key tiles: half a warp (16 lanes x 8 elements) has four rows in flight, whose
// sums and logarithms it takes side by side, and the team has as many warps as
// the batch's tiles have rows for on average (rows_team), so that all rows of a
// tile are under way at once.  A token's and a tile's largest are found in shared
// memory, two tiles' entries in turn, so that a tile costs one barrier of its
// team.  Bound by HBM: 25,920 tokens, 24/8 heads, 64 us with bf16 q/k, 82 with
// fp16 (256 threads a tile, two passes and logarithms row by row: 127).
constexpr int ROWS_THREADS = 512, ROWS_WARPS = ROWS_THREADS / 32;

template <bool NORMS>
__global__ void __launch_bounds__(ROWS_THREADS, 2)
    packed_bwd_rows_kernel(const PackedGeom g, const void *plan_base, const char *out, long out_stride,
                           const char *dout, long dout_stride, const char *v, long v_stride,
                           const float *__restrict__ lse, float2 *__restrict__ LD, const PackedTops tops,
                           const int team_warps) {
    extern __shared__ int best_of[];  // [team][tile's turn][|dO|, |D|][token], or [turn][0][key]: ordered
    const int lane = threadIdx.x & 31, sub = lane & 15, team = (int)threadIdx.x / 32 / team_warps;
    const int halves = 2 * team_warps, half = ((int)threadIdx.x >> 4) - team * halves;
    const int mine = (sub >> 2) * halves + half;  // the row, of those in flight, whose sums this lane gets
    int(*best)[2][128] = reinterpret_cast<int(*)[2][128]>(best_of + team * 512);
    const PackedPlan plan = packed_plan_at(const_cast<void *>(plan_base), g);
    if (!packed_plan_ok(*plan.head, g)) return;  // the next kernel reports it
    const uint32_t n_q = (uint32_t)plan.head->n_q, n_k = (uint32_t)plan.head->n_k;
    // the host keeps tokens * heads below 2^31
    const uint32_t q_units = n_q * (uint32_t)g.Hkv, units = q_units + (NORMS ? n_k * (uint32_t)g.Hkv : 0);
    const uint32_t teams = ROWS_WARPS / team_warps;
    if constexpr (NORMS) {
        for (int i = threadIdx.x; i < (int)teams * 512; i += ROWS_THREADS) best_of[i] = ordered(-INFINITY);
        __syncthreads();
    }
    int turn = 0;
    for (uint32_t u = blockIdx.x * teams + team; u < units; u += gridDim.x * teams) {
        int n;    // tokens or keys of the tile
        long at;  // [Hkv][Tq] or [Hkv][Tk] index of its first
        const bool keys = u >= q_units;
        if (!keys) {
            const int hk = (int)(u / n_q);
            const PackedItem it = plan.q[u - (uint32_t)hk * n_q];
            n = it.n_tok_hk, at = (long)hk * g.Tq + it.tok0;
            const int rows = n * g.G;
            for (int base = 0; base < rows; base += halves * 4) {
                uint4 a[4], b[4];
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const int r = min(base + i * halves + half, rows - 1);
                    const int t = r / g.G, h = hk * g.G + r - t * g.G;
                    a[i] = reinterpret_cast<const uint4 *>(out + (long)(it.tok0 + t) * out_stride + (long)h * 256)[sub];
                    b[i] = reinterpret_cast<const uint4 *>(dout + (long)(it.tok0 + t) * dout_stride + (long)h * 256)[sub];
                }
                const int r = min(base + mine, rows - 1), t = r / g.G;
                const float l = lse[(long)(hk * g.G + r - t * g.G) * g.Tq + it.tok0 + t];
                float s[4], q[4];
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const __nv_bfloat162 *x = reinterpret_cast<const __nv_bfloat162 *>(&a[i]);
                    const __nv_bfloat162 *y = reinterpret_cast<const __nv_bfloat162 *>(&b[i]);
                    s[i] = q[i] = 0.f;
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        const float2 fx = __bfloat1622float2(x[k]), fy = __bfloat1622float2(y[k]);
                        s[i] = fmaf(fx.x, fy.x, s[i]);
                        s[i] = fmaf(fx.y, fy.y, s[i]);
                        if (NORMS) q[i] = fmaf(fy.x, fy.x, fmaf(fy.y, fy.y, q[i]));
                    }
                }
                float d = fold_rows(s, sub);
                d += __shfl_xor_sync(0xffffffffu, d, 2);
                d += __shfl_xor_sync(0xffffffffu, d, 1);
                float top = 0.f;
                if constexpr (NORMS) {
                    float x = fold_rows(q, sub);
                    x += __shfl_xor_sync(0xffffffffu, x, 2);
                    x += __shfl_xor_sync(0xffffffffu, x, 1);
                    top = 0.5f * log2_squares(x, b, lane);
                }
                if (base + mine < rows && (sub & 3) == 0) {
                    const bool none = l == -INFINITY;  // the row sees nothing
                    LD[at * g.G + r] = make_float2(none ? INFINITY : l * pb::LOG2E, d);
                    if constexpr (NORMS) {
                        const float log_d = log2f(fabsf(d));
                        const bool has_do = !none && top < INFINITY, has_d = !none && log_d < INFINITY;
                        tops.row[at * g.G + r] = has_do ? top : -INFINITY;
                        if (has_do) atomicMax(&best[turn][0][t], ordered(top));
                        if (has_d) atomicMax(&best[turn][1][t], ordered(log_d));
                    }
                }
            }
        } else {
            const int hk = (int)((u - q_units) / n_k);
            const PackedKItem it = plan.k[u - q_units - (uint32_t)hk * n_k];
            n = it.n_key, at = (long)hk * g.Tk + it.krow0;
            for (int base = 0; base < n; base += halves * 4) {
                uint4 a[4];
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const int r = min(base + i * halves + half, n - 1);
                    a[i] = reinterpret_cast<const uint4 *>(v + (long)(it.krow0 + r) * v_stride + (long)hk * 256)[sub];
                }
                float q[4];
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const __nv_bfloat162 *x = reinterpret_cast<const __nv_bfloat162 *>(&a[i]);
                    q[i] = 0.f;
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        const float2 f = __bfloat1622float2(x[k]);
                        q[i] = fmaf(f.x, f.x, fmaf(f.y, f.y, q[i]));
                    }
                }
                float x = fold_rows(q, sub);
                x += __shfl_xor_sync(0xffffffffu, x, 2);
                x += __shfl_xor_sync(0xffffffffu, x, 1);
                float top = 0.5f * log2_squares(x, a, lane);
                if (!(top < INFINITY)) top = -INFINITY;
                if (base + mine < n && (sub & 3) == 0) {
                    tops.key[at + base + mine] = top;
                    best[turn][0][base + mine] = ordered(top);
                }
            }
        }
        if constexpr (NORMS) {
            if (team_warps == 1) __syncwarp();
            else asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(team_warps * 32) : "memory");
            if (half < 2) {  // the team's first warp
                float2 m = make_float2(-INFINITY, -INFINITY);
                for (int t = lane; t < n; t += 32) {
                    const float2 x = make_float2(unordered(best[turn][0][t]), unordered(best[turn][1][t]));
                    best[turn][0][t] = best[turn][1][t] = ordered(-INFINITY);  // next written behind the next barrier
                    if (!keys) tops.tok[at + t] = x;
                    m = make_float2(fmaxf(m.x, x.x), fmaxf(m.y, x.y));
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    m.x = fmaxf(m.x, __shfl_xor_sync(0xffffffffu, m.x, o));
                    m.y = fmaxf(m.y, __shfl_xor_sync(0xffffffffu, m.y, o));
                }
                if (lane == 0) {
                    if (keys) tops.ktile[at] = m.x;
                    else tops.tile[at] = m;
                }
            }
            turn ^= 1;
        }
    }
}

// ----------------------------------------------------------- shared set-up

template <int NB>
__device__ __forceinline__ uint32_t setup(uint8_t *smem, const int (&counts)[NB], uint64_t *&bars,
                                          volatile int *&abort_flag) {
    bars = reinterpret_cast<uint64_t *>(smem + pb::SMEM_DATA);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + NB);
    abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    if (threadIdx.x == 0) {
        for (int i = 0; i < NB; i++) mbar_init(bars + i, counts[i]);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (threadIdx.x / 32 == 9) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    return *tmem_slot;
}

__device__ __forceinline__ void teardown(uint32_t tmem) {
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x / 32 == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Two 64-element panels into dst (completing on bar).
__device__ __forceinline__ void load_panels(uint8_t *dst, const CUtensorMap *m, uint64_t *bar, int head, int row) {
    tma_load_4d(dst, m, bar, 0, head, row, 0);
    tma_load_4d(dst + pb::PANEL, m, bar, 64, head, row, 0);
}

// Rows [from, 128) of a tile in shared memory to zero, by one whole warp, before its MMAs read them.
__device__ __forceinline__ void zero_rows(uint8_t *tile, int from, int lane) {
    for (int c = from * 8 + lane; c < pb::BM * 8; c += 32) {
        *reinterpret_cast<uint4 *>(tile + c * 16) = make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4 *>(tile + pb::PANEL + c * 16) = make_uint4(0, 0, 0, 0);
    }
    fence_async_smem();
    __syncwarp();
}

// Step kk of a K-major SS MMA chain over d = 128.
__device__ __forceinline__ void mma_k(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, int kk) {
    const uint64_t off = (uint64_t)((kk >> 2) * pb::PANEL + (kk & 3) * 32) >> 4;
    mma_ss_w(d, a + off, b + off, idesc, kk > 0);
}

// 64 columns of this warp's 32 TMEM lanes (rows), times `scale`, as bf16: row i
// of the warp goes to dst(i) (null: not stored).  The warp turns its rows in
// `mine` (4 KB of shared memory that no MMA or copy uses any more) so that eight
// lanes store a row's 128 bytes, instead of 32 lanes 32 rows.
template <typename Dst>
__device__ __forceinline__ void store_rows(uint32_t taddr, uint8_t *mine, int lane, float scale, Dst dst) {
    auto chunk = [&](int row, int c) { return reinterpret_cast<uint4 *>(mine + row * 128 + (((c ^ row) & 7) << 4)); };
#pragma unroll
    for (int h = 0; h < 2; h++) {
        uint32_t o[32];
        tmem_ld32(taddr + h * 32, o);
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < 4; c++) {
            auto two = [&](int i) {
                return pack_bf16x2(__uint_as_float(o[c * 8 + i]) * scale, __uint_as_float(o[c * 8 + i + 1]) * scale);
            };
            *chunk(lane, h * 4 + c) = make_uint4(two(0), two(2), two(4), two(6));
        }
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const int row = 4 * i + lane / 8;
        __nv_bfloat16 *d = dst(row);
        if (d) *reinterpret_cast<uint4 *>(d + (lane % 8) * 8) = *chunk(row, lane % 8);
    }
    __syncwarp();
}

__device__ __forceinline__ void zero_half_row(__nv_bfloat16 *dst) {
#pragma unroll
    for (int k = 0; k < 64; k += 8) *reinterpret_cast<uint4 *>(dst + k) = make_uint4(0, 0, 0, 0);
}

// ------------------------------------------------------------------ dq kernel
//
// smem tiles: Q 0, dO 1, K slots 2-4, V slots 5-6.  Tensor memory: S buffers
// 0-127 and 128-255 (dS over each half's first 32 columns), dP 256-383, dQ
// 384-511.  With two S buffers the MMAs of a step (dP(t+1), dQ(t), S(t+2)) and
// the row pass (P(t+1) from S(t+1), then dS(t+1) once dP(t+1) is there) run side
// by side: 2,330 cycles a step, of which its products take 1,536 and shared
// memory (their operands and the copies) some 1,800.  (One S buffer, and S and dP
// both awaited before a row pass: 2,580.  Q and dO in tensor memory and steps of
// 64 keys, for the room: 3,100, since a product of N = 64 takes as long as one of
// 128.)

namespace dqk {
constexpr int STAT = 0, KFULL = 1, KEMPTY = 4, VFULL = 7, VEMPTY = 9, SFULL = 11, DPFULL = 13, DSFULL = 14, ACC = 15,
              DRAIN = 16, NB = 17;
}

// Row pass of the dq kernel, second half: dS of one query row and 64 keys from P
// in registers and dP in tensor memory, to `ds_at`; keys from rel on get dS = 0
// (MASKED).
template <bool MASKED>
__device__ __forceinline__ void dq_row(const float (&pr)[64], uint32_t dp_at, uint32_t ds_at, int rel, float d,
                                       int ds_f16) {
#pragma unroll
    for (int c = 0; c < 2; c++) {
        uint32_t pv[32], ds[16];
        tmem_ld32(dp_at + 32 * c, pv);
        tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
            float d0 = pr[32 * c + k] * (__uint_as_float(pv[k]) - d);
            float d1 = pr[32 * c + k + 1] * (__uint_as_float(pv[k + 1]) - d);
            if (MASKED) {
                if (32 * c + k >= rel) d0 = 0.f;
                if (32 * c + k + 1 >= rel) d1 = 0.f;
            }
            // dS in K's type (one MMA takes one type): 2^-8 (bf16) or 2^-11 (fp16) of each term
            ds[k / 2] = pack_ds(d0, d1, ds_f16);
        }
        tmem_st16(ds_at + 16 * c, ds);
    }
}

// One query tile of one key head (the whole block).
__device__ __forceinline__ void dq_item(uint8_t *smem, const CUtensorMap &tm_q, const CUtensorMap &tm_do,
                                        const CUtensorMap &tm_k, const CUtensorMap &tm_v, const PackedBwdParams &p,
                                        const PackedItem &it, int hk) {
    using namespace pb;
    using namespace dqk;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int T = it.kt1;
    // rows: lane quarter q4, key half g
    const int q4 = warp & 3, g = (warp >> 2) & 1;
    const int r = 32 * q4 + lane;
    const int rtok = r / p.g.G, rhead = r % p.g.G;
    const bool live = warp < 8 && rtok < it.n_tok_hk && r < p.g.rows;
    const long tok = (long)it.tok0 + (live ? rtok : 0);
    __nv_bfloat16 *drow = p.dq + tok * p.dq_stride + (long)(hk * p.g.G + rhead) * D + 64 * g;
    if (T <= 0) {  // no key is seen by any row of the tile
        if (live) zero_half_row(drow);
        return;
    }
    const int counts[NB] = {1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 256, 1, 1};
    uint64_t *bar;
    volatile int *abort_flag;
    const uint32_t tmem = setup<NB>(smem, counts, bar, abort_flag);
    const WaitCtx w{p.wait_limit_ns, p.err, abort_flag};
    uint8_t *sQ = smem, *sDO = smem + TILE, *sK = smem + 2 * TILE, *sV = smem + 5 * TILE;

    if (warp == 8) {
        const bool leader = elect_one();
        if (leader) {
            mbar_arrive_expect_tx(bar + STAT, 2u * (uint32_t)p.g.rows * 256u);
            load_panels(sQ, &tm_q, bar + STAT, hk * p.g.G, it.tok0);
            load_panels(sDO, &tm_do, bar + STAT, hk * p.g.G, it.tok0);
        }
        int nk = 0, nv = 0;  // K and V tiles issued
        for (int t = 0; t < T; t++) {
            const int ks = t % 3, vs = t & 1, row = it.krow0 + t * BM;
            if (!mbar_wait_w(bar + KEMPTY + ks, ((t / 3) & 1) ^ 1, w)) break;
            if (leader) {
                mbar_arrive_expect_tx(bar + KFULL + ks, TILE);
                load_panels(sK + ks * TILE, &tm_k, bar + KFULL + ks, hk, row);
            }
            nk++;
            if (!mbar_wait_w(bar + VEMPTY + vs, ((t >> 1) & 1) ^ 1, w)) break;
            if (leader) {
                mbar_arrive_expect_tx(bar + VFULL + vs, TILE);
                load_panels(sV + vs * TILE, &tm_v, bar + VFULL + vs, hk, row);
            }
            nv++;
        }
        // let copies in flight land before the CTA exits
        mbar_drain(bar + STAT, 0, DRAIN_NS);
        for (int t = nk > 3 ? nk - 3 : 0; t < nk; t++) mbar_drain(bar + KFULL + t % 3, (t / 3) & 1, DRAIN_NS);
        for (int t = nv > 2 ? nv - 2 : 0; t < nv; t++) mbar_drain(bar + VFULL + (t & 1), (t >> 1) & 1, DRAIN_NS);
        __syncwarp();
    } else if (warp == 9) {
        const uint32_t tS = tmem, tP = tmem + 256, tA = tmem + 384;
        const uint64_t dq_ = smem_desc_sw128(smem_u32(sQ), 16, 1024);
        const uint64_t ddo = smem_desc_sw128(smem_u32(sDO), 16, 1024);
        const uint64_t dk0 = smem_desc_sw128(smem_u32(sK), 16, 1024);
        const uint64_t dv0 = smem_desc_sw128(smem_u32(sV), 16, 1024);
        const uint64_t dkmn = smem_desc_sw128(smem_u32(sK), PANEL, 1024);
        auto issue_s = [&](int t) -> bool {  // S(t) = Q K^T into buffer t & 1
            const int ks = t % 3;
            if (!mbar_wait_w(bar + KFULL + ks, (t / 3) & 1, w)) return false;
            // keys behind the sequence enter dQ += dS K times zero
            if (it.Lk - t * BM < BM) zero_rows(sK + ks * TILE, it.Lk - t * BM, lane);
            tc_fence_after();
            const uint64_t kd = dk0 + (uint64_t)((ks * TILE) >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; kk++) mma_k(tS + (t & 1) * 128, dq_, kd, p.idesc_qk, kk);
            tc_commit_w(bar + SFULL + (t & 1));
            return true;
        };
        auto issue_dp = [&](int t) -> bool {  // dP(t) = dO V^T
            const int vs = t & 1;
            if (!mbar_wait_w(bar + VFULL + vs, (t >> 1) & 1, w)) return false;
            tc_fence_after();
            const uint64_t vd = dv0 + (uint64_t)((vs * TILE) >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; kk++) mma_k(tP, ddo, vd, p.idesc_bf16, kk);
            tc_commit_w(bar + VEMPTY + vs);
            tc_commit_w(bar + DPFULL);
            return true;
        };
        bool ok = mbar_wait_w(bar + STAT, 0, w) && issue_s(0) && issue_dp(0) && (T < 2 || issue_s(1));
        for (int t = 0; t < T && ok; t++) {
            // the row pass has read dP(t) and written dS(t) over S(t)
            if (!(ok = mbar_wait_w(bar + DSFULL, t & 1, w))) break;
            tc_fence_after();
            if (t + 1 < T && !(ok = issue_dp(t + 1))) break;
            const uint64_t kmn = dkmn + (uint64_t)(((t % 3) * TILE) >> 4);
            const uint32_t ads = tS + (t & 1) * 128;
#pragma unroll
            for (int kk = 0; kk < BM / 16; kk++)
                mma_ts_w(tA, ads + (kk >> 2) * 64 + (kk & 3) * 8, kmn + (uint64_t)((kk * 16 * 128) >> 4), p.idesc_ds_mn,
                         (t > 0 || kk > 0) ? 1u : 0u);  // dQ += dS K
            tc_commit_w(bar + KEMPTY + t % 3);
            if (t + 2 < T && !(ok = issue_s(t + 2))) break;  // MMAs of a thread run in order: dS(t) has been read
        }
        if (ok) tc_commit_w(bar + ACC);
        tc_commit_w(bar + DRAIN);
        mbar_drain(bar + DRAIN, 0, DRAIN_NS);
        __syncwarp();
    } else {
        const uint32_t lb = tmem + ((uint32_t)(32 * q4) << 16);
        int e = 0;
        const int lim = live ? packed_limit(it.pos0 + rtok, it.Lk, p.g.block) : it.Lk;
        float2 ld = make_float2(INFINITY, 0.f);
        const long at = ((long)hk * p.g.Tq + tok) * p.g.G + rhead;
        if (live) ld = p.LD[at];
        if (p.tops.row) {
            const float top = live ? p.tops.row[at] : -INFINITY;
            float v = -INFINITY;  // the largest |v_j| of the item's keys
            for (int t = lane; t < T; t += 32) v = fmaxf(v, p.tops.ktile[(long)hk * p.g.Tk + it.krow0 + t * BM]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
            e = ds_exponent(fmaxf(top + v, log2f(fabsf(ld.y))));
        }
        ld.x -= (float)e;  // P, and with it dS, is carried times 2^e
        const float sl2 = p.scale_log2;
        bool ok = true;
        for (int t = 0; t < T; t++) {
            if (!mbar_wait(bar + SFULL + (t & 1), (t >> 1) & 1, w)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t mine = lb + 128 * (t & 1) + 64 * g;  // this half's columns of S(t), and its dS(t)
            float pr[64];
#pragma unroll
            for (int c = 0; c < 2; c++) {
                uint32_t sv[32];
                tmem_ld32(mine + 32 * c, sv);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 32; k++) pr[32 * c + k] = ex2_in_order(fmaf(__uint_as_float(sv[k]), sl2, -ld.x));
            }
            if (!mbar_wait(bar + DPFULL, t & 1, w)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const int rel = lim - t * BM - 64 * g;  // columns below rel of this half are seen
            if (__any_sync(0xffffffffu, rel < 64)) dq_row<true>(pr, lb + 256 + 64 * g, mine, rel, ld.y, p.ds_f16);
            else dq_row<false>(pr, lb + 256 + 64 * g, mine, rel, ld.y, p.ds_f16);
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(bar + DSFULL);
        }
        if (ok && mbar_wait(bar + ACC, 0, w)) {
            tc_fence_after();
            store_rows(lb + 384 + 64 * g, smem + warp * 4096, lane, p.scale * pow2(-e), [&](int i) {
                const int rr = 32 * q4 + i;
                const int tk = (int)(((uint32_t)rr * p.inv_g) >> 16);  // rr / G
                return tk < it.n_tok_hk && rr < p.g.rows
                           ? p.dq + ((long)it.tok0 + tk) * p.dq_stride + (long)(hk * p.g.G + rr - tk * p.g.G) * D + 64 * g
                           : nullptr;
            });
        }
    }
    teardown(tmem);
}

// Row pass of the dk/dv kernel, first half: P of one key row and 64 queries from
// S^T in registers; sx holds the queries' lse (+inf for rows that are none).
// Queries below lo do not see the key: P = 0 (MASKED).
template <bool MASKED>
__device__ __forceinline__ void p_row(float (&pr)[64], const uint32_t (&sv)[2][32], const float *sx, int lo, float sl2) {
#pragma unroll
    for (int c = 0; c < 16; c++) {
        const float4 x = *reinterpret_cast<const float4 *>(sx + 4 * c);
        const float l2[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const int j = 4 * c + k;
            pr[j] = ex2_in_order(fmaf(__uint_as_float(sv[j / 32][j % 32]), sl2, -l2[k]));
            if (MASKED && j < lo) pr[j] = 0.f;
        }
    }
}

// Second half: dS^T = P (dP^T - D) of the 64 columns at taddr, times `sc`, into
// this thread's row of the swizzled dS^T panel at prow; sd holds the queries' D.
__device__ __forceinline__ void ds_row(const float (&pr)[64], const float *sd, uint32_t taddr, uint32_t prow, int r,
                                       int ds_f16, float sc) {
#pragma unroll
    for (int c = 0; c < 4; c++) {
        uint32_t pv[16], ds[8];
        tmem_ld16_here(taddr + 16 * c, pv);
        tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 16; k += 4) {
            const float4 d = *reinterpret_cast<const float4 *>(sd + 16 * c + k);
            float de[4] = {__uint_as_float(pv[k]) - d.x, __uint_as_float(pv[k + 1]) - d.y,
                           __uint_as_float(pv[k + 2]) - d.z, __uint_as_float(pv[k + 3]) - d.w};
#pragma unroll
            for (int e = 0; e < 4; e++) de[e] *= pr[16 * c + k + e];
            if (ds_f16) {
                ds[k / 2] = pack_ds(de[0] * sc, de[1] * sc, true);
                ds[k / 2 + 1] = pack_ds(de[2] * sc, de[3] * sc, true);
            } else {
                ds[k / 2] = pack_ds(de[0], de[1], false);
                ds[k / 2 + 1] = pack_ds(de[2], de[3], false);
            }
        }
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const int chunk = 2 * c + i;  // 16-byte chunk of the 128-byte row
            st_shared_16(prow + ((chunk ^ (r & 7)) << 4), ds[4 * i], ds[4 * i + 1], ds[4 * i + 2], ds[4 * i + 3]);
        }
    }
}

// The exponent of key row r's dS in a key tile (warps 0-7, 256 threads; `scratch`:
// 256 words of shared memory that nothing else uses until the function returns).
// The tile's keys fall into groups that the same queries see: frames of the mask,
// from the first key's on.  A query of group f sees the keys of the groups up to
// f, so key r takes the largest over the groups from its own on; queries behind
// the last group's first are taken by whole tiles.
__device__ __forceinline__ int dkv_exponent(const PackedBwdParams &p, const PackedKItem &it, int hk, int r, int *scratch) {
    const PackedGeom &g = p.g;
    const int t = threadIdx.x, lane = t & 31, F = g.block;
    const float v = r < it.n_key ? p.tops.key[(long)hk * g.Tk + it.krow0 + r] : -INFINITY;
    const int last = it.key0 + it.n_key - 1, frame0 = F ? it.key0 / F : 0, groups = F ? last / F - frame0 + 1 : 1;
    const int tile0 = (packed_first_query(last, it.off, F) + g.tpt - 1) / g.tpt;
    const int first = packed_first_query(it.key0, it.off, F) + t, end = min(tile0 * g.tpt, it.Lq);
    const long at = (long)hk * g.Tq + it.qrow0;
    const float2 none = make_float2(-INFINITY, -INFINITY);
    // the first of each is asked for before any is waited for: a short item has no more
    float2 m = tile0 + t < it.qt1 ? p.tops.tile[at + (long)(tile0 + t) * g.tpt] : none;
    float2 x = first < end ? p.tops.tok[at + first] : none;
    scratch[t] = ordered(-INFINITY);
    asm volatile("bar.sync 1, 256;" ::: "memory");
    for (int i = tile0 + t + 256; i < it.qt1; i += 256) {
        const float2 y = p.tops.tile[at + (long)i * g.tpt];
        m = make_float2(fmaxf(m.x, y.x), fmaxf(m.y, y.y));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        m.x = fmaxf(m.x, __shfl_xor_sync(0xffffffffu, m.x, o));
        m.y = fmaxf(m.y, __shfl_xor_sync(0xffffffffu, m.y, o));
    }
    if (lane == 0) {
        atomicMax(&scratch[groups - 1], ordered(m.x));
        atomicMax(&scratch[128 + groups - 1], ordered(m.y));
    }
    for (int i = first; i < end; i += 256) {
        if (i > first) x = p.tops.tok[at + i];
        const int f = F ? min(groups - 1, (i + it.off) / F - frame0) : 0;  // i + off >= frame0 F
        atomicMax(&scratch[f], ordered(x.x));
        atomicMax(&scratch[128 + f], ordered(x.y));
    }
    asm volatile("bar.sync 1, 256;" ::: "memory");
    if (groups > 1 && t < 64) {  // the largest from each group on: one warp each for |dO| and |D|, four groups a lane
        int4 *mine = reinterpret_cast<int4 *>(scratch + (t & 32) * 4) + lane;
        int4 x = *mine;
        x.z = max(x.z, x.w), x.y = max(x.y, x.z), x.x = max(x.x, x.y);
        int all = x.x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_down_sync(0xffffffffu, all, o);
            if (lane + o < 32) all = max(all, y);
        }
        int behind = __shfl_down_sync(0xffffffffu, all, 1);
        if (lane == 31) behind = ordered(-INFINITY);
        *mine = make_int4(max(x.x, behind), max(x.y, behind), max(x.z, behind), max(x.w, behind));
    }
    if (groups > 1) asm volatile("bar.sync 1, 256;" ::: "memory");
    const int f = F ? min(groups - 1, (it.key0 + r) / F - frame0) : 0;
    const float top = fmaxf(unordered(scratch[f]) + v, unordered(scratch[128 + f]));
    asm volatile("bar.sync 1, 256;" ::: "memory");
    return ds_exponent(top);
}

// ----------------------------------------------------------------- dkv kernel
//
// smem tiles: K 0, V 1, ring slot s: Q 2+2s, dO 3+2s; dS^T 6.  Tensor memory:
// S^T 0-127 (P^T over each half's first 32 columns), dP^T 128-255, dV 256-383,
// dK 384-511.  A step: P^T(t) is published as soon as S^T(t) is read, so that
// dV(t) and behind it S^T(t+1) run under the second half of the row pass
// (dS^T(t) from dP^T(t)); that half published, dK(t) and dP^T(t+1) follow under
// the next row pass: 3,100 cycles a step, its products 2,048.  (With dS^T over dP^T and P^T in shared memory, as in
// bwd_dkv_kernel, dP^T(t+1) had to wait for dK(t) and the row pass for both: a
// step took 3,550 cycles.)

namespace dkvk {
constexpr int STAT = 0, QFULL = 1, DOFULL = 3, QEMPTY = 5, DOEMPTY = 7, SREADY = 9, DPREADY = 10, PREADY = 11,
              DSREADY = 12, DSFREE = 13, ACC = 14, DRAIN = 15, NB = 16;
}

// One key tile of one key head (the whole block).
__device__ __forceinline__ void dkv_item(uint8_t *smem, const CUtensorMap &tm_q, const CUtensorMap &tm_do,
                                         const CUtensorMap &tm_k, const CUtensorMap &tm_v, const PackedBwdParams &p,
                                         const PackedKItem &it, int hk) {
    using namespace pb;
    using namespace dkvk;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int T = it.qt1 - it.qt0;
    // rows: key row r, query half g
    const int q4 = warp & 3, g = (warp >> 2) & 1;
    const int r = 32 * q4 + lane;
    const bool live = warp < 8 && r < it.n_key;
    __nv_bfloat16 *krow = p.dk + ((long)it.krow0 + (live ? r : 0)) * p.dk_stride + (long)hk * D + 64 * g;
    __nv_bfloat16 *vrow = p.dv + ((long)it.krow0 + (live ? r : 0)) * p.dv_stride + (long)hk * D + 64 * g;
    if (T <= 0) {  // no query sees any key of the tile
        if (live) {
            zero_half_row(krow);
            zero_half_row(vrow);
        }
        return;
    }
    const int counts[NB] = {1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 256, 256, 1, 1, 1};
    uint64_t *bar;
    volatile int *abort_flag;
    // rows that a copy of g.rows rows does not reach stay zero
    for (int t = 2; t < 6 && p.g.rows < BM; t++) {
        for (int c = p.g.rows * 8 + (int)threadIdx.x; c < BM * 8; c += THREADS) {
            *reinterpret_cast<uint4 *>(smem + t * TILE + c * 16) = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4 *>(smem + t * TILE + PANEL + c * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_async_smem();
    }
    // query rows of tile t (of the item's T) that belong to the sequence
    auto rows_of = [&](int t) { return min(p.g.rows, (it.Lq - (it.qt0 + t) * p.g.tpt) * p.g.G); };
    // {lse, D} of row i of tile t: P is 0 in a row that is none (its rows of Q and dO are zero, its D finite)
    const float2 *ld_h = p.LD + ((long)hk * p.g.Tq + it.qrow0) * p.g.G;
    auto row_ld = [&](int t, int i) {
        return t < T && i < rows_of(t) ? ld_h[(long)(it.qt0 + t) * p.g.rows + i] : make_float2(INFINITY, 0.f);
    };
    // the queries' lse and D, [tile parity][lse, D][128]: warps 0-3 bring the next tile's
    float *sLD = reinterpret_cast<float *>(smem + SMEM_LD);
    if (threadIdx.x < BM) {
        const float2 v = row_ld(0, threadIdx.x);
        sLD[threadIdx.x] = v.x, sLD[BM + threadIdx.x] = v.y;
    }
    const uint32_t tmem = setup<NB>(smem, counts, bar, abort_flag);
    const WaitCtx w{p.wait_limit_ns, p.err, abort_flag};
    uint8_t *sK = smem, *sV = smem + TILE, *sRing = smem + 2 * TILE, *sDS = smem + 6 * TILE;

    if (warp == 8) {
        const bool leader = elect_one();
        if (leader) {
            mbar_arrive_expect_tx(bar + STAT, 2 * TILE);
            load_panels(sK, &tm_k, bar + STAT, hk, it.krow0);
            load_panels(sV, &tm_v, bar + STAT, hk, it.krow0);
        }
        const uint32_t bytes = (uint32_t)p.g.rows * 256u;
        int nq = 0, ndo = 0;  // Q and dO tiles issued
        for (int t = 0; t < T; t++) {
            const int s = t & 1, row = it.qrow0 + (it.qt0 + t) * p.g.tpt;
            const uint32_t par = ((t >> 1) & 1) ^ 1;
            if (!mbar_wait_w(bar + QEMPTY + s, par, w)) break;
            if (leader) {
                mbar_arrive_expect_tx(bar + QFULL + s, bytes);
                load_panels(sRing + 2 * s * TILE, &tm_q, bar + QFULL + s, hk * p.g.G, row);
            }
            nq++;
            if (!mbar_wait_w(bar + DOEMPTY + s, par, w)) break;
            if (leader) {
                mbar_arrive_expect_tx(bar + DOFULL + s, bytes);
                load_panels(sRing + (2 * s + 1) * TILE, &tm_do, bar + DOFULL + s, hk * p.g.G, row);
            }
            ndo++;
        }
        mbar_drain(bar + STAT, 0, DRAIN_NS);
        for (int t = nq > 2 ? nq - 2 : 0; t < nq; t++) mbar_drain(bar + QFULL + (t & 1), (t >> 1) & 1, DRAIN_NS);
        for (int t = ndo > 2 ? ndo - 2 : 0; t < ndo; t++) mbar_drain(bar + DOFULL + (t & 1), (t >> 1) & 1, DRAIN_NS);
        __syncwarp();
    } else if (warp == 9) {
        const uint32_t tS = tmem, tP = tmem + 128, tV = tmem + 256, tK = tmem + 384;
        const uint64_t dk0 = smem_desc_sw128(smem_u32(sK), 16, 1024);
        const uint64_t dv0 = smem_desc_sw128(smem_u32(sV), 16, 1024);
        const uint64_t dring = smem_desc_sw128(smem_u32(sRing), 16, 1024);
        const uint64_t dring_mn = smem_desc_sw128(smem_u32(sRing), PANEL, 1024);
        const uint64_t dds = smem_desc_sw128(smem_u32(sDS), 16, 1024);
        // descriptor of tile `which` (0 Q, 1 dO) of the ring slot of tile t
        auto slot = [&](uint64_t base, int t, int which) {
            return base + (uint64_t)(((2 * (t & 1) + which) * TILE) >> 4);
        };
        // wait for tile t; queries behind the sequence enter dK and dV times zero
        auto wait_tile = [&](int t, int full, int which) {
            if (!mbar_wait_w(bar + full + (t & 1), (t >> 1) & 1, w)) return false;
            if (rows_of(t) < p.g.rows) zero_rows(sRing + (2 * (t & 1) + which) * TILE, rows_of(t), lane);
            return true;
        };
        auto wait_q = [&](int t) { return wait_tile(t, QFULL, 0); };
        auto wait_do = [&](int t) { return wait_tile(t, DOFULL, 1); };
        bool ok = mbar_wait_w(bar + STAT, 0, w) && wait_q(0);
        if (ok) {
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < D / 16; kk++) mma_k(tS, dk0, slot(dring, 0, 0), p.idesc_qk, kk);  // S^T = K Q^T
            tc_commit_w(bar + SREADY);
            ok = wait_do(0);
        }
        if (ok) {
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < D / 16; kk++) mma_k(tP, dv0, slot(dring, 0, 1), p.idesc_bf16, kk);  // dP^T = V dO^T
            tc_commit_w(bar + DPREADY);
        }
        for (int t = 0; t < T && ok; t++) {
            const bool next = t + 1 < T;
            // P^T(t) is in tensor memory
            if (!(ok = mbar_wait_w(bar + PREADY, t & 1, w))) break;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < BM / 16; kk++)  // dV += P^T dO; K-step kk covers queries 16 kk .. 16 kk + 15
                mma_ts_w(tV, tS + (kk >> 2) * 64 + (kk & 3) * 8, slot(dring_mn, t, 1) + (uint64_t)((kk * 16 * 128) >> 4),
                         p.idesc_bf16_mn, (t > 0 || kk > 0) ? 1u : 0u);
            tc_commit_w(bar + DOEMPTY + (t & 1));  // dO(t): dP^T(t) and dV(t) done
            if (next) {  // MMAs of a thread run in order: S^T(t+1) overwrites P^T(t) behind dV(t)
                if (!(ok = wait_q(t + 1))) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < D / 16; kk++) mma_k(tS, dk0, slot(dring, t + 1, 0), p.idesc_qk, kk);
                tc_commit_w(bar + SREADY);
            }
            // dS^T(t) is in shared memory, dP^T(t) read
            if (!(ok = mbar_wait_w(bar + DSREADY, t & 1, w))) break;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < BM / 16; kk++)  // dK += dS^T Q; ahead of dP^T(t+1), since Q(t+2) waits for its slot
                mma_ss_w(tK, dds + ((uint64_t)((kk >> 2) * PANEL + (kk & 3) * 32) >> 4),
                         slot(dring_mn, t, 0) + (uint64_t)((kk * 16 * 128) >> 4), p.idesc_ds_mn,
                         (t > 0 || kk > 0) ? 1u : 0u);
            tc_commit_w(bar + QEMPTY + (t & 1));  // Q(t): S^T(t) and dK(t) done
            tc_commit_w(bar + DSFREE);
            if (next) {
                if (!(ok = wait_do(t + 1))) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < D / 16; kk++) mma_k(tP, dv0, slot(dring, t + 1, 1), p.idesc_bf16, kk);  // dP^T(t+1)
                tc_commit_w(bar + DPREADY);
            }
        }
        if (ok) tc_commit_w(bar + ACC);
        tc_commit_w(bar + DRAIN);
        mbar_drain(bar + DRAIN, 0, DRAIN_NS);
        __syncwarp();
    } else {
        const uint32_t lb = tmem + ((uint32_t)(32 * q4) << 16);
        const float sl2 = p.scale_log2;
        // dS^T's tile is free until the first step writes it
        const int e = p.tops.row ? dkv_exponent(p, it, hk, r, reinterpret_cast<int *>(sDS)) : 0;
        const float sc = pow2(e);
        // the first query row (of the sequence, tokens x heads) that sees this key
        const long first = (long)packed_first_query(it.key0 + r, it.off, p.g.block) * p.g.G;
        // this thread's row of dS^T panel g: 8 chunks of 16 bytes, 128-byte swizzle
        const uint32_t prow = smem_u32(sDS) + g * PANEL + (r >> 3) * 1024 + (r & 7) * 128;
        bool ok = true;
        for (int t = 0; t < T; t++) {
            if (!mbar_wait(bar + SREADY, t & 1, w)) {
                ok = false;
                break;
            }
            tc_fence_after();
            uint32_t sv[2][32];
            tmem_ld32(lb + 64 * g, sv[0]);
            tmem_ld32(lb + 64 * g + 32, sv[1]);
            tmem_ld_wait();
            const long q0 = (long)(it.qt0 + t) * p.g.rows + 64 * g;  // first query row of this half
            const int lo = (int)max(-1L, min(first - q0, 64L));       // rows of this half from lo on see the key
            // the tile's {lse, D}, written before its writers' P^T(t-1) arrivals
            if (t > 0 && !mbar_wait(bar + PREADY, (t - 1) & 1, w)) {
                ok = false;
                break;
            }
            const float *sx = sLD + (t & 1) * 2 * BM + 64 * g;
            float2 nx = make_float2(0.f, 0.f);
            if (g == 0) nx = row_ld(t + 1, r);
            float pr[64];
            if (__any_sync(0xffffffffu, lo > 0)) p_row<true>(pr, sv, sx, lo, sl2);
            else p_row<false>(pr, sv, sx, lo, sl2);
            if (g == 0) {  // the other buffer was last read in step t-1, before its readers' dS^T(t-1) arrivals
                float *at = sLD + ((t + 1) & 1) * 2 * BM + r;
                if (t > 0 && !mbar_wait(bar + DSREADY, (t - 1) & 1, w)) {
                    ok = false;
                    break;
                }
                at[0] = nx.x, at[BM] = nx.y;
            }
            {  // P^T(t), rounded to bf16 (dO's type; one MMA takes one type), over this half's columns of S^T(t)
                uint32_t pk[32];
#pragma unroll
                for (int k = 0; k < 64; k += 2) pk[k / 2] = pack_bf16x2(pr[k], pr[k + 1]);
                tmem_st32(lb + 64 * g, pk);
            }
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(bar + PREADY);
            // dP^T(t) is in place, and dK(t-1) has read the dS^T buffer
            if (!mbar_wait(bar + DPREADY, t & 1, w) || (t > 0 && !mbar_wait(bar + DSFREE, (t - 1) & 1, w))) {
                ok = false;
                break;
            }
            tc_fence_after();
            ds_row(pr, sx + BM, lb + 128 + 64 * g, prow, r, p.ds_f16, sc);
            fence_async_smem();
            tc_fence_before();
            mbar_arrive(bar + DSREADY);
        }
        if (ok && mbar_wait(bar + ACC, 0, w)) {
            tc_fence_after();
            auto row_of = [&](__nv_bfloat16 *base, long stride) {
                return [=](int i) {
                    const int rr = 32 * q4 + i;
                    return rr < it.n_key ? base + ((long)it.krow0 + rr) * stride + (long)hk * D + 64 * g : nullptr;
                };
            };
            store_rows(lb + 384 + 64 * g, smem + warp * 4096, lane, p.scale * pow2(-e), row_of(p.dk, p.dk_stride));
            store_rows(lb + 256 + 64 * g, smem + warp * 4096, lane, 1.0f, row_of(p.dv, p.dv_stride));
        }
    }
    teardown(tmem);
}

// Key tiles first (their steps are the longer ones), query tiles behind them:
// one grid, so that the GPU drains once.
__global__ void __launch_bounds__(pb::THREADS, 1)
    packed_bwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
                      const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const PackedBwdParams p) {
    wait_previous_kernel();
    extern __shared__ __align__(1024) uint8_t smem[];
    if (smem_u32(smem) & 1023u) {  // the same for every thread: the CTA leaves before any barrier
        if (threadIdx.x == 0) atomicCAS(p.err, DEV_OK, DEV_LAYOUT);
        return;
    }
    const PackedPlan plan = packed_plan_at(const_cast<void *>(p.plan), p.g);
    if (!packed_plan_ok(*plan.head, p.g)) {
        if (threadIdx.x == 0) atomicCAS(p.err, DEV_OK, DEV_PLAN);
        return;
    }
    const bool keys = blockIdx.x < p.dkv_blocks;
    const uint32_t u = keys ? blockIdx.x : blockIdx.x - p.dkv_blocks;
    const uint32_t n_items = (uint32_t)(keys ? plan.head->n_k : plan.head->n_q);
    if (u >= n_items * (uint32_t)p.g.Hkv) return;
    const int hk = (int)(u / n_items);
    if (keys) dkv_item(smem, tm_q, tm_do, tm_k, tm_v, p, plan.k[u - (uint32_t)hk * n_items], hk);
    else dq_item(smem, tm_q, tm_do, tm_k, tm_v, p, plan.q[u - (uint32_t)hk * n_items], hk);
}

}  // namespace

// Tiles of the pre-pass, counted from above, of queries and (with norms) of keys.
static long rows_units(const PackedGeom &g, bool norms) {
    return (g.Tq ? (long)g.cap_q * g.Hkv : 0) + (norms && g.Tk ? (long)g.cap_k * g.Hkv : 0);
}

// Warps of a team: eight rows each, for the rows that a tile has on average.  us, fp16, a call: 1,300 sequences of 20
// tokens, 24/24 heads, 2,760 with this rule, 3,150 with 16 warps for every tile; long sequences get 16 either way.
static int rows_team(const PackedGeom &g, bool norms) {
    const long rows = (long)g.Tq * g.H + (norms ? (long)g.Tk * g.Hkv : 0), units = rows_units(g, norms);
    int warps = 1;
    while (warps < ROWS_WARPS && units * warps * 8 < rows) warps *= 2;
    return warps;
}

// Blocks of the pre-pass: a tile for each of their teams, up to two blocks a SM.
unsigned packed_bwd_rows_blocks(const PackedGeom &g, bool norms) {
    const long teams = ROWS_WARPS / rows_team(g, norms), want = (rows_units(g, norms) + teams - 1) / teams;
    return (unsigned)(want < 2L * g.sms ? want : 2L * g.sms);
}

// Workspace: LD, then the tops.
struct BwdLayout {
    size_t row, tok, tile, key, ktile, total;
    explicit BwdLayout(const PackedGeom &p) {
        const size_t q = (size_t)p.Tq * p.Hkv, k = (size_t)p.Tk * p.Hkv;
        row = round256(q * p.G * sizeof(float2));
        tok = row + round256(q * p.G * sizeof(float));
        tile = tok + round256(q * sizeof(float2));
        key = tile + round256(q * sizeof(float2));
        ktile = key + round256(k * sizeof(float));
        total = ktile + round256(k * sizeof(float));
    }
};

size_t packed_bwd_workspace(const PackedGeom &p) { return BwdLayout(p).total; }

cudaError_t launch_packed_bwd(const PackedGeom &g, const PackedPtrs &t, const void *out, long out_stride,
                              const void *dout, long dout_stride, const float *lse, void *dq, long dq_stride,
                              void *dk, long dk_stride, void *dv, long dv_stride, void *ws, cudaStream_t st,
                              const char **why) {
    if (g.Tq == 0 && g.Tk == 0) return cudaSuccess;
    // a side without rows is never loaded: its maps get the other's
    const void *q = g.Tq ? t.q : t.k, *d_o = g.Tq ? dout : t.v, *k = g.Tk ? t.k : t.q, *v = g.Tk ? t.v : dout;
    PackedGeom gq = g;
    if (!g.Tq) gq.Tq = g.Tk, gq.H = g.Hkv, gq.G = 1, gq.tpt = 128;
    CUtensorMap mq, mdo, mk, mv;
    const long krows = g.Tk ? g.Tk : g.Tq;
    const int kheads = g.Tk ? g.Hkv : 1;
    if (!packed_q_map(&mq, q, gq, g.Tq ? t.q_stride : t.k_stride, why) ||
        !packed_q_map(&mdo, d_o, gq, g.Tq ? dout_stride : t.v_stride, why) ||
        !packed_kv_map(&mk, k, krows, kheads, g.Tk ? t.k_stride : t.q_stride, why) ||
        !packed_kv_map(&mv, v, krows, kheads, g.Tk ? t.v_stride : dout_stride, why))
        return cudaErrorInvalidValue;
    cudaError_t e = set_max_dynamic_smem((const void *)packed_bwd_kernel, pb::SMEM_ALLOC);
    if (e != cudaSuccess) return e;
    float2 *LD = static_cast<float2 *>(ws);
    PackedTops tops = {};
    if (t.qk_f16) {
        const BwdLayout at(g);
        char *w = static_cast<char *>(ws);
        tops.row = reinterpret_cast<float *>(w + at.row);
        tops.tok = reinterpret_cast<float2 *>(w + at.tok);
        tops.tile = reinterpret_cast<float2 *>(w + at.tile);
        tops.key = reinterpret_cast<float *>(w + at.key);
        tops.ktile = reinterpret_cast<float *>(w + at.ktile);
    }
    if (g.Tq) {
        auto rows = [&](auto kernel) {
            const int team = rows_team(g, t.qk_f16);
            const size_t smem = t.qk_f16 ? (size_t)(ROWS_WARPS / team) * 512 * sizeof(int) : 0;
            kernel<<<packed_bwd_rows_blocks(g, t.qk_f16), ROWS_THREADS, smem, st>>>(
                g, t.plan, static_cast<const char *>(out), out_stride * 2, static_cast<const char *>(dout),
                dout_stride * 2, static_cast<const char *>(t.v), t.v_stride * 2, lse, LD, tops, team);
        };
        if (t.qk_f16) rows(packed_bwd_rows_kernel<true>);
        else rows(packed_bwd_rows_kernel<false>);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    PackedBwdParams p;
    p.g = g;
    p.plan = t.plan;
    p.scale = (float)(1.0 / sqrt(128.0));
    p.scale_log2 = (float)(1.4426950408889634 / sqrt(128.0));
    p.LD = LD;
    p.tops = tops;
    p.dq = static_cast<__nv_bfloat16 *>(dq), p.dk = static_cast<__nv_bfloat16 *>(dk);
    p.dv = static_cast<__nv_bfloat16 *>(dv);
    p.dq_stride = dq_stride, p.dk_stride = dk_stride, p.dv_stride = dv_stride;
    // A/B formats: bits 7-9 and 10-12 (0 = fp16, 1 = bf16); bit 16: B MN-major
    const uint32_t f16 = idesc_bf16_f32(128, 128, false) & ~((7u << 7) | (7u << 10));
    const uint32_t bf16 = f16 | (1u << 7) | (1u << 10);
    p.idesc_qk = t.qk_f16 ? f16 : bf16;                    // S = Q K^T
    p.idesc_bf16 = bf16;                                   // dP = dO V^T
    p.idesc_bf16_mn = bf16 | (1u << 16);                   // dV += P^T dO
    p.idesc_ds_mn = (t.qk_f16 ? f16 : bf16) | (1u << 16);  // dQ += dS K, dK += dS^T Q
    p.ds_f16 = t.qk_f16 ? 1 : 0;
    p.inv_g = (65536u + (uint32_t)g.G - 1) / (uint32_t)g.G;
    p.wait_limit_ns = t.wait_limit_ns;
    p.err = t.err;
    p.dkv_blocks = g.Tk ? (uint32_t)((long)g.cap_k * g.Hkv) : 0;
    const uint32_t blocks = p.dkv_blocks + (g.Tq ? (uint32_t)((long)g.cap_q * g.Hkv) : 0);
    return launch_after(packed_bwd_kernel, blocks, pb::THREADS, pb::SMEM_ALLOC, st, mq, mdo, mk, mv, p);
}

}  // namespace k6
