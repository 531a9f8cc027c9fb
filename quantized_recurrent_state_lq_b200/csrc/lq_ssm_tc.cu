// lq_ssm_tc.cu -- the selective state-space scan of f32 and f16 prompts in
// chunks of 32 tokens, on mma.sync m16n8k8 TF32 tiles with FP32-level accuracy.
//
// The chunk form is that of lq_ssm_umma.cu.  One CTA takes one head over one
// piece of a sequence; warp w keeps the transposed state of its 16 value
// columns, S^T [16][dk], in registers as accumulator tiles.  With the key rows
// of every 8-row block read in the order 0, 2, 4, 6, 1, 3, 5, 7 the same
// registers are the A operand of S^T C^T, so the state is never stored:
//   G = C B^T (lower tiles, shared among the warps), M = 2^(g_t - g_s) d_s G
//   Y^T = 2^(g_t) (S^T C^T) + X^T M^T + D X^T
//   S^T <- 2^(g_Q) S^T + X'^T B,  X'[s] = 2^(g_Q - g_s) d_s X[s]
// f16 operands are exact in TF32; S, M and X' (and f32 operands) enter as two
// TF32 parts, big x big + big x small + small x big: about 2^-22 of a term.
// Bound: with few CTAs latency (a chunk of a 64 x 64 head 10000 cycles, f32: rows
// 2000, G 2600, C S 1900, M X and the state 2700), with many the rate of mma.sync:
// two CTAs per SM for 128 value columns, four for 64.  3001 f16 tokens of 6 heads
// of 64 x 128: 35 us; 16384 f32 tokens of 16 heads of 128 x 128: 840 us.
#include "lq_ssm.h"

namespace lq {
namespace {

constexpr int Q = 32;   // tokens per chunk

__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// x = big + small, both rounded to TF32 (nearest, by adding half a unit to the
// bits): within 2^-22 of x.  Where that would pass the largest TF32 value (the last
// 2^-11 of the FP32 range) big is cut instead and small takes what is left; an
// infinity or a NaN is not finite in big, and small is whatever it is beside it.
__device__ __forceinline__ void split(float x, uint32_t &big, uint32_t &small) {
    const uint32_t u = __float_as_uint(x);
    big = (fabsf(x) < __int_as_float(0x7f7ff000) ? u + 0x1000u : u) & 0xffffe000u;
    small = (__float_as_uint(x - __uint_as_float(big)) + 0x1000u) & 0xffffe000u;
}

// c += A B with A in two parts and B exact in TF32.
__device__ __forceinline__ void mma_exact(float (&c)[4], const uint32_t (&ab)[4], const uint32_t (&as)[4], float b0,
                                          float b1) {
    mma_tf32(c, as, __float_as_uint(b0), __float_as_uint(b1));
    mma_tf32(c, ab, __float_as_uint(b0), __float_as_uint(b1));
}

// A B with both in two parts: the products of the big parts into c, the others
// (2^-11 of them) into d.  The tensor core's accumulation does not round to
// nearest, so f32 results keep their chains of large terms short: apart from the
// small ones, from the running state and (even and odd steps) from each other.
__device__ __forceinline__ void mma_split(float (&c)[4], float (&d)[4], const uint32_t (&ab)[4], const uint32_t (&as)[4],
                                          float b0, float b1) {
    uint32_t bb[2], bs[2];
    split(b0, bb[0], bs[0]);
    split(b1, bb[1], bs[1]);
    mma_tf32(d, as, bb[0], bb[1]);
    mma_tf32(d, ab, bs[0], bs[1]);
    mma_tf32(c, ab, bb[0], bb[1]);
}

__device__ __forceinline__ void split4(const float (&v)[4], uint32_t (&big)[4], uint32_t (&small)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) split(v[e], big[e], small[e]);
}

template <int DK, int DV>
struct Tiles {
    float C[Q][DK + 8];    // rows 8 banks apart: 8-byte fragments without conflicts
    float B[Q][DK + 4];    // rows 4 banks apart: its columns' fragments without
    float X[Q][DV + 4];    // and the outputs, at the end
    float M[Q][Q + 8];
    // of even and odd chunks:
    long long g[2][Q];     // log2 decay from the chunk's start (fixed point)
    float d[2][Q], eg[2][Q], w[2][Q];   // steps, 2^g, weights in the next state
    int first[2][DV];      // per value column, the first token whose x is not finite
    float keep[2];         // 2^(g_Q)
};

// Q rows of W elements as floats (zeros from the sequence's end on).  With first,
// an element that is not finite is replaced by 0 (times 0 it would reach earlier
// tokens) and its column marked from that token on.
template <typename T, int W, int NT, int LD>
__device__ __forceinline__ void load_rows(float (&dst)[Q][LD], const T *src, int64_t ld, const Piece &p, int t0,
                                          bool vec, int *first = nullptr) {
    auto finite = [&](float v, int t, int c) {
        if (fabsf(v) <= 3.402823466e38f) return v;
        atomicMin(first + c, t);
        return 0.0f;
    };
    if (vec) {
#pragma unroll
        for (int i = 0; i < Q * W / 8 / NT; ++i) {
            const int e = i * NT + threadIdx.x, t = e / (W / 8), j = e % (W / 8);
            Raw<T, 8> v;
            if (t0 + t < p.len) v.load(src + (p.row0 + (int64_t)(t0 + t) * p.step) * ld + 8 * j);
            else v.zero();
            float f[8];
            v.get(f);
            if (first)
#pragma unroll
                for (int k = 0; k < 8; ++k) f[k] = finite(f[k], t, 8 * j + k);
            float4 *o = reinterpret_cast<float4 *>(&dst[t][8 * j]);
            o[0] = make_float4(f[0], f[1], f[2], f[3]);
            o[1] = make_float4(f[4], f[5], f[6], f[7]);
        }
    } else {
        for (int e = threadIdx.x; e < Q * W; e += NT) {
            const int t = e / W, j = e % W;
            float v = t0 + t < p.len ? to_f<T>(src[(p.row0 + (int64_t)(t0 + t) * p.step) * ld + j]) : 0.0f;
            if (first) v = finite(v, t, j);
            dst[t][j] = v;
        }
    }
}

template <typename T, int DK, int DV, bool FULL>
__global__ void __launch_bounds__(2 * DV, DV == 128 ? 2 : 4) ssm_tc_kernel(SsmArgs a, int seg, int vec, int cut) {
    constexpr int NT = 2 * DV, NW = NT / 32;
    constexpr int PB = sizeof(T) == 4 ? 2 : 1;   // parts of B, C and X
    extern __shared__ __align__(16) unsigned char smem[];
    Tiles<DK, DV> &s = *reinterpret_cast<Tiles<DK, DV> *>(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gq = lane >> 2, tq = lane & 3;
    const int z = blockIdx.x / a.H, h = blockIdx.x % a.H;
    Piece p;
    const bool found = FULL ? find_piece(a.r, seg, z, p) : find_cut(a.r, seg, z, p);
    if (FULL) wait_for_kernel_before();
    if (!found) return;
    const int g = (int)((int64_t)h * a.G / a.H);
    const T *xp = static_cast<const T *>(a.x) + (int64_t)h * DV;
    const T *bp = static_cast<const T *>(a.Bm) + g * DK;
    const T *cp = static_cast<const T *>(a.Cm) + g * DK;
    const T *dp = static_cast<const T *>(a.dt) + h;
    const float A2 = a.A[h] * 1.4426950408889634f;   // log2 decay per unit step
    const float Dh = a.D ? a.D[h] : 0.0f, bias = a.dt_bias ? a.dt_bias[h] : 0.0f;
    const int pc = 16 * warp;   // this warp's value columns

    // S^T tile i: value columns pc + gq (+8), key rows 8 i + 2 tq (+1).
    float S[DK / 8][4];
    const int64_t sall = (int64_t)a.H * DK * DV, soff = (int64_t)h * DK * DV + pc + gq;
    const float *S0 = nullptr;
    if (FULL) {
        if (cut && p.n > 1) S0 = a.ws + p.id * sall + soff;
        else if (a.S0) S0 = a.S0 + p.b * sall + soff;
    }
#pragma unroll
    for (int i = 0; i < DK / 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[i][e] = S0 ? S0[(8 * i + 2 * tq + (e & 1)) * DV + (e >> 1) * 8] : 0.0f;

    // The last warp, whose share of the products before it is the least, forms the
    // decays of the chunk at t, a chunk ahead.
    const bool decays = warp == NW - 1;
    const int t_end = min(p.len, (p.j + 1) * seg);
    long long gsum = 0;
    auto step_at = [&](int t) {
        return t + lane < p.len ? to_f<T>(dp[(p.row0 + (int64_t)(t + lane) * p.step) * a.lddt]) : 0.0f;
    };
    auto form_decays = [&](float d, int t, int odd) {
        long long gt = 0;
        if (t + lane < p.len) {
            d += bias;
            if (a.softplus) d = softplus_f(d);
            gt = decay_of(d, A2);
        }
        gt = warp_scan(gt);
        const long long total = __shfl_sync(0xffffffffu, gt, 31);
        s.g[odd][lane] = gt;
        s.d[odd][lane] = d;
        s.eg[odd][lane] = exp2f(decay_f(gt));
        s.w[odd][lane] = d * exp2f(decay_f(total - gt));
        if (lane == 0) s.keep[odd] = exp2f(decay_f(total));
        gsum += total;
    };
    if (tid < DV) s.first[0][tid] = Q;
    if (decays && p.j * seg < t_end) form_decays(step_at(p.j * seg), p.j * seg, 0);

    int odd = 0;
    for (int t0 = p.j * seg; t0 < t_end; t0 += Q, odd ^= 1) {
        __syncthreads();   // the chunk before is done with the tiles
        const bool next = decays && t0 + Q < t_end;
        const float dn = next ? step_at(t0 + Q) : 0.0f;
        load_rows<T, DK, NT>(s.B, bp, a.ldb, p, t0, vec);
        load_rows<T, DV, NT>(s.X, xp, a.ldx, p, t0, vec, s.first[odd]);
        if (FULL) load_rows<T, DK, NT>(s.C, cp, a.ldc, p, t0, vec);
        if (tid < DV) s.first[odd ^ 1][tid] = Q;
        __syncthreads();
        if (FULL) {
            // lower 16 x 8 tiles of G, one at a time per warp
            for (int tile = warp; tile < 6; tile += NW) {
                const int rb = tile < 2 ? 0 : 16, cb = tile < 2 ? 8 * tile : 8 * (tile - 2);
                float acc[2][4] = {}, low[4] = {};   // two chains
#pragma unroll 4
                for (int k = 0; k < DK; k += 8) {
                    const float2 c0 = *reinterpret_cast<const float2 *>(&s.C[rb + gq][k + 2 * tq]);
                    const float2 c1 = *reinterpret_cast<const float2 *>(&s.C[rb + gq + 8][k + 2 * tq]);
                    const float2 b = *reinterpret_cast<const float2 *>(&s.B[cb + gq][k + 2 * tq]);
                    float(&c)[4] = acc[(k >> 3) & 1];
                    if constexpr (PB == 1) {
                        const uint32_t ar[4] = {__float_as_uint(c0.x), __float_as_uint(c1.x), __float_as_uint(c0.y),
                                                __float_as_uint(c1.y)};
                        mma_tf32(c, ar, __float_as_uint(b.x), __float_as_uint(b.y));
                    } else {
                        uint32_t ab[4], as[4];
                        const float av[4] = {c0.x, c1.x, c0.y, c1.y};
                        split4(av, ab, as);
                        mma_split(c, low, ab, as, b.x, b.y);
                    }
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int t = rb + gq + (e >> 1) * 8, u = cb + 2 * tq + (e & 1);
                    s.M[t][u] = u <= t ? exp2f(decay_f(s.g[odd][t] - s.g[odd][u])) * s.d[odd][u] * (acc[0][e] + acc[1][e] + low[e]) : 0.0f;
                }
            }
        }
        if (next) form_decays(dn, t0 + Q, odd ^ 1);
        float Y[Q / 8][4] = {};   // Y^T tile j: value columns pc + gq (+8), tokens 8 j + 2 tq (+1)
        if (FULL) {
            // (All token blocks in one pass over S: taken two at a time, S's parts are
            // kept for the second pass and spill, 944 us against 840 for 16384 tokens of
            // 16 f32 heads of 128 x 128.)
            float alt[Q / 8][4] = {}, low[Q / 8][4] = {};
#pragma unroll
            for (int i = 0; i < DK / 8; ++i) {
                uint32_t ab[4], as[4];
                const float sv[4] = {S[i][0], S[i][2], S[i][1], S[i][3]};
                split4(sv, ab, as);
#pragma unroll
                for (int j = 0; j < Q / 8; ++j) {
                    const float2 c = *reinterpret_cast<const float2 *>(&s.C[8 * j + gq][8 * i + 2 * tq]);
                    if constexpr (PB == 1) mma_exact(Y[j], ab, as, c.x, c.y);
                    else mma_split(i & 1 ? alt[j] : Y[j], low[j], ab, as, c.x, c.y);
                }
            }
            if constexpr (PB == 2)
#pragma unroll
                for (int j = 0; j < Q / 8; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) Y[j][e] += alt[j][e] + low[j][e];
#pragma unroll
            for (int j = 0; j < Q / 8; ++j) {
                const float e0 = s.eg[odd][8 * j + 2 * tq], e1 = s.eg[odd][8 * j + 2 * tq + 1];
                Y[j][0] *= e0; Y[j][1] *= e1; Y[j][2] *= e0; Y[j][3] *= e1;
            }
        }
        __syncthreads();   // M
        const float keep = s.keep[odd];
        auto x_at = [&](int u, float (&x)[4]) {
            x[0] = s.X[u][pc + gq];
            x[1] = s.X[u][pc + gq + 8];
            x[2] = s.X[u + 1][pc + gq];
            x[3] = s.X[u + 1][pc + gq + 8];
        };
        if constexpr (PB == 1) {
#pragma unroll
            for (int i = 0; i < DK / 8; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) S[i][e] *= keep;
#pragma unroll
            for (int k = 0; k < Q / 8; ++k) {   // 8 tokens
                const int u = 8 * k + 2 * tq;
                float x[4];
                x_at(u, x);
                if (FULL) {
                    const uint32_t ar[4] = {__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                                            __float_as_uint(x[3])};
#pragma unroll
                    for (int j = k; j < Q / 8; ++j) {
                        const float2 m = *reinterpret_cast<const float2 *>(&s.M[8 * j + gq][u]);
                        uint32_t mb[2], ms[2];
                        split(m.x, mb[0], ms[0]);
                        split(m.y, mb[1], ms[1]);
                        mma_tf32(Y[j], ar, ms[0], ms[1]);
                        mma_tf32(Y[j], ar, mb[0], mb[1]);
                    }
                }
                const float w0 = s.w[odd][u], w1 = s.w[odd][u + 1];
                const float xw[4] = {x[0] * w0, x[1] * w0, x[2] * w1, x[3] * w1};
                uint32_t ab[4], as[4];
                split4(xw, ab, as);
#pragma unroll
                for (int i = 0; i < DK / 8; ++i) mma_exact(S[i], ab, as, s.B[u][8 * i + gq], s.B[u + 1][8 * i + gq]);
            }
        } else {
            if (FULL)
#pragma unroll
                for (int j = 0; j < Q / 8; ++j) {
                    float acc[4] = {}, low[4] = {};
#pragma unroll
                    for (int k = 0; k <= j; ++k) {
                        const int u = 8 * k + 2 * tq;
                        float x[4];
                        x_at(u, x);
                        uint32_t ab[4], as[4];
                        split4(x, ab, as);
                        const float2 m = *reinterpret_cast<const float2 *>(&s.M[8 * j + gq][u]);
                        mma_split(acc, low, ab, as, m.x, m.y);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) Y[j][e] += acc[e] + low[e];
                }
#pragma unroll
            for (int kb = 0; kb < Q / 8; kb += 2) {   // 16 tokens
                uint32_t ab[2][4], as[2][4];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int u = 8 * (kb + k) + 2 * tq;
                    float x[4];
                    x_at(u, x);
                    const float w0 = s.w[odd][u], w1 = s.w[odd][u + 1];
                    const float xw[4] = {x[0] * w0, x[1] * w0, x[2] * w1, x[3] * w1};
                    split4(xw, ab[k], as[k]);
                }
#pragma unroll
                for (int i = 0; i < DK / 8; ++i) {
                    float acc[4] = {}, low[4] = {};
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int u = 8 * (kb + k) + 2 * tq;
                        mma_split(acc, low, ab[k], as[k], s.B[u][8 * i + gq], s.B[u + 1][8 * i + gq]);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) S[i][e] = fmaf(kb == 0 ? keep : 1.0f, S[i][e], acc[e] + low[e]);
                }
            }
        }
        // from a non-finite x on, its column has no finite state
        const int f0 = s.first[odd][pc + gq], f1 = s.first[odd][pc + gq + 8];
        const float nan = __int_as_float(0x7fffffff);
        if (f0 < Q || f1 < Q)
#pragma unroll
            for (int i = 0; i < DK / 8; ++i) {
                if (f0 < Q) S[i][0] = S[i][1] = nan;
                if (f1 < Q) S[i][2] = S[i][3] = nan;
            }
        if (FULL) {
            __syncwarp();   // this warp's columns of X have been read
#pragma unroll
            for (int j = 0; j < Q / 8; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int t = 8 * j + 2 * tq + (e & 1), c = pc + gq + (e >> 1) * 8;
                    const float y = fmaf(Dh, s.X[t][c], Y[j][e]);
                    s.X[t][c] = t >= ((e >> 1) ? f1 : f0) ? nan : y;
                }
            __syncthreads();
            T *yp = static_cast<T *>(a.y) + (int64_t)h * DV;
            if (vec) {
#pragma unroll
                for (int i = 0; i < Q * DV / 8 / NT; ++i) {
                    const int e = i * NT + tid, t = e / (DV / 8), j = e % (DV / 8);
                    const float4 *o = reinterpret_cast<const float4 *>(&s.X[t][8 * j]);
                    const float4 u = o[0], v = o[1];
                    const float f[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
                    Raw<T, 8> ry;
                    ry.set(f);
                    if (t0 + t < p.len) ry.store(yp + (p.row0 + (int64_t)(t0 + t) * p.step) * a.ldy + 8 * j);
                }
            } else {
                for (int e = tid; e < Q * DV; e += NT) {
                    const int t = e / DV, j = e % DV;
                    if (t0 + t < p.len) yp[(p.row0 + (int64_t)(t0 + t) * p.step) * a.ldy + j] = from_f<T>(s.X[t][j]);
                }
            }
        }
    }
    if (!FULL || p.j == p.n - 1) {
        float *so = (FULL ? a.S_out + p.b * sall : a.ws + p.id * sall) + soff;
#pragma unroll
        for (int i = 0; i < DK / 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) so[(8 * i + 2 * tq + (e & 1)) * DV + (e >> 1) * 8] = S[i][e];
    }
    if (!FULL && tid == NT - 32) ssm_decays(a, seg)[p.id * a.H + h] = exp2f(decay_f(gsum));
}

template <typename T, int DK, int DV>
cudaError_t launch(const SsmArgs &a, int seg, int vec, bool cut, cudaStream_t s) {
    constexpr int bytes = (int)sizeof(Tiles<DK, DV>), NT = 2 * DV;
    cudaError_t e = cudaFuncSetAttribute(ssm_tc_kernel<T, DK, DV, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         bytes);
    if (e != cudaSuccess) return e;
    if (cut) {
        e = cudaFuncSetAttribute(ssm_tc_kernel<T, DK, DV, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        ssm_tc_kernel<T, DK, DV, false><<<(unsigned)(cut_count(a.r, seg) * a.H), NT, bytes, s>>>(a, seg, vec, cut);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        e = launch_ssm_join(a, seg, false, s);
        if (e != cudaSuccess) return e;
        return launch_after(ssm_tc_kernel<T, DK, DV, true>, dim3((unsigned)(piece_count(a.r, seg) * a.H)), NT, bytes, s, a,
                            seg, vec, cut);
    }
    ssm_tc_kernel<T, DK, DV, true><<<(unsigned)(piece_count(a.r, seg) * a.H), NT, bytes, s>>>(a, seg, vec, cut);
    return cudaGetLastError();
}

template <typename T>
cudaError_t by_size(const SsmArgs &a, int seg, bool cut, cudaStream_t s) {
    const uintptr_t base = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.Bm) |
                           reinterpret_cast<uintptr_t>(a.Cm) | reinterpret_cast<uintptr_t>(a.y);
    const int u = 16 / (int)sizeof(T);
    const int vec = base % 16 == 0 && a.ldx % u == 0 && a.ldb % u == 0 && a.ldc % u == 0 && a.ldy % u == 0;
    if (a.dk == 64) return a.dv == 64 ? launch<T, 64, 64>(a, seg, vec, cut, s) : launch<T, 64, 128>(a, seg, vec, cut, s);
    return a.dv == 64 ? launch<T, 128, 64>(a, seg, vec, cut, s) : launch<T, 128, 128>(a, seg, vec, cut, s);
}

}  // namespace

cudaError_t launch_ssm_tc(const SsmArgs &a, int dtype, int seg, bool cut, cudaStream_t s) {
    return dtype == kF32 ? by_size<float>(a, seg, cut, s) : by_size<f16>(a, seg, cut, s);
}

}  // namespace lq
