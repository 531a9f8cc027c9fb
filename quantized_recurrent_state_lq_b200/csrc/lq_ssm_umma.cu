// lq_ssm_umma.cu -- the selective state-space scan of bf16 prompts in chunks of
// 128 tokens on the fifth-generation tensor cores.
//
// Per chunk, with g_t the cumulative log2 decay from the chunk's start:
//   G = C B^T                                    (128 x 128, K = dk)
//   M[t][s] = 2^(g_t - g_s) d_s G[t][s], s <= t
//   Y = 2^(g_t) (C S) + M X + D X
//   S <- 2^(g_Q) S + B^T X',  X'[s] = 2^(g_Q - g_s) d_s X[s]
// B, C and X are exact operands.  S and M enter as two bf16 parts (2^-17: Y is
// rounded to bf16, half a step 2^-9), X' as three (2^-25: the state is FP32);
// accumulators are FP32 in tensor memory, the state itself stays in FP32
// registers.  Every decay factor is 2^(difference), later token first, so a
// decaying state never forms a factor above 1.
//
// A CTA of four warps takes 64 value columns of one head over one piece of a
// sequence; thread r is token r, key row r and tensor-memory lane r.  Phases
// alternate between the tensor core and the threads, and two CTAs per SM (256
// tensor-memory columns, 112 KB of shared memory each) fill each other's gaps.
// Long sequences of a small batch are cut into pieces: a first pass forms each
// piece's own state, ssm_join_kernel chains them, the second pass starts every
// piece from its state (about a third more work for pieces x as much
// parallelism).
//
// Shared memory holds every operand as 16-byte chunks of 8 columns, chunk
// column j of 128 rows at 2048 j, row t at 16 t: read as rows x K it is
// K-major without swizzle, read as K x columns it is MN-major, so B serves
// C B^T and B^T X' from one copy.  A warp's 16-byte accesses touch 8
// consecutive rows of a chunk column (no bank conflicts).
//   [0, 32K) C, [32K, 64K) S parts   -- until C B^T and C S are done; then
//   [0, 48K) X' parts, [48K, ..) decay factors
//   [64K, 96K) B, [96K, 112K) X
#include "lq_act.cuh"
#include "lq_ssm.h"
#include "lq_tc.cuh"

namespace lq {
namespace {

constexpr int Q = 128;                 // tokens per chunk
constexpr int PW = 64;                 // value columns per CTA
constexpr int kNT = 128;
constexpr uint32_t kChunkB = Q * 16;   // bytes of a chunk column
constexpr int kOffC = 0, kOffS = 32768, kOffXw = 0, kOffF = 49152, kOffB = 65536, kOffX = 98304;
constexpr int kSmem = 114688;
constexpr uint32_t kTmemCols = 256, kColY = 128, kColS = 192;   // G and M: columns 0..127

// Instruction descriptors, kind::f16 with bf16 operands and FP32 accumulators.
constexpr uint32_t idesc(int N, int a_mn, int b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
           ((uint32_t)(N >> 3) << 17) | (8u << 24);   // M = 128
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t ad, uint64_t bd, uint32_t id, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(ad), "l"(bd), "r"(id), "r"(acc)
        : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t at, uint64_t bd, uint32_t id, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(at), "l"(bd), "r"(id), "r"(acc)
        : "memory");
}

// K-major: 8-row groups 128 B apart, chunk columns along K 2048 B apart.
__device__ __forceinline__ uint64_t desc_k(const void *p) { return umma_smem_desc(p, kChunkB, 128); }
// MN-major: 8-row groups along K 128 B apart, chunk columns 2048 B apart.
__device__ __forceinline__ uint64_t desc_mn(const void *p) { return umma_smem_desc(p, 128, kChunkB); }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool full) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(full ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// bf16 parts of a pair: returns the pair rounded to bf16 and leaves the rests.
__device__ __forceinline__ uint32_t take_part(float &a, float &b) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    const uint32_t w = *reinterpret_cast<const uint32_t *>(&p);
    a -= __uint_as_float(w << 16);
    b -= __uint_as_float(w & 0xffff0000u);
    return w;
}
__device__ __forceinline__ uint32_t last_part(float a, float b) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&p);
}

// Rows t0 .. t0 + Q - 1 of a sequence (zeros from `len` on), NCH chunks of 8
// elements each, into chunk columns.
template <int NCH>
__device__ __forceinline__ void load_tile(unsigned char *dst, const bf16 *src, int64_t ld, const Piece &p, int t0,
                                          bool vec) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < 16 * (NCH / 4) / 4; ++i) {
        const int grp = i * 4 + warp;                 // 8 rows x 4 chunks
        const int t = (grp & 15) * 8 + (lane & 7), j = (grp >> 4) * 4 + (lane >> 3);
        const bool in = t0 + t < p.len;
        const bf16 *s = src + (p.row0 + (in ? t0 + t : t0) * p.step) * ld + 8 * j;
        unsigned char *d = dst + j * kChunkB + t * 16;
        if (vec) {
            cp_async16(smem_u32(d), s, in);
        } else {
            uint32_t w[4] = {0u, 0u, 0u, 0u};
            const uint16_t *e = reinterpret_cast<const uint16_t *>(s);
            if (in)
#pragma unroll
                for (int k = 0; k < 4; ++k) w[k] = (uint32_t)e[2 * k] | ((uint32_t)e[2 * k + 1] << 16);
            *reinterpret_cast<uint4 *>(d) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

struct Fixed {
    uint64_t bar[3];     // G and C S done, Y done, B^T X' done
    double wsum[4];      // each warp's log2 decay
    uint32_t tmem;
    int bad;             // a wait ran out
    int nf;              // a non-finite x in this chunk
    int first[PW];       // per value column, the first token whose x is not finite
};

// FULL: outputs and the final state; else only the pieces' own states (from
// zero) and decays, for all but the last piece of each sequence.
template <bool FULL, int DK>
__global__ void __launch_bounds__(kNT, 2) ssm_umma_kernel(SsmArgs a, int seg, int units, int vec, int split) {
    extern __shared__ __align__(128) unsigned char sm[];
    __shared__ Fixed fx;
    const int r = threadIdx.x, warp = r >> 5, lane = r & 31;
    const int z = blockIdx.x / units, u = blockIdx.x % units;
    Piece p;
    if (!find_piece(a.r, seg, z, p) || (!FULL && p.j >= p.n - 1)) return;
    const int per = a.dv / PW;
    const int h = u / per, c0 = (u % per) * PW;
    const int g = (int)((int64_t)h * a.G / a.H);
    const bf16 *xp = static_cast<const bf16 *>(a.x) + (int64_t)h * a.dv + c0;
    const bf16 *bp = static_cast<const bf16 *>(a.Bm) + g * DK;
    const bf16 *cp = static_cast<const bf16 *>(a.Cm) + g * DK;
    const bf16 *dp = static_cast<const bf16 *>(a.dt) + h;
    const float A2 = a.A[h] * 1.4426950408889634f;   // log2 decay per unit step
    const float Dh = a.D ? a.D[h] : 0.0f, bias = a.dt_bias ? a.dt_bias[h] : 0.0f;

    if (warp == 0) tmem_alloc(&fx.tmem, kTmemCols);
    if (r == 0) {
        for (int i = 0; i < 3; ++i) mbar_init(&fx.bar[i], 1);
        fx.bad = 0;
        fence_mbar_init();
    }
    if (DK < 128) {   // B^T has 128 rows: the missing key rows are zero
        for (int i = r; i < (128 - DK) / 8 * (int)kChunkB / 16; i += kNT)
            reinterpret_cast<uint4 *>(sm + kOffB + DK / 8 * kChunkB)[i] = make_uint4(0u, 0u, 0u, 0u);
    }

    // The state's key row r, this CTA's columns.
    float S[PW];
    const int64_t soff = ((int64_t)h * DK + r) * a.dv + c0, sall = (int64_t)a.H * DK * a.dv;
    const float *S0 = nullptr;
    if (FULL && r < DK) {
        if (split && p.n > 1) S0 = a.ws + z * sall + soff;
        else if (a.S0) S0 = a.S0 + p.b * sall + soff;
    }
#pragma unroll
    for (int i = 0; i < PW / 4; ++i) {
        const float4 v = S0 ? reinterpret_cast<const float4 *>(S0)[i] : make_float4(0.f, 0.f, 0.f, 0.f);
        S[4 * i] = v.x; S[4 * i + 1] = v.y; S[4 * i + 2] = v.z; S[4 * i + 3] = v.w;
    }
    double gsum = 0.0;   // log2 decay of the piece so far
    const int t_end = min(p.len, (p.j + 1) * seg);
    int parity = 0;
    for (int t0 = p.j * seg; t0 < t_end; t0 += Q, parity ^= 1) {
        tc_fence_before();
        __syncthreads();   // the chunk before is done with shared and tensor memory
        if (fx.bad) break;
        load_tile<DK / 8>(sm + kOffB, bp, a.ldb, p, t0, vec);
        load_tile<PW / 8>(sm + kOffX, xp, a.ldx, p, t0, vec);
        if (FULL) load_tile<DK / 8>(sm + kOffC, cp, a.ldc, p, t0, vec);
        // This token's step and log2 decay, floored at -150 (a factor FP32
        // flushes to 0) so that no difference of sums is inf - inf; a NaN
        // passes the comparison by.
        float d = 0.0f, l = 0.0f;
        if (t0 + r < p.len) {
            d = __bfloat162float(dp[(p.row0 + (t0 + r) * p.step) * a.lddt]) + bias;
            if (a.softplus) d = softplus_f(d);
            l = d * A2;
            if (l < -150.0f) l = -150.0f;
        }
        double gw = l;   // inclusive sum within the warp
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const double o = __shfl_up_sync(0xffffffffu, gw, m);
            if (lane >= m) gw += o;
        }
        if (lane == 31) fx.wsum[warp] = gw;
        if (r == 0) fx.nf = 0;
        if (r < PW) fx.first[r] = Q;
        if (FULL && r < DK) {   // the state's two parts, chunk column by chunk column
#pragma unroll
            for (int j = 0; j < PW / 8; ++j) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float v0 = S[8 * j + 2 * k], v1 = S[8 * j + 2 * k + 1];
                    hi[k] = take_part(v0, v1);
                    lo[k] = last_part(v0, v1);
                }
                unsigned char *s = sm + kOffS + j * kChunkB + r * 16;
                *reinterpret_cast<uint4 *>(s) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4 *>(s + 16384) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
        }
        cp_async_wait();
        fence_async_smem();
        __syncthreads();
        const uint32_t tm = fx.tmem, tl = tm + ((uint32_t)warp << 21);   // this warp's lanes: 32 warp
        if (FULL && r == 0) {
            tc_fence_after();
            const uint64_t cd = desc_k(sm + kOffC), bd = desc_k(sm + kOffB), sd = desc_mn(sm + kOffS);
#pragma unroll
            for (int k = 0; k < DK / 16; ++k)
                mma_ss(tm, cd + (k * 2 * kChunkB >> 4), bd + (k * 2 * kChunkB >> 4), idesc(Q, 0, 0), k > 0);
#pragma unroll
            for (int part = 0; part < 2; ++part)
#pragma unroll
                for (int k = 0; k < DK / 16; ++k)
                    mma_ss(tm + kColY, cd + (k * 2 * kChunkB >> 4), sd + ((part * 16384 + k * 256) >> 4),
                           idesc(PW, 0, 1), part + k > 0);
            umma_commit(&fx.bar[0]);
        }
        double base = 0.0, total = 0.0;   // before this warp, and of the chunk
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            if (w < warp) base += fx.wsum[w];
            total += fx.wsum[w];
        }
        const double gt = base + gw;
        const float wr = d * exp2f((float)(total - gt));   // weight of this token in the next state
        if (FULL && !mbar_wait_bounded(&fx.bar[0], parity, nullptr)) fx.bad = 1;
        __syncwarp();
        tc_fence_after();
        float *fl = reinterpret_cast<float *>(sm + kOffF);   // [Q] sums within the warp, [Q] d, [3][Q] factors
        if (FULL) {
            fl[r] = (float)gw;
            fl[Q + r] = d;
            double end = 0.0;   // sum up to warp w: 2^(end - g_s) d_s for the rows of later warps
#pragma unroll
            for (int w = 0; w < 3; ++w) {
                end += fx.wsum[w];
                if (w >= warp) fl[(2 + w) * Q + r] = d * exp2f((float)(end - gt));
            }
        }
        // X' of this token in three parts; a non-finite x leaves X (times 0 it
        // would reach earlier tokens) and is marked instead.
#pragma unroll
        for (int j = 0; j < PW / 8; ++j) {
            unsigned char *s = sm + kOffX + j * kChunkB + r * 16;
            Raw<bf16, 8> rx;
            rx.a = *reinterpret_cast<const uint4 *>(s);
            float f[8];
            rx.get(f);
            float sum = 0.0f;   // 0 x finite = 0, else NaN
#pragma unroll
            for (int k = 0; k < 8; ++k) sum = fmaf(0.0f, f[k], sum);
            uint32_t w[3][4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float v0 = wr * f[2 * k], v1 = wr * f[2 * k + 1];
                w[0][k] = take_part(v0, v1);
                w[1][k] = take_part(v0, v1);
                w[2][k] = last_part(v0, v1);
            }
#pragma unroll
            for (int i = 0; i < 3; ++i)
                *reinterpret_cast<uint4 *>(sm + kOffXw + i * 16384 + j * kChunkB + r * 16) =
                    make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
            if (FULL && sum != 0.0f) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (!isfinite(f[k])) {
                        f[k] = 0.0f;
                        atomicMin(&fx.first[8 * j + k], r);
                    }
                rx.set(f);
                *reinterpret_cast<uint4 *>(s) = rx.a;
                fx.nf = 1;
            }
        }
        __syncwarp();
        if (FULL) {
            const float et = ex2((float)gt);   // 2^(g_t), on C S
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                uint32_t v[32];
                tmem_ld_32x32b<32>(tl + kColY + 32 * q, v);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(et * __uint_as_float(v[i]));
                tmem_st_32x32b_x32(tl + kColY + 32 * q, v);
            }
            __syncthreads();   // the factors
            // M over G, 32 columns at a time: 16 columns of first parts, 16 of
            // second.  Columns of earlier warps' tokens factor through the
            // boundary before this warp, later ones are zero.
            const float rf = ex2((float)gw);
            for (int q = 0; q < 4; ++q) {
                uint32_t v[32];
                if (q > warp) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = 0u;
                } else {
                    tmem_ld_32x32b<32>(tl + 32 * q, v);
                    tmem_ld_wait();
                    uint32_t hi[16], lo[16];
                    if (q < warp) {
                        const float4 *cf = reinterpret_cast<const float4 *>(fl + (1 + warp) * Q + 32 * q);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float4 c = cf[i];
                            float m[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
                            for (int k = 0; k < 4; ++k) m[k] *= rf * __uint_as_float(v[4 * i + k]);
                            hi[2 * i] = take_part(m[0], m[1]);
                            hi[2 * i + 1] = take_part(m[2], m[3]);
                            lo[2 * i] = last_part(m[0], m[1]);
                            lo[2 * i + 1] = last_part(m[2], m[3]);
                        }
                    } else {
                        const float4 *gs = reinterpret_cast<const float4 *>(fl + 32 * q);
                        const float4 *ds = reinterpret_cast<const float4 *>(fl + Q + 32 * q);
                        const float gwf = (float)gw;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float4 gv = gs[i], dv = ds[i];
                            const float ge[4] = {gv.x, gv.y, gv.z, gv.w}, de[4] = {dv.x, dv.y, dv.z, dv.w};
                            float m[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const float e = ex2(gwf - ge[k]) * de[k] * __uint_as_float(v[4 * i + k]);
                                m[k] = 4 * i + k <= lane ? e : 0.0f;
                            }
                            hi[2 * i] = take_part(m[0], m[1]);
                            hi[2 * i + 1] = take_part(m[2], m[3]);
                            lo[2 * i] = last_part(m[0], m[1]);
                            lo[2 * i + 1] = last_part(m[2], m[3]);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        v[i] = hi[i];
                        v[16 + i] = lo[i];
                    }
                }
                tmem_st_32x32b_x32(tl + 32 * q, v);
            }
            tmem_st_wait();
        }
        fence_async_smem();
        tc_fence_before();
        __syncthreads();
        if (r == 0) {
            tc_fence_after();
            if (FULL) {
                const uint64_t xd = desc_mn(sm + kOffX);
#pragma unroll
                for (int k = 0; k < Q / 16; ++k)
#pragma unroll
                    for (int part = 0; part < 2; ++part)
                        mma_ts(tm + kColY, tm + 32 * (k >> 1) + 16 * part + 8 * (k & 1), xd + (k * 256 >> 4),
                               idesc(PW, 0, 1), 1);
                umma_commit(&fx.bar[1]);
            }
            const uint64_t bd = desc_mn(sm + kOffB), wd = desc_mn(sm + kOffXw);
#pragma unroll
            for (int part = 0; part < 3; ++part)
#pragma unroll
                for (int k = 0; k < Q / 16; ++k)
                    mma_ss(tm + kColS, bd + (k * 256 >> 4), wd + ((part * 16384 + k * 256) >> 4), idesc(PW, 1, 1),
                           part + k > 0);
            umma_commit(&fx.bar[2]);
        }
        if (FULL) {
            if (!mbar_wait_bounded(&fx.bar[1], parity, nullptr)) fx.bad = 1;
            __syncwarp();
            tc_fence_after();
            const bool live = t0 + r < p.len;
            bf16 *yp = static_cast<bf16 *>(a.y) + (p.row0 + (live ? t0 + r : t0) * p.step) * a.ldy +
                       (int64_t)h * a.dv + c0;
            const bool nf = fx.nf != 0;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                uint32_t v[32];
                tmem_ld_32x32b<32>(tl + kColY + 32 * q, v);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    Raw<bf16, 8> rx;
                    rx.a = *reinterpret_cast<const uint4 *>(sm + kOffX + (4 * q + j) * kChunkB + r * 16);
                    float f[8];
                    rx.get(f);
#pragma unroll
                    for (int k = 0; k < 8; ++k) f[k] = fmaf(Dh, f[k], __uint_as_float(v[8 * j + k]));
                    if (nf)
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            if (fx.first[32 * q + 8 * j + k] <= r) f[k] = __int_as_float(0x7fffffff);
                    rx.set(f);
                    if (live) {
                        bf16 *dst = yp + 32 * q + 8 * j;
                        if (vec) {
                            rx.store(dst);
                        } else {
                            const uint32_t w[4] = {rx.a.x, rx.a.y, rx.a.z, rx.a.w};
                            uint16_t *e = reinterpret_cast<uint16_t *>(dst);
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                e[2 * k] = (uint16_t)w[k];
                                e[2 * k + 1] = (uint16_t)(w[k] >> 16);
                            }
                        }
                    }
                }
            }
        }
        if (!mbar_wait_bounded(&fx.bar[2], parity, nullptr)) fx.bad = 1;
        __syncwarp();
        tc_fence_after();
        const float keep = exp2f((float)total);
        gsum += total;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            uint32_t v[32];
            tmem_ld_32x32b<32>(tl + kColS + 32 * q, v);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) S[32 * q + i] = fmaf(keep, S[32 * q + i], __uint_as_float(v[i]));
        }
    }
    tc_fence_before();
    __syncthreads();
    // A wait that ran out leaves no state that looks like one.
    if (fx.bad)
#pragma unroll
        for (int i = 0; i < PW; ++i) S[i] = __int_as_float(0x7fffffff);
    if (r < DK && (!FULL || p.j == p.n - 1)) {
        float *so = FULL ? a.S_out + p.b * sall + soff : a.ws + z * sall + soff;
#pragma unroll
        for (int i = 0; i < PW / 4; ++i)
            reinterpret_cast<float4 *>(so)[i] = make_float4(S[4 * i], S[4 * i + 1], S[4 * i + 2], S[4 * i + 3]);
    }
    if (!FULL && r == 0 && c0 == 0) ssm_decays(a, seg)[(int64_t)z * a.H + h] = exp2f((float)gsum);
    if (warp == 0) {
        tmem_relinquish();
        tmem_dealloc(fx.tmem, kTmemCols);
    }
}

template <int DK>
cudaError_t launch(const SsmArgs &a, int seg, int vec, int split, cudaStream_t s) {
    const int units = a.H * (a.dv / PW);
    const int64_t grid = piece_count(a.r, seg) * units;
    cudaError_t e = cudaFuncSetAttribute(ssm_umma_kernel<true, DK>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    if (split) {
        e = cudaFuncSetAttribute(ssm_umma_kernel<false, DK>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        ssm_umma_kernel<false, DK><<<(unsigned)grid, kNT, kSmem, s>>>(a, seg, units, vec, split);
        e = launch_ssm_join(a, seg, s);
        if (e != cudaSuccess) return e;
    }
    ssm_umma_kernel<true, DK><<<(unsigned)grid, kNT, kSmem, s>>>(a, seg, units, vec, split);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_ssm_umma(const SsmArgs &a, int seg, bool split, cudaStream_t s) {
    // 16-byte copies need every row to start on a 16-byte boundary.
    const uintptr_t base = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.Bm) |
                           reinterpret_cast<uintptr_t>(a.Cm) | reinterpret_cast<uintptr_t>(a.y);
    const int vec = base % 16 == 0 && a.ldx % 8 == 0 && a.ldb % 8 == 0 && a.ldc % 8 == 0 && a.ldy % 8 == 0;
    return a.dk == 64 ? launch<64>(a, seg, vec, split, s) : launch<128>(a, seg, vec, split, s);
}

}  // namespace lq
