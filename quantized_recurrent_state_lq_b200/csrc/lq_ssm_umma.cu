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
// A group of eight warps takes 64 value columns of one head over one piece of
// a sequence: two threads per token, key row and tensor-memory lane, 32 columns
// each.  Its phases alternate between the tensor core and the threads, so a CTA
// runs two groups (256 tensor-memory columns, 112 KB of shared memory each)
// half a chunk apart: a kernel that uses tensor memory gets one CTA per SM here.
// Long sequences of a small batch are cut into pieces: a first pass forms each
// piece's own state, ssm_join_kernel chains them, the second pass starts every
// piece from its state (about a third more work for pieces x as much
// parallelism).
//
// Shared memory holds every operand as rows of 64 columns (128 bytes, the
// 16-byte chunks XOR-swizzled by the row's low 3 bits) in blocks of 16 KB:
// read as rows x K it is K-major, read as K x columns MN-major, so B serves
// C B^T and B^T X' from one copy, and a thread's accesses to its own row meet
// no bank conflict.  B, C and X arrive by TMA tensor copies, issued as soon as
// the chunk before has let go of their places:
//   [0, 32K) C, [32K, 64K) S parts   -- until C B^T and C S are done; then
//   [0, 48K) X' parts, [48K, ..) decay factors
//   [64K, 96K) B, [96K, 112K) X
// Rows that TMA cannot take (not 16-byte aligned) are copied by the threads.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "lq_act.cuh"
#include "lq_ssm.h"
#include "lq_tc.cuh"

namespace lq {
namespace {

constexpr int kSms = 148;
constexpr int Q = 128;                 // tokens per chunk
constexpr int PW = 64;                 // value columns of a group
constexpr int HW = PW / 2;             // and of a thread
constexpr int kNT = 256;               // threads of a group
constexpr int kBlk = Q * 128;          // bytes of 128 rows of 64 columns
constexpr int kOffC = 0, kOffS = 2 * kBlk, kOffXw = 0, kOffF = 3 * kBlk, kOffB = 4 * kBlk, kOffX = 6 * kBlk;
constexpr int kSmem = 7 * kBlk;
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

// 128-byte swizzle: 8-row groups 1024 B apart; MN-major operands of more than
// 64 columns continue a block further.
__device__ __forceinline__ uint64_t desc_sw(const void *p, uint32_t lbo) {
    return umma_smem_desc(p, lbo, 1024) | (2ull << 61);
}
__device__ __forceinline__ uint64_t desc_k(const void *p) { return desc_sw(p, 16); }
__device__ __forceinline__ uint64_t desc_mn(const void *p) { return desc_sw(p, kBlk); }
// 16 further along K: 32 bytes of a K-major block's rows (4 steps a block), 16
// rows of an MN-major one.
__device__ __forceinline__ constexpr uint64_t step_k(int k) { return (uint64_t)((k >> 2) * kBlk + (k & 3) * 32) >> 4; }
__device__ __forceinline__ constexpr uint64_t step_mn(int k) { return (uint64_t)(k * 16 * 128) >> 4; }

// 16-byte chunk j of a row.
__device__ __forceinline__ uint4 *chunk(unsigned char *tile, int row, int j) {
    return reinterpret_cast<uint4 *>(tile + (j >> 3) * kBlk + row * 128 + (((j & 7) ^ (row & 7)) << 4));
}

__device__ __forceinline__ void tma_rows(void *dst, const CUtensorMap *map, int col, int b, int t, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(col), "r"(b), "r"(t), "r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }

// bf16 parts of a pair: returns the pair rounded to bf16 and leaves the rests.
__device__ __forceinline__ uint32_t last_part(float2 v) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t *>(&p);
}
__device__ __forceinline__ uint32_t take_part(float2 &v) {
    const uint32_t w = last_part(v);
    v = ffma2(bf16x2_to_f2(w), f2(-1.0f, -1.0f), v);
    return w;
}

// Rows t0 .. t0 + Q - 1 of a sequence (zeros from its end on), NCH chunks of 8
// elements each, element by element: thread i of the group.
__device__ __forceinline__ void copy_tile(unsigned char *dst, int nch, const bf16 *src, int64_t ld, const Piece &p,
                                          int t0, int i) {
    for (; i < Q * nch; i += kNT) {
        const int t = i / nch, j = i % nch;
        uint32_t w[4] = {0u, 0u, 0u, 0u};
        if (t0 + t < p.len) {
            const uint16_t *e = reinterpret_cast<const uint16_t *>(src + (p.row0 + (t0 + t) * p.step) * ld + 8 * j);
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = (uint32_t)e[2 * k] | ((uint32_t)e[2 * k + 1] << 16);
        }
        *chunk(dst, t, j) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Token rows [T][B][width] of x, B and C as 3-D maps, boxes of 64 columns x 128
// tokens of one sequence (packed: one sequence of all rows).
struct alignas(64) SsmMaps {
    CUtensorMap x, b, c;
};

// One group's work: 64 value columns of one head over one piece.
struct Item {
    Piece p;
    int h, c0, g;
    int t_first, t_end;
    int tm_t, tm_b;      // where TMA finds token t: row tm_t + t of sequence tm_b
    bool valid;
};

// A group's share of the items: it takes every item that starts in its equal
// part of all chunks, the items in the order of sequences, pieces and units.
struct Walk {
    int64_t pos, end;    // start of the next item and end of the share, in chunks
    int b, j, u;         // the next item
};

struct Fixed {
    uint64_t bar[5];     // G and C S done, Y done, B^T X' done, B and C arrived, X arrived
    long long wsum[2][4];   // each warp's log2 decay (even, odd chunks)
    int bad;             // a wait ran out
    int nf[2];           // a non-finite x in this chunk (even, odd chunks)
    Item item[2];        // the item at work and the next
    Walk walk;
    int first[2][PW];    // per value column, the first token whose x is not finite
};

// X' of token r, this thread's columns, in three parts: w x.
__device__ __forceinline__ void split_x(unsigned char *sm, unsigned char *x, int r, int half, float w) {
#pragma unroll
    for (int i = 0; i < HW / 8; ++i) {
        const int j = half * (HW / 8) + i;
        Raw<bf16, 8> rx;
        rx.a = *chunk(x, r, j);
        float f[8];
        rx.get(f);
        uint32_t part[3][4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float2 v = mul2(f2(w, w), f2(f[2 * k], f[2 * k + 1]));
            part[0][k] = take_part(v);
            part[1][k] = take_part(v);
            part[2][k] = last_part(v);
        }
#pragma unroll
        for (int q = 0; q < 3; ++q)
            *chunk(sm + kOffXw + q * kBlk, r, j) = make_uint4(part[q][0], part[q][1], part[q][2], part[q][3]);
    }
}

// Outputs and final states.  Each group walks its share of the items; its second
// warp finds the next one and sends for its first tiles before the last one ends.
template <int DK>
__global__ void __launch_bounds__(2 * kNT, 1)
    ssm_umma_kernel(SsmArgs a, const __grid_constant__ SsmMaps maps, int seg, int tma, int split) {
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ uint32_t tmem;
    const int wid = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int grp = threadIdx.x / kNT, ti = threadIdx.x % kNT;
    unsigned char *sm = smem + grp * kSmem;
    Fixed &fx = reinterpret_cast<Fixed *>(smem + 2 * kSmem)[grp];
    const int warp = wid & 3, half = (wid >> 2) & 1, r = warp * 32 + lane;   // 32 rows, 32 columns of this warp
    // One thread of three warps issues for the group, so that none is held up for
    // long: C B^T, C S and B^T X'; M X and the copies of X; the copies of B and C.
    const bool lead = ti == 0, lead_x = ti == 128, finder = warp == 1 && half == 0;
    const int units = a.H * (a.dv / PW);
    const int64_t sall = (int64_t)a.H * DK * a.dv;
    auto sync = [&]() { asm volatile("bar.sync %0, %1;" ::"r"(1 + grp), "n"(kNT) : "memory"); };

    float S[HW];   // the state's key row r, this thread's columns
    // The item's state from its start, and to its end.
    auto state_at = [&](const Item &it) { return ((int64_t)it.h * DK + r) * a.dv + it.c0 + half * HW; };
    auto load_state = [&](const Item &it) {
        const float *S0 = nullptr;
        if (r < DK) {
            if (split && it.p.n > 1) S0 = a.ws + it.p.id * sall + state_at(it);
            else if (a.S0) S0 = a.S0 + it.p.b * sall + state_at(it);
        }
#pragma unroll
        for (int i = 0; i < HW / 4; ++i) {
            const float4 v = S0 ? reinterpret_cast<const float4 *>(S0)[i] : make_float4(0.f, 0.f, 0.f, 0.f);
            S[4 * i] = v.x; S[4 * i + 1] = v.y; S[4 * i + 2] = v.z; S[4 * i + 3] = v.w;
        }
    };
    auto store_state = [&](const Item &it) {
        if (r < DK && it.p.j == it.p.n - 1) {
            float *so = a.S_out + it.p.b * sall + state_at(it);
#pragma unroll
            for (int i = 0; i < HW / 4; ++i)
                reinterpret_cast<float4 *>(so)[i] = make_float4(S[4 * i], S[4 * i + 1], S[4 * i + 2], S[4 * i + 3]);
        }
    };
    const int64_t worker = 2 * (int64_t)blockIdx.x + grp, workers = 2 * (int64_t)gridDim.x;
    auto seq_len = [&](int b) {
        return a.r.cu ? max(cu_at(a.r, b + 1) - cu_at(a.r, b), 0) : a.r.rows / a.r.B;
    };
    // (Both by the group's second warp.)  The first item that starts in this
    // group's part.
    auto start_walk = [&]() {
        Walk w{};
        {
            int64_t all = 0;
            for (int b = lane; b < a.r.B; b += 32) all += (seq_len(b) + Q - 1) / Q;
            all = warp_scan(all);
            all = __shfl_sync(0xffffffffu, all, 31) * units;
            w.pos = all * worker / workers;
            w.end = all * (worker + 1) / workers;
            int64_t before = 0;   // chunks of the sequences before b
            w.b = a.r.B;
            for (int b0 = 0; b0 < a.r.B; b0 += 32) {
                const int64_t n = b0 + lane < a.r.B ? (int64_t)((seq_len(b0 + lane) + Q - 1) / Q) * units : 0;
                const int64_t upto = before + warp_scan(n);
                const unsigned in = __ballot_sync(0xffffffffu, upto > w.pos);
                if (in) {   // the sequence that holds the first position
                    const int l = __ffs(in) - 1;
                    w.b = b0 + l;
                    before = __shfl_sync(0xffffffffu, upto - n, l);
                    break;
                }
                before = __shfl_sync(0xffffffffu, upto, 31);
            }
            if (w.b < a.r.B) {
                const int len = seq_len(w.b), n = (len + seg - 1) / seg, whole = seg / Q;
                const int64_t o = w.pos - before, per = (int64_t)whole * units;
                w.j = (int)min(o / per, (int64_t)(n - 1));
                const int c = w.j < n - 1 ? whole : ((len - w.j * seg) + Q - 1) / Q;
                w.u = (int)((o - w.j * per + c - 1) / c);
                w.pos = before + w.j * per + (int64_t)w.u * c;
            }
        }
        if (lane == 0) fx.walk = w;
        __syncwarp();
    };
    auto next_item = [&](Item &out) {
        Walk w = fx.walk;
        Item it;
        it.valid = false;
        int u = 0;
        {
            while (w.pos < w.end && w.b < a.r.B && !it.valid) {
                const int c0 = a.r.cu ? cu_at(a.r, w.b) : 0, len = seq_len(w.b), n = (len + seg - 1) / seg;
                if (w.u >= units) {
                    w.u = 0;
                    ++w.j;
                }
                if (w.j >= n) {
                    w.j = w.u = 0;
                    ++w.b;
                    continue;
                }
                it.valid = true;
                it.p.b = w.b;
                it.p.j = w.j;
                it.p.len = len;
                it.p.n = n;
                it.p.row0 = a.r.cu ? c0 : w.b;
                it.p.step = a.r.cu ? 1 : a.r.B;
                it.p.id = (a.r.cu ? c0 / seg + w.b : (int64_t)w.b * n) + w.j;
                u = w.u++;
                w.pos += (min(len - w.j * seg, seg) + Q - 1) / Q;
            }
        }
        if (it.valid) {
            const int per = a.dv / PW;
            it.h = u / per;
            it.c0 = (u % per) * PW;
            it.g = (int)((int64_t)it.h * a.G / a.H);
            it.t_first = it.p.j * seg;
            it.t_end = min(it.p.len, it.t_first + seg);
            it.tm_t = a.r.cu ? (int)it.p.row0 : 0;
            it.tm_b = a.r.cu ? 0 : it.p.b;
        }
        __syncwarp();
        if (lane == 0) {
            out = it;
            fx.walk = w;
        }
        __syncwarp();
    };
    // B and C of a chunk: their places are free once B^T X' of the chunk before is
    // done.  X: once the outputs of the chunk before, in its place, have been stored.
    auto load_bc = [&](const Item &it, int t0) {
        mbar_arrive_expect_tx(&fx.bar[3], 2 * (DK / 64) * kBlk);
#pragma unroll
        for (int j = 0; j < DK / 64; ++j) {
            tma_rows(sm + kOffB + j * kBlk, &maps.b, it.g * DK + 64 * j, it.tm_b, it.tm_t + t0, &fx.bar[3]);
            tma_rows(sm + kOffC + j * kBlk, &maps.c, it.g * DK + 64 * j, it.tm_b, it.tm_t + t0, &fx.bar[3]);
        }
    };
    auto load_x = [&](const Item &it, int t0) {
        mbar_arrive_expect_tx(&fx.bar[4], kBlk);
        tma_rows(sm + kOffX, &maps.x, it.h * a.dv + it.c0, it.tm_b, it.tm_t + t0, &fx.bar[4]);
    };

    if (finder) {
        start_walk();
        next_item(fx.item[0]);
        if (lane == 0) {
            for (int i = 0; i < 5; ++i) mbar_init(&fx.bar[i], 1);
            fx.bad = 0;
            fence_mbar_init();
            if (tma && fx.item[0].valid) load_bc(fx.item[0], fx.item[0].t_first);
        }
    }
    if (a.r.cu) {   // a sequence without tokens hands its state through
        for (int b = blockIdx.x; b < a.r.B; b += gridDim.x)
            if (cu_at(a.r, b + 1) <= cu_at(a.r, b))
                for (int64_t i = threadIdx.x; i < sall / 4; i += 2 * kNT)
                    reinterpret_cast<float4 *>(a.S_out + b * sall)[i] =
                        a.S0 ? reinterpret_cast<const float4 *>(a.S0 + b * sall)[i] : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (wid == 1) tmem_alloc(&tmem, 2 * kTmemCols);
    if (ti < 2 * PW) (&fx.first[0][0])[ti] = Q;
    if (ti < 2) fx.nf[ti] = 0;
    if (DK < 128) {   // B^T has 128 rows: the missing key rows are zero
        for (int i = ti; i < kBlk / 16; i += kNT)
            reinterpret_cast<uint4 *>(sm + kOffB + kBlk)[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = tmem + grp * kTmemCols, tl = tm + ((uint32_t)warp << 21);   // this warp's lanes: 32 warp

    // This token's step and its log2 decay within its warp's 32, of the chunk
    // after the one at work; and of the chunk at work: the step, 2^ of the decay
    // within the warp and within the chunk, the weight in the next state, the
    // factors for the rows of later warps.
    float d_next, d, gwf, et, wr, keep, fac[3];
    long long gw_next;
    int parity = 0;
    // The second group starts half a chunk behind the first.
    if (grp == 0 && !fx.item[0].valid) asm volatile("bar.arrive 5, %0;" ::"n"(2 * kNT) : "memory");
    if (grp == 1) asm volatile("bar.sync 5, %0;" ::"n"(2 * kNT) : "memory");
    bool first = grp == 0;

    for (int sel = 0; fx.item[sel].valid; sel ^= 1) {
        const Item &it = fx.item[sel];
        const Piece &p = it.p;
        const int h = it.h, t_end = it.t_end;
        const bf16 *dp = static_cast<const bf16 *>(a.dt) + h;
        const float A2 = a.A[h] * 1.4426950408889634f;   // log2 decay per unit step
        const float Dh = a.D ? a.D[h] : 0.0f, bias = a.dt_bias ? a.dt_bias[h] : 0.0f;
        // (as it is stored: the conversion would wait for it)
        auto raw_step = [&](int t) -> unsigned short {
            return t < p.len ? reinterpret_cast<const unsigned short *>(dp)[(p.row0 + (int64_t)t * p.step) * a.lddt]
                             : (unsigned short)0;
        };
        auto scan_steps = [&](unsigned short raw, int t, int odd) {
            d_next = 0.0f;
            gw_next = 0;
            if (t < p.len) {
                d_next = bf16_to_f(raw) + bias;
                if (a.softplus) d_next = softplus_f(d_next);
                gw_next = decay_of(d_next, A2);
            }
            gw_next = warp_scan(gw_next);
            if (half == 0 && lane == 31) fx.wsum[odd][warp] = gw_next;
        };
        // The scanned chunk's factors, once every warp's sum is known.
        auto finish_steps = [&](int odd) {
            d = d_next;
            long long base = 0, total = 0;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const long long s = fx.wsum[odd][w];
                if (w < warp) base += s;
                total += s;
            }
            const long long gt = base + gw_next;
            gwf = decay_f(gw_next);
            et = ex2_f(decay_f(gt));
            wr = d * exp2f(decay_f(total - gt));
            keep = exp2f(decay_f(total));
            if (half == 1) {
                long long end = 0;
#pragma unroll
                for (int w = 0; w < 3; ++w) {
                    end += fx.wsum[odd][w];
                    fac[w] = d * exp2f(decay_f(end - gt));
                }
            }
        };
        auto split_state = [&]() {   // the state's two parts
            if (r < DK) {
#pragma unroll
                for (int j = 0; j < HW / 8; ++j) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float2 v = f2(S[8 * j + 2 * k], S[8 * j + 2 * k + 1]);
                        hi[k] = take_part(v);
                        lo[k] = last_part(v);
                    }
                    *chunk(sm + kOffS, r, half * (HW / 8) + j) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *chunk(sm + kOffS + kBlk, r, half * (HW / 8) + j) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
            }
        };
        const unsigned short raw0 = raw_step(it.t_first + r), raw1 = raw_step(it.t_first + Q + r);
        load_state(it);
        scan_steps(raw0, it.t_first + r, 0);
        split_state();
        sync();
        finish_steps(0);
        scan_steps(raw1, it.t_first + Q + r, 1);
        for (int t0 = it.t_first; t0 < t_end; t0 += Q, parity ^= 1) {
            const bool tail = t0 + Q > p.len, last = t0 + Q >= t_end;
            const int odd = ((t0 - it.t_first) / Q) & 1;
            fence_async_smem();
            tc_fence_before();
            sync();   // the chunk before is done with shared and tensor memory
            if (lead_x && tma) load_x(it, t0);
            if (fx.bad) {
                if (lead_x && tma) {   // the copies under way
                    mbar_wait_bounded(&fx.bar[3], parity, nullptr);
                    mbar_wait_bounded(&fx.bar[4], parity, nullptr);
                }
                break;
            }
            if (tma) {
                if (tail || lead) {
                    if (!mbar_wait_bounded(&fx.bar[3], parity, nullptr)) fx.bad = 1;
                }
                __syncwarp();
                if (tail) {
                    // a packed sequence's last tile continues into the next sequence
                    if (!mbar_wait_bounded(&fx.bar[4], parity, nullptr)) fx.bad = 1;
                    if (t0 + r >= p.len) {
                        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                        for (int j = 0; j < DK / 16; ++j) {
                            *chunk(sm + kOffB, r, half * (DK / 16) + j) = zero;
                            *chunk(sm + kOffC, r, half * (DK / 16) + j) = zero;
                        }
#pragma unroll
                        for (int j = 0; j < PW / 16; ++j) *chunk(sm + kOffX, r, half * (PW / 16) + j) = zero;
                    }
                    fence_async_smem();
                    sync();
                }
            } else {
                copy_tile(sm + kOffB, DK / 8, static_cast<const bf16 *>(a.Bm) + it.g * DK, a.ldb, p, t0, ti);
                copy_tile(sm + kOffX, PW / 8, static_cast<const bf16 *>(a.x) + (int64_t)h * a.dv + it.c0, a.ldx, p, t0,
                          ti);
                copy_tile(sm + kOffC, DK / 8, static_cast<const bf16 *>(a.Cm) + it.g * DK, a.ldc, p, t0, ti);
                fence_async_smem();
                sync();
            }
            if (lead) {
                tc_fence_after();
                const uint64_t cd = desc_k(sm + kOffC), bd = desc_k(sm + kOffB), sd = desc_mn(sm + kOffS);
#pragma unroll
                for (int k = 0; k < DK / 16; ++k) mma_ss(tm, cd + step_k(k), bd + step_k(k), idesc(Q, 0, 0), k > 0);
                // C S, its parts side by side: [kColY, kColS) and [kColS, 256)
#pragma unroll
                for (int k = 0; k < DK / 16; ++k)
                    mma_ss(tm + kColY, cd + step_k(k), sd + step_mn(k), idesc(2 * PW, 0, 1), k > 0);
                umma_commit(&fx.bar[0]);
            }
            __syncwarp();
            const unsigned short raw = raw_step(t0 + 2 * Q + r);
            if (ti < PW) fx.first[parity ^ 1][ti] = Q;
            if (ti == 0) fx.nf[parity ^ 1] = 0;
            if (tma && !mbar_wait_bounded(&fx.bar[4], parity, nullptr)) fx.bad = 1;
            if (!mbar_wait_bounded(&fx.bar[0], parity, nullptr)) fx.bad = 1;
            __syncwarp();
            tc_fence_after();
            float *fl = reinterpret_cast<float *>(sm + kOffF);   // [Q] sums within the warp, [Q] d, [3][Q] factors
            {
                if (half == 0) {
                    fl[r] = gwf;
                    fl[Q + r] = d;
                } else {
#pragma unroll
                    for (int w = 0; w < 3; ++w)
                        if (w >= warp) fl[(2 + w) * Q + r] = fac[w];
                }
            }
            // X' of this token in three parts; a non-finite x leaves X (times 0 it
            // would reach earlier tokens) and is marked instead.
#pragma unroll
            for (int i = 0; i < HW / 8; ++i) {
                const int j = half * (HW / 8) + i;
                Raw<bf16, 8> rx;
                rx.a = *chunk(sm + kOffX, r, j);
                float f[8];
                rx.get(f);
                uint32_t w[3][4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float2 v = mul2(f2(wr, wr), f2(f[2 * k], f[2 * k + 1]));
                    w[0][k] = take_part(v);
                    w[1][k] = take_part(v);
                    w[2][k] = last_part(v);
                }
#pragma unroll
                for (int q = 0; q < 3; ++q)
                    *chunk(sm + kOffXw + q * kBlk, r, j) = make_uint4(w[q][0], w[q][1], w[q][2], w[q][3]);
                {
                    const uint32_t wd[4] = {rx.a.x, rx.a.y, rx.a.z, rx.a.w};
                    __nv_bfloat162 n = __float2bfloat162_rn(0.0f);   // 0 x finite = 0, else NaN
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        n = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&wd[k]), __float2bfloat162_rn(0.0f), n);
                    if (*reinterpret_cast<const uint32_t *>(&n) & 0x7fff7fffu) {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            if (!isfinite(f[k])) {
                                f[k] = 0.0f;
                                atomicMin(&fx.first[parity][8 * j + k], r);
                            }
                        rx.set(f);
                        *chunk(sm + kOffX, r, j) = rx.a;
                        fx.nf[parity] = 1;
                    }
                }
            }
            __syncwarp();
            {
                // 2^(g_t) on the sum of C S's parts
#pragma unroll 1
                for (int q = 0; q < HW; q += 16) {
                    uint32_t v[16], v2[16];
                    tmem_ld_32x32b<16>(tl + kColY + half * HW + q, v);
                    tmem_ld_32x32b<16>(tl + kColS + half * HW + q, v2);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        v[i] = __float_as_uint(et * (__uint_as_float(v[i]) + __uint_as_float(v2[i])));
                    tmem_st_32x32b_x16(tl + kColY + half * HW + q, v);
                }
                sync();   // the factors
                // M over G, 16 tokens at a time: 8 columns of first parts, 8 of
                // second.  Tokens of earlier warps factor through the boundary
                // before this warp's, those after this one are zero.
                const float rf = ex2_f(gwf);
                for (int q = half; q < 8; q += 2) {
                    uint32_t v[16];
                    if (q > 2 * warp + 1) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) v[i] = 0u;
                    } else {
                        tmem_ld_32x32b<16>(tl + 16 * q, v);
                        tmem_ld_wait();
                        uint32_t hi[8], lo[8];
                        if (q < 2 * warp) {
                            const float4 *cf = reinterpret_cast<const float4 *>(fl + (1 + warp) * Q + 16 * q);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float4 c = cf[i];
                                const float2 cc[2] = {f2(c.x, c.y), f2(c.z, c.w)};
#pragma unroll
                                for (int k = 0; k < 2; ++k) {
                                    const float2 gg = f2(__uint_as_float(v[4 * i + 2 * k]),
                                                         __uint_as_float(v[4 * i + 2 * k + 1]));
                                    float2 m = mul2(cc[k], mul2(f2(rf, rf), gg));
                                    hi[2 * i + k] = take_part(m);
                                    lo[2 * i + k] = last_part(m);
                                }
                            }
                        } else {
                            const float4 *gs = reinterpret_cast<const float4 *>(fl + 16 * q);
                            const float4 *ds = reinterpret_cast<const float4 *>(fl + Q + 16 * q);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float4 gv = gs[i], dv = ds[i];
                                const float ge[4] = {gv.x, gv.y, gv.z, gv.w}, de[4] = {dv.x, dv.y, dv.z, dv.w};
                                float m[4];
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    const float e = ex2_f(gwf - ge[k]) * de[k] * __uint_as_float(v[4 * i + k]);
                                    m[k] = 16 * (q & 1) + 4 * i + k <= lane ? e : 0.0f;
                                }
#pragma unroll
                                for (int k = 0; k < 2; ++k) {
                                    float2 mm = f2(m[2 * k], m[2 * k + 1]);
                                    hi[2 * i + k] = take_part(mm);
                                    lo[2 * i + k] = last_part(mm);
                                }
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            v[i] = hi[i];
                            v[8 + i] = lo[i];
                        }
                    }
                    tmem_st_32x32b_x16(tl + 16 * q, v);
                }
                tmem_st_wait();
            }
            // The next chunk's factors and the decays of the one after: by the
            // issuing warp (which has little of M) before it is held up, by the
            // others while the MMAs run.
            const float keep_now = keep;
            if (!last && warp == 0) {
                finish_steps(odd ^ 1);
                scan_steps(raw, t0 + 2 * Q + r, odd);
            }
            fence_async_smem();
            tc_fence_before();
            sync();
            if (lead) {
                tc_fence_after();
                const uint64_t bd = desc_mn(sm + kOffB), wd = desc_mn(sm + kOffXw);
#pragma unroll
                for (int part = 0; part < 3; ++part)
#pragma unroll
                    for (int k = 0; k < Q / 16; ++k)
                        mma_ss(tm + kColS, bd + step_mn(k), wd + (part * kBlk >> 4) + step_mn(k), idesc(PW, 1, 1),
                               part + k > 0);
                umma_commit(&fx.bar[2]);
            }
            if (lead_x) {
                tc_fence_after();
                const uint64_t xd = desc_mn(sm + kOffX);
                {
#pragma unroll
                    for (int k = 0; k < Q / 16; ++k)
#pragma unroll
                        for (int part = 0; part < 2; ++part)
                            mma_ts(tm + kColY, tm + 16 * k + 8 * part, xd + step_mn(k),
                                   idesc(PW, 0, 1), 1);
                    umma_commit(&fx.bar[1]);
                }
            }
            __syncwarp();
            if (first) asm volatile("bar.arrive 5, %0;" ::"n"(2 * kNT) : "memory");
            first = false;
            if (!last && warp != 0) {
                finish_steps(odd ^ 1);
                scan_steps(raw, t0 + 2 * Q + r, odd);
            }
            if (last && finder) next_item(fx.item[sel ^ 1]);
            if (!mbar_wait_bounded(&fx.bar[2], parity, nullptr)) fx.bad = 1;
            if (finder && lane == 0 && tma) {
                if (!last) load_bc(it, t0 + Q);
                else if (fx.item[sel ^ 1].valid) load_bc(fx.item[sel ^ 1], fx.item[sel ^ 1].t_first);
            }
            __syncwarp();
            tc_fence_after();
#pragma unroll
            for (int q = 0; q < HW; q += 16) {
                uint32_t v[16];
                tmem_ld_32x32b<16>(tl + kColS + half * HW + q, v);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                    const float2 s = ffma2(f2(keep_now, keep_now), f2(S[q + i], S[q + i + 1]),
                                           f2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])));
                    S[q + i] = s.x;
                    S[q + i + 1] = s.y;
                }
            }
            if (!last) split_state();
            {
                // outputs into X's place
                if (!mbar_wait_bounded(&fx.bar[1], parity, nullptr)) fx.bad = 1;
                __syncwarp();
                tc_fence_after();
                const bool nf = fx.nf[parity] != 0;
#pragma unroll 1
                for (int q = 0; q < HW; q += 16) {
                    uint32_t v[16];
                    tmem_ld_32x32b<16>(tl + kColY + half * HW + q, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        uint4 *at8 = chunk(sm + kOffX, r, half * (HW / 8) + q / 8 + j);
                        Raw<bf16, 8> rx;
                        rx.a = *at8;
                        float f[8];
                        rx.get(f);
#pragma unroll
                        for (int k = 0; k < 8; ++k) f[k] = fmaf(Dh, f[k], __uint_as_float(v[8 * j + k]));
                        if (nf)
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                if (fx.first[parity][half * HW + q + 8 * j + k] <= r) f[k] = __int_as_float(0x7fffffff);
                        rx.set(f);
                        *at8 = rx.a;
                    }
                }
                // whole rows of 128 bytes at a time
                sync();
                const int col = h * a.dv + it.c0;
#pragma unroll
                for (int i = 0; i < Q * (PW / 8) / kNT; ++i) {
                    const int t = (i * kNT + ti) / (PW / 8), j = ti % (PW / 8);
                    if (t0 + t < p.len) {
                        const uint4 w4 = *chunk(sm + kOffX, t, j);
                        bf16 *dst = static_cast<bf16 *>(a.y) + (p.row0 + (int64_t)(t0 + t) * p.step) * a.ldy + col + 8 * j;
                        if (tma) {
                            *reinterpret_cast<uint4 *>(dst) = w4;
                        } else {
                            const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
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
        sync();   // the next item is known
        // A wait that ran out leaves no state that looks like one.
        if (fx.bad)
#pragma unroll
            for (int i = 0; i < HW; ++i) S[i] = __int_as_float(0x7fffffff);
        store_state(it);
        if (fx.bad) break;
    }
    tc_fence_before();
    __syncthreads();
    if (wid == 1) {
        tmem_relinquish();
        tmem_dealloc(tmem, 2 * kTmemCols);
    }
}

// The pieces' own states, from zero, and their decays, for every piece that is
// followed by another (all of them seg tokens long): only B^T X' and the state
// update.  Without C and S the tiles of X have two places, a chunk ahead, and
// the products of a chunk two accumulators, so that the update runs beside the
// next chunk's MMAs.
//   [0, 48K) X' parts, [48K, 64K) X of even chunks, [64K, 96K) B, [96K, 112K) X of odd chunks
template <int DK>
__global__ void __launch_bounds__(2 * kNT, 1)
    ssm_state_kernel(SsmArgs a, const __grid_constant__ SsmMaps maps, int seg, int64_t items, int tma) {
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ uint32_t tmem;
    const int wid = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int grp = threadIdx.x / kNT, ti = threadIdx.x % kNT;
    unsigned char *sm = smem + grp * kSmem;
    Fixed &fx = reinterpret_cast<Fixed *>(smem + 2 * kSmem)[grp];
    const int warp = wid & 3, half = (wid >> 2) & 1, r = warp * 32 + lane;
    const bool lead = ti == 0;
    const int units = a.H * (a.dv / PW), per = a.dv / PW, chunks = seg / Q;
    const int64_t sall = (int64_t)a.H * DK * a.dv;
    auto sync = [&]() { asm volatile("bar.sync %0, %1;" ::"r"(1 + grp), "n"(kNT) : "memory"); };
    auto x_tile = [&](int n) { return sm + (n & 1 ? kOffX : kOffF); };
    uint64_t *b_bar = &fx.bar[2], *mma_bar = &fx.bar[3];   // and bar[0], bar[1]: X of even and odd chunks

    if (lead) {
        for (int i = 0; i < 4; ++i) mbar_init(&fx.bar[i], 1);
        fx.bad = 0;
        fence_mbar_init();
    }
    if (wid == 1) tmem_alloc(&tmem, 256);
    if (DK < 128) {   // B^T has 128 rows: the missing key rows are zero
        for (int i = ti; i < kBlk / 16; i += kNT)
            reinterpret_cast<uint4 *>(sm + kOffB + kBlk)[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = tmem + grp * 128, tl = tm + ((uint32_t)warp << 21);   // this warp's lanes: 32 warp

    int n = 0;   // chunks so far: the barriers' phases
    // The second group starts half a chunk behind the first.
    if (grp == 1) asm volatile("bar.sync 5, %0;" ::"n"(2 * kNT) : "memory");
    for (int64_t at = 2 * (int64_t)blockIdx.x + grp; at < items; at += 2 * (int64_t)gridDim.x) {
        const int z = (int)(at / units), u = (int)(at - (int64_t)z * units), h = u / per, c0 = (u % per) * PW;
        Piece p;
        if (!find_cut(a.r, seg, z, p)) continue;
        const int g = (int)((int64_t)h * a.G / a.H), t_first = p.j * seg;
        const int tm_t = a.r.cu ? (int)p.row0 : 0, tm_b = a.r.cu ? 0 : p.b;
        const unsigned short *dp = static_cast<const unsigned short *>(a.dt) + h;
        const float A2 = a.A[h] * 1.4426950408889634f;   // log2 decay per unit step
        const float bias = a.dt_bias ? a.dt_bias[h] : 0.0f;
        auto load_x = [&](int i, int nth) {   // chunk i of the piece, the nth of all
            mbar_arrive_expect_tx(&fx.bar[nth & 1], kBlk);
            tma_rows(x_tile(nth), &maps.x, h * a.dv + c0, tm_b, tm_t + t_first + i * Q, &fx.bar[nth & 1]);
        };
        if (tma && lead) {
            load_x(0, n);
            if (chunks > 1) load_x(1, n + 1);
        }
        auto raw_step = [&](int i) -> unsigned short {
            return i < chunks ? dp[(p.row0 + (int64_t)(t_first + i * Q + r) * p.step) * a.lddt] : (unsigned short)0;
        };
        float d_next = 0.0f, wr = 0.0f, keep = 0.0f;
        long long gw_next = 0, gsum = 0;
        auto scan_steps = [&](unsigned short raw, int odd) {
            d_next = bf16_to_f(raw) + bias;
            if (a.softplus) d_next = softplus_f(d_next);
            gw_next = warp_scan(decay_of(d_next, A2));
            if (half == 0 && lane == 31) fx.wsum[odd][warp] = gw_next;
        };
        auto finish_steps = [&](int odd) {
            long long base = 0, total = 0;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const long long s = fx.wsum[odd][w];
                if (w < warp) base += s;
                total += s;
            }
            wr = d_next * exp2f(decay_f(total - base - gw_next));
            keep = exp2f(decay_f(total));
            gsum += total;
        };
        float S[HW];   // the state's key row r, this thread's columns
#pragma unroll
        for (int i = 0; i < HW; ++i) S[i] = 0.0f;
        // S <- decay S + the products of a chunk
        auto update = [&](int nth, float k) {
            tc_fence_after();
#pragma unroll
            for (int q = 0; q < HW; q += 16) {
                uint32_t v[16];
                tmem_ld_32x32b<16>(tl + (nth & 1) * PW + half * HW + q, v);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                    const float2 s = ffma2(f2(k, k), f2(S[q + i], S[q + i + 1]),
                                           f2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])));
                    S[q + i] = s.x;
                    S[q + i + 1] = s.y;
                }
            }
            tc_fence_before();
        };
        const unsigned short raw0 = raw_step(0);
        unsigned short raw = raw_step(1);
        scan_steps(raw0, 0);
        sync();
        finish_steps(0);
        scan_steps(raw, 1);
        float keep_before = 0.0f;
        for (int i = 0; i < chunks; ++i, ++n) {
            raw = raw_step(i + 2);
            // the chunk before has left X' and B
            if (i > 0 && !mbar_wait_bounded(mma_bar, (n - 1) & 1, nullptr)) fx.bad = 1;
            if (tma) {
                if (lead) {
                    mbar_arrive_expect_tx(b_bar, (DK / 64) * kBlk);
#pragma unroll
                    for (int j = 0; j < DK / 64; ++j)
                        tma_rows(sm + kOffB + j * kBlk, &maps.b, g * DK + 64 * j, tm_b, tm_t + t_first + i * Q, b_bar);
                }
                if (!mbar_wait_bounded(&fx.bar[n & 1], (n >> 1) & 1, nullptr)) fx.bad = 1;
            } else {
                const int t0 = t_first + i * Q;
                copy_tile(sm + kOffB, DK / 8, static_cast<const bf16 *>(a.Bm) + g * DK, a.ldb, p, t0, ti);
                copy_tile(x_tile(n), PW / 8, static_cast<const bf16 *>(a.x) + (int64_t)h * a.dv + c0, a.ldx, p, t0, ti);
                sync();
            }
            __syncwarp();
            split_x(sm, x_tile(n), r, half, wr);
            fence_async_smem();
            tc_fence_before();
            sync();
            if (n == 0 && grp == 0) asm volatile("bar.arrive 5, %0;" ::"n"(2 * kNT) : "memory");
            if (lead) {
                if (tma && !mbar_wait_bounded(b_bar, n & 1, nullptr)) fx.bad = 1;
                tc_fence_after();
                const uint64_t bd = desc_mn(sm + kOffB), wd = desc_mn(sm + kOffXw);
#pragma unroll
                for (int part = 0; part < 3; ++part)
#pragma unroll
                    for (int k = 0; k < Q / 16; ++k)
                        mma_ss(tm + (n & 1) * PW, bd + step_mn(k), wd + (part * kBlk >> 4) + step_mn(k),
                               idesc(PW, 1, 1), part + k > 0);
                umma_commit(mma_bar);
                if (tma && i + 2 < chunks) load_x(i + 2, n + 2);   // (X of this chunk has been read)
            }
            __syncwarp();
            if (i > 0) update(n - 1, keep_before);
            keep_before = keep;
            if (i + 1 < chunks) {
                finish_steps((i + 1) & 1);
                scan_steps(raw, i & 1);
            }
        }
        if (!mbar_wait_bounded(mma_bar, (n - 1) & 1, nullptr)) fx.bad = 1;
        __syncwarp();
        update(n - 1, keep_before);
        sync();   // every wait is over
        if (r < DK) {
            float4 *so = reinterpret_cast<float4 *>(a.ws + p.id * sall + ((int64_t)h * DK + r) * a.dv + c0 + half * HW);
            const float nan = __int_as_float(0x7fffffff);   // a wait that ran out leaves no state that looks like one
#pragma unroll
            for (int i = 0; i < HW / 4; ++i)
                so[i] = fx.bad ? make_float4(nan, nan, nan, nan)
                               : make_float4(S[4 * i], S[4 * i + 1], S[4 * i + 2], S[4 * i + 3]);
        }
        if (ti == 0 && c0 == 0) ssm_decays(a, seg)[p.id * a.H + h] = exp2f(decay_f(gsum));
        if (fx.bad) break;
    }
    if (n == 0 && grp == 0) asm volatile("bar.arrive 5, %0;" ::"n"(2 * kNT) : "memory");
    tc_fence_before();
    __syncthreads();
    if (wid == 1) {
        tmem_relinquish();
        tmem_dealloc(tmem, 256);
    }
}

// cuTensorMapEncodeTiled from the driver, looked up once.
PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        const bool ok = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
                        q == cudaDriverEntryPointSuccess;
        return ok ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p) : nullptr;
    }();
    return fn;
}

bool encode(CUtensorMap *m, const void *base, const Rows &r, int64_t width, int64_t ld) {
    const auto enc = encoder();
    if (!enc) return false;
    const bool packed = r.cu != nullptr;
    const cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)(packed ? 1 : r.B),
                                (cuuint64_t)(packed ? r.rows : r.rows / r.B)};
    const cuuint64_t strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)ld * 2 * (packed ? 1 : r.B)};
    const cuuint32_t box[3] = {64, 1, Q}, es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DK>
cudaError_t launch(const SsmArgs &a, const SsmMaps &maps, int seg, int tma, int split, cudaStream_t s) {
    constexpr int bytes = 2 * (kSmem + (int)sizeof(Fixed));
    static_assert(bytes <= 226 * 1024, "shared memory of one CTA");
    const int64_t units = (int64_t)a.H * (a.dv / PW);
    auto grid = [](int64_t items) { return (unsigned)(items < 2 * kSms ? (items + 1) / 2 : kSms); };
    cudaError_t e = cudaFuncSetAttribute(ssm_umma_kernel<DK>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    if (split) {
        e = cudaFuncSetAttribute(ssm_state_kernel<DK>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        const int64_t cuts = cut_count(a.r, seg) * units;
        ssm_state_kernel<DK><<<grid(cuts), 2 * kNT, bytes, s>>>(a, maps, seg, cuts, tma);
        e = launch_ssm_join(a, seg, s);
        if (e != cudaSuccess) return e;
    }
    ssm_umma_kernel<DK><<<grid(piece_count(a.r, seg) * units), 2 * kNT, bytes, s>>>(a, maps, seg, tma, split);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_ssm_umma(const SsmArgs &a, int seg, bool split, cudaStream_t s) {
    // Tensor copies and 16-byte stores need every row on a 16-byte boundary.
    const uintptr_t base = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.Bm) |
                           reinterpret_cast<uintptr_t>(a.Cm) | reinterpret_cast<uintptr_t>(a.y);
    SsmMaps maps{};
    const bool tma = base % 16 == 0 && a.ldx % 8 == 0 && a.ldb % 8 == 0 && a.ldc % 8 == 0 && a.ldy % 8 == 0 &&
                     encode(&maps.x, a.x, a.r, (int64_t)a.H * a.dv, a.ldx) &&
                     encode(&maps.b, a.Bm, a.r, (int64_t)a.G * a.dk, a.ldb) &&
                     encode(&maps.c, a.Cm, a.r, (int64_t)a.G * a.dk, a.ldc);
    return a.dk == 64 ? launch<64>(a, maps, seg, tma, split, s) : launch<128>(a, maps, seg, tma, split, s);
}

}  // namespace lq
