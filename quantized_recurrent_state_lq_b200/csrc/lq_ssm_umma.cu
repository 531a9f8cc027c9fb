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
// A CTA of 16 warps takes 128 value columns -- one head of 128 or two heads of 64
// of the same group of B and C -- over one piece of a sequence: four threads per
// token, key row and tensor-memory lane, 32 columns each.  A kernel that uses
// tensor memory gets one CTA per SM here, so the overlap is within the chunk:
//   C B^T, C S | M from C B^T, 2^(g_t) C S | M X beside X' | B^T X' beside the
//   outputs and the next chunk's decays | the state and its parts
// and the next chunk's tiles are on their way as soon as their places are free.
// 128 columns share one C B^T (and M, for one head) and run MMAs of N = 128 at 69
// cycles where two of N = 64 take 102: two independent groups of 64 columns took
// 16000 cycles a chunk against 11400 here.
// Long sequences of a small batch are cut into pieces: ssm_state_kernel forms each
// piece's own state, ssm_join_kernel chains them, and the scan starts every piece
// from its state (about a third more work for as many times the parallelism).
// 16384 rows of 40 sequences, 32 heads of 128 x 128: 300 us, tensor work 40% of a
// chunk's 11400 cycles and shared memory at work for 58% of them; one prompt of 16384,
// 32 heads of 128 x 64: 185 us (the pieces' states 42 of it, their join 6).
//
// Shared memory holds every operand as rows of 64 columns (128 bytes, the
// 16-byte chunks XOR-swizzled by the row's low 3 bits) in blocks of 16 KB:
// read as rows x K it is K-major, read as K x columns MN-major, so B serves
// C B^T and B^T X' from one copy, and a thread's accesses to its own row meet
// no bank conflict.  B, C and X arrive by TMA tensor copies:
//   [0, 32K) C, [32K, 64K) B, [64K, 96K) X and then the chunk's outputs,
//   [96K, 160K) S parts until C S is done, then [96K, 192K) X' parts
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
constexpr int CW = 32;                 // value columns of a thread
constexpr int kNT = 512;
constexpr int kBlk = Q * 128;          // bytes of 128 rows of 64 columns
constexpr int kOffC = 0, kOffB = 2 * kBlk, kOffX = 4 * kBlk, kOffU = 6 * kBlk, kOffF = 12 * kBlk;
// Decay factors of even and odd chunks, for up to two heads: [Q] sums within the
// warp (integer parts, negated), [Q] d, [3][Q] factors for the rows of later warps,
// [Q] the sums' fractions (negated).
constexpr int kFac = 6 * Q, kOffFixed = kOffF + 4 * kFac * 4;

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

// Thread l of the warp writes tensor-memory lane (taddr.lane + l), columns
// taddr.col .. taddr.col + 15 (shape 32x32b).
__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
        "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
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

// States: 32 columns x DK rows as 16-byte chunks of 4, swizzled like the tiles.
__device__ __forceinline__ void tma_state(void *dst, const CUtensorMap *map, int col, int row, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(col), "r"(row), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void tma_store_state(const CUtensorMap *map, const void *src, int col, int row) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(col), "r"(row), "r"(smem_u32(src))
                 : "memory");
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }

// bf16 parts of a pair: returns the pair rounded to bf16 and leaves the rests.
__device__ __forceinline__ uint32_t last_part(float2 v) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t *>(&p);
}
// (Values past the largest bf16 become that: the rest holds what is left of them,
// an infinity too.)
__device__ __forceinline__ uint32_t take_part(float2 &v) {
    uint32_t w;
    asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(v.y), "f"(v.x));
    v = ffma2(bf16x2_to_f2(w), f2(-1.0f, -1.0f), v);
    return w;
}

// Rows t0 .. t0 + Q - 1 of a sequence (zeros from its end on), NCH chunks of 8
// elements each, element by element.
__device__ __forceinline__ void copy_tile(unsigned char *dst, int nch, const bf16 *src, int64_t ld, const Piece &p,
                                          int t0) {
    for (int i = threadIdx.x; i < Q * nch; i += kNT) {
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
// The states as rows of dv floats, boxes of 32 columns x dk rows.
struct alignas(64) SsmMaps {
    CUtensorMap x, b, c, s0, ws, s_out;
};

// 128 value columns: one head of 128, or up to two heads of 64 of one group.
struct Unit {
    int h, heads, g;     // first head, heads, group of B and C
};

template <int HPC>
__host__ __device__ __forceinline__ int unit_count(int H, int G) {
    return HPC == 1 ? H : G * ((H / G + 1) / 2);
}

template <int HPC>
__device__ __forceinline__ Unit unit_of(int u, int H, int G) {
    const int hg = H / G;
    if (HPC == 1) return {u, 1, u / hg};
    const int pg = (hg + 1) / 2, g = u / pg, h = 2 * (u - g * pg);
    return {g * hg + h, min(2, hg - h), g};
}

// A CTA's work: one unit over one piece.
struct Item {
    Piece p;
    Unit u;
    int t_first, t_end;
    int tm_t, tm_b;      // where TMA finds token t: row tm_t + t of sequence tm_b
    bool valid;
};

// A CTA's share of the items: it takes every item that starts in its equal part
// of all chunks, the items in the order of sequences, pieces and units.
struct Walk {
    int64_t pos, end;    // start of the next item and end of the share, in chunks
    int b, j, u;         // the next item
};

struct Fixed {
    // G done; C S done; Y done; B^T X' done; B, C, X and the first state arrived
    uint64_t bar[8];
    long long wsum[2][2][4];   // each warp's log2 decay (even, odd chunks; heads)
    uint32_t tmem;
    int bad;             // a wait ran out
    int nf[2];           // a non-finite x in this chunk (even, odd chunks)
    Item item[2];        // the item at work and the next
    Walk walk;
    int first[2][2 * 64];   // per value column, the first token whose x is not finite
};
enum { kBarG, kBarCS, kBarY, kBarS, kBarB, kBarC, kBarX, kBarS0 };

// X' of token r, 32 columns from chunk j0 on, in three parts: w x.
__device__ __forceinline__ void split_x(unsigned char *dst, unsigned char *x, int r, int j0, float w) {
#pragma unroll
    for (int i = 0; i < CW / 8; ++i) {
        Raw<bf16, 8> rx;
        rx.a = *chunk(x, r, j0 + i);
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
            *chunk(dst + q * 2 * kBlk, r, j0 + i) = make_uint4(part[q][0], part[q][1], part[q][2], part[q][3]);
    }
}

// S <- k S + the products in tensor memory at `from`, 32 columns.
__device__ __forceinline__ void update_state(float (&S)[CW], uint32_t from, float k) {
#pragma unroll
    for (int q = 0; q < CW; q += 16) {
        uint32_t v[16];
        tmem_ld_32x32b<16>(from + q, v);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            const float2 s = ffma2(f2(k, k), f2(S[q + i], S[q + i + 1]),
                                   f2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])));
            S[q + i] = s.x;
            S[q + i + 1] = s.y;
        }
    }
}

// D[128][128] = B^T X', three parts, issued by one thread.
__device__ __forceinline__ void issue_state(uint32_t d, const unsigned char *b, const unsigned char *xw) {
    const uint64_t bd = desc_mn(b), wd = desc_mn(xw);
#pragma unroll
    for (int part = 0; part < 3; ++part)
#pragma unroll
        for (int k = 0; k < Q / 16; ++k)
            mma_ss(d, bd + step_mn(k), wd + (part * 2 * kBlk >> 4) + step_mn(k), idesc(2 * 64, 1, 1), part + k > 0);
}

// A token's step and decay: this thread's copy of its head's scan.
struct Steps {
    float d, A2, bias;
    long long gw;        // log2 decay up to this token within its warp's 32
    const unsigned short *dt;
    int64_t ld;
    bool softplus, on;

    __device__ __forceinline__ void head(const SsmArgs &a, int h, bool active) {
        on = active;
        softplus = a.softplus != 0;
        A2 = active ? a.A[h] * 1.4426950408889634f : 0.0f;   // log2 decay per unit step
        bias = active && a.dt_bias ? a.dt_bias[h] : 0.0f;
        dt = static_cast<const unsigned short *>(a.dt) + (active ? h : 0);
        ld = a.lddt;
    }
    // (as it is stored: the conversion would wait for it)
    __device__ __forceinline__ unsigned short load(const Piece &p, int t) const {
        return on && t < p.len ? dt[(p.row0 + (int64_t)t * p.step) * ld] : (unsigned short)0;
    }
    __device__ __forceinline__ void scan(unsigned short raw, bool live, long long *sum) {
        d = 0.0f;
        gw = 0;
        if (on && live) {
            d = bf16_to_f(raw) + bias;
            if (softplus) d = softplus_f(d);
            gw = decay_of(d, A2);
        }
        gw = warp_scan(gw);
        if (sum && (threadIdx.x & 31) == 31) *sum = gw;
    }
};

// Tokens of sequence b.
__device__ __forceinline__ int seq_len(const Rows &r, int b) {
    return r.cu ? max(cu_at(r, b + 1) - cu_at(r, b), 0) : r.rows / r.B;
}

__device__ __forceinline__ void place(const SsmArgs &a, int seg, Item &it) {
    it.t_first = it.p.j * seg;
    it.t_end = min(it.p.len, it.t_first + seg);
    it.tm_t = a.r.cu ? (int)it.p.row0 : 0;
    it.tm_b = a.r.cu ? 0 : it.p.b;
}

// The next item of the CTA's share (by one warp).
template <int HPC>
__device__ __forceinline__ void next_item(const SsmArgs &a, int seg, Fixed &fx, Item &out) {
    const int units = unit_count<HPC>(a.H, a.G);
    Walk w = fx.walk;
    Item it;
    it.valid = false;
    while (w.pos < w.end && w.b < a.r.B && !it.valid) {
        const int c0 = a.r.cu ? cu_at(a.r, w.b) : 0, len = seq_len(a.r, w.b), n = (len + seg - 1) / seg;
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
        it.u = unit_of<HPC>(w.u++, a.H, a.G);
        place(a, seg, it);
        w.pos += (it.t_end - it.t_first + Q - 1) / Q;
    }
    __syncwarp();
    if ((threadIdx.x & 31) == 0) {
        out = it;
        fx.walk = w;
    }
    __syncwarp();
}

// After a wait that ran out: NaN for the outputs and the final state of the item at
// work, item[sel], and of all that this CTA would have taken after it (item[sel ^ 1]
// holds the next one if `known`).  By the whole CTA; apart from the kernel, whose
// registers it would cost.
template <int DK, int HPC>
__device__ __noinline__ void leave_nan(const SsmArgs &a, int seg, Fixed &fx, int sel, bool known) {
    constexpr int DV = 128 / HPC;
    for (;; sel ^= 1, known = false) {
        const Item &it = fx.item[sel];
        const int width = it.u.heads * DV;
        for (int i = threadIdx.x; i < (it.t_end - it.t_first) * width; i += kNT) {
            const int64_t row = it.p.row0 + (int64_t)(it.t_first + i / width) * it.p.step;
            static_cast<uint16_t *>(a.y)[row * a.ldy + it.u.h * DV + i % width] = 0x7fff;
        }
        if (it.p.j == it.p.n - 1)
            for (int i = threadIdx.x; i < it.u.heads * DK * DV; i += kNT)
                a.S_out[((int64_t)it.p.b * a.H + it.u.h) * DK * DV + i] = __int_as_float(0x7fffffff);
        if (!known && threadIdx.x < 32) next_item<HPC>(a, seg, fx, fx.item[sel ^ 1]);
        __syncthreads();
        if (!fx.item[sel ^ 1].valid) return;
    }
}

// Outputs and final states.  Each CTA walks its share of the items; its second
// warp finds the next one and sends for its first tiles before the last one ends.
template <int DK, int HPC>
__global__ void __launch_bounds__(kNT, 1)
    ssm_umma_kernel(const __grid_constant__ SsmArgs a, const __grid_constant__ SsmMaps maps, int seg, int tma, int split,
                    int direct) {
    constexpr int DV = 128 / HPC;
    // Tensor memory: G at 0, Y with C S's first part at 128, its second at 256.
    // One head: M over G, the state's products at 384.  Two: M of the first at
    // 384, of the second at 256, the products over G.
    constexpr uint32_t kColY = 128, kColY2 = 256, kColS = HPC == 1 ? 384 : 0;
    extern __shared__ __align__(1024) unsigned char sm[];
    Fixed &fx = *reinterpret_cast<Fixed *>(sm + kOffFixed);
    const int ti = threadIdx.x, wid = ti >> 5, lane = ti & 31;
    const int warp = wid & 3, cq = wid >> 2, r = warp * 32 + lane;   // 32 rows, 32 columns of this warp
    const int hh = HPC == 2 ? cq >> 1 : 0;                           // this thread's head of the unit
    const int j0 = cq * (CW / 8);                                    // its first 16-byte chunk of a row
    // One thread of four warps issues, so that none is held up for long.
    const bool lead = ti == 0, lead_y = ti == 128, lead_x = ti == 256, finder = wid == 1;
    const int units = unit_count<HPC>(a.H, a.G);
    const int64_t sall = (int64_t)a.H * DK * DV;

    float S[CW];   // the state's key row r, this thread's columns
    // (Both by the second warp.)  The first item that starts in this CTA's part.
    auto start_walk = [&]() {
        Walk w{};
        auto seq_chunks = [&](int b) { return b < a.r.B ? (seq_len(a.r, b) + Q - 1) / Q : 0; };
        int64_t before = 0;   // chunks of the sequences before b
        w.b = a.r.B;
        if (!a.r.cu) {
            const int64_t each = (int64_t)seq_chunks(0) * units, all = each * a.r.B;
            w.pos = all * blockIdx.x / gridDim.x;
            w.end = all * (blockIdx.x + 1) / gridDim.x;
            if (w.pos < all) w.b = (int)(w.pos / each);
            before = w.b * each;
        } else {
            // The whole batch's chunks, then the sequence that holds the first
            // position: 8 sequences per lane and step.
            int64_t all = 0;
            for (int b0 = 0; b0 < a.r.B; b0 += 256)
#pragma unroll
                for (int i = 0; i < 8; ++i) all += seq_chunks(b0 + 8 * lane + i);
            all = warp_scan(all);
            all = __shfl_sync(0xffffffffu, all, 31) * units;
            w.pos = all * blockIdx.x / gridDim.x;
            w.end = all * (blockIdx.x + 1) / gridDim.x;
            for (int b0 = 0; b0 < a.r.B; b0 += 256) {
                int64_t n = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) n += (int64_t)seq_chunks(b0 + 8 * lane + i) * units;
                const int64_t upto = before + warp_scan(n);
                const unsigned in = __ballot_sync(0xffffffffu, upto > w.pos);
                if (in) {
                    const int l = __ffs(in) - 1;
                    before = __shfl_sync(0xffffffffu, upto - n, l);
                    w.b = b0 + 8 * l;
                    for (;;) {
                        const int64_t c = (int64_t)seq_chunks(w.b) * units;
                        if (before + c > w.pos) break;
                        before += c;
                        ++w.b;
                    }
                    break;
                }
                before = __shfl_sync(0xffffffffu, upto, 31);
            }
        }
        if (w.b < a.r.B) {
            const int len = seq_len(a.r, w.b), n = (len + seg - 1) / seg, whole = seg / Q;
            const int64_t o = w.pos - before, per = (int64_t)whole * units;
            w.j = (int)min(o / per, (int64_t)(n - 1));
            const int c = w.j < n - 1 ? whole : ((len - w.j * seg) + Q - 1) / Q;
            w.u = (int)((o - w.j * per + c - 1) / c);
            w.pos = before + w.j * per + (int64_t)w.u * c;
        }
        if (lane == 0) fx.walk = w;
        __syncwarp();
    };
    // No more items than CTAs: this one's is found without the walk (3000 cycles).
    auto only_item = [&]() {
        const int z = (int)(blockIdx.x / (unsigned)units);
        Item it;
        it.valid = find_piece(a.r, seg, z, it.p) && it.p.len > 0;
        it.u = unit_of<HPC>((int)(blockIdx.x - (unsigned)z * units), a.H, a.G);
        place(a, seg, it);
        if (lane == 0) {
            fx.item[0] = it;
            fx.walk = Walk{};
        }
        __syncwarp();
    };
    // B's place is free once B^T X' of the chunk before is done, C's once C S is,
    // X's once the outputs in it have been stored.
    auto load_b = [&](const Item &it, int t0) {
        mbar_arrive_expect_tx(&fx.bar[kBarB], DK / 64 * kBlk);
#pragma unroll
        for (int j = 0; j < DK / 64; ++j)
            tma_rows(sm + kOffB + j * kBlk, &maps.b, it.u.g * DK + 64 * j, it.tm_b, it.tm_t + t0, &fx.bar[kBarB]);
    };
    auto load_c = [&](const Item &it, int t0) {
        mbar_arrive_expect_tx(&fx.bar[kBarC], DK / 64 * kBlk);
#pragma unroll
        for (int j = 0; j < DK / 64; ++j)
            tma_rows(sm + kOffC + j * kBlk, &maps.c, it.u.g * DK + 64 * j, it.tm_b, it.tm_t + t0, &fx.bar[kBarC]);
    };
    auto load_x = [&](const Item &it, int t0) {
        const int blocks = HPC == 1 ? 2 : it.u.heads;
        mbar_arrive_expect_tx(&fx.bar[kBarX], blocks * kBlk);
        for (int j = 0; j < blocks; ++j)
            tma_rows(sm + kOffX + j * kBlk, &maps.x, it.u.h * DV + 64 * j, it.tm_b, it.tm_t + t0, &fx.bar[kBarX]);
    };
    // A state's 32-column blocks: on the way in where X and the third part of X'
    // go, on the way out where the first two parts went.
    auto s_in = [&](int c) { return sm + (c < 2 ? kOffX : kOffU + 2 * kBlk) + c * kBlk; };
    auto load_state = [&](const Item &it) {
        const bool cut = split && it.p.n > 1;
        if (!cut && !a.S0) return;
        const CUtensorMap *map = cut ? &maps.ws : &maps.s0;
        const int64_t head = (cut ? it.p.id : it.p.b) * a.H + it.u.h;
        const int blocks = it.u.heads * (DV / CW);
        mbar_arrive_expect_tx(&fx.bar[kBarS0], blocks * DK * 128);
        for (int c = 0; c < blocks; ++c)
            tma_state(s_in(c), map, c * CW % DV, (int)((head + c * CW / DV) * DK), &fx.bar[kBarS0]);
    };
    auto wait = [&](int bar, int parity) {
        if (!mbar_wait_bounded(&fx.bar[bar], parity, nullptr)) fx.bad = 1;
    };

    if (wid == 2) tmem_alloc(&fx.tmem, 512);
    if (finder) {
        if (direct) {
            only_item();
        } else {
            start_walk();
            next_item<HPC>(a, seg, fx, fx.item[0]);
        }
        if (lane == 0) {
            for (int i = 0; i < 8; ++i) mbar_init(&fx.bar[i], 1);
            fx.bad = 0;
            fence_mbar_init();
            if (fx.item[0].valid && tma) {
                load_b(fx.item[0], fx.item[0].t_first);
                load_c(fx.item[0], fx.item[0].t_first);
            }
        }
        wait_for_kernel_before();
        if (lane == 0 && fx.item[0].valid) load_state(fx.item[0]);
    }
    wait_for_kernel_before();
    if (a.r.cu) {   // a sequence without tokens hands its state through
        for (int b = blockIdx.x; b < a.r.B; b += gridDim.x)
            if (seq_len(a.r, b) == 0)
                for (int64_t i = ti; i < sall / 4; i += kNT)
                    reinterpret_cast<float4 *>(a.S_out + b * sall)[i] =
                        a.S0 ? reinterpret_cast<const float4 *>(a.S0 + b * sall)[i] : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (ti < 256) (&fx.first[0][0])[ti] = Q;
    if (ti < 2) fx.nf[ti] = 0;
    if (DK < 128) {   // B^T has 128 rows: the missing key rows are zero
        for (int i = ti; i < kBlk / 16; i += kNT)
            reinterpret_cast<uint4 *>(sm + kOffB + kBlk)[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = fx.tmem, tl = tm + ((uint32_t)warp << 21);   // this warp's lanes: 32 warp

    // Of the chunk at work: the log2 decay up to this token within its warp (integer
    // part and fraction), 2^ of that within the chunk, the token's weight in the next
    // state, the chunk's decay.
    float gi = 0.0f, gf = 0.0f, et = 0.0f, wr = 0.0f, keep = 0.0f;
    Steps st;
    int parity = 0, s_parity = 0;

    int sel = 0;
    bool known = false;
    for (; fx.item[sel].valid; sel ^= 1) {
        const Item &it = fx.item[sel];
        const Piece &p = it.p;
        const int t_end = it.t_end;
        const bool active = hh < it.u.heads;
        const int h = it.u.h + hh;
        const float Dh = active && a.D ? a.D[h] : 0.0f;
        st.head(a, h, active);
        // Of four (two) threads per token one writes its head's sums.
        auto scan = [&](unsigned short raw, int t, int odd) {
            st.scan(raw, t < p.len, (HPC == 2 ? (cq & 1) : cq) == 0 ? &fx.wsum[odd][hh][warp] : nullptr);
        };
        // The scanned chunk's factors, once every warp's sum is known.
        auto finish = [&](int odd) {
            long long base = 0, total = 0;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const long long s = fx.wsum[odd][hh][w];
                if (w < warp) base += s;
                total += s;
            }
            const long long gt = base + st.gw;
            decay_parts(st.gw, gi, gf);
            et = ex2_f(decay_f(gt));
            wr = st.d * exp2f(decay_f(total - gt));
            keep = exp2f(decay_f(total));
            // the threads of a token share the arrays out
            float *fl = reinterpret_cast<float *>(sm + kOffF) + (odd * 2 + hh) * kFac;
            const int part = HPC == 2 ? cq & 1 : cq;
            if (part == 0) {
                fl[r] = -gi;
                fl[Q + r] = st.d;
                fl[5 * Q + r] = -gf;
            }
            long long end = 0;   // 2^(sum to the end of tokens 32 w .. - g_s) d_s for the rows of later warps
#pragma unroll
            for (int w = 0; w < 3; ++w) {
                end += fx.wsum[odd][hh][w];
                if (w >= warp && part == (HPC == 2 ? 1 : w + 1)) fl[(2 + w) * Q + r] = st.d * exp2f(decay_f(end - gt));
            }
        };
        auto split_state = [&]() {   // the state's two parts
            if (r < DK) {
#pragma unroll
                for (int j = 0; j < CW / 8; ++j) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float2 v = f2(S[8 * j + 2 * k], S[8 * j + 2 * k + 1]);
                        hi[k] = take_part(v);
                        lo[k] = last_part(v);
                    }
                    *chunk(sm + kOffU, r, j0 + j) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *chunk(sm + kOffU + 2 * kBlk, r, j0 + j) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
            }
        };
        const unsigned short raw0 = st.load(p, it.t_first + r), raw1 = st.load(p, it.t_first + Q + r);
        scan(raw0, it.t_first + r, 0);
        const bool given = (split && p.n > 1) || a.S0;
        if (given) {
            wait(kBarS0, s_parity);
            s_parity ^= 1;
        }
        if (lead && p.row0 + it.t_first * p.step == a.fail_row) fx.bad = 1;
#pragma unroll
        for (int i = 0; i < CW / 4; ++i) {
            const uint4 z = make_uint4(0u, 0u, 0u, 0u), v = given && r < DK && active ? *chunk(s_in(cq), r, i) : z;
            S[4 * i] = __uint_as_float(v.x);
            S[4 * i + 1] = __uint_as_float(v.y);
            S[4 * i + 2] = __uint_as_float(v.z);
            S[4 * i + 3] = __uint_as_float(v.w);
        }
        __syncthreads();   // the state has been read, the one before has left
        split_state();
        if (HPC == 2 && !active) {   // no second head: zeros in its place
#pragma unroll
            for (int j = 0; j < CW / 8; ++j) *chunk(sm + kOffX, r, j0 + j) = make_uint4(0u, 0u, 0u, 0u);
        }
        finish(0);
        scan(raw1, it.t_first + Q + r, 1);
        int t0 = it.t_first;
        for (; t0 < t_end; t0 += Q, parity ^= 1) {
            const bool tail = t0 + Q > p.len, last = t0 + Q >= t_end;
            const int odd = ((t0 - it.t_first) / Q) & 1;
            fence_async_smem();
            tc_fence_before();
            __syncthreads();   // the chunk before is done with shared and tensor memory
            if (lead_x && tma) load_x(it, t0);
            if (fx.bad) {
                if (lead_x && tma) {   // the copies under way
                    wait(kBarB, parity);
                    wait(kBarC, parity);
                    wait(kBarX, parity);
                }
                break;
            }
            if (tma) {
                if (tail) {
                    // a packed sequence's last tile continues into the next sequence
                    wait(kBarB, parity);
                    wait(kBarC, parity);
                    wait(kBarX, parity);
                    if (t0 + r >= p.len) {
                        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                        for (int j = 0; j < DK / 32; ++j) {
                            *chunk(sm + kOffB, r, cq * (DK / 32) + j) = zero;
                            *chunk(sm + kOffC, r, cq * (DK / 32) + j) = zero;
                        }
#pragma unroll
                        for (int j = 0; j < CW / 8; ++j) *chunk(sm + kOffX, r, j0 + j) = zero;
                    }
                    fence_async_smem();
                    __syncthreads();
                }
            } else {
                copy_tile(sm + kOffB, DK / 8, static_cast<const bf16 *>(a.Bm) + it.u.g * DK, a.ldb, p, t0);
                copy_tile(sm + kOffC, DK / 8, static_cast<const bf16 *>(a.Cm) + it.u.g * DK, a.ldc, p, t0);
                copy_tile(sm + kOffX, it.u.heads * (DV / 8), static_cast<const bf16 *>(a.x) + (int64_t)it.u.h * DV, a.ldx,
                          p, t0);
                fence_async_smem();
                __syncthreads();
            }
            if (lead) {
                if (tma) {
                    wait(kBarB, parity);
                    wait(kBarC, parity);
                }
                tc_fence_after();
                const uint64_t cd = desc_k(sm + kOffC), bd = desc_k(sm + kOffB), sd = desc_mn(sm + kOffU);
#pragma unroll
                for (int k = 0; k < DK / 16; ++k) mma_ss(tm, cd + step_k(k), bd + step_k(k), idesc(Q, 0, 0), k > 0);
                umma_commit(&fx.bar[kBarG]);
                // C S, its parts side by side
#pragma unroll
                for (int k = 0; k < DK / 16; ++k)
                    mma_ss(tm + kColY, cd + step_k(k), sd + step_mn(k), idesc(256, 0, 1), k > 0);
                umma_commit(&fx.bar[kBarCS]);
            }
            __syncwarp();
            const unsigned short raw = st.load(p, t0 + 2 * Q + r);
            if (ti < 128) fx.first[parity ^ 1][ti] = Q;
            if (ti == 0) fx.nf[parity ^ 1] = 0;

            // 2^(g_t) on the sum of C S's parts.
            auto scale_cs = [&]() {
                wait(kBarCS, parity);
                __syncwarp();
                tc_fence_after();
#pragma unroll 1
                for (int q = 0; q < CW; q += 16) {
                    uint32_t v[16], v2[16];
                    tmem_ld_32x32b<16>(tl + kColY + cq * CW + q, v);
                    tmem_ld_32x32b<16>(tl + kColY2 + cq * CW + q, v2);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        v[i] = __float_as_uint(et * (__uint_as_float(v[i]) + __uint_as_float(v2[i])));
                    tmem_st_32x32b_x16(tl + kColY + cq * CW + q, v);
                }
            };
            if (HPC == 2) {   // the second M goes where C S's second part was
                scale_cs();
                tc_fence_before();
                __syncthreads();
                tc_fence_after();
            } else {
                wait(kBarG, parity);
                __syncwarp();
                tc_fence_after();
            }
            {
                // M from G, 16 tokens at a time: 8 columns of first parts, 8 of second.
                // Tokens of earlier warps factor through the boundary before this
                // warp's, those after this one are zero.  Within the warp the sums may be
                // large where their difference is small (31 tokens that wipe the state: 4650):
                // subtracted in two parts, the difference is good to 2^-24 (in one float
                // 2^-12 there, which showed in outputs whose terms cancel).
                const float *fl = reinterpret_cast<const float *>(sm + kOffF) + (odd * 2 + hh) * kFac;
                const uint32_t to = HPC == 1 ? tl : tl + (hh == 0 ? 384 : 256);
                const float rf = ex2_f(gi + gf);
                for (int q = HPC == 2 ? cq & 1 : cq; q < 8; q += HPC == 2 ? 2 : 4) {
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
                            const float4 *fs = reinterpret_cast<const float4 *>(fl + 5 * Q + 16 * q);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float4 gv = gs[i], dv = ds[i], fv = fs[i];
                                const float2 ge[2] = {f2(gv.x, gv.y), f2(gv.z, gv.w)}, de[2] = {f2(dv.x, dv.y), f2(dv.z, dv.w)};
                                const float2 fe[2] = {f2(fv.x, fv.y), f2(fv.z, fv.w)};
#pragma unroll
                                for (int k = 0; k < 2; ++k) {
                                    const float2 l = __fadd2_rn(__fadd2_rn(f2(gi, gi), ge[k]), __fadd2_rn(f2(gf, gf), fe[k]));
                                    const float2 gg = f2(__uint_as_float(v[4 * i + 2 * k]),
                                                         __uint_as_float(v[4 * i + 2 * k + 1]));
                                    float2 m = mul2(mul2(f2(ex2_f(l.x), ex2_f(l.y)), de[k]), gg);
                                    const int s = 16 * (q & 1) + 4 * i + 2 * k;
                                    if (s > lane) m.x = 0.0f;
                                    if (s + 1 > lane) m.y = 0.0f;
                                    hi[2 * i + k] = take_part(m);
                                    lo[2 * i + k] = last_part(m);
                                }
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            v[i] = hi[i];
                            v[8 + i] = lo[i];
                        }
                    }
                    tmem_st_32x32b_x16(to + 16 * q, v);
                }
            }
            if (HPC == 1) scale_cs();
            // A non-finite x leaves X (times 0 it would reach earlier tokens): its
            // column is marked from that token on, and has no finite state.
            bool poison = false;
            if (tma) wait(kBarX, parity);
#pragma unroll
            for (int i = 0; i < CW / 8; ++i) {
                const uint4 w4 = *chunk(sm + kOffX, r, j0 + i);
                const uint32_t wd[4] = {w4.x, w4.y, w4.z, w4.w};
                __nv_bfloat162 n = __float2bfloat162_rn(0.0f);   // 0 x finite = 0, else NaN
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    n = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&wd[k]), __float2bfloat162_rn(0.0f), n);
                poison |= (*reinterpret_cast<const uint32_t *>(&n) & 0x7fff7fffu) != 0;
            }
            if (poison) {
                for (int i = 0; i < CW / 8; ++i) {
                    Raw<bf16, 8> rx;
                    rx.a = *chunk(sm + kOffX, r, j0 + i);
                    float f[8];
                    rx.get(f);
                    for (int k = 0; k < 8; ++k)
                        if (!isfinite(f[k])) {
                            f[k] = 0.0f;
                            atomicMin(&fx.first[parity][8 * (j0 + i) + k], r);
                        }
                    rx.set(f);
                    *chunk(sm + kOffX, r, j0 + i) = rx.a;
                }
                fx.nf[parity] = 1;
            }
            __syncwarp();
            tmem_st_wait();
            fence_async_smem();
            tc_fence_before();
            __syncthreads();
            if (lead_y) {
                tc_fence_after();
                const uint64_t xd = desc_mn(sm + kOffX);
#pragma unroll
                for (int k = 0; k < Q / 16; ++k)
#pragma unroll
                    for (int part = 0; part < 2; ++part) {
                        if (HPC == 1) {
                            mma_ts(tm + kColY, tm + 16 * k + 8 * part, xd + step_mn(k), idesc(128, 0, 1), 1);
                        } else {
                            mma_ts(tm + kColY, tm + 384 + 16 * k + 8 * part, xd + step_mn(k), idesc(64, 0, 1), 1);
                            mma_ts(tm + kColY + 64, tm + 256 + 16 * k + 8 * part, xd + (kBlk >> 4) + step_mn(k),
                                   idesc(64, 0, 1), 1);
                        }
                    }
                umma_commit(&fx.bar[kBarY]);
            }
            if (finder && lane == 0 && tma && !last) load_c(it, t0 + Q);
            __syncwarp();
            split_x(sm + kOffU, sm + kOffX, r, j0, wr);
            fence_async_smem();
            tc_fence_before();
            __syncthreads();
            if (lead) {
                tc_fence_after();
                issue_state(tm + kColS, sm + kOffB, sm + kOffU);
                umma_commit(&fx.bar[kBarS]);
            }
            __syncwarp();
            const float keep_now = keep;
            if (!last) {
                finish(odd ^ 1);
                scan(raw, t0 + 2 * Q + r, odd);
            } else if (finder) {
                next_item<HPC>(a, seg, fx, fx.item[sel ^ 1]);
            }
            // outputs into X's place, then whole rows of 256 bytes at a time
            wait(kBarY, parity);
            __syncwarp();
            tc_fence_after();
            const bool nf = fx.nf[parity] != 0;
#pragma unroll 1
            for (int q = 0; q < CW; q += 16) {
                uint32_t v[16];
                tmem_ld_32x32b<16>(tl + kColY + cq * CW + q, v);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    uint4 *at8 = chunk(sm + kOffX, r, j0 + q / 8 + j);
                    Raw<bf16, 8> rx;
                    rx.a = *at8;
                    float f[8];
                    rx.get(f);
#pragma unroll
                    for (int k = 0; k < 8; ++k) f[k] = fmaf(Dh, f[k], __uint_as_float(v[8 * j + k]));
                    if (nf)
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            if (fx.first[parity][cq * CW + q + 8 * j + k] <= r) f[k] = __int_as_float(0x7fffffff);
                    rx.set(f);
                    *at8 = rx.a;
                }
            }
            __syncthreads();
            const int n8 = it.u.heads * (DV / 8);   // 16-byte chunks of a row
#pragma unroll
            for (int i = 0; i < Q * 16 / kNT; ++i) {
                const int t = (i * kNT + ti) / 16, j = ti % 16;
                if (t0 + t < p.len && j < n8) {
                    const uint4 w4 = *chunk(sm + kOffX, t, j);
                    bf16 *dst = static_cast<bf16 *>(a.y) + (p.row0 + (int64_t)(t0 + t) * p.step) * a.ldy + it.u.h * DV + 8 * j;
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
            wait(kBarS, parity);
            if (finder && lane == 0 && tma) {
                const Item &nx = fx.item[sel ^ 1];
                if (!last) {
                    load_b(it, t0 + Q);
                } else if (nx.valid) {
                    load_b(nx, nx.t_first);
                    load_c(nx, nx.t_first);
                }
            }
            __syncwarp();
            tc_fence_after();
            update_state(S, tl + kColS + cq * CW, keep_now);
            if (nf) {
#pragma unroll
                for (int i = 0; i < CW; ++i)
                    if (fx.first[parity][cq * CW + i] < Q) S[i] = __int_as_float(0x7fffffff);
            }
            if (!last) split_state();
        }
        // The last piece's state leaves.
        const bool ends = p.j == p.n - 1;
        if (ends && r < DK) {
#pragma unroll
            for (int i = 0; i < CW / 4; ++i)
                *chunk(sm + kOffU + cq * kBlk, r, i) =
                    make_uint4(__float_as_uint(S[4 * i]), __float_as_uint(S[4 * i + 1]), __float_as_uint(S[4 * i + 2]),
                               __float_as_uint(S[4 * i + 3]));
        }
        if (lead && p.row0 + (t_end - 1) * p.step == a.fail_row) fx.bad = 1;
        fence_async_smem();
        __syncthreads();   // (and the next item is known)
        if (fx.bad) {
            known = t0 >= t_end;
            if (known && lead_x && tma && fx.item[sel ^ 1].valid) {   // the next item's copies under way
                wait(kBarB, parity);
                wait(kBarC, parity);
            }
            break;
        }
        if (finder && lane == 0) {
            if (ends) {
                const int64_t head = (int64_t)p.b * a.H + it.u.h;
                for (int c = 0; c < it.u.heads * (DV / CW); ++c)
                    tma_store_state(&maps.s_out, sm + kOffU + c * kBlk, c * CW % DV, (int)((head + c * CW / DV) * DK));
                asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            }
            if (fx.item[sel ^ 1].valid) load_state(fx.item[sel ^ 1]);
            asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        }
        __syncwarp();
    }
    if (finder && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    if (fx.bad) leave_nan<DK, HPC>(a, seg, fx, sel, known);
    tc_fence_before();
    __syncthreads();
    if (wid == 2) {
        tmem_relinquish();
        tmem_dealloc(tm, 512);
    }
}

// The pieces' own states, from zero, and their decays, for every piece that is
// followed by another (all of them seg tokens long), one unit of one piece a CTA:
// only B^T X' and the state update.  Without C and S the tiles of B have two places,
// a chunk ahead, and the products of a chunk two accumulators, so that the update
// runs beside the next chunk's MMAs; a 17th warp issues the copies and the MMAs.
//   [0, 32K) B of even chunks, [32K, 64K) of odd ones, [64K, 96K) X, [96K, 192K) X' parts
template <int DK, int HPC>
__global__ void __launch_bounds__(kNT + 32, 1)
    ssm_state_kernel(SsmArgs a, const __grid_constant__ SsmMaps maps, int seg, int tma) {
    constexpr int DV = 128 / HPC;
    extern __shared__ __align__(1024) unsigned char sm[];
    Fixed &fx = *reinterpret_cast<Fixed *>(sm + kOffFixed);
    const int ti = threadIdx.x, wid = ti >> 5, lane = ti & 31;
    const int warp = wid & 3, cq = (wid >> 2) & 3, r = warp * 32 + lane;
    const int hh = HPC == 2 ? cq >> 1 : 0, j0 = cq * (CW / 8);
    const bool issuer = wid == kNT / 32, lead = ti == kNT;
    const int units = unit_count<HPC>(a.H, a.G), chunks = seg / Q;
    auto b_tile = [&](int n) { return sm + (n & 1 ? kOffB : kOffC); };
    uint64_t *x_bar = &fx.bar[2], *mma_bar = &fx.bar[3];   // and bar[0], bar[1]: B of even and odd chunks

    let_next_kernel_start();
    if (lead) {
        for (int i = 0; i < 4; ++i) mbar_init(&fx.bar[i], 1);
        fx.bad = 0;
        fence_mbar_init();
    }
    if (wid == 2) tmem_alloc(&fx.tmem, 256);
    if (DK < 128) {   // B^T has 128 rows: the missing key rows are zero
        for (int i = ti; i < kBlk / 16; i += kNT + 32)
            reinterpret_cast<uint4 *>(sm + kOffB + kBlk)[i] = reinterpret_cast<uint4 *>(sm + kOffC + kBlk)[i] =
                make_uint4(0u, 0u, 0u, 0u);
    }
    Piece p;   // found while tensor memory is allocated
    const int z = (int)(blockIdx.x / (unsigned)units);
    bool found = find_cut(a.r, seg, z, p);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = fx.tmem, tl = tm + ((uint32_t)warp << 21);   // this warp's lanes: 32 warp

    // (The issuing warp meets the others at the same barriers from code of its own.)
    auto sync = [&]() { asm volatile("bar.sync 1, %0;" ::"n"(kNT + 32) : "memory"); };
    int n = 0;   // chunks so far: the barriers' phases
    for (; found; found = false) {
        const Unit u = unit_of<HPC>((int)(blockIdx.x - (unsigned)z * units), a.H, a.G);
        const bool active = hh < u.heads;
        const int t_first = p.j * seg;
        const int tm_t = a.r.cu ? (int)p.row0 : 0, tm_b = a.r.cu ? 0 : p.b;
        auto load_x = [&](int i) {   // chunk i of the piece
            const int blocks = HPC == 1 ? 2 : u.heads;
            mbar_arrive_expect_tx(x_bar, blocks * kBlk);
            for (int j = 0; j < blocks; ++j)
                tma_rows(sm + kOffX + j * kBlk, &maps.x, u.h * DV + 64 * j, tm_b, tm_t + t_first + i * Q, x_bar);
        };
        auto load_b = [&](int i, int nth) {   // the nth of all
            uint64_t *bar = &fx.bar[nth & 1];
            mbar_arrive_expect_tx(bar, DK / 64 * kBlk);
#pragma unroll
            for (int j = 0; j < DK / 64; ++j)
                tma_rows(b_tile(nth) + j * kBlk, &maps.b, u.g * DK + 64 * j, tm_b, tm_t + t_first + i * Q, bar);
        };
        if (tma && lead) {
            load_x(0);
            load_b(0, n);
        }
        if (issuer) {
            sync();
            for (int i = 0; i < chunks; ++i, ++n) {
                // the chunk before has left X' and its B
                if (i > 0 && !mbar_wait_bounded(mma_bar, (n - 1) & 1, nullptr)) fx.bad = 1;
                if (tma && lead && i + 1 < chunks) load_b(i + 1, n + 1);
                if (!tma) sync();
                sync();   // X' is in place
                if (lead) {
                    if (tma && i + 1 < chunks) load_x(i + 1);   // (X of this chunk has been read)
                    if (tma && !mbar_wait_bounded(&fx.bar[n & 1], (n >> 1) & 1, nullptr)) fx.bad = 1;
                    tc_fence_after();
                    issue_state(tm + (n & 1) * 128, b_tile(n), sm + kOffU);
                    umma_commit(mma_bar);
                }
                __syncwarp();
            }
            if (!mbar_wait_bounded(mma_bar, (n - 1) & 1, nullptr)) fx.bad = 1;
            if (lead && p.row0 + t_first * p.step == a.fail_row) fx.bad = 1;
            sync();   // every wait is over
            sync();   // the state is where X' was
            if (lead) {
                const int64_t head = p.id * a.H + u.h;
                for (int c = 0; c < u.heads * (DV / CW); ++c)
                    tma_store_state(&maps.ws, sm + kOffU + c * kBlk, c * CW % DV, (int)((head + c * CW / DV) * DK));
                asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            }
            __syncwarp();
            if (fx.bad) break;
            continue;
        }
        if (HPC == 2 && !active) {   // no second head: zeros in its place
#pragma unroll
            for (int j = 0; j < CW / 8; ++j) *chunk(sm + kOffX, r, j0 + j) = make_uint4(0u, 0u, 0u, 0u);
        }
        Steps st;
        st.head(a, u.h + hh, active);
        float wr = 0.0f, keep = 0.0f, keep_before = 0.0f;
        long long gsum = 0;
        auto scan = [&](unsigned short raw, bool live, int odd) {
            st.scan(raw, live, (HPC == 2 ? (cq & 1) : cq) == 0 ? &fx.wsum[odd][hh][warp] : nullptr);
        };
        auto finish = [&](int odd) {
            long long base = 0, total = 0;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const long long s = fx.wsum[odd][hh][w];
                if (w < warp) base += s;
                total += s;
            }
            wr = st.d * exp2f(decay_f(total - base - st.gw));
            keep = exp2f(decay_f(total));
            gsum += total;
        };
        float S[CW];   // the state's key row r, this thread's columns
#pragma unroll
        for (int i = 0; i < CW; ++i) S[i] = 0.0f;
        const unsigned short raw0 = st.load(p, t_first + r);
        unsigned short raw = st.load(p, t_first + Q + r);
        scan(raw0, true, 0);
        sync();
        finish(0);
        scan(raw, chunks > 1, 1);
        for (int i = 0; i < chunks; ++i, ++n) {
            raw = st.load(p, t_first + (i + 2) * Q + r);
            // the chunk before has left X'
            if (i > 0 && !mbar_wait_bounded(mma_bar, (n - 1) & 1, nullptr)) fx.bad = 1;
            if (tma) {
                if (!mbar_wait_bounded(x_bar, n & 1, nullptr)) fx.bad = 1;
            } else {
                const int t0 = t_first + i * Q;
                copy_tile(b_tile(n), DK / 8, static_cast<const bf16 *>(a.Bm) + u.g * DK, a.ldb, p, t0);
                copy_tile(sm + kOffX, u.heads * (DV / 8), static_cast<const bf16 *>(a.x) + (int64_t)u.h * DV, a.ldx, p, t0);
                sync();
            }
            __syncwarp();
            split_x(sm + kOffU, sm + kOffX, r, j0, wr);
            fence_async_smem();
            tc_fence_before();
            sync();
            if (i > 0) {
                tc_fence_after();
                update_state(S, tl + ((n - 1) & 1) * 128 + cq * CW, keep_before);
                tc_fence_before();
            }
            keep_before = keep;
            if (i + 1 < chunks) {
                finish((i + 1) & 1);
                scan(raw, i + 2 < chunks, i & 1);
            }
        }
        if (!mbar_wait_bounded(mma_bar, (n - 1) & 1, nullptr)) fx.bad = 1;
        __syncwarp();
        tc_fence_after();
        update_state(S, tl + ((n - 1) & 1) * 128 + cq * CW, keep_before);
        tc_fence_before();
        sync();   // every wait is over
        const bool bad = fx.bad;   // after a wait that ran out: NaN
        if (r < DK) {
#pragma unroll
            for (int i = 0; i < CW / 4; ++i) {
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) w[k] = bad ? 0x7fffffffu : __float_as_uint(S[4 * i + k]);
                *chunk(sm + kOffU + cq * kBlk, r, i) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        fence_async_smem();
        sync();
        if (active && r == 0 && (HPC == 2 ? (cq & 1) : cq) == 0)
            ssm_decays(a, seg)[p.id * a.H + u.h + hh] = exp2f(decay_f(gsum));
        if (bad) break;
    }
    if (lead) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    tc_fence_before();
    __syncthreads();
    if (wid == 2) {
        tmem_relinquish();
        tmem_dealloc(tm, 256);
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

bool encode_states(CUtensorMap *m, const float *base, int64_t heads, int dk, int dv) {
    const auto enc = encoder();
    if (!enc) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)dv, (cuuint64_t)heads * dk}, strides[1] = {(cuuint64_t)dv * 4};
    const cuuint32_t box[2] = {CW, (cuuint32_t)dk}, es[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<float *>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DK, int HPC>
cudaError_t launch(const SsmArgs &a, const SsmMaps &maps, int seg, int tma, int split, cudaStream_t s) {
    constexpr int bytes = kOffFixed + (int)sizeof(Fixed);
    static_assert(bytes <= 227 * 1024, "shared memory of one CTA");
    const int64_t units = unit_count<HPC>(a.H, a.G);
    auto grid = [](int64_t items) { return (unsigned)(items < kSms ? items : kSms); };
    cudaError_t e = cudaFuncSetAttribute(ssm_umma_kernel<DK, HPC>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    if (split) {
        e = cudaFuncSetAttribute(ssm_state_kernel<DK, HPC>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        ssm_state_kernel<DK, HPC><<<(unsigned)(cut_count(a.r, seg) * units), kNT + 32, bytes, s>>>(a, maps, seg, tma);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        e = launch_ssm_join(a, seg, true, s);
        if (e != cudaSuccess) return e;
    }
    const int64_t items = piece_count(a.r, seg) * units;
    if (split) return launch_after(ssm_umma_kernel<DK, HPC>, grid(items), kNT, bytes, s, a, maps, seg, tma, split, items <= kSms);
    ssm_umma_kernel<DK, HPC><<<grid(items), kNT, bytes, s>>>(a, maps, seg, tma, split, items <= kSms);
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
    const int64_t heads = (int64_t)a.r.B * a.H;
    if (!encode_states(&maps.s_out, a.S_out, heads, a.dk, a.dv) ||
        (a.S0 && !encode_states(&maps.s0, a.S0, heads, a.dk, a.dv)) ||
        (split && !encode_states(&maps.ws, a.ws, piece_count(a.r, seg) * a.H, a.dk, a.dv)))
        return cudaErrorNotSupported;
    if (a.dv == 128)
        return a.dk == 64 ? launch<64, 1>(a, maps, seg, tma, split, s) : launch<128, 1>(a, maps, seg, tma, split, s);
    return a.dk == 64 ? launch<64, 2>(a, maps, seg, tma, split, s) : launch<128, 2>(a, maps, seg, tma, split, s);
}

}  // namespace lq
