// lq_ssm.cu -- the selective state-space scan, token by token:
//   d_t = softplus(dt_t + bias) (or dt_t),  a_t = exp(d_t A_h),
//   S_t = a_t S_{t-1} + d_t B_t x_t^T,      y_t = S_t^T C_t + D_h x_t
// for states S [dk][dv] of every head (key rows, value columns); head h reads
// group h * G / H of B and C.
//
// ssm_step_kernel: bound by HBM, the state is read and written once (8 dk dv
// bytes per head against 5 dk dv flops).  The state's value columns are
// independent, so a CTA takes CW columns of a head: 64 when the heads fill
// the GPU (16 16-byte loads in flight per thread), 16 when they do not (four
// times the CTAs, a quarter of the serial work each).  The state stays in
// registers over the tokens of a short prompt.  256 sequences of 32 heads of
// 128 x 128 (1.07 GB): 161 us, the copy rate.
#include <algorithm>

#include "lq_ssm.h"

namespace lq {
namespace {

constexpr int kStepThreads = 128;

template <typename T, int DK, int DV, int CW>
__global__ void __launch_bounds__(kStepThreads) ssm_step_kernel(SsmArgs a) {
    constexpr int LR = CW / 4;               // lanes per key row
    constexpr int RG = kStepThreads / LR;    // key rows side by side
    constexpr int NR = DK / RG;              // key rows per thread
    __shared__ float sB[2][DK], sC[2][DK], sx[2][CW], part[kStepThreads / 32][CW];
    const int tid = threadIdx.x;
    const int slice = blockIdx.x % (DV / CW);
    const int64_t bh = blockIdx.x / (DV / CW);
    const int b = (int)(bh / a.H), h = (int)(bh - (int64_t)b * a.H);
    const int g = (int)((int64_t)h * a.G / a.H);
    Piece p;
    p.row0 = b;
    p.step = a.r.B;
    p.len = a.r.rows / a.r.B;
    if (a.r.cu) {
        const int c0 = cu_at(a.r, b);
        p.row0 = c0;
        p.step = 1;
        p.len = max(cu_at(a.r, b + 1), c0) - c0;
    }
    const int col = 4 * (tid % LR), rg = tid / LR;
    const int64_t base = bh * DK * DV + slice * CW + col;
    float4 S[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i)
        S[i] = a.S0 ? *reinterpret_cast<const float4 *>(a.S0 + base + (int64_t)(rg + i * RG) * DV)
                    : make_float4(0.f, 0.f, 0.f, 0.f);
    const float A = a.A[h], Dh = a.D ? a.D[h] : 0.0f, bias = a.dt_bias ? a.dt_bias[h] : 0.0f;
    // A token's inputs, on their way while the one before is at work.
    T rB, rC, rx, rd;
    auto fetch = [&](int t) {
        const int64_t row = p.row0 + t * p.step;
        if (tid < DK) {
            rB = static_cast<const T *>(a.Bm)[row * a.ldb + g * DK + tid];
            rC = static_cast<const T *>(a.Cm)[row * a.ldc + g * DK + tid];
        }
        if (tid < CW) rx = static_cast<const T *>(a.x)[row * a.ldx + (int64_t)h * DV + slice * CW + tid];
        rd = static_cast<const T *>(a.dt)[row * a.lddt + h];
    };
    if (p.len > 0) fetch(0);
    for (int t = 0; t < p.len; ++t) {
        const int o = t & 1;
        if (tid < DK) {
            sB[o][tid] = to_f<T>(rB);
            sC[o][tid] = to_f<T>(rC);
        }
        if (tid < CW) sx[o][tid] = to_f<T>(rx);
        float d = to_f<T>(rd) + bias;
        if (t + 1 < p.len) fetch(t + 1);
        if (a.softplus) d = softplus_f(d);
        const float keep = expf(d * A);
        __syncthreads();
        const float4 x = *reinterpret_cast<const float4 *>(sx[o] + col);
        const float4 dx = make_float4(d * x.x, d * x.y, d * x.z, d * x.w);
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const float bn = sB[o][rg + i * RG], cn = sC[o][rg + i * RG];
            S[i].x = fmaf(bn, dx.x, keep * S[i].x);
            S[i].y = fmaf(bn, dx.y, keep * S[i].y);
            S[i].z = fmaf(bn, dx.z, keep * S[i].z);
            S[i].w = fmaf(bn, dx.w, keep * S[i].w);
            y.x = fmaf(cn, S[i].x, y.x);
            y.y = fmaf(cn, S[i].y, y.y);
            y.z = fmaf(cn, S[i].z, y.z);
            y.w = fmaf(cn, S[i].w, y.w);
        }
#pragma unroll
        for (int m = LR; m < 32; m <<= 1) {
            y.x += __shfl_xor_sync(0xffffffffu, y.x, m);
            y.y += __shfl_xor_sync(0xffffffffu, y.y, m);
            y.z += __shfl_xor_sync(0xffffffffu, y.z, m);
            y.w += __shfl_xor_sync(0xffffffffu, y.w, m);
        }
        if ((tid & 31) < LR) *reinterpret_cast<float4 *>(&part[tid >> 5][col]) = y;
        __syncthreads();
        if (tid < CW) {
            float s = Dh * sx[o][tid];
#pragma unroll
            for (int w = 0; w < kStepThreads / 32; ++w) s += part[w][tid];
            static_cast<T *>(a.y)[(p.row0 + t * p.step) * a.ldy + (int64_t)h * DV + slice * CW + tid] = from_f<T>(s);
        }
    }
#pragma unroll
    for (int i = 0; i < NR; ++i) *reinterpret_cast<float4 *>(a.S_out + base + (int64_t)(rg + i * RG) * DV) = S[i];
}

template <typename T, int DK, int DV>
cudaError_t step(const SsmArgs &a, cudaStream_t s) {
    // One token is bound by its loads: two CTAs of 64 columns per SM, or four times
    // as many; more tokens by what every CTA does for each: one CTA per SM (16 tokens
    // of 8 x 16 heads of 128 x 128: 12.5 us against 18.5).
    const int64_t heads = (int64_t)a.r.B * a.H;
    if (heads * (DV / 64) >= (a.r.rows > a.r.B ? 148 : 148 * 2))
        ssm_step_kernel<T, DK, DV, 64><<<(unsigned)(heads * (DV / 64)), kStepThreads, 0, s>>>(a);
    else
        ssm_step_kernel<T, DK, DV, 16><<<(unsigned)(heads * (DV / 16)), kStepThreads, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t step_sizes(const SsmArgs &a, cudaStream_t s) {
    if (a.dk == 64) return a.dv == 64 ? step<T, 64, 64>(a, s) : step<T, 64, 128>(a, s);
    return a.dv == 64 ? step<T, 128, 64>(a, s) : step<T, 128, 128>(a, s);
}

}  // namespace

cudaError_t launch_ssm_step(const SsmArgs &a, int dtype, cudaStream_t s) {
    if (dtype == kF32) return step_sizes<float>(a, s);
    if (dtype == kBF16) return step_sizes<bf16>(a, s);
    return step_sizes<f16>(a, s);
}

namespace {

constexpr int kJoin = 8, kJoinThreads = 128;

// One thread per 4 state elements; block y takes every gridDim.y-th sequence and
// skips those of one piece, 32 at a time.  kJoin pieces' states are on their way
// at a time (128 pieces of 2 heads of 64 x 64: 25 us less than one by one, of 62).
__global__ void __launch_bounds__(kJoinThreads) ssm_join_kernel(SsmArgs a, int seg, bool early) {
    const int64_t per = (int64_t)a.dk * a.dv / 4, all = per * a.H;
    const int64_t i = (int64_t)blockIdx.x * kJoinThreads + threadIdx.x;   // (head, element)
    const int lane = threadIdx.x & 31, step = gridDim.y;
    if (early) let_next_kernel_start();
    wait_for_kernel_before();
    for (int64_t b0 = blockIdx.y; b0 < a.r.B; b0 += 32 * step) {
        const int64_t bl = b0 + lane * step;
        unsigned todo = __ballot_sync(0xffffffffu, bl < a.r.B && pieces_of(a.r, seg, (int)bl) > 1);
        for (; todo; todo &= todo - 1) {
            const int b = (int)(b0 + (__ffs(todo) - 1) * step), n = pieces_of(a.r, seg, b);
            if (i >= all) continue;
            const int64_t id = first_piece(a.r, seg, b);
            const float *decay = ssm_decays(a, seg) + id * a.H + i / per;
            float4 *slot = reinterpret_cast<float4 *>(a.ws) + id * all + i;
            float4 S = a.S0 ? reinterpret_cast<const float4 *>(a.S0)[b * all + i] : make_float4(0.f, 0.f, 0.f, 0.f);
            for (int j0 = 0; j0 < n; j0 += kJoin) {
                float4 own[kJoin];
                float f[kJoin];
#pragma unroll
                for (int j = 0; j < kJoin; ++j)
                    if (j0 + j + 1 < n) {   // the last piece has no state of its own
                        own[j] = slot[j * all];
                        f[j] = decay[j * a.H];
                    }
#pragma unroll
                for (int j = 0; j < kJoin; ++j) {
                    if (j0 + j < n) slot[j * all] = S;
                    if (j0 + j + 1 < n)
                        S = make_float4(fmaf(f[j], S.x, own[j].x), fmaf(f[j], S.y, own[j].y),
                                        fmaf(f[j], S.z, own[j].z), fmaf(f[j], S.w, own[j].w));
                }
                slot += kJoin * all;
                decay += (int64_t)kJoin * a.H;
            }
        }
    }
}

// What runs side by side: for bf16 one CTA per SM and 128 value columns, else a
// head each, two per SM for 128 value columns and four for 64 (16384 tokens of 16
// heads of 64 x 64: 267 us against 407 with two).
struct Fit {
    int64_t units, slots, chunk;
    Fit(int dtype, int H, int G, int dv) : units(H), slots(dv == 64 ? 148 * 4 : 148 * 2), chunk(32) {
        if (dtype != kBF16) return;
        slots = 148;
        chunk = 128;
        if (dv == 64) units = (int64_t)G * ((H / G + 1) / 2);
    }
};

// Tokens per piece of sequences of unknown lengths: pieces are cut so that the
// batch gives about as many CTAs as the GPU runs side by side.  A batch with enough
// sequences and heads is cut only where a sequence is longer than a CTA's share of
// all tokens.  Pieces hold whole chunks, down to a single one.
int ragged_piece(const Fit &f, int64_t rows) {
    const int64_t share = f.units <= f.slots ? (rows + f.slots / f.units - 1) / (f.slots / f.units)
                                             : (rows * f.units + f.slots - 1) / f.slots;
    const int64_t seg = (share + f.chunk - 1) / f.chunk * f.chunk;
    return (int)(seg < f.chunk ? f.chunk : seg > (1 << 30) ? (1 << 30) : seg);
}

// The same of B equal sequences of T tokens, by the chunk times that it takes.  A cut
// costs two launches and the pieces' own states at a third (by mma.sync 0.45) of a
// chunk's time.  bf16: not cut, or in as many pieces as give each CTA one, or one more
// or half as many; more pieces than CTAs leave some CTAs with part of a piece more
// than their share.  (16000 tokens of 10 sequences, 8 heads of 128 x 128: 95 us uncut,
// 128 cut.)  f32, f16: not cut, or as above -- several CTAs share an SM, whose rate is
// what counts.  (3000 tokens of 20 sequences, 24 f32 heads of 64 x 64: 67 and 107 us.)
int even_piece(const Fit &f, int dtype, int64_t B, int64_t T) {
    const int64_t n = (T + f.chunk - 1) / f.chunk, all = B * f.units;
    if (dtype != kBF16) {
        const int seg = ragged_piece(f, B * T);
        const float share = (float)all * (float)n / (float)f.slots, len = (float)(seg / f.chunk);
        return (float)n <= 1.8f + 1.45f * std::max(share, len) ? (int)(n * f.chunk) : seg;
    }
    const int64_t fill = f.slots / all;
    int64_t best = n;
    float least = 3.0e38f;
    for (int64_t m : {(int64_t)1, fill / 2, fill, fill + 1}) {
        m = std::max((int64_t)1, std::min(m, n));
        const int64_t len = (n + m - 1) / m, cut = (n + len - 1) / len;   // chunks, pieces
        const int64_t waves = (all * (cut - 1) + f.slots - 1) / f.slots;
        float time = all * cut <= f.slots ? (float)len : (float)all * (float)n / (float)f.slots + 0.75f * (float)len;
        if (cut > 1) time += 1.8f + 0.33f * (float)(waves * len);
        if (time < least) {
            least = time;
            best = len;
        }
    }
    return (int)(best * f.chunk);
}

// Sequences of at most this length are not cut: the two launches more cost what
// four chunks of 32 do.
constexpr int kWhole = 128;

// The longest that a sequence can be.
int64_t longest(const Rows &r) { return r.cu ? r.rows : r.rows / r.B; }

}  // namespace

cudaError_t launch_ssm_join(const SsmArgs &a, int seg, bool early, cudaStream_t s) {
    const int64_t n = (int64_t)a.H * a.dk * a.dv / 4, x = (n + kJoinThreads - 1) / kJoinThreads;
    const int64_t y = (4 * 148 + x - 1) / x;   // about four CTAs per SM
    return launch_after(ssm_join_kernel, dim3((unsigned)x, (unsigned)(y < a.r.B ? y : a.r.B)), kJoinThreads, 0, s, a,
                        seg, early);
}

// Whether a prompt runs token by token.  A chunk costs about as much (13 us for
// bf16, 9 for f16, 14 for f32) whatever it holds, a token 0.35 us with fewer CTAs
// than SMs and 0.6 with more: so do sequences of at most 16 tokens, 24 of few heads
// (f16 chunks are of 32), and packed batches of at most 2 tokens a sequence on
// average and 512 in all (64 single tokens of 32 heads of 128 x 128: 45 us against
// 155), where one long sequence costs no more than 512 steps.
bool token_by_token(const SsmArgs &a, int dtype) {
    const Rows &r = a.r;
    const int most = dtype != kF16 && (int64_t)r.B * a.H * (a.dv / 64) < 148 ? 24 : 16;
    if (!r.cu) return r.rows / r.B <= most;
    return r.rows <= most || (r.rows <= 2 * (int64_t)r.B && r.rows <= 512);
}

size_t ssm_ws_bytes(int dtype, int B, int rows, int H, int G, int dk, int dv) {
    if (rows <= kWhole) return 0;
    // for either form of the batch: packed, at most rows / seg + B pieces, or equal lengths
    const Fit f(dtype, H, G, dv);
    const int64_t T = rows / B;
    int64_t pieces = 0;
    if (B > 1) {
        const int seg = ragged_piece(f, rows);
        if (rows > seg) pieces = rows / seg + B;
    }
    if (T > kWhole) {
        const int seg = even_piece(f, dtype, B, T);
        if (T > seg) pieces = std::max(pieces, B * ((T + seg - 1) / seg) + (B == 1));
    }
    return ((size_t)pieces * H * (dk * dv + 1) * 4 + 255) / 256 * 256;
}

cudaError_t launch_ssm_prefill(const SsmArgs &a, int dtype, cudaStream_t s) {
    if (token_by_token(a, dtype)) return launch_ssm_step(a, dtype, s);
    const Fit f(dtype, a.H, a.G, a.dv);
    const int64_t most = longest(a.r);
    const int seg = most <= kWhole                ? kWhole
                    : a.r.cu && a.r.B > 1 ? ragged_piece(f, a.r.rows)
                                          : even_piece(f, dtype, a.r.B, most);
    const bool cut = most > seg;
    if (dtype == kBF16) return launch_ssm_umma(a, seg, cut, s);
    return launch_ssm_tc(a, dtype, seg, cut, s);
}

}  // namespace lq
