// lq_conv.cu -- short causal depthwise convolution of a recurrent layer's
// inputs, over prompts and for single tokens:
//   y_t[c] = act(bias[c] + sum_{j < K} w[c][j] x_{t-K+1+j}[c]),
// rows before a sequence's first from its window (the last K-1 inputs) or 0.
//
// Bound: HBM (2 K flops per element read and written once), then the two
// hardware exponential / reciprocal operations a SiLU takes.  A thread walks
// kRun tokens of one sequence for 4 channels (one for widths or rows whose
// alignment does not allow that): 4 channels keep a warp's accesses whole lines
// at 4 K weights in registers, half the registers and twice the warps of 8
// channels (119 us against 66 us for 32768 x 2304 bf16).  The next kAhead rows
// are on their way while one batch is at work, and the K-1 inputs behind stay
// in registers, so an input is read once plus K-1 halo rows per run.  Sums are
// FP32, the output is rounded once; the window holds the inputs as they came.
// 66 us is 0.70 of the copy rate: instruction issue (62% of slots, the exponential
// and reciprocal of two channels at a time the largest part) beside the loads.
#include "lq_act.cuh"
#include "lq_common.cuh"

namespace lq {
namespace {

constexpr int kConvThreads = 128;
constexpr int kRun = 32;      // tokens per piece: halo (K-1)/32 more reads, mostly L2 hits
constexpr int kAhead = 4;     // rows loaded ahead of the rows at work
constexpr int kSeqs = 4;      // sequences of one thread's batch in a step

// The K taps and the bias of V channels (V = 4: w and bias 16-byte aligned).
template <int V, int K>
__device__ __forceinline__ void load_taps(const ConvArgs &a, int c, float (&w)[V][K], float (&bias)[V]) {
    if constexpr (V == 4) {
        float flat[V * K];
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const float4 v = reinterpret_cast<const float4 *>(a.w + (int64_t)c * K)[i];
            flat[4 * i] = v.x; flat[4 * i + 1] = v.y; flat[4 * i + 2] = v.z; flat[4 * i + 3] = v.w;
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < K; ++j) w[i][j] = flat[i * K + j];
        const float4 b = a.bias ? *reinterpret_cast<const float4 *>(a.bias + c) : make_float4(0.f, 0.f, 0.f, 0.f);
        bias[0] = b.x; bias[1] = b.y; bias[2] = b.z; bias[3] = b.w;
    } else {
#pragma unroll
        for (int j = 0; j < K; ++j) w[0][j] = a.w[(int64_t)c * K + j];
        bias[0] = a.bias ? a.bias[c] : 0.0f;
    }
}

// act(bias + sum of the taps over rows x[0 .. K-1]) of V channels, two channels
// per instruction where there are four.
template <typename T, int V, int K, int R>
__device__ __forceinline__ void conv_rows(const float (&w)[V][K], const float (&bias)[V], const float (&x)[R][V], int u,
                                          int act, float (&out)[V]) {
    if constexpr (V == 4) {
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            float2 s = f2(bias[i], bias[i + 1]);
#pragma unroll
            for (int j = 0; j < K; ++j) s = ffma2(f2(w[i][j], w[i + 1][j]), f2(x[u + j][i], x[u + j][i + 1]), s);
            if (act) s = silu2_f<sizeof(T) == 4>(s);
            out[i] = s.x;
            out[i + 1] = s.y;
        }
    } else {
        float s = bias[0];
#pragma unroll
        for (int j = 0; j < K; ++j) s = fmaf(w[0][j], x[u + j][0], s);
        out[0] = act ? silu_f<sizeof(T) == 4>(s) : s;
    }
}

template <typename T, int V, int K>
__global__ void __launch_bounds__(kConvThreads, sizeof(T) == 4 ? 5 : 8) conv_prefill_kernel(ConvArgs a) {
    const int c = (blockIdx.y * kConvThreads + threadIdx.x) * V;
    Piece p;
    if (!find_piece(a.r, kRun, blockIdx.x, p) || c >= a.C) return;
    const T *x = static_cast<const T *>(a.x) + c;
    const T *s0 = static_cast<const T *>(a.state0);
    if (s0) s0 += (int64_t)p.b * (K - 1) * a.C + c;
    // Row t >= 0 of the sequence, or its window for t = -(K-1) .. -1.
    auto row = [&](int t) {
        Raw<T, V> r;
        if (t >= 0) r.load(x + (p.row0 + t * p.step) * a.ldx);
        else if (s0) r.load(s0 + (int64_t)(t + K - 1) * a.C);
        else r.zero();
        return r;
    };
    const int t0 = p.j * kRun, t1 = min(p.len, t0 + kRun);
    float in[K - 1 + kAhead][V];   // rows t-K+1 .. t+kAhead-1
#pragma unroll
    for (int j = 0; j < K - 1; ++j) row(t0 - (K - 1) + j).get(in[j]);
    if (p.j == 0 && a.state_out) {
        // The next window.  Only the first piece reads the old one, and this
        // thread reads all it needs of it before it writes: it may be in place.
        Raw<T, V> last[K - 1];
#pragma unroll
        for (int j = 0; j < K - 1; ++j) last[j] = row(p.len - (K - 1) + j);
        T *so = static_cast<T *>(a.state_out) + (int64_t)p.b * (K - 1) * a.C + c;
#pragma unroll
        for (int j = 0; j < K - 1; ++j) last[j].store(so + (int64_t)j * a.C);
    }
    if (t0 >= t1) return;
    float w[V][K], bias[V];
    load_taps<V, K>(a, c, w, bias);
    const int64_t dx = p.step * a.ldx, dy = p.step * a.ldy;
    const T *xr = x + (p.row0 + t0 * p.step) * a.ldx;
    T *yr = static_cast<T *>(a.y) + c + (p.row0 + t0 * p.step) * a.ldy;
    Raw<T, V> next[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
        if (t0 + u < t1) next[u].load(xr + u * dx);
    for (int t = t0; t < t1; t += kAhead) {
        xr += kAhead * dx;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            next[u].get(in[K - 1 + u]);   // (beyond t1: not used)
            if (t + kAhead + u < t1) next[u].load(xr + u * dx);
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (t + u < t1) {
                float out[V];
                conv_rows<T, V, K>(w, bias, in, u, a.act, out);
                Raw<T, V> o;
                o.set(out);
                o.store(yr + u * dy);
            }
        }
#pragma unroll
        for (int j = 0; j < K - 1; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) in[j][i] = in[kAhead + j][i];
        yr += kAhead * dy;
    }
}

// One token per sequence: the window is read, the output formed and the window
// shifted by one, in place.  A thread takes `per` sequences with one load of
// its weights, kSeqs of them at a time.
template <typename T, int V, int K>
__global__ void __launch_bounds__(kConvThreads) conv_step_kernel(ConvArgs a, int per) {
    const int c = (blockIdx.y * kConvThreads + threadIdx.x) * V;
    if (c >= a.C) return;
    const int b0 = blockIdx.x * per, b1 = min(a.r.B, b0 + per);
    float w[V][K], bias[V];
    load_taps<V, K>(a, c, w, bias);
    T *s = static_cast<T *>(a.state_out) + (int64_t)b0 * (K - 1) * a.C + c;
    for (int b = b0; b < b1; b += kSeqs, s += (int64_t)kSeqs * (K - 1) * a.C) {
        Raw<T, V> r[kSeqs][K];
#pragma unroll
        for (int u = 0; u < kSeqs; ++u)
            if (b + u < b1) {
#pragma unroll
                for (int j = 0; j < K - 1; ++j) r[u][j].load(s + (int64_t)(u * (K - 1) + j) * a.C);
                r[u][K - 1].load(static_cast<const T *>(a.x) + (b + u) * a.ldx + c);
            }
#pragma unroll
        for (int u = 0; u < kSeqs; ++u)
            if (b + u < b1) {
                float in[K][V], out[V];
#pragma unroll
                for (int j = 0; j < K; ++j) r[u][j].get(in[j]);
                conv_rows<T, V, K>(w, bias, in, 0, a.act, out);
                Raw<T, V> o;
                o.set(out);
                o.store(static_cast<T *>(a.y) + (b + u) * a.ldy + c);
#pragma unroll
                for (int j = 0; j < K - 1; ++j) r[u][j + 1].store(s + (int64_t)(u * (K - 1) + j) * a.C);
            }
    }
}

template <typename T, int V, int K>
cudaError_t launch(const ConvArgs &a, bool step, cudaStream_t s) {
    const int cx = (a.C + kConvThreads * V - 1) / (kConvThreads * V);
    if (step) {
        // Enough CTAs to fill the SMs (12 of 128 threads each) before a thread
        // takes more than one sequence.
        const int64_t ctas = 148 * 12;
        const int64_t per = ((int64_t)a.r.B * cx + ctas - 1) / ctas;
        conv_step_kernel<T, V, K><<<dim3((unsigned)((a.r.B + per - 1) / per), cx), kConvThreads, 0, s>>>(a, (int)per);
        return cudaGetLastError();
    }
    const int64_t pieces = piece_count(a.r, kRun);
    conv_prefill_kernel<T, V, K><<<dim3((unsigned)pieces, cx), kConvThreads, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T, int V>
cudaError_t by_taps(const ConvArgs &a, bool step, cudaStream_t s) {
    switch (a.K) {
        case 2: return launch<T, V, 2>(a, step, s);
        case 3: return launch<T, V, 3>(a, step, s);
        default: return launch<T, V, 4>(a, step, s);
    }
}

template <typename T>
cudaError_t by_width(const ConvArgs &a, bool step, cudaStream_t s) {
    // Vectors of 4 channels need the width, the row strides and every base to
    // keep their alignment.
    const uintptr_t base = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.y) |
                           reinterpret_cast<uintptr_t>(a.state0) | reinterpret_cast<uintptr_t>(a.state_out);
    const uintptr_t par = reinterpret_cast<uintptr_t>(a.w) | reinterpret_cast<uintptr_t>(a.bias);
    if (a.C % 4 == 0 && a.ldx % 4 == 0 && a.ldy % 4 == 0 && base % (4 * sizeof(T)) == 0 && par % 16 == 0)
        return by_taps<T, 4>(a, step, s);
    return by_taps<T, 1>(a, step, s);
}

cudaError_t by_type(const ConvArgs &a, int dtype, bool step, cudaStream_t s) {
    if (dtype == kF32) return by_width<float>(a, step, s);
    if (dtype == kBF16) return by_width<bf16>(a, step, s);
    return by_width<f16>(a, step, s);
}

}  // namespace

cudaError_t launch_conv_prefill(const ConvArgs &a, int dtype, cudaStream_t s) { return by_type(a, dtype, false, s); }
cudaError_t launch_conv_step(const ConvArgs &a, int dtype, cudaStream_t s) { return by_type(a, dtype, true, s); }

}  // namespace lq
