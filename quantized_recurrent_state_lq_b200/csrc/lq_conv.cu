// lq_conv.cu -- short causal depthwise convolution of a recurrent layer's
// inputs, over prompts and for single tokens:
//   y_t[c] = act(bias[c] + sum_{j < K} w[c][j] x_{t-K+1+j}[c]),
// rows before a sequence's first from its window (the last K-1 inputs) or 0.
//
// Bound: HBM (2 K flops per element read and written once).  A thread walks
// kRun tokens of one sequence for 8 channels (one for widths or rows that are
// not 16-byte aligned) and keeps the K-1 inputs behind the current one in
// registers, so an input is read once plus K-1 halo rows per run.  Sums are
// FP32, the output is rounded once; the window holds the inputs as they came.
#include "lq_act.cuh"

namespace lq {
namespace {

constexpr int kConvThreads = 128;
constexpr int kRun = 64;      // tokens per piece: halo (K-1)/64 more reads, mostly L2 hits
constexpr int kAhead = 4;     // rows loaded before they are used

template <typename T, int V, int K>
__device__ __forceinline__ void load_taps(const ConvArgs &a, int c, float (&w)[V][K], float (&bias)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int j = 0; j < K; ++j) w[i][j] = a.w[(int64_t)(c + i) * K + j];
        bias[i] = a.bias ? a.bias[c + i] : 0.0f;
    }
}

template <typename T>
__device__ __forceinline__ float conv_act(float v, int act) {
    return act ? silu_f<sizeof(T) == 4>(v) : v;
}

template <typename T, int V, int K>
__global__ void __launch_bounds__(kConvThreads) conv_prefill_kernel(ConvArgs a) {
    const int c = (blockIdx.y * kConvThreads + threadIdx.x) * V;
    Piece p;
    if (!find_piece(a.r, kRun, blockIdx.x, p) || c >= a.C) return;
    const T *x = static_cast<const T *>(a.x) + c;
    const T *s0 = static_cast<const T *>(a.state0);
    if (s0) s0 += (int64_t)p.b * (K - 1) * a.C + c;
    T *y = static_cast<T *>(a.y) + c;
    // Row t >= 0 of the sequence, or its window for t = -(K-1) .. -1.
    auto row = [&](int t) {
        Raw<T, V> r;
        if (t >= 0) r.load(x + (p.row0 + t * p.step) * a.ldx);
        else if (s0) r.load(s0 + (int64_t)(t + K - 1) * a.C);
        else r.zero();
        return r;
    };
    const int t0 = p.j * kRun, t1 = min(p.len, t0 + kRun);
    float past[K - 1][V];   // rows t0-K+1 .. t0-1, shifted along
#pragma unroll
    for (int j = 0; j < K - 1; ++j) row(t0 - (K - 1) + j).get(past[j]);
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
    load_taps<T, V, K>(a, c, w, bias);
    for (int t = t0; t < t1; t += kAhead) {
        Raw<T, V> in[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (t + u < t1) in[u].load(x + (p.row0 + (t + u) * p.step) * a.ldx);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (t + u >= t1) break;
            float cur[V], out[V];
            in[u].get(cur);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float s = bias[i];
#pragma unroll
                for (int j = 0; j < K - 1; ++j) s = fmaf(w[i][j], past[j][i], s);
                out[i] = conv_act<T>(fmaf(w[i][K - 1], cur[i], s), a.act);
#pragma unroll
                for (int j = 0; j < K - 2; ++j) past[j][i] = past[j + 1][i];
                past[K - 2][i] = cur[i];
            }
            Raw<T, V> o;
            o.set(out);
            o.store(y + (p.row0 + (t + u) * p.step) * a.ldy);
        }
    }
}

// One token per sequence: the window is read, the output formed and the window
// shifted by one, in place.
template <typename T, int V, int K>
__global__ void __launch_bounds__(kConvThreads) conv_step_kernel(ConvArgs a) {
    const int c = (blockIdx.y * kConvThreads + threadIdx.x) * V;
    if (c >= a.C) return;
    const int b = blockIdx.x;
    T *s = static_cast<T *>(a.state_out) + (int64_t)b * (K - 1) * a.C + c;
    Raw<T, V> r[K];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) r[j].load(s + (int64_t)j * a.C);
    r[K - 1].load(static_cast<const T *>(a.x) + b * a.ldx + c);
    float w[V][K], out[V];
    load_taps<T, V, K>(a, c, w, out);
#pragma unroll
    for (int j = 0; j < K; ++j) {
        float f[V];
        r[j].get(f);
#pragma unroll
        for (int i = 0; i < V; ++i) out[i] = fmaf(w[i][j], f[i], out[i]);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) out[i] = conv_act<T>(out[i], a.act);
    Raw<T, V> o;
    o.set(out);
    o.store(static_cast<T *>(a.y) + b * a.ldy + c);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) r[j + 1].store(s + (int64_t)j * a.C);
}

template <typename T, int V, int K>
cudaError_t launch(const ConvArgs &a, bool step, cudaStream_t s) {
    const int cx = (a.C + kConvThreads * V - 1) / (kConvThreads * V);
    if (step) {
        conv_step_kernel<T, V, K><<<dim3(a.r.B, cx), kConvThreads, 0, s>>>(a);
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
    // Vectors of 8 channels need the width, the row strides and every base to
    // keep 16-byte alignment (two 16-byte accesses for f32).
    const int unit = 16 / (int)sizeof(T);
    const uintptr_t base = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.y) |
                           reinterpret_cast<uintptr_t>(a.state0) | reinterpret_cast<uintptr_t>(a.state_out);
    if (a.C % 8 == 0 && a.ldx % unit == 0 && a.ldy % unit == 0 && base % 16 == 0) return by_taps<T, 8>(a, step, s);
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
