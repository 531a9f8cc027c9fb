// lq_norm.cu -- the root-mean-square norms around a block:
//   norm_in:   h = res + scale x,           y = rms(h) w
//   norm_out:  y = res + scale [rms(x) w act(z)]   or, gate first,
//              y = res + scale [rms(x act(z)) w]
// with rms(u) = u / sqrt(mean u^2 + eps) over each group of D elements.
//
// Bound: HBM; every array is read and written once.  A team of threads holds
// its group's elements in registers between the statistic and the output (in
// FP32, unrounded; the output takes the one rounding), 8 elements per access
// when rows and strides are 16-byte aligned, else one.  Every element is read
// by the thread that writes it, after the whole group has been read, so y and
// h may be x, z or res themselves.  norm_in of 16384 rows of 4096 bf16 (537 MB):
// 89 us, 0.92 of the copy rate; norm_out of 16384 rows of 2048 f16 with gate and
// residual (268 MB): 53 us, 0.77 (issue at 76%, the gates' exponentials).
#include "lq_act.cuh"

namespace lq {
namespace {

// V consecutive FP32 parameters (16-byte aligned for V = 8), or a constant.
template <int V>
__device__ __forceinline__ void params(const float *p, float (&f)[V]) {
    Raw<float, V> r;
    r.load(p);
    r.get(f);
}

// The residual scale of V elements.
template <int V>
__device__ __forceinline__ void scales(const NormArgs &a, int64_t e, float (&f)[V]) {
    if (a.dscale) {
        params<V>(a.dscale + e, f);
#pragma unroll
        for (int k = 0; k < V; ++k) f[k] *= a.scale;
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k) f[k] = a.scale;
    }
}

// Sum over a team of TEAM threads: lanes of a warp, or the whole CTA.
template <int TEAM>
__device__ __forceinline__ float team_sum(float v) {
    constexpr int W = TEAM < 32 ? TEAM : 32;
#pragma unroll
    for (int m = W / 2; m >= 1; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    if constexpr (TEAM > 32) {
        __shared__ float part[TEAM / 32];
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < TEAM / 32; ++i) v += part[i];
    }
    return v;
}

template <typename T, typename TX, int V, int TEAM, int NV, bool IN>
__global__ void __launch_bounds__(TEAM > 128 ? TEAM : 128) norm_kernel(NormArgs a) {
    static_assert(TEAM <= 32 || TEAM >= 128, "a team is part of a warp, or the CTA");
    constexpr int kTeams = (TEAM > 128 ? TEAM : 128) / TEAM;
    constexpr bool EXACT = sizeof(T) == 4;
    const int tid = threadIdx.x % TEAM;
    const int64_t id = (int64_t)blockIdx.x * kTeams + threadIdx.x / TEAM;   // (row, group)
    // A team past the last group stays for the shuffles and does nothing else.
    const bool live = id < a.rows * a.G;
    const int64_t row = live ? id / a.G : 0;
    const int g = live ? (int)(id - row * a.G) : 0;
    const int n = live ? a.D / V : 0;
    const int64_t off = (int64_t)g * a.D;
    const TX *x = static_cast<const TX *>(a.x) + row * a.ldx + off;
    const T *z = a.z ? static_cast<const T *>(a.z) + row * a.ldz + off : nullptr;
    const T *res = a.res ? static_cast<const T *>(a.res) + row * a.ldres + off : nullptr;

    Raw<TX, V> rx[NV];
    Raw<T, V> rz[NV], rr[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = (i * TEAM + tid) * V;
        if (i * TEAM + tid < n) {
            rx[i].load(x + e);
            if (!IN && z) rz[i].load(z + e);
            if (res) rr[i].load(res + e);
        }
    }
    float u[NV][V];
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = (i * TEAM + tid) * V;
        if (i * TEAM + tid < n) {
            rx[i].get(u[i]);
            if constexpr (IN) {
                float r[V], sc[V];
                if (res) rr[i].get(r);
                scales<V>(a, off + e, sc);
#pragma unroll
                for (int k = 0; k < V; ++k) u[i][k] = res ? fmaf(sc[k], u[i][k], r[k]) : sc[k] * u[i][k];
            } else if (z && a.gate_first) {
                float f[V];
                rz[i].get(f);
#pragma unroll
                for (int k = 0; k < V; ++k) u[i][k] *= a.act ? sigmoid_f<EXACT>(f[k]) : silu_f<EXACT>(f[k]);
            }
#pragma unroll
            for (int k = 0; k < V; ++k) sum = fmaf(u[i][k], u[i][k], sum);
        }
    }
    sum = team_sum<TEAM>(sum);
    const float inv = 1.0f / sqrtf(sum / (float)a.D + a.eps);
    const float *w = a.w + (a.w_groups ? off : 0);
    T *y = static_cast<T *>(a.y) + row * a.ldy + off;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = (i * TEAM + tid) * V;
        if (i * TEAM + tid < n) {
            float o[V], f[V];
            params<V>(w + e, f);
#pragma unroll
            for (int k = 0; k < V; ++k) o[k] = u[i][k] * inv * f[k];
            if constexpr (IN) {
                if (a.h) {
                    Raw<T, V> rh;
                    rh.set(u[i]);
                    rh.store(static_cast<T *>(a.h) + row * a.ldh + off + e);
                }
            } else {
                if (z && !a.gate_first) {
                    rz[i].get(f);
#pragma unroll
                    for (int k = 0; k < V; ++k) o[k] *= a.act ? sigmoid_f<EXACT>(f[k]) : silu_f<EXACT>(f[k]);
                }
                float r[V];
                if (res) rr[i].get(r);
                scales<V>(a, off + e, f);
#pragma unroll
                for (int k = 0; k < V; ++k) o[k] = res ? fmaf(f[k], o[k], r[k]) : f[k] * o[k];
            }
            Raw<T, V> ro;
            ro.set(o);
            ro.store(y + e);
        }
    }
}

template <typename T, typename TX, int V, int TEAM, int NV, bool IN>
cudaError_t launch(const NormArgs &a, cudaStream_t s) {
    constexpr int kTeams = (TEAM > 128 ? TEAM : 128) / TEAM;
    const int64_t blocks = (a.rows * a.G + kTeams - 1) / kTeams;
    norm_kernel<T, TX, V, TEAM, NV, IN><<<(unsigned)blocks, kTeams * TEAM, 0, s>>>(a);
    return cudaGetLastError();
}

// Team and elements per thread by the group's size alone: few enough threads
// that most of them have work, few enough elements (up to 64 in registers) that
// small groups do not step through empty ones.  Without vector accesses the time
// goes to latency with every warp an SM holds at work, so what counts is the
// groups in flight: small teams of 4 to 12 elements a thread (norm_in of 67 M bf16
// elements, 537 MB in its four arrays, groups of 31: 184 us, 437 with a warp each; of
// 130: 163 and 438; of 1025: 159 and 328; a sixteenth of that, within L2: 14 and 29,
// 12 and 29, 12 and 23).
template <typename T, typename TX, bool IN>
cudaError_t by_size(const NormArgs &a, cudaStream_t s) {
    const uintptr_t base = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.z) |
                           reinterpret_cast<uintptr_t>(a.res) | reinterpret_cast<uintptr_t>(a.h) |
                           reinterpret_cast<uintptr_t>(a.y) | reinterpret_cast<uintptr_t>(a.w) |
                           reinterpret_cast<uintptr_t>(a.dscale);
    const int u = 16 / (int)sizeof(T), ux = 16 / (int)sizeof(TX);
    if (a.D % 8 == 0 && base % 16 == 0 && a.ldx % ux == 0 && a.ldz % u == 0 && a.ldres % u == 0 && a.ldh % u == 0 &&
        a.ldy % u == 0) {
        if (a.D <= 64) return launch<T, TX, 8, 8, 1, IN>(a, s);
        if (a.D <= 128) return launch<T, TX, 8, 16, 1, IN>(a, s);
        if (a.D <= 512) return launch<T, TX, 8, 32, 2, IN>(a, s);
        if (a.D <= 2048) return launch<T, TX, 8, 128, 2, IN>(a, s);
        if (a.D <= 4096) return launch<T, TX, 8, 256, 2, IN>(a, s);
        return launch<T, TX, 8, 512, 4, IN>(a, s);
    }
    if (a.D <= 16) return launch<T, TX, 1, 4, 4, IN>(a, s);
    if (a.D <= 32) return launch<T, TX, 1, 8, 4, IN>(a, s);
    if (a.D <= 48) return launch<T, TX, 1, 8, 6, IN>(a, s);
    if (a.D <= 64) return launch<T, TX, 1, 16, 4, IN>(a, s);
    if (a.D <= 96) return launch<T, TX, 1, 16, 6, IN>(a, s);
    if (a.D <= 128) return launch<T, TX, 1, 16, 8, IN>(a, s);
    if (a.D <= 192) return launch<T, TX, 1, 32, 6, IN>(a, s);
    if (a.D <= 256) return launch<T, TX, 1, 32, 8, IN>(a, s);
    if (a.D <= 384) return launch<T, TX, 1, 32, 12, IN>(a, s);
    if (a.D <= 512) return launch<T, TX, 1, 128, 4, IN>(a, s);
    if (a.D <= 1024) return launch<T, TX, 1, 128, 8, IN>(a, s);
    if (a.D <= 1536) return launch<T, TX, 1, 256, 6, IN>(a, s);
    if (a.D <= 2048) return launch<T, TX, 1, 256, 8, IN>(a, s);
    if (a.D <= 4096) return launch<T, TX, 1, 512, 8, IN>(a, s);
    return launch<T, TX, 1, 1024, 16, IN>(a, s);
}

}  // namespace

cudaError_t launch_norm_in(const NormArgs &a, int dtype, cudaStream_t s) {
    if (dtype == kF32) return by_size<float, float, true>(a, s);
    if (dtype == kBF16) return by_size<bf16, bf16, true>(a, s);
    return by_size<f16, f16, true>(a, s);
}

cudaError_t launch_norm_out(const NormArgs &a, int dtype, int x_dtype, cudaStream_t s) {
    if (dtype == kF32) return by_size<float, float, false>(a, s);
    if (dtype == kBF16)
        return x_dtype == kF32 ? by_size<bf16, float, false>(a, s) : by_size<bf16, bf16, false>(a, s);
    return x_dtype == kF32 ? by_size<f16, float, false>(a, s) : by_size<f16, f16, false>(a, s);
}

}  // namespace lq
