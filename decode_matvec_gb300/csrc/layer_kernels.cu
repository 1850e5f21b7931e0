// What a decoder layer needs between its attention and its experts: the norm of whole rows with the
// residual's addition, and the choice of experts from scores with a bias and groups.

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "device_common.cuh"

namespace {

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *(uint32_t*)&p;
}

// ---------------------------------------------------------------- norm of a row
//
// h = x + r, r' = bf16(h), y = h / sqrt(mean(h^2) + eps) w in fp32, rounded once to bf16; in 8 bits, with a scale for
// each row or each 128 values, s = max |y| / 448 and the code of y / s.  A row stays in registers between its sum and its
// output, so that every value is read once.
struct NormArgs {
    const void* x;
    const uint16_t* residual;
    uint16_t* residual_out;
    const uint16_t* weight;
    uint16_t* y;
    uint8_t* codes;
    float* scales;
    int64_t x_stride, res_stride, res_out_stride, y_stride;
    int T, n;
    int row_scale;     // one scale a row (0: one for each 128 values)
    float eps;
};

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

template <int V>
__device__ __forceinline__ void load_bf16(const uint16_t* p, float (&v)[V]) {
    if constexpr (V == 8) {
        const uint4 w = *(const uint4*)p;
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) v[2 * i] = bf16_lo(u[i]), v[2 * i + 1] = bf16_hi(u[i]);
    } else {
        v[0] = bf16_to_f32(*p);
    }
}

template <int V>
__device__ __forceinline__ void store_bf16(uint16_t* p, const float (&v)[V]) {
    if constexpr (V == 8) {
        *(uint4*)p = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
    } else {
        *p = (uint16_t)pack_bf16(v[0], v[0]);
    }
}

template <typename X, int V>
__device__ __forceinline__ void load_x(const X* p, float (&v)[V]) {
    if constexpr (sizeof(X) == 2) {
        load_bf16<V>((const uint16_t*)p, v);
    } else if constexpr (V == 8) {
        const float4 a = ((const float4*)p)[0], b = ((const float4*)p)[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
        v[0] = *p;
    }
}

// Reduction over the W warps of a row (slot: this row's place in shared memory).
template <bool kMax>
__device__ __forceinline__ float row_reduce(float v, int W, float* slot, int warp_in_row, int lane) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const float o = __shfl_xor_sync(QMOE_FULL_MASK, v, d);
        v = kMax ? max_nan(v, o) : v + o;
    }
    if (W == 1) return v;
    if (lane == 0) slot[warp_in_row] = v;
    __syncthreads();
    v = slot[lane & (W - 1)];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        if (d < W) {
            const float o = __shfl_xor_sync(QMOE_FULL_MASK, v, d);
            v = kMax ? max_nan(v, o) : v + o;
        }
    }
    return v;
}

// 8 codes of y / s.  A reciprocal is within a step of the quotient's last place, before a rounding to 4 bits; it
// overflows for scales near fp32's smallest, which divide.
template <int V>
__device__ __forceinline__ void store_codes(uint8_t* dst, const float (&y)[V], float s) {
    static_assert(V == 8, "codes are written eight at a time");
    float q[V];
    if (s >= 1e-37f) {
        const float inv = 1.f / s;
#pragma unroll
        for (int j = 0; j < V; ++j) q[j] = y[j] * inv;
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) q[j] = s > 0.f ? __fdiv_rn(y[j], s) : 0.f;      // (a NaN scale: codes 0)
    }
    uint32_t w[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
        w[j] = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(q[4 * j], q[4 * j + 1]), __NV_SATFINITE, __NV_E4M3) |
               (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(q[4 * j + 2], q[4 * j + 3]), __NV_SATFINITE, __NV_E4M3) << 16;
    *(uint2*)dst = make_uint2(w[0], w[1]);
}

// V values a lane and step (8: 16-byte accesses; 1: any width, stride and alignment), K steps, W warps a row.
template <typename X, int V, int K>
__global__ void __launch_bounds__(V == 8 ? 1024 : 1024) norm_kernel(NormArgs a, int W) {
    __shared__ float sum_s[32], max_s[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, in_row = warp & (W - 1), first = warp - in_row;
    const int rows = (blockDim.x >> 5) / W;
    const int64_t t = (int64_t)blockIdx.x * rows + warp / W;
    const bool on = t < a.T;
    const int c0 = in_row * 32 + lane, step = W * 32, chunks = on ? a.n / V : 0;
    const X* x = (const X*)a.x + t * a.x_stride;
    float h[K][V];
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
        for (int j = 0; j < V; ++j) h[k][j] = 0.f;
        if (c0 + k * step < chunks) load_x<X, V>(x + (int64_t)(c0 + k * step) * V, h[k]);
    }
    if (a.residual) {
        const uint16_t* r = a.residual + t * a.res_stride;
        uint16_t* ro = a.residual_out + t * a.res_out_stride;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (c0 + k * step < chunks) {
                float v[V];
                load_bf16<V>(r + (int64_t)(c0 + k * step) * V, v);
#pragma unroll
                for (int j = 0; j < V; ++j) h[k][j] += v[j];
                store_bf16<V>(ro + (int64_t)(c0 + k * step) * V, h[k]);
            }
    }
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) ss = fmaf(h[k][j], h[k][j], ss);
    ss = row_reduce<false>(ss, W, sum_s + first, in_row, lane);
    const float r = rsqrtf(ss / (float)a.n + a.eps);
    float big = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = c0 + k * step;
        if (c < chunks) {
            float w[V];
            if (a.weight) load_bf16<V>(a.weight + (int64_t)c * V, w);
#pragma unroll
            for (int j = 0; j < V; ++j) h[k][j] = h[k][j] * r * (a.weight ? w[j] : 1.f);
            if (a.y) store_bf16<V>(a.y + t * a.y_stride + (int64_t)c * V, h[k]);
        }
        if constexpr (V == 8) {
            if (a.codes) {
                float m = 0.f;
#pragma unroll
                for (int j = 0; j < V; ++j) m = max_nan(m, fabsf(h[k][j]));
                if (a.row_scale) {
                    big = max_nan(big, m);
                } else {       // 16 lanes hold 128 values
#pragma unroll
                    for (int d = 8; d > 0; d >>= 1) m = max_nan(m, __shfl_xor_sync(QMOE_FULL_MASK, m, d));
                    if (c < chunks) {
                        const float s = __fdiv_rn(m, 448.f);
                        if ((lane & 15) == 0) a.scales[t * ((a.n + 127) >> 7) + (c >> 4)] = s;
                        store_codes<V>(a.codes + t * a.n + (int64_t)c * V, h[k], s);
                    }
                }
            }
        }
    }
    if constexpr (V == 8) {
        if (a.codes && a.row_scale) {
            big = row_reduce<true>(big, W, max_s + first, in_row, lane);
            const float s = __fdiv_rn(big, 448.f);
            if (on && c0 == 0) a.scales[t] = s;
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (c0 + k * step < chunks) store_codes<V>(a.codes + t * a.n + (int64_t)(c0 + k * step) * V, h[k], s);
        }
    }
}

constexpr int kNormMaxWidth = 32768;

template <typename X, int V>
int launch_norm(const NormArgs& a, cudaStream_t st) {
    const int chunks = (a.n + V - 1) / V;
    constexpr int kMost = V == 8 ? 4 : 32;      // steps that a thread's registers hold
    // many rows: a few steps a thread; few rows: as many threads as a row has chunks
    int W = 1;
    while (W < 32 && W * 32 * (V == 8 ? 2 : 8) < chunks) W *= 2;
    if (a.T < 2 * qmoe::sm_count())
        while (W < 32 && W * 32 < chunks) W *= 2;
    const int need = (chunks + 32 * W - 1) / (32 * W), rows = std::max(1, 8 / W);
    const unsigned blocks = (unsigned)((a.T + rows - 1) / rows);
    const int threads = rows * W * 32;
    if constexpr (V == 8) {
        if (need <= 1) norm_kernel<X, V, 1><<<blocks, threads, 0, st>>>(a, W);
        else if (need <= 2) norm_kernel<X, V, 2><<<blocks, threads, 0, st>>>(a, W);
        else norm_kernel<X, V, kMost><<<blocks, threads, 0, st>>>(a, W);
    } else {
        if (need <= 8) norm_kernel<X, V, 8><<<blocks, threads, 0, st>>>(a, W);
        else norm_kernel<X, V, kMost><<<blocks, threads, 0, st>>>(a, W);
    }
    return qmoe::launch_check("add_rms_norm");
}

// ---------------------------------------------------------------- choice of experts
//
// Scores s = softmax(l) or 1 / (1 + e^-l); an expert's value c = s + bias; a group's value the sum of its best one or two
// c; the k best experts by c of the best groups; gates s, or s over the sum of the chosen, times a factor.
//
// The order is that of the values in 64 bits, equal ones to the lower index.  Without a bias an expert's order is its
// logit's, exactly.  Else the values are made in fp32 with a bound on their error, and a row in which two neighbours in
// the order are nearer than their bounds (and are not the same logit with the same bias) is decided again in fp64.
//
// A lane holds R neighbouring experts, so that among lanes with equal values the lowest has the lowest index: a round of
// the choice is a reduction of the lanes' best keys (one instruction) and a ballot.  A warp takes a token; above 1024 experts a
// block of 8 warps does, each warp's best k + 1 being merged by the first.
struct RouteArgs {
    const void* logits;
    const float* bias;
    int32_t* ids;
    float* gates;
    int64_t stride;
    int T, E, k, sigmoid, groups, top_groups, best, renorm;
    float scale;
};

constexpr int kRouteWarps = 8;
constexpr float kUlp = 5.9604645e-8f;       // 2^-24
constexpr float kLargest = 3.402823466e38f;

// fp32 -> integer of the same order (NaN is read as -infinity, -0 as 0); 0 stands for no value.
__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t u = __float_as_uint(v + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}
__device__ __forceinline__ unsigned long long key_of(double v) {
    const unsigned long long u = (unsigned long long)__double_as_longlong(v + 0.0);
    return u >> 63 ? ~u : u | 0x8000000000000000ull;
}

// A logit as it is read: NaN as -infinity, +infinity as the largest finite value.
template <typename X>
__device__ __forceinline__ float logit(const X* row, int e) {
    const float v = sizeof(X) == 2 ? bf16_to_f32(((const uint16_t*)row)[e]) : ((const float*)row)[e];
    return v == v ? fminf(v, kLargest) : -INFINITY;
}

// A value of the choice: NaN (an infinite bias of the other sign) as -infinity.
__device__ __forceinline__ float plain_value(float c) { return c == c ? c : -INFINITY; }

struct Pair {
    float a, b;      // the best and the second best
};
__device__ __forceinline__ Pair merge(Pair x, Pair y) {
    return Pair{fmaxf(x.a, y.a), fmaxf(fminf(x.a, y.a), fmaxf(x.b, y.b))};
}

// Which groups are kept (bit g of the result), from values that lane g holds for g < groups.
template <typename F>
__device__ __forceinline__ uint32_t best_groups(F v, int groups, int top, int lane) {
    int rank = 0;
    for (int g = 0; g < groups; ++g) {
        const F o = __shfl_sync(QMOE_FULL_MASK, v, g);
        rank += o > v || (o == v && g < lane);
    }
    return __ballot_sync(QMOE_FULL_MASK, lane < groups && rank < top);
}

__device__ __forceinline__ unsigned long long warp_max64(unsigned long long v) {
    const uint32_t hi = __reduce_max_sync(QMOE_FULL_MASK, (uint32_t)(v >> 32));
    const uint32_t lo = __reduce_max_sync(QMOE_FULL_MASK, (uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
    return (unsigned long long)hi << 32 | lo;
}

__device__ __forceinline__ double warp_sum_d(double v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(QMOE_FULL_MASK, v, d);
    return v;
}

struct ResolveShared {
    double sum[kRouteWarps];
    unsigned long long key[kRouteWarps];
};

// The choice in 64 bits, by NW warps: lane j of the first gets the j-th expert.  `cand`: bit i is set where expert e0 + i may be
// among the chosen (all of them where the groups are to be decided too).
template <typename X, int NW>
__device__ __noinline__ int resolve(const RouteArgs& a, const X* row, int e0, int R, float top, uint32_t cand, bool groups_too,
                                    ResolveShared* sh) {
    const int lane = threadIdx.x & 31, warp = NW == 1 ? 0 : threadIdx.x >> 5;
    double c[32], z = 1.0;
    if (!a.sigmoid) {
        double mine = 0.0;
        for (int i = 0; i < R; ++i) {
            const float l = e0 + i < a.E ? logit(row, e0 + i) : -INFINITY;
            if (l > -INFINITY) mine += exp((double)l - (double)top);
        }
        z = warp_sum_d(mine);
        if (NW > 1) {
            if (lane == 0) sh->sum[warp] = z;
            __syncthreads();
            z = 0.0;
            for (int w = 0; w < NW; ++w) z += sh->sum[w];
        }
    }
    for (int i = 0; i < R; ++i) {
        c[i] = -INFINITY;
        if (!((cand >> i) & 1)) continue;
        const double l = logit(row, e0 + i);
        double s = 0.0;
        if (l > -INFINITY) s = a.sigmoid ? 1.0 / (1.0 + exp(-l)) : exp(l - (double)top) / z;
        if (a.bias) s += (double)a.bias[e0 + i];
        c[i] = s == s ? s : -INFINITY;
    }
    if (groups_too) {
        const int size = a.E / a.groups;
        double mine = 0.0;
        for (int g = 0; g < a.groups; ++g) {
            double b0 = -INFINITY, b1 = -INFINITY;
            for (int i = 0; i < R; ++i) {
                const int e = e0 + i;
                if (e < g * size || e >= (g + 1) * size) continue;
                b1 = fmax(b1, fmin(b0, c[i]));
                b0 = fmax(b0, c[i]);
            }
            for (int d = 16; d > 0; d >>= 1) {
                const double o0 = __shfl_xor_sync(QMOE_FULL_MASK, b0, d), o1 = __shfl_xor_sync(QMOE_FULL_MASK, b1, d);
                b1 = fmax(fmin(b0, o0), fmax(b1, o1));
                b0 = fmax(b0, o0);
            }
            double v = a.best == 2 ? b0 + b1 : b0;
            if (v != v) v = -INFINITY;
            if (lane == g) mine = v;
        }
        const uint32_t kept = best_groups(mine, a.groups, a.top_groups, lane);
        for (int i = 0; i < R; ++i)
            if (e0 + i < a.E && !((kept >> ((e0 + i) / size)) & 1)) cand &= ~(1u << i);
    }
    // (without a bias the order is the logits'; sums of scores have decided the groups)
    if (!a.bias)
        for (int i = 0; i < R; ++i)
            if ((cand >> i) & 1) c[i] = logit(row, e0 + i);
    int got = 0;
    for (int j = 0; j < a.k; ++j) {
        unsigned long long best = 0;
        int at = 0;
        for (int i = 0; i < R; ++i)
            if ((cand >> i) & 1) {
                const unsigned long long key = key_of(c[i]);
                if (key > best) best = key, at = i;
            }
        unsigned long long m = warp_max64(best);
        bool here = true;
        if (NW > 1) {
            __syncthreads();
            if (lane == 0) sh->key[warp] = m;
            __syncthreads();
            const unsigned long long own = m;
            int from = 0;
            m = sh->key[0];
            for (int w = 1; w < NW; ++w)
                if (sh->key[w] > m) m = sh->key[w], from = w;
            here = from == warp && own == m;
        }
        const unsigned who = __ballot_sync(QMOE_FULL_MASK, here && best == m && m != 0);
        int e = 0;
        if (who) {
            const int w = __ffs(who) - 1;
            e = __shfl_sync(QMOE_FULL_MASK, e0 + at, w);
            if (lane == w) cand &= ~(1u << at);
        }
        if (NW > 1) {
            __syncthreads();
            if (lane == 0 && who) sh->key[0] = (unsigned long long)e;
            __syncthreads();
            e = (int)sh->key[0];
        }
        if (lane == j) got = e;
    }
    return got;
}

// The k + 1 best of the values that the lanes hold (R each, keys; 0: none): lane j gets the j-th one's key and tag, and
// the last round's go to every lane.  Keys are taken out of `key`.
template <int R>
__device__ __forceinline__ void choose(uint32_t (&key)[R], int rounds, int lane, uint32_t* my_key, int* my_at) {
    uint32_t best = 0;
    int at = 0;
#pragma unroll
    for (int i = 0; i < R; ++i)
        if (key[i] > best) best = key[i], at = i;
    *my_key = 0, *my_at = -1;
    for (int j = 0; j < rounds; ++j) {
        const uint32_t m = __reduce_max_sync(QMOE_FULL_MASK, best);
        const int w = __ffs(__ballot_sync(QMOE_FULL_MASK, best == m)) - 1;
        const int tag = __shfl_sync(QMOE_FULL_MASK, lane * R + at, w);
        if (lane == j) *my_key = m, *my_at = m ? tag : -1;
        if (lane == w) {
            best = 0;
            const int gone = at;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                if (i == gone) key[i] = 0;
                if (key[i] > best) best = key[i], at = i;
            }
        }
    }
}

// Gates of the experts that lanes 0 .. k - 1 hold, and the outputs of token t.  Renormalised weights are taken relative to the
// largest, so that scores below fp32's range keep their ratios.
template <typename X>
__device__ __forceinline__ void write_route(const RouteArgs& a, const X* row, int64_t t, int id, float top, float z, int lane) {
    const bool on = lane < a.k;
    const float l = on ? logit(row, id) : -INFINITY;
    float g = 0.f;
    if (a.renorm) {
        float big = l;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) big = fmaxf(big, __shfl_xor_sync(QMOE_FULL_MASK, big, d));
        if (l > -INFINITY) {
            if (!a.sigmoid)
                g = expf(l - big);
            else if (l >= 0.f)
                g = 1.f / (1.f + expf(-l));
            else
                g = expf(l - fminf(big, 0.f)) / (1.f + expf(l));
        }
        const float sum = warp_sum(g);
        g = sum > 0.f ? g / sum : 0.f;
    } else if (l > -INFINITY) {
        g = a.sigmoid ? (l >= 0.f ? 1.f / (1.f + expf(-l)) : expf(l) / (1.f + expf(l))) : expf(l - top) / z;
    }
    if (on) {
        a.ids[t * a.k + lane] = id;
        a.gates[t * a.k + lane] = g * a.scale;
    }
}

// R experts a lane; NW warps a token (1: kRouteWarps tokens a block).
template <typename X, int R, int NW>
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(RouteArgs a) {
    __shared__ ResolveShared rs;
    __shared__ float2 part_s[kRouteWarps];
    __shared__ uint32_t key_s[NW > 1 ? kRouteWarps * 32 : 1];
    __shared__ int id_s[NW > 1 ? kRouteWarps * 32 : 1];
    __shared__ float2 bound_s;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = NW == 1 ? (int64_t)blockIdx.x * kRouteWarps + warp : blockIdx.x;
    if (t >= a.T) return;
    const X* row = (const X*)a.logits + t * a.stride;
    const int e0 = (NW == 1 ? lane : (int)threadIdx.x) * R;
    float l[R];
#pragma unroll
    for (int i = 0; i < R; ++i) l[i] = e0 + i < a.E ? logit(row, e0 + i) : -INFINITY;
    // ---- softmax: largest logit and sum of exponentials
    float top = 0.f, z = 1.f;
    if (!a.sigmoid) {
        top = l[0];
#pragma unroll
        for (int i = 1; i < R; ++i) top = fmaxf(top, l[i]);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(QMOE_FULL_MASK, top, d));
        const float m = top > -INFINITY ? top : 0.f;
        z = 0.f;
#pragma unroll
        for (int i = 0; i < R; ++i) z += expf(l[i] - m);
        z = warp_sum(z);
        if (NW > 1) {
            if (lane == 0) part_s[warp] = make_float2(top, z);
            __syncthreads();
            const float2 p = part_s[lane & (NW - 1)];
            top = p.x;
#pragma unroll
            for (int d = NW / 2; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(QMOE_FULL_MASK, top, d));
            z = p.x > -INFINITY ? p.y * expf(p.x - top) : 0.f;
#pragma unroll
            for (int d = NW / 2; d > 0; d >>= 1) z += __shfl_xor_sync(QMOE_FULL_MASK, z, d);
        }
        if (!(top > -INFINITY)) top = 0.f, z = 1.f;      // nothing in the row: scores 0
    }
    // ---- values, and the bound on their error besides the last addition's: a score has at most (|x| + 3) 2^-24 of itself
    // from its exponential (x = l - top), the sum that and an addition's for each term; a sigmoid score 6 2^-24
    const bool by_logit = !a.bias;
    float c[R];
    const float slack = by_logit ? 0.f : fmaf(a.sigmoid ? 6.f : (float)(2 * R + 48) / z, kUlp, 1e-37f);
#pragma unroll
    for (int i = 0; i < R; ++i) {
        c[i] = l[i];
        if (!by_logit || (a.groups > 1 && a.best == 2)) {
            float s = a.sigmoid ? 1.f / (1.f + expf(-l[i])) : expf(l[i] - top) / z;
            if (a.bias) s = plain_value(s + (e0 + i < a.E ? a.bias[e0 + i] : 0.f));
            c[i] = s;
        }
    }
    bool again = false, groups_too = false;
    uint32_t in = 0;      // experts that may be chosen
#pragma unroll
    for (int i = 0; i < R; ++i) in |= e0 + i < a.E ? 1u << i : 0u;
    const uint32_t all = in;
    if constexpr (NW == 1) {
        if (a.groups > 1) {
            // ---- groups
            const int size = a.E / a.groups, lanes = size / R;
            Pair mine{-INFINITY, -INFINITY};
            if (size % R == 0 && (lanes & (lanes - 1)) == 0) {
                // a group is a power of two of whole lanes
                Pair p{-INFINITY, -INFINITY};
#pragma unroll
                for (int i = 0; i < R; ++i) p = merge(p, Pair{(all >> i) & 1 ? c[i] : -INFINITY, -INFINITY});
#pragma unroll
                for (int d = 1; d < 32; d <<= 1)
                    if (d < lanes) p = merge(p, Pair{__shfl_xor_sync(QMOE_FULL_MASK, p.a, d), __shfl_xor_sync(QMOE_FULL_MASK, p.b, d)});
                mine = Pair{__shfl_sync(QMOE_FULL_MASK, p.a, lane * lanes & 31), __shfl_sync(QMOE_FULL_MASK, p.b, lane * lanes & 31)};
            } else {
                for (int g = 0; g < a.groups; ++g) {
                    Pair p{-INFINITY, -INFINITY};
#pragma unroll
                    for (int i = 0; i < R; ++i)
                        if (e0 + i >= g * size && e0 + i < (g + 1) * size) p = merge(p, Pair{c[i], -INFINITY});
#pragma unroll
                    for (int d = 16; d > 0; d >>= 1) p = merge(p, Pair{__shfl_xor_sync(QMOE_FULL_MASK, p.a, d), __shfl_xor_sync(QMOE_FULL_MASK, p.b, d)});
                    if (lane == g) mine = p;
                }
            }
            const float v = plain_value(a.best == 2 ? mine.a + mine.b : mine.a);
            const uint32_t kept = best_groups(v, a.groups, a.top_groups, lane);
            if (!(by_logit && a.best == 1) && a.top_groups < a.groups) {
                // the last one kept and the best one dropped
                const float one = fmaf(a.sigmoid ? 6.f : (float)(2 * R + 48) / z, kUlp, 1e-37f);
                const float mag = fabsf(mine.a) + fabsf(mine.b);
                const float err = 2.f * one + (mag < kLargest ? 2.f * kUlp * mag : 0.f);
                const bool is = (kept >> lane) & 1;
                const float low = value_of(~__reduce_max_sync(QMOE_FULL_MASK, is ? ~key_of(v) : 0u));
                const uint32_t hk = __reduce_max_sync(QMOE_FULL_MASK, lane < a.groups && !is ? key_of(v) : 0u);
                const float gap = low - value_of(hk);
                const float err_all = __uint_as_float(__reduce_max_sync(QMOE_FULL_MASK, lane < a.groups ? __float_as_uint(err) : 0u));
                // (two groups of nothing but -infinity: a NaN, decided by the index as in 64 bits)
                again = groups_too = gap <= 2.f * err_all;
            }
#pragma unroll
            for (int i = 0; i < R; ++i)
                if (((all >> i) & 1) && !((kept >> ((e0 + i) / size)) & 1)) in &= ~(1u << i);
        }
    }
    // ---- the k best, and the next one
    uint32_t key[R];
#pragma unroll
    for (int i = 0; i < R; ++i) key[i] = (in >> i) & 1 ? key_of(by_logit ? l[i] : c[i]) : 0u;
    const int rounds = min(a.k + (by_logit ? 0 : 1), 32);
    uint32_t mk;
    int at;
    choose<R>(key, rounds, lane, &mk, &at);
    if constexpr (NW > 1) {
        key_s[warp * 32 + lane] = lane < rounds ? mk : 0u;
        id_s[warp * 32 + lane] = lane < rounds && mk ? warp * 32 * R + at : 0;
        __syncthreads();
        if (warp == 0) {
            // the warps' lists one behind the other, kRouteWarps of them a lane's worth at a time: lower lanes hold lower experts
            // among equal keys
            uint32_t mkeys[kRouteWarps];
#pragma unroll
            for (int i = 0; i < kRouteWarps; ++i) mkeys[i] = key_s[lane * kRouteWarps + i];
            choose<kRouteWarps>(mkeys, rounds, lane, &mk, &at);
            at = mk ? id_s[at] : -1;
        }
    }
    if (!by_logit && (NW == 1 || warp == 0)) {
        // ---- neighbours that are too near to tell (with k = 32 the 33rd is not known: then the last gap counts as too small)
        const uint32_t nk = __shfl_down_sync(QMOE_FULL_MASK, mk, 1);
        const int nat = __shfl_down_sync(QMOE_FULL_MASK, at, 1);
        bool near = false;
        if (lane < a.k && mk) {
            if (lane == 31) {
                near = a.k < a.E;
            } else if (nk) {
                const float v = value_of(mk), nv = value_of(nk);
                const float err = 2.f * slack + kUlp * (fabsf(v) + fabsf(nv));
                if (v > -INFINITY && v < INFINITY && nv > -INFINITY)
                    near = v - nv <= err;
                else
                    near = v == nv;
                if (near) near = !(logit(row, at) == logit(row, nat) && a.bias[at] == a.bias[nat]);
            }
        }
        again |= __any_sync(QMOE_FULL_MASK, near);
    }
    if constexpr (NW == 1) {
        if (__builtin_expect(again, 0)) {
            // what may be among the chosen: values down to the k-th's less the errors
            const float last = value_of(__shfl_sync(QMOE_FULL_MASK, mk, a.k - 1));
            uint32_t cand = groups_too ? all : 0u;
            if (!groups_too) {
#pragma unroll
                for (int i = 0; i < R; ++i)
                    if (((in >> i) & 1) && !(c[i] < last - (2.f * slack + 2.f * kUlp * fmaxf(fabsf(last), fabsf(c[i]))))) cand |= 1u << i;
            }
            at = resolve<X, 1>(a, row, e0, R, top, cand, groups_too, &rs);
        }
        write_route<X>(a, row, t, at < 0 ? 0 : at, top, z, lane);
    } else {
        if (!by_logit) {
            if (warp == 0) {
                const float last = value_of(__shfl_sync(QMOE_FULL_MASK, mk, a.k - 1));
                if (lane == 0) bound_s = make_float2(again ? 1.f : 0.f, last);
            }
            __syncthreads();
            if (__builtin_expect(bound_s.x != 0.f, 0)) {
                const float last = bound_s.y;
                uint32_t cand = 0u;
#pragma unroll
                for (int i = 0; i < R; ++i)
                    if (((in >> i) & 1) && !(c[i] < last - (2.f * slack + 2.f * kUlp * fmaxf(fabsf(last), fabsf(c[i]))))) cand |= 1u << i;
                at = resolve<X, NW>(a, row, e0, R, top, cand, false, &rs);
            }
        }
        if (warp == 0) write_route<X>(a, row, t, at < 0 ? 0 : at, top, z, lane);
    }
}

template <typename X>
int launch_route(const RouteArgs& a, cudaStream_t st) {
    const unsigned per_warp = (unsigned)((a.T + kRouteWarps - 1) / kRouteWarps);
    constexpr int threads = kRouteWarps * 32;
    if (a.E <= 32) route_kernel<X, 1, 1><<<per_warp, threads, 0, st>>>(a);
    else if (a.E <= 64) route_kernel<X, 2, 1><<<per_warp, threads, 0, st>>>(a);
    else if (a.E <= 128) route_kernel<X, 4, 1><<<per_warp, threads, 0, st>>>(a);
    else if (a.E <= 256) route_kernel<X, 8, 1><<<per_warp, threads, 0, st>>>(a);
    else if (a.E <= 512) route_kernel<X, 16, 1><<<per_warp, threads, 0, st>>>(a);
    else if (a.E <= 1024) route_kernel<X, 32, 1><<<per_warp, threads, 0, st>>>(a);
    else if (a.E <= 2048) route_kernel<X, 8, kRouteWarps><<<(unsigned)a.T, threads, 0, st>>>(a);
    else if (a.E <= 4096) route_kernel<X, 16, kRouteWarps><<<(unsigned)a.T, threads, 0, st>>>(a);
    else route_kernel<X, 32, kRouteWarps><<<(unsigned)a.T, threads, 0, st>>>(a);
    return qmoe::launch_check("qmoe_route_scored");
}

inline bool aligned(const void* p, int bytes) { return ((uintptr_t)p & (uintptr_t)(bytes - 1)) == 0; }

}  // namespace

extern "C" int add_rms_norm(const void* x, int x_is_f32, int64_t x_stride, const void* residual, int64_t residual_stride,
                            void* residual_out, int64_t residual_out_stride, const void* weight, int T, int n, float eps, void* y,
                            int64_t y_stride, void* codes, float* scales, int scale_group, void* stream) {
    qmoe::clear_error();
    if (T < 0 || n < 1 || n > kNormMaxWidth)
        return qmoe::fail(QMOE_EINVAL, "add_rms_norm: need T >= 0 and a row width of 1 .. 32768");
    if (!(eps >= 1.17549435e-38f) || !(eps < kLargest)) return qmoe::fail(QMOE_EINVAL, "add_rms_norm: eps must be positive and finite");
    if (!residual != !residual_out) return qmoe::fail(QMOE_EINVAL, "add_rms_norm: residual and residual_out go together");
    if (!codes != !scales) return qmoe::fail(QMOE_EINVAL, "add_rms_norm: codes and scales go together");
    if (codes && scale_group != 0 && scale_group != 128)
        return qmoe::fail(QMOE_EUNSUPPORTED, "add_rms_norm: scale_group must be 0 (a scale a row) or 128");
    if (T == 0) return QMOE_OK;
    if (!x || (!y && !codes)) return qmoe::fail(QMOE_EINVAL, "add_rms_norm: NULL pointer");
    if (T > 1 && (x_stride < n || (residual && (residual_stride < n || residual_out_stride < n)) || (y && y_stride < n)))
        return qmoe::fail(QMOE_EINVAL, "add_rms_norm: a row stride is smaller than the row");
    const int64_t strides = x_stride | (residual ? residual_stride | residual_out_stride : 0) | (y ? y_stride : 0);
    const bool wide = n % 8 == 0 && (T == 1 || strides % 8 == 0) && aligned(x, 16) && aligned(residual, 16) && aligned(residual_out, 16) &&
                      aligned(weight, 16) && aligned(y, 16);
    if (!aligned(x, x_is_f32 ? 4 : 2) || !aligned(residual, 2) || !aligned(residual_out, 2) || !aligned(weight, 2) || !aligned(y, 2) ||
        !aligned(scales, 4))
        return qmoe::fail(QMOE_EINVAL, "add_rms_norm: pointer not aligned to its type");
    if (codes && (!wide || !aligned(codes, 8)))
        return qmoe::fail(QMOE_EUNSUPPORTED, "add_rms_norm: codes need a row width and strides that are multiples of 8 and 16-byte aligned pointers");
    NormArgs a{x, (const uint16_t*)residual, (uint16_t*)residual_out, (const uint16_t*)weight, (uint16_t*)y, (uint8_t*)codes, scales,
               x_stride, residual_stride, residual_out_stride, y_stride, T, n, scale_group == 0, eps};
    cudaStream_t st = (cudaStream_t)stream;
    if (wide) return x_is_f32 ? launch_norm<float, 8>(a, st) : launch_norm<uint16_t, 8>(a, st);
    return x_is_f32 ? launch_norm<float, 1>(a, st) : launch_norm<uint16_t, 1>(a, st);
}

extern "C" int qmoe_route_scored(const void* logits, int logits_are_f32, int64_t row_stride, int T, int E, int k, int score,
                                 const float* bias, int n_groups, int top_groups, int group_best, int renormalise, float scale,
                                 int32_t* ids, float* gates, void* stream) {
    qmoe::clear_error();
    if (T < 0 || k < 1 || k > E || k > 32 || E > 8192)
        return qmoe::fail(QMOE_EINVAL, "qmoe_route_scored: need 1 <= k <= min(E, 32), E <= 8192, T >= 0");
    if (score != QMOE_SCORE_SOFTMAX && score != QMOE_SCORE_SIGMOID)
        return qmoe::fail(QMOE_EINVAL, "qmoe_route_scored: unknown score function");
    if (n_groups < 1 || n_groups > 32 || E % n_groups || top_groups < 1 || top_groups > n_groups)
        return qmoe::fail(QMOE_EINVAL, "qmoe_route_scored: need 1 <= top_groups <= n_groups <= 32 and E a multiple of n_groups");
    if ((group_best != 1 && group_best != 2) || (n_groups > 1 && group_best > E / n_groups))
        return qmoe::fail(QMOE_EINVAL, "qmoe_route_scored: group_best must be 1 or 2 and at most a group's experts");
    if (n_groups > 1 && (int64_t)top_groups * (E / n_groups) < k)
        return qmoe::fail(QMOE_EINVAL, "qmoe_route_scored: the kept groups have fewer than k experts");
    if (n_groups > 1 && E > 1024) return qmoe::fail(QMOE_EUNSUPPORTED, "qmoe_route_scored: groups need E <= 1024");
    if (!(scale > -kLargest && scale < kLargest)) return qmoe::fail(QMOE_EINVAL, "qmoe_route_scored: scale must be finite");
    if (T == 0) return QMOE_OK;
    if (!logits || !ids || !gates) return qmoe::fail(QMOE_EINVAL, "qmoe_route_scored: NULL pointer");
    if (T > 1 && row_stride < E) return qmoe::fail(QMOE_EINVAL, "qmoe_route_scored: the row stride is smaller than a row");
    if (!aligned(logits, logits_are_f32 ? 4 : 2) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(gates, 4))
        return qmoe::fail(QMOE_EINVAL, "qmoe_route_scored: pointer not aligned to its type");
    RouteArgs a{logits, bias, ids, gates, row_stride, T, E, k, score == QMOE_SCORE_SIGMOID, n_groups, top_groups, group_best,
                renormalise ? 1 : 0, scale};
    return logits_are_f32 ? launch_route<float>(a, (cudaStream_t)stream) : launch_route<uint16_t>(a, (cudaStream_t)stream);
}
