// What a decoder layer needs between its attention and its experts: the norm of whole rows with the
// residual's addition, and the choice of experts from scores with a bias and groups.

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "device_common.cuh"

namespace {

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *(uint32_t*)&p;
}

// Launches a kernel that waits for its predecessor itself.  Beginning before that has ended takes 2 us off calls in a row (4095 rows of
// 2080: 20.5 -> 18.0 us, 16383 tokens' routes 20.5 -> 16.8); the host pays 1 us for it, which with few rows is what bounds such calls (32
// rows 6.6 us plainly, 7.5 so).
template <typename... Args>
int launch_rows(void (*kernel)(Args...), int T, unsigned blocks, int threads, cudaStream_t st, const char* who, typename qmoe::Same<Args>::type... args) {
    if (T >= qmoe::sm_count()) return qmoe::launch_dependent(kernel, dim3(blocks), threads, 0, st, who, args...);
    kernel<<<blocks, threads, 0, st>>>(args...);
    return qmoe::launch_check(who);
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
    int x_stride, res_stride, res_out_stride, y_stride;
    int T, n;
    int row_scale;     // one scale a row (0: one for each 128 values)
    float eps;
};

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// A lane's values of a step: eight (16-byte accesses), or one (any width, stride and alignment).  (Packed pairs of fp32 take more
// instructions here, for the moves that line them up: 30.7 against 25.4 million for 16384 rows of 2048.)
template <int V>
struct Values {
    float v[V];
    __device__ __forceinline__ void add(const Values& o) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] += o.v[i];
    }
    __device__ __forceinline__ void times(const Values& o) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] *= o.v[i];
    }
    __device__ __forceinline__ void times(float f) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] *= f;
    }
    __device__ __forceinline__ float squares(float sum) const {
#pragma unroll
        for (int i = 0; i < V; ++i) sum = fmaf(v[i], v[i], sum);
        return sum;
    }
};

// The same as they are loaded.
template <typename X, int V>
struct Raw {
    uint32_t w[V * sizeof(X) / 4];
    __device__ __forceinline__ void load(const X* p) {
#pragma unroll
        for (int i = 0; i < (int)(V * sizeof(X) / 16); ++i) {
            const uint4 x = ((const uint4*)p)[i];
            w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
        }
    }
    __device__ __forceinline__ Values<V> values() const {
        Values<V> r;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if constexpr (sizeof(X) == 4) r.v[i] = __uint_as_float(w[i]);
            else r.v[i] = i & 1 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
        }
        return r;
    }
};
template <typename X>
struct Raw<X, 1> {
    X w;
    __device__ __forceinline__ void load(const X* p) { w = *p; }
    __device__ __forceinline__ Values<1> values() const {
        if constexpr (sizeof(X) == 4) return Values<1>{{w}};
        else return Values<1>{{bf16_to_f32(w)}};
    }
};

template <int V>
__device__ __forceinline__ void store_bf16(uint16_t* p, const Values<V>& v) {
    if constexpr (V == 8)
        *(uint4*)p = make_uint4(pack_bf16(v.v[0], v.v[1]), pack_bf16(v.v[2], v.v[3]), pack_bf16(v.v[4], v.v[5]), pack_bf16(v.v[6], v.v[7]));
    else
        *p = (uint16_t)pack_bf16(v.v[0], 0.f);
}

// Sum and largest of a row's values, over its W warps (slot: this row's places in shared memory).
template <bool kMax>
__device__ __forceinline__ float2 row_reduce(float sum, float big, int W, float2* slot, int warp_in_row, int lane) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        sum += __shfl_xor_sync(QMOE_FULL_MASK, sum, d);
        if (kMax) big = max_nan(big, __shfl_xor_sync(QMOE_FULL_MASK, big, d));
    }
    if (W == 1) return make_float2(sum, big);
    if (lane == 0) slot[warp_in_row] = make_float2(sum, big);
    __syncthreads();
    if (W <= 8) {
        float2 all = slot[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) {
            if (i >= W) break;
            const float2 o = slot[i];
            all.x += o.x;
            if (kMax) all.y = max_nan(all.y, o.y);
        }
        return all;
    }
    float2 all = lane < W ? slot[lane] : make_float2(0.f, 0.f);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        all.x += __shfl_xor_sync(QMOE_FULL_MASK, all.x, d);
        if (kMax) all.y = max_nan(all.y, __shfl_xor_sync(QMOE_FULL_MASK, all.y, d));
    }
    return all;
}

__device__ __forceinline__ float largest(const Values<8>& v) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max_nan(m, fabsf(v.v[i]));
    return m;
}

// 8 codes of v / s for s = m / 448, m = max |v| > 0.  448 / m is in two floats, as an error of it would move all the run's codes next to
// the middle of two values.  Where m is far from 1 a power of two brings the values near it first.
__device__ __forceinline__ void store_codes(uint8_t* dst, Values<8> v, float m) {
    if (__builtin_expect(!(m > 1e-30f && m < 1e30f), 0)) {
        const float g = __int_as_float(max((254 << 23) - (int)(__float_as_uint(m) & 0x7F800000u), 1 << 23));
        v.times(g), m *= g;
    }
    const float inv = __fdividef(448.f, m), rest = fmaf(-inv, m, 448.f) * inv * (1.f / 448.f);
    auto quotient = [&](float x) { return fmaf(x, inv, x * rest); };
    uint32_t w[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const float* x = v.v + 4 * j;
        w[j] = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(quotient(x[0]), quotient(x[1])), __NV_SATFINITE, __NV_E4M3) |
               (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(quotient(x[2]), quotient(x[3])), __NV_SATFINITE, __NV_E4M3) << 16;
    }
    *(uint2*)dst = make_uint2(w[0], w[1]);
}

// K steps of V values a lane, all loads under way at once; W warps a row.  Bound by memory: 16384 rows of 2048 bf16 with a residual, bf16
// and 8-bit outputs take 46.8 us for 303 MB, 6.5 TB/s, 95 % of a copy's rate; 32 rows from fp32 2.1 us, one launch.  A persistent grid
// that loads the next row ahead holds fewer rows in flight (53.8 us).
// v = h w, y = v f with f = 1 / sqrt(mean(h^2) + eps): codes are those of v relative to max |v|, without f and its roundings, and a row's largest
// v is found in the same exchange as its sum.
template <typename X, int V, int K>
__global__ void __launch_bounds__(1024) norm_kernel(NormArgs a, int W, int rows) {
    __shared__ float2 row_s[32];
    qmoe::depend_wait();
    qmoe::depend_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = W == 1 ? warp : warp / W, in_row = warp - row * W;
    const int64_t t64 = (int64_t)blockIdx.x * rows + row;
    const bool on = t64 < a.T;
    const int t = on ? (int)t64 : 0, c0 = in_row * 32 + lane, step = W * 32, chunks = on ? a.n / V : 0;
    Values<V> h[K];
    {
        Raw<X, V> x[K];
        Raw<uint16_t, V> r[K];
        const X* xp = (const X*)a.x + (int64_t)t * a.x_stride + c0 * V;
        const uint16_t* rp = a.residual + (int64_t)t * a.res_stride + c0 * V;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (c0 + k * step < chunks) x[k].load(xp + k * step * V);
        if (a.residual) {
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (c0 + k * step < chunks) r[k].load(rp + k * step * V);
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            h[k] = Values<V>{};
            if (c0 + k * step < chunks) {
                h[k] = x[k].values();
                if (a.residual) h[k].add(r[k].values());
            }
        }
    }
    if (a.residual) {
        uint16_t* ro = a.residual_out + (int64_t)t * a.res_out_stride + c0 * V;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (c0 + k * step < chunks) store_bf16<V>(ro + k * step * V, h[k]);
    }
    float part[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < K; ++k) part[k & 1] = h[k].squares(part[k & 1]);
    if (a.weight) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (c0 + k * step < chunks) {
                Raw<uint16_t, V> w;
                w.load(a.weight + (c0 + k * step) * V);
                h[k].times(w.values());
            }
        }
    }
    float big[K] = {};
    if constexpr (V == 8) {
        if (a.codes) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                big[k] = largest(h[k]);
                if (a.row_scale) {
                    if (k) big[0] = max_nan(big[0], big[k]);
                    continue;
                }
#pragma unroll
                for (int d = 8; d > 0; d >>= 1) big[k] = max_nan(big[k], __shfl_xor_sync(QMOE_FULL_MASK, big[k], d));      // (16 lanes hold 128 values)
            }
        }
    }
    const float2 all = V == 8 && a.codes && a.row_scale ? row_reduce<true>(part[0] + part[1], big[0], W, row_s + row * W, in_row, lane)
                                                        : row_reduce<false>(part[0] + part[1], 0.f, W, row_s + row * W, in_row, lane);
    const float f = rsqrtf(__fdividef(all.x, (float)a.n) + a.eps);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = c0 + k * step;
        if (c >= chunks) break;
        if constexpr (V == 8) {
            if (a.codes) {
                const float m = a.row_scale ? all.y : big[k], top = m * f;
                store_codes(a.codes + (int64_t)t * a.n + c * V, h[k], m);
                if (a.row_scale) {
                    if (c == 0) a.scales[t] = top * (1.f / 448.f);
                } else if ((lane & 15) == 0) {
                    a.scales[(int64_t)t * ((a.n + 127) >> 7) + (c >> 4)] = top * (1.f / 448.f);
                }
                h[k].times(f);
                if (__builtin_expect(!(top > 0.f && top < INFINITY), 0)) {
                    // no scale: 0 where all y are 0, and for finite y beside infinite ones; the rest NaN
                    uint32_t w[2] = {0, 0};
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        if (top != 0.f && !(top == INFINITY && fabsf(h[k].v[i]) < INFINITY)) w[i >> 2] |= 0x7Fu << 8 * (i & 3);
                    *(uint2*)(a.codes + (int64_t)t * a.n + c * V) = make_uint2(w[0], w[1]);
                }
                if (a.y) store_bf16<V>(a.y + (int64_t)t * a.y_stride + c * V, h[k]);
                continue;
            }
        }
        h[k].times(f);
        if (a.y) store_bf16<V>(a.y + (int64_t)t * a.y_stride + c * V, h[k]);
    }
}

constexpr int kNormMaxWidth = 32768;

template <typename X, int V, int K>
int launch_norm_steps(const NormArgs& a, cudaStream_t st) {
    const int W = (a.n / V + 32 * K - 1) / (32 * K), rows = std::max(1, 4 / W);
    return launch_rows(norm_kernel<X, V, K>, a.T, (unsigned)(((int64_t)a.T + rows - 1) / rows), rows * W * 32, st, "add_rms_norm", a, W, rows);
}

// Steps a lane.  With many rows two, or three where that leaves fewer lanes idle (16384 rows of 2048 with a residual and codes, us, with one
// to four steps: 50.2, 46.8, 46.9, 47.7; 4095 of 2080 from fp32 with a scale a row: 18.9, 17.7, 17.3, 19.6).  With few rows one, for the
// shortest chain; more where a row would take more than 16 warps.
template <typename X, int V>
int launch_norm(const NormArgs& a, cudaStream_t st) {
    const int chunks = a.n / V;
    if (chunks <= 512 && a.T < 8 * qmoe::sm_count()) return launch_norm_steps<X, V, 1>(a, st);
    if (chunks <= 1024 && V == 8 && (chunks + 95) / 96 * 3 < (chunks + 63) / 64 * 2) return launch_norm_steps<X, V, V == 8 ? 3 : 2>(a, st);
    if (chunks <= 1024) return launch_norm_steps<X, V, 2>(a, st);
    if constexpr (V == 8) return launch_norm_steps<X, V, 4>(a, st);
    else return chunks <= 4096 ? launch_norm_steps<X, V, 8>(a, st) : launch_norm_steps<X, V, 32>(a, st);
}

// ---------------------------------------------------------------- choice of experts
//
// Scores s = softmax(l) or 1 / (1 + e^-l); an expert's value c = s + bias; a group's value the sum of its best one or two
// c; the k best experts by c of the best groups; gates s, or s over the sum of the chosen, times a factor.
//
// The order is that of the values in 64 bits, equal ones to the lower index.  Without a bias an expert's order is its
// logit's, exactly.  Else the values are made in fp32 with a bound on their error (the approximate exponential and reciprocal
// are enough), and where two neighbours in the order are nearer than their bounds, and are not the same logit with the
// same bias, those are made in fp64: of the experts in question (fp64 runs at a 64th of fp32's rate here), of the groups' best
// ones, or of a whole row where more of its experts are in question than the list of the chosen holds.
//
// A lane holds R neighbouring experts as integer keys, and the 4 best of them sorted; among lanes with equal keys the
// lowest has the lowest index.  A round of the choice is a reduction of the lanes' heads (one instruction), a ballot, and the
// winner's list moving up.  Which expert a key was is looked up at the end, for all the chosen at once.  A warp takes a
// token.  Above 256 experts without groups a block of 4 warps does, another way (wide_route_kernel).
struct RouteArgs {
    const void* logits;
    const float* bias;
    int32_t* ids;
    float* gates;
    int64_t stride;
    int T, E, k, sigmoid, groups, top_groups, best, renorm;
    int group_size, group_lanes;      // experts of a group; lanes, where a group is a power of two of whole ones (else 0)
    int vec, vec_bias;      // rows (the bias) allow loads of 16 bytes, or of all of a lane's values where those are fewer
    float scale;
};

constexpr int kWideWarps = 4;               // of a block that works on one token
constexpr int kTokenWarps = 4;              // of a block whose warps take a token each (small blocks end and begin evenly)
constexpr float kUlp = 5.9604645e-8f;       // 2^-24
constexpr float kLargest = 3.402823466e38f;
constexpr float kLog2e = 1.4426950408889634f;

// fp32 -> integer of the same order (-0 as 0; key_of_sum: there is none); 0 stands for no value.
__device__ __forceinline__ uint32_t key_of_sum(float v) {
    const uint32_t u = __float_as_uint(v);
    return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ uint32_t key_of(float v) { return key_of_sum(v + 0.f); }
__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}
__device__ __forceinline__ unsigned long long key_of(double v) {
    const unsigned long long u = (unsigned long long)__double_as_longlong(v + 0.0);
    return u >> 63 ? ~u : u | 0x8000000000000000ull;
}

__device__ __forceinline__ double value_of(unsigned long long key) {
    return __longlong_as_double((long long)(key >> 63 ? key & 0x7FFFFFFFFFFFFFFFull : ~key));
}

// A logit as it is read: NaN as -infinity, +infinity as the largest finite value.
__device__ __forceinline__ float clean(float v) { return fminf(fmaxf(v, -INFINITY), kLargest); }
template <typename X>
__device__ __forceinline__ float logit(const X* row, int e) {
    return clean(sizeof(X) == 2 ? bf16_to_f32(((const uint16_t*)row)[e]) : ((const float*)row)[e]);
}

// R values from p[e0] on, `none` past E.
template <typename X, int R>
__device__ __forceinline__ void load_values(const X* p, int e0, int E, int vec, float none, float (&v)[R]) {
    constexpr int W = R * (int)sizeof(X) < 16 ? R : 16 / (int)sizeof(X);      // values of a wide load
#pragma unroll
    for (int i = 0; i < R; ++i) v[i] = none;
    if (vec) {
#pragma unroll
        for (int c = 0; c < R; c += W) {
            if (e0 + c >= E) break;      // (E is a multiple of W)
            uint32_t w[W * sizeof(X) >= 4 ? W * sizeof(X) / 4 : 1];
            if constexpr (W * sizeof(X) == 16) {
                const uint4 x = *(const uint4*)(p + e0 + c);
                w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
            } else if constexpr (W * sizeof(X) == 8) {
                const uint2 x = *(const uint2*)(p + e0 + c);
                w[0] = x.x, w[1] = x.y;
            } else if constexpr (W * sizeof(X) == 4) {
                w[0] = *(const uint32_t*)(p + e0 + c);
            } else {
                w[0] = *(const uint16_t*)(p + e0 + c);
            }
#pragma unroll
            for (int i = 0; i < W; ++i)
                v[c + i] = sizeof(X) == 4 ? __uint_as_float(w[sizeof(X) == 4 ? i : 0]) : i & 1 ? bf16_hi(w[sizeof(X) == 4 ? 0 : i / 2]) : bf16_lo(w[sizeof(X) == 4 ? 0 : i / 2]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (e0 + i < E) v[i] = sizeof(X) == 2 ? bf16_to_f32(((const uint16_t*)p)[e0 + i]) : ((const float*)p)[e0 + i];
    }
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Bound on a score's error: sigmoid_near's; or, with x = l - top, (2.5 |x| + 4) 2^-24 of itself from an exponential (|x| e^x <=
// 0.37), the same of the sum (|x| weighed by the scores is at most ln E) and R / 4 + 17 additions, and 9 of a quotient and factors.
__device__ __forceinline__ float sum_error(int R) { return (float)(R / 4 + 70) * kUlp; }      // (of itself)
__device__ __forceinline__ float error_bound(const RouteArgs& a, int R, float inv_z) {
    return (a.sigmoid ? 6.f * kUlp : sum_error(R) * inv_z) + 1e-37f;
}

// Within 6 2^-24: (1.5 |l| + 4) 2^-24 of the exponential, which the score's slope s (1 - s) makes 1.4, and 3 of the rest.
__device__ __forceinline__ float sigmoid_near(float l) { return rcp(1.f + ex2(-kLog2e * l)); }

// ---- sorted lists of keys, the largest first
__device__ __forceinline__ void order(uint32_t& a, uint32_t& b) {
    const uint32_t hi = max(a, b);
    b = min(a, b), a = hi;
}
template <int N>
__device__ __forceinline__ void sort_keys(uint32_t* v) {
    if constexpr (N == 2) {
        order(v[0], v[1]);
    } else if constexpr (N == 4) {
        order(v[0], v[1]), order(v[2], v[3]), order(v[0], v[2]), order(v[1], v[3]), order(v[1], v[2]);
    }
}
// The keys that a lane keeps sorted.  Four: a lane of the 32 rarely holds more of the chosen (then choose_slow goes through all
// of them), and a round moves the list up by one.
template <int R>
constexpr int kDepth = R < 4 ? R : 4;

// The best kDepth<R> of R keys.
template <int R>
__device__ __forceinline__ void best_keys(const uint32_t (&key)[R], uint32_t (&list)[kDepth<R>]) {
#pragma unroll
    for (int i = 0; i < kDepth<R>; ++i) list[i] = key[i];
    sort_keys<kDepth<R>>(list);
#pragma unroll
    for (int c = 4; c < R; c += 4) {
        uint32_t more[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) more[i] = key[c + i];
        sort_keys<4>(more);
        // the larger halves of a bitonic sequence, then its merge
#pragma unroll
        for (int i = 0; i < kDepth<R>; ++i) list[i] = max(list[i], more[3 - i]);
        if constexpr (R > 4) order(list[0], list[2]), order(list[1], list[3]), order(list[0], list[1]), order(list[2], list[3]);
    }
}

// The `rounds` best of all lanes' lists: lane j gets the j-th one's key and the lane that held it.
template <int N>
__device__ __forceinline__ void choose(uint32_t (&list)[N], int rounds, int lane, uint32_t* my_key, int* my_lane) {
    const unsigned below = (1u << lane) - 1;
    unsigned mine_held = 1;
    *my_key = 0;
    for (int j = 0; j < rounds; ++j) {
        const uint32_t m = __reduce_max_sync(QMOE_FULL_MASK, list[0]);
        const unsigned held = __ballot_sync(QMOE_FULL_MASK, list[0] == m);
        if (lane == j) *my_key = m, mine_held = held;
        const bool mine = list[0] == m && !(held & below);
#pragma unroll
        for (int i = 0; i + 1 < N; ++i) list[i] = mine ? list[i + 1] : list[i];
        list[N - 1] = mine ? 0u : list[N - 1];
    }
    *my_lane = __ffs(mine_held) - 1;
}

// Whether a lane's list (`had`: it was not empty) ran out while it held another of the `rounds` best.
template <int R>
__device__ __forceinline__ bool ran_out(const uint32_t (&key)[R], const uint32_t (&list)[kDepth<R>], bool had, int rounds, uint32_t my_key) {
    if (R <= kDepth<R>) return false;
    const bool empty = had && list[0] == 0;
    if (!__any_sync(QMOE_FULL_MASK, empty)) return false;
    const uint32_t last = __shfl_sync(QMOE_FULL_MASK, my_key, rounds - 1);
    int n = 0;
#pragma unroll
    for (int i = 0; i < R; ++i) n += key[i] && key[i] >= last;
    return __any_sync(QMOE_FULL_MASK, empty && n > kDepth<R>);
}

// Which of its lane's experts the key of lane j's choice was: the first with that key, or the one after where the same
// lane gave the same key the round before.
template <int R>
__device__ __forceinline__ int which(const uint32_t (&key)[R], uint32_t my_key, int my_lane, int lane) {
    const uint32_t before = __shfl_up_sync(QMOE_FULL_MASK, my_key, 1);
    const int from = __shfl_up_sync(QMOE_FULL_MASK, my_lane, 1);
    const unsigned starts = __ballot_sync(QMOE_FULL_MASK, lane == 0 || before != my_key || from != my_lane);
    int skip = lane - (31 - __clz((int)(starts & (0xFFFFFFFFu >> (31 - lane)))));
    int at = R - 1;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const bool hit = __shfl_sync(QMOE_FULL_MASK, key[i], my_lane) == my_key;
        if (hit && skip == 0) at = i;
        skip -= hit;
    }
    return my_lane * R + at;
}

// As choose and which, from the keys themselves (any number of a lane's), which it takes out; the slow way.
template <int R>
__device__ __noinline__ void choose_slow(uint32_t* key, int rounds, int lane, uint32_t* my_key, int* my_at) {
    *my_key = 0, *my_at = -1;
    for (int j = 0; j < rounds; ++j) {
        uint32_t best = 0;
        int at = 0;
        for (int i = 0; i < R; ++i)
            if (key[i] > best) best = key[i], at = i;
        const uint32_t m = __reduce_max_sync(QMOE_FULL_MASK, best);
        const int w = __ffs(__ballot_sync(QMOE_FULL_MASK, best == m)) - 1;
        const int tag = __shfl_sync(QMOE_FULL_MASK, lane * R + at, w);
        if (lane == j) *my_key = m, *my_at = m ? tag : -1;
        if (lane == w) key[at] = 0;
    }
}

struct Pair {
    uint32_t a, b;      // keys of the best and the second best
};
__device__ __forceinline__ Pair merge(Pair x, Pair y) { return Pair{max(x.a, y.a), max(min(x.a, y.a), max(x.b, y.b))}; }

// Which groups are kept (bit g of the result), from keys that lane g holds for g < groups (others 0); the last one kept and the
// best one dropped.
__device__ __forceinline__ uint32_t best_groups(uint32_t key, int top, int lane, uint32_t* last, uint32_t* next) {
    const unsigned below = (1u << lane) - 1;
    uint32_t kept = 0, m = 0;
    for (int j = 0; j < top; ++j) {
        m = __reduce_max_sync(QMOE_FULL_MASK, key);
        const unsigned held = __ballot_sync(QMOE_FULL_MASK, key == m);
        kept |= held & (0u - held);
        if (key == m && !(held & below)) key = 0;
    }
    *last = m, *next = __reduce_max_sync(QMOE_FULL_MASK, key);
    return kept;
}

// The same from values, by comparing each with each.
template <typename F>
__device__ __forceinline__ uint32_t best_groups(F v, int groups, int top, int lane) {
    int rank = 0;
    for (int g = 0; g < groups; ++g) {
        const F o = __shfl_sync(QMOE_FULL_MASK, v, g);
        rank += o > v || (o == v && g < lane);
    }
    return __ballot_sync(QMOE_FULL_MASK, lane < groups && rank < top);
}

// ---- in 64 bits
__device__ __forceinline__ unsigned long long warp_max64(unsigned long long v) {
    const uint32_t hi = __reduce_max_sync(QMOE_FULL_MASK, (uint32_t)(v >> 32));
    const uint32_t lo = __reduce_max_sync(QMOE_FULL_MASK, (uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
    return (unsigned long long)hi << 32 | lo;
}

struct ResolveShared {
    double sum[kWideWarps];
    unsigned long long key[kWideWarps];
};

// Sum of the row's exponentials, by NW warps that hold R experts a lane from e0 on (1 for sigmoid scores).
template <typename X, int NW>
__device__ __noinline__ double exact_sum(const RouteArgs& a, const X* row, int e0, int R, float top, ResolveShared* sh) {
    if (a.sigmoid) return 1.0;
    double z = 0.0;
    for (int i = 0; i < R && e0 + i < a.E; ++i) {
        const float l = logit(row, e0 + i);
        if (l > -INFINITY) z += exp((double)l - (double)top);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) z += __shfl_xor_sync(QMOE_FULL_MASK, z, d);
    if (NW > 1) {
        __syncthreads();
        if ((threadIdx.x & 31) == 0) sh->sum[threadIdx.x >> 5] = z;
        __syncthreads();
        z = 0.0;
        for (int w = 0; w < NW; ++w) z += sh->sum[w];
    }
    return z > 0.0 ? z : 1.0;
}

// Value c of expert e.
template <typename X>
__device__ __noinline__ double exact_value(const RouteArgs& a, const X* row, int e, float top, double z) {
    const double l = logit(row, e);
    double s = l > -INFINITY ? a.sigmoid ? 1.0 / (1.0 + exp(-l)) : exp(l - (double)top) / z : 0.0;
    if (a.bias) s += (double)a.bias[e];
    return s == s ? s : -INFINITY;
}

// Values of the groups in `which`, to lane g for group g, from the experts that each lane names (bit i of `cand`: e0 + i).
template <typename X>
__device__ __noinline__ double exact_groups(const RouteArgs& a, const X* row, int e0, int R, float top, uint32_t cand, uint32_t which_groups) {
    const int lane = threadIdx.x & 31, size = a.E / a.groups;
    const double z = exact_sum<X, 1>(a, row, e0, R, top, nullptr);
    unsigned long long c[32];
    for (uint32_t todo = cand; todo; todo &= todo - 1) c[__ffs(todo) - 1] = key_of(exact_value(a, row, e0 + __ffs(todo) - 1, top, z));
    __syncwarp();
    double mine = 0.0;
    for (uint32_t todo = which_groups; todo; todo &= todo - 1) {
        const int g = __ffs(todo) - 1;
        unsigned long long b0 = 0, b1 = 0;
        for (uint32_t left = cand; left; left &= left - 1) {
            const int i = __ffs(left) - 1, e = e0 + i;
            if (e < g * size || e >= (g + 1) * size) continue;
            b1 = max(b1, min(b0, c[i]));
            b0 = max(b0, c[i]);
        }
        __syncwarp();
        const unsigned long long best = warp_max64(b0);
        double v = value_of(best);
        if (a.best == 2) {
            // the second best: the next of the lane that held the best, or another lane's best
            const int w = __ffs(__ballot_sync(QMOE_FULL_MASK, b0 == best)) - 1;
            v += value_of(warp_max64(lane == w ? b1 : b0));
        }
        if (v != v) v = -INFINITY;
        if (lane == g) mine = v;
    }
    return mine;
}

// The choice among the experts that each lane names, by NW warps: lane j of each gets the j-th expert.  (Without a bias: by
// the logits themselves.)
template <typename X, int NW, typename Bits>
__device__ __noinline__ int exact_choice(const RouteArgs& a, const X* row, int e0, int R, float top, Bits cand, ResolveShared* sh) {
    constexpr int MOST = 8 * sizeof(Bits);
    const int lane = threadIdx.x & 31, warp = NW == 1 ? 0 : threadIdx.x >> 5;
    const double z = a.bias ? exact_sum<X, NW>(a, row, e0, R, top, sh) : 1.0;
    unsigned long long c[MOST];
    for (int i = 0; i < R; ++i) c[i] = 0ull;
    for (Bits todo = cand; todo; todo &= todo - 1) {
        const int i = sizeof(Bits) == 8 ? __ffsll((long long)todo) - 1 : __ffs((int)todo) - 1;
        c[i] = key_of(a.bias ? exact_value(a, row, e0 + i, top, z) : (double)logit(row, e0 + i));
    }
    __syncwarp();
    int got = 0;
    for (int j = 0; j < a.k; ++j) {
        unsigned long long best = 0;
        int at = 0;
        for (int i = 0; i < R; ++i)
            if (c[i] > best) best = c[i], at = i;
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
            if (lane == w) c[at] = 0;
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

// The list of lanes 0 .. n - 1 in the order of its values, those of lanes with `near` from scores in 64 bits.  The softmax's sum stays
// the fp32 one (256 exponentials in fp64 take 3 us here, 2048 some 22), within `error` of itself: that moves the difference of two
// values by so much of their scores' difference, which is no more than their biases'.  -1 where that still leaves a doubt.
template <typename X>
__device__ __noinline__ int exact_order(const RouteArgs& a, const X* row, int n, float value, int mine, bool near, float top, float z, float error) {
    const int lane = threadIdx.x & 31;
    double c = (double)value, p = 0.0;
    if (near) {
        const double l = logit(row, mine);
        p = l > -INFINITY ? a.sigmoid ? 1.0 / (1.0 + exp(-l)) : exp(l - (double)top) / (double)z : 0.0;
        c = p + (double)a.bias[mine];
        if (c != c) c = -INFINITY;
    }
    const unsigned long long key = key_of(c);
    int rank = 0, from = lane;
    for (int j = 0; j < n; ++j) {
        const unsigned long long o = __shfl_sync(QMOE_FULL_MASK, key, j);
        const int e = __shfl_sync(QMOE_FULL_MASK, mine, j);      // (outside the condition: every lane takes part)
        rank += o > key || (o == key && e < mine);
    }
    for (int j = 0; j < n; ++j)
        if (__shfl_sync(QMOE_FULL_MASK, rank, j) == lane) from = j;
    // neighbours in the new order (the same logit and bias give the same bits; infinite values are equal or not)
    bool sure = true;
    if (!a.sigmoid) {
        c = __shfl_sync(QMOE_FULL_MASK, c, from), p = __shfl_sync(QMOE_FULL_MASK, p, from);
        near = __shfl_sync(QMOE_FULL_MASK, (int)near, from) != 0;
        const double o = __shfl_down_sync(QMOE_FULL_MASK, c, 1), q = __shfl_down_sync(QMOE_FULL_MASK, p, 1);
        const bool both = __shfl_down_sync(QMOE_FULL_MASK, (int)near, 1) != 0 && near && lane + 1 < n;
        sure = !both || (o == c && q == p) || c - o > fabs(q - p) * (double)error + 4e-16 * (fabs(o) + fabs(c));
    }
    const int got = __shfl_sync(QMOE_FULL_MASK, mine, from);
    return __all_sync(QMOE_FULL_MASK, sure) ? got : -1;
}

// Gates of the experts that lanes 0 .. k - 1 hold (l: their logits), and the outputs of token t.  Renormalised weights are taken
// relative to the largest, so that scores below fp32's range keep their ratios.
__device__ __forceinline__ void write_route(const RouteArgs& a, int64_t t, int id, float l, float top, float z, int lane) {
    const bool on = lane < a.k;
    if (!on) l = -INFINITY;
    float g = 0.f;
    if (a.renorm) {
        float big = l;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) big = fmaxf(big, __shfl_xor_sync(QMOE_FULL_MASK, big, d));
        if (l > -INFINITY) {
            if (!a.sigmoid) {
                g = expf(l - big);
            } else {
                const float e = expf(-fabsf(l));      // 1 / (1 + e^-l) = e^l / (1 + e^l)
                g = (l >= 0.f ? 1.f : big >= 0.f ? e : expf(l - big)) * rcp(1.f + e);
            }
        }
        const float sum = warp_sum(g);
        // a quotient and one Newton step, which makes it exactly 1 for one expert (sum is 0.5 to 32; a correctly rounded division is 5 % of
        // the kernel's time)
        const float r = rcp(sum), q = g * r;
        g = sum > 0.f ? fmaf(fmaf(-q, sum, g), r, q) : 0.f;
    } else if (l > -INFINITY) {
        if (a.sigmoid) {
            const float e = expf(-fabsf(l));
            g = (l >= 0.f ? 1.f : e) * rcp(1.f + e);
        } else {
            g = expf(l - top) / z;
        }
    }
    if (on) {
        a.ids[t * a.k + lane] = id;
        a.gates[t * a.k + lane] = g * a.scale;
    }
}

// Which of the list that the lanes hold, largest first, are too near to tell apart (key mk of expert at, whose logit is l; one
// entry more than are chosen, where there is one).  Two neighbours of the same logit and bias are no doubt if they stand by index (the
// scores of one logit may differ in their last bits from warp to warp of wide_route_kernel, whose factors do).  Where they are the last one
// chosen and the one behind it, what stands behind both may still be larger than they are, and only what equals them may not.
struct Doubts {
    bool behind;     // some two neighbours, or what is behind the list has to be looked at (else nothing below is set)
    bool any;        // some two neighbours
    bool mine;       // this lane's entry is one of such a pair, or equal to one that is
    float last;      // value of the last one chosen
    float least;     // what is below that for certain
    int last_id;     // the last one chosen
};
__device__ __forceinline__ Doubts doubts_of(const RouteArgs& a, uint32_t mk, int at, float l, float slack, int lane) {
    const float v = value_of(mk);
    const uint32_t nk = __shfl_down_sync(QMOE_FULL_MASK, mk, 1);
    const int nat = __shfl_down_sync(QMOE_FULL_MASK, at, 1);
    const float nl = __shfl_down_sync(QMOE_FULL_MASK, l, 1);
    bool near = false, doubt = false, ask = false;
    if (lane < a.k && lane < 31 && mk && nk) {
        const float nv = value_of(nk);
        near = fabsf(v) < INFINITY && nv > -INFINITY ? v - nv <= 2.f * slack + kUlp * (fabsf(v) + fabsf(nv)) : v == nv;
        if (near) doubt = !(l == nl && a.bias[at] == a.bias[nat] && at < nat), ask = doubt || lane == a.k - 1;
    }
    Doubts d{};
    d.behind = __any_sync(QMOE_FULL_MASK, ask) || a.k == 32;
    if (__builtin_expect(d.behind, 0)) {
        const unsigned pairs = __ballot_sync(QMOE_FULL_MASK, near);
        d.any = __any_sync(QMOE_FULL_MASK, doubt) != 0;
        d.mine = ((pairs | pairs << 1) >> lane & 1) != 0;
        d.last = value_of(__shfl_sync(QMOE_FULL_MASK, mk, a.k - 1));
        d.least = d.last - (2.f * slack + 4.f * kUlp * fminf(fabsf(d.last), kLargest));
        d.last_id = __shfl_sync(QMOE_FULL_MASK, at, a.k - 1);
    }
    return d;
}
// Whether expert e equals the last one chosen and comes after it.  (With doubts in the list that one's place is open.)
template <typename X>
__device__ __forceinline__ bool comes_after(const RouteArgs& a, const X* row, int last, int e) {
    return e >= last && logit(row, e) == logit(row, last) && a.bias[e] == a.bias[last];
}
// The experts that do not, of those that a lane names (bit i: e0 + i).  Out of line, and behind a count that most rows end with: 16383
// tokens of 256 experts take 16.3 us without a look behind the list, 16.4 so and 16.7 with this in line and a second vote.
template <typename X>
__device__ __noinline__ uint32_t others(const RouteArgs& a, const X* row, int e0, uint32_t cand, int last) {
    uint32_t open = cand;
    for (uint32_t todo = cand; todo; todo &= todo - 1) {
        const int i = __ffs((int)todo) - 1;
        if (comes_after(a, row, last, e0 + i)) open &= ~(1u << i);
    }
    __syncwarp();
    return open;
}

// R experts a lane, a warp a token.  Instructions bound it, and the latency of a round (a reduction, a ballot, a list that moves up): 16383
// tokens of 256 experts in 8 groups, the best 8 by sigmoid scores and a bias, 16.4 us and 795 instructions a token, 65 % of the
// issue slots; 32 tokens 3.6 to 4.2 us.  A warp that goes on to another token with its logits loaded ahead took 19 us.
template <typename X, int R>
__global__ void __launch_bounds__(kTokenWarps * 32, R <= 8 ? 8 : 4) route_kernel(RouteArgs a) {
    qmoe::depend_wait();
    qmoe::depend_launch();
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * kTokenWarps + (threadIdx.x >> 5);
    if (t >= a.T) return;
    const X* row = (const X*)a.logits + t * a.stride;
    const int e0 = lane * R;
    float c[R];
    load_values<X, R>(row, e0, a.E, a.vec, -INFINITY, c);
#pragma unroll
    for (int i = 0; i < R; ++i) c[i] = clean(c[i]);
    // ---- softmax: largest logit and sum of exponentials, where they are needed
    const bool by_logit = !a.bias, sums = a.groups > 1 && a.best == 2;
    float top = 0.f, z = 1.f;
    if (!a.sigmoid && !(by_logit && a.renorm && !sums)) {
        top = c[0];
#pragma unroll
        for (int i = 1; i < R; ++i) top = fmaxf(top, c[i]);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(QMOE_FULL_MASK, top, d));
        if (!(top > -INFINITY)) top = 0.f;       // nothing in the row: scores 0
        float part[4] = {};
#pragma unroll
        for (int i = 0; i < R; ++i) part[i & 3] += ex2(kLog2e * (c[i] - top));
        z = warp_sum((part[0] + part[1]) + (part[2] + part[3]));
        if (!(z > 0.f)) z = 1.f;
    }
    // ---- values, and the bound on a score's error
    const float inv_z = rcp(z), score_err = error_bound(a, R, inv_z), slack = by_logit ? 0.f : score_err;
    auto score_near = [&](float l) { return a.sigmoid ? sigmoid_near(l) : ex2(kLog2e * (l - top)) * inv_z; };
    if (!by_logit) {
        float bias[R];
        load_values<float, R>(a.bias, e0, a.E, a.vec_bias, 0.f, bias);
#pragma unroll
        for (int i = 0; i < R; ++i) c[i] = fmaxf(score_near(c[i]) + bias[i], -INFINITY);      // (an infinite bias may give NaN; never -0)
    } else {
#pragma unroll
        for (int i = 0; i < R; ++i) c[i] += 0.f;
    }
    uint32_t key[R], list[kDepth<R>];
#pragma unroll
    for (int i = 0; i < R; ++i) key[i] = key_of_sum(c[i]);
    if (e0 + R > a.E) {
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (e0 + i >= a.E) key[i] = 0u;
    }
    best_keys<R>(key, list);
    if (a.groups > 1) {
        // ---- groups
        const int size = a.group_size, lanes = a.group_lanes;
        const bool whole = lanes > 0;
        Pair mine{0, 0};
        if (whole) {
            Pair p{list[0], R > 1 ? list[R > 1 ? 1 : 0] : 0u};
#pragma unroll
            for (int d = 1; d < 32; d <<= 1)
                if (d < lanes) p = merge(p, Pair{__shfl_xor_sync(QMOE_FULL_MASK, p.a, d), __shfl_xor_sync(QMOE_FULL_MASK, p.b, d)});
            mine = Pair{__shfl_sync(QMOE_FULL_MASK, p.a, lane * lanes & 31), __shfl_sync(QMOE_FULL_MASK, p.b, lane * lanes & 31)};
        } else {
            for (int g = 0; g < a.groups; ++g) {
                Pair p{0, 0};
#pragma unroll
                for (int i = 0; i < R; ++i)
                    if (e0 + i >= g * size && e0 + i < (g + 1) * size) p = merge(p, Pair{key[i], 0});
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) p = merge(p, Pair{__shfl_xor_sync(QMOE_FULL_MASK, p.a, d), __shfl_xor_sync(QMOE_FULL_MASK, p.b, d)});
                if (lane == g) mine = p;
            }
        }
        const bool on = lane < a.groups;
        uint32_t kept, last, next;
        if (by_logit && a.best == 1) {
            kept = best_groups(on ? mine.a : 0u, a.top_groups, lane, &last, &next);
        } else {
            float va = value_of(mine.a), vb = a.best == 2 ? value_of(mine.b) : 0.f;
            if (by_logit) va = score_near(va), vb = score_near(vb);      // (sums of scores)
            const float v = on ? fmaxf(va + vb, -INFINITY) : -INFINITY;
            kept = best_groups(on ? key_of(v) : 0u, a.top_groups, lane, &last, &next);
            if (a.top_groups < a.groups) {
                // the last one kept and the best one dropped
                const float mag = fabsf(va) + fabsf(vb);
                const float err = on ? 2.f * score_err + (mag < kLargest ? 2.f * kUlp * mag : 0.f) : 0.f;
                const float low = value_of(last), high = value_of(next);
                const float err2 = 2.f * __uint_as_float(__reduce_max_sync(QMOE_FULL_MASK, __float_as_uint(err)));
                // (infinite ones are equal or not, whatever the bits: NaN here)
                if (__builtin_expect(low - high <= err2, 0)) {
                    const uint32_t doubt = __ballot_sync(QMOE_FULL_MASK, on && v >= high - err2 && v <= low + err2);
                    // the experts that may be among the best of those groups
                    uint32_t cand = 0;
                    for (uint32_t todo = doubt; todo; todo &= todo - 1) {
                        const int g = __ffs(todo) - 1;
                        const uint32_t least = __shfl_sync(QMOE_FULL_MASK, a.best == 2 ? mine.b : mine.a, g);
                        const float from = value_of(least) - (2.f * slack + 2.f * kUlp * fminf(fabsf(value_of(least)), kLargest));
#pragma unroll
                        for (int i = 0; i < R; ++i)
                            if (e0 + i >= g * size && e0 + i < (g + 1) * size && (by_logit ? key[i] >= least : value_of(key[i]) >= from)) cand |= 1u << i;
                    }
                    const double exact = exact_groups(a, row, e0, R, top, cand, doubt);
                    kept = best_groups((doubt >> lane) & 1 ? exact : (double)v, a.groups, a.top_groups, lane);
                }
            }
        }
        if (whole) {
            const bool off = !((kept >> (lane >> (31 - __clz(lanes)))) & 1);      // (lanes past the last group hold nothing)
#pragma unroll
            for (int i = 0; i < R; ++i) key[i] = off ? 0u : key[i];
#pragma unroll
            for (int i = 0; i < kDepth<R>; ++i) list[i] = off ? 0u : list[i];
        } else {
#pragma unroll
            for (int i = 0; i < R; ++i)
                if (e0 + i < a.E && !((kept >> ((e0 + i) / size)) & 1)) key[i] = 0u;
            best_keys<R>(key, list);
        }
    }
    // ---- the k best, and the next one where the values are not exact
    const int rounds = min(a.k + (by_logit ? 0 : 1), 32);
    uint32_t mk;
    int at, from;
    const bool had = list[0] != 0;
    choose(list, rounds, lane, &mk, &from);
    if (__builtin_expect(ran_out<R>(key, list, had, rounds, mk), 0)) {
        uint32_t all[R];
#pragma unroll
        for (int i = 0; i < R; ++i) all[i] = key[i];
        choose_slow<R>(all, rounds, lane, &mk, &at);
    } else {
        at = which<R>(key, mk, from, lane);
    }
    // ---- the chosen ones' logits, and neighbours that are too near to tell
    const bool in_list = lane < rounds && mk;
    if (!in_list) at = 0;
    float l = in_list ? logit(row, at) : -INFINITY;
    if (!by_logit) {
        const Doubts d = doubts_of(a, mk, at, l, slack, lane);
        if (__builtin_expect(d.behind, 0)) {
            // experts outside the list that may belong into it: values down to the last one's less the errors
            uint32_t cand = 0;
#pragma unroll
            for (int i = 0; i < R; ++i)
                if (key[i] && !(value_of(key[i]) < d.least)) cand |= 1u << i;
            const bool listed = in_list && !(value_of(mk) < d.least);
            bool again = warp_sum_int(__popc(cand)) > __popc(__ballot_sync(QMOE_FULL_MASK, listed));
            if (again && !d.any)
                again = warp_sum_int(__popc(others(a, row, e0, cand, d.last_id))) >
                        __popc(__ballot_sync(QMOE_FULL_MASK, listed && !comes_after(a, row, d.last_id, at)));
            if (!again && d.any) {
                at = exact_order(a, row, __popc(__ballot_sync(QMOE_FULL_MASK, in_list)), value_of(mk), at, d.mine, top, z, sum_error(R));
                again = at < 0;
            }
            if (again) at = exact_choice<X, 1>(a, row, e0, R, top, cand, nullptr);
            if (lane < a.k) l = logit(row, at);
        }
    }
    write_route(a, t, at, l, top, z, lane);
}

// Many experts without groups: a block of 4 warps a token, R values a thread in loads that stand side by side.  In each warp
// the `rounds`-th largest of the lanes' maxima bounds the values to look at from below, and the largest of the warps' bounds
// does for all; the few values that reach it are put side by side in shared memory, and the first warp's rounds go over
// those, by key and index.  The three barriers of a row bound it: 4096 tokens of 2048 fp32 logits, 2 by softmax and a bias, 17.7 us, 1.9 TB/s,
// 51 % of the issue slots (a warp a token 21 to 23 us).
constexpr int kWideMost = 256;      // values put side by side; rows with more (many equal ones) take exact_choice

template <typename X, int R>
__global__ void __launch_bounds__(kWideWarps * 32, R <= 16 ? 10 : R <= 32 ? 5 : 3) wide_route_kernel(RouteArgs a) {
    constexpr int V = 16 / (int)sizeof(X), THREADS = kWideWarps * 32, CHUNK = R < 8 ? R : 8;
    __shared__ ResolveShared rs;
    __shared__ uint32_t key_s[kWideMost], bound_s[kWideWarps];
    __shared__ int id_s[kWideMost], count_s, again_s;
    __shared__ float2 part_s[kWideWarps];
    qmoe::depend_wait();
    qmoe::depend_launch();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t t = blockIdx.x;
    const X* row = (const X*)a.logits + t * a.stride;
    // expert of value i
    auto expert = [&](int i) { return a.vec ? (i / V) * (THREADS * V) + tid * V + i % V : i * THREADS + tid; };
    float c[R];
    if (a.vec) {
#pragma unroll
        for (int i = 0; i < R; i += V) {
            float v[V];
            load_values<X, V>(row, expert(i), a.E, 1, -INFINITY, v);
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (i + j < R) c[i + j] = clean(v[j]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < R; ++i) c[i] = i * THREADS + tid < a.E ? logit(row, i * THREADS + tid) : -INFINITY;
    }
    if (tid == 0) count_s = 0;
    const bool by_logit = !a.bias;
    // the bias, where registers hold it as well: behind the barrier of the sum it would be waited for (18.0 -> 17.5 us)
    constexpr bool kAhead = R <= 16;
    const bool vec_bias = a.vec && a.vec_bias;
    float bias[kAhead ? R : 4];
    auto load_bias = [&](int i, float* to) {
        float v[4];
        if (vec_bias) {
            load_values<float, 4>(a.bias, expert(i), a.E, 1, 0.f, v);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = expert(i + j) < a.E ? a.bias[expert(i + j)] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) to[j] = v[j];
    };
    if (kAhead && !by_logit) {
#pragma unroll
        for (int i = 0; i < R; i += 4) load_bias(i, bias + (kAhead ? i : 0));
    }
    float top = 0.f, z = 1.f, inv_z = 1.f, scale = 1.f;
    if (!a.sigmoid && !(by_logit && a.renorm)) {
        // a warp's exponentials are by its own largest logit until the block's is known
        float mine = c[0];
#pragma unroll
        for (int i = 1; i < R; ++i) mine = fmaxf(mine, c[i]);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) mine = fmaxf(mine, __shfl_xor_sync(QMOE_FULL_MASK, mine, d));
        const float by = mine > -INFINITY ? mine : 0.f;
        float part[4] = {};
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const float e = ex2(kLog2e * (c[i] - by));
            part[i & 3] += e;
            if (!by_logit) c[i] = e;
        }
        const float sum = warp_sum((part[0] + part[1]) + (part[2] + part[3]));
        if (lane == 0) part_s[warp] = make_float2(mine, sum);
        __syncthreads();
        const float2 p0 = part_s[0], p1 = part_s[1], p2 = part_s[2], p3 = part_s[3];
        top = fmaxf(fmaxf(p0.x, p1.x), fmaxf(p2.x, p3.x));
        if (!(top > -INFINITY)) top = 0.f;       // nothing in the row: scores 0
        z = fmaf(p0.y, ex2(kLog2e * (p0.x - top)), p1.y * ex2(kLog2e * (p1.x - top))) + fmaf(p2.y, ex2(kLog2e * (p2.x - top)), p3.y * ex2(kLog2e * (p3.x - top)));
        if (!(z > 0.f)) z = 1.f;
        inv_z = rcp(z), scale = mine > -INFINITY ? ex2(kLog2e * (by - top)) * inv_z : 0.f;
    }
    const float slack = by_logit ? 0.f : error_bound(a, R, inv_z);
    if (!by_logit) {
        if (a.sigmoid) {
#pragma unroll
            for (int i = 0; i < R; ++i) c[i] = sigmoid_near(c[i]);
        }
#pragma unroll
        for (int i = 0; i < R; i += 4) {
            if (!kAhead) load_bias(i, bias);
            const float* add = bias + (kAhead ? i : 0);
#pragma unroll
            for (int j = 0; j < 4; ++j) c[i + j] = fmaxf(fmaf(c[i + j], scale, add[j]), -INFINITY);
        }
        if (a.E < THREADS * R) {
#pragma unroll
            for (int i = 0; i < R; ++i)
                if (expert(i) >= a.E) c[i] = -INFINITY;
        }
    }
    // ---- the lanes' largest values, and the `rounds`-th of them
    float chunk[R / CHUNK], mine = -INFINITY;
#pragma unroll
    for (int i = 0; i < R / CHUNK; ++i) {
        chunk[i] = c[i * CHUNK];
#pragma unroll
        for (int j = 1; j < CHUNK; ++j) chunk[i] = fmaxf(chunk[i], c[i * CHUNK + j]);
        mine = fmaxf(mine, chunk[i]);
    }
    const int rounds = min(a.k + (by_logit ? 0 : 1), 32);
    uint32_t head = key_of(mine), bound = 0;
    for (int j = 0; j < rounds; ++j) {
        bound = __reduce_max_sync(QMOE_FULL_MASK, head);
        const int w = __ffs(__ballot_sync(QMOE_FULL_MASK, head == bound)) - 1;
        if (lane == w) head = 0;
    }
    if (lane == 0) bound_s[warp] = bound;
    __syncthreads();
    bound = max(max(bound_s[0], bound_s[1]), max(bound_s[2], bound_s[3]));
    // (less the errors, as doubts_of takes off the last one chosen: what may belong to the chosen is in the list)
    const float reach = value_of(bound), from = by_logit ? reach : reach - (2.f * slack + 4.f * kUlp * fminf(fabsf(reach), kLargest));
#pragma unroll
    for (int i = 0; i < R / CHUNK; ++i) {
        if (chunk[i] >= from) {
#pragma unroll
            for (int j = 0; j < CHUNK; ++j) {
                const int e = expert(i * CHUNK + j);
                if (c[i * CHUNK + j] >= from && e < a.E) {
                    const int at = atomicAdd(&count_s, 1);      // (their order does not matter)
                    if (at < kWideMost) key_s[at] = key_of(c[i * CHUNK + j]), id_s[at] = e;
                }
            }
        }
    }
    __syncthreads();
    bool again = false;
    int at = 0;
    float l = -INFINITY;
    if (warp == 0) {
        const int n = count_s;
        again = n > kWideMost;
        if (!again) {
            constexpr int MOST = kWideMost / 32;
            uint32_t key[MOST], mk = 0;
            int id[MOST];
            const int mine_n = (n + 31) / 32;
            bool in_list = false;
            auto take = [&]() {
                for (int j = 0; j < rounds; ++j) {
                    uint32_t best = key[0];
                    int e = id[0];
                    if (mine_n > 1) {
#pragma unroll
                        for (int i = 1; i < MOST; ++i)
                            if (key[i] > best || (key[i] == best && id[i] < e)) best = key[i], e = id[i];
                    }
                    const uint32_t m = __reduce_max_sync(QMOE_FULL_MASK, best);
                    const int first = (int)__reduce_min_sync(QMOE_FULL_MASK, best == m ? (unsigned)e : 0xFFFFFFFFu);
                    if (lane == j) mk = m, at = first;
#pragma unroll
                    for (int i = 0; i < MOST; ++i) {
                        if (i > 0 && mine_n == 1) break;
                        if (key[i] == m && id[i] == first) key[i] = 0;
                    }
                }
                in_list = lane < rounds && mk;
                if (!in_list) at = 0;
                l = in_list ? logit(row, at) : -INFINITY;
            };
#pragma unroll
            for (int i = 0; i < MOST; ++i) {
                key[i] = 0, id[i] = 0;
                if (i * 32 + lane < n) key[i] = key_s[i * 32 + lane], id[i] = id_s[i * 32 + lane];
            }
            take();
            if (!by_logit) {
                Doubts d = doubts_of(a, mk, at, l, slack, lane);
                if (__builtin_expect(d.behind && !a.sigmoid, 0)) {
                    // the listed values again, each by the block's largest logit and sum alone: what has the same logit and bias has the same
                    // bits, whichever warp it came from, and stands by index (what is not in the list is smaller for certain)
#pragma unroll
                    for (int i = 0; i < MOST; ++i)
                        if (i * 32 + lane < n) key[i] = key_of(fmaxf(fmaf(ex2(kLog2e * (logit(row, id[i]) - top)), inv_z, a.bias[id[i]]), -INFINITY));
                    mk = 0;
                    take();
                    d = doubts_of(a, mk, at, l, slack, lane);
                }
                if (__builtin_expect(d.behind, 0)) {
                    bool open = false;      // something that is left may belong to the chosen
#pragma unroll
                    for (int i = 0; i < MOST; ++i)
                        if (key[i] && !(value_of(key[i]) < d.least) && !(!d.any && comes_after(a, row, d.last_id, id[i]))) open = true;
                    again = __any_sync(QMOE_FULL_MASK, open);
                    if (!again && d.any) {
                        at = exact_order(a, row, __popc(__ballot_sync(QMOE_FULL_MASK, in_list)), value_of(mk), at, d.mine, top, z, sum_error(R));
                        again = at < 0;
                        if (in_list && !again) l = logit(row, at);
                    }
                }
            }
        }
        if (lane == 0) again_s = again;
    }
    if (by_logit ? count_s > kWideMost : true) {
        __syncthreads();
        if (__builtin_expect(again_s, 0)) {
            using Bits = std::conditional_t<(R > 32), unsigned long long, uint32_t>;
            const int have = min(max(a.E - tid * R, 0), R);      // all of the row, R neighbouring experts a thread
            const Bits cand = have == 0 ? 0 : ~(Bits)0 >> (8 * sizeof(Bits) - have);
            at = exact_choice<X, kWideWarps>(a, row, tid * R, R, top, cand, &rs);
            if (lane < a.k) l = logit(row, at);
        }
    }
    if (warp == 0) write_route(a, t, at, l, top, z, lane);
}

template <typename X>
int launch_route(const RouteArgs& a, cudaStream_t st) {
    const unsigned per_warp = ((unsigned)a.T + kTokenWarps - 1) / kTokenWarps, tokens = (unsigned)a.T;      // (T may be the largest int)
    constexpr int threads = kTokenWarps * 32, wide = kWideWarps * 32;
    auto launch = [&](void (*kernel)(RouteArgs), unsigned blocks, int n) { return launch_rows(kernel, a.T, blocks, n, st, "qmoe_route_scored", a); };
    if (a.E <= 32) return launch(route_kernel<X, 1>, per_warp, threads);
    if (a.E <= 64) return launch(route_kernel<X, 2>, per_warp, threads);
    if (a.E <= 128) return launch(route_kernel<X, 4>, per_warp, threads);
    if (a.E <= 256) return launch(route_kernel<X, 8>, per_warp, threads);
    if (a.groups > 1) return launch(a.E <= 512 ? route_kernel<X, 16> : route_kernel<X, 32>, per_warp, threads);
    if (a.E <= 1024) return launch(wide_route_kernel<X, 8>, tokens, wide);
    if (a.E <= 2048) return launch(wide_route_kernel<X, 16>, tokens, wide);
    if (a.E <= 4096) return launch(wide_route_kernel<X, 32>, tokens, wide);
    return launch(wide_route_kernel<X, 64>, tokens, wide);
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
    if (T == 1) x_stride = residual_stride = residual_out_stride = y_stride = 0;      // (not used)
    const int64_t strides = x_stride | (residual ? residual_stride | residual_out_stride : 0) | (y ? y_stride : 0);
    if (strides > 0x7FFFFFFF) return qmoe::fail(QMOE_EINVAL, "add_rms_norm: a row stride of 2^31 or more");
    const bool wide = n % 8 == 0 && strides % 8 == 0 && aligned(x, 16) && aligned(residual, 16) && aligned(residual_out, 16) &&
                      aligned(weight, 16) && aligned(y, 16);
    if (!aligned(x, x_is_f32 ? 4 : 2) || !aligned(residual, 2) || !aligned(residual_out, 2) || !aligned(weight, 2) || !aligned(y, 2) ||
        !aligned(scales, 4))
        return qmoe::fail(QMOE_EINVAL, "add_rms_norm: pointer not aligned to its type");
    if (codes && (!wide || !aligned(codes, 8)))
        return qmoe::fail(QMOE_EUNSUPPORTED, "add_rms_norm: codes need a row width and strides that are multiples of 8 and 16-byte aligned pointers");
    NormArgs a{x, (const uint16_t*)residual, (uint16_t*)residual_out, (const uint16_t*)weight, (uint16_t*)y, (uint8_t*)codes, scales,
               (int)x_stride, (int)residual_stride, (int)residual_out_stride, (int)y_stride, T, n, scale_group == 0, eps};
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
    // neighbouring experts of a lane (launch_route; 16 stands for more), and what its loads have to be multiples of
    const int R = E <= 32 ? 1 : E <= 64 ? 2 : E <= 128 ? 4 : E <= 256 ? 8 : 16, size = logits_are_f32 ? 4 : 2;
    const int wide = std::min(16, R * size), wide_bias = std::min(16, R * 4);
    const int per_lane = E > 512 && E <= 1024 ? 32 : R, group = E / n_groups, lanes = group / per_lane;
    RouteArgs a{};
    a.logits = logits, a.bias = bias, a.ids = ids, a.gates = gates, a.stride = row_stride;
    a.T = T, a.E = E, a.k = k, a.sigmoid = score == QMOE_SCORE_SIGMOID, a.groups = n_groups, a.top_groups = top_groups;
    a.best = group_best, a.renorm = renormalise ? 1 : 0, a.scale = scale;
    a.group_size = group, a.group_lanes = group % per_lane == 0 && (lanes & (lanes - 1)) == 0 ? lanes : 0;
    a.vec = aligned(logits, wide) && (T == 1 || row_stride * size % wide == 0) && E * size % wide == 0;
    a.vec_bias = aligned(bias, wide_bias) && E * 4 % wide_bias == 0;
    return logits_are_f32 ? launch_route<float>(a, (cudaStream_t)stream) : launch_route<uint16_t>(a, (cudaStream_t)stream);
}
