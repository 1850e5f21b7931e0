// Softmax attention over the 4-bit paged key/value cache.

#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "kv4_common.cuh"
#include "tc_common.cuh"

namespace {

__device__ int g_kv4_attention_error;

__device__ __forceinline__ void attn_set_error(int code) { atomicCAS(&g_kv4_attention_error, 0, code); }

struct AttnArgs {
    kv4::CacheView cache;
    const uint16_t* q;
    uint16_t* out;
    const int32_t *q_start, *kv_len, *table;
    int B, n_q_tokens, n_q_heads, group, max_blocks, max_q, max_kv;
    float scale;
    int causal, window;
};

// Whether request b can be run; what is wrong with it goes to the error word.
__device__ __forceinline__ bool request(const AttnArgs& a, int b, int* q0, int* q_len, int* kv_len, bool report) {
    const int s = a.q_start[b], e = a.q_start[b + 1], n = a.kv_len[b];
    *q0 = s, *q_len = e - s, *kv_len = n;
    if (s < 0 || e < s || e > a.n_q_tokens || n < 0) {
        if (report) attn_set_error(QMOE_EINVAL);
        return false;
    }
    if (e - s > a.max_q || n > a.max_kv) {
        if (report) attn_set_error(QMOE_ECAPACITY);
        return false;
    }
    return true;
}

// ---------------------------------------------------------------- few query rows: one pass over the codes
//
// A request's rows of one kv head (query n, head g of the group: row n * group + g) are few, so the
// cache's bytes bound the work.  With k_d = s u_d + z and v_d likewise,
//   scale q . k = scale (s (q . u) + z sum(q)),   sum_j p_j v_j = sum_j (p_j s_j) u_j + sum_j p_j z_j,
// the 4-bit codes are matrix operands as they are: a code in the low mantissa bits of an fp16 pattern
// is the subnormal u 2^-24 (u 2^-20 one nibble up), so two masks and a shift turn a 32-bit word into
// four operand registers, and scale and offset enter on the few scores.  Queries are scaled by a power
// of two per row into fp16's range (exact: bf16 has fewer significant bits), probabilities by the
// largest row scale seen, also a power of two, so that p s_v keeps fp16's 11 bits whatever the values'
// magnitude.  Statistics and sums are fp32.
//
// The products are S^T = U_k Q^T and O^T = U_v^T P^T (m16n8k16, keys or head values as the 16 rows, 8
// query rows as the 8 columns), so that one to eight rows fill the instruction; tcgen05's 128 rows
// would be idle and its operands would have to be expanded through shared memory.  The running maximum
// moves only when a score passes it by 2^8 (a vote per 16 tokens instead of a reduction).
//
// Work is cut into tiles of kTile tokens; the tiles of all (request, kv head) items in a row are dealt
// out to the blocks in equal runs, whatever the lengths.  A producer warp copies whole pages of one
// head (contiguous in the layout) into a ring of stages with bulk copies; four warps take 16 tokens of
// each 64.  An item that several blocks share leaves its parts (unnormalised sums, maximum, sum of
// weights) in the workspace for combine_kernel.
constexpr int kTile = 64;
constexpr int kStages = 4;
constexpr int kConsumers = 4;                        // warps that compute
constexpr int kDecodeThreads = 32 * (kConsumers + 1);
constexpr float kNoMax = -3.0e38f;                   // running maximum before any score
constexpr float kSlack = 8.f;                        // scores may pass the running maximum by 2^8
constexpr uint32_t kWaitLimit = 1u << 22;

// Tiles of request b for this path (0: not its request), and the first one.
__device__ __forceinline__ int tiles_of(const AttnArgs& a, int b, int max_rows, int* t0, bool report) {
    int q0, q_len, kv_len;
    *t0 = 0;
    if (!request(a, b, &q0, &q_len, &kv_len, report) || q_len == 0 || q_len * a.group > max_rows) return 0;
    const int first = a.causal ? kv_len - q_len : kv_len - 1;    // position of the first query
    const int lo = a.window ? max(0, first - a.window + 1) : 0;
    *t0 = lo / kTile;
    return max(1, (kv_len + kTile - 1) / kTile - *t0);
}

// Block-wide: units (tiles of all items) before request `want`'s first and in all, by a scan over the
// requests; or, with find >= 0, the request that holds unit `find`.  Every thread gets the results.
struct Found {
    long long total, before;
    int b;
};

template <int THREADS>
__device__ __forceinline__ Found scan_requests(const AttnArgs& a, int max_rows, long long want, bool by_request, int n_ctas,
                                               int cta, long long* chunk, bool report) {
    __shared__ long long warp_sum_s[THREADS / 32];
    __shared__ Found found;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (a.B + THREADS - 1) / THREADS;
    const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
    long long mine = 0;
    int t0;
    for (int b = b0; b < b1; ++b) mine += tiles_of(a, b, max_rows, &t0, report);
    mine *= a.cache.n_kv_heads;
    long long incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(QMOE_FULL_MASK, incl, d);
        if (lane >= d) incl += o;
    }
    if (lane == 31) warp_sum_s[warp] = incl;
    if (tid == 0) found.b = -1;
    __syncthreads();
    long long total = 0, before = incl - mine;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) before += warp_sum_s[w];
        total += warp_sum_s[w];
    }
    *chunk = max(1LL, (total + n_ctas - 1) / n_ctas);
    const long long target = by_request ? 0 : (long long)cta * *chunk;
    const bool here = by_request ? want >= b0 && want < b1 : target >= before && target < before + mine;
    if (here) {
        long long at = before;
        for (int b = b0; b < b1; ++b) {
            const long long n = (long long)tiles_of(a, b, max_rows, &t0, false) * a.cache.n_kv_heads;
            if (by_request ? b == want : target < at + n) {
                found.b = b;
                found.before = at;
                break;
            }
            at += n;
        }
    }
    __syncthreads();
    Found f = found;
    f.total = total;
    return f;
}

__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
    __half2 h = __floats2half2_rn(lo, hi);
    return *(uint32_t*)&h;
}

// Power of two 2^e as a float, e clamped to the normal range.
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((min(max(e, -126), 127) + 127) << 23); }

__device__ __forceinline__ void bulk_copy(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     qmoe_tc::smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(qmoe_tc::smem_u32(bar))
                 : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(qmoe_tc::smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void mbar_expect(uint64_t* bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(qmoe_tc::smem_u32(bar)), "r"(bytes) : "memory");
}

// What a stage holds.
struct StageInfo {
    int b, kh, tile, flags;
};
constexpr int kFirst = 1, kLast = 2, kWholeStart = 4, kWholeEnd = 8, kValid = 16;   // kValid << page of the tile

template <int D, int NT>
struct DecodeShared {
    // query operand of 16 or 32 rows (with 8 it is held in registers); every warp writes the same values
    alignas(16) uint2 qf[NT == 1 ? 1 : NT][D / 32][2][32];
    alignas(128) unsigned char stage[kStages][kTile * (D + 8)];
    alignas(16) float red[kConsumers][8][D + 4];
    float m[kConsumers][8], l[kConsumers][8];
    StageInfo info[kStages];
    uint64_t full[kStages], empty[kStages];
};

// fp32 parts of split items: slot 2 * block for an item that began before the block's run, 2 * block + 1
// for one that goes on after it; rows x (D sums, maximum, sum of weights).
__device__ __forceinline__ float* part_of(float* parts, long long cta, int which, int rows, int D) {
    return parts + ((size_t)cta * 2 + which) * (size_t)(rows * (D + 2));
}

template <int D, int NT>
__global__ void __launch_bounds__(kDecodeThreads, NT == 1 ? 4 : NT == 2 ? 3 : 2)
    decode_kernel(AttnArgs a, int max_rows, float* parts) {
    extern __shared__ unsigned char smem_raw[];
    DecodeShared<D, NT>& sh = *(DecodeShared<D, NT>*)(((uintptr_t)smem_raw + 127) & ~(uintptr_t)127);
    constexpr int W = D / 32;              // words of a key row that a lane reads
    constexpr int VW = D / 64;             // words of a value row that a lane reads
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            qmoe_tc::mbar_init(&sh.full[i], 1);
            qmoe_tc::mbar_init(&sh.empty[i], kConsumers);
        }
        qmoe_tc::fence_mbar_init();
    }
    long long chunk;
    const Found f = scan_requests<kDecodeThreads>(a, max_rows, 0, false, gridDim.x, blockIdx.x, &chunk, blockIdx.x == 0);
    const long long u0 = (long long)blockIdx.x * chunk, u1 = min(u0 + chunk, f.total);
    if (u0 >= u1) return;
    const int n_units = (int)(u1 - u0);

    if (warp == kConsumers) {
        // ---- producer: a warp, lane i copies the tile's i-th page
        const int per_tile = kTile >> a.cache.page_shift;
        const uint32_t page_copy = a.cache.head_bytes;
        int b = f.b, t0, n = tiles_of(a, b, max_rows, &t0, false);
        int kh = (int)((u0 - f.before) / n), tile = (int)((u0 - f.before) % n);
        int kv_len = a.kv_len[b];
        bool ok = true;
        int issued = 0;
        for (int u = 0; u < n_units && ok; ++u) {
            const int st = u % kStages;
            const int blk = (t0 + tile) * per_tile + lane;
            const bool mine = lane < per_tile && (blk << a.cache.page_shift) < kv_len;
            int page = -1;
            if (mine && blk < a.max_blocks) page = a.table[(int64_t)b * a.max_blocks + blk];
            const bool good = page >= 0 && page < a.cache.n_pages;
            if (mine && !good) attn_set_error(QMOE_EINVAL);
            const unsigned mask = __ballot_sync(QMOE_FULL_MASK, good);
            if (u >= kStages) ok = qmoe_tc::mbar_wait(&sh.empty[st], (uint32_t)((u / kStages - 1) & 1), kWaitLimit);
            if (!__all_sync(QMOE_FULL_MASK, ok)) {
                ok = false;
                break;
            }
            if (lane == 0) {
                int flags = (int)mask * kValid;
                if (u == 0 || tile == 0) flags |= kFirst;
                if (u == n_units - 1 || tile == n - 1) flags |= kLast;
                if (u >= tile) flags |= kWholeStart;            // the item's first tile is in this run
                if (u + (n - 1 - tile) < n_units) flags |= kWholeEnd;
                sh.info[st] = StageInfo{b, kh, t0 + tile, flags};
                mbar_expect(&sh.full[st], (uint32_t)__popc(mask) * page_copy);
            }
            __syncwarp();
            if (good) bulk_copy(sh.stage[st] + lane * page_copy, kv4::head_ptr(a.cache, page, kh), page_copy, &sh.full[st]);
            issued = u + 1;
            if (++tile == n) {
                tile = 0;
                if (++kh == a.cache.n_kv_heads) {
                    kh = 0;
                    if (u + 1 < n_units) {
                        do n = tiles_of(a, ++b, max_rows, &t0, false);
                        while (n == 0 && b + 1 < a.B);
                        kv_len = a.kv_len[b];
                    }
                }
            }
        }
        if (!ok) {
            // give up: report, and let the copies in flight land before the block's memory goes away
            if (lane == 0) attn_set_error(QMOE_ETIMEOUT);
            for (int u = max(0, issued - kStages); u < issued; ++u)
                qmoe_tc::mbar_wait(&sh.full[u % kStages], (uint32_t)((u / kStages) & 1), kWaitLimit);
        }
        return;
    }

    // ---- consumers
    const int g = lane >> 2, t = lane & 3;
    const int P = 1 << a.cache.page_shift;
    // this warp's 16 tokens of a tile: page of the tile and token in the page
    const int tok0 = warp * 16, pg = tok0 >> a.cache.page_shift, in0 = tok0 & (P - 1);
    const uint32_t page_off = (uint32_t)pg * a.cache.head_bytes;
    // row kappa of the product is token (kappa & 8) + ((kappa & 7) >> 1) + 4 (kappa & 1): the value operand's
    // lanes t then read four neighbouring rows
    const int kt = in0 + (g >> 1) + 4 * (g & 1);      // token of row g (row g + 8: kt + 8)
    const uint32_t k_off = page_off + (uint32_t)kt * (D / 2) + t * (W * 4);
    const uint32_t v_off = page_off + (uint32_t)(P + in0 + t) * (D / 2) + g * (VW * 4);
    const uint32_t kp_off = page_off + (uint32_t)P * D + kt * 4;
    const uint32_t vp_off = kp_off + (uint32_t)P * 4;

    uint2 qr[W][2];                // query operand of 8 rows: [word][nibble parity]
    float c1[NT][2], cz[NT][2];    // per row: factor of s (q . u), and factor times sum(q), in log2 units
    float m[NT][2], l[NT][2], pz[NT][2];
    float o[NT][4 * VW][4];
    float vs = 1.f, vlim = 1e-9f;  // probabilities carry vs (a power of two); a value scale >= vlim moves it
    int q0 = 0, q_len = 0, kv_len = 0;

    for (int u = 0; u < n_units; ++u) {
        const int st = u % kStages;
        if (!qmoe_tc::mbar_wait(&sh.full[st], (uint32_t)((u / kStages) & 1), kWaitLimit)) {
            if (lane == 0) attn_set_error(QMOE_ETIMEOUT);
            return;
        }
        const StageInfo in = sh.info[st];
        if (in.flags & kFirst) {
            q0 = a.q_start[in.b], q_len = a.q_start[in.b + 1] - q0, kv_len = a.kv_len[in.b];
            const int rows = q_len * a.group;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int row = nt * 8 + g;
                uint4 raw[W];
#pragma unroll
                for (int w = 0; w < W; ++w) raw[w] = make_uint4(0, 0, 0, 0);
                if (row < rows) {
                    const int n = row / a.group, h = in.kh * a.group + row - n * a.group;
                    const uint4* src = (const uint4*)(a.q + ((int64_t)(q0 + n) * a.n_q_heads + h) * D + t * (8 * W));
#pragma unroll
                    for (int w = 0; w < W; ++w) raw[w] = src[w];
                }
                float mx = 0.f, sum = 0.f;
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    const uint32_t r4[4] = {raw[w].x, raw[w].y, raw[w].z, raw[w].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        mx = fmaxf(mx, fmaxf(fabsf(bf16_lo(r4[i])), fabsf(bf16_hi(r4[i]))));
                        sum += bf16_lo(r4[i]) + bf16_hi(r4[i]);
                    }
                }
                mx = fmaxf(mx, __shfl_xor_sync(QMOE_FULL_MASK, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(QMOE_FULL_MASK, mx, 2));
                sum += __shfl_xor_sync(QMOE_FULL_MASK, sum, 1);
                sum += __shfl_xor_sync(QMOE_FULL_MASK, sum, 2);
                // the row's largest magnitude goes to [2^14, 2^15)
                const int e = mx > 0.f ? min(max((int)(__float_as_uint(mx) >> 23) - 127, -100), 126) : 0;
                const float up = pow2i(14 - e), f1 = a.scale * 1.4426950408889634f * pow2i(e - 14);
                sum *= up;
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    const uint32_t r4[4] = {raw[w].x, raw[w].y, raw[w].z, raw[w].w};
                    // registers of word w: values (0,1) (4,5) for even nibbles, (2,3) (6,7) for odd ones (u 16 times larger)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float s = i ? up * 0.0625f : up;
                        const uint2 v = make_uint2(half2_bits(bf16_lo(r4[i]) * s, bf16_hi(r4[i]) * s),
                                                   half2_bits(bf16_lo(r4[i + 2]) * s, bf16_hi(r4[i + 2]) * s));
                        if constexpr (NT == 1)
                            qr[w][i] = v;
                        else
                            sh.qf[nt][w][i][lane] = v;
                    }
                }
                const float fa = f1 * 16777216.f, fb = f1 * sum;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    c1[nt][i] = __shfl_sync(QMOE_FULL_MASK, fa, 8 * t + 4 * i);
                    cz[nt][i] = __shfl_sync(QMOE_FULL_MASK, fb, 8 * t + 4 * i);
                    m[nt][i] = kNoMax, l[nt][i] = 0.f, pz[nt][i] = 0.f;
                }
#pragma unroll
                for (int i = 0; i < 4 * VW; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[nt][i][j] = 0.f;
            }
            vs = 1.f, vlim = 1e-9f;
            __syncwarp();
        }
        const unsigned char* stg = sh.stage[st];
        // ---- scores of 16 tokens
        uint32_t kw[2][W];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            if constexpr (W == 4) {
                const uint4 x = *(const uint4*)(stg + k_off + r * 8 * (D / 2));
                kw[r][0] = x.x, kw[r][1] = x.y, kw[r][2] = x.z, kw[r][3] = x.w;
            } else {
                const uint2 x = *(const uint2*)(stg + k_off + r * 8 * (D / 2));
                kw[r][0] = x.x, kw[r][1] = x.y;
            }
        }
        float s[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[nt][j] = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const uint32_t x0 = kw[0][w], x1 = kw[1][w], y0 = x0 >> 8, y1 = x1 >> 8;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                uint2 qa, qb;
                if constexpr (NT == 1)
                    qa = qr[w][0], qb = qr[w][1];
                else
                    qa = sh.qf[nt][w][0][lane], qb = sh.qf[nt][w][1][lane];
                mma_16816(s[nt], x0 & 0x000F000Fu, x1 & 0x000F000Fu, y0 & 0x000F000Fu, y1 & 0x000F000Fu, qa.x, qa.y);
                mma_16816(s[nt], x0 & 0x00F000F0u, x1 & 0x00F000F0u, y0 & 0x00F000F0u, y1 & 0x00F000F0u, qb.x, qb.y);
            }
        }
        float sk[2], zk[2], sv[2], zv[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const float2 kp = __half22float2(*(const __half2*)(stg + kp_off + r * 32));
            const float2 vp = __half22float2(*(const __half2*)(stg + vp_off + r * 32));
            sk[r] = kp.x, zk[r] = kp.y, sv[r] = vp.x, zv[r] = vp.y;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    s[nt][2 * r + i] = fmaf(c1[nt][i], sk[r] * s[nt][2 * r + i], cz[nt][i] * zk[r]);
        // ---- tokens that some row does not see
        const int j0 = in.tile * kTile;
        const int first = a.causal ? kv_len - q_len : kv_len - 1;
        const int edge_lo = a.window ? max(0, (a.causal ? kv_len - 1 : first) - a.window + 1) : 0;
        if (j0 + kTile > first + 1 || j0 + kTile > kv_len || j0 < edge_lo ||
            (in.flags / kValid) != (1 << (kTile >> a.cache.page_shift)) - 1) {
            const bool page_ok = (in.flags / kValid >> pg) & 1;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int j = j0 + tok0 + (g >> 1) + 4 * (g & 1) + 8 * r;
                const bool there = page_ok && j < kv_len;
                if (!there) sv[r] = 0.f, zv[r] = 0.f;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int pos = a.causal ? first + (nt * 8 + 2 * t + i) / a.group : first;
                        if (!there || j > pos || (a.window && j <= pos - a.window)) s[nt][2 * r + i] = -INFINITY;
                    }
            }
        }
        // ---- move the maximum or the values' scale, rarely
        bool move = fmaxf(fabsf(sv[0]), fabsf(sv[1])) >= vlim;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) move |= fmaxf(s[nt][i], s[nt][2 + i]) > m[nt][i] + kSlack;
        if (__any_sync(QMOE_FULL_MASK, move)) {
            float v = fmaxf(fmaxf(fabsf(sv[0]), fabsf(sv[1])), vlim * 0.5f);
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) v = fmaxf(v, __shfl_xor_sync(QMOE_FULL_MASK, v, d));
            float fo = 1.f;
            if (v >= vlim) {
                const int k = (int)(__float_as_uint(v) >> 23) - 127;       // v in [2^k, 2^(k+1))
                const float nvs = pow2i(6 - k);
                fo = nvs / vs;
                vs = nvs;
                vlim = pow2i(k + 1);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float fr[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float mx = fmaxf(s[nt][i], s[nt][2 + i]);
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(QMOE_FULL_MASK, mx, d));
                    const float m2 = fmaxf(m[nt][i], mx), fm = ex2(m[nt][i] - m2);
                    m[nt][i] = m2;
                    l[nt][i] *= fm, pz[nt][i] *= fm;
                    fr[i] = fm * fo;
                }
#pragma unroll
                for (int i = 0; i < 4 * VW; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[nt][i][j] *= fr[j & 1];
            }
        }
        // ---- probabilities, as the value product's operand
        uint32_t pf[NT][2];
        const float w0 = sv[0] * vs, w1 = sv[1] * vs;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float p[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) p[j] = ex2(s[nt][j] - m[nt][j & 1]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                l[nt][i] += p[i] + p[2 + i];
                pz[nt][i] = fmaf(p[i], zv[0], fmaf(p[2 + i], zv[1], pz[nt][i]));
            }
            pf[nt][0] = movmatrix(half2_bits(p[0] * w0, p[1] * w0));
            pf[nt][1] = movmatrix(half2_bits(p[2] * w1, p[3] * w1));
        }
        // ---- values: words of tokens t, t + 4, t + 8, t + 12 of this warp's 16
        uint32_t vw[4][VW];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            if constexpr (VW == 2) {
                const uint2 x = *(const uint2*)(stg + v_off + r * 4 * (D / 2));
                vw[r][0] = x.x, vw[r][1] = x.y;
            } else {
                vw[r][0] = *(const uint32_t*)(stg + v_off + r * 4 * (D / 2));
            }
        }
#pragma unroll
        for (int w = 0; w < VW; ++w) {
            // pairs of tokens: (t, t + 4) and (t + 8, t + 12); even values in the low halves, odd ones in the high
            const uint32_t e0 = __byte_perm(vw[0][w], vw[1][w], 0x5410), d0 = __byte_perm(vw[0][w], vw[1][w], 0x7632);
            const uint32_t e1 = __byte_perm(vw[2][w], vw[3][w], 0x5410), d1 = __byte_perm(vw[2][w], vw[3][w], 0x7632);
            const uint32_t e0s = e0 >> 8, d0s = d0 >> 8, e1s = e1 >> 8, d1s = d1 >> 8;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                mma_16816(o[nt][4 * w], e0 & 0x000F000Fu, d0 & 0x000F000Fu, e1 & 0x000F000Fu, d1 & 0x000F000Fu, pf[nt][0], pf[nt][1]);
                mma_16816(o[nt][4 * w + 1], e0 & 0x00F000F0u, d0 & 0x00F000F0u, e1 & 0x00F000F0u, d1 & 0x00F000F0u, pf[nt][0], pf[nt][1]);
                mma_16816(o[nt][4 * w + 2], e0s & 0x000F000Fu, d0s & 0x000F000Fu, e1s & 0x000F000Fu, d1s & 0x000F000Fu, pf[nt][0], pf[nt][1]);
                mma_16816(o[nt][4 * w + 3], e0s & 0x00F000F0u, d0s & 0x00F000F0u, e1s & 0x00F000F0u, d1s & 0x00F000F0u, pf[nt][0], pf[nt][1]);
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.empty[st]);

        if (in.flags & kLast) {
            const int rows = q_len * a.group;
            const bool whole = (in.flags & kWholeStart) && (in.flags & kWholeEnd);
            float* part = part_of(parts, blockIdx.x, (in.flags & kWholeStart) ? 1 : 0, 8 * NT, D);
            const float unit = 16777216.f / vs;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                if (nt * 8 >= rows) break;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float ls = l[nt][i], ps = pz[nt][i];
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) {
                        ls += __shfl_xor_sync(QMOE_FULL_MASK, ls, d);
                        ps += __shfl_xor_sync(QMOE_FULL_MASK, ps, d);
                    }
                    const int row = 2 * t + i;
                    if (g == 0) sh.m[warp][row] = m[nt][i], sh.l[warp][row] = ls;
                    // values 8w + 2x, 8w + 2x + 1 of word w = VW g + (tile / 4)
#pragma unroll
                    for (int x = 0; x < 4 * VW; ++x) {
                        const float un = (x & 1) ? unit * 0.0625f : unit;
                        *(float2*)&sh.red[warp][row][8 * VW * g + 2 * x] =
                            make_float2(fmaf(o[nt][x][i], un, ps), fmaf(o[nt][x][2 + i], un, ps));
                    }
                }
                asm volatile("bar.sync 1, %0;" ::"n"(32 * kConsumers) : "memory");
                {
                    const int row = tid >> 4, d0 = (tid & 15) * (D / 16), r = nt * 8 + row;
                    float mm = sh.m[0][row];
#pragma unroll
                    for (int w = 1; w < kConsumers; ++w) mm = fmaxf(mm, sh.m[w][row]);
                    float ll = 0.f, acc[D / 16] = {};
#pragma unroll
                    for (int w = 0; w < kConsumers; ++w) {
                        const float fw = ex2(sh.m[w][row] - mm);
                        ll = fmaf(fw, sh.l[w][row], ll);
#pragma unroll
                        for (int d = 0; d < D / 16; ++d) acc[d] = fmaf(fw, sh.red[w][row][d0 + d], acc[d]);
                    }
                    if (r < rows) {
                        if (whole) {
                            const float inv = ll > 0.f ? 1.f / ll : (ll == 0.f ? 0.f : ll);
                            const int n = r / a.group, h = in.kh * a.group + r - n * a.group;
                            uint32_t* dst = (uint32_t*)(a.out + ((int64_t)(q0 + n) * a.n_q_heads + h) * D + d0);
#pragma unroll
                            for (int d = 0; d < D / 16; d += 2)
                                dst[d / 2] = (uint32_t)f32_to_bf16(acc[d] * inv) | ((uint32_t)f32_to_bf16(acc[d + 1] * inv) << 16);
                        } else {
                            float* dst = part + (size_t)r * D + d0;
#pragma unroll
                            for (int d = 0; d < D / 16; d += 4) *(float4*)(dst + d) = make_float4(acc[d], acc[d + 1], acc[d + 2], acc[d + 3]);
                            if ((tid & 15) == 0) *(float2*)(part + (size_t)8 * NT * D + 2 * r) = make_float2(mm, ll);
                        }
                    }
                }
                asm volatile("bar.sync 1, %0;" ::"n"(32 * kConsumers) : "memory");
            }
        }
    }
}

// Joins the parts of items that several blocks of decode_kernel shared.  One block per (request, kv head).
constexpr int kCombineThreads = 128;

template <int D>
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(AttnArgs a, int max_rows, int n_ctas, const float* parts) {
    const int b = blockIdx.x / a.cache.n_kv_heads, kh = blockIdx.x - b * a.cache.n_kv_heads;
    long long chunk;
    const Found f = scan_requests<kCombineThreads>(a, max_rows, b, true, n_ctas, 0, &chunk, false);
    int t0;
    const int n = tiles_of(a, b, max_rows, &t0, false);
    if (n == 0) return;
    const long long u0 = f.before + (long long)kh * n, u1 = u0 + n;
    const int c0 = (int)(u0 / chunk), c1 = (int)((u1 - 1) / chunk);
    if (c0 == c1) return;
    asm volatile("griddepcontrol.wait;" ::: "memory");      // the parts are written by the kernel before
    const int q0 = a.q_start[b], rows = (a.q_start[b + 1] - q0) * a.group;
    for (int i = threadIdx.x; i < rows * (D / 4); i += kCombineThreads) {
        const int r = i / (D / 4), d0 = (i - r * (D / 4)) * 4;
        float mm = kNoMax, ll = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = c0; c <= c1; ++c) {
            const float* p = part_of((float*)parts, c, u0 >= (long long)c * chunk ? 1 : 0, max_rows, D);
            const float2 ml = *(const float2*)(p + (size_t)max_rows * D + 2 * r);
            const float4 x = *(const float4*)(p + (size_t)r * D + d0);
            const float m2 = fmaxf(mm, ml.x), fa = ex2(mm - m2), fb = ex2(ml.x - m2);
            mm = m2;
            ll = ll * fa + ml.y * fb;
            acc.x = acc.x * fa + x.x * fb, acc.y = acc.y * fa + x.y * fb;
            acc.z = acc.z * fa + x.z * fb, acc.w = acc.w * fa + x.w * fb;
        }
        const float inv = ll > 0.f ? 1.f / ll : (ll == 0.f ? 0.f : ll);
        const int n_ = r / a.group, h = kh * a.group + r - n_ * a.group;
        uint2 w;
        w.x = (uint32_t)f32_to_bf16(acc.x * inv) | ((uint32_t)f32_to_bf16(acc.y * inv) << 16);
        w.y = (uint32_t)f32_to_bf16(acc.z * inv) | ((uint32_t)f32_to_bf16(acc.w * inv) << 16);
        *(uint2*)(a.out + ((int64_t)(q0 + n_) * a.n_q_heads + h) * D + d0) = w;
    }
}

// A warp per (query, head): a lane per key for the scores, head_dim / 32 values a lane for the sums.
template <int D>
__global__ void __launch_bounds__(128) attention_kernel(AttnArgs a, int max_rows) {
    __shared__ float qs[4][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = blockIdx.x * 4 + warp;
    const int b = blockIdx.z;
    int q0, q_len, len;
    if (!request(a, b, &q0, &q_len, &len, true) || q_len * a.group <= max_rows) return;
    const int n = blockIdx.y;
    if (n >= q_len || h >= a.n_q_heads) return;
    const int pos = a.causal ? len - q_len + n : len - 1;
    const int end = min(pos + 1, len);
    const int begin = a.window ? max(0, pos - a.window + 1) : 0;
    const int64_t row = ((int64_t)(q0 + n) * a.n_q_heads + h) * D;
    for (int i = lane; i < D; i += 32) qs[warp][i] = bf16_to_f32(a.q[row + i]);
    __syncwarp();
    const int kh = h / a.group, P = 1 << a.cache.page_shift;
    float m = -INFINITY, l = 0.f, o[D / 32] = {};
    for (int j0 = begin; j0 < end; j0 += 32) {
        const int j = j0 + lane;
        float s = -INFINITY;
        const unsigned char* hp = nullptr;
        if (j < end) {
            const int blk = j >> a.cache.page_shift;
            const int page = blk < a.max_blocks ? a.table[(int64_t)b * a.max_blocks + blk] : -1;
            if (page < 0 || page >= a.cache.n_pages) {
                attn_set_error(QMOE_EINVAL);
            } else {
                hp = kv4::head_ptr(a.cache, page, kh);
                const int r = j & (P - 1);
                float dot = 0.f, sum = 0.f;
                for (int w = 0; w < D / 8; ++w) {
                    const uint32_t word = ((const uint32_t*)hp)[r * (D / 8) + w];
                    for (int i = 0; i < 8; ++i) {
                        const float qv = qs[warp][8 * w + i];
                        dot += qv * (float)((word >> (4 * (i >> 1) + 16 * (i & 1))) & 15u);
                        sum += qv;
                    }
                }
                const uint32_t sz = ((const uint32_t*)(hp + P * D))[r];
                s = (f16_to_f32((uint16_t)sz) * dot + f16_to_f32((uint16_t)(sz >> 16)) * sum) * a.scale;
            }
        }
        float mx = s;
        for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(QMOE_FULL_MASK, mx, d));
        const float m2 = fmaxf(m, mx);
        if (m2 == -INFINITY) continue;
        const float f = expf(m - m2), p = expf(s - m2);
        m = m2;
        l = l * f + warp_sum(p);
        for (int i = 0; i < D / 32; ++i) o[i] *= f;
        for (int t = 0; t < min(32, end - j0); ++t) {
            const float pt = __shfl_sync(QMOE_FULL_MASK, p, t);
            const unsigned char* ht = (const unsigned char*)__shfl_sync(QMOE_FULL_MASK, (unsigned long long)hp, t);
            if (!ht) continue;
            const int r = P + ((j0 + t) & (P - 1));
            const uint32_t sz = ((const uint32_t*)(ht + P * D))[r];
            const float vs = f16_to_f32((uint16_t)sz), vz = f16_to_f32((uint16_t)(sz >> 16));
            for (int i = 0; i < D / 32; ++i) {
                const int d = lane + 32 * i;
                const uint32_t word = ((const uint32_t*)ht)[r * (D / 8) + d / 8];
                o[i] += pt * fmaf(vs, (float)((word >> (4 * ((d & 7) >> 1) + 16 * (d & 1))) & 15u), vz);
            }
        }
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    for (int i = 0; i < D / 32; ++i) a.out[row + lane + 32 * i] = f32_to_bf16(o[i] * inv);
}

// Query rows (a multiple of 8) that the few-row path takes per (request, kv head): the batch's largest where 32
// hold it, else enough for a single query (requests with more go to the tiles); 0 for groups above 32.
int decode_rows(int group, int max_q) {
    const long long all = (long long)group * max_q;
    const int rows = all <= 32 ? (int)all : group <= 32 ? group : 0;
    return rows == 0 ? 0 : rows <= 8 ? 8 : rows <= 16 ? 16 : 32;
}

// Blocks of the few-row path: as many as fit on the device, no more than tiles.
long long decode_blocks(int rows, int B, int n_kv_heads, int max_kv) {
    const long long fit = (long long)qmoe::sm_count() * (rows <= 8 ? 4 : rows <= 16 ? 3 : 2);
    return std::min(fit, (long long)B * n_kv_heads * std::max(1, (max_kv + kTile - 1) / kTile));
}

size_t decode_ws(int rows, int head_dim) {
    if (rows == 0) return 0;
    const size_t fit = (size_t)qmoe::sm_count() * (rows <= 8 ? 4 : rows <= 16 ? 3 : 2);
    return fit * 2 * rows * (head_dim + 2) * sizeof(float);
}

template <int D, int NT>
int launch_decode(const AttnArgs& a, float* parts, cudaStream_t st) {
    const int smem = (int)sizeof(DecodeShared<D, NT>) + 128;
    int rc = qmoe::smem_attr((const void*)decode_kernel<D, NT>, smem, "attention attr");
    if (rc) return rc;
    const long long blocks = decode_blocks(8 * NT, a.B, a.cache.n_kv_heads, a.max_kv);
    decode_kernel<D, NT><<<(unsigned)blocks, kDecodeThreads, smem, st>>>(a, 8 * NT, parts);
    if ((rc = qmoe::launch_check("decode_kernel"))) return rc;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)(a.B * a.cache.n_kv_heads));
    cfg.blockDim = dim3(kCombineThreads);
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return qmoe::cuda_check(cudaLaunchKernelEx(&cfg, combine_kernel<D>, a, 8 * NT, (int)blocks, (const float*)parts),
                            "combine_kernel");
}

int check_sizes(const char* who, int B, int n_q_heads, int n_kv_heads, int head_dim, int n_q_tokens, int max_q, int max_kv) {
    if (head_dim != 64 && head_dim != 128) return qmoe::fail(QMOE_EUNSUPPORTED, std::string(who) + ": head_dim must be 64 or 128");
    if (B < 0 || n_q_tokens < 0 || max_q < 0 || max_kv < 0 || n_kv_heads < 1 || n_q_heads < n_kv_heads ||
        n_q_heads % n_kv_heads)
        return qmoe::fail(QMOE_EINVAL, std::string(who) + ": bad sizes (n_q_heads must be a multiple of n_kv_heads)");
    if (n_q_heads / n_kv_heads > 128)
        return qmoe::fail(QMOE_EUNSUPPORTED, std::string(who) + ": more than 128 query heads per kv head");
    return QMOE_OK;
}

}  // namespace

namespace qmoe {
int kv4_attention_take_error() {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_kv4_attention_error, sizeof(int)) != cudaSuccess) return QMOE_ECUDA;
    const int z = 0;
    if (cudaMemcpyToSymbol(g_kv4_attention_error, &z, sizeof(int)) != cudaSuccess) return QMOE_ECUDA;
    return v;
}
}  // namespace qmoe

extern "C" int kv4_attention_ws_size(int B, int n_q_heads, int n_kv_heads, int head_dim, int n_q_tokens, int max_q,
                                     int max_kv, size_t* bytes) {
    qmoe::clear_error();
    if (!bytes) return qmoe::fail(QMOE_EINVAL, "kv4_attention_ws_size: NULL output");
    const int rc = check_sizes("kv4_attention_ws_size", B, n_q_heads, n_kv_heads, head_dim, n_q_tokens, max_q, max_kv);
    if (rc) return rc;
    *bytes = decode_ws(decode_rows(n_q_heads / n_kv_heads, max_q), head_dim);
    return QMOE_OK;
}

extern "C" int kv4_attention(const kv4_cache* cache, const void* q, int n_q_tokens, int n_q_heads, const int32_t* q_start,
                             const int32_t* kv_len, int B, const int32_t* table, int max_blocks, int max_q, int max_kv,
                             float scale, int causal, int window, void* out, void* workspace, size_t ws_bytes,
                             void* stream) {
    qmoe::clear_error();
    AttnArgs a{};
    int rc = kv4::view_of(cache, "kv4_attention", &a.cache);
    if (rc) return rc;
    rc = check_sizes("kv4_attention", B, n_q_heads, cache->n_kv_heads, cache->head_dim, n_q_tokens, max_q, max_kv);
    if (rc) return rc;
    if (max_blocks < 0 || window < 0) return qmoe::fail(QMOE_EINVAL, "kv4_attention: negative max_blocks or window");
    if (B == 0 || n_q_tokens == 0 || max_q == 0) return QMOE_OK;
    if (!q || !out || !q_start || !kv_len || (max_blocks > 0 && !table)) return qmoe::fail(QMOE_EINVAL, "kv4_attention: NULL pointer");
    if (!kv4::aligned16(q) || !kv4::aligned16(out)) return qmoe::fail(QMOE_EINVAL, "kv4_attention: pointer not 16-byte aligned");
    a.q = (const uint16_t*)q, a.out = (uint16_t*)out, a.q_start = q_start, a.kv_len = kv_len, a.table = table;
    a.B = B, a.n_q_tokens = n_q_tokens, a.n_q_heads = n_q_heads, a.group = n_q_heads / cache->n_kv_heads;
    a.max_blocks = max_blocks, a.max_q = max_q, a.max_kv = max_kv, a.scale = scale, a.causal = causal ? 1 : 0, a.window = window;
    cudaStream_t st = (cudaStream_t)stream;
    const int rows = decode_rows(a.group, max_q), D = cache->head_dim;
    if (ws_bytes < decode_ws(rows, D)) return qmoe::fail(QMOE_ECAPACITY, "kv4_attention: workspace too small");
    if (rows > 0 && (!workspace || !kv4::aligned16(workspace)))
        return qmoe::fail(QMOE_EINVAL, "kv4_attention: workspace NULL or not 16-byte aligned");
    if ((long long)B * cache->n_kv_heads > 0x7FFFFFFFLL) return qmoe::fail(QMOE_EINVAL, "kv4_attention: batch too large");
    float* parts = (float*)workspace;
    if (rows == 8) rc = D == 128 ? launch_decode<128, 1>(a, parts, st) : launch_decode<64, 1>(a, parts, st);
    if (rows == 16) rc = D == 128 ? launch_decode<128, 2>(a, parts, st) : launch_decode<64, 2>(a, parts, st);
    if (rows == 32) rc = D == 128 ? launch_decode<128, 4>(a, parts, st) : launch_decode<64, 4>(a, parts, st);
    if (rc || (long long)a.group * max_q <= rows) return rc;
    const dim3 grid((n_q_heads + 3) / 4, max_q, B);
    if (D == 128)
        attention_kernel<128><<<grid, 128, 0, st>>>(a, rows);
    else
        attention_kernel<64><<<grid, 128, 0, st>>>(a, rows);
    return qmoe::launch_check("kv4_attention");
}
