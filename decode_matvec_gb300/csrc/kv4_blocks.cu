// Choice of the blocks that a query attends to: bounds of the keys of each block of the 4-bit paged cache, scores of the
// blocks by them, and the best blocks of each query token and kv head.

#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "kv4_common.cuh"

namespace {

__device__ int g_kv4_blocks_error;

__device__ __forceinline__ void blocks_set_error(int code) { atomicCAS(&g_kv4_blocks_error, 0, code); }

// ---------------------------------------------------------------- bounds of a block's keys
struct BoundsArgs {
    kv4::CacheView cache;
    int8_t* codes;
    float* steps;
    const int32_t* slots;
    int n;
};

// A warp takes the tokens of one kv head that stand `span` from t0 on and bounds the block of each that is the last new one
// of its block: L = head_dim / 8 lanes a row of codes (a word, 8 channels, a lane), 32 / L rows at a time.
template <int L>
__global__ void __launch_bounds__(128) bounds_kernel(BoundsArgs a, int span) {
    constexpr int G = 32 / L, D = L * 8;
    const int lane = threadIdx.x & 31, gl = lane & (L - 1), g = lane / L;
    const int h = blockIdx.y;
    const int64_t t0 = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 5)) * span;
    if (t0 >= a.n) return;
    const int shift = a.cache.page_shift, P = 1 << shift;
    int slot = -1;
    bool last = false;
    if (lane < span && t0 + lane < a.n) {
        slot = a.slots[t0 + lane];
        if (slot < -1 || (slot >> shift) >= a.cache.n_pages) {
            blocks_set_error(QMOE_EINVAL);
            slot = -1;
        }
        const int next = t0 + lane + 1 < a.n ? a.slots[t0 + lane + 1] : -1;
        last = slot >= 0 && (next != slot + 1 || (next & (P - 1)) == 0);
    }
    for (unsigned todo = __ballot_sync(QMOE_FULL_MASK, last); todo; todo &= todo - 1) {
        const int s = __shfl_sync(QMOE_FULL_MASK, slot, __ffs(todo) - 1), page = s >> shift, count = (s & (P - 1)) + 1;
        const unsigned char* hp = kv4::head_ptr(a.cache, page, h);
        const uint32_t* words = (const uint32_t*)hp;
        const __half2* pairs = (const __half2*)(hp + (size_t)P * D);
        float lo[8], hi[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) lo[i] = INFINITY, hi[i] = -INFINITY;
#pragma unroll 4
        for (int r = g; r < count; r += G) {
            const uint32_t w = words[r * L + gl];
            const float2 sz = __half22float2(pairs[r]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float v = fmaf(sz.x, (float)((w >> (4 * (i >> 1) + 16 * (i & 1))) & 15u), sz.y);
                lo[i] = fminf(lo[i], v), hi[i] = fmaxf(hi[i], v);
            }
        }
        float big = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
#pragma unroll
            for (int d = L; d < 32; d <<= 1) {
                lo[i] = fminf(lo[i], __shfl_xor_sync(QMOE_FULL_MASK, lo[i], d));
                hi[i] = fmaxf(hi[i], __shfl_xor_sync(QMOE_FULL_MASK, hi[i], d));
            }
            big = fmaxf(big, fmaxf(fabsf(lo[i]), fabsf(hi[i])));
        }
#pragma unroll
        for (int d = L / 2; d > 0; d >>= 1) big = fmaxf(big, __shfl_xor_sync(QMOE_FULL_MASK, big, d));
        // big = m 2^e with m in [64, 127], or [63.5, 64) one power up; the quotients by a power of two are exact
        int e = (int)(__float_as_uint(big) >> 23) - 127 - 6;
        if (big > 127.f * __int_as_float((e + 127) << 23)) ++e;
        const float step = big > 0.f ? __int_as_float((e + 127) << 23) : 0.f, inv = big > 0.f ? __int_as_float((127 - e) << 23) : 0.f;
        const int64_t rec = (int64_t)page * a.cache.n_kv_heads + h;
        if (g < 2) {
            uint32_t w[2] = {0, 0};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int q = g == 0 ? __float2int_ru(hi[i] * inv) : __float2int_rd(lo[i] * inv);
                w[i >> 2] |= (uint32_t)(min(max(q, -127), 127) & 255) << (8 * (i & 3));
            }
            *(uint2*)(a.codes + (rec * 2 + g) * D + gl * 8) = make_uint2(w[0], w[1]);
        }
        if (lane == 0) a.steps[rec] = step;
    }
}

// ---------------------------------------------------------------- scores of the blocks
struct SelectArgs {
    const int8_t* codes;
    const float* steps;
    const uint16_t* q;
    const int32_t *q_start, *kv_len, *table;
    int32_t* sel;
    float* scores;         // [token][kv head][max_seen]
    int B, n, n_kv, group, n_pages, max_blocks, page_shift, max_kv, max_seen, top, first, last, bits;
};

// Blocks that query token t sees (-1: the token belongs to no request), and its request.
__device__ __forceinline__ int blocks_seen(const SelectArgs& a, int t, int* b, bool report) {
    *b = kv4::request_of(a.q_start, a.B, t);
    if (*b < 0) return -1;
    const int kv = a.kv_len[*b];
    if (kv < 0 || kv > a.max_kv) {
        if (report) blocks_set_error(kv < 0 ? QMOE_EINVAL : QMOE_ECAPACITY);
        return 0;
    }
    const int64_t pos = (int64_t)kv - ((int64_t)a.q_start[*b + 1] - t);
    return pos < 0 ? 0 : (int)(pos >> a.page_shift) + 1;
}

// The 16-bit products of 4 channels: acc + c[0] q0.lo + c[1] q0.hi + c[2] q1.lo + c[3] q1.hi.
__device__ __forceinline__ int dot4(uint32_t c, uint32_t q0, uint32_t q1, int acc) {
    acc = __dp2a_lo((int)q0, (int)c, acc);
    return __dp2a_hi((int)q1, (int)c, acc);
}

constexpr int kScoreThreads = 256, kScoreBlocks = 64;     // blocks of the cache that a thread block scores

// q as bf16, NaN as 0, infinities as the largest finite value
__device__ __forceinline__ float query_value(uint32_t bits) {
    const float v = __uint_as_float(bits << 16);
    return v == v ? fminf(fmaxf(v, -3.3895313892515355e38f), 3.3895313892515355e38f) : 0.f;
}

// A thread block scores kScoreBlocks blocks of one query token for every kv head.  L = 2 D / 16 lanes take a record (hi and lo
// codes), 16 codes a lane, against the group's summed queries, which a lane keeps in registers for one kv head.
template <int D>
__global__ void __launch_bounds__(kScoreThreads) score_kernel(SelectArgs a, int chunks) {
    constexpr int L = D / 8, SLOTS = kScoreThreads / L;     // groups of lanes
    const int t = blockIdx.x / chunks, chunk = blockIdx.x - t * chunks;
    int b;
    const int seen = blocks_seen(a, t, &b, chunk == 0 && threadIdx.x == 0);
    const int j0 = chunk * kScoreBlocks, j1 = min(j0 + kScoreBlocks, seen);
    if (seen <= a.top || j0 >= j1) return;      // few blocks are all taken
    const int sl = threadIdx.x / L, gl = threadIdx.x - sl * L;
    const int parts = max(1, SLOTS / a.n_kv);
    if (sl >= a.n_kv * parts) return;           // (whole groups of lanes: the shuffles below stay within a group)
    const unsigned mask = (L == 16 ? 0xFFFFu : 0xFFu) << (threadIdx.x & 31 & ~(L - 1));
    for (int h = sl % a.n_kv; h < a.n_kv; h += SLOTS) {
        // this lane's 16 channels: hi of 16 gl .., or lo
        const int d0 = (gl * 16) % D;
        const bool low = gl * 16 >= D;
        const uint16_t* q = a.q + ((int64_t)t * a.n_kv + h) * a.group * D + d0;
        float big = 0.f;
        for (int g = 0; g < a.group; ++g) {
            const uint4 x[2] = {((const uint4*)(q + g * D))[0], ((const uint4*)(q + g * D))[1]};
            const uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
#pragma unroll
            for (int i = 0; i < 8; ++i) big = fmaxf(big, fmaxf(fabsf(query_value(w[i] & 0xFFFFu)), fabsf(query_value(w[i] >> 16))));
        }
#pragma unroll
        for (int d = L / 2; d > 0; d >>= 1) big = fmaxf(big, __shfl_xor_sync(mask, big, d));
        // largest magnitude to [2^(bits-1), 2^bits): times 2^(bits - 1 - exponent), in two factors of normal size
        const int up = a.bits - 1 - (ilogbf(big > 0.f ? big : 1.f)), limit = (1 << a.bits) - 1;
        const float f1 = __int_as_float((min(up, 100) + 127) << 23), f2 = __int_as_float((max(up - 100, 0) + 127) << 23);
        int sum[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) sum[i] = 0;
        for (int g = 0; g < a.group; ++g) {
            const uint4 x[2] = {((const uint4*)(q + g * D))[0], ((const uint4*)(q + g * D))[1]};
            const uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float v = query_value(i & 1 ? w[i >> 1] >> 16 : w[i >> 1] & 0xFFFFu);
                const int r = min(max(__float2int_rn(v * f1 * f2), -limit), limit);
                sum[i] += low ? min(r, 0) : max(r, 0);
            }
        }
        uint32_t pk[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) pk[i] = __byte_perm((uint32_t)sum[2 * i], (uint32_t)sum[2 * i + 1], 0x5410);
        float* out = a.scores + ((int64_t)t * a.n_kv + h) * a.max_seen;
#pragma unroll 4
        for (int j = j0 + sl / a.n_kv; j < j1; j += parts) {
            const int page = j < a.max_blocks ? a.table[(int64_t)b * a.max_blocks + j] : -1;
            float score = -INFINITY;
            if (page >= 0 && page < a.n_pages) {
                const int64_t rec = (int64_t)page * a.n_kv + h;
                const uint4 c = *(const uint4*)(a.codes + rec * (2 * D) + gl * 16);
                int acc = dot4(c.x, pk[0], pk[1], 0);
                acc = dot4(c.y, pk[2], pk[3], acc);
                acc = dot4(c.z, pk[4], pk[5], acc);
                acc = dot4(c.w, pk[6], pk[7], acc);
#pragma unroll
                for (int d = L / 2; d > 0; d >>= 1) acc += __shfl_xor_sync(mask, acc, d);
                score = __fmul_rn((float)acc, a.steps[rec]);
            } else if (gl == 0 && h == 0) {
                blocks_set_error(QMOE_EINVAL);
            }
            if (gl == 0) out[j] = score;
        }
    }
}

// ---------------------------------------------------------------- the best blocks
constexpr int kPickThreads = 256;

__device__ __forceinline__ uint32_t score_key(float v) {
    const uint32_t u = __float_as_uint(v + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ int block_sum(int v, int* buf) {
    v = warp_sum_int(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    int s = 0;
#pragma unroll
    for (int w = 0; w < kPickThreads / 32; ++w) s += buf[w];
    return s;
}

// A thread block writes the list of one (token, kv head): the key of the last block taken by bisection, then the blocks above
// it and the first ones at it, in order (each warp those of an equal run of the blocks).
__global__ void __launch_bounds__(kPickThreads) pick_kernel(SelectArgs a) {
    __shared__ int buf[kPickThreads / 32], above_s[kPickThreads / 32], equal_s[kPickThreads / 32];
    const int t = blockIdx.x / a.n_kv, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int b;
    const int seen = blocks_seen(a, t, &b, false);
    if (seen < 0) return;
    int32_t* sel = a.sel + (int64_t)blockIdx.x * a.top;
    if (seen <= a.top) {
        for (int i = threadIdx.x; i < a.top; i += kPickThreads) sel[i] = i < seen ? i : -1;
        return;
    }
    const float* scores = a.scores + (int64_t)blockIdx.x * a.max_seen;
    const int lo = a.first, hi = seen - a.last, want = a.top - a.first - a.last;
    for (int i = threadIdx.x; i < a.first; i += kPickThreads) sel[i] = i;
    for (int i = threadIdx.x; i < a.last; i += kPickThreads) sel[a.top - a.last + i] = hi + i;
    if (want == 0) return;
    // largest key k with at least `want` keys >= k
    uint32_t key = 0;
    for (int bit = 31; bit >= 0; --bit) {
        const uint32_t probe = key | 1u << bit;
        int c = 0;
        for (int j = lo + threadIdx.x; j < hi; j += kPickThreads) c += score_key(scores[j]) >= probe;
        if (block_sum(c, buf) >= want) key = probe;
    }
    const int per = ((hi - lo + kPickThreads / 32 - 1) / (kPickThreads / 32) + 31) & ~31;
    const int w0 = min(lo + warp * per, hi), w1 = min(w0 + per, hi);
    int above = 0, equal = 0;
    for (int j = w0 + lane; j < w1; j += 32) {
        const uint32_t k = score_key(scores[j]);
        above += k > key, equal += k == key;
    }
    above = warp_sum_int(above), equal = warp_sum_int(equal);
    if (lane == 0) above_s[warp] = above, equal_s[warp] = equal;
    __syncthreads();
    int all_above = 0, above_before = 0, equal_before = 0;
#pragma unroll
    for (int w = 0; w < kPickThreads / 32; ++w) {
        all_above += above_s[w];
        if (w < warp) above_before += above_s[w], equal_before += equal_s[w];
    }
    const int room = want - all_above;          // of the equal ones
    for (int j0 = w0; j0 < w1; j0 += 32) {
        const int j = j0 + lane;
        const uint32_t k = j < w1 ? score_key(scores[j]) : 0u;
        const unsigned over = __ballot_sync(QMOE_FULL_MASK, j < w1 && k > key), same = __ballot_sync(QMOE_FULL_MASK, j < w1 && k == key);
        const unsigned before = (1u << lane) - 1;
        const int n_same = equal_before + __popc(same & before);
        const int at = above_before + __popc(over & before) + min(n_same, room);
        if (((over >> lane) & 1) || (((same >> lane) & 1) && n_same < room)) sel[a.first + at] = j;
        above_before += __popc(over), equal_before += __popc(same);
    }
}

int check_bounds(const kv4_bounds* b, const char* who) {
    const std::string name(who);
    if (!b || !b->codes || !b->steps) return qmoe::fail(QMOE_EINVAL, name + ": NULL bounds");
    if (b->page_size != 16 && b->page_size != 32 && b->page_size != 64) return qmoe::fail(QMOE_EINVAL, name + ": page_size must be 16, 32 or 64");
    if (b->head_dim != 64 && b->head_dim != 128) return qmoe::fail(QMOE_EUNSUPPORTED, name + ": head_dim must be 64 or 128");
    if (b->n_kv_heads < 1 || b->n_kv_heads > 1024 || b->n_pages < 1 || (int64_t)b->n_pages * b->page_size > 0x7FFFFFFFLL)
        return qmoe::fail(QMOE_EINVAL, name + ": n_kv_heads outside 1 .. 1024, or n_pages * page_size outside int32");
    if (!kv4::aligned16(b->codes) || ((uintptr_t)b->steps & 3)) return qmoe::fail(QMOE_EINVAL, name + ": codes not 16-byte aligned, or steps not 4-byte");
    return QMOE_OK;
}

int shift_of(int page_size) { return page_size == 16 ? 4 : page_size == 32 ? 5 : 6; }

// Scores of a (token, kv head), rounded up to 16 bytes.
int64_t score_row(int page_size, int max_kv) { return (((int64_t)max_kv + page_size - 1) / page_size + 3) & ~(int64_t)3; }

}  // namespace

namespace qmoe {
int kv4_blocks_take_error() {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_kv4_blocks_error, sizeof(int)) != cudaSuccess) return QMOE_ECUDA;
    if (v == 0) return 0;      // nothing to clear
    const int z = 0;
    if (cudaMemcpyToSymbol(g_kv4_blocks_error, &z, sizeof(int)) != cudaSuccess) return QMOE_ECUDA;
    return v;
}
}  // namespace qmoe

extern "C" int kv4_block_bounds(const kv4_cache* cache, const kv4_bounds* bounds, const int32_t* slots, int n, void* stream) {
    qmoe::clear_error();
    BoundsArgs a{};
    int rc = kv4::view_of(cache, "kv4_block_bounds", &a.cache);
    if (rc || (rc = check_bounds(bounds, "kv4_block_bounds"))) return rc;
    if (bounds->n_pages != cache->n_pages || bounds->page_size != cache->page_size || bounds->n_kv_heads != cache->n_kv_heads ||
        bounds->head_dim != cache->head_dim)
        return qmoe::fail(QMOE_EINVAL, "kv4_block_bounds: the bounds have other sizes than the cache");
    if (n < 0 || (n > 0 && !slots)) return qmoe::fail(QMOE_EINVAL, "kv4_block_bounds: negative n or NULL slots");
    if (n == 0) return QMOE_OK;
    a.codes = (int8_t*)bounds->codes, a.steps = bounds->steps, a.slots = slots, a.n = n;
    // few tokens: a warp each, so that blocks are bounded side by side; many: a warp a run of 32
    const int span = (int64_t)n * cache->n_kv_heads <= (int64_t)qmoe::sm_count() * 64 ? 1 : 32;
    const dim3 grid((unsigned)(((int64_t)n + 4 * span - 1) / (4 * span)), (unsigned)cache->n_kv_heads);
    if (cache->head_dim == 128) bounds_kernel<16><<<grid, 128, 0, (cudaStream_t)stream>>>(a, span);
    else bounds_kernel<8><<<grid, 128, 0, (cudaStream_t)stream>>>(a, span);
    return qmoe::launch_check("kv4_block_bounds");
}

extern "C" int kv4_select_blocks_ws_size(int n_q_tokens, int n_kv_heads, int page_size, int max_kv, size_t* bytes) {
    qmoe::clear_error();
    if (!bytes) return qmoe::fail(QMOE_EINVAL, "kv4_select_blocks_ws_size: NULL output");
    if (n_q_tokens < 0 || n_kv_heads < 1 || max_kv < 0 || (page_size != 16 && page_size != 32 && page_size != 64))
        return qmoe::fail(QMOE_EINVAL, "kv4_select_blocks_ws_size: bad sizes (page_size 16, 32 or 64)");
    *bytes = (size_t)n_q_tokens * n_kv_heads * (size_t)score_row(page_size, max_kv) * sizeof(float);
    return QMOE_OK;
}

extern "C" int kv4_select_blocks(const kv4_bounds* bounds, const void* q, int n_q_tokens, int n_q_heads, const int32_t* q_start,
                                 const int32_t* kv_len, int B, const int32_t* table, int max_blocks, int max_kv, int top, int first,
                                 int last, int32_t* sel, void* workspace, size_t ws_bytes, void* stream) {
    qmoe::clear_error();
    int rc = check_bounds(bounds, "kv4_select_blocks");
    if (rc) return rc;
    const int n_kv = bounds->n_kv_heads;
    if (B < 0 || n_q_tokens < 0 || max_kv < 0 || max_kv > 0x7FFFFFFF - 127 || max_blocks < 0 || n_q_heads < n_kv || n_q_heads % n_kv)
        return qmoe::fail(QMOE_EINVAL, "kv4_select_blocks: bad sizes (n_q_heads must be a multiple of n_kv_heads)");
    if (n_q_heads / n_kv > 128) return qmoe::fail(QMOE_EUNSUPPORTED, "kv4_select_blocks: more than 128 query heads per kv head");
    if (top < 1 || top > 65536 || first < 0 || last < 0 || (int64_t)first + last > top)
        return qmoe::fail(QMOE_EINVAL, "kv4_select_blocks: need 1 <= top <= 65536 and first + last <= top");
    if (B == 0 || n_q_tokens == 0) return QMOE_OK;
    if (!q || !q_start || !kv_len || !sel || (max_blocks > 0 && !table)) return qmoe::fail(QMOE_EINVAL, "kv4_select_blocks: NULL pointer");
    if (!kv4::aligned16(q)) return qmoe::fail(QMOE_EINVAL, "kv4_select_blocks: q not 16-byte aligned");
    SelectArgs a{};
    const int64_t row = score_row(bounds->page_size, max_kv);
    if (ws_bytes < (size_t)n_q_tokens * n_kv * (size_t)row * sizeof(float)) return qmoe::fail(QMOE_ECAPACITY, "kv4_select_blocks: workspace too small");
    a.codes = (const int8_t*)bounds->codes, a.steps = bounds->steps, a.q = (const uint16_t*)q;
    a.q_start = q_start, a.kv_len = kv_len, a.table = table, a.sel = sel, a.scores = (float*)workspace;
    a.B = B, a.n = n_q_tokens, a.n_kv = n_kv, a.group = n_q_heads / n_kv, a.n_pages = bounds->n_pages, a.max_blocks = max_blocks;
    a.page_shift = shift_of(bounds->page_size), a.max_kv = max_kv, a.max_seen = (int)row, a.top = top, a.first = first, a.last = last;
    a.bits = 15;
    while ((1 << (15 - a.bits)) < a.group) --a.bits;
    cudaStream_t st = (cudaStream_t)stream;
    const int64_t chunks = (row + kScoreBlocks - 1) / kScoreBlocks, blocks = chunks * n_q_tokens;
    if (blocks > 0x7FFFFFFFLL || (int64_t)n_q_tokens * n_kv > 0x7FFFFFFFLL)
        return qmoe::fail(QMOE_EINVAL, "kv4_select_blocks: too many query tokens in one call");
    if (row > top) {
        if (!workspace || !kv4::aligned16(workspace)) return qmoe::fail(QMOE_EINVAL, "kv4_select_blocks: workspace NULL or not 16-byte aligned");
        if (bounds->head_dim == 128) score_kernel<128><<<(unsigned)blocks, kScoreThreads, 0, st>>>(a, (int)chunks);
        else score_kernel<64><<<(unsigned)blocks, kScoreThreads, 0, st>>>(a, (int)chunks);
        if ((rc = qmoe::launch_check("kv4_select_blocks"))) return rc;
    }
    pick_kernel<<<(unsigned)(n_q_tokens * n_kv), kPickThreads, 0, st>>>(a);
    return qmoe::launch_check("kv4_select_blocks");
}
