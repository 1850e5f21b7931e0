// Choice of the blocks that a query attends to: bounds of the keys of each block of the 4-bit paged cache, scores of the
// blocks by them, and the best blocks of each query token and kv head.

#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "kv4_common.cuh"
#include "tc_common.cuh"

namespace {

__device__ int g_kv4_blocks_error;

__device__ __forceinline__ void blocks_set_error(int code) { atomicCAS(&g_kv4_blocks_error, 0, code); }

// Half-precision factors, one rounding to fp32: a's lower and upper halves times b's lower half, plus c.
__device__ __forceinline__ float2 fma_halves(uint32_t a, uint32_t b, float c) {
    float2 r;
    asm("{\n .reg .b16 al, ah, bl, bh;\n mov.b32 {al, ah}, %2;\n mov.b32 {bl, bh}, %3;\n fma.rn.f32.f16 %0, al, bl, %4;\n fma.rn.f32.f16 %1, ah, bl, %4;\n}"
        : "=f"(r.x), "=f"(r.y)
        : "r"(a), "r"(b), "f"(c));
    return r;
}

// ---------------------------------------------------------------- bounds of a block's keys
struct BoundsArgs {
    kv4::CacheView cache;
    int8_t* codes;
    float* steps;
    const int32_t* slots;
    int n;
};

// A thread block takes `span` tokens of one kv head and bounds the block of each that is the last new one of its block.
// L = head_dim / 8 lanes hold a row of codes (a word, 8 channels, a lane); the rows of a block are dealt out over the four
// warps, all of a lane's loads in flight together, and joined in shared memory, where a thread takes a channel.  The instructions bound
// it: 8 of a word's codes made fp32 values, exactly, and compared twice (16 prompts of 777 to 2048 tokens, 8 heads of 128, pages of 64:
// 8.1 us for 12 MB, 2000 instructions a block and head, 60 % of the issue slots; 9.4 us with codes made fp32 and packed fp32 arithmetic,
// 2300 instructions).
constexpr int kBoundsThreads = 128;

template <int L>
__global__ void __launch_bounds__(kBoundsThreads) bounds_kernel(BoundsArgs a, int span) {
    constexpr int D = L * 8, ROWS = kBoundsThreads / L, STEPS = 64 / ROWS, WARPS = kBoundsThreads / 32;
    __shared__ float lo_s[WARPS][D], hi_s[WARPS][D], big_s[WARPS];
    __shared__ int ends[kBoundsThreads], n_ends;
    kv4::depend_wait();
    kv4::depend_launch();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, gl = lane & (L - 1), row = tid / L;
    const int h = blockIdx.y, shift = a.cache.page_shift, P = 1 << shift;
    const int64_t t = (int64_t)blockIdx.x * span + tid;
    if (tid == 0) n_ends = 0;
    __syncthreads();
    if (tid < span && t < a.n) {
        int slot = a.slots[t];
        if (slot < -1 || (slot >> shift) >= a.cache.n_pages) {
            blocks_set_error(QMOE_EINVAL);
            slot = -1;
        }
        const int next = t + 1 < a.n ? a.slots[t + 1] : -1;
        if (slot >= 0 && (next != slot + 1 || (next & (P - 1)) == 0)) ends[atomicAdd(&n_ends, 1)] = slot;
    }
    __syncthreads();
    const int n = n_ends;
    for (int i = 0; i < n; ++i) {
        const int s = ends[i], page = s >> shift, count = (s & (P - 1)) + 1;
        const unsigned char* hp = kv4::head_ptr(a.cache, page, h);
        const uint32_t* words = (const uint32_t*)hp;
        const __half2* pairs = (const __half2*)(hp + (size_t)P * D);
        uint32_t w[STEPS];
        __half2 sz[STEPS];
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
            if ((k & ~1) * ROWS < P) {
                const int r = min(row + k * ROWS, count - 1);
                w[k] = words[r * L + gl], sz[k] = pairs[r];
            }
        }
        // Rows past the block's end repeat a row of it.  A code in the lowest bits of a half is u 2^-24 as a subnormal half, four bits up
        // 16 times that: s u + z comes out 2^-24 or 2^-20 of itself, with the same rounding, and is brought back at the end.
        float lo[8], hi[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) lo[c] = INFINITY, hi[c] = -INFINITY;
#pragma unroll
        for (int k = 0; k < STEPS; k += 2) {
            if (k * ROWS >= P) break;
            float v[2][8];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float z0 = __high2float(sz[k + x]) * (1.f / (1 << 24)), z1 = z0 * 16.f;
                const uint32_t s = *(const uint32_t*)&sz[k + x];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 r = fma_halves((w[k + x] >> (i & 2) * 4) & (i & 1 ? 0x00F000F0u : 0x000F000Fu), s, i & 1 ? z1 : z0);
                    v[x][2 * i] = r.x, v[x][2 * i + 1] = r.y;
                }
            }
#pragma unroll
            for (int c = 0; c < 8; ++c) lo[c] = fminf(fminf(lo[c], v[0][c]), v[1][c]), hi[c] = fmaxf(fmaxf(hi[c], v[0][c]), v[1][c]);
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) {
#pragma unroll
            for (int d = L; d < 32; d <<= 1) {
                lo[c] = fminf(lo[c], __shfl_xor_sync(QMOE_FULL_MASK, lo[c], d));
                hi[c] = fmaxf(hi[c], __shfl_xor_sync(QMOE_FULL_MASK, hi[c], d));
            }
            const float up = c >> 1 & 1 ? (float)(1 << 20) : (float)(1 << 24);
            lo[c] *= up, hi[c] *= up;
        }
        if (lane < L) {
#pragma unroll
            for (int c = 0; c < 8; c += 4) {
                *(float4*)&lo_s[warp][gl * 8 + c] = make_float4(lo[c], lo[c + 1], lo[c + 2], lo[c + 3]);
                *(float4*)&hi_s[warp][gl * 8 + c] = make_float4(hi[c], hi[c + 1], hi[c + 2], hi[c + 3]);
            }
        }
        __syncthreads();
        float l = 0.f, u = 0.f;
        if (tid < D) {
            l = lo_s[0][tid], u = hi_s[0][tid];
#pragma unroll
            for (int x = 1; x < WARPS; ++x) l = fminf(l, lo_s[x][tid]), u = fmaxf(u, hi_s[x][tid]);
        }
        float big = fmaxf(fabsf(l), fabsf(u));
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) big = fmaxf(big, __shfl_xor_sync(QMOE_FULL_MASK, big, d));
        if (lane == 0) big_s[warp] = big;
        __syncthreads();
#pragma unroll
        for (int x = 0; x < WARPS; ++x) big = fmaxf(big, big_s[x]);
        // big = m 2^e with m in [64, 127], or (63.5, 64) one power up; the quotients by a power of two are exact
        int e = (int)(__float_as_uint(big) >> 23) - 127 - 6;
        if (big > 127.f * __int_as_float((e + 127) << 23)) ++e;
        const float step = big > 0.f ? __int_as_float((e + 127) << 23) : 0.f, inv = big > 0.f ? __int_as_float((127 - e) << 23) : 0.f;
        const int64_t rec = (int64_t)page * a.cache.n_kv_heads + h;
        if (tid < D) {
            a.codes[rec * (2 * D) + tid] = (int8_t)min(max(__float2int_ru(u * inv), -127), 127);
            a.codes[rec * (2 * D) + D + tid] = (int8_t)min(max(__float2int_rd(l * inv), -127), 127);
        }
        if (tid == 0) a.steps[rec] = step;
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
    uint16_t* whole;       // [token][kv head][2 D]: sums of the group's queries as whole numbers
    int B, n, n_kv, group, n_pages, max_blocks, page_shift, max_kv, max_seen, top, first, last, bits;
};

// Blocks that query token t sees (-1: the token belongs to no request), and its request.
__device__ __forceinline__ int blocks_seen(const SelectArgs& a, int t, int* b, bool report) {
    int end, kv;
    *b = kv4::request_of<true>(a.q_start, a.kv_len, a.B, t, &end, &kv);
    if (*b < 0) return -1;
    if (kv < 0 || kv > a.max_kv) {
        if (report) blocks_set_error(kv < 0 ? QMOE_EINVAL : QMOE_ECAPACITY);
        return 0;
    }
    const int64_t pos = (int64_t)kv - ((int64_t)end - t);
    return pos < 0 ? 0 : (int)(pos >> a.page_shift) + 1;
}

// The 16-bit products of 4 channels: acc + c[0] q0.lo + c[1] q0.hi + c[2] q1.lo + c[3] q1.hi.
__device__ __forceinline__ int dot4(uint32_t c, uint32_t q0, uint32_t q1, int acc) {
    acc = __dp2a_lo((int)q0, (int)c, acc);
    return __dp2a_hi((int)q1, (int)c, acc);
}

constexpr int kScoreThreads = 128;

// q as bf16, NaN as 0, infinities as the largest finite value
__device__ __forceinline__ float query_value(uint32_t bits) {
    const float v = __uint_as_float(bits << 16);
    return v == v ? fminf(fmaxf(v, -3.3895313892515355e38f), 3.3895313892515355e38f) : 0.f;
}

// The queries of one token and kv head as whole numbers: sums over the group of the positive parts, then of the negative
// ones, 16 bits each.  A warp takes a (token, kv head), a lane D / 32 channels.  A kernel of its own: made again in every thread
// block of the scores they cost 2.5 us more for 64 requests of up to 32768 tokens.  One chain of loads bounds it, 2.5 us.
constexpr int kWholeThreads = 128;

template <int D>
__global__ void __launch_bounds__(kWholeThreads) whole_kernel(SelectArgs a) {
    constexpr int V = D / 32;
    kv4::depend_wait();        // (before the scores' kernel may begin: that reads what earlier calls wrote without waiting)
    kv4::depend_launch();
    const int64_t i = (int64_t)blockIdx.x * (kWholeThreads / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (i >= (int64_t)a.n * a.n_kv) return;
    const uint16_t* q = a.q + i * a.group * D + lane * V;
    auto load = [&](int g, uint32_t (&w)[V / 2]) {
        if constexpr (V == 4) {
            const uint2 x = *(const uint2*)(q + g * D);
            w[0] = x.x, w[1] = x.y;
        } else {
            w[0] = *(const uint32_t*)(q + g * D);
        }
    };
    float big = 0.f;
#pragma unroll 8
    for (int g = 0; g < a.group; ++g) {
        uint32_t w[V / 2];
        load(g, w);
#pragma unroll
        for (int k = 0; k < V / 2; ++k) big = fmaxf(big, fmaxf(fabsf(query_value(w[k] & 0xFFFFu)), fabsf(query_value(w[k] >> 16))));
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) big = fmaxf(big, __shfl_xor_sync(QMOE_FULL_MASK, big, d));
    // largest magnitude to [2^(bits-1), 2^bits): times 2^(bits - 1 - exponent), in two factors of normal size
    const int up = a.bits - 1 - ilogbf(big > 0.f ? big : 1.f), limit = (1 << a.bits) - 1;
    const float f1 = __int_as_float((min(up, 100) + 127) << 23), f2 = __int_as_float((max(up - 100, 0) + 127) << 23);
    int pos[V], neg[V];
#pragma unroll
    for (int k = 0; k < V; ++k) pos[k] = neg[k] = 0;
#pragma unroll 8
    for (int g = 0; g < a.group; ++g) {
        uint32_t w[V / 2];
        load(g, w);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const float v = query_value(k & 1 ? w[k >> 1] >> 16 : w[k >> 1] & 0xFFFFu);
            const int r = min(max(__float2int_rn(v * f1 * f2), -limit), limit);
            pos[k] += max(r, 0), neg[k] += min(r, 0);
        }
    }
    uint32_t* out = (uint32_t*)(a.whole + i * (2 * D)) + lane * (V / 2);
#pragma unroll
    for (int k = 0; k < V / 2; ++k) {
        out[k] = __byte_perm((uint32_t)pos[2 * k], (uint32_t)pos[2 * k + 1], 0x5410);
        out[D / 2 + k] = __byte_perm((uint32_t)neg[2 * k], (uint32_t)neg[2 * k + 1], 0x5410);
    }
}

// A thread block scores some blocks of one query token for up to kScoreHeads kv heads: it copies the records (hi and lo codes) of those
// heads of each page, which stand side by side, to shared memory, all at once and without registers, so that the blocks of a
// multiprocessor have what its bandwidth takes under way; then groups of L lanes (16 codes of a record each) multiply kRecords records
// of one kv head at a time with the group's summed queries, and the partial sums are added up crosswise, so that lane i ends with
// record i (mod kRecords).  What does not depend on the queries goes ahead of the wait for them.  The latency table - copy - product
// bounds it: 64 requests of up to 32768 tokens, 8 kv heads of 128, pages of 64, 37 MB, take 10.9 us behind whole_kernel's 2.5 (cold caches, 13 to 15: 40 % of the copy rate), 1.5 to 3 more where the records go
// through registers.
constexpr int kScoreBytes = 32768, kScoreHeads = 32, kRecords = 8, kMostPages = 256;
constexpr uint32_t kWaitLimit = 1u << 22;

// Pages of a thread block: what its shared memory holds, or fewer while every group of lanes still has kRecords and the blocks are
// few (131072 tokens in pages of 16, one kv head of 64: 132 blocks 12.4 us, 264 11.8).
inline int score_pages(int head_dim, int n_kv, int64_t row, int64_t tokens) {
    const int heads = std::min(n_kv, kScoreHeads), parts = std::max(1, kScoreThreads / (head_dim / 8) / heads);
    int p = std::min(kScoreBytes / (2 * head_dim) / heads, kMostPages);
    while (p >= 2 * kRecords * parts && (row + p - 1) / p * tokens < 2 * qmoe::sm_count()) p /= 2;
    return p;
}

template <int D>
__global__ void __launch_bounds__(kScoreThreads) score_kernel(SelectArgs a, int chunks, int pages) {
    constexpr int L = D / 8, GROUPS = kScoreThreads / L, TURNS = kMostPages / kScoreThreads;
    __shared__ alignas(128) unsigned char codes_s[kScoreBytes];
    __shared__ int page_s[kMostPages];
    __shared__ uint64_t full;
    kv4::depend_launch();
    const int tid = threadIdx.x, t = blockIdx.x / chunks, c = blockIdx.x - t * chunks;
    const int h0 = blockIdx.y * kScoreHeads, heads = min(a.n_kv - h0, kScoreHeads);
    const int j0 = c * pages;
    // (in a decode step token t is request t: its table entries are loaded beside the lengths that say so)
    int entry[TURNS];
#pragma unroll
    for (int i = 0; i < TURNS; ++i) {
        const int j = j0 + i * kScoreThreads + tid;
        entry[i] = i * kScoreThreads + tid < pages && t < a.B && j < a.max_blocks ? __ldcg(a.table + (int64_t)t * a.max_blocks + j) : -1;
    }
    int b;
    const int seen = blocks_seen(a, t, &b, c == 0 && tid == 0 && h0 == 0);
    if (seen <= a.top || j0 >= seen) {       // few blocks are all taken
        kv4::depend_wait();
        return;
    }
    if (tid == 0) {
        qmoe_tc::mbar_init(&full, 1);
        qmoe_tc::fence_mbar_init();
    }
    const uint32_t slice = (uint32_t)heads * (2 * D);
    int there = 0;
#pragma unroll
    for (int i = 0; i < TURNS; ++i) {
        const int at = i * kScoreThreads + tid, j = j0 + at;
        const bool mine = at < pages && j < seen;
        if (b != t) entry[i] = mine && j < a.max_blocks ? __ldcg(a.table + (int64_t)b * a.max_blocks + j) : -1;
        if (!mine || entry[i] < 0 || entry[i] >= a.n_pages) {
            if (mine && h0 == 0) blocks_set_error(QMOE_EINVAL);
            entry[i] = -1;
        }
        if (at < pages) page_s[at] = entry[i];
        there += __syncthreads_count(entry[i] >= 0);
    }
    if (tid == 0)
        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(qmoe_tc::smem_u32(&full)), "r"((uint32_t)there * slice) : "memory");
    __syncwarp();
#pragma unroll
    for (int i = 0; i < TURNS; ++i)
        if (entry[i] >= 0)
            asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                             qmoe_tc::smem_u32(codes_s) + (uint32_t)(i * kScoreThreads + tid) * slice),
                         "l"(a.codes + ((int64_t)entry[i] * a.n_kv + h0) * (2 * D)), "r"(slice), "r"(qmoe_tc::smem_u32(&full))
                         : "memory");
    const int grp = tid / L, gl = tid & (L - 1), rec = gl & (kRecords - 1);
    const unsigned mask = (L == 16 ? 0xFFFFu : 0xFFu) << (tid & 31 & ~(L - 1));
    const int parts = max(1, GROUPS / heads), part = grp / heads, span = (min(pages, seen - j0) + parts - 1) / parts;
    const int p0 = part * span, p1 = min(min(p0 + span, pages), seen - j0);
    kv4::depend_wait();
    bool landed = false;
    for (int h = grp - part * heads; h < heads && part < parts; h += GROUPS) {
        const uint4* q = (const uint4*)(a.whole + ((int64_t)t * a.n_kv + h0 + h) * (2 * D) + gl * 16);
        const uint4 q0 = q[0], q1 = q[1];
        for (int p = p0; p < p1; p += kRecords) {
            const int at = p + rec, page = at < p1 ? page_s[at] : -1;
            const float step = page >= 0 ? a.steps[(int64_t)page * a.n_kv + h0 + h] : 0.f;
            if (!landed && !qmoe_tc::mbar_wait(&full, 0, kWaitLimit)) {
                blocks_set_error(QMOE_ETIMEOUT);
                return;
            }
            landed = true;
            const unsigned char* from = codes_s + (uint32_t)p * slice + h * (2 * D) + gl * 16;
            int acc[kRecords];
#pragma unroll
            for (int r = 0; r < kRecords; ++r) {
                const uint4 x = p + r < p1 ? *(const uint4*)(from + r * slice) : make_uint4(0, 0, 0, 0);      // (a missing page's: whatever stands there)
                acc[r] = dot4(x.w, q1.z, q1.w, dot4(x.z, q1.x, q1.y, dot4(x.y, q0.z, q0.w, dot4(x.x, q0.x, q0.y, 0))));
            }
            if (L > kRecords) {
#pragma unroll
                for (int r = 0; r < kRecords; ++r) acc[r] += __shfl_xor_sync(mask, acc[r], kRecords);
            }
            // a lane keeps the records whose number has the lane's upper bits, and gives the others away
#pragma unroll
            for (int d = kRecords / 2; d > 0; d >>= 1) {
                const bool upper = gl & d;
#pragma unroll
                for (int r = 0; r < d; ++r) {
                    const int give = upper ? acc[r] : acc[r + d], keep = upper ? acc[r + d] : acc[r];
                    acc[r] = keep + __shfl_xor_sync(mask, give, d);
                }
            }
            // (a step that is NaN, which kv4_block_bounds never writes, gives a score like a missing page's)
            if (at < p1 && gl < kRecords)
                a.scores[((int64_t)t * a.n_kv + h0 + h) * a.max_seen + j0 + at] = page >= 0 ? fmaxf(__fmul_rn((float)acc[0], step), -INFINITY) : -INFINITY;
        }
    }
    // the copies land before the block's memory goes away
    if (!landed && !qmoe_tc::mbar_wait(&full, 0, kWaitLimit)) blocks_set_error(QMOE_ETIMEOUT);
}

// ---------------------------------------------------------------- the best blocks
//
// The list of one (token, kv head) is made by a warp (up to 1024 blocks to choose from) or a thread block.  Scores are kept in
// registers as integer keys, warp w those of the w-th equal run.  The key of the last one taken is found between the
// smallest and the largest by trying three keys at a time (a count each, all three in one word), until as many are above
// one of them as are wanted, or no more than 32 are left between: those are counted against each other.  Then every warp writes the
// blocks of its run that are above it, and the first ones at it.  Rounds one after the other, each a count and its sum, bound it: 64 requests' choice takes
// 13.4 us without this kernel and 17.7 with it (20.1 where the tries go on to the last key), 4 lists of 8192 scores 4.4 and 10.4 (11.5).
// Tries that are not a quarter apart as keys (as values; where the counts so far point to) take longer.
constexpr int kMostBlocks = 1 << 20;      // of a request
constexpr int kPickThreads = 128;        // of a block whose warps make a list each

// fp32 -> integer of the same order (-0 as 0); no key is 0.
__device__ __forceinline__ uint32_t score_key(float v) {
    const uint32_t u = __float_as_uint(v + 0.f);
    return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}

// WARPS a list (1: a block makes several), R scores a lane in registers; R = 0: any number, read again each time.
template <int WARPS, int R>
__global__ void __launch_bounds__(WARPS == 1 ? kPickThreads : WARPS * 32) pick_kernel(SelectArgs a) {
    __shared__ uint2 part_s[2][WARPS];
    __shared__ unsigned long long count_s[2][WARPS];
    constexpr int LISTS = WARPS == 1 ? kPickThreads / 32 : 1;
    __shared__ alignas(16) uint32_t left_s[LISTS][32];
    __shared__ int n_left_s[LISTS];
    const int lane = threadIdx.x & 31, warp = WARPS == 1 ? 0 : threadIdx.x >> 5;
    const int64_t list = WARPS == 1 ? (int64_t)blockIdx.x * (kPickThreads / 32) + (threadIdx.x >> 5) : blockIdx.x;
    const int tid = warp * 32 + lane;
    constexpr int THREADS = WARPS * 32;
    const int t = (int)(list / a.n_kv);
    int b, seen = -1;
    if (t < a.n) seen = blocks_seen(a, t, &b, a.max_seen <= a.top && tid == 0 && list == (int64_t)t * a.n_kv);
    kv4::depend_wait();        // (before any return: what follows the call waits for this kernel alone)
    kv4::depend_launch();
    if (seen < 0) return;
    int32_t* sel = a.sel + list * a.top;
    if (seen <= a.top) {
        for (int i = tid; i < a.top; i += THREADS) sel[i] = i < seen ? i : -1;
        return;
    }
    const float* scores = a.scores + list * a.max_seen;
    const int lo = a.first, hi = seen - a.last, want = a.top - a.first - a.last;
    for (int i = tid; i < a.first; i += THREADS) sel[i] = i;
    for (int i = tid; i < a.last; i += THREADS) sel[a.top - a.last + i] = hi + i;
    if (want == 0) return;
    const int per = R ? R * 32 : ((hi - lo + WARPS - 1) / WARPS + 31) & ~31;
    const int w0 = min(lo + warp * per, hi), w1 = min(w0 + per, hi), steps = R ? R : (w1 - w0 + 31) / 32;
    uint32_t* left = left_s[WARPS == 1 ? threadIdx.x >> 5 : 0];
    int* n_left = &n_left_s[WARPS == 1 ? threadIdx.x >> 5 : 0];
    if (warp == 0) {
        left[lane] = 0;
        if (lane == 0) *n_left = 0;
    }
    uint32_t key[R ? R : 1];
    if constexpr (R > 0) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int j = w0 + 32 * i + lane;
            key[i] = j < w1 ? score_key(scores[j]) : 0u;
        }
    }
    auto key_at = [&](int i) {
        if constexpr (R > 0) {
            return key[i];
        } else {
            const int j = w0 + 32 * i + lane;
            return j < w1 ? score_key(scores[j]) : 0u;
        }
    };
    // ---- all keys are in [least, end)
    uint32_t least = 0xFFFFFFFFu, end = 0;
#pragma unroll
    for (int i = 0; i < (R ? R : steps); ++i) {
        const uint32_t k = key_at(i);
        end = max(end, k);
        least = min(least, k ? k : 0xFFFFFFFFu);
    }
    least = __reduce_min_sync(QMOE_FULL_MASK, least), end = __reduce_max_sync(QMOE_FULL_MASK, end);
    if (WARPS > 1) {
        if (lane == 0) part_s[0][warp] = make_uint2(least, end);
        __syncthreads();
        const uint2 p = lane < WARPS ? part_s[0][lane] : make_uint2(0xFFFFFFFFu, 0u);
        least = __reduce_min_sync(QMOE_FULL_MASK, p.x), end = __reduce_max_sync(QMOE_FULL_MASK, p.y);
    }
    ++end;
    // ---- `from` keys are >= least, at least as many as are wanted; `above_end` are >= end, fewer
    int from = hi - lo, above_end = 0;
    for (int turn = 0; end - least > 1 && from > want && from - above_end > 32; turn ^= 1) {
        const uint32_t span = end - least, q = span >= 4 ? span >> 2 : 1;
        const uint32_t p1 = least + q, p2 = min(p1 + q, end), p3 = min(p2 + q, end);
        int n1 = 0, n2 = 0, n3 = 0;
#pragma unroll
        for (int i = 0; i < (R ? R : steps); ++i) {
            const uint32_t k = key_at(i);
            n1 += k >= p1, n2 += k >= p2, n3 += k >= p3;
        }
        if constexpr (R > 0) {
            // (a warp's counts are at most 512: ten bits)
            const uint32_t n = __reduce_add_sync(QMOE_FULL_MASK, (uint32_t)(n1 | n2 << 10 | n3 << 20));
            n1 = (int)(n & 1023u), n2 = (int)(n >> 10 & 1023u), n3 = (int)(n >> 20);
        } else {
            n1 = warp_sum_int(n1), n2 = warp_sum_int(n2), n3 = warp_sum_int(n3);
        }
        if (WARPS > 1) {
            // 21 bits each: a list chooses from at most kMostBlocks blocks
            static_assert(kMostBlocks < 1 << 21, "a count has 21 bits");
            if (lane == 0) count_s[turn][warp] = (unsigned long long)n1 | (unsigned long long)n2 << 21 | (unsigned long long)n3 << 42;
            __syncthreads();
            const unsigned long long v = lane < WARPS ? count_s[turn][lane] : 0ull;
            n1 = (int)__reduce_add_sync(QMOE_FULL_MASK, (uint32_t)(v & 0x1FFFFFu));
            n2 = (int)__reduce_add_sync(QMOE_FULL_MASK, (uint32_t)(v >> 21 & 0x1FFFFFu));
            n3 = (int)__reduce_add_sync(QMOE_FULL_MASK, (uint32_t)(v >> 42));
        }
        // (p3 >= p2 >= p1, counts the other way; a p at end counts none)
        if (n3 >= want) least = p3, from = n3;
        else if (n2 >= want) least = p2, from = n2, end = p3, above_end = n3;
        else if (n1 >= want) least = p1, from = n1, end = p2, above_end = n2;
        else end = p1, above_end = n1;
    }
    uint32_t cut = least;
    if (end - least > 1 && from > want) {
        // ---- at most 32 are between: side by side, a lane each, which counts the larger ones
        if (WARPS == 1) __syncwarp();
#pragma unroll
        for (int i = 0; i < (R ? R : steps); ++i) {
            const uint32_t k = key_at(i);
            if (k >= least && k < end) left[atomicAdd(n_left, 1)] = k;
        }
        if (WARPS == 1) __syncwarp();
        else __syncthreads();
        const int between = from - above_end;
        const uint32_t mine = left[lane];
        int larger = 0;
        for (int j = 0; j < between; j += 4) {
            const uint4 o = *(const uint4*)(left + j);
            larger += (o.x > mine) + (o.y > mine) + (o.z > mine) + (o.w > mine);
        }
        cut = __reduce_min_sync(QMOE_FULL_MASK, lane < between && above_end + larger < want ? mine : 0xFFFFFFFFu);
        from = above_end + __popc(__ballot_sync(QMOE_FULL_MASK, lane < between && mine >= cut));
    }
    const unsigned below = (1u << lane) - 1;
    if (from == want) {
        // ---- the blocks from `cut` on, all of them
        int before = 0;
        if (WARPS > 1) {
            int n = 0;
#pragma unroll
            for (int i = 0; i < (R ? R : steps); ++i) n += key_at(i) >= cut;
            n = (int)__reduce_add_sync(QMOE_FULL_MASK, (unsigned)n);
            if (lane == 0) part_s[1][warp] = make_uint2((unsigned)n, 0u);
            __syncthreads();
            before = (int)__reduce_add_sync(QMOE_FULL_MASK, lane < warp ? part_s[1][lane].x : 0u);
        }
#pragma unroll
        for (int i = 0; i < (R ? R : steps); ++i) {
            const bool in = key_at(i) >= cut;
            const unsigned hit = __ballot_sync(QMOE_FULL_MASK, in);
            if (in) sel[a.first + before + __popc(hit & below)] = w0 + 32 * i + lane;
            before += __popc(hit);
        }
        return;
    }
    // ---- the blocks above `cut`, and `room` of those at it
    int above = 0, equal = 0;
#pragma unroll
    for (int i = 0; i < (R ? R : steps); ++i) {
        const uint32_t k = key_at(i);
        above += k > cut, equal += k == cut;
    }
    above = (int)__reduce_add_sync(QMOE_FULL_MASK, (unsigned)above), equal = (int)__reduce_add_sync(QMOE_FULL_MASK, (unsigned)equal);
    int all_above = above, above_before = 0, equal_before = 0;
    if (WARPS > 1) {
        __syncthreads();
        if (lane == 0) part_s[1][warp] = make_uint2((unsigned)above, (unsigned)equal);
        __syncthreads();
        const uint2 p = lane < WARPS ? part_s[1][lane] : make_uint2(0u, 0u);
        all_above = (int)__reduce_add_sync(QMOE_FULL_MASK, p.x);
        above_before = (int)__reduce_add_sync(QMOE_FULL_MASK, lane < warp ? p.x : 0u);
        equal_before = (int)__reduce_add_sync(QMOE_FULL_MASK, lane < warp ? p.y : 0u);
    }
    const int room = want - all_above;
#pragma unroll
    for (int i = 0; i < (R ? R : steps); ++i) {
        const uint32_t k = key_at(i);
        const unsigned hit = __ballot_sync(QMOE_FULL_MASK, k >= cut);
        if (hit == 0) continue;
        const unsigned over = __ballot_sync(QMOE_FULL_MASK, k > cut), same = hit & ~over;
        const int n_same = equal_before + __popc(same & below);
        if (k > cut || (k == cut && n_same < room)) sel[a.first + above_before + __popc(over & below) + min(n_same, room)] = w0 + 32 * i + lane;
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

// Workspace: the queries as whole numbers (room for the larger head_dim), then the scores.
size_t whole_bytes(int n_q_tokens, int n_kv_heads) { return (size_t)n_q_tokens * n_kv_heads * (2 * 128) * sizeof(uint16_t); }

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
    // few tokens: a thread block each, so that their blocks are bounded side by side; many: a page's worth of them
    const int64_t share = (int64_t)n * cache->n_kv_heads / ((int64_t)qmoe::sm_count() * 16);
    const int span = (int)std::min<int64_t>(std::max<int64_t>(share, 1), cache->page_size);
    const dim3 grid((unsigned)(((int64_t)n + span - 1) / span), (unsigned)cache->n_kv_heads);
    return kv4::launch_dependent(cache->head_dim == 128 ? bounds_kernel<16> : bounds_kernel<8>, grid, kBoundsThreads, 0, (cudaStream_t)stream,
                                 "kv4_block_bounds", a, span);
}

extern "C" int kv4_select_blocks_ws_size(int n_q_tokens, int n_kv_heads, int page_size, int max_kv, size_t* bytes) {
    qmoe::clear_error();
    if (!bytes) return qmoe::fail(QMOE_EINVAL, "kv4_select_blocks_ws_size: NULL output");
    if (n_q_tokens < 0 || n_kv_heads < 1 || max_kv < 0 || (page_size != 16 && page_size != 32 && page_size != 64))
        return qmoe::fail(QMOE_EINVAL, "kv4_select_blocks_ws_size: bad sizes (page_size 16, 32 or 64)");
    *bytes = whole_bytes(n_q_tokens, n_kv_heads) + (size_t)n_q_tokens * n_kv_heads * (size_t)score_row(page_size, max_kv) * sizeof(float);
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
    if ((int64_t)max_kv > (int64_t)kMostBlocks * bounds->page_size)
        return qmoe::fail(QMOE_EUNSUPPORTED, "kv4_select_blocks: max_kv above 2^20 pages");
    if (top < 1 || top > 65536 || first < 0 || last < 0 || (int64_t)first + last > top)
        return qmoe::fail(QMOE_EINVAL, "kv4_select_blocks: need 1 <= top <= 65536 and first + last <= top");
    if (B == 0 || n_q_tokens == 0) return QMOE_OK;
    if (!q || !q_start || !kv_len || !sel || (max_blocks > 0 && !table)) return qmoe::fail(QMOE_EINVAL, "kv4_select_blocks: NULL pointer");
    if (!kv4::aligned16(q)) return qmoe::fail(QMOE_EINVAL, "kv4_select_blocks: q not 16-byte aligned");
    SelectArgs a{};
    const int64_t row = score_row(bounds->page_size, max_kv);
    const size_t whole = whole_bytes(n_q_tokens, n_kv);
    if (ws_bytes < whole + (size_t)n_q_tokens * n_kv * (size_t)row * sizeof(float)) return qmoe::fail(QMOE_ECAPACITY, "kv4_select_blocks: workspace too small");
    a.codes = (const int8_t*)bounds->codes, a.steps = bounds->steps, a.q = (const uint16_t*)q;
    a.q_start = q_start, a.kv_len = kv_len, a.table = table, a.sel = sel;
    a.whole = (uint16_t*)workspace, a.scores = (float*)((char*)workspace + whole);
    a.B = B, a.n = n_q_tokens, a.n_kv = n_kv, a.group = n_q_heads / n_kv, a.n_pages = bounds->n_pages, a.max_blocks = max_blocks;
    a.page_shift = shift_of(bounds->page_size), a.max_kv = max_kv, a.max_seen = (int)row, a.top = top, a.first = first, a.last = last;
    a.bits = 15;
    while ((1 << (15 - a.bits)) < a.group) --a.bits;
    cudaStream_t st = (cudaStream_t)stream;
    const int pages = score_pages(bounds->head_dim, n_kv, row, n_q_tokens);
    const int64_t chunks = (row + pages - 1) / pages, blocks = chunks * n_q_tokens;
    if (blocks > 0x7FFFFFFFLL || (int64_t)n_q_tokens * n_kv > 0x7FFFFFFFLL)
        return qmoe::fail(QMOE_EINVAL, "kv4_select_blocks: too many query tokens in one call");
    const unsigned lists = (unsigned)(n_q_tokens * n_kv), by_warps = (lists + kPickThreads / 32 - 1) / (kPickThreads / 32);
    const char* who = "kv4_select_blocks";
    if (row <= top) {
        // (launched plainly: it reads the lengths ahead of its wait, which only a kernel behind score_kernel may)
        pick_kernel<1, 0><<<by_warps, kPickThreads, 0, st>>>(a);      // every block that is there
        return qmoe::launch_check(who);
    }
    if (!workspace || !kv4::aligned16(workspace)) return qmoe::fail(QMOE_EINVAL, "kv4_select_blocks: workspace NULL or not 16-byte aligned");
    const unsigned whole_blocks = (lists + kWholeThreads / 32 - 1) / (kWholeThreads / 32);
    const bool d128 = bounds->head_dim == 128;
    if ((rc = kv4::launch_dependent(d128 ? whole_kernel<128> : whole_kernel<64>, dim3(whole_blocks), kWholeThreads, 0, st, who, a))) return rc;
    if ((rc = kv4::launch_dependent(d128 ? score_kernel<128> : score_kernel<64>, dim3((unsigned)blocks, (unsigned)((n_kv + kScoreHeads - 1) / kScoreHeads)), kScoreThreads, 0, st, who, a, (int)chunks, pages))) return rc;
    const int64_t most = ((int64_t)max_kv + bounds->page_size - 1) / bounds->page_size - first - last;      // blocks a list chooses from
    if (most <= 128) return kv4::launch_dependent(pick_kernel<1, 4>, dim3(by_warps), kPickThreads, 0, st, who, a);
    // (few lists by four warps each, for the shorter chain; us of a whole call of 4, 16, 64 and 256 requests with 8 kv heads, four warps a
    // list: 6.9, 8.7, 17.8, 39.7; one: 8.1, 9.7, 17.7, 39.1)
    if (most <= 512 && lists <= 2 * (unsigned)qmoe::sm_count()) return kv4::launch_dependent(pick_kernel<4, 4>, dim3(lists), 128, 0, st, who, a);
    if (most <= 512) return kv4::launch_dependent(pick_kernel<1, 16>, dim3(by_warps), kPickThreads, 0, st, who, a);
    if (most <= 2048) return kv4::launch_dependent(pick_kernel<8, 8>, dim3(lists), 256, 0, st, who, a);
    if (most <= 8192) return kv4::launch_dependent(pick_kernel<32, 8>, dim3(lists), 1024, 0, st, who, a);
    return kv4::launch_dependent(pick_kernel<32, 0>, dim3(lists), 1024, 0, st, who, a);
}
