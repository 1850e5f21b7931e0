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
    const int32_t* sel;      // lists of chosen blocks [query token][kv head][top], or NULL
    int top;
};

// Longest request: its keys, rounded up to a tile of either path, stay in int32.
constexpr int kMaxKv = 0x7FFFFFFF - 127;

// Whether request b can be run; what is wrong with it goes to the error word.
__device__ __forceinline__ bool request(const AttnArgs& a, int b, int* q0, int* q_len, int* kv_len, bool report) {
    const int s = a.q_start[b], e = a.q_start[b + 1], n = a.kv_len[b];
    *q0 = s, *q_len = e - s, *kv_len = n;
    if (s < 0 || e < s || e > a.n_q_tokens || n < 0 || n > kMaxKv) {
        if (report) attn_set_error(QMOE_EINVAL);
        return false;
    }
    if (e - s > a.max_q || n > a.max_kv) {
        if (report) attn_set_error(QMOE_ECAPACITY);
        return false;
    }
    return true;
}

// First token that a query at position pos sees (pos may be below 0: then it sees none, and pos - window would overflow).
__device__ __forceinline__ int first_seen(const AttnArgs& a, int pos) { return a.window && pos >= a.window ? pos - a.window + 1 : 0; }

// ---- with lists of chosen blocks every query token is a request of its own, with its list's blocks as its keys.  Bound by memory with
// many tokens: 64 of them over 64 blocks of 64 tokens, 32/8 heads of 128, 55.5 us for 260 MB (4.7 TB/s, 69 % of a copy's rate, the join
// and the items' beginnings among it; 49 % of the issue slots); one token over 128 blocks of 16, 16/16 heads, 9.6 us by latency.

// Whether query token t can be run: its request, its position, and the blocks that it sees.
__device__ __forceinline__ bool chosen_token(const AttnArgs& a, int t, int* b, int* pos, int* seen, bool report) {
    int end, n;
    *b = kv4::request_of<false>(a.q_start, a.kv_len, a.B, t, &end, &n);
    if (*b < 0) return false;
    if (n < 0 || n > kMaxKv) {
        if (report) attn_set_error(QMOE_EINVAL);
        return false;
    }
    const long long p = (long long)n - ((long long)end - t);      // (below 0 where q_start runs past kv_len)
    *pos = p < 0 ? -1 : (int)p;
    *seen = p < 0 ? 0 : (int)(p >> a.cache.page_shift) + 1;
    return true;
}

// What its list holds: entries that are read, the query's own block (the last that it sees) and the tokens it sees of that.
struct ChosenList {
    int req, listed, own_blk, in_own;
};
__device__ __forceinline__ ChosenList list_of(const AttnArgs& a, int t) {
    int req = 0, pos = -1, seen = 0;
    chosen_token(a, t, &req, &pos, &seen, false);
    return ChosenList{req, min(seen, a.top), seen - 1, pos - ((seen - 1) << a.cache.page_shift) + 1};
}

// ---------------------------------------------------------------- few query rows: one pass over the codes
//
// A request's rows of one kv head (query n, head g of the group: row n * group + g) are few, so the
// cache's bytes bound the work.  With k_d = s u_d + z and v_d likewise,
//   scale q . k = scale (s (q . u) + z sum(q)),   sum_j p_j v_j = sum_j (p_j s_j) u_j + sum_j p_j z_j,
// the 4-bit codes are matrix operands as they are: a code in the low mantissa bits of an fp16 pattern
// is the subnormal u 2^-24 (u 2^-20 one nibble up), so two masks and a shift turn a 32-bit word into
// four operand registers, and scale and offset enter on the few scores.  Queries are scaled by a power
// of two per row into fp16's range (exact: bf16 has fewer significant bits).  What is rounded to fp16
// (11 bits) is a weight times its value row's scale, p s_v: with p = 2^(score - m) each row's m follows
// its largest score + log2(s_v) so that its largest product stands between 2^6 and 2^14, and products
// down to 2^-20 of that keep all bits whatever the values' magnitudes are, also those of tokens that the
// row does not see.  Statistics and sums are fp32.
//
// The products are S^T = U_k Q^T and O^T = U_v^T P^T (m16n8k16, keys or head values as the 16 rows, 8
// query rows as the 8 columns), so that one to eight rows fill the instruction; tcgen05's 128 rows
// would be idle and its operands would have to be expanded through shared memory.  A row's m moves only
// when a product would pass 2^14 (a vote instead of a reduction).
//
// Work is cut into tiles of kTile tokens; the tiles of all (request, kv head) items in a row are dealt
// out to the blocks in equal runs, whatever the lengths.  A producer warp copies whole pages of one
// head (contiguous in the layout) into a ring of stages with bulk copies; four warps take 32 tokens of
// a tile each.  An item that several blocks share leaves its parts (unnormalised sums, maximum, sum of
// weights) in the workspace for join_kernel.
//
// Measured (one GB300): 64 requests of 1 to 16384 tokens, 32 query heads on 8 key heads of 128, 106 us in
// a graph = 5.5 TB/s of codes and pairs, 81 % of the copy rate (109 to 113 in a stream of calls from
// Python); issue slots 52 % used, tensor pipe 29 %.  What it took: 32 tokens a warp and stage instead of
// 16 (141 -> 127 us: fewer instructions beside the products), three stages and blocks a multiprocessor
// instead of two and four (120), runs that count an item's beginning and end (105).  The instances for 16
// and 32 rows of 128 spill 8 and 528 bytes of loads a thread; the others none.
constexpr int kTile = 128;
constexpr int kItemCost = 3;                         // what beginning and ending an item costs, in tiles
constexpr int kStages = 3;
constexpr int kConsumers = 4;                        // warps that compute
constexpr int kDecodeThreads = 32 * (kConsumers + 1);
constexpr float kNoMax = -3.0e38f;                   // running maximum before any score
constexpr float kTop = 6.f, kSlack = 14.f;           // few rows: the largest product is 2^6 when m moves, and 2^14 at most
constexpr float kLeastScale = 5.9604645e-8f;         // fp16's smallest scale but 0, 2^-24
constexpr uint32_t kWaitLimit = 1u << 22;

// Tiles of request b for this path (0: not its request), and the first one.
template <bool kSel>
__device__ __forceinline__ int tiles_of(const AttnArgs& a, int b, int max_rows, int* t0, bool report) {
    int q0, q_len, kv_len;
    *t0 = 0;
    if constexpr (kSel) {
        int r, pos, seen;
        if (!chosen_token(a, b, &r, &pos, &seen, report)) return 0;
        return max(1, (int)((((long long)min(seen, a.top) << a.cache.page_shift) + kTile - 1) / kTile));
    }
    if (!request(a, b, &q0, &q_len, &kv_len, report) || q_len == 0 || q_len * a.group > max_rows) return 0;
    const int first = a.causal ? kv_len - q_len : kv_len - 1;    // position of the first query
    *t0 = first_seen(a, first) / kTile;
    return max(1, (kv_len + kTile - 1) / kTile - *t0);
}

// Block-wide: the units (tiles of all items, and kItemCost for each item after its tiles) in all, the run of each block, and the request that holds this block's first
// unit with the units before it.  A scan over the requests; every thread gets the results.
struct Found {
    long long total, before;
    int b;
};

template <int THREADS, bool kSel>
__device__ __forceinline__ Found scan_requests(const AttnArgs& a, int max_rows, long long* chunk) {
    __shared__ long long warp_sum_s[THREADS / 32];
    __shared__ Found found;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int all = kSel ? a.n_q_tokens : a.B, per = (all + THREADS - 1) / THREADS;
    const int b0 = min(tid * per, all), b1 = min(b0 + per, all);
    long long mine = 0;
    int t0;
    for (int b = b0; b < b1; ++b) {
        const int n = tiles_of<kSel>(a, b, max_rows, &t0, blockIdx.x == 0);
        if (n) mine += n + kItemCost;
    }
    mine *= a.cache.n_kv_heads;
    long long incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(QMOE_FULL_MASK, incl, d);
        if (lane >= d) incl += o;
    }
    if (lane == 31) warp_sum_s[warp] = incl;
    __syncthreads();
    long long total = 0, before = incl - mine;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) before += warp_sum_s[w];
        total += warp_sum_s[w];
    }
    *chunk = max(1LL, (total + gridDim.x - 1) / gridDim.x);
    const long long target = (long long)blockIdx.x * *chunk;
    if (target >= before && target < before + mine) {
        for (int b = b0; b < b1; ++b) {
            const int tiles = tiles_of<kSel>(a, b, max_rows, &t0, false);
            const long long n = tiles ? (long long)(tiles + kItemCost) * a.cache.n_kv_heads : 0;
            if (target < before + n) {
                found.b = b;
                found.before = before;
                break;
            }
            before += n;
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

__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
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
constexpr int kFirst = 1, kLast = 2, kWholeStart = 4, kWholeEnd = 8, kEdge = 16, kEnd = 32, kValid = 64, kPartial = 1 << 16;
// kWholeStart, kWholeEnd: the item begins, ends in this run; kEdge: some row does not see all of the tile; kEnd: the run is
// over; kValid << page of the tile: the page is there; with chosen blocks, kPartial << page: the query sees its first tokens only

template <int D, int NT>
struct DecodeShared {
    // query operand of 16 to 32 rows (with 8 it is held in registers); every warp writes the same values
    alignas(16) uint2 qf[NT == 1 ? 1 : NT][D / 32][2][32];
    alignas(16) float4 qc[NT][4];          // and the factors of rows 2 t, 2 t + 1: of s (q . u), then of z
    alignas(128) unsigned char stage[kStages][kTile * (D + 8)];
    alignas(16) float red[kConsumers][8][D + 4];
    float m[kConsumers][8], l[kConsumers][8];
    StageInfo info[kStages];
    uint64_t full[kStages], empty[kStages], joint;
};

// fp32 parts of split items: slot 2 * block for an item that began before the block's run, 2 * block + 1
// for one that goes on after it; rows x (D sums, maximum, sum of weights).
__device__ __forceinline__ float* part_of(float* parts, long long cta, int which, int rows, int D) {
    return parts + ((size_t)cta * 2 + which) * (size_t)(rows * (D + 2));
}

// An item that a block began and left unfinished, and the last block that works on it (-1: none).
struct SplitItem {
    int b, kh, rb, last;
};

using kv4::depend_launch;
using kv4::depend_wait;

// Read where it stands: volatile, so that it is not read once for all tokens and kept.
__device__ __forceinline__ void load_factors(const float4* src, float (&c1)[2], float (&cz)[2]) {
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(c1[0]), "=f"(c1[1]), "=f"(cz[0]), "=f"(cz[1])
                 : "r"(qmoe_tc::smem_u32(src))
                 : "memory");
}

// The computing warps wait for each other; false (and reported) when one of them has given up.
__device__ __forceinline__ bool meet(uint64_t* bar, uint32_t& met) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
    const bool ok = qmoe_tc::mbar_wait(bar, met & 1, kWaitLimit);
    ++met;
    if (!ok) attn_set_error(QMOE_ETIMEOUT);
    return ok;
}

template <int D, int NT, bool kSel>
__global__ void __launch_bounds__(kDecodeThreads, NT <= 2 ? 3 : 2)
    decode_kernel(AttnArgs a, int max_rows, int direct, SplitItem* items, float* parts) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    DecodeShared<D, NT>& sh = *(DecodeShared<D, NT>*)smem_raw;
    constexpr int W = D / 32;              // words of a key row that a lane reads
    constexpr int VW = D / 64;             // words of a value row that a lane reads
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            qmoe_tc::mbar_init(&sh.full[i], 1);
            qmoe_tc::mbar_init(&sh.empty[i], kConsumers);
        }
        qmoe_tc::mbar_init(&sh.joint, kConsumers);
        qmoe_tc::fence_mbar_init();
    }
    long long chunk = 1, u0, u1;
    Found f;
    if (kSel) depend_wait();
    depend_launch();
    if (direct) {
        // a block an item: few tiles each, and nothing to join
        f.b = blockIdx.x / a.cache.n_kv_heads;
        int t0;
        const int n = tiles_of<kSel>(a, f.b, max_rows, &t0, blockIdx.x == f.b * a.cache.n_kv_heads);
        if (n == 0) return;
        f.before = 0;
        u0 = (long long)(blockIdx.x - f.b * a.cache.n_kv_heads) * (n + kItemCost);
        u1 = u0 + n;
        __syncthreads();
    } else {
        f = scan_requests<kDecodeThreads, kSel>(a, max_rows, &chunk);
        u0 = (long long)blockIdx.x * chunk, u1 = min(u0 + chunk, f.total);
        if (tid == 32 * kConsumers) items[blockIdx.x] = SplitItem{0, 0, 0, -1};
        if (u0 >= u1) return;
    }

    if (warp == kConsumers) {
        // ---- producer: a warp, lane i copies the tile's i-th page; 32 entries of the block table are read at a time
        const int per_tile = kTile >> a.cache.page_shift;
        const uint32_t page_copy = a.cache.head_bytes;
        int b = f.b, t0, n = tiles_of<kSel>(a, b, max_rows, &t0, false);
        int kh = (int)((u0 - f.before) / (n + kItemCost));
        long long begin = f.before + (long long)kh * (n + kItemCost);       // the item's first unit
        int tile = (int)(u0 - begin);
        int kv_len = 0, seen_lo = 0, seen_hi = 0;       // every row sees tokens [seen_lo, seen_hi)
        int blk_lo = 0;                                 // first block that some row sees: those before may have no page
        int held = 0, entry = -1;                       // lane i holds the entry of block held + i
        // chosen blocks: the token's list; the block that entry belongs to; and the same of the 32 entries that come after those
        // held, which are looked up while the copies before them are under way (a list's entry leads to a table's)
        ChosenList list{}, next_list{};
        int chosen = -1, next_chosen = -1, next_entry = -1, next_b = -1, next_kh = 0, next_blk = 0;
        bool looked = false;
        auto look_up = [&](const ChosenList& l, int token, int head, int blk, int* c, int* e) {
            *c = blk + lane < l.listed ? a.sel[((int64_t)token * a.cache.n_kv_heads + head) * a.top + blk + lane] : -1;
            *e = *c >= 0 && *c <= l.own_blk && *c < a.max_blocks ? a.table[(int64_t)l.req * a.max_blocks + *c] : -1;
        };
        bool ok = true, fresh = true;
        int issued = 0;
        for (int u = 0; ok; ++u) {
            const int st = u % kStages;
            // the next tile of the run: past an item's last one comes the next item's first
            bool over = begin + tile >= u1;
            while (!over && tile >= n) {
                begin += n + kItemCost;
                tile = 0;
                fresh = true;
                over = begin >= u1;
                if (!over && ++kh == a.cache.n_kv_heads) {
                    kh = 0;
                    do n = tiles_of<kSel>(a, ++b, max_rows, &t0, false);
                    while (n == 0 && b + 1 < (kSel ? a.n_q_tokens : a.B));
                }
            }
            if (over) {
                if (u >= kStages) ok = qmoe_tc::mbar_wait(&sh.empty[st], (uint32_t)((u / kStages - 1) & 1), kWaitLimit);
                if (ok && lane == 0) {
                    sh.info[st].flags = kEnd;
                    mbar_arrive(&sh.full[st]);
                }
                break;
            }
            const int end = (int)min((long long)n, u1 - begin);      // of the item's tiles in this run
            const int blk0 = (t0 + tile) * per_tile;
            const bool known = kSel && looked && next_b == b && next_kh == kh && next_blk == blk0;
            if (kSel && fresh) {
                list = known ? next_list : list_of(a, b);
            } else if (fresh) {
                const int q_len = a.q_start[b + 1] - a.q_start[b];
                kv_len = a.kv_len[b];
                seen_hi = a.causal ? kv_len - q_len + 1 : kv_len;
                seen_lo = a.window ? max(0, kv_len - a.window) : 0;
                blk_lo = first_seen(a, a.causal ? kv_len - q_len : kv_len - 1) >> a.cache.page_shift;
            }
            if (fresh || blk0 + per_tile > held + 32) {
                held = blk0;
                const int blk = blk0 + lane;
                if constexpr (kSel) {
                    if (known) chosen = next_chosen, entry = next_entry;
                    else look_up(list, b, kh, blk0, &chosen, &entry);
                    if (chosen < -1) attn_set_error(QMOE_EINVAL);
                    looked = false;
                } else {
                    entry = blk < a.max_blocks && ((long long)blk << a.cache.page_shift) < kv_len ? a.table[(int64_t)b * a.max_blocks + blk] : -1;
                }
            }
            const int page = __shfl_sync(QMOE_FULL_MASK, entry, (blk0 - held + lane) & 31);
            bool mine = lane < per_tile && blk0 + lane >= blk_lo && ((blk0 + lane) << a.cache.page_shift) < kv_len;
            unsigned partial = 0;
            if (kSel) {
                const int blk = __shfl_sync(QMOE_FULL_MASK, chosen, (blk0 - held + lane) & 31);
                mine = lane < per_tile && blk0 + lane < list.listed && blk >= 0 && blk <= list.own_blk;
                partial = __ballot_sync(QMOE_FULL_MASK, mine && blk == list.own_blk && list.in_own < 1 << a.cache.page_shift);
            }
            const bool good = mine && page >= 0 && page < a.cache.n_pages;
            if (mine && !good) attn_set_error(QMOE_EINVAL);
            const unsigned mask = __ballot_sync(QMOE_FULL_MASK, good);
            if (u >= kStages) ok = qmoe_tc::mbar_wait(&sh.empty[st], (uint32_t)((u / kStages - 1) & 1), kWaitLimit);
            if (!__all_sync(QMOE_FULL_MASK, ok)) {
                ok = false;
                break;
            }
            if (lane == 0) {
                int flags = (int)mask * kValid;
                if (fresh) flags |= kFirst;
                if (tile == end - 1) flags |= kLast;
                if (begin >= u0) flags |= kWholeStart;          // the item's first tile is in this run
                if (end == n) flags |= kWholeEnd;
                if (kSel) {
                    if ((int)mask != (1 << per_tile) - 1 || partial) flags |= kEdge | (int)partial * kPartial;
                } else if ((t0 + tile) * kTile < seen_lo || (t0 + tile + 1) * kTile > seen_hi || (int)mask != (1 << per_tile) - 1) flags |= kEdge;
                sh.info[st] = StageInfo{b, kh, kSel ? list.in_own : t0 + tile, flags};
                if ((flags & (kLast | kWholeStart | kWholeEnd)) == (kLast | kWholeStart))
                    items[blockIdx.x] = SplitItem{b, kh, 0, (int)((begin + n - 1) / chunk)};
                mbar_expect(&sh.full[st], (uint32_t)__popc(mask) * page_copy);
            }
            __syncwarp();
            if (good) bulk_copy(sh.stage[st] + lane * page_copy, kv4::head_ptr(a.cache, page, kh), page_copy, &sh.full[st]);
            issued = u + 1;
            fresh = false;
            ++tile;
            if (kSel && !looked && blk0 > held) {
                // the item's next entries, or the next item's first
                looked = true;
                next_b = b, next_kh = kh, next_blk = held + 32, next_list = list;
                if (next_blk >= min(list.listed, end * per_tile)) {
                    next_blk = 0;
                    if (++next_kh == a.cache.n_kv_heads) next_kh = 0, ++next_b;
                    if (begin + n + kItemCost >= u1 || next_b >= a.n_q_tokens) next_b = -1;
                    else if (next_b != b) next_list = list_of(a, next_b);
                }
                if (next_b >= 0) look_up(next_list, next_b, next_kh, next_blk, &next_chosen, &next_entry);
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
    // this warp's 32 tokens of a tile, in two halves of 16: page of the tile and token in the page
    const int tok0 = warp * 32, pg = tok0 >> a.cache.page_shift, in0 = tok0 & (P - 1);
    const uint32_t page_off = (uint32_t)pg * a.cache.head_bytes;
    // row kappa of the product is token (kappa & 8) + ((kappa & 7) >> 1) + 4 (kappa & 1): the value operand's
    // lanes t then read four neighbouring rows
    const int kt = in0 + (g >> 1) + 4 * (g & 1);      // token of row g (row g + 8: kt + 8)
    const uint32_t k_off = page_off + (uint32_t)kt * (D / 2) + t * (W * 4);
    const uint32_t v_off = page_off + (uint32_t)(P + in0 + t) * (D / 2) + g * (VW * 4);
    const uint32_t kp_off = page_off + (uint32_t)P * D + kt * 4;
    const uint32_t vp_off = kp_off + (uint32_t)P * 4;
    // from one half to the other: the next 16 rows, or the next page where a page has 16
    const uint32_t row_step = P == 16 ? a.cache.head_bytes : 16 * (D / 2), pair_step = P == 16 ? a.cache.head_bytes : 64;

    uint2 qr[W][2];                // query operand of 8 rows: [word][nibble parity]
    float c1[2], cz[2];            // of 8 rows, per row: factor of s (q . u), and factor times sum(q), in log2 units
    float m[NT][2], l[NT][2], pz[NT][2];
    float o[NT][4 * VW][4];
    uint32_t met = 0;              // times the computing warps have met
    int q0 = 0, q_len = 0, kv_len = 0;

    for (int u = 0;; ++u) {
        const int st = u % kStages;
        if (!qmoe_tc::mbar_wait(&sh.full[st], (uint32_t)((u / kStages) & 1), kWaitLimit)) {
            if (lane == 0) attn_set_error(QMOE_ETIMEOUT);
            return;
        }
        const StageInfo in = sh.info[st];
        if (in.flags & kEnd) return;
        if (in.flags & kFirst) {
            if (kSel) q0 = in.b, q_len = 1;
            else q0 = a.q_start[in.b], q_len = a.q_start[in.b + 1] - q0, kv_len = a.kv_len[in.b];
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
                    c1[i] = __shfl_sync(QMOE_FULL_MASK, fa, 8 * t + 4 * i);
                    cz[i] = __shfl_sync(QMOE_FULL_MASK, fb, 8 * t + 4 * i);
                    m[nt][i] = kNoMax, l[nt][i] = 0.f, pz[nt][i] = 0.f;
                }
                if (NT > 1) sh.qc[nt][t] = make_float4(c1[0], c1[1], cz[0], cz[1]);
#pragma unroll
                for (int i = 0; i < 4 * VW; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[nt][i][j] = 0.f;
            }
            __syncwarp();
        }
        const unsigned char* stg = sh.stage[st];
        // With 8 rows both halves go through each phase together (two chains to overlap, one vote); with more, whose sums
        // take the registers, one after the other.
        constexpr int J = NT == 1 ? 2 : 1;
#pragma unroll 1
        for (int half = 0; half < 2; half += J) {
            float s[J][NT][4], sv[J][2], zv[J][2];
#pragma unroll
            for (int j = 0; j < J; ++j) {
                // ---- scores of 16 tokens
                const unsigned char* kb = stg + k_off + (half + j) * row_step;
                uint32_t kw[2][W];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    if constexpr (W == 4) {
                        const uint4 x = *(const uint4*)(kb + r * 8 * (D / 2));
                        kw[r][0] = x.x, kw[r][1] = x.y, kw[r][2] = x.z, kw[r][3] = x.w;
                    } else {
                        const uint2 x = *(const uint2*)(kb + r * 8 * (D / 2));
                        kw[r][0] = x.x, kw[r][1] = x.y;
                    }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[j][nt][i] = 0.f;
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
                        mma_16816(s[j][nt], x0 & 0x000F000Fu, x1 & 0x000F000Fu, y0 & 0x000F000Fu, y1 & 0x000F000Fu, qa.x, qa.y);
                        mma_16816(s[j][nt], x0 & 0x00F000F0u, x1 & 0x00F000F0u, y0 & 0x00F000F0u, y1 & 0x00F000F0u, qb.x, qb.y);
                    }
                }
                float sk[2], zk[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float2 kp = __half22float2(*(const __half2*)(stg + kp_off + (half + j) * pair_step + r * 32));
                    const float2 vp = __half22float2(*(const __half2*)(stg + vp_off + (half + j) * pair_step + r * 32));
                    sk[r] = kp.x, zk[r] = kp.y, sv[j][r] = vp.x, zv[j][r] = vp.y;
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    // (with more rows they would cost the registers that the sums need)
                    if (NT > 1) load_factors(&sh.qc[nt][t], c1, cz);
#pragma unroll
                    for (int r = 0; r < 2; ++r)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            s[j][nt][2 * r + i] = fmaf(c1[i], sk[r] * s[j][nt][2 * r + i], cz[i] * zk[r]);
                }
                // ---- tokens that some row does not see
                if (kSel && __builtin_expect(in.flags & kEdge, 0)) {
                    const int page = (tok0 + 16 * (half + j)) >> a.cache.page_shift;
                    const bool page_ok = (in.flags / kValid >> page) & 1;
                    const int sees = (in.flags / kPartial >> page) & 1 ? in.tile : P;
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int tok = ((tok0 + 16 * (half + j)) & (P - 1)) + (g >> 1) + 4 * (g & 1) + 8 * r;
                        if (page_ok && tok < sees) continue;
                        sv[j][r] = 0.f, zv[j][r] = 0.f;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int i = 0; i < 2; ++i) s[j][nt][2 * r + i] = -INFINITY;
                    }
                } else if (!kSel && __builtin_expect(in.flags & kEdge, 0)) {
                    int first = a.causal ? kv_len - q_len : kv_len - 1;
                    asm volatile("" : "+r"(first));      // nothing of this is made ahead of the branch to it
                    const bool page_ok = (in.flags / kValid >> ((tok0 + 16 * (half + j)) >> a.cache.page_shift)) & 1;
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int tok = in.tile * kTile + tok0 + 16 * (half + j) + (g >> 1) + 4 * (g & 1) + 8 * r;
                        const bool there = page_ok && tok < kv_len;
                        if (!there) sv[j][r] = 0.f, zv[j][r] = 0.f;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const int pos = a.causal ? first + (nt * 8 + 2 * t + i) / a.group : first;
                                // (below position 0 nothing is seen, wherever pos - window wraps to)
                                if (!there || tok > pos || (a.window && tok <= (int)((unsigned)pos - (unsigned)a.window))) s[j][nt][2 * r + i] = -INFINITY;
                            }
                    }
                }
            }
            // ---- move a row's m, rarely (a row of values without a scale, all z, counts as one with the least scale)
            float ls[J][2];
#pragma unroll
            for (int j = 0; j < J; ++j) ls[j][0] = lg2(fmaxf(fabsf(sv[j][0]), kLeastScale)), ls[j][1] = lg2(fmaxf(fabsf(sv[j][1]), kLeastScale));
            bool move = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float mx = fmaxf(s[0][nt][i] + ls[0][0], s[0][nt][2 + i] + ls[0][1]);
                    if (J == 2) mx = fmaxf(mx, fmaxf(s[J - 1][nt][i] + ls[J - 1][0], s[J - 1][nt][2 + i] + ls[J - 1][1]));
                    // (scores above 2^24, whose last place is worth more than the slack, are always looked at)
                    move |= mx > fmaf(fabsf(m[nt][i]), -0x1p-21f, m[nt][i] + kSlack);
                }
            if (__builtin_expect(__any_sync(QMOE_FULL_MASK, move), 0)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float fr[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float mx = fmaxf(s[0][nt][i] + ls[0][0], s[0][nt][2 + i] + ls[0][1]);
                        if (J == 2) mx = fmaxf(mx, fmaxf(s[J - 1][nt][i] + ls[J - 1][0], s[J - 1][nt][2 + i] + ls[J - 1][1]));
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(QMOE_FULL_MASK, mx, d));
                        const float m2 = fmaxf(m[nt][i], mx - kTop);
                        fr[i] = ex2(m[nt][i] - m2);
                        m[nt][i] = m2;
                        l[nt][i] *= fr[i], pz[nt][i] *= fr[i];
                    }
#pragma unroll
                    for (int i = 0; i < 4 * VW; ++i)
#pragma unroll
                        for (int q = 0; q < 4; ++q) o[nt][i][q] *= fr[q & 1];
                }
            }
#pragma unroll
            for (int j = 0; j < J; ++j) {
                // ---- probabilities, as the value product's operand
                uint32_t pf[NT][2];
                const float w0 = sv[j][0], w1 = sv[j][1];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float p[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) p[i] = ex2(s[j][nt][i] - m[nt][i & 1]);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        l[nt][i] += p[i] + p[2 + i];
                        pz[nt][i] = fmaf(p[i], zv[j][0], fmaf(p[2 + i], zv[j][1], pz[nt][i]));
                    }
                    pf[nt][0] = movmatrix(half2_bits(p[0] * w0, p[1] * w0));
                    pf[nt][1] = movmatrix(half2_bits(p[2] * w1, p[3] * w1));
                }
                // ---- values: words of tokens t, t + 4, t + 8, t + 12 of the 16
                const unsigned char* vb = stg + v_off + (half + j) * row_step;
                uint32_t vw[4][VW];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    if constexpr (VW == 2) {
                        const uint2 x = *(const uint2*)(vb + r * 4 * (D / 2));
                        vw[r][0] = x.x, vw[r][1] = x.y;
                    } else {
                        vw[r][0] = *(const uint32_t*)(vb + r * 4 * (D / 2));
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
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.empty[st]);

        if (in.flags & kLast) {
            const int rows = q_len * a.group;
            const bool whole = (in.flags & kWholeStart) && (in.flags & kWholeEnd);
            float* part = part_of(parts, blockIdx.x, (in.flags & kWholeStart) ? 1 : 0, 8 * NT, D);
            constexpr float unit = 16777216.f;
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
                if (!meet(&sh.joint, met)) return;
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
                if (!meet(&sh.joint, met)) return;
            }
        }
    }
}

// Joins the parts of items that several blocks shared: block (c, slice) those of the item that block c began and left
// unfinished.  Its parts are slot 1 of block c and slot 0 of blocks c + 1 .. rec.last; a group of head_dim / 4 lanes
// adds up a row's parts, or every group some of them where there are many.
constexpr int kJoinThreads = 128;

template <int D, bool kSel>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(AttnArgs a, const SplitItem* items, const float* parts, int part_rows) {
    constexpr int LANES = D / 4, GROUPS = kJoinThreads / LANES;
    __shared__ float4 acc_s[GROUPS][LANES];
    __shared__ float2 ml_s[GROUPS];
    depend_wait();
    const SplitItem it = items[blockIdx.x];
    const int n_parts = it.last - (int)blockIdx.x + 1;
    if (n_parts < 2) return;
    depend_launch();
    const int q0 = kSel ? it.b : a.q_start[it.b];
    const int rows = kSel ? a.group : min(part_rows, (a.q_start[it.b + 1] - q0) * a.group - it.rb * part_rows);
    const int grp = threadIdx.x / LANES, ln = threadIdx.x - grp * LANES;
    const bool wide = n_parts > 4;
    for (int r0 = blockIdx.y * (wide ? 1 : GROUPS); r0 < rows; r0 += gridDim.y * (wide ? 1 : GROUPS)) {
        const int r = wide ? r0 : min(r0 + grp, rows - 1);
        float mm = kNoMax, ll = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int i = wide ? grp : 0; i < n_parts; i += wide ? GROUPS : 1) {
            const float* p = part_of((float*)parts, blockIdx.x + i, i == 0, part_rows, D);
            const float2 ml = *(const float2*)(p + (size_t)part_rows * D + 2 * r);
            const float4 x = *(const float4*)(p + (size_t)r * D + 4 * ln);
            const float m2 = fmaxf(mm, ml.x), fa = ex2(mm - m2), fb = ex2(ml.x - m2);
            mm = m2;
            ll = ll * fa + ml.y * fb;
            acc.x = acc.x * fa + x.x * fb, acc.y = acc.y * fa + x.y * fb;
            acc.z = acc.z * fa + x.z * fb, acc.w = acc.w * fa + x.w * fb;
        }
        if (wide) {
            acc_s[grp][ln] = acc;
            if (ln == 0) ml_s[grp] = make_float2(mm, ll);
            __syncthreads();
            if (grp == 0) {
#pragma unroll
                for (int g = 1; g < GROUPS; ++g) {
                    const float2 ml = ml_s[g];
                    const float4 x = acc_s[g][ln];
                    const float m2 = fmaxf(mm, ml.x), fa = ex2(mm - m2), fb = ex2(ml.x - m2);
                    mm = m2;
                    ll = ll * fa + ml.y * fb;
                    acc.x = acc.x * fa + x.x * fb, acc.y = acc.y * fa + x.y * fb;
                    acc.z = acc.z * fa + x.z * fb, acc.w = acc.w * fa + x.w * fb;
                }
            }
            __syncthreads();
        }
        if (wide ? grp == 0 : r0 + grp < rows) {
            const float inv = ll > 0.f ? 1.f / ll : (ll == 0.f ? 0.f : ll);
            const int row = it.rb * part_rows + r, n = row / a.group, h = it.kh * a.group + row - n * a.group;
            uint2 w;
            w.x = (uint32_t)f32_to_bf16(acc.x * inv) | ((uint32_t)f32_to_bf16(acc.y * inv) << 16);
            w.y = (uint32_t)f32_to_bf16(acc.z * inv) | ((uint32_t)f32_to_bf16(acc.w * inv) << 16);
            *(uint2*)(a.out + ((int64_t)(q0 + n) * a.n_q_heads + h) * D + 4 * ln) = w;
        }
    }
}

// ---------------------------------------------------------------- many query rows: tensor-core tiles
//
// A block takes 256 query rows of one (request, kv head) as two tiles of 128 and walks the keys 128 at
// a time: S = Q K^T into tensor memory, P = 2^(S c - m) back into tensor memory as fp16 (over S), O += P V
// (tcgen05, both products' accumulators fp32, P as the operand from tensor memory).  While one tile's
// softmax runs, the tensor core works on the other.  The codes are expanded once per block to fp16 in
// shared memory, k = s u + z rounded once to 11 bits (bf16 inputs and outputs have 8); P and the
// values are fp16 too, statistics and sums fp32.  Queries carry a power of two per row (exact), so any
// bf16 magnitude is inside fp16's range.  The running maximum moves, and O is rescaled, only when a
// row's weights by it pass 2^14; P carries 2^6, so that small weights stay above fp16's subnormals.
//
// Measured: 2048 query tokens behind 30011 cached ones, 32 query heads on 4 key heads of 128, 772 us = 1.35
// PFLOP/s, 72 % of cuBLAS's bf16 rate (690 to 775 by machine).  Leaving parts out in turn (no exponentials -5 %, one product of
// eight -1 %) shows no single limit: the four roles share the schedulers' issue slots (about 60 % used) and
// the instruction caches, which is why every loop is short.  A 64-key step has two score buffers a tile of
// rows, so that a softmax finds its next scores ready (128-key steps with one buffer: 951 us then, 895 with).
//
// Roles, one block per SM: 2 x 4 softmax warps (a thread per row), 4 warps that expand keys and values,
// a warp for each tile of rows that issues its products, one that copies pages.  For 128 keys at 256 rows
// and head_dim 128 the tensor core needs about 2500 cycles (its 64-column products run at 45 cycles instead
// of 32), the exponentials 1030 of a scheduler's; the walk takes 3400.
//
// Work is dealt out as in the few-row path: all (rows, kv head) items' key tiles in a row, in equal
// runs; items that several blocks share are joined by join_kernel.
constexpr int kKeys = 128;                       // keys of a tile (expanded at once)
constexpr int kStep = 64;                        // keys of a softmax step
constexpr int kTileItemCost = 3;                 // what beginning and ending an item costs, in tiles
constexpr int kRows = 256;                       // query rows of an item
constexpr int kTileThreads = 512;
constexpr int kExpandWarp = 8, kIssueWarp = 12, kCopyWarp = 13;
constexpr int kRawStages = 2, kExpanded = 3, kInfo = 8;
constexpr int kPlanTile = 1024;

// Work list of the tile path, in the workspace: pairs (request, block of 256 rows) in order.
struct alignas(16) PairInfo {
    long long unit;              // units before the pair: its kv heads' key tiles, and kTileItemCost for each item
    int n;                       // key tiles of one kv head, lo .. lo + n - 1
    int b, rb, q0, q_len, kv_len, lo;
    int s[2], e[2];              // steps, from 2 lo, that the two tiles of 128 rows see
    int pad[3];
};
static_assert(sizeof(PairInfo) == 64, "read as sixteen words");

struct TilePlan {
    int32_t* pair_start;         // [B + 1]
    int32_t* pair_b;             // [pairs]
    PairInfo* pairs;
    long long* total;            // units of the batch
    SplitItem* items;            // [blocks]
    int max_pairs;
};

// Blocks of `step` keys, [lo, hi), that rows [r0, r1) of a request see.
__device__ __forceinline__ void key_steps(const AttnArgs& a, int q_len, int kv_len, int r0, int r1, int step, int* lo, int* hi) {
    const int first = a.causal ? kv_len - q_len : kv_len - 1;
    const int p0 = a.causal ? first + r0 / a.group : first, p1 = a.causal ? first + (r1 - 1) / a.group : first;
    const int k1 = min(kv_len, p1 + 1), k0 = first_seen(a, p0);
    *lo = k0 / step;
    *hi = k1 > k0 ? (k1 + step - 1) / step : *lo;
}

// Inclusive scan over the block's 1024 threads; *total gets the sum.
__device__ __forceinline__ long long block_scan(long long v, long long* total) {
    __shared__ long long sums[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(QMOE_FULL_MASK, v, d);
        if (lane >= d) v += o;
    }
    if (lane == 31) sums[warp] = v;
    __syncthreads();
    long long before = 0, all = 0;
    for (int w = 0; w < 32; ++w) {
        if (w < warp) before += sums[w];
        all += sums[w];
    }
    __syncthreads();
    *total = all;
    return v + before;
}

__global__ void __launch_bounds__(kPlanTile) tile_plan_kernel(AttnArgs a, TilePlan p, int min_rows) {
    const int tid = threadIdx.x;
    depend_launch();
    long long base = 0, total;
    for (int b0 = 0; b0 < a.B; b0 += kPlanTile) {
        const int b = b0 + tid;
        int q0, q_len = 0, kv_len, pairs = 0;
        if (b < a.B && request(a, b, &q0, &q_len, &kv_len, min_rows == 0) && q_len * a.group > min_rows)
            pairs = (q_len * a.group + kRows - 1) / kRows;
        const long long end = base + block_scan(pairs, &total);
        if (b < a.B) {
            p.pair_start[b] = (int)(end - pairs);
            for (int i = 0; i < pairs; ++i)
                if (end - pairs + i < p.max_pairs) p.pair_b[end - pairs + i] = b;
        }
        base += total;
    }
    const int n_pairs = (int)min(base, (long long)p.max_pairs);
    if (tid == 0) p.pair_start[a.B] = n_pairs;
    __syncthreads();
    base = 0;
    for (int i0 = 0; i0 < n_pairs; i0 += kPlanTile) {
        const int i = i0 + tid;
        PairInfo w{};
        if (i < n_pairs) {
            w.b = p.pair_b[i], w.q0 = a.q_start[w.b], w.q_len = a.q_start[w.b + 1] - w.q0, w.kv_len = a.kv_len[w.b];
            w.rb = i - p.pair_start[w.b];
            const int r0 = w.rb * kRows, rows = w.q_len * a.group;
            int hi;
            key_steps(a, w.q_len, w.kv_len, r0, min(r0 + kRows, rows), kKeys, &w.lo, &hi);
            w.n = max(1, hi - w.lo);
            for (int x = 0; x < 2; ++x) {
                if (r0 + 128 * x >= rows) continue;
                int lo;
                key_steps(a, w.q_len, w.kv_len, r0 + 128 * x, min(r0 + 128 * x + 128, rows), kStep, &lo, &hi);
                w.s[x] = lo - 2 * w.lo, w.e[x] = hi - 2 * w.lo;
            }
        }
        const long long n = w.n ? (long long)(w.n + kTileItemCost) * a.cache.n_kv_heads : 0;
        const long long end = base + block_scan(n, &total);
        if (i < n_pairs) {
            w.unit = end - n;
            p.pairs[i] = w;
        }
        base += total;
    }
    if (tid == 0) *p.total = base;
    depend_wait();      // nothing before is read, but whoever waits for this kernel waits for those
}

struct TileCursor {
    PairInfo w;                  // the pair
    long long u, u1;             // next unit, end of the run
    int pair, kh, t0, t1, whole;
    int s[2], e[2];              // the tiles' steps inside [2 t0, 2 t1)
};

template <int D>
struct TileShared {
    // operand tiles in the 128-byte-swizzled K-major layout: atoms of 64 columns, a row of an atom 128 bytes, the 16-byte
    // piece i of row r at place i ^ (r % 8)
    // (a step's 64 keys: half the rows of K's atoms, one atom of V)
    static constexpr int kQAtom = 128 * 128, kVAtom = D * 128;      // Q and K (rows: queries, keys), V (rows: head values)
    static constexpr int kBuf = 128 * D * 2;
    alignas(1024) unsigned char q[2][kBuf];
    alignas(1024) unsigned char kv[kExpanded][kBuf];
    alignas(128) unsigned char raw[kRawStages][kKeys * (D + 8)];
    alignas(16) unsigned char rows[8][32 * 80];                  // a softmax warp's 64 bytes a row, on their way out
    uint64_t raw_full[kRawStages], raw_empty[kRawStages], kv_full[kExpanded], kv_empty[kExpanded];
    uint64_t q_full[2], s_full[2][2], p_full[2][2], o_full[2][2], fin[2];      // [tile of rows][step parity]
    uint32_t valid[kInfo];                                       // per tile: which groups of 16 tokens have a page
    uint32_t tmem;
    TileCursor cur[kTileThreads / 32];
};

// The next item of the run, or false: the pair's rows, kv head kh, key tiles w.lo + [t0, t1).  Each warp keeps its own
// cursor in shared memory.  Returns whether the place holds tiles (a run may begin or end in an item's extra units).
__device__ __forceinline__ bool place_item(const AttnArgs& a, TileCursor& c, bool first) {
    long long off = 0;
    if (first) {
        off = c.u - c.w.unit;
        c.kh = (int)(off / (c.w.n + kTileItemCost));
        off -= (long long)c.kh * (c.w.n + kTileItemCost);
    }
    const long long span = min(c.w.n + kTileItemCost - off, c.u1 - c.u);
    c.t0 = (int)min(off, (long long)c.w.n);
    c.t1 = (int)min(off + span, (long long)c.w.n);
    c.whole = c.t0 == 0 && c.t1 == c.w.n;
    for (int x = 0; x < 2; ++x) {
        const int s = max(c.w.s[x], 2 * c.t0), e = min(c.w.e[x], 2 * c.t1);
        c.s[x] = s < e ? s : 0, c.e[x] = s < e ? e : 0;
    }
    c.u += span;
    return c.t0 < c.t1;
}

// By one thread.
__device__ __forceinline__ bool next_item_alone(const AttnArgs& a, const TilePlan& p, TileCursor& c, bool first) {
    for (;; first = false) {
        if (c.u >= c.u1) return false;
        if (first || ++c.kh == a.cache.n_kv_heads) {
            c.kh = 0;
            if (!first) ++c.pair;
            const uint4* src = (const uint4*)(p.pairs + c.pair);
            const uint4 v[4] = {src[0], src[1], src[2], src[3]};
            for (int i = 0; i < 4; ++i) ((uint4*)&c.w)[i] = v[i];
        }
        if (place_item(a, c, first)) return true;
    }
}

// By a warp; ahead holds the pair after this one (a word a lane), loaded while this one is worked on.
__device__ __forceinline__ bool next_item(const AttnArgs& a, const TilePlan& p, int n_pairs, TileCursor& c, bool first, uint32_t& ahead) {
    const int lane = threadIdx.x & 31;
    for (;; first = false) {
        __syncwarp();
        if (c.u >= c.u1) return false;
        const bool load = first || c.kh + 1 == a.cache.n_kv_heads;
        const int pair = c.pair + (first ? 0 : 1);
        __syncwarp();
        if (load) {
            if (first && lane < 16) ahead = ((const uint32_t*)(p.pairs + pair))[lane];
            if (lane < 16) ((uint32_t*)&c.w)[lane] = ahead;
            if (lane < 16 && pair + 1 < n_pairs) ahead = ((const uint32_t*)(p.pairs + pair + 1))[lane];
            __syncwarp();
        }
        bool some = false;
        if (lane == 0) {
            if (load)
                c.kh = 0, c.pair = pair;
            else
                ++c.kh;
            some = place_item(a, c, first);
        }
        __syncwarp();      // all lanes read what lane 0 wrote (the shuffle orders no memory)
        if (__shfl_sync(QMOE_FULL_MASK, (int)some, 0)) return true;
    }
}

// Bounded wait; false when the tries ran out.  A few instructions, as every role's loop holds some of these and the
// roles' code shares the instruction caches; the hardware suspends the thread for part of each try.
constexpr uint32_t kTries = 1u << 21;
__device__ __forceinline__ bool tile_wait(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n .reg .b32 n;\n mov.b32 n, %3;\n"
        "AGAIN:\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n @p bra DONE;\n"
        " sub.u32 n, n, 1;\n setp.ne.u32 p, n, 0;\n @p bra AGAIN;\n setp.eq.u32 p, n, 1;\n"
        "DONE:\n selp.b32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(qmoe_tc::smem_u32(bar)), "r"(parity), "n"(kTries)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ void tmem_load32(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_store32(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

// Ends the loads before it; naming the registers keeps their uses behind it.
__device__ __forceinline__ void tmem_wait_load(uint32_t* r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                   "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}

// 64 columns, complete: the wait is in the same statement, so that the registers are used in place.
__device__ __forceinline__ void tmem_load64(uint32_t taddr, uint32_t (&r)[64]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
        "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, "
        "%22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32, %33, %34, %35, %36, %37, %38, %39, %40, %41, "
        "%42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, "
        "%62, %63 "
        "}, [%64];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
          "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
          "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
          "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
          "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(taddr)
        : "memory");
}

// Scores of 64 keys outside [lo, hi], or in a group of 16 whose bit of `groups` is clear, become -inf.
__device__ __forceinline__ void mask64(uint32_t* s, int lo, int hi, uint32_t groups) {
    asm volatile("" : "+r"(lo), "+r"(hi), "+r"(groups));      // nothing of this is made ahead of the branch to it
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int l = lo - 32 * h, u = hi - 32 * h;
        uint32_t keep = u < 0 ? 0u : u >= 31 ? 0xFFFFFFFFu : (2u << u) - 1u;
        keep &= l <= 0 ? 0xFFFFFFFFu : l > 31 ? 0u : 0xFFFFFFFFu << l;
        keep &= ((groups >> (2 * h)) & 1 ? 0xFFFFu : 0u) | ((groups >> (2 * h + 1)) & 1 ? 0xFFFF0000u : 0u);
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (!((keep >> i) & 1)) s[32 * h + i] = 0xFF800000u;
    }
}

__device__ __forceinline__ void tmem_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tmem_load16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_store16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// Two fp32 values in one 64-bit register: one instruction for both.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(lo), "f"(hi));
    return p;
}
__device__ __forceinline__ void unpair(uint64_t p, float* lo, float* hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(*lo), "=f"(*hi) : "l"(p)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// Arrival of a warp: one operation on the barrier, after all lanes.
__device__ __forceinline__ void arrive_warp(uint64_t* bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// One lane of a converged warp, always the same one.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred P;\n elect.sync _|P, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, P;\n}\n" : "=r"(p));
    return p != 0;
}

// Descriptor of a 128-byte-swizzled K-major operand, 8-row groups 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_sw128(const void* p) {
    return (uint64_t)((qmoe_tc::smem_u32(p) & 0x3FFFFu) >> 4) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 | 1ull << 46 | 2ull << 61;
}

// D += A B, the operands' descriptors as low words (plus off) and a high word: built at the instruction, so that they
// are not all kept in registers across the loop.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi, uint32_t off,
                                       uint32_t idesc, uint32_t accum) {
    asm volatile(
        "{\n .reg .pred p;\n .reg .b32 x, y;\n .reg .b64 A, B;\n setp.ne.b32 p, %7, 0;\n"
        " add.u32 x, %1, %5;\n add.u32 y, %3, %5;\n mov.b64 A, {x, %2};\n mov.b64 B, {y, %4};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], A, B, %6, p;\n}\n" ::"r"(d),
        "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(off), "r"(idesc), "r"(accum)
        : "memory");
}

// The same with A from tensor memory (fp16 pairs along K in 32-bit columns, from a + a_off).
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t a_off, uint32_t b_lo, uint32_t b_hi, uint32_t off,
                                       uint32_t idesc, uint32_t accum) {
    asm volatile(
        "{\n .reg .pred p;\n .reg .b32 x, y;\n .reg .b64 B;\n setp.ne.b32 p, %7, 0;\n"
        " add.u32 x, %1, %2;\n add.u32 y, %3, %5;\n mov.b64 B, {y, %4};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [x], B, %6, p;\n}\n" ::"r"(d),
        "r"(a), "r"(a_off), "r"(b_lo), "r"(b_hi), "r"(off), "r"(idesc), "r"(accum)
        : "memory");
}

// Four registers of a word of codes, (value 8w + 2i, value 8w + 2i + 1) each, as the integers 0..15 in fp16: 1024 + u
// (1024 + 16 u one nibble up) is an or into fp16's pattern of 1024, and taking the 1024 off is exact.
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t mask, uint32_t bits) {
    uint32_t d;      // one instruction; the compiler makes two of the same in C
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(mask), "r"(bits));
    return d;
}

__device__ __forceinline__ void code_integers(uint32_t w, __half2 (&u)[4]) {
    const uint32_t h = w >> 8, magic = 0x64006400u;
    const uint32_t x[4] = {and_or(w, 0x000F000Fu, magic), and_or(w, 0x00F000F0u, magic), and_or(h, 0x000F000Fu, magic),
                           and_or(h, 0x00F000F0u, magic)};
    const __half2 one = __float2half2_rn(1024.f), off = __float2half2_rn(-64.f), sixteenth = __float2half2_rn(0.0625f);
    u[0] = __hsub2(*(const __half2*)&x[0], one);
    u[1] = __hfma2(*(const __half2*)&x[1], sixteenth, off);
    u[2] = __hsub2(*(const __half2*)&x[2], one);
    u[3] = __hfma2(*(const __half2*)&x[3], sixteenth, off);
}

__device__ __forceinline__ uint32_t h2(const __half2& h) { return *(const uint32_t*)&h; }

// In key group (of 8) o of a V tile, place i holds key i ^ v_swap(o): the expanding lanes of four groups then read their
// words from different banks, and the softmax packs its pairs in the same order.
template <int D>
__host__ __device__ constexpr int v_swap(int o) {
    return D == 128 ? (o & 1) : (o & 3);
}

// Where row r of the item's rows is in q and out; -1 past the request's rows.
template <int D>
__device__ __forceinline__ int64_t row_at(const AttnArgs& a, const TileCursor& c, int r) {
    if (r >= c.w.q_len * a.group) return -1;
    const int n = r / a.group;
    return ((int64_t)(c.w.q0 + n) * a.n_q_heads + c.kh * a.group + r - n * a.group) * D;
}

// A warp's 32 query rows into the query tile, D / 8 lanes a row (a thread a row would touch 32 cache lines a load), each
// row's largest magnitude scaled to [2^14, 2^15).  Returns the factor that takes the thread's own row's scores to log2
// units.  Rows past the request's are zeros.
template <int D>
__device__ __forceinline__ float put_rows(const AttnArgs& a, const TileCursor& c, int x, TileShared<D>& sh) {
    if (c.e[x] <= c.s[x]) return 0.f;
    constexpr int LANES = D / 8, PER = 32 / LANES, LOADS = 32 / PER;      // lanes of a row, rows of a load, loads
    const int lane = threadIdx.x & 31, row0 = ((threadIdx.x >> 5) & 3) * 32, sub = lane / LANES, piece = lane % LANES;
    const int64_t mine = row_at<D>(a, c, c.w.rb * kRows + x * 128 + row0 + lane);
    int e_mine = 0;
#pragma unroll 1
    for (int i0 = 0; i0 < LOADS; i0 += 8) {
        uint4 raw[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t at = __shfl_sync(QMOE_FULL_MASK, mine, (i0 + i) * PER + sub);
            raw[i] = at >= 0 ? *(const uint4*)(a.q + at + piece * 8) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint4 v = raw[i];
            float mx = fmaxf(fmaxf(fmaxf(fabsf(bf16_lo(v.x)), fabsf(bf16_hi(v.x))), fmaxf(fabsf(bf16_lo(v.y)), fabsf(bf16_hi(v.y)))),
                             fmaxf(fmaxf(fabsf(bf16_lo(v.z)), fabsf(bf16_hi(v.z))), fmaxf(fabsf(bf16_lo(v.w)), fabsf(bf16_hi(v.w)))));
#pragma unroll
            for (int d = LANES / 2; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(QMOE_FULL_MASK, mx, d));
            const int e = mx > 0.f ? min(max((int)(__float_as_uint(mx) >> 23) - 127, -100), 126) : 0;
            const float up = a.scale < 0.f ? -pow2i(14 - e) : pow2i(14 - e);
            const int r = row0 + (i0 + i) * PER + sub;
            *(uint4*)(sh.q[x] + r * 128 + (piece >> 3) * TileShared<D>::kQAtom + (((piece & 7) ^ (r & 7)) << 4)) =
                make_uint4(half2_bits(bf16_lo(v.x) * up, bf16_hi(v.x) * up), half2_bits(bf16_lo(v.y) * up, bf16_hi(v.y) * up),
                           half2_bits(bf16_lo(v.z) * up, bf16_hi(v.z) * up), half2_bits(bf16_lo(v.w) * up, bf16_hi(v.w) * up));
            const int of = __shfl_sync(QMOE_FULL_MASK, e, (lane % PER) * LANES);
            if (lane / PER == i0 + i) e_mine = of;
        }
    }
    qmoe_tc::fence_async_shared();
    arrive_warp(&sh.q_full[x]);
    // not 0, so that a masked score's -inf stays one
    return fmaxf(fabsf(a.scale) * 1.4426950408889634f * pow2i(e_mine - 14), 1.2e-38f);
}

// 64 bytes of each of a warp's 32 rows to where the rows go (dst: the thread's own row's place, or NULL), four lanes a row.
__device__ __forceinline__ void rows_out(unsigned char* stage, const uint4 (&v)[4], unsigned char* dst) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < 4; ++j) *(uint4*)(stage + lane * 80 + 16 * j) = v[j];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 8 * i + (lane >> 2);
        unsigned char* to = (unsigned char*)__shfl_sync(QMOE_FULL_MASK, (unsigned long long)dst, r);
        const uint4 x = *(const uint4*)(stage + r * 80 + (lane & 3) * 16);
        if (to) *(uint4*)(to + (lane & 3) * 16) = x;
    }
    __syncwarp();
}

template <int D>
__global__ void __launch_bounds__(kTileThreads, 1) tile_kernel(AttnArgs a, TilePlan plan, float* parts) {
    using Sh = TileShared<D>;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    Sh& sh = *(Sh*)smem_raw;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    depend_launch();
    depend_wait();
    const int n_pairs = plan.pair_start[a.B];
    const long long total = *plan.total;
    const long long chunk = max(1LL, (total + gridDim.x - 1) / gridDim.x);
    if (tid == 32 * kCopyWarp) plan.items[blockIdx.x] = SplitItem{0, 0, 0, -1};
    const long long first_unit = (long long)blockIdx.x * chunk, end_unit = min(first_unit + chunk, total);
    if (first_unit >= end_unit) return;
    if (tid == 0) {
        for (int i = 0; i < kRawStages; ++i) qmoe_tc::mbar_init(&sh.raw_full[i], 1), qmoe_tc::mbar_init(&sh.raw_empty[i], 4);
        for (int i = 0; i < kExpanded; ++i) qmoe_tc::mbar_init(&sh.kv_full[i], 4), qmoe_tc::mbar_init(&sh.kv_empty[i], 2);
        for (int i = 0; i < 2; ++i) {
            qmoe_tc::mbar_init(&sh.q_full[i], 4);
            for (int j = 0; j < 2; ++j) {
                qmoe_tc::mbar_init(&sh.s_full[i][j], 1);
                qmoe_tc::mbar_init(&sh.p_full[i][j], 4);
                qmoe_tc::mbar_init(&sh.o_full[i][j], 1);
            }
        }
        for (int i = 0; i < 2; ++i) qmoe_tc::mbar_init(&sh.fin[i], 1);
        qmoe_tc::fence_mbar_init();
    }
    if (warp == kIssueWarp) qmoe_tc::tmem_alloc(&sh.tmem, 512);
    if (warp == kCopyWarp) {
        // last pair that starts at or before the run's first unit: 32 probes at a time
        int lo = 0, hi = n_pairs;     // the pair is in [lo, hi)
        while (hi - lo > 1) {
            const int step = (hi - lo + 31) / 32, at = lo + lane * step;
            const unsigned below = __ballot_sync(QMOE_FULL_MASK, at < hi && plan.pairs[at].unit <= first_unit);
            const int k = 31 - __clz(below);      // bit 0 is always set
            const int nlo = min(lo + k * step, hi);
            hi = min(nlo + step, hi);
            lo = nlo;
        }
        if (lane < kTileThreads / 32) sh.cur[lane].u = first_unit, sh.cur[lane].u1 = end_unit, sh.cur[lane].pair = lo;
    }
    __syncthreads();
    qmoe_tc::tc_fence_after();
    // all 512 columns were taken, so they begin at column 0
    constexpr uint32_t tmem = 0;
    TileCursor& c = sh.cur[warp];
    uint32_t ahead = 0;

    bool ok = true;
    if (warp < kExpandWarp) {
        // ---- softmax: a thread per query row.  2 x 128 threads of 160 registers and 256 of 96: what the block was launched with
        asm volatile("setmaxnreg.inc.sync.aligned.u32 160;");
        const int x = warp >> 2, row = tid & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;           // 32 lanes a warp, lane index in bits 16..
        const uint32_t ts = tmem + x * 128 + lanes, to = tmem + 256 + x * 128 + lanes;
        uint32_t n_s = 0;                                            // steps done (the step barriers take turns)
        int tiles = 0;                                               // tiles of the run before the item
        float factor = 0.f;                                          // of the item's scores, in log2 units
        bool more = next_item(a, plan, n_pairs, c, true, ahead);
        if (more) factor = put_rows<D>(a, c, x, sh);
        while (more) {
            const int t_s = c.s[x], t_e = c.e[x], t0 = c.t0, lo = c.w.lo;
            const bool whole = c.whole, some = t_e > t_s;
            const int r = c.w.rb * kRows + x * 128 + row;
            const int n = r / a.group;
            const int64_t base = row_at<D>(a, c, r);
            const bool live = base >= 0;
            float m = kNoMax, l = 0.f;
            const int first = a.causal ? c.w.kv_len - c.w.q_len : c.w.kv_len - 1;
            const int pos = a.causal ? first + n : first;
            const int k_hi = min(pos, c.w.kv_len - 1), k_lo = first_seen(a, pos);    // keys seen: [k_lo, k_hi]
            bool far = false;
            uint64_t mul2 = pair(factor, factor), nb2 = pair(6.f - m, 6.f - m);
            for (int t = t_s; t < t_e && ok; ++t) {
                const uint32_t tb = ts + (n_s & 1) * kStep;
                ok = tile_wait(&sh.s_full[x][n_s & 1], (n_s >> 1) & 1);
                if (!(ok = __all_sync(QMOE_FULL_MASK, ok))) break;
                qmoe_tc::tc_fence_after();
                const int j0 = lo * kKeys + t * kStep;
                const uint32_t valid = sh.valid[(tiles + (t >> 1) - t0) % kInfo] >> (4 * (t & 1)) & 15u;
                // (by a vote, so that it is a branch: predicated, the 64 tests would be issued in every step)
                const bool edge = __any_sync(QMOE_FULL_MASK, j0 + kStep - 1 > k_hi || j0 < k_lo || valid != 15u);
                // The weights are taken with the maximum as it stands; only when a row's sum shows that it has grown too
                // far (or there is none yet) the scores are read again, for their maximum and for the weights by it.
                uint32_t sr[kStep];
                float e0, e1;
#pragma unroll 1
                for (bool again = false;; again = true) {
                    tmem_load64(tb, sr);
                    if (__builtin_expect(edge, 0)) mask64(sr, k_lo - j0, k_hi - j0, valid);
                    if (__builtin_expect(far, 0)) {
#pragma unroll
                        for (int i = 0; i < kStep; ++i) sr[i] = __float_as_uint(__uint_as_float(sr[i]) * factor);
                    }
                    uint64_t l2[2] = {0, 0};
#pragma unroll
                    for (int i = 0; i < kStep; i += 2) {
                        unpair(fma2(pair(__uint_as_float(sr[i]), __uint_as_float(sr[i + 1])), mul2, nb2), &e0, &e1);
                        e0 = ex2(e0), e1 = ex2(e1);
                        l2[(i >> 1) & 1] = add2(l2[(i >> 1) & 1], pair(e0, e1));
                        sr[i] = __float_as_uint(e0), sr[i + 1] = __float_as_uint(e1);
                    }
                    unpair(add2(l2[0], l2[1]), &e0, &e1);
                    e0 += e1;
                    if (again || !__any_sync(QMOE_FULL_MASK, !(e0 < 16384.f))) break;
                    tmem_load64(tb, sr);
                    if (edge) mask64(sr, k_lo - j0, k_hi - j0, valid);
                    float mx = -INFINITY;
#pragma unroll
                    for (int i = 0; i < kStep; i += 2) mx = fmaxf(mx, fmaxf(__uint_as_float(sr[i]), __uint_as_float(sr[i + 1])));
                    const float m2 = fmaxf(m, mx * factor), f = ex2(m - m2);
                    m = m2;
                    l *= f;
                    if (t > t_s) {
                        // O as the step before left it
                        ok = tile_wait(&sh.o_full[x][(n_s - 1) & 1], ((n_s - 1) >> 1) & 1);
                        if (!(ok = __all_sync(QMOE_FULL_MASK, ok))) break;
                        qmoe_tc::tc_fence_after();
#pragma unroll 1
                        for (int i = 0; i < D; i += 16) {
                            uint32_t orr[16];
                            tmem_load16(to + i, orr);
#pragma unroll
                            for (int j = 0; j < 16; ++j) orr[j] = __float_as_uint(__uint_as_float(orr[j]) * f);
                            tmem_store16(to + i, orr);
                        }
                    }
                    // the fused product is not rounded before m is taken off: where m is so large that this shows, round first
                    far = __any_sync(QMOE_FULL_MASK, fabsf(m) > 65536.f && m != kNoMax);
                    mul2 = far ? pair(1.f, 1.f) : pair(factor, factor), nb2 = pair(6.f - m, 6.f - m);
                }
                if (!ok) break;
                l += e0;
                uint32_t pr[kStep / 2];
#pragma unroll
                for (int i = 0; i < kStep / 2; ++i)
                    pr[i] = half2_bits(__uint_as_float(sr[(2 * i) ^ v_swap<D>(i >> 2)]), __uint_as_float(sr[(2 * i + 1) ^ v_swap<D>(i >> 2)]));
                tmem_store32(tb, pr);      // over the scores
                tmem_wait_store();
                qmoe_tc::tc_fence_before();
                arrive_warp(&sh.p_full[x][n_s & 1]);
                ++n_s;
            }
            if (!ok) break;
            tiles += c.t1 - t0;
            // the next item's rows go into place first (this item's scores are done with them), so that its first products
            // run while this one's sums are written
            more = next_item(a, plan, n_pairs, c, false, ahead);
            if (more) factor = put_rows<D>(a, c, x, sh);
            if (some) ok = tile_wait(&sh.o_full[x][(n_s - 1) & 1], ((n_s - 1) >> 1) & 1);
            if (!(ok = __all_sync(QMOE_FULL_MASK, ok))) break;
            qmoe_tc::tc_fence_after();
            const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
            float* part = part_of(parts, blockIdx.x, t0 == 0 ? 1 : 0, kRows, D) + (size_t)(x * 128 + row) * D;
#pragma unroll 1
            for (int i = 0; i < D; i += 32) {
                uint32_t orr[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) orr[j] = 0;
                if (some) {
                    tmem_load32(to + i, orr);
                    tmem_wait_load(orr);
                }
                uint4 v[4];
                if (whole) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t w[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const __nv_bfloat162 b2 = __floats2bfloat162_rn(__uint_as_float(orr[8 * j + 2 * k]) * inv, __uint_as_float(orr[8 * j + 2 * k + 1]) * inv);
                            w[k] = *(const uint32_t*)&b2;
                        }
                        v[j] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    rows_out(sh.rows[warp], v, live ? (unsigned char*)(a.out + base + i) : nullptr);
                } else {
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) v[j] = make_uint4(orr[16 * hf + 4 * j], orr[16 * hf + 4 * j + 1], orr[16 * hf + 4 * j + 2], orr[16 * hf + 4 * j + 3]);
                        rows_out(sh.rows[warp], v, live ? (unsigned char*)(part + i + 16 * hf) : nullptr);
                    }
                }
            }
            if (live && !whole)
                *(float2*)(part_of(parts, blockIdx.x, t0 == 0 ? 1 : 0, kRows, D) + (size_t)kRows * D + 2 * (x * 128 + row)) = make_float2(m, l);
            qmoe_tc::tc_fence_before();
        }
    } else if (warp < kIssueWarp) {
        // ---- expand codes to fp16 tiles
        asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
        const int i = tid - kExpandWarp * 32;
        const int P = 1 << a.cache.page_shift, P1 = P - 1;
        // keys: thread i holds key i; which 16-byte piece first differs with the row, so that eight rows read different banks
        const uint32_t k_page = (uint32_t)(i >> a.cache.page_shift) * a.cache.head_bytes;
        const uint32_t k_row = k_page + (uint32_t)(i & P1) * (D / 2), k_pair = k_page + (uint32_t)P * D + (i & P1) * 4;
        constexpr int CH = D / 32, RP = 256 / D;
        const int c0 = (i & 7) / RP;
        const uint32_t k_dst = (uint32_t)i * 128;
        // values: a thread holds keys 8 o .. 8 o + 7 of its words (of 8 values each); the eight octets of a quarter-warp
        // store to different banks, and the words (and the order of the keys, v_swap) differ from octet to octet so that
        // the loads read different banks too
        const int ol = lane & 7, o = ol + 8 * ((warp - kExpandWarp) >> 1), ws = (lane >> 3) + 4 * (warp & 1);
        const int word0 = D == 128 ? 2 * ((ws + 2 * (ol >> 1)) & 7) : (ws + 4 * (ol >> 2)) & 7;
        const uint32_t v_page = (uint32_t)((8 * o) >> a.cache.page_shift) * a.cache.head_bytes;
        const int v_in = (8 * o) & P1;
        const uint32_t v_row = v_page + (uint32_t)(P + v_in) * (D / 2), v_pair = v_page + (uint32_t)P * D + (P + v_in) * 4;
        const int swap = v_swap<D>(o);
        uint32_t tile = 0, buf = 0, phase = 0;       // raw tiles done; next expanded buffer and its phase
        for (bool first = true; ok && next_item(a, plan, n_pairs, c, first, ahead); first = false) {
            for (int t = c.t0; t < c.t1; ++t, ++tile) {
                const int st = tile % kRawStages;
                ok = tile_wait(&sh.raw_full[st], (tile / kRawStages) & 1);
                if (ok && phase > 0) ok = tile_wait(&sh.kv_empty[buf], (phase - 1) & 1);
                if (!(ok = __all_sync(QMOE_FULL_MASK, ok))) break;
                const unsigned char* raw = sh.raw[st];
                const int j0 = (c.w.lo + t) * kKeys;
                const uint32_t valid = sh.valid[tile % kInfo];
                {
                    uint32_t sz = *(const uint32_t*)(raw + k_pair);
                    if (j0 + i >= c.w.kv_len || !((valid >> (i >> 4)) & 1)) sz = 0;
                    const __half2 s2 = __half2half2(__ushort_as_half((uint16_t)sz)), z2 = __half2half2(__ushort_as_half((uint16_t)(sz >> 16)));
                    unsigned char* dst = sh.kv[buf] + k_dst;
#pragma unroll 1
                    for (int s = 0; s < CH; ++s) {
                        const int ch = (c0 + s) & (CH - 1);
                        const uint4 w4 = *(const uint4*)(raw + k_row + ch * 16);
                        const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
                        // piece 4 ch + k of the row, at place (4 (ch & 1) + k) ^ (row % 8): the k only flips bits of the address
                        const uint32_t at = (ch >> 1) * Sh::kQAtom + (((4 * (ch & 1)) ^ (i & 7)) << 4);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            __half2 u[4];
                            code_integers(w[k], u);
                            *(uint4*)(dst + (at ^ (k << 4))) = make_uint4(h2(__hfma2(u[0], s2, z2)), h2(__hfma2(u[1], s2, z2)),
                                                                        h2(__hfma2(u[2], s2, z2)), h2(__hfma2(u[3], s2, z2)));
                        }
                    }
                }
                qmoe_tc::fence_async_shared();
                arrive_warp(&sh.kv_full[buf]);
                if (++buf == kExpanded) buf = 0, ++phase;
                ok = phase == 0 || tile_wait(&sh.kv_empty[buf], (phase - 1) & 1);
                if (!(ok = __all_sync(QMOE_FULL_MASK, ok))) break;
                {
                    __half2 s2[4], z2[4];
                    uint32_t pr[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) pr[k] = *(const uint32_t*)(raw + v_pair + (k ^ swap) * 4);
                    if (__builtin_expect(j0 + kKeys > c.w.kv_len || valid != 0xFFu, 0)) {
                        const bool page_ok = (valid >> (o >> 1)) & 1;
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            if (!page_ok || j0 + 8 * o + (k ^ swap) >= c.w.kv_len) pr[k] = 0;
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t ss = __byte_perm(pr[2 * k], pr[2 * k + 1], 0x5410), zz = __byte_perm(pr[2 * k], pr[2 * k + 1], 0x7632);
                        s2[k] = *(const __half2*)&ss, z2[k] = *(const __half2*)&zz;
                    }
                    unsigned char* dst0 = sh.kv[buf] + (o >> 3) * Sh::kVAtom;
#pragma unroll 1
                    for (int jj = 0; jj < D / 64; ++jj) {
                        const int word = word0 + (D == 128 ? jj ^ (lane >> 4) : 0);
                        uint32_t w[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) w[k] = *(const uint32_t*)(raw + v_row + (k ^ swap) * (D / 2) + word * 4);
#pragma unroll
                        for (int hh = 0; hh < 2; ++hh) {
                            uint32_t r[4][4];      // [value 2 v + hh][pair of keys]
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                __half2 u[4];
                                code_integers(__byte_perm(w[2 * k], w[2 * k + 1], hh ? 0x7632 : 0x5410), u);
#pragma unroll
                                for (int v = 0; v < 4; ++v) r[v][k] = h2(__hfma2(u[v], s2[k], z2[k]));
                            }
                            unsigned char* dst = dst0 + word * 1024 + hh * 128;
#pragma unroll
                            for (int v = 0; v < 4; ++v)
                                *(uint4*)(dst + v * 256 + (((ol ^ hh) ^ (2 * v)) << 4)) = make_uint4(r[v][0], r[v][1], r[v][2], r[v][3]);
                        }
                    }
                }
                qmoe_tc::fence_async_shared();
                arrive_warp(&sh.kv_full[buf]);
                if (++buf == kExpanded) buf = 0, ++phase;
                arrive_warp(&sh.raw_empty[st]);
            }
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
        if (warp == kIssueWarp || warp == kIssueWarp + 2) {
            // ---- issue the products of one tile of rows, by one elected thread
            const int x = (warp - kIssueWarp) >> 1;
            if (elect_one()) {
                constexpr uint32_t id_s = qmoe_tc::idesc_f16(128, kStep, false, false), id_o = qmoe_tc::idesc_f16(128, D, false, false);
                const uint64_t qd = desc_sw128(sh.q[x]), kvd = desc_sw128(sh.kv[0]);
                constexpr uint32_t kv_step = sizeof(sh.kv[0]) / 16;
                uint32_t n_q = 0, n_s = 0, n_p = 0;             // items, steps of scores and of values done
                uint32_t kb = 0, kph = 0, vb = 0, vph = 0;      // buffers and phases: keys, values
                for (bool first = true; ok && next_item_alone(a, plan, c, first); first = false) {
                    const int t0 = 2 * c.t0, t1 = 2 * c.t1, s = c.s[x], e = c.e[x];
                    // scores of step t + 1 go ahead of the values of step t, so that the softmax finds its next scores ready
#pragma unroll 1
                    for (int t = t0 - 1; t < t1 && ok; ++t) {
                        const uint32_t half = t & 1;            // of the values; the scores' is the other
                        if (half) {
                            if (t + 1 < t1) ok = tile_wait(&sh.kv_full[kb], kph);
                        } else {
                            vb = kb + 1, vph = kph;
                            if (vb == kExpanded) vb = 0, vph ^= 1;
                            ok = tile_wait(&sh.kv_full[vb], vph);
                        }
                        if (t + 1 >= s && t + 1 < e) {
                            if (t + 1 == s && ok) ok = tile_wait(&sh.q_full[x], n_q++ & 1);
                            if (!ok) break;
                            qmoe_tc::tc_fence_after();
                            const uint32_t k_lo = (uint32_t)kvd + kb * kv_step + (half ^ 1) * (kStep * 128 / 16), at = x * 128 + (n_s & 1) * kStep;
#pragma unroll
                            for (int k = 0; k < D / 16; ++k)
                                mma_ss(at, (uint32_t)qd, (uint32_t)(qd >> 32), k_lo, (uint32_t)(kvd >> 32), (k >> 2) * (Sh::kQAtom / 16) + (k & 3) * 2, id_s, k > 0);
                            qmoe_tc::mma_commit(&sh.s_full[x][n_s & 1]);
                            ++n_s;
                        }
                        if (t >= s && t < e) {
                            ok = ok && tile_wait(&sh.p_full[x][n_p & 1], (n_p >> 1) & 1);
                            if (!ok) break;
                            qmoe_tc::tc_fence_after();
                            const uint32_t v_lo = (uint32_t)kvd + vb * kv_step + half * (Sh::kVAtom / 16), at = x * 128 + (n_p & 1) * kStep;
#pragma unroll
                            for (int k = 0; k < kStep / 16; ++k)
                                mma_ts(256 + x * 128, at, k * 8, v_lo, (uint32_t)(kvd >> 32), k * 2, id_o, k > 0 || t > s);
                            qmoe_tc::mma_commit(&sh.o_full[x][n_p & 1]);
                            ++n_p;
                        }
                        // a tile's keys are done with after its second step's scores, its values after the second step's
                        if (t >= t0) {
                            qmoe_tc::mma_commit(&sh.kv_empty[half ? vb : kb]);
                            if (!half) {
                                kb = vb + 1, kph = vph;
                                if (kb == kExpanded) kb = 0, kph ^= 1;
                            }
                        }
                    }
                }
                // everything issued has ended before tensor memory is freed
                qmoe_tc::mma_commit(&sh.fin[x]);
                tile_wait(&sh.fin[x], 0);
            }
        } else if (warp == kCopyWarp) {
            // ---- copy pages: lane i the tile's i-th
            const int per_tile = kKeys >> a.cache.page_shift, per_page = (1 << a.cache.page_shift) / 16;
            uint32_t tile = 0;
            for (bool first = true; ok && next_item(a, plan, n_pairs, c, first, ahead); first = false) {
                if (lane == 0 && c.t0 == 0 && !c.whole)
                    plan.items[blockIdx.x] = SplitItem{c.w.b, c.kh, c.w.rb, (int)((c.w.unit + (long long)c.kh * (c.w.n + kTileItemCost) + c.w.n - 1) / chunk)};
                // the first block that a query of the request sees: those before may have no page
                const int blk_lo = first_seen(a, c.w.kv_len - (a.causal ? c.w.q_len : 1)) >> a.cache.page_shift;
                for (int t = c.t0; t < c.t1; ++t, ++tile) {
                    const int st = tile % kRawStages;
                    const int blk = (c.w.lo + t) * per_tile + lane;
                    const bool mine = lane < per_tile && blk >= blk_lo && (blk << a.cache.page_shift) < c.w.kv_len;
                    int page = -1;
                    if (mine && blk < a.max_blocks) page = a.table[(int64_t)c.w.b * a.max_blocks + blk];
                    const bool good = page >= 0 && page < a.cache.n_pages;
                    if (mine && !good) attn_set_error(QMOE_EINVAL);
                    const unsigned mask = __ballot_sync(QMOE_FULL_MASK, good);
                    if (tile >= kRawStages) ok = tile_wait(&sh.raw_empty[st], (tile / kRawStages - 1) & 1);
                    ok = __all_sync(QMOE_FULL_MASK, ok);
                    if (!ok) break;
                    if (lane == 0) {
                        uint32_t v = 0;
                        for (int i = 0; i < per_tile; ++i)
                            if ((mask >> i) & 1) v |= ((1u << per_page) - 1) << (i * per_page);
                        sh.valid[tile % kInfo] = v;
                        mbar_expect(&sh.raw_full[st], (uint32_t)__popc(mask) * a.cache.head_bytes);
                    }
                    __syncwarp();
                    if (good)
                        bulk_copy(sh.raw[st] + lane * a.cache.head_bytes, kv4::head_ptr(a.cache, page, c.kh), a.cache.head_bytes, &sh.raw_full[st]);
                }
            }
            // copies in flight land before the block's memory goes away
            for (uint32_t i = tile > kRawStages ? tile - kRawStages : 0; i < tile; ++i)
                qmoe_tc::mbar_wait(&sh.raw_full[i % kRawStages], (i / kRawStages) & 1, kWaitLimit);
        }
    }
    if (!ok) attn_set_error(QMOE_ETIMEOUT);
    qmoe_tc::tc_fence_before();
    __syncthreads();
    if (warp == kIssueWarp) {
        __syncwarp();
        qmoe_tc::tc_fence_after();
        qmoe_tc::tmem_dealloc(tmem, 512);
    }
}

// Query rows (a multiple of 8) that the few-row path takes per (request, kv head): the batch's largest where 32
// hold it, else enough for a single query (requests with more go to the tiles); 0 for groups above 32.
int decode_rows(int group, int max_q) {
    const long long all = (long long)group * max_q;
    const int rows = all <= 32 ? (int)all : group <= 32 ? group : 0;
    return (rows + 7) / 8 * 8;
}

// Blocks of the few-row path that are on the device together.
constexpr int kMaxFit = 3;
size_t decode_fit(int rows) { return (size_t)qmoe::sm_count() * (rows <= 16 ? kMaxFit : 2); }

size_t align256(size_t b) { return (b + 255) & ~(size_t)255; }

// Workspace of the few-row path: a record for each block (room for as many blocks as any row count has: what a longer
// draft needs then covers a shorter one), then the blocks' parts.
size_t decode_records() { return align256((size_t)qmoe::sm_count() * kMaxFit * sizeof(SplitItem)); }

size_t decode_ws(int rows, int head_dim) {
    return rows == 0 ? 0 : decode_records() + align256(decode_fit(rows) * 2 * rows * (head_dim + 2) * sizeof(float));
}

template <int D, int NT, bool kSel = false>
int launch_decode(const AttnArgs& a, void* ws, cudaStream_t st) {
    constexpr int rows = 8 * NT;
    const int smem = (int)sizeof(DecodeShared<D, NT>);
    int rc = qmoe::smem_attr((const void*)decode_kernel<D, NT, kSel>, smem, "attention attr");
    if (rc) return rc;
    const long long n_items = (long long)(kSel ? a.n_q_tokens : a.B) * a.cache.n_kv_heads;
    // tiles of the longest item (64 bits: the bounds may be the largest int32)
    long long tiles = ((long long)a.max_kv + kTile - 1) / kTile;
    if (kSel) tiles = (((long long)a.top << a.cache.page_shift) + kTile - 1) / kTile;
    if (a.window) tiles = std::min(tiles, ((long long)a.window + a.max_q + kTile - 1) / kTile + 1);
    // One block an item, or tiles spread over blocks and joined by a second kernel.  One request, 16/16 heads of 128, us in
    // a graph, one block / spread: 2 tiles 6.0 / 9.0, 4 7.8 / 9.0, 5 8.6 / 8.8, 6 9.4 / 9.1, 8 11.0 / 9.3; 16/1 heads of 64:
    // 4 8.7 / 9.2, 5 9.5 / 9.0.  More items cross later (8 requests of 32/8 heads: 6 9.6 / 10.6, 8 11.2 / 10.9; 32 of them:
    // 16 21.0 / 23.3), which is not counted on: the bound is the longest request's, and the others may be short.
    if (tiles <= 4 && n_items <= (long long)decode_fit(rows)) {
        if (kSel)
            return kv4::launch_dependent(decode_kernel<D, NT, kSel>, dim3((unsigned)n_items), kDecodeThreads, smem, st, "decode_kernel", a, rows, 1, nullptr, nullptr);
        decode_kernel<D, NT, kSel><<<(unsigned)n_items, kDecodeThreads, smem, st>>>(a, rows, 1, nullptr, nullptr);
        return qmoe::launch_check("decode_kernel");
    }
    const unsigned blocks = (unsigned)std::min((long long)decode_fit(rows), n_items * std::max(1LL, tiles));
    SplitItem* items = (SplitItem*)ws;
    float* parts = (float*)((char*)ws + decode_records());
    if (kSel) {
        rc = kv4::launch_dependent(decode_kernel<D, NT, kSel>, dim3(blocks), kDecodeThreads, smem, st, "decode_kernel", a, rows, 0, items, parts);
    } else {
        decode_kernel<D, NT, kSel><<<blocks, kDecodeThreads, smem, st>>>(a, rows, 0, items, parts);
        rc = qmoe::launch_check("decode_kernel");
    }
    if (rc) return rc;
    return kv4::launch_dependent(join_kernel<D, kSel>, dim3(blocks, kSel ? std::min(a.group, 16) : NT == 1 ? 8 : 16), kJoinThreads, 0, st, "join_kernel", a, items, parts, rows);
}

// Workspace of the tile path: the plan, then the blocks' parts.  max_pairs bounds the sum of ceil(rows / 256).
struct TileWs {
    TilePlan plan;
    float* parts;
    size_t bytes;
};

TileWs tile_ws(void* base, int B, int group, int head_dim, int n_q_tokens) {
    TileWs w{};
    size_t off = 0;
    auto take = [&](size_t bytes) {
        void* p = base ? (void*)((char*)base + off) : nullptr;
        off += align256(bytes);
        return p;
    };
    w.plan.max_pairs = (int)((long long)n_q_tokens * group / kRows + B);
    w.plan.pair_start = (int32_t*)take(sizeof(int32_t) * ((size_t)B + 1));
    w.plan.pair_b = (int32_t*)take(sizeof(int32_t) * (size_t)w.plan.max_pairs);
    w.plan.pairs = (PairInfo*)take(sizeof(PairInfo) * (size_t)w.plan.max_pairs);
    w.plan.total = (long long*)take(sizeof(long long));
    w.plan.items = (SplitItem*)take(sizeof(SplitItem) * (size_t)qmoe::sm_count());
    w.parts = (float*)take((size_t)qmoe::sm_count() * 2 * kRows * (head_dim + 2) * sizeof(float));
    w.bytes = off;
    return w;
}

template <int D>
int launch_tiles(const AttnArgs& a, const TileWs& w, int min_rows, cudaStream_t st) {
    const int smem = (int)sizeof(TileShared<D>), blocks = qmoe::sm_count();
    int rc = qmoe::smem_attr((const void*)tile_kernel<D>, smem, "attention attr");
    if (rc) return rc;
    if (min_rows == 0)      // the call's first kernel
        tile_plan_kernel<<<1, kPlanTile, 0, st>>>(a, w.plan, min_rows);
    else
        rc = kv4::launch_dependent(tile_plan_kernel, dim3(1), kPlanTile, 0, st, "tile_plan_kernel", a, w.plan, min_rows);
    if (rc || (rc = qmoe::launch_check("tile_plan_kernel"))) return rc;
    if ((rc = kv4::launch_dependent(tile_kernel<D>, dim3(blocks), kTileThreads, smem, st, "tile_kernel", a, w.plan, w.parts))) return rc;
    return kv4::launch_dependent(join_kernel<D, false>, dim3(blocks, 16), kJoinThreads, 0, st, "join_kernel", a, w.plan.items, w.parts, kRows);
}

// Whether some request of the batch has more rows than the few-row path takes.
bool has_tiles(int group, int max_q, int rows) { return (long long)group * max_q > rows; }

int check_sizes(const char* who, int B, int n_q_heads, int n_kv_heads, int head_dim, int n_q_tokens, int max_q, int max_kv) {
    if (head_dim != 64 && head_dim != 128) return qmoe::fail(QMOE_EUNSUPPORTED, std::string(who) + ": head_dim must be 64 or 128");
    if (B < 0 || n_q_tokens < 0 || max_q < 0 || max_kv < 0 || n_kv_heads < 1 || n_q_heads < n_kv_heads ||
        n_q_heads % n_kv_heads)
        return qmoe::fail(QMOE_EINVAL, std::string(who) + ": bad sizes (n_q_heads must be a multiple of n_kv_heads)");
    if ((long long)n_q_tokens * (n_q_heads / n_kv_heads) + (long long)kRows * B > 0x7FFFFFFFLL)
        return qmoe::fail(QMOE_EINVAL, std::string(who) + ": too many query rows in one call");
    if (n_q_heads / n_kv_heads > 128)
        return qmoe::fail(QMOE_EUNSUPPORTED, std::string(who) + ": more than 128 query heads per kv head");
    return QMOE_OK;
}

int check_chosen(const char* who, int n_q_tokens, int n_q_heads, int n_kv_heads, int head_dim, int top) {
    const int rc = check_sizes(who, 0, n_q_heads, n_kv_heads, head_dim, n_q_tokens, 0, 0);
    if (rc) return rc;
    if (n_q_heads / n_kv_heads > 32) return qmoe::fail(QMOE_EUNSUPPORTED, std::string(who) + ": more than 32 query heads per kv head");
    if (top < 1 || top > 65536) return qmoe::fail(QMOE_EINVAL, std::string(who) + ": need 1 <= top <= 65536");
    if ((long long)n_q_tokens * n_kv_heads > 0x7FFFFFFFLL) return qmoe::fail(QMOE_EINVAL, std::string(who) + ": too many query tokens in one call");
    return QMOE_OK;
}

}  // namespace

namespace qmoe {
int kv4_attention_take_error() {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_kv4_attention_error, sizeof(int)) != cudaSuccess) return QMOE_ECUDA;
    if (v == 0) return 0;      // nothing to clear
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
    const int group = n_q_heads / n_kv_heads, rows = decode_rows(group, max_q);
    *bytes = decode_ws(rows, head_dim) + (has_tiles(group, max_q, rows) ? tile_ws(nullptr, B, group, head_dim, n_q_tokens).bytes : 0);
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
    a.max_blocks = max_blocks, a.max_q = max_q, a.max_kv = max_kv, a.scale = scale, a.causal = causal ? 1 : 0;
    a.window = window >= max_kv ? 0 : window;      // as long as any request: it hides nothing
    cudaStream_t st = (cudaStream_t)stream;
    const int rows = decode_rows(a.group, max_q), D = cache->head_dim;
    const bool tiles = has_tiles(a.group, max_q, rows);
    const size_t few = decode_ws(rows, D);
    const TileWs tw = tiles ? tile_ws((char*)workspace + few, B, a.group, D, n_q_tokens) : TileWs{};
    if (ws_bytes < few + tw.bytes) return qmoe::fail(QMOE_ECAPACITY, "kv4_attention: workspace too small");
    if (!workspace || !kv4::aligned16(workspace)) return qmoe::fail(QMOE_EINVAL, "kv4_attention: workspace NULL or not 16-byte aligned");
    if ((long long)B * cache->n_kv_heads > 0x7FFFFFFFLL) return qmoe::fail(QMOE_EINVAL, "kv4_attention: batch too large");
    if (rows == 8) rc = D == 128 ? launch_decode<128, 1>(a, workspace, st) : launch_decode<64, 1>(a, workspace, st);
    if (rows == 16) rc = D == 128 ? launch_decode<128, 2>(a, workspace, st) : launch_decode<64, 2>(a, workspace, st);
    if (rows == 24) rc = D == 128 ? launch_decode<128, 3>(a, workspace, st) : launch_decode<64, 3>(a, workspace, st);
    if (rows == 32) rc = D == 128 ? launch_decode<128, 4>(a, workspace, st) : launch_decode<64, 4>(a, workspace, st);
    if (rc || !tiles) return rc;
    return D == 128 ? launch_tiles<128>(a, tw, rows, st) : launch_tiles<64>(a, tw, rows, st);
}

extern "C" int kv4_attention_blocks_ws_size(int n_q_tokens, int n_q_heads, int n_kv_heads, int head_dim, int page_size, int top,
                                            size_t* bytes) {
    qmoe::clear_error();
    if (!bytes) return qmoe::fail(QMOE_EINVAL, "kv4_attention_blocks_ws_size: NULL output");
    const int rc = check_chosen("kv4_attention_blocks_ws_size", n_q_tokens, n_q_heads, n_kv_heads, head_dim, top);
    if (rc) return rc;
    if (page_size != 16 && page_size != 32 && page_size != 64)
        return qmoe::fail(QMOE_EINVAL, "kv4_attention_blocks_ws_size: page_size must be 16, 32 or 64");
    *bytes = decode_ws(decode_rows(n_q_heads / n_kv_heads, 1), head_dim);
    return QMOE_OK;
}

extern "C" int kv4_attention_blocks(const kv4_cache* cache, const void* q, int n_q_tokens, int n_q_heads, const int32_t* q_start,
                                    const int32_t* kv_len, int B, const int32_t* table, int max_blocks, const int32_t* sel, int top,
                                    float scale, void* out, void* workspace, size_t ws_bytes, void* stream) {
    qmoe::clear_error();
    AttnArgs a{};
    int rc = kv4::view_of(cache, "kv4_attention_blocks", &a.cache);
    if (rc) return rc;
    if ((rc = check_chosen("kv4_attention_blocks", n_q_tokens, n_q_heads, cache->n_kv_heads, cache->head_dim, top))) return rc;
    if (B < 0 || max_blocks < 0) return qmoe::fail(QMOE_EINVAL, "kv4_attention_blocks: negative B or max_blocks");
    if (B == 0 || n_q_tokens == 0) return QMOE_OK;
    if (!q || !out || !q_start || !kv_len || !sel || (max_blocks > 0 && !table))
        return qmoe::fail(QMOE_EINVAL, "kv4_attention_blocks: NULL pointer");
    if (!kv4::aligned16(q) || !kv4::aligned16(out)) return qmoe::fail(QMOE_EINVAL, "kv4_attention_blocks: pointer not 16-byte aligned");
    a.q = (const uint16_t*)q, a.out = (uint16_t*)out, a.q_start = q_start, a.kv_len = kv_len, a.table = table, a.sel = sel;
    a.B = B, a.n_q_tokens = n_q_tokens, a.n_q_heads = n_q_heads, a.group = n_q_heads / cache->n_kv_heads;
    a.max_blocks = max_blocks, a.max_q = 1, a.scale = scale, a.causal = 1, a.top = top;
    const int rows = decode_rows(a.group, 1), D = cache->head_dim;
    if (ws_bytes < decode_ws(rows, D)) return qmoe::fail(QMOE_ECAPACITY, "kv4_attention_blocks: workspace too small");
    if (!workspace || !kv4::aligned16(workspace)) return qmoe::fail(QMOE_EINVAL, "kv4_attention_blocks: workspace NULL or not 16-byte aligned");
    cudaStream_t st = (cudaStream_t)stream;
    if (rows == 8) return D == 128 ? launch_decode<128, 1, true>(a, workspace, st) : launch_decode<64, 1, true>(a, workspace, st);
    if (rows == 16) return D == 128 ? launch_decode<128, 2, true>(a, workspace, st) : launch_decode<64, 2, true>(a, workspace, st);
    if (rows == 24) return D == 128 ? launch_decode<128, 3, true>(a, workspace, st) : launch_decode<64, 3, true>(a, workspace, st);
    return D == 128 ? launch_decode<128, 4, true>(a, workspace, st) : launch_decode<64, 4, true>(a, workspace, st);
}
