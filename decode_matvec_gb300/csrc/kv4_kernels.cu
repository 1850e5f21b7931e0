// What feeds attention over the 4-bit paged key/value cache: block tables and
// slot maps, the norms and the rotation of queries and keys, and the cache's
// writer and reader.  For a few tokens all are bound by a launch and one
// dependent chain of loads (2 to 4 us in a graph); for many the norm and the
// writer by instruction issue, the reader by memory.  Measured (one GB300):
// norm and rotation of 16383 tokens, 32 + 8 heads of 128, 73 us (4.7 TB/s of
// 6.8; 206 instructions for two heads, issue slots 79 % used), with the cache
// write 110; writing 16384 tokens of 16 heads of 128 59 us, reading them back 30;
// tables, slots and positions of 257 requests with 260 thousand new tokens 10 us.

#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "kv4_common.cuh"

namespace {

__device__ int g_kv4_error;

__device__ __forceinline__ void kv4_set_error(int code) { atomicCAS(&g_kv4_error, 0, code); }

// ---------------------------------------------------------------- block tables
constexpr int kPlanThreads = 1024;

struct TableArgs {
    const int32_t* cached;
    const int32_t* fresh;
    const int32_t* free_pages;
    const int32_t* n_free;
    int32_t* table;
    int32_t* q_start;
    int32_t* kv_len;
    int32_t* slots;
    int32_t* positions;
    int32_t* n_free_out;
    int B, page_shift, max_blocks, n_tokens;
    int max_free;     // places of the stack
    int vector4;      // slots and positions are 16-byte aligned
};

// Slot and position of new token t of request b (t in [q_start[b], q_start[b + 1])).
__device__ __forceinline__ void map_token(const TableArgs& a, int t, int b, int start, int* slot, int* pos) {
    *pos = max(a.cached[b], 0) + t - start;
    *slot = -1;
    const int blk = *pos >> a.page_shift;
    if (blk < a.max_blocks) {
        const int page = a.table[(int64_t)b * a.max_blocks + blk];
        if (page >= 0)
            *slot = (page << a.page_shift) + (*pos & ((1 << a.page_shift) - 1));
        else if (page != -1)
            kv4_set_error(QMOE_EINVAL);
    }
}

// Last i of [0, n) with start[i] <= t (start[0] <= t).
template <typename T>
__device__ __forceinline__ int last_start(const T* start, int n, T t) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= t)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// One block: prefix sums of the new tokens and new pages over the requests (1024 at a time), the new table entries (a
// thread a page, so that the loads from the stack do not wait for one another), and with kTokens the tokens' slots too
// (few tokens: one launch costs less than two).
template <bool kTokens>
__global__ void __launch_bounds__(kPlanThreads) block_tables_kernel(TableArgs a) {
    __shared__ long long warp_tok[32], warp_page[32];
    __shared__ long long page_at[kPlanThreads];
    __shared__ int have_s[kPlanThreads];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int P1 = (1 << a.page_shift) - 1;
    const int said = *a.n_free, n_free = min(max(said, 0), a.max_free);
    long long tok0 = 0, page0 = 0;
    bool bad = said > a.max_free;
    for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
        const int b = b0 + tid;
        int c = 0, n = 0;
        if (b < a.B) {
            c = a.cached[b];
            n = a.fresh[b];
            bad |= c < 0 || n < 0 || (long long)c + n > 0x7FFFFFFF - 64;
            c = max(c, 0);
            n = min(max(n, 0), 0x7FFFFFFF - 64 - c);
        }
        const int have = (int)(((unsigned)c + P1) >> a.page_shift);
        const int need = (int)(((unsigned)(c + n) + P1) >> a.page_shift) - have;
        long long ts = n, ps = need;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long to = __shfl_up_sync(QMOE_FULL_MASK, ts, d), po = __shfl_up_sync(QMOE_FULL_MASK, ps, d);
            if (lane >= d) {
                ts += to;
                ps += po;
            }
        }
        if (lane == 31) {
            warp_tok[warp] = ts;
            warp_page[warp] = ps;
        }
        __syncthreads();
        if (warp == 0) {
            long long tw = warp_tok[lane], pw = warp_page[lane];
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const long long to = __shfl_up_sync(QMOE_FULL_MASK, tw, d), po = __shfl_up_sync(QMOE_FULL_MASK, pw, d);
                if (lane >= d) {
                    tw += to;
                    pw += po;
                }
            }
            warp_tok[lane] = tw;
            warp_page[lane] = pw;
        }
        __syncthreads();
        const long long t_end = tok0 + ts + (warp ? warp_tok[warp - 1] : 0);
        page_at[tid] = ps - need + (warp ? warp_page[warp - 1] : 0);
        have_s[tid] = have;
        if (b < a.B) {
            a.q_start[b] = (int)min(t_end - n, (long long)a.n_tokens);
            a.kv_len[b] = c + n;
            if (have + need > a.max_blocks) bad = true;
        }
        __syncthreads();
        const long long pages = warp_page[31];
        for (long long i = tid; i < pages; i += kPlanThreads) {
            // requests without new pages begin where the next one does: the last of equals is the one that has the page
            const int r = last_start(page_at, min(kPlanThreads, a.B - b0), i);
            const long long entry = have_s[r] + i - page_at[r], at = n_free - 1 - page0 - i;
            if (entry < a.max_blocks) a.table[(int64_t)(b0 + r) * a.max_blocks + entry] = at >= 0 ? a.free_pages[at] : -1;
        }
        tok0 += warp_tok[31];
        page0 += pages;
        __syncthreads();
    }
    if (__syncthreads_or(bad) && tid == 0) kv4_set_error(QMOE_EINVAL);
    const int total = (int)min(tok0, (long long)a.n_tokens);
    if (tid == 0) {
        a.q_start[a.B] = total;
        *a.n_free_out = (int)max(n_free - page0, 0LL);
        if (page0 > n_free || tok0 > a.n_tokens) kv4_set_error(QMOE_ECAPACITY);
    }
    if (kTokens) {
        __syncthreads();   // the table and q_start, which this block wrote, are read below
        for (int t = tid; t < a.n_tokens; t += kPlanThreads) {
            int slot = -1, pos = 0;
            if (t < total) {
                const int b = last_start((const int32_t*)a.q_start, a.B, t);
                map_token(a, t, b, a.q_start[b], &slot, &pos);
            }
            a.slots[t] = slot;
            a.positions[t] = pos;
        }
    }
}

// Many tokens: a block maps 1024, four neighbours a thread.  Where they fit, the requests' starts are searched in
// shared memory (a search in global memory is a chain of about ten cache accesses).
constexpr int kMapTokens = 1024, kMapStarts = 4096;

__global__ void __launch_bounds__(kMapTokens / 4) slot_map_kernel(TableArgs a) {
    __shared__ int start_s[kMapStarts];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int total = a.q_start[a.B], t0 = blockIdx.x * kMapTokens + threadIdx.x * 4;
    const bool in_smem = a.B <= kMapStarts;
    if (in_smem) {
        for (int i = threadIdx.x; i < a.B; i += kMapTokens / 4) start_s[i] = a.q_start[i];
        __syncthreads();
    }
    if (t0 >= a.n_tokens) return;
    const int32_t* start = in_smem ? start_s : a.q_start;
    int slot[4], pos[4];
    int b = t0 < total ? last_start(start, a.B, t0) : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = t0 + i;
        slot[i] = -1, pos[i] = 0;
        if (t < total) {
            while (b + 1 < a.B && start[b + 1] <= t) ++b;
            map_token(a, t, b, start[b], &slot[i], &pos[i]);
        }
    }
    if (t0 + 3 < a.n_tokens && a.vector4) {
        *(int4*)(a.slots + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
        *(int4*)(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (t0 + i < a.n_tokens) a.slots[t0 + i] = slot[i], a.positions[t0 + i] = pos[i];
    }
}

// ---------------------------------------------------------------- norm, rotation, cache write
struct RopeArgs {
    const uint16_t *q, *k, *v;            // heads of one token contiguous
    int64_t q_stride, k_stride, v_stride;  // elements from token to token
    int T, n_q, n_kv, heads;               // heads: how many of a token's (q, k, v) heads are visited
    int q_blocks, kv_blocks;               // a warp's blocks of heads of one kind
    const uint16_t *wq, *wk;               // norm weights or NULL
    float eps;
    const float* cos_sin;                  // NULL: no rotation
    int rot, interleaved, n_pos;
    const int32_t* positions;
    uint16_t *q_out, *k_out;               // either may be NULL
    const int32_t* slots;                  // NULL: no cache
    kv4::CacheView cache;
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *(uint32_t*)&p;
}

template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int d = L / 2; d > 0; d >>= 1) v += __shfl_xor_sync(QMOE_FULL_MASK, v, d);
    return v;
}

__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
    const __nv_bfloat162 r = __hmin2(*(__nv_bfloat162*)&a, *(__nv_bfloat162*)&b);
    return *(const uint32_t*)&r;
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    const __nv_bfloat162 r = __hmax2(*(__nv_bfloat162*)&a, *(__nv_bfloat162*)&b);
    return *(const uint32_t*)&r;
}

// The code word of 8 values y by (s, z): u = clamp(rint((y - z) / s), 0, 15), the quotient rounded as the format defines it.
__device__ __forceinline__ uint32_t code_word(const float (&y)[8], float s, float z) {
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float u = fminf(fmaxf(rintf(__fdiv_rn(y[i] - z, s)), 0.f), 15.f);
        word |= (uint32_t)u << (4 * (i >> 1) + 16 * (i & 1));
    }
    return word;
}

// Quantises the row held as 8 bf16 values a lane by the L lanes of a group and stores its codes (one word a lane) and its
// (s, z) pair.  All lanes of the warp take part.
//
// Dividing 8 values a lane exactly would cost several times what the row's bytes do, so the quotient is taken as
// 15 saturate((y - z) (1 / (15 s))), within 1e-5 of it: its rounding is the same unless it lies that near a half, and a row
// with such a value, or with a NaN or a magnitude of 32768 or more, is done again with divisions.
template <int L>
__device__ __forceinline__ void store_row(const RopeArgs& a, uint4 o, int slot, int head, int side, int gl) {
    const uint32_t w4[4] = {o.x, o.y, o.z, o.w};
    uint32_t lo2 = min2(min2(o.x, o.y), min2(o.z, o.w)), hi2 = max2(max2(o.x, o.y), max2(o.z, o.w)), big = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) big |= (w4[i] & 0x7FFF7FFFu) + 0x39003900u;      // a half's top bit: magnitude >= 0x4700, 32768
#pragma unroll
    for (int d = L / 2; d > 0; d >>= 1) {
        lo2 = min2(lo2, __shfl_xor_sync(QMOE_FULL_MASK, lo2, d));
        hi2 = max2(hi2, __shfl_xor_sync(QMOE_FULL_MASK, hi2, d));
    }
    float y[8], lo = fminf(bf16_lo(lo2), bf16_hi(lo2)), hi = fmaxf(bf16_lo(hi2), bf16_hi(hi2));
#pragma unroll
    for (int i = 0; i < 4; ++i) y[2 * i] = bf16_lo(w4[i]), y[2 * i + 1] = bf16_hi(w4[i]);
    const bool odd = __any_sync(QMOE_FULL_MASK, (big & 0x80008000u) != 0);
    if (__builtin_expect(odd, 0)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            y[i] = fminf(fmaxf(y[i] == y[i] ? y[i] : 0.f, -32768.f), 32768.f);
            lo = i ? fminf(lo, y[i]) : y[i];
            hi = i ? fmaxf(hi, y[i]) : y[i];
        }
#pragma unroll
        for (int d = L / 2; d > 0; d >>= 1) {
            lo = fminf(lo, __shfl_xor_sync(QMOE_FULL_MASK, lo, d));
            hi = fmaxf(hi, __shfl_xor_sync(QMOE_FULL_MASK, hi, d));
        }
    }
    const __half zh = __float2half_rn(lo);
    const float z = __half2float(zh);
    // fp16 of (hi - z) / 15: the product with 1 / 15 is within 2 units of the quotient's last place, which decides unless
    // that is next to the middle of two fp16 values (or fp16 has no 11 bits there)
    float d15 = (hi - z) * (1.f / 15.f);
    if (__builtin_expect(((__float_as_uint(d15) + 2u) & 0x1FFFu) - 0x1000u <= 4u || d15 < 6.2e-5f, 0)) d15 = __fdiv_rn(hi - z, 15.f);
    const __half sh = __float2half_rn(d15);
    const float s = __half2float(sh);
    uint32_t word = 0;
    if (s > 0.f) {
        constexpr float kMagic = 12582912.f;       // 1.5 * 2^23: adding it leaves the nearest integer in the low bits
        constexpr uint32_t kBits = 0x4B400000u;
        const float r = __fdividef(1.f / 15.f, s);
        float worst = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float q = __saturatef((y[i] - z) * r), v = fmaf(q, 15.f, kMagic);
            worst = fmaxf(worst, fabsf(fmaf(q, 15.f, kMagic - v)));
            word += (__float_as_uint(v) - kBits) << (4 * (i >> 1) + 16 * (i & 1));
        }
        if (__builtin_expect(worst > 0.49999f || odd, 0)) word = code_word(y, s, z);
    }
    if (slot < 0) return;
    const int P = 1 << a.cache.page_shift;
    unsigned char* hp = kv4::head_ptr(a.cache, slot >> a.cache.page_shift, head);
    const int row = side * P + (slot & (P - 1));
    ((uint32_t*)hp)[row * L + gl] = word;
    if (gl == 0)
        ((uint32_t*)(hp + (size_t)2 * P * L * 4))[row] =
            (uint32_t)__half_as_ushort(sh) | ((uint32_t)__half_as_ushort(zh) << 16);
}

// A group of L = head_dim / 8 lanes holds one head, 8 values a lane (16-byte loads and stores); a warp takes up to
// `rounds` heads a group of one token and one kind (queries, keys or values), one after another (a loop, not unrolled:
// its code has to stay in the instruction caches), with the next head's load ahead of the present one's work.
//
// Norm and rotation are one linear map of the head, r (x_i w_i c_i + x_j w_j s_i) with j the value that i is paired with
// and r = 1 / sqrt(mean(x^2) + eps): w c and w s are made once a token, and the pair's values come from the partner's
// lane (or the same word, when pairs are neighbours) as they were loaded.
// kTurn: norm and rotation; kCache: keys and values go to the cache.
template <int L, bool kTurn, bool kCache>
__global__ void __launch_bounds__(256) rope_kernel(RopeArgs a, unsigned per_token, int rounds) {
    constexpr int G = 32 / L, D = L * 8;
    const int lane = threadIdx.x & 31, gl = lane & (L - 1), g = lane / L;
    const unsigned long long w = (unsigned long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (w >= (unsigned long long)a.T * per_token) return;
    const int t = w >> 32 ? (int)(w / per_token) : (int)((unsigned)w / per_token);
    int block = (int)(w - (unsigned long long)t * per_token), kind = 0;      // queries, keys, values in turn
    if (block >= a.q_blocks) {
        kind = block - a.q_blocks >= a.kv_blocks ? 2 : 1;
        block -= a.q_blocks + (kind == 2 ? a.kv_blocks : 0);
    }
    const int n = kind == 0 ? a.n_q : a.n_kv;
    int h = block * (rounds * G) + g;
    const uint16_t* src = (kind == 0 ? a.q + t * a.q_stride : kind == 1 ? a.k + t * a.k_stride : a.v + t * a.v_stride) + h * D + gl * 8;
    uint4 next = h < n ? *(const uint4*)src : make_uint4(0, 0, 0, 0);
    uint16_t* dst = !kTurn || kind == 2 ? nullptr : kind == 0 ? a.q_out : a.k_out;
    if (dst) dst += ((int64_t)t * n + h) * D + gl * 8;
    int slot = -1;
    if (kCache && kind > 0) {
        slot = a.slots[t];
        if (slot < -1 || (slot >> a.cache.page_shift) >= a.cache.n_pages) {
            kv4_set_error(QMOE_EINVAL);
            slot = -1;
        }
    }
    const uint16_t* wt = kind == 0 ? a.wq : kind == 1 ? a.wk : nullptr;
    const int hl = a.rot >> 4;                                   // lanes of half a rotation
    const bool turns = kTurn && gl * 8 < a.rot && kind < 2;
    const int partner = !turns || a.interleaved ? gl : gl < hl ? gl + hl : gl - hl;
    float wc[8], ws[8];
    if (kTurn) {
#pragma unroll
        for (int i = 0; i < 8; ++i) wc[i] = 1.f, ws[i] = 0.f;
        if (turns) {
            int pos = a.positions[t];
            if (pos < 0 || pos >= a.n_pos) {
                kv4_set_error(QMOE_EINVAL);
                pos = pos < 0 ? 0 : a.n_pos - 1;
            }
            const float* row = a.cos_sin + (int64_t)pos * a.rot;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int at = a.interleaved ? gl * 4 + i / 2 : (gl < hl ? gl : gl - hl) * 8 + i;
                const float s = row[(a.rot >> 1) + at];
                wc[i] = row[at];
                ws[i] = (a.interleaved ? (i & 1) == 0 : gl < hl) ? -s : s;
            }
        }
        if (wt) {
            const uint4 w4 = *(const uint4*)(wt + gl * 8), p4 = *(const uint4*)(wt + partner * 8);
            const uint32_t wo[4] = {w4.x, w4.y, w4.z, w4.w}, wp[4] = {p4.x, p4.y, p4.z, p4.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                wc[2 * i] *= bf16_lo(wo[i]), wc[2 * i + 1] *= bf16_hi(wo[i]);
                ws[2 * i] *= a.interleaved ? bf16_hi(wp[i]) : bf16_lo(wp[i]), ws[2 * i + 1] *= a.interleaved ? bf16_lo(wp[i]) : bf16_hi(wp[i]);
            }
        }
    }
#pragma unroll 1
    for (int k = 0; k < rounds; ++k) {
        uint4 o = next;
        const int at = h;
        h += G, src += G * D;
        if (k + 1 < rounds && h < n) next = *(const uint4*)src;
        if (kTurn && kind < 2) {
            uint32_t xw[4] = {o.x, o.y, o.z, o.w}, yw[4];
            float r = 1.f;
            if (wt) {
                float ss = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) ss = fmaf(bf16_lo(xw[i]), bf16_lo(xw[i]), fmaf(bf16_hi(xw[i]), bf16_hi(xw[i]), ss));
                ss = group_sum<L>(ss);
                r = rsqrtf(ss * (1.f / D) + a.eps);      // 2 ulp of fp32, before a rounding to 8 bits
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                yw[i] = a.interleaved ? __byte_perm(xw[i], 0, 0x1032) : __shfl_sync(QMOE_FULL_MASK, xw[i], partner, L);
                if (!turns) yw[i] = 0;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                xw[i] = pack_bf16(fmaf(bf16_lo(yw[i]), ws[2 * i], bf16_lo(xw[i]) * wc[2 * i]) * r,
                                  fmaf(bf16_hi(yw[i]), ws[2 * i + 1], bf16_hi(xw[i]) * wc[2 * i + 1]) * r);
            o = make_uint4(xw[0], xw[1], xw[2], xw[3]);
            if (dst) {
                if (at < n) *(uint4*)dst = o;
                dst += G * D;
            }
        }
        // what the cache holds are the values as k_out holds them (rounded to bf16)
        if (kCache && kind > 0) store_row<L>(a, o, at < n ? slot : -1, at, kind == 2, gl);
    }
}

// ---------------------------------------------------------------- cache reader
// As the writer: a group a row (token, side, head), HB rows a group, a word a lane.
template <int L, int HB>
__global__ void __launch_bounds__(256) gather_kernel(kv4::CacheView c, const int32_t* slots, int n, unsigned per_token, uint16_t* k_out,
                                                     uint16_t* v_out) {
    constexpr int G = 32 / L;
    const int lane = threadIdx.x & 31, gl = lane & (L - 1), g = lane / L;
    const unsigned long long w = (unsigned long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (w >= (unsigned long long)n * per_token) return;
    const int t = w >> 32 ? (int)(w / per_token) : (int)((unsigned)w / per_token);
    const int r0 = (int)(w - (unsigned long long)t * per_token) * (HB * G) + g;
    int slot = slots[t];
    if (slot < -1 || (slot >> c.page_shift) >= c.n_pages) {
        kv4_set_error(QMOE_EINVAL);
        slot = -1;
    }
    const int P = 1 << c.page_shift;
    uint32_t word[HB], sz[HB];
#pragma unroll
    for (int k = 0; k < HB; ++k) {
        const int r = r0 + k * G;
        word[k] = sz[k] = 0;
        if (r < 2 * c.n_kv_heads && slot >= 0) {
            const int side = r >= c.n_kv_heads, h = side ? r - c.n_kv_heads : r;
            const unsigned char* hp = kv4::head_ptr(c, slot >> c.page_shift, h);
            const int row = side * P + (slot & (P - 1));
            word[k] = ((const uint32_t*)hp)[row * L + gl];
            sz[k] = ((const uint32_t*)(hp + (size_t)2 * P * L * 4))[row];
        }
    }
#pragma unroll
    for (int k = 0; k < HB; ++k) {
        const int r = r0 + k * G;
        if (r >= 2 * c.n_kv_heads) break;
        const int side = r >= c.n_kv_heads, h = side ? r - c.n_kv_heads : r;
        const float s = f16_to_f32((uint16_t)sz[k]), z = f16_to_f32((uint16_t)(sz[k] >> 16));
        float x[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) x[q] = fmaf(s, (float)((word[k] >> (4 * (q >> 1) + 16 * (q & 1))) & 15u), z);
        *(uint4*)((side ? v_out : k_out) + ((int64_t)t * c.n_kv_heads + h) * (L * 8) + gl * 8) =
            make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
    }
}

// Heads a group of lanes takes: four where that still gives every scheduler of the device some eight warps, else one.
template <int L>
bool four_heads(long long T, int heads) {
    return T * ((heads + 4 * (32 / L) - 1) / (4 * (32 / L))) >= (long long)qmoe::sm_count() * 32;
}

// turn: norm and rotation (false: the rows as they are, for the cache alone).
template <int L>
int launch_rope(RopeArgs a, bool turn, const char* who, cudaStream_t st) {
    if (a.T == 0 || a.heads == 0) return QMOE_OK;
    const int rounds = four_heads<L>(a.T, a.heads) ? 4 : 1, span = rounds * (32 / L);
    a.q_blocks = (a.n_q + span - 1) / span, a.kv_blocks = (a.n_kv + span - 1) / span;
    const unsigned per_token = (unsigned)(a.q_blocks + (a.heads - a.n_q) / std::max(a.n_kv, 1) * a.kv_blocks);
    if (per_token == 0) return QMOE_OK;
    const long long blocks = ((long long)a.T * per_token + 7) / 8;
    if (blocks > 0x7FFFFFFFLL) return qmoe::fail(QMOE_EINVAL, std::string(who) + ": too many heads in one call");
    if (!turn)
        rope_kernel<L, false, true><<<(unsigned)blocks, 256, 0, st>>>(a, per_token, rounds);
    else if (a.slots)
        rope_kernel<L, true, true><<<(unsigned)blocks, 256, 0, st>>>(a, per_token, rounds);
    else
        rope_kernel<L, true, false><<<(unsigned)blocks, 256, 0, st>>>(a, per_token, rounds);
    return qmoe::launch_check(who);
}

template <int L, int HB>
int launch_gather(const kv4::CacheView& c, const int32_t* slots, int n, void* k_out, void* v_out, cudaStream_t st) {
    const unsigned per_token = (unsigned)((2 * c.n_kv_heads + HB * (32 / L) - 1) / (HB * (32 / L)));
    const long long blocks = ((long long)n * per_token + 7) / 8;
    if (blocks > 0x7FFFFFFFLL) return qmoe::fail(QMOE_EINVAL, "kv4_gather: too many rows in one call");
    gather_kernel<L, HB><<<(unsigned)blocks, 256, 0, st>>>(c, slots, n, per_token, (uint16_t*)k_out, (uint16_t*)v_out);
    return qmoe::launch_check("kv4_gather");
}

}  // namespace

namespace qmoe {
int kv4_take_error() {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_kv4_error, sizeof(int)) != cudaSuccess) return QMOE_ECUDA;
    if (v == 0) return 0;      // nothing to clear
    const int z = 0;
    if (cudaMemcpyToSymbol(g_kv4_error, &z, sizeof(int)) != cudaSuccess) return QMOE_ECUDA;
    return v;
}
}  // namespace qmoe

extern "C" int kv4_block_tables_bounded(const int32_t* cached, const int32_t* new_tokens, int B, const int32_t* free_pages,
                                        int max_free, const int32_t* n_free, int page_size, int32_t* table, int max_blocks,
                                        int32_t* q_start, int32_t* kv_len, int32_t* slots, int32_t* positions, int n_tokens,
                                        int32_t* n_free_out, void* stream) {
    qmoe::clear_error();
    if (page_size != 16 && page_size != 32 && page_size != 64)
        return qmoe::fail(QMOE_EINVAL, "kv4_block_tables: page_size must be 16, 32 or 64");
    if (B < 0 || n_tokens < 0 || max_blocks < 0 || max_free < 0) return qmoe::fail(QMOE_EINVAL, "kv4_block_tables: negative size");
    if (!n_free || !n_free_out || !q_start || (B > 0 && (!cached || !new_tokens || !table || !kv_len || !free_pages)) ||
        (n_tokens > 0 && (!slots || !positions)))
        return qmoe::fail(QMOE_EINVAL, "kv4_block_tables: NULL pointer");
    TableArgs a{cached, new_tokens, free_pages, n_free, table, q_start, kv_len, slots, positions, n_free_out,
                B, page_size == 16 ? 4 : page_size == 32 ? 5 : 6, max_blocks, n_tokens, max_free,
                kv4::aligned16(slots) && kv4::aligned16(positions)};
    cudaStream_t st = (cudaStream_t)stream;
    // up to four tokens a thread: one launch
    if (n_tokens <= 4 * kPlanThreads) {
        block_tables_kernel<true><<<1, kPlanThreads, 0, st>>>(a);
        return qmoe::launch_check("kv4_block_tables");
    }
    block_tables_kernel<false><<<1, kPlanThreads, 0, st>>>(a);
    const int rc = qmoe::launch_check("kv4_block_tables");
    if (rc) return rc;
    return kv4::launch_dependent(slot_map_kernel, dim3((unsigned)((n_tokens + kMapTokens - 1) / kMapTokens)), kMapTokens / 4, 0, st,
                                 "kv4_block_tables", a);
}

extern "C" int kv4_block_tables(const int32_t* cached, const int32_t* new_tokens, int B, const int32_t* free_pages,
                                const int32_t* n_free, int page_size, int32_t* table, int max_blocks,
                                int32_t* q_start, int32_t* kv_len, int32_t* slots, int32_t* positions, int n_tokens,
                                int32_t* n_free_out, void* stream) {
    return kv4_block_tables_bounded(cached, new_tokens, B, free_pages, 0x7FFFFFFF, n_free, page_size, table, max_blocks, q_start,
                                    kv_len, slots, positions, n_tokens, n_free_out, stream);
}

extern "C" int qk_norm_rope(const void* qkv, int64_t row_stride, int T, int n_q_heads, int n_kv_heads, int head_dim,
                            const void* q_weight, const void* k_weight, float eps, const float* cos_sin, int rot_dim,
                            int interleaved, int n_pos, const int32_t* positions, void* q_out, void* k_out,
                            const kv4_cache* cache, const int32_t* slots, void* stream) {
    qmoe::clear_error();
    if (head_dim != 64 && head_dim != 128) return qmoe::fail(QMOE_EUNSUPPORTED, "qk_norm_rope: head_dim must be 64 or 128");
    if (T < 0 || n_q_heads < 0 || n_kv_heads < 0 || n_q_heads > 65536 || n_kv_heads > 65536)
        return qmoe::fail(QMOE_EINVAL, "qk_norm_rope: bad sizes");
    if (!cos_sin != (rot_dim == 0) || rot_dim < 0 || rot_dim > head_dim || rot_dim % 16)
        return qmoe::fail(QMOE_EINVAL, "qk_norm_rope: rot_dim must be a multiple of 16 up to head_dim, 0 without cos_sin");
    if (cos_sin && (n_pos < 1 || (T > 0 && !positions)))
        return qmoe::fail(QMOE_EINVAL, "qk_norm_rope: a rotation needs positions and n_pos >= 1");
    if ((T > 0 && !qkv) || (T > 0 && n_q_heads > 0 && !q_out)) return qmoe::fail(QMOE_EINVAL, "qk_norm_rope: NULL pointer");
    if (!cache != !slots && T > 0) return qmoe::fail(QMOE_EINVAL, "qk_norm_rope: cache and slots go together");
    const int64_t width = (int64_t)(n_q_heads + (cache ? 2 : 1) * n_kv_heads) * head_dim;
    if (row_stride % 8 || (T > 1 && row_stride < width))
        return qmoe::fail(QMOE_EINVAL, "qk_norm_rope: row_stride must be a multiple of 8 and cover a token's heads");
    if (!kv4::aligned16(qkv) || !kv4::aligned16(q_weight) || !kv4::aligned16(k_weight) || !kv4::aligned16(cos_sin) ||
        !kv4::aligned16(q_out) || !kv4::aligned16(k_out))
        return qmoe::fail(QMOE_EINVAL, "qk_norm_rope: pointer not 16-byte aligned");
    RopeArgs a{};
    if (cache) {
        const int rc = kv4::view_of(cache, "qk_norm_rope", &a.cache);
        if (rc) return rc;
        if (cache->head_dim != head_dim || cache->n_kv_heads != n_kv_heads)
            return qmoe::fail(QMOE_EINVAL, "qk_norm_rope: the cache has another head layout");
    }
    const uint16_t* base = (const uint16_t*)qkv;
    a.q = base;
    a.k = base + (int64_t)n_q_heads * head_dim;
    a.v = a.k + (int64_t)n_kv_heads * head_dim;
    a.q_stride = a.k_stride = a.v_stride = row_stride;
    a.T = T, a.n_q = n_q_heads, a.n_kv = n_kv_heads, a.heads = n_q_heads + (cache ? 2 : 1) * n_kv_heads;
    a.wq = (const uint16_t*)q_weight, a.wk = (const uint16_t*)k_weight, a.eps = eps;
    a.cos_sin = cos_sin, a.rot = rot_dim, a.interleaved = interleaved ? 1 : 0, a.n_pos = n_pos, a.positions = positions;
    a.q_out = (uint16_t*)q_out, a.k_out = (uint16_t*)k_out, a.slots = cache ? slots : nullptr;
    if (!cache && !k_out) a.heads = n_q_heads;
    return head_dim == 128 ? launch_rope<16>(a, true, "qk_norm_rope", (cudaStream_t)stream) : launch_rope<8>(a, true, "qk_norm_rope", (cudaStream_t)stream);
}

extern "C" int kv4_append(const kv4_cache* cache, const void* k, int64_t k_stride, const void* v, int64_t v_stride, int T,
                          const int32_t* slots, void* stream) {
    qmoe::clear_error();
    RopeArgs a{};
    const int rc = kv4::view_of(cache, "kv4_append", &a.cache);
    if (rc) return rc;
    if (T < 0 || (T > 0 && (!k || !v || !slots))) return qmoe::fail(QMOE_EINVAL, "kv4_append: negative T or NULL pointer");
    const int64_t width = (int64_t)cache->n_kv_heads * cache->head_dim;
    if (k_stride % 8 || v_stride % 8 || (T > 1 && (k_stride < width || v_stride < width)) || !kv4::aligned16(k) ||
        !kv4::aligned16(v))
        return qmoe::fail(QMOE_EINVAL, "kv4_append: strides must be multiples of 8 that cover a token, pointers 16-byte aligned");
    a.k = (const uint16_t*)k, a.v = (const uint16_t*)v, a.k_stride = k_stride, a.v_stride = v_stride;
    a.T = T, a.n_kv = cache->n_kv_heads, a.heads = 2 * cache->n_kv_heads, a.slots = slots;
    return cache->head_dim == 128 ? launch_rope<16>(a, false, "kv4_append", (cudaStream_t)stream) : launch_rope<8>(a, false, "kv4_append", (cudaStream_t)stream);
}

extern "C" int kv4_gather(const kv4_cache* cache, const int32_t* slots, int n, void* k_out, void* v_out, void* stream) {
    qmoe::clear_error();
    kv4::CacheView c;
    const int rc = kv4::view_of(cache, "kv4_gather", &c);
    if (rc) return rc;
    if (n < 0 || (n > 0 && (!slots || !k_out || !v_out))) return qmoe::fail(QMOE_EINVAL, "kv4_gather: negative n or NULL pointer");
    if (!kv4::aligned16(k_out) || !kv4::aligned16(v_out)) return qmoe::fail(QMOE_EINVAL, "kv4_gather: pointer not 16-byte aligned");
    if (n == 0) return QMOE_OK;
    cudaStream_t st = (cudaStream_t)stream;
    if (cache->head_dim == 128)
        return four_heads<16>(n, 2 * c.n_kv_heads) ? launch_gather<16, 4>(c, slots, n, k_out, v_out, st) : launch_gather<16, 1>(c, slots, n, k_out, v_out, st);
    return four_heads<8>(n, 2 * c.n_kv_heads) ? launch_gather<8, 4>(c, slots, n, k_out, v_out, st) : launch_gather<8, 1>(c, slots, n, k_out, v_out, st);
}
