// Softmax attention over the 4-bit paged key/value cache.

#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "kv4_common.cuh"

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
__device__ __forceinline__ bool request(const AttnArgs& a, int b, int* q0, int* q_len, int* kv_len) {
    const int s = a.q_start[b], e = a.q_start[b + 1], n = a.kv_len[b];
    *q0 = s, *q_len = e - s, *kv_len = n;
    if (s < 0 || e < s || e > a.n_q_tokens || n < 0) {
        attn_set_error(QMOE_EINVAL);
        return false;
    }
    if (e - s > a.max_q || n > a.max_kv) {
        attn_set_error(QMOE_ECAPACITY);
        return false;
    }
    return true;
}

// A warp per (query, head): a lane per key for the scores, head_dim / 32 values a lane for the sums.
template <int D>
__global__ void __launch_bounds__(128) attention_kernel(AttnArgs a) {
    __shared__ float qs[4][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = blockIdx.x * 4 + warp;
    const int b = blockIdx.z;
    int q0, q_len, len;
    if (!request(a, b, &q0, &q_len, &len)) return;
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
    *bytes = 0;
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
    const dim3 grid((n_q_heads + 3) / 4, max_q, B);
    if (cache->head_dim == 128)
        attention_kernel<128><<<grid, 128, 0, (cudaStream_t)stream>>>(a);
    else
        attention_kernel<64><<<grid, 128, 0, (cudaStream_t)stream>>>(a);
    return qmoe::launch_check("kv4_attention");
}
