// Attention of one new token per request over a paged key-value cache:
//
//   s_t = scale <q, k_t>,  out = sum_t exp(s_t - m) v_t / sum_t exp(s_t - m)
//
// in one pass over the positions with the running maximum m and sum of the
// softmax: when a score above m comes, the sums so far are scaled by
// exp(m_old - m_new).
#include <cmath>

#include "llm.cuh"

namespace lbcsr {

namespace {

constexpr int kThreads = 128;
constexpr int kMaxDim = 256;

enum { kBadPage = 1, kBadLength = 2 };

// A warp per request and query head; lane l holds elements l, l + 32, ...
template <typename T>
__global__ void __launch_bounds__(kThreads) paged_attention_kernel(spmv_paged_attention_t a) {
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (item >= (int64_t)a.batch * a.q_heads) return;
    const int64_t b = item / a.q_heads, h = item % a.q_heads, c = h / (a.q_heads / a.kv_heads);
    const T *q = static_cast<const T *>(a.q) + b * a.q_stride[0] + h * a.q_stride[1];
    constexpr int R = kMaxDim / 32;
    float qr[R], acc[R], m = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        acc[r] = 0.0f;
        qr[r] = lane + 32 * r < a.head_dim ? to_float(q[lane + 32 * r]) : 0.0f;
    }
    int64_t len = a.lens[b];
    const int64_t most = (int64_t)a.max_pages * a.page_size;
    if (len < 0 || len > most) {
        len = len < 0 ? 0 : most;
        if (lane == 0) atomicOr(a.status, kBadLength);
    }
    for (int64_t t = 0; t < len; ++t) {
        const int32_t page = a.table[b * a.table_stride + t / a.page_size];
        if (page < 0 || page >= a.num_pages) {
            if (lane == 0) atomicOr(a.status, kBadPage);
            continue;
        }
        const T *k = static_cast<const T *>(a.k_cache) + page * a.k_stride[0] + t % a.page_size * a.k_stride[1] +
                     c * a.k_stride[2];
        const T *v = static_cast<const T *>(a.v_cache) + page * a.v_stride[0] + t % a.page_size * a.v_stride[1] +
                     c * a.v_stride[2];
        float s = 0.0f;
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (lane + 32 * r < a.head_dim) s = fmaf(qr[r], to_float(k[lane + 32 * r]), s);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        s *= a.scale;
        const float top = fmaxf(m, s), keep = top == -INFINITY ? 1.0f : expf(m - top);
        const float p = top == -INFINITY ? 0.0f : expf(s - top);
        m = top;
        sum = fmaf(sum, keep, p);
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (lane + 32 * r < a.head_dim) acc[r] = fmaf(acc[r], keep, p * to_float(v[lane + 32 * r]));
    }
    T *out = static_cast<T *>(a.out) + b * a.out_stride[0] + h * a.out_stride[1];
#pragma unroll
    for (int r = 0; r < R; ++r)
        if (lane + 32 * r < a.head_dim) out[lane + 32 * r] = from_float<T>(sum > 0.0f ? acc[r] / sum : 0.0f);
    if (lane == 0 && a.lse) a.lse[item] = m + logf(sum);
}

template <typename T>
cudaError_t launch_attention(const spmv_paged_attention_t &a, cudaStream_t stream) {
    const int64_t items = (int64_t)a.batch * a.q_heads;
    paged_attention_kernel<T><<<(unsigned)((items + kThreads / 32 - 1) / (kThreads / 32)), kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

const char *heads_bad(int32_t batch, int32_t q_heads, int32_t kv_heads, int32_t head_dim, int elem) {
    if (batch < 0 || q_heads < 0 || kv_heads < 0) return "negative size";
    if (!elem_ok(elem)) return "unknown element type";
    if (head_dim < 8 || head_dim > kMaxDim || head_dim % 8) return "head_dim must be a multiple of 8 in [8, 256]";
    if (kv_heads < 1 || q_heads % kv_heads) return "q_heads must be a multiple of kv_heads";
    if ((int64_t)batch * q_heads >= (1LL << 31)) return "batch * q_heads must be < 2^31";
    return nullptr;
}

}  // namespace

}  // namespace lbcsr

using namespace lbcsr;

extern "C" {

spmv_status_t spmv_paged_attention_workspace(int32_t max_batch, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                             spmv_elem_t elem, size_t *bytes) {
    if (!bytes) return llm_bad("bytes is NULL");
    *bytes = 0;
    if (const char *bad = heads_bad(max_batch, q_heads, kv_heads, head_dim, elem)) return llm_bad(bad);
    return SPMV_OK;
}

spmv_status_t spmv_paged_attention(const spmv_paged_attention_t *args, spmv_stream_t stream_handle) {
    if (!args) return llm_bad("args is NULL");
    const spmv_paged_attention_t &a = *args;
    if (const char *bad = heads_bad(a.batch, a.q_heads, a.kv_heads, a.head_dim, a.elem)) return llm_bad(bad);
    if (a.num_pages < 0 || a.max_pages < 0) return llm_bad("negative size");
    if (a.page_size < 1) return llm_bad("page_size must be at least 1");
    if ((int64_t)a.num_pages * a.page_size >= (1LL << 31)) return llm_bad("num_pages * page_size must be < 2^31");
    if (a.batch == 0 || a.q_heads == 0) return SPMV_OK;
    if (!a.q || !a.out || !a.lens || !a.status) return llm_bad("q, out, lens or status is NULL");
    if (a.max_pages > 0 && !a.table) return llm_bad("table is NULL");
    if (a.num_pages > 0 && (!a.k_cache || !a.v_cache)) return llm_bad("k_cache or v_cache is NULL");
    const int size = elem_size(a.elem);
    if (!aligned_to(a.q, size) || !aligned_to(a.out, size)) return llm_bad("q or out is not aligned to its type");
    if (!aligned_to(a.k_cache, 16) || !aligned_to(a.v_cache, 16)) return llm_bad("the caches must be 16-byte aligned");
    for (int i = 0; i < 3; ++i)
        if (a.k_stride[i] * size % 16 || a.v_stride[i] * size % 16)
            return llm_bad("the caches' strides must be multiples of 16 bytes");
    size_t need = 0;
    const spmv_status_t st =
        spmv_paged_attention_workspace(a.batch, a.q_heads, a.kv_heads, a.head_dim, (spmv_elem_t)a.elem, &need);
    if (st != SPMV_OK) return st;
    if (need && (!a.workspace || a.workspace_bytes < need || !aligned_to(a.workspace, 16)))
        return llm_bad("workspace is NULL, too small or not 16-byte aligned");
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_handle);
    const cudaError_t e = a.elem == SPMV_ELEM_F32    ? launch_attention<float>(a, stream)
                          : a.elem == SPMV_ELEM_BF16 ? launch_attention<__nv_bfloat16>(a, stream)
                                                     : launch_attention<__half>(a, stream);
    return llm_launched("spmv_paged_attention launch", e);
}

}  // extern "C"
