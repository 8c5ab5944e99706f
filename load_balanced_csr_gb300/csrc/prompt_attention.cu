// Attention of whole prompts, or of chunks of them, packed one behind the other:
//
//   s_ij = scale <q_i, k_j>,  out_i = sum_j exp(s_ij - m_i) v_j / sum_j exp(s_ij - m_i)
//
// with j over the keys of i's request, of them those up to i's own place where
// it is causal.
#include <cmath>

#include "internal.cuh"
#include "llm.cuh"

namespace lbcsr {

namespace {

enum { kBadQueries = 1, kBadKeys = 2 };

template <typename T>
__global__ void __launch_bounds__(128) prompt_attention_kernel(spmv_prompt_attention_t a) {
    after_previous();
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5), i = row / a.q_heads;
    const int head = (int)(row - i * a.q_heads), kvh = head / (a.q_heads / a.kv_heads);
    const int32_t *kv_ptr = a.kv_ptr ? a.kv_ptr : a.q_ptr;
    for (int r = threadIdx.x; blockIdx.x == 0 && r < a.requests; r += 128) {
        if (a.q_ptr[r] < 0 || a.q_ptr[r + 1] < a.q_ptr[r] || a.q_ptr[r + 1] > a.tokens) atomicOr(a.status, kBadQueries);
        else if (kv_ptr[r] < 0 || kv_ptr[r + 1] < kv_ptr[r] || kv_ptr[r + 1] > a.keys) atomicOr(a.status, kBadKeys);
    }
    if (i >= a.tokens) return;
    int r = 0;
    while (r < a.requests && !(a.q_ptr[r] <= i && i < a.q_ptr[r + 1])) ++r;
    if (r == a.requests) return;
    const int32_t q0 = a.q_ptr[r], q1 = a.q_ptr[r + 1], k0 = kv_ptr[r], k1 = kv_ptr[r + 1];
    if (q0 < 0 || q1 > a.tokens || k0 < 0 || k1 < k0 || k1 > a.keys) return;
    int64_t n = k1 - k0;
    if (a.causal) n = min(n, n - (q1 - q0) + (i - q0) + 1);
    const T *q = static_cast<const T *>(a.q) + i * a.q_stride[0] + head * a.q_stride[1];
    float o[8] = {}, m = -INFINITY, l = 0.0f;
    for (int64_t j0 = 0; j0 < n; j0 += 32) {
        const bool in = j0 + lane < n;
        float s = -INFINITY;
        if (in) {
            const T *k = static_cast<const T *>(a.k) + (k0 + j0 + lane) * a.k_stride[0] + kvh * a.k_stride[1];
            s = 0.0f;
            for (int d = 0; d < a.head_dim; ++d) s = fmaf(to_float(q[d]), to_float(k[d]), s);
            s *= a.scale;
        }
        float top = s;
        for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        top = fmaxf(top, m);
        const float base = top == -INFINITY ? 0.0f : top, keep = m == -INFINITY ? 0.0f : expf(m - base);
        const float w = in ? expf(s - base) : 0.0f;
        float sum = w;
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        l = l * keep + sum;
        m = top;
        for (int e = 0; e < 8; ++e) o[e] *= keep;
        for (int j = 0; j < 32 && j0 + j < n; ++j) {
            const float wj = __shfl_sync(0xffffffffu, w, j);
            const T *v = static_cast<const T *>(a.v) + (k0 + j0 + j) * a.v_stride[0] + kvh * a.v_stride[1];
            for (int e = 0; e < 8; ++e)
                if (lane + 32 * e < a.head_dim) o[e] = fmaf(wj, to_float(v[lane + 32 * e]), o[e]);
        }
    }
    T *out = static_cast<T *>(a.out) + i * a.out_stride[0] + head * a.out_stride[1];
    for (int e = 0; e < 8; ++e)
        if (lane + 32 * e < a.head_dim) out[lane + 32 * e] = from_float<T>(l == 0.0f ? 0.0f : o[e] / l);
    if (lane == 0 && a.lse) a.lse[i * a.q_heads + head] = l == 0.0f ? -INFINITY : m + logf(l);
}

const char *prompt_bad(const spmv_prompt_attention_t &a) {
    if (a.requests < 0 || a.tokens < 0 || a.keys < 0 || a.q_heads < 0) return "negative size";
    if (a.elem != SPMV_ELEM_BF16 && a.elem != SPMV_ELEM_F16) return "elements must be bf16 or f16";
    if (a.head_dim < 8 || a.head_dim > 256 || a.head_dim % 8) return "head_dim must be a multiple of 8 in [8, 256]";
    if (a.kv_heads < 1 || a.q_heads % a.kv_heads) return "q_heads must be a multiple of kv_heads";
    if (a.q_heads / a.kv_heads > 128) return "q_heads must be at most 128 times kv_heads";
    if ((int64_t)a.tokens * a.q_heads >= (1LL << 31)) return "tokens * q_heads must be < 2^31";
    if (a.requests == 0 || a.tokens == 0 || a.q_heads == 0) return nullptr;
    if (!a.q || !a.q_ptr || !a.out || !a.status) return "q, q_ptr, out or status is NULL";
    if (a.keys > 0 && (!a.k || !a.v)) return "k or v is NULL";
    if (!aligned_to(a.q_ptr, 4) || !aligned_to(a.kv_ptr, 4) || !aligned_to(a.lse, 4) || !aligned_to(a.status, 4))
        return "q_ptr, kv_ptr, lse or status is not aligned to its type";
    if (!aligned_to(a.q, 16) || !aligned_to(a.k, 16) || !aligned_to(a.v, 16) || !aligned_to(a.out, 16))
        return "q, k, v and out must be 16-byte aligned";
    for (int i = 0; i < 2; ++i)
        if (a.q_stride[i] % 8 || a.k_stride[i] % 8 || a.v_stride[i] % 8 || a.out_stride[i] % 8)
            return "strides must be multiples of 16 bytes";
    return nullptr;
}

}  // namespace

}  // namespace lbcsr

using namespace lbcsr;

extern "C" {

spmv_status_t spmv_prompt_attention(const spmv_prompt_attention_t *args, spmv_stream_t stream_handle) {
    if (!args) return llm_bad("args is NULL");
    const spmv_prompt_attention_t &a = *args;
    if (const char *bad = prompt_bad(a)) return llm_bad(bad);
    if (a.requests == 0 || a.tokens == 0 || a.q_heads == 0) return SPMV_OK;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_handle);
    const unsigned grid = (unsigned)(((int64_t)a.tokens * a.q_heads + 3) / 4);
    return llm_launched("spmv_prompt_attention launch",
                        a.elem == SPMV_ELEM_BF16 ? launch_chained(prompt_attention_kernel<__nv_bfloat16>, grid, 128, 0, 0, stream, a)
                                                 : launch_chained(prompt_attention_kernel<__half>, grid, 128, 0, 0, stream, a));
}

}  // extern "C"
