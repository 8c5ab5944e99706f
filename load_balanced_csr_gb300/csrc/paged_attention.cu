// C entry points of the paged attention, and its kernels for 32-bit elements
// (paged_attention.cuh has the kernel, paged_attention_bf16.cu and
// paged_attention_f16.cu the 16-bit ones).
#include "paged_attention.cuh"

namespace lbcsr {

namespace {

// Warps and stages: with more warps the instructions' latency matters less (16
// requests of up to 5,000 positions, 4 kv heads of 72 with 3 heads each: 47 us
// with 12 warps of 2 stages, 53 with 8 of 4), as far as registers and the
// shared memory for stages and queries go.
template <int GT, typename F>
auto with_f32(int dim, F f) {
    constexpr bool large = GT == 8;
    if (dim <= 64) return f(TileF32<64, GT, large ? 16 : 12, large ? 2 : 3>());
    if (dim <= 96) return f(TileF32<96, GT, large ? 8 : 12, large ? 3 : 2>());
    if (dim <= 128) return f(TileF32<128, GT, large ? 8 : 10, 2>());
    return f(TileF32<256, GT, large ? 4 : 5, 2>());
}
template <typename F>
auto with_f32(int dim, int group, F f) {
    return group == 1 ? with_f32<1>(dim, f) : group <= 4 ? with_f32<4>(dim, f) : with_f32<8>(dim, f);
}

// What is wrong with the arguments that both entry points share; `size`: bytes of an element of the caches.
const char *attention_bad(const spmv_paged_attention_t &a, int size) {
    if (a.num_pages < 0 || a.max_pages < 0) return "negative size";
    if (a.page_size < 1) return "page_size must be at least 1";
    if ((int64_t)a.num_pages * a.page_size >= (1LL << 31)) return "num_pages * page_size must be < 2^31";
    // one request's units (chunks of at least 8 positions, and its rows' own) are counted in 32 bits
    if ((int64_t)a.max_pages * a.page_size >= (1LL << 31) - 64 ||
        ((int64_t)a.max_pages * a.page_size / 8 + 1 + kRowCost) * std::max(a.q_heads, a.kv_heads) >= (1LL << 31))
        return "max_pages * page_size * q_heads is too large";
    if (a.batch == 0 || a.q_heads == 0) return nullptr;
    if (!a.q || !a.out || !a.lens || !a.status) return "q, out, lens or status is NULL";
    if (a.max_pages > 0 && !a.table) return "table is NULL";
    if (a.num_pages > 0 && (!a.k_cache || !a.v_cache)) return "k_cache or v_cache is NULL";
    const int own = elem_size(a.elem);
    if (!aligned_to(a.q, own) || !aligned_to(a.out, own)) return "q or out is not aligned to its type";
    if (!aligned_to(a.k_cache, 16) || !aligned_to(a.v_cache, 16)) return "the caches must be 16-byte aligned";
    for (int i = 0; i < 3; ++i)
        if (a.k_stride[i] * size % 16 || a.v_stride[i] * size % 16) return "the caches' strides must be multiples of 16 bytes";
    return nullptr;
}

const char *heads_bad(int32_t batch, int32_t q_heads, int32_t kv_heads, int32_t head_dim, int elem) {
    if (batch < 0 || q_heads < 0 || kv_heads < 0) return "negative size";
    if (!elem_ok(elem)) return "unknown element type";
    if (head_dim < 8 || head_dim > kMaxDim || head_dim % 8) return "head_dim must be a multiple of 8 in [8, 256]";
    if (kv_heads < 1 || q_heads % kv_heads) return "q_heads must be a multiple of kv_heads";
    if ((int64_t)batch * q_heads >= (1LL << 31)) return "batch * q_heads must be < 2^31";
    if ((int64_t)q_heads * head_dim >= (1LL << 30)) return "q_heads * head_dim must be < 2^30";
    return nullptr;
}

const char *codes_bad(int32_t head_dim, int elem) {
    if (elem == SPMV_ELEM_F32) return "over caches of codes q and out are bf16 or f16";
    return head_dim % 16 ? "over caches of codes head_dim must be a multiple of 16" : nullptr;
}

}  // namespace

size_t attention_workspace_f32(int dim, int group, int sms) {
    return with_f32(dim, group, [&](auto tile) { return workspace_of<decltype(tile)>(sms); });
}

cudaError_t launch_attention_f32(const spmv_paged_attention_t &a, int sms, cudaStream_t stream) {
    return with_f32(a.head_dim, a.q_heads / a.kv_heads,
                    [&](auto tile) { return launch_attention<decltype(tile)>(a, sms, stream); });
}

}  // namespace lbcsr

using namespace lbcsr;

extern "C" {

spmv_status_t spmv_paged_attention_workspace(int32_t max_batch, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                             spmv_elem_t elem, size_t *bytes) {
    if (!bytes) return llm_bad("bytes is NULL");
    *bytes = 0;
    if (const char *bad = heads_bad(max_batch, q_heads, kv_heads, head_dim, elem)) return llm_bad(bad);
    const int sms = device_sm_count();
    if (sms <= 0) return llm_fail(SPMV_ERR_CUDA, "no CUDA device");
    const int group = q_heads / kv_heads;
    *bytes = elem == SPMV_ELEM_F32    ? attention_workspace_f32(head_dim, group, sms)
             : elem == SPMV_ELEM_BF16 ? attention_workspace_bf16(head_dim, group, sms)
                                      : attention_workspace_f16(head_dim, group, sms);
    return SPMV_OK;
}

spmv_status_t spmv_paged_attention(const spmv_paged_attention_t *args, spmv_stream_t stream_handle) {
    if (!args) return llm_bad("args is NULL");
    const spmv_paged_attention_t &a = *args;
    if (const char *bad = heads_bad(a.batch, a.q_heads, a.kv_heads, a.head_dim, a.elem)) return llm_bad(bad);
    if (const char *bad = attention_bad(a, elem_size(a.elem))) return llm_bad(bad);
    if (a.batch == 0 || a.q_heads == 0) return SPMV_OK;
    size_t need = 0;
    const spmv_status_t st =
        spmv_paged_attention_workspace(a.batch, a.q_heads, a.kv_heads, a.head_dim, (spmv_elem_t)a.elem, &need);
    if (st != SPMV_OK) return st;
    if (need && (!a.workspace || a.workspace_bytes < need || !aligned_to(a.workspace, 16)))
        return llm_bad("workspace is NULL, too small or not 16-byte aligned");
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_handle);
    const int sms = device_sm_count();
    const cudaError_t e = a.elem == SPMV_ELEM_F32    ? launch_attention_f32(a, sms, stream)
                          : a.elem == SPMV_ELEM_BF16 ? launch_attention_bf16(a, sms, stream)
                                                     : launch_attention_f16(a, sms, stream);
    return llm_launched("spmv_paged_attention launch", e);
}

spmv_status_t spmv_paged_attention_e4m3_workspace(int32_t max_batch, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                                  spmv_elem_t elem, size_t *bytes) {
    if (!bytes) return llm_bad("bytes is NULL");
    *bytes = 0;
    if (const char *bad = heads_bad(max_batch, q_heads, kv_heads, head_dim, elem)) return llm_bad(bad);
    if (const char *bad = codes_bad(head_dim, elem)) return llm_bad(bad);
    const int sms = device_sm_count();
    if (sms <= 0) return llm_fail(SPMV_ERR_CUDA, "no CUDA device");
    *bytes = attention_workspace_e4m3(head_dim, q_heads / kv_heads, sms);
    return SPMV_OK;
}

spmv_status_t spmv_paged_attention_e4m3(const spmv_paged_attention_t *args, int32_t block, const float *k_scales,
                                        const int64_t *k_scale_stride, const float *v_scales, const int64_t *v_scale_stride,
                                        spmv_stream_t stream_handle) {
    if (!args) return llm_bad("args is NULL");
    const spmv_paged_attention_t &a = *args;
    if (const char *bad = heads_bad(a.batch, a.q_heads, a.kv_heads, a.head_dim, a.elem)) return llm_bad(bad);
    if (const char *bad = codes_bad(a.head_dim, a.elem)) return llm_bad(bad);
    if (const char *bad = attention_bad(a, 1)) return llm_bad(bad);
    if (block < 1 || a.page_size % block) return llm_bad("page_size must be a multiple of block");
    if (!k_scale_stride || !v_scale_stride) return llm_bad("a stride array is NULL");
    if (a.batch == 0 || a.q_heads == 0) return SPMV_OK;
    if (a.num_pages > 0 && (!k_scales || !v_scales)) return llm_bad("k_scales or v_scales is NULL");
    if (!aligned_to(k_scales, 4) || !aligned_to(v_scales, 4)) return llm_bad("the scales are not aligned to their type");
    size_t need = 0;
    const spmv_status_t st =
        spmv_paged_attention_e4m3_workspace(a.batch, a.q_heads, a.kv_heads, a.head_dim, (spmv_elem_t)a.elem, &need);
    if (st != SPMV_OK) return st;
    if (need && (!a.workspace || a.workspace_bytes < need || !aligned_to(a.workspace, 16)))
        return llm_bad("workspace is NULL, too small or not 16-byte aligned");
    AttendScales scales;
    scales.k = k_scales, scales.v = v_scales;
    std::copy(k_scale_stride, k_scale_stride + 3, scales.k_stride);
    std::copy(v_scale_stride, v_scale_stride + 3, scales.v_stride);
    set_divisor((uint32_t)block, &scales.mul, &scales.shift);
    return llm_launched("spmv_paged_attention_e4m3 launch",
                        launch_attention_e4m3(a, scales, device_sm_count(), reinterpret_cast<cudaStream_t>(stream_handle)));
}

}  // extern "C"
