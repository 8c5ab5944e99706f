// Page tables of a key-value cache and the stores through them.
//
// spmv_pages_append: with held_r = ceil(past_r / P), a prefix sum over the
// requests of (fresh_r, pages needed) gives each new token's place and each
// new page's place in the free list; then each token finds its request by
// binary search in the prefix sums (as a merge-path tile finds its first
// row), computes its slot from the table or, for a page not held before, from
// the free list, and the token that opens a page writes the table's entry.
// It is bound by latency when there are few tokens, by its instructions when
// there are many (0.69 of the issue slots): up to kBlockRequests requests every
// block makes the prefix sums for itself in shared memory, and there is one
// launch (256 requests with a token each 6.4 us a step, 2,048 requests with 860
// thousand tokens 10.4 us, of which its 6.9 MB are 1 us); beyond, one block
// makes them in global memory first.  One block's sums and a second launch took 11.6 and
// 21.8 us.
//
// spmv_paged_store: a copy, 16 bytes a lane, four in flight for keys and
// values each; 65,535 tokens of 8 heads of 128 f16, 5 % of them padding (510
// MB) 75.5 us: 6.75 TB/s, the measured copy's rate.  5 heads of 72 bf16 32.5
// us (28 at that rate); a warp per token, whose last turn such rows fill in
// part, took 47.
#include <algorithm>
#include <climits>

#include "internal.cuh"
#include "llm.cuh"

namespace lbcsr {

namespace {

// ---------------------------------------------------------------- append
constexpr int kAppendThreads = 1024;
constexpr int kRequestsPerThread = 4;  // consecutive: 4096 requests are read at once
static_assert(kAppendThreads == 1024, "a warp's lanes are the block's warps when their sums are added");
constexpr int kTokensPerThread = 4;    // consecutive, so that they are stored together
constexpr int kBlockRequests = 4096;

enum { kFreeEnded = 1, kRowShort = 2, kTooManyTokens = 4, kBadLength = 8, kBadPage = 16 };

// What the prefix sums leave of a request: where its new tokens begin, what it
// held, the place of its first new page in the free list (-1: not served).
struct Request {
    int32_t token, past, first;
};

struct AppendArgs {
    int32_t requests, page, num_pages, num_free, max_pages, max_tokens;
    const int32_t *past, *fresh, *free_pages;
    int32_t *table;
    int64_t ld_table;
    int32_t *token_ptr, *lens, *slots, *positions, *taken, *status;
    Request *made;  // workspace [requests], more than kBlockRequests only
    uint32_t page_mul, page_shift;  // division by the page size
};

// t / page for t < 2^32: (mulhi(t, page_mul) + t) >> page_shift without losing the sum's carry.
__device__ __forceinline__ uint32_t page_at(const AppendArgs &a, uint32_t t) {
    return (uint32_t)(((unsigned long long)__umulhi(t, a.page_mul) + t) >> a.page_shift);
}
// the pages of n tokens
__device__ __forceinline__ uint32_t pages_of(const AppendArgs &a, uint32_t n) { return n ? page_at(a, n - 1) + 1 : 0; }

__device__ __forceinline__ bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Fills req[0 .. requests] (the last one's token: the number of new tokens);
// the block that `writes` also gives the outputs per request.
__device__ __forceinline__ void scan_requests(const AppendArgs &a, Request *req, bool writes) {
    __shared__ long long warp_sum[kAppendThreads / 32];
    __shared__ int32_t all_used;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long carry = 0;  // pages << 32 | tokens
    int32_t flags = 0, used = 0;
    if (threadIdx.x == 0) all_used = 0;
    for (int64_t r0 = 0; r0 < a.requests; r0 += kAppendThreads * kRequestsPerThread) {
        const int64_t r1 = r0 + threadIdx.x * kRequestsPerThread;
        int32_t past[kRequestsPerThread], fresh[kRequestsPerThread], need[kRequestsPerThread];
        bool fits[kRequestsPerThread];
#pragma unroll
        for (int j = 0; j < kRequestsPerThread; ++j) {
            past[j] = r1 + j < a.requests ? a.past[r1 + j] : 0;
            fresh[j] = r1 + j < a.requests ? a.fresh[r1 + j] : 0;
        }
        long long mine = 0;
#pragma unroll
        for (int j = 0; j < kRequestsPerThread; ++j) {
            if (past[j] < 0 || fresh[j] < 0) flags |= kBadLength, past[j] = max(past[j], 0), fresh[j] = max(fresh[j], 0);
            const uint32_t held = pages_of(a, (uint32_t)past[j]), want = pages_of(a, (uint32_t)past[j] + (uint32_t)fresh[j]);
            fits[j] = true, need[j] = 0;
            if (held > (uint32_t)a.max_pages) fits[j] = false, flags |= kBadLength;
            else if (want > (uint32_t)a.max_pages) fits[j] = false, flags |= kRowShort;
            else need[j] = (int32_t)(want - held);
            mine += ((long long)need[j] << 32) + fresh[j];
        }
        long long scan = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long up = __shfl_up_sync(0xffffffffu, scan, d);
            if (lane >= d) scan += up;
        }
        if (lane == 31) warp_sum[warp] = scan;
        __syncthreads();
        long long before = lane < warp ? warp_sum[lane] : 0, all = warp_sum[lane];
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            before += __shfl_xor_sync(0xffffffffu, before, d);
            all += __shfl_xor_sync(0xffffffffu, all, d);
        }
        long long start = carry + before + scan - mine;
        carry += all;
#pragma unroll
        for (int j = 0; j < kRequestsPerThread; ++j) {
            const int64_t r = r1 + j;
            if (r >= a.requests) break;
            const int32_t first = (int32_t)(start >> 32), tokens = (int32_t)start;
            bool served = fits[j];
            if (need[j] > 0 && (long long)first + need[j] > a.num_free) served = false, flags |= kFreeEnded;
            if (fresh[j] > 0 && (long long)tokens + fresh[j] > a.max_tokens) served = false, flags |= kTooManyTokens;
            if (served && need[j] > 0) used = max(used, first + need[j]);
            req[r] = Request{tokens, past[j], served ? first : -1};
            if (writes) a.token_ptr[r] = tokens, a.lens[r] = served ? past[j] + fresh[j] : past[j];
            start += ((long long)need[j] << 32) + fresh[j];
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) req[a.requests].token = (int32_t)carry;
    __syncthreads();
    if (writes) {
        if (flags) atomicOr(a.status, flags);
        if (used) atomicMax(&all_used, used);
        __syncthreads();
        if (threadIdx.x == 0) a.token_ptr[a.requests] = (int32_t)carry, *a.taken = all_used;
    }
}

__global__ void __launch_bounds__(kAppendThreads) pages_scan_kernel(AppendArgs a) {
    after_previous();
    scan_requests(a, a.made, true);
}

// SCAN: the block makes the prefix sums itself.
template <bool SCAN>
__global__ void __launch_bounds__(kAppendThreads) pages_append_kernel(AppendArgs a) {
    extern __shared__ __align__(16) char smem[];
    const Request *req = a.made;
    after_previous();
    if (SCAN) {
        scan_requests(a, reinterpret_cast<Request *>(smem), blockIdx.x == 0);
        req = reinterpret_cast<const Request *>(smem);
    }
    const int32_t tokens = min(req[a.requests].token, a.max_tokens);
    const bool whole = aligned16(a.slots) && aligned16(a.positions);
    for (int64_t i0 = ((int64_t)blockIdx.x * kAppendThreads + threadIdx.x) * kTokensPerThread; i0 < a.max_tokens;
         i0 += (int64_t)gridDim.x * kAppendThreads * kTokensPerThread) {
        int r = 0;
        if (i0 < tokens) {
            int hi = a.requests - 1;  // the last request with token <= i0: the one that holds i0
            while (r < hi) {
                const int mid = (r + hi + 1) >> 1;
                if (req[mid].token <= i0) r = mid;
                else hi = mid - 1;
            }
        }
        // where each token's page number is, so that all are read together; then the slots
        int32_t slot[kTokensPerThread], position[kTokensPerThread], inside[kTokensPerThread], id[kTokensPerThread];
        const int32_t *from[kTokensPerThread];
        int32_t *opens[kTokensPerThread];  // the table's entry, for the token that opens a page
#pragma unroll
        for (int u = 0; u < kTokensPerThread; ++u) {
            const int64_t i = i0 + u;
            slot[u] = position[u] = -1, inside[u] = 0;
            from[u] = nullptr, opens[u] = nullptr;
            if (i >= tokens) continue;
            while (r + 1 < a.requests && req[r + 1].token <= i) ++r;
            const Request now = req[r];
            const int32_t at = now.past + (int32_t)(i - now.token);
            const int32_t page = (int32_t)page_at(a, (uint32_t)at);
            position[u] = at;
            inside[u] = at - page * a.page;
            if (now.first < 0 || at < 0 || page >= a.max_pages) continue;  // the last two only if sums passed 32 bits
            const int32_t held = (int32_t)pages_of(a, (uint32_t)now.past);
            const int64_t place = (int64_t)now.first + page - held;
            int32_t *entry = a.table + r * a.ld_table + page;
            if (page < held) {
                from[u] = entry;
            } else if (place < a.num_free) {
                from[u] = a.free_pages + place;
                if (inside[u] == 0) opens[u] = entry;
            }
        }
#pragma unroll
        for (int u = 0; u < kTokensPerThread; ++u) id[u] = from[u] ? *from[u] : -1;
#pragma unroll
        for (int u = 0; u < kTokensPerThread; ++u) {
            if (!from[u]) continue;
            if (opens[u]) *opens[u] = id[u];
            if ((uint32_t)id[u] < (uint32_t)a.num_pages) slot[u] = id[u] * a.page + inside[u];
            else atomicOr(a.status, kBadPage);
        }
        if (whole && i0 + kTokensPerThread <= a.max_tokens) {
            *reinterpret_cast<int4 *>(a.slots + i0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
            *reinterpret_cast<int4 *>(a.positions + i0) = make_int4(position[0], position[1], position[2], position[3]);
        } else {
#pragma unroll
            for (int u = 0; u < kTokensPerThread; ++u)
                if (i0 + u < a.max_tokens) a.slots[i0 + u] = slot[u], a.positions[i0 + u] = position[u];
        }
    }
}

// ---------------------------------------------------------------- store
constexpr int kStoreThreads = 256;

struct StoreArgs {
    int64_t items;            // vectors of all tokens
    int32_t row, vecs;        // vectors of a token, of a head
    int32_t num_pages, page;
    uint32_t row_mul, row_shift, vecs_mul, vecs_shift, page_mul, page_shift;
    const int32_t *slots;
    int64_t ks[2], vs[2], kc[3], vc[3];
};

__device__ __forceinline__ uint32_t divided(uint32_t t, uint32_t mul, uint32_t shift) {
    return (uint32_t)(((unsigned long long)__umulhi(t, mul) + t) >> shift);
}

// A block takes kStoreThreads * U neighbouring vectors, whichever tokens they
// are of, so that rows of any length fill its lanes.
template <typename T, int N, int U>
__global__ void __launch_bounds__(kStoreThreads)
paged_store_kernel(StoreArgs a, const T *k, const T *v, T *kc, T *vc) {
    using V = Vec<T, N>;
    after_previous();
    const int64_t first = (int64_t)blockIdx.x * (kStoreThreads * U), token0 = first / a.row;
    const uint32_t over = (uint32_t)(first - token0 * a.row) + threadIdx.x;
    int64_t token[U];
    uint32_t head[U], at[U];
    int32_t slot[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        // past the last vector: the first again, not stored
        const bool in = first + threadIdx.x + u * kStoreThreads < a.items;
        const uint32_t e = in ? over + u * kStoreThreads : 0, t = divided(e, a.row_mul, a.row_shift), in_row = e - t * a.row;
        token[u] = token0 + t;
        head[u] = divided(in_row, a.vecs_mul, a.vecs_shift);
        at[u] = (in_row - head[u] * a.vecs) * N;
        slot[u] = in ? a.slots[token[u]] : -1;
    }
    // read whatever the slot says, so that no load waits for it
    V kv[U], vv[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        kv[u] = *reinterpret_cast<const V *>(k + token[u] * a.ks[0] + head[u] * a.ks[1] + at[u]);
        vv[u] = *reinterpret_cast<const V *>(v + token[u] * a.vs[0] + head[u] * a.vs[1] + at[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t page = divided((uint32_t)slot[u], a.page_mul, a.page_shift);
        if (slot[u] < 0 || page >= (uint32_t)a.num_pages) continue;
        const int64_t in = (uint32_t)slot[u] - page * a.page;
        *reinterpret_cast<V *>(kc + page * a.kc[0] + in * a.kc[1] + head[u] * a.kc[2] + at[u]) = kv[u];
        *reinterpret_cast<V *>(vc + page * a.vc[0] + in * a.vc[1] + head[u] * a.vc[2] + at[u]) = vv[u];
    }
}

template <typename T, int N>
cudaError_t launch_store(const StoreArgs &a, const void *k, const void *v, void *kc, void *vc, cudaStream_t stream) {
    constexpr int U = N == 1 ? 8 : 4;
    const int64_t per_block = kStoreThreads * U;
    return launch_chained(paged_store_kernel<T, N, U>, (unsigned)((a.items + per_block - 1) / per_block), kStoreThreads, 0, 0,
                          stream, a, static_cast<const T *>(k), static_cast<const T *>(v), static_cast<T *>(kc),
                          static_cast<T *>(vc));
}

// n entries at a and m at b have bytes in common
bool overlap(const int32_t *a, int64_t n, const int32_t *b, int64_t m) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return n > 0 && m > 0 && x < y + 4 * (uintptr_t)m && y < x + 4 * (uintptr_t)n;
}

bool on_16(const void *p, const int64_t *strides, int n, int size) {
    if (!aligned_to(p, 16)) return false;
    for (int i = 0; i < n; ++i)
        if (strides[i] * size % 16) return false;
    return true;
}

}  // namespace

}  // namespace lbcsr

using namespace lbcsr;

extern "C" {

spmv_status_t spmv_pages_workspace(int32_t requests, size_t *bytes) {
    if (!bytes) return llm_bad("bytes is NULL");
    *bytes = 0;
    if (requests < 0) return llm_bad("negative size");
    *bytes = requests > kBlockRequests ? sizeof(Request) * ((size_t)requests + 1) : 0;
    return SPMV_OK;
}

spmv_status_t spmv_pages_append(int32_t requests, const int32_t *past, const int32_t *fresh, int32_t page_size,
                                int32_t num_pages, const int32_t *free_pages, int32_t num_free, int32_t *table,
                                int64_t ld_table, int32_t max_pages, int32_t max_tokens, int32_t *token_ptr,
                                int32_t *lens, int32_t *slots, int32_t *positions, int32_t *taken, int32_t *status,
                                void *workspace, size_t workspace_bytes, spmv_stream_t stream_handle) {
    size_t need = 0;
    const spmv_status_t st = spmv_pages_workspace(requests, &need);
    if (st != SPMV_OK) return st;
    if (num_pages < 0 || num_free < 0 || max_pages < 0 || max_tokens < 0) return llm_bad("negative size");
    if (page_size < 1) return llm_bad("page_size must be at least 1");
    if ((int64_t)num_pages * page_size >= (1LL << 31)) return llm_bad("num_pages * page_size must be < 2^31");
    if (!token_ptr || !taken || !status) return llm_bad("token_ptr, taken or status is NULL");
    if (requests > 0 && (!past || !fresh || !lens)) return llm_bad("past, fresh or lens is NULL");
    // every block reads the lengths while others write
    const int64_t n = requests;
    for (const int32_t *in : {past, fresh})
        if (overlap(in, n, lens, n) || overlap(in, n, token_ptr, n + 1) || overlap(in, n, slots, max_tokens) ||
            overlap(in, n, positions, max_tokens))
            return llm_bad("lens, token_ptr, slots and positions must not overlap past or fresh");
    if (requests > 0 && max_pages > 0 && !table) return llm_bad("table is NULL");
    if (ld_table < max_pages) return llm_bad("ld_table is smaller than max_pages");
    if (num_free > 0 && !free_pages) return llm_bad("free_pages is NULL");
    if (max_tokens > 0 && (!slots || !positions)) return llm_bad("slots or positions is NULL");
    if (need && (!workspace || workspace_bytes < need || !aligned_to(workspace, 16)))
        return llm_bad("workspace is NULL, too small or not 16-byte aligned");
    AppendArgs a;
    a.requests = requests, a.page = page_size, a.num_pages = num_pages, a.num_free = num_free;
    a.max_pages = max_pages, a.max_tokens = max_tokens;
    a.past = past, a.fresh = fresh, a.free_pages = free_pages;
    a.table = table, a.ld_table = ld_table;
    a.token_ptr = token_ptr, a.lens = lens, a.slots = slots, a.positions = positions, a.taken = taken;
    a.status = status;
    a.made = static_cast<Request *>(workspace);
    set_divisor((uint32_t)page_size, &a.page_mul, &a.page_shift);
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_handle);
    const int64_t per_block = (int64_t)kAppendThreads * kTokensPerThread;
    // one block an SM (its registers): more would make the prefix sums a second time
    const int blocks = (int)std::max<int64_t>(1, std::min<int64_t>((max_tokens + per_block - 1) / per_block, device_sm_count()));
    cudaError_t e = cudaSuccess;
    if (requests <= kBlockRequests) {
        const size_t smem = sizeof(Request) * ((size_t)requests + 1);
        if (smem > 47 * 1024)  // the function's limit is every host thread's: the most that any call needs
            e = cudaFuncSetAttribute(pages_append_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)(sizeof(Request) * (kBlockRequests + 1)));
        if (e == cudaSuccess) e = launch_chained(pages_append_kernel<true>, blocks, kAppendThreads, smem, 0, stream, a);
    } else {
        e = launch_chained(pages_scan_kernel, 1, kAppendThreads, 0, 0, stream, a);
        if (e == cudaSuccess && max_tokens > 0)
            e = launch_chained(pages_append_kernel<false>, blocks, kAppendThreads, 0, 0, stream, a);
    }
    return llm_launched("spmv_pages_append launch", e);
}

spmv_status_t spmv_paged_store(int32_t tokens, int32_t heads, int32_t head_dim, spmv_elem_t elem,
                               const int32_t *slots, int32_t num_pages, int32_t page_size, const void *k,
                               const int64_t *k_stride, const void *v, const int64_t *v_stride, void *k_cache,
                               const int64_t *k_cache_stride, void *v_cache, const int64_t *v_cache_stride,
                               spmv_stream_t stream_handle) {
    if (tokens < 0 || heads < 0 || head_dim < 0 || num_pages < 0) return llm_bad("negative size");
    if (page_size < 1) return llm_bad("page_size must be at least 1");
    if ((int64_t)num_pages * page_size >= (1LL << 31)) return llm_bad("num_pages * page_size must be < 2^31");
    if ((int64_t)heads * head_dim >= (1LL << 30)) return llm_bad("heads * head_dim must be < 2^30");
    if ((int64_t)tokens * heads * head_dim >= (1LL << 41)) return llm_bad("tokens * heads * head_dim must be < 2^41");
    if (!elem_ok(elem)) return llm_bad("unknown element type");
    if (!k_stride || !v_stride || !k_cache_stride || !v_cache_stride) return llm_bad("a stride array is NULL");
    if (tokens == 0 || heads == 0 || head_dim == 0 || num_pages == 0) return SPMV_OK;
    if (!slots || !k || !v || !k_cache || !v_cache) return llm_bad("slots, k, v or a cache is NULL");
    const int size = elem_size(elem);
    if (!aligned_to(k, size) || !aligned_to(v, size) || !aligned_to(k_cache, size) || !aligned_to(v_cache, size))
        return llm_bad("k, v or a cache is not aligned to its type");
    const bool wide = head_dim * size % 16 == 0 && on_16(k, k_stride, 2, size) && on_16(v, v_stride, 2, size) &&
                      on_16(k_cache, k_cache_stride, 3, size) && on_16(v_cache, v_cache_stride, 3, size);
    StoreArgs a;
    a.num_pages = num_pages, a.page = page_size, a.slots = slots;
    a.vecs = wide ? head_dim * size / 16 : head_dim;
    a.row = heads * a.vecs;
    a.items = (int64_t)tokens * a.row;
    set_divisor((uint32_t)a.row, &a.row_mul, &a.row_shift);
    set_divisor((uint32_t)a.vecs, &a.vecs_mul, &a.vecs_shift);
    set_divisor((uint32_t)page_size, &a.page_mul, &a.page_shift);
    for (int i = 0; i < 2; ++i) a.ks[i] = k_stride[i], a.vs[i] = v_stride[i];
    for (int i = 0; i < 3; ++i) a.kc[i] = k_cache_stride[i], a.vc[i] = v_cache_stride[i];
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_handle);
    const cudaError_t e = size == 4 ? (wide ? launch_store<float, 4>(a, k, v, k_cache, v_cache, stream)
                                            : launch_store<float, 1>(a, k, v, k_cache, v_cache, stream))
                                    : (wide ? launch_store<__half, 8>(a, k, v, k_cache, v_cache, stream)
                                            : launch_store<__half, 1>(a, k, v, k_cache, v_cache, stream));
    return llm_launched("spmv_paged_store launch", e);
}

}  // extern "C"
