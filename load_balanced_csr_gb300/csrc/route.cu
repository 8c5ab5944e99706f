// Routing tokens to experts: the transpose of the routing matrix (tokens by
// experts, top_k entries per row) by a stable counting sort, its product
// with the tokens' rows (dispatch), the weighted product back (combine) and
// the gradient of both.
//
//   build             slot = the stable rank of entry i = t * top_k + j by
//                     expert; entry = its inverse; expert_ptr = row pointers
//   dispatch          xs[slot(t, j)] = x[t]
//   combine           y[t] = sum_j w(t, j) ys[slot(t, j)]
//   combine_backward  dys[slot(t, j)] = w(t, j) dy[t],
//                     dw(t, j) = <dy[t], ys[slot(t, j)]>
//
// The rows' passes are bound by memory: each row of the experts' side is read
// or written once, and a token's own row once from memory.
#include <algorithm>

#include <cooperative_groups.h>

#include "llm.cuh"

namespace lbcsr {

namespace cg = cooperative_groups;

namespace {

// ---------------------------------------------------------------- build
// Bound by latency, not by its 20 bytes an entry: the ids are read once into
// registers, up to eight per thread, and ranked twice from there (counts per
// warp and expert, then positions).  Up to 131,072 entries are sorted by one
// launch of one cluster of up to 16 blocks, which read one another's counts
// in shared memory; more by two launches, the first of which counts.  On
// GB300: 512 entries of 128 experts 4.9 us alone (a launch and one block's
// trips to memory and between its barriers), 65,536 entries 9.0 us; with two
// launches and a tile per block 65,536 took 21 us, with clusters of 8 13.6.
constexpr int kBuildThreads = 1024;
constexpr int kBuildWarps = kBuildThreads / 32;
constexpr int kBuildKeys = 8;                               // ids of a thread at a time
constexpr int kBuildTile = kBuildThreads * kBuildKeys;      // entries of a block at a time
constexpr int kBuildCluster = 16;
constexpr int kMaxExperts = 2048;
constexpr int kMaxTiles = 152;                              // one tile per SM at most

bool build_clustered(int64_t n) { return n <= (int64_t)kBuildCluster * kBuildTile; }
// Entries of a block: in a cluster, spread over as many blocks as there are whole warps' loads for; else whole
// rounds of kBuildTile.
int64_t build_tile(int64_t n) {
    const int64_t blocks = build_clustered(n) ? kBuildCluster : kMaxTiles, step = build_clustered(n) ? kBuildThreads : kBuildTile;
    return std::max<int64_t>(step, (n + blocks * step - 1) / (blocks * step) * step);
}
int build_tiles(int64_t n) { return (int)std::max<int64_t>(1, (n + build_tile(n) - 1) / build_tile(n)); }

template <typename I>
__device__ __forceinline__ int key_of(const I *ids, int64_t ld, int k, int experts, int64_t i) {
    const I id = ld == k ? ids[i] : ids[(i / k) * ld + i % k];
    return id >= 0 && id < (I)experts ? (int)id : experts;  // the last bin: dropped
}

// The lanes whose key is this lane's, from one vote per bit of the keys
// (measured on 8,192 entries a block and 129 bins: the warp's match
// instruction takes about 210 clocks, more with more distinct keys; eight
// votes about 60).
__device__ __forceinline__ unsigned same_key(int key, int bits) {
    unsigned peers = 0xffffffffu;
    for (int b = 0; b < bits; b += 4) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const bool one = (key >> (b + u)) & 1;
            const unsigned vote = __ballot_sync(0xffffffffu, one);
            peers &= one ? vote : ~vote;
        }
    }
    return peers;
}

// hist[tile * (experts + 1) + bin]: entries of the tile in each bin
template <typename I>
__global__ void __launch_bounds__(kBuildThreads)
route_hist_kernel(const I *ids, int64_t ld, int k, int64_t n, int experts, int64_t tile, int32_t *hist) {
    extern __shared__ int32_t h[];
    after_previous();
    const int bins = experts + 1;
    for (int b = threadIdx.x; b < bins; b += kBuildThreads) h[b] = 0;
    __syncthreads();
    const int64_t t0 = (int64_t)blockIdx.x * tile, t1 = min(t0 + tile, n);
    constexpr int BATCH = 4;  // ids read together
    for (int64_t i0 = t0 + threadIdx.x; i0 < t1; i0 += BATCH * kBuildThreads) {
        int key[BATCH];
#pragma unroll
        for (int j = 0; j < BATCH; ++j)
            if (i0 + j * kBuildThreads < t1) key[j] = key_of(ids, ld, k, experts, i0 + j * kBuildThreads);
#pragma unroll
        for (int j = 0; j < BATCH; ++j)
            if (i0 + j * kBuildThreads < t1) atomicAdd(&h[key[j]], 1);
    }
    __syncthreads();
    for (int b = threadIdx.x; b < bins; b += kBuildThreads) hist[(int64_t)blockIdx.x * bins + b] = h[b];
}

// Positions of one tile.  Each warp owns a run of consecutive entries.
// counts[w][b]: the entries of bin b in warp w's run, then in the earlier
// warps' runs (a round has at most kBuildTile entries: 16 bits); base[b]: the
// position of the block's first entry in bin b, that is the bin's begin plus
// the earlier blocks' entries.  hist is null in a cluster.
template <typename I>
__global__ void __launch_bounds__(kBuildThreads)
route_rank_kernel(const I *ids, int64_t ld, int k, int64_t n, int experts, int64_t tile, int tiles, const int32_t *hist,
                  int32_t *expert_ptr, int32_t *entry, int32_t *slot) {
    extern __shared__ int32_t smem[];
    after_previous();
    __shared__ int32_t warp_sum[kBuildWarps];
    const int bins = experts + 1, bits = 32 - __clz(bins);  // keys, and `bins` for no entry
    int32_t *base = smem, *total = smem + bins, *sum = smem + 2 * bins;
    uint16_t *counts = reinterpret_cast<uint16_t *>(smem + 3 * bins);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned lt = (1u << lane) - 1u;
    const int64_t t0 = (int64_t)blockIdx.x * tile, t1 = min(t0 + tile, n);
    uint16_t *mine = counts + warp * bins;
    bool first = true;
    for (int64_t r0 = t0; first || r0 < t1; r0 += kBuildTile) {
        const int64_t r1 = min(r0 + kBuildTile, t1);
        // runs of whole multiples of 32, as short as the round allows
        const int run = (int)((max(r1 - r0, (int64_t)1) + kBuildThreads - 1) / kBuildThreads) * 32;
        const int64_t w0 = r0 + (int64_t)warp * run, w1 = min(w0 + run, r1);
        int key[kBuildKeys];
        unsigned peers[kBuildKeys];
#pragma unroll
        for (int j = 0; j < kBuildKeys; ++j) {
            const int64_t i = w0 + j * 32 + lane;
            key[j] = i < w1 ? key_of(ids, ld, k, experts, i) : bins;
        }
        for (int b = lane; b < bins; b += 32) mine[b] = 0;
        __syncwarp();
#pragma unroll
        for (int j = 0; j < kBuildKeys; ++j) {
            if (w0 + j * 32 >= w1) break;
            peers[j] = same_key(key[j], bits);
            if (key[j] < bins && lane == __ffs(peers[j]) - 1) mine[key[j]] += __popc(peers[j]);
            __syncwarp();
        }
        __syncthreads();
        for (int b = threadIdx.x; b < bins; b += kBuildThreads) {
            int32_t before = 0;
#pragma unroll 16
            for (int w = 0; w < kBuildWarps; ++w) {
                const int32_t c = counts[w * bins + b];
                counts[w * bins + b] = (uint16_t)before;
                before += c;
            }
            total[b] = before;
            if (first) base[b] = 0, sum[b] = 0;
        }
        if (first) {
            // base: the earlier blocks' entries of each bin; sum: all blocks'
            __syncthreads();
            if (hist) {
                constexpr int PER = (kMaxTiles + kBuildWarps - 1) / kBuildWarps;  // tiles of a warp
                for (int b = lane; b < bins; b += 32) {
                    int32_t c[PER], all = 0, before = 0;
#pragma unroll
                    for (int j = 0; j < PER; ++j) {
                        const int t = warp + j * kBuildWarps;
                        c[j] = t < tiles ? hist[(int64_t)t * bins + b] : 0;
                    }
#pragma unroll
                    for (int j = 0; j < PER; ++j) {
                        all += c[j];
                        if (warp + j * kBuildWarps < (int)blockIdx.x) before += c[j];
                    }
                    atomicAdd(sum + b, all);
                    atomicAdd(base + b, before);
                }
                __syncthreads();
            } else {
                cg::cluster_group cluster = cg::this_cluster();
                cluster.sync();
                for (int b = threadIdx.x; b < bins; b += kBuildThreads) {
                    int32_t all = 0, before = 0;
#pragma unroll
                    for (int t = 0; t < kBuildCluster; ++t) {
                        const int32_t c = t < tiles ? *cluster.map_shared_rank(total + b, t) : 0;
                        all += c;
                        if (t < blockIdx.x) before += c;
                    }
                    sum[b] = all, base[b] = before;
                }
                __syncthreads();
            }
            // plus each bin's begin: an exclusive prefix sum of `sum`, bins in blocks of one per thread
            int32_t carry = 0;
            for (int b0 = 0; b0 < bins; b0 += kBuildThreads) {
                const int b = b0 + threadIdx.x;
                const int32_t own = b < bins ? sum[b] : 0;
                int32_t scan = own;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int32_t up = __shfl_up_sync(0xffffffffu, scan, d);
                    if (lane >= d) scan += up;
                }
                if (lane == 31) warp_sum[warp] = scan;
                __syncthreads();
                int32_t before = lane < warp ? warp_sum[lane] : 0, all = warp_sum[lane];
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) {
                    before += __shfl_xor_sync(0xffffffffu, before, d);
                    all += __shfl_xor_sync(0xffffffffu, all, d);
                }
                const int32_t begin = carry + before + scan - own;
                carry += all;
                if (b < bins) {
                    base[b] += begin;
                    if (blockIdx.x == 0) expert_ptr[b] = begin;  // bin `experts` begins where the experts end
                }
                __syncthreads();
            }
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kBuildKeys; ++j) {
            if (w0 + j * 32 >= w1) break;
            if (key[j] < bins) {
                const int32_t p = base[key[j]] + mine[key[j]] + __popc(peers[j] & lt);
                const int64_t i = w0 + j * 32 + lane;
                entry[p] = (int32_t)i;
                slot[i] = key[j] < experts ? p : -1 - p;
            }
            __syncwarp();
            if (key[j] < bins && lane == __ffs(peers[j]) - 1) mine[key[j]] += __popc(peers[j]);
            __syncwarp();
        }
        if (r0 + kBuildTile < t1) {  // the next round goes on behind this one
            __syncthreads();
            for (int b = threadIdx.x; b < bins; b += kBuildThreads) base[b] += total[b];
            __syncthreads();
        }
        first = false;
    }
    // a block's counts stay until the others have read them
    if (!hist) cg::this_cluster().sync();
}

template <typename I>
cudaError_t launch_build(int64_t n, int k, int experts, const I *ids, int64_t ld, int32_t *expert_ptr, int32_t *entry,
                         int32_t *slot, int32_t *hist, cudaStream_t stream) {
    const int64_t tile = build_tile(n);
    const int tiles = build_tiles(n);
    constexpr int per_bin = 3 * 4 + kBuildWarps * 2;
    const size_t bins = (size_t)experts + 1, smem = bins * per_bin;
    if (smem > 47 * 1024) {
        // the function's limit is every host thread's: the most that any call needs, not this one
        const cudaError_t e = cudaFuncSetAttribute(route_rank_kernel<I>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (kMaxExperts + 1) * per_bin);
        if (e != cudaSuccess) return e;
    }
    const bool clustered = build_clustered(n);
    if (tiles > 8 && clustered) {  // more blocks than every device's clusters may have
        const cudaError_t e = cudaFuncSetAttribute(route_rank_kernel<I>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
    }
    if (!clustered) {
        const cudaError_t e = launch_chained(route_hist_kernel<I>, tiles, kBuildThreads, bins * 4, 0, stream, ids, ld, k, n,
                                             experts, tile, hist);
        if (e != cudaSuccess) return e;
    }
    return launch_chained(route_rank_kernel<I>, tiles, kBuildThreads, smem, clustered ? tiles : 0, stream, ids, ld, k, n,
                          experts, tile, tiles, clustered ? nullptr : hist, expert_ptr, entry, slot);
}

// ---------------------------------------------------------------- rows
constexpr int kRowThreads = 256;

// Dispatch and combine: one warp per (token, span of 32 * U vectors of its
// row).  A token's row is read (written) once and stays in registers while
// its top_k rows of the experts' side are written (read), each 16 bytes a
// lane; no sharing between warps, so nothing waits but for memory.  With
// 8,192 tokens, 8 choices and rows of 4,096 bf16 (604 MB) dispatch takes
// 91.9 us and combine 89.9: 6.57 and 6.72 TB/s, 0.98 and 1.00 of the measured
// copy; with 16,384 tokens and 2 choices (403 MB) 59.7 and 61.5 us.  Rows off
// 16-byte boundaries go element by element: 2,999 tokens, 6 choices, 1,001
// floats (84 MB) 13.5 and 10.7 us.
struct RowArgs {
    int64_t items;   // tokens * spans
    int32_t spans;
    int32_t k;
    int32_t vecs;    // vectors in a row
    const int32_t *slot;
    const float *w;
    int64_t ldw;
};

template <typename T, int N, int U>
__global__ void __launch_bounds__(kRowThreads)
route_dispatch_kernel(RowArgs a, const T *x, int64_t ldx, T *xs, int64_t ldxs) {
    using V = Vec<T, N>;
    after_previous();
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
    if (item >= a.items) return;
    const int64_t t = item / a.spans;
    const int v0 = (int)(item % a.spans) * (32 * U) + lane;
    const V *src = reinterpret_cast<const V *>(x + t * ldx);
    V row[U], none;
#pragma unroll
    for (int n = 0; n < N; ++n) none.v[n] = zero_of<T>();
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (v0 + 32 * u < a.vecs) row[u] = src[v0 + 32 * u];
    constexpr int BATCH = 4;  // slots read together
    for (int j0 = 0; j0 < a.k; j0 += BATCH) {
        int32_t p[BATCH];
#pragma unroll
        for (int j = 0; j < BATCH; ++j) p[j] = j0 + j < a.k ? a.slot[t * a.k + j0 + j] : 0;
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
            if (j0 + j >= a.k) break;
            V *dst = reinterpret_cast<V *>(xs + (int64_t)(p[j] < 0 ? -1 - p[j] : p[j]) * ldxs);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (v0 + 32 * u < a.vecs) dst[v0 + 32 * u] = p[j] < 0 ? none : row[u];
        }
    }
}

template <typename T, int N, int U>
__global__ void __launch_bounds__(kRowThreads)
route_combine_kernel(RowArgs a, const T *ys, int64_t ldys, T *y, int64_t ldy) {
    using V = Vec<T, N>;
    after_previous();
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
    if (item >= a.items) return;
    const int64_t t = item / a.spans;
    const int v0 = (int)(item % a.spans) * (32 * U) + lane;
    float sum[U][N];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int n = 0; n < N; ++n) sum[u][n] = 0.0f;
    if constexpr (U == 1) {
        // few or short rows: what counts is that the choices' rows are on their way together
        constexpr int BATCH = 4;
        for (int j0 = 0; j0 < a.k; j0 += BATCH) {
            int32_t p[BATCH];
            float w[BATCH];
            V r[BATCH];
#pragma unroll
            for (int j = 0; j < BATCH; ++j) {
                const bool in = j0 + j < a.k;
                p[j] = in ? a.slot[t * a.k + j0 + j] : -1;
                w[j] = in && a.w ? a.w[t * a.ldw + j0 + j] : 1.0f;
            }
#pragma unroll
            for (int j = 0; j < BATCH; ++j)
                if (p[j] >= 0 && v0 < a.vecs) r[j] = reinterpret_cast<const V *>(ys + (int64_t)p[j] * ldys)[v0];
#pragma unroll
            for (int j = 0; j < BATCH; ++j)
                if (p[j] >= 0 && v0 < a.vecs)
#pragma unroll
                    for (int n = 0; n < N; ++n) sum[0][n] = fmaf(w[j], to_float(r[j].v[n]), sum[0][n]);
        }
    } else {
        for (int j0 = 0; j0 < a.k; j0 += 32) {
            // the choices' slots and weights, one a lane, read together before the rows that they point to (a slot
            // read before each row: 101.9 us for the 8,192 tokens, 89.9 so)
            const bool in = j0 + lane < a.k;
            const int32_t ps = in ? a.slot[t * a.k + j0 + lane] : -1;
            const float ws = in && a.w ? a.w[t * a.ldw + j0 + lane] : 1.0f;
            const int choices = min(32, a.k - j0);
#pragma unroll 4
            for (int j = 0; j < choices; ++j) {
                const int32_t p = __shfl_sync(0xffffffffu, ps, j);
                const float w = __shfl_sync(0xffffffffu, ws, j);
                if (p < 0) continue;
                const V *src = reinterpret_cast<const V *>(ys + (int64_t)p * ldys);
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (v0 + 32 * u < a.vecs) {
                        const V r = src[v0 + 32 * u];
#pragma unroll
                        for (int n = 0; n < N; ++n) sum[u][n] = fmaf(w, to_float(r.v[n]), sum[u][n]);
                    }
            }
        }
    }
    V *dst = reinterpret_cast<V *>(y + t * ldy);
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (v0 + 32 * u < a.vecs) {
            V r;
#pragma unroll
            for (int n = 0; n < N; ++n) r.v[n] = from_float<T>(sum[u][n]);
            dst[v0 + 32 * u] = r;
        }
}

// A warp per entry (token, choice): it reads dy's and its expert row, writes
// its gradient row, and sums its dot product over its lanes.  The choices of
// a token are neighbouring warps, so dy's row comes from memory once and from
// L1 for the others.  With rows of 4,096 bf16: 16,384 tokens, 2 choices
// (671 MB) 99.8 us, 8,192 tokens, 8 choices (1,141 MB) 176 us: 6.7 and 6.5
// TB/s, 1.00 and 0.97 of the measured copy.  A block per token with dy's row
// in registers for all choices needed 130-170 registers, so few warps fit, and
// took 118 and 247 us.
template <typename T, int N, int U>
__global__ void __launch_bounds__(kRowThreads)
route_combine_backward_kernel(RowArgs a, const T *dy, int64_t lddy, const T *ys, int64_t ldys, T *dys, int64_t lddys,
                              float *dw, int64_t lddw) {
    using V = Vec<T, N>;
    after_previous();
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
    if (item >= a.items) return;
    const int64_t t = item / a.k;
    const int j = (int)(item - t * a.k);
    const int32_t p = a.slot[item];
    const float w = a.w ? a.w[t * a.ldw + j] : 1.0f;
    const V *g = reinterpret_cast<const V *>(dy + t * lddy);
    V *to = reinterpret_cast<V *>(dys + (int64_t)(p < 0 ? -1 - p : p) * lddys);
    if (p < 0) {
        V none;
#pragma unroll
        for (int n = 0; n < N; ++n) none.v[n] = zero_of<T>();
        for (int v = lane; v < a.vecs; v += 32) to[v] = none;
        if (dw && lane == 0) dw[t * lddw + j] = 0.0f;
        return;
    }
    const V *y = reinterpret_cast<const V *>(ys + (int64_t)p * ldys);
    // eight sums a lane: as one or two, a long row's were off by up to half as many units of the last place as they have terms
    constexpr int CHAINS = 8;
    float dot[CHAINS] = {};
    for (int v0 = lane; v0 < a.vecs; v0 += 32 * U) {
        V gv[U], yv[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (v0 + 32 * u < a.vecs) {
                if (dw) yv[u] = y[v0 + 32 * u];
                gv[u] = g[v0 + 32 * u];
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (v0 + 32 * u < a.vecs) {
                V r;
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    const float gf = to_float(gv[u].v[n]);
                    float &sum = dot[(u * N + n) % CHAINS];
                    if (dw) sum = fmaf(gf, to_float(yv[u].v[n]), sum);
                    r.v[n] = from_float<T>(w * gf);
                }
                to[v0 + 32 * u] = r;
            }
    }
    if (dw) {
#pragma unroll
        for (int c = CHAINS / 2; c > 0; c /= 2)
#pragma unroll
            for (int i = 0; i < c; ++i) dot[i] += dot[i + c];
        float d = dot[0];
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) d += __shfl_xor_sync(0xffffffffu, d, s);
        if (lane == 0) dw[t * lddw + j] = d;
    }
}

RowArgs row_args(int32_t tokens, int32_t k, int32_t hidden, int n, int u, const int32_t *slot, const float *w,
                 int64_t ldw) {
    RowArgs a;
    a.vecs = hidden / n;
    a.spans = (a.vecs + 32 * u - 1) / (32 * u);
    a.items = (int64_t)tokens * a.spans;
    a.k = k;
    a.slot = slot;
    a.w = w;
    a.ldw = ldw;
    return a;
}

unsigned row_blocks(const RowArgs &a) { return (unsigned)((a.items + kRowThreads / 32 - 1) / (kRowThreads / 32)); }

// A warp's span: with many rows, enough vectors per lane to keep the memory
// busy; with few (less than a vector for each of 64 warps an SM), one, so that
// the rows spread over the SMs: 64 tokens of 2,048 bf16 and 8 choices take
// 3.3 us by dispatch and 4.6 by combine, 5.1 and 7.6 with the large span; many
// rows with the small span 130 us instead of 63 (16,384 tokens, combine).
// Rows of one vector a lane have the small span anyway: 16,384 tokens, 8
// choices, 256 bf16 are combined in 10.7 us, 20.0 with the large one.
bool few_rows(int32_t tokens, int32_t hidden, int n) { return (int64_t)tokens * (hidden / n) < 152 * 64 * 32; }

template <typename T, int N, int U>
cudaError_t launch_dispatch_u(int32_t tokens, int32_t k, int32_t hidden, const int32_t *slot, const void *x, int64_t ldx,
                              void *xs, int64_t ldxs, cudaStream_t stream) {
    const RowArgs a = row_args(tokens, k, hidden, N, U, slot, nullptr, 0);
    return launch_chained(route_dispatch_kernel<T, N, U>, row_blocks(a), kRowThreads, 0, 0, stream, a,
                          static_cast<const T *>(x), ldx, static_cast<T *>(xs), ldxs);
}
template <typename T, int N>
cudaError_t launch_dispatch(int32_t tokens, int32_t k, int32_t hidden, const int32_t *slot, const void *x, int64_t ldx,
                            void *xs, int64_t ldxs, cudaStream_t stream) {
    return few_rows(tokens, hidden, N) ? launch_dispatch_u<T, N, 1>(tokens, k, hidden, slot, x, ldx, xs, ldxs, stream)
                                       : launch_dispatch_u<T, N, (N == 1 ? 8 : 4)>(tokens, k, hidden, slot, x, ldx, xs, ldxs, stream);
}

template <typename T, int N, int U>
cudaError_t launch_combine_u(int32_t tokens, int32_t k, int32_t hidden, const int32_t *slot, const float *w, int64_t ldw,
                             const void *ys, int64_t ldys, void *y, int64_t ldy, cudaStream_t stream) {
    const RowArgs a = row_args(tokens, k, hidden, N, U, slot, w, ldw);
    return launch_chained(route_combine_kernel<T, N, U>, row_blocks(a), kRowThreads, 0, 0, stream, a,
                          static_cast<const T *>(ys), ldys, static_cast<T *>(y), ldy);
}
template <typename T, int N>
cudaError_t launch_combine(int32_t tokens, int32_t k, int32_t hidden, const int32_t *slot, const float *w, int64_t ldw,
                           const void *ys, int64_t ldys, void *y, int64_t ldy, cudaStream_t stream) {
    return few_rows(tokens, hidden, N) || hidden / N <= 32 ? launch_combine_u<T, N, 1>(tokens, k, hidden, slot, w, ldw, ys, ldys, y, ldy, stream)
                                       : launch_combine_u<T, N, 4>(tokens, k, hidden, slot, w, ldw, ys, ldys, y, ldy, stream);
}

template <typename T, int N>
cudaError_t launch_combine_backward(int32_t tokens, int32_t k, int32_t hidden, const int32_t *slot, const float *w,
                                    int64_t ldw, const void *dy, int64_t lddy, const void *ys, int64_t ldys, void *dys,
                                    int64_t lddys, float *dw, int64_t lddw, cudaStream_t stream) {
    constexpr int U = N == 1 ? 8 : 2;
    RowArgs a = row_args(tokens, k, hidden, N, U, slot, w, ldw);
    a.items = (int64_t)tokens * k;
    return launch_chained(route_combine_backward_kernel<T, N, U>, row_blocks(a), kRowThreads, 0, 0, stream, a,
                          static_cast<const T *>(dy), lddy, static_cast<const T *>(ys), ldys, static_cast<T *>(dys), lddys,
                          dw, lddw);
}

// Rows whose addresses all fall on 16 bytes move in 16-byte vectors, others
// element by element.
bool rows_wide(int64_t hidden, int size, std::initializer_list<std::pair<const void *, int64_t>> rows) {
    if (hidden * size % 16) return false;
    for (const auto &r : rows)
        if (!aligned_to(r.first, 16) || r.second * size % 16) return false;
    return true;
}

// `size`-byte elements only (dispatch copies whatever they hold)
#define ROUTE_BY_SIZE(size, wide, F, ...)                                                     \
    ((size) == 4 ? ((wide) ? F<float, 4>(__VA_ARGS__) : F<float, 1>(__VA_ARGS__))             \
                 : ((wide) ? F<__half, 8>(__VA_ARGS__) : F<__half, 1>(__VA_ARGS__)))
#define ROUTE_BY_ELEM(elem, wide, F, ...)                                                                   \
    ((elem) == SPMV_ELEM_F32    ? ((wide) ? F<float, 4>(__VA_ARGS__) : F<float, 1>(__VA_ARGS__))            \
     : (elem) == SPMV_ELEM_BF16 ? ((wide) ? F<__nv_bfloat16, 8>(__VA_ARGS__) : F<__nv_bfloat16, 1>(__VA_ARGS__)) \
                                : ((wide) ? F<__half, 8>(__VA_ARGS__) : F<__half, 1>(__VA_ARGS__)))

// The checks the rows' passes share; null: they hold.
const char *rows_bad(int32_t tokens, int32_t top_k, int32_t hidden, int elem) {
    if (tokens < 0 || top_k < 0 || hidden < 0) return "negative size";
    if ((int64_t)tokens * top_k >= (1LL << 31)) return "tokens * top_k must be < 2^31";
    if (!elem_ok(elem)) return "unknown element type";
    // a lane's place in a row, up to 32 * 8 elements of its last turn past the end, is counted in 32 bits
    if (hidden >= INT32_MAX - 1023) return "hidden must be < 2^31 - 1024";
    // the passes' grids: eight warps a block, each of at least 32 elements of a token or of one of its entries
    if ((int64_t)tokens * ((hidden + 31) / 32) / 8 >= (1LL << 31) - 1) return "tokens * hidden is too large";
    return nullptr;
}

}  // namespace

}  // namespace lbcsr

using namespace lbcsr;

extern "C" {

spmv_status_t spmv_route_workspace(int32_t tokens, int32_t top_k, int32_t experts, size_t *bytes) {
    if (!bytes) return llm_bad("bytes is NULL");
    *bytes = 0;
    if (tokens < 0 || top_k < 0) return llm_bad("negative size");
    if (experts < 1 || experts > kMaxExperts) return llm_bad("experts must be in [1, 2048]");
    const int64_t n = (int64_t)tokens * top_k;
    if (n >= (1LL << 31)) return llm_bad("tokens * top_k must be < 2^31");
    // never below build_tiles of fewer entries, whose tiles may be smaller and more (152 of 1,245,184 entries, 77 of one more)
    *bytes = build_clustered(n) ? 0 : (size_t)std::min<int64_t>(kMaxTiles, (n + kBuildTile - 1) / kBuildTile) * (experts + 1) * 4;
    return SPMV_OK;
}

spmv_status_t spmv_route_build(int32_t tokens, int32_t top_k, int32_t experts, const void *expert_ids,
                               int32_t id_bytes, int64_t ld_ids, int32_t *expert_ptr, int32_t *entry, int32_t *slot,
                               void *workspace, size_t workspace_bytes, spmv_stream_t stream_handle) {
    size_t need = 0;
    const spmv_status_t st = spmv_route_workspace(tokens, top_k, experts, &need);
    if (st != SPMV_OK) return st;
    const int64_t n = (int64_t)tokens * top_k;
    if (id_bytes != 4 && id_bytes != 8) return llm_bad("id_bytes must be 4 or 8");
    if (!expert_ptr) return llm_bad("expert_ptr is NULL");
    if (n > 0 && (!expert_ids || !entry || !slot)) return llm_bad("expert_ids, entry or slot is NULL");
    if (!aligned_to(expert_ids, id_bytes)) return llm_bad("expert_ids is not aligned to its type");
    if (need && (!workspace || workspace_bytes < need || !aligned_to(workspace, 16)))
        return llm_bad("workspace is NULL, too small or not 16-byte aligned");
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_handle);
    int32_t *hist = static_cast<int32_t *>(workspace);
    const cudaError_t e =
        id_bytes == 8 ? launch_build(n, top_k, experts, static_cast<const int64_t *>(expert_ids), ld_ids, expert_ptr,
                                     entry, slot, hist, stream)
                      : launch_build(n, top_k, experts, static_cast<const int32_t *>(expert_ids), ld_ids, expert_ptr,
                                     entry, slot, hist, stream);
    return llm_launched("spmv_route_build launch", e);
}

spmv_status_t spmv_route_dispatch(int32_t tokens, int32_t top_k, int32_t hidden, spmv_elem_t elem,
                                  const int32_t *slot, const void *x, int64_t ldx, void *xs, int64_t ldxs,
                                  spmv_stream_t stream_handle) {
    if (const char *bad = rows_bad(tokens, top_k, hidden, elem)) return llm_bad(bad);
    if (tokens == 0 || top_k == 0 || hidden == 0) return SPMV_OK;
    if (!slot || !x || !xs) return llm_bad("slot, x or xs is NULL");
    if (ldxs < hidden) return llm_bad("ldxs is smaller than hidden");
    const int size = elem_size(elem);
    if (!aligned_to(x, size) || !aligned_to(xs, size)) return llm_bad("x or xs is not aligned to its type");
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_handle);
    const bool wide = rows_wide(hidden, size, {{x, ldx}, {xs, ldxs}});
    return llm_launched("spmv_route_dispatch launch",
                        ROUTE_BY_SIZE(size, wide, launch_dispatch, tokens, top_k, hidden, slot, x, ldx, xs, ldxs, stream));
}

spmv_status_t spmv_route_combine(int32_t tokens, int32_t top_k, int32_t hidden, spmv_elem_t elem,
                                 const int32_t *slot, const float *weights, int64_t ldw, const void *ys,
                                 int64_t ldys, void *y, int64_t ldy, spmv_stream_t stream_handle) {
    if (const char *bad = rows_bad(tokens, top_k, hidden, elem)) return llm_bad(bad);
    if (tokens == 0 || hidden == 0) return SPMV_OK;
    if (!y || (top_k > 0 && (!slot || !ys))) return llm_bad("slot, ys or y is NULL");
    if (ldy < hidden) return llm_bad("ldy is smaller than hidden");
    const int size = elem_size(elem);
    if (!aligned_to(ys, size) || !aligned_to(y, size)) return llm_bad("ys or y is not aligned to its type");
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_handle);
    const bool wide = rows_wide(hidden, size, {{ys, ldys}, {y, ldy}});
    return llm_launched("spmv_route_combine launch", ROUTE_BY_ELEM(elem, wide, launch_combine, tokens, top_k, hidden, slot,
                                                                   weights, ldw, ys, ldys, y, ldy, stream));
}

spmv_status_t spmv_route_combine_backward(int32_t tokens, int32_t top_k, int32_t hidden, spmv_elem_t elem,
                                          const int32_t *slot, const float *weights, int64_t ldw, const void *dy,
                                          int64_t lddy, const void *ys, int64_t ldys, void *dys, int64_t lddys,
                                          float *dweights, int64_t lddw, spmv_stream_t stream_handle) {
    if (const char *bad = rows_bad(tokens, top_k, hidden, elem)) return llm_bad(bad);
    if (tokens == 0 || top_k == 0) return SPMV_OK;
    if (!slot || (hidden > 0 && (!dy || !dys))) return llm_bad("slot, dy or dys is NULL");
    if (dweights && hidden > 0 && !ys) return llm_bad("ys is NULL");
    if (lddys < hidden) return llm_bad("lddys is smaller than hidden");
    if (dweights && lddw < top_k) return llm_bad("lddw is smaller than top_k");
    const int size = elem_size(elem);
    if (!aligned_to(dy, size) || !aligned_to(ys, size) || !aligned_to(dys, size))
        return llm_bad("dy, ys or dys is not aligned to its type");
    if (ys && ys == dys && ldys != lddys) return llm_bad("dys may be ys only with the same row stride");
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_handle);
    const bool wide = rows_wide(hidden, size, {{dy, lddy}, {ys, dweights ? ldys : 0}, {dys, lddys}});
    return llm_launched("spmv_route_combine_backward launch",
                        ROUTE_BY_ELEM(elem, wide, launch_combine_backward, tokens, top_k, hidden, slot, weights, ldw, dy,
                                      lddy, ys, ldys, dys, lddys, dweights, lddw, stream));
}

}  // extern "C"
