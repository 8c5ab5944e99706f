// Quantising stores into a paged cache of 8-bit codes, and reading a paged
// cache back.
//
// spmv_paged_store_e4m3: a block of tokens of one page and a head share a
// scale, the least power of two p with every finite |x| <= 448 p.  A power of
// two makes x / p exact, so a code is one rounding, and a block whose scale
// grows when more tokens come keeps its codes' values: code * old / new is
// exact until it is subnormal.  The tokens of one block that a call writes are
// neighbours in `slots` (a run); a warp takes one run of one head, of keys or
// of values: their rows into registers, the largest, the scale, the codes.
// A tile's runs are listed once, by votes.  With a scale per token a row is a
// run, and several rows share a warp.  65,504 tokens of 8 heads of 128 f16 (383
// MB) 72 us: 5.3 TB/s, bound by instructions (0.59 of the issue slots) and the
// trips of a run's chain together; so the usual run, all of it in registers
// and finite, has code of its own without other cases (98 us with them in the
// loops).
//
// spmv_paged_load: the same rows the other way, code * scale rounded once; a
// block looks up its tokens' slots first (token_ptr by binary search in
// shared memory), then moves 16 codes of keys and of values a thread: 139,000
// positions of 8 heads of 128 (856 MB) 146 us, 5.9 TB/s; with two vectors of
// each 175 us, for fewer warps fit.
#include <algorithm>
#include <type_traits>

#include "e4m3.cuh"
#include "internal.cuh"
#include "llm.cuh"

namespace lbcsr {

namespace {

constexpr int kMaxBlock = 64;  // tokens of a scale: a run's slots are 64 bits
constexpr int kCodeThreads = 256, kCodeWarps = kCodeThreads / 32;
constexpr int kTile = 32;      // tokens of a tile (64: 73 us instead of 72 below)
// Tokens of one block that are further apart in `slots` are not looked for: a
// long tail of skipped ones would be read to its end.
constexpr int kMaxGap = 64;

__device__ __forceinline__ uint32_t over(uint32_t t, uint32_t mul, uint32_t shift) {
    return (uint32_t)(((unsigned long long)__umulhi(t, mul) + t) >> shift);
}

struct Side {  // of keys, or of values
    const void *x;
    unsigned char *codes;
    float *scales;
    int64_t xs[2], cs[3], ss[3];  // token, head; page, position, head; page, block, head
};

struct StoreCodesArgs {
    Side side[2];
    int32_t tokens, heads, dim, num_pages, page, block, slices;
    uint32_t page_mul, page_shift, block_mul, block_shift, heads_mul, heads_shift;
    const int32_t *slots;
};

// ---------------------------------------------------------------- values and codes
// V neighbouring elements, held as they are read.
template <typename T, int V>
struct Raw {
    static constexpr int N = V == 1 ? 1 : 16 / sizeof(T);
    Vec<T, N> part[V / N];
    __device__ __forceinline__ void read(const T *at) {
#pragma unroll
        for (int i = 0; i < V / N; ++i) part[i] = reinterpret_cast<const Vec<T, N> *>(at)[i];
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < V; ++i) part[i / N].v[i % N] = zero_of<T>();
    }
    __device__ __forceinline__ float operator[](int i) const { return to_float(part[i / N].v[i % N]); }
};

// What the first pass over some elements finds: the bits of the largest finite |x|, and whether one is not finite.
struct Size {
    uint32_t bits;
    bool odd;
};
template <typename T, int V>
__device__ __forceinline__ void look(const Raw<T, V> &x, Size &s) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const uint32_t bits = __float_as_uint(x[i]) & 0x7fffffffu;
        if (bits < 0x7f800000u) s.bits = max(s.bits, bits);
        else s.odd = true;
    }
}
// 16-bit elements in pairs: their bits without the sign are in the order of their sizes
template <typename T>
__device__ __forceinline__ void look_pairs(const Raw<T, 8> &x, uint32_t &top) {
    static_assert(sizeof(T) == 2, "");
    uint4 w;
    memcpy(&w, &x, 16);
    top = __vmaxu2(top, __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu), __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu)));
}
// the least power of two p >= 2^-126 with size <= 448 p = 1.75 * 2^8 p
__device__ __forceinline__ float scale_for(uint32_t size_bits) {
    const int e = (int)(size_bits >> 23) - 8 + ((size_bits & 0x7fffffu) > 0x600000u);  // biased
    return __uint_as_float((uint32_t)max(e, 1) << 23);
}
// x / scale; a NaN stands for what is not finite.  PLAIN: the scale is a power of two, whose reciprocal is exact, and x
// is finite.
struct Divide {
    float scale, inverse;
    bool plain;
};
__device__ __forceinline__ Divide divide_by(float scale, bool odd) {
    return {scale, 1.0f / scale, !odd && (__float_as_uint(scale) & 0x7fffffu) == 0 && scale <= __uint_as_float(253u << 23)};
}
template <bool PLAIN>
__device__ __forceinline__ float divided(float x, const Divide &by) {
    if (PLAIN) return x * by.inverse;
    return (__float_as_uint(x) & 0x7f800000u) != 0x7f800000u ? x / by.scale : __int_as_float(0x7fffffff);
}
template <bool PLAIN, typename T, int V>
__device__ __forceinline__ void write_codes(unsigned char *to, const Raw<T, V> &x, const Divide &by) {
    auto q = [&](int i) { return divided<PLAIN>(x[i], by); };
    if constexpr (V == 1) {
        *to = (unsigned char)to_e4m3x2(q(0), 0.0f);
    } else {
        static_assert(V == 8, "");
        uint2 c;
        c.x = to_e4m3x2(q(0), q(1)) | to_e4m3x2(q(2), q(3)) << 16;
        c.y = to_e4m3x2(q(4), q(5)) | to_e4m3x2(q(6), q(7)) << 16;
        *reinterpret_cast<uint2 *>(to) = c;
    }
}
template <int V>
__device__ __forceinline__ void rescale_codes(unsigned char *at, float by) {
    if constexpr (V == 1) {
        *at = (unsigned char)to_e4m3x2(from_e4m3x2(*at).x * by, 0.0f);
    } else {
        uint2 c = *reinterpret_cast<const uint2 *>(at);
        auto again = [&](uint32_t w) {
            const float2 a = from_e4m3x2(w & 0xffffu), b = from_e4m3x2(w >> 16);
            return to_e4m3x2(a.x * by, a.y * by) | to_e4m3x2(b.x * by, b.y * by) << 16;
        };
        c.x = again(c.x), c.y = again(c.y);
        *reinterpret_cast<uint2 *>(at) = c;
    }
}

// ---------------------------------------------------------------- store, blocks of tokens
// A run of a tile: its tokens are entries first .. first + count - 1 of the tile's list.
struct Run {
    int32_t block, first, count;
};
constexpr int kListed = kTile + kMaxBlock;  // the tile's tokens, and those behind it of its last run

// L lanes take a row, 32 / L rows go at once; HELD batches of these stay in
// registers between the two passes.
template <typename T, int V, int L>
__global__ void __launch_bounds__(kCodeThreads, 4) paged_store_blocks_kernel(StoreCodesArgs a) {
    constexpr int G = 32 / L, HELD = sizeof(T) == 4 ? 2 : 8;
    __shared__ Run runs[kTile];
    __shared__ int num_runs;
    __shared__ int32_t token_of[kListed];
    __shared__ uint8_t place_of[kListed];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    after_previous();
    const uint32_t cache_slots = (uint32_t)a.num_pages * (uint32_t)a.page;
    const int64_t t0 = (int64_t)(blockIdx.x / a.slices) * kTile;
    const int slice = blockIdx.x % a.slices;
    if (warp == 0) {
        // a token's slot and the block of tokens that it goes to, or -1
        auto read = [&](int64_t i, int32_t &slot) {
            slot = i >= 0 && i < a.tokens ? a.slots[i] : -1;
            return (uint32_t)slot < cache_slots ? (int32_t)over((uint32_t)slot, a.block_mul, a.block_shift) : -1;
        };
        int before = -1;  // of the last token before these that goes anywhere
        int64_t before_at = 0;
        int32_t slot;
        for (int64_t i = t0 - 1; i >= t0 - kMaxGap && before < 0; i -= 32) {
            const int b = read(i - lane, slot);
            const uint32_t any = __ballot_sync(0xffffffffu, b >= 0);
            if (any) before = __shfl_sync(0xffffffffu, b, __ffs(any) - 1), before_at = i - (__ffs(any) - 1);
        }
        int n = 0, listed = 0;  // runs; tokens of them
        const uint32_t under_me = (1u << lane) - 1;
        for (int64_t i0 = t0;; i0 += 32) {
            const bool inside = i0 < t0 + kTile;  // behind the tile: the last run's tokens alone
            const int64_t i = i0 + lane;
            const int b = inside && i >= t0 + kTile ? -1 : read(i, slot);
            const uint32_t there = __ballot_sync(0xffffffffu, b >= 0), under = there & under_me;
            const int last = __shfl_sync(0xffffffffu, b, under ? 31 - __clz(under) : 0);
            const bool opens = b >= 0 && (under ? b != last : b != before || i - before_at > kMaxGap);
            uint32_t opened = __ballot_sync(0xffffffffu, opens), mine = there;
            if (!inside) {
                if (n == 0) break;
                mine &= opened ? (1u << (__ffs(opened) - 1)) - 1 : 0xffffffffu;
            } else if (n == 0) {  // tokens before the first run are of the tile's before
                mine &= opened ? ~((1u << (__ffs(opened) - 1)) - 1) : 0u;
            }
            const int at = listed + __popc(mine & under_me);
            if ((mine >> lane & 1) && at < kListed) {  // slots that tokens share could be more
                token_of[at] = (int32_t)i, place_of[at] = (uint8_t)(slot - b * a.block);
                if (inside && opens) runs[n + __popc(opened & under_me)] = Run{b, at, 0};
            }
            if (inside) n += __popc(opened);
            listed = min(listed + __popc(mine), kListed);
            if (!inside && (opened || (there ? false : i0 + 31 - before_at >= kMaxGap) || i0 + 32 >= a.tokens || listed == kListed)) break;
            if (there) {
                before = __shfl_sync(0xffffffffu, b, 31 - __clz(there));
                before_at = i0 + 31 - __clz(there);
            } else if (inside && i0 + 32 >= t0 + kTile && i0 + 31 - before_at >= kMaxGap) {
                break;
            }
            if (i0 + 32 >= a.tokens) break;
        }
        __syncwarp();
        for (int r = lane; r < n; r += 32) runs[r].count = min((r + 1 < n ? runs[r + 1].first : listed) - runs[r].first, a.block);
        if (lane == 0) num_runs = n;
    }
    __syncthreads();
    const int vecs = a.dim / V, sub = lane / L, col = lane % L;
    const int tasks = num_runs * 2 * a.heads;
    for (int task = slice * kCodeWarps + warp; task < tasks; task += a.slices * kCodeWarps) {
        const int of = (int)over((uint32_t)task >> 1, a.heads_mul, a.heads_shift), head = (task >> 1) - of * a.heads;
        const Side &side = a.side[task & 1];
        const Run run = runs[of];
        const int n = run.count;
        const uint32_t slot0 = (uint32_t)run.block * a.block, page = over(slot0, a.page_mul, a.page_shift), in0 = slot0 - page * a.page;
        float *scale = side.scales + page * side.ss[0] + over(in0, a.block_mul, a.block_shift) * side.ss[1] + head * side.ss[2];
        unsigned char *codes = side.codes + page * side.cs[0] + (int64_t)in0 * side.cs[1] + head * side.cs[2];
        const T *x = static_cast<const T *>(side.x) + head * side.xs[1];
        const float old = *scale;
        Size size = {0, false};
        uint32_t pairs = 0;
        auto look_at = [&](const Raw<T, V> &row) {
            if constexpr (sizeof(T) == 2 && V == 8) look_pairs(row, pairs);
            else look(row, size);
        };
        // one vector of row r
        auto read = [&](Raw<T, V> &to, int r, int c) { to.read(x + token_of[run.first + r] * side.xs[0] + c * V); };
        const bool whole = vecs <= L && n <= HELD * G;  // the registers hold the run
        Raw<T, V> held[HELD];
        if (whole) {
#pragma unroll
            for (int u = 0; u < HELD; ++u) {
                held[u].clear();
                if (u * G + sub < n && col < vecs) read(held[u], u * G + sub, col);
            }
#pragma unroll
            for (int u = 0; u < HELD; ++u) look_at(held[u]);
        } else {
            for (int r = sub; r < n; r += HELD * G)
                for (int c = col; c < vecs; c += L) {
#pragma unroll
                    for (int u = 0; u < HELD; ++u) {
                        held[u].clear();
                        if (r + u * G < n) read(held[u], r + u * G, c);
                    }
#pragma unroll
                    for (int u = 0; u < HELD; ++u) look_at(held[u]);
                }
        }
        if constexpr (sizeof(T) == 2 && V == 8) {
            pairs = __vmaxu2(pairs, pairs >> 16) & 0xffffu;
            pairs = __reduce_max_sync(0xffffffffu, pairs);
            T top;
            const uint16_t bits = (uint16_t)pairs;
            memcpy(&top, &bits, 2);
            size.bits = __float_as_uint(to_float(top));
            if (size.bits >= 0x7f800000u) {  // one of them is not finite: once more, leaving such out
                size = {0, true};
                for (int r = sub; r < n; r += G)
                    for (int c = col; c < vecs; c += L) {
                        Raw<T, V> again;
                        read(again, r, c);
                        look(again, size);
                    }
                size.odd = true;
                size.bits = __reduce_max_sync(0xffffffffu, size.bits);
            }
        } else {
            size.bits = __reduce_max_sync(0xffffffffu, size.bits);
            size.odd = __any_sync(0xffffffffu, size.odd);
        }
        uint32_t low = 0, high = 0;  // the places written
        for (int r = lane; r < n; r += 32) {
            const int place = place_of[run.first + r];
            if (place < 32) low |= 1u << place;
            else high |= 1u << (place - 32);
        }
        low = __reduce_or_sync(0xffffffffu, low);
        const bool begun = low & 1;
        const float need = scale_for(size.bits), now = begun ? need : fmaxf(old, need);
        const Divide by = divide_by(now, size.odd);
        if (whole && by.plain) {  // nearly always
#pragma unroll
            for (int u = 0; u < HELD; ++u)
                if (u * G + sub < n && col < vecs)
                    write_codes<true>(codes + place_of[run.first + u * G + sub] * side.cs[1] + col * V, held[u], by);
        } else {
            for (int r = sub; r < n; r += G)
                for (int c = col; c < vecs; c += L) {
                    Raw<T, V> again;
                    read(again, r, c);
                    unsigned char *to = codes + place_of[run.first + r] * side.cs[1] + c * V;
                    if (by.plain) write_codes<true>(to, again, by);
                    else write_codes<false>(to, again, by);
                }
        }
        if (!begun && now > old) {
            high = __reduce_or_sync(0xffffffffu, high);
            const float ratio = old / now;
            for (int r = sub; r < a.block; r += G) {
                if (((r < 32 ? low >> r : high >> (r - 32)) & 1)) continue;
                for (int c = col; c < vecs; c += L) rescale_codes<V>(codes + r * side.cs[1] + c * V, ratio);
            }
        }
        if (lane == 0) *scale = now;
    }
}

// ---------------------------------------------------------------- store, a scale per token
template <typename T, int V, int L>
__global__ void __launch_bounds__(kCodeThreads) paged_store_tokens_kernel(StoreCodesArgs a) {
    constexpr int U = sizeof(T) == 4 ? 1 : 2, ROWS = kCodeThreads / L * U;  // rows of a block of threads, keys and values each
    after_previous();
    const int lane = threadIdx.x % L, vecs = a.dim / V;
    const int64_t rows = (int64_t)a.tokens * a.heads, block0 = (int64_t)blockIdx.x * ROWS, token0 = block0 / a.heads;
    const uint32_t past = (uint32_t)(block0 - token0 * a.heads) + threadIdx.x / L;
    int32_t slot[U], head[U];
    int64_t token[U];
    Raw<T, V> held[U][2];
    Size size[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        // past the last row: the block's first token, not stored
        const bool in = block0 + threadIdx.x / L + u * (kCodeThreads / L) < rows;
        const uint32_t e = in ? past + u * (kCodeThreads / L) : 0, t = over(e, a.heads_mul, a.heads_shift);
        token[u] = token0 + t;
        head[u] = (int32_t)(e - t * a.heads);
        slot[u] = in ? a.slots[token[u]] : -1;
    }
    auto source = [&](int u, int s) { return static_cast<const T *>(a.side[s].x) + token[u] * a.side[s].xs[0] + head[u] * a.side[s].xs[1]; };
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            held[u][s].clear();
            if (lane < vecs) held[u][s].read(source(u, s) + lane * V);
        }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            size[u][s] = {0, false};
            look(held[u][s], size[u][s]);
            for (int c = lane + L; c < vecs; c += L) {
                Raw<T, V> more;
                more.read(source(u, s) + c * V);
                look(more, size[u][s]);
            }
            uint32_t all = size[u][s].bits | (size[u][s].odd ? 0x80000000u : 0u);
#pragma unroll
            for (int d = L / 2; d > 0; d >>= 1) {
                const uint32_t other = __shfl_xor_sync(0xffffffffu, all, d);
                all = max(all & 0x7fffffffu, other & 0x7fffffffu) | ((all | other) & 0x80000000u);
            }
            size[u][s] = {all & 0x7fffffffu, (all >> 31) != 0};
        }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t page = over((uint32_t)slot[u], a.page_mul, a.page_shift);
        if (slot[u] < 0 || page >= (uint32_t)a.num_pages) continue;
        const int64_t in = (uint32_t)slot[u] - page * a.page;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const Side &side = a.side[s];
            const float now = scale_for(size[u][s].bits);
            const Divide by = divide_by(now, size[u][s].odd);
            unsigned char *codes = side.codes + page * side.cs[0] + in * side.cs[1] + head[u] * side.cs[2];
            if (lane < vecs) {
                if (by.plain) write_codes<true>(codes + lane * V, held[u][s], by);
                else write_codes<false>(codes + lane * V, held[u][s], by);
            }
            for (int c = lane + L; c < vecs; c += L) {
                Raw<T, V> more;
                more.read(source(u, s) + c * V);
                write_codes<false>(codes + c * V, more, by);
            }
            if (lane == 0) side.scales[page * side.ss[0] + in * side.ss[1] + head[u] * side.ss[2]] = now;
        }
    }
}

template <typename T, int V, int L>
cudaError_t launch_store_codes(StoreCodesArgs &a, cudaStream_t stream) {
    if (a.block == 1) {
        constexpr int ROWS = kCodeThreads / L * (sizeof(T) == 4 ? 1 : 2);
        const int64_t blocks = ((int64_t)a.tokens * a.heads + ROWS - 1) / ROWS;
        return launch_chained(paged_store_tokens_kernel<T, V, L>, (unsigned)blocks, kCodeThreads, 0, 0, stream, a);
    }
    // few tokens: a tile's runs and heads go to several blocks
    const int sms = std::max(1, device_sm_count());
    const int64_t tiles = ((int64_t)a.tokens + kTile - 1) / kTile;
    const int64_t most = (std::min<int64_t>(kTile, a.tokens) * 2ll * a.heads + kCodeWarps - 1) / kCodeWarps;  // blocks that a tile could fill
    a.slices = (int)std::max<int64_t>(1, std::min<int64_t>(most, (2 * sms + tiles - 1) / tiles));
    return launch_chained(paged_store_blocks_kernel<T, V, L>, (unsigned)(tiles * a.slices), kCodeThreads, 0, 0, stream, a);
}
template <typename T>
cudaError_t launch_store_codes(StoreCodesArgs &a, bool wide, cudaStream_t stream) {
    if (!wide) return launch_store_codes<T, 1, 32>(a, stream);
    if (a.dim <= 64) return launch_store_codes<T, 8, 8>(a, stream);
    if (a.dim <= 128) return launch_store_codes<T, 8, 16>(a, stream);
    return launch_store_codes<T, 8, 32>(a, stream);
}

// ---------------------------------------------------------------- load
constexpr int kLoadRequests = 1024;  // token_ptr is read into shared memory up to so many
constexpr int kLoadThreads = 256;

struct LoadSide {
    const char *cache;
    const float *scales;
    char *out;
    int64_t cs[3], ss[3], os[2];
};
struct LoadArgs {
    LoadSide side[2];
    int64_t items;  // vectors of all rows
    int32_t requests, tokens, row, vecs, num_pages, page, max_pages;
    uint32_t row_mul, row_shift, vecs_mul, vecs_shift, page_mul, page_shift, block_mul, block_shift;
    const int32_t *table, *ptr;
    int64_t table_stride;
};

// The slot of row i: -1: left as it is, -2: zeros.
__device__ __forceinline__ int32_t slot_of_row(const LoadArgs &a, const int32_t *ptr, int64_t i) {
    if (i >= a.tokens || i < ptr[0] || i >= ptr[a.requests]) return -1;
    int lo = 0, hi = a.requests - 1;  // the last request that begins at or before i
    while (lo < hi) {
        const int mid = lo + ((hi - lo + 1) >> 1);  // lo + hi can pass 32 bits
        if (ptr[mid] <= i) lo = mid;
        else hi = mid - 1;
    }
    const int64_t t = i - ptr[lo];
    if (t < 0 || i >= ptr[lo + 1]) return -2;  // token_ptr falls somewhere
    const uint32_t p = over((uint32_t)t, a.page_mul, a.page_shift);
    if (p >= (uint32_t)a.max_pages) return -2;
    const int32_t page = a.table[lo * a.table_stride + p];
    if ((uint32_t)page >= (uint32_t)a.num_pages) return -2;
    return page * a.page + (int32_t)((uint32_t)t - p * a.page);
}

// CODES: the cache holds codes, N of them a vector, else elements T.
template <typename T, bool CODES, int N, int U>
__global__ void __launch_bounds__(kLoadThreads) paged_load_kernel(LoadArgs a) {
    using C = typename std::conditional<CODES, unsigned char, T>::type;
    extern __shared__ int32_t shared[];  // the block's tokens' slots, then token_ptr
    after_previous();
    const int64_t first = (int64_t)blockIdx.x * (kLoadThreads * U), token0 = first / a.row;
    const uint32_t skip = (uint32_t)(first - token0 * a.row);
    const int here = (int)((skip + kLoadThreads * U - 1) / a.row) + 1;  // tokens
    const int32_t *ptr = a.ptr;
    if (a.requests <= kLoadRequests) {
        int32_t *copy = shared + (kLoadThreads * U - 1) / a.row + 2;
        for (int r = threadIdx.x; r <= a.requests; r += kLoadThreads) copy[r] = a.ptr[r];
        __syncthreads();
        ptr = copy;
    }
    for (int i = threadIdx.x; i < here; i += kLoadThreads) shared[i] = slot_of_row(a, ptr, token0 + i);
    __syncthreads();
    // keys and values, all of a thread's, before any is stored
    Vec<C, N> in[2][U];
    float scale[2][U];
    int32_t slot[U];
    uint32_t token[U], head[U], at[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t e = skip + threadIdx.x + u * kLoadThreads, t = over(e, a.row_mul, a.row_shift), in_row = e - t * a.row;
        token[u] = t, head[u] = over(in_row, a.vecs_mul, a.vecs_shift), at[u] = (in_row - head[u] * a.vecs) * N;
        slot[u] = first + threadIdx.x + u * kLoadThreads < a.items ? shared[t] : -1;
        const bool there = slot[u] >= 0;
        const uint32_t page = there ? over((uint32_t)slot[u], a.page_mul, a.page_shift) : 0, inside = there ? (uint32_t)slot[u] - page * a.page : 0;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const LoadSide &side = a.side[s];
            scale[s][u] = 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i) in[s][u].v[i] = C{};
            if (!there) continue;
            in[s][u] = *reinterpret_cast<const Vec<C, N> *>(reinterpret_cast<const C *>(side.cache) + page * side.cs[0] +
                                                            inside * side.cs[1] + head[u] * side.cs[2] + at[u]);
            if (CODES)
                scale[s][u] = side.scales[page * side.ss[0] + over(inside, a.block_mul, a.block_shift) * side.ss[1] + head[u] * side.ss[2]];
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (slot[u] == -1) continue;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const LoadSide &side = a.side[s];
            T *to = reinterpret_cast<T *>(side.out) + (token0 + token[u]) * side.os[0] + head[u] * side.os[1] + at[u];
            if constexpr (CODES && N == 1) {
                *to = from_float<T>(from_e4m3x2(in[s][u].v[0]).x * scale[s][u]);
            } else if constexpr (CODES) {
                constexpr int W = 16 / sizeof(T);  // elements of a store
                uint32_t words[N / 4];
                memcpy(words, &in[s][u], N);
#pragma unroll
                for (int i = 0; i < N; i += W) {
                    Vec<T, W> out;
#pragma unroll
                    for (int j = 0; j < W; j += 2) {
                        const float2 x = from_e4m3x2(words[(i + j) / 4] >> ((i + j) % 4 * 8) & 0xffffu);
                        out.v[j] = from_float<T>(x.x * scale[s][u]), out.v[j + 1] = from_float<T>(x.y * scale[s][u]);
                    }
                    *reinterpret_cast<Vec<T, W> *>(to + i) = out;
                }
            } else {
                *reinterpret_cast<Vec<T, N> *>(to) = in[s][u];
            }
        }
    }
}

template <typename T, bool CODES, int N>
cudaError_t launch_load(const LoadArgs &a, cudaStream_t stream) {
    constexpr int U = N == 1 ? 4 : 1;
    const int64_t per_block = kLoadThreads * U;
    const size_t smem = 4 * ((per_block - 1) / a.row + 2 + (a.requests <= kLoadRequests ? a.requests + 1 : 0));
    return launch_chained(paged_load_kernel<T, CODES, N, U>, (unsigned)((a.items + per_block - 1) / per_block), kLoadThreads,
                          smem, 0, stream, a);
}

template <typename T>
cudaError_t launch_load_codes(const LoadArgs &a, int n, cudaStream_t stream) {
    return n == 16 ? launch_load<T, true, 16>(a, stream) : n == 8 ? launch_load<T, true, 8>(a, stream) : launch_load<T, true, 1>(a, stream);
}

bool strides_on(const void *p, const int64_t *strides, int n, int size, int bytes) {
    if (!aligned_to(p, bytes)) return false;
    for (int i = 0; i < n; ++i)
        if (strides[i] * size % bytes) return false;
    return true;
}

const char *cache_bad(const spmv_paged_cache_t *c, int32_t heads, int32_t head_dim) {
    if (!c) return "cache is NULL";
    if (heads < 0 || head_dim < 0 || c->num_pages < 0) return "negative size";
    if (c->page_size < 1) return "page_size must be at least 1";
    if ((int64_t)c->num_pages * c->page_size >= (1LL << 31)) return "num_pages * page_size must be < 2^31";
    if (c->block < 0 || (c->block > 0 && c->page_size % c->block)) return "page_size must be a multiple of block";
    if ((int64_t)heads * head_dim >= (1LL << 30)) return "heads * head_dim must be < 2^30";
    return nullptr;
}
const char *cache_missing(const spmv_paged_cache_t &c) {
    if (!c.k_cache || !c.v_cache) return "k_cache or v_cache is NULL";
    if (c.block && (!c.k_scales || !c.v_scales)) return "k_scales or v_scales is NULL";
    if (c.block && (!aligned_to(c.k_scales, 4) || !aligned_to(c.v_scales, 4))) return "the scales are not aligned to their type";
    return nullptr;
}

}  // namespace

}  // namespace lbcsr

using namespace lbcsr;

extern "C" {

spmv_status_t spmv_paged_store_e4m3(int32_t tokens, int32_t heads, int32_t head_dim, spmv_elem_t elem, const int32_t *slots,
                                    const spmv_paged_cache_t *cache, const void *k, const int64_t *k_stride, const void *v,
                                    const int64_t *v_stride, spmv_stream_t stream_handle) {
    if (tokens < 0) return llm_bad("negative size");
    if (const char *bad = cache_bad(cache, heads, head_dim)) return llm_bad(bad);
    const spmv_paged_cache_t &c = *cache;
    if (c.block < 1 || c.block > kMaxBlock) return llm_bad("block must be in [1, 64]");
    if ((int64_t)tokens * heads >= (1LL << 33)) return llm_bad("tokens * heads must be < 2^33");
    if (heads >= 1 << 24) return llm_bad("heads must be < 2^24");  // a tile's runs times heads are counted in 32 bits
    if (!elem_ok(elem)) return llm_bad("unknown element type");
    if (!k_stride || !v_stride) return llm_bad("a stride array is NULL");
    if (tokens == 0 || heads == 0 || head_dim == 0 || c.num_pages == 0) return SPMV_OK;
    if (!slots || !k || !v) return llm_bad("slots, k or v is NULL");
    if (const char *bad = cache_missing(c)) return llm_bad(bad);
    const int size = elem_size(elem);
    if (!aligned_to(slots, 4) || !aligned_to(k, size) || !aligned_to(v, size)) return llm_bad("slots, k or v is not aligned to its type");
    StoreCodesArgs a;
    a.side[0] = {k, static_cast<unsigned char *>(c.k_cache), c.k_scales, {}, {}, {}};
    a.side[1] = {v, static_cast<unsigned char *>(c.v_cache), c.v_scales, {}, {}, {}};
    std::copy(k_stride, k_stride + 2, a.side[0].xs), std::copy(v_stride, v_stride + 2, a.side[1].xs);
    std::copy(c.k_stride, c.k_stride + 3, a.side[0].cs), std::copy(c.v_stride, c.v_stride + 3, a.side[1].cs);
    std::copy(c.k_scale_stride, c.k_scale_stride + 3, a.side[0].ss), std::copy(c.v_scale_stride, c.v_scale_stride + 3, a.side[1].ss);
    bool wide = head_dim % 8 == 0;
    for (const Side &s : a.side) wide = wide && strides_on(s.x, s.xs, 2, size, 16) && strides_on(s.codes, s.cs, 3, 1, 8);
    a.tokens = tokens, a.heads = heads, a.dim = head_dim;
    a.num_pages = c.num_pages, a.page = c.page_size, a.block = c.block;
    a.slices = 0;
    a.slots = slots;
    set_divisor((uint32_t)c.page_size, &a.page_mul, &a.page_shift);
    set_divisor((uint32_t)c.block, &a.block_mul, &a.block_shift);
    set_divisor((uint32_t)heads, &a.heads_mul, &a.heads_shift);
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_handle);
    return llm_launched("spmv_paged_store_e4m3 launch", elem == SPMV_ELEM_F32    ? launch_store_codes<float>(a, wide, stream)
                                                        : elem == SPMV_ELEM_BF16 ? launch_store_codes<__nv_bfloat16>(a, wide, stream)
                                                                                 : launch_store_codes<__half>(a, wide, stream));
}

spmv_status_t spmv_paged_load(int32_t requests, int32_t tokens, int32_t heads, int32_t head_dim, spmv_elem_t elem,
                              const int32_t *table, int64_t table_stride, int32_t max_pages, const int32_t *token_ptr,
                              const spmv_paged_cache_t *cache, void *k, const int64_t *k_stride, void *v,
                              const int64_t *v_stride, spmv_stream_t stream_handle) {
    if (requests < 0 || tokens < 0 || max_pages < 0) return llm_bad("negative size");
    if (const char *bad = cache_bad(cache, heads, head_dim)) return llm_bad(bad);
    const spmv_paged_cache_t &c = *cache;
    if ((int64_t)tokens * heads * head_dim >= (1LL << 40)) return llm_bad("tokens * heads * head_dim must be < 2^40");
    if (!elem_ok(elem)) return llm_bad("unknown element type");
    if (!k_stride || !v_stride) return llm_bad("a stride array is NULL");
    if (requests == 0 || tokens == 0 || heads == 0 || head_dim == 0) return SPMV_OK;
    if (!token_ptr || !k || !v) return llm_bad("token_ptr, k or v is NULL");
    if (max_pages > 0 && !table) return llm_bad("table is NULL");
    if (c.num_pages > 0)
        if (const char *bad = cache_missing(c)) return llm_bad(bad);
    const int size = elem_size(elem), held = c.block ? 1 : size;
    if (!aligned_to(table, 4) || !aligned_to(token_ptr, 4)) return llm_bad("table or token_ptr is not aligned to its type");
    if (!aligned_to(k, size) || !aligned_to(v, size) || !aligned_to(c.k_cache, held) || !aligned_to(c.v_cache, held))
        return llm_bad("k, v or a cache is not aligned to its type");
    LoadArgs a;
    a.side[0] = {static_cast<const char *>(c.k_cache), c.k_scales, static_cast<char *>(k), {}, {}, {}};
    a.side[1] = {static_cast<const char *>(c.v_cache), c.v_scales, static_cast<char *>(v), {}, {}, {}};
    std::copy(k_stride, k_stride + 2, a.side[0].os), std::copy(v_stride, v_stride + 2, a.side[1].os);
    std::copy(c.k_stride, c.k_stride + 3, a.side[0].cs), std::copy(c.v_stride, c.v_stride + 3, a.side[1].cs);
    std::copy(c.k_scale_stride, c.k_scale_stride + 3, a.side[0].ss), std::copy(c.v_scale_stride, c.v_scale_stride + 3, a.side[1].ss);
    // 16 codes are one load of 16 bytes and two or four stores; 8 where heads or strides allow no more
    auto fits = [&](int n) {
        bool wide = head_dim % n == 0;
        for (const LoadSide &s : a.side) wide = wide && strides_on(s.cache, s.cs, 3, held, n * held) && strides_on(s.out, s.os, 2, size, 16);
        return wide;
    };
    const int n = c.block ? (fits(16) ? 16 : 8) : 16 / size;
    const bool wide = fits(n);
    a.vecs = wide ? head_dim / n : head_dim;
    a.row = heads * a.vecs;
    a.items = (int64_t)tokens * a.row;
    a.requests = requests, a.tokens = tokens, a.num_pages = c.num_pages, a.page = c.page_size, a.max_pages = max_pages;
    a.table = table, a.ptr = token_ptr, a.table_stride = table_stride;
    set_divisor((uint32_t)a.row, &a.row_mul, &a.row_shift);
    set_divisor((uint32_t)a.vecs, &a.vecs_mul, &a.vecs_shift);
    set_divisor((uint32_t)c.page_size, &a.page_mul, &a.page_shift);
    set_divisor((uint32_t)std::max(1, c.block), &a.block_mul, &a.block_shift);
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_handle);
    cudaError_t e;
    if (c.block)
        e = elem == SPMV_ELEM_F32    ? launch_load_codes<float>(a, wide ? n : 1, stream)
            : elem == SPMV_ELEM_BF16 ? launch_load_codes<__nv_bfloat16>(a, wide ? n : 1, stream)
                                     : launch_load_codes<__half>(a, wide ? n : 1, stream);
    else
        e = size == 4 ? (wide ? launch_load<float, false, 4>(a, stream) : launch_load<float, false, 1>(a, stream))
                      : (wide ? launch_load<__half, false, 8>(a, stream) : launch_load<__half, false, 1>(a, stream));
    return llm_launched("spmv_paged_load launch", e);
}

}  // extern "C"
