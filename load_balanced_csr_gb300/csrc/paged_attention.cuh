// Attention of one new token per request over a paged key-value cache:
//
//   s_t = scale <q, k_t>,  out = sum_t exp(s_t - m) v_t / sum_t exp(s_t - m)
//
// in one pass over the positions with the running maximum m and sum of the
// softmax: when a score above m comes, the sums so far are scaled by
// exp(m_old - m_new).  The maximum is the dot products' own, before their
// scale: a weight is 2^((x - m) scale / ln 2), whose difference is taken before
// anything is rounded, so that the highest score's weight is 1 however large
// the scores are.
//
// The work is a sparse product's with very uneven rows: row (request, kv
// head), one unit per chunk of positions and kRowCost for the row itself.
// Units in row order are cut into equal shares whatever the lengths (the
// merge-path SpMV's schedule), one per block, and those among the block's
// warps.  Each warp is a pipeline of its own: it copies its next chunks into
// its part of shared memory (cp.async, several chunks in flight) while it
// works on the present one, across row ends, with no barrier in the loop.  A
// row inside one share is written out by its warp; the parts of a row cut
// between warps are records (unnormalised sums, m and l per head) that the
// block joins in shared memory; the blocks' parts of a row cut between blocks
// are joined, in block order, by the last of them to arrive.  The order of
// every sum is fixed by the lengths, so results do not change between calls.
//
// Bound by memory where the cache is large: the steady loop moves 6.7 TB/s,
// the measured copy's rate.  One request of 131,071 positions, 8 kv heads of
// 128 bf16 (537 MB), 100 us: 5.35 TB/s, 0.80 of the copy.  Of the rest, about
// 7 us pass before the first chunk has come and 6 after the last warp's last;
// and groups of SMs get 14 % less of the memory than others when all ask at
// once (their blocks end at 88 us, most at 77), which equal shares cannot
// know.  Shares that warps take as they become free (small segments, parts
// joined by a second kernel) evened that out and cost more in parts: 120 us.
// Tensor Memory Accelerator copies are not used: pages may be of any size and
// strides, and the copies are not what it waits for.  The matrix instructions
// are the warp's own (16 x 8 x 16): a chunk's products have 8 or 16 rows of
// heads, and run while the warp's next chunks are on their way.
#pragma once

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <type_traits>

#include "internal.cuh"
#include "llm.cuh"

namespace lbcsr {

// One translation unit per element type holds its kernels.  group: query
// heads per kv head.
size_t attention_workspace_f32(int dim, int group, int sms);
size_t attention_workspace_bf16(int dim, int group, int sms);
size_t attention_workspace_f16(int dim, int group, int sms);
size_t attention_workspace_e4m3(int dim, int group, int sms);
cudaError_t launch_attention_f32(const spmv_paged_attention_t &a, int sms, cudaStream_t stream);
cudaError_t launch_attention_bf16(const spmv_paged_attention_t &a, int sms, cudaStream_t stream);
cudaError_t launch_attention_f16(const spmv_paged_attention_t &a, int sms, cudaStream_t stream);

// The scales of caches of 8-bit codes (paged_attention_e4m3.cu has the tile).
struct AttendScales {
    const float *k, *v;
    int64_t k_stride[3], v_stride[3];  // page, block in it, head
    uint32_t mul, shift;               // division by a block's positions
};
cudaError_t launch_attention_e4m3(const spmv_paged_attention_t &a, const AttendScales &scales, int sms, cudaStream_t stream);

namespace {

constexpr int kMaxDim = 256;
constexpr int kSmemAlign = 32;  // bytes, of a block's shared memory: what the widest vector read from it asks for
constexpr int kMaxSlice = 1024;  // requests per launch: their lengths and prefix sums live in shared memory
// Units a row costs beside its chunks (its queries, its output): without, a
// batch of 128 requests of 1 to 16,384 positions took 190 us instead of 158,
// the blocks with the short ones being last.
constexpr uint32_t kRowCost = 3;
// Rows of so few chunks are not cut between blocks, of so few not between
// warps: joining would take longer than the row (4 requests of up to 300
// positions, lengths even over the logarithm, 16 heads of 64 f16 over as many:
// 18.4 us with every row cut alike, 14.3 so; both with L2 flushed).
constexpr uint32_t kBlockRow = 32;
constexpr uint32_t kWarpRow = 2;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;

enum { kBadPage = 1, kBadLength = 2 };

struct AttendArgs {
    spmv_paged_attention_t a;
    int32_t group;   // query heads per kv head
    int32_t tiles;   // head tiles per kv head
    int32_t rows;    // kv_heads * tiles: rows per request
    float scale2;    // |scale| / ln 2
    uint32_t flip;   // sign bits of a pair of 16-bit elements, set when scale < 0: q is negated
    uint32_t page_mul, page_shift;  // t / page_size = (mulhi(t, page_mul) + t) >> page_shift
    int32_t q_pairs, out_pairs;     // pairs of elements of q, of out, are aligned
    int32_t same_strides;           // of the two caches
    int32_t *arrivals;   // [blocks], zero between calls
    float *warp_rec;     // [blocks * warps] records
    float *block_rec;    // [blocks][2] records: of the row that began earlier and ends here, of the one that goes on
};

struct ScaledArgs : AttendArgs {
    AttendScales scales;
};

__device__ __forceinline__ uint32_t smem_addr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
// 16 bytes from global to shared memory; zeros when !real (src is then not read)
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool real) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void *src, bool real) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(real ? 4 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t r[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4_t(uint32_t addr, uint32_t r[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
template <typename T>
__device__ __forceinline__ void mma16816(float c[4], const uint32_t a[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float c[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__half>(float c[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(T lo, T hi) {
    static_assert(sizeof(T) == 2, "");
    uint16_t l, h;
    memcpy(&l, &lo, 2);
    memcpy(&h, &hi, 2);
    return (uint32_t)l | ((uint32_t)h << 16);
}

// the pair with zeros in the place of infinities
__device__ __forceinline__ uint32_t no_infinities(uint32_t pair, __nv_bfloat16) {
    __nv_bfloat162 v;
    memcpy(&v, &pair, 4);
    return pair & ~__heq2_mask(__habs2(v), __bfloat162bfloat162(__ushort_as_bfloat16(0x7f80)));
}
__device__ __forceinline__ uint32_t no_infinities(uint32_t pair, __half) {
    __half2 v;
    memcpy(&v, &pair, 4);
    return pair & ~__heq2_mask(__habs2(v), __half2half2(__ushort_as_half(0x7c00)));
}

// 2^x by the hardware's instruction: 2 units in the last place, results
// below 2^-126 are zero (next to a row's largest weight of 1)
__device__ __forceinline__ float pow2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// the mask of a whole chunk
template <int CH>
constexpr uint32_t FULL_MASK = 0xffffffffu >> (32 - CH);

// what products are taken relative to; the running maximum m is -infinity
// until one has come, and nothing has weight then
__device__ __forceinline__ float base_of(float m) { return m == -INFINITY ? 0.0f : m; }
// what sums relative to m are worth relative to `base`, a maximum not below m
__device__ __forceinline__ float worth(float m, float base, float scale2) {
    return m == -INFINITY ? 0.0f : pow2((m - base) * scale2);
}

// ------------------------------------------------------------ 16-bit elements
// A chunk is 16 positions, or 32 of small heads, so that a chunk's fixed work
// is not most of it; a tile is 8 or 16 query heads of one kv head.  The
// scores are one 16 x CH product per chunk (heads by positions) and the
// output one 16 x DP product, on the warp's matrix instructions with 32-bit
// sums.  The weights go into the second product as hi + lo, two elements of
// the caches' type (p - hi is exact in 32 bits), so they carry 16 (bf16) or
// 22 (f16) bits: with hi alone the output's error against 64 bits is 1.4
// times that of one rounding.  A tile of 8 heads has hi in the product's
// first 8 rows and lo in its last 8, and so costs no more than hi alone.
// f16 weights are taken 2^15 times as large, as are the sums: its smallest
// step is then 2^-39 of a row's largest weight (2^-24 otherwise, below half of
// which a weight is lost: many positions behind one high score).
// An infinity in V is the hi product's alone: lo may be zero or negative, and
// would make it NaN.  A tile of 8 heads leaves lo's sum out where hi's is
// infinite; one of 16, whose halves share their sums, gives lo values without
// infinities.
template <typename T_, int GT_, int DP_, int CH_, int NW_, int STAGES_>
struct TileMma {
    using T = T_;
    using Cache = T;           // the caches' elements
    using Args = AttendArgs;
    static constexpr int SLICE = kMaxSlice;
    static constexpr bool SCALES = false;
    static constexpr int DP = DP_, NW = NW_, STAGES = STAGES_, GT = GT_, CH = CH_;
    static constexpr int PAGE_UNIT = 16;   // positions that lie in one page when page_size is a multiple
    static constexpr int NT = CH / 8;      // the scores' product in columns of 8 positions
    static constexpr int PITCH = DP * 2 + 16;  // bytes: rows 16 bytes apart modulo 128, so ldmatrix has no conflicts
    static constexpr int QBYTES = 0;
    static constexpr float LIFT = std::is_same<T, __half>::value ? 15.0f : 0.0f;  // log2 of a weight of 1
    static constexpr int H = GT / 8;  // heads of a lane: lane / 4 and, with 16, lane / 4 + 8

    static constexpr bool AHEAD = GT * DP <= 1024;  // registers for the next row's queries too

    uint32_t q[DP / 16][2 * H], next[AHEAD ? DP / 16 : 1][2 * H];
    float o[DP / 8][4];
    float m[H], l[H];  // l: this lane's part of the sum

    // the queries of a row, as the product's left operand
    __device__ __forceinline__ static void load(const AttendArgs &p, uint32_t (*to)[2 * H], int b, int h0, int heads, int lane) {
        const T *base = static_cast<const T *>(p.a.q) + b * p.a.q_stride[0] + h0 * p.a.q_stride[1];
        const int g = lane >> 2, t = (lane & 3) * 2;
#pragma unroll
        for (int s = 0; s < DP / 16; ++s)
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    const int head = g + h * 8, d = s * 16 + t + r * 8;
                    const T *at = base + head * p.a.q_stride[1] + d;
                    uint32_t pair = 0;
                    if (head < heads && d < p.a.head_dim)
                        pair = p.q_pairs ? *reinterpret_cast<const uint32_t *>(at) : pack2(at[0], at[1]);
                    to[s][r * H + h] = pair;
                }
    }
    // starts to load the next row's queries
    __device__ __forceinline__ void fetch(const AttendArgs &p, int b, int h0, int heads, int lane) {
        if (AHEAD) load(p, next, b, h0, heads, lane);
    }
    __device__ __forceinline__ void begin(const AttendArgs &p, int b, int h0, int heads, char *, int lane, bool fetched) {
        if (AHEAD && fetched) {
#pragma unroll
            for (int s = 0; s < DP / 16; ++s)
#pragma unroll
                for (int r = 0; r < 2 * H; ++r) q[s][r] = next[AHEAD ? s : 0][r];
        } else {
            load(p, q, b, h0, heads, lane);
        }
        if (p.flip) {  // a pair of zeros may become a pair of negative zeros: the products stay zeros
#pragma unroll
            for (int s = 0; s < DP / 16; ++s)
#pragma unroll
                for (int r = 0; r < 2 * H; ++r) q[s][r] ^= p.flip;
        }
#pragma unroll
        for (int n = 0; n < DP / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.0f;
#pragma unroll
        for (int h = 0; h < H; ++h) m[h] = -INFINITY, l[h] = 0.0f;
    }

    __device__ __forceinline__ void chunk(const AttendArgs &p, const char *stage, char *, uint32_t mask, int lane) {
        const uint32_t ks = smem_addr(stage), vs = ks + CH * PITCH;
        const int r8 = lane & 7, mat = lane >> 3;
        // with 16 positions, each score in two sums that do not wait for one another
        constexpr int SPLIT = CH == 16 ? 2 : 1;
        float sums[SPLIT][NT][4] = {};
        {
            const uint32_t at = ks + (r8 + (mat >> 1) * 8) * PITCH + (mat & 1) * 16;
#pragma unroll
            for (int i = 0; i < DP / 16; ++i) {
                const uint32_t qa[4] = {q[i][0], H == 2 ? q[i][H - 1] : 0u, q[i][H], H == 2 ? q[i][2 * H - 1] : 0u};
#pragma unroll
                for (int n = 0; n < NT; n += 2) {
                    uint32_t kb[4];
                    ldmatrix4(at + n * 8 * PITCH + i * 32, kb);
                    mma16816<T>(sums[i % SPLIT][n], qa, kb[0], kb[1]);
                    mma16816<T>(sums[i % SPLIT][n + 1], qa, kb[2], kb[3]);
                }
            }
        }
        const bool whole = mask == FULL_MASK<CH>;
        uint32_t hi[NT * H], lo[NT * H];  // [8 positions][head]
        float s[NT][H][2], top[H];
        bool higher = false;
#pragma unroll
        for (int h = 0; h < H; ++h) {
            float raw = -INFINITY;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    s[n][h][c] = sums[0][n][2 * h + c];
                    if (SPLIT == 2) s[n][h][c] += sums[SPLIT - 1][n][2 * h + c];
                    if (!whole && !((mask >> (n * 8 + (lane & 3) * 2 + c)) & 1)) s[n][h][c] = -INFINITY;
                    raw = fmaxf(raw, s[n][h][c]);
                }
            raw = fmaxf(raw, __shfl_xor_sync(0xffffffffu, raw, 1));
            raw = fmaxf(raw, __shfl_xor_sync(0xffffffffu, raw, 2));
            top[h] = fmaxf(m[h], raw);
            higher |= top[h] > m[h];
        }
        if (__any_sync(0xffffffffu, higher)) {
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const float keep = worth(m[h], top[h], p.scale2);
                l[h] *= keep;
                m[h] = top[h];
#pragma unroll
                for (int n = 0; n < DP / 8; ++n) {
                    o[n][2 * h] *= keep, o[n][2 * h + 1] *= keep;
                    if (H == 1) o[n][2] *= keep, o[n][3] *= keep;
                }
            }
        }
#pragma unroll
        for (int h = 0; h < H; ++h) {
            const float base = base_of(m[h]);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float w[2];
                T high[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    w[c] = pow2(fmaf(s[n][h][c] - base, p.scale2, LIFT));
                    if (!whole && !((mask >> (n * 8 + (lane & 3) * 2 + c)) & 1)) w[c] = 0.0f;
                    high[c] = from_float<T>(w[c]);
                }
                l[h] += w[0] + w[1];
                hi[n * H + h] = pack2(high[0], high[1]);
                lo[n * H + h] = pack2(from_float<T>(w[0] - to_float(high[0])), from_float<T>(w[1] - to_float(high[1])));
            }
        }
        const uint32_t at = vs + (r8 + (mat & 1) * 8) * PITCH + (mat >> 1) * 16;
#pragma unroll
        for (int k = 0; k < CH / 16; ++k) {
            const uint32_t *kh = hi + 2 * k * H, *kl = lo + 2 * k * H;
            const uint32_t pa[4] = {kh[0], H == 1 ? kl[0] : kh[H - 1], kh[H], H == 1 ? kl[1] : kh[2 * H - 1]};
            const uint32_t pl[4] = {kl[0], kl[H - 1], kl[H], kl[2 * H - 1]};
#pragma unroll
            for (int i = 0; i < DP / 16; ++i) {
                uint32_t vb[4];
                ldmatrix4_t(at + k * 16 * PITCH + i * 32, vb);
                mma16816<T>(o[2 * i], pa, vb[0], vb[1]);
                mma16816<T>(o[2 * i + 1], pa, vb[2], vb[3]);
            }
            if (H == 2) {
                // in a loop of its own, V read again: with both products at each V, 64 requests of 1 to 4,000 positions,
                // 4 kv heads with 16 heads each, took 168 us instead of 150 with 256 elements, 152 instead of 140 with 192
#pragma unroll
                for (int i = 0; i < DP / 16; ++i) {
                    uint32_t vb[4];
                    ldmatrix4_t(at + k * 16 * PITCH + i * 32, vb);
#pragma unroll
                    for (int j = 0; j < 4; ++j) vb[j] = no_infinities(vb[j], T());
                    mma16816<T>(o[2 * i], pl, vb[0], vb[1]);
                    mma16816<T>(o[2 * i + 1], pl, vb[2], vb[3]);
                }
            }
        }
    }

    __device__ __forceinline__ void sums() {
#pragma unroll
        for (int h = 0; h < H; ++h) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
        }
    }

    // hi and lo sums of a tile of 8 heads: an infinity of the first stands
    __device__ __forceinline__ static float joined(float hi, float lo) { return isinf(hi) ? hi : hi + lo; }

    // f(head, d, value at d, value at d + 1, l)
    template <typename F>
    __device__ __forceinline__ void each(int lane, F f) const {
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
            for (int n = 0; n < DP / 8; ++n) {
                const float x = H == 1 ? joined(o[n][0], o[n][2]) : o[n][2 * h], y = H == 1 ? joined(o[n][1], o[n][3]) : o[n][2 * h + 1];
                f((lane >> 2) + 8 * h, n * 8 + (lane & 3) * 2, x, y, l[h]);
            }
    }
    // f(head, m, l), once per head
    template <typename F>
    __device__ __forceinline__ void each_head(int lane, F f) const {
#pragma unroll
        for (int h = 0; h < H; ++h)
            if ((lane & 3) == 0) f((lane >> 2) + 8 * h, m[h], l[h]);
    }
};

// ------------------------------------------------------------ 32-bit elements
// A chunk is 8 positions; a tile is GT query heads.  For the scores lane
// (quarter, position) takes a quarter of the dot product of its position with
// every head of the tile; for the output lane l takes elements 2 l, 2 l + 1,
// 64 + 2 l, ... of every head.  Products and sums in 32 bits: there is no
// matrix instruction that keeps 32-bit inputs whole.  Bound by the latency of
// its instructions with 12 warps an SM: 16 requests of up to 5,000 positions,
// 4 kv heads of 72 and 3 query heads each, 7 positions a page (98 MB) 39 us;
// groups of 8 heads of 128 with a tile of 8 74 us, with two of 4 102 us.
template <int DP_, int GT_, int NW_, int STAGES_>
struct TileF32 {
    using T = float;
    using Cache = float;
    using Args = AttendArgs;
    static constexpr int SLICE = kMaxSlice;
    static constexpr bool SCALES = false;
    static constexpr int DP = DP_, NW = NW_, STAGES = STAGES_, GT = GT_, CH = 8, PAGE_UNIT = 8;
    static constexpr int PITCH = DP * 4 + 16;
    static constexpr float LIFT = 0.0f;
    static constexpr int WEIGHTS = GT * DP * 4;                // offset of the weights of a chunk behind the queries
    static constexpr int QBYTES = WEIGHTS + GT * CH * 4;
    using Weights = Vec<float, GT>;                            // of a position
    static_assert(kSmemAlign % alignof(Weights) == 0 && WEIGHTS % alignof(Weights) == 0, "a position's weights are aligned");
    static constexpr bool AHEAD = true;
    static constexpr int PAIRS = (DP + 63) / 64;               // pairs of elements of a lane; the last may not exist

    float2 o[GT][PAIRS];
    float m[GT], l[GT];       // l: this lane's part of the sum
    float next[GT][DP / 32];  // the next row's queries: elements lane, lane + 32, ...

    __device__ __forceinline__ static bool has_pair(int lane, int i) { return DP % 64 == 0 || 2 * (lane + 32 * i) < DP; }

    __device__ __forceinline__ void fetch(const AttendArgs &p, int b, int h0, int heads, int lane) {
        const float *base = static_cast<const float *>(p.a.q) + b * p.a.q_stride[0] + h0 * p.a.q_stride[1];
#pragma unroll
        for (int g = 0; g < GT; ++g)
#pragma unroll
            for (int i = 0; i < DP / 32; ++i)
                next[g][i] = g < heads && lane + 32 * i < p.a.head_dim ? base[g * p.a.q_stride[1] + lane + 32 * i] : 0.0f;
    }
    __device__ __forceinline__ void begin(const AttendArgs &p, int b, int h0, int heads, char *qs, int lane, bool fetched) {
        if (!fetched) fetch(p, b, h0, heads, lane);
        float *q = reinterpret_cast<float *>(qs);
        __syncwarp();
#pragma unroll
        for (int g = 0; g < GT; ++g) {
#pragma unroll
            for (int i = 0; i < DP / 32; ++i) q[g * DP + lane + 32 * i] = p.flip ? -next[g][i] : next[g][i];
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) o[g][i] = make_float2(0.0f, 0.0f);
            m[g] = -INFINITY;
            l[g] = 0.0f;
        }
        __syncwarp();
    }

    __device__ __forceinline__ void chunk(const AttendArgs &p, const char *stage, char *qs, uint32_t mask, int lane) {
        const int pos = lane & 7, quarter = lane >> 3;
        const float4 *k = reinterpret_cast<const float4 *>(stage + pos * PITCH) + quarter * (DP / 16);
        const float4 *q = reinterpret_cast<const float4 *>(qs) + quarter * (DP / 16);
        float s[GT], s2[GT], top[GT];
#pragma unroll
        for (int g = 0; g < GT; ++g) s[g] = s2[g] = 0.0f;
#pragma unroll
        for (int i = 0; i < DP / 16; ++i) {
            const float4 kv = k[i];
#pragma unroll
            for (int g = 0; g < GT; ++g) {
                const float4 qv = q[g * (DP / 4) + i];
                s[g] = fmaf(qv.x, kv.x, fmaf(qv.y, kv.y, s[g]));
                s2[g] = fmaf(qv.z, kv.z, fmaf(qv.w, kv.w, s2[g]));
            }
        }
        const bool live = (mask >> pos) & 1;
#pragma unroll
        for (int g = 0; g < GT; ++g) s[g] += s2[g];
#pragma unroll
        for (int d = 8; d < 32; d <<= 1)
#pragma unroll
            for (int g = 0; g < GT; ++g) s[g] += __shfl_xor_sync(0xffffffffu, s[g], d);
#pragma unroll
        for (int g = 0; g < GT; ++g) top[g] = live ? s[g] : -INFINITY;
#pragma unroll
        for (int d = 1; d < 8; d <<= 1)
#pragma unroll
            for (int g = 0; g < GT; ++g) top[g] = fmaxf(top[g], __shfl_xor_sync(0xffffffffu, top[g], d));
        bool higher = false;  // the same on every lane
#pragma unroll
        for (int g = 0; g < GT; ++g) {
            top[g] = fmaxf(m[g], top[g]);
            higher |= top[g] > m[g];
        }
        if (higher) {
#pragma unroll
            for (int g = 0; g < GT; ++g) {
                const float keep = worth(m[g], top[g], p.scale2);
                l[g] *= keep;
#pragma unroll
                for (int i = 0; i < PAIRS; ++i) o[g][i].x *= keep, o[g][i].y *= keep;
                m[g] = top[g];
            }
        }
        float *weights = reinterpret_cast<float *>(qs + WEIGHTS);  // [position][head]
#pragma unroll
        for (int j = 0; j < GT; j += 4) {  // a quarter stores one head of four
            float own = 0.0f;
#pragma unroll
            for (int g = j; g < GT && g < j + 4; ++g) {
                const float w = live ? pow2((s[g] - base_of(m[g])) * p.scale2) : 0.0f;
                if (quarter == 0) l[g] += w;
                if (quarter == g - j) own = w;
            }
            if (j + quarter < GT) weights[pos * GT + j + quarter] = own;
        }
        __syncwarp();
        const char *v = stage + CH * PITCH;
#pragma unroll
        for (int t = 0; t < CH; ++t) {
            float2 vv[PAIRS];
#pragma unroll
            for (int i = 0; i < PAIRS; ++i)
                vv[i] = has_pair(lane, i) ? reinterpret_cast<const float2 *>(v + t * PITCH)[lane + 32 * i] : make_float2(0.0f, 0.0f);
            const Weights w = *reinterpret_cast<const Weights *>(weights + t * GT);
#pragma unroll
            for (int g = 0; g < GT; ++g)
#pragma unroll
                for (int i = 0; i < PAIRS; ++i) {
                    o[g][i].x = fmaf(w.v[g], vv[i].x, o[g][i].x);
                    o[g][i].y = fmaf(w.v[g], vv[i].y, o[g][i].y);
                }
        }
    }

    __device__ __forceinline__ void sums() {
#pragma unroll
        for (int g = 0; g < GT; ++g)
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) l[g] += __shfl_xor_sync(0xffffffffu, l[g], d);
    }
    template <typename F>
    __device__ __forceinline__ void each(int lane, F f) const {
#pragma unroll
        for (int g = 0; g < GT; ++g)
#pragma unroll
            for (int i = 0; i < PAIRS; ++i)
                if (has_pair(lane, i)) f(g, 64 * i + 2 * lane, o[g][i].x, o[g][i].y, l[g]);
    }
    template <typename F>
    __device__ __forceinline__ void each_head(int lane, F f) const {
#pragma unroll
        for (int g = 0; g < GT; ++g)
            if (lane == 0) f(g, m[g], l[g]);
    }
};

// A part of a row, when the row is cut: GT rows of sums, then m and l of
// each head.
template <class P>
struct Record {
    static constexpr int ROW = P::DP + 8;  // the rows' first banks differ
    static constexpr int FLOATS = (P::GT * ROW + 2 * P::GT + 3) / 4 * 4;  // records are read 16 bytes at a time
    static constexpr int KV = 2 * P::CH * P::PITCH;                     // bytes of a chunk's K and V
    static constexpr int STAGE = KV + (P::SCALES ? 8 * P::CH : 0);      // and their scales
    static constexpr int WARP = P::STAGES * STAGE + P::QBYTES;          // bytes of a warp's shared memory
    static_assert(2 * FLOATS * 4 <= P::STAGES * STAGE, "both records of a warp fit its stages");
    static_assert(FLOATS % 4 == 0 && ROW % 4 == 0 && P::PITCH % 16 == 0 && P::QBYTES % 16 == 0, "16-byte accesses");
    static constexpr int PREFIX = (4 * (2 * P::SLICE + 1) + 127) / 128 * 128;
    static_assert(PREFIX % kSmemAlign == 0 && WARP % kSmemAlign == 0 && STAGE % kSmemAlign == 0, "as the block's shared memory");
    static constexpr int SMEM = PREFIX + P::NW * WARP;
};

// The rows: where each request's units begin.
struct Rows {
    const uint32_t *pre;   // [batch + 1]
    const int32_t *lens;   // [batch], within their tables
    int batch, rows;       // rows: per request

    // the request of unit c
    __device__ __forceinline__ int request(uint32_t c) const {
        int lo = 0, hi = batch - 1;  // the first with pre[b + 1] > c
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (pre[mid + 1] > c) hi = mid;
            else lo = mid + 1;
        }
        return lo;
    }
    __device__ __forceinline__ uint32_t units(int b) const { return (pre[b + 1] - pre[b]) / rows; }
    // a cut at unit c: one inside a short row, or before a row's first chunk, moves to the row's begin
    __device__ __forceinline__ uint32_t cut(uint32_t c, uint32_t short_row) const {
        if (c >= pre[batch]) return pre[batch];
        const int b = request(c);
        const uint32_t n = units(b), u = (c - pre[b]) % n;
        return n - kRowCost <= short_row || u <= kRowCost ? c - u : c;
    }
};

// A warp's place: chunk ch of nch of row vh of request b.
struct Place {
    int b, vh, len;
    uint32_t ch, nch;

    // the chunk that a share beginning at unit c begins with; returns its unit
    __device__ __forceinline__ uint32_t find(const Rows &r, uint32_t c) {
        b = r.request(c);
        const uint32_t n = r.units(b), u = (c - r.pre[b]) % n;
        vh = (int)((c - r.pre[b]) / n);
        nch = n - kRowCost;
        ch = u == 0 ? 0 : u - kRowCost;
        len = r.lens[b];
        return c - u + kRowCost + ch;
    }
    // the next row (only called while there is one)
    __device__ __forceinline__ void next_row(const Rows &r) {
        ch = 0;
        if (++vh < r.rows) return;
        vh = 0;
        do ++b;
        while (r.pre[b + 1] == r.pre[b]);
        nch = r.units(b) - kRowCost;
        len = r.lens[b];
    }
};

template <class P>
__device__ __forceinline__ void write_out(const AttendArgs &p, int b, int head, int d, float x, float y, float inv) {
    using T = typename P::T;
    if (d >= p.a.head_dim) return;
    T *out = static_cast<T *>(p.a.out) + b * p.a.out_stride[0] + head * p.a.out_stride[1] + d;
    if (p.out_pairs) {
        Vec<T, 2> v;
        v.v[0] = from_float<T>(x * inv), v.v[1] = from_float<T>(y * inv);
        *reinterpret_cast<Vec<T, 2> *>(out) = v;
    } else {
        out[0] = from_float<T>(x * inv), out[1] = from_float<T>(y * inv);
    }
}
// no weight at all: zeros (a NaN stays)
__device__ __forceinline__ float inverse(float l) { return l == 0.0f ? 0.0f : 1.0f / l; }
template <class P>
__device__ __forceinline__ void write_lse(const AttendArgs &p, int b, int head, float m, float l) {
    if (p.a.lse) p.a.lse[(int64_t)b * p.a.q_heads + head] = l == 0.0f ? -INFINITY : fmaf(m, p.scale2, log2f(l) - P::LIFT) * kLn2;
}

// Prefix sums of the requests' chunks into shared memory, with their lengths.
template <class P>
__device__ __forceinline__ Rows load_rows(const AttendArgs &p, char *smem) {
    constexpr int NT = P::NW * 32;
    __shared__ uint32_t warp_sum[P::NW];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t *pre = reinterpret_cast<uint32_t *>(smem);
    int32_t *lens = reinterpret_cast<int32_t *>(smem) + P::SLICE + 1;
    uint32_t carry = 0;
    for (int b0 = 0; b0 < p.a.batch; b0 += NT) {
        const int b = b0 + threadIdx.x;
        uint32_t n = 0;
        if (b < p.a.batch) {
            const int given = p.a.lens[b];
            const int len = given < 0 ? 0 : (int)min((long long)given, (long long)p.a.max_pages * p.a.page_size);
            if (blockIdx.x == 0 && len != given) atomicOr(p.a.status, kBadLength);
            n = len ? ((uint32_t)((len + P::CH - 1) / P::CH) + kRowCost) * p.rows : 0;
            lens[b] = len;
        }
        uint32_t scan = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t up = __shfl_up_sync(0xffffffffu, scan, d);
            if (lane >= d) scan += up;
        }
        if (lane == 31) warp_sum[warp] = scan;
        __syncthreads();
        uint32_t start = carry + scan - n;
#pragma unroll
        for (int w = 0; w < P::NW; ++w) {
            const uint32_t s = warp_sum[w];
            if (w < warp) start += s;
            carry += s;
        }
        if (b < p.a.batch) pre[b] = start;
        __syncthreads();
    }
    if (threadIdx.x == 0) pre[p.a.batch] = carry;
    __syncthreads();
    return Rows{pre, lens, p.a.batch, p.rows};
}

// Parts of a row that a block holds, in warps first .. last.
struct Part {
    int first, last;
    bool before, ended;  // the row begins in an earlier block; it ends in this one
    int b, vh;
};

// One warp joins `count` parts of a row for head g of its tile: part i has
// weight 2^((m_i - max m) scale2), and its record is at from + i * step + FLOATS, the
// last one's, if the row ends there, at from + i * step.  Writes the head's
// output, or the parts' sum to `to`.  GLOBAL: other blocks wrote the records,
// so they are read past L1.
template <class P, bool GLOBAL>
__device__ __forceinline__ void join(const AttendArgs &p, const float *from, int64_t step, const Part &part, int count, bool ended,
                                     int g, int lane, float *to) {
    using R = Record<P>;
    const int c = part.vh / p.tiles, t = part.vh - c * p.tiles, head = c * p.group + t * P::GT + g;
    if (g >= min(P::GT, p.group - t * P::GT)) return;
    auto record = [&](int i) { return from + i * step + (ended && i == count - 1 ? 0 : R::FLOATS); };
    auto one = [&](const float *at) { return GLOBAL ? __ldcg(at) : *at; };
    auto four = [&](const float *at) {
        return GLOBAL ? __ldcg(reinterpret_cast<const float4 *>(at)) : *reinterpret_cast<const float4 *>(at);
    };
    float m = -INFINITY, l = 0.0f;
    for (int i = lane; i < count; i += 32) m = fmaxf(m, one(record(i) + P::GT * R::ROW + g));
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    constexpr int QUADS = P::DP / 4, PER = (QUADS + 31) / 32;  // quads of elements, of a lane
    float4 sum[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) sum[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int i0 = 0; i0 < count; i0 += 32) {
        float w = 0.0f;
        if (i0 + lane < count) {
            const float *rec = record(i0 + lane) + P::GT * R::ROW + g;
            w = worth(one(rec), m, p.scale2);
            l = fmaf(w, one(rec + P::GT), l);
        }
        const int n = min(32, count - i0);
#pragma unroll 8
        for (int i = 0; i < n; ++i) {
            const float wi = __shfl_sync(0xffffffffu, w, i);
            const float *rec = record(i0 + i) + g * R::ROW;
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                const int quad = lane + 32 * j;
                if (QUADS % 32 == 0 || quad < QUADS) {
                    const float4 v = four(rec + 4 * quad);
                    sum[j].x = fmaf(wi, v.x, sum[j].x), sum[j].y = fmaf(wi, v.y, sum[j].y);
                    sum[j].z = fmaf(wi, v.z, sum[j].z), sum[j].w = fmaf(wi, v.w, sum[j].w);
                }
            }
        }
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
    const float inv = inverse(l);
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int d = 4 * (lane + 32 * j);
        if (QUADS % 32 != 0 && d >= P::DP) break;
        if (to) {
            *reinterpret_cast<float4 *>(to + g * R::ROW + d) = sum[j];
        } else {
            write_out<P>(p, part.b, head, d, sum[j].x, sum[j].y, inv);
            write_out<P>(p, part.b, head, d + 2, sum[j].z, sum[j].w, inv);
        }
    }
    if (lane == 0) {
        if (to) to[P::GT * R::ROW + g] = m, to[P::GT * R::ROW + P::GT + g] = l;
        else write_lse<P>(p, part.b, head, m, l);
    }
}

template <class P>
__global__ void __launch_bounds__(P::NW * 32, 1) paged_attention_kernel(typename P::Args p) {
    using R = Record<P>;
    using T = typename P::T;
    constexpr int NT = P::NW * 32;
    constexpr uint32_t FULL = FULL_MASK<P::CH>;
    enum { kFresh = 1, kBefore = 2, kRowEnd = 4, kShareEnd = 8 };
    extern __shared__ __align__(kSmemAlign) char smem[];
    __shared__ int4 notes[P::NW][P::STAGES];  // a stage's request, row, mask of positions, flags
    __shared__ int has[P::NW];                // bit 0: a head record, 1: a tail record, 2: its row began in an earlier warp
    __shared__ int rows_of[P::NW][4];         // head record's request and row, tail record's
    __shared__ Part parts[P::NW + 1];
    __shared__ int num_parts, last_arrived[2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    char *mine = smem + R::PREFIX + warp * R::WARP;
    char *qs = mine + P::STAGES * R::STAGE;
    after_previous();
    const Rows rows = load_rows<P>(p, smem);
    for (int b = blockIdx.x; b < p.a.batch; b += gridDim.x) {
        if (rows.pre[b + 1] != rows.pre[b]) continue;  // nothing to attend to: zeros
        T *out = static_cast<T *>(p.a.out) + b * p.a.out_stride[0];
        for (int e = threadIdx.x; e < p.a.q_heads * p.a.head_dim; e += NT)
            out[e / p.a.head_dim * p.a.out_stride[1] + e % p.a.head_dim] = zero_of<T>();
        for (int h = threadIdx.x; p.a.lse && h < p.a.q_heads; h += NT) p.a.lse[(int64_t)b * p.a.q_heads + h] = -INFINITY;
    }
    const uint32_t total = rows.pre[p.a.batch], share = (total + gridDim.x - 1) / gridDim.x;
    const uint32_t block0 = rows.cut(min(blockIdx.x * share, total), kBlockRow);
    const uint32_t block1 = rows.cut(min((blockIdx.x + 1) * share, total), kBlockRow);
    if (block0 >= block1) return;  // the whole block
    const uint32_t warp_share = (block1 - block0 + P::NW - 1) / P::NW;
    auto warp_cut = [&](int w) {
        const uint32_t c = block0 + w * warp_share;
        return w == 0 ? block0 : c >= block1 ? block1 : rows.cut(c, kWarpRow);
    };
    const uint32_t begin = warp_cut(warp), end = warp_cut(warp + 1);
    if (p.a.head_dim < P::DP) {  // the copies never write a row's padding: K's has to be zero
        for (int i = lane * 16; i < P::STAGES * R::STAGE; i += 512) *reinterpret_cast<uint4 *>(mine + i) = make_uint4(0, 0, 0, 0);
        __syncwarp();
    }

    P tile;

    // ---- the chunks to copy.  Under load a read takes longer than a chunk's
    // work, so what the next copies need is read well before: the pages in
    // batches of 32 units (a unit is PAGE_UNIT positions where these lie in one
    // page, else one), the next request's first batch, and the next
    // row's queries.
    Place load{};
    uint32_t at = 0;            // the next chunk's unit
    int32_t pages = 0, more_pages = 0, first_pages = 0, next_request_pages = 0;
    int base = 0;               // the first unit of `pages`
    int fetched_b = -1, fetched_vh = 0;  // the row whose queries are on their way
    int64_t kv_head = 0;
    bool live = begin < end, opened = true;
    const int tok = lane % P::CH;
    const bool one_page = p.a.page_size % P::PAGE_UNIT == 0;
    const int unit = one_page ? P::CH / P::PAGE_UNIT : P::CH;  // units in a chunk
    auto page_at = [&](int pos) { return (int)((__umulhi((uint32_t)pos, p.page_mul) + (uint32_t)pos) >> p.page_shift); };
    // this lane's entry of the batch of request b that begins at unit u
    auto read_pages = [&](int b, int len, int u) {
        const int64_t pos = (int64_t)(u + lane) * (one_page ? P::PAGE_UNIT : 1);
        return pos < len ? p.a.table[b * p.a.table_stride + page_at((int)pos)] : -1;
    };
    auto read_next_request = [&] {
        int b = load.b + 1;
        while (b < rows.batch && rows.pre[b + 1] == rows.pre[b]) ++b;
        next_request_pages = b < rows.batch ? read_pages(b, rows.lens[b], 0) : -1;
    };
    auto enter_row = [&] {
        kv_head = load.vh / p.tiles;
        if (P::AHEAD && fetched_b < 0) {
            const int t = load.vh % p.tiles;
            tile.fetch(p, load.b, (int)kv_head * p.group + t * P::GT, min(P::GT, p.group - t * P::GT), lane);
            fetched_b = load.b, fetched_vh = load.vh;
        }
    };
    // copies chunk `at` into a stage and moves on
    using C = typename P::Cache;
    constexpr int PER = 16 / sizeof(C), VPR = P::DP / PER;  // elements in a copy, copies in a row
    auto copy = [&](int stage) {
        const int pos = (int)load.ch * P::CH + tok;
        const int32_t page = __shfl_sync(0xffffffffu, pages, (int)load.ch * unit - base + (one_page ? tok / P::PAGE_UNIT : tok));
        const bool in = pos < load.len, real = in && (uint32_t)page < (uint32_t)p.a.num_pages;
        const uint32_t mask = __ballot_sync(0xffffffffu, real) & FULL;
        const bool row_end = load.ch + 1 == load.nch;
        if (lane == 0)
            notes[warp][stage] = make_int4(load.b, load.vh, (int)mask,
                                           (opened || load.ch == 0 ? kFresh : 0) | (opened && load.ch != 0 ? kBefore : 0) |
                                               (row_end ? kRowEnd : 0) | (at + 1 == end ? kShareEnd : 0));
        opened = false;
        const int inside = pos - page_at(pos) * p.a.page_size;
        const uint32_t dst = smem_addr(mine + stage * R::STAGE);
        if constexpr (P::SCALES) {
            const int64_t pg = real ? page : 0;
            const uint32_t in0 = real ? inside : 0, bl = (__umulhi(in0, p.scales.mul) + in0) >> p.scales.shift;
            if (lane < P::CH) {
                const AttendScales &s = p.scales;
                copy4(dst + R::KV + lane * 4, s.k + pg * s.k_stride[0] + bl * s.k_stride[1] + kv_head * s.k_stride[2], real);
                copy4(dst + R::KV + (P::CH + lane) * 4, s.v + pg * s.v_stride[0] + bl * s.v_stride[1] + kv_head * s.v_stride[2], real);
            }
        }
        if (32 % VPR == 0 && one_page && mask == FULL) {
            // a whole chunk: in a unit row r is r strides after row 0, and neighbouring lanes copy neighbours
            constexpr int STEP = 32 / VPR > 0 ? 32 / VPR : 1;  // rows a warp copies at once
            const int row0 = lane / VPR, col = lane % VPR;
            const int64_t kstep = STEP * p.a.k_stride[1], vstep = STEP * p.a.v_stride[1];
#pragma unroll
            for (int h = 0; h < P::CH / P::PAGE_UNIT; ++h) {
                const int64_t page_h = __shfl_sync(0xffffffffu, page, h * P::PAGE_UNIT);
                const int64_t in0 = __shfl_sync(0xffffffffu, inside, h * P::PAGE_UNIT) + row0;
                const C *ks = static_cast<const C *>(p.a.k_cache) + page_h * p.a.k_stride[0] + in0 * p.a.k_stride[1] +
                              kv_head * p.a.k_stride[2] + col * PER;
                const C *vs = static_cast<const C *>(p.a.v_cache) + page_h * p.a.v_stride[0] + in0 * p.a.v_stride[1] +
                              kv_head * p.a.v_stride[2] + col * PER;
                const uint32_t to = dst + (h * P::PAGE_UNIT + row0) * P::PITCH + col * 16;
                if (col * PER < p.a.head_dim) {
#pragma unroll
                    for (int i = 0; i < P::PAGE_UNIT / STEP; ++i) {
                        copy16(to + i * STEP * P::PITCH, ks, true);
                        copy16(to + (P::CH + i * STEP) * P::PITCH, vs, true);
                        ks += kstep, vs += vstep;
                    }
                }
            }
        } else {
            // row by row, each position's offsets from its lane; neighbouring lanes copy neighbours here too (each
            // lane copying a share of its own position's row took 313 us instead of 268 with 64-element heads
            // and 7 positions a page, 130 instead of 82 with one)
            if (in && !real && lane < P::CH) atomicOr(p.a.status, kBadPage);
            const int64_t pg = real ? page : 0, in0 = real ? inside : 0;
            const int64_t ko = pg * p.a.k_stride[0] + in0 * p.a.k_stride[1] + kv_head * p.a.k_stride[2];
            const int64_t vo = pg * p.a.v_stride[0] + in0 * p.a.v_stride[1] + kv_head * p.a.v_stride[2];
            const C *kc = static_cast<const C *>(p.a.k_cache), *vc = static_cast<const C *>(p.a.v_cache);
#pragma unroll
            for (int i = 0; i < P::CH * VPR / 32; ++i) {
                const int e = lane + 32 * i, row = e / VPR, col = e % VPR;
                const int64_t kr = __shfl_sync(0xffffffffu, ko, row);
                int64_t vr = kr;
                if (!p.same_strides) vr = __shfl_sync(0xffffffffu, vo, row);
                const bool there = (mask >> row) & 1;
                const uint32_t to = dst + row * P::PITCH + col * 16;
                if (col * PER < p.a.head_dim) {
                    copy16(to, kc + kr + col * PER, there);
                    copy16(to + P::CH * P::PITCH, vc + vr + col * PER, there);
                }
            }
        }
        if (++at >= end) {
            live = false;
        } else if (row_end) {
            at += kRowCost;
            const int b = load.b;
            load.next_row(rows);
            if (load.b != b) {
                first_pages = next_request_pages;
                read_next_request();
            }
            base = 0, pages = first_pages;
            more_pages = read_pages(load.b, load.len, 32);
            enter_row();
        } else {
            ++load.ch;
            if ((int)load.ch * unit - base == 32) {
                base += 32, pages = more_pages;
                more_pages = read_pages(load.b, load.len, base + 32);
            }
        }
    };
    if (live) {
        at = load.find(rows, begin);
        base = (int)load.ch * unit & ~31;
        pages = read_pages(load.b, load.len, base);
        more_pages = read_pages(load.b, load.len, base + 32);
        first_pages = base == 0 ? pages : read_pages(load.b, load.len, 0);
        read_next_request();
        enter_row();
    }

    // ---- the chunks copied
    auto write_record = [&](float *rec, int heads) {
        tile.each(lane, [&](int g, int d, float x, float y, float) {
            if (g < heads) *reinterpret_cast<float2 *>(rec + g * R::ROW + d) = make_float2(x, y);
        });
        tile.each_head(lane, [&](int g, float m, float l) {
            rec[P::GT * R::ROW + g] = m;
            rec[P::GT * R::ROW + P::GT + g] = l;
        });
    };
    float *head_rec = p.warp_rec + (int64_t)(blockIdx.x * P::NW + warp) * R::FLOATS;
    float *recs = reinterpret_cast<float *>(mine);  // both records, in the stages when these hold nothing any more
    int copied = 0, flags = 0, h0 = 0, heads = 0;  // of the present row
    auto heads_of = [&](int vh) {
        const int c = vh / p.tiles, t = vh - c * p.tiles;
        h0 = c * p.group + t * P::GT, heads = min(P::GT, p.group - t * P::GT);
    };
#pragma unroll
    for (int s = 0; s < P::STAGES - 1; ++s) {
        if (live) copy(s), ++copied;
        copy_commit();
    }
    bool before = false;  // the present row began in an earlier warp
    int stage = 0;
    for (int done = 0; done < copied; ++done) {
        if (live) copy(stage == 0 ? P::STAGES - 1 : stage - 1), ++copied;
        copy_commit();
        copy_wait<P::STAGES - 1>();
        __syncwarp();
        const int4 note = notes[warp][stage];
        if (note.w & kFresh) {
            heads_of(note.y);
            tile.begin(p, note.x, h0, heads, qs, lane, note.x == fetched_b && note.y == fetched_vh);
            fetched_b = -1;
            before = note.w & kBefore;
            __syncwarp();  // lanes without a head read nothing; the chunk's first instruction wants the whole warp
        }
        tile.chunk(p, mine + stage * R::STAGE, qs, (uint32_t)note.z, lane);
        __syncwarp();
        stage = stage + 1 == P::STAGES ? 0 : stage + 1;
        if (!(note.w & (kRowEnd | kShareEnd))) continue;
        tile.sums();
        if (!(note.w & kRowEnd)) {  // the last chunk
            flags |= before ? 6 : 2;
            if (lane == 0) rows_of[warp][2] = note.x, rows_of[warp][3] = note.y;
            write_record(recs + R::FLOATS, heads);
        } else if (before) {
            flags |= 1;
            if (lane == 0) rows_of[warp][0] = note.x, rows_of[warp][1] = note.y;
            write_record(head_rec, heads);
        } else {
            tile.each(lane, [&](int g, int d, float x, float y, float l) {
                if (g < heads) write_out<P>(p, note.x, h0 + g, d, x, y, inverse(l));
            });
            tile.each_head(lane, [&](int g, float m, float l) {
                if (g < heads) write_lse<P>(p, note.x, h0 + g, m, l);
            });
        }
    }
    copy_wait<0>();
    if (flags & 1) {
        __syncwarp();
#pragma unroll 8
        for (int e = lane; e < R::FLOATS / 4; e += 32)
            reinterpret_cast<float4 *>(recs)[e] = reinterpret_cast<const float4 *>(head_rec)[e];
    }
    if (lane == 0) has[warp] = flags;
    __syncthreads();

    // ---- the rows cut between this block's warps, and between blocks
    if (threadIdx.x == 0) {
        int n = 0, open = -1, tail = 0;
        bool from_before = false;
        for (int w = 0; w < P::NW; ++w) {
            if (open < 0 && (has[w] & 5)) open = w, from_before = true;  // only the first warp with any chunk
            if (open >= 0 && (has[w] & 1)) {
                parts[n++] = Part{open, w, from_before, true, rows_of[w][0], rows_of[w][1]};
                open = -1, from_before = false;
            }
            if ((has[w] & 6) == 2) open = w;
            if (has[w] & 2) tail = w;
        }
        if (open >= 0) parts[n++] = Part{open, tail, from_before, false, rows_of[tail][2], rows_of[tail][3]};
        num_parts = n;
        last_arrived[0] = last_arrived[1] = -1;
    }
    __syncthreads();
    const int most_heads = min(P::GT, p.group);
    for (int i = warp; i < num_parts * most_heads; i += P::NW) {
        const Part part = parts[i / most_heads];
        const float *from = reinterpret_cast<const float *>(smem + R::PREFIX + part.first * R::WARP);
        float *to = part.ended && !part.before ? nullptr : p.block_rec + ((int64_t)blockIdx.x * 2 + (part.ended ? 0 : 1)) * R::FLOATS;
        join<P, false>(p, from, R::WARP / 4, part, part.last - part.first + 1, part.ended, i % most_heads, lane, to);
    }
    if (num_parts == 0) return;
    const bool cut_before = parts[0].before, cut_after = !parts[num_parts - 1].ended;
    if (!cut_before && !cut_after) return;
    __threadfence();
    __syncthreads();
    // the blocks that hold a row's first and last chunk: cuts up to its first chunk move to its begin
    auto blocks_of = [&](const Part &part, int &first, int &last) {
        const uint32_t n = rows.units(part.b), start = rows.pre[part.b] + part.vh * n;
        first = (int)((start + kRowCost) / share);
        last = (int)((start + n - 1) / share);
    };
    if (threadIdx.x == 0) {
        for (int side = 0; side < 2; ++side) {
            const Part &part = parts[side ? num_parts - 1 : 0];
            if (side ? !cut_after || (cut_before && num_parts == 1) : !cut_before) continue;
            int first, last;
            blocks_of(part, first, last);
            if (atomicAdd(p.arrivals + first, 1) == last - first) {
                p.arrivals[first] = 0;  // for the next call
                last_arrived[side] = side ? num_parts - 1 : 0;
            }
        }
        __threadfence();
    }
    __syncthreads();
    for (int side = 0; side < 2; ++side) {
        if (last_arrived[side] < 0) continue;
        const Part part = parts[last_arrived[side]];
        int first, last;
        blocks_of(part, first, last);
        for (int g = warp; g < most_heads; g += P::NW)
            join<P, true>(p, p.block_rec + (int64_t)first * 2 * R::FLOATS, 2 * R::FLOATS, part, last - first + 1, true, g, lane, nullptr);
    }
}

// ------------------------------------------------------------ launch
constexpr size_t align16(size_t v) { return (v + 15) / 16 * 16; }

template <class P>
size_t workspace_of(int blocks) {
    return align16(4 * (size_t)blocks) + 4 * (size_t)Record<P>::FLOATS * blocks * (P::NW + 2);
}

template <class P>
cudaError_t launch_attention(const spmv_paged_attention_t &a, int sms, cudaStream_t stream, const AttendScales *scales = nullptr) {
    using R = Record<P>;
    using T = typename P::T;
    typename P::Args p;
    if constexpr (P::SCALES) p.scales = *scales;
    p.a = a;
    p.group = a.q_heads / a.kv_heads;
    p.tiles = (p.group + P::GT - 1) / P::GT;
    p.rows = a.kv_heads * p.tiles;
    p.scale2 = std::fabs(a.scale) * kLog2e;
    if constexpr (P::SCALES) p.scale2 = std::max(p.scale2, FLT_MIN);  // minus infinity times it has no weight
    p.flip = a.scale < 0.0f ? 0x80008000u : 0u;
    const int size = sizeof(T);
    auto pairs = [&](const void *at, const int64_t *strides) {  // pairs of elements are aligned
        return aligned_to(at, 2 * size) && strides[0] % 2 == 0 && strides[1] % 2 == 0;
    };
    p.q_pairs = pairs(a.q, a.q_stride);
    p.out_pairs = pairs(a.out, a.out_stride);
    p.same_strides = std::equal(a.k_stride, a.k_stride + 3, a.v_stride);
    set_divisor((uint32_t)a.page_size, &p.page_mul, &p.page_shift);
    char *w = static_cast<char *>(a.workspace);
    p.arrivals = reinterpret_cast<int32_t *>(w);
    p.warp_rec = reinterpret_cast<float *>(w + align16(4 * (size_t)sms));
    p.block_rec = p.warp_rec + (int64_t)sms * P::NW * R::FLOATS;
    cudaError_t e = cudaFuncSetAttribute(paged_attention_kernel<P>, cudaFuncAttributeMaxDynamicSharedMemorySize, R::SMEM);
    // a launch's units are counted in 32 bits
    const int64_t most = (((int64_t)a.max_pages * a.page_size + P::CH - 1) / P::CH + kRowCost) * p.rows;
    const int slice = (int)std::max<int64_t>(1, std::min<int64_t>(P::SLICE, ((1LL << 31) - 1) / std::max<int64_t>(1, most)));
    for (int b = 0; b < a.batch && e == cudaSuccess; b += slice) {
        p.a.batch = std::min(slice, a.batch - b);
        p.a.q = static_cast<const char *>(a.q) + (int64_t)b * a.q_stride[0] * size;
        p.a.out = static_cast<char *>(a.out) + (int64_t)b * a.out_stride[0] * size;
        p.a.lse = a.lse ? a.lse + (int64_t)b * a.q_heads : nullptr;
        p.a.table = a.table + b * a.table_stride;
        p.a.lens = a.lens + b;
        const int64_t blocks = std::min<int64_t>(sms, most * p.a.batch);
        e = launch_chained(paged_attention_kernel<P>, (unsigned)blocks, P::NW * 32, R::SMEM, 0, stream, p);
    }
    return e;
}

// Calls f with the tile of 16-bit elements T for the head size and group.
//
// Warps and stages: what an SM's registers and shared memory hold.  Of both
// measured ways for tiles of 8 heads (64 requests, their lengths even up to
// 4,000, 4 kv heads with 4 heads each, 16 positions a page, bf16, calls one
// after another): 96 elements (213 MB) 57.1 us with 10 warps of 3 stages, 58.5
// with 8 of 4; 128 elements (284 MB) 61.2 with 8 of 3, 65.9 with 10 of 2, whose
// registers do not suffice; 192 elements (426 MB) 89.3 with 8 of 2, 119.7 with
// 4 of 4; 256 elements (568 MB) 111.7 with 6 of 2, 116.4 with 4 of 3.  Tiles of
// 16 heads need their registers, and their records the stages' room.
template <typename T, int GT, typename F>
auto with_mma(int dim, F f) {
    constexpr bool small = GT == 8;
    if (dim <= 64) return f(TileMma<T, GT, 64, 32, 8, 3>());
    if (dim <= 96) return f(TileMma<T, GT, 96, 16, small ? 10 : 8, small ? 3 : 4>());
    if (dim <= 128) return f(TileMma<T, GT, 128, 16, 8, 3>());
    if (dim <= 192) return f(TileMma<T, GT, 192, 16, small ? 8 : 4, small ? 2 : 4>());
    return f(TileMma<T, GT, 256, 16, small ? 6 : 4, small ? 2 : 3>());
}
template <typename T, typename F>
auto with_mma(int dim, int group, F f) {
    return group <= 8 ? with_mma<T, 8>(dim, f) : with_mma<T, 16>(dim, f);
}

}  // namespace

}  // namespace lbcsr
