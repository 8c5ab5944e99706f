// Attention of one new token per request over a paged key-value cache:
//
//   s_t = scale <q, k_t>,  out = sum_t exp(s_t - m) v_t / sum_t exp(s_t - m)
//
// in one pass over the positions with the running maximum m and sum of the
// softmax: when a score above m comes, the sums so far are scaled by
// exp(m_old - m_new).  Scores are kept in units of ln 2, so the exponentials
// are powers of two.
//
// The work is a sparse product's with very uneven rows: row (request, kv
// head), one unit per chunk of positions.  Units in row order are cut into
// equal shares, one per warp, whatever the lengths (the merge-path SpMV's
// schedule).  Each warp is a pipeline of its own: it copies its next chunks
// into its part of shared memory (cp.async, several chunks in flight) while
// it works on the present one, across row ends, with no barrier in the loop.
// A row inside one share is written out by its warp; the parts of a row cut
// between warps are records (unnormalised sums, m and l per head) that the
// block joins in shared memory; the blocks' parts of a row cut between blocks
// are joined, in block order, by the last of them to arrive.  The order of
// every sum is fixed by the lengths, so results do not change between calls.
#pragma once

#include <algorithm>
#include <cmath>

#include "internal.cuh"
#include "llm.cuh"

namespace lbcsr {

// One translation unit per element type holds its kernels.  group: query
// heads per kv head.
size_t attention_workspace_f32(int dim, int group, int sms);
size_t attention_workspace_bf16(int dim, int group, int sms);
size_t attention_workspace_f16(int dim, int group, int sms);
cudaError_t launch_attention_f32(const spmv_paged_attention_t &a, int sms, cudaStream_t stream);
cudaError_t launch_attention_bf16(const spmv_paged_attention_t &a, int sms, cudaStream_t stream);
cudaError_t launch_attention_f16(const spmv_paged_attention_t &a, int sms, cudaStream_t stream);

namespace {

constexpr int kMaxDim = 256;
constexpr int kMaxSlice = 2048;  // requests per launch: their prefix sums live in shared memory
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
    int32_t *arrivals;   // [blocks], zero between calls
    float *warp_rec;     // [blocks * warps] records
    float *block_rec;    // [blocks][2] records
};

__device__ __forceinline__ uint32_t smem_addr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
// 16 bytes from global to shared memory; zeros when !real (src is then not read)
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool real) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
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

// 2^x by the hardware's instruction: 2 units in the last place, results
// below 2^-126 are zero (next to a row's largest weight of 1)
__device__ __forceinline__ float pow2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// what scores are taken relative to; the running maximum m is -infinity
// until a score has come, and nothing has weight then
__device__ __forceinline__ float base_of(float m) { return m == -INFINITY ? 0.0f : m; }

// ------------------------------------------------------------ 16-bit elements
// A chunk is 16 positions; a tile is 8 or 16 query heads of one kv head.  The
// scores are one 16 x 16 product per chunk (heads by positions) and the
// output one 16 x DP product, on the warp's matrix instructions with 32-bit
// sums.  The weights go into the second product as hi + lo, two elements of
// the caches' type (p - hi is exact in 32 bits), so they carry 16 (bf16) or
// 22 (f16) bits: with hi alone the output's error against 64 bits is 1.4
// times that of one rounding.  A tile of 8 heads has hi in the product's
// first 8 rows and lo in its last 8, and so costs no more than hi alone.
template <typename T_, int GT_, int DP_, int NW_, int STAGES_>
struct TileMma {
    using T = T_;
    static constexpr int DP = DP_, NW = NW_, STAGES = STAGES_, GT = GT_, CH = 16;
    static constexpr int PITCH = DP * 2 + 16;  // bytes: rows 16 bytes apart modulo 128, so ldmatrix has no conflicts
    static constexpr int QBYTES = 0;
    static constexpr int H = GT / 8;  // heads of a lane: lane / 4 and, with 16, lane / 4 + 8

    uint32_t q[DP / 16][2 * H];
    float o[DP / 8][4];
    float m[H], l[H];  // l: this lane's part of the sum

    __device__ __forceinline__ void begin(const AttendArgs &p, int b, int h0, int heads, char *, int lane) {
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
                    const bool real = head < heads && d < p.a.head_dim;
                    q[s][r * H + h] = real ? pack2(at[0], at[1]) ^ p.flip : 0u;
                }
#pragma unroll
        for (int n = 0; n < DP / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.0f;
#pragma unroll
        for (int h = 0; h < H; ++h) m[h] = -INFINITY, l[h] = 0.0f;
    }

    __device__ __forceinline__ void chunk(const AttendArgs &p, const char *stage, const char *, uint32_t mask, int lane) {
        const uint32_t ks = smem_addr(stage), vs = ks + CH * PITCH;
        const int r8 = lane & 7, mat = lane >> 3;
        // scores of positions 0-7 and 8-15, each in two sums that do not wait for one another
        float sums[2][2][4] = {};
        {
            const uint32_t at = ks + (r8 + (mat >> 1) * 8) * PITCH + (mat & 1) * 16;
#pragma unroll
            for (int i = 0; i < DP / 16; ++i) {
                uint32_t kb[4];
                ldmatrix4(at + i * 32, kb);
                const uint32_t qa[4] = {q[i][0], H == 2 ? q[i][H - 1] : 0u, q[i][H], H == 2 ? q[i][2 * H - 1] : 0u};
                mma16816<T>(sums[i & 1][0], qa, kb[0], kb[1]);
                mma16816<T>(sums[i & 1][1], qa, kb[2], kb[3]);
            }
        }
        const bool whole = mask == 0xffffu;
        uint32_t hi[2 * H], lo[2 * H];  // [positions 0-7, 8-15][head]
        float s[2][H][2], top[H];
        bool higher = false;
#pragma unroll
        for (int h = 0; h < H; ++h) {
            float raw = -INFINITY;
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    s[n][h][c] = sums[0][n][2 * h + c] + sums[1][n][2 * h + c];
                    if (!whole && !((mask >> (n * 8 + (lane & 3) * 2 + c)) & 1)) s[n][h][c] = -INFINITY;
                    raw = fmaxf(raw, s[n][h][c]);
                }
            raw = fmaxf(raw, __shfl_xor_sync(0xffffffffu, raw, 1));
            raw = fmaxf(raw, __shfl_xor_sync(0xffffffffu, raw, 2));
            top[h] = fmaxf(m[h], raw * p.scale2);
            higher |= top[h] > m[h];
        }
        if (__any_sync(0xffffffffu, higher)) {
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const float keep = pow2(m[h] - base_of(top[h]));
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
            for (int n = 0; n < 2; ++n) {
                float w[2];
                T high[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    w[c] = pow2(fmaf(s[n][h][c], p.scale2, -base));
                    if (!whole && !((mask >> (n * 8 + (lane & 3) * 2 + c)) & 1)) w[c] = 0.0f;
                    high[c] = from_float<T>(w[c]);
                }
                l[h] += w[0] + w[1];
                hi[n * H + h] = pack2(high[0], high[1]);
                lo[n * H + h] = pack2(from_float<T>(w[0] - to_float(high[0])), from_float<T>(w[1] - to_float(high[1])));
            }
        }
        const uint32_t at = vs + (r8 + (mat & 1) * 8) * PITCH + (mat >> 1) * 16;
        if (H == 1) {
            const uint32_t pa[4] = {hi[0], lo[0], hi[1], lo[1]};
#pragma unroll
            for (int i = 0; i < DP / 16; ++i) {
                uint32_t vb[4];
                ldmatrix4_t(at + i * 32, vb);
                mma16816<T>(o[2 * i], pa, vb[0], vb[1]);
                mma16816<T>(o[2 * i + 1], pa, vb[2], vb[3]);
            }
        } else {
            const uint32_t ph[4] = {hi[0], hi[H - 1], hi[H], hi[2 * H - 1]}, pl[4] = {lo[0], lo[H - 1], lo[H], lo[2 * H - 1]};
#pragma unroll
            for (int i = 0; i < DP / 16; ++i) {
                uint32_t vb[4];
                ldmatrix4_t(at + i * 32, vb);
                mma16816<T>(o[2 * i], ph, vb[0], vb[1]);
                mma16816<T>(o[2 * i + 1], ph, vb[2], vb[3]);
                mma16816<T>(o[2 * i], pl, vb[0], vb[1]);
                mma16816<T>(o[2 * i + 1], pl, vb[2], vb[3]);
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

    // f(head, d, value at d, value at d + 1, l)
    template <typename F>
    __device__ __forceinline__ void each(int lane, F f) const {
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
            for (int n = 0; n < DP / 8; ++n) {
                const float x = H == 1 ? o[n][0] + o[n][2] : o[n][2 * h], y = H == 1 ? o[n][1] + o[n][3] : o[n][2 * h + 1];
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
// matrix instruction that keeps 32-bit inputs whole.
template <int DP_, int GT_, int NW_, int STAGES_>
struct TileF32 {
    using T = float;
    static constexpr int DP = DP_, NW = NW_, STAGES = STAGES_, GT = GT_, CH = 8;
    static constexpr int PITCH = DP * 4 + 16;
    static constexpr int QBYTES = GT * DP * 4;

    float2 o[GT][DP / 64];
    float m[GT], l[GT];

    __device__ __forceinline__ void begin(const AttendArgs &p, int b, int h0, int heads, char *qs, int lane) {
        const float *base = static_cast<const float *>(p.a.q) + b * p.a.q_stride[0] + h0 * p.a.q_stride[1];
        float *q = reinterpret_cast<float *>(qs);
        __syncwarp();
#pragma unroll
        for (int g = 0; g < GT; ++g) {
            for (int d = lane; d < DP; d += 32)
                q[g * DP + d] = g < heads && d < p.a.head_dim ? (p.flip ? -1.0f : 1.0f) * base[g * p.a.q_stride[1] + d] : 0.0f;
#pragma unroll
            for (int i = 0; i < DP / 64; ++i) o[g][i] = make_float2(0.0f, 0.0f);
            m[g] = -INFINITY;
            l[g] = 0.0f;
        }
        __syncwarp();
    }

    __device__ __forceinline__ void chunk(const AttendArgs &p, const char *stage, const char *qs, uint32_t mask, int lane) {
        const int pos = lane & 7, quarter = lane >> 3;
        const float4 *k = reinterpret_cast<const float4 *>(stage + pos * PITCH) + quarter * (DP / 16);
        const float4 *q = reinterpret_cast<const float4 *>(qs) + quarter * (DP / 16);
        float s[GT];
#pragma unroll
        for (int g = 0; g < GT; ++g) s[g] = 0.0f;
#pragma unroll
        for (int i = 0; i < DP / 16; ++i) {
            const float4 kv = k[i];
#pragma unroll
            for (int g = 0; g < GT; ++g) {
                const float4 qv = q[g * (DP / 4) + i];
                s[g] = fmaf(qv.x, kv.x, fmaf(qv.y, kv.y, fmaf(qv.z, kv.z, fmaf(qv.w, kv.w, s[g]))));
            }
        }
        float pr[GT];
#pragma unroll
        for (int g = 0; g < GT; ++g) {
            s[g] += __shfl_xor_sync(0xffffffffu, s[g], 8);
            s[g] += __shfl_xor_sync(0xffffffffu, s[g], 16);
            const bool live = (mask >> pos) & 1;
            float top = live ? s[g] : -INFINITY;
#pragma unroll
            for (int d = 1; d < 8; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            top = fmaxf(m[g], top * p.scale2);
            const float base = base_of(top);
            if (top > m[g]) {  // the same on every lane
                const float keep = pow2(m[g] - base);
                l[g] *= keep;
#pragma unroll
                for (int i = 0; i < DP / 64; ++i) o[g][i].x *= keep, o[g][i].y *= keep;
                m[g] = top;
            }
            pr[g] = live ? pow2(fmaf(s[g], p.scale2, -base)) : 0.0f;
            if (quarter == 0) l[g] += pr[g];
        }
        const char *v = stage + CH * PITCH;
#pragma unroll
        for (int t = 0; t < CH; ++t) {
            float2 vv[DP / 64];
#pragma unroll
            for (int i = 0; i < DP / 64; ++i) vv[i] = reinterpret_cast<const float2 *>(v + t * PITCH)[lane + 32 * i];
#pragma unroll
            for (int g = 0; g < GT; ++g) {
                const float w = __shfl_sync(0xffffffffu, pr[g], t);
#pragma unroll
                for (int i = 0; i < DP / 64; ++i) {
                    o[g][i].x = fmaf(w, vv[i].x, o[g][i].x);
                    o[g][i].y = fmaf(w, vv[i].y, o[g][i].y);
                }
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
            for (int i = 0; i < DP / 64; ++i) f(g, 64 * i + 2 * lane, o[g][i].x, o[g][i].y, l[g]);
    }
    template <typename F>
    __device__ __forceinline__ void each_head(int lane, F f) const {
#pragma unroll
        for (int g = 0; g < GT; ++g)
            if (lane == 0) f(g, m[g], l[g]);
    }
};

// A record: GT rows of sums, then m and l of each head.
template <class P>
struct Record {
    static constexpr int ROW = P::DP + 8;  // the rows' first banks differ
    static constexpr int FLOATS = (P::GT * ROW + 2 * P::GT + 3) / 4 * 4;  // records are read 16 bytes at a time
    static constexpr int STAGE = 2 * P::CH * P::PITCH;                  // bytes of a chunk's K and V
    static constexpr int WARP = P::STAGES * STAGE + P::QBYTES;          // bytes of a warp's shared memory
    static_assert(2 * FLOATS * 4 <= P::STAGES * STAGE, "both records of a warp fit its stages");
    static_assert(FLOATS % 4 == 0 && ROW % 4 == 0 && P::PITCH % 16 == 0 && P::QBYTES % 16 == 0, "16-byte accesses");
    static constexpr int PREFIX = (4 * (kMaxSlice + 1) + 15) / 16 * 16;
    static constexpr int SMEM = PREFIX + P::NW * WARP;
};

// Where a warp is in its share: chunk ch of nch of row vh of request b.
struct Place {
    int b, vh;
    uint32_t ch, nch;
    int len;
};

__device__ __forceinline__ int clamped_len(const AttendArgs &p, int b) {
    const long long most = (long long)p.a.max_pages * p.a.page_size;
    const int len = __ldg(p.a.lens + b);
    return len < 0 ? 0 : (int)min((long long)len, most);
}

// The next chunk (only called while there is one).
__device__ __forceinline__ void next_row(const AttendArgs &p, const uint32_t *pre, Place &at) {
    at.ch = 0;
    if (++at.vh < p.rows) return;
    at.vh = 0;
    do ++at.b;
    while (pre[at.b + 1] == pre[at.b]);
    at.nch = (pre[at.b + 1] - pre[at.b]) / p.rows;
    at.len = clamped_len(p, at.b);
}

// Sums of records joined: record i has weight exp2(m_i - m); f gives record
// i's floats.  Writes head g's elements d .. d + 3 through out(g, d, values,
// l, m).
template <class P, typename Rec, typename Out>
__device__ __forceinline__ void join(int count, int heads, Rec rec, Out out) {
    for (int e = threadIdx.x; e < heads * (P::DP / 4); e += P::NW * 32) {
        const int g = e / (P::DP / 4), d = e % (P::DP / 4) * 4;
        float m = -INFINITY;
        for (int i = 0; i < count; ++i) m = fmaxf(m, rec(i, P::GT * Record<P>::ROW + g));
        const float base = base_of(m);
        float l = 0.0f;
        float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
        for (int i = 0; i < count; ++i) {
            const float w = pow2(rec(i, P::GT * Record<P>::ROW + g) - base);
            l = fmaf(w, rec(i, P::GT * Record<P>::ROW + P::GT + g), l);
            const float4 v = rec.quad(i, g * Record<P>::ROW + d);
            sum.x = fmaf(w, v.x, sum.x), sum.y = fmaf(w, v.y, sum.y);
            sum.z = fmaf(w, v.z, sum.z), sum.w = fmaf(w, v.w, sum.w);
        }
        out(g, d, sum, l, m);
    }
}

template <class P>
__device__ __forceinline__ void write_final(const AttendArgs &p, int b, int head, int d, const float *v, int n, float l,
                                            float m) {
    using T = typename P::T;
    T *out = static_cast<T *>(p.a.out) + b * p.a.out_stride[0] + head * p.a.out_stride[1] + d;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // no weight at all: zeros (a NaN stays)
    if (d < p.a.head_dim)
        for (int i = 0; i < n; ++i) out[i] = from_float<T>(v[i] * inv);
    if (d == 0 && p.a.lse) p.a.lse[(int64_t)b * p.a.q_heads + head] = (m + log2f(l)) * kLn2;
}

// Parts of a row that a block holds, in warps first .. last.
struct Part {
    int first, last;
    bool before, ended;  // the row begins in an earlier block; it ends in this one
    int b, vh;
};

template <class P>
__global__ void __launch_bounds__(P::NW * 32, 1) paged_attention_kernel(AttendArgs p) {
    using R = Record<P>;
    using T = typename P::T;
    constexpr int NT = P::NW * 32;
    extern __shared__ __align__(16) char smem[];
    __shared__ uint32_t warp_sum[P::NW];
    __shared__ uint32_t masks[P::NW][P::STAGES];
    __shared__ int has[P::NW];             // bit 0: a head record, 1: a tail record, 2: its row began in an earlier warp
    __shared__ int rows_of[P::NW][4];      // head record's request and row, tail record's
    __shared__ Part parts[P::NW + 1];
    __shared__ int num_parts, last_arrived[2];
    uint32_t *pre = reinterpret_cast<uint32_t *>(smem);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    char *mine = smem + R::PREFIX + warp * R::WARP;
    char *qs = mine + P::STAGES * R::STAGE;

    // ---- prefix sums of the requests' chunks
    uint32_t carry = 0;
    for (int b0 = 0; b0 < p.a.batch; b0 += NT) {
        const int b = b0 + threadIdx.x;
        uint32_t n = 0;
        if (b < p.a.batch) {
            const int len = clamped_len(p, b);
            n = (uint32_t)((len + P::CH - 1) / P::CH) * p.rows;
            if (blockIdx.x == 0 && len != __ldg(p.a.lens + b)) atomicOr(p.a.status, kBadLength);
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
    if (p.a.head_dim < P::DP) {  // the copies never write a row's padding: K's has to be zero
        for (int i = lane * 16; i < P::STAGES * R::STAGE; i += 512) *reinterpret_cast<uint4 *>(mine + i) = make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
    for (int b = blockIdx.x; b < p.a.batch; b += gridDim.x) {
        if (pre[b + 1] != pre[b]) continue;  // nothing to attend to: zeros
        T *out = static_cast<T *>(p.a.out) + b * p.a.out_stride[0];
        for (int e = threadIdx.x; e < p.a.q_heads * p.a.head_dim; e += NT)
            out[e / p.a.head_dim * p.a.out_stride[1] + e % p.a.head_dim] = zero_of<T>();
        for (int h = threadIdx.x; p.a.lse && h < p.a.q_heads; h += NT) p.a.lse[(int64_t)b * p.a.q_heads + h] = -INFINITY;
    }
    const uint32_t total = carry;
    const uint32_t share = (total + gridDim.x * P::NW - 1) / (gridDim.x * P::NW);
    const uint32_t block_share = share * P::NW;
    if (blockIdx.x * block_share >= total) return;  // the whole block
    const uint32_t c0 = min(blockIdx.x * block_share + warp * share, total), c1 = min(c0 + share, total);
    const int count = (int)(c1 - c0);

    // ---- this warp's share
    P tile;
    int flags = 0;
    if (count > 0) {
        Place load;
        {
            int lo = 0, hi = p.a.batch - 1;  // the first request with pre[b + 1] > c0
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (pre[mid + 1] > c0) hi = mid;
                else lo = mid + 1;
            }
            load.b = lo;
            load.nch = (pre[lo + 1] - pre[lo]) / p.rows;
            load.vh = (int)((c0 - pre[lo]) / load.nch);
            load.ch = (c0 - pre[lo]) % load.nch;
            load.len = clamped_len(p, lo);
        }
        Place work = load;
        const int tok = lane % P::CH;
        const bool one_page = p.a.page_size % P::CH == 0;  // every chunk lies in one page
        auto page_at = [&](int pos) { return (int)((__umulhi((uint32_t)pos, p.page_mul) + (uint32_t)pos) >> p.page_shift); };
        auto page_of = [&](const Place &at) {  // this lane's position's page, -1: none
            const int pos = (int)at.ch * P::CH + tok;
            return pos < at.len ? __ldg(p.a.table + at.b * p.a.table_stride + page_at(pos)) : -1;
        };
        int32_t page = page_of(load);
        int64_t head = load.vh / p.tiles;  // of `load`
        // copies chunk `load` into a stage and moves `load` on; `page` was loaded one chunk ahead
        constexpr int PER = 16 / sizeof(T), VPR = P::DP / PER;  // elements in a copy, copies in a row
        auto copy = [&](int stage, bool more) {
            const int first = (int)load.ch * P::CH, pos = first + tok;
            const bool in = pos < load.len, real = (uint32_t)page < (uint32_t)p.a.num_pages;
            const uint32_t mask = __ballot_sync(0xffffffffu, real) & ((1u << P::CH) - 1u);
            if (lane == 0) masks[warp][stage] = mask;
            const int inside = pos - page_at(pos) * p.a.page_size;
            const uint32_t dst = smem_addr(mine + stage * R::STAGE);
            if (one_page && mask == (1u << P::CH) - 1u) {
                // the whole chunk, in one page: row r is r strides after row 0
                const int row0 = lane / VPR, col = lane % VPR;
                const int64_t in0 = __shfl_sync(0xffffffffu, inside, 0) + row0;
                const T *ks = static_cast<const T *>(p.a.k_cache) + page * p.a.k_stride[0] + in0 * p.a.k_stride[1] +
                              head * p.a.k_stride[2] + col * PER;
                const T *vs = static_cast<const T *>(p.a.v_cache) + page * p.a.v_stride[0] + in0 * p.a.v_stride[1] +
                              head * p.a.v_stride[2] + col * PER;
                if (32 % VPR == 0) {
                    constexpr int STEP = 32 / VPR > 0 ? 32 / VPR : 1;  // rows a warp copies at once
                    const int64_t kstep = STEP * p.a.k_stride[1], vstep = STEP * p.a.v_stride[1];
                    const uint32_t to = dst + row0 * P::PITCH + col * 16;
                    if (col * PER < p.a.head_dim) {
#pragma unroll
                        for (int i = 0; i < P::CH / STEP; ++i) {
                            copy16(to + i * STEP * P::PITCH, ks, true);
                            copy16(to + (P::CH + i * STEP) * P::PITCH, vs, true);
                            ks += kstep, vs += vstep;
                        }
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < P::CH * VPR / 32; ++i) {
                        const int e = lane + 32 * i, row = e / VPR, c = e % VPR;
                        if (c * PER < p.a.head_dim) {
                            const uint32_t to = dst + row * P::PITCH + c * 16;
                            copy16(to, ks + (row - row0) * p.a.k_stride[1] + (c - col) * PER, true);
                            copy16(to + P::CH * P::PITCH, vs + (row - row0) * p.a.v_stride[1] + (c - col) * PER, true);
                        }
                    }
                }
            } else {
                if (in && !real && lane < P::CH) atomicOr(p.a.status, kBadPage);
                const int64_t pg = real ? page : 0;
                const int64_t ko = pg * p.a.k_stride[0] + inside * p.a.k_stride[1] + head * p.a.k_stride[2];
                const int64_t vo = pg * p.a.v_stride[0] + inside * p.a.v_stride[1] + head * p.a.v_stride[2];
#pragma unroll
                for (int i = 0; i < P::CH * VPR / 32; ++i) {
                    const int e = lane + 32 * i, row = e / VPR, col = e % VPR;
                    const int64_t kr = __shfl_sync(0xffffffffu, ko, row), vr = __shfl_sync(0xffffffffu, vo, row);
                    const bool live = (mask >> row) & 1;
                    if (col * PER < p.a.head_dim) {
                        const uint32_t to = dst + row * P::PITCH + col * 16;
                        copy16(to, static_cast<const T *>(p.a.k_cache) + (live ? kr + col * PER : 0), live);
                        copy16(to + P::CH * P::PITCH, static_cast<const T *>(p.a.v_cache) + (live ? vr + col * PER : 0), live);
                    }
                }
            }
            if (more) {
                if (++load.ch == load.nch) {
                    next_row(p, pre, load);
                    head = load.vh / p.tiles;
                }
                page = page_of(load);
            }
        };
        auto begin_row = [&] {
            const int c = work.vh / p.tiles, t = work.vh % p.tiles;
            tile.begin(p, work.b, c * p.group + t * P::GT, min(P::GT, p.group - t * P::GT), qs, lane);
        };
        auto write_record = [&](float *rec) {
            tile.sums();
            tile.each(lane, [&](int g, int d, float x, float y, float) {
                *reinterpret_cast<float2 *>(rec + g * R::ROW + d) = make_float2(x, y);
            });
            tile.each_head(lane, [&](int g, float m, float l) {
                rec[P::GT * R::ROW + g] = m;
                rec[P::GT * R::ROW + P::GT + g] = l;
            });
        };
        float *head_rec = p.warp_rec + (int64_t)(blockIdx.x * P::NW + warp) * R::FLOATS;
#pragma unroll
        for (int s = 0; s < P::STAGES - 1; ++s) {
            if (s < count) copy(s, s + 1 < count);
            copy_commit();
        }
        bool before = work.ch != 0;  // the present row began in an earlier warp
        begin_row();
        int stage = 0;
        for (int i = 0; i < count; ++i) {
            const int ahead = i + P::STAGES - 1;
            if (ahead < count) copy(stage == 0 ? P::STAGES - 1 : stage - 1, ahead + 1 < count);
            copy_commit();
            copy_wait<P::STAGES - 1>();
            __syncwarp();
            tile.chunk(p, mine + stage * R::STAGE, qs, masks[warp][stage], lane);
            __syncwarp();
            stage = stage + 1 == P::STAGES ? 0 : stage + 1;
            if (++work.ch < work.nch) continue;
            // the row ends here
            if (before) {
                write_record(head_rec);
                flags |= 1;
                if (lane == 0) rows_of[warp][0] = work.b, rows_of[warp][1] = work.vh;
                before = false;
            } else {
                const int c = work.vh / p.tiles, t = work.vh % p.tiles, h0 = c * p.group + t * P::GT;
                const int heads = min(P::GT, p.group - t * P::GT);
                tile.sums();
                tile.each(lane, [&](int g, int d, float x, float y, float l) {
                    const float v[2] = {x, y};
                    if (g < heads && d != 0) write_final<P>(p, work.b, h0 + g, d, v, 2, l, 0.0f);
                    else if (g < heads) {
                        T *out = static_cast<T *>(p.a.out) + work.b * p.a.out_stride[0] + (h0 + g) * p.a.out_stride[1];
                        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                        out[0] = from_float<T>(x * inv), out[1] = from_float<T>(y * inv);
                    }
                });
                if (p.a.lse)
                    tile.each_head(lane, [&](int g, float m, float l) {
                        if (g < heads) p.a.lse[(int64_t)work.b * p.a.q_heads + h0 + g] = (m + log2f(l)) * kLn2;
                    });
            }
            if (i + 1 < count) {
                next_row(p, pre, work);
                begin_row();
            }
        }
        copy_wait<0>();
        __syncwarp();
        // both records into this warp's stages, which hold nothing any more
        float *recs = reinterpret_cast<float *>(mine);
        if (work.ch < work.nch) {
            flags |= before ? 6 : 2;
            write_record(recs + R::FLOATS);
            if (lane == 0) rows_of[warp][2] = work.b, rows_of[warp][3] = work.vh;
        }
        if (flags & 1) {
            __syncwarp();
#pragma unroll 8
            for (int e = lane; e < R::FLOATS / 4; e += 32)
                reinterpret_cast<float4 *>(recs)[e] = reinterpret_cast<const float4 *>(head_rec)[e];
        }
    }
    if (lane == 0) has[warp] = flags;
    __syncthreads();

    // ---- the rows cut between this block's warps, and between blocks
    if (threadIdx.x == 0) {
        int n = 0, open = has[0] & 5 ? 0 : -1;
        bool before = open == 0;
        for (int w = 0; w < P::NW; ++w) {
            if (open >= 0 && (has[w] & 1)) {
                parts[n++] = Part{open, w, before, true, rows_of[w][0], rows_of[w][1]};
                open = -1, before = false;
            }
            if ((has[w] & 6) == 2) open = w;
        }
        if (open >= 0) parts[n++] = Part{open, P::NW - 1, before, false, rows_of[P::NW - 1][2], rows_of[P::NW - 1][3]};
        num_parts = n;
        last_arrived[0] = last_arrived[1] = -1;
    }
    __syncthreads();
    struct SharedRec {
        const char *base;
        Part part;
        __device__ __forceinline__ const float *at(int i) const {
            const int w = part.first + i;
            return reinterpret_cast<const float *>(base + w * R::WARP) + (w == part.last && part.ended ? 0 : R::FLOATS);
        }
        __device__ __forceinline__ float operator()(int i, int f) const { return at(i)[f]; }
        __device__ __forceinline__ float4 quad(int i, int f) const { return *reinterpret_cast<const float4 *>(at(i) + f); }
    };
    for (int n = 0; n < num_parts; ++n) {
        const Part part = parts[n];
        const int c = part.vh / p.tiles, t = part.vh % p.tiles, h0 = c * p.group + t * P::GT;
        const int heads = min(P::GT, p.group - t * P::GT);
        const SharedRec rec{smem + R::PREFIX, part};
        float *to = p.block_rec + ((int64_t)blockIdx.x * 2 + (part.ended ? 0 : 1)) * R::FLOATS;
        join<P>(part.last - part.first + 1, heads, rec, [&](int g, int d, float4 v, float l, float m) {
            if (part.ended && !part.before) {
                const float x[4] = {v.x, v.y, v.z, v.w};
                write_final<P>(p, part.b, h0 + g, d, x, 4, l, m);
            } else {
                *reinterpret_cast<float4 *>(to + g * R::ROW + d) = v;
                if (d == 0) to[P::GT * R::ROW + g] = m, to[P::GT * R::ROW + P::GT + g] = l;
            }
        });
    }
    if (num_parts == 0) return;
    const bool cut_before = parts[0].before, cut_after = !parts[num_parts - 1].ended;
    if (!cut_before && !cut_after) return;
    __threadfence();
    __syncthreads();
    auto row_blocks = [&](const Part &part, int &first, int &last) {
        const uint32_t nch = (pre[part.b + 1] - pre[part.b]) / p.rows, start = pre[part.b] + part.vh * nch;
        first = (int)(start / block_share);
        last = (int)((start + nch - 1) / block_share);
    };
    if (threadIdx.x == 0) {
        for (int side = 0; side < 2; ++side) {
            const Part &part = parts[side ? num_parts - 1 : 0];
            if (side ? !cut_after || (cut_before && num_parts == 1) : !cut_before) continue;
            int first, last;
            row_blocks(part, first, last);
            if (atomicAdd(p.arrivals + first, 1) == last - first) {
                p.arrivals[first] = 0;  // for the next call
                last_arrived[side] = side ? num_parts - 1 : 0;
            }
        }
        __threadfence();
    }
    __syncthreads();
    struct GlobalRec {
        const float *base;
        int first, last;
        __device__ __forceinline__ const float *at(int i) const {
            return base + ((int64_t)(first + i) * 2 + (first + i == last ? 0 : 1)) * R::FLOATS;
        }
        __device__ __forceinline__ float operator()(int i, int f) const { return __ldcg(at(i) + f); }
        __device__ __forceinline__ float4 quad(int i, int f) const {
            return __ldcg(reinterpret_cast<const float4 *>(at(i) + f));
        }
    };
    for (int side = 0; side < 2; ++side) {
        if (last_arrived[side] < 0) continue;
        const Part part = parts[last_arrived[side]];
        GlobalRec rec;
        rec.base = p.block_rec;
        row_blocks(part, rec.first, rec.last);
        const int c = part.vh / p.tiles, t = part.vh % p.tiles, h0 = c * p.group + t * P::GT;
        join<P>(rec.last - rec.first + 1, min(P::GT, p.group - t * P::GT), rec, [&](int g, int d, float4 v, float l, float m) {
            const float x[4] = {v.x, v.y, v.z, v.w};
            write_final<P>(p, part.b, h0 + g, d, x, 4, l, m);
        });
    }
}

// ------------------------------------------------------------ launch
constexpr size_t align16(size_t v) { return (v + 15) / 16 * 16; }

template <class P>
size_t workspace_of(int blocks) {
    return align16(4 * (size_t)blocks) + 4 * (size_t)Record<P>::FLOATS * blocks * (P::NW + 2);
}

template <class P>
cudaError_t launch_attention(const spmv_paged_attention_t &a, int sms, cudaStream_t stream) {
    using R = Record<P>;
    AttendArgs p;
    p.a = a;
    p.group = a.q_heads / a.kv_heads;
    p.tiles = (p.group + P::GT - 1) / P::GT;
    p.rows = a.kv_heads * p.tiles;
    p.scale2 = std::fabs(a.scale) * kLog2e;
    p.flip = a.scale < 0.0f ? 0x80008000u : 0u;
    // Division by a constant d < 2^31 of t < 2^31 ("Division by Invariant Integers using Multiplication", Granlund and
    // Montgomery, 1994, section 4): with 2^s >= d > 2^(s-1) and m = floor(2^32 (2^s - d) / d) + 1,
    // t / d = (mulhi(m, t) + t) >> s; the sum stays below 2^32.
    p.page_shift = 0;
    while ((1ull << p.page_shift) < (uint64_t)a.page_size) ++p.page_shift;
    p.page_mul = (uint32_t)(((1ull << 32) * ((1ull << p.page_shift) - (uint64_t)a.page_size)) / (uint64_t)a.page_size + 1);
    char *w = static_cast<char *>(a.workspace);
    p.arrivals = reinterpret_cast<int32_t *>(w);
    p.warp_rec = reinterpret_cast<float *>(w + align16(4 * (size_t)sms));
    p.block_rec = p.warp_rec + (int64_t)sms * P::NW * R::FLOATS;
    cudaError_t e = cudaFuncSetAttribute(paged_attention_kernel<P>, cudaFuncAttributeMaxDynamicSharedMemorySize, R::SMEM);
    // a launch's chunks are counted in 32 bits
    const int64_t most = ((int64_t)a.max_pages * a.page_size + P::CH - 1) / P::CH * p.rows;
    const int slice = (int)std::max<int64_t>(1, std::min<int64_t>(kMaxSlice, ((1LL << 31) - 1) / std::max<int64_t>(1, most)));
    const int size = sizeof(typename P::T);
    for (int b = 0; b < a.batch && e == cudaSuccess; b += slice) {
        p.a.batch = std::min(slice, a.batch - b);
        p.a.q = static_cast<const char *>(a.q) + (int64_t)b * a.q_stride[0] * size;
        p.a.out = static_cast<char *>(a.out) + (int64_t)b * a.out_stride[0] * size;
        p.a.lse = a.lse ? a.lse + (int64_t)b * a.q_heads : nullptr;
        p.a.table = a.table + b * a.table_stride;
        p.a.lens = a.lens + b;
        const int64_t blocks = std::min<int64_t>(sms, std::max<int64_t>(1, (most * p.a.batch + P::NW - 1) / P::NW));
        paged_attention_kernel<P><<<(unsigned)blocks, P::NW * 32, R::SMEM, stream>>>(p);
        e = cudaGetLastError();
    }
    return e;
}

// Calls f with the tile of 16-bit elements T for the head size and group.
template <typename T, int GT, typename F>
auto with_mma(int dim, F f) {
    if (dim <= 64) return f(TileMma<T, GT, 64, 8, 5>());
    if (dim <= 96) return f(TileMma<T, GT, 96, 8, 4>());
    if (dim <= 128) return f(TileMma<T, GT, 128, 8, 3>());
    if (dim <= 192) return f(TileMma<T, GT, 192, 4, 4>());
    return f(TileMma<T, GT, 256, 4, 3>());
}

template <typename T, typename F>
auto with_mma(int dim, int group, F f) {
    return group <= 8 ? with_mma<T, 8>(dim, f) : with_mma<T, 16>(dim, f);
}

}  // namespace

}  // namespace lbcsr
