// Paged attention over caches of 8-bit codes (e4m3) with a scale per block of
// positions and head: the kernel is paged_attention.cuh's, this is its tile.
//
//   s_t = scale ks_t <q, k_t>,  out = sum_t w_t vs_t v_t / sum_t w_t
//
// Codes are copied as they are, half the bytes of 16-bit elements, and become
// 16-bit values (f16, exactly) on their way into the warp's matrix
// instructions; a position's key scale goes onto its score, its value scale
// onto its weight.
//   Keys: ldmatrix gives a lane four neighbouring codes of a position, which
// the product takes as its elements 2 t, 2 t + 1 and 2 t + 8, 2 t + 9; q is
// laid out in the same order, and a dot product does not care.
//   Values: the transposing ldmatrix moves pairs of codes, (d, d + 1) of two
// positions; a byte permutation and the conversion make the pairs of positions
// that the product wants, even elements in one of its tiles and odd ones in
// the next.
//   q goes into f16 times a power of two that puts its row's largest element
// into [2^14, 2^15): bf16's 8 bits fit whole as far down as 2^-29 of it, and
// what is lost below is 2^-39 of it, less than the 32-bit sums round.
//   131,071 positions of 8 heads of 128, 8 query heads each (269 MB) 62 us: 0.64
// of the copy's rate.  Bound by latency: 760 instructions a warp for a chunk of
// 32 positions, each held up by the one before, and two warps a scheduler,
// which registers allow, fill 37 % of the issue slots while memory is at half
// of its peak; start and join take about 13 us.
//   Weights are taken 2^14 times as large, times vs / ref with ref the power of
// two below the largest value scale so far, as hi + lo; the sums, relative to
// ref, are rescaled when a larger scale comes.
#include "e4m3.cuh"
#include "paged_attention.cuh"

namespace lbcsr {

namespace {

// two 32-bit values at once
__device__ __forceinline__ uint64_t pair2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpair2(uint64_t v, float &lo, float &hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

template <typename T_, int GT_, int DP_, int CH_, int NW_, int STAGES_>
struct TileE4m3 {
    using T = T_;
    using Cache = unsigned char;
    using Args = ScaledArgs;
    static constexpr int SLICE = 512;
    static constexpr bool SCALES = true;
    static constexpr int DP = DP_, NW = NW_, STAGES = STAGES_, GT = GT_, CH = CH_;
    static constexpr int PAGE_UNIT = 16;
    static constexpr int NT = CH / 8;
    static constexpr int PITCH = DP + 16;  // an odd number of 16 bytes: ldmatrix has no conflicts
    static constexpr int QBYTES = 0;
    static constexpr float LIFT = 0.0f;    // what leaves the tile is taken down again
    static constexpr int H = GT / 8;
    static constexpr float UP = 14.0f;     // log2 of a weight of 1 in the products
    static constexpr bool AHEAD = GT * DP <= 1024;
    static constexpr bool BF16 = std::is_same<T, __nv_bfloat16>::value;
    static_assert(DP % 32 == 0 && CH % 16 == 0, "");

    uint32_t q[DP / 16][2 * H], next[AHEAD ? DP / 16 : 1][2 * H];
    float o[DP / 8][4];  // [32 elements][16 of them][even, odd]
    float m[H], l[H];
    float qf[H];         // what q was divided by
    float ref;           // of o: the same on every lane

    __device__ __forceinline__ static void load(const AttendArgs &p, uint32_t (*to)[2 * H], int b, int h0, int heads, int lane) {
        const T *base = static_cast<const T *>(p.a.q) + b * p.a.q_stride[0] + h0 * p.a.q_stride[1];
        const int g = lane >> 2, t = (lane & 3) * 4;
#pragma unroll
        for (int s = 0; s < DP / 16; ++s)
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    const int head = g + h * 8, d = s * 16 + t + r * 2;
                    const T *at = base + head * p.a.q_stride[1] + d;
                    uint32_t pair = 0;
                    if (head < heads && d < p.a.head_dim)
                        pair = p.q_pairs ? *reinterpret_cast<const uint32_t *>(at) : pack2(at[0], at[1]);
                    to[s][r * H + h] = pair;
                }
    }
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
#pragma unroll
        for (int s = 0; s < DP / 16; ++s)
#pragma unroll
            for (int r = 0; r < 2 * H; ++r) q[s][r] ^= p.flip;
#pragma unroll
        for (int h = 0; h < H; ++h) {
            qf[h] = 1.0f;
            if (!BF16) continue;
            uint32_t top = 0;  // the largest element's bits
#pragma unroll
            for (int s = 0; s < DP / 16; ++s)
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    top = max(top, max(q[s][r * H + h] & 0x7fffu, (q[s][r * H + h] >> 16) & 0x7fffu));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int shift = min(max(14 - ((int)(top >> 7) - 127), -114), 126);
            const float up = __int_as_float((127 + shift) << 23);
            qf[h] = __int_as_float((127 - shift) << 23);
#pragma unroll
            for (int s = 0; s < DP / 16; ++s)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    uint32_t &pair = q[s][r * H + h];
                    const __half2 v = __floats2half2_rn(__uint_as_float(pair << 16) * up, __uint_as_float(pair & 0xffff0000u) * up);
                    memcpy(&pair, &v, 4);
                }
        }
#pragma unroll
        for (int n = 0; n < DP / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.0f;
#pragma unroll
        for (int h = 0; h < H; ++h) m[h] = -INFINITY, l[h] = 0.0f;
        ref = __uint_as_float(1u << 23);
    }

    __device__ __forceinline__ void chunk(const AttendArgs &p, const char *stage, char *, uint32_t mask, int lane) {
        const uint32_t ks = smem_addr(stage), vs = ks + CH * PITCH;
        const float *k_scale = reinterpret_cast<const float *>(stage + 2 * CH * PITCH), *v_scale = k_scale + CH;
        const int r8 = lane & 7, mat = lane >> 3;
        float sums[NT][4] = {};
        {
            const uint32_t at = ks + (r8 + (mat >> 1) * 8) * PITCH + (mat & 1) * 16;
#pragma unroll
            for (int i = 0; i < DP / 32; ++i)
#pragma unroll
                for (int n = 0; n < NT; n += 2) {
                    uint32_t kb[4];  // [8 positions][16 codes]
                    ldmatrix4(at + n * 8 * PITCH + i * 32, kb);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint32_t(&qs)[2 * H] = q[2 * i + j];
                        const uint32_t qa[4] = {qs[0], H == 2 ? qs[H - 1] : 0u, qs[H], H == 2 ? qs[2 * H - 1] : 0u};
                        uint32_t b0, b1;
                        e4m3x4_to_half2(kb[j], b0, b1);
                        mma16816<__half>(sums[n], qa, b0, b1);
                        e4m3x4_to_half2(kb[2 + j], b0, b1);
                        mma16816<__half>(sums[n + 1], qa, b0, b1);
                    }
                }
        }
        // a value scale of twice ref, or more
        const uint32_t v_bits = __float_as_uint(v_scale[lane % CH]) & 0x7f800000u;
        bool higher = v_bits > __float_as_uint(ref);
        uint32_t hi[NT * H], lo[NT * H];
        float s[NT][H][2], top[H];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float2 scale = *reinterpret_cast<const float2 *>(k_scale + n * 8 + (lane & 3) * 2);
#pragma unroll
            for (int h = 0; h < H; ++h) {
                // What q was divided by goes onto the key scale first: a large one and small queries meet here, and the sum
                // of q's lifted products times the scale alone could pass 32 bits.
                uint64_t by = pair2(scale.x, scale.y);
                if (BF16) by = mul2(by, pair2(qf[h], qf[h]));
                unpair2(mul2(pair2(sums[n][2 * h], sums[n][2 * h + 1]), by), s[n][h][0], s[n][h][1]);
            }
        }
        if (mask != FULL_MASK<CH>) {  // their weights are 0: scale2 is not
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    if (!((mask >> (n * 8 + (lane & 3) * 2 + c)) & 1))
#pragma unroll
                        for (int h = 0; h < H; ++h) s[n][h][c] = -INFINITY;
        }
#pragma unroll
        for (int h = 0; h < H; ++h) {
            float raw = -INFINITY;
#pragma unroll
            for (int n = 0; n < NT; ++n) raw = fmaxf(raw, fmaxf(s[n][h][0], s[n][h][1]));
            raw = fmaxf(raw, __shfl_xor_sync(0xffffffffu, raw, 1));
            raw = fmaxf(raw, __shfl_xor_sync(0xffffffffu, raw, 2));
            top[h] = fmaxf(m[h], raw);
            higher |= top[h] > m[h];
        }
        if (__any_sync(0xffffffffu, higher)) {
            const float ref_now = __uint_as_float(max(__reduce_max_sync(0xffffffffu, v_bits), __float_as_uint(ref)));
            const float down = ref / ref_now;
            ref = ref_now;
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const float keep = worth(m[h], top[h], p.scale2), keep_o = keep * down;
                l[h] *= keep;
                m[h] = top[h];
#pragma unroll
                for (int n = 0; n < DP / 8; ++n) {
                    o[n][2 * h] *= keep_o, o[n][2 * h + 1] *= keep_o;
                    if (H == 1) o[n][2] *= keep_o, o[n][3] *= keep_o;
                }
            }
        }
        // ref is a power of two; the reciprocal of 2^127 is subnormal
        const float by_ref = __uint_as_float(max((254u << 23) - __float_as_uint(ref), 1u << 22));
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float2 scale = *reinterpret_cast<const float2 *>(v_scale + n * 8 + (lane & 3) * 2);
            scale.x *= by_ref, scale.y *= by_ref;
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const float base = base_of(m[h]);
                float x = pow2(fmaf(s[n][h][0] - base, p.scale2, UP)), y = pow2(fmaf(s[n][h][1] - base, p.scale2, UP));
                l[h] += x + y;
                x *= scale.x, y *= scale.y;
                const __half2 high = __floats2half2_rn(x, y);
                const float2 back = __half22float2(high);
                const __half2 low = __floats2half2_rn(x - back.x, y - back.y);
                memcpy(&hi[n * H + h], &high, 4);
                memcpy(&lo[n * H + h], &low, 4);
            }
        }
        const uint32_t at = vs + (r8 + (mat & 1) * 8) * PITCH + (mat >> 1) * 16;
#pragma unroll
        for (int k = 0; k < CH / 16; ++k) {
            const uint32_t *kh = hi + 2 * k * H, *kl = lo + 2 * k * H;
            const uint32_t pa[4] = {kh[0], H == 1 ? kl[0] : kh[H - 1], kh[H], H == 1 ? kl[1] : kh[2 * H - 1]};
            const uint32_t pl[4] = {kl[0], kl[H - 1], kl[H], kl[2 * H - 1]};
#pragma unroll
            for (int i = 0; i < DP / 32; ++i) {
                uint32_t vb[4];  // [16 codes][8 positions]
                ldmatrix4_t(at + k * 16 * PITCH + i * 32, vb);
#pragma unroll
                for (int j = 0; j < 4; ++j) vb[j] = __byte_perm(vb[j], 0, 0x3120);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    uint32_t b0[2], b1[2];  // even elements, odd ones
                    e4m3x4_to_half2(vb[2 * j], b0[0], b0[1]);
                    e4m3x4_to_half2(vb[2 * j + 1], b1[0], b1[1]);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        mma16816<__half>(o[4 * i + 2 * j + e], pa, b0[e], b1[e]);
                        if (H == 2) mma16816<__half>(o[4 * i + 2 * j + e], pl, b0[e], b1[e]);
                    }
                }
            }
        }
    }

    __device__ __forceinline__ void sums() {
        const float down = __int_as_float((127 - (int)UP) << 23);
#pragma unroll
        for (int h = 0; h < H; ++h) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
            l[h] *= down;
        }
#pragma unroll
        for (int n = 0; n < DP / 8; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) o[n][c] *= ref * down;
    }

    // f(head, d, value at d, value at d + 1, l)
    template <typename F>
    __device__ __forceinline__ void each(int lane, F f) const {
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
            for (int n = 0; n < DP / 8; n += 2)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float x = H == 1 ? o[n][c] + o[n][2 + c] : o[n][2 * h + c];
                    const float y = H == 1 ? o[n + 1][c] + o[n + 1][2 + c] : o[n + 1][2 * h + c];
                    f((lane >> 2) + 8 * h, n * 8 + (lane & 3) * 4 + 2 * c, x, y, l[h]);
                }
    }
    template <typename F>
    __device__ __forceinline__ void each_head(int lane, F f) const {
#pragma unroll
        for (int h = 0; h < H; ++h)
            if ((lane & 3) == 0) f((lane >> 2) + 8 * h, m[h], l[h]);
    }
};

// Positions of a chunk, warps and stages: what an SM's registers and shared
// memory hold, of the ways measured (64 requests, their lengths even up to
// 4,000, 4 kv heads, 16 positions a page, bf16; us with 4 and with 16 heads
// each).  64 elements: 8 warps of 4 stages 32.8 / 46.2, 12 of 3 31.4 / 46.2, 16
// of 2 32.3 / 42.7, but four requests of up to 300 positions take 10.3 with 8
// warps and 12.4 with more; 96: 8 of 3 42.3 / 54.8, 10 of 3 45.9; 128: 8 of 2
// chunks of 32 (one request of 131,071, 8 heads each: 65 us, 7 of 3 79, 10 of
// 2 80, 16 positions a chunk 83 and more); 192: 8 of 2 62.9 / 83.9, 16
// positions a chunk 65.2 / 137; 256: with 4 heads each 8 of 2 chunks of 16
// 74.0, 6 of 3 86, 6 of 2 of 32 87; with 16 6 of 2 of 32 142, 4 of 4 of 16 176.
template <typename T, int GT, typename F>
auto with_codes(int dim, F f) {
    constexpr bool small = GT == 8;
    if (dim <= 64) return f(TileE4m3<T, GT, 64, 32, small ? 8 : 16, small ? 4 : 2>());
    if (dim <= 96) return f(TileE4m3<T, GT, 96, 32, 8, 3>());
    if (dim <= 128) return f(TileE4m3<T, GT, 128, 32, 8, 2>());
    if (dim <= 192) return f(TileE4m3<T, GT, 192, 32, 8, 2>());
    return f(TileE4m3<T, GT, 256, small ? 16 : 32, small ? 8 : 6, 2>());
}
template <typename T, typename F>
auto with_codes(int dim, int group, F f) {
    return group <= 8 ? with_codes<T, 8>(dim, f) : with_codes<T, 16>(dim, f);
}

}  // namespace

// the records have no elements of T: both types need the same
size_t attention_workspace_e4m3(int dim, int group, int sms) {
    return with_codes<__half>(dim, group, [&](auto tile) { return workspace_of<decltype(tile)>(sms); });
}

cudaError_t launch_attention_e4m3(const spmv_paged_attention_t &a, const AttendScales &scales, int sms, cudaStream_t stream) {
    const int group = a.q_heads / a.kv_heads;
    auto launch = [&](auto tile) { return launch_attention<decltype(tile)>(a, sms, stream, &scales); };
    return a.elem == SPMV_ELEM_BF16 ? with_codes<__nv_bfloat16>(a.head_dim, group, launch) : with_codes<__half>(a.head_dim, group, launch);
}

}  // namespace lbcsr
