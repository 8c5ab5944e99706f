// Attention of whole prompts, or of chunks of them, packed one behind the other:
//
//   s_ij = scale <q_i, k_j>,  out_i = sum_j exp(s_ij - m_i) v_j / sum_j exp(s_ij - m_i)
//
// with j over the keys of i's request, of them those up to i's own place where
// it is causal, in one pass over the keys with the running maximum and sum of
// the softmax.
//
// A tile of queries is 128 rows of one kv head: neighbouring tokens times the
// query heads that share it, so that few tokens fill a tile and the keys are
// read once for all of them.  A block takes two tiles (heads of up to 192
// elements) or one, and goes through their keys 128 (heads of up to 128
// elements) or 64 at a time: what tensor memory holds.
// Its warps are
//   one that loads (TMA tensor copies, stages of a step's V and the next K),
//   one that issues the products (tcgen05, an elected lane),
//   one that plans: finds the rows of the next piece of work, this block's own
//   or that of a block not launched yet, and
//   four for each tile's softmax: a thread has a row.
// Scores S = Q K^T and outputs O live in tensor memory.  A thread takes its row
// of S into registers, and writes the weights over it as the left operand of
// O += P V.  The products of one tile run while the other's softmax does: with
// P_A ready the order is P_A V, then the next S_A, then P_B V, then the next
// S_B, each in the order of issue, so S needs one buffer a tile.  With one tile
// S has two buffers, and the next scores are there when the weights are done.
//
// The maximum that weights are relative to is raised only when a score is
// RAISE powers of two above it, so that O is rarely rescaled; by the row's own
// thread, which knows from the barrier of S that the product before is done.
//
// Keys and values behind a row's last are loaded with the tile.  Their weights
// are zero, which a NaN or infinity in V would survive as NaN: in tiles that
// any row sees in part the loading warp looks V over, puts zeros in the place
// of what is not finite and notes it; the rows that do see such a value then
// add it at the end, and where an output is NaN all the row's values are looked
// through.
//
// A weight is rounded to the elements' type, as an operand of the second
// product has to be; the sum it is divided by takes it whole.  That is an error
// of 2^-8 (f16 2^-11) of sum p |v| at most, and errors against 64 bits are 1.2
// to 1.4 times those of a softmax in 32 bits whose output is rounded once.  To
// keep more of it would take a product of what the rounding left: three where
// there are two, in a kernel that waits for products.
//
// 8,192 tokens, 64 over 8 heads of 128 bf16, causal (1.10 TFLOP): back to back,
// under the power limit, 706 us, 1,557 TFLOP/s, 0.92 of the library product's
// under the same limit; 20 at a time 647 us, 1,700 TFLOP/s, 0.90 of the library
// product's burst.  Bound by the matrix instructions: a step's 2,048 clocks of
// them take about 2,500.  Heads of 64 elements 957 TFLOP/s: matrix instructions
// 41 % of the time, the exponential unit too, for a tile's products wait while
// a thread goes through its row's 128 scores.  Of 192 1,270 (two tiles, 64 keys
// at a time; one tile 1,000).  Of 256 985: one tile, whose outputs fill half of
// tensor memory; matrix instructions 42 %, L2 24 %, 17 % of the issue slots: a
// step's chain of waits.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdlib>
#include <mutex>
#include <type_traits>

#include <cudaTypedefs.h>

#include "internal.cuh"
#include "llm.cuh"
#include "tcgen05.cuh"

namespace lbcsr {

namespace {

enum { kBadQueries = 1, kBadKeys = 2, kGaveUp = 4 };

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kRows = 128;
// Waits end, so that a fault ends with a flag and not with a GPU that hangs; where one runs out everybody gives up.  The
// planner, and warps that have nothing in a piece of work, wait for a whole piece (20 clocks a key of it where its rows
// are in step; a row's end can take as long again), and a search of all requests takes a few clocks each.  So what a wait
// may take goes with the keys and the requests: a second, and this much for each.
constexpr long long kEachClocks = 256;

// DP: the head's elements rounded up to 64; NQ: tiles of a block; CUT: the keys of its work are cut into shares.
template <typename T_, int DP_, int NQ_, bool CUT_>
struct Shape {
    using T = T_;
    static constexpr bool CUT = CUT_;
    static constexpr bool BF16 = std::is_same<T, __nv_bfloat16>::value;
    static constexpr int DP = DP_, NQ = NQ_, KEYS = DP <= 128 ? 128 : 64, HALVES = DP / 64;
    static constexpr int THREADS = NQ * 128 + 128;  // one of the last four warps has nothing to do
    static constexpr int QHALF = kRows * 128, QBYTES = HALVES * QHALF;    // 64 elements of a tile's rows; the tile
    static constexpr int KHALF = KEYS * 128, KVBYTES = HALVES * KHALF;
    // A stage holds the tiles that a step takes: V of tile j and K of tile j + 1.  Stage 0 begins with K of tile 0 alone.
    static constexpr int STAGES = DP == 64 ? 4 : 2, STAGE = 2 * KVBYTES;
    static constexpr int SMEM = 1024 + NQ * QBYTES + STAGES * STAGE;
    static constexpr uint32_t O = 2 * KEYS;                               // columns of tensor memory: S at 0 and KEYS, then O
    static_assert(O + NQ * DP <= 512 && SMEM <= 231 * 1024, "tensor memory and shared memory");
    // Weights are 2^LIFT times as large.  The maximum they are relative to is raised where a score is RAISE powers of
    // two above it, and looked for where a weight (f16), or a step's sum (bf16), is above LIMIT.  f16's weights stay below
    // 2^15, and its smallest step is 2^-35 of a row's largest.  bf16 has the range of 32 bits, in values too: a step's
    // weights sum to at most the number of its keys, so that O, a sum in 32 bits of weights times values, does not pass
    // its range before the plain sum of exp(s - m) v does, and the smallest values are 2^-16 times a weight still there.
    // (Without the lift the maximum would have to be raised wherever a score is above it: 857 us instead of 645 for 8,192
    // tokens whose scores have four times their usual spread.)
    static constexpr float LIFT = BF16 ? -16.0f : 11.0f, RAISE = BF16 ? 8.0f : 4.0f, LIMIT = BF16 ? (float)KEYS : 0x1p15f;
};

struct PromptArgs {
    spmv_prompt_attention_t a;
    int32_t group, tile_tokens;  // query heads per kv head; tokens of a tile
    uint32_t group_mul, group_shift;
    float scale2;                // |scale| / ln 2
    uint32_t negate;             // scale < 0
    int32_t splits;              // shares that each block's keys are cut into
    int64_t clocks;              // that a wait inside the kernel may take
    int64_t rows;                // tokens * q_heads
    float *sums, *stats;         // workspace of cut rows: [splits][rows][head_dim] sums, [splits][rows][2] m and l
};
constexpr int kLeast = 4;      // tiles of keys that a share has at least
constexpr int kMostSplits = 32;

__device__ __forceinline__ float pow2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The larger of two, a float or two 16-bit elements each, NaN where one is.
template <typename T>
__device__ __forceinline__ uint32_t max_nan(uint32_t a, uint32_t b) {
    uint32_t y;
    if constexpr (std::is_same<T, float>::value) asm("max.NaN.f32 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    else if constexpr (std::is_same<T, __half>::value) asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    else asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    return y;
}
template <typename T>
__device__ __forceinline__ bool any_nan(uint32_t x) {
    if constexpr (std::is_same<T, float>::value) return __uint_as_float(x) != __uint_as_float(x);
    constexpr uint32_t INF = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
    return (x & 0x7fffu) > INF || (x >> 16 & 0x7fffu) > INF;
}
template <typename T>
__device__ __forceinline__ uint32_t pack(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack<__nv_bfloat16>(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
template <>
__device__ __forceinline__ uint32_t pack<__half>(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Queries of a request and a kv head that a block works on at a time.  They
// are counted from the last request's last tokens, whose rows have most keys.
struct Work {
    int q0, nq, k0, nk;  // the request's rows
    int t0;              // the first token in it
    int kv_head, split;
    int more;            // 0: there is no more, and the rest says nothing
};

// Finds the requests of work numbers, which mostly rise: a warp's place in the requests.
template <class S>
struct Finder {
    static constexpr int EACH = 4;  // requests of a lane
    int base = 0, before = 0;       // requests passed, counted from the last, and their blocks

    // request r's rows; what is wrong with them
    __device__ __forceinline__ static int read(const PromptArgs &p, int r, Work &w) {
        const int32_t *kv_ptr = p.a.kv_ptr ? p.a.kv_ptr : p.a.q_ptr;
        const int q0 = p.a.q_ptr[r], q1 = p.a.q_ptr[r + 1], k0 = kv_ptr[r], k1 = kv_ptr[r + 1];
        w = Work{};
        if (q0 < 0 || q1 < q0 || q1 > p.a.tokens) return kBadQueries;
        if (k0 < 0 || k1 < k0 || k1 > p.a.keys) return kBadKeys;
        w.q0 = q0, w.nq = q1 - q0, w.k0 = k0, w.nk = k1 - k0;
        return 0;
    }
    // by a whole warp
    __device__ __forceinline__ bool find(const PromptArgs &p, int number, int lane, Work &work) {
        const int whole = S::CUT ? number / p.splits : number, block_tokens = S::NQ * p.tile_tokens, block = whole / p.a.kv_heads;
        if (block < before) base = before = 0;
        for (; base < p.a.requests; base += 32 * EACH) {
            Work w[EACH];
            int n[EACH], sum = 0;
#pragma unroll
            for (int i = 0; i < EACH; ++i) {
                const int r = p.a.requests - 1 - base - lane * EACH - i;
                w[i] = Work{};
                if (r >= 0) read(p, r, w[i]);
                n[i] = (w[i].nq + block_tokens - 1) / block_tokens;
                sum += n[i];
            }
            int scan = sum;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, scan, d);
                if (lane >= d) scan += up;
            }
            const int total = __shfl_sync(0xffffffffu, scan, 31);
            int at = before + scan - sum;
            bool mine = false;
#pragma unroll
            for (int i = 0; i < EACH; ++i) {
                if (block >= at && block < at + n[i]) {
                    mine = true;
                    work = w[i];
                    work.t0 = (n[i] - 1 - (block - at)) * block_tokens;
                }
                at += n[i];
            }
            const uint32_t who = __ballot_sync(0xffffffffu, mine);
            if (who) {
                const int from = __ffs(who) - 1;
                work.q0 = __shfl_sync(0xffffffffu, work.q0, from), work.nq = __shfl_sync(0xffffffffu, work.nq, from);
                work.k0 = __shfl_sync(0xffffffffu, work.k0, from), work.nk = __shfl_sync(0xffffffffu, work.nk, from);
                work.t0 = __shfl_sync(0xffffffffu, work.t0, from);
                work.kv_head = whole - block * p.a.kv_heads, work.split = S::CUT ? number - whole * p.splits : 0;
                work.more = 1;
                return true;
            }
            before += total;
        }
        return false;
    }
};

// What a piece of work is to a block.
template <class S>
struct Item {
    int begin;         // its first tile of keys; the others are counted from there
    int tiles[S::NQ];  // tiles of keys that a tile of queries sees
    int most;          // of them all
    int first_cut;     // the first that some of the rows see in part

    __device__ __forceinline__ static int keys_of(const PromptArgs &p, const Work &w, int token) {  // that a token sees
        return p.a.causal ? min(w.nk, max(0, token - w.nq + 1 + w.nk)) : w.nk;
    }
    __device__ __forceinline__ Item(const PromptArgs &p, const Work &w) {
        int all = 0;
#pragma unroll
        for (int t = 0; t < S::NQ; ++t) {
            const int first = w.t0 + t * p.tile_tokens, last = min(first + p.tile_tokens, w.nq) - 1;
            tiles[t] = last < first ? 0 : (keys_of(p, w, last) + S::KEYS - 1) / S::KEYS;
            all = max(all, tiles[t]);
        }
        begin = 0, most = all;
        first_cut = keys_of(p, w, w.t0) / S::KEYS;
        if constexpr (S::CUT) {  // the shares that there are tiles for, as equal as they go
            const int shares = min(p.splits, max(1, all / kLeast));
            begin = w.split < shares ? (int)((int64_t)all * w.split / shares) : all;
            const int end = w.split < shares ? (int)((int64_t)all * (w.split + 1) / shares) : all;
            most = 0;
#pragma unroll
            for (int t = 0; t < S::NQ; ++t) tiles[t] = max(0, min(tiles[t], end) - begin), most = max(most, tiles[t]);
            first_cut = max(0, first_cut - begin);
        }
    }
};

// Adds to a row's elements what is not finite among the values that the row sees: those of the first `whole` keys, which all
// rows of the warp see, looked for by all lanes and only where an element is NaN (search), and each row's others up to
// `end` (0: the row takes no part).  An element that a weight of 0 times an infinity made NaN becomes their sum.
template <typename T, typename Out>
__device__ __forceinline__ void add_not_finite(Out *out, int head_dim, const T *v, int64_t stride, bool search, int whole, int end, int lane) {
    constexpr uint32_t INF = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
#pragma unroll 1
    for (int c = 0; c < head_dim; c += 8) {
        __syncwarp();
        uint32_t found = 0;  // of eight elements: infinity, minus infinity, NaN
#pragma unroll 1
        for (int pass = search ? 0 : 1; pass < 2; ++pass) {
            const int last = pass == 0 ? whole : end, step = pass == 0 ? 32 : 1;
#pragma unroll 4
            for (int k = pass == 0 ? lane : whole; k < last; k += step) {
                const uint4 x = *reinterpret_cast<const uint4 *>(v + k * stride + c);
                const uint32_t words[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t bits = words[i / 2] >> (i % 2 * 16) & 0xffffu, size = bits & 0x7fffu;
                    if (size >= INF) found |= (size > INF ? 4u : bits >> 15 ? 2u : 1u) << (3 * i);
                }
            }
            __syncwarp();
            if (pass == 0) found = __reduce_or_sync(0xffffffffu, found);
        }
#pragma unroll 1
        for (int i = 0; i < 8 && end > 0; ++i) {
            const uint32_t what = found >> (3 * i) & 7u;
            if (what == 0) continue;
            const float x = what == 1 ? INFINITY : what == 2 ? -INFINITY : __int_as_float(0x7fffffff), now = to_float(out[c + i]);
            out[c + i] = from_float<Out>(now == now ? now + x : x);
        }
    }
    __syncwarp();
}

// Barriers' phases are counted over all work of a block: steps of a tile (scores, weights, and product with one tile),
// stages (full, empty), pieces of work (the others).
template <class S>
struct Shared {
    uint64_t q_full, q_empty, full[S::STAGES], empty[S::STAGES], scores[2], weights[2], product, done[S::NQ], last;
    uint64_t planned[2], taken[2], nearly, answered;
    uint4 answer;
    uint32_t tmem;
    int gave_up, not_finite[2];
    Work plan[2];
};

template <class S>
__global__ void __launch_bounds__(S::THREADS, 1)
prompt_attention_kernel(const __grid_constant__ PromptArgs p, const __grid_constant__ CUtensorMap q_map,
                        const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
    using T = typename S::T;
    extern __shared__ char dynamic[];
    __shared__ Shared<S> sh;
    after_previous();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    char *smem = dynamic + ((1024 - (tc::smem_u32(dynamic) & 1023)) & 1023);
    char *q_smem = smem, *kv_smem = smem + S::NQ * S::QBYTES;
    constexpr int kLoader = S::NQ * 4, kIssuer = kLoader + 1, kPlanner = kLoader + 2;

    if (threadIdx.x == 0) {
        tc::bar_init(&sh.q_full, 1), tc::bar_init(&sh.q_empty, 1), tc::bar_init(&sh.product, 1), tc::bar_init(&sh.last, 1);
        for (int i = 0; i < S::STAGES; ++i) tc::bar_init(&sh.full[i], 1), tc::bar_init(&sh.empty[i], 1);
        for (int i = 0; i < 2; ++i) {
            tc::bar_init(&sh.scores[i], 1), tc::bar_init(&sh.weights[i], 129);
            tc::bar_init(&sh.planned[i], 1), tc::bar_init(&sh.taken[i], S::NQ * 4 + 2);
        }
        for (int i = 0; i < S::NQ; ++i) tc::bar_init(&sh.done[i], 1);
        tc::bar_init(&sh.answered, 1), tc::bar_init(&sh.nearly, 1);
        sh.gave_up = 0;
        tc::bar_init_done();
    }
    __syncwarp();
    if (warp == kIssuer) tc::alloc(&sh.tmem, 512);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = sh.tmem;
    volatile int *gave_up = &sh.gave_up;
    auto wait = [&](uint64_t *bar, uint32_t parity) { return tc::bar_wait(bar, parity, gave_up, p.clocks); };
    // The next piece of work; the planner is one ahead of the last warp at work.
    auto next = [&](int item, Work &w) {
        if (!wait(&sh.planned[item & 1], item >> 1 & 1)) return false;
        w = sh.plan[item & 1];
        return w.more != 0;
    };
    auto finished = [&](int item) {
        __syncwarp();
        if (lane == 0) tc::bar_arrive(&sh.taken[item & 1]);
    };
    // Every warp's last step: all have stopped then, whoever came to its end before another one gave up.  Whether one did,
    // and all read the same.
    auto stopped = [&] {
        tc::fence_before();
        tc::block_barrier(1, S::THREADS);
        return sh.gave_up != 0;
    };
    // A row of 128 scores needs more registers than 384 threads have each: three times 168 are 72 + 2 * 216.
    static_assert(S::NQ == 1 || S::THREADS == 384, "the registers of the launch");
    if (warp >= kLoader) {
        if constexpr (S::NQ == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == kLoader) {
            bool ok = true;
            Work w;
            int pairs = 0, queries = 0;      // loaded so far
            int steps[2] = {0, 0};           // announced so far, of a tile (with one tile the first counts)
            for (int item = 0; ok && next(item, w); ++item) {
                const Item<S> of(p, w);
                const int most = of.most;
                if (lane == 0) sh.not_finite[item & 1] = 0;
                __syncwarp();
                if (most > 0) {
                    if (queries > 0) ok = wait(&sh.q_empty, (queries - 1) & 1);
                    if (!ok) break;
                    if (lane == 0) {
                        const uint32_t box = (uint32_t)(p.tile_tokens * p.group * 128 * S::HALVES);
                        const int n = S::NQ == 2 && of.tiles[S::NQ - 1] > 0 ? 2 : 1;
                        tma::mbar_expect_tx(&sh.q_full, n * box);
                        for (int t = 0; t < n; ++t)
                            for (int h = 0; h < S::HALVES; ++h)
                                tc::load_3d(q_smem + t * S::QBYTES + h * S::QHALF, &q_map, 64 * h, w.kv_head * p.group,
                                            w.q0 + w.t0 + t * p.tile_tokens, &sh.q_full);
                    }
                    ++queries;
                }
                const int pairs0 = pairs;  // pair i of this work is pair pairs0 + i
                // pair i: K of tile i, if there is one, and V of the tile before
                auto load = [&](int i) {
                    const int stage = pairs % S::STAGES, round = pairs / S::STAGES;
                    ok = round == 0 || wait(&sh.empty[stage], (round - 1) & 1);
                    if (!ok) return;
                    if (lane == 0) {
                        tma::mbar_expect_tx(&sh.full[stage], ((i < most) + (i > 0)) * S::KVBYTES);
                        for (int h = 0; h < S::HALVES; ++h) {
                            char *at = kv_smem + stage * S::STAGE + h * S::KHALF;
                            if (i < most) tc::load_3d(at, &k_map, 64 * h, w.kv_head, w.k0 + (of.begin + i) * S::KEYS, &sh.full[stage]);
                            if (i > 0) tc::load_3d(at + S::KVBYTES, &v_map, 64 * h, w.kv_head, w.k0 + (of.begin + i - 1) * S::KEYS, &sh.full[stage]);
                        }
                    }
                    ++pairs;
                };
                auto wait_pair = [&](int i) {
                    return wait(&sh.full[(pairs0 + i) % S::STAGES], (pairs0 + i) / S::STAGES & 1);
                };
                // puts zeros in the place of what is not finite among a stage's values
                auto look_over = [&](int stage) {
                    constexpr uint32_t EXPONENT = S::BF16 ? 0x7f807f80u : 0x7c007c00u, UNIT = S::BF16 ? 0x00800080u : 0x04000400u;
                    uint4 *v = reinterpret_cast<uint4 *>(kv_smem + stage * S::STAGE + S::KVBYTES);
                    auto bad = [&](uint32_t x) { return ((x & EXPONENT) + UNIT) & 0x80008000u; };  // its halves that are not finite
                    uint32_t any = 0;
#pragma unroll 8
                    for (int i = lane; i < S::KVBYTES / 16; i += 32) {
                        const uint4 x = v[i];
                        any |= bad(x.x) | bad(x.y) | bad(x.z) | bad(x.w);
                    }
                    if (any) {
                        auto zeroed = [&](uint32_t x) {
                            const uint32_t b = bad(x);
                            return x & ~((b >> 15) * 0xffffu);
                        };
                        for (int i = lane; i < S::KVBYTES / 16; i += 32) {
                            const uint4 x = v[i];
                            v[i] = make_uint4(zeroed(x.x), zeroed(x.y), zeroed(x.z), zeroed(x.w));
                        }
                        sh.not_finite[item & 1] = 1;
                        tc::shared_to_async();
                    }
                    __syncwarp();
                };
                // Tells the issuer, with the weights of step j, that what the step takes is there: V of tile j, looked over
                // if need be, and the keys behind it.
                auto announce = [&](int j) {
                    const int last = S::NQ == 2 ? j + 1 : min(j + 2, most);
                    for (int i = j + 1; i <= last && ok; ++i) ok = wait_pair(i);
                    if (ok && j >= of.first_cut) look_over((pairs0 + j + 1) % S::STAGES);
                    for (int t = 0; t < S::NQ && ok; ++t) {  // once a phase: the one before has to be over
                        if (j >= of.tiles[t]) continue;
                        const int step = steps[t]++, b = S::NQ == 2 ? t : step & 1, phase = S::NQ == 2 ? step : step >> 1;
                        if (phase > 0) ok = wait(&sh.weights[b], (phase - 1) & 1);
                        if (ok && lane == 0) tc::bar_arrive(&sh.weights[b]);
                    }
                };
                if (most > 0) load(0);
                if (most == 0 && lane == 0) tc::bar_arrive(&sh.nearly);
                for (int j = 0; j < most && ok; ++j) {
                    load(j + 1);
                    if (j + 1 == most && ok && lane == 0) tc::bar_arrive(&sh.nearly);
                    if (S::NQ == 1 && ok && j > 0) announce(j - 1);
                    if (S::NQ == 2 && ok) announce(j);
                }
                if (S::NQ == 1 && ok && most > 0) announce(most - 1);
                if (ok) finished(item);
            }
            if (stopped()) {  // nothing may be on its way into shared memory when the block ends
                if (queries > 0) tc::bar_wait(&sh.q_full, (queries - 1) & 1, nullptr);
                for (int i = std::max(0, pairs - S::STAGES); i < pairs; ++i)
                    tc::bar_wait(&sh.full[i % S::STAGES], i / S::STAGES & 1, nullptr);
            }
        } else if (warp == kIssuer) {
            // the whole warp goes through this, one lane issues
            const int n16 = (p.a.head_dim + 15) / 16;
            const uint32_t to = tc::uniform(tmem);
            const uint32_t scores_of = tc::product(S::BF16, kRows, S::KEYS, false, p.negate != 0);
            const uint32_t output_of = tc::product(S::BF16, kRows, 16 * n16, true, false);
            const uint32_t smem_at = tc::uniform(tc::smem_u32(smem));
            const tc::Operand q_at = tc::operand(smem_at, 1024, 0), k_at = tc::operand(smem_at + S::NQ * S::QBYTES, 1024, 0),
                              v_at = tc::operand(smem_at + S::NQ * S::QBYTES, 1024, S::KHALF);
            // The operands' places are constants apart, so that a product of 16 takes its thread a few instructions: with
            // descriptors made for each the products waited for that thread (about 130 clocks each, where they take 64).
            // S at column s = Q of tile t times a stage's K
            auto scores = [&](int t, int stage, uint32_t s) {
                const tc::Operand k = k_at.at(stage * S::STAGE), q = q_at.at(t * S::QBYTES);
#pragma unroll
                for (int i = 0; i < S::DP / 16; ++i)
                    if (i < n16)
                        tc::mma(to + s, q.at((i >> 2) * S::QHALF + (i & 3) * 32), k.at((i >> 2) * S::KHALF + (i & 3) * 32), scores_of,
                                i > 0);
            };
            // O of tile t (+)= the weights at column s times a stage's V
            auto output = [&](int t, int stage, uint32_t s, bool add) {
                const tc::Operand v = v_at.at(stage * S::STAGE + S::KVBYTES);
#pragma unroll
                for (int i = 0; i < S::KEYS / 16; ++i)
                    tc::mma_ts(to + S::O + t * S::DP, to + s + i * 8, v.at(i * 2048), output_of, i > 0 || add);
            };
            // the weights, and all that their step takes
            auto wait_weights = [&](int buffer, int parity) {
                const bool there = wait(&sh.weights[buffer], parity);
                tc::fence_after();
                return there;
            };
            bool ok = true;
            Work w;
            int stage = 0, stage_phase = 0;   // of the next pair
            int queries = 0, steps[2] = {0, 0};
            auto pass_stage = [&] {
                if (++stage == S::STAGES) stage = 0, stage_phase ^= 1;
            };
            // The queue of products is short, and every wait takes this warp 150 clocks and more even where nothing is waited
            // for: it waits once a tile and step.
            for (int item = 0; ok && next(item, w); ++item) {
                const Item<S> of(p, w);
                const int rounds = tc::uniform(of.most);
                if (rounds == 0) {
                    finished(item);
                    continue;
                }
                ok = wait(&sh.q_full, queries++ & 1) && wait(&sh.full[stage], stage_phase);
                if (!ok) break;
                if constexpr (S::NQ == 2) {
                    const int own[2] = {tc::uniform(of.tiles[0]), tc::uniform(of.tiles[1])};
                    if (tc::elect()) {
                        for (int t = 0; t < 2; ++t)
                            if (own[t] > 0) scores(t, stage, t * S::KEYS), tc::commit(&sh.scores[t]);
                        tc::commit(&sh.empty[stage]);
                        if (rounds == 1) tc::commit(&sh.q_empty);
                    }
                    __syncwarp();
                    pass_stage();
                    for (int j = 0; j < rounds && ok; ++j) {
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            if (j < own[t]) ok = wait_weights(t, (steps[t] + j) & 1);
                            if (!ok) break;
                            if (tc::elect()) {
                                if (j < own[t]) {
                                    output(t, stage, t * S::KEYS, j > 0);
                                    if (j + 1 < own[t]) scores(t, stage, t * S::KEYS), tc::commit(&sh.scores[t]);
                                    else tc::commit(&sh.done[t]);
                                }
                                if (t == 1) {
                                    tc::commit(&sh.empty[stage]);
                                    if (j + 2 == rounds) tc::commit(&sh.q_empty);
                                }
                            }
                            __syncwarp();
                        }
                        pass_stage();
                    }
                    steps[0] += own[0], steps[1] += own[1];
                } else {
                    const int step0 = steps[0];  // step j is step step0 + j of the block, in buffer (step0 + j) % 2
                    auto buffer = [&](int j) { return (uint32_t)((step0 + j) & 1); };
                    const int stage0 = stage;
                    if (tc::elect()) {
                        scores(0, stage0, buffer(0) * S::KEYS), tc::commit(&sh.scores[buffer(0)]);
                        tc::commit(&sh.empty[stage0]);
                        if (rounds == 1) tc::commit(&sh.q_empty);
                    }
                    __syncwarp();
                    pass_stage();
                    if (rounds > 1) {
                        ok = wait(&sh.full[stage], stage_phase);
                        if (ok && tc::elect()) {
                            scores(0, stage, buffer(1) * S::KEYS), tc::commit(&sh.scores[buffer(1)]);
                            if (rounds == 2) tc::commit(&sh.q_empty);
                        }
                        __syncwarp();
                    }
                    for (int j = 0; j < rounds && ok; ++j) {
                        ok = wait_weights(buffer(j), (step0 + j) >> 1 & 1);
                        if (!ok) break;
                        const int after = stage + 1 == S::STAGES ? 0 : stage + 1;
                        if (tc::elect()) {
                            output(0, stage, buffer(j) * S::KEYS, j > 0), tc::commit(&sh.product), tc::commit(&sh.empty[stage]);
                            if (j + 2 < rounds) scores(0, after, buffer(j) * S::KEYS), tc::commit(&sh.scores[buffer(j)]);
                            if (j + 3 == rounds) tc::commit(&sh.q_empty);
                            if (j + 1 == rounds) tc::commit(&sh.done[0]);
                        }
                        __syncwarp();
                        pass_stage();
                    }
                    steps[0] += rounds;
                }
                if (ok) finished(item);
            }
            if (stopped()) {  // no product may be under way when its memory is given back
                if (tc::elect()) tc::commit(&sh.last);
                __syncwarp();
                tc::bar_wait(&sh.last, 0, nullptr);
            }
            __syncwarp();
            tc::fence_after();
            tc::dealloc(tmem, 512);
        } else if (warp == kPlanner) {
            // Work for the other warps: this block's own, then that of blocks that have not begun, so that loads and first
            // scores run during the last piece's end.
            Finder<S> finder;
            int item = 0, asked = 0;
            bool ok = true;
            auto publish = [&](const Work &w) {
                if (lane == 0) sh.plan[item & 1] = w;
                __syncwarp();
                if (lane == 0) tc::bar_arrive(&sh.planned[item & 1]);
                ++item;
            };
            for (int number = blockIdx.x; number >= 0 && ok;) {
                Work w;
                if (finder.find(p, number, lane, w)) {
                    if (item >= 2) ok = wait(&sh.taken[item & 1], (item - 2) >> 1 & 1);
                    if (!ok) break;
                    publish(w);
                    // No more is taken over before this piece is nearly done: what waits here another block could do
                    // (asking when a piece begins: 263 us instead of 243 for eight chunks of 512 behind 3,500 to 7,000).
                    ok = wait(&sh.nearly, (item - 1) & 1);
                    if (!ok) break;
                }
                if (lane == 0) tc::ask_block(&sh.answer, &sh.answered);
                __syncwarp();
                // waited for by its own time alone: an answer must not come behind the block's end
                const bool there = tc::bar_wait(&sh.answered, asked++ & 1, nullptr);
                if (!there) *gave_up = 1, ok = false;
                number = there ? tc::answered_block(&sh.answer) : -1;
                tc::shared_to_async();  // read before it is written again
                __syncwarp();
            }
            if (ok && item >= 2) ok = wait(&sh.taken[item & 1], (item - 2) >> 1 & 1);
            if (ok) publish(Work{});
            if (blockIdx.x == 0)  // the first block looks all requests over
                for (int r = lane; r < p.a.requests; r += 32) {
                    Work w;
                    if (const int flag = Finder<S>::read(p, r, w)) atomicOr(p.a.status, flag);
                }
            if (stopped() && lane == 0) atomicOr(p.a.status, kGaveUp);
        } else {
            stopped();
        }
    } else {
        if constexpr (S::NQ == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        const int t = warp >> 2, row = threadIdx.x & 127;
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);  // this warp's 32 lanes
        const int in_tile = (int)((__umulhi((uint32_t)row, p.group_mul) + (uint32_t)row) >> p.group_shift);
        int steps = 0, pieces = 0;  // of this tile so far; with one tile step s is in buffer s % 2
        bool ok = true;
        Work w;
        for (int item = 0; ok && next(item, w); ++item) {
            const Item<S> of(p, w);
            const int n = of.tiles[t], first_cut = of.first_cut;
            const int token = w.t0 + t * p.tile_tokens + in_tile, head = w.kv_head * p.group + row - in_tile * p.group;
            const bool real = in_tile < p.tile_tokens && token < w.nq;
            const int seen = Item<S>::keys_of(p, w, token) - of.begin * S::KEYS;  // of its share's keys and those behind
            float m = -INFINITY, l = 0.0f;
            for (int j = 0; j < n; ++j) {
                const int step = steps + j, buffer = S::NQ == 2 ? t : step & 1;
                const uint32_t at = lanes + buffer * S::KEYS;
                ok = wait(&sh.scores[buffer], S::NQ == 2 ? step & 1 : step >> 1 & 1);
                if (!ok) break;
                tc::fence_after();
                const int left = seen - j * S::KEYS;  // keys that the row sees here
                const bool cut = j >= first_cut;
                // The instructions on tensor memory want a whole warp: where lanes may have gone different ways they meet
                // again before the next one, here and at the outputs.
                // Loops that few steps go through are not unrolled: the code of a step has to stay in the caches of
                // instructions beside that of the warp that issues the products.
                if (cut) {
#pragma unroll 1
                    for (int c = 0; c < S::KEYS; c += 32) {
                        float s[32];
                        tc::load32(at + c, reinterpret_cast<uint32_t *>(s));
                        tc::load32_wait(reinterpret_cast<uint32_t *>(s));
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (c + i >= left) s[i] = -INFINITY;
                        __syncwarp();
                        tc::store32(at + c, reinterpret_cast<uint32_t *>(s));
                    }
                    tc::store_wait();
                }
                // The weights are taken relative to the maximum so far, and the row's own is looked for only where one of
                // them comes out too large, or nothing was seen before.
                bool search = __any_sync(0xffffffffu, real && m == -INFINITY);
                uint32_t weights[S::KEYS / 2];
                float sum;
                for (;;) {
                    if (search) {
                        float high = m;
#pragma unroll 1
                        for (int c = 0; c < S::KEYS; c += 32) {
                            float s[32];
                            tc::load32(at + c, reinterpret_cast<uint32_t *>(s));
                            tc::load32_wait(reinterpret_cast<uint32_t *>(s));
#pragma unroll
                            for (int i = 0; i < 32; ++i) high = fmaxf(high, s[i]);
                        }
                        const bool raise = real && (high - m) * p.scale2 > S::RAISE;
                        if (__any_sync(0xffffffffu, raise)) {
                            const float keep = raise ? (m == -INFINITY ? 0.0f : pow2((m - high) * p.scale2)) : 1.0f;
                            if (raise) m = high;
                            __syncwarp();
                            l *= keep;
                            if (j > 0) {
                                if constexpr (S::NQ == 1) {  // with two tiles the barrier of S says it
                                    ok = wait(&sh.product, (step - 1) & 1);
                                    if (!ok) break;
                                    tc::fence_after();
                                }
                                const uint32_t o_at = lanes + S::O + t * S::DP;
#pragma unroll 1
                                for (int c = 0; c < p.a.head_dim; c += 32) {
                                    uint32_t o[32];
                                    tc::load32(o_at + c, o);
                                    tc::load32_wait(o);
#pragma unroll
                                    for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * keep);
                                    tc::store32(o_at + c, o);
                                }
                            }
                        }
                    }
                    const float base = m == -INFINITY ? 0.0f : m;
                    const uint64_t minus = tc::pair(-base, -base), by = tc::pair(p.scale2, p.scale2), lift = tc::pair(S::LIFT, S::LIFT);
                    uint64_t sums[2] = {0, 0};
                    float s[2][32];
                    __half2 top = __float2half2_rn(0.0f);
                    tc::load32(at, reinterpret_cast<uint32_t *>(s[0]));
#pragma unroll
                    for (int c = 0; c < S::KEYS; c += 32) {
                        float *x = s[c / 32 % 2];
                        tc::load32_wait(reinterpret_cast<uint32_t *>(x));
                        if (c + 32 < S::KEYS) tc::load32(at + c + 32, reinterpret_cast<uint32_t *>(s[(c / 32 + 1) % 2]));
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            float a, b;
                            tc::unpair(tc::fma2(tc::add2(tc::pair(x[i], x[i + 1]), minus), by, lift), a, b);
                            a = pow2(a), b = pow2(b);
                            sums[i / 2 % 2] = tc::add2(sums[i / 2 % 2], tc::pair(a, b));
                            const uint32_t w = weights[(c + i) / 2] = pack<T>(a, b);
                            if constexpr (!S::BF16) {
                                __half2 h;
                                memcpy(&h, &w, 4);
                                top = __hmax2(top, h);
                            }
                        }
                    }
                    float a, b;
                    tc::unpair(tc::add2(sums[0], sums[1]), a, b);
                    sum = a + b;
                    const float largest = S::BF16 ? sum : fmaxf(__low2float(top), __high2float(top));
                    if (search || !__any_sync(0xffffffffu, real && largest > S::LIMIT)) break;
                    search = true;
                }
                if (!ok) break;
                l += sum;
#pragma unroll
                for (int c = 0; c < S::KEYS / 2; c += 32) tc::store32(at + c, weights + c);
                tc::store_wait();
                tc::fence_before();
                tc::bar_arrive(&sh.weights[buffer]);
            }
            if (n > 0 && ok) {
                ok = wait(&sh.done[t], pieces++ & 1);
                tc::fence_after();
                // over long since; what the loading warp noted before it arrived here is read below
                const int step = steps + n - 1;
                ok = ok && wait(&sh.weights[S::NQ == 2 ? t : step & 1], S::NQ == 2 ? step & 1 : step >> 1 & 1);
            }
            steps += n;
            if (ok && w.t0 + t * p.tile_tokens < w.nq) {
                T *out = static_cast<T *>(p.a.out) + (int64_t)(w.q0 + token) * p.a.out_stride[0] + head * p.a.out_stride[1];
                const T *v = static_cast<const T *>(p.a.v) + (int64_t)(w.k0 + of.begin * S::KEYS) * p.a.v_stride[0] + w.kv_head * p.a.v_stride[1];
                const float inverse = S::CUT ? 1.0f : l == 0.0f ? 0.0f : 1.0f / l;
                const int64_t part = S::CUT ? w.split * p.rows + (int64_t)(w.q0 + token) * p.a.q_heads + head : 0;
                const bool weighs = n > 0 && l != 0.0f;  // some key
                const int end = S::CUT ? min(seen, n * S::KEYS) : seen, whole = min(first_cut, n) * S::KEYS;
                uint32_t probe[4] = {};  // NaN where an output is
                using Out = typename std::conditional<S::CUT, float, T>::type;
                for (int c = 0; c < p.a.head_dim && (!S::CUT || n > 0); c += 32) {
                    __syncwarp();
                    uint32_t o[32];
                    if (n > 0) {
                        tc::load32(lanes + S::O + t * S::DP + c, o);
                        tc::load32_wait(o);
                    }
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = weighs ? __float_as_uint(__uint_as_float(o[i]) * inverse) : 0u;
                    if (!real) continue;
                    if constexpr (S::CUT) {
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            if (c + i < p.a.head_dim) {
                                *reinterpret_cast<uint4 *>(p.sums + part * p.a.head_dim + c + i) = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                                for (int j = 0; j < 4; ++j) probe[j] = max_nan<float>(probe[j], o[i + j]);
                            }
                        continue;
                    }
#pragma unroll
                    for (int i = 0; i < 32; i += 8)
                        if (c + i < p.a.head_dim) {
                            uint32_t x[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                x[j] = pack<T>(__uint_as_float(o[i + 2 * j]), __uint_as_float(o[i + 2 * j + 1]));
                                probe[j] = max_nan<T>(probe[j], x[j]);
                            }
                            *reinterpret_cast<uint4 *>(out + c + i) = make_uint4(x[0], x[1], x[2], x[3]);
                        }
                }
                using Out = typename std::conditional<S::CUT, float, T>::type;
                // the weights do not explain it
                // Values that are not finite: taken out of the tiles seen in part, or times a weight of 0.  A sum of weights
                // that is NaN makes its row NaN whatever they are.
                const bool takes = real && weighs && l == l;
                const bool odd = takes && any_nan<Out>(max_nan<Out>(max_nan<Out>(probe[0], probe[1]), max_nan<Out>(probe[2], probe[3])));
                const bool search = __any_sync(0xffffffffu, odd);
                if (search || (n > 0 && sh.not_finite[item & 1])) {
                    if constexpr (S::CUT) add_not_finite<T>(p.sums + part * p.a.head_dim, p.a.head_dim, v, p.a.v_stride[0], search, whole, takes ? end : 0, lane);
                    else add_not_finite<T>(out, p.a.head_dim, v, p.a.v_stride[0], search, whole, takes ? end : 0, lane);
                }
                if constexpr (S::CUT) {
                    if (real) *reinterpret_cast<float2 *>(p.stats + 2 * part) = make_float2(m, l);
                } else if (real && p.a.lse)
                    p.a.lse[(int64_t)(w.q0 + token) * p.a.q_heads + head] =
                        l == 0.0f ? -INFINITY : fmaf(m == -INFINITY ? 0.0f : m, p.scale2, log2f(l) - S::LIFT) * kLn2;
            }
            if (ok) finished(item);
        }
        stopped();
    }
}

// ---------------------------------------------------------------- rows that were cut
// A warp joins a row's shares in their order, each weighted by its maximum's
// distance from the largest.
constexpr int kJoinWarps = 8;
template <typename T>
__global__ void __launch_bounds__(kJoinWarps * 32) prompt_join_kernel(PromptArgs p, float lift) {
    after_previous();
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * kJoinWarps + (threadIdx.x >> 5);
    if (row >= p.rows) return;
    const int64_t token = row / p.a.q_heads;
    const int head = (int)(row - token * p.a.q_heads);
    bool mine = false;  // the row is some request's
    for (int r0 = 0; r0 < p.a.requests && !mine; r0 += 32) {
        const int r = r0 + lane;
        bool in = false;
        if (r < p.a.requests) {
            const int32_t *kv_ptr = p.a.kv_ptr ? p.a.kv_ptr : p.a.q_ptr;
            const int q0 = p.a.q_ptr[r], q1 = p.a.q_ptr[r + 1], k0 = kv_ptr[r], k1 = kv_ptr[r + 1];
            in = q0 >= 0 && q0 <= token && token < q1 && q1 <= p.a.tokens && k0 >= 0 && k1 >= k0 && k1 <= p.a.keys;
        }
        mine = __any_sync(0xffffffffu, in);
    }
    if (!mine) return;
    float m = -INFINITY, l = 0.0f;
    if (lane < p.splits) {
        const float2 stat = *reinterpret_cast<const float2 *>(p.stats + 2 * (lane * p.rows + row));
        m = stat.x, l = stat.y;
    }
    float high = m;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, d));
    // a share without weights has no sums either
    const float weight = l == 0.0f ? 0.0f : m == -INFINITY ? 1.0f : pow2((m - high) * p.scale2);
    float sum = l * weight;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    const uint32_t there = __ballot_sync(0xffffffffu, !(weight == 0.0f));
    // of shares whose weight is 0 next to the others' what is not finite counts
    const uint32_t vanished = __ballot_sync(0xffffffffu, !(l == 0.0f)) & ~there;
    const float inverse = sum == 0.0f ? 0.0f : 1.0f / sum;
    T *out = static_cast<T *>(p.a.out) + token * p.a.out_stride[0] + head * p.a.out_stride[1];
    for (int c0 = 0; c0 < p.a.head_dim; c0 += 128) {
        const int c = c0 + lane * 4;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
        for (int i = 0; i < p.splits; ++i) {
            const float wi = __shfl_sync(0xffffffffu, weight, i);
            if (!(there >> i & 1) || c >= p.a.head_dim) continue;
            const float4 x = *reinterpret_cast<const float4 *>(p.sums + (i * p.rows + row) * p.a.head_dim + c);
            o.x = fmaf(wi, x.x, o.x), o.y = fmaf(wi, x.y, o.y), o.z = fmaf(wi, x.z, o.z), o.w = fmaf(wi, x.w, o.w);
        }
        for (uint32_t left = c < p.a.head_dim ? vanished : 0; left; left &= left - 1) {
            const int i = __ffs(left) - 1;
            const float4 x = *reinterpret_cast<const float4 *>(p.sums + (i * p.rows + row) * p.a.head_dim + c);
            auto add = [](float &sum, float y) { sum += fabsf(y) < INFINITY ? 0.0f : y; };
            add(o.x, x.x), add(o.y, x.y), add(o.z, x.z), add(o.w, x.w);
        }
        if (c < p.a.head_dim)
            *reinterpret_cast<uint2 *>(out + c) = make_uint2(pack<T>(o.x * inverse, o.y * inverse), pack<T>(o.z * inverse, o.w * inverse));
    }
    if (lane == 0 && p.a.lse) p.a.lse[row] = sum == 0.0f ? -INFINITY : fmaf(high == -INFINITY ? 0.0f : high, p.scale2, log2f(sum) - lift) * kLn2;
}

// ---------------------------------------------------------------- launch
PFN_cuTensorMapEncodeTiled_v12000 map_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    });
    return fn;
}

// rows x heads x head_dim elements at `at`; a copy takes 64 elements of box_heads heads of box_rows rows
bool make_map(CUtensorMap *map, bool bf16, const void *at, int head_dim, int heads, int rows, const int64_t *stride, int box_heads,
              int box_rows) {
    const auto encode = map_encoder();
    if (!encode) return false;
    // the stride of a dimension of one element is never used, but checked
    const int64_t head_stride = heads > 1 ? stride[1] : head_dim, row_stride = rows > 1 ? stride[0] : (int64_t)heads * head_dim;
    const cuuint64_t sizes[3] = {(cuuint64_t)head_dim, (cuuint64_t)heads, (cuuint64_t)rows};
    const cuuint64_t strides[2] = {(cuuint64_t)head_stride * 2, (cuuint64_t)row_stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows}, step[3] = {1, 1, 1};
    return encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void *>(at), sizes,
                  strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int DP, int NQ>
spmv_status_t launch_prompt(const spmv_prompt_attention_t &a, cudaStream_t stream) {
    using S = Shape<T, DP, NQ, false>;
    PromptArgs p;
    p.a = a;
    p.group = a.q_heads / a.kv_heads;
    p.tile_tokens = kRows / p.group;
    set_divisor((uint32_t)p.group, &p.group_mul, &p.group_shift);
    // weights of masked scores, minus infinity, have to be 0: a scale of 0 is taken as one that no score feels
    p.scale2 = std::max(std::fabs(a.scale) * kLog2e, FLT_MIN);
    p.negate = a.scale < 0.0f;
    p.clocks = (1ll << 31) + kEachClocks * ((int64_t)a.keys + a.requests);
#ifdef SPMV_DEBUG
    if (const char *clocks = std::getenv("SPMV_PROMPT_CLOCKS")) p.clocks = std::atoll(clocks);  // waits that run out
#endif
    CUtensorMap maps[3];
    const bool keys = a.keys > 0;  // without keys nothing is loaded
    if (!make_map(&maps[0], S::BF16, a.q, a.head_dim, a.q_heads, a.tokens, a.q_stride, p.group, p.tile_tokens) ||
        !make_map(&maps[1], S::BF16, keys ? a.k : a.q, a.head_dim, a.kv_heads, std::max(a.keys, 1), a.k_stride, 1, S::KEYS) ||
        !make_map(&maps[2], S::BF16, keys ? a.v : a.q, a.head_dim, a.kv_heads, std::max(a.keys, 1), a.v_stride, 1, S::KEYS))
        return llm_fail(SPMV_ERR_CUDA, "spmv_prompt_attention: the driver refused a tensor map");
    // no more pieces of work than this, whatever the lengths
    const int64_t block_tokens = S::NQ * p.tile_tokens, requests = std::min(a.requests, a.tokens);
    const int64_t pieces = (a.tokens + requests * (block_tokens - 1)) / block_tokens * a.kv_heads;
    // Few pieces leave most SMs without work: each one's keys are cut into shares then, as far as there are SMs, workspace,
    // keys (a share has four tiles at least) and bits to count them; a second kernel joins them.  64 queries behind 60,000
    // keys, 32 over 8 heads of 128: 487 us uncut.
    const int64_t sms = std::max(1, device_sm_count()), row_bytes = 4 * ((int64_t)a.head_dim + 2);
    p.rows = (int64_t)a.tokens * a.q_heads;
    const int64_t room = a.workspace ? (int64_t)std::min<uint64_t>(a.workspace_bytes, 1ull << 40) / (row_bytes * p.rows) : 0;
    p.splits = (int)std::max<int64_t>(1, std::min(std::min(sms / pieces, room), std::min<int64_t>(kMostSplits, a.keys / (kLeast * S::KEYS))));
    p.sums = static_cast<float *>(a.workspace);
    p.stats = p.sums + p.splits * p.rows * a.head_dim;
    auto launch = [&](auto kernel) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
        return e != cudaSuccess ? e
                                : launch_chained(kernel, (unsigned)(pieces * p.splits), S::THREADS, S::SMEM, 0, stream, p, maps[0], maps[1], maps[2]);
    };
    cudaError_t e = p.splits == 1 ? launch(prompt_attention_kernel<S>) : launch(prompt_attention_kernel<Shape<T, DP, NQ, true>>);
    if (e == cudaSuccess && p.splits > 1)
        e = launch_chained(prompt_join_kernel<T>, (unsigned)((p.rows + kJoinWarps - 1) / kJoinWarps), kJoinWarps * 32, 0, 0, stream, p,
                           S::LIFT);
    return llm_launched("spmv_prompt_attention launch", e);
}
template <typename T>
spmv_status_t launch_prompt_of(const spmv_prompt_attention_t &a, cudaStream_t stream) {
    if (a.head_dim <= 64) return launch_prompt<T, 64, 2>(a, stream);
    if (a.head_dim <= 128) return launch_prompt<T, 128, 2>(a, stream);
    if (a.head_dim <= 192) return launch_prompt<T, 192, 2>(a, stream);
    return launch_prompt<T, 256, 1>(a, stream);
}

const char *prompt_bad(const spmv_prompt_attention_t &a) {
    if (a.requests < 0 || a.tokens < 0 || a.keys < 0 || a.q_heads < 0) return "negative size";
    if (a.elem != SPMV_ELEM_BF16 && a.elem != SPMV_ELEM_F16) return "elements must be bf16 or f16";
    if (a.head_dim < 8 || a.head_dim > 256 || a.head_dim % 8) return "head_dim must be a multiple of 8 in [8, 256]";
    if (a.kv_heads < 1 || a.q_heads % a.kv_heads) return "q_heads must be a multiple of kv_heads";
    if (a.q_heads / a.kv_heads > 128) return "q_heads must be at most 128 times kv_heads";
    if ((int64_t)a.tokens * a.q_heads >= (1LL << 31)) return "tokens * q_heads must be < 2^31";
    // rows are counted up to the end of a block's tiles, requests 128 at a time
    if (std::max(std::max(a.tokens, a.keys), a.requests) > INT32_MAX - 512) return "requests, tokens and keys must be at most 2^31 - 513";
    if (a.requests == 0 || a.tokens == 0 || a.q_heads == 0) return nullptr;
    if (!a.q || !a.q_ptr || !a.out || !a.status) return "q, q_ptr, out or status is NULL";
    if (a.keys > 0 && (!a.k || !a.v)) return "k or v is NULL";
    if (!aligned_to(a.q_ptr, 4) || !aligned_to(a.kv_ptr, 4) || !aligned_to(a.lse, 4) || !aligned_to(a.status, 4))
        return "q_ptr, kv_ptr, lse or status is not aligned to its type";
    if (a.workspace && !aligned_to(a.workspace, 16)) return "the workspace must be 16-byte aligned";
    if (!aligned_to(a.q, 16) || !aligned_to(a.k, 16) || !aligned_to(a.v, 16) || !aligned_to(a.out, 16))
        return "q, k, v and out must be 16-byte aligned";
    const int sizes[2] = {a.tokens, a.q_heads}, kv_sizes[2] = {a.keys, a.kv_heads};
    for (int i = 0; i < 2; ++i)  // of a dimension with one element they are not used
        if ((sizes[i] > 1 && (a.q_stride[i] % 8 || a.out_stride[i] % 8)) || (kv_sizes[i] > 1 && (a.k_stride[i] % 8 || a.v_stride[i] % 8)))
            return "strides must be multiples of 16 bytes";
    for (int i = 0; i < 2; ++i)  // as tensor copies take them
        if ((sizes[i] > 1 && (a.q_stride[i] < 1 || a.q_stride[i] >= (1LL << 38))) ||
            (kv_sizes[i] > 1 && (a.k_stride[i] < 1 || a.k_stride[i] >= (1LL << 38) || a.v_stride[i] < 1 || a.v_stride[i] >= (1LL << 38))))
            return "strides of q, k and v must be positive and less than 2^38";
    return nullptr;
}

}  // namespace

}  // namespace lbcsr

using namespace lbcsr;

extern "C" {

spmv_status_t spmv_prompt_attention_workspace(int32_t q_heads, int32_t kv_heads, int32_t head_dim, spmv_elem_t elem, size_t *bytes) {
    if (!bytes) return llm_bad("bytes is NULL");
    *bytes = 0;
    spmv_prompt_attention_t a = {};
    a.q_heads = q_heads, a.kv_heads = kv_heads, a.head_dim = head_dim, a.elem = elem;
    if (const char *bad = prompt_bad(a)) return llm_bad(bad);
    const int sms = device_sm_count();
    if (sms <= 0) return llm_fail(SPMV_ERR_CUDA, "no CUDA device");
    // the rows of as many pieces of work as there are SMs
    *bytes = (size_t)sms * (head_dim <= 192 ? 2 : 1) * kRows * 4 * (head_dim + 2);
    return SPMV_OK;
}

spmv_status_t spmv_prompt_attention(const spmv_prompt_attention_t *args, spmv_stream_t stream_handle) {
    if (!args) return llm_bad("args is NULL");
    const spmv_prompt_attention_t &a = *args;
    if (const char *bad = prompt_bad(a)) return llm_bad(bad);
    if (a.requests == 0 || a.tokens == 0 || a.q_heads == 0) return SPMV_OK;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_handle);
    return a.elem == SPMV_ELEM_BF16 ? launch_prompt_of<__nv_bfloat16>(a, stream) : launch_prompt_of<__half>(a, stream);
}

}  // extern "C"
