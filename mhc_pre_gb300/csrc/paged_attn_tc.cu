// paged_attn_tc.cu -- attention of new tokens over a paged cache on the
// tensor cores (bf16, heads of at most 128, pages that divide 128 keys or are
// a multiple of 128).
//
// One CTA per SM walks the pieces of the plan (paged_attn.cuh).  Roles:
//   * warp 8 loads: key and value blocks of 128 keys go through a ring of
//     shared-memory stages, one TMA box per page and 64 columns (128-byte
//     swizzle); the page numbers are read one block ahead.  Queries come by TMA
//     too: a box of G heads x (128/G) tokens lies in shared memory in the order
//     of the rows.
//   * warp 9 issues the MMAs: S = Q K^T (128 rows x 128 keys, both operands in
//     shared memory) and O += P V with P read from tensor memory and V as it
//     lies in the cache (keys along K, so no transposition anywhere).
//   * warp 10 zeroes the value rows that no row of a tile sees (below).
//   * warp 11 walks the plan and hands the pieces to the others, a few ahead.
//   * two lanes of four warps run the softmax of up to 128 rows each, a thread
//     per row: scores are read from tensor memory to registers, the row's
//     maximum needs no exchange between threads, and the exponentials go back
//     as bf16 over the scores they came from.  While one lane is in its softmax
//     the tensor core works for the other.
// A tile of more rows than a lane has gives each lane its own rows and both
// use every key block; the lanes never wait for each other.  A smaller tile
// (decoding) gives both lanes the same rows and every other key block; lane 0
// adds lane 1's sums to its own at the end.
//
// The running maximum is only raised when a row's new maximum exceeds it by
// more than 2^8 in the exponentials' scale: float32 sums and bf16 exponentials
// lose nothing by a common factor of up to 2^8, and O in tensor memory is then
// rescaled a few times per row instead of at every block.  A cap below 52 bounds
// the scores so well that no maximum is needed at all (LOW_CAP).
//
// Keys outside what a tile's rows see (past the sequence's end, before the
// window) are masked in the scores, and their value rows are zeroed in shared
// memory before the MMA reads them, so that what the pages hold there (NaN,
// say) cannot reach a sum.  The keys and values of a page number outside the
// cache are zeros.
//
// Bounds and figures, 40 query and 8 key heads of 128 on one GB300: 2048 new
// tokens of 32768 keys take 0.80 to 0.85 ms in short runs, 1.6 PFLOP/s (0.81 of
// the library's burst rate for a plain product; the lanes' softmax and the
// products share the time, the tensor pipe is active for 62 % of it), and 0.93 to
// 0.97 ms as calls in a row, under the power cap.  One new token for each of 64
// sequences of up to 8192 keys takes 128 to 131 us with the plan, 5.9 TB/s, and
// two for each of 4 sequences of 131072 keys 325 us, 6.6 TB/s: there the keys and
// values coming from memory are the bound.  Tiles of few blocks (prompts with a
// window, heads of 64) take 6.8 us each and 1.03 a block without a cap, 3.0 and
// 2.2 with one of 30.
//
// Every wait is bounded (about one second); on expiry the kernel latches its
// error word, marks the plan as spent and all roles leave.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "launch.h"
#include "paged_attn.cuh"
#include "tc_ptx.cuh"

namespace mhc {

__device__ unsigned g_attn_tc_error;   // ATTN_ERR_* bits

static ErrorWord g_error_word;

cudaError_t read_and_clear_attn_tc_error(unsigned* word) { return g_error_word.read_and_clear(g_attn_tc_error, word); }

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();   // pre_tc.cu

namespace attn_tc {

constexpr int NTHREADS = 384;
constexpr int LOAD_WARP = 8, MMA_WARP = 9, BLANK_WARP = 10, WALK_WARP = 11;
// A softmax thread holds a row's 128 scores: 208 registers, taken from the
// third warpgroup.  256 * 208 + 128 * 88 = 384 * 168, the block's registers at
// its launch.
constexpr int SOFTMAX_REGS = 208, OTHER_REGS = 88;
constexpr int ROWS = 128, KEYS = 128;
constexpr int SUB = KEYS * 128;              // 128 rows x 64 columns: 16 KB
constexpr int RING_BYTES = 160 * 1024;
constexpr int TMEM_COLS = 512;
constexpr uint32_t S_COL = 0, O_COL = 256;   // two of each, 128 columns apart
constexpr uint64_t WAIT_LIMIT_NS = 1000000000ull;
constexpr float RAISE = 8.0f;                // see above
// Kinds of capping: none; a cap that bounds the scores so well that no maximum
// is needed (below); a higher one; one above HIGH_MOST, beside which ordinary
// scores are so small that their tanh needs more care (near4).
constexpr int NO_CAP = 0, LOW_CAP = 1, HIGH_CAP = 2, FAR_CAP = 3;
// With |z| <= cap (in base 2, cap <= LOW_MOST) every row takes the base
// min(cap, LOW_SPAN - cap): its exponentials then lie between 2^-90 and 2^60,
// where bf16 and float32 round as everywhere, sums of 2^31 of them times values
// of 2^30 stay finite, and a value below 2^-36 is the first that a row of
// lowest scores could lose.  The largest such softcap is 75 / log2 e = 51.98.
constexpr float LOW_MOST = 75.0f, LOW_SPAN = 90.0f;
constexpr uint32_t FULL = 0xffffffffu;

constexpr int PIECES = 4;                    // pieces handed out and not done with
constexpr int PIECE_BYTES = 64;
static_assert(sizeof(AttnPiece) <= PIECE_BYTES, "see Cfg::TOTAL");

template <int DP> struct Cfg {
    static constexpr int TILE = (DP / 64) * SUB;           // a block of keys, or 128 rows of queries
    static constexpr int STAGES = RING_BYTES / TILE;
    static constexpr int Q = 0;
    static constexpr int RING = 2 * TILE;
    static constexpr int BARS = RING + STAGES * TILE;
    static constexpr int B_FULL = 0, B_EMPTY = STAGES, B_S = 2 * STAGES, B_P = B_S + 2;
    static constexpr int B_Q = B_P + 4, B_QE = B_Q + 2, B_O = B_QE + 2, B_ASK = B_O + 2, B_Z = B_ASK + 1;
    static constexpr int B_X = B_Z + 1, B_XE = B_X + 4, B_PF = B_XE + 4, B_PE = B_PF + PIECES, NBARS = B_PE + PIECES;
    static constexpr int MISC = BARS + ((8 * NBARS + 15) / 16) * 16;   // TMEM address, abort flag
    static constexpr int ML = MISC + 16;                               // lane 1's maxima and sums
    static constexpr int PIECE = ML + 2 * ROWS * 4;
    static constexpr int TOTAL = PIECE + PIECES * PIECE_BYTES;
    static constexpr int SMEM = 232448;                                // all that a block may have
    static_assert(TOTAL <= SMEM, "shared memory of one SM");
};

__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = ptx::globaltimer();
    for (uint32_t it = 1;; ++it) {
        if (ptx::mbar_try_wait(bar, parity)) return true;
        if ((it & 63) == 0) {
            if (*abort_flag) return false;
            if (ptx::globaltimer() - t0 > WAIT_LIMIT_NS) {
                atomicOr(&g_attn_tc_error, ATTN_ERR_TIMEOUT);
                *abort_flag = 1;
                return false;
            }
        }
    }
}
// The same for a whole warp: all lanes go on, or none.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
    return __all_sync(FULL, wait_bar(bar, parity, abort_flag));
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// The lesser, or NaN if one is.
__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float rcp_ftz(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// 32 bytes in one store (32-byte aligned).
__device__ __forceinline__ void st32(void* p, const uint4& a, const uint4& b) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z),
                 "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
}

// Whether some of a block's keys lie outside [lo, hi).
__device__ __forceinline__ bool partly_seen(int k0, int lo, int hi) { return k0 < lo || k0 + KEYS > hi; }

// A warp's view of the pieces that the walking warp hands out.
template <int DP> struct Pieces {
    unsigned char* smem;
    uint32_t sbase;
    volatile int* abort_flag;
    uint32_t n;
    __device__ __forceinline__ Pieces(unsigned char* s, uint32_t b, volatile int* a)
        : smem(s), sbase(b), abort_flag(a), n(0) {}
    __device__ __forceinline__ uint32_t bar(int i) const {
        return sbase + Cfg<DP>::BARS + 8u * (static_cast<uint32_t>(i) + n % PIECES);
    }
    // The next piece; nb is 0 after the last one and when a role gave up.
    __device__ __forceinline__ const AttnPiece& get(bool& ok) const {
        ok = wait_warp(bar(Cfg<DP>::B_PF), (n / PIECES) & 1, abort_flag);
        return *reinterpret_cast<const AttnPiece*>(smem + Cfg<DP>::PIECE + (n % PIECES) * PIECE_BYTES);
    }
    // The warp is done with it.
    __device__ __forceinline__ void done(int lane) {
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(Cfg<DP>::B_PE));
        ++n;
    }
};

// cap tanh(scale s / cap) in base 2, plus `c` - cap: tanh(x) = 1 - 2 / (e^2x + 1),
// four quotients from one reciprocal of their denominators' product (so e^2x
// stays below 2^30: past it a denominator changes nothing in float32).  Pairs
// are neighbours in registers.  The difference leaves an error of about 2^-21
// of the cap, whatever the score is: up to HIGH_MOST at most 1.2e-4, a
// sixteenth of the exponentials' rounding to bf16.
constexpr float HIGH_MOST = 256.0f;
__device__ __forceinline__ void cap4(uint32_t* u, float in, float cap2, float c) {
    const float2 in2 = make_float2(in, in), one = make_float2(1.0f, 1.0f), c2 = make_float2(c, c);
    const float2 x = __fmul2_rn(make_float2(__uint_as_float(u[0]), __uint_as_float(u[1])), in2);
    const float2 y = __fmul2_rn(make_float2(__uint_as_float(u[2]), __uint_as_float(u[3])), in2);
    const float2 s = __fadd2_rn(make_float2(ex2(x.x), ex2(x.y)), one);
    const float2 t = __fadd2_rn(make_float2(ex2(y.x), ex2(y.y)), one);
    const float2 st = __fmul2_rn(s, t);
    const float r = rcp_ftz(st.x * st.y) * (-2.0f * cap2);
    const float2 q = make_float2(r * st.y, r * st.x);   // -2 cap / (s t) of each pair
    const float2 z = __ffma2_rn(q, t, c2), w = __ffma2_rn(q, s, c2);
    u[0] = __float_as_uint(z.x);
    u[1] = __float_as_uint(z.y);
    u[2] = __float_as_uint(w.x);
    u[3] = __float_as_uint(w.y);
}

// The same for x = scale s / cap of at most NEAR, with `c` in place of `c` - cap:
// scale s (tanh x) / x by the series of tanh to x^11, whose error is relative
// (2^-27 at NEAR, where the quotients' is 2^-19 of the score).  18 packed
// operations for four scores where the quotients have 7 and twice the MUFU's:
// 2048 tokens on 32768 keys with a cap of 1e5 take 2130 us, 1315 with one of 60.
constexpr float NEAR = 0.3f;
__device__ __forceinline__ float2 near2(float2 s, float in, float zscale, float c) {
    const float2 x = __fmul2_rn(s, make_float2(in, in)), w = __fmul2_rn(x, x);
    auto both = [](float v) { return make_float2(v, v); };
    float2 t = __ffma2_rn(w, both(-1382.0f / 155925.0f), both(62.0f / 2835.0f));
    t = __ffma2_rn(w, t, both(-17.0f / 315.0f));
    t = __ffma2_rn(w, t, both(2.0f / 15.0f));
    t = __ffma2_rn(w, t, both(-1.0f / 3.0f));
    t = __ffma2_rn(w, t, both(1.0f));
    return __ffma2_rn(__fmul2_rn(s, both(zscale)), t, both(c));
}
__device__ __forceinline__ void near4(uint32_t* u, float in, float zscale, float c) {
    const float2 a = near2(make_float2(__uint_as_float(u[0]), __uint_as_float(u[1])), in, zscale, c);
    const float2 b = near2(make_float2(__uint_as_float(u[2]), __uint_as_float(u[3])), in, zscale, c);
    u[0] = __float_as_uint(a.x);
    u[1] = __float_as_uint(a.y);
    u[2] = __float_as_uint(b.x);
    u[3] = __float_as_uint(b.y);
}

// Scores of 32 keys become `with` where `seen` has no bit.
constexpr uint32_t LOWEST = 0xff800000u;   // -inf
__device__ __forceinline__ void mask32(uint32_t* u, uint32_t seen, uint32_t with = LOWEST) {
#pragma unroll
    for (int e = 0; e < 32; ++e)
        if (!(seen & (1u << e))) u[e] = with;
}

// The keys [lo, hi) that a row sees, and the bounds of its warp's rows.
struct Seen {
    int lo, hi, lo_least, lo_most, hi_least, hi_most;
    // Of the 32 keys from g: no row of the warp sees any, all rows see all, and
    // which of them this row sees.
    __device__ __forceinline__ bool none(int g) const { return g >= hi_most || g + 32 <= lo_least; }
    __device__ __forceinline__ bool all(int g) const { return g >= lo_most && g + 32 <= hi_least; }
    __device__ __forceinline__ uint32_t bits(int g) const {
        const int from = max(lo - g, 0), to = min(hi - g, 32);
        return from < to ? (FULL << from) & (FULL >> (32 - to)) : 0u;
    }
};
template <bool V> struct Flag { static constexpr bool value = V; };

template <int DP, int CAP>
__device__ __forceinline__ void softmax_lanes(const AttnParams& p, unsigned char* smem, uint32_t sbase, uint32_t tmem) {
    using C = Cfg<DP>;
    auto bar = [&](int i) { return sbase + C::BARS + 8u * static_cast<uint32_t>(i); };
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC + 4);
    float* ml = reinterpret_cast<float*>(smem + C::ML);
    // what is the same in every lane of the warp is said to be: it then lives
    // in uniform registers
    auto same = [](int v) { return __shfl_sync(FULL, v, 0); };
    const int warp = same(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int L = warp >> 2, w4 = warp & 3, row_t = w4 * 32 + lane;
    const uint32_t t_lane = same(tmem) + (static_cast<uint32_t>(w4 * 32) << 16);
    const uint32_t t_s = t_lane + S_COL + L * 128, t_o = t_lane + O_COL + L * 128;
    const float zscale = CAP ? 1.0f : p.scale * LOG2E;
    const float cap2 = p.softcap * LOG2E, cap_in = CAP ? 2.0f * LOG2E * p.scale / p.softcap : 0.0f;
    const float low_base = fminf(cap2, LOW_SPAN - cap2);
    const float most = CAP ? 30.0f / cap_in : 0.0f;   // larger scores are capped as this one
    // scale / cap, scale in base 2, the largest score that is near zero beside the cap (FAR_CAP)
    const float near_in = p.scale / p.softcap, near_z = p.scale * LOG2E, near_most = NEAR * (p.softcap / p.scale);
    // rows of 32-byte multiples at 32-byte addresses are stored 32 bytes at a time
    // (the workspace's offsets are multiples of 256 bytes, its own address of 16)
    const bool wide = p.Dh % 16 == 0 && (reinterpret_cast<uintptr_t>(p.o) & 31u) == 0;
    const bool wide_part = (reinterpret_cast<uintptr_t>(p.ws) & 31u) == 0;
    uint32_t par_s = 0, par_o = 0, par_x = 0;
    bool ok = true, lent = false;   // lane 1's sums are with lane 0

    Pieces<DP> pieces(smem, sbase, abort_flag);
    while (ok) {
        const AttnPiece& pc = pieces.get(ok);
        if (!ok || pc.nb == 0) break;
        const int lane_rows = p.plan.lane_rows, left = same(pc.qlen * p.G - pc.row0);
        const bool pair = left > lane_rows;
        const int nb = same(pc.nb), blk = same(pc.blk);
        const int mine = pair ? nb : (nb + 1 - L) / 2;          // blocks of this lane
        const int rt = (pair ? L * lane_rows : 0) + row_t;      // row of the tile
        const int r = pc.row0 + rt;
        const bool valid = row_t < lane_rows && rt < left;
        const bool active = __any_sync(FULL, valid);            // a warp without rows only keeps the protocol
        int lo = 0, hi = 0x7fffffff;                            // rows that are not there need no mask
        const int tok = attn_token(p, valid ? r : 0);
        if (valid) attn_token_keys(pc, tok, p.window, lo, hi);
        const int lo_most = same(__reduce_max_sync(FULL, lo)), hi_least = same(__reduce_min_sync(FULL, hi));
        const int lo_least = same(__reduce_min_sync(FULL, valid ? lo : 0x7fffffff));
        const int hi_most = same(__reduce_max_sync(FULL, valid ? hi : 0));
        float m = -INFINITY, l = 0.0f;
        if (lent) {
            ok = wait_warp(bar(C::B_XE + w4), par_x, abort_flag);
            par_x ^= 1;
            lent = false;
            ptx::tc_fence_after();
        }
        for (int i = 0; ok && i < mine; ++i) {
            const int k0 = (blk + (pair ? i : 2 * i + L)) * KEYS;
            ok = wait_warp(bar(C::B_S + L), par_s, abort_flag);
            par_s ^= 1;
            if (!ok) break;
            ptx::tc_fence_after();
            if (active) {
                // Without a cap the scores stay in registers (128 of them) from
                // the maximum to the exponentials.  With one they are taken 32
                // at a time, by loops that are not unrolled: the capping is long
                // enough for the other warp's to cover the loads, and the code
                // of all 128 scores makes the warps wait for instructions (5
                // prompts with a window of 512 keys took 331 us, a chunk of 2048
                // tokens on 32768 keys 1550; with these loops 231 and 1338, and
                // 203 and 1135 without a maximum).  Of a block that not all rows
                // see whole, 32 keys that no row of the warp sees cost nothing,
                // and only the 32 at a border are masked.  Exponentials
                // overwrite scores already read.
                const bool partial = k0 < lo_most || k0 + KEYS > hi_least;
                const Seen see = {lo, hi, lo_least, lo_most, hi_least, hi_most};
                constexpr int HELD = CAP ? 32 : 128;
                uint32_t u[HELD];
                float top;
                if constexpr (CAP == NO_CAP) {
#pragma unroll
                    for (int c = 0; c < HELD / 32; ++c) ptx::tmem_ld32(t_s + c * 32, u + c * 32);
                    ptx::tmem_wait_ld();
                    if (partial) {
#pragma unroll
                        for (int c = 0; c < HELD / 32; ++c)
                            if (!see.all(k0 + 32 * c)) mask32(u + 32 * c, see.bits(k0 + 32 * c));
                    }
                    float mx[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) mx[e] = fmaxf(__uint_as_float(u[e]), __uint_as_float(u[4 + e]));
#pragma unroll
                    for (int e = 8; e < HELD; e += 8)
#pragma unroll
                        for (int f = 0; f < 4; ++f)
                            mx[f] = max3(mx[f], __uint_as_float(u[e + f]), __uint_as_float(u[e + 4 + f]));
                    top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * zscale;
                } else if constexpr (CAP == HIGH_CAP || CAP == FAR_CAP) {
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                    auto sweep = [&](auto borders) {
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            const int g = k0 + 32 * c;
                            if (borders.value && see.none(g)) continue;
                            ptx::tmem_ld32(t_s + c * 32, u);
                            ptx::tmem_wait_ld();
                            if (borders.value && !see.all(g)) mask32(u, see.bits(g));
#pragma unroll
                            for (int e = 0; e < 32; e += 8)
#pragma unroll
                                for (int f = 0; f < 4; ++f)
                                    mx[f] = max3(mx[f], __uint_as_float(u[e + f]), __uint_as_float(u[e + 4 + f]));
                        }
                    };
                    if (partial) sweep(Flag<true>{});
                    else sweep(Flag<false>{});
                    top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    // tanh keeps the order, so the capped maximum is the maximum's
                    uint32_t t[4] = {__float_as_uint(fminf(top, most)), 0u, 0u, 0u};
                    if (CAP == FAR_CAP && fabsf(top) <= near_most) near4(t, near_in, near_z, 0.0f);
                    else cap4(t, cap_in, cap2, cap2);
                    if (top > -INFINITY) top = __uint_as_float(t[0]);
                }
                if constexpr (CAP == LOW_CAP) top = m;
                const bool raise = top > m + RAISE || (m == -INFINITY && top > -INFINITY);
                if (CAP != LOW_CAP && __any_sync(FULL, raise)) {
                    // S of this block is complete, so every earlier MMA is: O stands still
                    const float f = raise ? ex2(m - top) : 1.0f;
                    if (raise) m = top;
                    l *= f;
                    if (i > 0) {
#pragma unroll 1
                        for (int c = 0; c < DP / 32; ++c) {
                            uint32_t o[32];
                            ptx::tmem_ld32(t_o + c * 32, o);
                            ptx::tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            ptx::tmem_st32(t_o + c * 32, o);
                        }
                    }
                }
                const float base = CAP == LOW_CAP ? low_base : m == -INFINITY ? 0.0f : m;
                const float2 z2 = make_float2(zscale, zscale), b2 = make_float2(-base, -base);
                float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
                if constexpr (CAP == NO_CAP) {
#pragma unroll
                    for (int h = 0; h < HELD / 64; ++h) {
                        uint32_t pk[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const float2 x = __ffma2_rn(
                                make_float2(__uint_as_float(u[64 * h + 2 * e]), __uint_as_float(u[64 * h + 2 * e + 1])), z2, b2);
                            const float2 y = make_float2(ex2(x.x), ex2(x.y));
                            sum[e & 1] = __fadd2_rn(sum[e & 1], y);
                            const __nv_bfloat162 t = __floats2bfloat162_rn(y.x, y.y);
                            pk[e] = *reinterpret_cast<const uint32_t*>(&t);
                        }
                        ptx::tmem_st32(t_s + h * 32, pk);
                        ptx::tmem_wait_st();
                        ptx::tc_fence_before();
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(bar(C::B_P + 2 * L + h));
                    }
                } else {
                    auto sweep = [&](auto borders) {
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            const int g = k0 + 32 * c;
                            uint32_t pk[16];
                            if (borders.value && see.none(g)) {
#pragma unroll
                                for (int e = 0; e < 16; ++e) pk[e] = 0u;
                            } else {
                                ptx::tmem_ld32(t_s + c * 32, u);
                                ptx::tmem_wait_ld();
                                const bool border = borders.value && !see.all(g);
                                // before the cap too: an unseen key's NaN must not reach its cap4's other three
                                if (border) mask32(u, see.bits(g), CAP == FAR_CAP ? 0u : LOWEST);
                                bool near = false;   // every score of the warp's is near zero beside the cap
                                if constexpr (CAP == FAR_CAP) {
                                    float mx[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                                    for (int e = 0; e < 32; e += 8)
#pragma unroll
                                        for (int f = 0; f < 4; ++f)
                                            mx[f] = max3(mx[f], fabsf(__uint_as_float(u[e + f])),
                                                         fabsf(__uint_as_float(u[e + 4 + f])));
                                    near = !__any_sync(FULL, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) > near_most);
                                }
                                if (near) {
#pragma unroll
                                    for (int e = 0; e < 32; e += 4) near4(u + e, near_in, near_z, -base);
                                } else if (CAP == FAR_CAP) {
#pragma unroll
                                    for (int e = 0; e < 32; e += 4) {
                                        uint32_t t[4] = {u[e], u[e + 1], u[e + 2], u[e + 3]}, q[4];
#pragma unroll
                                        for (int f = 0; f < 4; ++f)
                                            q[f] = __float_as_uint(min_nan(__uint_as_float(t[f]), most));
                                        cap4(q, cap_in, cap2, cap2 - base);
                                        near4(t, near_in, near_z, -base);
#pragma unroll
                                        for (int f = 0; f < 4; ++f)
                                            u[e + f] = fabsf(__uint_as_float(u[e + f])) <= near_most ? t[f] : q[f];
                                    }
                                } else {
#pragma unroll
                                    for (int e = 0; e < 32; ++e)
                                        u[e] = __float_as_uint(min_nan(__uint_as_float(u[e]), most));
#pragma unroll
                                    for (int e = 0; e < 32; e += 4) cap4(u + e, cap_in, cap2, cap2 - base);
                                }
                                if (border) mask32(u, see.bits(g));
#pragma unroll
                                for (int e = 0; e < 16; ++e) {
                                    const float2 y = make_float2(ex2(__uint_as_float(u[2 * e])),
                                                                 ex2(__uint_as_float(u[2 * e + 1])));
                                    sum[e & 1] = __fadd2_rn(sum[e & 1], y);
                                    const __nv_bfloat162 h = __floats2bfloat162_rn(y.x, y.y);
                                    pk[e] = *reinterpret_cast<const uint32_t*>(&h);
                                }
                            }
                            ptx::tmem_st16(t_s + c * 16, pk);
                            if (c & 1) {
                                // 64 keys' exponentials are there: their product may start
                                ptx::tmem_wait_st();
                                ptx::tc_fence_before();
                                __syncwarp();
                                if (lane == 0) ptx::mbar_arrive(bar(C::B_P + 2 * L + (c >> 1)));
                            }
                        }
                    };
                    if (partial) sweep(Flag<true>{});
                    else sweep(Flag<false>{});
                }
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
            } else {
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    ptx::mbar_arrive(bar(C::B_P + 2 * L));
                    ptx::mbar_arrive(bar(C::B_P + 2 * L + 1));
                }
            }
        }
        if (CAP == LOW_CAP) m = l != 0.0f ? low_base : -INFINITY;   // (NaN: as a row that saw something)
        if (ok && mine > 0) {
            ok = wait_warp(bar(C::B_O + L), par_o, abort_flag);
            par_o ^= 1;
        }
        if (!ok) break;
        ptx::tc_fence_after();
        if (active && !pair && L == 1) {
            // warp w4 of lane 0 adds this warp's rows to its own
            ml[row_t] = m;
            ml[ROWS + row_t] = l;
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(C::B_X + w4));
            lent = true;
        } else if (active) {
            // the rows' sums: to the output if this is the whole tile, else to
            // the workspace
            float w0 = 1.0f, w1 = 0.0f;
            if (!pair) {
                ok = wait_warp(bar(C::B_X + w4), par_x, abort_flag);
                par_x ^= 1;
                if (!ok) break;
                ptx::tc_fence_after();
                const float m1 = ml[row_t], l1 = ml[ROWS + row_t];
                const float M = fmaxf(m, m1), base = M == -INFINITY ? 0.0f : M;
                w0 = ex2(m - base);
                w1 = ex2(m1 - base);
                m = M;
                l = l * w0 + l1 * w1;
            }
            const bool whole = pc.whole != 0;
            const float inv = whole ? (l != 0.0f ? 1.0f / l : 0.0f) : 1.0f;
            w0 *= inv;
            w1 *= inv;
            const int64_t out = valid ? (pc.q0 + tok) * p.Hq + pc.head * p.G + (r - tok * p.G) : 0;
            float* part = attn_slot(p, pc.slot);
            const bool both = !pair && nb > 1;
#pragma unroll 1
            for (int c = 0; c < DP / 32; ++c) {
                uint32_t o[32];
                ptx::tmem_ld32(t_o + c * 32, o);
                ptx::tmem_wait_ld();
                float f[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) f[e] = __uint_as_float(o[e]) * w0;
                if (both) {
                    ptx::tmem_ld32(t_o + 128 + c * 32, o);   // lane 1's
                    ptx::tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e) f[e] = fmaf(__uint_as_float(o[e]), w1, f[e]);
                }
                if (valid && whole) {
                    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.o) + out * p.Dh + c * 32;
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        float t[2][8];
#pragma unroll
                        for (int e = 0; e < 16; ++e) t[e >> 3][e & 7] = f[16 * g + e];
                        const uint4 x = Vec<__nv_bfloat16>::pack(t[0]), y = Vec<__nv_bfloat16>::pack(t[1]);
                        if (wide) {
                            if (c * 32 + g * 16 < p.Dh) st32(dst + g * 16, x, y);
                        } else {
                            if (c * 32 + g * 16 < p.Dh) *reinterpret_cast<uint4*>(dst + g * 16) = x;
                            if (c * 32 + g * 16 + 8 < p.Dh) *reinterpret_cast<uint4*>(dst + g * 16 + 8) = y;
                        }
                    }
                } else if (valid) {
                    float* dst = part + static_cast<int64_t>(rt) * DP + c * 32;
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const uint4 x = make_uint4(__float_as_uint(f[8 * g]), __float_as_uint(f[8 * g + 1]),
                                                   __float_as_uint(f[8 * g + 2]), __float_as_uint(f[8 * g + 3]));
                        const uint4 y = make_uint4(__float_as_uint(f[8 * g + 4]), __float_as_uint(f[8 * g + 5]),
                                                   __float_as_uint(f[8 * g + 6]), __float_as_uint(f[8 * g + 7]));
                        if (wide_part) {
                            st32(dst + g * 8, x, y);
                        } else {
                            *reinterpret_cast<uint4*>(dst + g * 8) = x;
                            *reinterpret_cast<uint4*>(dst + g * 8 + 4) = y;
                        }
                    }
                }
                __syncwarp();
            }
            ptx::tc_fence_before();
            if (!pair) {
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar(C::B_XE + w4));
            }
            if (whole) {
                if (valid && p.lse != nullptr) p.lse[out] = attn_lse(m, l);
            } else {
                if (valid) {
                    part[static_cast<int64_t>(p.plan.slot_rows) * DP + rt] = m;
                    part[static_cast<int64_t>(p.plan.slot_rows) * (DP + 1) + rt] = l;
                }
                // the same warp of the CTA that comes last joins these rows
                __threadfence();
                __syncwarp();
                int last = 0;
                if (lane == 0) {
                    int* count = attn_counts(p) + pc.cnt + (pair ? L * 4 : 0) + w4;
                    last = atomicAdd(count, 1) == pc.last_cta - pc.first_cta;
                    if (last) *count = 0;   // back at zero for the next call with this plan
                    __threadfence();
                }
                __syncwarp();   // the others' reads come after lane 0's
                if (__shfl_sync(FULL, last, 0)) {
                    const int begin = __shfl_sync(FULL, rt, 0), n = __popc(__ballot_sync(FULL, valid));
                    attn_join<__nv_bfloat16, DP, DP == 128 ? 8 : 4, 3>(p, pc, begin, begin + n, lane);
                }
                __syncwarp();
            }
        }
        pieces.done(lane);
    }
}

template <int DP, int CAP>
__global__ void __launch_bounds__(NTHREADS, 1)
attn_tc_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
               const __grid_constant__ CUtensorMap tmap_v, const AttnParams p) {
    using C = Cfg<DP>;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* smem = smem_raw;
    const uint32_t sbase = ptx::smem_u32(smem);
    auto bar = [&](int i) { return sbase + C::BARS + 8u * static_cast<uint32_t>(i); };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC + 4);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = blockIdx.x;

    if (p.force_timeout != 0u) {
        // test hook: one bounded wait that runs out before anything async starts
        if (tid == 0 && ptx::forced_wait_runs_out(sbase, 100000ull)) {
            atomicOr(&g_attn_tc_error, ATTN_ERR_TIMEOUT);
            ptx::griddep_wait();   // the plan is written
            attn_plan_spent(p);
        }
        __syncthreads();
        return;
    }
    if ((sbase & 1023u) != 0) {   // the swizzle needs it; dynamic shared memory starts there without static arrays
        if (tid == 0) atomicOr(&g_attn_tc_error, ATTN_ERR_TIMEOUT);
        return;
    }
    if (tid == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            ptx::mbar_init(bar(C::B_FULL + s), 1);
            ptx::mbar_init(bar(C::B_EMPTY + s), 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(bar(C::B_S + i), 1);
            ptx::mbar_init(bar(C::B_P + 2 * i), 4);       // exponentials of the block's first 64 keys
            ptx::mbar_init(bar(C::B_P + 2 * i + 1), 4);   // and of the other 64
            ptx::mbar_init(bar(C::B_Q + i), 1);
            ptx::mbar_init(bar(C::B_QE + i), 1);
            ptx::mbar_init(bar(C::B_O + i), 1);
        }
        for (int i = 0; i < 4; ++i) {
            ptx::mbar_init(bar(C::B_X + i), 1);    // lane 1's rows of warp i are final
            ptx::mbar_init(bar(C::B_XE + i), 1);   // and have been taken
        }
        for (int i = 0; i < PIECES; ++i) {
            ptx::mbar_init(bar(C::B_PF + i), 1);
            ptx::mbar_init(bar(C::B_PE + i), 11);   // every other warp
        }
        ptx::mbar_init(bar(C::B_ASK), 1);
        ptx::mbar_init(bar(C::B_Z), 1);
        *abort_flag = 0;
        ptx::fence_mbar_init();
        ptx::prefetch_tmap(&tmap_q);
        ptx::prefetch_tmap(&tmap_k);
        ptx::prefetch_tmap(&tmap_v);
    }
    if (warp == MMA_WARP) {
        ptx::tmem_alloc(ptx::smem_u32(tmem_slot), TMEM_COLS);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    ptx::griddep_wait();   // the plan, the queries and the cache are written

    AttnWalk walk;
    const bool begun = walk.begin(p, cta), agrees = attn_plan_agrees(p);   // one round of loads
    if (!agrees && tid == 0) atomicOr(&g_attn_tc_error, ATTN_ERR_RANGE);
    const bool work = agrees && begun;
    if (warp >= LOAD_WARP) {
        ptx::regs_dec<OTHER_REGS>();
        Pieces<DP> pieces(smem, sbase, abort_flag);
        bool ok = true;
        if (work && warp == WALK_WARP) {
            // ------------------------------------------------------ walk ---
            for (uint32_t n = 0; ok; ++n) {
                ok = wait_warp(bar(C::B_PE + n % PIECES), ((n / PIECES) & 1) ^ 1, abort_flag);
                if (!ok) break;
                AttnPiece pc;
                const bool more = walk.next(p, cta, pc);
                if (lane == 0) {
                    *reinterpret_cast<AttnPiece*>(smem + C::PIECE + (n % PIECES) * PIECE_BYTES) = pc;
                    ptx::mbar_arrive(bar(C::B_PF + n % PIECES));
                }
                __syncwarp();
                if (!more) break;   // the piece without blocks ends every role
            }
        } else if (work && warp == LOAD_WARP) {
            // ------------------------------------------------------ loads ---
            const uint64_t policy = ptx::policy_evict_normal();
            const int box = p.page_size < KEYS ? p.page_size : KEYS;      // keys of one TMA box
            const int boxes = KEYS / box;                                 // of a block: at most 16
            int stage = 0;
            uint32_t round = 0, par_q = 1;
            {   // The first pieces' page numbers into the cache, before the walk has handed out the piece
                AttnPiece first;
                if (walk.next(p, cta, first)) {
                    const int key = first.blk * KEYS + lane * box;
                    if (lane < 2 * boxes && key < first.hi && key + box > first.lo) {
                        const int pg = p.page_shift >= 0 ? key >> p.page_shift : key / p.page_size;
                        asm volatile("prefetch.global.L1 [%0];" ::"l"(p.page_table + first.seq * p.table_stride + pg));
                    }
                }
            }
            while (ok) {
                const AttnPiece pc = pieces.get(ok);
                if (!ok || pc.nb == 0) break;
                pieces.done(lane);
                const int tlo = pc.lo, thi = pc.hi;
                const bool pair = pc.qlen * p.G - pc.row0 > p.plan.lane_rows;
                const int nb = pc.nb;
                const int32_t* row = p.page_table + pc.seq * p.table_stride;
                // lane i: the page of box i of a block, -1 where no row sees its keys.  In
                // place of a number outside the cache the page after the last one, of which
                // the copy makes zeros.
                auto page_of = [&](int j) {
                    const int key = (pc.blk + j) * KEYS + lane * box;
                    if (j >= nb || lane >= boxes || key + box <= tlo || key >= thi) return -1;
                    const int pg = p.page_shift >= 0 ? key >> p.page_shift : key / p.page_size;
                    const int page = row[pg];
                    if (page >= 0 && page < p.num_pages) return page;
                    atomicOr(&g_attn_tc_error, ATTN_ERR_RANGE);
                    return static_cast<int>(p.num_pages);
                };
                auto load = [&](const CUtensorMap* tm, int j, int page) {
                    if (!wait_warp(bar(C::B_EMPTY + stage), (round & 1) ^ 1, abort_flag)) return false;
                    const uint32_t full = bar(C::B_FULL + stage), dst = sbase + C::RING + stage * C::TILE;
                    const int n = __popc(__ballot_sync(FULL, page >= 0));
                    if (lane == 0) ptx::mbar_arrive_expect_tx(full, static_cast<uint32_t>(n * box * DP * 2));
                    __syncwarp();
                    if (page >= 0) {
                        const int key = (pc.blk + j) * KEYS + lane * box;
                        const int place = p.page_shift >= 0 ? key & (p.page_size - 1) : key % p.page_size;
#pragma unroll
                        for (int c = 0; c < DP / 64; ++c)
                            ptx::tma_load_4d(dst + c * SUB + lane * box * 128, tm, c * 64, place, pc.head, page, full,
                                             policy);
                    }
                    if (++stage == C::STAGES) {
                        stage = 0;
                        ++round;
                    }
                    return true;
                };
                // in the order of use: K0 V0 K1 V1 ... for a pair of lanes on
                // one block, K0 K1 V0 K2 V1 ... for lanes on alternate blocks
                int page = page_of(0), ahead = page_of(1);
                // each lane's queries, once its last scores have been formed
                for (int L = 0; ok && L < 2; ++L) {
                    ok = wait_warp(bar(C::B_QE + L), par_q, abort_flag);
                    if (ok && lane == 0) {
                        const uint32_t full = bar(C::B_Q + L);
                        ptx::mbar_arrive_expect_tx(full, static_cast<uint32_t>(p.plan.lane_rows * DP * 2));
                        const int64_t tok = pc.q0 + attn_token(p, pc.row0 + (pair ? L * p.plan.lane_rows : 0));
#pragma unroll
                        for (int c = 0; c < DP / 64; ++c)
                            ptx::tma_load_3d(sbase + C::Q + L * C::TILE + c * SUB, &tmap_q, c * 64, pc.head * p.G,
                                             static_cast<int32_t>(tok), full, policy);
                    }
                    __syncwarp();
                }
                par_q ^= 1;
                ok = ok && load(&tmap_k, 0, page);
                for (int j = 0; ok && j < nb; ++j) {
                    const int next = page_of(j + 2);
                    if (!pair && j + 1 < nb) ok = load(&tmap_k, j + 1, ahead);
                    ok = ok && load(&tmap_v, j, page);
                    if (pair && j + 1 < nb) ok = ok && load(&tmap_k, j + 1, ahead);
                    page = ahead;
                    ahead = next;
                }
            }
        } else if (work && warp == BLANK_WARP) {
            // ---------------------------------------------------- blanks ---
            // Value rows that no row of the tile sees become zeros before
            // their product.  Only a tile's first and last block can have some.
            uint32_t n = 0, par_a = 0;   // ring stages used by earlier pieces
            while (ok) {
                const AttnPiece pc = pieces.get(ok);
                if (!ok || pc.nb == 0) break;
                pieces.done(lane);
                const int tlo = pc.lo, thi = pc.hi;
                const bool pair = pc.qlen * p.G - pc.row0 > p.plan.lane_rows;
                for (int j = 0; ok && j < pc.nb; j = j == 0 && pc.nb > 1 ? pc.nb - 1 : pc.nb) {
                    const int k0 = (pc.blk + j) * KEYS;
                    if (!partly_seen(k0, tlo, thi)) continue;
                    // the loads' order: K0 V0 K1 V1 ... or K0 K1 V0 K2 V1 ...
                    const uint32_t at = n + (pair || j == pc.nb - 1 ? 2 * j + 1 : 2 * j + 2);
                    const int s = static_cast<int>(at % C::STAGES);
                    // the MMA thread saw the stage full and asks: this warp meets
                    // too few of the ring's stages to follow their parities itself
                    ok = wait_warp(bar(C::B_ASK), par_a, abort_flag);
                    par_a ^= 1;
                    if (!ok) break;
                    const int before = min(KEYS, max(0, tlo - k0)), from = max(before, min(KEYS, thi - k0));
                    for (int e = lane; e < (before + KEYS - from) * (DP / 8); e += 32) {
                        const int i = e / (DP / 8), c = e % (DP / 8), r = i < before ? i : from + i - before;
                        *reinterpret_cast<uint4*>(smem + C::RING + s * C::TILE + (c >> 3) * SUB + r * 128 +
                                                  (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(bar(C::B_Z));
                }
                n += 2u * static_cast<uint32_t>(pc.nb);
            }
        } else if (work && warp == MMA_WARP) {
            // -------------------------------------------------------- MMA ---
            // The warp runs this loop converged, on values that it knows to be
            // the same in every lane, and one lane's instructions take effect.
            constexpr uint32_t IDESC_S = ptx::idesc_bf16_f32(ROWS, KEYS);
            constexpr uint32_t IDESC_O = ptx::idesc_bf16_f32(ROWS, DP) | (1u << 16);   // B (V) MN-major
            const uint32_t on = ptx::elect_one();
            const uint32_t tm = __shfl_sync(FULL, tmem, 0);
            const uint64_t desc_q = ptx::sw128_kmajor_desc(sbase + C::Q);
            const uint64_t desc_k = ptx::sw128_kmajor_desc(sbase + C::RING);
            const uint64_t desc_v = ptx::sw128_mnmajor_desc(sbase + C::RING, SUB, 1024);
            int stage = 0;
            uint32_t par_f = 0, par_q = 0, par_z = 0, par_p[2] = {0, 0};
            auto take = [&]() {   // the ring's next stage, once it is full
                const int s = stage;
                ok = ok && wait_warp(bar(C::B_FULL + s), par_f, abort_flag);
                if (++stage == C::STAGES) {
                    stage = 0;
                    par_f ^= 1;
                }
                return s;
            };
            auto scores = [&](int L, int s) {
                const uint64_t a = ptx::desc_add(desc_q, L * C::TILE), b = ptx::desc_add(desc_k, s * C::TILE);
#pragma unroll
                for (int k = 0; k < DP / 16; ++k)
                    ptx::tc_mma_f16_if(on, tm + S_COL + L * 128, ptx::desc_add(a, (k / 4) * SUB + (k % 4) * 32),
                                    ptx::desc_add(b, (k / 4) * SUB + (k % 4) * 32), IDESC_S, k > 0);
                ptx::tc_commit_if(on, bar(C::B_S + L));
            };
            // the exponentials come in two halves: the first 64 keys' product
            // starts while the softmax still works on the others
            auto values = [&](int L, int s, bool add) {
                const uint64_t b = ptx::desc_add(desc_v, s * C::TILE);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    ok = ok && wait_warp(bar(C::B_P + 2 * L + h), par_p[L], abort_flag);
                    if (!ok) return false;
                    ptx::tc_fence_after();
#pragma unroll
                    for (int k = 4 * h; k < 4 * h + 4; ++k)
                        ptx::tc_mma_f16_ts_if(on, tm + O_COL + L * 128, tm + S_COL + L * 128 + k * 8,
                                           ptx::desc_add(b, k * 2048), IDESC_O, add || k > 0);
                }
                par_p[L] ^= 1;
                return true;
            };
            auto free_stage = [&](int s) { ptx::tc_commit_if(on, bar(C::B_EMPTY + s)); };
            while (ok) {
                const AttnPiece& pc = pieces.get(ok);
                if (!ok || pc.nb == 0) break;
                const int tlo = pc.lo, thi = pc.hi;
                const bool pair = __shfl_sync(FULL, pc.qlen * p.G - pc.row0, 0) > p.plan.lane_rows;
                const int nb = __shfl_sync(FULL, pc.nb, 0);
                const bool z0 = __all_sync(FULL, partly_seen(pc.blk * KEYS, tlo, thi));
                const bool z1 = __all_sync(FULL, partly_seen((pc.blk + nb - 1) * KEYS, tlo, thi));
                pieces.done(lane);
                auto blanked = [&](int j) {
                    if (ok && ((j == 0 && z0) || (j > 0 && j == nb - 1 && z1))) {
                        if (lane == 0) ptx::mbar_arrive(bar(C::B_ASK));
                        ok = wait_warp(bar(C::B_Z), par_z, abort_flag);
                        par_z ^= 1;
                    }
                };
                auto queries = [&](int L) { ok = ok && wait_warp(bar(C::B_Q + L), par_q, abort_flag); };
                auto free_queries = [&](int L) { ptx::tc_commit_if(on, bar(C::B_QE + L)); };
                if (pair) {
                    int sk = take();
                    queries(0);
                    if (!ok) break;
                    scores(0, sk);
                    queries(1);
                    if (!ok) break;
                    scores(1, sk);
                    free_stage(sk);
                    if (nb == 1) {
                        free_queries(0);
                        free_queries(1);
                    }
                    for (int j = 0; j < nb; ++j) {
                        const bool more = j + 1 < nb;
                        const int sv = take();
                        blanked(j);
                        if (!values(0, sv, j > 0)) break;
                        if (more) {
                            sk = take();
                            if (!ok) break;
                            scores(0, sk);
                            if (j + 2 == nb) free_queries(0);
                        } else {
                            ptx::tc_commit_if(on, bar(C::B_O + 0));
                        }
                        if (!values(1, sv, j > 0)) break;
                        free_stage(sv);
                        if (more) {
                            scores(1, sk);
                            free_stage(sk);
                            if (j + 2 == nb) free_queries(1);
                        } else {
                            ptx::tc_commit_if(on, bar(C::B_O + 1));
                        }
                    }
                } else {
                    for (int j = 0; ok && j < 2; ++j) {
                        queries(j);
                        if (j < nb) {
                            const int sk = take();
                            if (!ok) break;
                            scores(j, sk);
                            free_stage(sk);
                        }
                        if (j + 2 >= nb) free_queries(j);
                    }
                    for (int j = 0; ok && j < nb; ++j) {
                        const int L = j & 1;
                        const int sv = take();
                        blanked(j);
                        if (!values(L, sv, j > 1)) break;
                        free_stage(sv);
                        if (j + 2 < nb) {
                            const int sk = take();
                            if (!ok) break;
                            scores(L, sk);
                            free_stage(sk);
                            if (j + 4 >= nb) free_queries(L);
                        } else {
                            ptx::tc_commit_if(on, bar(C::B_O + L));
                        }
                    }
                }
                par_q ^= 1;
            }
        }
    } else {
        ptx::regs_inc<SOFTMAX_REGS>();
        if (work) softmax_lanes<DP, CAP>(p, smem, sbase, tmem);
    }
    __syncthreads();
    if (*abort_flag) {
        if (tid == 0) attn_plan_spent(p);
        // let copies already issued land before the shared memory goes away
        const uint64_t t0 = ptx::globaltimer();
        while (ptx::globaltimer() - t0 < 20000ull) {
        }
    }
    if (warp == MMA_WARP) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, TMEM_COLS);
    }
}

// ------------------------------------------------------------------ host ---

cudaError_t encode_q(PFN_cuTensorMapEncodeTiled_v12000 fn, CUtensorMap* tm, const AttnParams& p) {
    // (d, head, token); a box is 64 columns x G heads x as many whole tokens as a lane has rows for
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(p.Dh), static_cast<cuuint64_t>(p.Hq),
                                static_cast<cuuint64_t>(p.T)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(p.Dh) * 2, static_cast<cuuint64_t>(p.q_stride) * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(p.G), static_cast<cuuint32_t>(p.plan.lane_rows / p.G)};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p.q), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}

cudaError_t encode(PFN_cuTensorMapEncodeTiled_v12000 fn, CUtensorMap* tm, const void* cache, const AttnParams& p,
                   int64_t page_stride, int64_t slot_stride, int64_t head_stride) {
    // (d, place, head, page); a box is 64 columns x (a page or 128 places)
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(p.Dh), static_cast<cuuint64_t>(p.page_size),
                                static_cast<cuuint64_t>(p.Hk), static_cast<cuuint64_t>(p.num_pages)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(slot_stride * 2), static_cast<cuuint64_t>(head_stride * 2),
                                   static_cast<cuuint64_t>(page_stride * 2)};
    const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(p.page_size < KEYS ? p.page_size : KEYS), 1, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(cache), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}

template <int DP, int CAP>
cudaError_t launch(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const AttnParams& p, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};   // devices whose kernel has its shared memory allowed
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (bit == 0 || !(done.load() & bit)) {
        e = cudaFuncSetAttribute(attn_tc_kernel<DP, CAP>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<DP>::SMEM);
        if (e != cudaSuccess) return e;
        done.fetch_or(bit);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.plan.ncta));
    cfg.blockDim = dim3(NTHREADS);
    cfg.dynamicSmemBytes = Cfg<DP>::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_tc_kernel<DP, CAP>, tq, tk, tv, p);
}

template <int DP>
cudaError_t launch_cap(int cap, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const AttnParams& p,
                       cudaStream_t s) {
    switch (cap) {
        case NO_CAP: return launch<DP, NO_CAP>(tq, tk, tv, p, s);
        case LOW_CAP: return launch<DP, LOW_CAP>(tq, tk, tv, p, s);
        case HIGH_CAP: return launch<DP, HIGH_CAP>(tq, tk, tv, p, s);
        default: return launch<DP, FAR_CAP>(tq, tk, tv, p, s);
    }
}

}  // namespace attn_tc

// Boxes of 8 or more whole swizzle rows that tile a block of 128 keys, and a
// token's query heads of one key head within a lane's rows.
bool attn_tc_supports(bool bf16, int Hq, int Hk, int Dh, int page_size) {
    return bf16 && Hq / Hk <= 128 && Dh <= 128 && page_size >= 8 && (128 % page_size == 0 || page_size % 128 == 0);
}

cudaError_t launch_paged_attn_tc(const AttnParams& p, cudaStream_t s) {
    g_error_word.may_be_set();
    auto fn = tensor_map_encoder();
    if (fn == nullptr) return cudaErrorNotSupported;
    CUtensorMap tq, tk, tv;
    cudaError_t e = attn_tc::encode_q(fn, &tq, p);
    if (e == cudaSuccess) e = attn_tc::encode(fn, &tk, p.k_cache, p, p.k_page_stride, p.k_slot_stride, p.k_head_stride);
    if (e == cudaSuccess) e = attn_tc::encode(fn, &tv, p.v_cache, p, p.v_page_stride, p.v_slot_stride, p.v_head_stride);
    if (e != cudaSuccess) return e;
    const int cap = !(p.softcap > 0.0f)                       ? attn_tc::NO_CAP
                    : p.softcap * LOG2E <= attn_tc::LOW_MOST ? attn_tc::LOW_CAP
                    : p.softcap <= attn_tc::HIGH_MOST        ? attn_tc::HIGH_CAP
                                                             : attn_tc::FAR_CAP;
    return p.Dh <= 64 ? attn_tc::launch_cap<64>(cap, tq, tk, tv, p, s) : attn_tc::launch_cap<128>(cap, tq, tk, tv, p, s);
}

}  // namespace mhc
