// qk_norm_rope_bare.cu -- the position rotation without the normalisation
// (forward, backward, and into a paged cache), and the table of its angles.
//
//   (a, b) -> (a c - b s, b c + a s),   backward: the transpose, s -> -s.
// The transpose needs nothing of the forward, so its backward is the same pass.
// Many tokens go through turn_kernel below, fewer through the kernels of
// qk_norm_rope_fwd.cuh with NORM off.  Bound by memory: 32768 tokens of 40 + 8 heads
// of 128 in bf16 take 130 us (6.2 TB/s, 0.93 of the measured copy rate; 144 in those
// kernels, which store 8 bytes a lane), with neighbouring pairs 133, into the cache
// 164; in float32, whose rows leave room for 4 warps' stages only and so go through
// qk_norm_rope_fwd.cuh, 252 and 302 (0.95 and 0.93).  64 tokens 3.2 us: a position, then
// its angles, and the launch.  A table of 131072 x 128 takes 11.8 us
// (5.7 TB/s).
#include <math.h>

#include "qk_norm_rope_fwd.cuh"

namespace mhc {

static ErrorWord g_error_word;

cudaError_t read_and_clear_rope_error(unsigned* word) { return g_error_word.read_and_clear(g_qk_error, word); }

namespace qk {

// ------------------------------------------------------------- many tokens ---
// Nothing is summed over a head, so a warp takes a whole token by itself: its rows
// come to shared memory by bulk copies, are turned where they lie, and leave by bulk
// copies, so that global memory sees whole rows both ways.  A warp has a ring of
// stages; one is copied in while another is being turned and a third leaves.  A lane
// has 16 bytes of a's and 16 of b's (or 32 of pairs) of a head, at the same place of
// every head that it takes, so a token's angles are read once.
struct TurnRing {
    int rows[3], sizes[3];   // q, k, v: byte offsets in a stage, bytes (v: 0 unless it is appended)
    int angles, note;        // byte offsets
    int stage_bytes, stages, warps;
};

template <typename TA, bool ADJ>
__device__ __forceinline__ void turn_rows(TA* row, int heads, int Dh, int rot, const float* angles, float sign, int lane) {
    constexpr int V = 16 / static_cast<int>(sizeof(TA)), NG = V / 4;   // values of a piece, groups of four pairs
    const int units = rot / (2 * V), side = 32 / units;                // of a head, heads side by side
    const int u = lane % units, h0 = lane / units;
    if (h0 >= side) return;
    Coef k[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        const float4 c = *reinterpret_cast<const float4*>(angles + u * V + 4 * g);
        const float4 s = *reinterpret_cast<const float4*>(angles + rot / 2 + u * V + 4 * g);
        Angles a;
        a.c[0] = make_float2(c.x, c.y);
        a.c[1] = make_float2(c.z, c.w);
        a.s[0] = make_float2(s.x, s.y);
        a.s[1] = make_float2(s.z, s.w);
        k[g] = make_coef(a, sign);
    }
    using F = typename Four<TA>::T;
    for (int h = h0; h < heads; h += side) {
        TA* x = row + h * Dh + (ADJ ? 2 * u * V : u * V);
        TA* y = x + (ADJ ? V : rot / 2);
        F a[NG], b[NG];
        *reinterpret_cast<uint4*>(a) = *reinterpret_cast<const uint4*>(x);
        *reinterpret_cast<uint4*>(b) = *reinterpret_cast<const uint4*>(y);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            // neighbouring pairs of bf16: a piece holds both runs of its group
            F& lo = ADJ && NG == 2 ? (g == 0 ? a[0] : b[0]) : a[g];
            F& hi = ADJ && NG == 2 ? (g == 0 ? a[NG - 1] : b[NG - 1]) : b[g];
            Raw<TA> r;
            r.lo = lo;
            r.hi = hi;
            r = pack<TA, ADJ>(turn(unpack<TA, ADJ>(r), k[g]));
            lo = r.lo;
            hi = r.hi;
        }
        *reinterpret_cast<uint4*>(x) = *reinterpret_cast<const uint4*>(a);
        *reinterpret_cast<uint4*>(y) = *reinterpret_cast<const uint4*>(b);
    }
}

constexpr int TURN_WARPS = 16;

template <typename TA, bool ADJ, bool APPEND>
__global__ void __launch_bounds__(TURN_WARPS * 32)
turn_kernel(const QkParams p, const TurnRing ring) {
    extern __shared__ __align__(128) unsigned char smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, S = ring.stages;
    unsigned char* base = smem + warp * S * ring.stage_bytes;
    const uint32_t full = ptx::smem_u32(smem) + ring.warps * S * ring.stage_bytes + warp * S * 8;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * ring.warps + warp;
    const int64_t step = static_cast<int64_t>(gridDim.x) * ring.warps;
    const int64_t count = first < p.T ? (p.T - first + step - 1) / step : 0;
    if (lane == 0) {
        for (int s = 0; s < S; ++s) ptx::mbar_init(full + 8 * s, 1);
        ptx::fence_mbar_init();
        ptx::fence_proxy_async_smem();
    }
    __syncwarp();
    int next_pos = 0, put = 0;   // lane 0: the next token's position and slot, its stage
    int64_t next_slot = -1;
    auto numbers = [&](int64_t n) {
        if (n >= count) return;
        next_pos = p.positions[first + n * step];
        if (APPEND) next_slot = p.slots[first + n * step];
    };
    auto start = [&](int64_t n) {   // lane 0: the copies of token n
        if (n >= count) return;
        const int64_t t = first + n * step;
        unsigned char* stage = base + put * ring.stage_bytes;
        Note note;
        note.good = next_pos >= 0 && next_pos < p.max_pos;
        note.slot = next_slot;
        const bool bad_slot = APPEND && (note.slot < -1 || note.slot >= p.num_slots);
        if (bad_slot) note.slot = -1;
        if (!note.good || bad_slot) atomicOr(&g_qk_error, 2u);
        *reinterpret_cast<Note*>(stage + ring.note) = note;
        const uint32_t bar = full + 8 * put;
        ptx::mbar_arrive_expect_tx(bar, static_cast<uint32_t>(ring.sizes[0] + ring.sizes[1] + ring.sizes[2] + p.rot * 4));
        const char* const src[3] = {static_cast<const char*>(p.q) + t * p.q_stride * static_cast<int64_t>(sizeof(TA)),
                                    static_cast<const char*>(p.k) + t * p.k_stride * static_cast<int64_t>(sizeof(TA)),
                                    static_cast<const char*>(p.v) + t * p.v_stride * static_cast<int64_t>(sizeof(TA))};
#pragma unroll
        for (int i = 0; i < (APPEND ? 3 : 2); ++i)
            ptx::bulk_load(ptx::smem_u32(stage + ring.rows[i]), src[i], static_cast<uint32_t>(ring.sizes[i]), bar);
        ptx::bulk_load(ptx::smem_u32(stage + ring.angles), p.cos_sin + static_cast<int64_t>(note.good ? next_pos : 0) * p.rot,
                       static_cast<uint32_t>(p.rot) * 4u, bar);
        if (++put == S) put = 0;
        numbers(n + 1);
    };
    // With two stages a token's copies follow the one before out of its stage; with
    // more there is one stage between them, and the wait is over when it begins.
    const int ahead = S == 2 ? 1 : S - 2;
    if (lane == 0) {
        numbers(0);
        for (int n = 0; n < ahead; ++n) start(n);
    }
    int s = 0;
    uint32_t parity = 0;
    bool ok = true;
    for (int64_t n = 0; n < count; ++n) {
        if (lane == 0) {
            if (S == 2) ptx::bulk_wait_read<0>();
            else ptx::bulk_wait_read<1>();
            start(n + ahead);
        }
        __syncwarp();
        ok = __all_sync(0xffffffffu, wait_full(full + 8 * s, parity));
        if (!ok) break;
        unsigned char* stage = base + s * ring.stage_bytes;
        const Note note = *reinterpret_cast<const Note*>(stage + ring.note);
        TA *q = reinterpret_cast<TA*>(stage + ring.rows[0]), *k = reinterpret_cast<TA*>(stage + ring.rows[1]);
        const bool good = note.good != 0, write = APPEND && good && note.slot >= 0;
        if (good) {
            const float* angles = reinterpret_cast<const float*>(stage + ring.angles);
            turn_rows<TA, ADJ>(q, p.Hq, p.Dh, p.rot, angles, p.sine_sign, lane);
            if (!APPEND || write) turn_rows<TA, ADJ>(k, p.Hk, p.Dh, p.rot, angles, p.sine_sign, lane);
        } else {
            for (int i = lane; i < ring.sizes[0] / 16; i += 32) reinterpret_cast<uint4*>(q)[i] = make_uint4(0u, 0u, 0u, 0u);
            for (int i = lane; i < ring.sizes[1] / 16; i += 32) reinterpret_cast<uint4*>(k)[i] = make_uint4(0u, 0u, 0u, 0u);
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        const int64_t t = first + n * step;
        if (lane == 0) {
            ptx::bulk_store(static_cast<TA*>(p.q_out) + t * p.q_out_stride, ptx::smem_u32(q), static_cast<uint32_t>(ring.sizes[0]));
            if (!APPEND)
                ptx::bulk_store(static_cast<TA*>(p.k_out) + t * p.k_out_stride, ptx::smem_u32(k),
                                static_cast<uint32_t>(ring.sizes[1]));
        }
        if (write) {
            const TA* v = reinterpret_cast<const TA*>(stage + ring.rows[2]);
            const Place at = cache_place(p, note.slot);
            TA *ko = static_cast<TA*>(p.k_out) + at.k, *vo = static_cast<TA*>(p.v_out) + at.v;
            const uint32_t bytes = static_cast<uint32_t>(p.Dh) * sizeof(TA);
            if (lane == 0) {
                if (p.k_head_stride == p.Dh || p.Hk == 1) ptx::bulk_store(ko, ptx::smem_u32(k), bytes * p.Hk);
                else
                    for (int h = 0; h < p.Hk; ++h) ptx::bulk_store(ko + h * p.k_head_stride, ptx::smem_u32(k + h * p.Dh), bytes);
                if (p.v_head_stride == p.Dh || p.Hk == 1) ptx::bulk_store(vo, ptx::smem_u32(v), bytes * p.Hk);
                else
                    for (int h = 0; h < p.Hk; ++h) ptx::bulk_store(vo + h * p.v_head_stride, ptx::smem_u32(v + h * p.Dh), bytes);
            }
        }
        if (lane == 0) ptx::bulk_commit();
        if (++s == S) {
            s = 0;
            parity ^= 1;
        }
    }
    if (lane == 0) ptx::bulk_wait<0>();
    if (!ok) {   // let copies already issued land before the shared memory goes away
        const uint64_t t0 = ptx::globaltimer();
        while (ptx::globaltimer() - t0 < 20000ull) {
        }
    }
}

template <typename TA, bool ADJ, bool APPEND>
cudaError_t launch_turn(const QkParams& p, cudaStream_t s) {
    const int e = static_cast<int>(sizeof(TA)), q = p.Hq * p.Dh * e, k = p.Hk * p.Dh * e;
    TurnRing r = {};
    int at = 0;
    auto place = [&](int bytes) {
        const int here = at;
        at += (bytes + 127) & ~127;
        return here;
    };
    r.sizes[0] = q;
    r.sizes[1] = k;
    r.sizes[2] = APPEND ? k : 0;
    for (int i = 0; i < 3; ++i) r.rows[i] = place(r.sizes[i]);
    r.angles = place(p.rot * 4);
    r.note = place(static_cast<int>(sizeof(Note)));
    r.stage_bytes = at;
    const int room = (SM_SMEM - 1024) / (at + 8);   // stages of an SM
    r.warps = room / 2 < TURN_WARPS ? room / 2 : TURN_WARPS;
    r.stages = r.warps > 0 ? room / r.warps : 0;
    if (r.stages > 4) r.stages = 4;
    // fewer than 6 warps leave too little in flight, and each wants a few tokens: 4096
    // of 48 heads of 128 take 16.3 us here, 15.5 in the kernels with the norm off
    if (r.warps < 6 || p.T < 4ll * r.warps * sm_count()) return launch_fwd<TA, ADJ, APPEND, false>(p, s);
    static std::atomic<uint64_t> done{0};
    auto kernel = turn_kernel<TA, ADJ, APPEND>;
    const cudaError_t err = allow_smem(reinterpret_cast<const void*>(kernel), done);
    if (err != cudaSuccess) return err;
    const size_t smem = static_cast<size_t>(r.warps) * r.stages * (r.stage_bytes + 8);
    kernel<<<sm_count(), r.warps * 32, smem, s>>>(p, r);
    return cudaGetLastError();
}

}  // namespace qk

cudaError_t launch_rope(bool bf16, bool adjacent, bool append, const QkParams& p, cudaStream_t s) {
    g_error_word.may_be_set();
    using B = __nv_bfloat16;
    if (bf16) {
        if (append) return adjacent ? qk::launch_turn<B, true, true>(p, s) : qk::launch_turn<B, false, true>(p, s);
        return adjacent ? qk::launch_turn<B, true, false>(p, s) : qk::launch_turn<B, false, false>(p, s);
    }
    if (append) return adjacent ? qk::launch_turn<float, true, true>(p, s) : qk::launch_turn<float, false, true>(p, s);
    return adjacent ? qk::launch_turn<float, true, false>(p, s) : qk::launch_turn<float, false, false>(p, s);
}

// ------------------------------------------------------------------- table ---
namespace qk {

// Angles are counted in turns modulo 1, as 64-bit fractions: position p of a pair
// whose frequency is F / 2^64 turns a token is at p F / 2^64, and the product's
// overflow is whole turns.  That is exact for every position, where an angle in
// float32 has lost its fraction by p = 2^24, and costs no 64-bit floating point
// (1 instruction in 64 of this GPU's float32).  F itself comes from the host in
// double, u = 2^-53.  The exponent -2j/rot is off by u of it, which moves f by
// 0.37 u at most (x e^-x), the power by a unit in its last place and the rest of the
// unblended way by 9 u of f or of f / factor: 2^-49 max(1, 1/factor) p.  The turns over the
// trained length are off by 5.4 u of them, which are at most `high` inside the blend: 5.4 u
// high / (high - low) more.  F is cut off below 2^-64 turns: 2^-61 p.
struct TableParams {
    uint64_t turn[128];   // F of each pair
    float* out;           // [n, 2 half]: cosines, then sines
    int64_t n;
    int half, quads, rows;   // pairs of a row, runs of four of them, rows of a block
    float amplitude;
};

// a / 2^64 turns as the nearest quarter turn, in the top two bits, and what is left
// of it in the others: `a` has an eighth of a turn (and the rounding of its lower
// half) added, so that the rest is between -1/8 and 1/8.
constexpr uint64_t EIGHTH = (uint64_t(1) << 61) + (uint64_t(1) << 31);

// Cosines and sines of two angles, from the Taylor series of cos(pi x / 4) and
// sin(pi x / 4) for -1 <= x <= 1: their truncation is below 2^-29, the sine's
// first coefficient comes in two parts, and so both are right to 2^-24.
__device__ __forceinline__ void turned2(uint32_t a, uint32_t b, float2 amplitude, float2& c, float2& s) {
    auto both = [](float v) { return make_float2(v, v); };
    const float2 rest = make_float2(static_cast<float>(static_cast<int32_t>((a << 2) ^ 0x80000000u)),
                                    static_cast<float>(static_cast<int32_t>((b << 2) ^ 0x80000000u)));
    const float2 x = __fmul2_rn(rest, both(4.656612873077393e-10f)), w = __fmul2_rn(x, x);   // 2^-31
    float2 y = __ffma2_rn(w, both(3.13361689037812e-07f), both(-3.657620418217724e-05f));
    y = __ffma2_rn(w, y, both(0.00249039457019272f));
    y = __ffma2_rn(w, y, both(-0.08074551218828077f));
    y = __ffma2_rn(w, y, both(-2.1855695031547384e-08f));   // pi / 4 less the float below
    y = __ffma2_rn(x, both(0.78539818525314331f), __fmul2_rn(x, y));
    float2 z = __ffma2_rn(w, both(-2.461136950494199e-08f), both(3.590860448591509e-06f));
    z = __ffma2_rn(w, z, both(-0.00032599188692738996f));
    z = __ffma2_rn(w, z, both(0.0158543442438155f));
    z = __ffma2_rn(w, z, both(-0.30842513753404244f));
    z = __ffma2_rn(w, z, both(1.0f));
    y = __fmul2_rn(y, amplitude);
    z = __fmul2_rn(z, amplitude);
    // quarter turns 1 and 3 swap the two; the cosine is negative in 1 and 2, the sine in 2 and 3
    auto put = [](uint32_t q, float cos, float sin, float& oc, float& os) {
        const bool odd = q & 0x40000000u;
        oc = __uint_as_float(__float_as_uint(odd ? sin : cos) ^ ((q ^ (q << 1)) & 0x80000000u));
        os = __uint_as_float(__float_as_uint(odd ? cos : sin) ^ (q & 0x80000000u));
    };
    put(a, z.x, y.x, c.x, s.x);
    put(b, z.y, y.y, c.y, s.y);
}

__global__ void __launch_bounds__(256)
rope_table_kernel(const __grid_constant__ TableParams p) {
    const int q = static_cast<int>(threadIdx.x) % p.quads, r = static_cast<int>(threadIdx.x) / p.quads;
    if (r >= p.rows) return;
    const int64_t step = static_cast<int64_t>(gridDim.x) * p.rows;
    int64_t row = static_cast<int64_t>(blockIdx.x) * p.rows + r;
    uint64_t at[4], by[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t f = p.turn[4 * q + i];
        at[i] = f * static_cast<uint64_t>(row) + EIGHTH;
        by[i] = f * static_cast<uint64_t>(step);
    }
    const float2 amplitude = make_float2(p.amplitude, p.amplitude);
    float* out = p.out + row * (2 * p.half) + 4 * q;
    for (; row < p.n; row += step, out += step * (2 * p.half)) {
        float2 c[2], s[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            turned2(static_cast<uint32_t>(at[2 * i] >> 32), static_cast<uint32_t>(at[2 * i + 1] >> 32), amplitude, c[i],
                    s[i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) at[i] += by[i];
        *reinterpret_cast<float4*>(out) = make_float4(c[0].x, c[0].y, c[1].x, c[1].y);
        *reinterpret_cast<float4*>(out + p.half) = make_float4(s[0].x, s[0].y, s[1].x, s[1].y);
    }
}

}  // namespace qk

cudaError_t launch_rope_table(int64_t n, int rot, double base, double factor, double original, double low, double high,
                              float amplitude, float* cos_sin, cudaStream_t s) {
    constexpr double TAU = 6.283185307179586476925286766559;
    qk::TableParams p;
    p.half = rot / 2;
    for (int j = 0; j < p.half; ++j) {
        const double f = pow(base, -2.0 * j / rot);
        const double g = fmin(1.0, fmax(0.0, (original * f / TAU - low) / (high - low)));
        const double turn = f * (g + (1.0 - g) / factor) / TAU;
        p.turn[j] = static_cast<uint64_t>(ldexp(turn - floor(turn), 64));
    }
    p.out = cos_sin;
    p.n = n;
    p.quads = p.half / 4;
    p.rows = 256 / p.quads;
    p.amplitude = amplitude;
    int64_t blocks = (n + p.rows - 1) / p.rows;
    if (blocks > 8ll * sm_count()) blocks = 8ll * sm_count();
    qk::rope_table_kernel<<<static_cast<unsigned>(blocks), 256, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace mhc
