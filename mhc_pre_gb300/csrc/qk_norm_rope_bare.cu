// qk_norm_rope_bare.cu -- the position rotation without the normalisation
// (forward, backward, and into a paged cache), and the table of its angles.
//
// The rotation runs in the kernels of qk_norm_rope_fwd.cuh with NORM off:
//   (a, b) -> (a c - b s, b c + a s),   backward: the transpose, s -> -s.
// The transpose needs nothing of the forward, so its backward is the same pass.
#include <math.h>

#include "qk_norm_rope_fwd.cuh"

namespace mhc {

static ErrorWord g_error_word;

cudaError_t read_and_clear_rope_error(unsigned* word) { return g_error_word.read_and_clear(g_qk_error, word); }

cudaError_t launch_rope(bool bf16, bool adjacent, bool append, const QkParams& p, cudaStream_t s) {
    g_error_word.may_be_set();
    using B = __nv_bfloat16;
    if (bf16) {
        if (append) return adjacent ? qk::launch_fwd<B, true, true, false>(p, s) : qk::launch_fwd<B, false, true, false>(p, s);
        return adjacent ? qk::launch_fwd<B, true, false, false>(p, s) : qk::launch_fwd<B, false, false, false>(p, s);
    }
    if (append)
        return adjacent ? qk::launch_fwd<float, true, true, false>(p, s) : qk::launch_fwd<float, false, true, false>(p, s);
    return adjacent ? qk::launch_fwd<float, true, false, false>(p, s) : qk::launch_fwd<float, false, false, false>(p, s);
}

// ------------------------------------------------------------------- table ---
namespace qk {

// Angles are counted in turns modulo 1, as 64-bit fractions: position p of a pair
// whose frequency is F / 2^64 turns a token is at p F / 2^64, and the product's
// overflow is whole turns.  That is exact for every position, where an angle in
// float32 has lost its fraction by p = 2^24, and costs no 64-bit floating point
// (1 instruction in 64 of this GPU's float32).  F itself comes from the host in
// double: an angle is off by at most p f 2^-52.
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
