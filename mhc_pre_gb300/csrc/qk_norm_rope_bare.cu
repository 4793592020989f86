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

// Cosine and sine of a / 2^64 turns: the nearest quarter turn is taken off in
// integers, so that what is rounded to float32 is at most an eighth.
__device__ __forceinline__ void turned(uint64_t a, float amplitude, float& c, float& s) {
    const uint32_t top = static_cast<uint32_t>((a + 0x80000000ull) >> 32);
    const uint32_t quarter = (top + 0x20000000u) >> 30;
    const int32_t rest = static_cast<int32_t>(top - (quarter << 30));
    float y, x;
    sincospif(static_cast<float>(rest) * 4.656612873077393e-10f, &y, &x);   // 2^-31: in half turns
    const float u = (quarter & 1u) ? y : x, v = (quarter & 1u) ? x : y;
    c = amplitude * (((quarter + 1u) & 2u) ? -u : u);
    s = amplitude * ((quarter & 2u) ? -v : v);
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
        at[i] = f * static_cast<uint64_t>(row);
        by[i] = f * static_cast<uint64_t>(step);
    }
    for (; row < p.n; row += step) {
        float c[4], s[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            turned(at[i], p.amplitude, c[i], s[i]);
            at[i] += by[i];
        }
        float* out = p.out + row * (2 * p.half) + 4 * q;
        *reinterpret_cast<float4*>(out) = make_float4(c[0], c[1], c[2], c[3]);
        *reinterpret_cast<float4*>(out + p.half) = make_float4(s[0], s[1], s[2], s[3]);
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
