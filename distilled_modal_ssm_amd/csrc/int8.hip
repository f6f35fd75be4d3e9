// int8.hip -- products in 8-bit integers: rows of activations and of weights as
// whole multiples of a scale of their own, their products summed exactly in 32 bits
// on the matrix cores, the scales applied to the sums.
#include "hm_internal.hpp"

namespace hm {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ i32x4 mfma_i8(uint4 a, uint4 b, i32x4 c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}

// ------------------------------------------------------------------ rows in 8 bits

// rint(127 x / amax), the integer of the exact quotient: in float32, off by less than
// 127 * 2^-22, and again in float64 where that could matter (its product is exact, and
// a quotient of two 24-bit numbers is never nearer to a border than 2^-32 without
// being on it).
__device__ __forceinline__ int quantized(float x, float amax, float inverse) {
    const float r = x * inverse, n = rintf(r);
    if (fabsf(r - n) < 0.4999f && amax > 1e-30f) return (int)n;
    return (int)rint((double)x * 127.0 / (double)amax);
}

// One workgroup a row: the largest magnitude (as bits, where NaN and infinities come
// last) and the sum of squares, then the row again out of the cache.
template <int ACT>
__global__ __launch_bounds__(256) void quantize_rows_kernel(QuantArgs a) {
    using A = Act<ACT>;
    __shared__ uint32_t most[4];
    __shared__ float sums[4];
    const int64_t m = blockIdx.x;
    const typename A::T *x = static_cast<const typename A::T *>(a.x) + m * a.ldx;
    int8_t *q = a.q + m * a.ldq;
    const int tid = threadIdx.x, K = (int)a.K;
    uint32_t top = 0;
    float sum = 0.0f;
    for (int k = tid; k < K; k += 256) {
        const float v = A::ld(x + k);
        const uint32_t bits = __float_as_uint(v) & 0x7fffffffu;
        top = bits > top ? bits : top;
        sum = fmaf(v, v, sum);
    }
    for (int s = 32; s > 0; s >>= 1) {
        const uint32_t other = __shfl_xor(top, s);
        top = other > top ? other : top;
        sum += __shfl_xor(sum, s);
    }
    if (tid % 64 == 0) {
        most[tid / 64] = top;
        sums[tid / 64] = sum;
    }
    __syncthreads();
    for (int w = 0; w < 4; ++w) top = most[w] > top ? most[w] : top;
    sum = (sums[0] + sums[1]) + (sums[2] + sums[3]);
    const bool whole = top < 0x7f800000u;
    const float amax = __uint_as_float(top), inverse = 127.0f / amax;
    const int end = (K + 63) / 64 * 64;
    for (int k = tid; k < end; k += 256) q[k] = k < K && whole && top > 0 ? (int8_t)quantized(A::ld(x + k), amax, inverse) : 0;
    if (tid == 0) {
        float s = amax / 127.0f;
        if (a.rms) s = s / sqrtf(sum / (float)K + a.eps);
        a.scale[m] = whole ? s : __builtin_nanf("");
    }
}

// ------------------------------------------------------------------ products

// One wave 16 x 16 outputs.  The W fragment is the first operand: lane l holds row
// l % 16 of A's tile and columns 4 (l / 16) .. + 3.
template <int ACT>
__global__ __launch_bounds__(64) void dense_int8_kernel(Int8GemmArgs g) {
    using A = Act<ACT>;
    const int64_t tiles_n = (g.N + 15) / 16, m0 = blockIdx.x / tiles_n * 16, n0 = blockIdx.x % tiles_n * 16;
    const int lane = threadIdx.x, r = lane % 16, c = lane / 16;
    const int64_t m = m0 + r < g.M ? m0 + r : g.M - 1, n = n0 + r < g.N ? n0 + r : g.N - 1;
    const int8_t *pa = g.A + m * g.lda + 16 * c, *pw = g.W + n * g.ldw + 16 * c;
    i32x4 acc = {0, 0, 0, 0};
    for (int64_t k = 0; k < g.K; k += 64)
        acc = mfma_i8(*reinterpret_cast<const uint4 *>(pw + k), *reinterpret_cast<const uint4 *>(pa + k), acc);
    if (m0 + r >= g.M) return;
    const float sa = g.a_scale[m];
    for (int j = 0; j < 4; ++j) {
        const int64_t col = n0 + 4 * c + j;
        if (col < g.N) A::st(static_cast<typename A::T *>(g.C) + m * g.ldc + col, (float)acc[j] * sa * g.w_scale[col]);
    }
}

}  // namespace

hipError_t launch_quantize_rows(const QuantArgs &a, hipStream_t stream) {
    if (a.act == kBF16) quantize_rows_kernel<kBF16><<<dim3((unsigned)a.M), 256, 0, stream>>>(a);
    else quantize_rows_kernel<kF32><<<dim3((unsigned)a.M), 256, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_dense_int8(const Int8GemmArgs &g, hipStream_t stream) {
    const dim3 grid((unsigned)((g.M + 15) / 16 * ((g.N + 15) / 16)));
    if (g.act == kBF16) dense_int8_kernel<kBF16><<<grid, 64, 0, stream>>>(g);
    else dense_int8_kernel<kF32><<<grid, 64, 0, stream>>>(g);
    return hipGetLastError();
}

}  // namespace hm
