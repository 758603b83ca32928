// fp4.cu -- the 4-bit form's quantiser and dequantiser (the form and the rule:
// fp4.cuh).
//
// Quantise.  Two maxima (the row's and each block's), two multiplies and a
// conversion a value: memory bound, so a row is read once and stays in registers
// between its maximum and its codes.  A lane holds 4 contiguous fp32 values or 8
// of 16 bits, a block is 4 or 2 neighbouring lanes, and a row belongs to a warp
// (up to 1024 values) or to a CTA of 256 threads; rows beyond the registers are
// read a second time, from L2.
// Bytes a value: 4 or 2 read, 9 / 16 written.
#include "fp4.cuh"
#include "fp8w_internal.h"

namespace fp8w {

namespace {

constexpr int kFp4Threads = 256;
constexpr int kFp4WarpK = 1024;  // rows up to this go to a warp each

// V values of a row from piece i on, widened to fp32 (exact).
template <int kType>
struct Piece {
    static constexpr int kValues = kType == FP8W_F32 ? 4 : 8;
    uint4 raw;
    __device__ __forceinline__ void load(const void* row, int64_t i) { raw = __ldcs(static_cast<const uint4*>(row) + i); }
    __device__ __forceinline__ void widen(float* f) const {
        const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (kType == FP8W_F32) {
                f[e] = __uint_as_float(u[e]);
            } else {
                f[2 * e] = kType == FP8W_BF16 ? bf16_lo_to_f32(u[e]) : f16_lo_to_f32(u[e]);
                f[2 * e + 1] = kType == FP8W_BF16 ? bf16_hi_to_f32(u[e]) : f16_hi_to_f32(u[e]);
            }
        }
    }
};

// N pieces a thread in registers (0: read twice), T threads a row.
template <int kType, int N, int T>
__global__ void __launch_bounds__(kFp4Threads) quantize_fp4_kernel(const void* w, int64_t n, int64_t k, uint8_t* codes,
                                                                    uint8_t* blocks, float* scales) {
    using P = Piece<kType>;
    constexpr int V = P::kValues, kLanes = 16 / V;  // lanes a block
    const int tid = threadIdx.x % T;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (kFp4Threads / T) + threadIdx.x / T;
    if (T == 32 && row >= n) return;
    const int64_t pieces = k / V;
    const uint8_t* src = static_cast<const uint8_t*>(w) + row * k * (kType == FP8W_F32 ? 4 : 2);
    P held[N ? N : 1];
    float amax = 0.0f;
    auto take = [&](const P& p) {
        float f[V];
        p.widen(f);
#pragma unroll
        for (int e = 0; e < V; ++e) amax = fmaxf(amax, fabsf(f[e]));
    };
    if constexpr (N > 0) {
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (tid + j * T < pieces) held[j].load(src, tid + j * T);
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (tid + j * T < pieces) take(held[j]);
    } else {
        for (int64_t i = tid; i < pieces; i += T) {
            held[0].load(src, i);
            take(held[0]);
        }
    }
    // non-negative floats order like their bit patterns
    amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
    if constexpr (T > 32) {
        __shared__ float red[T / 32];
        if ((tid & 31) == 0) red[tid >> 5] = amax;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < T / 32; ++i) amax = fmaxf(amax, red[i]);
    }
    const float scale = fp4_scale(amax), inverse = __frcp_rn(scale);
    // pieces come in whole blocks (k % 32 == 0), and a block's lanes are in or out together
    auto put = [&](const P& p, int64_t i) {
        const bool in = i < pieces;
        float f[8] = {};
        if (in) p.widen(f);
        float top = 0.0f;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            f[e] = __fmul_rn(f[e], inverse);
            top = fmaxf(top, fabsf(f[e]));
        }
#pragma unroll
        for (int d = 1; d < kLanes; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        const uint32_t byte = fp4_block(top);
        const float bi = fp4_block_inverse(byte);
#pragma unroll
        for (int e = 0; e < V; ++e) f[e] = __fmul_rn(f[e], bi);
        if (!in) return;
        const int64_t at = row * pieces + i;
        if constexpr (V == 8)
            reinterpret_cast<uint32_t*>(codes)[at] = f32x8_to_e2m1(f);
        else
            reinterpret_cast<uint16_t*>(codes)[at] = f32x4_to_e2m1(f[0], f[1], f[2], f[3]);
        if ((i & (kLanes - 1)) == 0) blocks[at / kLanes] = static_cast<uint8_t>(byte);
    };
    if constexpr (N > 0) {
#pragma unroll
        for (int j = 0; j < N; ++j)
            if ((tid & ~31) + j * T < pieces) put(held[j], tid + j * T);
    } else {
        for (int64_t i = tid; (i & ~int64_t(31)) < pieces; i += T) {
            if (i < pieces) held[0].load(src, i);
            put(held[0], i);
        }
    }
    if (tid == 0) scales[row] = scale;
}

template <int kType, int N, int T>
cudaError_t quantize_form(const void* w, int64_t n, int64_t k, uint8_t* codes, uint8_t* blocks, float* scales, cudaStream_t st) {
    constexpr int kRows = kFp4Threads / T;
    quantize_fp4_kernel<kType, N, T><<<static_cast<unsigned>((n + kRows - 1) / kRows), kFp4Threads, 0, st>>>(w, n, k, codes, blocks, scales);
    return cudaGetLastError();
}

template <int kType>
cudaError_t quantize_type(const void* w, int64_t n, int64_t k, uint8_t* codes, uint8_t* blocks, float* scales, cudaStream_t st) {
    constexpr int V = Piece<kType>::kValues;
    const int64_t pieces = k / V;
    if (k <= kFp4WarpK) {
        if (pieces <= 32) return quantize_form<kType, 1, 32>(w, n, k, codes, blocks, scales, st);
        if (pieces <= 64) return quantize_form<kType, 2, 32>(w, n, k, codes, blocks, scales, st);
        return quantize_form<kType, kFp4WarpK / V / 32, 32>(w, n, k, codes, blocks, scales, st);
    }
    const int64_t each = (pieces + kFp4Threads - 1) / kFp4Threads;
    if (each <= 2) return quantize_form<kType, 2, kFp4Threads>(w, n, k, codes, blocks, scales, st);
    if (each <= 4) return quantize_form<kType, 4, kFp4Threads>(w, n, k, codes, blocks, scales, st);
    if (each <= 8) return quantize_form<kType, 8, kFp4Threads>(w, n, k, codes, blocks, scales, st);
    if (each <= 14) return quantize_form<kType, 14, kFp4Threads>(w, n, k, codes, blocks, scales, st);
    return quantize_form<kType, 0, kFp4Threads>(w, n, k, codes, blocks, scales, st);
}

// ------------------------------------------------------------ dequantise --
// The exact product of scale and e4m3 * e2m1 (fp32, 6 significant bits), rounded
// once: 16-bit results as in quantize.cu by hi = fp32(c * s) and its remainder.
// A thread makes 16 bytes a store, kFp4Unroll of them in flight; a word of codes
// lies in one block and one row.  Bytes a value: 9 / 16 read, 2 or 4 written.
constexpr int kFp4Unroll = 4;

template <int OUT>
__device__ __forceinline__ uint32_t fp4_round(float c, float s) {
    const float hi = __fmul_rn(c, s);
    if constexpr (OUT == 0) return __float_as_uint(hi);
    return OUT == 1 ? exact_to_bf16(hi, c, s) : exact_to_f16(hi, c, s);
}

// OUT: 0 fp32, 1 bf16, 2 fp16.
template <int OUT>
__global__ void __launch_bounds__(kFp4Threads) dequantize_fp4_kernel(const uint8_t* codes, const uint8_t* blocks, const float* scales,
                                                                      int64_t k, int64_t nchunk, void* out) {
    constexpr int U = kFp4Unroll, C = OUT == 0 ? 4 : 8;  // values a chunk
    const int64_t cpr = k / C, P = static_cast<int64_t>(gridDim.x) * kFp4Threads, step = U * P;
    const int64_t srow = step / cpr, scol = step - srow * cpr;
    const int64_t i0 = blockIdx.x * static_cast<int64_t>(kFp4Threads) + threadIdx.x;
    int64_t row[U], col[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        row[u] = (i0 + u * P) / cpr;
        col[u] = i0 + u * P - row[u] * cpr;
    }
    for (int64_t i = i0; i < nchunk; i += step) {
        uint32_t cw[U], bl[U];
        float sc[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t v = i + u * P;
            if (v >= nchunk) break;
            cw[u] = C == 8 ? __ldcs(reinterpret_cast<const uint32_t*>(codes) + v) : __ldcs(reinterpret_cast<const uint16_t*>(codes) + v);
            bl[u] = blocks[v / (16 / C)];
            sc[u] = scales[row[u]];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t v = i + u * P;
            if (v >= nchunk) break;
            uint32_t p[4], o[8];
            e2m1x8_to_f16x2(cw[u], p[0], p[1], p[2], p[3]);
            const uint32_t factor = both_lo(block_pair_f16(bl[u]));
#pragma unroll
            for (int e = 0; e < C / 2; ++e) {
                p[e] = f16x2_mul(p[e], factor);  // exact
                o[2 * e] = fp4_round<OUT>(f16_lo_to_f32(p[e]), sc[u]);
                o[2 * e + 1] = fp4_round<OUT>(f16_hi_to_f32(p[e]), sc[u]);
            }
            uint4* dst = static_cast<uint4*>(out) + v;
            if constexpr (OUT == 0)
                __stcs(dst, make_uint4(o[0], o[1], o[2], o[3]));
            else
                __stcs(dst, make_uint4(o[0] | (o[1] << 16), o[2] | (o[3] << 16), o[4] | (o[5] << 16), o[6] | (o[7] << 16)));
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            row[u] += srow;
            col[u] += scol;
            if (col[u] >= cpr) col[u] -= cpr, ++row[u];
        }
    }
}

}  // namespace

cudaError_t launch_quantize_fp4(const void* w, int w_dtype, int64_t n, int64_t k, uint8_t* codes, uint8_t* blocks, float* scales,
                                cudaStream_t st) {
    if (w_dtype == FP8W_F32) return quantize_type<FP8W_F32>(w, n, k, codes, blocks, scales, st);
    if (w_dtype == FP8W_BF16) return quantize_type<FP8W_BF16>(w, n, k, codes, blocks, scales, st);
    return quantize_type<FP8W_F16>(w, n, k, codes, blocks, scales, st);
}

cudaError_t launch_dequantize_fp4(const uint8_t* codes, const uint8_t* blocks, const float* scales, int64_t n, int64_t k,
                                  int out_dtype, void* w, cudaStream_t st) {
    int sms = 0;
    cudaError_t e = device_sm_count(sms);
    if (e != cudaSuccess) return e;
    const int64_t nchunk = n * (k / (out_dtype == 0 ? 4 : 8));
    int64_t grid = (nchunk + kFp4Threads * kFp4Unroll - 1) / (kFp4Threads * kFp4Unroll);
    if (grid > sms * 8) grid = sms * 8;
    const unsigned g = static_cast<unsigned>(grid);
    if (out_dtype == 1)
        dequantize_fp4_kernel<1><<<g, kFp4Threads, 0, st>>>(codes, blocks, scales, k, nchunk, w);
    else if (out_dtype == 2)
        dequantize_fp4_kernel<2><<<g, kFp4Threads, 0, st>>>(codes, blocks, scales, k, nchunk, w);
    else
        dequantize_fp4_kernel<0><<<g, kFp4Threads, 0, st>>>(codes, blocks, scales, k, nchunk, w);
    return cudaGetLastError();
}

}  // namespace fp8w
