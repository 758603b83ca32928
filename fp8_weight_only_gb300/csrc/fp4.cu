// fp4.cu -- the 4-bit form's quantiser and dequantiser (the form and the rule:
// fp4.cuh).
//
// Quantise.  Two maxima (the row's and each block's), two multiplies and a
// conversion a value: memory bound, so a row is read once and stays in registers
// between its maximum and its codes.  A lane holds 4 contiguous fp32 values or 8
// of 16 bits, a block is 4 or 2 neighbouring lanes, and a row belongs to a warp
// (up to 1024 values) or to a CTA of 256 threads; rows beyond the registers are
// read a second time, from L2.
// Bytes a value: 4 or 2 read, 9 / 16 written.  14336 x 4096 of fp32: 46.7 us, 5.7 TB/s
// (85% of the measured copy rate), of bf16 or fp16 32 us (70%).
#include <type_traits>

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
// The exact product of scale and e4m3 * e2m1 (6 significant bits, exact in fp16),
// rounded once.  16 bits: the fp32 product is taken towards zero with its last bit
// set where that dropped anything, so that the second rounding sees on which side of
// a middle the product lies (three instructions, and half of one for the pair).
// A thread takes a block of 16 values at a time, kFp4Unroll of them in flight.
// Bytes a value: 9 / 16 read, 2 or 4 written.  14336 x 4096 to bf16 27.9 us (80% of the
// measured copy rate), fp16 32.8 (68%), fp32 80.5 (49%: a thread's four 16-byte stores
// are 64 bytes from its neighbours').  To bf16 the schedulers issue 0.59 of the time, the
// ALU pipe is at 58% and the largest stall is for loads: neither alone bounds it.  (With
// a division by the row and single 16-bit conversions a quarter slower.)
constexpr int kFp4Unroll = 4;

// hi and a sticky last bit: rounds to fewer bits as the exact product does.  kTiny:
// for scales below kTinyScale, whose product can drop bits below fp32's subnormal
// numbers; what it drops is looked at 2^64 times as large, exactly.
constexpr float kTinyScale = 0x1p-100f;
template <bool kTiny>
__device__ __forceinline__ float mul_sticky(float c, float s) {
    const float hi = __fmul_rz(c, s);
    const float rest = kTiny ? fmaf(c * 0x1p64f, s, hi * -0x1p64f) : fmaf(c, s, -hi);
    // (an infinite scale's rest is NaN: its product is what it is)
    return fabsf(rest) > 0.0f ? __uint_as_float(__float_as_uint(hi) | 1u) : hi;
}

struct Fp4Walk {        // blocks of 16 values, a grid of threads apart
    int64_t blocks;     // of all rows
    int64_t per_row;    // of a row
    int64_t step_row;   // a grid of threads: rows and blocks of a row
    int64_t step_col;
};

// OUT: 0 fp32, 1 bf16, 2 fp16.
template <int OUT>
__global__ void __launch_bounds__(kFp4Threads) dequantize_fp4_kernel(const uint8_t* codes, const uint8_t* blocks, const float* scales,
                                                                      void* out, const __grid_constant__ Fp4Walk w) {
    const int64_t P = static_cast<int64_t>(gridDim.x) * kFp4Threads;
    int64_t i = blockIdx.x * static_cast<int64_t>(kFp4Threads) + threadIdx.x;
    // (one division, of 32 bits where that is enough)
    int64_t row = (w.blocks >> 32) == 0 ? static_cast<int64_t>(static_cast<uint32_t>(i) / static_cast<uint32_t>(w.per_row)) : i / w.per_row;
    int64_t col = i - row * w.per_row;
    while (i < w.blocks) {
        uint2 cw[kFp4Unroll];
        uint32_t bl[kFp4Unroll];
        float sc[kFp4Unroll];
#pragma unroll
        for (int u = 0; u < kFp4Unroll; ++u) {
            const int64_t v = i + u * P;
            if (v < w.blocks) {
                cw[u] = __ldcs(reinterpret_cast<const uint2*>(codes) + v);
                bl[u] = blocks[v];
                sc[u] = scales[row];
            }
            row += w.step_row;
            col += w.step_col;
            if (col >= w.per_row) col -= w.per_row, ++row;
        }
#pragma unroll
        for (int u = 0; u < kFp4Unroll; ++u) {
            const int64_t v = i + u * P;
            if (v >= w.blocks) break;
            const uint32_t factor = both_lo(block_pair_f16(bl[u]));
            constexpr int kWords = OUT == 0 ? 16 : 8;
            uint32_t o[kWords];
            auto convert = [&](auto tiny) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t p[4];
                    e2m1x8_to_f16x2(h ? cw[u].y : cw[u].x, p[0], p[1], p[2], p[3]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        p[e] = f16x2_mul(p[e], factor);  // exact
                        const float x = f16_lo_to_f32(p[e]), y = f16_hi_to_f32(p[e]);
                        if constexpr (OUT == 0) {
                            o[8 * h + 2 * e] = __float_as_uint(__fmul_rn(x, sc[u]));
                            o[8 * h + 2 * e + 1] = __float_as_uint(__fmul_rn(y, sc[u]));
                        } else {
                            constexpr bool kTiny = decltype(tiny)::value;
                            const float a = mul_sticky<kTiny>(x, sc[u]), b = mul_sticky<kTiny>(y, sc[u]);
                            if constexpr (OUT == 1)
                                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o[4 * h + e]) : "f"(b), "f"(a));
                            else
                                asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(o[4 * h + e]) : "f"(b), "f"(a));
                        }
                    }
                }
            };
            if (OUT == 1 && fabsf(sc[u]) < kTinyScale)
                convert(std::integral_constant<bool, OUT == 1>{});
            else
                convert(std::false_type{});
            uint4* dst = static_cast<uint4*>(out) + v * (kWords / 4);
#pragma unroll
            for (int q = 0; q < kWords; q += 4) __stcs(dst + q / 4, make_uint4(o[q], o[q + 1], o[q + 2], o[q + 3]));
        }
        i += kFp4Unroll * P;
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
                                  int out_dtype, void* w_out, cudaStream_t st) {
    int sms = 0;
    cudaError_t e = device_sm_count(sms);
    if (e != cudaSuccess) return e;
    Fp4Walk w;
    w.per_row = k / 16;
    w.blocks = n * w.per_row;
    int64_t grid = (w.blocks + kFp4Threads * kFp4Unroll - 1) / (kFp4Threads * kFp4Unroll);
    if (w.blocks <= static_cast<int64_t>(sms) * kFp4Threads * 2) grid = (w.blocks + kFp4Threads - 1) / kFp4Threads;  // few: one each
    if (grid > sms * 8) grid = sms * 8;
    const int64_t threads = grid * kFp4Threads;
    w.step_row = threads / w.per_row;
    w.step_col = threads - w.step_row * w.per_row;
    const unsigned g = static_cast<unsigned>(grid);
    if (out_dtype == 1)
        dequantize_fp4_kernel<1><<<g, kFp4Threads, 0, st>>>(codes, blocks, scales, w_out, w);
    else if (out_dtype == 2)
        dequantize_fp4_kernel<2><<<g, kFp4Threads, 0, st>>>(codes, blocks, scales, w_out, w);
    else
        dequantize_fp4_kernel<0><<<g, kFp4Threads, 0, st>>>(codes, blocks, scales, w_out, w);
    return cudaGetLastError();
}

}  // namespace fp8w
