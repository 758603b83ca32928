// rope.cu -- kernel K6: rotary positions, and the append of keys and values to
// a paged cache with the rotation applied on the way.
//
// A pair (a, b) of a head turns by its token's angle:
//   (a cos - b sin, b cos + a sin),  products and sums in fp32, each rounded
// once (no fused multiply-add: the result is then one function of the inputs,
// and codes made from it are too).  Keys and values for an e4m3 cache take the
// weight quantiser's rule on the fp32 row: scale = amax / 448 (1.0 if that is
// 0), code = nearest-even e4m3 of the IEEE quotient.
//
// Memory bound: every value is read and written once, and three operations a
// value are nothing beside that.  A lane holds 16 values of a head, the two
// 8-value chunks that make 8 whole pairs: chunks i and i + rot_dim / 16 with
// pairs in halves, 2 i and 2 i + 1 with interleaved ones, so one set of eight
// cosines and sines serves either form and a lane writes what it has read
// (in-place calls need no further order).  A warp takes a token, or with few
// tokens a part of its heads: 32 / P heads a step (P lanes a head), kAhead
// steps' loads in flight, the first before the position and the table row are
// asked for, and its cosines and sines stay in registers over the heads.  All
// loads are ordinary ones, none of the read-only path: the kernel starts while
// those ahead of it in the stream still write, and its wait orders ordinary loads.
// 16384 tokens of 40 heads of 128, three axes: 59.3 us, 5.8 TB/s (87% of the
// measured copy rate), one axis 54.8 us; 8192 tokens appended 34.6 us (88%), as
// codes 42.4 us (66%: sixteen IEEE divisions a lane); one token 1.7 us.
#include "fp8w_device.cuh"
#include "fp8w_internal.h"

namespace fp8w {

__device__ int g_rope_error;

namespace {

constexpr int kRopeWarps = 4;
constexpr int kRopeFill = 16;  // warps an SM up to which a token's heads are divided
constexpr int kAhead = 2;  // steps of a warp in flight: 2 KB
// Blocks an SM where a warp takes a whole token: the warps in flight count, and
// for them the registers (344 MB: 6 blocks 63.1 us, 7 58.5, 8 59.1; 8192 tokens
// appended 35.2, 33.9, 37.5; as codes, whose divisions take more of them, 4 blocks
// 47.1 us, 5 41.6, 6 43.1).  With fewer tokens a block's own time counts, and all
// registers help it (1161 tokens: 5.9 us when with the bound it was 7.6).
constexpr int kDenseBlocks = 7, kDenseBlocksCodes = 5;

struct RopeParams {
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    uint16_t* q_out;
    int64_t q_stride, k_stride, v_stride, q_out_stride, tokens;
    int q_heads, kv_heads, head_dim;
    const int32_t* positions;  // null: no rotation
    const float* table;
    int64_t max_pos;
    int rot_dim, interleaved, axes;
    int bound[4];  // pairs below bound[a] belong to axes 0 .. a
    const int64_t* slots;
    uint8_t* kc;
    uint8_t* vc;
    float* ks;
    float* vs;
    int64_t num_pages, page_stride, head_stride, token_stride;
    int page_size, log_page;
    int parts, per_part;  // warps a token, steps of each
};

template <bool kBf16>
__device__ __forceinline__ void widen(const uint4 v, float* f) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        f[2 * e] = kBf16 ? bf16_lo_to_f32(u[e]) : f16_lo_to_f32(u[e]);
        f[2 * e + 1] = kBf16 ? bf16_hi_to_f32(u[e]) : f16_hi_to_f32(u[e]);
    }
}

template <bool kBf16>
__device__ __forceinline__ uint4 narrow(const float* f) {
    uint32_t u[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if constexpr (kBf16)
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u[e]) : "f"(f[2 * e + 1]), "f"(f[2 * e]));
        else
            asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(u[e]) : "f"(f[2 * e + 1]), "f"(f[2 * e]));
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

// What a call does: rotate, or also append to a 16-bit cache or one of codes.
constexpr int kRotate = 0, kAppend16 = 1, kAppendCodes = 2;

// P lanes (a power of two >= head_dim / 16) work on a head.
template <int P, bool kBf16, int kKind, bool kDense>
__global__ void __launch_bounds__(kRopeWarps * 32, !kDense ? 1 : kKind == kAppendCodes ? kDenseBlocksCodes : kDenseBlocks) rope_kernel(const __grid_constant__ RopeParams p) {
    pdl_launch_dependents();
    constexpr int kHeads = 32 / P;  // heads a step
    constexpr bool kAppend = kKind != kRotate, kFp8 = kKind == kAppendCodes;
    const int lane = threadIdx.x & 31, item = lane & (P - 1);
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kRopeWarps + (threadIdx.x >> 5);
    // a token's parts are few where there are more than one: 32 bits
    const int64_t token = kDense ? unit : static_cast<int64_t>(static_cast<uint32_t>(unit) / static_cast<uint32_t>(p.parts));
    if (token >= p.tokens) return;
    const int part = kDense ? 0 : static_cast<int>(unit - token * p.parts);
    const bool live = item * 16 < p.head_dim;
    const int half = p.rot_dim >> 1;
    const bool turns = p.positions && item * 16 < p.rot_dim;
    // the item's two chunks (first values)
    const int c0 = turns ? (p.interleaved ? item * 16 : item * 8) : item * 16;
    const int c1 = turns && !p.interleaved ? half + item * 8 : c0 + 8;
    const int heads = p.q_heads + (kAppend ? 2 * p.kv_heads : 0), steps = (heads + kHeads - 1) / kHeads;
    const int first = part * p.per_part, last = min(first + p.per_part, steps);
    pdl_wait();

    int64_t slot = 0;
    if constexpr (kAppend) slot = p.slots[token];
    uint4 x[kAhead][2];
    auto head_of = [&](int step) { return step * kHeads + lane / P; };
    const uint16_t* const q_row = p.q + token * p.q_stride;
    const uint16_t* const k_row = p.k + token * p.k_stride;
    const uint16_t* const v_row = p.v + token * p.v_stride;
    auto load = [&](int step, uint4 (&y)[2]) {
        const int h = head_of(step);
        const bool is_q = !kAppend || h < p.q_heads, is_k = !is_q && h < p.q_heads + p.kv_heads;
        const int kvh = h - p.q_heads - (is_k ? 0 : p.kv_heads);
        const uint16_t* src = (is_q ? q_row : is_k ? k_row : v_row) + static_cast<int64_t>(is_q ? h : kvh) * p.head_dim;
        y[0] = y[1] = make_uint4(0u, 0u, 0u, 0u);
        if (live && step < last && h < heads) {
            // values that do not turn go by their item's own chunks
            y[0] = *reinterpret_cast<const uint4*>(src + (is_q || is_k ? c0 : item * 16));
            y[1] = *reinterpret_cast<const uint4*>(src + (is_q || is_k ? c1 : item * 16 + 8));
        }
    };
#pragma unroll
    for (int u = 0; u < kAhead; ++u) load(first + u, x[u]);

    float cs[8], sn[8];
    if (turns) {
        int64_t pos[4];
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            if (a >= p.axes) break;
            int64_t at = p.positions[a * p.tokens + token];
            if (at < 0 || at >= p.max_pos) {
                atomicCAS(&g_rope_error, 0, 6000 + kErrIndex);
                at = at < 0 ? 0 : p.max_pos - 1;
            }
            pos[a] = at;
        }
        auto axis_of = [&](int pair) {
            int a = 0;
#pragma unroll
            for (int i = 0; i < 3; ++i) a += (i + 1 < p.axes && pair >= p.bound[i]) ? 1 : 0;
            return a;
        };
        auto row_of = [&](int a) { return p.table + (a == 0 ? pos[0] : a == 1 ? pos[1] : a == 2 ? pos[2] : pos[3]) * p.rot_dim; };
        const int i0 = item * 8;
        if (axis_of(i0) == axis_of(i0 + 7)) {
            const float* row = row_of(axis_of(i0)) + i0;
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
                const float4 c = *reinterpret_cast<const float4*>(row + e);
                const float4 s = *reinterpret_cast<const float4*>(row + half + e);
                cs[e] = c.x, cs[e + 1] = c.y, cs[e + 2] = c.z, cs[e + 3] = c.w;
                sn[e] = s.x, sn[e + 1] = s.y, sn[e + 2] = s.z, sn[e + 3] = s.w;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float* row = row_of(axis_of(i0 + e)) + i0 + e;
                cs[e] = *row;
                sn[e] = row[half];
            }
        }
    }
    const int64_t page = kAppend && slot >= 0 ? slot >> p.log_page : 0, off = slot - page * p.page_size;
    bool kept = kAppend && slot >= 0;  // the token goes into the cache
    if (kAppend && kept && page >= p.num_pages) {
        atomicCAS(&g_rope_error, 0, 6000 + kErrIndex);
        kept = false;
    }

    uint16_t* const q_out_row = p.q_out + token * p.q_out_stride;
    auto finish = [&](int step, uint4 x0, uint4 x1) {
        const int h = head_of(step);
        const bool is_q = !kAppend || h < p.q_heads, is_k = !is_q && h < p.q_heads + p.kv_heads;
        const bool work = live && h < heads && (is_q || kept);
        const int kvh = is_q ? 0 : h - p.q_heads - (is_k ? 0 : p.kv_heads);
        const int s0 = (is_q || is_k) ? c0 : item * 16, s1 = (is_q || is_k) ? c1 : item * 16 + 8;
        float f[16];
        widen<kBf16>(x0, f);
        widen<kBf16>(x1, f + 8);
        if (turns && (is_q || is_k)) {
            if (p.interleaved) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float a = f[2 * e], b = f[2 * e + 1];
                    f[2 * e] = __fsub_rn(__fmul_rn(a, cs[e]), __fmul_rn(b, sn[e]));
                    f[2 * e + 1] = __fadd_rn(__fmul_rn(b, cs[e]), __fmul_rn(a, sn[e]));
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float a = f[e], b = f[8 + e];
                    f[e] = __fsub_rn(__fmul_rn(a, cs[e]), __fmul_rn(b, sn[e]));
                    f[8 + e] = __fadd_rn(__fmul_rn(b, cs[e]), __fmul_rn(a, sn[e]));
                }
            }
            x0 = narrow<kBf16>(f);
            x1 = narrow<kBf16>(f + 8);
        }
        if (is_q && work) {
            uint16_t* dst = q_out_row + static_cast<int64_t>(h) * p.head_dim;
            *reinterpret_cast<uint4*>(dst + s0) = x0;
            *reinterpret_cast<uint4*>(dst + s1) = x1;
        }
        if constexpr (kFp8) {
            if (__all_sync(0xffffffffu, is_q)) return;  // a step of queries only
            float amax = 0.0f;
#pragma unroll
            for (int e = 0; e < 16; ++e) amax = fmaxf(amax, fabsf(f[e]));
#pragma unroll
            for (int d = P / 2; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
            if (!is_q && work) {
                float s = __fdiv_rn(amax, 448.0f);
                s = s == 0.0f ? 1.0f : s;
                uint32_t c[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint16_t lo = f32x2_to_e4m3x2(__fdiv_rn(f[4 * e], s), __fdiv_rn(f[4 * e + 1], s));
                    const uint16_t hi = f32x2_to_e4m3x2(__fdiv_rn(f[4 * e + 2], s), __fdiv_rn(f[4 * e + 3], s));
                    c[e] = static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
                }
                uint8_t* dst = (is_k ? p.kc : p.vc) + page * p.page_stride + kvh * p.head_stride + off * p.token_stride;
                *reinterpret_cast<uint2*>(dst + s0) = make_uint2(c[0], c[1]);
                *reinterpret_cast<uint2*>(dst + s1) = make_uint2(c[2], c[3]);
                if (item == 0) (is_k ? p.ks : p.vs)[(page * p.kv_heads + kvh) * p.page_size + off] = s;
            }
        } else if (kAppend && !is_q && work) {
            uint16_t* dst = reinterpret_cast<uint16_t*>(is_k ? p.kc : p.vc) + page * p.page_stride +
                            kvh * p.head_stride + off * p.token_stride;
            *reinterpret_cast<uint4*>(dst + s0) = x0;
            *reinterpret_cast<uint4*>(dst + s1) = x1;
        }
    };
    for (int step = first; step < last; step += kAhead) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (step + u >= last) break;
            const uint4 x0 = x[u][0], x1 = x[u][1];
            load(step + u + kAhead, x[u]);
            finish(step + u, x0, x1);
        }
    }
}

template <int P, bool kDense>
cudaError_t launch_form(const cudaLaunchConfig_t& cfg, const RopeParams& p, bool bf16, bool fp8) {
    if (fp8)
        return bf16 ? cudaLaunchKernelEx(&cfg, rope_kernel<P, true, kAppendCodes, kDense>, p)
                    : cudaLaunchKernelEx(&cfg, rope_kernel<P, false, kAppendCodes, kDense>, p);
    if (p.kv_heads)
        return bf16 ? cudaLaunchKernelEx(&cfg, rope_kernel<P, true, kAppend16, kDense>, p)
                    : cudaLaunchKernelEx(&cfg, rope_kernel<P, false, kAppend16, kDense>, p);
    return bf16 ? cudaLaunchKernelEx(&cfg, rope_kernel<P, true, kRotate, kDense>, p)
                : cudaLaunchKernelEx(&cfg, rope_kernel<P, false, kRotate, kDense>, p);
}

template <int P>
cudaError_t launch_p(RopeParams p, bool bf16, bool fp8, cudaStream_t st) {
    int sms = 0;
    cudaError_t e = device_sm_count(sms);
    if (e != cudaSuccess) return e;
    // one warp a token; with few tokens a token's heads go to several
    const int steps = (p.q_heads + 2 * p.kv_heads + 32 / P - 1) / (32 / P);
    const int64_t want = (static_cast<int64_t>(sms) * kRopeFill + p.tokens - 1) / p.tokens;
    const int parts = static_cast<int>(want < steps ? want : steps);
    p.per_part = (((steps + parts - 1) / parts + kAhead - 1) / kAhead) * kAhead;  // whole rounds
    if (p.tokens * steps <= static_cast<int64_t>(sms) * kRopeFill) p.per_part = 1;  // a warp for each step
    p.parts = (steps + p.per_part - 1) / p.per_part;
    const int64_t blocks = (p.tokens * p.parts + kRopeWarps - 1) / kRopeWarps;
    if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(kRopeWarps * 32);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (p.parts > 1) return launch_form<P, false>(cfg, p, bf16, fp8);
    return launch_form<P, true>(cfg, p, bf16, fp8);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t st) {
    RopeParams p = {};
    p.q = static_cast<const uint16_t*>(a.q);
    p.q_out = static_cast<uint16_t*>(a.q_out);
    p.q_stride = a.q_stride;
    p.q_out_stride = a.q_out_stride;
    p.q_heads = a.q ? a.q_heads : 0;
    p.tokens = a.tokens;
    p.head_dim = a.head_dim;
    if (a.spec) {
        p.positions = a.positions;
        p.table = a.spec->table;
        p.max_pos = a.spec->max_pos;
        p.rot_dim = a.spec->rot_dim;
        p.interleaved = a.spec->interleaved;
        p.axes = a.spec->axes;
        for (int i = 0, sum = 0; i < 4; ++i) p.bound[i] = sum += a.spec->sections[i];
    }
    bool fp8 = false;
    if (a.cache) {
        const fp8w_kv_cache& c = *a.cache;
        p.k = static_cast<const uint16_t*>(a.k);
        p.v = static_cast<const uint16_t*>(a.v);
        p.k_stride = a.k_stride;
        p.v_stride = a.v_stride;
        p.kv_heads = c.kv_heads;
        p.slots = a.slots;
        p.kc = static_cast<uint8_t*>(c.k);
        p.vc = static_cast<uint8_t*>(c.v);
        p.ks = c.k_scales;
        p.vs = c.v_scales;
        p.num_pages = c.num_pages;
        p.page_stride = c.page_stride;
        p.head_stride = c.head_stride;
        p.token_stride = c.token_stride;
        p.page_size = c.page_size;
        while ((1 << p.log_page) < c.page_size) ++p.log_page;
        fp8 = c.dtype == FP8W_E4M3;
    }
    const bool bf16 = a.act == FP8W_BF16;
    const int items = a.head_dim / 16;
    if (items <= 1) return launch_p<1>(p, bf16, fp8, st);
    if (items <= 2) return launch_p<2>(p, bf16, fp8, st);
    if (items <= 4) return launch_p<4>(p, bf16, fp8, st);
    if (items <= 8) return launch_p<8>(p, bf16, fp8, st);
    return launch_p<16>(p, bf16, fp8, st);
}

int read_rope_device_error() {
    int v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_rope_error, sizeof v) != cudaSuccess) return -1;
    if (v != 0 && cudaMemcpyToSymbol(g_rope_error, &zero, sizeof zero) != cudaSuccess) return -1;
    return v;
}

}  // namespace fp8w
