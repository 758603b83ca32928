// attention.cuh -- what the two paged attention kernels share (attention.cu:
// many rows, on tcgen05; attention_few.cu: few rows): their parameters, the
// search for a tile's sequence, and small arithmetic wrappers.
#pragma once

#include "fp8w_device.cuh"
#include "fp8w_internal.h"

namespace fp8w {

constexpr float kLog2e = 1.4426950408889634f;
#define kNegInf __int_as_float(0xff800000)

// Forms of a cache: 16-bit values, e4m3 codes with a scale a slot and head, or the
// 4-bit form (fp4.cuh) with a scale a slot and head.
constexpr int kForm16 = 0, kFormE4m3 = 1, kFormFp4 = 2;

struct AttnParams {
    const uint16_t* q;
    uint16_t* out;
    int64_t q_stride, out_stride, tokens;
    const int32_t* table;
    const int32_t* lens;
    const int32_t* starts;
    int64_t table_width;
    const void* k;  // the cache, for the kernel that reads it without tensor maps
    const void* v;
    int64_t page_stride, head_stride, token_stride;
    const float* k_scales;
    const float* v_scales;
    const uint8_t* k_blocks;  // 4 bits: scales of blocks
    const uint8_t* v_blocks;
    int64_t num_pages;
    int seqs, kv_heads, group, head_dim, page_size, log_page;
    uint32_t group_inverse;  // 2^32 / group rounded up (0 for 1)
    float c;         // scale * log2(e)
    int64_t window;  // 0: none
    int row_tiles;   // bound on the row tiles of all sequences
    int cl;          // CTAs a cluster
};

// 16 bytes that are read once, not kept in L1.  An ordinary load, as all loads of
// operands here are: these kernels start while those ahead of them in the stream
// still write pages, scales and indices, and the wait for them orders ordinary
// loads only, not those of the read-only path (by which a decode batch of 1.2 GB
// took 222.8 us, and takes 224.6 so).
__device__ __forceinline__ uint4 ld_stream_v4(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// A tile of `tile_rows` rows (counted token * group + head) of one sequence.
struct SeqTile {
    int seq, inner;        // the sequence, the tile's number in it
    int64_t begin, count;  // its first new token, its new tokens
    int64_t len;           // its tokens in the cache (0 where that is out of range)
};

// The sequence of row tile `tile`, by a scan of the sequences' new tokens 32 at
// a time; every warp computes it alike.  Later rows see more keys, so a
// sequence's tiles come last rows first.  `report`: the warp that also looks at
// all of starts and records what is wrong with them.
__device__ __forceinline__ bool find_tile(const AttnParams& p, int tile_rows, int tile, bool report, int* error, SeqTile& f) {
    const int lane = threadIdx.x & 31;
    f.seq = -1;
    if (!p.starts) {
        const int per = (p.group + tile_rows - 1) / tile_rows;
        f.seq = tile / per;
        f.inner = tile - f.seq * per;
        if (f.seq >= p.seqs) return false;
        f.begin = f.seq;
        f.count = 1;
        f.len = p.lens[f.seq];
    } else {
        int64_t before = 0;
        for (int b0 = 0; b0 < p.seqs; b0 += 32) {
            const int b = b0 + lane;
            int64_t s = 0, n = 0;
            int size = 0;
            if (b < p.seqs) {
                size = p.lens[b];
                s = p.starts[b];
                n = p.starts[b + 1] - s;
                if (s < 0 || n < 0 || s + n > p.tokens) {
                    if (report) atomicCAS(error, 0, 7000 + kErrIndex);
                    n = 0;
                }
            }
            const int64_t t = (n * p.group + tile_rows - 1) / tile_rows;
            int64_t sum = t;  // inclusive prefix over the lanes
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int64_t o = __shfl_up_sync(0xffffffffu, sum, d);
                if (lane >= d) sum += o;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, before + sum > tile);
            if (hit && f.seq < 0) {
                const int l = __ffs(hit) - 1;
                f.seq = b0 + l;
                f.begin = __shfl_sync(0xffffffffu, s, l);
                f.count = __shfl_sync(0xffffffffu, n, l);
                f.len = __shfl_sync(0xffffffffu, size, l);
                f.inner = static_cast<int>(__shfl_sync(0xffffffffu, sum, l) + before - 1 - tile);
                if (!report) break;
            }
            before += __shfl_sync(0xffffffffu, sum, 31);
        }
        if (report && before > p.row_tiles && lane == 0) atomicCAS(error, 0, 7000 + kErrIndex);
        if (f.seq < 0) return false;
    }
    if (f.len < 0 || f.len > p.table_width * p.page_size) {
        if (lane == 0) atomicCAS(error, 0, 7000 + kErrIndex);
        f.len = 0;
    }
    return true;
}

// What a row's sum of weighted values is multiplied by.  A sum of weights is 0 where
// the row saw no key, and partial ones are left out of a join for that alone: one
// that is NaN (a query or score that is not finite) has to reach the output.  A row
// that sees keys and still has 0 has scores of -inf only, whose softmax is NaN too.
__device__ __forceinline__ float weight_inverse(float sum, bool sees) {
    return sum != 0.0f ? 1.0f / sum : sees ? __int_as_float(0x7fffffff) : 0.0f;
}

// Bound on the row tiles of all sequences, from what the host knows.
inline int64_t attention_row_tiles(const AttentionArgs& a, int group, int tile_rows) {
    const int64_t most_new = a.starts ? (a.max_new > 0 ? a.max_new : a.tokens) : 1;
    const int64_t tiles = a.seqs * ((most_new * group + tile_rows - 1) / tile_rows);
    const int64_t by_tokens = a.tokens * group / tile_rows + a.seqs;
    return a.starts && by_tokens < tiles ? by_tokens : tiles;
}

// About the most positions that a row tile reads.
inline int64_t attention_longest(const AttentionArgs& a) {
    const int64_t most_new = a.starts ? (a.max_new > 0 ? a.max_new : a.tokens) : 1;
    int64_t longest = a.table_width * a.cache->page_size;
    if (a.max_len > 0 && a.max_len < longest) longest = a.max_len;
    if (a.window > 0 && a.window + most_new < longest) longest = a.window + most_new;
    return longest;
}

inline AttnParams attention_params(const AttentionArgs& a) {
    const fp8w_kv_cache& c = *a.cache;
    AttnParams p = {};
    p.q = static_cast<const uint16_t*>(a.q);
    p.out = static_cast<uint16_t*>(a.out);
    p.q_stride = a.q_stride;
    p.out_stride = a.out_stride;
    p.tokens = a.tokens;
    p.table = a.block_table;
    p.lens = a.lens;
    p.starts = a.starts;
    p.table_width = a.table_width;
    p.k = c.k;
    p.v = c.v;
    p.page_stride = c.page_stride;
    p.head_stride = c.head_stride;
    p.token_stride = c.token_stride;
    p.k_scales = c.k_scales;
    p.v_scales = c.v_scales;
    p.k_blocks = c.k_blocks;
    p.v_blocks = c.v_blocks;
    p.num_pages = c.num_pages;
    p.seqs = static_cast<int>(a.seqs);
    p.kv_heads = c.kv_heads;
    p.group = a.q_heads / c.kv_heads;
    p.group_inverse = static_cast<uint32_t>(((1ull << 32) + p.group - 1) / p.group);
    p.head_dim = c.head_dim;
    p.page_size = c.page_size;
    while ((1 << p.log_page) < c.page_size) ++p.log_page;
    p.c = a.scale * kLog2e;
    p.window = a.window;
    return p;
}

// 2^x, approximate (2 ulp), subnormal results to zero.
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// fp16 weights (with codes: weights times value scales) are taken 2^kLiftF16 times
// as large, sums of them too: with references that lag by 2^8 at most they reach
// 2^15, and what a weight loses below fp16's normal numbers is at most 2^-32 of the
// largest (2^-25 without; a long tail of small weights may be all there is, where
// the largest ones' values are zero).
constexpr float kLiftF16 = 7.0f;

// log2 of a value scale for the reference of weight times value scale, with a
// floor (scales of 0 too): the sum of the weights alone, up to this much larger,
// stays finite, and smaller values are nothing in 16 bits.
__device__ __forceinline__ float log2_scale(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return fmaxf(y, -90.0f);
}

// Two fp32 -> packed 16-bit pair (first in the low half), rounded to nearest.
template <bool kBf16>
__device__ __forceinline__ uint32_t pack16(float first, float second) {
    uint32_t r;
    if constexpr (kBf16)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(second), "f"(first));
    else
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(second), "f"(first));
    return r;
}

// Shared memory of the cluster's CTAs.
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
__device__ __forceinline__ float2 ld_cluster_f2(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}

// Few rows (launch_attention decides): attention_few.cu.
cudaError_t launch_attention_few(const AttentionArgs& a, cudaStream_t st);
int read_attention_few_device_error();

}  // namespace fp8w
