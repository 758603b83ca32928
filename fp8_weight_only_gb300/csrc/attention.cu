// attention.cu -- kernel K7: attention of new tokens over a paged cache, on the
// tcgen05 tensor cores.
//
//   out[t, h] = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q.k_j - m),
// in one pass over the keys: for each row the running reference m and the sum
// of the p_j stay with one thread, the output's sum in tensor memory.
//
// Rows.  The g query heads that share a key head, for all new tokens of a
// sequence, are the rows of one matrix (row = token * g + head), so a page is
// read once for all of them.  A CTA takes one key head and up to 256 rows as
// two tiles of 128, and walks the keys 128 at a time:
//   S = Q K^T  (M = 128 rows, N = 128 keys; both operands in shared memory)
//   P = exp2(S c - m c), c = scale log2(e), rounded to the operand type
//   O += P V   (A = P from tensor memory, B = V in shared memory, N = head_dim)
// Two pipes, each with its own S and O (2 x 128 + 2 x 128 columns: all of the
// tensor memory), keep the tensor cores busy while the other's softmax runs.
// With more than 128 rows the pipes take the two row tiles and share every key
// tile; with fewer, both take the same rows and the key tiles in turn, and
// their two partial results are joined at the end.
//   warps 0-3, 4-7  softmax of pipe 0, 1: one row a thread
//   warp 8          TMA producer of key and value tiles, a lane a page
//   warp 9          MMA issue; owns TMEM
//   warps 12-15     (e4m3 cache) codes -> 16-bit operand tiles
// The reference m moves only when a row's maximum has grown by more than
// 2^8 (kSlack) over it: then the row's O is rescaled, after the MMA that is
// adding to it.  p stays below 2^8, and the sums are fp32.
//
// e4m3 caches: codes convert exactly; the key scales multiply the columns of S
// and the value scales those of P, in fp32, so no scale is ever rounded.
//
// Long caches and few rows: the CTAs of a cluster take equal runs of key tiles
// and join their (m, sum, O) in distributed shared memory, in rank order.
//
// Every wait is bounded; a CTA that gives up records a code, raises its abort
// flag, lets its copies and MMAs land and frees TMEM.
#include <mutex>

#include "fp8w_device.cuh"
#include "fp8w_internal.h"

namespace fp8w {

__device__ int g_attention_error;

namespace {

constexpr int kKeys = 128;            // keys a tile
constexpr int kRows = 128;            // rows a tile (TMEM lanes)
constexpr int kMaxAttnCluster = 16;
constexpr uint32_t kAttnTmemCols = 512;
constexpr int kLoadWarp = 8, kMmaWarp = 9, kConvWarp = 12;
constexpr int kBarSoftmax = 1;        // named barrier of the eight softmax warps
constexpr float kLog2e = 1.4426950408889634f;

template <int DP, bool kFp8>
struct AttnSmem {
    static constexpr uint32_t kSubs = DP / 64;                   // 64-value sub-tiles of a row (128 bytes)
    static constexpr uint32_t kTileBytes = kKeys * DP * 2;       // a 16-bit operand tile
    static constexpr uint32_t kRawBytes = kKeys * DP;            // a tile of codes
    static constexpr int kStages = kFp8 ? (DP == 128 ? 3 : 6) : (DP == 128 ? 5 : 10);
    static constexpr int kRaw = kFp8 ? (DP == 128 ? 3 : 6) : 0;
    // Key tile m is converted once ring position 2 m - 1 - kStages is free.  With
    // 3 stages that is value tile m - 3, so the softmax is done with tile m - 3;
    // with 6 it is key tile m - 3, multiplied after value tile m - 5 was.
    static constexpr int kScaleSlots = DP == 128 ? 4 : 8;
    static constexpr uint32_t kQOff = 0;                         // two row tiles; later a 128 x DP fp32 partial
    static constexpr uint32_t kRingOff = 2 * kTileBytes;
    static constexpr uint32_t kRawOff = kRingOff + kStages * kTileBytes;
    static constexpr uint32_t kScaleOff = kRawOff + kRaw * kRawBytes;  // [slot][k, v][128] fp32
    static constexpr uint32_t kMlOff = kScaleOff + (kFp8 ? kScaleSlots * 2 * kKeys * 4 : 0);
    static constexpr uint32_t kBarOff = kMlOff + kRows * 8;
    // full, empty [kStages] | rawfull, rawempty [kRaw] | sfull, pfull, ofull [2] | qfull | joinfull, joinfree | drain
    static constexpr uint32_t kNumBars = 2 * kStages + 2 * kRaw + 6 + 1 + 2 + 1;
    static constexpr uint32_t kMiscOff = kBarOff + kNumBars * 8;
    static constexpr uint32_t kBytes = kMiscOff + 16;
    static_assert(kBytes <= 227 * 1024, "shared memory");
    static constexpr int kThreads = kFp8 ? 512 : 384;
    // registers a thread after the split; the launch has 65536 / 512 = 128 or 65536 / 384 -> 168 a thread
    static constexpr int kRegsSoftmax = kFp8 ? 184 : 216;
    static constexpr int kRegsIssue = kFp8 ? 64 : 72;
    static constexpr int kRegsConv = 80;
    static_assert(256 * kRegsSoftmax + 128 * kRegsIssue + (kFp8 ? 128 * kRegsConv : 0) <= kThreads * (kFp8 ? 128 : 168),
                  "register split");
};

struct AttnParams {
    const uint16_t* q;
    uint16_t* out;
    int64_t q_stride, out_stride, tokens;
    const int32_t* table;
    const int32_t* lens;
    const int32_t* starts;
    int64_t table_width;
    const float* k_scales;
    const float* v_scales;
    int64_t num_pages;
    int seqs, kv_heads, group, head_dim, page_size, log_page;
    float c;         // scale * log2(e)
    int64_t window;  // 0: none
    int row_tiles;   // bound on the 256-row tiles of all sequences
    int cl;
};

__device__ __forceinline__ void attn_error(int code, volatile int* abort_flag) {
    *abort_flag = 1;
    atomicCAS(&g_attention_error, 0, 7000 + code);
}

template <int N>
__device__ __forceinline__ void reg_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, int32_t z,
                                            int32_t w, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}

// 32 consecutive columns of the thread's lane, without the wait.
__device__ __forceinline__ void tmem_ld_x32(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}
// The wait, tied to the registers it makes valid.
__device__ __forceinline__ void tmem_wait_ld_x32(uint32_t* r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                   "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                   "+r"(r[30]), "+r"(r[31])::"memory");
}
__device__ __forceinline__ void tmem_st_x32(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ float lo2(uint64_t v) { return __uint_as_float(static_cast<uint32_t>(v)); }
__device__ __forceinline__ float hi2(uint64_t v) { return __uint_as_float(static_cast<uint32_t>(v >> 32)); }

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

// B operand with its N values contiguous (the value tile: rows are keys, K of
// the product): 128-byte swizzled atoms of 8 keys x 64 values, 1024 bytes
// apart along the keys (SBO) and a sub-tile apart along the values (LBO).
__device__ __forceinline__ uint64_t smem_desc_sw128_nmajor(uint32_t addr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((addr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>((kKeys * 128u) >> 4) << 16;
    d |= static_cast<uint64_t>(1024u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(2u) << 61;
    return d;
}
constexpr uint32_t kIdescBNMajor = 1u << 16;

__device__ __forceinline__ void mbar_arrive_remote(uint32_t bar, uint32_t rank) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(mapa_shared(bar, rank)) : "memory");
}
// Bounded wait with cluster scope (another CTA's writes before its arrive).
__device__ __forceinline__ bool mbar_wait_cluster(uint32_t bar, uint32_t parity, const volatile int* abort_flag) {
    const long long t0 = cycles();
    for (uint32_t i = 1;; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
        if (ok) return true;
        if ((i & 63u) == 0 && (*abort_flag || cycles() - t0 > kWaitLimitCycles)) return false;
    }
}
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
__device__ __forceinline__ void softmax_bar() { asm volatile("bar.sync %0, 256;" ::"n"(kBarSoftmax) : "memory"); }

// What a CTA works on: rows [row0, row0 + rows) of sequence seq (rows counted
// token * group + head), key tiles [t0, t0 + cnt), of which pipe 0 takes the
// first cnt0 when the pipes have a row tile each.
struct Work {
    int seq, head, row0, rows, total_rows;
    int64_t token0;  // the sequence's first new token
    int pos0;        // its position
    int end;         // positions below this are loaded
    int t0, cnt, cnt0;
    int first_key;   // no row sees positions below this
    bool two;
};

// The sequence of 256-row tile `tile` and the tile's number in it, by a scan
// of the sequences' new tokens 32 at a time.  Every warp computes it alike.
__device__ __forceinline__ bool find_work(const AttnParams& p, int tile, int head, int rank, Work& w, bool report) {
    const int lane = threadIdx.x & 31;
    int64_t begin = 0, count = 0;
    int seq = -1, inner = 0;
    if (!p.starts) {
        const int per = (p.group + 2 * kRows - 1) / (2 * kRows);
        seq = tile / per;
        inner = tile - seq * per;
        if (seq >= p.seqs) return false;
        begin = seq;
        count = 1;
    } else {
        int64_t before = 0;
        for (int b0 = 0; b0 < p.seqs; b0 += 32) {
            const int b = b0 + lane;
            int64_t s = 0, n = 0, t = 0;
            if (b < p.seqs) {
                s = __ldg(p.starts + b);
                n = __ldg(p.starts + b + 1) - s;
                if (s < 0 || n < 0 || s + n > p.tokens) {
                    if (report) atomicCAS(&g_attention_error, 0, 7000 + kErrIndex);
                    n = 0;
                }
                t = (n * p.group + 2 * kRows - 1) / (2 * kRows);
            }
            int64_t sum = t;  // inclusive prefix over the lanes
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int64_t o = __shfl_up_sync(0xffffffffu, sum, d);
                if (lane >= d) sum += o;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, before + sum > tile);
            if (hit && seq < 0) {
                const int l = __ffs(hit) - 1;
                seq = b0 + l;
                inner = static_cast<int>(tile - before - __shfl_sync(0xffffffffu, sum - t, l));
                begin = __shfl_sync(0xffffffffu, s, l);
                count = __shfl_sync(0xffffffffu, n, l);
                // later rows see more keys: they go first
                inner = static_cast<int>((count * p.group + 2 * kRows - 1) / (2 * kRows)) - 1 - inner;
                if (!report) break;
            }
            before += __shfl_sync(0xffffffffu, sum, 31);
        }
        if (report && before > p.row_tiles && lane == 0) atomicCAS(&g_attention_error, 0, 7000 + kErrIndex);
        if (seq < 0) return false;
    }
    w.seq = seq;
    w.head = head;
    w.token0 = begin;
    w.total_rows = static_cast<int>(count * p.group);
    w.row0 = inner * 2 * kRows;
    w.rows = w.total_rows - w.row0 < 2 * kRows ? w.total_rows - w.row0 : 2 * kRows;
    w.two = w.rows > kRows;
    int64_t len = __ldg(p.lens + seq);
    if (len < 0 || len > p.table_width * p.page_size) {
        if (report || (head == 0 && rank == 0 && inner == 0 && threadIdx.x == 0))
            atomicCAS(&g_attention_error, 0, 7000 + kErrIndex);
        len = 0;
    }
    w.pos0 = static_cast<int>(len - count);
    const int last = w.pos0 + (w.row0 + w.rows - 1) / p.group;    // position of the last row
    const int low = w.pos0 + w.row0 / p.group;                    // and of the first
    const int mid = w.pos0 + (w.row0 + kRows - 1) / p.group;      // and of row tile 0's last
    w.end = last + 1 > 0 ? last + 1 : 0;
    const int64_t from = p.window > 0 ? static_cast<int64_t>(low) - p.window + 1 : 0;
    w.first_key = from > 0 ? static_cast<int>(from) : 0;
    const int lo = w.first_key / kKeys, hi = (w.end + kKeys - 1) / kKeys;
    const int per = (hi - lo + p.cl - 1) / p.cl;
    w.t0 = lo + rank * per;
    w.cnt = hi - w.t0 < per ? hi - w.t0 : per;
    if (w.cnt < 0) w.cnt = 0;
    const int hi0 = mid + 1 > 0 ? (mid + 1 + kKeys - 1) / kKeys : 0;
    w.cnt0 = hi0 - w.t0 < w.cnt ? hi0 - w.t0 : w.cnt;
    if (w.cnt0 < 0) w.cnt0 = 0;
    return true;
}

}  // namespace

template <int DP, bool kBf16, bool kFp8>
__global__ void __launch_bounds__(AttnSmem<DP, kFp8>::kThreads, 1)
    attention_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                     const __grid_constant__ AttnParams p) {
    using L = AttnSmem<DP, kFp8>;
    constexpr int kStages = L::kStages, kRaw = L::kRaw;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bar0 = sbase + L::kBarOff;
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (kStages + s); };
    auto rawfull = [&](int s) { return bar0 + 8u * (2 * kStages + s); };
    auto rawempty = [&](int s) { return bar0 + 8u * (2 * kStages + kRaw + s); };
    constexpr uint32_t kB = 2 * kStages + 2 * kRaw;
    auto sfull = [&](int i) { return bar0 + 8u * (kB + i); };
    auto pfull = [&](int i) { return bar0 + 8u * (kB + 2 + i); };
    auto ofull = [&](int i) { return bar0 + 8u * (kB + 4 + i); };
    const uint32_t qfull = bar0 + 8u * (kB + 6), joinfull = bar0 + 8u * (kB + 7), joinfree = bar0 + 8u * (kB + 8),
                   drain = bar0 + 8u * (kB + 9);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMiscOff);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMiscOff + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (warp == kMmaWarp) {
        tmem_alloc(smem_u32(tmem_slot), kAttnTmemCols);
        tmem_relinquish();
    } else if (warp == kLoadWarp) {
        if (lane == 0) {
            for (int s = 0; s < kStages; ++s) {
                mbar_init(full(s), kFp8 ? 4 : 1);  // the converting warps, or the producer
                mbar_init(empty(s), 1);            // MMA commit
            }
            for (int s = 0; s < kRaw; ++s) {
                mbar_init(rawfull(s), 1);
                mbar_init(rawempty(s), 4);
            }
            for (int i = 0; i < 2; ++i) {
                mbar_init(sfull(i), 1);
                mbar_init(pfull(i), 4);  // the pipe's softmax warps
                mbar_init(ofull(i), 1);
            }
            mbar_init(qfull, 8);
            mbar_init(joinfull, static_cast<uint32_t>(p.cl));
            mbar_init(joinfree, static_cast<uint32_t>(p.cl));
            mbar_init(drain, 1);
            *abort_flag = (sbase & 1023u) ? 1 : 0;  // the swizzled tiles need this alignment
            tma_prefetch_desc(&map_k);
            tma_prefetch_desc(&map_v);
        }
        fence_mbar_init();
    }
    tc_fence_before();
    if (p.cl > 1)
        cluster_sync_all();
    else
        __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_launch_dependents();
    pdl_wait();

    const int rank = p.cl > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int item = static_cast<int>(blockIdx.x) / p.cl;
    const int tile = item / p.kv_heads, head = item - tile * p.kv_heads;
    Work w = {};
    const bool have = !*abort_flag && find_work(p, tile, head, rank, w,
                                                blockIdx.x == 0 && warp == 0);
    if (!have) w = Work{};
    const int n = w.cnt;
    // ring position of key tile j and value tile j: K0 K1 V0 K2 V1 ...
    auto kpos = [&](int j) { return j == 0 ? 0 : 2 * j - 1; };
    auto vpos = [&](int j) { return j == n - 1 ? 2 * n - 1 : 2 * j + 2; };

    if (warp >= kLoadWarp && warp < kLoadWarp + 4) {
        reg_down<L::kRegsIssue>();
        if (warp == kLoadWarp && n > 0) {
            // ------------------------------------------------- producer --
            constexpr int kR = kFp8 ? kRaw : kStages;
            const int box = p.page_size < kKeys ? p.page_size : kKeys;
            const int boxes = kKeys / box;
            const int32_t* row = p.table + static_cast<int64_t>(w.seq) * p.table_width;
            auto page_of = [&](int t) -> int {  // page of this lane's box of key tile t, or one past the cache
                const int key = t * kKeys + lane * box;
                if (lane >= boxes || key >= w.end || key + box <= w.first_key) return static_cast<int>(p.num_pages);
                const int pg = __ldg(row + (key >> p.log_page));
                if (pg < 0 || pg >= p.num_pages) {
                    atomicCAS(&g_attention_error, 0, 7000 + kErrIndex);
                    return static_cast<int>(p.num_pages);
                }
                return pg;
            };
            // boxes past the cache read as zeros
            int pk = page_of(w.t0), pv = pk, next = n > 1 ? page_of(w.t0 + 1) : 0;
            bool ok = true;
            int i = 0;
            for (; i < 2 * n; ++i) {
                const int s = i % kR;
                const bool is_k = i == 0 || (i < 2 * n - 1 && (i & 1));
                const uint32_t fullb = kFp8 ? rawfull(s) : full(s), emptyb = kFp8 ? rawempty(s) : empty(s);
                const int j = i == 0 ? 0 : is_k ? (i + 1) / 2 : i == 2 * n - 1 ? n - 1 : (i - 2) / 2;
                int pg;
                if (is_k) {
                    if (j > 0) {
                        pv = pk;
                        pk = next;
                        next = j + 1 < n ? page_of(w.t0 + j + 1) : 0;
                    }
                    pg = pk;
                } else {
                    pg = j == n - 1 ? pk : pv;
                }
                if (!mbar_wait_warp(emptyb, static_cast<uint32_t>((i / kR) & 1) ^ 1u, abort_flag)) {
                    if (lane == 0) attn_error(kErrWaitSlot, abort_flag);
                    ok = false;
                    break;
                }
                if (lane == 0) mbar_arrive_expect_tx(fullb, kFp8 ? L::kRawBytes : L::kTileBytes);
                __syncwarp();
                if (lane < boxes) {
                    const CUtensorMap* map = is_k ? &map_k : &map_v;
                    const int slot = ((w.t0 + j) * kKeys + lane * box) & (p.page_size - 1);
                    if constexpr (kFp8) {
                        tma_load_4d(sbase + L::kRawOff + s * L::kRawBytes + lane * box * DP, map, 0, slot, w.head, pg, fullb);
                    } else {
#pragma unroll
                        for (uint32_t u = 0; u < L::kSubs; ++u)
                            tma_load_4d(sbase + L::kRingOff + s * L::kTileBytes + u * (kKeys * 128) + lane * box * 128, map,
                                        static_cast<int>(u) * 64, slot, w.head, pg, fullb);
                    }
                }
                __syncwarp();
            }
            if (!ok || *abort_flag) {
                // let the copies still in flight land before the CTA exits
                for (int c = i > kR ? i - kR : 0; c < i; ++c)
                    if (!mbar_wait_drain(kFp8 ? rawfull(c % kR) : full(c % kR), static_cast<uint32_t>((c / kR) & 1)))
                        atomicCAS(&g_attention_error, 0, 7000 + kErrWaitDrain);
            }
        } else if (warp == kMmaWarp && n > 0) {
            // ------------------------------------------------ MMA issue --
            constexpr uint32_t idesc_s = idesc_f16(kBf16, kKeys);
            constexpr uint32_t idesc_o = idesc_f16(kBf16, DP) | kIdescBNMajor;
            bool ok = true;
            auto wait_full = [&](int i) {
                if (!ok) return;
                ok = mbar_wait_warp(full(i % kStages), static_cast<uint32_t>((i / kStages) & 1), abort_flag);
                if (!ok && lane == 0) attn_error(kErrWaitTma, abort_flag);
                tc_fence_after();
            };
            auto release = [&](int i) { tc_commit_warp(empty(i % kStages)); };
            auto qk = [&](int pipe, int qtile, int i) {  // S_pipe = Q_qtile K^T
                const uint32_t a = sbase + L::kQOff + qtile * L::kTileBytes;
                const uint32_t b = sbase + L::kRingOff + (i % kStages) * L::kTileBytes;
#pragma unroll
                for (int kk = 0; kk < DP / 16; ++kk)
                    mma_f16_ss_warp(tmem + pipe * kKeys, smem_desc_sw128_kmajor(a + (kk >> 2) * (kRows * 128) + (kk & 3) * 32),
                                    smem_desc_sw128_kmajor(b + (kk >> 2) * (kKeys * 128) + (kk & 3) * 32), idesc_s, kk > 0);
                tc_commit_warp(sfull(pipe));
                __syncwarp();
            };
            int pv_n[2] = {0, 0};  // products P V of each pipe
            auto pv = [&](int pipe, int i) {  // O_pipe (+)= P_pipe V
                if (!mbar_wait_warp(pfull(pipe), static_cast<uint32_t>(pv_n[pipe] & 1), abort_flag)) {
                    if (lane == 0) attn_error(kErrWaitMma, abort_flag);
                    ok = false;
                    return;
                }
                tc_fence_after();
                const uint32_t b = sbase + L::kRingOff + (i % kStages) * L::kTileBytes;
#pragma unroll
                for (int kk = 0; kk < kKeys / 16; ++kk)
                    mma_f16_ts_warp(tmem + 2 * kKeys + pipe * DP, tmem + pipe * kKeys + kk * 8,
                                    smem_desc_sw128_nmajor(b + kk * 2048), idesc_o, pv_n[pipe] > 0 || kk > 0);
                tc_commit_warp(ofull(pipe));
                __syncwarp();
                ++pv_n[pipe];
            };
            // Slots past the sequence's end hold anything, a NaN perhaps, and
            // 0 * NaN is no zero: those rows of the last value tile are cleared
            // (pages past the end were never read; codes are cleared as they convert)
            auto clear_tail = [&](int j) {
                const int keep = w.end - (w.t0 + j) * kKeys;
                if (kFp8 || keep >= kKeys) return;
                const uint32_t b = sbase + L::kRingOff + (vpos(j) % kStages) * L::kTileBytes;
                for (int u = keep * 8 + lane; u < kKeys * 8; u += 32) {
#pragma unroll
                    for (uint32_t sub = 0; sub < L::kSubs; ++sub) sts128(b + sub * (kKeys * 128) + u * 16, 0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
                __syncwarp();
            };
            ok = mbar_wait_warp(qfull, 0, abort_flag);
            if (!ok && lane == 0) attn_error(kErrWaitDequant, abort_flag);
            tc_fence_after();
            if (w.two) {
                wait_full(kpos(0));
                if (ok) {
                    if (w.cnt0 > 0) qk(0, 0, kpos(0));
                    qk(1, 1, kpos(0));
                    release(kpos(0));
                }
                for (int j = 0; j < n && ok; ++j) {
                    wait_full(vpos(j));
                    if (!ok) break;
                    clear_tail(j);
                    if (j < w.cnt0) {
                        pv(0, vpos(j));
                        if (!ok) break;
                    }
                    if (j + 1 < n) wait_full(kpos(j + 1));
                    if (!ok) break;
                    if (j + 1 < w.cnt0) qk(0, 0, kpos(j + 1));
                    pv(1, vpos(j));
                    if (!ok) break;
                    release(vpos(j));
                    if (j + 1 < n) {
                        qk(1, 1, kpos(j + 1));
                        release(kpos(j + 1));
                    }
                }
            } else {
                for (int j = 0; j < 2 && j < n; ++j) {
                    wait_full(kpos(j));
                    if (!ok) break;
                    qk(j, 0, kpos(j));
                    release(kpos(j));
                }
                for (int j = 0; j < n && ok; ++j) {
                    wait_full(vpos(j));
                    if (!ok) break;
                    clear_tail(j);
                    pv(j & 1, vpos(j));
                    if (!ok) break;
                    release(vpos(j));
                    if (j + 2 < n) {
                        wait_full(kpos(j + 2));
                        if (!ok) break;
                        qk(j & 1, 0, kpos(j + 2));
                        release(kpos(j + 2));
                    }
                }
            }
            // every MMA issued above completes before TMEM is released
            tc_commit_warp(drain);
            if (!mbar_wait_drain(drain, 0) && lane == 0) atomicCAS(&g_attention_error, 0, 7000 + kErrWaitDrain);
            __syncwarp();
        }
    } else if (kFp8 && warp >= kConvWarp) {
        // --------------------------------------- codes to operand tiles --
        if constexpr (kFp8) {
            reg_down<L::kRegsConv>();
            const int r = (warp & 3) * 32 + lane;  // key of the tile
            const uint32_t swz = static_cast<uint32_t>(r & 7);
            const int32_t* row = p.table + static_cast<int64_t>(w.seq) * p.table_width;
            for (int i = 0; i < 2 * n; ++i) {
                const bool is_k = i == 0 || (i < 2 * n - 1 && (i & 1));
                const int j = i == 0 ? 0 : is_k ? (i + 1) / 2 : i == 2 * n - 1 ? n - 1 : (i - 2) / 2;
                const int key = (w.t0 + j) * kKeys + r;
                const bool live = key < w.end && key >= w.first_key;
                // the softmax needs both scales of a tile as soon as its scores are there
                float scale_k = 0.0f, scale_v = 0.0f;
                if (live && is_k) {
                    const int64_t pg = __ldg(row + (key >> p.log_page));
                    if (pg >= 0 && pg < p.num_pages) {
                        const int64_t at = (pg * p.kv_heads + w.head) * p.page_size + (key & (p.page_size - 1));
                        scale_k = __ldg(p.k_scales + at);
                        scale_v = __ldg(p.v_scales + at);
                    }
                }
                const int s = i % kRaw, d = i % kStages;
                if (!mbar_wait_warp(rawfull(s), static_cast<uint32_t>((i / kRaw) & 1), abort_flag)) {
                    if (lane == 0) attn_error(kErrWaitTma, abort_flag);
                    break;
                }
                uint4 c[DP / 16];
                const uint32_t src = sbase + L::kRawOff + s * L::kRawBytes + static_cast<uint32_t>(r) * DP;
#pragma unroll
                for (uint32_t u = 0; u < DP / 16; ++u) {
                    const uint32_t at = DP == 128 ? u ^ swz : u ^ (swz >> 1);  // 128- or 64-byte swizzle
                    c[u] = lds128(src + (at << 4));
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(rawempty(s));
                if (!mbar_wait_warp(empty(d), static_cast<uint32_t>((i / kStages) & 1) ^ 1u, abort_flag)) {
                    if (lane == 0) attn_error(kErrWaitMma, abort_flag);
                    break;
                }
                const uint32_t dst = sbase + L::kRingOff + d * L::kTileBytes + static_cast<uint32_t>(r) * 128u;
#pragma unroll
                for (uint32_t u = 0; u < DP / 16; ++u) {
                    const uint32_t w4[4] = {live ? c[u].x : 0u, live ? c[u].y : 0u, live ? c[u].z : 0u, live ? c[u].w : 0u};
                    uint32_t v[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if constexpr (kBf16)
                            e4m3x4_to_bf16x2(w4[e], v[2 * e], v[2 * e + 1]);
                        else
                            e4m3x4_to_f16x2(w4[e], v[2 * e], v[2 * e + 1]);
                    }
                    // 16 values: 16-byte chunks 2u and 2u + 1 of the row
                    const uint32_t sub = dst + (u >> 2) * (kKeys * 128);
                    sts128(sub + (((2 * u) & 7) ^ swz) * 16, v[0], v[1], v[2], v[3]);
                    sts128(sub + (((2 * u + 1) & 7) ^ swz) * 16, v[4], v[5], v[6], v[7]);
                }
                if (is_k) {
                    float* sc = reinterpret_cast<float*>(smem + L::kScaleOff) + (j % L::kScaleSlots) * 2 * kKeys + r;
                    sc[0] = scale_k;
                    sc[kKeys] = scale_v;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(full(d));
            }
        }
    } else {
        // ------------------------------------------------------ softmax --
        reg_up<L::kRegsSoftmax>();
        const int pipe = warp >> 2, quarter = warp & 3;
        const int tid = threadIdx.x;                    // 0..255
        const int r = quarter * 32 + lane;              // row of the tile == TMEM lane
        const int qtile = w.two ? pipe : 0;
        // Q rows: the two tiles, 16 bytes a step
        if (n > 0) {
            const int chunks = DP / 8;
            for (int u = tid; u < w.rows * chunks; u += 256) {
                const int rr = u / chunks, ch = u - rr * chunks;
                const int R = w.row0 + rr, t = R / p.group, g = R - t * p.group;
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                if (ch * 8 < p.head_dim)
                    v = *reinterpret_cast<const uint4*>(p.q + (w.token0 + t) * p.q_stride +
                                                        static_cast<int64_t>(w.head * p.group + g) * p.head_dim + ch * 8);
                const uint32_t a = sbase + L::kQOff + (rr >> 7) * L::kTileBytes + (ch >> 3) * (kRows * 128) +
                                   (rr & 127) * 128 + (((ch & 7) ^ (rr & 7)) << 4);
                sts128(a, v.x, v.y, v.z, v.w);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(qfull);
        }
        const int R = w.row0 + qtile * kRows + r;
        const bool valid = qtile * kRows + r < w.rows;
        const int pos = w.pos0 + R / p.group;
        const int hi = valid ? pos : -1;                                     // last position seen
        const int64_t from = p.window > 0 ? static_cast<int64_t>(pos) - p.window + 1 : 0;
        const int lo = from > 0 ? static_cast<int>(from) : 0;                // first
        const bool busy = __any_sync(0xffffffffu, valid);
        const int warp_hi = __reduce_min_sync(0xffffffffu, valid ? hi : 0x7fffffff);
        const int warp_lo = __reduce_max_sync(0xffffffffu, valid ? lo : 0);
        const uint32_t tq = static_cast<uint32_t>(quarter * 32) << 16;
        const uint32_t t_s = tmem + tq + pipe * kKeys, t_o = tmem + tq + 2 * kKeys + pipe * DP;
        // fp16 weights with e4m3 scales: p * v_scale * 2^8 keeps the products of
        // small scales among fp16's normal numbers, and cannot overflow with p <= 1
        // (scales reach 65504 / 448 = 146.2 for fp16 values): no slack there
        constexpr bool kScaledF16 = kFp8 && !kBf16;
        constexpr float kSlack = kScaledF16 ? 0.0f : 8.0f;
        constexpr float kPScale = kScaledF16 ? 256.0f : 1.0f;
        const float c = p.c;
        const uint64_t c2 = pack2(c, c);
        float m = __int_as_float(0xff800000), l = 0.0f;
        const int step = w.two ? 1 : 2, j0 = w.two ? 0 : pipe, jn = w.two && pipe == 0 ? w.cnt0 : n;
        int done = 0;  // tiles of this pipe
        bool ok = true;
        for (int j = j0; j < jn; j += step, ++done) {
            if (!mbar_wait_warp(sfull(pipe), static_cast<uint32_t>(done & 1), abort_flag)) {
                if (lane == 0) attn_error(kErrWaitMma, abort_flag);
                ok = false;
                break;
            }
            tc_fence_after();
            if (busy) {
                const int key0 = (w.t0 + j) * kKeys;
                uint32_t s[128];
#pragma unroll
                for (int b = 0; b < 4; ++b) tmem_ld_x32(t_s + 32 * b, s + 32 * b);
#pragma unroll
                for (int b = 0; b < 4; ++b) tmem_wait_ld_x32(s + 32 * b);
                const float* ksc = reinterpret_cast<const float*>(smem + L::kScaleOff) + (j % L::kScaleSlots) * 2 * kKeys;
                if constexpr (kFp8) {
#pragma unroll
                    for (int i = 0; i < 128; i += 4) {
                        const float4 f = *reinterpret_cast<const float4*>(ksc + i);
                        const uint64_t a = mul2(pack2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), pack2(f.x, f.y));
                        const uint64_t b = mul2(pack2(__uint_as_float(s[i + 2]), __uint_as_float(s[i + 3])), pack2(f.z, f.w));
                        s[i] = static_cast<uint32_t>(a), s[i + 1] = static_cast<uint32_t>(a >> 32);
                        s[i + 2] = static_cast<uint32_t>(b), s[i + 3] = static_cast<uint32_t>(b >> 32);
                    }
                }
                if (key0 + kKeys - 1 > warp_hi || key0 < warp_lo) {
                    const int top = hi - key0, bot = lo - key0;
#pragma unroll
                    for (int i = 0; i < 128; ++i)
                        if (i > top || i < bot) s[i] = 0xff800000u;
                }
                float mx = __uint_as_float(s[0]), my = __uint_as_float(s[1]);
#pragma unroll
                for (int i = 2; i < 126; i += 4) {
                    mx = max3(mx, __uint_as_float(s[i]), __uint_as_float(s[i + 1]));
                    my = max3(my, __uint_as_float(s[i + 2]), __uint_as_float(s[i + 3]));
                }
                mx = max3(mx, __uint_as_float(s[126]), __uint_as_float(s[127]));
                mx = fmaxf(mx, my);
                if (done == 0) {
                    m = mx;
                } else {
                    const bool grow = valid && (mx - m) * c > kSlack;  // -inf - -inf: no
                    if (__any_sync(0xffffffffu, grow)) {
                        float alpha = 1.0f;
                        if (grow) {
                            alpha = ex2((m - mx) * c);  // 0 while nothing was seen
                            m = mx;
                            l *= alpha;
                        }
                        // O is at rest once the last product has been added
                        if (!mbar_wait_warp(ofull(pipe), static_cast<uint32_t>((done - 1) & 1), abort_flag)) {
                            if (lane == 0) attn_error(kErrWaitMma, abort_flag);
                            ok = false;
                            break;
                        }
                        tc_fence_after();
#pragma unroll
                        for (int b = 0; b < DP; b += 32) {
                            uint32_t o[32];
                            tmem_ld_x32(t_o + b, o);
                            tmem_wait_ld_x32(o);
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                            tmem_st_x32(t_o + b, o);
                        }
                    }
                }
                const float mc = m == __int_as_float(0xff800000) ? 0.0f : -m * c;
                const uint64_t mc2 = pack2(mc, mc);
                uint64_t l0 = 0ull, l1 = 0ull;
                uint32_t o[32];
#pragma unroll
                for (int b = 0; b < 2; ++b) {
#pragma unroll
                    for (int i = 0; i < 64; i += 4) {
                        const int at = b * 64 + i;
                        const uint64_t x = fma2(pack2(__uint_as_float(s[at]), __uint_as_float(s[at + 1])), c2, mc2);
                        const uint64_t y = fma2(pack2(__uint_as_float(s[at + 2]), __uint_as_float(s[at + 3])), c2, mc2);
                        uint64_t e = pack2(ex2(lo2(x)), ex2(hi2(x))), f = pack2(ex2(lo2(y)), ex2(hi2(y)));
                        l0 = add2(l0, e);
                        l1 = add2(l1, f);
                        if constexpr (kFp8) {
                            const float4 v = *reinterpret_cast<const float4*>(ksc + kKeys + at);
                            e = mul2(e, pack2(v.x * kPScale, v.y * kPScale));
                            f = mul2(f, pack2(v.z * kPScale, v.w * kPScale));
                        }
                        o[i / 2] = pack16<kBf16>(lo2(e), hi2(e));
                        o[i / 2 + 1] = pack16<kBf16>(lo2(f), hi2(f));
                    }
                    tmem_st_x32(t_s + b * 32, o);
                }
                l0 = add2(l0, l1);
                l += lo2(l0) + hi2(l0);
                tmem_wait_st();
                tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(pfull(pipe));
        }
        // --------------------------------------------------- the result --
        if (ok && done > 0) {
            ok = mbar_wait_warp(ofull(pipe), static_cast<uint32_t>((done - 1) & 1), abort_flag);
            if (!ok && lane == 0) attn_error(kErrWaitMma, abort_flag);
            tc_fence_after();
        }
        constexpr float kUnscale = 1.0f / kPScale;
        float* stage = reinterpret_cast<float*>(smem + L::kQOff);  // [128][DP], 16-byte chunks swizzled by the row
        float2* ml = reinterpret_cast<float2*>(smem + L::kMlOff);
        auto stage_at = [&](int row, int chunk) { return stage + row * DP + ((chunk ^ (row & 7)) << 2); };
        auto write_row = [&](int b, const uint32_t* o, float inv) {  // 32 values from column b of this thread's row
            const int t = R / p.group, g = R - t * p.group;
            uint16_t* dst = p.out + (w.token0 + t) * p.out_stride + static_cast<int64_t>(w.head * p.group + g) * p.head_dim;
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
                if (b + i >= p.head_dim) break;
                uint32_t v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[e] = pack16<kBf16>(__uint_as_float(o[i + 2 * e]) * inv, __uint_as_float(o[i + 2 * e + 1]) * inv);
                *reinterpret_cast<uint4*>(dst + b + i) = make_uint4(v[0], v[1], v[2], v[3]);
            }
        };
        if (w.two && p.cl == 1) {
            if (ok && busy) {
                const float inv = l > 0.0f ? kUnscale / l : 0.0f;
#pragma unroll
                for (int b = 0; b < DP; b += 32) {
                    uint32_t o[32];
                    if (done > 0) {
                        tmem_ld_x32(t_o + b, o);
                        tmem_wait_ld_x32(o);
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = 0u;
                    }
                    if (valid) write_row(b, o, inv);
                }
            }
        } else if (have) {
            // Partial results through shared memory: the pipes' of this CTA, then
            // the cluster's.  Rounds: one, or one for each row tile.
            const int rounds = w.two ? 2 : 1;
            softmax_bar();  // both pipes' products are complete: Q's place is free
            for (int round = 0; round < rounds; ++round) {
                const int rows = w.two ? (round == 0 ? kRows : w.rows - kRows) : w.rows;
                if (round > 0) {
                    ok = ok && mbar_wait_cluster(joinfree, static_cast<uint32_t>((round - 1) & 1), abort_flag);
                    ok = __all_sync(0xffffffffu, ok);
                }
                if (w.two ? pipe == round : pipe == 1) {
                    if (valid) ml[r] = make_float2(m, done > 0 ? l : 0.0f);
                    if (ok && busy && done > 0) {
#pragma unroll
                        for (int b = 0; b < DP; b += 32) {
                            uint32_t o[32];
                            tmem_ld_x32(t_o + b, o);
                            tmem_wait_ld_x32(o);
                            if (valid)
#pragma unroll
                                for (int i = 0; i < 32; i += 4)
                                    *reinterpret_cast<uint4*>(stage_at(r, (b + i) / 4)) = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                        }
                    }
                }
                softmax_bar();
                if (!w.two && pipe == 0 && ok && busy) {
                    // add pipe 1's partial to this one's
                    float2 other = valid ? ml[r] : make_float2(0.0f, 0.0f);
                    const float mine_l = done > 0 ? l : 0.0f;
                    const float top = fmaxf(mine_l > 0.0f ? m : other.x, other.y > 0.0f ? other.x : m);
                    const float a0 = mine_l > 0.0f ? ex2((m - top) * c) : 0.0f;
                    const float a1 = other.y > 0.0f ? ex2((other.x - top) * c) : 0.0f;
                    const float sum = a0 * mine_l + a1 * other.y;
                    const float inv = sum > 0.0f ? kUnscale / sum : 0.0f;
#pragma unroll
                    for (int b = 0; b < DP; b += 32) {
                        uint32_t o[32];
                        if (done > 0) {
                            tmem_ld_x32(t_o + b, o);
                            tmem_wait_ld_x32(o);
                        }
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                            if (valid && a1 > 0.0f) v = *reinterpret_cast<const float4*>(stage_at(r, (b + i) / 4));
                            const float x[4] = {v.x * a1, v.y * a1, v.z * a1, v.w * a1};
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                o[i + e] = __float_as_uint(a0 > 0.0f ? fmaf(__uint_as_float(o[i + e]), a0, x[e]) : x[e]);
                        }
                        if (valid) {
                            if (p.cl == 1) {
                                write_row(b, o, inv);
                            } else {
#pragma unroll
                                for (int i = 0; i < 32; i += 4)
                                    *reinterpret_cast<uint4*>(stage_at(r, (b + i) / 4)) = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                            }
                        }
                    }
                    if (valid && p.cl > 1) ml[r] = make_float2(top, sum);
                }
                if (p.cl == 1) break;
                softmax_bar();
                if (tid < p.cl) mbar_arrive_remote(joinfull, static_cast<uint32_t>(tid));
                __syncwarp();
                bool all = mbar_wait_cluster(joinfull, static_cast<uint32_t>(round & 1), abort_flag);
                all = __all_sync(0xffffffffu, all);
                if (!all && lane == 0) attn_error(kErrWaitDequant, abort_flag);
                if (all) {
                    // each rank finishes its share of the rows' 16-byte chunks
                    const int units = rows * (DP / 4);
                    for (int u = rank * 256 + tid; u < units; u += p.cl * 256) {
                        const int row = u / (DP / 4), ch = u - row * (DP / 4);
                        const uint32_t ml_at = sbase + L::kMlOff + row * 8;
                        const uint32_t st_at = smem_u32(stage_at(row, ch));
                        float top = __int_as_float(0xff800000), sum = 0.0f;
                        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        for (int k = 0; k < p.cl; ++k) {
                            const float2 q = ld_cluster_f2(mapa_shared(ml_at, static_cast<uint32_t>(k)));
                            if (!(q.y > 0.0f)) continue;
                            const float4 v = ld_cluster_f4(mapa_shared(st_at, static_cast<uint32_t>(k)));
                            const float to = fmaxf(top, q.x);
                            const float a = ex2((top - to) * c), b = ex2((q.x - to) * c);
                            top = to;
                            sum = sum * a + q.y * b;
                            acc.x = acc.x * a + v.x * b;
                            acc.y = acc.y * a + v.y * b;
                            acc.z = acc.z * a + v.z * b;
                            acc.w = acc.w * a + v.w * b;
                        }
                        const float inv = sum > 0.0f ? kUnscale / sum : 0.0f;
                        if (ch * 4 < p.head_dim) {
                            const int RR = w.row0 + round * kRows + row, t = RR / p.group, g = RR - t * p.group;
                            uint16_t* dst = p.out + (w.token0 + t) * p.out_stride +
                                            static_cast<int64_t>(w.head * p.group + g) * p.head_dim + ch * 4;
                            *reinterpret_cast<uint2*>(dst) =
                                make_uint2(pack16<kBf16>(acc.x * inv, acc.y * inv), pack16<kBf16>(acc.z * inv, acc.w * inv));
                        }
                    }
                }
                softmax_bar();
                if (tid < p.cl) mbar_arrive_remote(joinfree, static_cast<uint32_t>(tid));
                __syncwarp();
            }
        }
    }

    // no CTA leaves while another may read its shared memory
    tc_fence_before();
    if (p.cl > 1)
        cluster_sync_all();
    else
        __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, kAttnTmemCols);
    }
}

namespace {

template <int DP, bool kBf16, bool kFp8>
cudaError_t launch_attn(const AttentionArgs& a, cudaStream_t st) {
    using L = AttnSmem<DP, kFp8>;
    auto kern = attention_kernel<DP, kBf16, kFp8>;
    static std::once_flag attr_once[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    int sms = 0;
    e = device_sm_count(sms);
    if (e != cudaSuccess) return e;
    cudaError_t attr_err = cudaSuccess;
    std::call_once(attr_once[dev], [&] {
        attr_err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes);
        if (attr_err == cudaSuccess)
            attr_err = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    });
    if (attr_err != cudaSuccess) return attr_err;

    const fp8w_kv_cache& c = *a.cache;
    const int group = a.q_heads / c.kv_heads;
    const uint64_t es = kFp8 ? 1 : 2;
    CUtensorMap map_k, map_v;
    const uint32_t box = static_cast<uint32_t>(c.page_size < kKeys ? c.page_size : kKeys);
    for (int i = 0; i < 2; ++i)
        if (!encode_pages(i ? &map_v : &map_k, kFp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16,
                          i ? c.v : c.k, static_cast<uint64_t>(c.head_dim), static_cast<uint64_t>(c.page_size),
                          static_cast<uint64_t>(c.kv_heads), static_cast<uint64_t>(c.num_pages),
                          static_cast<uint64_t>(c.token_stride) * es, static_cast<uint64_t>(c.head_stride) * es,
                          static_cast<uint64_t>(c.page_stride) * es, kFp8 ? DP : 64, box, kFp8 && DP == 64))
            return cudaErrorInvalidValue;

    // 256-row tiles of all sequences, at most
    const int64_t most_new = a.max_new > 0 && a.starts ? a.max_new : a.starts ? a.tokens : 1;
    int64_t tiles = a.seqs * ((most_new * group + 2 * kRows - 1) / (2 * kRows));
    if (a.starts) {
        const int64_t by_tokens = a.tokens * group / (2 * kRows) + a.seqs;
        tiles = tiles < by_tokens ? tiles : by_tokens;
    }
    const int64_t items = tiles * c.kv_heads;
    // CTAs a cluster: as many as fill the GPU, while each has two key tiles at least
    int64_t longest = a.table_width * c.page_size;
    if (a.max_len > 0 && a.max_len < longest) longest = a.max_len;
    if (a.window > 0 && a.window + most_new < longest) longest = a.window + most_new;
    const int64_t key_tiles = (longest + kKeys - 1) / kKeys;
    int cl = 1;
    while (cl < kMaxAttnCluster && items * cl * 2 <= sms && key_tiles >= cl * 4) cl *= 2;
    if (items * cl > 0x7fffffffll) return cudaErrorInvalidConfiguration;

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
    p.k_scales = c.k_scales;
    p.v_scales = c.v_scales;
    p.num_pages = c.num_pages;
    p.seqs = static_cast<int>(a.seqs);
    p.kv_heads = c.kv_heads;
    p.group = group;
    p.head_dim = c.head_dim;
    p.page_size = c.page_size;
    while ((1 << p.log_page) < c.page_size) ++p.log_page;
    p.c = a.scale * kLog2e;
    p.window = a.window;
    p.row_tiles = static_cast<int>(tiles);
    p.cl = cl;

    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cl);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(items * cl));
    cfg.blockDim = dim3(L::kThreads);
    cfg.dynamicSmemBytes = L::kBytes;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = cl > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, map_k, map_v, p);
}

template <int DP>
cudaError_t launch_dim(const AttentionArgs& a, cudaStream_t st) {
    const bool bf16 = a.act == FP8W_BF16;
    if (a.cache->dtype == FP8W_E4M3)
        return bf16 ? launch_attn<DP, true, true>(a, st) : launch_attn<DP, false, true>(a, st);
    return bf16 ? launch_attn<DP, true, false>(a, st) : launch_attn<DP, false, false>(a, st);
}

}  // namespace

cudaError_t launch_attention(const AttentionArgs& a, cudaStream_t st) {
    return a.cache->head_dim <= 64 ? launch_dim<64>(a, st) : launch_dim<128>(a, st);
}

int read_attention_device_error() {
    int v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_attention_error, sizeof v) != cudaSuccess) return -1;
    if (v != 0 && cudaMemcpyToSymbol(g_attention_error, &zero, sizeof zero) != cudaSuccess) return -1;
    return v;
}

}  // namespace fp8w
