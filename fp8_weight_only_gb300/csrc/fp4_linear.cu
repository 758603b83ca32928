// fp4_linear.cu -- kernel K9: the linear layer on 4-bit weights for few tokens.
//
//   y[m, n] = round(scale[n] * sum_k x[m, k] * e4m3(block) * e2m1(code) + bias[n])
// (the form: fp4.cuh).  With few tokens the weight's bytes, 9 bits for two
// values, are what counts, so the kernel is made for bytes in flight: codes go
// from memory straight into registers, in the layout that the warp's matrix
// instruction (m16n8k16) wants its operand in, with the next steps' loads
// outstanding meanwhile.  There is no staging of the weight and no barrier but
// one a tile of 16 output channels.
//
// Operands.  A step of a warp is 16 channels x 128 inputs.  A sum over the inputs
// runs in any order, so lane (g, t) = (lane / 4, lane % 4) reads 16 contiguous
// bytes of rows g and g + 8, the codes of inputs 32 t .. 32 t + 31, and these are
// its operands of eight products: four values of each row a product, against the
// same four inputs of token g.  Codes become fp16 by one conversion for two of
// them and one multiply by their block's scale, exactly.  The activations are in
// shared memory, in the order in which the warps read them (16 bytes a lane,
// lane by lane: no conflicts).
//
// bf16 activations go over to fp16 exactly but for a power of two a token and
// CTA, which takes their largest to [2^14, 2^15): what falls below fp16's normal
// numbers then is less than 2^-28 of the largest, and off by 2^-39 of it.
//
// Split.  G of a CTA's 16 warps share a tile's inputs and add their sums in shared
// memory in the warps' order; the CTAs of a cluster share the inputs too where
// there are too few tiles for the SMs (or too many activations for shared
// memory), and add theirs in distributed shared memory in rank order.  Each CTA
// goes over its tiles with the activations in place.
#include <mutex>

#include "fp4.cuh"
#include "fp8w_internal.h"

namespace fp8w {

namespace {

constexpr int kWarps = 16, kThreads = 32 * kWarps;
constexpr int kRowsTile = 16;      // output channels a tile
constexpr int kStepK = 128;        // inputs a step
constexpr int kMaxSplit = 8;       // CTAs a cluster
constexpr uint32_t kSmemMost = 224 * 1024;
constexpr uint32_t kPartialMost = 48 * 1024;  // a CTA's sums kept for its cluster, about
constexpr int kHeld = 4;           // 16-byte pieces of activations a thread keeps between its two looks at them

struct Fp4Params {
    const uint16_t* x;
    const uint8_t* codes;
    const uint8_t* blocks;
    const float* scales;
    const float* bias;
    uint16_t* y;
    int64_t m, n, k, tiles;
    int steps;     // of all inputs
    int per_rank;  // of a rank
    int cl;        // CTAs a cluster
    int g;         // warps a tile
    int batch;     // rounds of tiles between two joins of a cluster
    int early;
};

__device__ __forceinline__ uint4 ld_once_v4(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ uint32_t ld_u16(const void* p) {
    uint16_t v;
    asm volatile("ld.global.u16 %0, [%1];" : "=h"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void sts_f1(uint32_t addr, float v) { asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory"); }
__device__ __forceinline__ float lds_f1(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void group_bar(int group, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(threads) : "memory");
}

// Shared memory of a launch, in bytes from its start.
struct Fp4Layout {
    uint32_t x, red, part, top, total;
};
__host__ __device__ inline Fp4Layout fp4_layout(int nt, int tokens, int per_rank, int batch, int j, bool cluster) {
    Fp4Layout l;
    const uint32_t rows = nt == 1 ? tokens : 8 * nt;           // tokens stored of a step
    l.x = 0;
    l.red = l.x + static_cast<uint32_t>(per_rank) * rows * (kStepK * 2);
    l.part = l.red + 2 * kWarps * static_cast<uint32_t>(tokens) * kRowsTile * 4;  // [2][warp][token][channel]
    l.top = l.part + (cluster ? static_cast<uint32_t>(batch) * j * tokens * kRowsTile * 4 : 0);
    l.total = l.top + 8 * nt * 4 * 2;                           // largest bits, factor back
    return l;
}

// One step's codes of a lane: rows g and g + 8, and their blocks' scales.
struct Fp4Step {
    uint4 c0, c1;
    uint32_t b0, b1;
};

// The sums of `count` rounds of tiles from round `first` on, over the ranks in
// order, to the output.  Every CTA of the cluster calls it with the same rounds.
template <bool kBf16>
__device__ __noinline__ void join_ranks(const Fp4Params& p, uint32_t part, int first, int count, int J, int cluster, int clusters, int rank,
                                        int64_t m0, int slab, int tokens) {
    cluster_sync_all();
    const int per_tile = slab * kRowsTile, all = count * J * per_tile;
    for (int o = rank * kThreads + static_cast<int>(threadIdx.x); o < all; o += p.cl * kThreads) {
        const int n = o / per_tile, in = o - n * per_tile, token = in / kRowsTile, i = n / J;
        const int64_t row = ((static_cast<int64_t>(first + i) * clusters + cluster) * J + (n - i * J)) * kRowsTile + (in & (kRowsTile - 1));
        if (row >= p.n || token >= tokens) continue;
        float v[kMaxSplit], sum = 0.0f;
#pragma unroll
        for (int r = 0; r < kMaxSplit; ++r) v[r] = r < p.cl ? ld_shared_cluster_f32(mapa_shared(part + static_cast<uint32_t>(o) * 4, r)) : 0.0f;
#pragma unroll
        for (int r = 0; r < kMaxSplit; ++r) sum += v[r];
        p.y[(m0 + token) * p.n + row] = round_out<kBf16>(fmaf(sum, p.scales[row], p.bias ? p.bias[row] : 0.0f));
    }
    cluster_sync_all();  // the sums have been read: they may be written over, and CTAs may leave
}

}  // namespace

// NT: 8-token tiles of a slab.
template <int NT, bool kBf16, int kDepth>
__global__ void __launch_bounds__(kThreads, 1) fp4_few_kernel(const __grid_constant__ Fp4Params p) {
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int rank = p.cl > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int cluster = static_cast<int>(blockIdx.x) / p.cl, clusters = static_cast<int>(gridDim.x) / p.cl;
    const int64_t m0 = static_cast<int64_t>(blockIdx.y) * (8 * NT);
    const int tokens = p.m - m0 < 8 * NT ? static_cast<int>(p.m - m0) : 8 * NT;
    const int G = p.g, J = kWarps / G, group = warp / G, wk = warp - group * G;
    const int64_t span = static_cast<int64_t>(clusters) * J;
    const int rounds = static_cast<int>((p.tiles + span - 1) / span);
    // sizes by a full slab, so that all slabs and ranks have the same places
    const int slab = p.m < 8 * NT ? static_cast<int>(p.m) : 8 * NT;
    const Fp4Layout L = fp4_layout(NT, slab, p.per_rank, p.batch, J, p.cl > 1);
    const int rows = NT == 1 ? slab : 8 * NT;  // token rows of a step in shared memory (a tile of 8 at a time beyond 8)
    const int step0 = rank * p.per_rank;
    const int mine = p.steps - step0 < p.per_rank ? (p.steps > step0 ? p.steps - step0 : 0) : p.per_rank;
    const int S = (mine + G - 1) / G;          // steps of a warp a tile

    pdl_launch_dependents();
    if (!p.early) pdl_wait();

    // ---------------------------------------------------------------- loads --
    const int64_t code_row = p.k >> 1, block_row = p.k >> 4;
    // tile round i of this warp's group
    auto tile_at = [&](int i) { return (static_cast<int64_t>(i) * clusters + cluster) * J + group; };
    int li = 0, ls = 0;  // the load stream: round and step in it
    const uint8_t *c_at = nullptr, *b_at = nullptr;
    int64_t c_8 = 0, b_8 = 0;  // from row g to row g + 8 (0 where that is past the last)
    bool l_live = false;
    auto open = [&] {
        const int64_t tile = tile_at(li);
        l_live = li < rounds && tile < p.tiles;
        if (!l_live) return;
        // channels past the last read the last's: their sums go nowhere
        const int64_t r0 = tile * kRowsTile + g, a = r0 < p.n ? r0 : p.n - 1, b = r0 + 8 < p.n ? r0 + 8 : p.n - 1;
        c_at = p.codes + a * code_row;
        b_at = p.blocks + a * block_row;
        c_8 = (b - a) * code_row;
        b_8 = (b - a) * block_row;
    };
    open();
    auto load = [&](Fp4Step& s) {
        const int step = wk + ls * G;
        const int64_t k0 = static_cast<int64_t>(step0 + step) * kStepK + t * 32;
        s.c0 = s.c1 = make_uint4(0u, 0u, 0u, 0u);
        s.b0 = s.b1 = 0u;
        if (l_live && step < mine && k0 < p.k) {
            s.c0 = ld_once_v4(c_at + (k0 >> 1));
            s.c1 = ld_once_v4(c_at + c_8 + (k0 >> 1));
            s.b0 = ld_u16(b_at + (k0 >> 4));
            s.b1 = ld_u16(b_at + b_8 + (k0 >> 4));
        }
        if (++ls >= S) {
            ls = 0;
            ++li;
            open();
        }
    };
    Fp4Step held[kDepth];
#pragma unroll
    for (int d = 0; d < kDepth; ++d) load(held[d]);

    // ---------------------------------------------------------- activations --
    if (p.early) pdl_wait();  // x may come from the kernel before, y may still be read by it
    {
        const int pieces = mine * (kStepK / 8), total = slab * pieces;  // 8 values each; rows past the last are zeros
        const uint16_t* x = p.x + m0 * p.k + static_cast<int64_t>(step0) * kStepK;
        const int64_t k_left = p.k - static_cast<int64_t>(step0) * kStepK;
        auto fetch = [&](int token, int piece) {
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (token < tokens && piece * 8 < k_left) v = *reinterpret_cast<const uint4*>(x + token * p.k + piece * 8);
            return v;
        };
        // piece: inputs 8 (piece % 4) .. of lane t's 32 in step piece / 16
        auto put = [&](int token, int piece, const uint4& v) {
            const int step = piece >> 4, w = piece & 3, tt = (piece >> 2) & 3;
            const int part = NT == 1 ? rows : 8, tile = NT == 1 ? 0 : token >> 3, at = NT == 1 ? token : token & 7;
            sts128(sbase + L.x + ((((step * NT + tile) * 4 + w) * part + at) * 4 + tt) * 16, v.x, v.y, v.z, v.w);
        };
        uint32_t* top = reinterpret_cast<uint32_t*>(smem + L.top);
        float* back = reinterpret_cast<float*>(smem + L.top) + 8 * NT;
        if constexpr (kBf16) {
            if (tid < 8 * NT) top[tid] = 0u;
            __syncthreads();
            uint4 kept[kHeld];
            auto look = [&](int i, const uint4& v) {
                const int token = i / pieces;
                const uint32_t u[4] = {v.x, v.y, v.z, v.w};
                uint32_t mx = 0u;
#pragma unroll
                for (int e = 0; e < 4; ++e) mx = max(mx, max(u[e] & 0x7FFFu, (u[e] >> 16) & 0x7FFFu));
                if (mx) atomicMax(top + token, mx);
            };
            int u = 0;
#pragma unroll
            for (; u < kHeld; ++u) {
                const int i = tid + u * kThreads;
                kept[u] = make_uint4(0u, 0u, 0u, 0u);
                if (i < total) kept[u] = fetch(i / pieces, i % pieces);
            }
#pragma unroll
            for (int e = 0; e < kHeld; ++e)
                if (tid + e * kThreads < total) look(tid + e * kThreads, kept[e]);
            for (int i = tid + kHeld * kThreads; i < total; i += kThreads) look(i, fetch(i / pieces, i % pieces));
            __syncthreads();
            // exponent of the factor, 14 - (e - 127), within fp32's normal numbers
            auto up_of = [&](int token) { return min(max(127 + 14 - (static_cast<int>(top[token] >> 7) - 127), 1), 253); };
            if (tid < 8 * NT) back[tid] = __int_as_float((254 - up_of(tid)) << 23);
            auto turn = [&](int i, const uint4& v) {
                const int token = i / pieces;
                const float f = __int_as_float(up_of(token) << 23);
                auto two = [&](uint32_t w) {
                    uint32_t r;
                    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(bf16_hi_to_f32(w) * f), "f"(bf16_lo_to_f32(w) * f));
                    return r;
                };
                put(token, i - token * pieces, make_uint4(two(v.x), two(v.y), two(v.z), two(v.w)));
            };
#pragma unroll
            for (int e = 0; e < kHeld; ++e)
                if (tid + e * kThreads < total) turn(tid + e * kThreads, kept[e]);
            for (int i = tid + kHeld * kThreads; i < total; i += kThreads) turn(i, fetch(i / pieces, i % pieces));
        } else {
            for (int i0 = tid; i0 < total; i0 += kHeld * kThreads) {
                uint4 kept[kHeld];
#pragma unroll
                for (int e = 0; e < kHeld; ++e) {
                    const int i = i0 + e * kThreads;
                    if (i < total) kept[e] = fetch(i / pieces, i % pieces);
                }
#pragma unroll
                for (int e = 0; e < kHeld; ++e) {
                    const int i = i0 + e * kThreads;
                    if (i < total) put(i / pieces, i % pieces, kept[e]);
                }
            }
            if (tid < 8 * NT) back[tid] = 1.0f;
        }
        if constexpr (NT > 1) {
            // the last tile's rows past the slab
            const int spare = 8 * NT - slab;
            for (int i = tid; i < spare * pieces; i += kThreads) put(slab + i / pieces, i % pieces, make_uint4(0u, 0u, 0u, 0u));
        }
    }
    __syncthreads();

    // -------------------------------------------------------------- compute --
    float acc[NT][4];
    auto clear = [&] {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[j][e] = 0.0f;
    };
    clear();
    const bool reads = NT > 1 || g < rows;
    const uint32_t x_lane = sbase + L.x + (NT == 1 ? (g * 4 + t) : lane) * 16;
    const uint32_t x_word = (NT == 1 ? rows : 8) * 64, x_step = NT * 4 * x_word;
    auto compute = [&](int step, const Fp4Step& s) {
        const uint32_t at = x_lane + static_cast<uint32_t>(step) * x_step;
        const uint32_t f0 = block_pair_f16(s.b0), f1 = block_pair_f16(s.b1);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint32_t w0 = q == 0 ? s.c0.x : q == 1 ? s.c0.y : q == 2 ? s.c0.z : s.c0.w;
            const uint32_t w1 = q == 0 ? s.c1.x : q == 1 ? s.c1.y : q == 2 ? s.c1.z : s.c1.w;
            uint32_t a[4], b[4];
            fp4_operands<false>(w0, q < 2 ? both_lo(f0) : both_hi(f0), a);
            fp4_operands<false>(w1, q < 2 ? both_lo(f1) : both_hi(f1), b);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                uint4 x = make_uint4(0u, 0u, 0u, 0u);
                if (reads) x = lds128(at + (j * 4 + q) * x_word);
                mma_f16(acc[j], a[0], b[0], a[1], b[1], x.x, x.y);
                mma_f16(acc[j], a[2], b[2], a[3], b[3], x.z, x.w);
            }
        }
    };
    // sums of a tile: [warp][token][channel]
    const int gt = G * 32, gtid = tid - group * gt;
    const float* back = reinterpret_cast<const float*>(smem + L.top) + 8 * NT;
    const int channel = gtid & (kRowsTile - 1);  // of this thread's results in every tile (gt is a multiple of 16)
    float scale = 0.0f, bias = 0.0f;
    auto ask = [&](int i) {  // ahead of their use
        const int64_t row = tile_at(i) * kRowsTile + channel;
        if (p.cl == 1 && i < rounds && row < p.n) {
            scale = p.scales[row];
            bias = p.bias ? p.bias[row] : 0.0f;
        }
    };
    ask(0);
    auto finish = [&](int i) {
        const uint32_t buf = sbase + L.red + static_cast<uint32_t>((i & 1) * kWarps * slab * kRowsTile) * 4;
        const uint32_t own = buf + static_cast<uint32_t>(warp * slab * kRowsTile) * 4;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int token = 8 * j + 2 * t + (e & 1), ch = g + 8 * (e >> 1);
                if (token < slab) sts_f1(own + (token * kRowsTile + ch) * 4, acc[j][e]);
            }
        clear();
        if (G > 1)
            group_bar(group, gt);  // groups of 1 warp have no number for one
        else
            __syncwarp();
        const int64_t row = tile_at(i) * kRowsTile + channel;
        for (int o = gtid; o < slab * kRowsTile; o += gt) {
            const int token = o / kRowsTile;
            float sum = 0.0f;
            for (int w = 0; w < G; ++w) sum += lds_f1(buf + static_cast<uint32_t>((group * G + w) * slab * kRowsTile + o) * 4);
            sum *= back[token];
            if (p.cl > 1)
                sts_f1(sbase + L.part + static_cast<uint32_t>((i % p.batch * J + group) * slab * kRowsTile + o) * 4, sum);
            else if (token < tokens && row < p.n)
                p.y[(m0 + token) * p.n + row] = round_out<kBf16>(fmaf(sum, scale, bias));
        }
        ask(i + 1);
    };
    {
        int ci = 0, cs = 0;  // the compute stream
        // with a cluster all groups go through all rounds, and join
        auto goes_on = [&](int i) { return i < rounds && (p.cl > 1 || tile_at(i) < p.tiles); };
        bool more = goes_on(0);
        while (more) {
#pragma unroll
            for (int d = 0; d < kDepth; ++d) {
                if (more) {
                    const int step = wk + cs * G;
                    const Fp4Step s = held[d];
                    load(held[d]);
                    if (step < mine) compute(step, s);
                    if (++cs >= S) {
                        finish(ci);
                        cs = 0;
                        ++ci;
                        more = goes_on(ci);
                        if (p.cl > 1 && (ci % p.batch == 0 || !more)) {
                            const int first = (ci - 1) / p.batch * p.batch;
                            join_ranks<kBf16>(p, sbase + L.part, first, ci - first, J, cluster, clusters, rank, m0, slab, tokens);
                        }
                    }
                }
            }
        }
    }
}

namespace {

template <int NT, bool kBf16>
cudaError_t launch_form(const LinearArgs& a, cudaStream_t st) {
    auto kern = fp4_few_kernel<NT, kBf16, 4>;
    static std::once_flag attr_once[64];
    static int active[64][4];  // clusters of 1, 2, 4, 8 CTAs that fit the device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    int sms = 0;
    e = device_sm_count(sms);
    if (e != cudaSuccess) return e;
    cudaError_t attr_err = cudaSuccess;
    std::call_once(attr_once[dev], [&] {
        attr_err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMost);
        active[dev][0] = sms;
        for (int i = 1; i < 4 && attr_err == cudaSuccess; ++i) {
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = 1u << i;
            attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(static_cast<unsigned>(sms >> i << i));
            cfg.blockDim = dim3(kThreads);
            cfg.dynamicSmemBytes = kSmemMost;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            attr_err = cudaOccupancyMaxActiveClusters(&active[dev][i], kern, &cfg);
        }
    });
    if (attr_err != cudaSuccess) return attr_err;

    Fp4Params p = {};
    p.x = static_cast<const uint16_t*>(a.x);
    p.codes = a.codes;
    p.blocks = a.blocks;
    p.scales = a.scales;
    p.bias = a.bias;
    p.y = static_cast<uint16_t*>(a.y);
    p.m = a.m;
    p.n = a.n;
    p.k = a.k;
    p.tiles = (a.n + kRowsTile - 1) / kRowsTile;
    p.steps = static_cast<int>((a.k + kStepK - 1) / kStepK);
    p.early = a.early ? 1 : 0;
    const int64_t slabs = (a.m + 8 * NT - 1) / (8 * NT);
    const int slab = a.m < 8 * NT ? static_cast<int>(a.m) : 8 * NT;
    // Clusters and warps a tile that leave a warp the fewest steps, where the
    // activations fit; a tile's joins count as part of a step.
    double best = 1e30;
    int64_t grid = 0;
    uint32_t smem = 0;
    for (int c = 0; c < 4; ++c) {
        const int cl = 1 << c;
        if (active[dev][c] < 1 || (cl > 1 && cl > p.steps)) continue;
        const int per_rank = (p.steps + cl - 1) / cl;
        for (int g = 1; g <= kWarps; g <<= 1) {
            const int J = kWarps / g, S = (per_rank + g - 1) / g;
            const int64_t want = (p.tiles + J - 1) / J;  // clusters of work
            int64_t clusters = active[dev][c] / slabs > 1 ? active[dev][c] / slabs : 1;
            if (clusters > want) clusters = want;
            const int64_t rounds = (want + clusters - 1) / clusters;
            if (rounds > 0x3fffffff) continue;
            int64_t batch = static_cast<int64_t>(kPartialMost) / (static_cast<int64_t>(J) * slab * kRowsTile * 4);
            batch = batch < 1 ? 1 : batch < rounds ? batch : rounds;
            const Fp4Layout l = fp4_layout(NT, slab, per_rank, static_cast<int>(batch), J, cl > 1);
            if (l.total > kSmemMost) continue;
            const double waves = static_cast<double>((slabs * clusters * cl + sms - 1) / sms);
            const double joins = cl > 1 ? 1.5 * ((rounds + batch - 1) / batch) : 0.0;
            const double cost = waves * (rounds * (S + 0.4) + joins);
            if (cost < best) {
                best = cost;
                p.cl = cl;
                p.g = g;
                p.per_rank = per_rank;
                p.batch = static_cast<int>(batch);
                grid = clusters * cl;
                smem = l.total;
            }
        }
    }
    if (grid == 0) return cudaErrorNotSupported;
    if (slabs > 65535) return cudaErrorInvalidConfiguration;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(p.cl);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), static_cast<unsigned>(slabs));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = p.cl > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

// 8, 16 or 32 tokens a slab; fewer than there are where the activations of more
// do not fit a cluster's shared memory (32: k beyond 19 thousand or so).
template <bool kBf16>
static cudaError_t launch_act(const LinearArgs& a, cudaStream_t st) {
    cudaError_t e = cudaErrorNotSupported;
    if (a.m > 16) e = launch_form<4, kBf16>(a, st);
    if (e == cudaErrorNotSupported && a.m > 8) e = launch_form<2, kBf16>(a, st);
    if (e == cudaErrorNotSupported) e = launch_form<1, kBf16>(a, st);
    return e;
}

cudaError_t launch_fp4_few(const LinearArgs& a, cudaStream_t st) {
    return a.act == FP8W_BF16 ? launch_act<true>(a, st) : launch_act<false>(a, st);
}

}  // namespace fp8w
