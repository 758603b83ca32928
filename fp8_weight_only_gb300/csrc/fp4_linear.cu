// fp4_linear.cu -- kernel K9: the linear layer on 4-bit weights for up to 8 tokens.
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
// Split.  G of a CTA's 24 warps share a tile's inputs and add their sums in shared
// memory in the warps' order; the CTAs of a cluster share the inputs too where
// there are too few tiles for the SMs (or too many activations for shared
// memory), and add theirs in distributed shared memory in rank order.  Each CTA
// goes over its tiles with the activations in place.  The launch takes the split of
// which a model of the steps, the staging and the joins promises the least time.
//
// Measured (bf16, weights not in L2: 420 MB of them in turn): 14336 x 4096, 33 MB, 1
// token 10.5 us, 9.5 with the weights ready (47 and 51% of the measured copy rate; e4m3
// codes, 59 MB, take 12.9 and 12.0); 8 tokens 13.2; 4096 x 14336 12.3 and 15.8; 1024 x
// 4096 4.2 and 6.7.  A launch's start and end are 3 us of it.  The rest is latency: 0.47
// instructions issued a cycle and scheduler, no pipe above 34%, and the largest stall by
// far is for loads (two steps in flight a warp, 24 warps an SM, and not all of the time:
// set-up adds half again to the 105 instructions of a step).  Fewer instructions
// shortened it all the same (divisions on the device, a zeroing before each load and
// loads under a test each: 256 a step and 14.8 us; 32 warps of 64 registers spilled:
// 19.9).  Tiles of 16, 24 and 32 tokens in the same way took 17.4, 22 and 32 us where the
// skinny kernel takes 15.5 to 16.6 (both with 132 MB of weights in turn): the products
// (10 cycles each on a scheduler) and the staging.
#include "fp4.cuh"
#include "fp8w_internal.h"

namespace fp8w {

namespace {

constexpr int kTokens = 8;         // columns of a product: the most tokens of a CTA
constexpr int kWarps = 24, kThreads = 32 * kWarps;  // of a CTA (one an SM)
constexpr int kDepth = 2;          // steps of codes that a warp holds or awaits
constexpr int kRowsTile = 16;      // output channels a tile
constexpr int kPitch = 20;         // of a token's sums of a tile in shared memory (words): no two lanes of a store share a bank
constexpr int kStepK = 128;        // inputs a step
constexpr int kMaxSplit = 8;       // CTAs a cluster
constexpr uint32_t kSmemMost = 224 * 1024;
constexpr int kHeld = 4;           // 16-byte pieces of activations that a thread has in flight (bf16: and keeps between its two looks at them)

struct Fp4Params {
    const uint16_t* x;
    const uint8_t* codes;
    const uint8_t* blocks;
    const float* scales;
    const float* bias;
    uint16_t* y;
    int64_t m, n, k;
    int slab;      // tokens of a CTA, at most
    int tiles;     // of 16 channels
    int rounds;    // of tiles, of each cluster
    int steps;     // of all inputs
    int per_rank;  // of a rank, at most (rank r: from r steps / cl on)
    int cl, cl_log2;         // CTAs a cluster
    int g, j;      // warps a tile, tiles at a time
    uint32_t piece_inverse, tile_inverse, g_inverse, j_inverse;  // 2^32 / (16 per_rank), / results a tile, / g, / j, rounded up
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

// x / d by d's rounded-up reciprocal: exact for x d < 2^32 (0 stands for 2^32, d = 1).
__device__ __forceinline__ int divide(int x, uint32_t inverse) {
    return inverse ? static_cast<int>(__umulhi(static_cast<uint32_t>(x), inverse)) : x;
}
__host__ inline uint32_t inverse_of(int64_t d) { return static_cast<uint32_t>(((1ull << 32) + d - 1) / d); }

// Shared memory of a launch, in bytes from its start.
struct Fp4Layout {
    uint32_t x, red, part, top, total;
};
__host__ __device__ inline Fp4Layout fp4_layout(int tokens, int per_rank, int rounds, int j, bool cluster) {
    Fp4Layout l;
    l.x = 0;
    l.red = l.x + static_cast<uint32_t>(per_rank) * tokens * (kStepK * 2);
    l.part = l.red + 2 * kWarps * static_cast<uint32_t>(tokens) * kPitch * 4;  // [2][warp][token][channel]
    l.top = l.part + (cluster ? static_cast<uint32_t>(rounds) * j * tokens * kRowsTile * 4 : 0);
    l.total = l.top + kTokens * 4 * 2;                           // largest bits, factor back
    return l;
}

// One step's codes of a lane: rows g and g + 8, and their blocks' scales.
struct Fp4Step {
    uint4 c0, c1;
    uint32_t b0, b1;
};

}  // namespace

template <bool kBf16>
__global__ void __launch_bounds__(kThreads, 1) fp4_few_kernel(const __grid_constant__ Fp4Params p) {
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int rank = p.cl > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int cluster = static_cast<int>(blockIdx.x) >> p.cl_log2, clusters = static_cast<int>(gridDim.x) >> p.cl_log2;
    const int64_t m0 = static_cast<int64_t>(blockIdx.y) * p.slab;
    const int tokens = p.m - m0 < p.slab ? static_cast<int>(p.m - m0) : p.slab;
    const int G = p.g, J = p.j, group = divide(warp, p.g_inverse), wk = warp - group * G, rounds = p.rounds;
    // places by a full slab, the same for all slabs and ranks
    const int slab = p.slab;
    const Fp4Layout L = fp4_layout(slab, p.per_rank, rounds, J, p.cl > 1);
    const int step0 = rank * p.steps >> p.cl_log2, mine = ((rank + 1) * p.steps >> p.cl_log2) - step0;
    const int S = divide(mine - wk + G - 1, p.g_inverse);  // this warp's steps of a tile: 1 at least (the launch sees to it)

    pdl_launch_dependents();
    if (!p.early) pdl_wait();

    // ---------------------------------------------------------------- loads --
    // tile of this warp's group in round i
    auto tile_at = [&](int i) { return (i * clusters + cluster) * J + group; };
    // Rounds of this group.  With a cluster all groups go through all rounds, for they
    // join, and one without a tile takes the last again, for nothing.
    const int my_rounds = p.cl > 1 || tile_at(rounds - 1) < p.tiles ? rounds : rounds - 1;
    // A lane's bytes of codes in a row: from here on, G steps apart, and none past the
    // row's last (there it takes the last again: the activations are zeros).
    const int o_first = (step0 + wk) * (kStepK / 2) + t * 16, o_last = static_cast<int>(p.k >> 1) - 16, o_step = G * (kStepK / 2);
    int li = 0, ls = S, lo = o_first;  // the load stream: round, steps to come of it, offset
    const uint8_t *c0, *c1, *b0, *b1;  // rows g and g + 8 of its tile
    auto open = [&] {
        // channels past the last read the last's: their sums go nowhere
        const int64_t r0 = static_cast<int64_t>(min(tile_at(li), p.tiles - 1)) * kRowsTile + g;
        const int64_t a = r0 < p.n ? r0 : p.n - 1, b = r0 + 8 < p.n ? r0 + 8 : p.n - 1;
        c0 = p.codes + a * (p.k >> 1);
        c1 = p.codes + b * (p.k >> 1);
        b0 = p.blocks + a * (p.k >> 4);
        b1 = p.blocks + b * (p.k >> 4);
    };
    open();
    auto load = [&](Fp4Step& s) {
        if (li >= my_rounds) return;
        const uint32_t o = static_cast<uint32_t>(min(lo, o_last));
        s.c0 = ld_once_v4(c0 + o);
        s.c1 = ld_once_v4(c1 + o);
        s.b0 = ld_u16(b0 + (o >> 3));
        s.b1 = ld_u16(b1 + (o >> 3));
        lo += o_step;
        if (--ls == 0) {
            ls = S;
            lo = o_first;
            ++li;
            open();
        }
    };
    Fp4Step held[kDepth];
#pragma unroll
    for (int d = 0; d < kDepth; ++d) load(held[d]);

    // ---------------------------------------------------------- activations --
    if (p.early) pdl_wait();  // x may come from the kernel before, y may still be read by it
    uint32_t* top = reinterpret_cast<uint32_t*>(smem + L.top);
    float* back = reinterpret_cast<float*>(smem + L.top) + kTokens;
    {
        // pieces of 8 values, a rank's share of each token; beyond the inputs and the
        // tokens they are zeros
        const int pieces = p.per_rank * (kStepK / 8), total = slab * pieces;
        const uint16_t* x = p.x + m0 * p.k + static_cast<int64_t>(step0) * kStepK;
        const int inputs = static_cast<int>(p.k) - step0 * kStepK;
        auto token_of = [&](int i) { return divide(i, p.piece_inverse); };
        auto fetch = [&](int i) {
            const int token = token_of(i), piece = i - token * pieces;
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (token < tokens && piece * 8 < inputs) v = *reinterpret_cast<const uint4*>(x + token * p.k + piece * 8);
            return v;
        };
        // piece: inputs 8 (piece % 4) .. of lane t's 32 in step piece / 16
        auto put = [&](int token, int piece, const uint4& v) {
            const int step = piece >> 4, w = piece & 3, tt = (piece >> 2) & 3;
            sts128(sbase + L.x + (((step * 4 + w) * slab + token) * 4 + tt) * 16, v.x, v.y, v.z, v.w);
        };
        if constexpr (kBf16) {
            if (tid < kTokens) top[tid] = 0u;
            __syncthreads();
        }
        uint4 kept[kHeld];
        // a batch of pieces in flight, the first kept for the second look
        auto fetch_batch = [&](int i0) {
#pragma unroll
            for (int e = 0; e < kHeld; ++e) {
                const int i = i0 + tid + e * kThreads;
                kept[e] = make_uint4(0u, 0u, 0u, 0u);
                if (i < total) kept[e] = fetch(i);
            }
        };
        if constexpr (kBf16) {
            auto look = [&](int i0) {
#pragma unroll
                for (int e = 0; e < kHeld; ++e) {
                    const int i = i0 + tid + e * kThreads;
                    if (i - lane >= total) break;  // the warp's first piece
                    const uint4 v = kept[e];
                    uint32_t mx = 0u;  // largest magnitude of a lane's four pairs
                    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int q = 0; q < 4; ++q) mx = max(mx, max(u[q] & 0x7FFFu, (u[q] >> 16) & 0x7FFFu));
                    const int first = token_of(i - lane), last = token_of(min(i - lane + 31, total - 1));
                    if (first == last) {
                        mx = __reduce_max_sync(0xffffffffu, mx);
                        if (lane == 0 && mx) atomicMax(top + first, mx);
                    } else if (i < total && mx) {
                        atomicMax(top + token_of(i), mx);
                    }
                }
            };
            for (int i0 = kHeld * kThreads; i0 < total; i0 += kHeld * kThreads) {
                fetch_batch(i0);
                look(i0);
            }
            fetch_batch(0);
            look(0);
            __syncthreads();
            // exponent of the factor, 14 - (e - 127), within fp32's normal numbers
            auto up_of = [&](int token) { return min(max(127 + 14 - (static_cast<int>(top[token] >> 7) - 127), 1), 253); };
            if (tid < kTokens) back[tid] = __int_as_float((254 - up_of(tid)) << 23);
            for (int i0 = 0; i0 < total; i0 += kHeld * kThreads) {
                if (i0 > 0) fetch_batch(i0);
#pragma unroll
                for (int e = 0; e < kHeld; ++e) {
                    const int i = i0 + tid + e * kThreads;
                    if (i >= total) break;
                    const int token = token_of(i);
                    const float f = __int_as_float(up_of(token) << 23);
                    auto two = [&](uint32_t w) {
                        uint32_t r;
                        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(bf16_hi_to_f32(w) * f), "f"(bf16_lo_to_f32(w) * f));
                        return r;
                    };
                    put(token, i - token * pieces, make_uint4(two(kept[e].x), two(kept[e].y), two(kept[e].z), two(kept[e].w)));
                }
            }
        } else {
            for (int i0 = 0; i0 < total; i0 += kHeld * kThreads) {
                fetch_batch(i0);
#pragma unroll
                for (int e = 0; e < kHeld; ++e) {
                    const int i = i0 + tid + e * kThreads;
                    if (i >= total) break;
                    const int token = token_of(i);
                    put(token, i - token * pieces, kept[e]);
                }
            }
            if (tid < kTokens) back[tid] = 1.0f;
        }
    }
    __syncthreads();

    // -------------------------------------------------------------- compute --
    float acc[4];  // channels g (0, 1) and g + 8 (2, 3), tokens 2 t and 2 t + 1
    auto clear = [&] {
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = 0.0f;
    };
    clear();
    // Columns of tokens that are not there read another's: their sums go nowhere.
    const uint32_t x_word = slab * 64, x_step = 4 * x_word;
    const uint32_t x_first = sbase + L.x + (min(g, slab - 1) * 4 + t) * 16 + static_cast<uint32_t>(wk) * x_step;
    uint32_t x_at = x_first;
    auto compute = [&](const Fp4Step& s) {
        const uint32_t f0 = block_pair_f16(s.b0), f1 = block_pair_f16(s.b1);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint32_t w0 = q == 0 ? s.c0.x : q == 1 ? s.c0.y : q == 2 ? s.c0.z : s.c0.w;
            const uint32_t w1 = q == 0 ? s.c1.x : q == 1 ? s.c1.y : q == 2 ? s.c1.z : s.c1.w;
            uint32_t a[4], b[4];
            fp4_operands<false>(w0, q < 2 ? both_lo(f0) : both_hi(f0), a);
            fp4_operands<false>(w1, q < 2 ? both_lo(f1) : both_hi(f1), b);
            const uint4 x = lds128(x_at + q * x_word);
            mma_f16(acc, a[0], b[0], a[1], b[1], x.x, x.y);
            mma_f16(acc, a[2], b[2], a[3], b[3], x.z, x.w);
        }
    };
    // sums of a tile: [warp][token][channel]
    const int gt = G * 32, gtid = tid - group * gt;
    const int channel = gtid & (kRowsTile - 1);  // of this thread's results in every tile (gt is a multiple of 16)
    float scale = 0.0f, bias = 0.0f;
    auto ask = [&](int i) {  // ahead of their use
        const int64_t row = static_cast<int64_t>(tile_at(i)) * kRowsTile + channel;
        if (p.cl == 1 && gtid < slab * kRowsTile && i < rounds && row < p.n) {
            scale = p.scales[row];
            bias = p.bias ? p.bias[row] : 0.0f;
        }
    };
    ask(0);
    auto finish = [&](int i) {
        const uint32_t pitch = slab * kPitch * 4;  // of a warp's sums
        const uint32_t buf = sbase + L.red + static_cast<uint32_t>((i & 1) * kWarps) * pitch;
        const uint32_t own = buf + warp * pitch + (2 * t * kPitch + g) * 4;
#pragma unroll
        for (int e = 0; e < 2; ++e)
            if (2 * t + e < slab) {
                sts_f1(own + e * kPitch * 4, acc[e]);
                sts_f1(own + e * kPitch * 4 + 32, acc[2 + e]);
            }
        clear();
        if (G > 1)
            group_bar(group, gt);  // groups of 1 warp have no number for one
        else
            __syncwarp();
        const int64_t row = static_cast<int64_t>(tile_at(i)) * kRowsTile + channel;
        for (int o = gtid; o < slab * kRowsTile; o += gt) {
            const int token = o / kRowsTile;
            const uint32_t from = buf + group * G * pitch + (token * kPitch + channel) * 4;
            float sum = 0.0f;
#pragma unroll 4
            for (int w = 0; w < G; ++w) sum += lds_f1(from + w * pitch);
            sum *= back[token];
            if (p.cl > 1)
                sts_f1(sbase + L.part + static_cast<uint32_t>((i * J + group) * slab * kRowsTile + o) * 4, sum);
            else if (token < tokens && row < p.n)
                p.y[(m0 + token) * p.n + row] = round_out<kBf16>(fmaf(sum, scale, bias));
        }
        ask(i + 1);
    };
    int cs = S;  // steps to come of round ci
    for (int ci = 0; ci < my_rounds;) {
#pragma unroll
        for (int d = 0; d < kDepth; ++d) {
            compute(held[d]);
            load(held[d]);
            x_at += G * x_step;
            if (--cs == 0) {
                finish(ci);
                cs = S;
                x_at = x_first;
                if (++ci == my_rounds) break;
            }
        }
    }
    if (p.cl == 1) return;

    // ----------------------------------------------------------------- join --
    // the sums over the ranks in order, a share of them each
    cluster_sync_all();
    constexpr int kAtOnce = 4;  // results of a thread whose reads are in flight together
    const int per_tile = slab * kRowsTile, all = rounds * J * per_tile, stride = p.cl * kThreads;
    for (int o0 = rank * kThreads + tid; o0 < all; o0 += kAtOnce * stride) {
        float v[kAtOnce][kMaxSplit], sc[kAtOnce], bi[kAtOnce];
        int64_t at[kAtOnce];  // of the result, -1: none
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const int o = o0 + u * stride;
            const int n = divide(o, p.tile_inverse), in = o - n * per_tile, token = in / kRowsTile, i = divide(n, p.j_inverse);
            const int64_t row = static_cast<int64_t>((i * clusters + cluster) * J + (n - i * J)) * kRowsTile + (in & (kRowsTile - 1));
            const bool live = o < all && row < p.n && token < tokens;
            at[u] = live ? (m0 + token) * p.n + row : -1;
            sc[u] = live ? p.scales[row] : 0.0f;
            bi[u] = live && p.bias ? p.bias[row] : 0.0f;
#pragma unroll
            for (int r = 0; r < kMaxSplit; ++r)
                v[u][r] = live && r < p.cl ? ld_shared_cluster_f32(mapa_shared(sbase + L.part + static_cast<uint32_t>(o) * 4, r)) : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            float sum = 0.0f;
#pragma unroll
            for (int r = 0; r < kMaxSplit; ++r) sum += v[u][r];
            if (at[u] >= 0) p.y[at[u]] = round_out<kBf16>(fmaf(sum, sc[u], bi[u]));
        }
    }
    cluster_sync_all();  // no CTA leaves while another may read its shared memory
}

namespace {

template <bool kBf16>
cudaError_t launch_slab(const LinearArgs& a, int most, cudaStream_t st) {
    auto kern = fp4_few_kernel<kBf16>;
    static DeviceSetup setup;
    static int active[64][4];  // clusters of 1, 2, 4, 8 CTAs that fit the device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    int sms = 0;
    e = device_sm_count(sms);
    if (e != cudaSuccess) return e;
    e = setup(dev, [&] {
        cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMost);
        active[dev][0] = sms;
        for (int i = 1; i < 4 && err == cudaSuccess; ++i) {
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
            err = cudaOccupancyMaxActiveClusters(&active[dev][i], kern, &cfg);
        }
        return err;
    });
    if (e != cudaSuccess) return e;

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
    p.tiles = static_cast<int>((a.n + kRowsTile - 1) / kRowsTile);
    p.steps = static_cast<int>((a.k + kStepK - 1) / kStepK);
    p.early = a.early ? 1 : 0;
    const int slab = a.m < most ? static_cast<int>(a.m) : most;
    const int64_t slabs = (a.m + slab - 1) / slab;
    p.slab = slab;
    // Clusters and warps a tile that leave a warp the fewest steps, where the
    // activations fit; a tile's joins count as part of a step.
    double best = 1e30;
    int64_t grid = 0;
    uint32_t smem = 0;
    for (int c = 0; c < 4; ++c) {
        const int cl = 1 << c;
        if (active[dev][c] < 1) continue;
        const int per_rank = (p.steps + cl - 1) / cl;
        for (int g = 1; g <= kWarps && g <= p.steps / cl; ++g) {  // each warp has a step of each tile
            if (kWarps % g != 0) continue;
            const int J = kWarps / g, S = (per_rank + g - 1) / g;
            const int64_t want = (static_cast<int64_t>(p.tiles) + J - 1) / J;  // clusters of work
            int64_t clusters = active[dev][c] / slabs > 1 ? active[dev][c] / slabs : 1;
            if (clusters > want) clusters = want;
            const int64_t rounds = (want + clusters - 1) / clusters;
            if (rounds > 0x3fffffff) continue;
            // (where that many sums take over half of it, they do not fit)
            if (cl > 1 && rounds * J * slab * kRowsTile * 4 > kSmemMost / 2) continue;
            const Fp4Layout l = fp4_layout(slab, per_rank, static_cast<int>(rounds), J, cl > 1);
            if (l.total > kSmemMost) continue;
            const double waves = static_cast<double>((slabs * clusters * cl + sms - 1) / sms);
            const int pieces = (slab * per_rank * 16 + kThreads - 1) / kThreads, results = static_cast<int>((rounds * J * slab * kRowsTile / cl + kThreads - 1) / kThreads);
            const double cost = waves * (rounds * (S * kWarps * 56 + 200 + slab * J * g) + pieces * 250 + (cl > 1 ? 1500 + results * 200 : 0));
            if (cost < best) {
                best = cost;
                p.cl = cl;
                p.g = g;
                p.cl_log2 = c;
                p.j = J;
                p.rounds = static_cast<int>(rounds);
                p.per_rank = per_rank;
                grid = clusters * cl;
                smem = l.total;
            }
        }
    }
    if (grid == 0) return cudaErrorNotSupported;
    p.piece_inverse = inverse_of(16 * p.per_rank);
    p.tile_inverse = inverse_of(slab * kRowsTile);
    p.g_inverse = inverse_of(p.g);
    p.j_inverse = inverse_of(p.j);
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

// Fewer than 8 tokens a CTA where the activations of so many, or a cluster's sums of
// them, do not fit shared memory (8: k beyond 50 thousand or so; 1 fits always).
cudaError_t launch_fp4_few(const LinearArgs& a, cudaStream_t st) {
    cudaError_t e = cudaErrorNotSupported;
    for (int most = kTokens; e == cudaErrorNotSupported && most >= 1; most /= 2)
        e = a.act == FP8W_BF16 ? launch_slab<true>(a, most, st) : launch_slab<false>(a, most, st);
    return e;
}

}  // namespace fp8w
