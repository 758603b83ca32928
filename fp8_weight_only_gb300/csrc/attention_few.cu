// attention_few.cu -- kernel K8: attention of a few new tokens over a paged
// cache (decoding: one token a sequence, up to 16 query heads a tile).
//
// The mathematics of attention.cu with so few rows that the cache's bytes are
// all that counts: 4 * rows FLOPs a value of the cache, at 16 rows a
// thirtieth of what the tensor cores give beside the memory.  So the kernel is made for
// bytes in flight: no staging in shared memory and no barrier in the loop.
// A warp takes 16 to 64 keys at a time straight from the pages into
// registers, in the layout that the warp's matrix instruction (m16n8k16)
// wants its operands in, with the next keys' loads in flight meanwhile.
// Measured in this access pattern: 6.7 to 7.2 TB/s with 16- to 128-slot pages,
// against 4.3 to 5.2 by TMA boxes of a page into shared memory.
//
// Fragments.  The scores are computed transposed, 16 keys x 8 rows a matrix
// instruction (rows are few, keys are not), and the output too, 16 of the
// head's values x 8 rows.  A sum over the head's values runs in any order, so
// a thread reads 16 contiguous bytes of a key row and they are its operands of
// two (16-bit) or four (codes) steps; the queries are read in the same order.
// An output step's 16 values may be any of the head's, so a thread reads 8 or
// 16 contiguous values of four value rows and pairs them two rows to a word.
// The weights change from accumulators to operands by an 8 x 8 transposition.
//
// Softmax as in attention.cu: a row's reference moves only when its maximum
// has grown by more than 2^kSlack; until then no lane needs another's scores.
// Each warp has its own (m, l, O); a CTA's warps join theirs in shared memory
// and a cluster's CTAs theirs in distributed shared memory, in rank order.
//
// Measured: a decode batch of 96 sequences (1.2 GB of a 16-bit cache) 224 us, 5.4
// TB/s, 81% of the measured copy rate: the last CTAs of uneven sequences and each
// one's start, not the loop.  The same of codes: 146 us, 64%: conversions, 45% of
// the ALU pipe.  Heads of 64: 123 us, 73%, and of codes 113, 43%.  Two sequences of
// 90 and 131 thousand tokens of codes: 144 us, 52%: besides, 16 (sequence, head)
// pairs of at most 16 CTAs are 1.7 CTAs an SM.
// One short sequence: 8 us, four dependent reads of memory and a launch.
// 4 bits (fp4.cuh): the block's scale goes into the fp16 operands, exactly; a thread
// has 32 codes of a key row (two blocks) and 16 of a value row (one).  The decode batch,
// 349 MB of it, 129 us, 40%, the two long sequences 123, 35%: latency.  A warp needs 436
// instructions for 16 keys, of them 150 conversions, multiplies and products, and 244
// registers leave two warps a scheduler, too few to cover each other's waits: 0.37
// instructions issued a cycle, the busiest pipe (ALU) at 31%.  (Three warps, with 16 keys
// a step: 132.)
#include <type_traits>

#include "attention.cuh"
#include "fp4.cuh"

namespace fp8w {

__device__ int g_attention_few_error;

namespace {

constexpr int kFewWarps = 4;
constexpr int kMaxFewCluster = 16;
constexpr int kFewFill = 8;   // CTAs an SM up to which clusters grow
constexpr int kFewSteps = 2;  // steps a warp that stay at least

template <bool kBf16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint4& a, uint32_t b0, uint32_t b1) {
    if constexpr (kBf16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

// An 8 x 8 matrix of 16-bit values, a row to four lanes: its transpose.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// kForm: the cache's (attention.cuh).
template <int DP, int kForm, int NT>
struct FewShape {
    static constexpr bool kFp8 = kForm != kForm16, kFp4 = kForm == kFormFp4;
    static constexpr int kTile = 8 * NT;                               // rows
    static constexpr int kSubs = (DP == 64 ? 2 : 1) * (kFp8 && NT == 1 ? 2 : 1);  // 16-key parts a step of the loop
    static constexpr int kStepKeys = 16 * kSubs;
    static constexpr int kKeyPieces = kFp4 ? 1 : kFp8 ? DP / 64 : DP / 32;  // 16-byte pieces of a key row a thread (4 bits, DP 64: 8 bytes)
    static constexpr int kValuePieces = kFp8 ? 1 : DP / 64;            // pieces of a value row: 16 bytes (DP / 8 with codes, DP / 16 with 4 bits)
    static constexpr uint32_t kStageOff = 0;                           // fp32 [warps][rows][DP]
    static constexpr uint32_t kMlOff = kFewWarps * kTile * DP * 4;
    static constexpr uint32_t kJoinedOff = kMlOff + kFewWarps * kTile * 8;
    // Registers that a load leaves out keep their values: fewer instructions, but
    // they stay occupied, and the wide forms have none to spare (a decode batch of
    // heads of 64: 122 us against 143; of 128 no difference, its codes 191 against 142).
    static constexpr bool kKeeps = DP == 64 && !kFp8;
    // the queries' operands: registers, or shared memory where those are short
    static constexpr bool kQShared = NT == 2 && DP == 128 && !kFp8;
    static constexpr uint32_t kQOff = kJoinedOff + kTile * 8;
    static constexpr uint32_t kBytes = kQOff + (kQShared ? NT * DP / 16 * 32 * 8 : 0);
};

// What a thread holds of one step's keys (g = lane / 4, t = lane % 4).
template <int DP, int kForm, int NT>
struct Step {
    using S = FewShape<DP, kForm, NT>;
    static constexpr bool kFp8 = S::kFp8;
    uint4 k[S::kSubs][2][S::kKeyPieces];    // key rows g and g + 8
    uint4 v[S::kSubs][4][S::kValuePieces];  // value rows 2t, 2t + 1, 2t + 8, 2t + 9
    float ks[kFp8 ? S::kSubs : 1][2], vs[kFp8 ? S::kSubs : 1][2];  // scales of keys g and g + 8
    // 4 bits, bytes of blocks' scales: those of this thread's part of key rows g and
    // g + 8 (two, DP 64: one), and of its part of the four value rows (one each)
    uint32_t kb[S::kFp4 ? S::kSubs : 1][2], vb[S::kFp4 ? S::kSubs : 1][4];
};

}  // namespace

template <int DP, bool kBf16, int kForm, int NT>
__global__ void __launch_bounds__(kFewWarps * 32, 2) attention_few_kernel(const __grid_constant__ AttnParams p) {
    using S = FewShape<DP, kForm, NT>;
    using H = Step<DP, kForm, NT>;
    constexpr bool kFp8 = S::kFp8, kFp4 = S::kFp4;  // codes; of 4 bits
    constexpr int kSubs = S::kSubs, kStepKeys = S::kStepKeys, kTile = S::kTile;
    constexpr int kEl = kFp8 ? 1 : 2;  // bytes an element of the cache (4 bits: two values)
    // Codes are multiplied as fp16 whatever the activations' type: one conversion
    // instruction makes two of them, and the weights round to 11 bits.  bf16
    // queries go over exactly but for a power of two a row (below).
    constexpr bool kMmaBf16 = kBf16 && !kFp8;
    constexpr float kSlack = 8.0f, kLift = kMmaBf16 ? 0.0f : kLiftF16;
    __shared__ __align__(16) uint8_t smem[S::kBytes];
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;

    pdl_launch_dependents();
    pdl_wait();
    const int rank = p.cl > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int item = static_cast<int>(blockIdx.x) / p.cl;
    const int tile = item / p.kv_heads, head = item - tile * p.kv_heads;
    SeqTile f;
    const bool have = find_tile(p, kTile, tile, blockIdx.x == 0 && warp == 0, &g_attention_few_error, f);
    // ranks of a cluster share the tile, so all of them leave here
    if (!have) return;
    const int total = static_cast<int>(f.count * p.group), row0 = f.inner * kTile;
    const int rows = total - row0 < kTile ? total - row0 : kTile;
    const int pos0 = static_cast<int>(f.len - f.count);
    const int end = pos0 + (row0 + rows - 1) / p.group + 1;
    const int64_t from = p.window > 0 ? static_cast<int64_t>(pos0) + row0 / p.group - p.window + 1 : 0;
    const int first = from > 0 ? static_cast<int>(from) : 0;
    const int32_t* table = p.table + static_cast<int64_t>(f.seq) * p.table_width;
    auto row_at = [&](int row, int64_t stride) {  // element of an operand's row
        const int R = row0 + row, token = R / p.group, h = R - token * p.group;
        return (f.begin + token) * stride + static_cast<int64_t>(head * p.group + h) * p.head_dim;
    };

    // ------------------------------------------------------------- queries --
    // this thread's operands of step s for row tile n: row 8 n + g, four values
    uint2 q[S::kQShared ? 1 : NT][S::kQShared ? 1 : DP / 16];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int s = 0; s < DP / 16; ++s) {
            const int d = kFp4 ? t * (DP / 4) + s * 4 : kFp8 ? (s >> 2) * 64 + t * 16 + (s & 3) * 4 : (s >> 1) * 32 + t * 8 + (s & 1) * 4;
            uint2 y = make_uint2(0u, 0u);
            if (8 * n + g < rows && d < p.head_dim) y = *reinterpret_cast<const uint2*>(p.q + row_at(8 * n + g, p.q_stride) + d);
            if constexpr (!S::kQShared)
                q[n][s] = y;
            else if (warp == s % kFewWarps)
                asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(sbase + S::kQOff + ((n * (DP / 16) + s) * 32 + lane) * 8), "r"(y.x), "r"(y.y) : "memory");
        }
    if constexpr (S::kQShared) __syncthreads();
    // bf16 queries to fp16: each row times the power of two that takes its
    // largest value to [2^14, 2^15).  What falls below fp16's normal numbers then
    // is less than 2^-28 of the largest, off by 2^-39 of it.  The scores of rows
    // 2t, 2t + 1 get the factor back.
    float c[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        c[n][0] = c[n][1] = p.c;
        if constexpr (kFp8 && kBf16) {
            uint32_t top = 0u;  // bit pattern of the row's largest magnitude
#pragma unroll
            for (int s = 0; s < DP / 16; ++s)
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const uint32_t y = w ? q[n][s].y : q[n][s].x;
                    top = max(top, max(y & 0x7FFFu, (y >> 16) & 0x7FFFu));
                }
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // exponents of the row and of the factor, 14 - (e - 127), within fp32's normal numbers
            const int exponent = static_cast<int>(top >> 7);
            const int up = min(max(127 + 14 - (exponent - 127), 1), 253);
            const float factor = __int_as_float(up << 23), back = __int_as_float((254 - up) << 23) * p.c;
#pragma unroll
            for (int s = 0; s < DP / 16; ++s) {
                const uint2 y = q[n][s];
                q[n][s].x = pack16<false>(bf16_lo_to_f32(y.x) * factor, bf16_hi_to_f32(y.x) * factor);
                q[n][s].y = pack16<false>(bf16_lo_to_f32(y.y) * factor, bf16_hi_to_f32(y.y) * factor);
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) c[n][r] = __shfl_sync(0xffffffffu, back, 4 * (2 * t + r));
        }
    }

    // positions that rows 8 n + 2t and 8 n + 2t + 1 see
    int hi[NT][2], lo[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = 8 * n + 2 * t + i, pos = pos0 + (row0 + row) / p.group;
            const int64_t from_row = p.window > 0 ? static_cast<int64_t>(pos) - p.window + 1 : 0;
            hi[n][i] = row < rows ? pos : -1;
            lo[n][i] = from_row > 0 ? static_cast<int>(from_row) : 0;
        }
    const int all_hi = pos0 + row0 / p.group;                                       // every row sees up to here
    const int last = pos0 + (row0 + rows - 1) / p.group;
    const int64_t all_from = p.window > 0 ? static_cast<int64_t>(last) - p.window + 1 : 0;
    const int all_lo = all_from > 0 ? static_cast<int>(all_from) : 0;               // and from here

    // ---------------------------------------------------------------- loads --
    const int step0 = first / kStepKeys, steps = end > 0 ? (end + kStepKeys - 1) / kStepKeys : 0;
    const int workers = p.cl * kFewWarps;
    const int64_t token_bytes = p.token_stride * kEl, page_bytes = p.page_stride * kEl;
    const uint8_t* kbase = static_cast<const uint8_t*>(p.k) + static_cast<int64_t>(head) * p.head_stride * kEl;
    const uint8_t* vbase = static_cast<const uint8_t*>(p.v) + static_cast<int64_t>(head) * p.head_stride * kEl;
    // this thread's part of a 16-key block: key rows g and g + 8, value rows 2t, 2t + 1 and + 8
    constexpr int kKeyBytes = kFp4 ? DP / 8 : 16, kValueBytes = kFp4 ? DP / 16 : kFp8 ? DP / 8 : 16;  // of a piece
    const uint8_t* kthread = kbase + g * token_bytes + t * kKeyBytes;
    const uint8_t* vthread = vbase + 2 * t * token_bytes + g * kValueBytes;
    const int row_bytes = kFp4 ? p.head_dim >> 1 : p.head_dim * kEl, row_blocks = p.head_dim >> 4;
    auto load_codes = [&](const uint8_t* at, auto bytes) {  // a row's codes of this thread
        uint4 y = make_uint4(0u, 0u, 0u, 0u);
        if constexpr (bytes.value == 4) {
            y.x = *reinterpret_cast<const uint32_t*>(at);
        } else if constexpr (bytes.value == 16) {
            y = ld_stream_v4(at);
        } else {
            const uint2 z = *reinterpret_cast<const uint2*>(at);
            y.x = z.x, y.y = z.y;
        }
        return y;
    };
    // table entries of a step, one per 16 keys (a page has 16 slots or more);
    // read ahead of the step's loads
    auto entries = [&](int st, int (&e)[kSubs]) {
#pragma unroll
        for (int i = 0; i < kSubs; ++i) {
            const int key = st * kStepKeys + 16 * i;
            e[i] = st < steps && key < end && key + 16 > first ? table[key >> p.log_page] : -1;
        }
    };
    // 4 bits: this thread's places in the scales and the blocks' scales of page 0, slot 0
    const bool k_here = t * kKeyBytes < row_bytes, v_here = g * (DP / 8) < p.head_dim;
    const int64_t head_slot = static_cast<int64_t>(head) * p.page_size;
    const float* const ks_thread = kFp4 ? p.k_scales + head_slot + g : nullptr;
    const float* const vs_thread = kFp4 ? p.v_scales + head_slot + g : nullptr;
    const uint8_t* const kb_thread = kFp4 ? p.k_blocks + (head_slot + g) * row_blocks + t * (DP / 64) : nullptr;
    const uint8_t* const vb_thread = kFp4 ? p.v_blocks + (head_slot + 2 * t) * row_blocks + g * (DP / 8) / 16 : nullptr;
    const uint32_t page_slots = static_cast<uint32_t>(p.kv_heads) * static_cast<uint32_t>(p.page_size);
    auto load = [&](int st, const int (&e)[kSubs], H& x) {
        if constexpr (kFp4) {
            // Whole steps of keys that are all wanted, the most of a long cache, without
            // a test a load: with so few warps a warp's own instructions are the time (a
            // decode batch: 129 us, 167 without this).
            bool whole = st < steps && st * kStepKeys >= first && (st + 1) * kStepKeys <= end;
#pragma unroll
            for (int i = 0; i < kSubs; ++i) whole = whole && static_cast<uint32_t>(e[i]) < static_cast<uint32_t>(p.num_pages);
            if (whole) {
#pragma unroll
                for (int i = 0; i < kSubs; ++i) {
                    const int slot = (st * kStepKeys + 16 * i) & (p.page_size - 1);
                    const int64_t at = e[i] * page_bytes + slot * token_bytes;
                    const uint64_t sc = static_cast<uint64_t>(static_cast<uint32_t>(e[i])) * page_slots + static_cast<uint32_t>(slot);
                    const uint8_t *kr = kthread + at, *vr = vthread + at, *kb = kb_thread + sc * row_blocks, *vb = vb_thread + sc * row_blocks;
                    const float *ks = ks_thread + sc, *vs = vs_thread + sc;
                    if (k_here) {
                        x.k[i][0][0] = load_codes(kr, std::integral_constant<int, kKeyBytes>{});
                        x.k[i][1][0] = load_codes(kr + 8 * token_bytes, std::integral_constant<int, kKeyBytes>{});
                        if constexpr (DP == 128) {
                            x.kb[i][0] = *reinterpret_cast<const uint16_t*>(kb);
                            x.kb[i][1] = *reinterpret_cast<const uint16_t*>(kb + 8 * row_blocks);
                        } else {
                            x.kb[i][0] = *kb;
                            x.kb[i][1] = kb[8 * row_blocks];
                        }
                    }
                    x.ks[i][0] = ks[0];
                    x.ks[i][1] = ks[8];
                    x.vs[i][0] = vs[0];
                    x.vs[i][1] = vs[8];
                    if (v_here) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int r = (j >> 1) * 8 + (j & 1);
                            x.v[i][j][0] = load_codes(vr + r * token_bytes, std::integral_constant<int, kValueBytes>{});
                            x.vb[i][j] = vb[r * row_blocks];
                        }
                    }
                }
                return;
            }
        }
        // Slots at or past `end` may hold anything and are not read: zeros instead, or
        // (kKeeps) what an earlier step left in the registers, finite values whose
        // weights are 0.
#pragma unroll
        for (int i = 0; i < kSubs; ++i) {
            const int key16 = st * kStepKeys + 16 * i, slot = key16 & (p.page_size - 1);
            const bool wanted = st < steps && key16 < end && key16 + 16 > first;
            const bool page = wanted && e[i] >= 0 && e[i] < p.num_pages;
            if (wanted && !page) atomicCAS(&g_attention_few_error, 0, 7000 + kErrIndex);
            const int64_t at = e[i] * page_bytes + slot * token_bytes;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int key = key16 + g + 8 * r;
                const bool in = page && key < end && key >= first;
#pragma unroll
                for (int j = 0; j < S::kKeyPieces; ++j) {
                    if constexpr (!S::kKeeps) x.k[i][r][j] = make_uint4(0u, 0u, 0u, 0u);
                    if constexpr (kFp4) {
                        if (in && t * kKeyBytes < row_bytes)
                            x.k[i][r][j] = load_codes(kthread + at + 8 * r * token_bytes, std::integral_constant<int, kKeyBytes>{});
                    } else {
                        if (in && j * 64 + t * 16 < row_bytes) x.k[i][r][j] = ld_stream_v4(kthread + at + 8 * r * token_bytes + j * 64);
                    }
                }
                if constexpr (kFp8) {
                    const int64_t sc = (static_cast<int64_t>(e[i]) * p.kv_heads + head) * p.page_size + slot + g + 8 * r;
                    x.ks[i][r] = in ? p.k_scales[sc] : 0.0f;
                    x.vs[i][r] = in ? p.v_scales[sc] : 0.0f;
                    if constexpr (kFp4) {
                        x.kb[i][r] = 0u;
                        if (in && t * kKeyBytes < row_bytes) {
                            const uint8_t* b = p.k_blocks + sc * row_blocks + t * (DP / 64);
                            x.kb[i][r] = DP == 128 ? *reinterpret_cast<const uint16_t*>(b) : *b;
                        }
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = (j >> 1) * 8 + (j & 1), key = key16 + 2 * t + r;
                const bool in = page && key < end && key >= first;
                const uint8_t* row = vthread + at + r * token_bytes;
#pragma unroll
                for (int h = 0; h < S::kValuePieces; ++h) {
                    if constexpr (!S::kKeeps) x.v[i][j][h] = make_uint4(0u, 0u, 0u, 0u);
                    if constexpr (kFp8) {
                        const bool here = in && g * (DP / 8) < p.head_dim;
                        if (here) x.v[i][j][h] = load_codes(row, std::integral_constant<int, kValueBytes>{});
                        if constexpr (kFp4) {
                            x.vb[i][j] = 0u;
                            if (here) {
                                const int64_t sc = (static_cast<int64_t>(e[i]) * p.kv_heads + head) * p.page_size + slot + 2 * t + r;
                                x.vb[i][j] = p.v_blocks[sc * row_blocks + g * (DP / 8) / 16];
                            }
                        }
                    } else {
                        if (in && h * 64 + g * 8 < p.head_dim) x.v[i][j][h] = ld_stream_v4(row + h * 128);
                    }
                }
            }
        }
    };

    // -------------------------------------------------------------- compute --
    // rows 8 n + 2t and 8 n + 2t + 1: reference and sum; o[i][n] the i-th 16 values'
    // accumulators (value 2i and 2i + 1 of this thread's, for each of the rows)
    float m[NT][2], l[NT][2], o[DP / 16][NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        m[n][0] = m[n][1] = kNegInf;
        l[n][0] = l[n][1] = 0.0f;
#pragma unroll
        for (int i = 0; i < DP / 16; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[i][n][j] = 0.0f;
    }
    auto compute = [&](int st, const H& x) {
        uint32_t q_at = sbase + S::kQOff + lane * 8;
        if constexpr (S::kQShared) asm volatile("" : "+r"(q_at));  // read in every step, not kept
        float s[kSubs][NT][4];  // keys g (0, 1) and g + 8 (2, 3) of rows 2t, 2t + 1
#pragma unroll
        for (int i = 0; i < kSubs; ++i)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[i][n][j] = 0.0f;
#pragma unroll
        for (int k = 0; k < DP / 16; ++k) {
#pragma unroll
            for (int i = 0; i < kSubs; ++i) {
                uint4 a;
                if constexpr (kFp4) {
                    // half k & 1 of a word: four codes
                    const uint4 w = x.k[i][0][0], u = x.k[i][1][0];
                    const int q = k >> 1;
                    const uint32_t f = block_pair_f16(x.kb[i][0]), h = block_pair_f16(x.kb[i][1]);
                    const bool second = DP == 128 && q >= 2;  // of the thread's blocks
                    uint32_t c[4], d[4];
                    fp4_operands<false>(q == 0 ? w.x : q == 1 ? w.y : q == 2 ? w.z : w.w, second ? both_hi(f) : both_lo(f), c);
                    fp4_operands<false>(q == 0 ? u.x : q == 1 ? u.y : q == 2 ? u.z : u.w, second ? both_hi(h) : both_lo(h), d);
                    a = (k & 1) ? make_uint4(c[2], d[2], c[3], d[3]) : make_uint4(c[0], d[0], c[1], d[1]);
                } else if constexpr (kFp8) {
                    const uint4 w = x.k[i][0][k >> 2], u = x.k[i][1][k >> 2];
                    e4m3x4_to_f16x2((k & 3) == 0 ? w.x : (k & 3) == 1 ? w.y : (k & 3) == 2 ? w.z : w.w, a.x, a.z);
                    e4m3x4_to_f16x2((k & 3) == 0 ? u.x : (k & 3) == 1 ? u.y : (k & 3) == 2 ? u.z : u.w, a.y, a.w);
                } else {
                    const uint4 w = x.k[i][0][k >> 1], u = x.k[i][1][k >> 1];
                    a = (k & 1) ? make_uint4(w.z, u.z, w.w, u.w) : make_uint4(w.x, u.x, w.y, u.y);
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    uint2 b;
                    if constexpr (S::kQShared)
                        asm("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(b.x), "=r"(b.y) : "r"(q_at + (n * (DP / 16) + k) * 256));
                    else
                        b = q[n][k];
                    mma16816<kMmaBf16>(s[i][n], a, b.x, b.y);
                }
            }
        }
        const int key0 = st * kStepKeys;
        const bool masked = key0 + kStepKeys - 1 > all_hi || key0 < all_lo;
        // Exponents of two.  With codes m is the reference of weight times value
        // scale, which is what has to fit 16 bits; the sum of the weights alone is
        // fp32 and takes what stands against it.
        bool grow = false;
#pragma unroll
        for (int i = 0; i < kSubs; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int key = key0 + 16 * i + 8 * (j >> 1) + g;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float y = s[i][n][j] * c[n][j & 1];
                    if constexpr (kFp8) y *= x.ks[i][j >> 1];
                    if (masked && (key > hi[n][j & 1] || key < lo[n][j & 1])) y = kNegInf;
                    s[i][n][j] = y;
                    if constexpr (!kFp8) grow |= y - m[n][j & 1] > kSlack;  // -inf - -inf: no
                }
            }
        float vs[kFp8 ? kSubs : 1][2], lv[kFp8 ? kSubs : 1][2];
        if constexpr (kFp8) {
            // A row of zeros has the scale 1, as if its values reached 448: left so, a
            // large score there would set the reference and the weights of small values
            // would go below fp16.  So where a scale is 1, look at the codes: 0 for it.
            bool one = false;
#pragma unroll
            for (int i = 0; i < kSubs; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    vs[i][h] = x.vs[i][h];
                    one |= vs[i][h] == 1.0f;
                }
            if (__any_sync(0xffffffffu, one)) {
#pragma unroll
                for (int i = 0; i < kSubs; ++i) {
                    unsigned any = 0;  // a bit for each of the 16 keys
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint4 y = x.v[i][j][0];
                        if ((y.x | y.y | y.z | y.w) & (kFp4 ? 0x77777777u : 0x7F7F7F7Fu)) any |= 1u << (2 * t + (j >> 1) * 8 + (j & 1));
                    }
                    any = __reduce_or_sync(0xffffffffu, any);
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        if (!(any >> (g + 8 * h) & 1u)) vs[i][h] = 0.0f;
                }
            }
#pragma unroll
            for (int i = 0; i < kSubs; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    lv[i][h] = log2_scale(vs[i][h]);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int r = 0; r < 2; ++r) grow |= s[i][n][2 * h + r] + lv[i][h] - m[n][r] > kSlack;
                }
        }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float mx = kNegInf;
#pragma unroll
                    for (int i = 0; i < kSubs; ++i)
#pragma unroll
                        for (int h = 0; h < 2; ++h) mx = fmaxf(mx, s[i][n][2 * h + r] + (kFp8 ? lv[kFp8 ? i : 0][h] : 0.0f));
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                    if (mx - m[n][r] > kSlack) {  // by its own row alone: other rows of the tile change nothing in it
                        const float alpha = ex2(m[n][r] - mx);
                        m[n][r] = mx;
                        l[n][r] *= alpha;
#pragma unroll
                        for (int i = 0; i < DP / 16; ++i) o[i][n][r] *= alpha, o[i][n][2 + r] *= alpha;
                    }
                }
        }
#pragma unroll
        for (int i = 0; i < kSubs; ++i) {
            uint32_t b[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float ref0 = m[n][0] == kNegInf ? 0.0f : m[n][0] - kLift, ref1 = m[n][1] == kNegInf ? 0.0f : m[n][1] - kLift;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float e0 = ex2(s[i][n][2 * h] - ref0), e1 = ex2(s[i][n][2 * h + 1] - ref1);
                    l[n][0] += e0;
                    l[n][1] += e1;
                    if constexpr (kFp8) {
                        e0 *= vs[i][h];
                        e1 *= vs[i][h];
                    }
                    b[n][h] = transpose8(pack16<kMmaBf16>(e0, e1));
                }
            }
            // 16 values a product: this thread's values 2 j and 2 j + 1 of its four rows
#pragma unroll
            for (int j = 0; j < DP / 16; j += kFp4 ? 4 : kFp8 ? 2 : 1) {
                if constexpr (kFp4) {
                    // a word of 8 codes of each row, paired row by row: even values in
                    // the bytes of lo[], odd ones in those of hi[]
                    uint32_t lo[2], hi[2], f[2];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const uint4 y = x.v[i][2 * r][0], z = x.v[i][2 * r + 1][0];
                        const uint32_t a = j / 4 == 0 ? y.x : y.y, b = j / 4 == 0 ? z.x : z.y;
                        lo[r] = (a & 0x0F0F0F0Fu) | ((b << 4) & 0xF0F0F0F0u);
                        hi[r] = ((a >> 4) & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u);
                        f[r] = block_pair_f16(x.vb[i][2 * r] | (x.vb[i][2 * r + 1] << 8));
                    }
                    uint32_t v[2][2][4];  // [rows 2t or 2t + 8][even or odd value][pair of values]
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        e2m1x8_to_f16x2(lo[r], v[r][0][0], v[r][0][1], v[r][0][2], v[r][0][3]);
                        e2m1x8_to_f16x2(hi[r], v[r][1][0], v[r][1][1], v[r][1][2], v[r][1][3]);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint4 a = make_uint4(f16x2_mul(v[0][0][e], f[0]), f16x2_mul(v[0][1][e], f[0]), f16x2_mul(v[1][0][e], f[1]),
                                                   f16x2_mul(v[1][1][e], f[1]));
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma16816<kMmaBf16>(o[j + e][n], a, b[n][0], b[n][1]);
                    }
                } else if constexpr (kFp8) {
                    uint32_t c[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const uint4 y = x.v[i][r][0];
                        c[r] = j / 2 == 0 ? y.x : j / 2 == 1 ? y.y : j / 2 == 2 ? y.z : y.w;
                    }
                    uint4 a0, a1;
                    e4m3x4_to_f16x2(__byte_perm(c[0], c[1], 0x5140), a0.x, a0.y);
                    e4m3x4_to_f16x2(__byte_perm(c[0], c[1], 0x7362), a1.x, a1.y);
                    e4m3x4_to_f16x2(__byte_perm(c[2], c[3], 0x5140), a0.z, a0.w);
                    e4m3x4_to_f16x2(__byte_perm(c[2], c[3], 0x7362), a1.z, a1.w);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        mma16816<kMmaBf16>(o[j][n], a0, b[n][0], b[n][1]);
                        mma16816<kMmaBf16>(o[j + 1][n], a1, b[n][0], b[n][1]);
                    }
                } else {
                    uint32_t c[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const uint4 y = x.v[i][r][j / 4];
                        c[r] = j % 4 == 0 ? y.x : j % 4 == 1 ? y.y : j % 4 == 2 ? y.z : y.w;
                    }
                    const uint4 a = make_uint4(__byte_perm(c[0], c[1], 0x5410), __byte_perm(c[0], c[1], 0x7632),
                                               __byte_perm(c[2], c[3], 0x5410), __byte_perm(c[2], c[3], 0x7632));
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma16816<kMmaBf16>(o[j][n], a, b[n][0], b[n][1]);
                }
            }
        }
    };
    {
        // steps step0 + worker, + workers, ..: one in work, one in flight, the table
        // one further.  All in one straight line, loads and products: with a branch
        // around the loads of whole steps the same loop took a tenth longer.
        int st = step0 + rank * kFewWarps + warp;
        int e[kSubs];
        H x0 = {}, x1 = {};
        entries(st, e);
        load(st, e, x0);
        entries(st + workers, e);
        while (st < steps) {
            load(st + workers, e, x1);
            entries(st + 2 * workers, e);
            compute(st, x0);
            st += workers;
            if (st >= steps) break;
            load(st + workers, e, x0);
            entries(st + 2 * workers, e);
            compute(st, x1);
            st += workers;
        }
    }

    // ----------------------------------------------------------------- join --
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) l[n][r] += __shfl_xor_sync(0xffffffffu, l[n][r], d);
    auto stage_at = [&](int w, int row, int chunk) {  // 16-byte chunk of a warp's partial row
        return sbase + S::kStageOff + static_cast<uint32_t>((w * kTile + row) * DP + ((chunk ^ (row & 7)) << 2)) * 4u;
    };
    auto ml_at = [&](int w, int row) { return sbase + S::kMlOff + (w * kTile + row) * 8; };
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = 8 * n + 2 * t + r;
            if (row >= rows) continue;
            if (g == 0)
                asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(ml_at(warp, row)), "f"(m[n][r]), "f"(l[n][r]) : "memory");
            // this thread's values: kRun from g * kRun on (16-bit, 128 values: of each half)
            constexpr int kRun = kFp8 ? DP / 8 : 8;
#pragma unroll
            for (int j = 0; j < DP / 8; j += 4) {
                const int d = (j / kRun) * 64 + g * kRun + j % kRun;
                sts128(stage_at(warp, row, d / 4), __float_as_uint(o[j / 2][n][r]), __float_as_uint(o[j / 2][n][2 + r]),
                       __float_as_uint(o[j / 2 + 1][n][r]), __float_as_uint(o[j / 2 + 1][n][2 + r]));
            }
        }
    __syncthreads();
    auto write = [&](int row, int chunk, const float* acc, float sum) {
        const float inv = weight_inverse(sum, pos0 + (row0 + row) / p.group >= 0);
        if (chunk * 4 < p.head_dim)
            *reinterpret_cast<uint2*>(p.out + row_at(row, p.out_stride) + chunk * 4) =
                make_uint2(pack16<kBf16>(acc[0] * inv, acc[1] * inv), pack16<kBf16>(acc[2] * inv, acc[3] * inv));
    };
    const int units = rows * (DP / 4);
    for (int u = threadIdx.x; u < units; u += kFewWarps * 32) {
        const int row = u / (DP / 4), chunk = u - row * (DP / 4);
        float2 q[kFewWarps];
        float top = kNegInf, sum = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w) {
            asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(q[w].x), "=f"(q[w].y) : "r"(ml_at(w, row)) : "memory");
            if (q[w].y != 0.0f) top = fmaxf(top, q[w].x);
        }
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w) {
            if (q[w].y == 0.0f) continue;
            const uint4 y = lds128(stage_at(w, row, chunk));
            const float a = ex2(q[w].x - top);
            sum = fmaf(q[w].y, a, sum);
            acc[0] = fmaf(__uint_as_float(y.x), a, acc[0]);
            acc[1] = fmaf(__uint_as_float(y.y), a, acc[1]);
            acc[2] = fmaf(__uint_as_float(y.z), a, acc[2]);
            acc[3] = fmaf(__uint_as_float(y.w), a, acc[3]);
        }
        if (p.cl == 1) {
            write(row, chunk, acc, sum);
        } else {
            // in the first warp's place, which no other thread reads; (m, l) apart
            sts128(stage_at(0, row, chunk), __float_as_uint(acc[0]), __float_as_uint(acc[1]), __float_as_uint(acc[2]),
                   __float_as_uint(acc[3]));
            if (chunk == 0)
                asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(sbase + S::kJoinedOff + row * 8), "f"(top), "f"(sum) : "memory");
        }
    }
    if (p.cl == 1) return;
    cluster_sync_all();
    {
        // each rank finishes its share of the 16-byte chunks, several lanes to
        // one where there are few, each on some of the ranks
        const int share = (units + p.cl - 1) / p.cl;
        int lanes = 1;
        while (2 * lanes <= p.cl && 2 * share * lanes <= kFewWarps * 32) lanes *= 2;
        const int k0 = static_cast<int>(threadIdx.x) & (lanes - 1);
        for (int b = 0; b < share; b += kFewWarps * 32 / lanes) {
            const int i = b + static_cast<int>(threadIdx.x) / lanes, u = rank * share + i;
            const bool live = i < share && u < units;
            const int row = live ? u / (DP / 4) : 0, chunk = live ? u - row * (DP / 4) : 0;
            const uint32_t joined = sbase + S::kJoinedOff + row * 8, part = stage_at(0, row, chunk);
            float top = kNegInf, sum = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            auto add = [&](float o_top, float o_sum, const float (&y)[4]) {
                if (o_sum == 0.0f) return;
                const float to = fmaxf(top, o_top);
                const float a = ex2(top - to), z = ex2(o_top - to);
                top = to;
                sum = sum * a + o_sum * z;
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[e] = acc[e] * a + y[e] * z;
            };
            for (int k = k0; k < p.cl; k += 4 * lanes) {
                float2 q[4];
                float4 y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t other = static_cast<uint32_t>(k + e * lanes < p.cl ? k + e * lanes : k);
                    q[e] = ld_cluster_f2(mapa_shared(joined, other));
                    y[e] = ld_cluster_f4(mapa_shared(part, other));
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float z[4] = {y[e].x, y[e].y, y[e].z, y[e].w};
                    add(q[e].x, k + e * lanes < p.cl ? q[e].y : 0.0f, z);
                }
            }
            for (int d = lanes >> 1; d > 0; d >>= 1) {
                float z[4];
                const float o_top = __shfl_xor_sync(0xffffffffu, top, d), o_sum = __shfl_xor_sync(0xffffffffu, sum, d);
#pragma unroll
                for (int e = 0; e < 4; ++e) z[e] = __shfl_xor_sync(0xffffffffu, acc[e], d);
                add(o_top, o_sum, z);
            }
            if (live && k0 == 0) write(row, chunk, acc, sum);
        }
    }
    cluster_sync_all();  // no CTA leaves while another may read its shared memory
}

namespace {

template <int DP, bool kBf16, int kForm, int NT>
cudaError_t launch_few(const AttentionArgs& a, cudaStream_t st) {
    using S = FewShape<DP, kForm, NT>;
    auto kern = attention_few_kernel<DP, kBf16, kForm, NT>;
    static DeviceSetup setup;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    int sms = 0;
    e = device_sm_count(sms);
    if (e != cudaSuccess) return e;
    e = setup(dev, [&] { return cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1); });
    if (e != cudaSuccess) return e;

    AttnParams p = attention_params(a);
    const int64_t tiles = attention_row_tiles(a, p.group, S::kTile), items = tiles * p.kv_heads;
    const int64_t steps = (attention_longest(a) + S::kStepKeys - 1) / S::kStepKeys;
    int cl = 1;
    while (cl < kMaxFewCluster && items * cl <= kFewFill * sms && steps >= cl * 2 * kFewWarps * kFewSteps) cl *= 2;
    if (items * cl > 0x7fffffffll) return cudaErrorInvalidConfiguration;
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
    cfg.blockDim = dim3(kFewWarps * 32);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = cl > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int DP, int NT>
cudaError_t launch_few_dim(const AttentionArgs& a, cudaStream_t st) {
    const bool bf16 = a.act == FP8W_BF16;
    if (a.cache->dtype == FP8W_E2M1) return bf16 ? launch_few<DP, true, kFormFp4, NT>(a, st) : launch_few<DP, false, kFormFp4, NT>(a, st);
    if (a.cache->dtype == FP8W_E4M3) return bf16 ? launch_few<DP, true, kFormE4m3, NT>(a, st) : launch_few<DP, false, kFormE4m3, NT>(a, st);
    return bf16 ? launch_few<DP, true, kForm16, NT>(a, st) : launch_few<DP, false, kForm16, NT>(a, st);
}

}  // namespace

// Tiles of 8 rows where no sequence has more, else of 16.
cudaError_t launch_attention_few(const AttentionArgs& a, cudaStream_t st) {
    const int64_t most_new = a.starts ? (a.max_new > 0 ? a.max_new : a.tokens) : 1;
    const bool one = most_new * (a.q_heads / a.cache->kv_heads) <= 8;
    if (a.cache->head_dim <= 64) return one ? launch_few_dim<64, 1>(a, st) : launch_few_dim<64, 2>(a, st);
    return one ? launch_few_dim<128, 1>(a, st) : launch_few_dim<128, 2>(a, st);
}

int read_attention_few_device_error() {
    int v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_attention_few_error, sizeof v) != cudaSuccess) return -1;
    if (v != 0 && cudaMemcpyToSymbol(g_attention_few_error, &zero, sizeof zero) != cudaSuccess) return -1;
    return v;
}

}  // namespace fp8w
