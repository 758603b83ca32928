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
//   warps 0-7, 8-15 softmax of pipe 0, 1: two threads a row, half its keys each
//   warps 16, 18, 19 (with codes 16, 18) TMA producers of key and value tiles
//   warp 17         MMA issue, one thread; owns TMEM
//   warps 20-23     (a cache of codes) codes -> 16-bit operand tiles
// What bounds it: 8192 new tokens, 32 query heads of 128, 16-slot pages take 387
// us, 1421 TFLOP/s, 74% of the measured rate (calls back to back for longer: 407
// us).  Per key tile of 256 rows the products need 2048 cycles of the 3100 it
// takes; without the softmax's work 2700, without products and work 1900: a pipe's
// scores, weights and products wait for one another, and every instruction of the
// one thread that issues and of the producers waits behind sixteen softmax warps,
// so these loops are kept short.  Heads of 64: 351 us, 41%: the softmax is the same
// for half the products.  Heads of 80 and 96 are computed as heads of 128: 382 and
// 384 us, 47% and 56%.
// Codes: 697 us for chunks of 500 to 1030 tokens over 9000 to 16000, 45%: the
// softmax multiplies both scales too, and the conversion shares its schedulers
// (bf16, whose conversion takes more instructions: 734); 17% is the last wave (352
// row tiles on 152 SMs).
// 4 bits (fp4.cuh): the converting warps fold the blocks' scales into the operands,
// exactly, 32 codes and two scales a 16-byte chunk.  The products are of fp16 for bf16
// activations too: the chunks 724 us (43%), 818 with products of bf16, whose codes take
// five instructions a pair instead of two; fp16 activations 710 (44%).
// Measured and not kept for the prompt: a pair of CTAs sharing products of 256
// rows (cta_group::2, half of each key and value tile a CTA): 537 us when one CTA
// took 455, each product waiting for both CTAs' softmax; scores of 64 keys at a
// time in four buffers: 664; a persistent grid: 520 to 540 when this took 543, and
// 52 instead of 39 for mixed lengths; two CTAs a tile's keys, joined: 782.
// The reference m moves only when a row's maximum has grown by more than
// 2^8 (kSlack) over it: then the row's O is rescaled, after the MMA that is
// adding to it.  p stays below 2^8 (fp16: all of them 2^kLiftF16 times as large),
// and the sums are fp32.
//
// e4m3 caches: codes convert exactly; the key scales multiply the columns of S
// and the value scales those of P, in fp32, so what is rounded to 16 bits is a
// weight times its value scale.  With fp16 weights that product has to stay among
// fp16's numbers whatever the scales are, so m is then the reference of p v_scale
// (the maximum is taken of exponents plus log2 v_scale), and the sum of the p
// alone, which is fp32, takes what stands against it.  bf16 has the range anyway.
//
// Long caches and few rows: the CTAs of a cluster take equal runs of key tiles
// and join their (m, sum, O) in distributed shared memory, in rank order.
//
// Every wait on an mbarrier is bounded; a CTA that gives up records a code, raises
// its abort flag, lets its copies and MMAs land and frees TMEM.  The named barriers
// of the softmax warps have no bound, so no warp passes one by: what a wait came to
// decides what is worked on and written next, never who takes part in a barrier (a
// warp that gave up takes part in those of its remaining tiles).
#include <mutex>
#include <type_traits>

#include "attention.cuh"
#include "fp4.cuh"

namespace fp8w {

__device__ int g_attention_error;

namespace {

constexpr int kKeys = 128;            // keys a tile
constexpr int kRows = 128;            // rows a tile (TMEM lanes)
constexpr int kMaxAttnCluster = 16;
// Up to this many rows a key head (new tokens x its query heads) the kernel for
// few rows reads the cache faster.  It takes 16 rows at a time: with more a 16-bit
// cache is read twice (a decode batch of 1.2 GB, 16 rows: 248 us against 254 here,
// 24: 380 against 255), a cache of codes twice or thrice is still less than here
// (24: 287 against 395; 48: 388 against 408; 64: 491 against 411).
constexpr int kFewRows = 16, kFewRowsCodes = 48;
constexpr uint32_t kAttnTmemCols = 512;
constexpr int kSoftmaxThreads = 512;   // sixteen warps
constexpr int kLoadWarp = 16, kMmaWarp = 17, kConvWarp = 20;
constexpr int kBarSoftmax = 1;        // named barrier of the softmax warps; 2..9: of the pairs that share rows

template <int DP, int kForm>
struct AttnSmem {
    static constexpr bool kFp8 = kForm != kForm16;               // codes
    static constexpr uint32_t kRawRow = kForm == kFormFp4 ? DP / 2 : DP;  // bytes of a key's or value's codes
    static constexpr uint32_t kSubs = DP / 64;                   // 64-value sub-tiles of a row (128 bytes)
    static constexpr uint32_t kTileBytes = kKeys * DP * 2;       // a 16-bit operand tile
    static constexpr uint32_t kRawBytes = kKeys * kRawRow;       // a tile of codes
    static constexpr int kStages = kFp8 ? (DP == 128 ? 3 : 6) : (DP == 128 ? 5 : 10);
    static constexpr int kRaw = kFp8 ? (DP == 128 ? 3 : 6) : 0;
    // Key tile m is converted once ring position 2 m - 1 - kStages is free.  With
    // 3 stages that is value tile m - 3, so the softmax is done with tile m - 3;
    // with 6 it is key tile m - 3, multiplied after value tile m - 5 was.
    static constexpr int kLoaders = kFp8 ? 2 : 3;                // warps that load: kLoadWarp and those after kMmaWarp
    static constexpr int kScaleSlots = DP == 128 ? 4 : 8;
    static constexpr int kScaleWords = 3 * kKeys + 64;           // of a slot (4 of the 64 are used)
    static constexpr uint32_t kQOff = 0;                         // two row tiles; later a 128 x DP fp32 partial
    static constexpr uint32_t kRingOff = 2 * kTileBytes;
    static constexpr uint32_t kRawOff = kRingOff + kStages * kTileBytes;
    static constexpr uint32_t kScaleOff = kRawOff + kRaw * kRawBytes;  // [slot][k, v, log2 v][128], each warp's largest log2 v [4], fp32
    static constexpr uint32_t kMlOff = kScaleOff + (kFp8 ? kScaleSlots * kScaleWords * 4 : 0);
    static constexpr uint32_t kJoinedOff = kMlOff + kRows * 8;   // (m, l) of the CTA's rows, for the cluster
    static constexpr uint32_t kBarOff = kJoinedOff + kRows * 8;
    // full, empty [kStages] | rawfull, rawempty [kRaw] | sfull, pfull, ofull [2] | qfull | joinfull, joinfree | drain | tail
    static constexpr uint32_t kNumBars = 2 * kStages + 2 * kRaw + 6 + 1 + 2 + 1 + 1;
    static constexpr uint32_t kMiscOff = kBarOff + kNumBars * 8;
    static constexpr uint32_t kTurnOff = kMiscOff + 16;          // (4 bits) factors of the two row tiles' queries
    static constexpr uint32_t kBytes = kTurnOff + (kForm == kFormFp4 ? 2 * kRows * 4 : 0);
    static_assert(kBytes <= 227 * 1024 && kMlOff % 1024 == 0, "shared memory");
    static constexpr int kThreads = kSoftmaxThreads + 128 + (kFp8 ? 128 : 0);
    // registers a thread at launch and after the split
    static constexpr int kRegs = 65536 / kThreads / 8 * 8;
    static constexpr int kRegsSoftmax = kFp8 ? 88 : 104;
    static constexpr int kRegsIssue = kFp8 ? 56 : 64;
    static constexpr int kRegsConv = 72;
    static_assert(kSoftmaxThreads * kRegsSoftmax + 128 * kRegsIssue + (kFp8 ? 128 * kRegsConv : 0) <= kThreads * kRegs, "register split");
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

// 32 consecutive columns of the thread's lane, with the wait in the same
// statement: registers named by a load that is still in flight may be copied
// by the compiler before a wait that stands apart.
__device__ __forceinline__ void tmem_ld_x32_sync(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]),
          "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
          "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
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

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// Products in a row, issued by one thread.  Sixteen a key tile have to be issued
// beside sixteen busy softmax warps, so descriptors advance by an add.
// D[tmem] = (or +=) sum of A[smem] B[smem] over the 64 values of a sub-tile, a
// 16-value step being 32 bytes.
__device__ __forceinline__ void mma_scores(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, t;\n\t.reg .b64 x, y;\n\t.reg .b32 u, v;\n\t"
        "setp.ne.b32 p, %5, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
        "mov.b64 x, {%1, %3};\n\tmov.b64 y, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p;\n\t"
        "add.u32 u, %1, 2;\n\tadd.u32 v, %2, 2;\n\tmov.b64 x, {u, %3};\n\tmov.b64 y, {v, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, t;\n\t"
        "add.u32 u, %1, 4;\n\tadd.u32 v, %2, 4;\n\tmov.b64 x, {u, %3};\n\tmov.b64 y, {v, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, t;\n\t"
        "add.u32 u, %1, 6;\n\tadd.u32 v, %2, 6;\n\tmov.b64 x, {u, %3};\n\tmov.b64 y, {v, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, t;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate ? 1u : 0u)
        : "memory");
}
// D[tmem] (+)= A[tmem] B[smem] over 128 keys: 8 columns of A and 16 key rows
// (2048 bytes) a step, the second 64 keys' columns 64 behind the first's.
__device__ __forceinline__ void mma_values(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t hi, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, t;\n\t.reg .b64 y;\n\t.reg .b32 u, v;\n\t"
        "setp.ne.b32 p, %5, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
        "mov.b64 y, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n\t"
        "add.u32 u, %1, 8;\n\tadd.u32 v, %2, 128;\n\tmov.b64 y, {v, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [u], y, %4, t;\n\t"
        "add.u32 u, %1, 16;\n\tadd.u32 v, %2, 256;\n\tmov.b64 y, {v, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [u], y, %4, t;\n\t"
        "add.u32 u, %1, 24;\n\tadd.u32 v, %2, 384;\n\tmov.b64 y, {v, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [u], y, %4, t;\n\t"
        "add.u32 u, %1, 64;\n\tadd.u32 v, %2, 512;\n\tmov.b64 y, {v, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [u], y, %4, t;\n\t"
        "add.u32 u, %1, 72;\n\tadd.u32 v, %2, 640;\n\tmov.b64 y, {v, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [u], y, %4, t;\n\t"
        "add.u32 u, %1, 80;\n\tadd.u32 v, %2, 768;\n\tmov.b64 y, {v, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [u], y, %4, t;\n\t"
        "add.u32 u, %1, 88;\n\tadd.u32 v, %2, 896;\n\tmov.b64 y, {v, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [u], y, %4, t;\n\t}" ::"r"(d),
        "r"(a), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate ? 1u : 0u)
        : "memory");
}

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
// Shared-memory accesses by address.  lds_f4 is free to move (its address
// says after what).
__device__ __forceinline__ float4 lds_f4(uint32_t addr) {
    float4 v;
    asm("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
    return v;
}
__device__ __forceinline__ float2 lds_f2(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void sts_f2(uint32_t addr, float x, float y) {
    asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(x), "f"(y) : "memory");
}
// x / group, for x < 2^15 + group (x * group < 2^32: the rounded-up reciprocal is exact).
__device__ __forceinline__ int by_group(const AttnParams& p, int x) { return static_cast<int>(__umulhi(static_cast<uint32_t>(x), p.group_inverse)) + (p.group == 1 ? x : 0); }
__device__ __forceinline__ void softmax_bar() { asm volatile("bar.sync %0, %1;" ::"n"(kBarSoftmax), "n"(kSoftmaxThreads) : "memory"); }

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

__device__ __forceinline__ bool find_work(const AttnParams& p, int tile, int head, int rank, Work& w, bool report) {
    SeqTile f;
    if (!find_tile(p, 2 * kRows, tile, report, &g_attention_error, f)) return false;
    w.seq = f.seq;
    w.head = head;
    w.token0 = f.begin;
    w.total_rows = static_cast<int>(f.count * p.group);
    w.row0 = f.inner * 2 * kRows;
    w.rows = w.total_rows - w.row0 < 2 * kRows ? w.total_rows - w.row0 : 2 * kRows;
    w.two = w.rows > kRows;
    w.pos0 = static_cast<int>(f.len - f.count);
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

// What a softmax thread takes to the join.
struct Join {
    uint32_t sbase, t_o, joinfull, joinfree;
    int rank, split, done;
    bool ok, valid;
    float m, l;
};

// The largest of a row's exponents plus log2 of the value scales, less m, over
// `width` columns of scores from taddr on (ksc: their first key scale; turn: the
// row's factor); top, bot: the last and first column that the row sees.  Out of line, for the loop over the
// tiles has no registers to spare for it (773 us for the chunks of codes that take
// 696 so).
template <bool kTurn>
__device__ __noinline__ float scaled_peak(uint32_t taddr, uint32_t ksc, int width, float less_m, float turn, bool masked, int top, int bot) {
    float mx = kNegInf, my = kNegInf;
    const uint64_t less_m2 = pack2(less_m, less_m), turn2 = pack2(turn, turn);
#pragma unroll 1
    for (int b = 0; b < width; b += 16) {
        uint32_t v[16];
        tmem_ld_x16_sync(taddr + b, v);
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            const float4 f = lds_f4(ksc + (b + i) * 4), g = lds_f4(ksc + (2 * kKeys + b + i) * 4);
            uint64_t x = fma2(pack2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), kTurn ? mul2(pack2(f.x, f.y), turn2) : pack2(f.x, f.y), less_m2);
            uint64_t y = fma2(pack2(__uint_as_float(v[i + 2]), __uint_as_float(v[i + 3])), kTurn ? mul2(pack2(f.z, f.w), turn2) : pack2(f.z, f.w), less_m2);
            x = add2(x, pack2(g.x, g.y));
            y = add2(y, pack2(g.z, g.w));
            auto seen = [&](int e, float z) { return masked && (b + i + e > top || b + i + e < bot) ? kNegInf : z; };
            mx = max3(mx, seen(0, lo2(x)), seen(1, hi2(x)));
            my = max3(my, seen(2, lo2(y)), seen(3, hi2(y)));
        }
    }
    return fmaxf(mx, my);
}

// Partial results through shared memory to the output: the pipes', the copies'
// and then the cluster's.  Rounds: one, or one for each row tile.  A function of
// its own: inlined, it took registers from the loop before it.  All softmax
// threads call it.
template <int DP, bool kBf16, int kForm>
__device__ __noinline__ void join_results(const AttnParams& p, const Work& w, const Join& a, volatile int* abort_flag) {
    using L = AttnSmem<DP, kForm>;
    const uint32_t sbase = a.sbase, t_o = a.t_o, joinfull = a.joinfull, joinfree = a.joinfree;
    const int rank = a.rank, tid = threadIdx.x, split = a.split, done = a.done, per_copy = kRows / split;
    constexpr int kHalf = DP / 2;          // output columns a thread
    const int lane = tid & 31, pipe = tid >> 8, half = (tid >> 7) & 1, r = tid & 127, cout = half * kHalf;
    const uint32_t pair = 2 + pipe * 4 + ((tid >> 5) & 3);
    const bool valid = a.valid;
    const float m = a.m, l = a.l;
    bool ok = a.ok;
    const bool busy = __any_sync(0xffffffffu, valid);
    const uint32_t ml = sbase + L::kMlOff, joined = sbase + L::kJoinedOff;
    // fp32 partials [128][DP] where Q was, 16-byte chunks swizzled by the row
    auto stage_at = [&](int row, int chunk) { return sbase + L::kQOff + static_cast<uint32_t>(row * DP + ((chunk ^ (row & 7)) << 2)) * 4u; };
    uint16_t* out = p.out + w.token0 * p.out_stride + static_cast<int64_t>(w.head * p.group) * p.head_dim;
    auto out_at = [&](int row) {
        const int t = row / p.group, g = row - t * p.group;
        return out + t * p.out_stride + g * p.head_dim;
    };
    const int64_t sees_from = -static_cast<int64_t>(w.pos0) * p.group - w.row0;  // the CTA's first row at position 0 or above
    auto sees = [&](int row) { return row >= sees_from; };
    const int rounds = w.two ? 2 : 1;
    softmax_bar();  // both pipes' products are complete: Q's place is free
    for (int round = 0; round < rounds; ++round) {
        const int rows = w.two ? (round == 0 ? kRows : w.rows - kRows) : w.rows;
        if (round > 0) {
            ok = ok && mbar_wait_cluster(joinfree, static_cast<uint32_t>((round - 1) & 1), abort_flag);
            ok = __all_sync(0xffffffffu, ok);
        }
        if (w.two ? pipe == round : pipe == 1) {
            if (valid && half == 0) sts_f2(ml + r * 8, m, done > 0 ? l : 0.0f);
            if (ok && busy && done > 0) {
#pragma unroll
                for (int b = 0; b < kHalf; b += 32) {
                    uint32_t o[32];
                    tmem_ld_x32_sync(t_o + b, o);
                    if (valid)
#pragma unroll
                        for (int i = 0; i < 32; i += 4) sts128(stage_at(r, (cout + b + i) / 4), o[i], o[i + 1], o[i + 2], o[i + 3]);
                }
            }
        }
        softmax_bar();
        if (!w.two) {
            const bool direct = split == 1 && p.cl == 1;
            if (pipe == 0 && busy) {
                // add pipe 1's partial to this one's
                const float2 other = valid ? lds_f2(ml + r * 8) : make_float2(0.0f, 0.0f);
                const float mine_l = done > 0 ? l : 0.0f;
                const float top = fmaxf(mine_l != 0.0f ? m : other.x, other.y != 0.0f ? other.x : m);
                const float a0 = mine_l != 0.0f ? ex2(m - top) : 0.0f;
                const float a1 = other.y != 0.0f ? ex2(other.x - top) : 0.0f;
                const float sum = a0 * mine_l + a1 * other.y;
                const float inv = weight_inverse(sum, sees(r));
                // both threads of the row have read its (m, l)
                asm volatile("bar.sync %0, 64;" ::"r"(pair) : "memory");
#pragma unroll
                for (int b = 0; b < kHalf; b += 32) {
                    uint32_t o[32];
                    if (done > 0) {
                        tmem_ld_x32_sync(t_o + b, o);
                    }
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        uint4 v = make_uint4(0u, 0u, 0u, 0u);
                        if (valid && a1 > 0.0f) v = lds128(stage_at(r, (cout + b + i) / 4));
                        const float x[4] = {__uint_as_float(v.x) * a1, __uint_as_float(v.y) * a1, __uint_as_float(v.z) * a1,
                                            __uint_as_float(v.w) * a1};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            o[i + e] = __float_as_uint(a0 > 0.0f ? fmaf(__uint_as_float(o[i + e]), a0, x[e]) : x[e]);
                    }
                    if (valid && direct && ok) {
                        uint16_t* dst = out_at(w.row0 + r);
#pragma unroll
                        for (int i = 0; i < 32; i += 8) {
                            if (cout + b + i >= p.head_dim) break;
                            uint32_t v[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                v[e] = pack16<kBf16>(__uint_as_float(o[i + 2 * e]) * inv, __uint_as_float(o[i + 2 * e + 1]) * inv);
                            *reinterpret_cast<uint4*>(dst + cout + b + i) = make_uint4(v[0], v[1], v[2], v[3]);
                        }
                    } else if (valid && !direct) {
#pragma unroll
                        for (int i = 0; i < 32; i += 4) sts128(stage_at(r, (cout + b + i) / 4), o[i], o[i + 1], o[i + 2], o[i + 3]);
                    }
                }
                if (valid && half == 0) sts_f2(ml + r * 8, top, sum);
            }
            if (direct) break;
            softmax_bar();
        }
        // the copies of a row into the first of them (its (m, l) apart: other
        // threads of the row still read the copies')
        const int units = rows * (DP / 4);
        for (int u = tid; u < units; u += kSoftmaxThreads) {
            const int row = u / (DP / 4), ch = u - row * (DP / 4);
            float2 q[4];
            float top = kNegInf, sum = 0.0f;
#pragma unroll
            for (int f = 0; f < 4; ++f) {
                q[f] = f < split ? lds_f2(ml + (f * per_copy + row) * 8) : make_float2(kNegInf, 0.0f);
                if (q[f].y != 0.0f) top = fmaxf(top, q[f].x);
            }
            float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int f = 0; f < 4; ++f) {
                if (q[f].y == 0.0f) continue;
                const uint4 v = lds128(stage_at(f * per_copy + row, ch));
                const float a = ex2(q[f].x - top);
                sum = fmaf(q[f].y, a, sum);
                acc[0] = fmaf(__uint_as_float(v.x), a, acc[0]);
                acc[1] = fmaf(__uint_as_float(v.y), a, acc[1]);
                acc[2] = fmaf(__uint_as_float(v.z), a, acc[2]);
                acc[3] = fmaf(__uint_as_float(v.w), a, acc[3]);
            }
            if (p.cl == 1) {
                const float inv = weight_inverse(sum, sees(round * kRows + row));
                if (ch * 4 < p.head_dim)
                    *reinterpret_cast<uint2*>(out_at(w.row0 + row) + ch * 4) =
                        make_uint2(pack16<kBf16>(acc[0] * inv, acc[1] * inv), pack16<kBf16>(acc[2] * inv, acc[3] * inv));
            } else {
                sts128(stage_at(row, ch), __float_as_uint(acc[0]), __float_as_uint(acc[1]), __float_as_uint(acc[2]),
                       __float_as_uint(acc[3]));
                if (ch == 0) sts_f2(joined + row * 8, top, sum);
            }
        }
        if (p.cl == 1) break;
        softmax_bar();
        if (tid < p.cl) mbar_arrive_remote(joinfull, static_cast<uint32_t>(tid));
        __syncwarp();
        bool all = mbar_wait_cluster(joinfull, static_cast<uint32_t>(round & 1), abort_flag);
        all = __all_sync(0xffffffffu, all);
        if (!all && lane == 0) attn_error(kErrWaitDequant, abort_flag);
        if (all) {
            // each rank finishes its share of the rows' 16-byte chunks; with
            // few of them several lanes share one, each reading some ranks'
            // partials (one remote read's time instead of a rank count's)
            const int share = (units + p.cl - 1) / p.cl;
            int lanes = p.cl;
            while (lanes > 1 && share * lanes > kSoftmaxThreads) lanes >>= 1;
            const int k0 = tid & (lanes - 1);
            for (int b = 0; b < share; b += kSoftmaxThreads / lanes) {
                const int i = b + tid / lanes, u = rank * share + i;
                const bool live = i < share && u < units;
                const int row = live ? u / (DP / 4) : 0, ch = live ? u - row * (DP / 4) : 0;
                const uint32_t ml_at = joined + row * 8, st_at = stage_at(row, ch);
                float top = kNegInf, sum = 0.0f;
                float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                for (int k = k0; k < p.cl; k += 4 * lanes) {
                    float2 q[4];
                    float4 v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t from_rank = static_cast<uint32_t>(k + e * lanes < p.cl ? k + e * lanes : k);
                        q[e] = ld_cluster_f2(mapa_shared(ml_at, from_rank));
                        v[e] = ld_cluster_f4(mapa_shared(st_at, from_rank));
                        if (k + e * lanes >= p.cl) q[e].y = 0.0f;
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (q[e].y == 0.0f) continue;
                        const float to = fmaxf(top, q[e].x);
                        const float x = ex2(top - to), y = ex2(q[e].x - to);
                        top = to;
                        sum = sum * x + q[e].y * y;
                        acc.x = acc.x * x + v[e].x * y;
                        acc.y = acc.y * x + v[e].y * y;
                        acc.z = acc.z * x + v[e].z * y;
                        acc.w = acc.w * x + v[e].w * y;
                    }
                }
                for (int d = lanes >> 1; d > 0; d >>= 1) {
                    const float o_top = __shfl_xor_sync(0xffffffffu, top, d), o_sum = __shfl_xor_sync(0xffffffffu, sum, d);
                    const float4 o = make_float4(__shfl_xor_sync(0xffffffffu, acc.x, d), __shfl_xor_sync(0xffffffffu, acc.y, d),
                                                 __shfl_xor_sync(0xffffffffu, acc.z, d), __shfl_xor_sync(0xffffffffu, acc.w, d));
                    const float to = fmaxf(top, o_top);
                    const float x = sum != 0.0f ? ex2(top - to) : 0.0f, y = o_sum != 0.0f ? ex2(o_top - to) : 0.0f;
                    top = to;
                    sum = sum * x + o_sum * y;
                    acc.x = acc.x * x + o.x * y;
                    acc.y = acc.y * x + o.y * y;
                    acc.z = acc.z * x + o.z * y;
                    acc.w = acc.w * x + o.w * y;
                }
                const float inv = weight_inverse(sum, sees(round * kRows + row));
                if (live && k0 == 0 && ch * 4 < p.head_dim)
                    *reinterpret_cast<uint2*>(out_at(w.row0 + round * kRows + row) + ch * 4) =
                        make_uint2(pack16<kBf16>(acc.x * inv, acc.y * inv), pack16<kBf16>(acc.z * inv, acc.w * inv));
            }
        }
        softmax_bar();
        if (tid < p.cl) mbar_arrive_remote(joinfree, static_cast<uint32_t>(tid));
        __syncwarp();
    }
}

}  // namespace

template <int DP, bool kBf16, int kForm>
__global__ void __launch_bounds__(AttnSmem<DP, kForm>::kThreads, 1)
    attention_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                     const __grid_constant__ AttnParams p) {
    using L = AttnSmem<DP, kForm>;
    constexpr bool kFp8 = L::kFp8, kFp4 = kForm == kFormFp4;  // codes; of 4 bits
    // With 4 bits the products are of fp16 whatever the activations' type: the codes
    // take two instructions a pair instead of five, and the weights round to 11 bits.
    // bf16 queries go over exactly but for a power of two a row.
    constexpr bool kTurn = kFp4 && kBf16, kMmaBf16 = kBf16 && !kFp4;
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
                   drain = bar0 + 8u * (kB + 9), tail = bar0 + 8u * (kB + 10);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMiscOff);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMiscOff + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr float kSlack = 8.0f, kLift = kMmaBf16 ? 0.0f : kLiftF16;
    constexpr bool kScaledF16 = kFp8 && !kMmaBf16;  // m is the reference of weight times value scale

    if (warp == kMmaWarp) {
        tmem_alloc(smem_u32(tmem_slot), kAttnTmemCols);
        tmem_relinquish();
    } else if (warp == kLoadWarp) {
        if (lane == 0) {
            for (int s = 0; s < kStages; ++s) {
                mbar_init(full(s), kFp8 ? 4 : L::kLoaders);  // the converting warps, or the producers
                mbar_init(empty(s), 1);  // MMA commit
            }
            for (int s = 0; s < kRaw; ++s) {
                mbar_init(rawfull(s), L::kLoaders);
                mbar_init(rawempty(s), 4);
            }
            for (int i = 0; i < 2; ++i) {
                mbar_init(sfull(i), 1);
                mbar_init(pfull(i), 8);  // the pipe's softmax warps
                mbar_init(ofull(i), 1);
            }
            mbar_init(qfull, kSoftmaxThreads / 32);
            mbar_init(joinfull, static_cast<uint32_t>(p.cl));
            mbar_init(joinfree, static_cast<uint32_t>(p.cl));
            mbar_init(drain, 1);
            mbar_init(tail, 1);
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
    // the same for all threads (not by the abort flag, which a warp may raise meanwhile)
    const bool have = !(sbase & 1023u) && find_work(p, tile, head, rank, w, blockIdx.x == 0 && warp == 0);
    if (!have) w = Work{};
    const int n = w.cnt;
    // Ring positions: K0 K1 V0 K2 V1 .. K(n-1) V(n-2) V(n-1).
    // Release e is of positions 2 e - 1 and 2 e: key tile e and value tile e - 1,
    // which one commit gives back; position i may be filled again after release
    // (i - kStages + 1) / 2.  Those who fill wait for each release in turn; the last
    // one lies less than kStages after the one that is waited for.

    if (warp >= kLoadWarp && warp < kLoadWarp + 4) {
        reg_down<L::kRegsIssue>();
        if (warp != kMmaWarp && warp < kLoadWarp + L::kLoaders + 1 && n > 0) {
            // ------------------------------------------------- producer --
            constexpr int kR = kFp8 ? kRaw : kStages;
            // A tile is up to 16 copies of a page's 64-value sub-tile (a page's codes),
            // one a lane, of three warps in turn: a warp alone issues them too slowly,
            // and each instruction here waits behind the softmax warps' (8192 tokens on
            // 16-slot pages: 543 us with one warp when two took 455; 434 with two when
            // three took 415).  Codes are half the copies: two warps, 707 us against 709.
            constexpr int kCopies = kFp8 ? 1 : static_cast<int>(L::kSubs);  // of a box
            const int loader = warp == kLoadWarp ? 0 : warp - kMmaWarp;
            const int box = p.page_size < kKeys ? p.page_size : kKeys;
            const int mine = lane * L::kLoaders + loader, sub = mine % kCopies, at = mine / kCopies * box;
            const bool lives = at < kKeys;
            const uint32_t bytes = static_cast<uint32_t>(__popc(__ballot_sync(0xffffffffu, lives)) * box) * (kFp8 ? L::kRawRow : 128);
            const uint32_t dst0 = sbase + (kFp8 ? L::kRawOff + at * L::kRawRow : L::kRingOff + sub * (kKeys * 128) + at * 128);
            const int32_t* row = p.table + static_cast<int64_t>(w.seq) * p.table_width;
            // A lane's table entry is read two key tiles before its use and checked
            // there, so the table is not waited for.  One past the cache (which reads as
            // zeros) stands for no page, and for positions that no row sees.
            const int none = static_cast<int>(p.num_pages), key0 = w.t0 * kKeys + at;
            auto wanted = [&](int j) {
                const int key = key0 + j * kKeys;
                return j < n && lives && key < w.end && key + box > w.first_key;
            };
            auto entry_of = [&](int j) { return wanted(j) ? row[(key0 + j * kKeys) >> p.log_page] : none; };
            auto page_of = [&](int j, int entry) {
                if (static_cast<uint32_t>(entry) < static_cast<uint32_t>(none)) return entry;
                if (wanted(j)) atomicCAS(&g_attention_error, 0, 7000 + kErrIndex);
                return none;
            };
            uint32_t s = 0, phase = 0;               // stage of the position, use of it
            uint32_t freed = 0, fs = 0, fphase = 0;  // releases waited for; the next one's barrier and phase
            int e0 = entry_of(0), e1 = entry_of(1), now = none, before = none;  // now: the newest key tile's page
            bool ok = true;
            int i = 0;
#pragma unroll 1
            for (; i < 2 * n; ++i) {  // one body: a small loop fetches its instructions faster
                const bool is_k = i == 0 || (i < 2 * n - 1 && (i & 1));
                const int j = (i + (is_k ? 1 : i == 2 * n - 1 ? -1 : -2)) / 2;
                if (is_k) {
                    before = now;
                    now = page_of(j, e0);
                    e0 = e1;
                    e1 = entry_of(j + 2);
                }
                if constexpr (kFp8) {
                    ok = mbar_wait_warp(rawempty(s), phase ^ 1u, abort_flag);
                } else if (i >= kStages && i + 1 >= kStages + 2 * static_cast<int>(freed)) {
                    ok = mbar_wait_warp(empty(fs), fphase, abort_flag);
                    ++freed;
                    if (++fs == kStages) fs = 0, fphase ^= 1u;
                }
                if (!ok) {
                    if (lane == 0) attn_error(kErrWaitSlot, abort_flag);
                    break;
                }
                const uint32_t bar = kFp8 ? rawfull(s) : full(s);
                if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
                if (lives)
                    tma_load_4d(dst0 + s * (kFp8 ? L::kRawBytes : L::kTileBytes), is_k ? &map_k : &map_v, sub * 64,
                                (key0 + j * kKeys) & (p.page_size - 1), w.head, is_k || j == n - 1 ? now : before, bar);
                __syncwarp();
                if (++s == kR) s = 0, phase ^= 1u;
            }
            // Slots past the sequence's end hold anything, a NaN perhaps, and
            // 0 * NaN is no zero: those rows of the last value tile are cleared
            // (pages past the end were never read; codes are cleared as they convert)
            const int keep = w.end - (w.t0 + n - 1) * kKeys;
            if (!kFp8 && ok && loader == 0 && keep < kKeys) {
                const int s = (2 * n - 1) % kStages;  // the stage filled last
                ok = mbar_wait_warp(full(s), static_cast<uint32_t>(((2 * n - 1) / kStages) & 1), abort_flag);
                if (ok) {
                    const uint32_t b = sbase + L::kRingOff + s * L::kTileBytes;
                    for (int u = keep * 8 + lane; u < kKeys * 8; u += 32) {
#pragma unroll
                        for (uint32_t v = 0; v < L::kSubs; ++v) sts128(b + v * (kKeys * 128) + u * 16, 0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(tail);
                } else if (lane == 0) {
                    attn_error(kErrWaitTma, abort_flag);
                }
            }
            if (!ok || *abort_flag) {
                // let the copies still in flight land before the CTA exits
                for (int c = i > kR ? i - kR : 0; c < i; ++c)
                    if (!mbar_wait_drain(kFp8 ? rawfull(c % kR) : full(c % kR), static_cast<uint32_t>((c / kR) & 1)))
                        atomicCAS(&g_attention_error, 0, 7000 + kErrWaitDrain);
            }
        } else if (warp == kMmaWarp && n > 0) {
            // ------------------------------------------------ MMA issue --
            // One thread, and no more instructions than it needs: it shares its
            // scheduler with four softmax warps, and the tensor cores wait for it
            // (8192 tokens: a whole warp that elects for each statement 447 us, this 434).
            if (elect_one()) {
                constexpr uint32_t idesc_s = idesc_f16(kMmaBf16, kKeys);
                constexpr uint32_t idesc_o = idesc_f16(kMmaBf16, DP) | kIdescBNMajor;
                const uint64_t qd = smem_desc_sw128_kmajor(sbase + L::kQOff), kd = smem_desc_sw128_kmajor(sbase + L::kRingOff),
                               vd = smem_desc_sw128_nmajor(sbase + L::kRingOff);
                const uint32_t q_lo = static_cast<uint32_t>(qd), k_lo = static_cast<uint32_t>(kd), v_lo = static_cast<uint32_t>(vd);
                const uint32_t k_hi = static_cast<uint32_t>(kd >> 32), v_hi = static_cast<uint32_t>(vd >> 32);
                bool ok = true;
                auto wait = [&](uint32_t bar, uint32_t parity, int code) {
                    ok = mbar_wait(bar, parity, abort_flag);
                    if (!ok) attn_error(code, abort_flag);
                    return ok;
                };
                auto qk = [&](int pipe, int qtile, uint32_t stage) {  // S_pipe = Q_qtile K^T
#pragma unroll
                    for (uint32_t u = 0; u < L::kSubs; ++u)
                        mma_scores(tmem + pipe * kKeys, q_lo + qtile * (L::kTileBytes >> 4) + u * (kRows * 128 >> 4),
                                   k_lo + stage * (L::kTileBytes >> 4) + u * (kKeys * 128 >> 4), k_hi, idesc_s, u > 0);
                    tc_commit(sfull(pipe));
                };
                auto pv = [&](int pipe, uint32_t done, uint32_t stage, bool last) {  // O_pipe (+)= P_pipe V, the pipe's product number `done`
                    if (!wait(pfull(pipe), done & 1, kErrWaitMma)) return false;
                    tc_fence_after();
                    mma_values(tmem + 2 * kKeys + pipe * DP, tmem + pipe * kKeys, v_lo + stage * (L::kTileBytes >> 4), v_hi, idesc_o,
                               done > 0);
                    if (last) tc_commit(ofull(pipe));
                    return true;
                };
                // the last value tile: a producer clears what lies past the end
                auto wait_tail = [&] { return kFp8 || w.end - (w.t0 + n - 1) * kKeys >= kKeys || wait(tail, 0, kErrWaitTma); };
                // ring stage and phase of position 2 j + 1, and of the one behind it
                uint32_t a = 1, a_ph = 0;
                auto behind = [&](uint32_t& stage, uint32_t& phase) { stage = a + 1 == kStages ? 0 : a + 1, phase = a_ph ^ (a + 1 == kStages); };
                auto advance = [&] {
                    a += 2;
                    if (a >= kStages) a -= kStages, a_ph ^= 1;
                };
                ok = wait(qfull, 0, kErrWaitDequant) && wait(full(0), 0, kErrWaitTma);
                if (ok) tc_fence_after();
                if (ok && w.two) {
                    if (w.cnt0 > 0) qk(0, 0, 0);
                    qk(1, 1, 0);
                    tc_commit(empty(0));
                    uint32_t free_at = 1;  // barrier of release j + 1
                    for (int j = 0; j < n; ++j, advance()) {
                        const bool last = j == n - 1;
                        uint32_t b, b_ph;
                        behind(b, b_ph);
                        if (last) b = a, b_ph = a_ph;  // no key tile between
                        if (!wait(full(b), b_ph, kErrWaitTma) || (last && !wait_tail())) break;
                        if (j < w.cnt0 && !pv(0, j, b, j == w.cnt0 - 1)) break;
                        if (!last) {
                            if (!wait(full(a), a_ph, kErrWaitTma)) break;
                            if (j + 1 < w.cnt0) qk(0, 0, a);
                        }
                        if (!pv(1, j, b, last)) break;
                        if (!last) {
                            qk(1, 1, a);
                            tc_commit(empty(free_at));
                            free_at = free_at + 1 == kStages ? 0 : free_at + 1;
                        }
                    }
                } else if (ok) {
                    qk(0, 0, 0);
                    tc_commit(empty(0));
                    if (n > 1 && wait(full(1), 0, kErrWaitTma)) qk(1, 0, 1);
                    uint32_t free_at = 1;
                    for (int j = 0; j < n && ok; ++j) {
                        const bool last = j == n - 1;
                        uint32_t b, b_ph;
                        behind(b, b_ph);
                        if (last) b = a, b_ph = a_ph;
                        if (!wait(full(b), b_ph, kErrWaitTma) || (last && !wait_tail())) break;
                        if (!pv(j & 1, j >> 1, b, j >= n - 2)) break;
                        tc_commit(empty(free_at));
                        free_at = free_at + 1 == kStages ? 0 : free_at + 1;
                        advance();
                        if (j + 2 < n) {
                            if (!wait(full(a), a_ph, kErrWaitTma)) break;
                            qk(j & 1, 0, a);
                        }
                    }
                }
                // every MMA issued above completes before TMEM is released
                tc_commit(drain);
                if (!mbar_wait_drain(drain, 0)) atomicCAS(&g_attention_error, 0, 7000 + kErrWaitDrain);
            }
            __syncwarp();
        }
    } else if (kFp8 && warp >= kConvWarp) {
        // --------------------------------------- codes to operand tiles --
        if constexpr (kFp8) {
            reg_down<L::kRegsConv>();
            // One key a thread.  (Two warpgroups, half a key a thread each: 769 us for the
            // chunks that take 720 so; the schedulers have no room for more.)
            constexpr int kChunks = L::kRawRow / 16;  // 16-byte chunks
            const int r = (warp & 3) * 32 + lane;  // key of the tile
            const uint32_t swz = static_cast<uint32_t>(r & 7);
            const int32_t* row = p.table + static_cast<int64_t>(w.seq) * p.table_width;
            auto live_at = [&](int j) {
                const int key = (w.t0 + j) * kKeys + r;
                return j < n && key < w.end && key >= w.first_key;
            };
            // Behind a tile's page stand its scales: the page is read two key tiles
            // ahead and the scales one, and neither is used before it is needed, so
            // neither is waited for.
            const int64_t head_scales = static_cast<int64_t>(w.head) * p.page_size;
            const int64_t page_scales = static_cast<int64_t>(p.kv_heads) * p.page_size;
            auto page_at = [&](int j) { return live_at(j) ? row[((w.t0 + j) * kKeys + r) >> p.log_page] : -1; };
            auto scales_at = [&](int j, int pg) {
                if (pg < 0 || pg >= p.num_pages) return make_float2(0.0f, 0.0f);
                const int64_t at = head_scales + pg * page_scales + (((w.t0 + j) * kKeys + r) & (p.page_size - 1));
                return make_float2(p.k_scales[at], p.v_scales[at]);
            };
            // Whether a value row is all zeros.  Its scale is 1 then, as if its values
            // reached 448, and a large score there would set the reference of the weights
            // of small values.  Its codes are looked at where they are, ahead of their
            // tile: rows of other values that have this very scale mostly end with the
            // first chunk (the chunks of codes with this scale in all slots: 812 us, else 697).
            auto zero_row = [&](int j) {
                const int pg = page_at(j), slot = ((w.t0 + j) * kKeys + r) & (p.page_size - 1);
                if (pg < 0 || pg >= p.num_pages) return true;
                const uint8_t* at = static_cast<const uint8_t*>(p.v) + pg * p.page_stride + w.head * p.head_stride + slot * p.token_stride;
                for (int u = 0; u < (kFp4 ? p.head_dim >> 1 : p.head_dim); u += 16) {
                    const uint4 y = *reinterpret_cast<const uint4*>(at + u);
                    if ((y.x | y.y | y.z | y.w) & (kFp4 ? 0x77777777u : 0x7F7F7F7Fu)) return false;
                }
                return true;
            };
            // 4 bits: the scales of a key's or value's blocks, two blocks a load, read
            // one ring position ahead.
            constexpr int kPairs = DP / 32;
            struct Blocks {
                uint32_t two[kFp4 ? kPairs : 1];
            };
            auto blocks_at = [&](bool of_k, int j, int pg) {
                Blocks b = {};
                if constexpr (kFp4) {
                    if (live_at(j) && pg >= 0 && pg < p.num_pages) {
                        const int64_t at = head_scales + pg * page_scales + (((w.t0 + j) * kKeys + r) & (p.page_size - 1));
                        const uint8_t* from = (of_k ? p.k_blocks : p.v_blocks) + at * (p.head_dim >> 4);
#pragma unroll
                        for (int u = 0; u < kPairs; ++u)
                            if (u * 32 < p.head_dim) b.two[u] = *reinterpret_cast<const uint16_t*>(from + 2 * u);
                    }
                }
                return b;
            };
            const int page0 = page_at(0);
            float2 next = scales_at(0, page0);
            int page = page_at(1);
            int next_page = -1, k_page = page0, v_page = -1;  // of the tile behind the newest key tile, of that, and of the one before
            Blocks ahead = blocks_at(true, 0, page0);
            uint32_t s = 0, phase = 0, d = 0;        // raw stage of the position, use of it, ring stage
            uint32_t freed = 0, fs = 0, fphase = 0;  // releases waited for; the next one's barrier and phase
            // One body for key and value tiles: two copies of it took 753 us where this takes 720.
#pragma unroll 1
            for (int i = 0; i < 2 * n; ++i) {
                const bool is_k = i == 0 || (i < 2 * n - 1 && (i & 1));
                const int j = i == 0 ? 0 : is_k ? (i + 1) / 2 : i == 2 * n - 1 ? n - 1 : (i - 2) / 2;
                const bool live = live_at(j);
                const float2 scale = next;
                if (is_k) {
                    if constexpr (kFp4) {
                        if (j > 0) v_page = k_page, k_page = next_page;
                        next_page = page;
                    }
                    next = scales_at(j + 1, page);
                    page = page_at(j + 2);
                }
                Blocks blocks = {};
                if constexpr (kFp4) {
                    // positions go K0 K1 V0 K2 V1 .. V(n-1): after a key tile (but the first)
                    // comes the value tile before it, after a value tile the next key tile
                    blocks = ahead;
                    if (i == 0 ? n > 1 : !is_k && j + 2 < n)
                        ahead = blocks_at(true, i == 0 ? 1 : j + 2, next_page);
                    else if (is_k && j > 0)
                        ahead = blocks_at(false, j - 1, v_page);
                    else if (i + 1 < 2 * n)
                        ahead = blocks_at(false, n - 1, k_page);
                }
                if (!mbar_wait_warp(rawfull(s), phase, abort_flag)) {
                    if (lane == 0) attn_error(kErrWaitTma, abort_flag);
                    break;
                }
                uint4 c[kChunks];
                const uint32_t src = sbase + L::kRawOff + s * L::kRawBytes + static_cast<uint32_t>(r) * L::kRawRow;
#pragma unroll
                for (uint32_t u = 0; u < kChunks; ++u) {
                    // 128-, 64- or 32-byte swizzle
                    c[u] = lds128(src + ((L::kRawRow == 128 ? u ^ swz : L::kRawRow == 64 ? u ^ (swz >> 1) : u ^ (swz >> 2)) << 4));
                }
                if (i >= kStages && i + 1 >= kStages + 2 * static_cast<int>(freed)) {
                    if (!mbar_wait_warp(empty(fs), fphase, abort_flag)) {
                        if (lane == 0) attn_error(kErrWaitMma, abort_flag);
                        break;
                    }
                    ++freed;
                    if (++fs == kStages) fs = 0, fphase ^= 1u;
                }
                const uint32_t dst = sbase + L::kRingOff + d * L::kTileBytes + static_cast<uint32_t>(r) * 128u;
#pragma unroll
                for (uint32_t u = 0; u < kChunks; ++u) {
                    const uint32_t w4[4] = {live ? c[u].x : 0u, live ? c[u].y : 0u, live ? c[u].z : 0u, live ? c[u].w : 0u};
                    if constexpr (kFp4) {  // 32 values: 16-byte chunks 4 u .. 4 u + 3 of the row
                        const uint32_t f = block_pair_f16(blocks.two[u]);
                        const uint32_t sub = dst + (u >> 1) * (kKeys * 128);
#pragma unroll
                        for (uint32_t e = 0; e < 4; ++e) {
                            uint32_t v[4];
                            fp4_operands<false>(w4[e], e < 2 ? both_lo(f) : both_hi(f), v);
                            sts128(sub + (((4 * u + e) & 7) ^ swz) * 16, v[0], v[1], v[2], v[3]);
                        }
                        continue;
                    }
                    uint32_t v[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if constexpr (kBf16)
                            e4m3x4_to_bf16x2(w4[e], v[2 * e], v[2 * e + 1]);
                        else
                            e4m3x4_to_f16x2(w4[e], v[2 * e], v[2 * e + 1]);
                    }
                    // 16 values: 16-byte chunks 2 u and 2 u + 1 of the row
                    const uint32_t sub = dst + (u >> 2) * (kKeys * 128);
                    sts128(sub + (((2 * u) & 7) ^ swz) * 16, v[0], v[1], v[2], v[3]);
                    sts128(sub + (((2 * u + 1) & 7) ^ swz) * 16, v[4], v[5], v[6], v[7]);
                }
                if (is_k) {  // the softmax needs both as soon as the tile's scores are there
                    float* sc = reinterpret_cast<float*>(smem + L::kScaleOff) + (j % L::kScaleSlots) * L::kScaleWords + r;
                    sc[0] = scale.x * p.c;
                    if constexpr (kScaledF16) {
                        const float vs = scale.y == 1.0f && zero_row(j) ? 0.0f : scale.y;
                        sc[kKeys] = vs;
                        const float log2_vs = log2_scale(vs);  // above -128: the sum's bits are in its order
                        sc[2 * kKeys] = log2_vs;
                        const int top = __reduce_max_sync(0xffffffffu, __float_as_int(log2_vs + 128.0f));
                        if (lane == 0) sc[3 * kKeys - r + (warp & 3)] = __int_as_float(top) - 128.0f;
                    } else {
                        sc[kKeys] = scale.y;
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(full(d));
                    // behind the stores of what was read from the slot: sooner gained no time
                    mbar_arrive(rawempty(s));
                }
                if (++s == kRaw) s = 0, phase ^= 1u;
                if (++d == kStages) d = 0;
            }
        }
    } else {
        // ------------------------------------------------------ softmax --
        reg_up<L::kRegsSoftmax>();
        const int pipe = warp >> 3, half = (warp >> 2) & 1, quarter = warp & 3;
        const int tid = threadIdx.x;                    // 0..511
        const int r = quarter * 32 + lane;              // TMEM lane
        const int qtile = w.two ? pipe : 0;
        // Few rows: copies of them in the lanes' halves or quarters, each copy's
        // threads on its own part of the keys (its P is zero elsewhere), so all
        // warps share a tile's softmax.  The copies' results are joined.
        const int split = w.two ? 1 : w.rows <= kRows / 4 ? 4 : w.rows <= kRows / 2 ? 2 : 1;
        const int per_copy = kRows / split;
        const int copy = r / per_copy, rr = r - copy * per_copy;
        const int width = kKeys / 2 / split;            // keys of a tile for this thread
        const int cbeg = (copy * 2 + half) * width;     // the first of them
        // Q rows, 16 bytes a step, eight steps' reads in flight
        if (n > 0) {
            constexpr int kChunks = DP / 8, kLines = kSoftmaxThreads / kChunks;
            const int ch = tid % kChunks, lines = w.rows * split;
            const bool inside = ch * 8 < p.head_dim;
            const int token = w.row0 / p.group, over = w.row0 - token * p.group;
            const uint16_t* q_head = p.q + (w.token0 + token) * p.q_stride + static_cast<int64_t>(w.head * p.group) * p.head_dim + ch * 8;
            for (int line0 = tid / kChunks; line0 < lines; line0 += 8 * kLines) {
                uint4 v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int line = line0 + i * kLines;
                    v[i] = make_uint4(0u, 0u, 0u, 0u);
                    if (line < lines && inside) {
                        const int row = over + (split > 1 ? line % w.rows : line), t = by_group(p, row), g = row - t * p.group;
                        v[i] = *reinterpret_cast<const uint4*>(q_head + t * p.q_stride + g * p.head_dim);
                    }
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int line = line0 + i * kLines;
                    if (line >= lines) break;
                    const int f = split > 1 ? line / w.rows : 0, at = f * per_copy + line - f * w.rows;  // row of the two tiles
                    const uint32_t a = sbase + L::kQOff + (at >> 7) * L::kTileBytes + (ch >> 3) * (kRows * 128) +
                                       (at & 127) * 128 + (((ch & 7) ^ (at & 7)) << 4);
                    if constexpr (kTurn) {
                        // the row's largest value to [2^14, 2^15): what falls below fp16's
                        // normal numbers then is less than 2^-28 of it, off by 2^-39 of it
                        uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w}, top = 0u;
#pragma unroll
                        for (int e = 0; e < 4; ++e) top = max(top, max(u[e] & 0x7FFFu, (u[e] >> 16) & 0x7FFFu));
                        // (the lanes of a row are here together)
                        const unsigned lanes = static_cast<unsigned>((1ull << kChunks) - 1) << (lane & (32 - kChunks));
#pragma unroll
                        for (int d = 1; d < kChunks; d <<= 1) top = max(top, __shfl_xor_sync(lanes, top, d));
                        const int up = min(max(127 + 14 - (static_cast<int>(top >> 7) - 127), 1), 253);
                        const float factor = __int_as_float(up << 23);
#pragma unroll
                        for (int e = 0; e < 4; ++e) u[e] = pack16<false>(bf16_lo_to_f32(u[e]) * factor, bf16_hi_to_f32(u[e]) * factor);
                        v[i] = make_uint4(u[0], u[1], u[2], u[3]);
                        if (ch == 0) reinterpret_cast<float*>(smem + L::kTurnOff)[at] = __int_as_float((254 - up) << 23);
                    }
                    sts128(a, v[i].x, v[i].y, v[i].z, v[i].w);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(qfull);
            if constexpr (kTurn) softmax_bar();  // the rows' factors are there
        }
        const int R = w.row0 + qtile * kRows + rr;
        const bool valid = qtile * kRows + rr < w.rows;
        const int pos = w.pos0 + R / p.group;
        const int hi = valid ? pos : -1;                                     // last position seen
        const int64_t from = p.window > 0 ? static_cast<int64_t>(pos) - p.window + 1 : 0;
        const int lo = from > 0 ? static_cast<int>(from) : 0;                // first
        const bool busy = __any_sync(0xffffffffu, valid);
        const int warp_hi = __reduce_min_sync(0xffffffffu, valid ? hi : 0x7fffffff);
        const int warp_lo = __reduce_max_sync(0xffffffffu, valid ? lo : 0);
        const uint32_t tq = static_cast<uint32_t>(quarter * 32) << 16;
        const uint32_t t_s = tmem + tq + pipe * kKeys, t_o = tmem + tq + 2 * kKeys + pipe * DP + half * (DP / 2);
        const float c = p.c;
        const uint64_t c2 = pack2(c, c);
        // what the row's scores are multiplied by beside the keys' scales
        const float turn = kTurn && n > 0 && valid ? reinterpret_cast<const float*>(smem + L::kTurnOff)[qtile * kRows + r] : 1.0f;
        const uint64_t turn2 = pack2(turn, turn);
        float m = kNegInf, l = 0.0f;  // the row's reference, in exponents of two and less kLift, and its sum
        int done = 0;                 // tiles of this pipe
        bool ok = true;

        // One tile for this thread's row and W keys from cbeg: P over S, m, l and,
        // where m moved, its half of O.  The row's other thread has the same m.
        const uint32_t pair = 2 + pipe * 4 + quarter;   // the pair's barrier
        const uint32_t mine = sbase + L::kMlOff + ((pipe * 2 + half) * kRows + r) * 4;
        auto softmax_tile = [&](auto w_tag, int j) {
            constexpr int W = decltype(w_tag)::value;
            // columns a load: 16 leave registers where the head is wide (8192 tokens 380
            // us against 387; codes 695 against 688, heads of 64 no difference)
            constexpr int kStep = W < 32 ? W : !kFp8 && DP == 128 ? 16 : 32;
            const int key0 = (w.t0 + j) * kKeys + cbeg;
            const bool masked = key0 + W - 1 > warp_hi || key0 < warp_lo;
            // address taken after the wait, so the reads below stay behind it
            uint32_t ksc = sbase + L::kScaleOff + (j % L::kScaleSlots) * (L::kScaleWords * 4) + cbeg * 4;
            asm volatile("" : "+r"(ksc)::"memory");
            // kStep exponents from the b-th on: scores times c (with codes, times key
            // scales that hold it) less m, masked
            auto exponents = [&](int b, uint64_t less_m, uint32_t (&v)[kStep]) {
                if constexpr (kStep == 16)
                    tmem_ld_x16_sync(t_s + cbeg + b, v);
                else
                    tmem_ld_x32_sync(t_s + cbeg + b, v);
#pragma unroll
                for (int i = 0; i < kStep; i += 4) {
                    uint64_t x = pack2(__uint_as_float(v[i]), __uint_as_float(v[i + 1]));
                    uint64_t y = pack2(__uint_as_float(v[i + 2]), __uint_as_float(v[i + 3]));
                    if constexpr (kFp8) {
                        const float4 f = lds_f4(ksc + (b + i) * 4);
                        uint64_t f0 = pack2(f.x, f.y), f1 = pack2(f.z, f.w);
                        if constexpr (kTurn) f0 = mul2(f0, turn2), f1 = mul2(f1, turn2);
                        x = fma2(x, f0, less_m);
                        y = fma2(y, f1, less_m);
                    } else {
                        x = fma2(x, c2, less_m);
                        y = fma2(y, c2, less_m);
                    }
                    v[i] = static_cast<uint32_t>(x), v[i + 1] = static_cast<uint32_t>(x >> 32);
                    v[i + 2] = static_cast<uint32_t>(y), v[i + 3] = static_cast<uint32_t>(y >> 32);
                }
                if (masked) {
                    const int top = hi - key0 - b, bot = lo - key0 - b;
#pragma unroll
                    for (int i = 0; i < kStep; ++i)
                        if (i > top || i < bot) v[i] = 0xff800000u;
                }
            };
            // m of the larger of both threads' maxima
            auto exchange = [&](float x) {
                asm volatile("st.shared.f32 [%0], %1;" ::"r"(mine), "f"(x) : "memory");
                asm volatile("bar.sync %0, 64;" ::"r"(pair) : "memory");
                float other;
                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(other) : "r"(mine ^ (kRows * 4)) : "memory");
                return fmaxf(x, other);
            };
            float mx = kNegInf, my = kNegInf;
            // The maximum of what m is the reference of, less m.
            auto peak = [&](float less) {
                if constexpr (kScaledF16) return scaled_peak<kTurn>(t_s + cbeg, ksc, W, less, turn, masked, hi - key0, lo - key0);
                const uint64_t less2 = pack2(less, less);
#pragma unroll 1
                for (int b = 0; b < W; b += kStep) {
                    uint32_t v[kStep];
                    exponents(b, less2, v);
#pragma unroll
                    for (int i = 0; i < kStep; i += 4) {
                        mx = max3(mx, __uint_as_float(v[i]), __uint_as_float(v[i + 1]));
                        my = max3(my, __uint_as_float(v[i + 2]), __uint_as_float(v[i + 3]));
                    }
                }
                return fmaxf(mx, my);
            };
            if (done == 0) m = exchange(peak(0.0f)) - kLift;  // the first tile's maximum is the first m
            uint32_t o[W / 2];
            uint64_t l0, l1;
            // The weights are taken with the m of the tiles before, without waiting
            // for this one's maximum.  Where that turns out to lie too far above, m
            // moves and they are taken again; both threads of a row have the same m.
            // With kScaledF16 the largest exponent and the tile's largest scale bound what
            // m is the reference of; its own maximum, which reads log2 of each scale, is
            // looked for where that bound lies above only (in every tile: 766 us for the
            // chunks of codes that take 696 so).
            auto weights = [&] {
                const float mc = m == kNegInf ? 0.0f : -m;  // while nothing was seen, exponents are not reduced
                const uint64_t mc2 = pack2(mc, mc);
                mx = my = kNegInf;
                l0 = l1 = 0ull;
#pragma unroll
                for (int b = 0; b < W; b += kStep) {
                    uint32_t v[kStep];
                    exponents(b, mc2, v);
#pragma unroll
                    for (int i = 0; i < kStep; i += 4) {
                        mx = max3(mx, __uint_as_float(v[i]), __uint_as_float(v[i + 1]));
                        my = max3(my, __uint_as_float(v[i + 2]), __uint_as_float(v[i + 3]));
                        uint64_t x = pack2(__uint_as_float(v[i]), __uint_as_float(v[i + 1]));
                        uint64_t y = pack2(__uint_as_float(v[i + 2]), __uint_as_float(v[i + 3]));
                        x = pack2(ex2(lo2(x)), ex2(hi2(x)));
                        y = pack2(ex2(lo2(y)), ex2(hi2(y)));
                        l0 = add2(l0, x);
                        l1 = add2(l1, y);
                        if constexpr (kFp8) {
                            const float4 f = lds_f4(ksc + (kKeys + b + i) * 4);
                            x = mul2(x, pack2(f.x, f.y));
                            y = mul2(y, pack2(f.z, f.w));
                        }
                        o[(b + i) / 2] = pack16<kMmaBf16>(lo2(x), hi2(x));
                        o[(b + i) / 2 + 1] = pack16<kMmaBf16>(lo2(y), hi2(y));
                    }
                    if constexpr (kFp8) asm volatile("" : "+r"(ksc));  // scales of one part at a time
                }
                mx = fmaxf(mx, my);
            };
            auto store = [&] {
                if constexpr (W == 64) {
                    tmem_st_x16(t_s + cbeg, o);
                    tmem_st_x16(t_s + cbeg + 16, o + 16);
                } else {
#pragma unroll
                    for (int f = 0; f < kKeys / 2 / W; ++f) {  // zero in the other copies' keys
                        uint32_t v[W / 2];
#pragma unroll
                        for (int i = 0; i < W / 2; ++i) v[i] = f == copy ? o[i] : 0u;
                        const int key = (f * 2 + half) * W, col = key / 2 + (key >= kKeys / 2 ? kKeys / 4 : 0);
                        if constexpr (W == 32)
                            tmem_st_x16(t_s + col, v);
                        else
                            tmem_st_x8(t_s + col, v);
                    }
                }
            };
            // No thread writes P before the other of its row knows whether m moves: with
            // 64 keys its own scores go under it, with fewer those of others too.
            // (Storing them before the vote, to be scaled by a power of two if m moves:
            // 398 us for the 8192 tokens that take 382 so, the registers run short.)
            weights();
            tc_fence_before();
            if constexpr (kScaledF16) {
                const float4 f = lds_f4(ksc + (3 * kKeys - cbeg) * 4);
                mx += max3(fmaxf(f.x, f.y), f.z, f.w);
            }
            const bool moves = bar_red_or(pair, 64, valid && mx > (m == kNegInf ? kNegInf : kSlack + kLift));
            tc_fence_after();
            if (moves) {
                if constexpr (kScaledF16) mx = peak(m == kNegInf ? 0.0f : -m);
                const float top = exchange(mx) + (m == kNegInf ? 0.0f : m) - kLift;
                float alpha = 1.0f;
                if (valid && top - m > kSlack) {  // -inf - -inf: no
                    alpha = ex2(m - top);  // 0 while nothing was seen
                    m = top;
                    l *= alpha;
                }
                weights();
                if constexpr (W < 64) asm volatile("bar.sync %0, 64;" ::"r"(pair) : "memory");
                // O is at rest: the product of the tile before was issued before
                // these scores, whose commit stands for it too
                if (done > 0) {
#pragma unroll 1
                    for (int b = 0; b < DP / 2; b += 16) {
                        uint32_t v[16];
                        tmem_ld_x16_sync(t_o + b, v);
#pragma unroll
                        for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * alpha);
                        tmem_st_x16(t_o + b, v);
                    }
                }
            }
            store();
            l0 = add2(l0, l1);
            l += lo2(l0) + hi2(l0);
            tmem_wait_st();
            tc_fence_before();
        };

        const int step = w.two ? 1 : 2, jn = w.two && pipe == 0 ? w.cnt0 : n;
        // A pipe without a tile (none of its rows sees a key) waits for no product, and
        // the results go where the other warps may still be putting queries.
        if (jn == 0 && n > 0 && !mbar_wait_warp(qfull, 0, abort_flag) && lane == 0) attn_error(kErrWaitDequant, abort_flag);
        int j = w.two ? 0 : pipe;
        for (; j < jn; j += step, ++done) {
            if (!mbar_wait_warp(sfull(pipe), static_cast<uint32_t>(done & 1), abort_flag)) {
                if (lane == 0) attn_error(kErrWaitMma, abort_flag);
                ok = false;
                break;
            }
            tc_fence_after();
            if (busy) {
                if (split == 4)
                    softmax_tile(std::integral_constant<int, 16>{}, j);
                else if (split == 2)
                    softmax_tile(std::integral_constant<int, 32>{}, j);
                else
                    softmax_tile(std::integral_constant<int, 64>{}, j);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(pfull(pipe));
        }
        // The tiles of a warp that gave up: softmax_tile's barriers, for the row's other
        // warp may still take them.  (Going on in the loop above without its waits: 418 us
        // for the 8192 tokens that take 406 so.)
        for (; j < jn && busy; j += step, ++done) {
            if (done == 0) asm volatile("bar.sync %0, 64;" ::"r"(pair) : "memory");
            if (bar_red_or(pair, 64, false)) {
                asm volatile("bar.sync %0, 64;" ::"r"(pair) : "memory");
                if (split > 1) asm volatile("bar.sync %0, 64;" ::"r"(pair) : "memory");
            }
        }
        // --------------------------------------------------- the result --
        if (ok && done > 0) {
            ok = mbar_wait_warp(ofull(pipe), 0, abort_flag);
            if (!ok && lane == 0) attn_error(kErrWaitMma, abort_flag);
            tc_fence_after();
        }
        if (busy) {  // the row's sum: both threads'
            asm volatile("bar.sync %0, 64;" ::"r"(pair) : "memory");  // the last exchange above has been read
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(mine), "f"(l) : "memory");
            asm volatile("bar.sync %0, 64;" ::"r"(pair) : "memory");
            float other;
            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(other) : "r"(mine ^ (kRows * 4)) : "memory");
            l += other;
        }
        if (w.two && p.cl == 1) {
            if (ok && busy) {
                // Each warp through its own rows of this pipe's Q tile, which no product
                // reads any more (half a row a warp): 16-byte chunks swizzled by the row,
                // then 16 bytes a lane along the rows to memory.
                constexpr int kHalf = DP / 2, kChunks = kHalf / 8, kRowsAtOnce = 32 / kChunks;
                const float inv = weight_inverse(l, hi >= 0);
                const uint32_t mine = sbase + L::kQOff + pipe * L::kTileBytes + (half * 4 + quarter) * (32 * kHalf * 2);
#pragma unroll
                for (int b = 0; b < kHalf; b += 32) {
                    uint32_t o[32];
                    if (done > 0) {
                        tmem_ld_x32_sync(t_o + b, o);
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = 0u;
                    }
#pragma unroll
                    for (int i = 0; i < 32; i += 8) {
                        uint32_t v[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            v[e] = pack16<kBf16>(__uint_as_float(o[i + 2 * e]) * inv, __uint_as_float(o[i + 2 * e + 1]) * inv);
                        sts128(mine + lane * (kHalf * 2) + ((((b + i) / 8) ^ (lane & (kChunks - 1))) << 4), v[0], v[1], v[2], v[3]);
                    }
                }
                __syncwarp();
                const int row0 = w.row0 + qtile * kRows + quarter * 32, token = row0 / p.group, over = row0 - token * p.group;
                const int left = w.rows - qtile * kRows - quarter * 32, ch = lane % kChunks, col = half * kHalf + ch * 8;
                uint16_t* out = p.out + (w.token0 + token) * p.out_stride + static_cast<int64_t>(w.head * p.group) * p.head_dim + col;
                if (col < p.head_dim) {
#pragma unroll 4
                    for (int i = lane / kChunks; i < 32; i += kRowsAtOnce) {
                        if (i >= left) break;
                        const uint4 v = lds128(mine + i * (kHalf * 2) + ((ch ^ (i & (kChunks - 1))) << 4));
                        const int t = by_group(p, over + i), g = over + i - t * p.group;
                        *reinterpret_cast<uint4*>(out + t * p.out_stride + g * p.head_dim) = v;
                    }
                }
            }
        } else if (have) {
            Join j;
            j.sbase = sbase;
            j.t_o = t_o;
            j.joinfull = joinfull;
            j.joinfree = joinfree;
            j.rank = rank;
            j.split = split;
            j.done = done;
            j.ok = ok;
            j.valid = valid;
            j.m = m;
            j.l = l;
            join_results<DP, kBf16, kForm>(p, w, j, abort_flag);
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

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_tiled() {
    static std::once_flag once;
    static EncodeTiledFn fn = nullptr;
    std::call_once(once, [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(f);
    });
    return fn;
}

// Tensor map over one half of a paged cache: (value, slot, head, page), boxes of
// box_inner values (4 bits: bytes) x box_slots slots, 128-byte swizzle (64 or 32 for
// boxes of so many bytes).
bool encode_pages(CUtensorMap* map, const fp8w_kv_cache& c, const void* base, uint32_t box_inner, uint32_t box_slots) {
    EncodeTiledFn fn = encode_tiled();
    if (!fn) return false;
    const bool codes = c.dtype == FP8W_E4M3 || c.dtype == FP8W_E2M1;
    const cuuint64_t es = codes ? 1 : 2;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c.dtype == FP8W_E2M1 ? c.head_dim / 2 : c.head_dim), static_cast<cuuint64_t>(c.page_size),
                                static_cast<cuuint64_t>(c.kv_heads), static_cast<cuuint64_t>(c.num_pages)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(c.token_stride) * es, static_cast<cuuint64_t>(c.head_stride) * es,
                                   static_cast<cuuint64_t>(c.page_stride) * es};
    const cuuint32_t box[4] = {box_inner, box_slots, 1, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(map, codes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, const_cast<void*>(base), dims,
              strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              box_inner * es == 32   ? CU_TENSOR_MAP_SWIZZLE_32B
              : box_inner * es == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                     : CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DP, bool kBf16, int kForm>
cudaError_t launch_attn(const AttentionArgs& a, cudaStream_t st) {
    using L = AttnSmem<DP, kForm>;
    auto kern = attention_kernel<DP, kBf16, kForm>;
    static DeviceSetup setup;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    int sms = 0;
    e = device_sm_count(sms);
    if (e != cudaSuccess) return e;
    e = setup(dev, [&] {
        const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes);
        return err != cudaSuccess ? err : cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    });
    if (e != cudaSuccess) return e;

    const fp8w_kv_cache& c = *a.cache;
    const int group = a.q_heads / c.kv_heads;
    CUtensorMap map_k, map_v;
    const uint32_t box = static_cast<uint32_t>(c.page_size < kKeys ? c.page_size : kKeys);
    constexpr uint32_t kInner = L::kFp8 ? L::kRawRow : 64;
    if (!encode_pages(&map_k, c, c.k, kInner, box) || !encode_pages(&map_v, c, c.v, kInner, box))
        return cudaErrorInvalidValue;

    const int64_t tiles = attention_row_tiles(a, group, 2 * kRows), items = tiles * c.kv_heads;
    // CTAs a cluster: as many as fill the GPU, while each has two key tiles at least
    const int64_t key_tiles = (attention_longest(a) + kKeys - 1) / kKeys;
    int cl = 1;
    while (cl < kMaxAttnCluster && items * cl * 2 <= sms && key_tiles >= cl * 4) cl *= 2;
    if (items * cl > 0x7fffffffll) return cudaErrorInvalidConfiguration;

    AttnParams p = attention_params(a);
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
    if (a.cache->dtype == FP8W_E2M1)
        return bf16 ? launch_attn<DP, true, kFormFp4>(a, st) : launch_attn<DP, false, kFormFp4>(a, st);
    if (a.cache->dtype == FP8W_E4M3)
        return bf16 ? launch_attn<DP, true, kFormE4m3>(a, st) : launch_attn<DP, false, kFormE4m3>(a, st);
    return bf16 ? launch_attn<DP, true, kForm16>(a, st) : launch_attn<DP, false, kForm16>(a, st);
}

}  // namespace

cudaError_t launch_attention(const AttentionArgs& a, cudaStream_t st) {
    const int64_t most_new = a.starts ? (a.max_new > 0 ? a.max_new : a.tokens) : 1;
    if (most_new * (a.q_heads / a.cache->kv_heads) <= (a.cache->dtype == FP8W_E4M3 || a.cache->dtype == FP8W_E2M1 ? kFewRowsCodes : kFewRows))
        return launch_attention_few(a, st);
    return a.cache->head_dim <= 64 ? launch_dim<64>(a, st) : launch_dim<128>(a, st);
}

int read_attention_device_error() {
    int v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_attention_error, sizeof v) != cudaSuccess) return -1;
    if (v != 0 && cudaMemcpyToSymbol(g_attention_error, &zero, sizeof zero) != cudaSuccess) return -1;
    const int few = read_attention_few_device_error();
    return v ? v : few;
}

}  // namespace fp8w
