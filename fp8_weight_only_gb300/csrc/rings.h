// rings.h -- the rings between the roles of the tensor-core kernels K3 (skinny.cu)
// and K4 (prefill.cu): their depths, and who takes which slot and barrier.  Plain
// C++, so that tests/test_rings.py runs a model of the barriers on these same
// numbers and functions.
//
// A wait on an mbarrier asks for the parity of a phase, one bit: it tells "use u of
// this slot is over" from "use u is still going on", but takes "use u - 1 is not over
// yet" for "use u is over".  So whoever waits for use u has to know already that use
// u - 1 was over, from its own wait for it: each barrier is waited on, use after use,
// by the same warps.
#pragma once

#ifdef __CUDACC__
#define FP8W_HD __host__ __device__ __forceinline__
#else
#define FP8W_HD inline
#endif

namespace fp8w {

// K4, tiles of BN tokens: stages of codes, of dequantised weights and of activations.
template <int BN>
struct PrefillRings {
    static constexpr int kPCS = BN == 128 ? 6 : 4;  // code stages (16 KB)
    static constexpr int kPAS = 4;                  // dequantised A stages (16 KB)
    static constexpr int kPXS = BN == 128 ? 4 : 3;  // x stages (BN x 64 x 2 B)
};

// K4's 4-bit form: so many warpgroups, each taking one of the four k-blocks of a code
// stage.
constexpr int kPFp4Groups = 4;
// Which of a stage's four a warpgroup takes in a tile before which the CTA has had
// `before` k-blocks: the one that goes to its own A stage, (before + j) % 4 == group,
// so that it waits for each use of that stage.  (Part `group` in every tile is another
// stage in the next tile where a tile's k-blocks are no multiple of four.)
FP8W_HD int prefill_fp4_part(int group, long long before) {
    return static_cast<int>((group - before) & (kPFp4Groups - 1));
}

// K3, launches of NT tokens.  Three warpgroups dequantise the units in turn, two MMA
// warps issue them in turn.
template <int NT, bool kFp4>
struct SkinnyRings {
    static constexpr int kLanes = 3;                                         // dequantising warpgroups
    static constexpr int kMmaWarps = 2;
    static constexpr int kASlots = kFp4 ? 1 : 2;                             // TMEM A slots a warpgroup
    static constexpr int kASlotsAll = kLanes * kASlots;                      // unit u: slot u % kASlotsAll
    // aready barriers, unit u's the one u % kReady.  As many as take both the warpgroups
    // and the MMA warps round, so that one MMA warp waits for all uses of a barrier,
    // whatever the number of slots.
    static constexpr int kReady = kLanes * kMmaWarps;
    // per warpgroup: freed as soon as read (9 tiles in flight per SM: deeper
    // rings on every SM make the HBM stream slower, not faster)
    static constexpr int kCodeSlots = NT <= 32 ? 3 : 2;
    static constexpr int kXSlots = (NT == 16 ? 12 : 8) / (kFp4 ? 2 : 1);     // activation ring (freed when the unit's MMAs are done)
    // accumulator buffers per MMA warp: two (the epilogue drains one tile
    // while the next accumulates) where TMEM has room, one for 64 tokens
    static constexpr int kDBuf = NT <= 32 ? 2 : 1;
    static constexpr int kDoneSlots = NT == 16 ? 12 : 24;
    static_assert(kReady % kMmaWarps == 0 && kXSlots % kMmaWarps == 0, "one MMA warp waits for all uses of a barrier");
    static_assert(kReady % kASlotsAll == 0, "a barrier belongs to one slot");
    static_assert(kDoneSlots % kASlotsAll == 0 && kDoneSlots % kXSlots == 0, "unit-done ring");
};

}  // namespace fp8w
