// rings.h -- the rings between the roles of the tensor-core kernel K4 (prefill.cu):
// their depths, and who takes which slot and barrier.  Plain C++, so that
// tests/test_rings.py runs a model of the barriers on these same numbers and
// functions.
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

}  // namespace fp8w
