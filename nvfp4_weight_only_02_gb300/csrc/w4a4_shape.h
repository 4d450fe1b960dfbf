// w4a4_shape.h -- shared memory, TMEM and split of the W4A4 product for few
// tokens (gemm_w4a4.cu).  Host arithmetic only: plain C++.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <algorithm>

namespace nvfp4 {

constexpr int kWsRows = 128;     // weight rows per CTA
constexpr int kWsK = 256;        // elements of K per stage (128 bytes of codes a row)
constexpr int kWsSmem = 113 * 1024;  // two CTAs share an SM
constexpr int kWsMaxStages = 6;

// Tokens as the kernel gets them: quantised, or bf16 / FP32 to be quantised here.
enum Tokens { kCodes, kBf16, kFp32 };

// A CTA that waits for TMEM columns waits without a limit, and one that holds
// columns may itself wait for a CTA of its cluster on another SM.  So the CTAs
// that fit into an SM's 228 KB of shared memory (1 KB more than its own for
// each) must never want more than its 512 columns together.  Kernels allocate
// multiples of 128: more than 512 is 640 at least, which at 46 KB for 128
// columns comes to 5 x 46 KB and 1 KB for each of three CTAs or more, 233 KB.
// (The tile kernels, with all 512 columns, leave no room for another CTA.)
constexpr size_t kWsSmemPer128Columns = 46 * 1024;

template <bool kNv, int NT, Tokens kTok>
struct WsShape {
    static constexpr int kTiles = kNv ? 4 : 2;                    // scale tiles per stage and operand
    static constexpr int kScaleBytes = kTiles * 512;
    static constexpr int kWBytes = kWsRows * 128 + kScaleBytes, kXBytes = NT * 128 + kScaleBytes;
    static constexpr bool kOwn = kTok != kCodes;                  // tokens quantised here stay for all stages
    static constexpr int kFixed = 1024 + 256;
    static constexpr int kAccCols = NT < 64 ? 64 : NT;
    static constexpr int kSfCols = 2 * kTiles * 4;                // one stage's scales of both operands
    static constexpr int kSfBufs = kNv && NT <= 64 ? 2 : 4;       // stages whose scales fit beside the accumulator
    static constexpr int kTmemCols = kAccCols + kSfBufs * kSfCols <= 128 ? 128 : 256;
    static_assert(kAccCols + kSfBufs * kSfCols <= kTmemCols, "TMEM");
    // ring stages beside `nk` stages of own tokens; 0: they do not fit
    static int stages(int nk)
    {
        const int room = kWsSmem - kFixed - (kOwn ? nk * kXBytes : 0);
        const int fit = room / (kOwn ? kWBytes : kWBytes + kXBytes);
        return std::max(0, std::min({fit, kWsMaxStages, std::max(nk, 2)}));
    }
    static size_t smem(int nk, int stages)
    {
        const size_t ring = (size_t)stages * (kOwn ? kWBytes : kWBytes + kXBytes) + (kOwn ? (size_t)nk * kXBytes : 0);
        // the ring also holds the shares of a split K
        return std::max(kFixed + std::max(ring, (size_t)NT * 512), kTmemCols / 128 * kWsSmemPer128Columns);
    }
};

// K is split while the tiles leave CTA places free: two per SM, at most 8 CTAs to a cluster.
inline int ws_split(int64_t tiles, int64_t K, int num_sms)
{
    const int64_t ksteps = (K + kWsK - 1) / kWsK;
    return (int)std::max<int64_t>(1, std::min<int64_t>({8, ksteps, 2 * num_sms / tiles}));
}

// Whether the tokens (FP32 or bf16) are quantised in the product's kernel, not by a kernel of their own.  Every CTA
// quantises its part of K for all tokens again, so what it takes and how many turns of CTAs do that decide, against a
// launch and about 1.5 us; many stages to multiply behind that hide some of it.  6144 bf16 elements are the loads that
// a CTA has on their way at once, in FP32 half as many.  One kernel / two, us:
//   bf16: 3584 x 18944, split 8, ten stages a CTA: 4 tokens (10240 elements) 11.1 / 11.5, 6 (15360) 12.0 / 11.5;
//   18944 x 3584, split 2, seven: 6 (10752) 10.2 / 10.9, 7 (12544) 11.3 / 11.0; 12288 x 4096, split 3, six: 8 (12288)
//   10.2 / 10.4; 1024 x 10240, split 8, five: 5 (6400) 6.8 / 6.9, 9 (11520) 7.2 / 7.0; 1024 x 8192, split 8, four:
//   6 (6144) 5.4 / 6.4, 7 (7168) 6.5 / 6.1; 3584 x 3584, split 8, two: 12 (6144) 6.2 / 7.1, 16 (8192) 7.2 / 7.1;
//   27648 x 5120, no split, twenty: 2 (10240) 16.3 / 16.5, 3 (15360) 17.8 / 16.5; 76032 x 3584, two turns: 1 (7168)
//   25.9 / 27.5, 2 (14336) 28.8 / 27.7.
//   FP32: 3584 x 18944: 4 (10240) 11.6 / 12.1, 5 (12800) 12.1 / 11.9; 18944 x 3584: 5 (8960) 10.6 / 10.9, 6 (10752)
//   11.3 / 10.8; without a split 27648 x 5120: 2 (10240) 17.7 / 16.5; 40000 x 2048, two turns: 2 (8192) 15.0 / 14.4;
//   76032 x 3584, two turns: 1 (7168) 27.0 / 27.5.
inline bool ws_takes_tokens(int64_t M, int64_t N, int64_t K, bool fp32, int num_sms)
{
    if (M > 16)
        return false;
    const int64_t tiles = (N + kWsRows - 1) / kWsRows, ksteps = (K + kWsK - 1) / kWsK;
    const int64_t split = ws_split(tiles, K, num_sms), nk = (ksteps + split - 1) / split;
    const int64_t turns = (tiles * split + 2 * num_sms - 1) / (2 * num_sms);
    const int64_t most = nk < 6 ? 6144 : !fp32 ? 12288 : split > 1 ? 10240 : 7680;
    if (M * nk * kWsK * turns > most)
        return false;
    // at least three stages of weights beside the tokens
    return nk <= 64 && WsShape<false, 16, kBf16>::stages((int)nk) >= std::min<int64_t>(3, std::max<int64_t>(nk, 2));
}

}  // namespace nvfp4
