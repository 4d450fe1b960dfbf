// w4a4_shape.h -- shared memory and TMEM of the W4A4 product for few tokens
// (gemm_w4a4.cu).  Host arithmetic only: plain C++.
#pragma once

#include <stddef.h>

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

}  // namespace nvfp4
