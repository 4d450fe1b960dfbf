// moe_route.cu -- routing of tokens to experts: the k best experts of a token
// and their weights, the grouping of the (token, choice) slots by expert, the
// gradient of the router's logits, and the weighted sum of the experts' rows
// back to the tokens with its gradient.
//
// Mathematics.  Of a token's E logits z the k largest are taken (of score plus
// bias with a bias), ties to the lowest index; with l = z or log sigmoid(z) the
// weights are scale * softmax of l over the taken ones, or scale * softmax(z)
// (sigmoid(z)) of each.  Softmax over the taken ones is formed from the
// differences to their largest, so it has no 0 / 0 where the scores underflow.
//
// Grouping is a counting sort, stable in the slot number t k + j, so that it
// depends on nothing but the experts: a warp counts its run of slots 32 at a
// time (lanes with equal experts rank themselves by match), counts are summed
// over warps and CTAs, and the second pass places each slot.
//
// What bounds it.  16384 tokens, 8 of 256 experts: 22 us, of which choosing 16
// (instructions) and placing 6 (the second kernel waits for each CTA's counts,
// 152 x 256 of them read by every CTA; 9 when a thread asked for few of them at a
// time and for its slots afterwards); gradient 4.5 (issue 55 %, latency; its 17 MB
// stay in L2), 10.3 with scores over all experts (issue 76 %).  8192 tokens, 8 rows
// each of 4096 in bf16: sum 87.5 us, its gradients 169 (99 % of the copy rate or more).
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "moe_plan.h"

namespace nvfp4 {

namespace {

constexpr int kRtThreads = 1024, kRtWarps = kRtThreads / 32;
constexpr uint32_t kAll = 0xffffffffu;

struct RouteParams {
    const void *z;          // T x E, ldz; null: the experts are given
    int z_fp32;
    int64_t T, ldz;
    int E, k;
    int sigmoid, renorm;
    const float *bias;      // E or null
    float scale;
    float *weights;         // T x k
    int32_t *experts;       // T x k: written, or read where they are given
    int32_t *plan;
    int64_t offsets, first_block, position, order, padded, blocks, tiles, counts;
    int tile_rows;
    int64_t slots;
    int chunk;              // tokens of a CTA
    uint32_t *ctl;          // status words or null
};

__device__ __forceinline__ float load_z(const void *z, int fp32, int64_t at)
{
    return fp32 ? reinterpret_cast<const float *>(z)[at]
                : __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(z)[at]);
}

// log sigmoid(z) without overflow on either side
__device__ __forceinline__ float log_sigmoid(float z) { return fminf(z, 0.0f) - log1pf(expf(-fabsf(z))); }
__device__ __forceinline__ float sigmoid(float z)
{
    const float e = expf(-fabsf(z));
    return (z >= 0.0f ? 1.0f : e) / (1.0f + e);
}

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int d = 16; d; d >>= 1)
        v = fmaxf(v, __shfl_xor_sync(kAll, v, d));
    return v;
}
__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int d = 16; d; d >>= 1)
        v += __shfl_xor_sync(kAll, v, d);
    return v;
}

// Order-preserving key of a score; 0 for what is never taken (NaN, -inf).
__device__ __forceinline__ uint32_t key_of(float v)
{
    const uint32_t u = __float_as_uint(v + 0.0f);   // -0 ranks with +0
    return v > -INFINITY ? u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u) : 0u;
}

// The k experts of the largest keys, in order; equal keys by index.  A lane has
// kPer experts behind one another, so of equal keys the lowest lane's is first.
// Returns lane j's choice j, -1 where there is none.
//
// Up to 16 choices: the k-th of the lanes' largest keys (each distinct one
// counted once) is a bound that the k best reach and few others, about 9 keys for
// k = 8 and 21 for k = 16 whatever E is, when experts are in no order.  Those that
// reach it are collected, a lane each, and a key's place is the number of larger
// ones.  Where more than 32 reach it, and for more choices, each round looks at
// all keys.  Routing 16384 tokens, 8 of 256, 8 of 512, 16 of 1024 experts takes 22, 34
// and 54 us; with rounds over all keys the 512 took 12 more and the 1024 45, with each
// lane's keys sorted first the 256 2 more.
constexpr int kRtFew = 16;
struct Candidates {
    uint32_t key[32];
    int expert[32];
};
template <int kPer>
__device__ __forceinline__ int choose(const uint32_t (&key)[kPer], int k, int lane, Candidates &c)
{
    int mine = -1;
    if (k <= kRtFew) {
        uint32_t head = key[0];
#pragma unroll
        for (int i = 1; i < kPer; i++)
            head = max(head, key[i]);
        uint32_t bound = 0;
        for (int j = 0; j < k; j++) {
            bound = __reduce_max_sync(kAll, head);
            if (bound == 0)
                break;
            head = head == bound ? 0u : head;
        }
        bound = max(bound, 1u);
        int n = 0;
#pragma unroll
        for (int i = 0; i < kPer; i++)
            n += key[i] >= bound;
        // keys of the lanes before, and of all
        int at = 0, all = 0;
#pragma unroll
        for (int bit = 1; bit <= kPer; bit *= 2) {
            const uint32_t has = __ballot_sync(kAll, n & bit);
            at += bit * __popc(has & ((1u << lane) - 1u));
            all += bit * __popc(has);
        }
        if (all <= 32) {
#pragma unroll
            for (int i = 0; i < kPer; i++) {
                if (key[i] >= bound) {
                    c.key[at] = key[i];
                    c.expert[at++] = lane * kPer + i;
                }
            }
            __syncwarp();
            const uint32_t own = lane < all ? c.key[lane] : 0u;
            const int expert = lane < all ? c.expert[lane] : -1;
            int place = 0;
            for (int j = 0; j < all; j += 4) {
#pragma unroll
                for (int i = 0; i < 4; i++)     // behind the last one: 0, above nothing
                    place += __shfl_sync(kAll, own, j + i) + (j + i < lane) > own;
            }
            __syncwarp();
            if (lane < all && place < k)
                c.expert[place] = expert;
            __syncwarp();
            mine = lane < min(k, all) ? c.expert[lane] : -1;
            __syncwarp();
            return mine;
        }
    }
    uint32_t left[kPer];
#pragma unroll
    for (int i = 0; i < kPer; i++)
        left[i] = key[i];
    for (int j = 0; j < k; j++) {
        uint32_t head = left[0];
#pragma unroll
        for (int i = 1; i < kPer; i++)
            head = max(head, left[i]);
        const uint32_t top = __reduce_max_sync(kAll, head);
        if (top == 0)
            break;
        const int from = __ffs(__ballot_sync(kAll, head == top)) - 1;
        int at = 0;
#pragma unroll
        for (int i = kPer - 1; i >= 0; i--)
            at = left[i] == top ? i : at;
        at = __shfl_sync(kAll, at, from);
#pragma unroll
        for (int i = 0; i < kPer; i++)
            left[i] = lane == from && i == at ? 0u : left[i];
        mine = lane == j ? from * kPer + at : mine;
    }
    return mine;
}

// kPer logits behind one another from element `at` (of row t), -inf behind the last expert.
template <int kPer, bool kF32>
__device__ __forceinline__ void load_logits(const RouteParams &p, int64_t t, int e0, float (&z)[kPer])
{
    constexpr int kBytes = kPer * (kF32 ? 4 : 2), kStep = kBytes < 16 ? kBytes : 16;
    const char *src = reinterpret_cast<const char *>(p.z) + (t * p.ldz + e0) * (kF32 ? 4 : 2);
    if (e0 + kPer <= p.E && p.ldz * (kF32 ? 4 : 2) % kStep == 0) {
        uint32_t w[kBytes / 4];
#pragma unroll
        for (int i = 0; i < kBytes / kStep; i++) {
            if constexpr (kStep == 16) {
                const uint4 a = ld_once_u4(src + 16 * i);
                w[4 * i] = a.x, w[4 * i + 1] = a.y, w[4 * i + 2] = a.z, w[4 * i + 3] = a.w;
            } else if constexpr (kStep == 8) {
                const uint2 a = *reinterpret_cast<const uint2 *>(src);
                w[0] = a.x, w[1] = a.y;
            } else {
                w[0] = *reinterpret_cast<const uint32_t *>(src);
            }
        }
#pragma unroll
        for (int i = 0; i < kPer; i++)
            z[i] = kF32 ? __uint_as_float(w[i]) : __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    } else {
#pragma unroll
        for (int i = 0; i < kPer; i++)
            z[i] = e0 + i < p.E ? load_z(p.z, kF32, t * p.ldz + e0 + i) : -INFINITY;
    }
}

// One token by one warp, kPer experts a lane.
template <int kPer, bool kF32>
__device__ __forceinline__ void route_token(const RouteParams &p, int64_t t, const float (&z)[kPer], int lane, Candidates &s_cand)
{
    bool nan = false;   // the softmax of the row has no value
#pragma unroll
    for (int i = 0; i < kPer; i++)
        nan |= p.sigmoid ? z[i] != z[i] : !(z[i] < INFINITY);
    nan = __any_sync(kAll, nan);
    // statistics of the softmax over all experts
    float zmax = -INFINITY, denom = 0.0f;
    if (!p.sigmoid && (!p.renorm || p.bias)) {
#pragma unroll
        for (int i = 0; i < kPer; i++)
            zmax = fmaxf(zmax, z[i]);
        zmax = warp_max(zmax);
#pragma unroll
        for (int i = 0; i < kPer; i++)
            denom += z[i] > -INFINITY ? expf(z[i] - zmax) : 0.0f;
        denom = warp_sum(denom);
    }
    uint32_t key[kPer];
    if (p.bias) {
#pragma unroll
        for (int i = 0; i < kPer; i++) {
            const int e = lane * kPer + i;
            float v = z[i];
            if (e < p.E && v > -INFINITY)
                v = (p.sigmoid ? sigmoid(v) : expf(v - zmax) / denom) + p.bias[e];
            key[i] = key_of(v);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kPer; i++)
            key[i] = key_of(z[i]);
    }
    const int mine = choose<kPer>(key, p.k, lane, s_cand);
    const float zj = mine >= 0 ? load_z(p.z, kF32, t * p.ldz + mine) : -INFINITY;
    float w = 0.0f;
    if (p.renorm) {
        const float l = mine >= 0 && p.sigmoid ? log_sigmoid(zj) : zj;
        const float lmax = warp_max(l);
        const float e = mine >= 0 ? expf(l - lmax) : 0.0f;
        const float sum = warp_sum(e);
        w = mine >= 0 ? e / sum : 0.0f;
    } else if (mine >= 0) {
        w = p.sigmoid ? sigmoid(zj) : expf(zj - zmax) / denom;
    }
    if (lane < p.k) {
        p.weights[t * p.k + lane] = nan ? __uint_as_float(0x7FC00000u) : w * p.scale;
        p.experts[t * p.k + lane] = mine;
    }
}

// The tokens t0, t0 + step, ... below t1; up to eight experts a lane the next one's logits are on their way meanwhile.
template <int kPer, bool kF32>
__device__ __forceinline__ void route_run(const RouteParams &p, int64_t t0, int64_t t1, int step, int lane, Candidates &s_cand)
{
    constexpr bool kAhead = kPer <= 8;
    float z[kPer], next[kAhead ? kPer : 1];
    if constexpr (kAhead) {
        if (t0 < t1)
            load_logits<kPer, kF32>(p, t0, lane * kPer, next);
    }
    for (int64_t t = t0; t < t1; t += step) {
        if constexpr (kAhead) {
#pragma unroll
            for (int i = 0; i < kPer; i++)
                z[i] = next[i];
            if (t + step < t1)
                load_logits<kPer, kF32>(p, t + step, lane * kPer, next);
        } else {
            load_logits<kPer, kF32>(p, t, lane * kPer, z);
        }
        route_token<kPer, kF32>(p, t, z, lane, s_cand);
    }
}

template <bool kF32>
__device__ __forceinline__ void route_tokens(const RouteParams &p, int64_t t0, int64_t t1, int step, int lane, Candidates &s_cand)
{
    if (p.E <= 64)
        route_run<2, kF32>(p, t0, t1, step, lane, s_cand);
    else if (p.E <= 128)
        route_run<4, kF32>(p, t0, t1, step, lane, s_cand);
    else if (p.E <= 256)
        route_run<8, kF32>(p, t0, t1, step, lane, s_cand);
    else if (p.E <= 512)
        route_run<16, kF32>(p, t0, t1, step, lane, s_cand);
    else
        route_run<32, kF32>(p, t0, t1, step, lane, s_cand);
}

// Calls f(slot, expert, rank) for the slots of this warp's run in groups of
// 32, expert -1 for none; rank counts lanes of the group before this one with
// the same expert, `last` tells the lane that ranks highest.
template <typename F>
__device__ __forceinline__ void each_slot(const RouteParams &p, int64_t s0, int64_t s1, int lane, F f)
{
    for (int64_t s = s0; s < s1; s += 32) {
        int e = -1;
        if (s + lane < s1) {
            e = p.experts[s + lane];
            if (e >= p.E || e < 0)
                e = -1;
        }
        const uint32_t same = __match_any_sync(kAll, e);
        const int rank = __popc(same & ((1u << lane) - 1u));
        f(s + lane, e, rank, rank + 1 == __popc(same));
        __syncwarp();
    }
}

// Inclusive sums over the block of three values a thread.
__device__ __forceinline__ void block_scan3(int (&v)[3], int (*s_warp)[3], int warp, int lane)
{
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
#pragma unroll
        for (int c = 0; c < 3; c++) {
            const int o = __shfl_up_sync(kAll, v[c], d);
            v[c] += lane >= d ? o : 0;
        }
    }
    if (lane == 31)
        for (int c = 0; c < 3; c++)
            s_warp[warp][c] = v[c];
    __syncthreads();
    if (warp == 0) {
        const bool is = lane < (int)(blockDim.x >> 5);
        int w[3] = {is ? s_warp[lane][0] : 0, is ? s_warp[lane][1] : 0, is ? s_warp[lane][2] : 0};
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
#pragma unroll
            for (int c = 0; c < 3; c++) {
                const int o = __shfl_up_sync(kAll, w[c], d);
                w[c] += lane >= d ? o : 0;
            }
        }
        for (int c = 0; c < 3; c++)
            s_warp[lane][c] = w[c];
    }
    __syncthreads();
    if (warp > 0)
        for (int c = 0; c < 3; c++)
            v[c] += s_warp[warp - 1][c];
}

// kFirst: experts (where there are logits), each slot's rank among the CTA's
// slots of its expert, and the CTA's counts.  kSecond: offsets, lists and the
// slots' places.  Both: one CTA does it all.
// kTopk: there are logits.  As many warps as the experts and the slots of a CTA
// need: fewer meet faster at the barriers (the plan of one token with 8 of 128
// experts: 3.9 us, 5.1 with 32 warps).
template <bool kTopk, bool kFirst, bool kSecond>
__global__ void __launch_bounds__(kRtThreads) route_kernel(const RouteParams p)
{
    extern __shared__ uint16_t s_hist[];            // [warps][E]
    __shared__ int s_base[kMoeMaxExperts];          // row of the expert's first slot of this CTA
    __shared__ int s_off[kMoeMaxExperts + 1], s_fb[kMoeMaxExperts + 1], s_ft[kMoeMaxExperts + 1];
    __shared__ int s_warp[kRtWarps][3];
    __shared__ Candidates s_cand[kTopk ? kRtWarps : 1];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, threads = blockDim.x, warps = threads >> 5;
    const int64_t t0 = (int64_t)blockIdx.x * p.chunk, t1 = min(p.T, t0 + p.chunk);
    const int64_t c0 = t0 * p.k, c1 = max(c0, t1 * p.k);    // the CTA's slots
    int32_t *counts = p.plan + p.counts, *position = p.plan + p.position;
    pdl_launch_dependents();
    pdl_wait();
    int total = 0, before = 0;
    int expert = -1, rank = 0;      // of the thread's next slot
    if (!kFirst && c0 + tid < c1) {
        expert = p.experts[c0 + tid];
        rank = position[c0 + tid];
    }
    if (kFirst) {
        if constexpr (kTopk) {
            if (p.z_fp32)
                route_tokens<true>(p, t0 + warp, t1, warps, lane, s_cand[warp]);
            else
                route_tokens<false>(p, t0 + warp, t1, warps, lane, s_cand[warp]);
        }
        uint16_t *hist = s_hist + warp * p.E;
        for (int i = lane; i < p.E; i += 32)
            hist[i] = 0;
        __syncthreads();
        // this warp's run of the CTA's slots
        const int64_t per = (c1 - c0 + threads - 1) / threads * 32;
        const int64_t s0 = min(c1, c0 + warp * per), s1 = min(c1, s0 + per);
        bool bad = false;
        each_slot(p, s0, s1, lane, [&](int64_t s, int e, int rank, bool last) {
            if (!kTopk && s < s1)
                bad |= p.experts[s] >= p.E;
            const int h = e >= 0 ? hist[e] : 0;
            __syncwarp();
            if (e >= 0 && last)
                hist[e] = (uint16_t)(h + rank + 1);
            if (s < s1)
                position[s] = h + rank;     // among this warp's slots
        });
        if (bad && p.ctl)
            record_status(p.ctl, NVFP4_ERR_INDEX);
        __syncthreads();
        // per expert: counts of the warps before, and the CTA's
        if (tid < p.E) {
#pragma unroll 8
            for (int w = 0; w < warps; w++) {
                const int c = s_hist[w * p.E + tid];
                s_hist[w * p.E + tid] = (uint16_t)total;
                total += c;
            }
            if (!kSecond)
                counts[(int64_t)blockIdx.x * p.E + tid] = total;
        }
        __syncthreads();
        for (int64_t s = s0 + lane; s < s1; s += 32) {
            const int e = p.experts[s];
            if (e >= 0 && e < p.E)
                position[s] += hist[e];
        }
        if (!kSecond)
            return;
    } else {
        // counts of all CTAs, 16 a thread on their way at once; the threads share out the CTAs where there are few experts
        __shared__ int s_before[kMoeMaxExperts], s_total[kMoeMaxExperts];
        s_before[tid] = s_total[tid] = 0;   // 1024 threads
        __syncthreads();
        const int width = (p.E + 31) / 32 * 32, groups = threads / width, g = tid / width, e = tid % width;
        if (g < groups && e < p.E) {
            int b = 0, all = 0;
            for (int first = g; first < (int)gridDim.x; first += 16 * groups) {
                int v[16];
#pragma unroll
                for (int i = 0; i < 16; i++) {
                    const int c = first + i * groups;
                    v[i] = c < (int)gridDim.x ? counts[(int64_t)c * p.E + e] : 0;
                }
#pragma unroll
                for (int i = 0; i < 16; i++) {
                    all += v[i];
                    b += first + i * groups < (int)blockIdx.x ? v[i] : 0;
                }
            }
            atomicAdd(&s_before[e], b);
            atomicAdd(&s_total[e], all);
        }
        __syncthreads();
        if (tid < p.E) {
            before = s_before[tid];
            total = s_total[tid];
        }
    }
    int v[3] = {total, (total + kMoeBlock - 1) / kMoeBlock, (total + p.tile_rows - 1) / p.tile_rows};
    const int mine[3] = {v[0], v[1], v[2]};
    block_scan3(v, s_warp, warp, lane);
    if (tid < p.E) {
        s_off[tid] = v[0] - mine[0];
        s_fb[tid] = v[1] - mine[1];
        s_ft[tid] = v[2] - mine[2];
        s_base[tid] = s_off[tid] + before;
        if (tid == p.E - 1) {
            s_off[p.E] = v[0];
            s_fb[p.E] = v[1];
            s_ft[p.E] = v[2];
        }
    }
    __syncthreads();
    const int rows = s_off[p.E];
    if (blockIdx.x == 0) {
        for (int e = tid; e <= p.E; e += threads) {
            p.plan[p.offsets + e] = s_off[e];
            p.plan[p.first_block + e] = s_fb[e];
        }
        if (tid < kMoeHeader)
            p.plan[tid] = tid == kMoeRows ? rows : tid == kMoeBlocks ? s_fb[p.E] : tid == kMoeTiles ? s_ft[p.E] : 0;
    }
    // lists of blocks and tiles: expert, first row of the padded and of the compact order, rows
    auto list = [&](const int *first, int size, int4 *out) {
        for (int i = (int)blockIdx.x * threads + tid; i < first[p.E]; i += (int)gridDim.x * threads) {
            int e = 0;   // the last expert whose first is i or below
            for (int step = kMoeMaxExperts / 2; step; step >>= 1)
                if (e + step < p.E && first[e + step] <= i)
                    e += step;
            const int r = (i - first[e]) * size;
            out[i] = make_int4(e, s_fb[e] * kMoeBlock + r, s_off[e] + r, min(size, s_off[e + 1] - s_off[e] - r));
        }
    };
    list(s_fb, kMoeBlock, reinterpret_cast<int4 *>(p.plan + p.blocks));
    list(s_ft, p.tile_rows, reinterpret_cast<int4 *>(p.plan + p.tiles));
    for (int64_t r = rows + (int64_t)blockIdx.x * threads + tid; r < p.slots; r += (int64_t)gridDim.x * threads)
        p.plan[p.order + r] = -1;
    // places; in one CTA each thread meets the ranks that another warp wrote before the last barriers
    if (kFirst && c0 + tid < c1) {
        expert = p.experts[c0 + tid];
        rank = position[c0 + tid];
    }
    for (int64_t s = c0 + tid; s < c1; s += threads) {
        const int e = expert, r = rank;
        int pos = -1, pad = -1;
        if (s + threads < c1) {
            expert = p.experts[s + threads];
            rank = position[s + threads];
        }
        if (e >= 0 && e < p.E) {
            pos = s_base[e] + r;
            pad = s_fb[e] * kMoeBlock + pos - s_off[e];
            p.plan[p.order + pos] = (int32_t)s;
        }
        position[s] = pos;
        p.plan[p.padded + s] = pad;
    }
}

// dz of the router, a warp a token.
//
// With u = w / scale, a softmax over the taken ones (j among them), dl_i = w_i (dw_i -
// sum_j u_j dw_j): with a weight near 1, or dw that share an offset, the difference
// cancels (logits 14, 0, -1, -2: the largest one's gradient off by 3 %).  So the dw
// of the largest weight, r, is taken off all of them first, d = dw - dw_r; then
//     dl_i = w_i (d_i - sum_j u_j d_j),
// whose sum is all that r has and which cancels k-fold at most for the others.  With
// scores over all experts, of which A are taken and B = 1 - A are not (each summed by
// itself), dl_i = w_i (A d_i + B dw_i - sum_j u_j d_j).
struct RouteGradParams {
    const void *z;
    int z_fp32;
    int64_t T, ldz;
    int E, k;
    int sigmoid, renorm;
    float scale;
    const float *weights, *dw;
    const int32_t *experts;
    void *dz;
    int64_t lddz;
};

__device__ __forceinline__ void put_dz(const RouteGradParams &p, int64_t at, float v)
{
    if (p.z_fp32)
        reinterpret_cast<float *>(p.dz)[at] = v;
    else
        reinterpret_cast<__nv_bfloat16 *>(p.dz)[at] = __float2bfloat16_rn(v);
}

// A row whose scores are a softmax over all experts, lane, lane + 32, ... of them a
// lane's.  e, w, dw: this lane's slot (e < 0: none); d, sum as above; own = w dw.
template <int kPer>
__device__ __forceinline__ void softmax_grad(const RouteGradParams &p, int64_t t, int lane, int e, float w, float dw, float d,
                                             float sum, float own)
{
    uint32_t taken = 0;
    for (int j = 0; j < p.k; j++) {
        const int apart = __shfl_sync(kAll, e, j) - lane;   // no expert: not a multiple of 32 apart, or below 0
        taken |= apart >= 0 && (apart & 31) == 0 ? 1u << (apart >> 5) : 0u;
    }
    float s[kPer], zmax = -INFINITY, in = 0.0f, out = 0.0f;
#pragma unroll
    for (int u = 0; u < kPer; u++) {
        const int i = lane + 32 * u;
        s[u] = i < p.E ? load_z(p.z, p.z_fp32, t * p.ldz + i) : -INFINITY;
        zmax = fmaxf(zmax, s[u]);
    }
    zmax = warp_max(zmax);
#pragma unroll
    for (int u = 0; u < kPer; u++) {
        s[u] = s[u] == -INFINITY ? 0.0f : expf(s[u] - zmax);
        in += taken >> u & 1u ? s[u] : 0.0f;
        out += taken >> u & 1u ? 0.0f : s[u];
    }
    in = warp_sum(in);
    out = warp_sum(out);
    const float denom = in + out, dot = warp_sum(own), share = dot / denom;
#pragma unroll
    for (int u = 0; u < kPer; u++) {
        const int i = lane + 32 * u;
        if (i < p.E)
            put_dz(p, t * p.lddz + i, dot != dot ? dot : s[u] == 0.0f ? 0.0f : -s[u] * share);
    }
    __syncwarp();   // the chosen ones over what their lanes' neighbours wrote
    if (e >= 0)
        put_dz(p, t * p.lddz + e, dot != dot ? dot : w * ((in * d + out * dw) / denom - sum));
}

// kPer: experts a lane where the scores are a softmax over all of them, else 0.
template <int kPer>
__global__ void __launch_bounds__(256) route_grad_kernel(const RouteGradParams p)
{
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    pdl_wait();
    pdl_launch_dependents();
    if (t >= p.T)
        return;
    int e = -1;
    float w = 0.0f, dw = 0.0f;
    if (lane < p.k) {
        e = p.experts[t * p.k + lane];
        if (e >= p.E || e < 0)
            e = -1;
        w = p.weights[t * p.k + lane];
        dw = p.dw[t * p.k + lane];
    }
    const bool none = e < 0;
    // a NaN weight reaches the gradient of its row, an unused slot's dw does not
    const float own = none ? w * 0.0f : w * dw;
    float d = dw, sum = 0.0f;
    bool nan = false;
    if (p.renorm || kPer > 0) {
        const uint32_t size = none ? 0u : __float_as_uint(fabsf(w));
        const int r = __ffs(__ballot_sync(kAll, size == __reduce_max_sync(kAll, size))) - 1;
        const float dr = __shfl_sync(kAll, dw, r);
        d = lane == r ? 0.0f : dw - dr;
        sum = warp_sum(none || lane == r ? 0.0f : w * d);
        sum = p.scale != 0.0f ? sum / p.scale : 0.0f;
        nan = __any_sync(kAll, own != own);
    }
    if constexpr (kPer > 0) {
        softmax_grad<kPer>(p, t, lane, e, w, dw, d, sum, own);
        return;
    }
    const float v = nan ? __uint_as_float(0x7FC00000u) : 0.0f;   // a row without a value
    float g = w * (d - sum);
    if (p.sigmoid && !none)
        g *= sigmoid(-load_z(p.z, p.z_fp32, t * p.ldz + e));
    const int size = p.z_fp32 ? 4 : 2;
    char *row = reinterpret_cast<char *>(p.dz) + t * p.lddz * size;
    if (p.E * size % 16 == 0 && p.lddz * size % 16 == 0 && !nan) {
        for (int i = lane; i < p.E * size / 16; i += 32)
            reinterpret_cast<uint4 *>(row)[i] = make_uint4(0u, 0u, 0u, 0u);
    } else {
        for (int i = lane; i < p.E; i += 32)
            put_dz(p, t * p.lddz + i, v);
    }
    __syncwarp();   // the chosen ones over what their lanes' neighbours wrote
    if (!none)
        put_dz(p, t * p.lddz + e, nan ? v : g);
}

// ---------------------------------------------------------------- combine
// kVec elements of a row at a time: 16 bytes of the widest type involved (a
// thread with two of them would ask for each 32-byte sector twice), or single
// elements where rows do not start on 16-byte boundaries.
template <typename T, int kVec>
__device__ __forceinline__ void load_vec(const T *src, float (&v)[kVec])
{
    if constexpr (kVec == 1) {
        v[0] = (float)src[0];
    } else if constexpr (sizeof(T) == 2 && kVec == 4) {
        const uint2 a = *reinterpret_cast<const uint2 *>(src);
        v[0] = __uint_as_float(a.x << 16);
        v[1] = __uint_as_float(a.x & 0xFFFF0000u);
        v[2] = __uint_as_float(a.y << 16);
        v[3] = __uint_as_float(a.y & 0xFFFF0000u);
    } else if constexpr (sizeof(T) == 2) {
        static_assert(kVec == 8, "16 bytes");
        const uint4 a = ld_once_u4(src);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kVec; i += 4) {
            const uint4 a = ld_once_u4(src + i);
            v[i] = __uint_as_float(a.x);
            v[i + 1] = __uint_as_float(a.y);
            v[i + 2] = __uint_as_float(a.z);
            v[i + 3] = __uint_as_float(a.w);
        }
    }
}

// Rows that are written once: evicted first.
template <typename T, int kVec>
__device__ __forceinline__ void store_vec(T *dst, const float (&v)[kVec])
{
    if constexpr (kVec == 1) {
        if constexpr (sizeof(T) == 2)
            dst[0] = __float2bfloat16_rn(v[0]);
        else
            dst[0] = v[0];
    } else if constexpr (sizeof(T) == 2) {
        uint32_t w[kVec / 2];
#pragma unroll
        for (int i = 0; i < kVec / 2; i++) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        if constexpr (kVec == 8)
            __stcs(reinterpret_cast<uint4 *>(dst), make_uint4(w[0], w[1], w[2], w[3]));
        else
            *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
        for (int i = 0; i < kVec; i += 4)
            __stcs(reinterpret_cast<float4 *>(dst + i), make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]));
    }
}

// The same, unconverted: what is on its way of a row in a thread.
template <typename T, int kVec>
struct Vec;
template <>
struct Vec<__nv_bfloat16, 8> {
    uint32_t w[4];
    __device__ __forceinline__ void zero() { w[0] = w[1] = w[2] = w[3] = 0u; }
    __device__ __forceinline__ void load(const __nv_bfloat16 *p)
    {
        const uint4 a = ld_once_u4(p);
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
    }
    __device__ __forceinline__ float get(int e) const
    {
        return __uint_as_float(e & 1 ? w[e / 2] & 0xFFFF0000u : w[e / 2] << 16);
    }
};
template <>
struct Vec<__nv_bfloat16, 4> {
    uint2 w;
    __device__ __forceinline__ void zero() { w = make_uint2(0u, 0u); }
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { w = *reinterpret_cast<const uint2 *>(p); }
    __device__ __forceinline__ float get(int e) const
    {
        const uint32_t u = e & 2 ? w.y : w.x;
        return __uint_as_float(e & 1 ? u & 0xFFFF0000u : u << 16);
    }
};
template <>
struct Vec<float, 4> {
    float w[4];
    __device__ __forceinline__ void zero() { w[0] = w[1] = w[2] = w[3] = 0.0f; }
    __device__ __forceinline__ void load(const float *p) { load_vec<float, 4>(p, w); }
    __device__ __forceinline__ float get(int e) const { return w[e]; }
};
template <typename T>
struct Vec<T, 1> {
    float w;
    __device__ __forceinline__ void zero() { w = 0.0f; }
    __device__ __forceinline__ void load(const T *p) { w = (float)p[0]; }
    __device__ __forceinline__ float get(int) const { return w; }
};

struct CombineParams {
    const void *y, *base, *dout;
    const float *weights;
    const int32_t *position;
    void *out, *dy;
    float *dw;
    int64_t T;
    int N, k;
};

// out[t] = base[t] + sum_j w[t][j] y[position[t][j]], in FP32, j ascending.  A
// CTA takes a token, or a part of its row, eight rows' loads on their way at once:
// bounds that leave registers for them, 5 CTAs an SM for rows in FP32 or element by
// element, 6 for bf16 rows summed to FP32, else 4.  8192 x 8 rows of 4096 in bf16 take
// 87.5 us (93.5 with 5, 112 without a bound, in 40 registers), 8192 x 4 in FP32 96.7 (99.4
// with 4), 4096 x 4 in bf16 to FP32 35.3 (38.3 with 7), 1000 x 8 of 2601 25.7 (35.7 without).
constexpr int kCbRows = 8;

template <typename TY, typename TO, int kVec, bool kWeights>
__global__ void __launch_bounds__(256, kVec == 1 || sizeof(TY) == 4 ? 5 : sizeof(TO) == 4 ? 6 : 4)
    combine_kernel(const CombineParams p)
{
    const int64_t t = blockIdx.x;
    pdl_wait();
    pdl_launch_dependents();
    const TY *y = reinterpret_cast<const TY *>(p.y);
    int pos[kCbRows];
    float w[kCbRows];
    // all asked for before any row is; for up to eight slots once, not again for each piece of the row
    auto slots = [&](int j0) {
#pragma unroll
        for (int j = 0; j < kCbRows; j++) {
            pos[j] = j0 + j < p.k ? p.position[t * p.k + j0 + j] : -1;
            w[j] = !kWeights ? 1.0f : j0 + j < p.k ? p.weights[t * p.k + j0 + j] : 0.0f;
        }
        if (kWeights) {
#pragma unroll
            for (int j = 0; j < kCbRows; j++)   // without an expert nothing is added, be the weight infinite; a NaN shows
                w[j] = pos[j] >= 0 || w[j] != w[j] ? w[j] : 0.0f;
        }
    };
    const bool once = p.k <= kCbRows;
    if (once)
        slots(0);
    for (int c = (blockIdx.y * blockDim.x + threadIdx.x) * kVec; c < p.N; c += gridDim.y * blockDim.x * kVec) {
        float acc[kVec];
#pragma unroll
        for (int e = 0; e < kVec; e++)
            acc[e] = 0.0f;
        if (p.base)
            load_vec<TO, kVec>(reinterpret_cast<const TO *>(p.base) + t * p.N + c, acc);
        for (int j0 = 0; j0 < p.k; j0 += kCbRows) {
            if (!once)
                slots(j0);
            Vec<TY, kVec> v[kCbRows];
#pragma unroll
            for (int j = 0; j < kCbRows; j++) {
                v[j].zero();
                if (pos[j] >= 0)
                    v[j].load(y + (int64_t)pos[j] * p.N + c);
            }
#pragma unroll
            for (int j = 0; j < kCbRows; j++)
#pragma unroll
                for (int e = 0; e < kVec; e++)
                    acc[e] = fmaf(w[j], v[j].get(e), acc[e]);
        }
        store_vec<TO, kVec>(reinterpret_cast<TO *>(p.out) + t * p.N + c, acc);
    }
}

// dy[position[t][j]] = w[t][j] dout[t], dw[t][j] = <dout[t], y[position[t][j]]>: a CTA a token, dout read once for
// kRows slots, whose rows of y are on their way while the rows of dy are written.  Registers for that many loads and
// CTAs for the rest: bounds of 3 (bf16, eight rows), 5 (four), 4 and 6 (FP32).  8192 tokens of 4096 in bf16, eight
// rows each: 169 us (187 with loads as they are used, in 40 registers), four rows 92 (105); bounds of 2 and 4: 177, 183.
template <typename T, int kVec, int kRows>
__global__ void __launch_bounds__(256, kVec == 8 ? (kRows == 8 ? 3 : 5)
                                             : kVec == 4 ? (kRows == 8 ? 4 : 6) : 1) combine_grad_kernel(const CombineParams p)
{
    __shared__ float s_part[8][kRows];
    const int64_t t = blockIdx.x;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, warps = blockDim.x >> 5;
    pdl_wait();
    pdl_launch_dependents();
    const T *dout = reinterpret_cast<const T *>(p.dout) + t * p.N, *y = reinterpret_cast<const T *>(p.y);
    T *dy = reinterpret_cast<T *>(p.dy);
    for (int j0 = 0; j0 < p.k; j0 += kRows) {
        float dot[kRows], w[kRows];
        int pos[kRows];
#pragma unroll
        for (int j = 0; j < kRows; j++) {
            dot[j] = 0.0f;
            pos[j] = j0 + j < p.k ? p.position[t * p.k + j0 + j] : -1;
            w[j] = pos[j] >= 0 ? p.weights[t * p.k + j0 + j] : 0.0f;
        }
        for (int c = tid * kVec; c < p.N; c += blockDim.x * kVec) {
            float d[kVec];
            load_vec<T, kVec>(dout + c, d);
            Vec<T, kVec> v[kRows];
            if (p.dw) {
#pragma unroll
                for (int j = 0; j < kRows; j++) {
                    v[j].zero();
                    if (pos[j] >= 0)
                        v[j].load(y + (int64_t)pos[j] * p.N + c);
                }
            }
            if (dy) {   // while y's rows are on their way
#pragma unroll
                for (int j = 0; j < kRows; j++) {
                    if (pos[j] >= 0) {
                        float o[kVec];
#pragma unroll
                        for (int e = 0; e < kVec; e++)
                            o[e] = w[j] * d[e];
                        store_vec<T, kVec>(dy + (int64_t)pos[j] * p.N + c, o);
                    }
                }
            }
            if (p.dw) {
#pragma unroll
                for (int j = 0; j < kRows; j++)
#pragma unroll
                    for (int e = 0; e < kVec; e++)
                        dot[j] = fmaf(d[e], v[j].get(e), dot[j]);
            }
        }
        if (p.dw) {
#pragma unroll
            for (int j = 0; j < kRows; j++) {
                // a slot without an expert adds nothing, whatever dout holds
                const float s = warp_sum(pos[j] >= 0 ? dot[j] : 0.0f);
                if (lane == 0)
                    s_part[warp][j] = s;
            }
            __syncthreads();
            if (tid < kRows && j0 + tid < p.k) {
                float s = 0.0f;
                for (int i = 0; i < warps; i++)
                    s += s_part[i][tid];
                p.dw[t * p.k + j0 + tid] = s;
            }
            __syncthreads();
        }
    }
}

constexpr size_t kRtMaxSmem = (size_t)kRtWarps * kMoeMaxExperts * 2;

// Threads of a token's CTA.
int combine_threads(int64_t N, int vec)
{
    const int64_t items = (N + vec - 1) / vec;
    return (int)std::min<int64_t>(256, (items + 31) / 32 * 32);
}

template <typename TY, typename TO, bool kWeights>
cudaError_t run_combine(const MoeCombineArgs &a, const CombineParams &p, cudaStream_t s)
{
    // rows that are no multiple of the vector go element by element: 8192 x 8 rows of 2601 in bf16 149 us, of 2600 55
    constexpr int kVec = sizeof(TY) == 4 || sizeof(TO) == 4 ? 4 : 8;
    const int vec = a.N % kVec == 0 ? kVec : 1, threads = combine_threads(a.N, vec);
    // few tokens: a row's vectors over several CTAs, many: one for all of them.  Rows of 4096 in bf16, us over several /
    // in one, for 64, 256, 512, 1536, 4096 tokens: eight rows each 2.7 / 3.4, 3.9 / 4.1, 8.2 / 7.5, 19.9 / 19.6, 46.8 /
    // 45.8; two 2.7 / 2.8, 3.4 / 3.4, 4.8 / 4.8, 11.1 / 10.3, 26.7 / 23.9; rows of 7168, eight each: 2.8 / 4.1, 6.9 / 8.2,
    // 13.0 / 12.3, 33.3 / 32.5, 81.4 / 78.4
    const int64_t pieces = std::min<int64_t>((a.N + vec * threads - 1) / (vec * threads), 65535);   // a grid's most in y
    const dim3 grid((unsigned)a.T, a.T < 512 ? (unsigned)pieces : 1u);
    return vec > 1 ? launch_dependent(combine_kernel<TY, TO, kVec, kWeights>, grid, threads, 0, s, p)
                   : launch_dependent(combine_kernel<TY, TO, 1, kWeights>, grid, threads, 0, s, p);
}

template <bool kWeights>
cudaError_t run_combine_types(const MoeCombineArgs &a, const CombineParams &p, cudaStream_t s)
{
    using B = __nv_bfloat16;
    if (a.y_fp32)
        return a.out_fp32 ? run_combine<float, float, kWeights>(a, p, s) : run_combine<float, B, kWeights>(a, p, s);
    return a.out_fp32 ? run_combine<B, float, kWeights>(a, p, s) : run_combine<B, B, kWeights>(a, p, s);
}

template <typename T, int kRows>
cudaError_t run_combine_grad(const MoeCombineArgs &a, const CombineParams &p, cudaStream_t s)
{
    // element by element as above: 313 us instead of 126.  A CTA a token however few there are: 16 tokens, eight rows of
    // 4096 each, 4.1 us.
    constexpr int kVec = 16 / sizeof(T);
    const dim3 grid((unsigned)a.T);
    return a.N % kVec == 0
               ? launch_dependent(combine_grad_kernel<T, kVec, kRows>, grid, combine_threads(a.N, kVec), 0, s, p)
               : launch_dependent(combine_grad_kernel<T, 1, kRows>, grid, combine_threads(a.N, 1), 0, s, p);
}

CombineParams combine_params(const MoeCombineArgs &a)
{
    CombineParams p = {};
    p.y = a.y;
    p.base = a.base;
    p.dout = a.dout;
    p.weights = a.weights;
    p.position = a.position;
    p.out = a.out;
    p.dy = a.dy;
    p.dw = a.dw;
    p.T = a.T;
    p.N = (int)a.N;
    p.k = a.k;
    return p;
}

template <bool kTopk>
cudaError_t run_route(const RouteParams &p, const MoeLayout &l, cudaStream_t s, const DeviceInfo &dev)
{
    if (l.ctas == 1) {
        // a thread for each expert and each slot, a warp for each token
        const int64_t want = std::max<int64_t>({p.E, l.slots, kTopk ? 32 * p.T : 0});
        const int threads = (int)std::min<int64_t>(kRtThreads, (want + 31) / 32 * 32);
        const cudaError_t e = allow_smem<route_kernel<kTopk, true, true>>(kRtMaxSmem, dev);
        return e != cudaSuccess ? e : launch_dependent(route_kernel<kTopk, true, true>, 1, threads,
                                                       (size_t)(threads / 32) * p.E * 2, s, p);
    }
    cudaError_t e = allow_smem<route_kernel<kTopk, true, false>>(kRtMaxSmem, dev);
    if (e == cudaSuccess)
        e = launch_dependent(route_kernel<kTopk, true, false>, (unsigned)l.ctas, kRtThreads, (size_t)kRtWarps * p.E * 2, s,
                             p);
    if (e == cudaSuccess)
        e = launch_dependent(route_kernel<false, false, true>, (unsigned)l.ctas, kRtThreads, 0, s, p);
    return e;
}

}  // namespace

cudaError_t launch_moe_route(const MoeRouteArgs &a, cudaStream_t s, const DeviceInfo &dev)
{
    const MoeLayout l(a.T, a.k, a.E);
    RouteParams p = {};
    p.z = a.z;
    p.z_fp32 = a.z_fp32 ? 1 : 0;
    p.T = a.T;
    p.ldz = a.ldz;
    p.E = a.E;
    p.k = a.k;
    p.sigmoid = a.sigmoid ? 1 : 0;
    p.renorm = a.renorm ? 1 : 0;
    p.bias = a.bias;
    p.scale = a.scale;
    p.weights = a.weights;
    p.experts = a.experts;
    p.plan = a.plan;
    p.offsets = l.offsets;
    p.first_block = l.first_block;
    p.position = l.position;
    p.order = l.order;
    p.padded = l.padded;
    p.blocks = l.blocks;
    p.tiles = l.tiles;
    p.counts = l.counts;
    p.tile_rows = l.tile_rows;
    p.slots = l.slots;
    p.ctl = a.ctl;
    p.chunk = (int)((a.T + l.ctas - 1) / l.ctas);
    return a.z ? run_route<true>(p, l, s, dev) : run_route<false>(p, l, s, dev);
}

cudaError_t launch_moe_route_backward(const MoeRouteArgs &a, const float *dw, void *dz, int64_t lddz, cudaStream_t s)
{
    RouteGradParams p = {};
    p.z = a.z;
    p.z_fp32 = a.z_fp32 ? 1 : 0;
    p.T = a.T;
    p.ldz = a.ldz;
    p.E = a.E;
    p.k = a.k;
    p.sigmoid = a.sigmoid ? 1 : 0;
    p.renorm = a.renorm ? 1 : 0;
    p.scale = a.scale;
    p.weights = a.weights;
    p.dw = dw;
    p.experts = a.experts;
    p.dz = dz;
    p.lddz = lddz;
    const dim3 grid((unsigned)((a.T + 7) / 8));
    if (a.sigmoid || a.renorm)
        return launch_dependent(route_grad_kernel<0>, grid, 256, 0, s, p);
    return a.E <= 256 ? launch_dependent(route_grad_kernel<8>, grid, 256, 0, s, p)
                      : launch_dependent(route_grad_kernel<32>, grid, 256, 0, s, p);
}

cudaError_t launch_moe_combine(const MoeCombineArgs &a, cudaStream_t s)
{
    const CombineParams p = combine_params(a);
    return a.weights ? run_combine_types<true>(a, p, s) : run_combine_types<false>(a, p, s);
}

cudaError_t launch_moe_combine_backward(const MoeCombineArgs &a, cudaStream_t s)
{
    const CombineParams p = combine_params(a);
    if (a.k <= 4)
        return a.y_fp32 ? run_combine_grad<float, 4>(a, p, s) : run_combine_grad<__nv_bfloat16, 4>(a, p, s);
    return a.y_fp32 ? run_combine_grad<float, 8>(a, p, s) : run_combine_grad<__nv_bfloat16, 8>(a, p, s);
}

}  // namespace nvfp4
