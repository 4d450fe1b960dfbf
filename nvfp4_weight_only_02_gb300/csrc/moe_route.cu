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
    return v > -INFINITY ? (u & 0x80000000u ? ~u : u | 0x80000000u) : 0u;
}

// One token by one warp.  kPer values a lane: expert lane + 32 i.
template <int kPer>
__device__ __forceinline__ void route_token(const RouteParams &p, int64_t t, int lane)
{
    float z[kPer];
#pragma unroll
    for (int i = 0; i < kPer; i++) {
        const int e = lane + 32 * i;
        z[i] = e < p.E ? load_z(p.z, p.z_fp32, t * p.ldz + e) : -INFINITY;
    }
    bool nan = false;   // the softmax of the row has no value
#pragma unroll
    for (int i = 0; i < kPer; i++)
        nan |= z[i] != z[i] || (!p.sigmoid && z[i] == INFINITY);
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
#pragma unroll
    for (int i = 0; i < kPer; i++) {
        float v = z[i];
        const int e = lane + 32 * i;
        if (p.bias && e < p.E && v > -INFINITY)
            v = (p.sigmoid ? sigmoid(v) : expf(v - zmax) / denom) + p.bias[e];
        key[i] = key_of(v);
    }
    int mine = -1;   // lane j: expert of slot j
    for (int j = 0; j < p.k; j++) {
        uint32_t best = 0;
        int at = 0;
#pragma unroll
        for (int i = 0; i < kPer; i++)
            if (key[i] > best) {
                best = key[i];
                at = i;
            }
        const uint32_t top = __reduce_max_sync(kAll, best);
        if (top == 0)
            break;
        const uint32_t idx = __reduce_min_sync(kAll, best == top ? (uint32_t)(lane + 32 * at) : kAll);
        if ((idx & 31) == (uint32_t)lane) {
#pragma unroll
            for (int i = 0; i < kPer; i++)
                if (i == (int)(idx >> 5))
                    key[i] = 0;
        }
        if (lane == j)
            mine = (int)idx;
    }
    const float zj = mine >= 0 ? load_z(p.z, p.z_fp32, t * p.ldz + mine) : -INFINITY;
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

__device__ __forceinline__ void route_any(const RouteParams &p, int64_t t, int lane)
{
    if (p.E <= 64)
        route_token<2>(p, t, lane);
    else if (p.E <= 128)
        route_token<4>(p, t, lane);
    else if (p.E <= 256)
        route_token<8>(p, t, lane);
    else if (p.E <= 512)
        route_token<16>(p, t, lane);
    else
        route_token<32>(p, t, lane);
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
        int w[3] = {s_warp[lane][0], s_warp[lane][1], s_warp[lane][2]};
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

// kFirst: experts (where there are logits) and the CTA's counts.  kSecond:
// offsets, lists and the slots' places.  Both: one CTA does it all.
template <bool kFirst, bool kSecond>
__global__ void __launch_bounds__(kRtThreads) route_kernel(const RouteParams p)
{
    extern __shared__ uint16_t s_hist[];            // [warps][E]
    __shared__ int s_base[kMoeMaxExperts];          // row of the expert's first slot of this CTA
    __shared__ int s_off[kMoeMaxExperts + 1], s_fb[kMoeMaxExperts + 1], s_ft[kMoeMaxExperts + 1];
    __shared__ int s_warp[kRtWarps][3];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t t0 = (int64_t)blockIdx.x * p.chunk, t1 = min(p.T, t0 + p.chunk);
    int32_t *counts = p.plan + p.counts;
    if (kSecond && !kFirst)
        pdl_wait();
    pdl_launch_dependents();
    if (kFirst && !kSecond)
        pdl_wait();     // the buffers may be in use by the kernel before
    if (kFirst && kSecond)
        pdl_wait();
    if (kFirst && p.z) {
        for (int64_t t = t0 + warp; t < t1; t += kRtWarps)
            route_any(p, t, lane);
    }
    for (int i = tid; i < kRtWarps * p.E; i += kRtThreads)
        s_hist[i] = 0;
    __syncthreads();
    // this warp's run of the CTA's slots
    const int64_t c0 = t0 * p.k, c1 = t1 * p.k;
    const int64_t per = (c1 - c0 + 32 * kRtWarps - 1) / (32 * kRtWarps) * 32;
    const int64_t s0 = min(c1, c0 + warp * per), s1 = min(c1, s0 + per);
    uint16_t *hist = s_hist + warp * p.E;
    bool bad = false;
    each_slot(p, s0, s1, lane, [&](int64_t s, int e, int rank, bool last) {
        if (kFirst && !p.z && s < s1)
            bad |= p.experts[s] >= p.E;
        if (e >= 0 && last)
            hist[e] += rank + 1;
    });
    if (bad && p.ctl)
        record_status(p.ctl, NVFP4_ERR_INDEX);
    __syncthreads();
    // per expert: counts of the warps before, and the CTA's
    int n = 0;
    if (tid < p.E) {
        for (int w = 0; w < kRtWarps; w++) {
            const int c = s_hist[w * p.E + tid];
            s_hist[w * p.E + tid] = (uint16_t)n;
            n += c;
        }
    }
    if (!kSecond) {
        if (tid < p.E)
            counts[(int64_t)blockIdx.x * p.E + tid] = n;
        return;
    }
    int before = 0, total = n;
    if (!kFirst) {
        // counts of the other CTAs; the threads share out the CTAs where there are few experts
        __shared__ int s_before[kMoeMaxExperts], s_total[kMoeMaxExperts];
        s_before[tid] = s_total[tid] = 0;
        __syncthreads();
        const int width = (p.E + 31) / 32 * 32, groups = kRtThreads / width, g = tid / width, e = tid % width;
        if (g < groups && e < p.E) {
            int b = 0, all = 0;
            for (int c = g; c < (int)gridDim.x; c += groups) {
                const int v = counts[(int64_t)c * p.E + e];
                all += v;
                b += c < (int)blockIdx.x ? v : 0;
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
    if (tid >= p.E)
        total = 0;
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
        for (int e = tid; e <= p.E; e += kRtThreads) {
            p.plan[p.offsets + e] = s_off[e];
            p.plan[p.first_block + e] = s_fb[e];
        }
        if (tid < kMoeHeader)
            p.plan[tid] = tid == kMoeRows ? rows : tid == kMoeBlocks ? s_fb[p.E] : tid == kMoeTiles ? s_ft[p.E]
                          : tid == kMoeTileRows ? p.tile_rows : 0;
    }
    // lists of blocks and tiles: expert, first row of the padded and of the compact order, rows
    int4 *blocks = reinterpret_cast<int4 *>(p.plan + p.blocks), *tiles = reinterpret_cast<int4 *>(p.plan + p.tiles);
    for (int e = (int)blockIdx.x * kRtWarps + warp; e < p.E; e += (int)gridDim.x * kRtWarps) {
        const int ne = s_off[e + 1] - s_off[e];
        for (int b = lane; b < s_fb[e + 1] - s_fb[e]; b += 32)
            blocks[s_fb[e] + b] = make_int4(e, (s_fb[e] + b) * kMoeBlock, s_off[e] + b * kMoeBlock,
                                            min(kMoeBlock, ne - b * kMoeBlock));
        for (int b = lane; b < s_ft[e + 1] - s_ft[e]; b += 32)
            tiles[s_ft[e] + b] = make_int4(e, s_fb[e] * kMoeBlock + b * p.tile_rows, s_off[e] + b * p.tile_rows,
                                           min(p.tile_rows, ne - b * p.tile_rows));
    }
    for (int64_t r = rows + (int64_t)blockIdx.x * kRtThreads + tid; r < p.slots; r += (int64_t)gridDim.x * kRtThreads)
        p.plan[p.order + r] = -1;
    // places: hist holds the counts of the warps before, and counts on
    each_slot(p, s0, s1, lane, [&](int64_t s, int e, int rank, bool last) {
        int pos = -1, pad = -1;
        if (e >= 0) {
            const int h = hist[e];
            pos = s_base[e] + h + rank;
            pad = s_fb[e] * kMoeBlock + pos - s_off[e];
        }
        __syncwarp();
        if (e >= 0) {
            if (last)
                hist[e] += rank + 1;
            p.plan[p.order + pos] = (int32_t)s;
        }
        if (s < s1) {
            p.plan[p.position + s] = pos;
            p.plan[p.padded + s] = pad;
        }
    });
}

// dz of the router, a warp a token.
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

__global__ void __launch_bounds__(256) route_grad_kernel(const RouteGradParams p)
{
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (t >= p.T)
        return;
    int e = -1;
    float w = 0.0f, dw = 0.0f, g = 0.0f;
    if (lane < p.k) {
        e = p.experts[t * p.k + lane];
        if (e >= p.E)
            e = -1;
        w = p.weights[t * p.k + lane];
        dw = p.dw[t * p.k + lane];
    }
    const bool none = e < 0;
    const bool softmax_all = !p.sigmoid && !p.renorm;
    // a NaN weight reaches the gradient of its row, an unused slot's dw does not
    const float dot = p.renorm || softmax_all ? warp_sum(none ? w * 0.0f : w * dw) : 0.0f;
    if (!none) {
        if (p.renorm) {
            // w = scale u: scale u (dw - sum u dw) = w dw - w (sum w dw) / scale
            g = w * (dw - (p.scale != 0.0f ? dot / p.scale : 0.0f));
            if (p.sigmoid)
                g *= sigmoid(-load_z(p.z, p.z_fp32, t * p.ldz + e));
        } else if (p.sigmoid) {
            g = w * dw * sigmoid(-load_z(p.z, p.z_fp32, t * p.ldz + e));
        } else {
            g = w * dw;
        }
    }
    float zmax = -INFINITY, denom = 0.0f;
    if (softmax_all) {
        for (int i = lane; i < p.E; i += 32)
            zmax = fmaxf(zmax, load_z(p.z, p.z_fp32, t * p.ldz + i));
        zmax = warp_max(zmax);
        for (int i = lane; i < p.E; i += 32) {
            const float z = load_z(p.z, p.z_fp32, t * p.ldz + i);
            denom += z == -INFINITY ? 0.0f : expf(z - zmax);
        }
        denom = warp_sum(denom);
    }
    for (int i0 = 0; i0 < p.E; i0 += 32) {
        const int i = i0 + lane;
        float v = dot != dot ? dot : 0.0f;
        if (softmax_all && i < p.E) {
            const float z = load_z(p.z, p.z_fp32, t * p.ldz + i);
            v = z == -INFINITY ? 0.0f : -expf(z - zmax) / denom * dot;
        }
        for (int j = 0; j < p.k; j++) {
            const int ej = __shfl_sync(kAll, e, j);
            const float gj = __shfl_sync(kAll, g, j);
            if (ej == i)
                v += gj;
        }
        if (i < p.E) {
            if (p.z_fp32)
                reinterpret_cast<float *>(p.dz)[t * p.lddz + i] = v;
            else
                reinterpret_cast<__nv_bfloat16 *>(p.dz)[t * p.lddz + i] = __float2bfloat16_rn(v);
        }
    }
}

// ---------------------------------------------------------------- combine
// kVec elements of a row at a time: 16 bytes of the wider type's partner or,
// where rows do not start on 16-byte boundaries, single elements.
template <typename T, int kVec>
__device__ __forceinline__ void load_vec(const T *src, float (&v)[kVec])
{
    if constexpr (kVec == 1) {
        v[0] = (float)src[0];
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

template <typename T, int kVec>
__device__ __forceinline__ void store_vec(T *dst, const float (&v)[kVec])
{
    if constexpr (kVec == 1) {
        if constexpr (sizeof(T) == 2)
            dst[0] = __float2bfloat16_rn(v[0]);
        else
            dst[0] = v[0];
    } else if constexpr (sizeof(T) == 2) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
        for (int i = 0; i < kVec; i += 4)
            *reinterpret_cast<float4 *>(dst + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    }
}

struct CombineParams {
    const void *y, *base, *dout;
    const float *weights;
    const int32_t *position;
    void *out, *dy;
    float *dw;
    int64_t T;
    int N, k;
};

// out[t] = base[t] + sum_j w[t][j] y[position[t][j]], in FP32, j ascending.
template <typename TY, typename TO, int kVec>
__global__ void __launch_bounds__(256) combine_kernel(const CombineParams p)
{
    pdl_wait();
    pdl_launch_dependents();
    const int nv = p.N / kVec;
    const int64_t n = p.T * nv, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n)
        return;
    const int64_t t = i / nv;
    const int c = (int)(i % nv) * kVec;
    float acc[kVec];
#pragma unroll
    for (int e = 0; e < kVec; e++)
        acc[e] = 0.0f;
    if (p.base)
        load_vec<TO, kVec>(reinterpret_cast<const TO *>(p.base) + t * p.N + c, acc);
    const TY *y = reinterpret_cast<const TY *>(p.y) + c;
    for (int j0 = 0; j0 < p.k; j0 += 4) {
        float v[4][kVec], w[4];
        int pos[4];
#pragma unroll
        for (int j = 0; j < 4; j++) {
            pos[j] = -1;
            w[j] = 0.0f;
            if (j0 + j < p.k) {
                pos[j] = p.position[t * p.k + j0 + j];
                w[j] = p.weights ? p.weights[t * p.k + j0 + j] : 1.0f;
            }
        }
#pragma unroll
        for (int j = 0; j < 4; j++) {
#pragma unroll
            for (int e = 0; e < kVec; e++)
                v[j][e] = 0.0f;
            if (pos[j] >= 0)
                load_vec<TY, kVec>(y + (int64_t)pos[j] * p.N, v[j]);
        }
#pragma unroll
        for (int j = 0; j < 4; j++)
#pragma unroll
            for (int e = 0; e < kVec; e++)
                acc[e] = fmaf(w[j], v[j][e], acc[e]);
    }
    store_vec<TO, kVec>(reinterpret_cast<TO *>(p.out) + t * p.N + c, acc);
}

// dy[position[t][j]] = w[t][j] dout[t], dw[t][j] = <dout[t], y[position[t][j]]>: a CTA a token.
template <typename T, int kVec>
__global__ void __launch_bounds__(256) combine_grad_kernel(const CombineParams p)
{
    __shared__ float s_part[8][kMoeMaxK];
    const int64_t t = blockIdx.x;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const T *dout = reinterpret_cast<const T *>(p.dout) + t * p.N;
    for (int j = 0; j < p.k; j++) {
        const int pos = p.position[t * p.k + j];
        float dot = 0.0f;
        if (pos >= 0) {
            const T *y = reinterpret_cast<const T *>(p.y) + (int64_t)pos * p.N;
            T *dy = reinterpret_cast<T *>(p.dy) + (int64_t)pos * p.N;
            const float w = p.weights[t * p.k + j];
            for (int c = tid * kVec; c < p.N; c += 256 * kVec) {
                float d[kVec], v[kVec];
                load_vec<T, kVec>(dout + c, d);
                if (p.dw)
                    load_vec<T, kVec>(y + c, v);
#pragma unroll
                for (int e = 0; e < kVec; e++) {
                    if (p.dw)
                        dot = fmaf(d[e], v[e], dot);
                    d[e] *= w;
                }
                if (p.dy)
                    store_vec<T, kVec>(dy + c, d);
            }
        }
        dot = warp_sum(dot);
        if (lane == 0)
            s_part[warp][j] = dot;
    }
    __syncthreads();
    if (p.dw && tid < p.k) {
        float s = 0.0f;
        for (int w = 0; w < 8; w++)
            s += s_part[w][tid];
        p.dw[t * p.k + tid] = s;
    }
}

constexpr size_t kRtMaxSmem = (size_t)kRtWarps * kMoeMaxExperts * 2;

template <typename TY, typename TO>
cudaError_t run_combine(const MoeCombineArgs &a, const CombineParams &p, cudaStream_t s)
{
    const bool vec = a.N % 8 == 0;
    const int64_t n = a.T * (vec ? a.N / 8 : a.N);
    const unsigned grid = (unsigned)((n + 255) / 256);
    return vec ? launch_dependent(combine_kernel<TY, TO, 8>, grid, 256, 0, s, p)
               : launch_dependent(combine_kernel<TY, TO, 1>, grid, 256, 0, s, p);
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
    const size_t smem = (size_t)kRtWarps * a.E * 2;
    if (l.ctas == 1) {
        const cudaError_t e = allow_smem<route_kernel<true, true>>(kRtMaxSmem, dev);
        return e != cudaSuccess ? e : launch_dependent(route_kernel<true, true>, 1, kRtThreads, smem, s, p);
    }
    cudaError_t e = allow_smem<route_kernel<true, false>>(kRtMaxSmem, dev);
    if (e == cudaSuccess)
        e = allow_smem<route_kernel<false, true>>(kRtMaxSmem, dev);
    if (e == cudaSuccess)
        e = launch_dependent(route_kernel<true, false>, (unsigned)l.ctas, kRtThreads, smem, s, p);
    if (e == cudaSuccess)
        e = launch_dependent(route_kernel<false, true>, (unsigned)l.ctas, kRtThreads, smem, s, p);
    return e;
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
    route_grad_kernel<<<(unsigned)((a.T + 7) / 8), 256, 0, s>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_moe_combine(const MoeCombineArgs &a, cudaStream_t s)
{
    const CombineParams p = combine_params(a);
    if (a.y_fp32)
        return a.out_fp32 ? run_combine<float, float>(a, p, s) : run_combine<float, __nv_bfloat16>(a, p, s);
    return a.out_fp32 ? run_combine<__nv_bfloat16, float>(a, p, s) : run_combine<__nv_bfloat16, __nv_bfloat16>(a, p, s);
}

cudaError_t launch_moe_combine_backward(const MoeCombineArgs &a, cudaStream_t s)
{
    const CombineParams p = combine_params(a);
    const bool vec = a.N % 8 == 0;
    const unsigned grid = (unsigned)a.T;
    if (a.y_fp32) {
        if (vec)
            combine_grad_kernel<float, 8><<<grid, 256, 0, s>>>(p);
        else
            combine_grad_kernel<float, 1><<<grid, 256, 0, s>>>(p);
    } else if (vec) {
        combine_grad_kernel<__nv_bfloat16, 8><<<grid, 256, 0, s>>>(p);
    } else {
        combine_grad_kernel<__nv_bfloat16, 1><<<grid, 256, 0, s>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace nvfp4
