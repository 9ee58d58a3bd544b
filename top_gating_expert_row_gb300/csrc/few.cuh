// The layer for a few pairs (decode of one to a few tokens), on the CUDA cores
// and without a sort: two launches, a warp per row of the weights.
//
//   up    h[p][i] = act(w13[e][i] . x_t) * (w13[e][I + i] . x_t)
//   down  out[t][c] = sum_j weight[t][j] * (w2[e_j][c] . h[t][j])
//
// k_experts_few (experts.cu) is either for a given choice of experts, k_layer_few
// (layer_few.cu) with the routing.
//
// A pair's product is a matrix-vector one: each weight is used once, two
// operations a weight, so the time is that of streaming the weights, and what
// is left to save is latency. Hence no tensor memory, no barriers, no counters:
// a warp of `down` holds a whole output element, and both kernels route the
// tokens themselves (each CTA all of them: they are few, and it costs what
// waiting for another launch would). `down` starts beside `up`, brings its
// weights to L2 meanwhile and waits only for h.
//
// Measured (CUDA graph, states that do not fit L2): T=1 E=256 k=8 H=2048 I=768 22.0
// us for 75 MB, 11.1 at the memory's rate; about 2 us of it routing, the rest
// that a warp holds one row pair's loads in flight and has two or three pairs one
// after the other. T=1 E=8 k=2 H=512 I=256 6.6 us, all latency.
#pragma once

#include "experts.h"
#include "route.cuh"

namespace mr {

constexpr int kFewThreads = 256;
constexpr int kFewWarps = kFewThreads / 32;

struct FewArgs {
    const __nv_bfloat16* x;
    const __nv_bfloat16* w13;
    const __nv_bfloat16* w2;
    float* h;               // [P][I]: few enough values to keep them unrounded
    __nv_bfloat16* out;
    const int32_t* idx;     // given choice (no routing)
    const float* w;
    int32_t* idx_out;       // the routing's outputs (nullable)
    float* w_out;
    int32_t* status;        // MR_ERANGE (nullable)
    int T, topk, H, I, E, act;
};

__host__ __device__ inline int few_pairs_bytes(int P) { return align16(P * 4) * 2; }


// a . b over 8 bf16 each, added to s.
__device__ __forceinline__ float dot8(uint4 a, uint4 b, float s)
{
    const uint32_t p[4] = {a.x, a.y, a.z, a.w}, q[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        s = fmaf(__uint_as_float(p[i] << 16), __uint_as_float(q[i] << 16), s);
        s = fmaf(__uint_as_float(p[i] & 0xffff0000u), __uint_as_float(q[i] & 0xffff0000u), s);
    }
    return s;
}

__device__ __forceinline__ float dot8(uint4 a, const float4* b, float s)
{
    const uint32_t p[4] = {a.x, a.y, a.z, a.w};
    const float4 u = b[0], v = b[1];
    s = fmaf(__uint_as_float(p[0] << 16), u.x, s);
    s = fmaf(__uint_as_float(p[0] & 0xffff0000u), u.y, s);
    s = fmaf(__uint_as_float(p[1] << 16), u.z, s);
    s = fmaf(__uint_as_float(p[1] & 0xffff0000u), u.w, s);
    s = fmaf(__uint_as_float(p[2] << 16), v.x, s);
    s = fmaf(__uint_as_float(p[2] & 0xffff0000u), v.y, s);
    s = fmaf(__uint_as_float(p[3] << 16), v.z, s);
    return fmaf(__uint_as_float(p[3] & 0xffff0000u), v.w, s);
}

// Weights are read once: past L1.
__device__ __forceinline__ uint4 load_weights(const uint4* p)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

// h of every pair; x in shared memory. A warp takes ROWS neighbouring rows at a
// time, so that short rows (H of 1024 and less) keep as many loads in flight.
template <int ROWS>
__device__ __forceinline__ void few_up(const FewArgs& a, const int32_t* s_idx, const unsigned char* s_x)
{
    constexpr int kChunks = 8 / ROWS;  // 16-byte chunks of each row in flight a lane
    const int lane = threadIdx.x & 31, P = a.T * a.topk, H8 = a.H / 8, groups = (a.I + ROWS - 1) / ROWS;
    const int warps = gridDim.x * kFewWarps;
    for (int u = blockIdx.x * kFewWarps + (threadIdx.x >> 5); u < P * groups; u += warps) {
        const int p = u / groups, i0 = (u - p * groups) * ROWS;
        const int e = s_idx[p];
        if (e < 0 || e >= a.E) continue;
        const uint4* g = reinterpret_cast<const uint4*>(a.w13 + (static_cast<long long>(e) * 2 * a.I + i0) * a.H);
        const uint4* v = g + static_cast<long long>(a.I) * H8;
        const uint4* x = reinterpret_cast<const uint4*>(s_x) + p / a.topk * H8;
        float sg[ROWS] = {}, sv[ROWS] = {};
        for (int c0 = lane; c0 < H8; c0 += 32 * kChunks) {
            uint4 wg[kChunks][ROWS], wv[kChunks][ROWS];
#pragma unroll
            for (int c = 0; c < kChunks; ++c)
#pragma unroll
                for (int r = 0; r < ROWS; ++r)
                    if (c0 + c * 32 < H8 && i0 + r < a.I) {
                        wg[c][r] = load_weights(g + r * H8 + c0 + c * 32);
                        wv[c][r] = load_weights(v + r * H8 + c0 + c * 32);
                    }
#pragma unroll
            for (int c = 0; c < kChunks; ++c)
                if (c0 + c * 32 < H8) {
                    const uint4 xc = x[c0 + c * 32];
#pragma unroll
                    for (int r = 0; r < ROWS; ++r)
                        if (i0 + r < a.I) {
                            sg[r] = dot8(wg[c][r], xc, sg[r]);
                            sv[r] = dot8(wv[c][r], xc, sv[r]);
                        }
                }
        }
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            const float gs = warp_sum(sg[r]), vs = warp_sum(sv[r]);
            if (lane == 0 && i0 + r < a.I) a.h[static_cast<long long>(p) * a.I + i0 + r] = act_f32(gs, a.act) * vs;
        }
    }
}

__host__ __device__ inline int few_rows(int H) { return H <= 512 ? 4 : H <= 1024 ? 2 : 1; }

// This warp's weights of `down`, to L2.
__device__ __forceinline__ void few_down_prefetch(const FewArgs& a, const int32_t* s_idx)
{
    const int lane = threadIdx.x & 31, warps = gridDim.x * kFewWarps;
    for (long long u = static_cast<long long>(blockIdx.x) * kFewWarps + (threadIdx.x >> 5); u < static_cast<long long>(a.T) * a.H;
         u += warps) {
        const int t = static_cast<int>(u / a.H), c = static_cast<int>(u - static_cast<long long>(t) * a.H);
        for (int j = lane; j < a.topk; j += 32) {
            const int e = s_idx[t * a.topk + j];
            if (e >= 0 && e < a.E) prefetch_l2(a.w2 + (static_cast<long long>(e) * a.H + c) * a.I, a.I * 2);
        }
    }
}

// out of every token; h in shared memory.
__device__ __forceinline__ void few_down(const FewArgs& a, const int32_t* s_idx, const float* s_w, const unsigned char* s_h)
{
    constexpr int kChunks = 8;
    const int lane = threadIdx.x & 31, I8 = a.I / 8;
    const int warps = gridDim.x * kFewWarps;
    for (long long u = static_cast<long long>(blockIdx.x) * kFewWarps + (threadIdx.x >> 5); u < static_cast<long long>(a.T) * a.H;
         u += warps) {
        const int t = static_cast<int>(u / a.H), c = static_cast<int>(u - static_cast<long long>(t) * a.H);
        // the token's slots one after the other: step q is piece q % n of slot q / n
        const int n = (I8 + 31) / 32, steps = a.topk * n;
        int j = 0, piece = 0;
        float sum = 0.0f;
        for (int q = 0; q < steps; q += kChunks) {
            uint4 w[kChunks];
            int src[kChunks];
            float weight[kChunks];
#pragma unroll
            for (int k = 0; k < kChunks; ++k) {
                const int at = piece * 32 + lane, p = t * a.topk + j;
                const int e = q + k < steps ? s_idx[p] : -1;
                src[k] = e >= 0 && e < a.E && at < I8 ? p * I8 + at : -1;
                if (src[k] >= 0) {
                    weight[k] = s_w[p];
                    w[k] = load_weights(reinterpret_cast<const uint4*>(a.w2 + (static_cast<long long>(e) * a.H + c) * a.I) + at);
                }
                if (++piece == n) {
                    piece = 0;
                    ++j;
                }
            }
#pragma unroll
            for (int k = 0; k < kChunks; ++k)
                if (src[k] >= 0) sum = fmaf(weight[k], dot8(w[k], reinterpret_cast<const float4*>(s_h) + src[k] * 2, 0.0f), sum);
        }
        sum = warp_sum(sum);
        if (lane == 0) a.out[u] = __float2bfloat16_rn(sum);
    }
}

// Copies n16 16-byte pieces to shared memory.
__device__ __forceinline__ void few_stage(unsigned char* dst, const void* src, int n16)
{
    for (int i = threadIdx.x; i < n16; i += kFewThreads)
        reinterpret_cast<uint4*>(dst)[i] = __ldcg(reinterpret_cast<const uint4*>(src) + i);
}

// Shared memory: the pairs, then x (up) or h (down), then the routing's rows.
template <bool DOWN, typename Choose>
__device__ __forceinline__ void few_body(const FewArgs& a, unsigned char* smem, Choose choose)
{
    const int P = a.T * a.topk;
    int32_t* s_idx = reinterpret_cast<int32_t*>(smem);
    float* s_w = reinterpret_cast<float*>(smem + align16(P * 4));
    unsigned char* s_v = smem + few_pairs_bytes(P);
    if (!DOWN) {
        pdl_wait();
        pdl_trigger();
        few_stage(s_v, a.x, a.T * a.H / 8);
    }
    choose(s_idx, s_w);
    __syncthreads();
    if (!DOWN) {
        const int rows = few_rows(a.H);
        if (rows == 4) few_up<4>(a, s_idx, s_v);
        else if (rows == 2) few_up<2>(a, s_idx, s_v);
        else few_up<1>(a, s_idx, s_v);
    } else {
        few_down_prefetch(a, s_idx);
        pdl_trigger();
        pdl_wait();
        few_stage(s_v, a.h, P * a.I / 4);
        __syncthreads();
        few_down(a, s_idx, s_w, s_v);
    }
}

inline size_t few_smem(const FewArgs& a, bool down, size_t route_bytes)
{
    return few_pairs_bytes(a.T * a.topk) + static_cast<size_t>(align16(down ? a.T * a.topk * a.I * 4 : a.T * a.H * 2)) + route_bytes;
}

}  // namespace mr
