// Shared by the translation units of the layer behind the router.
#pragma once

#include <cuda.h>

#include "internal.h"
#include "moe_router.h"

namespace mr {

// act(g) in fp32: SiLU g / (1 + exp(-g)), or GELU g * Phi(g). The hardware's
// base-2 exponential and reciprocal are off by a few units of the last place (the
// exponential by |g| / 2 of them more), below the 16 bits that h keeps. Phi(g) is
// erfc(-g / sqrt 2) / 2, which keeps them for g below zero as well (1 + erf(g /
// sqrt 2) cancels: 10 bits at -4, none below -5.5); the rounding of its argument
// enters the value g^2 times, 2^-17 at g = -8.
__device__ __forceinline__ float act_f32(float g, int act)
{
    if (act == MR_SILU) return __fdividef(g, 1.0f + exp2_hw(-g * kLog2e));
    return 0.5f * g * erfcf(-g * 0.70710678118654752f);
}

// v as hi + lo, two bf16 (their bits), to 16 significant bits: hi is v cut off, lo
// the rest rounded; v that has no rest, or is an infinity, is halved instead. So
// both parts have v's sign and neither is zero unless v is (or is below 2^-100):
// an infinite weight times either is the same infinity, the one of w * v. (Of hi
// rounded to nearest, which would spare one bit more, the rest has the other sign
// half of the time, and inf - inf and inf * 0 are NaN. A tiny stand-in for a rest
// of zero costs exact sums their last bit: the tensor cores cut off, they do not
// round.)
__device__ __forceinline__ void split_f32(float v, uint32_t& hi, uint32_t& lo)
{
    const uint32_t bits = __float_as_uint(v);
    const float rest = v - __uint_as_float(bits & 0xffff0000u);  // exact; NaN for an infinity
    if (fabsf(rest) > 0.0f) {
        hi = bits >> 16;
        lo = __bfloat16_as_ushort(__float2bfloat16_rn(rest));
    } else {
        hi = lo = __float_as_uint(0.5f * v) >> 16;
    }
}

// Waits on copies in flight when a CTA gives up (attempts of about a microsecond).
constexpr uint32_t kDrainTries = 1u << 14;

// What the experts' kernels work on (device pointers; the sorted layout with
// blocks of nt pairs).
struct ExpertArgs {
    const __nv_bfloat16* x;  // [T][H]
    __nv_bfloat16* xs;     // [cap][H] rows of x in sorted order, where blocks are wide
    const int32_t* sids;   // sorted pair ids, P at sentinels
    const int32_t* eids;   // expert of each block
    const int32_t* npp;    // rows of the sorted layout
    const int32_t* idx;    // [T][topk]
    const float* w;        // [T][topk]
    __nv_bfloat16* h;      // [cap][I], in sorted order (narrow blocks: hi, then lo)
    float* y;              // [T * topk][H], weighted
    __nv_bfloat16* out;    // [T][H]
    int32_t* status;
    int T, topk, H, I, E, P, cap;
    int mt;                // row tiles of this kernel
    int stages, act, drop;
    int out16;             // out allows 16-byte stores
    uint32_t tries;
};

// Blocks of this many pairs or more read x from a copy in sorted order.
constexpr int kGatherColumns = 32;
// Blocks of at most this many pairs keep h as two bf16 parts (16 significant bits):
// up to 128 columns a product takes 70 clocks, so twice 64 cost nothing. Wider
// blocks round h to bf16, as x and the weights are. Two parts would cost blocks of
// 128 4 to 5% (T=512 E=32 k=4 H=2048 I=1024 100 -> 105 us, graph); blocks of 256 have
// no tensor memory for them and would have to be blocks of 128 (T=2048 E=64 k=4 198
// -> 220, T=8192 E=8 k=2 H=I=2048 320 -> 497). The error against 64 bits is 2.3e-3 of
// the output's norm there and 1.7e-3, the output's own rounding, with two parts.
constexpr int kSplitColumns = 64;
// Rows of one copy of the token operand.
inline int token_box(int nt) { return nt >= 64 ? nt / 4 : 16; }

int launch_experts_gather(const ExpertArgs& a, cudaStream_t st);
int launch_experts_sum(const ExpertArgs& a, cudaStream_t st);
int launch_experts_up(int nt, const CUtensorMap& map_w, const CUtensorMap& map_t, const ExpertArgs& a, long long units,
                      cudaStream_t st);
int launch_experts_down(int nt, const CUtensorMap& map_w, const CUtensorMap& map_t, const ExpertArgs& a,
                        long long units, cudaStream_t st);

// What the adapter projection's kernels work on.
struct AdapterArgs {
    const __nv_bfloat16* b;    // [n_adapters][N][rank]
    const int32_t* adapter;    // [T]
    const float* scale;        // [n_adapters] or null
    float* low;                // [slices][T][rank] rank-space values, scaled
    int32_t* same;             // wide tiles: the adapter of all the tile's tokens, or -1
    __nv_bfloat16* split;      // wide tiles: [T][ranks / 32][hi of 32 ranks, lo of them]
    void* out;                 // [T][N]
    int32_t* status;           // timeouts
    int32_t* range_status;     // ids past the adapters (nullable)
    int T, K, N, n_adapters, rank;
    int tiles;                 // of at most nt tokens
    int mt;                    // row tiles
    int ways;                  // CTAs (a cluster) that share the sum over K of a unit
    int slices;                // of K, in k_adapter_low
    int stages, stages_low, drop;
    uint32_t tries;
};

int launch_adapter_low(int nt, const CUtensorMap& map_a, const CUtensorMap& map_x, const AdapterArgs& a, int groups,
                       cudaStream_t st);
int launch_adapter_low_rows(const void* x, const void* wa, const AdapterArgs& a, cudaStream_t st);
int launch_adapter_few(const void* x, const void* w, const void* wa, bool fused, bool f32, const AdapterArgs& a,
                       cudaStream_t st);
int launch_adapter_split(int nt, const AdapterArgs& a, cudaStream_t st);
int launch_adapter_proj(int nt, bool f32, const CUtensorMap& map_w, const CUtensorMap& map_x, const CUtensorMap& map_b,
                        const CUtensorMap& map_s, const AdapterArgs& a, cudaStream_t st);

// A tensor map of bf16 [planes][height][width] (planes 0: a matrix) with boxes
// of box_h rows by 64 columns, 128-byte swizzled; elements outside read as 0.
bool encode_map(CUtensorMap* m, const void* base, long long width, long long height, long long planes, int box_h);

// The validation of the forward calls' options, the per-device status word and
// the wait-test settings (api.cu).
int router_check(const mr_router_params* p);
RouteArgs router_args(const mr_router_params* p, const void* logits);
bool router_forced_select();
int32_t* status_word(int32_t* status);
void wait_test(uint32_t* tries, int* drop);

}  // namespace mr
