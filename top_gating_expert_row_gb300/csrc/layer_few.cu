// The layer for a few pairs from the router's logits: few.cuh's two kernels
// with the routing of the call's tokens inside, for one (score function, logits
// dtype) pair per translation unit.
#include <algorithm>

#include "few.cuh"

#ifndef MR_SCORE_FN
#error "MR_SCORE_FN must be defined (0 softmax, 1 sigmoid)"
#endif
#ifndef MR_IN_BF16
#error "MR_IN_BF16 must be defined (0 fp32, 1 bf16)"
#endif

#define MR_CAT2(a, b) a##b
#define MR_CAT(a, b) MR_CAT2(a, b)
#define MR_SUFFIX MR_CAT(MR_CAT(_s, MR_SCORE_FN), MR_CAT(_d, MR_IN_BF16))

namespace mr {

#if MR_IN_BF16
using InT = __nv_bfloat16;
#else
using InT = float;
#endif

// Each CTA routes every token: warp w tokens w, w + 8, ... by the repeated
// arg-max, whose results are the threshold select's bit for bit.
template <int NV, bool FULL, bool DOWN>
__global__ void __launch_bounds__(kFewThreads, 2) k_layer_few(RouteArgs r, FewArgs a)
{
    extern __shared__ __align__(16) unsigned char smem[];
    few_body<DOWN>(a, smem, [&](int32_t* s_idx, float* s_w) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        const WarpLayout L = warp_layout(r.k_r, r.stop, r.E, false, r.n_group > 0);
        unsigned char* wsm = smem + few_pairs_bytes(a.T * a.topk) +
                             align16(DOWN ? a.T * a.topk * a.I * 4 : a.T * a.H * 2) + static_cast<size_t>(warp) * L.bytes;
        for (int t = warp; t < a.T; t += kFewWarps) {
            uint32_t warm = 0u;
            const float scale = route_row<MR_SCORE_FN, InT, NV, false, FULL>(r, t, wsm, L, lane, warm);
            const uint32_t* win_idx = reinterpret_cast<const uint32_t*>(wsm + L.win_idx);
            const float* win_val = reinterpret_cast<const float*>(wsm + L.win_val);
            for (int j = lane; j < a.topk; j += 32) {
                const bool routed = j < r.k_r;
                const int32_t id = routed ? static_cast<int32_t>(win_idx[j]) : r.E + (j - r.k_r);
                const float wv = routed ? __fmul_rn(win_val[j], scale) : r.shared_weight;
                const int o = t * a.topk + j;
                s_idx[o] = id;
                s_w[o] = wv;
                if (!DOWN && blockIdx.x == 0) {
                    if (a.idx_out) a.idx_out[o] = id;
                    if (a.w_out) a.w_out[o] = wv;
                }
            }
            __syncwarp();
        }
    });
}

int MR_CAT(launch_layer_few, MR_SUFFIX)(const RouteArgs& r, const FewArgs& a, int nv_idx, bool down, cudaStream_t st)
{
    using Fn = void (*)(RouteArgs, FewArgs);
    const bool full = r.vec && r.E == 128 * kNvBuckets[nv_idx];
    Fn f = nullptr;
#define MR_FEW(NV)                                                                                        \
    case NV:                                                                                              \
        f = down ? (full ? k_layer_few<NV, true, true> : k_layer_few<NV, false, true>)                    \
                 : (full ? k_layer_few<NV, true, false> : k_layer_few<NV, false, false>);                 \
        break;
    switch (kNvBuckets[nv_idx]) {
        MR_FEW(1)
        MR_FEW(2)
        MR_FEW(3)
        MR_FEW(4)
        MR_FEW(6)
        MR_FEW(8)
    }
#undef MR_FEW
    if (!f) return cudaErrorInvalidValue;
    const WarpLayout L = warp_layout(r.k_r, r.stop, r.E, false, r.n_group > 0);
    const size_t smem = few_smem(a, down, static_cast<size_t>(L.bytes) * std::min(a.T, kFewWarps));
    const int e = ensure_smem(reinterpret_cast<const void*>(f), smem);
    if (e != cudaSuccess) return e;
    const long long tasks = down ? static_cast<long long>(a.T) * a.H
                                 : static_cast<long long>(a.T) * a.topk * ((a.I + few_rows(a.H) - 1) / few_rows(a.H));
    const int grid = persistent_grid(reinterpret_cast<const void*>(f), kFewThreads, smem, (tasks + kFewWarps - 1) / kFewWarps);
    if (grid < 1) return cudaErrorLaunchOutOfResources;
    return launch_kernel(f, dim3(grid), dim3(kFewThreads), smem, st, 0, r, a);
}

}  // namespace mr
