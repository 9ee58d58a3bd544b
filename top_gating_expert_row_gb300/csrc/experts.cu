// The layer behind the router: argument checks, path choice and launches of
// moe_experts_fwd, moe_layer_fwd and moe_adapter_proj_fwd, and their plain
// kernels (any size, any alignment).
#include <climits>
#include <cudaTypedefs.h>

#include <algorithm>

#include "few.cuh"

namespace mr {

// cuTensorMapEncodeTiled, from the driver that is loaded (the library itself
// links no driver); nullptr where there is none.
static PFN_cuTensorMapEncodeTiled_v12000 encode_function()
{
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult found = cudaDriverEntryPointSymbolNotFound;
        const cudaError_t e =
            cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found);
        return e == cudaSuccess && found == cudaDriverEntryPointSuccess
                   ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f)
                   : nullptr;
    }();
    return fn;
}

bool encode_map(CUtensorMap* m, const void* base, long long width, long long height, long long planes, int box_h)
{
    const auto fn = encode_function();
    if (!fn) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(height),
                                static_cast<cuuint64_t>(planes > 0 ? planes : 1)};
    const cuuint64_t strides[2] = {dims[0] * 2, dims[0] * dims[1] * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_h), 1};
    const cuuint32_t steps[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, planes > 0 ? 3 : 2, const_cast<void*>(base), dims, strides, box, steps,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// ---------------------------------------------------------------------------
// Plain kernels: a warp per output element, lanes over the summed index, fp32
// sums (each lane's in ascending order, then a fixed tree), no shared memory
// and no alignment beyond the element's. They serve rows that the tensor-core
// kernels' 16-byte copies cannot address.
// ---------------------------------------------------------------------------
__device__ __forceinline__ float value(const __nv_bfloat16* p)
{
    return bf16_bits_to_f32(__ldcg(reinterpret_cast<const unsigned short*>(p)));
}

__device__ __forceinline__ float value(const float* p) { return __ldcg(p); }

template <typename B>
__device__ __forceinline__ float warp_dot(const __nv_bfloat16* a, const B* b, int n, int lane)
{
    float s = 0.0f;
    for (int i = lane; i < n; i += 32) s = fmaf(value(a + i), value(b + i), s);
    return warp_sum(s);
}

// h[pair][i] = act(w13[e][i] . x[t]) * (w13[e][I + i] . x[t]); pairs without an expert are left out
__global__ void k_experts_up_plain(const __nv_bfloat16* x, const int32_t* idx, const __nv_bfloat16* w13,
                                   float* h, long long P, int topk, int H, int I, int E, int act,
                                   int32_t* status)
{
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const long long warps = static_cast<long long>(gridDim.x) * (blockDim.x >> 5);
    for (long long u = static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5); u < P * I;
         u += warps) {
        const long long pair = u / I;
        const int i = static_cast<int>(u - pair * I);
        const int e = __ldcg(idx + pair);
        if (e < 0 || e >= E) {
            if (i == 0 && lane == 0) report_status(status, kStatusRange);
            continue;
        }
        const __nv_bfloat16* row = x + pair / topk * H;
        const __nv_bfloat16* w = w13 + (static_cast<long long>(e) * 2 * I + i) * H;
        const float g = warp_dot(w, row, H, lane);
        const float v = warp_dot(w + static_cast<long long>(I) * H, row, H, lane);
        if (lane == 0) h[u] = act_f32(g, act) * v;
    }
}

// out[t][c] = sum_j weight[t][j] * (w2[e_j][c] . h[t][j])
__global__ void k_experts_down_plain(const float* h, const int32_t* idx, const float* weight,
                                     const __nv_bfloat16* w2, __nv_bfloat16* out, long long T, int topk, int H, int I,
                                     int E)
{
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const long long warps = static_cast<long long>(gridDim.x) * (blockDim.x >> 5);
    for (long long u = static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5); u < T * H;
         u += warps) {
        const long long t = u / H;
        const int c = static_cast<int>(u - t * H);
        float acc = 0.0f;
        for (int j = 0; j < topk; ++j) {
            const long long pair = t * topk + j;
            const int e = __ldcg(idx + pair);
            if (e < 0 || e >= E) continue;
            const float y = warp_dot(w2 + (static_cast<long long>(e) * H + c) * I, h + pair * I, I, lane);
            acc = fmaf(__ldcg(weight + pair), y, acc);
        }
        if (lane == 0) out[u] = __float2bfloat16_rn(acc);
    }
}

// s[t][q] = scale * (a[adapter][q] . x[t])
__global__ void k_adapter_low_plain(const __nv_bfloat16* x, const __nv_bfloat16* a, const int32_t* adapter,
                                    const float* scale, float* s, long long T, int K, int rank, int n_adapters,
                                    int32_t* status)
{
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const long long warps = static_cast<long long>(gridDim.x) * (blockDim.x >> 5);
    for (long long u = static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5); u < T * rank;
         u += warps) {
        const long long t = u / rank;
        const int q = static_cast<int>(u - t * rank);
        const int ad = __ldcg(adapter + t);
        if (ad >= n_adapters && q == 0 && lane == 0) report_status(status, kStatusRange);
        if (ad < 0 || ad >= n_adapters) continue;
        const float d = warp_dot(a + (static_cast<long long>(ad) * rank + q) * K, x + t * K, K, lane);
        if (lane == 0) s[u] = scale ? d * __ldcg(scale + ad) : d;
    }
}

template <typename OutT>
__global__ void k_adapter_proj_plain(const __nv_bfloat16* x, const __nv_bfloat16* w, const __nv_bfloat16* b,
                                     const int32_t* adapter, const float* s, OutT* out, long long T, int K, int N,
                                     int rank, int n_adapters)
{
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const long long warps = static_cast<long long>(gridDim.x) * (blockDim.x >> 5);
    for (long long u = static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5); u < T * N;
         u += warps) {
        const long long t = u / N;
        const int c = static_cast<int>(u - t * N);
        float acc = warp_dot(w + static_cast<long long>(c) * K, x + t * K, K, lane);
        const int ad = n_adapters > 0 ? __ldcg(adapter + t) : -1;
        if (ad >= 0 && ad < n_adapters) {
            const __nv_bfloat16* brow = b + (static_cast<long long>(ad) * N + c) * rank;
            float v = 0.0f;
            for (int q = lane; q < rank; q += 32) v = fmaf(value(brow + q), __ldcg(s + t * rank + q), v);
            acc += warp_sum(v);
        }
        if (lane == 0) store_scalar(out + u, acc);
    }
}

// ---- a few pairs ---------------------------------------------------------------------------------------------------

// few.cuh's kernels for a given choice of experts.
template <bool DOWN>
__global__ void __launch_bounds__(kFewThreads, 2) k_experts_few(FewArgs a)
{
    extern __shared__ __align__(16) unsigned char smem[];
    few_body<DOWN>(a, smem, [&](int32_t* s_idx, float* s_w) {
        for (int p = threadIdx.x; p < a.T * a.topk; p += kFewThreads) {
            const int e = __ldcg(a.idx + p);
            s_idx[p] = e;
            s_w[p] = __ldcg(a.w + p);
            if (!DOWN && blockIdx.x == 0 && (e < 0 || e >= a.E)) report_status(a.status, kStatusRange);
        }
    });
}

int launch_layer_few_s0_d0(const RouteArgs&, const FewArgs&, int, bool, cudaStream_t);
int launch_layer_few_s0_d1(const RouteArgs&, const FewArgs&, int, bool, cudaStream_t);
int launch_layer_few_s1_d0(const RouteArgs&, const FewArgs&, int, bool, cudaStream_t);
int launch_layer_few_s1_d1(const RouteArgs&, const FewArgs&, int, bool, cudaStream_t);

namespace {

constexpr int kPlainThreads = 256;

int plain_grid(const void* func, long long warps)
{
    return persistent_grid(func, kPlainThreads, 0, (warps + kPlainThreads / 32 - 1) / (kPlainThreads / 32));
}

int from_cuda(int e) { return e == cudaSuccess ? MR_OK : MR_ECUDA; }
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int check_experts(const mr_expert_params* p)
{
    if (!p) return MR_EINVAL;
    if (p->T < 0 || p->H < 1 || p->I < 1 || p->E < 1 || p->topk < 1) return MR_EINVAL;
    if (p->dtype != MR_F32 && p->dtype != MR_BF16) return MR_EINVAL;
    if (p->act != MR_SILU && p->act != MR_GELU) return MR_EINVAL;
    if (static_cast<long long>(p->T) * p->topk >= INT_MAX) return MR_EINVAL;
    if (p->dtype != MR_BF16) return MR_EUNSUPPORTED;
    if (p->H > MR_MAX_WIDTH || p->I > MR_MAX_WIDTH || p->E > MR_MAX_SORT_EXPERTS) return MR_EUNSUPPORTED;
    return MR_OK;
}

// The router's options as expert options (E_tot experts).
mr_expert_params layer_experts(const mr_router_params* p, int H, int I, int act)
{
    mr_expert_params q;
    q.T = p->T;
    q.H = H;
    q.I = I;
    q.E = p->E + p->n_shared;
    q.topk = p->topk;
    q.dtype = MR_BF16;
    q.act = act;
    return q;
}

int check_adapter(const mr_adapter_params* p)
{
    if (!p) return MR_EINVAL;
    if (p->T < 0 || p->K < 1 || p->N < 1 || p->n_adapters < 0 || (p->n_adapters > 0 && p->rank < 1)) return MR_EINVAL;
    if (p->dtype != MR_F32 && p->dtype != MR_BF16) return MR_EINVAL;
    if (p->out_dtype != MR_F32 && p->out_dtype != MR_BF16) return MR_EINVAL;
    if (p->dtype != MR_BF16) return MR_EUNSUPPORTED;
    if (p->K > MR_MAX_WIDTH || p->N > MR_MAX_WIDTH || (p->n_adapters > 0 && p->rank > MR_MAX_WIDTH))
        return MR_EUNSUPPORTED;
    return MR_OK;
}

// Workspace of the experts' products: offsets of its parts. The plain kernels
// use idx, w and h alone.
struct ExpertPlan {
    size_t idx, w, h, xs, sids, eids, npp, y, sort, sort_bytes, bytes;
    int nt, cap, mt_up, mt_down;
    bool tensor;  // the sizes allow the tensor-core kernels (else cap and the parts beyond h are 0)
};

// Rows of the sorted layout and units that the tensor-core kernels count in 32
// bits: a row index goes up by a grid's worth of warps past the last one, and is
// doubled where h has two parts; a unit goes up by the grid. Larger calls take
// the plain kernels, which count in 64.
constexpr size_t kMaxRows = (size_t(1) << 30) - (1 << 16);
constexpr long long kMaxUnits = INT_MAX - (1 << 16);

size_t part(size_t& o, size_t bytes)
{
    const size_t at = o;
    o += (bytes + 255) / 256 * 256;
    return at;
}

// Units that keep the SMs busy (one CTA each).
constexpr int kFullGrid = 148;

// Columns (pairs) of a block: four times the mean load of an expert that has any,
// up to 128, so that few experts need a second block (which reads their weights
// again); twice and eight times are slower (T=512 E=384+1 k=9 with skewed loads:
// 110 and 106 us against 104). A product only takes the columns that its block
// fills, so wide blocks cost shared memory, not time. 256, which pairs of CTAs
// take, from a mean of 112 on: at 100 113.9 us against 110.8 with 128 (E=32 k=2
// H=2048 I=1024), at 150 123.7 against 131.6.
int columns_for(long long P, int E)
{
    const long long active = std::min<long long>(P, E), load = (P + active - 1) / active;
    int nt = 16;
    while (nt < 128 && nt < 4 * load) nt *= 2;
    return load > 112 ? 256 : nt;
}

// route: the routing options when the call routes too (room for its outputs and workspace)
ExpertPlan expert_plan(const mr_expert_params& p, const mr_router_params* route)
{
    const size_t P = static_cast<size_t>(p.T) * p.topk;
    ExpertPlan w;
    w.nt = columns_for(static_cast<long long>(P), p.E);
    const size_t cap = moe_sort_capacity(p.T, p.topk, p.E, w.nt);
    w.mt_up = (p.I + 63) / 64;
    w.mt_down = (p.H + 127) / 128;
    // whole 16-byte rows, an expert's weights below 2^40 bytes, counts of 32 bits
    w.tensor = p.H % 8 == 0 && p.I % 8 == 0 && static_cast<long long>(p.I) * p.H < (1ll << 37) && cap <= kMaxRows &&
               static_cast<long long>(cap / w.nt + 1) * std::max(w.mt_up, w.mt_down) <= kMaxUnits;
    const size_t rows = w.tensor ? cap : 0;
    w.cap = static_cast<int>(rows);
    size_t o = 0;
    w.idx = part(o, route ? P * 4 : 0);
    w.w = part(o, route ? P * 4 : 0);
    w.sids = part(o, rows * 4);
    w.eids = part(o, w.tensor ? (rows / w.nt + 1) * 4 : 0);
    w.npp = part(o, w.tensor ? 4 : 0);
    w.sort_bytes = w.tensor ? moe_sort_workspace_bytes(p.T, p.topk, p.E, w.nt) : 0;
    if (route && w.tensor) w.sort_bytes = std::max(w.sort_bytes, moe_router_fused_workspace_bytes(route, w.nt));
    w.sort = part(o, w.sort_bytes);
    // few pairs and plain kernels: fp32; narrow blocks: two parts
    w.h = part(o, std::max(w.nt <= kSplitColumns ? 2 * rows : rows, 2 * P) * p.I * 2);
    w.xs = part(o, w.nt >= kGatherColumns ? rows * p.H * 2 : 0);
    w.y = part(o, w.tensor ? P * p.H * 4 : 0);
    w.bytes = o;
    return w;
}

// Few pairs: each pair's weights are read by itself, as fast as the tensor cores'
// path reads them up to about 100 MB and without its 5 us of set-up. Layers in a
// CUDA graph, this path against that one, us: at 8.4M products 17.8 / 22.2 (T=1 k=8
// H=2048), 16.4 / 20.8 (T=2 k=4 H=2048); at 12.6M 22.2 / 24.8, 21.4 / 23.4; at 16.8M
// 25.9 / 27.9, 25.1 / 26.8, 25.6 / 26.5 (T=4 k=4 H=1024), 23.1 / 22.9 (T=8 k=4
// H=512); at 15.7M 27.8 / 27.5 (T=1 k=4 H=2560); at 21.0M, past the border, 34.0 /
// 31.1 there, but 31.1 / 35.3 (T=1 k=8 H=2048). Eager calls save the host two launches
// (26 / 33) as long as that bounds them, up to about 17M.
constexpr int kFewPairs = 32, kFewTokens = 8;
constexpr long long kFewProducts = 17000000;  // P * H * I
constexpr size_t kFewSmem = 64 * 1024;

bool few_path(const mr_expert_params& p, const void* x, const void* w13, const void* w2)
{
    const long long P = static_cast<long long>(p.T) * p.topk;
    return P <= kFewPairs && p.T <= kFewTokens && P * p.H * p.I <= kFewProducts && p.H % 8 == 0 && p.I % 8 == 0 && aligned(x, 16) && aligned(w13, 16) &&
           aligned(w2, 16) && static_cast<size_t>(P) * p.I * 4 <= kFewSmem && static_cast<size_t>(p.T) * p.H * 2 <= kFewSmem;
}

FewArgs few_args(const mr_expert_params& p, const void* x, const void* w13, const void* w2, void* out, void* h)
{
    FewArgs a;
    a.x = static_cast<const __nv_bfloat16*>(x);
    a.w13 = static_cast<const __nv_bfloat16*>(w13);
    a.w2 = static_cast<const __nv_bfloat16*>(w2);
    a.h = static_cast<float*>(h);
    a.out = static_cast<__nv_bfloat16*>(out);
    a.idx = nullptr;
    a.w = nullptr;
    a.idx_out = nullptr;
    a.w_out = nullptr;
    a.status = nullptr;
    a.T = p.T;
    a.topk = p.topk;
    a.H = p.H;
    a.I = p.I;
    a.E = p.E;
    a.act = p.act;
    return a;
}

template <bool DOWN>
int launch_experts_few(const FewArgs& a, cudaStream_t st)
{
    const void* f = reinterpret_cast<const void*>(&k_experts_few<DOWN>);
    const size_t smem = few_smem(a, DOWN, 0);
    const int e = ensure_smem(f, smem);
    if (e != cudaSuccess) return e;
    const long long tasks = static_cast<long long>(a.T) * (DOWN ? a.H : a.topk * ((a.I + few_rows(a.H) - 1) / few_rows(a.H)));
    const int grid = persistent_grid(f, kFewThreads, smem, (tasks + kFewWarps - 1) / kFewWarps);
    if (grid < 1) return cudaErrorLaunchOutOfResources;
    return launch_kernel(&k_experts_few<DOWN>, dim3(grid), dim3(kFewThreads), smem, st, 0, a);
}

int launch_layer_few(const mr_router_params* p, const RouteArgs& r, const FewArgs& a, bool down, cudaStream_t st)
{
    const int nv = nv_index(p->E);
    if (p->score_fn == MR_SOFTMAX)
        return p->in_dtype == MR_BF16 ? launch_layer_few_s0_d1(r, a, nv, down, st) : launch_layer_few_s0_d0(r, a, nv, down, st);
    return p->in_dtype == MR_BF16 ? launch_layer_few_s1_d1(r, a, nv, down, st) : launch_layer_few_s1_d0(r, a, nv, down, st);
}

// Whether the tensor-core kernels' copies can address these arrays: 16-byte
// aligned bases.
bool tensor_path(const ExpertPlan& plan, const void* x, const void* w13, const void* w2)
{
    return plan.tensor && aligned(x, 16) && aligned(w13, 16) && aligned(w2, 16);
}

int experts_tensor(const mr_expert_params& p, const void* x, const int32_t* idx, const float* w, const void* w13,
                   const void* w2, void* out, unsigned char* ws, const ExpertPlan& plan, int32_t* status,
                   cudaStream_t st)
{
    CUtensorMap map13, mapx, map2, maph;
    const bool gather = plan.nt >= kGatherColumns;
    const int box = token_box(plan.nt);
    if (!encode_map(&map13, w13, p.H, 2ll * p.I, p.E, 16) ||
        !encode_map(&mapx, gather ? ws + plan.xs : x, p.H, gather ? plan.cap : p.T, 0, gather ? box : 1) ||
        !encode_map(&map2, w2, p.I, p.H, p.E, 128) || !encode_map(&maph, ws + plan.h, p.I, plan.nt <= kSplitColumns ? 2ll * plan.cap : plan.cap, 0, box))
        return MR_ECUDA;
    ExpertArgs a;
    a.x = static_cast<const __nv_bfloat16*>(x);
    a.xs = reinterpret_cast<__nv_bfloat16*>(ws + plan.xs);
    a.out16 = aligned(out, 16);
    a.sids = reinterpret_cast<int32_t*>(ws + plan.sids);
    a.eids = reinterpret_cast<int32_t*>(ws + plan.eids);
    a.npp = reinterpret_cast<int32_t*>(ws + plan.npp);
    a.idx = idx;
    a.w = w;
    a.h = reinterpret_cast<__nv_bfloat16*>(ws + plan.h);
    a.y = reinterpret_cast<float*>(ws + plan.y);
    a.out = static_cast<__nv_bfloat16*>(out);
    a.status = status_word(status);
    a.T = p.T;
    a.topk = p.topk;
    a.H = p.H;
    a.I = p.I;
    a.E = p.E;
    a.P = p.T * p.topk;
    a.cap = plan.cap;
    a.act = p.act;
    wait_test(&a.tries, &a.drop);
    const long long blocks = plan.cap / plan.nt;
    a.mt = plan.mt_up;
    int e = gather ? launch_experts_gather(a, st) : cudaSuccess;
    if (e != cudaSuccess) return MR_ECUDA;
    e = launch_experts_up(plan.nt, map13, mapx, a, blocks * a.mt, st);
    if (e != cudaSuccess) return MR_ECUDA;
    a.mt = plan.mt_down;
    e = launch_experts_down(plan.nt, map2, maph, a, blocks * a.mt, st);
    return e != cudaSuccess ? MR_ECUDA : from_cuda(launch_experts_sum(a, st));
}

// Workspace of the adapter projection (the rank-space values; the plain kernels
// use one slice) and its shapes.
struct AdapterPlan {
    size_t same, split, bytes;
    int nt, tiles, mt, ways, slices, groups;
    bool low_rows;
};

// Rank-space values: up to this many products a warp per four of them, above
// it the tensor cores.
constexpr double kLowRowsProducts = 64 << 20;
// What the projection on the CUDA cores takes: up to 4 tokens, and products up
// to T*N*K = 10M (T=1 K=4096: 7.0 us against 7.7 on the tensor cores at N=2048,
// 11.5 against 8.6 at N=4096; T=2 K=N=2048: 6.7 against 7.5).
constexpr int kFewProjTokens = 4;
constexpr long long kFewProjProducts = 10000000;
// Rank-space values that every CTA of it makes for itself (one token), up to this
// many products: a launch less saves an eager call's host 3.3 us at any of them
// (18.4 / 21.7), and what the GPU takes more stays below that: at 32K products 5.0 /
// 3.9 (K=2048 N=256), 7.2 / 5.0 (K=4096 N=256), 7.4 / 6.6 (K=4096 N=1024), 5.6 / 6.0
// (K=N=2048); at 48K, past the border, 7.0 / 3.9 (K=2048 N=256), at 64K 7.3 / 4.9
// (K=4096 N=256), 7.7 / 4.8 (K=N=2048). (CUDA graph, us, made by each CTA / by a launch.)
constexpr long long kFusedLowProducts = 32 << 10;

AdapterPlan adapter_plan(const mr_adapter_params& p)
{
    AdapterPlan w;
    // wide tiles of tokens read w less often; narrower ones while wide ones
    // leave SMs without a unit, and for fp32 outputs (k_adapter_proj says why)
    w.nt = 16;
    while (w.nt < 64 && w.nt < p.T) w.nt *= 2;
    const long long mt = (p.N + 127) / 128;
    const long long T = p.T;
    while (p.out_dtype == MR_BF16 && w.nt >= 64 && w.nt < 256 && (T + 2 * w.nt - 1) / (2 * w.nt) * mt >= kFullGrid) w.nt *= 2;
    w.tiles = static_cast<int>((T + w.nt - 1) / w.nt);
    w.mt = static_cast<int>(mt);
    // a cluster shares a unit's sum over K while that gives idle SMs work
    // (clusters of 8 fit the GPU's partitions badly when there are many)
    const int steps = (p.K + 63) / 64;
    w.ways = 1;
    while (w.nt <= 64 && w.ways < 8 && 2ll * w.ways * w.tiles * w.mt <= kFullGrid && steps / (2 * w.ways) >= 4 &&
           (w.ways < 4 || w.tiles * w.mt <= 8))
        w.ways *= 2;
    w.slices = 1;
    w.groups = 1;
    w.bytes = 0;
    w.low_rows = static_cast<double>(T) * p.rank * p.K <= kLowRowsProducts;
    if (p.n_adapters == 0) return w;
    if (w.low_rows) {
        // slices of K while there are fewer warps than the SMs hold in flight
        const long long warps = static_cast<long long>(p.T) * ((p.rank + 3) / 4);
        while (w.slices < 8 && warps * w.slices < 1024 && p.K / (w.slices * 2) >= 512) w.slices *= 2;
    } else if (p.rank <= 128) {
        // as many CTAs as SMs or a little fewer: slices of K first (a prompt's
        // tile names one adapter), then groups of as many adapters as a tile's
        // tokens can name
        const int ksteps = (p.K + 63) / 64;
        w.slices = std::max(1, std::min(std::min(ksteps, 16), 144 / w.tiles));
        const int distinct = std::min(std::min(w.nt, p.T), p.n_adapters);
        const int per_group = 128 / p.rank;
        w.groups = std::max(1, std::min((distinct + per_group - 1) / per_group, 144 / (w.tiles * w.slices)));
    }
    size_t o = 0;
    part(o, static_cast<size_t>(w.slices) * p.T * p.rank * 4);
    w.same = part(o, w.nt > 64 ? static_cast<size_t>(w.tiles) * 4 : 0);
    w.split = part(o, w.nt > 64 ? static_cast<size_t>(p.T) * ((p.rank + 31) / 32) * 128 : 0);
    w.bytes = o;
    return w;
}

bool adapter_tensor_path(const mr_adapter_params& p, const AdapterPlan& plan, const void* x, const void* w,
                         const void* a, const void* b)
{
    return p.K % 8 == 0 && aligned(x, 16) && aligned(w, 16) && static_cast<long long>(plan.tiles) * plan.mt <= kMaxUnits &&
           (p.n_adapters == 0 || (p.rank % 8 == 0 && p.rank <= 128 && aligned(a, 16) && aligned(b, 16)));
}

int experts_plain(const mr_expert_params& p, const void* x, const int32_t* idx, const float* w, const void* w13,
                  const void* w2, void* out, unsigned char* ws, const ExpertPlan& plan, int32_t* status,
                  cudaStream_t st)
{
    using B = __nv_bfloat16;
    float* h = reinterpret_cast<float*>(ws + plan.h);
    const long long P = static_cast<long long>(p.T) * p.topk;
    int g = plain_grid(reinterpret_cast<const void*>(&k_experts_up_plain), P * p.I);
    if (g < 1) return MR_ECUDA;
    int e = launch_kernel(k_experts_up_plain, dim3(g), dim3(kPlainThreads), 0, st, 0, static_cast<const B*>(x), idx,
                          static_cast<const B*>(w13), h, P, p.topk, p.H, p.I, p.E, p.act, status);
    if (e != cudaSuccess) return MR_ECUDA;
    g = plain_grid(reinterpret_cast<const void*>(&k_experts_down_plain), static_cast<long long>(p.T) * p.H);
    if (g < 1) return MR_ECUDA;
    return from_cuda(launch_kernel(k_experts_down_plain, dim3(g), dim3(kPlainThreads), 0, st, 0,
                                   static_cast<const float*>(h), idx, w, static_cast<const B*>(w2), static_cast<B*>(out),
                                   static_cast<long long>(p.T), p.topk, p.H, p.I, p.E));
}

}  // namespace
}  // namespace mr

using namespace mr;

extern "C" {

size_t moe_experts_workspace_bytes(const mr_expert_params* p)
{
    if (check_experts(p) != MR_OK || p->T == 0) return 0;
    return expert_plan(*p, nullptr).bytes;
}

int moe_experts_fwd(const mr_expert_params* p, const void* x, const int32_t* topk_idx, const float* topk_w,
                    const void* w13, const void* w2, void* out, void* workspace, size_t ws_bytes, int32_t* status,
                    mr_stream_t stream)
{
    const int rc = check_experts(p);
    if (rc != MR_OK) return rc;
    if (p->T == 0) return MR_OK;
    if (!x || !topk_idx || !topk_w || !w13 || !w2 || !out || !workspace) return MR_EINVAL;
    if (!aligned(x, 2) || !aligned(w13, 2) || !aligned(w2, 2) || !aligned(out, 2)) return MR_EINVAL;
    if (!aligned(topk_idx, 4) || !aligned(topk_w, 4) || !aligned(status, 4)) return MR_EINVAL;
    const ExpertPlan plan = expert_plan(*p, nullptr);
    if (ws_bytes < plan.bytes || !aligned(workspace, 256)) return MR_EINVAL;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    if (few_path(*p, x, w13, w2)) {
        FewArgs a = few_args(*p, x, w13, w2, out, ws + plan.h);
        a.idx = topk_idx;
        a.w = topk_w;
        a.status = status;
        const int e = launch_experts_few<false>(a, st);
        return e != cudaSuccess ? MR_ECUDA : from_cuda(launch_experts_few<true>(a, st));
    }
    if (!tensor_path(plan, x, w13, w2))
        return experts_plain(*p, x, topk_idx, topk_w, w13, w2, out, ws, plan, status, st);
    const int e = moe_sort(topk_idx, nullptr, p->T, p->topk, p->E, plan.nt, reinterpret_cast<int32_t*>(ws + plan.sids),
                           nullptr, reinterpret_cast<int32_t*>(ws + plan.eids),
                           reinterpret_cast<int32_t*>(ws + plan.npp), ws + plan.sort, plan.sort_bytes, status, stream);
    if (e != MR_OK) return e;
    return experts_tensor(*p, x, topk_idx, topk_w, w13, w2, out, ws, plan, status, st);
}

size_t moe_layer_workspace_bytes(const mr_router_params* p, int H, int I, int act)
{
    if (router_check(p) != MR_OK || p->T == 0 || p->n_shared > MR_MAX_SORT_EXPERTS) return 0;
    const mr_expert_params q = layer_experts(p, H, I, act);
    if (check_experts(&q) != MR_OK) return 0;
    return expert_plan(q, p).bytes;
}

int moe_layer_fwd(const mr_router_params* p, int H, int I, int act, const void* x, const void* logits,
                  const void* w13, const void* w2, void* out, int32_t* topk_idx, float* topk_w, void* workspace,
                  size_t ws_bytes, int32_t* status, mr_stream_t stream)
{
    int rc = router_check(p);
    if (rc != MR_OK) return rc;
    if (p->n_shared > MR_MAX_SORT_EXPERTS) return MR_EUNSUPPORTED;
    const mr_expert_params q = layer_experts(p, H, I, act);
    rc = check_experts(&q);
    if (rc != MR_OK) return rc;
    if (p->T == 0) return MR_OK;
    if (!x || !logits || !w13 || !w2 || !out || !workspace) return MR_EINVAL;
    if (!aligned(x, 2) || !aligned(w13, 2) || !aligned(w2, 2) || !aligned(out, 2)) return MR_EINVAL;
    if (!aligned(topk_idx, 4) || !aligned(topk_w, 4) || !aligned(status, 4)) return MR_EINVAL;
    if (!aligned(logits, p->in_dtype == MR_BF16 ? 2 : 4)) return MR_EINVAL;
    const ExpertPlan plan = expert_plan(q, p);
    if (ws_bytes < plan.bytes || !aligned(workspace, 256)) return MR_EINVAL;
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    int32_t* idx = topk_idx ? topk_idx : reinterpret_cast<int32_t*>(ws + plan.idx);
    float* w = topk_w ? topk_w : reinterpret_cast<float*>(ws + plan.w);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (few_path(q, x, w13, w2) && p->E <= 128 * kRegisterMaxNv && !router_forced_select()) {
        FewArgs a = few_args(q, x, w13, w2, out, ws + plan.h);
        a.idx_out = topk_idx;
        a.w_out = topk_w;
        const RouteArgs r = router_args(p, logits);
        const int e = launch_layer_few(p, r, a, false, st);
        return e != cudaSuccess ? MR_ECUDA : from_cuda(launch_layer_few(p, r, a, true, st));
    }
    if (!tensor_path(plan, x, w13, w2)) {
        rc = moe_router_fwd(p, logits, nullptr, nullptr, nullptr, idx, w, status, stream);
        return rc != MR_OK ? rc : experts_plain(q, x, idx, w, w13, w2, out, ws, plan, status, st);
    }
    int32_t* sids = reinterpret_cast<int32_t*>(ws + plan.sids);
    int32_t* eids = reinterpret_cast<int32_t*>(ws + plan.eids);
    int32_t* npp = reinterpret_cast<int32_t*>(ws + plan.npp);
    rc = moe_router_fused_fwd_sort(p, logits, plan.nt, idx, w, sids, nullptr, eids, npp, ws + plan.sort,
                                   plan.sort_bytes, status, stream);
    if (rc == MR_EUNSUPPORTED) {  // few tokens with more slots than the one-launch form's shared memory holds
        rc = moe_router_fwd(p, logits, nullptr, nullptr, nullptr, idx, w, status, stream);
        if (rc == MR_OK)
            rc = moe_sort(idx, nullptr, q.T, q.topk, q.E, plan.nt, sids, nullptr, eids, npp, ws + plan.sort,
                          plan.sort_bytes, status, stream);
    }
    if (rc != MR_OK) return rc;
    return experts_tensor(q, x, idx, w, w13, w2, out, ws, plan, status, st);
}

size_t moe_adapter_proj_workspace_bytes(const mr_adapter_params* p)
{
    if (check_adapter(p) != MR_OK || p->T == 0 || p->n_adapters == 0) return 0;
    return adapter_plan(*p).bytes;
}

int moe_adapter_proj_fwd(const mr_adapter_params* p, const void* x, const void* w, const void* a, const void* b,
                         const int32_t* adapter, const float* scale, void* out, void* workspace, size_t ws_bytes,
                         int32_t* status, mr_stream_t stream)
{
    const int rc = check_adapter(p);
    if (rc != MR_OK) return rc;
    if (p->T == 0) return MR_OK;
    if (!x || !w || !out || !aligned(x, 2) || !aligned(w, 2)) return MR_EINVAL;
    if (!aligned(out, p->out_dtype == MR_F32 ? 4 : 2) || !aligned(status, 4)) return MR_EINVAL;
    if (p->n_adapters > 0) {
        if (!a || !b || !adapter || !aligned(a, 2) || !aligned(b, 2) || !aligned(adapter, 4) || !aligned(scale, 4))
            return MR_EINVAL;
        if (!workspace || ws_bytes < moe_adapter_proj_workspace_bytes(p) || !aligned(workspace, 256)) return MR_EINVAL;
    }
    using B = __nv_bfloat16;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    float* s = static_cast<float*>(workspace);
    const AdapterPlan plan = adapter_plan(*p);
    if (adapter_tensor_path(*p, plan, x, w, a, b)) {
        CUtensorMap mapw, mapx, mapa, mapb, maps;
        const bool few = p->T <= kFewProjTokens && plan.low_rows &&
                         static_cast<long long>(p->T) * p->N * p->K <= kFewProjProducts && static_cast<size_t>(p->T) * p->K * 2 <= kFewSmem;
        if (!few && (!encode_map(&mapw, w, p->K, p->N, 0, 128) || !encode_map(&mapx, x, p->K, p->T, 0, plan.nt)))
            return MR_ECUDA;
        AdapterArgs d;
        d.b = static_cast<const B*>(b);
        d.adapter = adapter;
        d.scale = scale;
        d.low = s;
        d.out = out;
        d.status = status_word(status);
        d.range_status = status;
        d.T = p->T;
        d.K = p->K;
        d.N = p->N;
        d.n_adapters = p->n_adapters;
        d.rank = p->rank;
        d.tiles = plan.tiles;
        d.mt = plan.mt;
        d.ways = plan.ways;
        d.slices = plan.slices;
        wait_test(&d.tries, &d.drop);
        const bool fused = few && p->T == 1 && p->n_adapters > 0 && static_cast<long long>(p->rank) * p->K <= kFusedLowProducts;
        if (fused) return from_cuda(launch_adapter_few(x, w, a, true, p->out_dtype == MR_F32, d, st));
        if (p->n_adapters > 0 && plan.low_rows) {
            if (launch_adapter_low_rows(x, a, d, st) != cudaSuccess) return MR_ECUDA;
        } else if (p->n_adapters > 0) {
            if (!encode_map(&mapa, a, p->K, p->rank, p->n_adapters, p->rank)) return MR_ECUDA;
            if (launch_adapter_low(plan.nt, mapa, mapx, d, plan.groups, st) != cudaSuccess) return MR_ECUDA;
        }
        if (few) return from_cuda(launch_adapter_few(x, w, a, false, p->out_dtype == MR_F32, d, st));
        mapb = mapw;  // not read without adapters or by narrow tiles
        maps = mapw;
        if (p->n_adapters > 0 && plan.nt > 64) {
            unsigned char* ws = static_cast<unsigned char*>(workspace);
            d.same = reinterpret_cast<int32_t*>(ws + plan.same);
            d.split = reinterpret_cast<B*>(ws + plan.split);
            if (!encode_map(&mapb, b, p->rank, p->N, p->n_adapters, 128) ||
                !encode_map(&maps, d.split, (p->rank + 31) / 32 * 64, p->T, 0, plan.nt))
                return MR_ECUDA;
            if (launch_adapter_split(plan.nt, d, st) != cudaSuccess) return MR_ECUDA;
        }
        return from_cuda(launch_adapter_proj(plan.nt, p->out_dtype == MR_F32, mapw, mapx, mapb, maps, d, st));
    }
    const long long T = p->T;
    if (p->n_adapters > 0) {
        const int g = plain_grid(reinterpret_cast<const void*>(&k_adapter_low_plain), T * p->rank);
        if (g < 1) return MR_ECUDA;
        const int e = launch_kernel(k_adapter_low_plain, dim3(g), dim3(kPlainThreads), 0, st, 0,
                                    static_cast<const B*>(x), static_cast<const B*>(a), adapter, scale, s, T, p->K,
                                    p->rank, p->n_adapters, status);
        if (e != cudaSuccess) return MR_ECUDA;
    }
    auto go = [&](auto kernel, auto* o) {
        const int g = plain_grid(reinterpret_cast<const void*>(kernel), T * p->N);
        if (g < 1) return static_cast<int>(MR_ECUDA);
        return from_cuda(launch_kernel(kernel, dim3(g), dim3(kPlainThreads), 0, st, 0, static_cast<const B*>(x),
                                       static_cast<const B*>(w), static_cast<const B*>(b), adapter,
                                       static_cast<const float*>(s), o, T, p->K, p->N, p->rank, p->n_adapters));
    };
    return p->out_dtype == MR_F32 ? go(&k_adapter_proj_plain<float>, static_cast<float*>(out))
                                  : go(&k_adapter_proj_plain<B>, static_cast<B*>(out));
}

}  // extern "C"
