// The adapter projection on the tensor cores.
//
//   k_adapter_low   s[t] = scale * (a[i] . x_t), the rank-space values of each token's adapter i, as
//                   partial sums over slices of K
//   k_adapter_proj  out[t] = w . x_t + b[i] . s[t]
//
// Tokens are taken in tiles of at most NT and need no sorting by adapter.
//
// The second part of k_adapter_proj, rank multiply-adds an output:
// * A wide tile (128 or 256 tokens) whose tokens all name the same adapter, the
//   usual one of a prompt, takes it as further steps of the tensor cores' sum,
//   with s as two bf16 parts (s = hi + lo to 16 significant bits, made by
//   k_adapter_split) against the same b[i]: 2 steps of 66 at rank 64, K 4096,
//   where the epilogue's multiply-adds took three times the products' time.
// * Otherwise the epilogue warps take it in fp32, each token's with its own
//   b[i] only. (In the tensor cores' sum the tokens of other adapters would meet
//   b[i] with zeros, and an infinity in one request's adapter would reach every
//   token of the tile.) In narrow tiles that is done before the sum over K is.
//
// Calls with fewer units than SMs share each unit's sum over K among the CTAs
// of a cluster, which add their parts through distributed shared memory.
//
// Measured (CUDA graph, one GB300): T=48 K=N=4096 rank 16, an adapter each, 14.4 us
// (33.5 MB of w are 4.9 us; the rest is the chain rank-space values, b, cluster
// sum); T=333 K=1544 N=1000 rank 8 17.1 us; T=4096 K=N=4096 rank 64 124 us, of it
// the projection 101 (1.4 PFLOP/s; its 512 units are 4 rounds on 152 SMs where
// 3.4 would do), the rank-space values 26 and their split 8 beside it; T=8 K=N=4096
// rank 16 9.9 us.
//
// Those prompts end on tile edges. One token of another adapter, or of none, sends
// its whole tile to the epilogue: T=4096 K=N=4096 rank 64 with requests of 512 tokens
// 123 us, of 500 454, of 300 579, of 200 586, of 29 1131, of one 1619. fp32 outputs take
// tiles of 64 and always the epilogue: T=3600 K=3696 N=512 rank 32 94 us (73 in bf16,
// N being small for wide tiles).
//
// k_adapter_proj starts while k_adapter_low runs (its sum over K needs nothing
// of it), so the low-rank product costs little time of its own once w is large.
#include <type_traits>

#include "few.cuh"
#include "gemm.cuh"

namespace mr {

namespace {
constexpr int kChunkRanks = 32;  // ranks of a further step (hi and lo)
constexpr int kSegment = 4;      // k-steps between readings of the accumulator, fp32 output
constexpr int kSmallTile = 64;   // tiles up to this keep the adapters' part of a whole unit in shared memory

struct AdapterLayout {
    uint32_t a, b, ids, list, low, part, bars, bytes;
};
}  // namespace

// rank: 0 for a kernel (or call) without the adapters' part. low: rank-space
// values (small tiles: of all tokens; else of 16, rank-major); part: small
// tiles: the adapters' part of the unit; else b[i]'s rows of the unit.
__host__ __device__ inline AdapterLayout adapter_layout(int nt, int stages, int rank)
{
    AdapterLayout L;
    uint32_t o = 0;
    L.a = o; o += static_cast<uint32_t>(stages) * kRows * kStepBytes;
    L.b = o; o += static_cast<uint32_t>(stages) * nt * kStepBytes;
    L.ids = o; o += static_cast<uint32_t>(nt) * 4;
    L.list = o; o += static_cast<uint32_t>(nt) * 4 + 16;
    o = (o + 15) / 16 * 16;
    L.low = o; o += static_cast<uint32_t>(nt <= kSmallTile ? nt : 16) * rank * 4;
    L.part = o; o += rank == 0 ? 0 : nt <= kSmallTile ? static_cast<uint32_t>(nt) * kRows * 4
                                                      : static_cast<uint32_t>(kRows) * (rank + 8) * 2;
    o = (o + 15) / 16 * 16;
    L.bars = o; o += sizeof(GemmBars);
    L.bytes = o + 1024;
    return L;
}

// ---- rank-space values -------------------------------------------------------------------------------------------

// A CTA works on one tile of tokens, one slice of K, and every gridDim.z-th
// group of the tile's distinct adapters; a group is as many adapters as fill
// the 128 rows of a product.
template <int NT>
__global__ void __launch_bounds__(kGemmThreads, 1)
    k_adapter_low(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_x,
                  const __grid_constant__ AdapterArgs a)
{
    extern __shared__ unsigned char raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    const AdapterLayout L = adapter_layout(NT, a.stages_low, 0);
    GemmBars& bars = *reinterpret_cast<GemmBars*>(smem + L.bars);
    int* slot = reinterpret_cast<int*>(smem + L.ids);    // token -> place in the list, -1: none
    int* list = reinterpret_cast<int*>(smem + L.list);   // the tile's distinct adapters, by first appearance
    int* count = list + NT;
    __shared__ int warp_first[kGemmThreads / 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr uint32_t kColumns = 2 * NT;
    const int group = 128 / a.rank;
    const uint32_t ring_a = smem_addr(smem + L.a), ring_b = smem_addr(smem + L.b);
    const int t0 = blockIdx.x * NT, tokens = min(NT, a.T - t0);

    if (warp == 1) tmem_alloc(&bars.tmem, kColumns);
    if (threadIdx.x == 0) {
        for (int i = 0; i < a.stages_low; ++i) {
            mbar_init(&bars.full[i], 2);
            mbar_init(&bars.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.acc_full[i], 1);
            mbar_init(&bars.acc_empty[i], kEpilogueThreads);
        }
        mbar_init(&bars.drained, 1);
        bars.gone = 0;
        prefetch_map(&map_a);
        prefetch_map(&map_x);
    }
    pdl_wait();
    // the distinct adapters of the tile
    for (int t = threadIdx.x; t < NT; t += kGemmThreads) {
        const int id = t < tokens ? __ldcg(a.adapter + t0 + t) : -1;
        if (id >= a.n_adapters && blockIdx.y == 0 && blockIdx.z == 0) report_status(a.range_status, kStatusRange);
        slot[t] = id >= 0 && id < a.n_adapters ? id : -1;
    }
    __syncthreads();
    pdl_trigger();  // after this CTA has its tensor memory: the next kernel takes some too, and waits for this one
    // a token is its adapter's first if no earlier one names it (the previous
    // one does, mostly); the first ones are listed in order
    int id = -1;
    bool first = false;
    if (threadIdx.x < NT) {
        id = slot[threadIdx.x];
        first = id >= 0;
        for (int t = static_cast<int>(threadIdx.x) - 1; first && t >= 0; --t) first = slot[t] != id;
    }
    const uint32_t firsts = __ballot_sync(kFull, first);
    if (lane == 0) warp_first[warp] = __popc(firsts);
    __syncthreads();
    if (first) {
        int place = __popc(firsts & lanemask_lt());
        for (int w = 0; w < warp; ++w) place += warp_first[w];
        list[place] = id;
    }
    if (threadIdx.x == 0) {
        int n = 0;
        for (int w = 0; w < kGemmThreads / 32; ++w) n += warp_first[w];
        *count = n;
    }
    __syncthreads();
    if (id >= 0) {
        int place = 0;
        while (list[place] != id) ++place;
        slot[threadIdx.x] = place;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars.tmem;
    const int distinct = *count;

    const Waits wait{&bars.gone, a.tries};
    const uint32_t drain = min(a.tries, kDrainTries);
    const int groups = (distinct + group - 1) / group;
    const int ksteps = (a.K + kStepK - 1) / kStepK;
    const int k0 = static_cast<int>(static_cast<long long>(ksteps) * blockIdx.y / gridDim.y);
    const int k1 = static_cast<int>(static_cast<long long>(ksteps) * (blockIdx.y + 1) / gridDim.y);
    const int cols = (tokens + 15) & ~15;
    RingPos pos;
    int issued = 0;
    bool ok = true;

    if (warp == 0) {
        for (int g = blockIdx.z; ok && g < groups; g += gridDim.z) {
            const int n = min(group, distinct - g * group);
            for (int k = k0; k < k1; ++k) {
                ok = __all_sync(kFull, pos.wraps == 0 || wait(&bars.empty[pos.s], (pos.wraps - 1) & 1));
                if (!ok) break;
                uint64_t* full = &bars.full[pos.s];
                if (lane == 0) mbar_expect(full, n * a.rank * kStepBytes);
                ++issued;
                __syncwarp();
                if (lane < n && !a.drop)
                    load_box3(ring_a + pos.s * (128 * kStepBytes) + lane * a.rank * kStepBytes, &map_a, k * kStepK, 0,
                              list[g * group + lane], full);
                pos.next(a.stages_low);
            }
        }
    } else if (warp == 2) {
        if (elect_one())
            for (int g = blockIdx.z; ok && g < groups; g += gridDim.z)
                for (int k = k0; k < k1; ++k) {
                    ok = pos.wraps == 0 || wait(&bars.empty[pos.s], (pos.wraps - 1) & 1);
                    if (!ok) break;
                    uint64_t* full = &bars.full[pos.s];
                    mbar_expect(full, NT * kStepBytes);
                    ++issued;
                    if (!a.drop) load_box2(ring_b + pos.s * (NT * kStepBytes), &map_x, k * kStepK, t0, full);
                    pos.next(a.stages_low);
                }
    } else if (warp == 1) {
        if (elect_one()) {
            int seen = 0;
            StagePoll poll;
            const uint32_t desc = product_desc(cols);
            for (int g = blockIdx.z; ok && g < groups; g += gridDim.z, ++seen) {
                const int buf = seen & 1;
                ok = seen < 2 || wait(&bars.acc_empty[buf], ((seen >> 1) - 1) & 1);
                if (!ok) break;
                tc_fence_after();
                for (int k = k0; k < k1; ++k) {
                    ok = poll.take(wait, bars, pos, a.stages_low);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t da = operand_desc(ring_a + pos.s * (128 * kStepBytes));
                    const uint64_t db = operand_desc(ring_b + pos.s * (NT * kStepBytes));
#pragma unroll
                    for (int q = 0; q < kStepK / 16; ++q) mma16(tmem + buf * NT, da + q * 2, db + q * 2, desc, k > k0 || q > 0);
                    mma_commit(&bars.empty[pos.s]);
                    pos.next(a.stages_low);
                }
                if (ok) mma_commit(&bars.acc_full[buf]);
            }
            if (!ok) {
                mma_commit(&bars.drained);
                mbar_wait(&bars.drained, 0, drain);
            }
        }
    } else if (warp >= 4) {
        const int et = threadIdx.x - kEpilogueThreads, q = warp - 4;
        const int j = et / a.rank, r = et - j * a.rank;
        float* part = a.low + static_cast<long long>(blockIdx.y) * a.T * a.rank;
        int seen = 0;
        for (int g = blockIdx.z; g < groups; g += gridDim.z, ++seen) {
            const int buf = seen & 1;
            if (!epilogue_wait(wait, &bars.acc_full[buf], (seen >> 1) & 1)) break;
            tc_fence_after();
            const int mine = j < group && g * group + j < distinct ? g * group + j : -2;
            const float sc = mine < 0 ? 0.0f : (a.scale ? __ldcg(a.scale + list[mine]) : 1.0f);
            const uint32_t acc = tmem + buf * NT + (static_cast<uint32_t>(q * 32) << 16);
            for (int c0 = 0; c0 < tokens; c0 += 16) {
                float v[16];
                tmem_load16(acc + c0, v);
#pragma unroll
                for (int c = 0; c < 16; ++c)
                    if (c0 + c < tokens && slot[c0 + c] == mine)
                        part[static_cast<long long>(t0 + c0 + c) * a.rank + r] = v[c] * sc;
            }
            tc_fence_before();
            mbar_arrive(&bars.acc_empty[buf]);
        }
    }
    if ((warp == 0 || warp == 2) && !ok)
        for (int s = 0; s < a.stages_low && s < issued; ++s)
            mbar_wait(&bars.full[s], ((issued - 1 - s) / a.stages_low) & 1, drain);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_free(tmem, kColumns);
    }
    if (threadIdx.x == 0 && bars.gone) report_status(a.status, kStatusTimeout);
}

// The same without tiles, for calls whose products are few: a warp takes four
// ranks of one token over a slice of K, and a's rows come from L2 again for
// each token.
__global__ void __launch_bounds__(256) k_adapter_low_rows(const __nv_bfloat16* x, const __nv_bfloat16* wa, AdapterArgs a)
{
    pdl_wait();
    pdl_trigger();
    constexpr int kAtOnce = 4;
    const int lane = threadIdx.x & 31, K8 = a.K / 8, quads = a.rank / 4;
    const int part = (K8 + a.slices - 1) / a.slices;
    const long long warps = static_cast<long long>(gridDim.x) * 8;
    for (long long u = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5); u < static_cast<long long>(a.T) * quads * a.slices;
         u += warps) {
        const long long v = u / a.slices, t = v / quads;
        const int slice = static_cast<int>(u - v * a.slices), r0 = static_cast<int>(v - t * quads) * 4;
        const int end = min(K8, (slice + 1) * part);
        const int id = __ldcg(a.adapter + t);
        if (id >= a.n_adapters && r0 == 0 && slice == 0 && lane == 0) report_status(a.range_status, kStatusRange);
        if (id < 0 || id >= a.n_adapters) continue;
        const uint4* xr = reinterpret_cast<const uint4*>(x + t * a.K);
        const uint4* ar = reinterpret_cast<const uint4*>(wa + (static_cast<long long>(id) * a.rank + r0) * a.K);
        float sum[4] = {0, 0, 0, 0};  // rank is a multiple of 8: all four rows are there
        for (int c0 = slice * part + lane; c0 < end; c0 += 32 * kAtOnce) {
            uint4 xc[kAtOnce], ac[kAtOnce][4];
#pragma unroll
            for (int c = 0; c < kAtOnce; ++c)
                if (c0 + c * 32 < end) {
                    xc[c] = __ldcg(xr + c0 + c * 32);
#pragma unroll
                    for (int q = 0; q < 4; ++q) ac[c][q] = __ldcg(ar + static_cast<long long>(q) * K8 + c0 + c * 32);
                }
#pragma unroll
            for (int c = 0; c < kAtOnce; ++c)
                if (c0 + c * 32 < end) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) sum[q] = dot8(ac[c][q], xc[c], sum[q]);
                }
        }
        const float sc = a.scale ? __ldcg(a.scale + id) : 1.0f;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float v = warp_sum(sum[q]);
            if (lane == q) a.low[(static_cast<long long>(slice) * a.T + t) * a.rank + r0 + q] = v * sc;
        }
    }
}

// One to TOKENS tokens: a warp per row of w, on the CUDA cores (few.cuh says
// why). The row's product, and the loads of b's row, come before the rank-space
// values are needed; the lanes share out the ranks. FUSED (one token): every CTA
// makes the rank-space values itself, at most 64 KB of a from L2: a launch less
// for the host, which costs an eager call 3.3 us, and up to 2.2 us more on the GPU
// (kFusedLowProducts, in experts.cu, has the figures).
__host__ __device__ constexpr int few_threads(bool fused) { return fused ? 512 : 256; }

template <int TOKENS, bool FUSED, typename OutT>
__global__ void __launch_bounds__(few_threads(FUSED)) k_adapter_few(const __nv_bfloat16* x, const __nv_bfloat16* w,
                                                     const __nv_bfloat16* wa, AdapterArgs a)
{
    extern __shared__ __align__(16) unsigned char smem[];
    const bool low = a.n_adapters > 0;
    if (!low || FUSED) pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, K8 = a.K / 8;
    const uint4* xs = reinterpret_cast<const uint4*>(smem);
    float* s_low = reinterpret_cast<float*>(smem + static_cast<size_t>(a.T) * a.K * 2);
    constexpr int kChunks = 8, kThreads = few_threads(FUSED), kWarps = kThreads / 32;
    bool waited = !low || FUSED;
    // the first part of the warp's first row is on its way while x is staged
    int row = blockIdx.x * kWarps + warp;
    uint4 wc[kChunks];
    auto load = [&](int c0) {
        const uint4* wr = reinterpret_cast<const uint4*>(w + static_cast<long long>(row) * a.K);
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
            if (c0 + c * 32 < K8) wc[c] = load_weights(wr + c0 + c * 32);
    };
    if (row < a.N) load(lane);
    for (int i = threadIdx.x; i < a.T * K8; i += kThreads)
        reinterpret_cast<uint4*>(smem)[i] = __ldcg(reinterpret_cast<const uint4*>(x) + i);
    __syncthreads();
    if (FUSED && low) {
        for (int u = warp; u < a.T * a.rank; u += kWarps) {
            const int t = u / a.rank, r = u - t * a.rank, id = __ldcg(a.adapter + t);
            if (id >= a.n_adapters && r == 0 && lane == 0 && blockIdx.x == 0) report_status(a.range_status, kStatusRange);
            if (id < 0 || id >= a.n_adapters) continue;
            const uint4* ar = reinterpret_cast<const uint4*>(wa + (static_cast<long long>(id) * a.rank + r) * a.K);
            float v = 0.0f;
#pragma unroll 8
            for (int c = lane; c < K8; c += 32) v = dot8(__ldcg(ar + c), xs[t * K8 + c], v);
            v = warp_sum(v);
            if (lane == 0) s_low[u] = a.scale ? v * __ldcg(a.scale + id) : v;
        }
        __syncthreads();
    }
    for (; row < a.N; row += gridDim.x * kWarps) {
        float sum[TOKENS] = {};
        for (int c0 = lane; c0 < K8; c0 += 32 * kChunks) {
            if (c0 != lane || row != static_cast<int>(blockIdx.x) * kWarps + warp) load(c0);
#pragma unroll
            for (int c = 0; c < kChunks; ++c)
                if (c0 + c * 32 < K8) {
#pragma unroll
                    for (int t = 0; t < TOKENS; ++t)
                        if (t < a.T) sum[t] = dot8(wc[c], xs[t * K8 + c0 + c * 32], sum[t]);
                }
        }
        if (low) {
            int id[TOKENS];
            float b0[TOKENS];
#pragma unroll
            for (int t = 0; t < TOKENS; ++t) {
                id[t] = t < a.T ? __ldcg(a.adapter + t) : -1;
                if (id[t] >= a.n_adapters) id[t] = -1;
                b0[t] = 0.0f;
                if (id[t] >= 0 && lane < a.rank)
                    b0[t] = load_scalar(a.b + (static_cast<long long>(id[t]) * a.N + row) * a.rank + lane);
            }
            if (!waited) pdl_wait();
            waited = true;
#pragma unroll
            for (int t = 0; t < TOKENS; ++t) {
                if (id[t] < 0) continue;
                const __nv_bfloat16* br = a.b + (static_cast<long long>(id[t]) * a.N + row) * a.rank;
                const float* s = a.low + static_cast<long long>(t) * a.rank;
                for (int r = lane; r < a.rank; r += 32) {
                    float v = 0.0f;
                    if (FUSED) v = s_low[t * a.rank + r];
                    else
                        for (int p = 0; p < a.slices; ++p) v += __ldcg(s + static_cast<long long>(p) * a.T * a.rank + r);
                    sum[t] = fmaf(r == lane ? b0[t] : load_scalar(br + r), v, sum[t]);
                }
            }
        }
#pragma unroll
        for (int t = 0; t < TOKENS; ++t) {
            const float v = warp_sum(sum[t]);
            if (lane == 0 && t < a.T) store_scalar(static_cast<OutT*>(a.out) + static_cast<long long>(t) * a.N + row, v);
        }
    }
    if (!waited) pdl_wait();  // a kernel never ends before the one it follows
}

// ---- projection --------------------------------------------------------------------------------------------------

// Sum over the slices of four rank-space values.
__device__ __forceinline__ float4 low4(const AdapterArgs& a, long long t, int r)
{
    const float* s = a.low + t * a.rank + r;
    float4 v = make_float4(0, 0, 0, 0);
#pragma unroll 4
    for (int p = 0; p < a.slices; ++p) {
        const float4 x = __ldcg(reinterpret_cast<const float4*>(s + static_cast<long long>(p) * a.T * a.rank));
        v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
    }
    return v;
}

__device__ __forceinline__ void unpack8(uint4 p, float (&v)[8])
{
    const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// hi and lo of 8 consecutive ranks, packed.
__device__ __forceinline__ void split8(const float (&v)[8], uint4& hi, uint4& lo)
{
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t h0, l0, h1, l1;
        split_f32(v[2 * i], h0, l0);
        split_f32(v[2 * i + 1], h1, l1);
        h[i] = h0 | h1 << 16;
        l[i] = l0 | l1 << 16;
    }
    hi = make_uint4(h[0], h[1], h[2], h[3]);
    lo = make_uint4(l[0], l[1], l[2], l[3]);
}

// Wide tiles: whether all tokens of the tile name one adapter, and if so their
// rank-space values as the token operand of k_adapter_proj's further steps.
// Grid: tiles by 8 parts of a tile.
template <int NT>
__global__ void __launch_bounds__(256) k_adapter_split(AdapterArgs a)
{
    pdl_wait();
    pdl_trigger();
    const int t0 = blockIdx.x * NT, tokens = min(NT, a.T - t0);
    const int ad = __ldcg(a.adapter + t0);
    const int mine = static_cast<int>(threadIdx.x) < tokens ? __ldcg(a.adapter + t0 + threadIdx.x) : ad;
    const bool same = __syncthreads_and(mine == ad) && ad >= 0 && ad < a.n_adapters;
    if (blockIdx.y == 0 && threadIdx.x == 0) a.same[blockIdx.x] = same ? ad : -1;
    if (!same) return;
    const int octets = (a.rank + kChunkRanks - 1) / kChunkRanks * (kChunkRanks / 8), part = NT / 8;
    for (int f = threadIdx.x; f < part * octets; f += 256) {
        const int t = blockIdx.y * part + f / octets, o = f % octets;
        if (t >= tokens) break;
        float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (o * 8 < a.rank) {
            const float4 x = low4(a, t0 + t, o * 8), y = low4(a, t0 + t, o * 8 + 4);
            v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
            v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
        }
        uint4 hi, lo;
        split8(v, hi, lo);
        uint4* row = reinterpret_cast<uint4*>(a.split + (static_cast<long long>(t0 + t) * octets + o / 4 * 4) * 16);
        row[o % 4] = hi;
        row[4 + o % 4] = lo;
    }
}

// Output in fp32: the tensor cores add to their accumulator without rounding
// the last bit, off by 4.4e-6 of the output's norm at K = 4096 (1.0e-6 at 1024), so
// it is taken out every kSegment steps and the parts are summed in registers
// (tiles of at most 64 tokens, whose sums fit there): 2.4e-7 at any K, 4.7e-7 with
// parts twice as long, which are 4% faster. In bf16 one segment does.
template <int NT, typename OutT>
__global__ void __launch_bounds__(kGemmThreads, 1)
    k_adapter_proj(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                   const __grid_constant__ CUtensorMap map_b, const __grid_constant__ CUtensorMap map_s,
                   const __grid_constant__ AdapterArgs a)
{
    extern __shared__ unsigned char raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    const AdapterLayout L = adapter_layout(NT, a.stages, a.n_adapters > 0 ? a.rank : 0);
    GemmBars& bars = *reinterpret_cast<GemmBars*>(smem + L.bars);
    const int warp = threadIdx.x >> 5;
    constexpr uint32_t kColumns = 2 * NT;
    constexpr uint32_t a_bytes = kRows * kStepBytes, b_bytes = NT * kStepBytes;
    const uint32_t ring_a = smem_addr(smem + L.a), ring_b = smem_addr(smem + L.b);

    if (warp == 1) tmem_alloc(&bars.tmem, kColumns);
    if (threadIdx.x == 0) {
        for (int i = 0; i < a.stages; ++i) {
            mbar_init(&bars.full[i], 2);
            mbar_init(&bars.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.acc_full[i], 1);
            mbar_init(&bars.acc_empty[i], kEpilogueThreads);
        }
        mbar_init(&bars.drained, 1);
        bars.gone = 0;
        prefetch_map(&map_w);
        prefetch_map(&map_x);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars.tmem;
    // Alone in the call, it follows whatever made x. After k_adapter_low, whose
    // trigger comes after its own wait, x and w are there already.
    const bool low = a.n_adapters > 0;
    if (!low) pdl_wait();
    pdl_trigger();

    const Waits wait{&bars.gone, a.tries};
    const uint32_t drain = min(a.tries, kDrainTries);
    const int units = a.tiles * a.mt;
    // With fewer units than SMs a cluster of `ways` CTAs shares one, each a
    // range of K (narrow tiles; one unit a cluster then).
    const int ways = NT <= kSmallTile ? a.ways : 1, share = ways > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int first_unit = blockIdx.x / ways, stride = gridDim.x / ways;
    const int all_steps = (a.K + kStepK - 1) / kStepK;
    const int k_first = all_steps * share / ways, ksteps = all_steps * (share + 1) / ways - k_first;
    RingPos pos;
    int issued = 0;
    bool ok = true;

    constexpr bool kWide = NT > kSmallTile, kSegments = std::is_same<OutT, float>::value;
    const int segments = kSegments ? (ksteps + kSegment - 1) / kSegment : 1;
    const int chunks = (a.rank + kChunkRanks - 1) / kChunkRanks;  // further steps of a tile with one adapter
    bool waited = !low;
    // the adapter whose steps follow the sum over K, or -1; asked for at the
    // unit's start once it is known by then
    constexpr int kUnknown = -2;
    auto early_adapter = [&](int b) { return !kWide || !low ? -1 : waited ? __ldcg(a.same + b) : kUnknown; };
    auto one_adapter = [&](int b, int early) {
        if (early != kUnknown) return early;
        pdl_wait();
        waited = true;
        return __ldcg(a.same + b);
    };

    if (warp == 0 || warp == 2) {
        if (elect_one()) {
            for (int u = first_unit; ok && u < units; u += stride) {
                const int b = u / a.mt, m = u - b * a.mt;
                int steps = ksteps, ad = early_adapter(b);
                for (int k = 0; k < steps; ++k) {
                    ok = pos.wraps == 0 || wait(&bars.empty[pos.s], (pos.wraps - 1) & 1);
                    if (!ok) break;
                    uint64_t* full = &bars.full[pos.s];
                    mbar_expect(full, warp == 0 ? a_bytes : b_bytes);
                    ++issued;
                    if (!a.drop) {
                        const uint32_t dst = warp == 0 ? ring_a + pos.s * a_bytes : ring_b + pos.s * b_bytes;
                        if (k < ksteps) {
                            if (warp == 0) load_box2(dst, &map_w, (k_first + k) * kStepK, m * kRows, full);
                            else load_box2(dst, &map_x, (k_first + k) * kStepK, b * NT, full);
                        } else {
                            const int c = k - ksteps;
                            if (warp == 0) load_box3(dst, &map_b, c * kChunkRanks, m * kRows, ad, full);
                            else load_box2(dst, &map_s, c * kStepK, b * NT, full);
                        }
                    }
                    pos.next(a.stages);
                    if (k == ksteps - 1) {
                        ad = one_adapter(b, ad);
                        if (ad >= 0) steps += chunks;
                    }
                }
            }
            if (!ok)
                for (int s = 0; s < a.stages && s < issued; ++s)
                    mbar_wait(&bars.full[s], ((issued - 1 - s) / a.stages) & 1, drain);
        }
    } else if (warp == 1) {
        if (elect_one()) {
            int seen = 0;
            StagePoll poll;
            for (int u = first_unit; ok && u < units; u += stride) {
                const int b = u / a.mt;
                const uint32_t desc = product_desc((min(NT, a.T - b * NT) + 15) & ~15);
                const int early = early_adapter(b);
                for (int g = 0; ok && g < segments; ++g, ++seen) {
                    const int buf = seen & 1, k1 = kSegments ? min(ksteps, (g + 1) * kSegment) : ksteps;
                    const uint32_t d = tmem + buf * NT;
                    ok = seen < 2 || wait(&bars.acc_empty[buf], ((seen >> 1) - 1) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    bool add = false;
                    for (int k = kSegments ? g * kSegment : 0; k < k1; ++k) {
                        ok = poll.take(wait, bars, pos, a.stages);
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t da = operand_desc(ring_a + pos.s * a_bytes), db = operand_desc(ring_b + pos.s * b_bytes);
#pragma unroll
                        for (int q = 0; q < kStepK / 16; ++q) {
                            mma16(d, da + q * 2, db + q * 2, desc, add);
                            add = true;
                        }
                        mma_commit(&bars.empty[pos.s]);
                        pos.next(a.stages);
                    }
                    if (ok && one_adapter(b, early) >= 0)
                        for (int c = 0; c < chunks; ++c) {
                            ok = poll.take(wait, bars, pos, a.stages);
                            if (!ok) break;
                            tc_fence_after();
                            const uint64_t da = operand_desc(ring_a + pos.s * a_bytes), db = operand_desc(ring_b + pos.s * b_bytes);
                            const int nq = (min(a.rank - c * kChunkRanks, kChunkRanks) + 15) / 16;
                            for (int q = 0; q < nq; ++q) {
                                mma16(d, da + q * 2, db + q * 2, desc, true);
                                mma16(d, da + q * 2, db + (2 + q) * 2, desc, true);
                            }
                            mma_commit(&bars.empty[pos.s]);
                            pos.next(a.stages);
                        }
                    if (ok) mma_commit(&bars.acc_full[buf]);
                }
            }
            if (!ok) {
                mma_commit(&bars.drained);
                mbar_wait(&bars.drained, 0, drain);
            }
        }
    } else if (warp >= 4) {
        const int et = threadIdx.x - kEpilogueThreads, q = warp - 4;
        int* mine = reinterpret_cast<int*>(smem + L.ids);      // the tile's adapters, -1: none
        float* s = reinterpret_cast<float*>(smem + L.low);
        float* part = reinterpret_cast<float*>(smem + L.part);
        __nv_bfloat16* rows_b = reinterpret_cast<__nv_bfloat16*>(smem + L.part);
        float* sums = reinterpret_cast<float*>(smem + L.a);    // shared unit: this CTA's sums, over the ring's first stages
        const int rank = a.rank, pitch = rank + 8;             // 16 bytes more a row: no bank conflicts
        if (low && NT <= kSmallTile && first_unit < units) {
            // b's rows of the first unit come to L2 while the rank-space values are made
            const int b = first_unit / a.mt, m = first_unit - b * a.mt, t = b * NT + share + et * ways;
            const int id = et * ways + share < NT && t < a.T ? __ldcg(a.adapter + t) : -1;
            if (id >= 0 && id < a.n_adapters)
                prefetch_l2(a.b + (static_cast<long long>(id) * a.N + m * kRows) * rank, min(kRows, a.N - m * kRows) * rank * 2);
        }
        int seen = 0, tile = -1;
        for (int u = first_unit; u < units; u += stride) {
            const int b = u / a.mt, m = u - b * a.mt, t0 = b * NT, tokens = min(NT, a.T - t0);
            const int row = m * kRows + et;
            const bool there = row < a.N;
            if (low) {
                epilogue_sync();  // the last unit's values have been read
                if (b != tile)
                    for (int t = et; t < NT; t += kEpilogueThreads) {
                        const int id = t < tokens ? __ldcg(a.adapter + t0 + t) : -1;
                        mine[t] = id < a.n_adapters ? max(id, -1) : -1;
                    }
                if (NT <= kSmallTile) epilogue_sync();
                if (!waited) pdl_wait();  // for the rank-space values
                waited = true;
                if (NT <= kSmallTile) {
                    if (b != tile)
                        for (int f = et; share + f / (rank >> 2) * ways < tokens; f += kEpilogueThreads) {
                            const int t = share + f / (rank >> 2) * ways, r = f % (rank >> 2) * 4;
                            if (mine[t] >= 0) *reinterpret_cast<float4*>(s + t * rank + r) = low4(a, t0 + t, r);
                        }
                    epilogue_sync();
                    // this thread's row of the unit, 8 of this CTA's tokens at a time
                    for (int tb = share; tb < tokens; tb += 8 * ways) {
                        float v[8] = {};
                        const __nv_bfloat16* brow[8];
                        bool use[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const int t = tb + k * ways;
                            use[k] = t < tokens && mine[t] >= 0 && row < a.N;
                            brow[k] = a.b + (use[k] ? (static_cast<long long>(mine[t]) * a.N + row) * rank : 0);
                        }
#pragma unroll 2
                        for (int r = 0; r < rank; r += 8) {
                            uint4 p[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                if (use[k]) p[k] = __ldcg(reinterpret_cast<const uint4*>(brow[k] + r));
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                if (!use[k]) continue;
                                float w[8];
                                unpack8(p[k], w);
                                const float4* x = reinterpret_cast<const float4*>(s + (tb + k * ways) * rank + r);
                                const float4 y = x[0], z = x[1];
                                v[k] = fmaf(w[0], y.x, fmaf(w[1], y.y, fmaf(w[2], y.z, fmaf(w[3], y.w, v[k]))));
                                v[k] = fmaf(w[4], z.x, fmaf(w[5], z.y, fmaf(w[6], z.z, fmaf(w[7], z.w, v[k]))));
                            }
                        }
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            if (tb + k * ways < tokens) part[(tb + k * ways) * kRows + et] = v[k];
                    }
                }
                tile = b;
            }
            // the adapter's part is in the accumulator
            const bool summed = kWide && low && __ldcg(a.same + b) >= 0;
            // the parts of all segments but the last
            float sum[kSegments ? NT : 1];
            if (kSegments) {
#pragma unroll
                for (int c = 0; c < NT; ++c) sum[c] = 0.0f;
                for (int g = 0; ok && g < segments - 1; ++g, ++seen) {
                    ok = epilogue_wait(wait, &bars.acc_full[seen & 1], (seen >> 1) & 1);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int c0 = 0; c0 < NT; c0 += 16)
                        if (c0 < tokens) {
                            float v[16];
                            tmem_load16(tmem + (seen & 1) * NT + (static_cast<uint32_t>(q * 32) << 16) + c0, v);
#pragma unroll
                            for (int c = 0; c < 16; ++c) sum[c0 + c] += v[c];
                        }
                    tc_fence_before();
                    mbar_arrive(&bars.acc_empty[seen & 1]);
                }
                if (!ok) break;
            }
            const int buf = seen & 1;
            ok = epilogue_wait(wait, &bars.acc_full[buf], (seen >> 1) & 1);
            if (!ok) break;
            ++seen;
            tc_fence_after();
            const uint32_t acc = tmem + buf * NT + (static_cast<uint32_t>(q * 32) << 16);
            OutT* out = static_cast<OutT*>(a.out) + static_cast<long long>(t0) * a.N + row;
            int held = -1;  // the adapter whose rows are in rows_b
            constexpr int kUnroll = kSegments ? NT / 16 : 1;  // `sum` stays in registers
#pragma unroll kUnroll
            for (int c0 = 0; c0 < NT; c0 += 16) {
                if (c0 >= tokens) continue;
                float v[16];
                tmem_load16(acc + c0, v);
                if (kSegments) {
#pragma unroll
                    for (int c = 0; c < 16; ++c) v[c] += sum[kSegments ? c0 + c : 0];
                }
                if (ways > 1) {  // to the cluster, below
#pragma unroll
                    for (int c = 0; c < 16; ++c) sums[(c0 + c) * kRows + et] = v[c];
                    continue;
                }
                if (low && NT <= kSmallTile) {
#pragma unroll
                    for (int c = 0; c < 16; ++c)
                        if (c0 + c < tokens) v[c] += part[(c0 + c) * kRows + et];
                } else if (low && !summed) {
                    const int ad = mine[c0];
                    bool same = true, any = false;
                    for (int c = 0; c < 16; ++c) {
                        same = same && (c0 + c >= tokens || mine[c0 + c] == ad);
                        any = any || mine[c0 + c] >= 0;
                    }
                    if (any) {
                        epilogue_sync();  // the last 16 tokens' values have been read
                        for (int f = et; f < 16 * (rank >> 2); f += kEpilogueThreads) {
                            const int c = f & 15, r = (f >> 4) * 4;
                            float4 x = make_float4(0, 0, 0, 0);
                            if (mine[c0 + c] >= 0) x = low4(a, t0 + c0 + c, r);
                            s[r * 16 + c] = x.x;
                            s[(r + 1) * 16 + c] = x.y;
                            s[(r + 2) * 16 + c] = x.z;
                            s[(r + 3) * 16 + c] = x.w;
                        }
                        if (same && ad != held) {
                            for (int f = et; f < kRows * (rank >> 3); f += kEpilogueThreads) {
                                const int i = f / (rank >> 3), r = (f - i * (rank >> 3)) * 8;
                                if (m * kRows + i < a.N)
                                    *reinterpret_cast<uint4*>(rows_b + i * pitch + r) = __ldcg(reinterpret_cast<const uint4*>(
                                        a.b + (static_cast<long long>(ad) * a.N + m * kRows + i) * rank + r));
                            }
                            held = ad;
                        }
                        epilogue_sync();
                        if (there && same) {
                            for (int r = 0; r < rank; r += 8) {
                                float w[8];
                                unpack8(*reinterpret_cast<const uint4*>(rows_b + et * pitch + r), w);
#pragma unroll
                                for (int i = 0; i < 8; ++i) {
                                    const float4* x = reinterpret_cast<const float4*>(s + (r + i) * 16);
#pragma unroll
                                    for (int g = 0; g < 4; ++g) {
                                        const float4 y = x[g];
                                        const float2 p = __ffma2_rn(make_float2(w[i], w[i]), make_float2(y.x, y.y),
                                                                    make_float2(v[g * 4], v[g * 4 + 1]));
                                        const float2 z = __ffma2_rn(make_float2(w[i], w[i]), make_float2(y.z, y.w),
                                                                    make_float2(v[g * 4 + 2], v[g * 4 + 3]));
                                        v[g * 4] = p.x;
                                        v[g * 4 + 1] = p.y;
                                        v[g * 4 + 2] = z.x;
                                        v[g * 4 + 3] = z.y;
                                    }
                                }
                            }
                        } else if (there) {
                            // each token with its own row of b, 16 loads in flight
                            for (int r = 0; r < rank; r += 8) {
                                uint4 p[16];
#pragma unroll
                                for (int c = 0; c < 16; ++c)
                                    if (mine[c0 + c] >= 0)
                                        p[c] = __ldcg(reinterpret_cast<const uint4*>(
                                            a.b + (static_cast<long long>(mine[c0 + c]) * a.N + row) * rank + r));
#pragma unroll
                                for (int c = 0; c < 16; ++c) {
                                    if (mine[c0 + c] < 0) continue;
                                    float w[8];
                                    unpack8(p[c], w);
#pragma unroll
                                    for (int i = 0; i < 8; ++i) v[c] = fmaf(w[i], s[(r + i) * 16 + c], v[c]);
                                }
                            }
                        }
                    }
                }
#pragma unroll
                for (int c = 0; c < 16; ++c)
                    if (there && c0 + c < tokens) store_scalar(out + static_cast<long long>(c0 + c) * a.N, v[c]);
            }
            tc_fence_before();
            mbar_arrive(&bars.acc_empty[buf]);
        }
    }
    if (ways > 1) {
        // every CTA adds up its share of the tokens: the CTAs' sums in order of K
        __syncwarp();
        cluster_sync();
        if (warp >= 4 && !bars.gone && first_unit < units) {
            const int et = threadIdx.x - kEpilogueThreads, b = first_unit / a.mt, m = first_unit - b * a.mt, t0 = b * NT;
            const int tokens = min(NT, a.T - t0), row = m * kRows + et;
            const float* part = reinterpret_cast<const float*>(smem + L.part);
            const float* sums = reinterpret_cast<const float*>(smem + L.a) + et;
            OutT* out = static_cast<OutT*>(a.out) + static_cast<long long>(t0) * a.N + row;
            constexpr int kAtOnce = 4;  // tokens whose parts are in flight together
            if (row < a.N)
                for (int t = share; t < tokens; t += kAtOnce * ways) {
                    float p[kAtOnce][8];
#pragma unroll
                    for (int k = 0; k < kAtOnce; ++k)
#pragma unroll
                        for (int r = 0; r < 8; ++r)
                            p[k][r] = r < ways && t + k * ways < tokens ? *cluster_peer(sums + (t + k * ways) * kRows, r) : 0.0f;
#pragma unroll
                    for (int k = 0; k < kAtOnce; ++k) {
                        if (t + k * ways >= tokens) break;
                        float v = p[k][0];
#pragma unroll
                        for (int r = 1; r < 8; ++r) v += p[k][r];
                        if (low) v += part[(t + k * ways) * kRows + et];
                        store_scalar(out + static_cast<long long>(t + k * ways) * a.N, v);
                    }
                }
        }
        __syncwarp();
        cluster_sync();  // no CTA leaves while its sums may be read
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_free(tmem, kColumns);
    }
    if (threadIdx.x == 0 && bars.gone) report_status(a.status, kStatusTimeout);
}

namespace {

// With narrow tiles k_adapter_proj leaves room for a CTA of k_adapter_low beside it.
constexpr int kLowBudget = 60 * 1024, kProjBudget = 164 * 1024;

int stages_for(int nt, int rank, int budget)
{
    int s = kMaxStages;
    while (s > 2 && static_cast<int>(adapter_layout(nt, s, rank).bytes) > budget) --s;
    return s;
}

template <int NT>
int launch_low(const CUtensorMap& map_a, const CUtensorMap& map_x, AdapterArgs a, int groups, cudaStream_t st)
{
    a.stages_low = stages_for(NT, 0, NT > kSmallTile ? kProjBudget : kLowBudget);
    const size_t smem = adapter_layout(NT, a.stages_low, 0).bytes;
    const int e = ensure_smem(reinterpret_cast<const void*>(&k_adapter_low<NT>), smem);
    if (e != cudaSuccess) return e;
    return launch_kernel(&k_adapter_low<NT>, dim3(a.tiles, a.slices, groups), dim3(kGemmThreads), smem, st, 0, map_a,
                         map_x, a);
}

template <int NT, typename OutT>
int launch_proj(const CUtensorMap& map_w, const CUtensorMap& map_x, const CUtensorMap& map_b, const CUtensorMap& map_s,
                AdapterArgs a, cudaStream_t st)
{
    const int rank = a.n_adapters > 0 ? a.rank : 0;
    a.stages = stages_for(NT, rank, NT > kSmallTile ? 226 * 1024 : kProjBudget);
    const size_t smem = adapter_layout(NT, a.stages, rank).bytes;
    const void* f = reinterpret_cast<const void*>(&k_adapter_proj<NT, OutT>);
    const int e = ensure_smem(f, smem);
    if (e != cudaSuccess) return e;
    while (a.ways > 1 && !cluster_fits(f, kGemmThreads, smem, a.ways)) a.ways /= 2;
    int grid = a.tiles * a.mt * a.ways;
    if (a.ways == 1) grid = persistent_grid(f, kGemmThreads, smem, static_cast<long long>(a.tiles) * a.mt);
    if (grid < 1) return cudaErrorLaunchOutOfResources;
    return launch_kernel(&k_adapter_proj<NT, OutT>, dim3(grid), dim3(kGemmThreads), smem, st, a.ways > 1 ? a.ways : 0, map_w, map_x, map_b, map_s, a);
}

}  // namespace

int launch_adapter_low_rows(const void* x, const void* wa, const AdapterArgs& a, cudaStream_t st)
{
    const long long warps = static_cast<long long>(a.T) * (a.rank / 4) * a.slices;
    const int grid = persistent_grid(reinterpret_cast<const void*>(&k_adapter_low_rows), 256, 0, (warps + 7) / 8);
    if (grid < 1) return cudaErrorLaunchOutOfResources;
    return launch_kernel(&k_adapter_low_rows, dim3(grid), dim3(256), 0, st, 0, static_cast<const __nv_bfloat16*>(x),
                         static_cast<const __nv_bfloat16*>(wa), a);
}

int launch_adapter_few(const void* x, const void* w, const void* wa, bool fused, bool f32, const AdapterArgs& a,
                       cudaStream_t st)
{
    using B = __nv_bfloat16;
    const size_t smem = static_cast<size_t>(a.T) * a.K * 2 + (fused && a.n_adapters > 0 ? static_cast<size_t>(a.T) * a.rank * 4 : 0);
    auto go = [&](auto kernel) -> int {
        const void* f = reinterpret_cast<const void*>(kernel);
        const int e = ensure_smem(f, smem);
        if (e != cudaSuccess) return e;
        const int threads = few_threads(fused), grid = persistent_grid(f, threads, smem, (a.N + threads / 32 - 1) / (threads / 32));
        if (grid < 1) return cudaErrorLaunchOutOfResources;
        return launch_kernel(kernel, dim3(grid), dim3(threads), smem, st, 0, static_cast<const B*>(x), static_cast<const B*>(w),
                             static_cast<const B*>(wa), a);
    };
    auto out = [&](auto as_f32, auto as_bf16) { return f32 ? go(as_f32) : go(as_bf16); };
    if (fused) return out(&k_adapter_few<1, true, float>, &k_adapter_few<1, true, B>);
    if (a.T == 1) return out(&k_adapter_few<1, false, float>, &k_adapter_few<1, false, B>);
    if (a.T == 2) return out(&k_adapter_few<2, false, float>, &k_adapter_few<2, false, B>);
    return out(&k_adapter_few<4, false, float>, &k_adapter_few<4, false, B>);
}

int launch_adapter_low(int nt, const CUtensorMap& map_a, const CUtensorMap& map_x, const AdapterArgs& a, int groups,
                       cudaStream_t st)
{
    switch (nt) {
        case 16: return launch_low<16>(map_a, map_x, a, groups, st);
        case 32: return launch_low<32>(map_a, map_x, a, groups, st);
        case 64: return launch_low<64>(map_a, map_x, a, groups, st);
        case 128: return launch_low<128>(map_a, map_x, a, groups, st);
        default: return launch_low<256>(map_a, map_x, a, groups, st);
    }
}

int launch_adapter_split(int nt, const AdapterArgs& a, cudaStream_t st)
{
    return nt == 128 ? launch_kernel(&k_adapter_split<128>, dim3(a.tiles, 8), dim3(256), 0, st, 0, a)
                     : launch_kernel(&k_adapter_split<256>, dim3(a.tiles, 8), dim3(256), 0, st, 0, a);
}

int launch_adapter_proj(int nt, bool f32, const CUtensorMap& map_w, const CUtensorMap& map_x, const CUtensorMap& map_b,
                        const CUtensorMap& map_s, const AdapterArgs& a, cudaStream_t st)
{
    using B = __nv_bfloat16;
    auto go = [&](auto f) { return f(map_w, map_x, map_b, map_s, a, st); };
    switch (nt) {
        case 16: return f32 ? go(&launch_proj<16, float>) : go(&launch_proj<16, B>);
        case 32: return f32 ? go(&launch_proj<32, float>) : go(&launch_proj<32, B>);
        case 64: return f32 ? go(&launch_proj<64, float>) : go(&launch_proj<64, B>);
        case 128: return go(&launch_proj<128, B>);
        default: return go(&launch_proj<256, B>);
    }
}

}  // namespace mr
