// The experts' products on the tensor cores, over the sorted layout (blocks of
// at most NT pairs of one expert).
//
//   k_experts_up    h[p][i] = act(w13[e][i] . x_t) * (w13[e][I + i] . x_t), as two bf16 parts (16
//                   significant bits) in blocks of at most 64 pairs, else rounded to bf16
//   k_experts_down  y[t][j] = weight * (w2[e] . h[p])
//   k_experts_sum   out[t] = sum_j y[t][j], in slot order
//
// The first two are one persistent CTA per SM over units (block, row tile); see
// gemm.cuh for the operands' roles. A unit of `up` holds 64 gate rows and the same
// 64 up rows, alternating by 16, so that a warp of the epilogue has both factors
// of h and one shuffle brings them together.
//
// Blocks of 32 pairs and more read x from a copy in sorted order that
// k_experts_gather makes: a copy of 4 scattered rows takes the tensor-copy
// engine 80 clocks, of 64 consecutive rows 120, and each row tile of w13 reads
// the block's rows again.
//
// The sum over a token's slots is a kernel of its own. Taken by the unit that
// completes a token (a counter per token and row tile), it cost `down` a fence,
// an atomic and a fence a unit, 4 us of latency that the next unit's products
// did not cover (T=16 E=256 k=8: 83 us instead of 55; T=8192 E=8 k=2: 208 instead
// of 114).
//
// Measured (one GB300, HBM copy 6.78 TB/s, products 1.92 PFLOP/s): T=16 E=256 k=8
// H=2048 I=768 `up` 107 us for 661 MB (6.2 TB/s), `down` 55 us for 333 MB (6.1),
// the sum 7: weights stream at the memory's rate. T=8192 E=8 k=2 H=I=2048 `up` 176
// us (1.56 PFLOP/s), `down` 100 (1.37, beside 134 MB of y), the copy of x 20, the
// sum 25 (5.4 TB/s): the products' rate and what surrounds them.
#include <algorithm>

#include "experts.h"
#include "gemm.cuh"

namespace mr {

namespace {
template <int NT>
constexpr int kTokenBox = NT >= 64 ? NT / 4 : 16;
}  // namespace

// Rows of the token operand: h in two parts is twice as many columns, which cost
// a product nothing up to 128 (gemm.cuh) and spare h the rounding to bf16. A pair's
// CTAs hold half each.
__host__ __device__ constexpr int token_rows(int nt, bool down)
{
    return nt >= kPairColumns ? nt / 2 : down && nt <= kSplitColumns ? 2 * nt : nt;
}

struct CtaLayout {
    uint32_t a, b, info, bars, bytes;
};

// Offsets from the first 1024-byte boundary of the CTA's shared memory.
__host__ __device__ inline CtaLayout cta_layout(int nt, bool down, int stages)
{
    CtaLayout L;
    uint32_t o = 0;
    L.a = o; o += static_cast<uint32_t>(stages) * kRows * kStepBytes;
    L.b = o; o += static_cast<uint32_t>(stages) * token_rows(nt, down) * kStepBytes;
    L.info = o; o += static_cast<uint32_t>(nt) * 8;
    o = (o + 15) / 16 * 16;
    L.bars = o; o += sizeof(GemmBars);
    L.bytes = o + 1024;  // the base is aligned inside
    return L;
}

// Number of this block's pairs: the sort puts them first, then sentinels (ids
// of P). Every lane of the warp calls it.
template <int NT>
__device__ __forceinline__ int block_pairs(const int32_t* ids, int P, int lane)
{
    int n = 0;
#pragma unroll
    for (int i = 0; i < (NT + 31) / 32; ++i) {
        const int c = i * 32 + lane;
        const int id = c < NT ? __ldcg(ids + c) : P;
        n += __popc(__ballot_sync(kFull, id >= 0 && id < P));
    }
    return n;
}

// xs[r] = x[token of sorted row r]; a warp per row.
__global__ void __launch_bounds__(256) k_experts_gather(const __grid_constant__ ExpertArgs a)
{
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = blockIdx.x * 8 + (threadIdx.x >> 5), warps = gridDim.x * 8;
    const int rows = min(__ldcg(a.npp), a.cap);
    for (int r = warp; r < rows; r += warps) {
        const int id = __ldcg(a.sids + r);
        if (id < 0 || id >= a.P) continue;
        const uint4* src = reinterpret_cast<const uint4*>(a.x + static_cast<long long>(id / a.topk) * a.H);
        uint4* dst = reinterpret_cast<uint4*>(a.xs + static_cast<long long>(r) * a.H);
#pragma unroll 4
        for (int c = lane; c < a.H / 8; c += 32) dst[c] = __ldcg(src + c);
    }
}

// out[t] = sum of the token's weighted products in slot order (zeros where no
// slot has an expert); a thread takes 8 columns of a token.
__global__ void __launch_bounds__(256) k_experts_sum(const __grid_constant__ ExpertArgs a)
{
    pdl_wait();
    pdl_trigger();
    const int H8 = a.H / 8;
    const long long n = static_cast<long long>(a.T) * H8;
    for (long long u = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; u < n; u += static_cast<long long>(gridDim.x) * 256) {
        const long long t = u / H8;
        const int c = static_cast<int>(u - t * H8) * 8;
        float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 4
        for (int j = 0; j < a.topk; ++j) {
            const long long pair = t * a.topk + j;
            const int e = __ldcg(a.idx + pair);
            const float4* y = reinterpret_cast<const float4*>(a.y + pair * a.H + c);
            const float4 p = __ldcs(y), q = __ldcs(y + 1);  // of a slot without an expert: whatever is there
            if (e >= 0 && e < a.E) {
                v[0] += p.x; v[1] += p.y; v[2] += p.z; v[3] += p.w;
                v[4] += q.x; v[5] += q.y; v[6] += q.z; v[7] += q.w;
            }
        }
        __nv_bfloat16* o = a.out + t * a.H + c;
        if (a.out16) {
            uint4 w;
            uint32_t* wp = &w.x;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                wp[i] = *reinterpret_cast<const uint32_t*>(&b);
            }
            *reinterpret_cast<uint4*>(o) = w;
        } else {
            for (int i = 0; i < 8; ++i) o[i] = __float2bfloat16_rn(v[i]);
        }
    }
}

template <int NT, bool DOWN>
__global__ void __launch_bounds__(kGemmThreads, 1)
    k_experts(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_t,
              const __grid_constant__ ExpertArgs a)
{
    extern __shared__ unsigned char raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    const CtaLayout L = cta_layout(NT, DOWN, a.stages);
    GemmBars& bars = *reinterpret_cast<GemmBars*>(smem + L.bars);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr bool kPair = NT >= kPairColumns;
    constexpr int kCtas = kPair ? 2 : 1;
    const int rank = kPair ? static_cast<int>(cluster_ctarank()) : 0;
    constexpr bool kSplit = NT <= kSplitColumns;  // h in two parts
    constexpr int kAcc = DOWN && kSplit ? 2 * NT : NT;
    constexpr uint32_t kColumns = 2 * kAcc;  // two accumulators: one fills while the other is read
    constexpr uint32_t a_bytes = kRows * kStepBytes, b_bytes = token_rows(NT, DOWN) * kStepBytes;
    const uint32_t ring_a = smem_addr(smem + L.a), ring_b = smem_addr(smem + L.b);

    if (warp == 1) tmem_alloc<kPair>(&bars.tmem, kColumns);
    if (threadIdx.x == 0) {
        for (int i = 0; i < a.stages; ++i) {
            mbar_init(&bars.full[i], 2);
            mbar_init(&bars.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.acc_full[i], 1);
            mbar_init(&bars.acc_empty[i], 4 * kCtas);  // a warp's arrival each, of both CTAs in the first one's
        }
        mbar_init(&bars.drained, 1);
        bars.gone = 0;
        prefetch_map(&map_w);
        prefetch_map(&map_t);
    }
    tc_fence_before();
    __syncthreads();
    if (kPair) cluster_sync();  // the other CTA's barriers are ready
    tc_fence_after();
    const uint32_t tmem = bars.tmem;

    // `up` follows the sort and lets `down` start; `down` knows then that the
    // sort is done (up's trigger comes after up's own wait) and may fetch
    // weights before `up` ends. Every kernel after them waits before it reads.
    if (!DOWN) pdl_wait();
    pdl_trigger();
    const Waits wait{&bars.gone, a.tries};
    const uint32_t drain = min(a.tries, kDrainTries);
    const int nblk = min(__ldcg(a.npp), a.cap) / NT;
    const int mts = (a.mt + kCtas - 1) / kCtas;  // row tiles, a pair's two as one (the last second one may be past the rows)
    const int units = nblk * mts, first_unit = blockIdx.x / kCtas, stride = gridDim.x / kCtas;
    const int ksteps = ((DOWN ? a.I : a.H) + kStepK - 1) / kStepK;
    RingPos pos;
    int issued = 0;

    if (warp == 0) {
        if (elect_one()) {
            bool ok = true;
            for (int u = first_unit; ok && u < units; u += stride) {
                const int b = u / mts, m = (u - b * mts) * kCtas + rank;
                const int e = min(max(__ldcg(a.eids + b), 0), a.E - 1);
                for (int k = 0; k < ksteps; ++k) {
                    if (DOWN && issued == a.stages) pdl_wait();
                    ok = pos.wraps == 0 || wait(&bars.empty[pos.s], (pos.wraps - 1) & 1);
                    if (!ok) break;
                    uint64_t* full = &bars.full[pos.s];
                    const uint32_t dst = ring_a + pos.s * a_bytes;
                    // a pair's first CTA counts what both bring
                    if (rank == 0) mbar_expect(full, a_bytes * kCtas);
                    ++issued;
                    if (!a.drop) {
                        const uint32_t counted = kPair ? cluster_addr(full, 0) : 0;
                        auto load = [&](uint32_t to, int row) {
                            if (kPair) load_box3_pair(to, &map_w, k * kStepK, row, e, counted);
                            else load_box3(to, &map_w, k * kStepK, row, e, full);
                        };
                        if (DOWN) {
                            load(dst, m * kRows);
                        } else {
                            const int i = m * (kRows / 2);
                            for (int g = 0; g < kRows / 32; ++g) {
                                load(dst + g * 32 * kStepBytes, i + g * 16);
                                load(dst + (g * 32 + 16) * kStepBytes, a.I + i + g * 16);
                            }
                        }
                    }
                    pos.next(a.stages);
                }
            }
            if (!ok)  // copies in flight land before the CTA leaves
                for (int s = 0; s < a.stages && s < issued; ++s)
                    mbar_wait(&bars.full[s], ((issued - 1 - s) / a.stages) & 1, drain);
        }
    } else if (warp == 2) {
        if (DOWN) pdl_wait();
        constexpr bool kScattered = !DOWN && NT < kGatherColumns;
        const int box = kTokenBox<NT>;
        bool ok = true;
        for (int u = first_unit; ok && u < units; u += stride) {
            const int b = u / mts;
            const int32_t* ids = a.sids + static_cast<long long>(b) * NT;
            const int n = block_pairs<NT>(ids, a.P, lane);
            // (a pair's CTAs bring half of the columns' tokens each)
            constexpr int kRound = 16 * kCtas;
            const int cols = max((n + kRound - 1) / kRound, 1) * kRound, boxes = (cols / kCtas + box - 1) / box;
            constexpr int kParts = DOWN && kSplit ? 2 : 1;
            int4 row[kScattered ? NT / 4 : 1];
            if (kScattered) {
#pragma unroll
                for (int g = 0; g < NT / 4; ++g) {
                    const int4 id = __ldcg(reinterpret_cast<const int4*>(ids + g * 4));
                    // a sentinel's column is never read
                    row[g] = make_int4(id.x >= 0 && id.x < a.P ? id.x / a.topk : 0, id.y >= 0 && id.y < a.P ? id.y / a.topk : 0,
                                       id.z >= 0 && id.z < a.P ? id.z / a.topk : 0, id.w >= 0 && id.w < a.P ? id.w / a.topk : 0);
                }
            }
            if (elect_one()) {
                for (int k = 0; k < ksteps; ++k) {
                    ok = pos.wraps == 0 || wait(&bars.empty[pos.s], (pos.wraps - 1) & 1);
                    if (!ok) break;
                    uint64_t* full = &bars.full[pos.s];
                    const uint32_t dst = ring_b + pos.s * b_bytes;
                    if (k == 0) bars.cols[pos.s] = cols * kParts;
                    if (rank == 0) mbar_expect(full, (kScattered ? cols : boxes * box * kCtas * kParts) * kStepBytes);
                    ++issued;
                    if (!a.drop) {
                        if (kScattered) {
#pragma unroll
                            for (int g = 0; g < NT / 4; ++g)
                                if (g * 4 < cols) load_rows4(dst + g * 4 * kStepBytes, &map_t, k * kStepK, row[g], full);
                        } else {
                            const int first = b * NT + rank * (cols / kCtas);
                            for (int g = 0; g < boxes; ++g) {
                                const uint32_t to = dst + g * box * kStepBytes;
                                if (kPair) load_box2_pair(to, &map_t, k * kStepK, first + g * box, cluster_addr(full, 0));
                                else load_box2(to, &map_t, k * kStepK, first + g * box, full);
                                if (kParts == 2) load_box2(to + cols * kStepBytes, &map_t, k * kStepK, a.cap + first + g * box, full);
                            }
                        }
                    }
                    pos.next(a.stages);
                }
                if (!ok)
                    for (int s = 0; s < a.stages && s < issued; ++s)
                        mbar_wait(&bars.full[s], ((issued - 1 - s) / a.stages) & 1, drain);
            }
            ok = __all_sync(kFull, ok);
        }
    } else if (warp == 1) {
        if (rank == 0 && elect_one()) {
            if (DOWN) pdl_wait();
            int seen = 0;
            bool ok = true;
            StagePoll poll;
            for (int u = first_unit; ok && u < units; u += stride, ++seen) {
                const int buf = seen & 1;
                ok = seen < 2 || wait(&bars.acc_empty[buf], ((seen >> 1) - 1) & 1);
                if (!ok) break;
                tc_fence_after();
                const uint32_t d = tmem + buf * kAcc;
                uint32_t desc = 0;
                for (int k = 0; k < ksteps; ++k) {
                    ok = poll.take(wait, bars, pos, a.stages);
                    if (!ok) break;
                    tc_fence_after();
                    if (k == 0) desc = product_desc(bars.cols[pos.s], kPair);
                    const uint64_t da = operand_desc(ring_a + pos.s * a_bytes), db = operand_desc(ring_b + pos.s * b_bytes);
#pragma unroll
                    for (int q = 0; q < kStepK / 16; ++q) mma16<kPair>(d, da + q * 2, db + q * 2, desc, k > 0 || q > 0);
                    if (kPair) mma_commit_pair(&bars.empty[pos.s], 3);
                    else mma_commit(&bars.empty[pos.s]);
                    pos.next(a.stages);
                }
                if (ok && kPair) mma_commit_pair(&bars.acc_full[buf], 3);
                else if (ok) mma_commit(&bars.acc_full[buf]);
            }
            if (!ok) {
                if (kPair) mma_commit_pair(&bars.drained, 1);
                else mma_commit(&bars.drained);
                mbar_wait(&bars.drained, 0, drain);
            }
        }
    } else if (warp >= 4) {
        const int et = threadIdx.x - kEpilogueThreads, q = warp - 4;  // this thread's row of the accumulator
        if (DOWN) pdl_wait();
        int* info = reinterpret_cast<int*>(smem + L.info);  // NT pair ids, NT weights
        float* info_w = reinterpret_cast<float*>(info + NT);
        int seen = 0;
        for (int u = first_unit; u < units; u += stride, ++seen) {
            const int b = u / mts, m = (u - b * mts) * kCtas + rank, buf = seen & 1;
            const int32_t* ids = a.sids + static_cast<long long>(b) * NT;
            const int n = block_pairs<NT>(ids, a.P, lane);
            if (DOWN) {
                for (int c = et; c < n; c += kEpilogueThreads) {
                    const int id = __ldcg(ids + c);
                    info[c] = id;
                    info_w[c] = __ldcg(a.w + id);
                }
            }
            if (!epilogue_wait(wait, &bars.acc_full[buf], (seen >> 1) & 1)) break;
            tc_fence_after();
            const uint32_t acc = tmem + buf * kAcc + (static_cast<uint32_t>(q * 32) << 16);
            if (DOWN) {
                const int row = m * kRows + et;
                const bool mine = row < a.H;
                for (int c0 = 0; c0 < n; c0 += 16) {
                    float v[16];
                    tmem_load16(acc + c0, v);
                    if (kSplit) {
                        float lo[16];
                        tmem_load16(acc + ((n + 15) & ~15) + c0, lo);
#pragma unroll
                        for (int c = 0; c < 16; ++c) v[c] += lo[c];
                    }
#pragma unroll
                    for (int c = 0; c < 16; ++c)
                        if (mine && c0 + c < n)
                            a.y[static_cast<long long>(info[c0 + c]) * a.H + row] = v[c] * info_w[c0 + c];
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (kPair) mbar_arrive_cluster(cluster_addr(&bars.acc_empty[buf], 0));
                    else mbar_arrive(&bars.acc_empty[buf]);
                }
                epilogue_sync();  // the next unit overwrites info
            } else {
                // lanes 0-15 hold gate rows, lanes 16-31 the same up rows: the
                // first finish the even columns, the others the odd ones
                const bool low = lane < 16;
                const int col = m * (kRows / 2) + q * 16 + (lane & 15);
                const bool mine = col < a.I;
                __nv_bfloat16* h = a.h + (static_cast<long long>(b) * NT + (low ? 0 : 1)) * a.I + col;
                for (int c0 = 0; c0 < n; c0 += 16) {
                        float v[16];
                        tmem_load16(acc + c0, v);
#pragma unroll
                        for (int c = 0; c < 16; c += 2) {
                            const float other = __shfl_xor_sync(kFull, low ? v[c + 1] : v[c], 16);
                            const float g = low ? v[c] : other, w = low ? other : v[c + 1];
                            if (mine && c0 + c + (low ? 0 : 1) < n) {
                                const float f = act_f32(g, a.act) * w;
                                __nv_bfloat16* to = h + static_cast<long long>(c0 + c) * a.I;
                                if (kSplit) {
                                    uint32_t hi, lo;
                                    split_f32(f, hi, lo);
                                    *to = __ushort_as_bfloat16(static_cast<unsigned short>(hi));
                                    to[static_cast<long long>(a.cap) * a.I] = __ushort_as_bfloat16(static_cast<unsigned short>(lo));
                                } else {
                                    *to = __float2bfloat16_rn(f);
                                }
                            }
                        }
                    }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (kPair) mbar_arrive_cluster(cluster_addr(&bars.acc_empty[buf], 0));
                    else mbar_arrive(&bars.acc_empty[buf]);
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    if (kPair) cluster_sync();  // no CTA leaves while the other may use its memory or its barriers
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_free<kPair>(tmem, kColumns);
    }
    if (threadIdx.x == 0 && bars.gone) report_status(a.status, kStatusTimeout);
}

int launch_experts_gather(const ExpertArgs& a, cudaStream_t st)
{
    const int grid = persistent_grid(reinterpret_cast<const void*>(&k_experts_gather), 256, 0, (a.cap + 7) / 8);
    if (grid < 1) return cudaErrorLaunchOutOfResources;
    return launch_kernel(&k_experts_gather, dim3(grid), dim3(256), 0, st, 0, a);
}

int launch_experts_sum(const ExpertArgs& a, cudaStream_t st)
{
    const long long n = static_cast<long long>(a.T) * (a.H / 8);
    const int grid = persistent_grid(reinterpret_cast<const void*>(&k_experts_sum), 256, 0, (n + 255) / 256);
    if (grid < 1) return cudaErrorLaunchOutOfResources;
    return launch_kernel(&k_experts_sum, dim3(grid), dim3(256), 0, st, 0, a);
}

namespace {

constexpr int kSmemBudget = 200 * 1024;

// As many stages as the budget holds.
int stages_for(int nt, bool down)
{
    int s = kMaxStages;
    while (s > 2 && cta_layout(nt, down, s).bytes > kSmemBudget) --s;
    return s;
}

template <int NT, bool DOWN>
int launch_one(const CUtensorMap& map_w, const CUtensorMap& map_t, ExpertArgs a, long long units, cudaStream_t st)
{
    a.stages = stages_for(NT, DOWN);
    const size_t smem = cta_layout(NT, DOWN, a.stages).bytes;
    const void* f = reinterpret_cast<const void*>(&k_experts<NT, DOWN>);
    const int e = ensure_smem(f, smem);
    if (e != cudaSuccess) return e;
    constexpr int kCtas = NT >= kPairColumns ? 2 : 1;
    const int grid = kCtas == 1 ? persistent_grid(f, kGemmThreads, smem, units)
                                : 2 * static_cast<int>(std::min<long long>(active_clusters(f, kGemmThreads, smem, 2), (units + 1) / 2));
    if (grid < 1) return cudaErrorLaunchOutOfResources;
    return launch_kernel(&k_experts<NT, DOWN>, dim3(grid), dim3(kGemmThreads), smem, st, kCtas == 2 ? 2 : 0, map_w, map_t, a);
}

template <bool DOWN>
int launch_any(int nt, const CUtensorMap& map_w, const CUtensorMap& map_t, const ExpertArgs& a, long long units,
               cudaStream_t st)
{
    switch (nt) {
        case 16: return launch_one<16, DOWN>(map_w, map_t, a, units, st);
        case 32: return launch_one<32, DOWN>(map_w, map_t, a, units, st);
        case 64: return launch_one<64, DOWN>(map_w, map_t, a, units, st);
        case 128: return launch_one<128, DOWN>(map_w, map_t, a, units, st);
        default: return launch_one<256, DOWN>(map_w, map_t, a, units, st);
    }
}

}  // namespace

int launch_experts_up(int nt, const CUtensorMap& map_w, const CUtensorMap& map_t, const ExpertArgs& a, long long units,
                      cudaStream_t st)
{
    return launch_any<false>(nt, map_w, map_t, a, units, st);
}

int launch_experts_down(int nt, const CUtensorMap& map_w, const CUtensorMap& map_t, const ExpertArgs& a,
                        long long units, cudaStream_t st)
{
    return launch_any<true>(nt, map_w, map_t, a, units, st);
}

}  // namespace mr
