// The experts' products on the tensor cores, over the sorted layout (blocks of
// at most NT pairs of one expert).
//
//   k_experts_up    h[p][i] = act(w13[e][i] . x_t) * (w13[e][I + i] . x_t)
//   k_experts_down  y[t][j] = weight * (w2[e] . h[p]), then out[t] = sum_j y[t][j]
//
// Both are one persistent CTA per SM over units (block, row tile); see gemm.cuh
// for the operands' roles. A unit of `up` holds rows/2 gate rows and the same
// rows/2 up rows, so that one accumulator has both factors of h.
//
// The sum over a token's slots is taken in slot order by whichever unit
// completes the token's last slot (a counter per token and row tile): the same
// bits whatever the order of arrival, and no launch for it.
#include "experts.h"
#include "gemm.cuh"

namespace mr {

struct CtaLayout {
    uint32_t a, b, xchg, info, bars, bytes;
};

// Offsets from the first 1024-byte boundary of the CTA's shared memory.
__host__ __device__ inline CtaLayout cta_layout(int nt, int rows, int stages)
{
    CtaLayout L;
    uint32_t o = 0;
    L.a = o; o += static_cast<uint32_t>(stages) * rows * kStepBytes;
    L.b = o; o += static_cast<uint32_t>(stages) * nt * kStepBytes;
    // a product reads 128 rows from the start of a stage, also of the last one
    const uint32_t reach = static_cast<uint32_t>(stages - 1) * rows * kStepBytes + 128 * kStepBytes;
    if (o < reach) o = reach;
    L.xchg = o; o += 2 * 64 * 17 * 4;
    L.info = o; o += static_cast<uint32_t>(nt) * 8 + 16;
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

template <int NT, bool DOWN>
__global__ void __launch_bounds__(kGemmThreads, 1)
    k_experts(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_t,
              const __grid_constant__ ExpertArgs a)
{
    extern __shared__ unsigned char raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    const CtaLayout L = cta_layout(NT, a.rows, a.stages);
    GemmBars& bars = *reinterpret_cast<GemmBars*>(smem + L.bars);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr uint32_t kColumns = 2 * NT;  // two accumulators: one fills while the other is read
    const uint32_t a_bytes = a.rows * kStepBytes, b_bytes = NT * kStepBytes;
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
        prefetch_map(&map_t);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars.tmem;

    // `up` follows the sort and lets `down` start; `down` knows then that the
    // sort is done (up's trigger comes after up's own wait) and may fetch
    // weights before `up` ends.
    if (!DOWN) {
        pdl_wait();
        pdl_trigger();
    }
    const Waits wait{&bars.gone, a.tries};
    const uint32_t drain = min(a.tries, kDrainTries);
    const int nblk = min(__ldcg(a.npp), a.cap) / NT;
    const int units = nblk * a.mt;
    const int ksteps = ((DOWN ? a.I : a.H) + kStepK - 1) / kStepK;
    RingPos pos;
    int issued = 0;

    if (warp == 0) {
        if (lane == 0) {
            bool ok = true;
            for (int u = blockIdx.x; ok && u < units; u += gridDim.x) {
                const int b = u / a.mt, m = u - b * a.mt;
                const int e = min(max(__ldcg(a.eids + b), 0), a.E - 1);
                for (int k = 0; k < ksteps; ++k) {
                    if (DOWN && issued == a.stages) pdl_wait();
                    ok = pos.wraps == 0 || wait(&bars.empty[pos.s], (pos.wraps - 1) & 1);
                    if (!ok) break;
                    uint64_t* full = &bars.full[pos.s];
                    const uint32_t dst = ring_a + pos.s * a_bytes;
                    mbar_expect(full, a_bytes);
                    ++issued;
                    if (!a.drop) {
                        if (DOWN) {
                            load_box3(dst, &map_w, k * kStepK, m * a.rows, e, full);
                        } else {
                            const int half = a.rows >> 1;
                            load_box3(dst, &map_w, k * kStepK, m * half, e, full);
                            load_box3(dst + half * kStepBytes, &map_w, k * kStepK, a.I + m * half, e, full);
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
        bool ok = true;
        for (int u = blockIdx.x; ok && u < units; u += gridDim.x) {
            const int b = u / a.mt;
            const int32_t* ids = a.sids + static_cast<long long>(b) * NT;
            const int n = block_pairs<NT>(ids, a.P, lane);
            const int cols = max((n + 15) & ~15, 16);
            constexpr int kGathers = (NT / 4 + 31) / 32;
            int4 row[kGathers];
            if (!DOWN) {
#pragma unroll
                for (int i = 0; i < kGathers; ++i) {
                    const int g = i * 32 + lane;
                    int r[4] = {0, 0, 0, 0};
                    if (g * 4 < cols)
                        for (int q = 0; q < 4; ++q) {
                            const int id = __ldcg(ids + g * 4 + q);
                            r[q] = id >= 0 && id < a.P ? id / a.topk : 0;  // a sentinel's column is never read
                        }
                    row[i] = make_int4(r[0], r[1], r[2], r[3]);
                }
            }
            for (int k = 0; k < ksteps; ++k) {
                ok = __all_sync(kFull, pos.wraps == 0 || wait(&bars.empty[pos.s], (pos.wraps - 1) & 1));
                if (!ok) break;
                uint64_t* full = &bars.full[pos.s];
                const uint32_t dst = ring_b + pos.s * b_bytes;
                if (lane == 0) {
                    if (k == 0) bars.cols[pos.s] = cols;
                    mbar_expect(full, cols * kStepBytes);
                }
                ++issued;
                __syncwarp();
                if (!a.drop) {
                    if (DOWN) {
                        if (lane * 16 < cols)
                            load_box2(dst + lane * 16 * kStepBytes, &map_t, k * kStepK, b * NT + lane * 16, full);
                    } else {
#pragma unroll
                        for (int i = 0; i < kGathers; ++i) {
                            const int g = i * 32 + lane;
                            if (g * 4 < cols) load_rows4(dst + g * 4 * kStepBytes, &map_t, k * kStepK, row[i], full);
                        }
                    }
                }
                pos.next(a.stages);
            }
        }
        if (!ok && lane == 0)
            for (int s = 0; s < a.stages && s < issued; ++s)
                mbar_wait(&bars.full[s], ((issued - 1 - s) / a.stages) & 1, drain);
    } else if (warp == 1) {
        if (lane == 0) {
            if (DOWN) pdl_wait();
            int seen = 0;
            bool ok = true;
            for (int u = blockIdx.x; ok && u < units; u += gridDim.x, ++seen) {
                const int buf = seen & 1;
                ok = seen < 2 || wait(&bars.acc_empty[buf], ((seen >> 1) - 1) & 1);
                if (!ok) break;
                tc_fence_after();
                const uint32_t d = tmem + buf * NT;
                uint32_t desc = 0;
                for (int k = 0; k < ksteps; ++k) {
                    ok = wait(&bars.full[pos.s], pos.wraps & 1);
                    if (!ok) break;
                    tc_fence_after();
                    if (k == 0) desc = product_desc(bars.cols[pos.s]);
                    const uint64_t da = operand_desc(ring_a + pos.s * a_bytes), db = operand_desc(ring_b + pos.s * b_bytes);
#pragma unroll
                    for (int q = 0; q < kStepK / 16; ++q) mma16(d, da + q * 2, db + q * 2, desc, k > 0 || q > 0);
                    mma_commit(&bars.empty[pos.s]);
                    pos.next(a.stages);
                }
                if (ok) mma_commit(&bars.acc_full[buf]);
            }
            if (!ok) {
                mma_commit(&bars.drained);
                mbar_wait(&bars.drained, 0, drain);
            }
        }
    } else if (warp >= 4) {
        const int et = threadIdx.x - kEpilogueThreads, q = warp - 4;  // this thread's row of the accumulator
        if (DOWN) pdl_wait();
        if (!DOWN) {
            // the counters of `down`, and the rows of tokens without any expert
            for (int t = blockIdx.x * 4 + q; t < a.T; t += gridDim.x * 4) {
                int none = 0;
                for (int j = lane; j < a.topk; j += 32) {
                    const int e = __ldcg(a.idx + static_cast<long long>(t) * a.topk + j);
                    none += e < 0 || e >= a.E;
                }
                for (int o = 16; o > 0; o >>= 1) none += __shfl_xor_sync(kFull, none, o);
                for (int m = lane; m < a.mt_down; m += 32) a.count[static_cast<long long>(t) * a.mt_down + m] = none;
                if (none == a.topk)
                    for (int c = lane; c < a.H; c += 32)
                        a.out[static_cast<long long>(t) * a.H + c] = __float2bfloat16_rn(0.0f);
            }
        }
        float* xchg = reinterpret_cast<float*>(smem + L.xchg);
        int* info = reinterpret_cast<int*>(smem + L.info);  // NT pair ids, then NT weights
        float* info_w = reinterpret_cast<float*>(info + NT);
        int* ndone = info + 2 * NT;
        int seen = 0;
        for (int u = blockIdx.x; u < units; u += gridDim.x, ++seen) {
            const int b = u / a.mt, m = u - b * a.mt, buf = seen & 1;
            const int32_t* ids = a.sids + static_cast<long long>(b) * NT;
            const int n = block_pairs<NT>(ids, a.P, lane);
            if (DOWN) {
                for (int c = et; c < n; c += kEpilogueThreads) {
                    const int id = __ldcg(ids + c);
                    info[c] = id;
                    info_w[c] = __ldcg(a.w + id);
                }
                if (et == 0) *ndone = 0;
            }
            if (!epilogue_wait(wait, &bars.acc_full[buf], (seen >> 1) & 1)) break;
            tc_fence_after();
            const uint32_t acc = tmem + buf * NT + (static_cast<uint32_t>(q * 32) << 16);
            if (DOWN) {
                const int row = m * a.rows + et;
                const bool mine = et < a.rows && row < a.H;
                for (int c0 = 0; c0 < n; c0 += 16) {
                    float v[16];
                    tmem_load16(acc + c0, v);
#pragma unroll
                    for (int c = 0; c < 16; ++c)
                        if (mine && c0 + c < n)
                            a.y[static_cast<long long>(info[c0 + c]) * a.H + row] = v[c] * info_w[c0 + c];
                }
                tc_fence_before();
                mbar_arrive(&bars.acc_empty[buf]);
                __threadfence();
                epilogue_sync();
                for (int c = et; c < n; c += kEpilogueThreads) {
                    const int t = info[c] / a.topk;
                    const int old = atomicAdd(a.count + static_cast<long long>(t) * a.mt_down + m, 1);
                    if (old == a.topk - 1) reinterpret_cast<int*>(xchg)[atomicAdd(ndone, 1)] = t;
                }
                epilogue_sync();
                __threadfence();
                const int done = *ndone;
                for (int i = 0; i < done; ++i) {
                    const long long t = reinterpret_cast<int*>(xchg)[i];
                    if (!mine) continue;
                    float sum = 0.0f;
                    for (int j = 0; j < a.topk; ++j) {
                        const int e = __ldcg(a.idx + t * a.topk + j);
                        const float y = __ldcg(a.y + (t * a.topk + j) * a.H + row);
                        if (e >= 0 && e < a.E) sum += y;
                    }
                    a.out[t * a.H + row] = __float2bfloat16_rn(sum);
                }
                epilogue_sync();  // the next unit overwrites info
            } else {
                const int half = a.rows >> 1;
                const bool gate = et < half, up = et >= half && et < a.rows;
                const int i = gate ? et : et - half, col = m * half + i;
                const bool mine = (gate || up) && col < a.I;
                float* to_up = xchg + i * 17;              // gate rows' later columns
                float* to_gate = xchg + (64 + i) * 17;     // up rows' earlier columns
                for (int c0 = 0; c0 < n; c0 += 16) {
                    float v[16];
                    tmem_load16(acc + c0, v);
                    if (gate)
                        for (int c = 8; c < 16; ++c) to_up[c] = v[c];
                    else if (up)
                        for (int c = 0; c < 8; ++c) to_gate[c] = v[c];
                    epilogue_sync();
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const int at = c0 + (gate ? c : c + 8);
                        const float g = gate ? v[c] : to_up[c + 8], w = gate ? to_gate[c] : v[c + 8];
                        if (mine && at < n)
                            a.h[(static_cast<long long>(b) * NT + at) * a.I + col] = __float2bfloat16_rn(act_f32(g, a.act) * w);
                    }
                    epilogue_sync();
                }
                tc_fence_before();
                mbar_arrive(&bars.acc_empty[buf]);
            }
        }
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

constexpr int kSmemBudget = 200 * 1024;

// As many stages as the budget holds.
int stages_for(int nt, int rows, int ksteps)
{
    int s = kMaxStages;
    while (s > 2 && cta_layout(nt, rows, s).bytes > kSmemBudget) --s;
    (void)ksteps;
    return s;
}

template <int NT, bool DOWN>
int launch_one(const CUtensorMap& map_w, const CUtensorMap& map_t, ExpertArgs a, long long units, cudaStream_t st)
{
    a.stages = stages_for(NT, a.rows, 0);
    const size_t smem = cta_layout(NT, a.rows, a.stages).bytes;
    const void* f = reinterpret_cast<const void*>(&k_experts<NT, DOWN>);
    const int e = ensure_smem(f, smem);
    if (e != cudaSuccess) return e;
    const int grid = persistent_grid(f, kGemmThreads, smem, units);
    if (grid < 1) return cudaErrorLaunchOutOfResources;
    return launch_kernel(&k_experts<NT, DOWN>, dim3(grid), dim3(kGemmThreads), smem, st, 0, map_w, map_t, a);
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
