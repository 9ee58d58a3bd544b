// Tokens to rows sorted by expert and back, with their gradients: moe_permute_fwd / bwd and moe_combine_fwd / bwd.
//
//   rows[r(t,j)] = x[t], 0 at the sort's padding                 (permute; its gradient sums a token's rows)
//   out[t] = residual[t] + m[t] * sum_j w[t,j] rows[r(t,j)]      (combine; m: dropout's factors, see rows.cuh)
//   g = m[t] grad_out[t]:  grad_rows[r(t,j)] = w[t,j] g,  grad_w[t,j] = <g, rows[r(t,j)]>;  a dropped element's part of
//   both is 0 whatever weight or row hold
// All are bound by memory. A token's slots are summed in slot order in fp32 and rounded once: no atomic sums, the same
// bits each time.
#include <algorithm>
#include <climits>

#include "rows.cuh"

namespace mr {
namespace {

// ---- permute ---------------------------------------------------------------

struct PermuteArgs {
    const void* x;
    const int32_t* topk_idx;
    const int32_t* ids;
    const int32_t* npp;
    void* rows;
    int32_t* pair_row;
    int32_t* status;
    int P, topk, n_rows, E_tot;
    int words;  // of a row
    int wc;
};

__device__ __forceinline__ int load_relaxed(const int32_t* p)
{
    int v;
    asm volatile("ld.relaxed.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void store_relaxed(int32_t* p, int v)
{
    asm volatile("st.relaxed.gpu.global.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// A row writes its number to its pair's entry of pair_row, unless topk_idx drops the pair; a pair that no row holds (the
// sort dropped it, its row lies behind the buffer, its id is missing) gets -1 without a pass before this one: what its
// entry held before, whatever that is, stands only where the row of that number holds the pair, and is exchanged for -1
// otherwise, unless the row's own number has come in meanwhile.
//
// A warp copies 32 * N words of a row, all of its loads in flight before the first store, the next row's id behind them.
// Bound by the writes: rows are evicted first, which leaves L2 to x, whose rows are read topk times (8192 tokens, 64
// experts, topk 8, 2048 columns in bf16: 62 us instead of 68), and handed out in eight waves of CTAs, since memory
// serves some SMs faster than others (51 us, 6.1 TB/s; two waves 58, each SM an equal share 62, a CTA for every few rows
// 61).
template <typename Word, int N>
__global__ void __launch_bounds__(kRowsThreads) k_permute(const __grid_constant__ PermuteArgs a)
{
    pdl_trigger_small();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int across = 1 << a.wc, tall = (kRowsThreads / 32) >> a.wc;
    const int first = (static_cast<int>(blockIdx.y) * across + (warp & (across - 1))) * 32 * N;
    const long long pairs_step = static_cast<long long>(gridDim.x) * kRowsThreads;
    long long pair = static_cast<long long>(blockIdx.x) * kRowsThreads + threadIdx.x;
    int expert = 0, was = -1;
    auto look = [&] {
        if (blockIdx.y != 0 || pair >= a.P) return false;
        expert = __ldcg(a.topk_idx + pair);
        was = load_relaxed(a.pair_row + pair);
        return true;
    };
    bool mine = look();
    int rows = __ldcg(a.npp);
    if (rows > a.n_rows) {
        if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) report_status(a.status, kStatusRange);
        rows = a.n_rows;
    }
    const long long step = static_cast<long long>(gridDim.x) * tall;
    long long r = static_cast<long long>(blockIdx.x) * tall + (warp >> a.wc);
    int next = r < rows ? __ldcg(a.ids + r) : 0;
    while (mine) {
        if (expert < 0 || expert >= a.E_tot) store_relaxed(a.pair_row + pair, -1);
        else if (was != -1 && (was < 0 || was >= rows || __ldcg(a.ids + was) != pair)) atomicCAS(a.pair_row + pair, was, -1);
        pair += pairs_step;
        mine = look();
    }
    if (first >= a.words) return;
    for (; r < rows; r += step) {
        const int id = next;
        if (r + step < rows) next = __ldcg(a.ids + r + step);
        const bool real = id >= 0 && id < a.P;
        const int of = real && first == 0 && lane == 0 ? __ldcg(a.topk_idx + id) : -1;
        Word v[N];
        const Word* src = static_cast<const Word*>(a.x) + static_cast<long long>(real ? id / a.topk : 0) * a.words;
        Word* dst = static_cast<Word*>(a.rows) + r * a.words;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = first + 32 * i + lane;
            v[i] = Word{};
            if (real && c < a.words) v[i] = src[c];
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = first + 32 * i + lane;
            if (c < a.words) __stcs(dst + c, v[i]);
        }
        if (first == 0 && lane == 0) {
            if (of >= 0 && of < a.E_tot) store_relaxed(a.pair_row + id, static_cast<int32_t>(r));
            else if (real || id != a.P) report_status(a.status, kStatusRange);
        }
    }
}

// ---- a token's rows, summed ------------------------------------------------

struct CombineArgs {
    const void* rows;
    const int32_t* pair_row;
    const float* w;         // null: ones
    const void* residual;   // null: none
    void* out;
    int32_t* status;
    DropArgs drop;
    int T, topk, n_rows, W, wc;
};

// A warp sums a span of a token: the rows' numbers and weights a lane each, then the rows four at a time. Bound by memory
// and, behind it, by the loads in flight: five CTAs an SM with four rows a warp (8192 tokens, topk 8, 2048 columns in bf16
// with dropout and residual: 54.7 us, 6.1 TB/s) do better than three with eight (57.8) or six (55.9), which spill more
// (five: 8 bytes, with dropout), and four waves than one where topk is small (4096 tokens, topk 4: 13.4 us against 14.1,
// 16.7 with eight rows). fp32 rows take 32 bytes a lane and are best left alone, in one wave (8192 tokens, topk 2, 4096
// columns with dropout: 68.7 us, 5.9 TB/s; three 70.8).
template <typename T, bool VEC>
constexpr int combine_ctas() { return sizeof(T) == 2 && VEC ? 5 : 0; }  // 0: the compiler's choice

template <typename T, bool VEC, bool DROP>
__global__ void __launch_bounds__(kRowsThreads, combine_ctas<T, VEC>()) k_combine(const __grid_constant__ CombineArgs a)
{
    constexpr int kBatch = 4;
    pdl_trigger_small();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int across = 1 << a.wc, tall = (kRowsThreads / 32) >> a.wc;
    const int c0 = (static_cast<int>(blockIdx.y) * across + (warp & (across - 1))) * kSpan;
    if (c0 >= a.W) return;
    const T* rows = static_cast<const T*>(a.rows);
    DropState ds;
    if constexpr (DROP) ds = drop_state(a.drop);
    for (long long t = static_cast<long long>(blockIdx.x) * tall + (warp >> a.wc); t < a.T;
         t += static_cast<long long>(gridDim.x) * tall) {
        Pack<T> q;
        float v[8] = {};
        for (int j0 = 0; j0 < a.topk; j0 += 32) {
            int r = -1;
            float w = 1.0f;
            if (j0 + lane < a.topk) {
                r = __ldcg(a.pair_row + t * a.topk + j0 + lane);
                if (a.w) w = __ldcg(a.w + t * a.topk + j0 + lane);
                if (r < -1 || r >= a.n_rows) {
                    report_status(a.status, kStatusRange);
                    r = -1;
                }
            }
            const int n = min(32, a.topk - j0);
            for (int j = 0; j < n; j += kBatch) {
                Pack<T> p[kBatch];
                int rj[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    rj[i] = __shfl_sync(kFull, r, (j + i) & 31);
                    if (j + i >= n) rj[i] = -1;
                    if (rj[i] >= 0) load_span<VEC>(rows + static_cast<long long>(rj[i]) * a.W, c0, a.W, lane, p[i]);
                }
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const float wj = __shfl_sync(kFull, w, (j + i) & 31);
                    if (rj[i] < 0) continue;
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = fmaf(wj, p[i].get(e), v[e]);
                }
            }
        }
        if constexpr (DROP) drop_span<VEC>(a.drop, ds, static_cast<uint32_t>(t), c0, lane, v);
        if (a.residual) {
            Pack<T> p;
            load_span<VEC>(static_cast<const T*>(a.residual) + t * a.W, c0, a.W, lane, p);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += p.get(e);
        }
        q.set(v);
        store_span<VEC>(static_cast<T*>(a.out) + t * a.W, c0, a.W, lane, q);
    }
}

// ---- the weighted sum's gradient ---------------------------------------------

struct CombineBwdArgs {
    const void* grad_out;
    const void* rows;
    const int32_t* pair_row;
    const float* w;
    const int32_t* ids;
    const int32_t* npp;
    void* grad_rows;
    float* grad_w;
    int32_t* status;
    DropArgs drop;
    int T, topk, n_rows, W, wc;
    int pad_span, pads;  // sorted positions of a share, shares
};

// Zeroes the padding rows among the sorted positions from u * pad_span on, pad_span of them (at most 32).
template <bool VEC, typename T>
__device__ __forceinline__ void zero_padding(const CombineBwdArgs& a, long long u, int lane)
{
    const long long first = u * a.pad_span;
    bool pad = false;
    if (lane < a.pad_span && first + lane < min(__ldcg(a.npp), a.n_rows)) {
        const int id = __ldcg(a.ids + first + lane);
        pad = id < 0 || id >= static_cast<long long>(a.T) * a.topk;
    }
    for (unsigned m = __ballot_sync(kFull, pad); m; m &= m - 1) {
        T* row = static_cast<T*>(a.grad_rows) + (first + __ffs(m) - 1) * a.W;
        const Pack<T> zero = {};
        for (int c0 = 0; c0 < a.W; c0 += kSpan) store_span<VEC>(row, c0, a.W, lane, zero);
    }
}

// A warp per pair, a token's pairs side by side so that its gradient comes from L2 or L1 after the first; behind the
// pairs the padding rows. The kernel without dropout: 8192 tokens, topk 8, 2048 columns in bf16 take 93 us (6.2 TB/s),
// 98 with a token's pairs in one warp.
template <typename T, bool VEC, bool DROP>
__global__ void __launch_bounds__(kRowsThreads) k_combine_bwd_pairs(const __grid_constant__ CombineBwdArgs a)
{
    constexpr int kBatch = sizeof(T) == 2 ? 4 : 2;
    pdl_trigger_small();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const long long P = static_cast<long long>(a.T) * a.topk, warps = static_cast<long long>(gridDim.x) * (kRowsThreads / 32);
    const long long units = P + a.pads;
    DropState ds;
    if constexpr (DROP) ds = drop_state(a.drop);
    for (long long u = static_cast<long long>(blockIdx.x) * (kRowsThreads / 32) + (threadIdx.x >> 5); u < units; u += warps) {
        if (u >= P) {
            zero_padding<VEC, T>(a, u - P, lane);
            continue;
        }
        int r = __ldcg(a.pair_row + u);
        const float w = __ldcg(a.w + u);
        if (r < -1 || r >= a.n_rows) {
            if (lane == 0) report_status(a.status, kStatusRange);
            r = -1;
        }
        float dot = 0.0f;
        if (r >= 0) {
            const uint32_t t = static_cast<uint32_t>(u / a.topk);
            const T* g = static_cast<const T*>(a.grad_out) + static_cast<long long>(t) * a.W;
            const T* row = static_cast<const T*>(a.rows) + static_cast<long long>(r) * a.W;
            T* grad = static_cast<T*>(a.grad_rows) + static_cast<long long>(r) * a.W;
            for (int c = 0; c < a.W; c += kBatch * kSpan) {
                Pack<T> pg[kBatch], pr[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    load_span<VEC, false>(row, c + i * kSpan, a.W, lane, pr[i]);
                    load_span<VEC, false>(g, c + i * kSpan, a.W, lane, pg[i], false);
                }
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int c0 = c + i * kSpan;
                    if (c0 >= a.W) break;
                    float v[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = pg[i].get(e);
                    Keep<T> keep;
                    if constexpr (DROP) {
                        drop_span<VEC>(a.drop, ds, t, c0, lane, v, keep);
                        keep.apply(pr[i]);
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        dot = fmaf(v[e], pr[i].get(e), dot);
                        v[e] *= w;
                    }
                    Pack<T> q;
                    q.set(v);
                    if constexpr (DROP) keep.apply(q);
                    store_span<VEC>(grad, c0, a.W, lane, q);
                }
            }
        }
        dot = warp_sum(dot);
        if (lane == 0) a.grad_w[u] = dot;
    }
}

__device__ __forceinline__ bool not_finite(float v) { return (__float_as_uint(v) & 0x7f800000u) == 0x7f800000u; }

// A warp's spans c0, c0 + step, ... of the pair of token t and row r once more, where an infinity or a NaN has met a dropped
// element: gives the lanes' sum of <g, row> over the kept elements, and writes the row's gradient, 0 at the others. A sum
// that is NaN or a weight that is not finite brings a pair here (0 times an infinity is NaN, so nothing else can hide): a
// look at each element, which the kernel of pairs takes, holds this one's four rows up (8192 tokens, topk 4, 4096 columns
// in bf16 99 us against 97.5; 1001 columns 79 against 61).
template <typename T, bool VEC>
__device__ __forceinline__ float pair_again(const CombineBwdArgs& a, long long t, int r, float w, int c0, int step, int lane)
{
    const T* g = static_cast<const T*>(a.grad_out) + t * a.W;
    const T* row = static_cast<const T*>(a.rows) + static_cast<long long>(r) * a.W;
    T* grad = static_cast<T*>(a.grad_rows) + static_cast<long long>(r) * a.W;
    float dot = 0.0f;
    for (; c0 < a.W; c0 += step) {
#pragma unroll 1
        for (int e = 0; e < 8; ++e) {
            const int c = span_column<VEC>(c0, lane, e);
            if (c >= a.W) break;
            const float m = drop_factor(a.drop, drop_state(a.drop), static_cast<uint32_t>(t), c);
            const float v = m != 0.0f ? static_cast<float>(g[c]) * m : 0.0f;
            if (m != 0.0f) dot = fmaf(v, static_cast<float>(row[c]), dot);
            grad[c] = static_cast<T>(m != 0.0f ? v * w : 0.0f);
        }
    }
    return warp_sum(dot);
}

// With dropout: 2^wc warps share a token. Each takes every 2^wc-th span of its gradient, makes the factors there once
// for kTokenRows of the token's rows at a time, and adds their dot products over its lanes, then the warps' in their
// order. 8192 tokens, topk 4, 4096 columns in bf16: 97.7 us (6.4 TB/s) against 127 with the factors made for every pair;
// where four rows and four warps took 97, eight rows took 110, eight warps a token 100, one 106. Behind the tokens the
// padding rows.
constexpr int kTokenRows = 4;
constexpr int kTokenWarpsLog2 = 2;

template <typename T, bool VEC>
__global__ void __launch_bounds__(kRowsThreads) k_combine_bwd_tokens(const __grid_constant__ CombineBwdArgs a)
{
    constexpr int KB = kTokenRows;
    __shared__ float part[2][kRowsThreads / 32][KB];
    pdl_trigger_small();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int across = 1 << a.wc, tall = (kRowsThreads / 32) >> a.wc, mine = warp & (across - 1);
    const DropState ds = drop_state(a.drop);
    int turn = 0;
    for (long long t0 = static_cast<long long>(blockIdx.x) * tall; t0 < a.T; t0 += static_cast<long long>(gridDim.x) * tall) {
        const long long t = t0 + (warp >> a.wc);
        const T* g = static_cast<const T*>(a.grad_out) + t * a.W;
        for (int j0 = 0; j0 < a.topk; j0 += KB) {
            int r = -1;
            float w = 0.0f;
            if (t < a.T && lane < KB && j0 + lane < a.topk) {
                r = __ldcg(a.pair_row + t * a.topk + j0 + lane);
                w = __ldcg(a.w + t * a.topk + j0 + lane);
                if (r < -1 || r >= a.n_rows) {
                    if (mine == 0) report_status(a.status, kStatusRange);
                    r = -1;
                }
            }
            const bool any = __any_sync(kFull, r >= 0);
            float dot[KB] = {};
            for (int c0 = mine * kSpan; any && c0 < a.W; c0 += across * kSpan) {
                Pack<T> pg, pr[KB];
                load_span<VEC>(g, c0, a.W, lane, pg, j0 + KB >= a.topk);
#pragma unroll
                for (int j = 0; j < KB; ++j) {
                    const int rj = __shfl_sync(kFull, r, j);
                    if (rj >= 0) load_span<VEC>(static_cast<const T*>(a.rows) + static_cast<long long>(rj) * a.W, c0, a.W, lane, pr[j]);
                }
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = pg.get(e);
                drop_span<VEC>(a.drop, ds, static_cast<uint32_t>(t), c0, lane, v);
#pragma unroll
                for (int j = 0; j < KB; ++j) {
                    const int rj = __shfl_sync(kFull, r, j);
                    const float wj = __shfl_sync(kFull, w, j);
                    if (rj < 0) continue;
                    float o[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        dot[j] = fmaf(v[e], pr[j].get(e), dot[j]);
                        o[e] = v[e] * wj;
                    }
                    Pack<T> q;
                    q.set(o);
                    store_span<VEC>(static_cast<T*>(a.grad_rows) + static_cast<long long>(rj) * a.W, c0, a.W, lane, q);
                }
            }
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < KB; ++j) {
                const float s = warp_sum(dot[j]);
                if (lane == j) sum = s;
            }
            for (unsigned redo = __ballot_sync(kFull, r >= 0 && (sum != sum || not_finite(w))); redo; redo &= redo - 1) {
                const int j = __ffs(redo) - 1;
                const float s = pair_again<T, VEC>(a, t, __shfl_sync(kFull, r, j), __shfl_sync(kFull, w, j), mine * kSpan,
                                                   across * kSpan, lane);
                if (lane == j) sum = s;
            }
            if (across > 1) {
                if (lane < KB) part[turn][warp][lane] = sum;
                __syncthreads();
                if (mine == 0 && lane < KB)
                    for (int i = 1; i < across; ++i) sum += part[turn][warp + i][lane];
                turn ^= 1;
            }
            if (mine == 0 && t < a.T && lane < KB && j0 + lane < a.topk) a.grad_w[t * a.topk + j0 + lane] = sum;
        }
    }
    const long long warps = static_cast<long long>(gridDim.x) * (kRowsThreads / 32);
    for (long long u = static_cast<long long>(blockIdx.x) * (kRowsThreads / 32) + warp; u < a.pads; u += warps)
        zero_padding<VEC, T>(a, u, lane);
}

// ---- host --------------------------------------------------------------------

int check_rows(const mr_rows_params* p)
{
    if (!p) return MR_EINVAL;
    if (p->T < 0 || p->H < 1 || p->topk < 1 || p->n_rows < 0) return MR_EINVAL;
    if (p->dtype != MR_F32 && p->dtype != MR_BF16) return MR_EINVAL;
    if (static_cast<long long>(p->T) * p->topk >= INT_MAX) return MR_EINVAL;
    return p->H > MR_MAX_WIDTH ? MR_EUNSUPPORTED : MR_OK;
}

template <typename Word, int N>
int permute(PermuteArgs a, size_t row_bytes, cudaStream_t st)
{
    a.words = static_cast<int>(row_bytes / sizeof(Word));
    const int spans = (a.words + 32 * N - 1) / (32 * N);
    a.wc = warps_across(spans);
    const dim3 grid = span_grid(reinterpret_cast<const void*>(k_permute<Word, N>), a.n_rows, spans, a.wc, 8);
    if (grid.x < 1) return MR_ECUDA;
    const int e = launch_kernel(k_permute<Word, N>, grid, dim3(kRowsThreads), 0, st, 0, a);
    return e == cudaSuccess ? MR_OK : MR_ECUDA;
}

template <typename T, bool VEC, bool DROP>
int combine(CombineArgs a, cudaStream_t st)
{
    const int spans = spans_of(a.W);
    a.wc = warps_across(spans);
    const dim3 grid = span_grid(reinterpret_cast<const void*>(k_combine<T, VEC, DROP>), a.T, spans, a.wc, sizeof(T) == 2 ? 4 : 0);
    if (grid.x < 1) return MR_ECUDA;
    const int e = launch_kernel(k_combine<T, VEC, DROP>, grid, dim3(kRowsThreads), 0, st, 0, a);
    return e == cudaSuccess ? MR_OK : MR_ECUDA;
}

template <typename T>
int combine_of(const CombineArgs& a, cudaStream_t st)
{
    const size_t n = kVecBytes<T>;
    const bool vec = a.W % 8 == 0 && at_multiple(a.rows, n) && at_multiple(a.out, n) && at_multiple(a.residual, n);
    if (a.drop.cut) return vec ? combine<T, true, true>(a, st) : combine<T, false, true>(a, st);
    return vec ? combine<T, true, false>(a, st) : combine<T, false, false>(a, st);
}

template <typename T, bool VEC, bool DROP>
int combine_bwd(CombineBwdArgs a, cudaStream_t st)
{
    const int warps = kRowsThreads / 32;
    const long long pairs = static_cast<long long>(a.T) * a.topk;
    // a warp's share of the padding: small layouts are mostly padding and want all SMs for it (64 tokens, 256 experts,
    // topk 8, blocks of 16, H=2048: 5.2 us against 16.1 with 32 rows a warp; 2048 tokens, 64 experts, topk 4, blocks of 64
    // 16.7 against 18.6), in large ones there is little to do and both do alike (8192 tokens, topk 8, 64 experts 93.0 with
    // 32, 93.6 with 4). It is the part of padding that counts, not the number of rows: a large layout that is mostly
    // padding is on the wrong side (512 tokens, 384 experts, topk 8, blocks of 128: 45.0 us, 38.2 with 4)
    a.pad_span = a.n_rows <= 32768 ? 4 : 32;
    a.pads = static_cast<int>((static_cast<long long>(a.n_rows) + a.pad_span - 1) / a.pad_span);  // n_rows may be INT_MAX
    if constexpr (DROP) {
        // bf16, H=2048, by tokens (pair by pair): T=1024 topk 4 12.7 us (14.0), T=2048 topk 4 19.4 (24.0); below the rule's
        // sizes T=1024 topk 1 10.5 (7.8), T=512 topk 4 10.0 (8.6), T=2048 topk 2 15.7 (13.9). At its border pairs are
        // still better: T=512 topk 8 15.1 (13.8), T=1366 topk 3 15.3 (14.0)
        if (a.topk >= 3 && pairs >= 4096) {
            const auto kernel = k_combine_bwd_tokens<T, VEC>;
            a.wc = std::min(warps_across(spans_of(a.W)), kTokenWarpsLog2);
            const int tall = warps >> a.wc;
            const long long g = dynamic_grid(reinterpret_cast<const void*>(kernel), (a.T + tall - 1) / tall, 4);
            if (g < 1) return MR_ECUDA;
            const int e = launch_kernel(kernel, dim3(static_cast<unsigned>(g)), dim3(kRowsThreads), 0, st, 0, a);
            return e == cudaSuccess ? MR_OK : MR_ECUDA;
        }
    }
    const auto kernel = k_combine_bwd_pairs<T, VEC, DROP>;
    const int g = persistent_grid(reinterpret_cast<const void*>(kernel), kRowsThreads, 0, (pairs + a.pads + warps - 1) / warps, true);
    if (g < 1) return MR_ECUDA;
    const int e = launch_kernel(kernel, dim3(g), dim3(kRowsThreads), 0, st, 0, a);
    return e == cudaSuccess ? MR_OK : MR_ECUDA;
}

template <typename T>
int combine_bwd_of(const CombineBwdArgs& a, cudaStream_t st)
{
    const size_t n = kVecBytes<T>;
    const bool vec = a.W % 8 == 0 && at_multiple(a.rows, n) && at_multiple(a.grad_out, n) && at_multiple(a.grad_rows, n);
    if (a.drop.cut) return vec ? combine_bwd<T, true, true>(a, st) : combine_bwd<T, false, true>(a, st);
    return vec ? combine_bwd<T, true, false>(a, st) : combine_bwd<T, false, false>(a, st);
}

int combine_call(const mr_rows_params& p, const void* rows, const int32_t* pair_row, const float* w, const void* residual,
                 const DropArgs& drop, void* out, int32_t* status, cudaStream_t st)
{
    const CombineArgs a = {rows, pair_row, w, residual, out, status, drop, p.T, p.topk, p.n_rows, p.H, 0};
    return p.dtype == MR_F32 ? combine_of<float>(a, st) : combine_of<__nv_bfloat16>(a, st);
}

}  // namespace
}  // namespace mr

using namespace mr;

extern "C" {

int moe_permute_fwd(const mr_rows_params* p, int E_tot, const void* x, const int32_t* topk_idx,
                    const int32_t* sorted_token_ids, const int32_t* num_tokens_post_pad, void* rows, int32_t* pair_row,
                    int32_t* status, mr_stream_t stream)
{
    const int rc = check_rows(p);
    if (rc != MR_OK) return rc;
    if (E_tot < 1) return MR_EINVAL;
    if (p->T == 0) return MR_OK;
    const size_t size = element(p->dtype);
    if (!x || !topk_idx || !num_tokens_post_pad || !pair_row || (p->n_rows > 0 && (!sorted_token_ids || !rows))) return MR_EINVAL;
    if (!at_multiple(x, size) || !at_multiple(rows, size) || !at_multiple(topk_idx, 4) || !at_multiple(sorted_token_ids, 4) ||
        !at_multiple(num_tokens_post_pad, 4) || !at_multiple(pair_row, 4) || !at_multiple(status, 4))
        return MR_EINVAL;
    const PermuteArgs a = {x, topk_idx, sorted_token_ids, num_tokens_post_pad, rows, pair_row, status,
                           p->T * p->topk, p->topk, p->n_rows, E_tot, 0, 0};
    const size_t bytes = size * p->H;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    auto fits = [&](size_t n) { return bytes % n == 0 && at_multiple(x, n) && at_multiple(rows, n); };
    if (fits(16)) return permute<uint4, 4>(a, bytes, st);
    return fits(4) ? permute<uint32_t, 8>(a, bytes, st) : permute<uint16_t, 8>(a, bytes, st);
}

int moe_permute_bwd(const mr_rows_params* p, const void* grad_rows, const int32_t* pair_row, void* grad_x,
                    int32_t* status, mr_stream_t stream)
{
    const int rc = check_rows(p);
    if (rc != MR_OK) return rc;
    if (p->T == 0) return MR_OK;
    const size_t size = element(p->dtype);
    if ((p->n_rows > 0 && !grad_rows) || !pair_row || !grad_x) return MR_EINVAL;
    if (!at_multiple(grad_rows, size) || !at_multiple(grad_x, size) || !at_multiple(pair_row, 4) || !at_multiple(status, 4))
        return MR_EINVAL;
    return combine_call(*p, grad_rows, pair_row, nullptr, nullptr, DropArgs{}, grad_x, status,
                        reinterpret_cast<cudaStream_t>(stream));
}

int moe_combine_fwd(const mr_rows_params* p, const void* rows, const int32_t* pair_row, const float* topk_w,
                    const void* residual, float drop_p, const void* rng, void* out, int32_t* status, mr_stream_t stream)
{
    const int rc = check_rows(p);
    if (rc != MR_OK) return rc;
    DropArgs drop;
    if (!drop_args(drop_p, rng, drop)) return MR_EINVAL;
    if (p->T == 0) return MR_OK;
    const size_t size = element(p->dtype);
    if ((p->n_rows > 0 && !rows) || !pair_row || !topk_w || !out) return MR_EINVAL;
    if (!at_multiple(rows, size) || !at_multiple(out, size) || !at_multiple(residual, size) || !at_multiple(pair_row, 4) ||
        !at_multiple(topk_w, 4) || !at_multiple(status, 4))
        return MR_EINVAL;
    return combine_call(*p, rows, pair_row, topk_w, residual, drop, out, status, reinterpret_cast<cudaStream_t>(stream));
}

int moe_combine_bwd(const mr_rows_params* p, const void* grad_out, const void* rows, const int32_t* pair_row,
                    const float* topk_w, const int32_t* sorted_token_ids, const int32_t* num_tokens_post_pad,
                    float drop_p, const void* rng, void* grad_rows, float* grad_w, int32_t* status, mr_stream_t stream)
{
    const int rc = check_rows(p);
    if (rc != MR_OK) return rc;
    DropArgs drop;
    if (!drop_args(drop_p, rng, drop)) return MR_EINVAL;
    if (p->T == 0) return MR_OK;
    const size_t size = element(p->dtype);
    if (!grad_out || !pair_row || !topk_w || !num_tokens_post_pad || !grad_w ||
        (p->n_rows > 0 && (!rows || !grad_rows || !sorted_token_ids)))
        return MR_EINVAL;
    if (!at_multiple(grad_out, size) || !at_multiple(rows, size) || !at_multiple(grad_rows, size) || !at_multiple(pair_row, 4) ||
        !at_multiple(topk_w, 4) || !at_multiple(sorted_token_ids, 4) || !at_multiple(num_tokens_post_pad, 4) ||
        !at_multiple(grad_w, 4) || !at_multiple(status, 4))
        return MR_EINVAL;
    const CombineBwdArgs a = {grad_out, rows, pair_row, topk_w, sorted_token_ids, num_tokens_post_pad, grad_rows, grad_w,
                              status, drop, p->T, p->topk, p->n_rows, p->H, 0, 0, 0};
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return p->dtype == MR_F32 ? combine_bwd_of<float>(a, st) : combine_bwd_of<__nv_bfloat16>(a, st);
}

}  // extern "C"
