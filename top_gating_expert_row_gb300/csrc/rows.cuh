// Building blocks of the row-wise steps around the experts' products (rows.cu, act.cu): a warp works on a span of
// 256 columns of one row, eight to a lane.
#pragma once

#include <algorithm>
#include <type_traits>

#include <cuda_bf16.h>

#include "internal.h"
#include "moe_router.h"

namespace mr {

constexpr int kSpan = 256;          // columns a warp takes at a time
constexpr int kRowsThreads = 256;   // 8 warps

inline int spans_of(int width) { return (width + kSpan - 1) / kSpan; }

// Eight elements as they lie in memory. With VEC the lane holds columns c0 + 8 lane + i of the span, in one load of
// 16 (bf16) or 32 bytes (fp32); rows at other alignments are read and written an element at a time, neighbouring
// lanes side by side: column c0 + 32 i + lane.
template <typename T>
struct Pack;
template <>
struct Pack<__nv_bfloat16> {
    uint32_t w[4];
    __device__ __forceinline__ float get(int i) const
    {
        return (i & 1) ? __uint_as_float(w[i >> 1] & 0xffff0000u) : __uint_as_float(w[i >> 1] << 16);
    }
    __device__ __forceinline__ void set(const float (&v)[8])
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&p);
        }
    }
};
template <>
struct Pack<float> {
    uint32_t w[8];
    __device__ __forceinline__ float get(int i) const { return __uint_as_float(w[i]); }
    __device__ __forceinline__ void set(const float (&v)[8])
    {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[i]);
    }
};

// The alignment that VEC asks of a base and of a row's bytes.
template <typename T>
constexpr int kVecBytes = 8 * sizeof(T);

template <bool VEC>
__device__ __forceinline__ int span_column(int c0, int lane, int i)
{
    return VEC ? c0 + 8 * lane + i : c0 + 32 * i + lane;
}

__device__ __forceinline__ void load_vec(const __nv_bfloat16* p, Pack<__nv_bfloat16>& q, bool once)
{
    const uint4 v = once ? __ldcs(reinterpret_cast<const uint4*>(p)) : *reinterpret_cast<const uint4*>(p);
    q.w[0] = v.x; q.w[1] = v.y; q.w[2] = v.z; q.w[3] = v.w;
}
__device__ __forceinline__ void load_vec(const float* p, Pack<float>& q, bool once)
{
    (void)once;
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(q.w[0]), "=r"(q.w[1]), "=r"(q.w[2]), "=r"(q.w[3]), "=r"(q.w[4]), "=r"(q.w[5]), "=r"(q.w[6]),
                   "=r"(q.w[7])
                 : "l"(p)
                 : "memory");
}
__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const Pack<__nv_bfloat16>& q)
{
    *reinterpret_cast<uint4*>(p) = make_uint4(q.w[0], q.w[1], q.w[2], q.w[3]);
}
__device__ __forceinline__ void store_vec(float* p, const Pack<float>& q)
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 :
                 : "l"(p), "r"(q.w[0]), "r"(q.w[1]), "r"(q.w[2]), "r"(q.w[3]), "r"(q.w[4]), "r"(q.w[5]), "r"(q.w[6]),
                   "r"(q.w[7])
                 : "memory");
}

// The lane's eight elements of the span at column c0 of a row of W; zeros past its end. once: read by this warp
// alone (evicted first). BRANCH: whole spans of unaligned rows without comparisons, at offsets that the loads hold
// themselves; a kernel that asks for several spans in a row does without, the branches would hold its loads up.
template <bool VEC, bool BRANCH = true, typename T>
__device__ __forceinline__ void load_span(const T* row, int c0, int W, int lane, Pack<T>& q, bool once = true)
{
    if constexpr (VEC) {
        if (c0 + 8 * lane < W) {
            load_vec(row + c0 + 8 * lane, q, once);
        } else {
#pragma unroll
            for (int i = 0; i < static_cast<int>(sizeof(q.w) / 4); ++i) q.w[i] = 0u;
        }
    } else {
        using E = std::conditional_t<sizeof(T) == 4, uint32_t, unsigned short>;
        const E* p = reinterpret_cast<const E*>(row) + c0 + lane;
        uint32_t b[8];
        if (BRANCH && c0 + kSpan <= W) {
#pragma unroll
            for (int i = 0; i < 8; ++i) b[i] = once ? __ldcs(p + 32 * i) : p[32 * i];
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) b[i] = c0 + 32 * i + lane < W ? (once ? __ldcs(p + 32 * i) : p[32 * i]) : 0u;
        }
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 8; ++i) q.w[i] = b[i];
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) q.w[i] = b[2 * i] | b[2 * i + 1] << 16;
        }
    }
}

// Aligned rows through shared memory: a thread asks for its eight elements of rows ahead without holding registers for
// them, and takes them up itself (so no barrier). N tensors, D rows; at most D - 1 of them are on their way, so that a
// place is asked for again one row after it was read.
template <typename T, int N, int D>
struct Ring {
    static constexpr int kWords = sizeof(T) / 2;  // of 16 bytes
    uint4 place[D][N * kWords][kRowsThreads];

    __device__ __forceinline__ void ask(int stage, int tensor, const T* p)
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(&place[stage][tensor * kWords + i][threadIdx.x]));
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(p + i * (8 / kWords)) : "memory");
        }
    }
    __device__ __forceinline__ static void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
    // the oldest of D - 1 rows asked for has arrived
    __device__ __forceinline__ static void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(D - 2) : "memory"); }
    __device__ __forceinline__ void take(int stage, int tensor, Pack<T>& q) const
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            const uint4 v = place[stage][tensor * kWords + i][threadIdx.x];
            q.w[4 * i] = v.x; q.w[4 * i + 1] = v.y; q.w[4 * i + 2] = v.z; q.w[4 * i + 3] = v.w;
        }
    }
};

template <bool VEC, typename T>
__device__ __forceinline__ void store_span(T* row, int c0, int W, int lane, const Pack<T>& q)
{
    if constexpr (VEC) {
        if (c0 + 8 * lane < W) store_vec(row + c0 + 8 * lane, q);
    } else {
        using E = std::conditional_t<sizeof(T) == 4, uint32_t, unsigned short>;
        E* p = reinterpret_cast<E*>(row) + c0 + lane;
        auto value = [&](int i) {
            if constexpr (sizeof(T) == 4) return q.w[i];
            else return static_cast<E>(q.w[i >> 1] >> (16 * (i & 1)));
        };
        if (c0 + kSpan <= W) {
#pragma unroll
            for (int i = 0; i < 8; ++i) p[32 * i] = value(i);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c0 + 32 * i + lane < W) p[32 * i] = value(i);
        }
    }
}

// ---------------------------------------------------------------------------
// Dropout. Element (row, column) is kept iff its 16 random bits are at least `cut` (p * 2^16, rounded), and then
// scaled by 2^16 / (2^16 - cut), so that the expectation is exact for the p that is used. The bits are those of
// Philox 4x32 with ten rounds (J. Salmon et al., "Parallel random numbers: as easy as 1, 2, 3", SC 2011): the key is
// the seed, the counter (column / 8, row, offset), element i of a block of eight takes 16 bits of word i / 2, the low
// ones first. Every row starts a block of its own, so the mask depends on nothing but these, whatever the kernel, and
// a backward pass computes it again instead of reading it. 16 bits rather than 32 halve the generator's work, which
// is what a bf16 element's 4 bytes of traffic leave room for (about 20 instructions at this GPU's rates).
// ---------------------------------------------------------------------------
struct DropArgs {
    const unsigned long long* rng;  // {seed, offset}
    uint32_t cut;                   // 1..65536 (0: nothing is dropped, and the kernels without dropout run)
    uint32_t above;                 // cut * 2^16 - 1: 16 bits on top of a word keep their element iff the word is above
    float scale;                    // 0 where nothing is kept
};

struct DropState {
    uint32_t k0, k1, o0, o1;
};

__device__ __forceinline__ DropState drop_state(const DropArgs& d)
{
    const unsigned long long seed = __ldcg(d.rng), offset = __ldcg(d.rng + 1);
    return {static_cast<uint32_t>(seed), static_cast<uint32_t>(seed >> 32), static_cast<uint32_t>(offset),
            static_cast<uint32_t>(offset >> 32)};
}

__device__ __forceinline__ uint4 philox(const DropState& s, uint32_t block, uint32_t row)
{
    uint32_t a = block, b = row, c = s.o0, d = s.o1, k0 = s.k0, k1 = s.k1;
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const unsigned long long x = 0xD2511F53ull * a, y = 0xCD9E8D57ull * c;
        a = static_cast<uint32_t>(y >> 32) ^ b ^ k0;
        b = static_cast<uint32_t>(y);
        c = static_cast<uint32_t>(x >> 32) ^ d ^ k1;
        d = static_cast<uint32_t>(x);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return make_uint4(a, b, c, d);
}

// Ones in the places of a pack whose elements are kept, zeros in the others.
template <typename T>
struct Keep {
    uint32_t w[2 * sizeof(T)];
    __device__ __forceinline__ void set(int i, bool kept)
    {
        if constexpr (sizeof(T) == 4) w[i] = kept ? 0xffffffffu : 0u;
        else if (i & 1) w[i >> 1] |= kept ? 0xffff0000u : 0u;
        else w[i >> 1] = kept ? 0x0000ffffu : 0u;
    }
    __device__ __forceinline__ void apply(Pack<T>& p) const
    {
#pragma unroll
        for (int i = 0; i < static_cast<int>(2 * sizeof(T)); ++i) p.w[i] &= w[i];
    }
};
struct NoKeep {
    __device__ __forceinline__ void set(int, bool) {}
};

// v[i] times its factor, for the lane's elements of the span at column c0 of `row`; a dropped element is 0 whatever it
// held. All 32 lanes take part. keep: which are kept, for what else meets them.
template <bool VEC, typename K = NoKeep>
__device__ __forceinline__ void drop_span(const DropArgs& d, const DropState& s, uint32_t row, int c0, int lane,
                                          float (&v)[8], K&& keep = {})
{
    const uint4 r = philox(s, static_cast<uint32_t>(c0 / 8 + lane), row);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool kept = ((i & 1) ? w[i >> 1] : w[i >> 1] << 16) > d.above;
            v[i] = kept ? v[i] * d.scale : 0.0f;
            keep.set(i, kept);
        }
    } else {
        // lane l made block c0 / 8 + l: its eight bits go to the lanes that hold these columns
        uint32_t bits = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) bits |= (((i & 1) ? w[i >> 1] : w[i >> 1] << 16) > d.above ? 1u : 0u) << i;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t k = __shfl_sync(kFull, bits, 4 * i + (lane >> 3));
            const bool kept = (k >> (lane & 7)) & 1u;
            v[i] = kept ? v[i] * d.scale : 0.0f;
            keep.set(i, kept);
        }
    }
}

// The factor of one element.
__device__ __forceinline__ float drop_factor(const DropArgs& d, const DropState& s, uint32_t row, int column)
{
    const uint4 r = philox(s, static_cast<uint32_t>(column / 8), row);
    const int i = column & 7;
    const uint32_t w = i < 4 ? (i < 2 ? r.x : r.y) : (i < 6 ? r.z : r.w);
    return ((i & 1) ? w : w << 16) > d.above ? d.scale : 0.0f;
}

// How a CTA's 8 warps are laid over (rows, spans): 2^wc spans side by side, the rest on further rows. As many spans
// as leave at most an eighth of the warps without work.
inline int warps_across(int spans)
{
    for (int wc = 3; wc > 0; --wc) {
        const int n = 1 << wc, padded = (spans + n - 1) / n * n;
        if ((padded - spans) * 8 <= padded) return wc;
    }
    return 0;
}

// CTAs for `units` of work. waves 0: no more than are resident, each with the same number of units in turn. Otherwise,
// where there are units for it, `waves` times as many as are resident, handed out as others end, so that SMs that memory
// serves faster take more (whole waves: a few CTAs behind the last would have the GPU to themselves, which cost up to a
// quarter of the time). A CTA's start costs too: which is better differs from kernel to kernel, as measured there. -1 on
// an error.
inline long long dynamic_grid(const void* kernel, long long units, int waves)
{
    const long long resident = persistent_grid(kernel, kRowsThreads, 0, units, false);
    if (resident < 1) return -1;
    if (units < 1) return 1;
    if (waves > 0 && units >= resident * waves) return resident * waves;
    const long long each = (units + resident - 1) / resident;
    return (units + each - 1) / each;
}

// A grid of (row groups, span groups) for CTAs that take 2^wc spans of 8 >> wc rows at a time; x is 0 on an error. Waves
// are rounded up to whole row groups: where y does not divide the resident CTAs the few behind the last wave cost nothing
// that could be measured (16384 x 1280, five spans: 20.2 us, 20.1 rounded down).
inline dim3 span_grid(const void* kernel, long long rows, int spans, int wc, int waves)
{
    const int tall = (kRowsThreads / 32) >> wc;
    const unsigned y = static_cast<unsigned>((spans + (1 << wc) - 1) >> wc);
    const long long need = rows > tall ? (rows + tall - 1) / tall : 1;
    const long long g = dynamic_grid(kernel, need * y, waves);
    if (g < 1) return dim3(0);
    return dim3(static_cast<unsigned>(std::min((g + y - 1) / y, need)), y);
}

// Host side of dropout's arguments: p in [0, 1] and, where it drops anything, the generator's state. False if either
// is not valid; cut 0: nothing is dropped.
inline bool drop_args(float p, const void* rng, DropArgs& d)
{
    if (!(p >= 0.0f && p <= 1.0f)) return false;
    d.cut = static_cast<uint32_t>(static_cast<double>(p) * 65536.0 + 0.5);
    d.above = (d.cut << 16) - 1u;  // nothing is above where cut is 2^16
    d.scale = d.cut < 65536u ? static_cast<float>(65536.0 / (65536.0 - d.cut)) : 0.0f;
    d.rng = static_cast<const unsigned long long*>(rng);
    return d.cut == 0 || (rng && (reinterpret_cast<uintptr_t>(rng) & 7) == 0);
}

inline size_t element(int dtype) { return dtype == MR_F32 ? 4 : 2; }
inline bool at_multiple(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

}  // namespace mr
