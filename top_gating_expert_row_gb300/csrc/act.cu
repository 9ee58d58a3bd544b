// The gated activation of the experts' rows with expert dropout, and dropout of hidden states, with their gradients:
// moe_expert_act_fwd / bwd and moe_dropout_fwd / bwd.
//
//   h = m * act(g) * u                                    for the rows (g, u) in use; m: dropout's factors (rows.cuh)
//   d = m * grad_h:  grad_u = d act(g),  grad_g = d u act'(g);  h again where it is asked for
//   y = residual + m * x;  grad_x = m * grad_y
//   SiLU: act = g s, act' = s + g s (1 - s), s = 1 / (1 + exp -g);  GELU: act = g Phi(g), act' = Phi(g) + g phi(g)
// Bound by memory, but for what the generator and the exponentials cost in bf16.
#include <climits>

#include "rows.cuh"

namespace mr {
namespace {

__device__ __forceinline__ float rcp_hw(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// act(g) and act'(g) in fp32, for outputs of type T. The sigmoid is a hardware exponential and reciprocal. Phi(-a) =
// exp(-a^2 / 2) R(s), s = a / (4 + a): R, half the scaled complementary error function of a / sqrt 2, is smooth in s and
// is a polynomial of degree 9, fitted here by least squares that are weighted again until the errors level (Lawson's
// method), for a up to 14. Near a = 0 an error of s counts little, and behind it R's grows no faster than the
// exponential's. Phi(a) = 1 - Phi(-a).
// Errors: the exponential's argument is rounded, so they grow with it: at most (|g| + 12) 2^-24 of SiLU (tens of units of
// the last place at g = -80) and (2 g^2 + 10) 2^-24 of GELU's negative side (1e-5 at -13), relative.
// exp g and exp(-g^2 / 2) become subnormal, which the fast forms flush to 0, while act and act' are still normal numbers.
// So the exponent is moved by kShift where it matters, and the result moved back by a product: in fp32, where exponents of
// 100 and more are met (far is 0 or 1, a saturated product: exponents there are multiples of 2^-17), which gives all that
// fp32 holds; in bf16 always, in one product with log2 e, since the roundings of 2^-20 that this costs are far below
// bf16's, and g times 2^-16 is exact for bf16's subnormal numbers too. There act is 0 below 2^-135, which bf16 cannot
// hold.
// Two values at a time, in packed instructions where there are any (each half rounds as the single one does).
template <typename T, int ACT, bool GRAD>
__device__ __forceinline__ float2 gate(float2 g, float2& da)
{
    constexpr bool kShort = sizeof(T) == 2;
    auto both = [](float v) { return make_float2(v, v); };
    auto ex2 = [](float2 v) { return make_float2(exp2_hw(v.x), exp2_hw(v.y)); };
    auto rcp = [](float2 v) { return make_float2(rcp_hw(v.x), rcp_hw(v.y)); };
    constexpr float kShift = kShort ? 16.0f : 24.0f, kBack = kShort ? 0x1p-16f : 0x1p-24f;
    const float2 one = both(1.0f);
    // fp32: x log2 e, moved towards 0 by kShift where it is beyond 100, and what moves the result back
    auto exponent = [&](float2 x, float sign, float2& back) {
        const float2 y = __ffma2_rn(x, both(kLog2eHi), __fmul2_rn(x, both(kLog2eLo)));
        auto beyond = [&](float v) { return __saturatef(fmaf(v, sign * 0x1p20f, -100.0f * 0x1p20f)); };
        const float2 far = make_float2(beyond(y.x), beyond(y.y));
        back = __ffma2_rn(far, both(kBack - 1.0f), one);
        return __ffma2_rn(far, both(-sign * kShift), y);
    };
    if constexpr (ACT == MR_SILU) {
        float2 a, s;
        if constexpr (kShort) {
            const float2 r = rcp(__fadd2_rn(both(kBack), ex2(__ffma2_rn(g, both(-kLog2eHi), both(-kShift)))));
            a = __fmul2_rn(__fmul2_rn(g, both(kBack)), r);
            s = __fmul2_rn(r, both(kBack));
        } else {
            float2 back;
            const float2 r = rcp(__fadd2_rn(one, ex2(exponent(make_float2(-g.x, -g.y), 1.0f, back))));
            a = __fmul2_rn(__fmul2_rn(g, r), back);
            s = __fmul2_rn(r, back);
        }
        if constexpr (GRAD) da = __ffma2_rn(a, __fadd2_rn(one, make_float2(-s.x, -s.y)), s);
        return a;
    } else {
        constexpr float kR[] = {0.5f, -1.5957679748535156f, 2.4041967391967773f, -2.1061601638793945f, 0.8699361681938171f,
                                0.10994171351194382f, -0.2098998725414276f, -0.04766450077295303f, 0.10934294760227203f,
                                -0.03394665941596031f};
        constexpr float kScale = kShort ? kBack : 1.0f;  // of R and of the density
        const float2 q = __fmul2_rn(both(0.25f), make_float2(fminf(fabsf(g.x), 14.0f), fminf(fabsf(g.y), 14.0f)));
        const float2 s = __fmul2_rn(q, rcp(__fadd2_rn(one, q)));
        float2 e, back = one;
        if constexpr (kShort) e = ex2(__ffma2_rn(__fmul2_rn(g, g), both(-0.5f * kLog2eHi), both(kShift)));
        else e = ex2(exponent(__fmul2_rn(__fmul2_rn(both(-0.5f), g), g), -1.0f, back));
        float2 t = both(kScale * kR[9]);
#pragma unroll
        for (int i = 8; i >= 0; --i) t = __ffma2_rn(t, s, both(kScale * kR[i]));
        t = __fmul2_rn(t, e);
        if constexpr (!kShort) t = __fmul2_rn(t, back);
        const float2 cdf = make_float2(g.x > 0.0f ? 1.0f - t.x : t.x, g.y > 0.0f ? 1.0f - t.y : t.y);
        if constexpr (GRAD) {
            float2 density = __fmul2_rn(both(kScale * 0.39894228040143268f), e);
            if constexpr (!kShort) density = __fmul2_rn(density, back);
            da = __ffma2_rn(g, density, cdf);
        }
        return __fmul2_rn(g, cdf);
    }
}

struct ActArgs {
    const void* grad_h;  // backward only
    const void* gu;
    const int32_t* used;  // null: all n_rows
    void* grad_gu;        // backward only
    void* h;              // backward: nullable
    DropArgs drop;
    int n_rows, W, wc;
};

// bf16 rows at aligned widths are asked for two ahead through shared memory, which holds what registers would: 30016 of
// 32768 x 1024 with dropout 31.4 us (5.9 TB/s) against 35.7 with loads to registers, GELU 32768 x 1024 32.4 against 36.5,
// the gradient of 32000 x 2048 with dropout 121.4 (6.5 TB/s) against 123.8, of 8000 x 768 13.0 against 13.7; ahead in
// registers 37 (fewer warps). A gradient whose warps have few rows each loses by it (2000 x 1024 6.0 us against 5.5; the
// forward 3.6 against 3.8). fp32 takes twice the shared memory and is slower for it (16384 x 2048 GELU 88 us against 65,
// its gradient 82 against 64 at half the rows).
template <typename T, bool VEC, int ACT, bool DROP, bool BWD>
__global__ void __launch_bounds__(kRowsThreads) k_act(const __grid_constant__ ActArgs a)
{
    pdl_trigger_small();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int across = 1 << a.wc, tall = (kRowsThreads / 32) >> a.wc;
    const int c0 = (static_cast<int>(blockIdx.y) * across + (warp & (across - 1))) * kSpan;
    if (c0 >= a.W) return;
    const int rows = a.used ? min(__ldcg(a.used), a.n_rows) : a.n_rows;
    DropState ds;
    if constexpr (DROP) ds = drop_state(a.drop);
    const long long step = static_cast<long long>(gridDim.x) * tall;
    const long long first = static_cast<long long>(blockIdx.x) * tall + (warp >> a.wc);
    constexpr bool kAhead = VEC && sizeof(T) == 2;
    constexpr int D = 3;
    __shared__ Ring<T, BWD ? 3 : 2, kAhead ? D : 1> ring;
    int stage = 0;
    const bool mine = c0 + 8 * lane < a.W;
    auto ask = [&](long long r, int at) {
        if constexpr (kAhead) {
            if (r < rows && mine) {
                const T* gu = static_cast<const T*>(a.gu) + r * 2 * a.W + c0 + 8 * lane;
                ring.ask(at, 0, gu);
                ring.ask(at, 1, gu + a.W);
                if constexpr (BWD) ring.ask(at, 2, static_cast<const T*>(a.grad_h) + r * a.W + c0 + 8 * lane);
            }
            ring.commit();
        }
    };
    if constexpr (kAhead) {
#pragma unroll
        for (int i = 0; i < D - 1; ++i) ask(first + i * step, i);
    }
    for (long long r = first; r < rows; r += step) {
        Pack<T> pg = {}, pu = {}, pd = {};
        if constexpr (kAhead) {
            ring.wait();
            if (mine) {
                ring.take(stage, 0, pg);
                ring.take(stage, 1, pu);
                if constexpr (BWD) ring.take(stage, 2, pd);
            }
            ask(r + (D - 1) * step, stage == 0 ? D - 1 : stage - 1);
            stage = stage == D - 1 ? 0 : stage + 1;
        } else {
            const T* gu = static_cast<const T*>(a.gu) + r * 2 * a.W;
            load_span<VEC>(gu, c0, a.W, lane, pg);
            load_span<VEC>(gu + a.W, c0, a.W, lane, pu);
            if constexpr (BWD) load_span<VEC>(static_cast<const T*>(a.grad_h) + r * a.W, c0, a.W, lane, pd);
        }
        if constexpr (!BWD) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                float2 da;
                const float2 act = gate<T, ACT, false>(make_float2(pg.get(e), pg.get(e + 1)), da);
                v[e] = act.x * pu.get(e);
                v[e + 1] = act.y * pu.get(e + 1);
            }
            if constexpr (DROP) drop_span<VEC>(a.drop, ds, static_cast<uint32_t>(r), c0, lane, v);
            Pack<T> q;
            q.set(v);
            store_span<VEC>(static_cast<T*>(a.h) + r * a.W, c0, a.W, lane, q);
        } else {
            float m[8], v[8], gg[8], gq[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) m[e] = 1.0f;
            if constexpr (DROP) drop_span<VEC>(a.drop, ds, static_cast<uint32_t>(r), c0, lane, m);
#pragma unroll
            for (int e0 = 0; e0 < 8; e0 += 2) {
                float2 da2;
                const float2 act2 = gate<T, ACT, true>(make_float2(pg.get(e0), pg.get(e0 + 1)), da2);
#pragma unroll
                for (int e = e0; e < e0 + 2; ++e) {
                    const float act = e == e0 ? act2.x : act2.y, da = e == e0 ? da2.x : da2.y, u = pu.get(e);
                    // a dropped element is 0 whatever it held
                    const bool kept = !DROP || m[e] != 0.0f;
                    const float d = kept ? m[e] * pd.get(e) : 0.0f;
                    v[e] = kept ? act * u * m[e] : 0.0f;  // in the forward's order: the same bits
                    gq[e] = kept ? d * act : 0.0f;
                    gg[e] = kept ? d * u * da : 0.0f;
                }
            }
            T* grad = static_cast<T*>(a.grad_gu) + r * 2 * a.W;
            Pack<T> q;
            q.set(gg);
            store_span<VEC>(grad, c0, a.W, lane, q);
            q.set(gq);
            store_span<VEC>(grad + a.W, c0, a.W, lane, q);
            if (a.h) {
                q.set(v);
                store_span<VEC>(static_cast<T*>(a.h) + r * a.W, c0, a.W, lane, q);
            }
        }
    }
}

struct DropoutArgs {
    const void* x;
    const void* residual;  // nullable
    void* y;
    DropArgs drop;
    int T, W, wc;
};

// Without a residual a warp has one load of 512 bytes in flight beside the generator's chain of dependent products:
// what counts is the number of warps, so these kernels keep to 32 registers: bf16 takes 30 by itself (16384 x 4096: 49.4
// us, 5.4 TB/s), fp32 36 without the limit (16384 x 4096 84.3 us, 6.4 TB/s, against 85.4; 4096 x 1024 8.3 against 7.5). Two
// rows a warp or the next row's load ahead took more registers and 56 to 62 us in bf16. With a residual there are twice
// the loads a warp, and the compiler's choice stands (16384 x 2048 in bf16: 31.2 us, 6.5 TB/s).
constexpr int dropout_ctas(bool few_registers) { return few_registers ? 8 : 0; }  // 0: the compiler's choice

template <typename T, bool VEC, bool DROP, bool RES>
__global__ void __launch_bounds__(kRowsThreads, dropout_ctas(VEC && !RES)) k_dropout(const __grid_constant__ DropoutArgs a)
{
    pdl_trigger_small();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int across = 1 << a.wc, tall = (kRowsThreads / 32) >> a.wc;
    const int c0 = (static_cast<int>(blockIdx.y) * across + (warp & (across - 1))) * kSpan;
    if (c0 >= a.W) return;
    DropState ds;
    if constexpr (DROP) ds = drop_state(a.drop);
    for (long long t = static_cast<long long>(blockIdx.x) * tall + (warp >> a.wc); t < a.T;
         t += static_cast<long long>(gridDim.x) * tall) {
        Pack<T> p, q;
        load_span<VEC>(static_cast<const T*>(a.x) + t * a.W, c0, a.W, lane, p);
        if constexpr (RES) load_span<VEC>(static_cast<const T*>(a.residual) + t * a.W, c0, a.W, lane, q);
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = p.get(e);
        if constexpr (DROP) drop_span<VEC>(a.drop, ds, static_cast<uint32_t>(t), c0, lane, v);
        if constexpr (RES) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += q.get(e);
        }
        q.set(v);
        store_span<VEC>(static_cast<T*>(a.y) + t * a.W, c0, a.W, lane, q);
    }
}

// ---- host --------------------------------------------------------------------

// Launches a kernel whose warps take a row and a span at a time, in three waves (with one, with six): 32768 x 1024 GELU
// 32.2 us (35.0, 33.8), 30016 x 1024 with dropout 31.3 (32.4, 33.1), dropout 16384 x 2048 with residual 31.2 (31.6, 32.6).
// Not everywhere the best: 16384 x 1001 with dropout 30.5 (29.2, 31.4), dropout 16384 x 1280 20.2 (18.0, 29.9).
template <typename Args>
int launch_spans(void (*kernel)(Args), Args a, long long rows, cudaStream_t st)
{
    const int spans = spans_of(a.W);
    a.wc = warps_across(spans);
    const dim3 grid = span_grid(reinterpret_cast<const void*>(kernel), rows, spans, a.wc, 3);
    if (grid.x < 1) return MR_ECUDA;
    return launch_kernel(kernel, grid, dim3(kRowsThreads), 0, st, 0, a) == cudaSuccess ? MR_OK : MR_ECUDA;
}

template <typename T, int ACT, bool BWD>
int act_of(const ActArgs& a, cudaStream_t st)
{
    const size_t n = kVecBytes<T>;
    const bool vec = a.W % 8 == 0 && at_multiple(a.gu, n) && at_multiple(a.h, n) && at_multiple(a.grad_h, n) &&
                     at_multiple(a.grad_gu, n);
    if (a.drop.cut)
        return vec ? launch_spans(k_act<T, true, ACT, true, BWD>, a, a.n_rows, st)
                   : launch_spans(k_act<T, false, ACT, true, BWD>, a, a.n_rows, st);
    return vec ? launch_spans(k_act<T, true, ACT, false, BWD>, a, a.n_rows, st)
               : launch_spans(k_act<T, false, ACT, false, BWD>, a, a.n_rows, st);
}

template <bool BWD>
int act_call(const ActArgs& a, int act, int dtype, cudaStream_t st)
{
    using B = __nv_bfloat16;
    if (act == MR_SILU) return dtype == MR_F32 ? act_of<float, MR_SILU, BWD>(a, st) : act_of<B, MR_SILU, BWD>(a, st);
    return dtype == MR_F32 ? act_of<float, MR_GELU, BWD>(a, st) : act_of<B, MR_GELU, BWD>(a, st);
}

template <typename T, bool VEC>
int dropout_vec(const DropoutArgs& a, cudaStream_t st)
{
    if (a.drop.cut)
        return a.residual ? launch_spans(k_dropout<T, VEC, true, true>, a, a.T, st)
                          : launch_spans(k_dropout<T, VEC, true, false>, a, a.T, st);
    return a.residual ? launch_spans(k_dropout<T, VEC, false, true>, a, a.T, st)
                      : launch_spans(k_dropout<T, VEC, false, false>, a, a.T, st);
}

template <typename T>
int dropout_of(const DropoutArgs& a, cudaStream_t st)
{
    const size_t n = kVecBytes<T>;
    const bool vec = a.W % 8 == 0 && at_multiple(a.x, n) && at_multiple(a.residual, n) && at_multiple(a.y, n);
    return vec ? dropout_vec<T, true>(a, st) : dropout_vec<T, false>(a, st);
}

int check_act(const mr_act_params* p)
{
    if (!p || p->n_rows < 0 || p->I < 1) return MR_EINVAL;
    if (p->act != MR_SILU && p->act != MR_GELU) return MR_EINVAL;
    if (p->dtype != MR_F32 && p->dtype != MR_BF16) return MR_EINVAL;
    return p->I > MR_MAX_WIDTH ? MR_EUNSUPPORTED : MR_OK;
}

int dropout_call(int T, int H, int dtype, const void* x, const void* residual, float drop_p, const void* rng, void* y,
                 cudaStream_t st)
{
    if (T < 0 || H < 1 || (dtype != MR_F32 && dtype != MR_BF16)) return MR_EINVAL;
    if (H > MR_MAX_WIDTH) return MR_EUNSUPPORTED;
    DropArgs drop;
    if (!drop_args(drop_p, rng, drop)) return MR_EINVAL;
    if (T == 0) return MR_OK;
    const size_t size = element(dtype);
    if (!x || !y || !at_multiple(x, size) || !at_multiple(y, size) || !at_multiple(residual, size)) return MR_EINVAL;
    const DropoutArgs a = {x, residual, y, drop, T, H, 0};
    return dtype == MR_F32 ? dropout_of<float>(a, st) : dropout_of<__nv_bfloat16>(a, st);
}

}  // namespace
}  // namespace mr

using namespace mr;

extern "C" {

int moe_expert_act_fwd(const mr_act_params* p, const void* gu, const int32_t* num_rows, float drop_p, const void* rng,
                       void* h, mr_stream_t stream)
{
    const int rc = check_act(p);
    if (rc != MR_OK) return rc;
    DropArgs drop;
    if (!drop_args(drop_p, rng, drop)) return MR_EINVAL;
    if (p->n_rows == 0) return MR_OK;
    const size_t size = element(p->dtype);
    if (!gu || !h || !at_multiple(gu, size) || !at_multiple(h, size) || !at_multiple(num_rows, 4)) return MR_EINVAL;
    const ActArgs a = {nullptr, gu, num_rows, nullptr, h, drop, p->n_rows, p->I, 0};
    return act_call<false>(a, p->act, p->dtype, reinterpret_cast<cudaStream_t>(stream));
}

int moe_expert_act_bwd(const mr_act_params* p, const void* grad_h, const void* gu, const int32_t* num_rows, float drop_p,
                       const void* rng, void* grad_gu, void* h, mr_stream_t stream)
{
    const int rc = check_act(p);
    if (rc != MR_OK) return rc;
    DropArgs drop;
    if (!drop_args(drop_p, rng, drop)) return MR_EINVAL;
    if (p->n_rows == 0) return MR_OK;
    const size_t size = element(p->dtype);
    if (!grad_h || !gu || !grad_gu || !at_multiple(grad_h, size) || !at_multiple(gu, size) || !at_multiple(grad_gu, size) ||
        !at_multiple(h, size) || !at_multiple(num_rows, 4))
        return MR_EINVAL;
    const ActArgs a = {grad_h, gu, num_rows, grad_gu, h, drop, p->n_rows, p->I, 0};
    return act_call<true>(a, p->act, p->dtype, reinterpret_cast<cudaStream_t>(stream));
}

int moe_dropout_fwd(int T, int H, int dtype, const void* x, const void* residual, float drop_p, const void* rng, void* y,
                    mr_stream_t stream)
{
    return dropout_call(T, H, dtype, x, residual, drop_p, rng, y, reinterpret_cast<cudaStream_t>(stream));
}

int moe_dropout_bwd(int T, int H, int dtype, const void* grad_y, float drop_p, const void* rng, void* grad_x,
                    mr_stream_t stream)
{
    return dropout_call(T, H, dtype, grad_y, nullptr, drop_p, rng, grad_x, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
