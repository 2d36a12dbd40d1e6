// Routing from given logits: scores (softmax or sigmoid), a bias that steers the choice alone, groups of
// experts, top-k, renormalised weights; and the gradient of the logits.
//
// The choice is that of the keys in exact arithmetic wherever 64 bits tell them apart: without a bias the
// order of the scores is that of the logits, which are compared as they are; keys that are sums (a score and
// a bias, or a group's two largest) are formed in 32 bits, and a token of which two neighbouring keys lie
// nearer than their rounding can be is chosen again with keys in 64 bits (about one token in a thousand).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>

#include "kernels.cuh"

namespace moe {

namespace {

constexpr uint32_t kAll = 0xffffffffu;

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ void from_f32(float v, float& o) { o = v; }
__device__ __forceinline__ void from_f32(float v, __nv_bfloat16& o) { o = __float2bfloat16_rn(v); }
__device__ __forceinline__ void from_f32(float v, __half& o) { o = __float2half_rn(v); }

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}
__device__ __forceinline__ double warp_sum(double v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

// Keys as unsigned numbers in the same order (NaN does not occur; -0 counts as +0): 0 is below every key.
__device__ __forceinline__ uint32_t ordered(float v)
{
    const uint32_t b = __float_as_uint(v + 0.0f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ uint64_t ordered(double v)
{
    const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
    return b ^ ((uint64_t)((int64_t)b >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ float unordered(uint32_t k)
{
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(kAll, v); }
__device__ __forceinline__ uint64_t warp_max(uint64_t v)
{
    const uint32_t hi = __reduce_max_sync(kAll, (uint32_t)(v >> 32));
    const uint32_t lo = __reduce_max_sync(kAll, (uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
    return (uint64_t)hi << 32 | lo;
}

// The largest of the lanes' keys (expert 32 i + lane at key[i]) and the lowest expert that has it, taken out.
template <int PL, typename K>
__device__ __forceinline__ K take_max(K (&key)[PL], int& expert)
{
    const int lane = threadIdx.x & 31;
    K m = key[0];
    int at = 0;
#pragma unroll
    for (int i = 1; i < PL; ++i)
        if (key[i] > m) {
            m = key[i];
            at = i;
        }
    const K best = warp_max(m);
    const uint32_t e = __reduce_min_sync(kAll, m == best ? (uint32_t)(32 * at + lane) : 0xffffffffu);
#pragma unroll
    for (int i = 0; i < PL; ++i)
        if (e == (uint32_t)(32 * i + lane)) key[i] = 0;
    expert = (int)e;
    return best;
}

// Bit g: group g is among the topk_groups best; ties go to the lower group.  score: lane g's group.  `edge`
// receives the scores of the last group taken and the first left out.
template <typename F>
__device__ __forceinline__ uint32_t best_groups(F score, int groups, int take, F (&edge)[2])
{
    const int lane = threadIdx.x & 31;
    int before = 0;
    for (int g = 0; g < groups; ++g) {
        const F s = __shfl_sync(kAll, score, g);
        before += s > score || (s == score && g < lane);
    }
    const bool in = lane < groups;
    const uint32_t last = __ballot_sync(kAll, in && before == take - 1);
    const uint32_t next = __ballot_sync(kAll, in && before == take);
    edge[0] = __shfl_sync(kAll, score, __ffs(last) - 1);
    edge[1] = __shfl_sync(kAll, score, next ? __ffs(next) - 1 : 0);
    return __ballot_sync(kAll, in && before < take);
}

// Lane g < groups: the score of group g, keys [E] in shared memory: its largest, or the sum of its two
// largest (the largest alone where the second is -infinity).  32 / (groups rounded up to a power of two)
// lanes look at a group together.
template <typename F>
__device__ __forceinline__ F group_score(const F* keys, int groups, int n, bool two)
{
    const int lane = threadIdx.x & 31;
    int per = 32;
    while (per * groups > 32) per >>= 1;
    const int g = lane / per;
    F a = -(F)INFINITY, b = -(F)INFINITY;
    if (g < groups)
        for (int i = lane % per; i < n; i += per) {
            const F v = keys[g * n + i];
            if (v > a) {
                b = a;
                a = v;
            } else if (v > b) {
                b = v;
            }
        }
    for (int o = 1; o < per; o <<= 1) {
        const F c = __shfl_xor_sync(kAll, a, o), d = __shfl_xor_sync(kAll, b, o);
        b = fmax(fmin(a, c), fmax(b, d));
        a = fmax(a, c);
    }
    const F s = two && b > -(F)INFINITY ? a + b : a;
    return __shfl_sync(kAll, s, (lane * per) & 31);
}

// The choice with keys in 64 bits: expert j of lane j.  (Out of line: few tokens need it.)
template <int PL>
__device__ __noinline__ int choose_64(const RouteArgs& a, const float (&l)[PL], double* s_keys)
{
    const int lane = threadIdx.x & 31;
    double m = -INFINITY, sum = 0.0;
    if (a.score == MOE_SCORE_SOFTMAX) {
        float mf = -INFINITY;
#pragma unroll
        for (int i = 0; i < PL; ++i) mf = fmaxf(mf, l[i]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mf = fmaxf(mf, __shfl_xor_sync(kAll, mf, o));
        m = mf;
        for (int i = 0; i < PL; ++i)
            if (l[i] > -INFINITY) sum += l[i] == m ? 1.0 : exp((double)l[i] - m);
        sum = warp_sum(sum);
    }
    uint64_t key[PL];
    const int n = a.E / a.groups;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
        const int e = 32 * i + lane;
        key[i] = 0;
        if (e >= a.E) continue;
        double v = -INFINITY, own = l[i];
        if (l[i] > -INFINITY) {
            v = a.score == MOE_SCORE_SOFTMAX ? (l[i] == m ? 1.0 : exp((double)l[i] - m)) / sum : 1.0 / (1.0 + exp(-(double)l[i]));
            if (a.bias) v += (double)a.bias[e];
            if (!(v >= -DBL_MAX)) v = -INFINITY;  // a bias of -infinity or NaN
            if (a.bias) own = v;
        }
        if (a.groups > 1) s_keys[e] = v;
        key[i] = ordered(own);
    }
    if (a.groups > 1) {
        __syncwarp();
        double edge[2];
        const uint32_t in = best_groups(group_score(s_keys, a.groups, n, a.group_score == MOE_GROUP_TOP2),
                                        a.groups, a.topk_groups, edge);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            const int e = 32 * i + lane;
            if (e < a.E && !(in >> (e / n) & 1)) key[i] = 0;
        }
    }
    int mine = 0;
    for (int j = 0; j < a.k; ++j) {
        int e;
        take_max<PL>(key, e);
        if (lane == j) mine = e;
    }
    return mine;
}

}  // namespace

// A warp per token, expert 32 i + lane in the registers of a lane.
template <int PL, typename T>
__global__ void __launch_bounds__(32 * kRouteWarps) route_scores_kernel(RouteArgs a)
{
    extern __shared__ double s_all[];  // [kRouteWarps][E] keys, where there are groups
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp;
    if (t >= a.T) return;
    double* s_keys = s_all + (a.groups > 1 ? (size_t)warp * a.E : 0);
    const T* x = static_cast<const T*>(a.logits) + t * a.stride;
    float l[PL];
    const bool softmax = a.score == MOE_SCORE_SOFTMAX;
    bool nan = false;  // of this token's weights: a logit is NaN, which ranks last, or has no softmax
#pragma unroll
    for (int i = 0; i < PL; ++i) {
        const int e = 32 * i + lane;
        l[i] = e < a.E ? to_f32(x[e]) : -INFINITY;
        nan = nan || l[i] != l[i] || (softmax && l[i] == INFINITY);
        if (l[i] != l[i]) l[i] = -INFINITY;
    }
    const bool summed = a.bias || (a.groups > 1 && a.group_score == MOE_GROUP_TOP2);  // keys of sums
    float m = 0.0f, inv = 1.0f;
    if (softmax && (summed || !a.renorm)) {
        m = -INFINITY;
#pragma unroll
        for (int i = 0; i < PL; ++i) m = fmaxf(m, l[i]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
        if (m == -INFINITY) m = 0.0f;
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < PL; ++i) sum += expf(l[i] == m ? 0.0f : l[i] - m);
        sum = warp_sum(sum);
        inv = sum > 0.0f ? 1.0f / sum : 0.0f;
    }
    auto score = [&](float v) { return softmax ? expf(v == m ? 0.0f : v - m) * inv : 1.0f / (1.0f + expf(-v)); };
    uint32_t key[PL];
    const int n = a.E / a.groups;
    // How far apart two 32-bit keys are that may be in the other order: twice the rounding of a key, itself
    // within 2^-22 of a sigmoid (of the largest softmax score 2^-19: the sum's terms) and 2^-24 of the sum.
    const float slack = softmax ? inv * 0x1p-17f : 0x1p-20f;
    auto near = [&](float hi, float lo) {
        return hi - lo <= slack + 0x1p-22f * fminf(fmaxf(fabsf(hi), fabsf(lo)), FLT_MAX);
    };
    bool again = false;
    float* keys32 = reinterpret_cast<float*>(s_keys);
    const bool sums = a.groups > 1 && a.group_score == MOE_GROUP_TOP2;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
        const int e = 32 * i + lane;
        key[i] = 0;
        if (e >= a.E) continue;
        float v = l[i], s = v;  // the expert's key, and what its group's score is made of
        if (summed && v > -INFINITY) {
            s = score(v);
            if (a.bias) {
                s += a.bias[e];
                if (!(s >= -FLT_MAX)) s = -INFINITY;  // a bias of -infinity or NaN
                v = s;
            }
        }
        if (a.groups > 1) keys32[e] = sums ? s : v;
        key[i] = ordered(v);
    }
    if (a.groups > 1) {
        __syncwarp();
        float edge[2];
        const uint32_t in = best_groups(group_score(keys32, a.groups, n, sums), a.groups, a.topk_groups, edge);
        __syncwarp();
        // (a group's score is two keys)
        if (summed && a.topk_groups < a.groups) again = near(0.25f * edge[0], 0.25f * edge[1]);
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            const int e = 32 * i + lane;
            if (e < a.E && !(in >> (e / n) & 1)) key[i] = 0;
        }
    }
    int mine = 0;
    if (!again) {
        // lane j: the key and expert taken j-th; one more than k where the order of sums may need 64 bits
        const int rounds = a.bias && a.k < a.E ? a.k + 1 : a.k;
        uint32_t kept = 0, k = 0;
        int e = 0;
        for (int j = 0; j < rounds; ++j) {
            k = take_max<PL>(key, e);
            if (lane == j) {
                mine = e;
                kept = k;
            }
        }
        if (a.bias) {
            uint32_t next = __shfl_down_sync(kAll, kept, 1);
            int after = __shfl_down_sync(kAll, mine, 1);
            if (lane == 31) {  // (of 32 taken, the 33rd)
                next = rounds == 33 ? k : 0u;
                after = e;
            }
            // (the sums of equal terms are equal)
            bool apart = lane >= rounds - 1 || !next || !near(unordered(kept), unordered(next));
            apart = apart || (to_f32(x[mine]) == to_f32(x[after]) && a.bias[mine] == a.bias[after]);
            again = !__all_sync(kAll, apart);
        }
    }
    if (again) mine = choose_64<PL>(a, l, s_keys);
    // lane j < k: the chosen expert's logit and weight
    const bool chosen = lane < a.k;
    float v = chosen ? to_f32(x[mine]) : -INFINITY, w;
    if (v != v) v = -INFINITY;
    if (!a.renorm) {
        w = v > -INFINITY ? score(v) : 0.0f;
    } else {
        // of softmax scores the same factor falls out; sigmoids of very negative logits are taken relative
        // to the largest: 1 / (1 + e^-l) = e^l / (1 + e^l)
        float top = v;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
        if (top == -INFINITY) top = 0.0f;
        if (softmax) w = expf(v - top);
        else if (top < 0.0f) w = expf(v - top) / (1.0f + expf(v));
        else w = 1.0f / (1.0f + expf(-v));
        if (!chosen) w = 0.0f;
        const float sum = warp_sum(w);
        w = sum > 0.0f ? w / sum : sum;  // (no expert left: 0)
    }
    if (__any_sync(kAll, nan)) w = NAN;
    if (chosen) {
        a.ids[t * a.k + lane] = mine;
        a.w[t * a.k + lane] = w * a.scale;
    }
}

// A warp per token.  Scores of their own and renormalised ones: the chosen experts' logits alone have
// gradients, q (g - r) f with g_j = scale dw_j, q the weight / scale, r = sum_i g_i q_i, f the score's own
// derivative over it (softmax 1, sigmoid 1 - s); not renormalised sigmoids g s (1 - s).  Softmax scores that
// are not renormalised: p_e (sum of the g_j of expert e - sum_j g_j p_j), for every expert e.
template <typename T>
__global__ void __launch_bounds__(32 * kRouteWarps) route_back_kernel(RouteBackArgs a)
{
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp;
    if (t >= a.T) return;
    const T* x = static_cast<const T*>(a.logits) + t * a.stride;
    T* dx = static_cast<T*>(a.dlogits) + t * a.dstride;
    const bool softmax = a.score == MOE_SCORE_SOFTMAX;
    int id = lane < a.k ? a.ids[t * a.k + lane] : -1;
    if (id >= a.E) id = -1;  // (an id out of range has no gradient)
    const bool chosen = id >= 0;
    const float v = chosen ? to_f32(x[id]) : -INFINITY;
    float g = chosen ? a.dw[t * a.k + lane] * a.scale : 0.0f;
    float d = 0.0f;
    if (softmax && !a.renorm) {
        float m = -INFINITY, sum = 0.0f;
        for (int e = lane; e < a.E; e += 32) m = fmaxf(m, to_f32(x[e]));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
        if (m == -INFINITY) m = 0.0f;
        for (int e = lane; e < a.E; e += 32) sum += expf(to_f32(x[e]) - m);
        sum = warp_sum(sum);
        const float inv = sum > 0.0f ? 1.0f / sum : sum;
        const float p = chosen ? expf(v - m) * inv : 0.0f;
        const float r = warp_sum(chosen ? g * p : 0.0f);
        for (int e = lane; e < a.E; e += 32) from_f32(-expf(to_f32(x[e]) - m) * inv * r, dx[e]);
        float all = 0.0f;  // of the positions that chose the same expert
        for (int j = 0; j < a.k; ++j) {
            const int other = __shfl_sync(kAll, id, j);
            const float gj = __shfl_sync(kAll, g, j);
            if (other == id) all += gj;
        }
        d = p * (all - r);
    } else {
        for (int e = lane; e < a.E; e += 32) from_f32(0.0f, dx[e]);
        if (a.renorm) {
            float top = v;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
            if (top == -INFINITY) top = 0.0f;
            float q, f = 1.0f;
            if (softmax) {
                q = expf(v - top);
            } else {
                q = top < 0.0f ? expf(v - top) / (1.0f + expf(v)) : 1.0f / (1.0f + expf(-v));
                f = 1.0f / (1.0f + expf(v));
            }
            if (!chosen) q = 0.0f;
            const float sum = warp_sum(q);
            q = sum > 0.0f ? q / sum : sum;
            const float r = warp_sum(chosen ? g * q : 0.0f);
            g = chosen ? q * (g - r) * f : 0.0f;
        } else {
            const float s = 1.0f / (1.0f + expf(-v));
            g = chosen ? g * s / (1.0f + expf(v)) : 0.0f;
        }
        for (int j = 0; j < a.k; ++j) {
            const int other = __shfl_sync(kAll, id, j);
            const float gj = __shfl_sync(kAll, g, j);
            if (other == id) d += gj;
        }
    }
    __syncwarp();  // the row is written; its chosen experts' are written again
    if (chosen) from_f32(d, dx[id]);
}

template <typename T>
static RouteKernel route_of(int E)
{
    return E <= 64 ? route_scores_kernel<2, T> : E <= 128 ? route_scores_kernel<4, T>
         : E <= 256 ? route_scores_kernel<8, T> : E <= 384 ? route_scores_kernel<12, T>
         : E <= 512 ? route_scores_kernel<16, T> : route_scores_kernel<32, T>;
}

RouteKernel route_scores_kernel_for(int dtype, int E)
{
    switch (dtype) {
        case MOE_BF16: return route_of<__nv_bfloat16>(E);
        case MOE_FP16: return route_of<__half>(E);
        default: return route_of<float>(E);
    }
}

RouteBackKernel route_back_kernel_for(int dtype)
{
    switch (dtype) {
        case MOE_BF16: return route_back_kernel<__nv_bfloat16>;
        case MOE_FP16: return route_back_kernel<__half>;
        default: return route_back_kernel<float>;
    }
}

}  // namespace moe
