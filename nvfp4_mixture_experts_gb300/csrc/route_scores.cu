// Routing from given logits: scores (softmax or sigmoid), a bias that steers the choice alone, groups of
// experts, top-k, renormalised weights; and the gradient of the logits.
//
// The choice is that of the keys in exact arithmetic wherever 64 bits tell them apart: without a bias the
// order of the scores is that of the logits, which are compared as they are; keys that are sums (a score and
// a bias, or a group's two largest) are formed in 32 bits, and a token of which two neighbouring keys lie
// nearer than their rounding can be is chosen again with keys in 64 bits (about one token in a thousand): of
// the chosen experts where the next one is apart, else of the candidates for the choice, or of the largest
// keys of the groups at the border, a lane each, because 64-bit exponentials take microseconds (all keys of
// such a token: 43 us where 8192 tokens took 18).
//
// A warp has a token, so that a row is read once, in its lanes' registers, and nothing waits for other warps.
// What bounds it is the work on each token (800 instructions for top-8 of 320 logits, 1380 with sigmoids, a
// bias and eight groups), not the row's 1280 bytes: 8192 tokens top-8 of 320 9.4 us, with sigmoids, a bias and
// groups 16.0, of which the few tokens with 64-bit keys are 1.5; with softmax scores 18, of which they are 3
// (23 with all of such a token's exponentials in 64 bits, which are now for what 32-bit ones do not settle); one
// token 3.3 us.  The gradient is bound by its launch and memory: 4.4 us, 21 MB (where one score is nearly all 6.2);
// renormalised 5.2.
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

// The lanes' numbers sorted, the largest in lane 0 (a bitonic network).
__device__ __forceinline__ uint32_t warp_sort(uint32_t x)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
        for (int j = k >> 1; j; j >>= 1) {
            const uint32_t y = __shfl_xor_sync(kAll, x, j);
            const bool larger = ((lane & j) == 0) == ((lane & k) == 0);
            x = larger ? max(x, y) : min(x, y);
        }
    return x;
}

// The `rounds` largest keys (at 32 i + lane in key[i]; 0: none) in order, equal ones by position: that of lane
// j in `kept` and its position in `mine`.  Keys as large as the rounds-th largest of the lanes' maxima are the
// only ones that can be among them: mostly few, which are put together with their positions and ranked by
// counting, a lane each (8192 tokens of 320 experts, top-8: 567 instructions a token with the bound found and
// the keys put together in votes, 10.6 us).  More than 32, as of equal logits: in rounds over all keys.
template <int PL>
__device__ __forceinline__ void choose_32(const uint32_t (&key)[PL], int rounds, uint64_t* s_key, uint32_t& kept,
                                          int& mine)
{
    const int lane = threadIdx.x & 31;
    uint32_t x = key[0];
#pragma unroll
    for (int i = 1; i < PL; ++i) x = max(x, key[i]);
    const uint32_t bound = rounds > 32 ? 1u : max(__shfl_sync(kAll, warp_sort(x), rounds - 1), 1u);
    int own = 0;
#pragma unroll
    for (int i = 0; i < PL; ++i) own += key[i] >= bound;
    int n = own;   // of this lane and those before it
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kAll, n, o);
        if (lane >= o) n += y;
    }
    int at = n - own;
    n = __shfl_sync(kAll, n, 31);
    kept = 0;
    mine = 0;
    if (n <= 32) {
        // key and, of equal keys the larger for the lower position, its complement; an even number of them
        s_key[lane] = 0;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < PL; ++i)
            if (key[i] >= bound) s_key[at++] = (uint64_t)key[i] << 32 | ~(uint32_t)(32 * i + lane);
        __syncwarp();
        const uint64_t k = s_key[lane];
        int rank = 0;
        for (int j = 0; j < n; j += 2) {
            const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(s_key + j);
            rank += o.x > k;
            rank += o.y > k;
        }
        __syncwarp();
        if (lane < n) s_key[rank] = k;
        __syncwarp();
        if (lane < min(n, rounds)) {
            const uint64_t r = s_key[lane];
            kept = (uint32_t)(r >> 32);
            mine = (int)~(uint32_t)r;
        }
        return;
    }
    uint32_t left[PL];
#pragma unroll
    for (int i = 0; i < PL; ++i) left[i] = key[i];
    for (int j = 0; j < min(rounds, 32); ++j) {
        int e;
        const uint32_t k = take_max<PL>(left, e);
        if (lane == j) {
            kept = k;
            mine = e;
        }
    }
}

__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ float smaller(float a, float b) { return fminf(a, b); }
__device__ __forceinline__ double larger(double a, double b) { return a > b ? a : b; }
__device__ __forceinline__ double smaller(double a, double b) { return a < b ? a : b; }

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
// lanes look at a group together.  least: the smaller of the two keys, or the largest where the score is of one.
template <typename F>
__device__ __forceinline__ F group_score(const F* keys, int groups, int n, bool two, F* least = nullptr)
{
    const int lane = threadIdx.x & 31;
    int per = 32;
    while (per * groups > 32) per >>= 1;
    const int g = lane / per;
    F a = -(F)INFINITY, b = -(F)INFINITY;
    if (g < groups)
#pragma unroll 4
        for (int i = lane % per; i < n; i += per) {
            const F v = keys[g * n + i];
            b = larger(b, smaller(a, v));
            a = larger(a, v);
        }
    for (int o = 1; o < per; o <<= 1) {
        const F c = __shfl_xor_sync(kAll, a, o), d = __shfl_xor_sync(kAll, b, o);
        b = larger(smaller(a, c), larger(b, d));
        a = larger(a, c);
    }
    const bool sum = two && b > -(F)INFINITY;
    const F s = sum ? a + b : a;
    if (least) *least = __shfl_sync(kAll, sum ? b : a, (lane * per) & 31);
    return __shfl_sync(kAll, s, (lane * per) & 31);
}

// A token's scores in 64 bits.  (What follows is out of line and reads the logits again: few tokens need it.)
// `quick`: a softmax's sum is one of 32-bit exponentials, added in 64 bits.  Each term is within 2^-22 + 2^-24
// of itself (expf by two units at most; what the rounding of l - m left out is multiplied back in, which is
// rounded once), so the scores are all off by one factor, within 2^-21 of 1.
template <typename T>
struct Scores64 {
    const RouteArgs& a;
    const T* x;
    double m, sum, off;
    __device__ __forceinline__ float logit(int e) const
    {
        const float l = to_f32(x[e]);
        return l != l ? -INFINITY : l;
    }
    __device__ Scores64(const RouteArgs& a, const T* x, bool quick) : a(a), x(x), m(0.0), sum(1.0), off(0.0)
    {
        if (a.score != MOE_SCORE_SOFTMAX) return;
        const int lane = threadIdx.x & 31;
        float top = -INFINITY;
        for (int e = lane; e < a.E; e += 32) top = fmaxf(top, logit(e));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
        m = top;
        sum = 0.0;
        if (quick && fabsf(top) <= FLT_MAX) {
            off = 0x1p-21;
            for (int e = lane; e < a.E; e += 32) {
                const float l = logit(e), d = l - top;
                if (!(d >= -FLT_MAX)) continue;   // (e^d is 0 in 64 bits, too)
                // l - top is d + rest (two numbers' difference and what its rounding left out: Knuth's)
                const float back = d + top, rest = (l - back) + ((back - d) - top);
                const float p = expf(d);
                sum += (double)fmaf(p, rest, p);
            }
            sum = warp_sum(sum);
            return;
        }
        double part[4] = {};   // (four exponentials at a time: 64-bit instructions take long)
        for (int e0 = lane; e0 < a.E; e0 += 128)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float l = e0 + 32 * q < a.E ? logit(e0 + 32 * q) : -INFINITY;
                part[q] += l == -INFINITY ? 0.0 : l == m ? 1.0 : exp((double)l - m);
            }
        sum = warp_sum((part[0] + part[1]) + (part[2] + part[3]));
    }
    // the key of a sum: score (of which `score` receives what may be off) and bias
    __device__ double key(int e, double& score) const
    {
        score = 0.0;
        const float l = logit(e);
        if (l == -INFINITY) return -INFINITY;
        score = a.score == MOE_SCORE_SOFTMAX ? (l == m ? 1.0 : exp((double)l - m)) / sum
                                             : 1.0 / (1.0 + exp(-(double)l));
        const double v = a.bias ? score + (double)a.bias[e] : score;
        return v >= -DBL_MAX ? v : -INFINITY;  // a bias of -infinity or NaN
    }
};

// The choice with all keys in 64 bits: expert j of lane j.
template <int PL, typename T>
__device__ __noinline__ int choose_64(const RouteArgs& a, const T* x, double* s_keys)
{
    const int lane = threadIdx.x & 31;
    const Scores64<T> sc(a, x, false);
    uint64_t key[PL];
    for (int i = 0; i < PL; ++i) {
        const int e = 32 * i + lane;
        key[i] = 0;
        if (e >= a.E) continue;
        double score;
        const double v = sc.key(e, score);
        if (a.groups > 1) s_keys[e] = v;
        key[i] = ordered(a.bias ? v : (double)sc.logit(e));
    }
    if (a.groups > 1) {
        __syncwarp();
        double edge[2];
        const uint32_t in = best_groups(group_score(s_keys, a.groups, a.E / a.groups, a.group_score == MOE_GROUP_TOP2),
                                        a.groups, a.topk_groups, edge);
        __syncwarp();
        for (int i = 0; i < PL; ++i) {
            const int e = 32 * i + lane;
            if (e < a.E && !(in >> (e * a.group_mul >> 20 & 31) & 1)) key[i] = 0;
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

// The kept groups where scores lie nearer to the border than 32-bit keys can tell: lane g's group has the
// score `score`, made of keys of at least `least`, and its keys are keys[g n ..]; edge: the border's scores;
// near: whether two keys may be in the other order.  Groups well above the border are in; those near it have
// their few largest keys, four at most, taken in 64 bits, a lane each.  False: more keys than that are near
// one another.
template <typename T, typename Near>
__device__ __noinline__ bool border_groups(const RouteArgs& a, const T* x, const float* keys, float score,
                                           float least, const float (&edge)[2], Near near, int* s_expert,
                                           uint32_t& in)
{
    const int lane = threadIdx.x & 31, n = a.group;
    const bool two = a.group_score == MOE_GROUP_TOP2;
    const bool mine = lane < a.groups;
    // (a group's score is two keys; the border's two scores are near each other)
    auto by = [&](float hi, float lo) { return near(0.125f * hi, 0.125f * lo); };
    const bool border = mine && (by(fmaxf(score, edge[0]), fminf(score, edge[0])) ||
                                 by(fmaxf(score, edge[1]), fminf(score, edge[1])));
    const uint32_t borders = __ballot_sync(kAll, border);
    const uint32_t above = __ballot_sync(kAll, mine && !border && score > edge[0]);
    if (__popc(borders) > 8) return false;
    // candidate i of the r-th group at the border in s_expert[4 r + i], where there is one
    int e = -1, r = 0;   // lane 4 r + i: that candidate
    s_expert[lane] = -1;
    __syncwarp();
    for (uint32_t left = borders; left; left &= left - 1, ++r) {
        const int g = __ffs(left) - 1;
        const float low = __shfl_sync(kAll, least, g);
        int count = 0;
        for (int i0 = 0; i0 < n; i0 += 32) {
            const float k = i0 + lane < n ? keys[g * n + i0 + lane] : -INFINITY;
            const bool is = k > -INFINITY && (k >= low || near(low, k));
            const uint32_t mask = __ballot_sync(kAll, is);
            const int at = count + __popc(mask & ((1u << lane) - 1));
            if (is && at < 4) s_expert[4 * r + at] = g * n + i0 + lane;
            count += __popc(mask);
        }
        if (count > 4) return false;
    }
    __syncwarp();
    e = s_expert[lane];
    for (bool quick = a.score == MOE_SCORE_SOFTMAX;; quick = false) {
        const Scores64<T> sc(a, x, quick);
        double score;
        const double v = e >= 0 ? sc.key(e, score) : -INFINITY;
        if (e < 0) score = 0.0;
        const int rank = __popc(borders & ((1u << lane) - 1));
        double p = -INFINITY, q = -INFINITY, most = 0.0;   // most: of the candidates' scores
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const double c = __shfl_sync(kAll, v, (4 * rank + i) & 31);
            most = larger(most, __shfl_sync(kAll, score, (4 * rank + i) & 31));
            q = larger(q, smaller(p, c));
            p = larger(p, c);
        }
        const double exact = two && q > -INFINITY ? p + q : p;
        // a group's score is off by what two of its keys are (and 2^-50 of rounding), the border's order known
        // where the scores are further apart
        const double mine_off = 2.0 * sc.off * most + 0x1p-50 * fabs(exact);
        bool known = true;
        int before = __popc(above);
        for (uint32_t left = borders; left; left &= left - 1) {
            const int g = __ffs(left) - 1;
            const double o = __shfl_sync(kAll, exact, g), off = __shfl_sync(kAll, mine_off, g);
            before += o > exact || (o == exact && g < lane);
            known = known && (g == lane || fabs(o - exact) > off + mine_off);
        }
        if (quick && !__all_sync(kAll, known || !border)) continue;
        in = above | __ballot_sync(kAll, border && before < a.topk_groups);
        return true;
    }
}

// The order of n candidates, one a lane, by their keys in 64 bits: expert j of lane j.
template <typename T>
__device__ __noinline__ int order_64(const RouteArgs& a, const T* x, int mine, int n)
{
    const int lane = threadIdx.x & 31;
    for (bool quick = a.score == MOE_SCORE_SOFTMAX;; quick = false) {
        const Scores64<T> sc(a, x, quick);
        double score = 0.0;
        const double k = lane < n ? sc.key(mine, score) : -INFINITY;
        int rank = 0;
        for (int j = 0; j < n; ++j) {
            const double o = __shfl_sync(kAll, k, j);
            const int e = __shfl_sync(kAll, mine, j);
            rank += o > k || (o == k && e < mine);
        }
        // what of a key may be off; the order is known where neighbours are further apart, or of equal terms
        const double off = sc.off * score + 0x1p-50 * fabs(k);
        int out = 0, from = 0;
        for (int j = 0; j < n; ++j) {
            const int r = __shfl_sync(kAll, rank, j), e = __shfl_sync(kAll, mine, j);
            if (r == lane) {
                out = e;
                from = j;
            }
        }
        if (!quick) return out;
        const int next = __shfl_down_sync(kAll, from, 1), after = __shfl_down_sync(kAll, out, 1);
        const double hi = __shfl_sync(kAll, k, from), lo = __shfl_sync(kAll, k, next);
        const double offs = __shfl_sync(kAll, off, from) + __shfl_sync(kAll, off, next);
        const bool known = lane >= n - 1 || hi - lo > offs || lo == -INFINITY ||
                           (sc.logit(out) == sc.logit(after) && a.bias[out] == a.bias[after]);
        if (__all_sync(kAll, known)) return out;
    }
}

__device__ __forceinline__ float ex2_approx(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float rcp_approx(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

constexpr float kLog2e = 1.4426950408889634f;

// The 32-bit key of a sum: of a logit v's score and a bias (m, inv: the softmax's largest logit and the inverse
// of its sum).
__device__ __forceinline__ float sum_key(bool softmax, float v, float m, float inv, float bias)
{
    const float s = softmax ? ex2_approx(kLog2e * (v == m ? 0.0f : v - m)) * inv
                            : rcp_approx(1.0f + ex2_approx(-kLog2e * v));
    const float key = s + bias;
    return v == -INFINITY || !(key >= -FLT_MAX) ? -INFINITY : key;  // masked; a bias of -infinity or NaN
}

// Whether two keys may be in the other order in exact arithmetic.
__device__ __forceinline__ bool near_keys(float hi, float lo, float slack)
{
    return hi - lo <= slack + 0x1p-22f * fminf(fmaxf(fabsf(hi), fabsf(lo)), FLT_MAX);
}

// Whether all experts with keys near that of expert `kth` have its logit and its bias.
template <typename T>
__device__ __noinline__ bool near_are_equal(const RouteArgs& a, const T* x, float m, float inv, float slack, int kth)
{
    const bool softmax = a.score == MOE_SCORE_SOFTMAX;
    const float l = to_f32(x[kth]), b = a.bias[kth], at = sum_key(softmax, l, m, inv, b);
    bool same = true;
    for (int e = threadIdx.x & 31; e < a.E; e += 32) {
        const float v = fmaxf(to_f32(x[e]), -INFINITY), o = sum_key(softmax, v, m, inv, a.bias[e]);
        if (near_keys(fmaxf(at, o), fminf(at, o), slack)) same = same && v == l && a.bias[e] == b;
    }
    return __all_sync(kAll, same);
}

}  // namespace

// A warp per token, expert 32 i + lane in the registers of a lane.
template <int PL, typename T>
__global__ void __launch_bounds__(32 * kRouteWarps, PL <= 12 ? 7 : 1) route_scores_kernel(RouteArgs a)
{
    extern __shared__ double s_all[];  // [kRouteWarps][E] keys, where there are groups
    __shared__ alignas(16) uint64_t s_key[kRouteWarps][32];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp;
    if (t >= a.T) return;
    double* s_keys = s_all + (a.groups > 1 ? (size_t)warp * a.E : 0);
    const T* x = static_cast<const T*>(a.logits) + t * a.stride;
    float l[PL];
    const bool softmax = a.score == MOE_SCORE_SOFTMAX;
#pragma unroll
    for (int i = 0; i < PL; ++i) l[i] = 32 * i + lane < a.E ? to_f32(x[32 * i + lane]) : -INFINITY;
    float bias[PL];    // (loaded here: no load passes the stores to shared memory below)
#pragma unroll
    for (int i = 0; i < PL; ++i) bias[i] = a.bias && 32 * i + lane < a.E ? a.bias[32 * i + lane] : 0.0f;
    bool nan = false;  // of this token's weights: a logit is NaN, which ranks last, or has no softmax
#pragma unroll
    for (int i = 0; i < PL; ++i) {
        nan = nan || l[i] != l[i];
        l[i] = fmaxf(l[i], -INFINITY);
    }
    const bool top2 = a.groups > 1 && a.group_score == MOE_GROUP_TOP2;
    const bool summed = a.bias || top2;  // keys of sums
    float m = 0.0f, inv = 1.0f;
    if (softmax && (summed || !a.renorm)) {
        m = -INFINITY;
#pragma unroll
        for (int i = 0; i < PL; ++i) m = fmaxf(m, l[i]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
        nan = nan || m == INFINITY;
        if (m == -INFINITY) m = 0.0f;
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < PL; ++i) sum += ex2_approx(kLog2e * (l[i] == m ? 0.0f : l[i] - m));
        sum = warp_sum(sum);
        inv = sum > 0.0f ? 1.0f / sum : 0.0f;
    }
    uint32_t key[PL];
    // How far apart two 32-bit keys are that may be in the other order, twice a key's own error: of a
    // sigmoid 2^-22 (its instructions are within 2^-22 and 2^-23 of their results, its exponent within
    // |l| 2^-24), of a softmax score 2^-18 of the largest (a lane's sum of up to 32 terms), and 2^-24 of
    // the sum with the bias.
    const float slack = softmax ? inv * 0x1p-17f : 0x1p-20f;
    auto near = [&](float hi, float lo) { return near_keys(hi, lo, slack); };
    float* keys32 = reinterpret_cast<float*>(s_keys);
#pragma unroll
    for (int i = 0; i < PL; ++i) {
        const int e = 32 * i + lane;
        key[i] = 0;
        if (e >= a.E) continue;
        float v = l[i], s = v;  // the expert's key, and what its group's score is made of
        if (summed) {
            s = sum_key(softmax, v, m, inv, bias[i]);
            if (a.bias) v = s;
        }
        if (a.groups > 1) keys32[e] = top2 ? s : v;
        key[i] = ordered(v);
    }
    bool again = false;
    if (a.groups > 1) {
        __syncwarp();
        float edge[2];
        float least;
        const float score = group_score(keys32, a.groups, a.group, top2, &least);
        uint32_t in = best_groups(score, a.groups, a.topk_groups, edge);
        if (summed && near(0.25f * edge[0], 0.25f * edge[1]))
            again = !border_groups(a, x, keys32, score, least, edge, near, reinterpret_cast<int*>(s_key[warp]), in);
#pragma unroll
        for (int i = 0; i < PL; ++i)
            if (!(in >> ((32 * i + lane) * a.group_mul >> 20 & 31) & 1)) key[i] = 0;
        __syncwarp();
    }
    int mine = 0;
    if (!again) {
        // one more than k where the order of sums may need 64 bits
        const int rounds = a.bias && a.k < a.E ? a.k + 1 : a.k;
        uint32_t kept;
        choose_32<PL>(key, rounds, s_key[warp], kept, mine);
        if (a.bias) {
            const uint32_t next = __shfl_down_sync(kAll, kept, 1);
            const int after = __shfl_down_sync(kAll, mine, 1);
            const bool apart = lane >= rounds - 1 || lane == 31 || !next || !near(unordered(kept), unordered(next));
            bool all = __all_sync(kAll, apart);
            if (!all || rounds > 32) {
                // the k are known where the next key is apart from the k-th, and so from all of them; or where the two
                // are of equal terms (whose sums are equal), if all keys near them are
                const bool equal = to_f32(x[mine]) == to_f32(x[after]) && a.bias[mine] == a.bias[after];
                const bool clear = __ballot_sync(kAll, apart) >> (a.k - 1) & 1;
                const bool even = __ballot_sync(kAll, equal) >> (a.k - 1) & 1;
                if (rounds <= 32 && (clear || even)) {
                    all = __all_sync(kAll, apart || equal || lane >= a.k - 1);
                    if (!clear && !near_are_equal(a, x, m, inv, slack, __shfl_sync(kAll, mine, a.k - 1)))
                        again = true;   // (the loop below would have the keys live across the call: 17.3 us where 16.0)
                    else if (!all)
                        mine = order_64(a, x, mine, a.k);
                } else {
                    // every expert that may be among the k: those with keys near the k-th, or before it
                    int c = 0;
                    float last = 0.0f;
                    for (bool more = true; more;) {
                        int p;
                        const uint32_t k = take_max<PL>(key, p);
                        more = k && (c < a.k || near(last, unordered(k)));
                        if (!more) break;
                        if (c == 32) again = true;
                        if (again) break;
                        if (lane == c) mine = p;
                        if (c < a.k) last = unordered(k);
                        ++c;
                    }
                    if (!again) mine = order_64(a, x, mine, c);
                }
            }
        }
    }
    if (again) mine = choose_64<PL>(a, x, s_keys);
    // lane j < k: the chosen expert's logit and weight
    const bool chosen = lane < a.k;
    float v = chosen ? to_f32(x[mine]) : -INFINITY, w;
    if (v != v) v = -INFINITY;
    if (!a.renorm) {
        w = v == -INFINITY ? 0.0f : softmax ? expf(v - m) * inv : 1.0f / (1.0f + expf(-v));
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

// A warp per token.  Renormalised scores and sigmoids: the chosen experts' logits alone have gradients,
// q (g - r) f with g the weights' gradients, q the weight / scale, r = sum_i g_i q_i, f the score's own derivative
// over it (softmax 1, sigmoid 1 - s); not renormalised g s (1 - s); each times scale.  Softmax scores that are not
// renormalised: p_e (sum of the g_j of expert e - sum_j g_j p_j), for every expert e (DENSE); of a chosen
// one the difference as a sum of differences.  Expert 32 i + lane is in the registers of a lane.  All of a
// token's are NaN where its weights are.
template <int PL, bool DENSE, typename T>
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
    // (the scale comes last: it would round the gradients whose differences count)
    float g = chosen ? a.dw[t * a.k + lane] : 0.0f;
    float p = 0.0f, r = 0.0f, inv = 0.0f, mass = 0.0f;   // mass: the positions' scores together
    float l[PL];
#pragma unroll
    for (int i = 0; i < PL; ++i) l[i] = 32 * i + lane < a.E ? to_f32(x[32 * i + lane]) : -INFINITY;
    if constexpr (DENSE) {
        float m = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int i = 0; i < PL; ++i) m = fmaxf(m, l[i]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
        if (m == -INFINITY) m = 0.0f;
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            l[i] = expf(l[i] - m);
            sum += l[i];
        }
        sum = warp_sum(sum);
        inv = sum > 0.0f ? 1.0f / sum : sum;
        p = chosen ? expf(v - m) * inv : 0.0f;
        mass = p;
        r = chosen ? g * p : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            mass += __shfl_xor_sync(kAll, mass, o);
            r += __shfl_xor_sync(kAll, r, o);
        }
        const float less = -(inv * r) * a.scale;
#pragma unroll
        for (int i = 0; i < PL; ++i)
            if (32 * i + lane < a.E) from_f32(l[i] * less, dx[32 * i + lane]);
    } else {
        // the row is read for its token's weights: NaN with a NaN logit, or an infinite one's softmax
        bool nan = false;
#pragma unroll
        for (int i = 0; i < PL; ++i) nan = nan || l[i] != l[i] || (softmax && l[i] == INFINITY);
        nan = __any_sync(kAll, nan);
#pragma unroll
        for (int i = 0; i < PL; ++i)
            if (32 * i + lane < a.E) from_f32(nan ? NAN : 0.0f, dx[32 * i + lane]);
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
            // g - r as the sum of q_i (g - g_i): where one weight is nearly all, g - r cancels
            float d = 0.0f;
            for (int i = 0; i < a.k; ++i)
                d = fmaf(__shfl_sync(kAll, q, i), g - __shfl_sync(kAll, g, i), d);
            g = chosen ? q * d * f : 0.0f;
        } else {
            const float s = 1.0f / (1.0f + expf(-v));
            g = chosen ? g * s / (1.0f + expf(v)) : 0.0f;
        }
        if (nan) g = NAN;
    }
    float all = 0.0f;  // of the positions that chose the same expert
    for (int j = 0; j < a.k; ++j) {
        const int other = __shfl_sync(kAll, id, j);
        const float gj = __shfl_sync(kAll, g, j);
        if (other == id) all += gj;
    }
    if constexpr (DENSE) {
        if (mass <= 0.75f) {
            all = p * (all - r);
        } else {
            // Where the others have few of the scores, all - r cancels (one logit 20 above 319 others: nothing is
            // left of it).  As differences: all times the others' scores, and the sum of p_i (all - all_i) over
            // the chosen experts.  (While the others have a quarter, |all| is at most four times the magnitudes of
            // these terms, all - r as good within that, and cheaper: 8192 tokens of 320, top-8, 4.4 us, with all
            // of them here 6.2.)
            uint32_t own = 0;      // bit i: this lane's expert 32 i + lane is chosen
            bool first = chosen;   // of the positions with this expert
#pragma unroll 4
            for (int j = 0; j < a.k; ++j) {
                const int other = __shfl_sync(kAll, id, j);
                if (other >= 0 && (other & 31) == lane) own |= 1u << (other >> 5);
                if (other == id && j < lane) first = false;
            }
            float rest = 0.0f;
#pragma unroll
            for (int i = 0; i < PL; ++i) rest += own >> i & 1 ? 0.0f : l[i];
            float d = all * (warp_sum(rest) * inv);
            const float q = first ? p : 0.0f;
#pragma unroll 4
            for (int j = 0; j < a.k; ++j)
                d = fmaf(__shfl_sync(kAll, q, j), all - __shfl_sync(kAll, all, j), d);
            all = p * d;
        }
    }
    __syncwarp();  // the row is written; its chosen experts' are written again
    if (chosen) from_f32(all * a.scale, dx[id]);
}

// Registers of a lane for a token's experts: powers of two and steps between them (320 experts in 10, not 16).
template <template <int, typename> class K, typename T, typename F>
static F with_pl(int E)
{
    return E <= 64 ? K<2, T>::get() : E <= 128 ? K<4, T>::get() : E <= 192 ? K<6, T>::get()
         : E <= 256 ? K<8, T>::get() : E <= 320 ? K<10, T>::get() : E <= 384 ? K<12, T>::get()
         : E <= 512 ? K<16, T>::get() : K<32, T>::get();
}
template <int PL, typename T>
struct Forward {
    static RouteKernel get() { return route_scores_kernel<PL, T>; }
};
template <int PL, typename T>
struct Dense {
    static RouteBackKernel get() { return route_back_kernel<PL, true, T>; }
};
template <int PL, typename T>
struct Sparse {
    static RouteBackKernel get() { return route_back_kernel<PL, false, T>; }
};
template <typename T>
static RouteBackKernel back_of(bool dense, int E)
{
    return dense ? with_pl<Dense, T, RouteBackKernel>(E) : with_pl<Sparse, T, RouteBackKernel>(E);
}

RouteKernel route_scores_kernel_for(int dtype, int E)
{
    switch (dtype) {
        case MOE_BF16: return with_pl<Forward, __nv_bfloat16, RouteKernel>(E);
        case MOE_FP16: return with_pl<Forward, __half, RouteKernel>(E);
        default: return with_pl<Forward, float, RouteKernel>(E);
    }
}

RouteBackKernel route_back_kernel_for(int dtype, bool dense, int E)
{
    switch (dtype) {
        case MOE_BF16: return back_of<__nv_bfloat16>(dense, E);
        case MOE_FP16: return back_of<__half>(dense, E);
        default: return back_of<float>(dense, E);
    }
}

}  // namespace moe
