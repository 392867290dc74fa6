// ep_router.hip -- the choice of experts: scores of each token's logits, the
// k best experts with their weights, and the gradient back to the logits.
//
//   score_e  = softmax_e(logits)            or  1 / (1 + exp(-logit_e))
//   value_e  = score_e + bias_e             (bias steers the choice only)
//   groups   of E/G consecutive experts are rated by the sum of their
//            group_top best values; the topk_groups best groups stay
//   choice   the k best experts left, best first, ties to the lowest index;
//            without a bias by logit, which orders like the score
//   weight_j = scale * score_ij [ / sum_j score_ij ]
//
// A logit of -inf or NaN takes the expert out: it is never chosen and its
// score is 0.  A value of -inf or NaN keeps it from being chosen, wherever
// values steer the choice (a bias, or groups rated by two).  With a logit of
// +inf all softmax scores of its row are NaN, and so are the weights of what
// is chosen by logit; by value nothing is left to choose.
//
// Backward, with r_j the renormalised weights and the choice held constant:
//   renormalised:  d logit_ij += scale * r_j (g_j - sum r g) * (softmax: 1,
//                  sigmoid: 1 - score_ij)
//   else           the gradient scale * g_j joins grad_probs at i_j
//   grad_probs B:  softmax: d logit_e += p_e (B_e - sum p B);
//                  sigmoid: d logit_e += p_e (1 - p_e) B_e
//
// Values near one another decide whole numbers, so wherever the choice
// depends on computed scores (a bias, or groups rated by a sum) scores and
// sums are formed in 64 bits (a fp64 multiply-add costs this chip no more
// than a fp32 one); a choice by logits alone compares the logits themselves.
//
// Design: a row is held by LPR lanes, VV vectors of four experts each
// (expert (i * LPR + lane) * 4 + c), so a row of up to 256 experts takes 16
// lanes and a wavefront works on four rows.  Every reduction is a butterfly
// inside the LPR lanes, in registers (lane moves of the DPP kind up to 16
// lanes), and the k best are taken one at a time, each round a scan of the
// lane's own values and one butterfly for the largest value, another for the
// lowest expert that has it.  Those rounds bound it: 8192 tokens of 256 fp32
// logits, k 8, take 6.3 us, 8.8 with all scores written (17 MB, 2.6 us of
// copying), and 16.8 with sigmoid, a bias and 8 groups, where the rounds scan
// 64-bit values and every score is a 64-bit exponential; the backward of the
// softmax with all scores 8.1.

#include "ep_internal.h"
#include "ep_layer.h"
#include "ep_types.h"

namespace ep {
namespace {

constexpr int kThreads = 256;
constexpr float kNegInf = -__builtin_inff();

// lane ^ STEP.  Up to 8 a DPP move (the mirror forms pair lane i with 7 - i
// and 15 - i, which meets lane ^ 4's and ^ 8's half: what is moved is the
// same in all lanes of a half); 16 and 32 swap rows of two registers, here
// copies of one, and take the half that is not the lane's own.
template <int STEP>
__device__ __forceinline__ uint32_t exchange(uint32_t v)
{
    if constexpr (STEP == 1) return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true);
    else if constexpr (STEP == 2) return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true);
    else if constexpr (STEP == 4) return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, true);
    else if constexpr (STEP == 8) return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, true);
    else if constexpr (STEP == 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        return (threadIdx.x & 16) ? r[0] : r[1];
    } else {
        const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        return (threadIdx.x & 32) ? r[0] : r[1];
    }
}
template <int STEP>
__device__ __forceinline__ float exchange(float v)
{
    return __uint_as_float(exchange<STEP>(__float_as_uint(v)));
}
template <int STEP>
__device__ __forceinline__ double exchange(double v)
{
    const uint64_t u = (uint64_t)__double_as_longlong(v);
    const uint32_t lo = exchange<STEP>((uint32_t)u), hi = exchange<STEP>((uint32_t)(u >> 32));
    return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}

template <int LPR, int STEP = 1, typename S>
__device__ __forceinline__ S row_sum(S v)
{
    if constexpr (STEP < LPR) return row_sum<LPR, STEP * 2>(v + exchange<STEP>(v));
    else return v;
}
__device__ __forceinline__ float larger(float a, float b) { return __builtin_fmaxf(a, b); }
__device__ __forceinline__ double larger(double a, double b) { return __builtin_fmax(a, b); }
template <int LPR, int STEP = 1, typename S>
__device__ __forceinline__ S row_max(S v)
{
    if constexpr (STEP < LPR) return row_max<LPR, STEP * 2>(larger(v, exchange<STEP>(v)));
    else return v;
}
template <int LPR, int STEP = 1>
__device__ __forceinline__ uint32_t row_min(uint32_t v)
{
    if constexpr (STEP < LPR) {
        const uint32_t o = exchange<STEP>(v);
        return row_min<LPR, STEP * 2>(o < v ? o : v);
    } else {
        return v;
    }
}
// the two largest of a >= b and c >= d
template <typename S>
__device__ __forceinline__ void two_best(S& a, S& b, S c, S d)
{
    const S lo = c > a ? a : c;
    a = c > a ? c : a;
    b = d > b ? d : b;
    b = lo > b ? lo : b;
}
// the two largest keys of `width` lanes (a power of two)
template <int LPR, int STEP = 1, typename S>
__device__ __forceinline__ void group_top2(S& a, S& b, int width)
{
    if constexpr (STEP < LPR) {
        if (STEP >= width) return;
        two_best(a, b, exchange<STEP>(a), exchange<STEP>(b));
        group_top2<LPR, STEP * 2>(a, b, width);
    }
}

// Four experts from `e` on: logits of a row in fp32; past E, and where the
// logit is NaN, -inf.
template <typename T>
__device__ __forceinline__ void load4(const T* row, int e, int E, float (&f)[4])
{
    if (e + 4 <= E) {
        T raw[4];
        __builtin_memcpy(raw, row + e, sizeof raw);
#pragma unroll
        for (int c = 0; c < 4; ++c) f[c] = to_float(raw[c]);
    } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) f[c] = e + c < E ? to_float(row[e + c]) : kNegInf;
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) f[c] = f[c] == f[c] ? f[c] : kNegInf;
}

// A row of logits for a second reading by few: hidden from the compiler that
// it is the same, which would hold the first reading's values for all (8192 x
// 512 with a bias: 48.3 us against 44.8).
template <typename T>
__device__ __forceinline__ const T* read_again(const T* row)
{
    asm("" : "+v"(row));
    return row;
}

// WIDE: 64-bit values (score + bias) rate the groups and, with a bias, make the
// choice; else both are by the logits.
template <typename T, int LPR, int VV, bool WIDE>
__global__ __launch_bounds__(kThreads)
void router_kernel(const T* __restrict__ logits, int64_t num_tokens, int E, int64_t ld, int k,
                   int softmax, const float* __restrict__ bias, int num_groups, int topk_groups,
                   int group_top, int renormalize, float scale, int64_t* __restrict__ topk_idx,
                   float* __restrict__ topk_weights, float* __restrict__ probs)
{
    using Key = typename std::conditional<WIDE, double, float>::type;
    constexpr int kRows = kThreads / LPR;
    constexpr int kSel = 64 / LPR;     // choices held per lane (k <= 64)
    __shared__ Key rating[kRows][64];
    const int lr = threadIdx.x % LPR;
    const int r = threadIdx.x / LPR;
    const int64_t row = (int64_t)blockIdx.x * kRows + r;
    const bool live = row < num_tokens;
    const T* x = logits + (live ? row : num_tokens - 1) * ld;

    float l[VV][4];
#pragma unroll
    for (int i = 0; i < VV; ++i) load4(x, (i * LPR + lr) * 4, E, l[i]);

    // softmax statistics: m the largest logit (0 for a row with none left),
    // z the sum of exp(l - m), NaN where m is +inf
    float m = 0.0f;
    if (softmax) {
        m = kNegInf;
#pragma unroll
        for (int i = 0; i < VV; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) m = l[i][c] > m ? l[i][c] : m;
        m = row_max<LPR>(m);
        m = m == kNegInf ? 0.0f : m;
    }
    Key val[VV][4];
    Key z = 0;
    if constexpr (WIDE) {
#pragma unroll
        for (int i = 0; i < VV; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const double d = softmax ? exp((double)l[i][c] - (double)m)
                                         : 1.0 / (1.0 + exp(-(double)l[i][c]));
                val[i][c] = d;
                z += d;
            }
        if (softmax) z = row_sum<LPR>(z);
        const double inv = softmax ? 1.0 / (z == 0 ? 1.0 : z) : 1.0;
#pragma unroll
        for (int i = 0; i < VV; ++i) {
            const int e = (i * LPR + lr) * 4;
            if (probs != nullptr && live) {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (e + c < E)
                        probs[row * E + e + c] = l[i][c] > kNegInf ? (float)(val[i][c] * inv) : 0.0f;
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const double b = bias != nullptr && e + c < E ? (double)bias[e + c] : 0.0;
                const double v = val[i][c] * inv + b;
                val[i][c] = l[i][c] > kNegInf && v == v ? v : (double)kNegInf;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < VV; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) val[i][c] = l[i][c];
        if (probs != nullptr || (softmax && !renormalize)) {
            float p[VV][4];
#pragma unroll
            for (int i = 0; i < VV; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    p[i][c] = softmax ? expf(l[i][c] - m) : 1.0f / (1.0f + expf(-l[i][c]));
                    z += p[i][c];
                }
            if (softmax) z = row_sum<LPR>(z);
            if (probs != nullptr && live) {
                const float inv = softmax ? 1.0f / (z == 0 ? 1.0f : z) : 1.0f;
#pragma unroll
                for (int i = 0; i < VV; ++i) {
                    const int e = (i * LPR + lr) * 4;
#pragma unroll
                    for (int c = 0; c < 4; ++c) p[i][c] = l[i][c] > kNegInf ? p[i][c] * inv : 0.0f;
                    if (e + 4 <= E && (E & 3) == 0) {
                        *reinterpret_cast<float4*>(probs + row * E + e) =
                            make_float4(p[i][0], p[i][1], p[i][2], p[i][3]);
                    } else {
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            if (e + c < E) probs[row * E + e + c] = p[i][c];
                    }
                }
            }
        }
    }

    if (num_groups > 1) {
        // rate each group, then keep those with fewer than topk_groups better
        // ones (ties to the lower group)
        const int per = E / num_groups;
        const int seg = per / 4;            // lanes of a group, if it is whole vectors
        if (per % 4 == 0 && seg <= LPR && (seg & (seg - 1)) == 0) {
            // each vector's lanes hold whole groups side by side: the two best
            // of the vector, then of the group's lanes
#pragma unroll
            for (int i = 0; i < VV; ++i) {
                Key a = (Key)kNegInf, b = (Key)kNegInf;
#pragma unroll
                for (int c = 0; c < 4; ++c) two_best(a, b, val[i][c], (Key)kNegInf);
                group_top2<LPR>(a, b, seg);
                if (group_top > 1 && b > (Key)kNegInf) a += b;
                const int g = (i * LPR + lr) / seg;
                if (lr % seg == 0 && g < num_groups) rating[r][g] = a;
            }
        } else {
            for (int g = 0; g < num_groups; ++g) {
                Key a = (Key)kNegInf, b = (Key)kNegInf;
#pragma unroll
                for (int i = 0; i < VV; ++i)
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int e = (i * LPR + lr) * 4 + c;
                        const Key v = e >= g * per && e < (g + 1) * per ? val[i][c] : (Key)kNegInf;
                        two_best(a, b, v, (Key)kNegInf);
                    }
                group_top2<LPR>(a, b, LPR);
                if (group_top > 1 && b > (Key)kNegInf) a += b;
                if (lr == 0) rating[r][g] = a;
            }
        }
        __syncthreads();
        uint64_t keep = 0;
#pragma unroll
        for (int q = 0; q < kSel; ++q) {
            const int g = q * LPR + lr;
            bool in = false;
            if (g < num_groups) {
                const Key mine = rating[r][g];
                int better = 0;
                for (int o = 0; o < num_groups; ++o) {
                    const Key other = rating[r][o];
                    better += other > mine || (other == mine && o < g);
                }
                in = better < topk_groups;
            }
            const uint64_t all = __ballot(in) >> ((threadIdx.x & 63) / LPR * LPR);
            keep |= (LPR == 64 ? all : all & ((1ull << (LPR % 64)) - 1)) << (q * LPR);
        }
#pragma unroll
        for (int i = 0; i < VV; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int e = (i * LPR + lr) * 4 + c;
                const int g = e < E ? e / per : 0;
                if (!((keep >> g) & 1)) val[i][c] = (Key)kNegInf;
            }
        if constexpr (WIDE) {
            if (bias == nullptr) {
                // the scores have rated the groups; the choice is by logit,
                // also among scores that are the same number
                const T* again = read_again(x);
#pragma unroll
                for (int i = 0; i < VV; ++i) {
                    float f[4];
                    load4(again, (i * LPR + lr) * 4, E, f);
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (val[i][c] > (Key)kNegInf) val[i][c] = (Key)f[c];
                }
            }
        }
    }

    // the k best, one a round; lane j % LPR keeps choice j
    int sel[kSel];
#pragma unroll
    for (int q = 0; q < kSel; ++q) sel[q] = -1;
    for (int j = 0; j < k; ++j) {
        // the largest value of the row, then the lowest expert that has it
        Key best = (Key)kNegInf;
#pragma unroll
        for (int i = 0; i < VV; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) best = larger(best, val[i][c]);
        best = row_max<LPR>(best);
        uint32_t at = 0xFFFFFFFFu;
#pragma unroll
        for (int i = VV - 1; i >= 0; --i)
#pragma unroll
            for (int c = 3; c >= 0; --c)
                at = val[i][c] == best ? (uint32_t)((i * LPR + lr) * 4 + c) : at;
        at = row_min<LPR>(at);
#pragma unroll
        for (int i = 0; i < VV; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (at == (uint32_t)((i * LPR + lr) * 4 + c)) val[i][c] = (Key)kNegInf;
#pragma unroll
        for (int q = 0; q < kSel; ++q)
            if (j == q * LPR + lr) sel[q] = best > (Key)kNegInf ? (int)at : -1;
    }

    // weights of the choices, from their logits, in 64 bits: a renormalised
    // softmax relative to the largest chosen logit, so it cannot underflow
    double w[kSel];
    float ls[kSel];
    float ms = kNegInf;
#pragma unroll
    for (int q = 0; q < kSel; ++q) {
        ls[q] = sel[q] >= 0 ? to_float(x[sel[q]]) : kNegInf;
        ms = ls[q] > ms ? ls[q] : ms;
    }
    if (softmax && renormalize) {
        ms = row_max<LPR>(ms);
        ms = ms == kNegInf ? 0.0f : ms;
    } else {
        ms = m;
    }
    double sum = 0.0;
#pragma unroll
    for (int q = 0; q < kSel; ++q) {
        w[q] = 0.0;
        if (sel[q] >= 0)
            w[q] = softmax ? exp((double)ls[q] - (double)ms) : 1.0 / (1.0 + exp(-(double)ls[q]));
        sum += w[q];
    }
    double div = 1.0;
    if (renormalize) div = row_sum<LPR>(sum);
    else if (softmax) div = (double)z;
    const double f = div > 0.0 || div != div ? (double)scale / div : 0.0;
#pragma unroll
    for (int q = 0; q < kSel; ++q) {
        const int j = q * LPR + lr;
        if (live && j < k) {
            topk_idx[row * k + j] = sel[q];
            topk_weights[row * k + j] = sel[q] >= 0 ? (float)(w[q] * f) : 0.0f;
        }
    }
}

template <typename T, int LPR, int VV>
__global__ __launch_bounds__(kThreads)
void router_backward_kernel(const T* __restrict__ logits, int64_t num_tokens, int E, int64_t ld,
                            int k, int softmax, int renormalize, float scale,
                            const int64_t* __restrict__ topk_idx,
                            const float* __restrict__ grad_weights,
                            const float* __restrict__ grad_probs, T* __restrict__ grad_logits)
{
    constexpr int kRows = kThreads / LPR;
    constexpr int kSel = 64 / LPR;
    const int lr = threadIdx.x % LPR;
    const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / LPR;
    const bool live = row < num_tokens;
    const int64_t at = live ? row : num_tokens - 1;
    const T* x = logits + at * ld;

    // choices: lane j % LPR holds choice j, its gradient and its logit
    int sel[kSel];
    float gw[kSel], ls[kSel];
    float ms = kNegInf;
#pragma unroll
    for (int q = 0; q < kSel; ++q) {
        const int j = q * LPR + lr;
        sel[q] = -1;
        gw[q] = 0.0f;
        ls[q] = kNegInf;
        if (j < k) {
            const int64_t e = topk_idx[at * k + j];
            if (e >= 0 && e < E) {
                ls[q] = to_float(x[e]);
                if (ls[q] > kNegInf) {
                    sel[q] = (int)e;
                    gw[q] = grad_weights[at * k + j] * scale;
                    ms = ls[q] > ms ? ls[q] : ms;
                }
            }
        }
    }
    float direct[kSel];
    if (renormalize) {
        ms = row_max<LPR>(ms);
        ms = ms == kNegInf ? 0.0f : ms;
        // Scores relative to the largest chosen one, so that they do not
        // vanish in fp32 where the forward's 64 bits hold them.  Sigmoid with
        // all chosen logits below 0: exp(l - ms) / (1 + exp(l)), the score
        // over exp(ms).  Where the forward's scores are 0 (exp(-ms) is past
        // the largest double) so are its weights, and these.
        const bool below = !softmax && ms < 0.0f;
        const bool zero = below && (double)ms < -709.782712893384;
        float s[kSel], sum = 0.0f, dot = 0.0f;
#pragma unroll
        for (int q = 0; q < kSel; ++q) {
            s[q] = 0.0f;
            if (q * LPR >= k) continue;         // no choice here in any row
            s[q] = softmax || below ? expf(ls[q] - ms) : 1.0f;
            if (!softmax) s[q] /= 1.0f + expf(below ? ls[q] : -ls[q]);
            if (sel[q] < 0 || zero) s[q] = 0.0f;
            sum += s[q];
            dot = __builtin_fmaf(s[q], gw[q], dot);
        }
        sum = row_sum<LPR>(sum);
        dot = row_sum<LPR>(dot);
        const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
        for (int q = 0; q < kSel; ++q) {
            direct[q] = 0.0f;
            if (q * LPR >= k) continue;
            direct[q] = s[q] * inv * (gw[q] - dot * inv);
            if (!softmax) direct[q] *= 1.0f / (1.0f + expf(ls[q]));    // 1 - score
            if (sel[q] < 0) direct[q] = 0.0f;
        }
    }

    float out[VV][4];
    float whole = 0.0f;             // the softmax's sum: NaN in a row with a logit of +inf
    const bool dense = grad_probs != nullptr || !renormalize;
    if (dense) {
        float l[VV][4], b[VV][4];
#pragma unroll
        for (int i = 0; i < VV; ++i) {
            const int e = (i * LPR + lr) * 4;
            load4(x, e, E, l[i]);
            if (grad_probs != nullptr && e + 4 <= E) {
                __builtin_memcpy(b[i], grad_probs + at * E + e, 16);
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    b[i][c] = grad_probs != nullptr && e + c < E ? grad_probs[at * E + e + c] : 0.0f;
            }
        }
        if (!renormalize) {
            for (int j = 0; j < k; ++j) {
                int ej = -1;
                float gj = 0.0f;
#pragma unroll
                for (int q = 0; q < kSel; ++q)
                    if (j / LPR == q) {
                        ej = __shfl(sel[q], j % LPR, LPR);
                        gj = __shfl(gw[q], j % LPR, LPR);
                    }
#pragma unroll
                for (int i = 0; i < VV; ++i)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        b[i][c] += ej == (i * LPR + lr) * 4 + c ? gj : 0.0f;
            }
        }
        if (softmax) {
            float m = kNegInf;
#pragma unroll
            for (int i = 0; i < VV; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) m = l[i][c] > m ? l[i][c] : m;
            m = row_max<LPR>(m);
            m = m == kNegInf ? 0.0f : m;
            float z = 0.0f, dot = 0.0f;
#pragma unroll
            for (int i = 0; i < VV; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float p = expf(l[i][c] - m);
                    z += p;
                    // a masked expert's probability is 0 whatever its gradient
                    dot = p != 0.0f ? __builtin_fmaf(p, b[i][c], dot) : dot;
                    l[i][c] = p;
                }
            z = row_sum<LPR>(z);
            dot = row_sum<LPR>(dot);
            const float inv = z != 0.0f ? 1.0f / z : 0.0f;
#pragma unroll
            for (int i = 0; i < VV; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    out[i][c] = l[i][c] != 0.0f ? l[i][c] * inv * (b[i][c] - dot * inv) : 0.0f;
            whole = z;
        } else {
#pragma unroll
            for (int i = 0; i < VV; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float p = 1.0f / (1.0f + expf(-l[i][c]));
                    const float q = 1.0f / (1.0f + expf(l[i][c]));
                    out[i][c] = l[i][c] > kNegInf ? b[i][c] * p * q : 0.0f;
                }
        }
    } else {
#pragma unroll
        for (int i = 0; i < VV; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) out[i][c] = 0.0f;
    }
    if (renormalize) {
        for (int j = 0; j < k; ++j) {
            int ej = -1;
            float gj = 0.0f;
#pragma unroll
            for (int q = 0; q < kSel; ++q)
                if (j / LPR == q) {
                    ej = __shfl(sel[q], j % LPR, LPR);
                    gj = __shfl(direct[q], j % LPR, LPR);
                }
#pragma unroll
            for (int i = 0; i < VV; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    out[i][c] += ej == (i * LPR + lr) * 4 + c ? gj : 0.0f;
        }
    }
    if (!live) return;
    T* o = grad_logits + row * E;
    if (whole != whole) {           // every gradient of the row, its masked experts apart
        for (int i = 0; i < VV; ++i) {
            const int e = (i * LPR + lr) * 4;
            float f[4];
            load4(x, e, E, f);
            for (int c = 0; c < 4; ++c)
                if (e + c < E) o[e + c] = from_float<T>(f[c] > kNegInf ? whole : 0.0f);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < VV; ++i) {
        const int e = (i * LPR + lr) * 4;
        if (e + 4 <= E) {
            T raw[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) raw[c] = from_float<T>(out[i][c]);
            __builtin_memcpy(o + e, raw, sizeof raw);
        } else {
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (e + c < E) o[e + c] = from_float<T>(out[i][c]);
        }
    }
}

// f(lanes per row, vectors per lane) for a row of E experts: 4 lanes up to
// 16 experts, 16 up to 256, 64 beyond.  Few rows leave the chip idle and only
// the length of the chain counts: then 65 to 256 experts take 64 lanes too.
// Measured on MI355X, us in a graph, 16 against 64 lanes, in brackets with
// sigmoid, a bias and 8 groups: 256 experts, 1 token 5.0 / 3.7 (12.9 / 6.1),
// 2048 tokens 5.4 / 4.9 (13.7 / 8.3), 4096 5.5 / 6.8 (13.9 / 11.1), 8192 6.4 /
// 11.0 (17.0 / 18.5); 128 experts, 1024 tokens 4.3 / 4.2 (8.6 / 6.6), 2048 4.4
// / 4.9 (8.7 / 8.1); 96 experts, 1 token 4.0 / 3.8 (11.1 / 9.1), 1024 tokens
// 4.4 / 4.2 (11.6 / 9.6), 2048 4.4 / 4.9 (11.6 / 12.5); the backward at 256
// experts, 1 token 4.3 / 3.0, 2048 4.8 / 3.6, 4096 5.1 / 4.5, 8192 5.4 / 6.4.
template <typename F>
hipError_t with_row_shape(int E, int64_t num_tokens, F&& f)
{
    if (E <= 16) return f(std::integral_constant<int, 4>(), std::integral_constant<int, 1>());
    if (E <= 64) return f(std::integral_constant<int, 16>(), std::integral_constant<int, 1>());
    if (E <= 256 && num_tokens <= (E <= 128 ? 1024 : 2048))
        return f(std::integral_constant<int, 64>(), std::integral_constant<int, 1>());
    if (E <= 128) return f(std::integral_constant<int, 16>(), std::integral_constant<int, 2>());
    if (E <= 256) return f(std::integral_constant<int, 16>(), std::integral_constant<int, 4>());
    return f(std::integral_constant<int, 64>(), std::integral_constant<int, 4>());
}

template <typename T>
hipError_t router_of(const RouterArgs& a, hipStream_t stream)
{
    const bool wide = a.bias != nullptr || (a.num_groups > 1 && a.group_top > 1);
    return with_row_shape(a.num_experts, a.num_tokens, [&](auto lpr, auto vv) {
        constexpr int kRows = kThreads / decltype(lpr)::value;
        const dim3 grid((unsigned)((a.num_tokens + kRows - 1) / kRows));
        auto go = [&](auto w) {
            hipLaunchKernelGGL((router_kernel<T, decltype(lpr)::value, decltype(vv)::value,
                                              decltype(w)::value>),
                               grid, dim3(kThreads), 0, stream, static_cast<const T*>(a.logits),
                               a.num_tokens, a.num_experts, a.ld, a.num_topk, a.softmax, a.bias,
                               a.num_groups, a.topk_groups, a.group_top, a.renormalize, a.scale,
                               a.topk_idx, a.topk_weights, a.probs);
            return hipGetLastError();
        };
        return wide ? go(std::true_type()) : go(std::false_type());
    });
}

template <typename T>
hipError_t router_backward_of(const RouterBackwardArgs& a, hipStream_t stream)
{
    return with_row_shape(a.num_experts, a.num_tokens, [&](auto lpr, auto vv) {
        constexpr int kRows = kThreads / decltype(lpr)::value;
        const dim3 grid((unsigned)((a.num_tokens + kRows - 1) / kRows));
        hipLaunchKernelGGL((router_backward_kernel<T, decltype(lpr)::value, decltype(vv)::value>),
                           grid, dim3(kThreads), 0, stream, static_cast<const T*>(a.logits),
                           a.num_tokens, a.num_experts, a.ld, a.num_topk, a.softmax, a.renormalize,
                           a.scale, a.topk_idx, a.grad_weights, a.grad_probs,
                           static_cast<T*>(a.grad_logits));
        return hipGetLastError();
    });
}

}  // namespace

hipError_t launch_router(int dtype, const RouterArgs& a, hipStream_t stream)
{
    if (dtype == 0) return router_of<Bf16>(a, stream);
    if (dtype == 1) return router_of<Fp16>(a, stream);
    return router_of<float>(a, stream);
}

hipError_t launch_router_backward(int dtype, const RouterBackwardArgs& a, hipStream_t stream)
{
    if (dtype == 0) return router_backward_of<Bf16>(a, stream);
    if (dtype == 1) return router_backward_of<Fp16>(a, stream);
    return router_backward_of<float>(a, stream);
}

}  // namespace ep
