// ep_route.hip -- the router: scores, the K best experts of every token and
// their weights, the balance loss of each source, and the gradient of the
// logits.
//
// One wave per token; lane i holds the PER neighbouring experts i*PER..., so a
// row is one coalesced load, "the lowest index" is the lowest lane, and all
// state stays in registers.  The K best are found by K rounds of a wave maximum
// (six register steps) and a ballot for the lane that holds it.
#include "ep_kernels.h"
#include "ep_wave.h"

namespace ep {
namespace {

constexpr int kWaves = 4;
constexpr int kThreads = kWaves * kWave;
constexpr int kManyTokens = 8192;
// Waves of a forward workgroup.  With the balance loss each workgroup leaves one
// partial sum per expert to be added, so for many tokens there are few, large
// ones (as much as their LDS allows); up to kFewTokens small ones, which wait
// less for each other (38 tokens over 384 experts, top-11: 27 us with sixteen
// waves).
constexpr int kFewTokens = 1024;
constexpr int large_waves(int per) { return per > 8 ? 8 : 16; }

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float lowest(const float *) { return -3.402823466e+38f; }
__device__ __forceinline__ float lowest(const uint16_t *) { return __uint_as_float(0xff7f0000u); }
__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ void narrow(float v, float &o) { o = v; }
__device__ __forceinline__ void narrow(float v, uint16_t &o) { o = (uint16_t)to_bf16(v); }

template <typename T, int PER>
struct alignas(sizeof(T) * PER < 16 ? sizeof(T) * PER : 16) Pack {
    T v[PER];
};

// The lane's logits; masked ones (and places beyond E) as -inf, +inf as the
// type's largest value.
template <typename T, int PER>
__device__ __forceinline__ void load_logits(const T *row, int E, int lane, bool open, bool vec, float (&l)[PER]) {
    Pack<T, PER> p;
    const int e0 = lane * PER;
    const bool full = e0 + PER <= E;
    if (vec) {
        if (full) p = *reinterpret_cast<const Pack<T, PER> *>(row + e0);
    } else {
#pragma unroll
        for (int j = 0; j < PER; ++j)
            if (e0 + j < E) p.v[j] = row[e0 + j];
    }
    const float lo = lowest(row);
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const bool in = vec ? full : e0 + j < E;
        const float v = in ? widen(p.v[j]) : lo;
        l[j] = open && v > lo ? fminf(v, -lo) : -INFINITY;
    }
}

// exp(d + e), d <= 0, e far below d, from the hardware's exp2: the argument's
// product with log2(e) is carried in two parts, so the error is a few 2^-24 of
// the value however long the argument is (with one part: |d| 2^-24).
__device__ __forceinline__ float exp_of(float d, float e) {
    const float p = d * 1.44269502f;
    const float r = fmaf(e, 1.44269502f, fmaf(d, 1.92596303e-8f, fmaf(d, 1.44269502f, -p)));
    return __builtin_amdgcn_exp2f(p) * fmaf(r, 0.69314718f, 1.0f);
}
// exp(l - top), l <= top, with the difference's own rounding; 0 where it is
// below the normal numbers (and for -inf).
__device__ __forceinline__ float exp_below(float l, float top) {
    const float d = l - top, z = d - l, e = (l - (d - z)) - (top + z);
    const float v = exp_of(d, e);
    return d > -110.0f ? v : 0.0f;
}

// 1 / (1 + exp(-l)) without overflow on either side; 0 for -inf.
__device__ __forceinline__ float sigmoid(float l) {
    const float z = expf(-fabsf(l));
    return (l >= 0.0f ? 1.0f : z) / (1.0f + z);
}
__device__ __forceinline__ double sigmoid(double l) {
    const double z = exp(-fabs(l));
    return (l >= 0.0 ? 1.0 : z) / (1.0 + z);
}

// Keys s + bias in 32 bits that lie closer than this times max(1, |key|) are
// compared in 64 bits.  The error of their difference, u = 2^-24: the softmax sum
// is off by a step of u at each addition, 15 in a lane and 6 across the lanes, by
// 4 u of its exponentials, the division by u; that scales both scores and moves
// their difference, at most 1, by 26 u.  Each score has 5 u more of its own (the
// two are at most 1 together) and each sum with the bias rounds once: 33 u, and 3
// for the difference and its bound.  (A sigmoid score is off by 3 u.)
constexpr float kKeyError = 36.0f * 0x1p-24f;

// K rounds of "largest key, lowest index".  Lane k of the result holds the k-th
// expert and its logit, bit j of `taken` says that the lane's j-th expert was
// chosen, `close` that two of the K+1 best keys lie closer than rounding tells
// apart.
template <int PER, typename Key>
__device__ __forceinline__ int select(Key (&key)[PER], const float (&l)[PER], int K, int lane, bool want_gap, int &idx,
                                      float &lsel, uint32_t &taken, bool &close) {
    idx = -1;
    taken = 0;
    lsel = -INFINITY;
    close = false;
    int n = 0;
    Key prev = 0;
    const int rounds = want_gap ? K + 1 : K;
    for (int k = 0; k < rounds; ++k) {
        Key best = key[0];
        int at = 0;
        float lv = l[0];
#pragma unroll
        for (int j = 1; j < PER; ++j) {
            const Key kj = key[j];
            const float lj = l[j];
            const bool more = kj > best;
            best = more ? kj : best;
            at = more ? j : at;
            lv = more ? lj : lv;
        }
        const Key top = wave_max(best);
        if (!(top > (Key)-INFINITY)) break;
        if (want_gap && k > 0) {
            const Key a = top < 0 ? -top : top, b = prev < 0 ? -prev : prev;
            const Key unit = a > b ? (a > 1 ? a : (Key)1) : (b > 1 ? b : (Key)1);
            if (!(prev - top > (Key)kKeyError * unit)) close = true;
        }
        prev = top;
        if (k == K) break;
        const int owner = __builtin_ctzll(ballot(best == top));
        const int e = owner * PER + read_lane(at, owner);
        const float le = read_lane_f(lv, owner);
        if (lane == k) {
            idx = e;
            lsel = le;
        }
        n = k + 1;
#pragma unroll
        for (int j = 0; j < PER; ++j)
            if (lane * PER + j == e) {
                key[j] = (Key)-INFINITY;
                taken |= 1u << j;
            }
    }
    return n;
}

template <int PER>
__device__ __forceinline__ float sum_of(const float (&v)[PER]) {
    float t = 0.0f;
#pragma unroll
    for (int j = 0; j < PER; ++j) t += v[j];
    return wave_sum(t);
}

// Scores of the lane's experts from their logits: sigmoid, or softmax with the
// given maximum; `all` = the sum over the token's experts (softmax: of the
// exponentials, already divided out).
template <int PER, bool SIG>
__device__ __forceinline__ void scores(const float (&l)[PER], float top, float (&s)[PER], float &inv, float &all) {
#pragma unroll
    for (int j = 0; j < PER; ++j) s[j] = SIG ? sigmoid(l[j]) : exp_below(l[j], top);
    all = sum_of(s);
    inv = 1.0f;
    if (!SIG) {
        inv = 1.0f / fmaxf(all, 1e-30f);
#pragma unroll
        for (int j = 0; j < PER; ++j) s[j] *= inv;
    }
}

template <int PER>
__device__ __forceinline__ float top_of(const float (&l)[PER]) {
    float m = l[0];
#pragma unroll
    for (int j = 1; j < PER; ++j) m = fmaxf(m, l[j]);
    return wave_max(m);
}

// blockIdx.y = source, blockIdx.x = block of that source's tokens; each wave
// takes tokens wave0, wave0 + nwaves, ...
template <typename T, int PER, bool SIG, bool BAL, int W>
__global__ void __launch_bounds__(kWave *W) k_route(RouteArgs a) {
    constexpr int kWaves = W, kThreads = kWaves * kWave;
    const int lane = lane_id(), wave = threadIdx.x / kWave;
    const int s = blockIdx.y, E = a.E, K = a.K;
    double psum[PER];  // equal probabilities round one way: 1024 additions in fp32 were off by 1.5e-5
    int cnt[PER], seen = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) psum[j] = 0.0, cnt[j] = 0;
    if (BAL && blockIdx.x == 0 && threadIdx.x == 0) a.part_done[s] = 0;  // for k_route_sum
    for (int64_t t = (int64_t)blockIdx.x * kWaves + wave; t < a.T; t += (int64_t)gridDim.x * kWaves) {
        const int64_t g = (int64_t)s * a.T + t;
        const bool open = !a.token_mask || a.token_mask[g] != 0;
        float l[PER], sc[PER];
        load_logits<T, PER>(static_cast<const T *>(a.logits) + g * E, E, lane, open, a.vec, l);
        const float top = top_of(l);
        const bool any = top > -INFINITY;
        float inv, all;
        scores<PER, SIG>(l, any ? top : 0.0f, sc, inv, all);
        int idx, n;
        float lsel;
        bool close = false;
        uint32_t taken;
        float key[PER];
        if (!a.bias) {
#pragma unroll
            for (int j = 0; j < PER; ++j) key[j] = l[j];
            n = select<PER>(key, l, K, lane, false, idx, lsel, taken, close);
        } else {
            float b[PER];
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                const int e = lane * PER + j;
                b[j] = e < E ? a.bias[e] : 0.0f;
                const float v = sc[j] + b[j];
                key[j] = l[j] > -INFINITY && b[j] == b[j] ? v : -INFINITY;
            }
            n = select<PER>(key, l, K, lane, true, idx, lsel, taken, close);
            if (close) {  // rare: settle the order in 64 bits
                double kd[PER], sum = 0.0;
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    kd[j] = SIG ? sigmoid((double)l[j]) : exp((double)l[j] - (double)top);
                    if (!SIG) sum += kd[j];
                }
                if (!SIG) {
#pragma unroll
                    for (int d = 32; d; d >>= 1)
                        sum += __hiloint2double(shfl(__double2hiint(sum), lane ^ d), shfl(__double2loint(sum), lane ^ d));
                }
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    const double v = (SIG ? kd[j] : kd[j] / sum) + (double)b[j];
                    kd[j] = l[j] > -INFINITY && b[j] == b[j] ? v : -(double)INFINITY;
                }
                bool none;
                n = select<PER>(kd, l, K, lane, false, idx, lsel, taken, none);
            }
        }
        const bool chosen = lane < n;
        const float sk = chosen ? (SIG ? sigmoid(lsel) : exp_below(lsel, top) * inv) : 0.0f;
        const float D = wave_sum(sk) + 1e-20f;
        if (lane < K) {
            a.topk_idx[g * K + lane] = idx;
            a.topk_weights[g * K + lane] = chosen ? a.scale * (sk / D) : 0.0f;
        }
        if (BAL) {
            seen += any ? 1 : 0;
            const float r = SIG ? 1.0f / (all + 1e-20f) : 1.0f;
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                psum[j] += (double)(any ? sc[j] * r : 0.0f);
                cnt[j] += (taken >> j) & 1u;
            }
        }
    }
    if (BAL) {
        // The block's sums, waves in order; one place per (source, block, expert).
        __shared__ float lp[kWaves][kWave * PER];
        __shared__ int lc[kWaves][kWave * PER];
        __shared__ int ls[kWaves];
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            lp[wave][lane * PER + j] = (float)psum[j];
            lc[wave][lane * PER + j] = cnt[j];
        }
        if (lane == 0) ls[wave] = seen;
        __syncthreads();
        const int64_t unit = (int64_t)s * gridDim.x + blockIdx.x;
        for (int e = threadIdx.x; e < a.pitch; e += kThreads) {
            double p = 0.0;
            int c = 0;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) p += (double)lp[w][e], c += lc[w][e];
            a.part_p[unit * a.pitch + e] = (float)p;
            a.part_cnt[unit * a.pitch + e] = c;
        }
        if (threadIdx.x == 0) {
            int n = 0;
            for (int w = 0; w < kWaves; ++w) n += ls[w];
            a.part_seen[unit] = n;
        }
    }
}

// Counts, valid tokens and the loss of source blockIdx.y from the workgroups'
// partial sums, 32 experts per workgroup.  Thread (quad, part) adds every 32nd
// partial sum of four neighbouring experts in order, eight loads in flight (one
// at a time took 74 us instead of 6 at 1024 partial sums of 256 experts).  The
// last workgroup to finish adds the shares of the loss, in order.  Sums over
// tokens and experts are held in 64 bits; a wave's and a workgroup's sums are
// rounded to 32 once each.
constexpr int kSumThreads = 256, kSumExperts = 32, kSumQuads = kSumExperts / 4, kSumParts = kSumThreads / kSumQuads;
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
__global__ void __launch_bounds__(kSumThreads) k_route_sum(RouteArgs a, int blocks) {
    __shared__ double lp[kSumParts][kSumExperts + 1];
    __shared__ int lc[kSumParts][kSumExperts + 1];
    __shared__ int seen, last;
    constexpr int G = 8;
    const int s = blockIdx.y, E = a.E, tid = threadIdx.x;
    const int q = tid % kSumQuads, part = tid / kSumQuads, e0 = blockIdx.x * kSumExperts + q * 4;
    const int64_t u0 = (int64_t)s * blocks;
    if (tid < kWave) {
        int v = 0;
        for (int b = tid; b < blocks; b += kWave) v += a.part_seen[u0 + b];
#pragma unroll
        for (int d = 32; d; d >>= 1) v += shfl(v, tid ^ d);
        if (tid == 0) seen = v;
    }
    double p[4] = {0.0, 0.0, 0.0, 0.0};
    i32x4 c = {0, 0, 0, 0};
    if (e0 < a.pitch)
        for (int b0 = part; b0 < blocks; b0 += kSumParts * G) {
            f32x4 pv[G];
            i32x4 cv[G];
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const int64_t at = (u0 + min(b0 + g * kSumParts, blocks - 1)) * a.pitch + e0;
                pv[g] = *reinterpret_cast<const f32x4 *>(a.part_p + at);
                cv[g] = *reinterpret_cast<const i32x4 *>(a.part_cnt + at);
            }
#pragma unroll
            for (int g = 0; g < G; ++g) {
                if (b0 + g * kSumParts >= blocks) continue;
                c += cv[g];
#pragma unroll
                for (int j = 0; j < 4; ++j) p[j] += (double)pv[g][j];
            }
        }
#pragma unroll
    for (int j = 0; j < 4; ++j) lp[part][q * 4 + j] = p[j], lc[part][q * 4 + j] = c[j];
    __syncthreads();
    if (tid < kWave) {
        const int e = blockIdx.x * kSumExperts + tid;
        double term = 0.0;
        if (tid < kSumExperts && e < E) {
            double all = 0.0;
            int count = 0;
#pragma unroll 8
            for (int o = 0; o < kSumParts; ++o) all += lp[o][tid], count += lc[o][tid];
            a.tokens_per_expert[(int64_t)s * E + e] = count;
            const double v = seen > 0 ? (double)seen : 1.0;
            term = (double)count * E / (a.K * v) * (all / v);
        }
        // A fixed order: halves of the lanes.
#pragma unroll
        for (int d = 32; d; d >>= 1)
            term += __hiloint2double(shfl(__double2hiint(term), tid ^ d), shfl(__double2loint(term), tid ^ d));
        if (tid == 0) {
            __hip_atomic_store(&a.part_loss[(int64_t)s * gridDim.x + blockIdx.x], term, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            last = __hip_atomic_fetch_add(&a.part_done[s], 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == (int)gridDim.x - 1;
            if (last) {
                double sum = 0.0;
                for (int b = 0; b < (int)gridDim.x; ++b)
                    sum += __hip_atomic_load(&a.part_loss[(int64_t)s * gridDim.x + b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                a.balance_loss[s] = (float)sum;
                a.tokens_valid[s] = seen;
            }
        }
    }
}

// Gradient of the logits: with u_e the gradient of s_e,
//   softmax  dl = s (u - sum u s),   sigmoid  dl = u s (1 - s),
// u = the chosen lanes' scale (dw - sum dw s / D) / D, plus the loss's share a_e
// (softmax) or (a_e - sum a p) / (sum s) (sigmoid).
template <typename T, int PER, bool SIG>
__global__ void __launch_bounds__(kThreads) k_route_backward(RouteArgs a) {
    const int lane = lane_id(), wave = threadIdx.x / kWave;
    const int s = blockIdx.y, E = a.E, K = a.K;
    float ae[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) ae[j] = 0.0f;
    if (a.d_loss) {
        const int tv = a.tokens_valid[s];
        const double v = tv > 0 ? (double)tv : 1.0;
        const double f = (double)a.d_loss[s] * E / (a.K * v * v);
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int e = lane * PER + j;
            if (e < E) ae[j] = (float)(f * a.tokens_per_expert[(int64_t)s * E + e]);
        }
    }
    for (int64_t t = (int64_t)blockIdx.x * kWaves + wave; t < a.T; t += (int64_t)gridDim.x * kWaves) {
        const int64_t g = (int64_t)s * a.T + t;
        const bool open = !a.token_mask || a.token_mask[g] != 0;
        const T *row = static_cast<const T *>(a.logits) + g * E;
        float l[PER], sc[PER], u[PER];
        load_logits<T, PER>(row, E, lane, open, a.vec, l);
        int idx = -1;
        float dw = 0.0f;
        if (lane < K && a.d_weights) {
            const int64_t i = a.topk_idx[g * K + lane];
            idx = i >= 0 && i < E ? (int)i : -1;
            if (idx >= 0) dw = a.d_weights[g * K + lane];
        }
        const float top = top_of(l);
        const bool any = top > -INFINITY;
        float inv, all;
        scores<PER, SIG>(l, any ? top : 0.0f, sc, inv, all);
#pragma unroll
        for (int j = 0; j < PER; ++j) u[j] = 0.0f;
        if (a.d_weights) {
            // The chosen lanes' scores, from the lanes that hold them.
            float sk = 0.0f;
            for (int k = 0; k < K; ++k) {
                const int e = read_lane(idx, k);
                if (e < 0) continue;
                float mine = 0.0f;
#pragma unroll
                for (int j = 0; j < PER; ++j) mine = lane * PER + j == e ? sc[j] : mine;
                const float v = read_lane_f(mine, e / PER);
                if (lane == k) sk = v;
            }
            const float D = wave_sum(sk) + 1e-20f;
            const float dot = wave_sum(dw * (sk / D));
            const float dk = idx >= 0 ? a.scale * (dw - dot) / D : 0.0f;
            for (int k = 0; k < K; ++k) {
                const int e = read_lane(idx, k);
                if (e < 0) continue;
                const float v = read_lane_f(dk, k);
#pragma unroll
                for (int j = 0; j < PER; ++j) u[j] = lane * PER + j == e ? v : u[j];
            }
        }
        if (SIG) {
            const float r = 1.0f / (all + 1e-20f);
            float dot = 0.0f;
#pragma unroll
            for (int j = 0; j < PER; ++j) dot += ae[j] * (sc[j] * r);
            dot = wave_sum(dot);
#pragma unroll
            for (int j = 0; j < PER; ++j) u[j] = (u[j] + (ae[j] - dot) * r) * sc[j] * sigmoid(-l[j]);
        } else {
            float dot = 0.0f;
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                u[j] += ae[j];
                dot += u[j] * sc[j];
            }
            dot = wave_sum(dot);
#pragma unroll
            for (int j = 0; j < PER; ++j) u[j] = sc[j] * (u[j] - dot);
        }
        T *out = static_cast<T *>(a.d_logits) + g * E;
        Pack<T, PER> p;
        const int e0 = lane * PER;
#pragma unroll
        for (int j = 0; j < PER; ++j) narrow(l[j] > -INFINITY ? u[j] : 0.0f, p.v[j]);
        if (a.vec) {
            if (e0 + PER <= E) *reinterpret_cast<Pack<T, PER> *>(out + e0) = p;
        } else {
#pragma unroll
            for (int j = 0; j < PER; ++j)
                if (e0 + j < E) out[e0 + j] = p.v[j];
        }
    }
}

// ---- Many tokens: several per wave ----
//
// With a token per wave the rounds of the choice are bound by issuing 70
// instructions per token and round for one maximum; with L = 16 (E <= 256) or 32
// lanes per token, one maximum inside a row of lanes serves four or two tokens.
// Keys are whole numbers of the same order as the floats, their low bits
// replaced by the expert (lowest first), so that keys differ and a round is a
// maximum, a comparison and the owner's removal.  Where neighbours among the
// K + 1 best agree in the bits that are left (with a bias: the last two do, or
// two lie closer than their rounding tells apart, the K-th and the end of the next
// bin included), the choice is made again from whole keys, in 64 bits with a bias.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_bits(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false);
}
constexpr int kRor1 = 0x121, kRor2 = 0x122, kRor4 = 0x124, kRor8 = 0x128;  // rotate a row of 16 lanes

// The group's result in each of its lanes.
template <int L, typename F>
__device__ __forceinline__ uint32_t group_fold(uint32_t v, F f) {
    v = f(v, dpp_bits<kRor8>(v));
    v = f(v, dpp_bits<kRor4>(v));
    v = f(v, dpp_bits<kRor2>(v));
    v = f(v, dpp_bits<kRor1>(v));
    if (L == 32) v = f(v, (uint32_t)shfl((int)v, lane_id() ^ 16));
    return v;
}
template <int L>
__device__ __forceinline__ uint32_t group_max_bits(uint32_t v) {
    return group_fold<L>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
template <int L>
__device__ __forceinline__ int group_min_int(int v) {
    return (int)group_fold<L>((uint32_t)v, [](uint32_t a, uint32_t b) { return (int)a < (int)b ? a : b; });
}
template <int L>
__device__ __forceinline__ float group_max(float v) {
    return __uint_as_float(group_fold<L>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
        return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    }));
}
template <int L>
__device__ __forceinline__ float group_sum(float v) {
    return __uint_as_float(group_fold<L>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }));
}
template <int L>
__device__ __forceinline__ double group_max(double v) {
#pragma unroll
    for (int d = L / 2; d; d >>= 1) {
        const int from = lane_id() ^ d;
        v = fmax(v, __hiloint2double(shfl(__double2hiint(v), from), shfl(__double2loint(v), from)));
    }
    return v;
}
template <int L>
__device__ __forceinline__ double group_sum(double v) {
#pragma unroll
    for (int d = L / 2; d; d >>= 1) {
        const int from = lane_id() ^ d;
        v += __hiloint2double(shfl(__double2hiint(v), from), shfl(__double2loint(v), from));
    }
    return v;
}

__device__ __forceinline__ float fast_sigmoid(float l) {
    const float m = fabsf(l), v = exp_of(-m, 0.0f), z = m < 110.0f ? v : 0.0f;
    return (l >= 0.0f ? 1.0f : z) * __builtin_amdgcn_rcpf(1.0f + z);
}

// One logit as the router takes it: masked ones -inf, +inf the largest value.
template <typename T>
__device__ __forceinline__ float take(T raw, float lo, bool open) {
    const float v = widen(raw);
    return open && v > lo ? fminf(v, -lo) : -INFINITY;
}

template <typename T, int PER>
__device__ __forceinline__ void load_row(const T *row, int e0, int E, bool open, bool vec, float (&l)[PER]) {
    const float lo = lowest(row);
    typedef T quad __attribute__((ext_vector_type(4)));
    if (vec) {
        quad p[PER / 4];
#pragma unroll
        for (int c = 0; c < PER / 4; ++c)
            p[c] = e0 + 4 * c < E ? *reinterpret_cast<const quad *>(row + e0 + 4 * c) : quad{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < PER; ++j) l[j] = take<T>(p[j / 4][j % 4], lo, open && e0 + j / 4 * 4 < E);
    } else {
#pragma unroll
        for (int j = 0; j < PER; ++j) l[j] = e0 + j < E ? take<T>(row[e0 + j], lo, open) : -INFINITY;
    }
}

// K rounds of "largest key, lowest index" on whole keys.
template <int L, int PER, typename Key>
__device__ __forceinline__ int choose_exact(Key (&key)[PER], int K, int li) {
    int idx = -1;
    for (int k = 0; k < K; ++k) {
        Key best = key[0];
#pragma unroll
        for (int j = 1; j < PER; ++j) best = key[j] > best ? key[j] : best;
        const Key top = group_max<L>(best);
        int at = 1 << 20;
#pragma unroll
        for (int j = PER - 1; j >= 0; --j)
            if (key[j] == top) at = li * PER + j;
        const int e = group_min_int<L>(at);
        const bool some = top > (Key)-INFINITY;
        if (li == k) idx = some ? e : -1;
#pragma unroll
        for (int j = 0; j < PER; ++j)
            if (li * PER + j == e) key[j] = (Key)-INFINITY;
    }
    return idx;
}

// Scores from logits, the group's sum of them (softmax: already divided out).
template <int L, int PER, bool SIG>
__device__ __forceinline__ void group_scores(const float (&l)[PER], float top, float (&s)[PER], float &inv, float &all) {
    float t = 0.0f;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        s[j] = SIG ? fast_sigmoid(l[j]) : exp_below(l[j], top);
        t += s[j];
    }
    all = group_sum<L>(t);
    inv = 1.0f;
    if (!SIG) {
        inv = 1.0f / fmaxf(all, 1e-30f);
#pragma unroll
        for (int j = 0; j < PER; ++j) s[j] *= inv;
    }
}

template <typename T, int L, int PER, bool SIG, bool BAL>
__global__ void __launch_bounds__(kThreads) k_route_rows(RouteArgs a) {
    constexpr int G = kWave / L, kLow = L == 16 ? 255 : 511, kAll = L * PER;
    __shared__ int hist[BAL ? kAll : 1];
    __shared__ float lp[BAL ? kWaves : 1][BAL ? kAll : 1];
    __shared__ int ls[kWaves];
    const int lane = lane_id(), wave = threadIdx.x / kWave, li = lane % L, e0 = li * PER;
    const int s = blockIdx.y, E = a.E, K = a.K;
    double psum[PER];  // as in k_route
    int seen = 0;
    if (BAL) {
#pragma unroll
        for (int j = 0; j < PER; ++j) psum[j] = 0.0;
        for (int e = threadIdx.x; e < kAll; e += kThreads) hist[e] = 0;
        if (blockIdx.x == 0 && threadIdx.x == 0) a.part_done[s] = 0;  // for k_route_sum
        __syncthreads();
    }
    for (int64_t t0 = ((int64_t)blockIdx.x * kWaves + wave) * G; t0 < a.T; t0 += (int64_t)gridDim.x * kWaves * G) {
        const bool live = t0 + lane / L < a.T;
        const int64_t g = (int64_t)s * a.T + (live ? t0 + lane / L : t0);
        const bool open = live && (!a.token_mask || a.token_mask[g] != 0);
        const T *row = static_cast<const T *>(a.logits) + g * E;
        float l[PER], sc[PER];
        load_row<T, PER>(row, e0, E, open, a.vec, l);
        float m = l[0];
#pragma unroll
        for (int j = 1; j < PER; ++j) m = fmaxf(m, l[j]);
        m = group_max<L>(m);
        const bool any = m > -INFINITY;
        const float top = any ? m : 0.0f;
        float inv = 1.0f, all = 0.0f;
        if (BAL || a.bias) group_scores<L, PER, SIG>(l, top, sc, inv, all);
        uint32_t key[PER];
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            float v = l[j];
            if (a.bias) {
                const float b = e0 + j < E ? a.bias[e0 + j] : 0.0f;
                v = v > -INFINITY && b == b ? sc[j] + b : -INFINITY;
            }
            const uint32_t u = __float_as_uint(v + 0.0f);  // -0 is +0: they tie, and their bits would not
            const uint32_t up = u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
            key[j] = v > -INFINITY ? (up & ~(uint32_t)kLow) | (uint32_t)(kLow - (e0 + j)) : 0u;
        }
        int idx = -1;
        bool again = false;
        uint32_t prev = 0u;
        for (int k = 0;; ++k) {
            uint32_t best = key[0];
#pragma unroll
            for (int j = 1; j < PER; ++j) best = best > key[j] ? best : key[j];
            const uint32_t first = group_max_bits<L>(best);
            if (k > 0 && first != 0u && (!a.bias || k == K)) again |= ((prev ^ first) & ~(uint32_t)kLow) == 0u;
            prev = first;
            if (li == k) idx = first != 0u ? kLow - (int)(first & kLow) : -1;
            if (k == K) break;
#pragma unroll
            for (int j = 0; j < PER; ++j) key[j] = key[j] == first ? 0u : key[j];
        }
        // Without a bias the best is among the chosen, so softmax weights need no
        // division by the whole sum (and are the same with or without the loss).
        const float by = a.bias ? inv : 1.0f;
        float lk = idx >= 0 ? take<T>(row[idx], lowest(row), true) : 0.0f;
        float sk = idx < 0 ? 0.0f : (SIG ? fast_sigmoid(lk) : exp_below(lk, top) * by);
        if (a.bias) {
            // Past the K-th the order inside a bin is not known: the end of the
            // (K+1)-th's bin bounds every key that was not chosen.
            const uint32_t end = prev | (uint32_t)kLow;
            float mine = idx >= 0 ? sk + a.bias[idx] : -INFINITY;
            if (li == K && idx >= 0) mine = __uint_as_float(end ^ (end >> 31 ? 0x80000000u : 0xffffffffu));
            const float next = __int_as_float(shfl(__float_as_int(mine), lane + 1));
            const float unit = fmaxf(1.0f, fmaxf(fabsf(mine), fabsf(next)));
            again |= li < K && next > -INFINITY && !(mine - next > kKeyError * unit);
        }
        // bf16 logits lie in the bits that are left: equal ones are equal.
        if (sizeof(T) == 2 && !a.bias) again = false;
        if (ballot(again)) {
            if (!a.bias) {
                float kf[PER];
#pragma unroll
                for (int j = 0; j < PER; ++j) kf[j] = l[j];
                idx = choose_exact<L>(kf, K, li);
            } else {
                double kd[PER], sum = 0.0;
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    kd[j] = SIG ? sigmoid((double)l[j]) : exp((double)l[j] - (double)top);
                    sum += kd[j];
                }
                if (!SIG) sum = group_sum<L>(sum);
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    const float b = e0 + j < E ? a.bias[e0 + j] : 0.0f;
                    const double v = (SIG ? kd[j] : kd[j] / sum) + (double)b;
                    kd[j] = l[j] > -INFINITY && b == b ? v : -(double)INFINITY;
                }
                idx = choose_exact<L>(kd, K, li);
            }
            lk = idx >= 0 ? take<T>(row[idx], lowest(row), true) : 0.0f;
            sk = idx < 0 ? 0.0f : (SIG ? fast_sigmoid(lk) : exp_below(lk, top) * by);
        }
        if (li >= K) idx = -1, sk = 0.0f;  // the first that was not chosen
        const float D = group_sum<L>(sk) + 1e-20f;
        if (live && li < K) {
            a.topk_idx[g * K + li] = idx;
            a.topk_weights[g * K + li] = a.scale * (sk / D);
        }
        if (BAL) {
            if (idx >= 0) atomicAdd(&hist[idx], 1);
            seen += any && li == 0;
            const float r = !any ? 0.0f : (SIG ? 1.0f / (all + 1e-20f) : 1.0f);
#pragma unroll
            for (int j = 0; j < PER; ++j) psum[j] += (double)(sc[j] * r);
        }
    }
    if (BAL) {
        // The workgroup's sums in order: over a wave's groups, then the waves.
#pragma unroll
        for (int d = L; d < kWave; d <<= 1) {
#pragma unroll
            for (int j = 0; j < PER; ++j)
                psum[j] += __hiloint2double(shfl(__double2hiint(psum[j]), lane ^ d), shfl(__double2loint(psum[j]), lane ^ d));
        }
#pragma unroll
        for (int d = 32; d; d >>= 1) seen += shfl(seen, lane ^ d);
        if (lane < L) {
#pragma unroll
            for (int j = 0; j < PER; ++j) lp[wave][e0 + j] = (float)psum[j];
        }
        if (lane == 0) ls[wave] = seen;
        __syncthreads();
        const int64_t unit = (int64_t)s * gridDim.x + blockIdx.x;
        for (int e = threadIdx.x; e < a.pitch; e += kThreads) {
            double p = 0.0;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) p += (double)lp[w][e];
            a.part_p[unit * a.pitch + e] = (float)p;
            a.part_cnt[unit * a.pitch + e] = hist[e];
        }
        if (threadIdx.x == 0) a.part_seen[unit] = ls[0] + ls[1] + ls[2] + ls[3];
    }
}

// The gradient (see k_route_backward) for several tokens per wave; the chosen
// lanes' gradients reach their experts' lanes through LDS.
template <typename T, int L, int PER, bool SIG>
__global__ void __launch_bounds__(kThreads) k_route_rows_backward(RouteArgs a) {
    constexpr int G = kWave / L, kAll = L * PER;
    __shared__ __align__(16) float lu[kWaves][G][kAll];
    const int lane = lane_id(), wave = threadIdx.x / kWave, li = lane % L, e0 = li * PER;
    const int s = blockIdx.y, E = a.E, K = a.K;
    float *mine = lu[wave][lane / L];
    float ae[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) ae[j] = 0.0f;
    if (a.d_loss) {
        const int tv = a.tokens_valid[s];
        const double v = tv > 0 ? (double)tv : 1.0;
        const double f = (double)a.d_loss[s] * E / (a.K * v * v);
#pragma unroll
        for (int j = 0; j < PER; ++j)
            if (e0 + j < E) ae[j] = (float)(f * a.tokens_per_expert[(int64_t)s * E + e0 + j]);
    }
    for (int64_t t0 = ((int64_t)blockIdx.x * kWaves + wave) * G; t0 < a.T; t0 += (int64_t)gridDim.x * kWaves * G) {
        const bool live = t0 + lane / L < a.T;
        const int64_t g = (int64_t)s * a.T + (live ? t0 + lane / L : t0);
        const bool open = !a.token_mask || a.token_mask[g] != 0;
        const T *row = static_cast<const T *>(a.logits) + g * E;
        int idx = -1;
        float dw = 0.0f;
        T raw = 0;
        if (li < K && a.d_weights) {
            const int64_t i = a.topk_idx[g * K + li];
            idx = i >= 0 && i < E ? (int)i : -1;
            if (idx >= 0) dw = a.d_weights[g * K + li], raw = row[idx];
        }
        float l[PER], sc[PER], u[PER];
        load_row<T, PER>(row, e0, E, open, a.vec, l);
        float m = l[0];
#pragma unroll
        for (int j = 1; j < PER; ++j) m = fmaxf(m, l[j]);
        m = group_max<L>(m);
        const float top = m > -INFINITY ? m : 0.0f;
        float inv, all;
        group_scores<L, PER, SIG>(l, top, sc, inv, all);
#pragma unroll
        for (int j = 0; j < PER; ++j) u[j] = 0.0f;
        if (a.d_weights) {
            const float lk = take<T>(raw, lowest(row), open && idx >= 0);
            const float sk = idx < 0 ? 0.0f : (SIG ? fast_sigmoid(lk) : exp_below(lk, top) * inv);
            const float D = group_sum<L>(sk) + 1e-20f;
            const float dot = group_sum<L>(dw * (sk / D));
#pragma unroll
            for (int j = 0; j < PER; j += 4) *reinterpret_cast<f32x4 *>(mine + e0 + j) = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            __builtin_amdgcn_wave_barrier();
            if (idx >= 0) mine[idx] = a.scale * (dw - dot) / D;
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int j = 0; j < PER; j += 4) {
                const f32x4 v = *reinterpret_cast<const f32x4 *>(mine + e0 + j);
#pragma unroll
                for (int i = 0; i < 4; ++i) u[j + i] = v[i];
            }
            __builtin_amdgcn_wave_barrier();
        }
        float dot = 0.0f;
        if (SIG) {
            const float r = 1.0f / (all + 1e-20f);
#pragma unroll
            for (int j = 0; j < PER; ++j) dot += ae[j] * (sc[j] * r);
            dot = group_sum<L>(dot);
#pragma unroll
            for (int j = 0; j < PER; ++j) u[j] = (u[j] + (ae[j] - dot) * r) * sc[j] * fast_sigmoid(-l[j]);
        } else {
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                u[j] += ae[j];
                dot += u[j] * sc[j];
            }
            dot = group_sum<L>(dot);
#pragma unroll
            for (int j = 0; j < PER; ++j) u[j] = sc[j] * (u[j] - dot);
        }
        if (!live) continue;
        T *out = static_cast<T *>(a.d_logits) + g * E;
        typedef T quad __attribute__((ext_vector_type(4)));
        T o[PER];
#pragma unroll
        for (int j = 0; j < PER; ++j) narrow(l[j] > -INFINITY ? u[j] : 0.0f, o[j]);
        if (a.vec) {
#pragma unroll
            for (int j = 0; j < PER; j += 4)
                if (e0 + j < E) *reinterpret_cast<quad *>(out + e0 + j) = quad{o[j], o[j + 1], o[j + 2], o[j + 3]};
        } else {
#pragma unroll
            for (int j = 0; j < PER; ++j)
                if (e0 + j < E) out[e0 + j] = o[j];
        }
    }
}

bool few_tokens(int S, int T) { return (int64_t)S * T <= kFewTokens; }

int per_lane(int E) {
    int per = 1;
    while (per * kWave < E) per *= 2;
    return per;
}

template <typename T, int PER, bool SIG>
hipError_t run(const RouteArgs &a, bool backward, int blocks, hipStream_t st) {
    const dim3 grid(blocks, a.S);
    constexpr int L = large_waves(PER);
    if (backward) hipLaunchKernelGGL((k_route_backward<T, PER, SIG>), grid, dim3(kThreads), 0, st, a);
    else if (!a.part_p) hipLaunchKernelGGL((k_route<T, PER, SIG, false, kWaves>), grid, dim3(kThreads), 0, st, a);
    else if (few_tokens(a.S, a.T)) hipLaunchKernelGGL((k_route<T, PER, SIG, true, kWaves>), grid, dim3(kThreads), 0, st, a);
    else hipLaunchKernelGGL((k_route<T, PER, SIG, true, L>), grid, dim3(kWave * L), 0, st, a);
    return hipGetLastError();
}

template <typename T, int PER>
hipError_t run(const RouteArgs &a, bool backward, int blocks, hipStream_t st) {
    return a.sigmoid ? run<T, PER, true>(a, backward, blocks, st) : run<T, PER, false>(a, backward, blocks, st);
}

template <typename T>
hipError_t run(RouteArgs a, bool backward, int blocks, hipStream_t st) {
    const int per = per_lane(a.E);
    const uintptr_t ends = reinterpret_cast<uintptr_t>(a.logits) | (backward ? reinterpret_cast<uintptr_t>(a.d_logits) : 0);
    a.vec = a.E % per == 0 && ends % alignof(Pack<T, 16>) == 0;
    switch (per) {
        case 1: return run<T, 1>(a, backward, blocks, st);
        case 2: return run<T, 2>(a, backward, blocks, st);
        case 4: return run<T, 4>(a, backward, blocks, st);
        case 8: return run<T, 8>(a, backward, blocks, st);
        default: return run<T, 16>(a, backward, blocks, st);
    }
}

template <typename T, int L, int PER, bool SIG>
hipError_t run_rows(const RouteArgs &a, bool backward, int blocks, hipStream_t st) {
    const dim3 grid(blocks, a.S);
    if (backward) hipLaunchKernelGGL((k_route_rows_backward<T, L, PER, SIG>), grid, dim3(kThreads), 0, st, a);
    else if (a.part_p) hipLaunchKernelGGL((k_route_rows<T, L, PER, SIG, true>), grid, dim3(kThreads), 0, st, a);
    else hipLaunchKernelGGL((k_route_rows<T, L, PER, SIG, false>), grid, dim3(kThreads), 0, st, a);
    return hipGetLastError();
}

template <typename T, int L, int PER>
hipError_t run_rows(const RouteArgs &a, bool backward, int blocks, hipStream_t st) {
    return a.sigmoid ? run_rows<T, L, PER, true>(a, backward, blocks, st)
                     : run_rows<T, L, PER, false>(a, backward, blocks, st);
}

template <typename T>
hipError_t run_rows(RouteArgs a, bool backward, int blocks, hipStream_t st) {
    const uintptr_t ends = reinterpret_cast<uintptr_t>(a.logits) | (backward ? reinterpret_cast<uintptr_t>(a.d_logits) : 0);
    a.vec = a.E % 4 == 0 && ends % (4 * sizeof(T)) == 0;
    if (a.E <= 64) return run_rows<T, 16, 4>(a, backward, blocks, st);
    if (a.E <= 128) return run_rows<T, 16, 8>(a, backward, blocks, st);
    if (a.E <= 192) return run_rows<T, 16, 12>(a, backward, blocks, st);
    if (a.E <= 256) return run_rows<T, 16, 16>(a, backward, blocks, st);
    if (a.E <= 384) return run_rows<T, 32, 12>(a, backward, blocks, st);
    return run_rows<T, 32, 16>(a, backward, blocks, st);
}

// Several tokens per wave: from kManyTokens on, where there are waves enough
// for the card either way (256 experts, top-8, forward: 4096 tokens 6.8 us with
// a token per wave, 8.5 with four; 8192 10.5 and 9.2; 32768 35 and 19), and
// sooner with few experts, which leave a wave's lanes with one each (64 experts,
// 6555 tokens, top-11 with a bias: 13.4 us).
bool many_tokens(int S, int T, int E, int K) {
    return (int64_t)S * T >= (E <= 64 ? kManyTokens / 4 : kManyTokens) && E <= 512 && K < (E <= 256 ? 16 : 32);
}

}  // namespace

// Blocks per source: a wave for every token until there are `most` blocks in
// all, then a loop over tokens.
int blocks_for(int S, int T, int waves, int most) {
    const int want = (int)(((int64_t)T + waves - 1) / waves);
    most = most / S > 1 ? most / S : 1;
    return want < 1 ? 1 : (want < most ? want : most);
}

// Blocks of the forward pass with the balance loss, per source: few, for their
// partial sums are to be added.
int route_blocks(int S, int T, int E, int K) {
    if (many_tokens(S, T, E, K)) return blocks_for(S, T, kWaves * (E <= 256 ? 4 : 2), 512);
    return blocks_for(S, T, few_tokens(S, T) ? kWaves : large_waves(per_lane(E)), 256);
}
int route_sum_blocks(int E) { return (E + kSumExperts - 1) / kSumExperts; }

hipError_t launch_route(const RouteArgs &a, hipStream_t st) {
    if (a.T == 0 && !a.part_p) return hipSuccess;
    const bool many = many_tokens(a.S, a.T, a.E, a.K);
    const int waves = many ? kWaves * (a.E <= 256 ? 4 : 2) : kWaves;
    const int blocks = a.part_p ? route_blocks(a.S, a.T, a.E, a.K) : blocks_for(a.S, a.T, waves, 2048);
    hipError_t rc;
    if (many) rc = a.logits_bf16 ? run_rows<uint16_t>(a, false, blocks, st) : run_rows<float>(a, false, blocks, st);
    else rc = a.logits_bf16 ? run<uint16_t>(a, false, blocks, st) : run<float>(a, false, blocks, st);
    if (rc != hipSuccess || !a.part_p) return rc;
    hipLaunchKernelGGL(k_route_sum, dim3(route_sum_blocks(a.E), a.S), dim3(kSumThreads), 0, st, a, blocks);
    return hipGetLastError();
}

hipError_t launch_route_backward(const RouteArgs &a, hipStream_t st) {
    if (a.T == 0) return hipSuccess;
    if (many_tokens(a.S, a.T, a.E, a.K)) {
        const int blocks = blocks_for(a.S, a.T, kWaves * (a.E <= 256 ? 4 : 2), 2048);
        return a.logits_bf16 ? run_rows<uint16_t>(a, true, blocks, st) : run_rows<float>(a, true, blocks, st);
    }
    const int blocks = blocks_for(a.S, a.T, kWaves, 2048);
    return a.logits_bf16 ? run<uint16_t>(a, true, blocks, st) : run<float>(a, true, blocks, st);
}

}  // namespace ep
