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
// Waves of a forward workgroup.  With the balance loss each workgroup leaves one
// partial sum per expert for a single workgroup to add, so there are few, large
// ones (as much as their LDS allows).
constexpr int route_waves(int per, bool balance) { return balance ? (per > 8 ? 8 : 16) : kWaves; }

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

// 1 / (1 + exp(-l)) without overflow on either side; 0 for -inf.
__device__ __forceinline__ float sigmoid(float l) {
    const float z = expf(-fabsf(l));
    return (l >= 0.0f ? 1.0f : z) / (1.0f + z);
}
__device__ __forceinline__ double sigmoid(double l) {
    const double z = exp(-fabs(l));
    return (l >= 0.0 ? 1.0 : z) / (1.0 + z);
}

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
            // A key s + bias in 32 bits is within 5e-7 * max(1, |key|) of its
            // value (s to 3 * 2^-24, the sum's rounding 2^-24 relative).
            const Key a = top < 0 ? -top : top, b = prev < 0 ? -prev : prev;
            const Key unit = a > b ? (a > 1 ? a : (Key)1) : (b > 1 ? b : (Key)1);
            if (!(prev - top > (Key)1e-6 * unit)) close = true;
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
    for (int j = 0; j < PER; ++j) s[j] = SIG ? sigmoid(l[j]) : expf(l[j] - top);
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
template <typename T, int PER, bool SIG, bool BAL>
__global__ void __launch_bounds__(kWave *route_waves(PER, BAL)) k_route(RouteArgs a) {
    constexpr int kWaves = route_waves(PER, BAL), kThreads = kWaves * kWave;
    const int lane = lane_id(), wave = threadIdx.x / kWave;
    const int s = blockIdx.y, E = a.E, K = a.K;
    float psum[PER];
    int cnt[PER], seen = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) psum[j] = 0.0f, cnt[j] = 0;
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
        const float sk = chosen ? (SIG ? sigmoid(lsel) : expf(lsel - top) * inv) : 0.0f;
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
                psum[j] += any ? sc[j] * r : 0.0f;
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
            lp[wave][lane * PER + j] = psum[j];
            lc[wave][lane * PER + j] = cnt[j];
        }
        if (lane == 0) ls[wave] = seen;
        __syncthreads();
        const int64_t unit = (int64_t)s * gridDim.x + blockIdx.x;
        for (int e = threadIdx.x; e < a.pitch; e += kThreads) {
            float p = 0.0f;
            int c = 0;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) p += lp[w][e], c += lc[w][e];
            a.part_p[unit * a.pitch + e] = p;
            a.part_cnt[unit * a.pitch + e] = c;
        }
        if (threadIdx.x == 0) {
            int n = 0;
            for (int w = 0; w < kWaves; ++w) n += ls[w];
            a.part_seen[unit] = n;
        }
    }
}

// Counts, valid tokens and the loss of source blockIdx.x from the blocks'
// partial sums.  Thread (quad, part) adds every parts-th block of four
// neighbouring experts in order, eight blocks' loads in flight: one workgroup
// reads it all, and only loads in flight hide the latency (one at a time: 74 us
// instead of 6 at 1024 partial sums of 256 experts).  Sums over tokens and
// experts are held in 64 bits.
constexpr int kSumThreads = 1024;
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
__global__ void __launch_bounds__(kSumThreads) k_route_sum(RouteArgs a, int blocks, int parts) {
    __shared__ double lp[kSumThreads][4];
    __shared__ i32x4 lc[kSumThreads];
    __shared__ int seen;
    constexpr int G = 8;
    const int s = blockIdx.x, E = a.E, tid = threadIdx.x, quads = a.pitch / 4;
    const int q = tid % quads, part = tid / quads;
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
    if (part < parts)
        for (int b0 = part; b0 < blocks; b0 += parts * G) {
            f32x4 pv[G];
            i32x4 cv[G];
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const int64_t at = (u0 + min(b0 + g * parts, blocks - 1)) * a.pitch + 4 * q;
                pv[g] = *reinterpret_cast<const f32x4 *>(a.part_p + at);
                cv[g] = *reinterpret_cast<const i32x4 *>(a.part_cnt + at);
            }
#pragma unroll
            for (int g = 0; g < G; ++g) {
                if (b0 + g * parts >= blocks) continue;
                c += cv[g];
#pragma unroll
                for (int j = 0; j < 4; ++j) p[j] += (double)pv[g][j];
            }
        }
#pragma unroll
    for (int j = 0; j < 4; ++j) lp[tid][j] = p[j];
    lc[tid] = c;
    __syncthreads();
    double term = 0.0;
    if (part == 0) {
        for (int o = 1; o < parts; ++o) {
            c += lc[tid + o * quads];
#pragma unroll
            for (int j = 0; j < 4; ++j) p[j] += lp[tid + o * quads][j];
        }
        const double v = seen > 0 ? (double)seen : 1.0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (4 * q + j < E) {
                a.tokens_per_expert[(int64_t)s * E + 4 * q + j] = c[j];
                term += (double)c[j] * E / (a.K * v) * (p[j] / v);
            }
    }
    // The terms' sum in a fixed order: inside the waves, then over them.
#pragma unroll
    for (int d = 32; d; d >>= 1)
        term += __hiloint2double(shfl(__double2hiint(term), lane_id() ^ d), shfl(__double2loint(term), lane_id() ^ d));
    __syncthreads();
    if (tid % kWave == 0) lp[tid / kWave][0] = term;
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < kSumThreads / kWave; ++w) term += lp[w][0];
        a.balance_loss[s] = (float)term;
        a.tokens_valid[s] = seen;
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

int per_lane(int E) {
    int per = 1;
    while (per * kWave < E) per *= 2;
    return per;
}

template <typename T, int PER, bool SIG>
hipError_t run(const RouteArgs &a, bool backward, int blocks, hipStream_t st) {
    const dim3 grid(blocks, a.S);
    const dim3 threads(kWave * route_waves(PER, !backward && a.part_p));
    if (backward) hipLaunchKernelGGL((k_route_backward<T, PER, SIG>), grid, dim3(kThreads), 0, st, a);
    else if (a.part_p) hipLaunchKernelGGL((k_route<T, PER, SIG, true>), grid, threads, 0, st, a);
    else hipLaunchKernelGGL((k_route<T, PER, SIG, false>), grid, threads, 0, st, a);
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

}  // namespace

// Blocks per source: a wave for every token until there are `most` blocks in
// all, then a loop over tokens.
int blocks_for(int S, int T, int waves, int most) {
    const int want = (int)(((int64_t)T + waves - 1) / waves);
    most = most / S > 1 ? most / S : 1;
    return want < 1 ? 1 : (want < most ? want : most);
}

// Blocks of the forward pass with the balance loss, per source: at most one for
// every CU in all.
int route_blocks(int S, int T, int E) { return blocks_for(S, T, route_waves(per_lane(E), true), 256); }

hipError_t launch_route(const RouteArgs &a, hipStream_t st) {
    if (a.T == 0 && !a.part_p) return hipSuccess;
    const int blocks = a.part_p ? route_blocks(a.S, a.T, a.E) : blocks_for(a.S, a.T, kWaves, 2048);
    hipError_t rc = a.logits_bf16 ? run<uint16_t>(a, false, blocks, st) : run<float>(a, false, blocks, st);
    if (rc != hipSuccess || !a.part_p) return rc;
    int parts = kSumThreads / (a.pitch / 4);
    parts = parts < blocks ? parts : blocks;
    hipLaunchKernelGGL(k_route_sum, dim3(a.S), dim3(kSumThreads), 0, st, a, blocks, parts);
    return hipGetLastError();
}

hipError_t launch_route_backward(const RouteArgs &a, hipStream_t st) {
    if (a.T == 0) return hipSuccess;
    const int blocks = blocks_for(a.S, a.T, kWaves, 2048);
    return a.logits_bf16 ? run<uint16_t>(a, true, blocks, st) : run<float>(a, true, blocks, st);
}

}  // namespace ep
