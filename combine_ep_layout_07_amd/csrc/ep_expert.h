// ep_expert.h -- arguments and device helpers of the experts' products.
#pragma once

#include "ep_wave.h"

namespace ep {

enum { kActNone = 0, kActRelu = 1, kActGelu = 2, kActSilu = 3, kActSwiglu = 4 };

// Rows of a tile of the activation's backward pass (each leaves one partial sum
// per column for d_bias).
constexpr int kActRows = 16;

// Tiles of `size` rows that E segments of `rows` rows in all can make, at most.
inline int64_t expert_row_tiles(int64_t rows, int E, int size) { return rows / size + (rows < E ? rows : E); }

struct ExpertArgs {
    int E, I, N, Nw;  // Nw = weight rows per expert: 2N for swiglu, else N
    int act, fp8;
    int64_t rows;
    const int32_t *base;  // [E+1]
    const void *x, *w;
    const float *x_sf, *w_sf;  // fp8: [rows][I/128], [E][ceil(Nw/128)][I/128]
    const float *bias;         // [E][Nw] or null
    const uint16_t *residual;  // [rows][N] or null
    uint16_t *out;             // [rows][N]
    uint16_t *pre;             // [rows][Nw] or null; backward: read
    const uint16_t *d_out;     // backward [rows][N]
    uint16_t *d;               // scratch [rows][Nw]: gradient of the pre-activation (d_out itself without one)
    float *part;               // scratch [part_tiles][Nw]
    int64_t part_tiles;
    uint16_t *d_x, *d_w;       // either may be null
    float *d_bias;             // or null
};

struct Segment {
    int e;       // -1: none
    int64_t r0;  // first row
    int n;       // rows
};

// Rows of expert e, inside [0, rows] whatever the table holds.
__device__ __forceinline__ Segment segment_of(const int32_t *base, int e, int64_t rows) {
    const int64_t lo = base[e], hi = base[e + 1];
    const int64_t a = lo < 0 ? 0 : (lo < rows ? lo : rows);
    const int64_t b = hi < a ? a : (hi < rows ? hi : rows);
    return {e, a, (int)(b - a)};
}

// Inclusive sum over the wave's lanes.
__device__ __forceinline__ int wave_scan(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, kRowShr1, 0xf, 0xf, true);
    v += __builtin_amdgcn_update_dpp(0, v, kRowShr2, 0xf, 0xf, true);
    v += __builtin_amdgcn_update_dpp(0, v, kRowShr4, 0xf, 0xf, true);
    v += __builtin_amdgcn_update_dpp(0, v, kRowShr8, 0xf, 0xf, true);
    v += __builtin_amdgcn_update_dpp(0, v, kRowBcast15, 0xa, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, kRowBcast31, 0xc, 0xf, false);
    return v;
}

// All tiles of `size` rows of the first E experts' segments.  A table that
// decreases can count every row hundreds of times; a grid holds 2^24 workgroups,
// so the lanes' bound changes no count that a launch uses and keeps the sum
// positive.
__device__ __forceinline__ int count_tiles(const int32_t *base, int E, int64_t rows, int size) {
    int n = 0;
    for (int e = lane_id(); e < E; e += kWave) n += (segment_of(base, e, rows).n + size - 1) / size;
    return read_lane(wave_scan(min(n, (1 << 25) - 1)), kWave - 1);
}

// Tile `tile` of `size` rows, counted over the experts in order: a scan over
// the experts by the whole wave, 64 at a time.
__device__ __forceinline__ Segment find_tile(const int32_t *base, int E, int64_t rows, int size, int64_t tile) {
    const int lane = lane_id();
    int64_t before = 0;
    for (int e0 = 0; e0 < E; e0 += kWave) {
        const int e = e0 + lane;
        const Segment g = e < E ? segment_of(base, e, rows) : Segment{e, 0, 0};
        const int mine = (g.n + size - 1) / size;
        const int incl = wave_scan(mine);
        const uint64_t past = ballot(before + incl > tile);
        if (past) {
            const int o = __builtin_ctzll(past);
            const int64_t at = tile - before - (read_lane(incl, o) - read_lane(mine, o));
            const int64_t r0 = (int64_t)read_lane((int)g.r0, o) + at * size;
            const int64_t left = read_lane(g.n, o) - at * size;
            return {e0 + o, r0, (int)(left < size ? left : size)};
        }
        before += read_lane(incl, kWave - 1);
    }
    return {-1, 0, 0};
}

// 1 / (1 + exp(-v)) without overflow on either side, from the hardware's exp2
// and reciprocal: off by a few 2^-24 of 1 (the library's expf and division took
// half of the time of an epilogue).  exp2 returns nothing below the normal
// numbers, so exp(-|v|) is the square of half the exponent's: v times it is
// normal down to -91.
__device__ __forceinline__ float logistic(float v) {
    const float y = __builtin_amdgcn_exp2f(fabsf(v) * -0.72134752f), z = y * y;
    return (v >= 0.0f ? 1.0f : z) * __builtin_amdgcn_rcpf(1.0f + z);
}

// The normal distribution's Phi(v) and exp(-v*v/2).  With t = 1 / (1 + 0.305 |v|)
// the smaller side is exp(-v*v/2) t P(t): P is a least-maximum fit of relative
// error 1e-7 to erfc(|v| / sqrt 2) / (2 t exp(-v*v/2)) for |v| up to 14, so the
// tail keeps its relative accuracy, (1.5 v*v + 24) 2^-24 with the exponential's
// rounding, until it leaves the normal numbers (a fit of absolute error 1.5e-7
// was off by 1% at -8).
__device__ __forceinline__ float normal_cdf(float v, float &bell) {
    const float t = __builtin_amdgcn_rcpf(fmaf(0.305f, fabsf(v), 1.0f));
    bell = __builtin_amdgcn_exp2f(v * v * -0.72134752f);
    float p = fmaf(0.036699183f, t, -0.15298828f);
    p = fmaf(p, t, 0.18571684f);
    p = fmaf(p, t, -0.03797677f);
    p = fmaf(p, t, 0.12102165f);
    p = fmaf(p, t, 0.103420876f);
    p = fmaf(p, t, 0.12246682f);
    p = fmaf(p, t, 0.121639736f);
    const float tail = p * t * bell;
    return v < 0.0f ? tail : 1.0f - tail;
}

// The activations of one argument.
__device__ __forceinline__ float activate(int act, float v) {
    float bell;
    if (act == kActRelu) return v < 0.0f ? 0.0f : v;
    if (act == kActGelu) return v * normal_cdf(v, bell);
    if (act == kActSilu) return v * logistic(v);
    return v;
}
// Their derivatives.
__device__ __forceinline__ float activate_slope(int act, float v) {
    if (act == kActRelu) return v > 0.0f ? 1.0f : 0.0f;
    if (act == kActGelu) {
        float bell;
        const float c = normal_cdf(v, bell);
        return fmaf(v * bell, 0.39894228f, c);
    }
    if (act == kActSilu) {
        const float s = logistic(v);
        return s * (1.0f + v * (1.0f - s));
    }
    return 1.0f;
}

// Rows of the tiles that the products take (0: no such product).
void expert_tiles(const ExpertArgs &a, int *forward, int *d_x, int *d_w);
hipError_t launch_expert(const ExpertArgs &a, hipStream_t st);
hipError_t launch_expert_backward(const ExpertArgs &a, hipStream_t st);

}  // namespace ep
