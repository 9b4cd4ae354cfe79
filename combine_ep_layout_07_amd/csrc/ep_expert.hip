// ep_expert.hip -- the experts' products over rows grouped by expert, with
// bias, activation and residual in the epilogue, and their gradients.
//
// All three products are D = sum over k of Q[., k] P[k, .] with D's contiguous
// dimension on P's side:
//   forward  Q = x,  P = W_e^T  (k = I, both operands contiguous in k)
//   d_x      Q = d,  P = W_e    (k = Nw, P contiguous across k)
//   d_w      Q = d^T, P = x     (k = the expert's rows, both across k)
#include "ep_expert.h"
#include "ep_kernels.h"

namespace ep {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 64, kDepth = 32, kPitch = kDepth + 8;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

enum { kForward = 0, kDx = 1, kDw = 2 };

// e4m3fn to bf16 (exact: 4 bits of mantissa, exponents -9..8).
__device__ __forceinline__ uint32_t e4m3_to_bf16(uint32_t b) {
    const uint32_t sign = (b & 0x80u) << 8, m = b & 0x7fu;
    if (m == 0x7fu) return sign | 0x7fc0u;
    if (m < 8) return sign | (__float_as_uint((float)m * 0.001953125f) >> 16);
    return sign | ((m << 4) + (120u << 7));
}

// Eight operands of 8 neighbouring elements, zeros where `ok` is false.
template <bool FP8>
__device__ __forceinline__ u32x4 load8(const void *p, int64_t i, bool ok) {
    u32x4 v = {0u, 0u, 0u, 0u};
    if (!ok) return v;
    if (!FP8) return *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(p) + i);
    const u32x2 b = *reinterpret_cast<const u32x2 *>(static_cast<const uint8_t *>(p) + i);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint32_t two = b[q / 2] >> (q % 2 * 16);
        v[q] = e4m3_to_bf16(two & 0xffu) | (e4m3_to_bf16((two >> 8) & 0xffu) << 16);
    }
    return v;
}

// One operand tile of kTile x kDepth to LDS rows of k.  ALONG: the operand's
// rows are contiguous in k (row r of `rows` at src + r * pitch); otherwise its
// k-rows are contiguous across (element (r, k) at src + k * pitch + r).
template <bool ALONG, bool FP8>
__device__ __forceinline__ void stage(uint16_t *lds, const void *src, int64_t at, int64_t pitch, int rows, int k0, int k1) {
    const int t = threadIdx.x;
    if (ALONG) {
        const int r = t / 4, k = k0 + t % 4 * 8;
        *reinterpret_cast<u32x4 *>(lds + r * kPitch + t % 4 * 8) = load8<FP8>(src, at + r * pitch + k, r < rows && k < k1);
    } else {
        const int k = t / 8, r = t % 8 * 8;
        const u32x4 v = load8<FP8>(src, at + (k0 + k) * pitch + r, r < rows && k0 + k < k1);
#pragma unroll
        for (int j = 0; j < 8; ++j) lds[(r + j) * kPitch + k] = (uint16_t)(v[j / 2] >> (j % 2 * 16));
    }
}

// Four waves, each 32 x 32 of a 64 x 64 tile.
template <int MODE, bool FP8>
__global__ void __launch_bounds__(kThreads) k_expert_simple(ExpertArgs a, int cols) {
    __shared__ __align__(16) uint16_t lp[kTile * kPitch], lq[kTile * kPitch];
    const int lane = lane_id(), wave = threadIdx.x / kWave;
    const int wp = wave % 2 * 32, wq = wave / 2 * 32;
    const int col = blockIdx.x % cols;
    const bool gated = MODE == kForward && a.act == kActSwiglu;
    Segment g;
    int q0 = 0;
    if (MODE == kDw) {
        const int per = (a.Nw + kTile - 1) / kTile, at = blockIdx.x / cols;
        g = segment_of(a.base, at / per, a.rows);
        q0 = at % per * kTile;
    } else {
        g = find_tile(a.base, a.E, a.rows, kTile, blockIdx.x / cols);
        if (g.e < 0) return;
    }
    const int K = MODE == kForward ? a.I : (MODE == kDx ? a.Nw : g.n);
    const int P = MODE == kForward ? a.N : a.I;  // output columns
    const int p0 = col * (gated ? kTile / 2 : kTile);
    const int np = P - p0 < kTile ? P - p0 : kTile;
    const int nq = MODE == kDw ? (a.Nw - q0 < kTile ? a.Nw - q0 : kTile) : g.n;
    const int64_t we = (int64_t)g.e * a.Nw * a.I;
    f32x4 acc[2][2], part[2][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i / 2][i % 2] = part[i / 2][i % 2] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int k0 = 0; k0 < K; k0 += kDepth) {
        if (MODE == kForward) {
            stage<true, FP8>(lq, a.x, g.r0 * a.I, a.I, nq, k0, K);
            if (gated) {  // 16 gate rows, then their 16 up rows
                const int r = threadIdx.x / 4, n = p0 + r / 32 * 16 + r % 16, k = k0 + threadIdx.x % 4 * 8;
                const int64_t row = n + (r / 16 % 2 ? a.N : 0);
                *reinterpret_cast<u32x4 *>(lp + r * kPitch + threadIdx.x % 4 * 8) =
                    load8<FP8>(a.w, we + row * a.I + k, n < a.N && k < K);
            } else {
                stage<true, FP8>(lp, a.w, we + (int64_t)p0 * a.I, a.I, np, k0, K);
            }
        } else if (MODE == kDx) {
            stage<true, false>(lq, a.d, g.r0 * a.Nw, a.Nw, nq, k0, K);
            stage<false, false>(lp, a.w, we + p0, a.I, np, k0, K);
        } else {
            stage<false, false>(lq, a.d, g.r0 * a.Nw + q0, a.Nw, nq, k0, K);
            stage<false, false>(lp, a.x, g.r0 * a.I + p0, a.I, np, k0, K);
        }
        __syncthreads();
        bf16x8 fp[2], fq[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            fp[i] = *reinterpret_cast<const bf16x8 *>(lp + (wp + i * 16 + lane % 16) * kPitch + lane / 16 * 8);
            fq[i] = *reinterpret_cast<const bf16x8 *>(lq + (wq + i * 16 + lane % 16) * kPitch + lane / 16 * 8);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                f32x4 &c = FP8 ? part[i][j] : acc[i][j];
                c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fp[i], fq[j], c, 0, 0, 0);
            }
        if (FP8 && k0 % 128 == 96) {  // the scales of 128 elements
            const int kb = k0 / 128, nkb = a.I / 128, nb = (a.Nw + 127) / 128;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int q = wq + j * 16 + lane % 16;
                    const float xs = q < nq ? a.x_sf[(g.r0 + q) * nkb + kb] : 0.0f;
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int pl = wp + i * 16 + lane / 16 * 4 + r;
                        const int n = gated ? p0 + pl / 32 * 16 + pl % 16 : p0 + pl;
                        const int row = n + (gated && pl / 16 % 2 ? a.N : 0);
                        const float ws = n < a.N ? a.w_sf[((int64_t)g.e * nb + row / 128) * nkb + kb] : 0.0f;
                        acc[i][j][r] = fmaf(part[i][j][r], xs * ws, acc[i][j][r]);
                        part[i][j][r] = 0.0f;
                    }
                }
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int q = wq + j * 16 + lane % 16, pl = wp + i * 16 + lane / 16 * 4;
            if (q >= nq) continue;
            if (MODE == kForward) {
                const int64_t r = g.r0 + q;
                if (gated && i == 1) continue;
                const int n = gated ? p0 + pl / 32 * 16 + pl % 16 : p0 + pl;
                if (n >= a.N) continue;
                float o[4];
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    float f = acc[i][j][v];
                    if (a.bias) f += a.bias[(int64_t)g.e * a.Nw + n + v];
                    if (a.pre) a.pre[r * a.Nw + n + v] = (uint16_t)to_bf16(f);
                    if (gated) {
                        float u = acc[1][j][v];
                        if (a.bias) u += a.bias[(int64_t)g.e * a.Nw + a.N + n + v];
                        if (a.pre) a.pre[r * a.Nw + a.N + n + v] = (uint16_t)to_bf16(u);
                        f = f * logistic(f) * u;
                    } else {
                        f = activate(a.act, f);
                    }
                    if (a.residual) f += __uint_as_float((uint32_t)a.residual[r * a.N + n + v] << 16);
                    o[v] = f;
                }
                *reinterpret_cast<u32x2 *>(a.out + r * a.N + n) = u32x2{pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3])};
            } else if (pl < np) {
                uint16_t *dst = MODE == kDx ? a.d_x + (g.r0 + q) * a.I : a.d_w + we + (int64_t)(q0 + q) * a.I;
                *reinterpret_cast<u32x2 *>(dst + p0 + pl) =
                    u32x2{pack_bf16(acc[i][j][0], acc[i][j][1]), pack_bf16(acc[i][j][2], acc[i][j][3])};
            }
        }
}

// Gradient of the pre-activation, bf16, and the columns' sums of its unrounded
// values for d_bias.  blockIdx: x = 512 columns of N, y = expert, z = split of
// its rows; the four waves take rows in turn, and their sums are added in
// order.
template <bool GATED>
__global__ void __launch_bounds__(kThreads) k_expert_act_backward(ExpertArgs a) {
    __shared__ float sum[kThreads / kWave - 1][kWave][GATED ? 17 : 9];
    const int lane = lane_id(), wave = threadIdx.x / kWave, e = blockIdx.y;
    const Segment g = segment_of(a.base, e, a.rows);
    const int each = (g.n + gridDim.z - 1) / gridDim.z;
    const int lo = min(g.n, (int)blockIdx.z * each), hi = min(g.n, lo + each);
    const int n = (blockIdx.x * kWave + lane) * 8;
    float sg[8], su[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) sg[j] = su[j] = 0.0f;
    if (n < a.N)
        for (int i = lo + wave; i < hi; i += kThreads / kWave) {
            const int64_t r = g.r0 + i;
            const u32x4 d = *reinterpret_cast<const u32x4 *>(a.d_out + r * a.N + n);
            u32x4 v = {0u, 0u, 0u, 0u}, u = v, od, ou;
            if (a.act != kActNone) v = *reinterpret_cast<const u32x4 *>(a.pre + r * a.Nw + n);
            if (GATED) u = *reinterpret_cast<const u32x4 *>(a.pre + r * a.Nw + a.N + n);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float dg[2], du[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float dv = h ? bf16_hi(d[q]) : bf16_lo(d[q]), p = h ? bf16_hi(v[q]) : bf16_lo(v[q]);
                    if (GATED) {
                        const float s = logistic(p), w = h ? bf16_hi(u[q]) : bf16_lo(u[q]);
                        dg[h] = dv * w * s * (1.0f + p * (1.0f - s));
                        du[h] = dv * p * s;
                        su[2 * q + h] += du[h];
                    } else {
                        dg[h] = a.act == kActRelu ? (p > 0.0f ? dv : 0.0f) : dv * activate_slope(a.act, p);
                    }
                    sg[2 * q + h] += dg[h];
                }
                od[q] = pack_bf16(dg[0], dg[1]);
                if (GATED) ou[q] = pack_bf16(du[0], du[1]);
            }
            if (a.act != kActNone) *reinterpret_cast<u32x4 *>(a.d + r * a.Nw + n) = od;
            if (GATED) *reinterpret_cast<u32x4 *>(a.d + r * a.Nw + a.N + n) = ou;
        }
    if (!a.d_bias) return;
    if (wave > 0)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            sum[wave - 1][lane][j] = sg[j];
            if (GATED) sum[wave - 1][lane][8 + j] = su[j];
        }
    __syncthreads();
    if (wave > 0 || n >= a.N) return;
    float *to = gridDim.z == 1 ? a.d_bias + (int64_t)e * a.Nw : a.part + ((int64_t)e * gridDim.z + blockIdx.z) * a.Nw;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        for (int w = 0; w < kThreads / kWave - 1; ++w) {
            sg[j] += sum[w][lane][j];
            if (GATED) su[j] += sum[w][lane][8 + j];
        }
        to[n + j] = sg[j];
        if (GATED) to[a.N + n + j] = su[j];
    }
}

__global__ void __launch_bounds__(kThreads) k_expert_bias_sum(ExpertArgs a, int splits) {
    const int n = blockIdx.x * kThreads + threadIdx.x, e = blockIdx.y;
    if (n >= a.Nw) return;
    float s = 0.0f;
    for (int z = 0; z < splits; ++z) s += a.part[((int64_t)e * splits + z) * a.Nw + n];
    a.d_bias[(int64_t)e * a.Nw + n] = s;
}

int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

// Tiles of `size` rows that E segments of `rows` rows can make.
int64_t row_tiles(const ExpertArgs &a, int size) { return a.rows / size + (a.rows < a.E ? a.rows : a.E); }

}  // namespace

hipError_t launch_expert(const ExpertArgs &a, hipStream_t st) {
    if (a.rows == 0) return hipSuccess;
    const int cols = ceil_div(a.N, a.act == kActSwiglu ? kTile / 2 : kTile);
    const dim3 grid((uint32_t)(cols * row_tiles(a, kTile)));
    if (a.fp8) hipLaunchKernelGGL((k_expert_simple<kForward, true>), grid, dim3(kThreads), 0, st, a, cols);
    else hipLaunchKernelGGL((k_expert_simple<kForward, false>), grid, dim3(kThreads), 0, st, a, cols);
    return hipGetLastError();
}

hipError_t launch_expert_backward(const ExpertArgs &args, hipStream_t st) {
    ExpertArgs a = args;
    hipError_t rc = hipSuccess;
    if (a.act == kActNone) a.d = const_cast<uint16_t *>(a.d_out);
    if (a.d_bias || a.act != kActNone) {
        const int cols = ceil_div(a.N, 512);
        // About 2048 workgroups, at least 16 rows each on average.
        int splits = 1;
        while (splits < kActSplits && splits * a.E * cols < 2048 && a.rows / a.E > splits * 32) splits *= 2;
        const dim3 grid(cols, a.E, splits);
        if (a.act == kActSwiglu) hipLaunchKernelGGL(k_expert_act_backward<true>, grid, dim3(kThreads), 0, st, a);
        else hipLaunchKernelGGL(k_expert_act_backward<false>, grid, dim3(kThreads), 0, st, a);
        if ((rc = hipGetLastError()) != hipSuccess) return rc;
        if (a.d_bias && splits > 1) {
            hipLaunchKernelGGL(k_expert_bias_sum, dim3(ceil_div(a.Nw, kThreads), a.E), dim3(kThreads), 0, st, a, splits);
            if ((rc = hipGetLastError()) != hipSuccess) return rc;
        }
    }
    const int cols = ceil_div(a.I, kTile);
    if (a.d_x && a.rows > 0) {
        const dim3 grid((uint32_t)(cols * row_tiles(a, kTile)));
        hipLaunchKernelGGL((k_expert_simple<kDx, false>), grid, dim3(kThreads), 0, st, a, cols);
        if ((rc = hipGetLastError()) != hipSuccess) return rc;
    }
    if (a.d_w) {
        const dim3 grid((uint32_t)((int64_t)cols * ceil_div(a.Nw, kTile) * a.E));
        hipLaunchKernelGGL((k_expert_simple<kDw, false>), grid, dim3(kThreads), 0, st, a, cols);
        rc = hipGetLastError();
    }
    return rc;
}

}  // namespace ep
