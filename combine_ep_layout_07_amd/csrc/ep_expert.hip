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
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

enum { kForward = 0, kDx = 1, kDw = 2 };

// Bias, activation and residual of four neighbouring outputs, from the fp32
// sums `v` (and, gated, the up projection's).
__device__ __forceinline__ void finish(const ExpertArgs &a, int e, int64_t r, int c, f32x4 v, f32x4 up) {
    const bool gated = a.act == kActSwiglu;
    const int64_t b = (int64_t)e * a.Nw + c;
    if (a.bias) {
        v += *reinterpret_cast<const f32x4 *>(a.bias + b);
        if (gated) up += *reinterpret_cast<const f32x4 *>(a.bias + b + a.N);
    }
    if (a.pre) {
        uint16_t *to = a.pre + r * a.Nw + c;
        *reinterpret_cast<u32x2 *>(to) = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
        if (gated) *reinterpret_cast<u32x2 *>(to + a.N) = u32x2{pack_bf16(up[0], up[1]), pack_bf16(up[2], up[3])};
    }
    u32x2 res = {0u, 0u};
    if (a.residual) res = *reinterpret_cast<const u32x2 *>(a.residual + r * a.N + c);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = gated ? v[i] * logistic(v[i]) * up[i] : activate(a.act, v[i]);
        if (a.residual) v[i] += i % 2 ? bf16_hi(res[i / 2]) : bf16_lo(res[i / 2]);
    }
    *reinterpret_cast<u32x2 *>(a.out + r * a.N + c) = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
}

// ---- The tiled product ----
//
// A tile of BQ rows x BP columns by WQ x WP waves.  A step of the sum is 128
// bytes of k (64 bf16, 128 fp8) of both operands: the DMA path writes them to
// LDS (16 bytes a lane, no registers), one step ahead of the matrix units, in
// two stages.  D comes transposed from the matrix unit (its rows are P's
// columns), so that a lane holds four neighbours of a row of the output.
//
// An operand contiguous in k lies in LDS as rows of 128 bytes, chunk c of row r
// at slot c ^ (r & 7).  One contiguous across k lies as 64 rows of k, the
// 32-byte unit u of row k at u ^ ((k & 3) | (k & 8) >> 1), and is read by the
// transposing LDS load.  Both place every read's lanes in different banks; the
// permutation is made by each lane's global address, since the DMA writes a
// wave's 1 KiB in lane order.
constexpr uint32_t kOutside = 0x80000000u;  // past every buffer: the load returns zeros

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) char lds_char;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

__device__ __forceinline__ int64_t uniform64(int64_t v) {
    return (int64_t)(uint32_t)uniform((int)v) | (int64_t)uniform((int)(v >> 32)) << 32;
}

// One operand's part of a stage, of B rows (ALONG k) or B columns.
template <bool ALONG, int B, int NW>
struct Loader {
    static constexpr int kLoads = B / 8 / NW;         // of 1 KiB, per wave
    static constexpr int kLanes = ALONG ? 8 : B / 8;  // lanes of one row
    static constexpr int kRows = kWave / kLanes;      // rows of one load
    const char *at;
    int64_t step;
    uint32_t off[kLoads];
    int place;  // ALONG: the lane's chunk; else its k row in the wave's first load

    __device__ __forceinline__ static int row(int j, int wave, int lane) { return (j * NW + wave) * kRows + lane / kLanes; }
    __device__ __forceinline__ static int chunk(int r, int lane) {
        return ALONG ? (lane % 8) ^ (r & 7) : (lane % kLanes) ^ (((r & 3) | (r & 8) >> 1) << 1);
    }
    // Issues the loads of one stage; `left` chunks (ALONG) or rows of k remain.
    __device__ __forceinline__ void issue(char *stage, int wave, int left) {
        const __amdgpu_buffer_rsrc_t rs =
            __builtin_amdgcn_make_buffer_rsrc(const_cast<char *>(at), 0, 0x7fffffff, 0x00020000);
        const bool whole = left >= (ALONG ? 8 : 64);
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            uint32_t o = off[j];
            if (!whole && (ALONG ? place : place + j * NW * kRows) >= left) o = kOutside;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_char *)(stage + (j * NW + wave) * 1024), 16, o, 0, 0, 0);
        }
        at += step;
    }
};

// The lane's share of a 16-wide fragment for 32 steps of k (bf16).
template <bool ALONG, int B>
struct Reader {
    int addr, swz;
    __device__ __forceinline__ void init(int first, int lane) {  // first: the wave's first row or column
        const int g = lane / 16, m = lane % 16;
        if (ALONG) {
            addr = (first + m) * 128 + ((g ^ (m & 7)) * 16);
        } else {
            addr = (g * 8 + m / 4) * (2 * B) + m % 4 * 8;
            swz = (first / 16) ^ ((m / 4) | (g & 1) << 2);
        }
    }
    __device__ __forceinline__ bf16x8 read(const char *lds, int i, int kk) const {
        if (ALONG) return *reinterpret_cast<const bf16x8 *>(lds + ((addr + i * 2048) ^ (kk * 64)));
        const char *p = lds + addr + (swz ^ i) * 32 + kk * 64 * B;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p);
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 8 * B));
        return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
};

// All tiles of `size` rows of the experts' segments.
__device__ __forceinline__ int count_tiles(const int32_t *base, int E, int64_t rows, int size) {
    int n = 0;
    for (int e = lane_id(); e < E; e += kWave) n += (segment_of(base, e, rows).n + size - 1) / size;
#pragma unroll
    for (int d = 32; d; d >>= 1) n += shfl(n, lane_id() ^ d);
    return uniform(n);
}

// Workgroups go round the 8 XCDs; each XCD takes a contiguous eighth of the
// tiles, in groups of 8 rows of tiles walked column by column, so that the
// tiles it works on together share their operands in its L2.
constexpr int kXcds = 8, kGroup = 8;
__device__ __forceinline__ bool place_tile(int b, int rows, int cols, int &row, int &col) {
    const int total = rows * cols, per = (total + kXcds - 1) / kXcds;
    const int i = b % kXcds * per + b / kXcds;
    if (b / kXcds >= per || i >= total) return false;
    const int first = i / (kGroup * cols) * kGroup, in = i % (kGroup * cols);
    const int high = rows - first < kGroup ? rows - first : kGroup;
    row = first + in % high;
    col = in / high;
    return true;
}

template <int MODE, bool FP8, int BQ, int BP, int WQ, int WP>
__global__ void __launch_bounds__(WQ *WP *kWave, 2) k_expert_tile(ExpertArgs a, int cols) {
    constexpr int NW = WQ * WP, NQ = BQ / WQ / 16, NP = BP / WP / 16;
    constexpr bool QA = MODE != kDw, PA = MODE == kForward;
    constexpr int kStage = (BQ + BP) * 128;
    __shared__ __align__(1024) char smem[2][kStage];
    const int lane = lane_id(), wave = uniform(threadIdx.x / kWave);
    const int wq = wave % WQ * (BQ / WQ), wp = wave / WQ * (BP / WP);
    const bool gated = MODE == kForward && a.act == kActSwiglu;
    int trow, tcol, q0 = 0;
    Segment g;
    if (MODE == kDw) {
        const int per = (a.Nw + BQ - 1) / BQ;
        if (!place_tile(blockIdx.x, per * a.E, cols, trow, tcol)) return;
        g = segment_of(a.base, trow / per, a.rows);
        q0 = trow % per * BQ;
    } else {
        if (!place_tile(blockIdx.x, count_tiles(a.base, a.E, a.rows, BQ), cols, trow, tcol)) return;
        g = find_tile(a.base, a.E, a.rows, BQ, trow);
        if (g.e < 0) return;
    }
    const int64_t r0 = uniform64(g.r0);
    const int e = uniform(g.e), n = uniform(g.n);
    constexpr int EL = FP8 ? 1 : 2;
    const int K = MODE == kForward ? a.I : (MODE == kDx ? a.Nw : n);
    const int64_t pitchx = (int64_t)a.I * EL, pitchd = (int64_t)a.Nw * 2;
    const int64_t we = (int64_t)e * a.Nw * a.I;
    const int P = MODE == kForward ? a.N : a.I;  // output columns
    const int p0 = tcol * (gated ? BP / 2 : BP);
    const int nq = MODE == kDw ? min(a.Nw - q0, BQ) : n;

    Loader<QA, BQ, NW> lq;
    Loader<PA, BP, NW> lp;
    const char *d = reinterpret_cast<const char *>(a.d), *x = static_cast<const char *>(a.x), *w = static_cast<const char *>(a.w);
    if (MODE == kForward) {
        lq.at = x + r0 * pitchx;
        // Rows of the tile alternate between 16 of the gate and 16 of the up
        // projection; a wave's loads all lie in one of the two.
        const bool up = gated && wave / 2 % 2;
        lp.at = w + (we + (int64_t)(p0 + (up ? a.N : 0)) * a.I) * EL;
    } else if (MODE == kDx) {
        lq.at = d + r0 * pitchd;
        lp.at = w + (we + p0) * 2;
    } else {
        lq.at = d + r0 * pitchd + (int64_t)q0 * 2;
        lp.at = x + r0 * pitchx + (int64_t)p0 * 2;
    }
    lq.step = QA ? 128 : 64 * pitchd;
    lp.step = PA ? 128 : 64 * pitchx;
#pragma unroll
    for (int j = 0; j < lq.kLoads; ++j) {
        const int r = lq.row(j, wave, lane), c = lq.chunk(r, lane);
        const bool in = QA ? r < nq : c * 8 < nq;
        lq.off[j] = in ? (uint32_t)(r * (QA && MODE == kForward ? pitchx : pitchd)) + c * 16 : kOutside;
        if (j == 0) lq.place = QA ? c : r;
    }
#pragma unroll
    for (int j = 0; j < lp.kLoads; ++j) {
        const int r = lp.row(j, wave, lane), c = lp.chunk(r, lane);
        const int local = gated ? r / 32 * 16 + r % 16 : r;
        const bool in = PA ? p0 + local < P : p0 + c * 8 < P;
        lp.off[j] = in ? (uint32_t)(local * pitchx) + c * 16 : kOutside;
        if (j == 0) lp.place = PA ? c : r;
    }
    Reader<QA, BQ> rq;
    Reader<PA, BP> rp;
    rq.init(wq, lane);
    rp.init(wp, lane);

    f32x4 acc[NP][NQ];
#pragma unroll
    for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int j = 0; j < NQ; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    // fp8: places of the lane's scales
    const int nkb = a.I / 128;
    const float *xs_at[FP8 ? NQ : 1], *ws_at[FP8 ? NP : 1];
    float xs[FP8 ? NQ : 1], ws[FP8 ? NP : 1];
    if (FP8) {
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
            const int q = wq + j * 16 + lane % 16;
            xs_at[j] = a.x_sf + (r0 + min(q, nq - 1)) * nkb;
        }
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int pl = wp + i * 16 + lane / 16 * 4;
            const int c = min(gated ? p0 + pl / 32 * 16 + pl % 16 : p0 + pl, a.N - 1);
            const int row = c + (gated && i % 2 ? a.N : 0);
            ws_at[i] = a.w_sf + ((int64_t)e * ((a.Nw + 127) / 128) + row / 128) * nkb;
        }
    }

    const int per_step = FP8 ? 128 : 64;
    const int steps = (K + per_step - 1) / per_step;
    auto issue = [&](int t, char *stage) {
        const int left = K - t * per_step;
        lq.issue(stage, wave, QA ? left / (16 / EL) : left);
        lp.issue(stage + BQ * 128, wave, PA ? left / (16 / EL) : left);
    };
    if (steps > 0) issue(0, smem[0]);
    for (int t = 0; t < steps; ++t) {
        // The stage's loads have landed, and every wave is done with the other
        // stage (its reads fed matrix operations that were issued before).
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        if (FP8) {
#pragma unroll
            for (int j = 0; j < NQ; ++j) xs[j] = xs_at[j][t];
#pragma unroll
            for (int i = 0; i < NP; ++i) ws[i] = ws_at[i][t];
        }
        if (t + 1 < steps) issue(t + 1, smem[(t + 1) & 1]);
        const char *sq = smem[t & 1], *sp = sq + BQ * 128;
        if (!FP8) {
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                bf16x8 fq[NQ], fp[NP];
#pragma unroll
                for (int j = 0; j < NQ; ++j) fq[j] = rq.read(sq, j, kk);
#pragma unroll
                for (int i = 0; i < NP; ++i) fp[i] = rp.read(sp, i, kk);
#pragma unroll
                for (int i = 0; i < NP; ++i)
#pragma unroll
                    for (int j = 0; j < NQ; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fp[i], fq[j], acc[i][j], 0, 0, 0);
            }
        } else {
            auto wide = [](bf16x8 lo, bf16x8 hi) {
                typedef int i32x4 __attribute__((ext_vector_type(4)));
                return __builtin_shufflevector(__builtin_bit_cast(i32x4, lo), __builtin_bit_cast(i32x4, hi), 0, 1, 2, 3, 4, 5, 6, 7);
            };
            i32x8 fq[NQ];
#pragma unroll
            for (int j = 0; j < NQ; ++j) fq[j] = wide(rq.read(sq, j, 0), rq.read(sq, j, 1));
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const i32x8 fp = wide(rp.read(sp, i, 0), rp.read(sp, i, 1));
#pragma unroll
                for (int j = 0; j < NQ; ++j) {
                    const f32x4 part = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        fp, fq[j], f32x4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, 0x7f7f7f7f, 0, 0x7f7f7f7f);
                    const float sc = xs[j] * ws[i];
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[i][j][r] = fmaf(part[r], sc, acc[i][j][r]);
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
            const int q = wq + j * 16 + lane % 16, pl = wp + i * 16 + lane / 16 * 4;
            if (q >= nq) continue;
            if (MODE == kForward) {
                if (gated && i % 2) continue;
                const int c = gated ? p0 + pl / 32 * 16 + pl % 16 : p0 + pl;
                if (c < a.N) finish(a, e, r0 + q, c, acc[i][j], acc[i | 1][j]);
            } else if (p0 + pl < P) {
                uint16_t *dst = MODE == kDx ? a.d_x + (r0 + q) * a.I : a.d_w + we + (int64_t)(q0 + q) * a.I;
                *reinterpret_cast<u32x2 *>(dst + p0 + pl) =
                    u32x2{pack_bf16(acc[i][j][0], acc[i][j][1]), pack_bf16(acc[i][j][2], acc[i][j][3])};
            }
        }
}

// Gradient of the pre-activation, bf16, and the columns' sums of its unrounded
// values for d_bias.  A workgroup takes 512 columns of one tile of kActRows
// rows of an expert (so that one expert with most of the rows is no slower),
// each wave a quarter of the rows, four in flight; the waves' sums are added in
// order, and a second launch adds the tiles' in order.
template <bool GATED>
__global__ void __launch_bounds__(kThreads) k_expert_act_backward(ExpertArgs a, int cols) {
    constexpr int kMore = kThreads / kWave - 1, kEach = kActRows / (kMore + 1), G = 4;
    __shared__ float sum[kMore][kWave][GATED ? 17 : 9];
    const int lane = lane_id(), wave = threadIdx.x / kWave;
    const int64_t tile = blockIdx.x / cols;
    const Segment g = find_tile(a.base, a.E, a.rows, kActRows, tile);
    if (g.e < 0) return;
    const int n = (blockIdx.x % cols * kWave + lane) * 8;
    float sg[8], su[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) sg[j] = su[j] = 0.0f;
    if (n < a.N)
        for (int i0 = 0; i0 < kEach; i0 += G) {
            const int64_t first = g.r0 + wave * kEach + i0;
            const int left = g.n - wave * kEach - i0;
            u32x4 d[G], v[G], u[G];
#pragma unroll
            for (int i = 0; i < G; ++i) {
                const int64_t r = first + (i < left ? i : 0);
                d[i] = v[i] = u[i] = u32x4{0u, 0u, 0u, 0u};
                if (left > 0) {
                    d[i] = *reinterpret_cast<const u32x4 *>(a.d_out + r * a.N + n);
                    if (a.act != kActNone) v[i] = *reinterpret_cast<const u32x4 *>(a.pre + r * a.Nw + n);
                    if (GATED) u[i] = *reinterpret_cast<const u32x4 *>(a.pre + r * a.Nw + a.N + n);
                }
            }
#pragma unroll
            for (int i = 0; i < G; ++i) {
                if (i >= left) continue;
                const int64_t r = first + i;
                u32x4 od, ou;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float dg[2], du[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float dv = h ? bf16_hi(d[i][q]) : bf16_lo(d[i][q]), p = h ? bf16_hi(v[i][q]) : bf16_lo(v[i][q]);
                        if (GATED) {
                            const float s = logistic(p), w = h ? bf16_hi(u[i][q]) : bf16_lo(u[i][q]);
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
    float *to = a.part + tile * a.Nw;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        for (int w = 0; w < kMore; ++w) {
            sg[j] += sum[w][lane][j];
            if (GATED) su[j] += sum[w][lane][8 + j];
        }
        to[n + j] = sg[j];
        if (GATED) to[a.N + n + j] = su[j];
    }
}

// d_bias: the sums of the expert's tiles, each wave every fourth, then the
// waves in order.
__global__ void __launch_bounds__(kThreads) k_expert_bias_sum(ExpertArgs a) {
    __shared__ float sum[kThreads / kWave][kWave];
    const int lane = lane_id(), wave = threadIdx.x / kWave, e = blockIdx.y;
    const int n = blockIdx.x * kWave + lane;
    const int first = count_tiles(a.base, e, a.rows, kActRows);
    const int tiles = (segment_of(a.base, e, a.rows).n + kActRows - 1) / kActRows;
    // (A table that decreases counts more tiles than there are: stay inside.)
    const int last = (int)min((int64_t)first + tiles, a.part_tiles);
    float s = 0.0f;
    if (n < a.Nw) {
#pragma unroll 4
        for (int t = first + wave; t < last; t += kThreads / kWave) s += a.part[(int64_t)t * a.Nw + n];
    }
    sum[wave][lane] = s;
    __syncthreads();
    if (wave > 0 || n >= a.Nw) return;
    for (int w = 1; w < kThreads / kWave; ++w) s += sum[w][lane];
    a.d_bias[(int64_t)e * a.Nw + n] = s;
}

int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

int64_t row_tiles(const ExpertArgs &a, int size) { return expert_row_tiles(a.rows, a.E, size); }

template <int MODE, bool FP8, int BQ, int BP, int WQ, int WP>
hipError_t run_tile(const ExpertArgs &a, hipStream_t st) {
    const bool gated = MODE == kForward && a.act == kActSwiglu;
    const int64_t cols = ceil_div(MODE == kForward ? a.N : a.I, gated ? BP / 2 : BP);
    const int64_t tiles = MODE == kDw ? (int64_t)ceil_div(a.Nw, BQ) * a.E : row_tiles(a, BQ);
    const int64_t blocks = (tiles * cols + kXcds - 1) / kXcds * kXcds;
    if (blocks > 4294967295ll / (WQ * WP * kWave)) return hipErrorInvalidValue;
    hipLaunchKernelGGL((k_expert_tile<MODE, FP8, BQ, BP, WQ, WP>), dim3((uint32_t)blocks), dim3(WQ * WP * kWave), 0, st,
                       a, (int)cols);
    return hipGetLastError();
}

template <int MODE, bool FP8>
hipError_t run(const ExpertArgs &a, hipStream_t st) {
    const int64_t each = MODE == kDw ? a.Nw : a.rows / a.E;
    if (each >= 256) return run_tile<MODE, FP8, 256, 256, 4, 2>(a, st);
    return run_tile<MODE, FP8, 128, 128, 2, 2>(a, st);
}

}  // namespace

hipError_t launch_expert(const ExpertArgs &a, hipStream_t st) {
    if (a.rows == 0) return hipSuccess;
    return a.fp8 ? run<kForward, true>(a, st) : run<kForward, false>(a, st);
}

hipError_t launch_expert_backward(const ExpertArgs &args, hipStream_t st) {
    ExpertArgs a = args;
    hipError_t rc = hipSuccess;
    if (a.act == kActNone) a.d = const_cast<uint16_t *>(a.d_out);
    if (a.rows > 0 && (a.d_bias || a.act != kActNone)) {
        const int cols = ceil_div(a.N, kWave * 8);
        const int64_t blocks = cols * a.part_tiles;
        if (blocks > 4294967295ll / kThreads) return hipErrorInvalidValue;
        if (a.act == kActSwiglu)
            hipLaunchKernelGGL(k_expert_act_backward<true>, dim3((uint32_t)blocks), dim3(kThreads), 0, st, a, cols);
        else
            hipLaunchKernelGGL(k_expert_act_backward<false>, dim3((uint32_t)blocks), dim3(kThreads), 0, st, a, cols);
        if ((rc = hipGetLastError()) != hipSuccess) return rc;
    }
    if (a.d_bias) {
        hipLaunchKernelGGL(k_expert_bias_sum, dim3(ceil_div(a.Nw, kWave), a.E), dim3(kThreads), 0, st, a);
        if ((rc = hipGetLastError()) != hipSuccess) return rc;
    }
    if (a.d_x && a.rows > 0 && (rc = run<kDx, false>(a, st)) != hipSuccess) return rc;
    return a.d_w ? run<kDw, false>(a, st) : rc;
}

}  // namespace ep
