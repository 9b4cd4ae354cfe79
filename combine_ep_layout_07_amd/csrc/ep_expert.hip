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

// ---- The tiled product ----
//
// A tile of BQ rows x BP columns by WQ x WP waves.  The sum runs in steps of SB
// bytes of k (64 bytes: 32 bf16); the DMA path writes both operands of a step to
// one of NST stages of LDS (16 bytes a lane, no registers), NST - 1 steps ahead
// of the matrix unit.  D comes transposed from the matrix unit (its rows are
// P's columns), so that a lane holds four neighbours of a row of the output.
//
// An operand contiguous in k lies in LDS as rows of SB bytes, chunk c (16 bytes)
// of row r at slot c ^ (r & 7) (SB 128) or c ^ (r / 2 & 3) (SB 64).  One
// contiguous across k lies as rows of k, the 32-byte unit u of row k at
// u ^ ((k & 3) | (k & 8) >> 1), and is read by the transposing LDS load.  Both
// place the lanes of every read in different banks; the permutation is made by
// each lane's global address, since the DMA writes a wave's 1 KiB in lane order.
constexpr uint32_t kOutside = 0x80000000u;  // past every buffer: the load returns zeros

// s_waitcnt: at most `vm` loads and `lds` LDS operations outstanding.
constexpr int wait_for(int vm, int lds) { return (vm & 15) | (vm >> 4) << 14 | 7 << 4 | lds << 8; }
constexpr int kAnyLds = 15, kAnyLoads = 63;

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) char lds_char;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

__device__ __forceinline__ int64_t uniform64(int64_t v) {
    return (int64_t)(uint32_t)uniform((int)v) | (int64_t)uniform((int)(v >> 32)) << 32;
}

// One operand's part of a stage, of B rows (ALONG k) or B columns.
template <bool ALONG, int B, int NW, int SB>
struct Loader {
    static constexpr int kLoads = B * SB / 1024 / NW;       // of 1 KiB, per wave
    static constexpr int kLanes = ALONG ? SB / 16 : B / 8;  // lanes of one row
    static constexpr int kRows = kWave / kLanes;            // rows of one load
    static constexpr int kFull = ALONG ? SB / 16 : SB / 2;  // chunks or rows of k of a whole step
    const char *at;
    int64_t step;
    uint32_t off;    // of the wave's first load; kOutside: the lane's column does not exist
    uint32_t apart;  // bytes between the wave's loads
    uint32_t bytes;  // rows at or past the tile's end lie outside
    int place;       // ALONG: the lane's chunk; else its k row in the wave's first load

    __device__ __forceinline__ static int row(int j, int wave, int lane) { return (j * NW + wave) * kRows + lane / kLanes; }
    __device__ __forceinline__ static int chunk(int r, int lane) {
        if (!ALONG) return (lane % kLanes) ^ (((r & 3) | (r & 8) >> 1) << 1);
        return (lane % kLanes) ^ (SB == 128 ? r & 7 : r / 2 & 3);
    }
    // Issues the loads of one stage; `left` chunks (ALONG) or rows of k remain
    // (none: zeros, so that every step has as many loads).
    __device__ __forceinline__ void issue(char *stage, int wave, int left) {
        const __amdgpu_buffer_rsrc_t rs =
            __builtin_amdgcn_make_buffer_rsrc(const_cast<char *>(at), 0, bytes, 0x00020000);
        const bool whole = left >= kFull;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            uint32_t o = off + j * apart;
            if (!whole && (ALONG ? place : place + j * NW * kRows) >= left) o = kOutside;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_char *)(stage + (j * NW + wave) * 1024), 16, o, 0, 0, 0);
        }
        at += step;
    }
};

// The lane's share of a 16-wide fragment: 16 bytes of k of its row, for 64 bytes
// of k over the four lane groups.
template <bool ALONG, int B, int SB>
struct Reader {
    int addr, swz;  // ALONG: addresses of the first and the second 64 bytes of k
    __device__ __forceinline__ void init(int first, int lane) {  // first: the wave's first row or column
        const int g = lane / 16, m = lane % 16;
        if (ALONG) {
            addr = (first + m) * SB + ((g ^ (SB == 128 ? m & 7 : m / 2 & 3)) * 16);
            swz = addr ^ 64;
        } else {
            addr = (g * 8 + m / 4) * (2 * B) + m % 4 * 8;
            swz = (first / 16) ^ ((m / 4) | (g & 1) << 2);
        }
    }
    __device__ __forceinline__ bf16x8 read(const char *lds, int i, int kk) const {
        if (ALONG) return *reinterpret_cast<const bf16x8 *>(lds + (kk ? swz : addr) + i * 16 * SB);
        const char *p = lds + addr + (swz ^ i) * 32 + kk * 64 * B;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p);
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 8 * B));
        return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
};

// Workgroups go round the 8 XCDs.  Of every 128 tiles in order each XCD takes 16
// neighbours, 4 rows of tiles by 4 columns, which share their operands in its
// L2, while all XCDs together stay within one or two experts: at 32768 rows,
// 16 experts, 7168 to 2 x 2048 that took 1.71 ms, a contiguous eighth of all
// tiles per XCD 1.86 ms (fewer L2 misses, but twice as many rows open in the
// memory behind), tiles in launch order 1.77 ms.
constexpr int kXcds = 8, kPatch = 16, kGroup = 4;
__device__ __forceinline__ bool place_tile(int b, int rows, int cols, int &row, int &col) {
    const int i = b / (kXcds * kPatch) * (kXcds * kPatch) + b % kXcds * kPatch + b / kXcds % kPatch;
    if (i >= rows * cols) return false;
    const int first = i / (kGroup * cols) * kGroup, in = i % (kGroup * cols);
    const int high = rows - first < kGroup ? rows - first : kGroup;
    row = first + in % high;
    col = in / high;
    return true;
}

// The workgroup's tile of `size` rows of an expert's segment and its column.
__device__ __forceinline__ bool locate(const ExpertArgs &a, int size, int cols, Segment &g, int &col) {
    int row;
    if (a.E > kWave) {
        if (!place_tile(blockIdx.x, count_tiles(a.base, a.E, a.rows, size), cols, row, col)) return false;
        g = find_tile(a.base, a.E, a.rows, size, row);
        return g.e >= 0;
    }
    const int lane = lane_id();
    g = lane < a.E ? segment_of(a.base, lane, a.rows) : Segment{lane, 0, 0};
    const int mine = (g.n + size - 1) / size, incl = wave_scan(mine);
    if (!place_tile(blockIdx.x, read_lane(incl, kWave - 1), cols, row, col)) return false;
    const int o = __builtin_ctzll(ballot(incl > row));
    const int at = row - (read_lane(incl, o) - read_lane(mine, o));
    const int left = read_lane(g.n, o) - at * size;
    g = {o, (int64_t)read_lane((int)g.r0, o) + (int64_t)at * size, left < size ? left : size};
    return true;
}

// W neighbouring values, W 4 or 8.
template <int W>
__device__ __forceinline__ void store_bf16(uint16_t *to, const float (&v)[W]) {
    typedef uint32_t bits __attribute__((ext_vector_type(W / 2)));
    bits o;
#pragma unroll
    for (int i = 0; i < W / 2; ++i) o[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<bits *>(to) = o;
}
template <int W>
__device__ __forceinline__ void load_bf16(const uint16_t *p, uint32_t (&v)[W / 2]) {
    typedef uint32_t bits __attribute__((ext_vector_type(W / 2)));
    const bits o = *reinterpret_cast<const bits *>(p);
#pragma unroll
    for (int i = 0; i < W / 2; ++i) v[i] = o[i];
}
template <int W>
__device__ __forceinline__ void load_float(const float *p, float (&v)[W]) {
#pragma unroll
    for (int i = 0; i < W; i += 4) {
        const f32x4 o = *reinterpret_cast<const f32x4 *>(p + i);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[i + j] = o[j];
    }
}

// W neighbouring outputs from the biased fp32 sums `v` (and, gated, those of
// the up projection): the kept pre-activation, activation and residual.
template <bool GATED, int W>
__device__ __forceinline__ void finish(const ExpertArgs &a, int64_t r, int c, float (&v)[W], const float (&up)[W],
                                       const uint32_t (&res)[W / 2]) {
    if (a.pre) {
        uint16_t *to = a.pre + r * a.Nw + c;
        store_bf16<W>(to, v);
        if (GATED) store_bf16<W>(to + a.N, up);
    }
    if (GATED) {
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] = v[i] * logistic(v[i]) * up[i];
    } else if (a.act == kActGelu) {
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] = activate(kActGelu, v[i]);
    } else if (a.act == kActSilu) {
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] = activate(kActSilu, v[i]);
    } else if (a.act == kActRelu) {
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] = activate(kActRelu, v[i]);
    }
    if (a.residual) {
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] += i % 2 ? bf16_hi(res[i / 2]) : bf16_lo(res[i / 2]);
    }
    store_bf16<W>(a.out + r * a.N + c, v);
}

__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_s_waitcnt(wait_for(kAnyLoads, 0));
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// The forward tile through LDS in fp32, as many rows at a time as fit, and the
// epilogue in row order: a thread keeps its eight columns, so their bias is
// loaded once, and has the residual of all its rows in flight before the sums
// are in LDS (loaded row by row the epilogue took half of a small product).
template <bool GATED, int BQ, int BP, int NW, int NP, int NQ, typename ACC>
__device__ __forceinline__ void forward_rows(const ExpertArgs &a, char *smem, ACC (&acc)[NP][NQ], int e, int64_t r0, int p0,
                                             int nq, int wq, int wp, int lane) {
    constexpr int kRowsPer = BQ < 128 ? BQ : 128, kPer = BP / (GATED ? 16 : 8);
    constexpr int kApart = NW * kWave / kPer, kItems = (kRowsPer + kApart - 1) / kApart;
    const int c8 = threadIdx.x % kPer, q0 = threadIdx.x / kPer, c = p0 + c8 * 8;
    const int c4 = GATED ? c8 / 2 * 8 + c8 % 2 * 2 : c8 * 2;
    float bv[8], bu[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) bv[i] = bu[i] = 0.0f;
    if (a.bias && c < a.N) {
        load_float<8>(a.bias + (int64_t)e * a.Nw + c, bv);
        if (GATED) load_float<8>(a.bias + (int64_t)e * a.Nw + a.N + c, bu);
    }
#pragma unroll
    for (int h = 0; h < BQ / kRowsPer; ++h) {
        uint32_t res[kItems][4];
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            const int q = h * kRowsPer + q0 + k * kApart;
            res[k][0] = res[k][1] = res[k][2] = res[k][3] = 0u;
            if (a.residual && q0 + k * kApart < kRowsPer && q < nq && c < a.N) load_bf16<8>(a.residual + (r0 + q) * a.N + c, res[k]);
        }
        lds_barrier();
        if (wq / kRowsPer == h) {
#pragma unroll
            for (int i = 0; i < NP; ++i)
#pragma unroll
                for (int j = 0; j < NQ; ++j) {
                    const int q = wq % kRowsPer + j * 16 + lane % 16, at = (wp + i * 16) / 4 + lane / 16;
                    *reinterpret_cast<f32x4 *>(smem + q * BP * 4 + (at ^ (q & 7)) * 16) =
                        f32x4{acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
                }
        }
        lds_barrier();
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            const int q = q0 + k * kApart;
            if (q >= kRowsPer || h * kRowsPer + q >= nq || c >= a.N) continue;
            const char *row = smem + q * BP * 4;
            float v[8], up[8];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const f32x4 l = *reinterpret_cast<const f32x4 *>(row + ((c4 + i) ^ (q & 7)) * 16);
                f32x4 u = l;
                if (GATED) u = *reinterpret_cast<const f32x4 *>(row + ((c4 + 4 + i) ^ (q & 7)) * 16);
#pragma unroll
                for (int r = 0; r < 4; ++r) v[4 * i + r] = l[r] + bv[4 * i + r], up[4 * i + r] = u[r] + bu[4 * i + r];
            }
            finish<GATED, 8>(a, r0 + h * kRowsPer + q, c, v, up, res[k]);
        }
    }
}

// A lane's four sums: the matrix unit's own registers, or, for fp8, four that
// stay apart (as a vector the compiler moved them at every step).
struct Four {
    float v[4];
    __device__ __forceinline__ float &operator[](int i) { return v[i]; }
};
template <bool FP8>
struct Sum {
    typedef f32x4 type;
};
template <>
struct Sum<true> {
    typedef Four type;
};

template <int MODE, bool FP8, int BQ, int BP, int WQ, int WP, int SB, int NST>
__global__ void __launch_bounds__(WQ *WP *kWave, 2) k_expert_tile(ExpertArgs a, int cols) {
    constexpr int NW = WQ * WP, NQ = BQ / WQ / 16, NP = BP / WP / 16;
    constexpr bool QA = MODE != kDw, PA = MODE == kForward;
    constexpr int kStage = (BQ + BP) * SB;
    __shared__ __align__(1024) char smem[NST * kStage];
    const int lane = lane_id(), wave = uniform(threadIdx.x / kWave);
    const int wq = wave % WQ * (BQ / WQ), wp = wave / WQ * (BP / WP);
    const bool gated = MODE == kForward && a.act == kActSwiglu;
    int tcol, q0 = 0;
    Segment g;
    if (MODE == kDw) {
        const int per = (a.Nw + BQ - 1) / BQ;
        int trow;
        if (!place_tile(blockIdx.x, per * a.E, cols, trow, tcol)) return;
        g = segment_of(a.base, trow / per, a.rows);
        q0 = trow % per * BQ;
    } else if (!locate(a, BQ, cols, g, tcol)) {
        return;
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

    Loader<QA, BQ, NW, SB> lq;
    Loader<PA, BP, NW, SB> lp;
    const char *d = reinterpret_cast<const char *>(a.d), *x = static_cast<const char *>(a.x), *w = static_cast<const char *>(a.w);
    if (MODE == kForward) {
        lq.at = x + r0 * pitchx;
        lp.at = w + (we + (int64_t)p0 * a.I) * EL;
        // Rows of the tile alternate between 16 of the gate and 16 of the up
        // projection; all of a wave's loads lie in one of the two.
        static_assert(MODE != kForward || NW * lp.kRows % 32 == 0, "a wave's loads keep their side");
        if (gated && wave * lp.kRows / 16 % 2) lp.at += (int64_t)a.N * pitchx;
    } else if (MODE == kDx) {
        lq.at = d + r0 * pitchd;
        lp.at = w + (we + p0) * 2;
    } else {
        lq.at = d + r0 * pitchd + (int64_t)q0 * 2;
        lp.at = x + r0 * pitchx + (int64_t)p0 * 2;
    }
    lq.step = QA ? SB : SB / 2 * pitchd;
    lp.step = PA ? SB : SB / 2 * pitchx;
    {
        // Along k: the offsets grow with the row, so a bound at the end of the
        // tile's last row turns the rows after it into zeros.  Across k: columns
        // outside by the lane's offset, rows of k by `left`.
        const int r = lq.row(0, wave, lane), c = lq.chunk(r, lane);
        const uint32_t pitch = (uint32_t)(QA && MODE == kForward ? pitchx : pitchd);
        lq.off = QA || c * 8 < nq ? r * pitch + c * 16 : kOutside;
        lq.apart = NW * lq.kRows * pitch;
        lq.bytes = QA ? (nq - 1) * pitch + SB : kOutside;
        lq.place = QA ? c : r;
    }
    {
        const int r = lp.row(0, wave, lane), c = lp.chunk(r, lane);
        const uint32_t pitch = (uint32_t)pitchx;
        lp.off = PA || p0 + c * 8 < P ? (gated ? r / 32 * 16 + r % 16 : r) * pitch + c * 16 : kOutside;
        lp.apart = NW * lp.kRows / (gated ? 2 : 1) * pitch;
        lp.bytes = PA ? (min(P - p0, gated ? BP / 2 : BP) - 1) * pitch + SB : kOutside;
        lp.place = PA ? c : r;
    }
    Reader<QA, BQ, SB> rq;
    Reader<PA, BP, SB> rp;
    rq.init(wq, lane);
    rp.init(wp, lane);

    typename Sum<FP8>::type acc[NP][NQ];
#pragma unroll
    for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int j = 0; j < NQ; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[i][j][r] = 0.0f;

    // fp8: the scales of eight steps at a time go to LDS, [row][8] for x, and
    // for the weights the tile's two or three blocks of 128 weight rows: its
    // columns', or gated the gate's one and the up projection's two at most.
    // (Loaded by each lane at each step they took a third of the time: a line
    // for every row, every time anew.)
    constexpr int kBlocks = 8;
    __shared__ float sxs[FP8 ? 2 : 1][FP8 ? BQ * kBlocks : 1], sws[FP8 ? 2 : 1][FP8 ? kWave : 1];
    const int nkb = a.I / 128;
    const int up_from = ((a.N + p0) / 128 + 1) * 128 - a.N - p0 - wp / 2;  // the wave's columns from here on take the third
    auto load_scales = [&](int kb0) {
        const int to = kb0 / kBlocks % 2, kb = kb0 + lane % kBlocks;
        const __amdgpu_buffer_rsrc_t rx =
            __builtin_amdgcn_make_buffer_rsrc(const_cast<float *>(a.x_sf + r0 * nkb), 0, kOutside, 0x00020000);
#pragma unroll
        for (int j = 0; j < BQ * kBlocks / kWave / NW; ++j) {
            const int row = (j * NW + wave) * (kWave / kBlocks) + lane / kBlocks;
            const uint32_t o = row < nq && kb < nkb ? (row * nkb + kb) * 4 : kOutside;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_char *)&sxs[to][(j * NW + wave) * kWave], 4, o, 0, 0, 0);
        }
        if (wave == 0) {
            const int blocks = (a.Nw + 127) / 128, slot = lane / kBlocks;
            const int block = gated && slot > 0 ? (a.N + p0) / 128 + slot - 1 : p0 / 128 + slot;
            const uint32_t o = slot < 3 && block < blocks && kb < nkb ? (block * nkb + kb) * 4 : kOutside;
            const __amdgpu_buffer_rsrc_t rw = __builtin_amdgcn_make_buffer_rsrc(
                const_cast<float *>(a.w_sf + (int64_t)e * blocks * nkb), 0, kOutside, 0x00020000);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_char *)&sws[to][0], 4, o, 0, 0, 0);
        }
    };
    auto x_scale = [&](int t, int j) {
        return sxs[t / kBlocks % 2][(wq + j * 16 + lane % 16) * kBlocks + t % kBlocks];
    };
    // The scales of even and of odd 16 columns of the wave, the latter up to
    // and from up_from on.
    auto w_scales = [&](int t) {
        const float *s = &sws[t / kBlocks % 2][t % kBlocks];
        const float first = s[gated ? 0 : wp / 128 * kBlocks], lo = s[kBlocks], hi = s[2 * kBlocks];
        return f32x4{first, gated ? lo : first, gated ? hi : first, 0.0f};
    };
    auto w_scale = [&](f32x4 s, int i) { return i % 2 == 0 ? s[0] : (i / 2 * 16 + lane / 16 * 4 < up_from ? s[1] : s[2]); };
    auto both = [](bf16x8 lo, bf16x8 hi) {
        return __builtin_shufflevector(__builtin_bit_cast(i32x4, lo), __builtin_bit_cast(i32x4, hi), 0, 1, 2, 3, 4, 5, 6, 7);
    };
    auto mfma8 = [](i32x8 p, i32x8 q) {
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(p, q, f32x4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, 0, 0, 0);
    };
    auto add_scaled = [](typename Sum<FP8>::type &c, f32x4 part, float sc) {
#pragma unroll
        for (int r = 0; r < 4; ++r) c[r] = fmaf(part[r], sc, c[r]);
        // Here and not later: left to itself the compiler holds the products of
        // a whole step until its end, which spills.
        asm volatile("" : "+v"(c[0]), "+v"(c[1]), "+v"(c[2]), "+v"(c[3]));
    };

    constexpr int kPerStep = SB / EL, kIssued = lq.kLoads + lp.kLoads;
    const int steps = (K + kPerStep - 1) / kPerStep;
    auto issue = [&](int t, int stage) {
        if (FP8 && t % kBlocks == 0 && t < steps) load_scales(t);
        const int left = K - t * kPerStep;
        char *to = smem + stage * kStage;
        lq.issue(to, wave, QA ? left / (16 / EL) : left);
        lp.issue(to + BQ * SB, wave, PA ? left / (16 / EL) : left);
    };
    auto next = [](int stage) { return stage + 1 == NST ? 0 : stage + 1; };
    // The oldest step's loads are done when those of NST - 2 steps may be out.
    constexpr int kLanded = (NST - 2) * kIssued;
    // (Loads end in order, and a step's scales are issued before its operands.)
    static_assert(kLanded < kAnyLoads, "vmcnt");
    if (steps > 0)
        for (int t = 0; t < NST - 1; ++t) issue(t, t);
    int rd = 0, wr = NST - 1;
    if constexpr (NW == 8) {
        // Two waves on each SIMD, of the two halves of the workgroup: one reads
        // its fragments while the other keeps the matrix unit, and at the next
        // barrier they change places; the second half runs one turn behind,
        // held by one barrier more at the start.  fp8 has two such turns per
        // step (the halves of P; all fragments of a step would not fit the
        // registers).  A stage is written again from the turn after the second
        // half's last read of it on.  Each wave waits for its own loads in the
        // last turn before the first half reads them.
        constexpr int kTurns = FP8 ? 2 : 1;
        static_assert(NW != 8 || (FP8 ? SB == 128 : SB == 64), "one turn's fragments");
        const bool second = wave >= 4;
        auto turn = [] {
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_barrier();
            __builtin_amdgcn_sched_barrier(0);
        };
        if (steps > 0) __builtin_amdgcn_s_waitcnt(wait_for(kLanded, kAnyLds));
        asm volatile("" ::: "memory");
        turn();
        if (second) turn();
        for (int t = 0; t < steps; ++t) {
            const char *sq = smem + rd * kStage, *sp = sq + BQ * SB;
            i32x8 wideq[FP8 ? NQ : 1], widep[FP8 ? NP / 2 : 1];
            float xs[FP8 ? NQ : 1];
            f32x4 ws;
#pragma unroll
            for (int h = 0; h < kTurns; ++h) {
                const int p1 = h * (NP / 2);
                asm volatile("" ::: "memory");
                bf16x8 fq[FP8 ? 1 : NQ], fp[FP8 ? 1 : NP];
                if (FP8) {
                    if (h == 0) {
                        ws = w_scales(t);
#pragma unroll
                        for (int j = 0; j < NQ; ++j) {
                            xs[j] = x_scale(t, j);
                            wideq[j] = both(rq.read(sq, j, 0), rq.read(sq, j, 1));
                        }
                    }
#pragma unroll
                    for (int i = 0; i < NP / 2; ++i) widep[i] = both(rp.read(sp, p1 + i, 0), rp.read(sp, p1 + i, 1));
                } else {
#pragma unroll
                    for (int j = 0; j < NQ; ++j) fq[j] = rq.read(sq, j, 0);
#pragma unroll
                    for (int i = 0; i < NP; ++i) fp[i] = rp.read(sp, i, 0);
                }
                if (h == 0) issue(t + NST - 1, wr);
                asm volatile("" ::: "memory");
                if (h == kTurns - 1 && second) __builtin_amdgcn_s_waitcnt(wait_for(kLanded, 0));
                else __builtin_amdgcn_s_waitcnt(wait_for(kAnyLoads, 0));
                turn();
                __builtin_amdgcn_s_setprio(1);
                if constexpr (FP8) {
                    // Two products, and the scaling of the two before, at a time.
                    constexpr int kPairs = NP / 2 * NQ / 2;
                    f32x4 part[2][2];
#pragma unroll
                    for (int u = 0; u <= kPairs; ++u) {
#pragma unroll
                        for (int v = 0; v < 2 && u < kPairs; ++v)
                            part[u % 2][v] = mfma8(widep[u * 2 / NQ], wideq[u * 2 % NQ + v]);
#pragma unroll
                        for (int v = 0; v < 2 && u > 0; ++v) {
                            const int i = p1 + (u - 1) * 2 / NQ, j = (u - 1) * 2 % NQ + v;
                            add_scaled(acc[i][j], part[(u - 1) % 2][v], xs[j] * w_scale(ws, i));
                        }
                        __builtin_amdgcn_sched_barrier(0);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < NP; ++i)
#pragma unroll
                        for (int j = 0; j < NQ; ++j)
                            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fp[i], fq[j], acc[i][j], 0, 0, 0);
                }
                __builtin_amdgcn_s_setprio(0);
                asm volatile("" ::: "memory");
                if (h == kTurns - 1 && !second) __builtin_amdgcn_s_waitcnt(wait_for(kLanded, kAnyLds));
                turn();
            }
            rd = next(rd);
            wr = next(wr);
        }
        if (!second) turn();
    } else {
        for (int t = 0; t < steps; ++t) {
            // The step's loads have landed, and every wave is done with the
            // stage that is written next.
            __builtin_amdgcn_s_waitcnt(wait_for(kLanded, 0));
            asm volatile("" ::: "memory");
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            issue(t + NST - 1, wr);
            const char *sq = smem + rd * kStage, *sp = sq + BQ * SB;
            if constexpr (!FP8) {
#pragma unroll
                for (int kk = 0; kk < SB / 64; ++kk) {
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
                i32x8 fq[NQ];
                float xs[NQ];
                const f32x4 ws = w_scales(t);
#pragma unroll
                for (int j = 0; j < NQ; ++j) xs[j] = x_scale(t, j), fq[j] = both(rq.read(sq, j, 0), rq.read(sq, j, 1));
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    const i32x8 fp = both(rp.read(sp, i, 0), rp.read(sp, i, 1));
#pragma unroll
                    for (int j = 0; j < NQ; ++j) add_scaled(acc[i][j], mfma8(fp, fq[j]), xs[j] * w_scale(ws, i));
                }
            }
            rd = next(rd);
            wr = next(wr);
        }
    }

    // The tile goes through LDS, so that rows leave in 16-byte pieces of whole
    // lines (stored from the accumulators they leave as 8-byte pieces of 16
    // rows: 12 us per 256 x 256 tile), gradients already rounded.
    __builtin_amdgcn_s_waitcnt(wait_for(0, 0));
    if (MODE == kForward) {
        static_assert((BQ < 128 ? BQ : 128) * BP * 4 <= NST * kStage, "LDS");
        if (gated) forward_rows<true, BQ, BP, NW>(a, smem, acc, e, r0, p0, nq, wq, wp, lane);
        else forward_rows<false, BQ, BP, NW>(a, smem, acc, e, r0, p0, nq, wq, wp, lane);
    } else {
        static_assert(MODE == kForward || BQ * BP * 2 <= NST * kStage, "LDS");
        lds_barrier();
#pragma unroll
        for (int i = 0; i < NP; ++i)
#pragma unroll
            for (int j = 0; j < NQ; ++j) {
                const int q = wq + j * 16 + lane % 16, p = wp + i * 16 + lane / 16 * 4;
                *reinterpret_cast<u32x2 *>(smem + q * BP * 2 + (p / 8 ^ (q & 15)) * 16 + p % 8 * 2) =
                    u32x2{pack_bf16(acc[i][j][0], acc[i][j][1]), pack_bf16(acc[i][j][2], acc[i][j][3])};
            }
        lds_barrier();
        uint16_t *to = MODE == kDx ? a.d_x + r0 * a.I : a.d_w + we + (int64_t)q0 * a.I;
        constexpr int kPer = BP / 8, kApart = NW * kWave / kPer, kItems = BQ / kApart, kOnce = kItems < 8 ? kItems : 8;
        const int c = threadIdx.x % kPer, q0 = threadIdx.x / kPer;
        to += (int64_t)q0 * a.I + p0 + c * 8;
        if (p0 + c * 8 < P)
#pragma unroll
            for (int k0 = 0; k0 < kItems; k0 += kOnce) {
                u32x4 v[kOnce];
#pragma unroll
                for (int k = 0; k < kOnce; ++k) {
                    const int q = q0 + (k0 + k) * kApart;
                    v[k] = *reinterpret_cast<const u32x4 *>(smem + q * BP * 2 + (c ^ (q & 15)) * 16);
                }
#pragma unroll
                for (int k = 0; k < kOnce; ++k)
                    if (q0 + (k0 + k) * kApart < nq)
                        *reinterpret_cast<u32x4 *>(to + (int64_t)((k0 + k) * kApart) * a.I) = v[k];
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
#pragma unroll 8
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

template <int MODE, bool FP8, int BQ, int BP, int WQ, int WP, int SB, int NST>
hipError_t run_tile(const ExpertArgs &a, hipStream_t st) {
    const bool gated = MODE == kForward && a.act == kActSwiglu;
    const int64_t cols = ceil_div(MODE == kForward ? a.N : a.I, gated ? BP / 2 : BP);
    const int64_t tiles = MODE == kDw ? (int64_t)ceil_div(a.Nw, BQ) * a.E : row_tiles(a, BQ);
    const int64_t blocks = (tiles * cols + kXcds * kPatch - 1) / (kXcds * kPatch) * (kXcds * kPatch);
    if (blocks > 4294967295ll / (WQ * WP * kWave)) return hipErrorInvalidValue;
    hipLaunchKernelGGL((k_expert_tile<MODE, FP8, BQ, BP, WQ, WP, SB, NST>), dim3((uint32_t)blocks), dim3(WQ * WP * kWave),
                       0, st, a, (int)cols);
    return hipGetLastError();
}

// Microseconds that a product of `steps` 128-byte steps takes in tiles of BQ x
// BP: so many rounds of as many tiles as the card holds at once, each with a
// start and an epilogue; a step takes `full` in a round that fills the card,
// `least` with one tile alone.  Measured on 16 experts of 4 to 1024 rows, 2048
// to 2 x 1024 and 4096 to 2048 (at 192 rows: 72 us in 32-row tiles, 38 in
// 64-row, 34 in 128-row, 46 in 256-row tiles; at 1024 rows 302, 160, 131, 116).
double tile_cost(const ExpertArgs &a, bool dw, int columns, int BQ, int BP, int slots, int steps, double start,
                 double least, double full) {
    const int64_t some = a.rows < a.E ? a.rows : a.E;
    int64_t tiles = a.rows / BQ + some / 2;  // on average half a tile is missing from each expert's last
    tiles = dw ? (int64_t)a.E * ceil_div(a.Nw, BQ) : (tiles > some ? tiles : some);
    tiles *= ceil_div(columns, BP);
    const int64_t rounds = tiles / slots, rest = tiles % slots;
    return rounds * (start + steps * full) + (rest ? start + steps * (least + (full - least) * rest / slots) : 0.0);
}

template <int MODE, bool FP8>
hipError_t run(const ExpertArgs &a, hipStream_t st) {
    constexpr bool F = MODE == kForward, W = MODE == kDw;
    const int K = F ? a.I : (W ? (int)(a.rows / a.E) : a.Nw), steps = ceil_div(K, FP8 ? 128 : 64);
    const int columns = F ? a.Nw : a.I;
    const double c256 = tile_cost(a, W, columns, 256, 256, 256, steps, 8, 1.1, 1.85);
    const double c128 = tile_cost(a, W, columns, 128, 128, 512, steps, 5, 0.55, 1.15);
    if constexpr (!W) {
        const double c64 = tile_cost(a, W, columns, 64, 128, 512, steps, 3.5, 0.35, 0.7);
        const double c32 = F ? tile_cost(a, W, columns, 32, 64, 512, steps, 3, 0.2, 0.32)
                             : tile_cost(a, W, columns, 32, 128, 512, steps, 3, 0.3, 0.69);
        const double best = c64 < c32 ? c64 : c32;
        if (best <= c128 && best <= c256) {
            if (c64 < c32) return run_tile<MODE, FP8, 64, 128, 2, 2, 128, 3>(a, st);
            return run_tile<MODE, FP8, 32, F ? 64 : 128, F ? 2 : 1, F ? 2 : 4, 128, F ? 6 : 4>(a, st);
        }
    }
    if (c128 < c256) return run_tile<MODE, FP8, 128, 128, 2, 2, 128, 2>(a, st);
    return run_tile<MODE, FP8, 256, 256, 4, 2, FP8 ? 128 : 64, FP8 ? 2 : 5>(a, st);
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
