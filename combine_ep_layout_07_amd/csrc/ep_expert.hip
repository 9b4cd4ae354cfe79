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

    // `rows` rows (ALONG) or columns from `from` on, `pitch` bytes apart; gated:
    // alternating 16 of the gate, 16 of the up projection, whose rows are apart.
    // Along k the offsets grow with the row, so a bound at the end of the last
    // row turns the rows after it into zeros.  Across k columns outside do so by
    // the lane's offset, rows of k by issue's `left`.
    __device__ __forceinline__ void init(const char *from, uint32_t pitch, int rows, bool gated, int wave, int lane) {
        const int r = wave * kRows + lane / kLanes;
        int c = (lane % kLanes) ^ (((r & 3) | (r & 8) >> 1) << 1);
        if (ALONG) c = (lane % kLanes) ^ (SB == 128 ? r & 7 : r / 2 & 3);
        at = from;
        step = ALONG ? SB : SB / 2 * (int64_t)pitch;
        off = ALONG || c * 8 < rows ? (gated ? r / 32 * 16 + r % 16 : r) * pitch + c * 16 : kOutside;
        apart = NW * kRows / (gated ? 2 : 1) * pitch;
        bytes = !ALONG ? kOutside : (rows > 0 ? (rows - 1) * pitch + (pitch < SB ? pitch : SB) : 0);
        place = ALONG ? c : r;
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
__device__ __forceinline__ bool locate(const ExpertArgs &a, int block, int size, int cols, Segment &g, int &col) {
    int row;
    if (a.E > kWave) {
        if (!place_tile(block, count_tiles(a.base, a.E, a.rows, size), cols, row, col)) return false;
        g = find_tile(a.base, a.E, a.rows, size, row);
        return g.e >= 0;
    }
    const int lane = lane_id();
    g = lane < a.E ? segment_of(a.base, lane, a.rows) : Segment{lane, 0, 0};
    const int mine = (g.n + size - 1) / size, incl = wave_scan(mine);
    if (!place_tile(block, read_lane(incl, kWave - 1), cols, row, col)) return false;
    const uint64_t past = ballot(incl > row);
    if (!past) return false;
    const int o = __builtin_ctzll(past);
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
    __builtin_nontemporal_store(o, reinterpret_cast<bits *>(to));
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
// the up projection): the kept pre-activation, activation and residual; stored
// where `in`.
template <bool GATED, int W>
__device__ __forceinline__ void finish(const ExpertArgs &a, bool in, int64_t r, int c, float (&v)[W], const float (&up)[W],
                                       const uint32_t (&res)[W / 2]) {
    if (a.pre && in) {
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
    if (in) store_bf16<W>(a.out + r * a.N + c, v);
}

__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_s_waitcnt(wait_for(kAnyLoads, 0));
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// First column in the tile of a wave's fragment i; the wide tile's waves take
// columns of both halves.
template <int NP, bool WIDE>
__device__ __forceinline__ int column_of(int wp, int i) {
    return WIDE ? i / (NP / 2) * 128 + wp + i % (NP / 2) * 16 : wp + i * 16;
}

// The forward tile through LDS in fp32, as many rows at a time as fit, and the
// epilogue in row order: a thread keeps its eight columns, so their bias is
// loaded once, and has the residual of all its rows in flight before the sums
// are in LDS (loaded row by row the epilogue took half of a small product).
template <bool GATED, int BQ, int BP, int NW, int NP, int NQ, bool WIDE, typename ACC>
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
                    const int q = wq % kRowsPer + j * 16 + lane % 16, at = column_of<NP, WIDE>(wp, i) / 4 + lane / 16;
                    *reinterpret_cast<f32x4 *>(smem + q * BP * 4 + (at ^ (q & 7)) * 16) =
                        f32x4{acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
                }
        }
        lds_barrier();
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            // No branch around the arithmetic, so that items overlap.
            const int q = kItems * kApart > kRowsPer ? min(q0 + k * kApart, kRowsPer - 1) : q0 + k * kApart;
            const bool in = q0 + k * kApart < kRowsPer && h * kRowsPer + q < nq && c < a.N;
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
            finish<GATED, 8>(a, in, r0 + h * kRowsPer + q, c, v, up, res[k]);
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

// A tile's place: rows r0 .. r0 + nq of Q's side, columns p0 .. of P's, and the
// bases of both operands at k = 0.
struct Tile {
    int64_t r0, we;  // first row, first weight of the expert
    const char *q, *p;
    uint32_t pitchq, pitchp;  // bytes between rows
    int e, K, nq, np, q0, p0;
};

template <int MODE, bool FP8, int BQ, int BP>
__device__ __forceinline__ bool find(const ExpertArgs &a, int block, int cols, Tile &t) {
    constexpr int EL = FP8 ? 1 : 2;
    int tcol;
    Segment g;
    t.q0 = 0;
    if (MODE == kDw) {
        const int per = (a.Nw + BQ - 1) / BQ;
        int trow;
        if (!place_tile(block, per * a.E, cols, trow, tcol)) return false;
        g = segment_of(a.base, trow / per, a.rows);
        t.q0 = trow % per * BQ;
    } else if (!locate(a, block, BQ, cols, g, tcol)) {
        return false;
    }
    const bool gated = MODE == kForward && a.act == kActSwiglu;
    t.r0 = uniform64(g.r0);
    t.e = uniform(g.e);
    const int n = uniform(g.n);
    t.we = (int64_t)t.e * a.Nw * a.I;
    t.K = MODE == kForward ? a.I : (MODE == kDx ? a.Nw : n);
    t.p0 = tcol * (gated ? BP / 2 : BP);
    t.np = min((MODE == kForward ? a.N : a.I) - t.p0, gated ? BP / 2 : BP);
    t.nq = MODE == kDw ? min(a.Nw - t.q0, BQ) : n;
    const char *d = reinterpret_cast<const char *>(a.d), *x = static_cast<const char *>(a.x), *w = static_cast<const char *>(a.w);
    const uint32_t pitchx = a.I * EL, pitchd = a.Nw * 2;
    t.pitchq = MODE == kForward ? pitchx : pitchd;
    t.pitchp = pitchx;
    if (MODE == kForward) t.q = x + t.r0 * pitchx, t.p = w + (t.we + (int64_t)t.p0 * a.I) * EL;
    else if (MODE == kDx) t.q = d + t.r0 * pitchd, t.p = w + (t.we + t.p0) * 2;
    else t.q = d + t.r0 * pitchd + (int64_t)t.q0 * 2, t.p = x + t.r0 * pitchx + (int64_t)t.p0 * 2;
    return true;
}

// The fp8 scales of eight steps at a time in LDS, [row][8] for x, and for the
// weights the tile's two or three blocks of 128 weight rows: its columns', or
// gated the gate's one and the up projection's two at most.  (Loaded by each
// lane at each step they took a third of the time: a line for every row, every
// time anew.)
constexpr int kBlocks = 8;
template <int BQ, int NW>
__device__ __forceinline__ void load_scales(const ExpertArgs &a, const Tile &t, float (*sxs)[BQ * kBlocks], float (*sws)[kWave],
                                            bool gated, int kb0, int wave, int lane) {
    const int to = kb0 / kBlocks % 2, kb = kb0 + lane % kBlocks, nkb = a.I / 128;
    const __amdgpu_buffer_rsrc_t rx =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<float *>(a.x_sf + t.r0 * nkb), 0, kOutside, 0x00020000);
#pragma unroll
    for (int j = 0; j < BQ * kBlocks / kWave / NW; ++j) {
        const int row = (j * NW + wave) * (kWave / kBlocks) + lane / kBlocks;
        const uint32_t o = row < t.nq && kb < nkb ? (row * nkb + kb) * 4 : kOutside;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_char *)&sxs[to][(j * NW + wave) * kWave], 4, o, 0, 0, 0);
    }
    if (wave == 0) {
        const int blocks = (a.Nw + 127) / 128, slot = lane / kBlocks;
        const int block = gated && slot > 0 ? (a.N + t.p0) / 128 + slot - 1 : t.p0 / 128 + slot;
        const uint32_t o = slot < 3 && block < blocks && kb < nkb ? (block * nkb + kb) * 4 : kOutside;
        const __amdgpu_buffer_rsrc_t rw = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<float *>(a.w_sf + (int64_t)t.e * blocks * nkb), 0, kOutside, 0x00020000);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_char *)&sws[to][0], 4, o, 0, 0, 0);
    }
}
// The step's scale of a row of x, and of the weights' columns: [0] the first
// block (gated: the gate's), [1] the second (the up projection's first), [2]
// the up projection's second.
__device__ __forceinline__ float x_scale(const float *sxs, int row, int step) { return sxs[row * kBlocks + step % kBlocks]; }
__device__ __forceinline__ f32x4 w_scales(const float *sws, int step) {
    const float *s = sws + step % kBlocks;
    return f32x4{s[0], s[kBlocks], s[2 * kBlocks], 0.0f};
}

__device__ __forceinline__ i32x8 join(bf16x8 lo, bf16x8 hi) {
    return __builtin_shufflevector(__builtin_bit_cast(i32x4, lo), __builtin_bit_cast(i32x4, hi), 0, 1, 2, 3, 4, 5, 6, 7);
}
__device__ __forceinline__ f32x4 mfma8(i32x8 p, i32x8 q) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(p, q, f32x4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ void add_scaled(Four &c, f32x4 part, float sc) {
#pragma unroll
    for (int r = 0; r < 4; ++r) c[r] = fmaf(part[r], sc, c[r]);
    // Here and not later: left to itself the compiler holds the products of a
    // whole step until its end, which spills.
    asm volatile("" : "+v"(c[0]), "+v"(c[1]), "+v"(c[2]), "+v"(c[3]));
}

// The finished tile leaves through LDS, so that rows go out in 16-byte pieces
// of whole lines (stored from the accumulators they go as 8-byte pieces of 16
// rows: 12 us per 256 x 256 tile), gradients already rounded.  Nontemporal: all
// tiles finish together, and their lines would push the operands out of L2
// (unbalanced gradients 88 us, 73 with it).
template <int MODE, int BQ, int BP, int NW, int NP, int NQ, bool WIDE, typename ACC>
__device__ __forceinline__ void put_tile(const ExpertArgs &a, char *smem, ACC (&acc)[NP][NQ], const Tile &t, int wq, int wp, int lane) {
    __builtin_amdgcn_s_waitcnt(wait_for(0, 0));
    if (MODE == kForward) {
        if (a.act == kActSwiglu) forward_rows<true, BQ, BP, NW, NP, NQ, WIDE>(a, smem, acc, t.e, t.r0, t.p0, t.nq, wq, wp, lane);
        else forward_rows<false, BQ, BP, NW, NP, NQ, WIDE>(a, smem, acc, t.e, t.r0, t.p0, t.nq, wq, wp, lane);
        return;
    }
    lds_barrier();
#pragma unroll
    for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
            const int q = wq + j * 16 + lane % 16, p = column_of<NP, WIDE>(wp, i) + lane / 16 * 4;
            *reinterpret_cast<u32x2 *>(smem + q * BP * 2 + (p / 8 ^ (q & 15)) * 16 + p % 8 * 2) =
                u32x2{pack_bf16(acc[i][j][0], acc[i][j][1]), pack_bf16(acc[i][j][2], acc[i][j][3])};
        }
    lds_barrier();
    constexpr int kPer = BP / 8, kApart = NW * kWave / kPer, kItems = BQ / kApart, kOnce = kItems < 8 ? kItems : 8;
    const int c = threadIdx.x % kPer, q0 = threadIdx.x / kPer;
    if (c * 8 >= t.np) return;
    uint16_t *to = (MODE == kDx ? a.d_x + t.r0 * a.I : a.d_w + t.we + (int64_t)t.q0 * a.I) + (int64_t)q0 * a.I + t.p0 + c * 8;
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
            if (q0 + (k0 + k) * kApart < t.nq)
                __builtin_nontemporal_store(v[k], reinterpret_cast<u32x4 *>(to + (int64_t)((k0 + k) * kApart) * a.I));
    }
}

// Tiles of up to 128 x 128 by four waves, two workgroups on a CU: one reads
// while the other multiplies, by chance.  SB bytes of k per step, NST stages.
template <int MODE, bool FP8, int BQ, int BP, int WQ, int WP, int SB, int NST>
__global__ void __launch_bounds__(WQ *WP *kWave, 2) k_expert_tile(ExpertArgs a, int cols) {
    constexpr int NW = WQ * WP, NQ = BQ / WQ / 16, NP = BP / WP / 16;
    constexpr bool QA = MODE != kDw, PA = MODE == kForward;
    constexpr int kStage = (BQ + BP) * SB;
    __shared__ __align__(1024) char smem[NST * kStage];
    __shared__ float sxs[2][FP8 ? BQ * kBlocks : 1], sws[2][FP8 ? kWave : 1];
    const int lane = lane_id(), wave = uniform(threadIdx.x / kWave);
    const int wq = wave % WQ * (BQ / WQ), wp = wave / WQ * (BP / WP);
    const bool gated = MODE == kForward && a.act == kActSwiglu;
    Tile t;
    if (!find<MODE, FP8, BQ, BP>(a, blockIdx.x, cols, t)) return;

    Loader<QA, BQ, NW, SB> lq;
    Loader<PA, BP, NW, SB> lp;
    lq.init(t.q, t.pitchq, t.nq, false, wave, lane);
    lp.init(t.p, t.pitchp, t.np, gated, wave, lane);
    // Rows of the tile alternate between 16 of the gate and 16 of the up
    // projection; all of a wave's loads lie in one of the two.
    static_assert(MODE != kForward || NW * lp.kRows % 32 == 0, "a wave's loads keep their side");
    if (gated && wave * lp.kRows / 16 % 2) lp.at += (int64_t)a.N * t.pitchp;
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

    constexpr int EL = FP8 ? 1 : 2, kPerStep = SB / EL, kIssued = lq.kLoads + lp.kLoads;
    const int steps = (t.K + kPerStep - 1) / kPerStep;
    auto issue = [&](int s, int stage) {
        if constexpr (FP8)
            if (s % kBlocks == 0 && s < steps) load_scales<BQ, NW>(a, t, sxs, sws, gated, s, wave, lane);
        const int left = t.K - s * kPerStep;
        char *to = smem + stage * kStage;
        lq.issue(to, wave, QA ? left / (16 / EL) : left);
        lp.issue(to + BQ * SB, wave, PA ? left / (16 / EL) : left);
    };
    auto next = [](int stage) { return stage + 1 == NST ? 0 : stage + 1; };
    // The oldest step's loads are done when those of NST - 2 steps may be out.
    // (Loads end in order, and a step's scales are issued before its operands.)
    constexpr int kLanded = (NST - 2) * kIssued;
    static_assert(kLanded < kAnyLoads, "vmcnt");
    if (steps > 0)
        for (int s = 0; s < NST - 1; ++s) issue(s, s);
    int rd = 0, wr = NST - 1;
    const int up_from = ((a.N + t.p0) / 128 + 1) * 128 - a.N - t.p0;  // gated: up columns from here on take the third scale
    for (int s = 0; s < steps; ++s) {
        // The step's loads have landed, and every wave is done with the stage
        // that is written next.
        __builtin_amdgcn_s_waitcnt(wait_for(kLanded, 0));
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        issue(s + NST - 1, wr);
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
            const float *sx = sxs[s / kBlocks % 2];
            const f32x4 ws = w_scales(sws[s / kBlocks % 2], s);
#pragma unroll
            for (int j = 0; j < NQ; ++j) {
                xs[j] = x_scale(sx, wq + j * 16 + lane % 16, s);
                fq[j] = join(rq.read(sq, j, 0), rq.read(sq, j, 1));
            }
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const i32x8 fp = join(rp.read(sp, i, 0), rp.read(sp, i, 1));
                const float up = wp / 2 + i / 2 * 16 + lane / 16 * 4 < up_from ? ws[1] : ws[2];
                const float wsc = gated && i % 2 ? up : ws[0];
#pragma unroll
                for (int j = 0; j < NQ; ++j) add_scaled(acc[i][j], mfma8(fp, fq[j]), xs[j] * wsc);
            }
        }
        rd = next(rd);
        wr = next(wr);
    }
    static_assert((MODE == kForward ? (BQ < 128 ? BQ : 128) * BP * 4 : BQ * BP * 2) <= NST * kStage, "LDS");
    put_tile<MODE, BQ, BP, NW, NP, NQ, false>(a, smem, acc, t, wq, wp, lane);
}

// Tiles of 256 x 256 by eight waves, one workgroup on a CU.
//
// Two waves on each SIMD, of the two halves of the workgroup: one reads its
// fragments while the other keeps the matrix unit, and at the next barrier they
// change places; the second half runs one turn behind, held by one barrier more
// at the start.  A step is 128 bytes of k (whole lines: half lines cost the L2
// twice the requests) in two turns: Q's fragments and those of P's first half,
// then those of P's second half.
//
// LDS is a ring of R units of 16 KiB: the halves of 128 rows of Q (0, 1) and of
// P (2, 3) of a step.  Units 0 to 2 are free when the second half has read them
// in its first turn, unit 3 after its second, and each is refilled from the
// next turn on with the unit R further: one in a step's first turn, three in
// its second, two loads per wave each.  So R - 4 units are on their way at
// every wait, 6 to 10 turns before they are read.  (In stages of whole steps,
// or of half lines, the same product took 15 and 10% longer.)
constexpr int kUnit = 128 * 128;
template <int MODE, bool FP8, int R>
__device__ __forceinline__ void wide_tile(const ExpertArgs &a, int block, int cols, char *smem, float (*sxs)[256 * kBlocks],
                                          float (*sws)[kWave]) {
    constexpr int NW = 8, BQ = 256, BP = 256, NQ = 4, NP = 8, SB = 128;
    constexpr bool QA = MODE != kDw, PA = MODE == kForward;
    const int lane = lane_id(), wave = uniform(threadIdx.x / kWave);
    const int wq = wave % 4 * 64, wp = wave / 4 * 64;  // columns wp .. and 128 + wp ..
    const bool gated = MODE == kForward && a.act == kActSwiglu, second = wave >= 4;
    Tile t;
    if (!find<MODE, FP8, BQ, BP>(a, block, cols, t)) return;

    Loader<QA, 128, NW, SB> l0, l1;
    Loader<PA, 128, NW, SB> l2, l3;
    l0.init(t.q, t.pitchq, min(t.nq, 128), false, wave, lane);
    l1.init(t.q + (QA ? 128 * (int64_t)t.pitchq : 256), t.pitchq, t.nq - 128, false, wave, lane);
    const int ph = gated ? 64 : 128;
    l2.init(t.p, t.pitchp, min(t.np, ph), gated, wave, lane);
    l3.init(t.p + (PA ? ph * (int64_t)t.pitchp : 256), t.pitchp, t.np - ph, gated, wave, lane);
    if (gated && wave / 2 % 2) {  // a wave's loads are all the gate's or all the up projection's
        l2.at += (int64_t)a.N * t.pitchp;
        l3.at += (int64_t)a.N * t.pitchp;
    }
    Reader<QA, 128, SB> rq;
    Reader<PA, 128, SB> rp;
    rq.init(wq % 128, lane);
    rp.init(wp, lane);

    typename Sum<FP8>::type acc[NP][NQ];
#pragma unroll
    for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int j = 0; j < NQ; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[i][j][r] = 0.0f;

    constexpr int EL = FP8 ? 1 : 2, kPerStep = SB / EL;
    const int steps = (t.K + kPerStep - 1) / kPerStep;
    // Unit 4 s + kind into place `at` of the ring.
    auto issue = [&](int s, int kind, int at) {
        const int left = t.K - s * kPerStep, lq = QA ? left / (16 / EL) : left, lp = PA ? left / (16 / EL) : left;
        char *to = smem + at * kUnit;
        if constexpr (FP8)
            if (kind == 0 && s % kBlocks == 0 && s < steps) load_scales<BQ, NW>(a, t, sxs, sws, gated, s, wave, lane);
        if (kind == 0) l0.issue(to, wave, lq);
        else if (kind == 1) l1.issue(to, wave, lq);
        else if (kind == 2) l2.issue(to, wave, lp);
        else l3.issue(to, wave, lp);
    };
    auto wrap = [](int at) { return at >= R ? at - R : at; };
    auto turn = [] {
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
    };
    // Loads end in order: a unit's are done when those of the R - 4 after it
    // may be out.  Every wave waits for its own before the barrier after which
    // the first half reads them.
    constexpr int kLanded = (R - 4) * 2;
    static_assert(l0.kLoads == 2 && l2.kLoads == 2 && kLanded < kAnyLoads, "two loads per unit");
    const int up_from = ((a.N + t.p0) / 128 + 1) * 128 - a.N - t.p0;  // gated: up columns from here on take the third scale
    if (steps > 0) {
#pragma unroll
        for (int u = 0; u < R - 1; ++u) issue(u / 4, u % 4, u);
        __builtin_amdgcn_s_waitcnt(wait_for(kLanded, kAnyLds));
        asm volatile("" ::: "memory");
    }
    turn();
    if (second) turn();
    int at = 0;  // place of the step's unit 0
    for (int s = 0; s < steps; ++s) {
        const char *sq = smem + wrap(at + wave % 4 / 2) * kUnit;
        bf16x8 fq[NQ][2];
        float xs[NQ];
        f32x4 ws;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const char *sp = smem + wrap(at + 2 + h) * kUnit;
            bf16x8 fp[NP / 2][2];
            asm volatile("" ::: "memory");
            if (h == 0) {
                if (FP8) ws = w_scales(sws[s / kBlocks % 2], s);
#pragma unroll
                for (int j = 0; j < NQ; ++j) {
                    if (FP8) xs[j] = x_scale(sxs[s / kBlocks % 2], wq + j * 16 + lane % 16, s);
                    fq[j][0] = rq.read(sq, j, 0);
                    fq[j][1] = rq.read(sq, j, 1);
                }
            }
#pragma unroll
            for (int i = 0; i < NP / 2; ++i) {
                fp[i][0] = rp.read(sp, i, 0);
                fp[i][1] = rp.read(sp, i, 1);
            }
            if (h == 0) {
                issue(s + (R - 1) / 4, (R - 1) % 4, wrap(at + R - 1));
            } else {
                issue(s + R / 4, R % 4, at);
                issue(s + (R + 1) / 4, (R + 1) % 4, wrap(at + 1));
                issue(s + (R + 2) / 4, (R + 2) % 4, wrap(at + 2));
            }
            asm volatile("" ::: "memory");
            if (second) __builtin_amdgcn_s_waitcnt(wait_for(kLanded, 0));
            else __builtin_amdgcn_s_waitcnt(wait_for(kAnyLoads, 0));
            turn();
            __builtin_amdgcn_s_setprio(1);
            if constexpr (FP8) {
                // Two products at a time, then the scaling of the pair two
                // before, which is ready by then: closer together the matrix
                // unit idles until the scaling is done (595 us, 4096 tokens).
                constexpr int kPairs = NP / 2 * NQ / 2, kAfter = 2;
                f32x4 part[kAfter + 1][2];
#pragma unroll
                for (int u = 0; u < kPairs + kAfter; ++u) {
#pragma unroll
                    for (int v = 0; v < 2 && u < kPairs; ++v) {
                        const int i = u * 2 / NQ, j = u * 2 % NQ + v;
                        part[u % (kAfter + 1)][v] = mfma8(join(fp[i][0], fp[i][1]), join(fq[j][0], fq[j][1]));
                    }
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int v = 0; v < 2 && u >= kAfter; ++v) {
                        const int o = u - kAfter, i = o * 2 / NQ, j = o * 2 % NQ + v;
                        const int c = (h * 128 + wp) / 2 + i / 2 * 16 + lane / 16 * 4;
                        const float up = c < up_from ? ws[1] : ws[2];
                        const float wsc = gated ? (i % 2 ? up : ws[0]) : ws[h];
                        add_scaled(acc[h * (NP / 2) + i][j], part[o % (kAfter + 1)][v], xs[j] * wsc);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
            } else {
#pragma unroll
                for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                    for (int i = 0; i < NP / 2; ++i)
#pragma unroll
                        for (int j = 0; j < NQ; ++j)
                            acc[h * (NP / 2) + i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                fp[i][kk], fq[j][kk], acc[h * (NP / 2) + i][j], 0, 0, 0);
            }
            __builtin_amdgcn_s_setprio(0);
            asm volatile("" ::: "memory");
            if (!second) __builtin_amdgcn_s_waitcnt(wait_for(kLanded, kAnyLds));
            turn();
        }
        at = wrap(at + 4);
    }
    if (!second) turn();
    static_assert((MODE == kForward ? 128 * BP * 4 : BQ * BP * 2) <= R * kUnit, "LDS");
    put_tile<MODE, BQ, BP, NW, NP, NQ, true>(a, smem, acc, t, wq, wp, lane);
}

// All of LDS; with fp8 the scales take the room of two units.
template <bool FP8>
__global__ void __launch_bounds__(512, 2) k_expert_wide(ExpertArgs a, int cols) {
    __shared__ __align__(1024) char smem[(FP8 ? 8 : 10) * kUnit];
    __shared__ float sxs[FP8 ? 2 : 1][256 * kBlocks / (FP8 ? 1 : 256 * kBlocks)], sws[FP8 ? 2 : 1][FP8 ? kWave : 1];
    wide_tile<kForward, FP8, FP8 ? 8 : 10>(a, blockIdx.x, cols, smem, reinterpret_cast<float(*)[256 * kBlocks]>(sxs),
                                           reinterpret_cast<float(*)[kWave]>(sws));
}

// The gradients' tiles of 256 x 256 in one launch, those of d_x first (blocks
// below `dx`): the tiles of d_w, with few steps each, fill what the last ones of
// d_x leave idle.
__global__ void __launch_bounds__(512, 2) k_expert_wide_back(ExpertArgs a, int cols, int dx) {
    __shared__ __align__(1024) char smem[10 * kUnit];
    const int block = blockIdx.x;
    if (block < dx) wide_tile<kDx, false, 10>(a, block, cols, smem, nullptr, nullptr);
    else wide_tile<kDw, false, 10>(a, block - dx, cols, smem, nullptr, nullptr);
}

// Gradient of the pre-activation and the columns' sums of its unrounded values
// for d_bias.  It is stored as bf16, which the matrix unit takes: the error of d_x
// and d_w against 64 bits is 0.0023 of their norm with an activation and 0.0017,
// the results' own rounding, without; a second product with the remainder would
// double their time.  A workgroup takes 512 columns of one tile of kActRows
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
#pragma unroll
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

template <int MODE>
int64_t count_blocks(const ExpertArgs &a, int BQ, int BP, int threads, int *cols) {
    const bool gated = MODE == kForward && a.act == kActSwiglu;
    *cols = ceil_div(MODE == kForward ? a.N : a.I, gated ? BP / 2 : BP);
    const int64_t tiles = (MODE == kDw ? (int64_t)ceil_div(a.Nw, BQ) * a.E : row_tiles(a, BQ)) * *cols;
    const int64_t blocks = (tiles + kXcds * kPatch - 1) / (kXcds * kPatch) * (kXcds * kPatch);
    return blocks > 4294967295ll / threads ? 0 : blocks;
}

template <int MODE, bool FP8, int BQ, int BP, int WQ, int WP, int SB, int NST>
hipError_t run_tile(const ExpertArgs &a, hipStream_t st) {
    int cols;
    const int64_t blocks = count_blocks<MODE>(a, BQ, BP, WQ * WP * kWave, &cols);
    if (!blocks) return hipErrorInvalidValue;
    hipLaunchKernelGGL((k_expert_tile<MODE, FP8, BQ, BP, WQ, WP, SB, NST>), dim3((uint32_t)blocks), dim3(WQ * WP * kWave),
                       0, st, a, cols);
    return hipGetLastError();
}

template <bool FP8>
hipError_t run_wide(const ExpertArgs &a, hipStream_t st) {
    int cols;
    const int64_t blocks = count_blocks<kForward>(a, 256, 256, 512, &cols);
    if (!blocks) return hipErrorInvalidValue;
    hipLaunchKernelGGL(k_expert_wide<FP8>, dim3((uint32_t)blocks), dim3(512), 0, st, a, cols);
    return hipGetLastError();
}

// The gradients in wide tiles, one or both.
hipError_t run_wide_back(const ExpertArgs &a, bool d_x, bool d_w, hipStream_t st) {
    int cols;
    const int64_t bx = count_blocks<kDx>(a, 256, 256, 512, &cols), bw = count_blocks<kDw>(a, 256, 256, 512, &cols);
    const int64_t blocks = (d_x ? bx : 0) + (d_w ? bw : 0);
    if (!bx || !bw || blocks > 4294967295ll / 512) return hipErrorInvalidValue;
    hipLaunchKernelGGL(k_expert_wide_back, dim3((uint32_t)blocks), dim3(512), 0, st, a, cols, d_x ? (int)bx : 0);
    return hipGetLastError();
}

// Microseconds that a product of `steps` 128-byte steps takes in tiles of one
// size: so many rounds of as many tiles as the card holds at once, each with a
// start and an epilogue; a step takes `full` in a round that fills the card,
// `least` with one tile alone.  Fitted to 16 experts of 4 to 1024 rows, 2048 to
// 2 x 1024 and 4096 to 2048 features.  Forward, 4096 to 2048, at 4 rows: 40 us
// in 32-row tiles, 77 in 256-row tiles; at 128: 64 in 64-row, 66 in 128-row, 83
// in 256-row; at 256: 88 in 128-row, 90 in 256-row; at 1024: 273 in 128-row, 206
// in 256-row tiles.
template <int MODE, bool FP8>
double cost(const ExpertArgs &a, int BQ, int BP, int slots, double start, double least, double full) {
    const int64_t some = a.rows < a.E ? a.rows : a.E;
    int64_t tiles = a.rows / BQ + some / 2;  // on average half a tile is missing from each expert's last
    tiles = MODE == kDw ? (int64_t)a.E * ceil_div(a.Nw, BQ) : (tiles > some ? tiles : some);
    tiles *= ceil_div(MODE == kForward ? a.Nw : a.I, BP);
    const int steps = ceil_div(MODE == kForward ? a.I : (MODE == kDw ? a.rows / a.E : a.Nw), FP8 ? 128 : 64);
    const int64_t rounds = tiles / slots, rest = tiles % slots;
    return rounds * (start + steps * full) + (rest ? start + steps * (least + (full - least) * rest / slots) : 0.0);
}
template <int MODE, bool FP8>
double cost_wide(const ExpertArgs &a) {
    if (MODE == kDw) return cost<MODE, FP8>(a, 256, 256, 256, 7.7, 1.1, 1.43);
    return FP8 ? cost<MODE, FP8>(a, 256, 256, 256, 5, 1.55, 2.05) : cost<MODE, FP8>(a, 256, 256, 256, 5, 1.15, 1.55);
}
template <int MODE, bool FP8>
double cost_128(const ExpertArgs &a) {
    if (MODE == kDw) return cost<MODE, FP8>(a, 128, 128, 512, 3.4, 0.6, 1.0);
    return FP8 ? cost<MODE, FP8>(a, 128, 128, 512, 5, 1.15, 1.3) : cost<MODE, FP8>(a, 128, 128, 512, 5, 0.6, 1.0);
}
template <int MODE, bool FP8>
double cost_64(const ExpertArgs &a) {
    return FP8 ? cost<MODE, FP8>(a, 64, 128, 512, 3.5, 0.9, 1.1) : cost<MODE, FP8>(a, 64, 128, 512, 3.5, 0.4, 0.72);
}
template <int MODE, bool FP8>
double cost_32(const ExpertArgs &a) {
    if (MODE != kForward) return cost<MODE, FP8>(a, 32, 128, 512, 3, 0.3, 0.69);
    return FP8 ? cost<MODE, FP8>(a, 32, 64, 512, 3, 0.65, 0.7) : cost<MODE, FP8>(a, 32, 64, 512, 3, 0.2, 0.32);
}

// Rows of the cheapest tiles: 32, 64, 128 or 256 (d_w: 128 or 256).
template <int MODE, bool FP8>
int tile_rows(const ExpertArgs &a) {
    double c = cost_128<MODE, FP8>(a);
    int rows = 128;
    if (MODE != kDw) {
        const double c64 = cost_64<MODE, FP8>(a), c32 = cost_32<MODE, FP8>(a);
        if (c64 <= c) c = c64, rows = 64;
        if (c32 <= c) c = c32, rows = 32;
    }
    return cost_wide<MODE, FP8>(a) < c ? 256 : rows;
}
template <int MODE, bool FP8>
hipError_t run_small(const ExpertArgs &a, int rows, hipStream_t st) {
    constexpr bool F = MODE == kForward;
    if constexpr (MODE != kDw) {
        if (rows == 32) return run_tile<MODE, FP8, 32, F ? 64 : 128, F ? 2 : 1, F ? 2 : 4, 128, F ? 6 : 4>(a, st);
        if (rows == 64) return run_tile<MODE, FP8, 64, 128, 2, 2, 128, 3>(a, st);
    }
    return run_tile<MODE, FP8, 128, 128, 2, 2, 128, 2>(a, st);
}

template <bool FP8>
hipError_t run_forward(const ExpertArgs &a, hipStream_t st) {
    const int rows = tile_rows<kForward, FP8>(a);
    return rows == 256 ? run_wide<FP8>(a, st) : run_small<kForward, FP8>(a, rows, st);
}

// Both gradients go in one launch where both are best in wide tiles (565 us in
// two, 555 in one; 2331 rows of 24 experts, d_x best in 64-row tiles: 73 in two,
// 82 in one).
hipError_t run_back(const ExpertArgs &a, hipStream_t st) {
    const bool x = a.d_x && a.rows > 0, w = a.d_w;
    const int rows_x = tile_rows<kDx, false>(a), rows_w = tile_rows<kDw, false>(a);
    const bool wide_x = x && rows_x == 256, wide_w = w && rows_w == 256;
    hipError_t rc = hipSuccess;
    if (wide_x || wide_w) rc = run_wide_back(a, wide_x, wide_w, st);
    if (rc == hipSuccess && x && !wide_x) rc = run_small<kDx, false>(a, rows_x, st);
    if (rc == hipSuccess && w && !wide_w) rc = run_small<kDw, false>(a, rows_w, st);
    return rc;
}

}  // namespace

void expert_tiles(const ExpertArgs &a, int *forward, int *d_x, int *d_w) {
    *forward = a.fp8 ? tile_rows<kForward, true>(a) : tile_rows<kForward, false>(a);
    *d_x = a.fp8 ? 0 : tile_rows<kDx, false>(a);
    *d_w = a.fp8 ? 0 : tile_rows<kDw, false>(a);
}

hipError_t launch_expert(const ExpertArgs &a, hipStream_t st) {
    if (a.rows == 0) return hipSuccess;
    return a.fp8 ? run_forward<true>(a, st) : run_forward<false>(a, st);
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
    return run_back(a, st);
}

}  // namespace ep
