// MXFP4 grouped SwiGLU GEMMs on gfx950's block-scaled MFMA
// (v_mfma_scale_f32_32x32x64_f8f6f4 with both operands E2M1, one E8M0 scale
// per 32 k): the forward of the experts with weights and activations held in
// 4 bits.
//   gate/up  gu = x [Wg | Wu]^T, h = silu(g) * u   x row-wise (dispatch payload)
//   down     y = h Wd^T                            h row-wise (made by the gate/up epilogue)
// A 128-byte tile row is 256 codes, so tiles, LDS layout, device schedule and
// staged stores are those of the bf16 kernels with a K-step four times as
// deep.  A fragment of 32 rows x 64 k is 16 bytes per lane: lane i holds
// row (i & 31)'s 32 codes of k-block (i >> 5), and its scale operand that
// block's scale (checked on the hardware against a host product with random
// codes and scales, in all four byte positions of the scale operand).
#include <algorithm>

#include "gemm_common.h"
#include "mx4.h"

namespace moe {
namespace {

using namespace gemm;

typedef __attribute__((ext_vector_type(8))) int i32x8;
typedef __attribute__((ext_vector_type(4))) float f32x4_t;

constexpr int KB = 256;          // codes per K-step (128 bytes per row)
constexpr int NW4 = 8;           // waves per workgroup



// K-major MXFP4 operand rows: codes [rows][K/2] bytes, scales [rows][K/32]
struct Src4 {
    const uint8_t* c0;   // codes of rows [0, half)
    const uint8_t* c1;   // codes of rows [half, 2*half)
    const uint8_t* s0;   // scales of the same rows
    const uint8_t* s1;
    int rows0, rows1;
    int K;               // multiple of 128
};

__device__ __forceinline__ TileSrc codes_as_tile(const Src4& s)
{
    TileSrc t;           // four codes per 16-bit "element"
    t.p0 = reinterpret_cast<const uint16_t*>(s.c0);
    t.p1 = reinterpret_cast<const uint16_t*>(s.c1);
    t.ld = s.K / 4;
    t.rows0 = s.rows0;
    t.rows1 = s.rows1;
    t.K = (s.K + KB - 1) / KB * 64;   // whole K-steps: what lies past K is loaded and never multiplied
    return t;
}

__device__ __forceinline__ i32x8 read_frag4(const uint8_t* tile, int row_base, int ks, int lane)
{
    const int row = row_base + (lane & 31);
    const uint4 v = *reinterpret_cast<const uint4*>(tile + row * 128 + lds_chunk<false, 64>(row, ks * 2 + (lane >> 5)) * 16);
    return i32x8{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
}

// acc += a b^T over 64 k; sel: byte of the scale words (this lane's k-block)
template <int SEL>
__device__ __forceinline__ f32x16 mfma4(i32x8 b, i32x8 a, f32x16 acc, uint32_t sb, uint32_t sa)
{
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b, a, acc, 4, 4, SEL, (int)sb, SEL, (int)sa);
}

// LDS: stages of codes, then two stages of scales.  A scale stage holds 16
// bytes of every operand row (512 codes, two K-steps), A rows first: read a
// K-step at a time, 4 bytes per 128 codes, every row would cost a cache line
// per K-step, as much traffic as the codes.  The loads of a row's last 16
// bytes may run into the next row (never multiplied) or past the descriptor's
// range, where each 4-byte word by itself reads zero (checked on the hardware).
constexpr int SROWS = 512;
constexpr int SSTAGE = SROWS * 16;

// this wave's 64 rows of a scale stage: rows 64 w .. 64 w + 63 of A's BM rows
// followed by B's 256
template <int BM>
struct ScaleLoader4 {
    desc_t d;
    uint32_t off;
    uint32_t lds;     // LDS byte address of the wave's rows in stage 0
    __device__ __forceinline__ void init(const Src4& a, const Src4& b, uint32_t lds_scales)
    {
        const int lane = threadIdx.x & 63;
        const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int row = w * 64;
        const int ld = a.K / 32;
        const bool isb = row >= BM;
        const int r = isb ? row - BM : row;
        // a 64-row A tile keeps its two 32-row halves in one wave's rows: they are consecutive in memory
        const int half = BM == 64 && !isb ? 64 : (isb ? 128 : BM / 2);
        const bool hi = r >= half;
        const uint8_t* base = isb ? (hi ? b.s1 : b.s0) : (hi ? a.s1 : a.s0);
        const int rows = isb ? (hi ? b.rows1 : b.rows0) : (BM == 64 ? a.rows0 + a.rows1 : (hi ? a.rows1 : a.rows0));
        const bool none = row >= BM + BN;
        d = wave_uniform(make_desc(base, none ? 0 : (int64_t)rows * ld));
        off = none ? kOOB : (uint32_t)((r - (hi ? half : 0) + lane) * ld);
        lds = lds_scales + (uint32_t)row * 16u;
    }
    // chunk c (two K-steps) into its stage; outside: zeros
    __device__ __forceinline__ void issue(int c, bool inside = true)
    {
        dma16_to_lds_at(d, lds + (uint32_t)(c & 1) * SSTAGE, off, inside ? (uint32_t)c * 16u : d[2]);
    }
};

// the scale word of half K-step hs (128 k) of scale-stage row `row`, shifted
// so that bytes 0 and 2 are this lane's k-blocks of its two k-slices
__device__ __forceinline__ uint32_t scale_word(const uint8_t* scales, int row, int hs, int lane)
{
    return *reinterpret_cast<const uint32_t*>(scales + ((hs >> 2) & 1) * SSTAGE + (row + (lane & 31)) * 16 + (hs & 3) * 4);
}

// BM x 256 tile (BM = 64, 128: the tail tiles) through a ring of three LDS
// stages: the loads of K-step kt + 2 go out while K-step kt's MFMAs run, also
// past the end of K, where they write zeros to a stage nobody reads, so that
// the wait at each K-step counts a known number of younger operations.
template <int BM>
__device__ __forceinline__ void mainloop4(const Src4& sa, const Src4& sb, f32x16 (&acc)[BM / 64][2], uint8_t* smem)
{
    constexpr int MI = BM / 64, NJ = 2, NS = 3;
    constexpr int STAGE = (BM + BN) * 128;
    using LA = DirectLoader<BM, 64, false, NW4>;
    using LB = DirectLoader<BN, 64, false, NW4>;
    constexpr int NQ = LA::PER_WAVE + LB::PER_WAVE;
    uint8_t* scales = smem + NS * STAGE;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int wm = WL<NW4>::wm(wave), wn = WL<NW4>::wn(wave);
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
    const int nk = (sa.K + KB - 1) / KB;
    LA la;
    LB lb;
    ScaleLoader4<BM> sc;
    la.init(codes_as_tile(sa), lds_addr(smem));
    lb.init(codes_as_tile(sb), lds_addr(smem + BM * 128));
    sc.init(sa, sb, lds_addr(scales));
    auto issue = [&](int kt) __attribute__((always_inline)) {
        const bool inside = kt < nk;
        const uint32_t so = (uint32_t)(kt % NS) * STAGE;
        if ((kt & 1) == 0) sc.issue(kt >> 1, inside);
#pragma unroll
        for (int q = 0; q < LA::PER_WAVE; ++q) la.issue_ring(so, kt, q, inside);
#pragma unroll
        for (int q = 0; q < LB::PER_WAVE; ++q) lb.issue_ring(so, kt, q, inside);
    };
#pragma unroll
    for (int j = 0; j < NS - 1; ++j) issue(j);
    for (int kt = 0; kt < nk; ++kt) {
        // younger operations: K-step kt + 1's, with a scale load when it is even
        if (kt & 1) wait_vmcnt<NQ + 1>();
        else wait_vmcnt<NQ>();
        __syncthreads();
        issue(kt + NS - 1);
        const uint8_t* a_s = smem + (kt % NS) * STAGE;
        const uint8_t* b_s = a_s + BM * 128;
        auto half = [&](int h) __attribute__((always_inline)) {
            const int hs = kt * 2 + h;
            uint32_t wa[MI], wb[NJ];
#pragma unroll
            for (int i = 0; i < MI; ++i)
                wa[i] = scale_word(scales, wm * (BM / 2) + i * 32, hs, lane) >> (8 * (lane >> 5));
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                wb[j] = scale_word(scales, BM + WL<NW4>::sub_col(wn, j), hs, lane) >> (8 * (lane >> 5));
            i32x8 af[2][MI], bf[2][NJ];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
#pragma unroll
                for (int i = 0; i < MI; ++i) af[q][i] = read_frag4(a_s, wm * (BM / 2) + i * 32, h * 2 + q, lane);
#pragma unroll
                for (int j = 0; j < NJ; ++j) bf[q][j] = read_frag4(b_s, WL<NW4>::sub_col(wn, j), h * 2 + q, lane);
            }
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < NJ; ++j) acc[i][j] = mfma4<0>(bf[0][j], af[0][i], acc[i][j], wb[j], wa[i]);
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < NJ; ++j) acc[i][j] = mfma4<2>(bf[1][j], af[1][i], acc[i][j], wb[j], wa[i]);
        };
        half(0);
        if (kt * KB + 128 < sa.K) half(1);
    }
    wait_vmcnt<0>();   // the zero loads past K have landed too
    __syncthreads();
}

// this wave's direct loads of half of a 256-row operand tile: 1 KB chunks
// half*16 + 4i + w4, i = 0..3, of the 32 of a K-step
struct HalfLoader4 {
    desc_t d;
    uint32_t off[4];
    uint32_t m0w;
    __device__ __forceinline__ void init(const Src4& s, uint32_t lds_tile, int half, int w4)
    {
        const int lane = threadIdx.x & 63;
        m0w = lds_tile + (uint32_t)(half * 16 + w4) * 1024u;
        d = wave_uniform(half ? make_desc(s.c1, (int64_t)s.rows1 * (s.K / 2)) : make_desc(s.c0, (int64_t)s.rows0 * (s.K / 2)));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = (half * 16 + i * 4 + w4) * 8 + lane / 8;
            off[i] = (uint32_t)((row - half * 128) * (s.K / 2)) + lds_chunk<false, 64>(row, lane % 8) * 16u;
        }
    }
    __device__ __forceinline__ void issue(uint32_t stage_off, int kt)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            dma16_to_lds_at(d, m0w + stage_off + (uint32_t)i * 4096u, off[i], (uint32_t)kt * 128u);
    }
};

// Ping-pong main loop of a 256 x 256 tile: the two waves of a SIMD belong to
// different groups (waves 0..3: tile rows 0..127, waves 4..7: rows 128..255)
// that alternate, tick by tick, between a compute tick (the 16 MFMAs of a half
// K-step from registers, with the next half's 12 fragments and 6 scale words
// read from LDS in their shadow) and a memory tick (this wave's 4 direct loads
// of a quarter of a K-step); group 1 runs one tick behind group 0 and a
// barrier ends every tick, so on every SIMD one wave feeds the matrix unit
// while the other issues loads.  An MXFP4 fragment is 16 bytes per lane, as a
// bf16 one is, and its MFMA as long, so the schedule is the bf16 kernels':
// the quarters of K-step j (two LDS stages) go out at ticks 4j-7 (A rows
// 0..127, group 0), 4j-6 (B half 0, group 1), 4j-5 (B half 1, group 0) and
// 4j-4 (A rows 128..255, group 1); group 0 reads K-step j at ticks 4j-2 and
// 4j, group 1 at 4j-1 and 4j+1.  The scales of K-steps 2c, 2c+1 go out ahead
// of the first quarter a group loads of K-step 2c (A's at tick 8c-7 by group
// 0, B's at 8c-6 by group 1), after the last read of their stage (8c-11).
// When K is an odd multiple of 128, the last half K-step is loaded and read
// like any other and its MFMAs are left out.
__device__ __forceinline__ void mainloop4_pp(const Src4& sa, const Src4& sb, f32x16 (&acc)[4][2], uint8_t* smem)
{
    constexpr int BM = 256, MI = 4, NJ = 2;
    constexpr int STAGE = (BM + BN) * 128;
    uint8_t* scales = smem + 2 * STAGE;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = wave >> 2;    // group
    const int w4 = wave & 3;    // wave column (and SIMD)
    const int sh = 8 * (lane >> 5);
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

    const int nk = (sa.K + KB - 1) / KB;
    const int H = 2 * nk;       // half K-steps
    const bool whole = sa.K % KB == 0;
    HalfLoader4 ha, hb;
    ScaleLoader4<BM> sc;
    ha.init(sa, lds_addr(smem), g, w4);
    hb.init(sb, lds_addr(smem + BM * 128), 1 - g, w4);
    sc.init(sa, sb, lds_addr(scales));
    sc.issue(0);
    ha.issue(0, 0);
    hb.issue(0, 0);
    if (nk > 1) {
        ha.issue(STAGE, 1);
        hb.issue(STAGE, 1);
        wait_vmcnt<8>();
    } else {
        wait_vmcnt<0>();
    }
    __syncthreads();

    // fragments of one 64-deep k-slice: 4 A sub-tiles, 2 B sub-tiles
    struct Slot {
        i32x8 a[MI], b[NJ];
    };
    struct Words {
        uint32_t a[MI], b[NJ];
    };
    // LDS offsets of this lane's part of a fragment, per k-slice of a K-step:
    // the chunk swizzle depends on the lane alone, so sub-tiles are constant
    // offsets from one address
    uint32_t vo[4];
#pragma unroll
    for (int ks = 0; ks < 4; ++ks)
        vo[ks] = (uint32_t)((lane & 31) * 128) + lds_chunk<false, 64>(lane & 31, ks * 2 + (lane >> 5)) * 16u;
    const uint32_t vs = (uint32_t)(2 * STAGE + (lane & 31) * 16);
    // where half K-step hs is read: scalars, opaque so that the per-lane
    // addresses are made where they are used and not kept for every stage
    struct At {
        uint32_t a, b, s;
    };
    auto at = [&](int hs) __attribute__((always_inline)) {
        const uint32_t st = (uint32_t)((hs >> 1) & 1) * STAGE;
        At r{st + (uint32_t)g * (128 * 128), st + BM * 128 + (uint32_t)w4 * (32 * 128),
             (uint32_t)((hs >> 2) & 1) * SSTAGE + (uint32_t)(hs & 3) * 4u};
        asm volatile("" : "+s"(r.a), "+s"(r.b), "+s"(r.s));
        return r;
    };
    // fragment m (A 0..3, B 4..5) of k-slice s2 of half K-step hs
    auto read_one = [&](const At& p, int odd, int s2, int m, Slot& dst) __attribute__((always_inline)) {
        const uint32_t v = vo[odd * 2 + s2];
        const uint4 x = m < MI ? *reinterpret_cast<const uint4*>(smem + (v + p.a) + m * (32 * 128))
                               : *reinterpret_cast<const uint4*>(smem + (v + p.b) + (m - MI) * (128 * 128));
        const i32x8 f = {(int)x.x, (int)x.y, (int)x.z, (int)x.w, 0, 0, 0, 0};
        if (m < MI) dst.a[m] = f;
        else dst.b[m - MI] = f;
    };
    auto read_word = [&](const At& p, int m, Words& w) __attribute__((always_inline)) {
        const uint32_t x = *reinterpret_cast<const uint32_t*>(
            smem + (vs + p.s) + (m < MI ? (uint32_t)g * 2048u : 4096u + (uint32_t)w4 * 512u) +
            (m < MI ? m * 512 : (m - MI) * 2048));
        if (m < MI) w.a[m] = x;
        else w.b[m - MI] = x;
    };
    auto barrier = [&]() __attribute__((always_inline)) {
        __builtin_amdgcn_sched_barrier(0);
        __syncthreads();
        __builtin_amdgcn_sched_barrier(0);
    };
    // A compute tick: the 16 MFMAs of k-slices p (first) and c1 (second) under
    // the scale words w; with RD, what half K-step hs needs is read in their
    // shadow: its second k-slice into n1, its scale words into wn, its first
    // k-slice into p, each register once the MFMAs that use it have issued.
    // The tick's barrier (after `waits`) comes kAfter MFMAs before the end, so
    // that the other group's first ones queue up behind this one's last: with
    // the barrier after all 16 the matrix unit idled a quarter of the time.
    constexpr int kAfter = 3;
    auto compute = [&](auto RD, auto ODD, int hs, Slot& p, Slot& c1, Slot& n1, Words& w, Words& wn,
                       auto&& waits) __attribute__((always_inline)) {
        constexpr int odd = decltype(ODD)::value;
        At pt{};
        if constexpr (decltype(RD)::value) pt = at(hs);
        __builtin_amdgcn_s_setprio(1);   // ahead of the memory-phase wave of this SIMD
#pragma unroll
        for (int n = 0; n < 16; ++n) {
            const int i = (n >> 1) & 3, j = n & 1;
            if (n == 16 - kAfter) {
                waits();
                barrier();
            }
            if (n < 8) acc[i][j] = mfma4<0>(p.b[j], p.a[i], acc[i][j], w.b[j], w.a[i]);
            else acc[i][j] = mfma4<2>(c1.b[j], c1.a[i], acc[i][j], w.b[j], w.a[i]);
            if constexpr (decltype(RD)::value) {
                if (n < 3) {
                    read_one(pt, odd, 1, 2 * n, n1);
                    read_one(pt, odd, 1, 2 * n + 1, n1);
                }
                if (n == 3 || n == 5) {
#pragma unroll
                    for (int m = 0; m < 3; ++m) read_word(pt, (n - 3) / 2 * 3 + m, wn);
                }
                if (n == 2 || n == 4 || n == 6 || n == 8) read_one(pt, odd, 0, n / 2 - 1, p);
                if (n == 8 || n == 9) read_one(pt, odd, 0, n - 4, p);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        // the MFMAs belong to this tick: the compiler would sink some of them
        // past the branches that follow (with 190 spilled registers)
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j) asm volatile("" : "+v"(acc[i][j]));
        __builtin_amdgcn_s_setprio(0);
    };
    // the scale words read in the last compute tick, shifted for this lane's
    // k-blocks (in memory ticks: not between the barrier and the MFMAs)
    auto shift = [&](Words& w) __attribute__((always_inline)) {
#pragma unroll
        for (int m = 0; m < MI; ++m) w.a[m] >>= sh;
#pragma unroll
        for (int m = 0; m < NJ; ++m) w.b[m] >>= sh;
    };
    // this wave's direct loads of memory tick t
    auto loads = [&](int t) __attribute__((always_inline)) {
        int j;
        if (g == 0) {
            if ((t & 3) == 1) {          // A half 0 of K-step j, the A scales of K-steps j, j + 1
                j = (t + 7) >> 2;
                if (j >= 2 && j < nk) {
                    if ((j & 1) == 0) sc.issue(j >> 1);
                    ha.issue((uint32_t)(j & 1) * STAGE, j);
                }
            } else {                     // t % 4 == 3: B half 1
                j = (t + 5) >> 2;
                if (j >= 2 && j < nk) hb.issue((uint32_t)(j & 1) * STAGE, j);
            }
        } else {
            if ((t & 3) == 2) {          // B half 0 of K-step j, the B scales of K-steps j, j + 1
                j = (t + 6) >> 2;
                if (j >= 2 && j < nk) {
                    if ((j & 1) == 0) sc.issue(j >> 1);
                    hb.issue((uint32_t)(j & 1) * STAGE, j);
                }
            } else {                     // t % 4 == 0: A half 1
                j = (t + 4) >> 2;
                if (j >= 2 && j < nk) ha.issue((uint32_t)(j & 1) * STAGE, j);
            }
        }
    };
    // end of tick t: what the next tick reads has landed, then the barrier.
    // What was issued this tick (or, for group 1 at t % 4 == 1, the tick
    // before) may stay in flight: 4 loads, and the scales ahead of them when
    // they went out this tick
    auto waits = [&](int t) __attribute__((always_inline)) {
        if ((t & 3) == 1) {
            const int j = (t + 3) >> 2;
            const int jn = g == 0 ? j + 1 : j;
            if (jn < 2 || jn >= nk) wait_vmcnt<0>();
            else if (g == 0 && (jn & 1) == 0) wait_vmcnt<5>();
            else wait_vmcnt<4>();
        } else if ((t & 3) == 2 && g == 1) {
            const int jn = ((t + 2) >> 2) + 1;
            if (jn < 2 || jn >= nk) wait_vmcnt<0>();
            else if ((jn & 1) == 0) wait_vmcnt<5>();
            else wait_vmcnt<4>();
        }
    };
    auto end_tick = [&](int t) __attribute__((always_inline)) {
        waits(t);
        barrier();
    };
    auto none = []() __attribute__((always_inline)) {};
    auto wait4 = []() __attribute__((always_inline)) { wait_vmcnt<4>(); };
    const std::integral_constant<bool, true> rd;
    const std::integral_constant<bool, false> no_rd;
    const std::integral_constant<int, 1> odd;    // of the half K-step that is read
    const std::integral_constant<int, 0> even;
    Slot sp, sq, sr;   // first k-slice; second k-slice, alternating between sq and sr
    Words wq, wr;
    auto read_all = [&]() __attribute__((always_inline)) {
        const At p0 = at(0);
#pragma unroll
        for (int m = 0; m < 6; ++m) read_one(p0, 0, 0, m, sp);
#pragma unroll
        for (int m = 0; m < 6; ++m) read_one(p0, 0, 1, m, sq);
#pragma unroll
        for (int m = 0; m < 6; ++m) read_word(p0, m, wq);
    };

    // the last half K-step, in tick t
    auto last = [&](int t) __attribute__((always_inline)) {
        if (whole) compute(no_rd, even, 0, sp, sr, sq, wr, wq, [&] { waits(t); });
        else end_tick(t);
    };
    // Two K-steps (2c, 2c + 1; their loads are of 2c + 2, 2c + 3) are eight
    // ticks whose loads and waits are known when all of those K-steps exist
    // (and, for group 1, c > 0): no branches there.  With the conditions
    // tested in every tick, and the barrier after the last MFMA, a tick took 800
    // cycles; so it takes 625 (16 MFMAs are 512).
    if (g == 0) {
        read_all();
        shift(wq);
        int u = 0;
        for (int c = 0; 2 * c + 3 < nk; ++c, u += 4) {
            compute(rd, odd, u + 1, sp, sq, sr, wq, wr, none);                       // tick 8c
            sc.issue(c + 1);
            ha.issue(0, 2 * c + 2);
            shift(wr);
            wait_vmcnt<5>();
            barrier();
            compute(rd, even, u + 2, sp, sr, sq, wr, wq, none);                      // tick 8c+2
            hb.issue(0, 2 * c + 2);
            shift(wq);
            barrier();
            compute(rd, odd, u + 3, sp, sq, sr, wq, wr, none);                       // tick 8c+4
            ha.issue(STAGE, 2 * c + 3);
            shift(wr);
            wait_vmcnt<4>();
            barrier();
            compute(rd, even, u + 4, sp, sr, sq, wr, wq, none);                      // tick 8c+6
            hb.issue(STAGE, 2 * c + 3);
            shift(wq);
            barrier();
        }
        for (; u + 2 < H; u += 2) {
            compute(rd, odd, u + 1, sp, sq, sr, wq, wr, [&] { waits(2 * u); });      // tick 2u
            loads(2 * u + 1);                                    // tick 2u+1
            shift(wr);
            end_tick(2 * u + 1);
            compute(rd, even, u + 2, sp, sr, sq, wr, wq, [&] { waits(2 * u + 2); }); // tick 2u+2
            loads(2 * u + 3);                                    // tick 2u+3
            shift(wq);
            end_tick(2 * u + 3);
        }
        compute(rd, odd, u + 1, sp, sq, sr, wq, wr, [&] { waits(2 * u); });      // tick 2H-4
        loads(2 * u + 1);
        shift(wr);
        end_tick(2 * u + 1);
        last(2 * u + 2);                                         // tick 2H-2
        loads(2 * u + 3);
        end_tick(2 * u + 3);
    } else {
        loads(0);                                                // tick 0
        read_all();
        shift(wq);
        end_tick(0);
        int u = 0;
        auto generic = [&](int end) __attribute__((always_inline)) {
            for (; u + 2 < end; u += 2) {
                compute(rd, odd, u + 1, sp, sq, sr, wq, wr, [&] { waits(2 * u + 1); });  // tick 2u+1
                loads(2 * u + 2);                                // tick 2u+2
                shift(wr);
                end_tick(2 * u + 2);
                compute(rd, even, u + 2, sp, sr, sq, wr, wq, [&] { waits(2 * u + 3); }); // tick 2u+3
                loads(2 * u + 4);                                // tick 2u+4
                shift(wq);
                end_tick(2 * u + 4);
            }
        };
        if (nk > 5) {
            generic(5);
            for (int c = 1; 2 * c + 3 < nk; ++c, u += 4) {
                compute(rd, odd, u + 1, sp, sq, sr, wq, wr, wait4);                      // tick 8c+1
                sc.issue(c + 1);
                hb.issue(0, 2 * c + 2);
                shift(wr);
                wait_vmcnt<5>();
                barrier();
                compute(rd, even, u + 2, sp, sr, sq, wr, wq, none);                      // tick 8c+3
                ha.issue(0, 2 * c + 2);
                shift(wq);
                barrier();
                compute(rd, odd, u + 3, sp, sq, sr, wq, wr, wait4);                      // tick 8c+5
                hb.issue(STAGE, 2 * c + 3);
                shift(wr);
                wait_vmcnt<4>();
                barrier();
                compute(rd, even, u + 4, sp, sr, sq, wr, wq, none);                      // tick 8c+7
                ha.issue(STAGE, 2 * c + 3);
                shift(wq);
                barrier();
            }
        }
        generic(H);
        compute(rd, odd, u + 1, sp, sq, sr, wq, wr, [&] { waits(2 * u + 1); });  // tick 2H-3
        loads(2 * u + 2);
        shift(wr);
        end_tick(2 * u + 2);
        last(2 * u + 3);                                         // tick 2H-1
    }
}

// The tile of this workgroup in schedule_m's order (expert-major; a contiguous
// range of tiles per XCD), with every lane's group bounds loaded at once and
// the chosen expert's taken from the lane that holds them: one round trip to
// memory ahead of the operands instead of three, which nothing hides with one
// workgroup per CU (268 rows of 128 experts, d = 4096, f = 1536: gate/up 152 ->
// 141 us, down 101 -> 86; 65536 rows 656 -> 634 and 418 -> 383).  With 64-row
// tiles all column tiles of a row tile go before the next: they run together
// and share its rows.
template <int PER, int BM>   // experts per lane, E <= 64 PER; M-tiles of BM rows
__device__ __forceinline__ bool schedule_per(const int32_t* group_off, int capacity, int E, int64_t n_rows64, int ntn,
                                             MTile& t)
{
    const int lane = threadIdx.x & 63;
    const int gb = lane * PER;
    const int n_rows = (int)n_rows64;   // below 2^31
    int bnd[PER + 1];
    if (capacity > 0) {
#pragma unroll
        for (int k = 0; k <= PER; ++k) bnd[k] = (int)min((int64_t)min(gb + k, E) * capacity, n_rows64);
    } else {
#pragma unroll
        for (int k = 0; k <= PER; ++k) bnd[k] = group_off[min(gb + k, E)];
    }
    int cnt = 0, c[PER];
#pragma unroll
    for (int k = 0; k <= PER; ++k) bnd[k] = min(max(bnd[k], 0), n_rows);
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        c[k] = (int)((uint32_t)(max(bnd[k + 1] - bnd[k], 0) + BM - 1) / BM) * ntn;
        cnt += c[k];
    }
    // inclusive scan by lane permutations: within rows of 16 (row_shr 1, 2, 4,
    // 8), then each row's last lane into the rows behind it (row_bcast 15, 31)
    int incl = cnt;
    incl += __builtin_amdgcn_update_dpp(0, incl, 0x111, 0xF, 0xF, true);
    incl += __builtin_amdgcn_update_dpp(0, incl, 0x112, 0xF, 0xF, true);
    incl += __builtin_amdgcn_update_dpp(0, incl, 0x114, 0xF, 0xF, true);
    incl += __builtin_amdgcn_update_dpp(0, incl, 0x118, 0xF, 0xF, true);
    incl += __builtin_amdgcn_update_dpp(0, incl, 0x142, 0xA, 0xF, true);
    incl += __builtin_amdgcn_update_dpp(0, incl, 0x143, 0xC, 0xF, true);
    const int total = __builtin_amdgcn_readlane(incl, 63);
    const int per_xcd = (total + 7) / 8;
    const int slot = blockIdx.x / 8;
    const int L = (int)(blockIdx.x % 8) * per_xcd + slot;
    if (slot >= per_xcd || L >= total) return false;
    int run = incl - cnt;
    const int src = __ffsll((unsigned long long)__ballot(run <= L && L < incl)) - 1;
    int e = gb, first = run, b0 = 0, rows = 0;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        if (L >= run && L < run + c[k]) {
            e = gb + k;
            first = run;
            b0 = bnd[k];
            rows = bnd[k + 1] - bnd[k];
        }
        run += c[k];
    }
    t.e = __builtin_amdgcn_readlane(e, src);
    const int local = L - __builtin_amdgcn_readlane(first, src);
    const int m_e = __builtin_amdgcn_readlane(rows, src);
    grouped_tile(local, (m_e + BM - 1) / BM, ntn, BM == 64 ? 1 : kMTileGroup, t.mt, t.nt);
    t.row0 = (int64_t)__builtin_amdgcn_readlane(b0, src) + (int64_t)t.mt * BM;
    t.rows_valid = min(BM, m_e - t.mt * BM);
    return true;
}
template <int BM>
__device__ __forceinline__ bool schedule4(const int32_t* group_off, int capacity, int E, int64_t n_rows, int ntn, MTile& t)
{
    if (E <= 128) return schedule_per<2, BM>(group_off, capacity, E, n_rows, ntn, t);
    return schedule_per<16, BM>(group_off, capacity, E, n_rows, ntn, t);
}

struct Mx4Params {
    MParams p;             // shapes, schedule and outputs (p.A / p.B unused; p.C, p.H may be null)
    const uint8_t* Aq;     // [n_rows, K/2] codes
    const uint8_t* As;     // [n_rows, K/32] scales
    const uint8_t* Bq;     // per expert [N_total, K/2] codes at Bq + e * sBq
    const uint8_t* Bs;     // per expert [N_total, K/32] scales at Bs + e * sBq / 16
    int64_t sBq;
};

// SwiGLU forward epilogue: [g | u] (when p.C is given), h in bf16 (when p.H
// is), and always the MXFP4 copy of the bf16 h, which the down GEMM reads.
// A wave's 32 x 32 sub-tile has a row in the lanes l and l + 32, four columns
// in turn: columns 8 q + 4 (lane >> 5) .. + 3 in registers 4 q .. 4 q + 3.  Rounded
// to bf16 and with its middle quarters exchanged between the lanes' halves,
// lane l holds columns 0 .. 15 and lane l + 32 columns 16 .. 31: MXFP4 blocks
// are made there, and only bf16 rows go through the LDS, for stores of whole
// lines (stored from the registers, 64 bytes of a row by two lanes, the outputs
// of 65536 rows cost more: gate/up with gu and h 649 -> 665 us, down 406 -> 443).
template <int BM>
__device__ __forceinline__ void epilogue_swiglu4(const f32x16 (&acc)[BM / 64][2], const MParams& p, int64_t row0,
                                                 int rows_valid, int nt, uint8_t* lds)
{
    constexpr int NT = WL<NW4>::NT;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    const int wm = WL<NW4>::wm(wave), wn = WL<NW4>::wn(wave);
    const int n0 = nt * 128;   // (f is a multiple of 128: a tile's columns all exist)
    if (p.C) {
        stage_acc<BM, NW4>(acc, lds);
        stage_flush<BM, 32, NT>(lds, [&](int r, int c, uint4 v) {
            const int n = n0 + 8 * (c & 15);
            if (r < rows_valid) *reinterpret_cast<uint4*>(p.C + (row0 + r) * p.ldc + (c < 16 ? n : p.f + n)) = v;
        });
    }
#pragma unroll
    for (int i = 0; i < BM / 64; ++i) {
        uint2 w[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float hv[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) hv[e] = silu_f(acc[i][0][4 * q + e]) * acc[i][1][4 * q + e];
            w[q] = pack4_bf16(hv[0], hv[1], hv[2], hv[3]);
        }
        uint4 v[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const auto x = __builtin_amdgcn_permlane32_swap(w[q].x, w[q + 2].x, false, false);
            const auto y = __builtin_amdgcn_permlane32_swap(w[q].y, w[q + 2].y, false, false);
            v[q] = make_uint4(x[0], y[0], x[1], y[1]);
        }
        const uint32_t m = max(mx4::amax8(v[0]), mx4::amax8(v[1]));
        const auto o = __builtin_amdgcn_permlane32_swap(m, m, false, false);
        const uint32_t s = mx4::scale_byte(max(o[0], o[1]));
        const int r = wm * (BM / 2) + i * 32 + (lane & 31);
        const int col = wn * 32 + 16 * (lane >> 5);
        if (r < rows_valid) {
            const int64_t at = (row0 + r) * p.ldq + n0 + col;
            *reinterpret_cast<uint2*>(p.Mq + at / 2) = make_uint2(mx4::encode8(v[0], s), mx4::encode8(v[1], s));
            if (lane < 32) p.Ms[at / 32] = (uint8_t)s;
        }
        if (p.H) {
            *reinterpret_cast<uint4*>(lds + stage_off<16>(r, col)) = v[0];
            *reinterpret_cast<uint4*>(lds + stage_off<16>(r, col + 8)) = v[1];
        }
    }
    if (p.H)
        stage_flush<BM, 16, NT>(lds, [&](int r, int c, uint4 v) {
            if (r < rows_valid) *reinterpret_cast<uint4*>(p.H + (row0 + r) * p.ldh + n0 + 8 * c) = v;
        });
}

template <int EPI, int BM>   // M-tiles of BM rows
__global__ MOE_GEMM_KERNEL_ATTRS_NW(NW4) void mx4_grouped_m_kernel(Mx4Params mp)
{
    // all of the LDS: the 128-row ring with its scales
    __shared__ __align__(16) uint8_t smem[3 * (128 + BN) * 128 + 2 * SSTAGE];
    static_assert(sizeof(smem) >= 2 * (BM + BN) * 128 + 2 * SSTAGE && sizeof(smem) <= 160 * 1024, "LDS");
    const MParams& p = mp.p;
    MTile tile;
    if (!schedule4<BM>(p.group_off, p.capacity, p.E, p.n_rows, p.ntn, tile)) return;
    const int nt = tile.nt;
    const int64_t cb = p.K / 2, sbk = p.K / 32;   // bytes per row: codes, scales

    Src4 sa;
    sa.c0 = mp.Aq + tile.row0 * cb;
    sa.s0 = mp.As + tile.row0 * sbk;
    sa.K = p.K;
    Src4 sb;
    int r_lo, r_hi;
    if constexpr (EPI == EPI_SWIGLU_FWD) {
        r_lo = nt * 128;
        r_hi = p.f + r_lo;
        sb.rows0 = sb.rows1 = min(128, p.f - r_lo);
    } else {
        r_lo = nt * BN;
        r_hi = r_lo + 128;
        sb.rows0 = max(min(128, p.N - r_lo), 0);
        sb.rows1 = max(min(128, p.N - r_hi), 0);
    }
    const uint8_t* Bq = mp.Bq + (int64_t)tile.e * mp.sBq;
    const uint8_t* Bs = mp.Bs + (int64_t)tile.e * (mp.sBq / 16);
    sb.c0 = Bq + r_lo * cb;
    sb.c1 = Bq + r_hi * cb;
    sb.s0 = Bs + r_lo * sbk;
    sb.s1 = Bs + r_hi * sbk;
    sb.K = p.K;

    // the last M-tile of an expert with at most 64 (128) rows: a smaller tile
    auto run = [&](auto BMS_) __attribute__((always_inline)) {
        constexpr int BMS = decltype(BMS_)::value;
        sa.c1 = sa.c0 + (BMS / 2) * cb;
        sa.s1 = sa.s0 + (BMS / 2) * sbk;
        sa.rows0 = min(tile.rows_valid, BMS / 2);
        sa.rows1 = max(tile.rows_valid - BMS / 2, 0);
        f32x16 acc[BMS / 64][2];
        if constexpr (BMS == 256) mainloop4_pp(sa, sb, acc, smem);
        else mainloop4<BMS>(sa, sb, acc, smem);
        if constexpr (EPI == EPI_SWIGLU_FWD)
            epilogue_swiglu4<BMS>(acc, p, tile.row0, tile.rows_valid, nt, smem);
        else
            epilogue_m<BMS, EPI_STORE, NW4>(acc, p, tile.row0, tile.rows_valid, nt, smem);
    };
    if constexpr (BM == 64) {
        run(std::integral_constant<int, 64>{});
    } else {
        if (tile.rows_valid <= 64) run(std::integral_constant<int, 64>{});
        else if (BM == 128 || tile.rows_valid <= 128) run(std::integral_constant<int, 128>{});
        else if constexpr (BM == 256) run(std::integral_constant<int, 256>{});
    }
}

// ---------------------------------------------------------------- few rows
// The form for few rows per expert (single tokens, small batches): the
// weights are read once and that bounds it, so a workgroup takes 32 output
// columns (32 gate and 32 up rows of W13) of one expert against up to 64 of
// its rows, and its 8 waves split K in units of 256 k, 128 bytes of a row: a
// panel is U units of every wave.  A wave's weights of a panel come into its
// own part of the LDS by direct loads, all in flight together and whole
// 128-byte lines at a time (read straight into the registers of a fragment, 64
// bytes of each of 16 rows, the same bytes took 1.25 times as long from HBM,
// twice as long from the L2); the panel's scales, which are consecutive in
// every row, are loaded once for all waves (each wave fetching its own 16
// bytes of 64 rows made the kernel half as fast).  They are multiplied with 16
// rows at a time (v_mfma_scale_f32_16x16x128: lane i holds weight row, or
// token, i & 15 and k-block i >> 4 of 128 k).  The waves' sums meet in LDS, in
// wave order.
constexpr int FROWS = 64, FCOLS = 32;

struct Few4Params {
    const uint8_t *Aq, *As;    // rows: codes, scales
    const uint8_t *Bq, *Bs;    // weights of expert 0; sBq bytes between experts' codes
    int64_t sBq;
    int K;
    int f;                     // gate/up: W13's up rows start here
    int ntn;                   // column tiles: f / 32 or d / 32
    const int32_t* group_off;
    int capacity, E;
    int64_t n_rows;
    uint16_t* C;               // gate/up: gu [n_rows, 2f] or null; down: y [n_rows, ldc]
    int64_t ldc;
    uint16_t* H;               // gate/up: h [n_rows, f] or null
    uint8_t *Mq, *Ms;          // gate/up: MXFP4 h
};

template <int EPI, int U>   // U: units a wave has in flight
__global__ __launch_bounds__(64 * NW4) void mx4_few_rows_kernel(Few4Params p)
{
    constexpr int NTILE = EPI == EPI_SWIGLU_FWD ? 4 : 2;   // 16-row weight tiles: gate, gate, up, up
    constexpr int NCH = FROWS / 16;                        // 16-row chunks of the rows
    constexpr int WROWS = 16 * NTILE;                      // weight rows of the workgroup
    constexpr int WBYTES = U * WROWS * 128;                // a wave's weights
    constexpr int RBYTES = NTILE * 64 * 16;                // a wave's sums, in the same place afterwards
    constexpr int SB = 64 * U;                             // scale bytes of a row and panel
    constexpr int SPIECE = SB / 16;                        // ... in 16-byte pieces
    constexpr int NOUT = EPI == EPI_SWIGLU_FWD ? 3 : 1;
    __shared__ __align__(16) uint8_t lds[NW4 * (WBYTES > RBYTES ? WBYTES : RBYTES)];
    __shared__ __align__(16) uint8_t lsc[WROWS * SB];
    __shared__ __align__(16) uint16_t out[NOUT][16 * FCOLS];
    auto red = reinterpret_cast<f32x4_t(*)[NTILE][64]>(lds);
    MTile t;
    if (!schedule4<FROWS>(p.group_off, p.capacity, p.E, p.n_rows, p.ntn, t)) return;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r16 = lane & 15, kb = lane >> 4;
    const int64_t cb = p.K / 2, sbk = p.K / 32;
    const int n0 = t.nt * FCOLS;
    const int nch = (t.rows_valid + 15) / 16;

    // this wave's units; steps of 128 k
    const int n128 = p.K / 128, n256 = (n128 + 1) / 2;
    // 32 consecutive rows of W13's gate half and of its up half (of W2)
    const uint8_t* Bq = p.Bq + (int64_t)t.e * p.sBq + n0 * cb;
    const uint8_t* Bs = p.Bs + (int64_t)t.e * (p.sBq / 16) + n0 * sbk;
    desc_t d[NTILE / 2];
#pragma unroll
    for (int h = 0; h < NTILE / 2; ++h) d[h] = wave_uniform(make_desc(Bq + h * (p.f * cb), FCOLS * cb));
    // direct loads of scales: 64 / SPIECE rows each, this wave's is number `wave`;
    // piece c of row r at piece c ^ (r & (SPIECE - 1))
    constexpr int SINSTR = WROWS * SPIECE / 64;
    const int srow = wave * (64 / SPIECE) + lane / SPIECE;   // of WROWS
    const int shalf = __builtin_amdgcn_readfirstlane(srow) / FCOLS;
    const desc_t ds = wave_uniform(make_desc(Bs + shalf * (p.f * sbk), wave < SINSTR ? FCOLS * sbk : 0));
    const uint32_t soff = (uint32_t)((srow % FCOLS) * sbk) + (((uint32_t)lane % SPIECE) ^ ((uint32_t)srow & (SPIECE - 1))) * 16u;
    const uint32_t sm0 = lds_addr(lsc) + (uint32_t)wave * 1024u;
    // direct load q of a unit: rows 8q .. 8q+7 of WROWS, 16-byte chunk c of row
    // r at chunk c ^ ((r >> 1) & 7), so that a fragment's 16 rows of one chunk
    // lie in 16 different bank groups
    uint32_t voff[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int row = 8 * q + (lane >> 3);               // of a half's 32
        voff[q] = (uint32_t)(row * cb) + (((uint32_t)lane & 7u) ^ ((row >> 1) & 7u)) * 16u;
    }
    uint8_t* mine = lds + wave * WBYTES;
    const uint32_t m0 = lds_addr(mine);
    // the scale words of a unit's two steps of 128 k
    struct __attribute__((packed, aligned(4))) Words2 { uint32_t v[2]; };
    auto scales = [&](const uint8_t* row, int u) __attribute__((always_inline)) {
        Words2 x;
        if (2 * u + 1 < n128) {
            x = *reinterpret_cast<const Words2*>(row + u * 8);
        } else {
            x.v[0] = *reinterpret_cast<const uint32_t*>(row + u * 8);
            x.v[1] = 0;
        }
        return x;
    };
    f32x4_t acc[NCH][NTILE];
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
        for (int i = 0; i < NTILE; ++i) acc[c][i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    for (int p0 = 0; p0 < n256; p0 += NW4 * U) {
        const int u0 = p0 + wave * U, u_end = n256;        // this wave's units of the panel
        if (wave < SINSTR) dma16_to_lds_at(ds, sm0, soff, (uint32_t)p0 * 8u);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (u0 + u >= u_end) break;
#pragma unroll
            for (int q = 0; q < 2 * NTILE; ++q)
                dma16_to_lds_at(d[q >> 2], m0 + (uint32_t)(u * WROWS * 128 + q * 1024), voff[q & 3], (uint32_t)(u0 + u) * 128u);
        }
        Words2 sw[U][NTILE];
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            if (c >= nch) break;
            // rows past the last valid one repeat it (their sums are not stored)
            const int64_t row = t.row0 + min(c * 16 + r16, t.rows_valid - 1);
            const uint8_t* xr = p.Aq + row * cb + kb * 16;
            uint4 x[U][2];
            Words2 sx[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (u0 + u >= u_end) break;
                sx[u] = scales(p.As + row * sbk, u0 + u);
                x[u][0] = *reinterpret_cast<const uint4*>(xr + (int64_t)(u0 + u) * 128);
                x[u][1] = 2 * (u0 + u) + 1 < n128 ? *reinterpret_cast<const uint4*>(xr + (int64_t)(u0 + u) * 128 + 64)
                                                  : make_uint4(0, 0, 0, 0);
            }
            if (c == 0) {
                // all waves' direct loads have landed
                asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
                __syncthreads();
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int i = 0; i < NTILE; ++i) {
                        const int row = i * 16 + r16, at = (wave * U + u) * 8;
                        const uint2 x2 = *reinterpret_cast<const uint2*>(
                            lsc + row * SB + (((at >> 4) ^ (row & (SPIECE - 1))) << 4) + (at & 8));
                        sw[u][i].v[0] = x2.x;
                        sw[u][i].v[1] = x2.y;
                    }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (u0 + u >= u_end) break;
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    if (2 * (u0 + u) + s >= n128) break;
                    const i32x8 b = {(int)x[u][s].x, (int)x[u][s].y, (int)x[u][s].z, (int)x[u][s].w, 0, 0, 0, 0};
                    const int sb = (int)(sx[u].v[s] >> (8 * kb));
#pragma unroll
                    for (int i = 0; i < NTILE; ++i) {
                        const uint4 w = *reinterpret_cast<const uint4*>(
                            mine + (u * WROWS + i * 16 + r16) * 128 + ((s * 4 + kb) ^ ((r16 >> 1) & 7)) * 16);
                        const i32x8 a = {(int)w.x, (int)w.y, (int)w.z, (int)w.w, 0, 0, 0, 0};
                        acc[c][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc[c][i], 4, 4, 0,
                                                                                     (int)(sw[u][i].v[s] >> (8 * kb)), 0, sb);
                    }
                }
            }
        }
        // the next panel, or the sums, take the weights' and scales' place
        __syncthreads();
    }
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
        if (c >= nch) break;
#pragma unroll
        for (int i = 0; i < NTILE; ++i) red[wave][i][lane] = acc[c][i];
        __syncthreads();
        // 16 rows x 32 columns; lane (col / 4 % 4) * 16 + row holds columns 4g .. 4g+3 of a tile
        for (int o = tid; o < 16 * FCOLS; o += 64 * NW4) {
            const int r = o & 15, col = o >> 4;
            const int l = ((col & 15) >> 2) * 16 + r, q = col & 3, tl = col >> 4;
            float v = red[0][tl][l][q], u = 0.0f;
#pragma unroll
            for (int w = 1; w < NW4; ++w) v += red[w][tl][l][q];
            if constexpr (EPI == EPI_SWIGLU_FWD) {
                u = red[0][2 + tl][l][q];
#pragma unroll
                for (int w = 1; w < NW4; ++w) u += red[w][2 + tl][l][q];
                out[1][r * FCOLS + col] = (uint16_t)f32_to_bf16_bits(v);
                out[2][r * FCOLS + col] = (uint16_t)f32_to_bf16_bits(u);
                v = silu_f(v) * u;
            }
            out[0][r * FCOLS + col] = (uint16_t)f32_to_bf16_bits(v);
        }
        __syncthreads();
        // a wave stores one 16 x 32 tile, 16 bytes per lane: h (or y), g, u
        const int r = lane >> 2, col = 8 * (lane & 3);
        const int64_t row = t.row0 + c * 16 + r;
        const bool valid = c * 16 + r < t.rows_valid;
        if (wave < NOUT) {
            const uint4 v = *reinterpret_cast<const uint4*>(&out[wave][r * FCOLS + col]);
            if constexpr (EPI == EPI_SWIGLU_FWD) {
                if (wave == 0) {
                    uint32_t q;
                    const uint32_t s = mx4::quant8_quad(v, q);
                    if (valid) {
                        if (p.H) *reinterpret_cast<uint4*>(p.H + row * p.f + n0 + col) = v;
                        *reinterpret_cast<uint32_t*>(p.Mq + row * (p.f / 2) + (n0 + col) / 2) = q;
                        if ((lane & 3) == 0) p.Ms[row * (p.f / 32) + n0 / 32] = (uint8_t)s;
                    }
                } else if (valid && p.C) {
                    *reinterpret_cast<uint4*>(p.C + row * p.ldc + (wave == 2 ? p.f : 0) + n0 + col) = v;
                }
            } else {
                if (valid) *reinterpret_cast<uint4*>(p.C + row * p.ldc + n0 + col) = v;
            }
        }
        // (the next chunk's sums go to red, which nobody reads any more; out is
        // written again after the barrier that follows them)
    }
}

// The tiles of bm rows that the groups can have: sum ceil(m_e / bm) over the
// groups with rows, at most e of them, is sum 1 + floor((m_e - 1) / bm).
inline int64_t row_tiles(int64_t n_rows, int E, int bm)
{
    const int64_t e = std::min<int64_t>(E, n_rows);
    return e + (n_rows - e) / bm;
}

// Whether the few-row form runs: with more than 32 rows per expert on average
// when its workgroups (at most) are one per CU, else when they run in one round
// (one per CU with two units a wave, 139 KB of LDS, two with one), with at most
// 16 rows in one and a half.  Measured, this form and the tile form (us):
//   one per CU: 1 row of 1 expert, d = 4096, f = 1536, gate/up 5.5 16.1 and down
//     3.9 8.3; 256 rows of 1 expert, gate/up 15.0 16.6 (down, two per CU, 9.2 8.7)
//   one round: 256 rows of 8, d = 2048, f = 1152, 9.7 9.9 (384 rows 12.3 10.2)
//   1.5 rounds: 64 rows of 8, d = 4096, 15.8 16.6; 256 rows of 32, d = 1024, 5.8
//     6.9 (but 1024 rows 8.2 7.0)
//   more: 64 rows of 8, down (2 rounds) 8.2 8.4; 256 of 32, d = 1024, f = 512,
//     7.5 5.4; 16 rows of 16 25.0 18.5; 256 rows of 128 198 147 and 131 89: there
//     the tile form streams the weights faster.
inline bool few_rows(const GroupSpec& g, int K, int ntn)
{
    const int64_t n = g.n_rows, e = std::min<int64_t>(g.E, n);
    const int64_t wgs = row_tiles(n, g.E, FROWS) * ntn, round = 256 * (K <= NW4 * 256 ? 2 : 1);
    if (n > 32 * e) return wgs <= 256;
    return n > 16 * e ? wgs <= round : 2 * wgs <= 3 * round;
}

template <int EPI>
hipError_t launch_few4(const Few4Params& p, hipStream_t s)
{
    const int64_t grid = (row_tiles(p.n_rows, p.E, FROWS) * p.ntn + 7) / 8 * 8;
    if (p.K <= NW4 * 256)   // one unit per wave
        hipLaunchKernelGGL((mx4_few_rows_kernel<EPI, 1>), dim3((unsigned)grid), dim3(64 * NW4), 0, s, p);
    else
        hipLaunchKernelGGL((mx4_few_rows_kernel<EPI, 2>), dim3((unsigned)grid), dim3(64 * NW4), 0, s, p);
    return hipGetLastError();
}

// Tiles of 64 or 128 rows, the smallest whose number (its host-known bound)
// runs in one round on the 256 CUs, else of 256 rows, whose loop does the most
// per byte read.  Measured (64, 128, 256 rows a tile, us): 838 rows of 3
// experts, d = 2048, f = 1280, gate/up 12.5 14.6 17.4 and down 9.3 10.0 13.8;
// 2000 rows of 8, f = 1152, 21.9 15.4 18.4 and 16.2 11.6 15.5 (342 and 304
// tiles of 64 rows); 16576 rows of 43, d = f = 1024, 62.4 46.1 42.4 and 34.6
// 28.6 27.0.
template <int EPI>
hipError_t launch_mx4_m(const Mx4Params& mp, hipStream_t s)
{
    auto tiles = [&](int bm) { return row_tiles(mp.p.n_rows, mp.p.E, bm) * mp.p.ntn; };
    auto go = [&](auto BM) {
        const int64_t grid = (tiles(decltype(BM)::value) + 7) / 8 * 8;
        if (grid > 0)
            hipLaunchKernelGGL((mx4_grouped_m_kernel<EPI, decltype(BM)::value>), dim3((unsigned)grid), dim3(64 * NW4), 0,
                               s, mp);
    };
    if (tiles(64) <= 256) go(std::integral_constant<int, 64>{});
    else if (tiles(128) <= 256) go(std::integral_constant<int, 128>{});
    else go(std::integral_constant<int, 256>{});
    return hipGetLastError();
}

inline size_t al(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace

// the row-wise MXFP4 h that the gate/up stage leaves for the down stage
size_t gemm_ws_mxfp4(int64_t n_rows, int f)
{
    return al((size_t)n_rows * f / 2) + al((size_t)n_rows * f / 32) + 256;   // never empty
}

hipError_t gemm_op_mxfp4(int op, const moe_gemm_tensors& t, GroupSpec g, int d, int f, hipStream_t s)
{
    uint8_t* hq = static_cast<uint8_t*>(t.ws);
    uint8_t* hs = hq + al((size_t)g.n_rows * f / 2);
    Mx4Params a{};
    a.p.group_off = g.group_off;
    a.p.capacity = g.capacity;
    a.p.E = g.E;
    a.p.n_rows = g.n_rows;
    a.p.f = f;
    if (op != MOE_GEMM_GATE_UP && op != MOE_GEMM_DOWN) return hipErrorInvalidValue;
    if (g.n_rows == 0) return hipSuccess;
    const bool up = op == MOE_GEMM_GATE_UP;
    if (few_rows(g, up ? d : f, (up ? f : d) / FCOLS)) {
        Few4Params p{};
        p.group_off = g.group_off;
        p.capacity = g.capacity;
        p.E = g.E;
        p.n_rows = g.n_rows;
        p.f = f;
        p.K = up ? d : f;
        p.ntn = (up ? f : d) / FCOLS;
        p.Aq = up ? static_cast<const uint8_t*>(t.x_perm) : hq;
        p.As = up ? t.x_perm_scales : hs;
        p.Bq = static_cast<const uint8_t*>(up ? t.w13 : t.w2);
        p.Bs = up ? t.w13_scales : t.w2_scales;
        p.sBq = (int64_t)d * f * (up ? 2 : 1) / 2;
        p.C = static_cast<uint16_t*>(up ? t.gu : t.y_perm);
        p.ldc = up ? 2 * f : d;
        p.H = static_cast<uint16_t*>(t.h);
        p.Mq = hq;
        p.Ms = hs;
        return up ? launch_few4<EPI_SWIGLU_FWD>(p, s) : launch_few4<EPI_STORE>(p, s);
    }
    if (up) {
        a.p.N = f;
        a.p.K = d;
        a.p.ntn = (f + 127) / 128;
        a.p.C = static_cast<uint16_t*>(t.gu);
        a.p.ldc = 2 * f;
        a.p.H = static_cast<uint16_t*>(t.h);
        a.p.ldh = f;
        a.p.Mq = hq;
        a.p.Ms = hs;
        a.p.ldq = f;
        a.Aq = static_cast<const uint8_t*>(t.x_perm);
        a.As = t.x_perm_scales;
        a.Bq = static_cast<const uint8_t*>(t.w13);
        a.Bs = t.w13_scales;
        a.sBq = (int64_t)2 * f * (d / 2);
        return launch_mx4_m<EPI_SWIGLU_FWD>(a, s);
    }
    a.p.N = d;
    a.p.K = f;
    a.p.ntn = (d + BN - 1) / BN;
    a.p.C = static_cast<uint16_t*>(t.y_perm);
    a.p.ldc = d;
    a.Aq = hq;
    a.As = hs;
    a.Bq = static_cast<const uint8_t*>(t.w2);
    a.Bs = t.w2_scales;
    a.sBq = (int64_t)d * (f / 2);
    return launch_mx4_m<EPI_STORE>(a, s);
}

}  // namespace moe
