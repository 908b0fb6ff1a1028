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
#include "gemm_common.h"
#include "mx4.h"

namespace moe {
namespace {

using namespace gemm;

typedef __attribute__((ext_vector_type(8))) int i32x8;

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

// BM x 256 tile, two LDS stages of codes, scales read from memory
template <int BM>
__device__ __forceinline__ void mainloop4(const Src4& sa, const Src4& sb, f32x16 (&acc)[BM / 64][2], uint8_t* smem)
{
    constexpr int MI = BM / 64, NJ = 2;
    constexpr int STAGE = (BM + BN) * 128;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int wm = WL<NW4>::wm(wave), wn = WL<NW4>::wn(wave);
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
    const int nk = (sa.K + KB - 1) / KB;
    if (nk == 0) return;
    DirectLoader<BM, 64, false, NW4> la;
    DirectLoader<BN, 64, false, NW4> lb;
    la.init(codes_as_tile(sa));
    lb.init(codes_as_tile(sb));
    auto issue = [&](int kt, int stage) {
        la.issue(reinterpret_cast<uint16_t*>(smem + stage * STAGE), kt);
        lb.issue(reinterpret_cast<uint16_t*>(smem + stage * STAGE + BM * 128), kt);
    };
    // a row's scale word (128 k), 0 outside the operand
    auto scale_word = [&](const Src4& s, int row, int half, int w) {
        const bool hi = row >= half;
        const int r = hi ? row - half : row;
        return r < (hi ? s.rows1 : s.rows0) && w * 128 < s.K
                   ? *reinterpret_cast<const uint32_t*>((hi ? s.s1 : s.s0) + (int64_t)r * (s.K / 32) + w * 4) : 0u;
    };
    issue(0, 0);
    for (int kt = 0; kt < nk; ++kt) {
        wait_vmcnt<0>();
        __syncthreads();
        if (kt + 1 < nk) issue(kt + 1, (kt + 1) & 1);
        const uint8_t* a_s = smem + (kt & 1) * STAGE;
        const uint8_t* b_s = a_s + BM * 128;
        for (int hs = 0; hs < 2 && kt * KB + hs * 128 < sa.K; ++hs) {
            uint32_t wa[MI], wb[NJ];
#pragma unroll
            for (int i = 0; i < MI; ++i)
                wa[i] = scale_word(sa, wm * (BM / 2) + i * 32 + (lane & 31), BM / 2, kt * 2 + hs) >> (8 * (lane >> 5));
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                wb[j] = scale_word(sb, WL<NW4>::sub_col(wn, j) + (lane & 31), 128, kt * 2 + hs) >> (8 * (lane >> 5));
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                i32x8 af[MI], bf[NJ];
#pragma unroll
                for (int i = 0; i < MI; ++i) af[i] = read_frag4(a_s, wm * (BM / 2) + i * 32, hs * 2 + q, lane);
#pragma unroll
                for (int j = 0; j < NJ; ++j) bf[j] = read_frag4(b_s, WL<NW4>::sub_col(wn, j), hs * 2 + q, lane);
#pragma unroll
                for (int i = 0; i < MI; ++i)
#pragma unroll
                    for (int j = 0; j < NJ; ++j)
                        acc[i][j] = q ? mfma4<2>(bf[j], af[i], acc[i][j], wb[j], wa[i])
                                      : mfma4<0>(bf[j], af[i], acc[i][j], wb[j], wa[i]);
            }
        }
    }
    __syncthreads();
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
// is), and always the MXFP4 copy of the bf16 h, which the down GEMM reads
template <int BM>
__device__ __forceinline__ void epilogue_swiglu4(const f32x16 (&acc)[BM / 64][2], const MParams& p, int64_t row0,
                                                 int rows_valid, int nt, uint8_t* lds)
{
    constexpr int NT = WL<NW4>::NT;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    const int wm = WL<NW4>::wm(wave), wn = WL<NW4>::wn(wave);
    const int n0 = nt * 128;
    if (p.C) {
        stage_acc<BM, NW4>(acc, lds);
        stage_flush<BM, 32, NT>(lds, [&](int r, int c, uint4 v) {
            const int n = n0 + 8 * (c & 15);
            if (r < rows_valid && n < p.f)
                *reinterpret_cast<uint4*>(p.C + (row0 + r) * p.ldc + (c < 16 ? n : p.f + n)) = v;
        });
    }
#pragma unroll
    for (int i = 0; i < BM / 64; ++i)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            float hv[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) hv[q] = silu_f(acc[i][0][4 * g + q]) * acc[i][1][4 * g + q];
            stage_put(lds, stage_off<16>(wm * (BM / 2) + i * 32 + (lane & 31), acc_col<NW4>(wn, 0, g, lane)),
                      pack4_bf16(hv[0], hv[1], hv[2], hv[3]));
        }
    stage_flush<BM, 16, NT>(lds, [&](int r, int c, uint4 v) {
        const int n = n0 + 8 * c;
        uint32_t q;
        const uint32_t s = mx4::quant8_quad(v, q);
        if (r < rows_valid && n < p.f) {
            if (p.H) *reinterpret_cast<uint4*>(p.H + (row0 + r) * p.ldh + n) = v;
            *reinterpret_cast<uint32_t*>(p.Mq + (row0 + r) * (p.ldq / 2) + n / 2) = q;
            if ((c & 3) == 0) p.Ms[(row0 + r) * (p.ldq / 32) + n / 32] = (uint8_t)s;
        }
    });
}

template <int EPI>
__global__ MOE_GEMM_KERNEL_ATTRS_NW(NW4) void mx4_grouped_m_kernel(Mx4Params mp)
{
    constexpr int BM = 256;
    __shared__ __align__(16) uint8_t smem[2 * (BM + BN) * 128];
    const MParams& p = mp.p;
    MTile tile;
    if (!schedule_m<BM>(p.group_off, p.capacity, p.E, p.n_rows, p.ntn, tile)) return;
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
        mainloop4<BMS>(sa, sb, acc, smem);
        if constexpr (EPI == EPI_SWIGLU_FWD)
            epilogue_swiglu4<BMS>(acc, p, tile.row0, tile.rows_valid, nt, smem);
        else
            epilogue_m<BMS, EPI_STORE, NW4>(acc, p, tile.row0, tile.rows_valid, nt, smem);
    };
    if (tile.rows_valid <= 64) run(std::integral_constant<int, 64>{});
    else if (tile.rows_valid <= 128) run(std::integral_constant<int, 128>{});
    else run(std::integral_constant<int, 256>{});
}

template <int EPI>
hipError_t launch_mx4_m(const Mx4Params& mp, hipStream_t s)
{
    const int64_t bound = (mp.p.n_rows / 256 + mp.p.E) * (int64_t)mp.p.ntn;
    const int64_t grid = (bound + 7) / 8 * 8;
    if (grid == 0 || mp.p.n_rows == 0) return hipSuccess;
    hipLaunchKernelGGL((mx4_grouped_m_kernel<EPI>), dim3((unsigned)grid), dim3(64 * NW4), 0, s, mp);
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
    if (op == MOE_GEMM_GATE_UP) {
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
    if (op == MOE_GEMM_DOWN) {
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
    return hipErrorInvalidValue;
}

}  // namespace moe
