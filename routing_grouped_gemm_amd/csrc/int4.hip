// Experts in 4-bit integers with group scales: the quantiser and its inverse,
// and the layer's feed-forward for few tokens (moe_int4_ffn).
//
// The products are bound by the weights' bytes: half a byte an element plus a
// scale (and zero point) a group, each read once.
//
// Codes become matrix operands without a conversion: bf16 has seven fraction
// bits, so a code q put at bits 3..6 of the word 0x4180 is the bf16 number
// 16 + q, and one shift and one and-or make two of them.  With X the sum of
// a row's x over a group,
//     sum x (q - z) s = s * (sum x (16 + q) - (16 + z) X),
// the products exact in fp32, the two sums held in fp32 and the scale applied to
// their difference: weights are never rounded.  X comes from one more MFMA with
// ones for weights, which serves every column of the tile.  (At bits 0..3, for
// 128 + q, the shift of the first code is free, but the difference then loses
// three more bits.)
//
// v_mfma_f32_16x16x32_bf16: rows of x are the M side (lane & 15), weight rows the
// N side (lane & 15), K in eighths (lane >> 4).  A wave reads 16 weight rows x 128
// codes, 16 bytes a lane: lane group g holds codes 32g .. 32g + 31 of the row.
// With groups of 128 the K order within the group is free, and MFMA i takes
// codes 32g + 8i .. + 7.  With smaller groups each MFMA must stay within one:
// a 4 x 4 exchange of words among the lane groups gives MFMA i the codes
// 32i + 8g .. + 7.  Within a word the pairs are (j, j + 4), and x is put in the
// same order.
#include "gemm_common.h"

namespace moe {
namespace {

using gemm::bf16x8;
typedef __attribute__((ext_vector_type(4))) float f32x4;

// ---------------------------------------------------------------- quantiser
// A lane takes 8 elements, a group's G / 8 lanes (4, 8 or 16 neighbours) find its
// extremes together.
template <int G, bool ZEROS>
__global__ __launch_bounds__(256) void quantize_int4_kernel(const uint4* __restrict__ src, int64_t n8,
                                                            uint32_t* __restrict__ codes, uint16_t* __restrict__ scales,
                                                            uint8_t* __restrict__ zeros)
{
    constexpr int LG = G / 8;
    for (int64_t base = (int64_t)blockIdx.x * 256; base < n8; base += (int64_t)gridDim.x * 256) {
        const int64_t i = base + threadIdx.x;
        const bool on = i < n8;   // whole groups are on or off
        const uint4 in = on ? src[i] : make_uint4(0, 0, 0, 0);
        const uint32_t w[4] = {in.x, in.y, in.z, in.w};
        float v[8];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            v[2 * p] = bf16_lo(w[p]);
            v[2 * p + 1] = bf16_hi(w[p]);
        }
        float hi = 0.0f, lo = 0.0f;
        bool finite = true;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            hi = fmaxf(hi, v[j]);
            lo = fminf(lo, v[j]);
            finite &= fabsf(v[j]) <= 3.402823466e38f;
        }
#pragma unroll
        for (int off = 1; off < LG; off <<= 1) {
            hi = fmaxf(hi, __shfl_xor(hi, off, 64));
            lo = fminf(lo, __shfl_xor(lo, off, 64));
            finite &= __shfl_xor((int)finite, off, 64) != 0;
        }
        const float s0 = ZEROS ? (0.5f * hi - 0.5f * lo) / 7.5f : fmaxf(hi, -lo) / 7.0f;
        uint32_t sb = f32_to_bf16_bits(s0);
        if (sb < 0x0080u) sb = 0x0080u;                 // 2^-126
        const float s = __uint_as_float(sb << 16);
        float z = 8.0f;
        if constexpr (ZEROS) z = fminf(fmaxf(rintf(-lo / s), 0.0f), 15.0f);
        uint32_t out = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float q = ZEROS ? rintf(v[j] / s) + z : fmaxf(rintf(v[j] / s), -8.0f) + 8.0f;
            out |= (uint32_t)fminf(fmaxf(q, 0.0f), 15.0f) << (4 * j);
        }
        if (!finite) {
            out = 0x88888888u;
            sb = 0x7fc0u;
            z = 8.0f;
        }
        if (!on) continue;
        codes[i] = out;
        if (threadIdx.x % LG == 0) {
            scales[i / LG] = (uint16_t)sb;
            if constexpr (ZEROS) zeros[i / LG] = (uint8_t)z;
        }
    }
}

template <int G>
__global__ __launch_bounds__(256) void dequantize_int4_kernel(const uint32_t* __restrict__ codes,
                                                              const uint16_t* __restrict__ scales,
                                                              const uint8_t* __restrict__ zeros, int64_t n8,
                                                              uint4* __restrict__ dst)
{
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n8; i += (int64_t)gridDim.x * 256) {
        const uint32_t c = codes[i];
        const float s = bf16_to_f32(scales[i / (G / 8)]);
        const float z = zeros ? (float)zeros[i / (G / 8)] : 8.0f;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = ((float)((c >> (4 * j)) & 15u) - z) * s;
        dst[i] = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                            pack_bf16x2(v[6], v[7]));
    }
}

// ---------------------------------------------------------------- products
__device__ __forceinline__ bf16x8 as_bf16x8(uint4 v) { return __builtin_bit_cast(bf16x8, v); }

// the bf16 numbers 16 + q of eight codes: pairs (0,4) (1,5) (2,6) (3,7)
__device__ __forceinline__ uint4 codes_to_bf16(uint32_t w)
{
    return make_uint4(((w << 3) & 0x00780078u) | 0x41804180u, ((w >> 1) & 0x00780078u) | 0x41804180u,
                      ((w >> 5) & 0x00780078u) | 0x41804180u, ((w >> 9) & 0x00780078u) | 0x41804180u);
}

// eight x in the same order
__device__ __forceinline__ uint4 pair_order(uint4 v)
{
    return make_uint4(__builtin_amdgcn_perm(v.z, v.x, 0x05040100u), __builtin_amdgcn_perm(v.z, v.x, 0x07060302u),
                      __builtin_amdgcn_perm(v.w, v.y, 0x05040100u), __builtin_amdgcn_perm(v.w, v.y, 0x07060302u));
}

// word i of lane group g <-> word g of lane group i
__device__ __forceinline__ uint4 exchange4(uint4 v)
{
    const auto a = __builtin_amdgcn_permlane32_swap(v.x, v.z, false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(v.y, v.w, false, false);
    const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    return make_uint4(c[0], c[1], d[0], d[1]);
}

// one weight row of a lane: codes, scales and zero points from the row's start
struct WRow {
    const uint8_t* codes;
    const uint16_t* scales;
    const uint8_t* zeros;    // or nullptr
};

__device__ __forceinline__ WRow w_row(const moe_int4& w, int64_t row, int K, int group)
{
    const int64_t n = row * (K / group);
    return {w.codes + row * (K / 2), (const uint16_t*)w.scales + n, w.zeros ? w.zeros + n : nullptr};
}

// acc[t] += (x rows) . (weight rows of column tile t) over chunk c of 128 codes.
// x: the lane's row (nullptr: a row of zeros).  Nothing past K is read.
template <int G, int NT>
__device__ __forceinline__ void chunk_product(f32x4 (&acc)[NT], const uint16_t* x, const WRow (&w)[NT], int c, int K,
                                              float factor)
{
    const int g = (threadIdx.x & 63) >> 4;
    const int kb = c * 128;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    uint4 q[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
        q[t] = kb + 32 * g < K ? *reinterpret_cast<const uint4*>(w[t].codes + kb / 2 + 16 * g) : zero;
    bf16x8 xf[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int block = G == 128 ? g : i;             // which 32 codes
        const int k = kb + 32 * block + 8 * (G == 128 ? i : g);
        const uint4 v = x && kb + 32 * block < K ? *reinterpret_cast<const uint4*>(x + k) : zero;
        xf[i] = as_bf16x8(pair_order(v));
    }
    if constexpr (G != 128) {
#pragma unroll
        for (int t = 0; t < NT; ++t) q[t] = exchange4(q[t]);
    }
    constexpr int PER = G / 32;                          // MFMAs of a group
#pragma unroll
    for (int b = 0; b < 4 / PER; ++b) {
        if (kb + b * G >= K) break;
        const bf16x8 ones = as_bf16x8(make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u));
        f32x4 X = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < PER; ++i) X = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[b * PER + i], ones, X, 0, 0, 0);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const uint32_t qw[4] = {q[t].x, q[t].y, q[t].z, q[t].w};
            f32x4 p = {0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < PER; ++i)
                p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[b * PER + i], as_bf16x8(codes_to_bf16(qw[b * PER + i])), p,
                                                            0, 0, 0);
            const int gi = (kb + b * G) / G;
            const float s = bf16_to_f32(w[t].scales[gi]) * factor;
            const float z = 16.0f + (w[t].zeros ? (float)w[t].zeros[gi] : 8.0f);
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[t][r] = fmaf(s, fmaf(-z, X[r], p[r]), acc[t][r]);
        }
    }
}

constexpr int kW = 4;   // waves of a workgroup: they split K and add up in LDS

// sum over the waves of element idx (row idx / 16, column idx % 16) of column tile t
template <int NT>
__device__ __forceinline__ float wave_sum(const float (&red)[kW][NT][256], int t, int idx)
{
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kW; ++w) v += red[w][t][idx];
    return v;
}

template <int NT>
__device__ __forceinline__ void put_acc(float (&red)[kW][NT][256], const f32x4 (&acc)[NT])
{
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) red[wave][t][((lane >> 4) * 4 + r) * 16 + (lane & 15)] = acc[t][r];
    __syncthreads();
}

struct Rows {
    int e;             // expert
    int64_t row0;      // first row of h (and y)
    int valid;         // rows of the tile
    int nt;            // column tile
};

// PAIR: one row a workgroup, that of slot blockIdx.y, whose expert topk_idx names
// (row = slot).  Otherwise up to 16 rows of an expert's group.
template <bool PAIR>
__device__ __forceinline__ bool find_rows(const Int4Ffn& a, int ntn, Rows& o)
{
    if constexpr (PAIR) {
        const int p = blockIdx.y;
        o.e = a.topk_idx[p];
        const int32_t dst = a.dst_row[p];
        const bool bad = o.e < 0 || o.e >= a.E || dst >= a.T * a.k;
        if (bad && a.dev_err && threadIdx.x == 0) atomicOr(a.dev_err, (int)MOE_ERR_ROW_RANGE);
        o.row0 = p;
        o.valid = 1;
        o.nt = blockIdx.x;
        return !bad && dst >= 0;
    } else {
        gemm::MTile m;
        if (!gemm::schedule_m<16>(a.group_off, 0, a.E, (int64_t)a.T * a.k, ntn, m)) return false;
        o = Rows{m.e, m.row0, m.rows_valid, m.nt};
        return true;
    }
}

// h = a(g') u' of 16 columns
template <int G, bool PAIR>
__global__ __launch_bounds__(64 * kW) void int4_gate_up_kernel(Int4Ffn a, uint16_t* __restrict__ h)
{
    __shared__ float red[kW][2][256];
    Rows o;
    if (!find_rows<PAIR>(a, a.f / 16, o)) return;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int m = lane & 15;
    const uint16_t* x = nullptr;
    if (m < o.valid) {
        const int64_t slot = PAIR ? o.row0 : a.src_slot[o.row0 + m];
        if (slot >= 0 && slot < (int64_t)a.T * a.k) x = a.x + slot / a.k * a.d;
        else if (slot >= 0 && a.dev_err) atomicOr(a.dev_err, (int)MOE_ERR_ROW_RANGE);
    }
    const int64_t n = (int64_t)o.e * 2 * a.f + o.nt * 16 + m;
    const WRow w[2] = {w_row(a.w13, n, a.d, G), w_row(a.w13, n + a.f, a.d, G)};
    f32x4 acc[2] = {};
    const int chunks = (a.d + 127) / 128;
    for (int c = wave; c < chunks; c += kW) chunk_product<G, 2>(acc, x, w, c, a.d, 1.0f);
    put_acc(red, acc);
    const int idx = threadIdx.x, r = idx >> 4;
    if (r >= o.valid) return;
    const float L = a.glu.limit;
    const float g = limit_g(wave_sum(red, 0, idx), L), u = limit_u(wave_sum(red, 1, idx), L);
    float v = 0.0f;
    with_act(a.glu.act, [&](auto A) { v = act_of<decltype(A)::value, true>(g) * u; });
    h[(o.row0 + r) * a.f + o.nt * 16 + (idx & 15)] = (uint16_t)f32_to_bf16_bits(v);
}

// y = h W2^T of 32 columns
template <int G>
__global__ __launch_bounds__(64 * kW) void int4_down_kernel(Int4Ffn a, const uint16_t* __restrict__ h,
                                                            uint16_t* __restrict__ y)
{
    __shared__ float red[kW][2][256];
    Rows o;
    if (!find_rows<false>(a, a.d / 32, o)) return;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int m = lane & 15;
    const uint16_t* x = m < o.valid ? h + (o.row0 + m) * a.f : nullptr;
    const int64_t n = (int64_t)o.e * a.d + o.nt * 32 + m;
    const WRow w[2] = {w_row(a.w2, n, a.f, G), w_row(a.w2, n + 16, a.f, G)};
    f32x4 acc[2] = {};
    const int chunks = (a.f + 127) / 128;
    for (int c = wave; c < chunks; c += kW) chunk_product<G, 2>(acc, x, w, c, a.f, 1.0f);
    put_acc(red, acc);
    const int idx = threadIdx.x, r = idx >> 4;
    if (r >= o.valid) return;
#pragma unroll
    for (int t = 0; t < 2; ++t)
        y[(o.row0 + r) * a.d + o.nt * 32 + 16 * t + (idx & 15)] = (uint16_t)f32_to_bf16_bits(wave_sum(red, t, idx));
}

// out[t] = sum_j topk_w_j (h_j W2[e_j]^T) of 16 columns of token blockIdx.y: the
// slots' K ranges are one long sum, each slot's scales times its weight
template <int G>
__global__ __launch_bounds__(64 * kW) void int4_down_token_kernel(Int4Ffn a, const uint16_t* __restrict__ h)
{
    __shared__ float red[kW][1][256];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int t = blockIdx.y, m = lane & 15;
    const int chunks = (a.f + 127) / 128;
    f32x4 acc[1] = {};
    for (int i = wave; i < a.k * chunks; i += kW) {
        const int j = i / chunks;
        const int64_t p = (int64_t)t * a.k + j;
        const int e = a.topk_idx[p], dst = a.dst_row[p];
        if (e < 0 || e >= a.E || dst < 0 || dst >= a.T * a.k) continue;
        const uint16_t* x = m == 0 ? h + p * a.f : nullptr;
        const WRow w[1] = {w_row(a.w2, (int64_t)e * a.d + blockIdx.x * 16 + m, a.f, G)};
        chunk_product<G, 1>(acc, x, w, i - j * chunks, a.f, a.topk_w[p]);
    }
    put_acc(red, acc);
    if (threadIdx.x < 16)
        a.out[(int64_t)t * a.d + blockIdx.x * 16 + threadIdx.x] = (uint16_t)f32_to_bf16_bits(wave_sum(red, 0, threadIdx.x));
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

constexpr int64_t kMaxBlocks = 1 << 20;
unsigned grid_of(int64_t n) { return (unsigned)(n < 256 * kMaxBlocks ? (n + 255) / 256 : kMaxBlocks); }

template <class F>
hipError_t with_group(int group, F&& f)
{
    switch (group) {
    case 32: f(std::integral_constant<int, 32>{}); break;
    case 64: f(std::integral_constant<int, 64>{}); break;
    case 128: f(std::integral_constant<int, 128>{}); break;
    default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_int4(const uint16_t* src, int64_t rows, int K, int group, uint8_t* codes, uint16_t* scales,
                                uint8_t* zeros, hipStream_t s)
{
    const int64_t n8 = rows * (K / 8);
    if (n8 == 0) return hipSuccess;
    return with_group(group, [&](auto g) {
        constexpr int G = decltype(g)::value;
        if (zeros)
            hipLaunchKernelGGL((quantize_int4_kernel<G, true>), dim3(grid_of(n8)), dim3(256), 0, s, (const uint4*)src, n8,
                               (uint32_t*)codes, scales, zeros);
        else
            hipLaunchKernelGGL((quantize_int4_kernel<G, false>), dim3(grid_of(n8)), dim3(256), 0, s, (const uint4*)src, n8,
                               (uint32_t*)codes, scales, zeros);
    });
}

hipError_t launch_dequantize_int4(const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros, int64_t rows,
                                  int K, int group, uint16_t* dst, hipStream_t s)
{
    const int64_t n8 = rows * (K / 8);
    if (n8 == 0) return hipSuccess;
    return with_group(group, [&](auto g) {
        hipLaunchKernelGGL((dequantize_int4_kernel<decltype(g)::value>), dim3(grid_of(n8)), dim3(256), 0, s,
                           (const uint32_t*)codes, scales, zeros, n8, (uint4*)dst);
    });
}

size_t int4_ws_bytes(int64_t n_rows, int d, int f)
{
    return up256((size_t)n_rows * f * 2) + up256((size_t)n_rows * d * 2) + 256;
}

hipError_t launch_int4_ffn(const Int4Ffn& a, hipStream_t s)
{
    if (a.T == 0) return hipSuccess;
    const int64_t R = (int64_t)a.T * a.k;
    uint16_t* h = reinterpret_cast<uint16_t*>(a.ws);
    uint16_t* y = reinterpret_cast<uint16_t*>(reinterpret_cast<uint8_t*>(a.ws) + up256((size_t)R * a.f * 2));
    const dim3 blk(64 * kW);
    if (a.T == 1) {
        return with_group(a.group, [&](auto g) {
            constexpr int G = decltype(g)::value;
            hipLaunchKernelGGL((int4_gate_up_kernel<G, true>), dim3(a.f / 16, (unsigned)R), blk, 0, s, a, h);
            hipLaunchKernelGGL((int4_down_token_kernel<G>), dim3(a.d / 16, (unsigned)a.T), blk, 0, s, a, h);
        });
    }
    // tiles of up to 16 rows: no more than the rows, nor than the full ones and one of each expert
    const int64_t mt = R < R / 16 + a.E ? R : R / 16 + a.E;
    auto grid = [&](int ntn) { return dim3((unsigned)((mt * ntn + 7) / 8 * 8)); };
    const hipError_t e = with_group(a.group, [&](auto g) {
        constexpr int G = decltype(g)::value;
        hipLaunchKernelGGL((int4_gate_up_kernel<G, false>), grid(a.f / 16), blk, 0, s, a, h);
        hipLaunchKernelGGL((int4_down_kernel<G>), grid(a.d / 32), blk, 0, s, a, h, y);
    });
    if (e != hipSuccess) return e;
    return launch_combine(MOE_BF16, y, a.dst_row, a.topk_w, a.T, a.k, a.d, R, a.out, a.dev_err, s);
}

}  // namespace moe
