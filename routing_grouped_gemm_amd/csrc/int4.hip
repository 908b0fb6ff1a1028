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
//
// h between the two products is fp16 with a power of two for each row (or 16
// columns of it) that puts its largest element into [2^7, 2^8): eleven
// significant bits.  In bf16, with eight, its rounding costs as much as the
// output's own, and more where a limit makes many elements of h the same and
// their errors add up (outputs of 80 random calls against 64 bits: 2.3e-3 to
// 2.8e-3 of their size off with h in bf16, 1.7e-3 so, their own rounding).
// The down product's operands are fp16 then: a code at bits 6..9 of 0x4c00 is
// 16 + q.  Where matrix instructions need a whole row's scale, the first
// product leaves h in fp32 and a pass of 3 to 5 us a call narrows it.  (Scales
// of 16 columns from the first product's epilogue, brought to one where the
// second loads its rows, are dearer: 245 against 239 us for the few-row
// kernel's example.)
#include "gemm_common.h"

namespace moe {
namespace {

using gemm::bf16x8;
typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
typedef __attribute__((ext_vector_type(8))) _Float16 f16x8;
typedef __attribute__((ext_vector_type(2))) _Float16 f16x2;

// ---------------------------------------------------------------- quantiser
// A lane takes 8 elements, a group's G / 8 lanes (4, 8 or 16 neighbours) find its extremes together.  Bound by the
// reads and writes as long as an element costs few instructions, so:
//   - extremes are found on the bf16 patterns, two to an instruction: as signed integers the largest is the largest
//     positive value, as unsigned ones the largest is the negative value of largest magnitude (if there is one), and
//     either is at least 0x7f80 in its magnitude if an element is not finite;
//   - v / scale is v times the reciprocal r of the scale, moved to a multiple of 2^-13.  v and the scale have 8-bit
//     significands, so the exact quotient is a tie k + 1/2 (a multiple of 2^-13) or at least 2^-10 from one; the
//     product is within 2^-19 of it (|quotient| < 16, two roundings), so moving it lands on the tie if it was one and
//     crosses none if it was not: what is rounded to an integer rounds as the exact quotient does;
//   - the integer comes from adding 1.5 * 2^23 + 16 (even: ties stay ties of the same parity), four of them share a word
//     from there on.
// [49152, 4096] with groups of 128: quantised in 82 us (6.2 TB/s, caches cold or not; with a division an element twice as
// long), decoded in 109 with the caches cold (4.7 TB/s) and 70 where they hold part of the codes.
constexpr int kVec = 2;                   // vectors a thread, their loads in flight together
constexpr int64_t kMaxBlocks = 1 << 20;
typedef __attribute__((ext_vector_type(4))) uint32_t vu4;
typedef __attribute__((ext_vector_type(2))) short s16x2;
typedef __attribute__((ext_vector_type(2))) unsigned short u16x2;

__device__ __forceinline__ uint32_t max_i16(uint32_t a, uint32_t b)
{
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(s16x2, a), __builtin_bit_cast(s16x2, b)));
}
__device__ __forceinline__ uint32_t max_u16(uint32_t a, uint32_t b)
{
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}

// v of the lane `1 << step` away among 16 neighbours
__device__ __forceinline__ uint32_t neighbour(uint32_t v, int step)
{
    switch (step) {
    case 0: return __builtin_amdgcn_update_dpp(0, v, 0xB1, 0xF, 0xF, true);      // lane ^ 1
    case 1: return __builtin_amdgcn_update_dpp(0, v, 0x4E, 0xF, 0xF, true);      // lane ^ 2
    case 2: return __builtin_amdgcn_update_dpp(0, v, 0x141, 0xF, 0xF, true);     // 7 - lane: the other four
    default: return __builtin_amdgcn_update_dpp(0, v, 0x140, 0xF, 0xF, true);    // 15 - lane: the other eight
    }
}

template <int G, bool ZEROS>
__device__ __forceinline__ uint32_t quantize8(vu4 x, uint32_t& scale, uint32_t& zero)
{
    constexpr int STEPS = G == 32 ? 2 : G == 64 ? 3 : 4;
    float hi, lo = 0.0f;
    bool finite;
    if constexpr (ZEROS) {
        uint32_t p = 0, n = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            p = max_i16(p, x[i]);
            n = max_u16(n, x[i]);
        }
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
            p = max_i16(p, neighbour(p, i));
            n = max_u16(n, neighbour(n, i));
        }
        p = max_i16(p, p >> 16) & 0xffffu;
        n = max_u16(n, n >> 16) & 0xffffu;
        hi = __uint_as_float(p << 16);
        lo = n >= 0x8000u ? __uint_as_float(n << 16) : 0.0f;
        finite = p < 0x7f80u && (n & 0x7fffu) < 0x7f80u;
    } else {
        uint32_t p = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) p = max_u16(p, x[i] & 0x7fff7fffu);
#pragma unroll
        for (int i = 0; i < STEPS; ++i) p = max_u16(p, neighbour(p, i));
        p = max_u16(p, p >> 16) & 0xffffu;
        hi = __uint_as_float(p << 16);
        finite = p < 0x7f80u;
    }
    uint32_t sb = f32_to_bf16_bits(ZEROS ? (0.5f * hi - 0.5f * lo) / 7.5f : hi / 7.0f);
    if (sb < 0x0080u) sb = 0x0080u;                      // 2^-126
    const float r = 1.0f / __uint_as_float(sb << 16);
    auto quotient = [r](float v) __attribute__((always_inline)) { return (v * r + 1536.0f) - 1536.0f; };
    const float z = ZEROS ? fminf(rintf(quotient(-lo)), 15.0f) : 8.0f;
    uint32_t b[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        b[2 * i] = __float_as_uint(__builtin_amdgcn_fmed3f(quotient(bf16_lo(x[i])), -z, 15.0f - z) + 12582928.0f);
        b[2 * i + 1] = __float_as_uint(__builtin_amdgcn_fmed3f(quotient(bf16_hi(x[i])), -z, 15.0f - z) + 12582928.0f);
    }
    zero = (uint32_t)z;
    uint32_t out[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        // bytes 16 + round(v / s) of four elements, then the codes, then two codes to a byte
        const uint32_t ab = __builtin_amdgcn_perm(b[4 * i + 1], b[4 * i], 0x0c0c0400u);
        const uint32_t cd = __builtin_amdgcn_perm(b[4 * i + 3], b[4 * i + 2], 0x04000c0cu);
        const uint32_t q = (ab | cd) + zero * 0x01010101u - 0x10101010u;
        out[i] = q | (q >> 4);
    }
    scale = finite ? sb : 0x7fc0u;
    if (!finite) zero = 8;
    return finite ? __builtin_amdgcn_perm(out[1], out[0], 0x06040200u) : 0x88888888u;
}

// runs of 256 kVec vectors a workgroup; STREAM: non-temporal access, for sources past the last-level cache
template <int G, bool ZEROS, bool STREAM>
__global__ __launch_bounds__(256) void quantize_int4_kernel(const vu4* __restrict__ src, int64_t n8,
                                                            uint32_t* __restrict__ codes, uint16_t* __restrict__ scales,
                                                            uint8_t* __restrict__ zeros)
{
    constexpr int LG = G / 8;
    for (int64_t i0 = (int64_t)blockIdx.x * (256 * kVec) + threadIdx.x; i0 < n8; i0 += (int64_t)gridDim.x * (256 * kVec)) {
        vu4 x[kVec];
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            const int64_t i = i0 + 256 * j;
            if (i < n8) x[j] = STREAM ? __builtin_nontemporal_load(src + i) : src[i];
        }
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            const int64_t i = i0 + 256 * j;
            if (i >= n8) break;                          // whole groups stay
            uint32_t s, z;
            const uint32_t c = quantize8<G, ZEROS>(x[j], s, z);
            if constexpr (STREAM) __builtin_nontemporal_store(c, codes + i);
            else codes[i] = c;
            if (threadIdx.x % LG == 0) {
                scales[i / LG] = (uint16_t)s;
                if constexpr (ZEROS) zeros[i / LG] = (uint8_t)z;
            }
        }
    }
}

template <int G, bool STREAM>
__global__ __launch_bounds__(256) void dequantize_int4_kernel(const uint32_t* __restrict__ codes,
                                                              const uint16_t* __restrict__ scales,
                                                              const uint8_t* __restrict__ zeros, int64_t n8,
                                                              vu4* __restrict__ dst)
{
    constexpr int LG = G / 8;
    for (int64_t i0 = (int64_t)blockIdx.x * (256 * kVec) + threadIdx.x; i0 < n8; i0 += (int64_t)gridDim.x * (256 * kVec)) {
        uint32_t c[kVec], s[kVec], z[kVec];
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            const int64_t i = i0 + 256 * j;
            if (i >= n8) break;
            c[j] = codes[i];
            s[j] = scales[i / LG];
            z[j] = zeros ? zeros[i / LG] : 8u;
        }
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            const int64_t i = i0 + 256 * j;
            if (i >= n8) break;
            const float sc = bf16_lo(s[j]), zf = (float)z[j];
            const uint32_t even = c[j] & 0x0f0f0f0fu, odd = (c[j] >> 4) & 0x0f0f0f0fu;   // codes 0 2 4 6 and 1 3 5 7
            vu4 o;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const bf16x2 v = {(__bf16)(((float)((even >> (8 * q)) & 0xffu) - zf) * sc),
                                  (__bf16)(((float)((odd >> (8 * q)) & 0xffu) - zf) * sc)};
                o[q] = __builtin_bit_cast(uint32_t, v);
            }
            if constexpr (STREAM) __builtin_nontemporal_store(o, dst + i);
            else dst[i] = o;
        }
    }
}

// ---------------------------------------------------------------- products
// The two products' operand types: x of the gate and up products is bf16, h of the down product fp16.  What they have in
// common is written once, for words of two elements each.
struct Bf16 {
    static constexpr uint32_t one = 0x3f803f80u, sixteen = 0x41804180u;
    static constexpr int at = 3;          // a code's lowest bit in 16 + q
    static __device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float c)
    {
        return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, a), __builtin_bit_cast(bf16x2, b), c, false);
    }
    static __device__ __forceinline__ f32x4 mfma(uint4 a, uint4 b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    }
    // three numbers that add up to X exactly, two and one to a word
    static __device__ __forceinline__ uint2 split(float X)
    {
        const uint32_t hi = __float_as_uint(X) & 0xffff0000u;
        const float r = X - __uint_as_float(hi);
        const uint32_t mid = __float_as_uint(r) & 0xffff0000u;
        const uint32_t lo = __float_as_uint(r - __uint_as_float(mid));
        return make_uint2((hi >> 16) | mid, lo >> 16);
    }
};

struct F16 {
    static constexpr uint32_t one = 0x3c003c00u, sixteen = 0x4c004c00u;
    static constexpr int at = 6;
    static __device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float c)
    {
        return __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, a), __builtin_bit_cast(f16x2, b), c, false);
    }
    static __device__ __forceinline__ f32x4 mfma(uint4 a, uint4 b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ uint32_t bits(float v) { return __builtin_bit_cast(unsigned short, (_Float16)v); }
    // (a group's sum stays below 128 * 2^8; parts below 2^-24, 2^-32 of a row's largest element, are lost)
    static __device__ __forceinline__ uint2 split(float X)
    {
        const float hi = __uint_as_float(__float_as_uint(X) & 0xffffe000u), r = X - hi;
        const float mid = __uint_as_float(__float_as_uint(r) & 0xffffe000u);
        return make_uint2(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(hi, mid)),
                          __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(r - mid, 0.0f)));
    }
};

// h's scale: the power of two that puts the magnitude with these bits (the largest of a row) into [2^7, 2^8), and its
// inverse, both of them normal numbers.  An infinity or a NaN stays one.
__device__ __forceinline__ float h_scale(uint32_t largest, float& inverse)
{
    const uint32_t e = 261u - (largest >> 23);                  // 127 + 7 - (exponent - 127)
    const uint32_t c = e > 253u ? 253u : e;
    inverse = __uint_as_float((254u - c) << 23);
    return __uint_as_float(c << 23);
}
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// The constants of a conversion, one in a vector register: with two literals the and-or would be two instructions
struct Conv {
    uint32_t mask, base;
};
template <class T>
__device__ __forceinline__ Conv conv()
{
    Conv c{0x000f000fu << T::at, T::sixteen};
    asm("" : "+s"(c.mask));
    asm("" : "+v"(c.base));
    return c;
}

// the numbers 16 + q of eight codes: pairs (0,4) (1,5) (2,6) (3,7)
template <class T>
__device__ __forceinline__ uint4 codes_to(uint32_t w, Conv c)
{
    constexpr int at = T::at;
    return make_uint4(((w << at) & c.mask) | c.base, ((at >= 4 ? w << (at & 3) : w >> 1) & c.mask) | c.base,
                      ((w >> (8 - at)) & c.mask) | c.base, ((w >> (12 - at)) & c.mask) | c.base);
}

// The products' zero points come off by a matrix instruction too: X, a row's sum of x over a group, as three
// numbers that add up to it, times -(16 + z).  x side: lane group 0 has the three (row = lane & 15), the
// others zeros; weight side: the number -(16 + z) of the lane's column.  (The same 32-deep instruction as the
// products': a 16-deep one would do, but a product that took its result as the sum to add to read it too soon,
// without the wait states that mixed depths need.)
template <class T>
__device__ __forceinline__ uint4 split_sum(float X)
{
    const uint2 v = T::split(X);
    return make_uint4(v.x, v.y, 0, 0);
}

template <class T>
__device__ __forceinline__ f32x4 minus_zeros(uint4 X, uint32_t z)
{
    const uint32_t v = (T::sixteen | 0x80008000u) + z * (0x00010001u << T::at);
    return T::mfma(X, make_uint4(v, v, v, v), f32x4{0, 0, 0, 0});
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

// Buffer descriptors over one expert's matrix (zeros: over nothing if there are none, so that they load as 0).
// Sizes stay below 2^31 bytes (checked on the host).
struct WBuf {
    __amdgpu_buffer_rsrc_t codes, scales, zeros;
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buf_of(const void* p, int64_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)bytes, 0x00020000);
}

__device__ __forceinline__ WBuf w_buf(const moe_int4& w, int e, int N, int K, int group)
{
    const int64_t n = (int64_t)N * K, ng = n / group;
    return {buf_of(w.codes + e * (n / 2), n / 2), buf_of((const uint16_t*)w.scales + e * ng, ng * 2),
            buf_of(w.zeros + (w.zeros ? e * ng : 0), w.zeros ? ng : 0)};
}

// (the whole offset in the lane's register: the hardware checks it against the size, and a scalar offset past the
// size of a small buffer could wrap that check)
__device__ __forceinline__ uint4 load16(__amdgpu_buffer_rsrc_t r, uint32_t off)
{
    return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0));
}

// A pair of consecutive chunks of 128 codes of NT column tiles on their way: 16 rows x 128 bytes each in two loads,
// eight neighbouring lanes a row's 128 bytes.  (Each lane loading the codes of its own column, as the matrix operand
// has them, touches 16 rows with every 16 lanes: the address path then bounds the kernel, 168 us where turned codes took
// 145, before later steps, for the gate and up products of the few-row kernel's example.)
// Scale and zero point: lane 4r + j has those of row r and every fourth group, from the j-th on.
template <int G, int NT>
struct Codes {
    static constexpr int NS = (256 / G + 3) / 4;
    uint4 q[NT][2];
    uint32_t s[NS][NT], z[NS][NT];
};

// Where a step's codes lie: the expert's matrix, and the lane's offsets of its rows' first codes and scales.  A step
// that loads nothing has offsets past every buffer.
template <int NT>
struct Where {
    WBuf w;
    uint32_t code[NT], scale[NT];
    int left;                // groups from this lane's first on to the row's end
};
constexpr uint32_t kPast = 0x80000000u;

// column tiles from row0[t] on, chunks from c on
template <int G, int NT>
__device__ __forceinline__ Where<NT> where_of(const WBuf& w, const int (&row0)[NT], int c, int K, bool live)
{
    const int lane = threadIdx.x & 63;
    // (chunks past the row's end within a wave's share are other rows' codes, and not used)
    const uint32_t past = live && c * 128 < K ? 0 : kPast;
    Where<NT> p;
    p.w = w;
    p.left = K / G - c * (128 / G) - (lane & 3);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        p.code[t] = (uint32_t)((row0[t] + (lane >> 3)) * (K / 2) + c * 64 + 16 * (lane & 7)) | past;
        p.scale[t] = (uint32_t)((row0[t] + (lane >> 2)) * (K / G) + c * (128 / G) + (lane & 3)) | past >> 1;
    }
    return p;
}

template <int G, int NT>
__device__ __forceinline__ void load_pair(Codes<G, NT>& o, const Where<NT>& p, int K)
{
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        o.q[t][0] = load16(p.w.codes, p.code[t]);
        o.q[t][1] = load16(p.w.codes, p.code[t] + 4 * K);     // eight rows on
    }
}

template <int G, int NT>
__device__ __forceinline__ void load_scales(Codes<G, NT>& o, const Where<NT>& p, int i)
{
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        // a group past the row's end is the next row's, whose scale may be a NaN: none is loaded for it
        const uint32_t past = p.left > 4 * i ? 0 : kPast;
        o.s[i][t] = __builtin_amdgcn_raw_buffer_load_b16(p.w.scales, (int)((p.scale[t] * 2 + 8 * i) | past), 0, 0);
        o.z[i][t] = __builtin_amdgcn_raw_buffer_load_b8(p.w.zeros, (int)((p.scale[t] + 4 * i) | past), 0, 0);
    }
}

template <int G, int NT>
__device__ __forceinline__ void load_all(Codes<G, NT>& o, const Where<NT>& p, int K)
{
    // in the order in which they will be waited for, here as in the loop: the compiler counts the loads in flight
    load_scales(o, p, 0);
    __builtin_amdgcn_sched_barrier(0);
    load_pair(o, p, K);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (Codes<G, NT>::NS == 2) load_scales(o, p, 1);
    __builtin_amdgcn_sched_barrier(0);
}

// A wave's own LDS: a pair of chunks passes through it from the lanes that loaded it to those whose column it is.
// Part p (16 bytes) of row r lies at part p ^ (r / 2), so that the sixteen rows of a lane group's read and the eight
// parts of a row's write each fall on different banks.
template <int NT>
struct Turn {
    uint4 part[NT][16][8];
};

__device__ __forceinline__ void wave_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

template <int G, int NT>
__device__ __forceinline__ void put_pair(Turn<NT>& turn, const Codes<G, NT>& w)
{
    const int lane = threadIdx.x & 63, r = lane >> 3, p = lane & 7;
    wave_fence();
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        turn.part[t][r][p ^ (r >> 1)] = w.q[t][0];
        turn.part[t][r + 8][p ^ ((r + 8) >> 1)] = w.q[t][1];
    }
    wave_fence();
}

// A pair of chunks of a lane's row of x (bf16) or h (fp16, in the codes' order already) as matrix operands, and each
// group's sum over the row (lane group 0; 0 in the others)
template <int G, class T>
struct XRows {
    static constexpr int U = 2;
    static constexpr int PER = G / 32;                           // MFMAs of a group
    static constexpr int GROUPS = U * 128 / G;
    uint4 f[U][4];
    float X[GROUPS];

    // chunks c and c + 1 of the row at byte `at`
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t x, uint32_t at, int c, int K)
    {
        const int g = (threadIdx.x & 63) >> 4;
        const uint32_t off = at + c * 256 + (G == 128 ? 64 * g : 16 * g);
        uint4 v[U][4];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) v[u][i] = load16(x, off + 256 * u + (G == 128 ? 16 : 64) * i);
        if ((c + U) * 128 > K) {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if ((c + u) * 128 + 32 * (G == 128 ? g : i) >= K) v[u][i] = make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) f[u][i] = std::is_same_v<T, F16> ? v[u][i] : pair_order(v[u][i]);
        const uint4 ones = make_uint4(T::one, T::one, T::one, T::one);
#pragma unroll
        for (int n = 0; n < GROUPS; ++n) {
            f32x4 s = {0, 0, 0, 0};                              // ones on the weight side's place: column = row of x
#pragma unroll
            for (int i = 0; i < PER; ++i) s = T::mfma(ones, f[(n * PER + i) / 4][(n * PER + i) % 4], s);
            X[n] = g == 0 ? s[0] : 0.0f;
        }
    }
};

// acc[t] += (x rows) . (weight rows) over the first n chunks.  ahead() is called when the codes have left their
// registers, ahead_scales(i) when the i-th scales have.
template <int G, int NT, class T, class F, class S>
__device__ __forceinline__ void product(f32x4 (&acc)[NT], const XRows<G, T>& x, Codes<G, NT>& w, Turn<NT>& turn, uint32_t z8,
                                        int n, Conv cv, F&& ahead, S&& ahead_scales)
{
    constexpr int PER = G / 32, GC = 128 / G;                    // MFMAs of a group, groups of a chunk
    const int lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
    uint32_t sz[NT][4];      // bf16 scale in the upper half, zero point below
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        if (u * GC % 4 == 0) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const uint32_t v = (w.s[u * GC / 4][t] << 16) | (w.z[u * GC / 4][t] + z8);
#pragma unroll
                for (int j = 0; j < 4; ++j) sz[t][j] = __builtin_amdgcn_ds_bpermute(4 * (4 * m + j), (int)v);
            }
            ahead_scales(u * GC / 4);
        }
        if (u == 0) {
            put_pair(turn, w);
            ahead();
        }
        if (u < n) {
            uint4 q[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                q[t] = turn.part[t][m][(4 * u + g) ^ (m >> 1)];
                if constexpr (G != 128) q[t] = exchange4(q[t]);
            }
#pragma unroll
            for (int b = 0; b < GC; ++b) {
                const int gi = u * GC + b;
                const uint4 X = split_sum<T>(x.X[gi]);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const uint32_t qw[4] = {q[t].x, q[t].y, q[t].z, q[t].w};
                    f32x4 p = minus_zeros<T>(X, sz[t][gi % 4] & 0xffu);
#pragma unroll
                    for (int i = 0; i < PER; ++i) p = T::mfma(x.f[u][b * PER + i], codes_to<T>(qw[b * PER + i], cv), p);
                    const float sc = bf16_hi(sz[t][gi % 4]);
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[t][r] = fmaf(sc, p[r], acc[t][r]);
                }
            }
        }
    }
}

constexpr int kWaves = 16;     // most waves of a workgroup

// sum over the waves of element idx (row idx / 16, column idx % 16) of column tile t
template <int NT>
__device__ __forceinline__ float wave_sum(const float (*red)[NT][256], int waves, int t, int idx)
{
    // (eight reads on their way together: those past the last wave's are that one's again, and not added)
    float v = 0.0f;
    for (int w0 = 0; w0 < waves; w0 += 8) {
        float p[8];
#pragma unroll
        for (int w = 0; w < 8; ++w) p[w] = red[min(w0 + w, waves - 1)][t][idx];
#pragma unroll
        for (int w = 0; w < 8; ++w) v += w0 + w < waves ? p[w] : 0.0f;
    }
    return v;
}

template <int NT>
__device__ __forceinline__ void put_acc(float (*red)[NT][256], const f32x4 (&acc)[NT])
{
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) red[wave][t][((lane >> 4) * 4 + r) * 16 + (lane & 15)] = acc[t][r];
    __syncthreads();
}

// s_pref[e] = tiles of the experts before e (ceil(rows / 16) * ntn each), s_pref[E] = all: the first wave scans the
// offsets, up to 16 experts a lane
__device__ __forceinline__ int tile_prefix(const Int4Ffn& a, int ntn, int* s_pref)
{
    if (threadIdx.x < 64) {
        const int per = (a.E + 63) >> 6, g0 = threadIdx.x * per;
        const int64_t R = (int64_t)a.T * a.k;
        int cnt = 0;
        for (int i = 0; i < per && g0 + i < a.E; ++i) cnt += (int)((group_rows(a.group_off, 0, g0 + i, R) + 15) / 16) * ntn;
        int incl = cnt;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int v = __shfl_up(incl, off, 64);
            if ((int)threadIdx.x >= off) incl += v;
        }
        int run = incl - cnt;
        for (int i = 0; i < per && g0 + i < a.E; ++i) {
            s_pref[g0 + i] = run;
            run += (int)((group_rows(a.group_off, 0, g0 + i, R) + 15) / 16) * ntn;
        }
        if (threadIdx.x == 63) s_pref[a.E] = incl;
    }
    __syncthreads();
    return s_pref[a.E];
}

// The products of up to 16 rows of an expert with 16 NC of its columns (a tile), tiles expert after expert, rows
// then columns.  A workgroup takes a run of tiles; its W waves share K, a pair of chunks each.  The rows' operands and
// sums stay in registers from tile to tile, and the next tile's codes are on their way while one is multiplied, so that a
// workgroup's loads never stop.  K over 256 W takes several steps a tile, which load the rows each time.
// Four waves a SIMD (at most 128 registers): a workgroup's waves go to the SIMDs in turn from the first, so two of six
// waves each put four on it, and with registers for three the second would wait for the first to end (down product of 64
// experts, K = 1408: 114 us a pass so, 88 with four).
// 67 tokens, top-4 of 128 experts, d 4096, f 1536, groups of 128 with zero points, passes apart: 141 us for the gate and up
// products (5.3 TB/s of codes and scales; loads alone, multiplied with nothing, 137), 91 for the down one (4.1 TB/s; 75: its
// tiles are shorter, and each ends with a sum over the waves).  Passes back to back take 20% longer in the median, the power
// limit lowers the clock: 162 and 107.
//   GATE_UP  h = a(g') u', in fp32: column tiles 0 .. NC - 1 are the gate's, then the up ones.
//   else     y = h W2^T, h as int4_narrow_kernel leaves it
template <int G, bool GATE_UP>
__global__ __launch_bounds__(64 * kWaves) __attribute__((amdgpu_waves_per_eu(4))) void int4_rows_kernel(
    Int4Ffn a, float* __restrict__ h32, const uint16_t* __restrict__ h, const float* __restrict__ hinv, float* __restrict__ y)
{
    using T = std::conditional_t<GATE_UP, Bf16, F16>;
    constexpr int NC = GATE_UP ? 1 : 2, NT = 2, U = 2;
    const int W = blockDim.x >> 6;
    extern __shared__ __align__(16) uint8_t smem[];
    Turn<NT>* turn = reinterpret_cast<Turn<NT>*>(smem);
    float (*red)[NT][256] = reinterpret_cast<float (*)[NT][256]>(smem + W * sizeof(Turn<NT>));   // [2 W]
    __shared__ float factor[2][16];      // of a row's results: 0 for a foreign one
    __shared__ int s_pref[kMaxExperts + 1];
    const int N = GATE_UP ? a.f : a.d, K = GATE_UP ? a.d : a.f;
    const int ntn = (N + 16 * NC - 1) / (16 * NC);
    const int total = tile_prefix(a, ntn, s_pref);
    const int first = (int)((int64_t)blockIdx.x * total / gridDim.x);
    const int last = (int)((int64_t)(blockIdx.x + 1) * total / gridDim.x);
    if (first >= last) return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int m = lane & 15;
    const int chunks = (K + 127) / 128;
    const int blocks = (chunks + W * U - 1) / (W * U);           // steps a tile

    struct Tile {
        int e, nt, valid;
        int64_t row0;
    };
    const int64_t R = (int64_t)a.T * a.k;
    auto tile_at = [&](int L) __attribute__((always_inline)) {
        Tile t;
        t.e = find_group(s_pref, a.E, L);
        const int local = L - s_pref[t.e], mt = local / ntn;
        t.nt = local - mt * ntn;
        t.row0 = group_begin(a.group_off, 0, t.e, R) + 16 * mt;
        t.valid = (int)min((int64_t)16, group_rows(a.group_off, 0, t.e, R) - 16 * mt);
        return t;
    };

    const int steps = (last - first) * blocks;
    const auto xb = GATE_UP ? buf_of(a.x, (int64_t)a.T * a.d * 2) : buf_of(h, R * a.f * 2);
    uint32_t xat = 0;
    float mine = 1.0f;
    int64_t have = -1;       // row of h whose tile's operands are held
    XRows<G, T> x;
    f32x4 acc[NT];
    int buf = 0;

    auto where = [&](const Tile& t, int kb, bool live) __attribute__((always_inline)) {
        int row[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) row[i] = (i < NC ? 0 : N) + min((t.nt * NC + i % NC) * 16, N - 16);
        return where_of<G>(w_buf(GATE_UP ? a.w13 : a.w2, t.e, GATE_UP ? 2 * N : N, K, G), row, (kb * W + wave) * U, K, live);
    };
    const uint32_t z8 = (GATE_UP ? a.w13 : a.w2).zeros ? 0 : 8;
    const Conv cv = conv<T>();
    auto step = [&](Codes<G, NT>& c, const Tile& t, int kb, const Where<NT>& p) __attribute__((always_inline)) {
        const int c0 = (kb * W + wave) * U, n = min(U, chunks - c0);
        if (have != t.row0 || blocks > 1) {
            if (have != t.row0) {
                // rows past the tile's last are that one again
                const int64_t row = t.row0 + min(m, t.valid - 1);
                if constexpr (GATE_UP) {
                    const int64_t slot = a.src_slot[row];
                    const bool in = slot >= 0 && slot < R;
                    mine = in ? 1.0f : 0.0f;
                    if (slot >= R && a.dev_err && threadIdx.x < 16)
                        atomicOr(a.dev_err, (int)MOE_ERR_ROW_RANGE);
                    xat = in ? (uint32_t)(slot / a.k * a.d * 2) : 0;
                } else {
                    xat = (uint32_t)(row * a.f * 2);
                    mine = hinv[row];
                }
                have = t.row0;
            }
            x.load(xb, xat, c0, K);
        }
        if (kb == 0) {
#pragma unroll
            for (int i = 0; i < NT; ++i) acc[i] = f32x4{0, 0, 0, 0};
        }
        product<G, NT, T>(acc, x, c, turn[wave], z8, n, cv, [&]() __attribute__((always_inline)) { load_pair(c, p, K); },
                       [&](int i) __attribute__((always_inline)) { load_scales(c, p, i); });
        if (kb + 1 < blocks) return;
        if (threadIdx.x < 16) factor[buf][m] = mine;
        put_acc<NT>(red + buf * W, acc);
        for (int i = threadIdx.x; i < NC * 256; i += 64 * W) {
            const int idx = i & 255, j = i >> 8, r = idx >> 4, col = (t.nt * NC + j) * 16 + (idx & 15);
            if (r >= t.valid || col >= N) continue;
            float v = wave_sum<NT>(red + buf * W, W, j, idx);
            if constexpr (GATE_UP) {
                const float L = a.glu.limit, g = limit_g(v, L), u = limit_u(wave_sum<NT>(red + buf * W, W, j + NC, idx), L);
                with_act(a.glu.act, [&](auto A) __attribute__((always_inline)) { v = act_of<decltype(A)::value, true>(g) * u; });
                h32[(t.row0 + r) * a.f + col] = factor[buf][r] ? v : 0.0f;
            } else {
                y[(t.row0 + r) * a.d + col] = v * factor[buf][r];
            }
        }
        buf ^= 1;
    };
    // a chunk's registers take the next step's codes as soon as they are used
    Codes<G, NT> codes;
    Tile t = tile_at(first), tn = t;
    load_all(codes, where(t, 0, true), K);
    for (int s = 0, at = first, kb = 0; s < steps; ++s) {
        int kn = kb + 1;
        if (kn == blocks) {
            kn = 0;
            ++at;
            if (++tn.nt == ntn && at < last) tn = tile_at(at);
        }
        step(codes, t, kb, where(tn, kn, s + 1 < steps));
        t = tn;
        kb = kn;
    }
}

// ---------------------------------------------------------------- many rows an expert
// Tiles of 64 rows: each of four waves has 32 columns (16 and 16 of gate and up) of its own and all the rows, so that
// a code is converted once for 64 products.  x passes through LDS in chunks of 128, two in turn and one barrier a chunk;
// codes as in the kernel for few rows.  Bound by the issue of vector instructions, so what a row needs once is not done
// again for each tile of columns: rows come in the codes' order with their sums (fp32, over each 32), x from
// int4_order_kernel, h from int4_narrow_kernel.
// 1000 tokens, top-2 of 8 experts, d 2048, f 1152, groups of 64 with zero points: 54 us for the gate and up products, 34
// for the down one (350 and 280 TFLOP/s), 5 each for the order of x and h's narrowing; with order and sums made in every
// tile and the compiler's order of loads from LDS 62 and 39.  Eight waves a workgroup, which share x among more columns: 71.
constexpr int kTileRows = 64, kTileWaves = 4;

struct XStage {
    uint4 part[2][kTileRows][16];            // part p of row r at p ^ (r & 15)
    uint4 sum[2][4][kTileRows];              // a row's sum over group b of the chunk, as split_sum has it
    uint4 none[kTileRows];                   // zeros, what lane groups 1 to 3 take for it
};

// eight elements of a row in the codes' order, and in each of four neighbouring lanes the sum of their 32
template <class T>
__device__ __forceinline__ uint4 order_and_sum(uint4 v, float& sum)
{
    v = pair_order(v);
    sum = T::dot2(v.x, T::one, T::dot2(v.y, T::one, T::dot2(v.z, T::one, T::dot2(v.w, T::one, 0.0f))));
    sum += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(sum), 0xB1, 0xF, 0xF, true));
    sum += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(sum), 0x4E, 0xF, 0xF, true));
    return v;
}

// x [n8 vectors] in that order, and its sums
__global__ __launch_bounds__(256) void int4_order_kernel(const uint4* __restrict__ x, int64_t n8, uint4* __restrict__ xo,
                                                         float* __restrict__ sums)
{
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n8; i += (int64_t)gridDim.x * 256) {
        float sum;
        xo[i] = order_and_sum<Bf16>(x[i], sum);
        if (threadIdx.x % 4 == 0) sums[i / 4] = sum;
    }
}

// h in fp32 -> fp16 in the codes' order, a scale for each row and its inverse (hinv), and the sums of what is stored.
// TPR threads share a row; a thread's first eight elements stay in its registers between the row's largest and the
// rounding, the others are read again.
template <int TPR>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void int4_narrow_kernel(const float* __restrict__ h32, int64_t rows, int f,
                                                                          uint4* __restrict__ h, float* __restrict__ hsum,
                                                                          float* __restrict__ hinv)
{
    constexpr int ROWS = TPR < 256 ? 256 / TPR : 1;
    const int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / TPR;
    const int lane = threadIdx.x % TPR, n8 = f / 8;
    if (row >= rows) return;                             // (whole waves; a row of several has its workgroup to itself)
    const float4* src = reinterpret_cast<const float4*>(h32 + row * f);
    auto largest_of = [](float4 a, float4 b) __attribute__((always_inline)) {
        const uint32_t p = max(max(magnitude(a.x), magnitude(a.y)), max(magnitude(a.z), magnitude(a.w)));
        return max(p, max(max(magnitude(b.x), magnitude(b.y)), max(magnitude(b.z), magnitude(b.w))));
    };
    float4 a{}, b{};
    if (lane < n8) {
        a = src[2 * lane];
        b = src[2 * lane + 1];
    }
    uint32_t largest = largest_of(a, b);
    for (int i = lane + TPR; i < n8; i += TPR) largest = max(largest, largest_of(src[2 * i], src[2 * i + 1]));
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) largest = max(largest, (uint32_t)__shfl_xor((int)largest, o, 64));
    if constexpr (TPR > 64) {
        __shared__ uint32_t of_wave[TPR / 64];
        if (threadIdx.x % 64 == 0) of_wave[threadIdx.x / 64] = largest;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < TPR / 64; ++i) largest = max(largest, of_wave[i]);
    }
    float inverse;
    const float scale = h_scale(largest, inverse);
    if (lane == 0) hinv[row] = inverse;
    for (int i = lane; i < n8; i += TPR) {               // (n8 is a multiple of 4: four neighbours stay together)
        if (i != lane) {
            a = src[2 * i];
            b = src[2 * i + 1];
        }
        const uint4 v = make_uint4(F16::bits(a.x * scale) | F16::bits(a.y * scale) << 16,
                                   F16::bits(a.z * scale) | F16::bits(a.w * scale) << 16,
                                   F16::bits(b.x * scale) | F16::bits(b.y * scale) << 16,
                                   F16::bits(b.z * scale) | F16::bits(b.w * scale) << 16);
        float sum;
        h[row * n8 + i] = order_and_sum<F16>(v, sum);
        if (lane % 4 == 0) hsum[(row * n8 + i) / 4] = sum;
    }
}

// rows of x (else: of h) and their sums as above -> h in fp32 (y)
template <int G, bool GATE_UP>
__global__ __launch_bounds__(64 * kTileWaves) __attribute__((amdgpu_waves_per_eu(2))) void int4_tile_kernel(
    Int4Ffn a, const uint16_t* __restrict__ rows, const float* __restrict__ sums, const float* __restrict__ hinv,
    float* __restrict__ result)
{
    using T = std::conditional_t<GATE_UP, Bf16, F16>;
    constexpr int NT = 2, NC = GATE_UP ? 1 : 2, MT = kTileRows / 16, GC = 128 / G, PER = G / 32;
    constexpr int XR = kTileRows / (4 * kTileWaves);     // rows that a thread brings in
    extern __shared__ __align__(16) uint8_t smem[];
    XStage& xs = *reinterpret_cast<XStage*>(smem);
    Turn<NT>* turn = reinterpret_cast<Turn<NT>*>(smem + sizeof(XStage));
    const int N = GATE_UP ? a.f : a.d, K = GATE_UP ? a.d : a.f;
    const int64_t R = (int64_t)a.T * a.k;
    gemm::MTile tile;
    if (!gemm::schedule_m<kTileRows>(a.group_off, 0, a.E, R, (N + 16 * NC * kTileWaves - 1) / (16 * NC * kTileWaves), tile)) return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int m = lane & 15, g = lane >> 4;
    const int chunks = (K + 127) / 128;

    // this thread's rows (threadIdx.x / 16 + 16 i) and 16 bytes of each chunk; and one row's sum over 32
    const int64_t n = GATE_UP ? a.T : R;
    const auto xb = buf_of(rows, n * K * 2), sb = buf_of(sums, n * (K / 32) * 4);
    auto row_of = [&](int r) __attribute__((always_inline)) {
        const int64_t row = tile.row0 + min(r, tile.rows_valid - 1);
        if constexpr (GATE_UP) {
            const int64_t slot = a.src_slot[row];
            if (slot >= R && a.dev_err) atomicOr(a.dev_err, (int)MOE_ERR_ROW_RANGE);
            return slot >= 0 && slot < R ? slot / a.k : (int64_t)-1;     // a foreign row is one of zeros: so is its h
        } else {
            return row;
        }
    };
    const int xp = threadIdx.x & 15, sr = 16 * wave + (lane >> 2), s32 = lane & 3;
    uint32_t xat[XR];
#pragma unroll
    for (int i = 0; i < XR; ++i) {
        const int64_t row = row_of((threadIdx.x >> 4) + 4 * kTileWaves * i);
        xat[i] = row < 0 ? kPast : (uint32_t)(row * K * 2 + 16 * xp);
    }
    const int64_t srow = row_of(sr);
    const uint32_t sat = srow < 0 ? kPast : (uint32_t)((srow * (K / 32) + s32) * 4);
    uint4 xr[XR];
    float xsum;
    auto load_x = [&](int c, int i) __attribute__((always_inline)) {
        xr[i] = load16(xb, (xat[i] + c * 256) | (c * 128 + 8 * xp < K ? 0 : kPast));
    };
    auto load_sum = [&](int c) __attribute__((always_inline)) {
        xsum = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(sb, (int)((sat + c * 16) | (c * 128 + 32 * s32 < K ? 0 : kPast)), 0, 0));
    };
    auto put_x = [&](int st, int i) __attribute__((always_inline)) {
        const int r = (threadIdx.x >> 4) + 4 * kTileWaves * i;
        xs.part[st][r][xp ^ (r & 15)] = xr[i];
    };
    auto put_sum = [&](int st) __attribute__((always_inline)) {
        float v = xsum;
        if constexpr (G >= 64) v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xF, 0xF, true));
        if constexpr (G >= 128) v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4E, 0xF, 0xF, true));
        xs.sum[st][s32 / (G / 32)][sr] = split_sum<T>(v);       // (by each of a group's lanes: no branch among the products)
    };

    int row0[NT];
    const int wn = tile.nt * kTileWaves + wave;      // this wave's columns
#pragma unroll
    for (int t = 0; t < NT; ++t) row0[t] = (t < NC ? 0 : N) + min((wn * NC + t % NC) * 16, N - 16);
    const WBuf wb = w_buf(GATE_UP ? a.w13 : a.w2, tile.e, GATE_UP ? 2 * N : N, K, G);
    const bool live = wn * NC * 16 < N;

    f32x4 acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[i][t] = f32x4{0, 0, 0, 0};
    Codes<G, NT> w;
    uint32_t sz[NT][4];
    const uint32_t z8 = (GATE_UP ? a.w13 : a.w2).zeros ? 0 : 8;
    const Conv cv = conv<T>();
    if (threadIdx.x < kTileRows) xs.none[threadIdx.x] = make_uint4(0, 0, 0, 0);
    load_all(w, where_of<G>(wb, row0, 0, K, live), K);
#pragma unroll
    for (int i = 0; i < XR; ++i) load_x(0, i);
    load_sum(0);
#pragma unroll
    for (int i = 0; i < XR; ++i) {
        put_x(0, i);
        load_x(1, i);
    }
    put_sum(0);
    load_sum(1);
    __syncthreads();
    // Four 32-deep steps a chunk.  Each has the next one's operands on their way from LDS, and brings in a share of the
    // next chunk's x beside its products; the barriers to the scheduler keep that order.
    auto chunk = [&](int c, auto U_) __attribute__((always_inline)) {
        constexpr int u = decltype(U_)::value;           // which of the pair
        if (u * GC % 4 == 0) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const uint32_t v = (w.s[u * GC / 4][t] << 16) | (w.z[u * GC / 4][t] + z8);
#pragma unroll
                for (int j = 0; j < 4; ++j) sz[t][j] = __builtin_amdgcn_ds_bpermute(4 * (4 * m + j), (int)v);
            }
            load_scales(w, where_of<G>(wb, row0, c + 2 - u, K, live), u * GC / 4);
        }
        if (u == 0) {
            put_pair(turn[wave], w);
            load_pair(w, where_of<G>(wb, row0, c + 2, K, live), K);
        }
        uint4 q[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) q[t] = turn[wave].part[t][m][(4 * u + g) ^ (m >> 1)];
        uint4 xf[2][MT];
        uint4 X[MT];
        auto read = [&](int j) __attribute__((always_inline)) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                if (j % PER == 0) X[mt] = (g == 0 ? xs.sum[u][j / PER] : xs.none)[16 * mt + m];
                xf[j & 1][mt] = xs.part[u][16 * mt + m][(G == 128 ? 4 * g + j : 4 * j + g) ^ m];
            }
        };
        read(0);
        if constexpr (G != 128) {
#pragma unroll
            for (int t = 0; t < NT; ++t) q[t] = exchange4(q[t]);
        }
        f32x4 p[MT][NT];
        auto begin = [&](int t, int b) __attribute__((always_inline)) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) p[mt][t] = minus_zeros<T>(X[mt], sz[t][(u * GC + b) % 4] & 0xffu);
        };
#pragma unroll
        for (int t = 0; t < NT; ++t) begin(t, 0);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            __builtin_amdgcn_sched_barrier(0);
            if (j < 3) read(j + 1);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const uint4 wf = codes_to<T>(j == 0 ? q[t].x : j == 1 ? q[t].y : j == 2 ? q[t].z : q[t].w, cv);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) p[mt][t] = T::mfma(xf[j & 1][mt], wf, p[mt][t]);
            }
#pragma unroll
            for (int i = j * XR / 4; i < (j + 1) * XR / 4; ++i) {
                put_x(1 - u, i);
                load_x(c + 2, i);
            }
            if (j == 3) {
                put_sum(1 - u);
                load_sum(c + 2);
            }
            if (j % PER < PER - 1) continue;
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                // (one column tile's sums are scaled while the other's next group begins)
                const float sc = bf16_hi(sz[t][(u * GC + j / PER) % 4]);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[mt][t][r] = fmaf(sc, p[mt][t][r], acc[mt][t][r]);
                __builtin_amdgcn_sched_barrier(0);
                if (j < 3) begin(t, (j + 1) / PER);
            }
        }
        __syncthreads();
    };
    for (int c = 0; c + 1 < chunks; c += 2) {
        chunk(c, std::integral_constant<int, 0>{});
        chunk(c + 1, std::integral_constant<int, 1>{});
    }
    if (chunks & 1) chunk(chunks - 1, std::integral_constant<int, 0>{});

    // the tile leaves through LDS as rows (the loop's last barrier has freed it)
    constexpr int COLS = 16 * NC * kTileWaves, PITCH = COLS + 4;
    static_assert(kTileRows * PITCH * sizeof(float) <= sizeof(XStage) + kTileWaves * sizeof(Turn<NT>), "the tile fits");
    float* out = reinterpret_cast<float*>(smem);
    auto stage = [&](auto&& value) __attribute__((always_inline)) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int t = 0; t < NC; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) out[(16 * mt + 4 * g + r) * PITCH + (wave * NC + t) * 16 + m] = value(mt, t, r);
    };
    if constexpr (GATE_UP) {
        const float L = a.glu.limit;
        with_act(a.glu.act, [&](auto A) __attribute__((always_inline)) {
            stage([&](int mt, int t, int r) __attribute__((always_inline)) {
                return act_of<decltype(A)::value, true>(limit_g(acc[mt][t][r], L)) * limit_u(acc[mt][t + NC][r], L);
            });
        });
    } else {
        stage([&](int mt, int t, int r) __attribute__((always_inline)) { return acc[mt][t][r]; });
    }
    __syncthreads();
    for (int i = threadIdx.x; i < tile.rows_valid * (COLS / 4); i += 64 * kTileWaves) {
        const int r = i / (COLS / 4), c = 4 * (i % (COLS / 4)), col = tile.nt * COLS + c;
        if (col >= N) continue;
        float4 v = *reinterpret_cast<const float4*>(out + r * PITCH + c);
        if constexpr (!GATE_UP) {
            const float k = hinv[tile.row0 + r];
            v = make_float4(v.x * k, v.y * k, v.z * k, v.w * k);
        }
        *reinterpret_cast<float4*>(result + (tile.row0 + r) * N + col) = v;
    }
}

// ---------------------------------------------------------------- one row at a time
constexpr int kTokenWaves = 8;
// A single row of x has no use for a matrix instruction.  Here a lane multiplies the codes where they arrive: eight
// neighbouring lanes have 256 consecutive codes of a row, 32 each, the same 32 of every row that passes, so that the
// lane's x stay in registers; a wave instruction is eight rows x 128 bytes.  Two products an instruction
// (v_dot2c_f32_bf16, v_dot2c_f32_f16) on the same 16 + q operands.  One token, 4 of 128 experts, d 4096, f 1536: 9.0 and
// 4.5 us for the two kernels, a launch and one chain of load latencies each (its 39 MB take 6.1 us at 6.4 TB/s); with the few-row
// kernel 20 us for the pass.
// 32 consecutive x of a lane in the codes' order, and their sum
struct X32 {
    uint4 v[4];
    float sum;

    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t x, uint32_t at)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = load16(x, at + 16 * i);
    }
    __device__ __forceinline__ void order()
    {
        float a = 0.0f, b = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = pair_order(v[i]);
            a = Bf16::dot2(v[i].x, Bf16::one, a);
            b = Bf16::dot2(v[i].y, Bf16::one, b);
            a = Bf16::dot2(v[i].z, Bf16::one, a);
            b = Bf16::dot2(v[i].w, Bf16::one, b);
        }
        sum = a + b;
    }
    // sum x (q - zero) over a lane's 32 codes
    __device__ __forceinline__ float times(uint4 q, float zero16, Conv cv) const
    {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
        float a = 0.0f, b = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 c = codes_to<Bf16>(w[i], cv);
            a = Bf16::dot2(c.x, v[i].x, a);
            b = Bf16::dot2(c.y, v[i].y, b);
            a = Bf16::dot2(c.z, v[i].z, a);
            b = Bf16::dot2(c.w, v[i].w, b);
        }
        return fmaf(-zero16, sum, a + b);
    }
};

// 32 consecutive h, fp16 with a scale for each 16: the columns that one workgroup of the gate and up products makes
struct H32 {
    uint4 v[4];
    float inv[2], sum;

    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t h, __amdgpu_buffer_rsrc_t hinv, uint32_t at, uint32_t past)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = load16(h, (at * 2 | past) + 16 * i);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            inv[i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(hinv, (int)((at / 4 | past) + 4 * i), 0, 0));
    }
    // the two halves' sums of products with c, each with its scale
    template <class F>
    __device__ __forceinline__ float halves(F&& c) const
    {
        float part[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 w = c(i);
            part[i / 2] = F16::dot2(w.x, v[i].x, part[i / 2]);
            part[i / 2] = F16::dot2(w.y, v[i].y, part[i / 2]);
            part[i / 2] = F16::dot2(w.z, v[i].z, part[i / 2]);
            part[i / 2] = F16::dot2(w.w, v[i].w, part[i / 2]);
        }
        return fmaf(part[0], inv[0], part[1] * inv[1]);
    }
    __device__ __forceinline__ void order()
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = pair_order(v[i]);
        sum = halves([](int) __attribute__((always_inline)) { return make_uint4(F16::one, F16::one, F16::one, F16::one); });
    }
    __device__ __forceinline__ float times(uint4 q, float zero16, Conv cv) const
    {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
        return fmaf(-zero16, sum, halves([&](int i) __attribute__((always_inline)) { return codes_to<F16>(w[i], cv); }));
    }
};

// one load of a lane: its 32 codes of a row, their scale and zero point
struct Q32 {
    uint4 q;
    uint32_t s, z;

    __device__ __forceinline__ void load(const WBuf& w, int row, int k0, int K, int G, uint32_t past)
    {
        const uint32_t at = row * (K / G) + k0 / G;
        q = load16(w.codes, (uint32_t)(row * (K / 2) + k0 / 2) | past);
        s = __builtin_amdgcn_raw_buffer_load_b16(w.scales, (int)(at * 2 | past), 0, 0);
        z = __builtin_amdgcn_raw_buffer_load_b8(w.zeros, (int)(at | past), 0, 0);
    }
    template <class X>
    __device__ __forceinline__ float times(const X& x, uint32_t z8, Conv cv) const
    {
        return bf16_lo(s) * x.times(q, (float)(16 + z8 + z), cv);
    }
};

// sum over eight neighbouring lanes, in each of them
__device__ __forceinline__ float sum8(float v)
{
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xF, 0xF, true));    // lane ^ 1
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4E, 0xF, 0xF, true));    // lane ^ 2
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x141, 0xF, 0xF, true));   // 7 - lane
    return v;
}

// the expert of slot p, or -1 for a slot that adds nothing (flagged if it is out of range)
__device__ __forceinline__ int expert_of(const Int4Ffn& a, int64_t p, bool flag)
{
    const int e = a.topk_idx[p], dst = a.dst_row[p];
    const bool bad = e < 0 || e >= a.E || dst >= a.T * a.k;
    if (bad && flag && a.dev_err && threadIdx.x == 0) atomicOr(a.dev_err, (int)MOE_ERR_ROW_RANGE);
    return bad || dst < 0 ? -1 : e;
}

// h = a(g') u' of 16 columns for slot blockIdx.y, with their scale's inverse: eight waves share K in slices of 256, two at
// a time
template <int G>
__global__ __launch_bounds__(64 * kTokenWaves) void int4_gate_up_token_kernel(Int4Ffn a, uint16_t* __restrict__ h,
                                                                            float* __restrict__ hinv)
{
    constexpr int U = 2;
    __shared__ float red[kTokenWaves][32];
    const int64_t p = blockIdx.y;
    const int e = expert_of(a, p, blockIdx.x == 0);
    if (e < 0) return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int K = a.d, slices = (K + 255) / 256;
    const WBuf w = w_buf(a.w13, e, 2 * a.f, K, G);
    const auto xb = buf_of(a.x, (int64_t)a.T * K * 2);
    const uint32_t xat = (uint32_t)(p / a.k * K * 2), z8 = a.w13.zeros ? 0 : 8;
    const int row = blockIdx.x * 16 + (lane >> 3);
    const Conv cv = conv<Bf16>();
    float acc[4] = {};
    for (int s0 = wave * U; s0 < slices; s0 += kTokenWaves * U) {
        Q32 q[U][4];
        X32 x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k0 = (s0 + u) * 256 + 32 * (lane & 7);
            const uint32_t past = k0 < K ? 0 : kPast;
#pragma unroll
            for (int i = 0; i < 4; ++i) q[u][i].load(w, row + (i & 1) * 8 + (i >> 1) * a.f, k0, K, G, past);
            x[u].load(xb, (xat + k0 * 2) | past);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            x[u].order();
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] += q[u][i].times(x[u], z8, cv);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float v = sum8(acc[i]);
        if ((lane & 7) == 0) red[wave][i * 8 + (lane >> 3)] = v;
    }
    __syncthreads();
    if (threadIdx.x >= 16) return;
    float g = 0.0f, u = 0.0f;
#pragma unroll
    for (int i = 0; i < kTokenWaves; ++i) {
        g += red[i][threadIdx.x];
        u += red[i][16 + threadIdx.x];
    }
    g = limit_g(g, a.glu.limit);
    u = limit_u(u, a.glu.limit);
    float v = 0.0f;
    with_act(a.glu.act, [&](auto A) __attribute__((always_inline)) { v = act_of<decltype(A)::value, true>(g) * u; });
    uint32_t largest = magnitude(v);
#pragma unroll
    for (int i = 0; i < 4; ++i) largest = max(largest, neighbour(largest, i));
    float inverse;
    const float scale = h_scale(largest, inverse);
    h[p * a.f + blockIdx.x * 16 + threadIdx.x] = (uint16_t)F16::bits(v * scale);
    if (threadIdx.x == 0) hinv[p * (a.f / 16) + blockIdx.x] = inverse;
}

// out[t] = sum_j topk_w_j (h_j W2[e_j]^T) of 16 columns of token blockIdx.y: the slices of all its slots are shared by
// eight waves, three at a time, a slice's sum times its slot's weight, so that one sum over the waves is the combine
template <int G>
__global__ __launch_bounds__(64 * kTokenWaves) void int4_down_token_kernel(Int4Ffn a, const uint16_t* __restrict__ h,
                                                                         const float* __restrict__ hinv)
{
    constexpr int U = 3;
    __shared__ float red[kTokenWaves][16];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int64_t t = blockIdx.y;
    const int K = a.f, slices = (K + 255) / 256, items = a.k * slices;
    const auto hb = buf_of(h, (int64_t)a.T * a.k * K * 2), ib = buf_of(hinv, (int64_t)a.T * a.k * (K / 16) * 4);
    const uint32_t z8 = a.w2.zeros ? 0 : 8;
    const int row = blockIdx.x * 16 + (lane >> 3);
    const Conv cv = conv<F16>();
    float acc[2] = {};
    for (int i0 = wave; i0 < items; i0 += kTokenWaves * U) {
        Q32 q[U][2];
        H32 x[U];
        float c[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = min(i0 + u * kTokenWaves, items - 1);
            const int j = i / slices;
            const int64_t p = t * a.k + j;
            const int e = expert_of(a, p, false);
            const bool on = e >= 0 && i0 + u * kTokenWaves < items;
            c[u] = on ? a.topk_w[p] : 0.0f;
            const int k0 = (i - j * slices) * 256 + 32 * (lane & 7);
            const uint32_t past = on && k0 < K ? 0 : kPast;
            const WBuf w = w_buf(a.w2, max(e, 0), a.d, K, G);
            q[u][0].load(w, row, k0, K, G, past);
            q[u][1].load(w, row + 8, k0, K, G, past);
            x[u].load(hb, ib, (uint32_t)(p * K + k0), past);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            x[u].order();
            acc[0] = fmaf(c[u], q[u][0].times(x[u], z8, cv), acc[0]);
            acc[1] = fmaf(c[u], q[u][1].times(x[u], z8, cv), acc[1]);
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float v = sum8(acc[i]);
        if ((lane & 7) == 0) red[wave][i * 8 + (lane >> 3)] = v;
    }
    __syncthreads();
    if (threadIdx.x >= 16) return;
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < kTokenWaves; ++i) v += red[i][threadIdx.x];
    a.out[t * a.d + blockIdx.x * 16 + threadIdx.x] = (uint16_t)f32_to_bf16_bits(v);
}

// out[t] = sum_j topk_w[t, j] * y[dst_row[t, j]] over the slots that have an expert and a row, rounded once: y is fp32, as a
// rounding of it to bf16 would cost as much of the result's accuracy as the output's.  A thread makes 8 columns.
template <int K>
__global__ __launch_bounds__(256) void int4_combine_kernel(const float4* __restrict__ y, const int32_t* __restrict__ topk_idx,
                                                           const int32_t* __restrict__ dst_row, const float* __restrict__ w,
                                                           int T, int E, int d8, uint4* __restrict__ out, int32_t* dev_err)
{
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < (int64_t)T * d8; i += (int64_t)gridDim.x * 256) {
        const int64_t t = i / d8;
        const int v = (int)(i - t * d8);
        float4 a[K], b[K];
        float c[K];
        bool on[K], bad = false;
#pragma unroll
        for (int j = 0; j < K; ++j) {
            const int32_t dst = dst_row[t * K + j];
            const bool foreign = (uint32_t)topk_idx[t * K + j] >= (uint32_t)E || dst >= T * K;
            on[j] = !foreign && dst >= 0;
            bad |= foreign;
            c[j] = w[t * K + j];
            const int64_t at = ((int64_t)(on[j] ? dst : 0) * d8 + v) * 2;
            a[j] = y[at];
            b[j] = y[at + 1];
        }
        float o[8] = {};
#pragma unroll
        for (int j = 0; j < K; ++j) {
            if (!on[j]) continue;
            const float e[8] = {a[j].x, a[j].y, a[j].z, a[j].w, b[j].x, b[j].y, b[j].z, b[j].w};
#pragma unroll
            for (int q = 0; q < 8; ++q) o[q] = fmaf(c[j], e[q], o[q]);
        }
        out[i] = make_uint4(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]), pack_bf16x2(o[4], o[5]), pack_bf16x2(o[6], o[7]));
        if (bad && dev_err) atomicOr(dev_err, (int)MOE_ERR_ROW_RANGE);
    }
}

// CUs of the current device
int cu_count()
{
    int dev = 0, n = 0;
    if (hipGetDevice(&dev) != hipSuccess ||
        hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n < 1)
        n = 256;
    return n;
}

// Where a pass's h and expert outputs lie in the workspace
struct Int4Ws {
    float* h32;       // [R, f]; for single tokens the inverse scales [R, f / 16]
    uint16_t* h;      // [R, f]
    float* hsum;      // [R, f / 32]
    float* hinv;      // [R]
    float* y;         // [R, d]
};

template <int G, bool UP>
void launch_rows(const Int4Ffn& a, const Int4Ws& w, hipStream_t s)
{
    constexpr int NT = 2, COLS = UP ? 16 : 32;
    const int N = UP ? a.f : a.d, K = UP ? a.d : a.f, need = (K + 255) / 256, W = need < kWaves ? need : kWaves;
    const int64_t R = (int64_t)a.T * a.k, cus = cu_count();
    // tiles of up to 16 rows: no more than the rows, nor than the full ones and one of each expert
    const int64_t mt = R < R / 16 + a.E ? R : R / 16 + a.E, tiles = mt * ((N + COLS - 1) / COLS);
    // As many workgroups as fit, 16 waves a CU (64 experts of d 2048, f 1024, 48 tokens of 4: 61 us a pass; with 12 waves
    // 69); 12 where a workgroup would have fewer than two tiles (8 experts, 48 tokens of 2: 27 us; with 16 waves 28.5).
    int64_t per_cu = kWaves / W;
    if (tiles < 2 * cus * per_cu) per_cu = kWaves * 3 / 4 / W;
    const size_t lds = W * (sizeof(Turn<NT>) + 2 * NT * 1024);
    const int64_t fit = (int64_t)(156 << 10) / (lds + 4 * kMaxExperts + 256);
    per_cu = per_cu < 1 ? 1 : per_cu < fit ? per_cu : fit;
    hipLaunchKernelGGL((int4_rows_kernel<G, UP>), dim3((unsigned)(tiles < cus * per_cu ? tiles : cus * per_cu)), dim3(64 * W),
                       lds, s, a, w.h32, w.h, w.hinv, w.y);
}

void launch_narrow(const Int4Ffn& a, const Int4Ws& w, hipStream_t s)
{
    const int64_t R = (int64_t)a.T * a.k;
    // a vector of eight a thread, where a workgroup is that long
    if (a.f <= 8 * 64)
        hipLaunchKernelGGL(int4_narrow_kernel<64>, dim3((unsigned)((R + 3) / 4)), dim3(256), 0, s, w.h32, R, a.f, (uint4*)w.h,
                           w.hsum, w.hinv);
    else if (a.f <= 8 * 256)
        hipLaunchKernelGGL(int4_narrow_kernel<256>, dim3((unsigned)R), dim3(256), 0, s, w.h32, R, a.f, (uint4*)w.h, w.hsum,
                           w.hinv);
    else
        hipLaunchKernelGGL(int4_narrow_kernel<1024>, dim3((unsigned)R), dim3(1024), 0, s, w.h32, R, a.f, (uint4*)w.h, w.hsum,
                           w.hinv);
}

template <int G>
void launch_tiles(const Int4Ffn& a, const Int4Ws& w, hipStream_t s)
{
    const int64_t R = (int64_t)a.T * a.k, mt = R / kTileRows + (R < a.E ? R : a.E);
    auto go = [&](auto UP_, const uint16_t* rows, const float* sums, float* result) {
        constexpr bool UP = decltype(UP_)::value;
        constexpr int COLS = (UP ? 16 : 32) * kTileWaves;
        const int64_t ntn = ((UP ? a.f : a.d) + COLS - 1) / COLS;
        hipLaunchKernelGGL((int4_tile_kernel<G, UP>), dim3((unsigned)((mt * ntn + 7) / 8 * 8)), dim3(64 * kTileWaves),
                           sizeof(XStage) + kTileWaves * sizeof(Turn<2>), s, a, rows, sums, w.hinv, result);
    };
    // x in the codes' order and its sums lie where y will, which is longer
    const int64_t n8 = (int64_t)a.T * (a.d / 8), blocks = (n8 + 255) / 256;
    uint16_t* xo = reinterpret_cast<uint16_t*>(w.y);
    float* xsum = reinterpret_cast<float*>(xo + (int64_t)a.T * a.d);
    hipLaunchKernelGGL(int4_order_kernel, dim3((unsigned)(blocks < kMaxBlocks ? blocks : kMaxBlocks)), dim3(256), 0, s,
                       (const uint4*)a.x, n8, (uint4*)xo, xsum);
    go(std::true_type{}, xo, xsum, w.h32);
    launch_narrow(a, w, s);
    go(std::false_type{}, w.h, w.hsum, w.y);
}

// Which kernels.  Times of a whole pass, us, in a graph; A: d 4096, f 1536, top-4 of 128; B: d 2048, f 1024, 8 experts;
// C: d 2048, f 1408, top-6 of 64; D: d 5120, f 2560, top-2 of 16.  (With h in bf16; in fp16 a pass takes 0 to 3 us more
// by slot, 2 to 5 in rows.)
// Slot by slot or rows together: a slot by itself reads its expert's matrices once more, which costs nothing while
// few slots share one, or the second reading is from a cache.
//   slots      A: 16  32  48  64      B, top-2: 8  12  16    B, top-4: 16  24      C: 30  48      D: 32
//   by slot       40  68  95 122             17  21  24              21  26         43  60        125
//   rows          49  76 100 118             22  23  23              23  24         51  63        103
// so up to 48 slots, and up to one and a half an expert.
// Tiles of 16 or of 64 rows: with 16, each tile reads its matrices anew, from the caches.
//   rows an expert   A: 16  24  32      B: 32  48  64
//   tiles of 16         389 484 656        39  46  54
//   tiles of 64         458 470 485        44  45  46
// so tiles of 64 from 32 rows an expert on.
constexpr int kTokenSlots = 48, kTileMinRows = 32;

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

unsigned grid_of(int64_t n8)
{
    const int64_t n = (n8 + 256 * kVec - 1) / (256 * kVec);
    return (unsigned)(n < kMaxBlocks ? n : kMaxBlocks);
}

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
    // past the last-level cache (256 MB) the elements are read once and pass it by
    const bool stream = rows * (int64_t)K * 2 > ((int64_t)256 << 20);
    return with_group(group, [&](auto g) {
        constexpr int G = decltype(g)::value;
        auto go = [&](auto z, auto st) {
            hipLaunchKernelGGL((quantize_int4_kernel<G, decltype(z)::value, decltype(st)::value>), dim3(grid_of(n8)), dim3(256),
                               0, s, (const vu4*)src, n8, (uint32_t*)codes, scales, zeros);
        };
        using Y = std::true_type;
        using N = std::false_type;
        if (zeros) stream ? go(Y{}, Y{}) : go(Y{}, N{});
        else stream ? go(N{}, Y{}) : go(N{}, N{});
    });
}

hipError_t launch_dequantize_int4(const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros, int64_t rows,
                                  int K, int group, uint16_t* dst, hipStream_t s)
{
    const int64_t n8 = rows * (K / 8);
    if (n8 == 0) return hipSuccess;
    const bool stream = rows * (int64_t)K * 2 > ((int64_t)256 << 20);
    return with_group(group, [&](auto g) {
        constexpr int G = decltype(g)::value;
        if (stream)
            hipLaunchKernelGGL((dequantize_int4_kernel<G, true>), dim3(grid_of(n8)), dim3(256), 0, s, (const uint32_t*)codes,
                               scales, zeros, n8, (vu4*)dst);
        else
            hipLaunchKernelGGL((dequantize_int4_kernel<G, false>), dim3(grid_of(n8)), dim3(256), 0, s,
                               (const uint32_t*)codes, scales, zeros, n8, (vu4*)dst);
    });
}

size_t int4_ws_bytes(int64_t n_rows, int d, int f)
{
    const size_t R = (size_t)n_rows;
    return up256(R * f * 4) + up256(R * f * 2) + up256(R * (f / 32) * 4) + up256(R * 4) + up256(R * d * 4) + 256;
}

hipError_t launch_int4_ffn(const Int4Ffn& a, hipStream_t s)
{
    if (a.T == 0) return hipSuccess;
    const int64_t R = (int64_t)a.T * a.k;
    uint8_t* at = reinterpret_cast<uint8_t*>(a.ws);
    auto take = [&](size_t bytes) {
        uint8_t* p = at;
        at += up256(bytes);
        return p;
    };
    Int4Ws w;
    w.h32 = reinterpret_cast<float*>(take((size_t)R * a.f * 4));
    w.h = reinterpret_cast<uint16_t*>(take((size_t)R * a.f * 2));
    w.hsum = reinterpret_cast<float*>(take((size_t)R * (a.f / 32) * 4));
    w.hinv = reinterpret_cast<float*>(take((size_t)R * 4));
    w.y = reinterpret_cast<float*>(take((size_t)R * a.d * 4));
    hipError_t e;
    if (R <= kTokenSlots && 2 * R <= 3 * a.E) {
        return with_group(a.group, [&](auto g) {
            constexpr int G = decltype(g)::value;
            hipLaunchKernelGGL((int4_gate_up_token_kernel<G>), dim3(a.f / 16, (unsigned)R), dim3(64 * kTokenWaves), 0, s, a, w.h,
                               w.h32);
            hipLaunchKernelGGL((int4_down_token_kernel<G>), dim3(a.d / 16, (unsigned)a.T), dim3(64 * kTokenWaves), 0, s, a, w.h,
                               w.h32);
        });
    }
    if (R >= (int64_t)kTileMinRows * a.E) {
        e = with_group(a.group, [&](auto g) { launch_tiles<decltype(g)::value>(a, w, s); });
    } else {
        e = with_group(a.group, [&](auto g) {
            launch_rows<decltype(g)::value, true>(a, w, s);
            launch_narrow(a, w, s);
            launch_rows<decltype(g)::value, false>(a, w, s);
        });
    }
    if (e != hipSuccess) return e;
    const int64_t n = (int64_t)a.T * (a.d / 8), blocks = (n + 255) / 256;
    e = with_k(a.k, [&](auto kc) {
        hipLaunchKernelGGL((int4_combine_kernel<decltype(kc)::value>), dim3((unsigned)(blocks < kMaxBlocks ? blocks : kMaxBlocks)),
                           dim3(256), 0, s, (const float4*)w.y, a.topk_idx, a.dst_row, a.topk_w, a.T, a.E, a.d / 8, (uint4*)a.out,
                           a.dev_err);
    });
    if (e != hipSuccess) return e;
    return hipGetLastError();
}

}  // namespace moe
