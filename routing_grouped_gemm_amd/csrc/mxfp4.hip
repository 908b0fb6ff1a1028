// MXFP4 quantiser, its inverse, and the MXFP4 dispatch.
//
// All three stream: bf16 in 16-byte vectors, consecutive lanes on consecutive
// vectors of a row, one 32-element block per quad of lanes, which share the
// block's maximum by lane permutations (one lane per block would read with
// a stride of 64 bytes).  A lane writes (reads) the 4 bytes of its 8 codes, so
// a wave's codes are 256 contiguous bytes.
#include <algorithm>

#include "mx4.h"

namespace moe {
namespace {

// A workgroup takes runs of 256 NV vectors of [rows, K] (nvec = rows * K / 8 in
// all, a multiple of 4), NV a thread, all of its loads in flight together;
// runs past the grid's end are taken in turn.  STREAM: non-temporal access, for
// sources past the 256 MB last-level cache.  Bound by the reads and writes:
// called again and again, [49152, 4096] quantises in 79 us (6.4 TB/s, with plain
// accesses 90) and decodes in 70 (7.2 TB/s; 92); one after the other 80 and 76
// (6.7 TB/s); with the caches full of other data 84 and 100.  [16384, 4096], which
// the last-level cache holds, takes 24 and 25.  One vector a thread took 85 and
// 95 us, eight 82 and 73.
constexpr int NV = 2;
constexpr int kMaxGrid = 1 << 20;
typedef __attribute__((ext_vector_type(4))) uint32_t vu4;

template <bool STREAM>
__global__ __launch_bounds__(256) void quant_rows4_kernel(const vu4* __restrict__ src, int64_t nvec,
                                                          uint32_t* __restrict__ codes, uint8_t* __restrict__ scales)
{
    for (int64_t i0 = (int64_t)blockIdx.x * (256 * NV) + threadIdx.x; i0 < nvec; i0 += (int64_t)gridDim.x * (256 * NV)) {
        vu4 x[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t i = i0 + 256 * j;
            if (i < nvec) x[j] = STREAM ? __builtin_nontemporal_load(src + i) : src[i];
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t i = i0 + 256 * j;
            if (i >= nvec) break;   // whole quads stay
            uint32_t c;
            const uint32_t s = mx4::quant8_quad(make_uint4(x[j][0], x[j][1], x[j][2], x[j][3]), c);
            if constexpr (STREAM) __builtin_nontemporal_store(c, codes + i);
            else codes[i] = c;
            if ((threadIdx.x & 3) == 0) scales[i >> 2] = (uint8_t)s;
        }
    }
}

template <bool STREAM>
__global__ __launch_bounds__(256) void dequant_rows4_kernel(const uint32_t* __restrict__ codes,
                                                            const uint8_t* __restrict__ scales, int64_t nvec,
                                                            vu4* __restrict__ dst)
{
    for (int64_t i0 = (int64_t)blockIdx.x * (256 * NV) + threadIdx.x; i0 < nvec; i0 += (int64_t)gridDim.x * (256 * NV)) {
        uint32_t c[NV], s[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t i = i0 + 256 * j;
            if (i >= nvec) break;
            c[j] = codes[i];
            s[j] = scales[i >> 2];
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t i = i0 + 256 * j;
            if (i >= nvec) break;
            const uint4 v = mx4::decode8(c[j], s[j]);
            const vu4 o = {v.x, v.y, v.z, v.w};
            if constexpr (STREAM) __builtin_nontemporal_store(o, dst + i);
            else dst[i] = o;
        }
    }
}

// MXFP4 dispatch: a token's row is quantised once and its codes go to the K
// destination rows.  K (= top-k) is a template parameter: the destinations are
// read first and the K stores go out back to back.  ROW (rows of at least 256
// vectors): one workgroup per token, thread v on vectors v, v + 256, ..., its
// destinations workgroup-uniform (scalar loads, once per token); otherwise
// thread i quantises vector (i % nvec) of token row (i / nvec).  Bound by the
// reads and writes: called again and again, 32768 tokens of 4096 to one row each
// 62 us (5.5 TB/s; 68 without ROW), 16384 of 2048 to eight 33 us (6.3 TB/s);
// without ROW 65536 of 1024 to one 31 us (5.5 TB/s), 32768 of 1024 to four 24 us,
// 262144 of 256 to two 38 us (5.5 TB/s).  Between products, which fill the caches
// with other data, the first takes 75 to 78 us.  The codes are stored for the
// product that reads them next: past the caches the dispatch is 50 us called
// again and again, but dispatch and product together go from 510 to 520.
template <int K, bool ROW>
__global__ __launch_bounds__(256) void permute_mx4_kernel(const uint4* __restrict__ x, int T, int nvec,
                                                          const int32_t* __restrict__ dst_row, int64_t n_rows,
                                                          uint32_t* __restrict__ codes, uint8_t* __restrict__ scales,
                                                          int32_t* __restrict__ dev_err)
{
    bool bad = false;
    auto token = [&](int64_t t, int v0) {
        int32_t dst[K];
#pragma unroll
        for (int j = 0; j < K; ++j) {
            dst[j] = dst_row[t * K + j];
            bad |= dst[j] >= n_rows;
        }
        for (int v = v0; v < nvec; v += ROW ? 256 : nvec) {   // whole quads stay
            uint32_t c;
            const uint32_t s = mx4::quant8_quad(x[t * nvec + v], c);
#pragma unroll
            for (int j = 0; j < K; ++j) {
                if (dst[j] < 0 || dst[j] >= n_rows) continue;
                codes[(int64_t)dst[j] * nvec + v] = c;
                if ((v & 3) == 0) scales[(int64_t)dst[j] * (nvec >> 2) + (v >> 2)] = (uint8_t)s;
            }
        }
    };
    if constexpr (ROW) {
        for (int64_t t = blockIdx.x; t < T; t += gridDim.x) token(t, threadIdx.x);
        bad &= threadIdx.x == 0;
    } else {
        const int64_t n = (int64_t)T * nvec;
        for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
            token(i / nvec, (int)(i % nvec));
    }
    if (bad && dev_err) atomicOr(dev_err, (int)MOE_ERR_ROW_RANGE);
}

template <int K>
hipError_t permute_mx4(const void* x, int T, int d, const int32_t* dst_row, int64_t n_rows, void* codes,
                       uint8_t* scales, int32_t* dev_err, hipStream_t s)
{
    const int nvec = d / 8;
    const int64_t nblk = nvec >= 256 ? (int64_t)T : ((int64_t)T * nvec + 255) / 256;
    const dim3 grid((unsigned)std::min<int64_t>(nblk, kMaxGrid));
    if (nvec >= 256)
        hipLaunchKernelGGL((permute_mx4_kernel<K, true>), grid, dim3(256), 0, s, (const uint4*)x, T, nvec, dst_row, n_rows,
                           (uint32_t*)codes, scales, dev_err);
    else
        hipLaunchKernelGGL((permute_mx4_kernel<K, false>), grid, dim3(256), 0, s, (const uint4*)x, T, nvec, dst_row, n_rows,
                           (uint32_t*)codes, scales, dev_err);
    return hipGetLastError();
}

constexpr int64_t kStreamVectors = (256 << 20) / 16;   // bf16 vectors of 256 MB

}  // namespace

hipError_t launch_quantize_rows4(const uint16_t* src, int64_t rows, int K, uint8_t* codes, uint8_t* scales,
                                 hipStream_t s)
{
    const int64_t n = rows * (K / 8);
    if (n == 0) return hipSuccess;
    const dim3 grid((unsigned)std::min<int64_t>((n + 256 * NV - 1) / (256 * NV), kMaxGrid));
    if (n >= kStreamVectors)
        hipLaunchKernelGGL(quant_rows4_kernel<true>, grid, dim3(256), 0, s, (const vu4*)src, n, (uint32_t*)codes, scales);
    else
        hipLaunchKernelGGL(quant_rows4_kernel<false>, grid, dim3(256), 0, s, (const vu4*)src, n, (uint32_t*)codes, scales);
    return hipGetLastError();
}

hipError_t launch_dequantize_rows4(const uint8_t* codes, const uint8_t* scales, int64_t rows, int K, uint16_t* dst,
                                   hipStream_t s)
{
    const int64_t n = rows * (K / 8);
    if (n == 0) return hipSuccess;
    const dim3 grid((unsigned)std::min<int64_t>((n + 256 * NV - 1) / (256 * NV), kMaxGrid));
    if (n >= kStreamVectors)
        hipLaunchKernelGGL(dequant_rows4_kernel<true>, grid, dim3(256), 0, s, (const uint32_t*)codes, scales, n, (vu4*)dst);
    else
        hipLaunchKernelGGL(dequant_rows4_kernel<false>, grid, dim3(256), 0, s, (const uint32_t*)codes, scales, n, (vu4*)dst);
    return hipGetLastError();
}

hipError_t launch_permute_mx4(const void* x, int T, int d, int k, const int32_t* dst_row, int64_t n_rows,
                              void* codes, uint8_t* scales, int32_t* dev_err, hipStream_t s)
{
    if (T == 0 || d == 0) return hipSuccess;
    switch (k) {
    case 1: return permute_mx4<1>(x, T, d, dst_row, n_rows, codes, scales, dev_err, s);
    case 2: return permute_mx4<2>(x, T, d, dst_row, n_rows, codes, scales, dev_err, s);
    case 3: return permute_mx4<3>(x, T, d, dst_row, n_rows, codes, scales, dev_err, s);
    case 4: return permute_mx4<4>(x, T, d, dst_row, n_rows, codes, scales, dev_err, s);
    case 5: return permute_mx4<5>(x, T, d, dst_row, n_rows, codes, scales, dev_err, s);
    case 6: return permute_mx4<6>(x, T, d, dst_row, n_rows, codes, scales, dev_err, s);
    case 7: return permute_mx4<7>(x, T, d, dst_row, n_rows, codes, scales, dev_err, s);
    default: return permute_mx4<8>(x, T, d, dst_row, n_rows, codes, scales, dev_err, s);
    }
}

}  // namespace moe
