// MXFP4 quantiser, its inverse, and the MXFP4 dispatch.
//
// All three stream: bf16 in 16-byte vectors, consecutive lanes on consecutive
// vectors of a row, one 32-element block per quad of lanes, which share the
// block's maximum by lane permutations (one lane per block would read with
// a stride of 64 bytes).  A lane writes (reads) the 4 bytes of its 8 codes, so
// a wave's codes are 256 contiguous bytes.
#include "mx4.h"

namespace moe {
namespace {

// thread i quantises vector i of [rows, K] (nvec = rows * K / 8)
__global__ __launch_bounds__(256) void quant_rows4_kernel(const uint4* __restrict__ src, int64_t nvec,
                                                          uint32_t* __restrict__ codes, uint8_t* __restrict__ scales)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= nvec) return;   // nvec is a multiple of 4: whole quads stay
    uint32_t c;
    const uint32_t s = mx4::quant8_quad(src[i], c);
    codes[i] = c;
    if ((threadIdx.x & 3) == 0) scales[i >> 2] = (uint8_t)s;
}

__global__ __launch_bounds__(256) void dequant_rows4_kernel(const uint32_t* __restrict__ codes,
                                                            const uint8_t* __restrict__ scales, int64_t nvec,
                                                            uint4* __restrict__ dst)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= nvec) return;
    dst[i] = mx4::decode8(codes[i], scales[i >> 2]);
}

// MXFP4 dispatch: thread i quantises vector (i % nvec) of token row (i / nvec)
// and writes its codes to the k destination rows
__global__ __launch_bounds__(256) void permute_mx4_kernel(const uint4* __restrict__ x, int T, int nvec, int k,
                                                          const int32_t* __restrict__ dst_row, int64_t n_rows,
                                                          uint32_t* __restrict__ codes, uint8_t* __restrict__ scales,
                                                          int32_t* __restrict__ dev_err)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= (int64_t)T * nvec) return;
    const int64_t t = i / nvec;
    const int v = (int)(i - t * nvec);
    uint32_t c;
    const uint32_t s = mx4::quant8_quad(x[i], c);
    bool bad = false;
    for (int j = 0; j < k; ++j) {
        const int64_t dst = dst_row[t * k + j];
        bad |= dst >= n_rows;
        if (dst < 0 || dst >= n_rows) continue;
        codes[dst * nvec + v] = c;
        if ((v & 3) == 0) scales[dst * (nvec >> 2) + (v >> 2)] = (uint8_t)s;
    }
    if (bad && dev_err) atomicOr(dev_err, (int)MOE_ERR_ROW_RANGE);
}

inline unsigned grid_for(int64_t n) { return (unsigned)((n + 255) / 256); }

}  // namespace

hipError_t launch_quantize_rows4(const uint16_t* src, int64_t rows, int K, uint8_t* codes, uint8_t* scales,
                                 hipStream_t s)
{
    const int64_t n = rows * (K / 8);
    if (n == 0) return hipSuccess;
    hipLaunchKernelGGL(quant_rows4_kernel, dim3(grid_for(n)), dim3(256), 0, s, (const uint4*)src, n,
                       (uint32_t*)codes, scales);
    return hipGetLastError();
}

hipError_t launch_dequantize_rows4(const uint8_t* codes, const uint8_t* scales, int64_t rows, int K, uint16_t* dst,
                                   hipStream_t s)
{
    const int64_t n = rows * (K / 8);
    if (n == 0) return hipSuccess;
    hipLaunchKernelGGL(dequant_rows4_kernel, dim3(grid_for(n)), dim3(256), 0, s, (const uint32_t*)codes, scales,
                       n, (uint4*)dst);
    return hipGetLastError();
}

hipError_t launch_permute_mx4(const void* x, int T, int d, int k, const int32_t* dst_row, int64_t n_rows,
                              void* codes, uint8_t* scales, int32_t* dev_err, hipStream_t s)
{
    const int64_t n = (int64_t)T * (d / 8);
    if (n == 0) return hipSuccess;
    hipLaunchKernelGGL(permute_mx4_kernel, dim3(grid_for(n)), dim3(256), 0, s, (const uint4*)x, T, d / 8, k,
                       dst_row, n_rows, (uint32_t*)codes, scales, dev_err);
    return hipGetLastError();
}

}  // namespace moe
