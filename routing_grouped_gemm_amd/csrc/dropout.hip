// Dropout without a stored mask (moe_dropout), and the combine with dropout
// and a residual in its epilogue (moe_combine_dropout).
//
// Both are bound by HBM: every element is read and written once, and the mask
// comes from an eighth of a generator call (philox.h).  A thread makes eight
// consecutive elements, one generator block, from whole 16-byte vectors.
#include <algorithm>
#include <type_traits>

#include "philox.h"

namespace moe {
namespace {

typedef __attribute__((ext_vector_type(4))) uint32_t vu4;

constexpr int64_t kMaxBlocks = 1 << 20;   // workgroups of a launch; longer tensors are walked

__device__ __forceinline__ void unpack8(vu4 v, float (&o)[8])
{
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        o[2 * p] = bf16_lo(v[p]);
        o[2 * p + 1] = bf16_hi(v[p]);
    }
}

__device__ __forceinline__ vu4 pack8(const float (&o)[8])
{
    return vu4{pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]), pack_bf16x2(o[4], o[5]), pack_bf16x2(o[6], o[7])};
}

// element j of a generator block
__device__ __forceinline__ bool kept(uint4 r, int j, uint32_t thr)
{
    const uint32_t w = j < 2 ? r.x : j < 4 ? r.y : j < 6 ? r.z : r.w;
    return (j & 1) ? keep_hi(w, thr) : keep_lo(w, thr);
}

// thread i makes elements 8i .. 8i + 7 of the flat tensor (fp32: two vectors,
// the second absent where n ends on an odd one)
template <bool BF16, bool RES, bool DROP>
__global__ __launch_bounds__(256) void dropout_kernel(const vu4* x, const vu4* residual, int64_t n, uint32_t thr,
                                                      float scale, const uint64_t* rng, vu4* out)
{
    PhiloxKey key{};
    if constexpr (DROP) key = philox_key(rng);
    const int64_t nblk = (n + 7) / 8;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < nblk; i += (int64_t)gridDim.x * 256) {
        float v[8], r[8];
        bool two = true;
        if constexpr (BF16) {
            unpack8(x[i], v);
            if constexpr (RES) unpack8(residual[i], r);
        } else {
            two = 8 * i + 4 < n;
            const vu4 a = x[2 * i], b = two ? x[2 * i + 1] : vu4{0, 0, 0, 0};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                v[q] = __uint_as_float(a[q]);
                v[4 + q] = __uint_as_float(b[q]);
            }
            if constexpr (RES) {
                const vu4 c = residual[2 * i], e = two ? residual[2 * i + 1] : vu4{0, 0, 0, 0};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    r[q] = __uint_as_float(c[q]);
                    r[4 + q] = __uint_as_float(e[q]);
                }
            }
        }
        uint4 w = make_uint4(0, 0, 0, 0);
        if constexpr (DROP) w = philox(key, (uint64_t)i);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if constexpr (DROP) v[j] = kept(w, j, thr) ? v[j] * scale : 0.0f;
            if constexpr (RES) v[j] += r[j];
        }
        if constexpr (BF16) {
            out[i] = pack8(v);
        } else {
            vu4 a, b;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                a[q] = __float_as_uint(v[q]);
                b[q] = __float_as_uint(v[4 + q]);
            }
            out[2 * i] = a;
            if (two) out[2 * i + 1] = b;
        }
    }
}

// thread i makes vector (i % nvec) of token (i / nvec), as the plain combine
// does: the K row loads in flight together, the sum in slot order, all streams
// non-temporal (16384 tokens of 4 x 4096: 138 -> 131 us, 6.1 TB/s)
template <bool BF16, int K>
__global__ __launch_bounds__(256) void combine_dropout_kernel(const vu4* __restrict__ y,
                                                              const int32_t* __restrict__ dst_row,
                                                              const float* __restrict__ wt, const vu4* residual,
                                                              int T, int nvec, int64_t n_rows, uint32_t thr,
                                                              float scale, const uint64_t* rng, vu4* out,
                                                              int32_t* dev_err)
{
    constexpr int NE = BF16 ? 8 : 4;
    PhiloxKey key{};
    if (thr) key = philox_key(rng);
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < (int64_t)T * nvec; i += (int64_t)gridDim.x * 256) {
        const int64_t t = i / nvec;
        const int v = (int)(i - t * nvec);
        vu4 val[K];
        float w[K];
        bool on[K], bad = false;
#pragma unroll
        for (int j = 0; j < K; ++j) {
            const int32_t dst = dst_row[t * K + j];
            w[j] = wt ? wt[t * K + j] : 1.0f;
            on[j] = dst >= 0 && dst < n_rows;
            bad |= dst >= n_rows;
            val[j] = on[j] ? __builtin_nontemporal_load(y + (int64_t)dst * nvec + v) : vu4{0, 0, 0, 0};
        }
        const vu4 res = residual ? __builtin_nontemporal_load(residual + i) : vu4{0, 0, 0, 0};
        float acc[NE];
#pragma unroll
        for (int q = 0; q < NE; ++q) acc[q] = 0.0f;
#pragma unroll
        for (int j = 0; j < K; ++j) {
            if (!on[j]) continue;
#pragma unroll
            for (int q = 0; q < NE; ++q) {
                const float e = BF16 ? ((q & 1) ? bf16_hi(val[j][q / 2]) : bf16_lo(val[j][q / 2]))
                                     : __uint_as_float(val[j][q & 3]);
                acc[q] = fmaf(w[j], e, acc[q]);
            }
        }
        if (thr) {
            // an fp32 vector is half a generator block, an odd vector its second half
            uint4 r = philox(key, (uint64_t)(BF16 ? i : i >> 1));
            if (!BF16 && (i & 1)) r = make_uint4(r.z, r.w, 0, 0);
#pragma unroll
            for (int q = 0; q < NE; ++q) acc[q] = kept(r, q, thr) ? acc[q] * scale : 0.0f;
        }
        if (residual) {
#pragma unroll
            for (int q = 0; q < NE; ++q)
                acc[q] += BF16 ? ((q & 1) ? bf16_hi(res[q / 2]) : bf16_lo(res[q / 2])) : __uint_as_float(res[q & 3]);
        }
        vu4 o;
        if constexpr (BF16) {
            o = vu4{pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]), pack_bf16x2(acc[4], acc[5]),
                    pack_bf16x2(acc[6], acc[7])};
        } else {
            o = vu4{__float_as_uint(acc[0]), __float_as_uint(acc[1]), __float_as_uint(acc[2]), __float_as_uint(acc[3])};
        }
        __builtin_nontemporal_store(o, out + i);
        if (bad && dev_err) atomicOr(dev_err, (int)MOE_ERR_ROW_RANGE);
    }
}

unsigned grid_of(int64_t n) { return (unsigned)std::min<int64_t>((n + 255) / 256, kMaxBlocks); }

}  // namespace

hipError_t launch_dropout(int dtype, const void* x, const void* residual, int64_t n, DropSpec dr, void* out,
                          hipStream_t s)
{
    if (n == 0) return hipSuccess;
    const dim3 grid(grid_of((n + 7) / 8)), blk(256);
    auto go = [&](auto BF_, auto RES_, auto DROP_) {
        hipLaunchKernelGGL((dropout_kernel<decltype(BF_)::value, decltype(RES_)::value, decltype(DROP_)::value>), grid,
                           blk, 0, s, (const vu4*)x, (const vu4*)residual, n, dr.thr, dr.scale, dr.rng, (vu4*)out);
    };
    using Y = std::true_type;
    using N = std::false_type;
    auto drop = [&](auto BF_, auto RES_) { dr.thr ? go(BF_, RES_, Y{}) : go(BF_, RES_, N{}); };
    auto res = [&](auto BF_) { residual ? drop(BF_, Y{}) : drop(BF_, N{}); };
    dtype == MOE_BF16 ? res(Y{}) : res(N{});
    return hipGetLastError();
}

hipError_t launch_combine_dropout(int dtype, const void* y_perm, const int32_t* dst_row, const float* w,
                                  const void* residual, int T, int k, int d, int64_t n_rows, DropSpec dr, void* out,
                                  int32_t* dev_err, hipStream_t s)
{
    const bool bf = dtype == MOE_BF16;
    const int nvec = bf ? d / 8 : d / 4;
    if ((int64_t)T * nvec == 0) return hipSuccess;
    const dim3 grid(grid_of((int64_t)T * nvec)), blk(256);
    const hipError_t e = with_k(k, [&](auto kc) {
        constexpr int K = decltype(kc)::value;
        if (bf)
            hipLaunchKernelGGL((combine_dropout_kernel<true, K>), grid, blk, 0, s, (const vu4*)y_perm, dst_row, w,
                               (const vu4*)residual, T, nvec, n_rows, dr.thr, dr.scale, dr.rng, (vu4*)out, dev_err);
        else
            hipLaunchKernelGGL((combine_dropout_kernel<false, K>), grid, blk, 0, s, (const vu4*)y_perm, dst_row, w,
                               (const vu4*)residual, T, nvec, n_rows, dr.thr, dr.scale, dr.rng, (vu4*)out, dev_err);
    });
    if (e != hipSuccess) return e;
    return hipGetLastError();
}

}  // namespace moe
