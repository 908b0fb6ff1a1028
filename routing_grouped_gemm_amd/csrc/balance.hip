// The router's balance loss and z loss over packed sequences, with the
// per-expert counts, and their gradient to the router logits.
//
// With p_t = softmax(logits[t]) over all E experts and, for sequence s of n_s
// counted tokens, f_se its share of the routed pairs and P_se the mean of p_te:
//   balance = c_b * E * sum_s (n_s / N) sum_e f_se P_se
//   z       = c_z / N * sum_t lse_t^2,   lse_t = log sum_e exp(logits[t, e])
//   dlogits = p_te * (g_b c_b E / N (f_se - sum_j f_sj p_tj) + g_z 2 c_z / N lse_t)
// (the counts are piecewise constant).  Forward, two kernels:
//   1. balance_tokens_kernel: a workgroup takes a run of TB tokens; LPT lanes
//      hold one token's logits, so its softmax is a few lane exchanges, and
//      every lane keeps the running sums of p of its experts in registers.
//      A run is cut where a sequence ends; the piece of run b in sequence s
//      leaves its sums in row b + s of the workspace (run and sequence never
//      decrease from piece to piece and one of them grows, so rows are distinct).
//   2. balance_reduce_kernel: per sequence, the sums of its pieces' rows in a
//      fixed order; the last workgroup to finish adds up the losses.
// Backward, one kernel: the softmax again from the logits (p from a rounded lse
// would lose |lse| * 2^-24 of relative accuracy).  No floating-point atomics:
// results are the same bits on every run.
#include <type_traits>

#include "moe_internal.h"

namespace moe {
namespace {

constexpr int NT = 512;

struct Tokens {
    const float* logits;
    const uint8_t* mask;       // [T], 0 = not counted; may be null
    const int32_t* seg_off;    // [S + 1]; null: one sequence of all T tokens
    int T, E, S, TB;
};

__device__ __forceinline__ int seg_at(const Tokens& a, int i)
{
    const int v = a.seg_off ? a.seg_off[i] : (i ? a.T : 0);
    return min(max(v, 0), a.T);
}

// Calls f(s, begin, end) for the pieces of [t0, t1) in order; s < 0 for tokens
// outside every sequence.  Every piece holds a token whatever seg_off holds.
template <class F>
__device__ __forceinline__ void for_pieces(const Tokens& a, int t0, int t1, F&& f)
{
    int lo = 0, hi = a.S;   // first sequence that ends past t0
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (seg_at(a, mid + 1) > t0) hi = mid;
        else lo = mid + 1;
    }
    int s = lo;
    const int first = seg_at(a, 0);
    for (int cur = t0; cur < t1;) {
        if (cur < first) {
            const int end = min(t1, first);
            f(-1, cur, end);
            cur = end;
            continue;
        }
        while (s < a.S && seg_at(a, s + 1) <= cur) ++s;
        const int end = s < a.S ? min(t1, seg_at(a, s + 1)) : t1;
        f(s < a.S ? s : -1, cur, end);
        cur = end;
    }
}

// op over aligned segments of L lanes, every lane ending with the result:
// within 16 lanes by DPP (quad swaps, mirrored half-rows and rows)
template <int L, class F>
__device__ __forceinline__ float segment_op(float x, F&& op)
{
    auto dpp = [](float v, auto CTRL) __attribute__((always_inline)) {
        return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), decltype(CTRL)::value, 0xF, 0xF, false));
    };
    if constexpr (L >= 2) x = op(x, dpp(x, std::integral_constant<int, 0xB1>{}));
    if constexpr (L >= 4) x = op(x, dpp(x, std::integral_constant<int, 0x4E>{}));
    if constexpr (L >= 8) x = op(x, dpp(x, std::integral_constant<int, 0x141>{}));
    if constexpr (L >= 16) x = op(x, dpp(x, std::integral_constant<int, 0x140>{}));
#pragma unroll
    for (int off = 16; off < L; off <<= 1) x = op(x, __shfl_xor(x, off, 64));
    return x;
}
template <int L>
__device__ __forceinline__ float segment_sum(float x)
{
    return segment_op<L>(x, [](float a, float b) __attribute__((always_inline)) { return a + b; });
}
template <int L>
__device__ __forceinline__ float segment_max(float x)
{
    return segment_op<L>(x, [](float a, float b) __attribute__((always_inline)) { return fmaxf(a, b); });
}

// Lane l of a token's LPT holds NCH chunks of 4 experts, chunk q at expert
// 4 * (q * LPT + l): consecutive lanes on consecutive 16 bytes of the row.
// VEC: E is a multiple of 4 and rows are 16-byte aligned.
template <int LPT, int NCH, bool VEC>
struct Row {
    float v[4 * NCH];
    __device__ __forceinline__ static int col(int l, int i) { return 4 * ((i >> 2) * LPT + l) + (i & 3); }
    __device__ __forceinline__ void load(const float* row, int E, int l, float pad)
    {
#pragma unroll
        for (int q = 0; q < NCH; ++q) {
            const int c = col(l, 4 * q);
            if constexpr (VEC) {
                const float4 x = c < E ? *reinterpret_cast<const float4*>(row + c) : make_float4(pad, pad, pad, pad);
                v[4 * q] = x.x;
                v[4 * q + 1] = x.y;
                v[4 * q + 2] = x.z;
                v[4 * q + 3] = x.w;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) v[4 * q + i] = c + i < E ? row[c + i] : pad;
            }
        }
    }
    __device__ __forceinline__ void store(float* row, int E, int l) const
    {
#pragma unroll
        for (int q = 0; q < NCH; ++q) {
            const int c = col(l, 4 * q);
            if constexpr (VEC) {
                if (c < E) *reinterpret_cast<float4*>(row + c) = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (c + i < E) row[c + i] = v[4 * q + i];
            }
        }
    }
    // Softmax in place over the segment; returns the log of the sum of exps.
    // A logit that is not finite counts as -infinity (as in the route; bad is
    // set); a row with no finite logit has p = 0 and lse = 0.
    __device__ __forceinline__ float softmax(int E, int l, bool& bad)
    {
        // x * 0 is NaN for an x that is not finite: one operation per logit
        // tells whether any needs to be replaced
        float odd = 0.0f, top = -INFINITY;
#pragma unroll
        for (int i = 0; i < 4 * NCH; ++i) {
            odd = fmaf(v[i], 0.0f, odd);
            top = fmaxf(top, v[i]);
        }
        bool none = false;
        if (__builtin_expect(__any(odd != 0.0f), 0)) {   // (also where a lane's chunk lies past E)
            top = -INFINITY;
#pragma unroll
            for (int i = 0; i < 4 * NCH; ++i) {
                const bool fin = fabsf(v[i]) <= 3.402823466e38f;
                bad |= !fin && col(l, i) < E;
                v[i] = fin ? v[i] : -INFINITY;
                top = fmaxf(top, v[i]);
            }
            top = segment_max<LPT>(top);
            none = top == -INFINITY;
            top = none ? 0.0f : top;                     // exp(-infinity - 0) = 0
        } else {
            top = segment_max<LPT>(top);
        }
        float den = 0.0f;
#pragma unroll
        for (int i = 0; i < 4 * NCH; ++i) {
            v[i] = __expf(v[i] - top);
            den += v[i];
        }
        den = segment_sum<LPT>(den);
        const float r = none ? 0.0f : __builtin_amdgcn_rcpf(den);   // (one unit in the last place)
#pragma unroll
        for (int i = 0; i < 4 * NCH; ++i) v[i] *= r;
        return none ? 0.0f : top + __logf(den);
    }
};

// workspace: the ticket (first 256 bytes), then per piece a row of floats (the
// sums of p, then the sum of lse^2) and a row of counts (pairs per expert,
// then tokens)
constexpr size_t kTicketBytes = 256;
__host__ __device__ inline int row_stride(int E) { return (E + 4) & ~3; }

template <int LPT, int NCH, bool VEC>
__global__ __launch_bounds__(NT) void balance_tokens_kernel(Tokens a, const int32_t* __restrict__ topk_idx, int k,
                                                            uint32_t over_k,   // ceil(2^32 / k), k > 1
                                                            float* __restrict__ lse_out, float* __restrict__ fpart,
                                                            int32_t* __restrict__ ipart, int* __restrict__ ticket,
                                                            int32_t* __restrict__ dev_err)
{
    constexpr int NG = NT / LPT, GW = 64 / LPT;   // lane groups per workgroup, per wave
    constexpr int U = NCH == 1 ? 4 : 2;           // tokens in flight per group
    __shared__ float s_p[NT / 64][kMaxExperts];
    __shared__ float s_z[NT / 64];
    __shared__ int s_n[NT / 64];
    __shared__ int s_cnt[kMaxExperts];
    const int tid = threadIdx.x, l = tid % LPT, grp = tid / LPT, wave = tid >> 6;
    const int E = a.E, stride = row_stride(E);
    if (blockIdx.x == 0 && tid == 0) *ticket = 0;
    const int t0 = blockIdx.x * a.TB, t1 = min(t0 + a.TB, a.T);
    bool bad = false;
    for_pieces(a, t0, t1, [&](int s, int begin, int end) {
        if (s < 0) {
            if (lse_out)
                for (int t = begin + tid; t < end; t += NT) lse_out[t] = 0.0f;
            return;
        }
        for (int e = tid; e < E; e += NT) s_cnt[e] = 0;
        // The piece's routed pairs, PQ per thread and pass; the first pass is
        // loaded ahead of the logits.  A pair's token is its number within the
        // piece over k, by multiplication (numbers below 2^24: exact).
        constexpr int PQ = 4;
        const int32_t* idx = topk_idx + (int64_t)begin * k;
        const int pairs = (end - begin) * k;
        auto load_pairs = [&](int i0, int (&e)[PQ]) __attribute__((always_inline)) {
#pragma unroll
            for (int q = 0; q < PQ; ++q) {
                const int i = i0 + q * NT;
                e[q] = i < pairs ? idx[i] : -1;
                if (a.mask && i < pairs && !a.mask[begin + (k == 1 ? i : (int)__umulhi((uint32_t)i, over_k))]) e[q] = -1;
            }
        };
        int ev[PQ];
        load_pairs(tid, ev);
        int n = 0;
        float sum[4 * NCH], z = 0.0f;
#pragma unroll
        for (int i = 0; i < 4 * NCH; ++i) sum[i] = 0.0f;
        for (int t = begin + grp; t < end; t += NG * U) {
            Row<LPT, NCH, VEC> r[U];
            bool on[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int tt = t + u * NG;
                on[u] = tt < end && (!a.mask || a.mask[tt]);
                r[u].load(a.logits + (int64_t)(tt < end ? tt : begin) * E, E, l, -INFINITY);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int tt = t + u * NG;
                bool b = false;
                const float lse = r[u].softmax(E, l, b);
                bad |= b && on[u];
                if (on[u]) {
                    ++n;
#pragma unroll
                    for (int i = 0; i < 4 * NCH; ++i) sum[i] += r[u].v[i];
                    z = fmaf(lse, lse, z);
                }
                if (lse_out && l == 0 && tt < end) lse_out[tt] = on[u] ? lse : 0.0f;
            }
        }
        // the wave's groups, then the waves, each in a fixed order
#pragma unroll
        for (int off = LPT; off < 64; off <<= 1) {
#pragma unroll
            for (int i = 0; i < 4 * NCH; ++i) sum[i] += __shfl_xor(sum[i], off, 64);
            z += __shfl_xor(z, off, 64);
            n += __shfl_xor(n, off, 64);
        }
        if (grp % GW == 0) {
#pragma unroll
            for (int i = 0; i < 4 * NCH; ++i)
                if (Row<LPT, NCH, VEC>::col(l, i) < E) s_p[wave][Row<LPT, NCH, VEC>::col(l, i)] = sum[i];
            if (l == 0) {
                s_z[wave] = z;
                s_n[wave] = n;
            }
        }
        __syncthreads();   // s_cnt is clear, too
        for (int i0 = tid; i0 < pairs; i0 += NT * PQ) {
            if (i0 != tid) load_pairs(i0, ev);
#pragma unroll
            for (int q = 0; q < PQ; ++q)
                if (ev[q] >= 0 && ev[q] < E) atomicAdd(&s_cnt[ev[q]], 1);   // integer: the order does not matter
        }
        __syncthreads();
        float* fo = fpart + (int64_t)(blockIdx.x + s) * stride;
        int32_t* io = ipart + (int64_t)(blockIdx.x + s) * stride;
        for (int e = tid; e <= E; e += NT) {
            float v = e < E ? s_p[0][e] : s_z[0];
            int c = e < E ? s_cnt[e] : s_n[0];
#pragma unroll
            for (int w = 1; w < NT / 64; ++w) {
                v += e < E ? s_p[w][e] : s_z[w];
                c += e < E ? 0 : s_n[w];
            }
            fo[e] = v;
            io[e] = c;
        }
        __syncthreads();   // the next piece clears the counts
    });
    if (bad && dev_err) atomicOr(dev_err, (int)MOE_ERR_NONFINITE_LOGIT);
}

// One workgroup per sequence: the sums of its pieces' rows, R rows at a time
// (a thread takes 4 columns of every R-th row), then R to 1 through LDS.  With
// one sequence it also makes the losses; else the last workgroup to finish does.
constexpr int RT = 1024;

__global__ __launch_bounds__(RT) void balance_reduce_kernel(Tokens a, float cb, float cz,
                                                            const float4* __restrict__ fpart,
                                                            const int4* __restrict__ ipart,
                                                            int* __restrict__ ticket, float* __restrict__ partial,
                                                            float* __restrict__ losses, int32_t* __restrict__ counts,
                                                            float* __restrict__ probs, int32_t* __restrict__ tokens)
{
    __shared__ float4 s_f[RT];
    __shared__ int4 s_i[RT];
    __shared__ double s_b[RT / 64], s_zz[RT / 64];
    __shared__ int s_n[RT / 64];
    __shared__ int s_last;
    const int s = blockIdx.x, tid = threadIdx.x;
    const int E = a.E, nv = row_stride(E) / 4;
    const int begin = seg_at(a, s), end = seg_at(a, s + 1);
    const int b0 = begin / a.TB, b1 = end > begin ? (end - 1) / a.TB + 1 : b0;
    int R = 1;   // a power of two, for the steps below
    while (2 * R * nv <= RT && R < b1 - b0) R *= 2;
    const int c = tid % nv, r = tid / nv;
    float4 fv = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    int4 iv = make_int4(0, 0, 0, 0);
    if (r < R) {
#pragma unroll 4
        for (int b = b0 + r; b < b1; b += R) {
            const int64_t at = (int64_t)(b + s) * nv + c;
            const float4 f = fpart[at];
            const int4 i = ipart[at];
            fv.x += f.x;
            fv.y += f.y;
            fv.z += f.z;
            fv.w += f.w;
            iv.x += i.x;
            iv.y += i.y;
            iv.z += i.z;
            iv.w += i.w;
        }
        s_f[tid] = fv;
        s_i[tid] = iv;
    }
    __syncthreads();
    for (int h = R / 2; h >= 1; h /= 2) {
        if (r < h) {
            const float4 f = s_f[tid + h * nv];
            const int4 i = s_i[tid + h * nv];
            fv.x += f.x;
            fv.y += f.y;
            fv.z += f.z;
            fv.w += f.w;
            iv.x += i.x;
            iv.y += i.y;
            iv.z += i.z;
            iv.w += i.w;
            s_f[tid] = fv;
            s_i[tid] = iv;
        }
        __syncthreads();
    }
    // row 0: the sums of p and the pairs per expert, then sum lse^2; tokens and pairs
    const float* sum = reinterpret_cast<const float*>(s_f);
    const int* cnt = reinterpret_cast<const int*>(s_i);
    const int n = cnt[E];
    const float rn = n ? 1.0f / (float)n : 0.0f;
    double vb = 0.0;
    int m = 0;
    for (int e = tid; e < E; e += RT) {
        counts[(int64_t)s * E + e] = cnt[e];
        probs[(int64_t)s * E + e] = sum[e] * rn;
        vb += (double)cnt[e] * sum[e];                        // m n_s f_se P_se, m the pairs
        m += cnt[e];
    }
    // sums over the workgroup, in a fixed order
    auto block_sum = [&](double& b, double& z, int& k) __attribute__((always_inline)) {
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) {
            b += __shfl_xor(b, off, 64);
            z += __shfl_xor(z, off, 64);
            k += __shfl_xor(k, off, 64);
        }
        if ((tid & 63) == 0) {
            s_b[tid >> 6] = b;
            s_zz[tid >> 6] = z;
            s_n[tid >> 6] = k;
        }
        __syncthreads();
        b = z = 0.0;
        k = 0;
        for (int w = 0; w < RT / 64; ++w) {
            b += s_b[w];
            z += s_zz[w];
            k += s_n[w];
        }
        __syncthreads();
    };
    double vz = tid == 0 ? (double)sum[E] : 0.0;
    int vn = n;
    block_sum(vb, vz, m);
    vb = m ? vb / m : 0.0;
    if (a.S > 1) {
        if (tid == 0) {
            partial[2 * s] = (float)vb;
            partial[2 * s + 1] = (float)vz;
            tokens[s] = n;
            __threadfence();
            s_last = atomicAdd(ticket, 1) == a.S - 1;
        }
        __syncthreads();
        if (!s_last) return;
        __threadfence();
        vb = vz = 0.0;
        vn = 0;
        // (each sequence's sums were rounded to 32 bits once)
        for (int i = tid; i < a.S; i += RT) {
            vb += __hip_atomic_load(partial + 2 * i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            vz += __hip_atomic_load(partial + 2 * i + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            vn += __hip_atomic_load(tokens + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        block_sum(vb, vz, vn);
    } else if (tid == 0) {
        tokens[0] = n;
    }
    if (tid == 0) {
        const double inv = vn ? 1.0 / vn : 0.0;
        losses[0] = (float)((double)cb * E * inv * vb);
        // (a row of the type's lowest value has an lse^2 past fp32: no 0 * infinity)
        losses[1] = cz == 0.0f ? 0.0f : (float)((double)cz * inv * vz);
        tokens[a.S] = vn;
    }
}

template <int LPT, int NCH, bool VEC>
__global__ __launch_bounds__(NT) void balance_bwd_kernel(Tokens a, const int32_t* __restrict__ counts,
                                                         const int32_t* __restrict__ tokens, float cb, float cz,
                                                         const float* __restrict__ dlosses, const float* add,
                                                         float* dlogits)
{
    constexpr int NG = NT / LPT;
    constexpr int U = NCH == 1 ? 4 : 2;
    using R = Row<LPT, NCH, VEC>;
    const int tid = threadIdx.x, l = tid % LPT, grp = tid / LPT;
    const int E = a.E;
    const int t0 = blockIdx.x * a.TB, t1 = min(t0 + a.TB, a.T);
    const int N = tokens[a.S];
    const float inv = N > 0 ? 1.0f / (float)N : 0.0f;
    const float kb = (dlosses ? dlosses[0] : 1.0f) * cb * (float)E * inv;
    const float kz = (dlosses ? dlosses[1] : 1.0f) * cz * 2.0f * inv;
    for_pieces(a, t0, t1, [&](int s, int begin, int end) {
        float f[4 * NCH], m = 0.0f;
#pragma unroll
        for (int i = 0; i < 4 * NCH; ++i) {
            f[i] = s >= 0 && R::col(l, i) < E ? (float)counts[(int64_t)s * E + R::col(l, i)] : 0.0f;
            m += f[i];
        }
        m = segment_sum<LPT>(m);
#pragma unroll
        for (int i = 0; i < 4 * NCH; ++i) f[i] = m > 0.0f ? f[i] / m : 0.0f;
        for (int t = begin + grp; t < end; t += NG * U) {
            R x[U], o[U];
            bool on[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int tt = t + u * NG < end ? t + u * NG : begin;
                on[u] = s >= 0 && (!a.mask || a.mask[tt]);
                x[u].load(a.logits + (int64_t)tt * E, E, l, -INFINITY);
                if (add && t + u * NG < end) o[u].load(add + (int64_t)tt * E, E, l, 0.0f);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                bool bad = false;
                const float lse = x[u].softmax(E, l, bad);
                float dot = 0.0f;
#pragma unroll
                for (int i = 0; i < 4 * NCH; ++i) dot = fmaf(f[i], x[u].v[i], dot);
                dot = segment_sum<LPT>(dot);
                const float c0 = fmaf(kz, lse, -kb * dot);
#pragma unroll
                for (int i = 0; i < 4 * NCH; ++i) {
                    const float gr = on[u] ? x[u].v[i] * fmaf(kb, f[i], c0) : 0.0f;
                    o[u].v[i] = add ? o[u].v[i] + gr : gr;
                }
                if (t + u * NG < end) o[u].store(dlogits + (int64_t)(t + u * NG) * E, E, l);
            }
        }
    });
}

// tokens per workgroup: 64, or as many as leave 1024 workgroups
int tokens_per_block(int T)
{
    const int64_t tb = ((int64_t)T + 1023) / 1024;
    return (int)((tb + 63) / 64 * 64 > 64 ? (tb + 63) / 64 * 64 : 64);
}

template <class F>
void with_shape(int E, bool vec, F&& f)
{
    auto go = [&](auto L, auto N) {
        if (vec) f(L, N, std::true_type{});
        else f(L, N, std::false_type{});
    };
    using std::integral_constant;
    if (E <= 4) go(integral_constant<int, 1>{}, integral_constant<int, 1>{});
    else if (E <= 8) go(integral_constant<int, 2>{}, integral_constant<int, 1>{});
    else if (E <= 16) go(integral_constant<int, 4>{}, integral_constant<int, 1>{});
    else if (E <= 32) go(integral_constant<int, 8>{}, integral_constant<int, 1>{});
    else if (E <= 64) go(integral_constant<int, 16>{}, integral_constant<int, 1>{});
    else if (E <= 128) go(integral_constant<int, 16>{}, integral_constant<int, 2>{});
    else if (E <= 256) go(integral_constant<int, 16>{}, integral_constant<int, 4>{});
    else if (E <= 512) go(integral_constant<int, 32>{}, integral_constant<int, 4>{});
    else go(integral_constant<int, 64>{}, integral_constant<int, 4>{});
}

inline int64_t piece_rows(int T, int S) { return ((int64_t)T + tokens_per_block(T) - 1) / tokens_per_block(T) + S; }

inline bool vec_ok(int E, const void* p) { return E % 4 == 0 && (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

size_t balance_ws_bytes(int T, int E, int S)
{
    return kTicketBytes + ((size_t)S * 2 * 4 + 255) / 256 * 256 + (size_t)piece_rows(T, S) * row_stride(E) * 8;
}

hipError_t launch_balance(const float* logits, const int32_t* topk_idx, const uint8_t* mask, const int32_t* seg_off,
                          int S, int T, int E, int k, float cb, float cz, float* losses, int32_t* counts,
                          float* probs, float* lse, int32_t* tokens, void* ws, int32_t* dev_err, hipStream_t s)
{
    const Tokens a{logits, mask, seg_off, T, E, S, tokens_per_block(T)};
    uint8_t* w = static_cast<uint8_t*>(ws);
    int* ticket = reinterpret_cast<int*>(w);
    float* partial = reinterpret_cast<float*>(w + kTicketBytes);
    float* fpart = reinterpret_cast<float*>(w + kTicketBytes + ((size_t)S * 2 * 4 + 255) / 256 * 256);
    int32_t* ipart = reinterpret_cast<int32_t*>(fpart + piece_rows(T, S) * row_stride(E));
    const int nblk = T > 0 ? (T + a.TB - 1) / a.TB : 1;
    with_shape(E, vec_ok(E, logits), [&](auto L, auto N, auto V) {
        hipLaunchKernelGGL((balance_tokens_kernel<decltype(L)::value, decltype(N)::value, decltype(V)::value>),
                           dim3((unsigned)nblk), dim3(NT), 0, s, a, topk_idx, k,
                           (uint32_t)(((1ull << 32) + k - 1) / k), lse, fpart, ipart, ticket, dev_err);
    });
    hipLaunchKernelGGL(balance_reduce_kernel, dim3((unsigned)S), dim3(RT), 0, s, a, cb, cz,
                       reinterpret_cast<const float4*>(fpart), reinterpret_cast<const int4*>(ipart), ticket, partial, losses, counts, probs, tokens);
    return hipGetLastError();
}

hipError_t launch_balance_bwd(const float* logits, const uint8_t* mask, const int32_t* seg_off, int S, int T, int E,
                              const int32_t* counts, const int32_t* tokens, float cb, float cz, const float* dlosses,
                              const float* add, float* dlogits, hipStream_t s)
{
    if (T == 0) return hipSuccess;
    const Tokens a{logits, mask, seg_off, T, E, S, tokens_per_block(T)};
    const int nblk = (T + a.TB - 1) / a.TB;
    const bool vec = vec_ok(E, logits) && vec_ok(E, dlogits) && vec_ok(E, add);
    with_shape(E, vec, [&](auto L, auto N, auto V) {
        hipLaunchKernelGGL((balance_bwd_kernel<decltype(L)::value, decltype(N)::value, decltype(V)::value>),
                           dim3((unsigned)nblk), dim3(NT), 0, s, a, counts, tokens, cb, cz, dlosses, add, dlogits);
    });
    return hipGetLastError();
}

}  // namespace moe
