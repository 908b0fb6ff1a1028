// The router's balance loss and z loss over packed sequences, with the
// per-expert counts, and their gradient to the router logits.
//
// With p_t = softmax(logits[t]) over all E experts and, for sequence s of n_s
// counted tokens, f_se its share of the routed pairs and P_se the mean of p_te:
//   balance = c_b * E * sum_s (n_s / N) sum_e f_se P_se
//   z       = c_z / N * sum_t lse_t^2,   lse_t = log sum_e exp(logits[t, e])
//   dlogits = p_te * (g_b c_b E / N (f_se - sum_j f_sj p_tj) + g_z 2 c_z / N lse_t)
// (the counts are piecewise constant).  Forward, two kernels (few tokens: the
// first alone, in a single workgroup that finishes by itself; many sequences: a
// third for the losses):
//   1. balance_tokens_kernel: a workgroup takes a run of TB tokens; LPT lanes
//      hold one token's logits, so its softmax is a few lane exchanges, and
//      every lane keeps the running sums of p of its experts in registers.
//      A run is cut where a sequence ends; the piece of run b in sequence s
//      leaves its sums in row b + s of the workspace (run and sequence never
//      decrease from piece to piece and one of them grows, so rows are distinct).
//   2. balance_reduce_kernel: per sequence and group of experts, the sums of
//      its pieces' rows in a fixed order; the last workgroup to finish adds up
//      the losses (or balance_losses_kernel does).
// Backward, one kernel: the softmax again from the logits (p from a rounded lse
// would lose |lse| * 2^-24 of relative accuracy).  No floating-point atomics:
// results are the same bits on every run.
#include <algorithm>
#include <type_traits>

#include "moe_internal.h"

namespace moe {
namespace {

constexpr int NT = 512, NTB = 256;   // threads of the forward's and the backward's workgroups

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
// The first sequence that ends past t0 is searched by all 64 lanes at once, a
// round trip to memory per factor of 64 (halving took 5 for 23 sequences: 2 us
// of each kernel).
template <class F>
__device__ __forceinline__ void for_pieces(const Tokens& a, int t0, int t1, F&& f)
{
    const int first = seg_at(a, 0);
    int s = 0, end_s = a.T;   // the sequence, and its end
    if (a.seg_off) {
        const int lane = threadIdx.x & 63;
        int lo = 0, hi = a.S;
        for (;;) {
            const int step = (hi - lo + 63) >> 6;
            const int i = min(lo + lane * step + step - 1, hi - 1);
            const int v = seg_at(a, i + 1);
            const unsigned long long past = __ballot(v > t0);
            if (!past) {
                s = a.S;
                break;
            }
            const int l = __ffsll(past) - 1;
            s = __builtin_amdgcn_readlane(i, l);
            end_s = __builtin_amdgcn_readlane(v, l);
            if (step == 1) break;
            lo = s - min(step - 1, s - lo);
            hi = s + 1;
        }
    }
    for (int cur = t0; cur < t1;) {
        if (cur < first) {
            const int end = min(t1, first);
            f(-1, cur, end);
            cur = end;
            continue;
        }
        while (s < a.S && end_s <= cur)
            if (++s < a.S) end_s = seg_at(a, s + 1);
        const int end = s < a.S ? min(t1, end_s) : t1;
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
// STREAM: loads and stores that do not displace what the caches hold, for
// logits that do not fit there (the 256 MB last-level cache) between the
// forward and the backward anyway.  At 2^20 x 128: forward 113 -> 98 us,
// backward with an addend 317 -> 303 us; at 2^16 x 128 the backward goes 19.5
// -> 21.1 us with them.
typedef __attribute__((ext_vector_type(4))) float vf4;
template <int LPT, int NCH, bool VEC, bool STREAM>
struct Row {
    float v[4 * NCH];
    __device__ __forceinline__ static int col(int l, int i) { return 4 * ((i >> 2) * LPT + l) + (i & 3); }
    __device__ __forceinline__ void load(const float* row, int E, int l, float pad)
    {
#pragma unroll
        for (int q = 0; q < NCH; ++q) {
            const int c = col(l, 4 * q);
            if constexpr (VEC) {
                const vf4* at = reinterpret_cast<const vf4*>(row + c);
                vf4 x = {pad, pad, pad, pad};
                if (c < E) x = STREAM ? __builtin_nontemporal_load(at) : *at;
#pragma unroll
                for (int i = 0; i < 4; ++i) v[4 * q + i] = x[i];
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
                const vf4 x = {v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
                vf4* at = reinterpret_cast<vf4*>(row + c);
                if (c < E) {
                    if constexpr (STREAM) __builtin_nontemporal_store(x, at);
                    else *at = x;
                }
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

// workspace: the ticket (first 256 bytes), the reduction's partial losses, then
// per piece the sums of p and, apart, the pairs per expert, in vectors of 4
// experts with one more vector at the end: the sum of lse^2; the tokens and the
// pairs.  Vector v of all pieces is contiguous, so that the reduction reads
// whole lines.
constexpr size_t kTicketBytes = 256;
__host__ __device__ inline int last_vector(int E) { return (E + 3) / 4; }

struct Results {
    float cb, cz;
    float* losses;      // [2]
    int32_t* counts;    // [S, E]
    float* probs;       // [S, E]
    int32_t* tokens;    // [S + 1]
};
__device__ __forceinline__ void write_losses(const Results& o, int E, int S, float vb, float vz, int N)
{
    const float inv = N ? 1.0f / (float)N : 0.0f;
    o.losses[0] = o.cb * (float)E * inv * vb;
    // (a row of the type's lowest value has an lse^2 past fp32: no 0 * infinity)
    o.losses[1] = o.cz == 0.0f ? 0.0f : o.cz * inv * vz;
    o.tokens[S] = N;
}

// ONE: a single workgroup has all tokens, so every piece is a whole sequence
// and its sums are the results.
template <int LPT, int NCH, bool VEC, bool STREAM, bool ONE>
__global__ __launch_bounds__(NT) void balance_tokens_kernel(Tokens a, const int32_t* __restrict__ topk_idx, int k,
                                                            uint32_t over_k,   // ceil(2^32 / k), k > 1
                                                            float* __restrict__ lse_out, float4* __restrict__ fpart,
                                                            int4* __restrict__ ipart, int rows,
                                                            int* __restrict__ ticket, Results o,
                                                            int32_t* __restrict__ dev_err)
{
    constexpr int NG = NT / LPT, GW = 64 / LPT;   // lane groups per workgroup, per wave
    constexpr int U = NCH == 1 ? 4 : 2;           // tokens in flight per group
    __shared__ float s_p[NT / 64][kMaxExperts];
    __shared__ float s_z[NT / 64];
    __shared__ int s_n[NT / 64], s_m[NT / 64];
    __shared__ int s_cnt[kMaxExperts];
    const int tid = threadIdx.x, l = tid % LPT, grp = tid / LPT, wave = tid >> 6;
    const int E = a.E, vl = last_vector(E);
    float all_b = 0.0f, all_z = 0.0f;   // ONE, wave 0: over the sequences so far
    int all_n = 0;
    if constexpr (ONE) {   // sequences without a token
        for (int64_t i = tid; i < (int64_t)a.S * E; i += NT) {
            o.counts[i] = 0;
            o.probs[i] = 0.0f;
        }
        for (int i = tid; i < a.S; i += NT) o.tokens[i] = 0;
        __syncthreads();
    } else if (blockIdx.x == 0 && tid == 0) {
        *ticket = 0;
    }
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
            Row<LPT, NCH, VEC, STREAM> r[U];
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
                if (Row<LPT, NCH, VEC, STREAM>::col(l, i) < E) s_p[wave][Row<LPT, NCH, VEC, STREAM>::col(l, i)] = sum[i];
            if (l == 0) {
                s_z[wave] = z;
                s_n[wave] = n;
            }
        }
        __syncthreads();   // s_cnt is clear, too
        int m = 0;   // the wave's pairs
        for (int i0 = tid; i0 - tid < pairs; i0 += NT * PQ) {
            if (i0 != tid) load_pairs(i0, ev);
#pragma unroll
            for (int q = 0; q < PQ; ++q) {
                const bool valid = ev[q] >= 0 && ev[q] < E;
                if (valid) atomicAdd(&s_cnt[ev[q]], 1);   // integer: the order does not matter
                m += __popcll(__ballot(valid));
            }
        }
        if ((tid & 63) == 0) s_m[wave] = m;
        __syncthreads();
        auto vector = [&](int v, float (&f)[4], int (&c)[4]) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int e = min(4 * v + i, E - 1);   // (past E: nobody looks)
                f[i] = s_p[0][e];
#pragma unroll
                for (int w = 1; w < NT / 64; ++w) f[i] += s_p[w][e];
                c[i] = s_cnt[e];
            }
        };
        float zz = 0.0f;
        int nn = 0, mm = 0;
        auto scalars = [&]() __attribute__((always_inline)) {
#pragma unroll
            for (int w = 0; w < NT / 64; ++w) {
                zz += s_z[w];
                nn += s_n[w];
                mm += s_m[w];
            }
        };
        if constexpr (ONE) {
            if (wave == 0) {
                scalars();
                float vb = 0.0f;
                for (int v = tid; v < vl; v += 64) {
                    float f[4];
                    int c[4];
                    vector(v, f, c);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int64_t at = (int64_t)s * E + 4 * v + i;
                        if (4 * v + i >= E) break;
                        o.counts[at] = c[i];
                        o.probs[at] = nn ? f[i] / (float)nn : 0.0f;
                        vb += mm ? (float)c[i] / (float)mm * f[i] : 0.0f;   // n f P
                    }
                }
                all_b += segment_sum<64>(vb);
                all_z += zz;
                all_n += nn;
                if (tid == 0) o.tokens[s] = nn;
            }
        } else {
            const int64_t piece = (int64_t)blockIdx.x + s;
            for (int v = tid; v < vl; v += NT) {
                float f[4];
                int c[4];
                vector(v, f, c);
                fpart[v * (int64_t)rows + piece] = make_float4(f[0], f[1], f[2], f[3]);
                ipart[v * (int64_t)rows + piece] = make_int4(c[0], c[1], c[2], c[3]);
            }
            if (tid == NT - 1) {
                scalars();
                fpart[vl * (int64_t)rows + piece] = make_float4(zz, 0.0f, 0.0f, 0.0f);
                ipart[vl * (int64_t)rows + piece] = make_int4(nn, mm, 0, 0);
            }
        }
        __syncthreads();   // the next piece clears the counts
    });
    if (ONE && tid == 0) write_losses(o, E, a.S, all_b, all_z, all_n);
    if (bad && dev_err) atomicOr(dev_err, (int)MOE_ERR_NONFINITE_LOGIT);
}

// Workgroup (s, g): the sums of sequence s's pieces' rows over RW - 1 4-column
// vectors (group g of them) and the rows' last vector: a wave per vector, a lane per row (every 64th), then the lanes.  The
// last workgroup to finish (TICKET) or a kernel behind this one makes the losses
// from what each left in `partial`.
constexpr int RW = 8, RT = 64 * RW;

struct Partial {
    float b, z;      // its experts' n f P; sum of lse^2 (group 0, else 0)
};

template <int L>
__device__ __forceinline__ int segment_sum(int x)
{
#pragma unroll
    for (int off = 1; off < L; off <<= 1) x += __shfl_xor(x, off, 64);
    return x;
}

// The losses from the partial ones of all sequences and groups (one workgroup).
// ATOMIC: they were left by other workgroups of the same launch.
template <bool ATOMIC>
__device__ __forceinline__ void add_losses(const Partial* partial, int n, const Results& o, int S, int E)
{
    __shared__ float s_b[RW], s_z[RW];
    __shared__ int s_n[RW];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    float vb = 0.0f, vz = 0.0f;
    int N = 0;
    for (int i = tid; i < n; i += RT) {
        if constexpr (ATOMIC) {
            vb += __hip_atomic_load(&partial[i].b, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            vz += __hip_atomic_load(&partial[i].z, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            if (i < S) N += __hip_atomic_load(o.tokens + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        } else {
            vb += partial[i].b;
            vz += partial[i].z;
            if (i < S) N += o.tokens[i];
        }
    }
    vb = segment_sum<64>(vb);
    vz = segment_sum<64>(vz);
    N = segment_sum<64>(N);
    if (lane == 0) {
        s_b[wave] = vb;
        s_z[wave] = vz;
        s_n[wave] = N;
    }
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < RW; ++w) {
            vb += s_b[w];
            vz += s_z[w];
            N += s_n[w];
        }
        write_losses(o, E, S, vb, vz, N);
    }
}

__global__ __launch_bounds__(RT) void balance_losses_kernel(const Partial* __restrict__ partial, int n, Results o, int S,
                                                            int E)
{
    add_losses<false>(partial, n, o, S, E);
}

template <bool TICKET>
__global__ __launch_bounds__(RT) void balance_reduce_kernel(Tokens a, const float4* __restrict__ fpart,
                                                            const int4* __restrict__ ipart, int rows,
                                                            int* __restrict__ ticket, Partial* __restrict__ partial,
                                                            Results o)
{
    __shared__ float s_f[RW][4];
    __shared__ int s_i[RW][4];
    __shared__ int s_last;
    const int s = blockIdx.x, g = blockIdx.y, ng = gridDim.y, tid = threadIdx.x;
    const int lane = tid & 63, wave = tid >> 6;
    const int E = a.E, vl = last_vector(E);
    const int begin = seg_at(a, s), end = seg_at(a, s + 1);
    const int b0 = begin / a.TB, b1 = end > begin ? (end - 1) / a.TB + 1 : b0;
    const int v = wave < RW - 1 ? g * (RW - 1) + wave : vl;
    if (wave == RW - 1 || v < vl) {
        float f[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        int c[4] = {0, 0, 0, 0};
#pragma unroll 4
        for (int b = b0 + lane; b < b1; b += 64) {
            const int64_t at = v * (int64_t)rows + b + s;
            const float4 x = fpart[at];
            const int4 i = ipart[at];
            f[0] += x.x;
            f[1] += x.y;
            f[2] += x.z;
            f[3] += x.w;
            c[0] += i.x;
            c[1] += i.y;
            c[2] += i.z;
            c[3] += i.w;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[i] = segment_sum<64>(f[i]);
            c[i] = segment_sum<64>(c[i]);
            if (lane == 0) {
                s_f[wave][i] = f[i];
                s_i[wave][i] = c[i];
            }
        }
    }
    __syncthreads();
    const int n = s_i[RW - 1][0], m = s_i[RW - 1][1];
    if (wave == 0) {
        const int w = lane >> 2, e = 4 * (g * (RW - 1) + w) + (lane & 3);
        float vb = 0.0f;
        if (w < RW - 1 && e < E) {
            const float p = s_f[w][lane & 3];
            const int c = s_i[w][lane & 3];
            o.counts[(int64_t)s * E + e] = c;
            o.probs[(int64_t)s * E + e] = n ? p / (float)n : 0.0f;
            vb = m ? (float)c / (float)m * p : 0.0f;          // n f P
        }
        vb = segment_sum<32>(vb);
        // What passes between workgroups does so through device-scope atomics
        // alone, which are performed where all XCDs see them: each exchange has
        // been when its old value is back, and the ticket is taken after that.
        // (With plain stores between fences the kernel took 4 us longer: a
        // release writes back the XCD's whole L2.)
        if (lane == 0) {
            Partial* q = partial + s * ng + g;
            const float vz = g == 0 ? s_f[RW - 1][0] : 0.0f;
            if constexpr (TICKET) {
                const int o0 = atomicExch(reinterpret_cast<int*>(&q->b), __float_as_int(vb));
                const int o1 = atomicExch(reinterpret_cast<int*>(&q->z), __float_as_int(vz));
                const int o2 = g == 0 ? atomicExch(o.tokens + s, n) : 0;
                asm volatile("" :: "v"(o0), "v"(o1), "v"(o2) : "memory");
                s_last = atomicAdd(ticket, 1) == a.S * ng - 1;
            } else {
                q->b = vb;
                q->z = vz;
                if (g == 0) o.tokens[s] = n;
            }
        }
    }
    if constexpr (TICKET) {
        __syncthreads();
        if (s_last) add_losses<true>(partial, a.S * ng, o, a.S, E);
    }
}

template <int LPT, int NCH, bool VEC, bool STREAM>
__global__ __launch_bounds__(NTB) void balance_bwd_kernel(Tokens a, const int32_t* __restrict__ counts,
                                                         const int32_t* __restrict__ tokens, float cb, float cz,
                                                         const float* __restrict__ dlosses, const float* add,
                                                         float* dlogits)
{
    constexpr int NG = NTB / LPT;
    constexpr int U = NCH == 1 ? 4 : 2;
    using R = Row<LPT, NCH, VEC, STREAM>;
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

// tokens per workgroup: `least`, or as many as leave `most` workgroups
int tokens_per_block(int T, int least, int most)
{
    const int64_t tb = (((int64_t)T + most - 1) / most + 15) / 16 * 16;
    return (int)(tb > least ? tb : least);
}
// forward: two workgroups per CU, since each leaves a row of sums to add up
// (2^16 tokens of 128 experts: 29 us with 1024 workgroups, 17 with 512)
constexpr int kLeastFwd = 64, kMostFwd = 512;
// A workgroup takes the sequences of its run one after another: no longer runs
// than a sequence is on average, down to kShort tokens (300 tokens in 40
// sequences: forward 33 -> 19 us, backward 17.5 -> 11.6; 16 tokens 24 and 15.5, 4
// tokens as 8).
constexpr int kShort = 8;
int not_past_sequences(int tb, int T, int S)
{
    return std::min(tb, std::max((T / S + 7) / 8 * 8, kShort));
}
int tokens_per_block_fwd(int T, int S)
{
    return not_past_sequences(tokens_per_block(T, kLeastFwd, kMostFwd), T, S);
}
// Up to so many workgroups of the reduction take a ticket; more of them would
// wait at it, one after another, for longer than another launch takes (64
// sequences, 64 experts, 192 workgroups: 17.8 -> 16.2 us; 200 of 128, 1000: 30 ->
// 22; 8 of 64, 24: 12.1 -> 12.4, a call 12.3 -> 14.2).
constexpr int kTickets = 64;
// backward: 32 KB of logits a workgroup, nothing to add up after it (2^20
// tokens of 128 experts, with the gradient added on: 263 us; 64 KB 283, 128 KB
// 303; of 16: 32.5, 33.0, 33.9), at least 32 tokens, and 512 workgroups before
// they grow past that
constexpr int kLeastBwd = 32, kElemsBwd = 8192, kFillBwd = 512;
int tokens_per_block_bwd(int T, int E, int S)
{
    int64_t tb = kElemsBwd / E;
    tb = std::min<int64_t>(tb, T / kFillBwd) / 16 * 16;
    return not_past_sequences((int)(tb > kLeastBwd ? tb : kLeastBwd), T, S);
}

template <class F>
void with_shape(int T, int E, bool vec, F&& f)
{
    const bool stream = (int64_t)T * E * 4 >= ((int64_t)256 << 20);
    auto go = [&](auto L, auto N) {
        if (vec && stream) f(L, N, std::true_type{}, std::true_type{});
        else if (vec) f(L, N, std::true_type{}, std::false_type{});
        else f(L, N, std::false_type{}, std::false_type{});
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

// A single workgroup saves the second kernel while it does not take longer
// than that: with 128 experts 128 tokens take 6.1 us (two kernels 9.2), 256 7.9
// (9.0), 512 12.0 (9.3); with 8 experts 2048 take 7.0 (8.8), 4096 10.1 (8.4); it
// takes sequences one after another (256 tokens of 8 experts in two 9.0 us, two
// kernels 11.6; in three 12.0 and 11.7).
inline bool one_workgroup(int T, int E, int S) { return (int64_t)T * E <= 32768 && T <= 2048 && S <= 2; }

inline int64_t piece_rows(int T, int S)
{
    const int tb = tokens_per_block_fwd(T, S);
    return ((int64_t)T + tb - 1) / tb + S;
}

inline int reduce_groups(int E)
{
    return (last_vector(E) + RW - 2) / (RW - 1);
}
inline size_t partial_bytes(int E, int S)
{
    return ((size_t)S * reduce_groups(E) * sizeof(Partial) + 255) / 256 * 256;
}

inline bool vec_ok(int E, const void* p) { return E % 4 == 0 && (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

size_t balance_ws_bytes(int T, int E, int S)
{
    return kTicketBytes + partial_bytes(E, S) + (size_t)piece_rows(T, S) * (last_vector(E) + 1) * 32;
}

hipError_t launch_balance(const float* logits, const int32_t* topk_idx, const uint8_t* mask, const int32_t* seg_off,
                          int S, int T, int E, int k, float cb, float cz, float* losses, int32_t* counts,
                          float* probs, float* lse, int32_t* tokens, void* ws, int32_t* dev_err, hipStream_t s)
{
    const Results o{cb, cz, losses, counts, probs, tokens};
    const uint32_t over_k = (uint32_t)(((1ull << 32) + k - 1) / k);
    if (one_workgroup(T, E, S)) {
        const Tokens a{logits, mask, seg_off, T, E, S, T};
        with_shape(T, E, vec_ok(E, logits), [&](auto L, auto N, auto V, auto) {
            hipLaunchKernelGGL((balance_tokens_kernel<decltype(L)::value, decltype(N)::value, decltype(V)::value, false,
                                true>),
                               dim3(1), dim3(NT), 0, s, a, topk_idx, k, over_k, lse, nullptr, nullptr, 0, nullptr, o,
                               dev_err);
        });
        return hipGetLastError();
    }
    const Tokens a{logits, mask, seg_off, T, E, S, tokens_per_block_fwd(T, S)};
    uint8_t* w = static_cast<uint8_t*>(ws);
    int* ticket = reinterpret_cast<int*>(w);
    Partial* partial = reinterpret_cast<Partial*>(w + kTicketBytes);
    const int rows = (int)piece_rows(T, S);
    float4* fpart = reinterpret_cast<float4*>(w + kTicketBytes + partial_bytes(E, S));
    int4* ipart = reinterpret_cast<int4*>(fpart + (int64_t)rows * (last_vector(E) + 1));
    const int nblk = T > 0 ? (T + a.TB - 1) / a.TB : 1;
    with_shape(T, E, vec_ok(E, logits), [&](auto L, auto N, auto V, auto ST) {
        hipLaunchKernelGGL((balance_tokens_kernel<decltype(L)::value, decltype(N)::value, decltype(V)::value,
                            decltype(ST)::value, false>),
                           dim3((unsigned)nblk), dim3(NT), 0, s, a, topk_idx, k, over_k, lse, fpart, ipart, rows, ticket,
                           o, dev_err);
    });
    const int ng = reduce_groups(E);
    const dim3 grid((unsigned)S, (unsigned)ng);
    if ((int64_t)S * ng <= kTickets) {
        hipLaunchKernelGGL(balance_reduce_kernel<true>, grid, dim3(RT), 0, s, a, fpart, ipart, rows, ticket, partial, o);
    } else {
        hipLaunchKernelGGL(balance_reduce_kernel<false>, grid, dim3(RT), 0, s, a, fpart, ipart, rows, ticket, partial, o);
        hipLaunchKernelGGL(balance_losses_kernel, dim3(1), dim3(RT), 0, s, partial, S * ng, o, S, E);
    }
    return hipGetLastError();
}

hipError_t launch_balance_bwd(const float* logits, const uint8_t* mask, const int32_t* seg_off, int S, int T, int E,
                              const int32_t* counts, const int32_t* tokens, float cb, float cz, const float* dlosses,
                              const float* add, float* dlogits, hipStream_t s)
{
    if (T == 0) return hipSuccess;
    const Tokens a{logits, mask, seg_off, T, E, S, tokens_per_block_bwd(T, E, S)};
    const int nblk = (T + a.TB - 1) / a.TB;
    const bool vec = vec_ok(E, logits) && vec_ok(E, dlogits) && vec_ok(E, add);
    with_shape(T, E, vec, [&](auto L, auto N, auto V, auto ST) {
        hipLaunchKernelGGL((balance_bwd_kernel<decltype(L)::value, decltype(N)::value, decltype(V)::value,
                            decltype(ST)::value>),
                           dim3((unsigned)nblk), dim3(NTB), 0, s, a, counts, tokens, cb, cz, dlosses, add, dlogits);
    });
    return hipGetLastError();
}

}  // namespace moe
