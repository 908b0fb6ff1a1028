// Grouped SwiGLU GEMMs in fp32 on the vector ALUs (the fp32 workload: fp32
// activations and weights, fp32 accumulate).  Same device tile schedule and
// epilogue semantics as the bf16 MFMA path; 64 x 64 tiles, 256 threads with a
// 4 x 4 register micro-tile each, operands staged in LDS as [k][row].
// For the SwiGLU forward a tile's 64 logical columns are 32 gate columns and
// the same 32 up columns, so the epilogue (through LDS) forms h = silu(g) * u.
// The activation-side stages take 32 x 32 tiles (2 x 2 a thread) where 64 x 64
// ones would not fill the GPU twice.  Either way an element is one chain of fmaf
// over ascending k, so the tile does not change a bit of the result.
#include "glu.h"

namespace moe {
namespace {

constexpr int TM = 64, TN = 64, TK = 16;
typedef __attribute__((ext_vector_type(4))) float f32x4;

// GLU: the gate, limit and dropout given at run time (F32M::glu)
enum { EPI_STORE = 0, EPI_SWIGLU_FWD = 1, EPI_SWIGLU_BWD = 2, EPI_GLU_FWD = 3, EPI_GLU_BWD = 4 };
constexpr bool is_gate_up(int epi) { return epi == EPI_SWIGLU_FWD || epi == EPI_GLU_FWD; }

struct F32M {
    const float* A;        // [n_rows, K] grouped rows
    int64_t lda;
    const float* B;        // per-expert weight, B + e * sB
    int64_t ldb, sB;
    bool b_mn;             // B_e stored [K, N] (else [N, K])
    int N, K;
    const int32_t* group_off;
    int capacity, E, ntn;
    int64_t n_rows;
    float* C;
    int64_t ldc;
    float* H;
    int64_t ldh;
    const float* G;
    int64_t ldg;
    int f;
    GluSpec glu;
};

__device__ __forceinline__ float silu(float g) { return g / (1.0f + expf(-g)); }

// the factor of element i of h: 0 where it is dropped.  (A generator call for
// each element, of which it uses an eighth: this path is the small fp32 one.)
__device__ __forceinline__ float drop_factor(const DropSpec& dr, PhiloxKey key, int64_t i)
{
    if (!dr.thr) return 1.0f;
    const uint4 w = philox(key, (uint64_t)i >> 3);
    const int j = (int)(i & 7);
    const uint32_t r = j < 2 ? w.x : j < 4 ? w.y : j < 6 ? w.z : w.w;
    return ((j & 1) ? keep_hi(r, dr.thr) : keep_lo(r, dr.thr)) ? dr.scale : 0.0f;
}

// Bound by latency at the sizes this path is for, so the next four K-steps' operands are on their way in registers
// while one is multiplied, and two LDS stages leave one barrier a K-step (512 rows of 8 experts, d = 128, f = 256: 12 and
// 10 us for the two forward stages; one K-step ahead 12.5 and 14, 64 x 64 tiles with loads between the barriers 24 and 38).
template <int EPI, int T>
__global__ __launch_bounds__(256) void f32_grouped_m_kernel(F32M p)
{
    constexpr int TM = T, TN = T, M = T / 16, TK = 1024 / T, D = 4;
    __shared__ __align__(16) float sA[2][TK][TM + 4];
    __shared__ __align__(16) float sB[2][TK][TN + 4];
    __shared__ float sC[TM][TN + 1];
    __shared__ int s_pref[kMaxExperts + 1];
    __shared__ int s_part[256];

    const int total =
        block_tile_prefix<256>(p.group_off, p.capacity, p.E, p.n_rows, TM, p.ntn, s_pref, s_part);
    if ((int)blockIdx.x >= total) return;
    const int L = blockIdx.x;
    const int e = find_group(s_pref, p.E, L);
    const int64_t g0 = group_begin(p.group_off, p.capacity, e, p.n_rows);
    const int m_e = (int)group_rows(p.group_off, p.capacity, e, p.n_rows);
    const int mt_e = (m_e + TM - 1) / TM;
    const int local = L - s_pref[e];
    const int nt = local / mt_e;
    const int mt = local - nt * mt_e;
    const int64_t row0 = g0 + (int64_t)mt * TM;
    const int rows_valid = min(TM, m_e - mt * TM);
    const float* Be = p.B + (int64_t)e * p.sB;
    const int n0 = is_gate_up(EPI) ? nt * (TN / 2) : nt * TN;

    const int tid = threadIdx.x;
    const int tx = tid % 16, ty = tid / 16;
    // one 16-byte piece of A and of B a thread and K-step: row (or column) r, k .. k + 3; a [K, N] weight: k-row kb,
    // columns nb .. nb + 3.  K and N are multiples of 4, so a piece is inside or outside as a whole.
    const int r = tid / (TK / 4), k = 4 * (tid % (TK / 4));
    const int kb = tid / (TN / 4), nb = 4 * (tid % (TN / 4));
    const f32x4 zero4 = {0.0f, 0.0f, 0.0f, 0.0f};
    int64_t brow = n0 + r;
    bool b_ok = brow < p.N;
    if (is_gate_up(EPI)) {
        const int n = n0 + r % (TN / 2);
        b_ok = n < p.f;
        brow = r < TN / 2 ? n : p.f + n;
    }
    const uint32_t K = p.K;          // (a step past it fits 32 bits)
    f32x4 ar[D], br[D];
    auto load = [&](uint32_t k0, f32x4& a4, f32x4& b4) __attribute__((always_inline)) {
        a4 = r < rows_valid && k0 + k < K ? *reinterpret_cast<const f32x4*>(p.A + (row0 + r) * p.lda + k0 + k) : zero4;
        if (p.b_mn)
            b4 = k0 + kb < K && n0 + nb < p.N ? *reinterpret_cast<const f32x4*>(Be + (int64_t)(k0 + kb) * p.ldb + n0 + nb)
                                                : zero4;
        else
            b4 = b_ok && k0 + k < K ? *reinterpret_cast<const f32x4*>(Be + brow * p.ldb + k0 + k) : zero4;
    };
    auto store = [&](int st, f32x4 a4, f32x4 b4) __attribute__((always_inline)) {
        sA[st][k][r] = a4.x;
        sA[st][k + 1][r] = a4.y;
        sA[st][k + 2][r] = a4.z;
        sA[st][k + 3][r] = a4.w;
        if (p.b_mn) {
            *reinterpret_cast<f32x4*>(&sB[st][kb][nb]) = b4;
        } else {
            sB[st][k][r] = b4.x;
            sB[st][k + 1][r] = b4.y;
            sB[st][k + 2][r] = b4.z;
            sB[st][k + 3][r] = b4.w;
        }
    };
    float acc[M][M] = {};
#pragma unroll
    for (int d = 0; d < D; ++d) load(d * TK, ar[d], br[d]);
    for (uint32_t k0 = 0; k0 < K; k0 += D * TK) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (k0 + d * TK >= K) break;
            store(d & 1, ar[d], br[d]);
            __syncthreads();
            load(k0 + (D + d) * TK, ar[d], br[d]);
#pragma unroll
            for (int kk = 0; kk < TK; ++kk) {
                float a[M], b[M];
#pragma unroll
                for (int i = 0; i < M; ++i) a[i] = sA[d & 1][kk][ty * M + i];
#pragma unroll
                for (int j = 0; j < M; ++j) b[j] = sB[d & 1][kk][tx * M + j];
#pragma unroll
                for (int i = 0; i < M; ++i)
#pragma unroll
                    for (int j = 0; j < M; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < M; ++i)
#pragma unroll
        for (int j = 0; j < M; ++j) sC[ty * M + i][tx * M + j] = acc[i][j];
    __syncthreads();
    PhiloxKey key{};
    if ((EPI == EPI_GLU_FWD || EPI == EPI_GLU_BWD) && p.glu.drop.thr) key = philox_key(p.glu.drop.rng);
    if (is_gate_up(EPI)) {
        for (int idx = tid; idx < TM * (TN / 2); idx += 256) {
            const int r = idx / (TN / 2), c = idx % (TN / 2);
            const int n = n0 + c;
            if (r >= rows_valid || n >= p.f) continue;
            const float g = sC[r][c], u = sC[r][c + TN / 2];
            const int64_t row = row0 + r;
            p.C[row * p.ldc + n] = g;
            p.C[row * p.ldc + p.f + n] = u;
            if constexpr (EPI == EPI_GLU_FWD) {
                const float c = drop_factor(p.glu.drop, key, row * p.f + n), L = p.glu.limit;
                with_act(p.glu.act, [&](auto A) {
                    const float h = act_of<decltype(A)::value, false>(limit_g(g, L)) * limit_u(u, L);
                    p.H[row * p.ldh + n] = c == 0.0f ? 0.0f : h * c;
                });
            } else {
                p.H[row * p.ldh + n] = silu(g) * u;
            }
        }
    } else {
        for (int idx = tid; idx < TM * TN; idx += 256) {
            const int r = idx / TN, c = idx % TN;
            const int n = n0 + c;
            if (r >= rows_valid || n >= p.N) continue;
            const int64_t row = row0 + r;
            const float v = sC[r][c];
            if constexpr (EPI == EPI_STORE) {
                p.C[row * p.ldc + n] = v;
            } else if constexpr (EPI == EPI_GLU_BWD) {
                const float g = p.G[row * p.ldg + n], u = p.G[row * p.ldg + p.f + n];
                const float c = drop_factor(p.glu.drop, key, row * p.f + n), L = p.glu.limit;
                with_act(p.glu.act, [&](auto A) {
                    float a, da;
                    act_and_slope<decltype(A)::value, false>(limit_g(g, L), a, da);
                    const float dh = v * c;
                    p.C[row * p.ldc + n] = c == 0.0f || g > L ? 0.0f : dh * limit_u(u, L) * da;
                    p.C[row * p.ldc + p.f + n] = c == 0.0f || u > L || u < -L ? 0.0f : dh * a;
                });
            } else {
                const float g = p.G[row * p.ldg + n], u = p.G[row * p.ldg + p.f + n];
                const float s = 1.0f / (1.0f + expf(-g));
                const float da = v * u;
                p.C[row * p.ldc + n] = da * s * (1.0f + g * (1.0f - s));
                p.C[row * p.ldc + p.f + n] = v * g * s;
            }
        }
    }
}

struct F32KProblem {
    const float* A;        // [n_rows, M]
    int64_t lda;
    const float* B;        // [n_rows, N]
    int64_t ldb;
    int M, N, mtn, ntn;
    float* C;              // [E, M, N]
    int64_t ldc, sC;
};

struct F32K {
    F32KProblem pr[2];
    int nprob;
    const int32_t* group_off;
    int capacity, E;
    int64_t n_rows;
};

// The weight gradients, K the group's rows: the same loop, 64 x 64 tiles (a layer's backward, us, with loads between the
// barriers and so: 2100 rows of 5 experts, d 132, f 68, 104 and 69; 6000 of 8, d = f = 512, 380 and 316)
__global__ __launch_bounds__(256) void f32_grouped_k_kernel(F32K p)
{
    constexpr int D = 4;
    __shared__ __align__(16) float sA[2][TK][TM + 4];
    __shared__ __align__(16) float sB[2][TK][TN + 4];
    const int t0 = p.pr[0].mtn * p.pr[0].ntn;
    const int tiles_e = t0 + (p.nprob > 1 ? p.pr[1].mtn * p.pr[1].ntn : 0);
    const int L = blockIdx.x;
    const int e = L / tiles_e;
    int local = L - e * tiles_e;
    const int which = local < t0 ? 0 : 1;
    if (which) local -= t0;
    const F32KProblem& q = p.pr[which];
    const int mt = local / q.ntn, nt = local - (local / q.ntn) * q.ntn;
    const int64_t g0 = group_begin(p.group_off, p.capacity, e, p.n_rows);
    const uint32_t m_e = (uint32_t)group_rows(p.group_off, p.capacity, e, p.n_rows);     // (a step past it fits 32 bits)
    const int m0 = mt * TM, n0 = nt * TN;
    const int tid = threadIdx.x;
    const int tx = tid % 16, ty = tid / 16;
    // one 16-byte piece of A and of B a thread and K-step (M and N are multiples of 4: inside or outside as a whole)
    const int kr = tid / 16, c = 4 * (tid % 16);
    const bool a_ok = m0 + c < q.M, b_ok = n0 + c < q.N;
    f32x4 ar[D], br[D];
    auto load = [&](uint32_t k, f32x4& a4, f32x4& b4) __attribute__((always_inline)) {
        const f32x4 zero4 = {0.0f, 0.0f, 0.0f, 0.0f};
        a4 = a_ok && k < m_e ? *reinterpret_cast<const f32x4*>(q.A + (g0 + k) * q.lda + m0 + c) : zero4;
        b4 = b_ok && k < m_e ? *reinterpret_cast<const f32x4*>(q.B + (g0 + k) * q.ldb + n0 + c) : zero4;
    };
    float acc[4][4] = {};
#pragma unroll
    for (int d = 0; d < D; ++d) load(d * TK + kr, ar[d], br[d]);
    for (uint32_t k0 = 0; k0 < m_e; k0 += D * TK) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (k0 + d * TK >= m_e) break;
            *reinterpret_cast<f32x4*>(&sA[d & 1][kr][c]) = ar[d];
            *reinterpret_cast<f32x4*>(&sB[d & 1][kr][c]) = br[d];
            __syncthreads();
            load(k0 + (D + d) * TK + kr, ar[d], br[d]);
#pragma unroll
            for (int kk = 0; kk < TK; ++kk) {
                float a[4], b[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) a[i] = sA[d & 1][kk][ty * 4 + i];
#pragma unroll
                for (int j = 0; j < 4; ++j) b[j] = sB[d & 1][kk][tx * 4 + j];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
            }
        }
    }
    float* Ce = q.C + (int64_t)e * q.sC;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int m = m0 + ty * 4 + i, n = n0 + tx * 4;
        if (m < q.M && n < q.N)
            *reinterpret_cast<f32x4*>(Ce + (int64_t)m * q.ldc + n) = f32x4{acc[i][0], acc[i][1], acc[i][2], acc[i][3]};
    }
}

template <int EPI>
hipError_t launch_m(F32M p, int64_t n_rows, hipStream_t s)
{
    const int cols = is_gate_up(EPI) ? 2 * p.N : p.N;
    auto grid = [&](int T) {
        p.ntn = (cols + T - 1) / T;
        return (n_rows / T + p.E) * (int64_t)p.ntn;
    };
    // 64 x 64 tiles from two for each of 256 CUs on (an upper bound of their number is what is known here)
    const int64_t big = grid(64);
    if (big >= 512) {
        hipLaunchKernelGGL((f32_grouped_m_kernel<EPI, 64>), dim3((unsigned)big), dim3(256), 0, s, p);
    } else {
        const int64_t n = grid(32);
        if (n > 0) hipLaunchKernelGGL((f32_grouped_m_kernel<EPI, 32>), dim3((unsigned)n), dim3(256), 0, s, p);
    }
    return hipGetLastError();
}

hipError_t launch_k(const F32K& p, hipStream_t s)
{
    int64_t tiles_e = 0;
    for (int i = 0; i < p.nprob; ++i) tiles_e += (int64_t)p.pr[i].mtn * p.pr[i].ntn;
    const int64_t grid = (int64_t)p.E * tiles_e;
    if (grid > 0) hipLaunchKernelGGL(f32_grouped_k_kernel, dim3((unsigned)grid), dim3(256), 0, s, p);
    return hipGetLastError();
}

}  // namespace

hipError_t gemm_op_f32(int op, const moe_gemm_tensors& t, GroupSpec g, const GluSpec& glu, int d, int f,
                       hipStream_t s)
{
    F32M p{};
    p.group_off = g.group_off;
    p.capacity = g.capacity;
    p.E = g.E;
    p.n_rows = g.n_rows;
    p.f = f;
    p.glu = glu;
    const bool plain = plain_swiglu(glu);
    switch (op) {
    case MOE_GEMM_GATE_UP:
        p.A = (const float*)t.x_perm;
        p.lda = d;
        p.B = (const float*)t.w13;
        p.ldb = d;
        p.sB = (int64_t)2 * f * d;
        p.b_mn = false;
        p.N = f;
        p.K = d;
        p.C = (float*)t.gu;
        p.ldc = 2 * f;
        p.H = (float*)t.h;
        p.ldh = f;
        if (!plain) return launch_m<EPI_GLU_FWD>(p, g.n_rows, s);
        return launch_m<EPI_SWIGLU_FWD>(p, g.n_rows, s);
    case MOE_GEMM_DOWN:
        p.A = (const float*)t.h;
        p.lda = f;
        p.B = (const float*)t.w2;
        p.ldb = f;
        p.sB = (int64_t)d * f;
        p.b_mn = false;
        p.N = d;
        p.K = f;
        p.C = (float*)t.y_perm;
        p.ldc = d;
        return launch_m<EPI_STORE>(p, g.n_rows, s);
    case MOE_GEMM_DGRAD_DOWN:
        p.A = (const float*)t.dy_perm;
        p.lda = d;
        p.B = (const float*)t.w2;
        p.ldb = f;
        p.sB = (int64_t)d * f;
        p.b_mn = true;
        p.N = f;
        p.K = d;
        p.C = (float*)t.dgu;
        p.ldc = 2 * f;
        p.G = (const float*)t.gu;
        p.ldg = 2 * f;
        if (!plain) return launch_m<EPI_GLU_BWD>(p, g.n_rows, s);
        return launch_m<EPI_SWIGLU_BWD>(p, g.n_rows, s);
    case MOE_GEMM_DGRAD_GATE_UP:
        p.A = (const float*)t.dgu;
        p.lda = 2 * f;
        p.B = (const float*)t.w13;
        p.ldb = d;
        p.sB = (int64_t)2 * f * d;
        p.b_mn = true;
        p.N = d;
        p.K = 2 * f;
        p.C = (float*)t.dx_perm;
        p.ldc = d;
        return launch_m<EPI_STORE>(p, g.n_rows, s);
    case MOE_GEMM_WGRAD: {
        F32K k{};
        k.group_off = g.group_off;
        k.capacity = g.capacity;
        k.E = g.E;
        k.n_rows = g.n_rows;
        k.nprob = 2;
        F32KProblem& a = k.pr[0];
        a.A = (const float*)t.dy_perm;
        a.lda = d;
        a.B = (const float*)t.h;
        a.ldb = f;
        a.M = d;
        a.N = f;
        a.mtn = (d + TM - 1) / TM;
        a.ntn = (f + TN - 1) / TN;
        a.C = (float*)t.dw2;
        a.ldc = f;
        a.sC = (int64_t)d * f;
        F32KProblem& b = k.pr[1];
        b.A = (const float*)t.dgu;
        b.lda = 2 * f;
        b.B = (const float*)t.x_perm;
        b.ldb = d;
        b.M = 2 * f;
        b.N = d;
        b.mtn = (2 * f + TM - 1) / TM;
        b.ntn = (d + TN - 1) / TN;
        b.C = (float*)t.dw13;
        b.ldc = d;
        b.sC = (int64_t)2 * f * d;
        return launch_k(k, s);
    }
    default:
        return hipErrorInvalidValue;
    }
}

}  // namespace moe
