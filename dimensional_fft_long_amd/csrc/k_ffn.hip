// k_ffn.hip -- the gated feed-forward block, forward and backward: products of
// weights and activations with the activation and the gate product in their
// epilogues.
#include "block_dev.h"

namespace hyenand {
namespace {

// A matrix of activations or weights: element (r, t) at
// r * sr + (t / L) * sb + (t % L) * st.
struct View {
    const void* p;
    long long sr, st, L, sb;
};

struct GemmArgs {
    View A[2], B[2];  // C[n] = sum_k A[n](m, k) B[n](k, t): k is B's row index, or its column index with BT
    int nprod;        // products (accumulated into one result, or kept apart with DUAL)
    int M, N;
    long long K;
    void *o0, *o1, *o2;            // outputs, [M][ldo] or through oL / osb
    const void *i0, *i1;           // saved g and u (backward epilogue)
    long long osr, oL, osb;
    int act;
};

template <class T>
__device__ __forceinline__ float at(const View& v, long long r, long long t)
{
    return (float)((const T*)v.p)[r * v.sr + (t / v.L) * v.sb + (t % v.L) * v.st];
}

enum { kEpiStore = 0, kEpiGate = 1, kEpiGrad = 2 };

// 64 x 64 outputs by 256 threads, 4 x 4 each, through LDS tiles of 16 terms.
template <class T, bool BT, int EPI>
__global__ __launch_bounds__(256) void k_ffn_gemm(GemmArgs a)
{
    __shared__ float As[16][65], Bs[16][65];
    constexpr int NACC = EPI == kEpiGate ? 2 : 1;
    const int t = (int)threadIdx.x, tx = t & 15, ty = t >> 4;
    const long long m0 = (long long)blockIdx.y * 64, n0 = (long long)blockIdx.x * 64;
    float acc[NACC][4][4] = {};
    for (int p = 0; p < a.nprod; ++p) {
        const View va = a.A[p], vb = a.B[p];
        for (long long k0 = 0; k0 < a.K; k0 += 16) {
            for (int i = t; i < 1024; i += 256) {
                const int kk = i >> 6, c = i & 63;
                const long long k = k0 + kk;
                As[kk][c] = (k < a.K && m0 + c < a.M) ? at<T>(va, m0 + c, k) : 0.0f;
                Bs[kk][c] = (k < a.K && n0 + c < a.N) ? (BT ? at<T>(vb, n0 + c, k) : at<T>(vb, k, n0 + c)) : 0.0f;
            }
            __syncthreads();
            for (int kk = 0; kk < 16; ++kk) {
                float ra[4], rb[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    ra[i] = As[kk][ty * 4 + i];
                    rb[i] = Bs[kk][tx * 4 + i];
                }
#pragma unroll
                for (int n = 0; n < NACC; ++n)
                    if (NACC == 1 || n == p)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int j = 0; j < 4; ++j) acc[n][i][j] += ra[i] * rb[j];
            }
            __syncthreads();
        }
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const long long m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
            if (m >= a.M || n >= a.N) continue;
            const long long o = m * a.osr + (n / a.oL) * a.osb + n % a.oL;
            if constexpr (EPI == kEpiStore) {
                ((T*)a.o0)[o] = (T)acc[0][i][j];
            } else if constexpr (EPI == kEpiGate) {
                const float g = acc[0][i][j], u = acc[NACC - 1][i][j];
                ((T*)a.o0)[o] = (T)(act_fwd(a.act, g) * u);
                if (a.o1) {
                    ((T*)a.o1)[o] = (T)g;
                    ((T*)a.o2)[o] = (T)u;
                }
            } else {
                const float g = (float)((const T*)a.i0)[o], u = (float)((const T*)a.i1)[o], dh = acc[0][i][j];
                float ga, da;
                act_both(a.act, g, ga, da);
                ((T*)a.o1)[o] = (T)(dh * u * da);
                ((T*)a.o2)[o] = (T)(dh * ga);
            }
        }
}

template <class T, bool BT, int EPI>
hipError_t gemm(const GemmArgs& a, hipStream_t st)
{
    if (a.M <= 0 || a.N <= 0) return hipSuccess;
    hipLaunchKernelGGL((k_ffn_gemm<T, BT, EPI>), dim3((unsigned)((a.N + 63) / 64), (unsigned)((a.M + 63) / 64)),
                       dim3(256), 0, st, a);
    return launch_status();
}

constexpr long long kFar = 1ll << 62;

template <class T>
hipError_t forward(const FfnArgs& a, bool save, hipStream_t st)
{
    const long long Tn = a.B * a.L;
    T* h = (T*)a.ws;
    const View x{a.x, a.L, 1, a.L, a.C * a.L}, wg{a.Wg, a.C, 1, kFar, 0}, wu{a.Wu, a.C, 1, kFar, 0};
    GemmArgs g{};
    g.A[0] = wg;
    g.A[1] = wu;
    g.B[0] = g.B[1] = x;
    g.nprod = 2;
    g.M = a.F;
    g.N = (int)Tn;
    g.K = a.C;
    g.o0 = h;
    if (save) {
        g.o1 = h + a.F * Tn;
        g.o2 = h + 2 * a.F * Tn;
    }
    g.osr = Tn;
    g.oL = kFar;
    g.act = a.act;
    hipError_t e = gemm<T, false, kEpiGate>(g, st);
    if (e != hipSuccess || save) return e;
    GemmArgs d{};
    d.A[0] = View{a.Wd, a.F, 1, kFar, 0};
    d.B[0] = View{h, Tn, 1, kFar, 0};
    d.nprod = 1;
    d.M = a.C;
    d.N = (int)Tn;
    d.K = a.F;
    d.o0 = a.y;
    d.osr = a.L;
    d.oL = a.L;
    d.osb = a.C * a.L;
    return gemm<T, false, kEpiStore>(d, st);
}

template <class T>
hipError_t backward(const FfnArgs& a, hipStream_t st)
{
    const long long Tn = a.B * a.L;
    T *h = (T*)a.ws, *dg = h + a.F * Tn, *du = dg + a.F * Tn;
    const View x{a.x, a.L, 1, a.L, a.C * a.L}, dy{a.dy, a.L, 1, a.L, a.C * a.L};
    const View vh{h, Tn, 1, kFar, 0}, vdg{dg, Tn, 1, kFar, 0}, vdu{du, Tn, 1, kFar, 0};
    hipError_t e = forward<T>(a, true, st);  // h, g, u
    if (e != hipSuccess) return e;
    GemmArgs g{};
    g.A[0] = View{a.Wd, 1, a.F, kFar, 0};  // Wd^T
    g.B[0] = dy;
    g.nprod = 1;
    g.M = a.F;
    g.N = (int)Tn;
    g.K = a.C;
    g.i0 = g.o1 = dg;  // g and u are read and replaced by their gradients
    g.i1 = g.o2 = du;
    g.osr = Tn;
    g.oL = kFar;
    g.act = a.act;
    if ((e = gemm<T, false, kEpiGrad>(g, st)) != hipSuccess) return e;
    GemmArgs d{};
    d.A[0] = View{a.Wg, 1, a.C, kFar, 0};
    d.A[1] = View{a.Wu, 1, a.C, kFar, 0};
    d.B[0] = vdg;
    d.B[1] = vdu;
    d.nprod = 2;
    d.M = a.C;
    d.N = (int)Tn;
    d.K = a.F;
    d.o0 = a.dx;
    d.osr = a.L;
    d.oL = a.L;
    d.osb = a.C * a.L;
    if ((e = gemm<T, false, kEpiStore>(d, st)) != hipSuccess) return e;
    for (int i = 0; i < 3; ++i) {
        GemmArgs w{};
        w.A[0] = i == 0 ? vdg : i == 1 ? vdu : dy;
        w.B[0] = i < 2 ? x : vh;
        w.nprod = 1;
        w.M = i < 2 ? a.F : a.C;
        w.N = i < 2 ? a.C : a.F;
        w.K = Tn;
        w.o0 = i == 0 ? a.dWg : i == 1 ? a.dWu : a.dWd;
        w.osr = w.N;
        w.oL = kFar;
        if ((e = gemm<T, true, kEpiStore>(w, st)) != hipSuccess) return e;
    }
    return hipSuccess;
}

__global__ __launch_bounds__(256) void k_ffn_zero(unsigned short* p, long long n)
{
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i < n) p[i] = 0;
}

}  // namespace

hipError_t launch_ffn_zero(void* p, long long bytes, hipStream_t st)
{
    const long long n = bytes / 2;
    hipLaunchKernelGGL(k_ffn_zero, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st, (unsigned short*)p, n);
    return launch_status();
}

size_t ffn_workspace(int B, int C, int F, long long L, bool bf16, bool bwd)
{
    (void)C;
    return (size_t)B * (size_t)L * (size_t)F * (bf16 ? 2u : 4u) * (bwd ? 3u : 1u);
}

hipError_t launch_ffn_fwd(const FfnArgs& a, hipStream_t st)
{
    return a.bf16 ? forward<__bf16>(a, false, st) : forward<float>(a, false, st);
}

hipError_t launch_ffn_bwd(const FfnArgs& a, hipStream_t st)
{
    return a.bf16 ? backward<__bf16>(a, st) : backward<float>(a, st);
}

}  // namespace hyenand
