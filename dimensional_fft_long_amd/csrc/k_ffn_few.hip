// k_ffn_few.hip -- the gated feed-forward block's forward for few positions
// (single tokens of a few streams): the weights are the traffic, each read once.
//
// A workgroup owns 16 rows of the weights and all positions (16 per matrix
// column tile); its waves deal the summation index among themselves in steps of
// 32 and are joined through LDS in a fixed order.  Weights go from memory
// straight into the matrix instruction's operand registers (16 bytes of a row a
// lane), four steps in flight per wave: with one workgroup per 16 rows the
// whole weight matrix is requested at once, which is what a launch this short
// is bounded by.  Nothing is packed: rows may start anywhere and K may be any
// length.  fp32 splits into three bf16 planes in registers.  Measured on one
// MI355X, four positions, C = 1024, F = 4096, bf16: 7.2 and 8.3 us (16.8 and 8.4
// MB), against 16.7 and 43.3 us through the tiles.
#include "ffn_tile.h"

namespace hyenand {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

struct FewArgs {
    const void *w0, *w1;  // [M][K]
    const void* x;        // element (k, n) at n * xn + k * xk, or (n / xL) * xb + n % xL + k * xk
    long long xk, xb;
    int xL;
    void* out;            // element (m, n) at (n / oL) * ob + n % oL + m * om
    long long om, ob;
    int oL;
    int M, K, N, act;
};

template <class T>
struct Terms {
    static constexpr int NPL = sizeof(T) == 2 ? 1 : 3;
    bf16x8 p[NPL];
};

// Eight consecutive terms, zeros from nv on; stride in elements.
template <class T, bool CONTIG>
__device__ __forceinline__ Terms<T> load_terms(const T* p, int nv, long long stride)
{
    Terms<T> r;
    Pack<T, 8> q;
    if constexpr (CONTIG) {
        q = load_pack<T, 8>(p, nv);
    } else {
#pragma unroll
        for (int i = 0; i < Pack<T, 8>::N; ++i) q.w[i] = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < nv) {
                const unsigned b = bits_of(p[i * stride]);
                if constexpr (sizeof(T) == 2) q.w[i >> 1] |= b << (16 * (i & 1));
                else q.w[i] = b;
            }
    }
    if constexpr (sizeof(T) == 2) {
        r.p[0] = __builtin_bit_cast(bf16x8, u32x4{q.w[0], q.w[1], q.w[2], q.w[3]});
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float s[3];
            split3(q.get(i), s);
#pragma unroll
            for (int k = 0; k < 3; ++k) r.p[k][i] = (__bf16)s[k];
        }
    }
    return r;
}

template <class T>
__device__ __forceinline__ f32x4 multiply_terms(const Terms<T>& a, const Terms<T>& b, f32x4 c)
{
    if constexpr (sizeof(T) == 4) {  // pairs of planes, smallest first
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.p[2], b.p[0], c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.p[1], b.p[1], c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.p[0], b.p[2], c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.p[1], b.p[0], c, 0, 0, 0);
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.p[0], b.p[1], c, 0, 0, 0);
    }
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.p[0], b.p[0], c, 0, 0, 0);
}

// GATE: out = a(w0 x) (w1 x), else out = w0 x.  NT: column tiles of 16 positions.
template <class T, bool GATE, bool XCONTIG, int NT>
__global__ __launch_bounds__(1024) void k_ffn_few(FewArgs a)
{
    extern __shared__ __align__(16) float red[];
    constexpr int G = GATE ? 2 : 1;
    const int t = (int)threadIdx.x, lane = t & 63, w = t >> 6, nw = (int)blockDim.x >> 6;
    const int m0 = (int)blockIdx.x * 16, kq = (lane >> 4) * 8, r = lane & 15;
    const int m = m0 + r < a.M ? m0 + r : a.M - 1;
    const T *p0 = (const T*)a.w0 + (long long)m * a.K, *p1 = GATE ? (const T*)a.w1 + (long long)m * a.K : nullptr;
    const T* px[NT];
    bool live[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int n = j * 16 + r;
        live[j] = n < a.N;
        const int nn = live[j] ? n : 0, q = nn / a.xL;
        px[j] = (const T*)a.x + q * a.xb + (nn - q * a.xL);
    }
    f32x4 acc[G][NT] = {};
    const int steps = (a.K + 31) / 32;
    constexpr int U = sizeof(T) == 2 ? (NT <= 2 ? 4 : 2) : (NT == 1 ? 2 : 1);  // steps in flight
    for (int s0 = w; s0 < steps; s0 += U * nw) {
        Terms<T> fa[G][U], fb[U][NT];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int k = (s0 + i * nw) * 32 + kq, left = a.K - k, nv = left >= 8 ? 8 : left > 0 ? left : 0;
            fa[0][i] = load_terms<T, true>(p0 + k, nv, 1);
            if constexpr (GATE) fa[G - 1][i] = load_terms<T, true>(p1 + k, nv, 1);
#pragma unroll
            for (int j = 0; j < NT; ++j)
                fb[i][j] = load_terms<T, XCONTIG>(px[j] + k * a.xk, live[j] ? nv : 0, a.xk);
        }
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int g = 0; g < G; ++g) acc[g][j] = multiply_terms<T>(fa[g][i], fb[i][j], acc[g][j]);
    }
    // Join the waves: [wave][group][tile][lane] of four rows.
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
        for (int j = 0; j < NT; ++j)
            *reinterpret_cast<f32x4*>(red + (((w * G + g) * NT + j) * 64 + lane) * 4) = acc[g][j];
    __syncthreads();
    for (int e = t; e < NT * 64; e += (int)blockDim.x) {
        f32x4 v[G] = {};
        for (int i = 0; i < nw; ++i)
#pragma unroll
            for (int g = 0; g < G; ++g)
                v[g] += *reinterpret_cast<const f32x4*>(red + ((i * G + g) * NT * 64 + e) * 4);
        const int n = e >> 6 << 4 | (e & 15), mr = m0 + ((e >> 4) & 3) * 4;
        if (n >= a.N) continue;
        const int q = n / a.oL;
        T* o = (T*)a.out + q * a.ob + (n - q * a.oL);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float f = v[0][i];
            if constexpr (GATE) f = act_fwd(a.act, f) * v[G - 1][i];
            if (mr + i < a.M) o[(mr + i) * a.om] = (T)f;
        }
    }
}

template <class T, bool GATE, bool XCONTIG, int NT>
hipError_t few(const FewArgs& a, hipStream_t st)
{
    // Waves: about four steps each, as many as the join's LDS takes.
    const int steps = (a.K + 31) / 32;
    int nw = (steps + 3) / 4;
    const int most = 32 / ((GATE ? 2 : 1) * NT) < 16 ? 32 / ((GATE ? 2 : 1) * NT) : 16;
    nw = nw < 1 ? 1 : nw > most ? most : nw;
    const size_t lds = (size_t)nw * (GATE ? 2 : 1) * NT * 1024;
    hipLaunchKernelGGL((k_ffn_few<T, GATE, XCONTIG, NT>), dim3((unsigned)((a.M + 15) / 16)), dim3(64 * nw), lds, st, a);
    return launch_status();
}

template <class T, bool GATE, bool XCONTIG>
hipError_t few_n(const FewArgs& a, hipStream_t st)
{
    if (a.N <= 16) return few<T, GATE, XCONTIG, 1>(a, st);
    if (a.N <= 32) return few<T, GATE, XCONTIG, 2>(a, st);
    return few<T, GATE, XCONTIG, 4>(a, st);
}

template <class T>
hipError_t forward(const FfnArgs& f, hipStream_t st)
{
    const int N = (int)(f.B * f.L);
    FewArgs a{};
    a.w0 = f.Wg;
    a.w1 = f.Wu;
    a.x = f.x;
    a.xk = f.L;
    a.xb = f.C * f.L;
    a.xL = (int)f.L;
    a.out = f.ws;  // h [position][F]
    a.om = 1;
    a.ob = f.F;
    a.oL = 1;
    a.M = f.F;
    a.K = f.C;
    a.N = N;
    a.act = f.act;
    hipError_t e = f.L == 1 ? few_n<T, true, true>(a, st) : few_n<T, true, false>(a, st);
    if (e != hipSuccess) return e;
    FewArgs d{};
    d.w0 = f.Wd;
    d.x = f.ws;
    d.xk = 1;
    d.xb = f.F;
    d.xL = 1;
    d.out = f.y;
    d.om = f.L;
    d.ob = f.C * f.L;
    d.oL = (int)f.L;
    d.M = f.C;
    d.K = f.F;
    d.N = N;
    return few_n<T, false, true>(d, st);
}

}  // namespace

hipError_t launch_ffn_few(const FfnArgs& a, hipStream_t st)
{
    return a.bf16 ? forward<__bf16>(a, st) : forward<float>(a, st);
}

}  // namespace hyenand
