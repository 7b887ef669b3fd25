// block_dev.h -- device pieces shared by the residual block's kernels: I/O of
// rows at any alignment, the gate activations and the dropout generator.
#pragma once

#include <type_traits>

#include "block.h"

namespace hyenand {
namespace {

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

inline hipError_t launch_status() { return hipGetLastError(); }

typedef __attribute__((address_space(3))) void lds_void;

// 16 bytes a lane from global memory to LDS at the wave-uniform address l plus
// 16 times the lane.  In assembly because the compiler, which cannot tell the
// stage being filled from the one being read, waits for the builtin's load
// before the next LDS read.  The instruction has no destination register; it is
// complete at wait_loads(), which comes before the barrier ahead of its use.
__device__ __forceinline__ void to_lds(const void* g, unsigned l)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(l), "v"(g) : "memory");
}

// All but the newest N of this wave's loads are complete.
template <int N = 0>
__device__ __forceinline__ void wait_loads()
{
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

__device__ __forceinline__ unsigned lds_address(const void* p)
{
    return (unsigned)(unsigned long long)(lds_void*)p;
}

// V consecutive elements of type T (float or __bf16), kept as loaded (two bf16
// a register).  A group need not be aligned beyond its element: gfx950's vector
// memory instructions take any address, so a row that starts at an odd element
// still moves in wide accesses.
template <int N, int ALIGN>
struct __attribute__((packed, aligned(ALIGN))) WordsMem {
    unsigned w[N];
};

template <class T, int V>
struct Pack {
    static constexpr bool kHalf = sizeof(T) == 2;
    static constexpr int N = kHalf ? (V + 1) / 2 : V;
    unsigned w[N];
    __device__ __forceinline__ float get(int v) const
    {
        if constexpr (!kHalf) return __builtin_bit_cast(float, w[v]);
        else return __builtin_bit_cast(float, (v & 1) ? w[v >> 1] & 0xffff0000u : w[v >> 1] << 16);
    }
};

__device__ __forceinline__ unsigned bits_of(float f) { return __builtin_bit_cast(unsigned, f); }
__device__ __forceinline__ unsigned bits_of(__bf16 f) { return __builtin_bit_cast(unsigned short, f); }

// The nv <= V first elements of p (zeros behind them).
template <class T, int V>
__device__ __forceinline__ Pack<T, V> load_pack(const T* p, int nv)
{
    Pack<T, V> r;
    if constexpr (V == 1) {
        r.w[0] = nv > 0 ? bits_of(p[0]) : 0u;
    } else {
        if (nv == V) {
            const auto q = *reinterpret_cast<const WordsMem<Pack<T, V>::N, sizeof(T)>*>(p);
#pragma unroll
            for (int i = 0; i < Pack<T, V>::N; ++i) r.w[i] = q.w[i];
        } else if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int i = 0; i < V / 2; ++i)
                r.w[i] = (2 * i < nv ? bits_of(p[2 * i]) : 0u) | (2 * i + 1 < nv ? bits_of(p[2 * i + 1]) << 16 : 0u);
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) r.w[v] = v < nv ? bits_of(p[v]) : 0u;
        }
    }
    return r;
}

// Stores round to nearest even.
template <class T, int V>
__device__ __forceinline__ void store_pack(T* p, const float (&f)[V], int nv)
{
    if constexpr (V > 1) {
        if (nv == V) {
            WordsMem<Pack<T, V>::N, sizeof(T)> q;
#pragma unroll
            for (int i = 0; i < Pack<T, V>::N; ++i) {
                if constexpr (sizeof(T) == 2) q.w[i] = bits_of((T)f[2 * i]) | bits_of((T)f[2 * i + 1]) << 16;
                else q.w[i] = bits_of(f[i]);
            }
            *reinterpret_cast<WordsMem<Pack<T, V>::N, sizeof(T)>*>(p) = q;
            return;
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (v < nv) p[v] = (T)f[v];
}

constexpr float kLog2e = 1.44269504088896341f;

// exp(-v), capped below infinity so that its products with the logistic of v
// stay finite; NaN stays NaN.
__device__ __forceinline__ float exp_neg(float v)
{
    float t = -v * kLog2e;
    t = t > 126.0f ? 126.0f : t;
    return __builtin_amdgcn_exp2f(t);
}

enum { kActNone = 0, kActSigmoid = 1, kActSilu = 2, kActGelu = 3, kActOne = 4 };  // One: no gate at all

// Activation a(v) and its derivative.  1 - s is taken as exp(-v) s, which keeps
// its relative accuracy where s rounds to one.
__device__ __forceinline__ float act_fwd(int act, float v)
{
    if (act == kActOne) return 1.0f;
    if (act == kActNone) return v;
    if (act == kActGelu) return 0.5f * v * (1.0f + erff(v * 0.707106781186547524f));
    const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-v * kLog2e));
    return act == kActSilu ? v * s : s;
}

__device__ __forceinline__ void act_both(int act, float v, float& a, float& da)
{
    if (act == kActOne) {
        a = 1.0f;
        da = 0.0f;
        return;
    }
    if (act == kActNone) {
        a = v;
        da = 1.0f;
        return;
    }
    if (act == kActGelu) {
        const float cdf = 0.5f * (1.0f + erff(v * 0.707106781186547524f));
        a = v * cdf;
        da = cdf + v * (0.398942280401432678f * __builtin_amdgcn_exp2f(-0.5f * v * v * kLog2e));
        return;
    }
    const float e = exp_neg(v), s = __builtin_amdgcn_rcpf(1.0f + e), q = e * s;  // q = 1 - s
    if (act == kActSilu) {
        a = v * s;
        da = s * (1.0f + v * q);
    } else {
        a = s;
        da = s * q;
    }
}

// f(the activation as a constant): loops over elements then hold no branches.
template <class F>
__device__ __forceinline__ void with_act(int act, F&& f)
{
    if (act == kActSilu) f(std::integral_constant<int, kActSilu>{});
    else if (act == kActSigmoid) f(std::integral_constant<int, kActSigmoid>{});
    else f(std::integral_constant<int, kActGelu>{});
}

// The same for a join's gate.
template <class F>
__device__ __forceinline__ void with_gate(bool gate, int act, F&& f)
{
    if (!gate) f(std::integral_constant<int, kActOne>{});
    else if (act == kActSigmoid) f(std::integral_constant<int, kActSigmoid>{});
    else if (act == kActSilu) f(std::integral_constant<int, kActSilu>{});
    else f(std::integral_constant<int, kActNone>{});
}

// Four words of the counter-based generator Philox 4x32 with 10 rounds (Salmon
// et al., "Parallel random numbers: as easy as 1, 2, 3", 2011) at counter ctr.
__device__ __forceinline__ void random4(unsigned long long key, unsigned long long ctr, unsigned (&w)[4])
{
    unsigned c0 = (unsigned)ctr, c1 = (unsigned)(ctr >> 32), c2 = 0, c3 = 0;
    unsigned k0 = (unsigned)key, k1 = (unsigned)(key >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const unsigned long long a = (unsigned long long)c0 * 0xD2511F53u, b = (unsigned long long)c2 * 0xCD9E8D57u;
        c0 = (unsigned)(b >> 32) ^ c1 ^ k0;
        c1 = (unsigned)b;
        c2 = (unsigned)(a >> 32) ^ c3 ^ k1;
        c3 = (unsigned)a;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    w[0] = c0;
    w[1] = c1;
    w[2] = c2;
    w[3] = c3;
}

// Keep bits of the V consecutive elements from linear index e0 on: bit v set
// iff element e0 + v is kept.  Element e takes word e % 4 of the block at
// counter offset + e / 4.  `whole` (the same for all lanes): no group of four
// reaches past ceil(V / 4) blocks, the case of rows that are multiples of four.
template <int V>
__device__ __forceinline__ unsigned keep_bits(unsigned long long seed, unsigned long long offset, unsigned thr,
                                              unsigned long long e0, bool whole)
{
    const unsigned sh = (unsigned)e0 & 3u;
    const unsigned long long q = offset + (e0 >> 2);
    constexpr int G = (V + 3) / 4;
    unsigned bits = 0;
    const auto block = [&](int g) {
        unsigned w[4];
        random4(seed, q + g, w);
#pragma unroll
        for (int j = 0; j < 4; ++j) bits |= (w[j] >= thr ? 1u : 0u) << (4 * g + j);
    };
#pragma unroll
    for (int g = 0; g < G; ++g) block(g);
    if constexpr (V > 1) {
        if (!whole) block(G);
    }
    return bits >> sh;
}

}  // namespace
}  // namespace hyenand
