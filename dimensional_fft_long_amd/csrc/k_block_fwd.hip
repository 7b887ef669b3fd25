// k_block_fwd.hip -- the norm ahead of a block, the join behind it (norm of the
// block's output, gate, residual scale, dropout, residual sum, the next norm),
// forward, and dropout.
//
// Measured on one MI355X (a large copy moves 5.1 TB/s): norm of 32 x 128^3 fp32
// 102 us, 5.2 TB/s; join of 8 x 64 x 256^2 fp32 (five tensors) 132 us, 5.1 TB/s;
// join of 2 x 128 x 1024^2 bf16 0.67 ms, 4.0 TB/s (its rows lie 2 MB apart, and
// rows a power of two apart cost about a tenth against rows 2.002 MB apart).
#include "block_tile.h"

namespace hyenand {
namespace {

// Four waves a SIMD (128 registers) also where a few registers then spill: with
// eight positions and four groups of channels a thread, the join of 2 x 128 x
// 1024^2 bf16 takes 675 us so and 780 us with two waves.  fp32 with eight groups
// keeps two waves of 256 registers (717 channels by 131072: 962 -> 492 us).
template <class T, bool JOIN, int V, int K, bool ROW, int NT>
__global__ __launch_bounds__(NT, V * K * (JOIN ? (int)sizeof(T) : 2) <= 64 ? 4 : 2) void k_block_fwd(BlockArgs a, Lay g)
{
    __shared__ __align__(16) float red[2 * red_floats(NT)];
    int turn = 0;
    const float invC = 1.0f / (float)a.C;
    unsigned long long seed = 0, offs = 0;
    const bool drop = JOIN && a.drop.rng;
    if (drop) {
        seed = a.drop.rng[0];
        offs = a.drop.rng[1];
    }
    Params<V, K, ROW> wpost, sc, wpre;
    {
        const Where<V, ROW> w(a, g);  // channels only
        if (JOIN) {
            wpost.load(a.w_post, w, 1.0f);
            sc.load(a.scale, w, 1.0f);
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < (ROW ? V : 1); ++i) sc.v[k][i] *= wpost.v[k][i] * (drop ? a.drop.up : 1.0f);
        }
        wpre.load(a.w_pre, w, 0.0f);
    }
    Where<V, ROW> w(a, g);
    const Run tiles(g);
    for (long long tile = tiles.first; tile < tiles.end; tile += tiles.step) {
        w.at(a, g, tile);
        Pack<T, V> xr[K], mr[JOIN ? K : 1], gr[JOIN ? K : 1];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (JOIN) mr[k] = load_group<T, V, ROW>(a.m, w, k);
            xr[k] = load_group<T, V, ROW>(a.x, w, k);
            if (JOIN && a.gate) gr[k] = load_group<T, V, ROW>(a.gate, w, k);
        }
        // Dropout's words while the loads are in flight.
        unsigned keep[JOIN ? K : 1];
        if (JOIN) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                keep[k] = ~0u;
                if (drop) keep[k] = keep_bits<V>(seed, offs, a.drop.thr, (unsigned long long)w.off(k), g.whole4);
            }
        }
        float rm[1][V];
#pragma unroll
        for (int v = 0; v < V; ++v) rm[0][v] = 1.0f;
        if (JOIN && a.w_post) {
#pragma unroll
            for (int v = 0; v < V; ++v) rm[0][v] = 0.0f;
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (!ROW || w.mine(k, v)) rm[0][v] += mr[k].get(v) * mr[k].get(v);
            sum_channels<1, V, ROW, NT>(rm, red, turn, g.lxs);
#pragma unroll
            for (int v = 0; v < V; ++v) rm[0][v] = __builtin_amdgcn_rsqf(rm[0][v] * invC + a.eps);
        }
        float o[K][V], ro[1][V];
#pragma unroll
        for (int v = 0; v < V; ++v) ro[0][v] = 0.0f;
        if constexpr (JOIN) {
            with_gate(a.gate != nullptr, a.act, [&](auto act) __attribute__((always_inline)) {
#pragma unroll
                for (int k = 0; k < K; ++k) {
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        const float b = sc.at(k, v) * act_fwd(act, gr[k].get(v)) * (mr[k].get(v) * rm[0][v]);
                        const float val = xr[k].get(v);
                        o[k][v] = val + kept(keep[k], v, b);
                    }
                    store_group<T, V, ROW>(a.out, w, k, o[k]);
                }
            });
        } else {
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int v = 0; v < V; ++v) o[k][v] = xr[k].get(v);
        }
        if (a.w_pre) {
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (!ROW || w.mine(k, v)) ro[0][v] += o[k][v] * o[k][v];
            sum_channels<1, V, ROW, NT>(ro, red, turn, g.lxs);
#pragma unroll
            for (int v = 0; v < V; ++v) ro[0][v] = __builtin_amdgcn_rsqf(ro[0][v] * invC + a.eps);
#pragma unroll
            for (int k = 0; k < K; ++k) {
#pragma unroll
                for (int v = 0; v < V; ++v) o[k][v] *= ro[0][v] * wpre.at(k, v);
                store_group<T, V, ROW>(a.h, w, k, o[k]);
            }
        }
    }
}

template <class T, bool JOIN, int V, int K, bool ROW, int NT = 512>
hipError_t run(const BlockArgs& a, const Shape& s, hipStream_t st)
{
    const long long cap = 1ll << 30;
    const unsigned grid = (unsigned)(s.g.tiles < cap ? s.g.tiles : cap);
    hipLaunchKernelGGL((k_block_fwd<T, JOIN, V, K, ROW, NT>), dim3(grid), dim3(s.nt), 0, st, a, s.g);
    return launch_status();
}

template <class T, bool JOIN>
hipError_t dispatch(const BlockArgs& a, hipStream_t st)
{
    constexpr int V = 16 / (int)sizeof(T);
    const Shape s = pick(a, V, 512, 4, 8);
    if (s.row) {
        if (s.K == 1) return run<T, JOIN, V, 1, true>(a, s, st);
        if (s.K == 2) return run<T, JOIN, V, 2, true>(a, s, st);
        return run<T, JOIN, V, 4, true>(a, s, st);
    }
    if (s.V > 1) {
        if (s.nt == 64) return run<T, JOIN, V, 1, false, 64>(a, s, st);
        if (s.nt == 128) return run<T, JOIN, V, 1, false, 128>(a, s, st);
        if (s.nt == 256) return run<T, JOIN, V, 1, false, 256>(a, s, st);
        if (s.K == 1) return run<T, JOIN, V, 1, false>(a, s, st);
        if (s.K == 2) return run<T, JOIN, V, 2, false>(a, s, st);
        if (s.K == 4) return run<T, JOIN, V, 4, false>(a, s, st);
        if (s.K == 8) return run<T, JOIN, V, 8, false>(a, s, st);
        return run<T, JOIN, V / 2, 16, false>(a, s, st);
    }
    if (s.K == 1) return run<T, JOIN, 1, 1, false>(a, s, st);
    if (s.K == 2) return run<T, JOIN, 1, 2, false>(a, s, st);
    if (s.K == 4) return run<T, JOIN, 1, 4, false>(a, s, st);
    if (s.K == 8) return run<T, JOIN, 1, 8, false>(a, s, st);
    return run<T, JOIN, 1, 16, false>(a, s, st);
}

// ------------------------------------------------------------------ dropout
template <class T, int V>
__global__ __launch_bounds__(256) void k_dropout(const T* x, T* y, long long n, DropArgs d)
{
    const long long i = ((long long)blockIdx.x * 256 + threadIdx.x) * V;
    if (i >= n) return;
    const int nv = n - i >= V ? V : (int)(n - i);
    const Pack<T, V> r = load_pack<T, V>(x + i, nv);
    const unsigned keep = d.rng ? keep_bits<V>(d.rng[0], d.rng[1], d.thr, (unsigned long long)i, true) : ~0u;
    float f[V];
#pragma unroll
    for (int v = 0; v < V; ++v) f[v] = (keep >> v & 1u) ? r.get(v) * d.up : 0.0f;
    store_pack<T, V>(y + i, f, nv);
}

}  // namespace

hipError_t launch_block_fwd(const BlockArgs& a, hipStream_t st)
{
    if (a.m) return a.bf16 ? dispatch<__bf16, true>(a, st) : dispatch<float, true>(a, st);
    return a.bf16 ? dispatch<__bf16, false>(a, st) : dispatch<float, false>(a, st);
}

hipError_t launch_dropout(const void* x, void* y, long long n, bool bf16, const DropArgs& d, hipStream_t st)
{
    const int V = bf16 ? 8 : 4;
    const unsigned grid = (unsigned)((n + 256ll * V - 1) / (256ll * V));
    if (bf16) hipLaunchKernelGGL((k_dropout<__bf16, 8>), dim3(grid), dim3(256), 0, st, (const __bf16*)x, (__bf16*)y, n, d);
    else hipLaunchKernelGGL((k_dropout<float, 4>), dim3(grid), dim3(256), 0, st, (const float*)x, (float*)y, n, d);
    return launch_status();
}

}  // namespace hyenand
