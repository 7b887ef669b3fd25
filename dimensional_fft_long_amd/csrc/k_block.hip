// k_block.hip -- the norm ahead of a block, the join behind it (norm of the
// block's output, gate, residual scale, dropout, residual sum, the next norm)
// and dropout, forward and backward.
//
// One workgroup holds a tile of positions with ALL their channels in registers,
// so every tensor crosses HBM once: the sums over channels (the norms' mean
// squares and, backward, their products with the gradient) go through lane
// exchanges and LDS between the passes over the registers.  These operators do
// a few operations per byte; HBM traffic is what bounds them.
#include "block_dev.h"

namespace hyenand {
namespace {

constexpr int kNT = 512;     // threads of a workgroup, at most
constexpr int kMaxP = 256;   // positions of a tile, at most

// How a launch lays its threads over a tile.
struct Lay {
    int lxs;            // log2 of the lanes along positions
    long long tiles_b;  // tiles per batch entry
    long long tiles;
};

// Sum of N values per position over the channels of the workgroup.  Rows: one
// position, every lane holds channels.  Else lane t holds positions
// (t & (LX-1)) * V + v.  `red` has two halves used in turn, so one barrier per
// sum is enough: a half is written again only after the barrier of the sum in
// between.
template <int N, int V, bool ROW>
__device__ __forceinline__ void sum_channels(float (&s)[N][V], float* red, int& turn, int lxs)
{
    const int t = (int)threadIdx.x, nw = (int)blockDim.x >> 6, w = t >> 6;
    float* buf = red + turn * (2 * (kNT / 64) * kMaxP);
    turn ^= 1;
    if constexpr (ROW) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            float a = s[n][0];
#pragma unroll
            for (int v = 1; v < V; ++v) a += s[n][v];
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) a += __shfl_xor(a, o);
            if ((t & 63) == 0) buf[n * (kNT / 64) + w] = a;
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < N; ++n) {
            float a = 0.0f;
            for (int i = 0; i < nw; ++i) a += buf[n * (kNT / 64) + i];
#pragma unroll
            for (int v = 0; v < V; ++v) s[n][v] = a;
        }
    } else {
        const int LX = 1 << lxs, lane = t & 63, lx = t & (LX - 1), P = LX * V;
        for (int o = LX; o < 64; o <<= 1) {
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int v = 0; v < V; ++v) s[n][v] += __shfl_xor(s[n][v], o);
        }
        if (lane < LX) {
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int v = 0; v < V; ++v) buf[(n * nw + w) * P + v * LX + lx] = s[n][v];
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float a = 0.0f;
                for (int i = 0; i < nw; ++i) a += buf[(n * nw + i) * P + v * LX + lx];
                s[n][v] = a;
            }
    }
}

// Where a thread's k-th group of V elements lies: offset into the tensor,
// number of valid elements, and the channel of element v.
template <int V, bool ROW>
struct Where {
    long long base;
    int nv0, cy, step, C;
    long long L;
    __device__ Where(const BlockArgs& a, const Lay& g, long long tile)
    {
        const int t = (int)threadIdx.x;
        C = a.C;
        L = a.L;
        if constexpr (ROW) {
            base = tile * a.C;
            nv0 = 0;
            cy = t * V;
            step = (int)blockDim.x * V;
        } else {
            const int LX = 1 << g.lxs;
            const long long b = tile / g.tiles_b;
            const long long l0 = (tile - b * g.tiles_b) * (LX * V) + (t & (LX - 1)) * V;
            base = b * a.C * a.L + l0;
            const long long left = a.L - l0;
            nv0 = left >= V ? V : left > 0 ? (int)left : 0;
            cy = t >> g.lxs;
            step = (int)blockDim.x >> g.lxs;
        }
    }
    __device__ int chan(int k, int v) const { return ROW ? cy + k * step + v : cy + k * step; }
    __device__ long long off(int k) const
    {
        return ROW ? base + chan(k, 0) : base + (long long)chan(k, 0) * L;
    }
    __device__ int nv(int k) const
    {
        const int c = chan(k, 0);
        if constexpr (ROW) return c + V <= C ? V : c < C ? C - c : 0;
        return c < C ? nv0 : 0;
    }
};

// Channel parameter p[c] of element v of group k (dflt where p is null or the
// channel is past the end).
template <int V, bool ROW>
__device__ __forceinline__ float param(const float* p, const Where<V, ROW>& w, int k, int v, float dflt)
{
    const int c = w.chan(k, v);
    return p && c < w.C ? p[c] : dflt;
}

template <class T, bool JOIN, int V, int K, bool ROW>
__global__ __launch_bounds__(kNT) void k_block_fwd(BlockArgs a, Lay g)
{
    __shared__ float red[2 * 2 * (kNT / 64) * kMaxP];
    int turn = 0;
    const float invC = 1.0f / (float)a.C;
    unsigned long long seed = 0, offs = 0;
    if (JOIN && a.drop.rng) {
        seed = a.drop.rng[0];
        offs = a.drop.rng[1];
    }
    for (long long tile = blockIdx.x; tile < g.tiles; tile += gridDim.x) {
        const Where<V, ROW> w(a, g, tile);
        Pack<T, V> xr[K], mr[JOIN ? K : 1], gr[JOIN ? K : 1];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int nv = w.nv(k);
            const long long o = w.off(k);
            if (JOIN) mr[k] = load_pack<T, V>((const T*)a.m + o, nv);
            xr[k] = load_pack<T, V>((const T*)a.x + o, nv);
            if (JOIN && a.gate) gr[k] = load_pack<T, V>((const T*)a.gate + o, nv);
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
                for (int v = 0; v < V; ++v) rm[0][v] += mr[k].get(v) * mr[k].get(v);
            sum_channels<1, V, ROW>(rm, red, turn, g.lxs);
#pragma unroll
            for (int v = 0; v < V; ++v) rm[0][v] = rsqrtf(rm[0][v] * invC + a.eps);
        }
        float o[K][V], ro[1][V];
#pragma unroll
        for (int v = 0; v < V; ++v) ro[0][v] = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int nv = w.nv(k);
            unsigned keep = ~0u;
            if (JOIN && a.drop.rng && nv > 0) keep = keep_bits<V>(seed, offs, a.drop.thr, (unsigned long long)w.off(k));
            const float up = JOIN && a.drop.rng ? a.drop.up : 1.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float val = xr[k].get(v);
                if (JOIN) {
                    const float ga = a.gate ? act_fwd(a.act, gr[k].get(v)) : 1.0f;
                    const float n = mr[k].get(v) * rm[0][v] * param(a.w_post, w, k, v, 1.0f);
                    const float b = param(a.scale, w, k, v, 1.0f) * ga * n * up;
                    val = (keep >> v & 1u) ? val + b : val;
                }
                o[k][v] = val;
                ro[0][v] += v < nv ? val * val : 0.0f;
            }
            if (JOIN && nv > 0) store_pack<T, V>((T*)a.out + w.off(k), o[k], nv);
        }
        if (a.w_pre) {
            sum_channels<1, V, ROW>(ro, red, turn, g.lxs);
#pragma unroll
            for (int v = 0; v < V; ++v) ro[0][v] = rsqrtf(ro[0][v] * invC + a.eps);
#pragma unroll
            for (int k = 0; k < K; ++k) {
#pragma unroll
                for (int v = 0; v < V; ++v) o[k][v] *= ro[0][v] * param(a.w_pre, w, k, v, 0.0f);
                if (w.nv(k) > 0) store_pack<T, V>((T*)a.h + w.off(k), o[k], w.nv(k));
            }
        }
    }
}

// Backward.  With n = m r_m w_post, b = s a(gate) n up keep, out = x + b and
// h = out r_o w_pre:
//   do  = dout + r_o dn - out r_o^3 mean_c(dn out),  dn = dh w_pre
//   dx  = do,  db = do up keep,  dgate = db s n a'
//   e   = db s a,  dm = r_m e w_post - m r_m^3 mean_c(e w_post m)   (e without the post norm)
//   Q_c = sum db a m r_m: dscale = w_post Q, dw_post = s Q;  dw_pre = sum dh out r_o
// Both channel sums stay in registers over all of a workgroup's tiles and are
// joined in a fixed order by k_block_reduce.
template <class T, bool JOIN, int V, int K, bool ROW>
__global__ __launch_bounds__(kNT) void k_block_bwd(BlockArgs a, Lay g)
{
    __shared__ float red[2 * 2 * (kNT / 64) * kMaxP];
    int turn = 0;
    const float invC = 1.0f / (float)a.C;
    unsigned long long seed = 0, offs = 0;
    if (JOIN && a.drop.rng) {
        seed = a.drop.rng[0];
        offs = a.drop.rng[1];
    }
    const float up = JOIN && a.drop.rng ? a.drop.up : 1.0f;
    constexpr int VA = ROW ? V : 1;
    float Q[K][VA], S[K][VA];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int v = 0; v < VA; ++v) Q[k][v] = S[k][v] = 0.0f;
    for (long long tile = blockIdx.x; tile < g.tiles; tile += gridDim.x) {
        const Where<V, ROW> w(a, g, tile);
        Pack<T, V> xr[K], mr[JOIN ? K : 1], gr[JOIN ? K : 1], hr[K], dr[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int nv = w.nv(k);
            const long long o = w.off(k);
            if (JOIN) mr[k] = load_pack<T, V>((const T*)a.m + o, nv);
            xr[k] = load_pack<T, V>((const T*)a.x + o, nv);
            if (JOIN && a.gate) gr[k] = load_pack<T, V>((const T*)a.gate + o, nv);
            if (a.dh) hr[k] = load_pack<T, V>((const T*)a.dh + o, nv);
            if (a.dout) dr[k] = load_pack<T, V>((const T*)a.dout + o, nv);
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
                for (int v = 0; v < V; ++v) rm[0][v] += mr[k].get(v) * mr[k].get(v);
            sum_channels<1, V, ROW>(rm, red, turn, g.lxs);
#pragma unroll
            for (int v = 0; v < V; ++v) rm[0][v] = rsqrtf(rm[0][v] * invC + a.eps);
        }
        float o[K][V], s2[2][V];
        unsigned keep[K];
#pragma unroll
        for (int v = 0; v < V; ++v) s2[0][v] = s2[1][v] = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int nv = w.nv(k);
            keep[k] = ~0u;
            if (JOIN && a.drop.rng && nv > 0)
                keep[k] = keep_bits<V>(seed, offs, a.drop.thr, (unsigned long long)w.off(k));
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float val = xr[k].get(v);
                if (JOIN) {
                    const float ga = a.gate ? act_fwd(a.act, gr[k].get(v)) : 1.0f;
                    const float n = mr[k].get(v) * rm[0][v] * param(a.w_post, w, k, v, 1.0f);
                    const float b = param(a.scale, w, k, v, 1.0f) * ga * n * up;
                    val = (keep[k] >> v & 1u) ? val + b : val;
                }
                o[k][v] = val;
                if (a.dh && v < nv) {
                    s2[0][v] += val * val;
                    s2[1][v] += hr[k].get(v) * param(a.w_pre, w, k, v, 0.0f) * val;
                }
            }
        }
        float ro[V], co[V];
        if (a.dh) {
            sum_channels<2, V, ROW>(s2, red, turn, g.lxs);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                ro[v] = rsqrtf(s2[0][v] * invC + a.eps);
                co[v] = ro[v] * ro[v] * ro[v] * (s2[1][v] * invC);
            }
        }
        float e[JOIN ? K : 1][V], em[1][V];
#pragma unroll
        for (int v = 0; v < V; ++v) em[0][v] = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int nv = w.nv(k);
            float dx[V], dg[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float d = a.dout ? dr[k].get(v) : 0.0f;
                if (a.dh) {
                    const float dhv = hr[k].get(v);
                    d += ro[v] * dhv * param(a.w_pre, w, k, v, 0.0f) - o[k][v] * co[v];
                    if (v < nv) S[k][ROW ? v : 0] += dhv * o[k][v] * ro[v];
                }
                dx[v] = d;
                if (JOIN) {
                    float ga = 1.0f, da = 0.0f;
                    if (a.gate) act_both(a.act, gr[k].get(v), ga, da);
                    const float db = (keep[k] >> v & 1u) ? d * up : 0.0f;
                    const float mn = mr[k].get(v) * rm[0][v], wp = param(a.w_post, w, k, v, 1.0f);
                    const float sc = param(a.scale, w, k, v, 1.0f);
                    dg[v] = db * sc * (mn * wp) * da;
                    const float dba = db * ga;
                    if (v < nv) Q[k][ROW ? v : 0] += dba * mn;
                    e[k][v] = dba * sc * wp;
                    if (v < nv) em[0][v] += e[k][v] * mr[k].get(v);
                }
            }
            if (nv > 0) {
                store_pack<T, V>((T*)a.dx + w.off(k), dx, nv);
                if (JOIN && a.gate) store_pack<T, V>((T*)a.dgate + w.off(k), dg, nv);
            }
        }
        if (JOIN) {
            if (a.w_post) {
                sum_channels<1, V, ROW>(em, red, turn, g.lxs);
#pragma unroll
                for (int v = 0; v < V; ++v) em[0][v] *= rm[0][v] * rm[0][v] * rm[0][v] * invC;
            }
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (a.w_post) {
#pragma unroll
                    for (int v = 0; v < V; ++v) e[k][v] = e[k][v] * rm[0][v] - mr[k].get(v) * em[0][v];
                }
                if (w.nv(k) > 0) store_pack<T, V>((T*)a.dm + w.off(k), e[k], w.nv(k));
            }
        }
    }
    // Partial sums of this workgroup's tiles.
    float* part = a.part + (long long)blockIdx.x * 2 * a.C;
    const Where<V, ROW> w(a, g, 0);
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
        for (int v = 0; v < VA; ++v) {
            float q = Q[k][v], s = S[k][v];
            if constexpr (!ROW) {
                for (int of = 1; of < (1 << g.lxs); of <<= 1) {
                    q += __shfl_xor(q, of);
                    s += __shfl_xor(s, of);
                }
                if ((int)threadIdx.x & ((1 << g.lxs) - 1)) continue;
            }
            const int c = w.chan(k, v);
            if (c < a.C) {
                part[c] = q;
                part[a.C + c] = s;
            }
        }
    }
}

// Channel gradients from the workgroups' partial sums, in double and in a fixed
// order: 16 channels by 64 groups of workgroups.
__global__ __launch_bounds__(1024) void k_block_reduce(BlockArgs a, int parts)
{
    __shared__ double R[2][64][16];
    const int lc = (int)threadIdx.x & 15, gr = (int)threadIdx.x >> 4, c = (int)blockIdx.x * 16 + lc;
    double q = 0.0, s = 0.0;
    if (c < a.C)
        for (int p = gr; p < parts; p += 64) {
            const float* r = a.part + (long long)p * 2 * a.C;
            q += (double)r[c];
            s += (double)r[a.C + c];
        }
    R[0][gr][lc] = q;
    R[1][gr][lc] = s;
    __syncthreads();
    for (int h = 32; h > 0; h >>= 1) {
        if (gr < h) {
            R[0][gr][lc] += R[0][gr + h][lc];
            R[1][gr][lc] += R[1][gr + h][lc];
        }
        __syncthreads();
    }
    if (gr == 0 && c < a.C) {
        const double Q = R[0][0][lc];
        if (a.dscale) a.dscale[c] = (float)(a.w_post ? Q * (double)a.w_post[c] : Q);
        if (a.dw_post) a.dw_post[c] = (float)(a.scale ? Q * (double)a.scale[c] : Q);
        if (a.dw_pre) a.dw_pre[c] = (float)R[1][0][lc];
    }
}

// ------------------------------------------------------------------ dropout
template <class T, int V>
__global__ __launch_bounds__(256) void k_dropout(const T* x, T* y, long long n, DropArgs d)
{
    const long long i = ((long long)blockIdx.x * 256 + threadIdx.x) * V;
    if (i >= n) return;
    const int nv = n - i >= V ? V : (int)(n - i);
    const Pack<T, V> r = load_pack<T, V>(x + i, nv);
    const unsigned keep = d.rng ? keep_bits<V>(d.rng[0], d.rng[1], d.thr, (unsigned long long)i) : ~0u;
    float f[V];
#pragma unroll
    for (int v = 0; v < V; ++v) f[v] = (keep >> v & 1u) ? r.get(v) * d.up : 0.0f;
    store_pack<T, V>(y + i, f, nv);
}

// ------------------------------------------------------------------ dispatch
struct Shape {
    bool row;
    bool wide;   // 16 bytes along positions per lane (else one element)
    int K, nt;
    Lay g;
};

Shape pick(const BlockArgs& a)
{
    Shape s{};
    s.row = a.L == 1;
    const int full = a.bf16 ? 8 : 4;
    if (s.row) {
        s.wide = true;
        s.nt = 256;
        int K = (a.C + s.nt * full - 1) / (s.nt * full);
        if (K > 4) s.nt = 512, K = (a.C + s.nt * full - 1) / (s.nt * full);
        s.K = K <= 1 ? 1 : K <= 2 ? 2 : 4;
        s.g = Lay{0, 1, a.B};
        return s;
    }
    s.wide = a.L >= full;
    const int V = s.wide ? full : 1;
    s.nt = kNT;
    // Lanes along positions: as many as a tile may have while the channels still
    // fit K <= 8 groups per thread and there are tiles for the whole device.
    int lxs = 5;
    while (lxs > 0) {
        const long long tiles = a.B * ((a.L + (V << lxs) - 1) / (V << lxs));
        const int cy = s.nt >> lxs, K = (a.C + cy - 1) / cy;
        if (K <= 8 && tiles >= 512 && (K <= 1 || lxs <= 3)) break;
        --lxs;
    }
    const int cy = s.nt >> lxs, K = (a.C + cy - 1) / cy;
    s.K = K <= 1 ? 1 : K <= 2 ? 2 : K <= 4 ? 4 : K <= 8 ? 8 : 16;
    const long long tb = (a.L + (V << lxs) - 1) / (V << lxs);
    s.g = Lay{lxs, tb, tb * a.B};
    return s;
}

template <class T, bool JOIN, int V, int K, bool ROW>
hipError_t run(const BlockArgs& a, const Shape& s, bool bwd, hipStream_t st)
{
    const long long cap = bwd ? kBlockMaxParts : (1ll << 30);
    const unsigned grid = (unsigned)(s.g.tiles < cap ? s.g.tiles : cap);
    if (!bwd) {
        hipLaunchKernelGGL((k_block_fwd<T, JOIN, V, K, ROW>), dim3(grid), dim3(s.nt), 0, st, a, s.g);
        return launch_status();
    }
    hipLaunchKernelGGL((k_block_bwd<T, JOIN, V, K, ROW>), dim3(grid), dim3(s.nt), 0, st, a, s.g);
    hipError_t e = launch_status();
    if (e != hipSuccess || !(a.dscale || a.dw_post || a.dw_pre)) return e;
    hipLaunchKernelGGL(k_block_reduce, dim3((a.C + 15) / 16), dim3(1024), 0, st, a, (int)grid);
    return launch_status();
}

template <class T, bool JOIN>
hipError_t pick_and_run(const BlockArgs& a, bool bwd, hipStream_t st)
{
    const Shape s = pick(a);
    constexpr int V = 16 / (int)sizeof(T);
    if (s.row) {
        if (s.K == 1) return run<T, JOIN, V, 1, true>(a, s, bwd, st);
        if (s.K == 2) return run<T, JOIN, V, 2, true>(a, s, bwd, st);
        return run<T, JOIN, V, 4, true>(a, s, bwd, st);
    }
    if (s.wide) {
        if (s.K == 1) return run<T, JOIN, V, 1, false>(a, s, bwd, st);
        if (s.K == 2) return run<T, JOIN, V, 2, false>(a, s, bwd, st);
        if (s.K == 4) return run<T, JOIN, V, 4, false>(a, s, bwd, st);
        if (s.K == 8) return run<T, JOIN, V, 8, false>(a, s, bwd, st);
        // More than 4096 channels: twice the groups of half the width.
        Shape h = s;
        h.g.tiles_b = (a.L + V / 2 - 1) / (V / 2);
        h.g.tiles = h.g.tiles_b * a.B;
        return run<T, JOIN, V / 2, 16, false>(a, h, bwd, st);
    }
    if (s.K == 1) return run<T, JOIN, 1, 1, false>(a, s, bwd, st);
    if (s.K == 2) return run<T, JOIN, 1, 2, false>(a, s, bwd, st);
    if (s.K == 4) return run<T, JOIN, 1, 4, false>(a, s, bwd, st);
    if (s.K == 8) return run<T, JOIN, 1, 8, false>(a, s, bwd, st);
    return run<T, JOIN, 1, 16, false>(a, s, bwd, st);
}

hipError_t launch_block(const BlockArgs& a, bool bwd, hipStream_t st)
{
    if (a.m) return a.bf16 ? pick_and_run<__bf16, true>(a, bwd, st) : pick_and_run<float, true>(a, bwd, st);
    return a.bf16 ? pick_and_run<__bf16, false>(a, bwd, st) : pick_and_run<float, false>(a, bwd, st);
}

}  // namespace

hipError_t launch_block_fwd(const BlockArgs& a, hipStream_t st) { return launch_block(a, false, st); }
hipError_t launch_block_bwd(const BlockArgs& a, hipStream_t st) { return launch_block(a, true, st); }

hipError_t launch_dropout(const void* x, void* y, long long n, bool bf16, const DropArgs& d, hipStream_t st)
{
    const int V = bf16 ? 8 : 4;
    const unsigned grid = (unsigned)((n + 256ll * V - 1) / (256ll * V));
    if (bf16) hipLaunchKernelGGL((k_dropout<__bf16, 8>), dim3(grid), dim3(256), 0, st, (const __bf16*)x, (__bf16*)y, n, d);
    else hipLaunchKernelGGL((k_dropout<float, 4>), dim3(grid), dim3(256), 0, st, (const float*)x, (float*)y, n, d);
    return launch_status();
}

}  // namespace hyenand
