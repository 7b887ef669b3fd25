// k_block_bwd.hip -- the norm and the join, backward.
//
// Measured on one MI355X: norm of 2 x 1024 x 16384 bf16 (three tensors) 81 us,
// 2.5 TB/s; join of 2 x 128 x 1024^2 bf16 (eight tensors) 2.0 ms, 2.1 TB/s.  The
// join issues 133 vector instructions an element (46% of the issue slots) and
// its waves wait for 67% of their cycles: four waves a SIMD of 128 registers
// are what the five tensors leave, with three sums (each behind two barriers)
// a tile between the loads and the stores.
#include "block_tile.h"

namespace hyenand {
namespace {

constexpr int kCUs = 256;

// Backward.  With n = m r_m w_post, b = s a(gate) n up keep, out = x + b and
// h = out r_o w_pre:
//   do  = dout + r_o dn - out r_o^3 mean_c(dn out),  dn = dh w_pre
//   dx  = do,  db = do up keep,  dgate = db s n a'
//   e   = db s a,  dm = r_m e w_post - m r_m^3 mean_c(e w_post m)   (e without the post norm)
//   Q_c = sum db a m r_m: dscale = w_post Q, dw_post = s Q;  dw_pre = sum dh out r_o
// Both channel sums stay in registers over all of a workgroup's tiles and are
// joined in a fixed order by k_block_reduce.
template <class T, bool JOIN, int V, int K, bool ROW, int NT>
__global__ __launch_bounds__(NT, NT == 1024 ? 4 : V * K <= (JOIN ? 8 : 16) ? 4 : 2) void k_block_bwd(BlockArgs a, Lay g)
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
    const float up = drop ? a.drop.up : 1.0f;
    Params<V, K, ROW> sw, wpre;  // scale w_post, w_pre
    {
        const Where<V, ROW> w(a, g);  // channels only
        if (JOIN) {
            Params<V, K, ROW> sc;
            sw.load(a.w_post, w, 1.0f);
            sc.load(a.scale, w, 1.0f);
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < (ROW ? V : 1); ++i) sw.v[k][i] *= sc.v[k][i];
        }
        wpre.load(a.w_pre, w, 0.0f);
    }
    constexpr int VA = ROW ? V : 1;
    float Q[K][VA], S[K][VA];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int v = 0; v < VA; ++v) Q[k][v] = S[k][v] = 0.0f;
    Pack<T, V> xr[K], mr[JOIN ? K : 1], gr[JOIN ? K : 1], hr[K], dr[K];
    const auto load = [&](const Where<V, ROW>& at) __attribute__((always_inline)) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (JOIN) mr[k] = load_group<T, V, ROW>(a.m, at, k);
            if (a.dh) {
                xr[k] = load_group<T, V, ROW>(a.x, at, k);
                hr[k] = load_group<T, V, ROW>(a.dh, at, k);
            }
            if (JOIN && a.gate) gr[k] = load_group<T, V, ROW>(a.gate, at, k);
        }
    };
    // The norm asks for the next tile's tensors ahead of this tile's stores (89 ->
    // 81 us at 2 x 1024 x 16384 bf16; nothing gained for the join's five tensors).
    constexpr bool AHEAD = !JOIN;
    const Run tiles(g);
    Where<V, ROW> w(a, g), wn(a, g);
    if (AHEAD && tiles.first < tiles.end) {
        w.at(a, g, tiles.first);
        load(w);
    }
    for (long long tile = tiles.first; tile < tiles.end; tile += tiles.step) {
        const bool more = AHEAD && tile + tiles.step < tiles.end;
        if (more) wn.at(a, g, tile + tiles.step);
        if (!AHEAD) {
            w.at(a, g, tile);
            load(w);
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
        with_gate(JOIN && a.gate, a.act, [&](auto act) __attribute__((always_inline)) {
            // out of element (k, v), computed where it is needed.
            const auto out_at = [&](int k, int v) __attribute__((always_inline)) {
                float val = xr[k].get(v);
                if constexpr (JOIN) {
                    const float b = sw.at(k, v) * act_fwd(act, gr[k].get(v)) * (mr[k].get(v) * rm[0][v]) * up;
                    val += kept(keep[k], v, b);
                }
                return val;
            };
            // 0 for the positions that another lane counts, else 1.
            float once[V];
#pragma unroll
            for (int v = 0; v < V; ++v) once[v] = ROW || v >= w.skip ? 1.0f : 0.0f;
            float s2[2][V], ro[V], co[V];
            if (a.dh) {
#pragma unroll
                for (int v = 0; v < V; ++v) s2[0][v] = s2[1][v] = 0.0f;
#pragma unroll
                for (int k = 0; k < K; ++k) {
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        const float val = out_at(k, v);
                        if (!ROW || w.mine(k, v)) {
                            s2[0][v] += val * val;
                            s2[1][v] += hr[k].get(v) * wpre.at(k, v) * val;
                        }
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (a.dout) dr[k] = load_group<T, V, ROW>(a.dout, w, k);
                else dr[k] = Pack<T, V>{};
            }
            if (a.dh) {
                sum_channels<2, V, ROW, NT>(s2, red, turn, g.lxs);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    ro[v] = __builtin_amdgcn_rsqf(s2[0][v] * invC + a.eps);
                    co[v] = ro[v] * ro[v] * ro[v] * (s2[1][v] * invC);
                }
            }
            float ev[JOIN ? K : 1][V], em[1][V];  // e w_post
#pragma unroll
            for (int v = 0; v < V; ++v) em[0][v] = 0.0f;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                float dv[V], dg[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    dv[v] = dr[k].get(v);
                    if (a.dh) {
                        const float dhr = hr[k].get(v) * ro[v], val = out_at(k, v);
                        dv[v] += dhr * wpre.at(k, v) - val * co[v];
                        S[k][ROW ? v : 0] += dhr * val * once[v];
                    }
                }
                store_group<T, V, ROW>(a.dx, w, k, dv);
                if constexpr (JOIN) {
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        float ga, da;
                        act_both(act, gr[k].get(v), ga, da);
                        const float db = kept(keep[k], v, dv[v] * up);
                        const float mn = mr[k].get(v) * rm[0][v], dbs = db * sw.at(k, v);
                        dg[v] = dbs * mn * da;
                        ev[k][v] = dbs * ga;
                        Q[k][ROW ? v : 0] += db * ga * mn * once[v];
                        if (!ROW || w.mine(k, v)) em[0][v] += ev[k][v] * mr[k].get(v);
                    }
                    if (act != kActOne) store_group<T, V, ROW>(a.dgate, w, k, dg);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            if (more) load(wn);
            if constexpr (JOIN) {
                if (a.w_post) {
                    sum_channels<1, V, ROW, NT>(em, red, turn, g.lxs);
#pragma unroll
                    for (int v = 0; v < V; ++v) em[0][v] *= rm[0][v] * rm[0][v] * rm[0][v] * invC;
                }
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    if (a.w_post) {
#pragma unroll
                        for (int v = 0; v < V; ++v) ev[k][v] = ev[k][v] * rm[0][v] - mr[k].get(v) * em[0][v];
                    }
                    store_group<T, V, ROW>(a.dm, w, k, ev[k]);
                }
            }
        });
        if (AHEAD) w = wn;
    }
    // Partial sums of this workgroup's tiles.
    float* part = a.part + (long long)blockIdx.x * 2 * a.C;
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
            if (w.cy + k * w.step < a.C) {
                part[w.chan(k, v)] = q;
                part[a.C + w.chan(k, v)] = s;
            }
        }
    }
}

// The join's backward with its tensors staged in LDS, for tiles whose channels
// would take more than two groups a thread of the kernel above (more than about
// 256 channels): five tensors of so many groups leave too few registers, and
// narrower rows too little bandwidth.  What a thread reads of m, the gate, x and
// dh (16 bytes a group of channels each) lies in its own part of LDS, 32 KB a
// group and workgroup, and only the group at work is in registers.  Where rows
// are whole 16-byte pieces (DMA) the loads go straight to LDS, and a group's
// next tile is asked for as soon as this tile no longer needs it; else they pass
// through registers, a tile at a time.  No barrier guards the stage: every lane
// reads back its own wave's loads alone.  Measured against the kernel above, bf16: 717
// channels by 131072 positions 1180 -> 576 us, 260 by 131072 552 -> 248, 283 by
// 20074 (no DMA) 150 -> 72; fp32: 1000 by 131072 1876 -> 1297 us.  Up to 128
// channels, two groups, the two are level (2 x 128 x 1024^2 bf16: 1.97 against
// 2.0 ms) or this one behind (3 x 100 x 37 x 53: 24 against 17 us).
constexpr int kStageP = 64;  // positions of a staged tile, at most
template <class T>
constexpr int V_of = 16 / (int)sizeof(T);

template <class T, int K, bool DMA>
__global__ __launch_bounds__(512, V_of<T> * K <= 8 ? 4 : 2) void k_join_bwd_staged(BlockArgs a, Lay g)
{
    constexpr int V = V_of<T>, NT = 512;
    typedef Where<V, false> W;
    __shared__ __align__(16) char stage[K * 4 * NT * 16];
    __shared__ __align__(16) float red[2 * red_floats(NT, kStageP)];
    int turn = 0;
    const int t = (int)threadIdx.x;
    constexpr int qg = 1, qx = 2, qh = 3, ns = 4;
    const unsigned wave0 = lds_address(stage) + __builtin_amdgcn_readfirstlane(t >> 6) * 1024;
    const float invC = 1.0f / (float)a.C;
    unsigned long long seed = 0, offs = 0;
    const bool drop = a.drop.rng;
    if (drop) {
        seed = a.drop.rng[0];
        offs = a.drop.rng[1];
    }
    const float up = drop ? a.drop.up : 1.0f;
    W w(a, g), wn(a, g);
    Params<V, K, false> sw, wpre;  // scale w_post, w_pre
    {
        Params<V, K, false> sc;
        sw.load(a.w_post, w, 1.0f);
        sc.load(a.scale, w, 1.0f);
#pragma unroll
        for (int k = 0; k < K; ++k) sw.v[k][0] *= sc.v[k][0];
        wpre.load(a.w_pre, w, 0.0f);
    }
    float Q[K], S[K];
#pragma unroll
    for (int k = 0; k < K; ++k) Q[k] = S[k] = 0.0f;
    const auto fetch = [&](int q, const void* p, const W& at, int k) __attribute__((always_inline)) {
        to_lds((const T*)p + at.off(k), wave0 + (k * ns + q) * (NT * 16));
    };
    const auto keep_group = [&](int q, int k, const Pack<T, V>& v) __attribute__((always_inline)) {
        *reinterpret_cast<u32x4*>(stage + (k * ns + q) * (NT * 16) + t * 16) = u32x4{v.w[0], v.w[1], v.w[2], v.w[3]};
    };
    const auto group = [&](int q, int k) __attribute__((always_inline)) {
        const u32x4 v = *reinterpret_cast<const u32x4*>(stage + (k * ns + q) * (NT * 16) + t * 16);
        Pack<T, V> r{{v[0], v[1], v[2], v[3]}};
        if (!w.all_live(k) && w.cy + k * w.step >= w.C) r = Pack<T, V>{};
        return r;
    };
    const auto fetch_rest = [&](const W& at, int k) __attribute__((always_inline)) {
        if (a.gate) fetch(qg, a.gate, at, k);
        if (a.dh) {
            fetch(qx, a.x, at, k);
            fetch(qh, a.dh, at, k);
        }
    };
    const Run tiles(g);
    if (DMA && tiles.first < tiles.end) {
        w.at(a, g, tiles.first);
#pragma unroll
        for (int k = 0; k < K; ++k) fetch(0, a.m, w, k);
#pragma unroll
        for (int k = 0; k < K; ++k) fetch_rest(w, k);
    }
    for (long long tile = tiles.first; tile < tiles.end; tile += tiles.step) {
        const bool more = DMA && tile + tiles.step < tiles.end;
        w.at(a, g, tile);
        if (more) wn.at(a, g, tile + tiles.step);
        if constexpr (!DMA) {
            // Two groups' loads in flight a thread.
#pragma unroll
            for (int k0 = 0; k0 < K; k0 += 2) {
                Pack<T, V> raw[2][4];
#pragma unroll
                for (int k = k0; k < k0 + 2 && k < K; ++k) {
                    raw[k - k0][0] = load_group<T, V, false>(a.m, w, k);
                    if (a.gate) raw[k - k0][1] = load_group<T, V, false>(a.gate, w, k);
                    if (a.dh) {
                        raw[k - k0][2] = load_group<T, V, false>(a.x, w, k);
                        raw[k - k0][3] = load_group<T, V, false>(a.dh, w, k);
                    }
                }
#pragma unroll
                for (int k = k0; k < k0 + 2 && k < K; ++k) {
                    keep_group(0, k, raw[k - k0][0]);
                    if (a.gate) keep_group(qg, k, raw[k - k0][1]);
                    if (a.dh) {
                        keep_group(qx, k, raw[k - k0][2]);
                        keep_group(qh, k, raw[k - k0][3]);
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        // Dropout's words (with DMA while the loads are in flight).
        unsigned keep[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            keep[k] = ~0u;
            if (drop) keep[k] = keep_bits<V>(seed, offs, a.drop.thr, (unsigned long long)w.off(k), g.whole4);
        }
        if constexpr (DMA) wait_loads();
        float rm[1][V];
#pragma unroll
        for (int v = 0; v < V; ++v) rm[0][v] = a.w_post ? 0.0f : 1.0f;
        if (a.w_post) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const Pack<T, V> m = group(0, k);
#pragma unroll
                for (int v = 0; v < V; ++v) rm[0][v] += m.get(v) * m.get(v);
            }
            sum_channels<1, V, false, NT, kStageP>(rm, red, turn, g.lxs);
#pragma unroll
            for (int v = 0; v < V; ++v) rm[0][v] = __builtin_amdgcn_rsqf(rm[0][v] * invC + a.eps);
        }
        with_gate(a.gate != nullptr, a.act, [&](auto act) __attribute__((always_inline)) {
            const auto rest = [&](int q, int k) __attribute__((always_inline)) { return act == kActOne ? Pack<T, V>{} : group(q, k); };
            const auto out_at = [&](const Pack<T, V>& m, const Pack<T, V>& x, int k, int v, float ga) __attribute__((always_inline)) {
                return x.get(v) + kept(keep[k], v, sw.at(k, v) * ga * (m.get(v) * rm[0][v]) * up);
            };
            // 0 for the positions that another lane counts, else 1.
            float once[V];
#pragma unroll
            for (int v = 0; v < V; ++v) once[v] = v >= w.skip ? 1.0f : 0.0f;
            Pack<T, V> dr[K];
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (a.dout) dr[k] = load_group<T, V, false>(a.dout, w, k);
                else dr[k] = Pack<T, V>{};
            }
            float s2[2][V];
            if (a.dh) {
#pragma unroll
                for (int v = 0; v < V; ++v) s2[0][v] = s2[1][v] = 0.0f;
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const Pack<T, V> m = group(0, k), gt = rest(qg, k), x = group(qx, k), h = group(qh, k);
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        const float val = out_at(m, x, k, v, act_fwd(act, gt.get(v)));
                        s2[0][v] += val * val;
                        s2[1][v] += h.get(v) * wpre.at(k, v) * val;
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
                sum_channels<2, V, false, NT, kStageP>(s2, red, turn, g.lxs);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float ro = __builtin_amdgcn_rsqf(s2[0][v] * invC + a.eps);
                    s2[1][v] = ro * ro * ro * (s2[1][v] * invC);
                    s2[0][v] = ro;
                }
            }
            // dout is complete ahead of the next tile's loads, which the compiler's
            // waits do not count: it would wait for them too.
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < Pack<T, V>::N; ++i) asm volatile("" : "+v"(dr[k].w[i]));
            float ev[K][V], em[1][V];  // e w_post
#pragma unroll
            for (int v = 0; v < V; ++v) em[0][v] = 0.0f;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                float dv[V], dg[V];
                const Pack<T, V> m = group(0, k), gt = rest(qg, k);
                Pack<T, V> x{}, h{};
                if (a.dh) {
                    x = group(qx, k);
                    h = group(qh, k);
                }
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float ga, da;
                    act_both(act, gt.get(v), ga, da);
                    dv[v] = dr[k].get(v);
                    if (a.dh) {
                        const float dhr = h.get(v) * s2[0][v], val = out_at(m, x, k, v, ga);
                        dv[v] += dhr * wpre.at(k, v) - val * s2[1][v];
                        S[k] += dhr * val * once[v];
                    }
                    const float db = kept(keep[k], v, dv[v] * up);
                    const float mn = m.get(v) * rm[0][v], dbs = db * sw.at(k, v);
                    dg[v] = dbs * mn * da;
                    ev[k][v] = dbs * ga;
                    Q[k] += db * ga * mn * once[v];
                    em[0][v] += ev[k][v] * m.get(v);
                }
                store_group<T, V, false>(a.dx, w, k, dv);
                if (act != kActOne) store_group<T, V, false>(a.dgate, w, k, dg);
                if (more) {
                    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // this group's reads are done
                    fetch_rest(wn, k);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            if (a.w_post) {
                sum_channels<1, V, false, NT, kStageP>(em, red, turn, g.lxs);
#pragma unroll
                for (int v = 0; v < V; ++v) em[0][v] *= rm[0][v] * rm[0][v] * rm[0][v] * invC;
            }
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (a.w_post) {
                    const Pack<T, V> m = group(0, k);
#pragma unroll
                    for (int v = 0; v < V; ++v) ev[k][v] = ev[k][v] * rm[0][v] - m.get(v) * em[0][v];
                }
                store_group<T, V, false>(a.dm, w, k, ev[k]);
                if (more) {
                    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                    fetch(0, a.m, wn, k);
                }
            }
        });
    }
    float* part = a.part + (long long)blockIdx.x * 2 * a.C;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        float q = Q[k], s = S[k];
        for (int of = 1; of < (1 << g.lxs); of <<= 1) {
            q += __shfl_xor(q, of);
            s += __shfl_xor(s, of);
        }
        if (((int)threadIdx.x & ((1 << g.lxs) - 1)) == 0 && w.cy + k * w.step < a.C) {
            part[w.chan(k, 0)] = q;
            part[a.C + w.chan(k, 0)] = s;
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
#pragma unroll 8
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

template <class T, bool JOIN, int V, int K, bool ROW, int NT>
hipError_t run(const BlockArgs& a, const Shape& s, hipStream_t st)
{
    const unsigned grid = (unsigned)(s.g.tiles < block_parts(a.C) ? s.g.tiles : block_parts(a.C));
    hipLaunchKernelGGL((k_block_bwd<T, JOIN, V, K, ROW, NT>), dim3(grid), dim3(s.nt), 0, st, a, s.g);
    const hipError_t e = launch_status();
    if (e != hipSuccess || !(a.dscale || a.dw_post || a.dw_pre)) return e;
    hipLaunchKernelGGL(k_block_reduce, dim3((a.C + 15) / 16), dim3(1024), 0, st, a, (int)grid);
    return launch_status();
}

template <class T, int K>
hipError_t run_staged(const BlockArgs& a, const Shape& s, hipStream_t st)
{
    const long long most = kCUs * (V_of<T> * K <= 8 ? 2 : 1);  // what the device holds at once
    const unsigned grid = (unsigned)(s.g.tiles < most ? s.g.tiles : most);
    const auto whole = [](const void* p) { return (uintptr_t)p % 16 == 0; };
    const bool dma = a.L % V_of<T> == 0 && whole(a.x) && whole(a.m) && whole(a.gate) && whole(a.dh);
    if (dma) hipLaunchKernelGGL((k_join_bwd_staged<T, K, true>), dim3(grid), dim3(512), 0, st, a, s.g);
    else hipLaunchKernelGGL((k_join_bwd_staged<T, K, false>), dim3(grid), dim3(512), 0, st, a, s.g);
    const hipError_t e = launch_status();
    if (e != hipSuccess || !(a.dscale || a.dw_post || a.dw_pre)) return e;
    hipLaunchKernelGGL(k_block_reduce, dim3((a.C + 15) / 16), dim3(1024), 0, st, a, (int)grid);
    return launch_status();
}

template <class T, bool JOIN>
hipError_t dispatch(const BlockArgs& a, hipStream_t st)
{
    // The join holds five tensors: four elements a lane keep two groups of
    // channels within 128 registers (bf16; eight elements a lane spill).  Workgroups
    // of 1024 threads give rows of 128 bytes at 128 channels where there are many
    // tiles (2.01 against 2.13 ms at 2 x 128 x 1024^2), of 512 threads twice the
    // tiles where there are few (17 against 24 us at 3 x 100 x 37 x 53).  More groups
    // than two go through LDS where that holds them (up to 2048 channels).
    constexpr int F = 16 / (int)sizeof(T), V = JOIN ? 4 : F;
    Shape s = JOIN ? pick(a, V, 1024, 2, 4) : pick(a, V, 512, 4, 8);
    if (JOIN && !s.row && s.V > 1 && s.nt == 1024 && s.g.tiles < 2048 && a.C <= 2048) s = pick(a, V, 512, 2, 4);
    if constexpr (JOIN) {
        if (!s.row && s.V > 1 && s.K > 2) {
            const Shape q = pick(a, F, 512, 2, 4, kStageP);
            const int step = 512 >> q.g.lxs, K = (a.C + step - 1) / step;
            if (q.V == F && K <= 2) return run_staged<T, 2>(a, q, st);
            if (q.V == F && K == 3) return run_staged<T, 3>(a, q, st);
            if (q.V == F && K == 4) return run_staged<T, 4>(a, q, st);
        }
    }
    if (s.row) {
        if (s.K == 1) return run<T, JOIN, F, 1, true, 512>(a, s, st);
        if (s.K == 2) return run<T, JOIN, F, 2, true, 512>(a, s, st);
        return run<T, JOIN, F, 4, true, 512>(a, s, st);
    }
    if (s.V > 1) {
        if (s.nt == 64) return run<T, JOIN, V, 1, false, 64>(a, s, st);
        if (s.nt == 128) return run<T, JOIN, V, 1, false, 128>(a, s, st);
        if (s.nt == 256) return run<T, JOIN, V, 1, false, 256>(a, s, st);
        if constexpr (JOIN) {
            if (s.nt == 1024) {
                if (s.K == 1) return run<T, JOIN, V, 1, false, 1024>(a, s, st);
                if (s.K == 2) return run<T, JOIN, V, 2, false, 1024>(a, s, st);
                if (s.K == 4) return run<T, JOIN, V, 4, false, 1024>(a, s, st);
                return run<T, JOIN, V, 8, false, 1024>(a, s, st);  // 8192 channels at most
            }
            if (s.K == 1) return run<T, JOIN, V, 1, false, 512>(a, s, st);
            if (s.K == 2) return run<T, JOIN, V, 2, false, 512>(a, s, st);
            return run<T, JOIN, V, 4, false, 512>(a, s, st);  // 2048 channels at most
        } else {
            if (s.K == 1) return run<T, JOIN, V, 1, false, 512>(a, s, st);
            if (s.K == 2) return run<T, JOIN, V, 2, false, 512>(a, s, st);
            if (s.K == 4) return run<T, JOIN, V, 4, false, 512>(a, s, st);
            if (s.K == 8) return run<T, JOIN, V, 8, false, 512>(a, s, st);
            return run<T, JOIN, V / 2, 16, false, 512>(a, s, st);
        }
    }
    if (s.K == 1) return run<T, JOIN, 1, 1, false, 512>(a, s, st);
    if (s.K == 2) return run<T, JOIN, 1, 2, false, 512>(a, s, st);
    if (s.K == 4) return run<T, JOIN, 1, 4, false, 512>(a, s, st);
    if (s.K == 8) return run<T, JOIN, 1, 8, false, 512>(a, s, st);
    return run<T, JOIN, 1, 16, false, 512>(a, s, st);
}

}  // namespace

hipError_t launch_block_bwd(const BlockArgs& a, hipStream_t st)
{
    if (a.m) return a.bf16 ? dispatch<__bf16, true>(a, st) : dispatch<float, true>(a, st);
    return a.bf16 ? dispatch<__bf16, false>(a, st) : dispatch<float, false>(a, st);
}

}  // namespace hyenand
