// block_tile.h -- what the norm's and the join's kernels share: a workgroup's
// tile of positions with all their channels, and the sums over channels.
//
// One workgroup holds a tile of positions with ALL their channels in registers,
// so every tensor crosses HBM once: the sums over channels (the norms' mean
// squares and, backward, their products with the gradient) go through lane
// exchanges and LDS between the passes over the registers.  These operators do
// a few operations per byte; HBM traffic bounds them, and, backward, how many
// bytes a CU keeps in flight next to the values that it holds.
#pragma once

#include "block_dev.h"

namespace hyenand {
namespace {

constexpr int kMaxP = 256;  // positions of a tile, at most
// Floats of a sum over a workgroup's waves: every wave's values and the joined ones.
constexpr int red_floats(int NT, int P = kMaxP) { return (NT / 64 + 1) * 2 * P; }

// How a launch lays its threads over a tile.
struct Lay {
    int lxs;            // log2 of the lanes along positions
    long long tiles_b;  // tiles per batch entry
    long long tiles;
    bool whole4;        // rows (of positions, or of channels) are multiples of four elements
    bool runs;          // a contiguous run of tiles for each XCD
};

// The tiles of a workgroup: every gridDim-th one, or, where a tile's rows are
// shorter than the 128-byte lines (`runs`), from a contiguous run for each XCD
// (workgroups are dealt to the eight XCDs in turn), so that neighbours, which
// share lines, share an L2: norm of 2 x 1024 x 16384 bf16, 64-byte rows, 35 ->
// 27 us forward, 97 -> 90 us backward.  Rows of whole lines are faster dealt
// singly (142 against 149 us for the join of 8 x 64 x 256^2 fp32).
struct Run {
    long long first, end, step;
    __device__ __forceinline__ Run(const Lay& g)
    {
        const unsigned x = blockIdx.x & 7u, n = gridDim.x;
        first = blockIdx.x;
        end = g.tiles;
        step = n;
        if (g.runs && n >= 64) {
            const long long lo = g.tiles * x / 8;
            end = g.tiles * (x + 1) / 8;
            first = lo + (blockIdx.x >> 3);
            step = (n >> 3) + (x < (n & 7u) ? 1 : 0);
        }
    }
};

__device__ __forceinline__ float from_bits(unsigned u) { return __builtin_bit_cast(float, u); }

template <int CTRL>
__device__ __forceinline__ float add_rotated(float a)
{
    return a + from_bits((unsigned)__builtin_amdgcn_update_dpp(0, (int)bits_of(a), CTRL, 0xf, 0xf, false));
}

// Sum over the lanes that agree in their lowest bits (lane % 2^lxs), in all of
// them.  Rotations inside a row of 16 lanes, then exchanges of rows and halves:
// vector instructions alone.  Both partners add the same two values, so every
// lane of a sum holds the same bits.
__device__ __forceinline__ float sum_lanes(float a, int lxs)
{
    if (lxs <= 3) a = add_rotated<0x128>(a);  // by 8
    if (lxs <= 2) a = add_rotated<0x124>(a);  // by 4
    if (lxs <= 1) a = add_rotated<0x122>(a);  // by 2
    if (lxs <= 0) a = add_rotated<0x121>(a);  // by 1
    if (lxs <= 4) {
        const auto r = __builtin_amdgcn_permlane16_swap(bits_of(a), bits_of(a), false, false);
        a = from_bits(r[0]) + from_bits(r[1]);
    }
    if (lxs <= 5) {
        const auto r = __builtin_amdgcn_permlane32_swap(bits_of(a), bits_of(a), false, false);
        a = from_bits(r[0]) + from_bits(r[1]);
    }
    return a;
}

// Sum of N values per position over the channels of the workgroup.  Rows: one
// position, every lane holds channels.  Else lane t holds positions
// (t & (LX-1)) * V + v: each wave's sums go to LDS, one thread per value joins
// the waves in order, and everyone reads the joined values.  `red` has two
// parts used in turn: a part is written again only behind the barriers of the
// sum in between.
template <int N, int V, bool ROW, int NT, int MP = kMaxP>
__device__ __forceinline__ void sum_channels(float (&s)[N][V], float* red, int& turn, int lxs)
{
    const int t = (int)threadIdx.x, nw = (int)blockDim.x >> 6, w = t >> 6, lane = t & 63;
    float* buf = red + turn * red_floats(NT, MP);
    turn ^= 1;
    if constexpr (ROW) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            float a = s[n][0];
#pragma unroll
            for (int v = 1; v < V; ++v) a += s[n][v];
            a = sum_lanes(a, 0);
            if (lane == 0) buf[n * (NT / 64) + w] = a;
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < N; ++n) {
            float a = 0.0f;
            for (int i = 0; i < nw; ++i) a += buf[n * (NT / 64) + i];
#pragma unroll
            for (int v = 0; v < V; ++v) s[n][v] = a;
        }
    } else {
        const int LX = 1 << lxs, lx = t & (LX - 1), P = LX * V;
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int v = 0; v < V; ++v) s[n][v] = sum_lanes(s[n][v], lxs);
        if constexpr (NT == 64) return;
        if (lane < LX) {
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int v = 0; v < V; ++v) buf[(w * N + n) * P + lx * V + v] = s[n][v];
        }
        __syncthreads();
        float* tot = buf + NT / 64 * 2 * MP;
        for (int e = t; e < N * P; e += (int)blockDim.x) {
            float a = 0.0f;
            for (int i = 0; i < nw; ++i) a += buf[i * N * P + e];
            tot[e] = a;
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int v = 0; v < V; ++v) s[n][v] = tot[n * P + lx * V + v];
    }
}

// Where a thread's k-th group of V elements lies.  Every access is a whole
// group: one that would leave its row (of positions, or of channels with ROW)
// is moved back to the row's last V elements, and the elements that another
// lane holds too stay out of the sums that they would enter twice (both lanes
// store the same values).  Groups past the last channel read another channel of
// their thread and count as zeros.
template <int V, bool ROW>
struct Where {
    long long lane;   // this thread's part of the offsets, the same for every tile
    long long tile;   // the tile's part, the same for every thread
    long long kstep;  // from group to group
    int l0, skip, cy, step, C;
    __device__ __forceinline__ Where(const BlockArgs& a, const Lay& g)
    {
        const int t = (int)threadIdx.x;
        C = a.C;
        tile = lane = 0;
        skip = l0 = 0;
        if constexpr (ROW) {
            cy = t * V;
            step = (int)blockDim.x * V;
            kstep = step;
        } else {
            cy = t >> g.lxs;
            step = (int)blockDim.x >> g.lxs;
            kstep = step * a.L;
            l0 = (t & ((1 << g.lxs) - 1)) * V;
        }
    }
    __device__ __forceinline__ void at(const BlockArgs& a, const Lay& g, long long i)
    {
        if constexpr (ROW) {
            tile = i * a.C;
        } else {
            const long long b = g.tiles < (1ll << 31) ? (unsigned)i / (unsigned)g.tiles_b : i / g.tiles_b;
            const long long start = (i - b * g.tiles_b) * (long long)(V << g.lxs);
            tile = b * a.C * a.L + start;
            const long long over = start + l0 + V - a.L;  // elements past the row's end
            skip = over > 0 ? (int)(over < V ? over : V) : 0;
            lane = (cy < C ? cy : C - 1) * a.L + l0 - (over > 0 ? over : 0);
            // Not to be added to the groups' steps ahead of the loop over the tiles:
            // that would hold an address for every group.
            asm volatile("" : "+v"(lane));
        }
    }
    __device__ __forceinline__ bool live(int k) const { return cy + k * step < C && skip < V; }
    __device__ __forceinline__ bool all_live(int k) const { return (ROW ? (int)blockDim.x * V : step) * (k + 1) <= C; }
    __device__ __forceinline__ int chan(int k, int v) const
    {
        const int c = cy + k * step;
        return ROW ? (c + V <= C ? c : C - V) + v : c;
    }
    __device__ __forceinline__ long long off(int k) const
    {
        if constexpr (ROW) return tile + chan(k, 0);
        return lane + (tile + (all_live(k) || cy + k * step < C ? k * kstep : 0));
    }
    // ROW: whether element v of group k is this lane's to count.
    __device__ __forceinline__ bool mine(int k, int v) const
    {
        const int c = cy + k * step;
        return c + V <= C || (c < C && v >= c + V - C);
    }
};

// f where bit v of keep is set, else 0, whatever f holds.
__device__ __forceinline__ float kept(unsigned keep, int v, float f)
{
    return __builtin_bit_cast(float, __builtin_bit_cast(unsigned, f) & (unsigned)((int)(keep << (31 - v)) >> 31));
}

template <class T, int V, bool ROW>
__device__ __forceinline__ Pack<T, V> load_group(const void* p, const Where<V, ROW>& w, int k)
{
    Pack<T, V> r = load_pack<T, V>((const T*)p + w.off(k), V);
    if constexpr (!ROW) {
        if (!w.all_live(k) && w.cy + k * w.step >= w.C) r = Pack<T, V>{};
    }
    return r;
}

template <class T, int V, bool ROW>
__device__ __forceinline__ void store_group(void* p, const Where<V, ROW>& w, int k, const float (&f)[V])
{
    if (w.live(k)) store_pack<T, V>((T*)p + w.off(k), f, V);
}

// Channel parameters of a thread's groups, the same for every tile: p[c], or
// dflt where p is null (and for channels past the end, which are not stored).
template <int V, int K, bool ROW>
struct Params {
    float v[K][ROW ? V : 1];
    __device__ __forceinline__ void load(const float* p, const Where<V, ROW>& w, float dflt)
    {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < (ROW ? V : 1); ++i) v[k][i] = p && w.cy + k * w.step < w.C ? p[w.chan(k, i)] : dflt;
    }
    __device__ __forceinline__ float at(int k, int i) const { return v[k][ROW ? i : 0]; }
};

// How a launch is cut: V elements along positions per lane (rows: along
// channels), K groups per thread, nt threads.
struct Shape {
    bool row;
    int V, K, nt;
    Lay g;
};

inline long long tile_count(const BlockArgs& a, int V, int lxs)
{
    return a.B * ((a.L + (V << lxs) - 1) / (V << lxs));
}

// Lanes along positions: the widest rows (DRAM and the address translation work
// on long runs: 128 to 512 bytes measured 1.2 to 4 times the rate of 32) whose
// channels fit `good` groups per thread, while there are tiles for the whole
// device; short rows take up to `most` groups, where a few spilled registers
// cost less than the row's length gives.  Few channels take workgroups of fewer
// waves, so that every row of threads has one (norm of 8 x 1 x 6.6 million bf16
// 577 -> 73 us, join of 7 x 2 x 9.2 million fp32 1638 -> 575).  A single
// position per batch entry is a row of channels.
inline Shape pick(const BlockArgs& a, int V, int nt, int good, int most, int maxp = kMaxP)
{
    const int es = a.bf16 ? 2 : 4, full = 16 / es;
    Shape s{};
    if (a.L == 1 && a.C >= full) {
        s.row = true;
        s.V = full;
        s.nt = a.C <= 1024 * full ? 256 : 512;
        const int K = (a.C + s.nt * full - 1) / (s.nt * full);
        s.K = K <= 1 ? 1 : K <= 2 ? 2 : 4;
        s.g = Lay{0, 1, a.B, a.C % 4 == 0, false};
        return s;
    }
    s.V = a.L >= V ? V : 1;
    s.nt = s.V > 1 ? nt : 512;
    const auto groups = [&](int lxs) { return (a.C + (s.nt >> lxs) - 1) / (s.nt >> lxs); };
    int top = 6;
    while (s.V > 1 && (s.V << top) > maxp) --top;
    const long long enough = s.nt == 1024 ? 256 : 512;
    if (s.V > 1 && a.C <= kFewChannels && tile_count(a, s.V, top) >= 4 * enough)
        while (s.nt > 64 && (s.nt >> (top + 1)) >= a.C) s.nt /= 2;
    int lxs = top;
    while (lxs > 0 && (groups(lxs) > good || tile_count(a, s.V, lxs) < enough)) --lxs;
    while (lxs < top && (s.V << lxs) * es < 64 && groups(lxs + 1) <= most && tile_count(a, s.V, lxs + 1) >= 256) ++lxs;
    const int K = groups(lxs);
    s.K = K <= 1 ? 1 : K <= 2 ? 2 : K <= 4 ? 4 : K <= 8 ? 8 : 16;
    if (s.K == 16 && s.V > 1) s.V /= 2;  // more than 4096 channels: twice the groups of half the width
    const long long tb = (a.L + (s.V << lxs) - 1) / (s.V << lxs);
    s.g = Lay{lxs, tb, tb * a.B, a.L % 4 == 0, (s.V << lxs) * es < 128};
    return s;
}

}  // namespace
}  // namespace hyenand
