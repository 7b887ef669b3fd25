// ffn_tile.h -- the matrix-core product of the gated feed-forward block: a
// workgroup computes one or two row groups of A times one tile of B, with the
// operation's epilogue on the accumulators.
//
// Every operand is a bf16 matrix in rows of 16-byte multiples.  A (weights, or
// gradients in the weight gradients) has its summation index k contiguous.  B
// is either k-contiguous too, or (activations of a [channel][position] layout)
// contiguous along its columns; then the transposing LDS read brings four
// consecutive k of a column into a lane, so activations are used where they lie.
//
// fp32 operands come as three bf16 planes whose sum is the value (8 bits each,
// split by truncation: exact, and the leading plane cannot overflow).  A step
// reads the three planes of both operands once and multiplies six pairs of
// them; the three pairs left out are below 2^-23 of |a| |b|.  The leading pair
// has an accumulator of its own, so the five small ones do not add to its
// roundings.  Six bf16 products have 2.7 times the rate of the fp32 matrix
// instruction (2.5 / 6 against 0.157 PFLOP/s).
//
// Pipeline: NST LDS stages of BK terms, filled from global memory directly (16
// bytes a lane) NST - 1 stages ahead; one barrier per stage.
//
// Measured on one MI355X at 1024 channels, 4096 hidden, 32768 positions, bf16:
// 1.0 to 1.15 PFLOP/s (y 0.24 to 0.26 ms, both weight gradients of the hidden
// layer 0.55 ms), half of the matrix cores' cycles at the 1.8 GHz that the card
// holds under this load, no LDS bank conflicts; library products of that size
// reach 1.27 to 1.52.  A tile reads 192 KB of fragments from LDS and takes 64 KB
// of loads for each 2048 matrix cycles, which is all that LDS moves (124 bytes a
// clock measured).
#pragma once

#include <type_traits>

#include "block_dev.h"

namespace hyenand {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int kPiece = 64;       // pieces of K (weight gradients) are multiples of this
constexpr int kMaxPhases = 3;
constexpr int kTileRows = 8;     // row tiles of a band

__device__ __align__(16) const unsigned g_zeros[4] = {0, 0, 0, 0};

// k-contiguous rows: element (r, k) at r * ld + (k / L) * sb + k % L (L: the
// positions of a batch entry, or more than K for one piece; pieces only where
// B is k-contiguous too, in the weight gradients).
// Column-contiguous (B only): element (k, n) at k * ld + (n / L) * sb + n % L.
// plane: distance of the planes of fp32.
struct Mat {
    long long ld, sb, plane;
    int L;
};

struct TileArgs {
    // Phase p adds A[p][g] B[p] to row group g of the accumulators; phase n1 (of
    // the gradient epilogue) adds to the third group, with K2 terms.
    const __bf16 *A0[kMaxPhases], *A1[kMaxPhases], *B[kMaxPhases];
    int n1;
    Mat ma, mb, ma2, mb2;
    int M, N, K, K2;
    int goff;            // rows between the two groups (0: two matrices of the same rows)
    int tm, tn, splits;  // tiles along M and N, pieces of K
    int kper;            // terms of a piece
    // outputs
    void *o0, *o1, *o2;  // stored rows; planes: first plane of each
    long long ldo, osb;  // row stride, batch stride of the output
    int oL;              // positions of a batch entry of the output
    long long plane;     // distance of the planes of an output
    int act;
    bool out32;          // fp32 output (else bf16)
};

enum { kEpiOut = 0, kEpiGate = 1, kEpiGrad = 2, kEpiPart = 3 };

template <int WM_, int WN_, int MT_, int NT_, int BK_, int NST_, int NPL_>
struct TileCfg {
    static constexpr int WM = WM_, WN = WN_, MT = MT_, NT = NT_, BK = BK_, NST = NST_, NPL = NPL_;
    static constexpr int NTH = 64 * WM * WN;
    static constexpr int BMG = 32 * WM * MT;  // rows of a group
    static constexpr int BN = 32 * WN * NT;
    static constexpr int PR = BK / 8;         // 16-byte pieces of a k-contiguous row
    static constexpr int kA1 = 2 * BMG * BK * 2, kB1 = BN * BK * 2;  // bytes of a plane's tile
    static constexpr int kStage = NPL * (kA1 + kB1);
    static constexpr int NACC = NPL == 1 ? 1 : 2;  // accumulators: the leading pair's, the small pairs'
};

// Swizzle of the 16-byte pieces of a k-contiguous row: with rows of 64 (128,
// 256) bytes, 16 rows of one piece then lie in 16 different bank groups.
template <int PR>
__device__ __forceinline__ int piece_swizzle(int row)
{
    return PR == 16 ? row & 15 : PR == 8 ? (row >> 1) & 7 : (row >> 2) & 3;
}

// Column-contiguous tiles are [term][BN / 8 pieces]; a transposing read takes 64
// bytes of each of four consecutive terms.  The 64-byte unit u of term k lies at
// u ^ unit_swizzle(k), which puts the four into different quarters of the banks
// (rows of 128 bytes already alternate between two of them).
template <int BN>
__device__ __forceinline__ int unit_swizzle(int k)
{
    return BN >= 128 ? k & 3 : (k >> 1) & 1;
}

// Fragments of 16 terms: row pieces of A and columns of B.
template <class Cfg, int G>
struct Frags {
    bf16x8 a[Cfg::NPL][G][Cfg::MT], b[Cfg::NPL][Cfg::NT];
};

template <class Cfg, int G>
struct Acc {
    f32x16 v[Cfg::NACC][G][Cfg::MT][Cfg::NT];
};

// aoff and boff are the lane's read offsets, swa its piece swizzle.
template <class Cfg, int G, bool BTR>
__device__ __forceinline__ void load_frags(Frags<Cfg, G>& f, const char* stage, int ks, int aoff,
                                           const int (&boff)[Cfg::NT], int h, int swa)
{
    const int piece = ((ks * 2 + h) ^ swa) << 4;
#pragma unroll
    for (int p = 0; p < Cfg::NPL; ++p) {
        const char *sa = stage + p * Cfg::kA1, *sb = stage + Cfg::NPL * Cfg::kA1 + p * Cfg::kB1;
#pragma unroll
        for (int j = 0; j < Cfg::NT; ++j) {
            if constexpr (BTR) {
                typedef __attribute__((address_space(3))) s16x4 lds4;
                const char* q = sb + boff[j] + ks * (16 * Cfg::BN * 2);
                const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)q);
                const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(q + 4 * Cfg::BN * 2));
                f.b[p][j] = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
            } else {
                f.b[p][j] = *reinterpret_cast<const bf16x8*>(sb + boff[j] + piece);
            }
        }
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int i = 0; i < Cfg::MT; ++i)
                f.a[p][g][i] = *reinterpret_cast<const bf16x8*>(sa + (g * Cfg::BMG + i * Cfg::WM * 32) * (Cfg::BK * 2) +
                                                                aoff + piece);
    }
}

// Columns of B along the accumulator's rows: a lane then holds runs of four
// consecutive columns of one row of the result.
template <class Cfg, int G>
__device__ __forceinline__ void multiply(const Frags<Cfg, G>& f, Acc<Cfg, G>& acc)
{
    const auto pair = [&](auto pa, auto pb, auto to) {
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int i = 0; i < Cfg::MT; ++i)
#pragma unroll
                for (int j = 0; j < Cfg::NT; ++j)
                    acc.v[to][g][i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.b[pb][j], f.a[pa][g][i],
                                                                                  acc.v[to][g][i][j], 0, 0, 0);
    };
    constexpr std::integral_constant<int, 0> c0{};
    if constexpr (Cfg::NPL == 3) {
        constexpr std::integral_constant<int, 1> c1{};
        constexpr std::integral_constant<int, 2> c2{};
        pair(c2, c0, c1);
        pair(c1, c1, c1);
        pair(c0, c2, c1);
        pair(c1, c0, c1);
        pair(c0, c1, c1);
    }
    pair(c0, c0, c0);
}

// Sum over phases [p0, p0 + np) into acc, G row groups.
template <class Cfg, int G, bool BTR>
__device__ __forceinline__ void tile_product(const TileArgs& a, int p0, int np, const Mat& ma, const Mat& mb, int K,
                                             int kb, int ke, int m0, int n0, char* S, Acc<Cfg, G>& acc)
{
    constexpr int NTH = Cfg::NTH, BN = Cfg::BN, BMG = Cfg::BMG, BK = Cfg::BK, PR = Cfg::PR, NST = Cfg::NST;
    constexpr int NA = G * BMG * PR / NTH, NB = BN * PR / NTH, RP = NTH / PR;  // pieces a thread, rows a pass
    constexpr int kPer = Cfg::NPL * (NA + NB);                                // loads a thread and stage
    static_assert(NA * NTH == G * BMG * PR && NB * NTH == BN * PR && RP % 16 == 0 && BMG % RP == 0);
    static_assert((NST - 1) * kPer < 64, "vmcnt");
    const int t = (int)threadIdx.x, lane = t & 63;
    const int w = __builtin_amdgcn_readfirstlane(t >> 6), wm = w / Cfg::WN, wn = w % Cfg::WN;
    const int steps = (ke - kb + BK - 1) / BK;
    if (steps <= 0 || np <= 0) return;
    // This thread's pieces; k-contiguous tiles are [row][PR pieces of 8 terms].
    const int ar = t / PR, ac = ((t % PR) ^ piece_swizzle<PR>(ar)) * 8;
    const __bf16 *pa[NA], *pb[NB];
    int la = 0, lb = 0;
    const auto start = [&](int p) {
        const long long k = kb + ac, qa = ma.L > k ? 0 : k / ma.L;
        la = (int)(k - qa * ma.L);
#pragma unroll
        for (int j = 0; j < NA; ++j) {
            const int r = j * RP + ar, g = G > 1 && r >= BMG ? 1 : 0;
            int row = m0 + (r - g * BMG) + (g ? a.goff : 0);
            row = row < a.M ? row : a.M - 1;  // rows past the end are computed and not stored
            pa[j] = (g ? a.A1[p] : a.A0[p]) + (long long)row * ma.ld + qa * ma.sb + la;
        }
        if constexpr (BTR) {
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                const int e = j * NTH + t, kk = e / (BN / 8), c = (e % (BN / 8)) ^ (unit_swizzle<BN>(kk) << 2);
                int n = n0 + c * 8;
                n = n < a.N ? n : 0;
                const int q = n / mb.L;
                pb[j] = a.B[p] + (long long)(kb + kk) * mb.ld + q * mb.sb + (n - q * mb.L);
            }
        } else {
            const long long q = mb.L > k ? 0 : k / mb.L;
            lb = (int)(k - q * mb.L);
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                int row = n0 + j * RP + ar;
                row = row < a.N ? row : a.N - 1;
                pb[j] = a.B[p] + (long long)row * mb.ld + q * mb.sb + lb;
            }
        }
    };
    int ip = p0, ik = kb, ib = 0;  // next stage to load: phase, first term, buffer
    const unsigned lds0 = lds_address(S) + w * 1024;
    const auto issue = [&] {
        const void* z = g_zeros;
        const unsigned d = lds0 + ib * Cfg::kStage;
        const auto load = [&](auto whole) {
            const bool oka = whole || ik + ac < K;
#pragma unroll
            for (int j = 0; j < NA; ++j)
#pragma unroll
                for (int p = 0; p < Cfg::NPL; ++p)
                    to_lds(oka ? (const void*)(pa[j] + p * ma.plane) : z, d + p * Cfg::kA1 + j * (NTH * 16));
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                const bool ok = whole || (BTR ? ik + (j * NTH + t) / (BN / 8) < K : oka);
#pragma unroll
                for (int p = 0; p < Cfg::NPL; ++p)
                    to_lds(ok ? (const void*)(pb[j] + p * mb.plane) : z,
                           d + Cfg::NPL * Cfg::kA1 + p * Cfg::kB1 + j * (NTH * 16));
            }
        };
        if (ik + BK <= K) load(std::true_type{});
        else load(std::false_type{});  // zeros past the last term
#pragma unroll
        for (int j = 0; j < NA; ++j) pa[j] += BK;
#pragma unroll
        for (int j = 0; j < NB; ++j) pb[j] += BTR ? (long long)BK * mb.ld : (long long)BK;
        if constexpr (!BTR) {
            // Positions as terms (weight gradients): on to the next batch entry.
            la += BK;
            while (la >= ma.L) {
                la -= ma.L;
#pragma unroll
                for (int j = 0; j < NA; ++j) pa[j] += ma.sb - ma.L;
            }
            lb += BK;
            while (lb >= mb.L) {
                lb -= mb.L;
#pragma unroll
                for (int j = 0; j < NB; ++j) pb[j] += mb.sb - mb.L;
            }
        }
        ib = ib + 1 < NST ? ib + 1 : 0;
        ik += BK;
        if (ik >= ke) {
            ik = kb;
            if (++ip < p0 + np) start(ip);
        }
    };
    // Read addresses.
    const int h = lane >> 5, swa = piece_swizzle<PR>(lane & 31);
    const int arow = (wm * 32 + (lane & 31)) * (BK * 2);
    int boff[Cfg::NT];
#pragma unroll
    for (int j = 0; j < Cfg::NT; ++j) {
        const int nb = (j * Cfg::WN + wn) * 32;
        if constexpr (BTR) {
            const int i = lane & 15, kk = 8 * h + (i >> 2);
            boff[j] = kk * (BN * 2) + (((nb >> 5) ^ unit_swizzle<BN>(i >> 2)) << 6) + ((lane >> 4) & 1) * 32 + (i & 3) * 8;
        } else {
            boff[j] = (nb + (lane & 31)) * (BK * 2);
        }
    }
    const int total = steps * np;
    start(p0);
    for (int i = 0; i < NST && i < total; ++i) issue();
    if (total >= NST) wait_loads<(NST - 1) * kPer>();
    else wait_loads();
    __syncthreads();
    // A step's fragments are read while the step before multiplies.  The barrier
    // that ends a stage comes before its last multiplication: by then every wave
    // has the stage's last fragments in registers, so its buffer can be filled
    // again, and the next stage's first fragments are read behind that work.
    constexpr int KS = BK / 16;
    static_assert(KS % 2 == 0);
    Frags<Cfg, G> f[2];
    int buf = 0;
    load_frags<Cfg, G, BTR>(f[0], S, 0, arow, boff, h, swa);
    for (int it = 0; it < total; ++it) {
        const char* stage = S + buf * Cfg::kStage;
        buf = buf + 1 < NST ? buf + 1 : 0;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            if (ks + 1 < KS) {
                load_frags<Cfg, G, BTR>(f[(ks + 1) & 1], stage, ks + 1, arow, boff, h, swa);
            } else if (it + 1 < total) {
                if (it + NST <= total) wait_loads<(NST - 2) * kPer>();
                else wait_loads();
                __syncthreads();
                if (it + NST < total) issue();
                load_frags<Cfg, G, BTR>(f[0], S + buf * Cfg::kStage, 0, arow, boff, h, swa);
            }
            multiply<Cfg, G>(f[ks & 1], acc);
            // One read, one multiplication at a time (3% on the training step's launches).
#pragma unroll
            for (int i = 0; i < Cfg::NPL * (G * Cfg::MT + Cfg::NT * (BTR ? 2 : 1)); ++i) {
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
            }
        }
    }
    if constexpr (Cfg::NPL == 3) {
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int i = 0; i < Cfg::MT; ++i)
#pragma unroll
                for (int j = 0; j < Cfg::NT; ++j) acc.v[0][g][i][j] += acc.v[1][g][i][j];
    }
}

__device__ __forceinline__ float truncated(float v)
{
    return __builtin_bit_cast(float, __builtin_bit_cast(unsigned, v) & 0xffff0000u);
}

// The three planes of v (see above).  Non-finite values keep their leading
// plane alone.
__device__ __forceinline__ void split3(float v, float (&p)[3])
{
    p[0] = truncated(v);
    // A NaN whose payload lies in the low half would lose it.
    if (v != v) p[0] = v;
    const bool fin = __builtin_fabsf(p[0]) < __builtin_inff();
    const float r = fin ? v - p[0] : 0.0f;
    p[1] = truncated(r);
    p[2] = r - p[1];
}

// Epilogue.  The accumulators' 32 x 32 blocks (i, j) of all waves form an
// SR x SC sub-tile of consecutive rows and columns; one sub-tile at a time goes
// through LDS (fp32, of every accumulator group) and is finished in pieces of
// eight columns a thread: results leave in rows of 16 bytes a lane, and the
// activation's code exists once per sub-tile instead of once per register.
template <class Cfg>
struct Sub {
    static constexpr int SR = 32 * Cfg::WM, SC = 32 * Cfg::WN;
    // Rows are 16 bytes longer than their columns: 16 rows at one column start in different banks.
    static constexpr int LD = SC * 4 + 16, kBytes = SR * LD;

    static __device__ __forceinline__ void put(char* S, const f32x16& v)
    {
        const int t = (int)threadIdx.x, lane = t & 63, w = t >> 6, wm = w / Cfg::WN, wn = w % Cfg::WN;
        // A lane holds runs of four consecutive columns of one row.
        char* d = S + (wm * 32 + (lane & 31)) * LD + (wn * 32 + 4 * (lane >> 5)) * 4;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            u32x4 o;
#pragma unroll
            for (int r = 0; r < 4; ++r) o[r] = bits_of((float)v[4 * q + r]);
            *reinterpret_cast<u32x4*>(d + q * 32) = o;
        }
    }

    static __device__ __forceinline__ void get(const char* S, int row, int col, float (&f)[8])
    {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const u32x4 q = *reinterpret_cast<const u32x4*>(S + row * LD + (col + 4 * k) * 4);
#pragma unroll
            for (int r = 0; r < 4; ++r) f[4 * k + r] = __builtin_bit_cast(float, (unsigned)q[r]);
        }
    }

    // piece(row, column) for every eight columns of the sub-tile.
    template <class F>
    static __device__ __forceinline__ void pieces(F&& piece)
    {
        static_assert(SR * SC / 8 % Cfg::NTH == 0);
#pragma unroll 1
        for (int e = (int)threadIdx.x; e < SR * SC / 8; e += Cfg::NTH) piece(e / (SC / 8), e % (SC / 8) * 8);
    }
};

// Eight columns of row m into the planes of an intermediate matrix; columns past
// N are written as zeros up to the row's padding, where the weight gradients
// read them as terms.
template <int NPL>
__device__ __forceinline__ void store_plane(const TileArgs& a, void* o, int m, int n, float (&f)[8])
{
    if (n >= a.ldo) return;
    if (n + 8 > a.N) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = n + i < a.N ? f[i] : 0.0f;
    }
    __bf16* q = (__bf16*)o + (long long)m * a.ldo + n;
    if constexpr (NPL == 1) {
        store_pack<__bf16, 8>(q, f, 8);
        return;
    }
    float s[3][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float p[3];
        split3(f[i], p);
#pragma unroll
        for (int k = 0; k < 3; ++k) s[k][i] = p[k];
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) store_pack<__bf16, 8>(q + k * a.plane, s[k], 8);
}

// Eight columns of row m into a result of the caller's layout.
template <class T>
__device__ __forceinline__ void store_out(const TileArgs& a, void* o, int m, int n, const float (&f)[8])
{
    if (n >= a.N) return;
    T* r = (T*)o + (long long)m * a.ldo;
    const int q = n / a.oL, l = n - q * a.oL;
    if (n + 8 <= a.N && l + 8 <= a.oL) {
        store_pack<T, 8>(r + q * a.osb + l, f, 8);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int c = n + i, qq = c / a.oL;
        if (c < a.N) r[qq * a.osb + (c - qq * a.oL)] = (T)f[i];
    }
}

template <class Cfg, int EPI>
constexpr int tile_lds()
{
    const int stages = Cfg::NST * Cfg::kStage, out = (EPI == kEpiGrad ? 3 : 2) * Sub<Cfg>::kBytes;
    return stages > out ? stages : out;
}

template <class Cfg, bool BTR, int EPI>
__global__ __launch_bounds__(Cfg::NTH) void k_ffn_tile(TileArgs a)
{
    __shared__ __align__(1024) char S[tile_lds<Cfg, EPI>()];
    // Workgroups are dealt to the eight XCDs in turn: each takes a contiguous run
    // of tiles, in columns of up to kTileRows row tiles, so that the operands
    // its workgroups share stay in its own L2.
    const int G = (int)gridDim.x, xcd = (int)blockIdx.x & 7, per = G >> 3, rem = G & 7;
    const int id = xcd * per + (xcd < rem ? xcd : rem) + ((int)blockIdx.x >> 3);
    const int tiles = a.tm * a.tn, s = id / tiles, tile = id - s * tiles;
    const int band = tile / (kTileRows * a.tn), in = tile - band * (kTileRows * a.tn);
    const int left = a.tm - band * kTileRows, bm = left < kTileRows ? left : kTileRows;
    const int m0 = (band * kTileRows + in % bm) * (a.goff ? 2 * Cfg::BMG : Cfg::BMG), n0 = (in / bm) * Cfg::BN;
    const int kb = s * a.kper, ke = kb + a.kper < a.K ? kb + a.kper : a.K;
    Acc<Cfg, 2> acc{};
    tile_product<Cfg, 2, BTR>(a, 0, a.n1, a.ma, a.mb, a.K, kb, ke, m0, n0, S, acc);
    Acc<Cfg, 1> dh{};
    if constexpr (EPI == kEpiGrad) {
        __syncthreads();
        tile_product<Cfg, 1, BTR>(a, a.n1, 1, a.ma2, a.mb2, a.K2, 0, a.K2, m0, n0, S, dh);
    }
    typedef Sub<Cfg> E;
    char *S0 = S, *S1 = S + E::kBytes, *S2 = S + 2 * E::kBytes;
#pragma unroll
    for (int i = 0; i < Cfg::MT; ++i)
#pragma unroll
        for (int j = 0; j < Cfg::NT; ++j) {
            __syncthreads();
            E::put(S0, acc.v[0][0][i][j]);
            E::put(S1, acc.v[0][1][i][j]);
            if constexpr (EPI == kEpiGrad) E::put(S2, dh.v[0][0][i][j]);
            __syncthreads();
            E::pieces([&](int row, int col) {
                const int m = m0 + i * E::SR + row, n = n0 + j * E::SC + col;
                float f0[8], f1[8];
                E::get(S0, row, col, f0);
                E::get(S1, row, col, f1);
                if constexpr (EPI == kEpiOut || EPI == kEpiPart) {
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        const int mg = m + g * a.goff;
                        if (mg >= a.M) return;  // the second group's rows come after the first's
                        const float(&f)[8] = g ? f1 : f0;
                        void* o = g && !a.goff ? a.o1 : a.o0;
                        if (EPI == kEpiPart && a.splits > 1) {
                            // [piece][row][column], the second matrix's rows behind the first's
                            const int rows = a.goff ? a.M : 2 * a.M, at = g && !a.goff ? a.M : 0;
                            store_out<float>(a, (float*)a.o2 + ((long long)s * rows + at) * a.N, mg, n, f);
                        } else if (a.out32) {
                            store_out<float>(a, o, mg, n, f);
                        } else {
                            store_out<__bf16>(a, o, mg, n, f);
                        }
                    }
                } else if (m < a.M) {
                    if constexpr (EPI == kEpiGate) {
                        with_act(a.act, [&](auto act) {
#pragma unroll
                            for (int r = 0; r < 8; ++r) f0[r] = act_fwd(act, f0[r]) * f1[r];
                        });
                        store_plane<Cfg::NPL>(a, a.o0, m, n, f0);
                    } else {
                        float d[8], du[8];
                        E::get(S2, row, col, d);
                        with_act(a.act, [&](auto act) {
#pragma unroll
                            for (int r = 0; r < 8; ++r) {
                                float ga, da;
                                act_both(act, f0[r], ga, da);
                                f0[r] = ga * f1[r];
                                du[r] = d[r] * ga;
                                f1[r] = d[r] * f1[r] * da;
                            }
                        });
                        store_plane<Cfg::NPL>(a, a.o0, m, n, f0);
                        store_plane<Cfg::NPL>(a, a.o1, m, n, f1);
                        store_plane<Cfg::NPL>(a, a.o2, m, n, du);
                    }
                }
            });
        }
}

}  // namespace
}  // namespace hyenand
