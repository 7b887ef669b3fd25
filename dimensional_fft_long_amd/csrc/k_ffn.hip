// k_ffn.hip -- the gated feed-forward block, forward and backward: the launch
// chains over the matrix-core product of ffn_tile.h, operands brought into its
// layout, and the weight gradients' sum over pieces.
//
//   forward   h  = a(Wg x) (Wu x)            one launch, both products and the gate in its epilogue
//             y  = Wd h
//   backward  g, u, dh = Wd^T dy -> h, dg, du  one launch: g, u and dh stay in the accumulators
//             dx = Wg^T dg + Wu^T du          one launch, both products into one accumulator
//             dWg, dWu = dg x^T, du x^T       one launch (x is read once for both)
//             dWd = dy h^T
//
// The hidden values are planes [F][positions of all batch entries], padded to
// eight.  Operands are used where they lie if their rows are multiples of 16
// bytes (bf16, C, F and L multiples of eight); else, and for fp32, a pass
// writes them as padded bf16 planes first, all of a chain's operands in one
// launch.  Measured on one MI355X, training step (forward and backward): 1024
// channels, 4096 hidden, 32768 positions, bf16 3.03 ms (22 C F T operations with
// the recomputed products: 1.0 PFLOP/s); 100 channels, 333 hidden, 5883
// positions, fp32 178 us in eleven launches.
#include "ffn_tile.h"

#include <climits>

namespace hyenand {
namespace {

constexpr long long kFar = 1ll << 62;

// Source of a pass: element (r, t) at r * sr + (t / L) * sb + (t % L) * st.
struct View {
    const void* p;
    long long sr, st, L, sb;
};

// One operand to bring into planes; a launch does all of a chain's.
struct PackJob {
    View v;
    __bf16* dst;
    long long plane;
    int rows, cols, ld;
    bool by_row;          // threads along the rows (the direction contiguous in the source)
    unsigned first;       // first workgroup
};
constexpr int kMaxJobs = 7;
struct PackJobs {
    PackJob j[kMaxJobs];
    int n;
};

template <class T, int NPL>
__global__ __launch_bounds__(256) void k_ffn_pack(PackJobs jobs)
{
    int which = 0;
    while (which + 1 < jobs.n && blockIdx.x >= jobs.j[which + 1].first) ++which;
    const PackJob& job = jobs.j[which];
    const View& v = job.v;
    const int rows = job.rows, cols = job.cols, ld = job.ld;
    const long long i = (long long)(blockIdx.x - job.first) * 256 + threadIdx.x;
    const int gc = ld / 8;
    const long long r = job.by_row ? i % rows : i / gc, g = job.by_row ? i / rows : i % gc;
    if (r >= rows || g >= gc) return;
    const long long t0 = g * 8;
    float f[8];
    const long long q = t0 / v.L, l = t0 - q * v.L;
    const T* s = (const T*)v.p + r * v.sr;
    if (v.st == 1 && t0 + 8 <= cols && l + 8 <= v.L) {
        const Pack<T, 8> k = load_pack<T, 8>(s + q * v.sb + l, 8);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = k.get(j);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const long long t = t0 + j, qq = t / v.L;
            f[j] = t < cols ? (float)s[qq * v.sb + (t - qq * v.L) * v.st] : 0.0f;
        }
    }
    __bf16* d = job.dst + r * ld + t0;
    if constexpr (NPL == 1) {
        store_pack<__bf16, 8>(d, f, 8);
    } else {
        float s3[3][8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float p[3];
            split3(f[j], p);
#pragma unroll
            for (int k = 0; k < 3; ++k) s3[k][j] = p[k];
        }
#pragma unroll
        for (int k = 0; k < 3; ++k) store_pack<__bf16, 8>(d + k * job.plane, s3[k], 8);
    }
}

// Weight gradients: the pieces' partial sums [splits][rows][N] in order, the
// first M rows to o0 and the rest to o1.
template <class T>
__global__ __launch_bounds__(256) void k_ffn_sum(const float* part, int splits, long long n, long long n0, T* o0, T* o1)
{
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    float s = 0.0f;
#pragma unroll 8
    for (int p = 0; p < splits; ++p) s += part[(long long)p * n + i];
    if (i < n0) o0[i] = (T)s;
    else o1[i - n0] = (T)s;
}

__global__ __launch_bounds__(256) void k_ffn_zero(unsigned short* p, long long n)
{
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) p[i] = 0;
}

// Tiles.  bf16: Big fills a CU (128 KB of stages, eight waves); Mid runs two
// workgroups a CU where Big has too few tiles; Small adds stages in flight for
// launches that cannot fill the device.  fp32 (three planes): Wide and Slim.
typedef TileCfg<2, 4, 2, 2, 64, 2, 1> Big;    // 128 (x 2 groups) x 256
typedef TileCfg<2, 2, 1, 2, 64, 2, 1> Mid;    // 64 (x 2) x 128
typedef TileCfg<2, 2, 1, 1, 64, 4, 1> Small;  // 64 (x 2) x 64
typedef TileCfg<2, 2, 1, 2, 32, 3, 3> Wide;   // 64 (x 2) x 128
typedef TileCfg<2, 2, 1, 1, 32, 4, 3> Slim;   // 64 (x 2) x 64
enum Tile { kBig, kMid, kSmall, kWide, kSlim };
constexpr int kCUs = 256;

struct TileSize {
    int bmg, bn, slots;
};

TileSize tile_size(Tile t)
{
    switch (t) {
    case kBig: return {Big::BMG, Big::BN, kCUs};
    case kMid: return {Mid::BMG, Mid::BN, 2 * kCUs};
    case kSmall: return {Small::BMG, Small::BN, kCUs};
    case kWide: return {Wide::BMG, Wide::BN, kCUs};
    default: return {Slim::BMG, Slim::BN, kCUs};
    }
}

long long tiles_of(Tile t, long long rows, long long cols, bool dual)
{
    const TileSize s = tile_size(t);
    const long long m = s.bmg * (dual ? 1 : 2);
    return ((rows + m - 1) / m) * ((cols + s.bn - 1) / s.bn);
}

// The largest tile that still gives (most of) the device's CUs one.
Tile pick_tile(bool bf16, long long rows, long long cols, bool dual)
{
    if (!bf16) return tiles_of(kWide, rows, cols, dual) >= kCUs * 3 / 4 ? kWide : kSlim;
    if (tiles_of(kBig, rows, cols, dual) >= kCUs * 3 / 4) return kBig;
    return tiles_of(kMid, rows, cols, dual) >= kCUs * 3 / 4 ? kMid : kSmall;
}

long long round8(long long v) { return (v + 7) & ~7ll; }

// Row stride of the position planes: an odd multiple of 128 bytes, so that the
// rows a stage reads (one column block of 64 rows) lie on different memory
// channels whatever the number of positions.
long long spread(long long v)
{
    const long long lines = (v + 63) / 64;
    return (lines | 1) * 64;
}

// A packed operand or intermediate: planes of [rows][ld].
struct Planes {
    __bf16* p;
    long long ld, plane;
};

// How the weight gradients' sum over positions is cut: pieces of whole stages so
// that the tiles fill the device's workgroup slots, weighed against the partial
// sums' traffic (time in units of one stage of the big tile, about a microsecond).
int pieces(long long tiles, int slots, long long K, long long elems)
{
    const long long steps = (K + kPiece - 1) / kPiece;
    double best = 0.0;
    int pick = 1;
    for (int s = 1; s <= 128 && s <= steps; ++s) {
        const double waves = (double)((tiles * s + slots - 1) / slots), per = (double)((steps + s - 1) / s);
        const double cost = waves * (per + 6.0) + (s > 1 ? 10.0 + (double)elems * s * 8.0 / 4.0e6 : 0.0);
        if (s == 1 || cost < best) best = cost, pick = s;
    }
    return pick;
}

struct Cut {
    Tile tile;
    int splits;
};

Cut cut_dw(bool bf16, long long rows, long long cols, long long K, bool dual)
{
    const Tile t = !bf16 ? kWide : rows >= Big::BMG && cols >= Big::BN ? kBig : kMid;
    return Cut{t, pieces(tiles_of(t, rows, cols, dual), tile_size(t).slots, K, rows * cols * (dual ? 2 : 1))};
}

struct Layout {
    int npl;
    long long T, Tp, Cp, Fp;
    bool xdirect, wdirect;
    size_t h, dg, du, x, dy, wg, wu, wd, wgt, wut, wdt, part, total;
};

Layout layout(int B, int C, int F, long long L, bool bf16, bool bwd)
{
    Layout o{};
    o.npl = bf16 ? 1 : 3;
    o.T = B * L;
    o.Tp = spread(o.T);
    o.Cp = round8(C);
    o.Fp = round8(F);
    o.xdirect = bf16 && L % 8 == 0;
    o.wdirect = bf16 && C % 8 == 0 && F % 8 == 0;
    size_t at = 0;
    const auto take = [&](size_t& off, long long rows, long long ld) {
        off = at;
        at += ((size_t)rows * (size_t)ld * 2u * (size_t)o.npl + 255u) & ~(size_t)255u;
    };
    take(o.h, F, o.Tp);
    if (!o.xdirect) take(o.x, C, o.Tp);
    if (!o.wdirect) {
        take(o.wg, F, o.Cp);
        take(o.wu, F, o.Cp);
        if (!bwd) take(o.wd, C, o.Fp);
    }
    if (bwd) {
        take(o.dg, F, o.Tp);
        take(o.du, F, o.Tp);
        if (!o.xdirect) take(o.dy, C, o.Tp);
        take(o.wgt, C, o.Fp);
        take(o.wut, C, o.Fp);
        take(o.wdt, F, o.Cp);
        const Cut c1 = cut_dw(bf16, F, C, o.T, true), c2 = cut_dw(bf16, C, F, o.T, false);
        const size_t e1 = c1.splits > 1 ? (size_t)c1.splits * 2u : 0u, e2 = c2.splits > 1 ? (size_t)c2.splits : 0u;
        o.part = at;
        at += (e1 > e2 ? e1 : e2) * (size_t)F * (size_t)C * 4u;
    }
    o.total = at;
    return o;
}

template <class Cfg, bool BTR, int EPI>
hipError_t run_tiles(TileArgs& a, hipStream_t st)
{
    const long long gm = a.goff ? 2 * Cfg::BMG : Cfg::BMG;
    if (a.goff) a.goff = Cfg::BMG;
    const long long tm = (a.M + gm - 1) / gm, tn = ((long long)a.N + Cfg::BN - 1) / Cfg::BN;
    if (tm * tn * a.splits > INT_MAX) return hipErrorInvalidValue;
    a.tm = (int)tm;
    a.tn = (int)tn;
    hipLaunchKernelGGL((k_ffn_tile<Cfg, BTR, EPI>), dim3((unsigned)(tm * tn * a.splits)), dim3(Cfg::NTH), 0, st, a);
    return launch_status();
}

template <bool BTR, int EPI>
hipError_t run_any(TileArgs& a, Tile t, hipStream_t st)
{
    switch (t) {
    case kBig: return run_tiles<Big, BTR, EPI>(a, st);
    case kMid: return run_tiles<Mid, BTR, EPI>(a, st);
    case kSmall:
        if constexpr (EPI != kEpiPart) return run_tiles<Small, BTR, EPI>(a, st);
        return hipErrorInvalidValue;
    case kWide: return run_tiles<Wide, BTR, EPI>(a, st);
    case kSlim:
        if constexpr (EPI != kEpiPart) return run_tiles<Slim, BTR, EPI>(a, st);
        return hipErrorInvalidValue;
    }
    return hipErrorInvalidValue;
}

void set_phase(TileArgs& a, int i, const Planes& A0, const Planes& A1, const Planes& B)
{
    a.A0[i] = A0.p;
    a.A1[i] = A1.p;
    a.B[i] = B.p;
}

struct Chain {
    const FfnArgs& f;
    Layout o;
    hipStream_t st;
    char* ws;
    PackJobs jobs{};
    unsigned blocks = 0;

    Chain(const FfnArgs& a, bool bwd, hipStream_t s)
        : f(a), o(layout(a.B, a.C, a.F, a.L, a.bf16, bwd)), st(s), ws((char*)a.ws)
    {
    }
    Planes planes(size_t off, long long rows, long long ld) const { return {(__bf16*)(ws + off), ld, rows * ld}; }

    void pack(const View& v, int rows, int cols, const Planes& d, bool by_row)
    {
        PackJob& j = jobs.j[jobs.n++];
        j = PackJob{v, d.p, d.plane, rows, cols, (int)d.ld, by_row, blocks};
        blocks += (unsigned)((rows * (d.ld / 8) + 255) / 256);
    }

    // The passes asked for so far, in one launch.
    hipError_t run_packs() const
    {
        if (jobs.n == 0) return hipSuccess;
        if (f.bf16) hipLaunchKernelGGL((k_ffn_pack<__bf16, 1>), dim3(blocks), dim3(256), 0, st, jobs);
        else hipLaunchKernelGGL((k_ffn_pack<float, 3>), dim3(blocks), dim3(256), 0, st, jobs);
        return launch_status();
    }

    // Activations [B][C][L] as an operand: where they lie, or packed at off.
    void act(const void* x, size_t off, Planes* p, Mat* m)
    {
        if (o.xdirect) {
            *p = Planes{(__bf16*)x, f.L, 0};
            *m = Mat{f.L, f.C * f.L, 0, (int)f.L};
            return;
        }
        *p = planes(off, f.C, o.Tp);
        *m = Mat{o.Tp, 0, p->plane, INT_MAX};
        // One position per batch entry: rows of channels, read along them.
        const View v = f.L == 1 ? View{x, 1, f.C, kFar, 0} : View{x, f.L, 1, f.L, f.C * f.L};
        pack(v, f.C, (int)o.T, *p, f.L == 1);
    }

    void weight(const void* w, size_t off, int rows, int cols, Planes* p, Mat* m)
    {
        const long long ld = o.wdirect ? cols : round8(cols);
        *p = o.wdirect ? Planes{(__bf16*)w, ld, 0} : planes(off, rows, ld);
        *m = Mat{ld, 0, p->plane, INT_MAX};
        if (!o.wdirect) pack(View{w, cols, 1, kFar, 0}, rows, cols, *p, false);
    }

    // w [cols][rows] transposed.
    void weight_t(const void* w, size_t off, int rows, int cols, Planes* p, Mat* m)
    {
        const long long ld = round8(cols);
        *p = planes(off, rows, ld);
        *m = Mat{ld, 0, p->plane, INT_MAX};
        pack(View{w, 1, rows, kFar, 0}, rows, cols, *p, true);
    }

    TileArgs base(int M, long long N, int K) const
    {
        TileArgs a{};
        a.M = M;
        a.N = (int)N;
        a.K = a.kper = K;
        a.splits = 1;
        a.act = f.act;
        a.out32 = !f.bf16;
        a.oL = INT_MAX;
        return a;
    }

    // y or dx: rows of C channels in the caller's layout.
    void to_grid(TileArgs& a, void* out) const
    {
        a.o0 = out;
        a.ldo = f.L;
        a.osb = f.C * f.L;
        a.oL = (int)f.L;
        a.goff = 1;
    }

    // Few channels, and few hidden rows or many positions.  A workgroup of the
    // one-launch form goes through all hidden rows by itself, 1.8 to 2.6 us a
    // hundred, however few workgroups there are.  Measured, us, one launch
    // against tiles at 32 (128) channels: 1024 positions, 256 hidden 12 (12) / 15 (15),
    // 1024 hidden 20 (31) / 17 (18), 4096 hidden 71 (109) / 42 (43); 8192
    // positions, 1024 hidden 21 (33) / 24 (27); 32768 positions, 1024 hidden
    // 22 (37) / 58 (68), 4096 hidden 77 (131) / 216 (260).
    bool one_launch() const { return f.bf16 && f.C <= kFusedMaxC && (f.F <= 512 || o.T >= 16384); }

    hipError_t forward()
    {
        Planes x, wg, wu, wd, h = planes(o.h, f.F, o.Tp);
        Mat mx, mw, md;
        hipError_t e;
        act(f.x, o.x, &x, &mx);
        weight(f.Wg, o.wg, f.F, f.C, &wg, &mw);
        weight(f.Wu, o.wu, f.F, f.C, &wu, &mw);
        weight(f.Wd, o.wd, f.C, f.F, &wd, &md);
        if ((e = run_packs()) != hipSuccess) return e;
        if (one_launch())
            return launch_ffn_fused(FusedFfn{x.p, wg.p, wu.p, wd.p, f.y, mx.ld, mx.sb, mx.L, mw.ld, md.ld, f.C, f.F,
                                             (int)o.T, f.act, f.L, f.C * f.L, (int)f.L}, st);
        TileArgs a = base(f.F, o.T, f.C);
        a.n1 = 1;
        set_phase(a, 0, wg, wu, x);
        a.ma = mw;
        a.mb = mx;
        a.o0 = h.p;
        a.ldo = o.Tp;
        a.plane = h.plane;
        if ((e = run_any<true, kEpiGate>(a, pick_tile(f.bf16, f.F, o.T, true), st)) != hipSuccess) return e;
        TileArgs d = base(f.C, o.T, f.F);
        d.n1 = 1;
        set_phase(d, 0, wd, wd, h);
        d.ma = md;
        d.mb = Mat{o.Tp, 0, h.plane, INT_MAX};
        to_grid(d, f.y);
        return run_any<true, kEpiOut>(d, pick_tile(f.bf16, f.C, o.T, false), st);
    }

    hipError_t weight_grad(TileArgs& a, bool dual, void* o0, void* o1) const
    {
        const Cut c = cut_dw(f.bf16, a.M, a.N, o.T, dual);
        a.splits = c.splits;
        a.kper = (int)(((o.T + kPiece - 1) / kPiece + c.splits - 1) / c.splits) * kPiece;
        a.goff = dual ? 0 : 1;
        a.o0 = o0;
        a.o1 = o1;
        a.o2 = ws + o.part;
        a.ldo = a.N;
        hipError_t e = run_any<false, kEpiPart>(a, c.tile, st);
        if (e != hipSuccess || c.splits == 1) return e;
        const long long n0 = (long long)a.M * a.N, n = n0 * (dual ? 2 : 1);
        const unsigned grid = (unsigned)((n + 255) / 256);
        if (f.bf16)
            hipLaunchKernelGGL(k_ffn_sum<__bf16>, dim3(grid), dim3(256), 0, st, (const float*)a.o2, c.splits, n, n0,
                               (__bf16*)o0, (__bf16*)o1);
        else
            hipLaunchKernelGGL(k_ffn_sum<float>, dim3(grid), dim3(256), 0, st, (const float*)a.o2, c.splits, n, n0,
                               (float*)o0, (float*)o1);
        return launch_status();
    }

    hipError_t backward()
    {
        Planes x, dy, wg, wu, wgt, wut, wdt;
        const Planes h = planes(o.h, f.F, o.Tp), dg = planes(o.dg, f.F, o.Tp), du = planes(o.du, f.F, o.Tp);
        Mat mx, mw, mt, mdt;
        const Mat mh{o.Tp, 0, h.plane, INT_MAX};
        hipError_t e;
        act(f.x, o.x, &x, &mx);
        act(f.dy, o.dy, &dy, &mx);
        weight(f.Wg, o.wg, f.F, f.C, &wg, &mw);
        weight(f.Wu, o.wu, f.F, f.C, &wu, &mw);
        weight_t(f.Wg, o.wgt, f.C, f.F, &wgt, &mt);
        weight_t(f.Wu, o.wut, f.C, f.F, &wut, &mt);
        weight_t(f.Wd, o.wdt, f.F, f.C, &wdt, &mdt);
        if ((e = run_packs()) != hipSuccess) return e;
        // h, dg, du
        TileArgs a = base(f.F, o.T, f.C);
        a.n1 = 1;
        set_phase(a, 0, wg, wu, x);
        set_phase(a, 1, wdt, wdt, dy);
        a.ma = mw;
        a.mb = a.mb2 = mx;
        a.ma2 = mdt;
        a.K2 = f.C;
        a.o0 = h.p;
        a.o1 = dg.p;
        a.o2 = du.p;
        a.ldo = o.Tp;
        a.plane = h.plane;
        if ((e = run_any<true, kEpiGrad>(a, pick_tile(f.bf16, f.F, o.T, true), st)) != hipSuccess) return e;
        // dx
        TileArgs d = base(f.C, o.T, f.F);
        d.n1 = 2;
        set_phase(d, 0, wgt, wgt, dg);
        set_phase(d, 1, wut, wut, du);
        d.ma = mt;
        d.mb = mh;
        to_grid(d, f.dx);
        if ((e = run_any<true, kEpiOut>(d, pick_tile(f.bf16, f.C, o.T, false), st)) != hipSuccess) return e;
        // dWg, dWu
        TileArgs w = base(f.F, f.C, (int)o.T);
        w.n1 = 1;
        set_phase(w, 0, dg, du, x);
        w.ma = mh;
        w.mb = mx;
        if ((e = weight_grad(w, true, f.dWg, f.dWu)) != hipSuccess) return e;
        // dWd
        TileArgs v = base(f.C, f.F, (int)o.T);
        v.n1 = 1;
        set_phase(v, 0, dy, dy, h);
        v.ma = mx;
        v.mb = mh;
        return weight_grad(v, false, f.dWd, nullptr);
    }
};

}  // namespace

hipError_t launch_ffn_zero(void* p, long long bytes, hipStream_t st)
{
    // A launch holds fewer than 2^32 threads; the largest weights have more halves.
    const long long n = bytes / 2, blocks = (n + 255) / 256;
    hipLaunchKernelGGL(k_ffn_zero, dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(256), 0, st, (unsigned short*)p, n);
    return launch_status();
}

size_t ffn_workspace(int B, int C, int F, long long L, bool bf16, bool bwd) { return layout(B, C, F, L, bf16, bwd).total; }

hipError_t launch_ffn_fwd(const FfnArgs& a, hipStream_t st)
{
    if (a.B * a.L <= kFewPositions) return launch_ffn_few(a, st);
    return Chain(a, false, st).forward();
}

hipError_t launch_ffn_bwd(const FfnArgs& a, hipStream_t st) { return Chain(a, true, st).backward(); }

}  // namespace hyenand
