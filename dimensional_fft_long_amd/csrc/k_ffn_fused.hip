// k_ffn_fused.hip -- the gated feed-forward block's forward in one launch for
// few channels (bf16, C <= 128): the hidden values never leave the registers.
//
// A wave owns 32 positions.  Its x fragments (all channels) and its y
// accumulators (all channels) stay in registers while the hidden rows go by in
// chunks of 32: g and u of the chunk (two 32 x 32 products over C), h = a(g) u,
// then y += Wd[:, chunk] h.  The accumulator layout of the first products is
// the operand layout of the last one up to the order of the hidden rows inside
// the chunk, so h only rounds to bf16 in place: a lane holds accumulator rows
// 16 s + 8 a + 4 h + b (h its half of the wave) and the operand wants terms
// 16 s + 8 h + 4 a + b, so the rows of Wg and Wu are read with these two bits
// exchanged.  Weights stream through LDS in two stages (24 KB a chunk at
// C = 128), shared by the four waves of a workgroup.
//
// The two-launch form moves h through HBM twice (2 F positions x 2 bytes each
// way, 4.3 GB at C = 128, F = 512, two million positions, against 1.1 GB for x
// and y), and its products have only C = 128 terms, too few to hide a tile's
// start and end.  Here the bound is shared by the matrix cores (48 cycles a
// hidden value a lane at C = 128) and the activation's vector instructions (54
// cycles, two of them quarter-rate); two workgroups per CU let one wave of a
// SIMD multiply while the other evaluates.  Measured on one MI355X at C = 128,
// F = 512, two million positions: 0.93 to 1.1 ms against 2.56 ms in two
// launches; 230 us plus 1.4 us a hidden row, matrix cores 41% and vector
// instructions 55% busy at 1.65 GHz.
#include "ffn_tile.h"

namespace hyenand {
namespace {

constexpr int kFusedCols = 128;  // positions of a workgroup (four waves of 32)

struct FusedArgs {
    const __bf16 *x, *wg, *wu, *wd;
    void* y;
    Mat mx;           // x: element (c, n), column-contiguous
    long long ldw, ldd;  // row strides of Wg / Wu and of Wd
    int C, F, N, act;
    long long ldo, osb;
    int oL;
};

// KC: 32-channel groups (C <= 32 KC).
template <int KC>
struct FusedCfg {
    static constexpr int PR = KC <= 1 ? 4 : KC == 2 ? 8 : 16;  // 16-byte pieces of a weight row in LDS
    static constexpr int kW = 32 * PR * 16;                    // bytes of a chunk of Wg (and of Wu)
    static constexpr int kD = KC * 32 * 64;                    // bytes of a chunk of Wd: rows of 32 hidden values
    static constexpr int kStage = 2 * kW + kD;
    static constexpr int kX = KC * 32 * kFusedCols * 2;
    static constexpr int kOut = KC * 32 * (kFusedCols * 2 + 16);
    static constexpr int kBytes = 2 * kStage + kX > kOut ? 2 * kStage + kX : kOut;
};

template <int KC>
__global__ __launch_bounds__(256, 2) void k_ffn_fused(FusedArgs a)
{
    typedef FusedCfg<KC> G;
    __shared__ __align__(1024) char S[G::kBytes];
    const int t = (int)threadIdx.x, lane = t & 63, h = lane >> 5;
    const int w = __builtin_amdgcn_readfirstlane(t >> 6);
    const int n0 = (int)blockIdx.x * kFusedCols;
    const void* z = g_zeros;
    const unsigned lds = lds_address(S) + w * 1024;
    char* X = S + 2 * G::kStage;

    // Weights of a stage: chunk ch of Wg and Wu, and chunk ch - 1 of Wd.
    constexpr int JW = (G::kW + 4095) / 4096, JD = (G::kD + 4095) / 4096;
    const __bf16 *pg[JW], *pu[JW], *pd[JD];
    bool okw[JW], okd[JD];
    int fr[JW], fc[JD];  // hidden rows and columns of this thread's pieces inside a chunk
#pragma unroll
    for (int j = 0; j < JW; ++j) {
        const int e = j * 256 + t, row = e / G::PR, c = ((e % G::PR) ^ piece_swizzle<G::PR>(row)) * 8;
        fr[j] = row;
        okw[j] = c < a.C;
        pg[j] = a.wg + row * a.ldw + c;
        pu[j] = a.wu + row * a.ldw + c;
    }
#pragma unroll
    for (int j = 0; j < JD; ++j) {
        const int e = j * 256 + t, row = e >> 2;
        fc[j] = ((e & 3) ^ ((row >> 2) & 3)) * 8;
        okd[j] = row < a.C;
        pd[j] = a.wd + row * a.ldd + fc[j];
    }
    const auto issue = [&](int ch, int buf) {
        const unsigned d = lds + buf * G::kStage;
        if (ch * 32 < a.F) {
            const bool full = ch * 32 + 32 <= a.F;
#pragma unroll
            for (int j = 0; j < JW; ++j) {
                const bool ok = okw[j] && (full || ch * 32 + fr[j] < a.F);
                if (G::kW - j * 4096 >= 4096 || w < (G::kW - j * 4096) / 1024) {
                    to_lds(ok ? (const void*)pg[j] : z, d + j * 4096);
                    to_lds(ok ? (const void*)pu[j] : z, d + G::kW + j * 4096);
                }
                pg[j] += 32 * a.ldw;
                pu[j] += 32 * a.ldw;
            }
        }
        if (ch > 0) {
            const bool full = ch * 32 <= a.F;
#pragma unroll
            for (int j = 0; j < JD; ++j) {
                const bool ok = okd[j] && (full || ch * 32 - 32 + fc[j] < a.F);
                if (G::kD - j * 4096 >= 4096 || w < (G::kD - j * 4096) / 1024)
                    to_lds(ok ? (const void*)pd[j] : z, d + 2 * G::kW + j * 4096);
                pd[j] += 32;
            }
        }
    };

    // x tile: [channel][128 positions], pieces swizzled for the transposing read.
#pragma unroll
    for (int j = 0; j < G::kX / 4096; ++j) {
        const int e = j * 256 + t, k = e >> 4, c = (e & 15) ^ ((k & 3) << 2);
        int n = n0 + c * 8;
        n = n < a.N ? n : 0;
        const int q = n / a.mx.L;
        const __bf16* p = a.x + (long long)k * a.mx.ld + q * a.mx.sb + (n - q * a.mx.L);
        to_lds(k < a.C ? (const void*)p : z, lds + 2 * G::kStage + j * 4096);
    }
    issue(0, 0);
    wait_loads();
    __syncthreads();
    bf16x8 xb[2 * KC];
    {
        const int i = lane & 15;
        const char* q = X + (8 * h + (i >> 2)) * 256 + ((w ^ (i >> 2)) << 6) + ((lane >> 4) & 1) * 32 + (i & 3) * 8;
#pragma unroll
        for (int ks = 0; ks < 2 * KC; ++ks) {
            typedef __attribute__((address_space(3))) s16x4 lds4;
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(q + ks * 4096));
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(q + ks * 4096 + 1024));
            xb[ks] = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        }
    }
    const int r32 = lane & 31, row = (r32 & 19) | ((r32 & 4) << 1) | ((r32 & 8) >> 1);  // bits 2 and 3 exchanged
    const int swz = piece_swizzle<G::PR>(row);
    f32x16 y[KC] = {};
    const int chunks = (a.F + 31) / 32;
    const char *sw = S + row * (G::PR * 16), *sd = S + 2 * G::kW + r32 * 64;
    int ow[2 * KC];  // offsets of the pieces of a weight row
#pragma unroll
    for (int ks = 0; ks < 2 * KC; ++ks) ow[ks] = ((2 * ks + h) ^ swz) << 4;
    const int od = (h ^ ((r32 >> 2) & 3)) << 4;
    struct Hidden {
        f32x16 g, u;
    };
    const auto product = [&](auto buf) {
        Hidden v{};
#pragma unroll
        for (int ks = 0; ks < 2 * KC; ++ks) {
            const char* q = sw + buf * G::kStage + ow[ks];
            v.g = __builtin_amdgcn_mfma_f32_32x32x16_bf16(*reinterpret_cast<const bf16x8*>(q), xb[ks], v.g, 0, 0, 0);
            v.u = __builtin_amdgcn_mfma_f32_32x32x16_bf16(*reinterpret_cast<const bf16x8*>(q + G::kW), xb[ks], v.u, 0, 0, 0);
        }
        return v;
    };
    const auto down = [&](auto buf, const bf16x8 (&hb)[2]) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int c = 0; c < KC; ++c)
                y[c] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                    *reinterpret_cast<const bf16x8*>(sd + buf * G::kStage + c * 2048 + (od ^ (s << 5))), hb[s], y[c], 0, 0, 0);
    };
    constexpr std::integral_constant<int, 0> b0{};
    constexpr std::integral_constant<int, 1> b1{};
    with_act(a.act, [&](auto act) {
        const auto hidden = [&](const Hidden& v, bf16x8 (&hb)[2]) {
#pragma unroll
            for (int e = 0; e < 16; ++e) hb[e >> 3][e & 7] = (__bf16)(act_fwd(act, v.g[e]) * v.u[e]);
        };
        // Chunk ch: its activation beside the next chunk's products (independent,
        // so the vector and the matrix instructions interleave), then its share of y.
        const auto step = [&](int ch, auto buf, const Hidden& cur, Hidden& next) {
            wait_loads();
            __syncthreads();  // the stage has arrived; the other one is no longer read
            if (ch + 2 <= chunks) issue(ch + 2, 1 - buf);
            bf16x8 hb[2];
            next = product(buf);
            hidden(cur, hb);
            down(buf, hb);
            // Four fragments ahead, then one multiplication, five vector instructions and
            // one read at a time (left alone the compiler bunches each kind; 967 -> 943 us).
            __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
#pragma unroll
            for (int i = 0; i < 4 * KC + 2 * KC - 4; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x2, 5, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            }
        };
        const auto last = [&](auto buf, const Hidden& cur) {
            wait_loads();
            __syncthreads();
            bf16x8 hb[2];
            hidden(cur, hb);
            down(buf, hb);
        };
        issue(1, 1);
        Hidden v0 = product(b0), v1;
        int ch = 0;
        for (; ch + 2 < chunks; ch += 2) {
            step(ch, b1, v0, v1);
            step(ch + 1, b0, v1, v0);
        }
        if (ch + 1 < chunks) {
            step(ch, b1, v0, v1);
            last(b0, v1);
        } else {
            last(b1, v0);
        }
    });
    // y through LDS: rows of channels, 16 bytes a lane.
    __syncthreads();
    constexpr int LD = kFusedCols * 2 + 16;
#pragma unroll
    for (int c = 0; c < KC; ++c)
#pragma unroll
        for (int i = 0; i < 16; ++i)
            *reinterpret_cast<__bf16*>(S + (c * 32 + 8 * (i >> 2) + 4 * h + (i & 3)) * LD + (w * 32 + r32) * 2) =
                (__bf16)y[c][i];
    __syncthreads();
#pragma unroll 2
    for (int e = t; e < KC * 32 * 16; e += 256) {
        const int c = e >> 4, n = n0 + (e & 15) * 8;
        if (c >= a.C || n >= a.N) continue;
        const u32x4 v = *reinterpret_cast<const u32x4*>(S + c * LD + (e & 15) * 16);
        __bf16* r = (__bf16*)a.y + (long long)c * a.ldo;
        const int q = n / a.oL, l = n - q * a.oL;
        if (n + 8 <= a.N && l + 8 <= a.oL) {
            WordsMem<4, 2> m;
#pragma unroll
            for (int i = 0; i < 4; ++i) m.w[i] = v[i];
            *reinterpret_cast<WordsMem<4, 2>*>(r + q * a.osb + l) = m;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int cn = n + i, qq = cn / a.oL;
                if (cn < a.N)
                    *reinterpret_cast<unsigned short*>(r + qq * a.osb + (cn - qq * a.oL)) =
                        (unsigned short)(i & 1 ? v[i >> 1] >> 16 : v[i >> 1]);
            }
        }
    }
}

}  // namespace

hipError_t launch_ffn_fused(const FusedFfn& f, hipStream_t st)
{
    FusedArgs a{};
    a.x = (const __bf16*)f.x;
    a.wg = (const __bf16*)f.wg;
    a.wu = (const __bf16*)f.wu;
    a.wd = (const __bf16*)f.wd;
    a.y = f.y;
    a.mx = Mat{f.ldx, f.sbx, 0, f.Lx};
    a.ldw = f.ldw;
    a.ldd = f.ldd;
    a.C = f.C;
    a.F = f.F;
    a.N = f.N;
    a.act = f.act;
    a.ldo = f.ldo;
    a.osb = f.osb;
    a.oL = f.oL;
    const dim3 grid((unsigned)((f.N + kFusedCols - 1) / kFusedCols));
    if (f.C <= 32) hipLaunchKernelGGL((k_ffn_fused<1>), grid, dim3(256), 0, st, a);
    else if (f.C <= 64) hipLaunchKernelGGL((k_ffn_fused<2>), grid, dim3(256), 0, st, a);
    else if (f.C <= 96) hipLaunchKernelGGL((k_ffn_fused<3>), grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL((k_ffn_fused<4>), grid, dim3(256), 0, st, a);
    return launch_status();
}

}  // namespace hyenand
