// block.h -- arguments and launchers of the residual block's operators (norm,
// join, dropout, gated feed-forward).  The launchers validate nothing (the C
// ABI does) and return hipSuccess or the launch error.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

namespace hyenand {

// Dropout: an element is kept iff its random word is >= thr; kept values are
// multiplied by `up` = 1 / (1 - p).
struct DropArgs {
    const unsigned long long* rng;  // device {seed, offset}; null: no dropout
    unsigned thr;
    float up;
};

// Norm (m == null: out is x itself and is not written) and join, forward and
// backward.  Tensors are [B][C][L].
struct BlockArgs {
    const void *x, *m, *gate, *dout, *dh;
    const float *scale, *w_post, *w_pre;
    void *out, *h, *dx, *dm, *dgate;
    float *dscale, *dw_post, *dw_pre;
    float* part;  // [workgroups][2][C] partial sums of the channel gradients (backward)
    DropArgs drop;
    float eps;
    int act;
    int B, C;
    long long L;
    bool bf16;
};

constexpr int kBlockMaxC = 8192;      // channels of a norm or join (held in registers by one workgroup)
// Workgroups of a backward launch, at most; up to eight channels may take
// workgroups of a wave.
constexpr int kFewChannels = 8;
constexpr int block_parts(int C) { return C <= kFewChannels ? 4096 : 1024; }

hipError_t launch_block_fwd(const BlockArgs& a, hipStream_t st);
hipError_t launch_block_bwd(const BlockArgs& a, hipStream_t st);
hipError_t launch_dropout(const void* x, void* y, long long n, bool bf16, const DropArgs& d, hipStream_t st);

// Gated feed-forward: h = act(Wg x) (Wu x), y = Wd h per position.
struct FfnArgs {
    const void *x, *Wg, *Wu, *Wd, *dy;
    void *y, *dx, *dWg, *dWu, *dWd;
    void* ws;
    int act;
    int B, C, F;
    long long L;
    bool bf16;
};

// The one-launch forward for few channels (bf16, at most kFusedMaxC): operands in
// rows of 16-byte multiples, x and y as in FfnArgs or packed.
constexpr int kFusedMaxC = 128;
struct FusedFfn {
    const void *x, *wg, *wu, *wd;
    void* y;
    long long ldx, sbx;  // x: element (c, n) at c ldx + (n / Lx) sbx + n % Lx
    int Lx;
    long long ldw, ldd;  // row strides of Wg / Wu and Wd
    int C, F, N, act;
    long long ldo, osb;  // y likewise
    int oL;
};
hipError_t launch_ffn_fused(const FusedFfn& f, hipStream_t st);

// The forward for few positions, straight from the caller's weights.
constexpr int kFewPositions = 64;
hipError_t launch_ffn_few(const FfnArgs& a, hipStream_t st);

size_t ffn_workspace(int B, int C, int F, long long L, bool bf16, bool bwd);
hipError_t launch_ffn_fwd(const FfnArgs& a, hipStream_t st);
hipError_t launch_ffn_bwd(const FfnArgs& a, hipStream_t st);
// Zero fill of an even number of bytes at a 2-byte aligned address.
hipError_t launch_ffn_zero(void* p, long long bytes, hipStream_t st);

}  // namespace hyenand
