// api_block.cpp -- the C ABI of the residual block's operators (norm, join,
// dropout, gated feed-forward): argument validation, workspace sizes, launch
// and error mapping.
#include <hip/hip_runtime.h>

#include <cfloat>
#include <cmath>

#include "../../include/hyenand.h"
#include "block.h"
#include "launch.h"

using namespace hyenand;

namespace {

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

constexpr long long kMaxElems = 1ll << 60;

// Positions of one batch entry; false for a null or negative extent or a
// product that leaves 64 bits once multiplied out.
bool positions(int B, int C, int d, const int64_t* dims, long long* L)
{
    long long n = 1;
    bool zero = false;
    for (int i = 0; i < d; ++i) {
        if (dims[i] < 0) return false;
        if (dims[i] == 0) zero = true;
        else if (n > kMaxElems / dims[i]) return false;
        else n *= dims[i];
    }
    *L = zero ? 0 : n;
    const long long pairs = (long long)(B > 0 ? B : 1) * (C > 0 ? C : 1);
    return zero || n <= kMaxElems / pairs;
}

// The checks every entry point shares.
int common(int B, int C, int d, const int64_t* dims, int dtype, long long* L)
{
    if (B < 0 || C < 0) return HYENAND_ERR_INVALID_ARG;
    if (dtype != HYENAND_F32 && dtype != HYENAND_BF16) return HYENAND_ERR_INVALID_ARG;
    if (d < 1 || d > 3) return HYENAND_ERR_UNSUPPORTED;
    if (!dims) return HYENAND_ERR_INVALID_ARG;
    for (int i = 0; i < d; ++i)
        if (dims[i] < 0) return HYENAND_ERR_INVALID_ARG;
    if (!positions(B, C, d, dims, L)) return HYENAND_ERR_UNSUPPORTED;
    return HYENAND_OK;
}

// A normal positive number: the hardware's reciprocal square root takes no others.
int checked_eps(float eps)
{
    return eps >= FLT_MIN && std::isfinite(eps) ? HYENAND_OK : HYENAND_ERR_INVALID_ARG;
}

// Dropout probability and generator; p = 0 draws nothing.
int drop_args(double p, const void* rng, DropArgs* d)
{
    *d = DropArgs{nullptr, 0, 1.0f};
    if (!(p >= 0.0 && p < 1.0)) return HYENAND_ERR_INVALID_ARG;
    if (p == 0.0) return HYENAND_OK;
    if (!rng || !aligned(rng, 8)) return HYENAND_ERR_INVALID_ARG;
    d->rng = static_cast<const unsigned long long*>(rng);
    d->thr = (unsigned)(p * 4294967296.0);
    d->up = (float)(1.0 / (1.0 - p));
    return HYENAND_OK;
}

bool bad(const void* p, size_t a) { return !p || !aligned(p, a); }
bool bad_opt(const void* p, size_t a) { return p && !aligned(p, a); }

size_t parts_bytes(int B, int C, long long L)
{
    return B <= 0 || C <= 0 || L <= 0 ? 0 : (size_t)block_parts(C) * 2u * (size_t)C * sizeof(float);
}

size_t part_workspace(int B, int C, int d, const int64_t* dims, int dtype)
{
    long long L;
    if (common(B, C, d, dims, dtype, &L) != HYENAND_OK || C > kBlockMaxC) return 0;
    return parts_bytes(B, C, L);
}

int check_ws(void* ws, size_t have, size_t need, size_t align)
{
    if (need == 0) return HYENAND_OK;
    if (!ws || have < need) return HYENAND_ERR_WORKSPACE;
    return aligned(ws, align) ? HYENAND_OK : HYENAND_ERR_INVALID_ARG;
}

// The gate, scales and dropout of a join.
int join_args(const hyenand_join* j, size_t es, BlockArgs* a)
{
    if (!j) return HYENAND_ERR_INVALID_ARG;
    if (j->gate_act != HYENAND_ACT_NONE && j->gate_act != HYENAND_ACT_SIGMOID && j->gate_act != HYENAND_ACT_SILU)
        return HYENAND_ERR_INVALID_ARG;
    if (checked_eps(j->eps) != HYENAND_OK) return HYENAND_ERR_INVALID_ARG;
    if (bad_opt(j->gate, es) || bad_opt(j->scale, 4) || bad_opt(j->w_post, 4) || bad_opt(j->w_pre, 4))
        return HYENAND_ERR_INVALID_ARG;
    a->gate = j->gate;
    a->scale = j->scale;
    a->w_post = j->w_post;
    a->w_pre = j->w_pre;
    a->act = j->gate_act;
    a->eps = j->eps;
    return drop_args(j->p, j->rng, &a->drop);
}

void shape(BlockArgs* a, int B, int C, long long L, int dtype)
{
    a->B = B;
    a->C = C;
    a->L = L;
    a->bf16 = dtype == HYENAND_BF16;
}

int zero(float* p, int n, hipStream_t st)
{
    return !p || launch_zero(p, n, st) == hipSuccess ? HYENAND_OK : HYENAND_ERR_HIP;
}

// The checks of the gated feed-forward entry points.
int ffn_check(int B, int C, int F, int d, const int64_t* dims, int dtype, int act, long long* L)
{
    const int rc = common(B, C, d, dims, dtype, L);
    if (rc != HYENAND_OK) return rc;
    if (F < 1) return HYENAND_ERR_INVALID_ARG;
    if (act != HYENAND_ACT_SIGMOID && act != HYENAND_ACT_SILU && act != HYENAND_ACT_GELU)
        return HYENAND_ERR_INVALID_ARG;
    if (C > HYENAND_FFN_MAX_WIDTH || F > HYENAND_FFN_MAX_WIDTH) return HYENAND_ERR_UNSUPPORTED;
    if ((long long)B > 0 && *L > HYENAND_FFN_MAX_POSITIONS / B) return HYENAND_ERR_UNSUPPORTED;
    return HYENAND_OK;
}

size_t ffn_ws(int B, int C, int F, int d, const int64_t* dims, int dtype, bool bwd)
{
    long long L;
    if (ffn_check(B, C, F, d, dims, dtype, HYENAND_ACT_SILU, &L) != HYENAND_OK || B == 0 || C == 0 || L == 0) return 0;
    return ffn_workspace(B, C, F, L, dtype == HYENAND_BF16, bwd);
}

}  // namespace

extern "C" {

int hyenand_block_norm_fwd(const void* x, const float* w, void* h, int B, int C, int d, const int64_t* dims, int dtype,
                           float eps, void* stream)
{
    long long L;
    const int rc = common(B, C, d, dims, dtype, &L);
    if (rc != HYENAND_OK) return rc;
    if (checked_eps(eps) != HYENAND_OK) return HYENAND_ERR_INVALID_ARG;
    if (C > kBlockMaxC) return HYENAND_ERR_UNSUPPORTED;
    if (B == 0 || C == 0 || L == 0) return HYENAND_OK;
    const size_t es = dtype == HYENAND_BF16 ? 2 : 4;
    if (bad(x, es) || bad(h, es) || bad(w, 4)) return HYENAND_ERR_INVALID_ARG;
    BlockArgs a{};
    shape(&a, B, C, L, dtype);
    a.x = x;
    a.w_pre = w;
    a.h = h;
    a.eps = eps;
    return launch_block_fwd(a, static_cast<hipStream_t>(stream)) == hipSuccess ? HYENAND_OK : HYENAND_ERR_HIP;
}

size_t hyenand_block_norm_bwd_workspace_bytes(int B, int C, int d, const int64_t* dims, int dtype)
{
    return part_workspace(B, C, d, dims, dtype);
}

int hyenand_block_norm_bwd(const void* x, const float* w, const void* dh, void* dx, float* dw, int B, int C, int d,
                           const int64_t* dims, int dtype, float eps, void* workspace, size_t workspace_bytes,
                           void* stream)
{
    long long L;
    int rc = common(B, C, d, dims, dtype, &L);
    if (rc != HYENAND_OK) return rc;
    if (checked_eps(eps) != HYENAND_OK) return HYENAND_ERR_INVALID_ARG;
    if (C > kBlockMaxC) return HYENAND_ERR_UNSUPPORTED;
    if (C == 0) return HYENAND_OK;
    if (bad(dw, 4)) return HYENAND_ERR_INVALID_ARG;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (B == 0 || L == 0) return zero(dw, C, st);
    const size_t es = dtype == HYENAND_BF16 ? 2 : 4;
    if (bad(x, es) || bad(dh, es) || bad(dx, es) || bad(w, 4)) return HYENAND_ERR_INVALID_ARG;
    if ((rc = check_ws(workspace, workspace_bytes, parts_bytes(B, C, L), 4)) != HYENAND_OK) return rc;
    BlockArgs a{};
    shape(&a, B, C, L, dtype);
    a.x = x;
    a.dh = dh;
    a.dx = dx;
    a.w_pre = w;
    a.dw_pre = dw;
    a.eps = eps;
    a.part = static_cast<float*>(workspace);
    return launch_block_bwd(a, st) == hipSuccess ? HYENAND_OK : HYENAND_ERR_HIP;
}

int hyenand_block_join_fwd(const void* x, const void* m, const hyenand_join* j, void* out, void* h, int B, int C,
                           int d, const int64_t* dims, int dtype, void* stream)
{
    long long L;
    int rc = common(B, C, d, dims, dtype, &L);
    if (rc != HYENAND_OK) return rc;
    const size_t es = dtype == HYENAND_BF16 ? 2 : 4;
    BlockArgs a{};
    if ((rc = join_args(j, es, &a)) != HYENAND_OK) return rc;
    if (C > kBlockMaxC) return HYENAND_ERR_UNSUPPORTED;
    if (B == 0 || C == 0 || L == 0) return HYENAND_OK;
    if (bad(x, es) || bad(m, es) || bad(out, es)) return HYENAND_ERR_INVALID_ARG;
    if (j->w_pre ? bad(h, es) : h != nullptr) return HYENAND_ERR_INVALID_ARG;
    shape(&a, B, C, L, dtype);
    a.x = x;
    a.m = m;
    a.out = out;
    a.h = h;
    return launch_block_fwd(a, static_cast<hipStream_t>(stream)) == hipSuccess ? HYENAND_OK : HYENAND_ERR_HIP;
}

size_t hyenand_block_join_bwd_workspace_bytes(int B, int C, int d, const int64_t* dims, int dtype)
{
    return part_workspace(B, C, d, dims, dtype);
}

int hyenand_block_join_bwd(const void* x, const void* m, const hyenand_join* j, const void* dout, const void* dh,
                           const hyenand_join_grads* grads, int B, int C, int d, const int64_t* dims, int dtype,
                           void* workspace, size_t workspace_bytes, void* stream)
{
    long long L;
    int rc = common(B, C, d, dims, dtype, &L);
    if (rc != HYENAND_OK) return rc;
    const size_t es = dtype == HYENAND_BF16 ? 2 : 4;
    BlockArgs a{};
    if ((rc = join_args(j, es, &a)) != HYENAND_OK) return rc;
    if (!grads) return HYENAND_ERR_INVALID_ARG;
    if (C > kBlockMaxC) return HYENAND_ERR_UNSUPPORTED;
    if (C == 0) return HYENAND_OK;
    const hyenand_join_grads& g = *grads;
    // A gradient is asked for exactly where the forward has the input.
    if (j->scale ? bad(g.dscale, 4) : g.dscale != nullptr) return HYENAND_ERR_INVALID_ARG;
    if (j->w_post ? bad(g.dw_post, 4) : g.dw_post != nullptr) return HYENAND_ERR_INVALID_ARG;
    if (j->w_pre ? bad(g.dw_pre, 4) : g.dw_pre != nullptr) return HYENAND_ERR_INVALID_ARG;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (B == 0 || L == 0) {
        if ((rc = zero(g.dscale, C, st)) != HYENAND_OK || (rc = zero(g.dw_post, C, st)) != HYENAND_OK) return rc;
        return zero(g.dw_pre, C, st);
    }
    if (bad(x, es) || bad(m, es) || bad_opt(dout, es) || bad_opt(dh, es) || bad(g.dx, es) || bad(g.dm, es))
        return HYENAND_ERR_INVALID_ARG;
    if (!j->w_pre && dh) return HYENAND_ERR_INVALID_ARG;
    if (j->gate ? bad(g.dgate, es) : g.dgate != nullptr) return HYENAND_ERR_INVALID_ARG;
    if ((rc = check_ws(workspace, workspace_bytes, parts_bytes(B, C, L), 4)) != HYENAND_OK) return rc;
    shape(&a, B, C, L, dtype);
    a.x = x;
    a.m = m;
    a.dout = dout;
    a.dh = dh;
    a.dx = g.dx;
    a.dm = g.dm;
    a.dgate = g.dgate;
    a.dscale = g.dscale;
    a.dw_post = g.dw_post;
    a.dw_pre = g.dw_pre;
    a.part = static_cast<float*>(workspace);
    return launch_block_bwd(a, st) == hipSuccess ? HYENAND_OK : HYENAND_ERR_HIP;
}

int hyenand_dropout(const void* x, void* y, int64_t n, int dtype, double p, const uint64_t* rng, void* stream)
{
    if (n < 0 || (dtype != HYENAND_F32 && dtype != HYENAND_BF16)) return HYENAND_ERR_INVALID_ARG;
    DropArgs d;
    const int rc = drop_args(p, rng, &d);
    if (rc != HYENAND_OK) return rc;
    if (n > HYENAND_DROPOUT_MAX_ELEMENTS) return HYENAND_ERR_UNSUPPORTED;
    if (n == 0) return HYENAND_OK;
    const size_t es = dtype == HYENAND_BF16 ? 2 : 4;
    if (bad(x, es) || bad(y, es)) return HYENAND_ERR_INVALID_ARG;
    return launch_dropout(x, y, n, dtype == HYENAND_BF16, d, static_cast<hipStream_t>(stream)) == hipSuccess
               ? HYENAND_OK
               : HYENAND_ERR_HIP;
}

size_t hyenand_gated_ffn_workspace_bytes(int B, int C, int F, int d, const int64_t* dims, int dtype)
{
    return ffn_ws(B, C, F, d, dims, dtype, false);
}

size_t hyenand_gated_ffn_bwd_workspace_bytes(int B, int C, int F, int d, const int64_t* dims, int dtype)
{
    return ffn_ws(B, C, F, d, dims, dtype, true);
}

int hyenand_gated_ffn_fwd(const void* x, const void* Wg, const void* Wu, const void* Wd, void* y, int B, int C, int F,
                          int d, const int64_t* dims, int dtype, int act, void* workspace, size_t workspace_bytes,
                          void* stream)
{
    long long L;
    int rc = ffn_check(B, C, F, d, dims, dtype, act, &L);
    if (rc != HYENAND_OK) return rc;
    if (B == 0 || C == 0 || L == 0) return HYENAND_OK;
    if (bad(x, 16) || bad(y, 16) || bad(Wg, 16) || bad(Wu, 16) || bad(Wd, 16)) return HYENAND_ERR_INVALID_ARG;
    const bool bf16 = dtype == HYENAND_BF16;
    if ((rc = check_ws(workspace, workspace_bytes, ffn_workspace(B, C, F, L, bf16, false), 256)) != HYENAND_OK)
        return rc;
    FfnArgs a{};
    a.x = x;
    a.Wg = Wg;
    a.Wu = Wu;
    a.Wd = Wd;
    a.y = y;
    a.ws = workspace;
    a.act = act;
    a.B = B;
    a.C = C;
    a.F = F;
    a.L = L;
    a.bf16 = bf16;
    return launch_ffn_fwd(a, static_cast<hipStream_t>(stream)) == hipSuccess ? HYENAND_OK : HYENAND_ERR_HIP;
}

int hyenand_gated_ffn_bwd(const void* x, const void* Wg, const void* Wu, const void* Wd, const void* dy, void* dx,
                          void* dWg, void* dWu, void* dWd, int B, int C, int F, int d, const int64_t* dims, int dtype,
                          int act, void* workspace, size_t workspace_bytes, void* stream)
{
    long long L;
    int rc = ffn_check(B, C, F, d, dims, dtype, act, &L);
    if (rc != HYENAND_OK) return rc;
    if (C == 0) return HYENAND_OK;
    if (bad(dWg, 16) || bad(dWu, 16) || bad(dWd, 16)) return HYENAND_ERR_INVALID_ARG;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const bool bf16 = dtype == HYENAND_BF16;
    if (B == 0 || L == 0) {
        // Sums over no positions.
        const long long n = (long long)C * F;
        void* const dw[3] = {dWg, dWu, dWd};
        for (void* p : dw)
            if (launch_ffn_zero(p, n * (bf16 ? 2 : 4), st) != hipSuccess) return HYENAND_ERR_HIP;
        return HYENAND_OK;
    }
    if (bad(x, 16) || bad(dy, 16) || bad(dx, 16) || bad(Wg, 16) || bad(Wu, 16) || bad(Wd, 16))
        return HYENAND_ERR_INVALID_ARG;
    if ((rc = check_ws(workspace, workspace_bytes, ffn_workspace(B, C, F, L, bf16, true), 256)) != HYENAND_OK)
        return rc;
    FfnArgs a{};
    a.x = x;
    a.Wg = Wg;
    a.Wu = Wu;
    a.Wd = Wd;
    a.dy = dy;
    a.dx = dx;
    a.dWg = dWg;
    a.dWu = dWu;
    a.dWd = dWd;
    a.ws = workspace;
    a.act = act;
    a.B = B;
    a.C = C;
    a.F = F;
    a.L = L;
    a.bf16 = bf16;
    return launch_ffn_bwd(a, st) == hipSuccess ? HYENAND_OK : HYENAND_ERR_HIP;
}

}  // extern "C"
