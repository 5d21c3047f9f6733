// The C ABI of the selective scan: argument checks, the sequence split, workspace layout and launch order.
#include <cstring>

#include "gla_span.h"
#include "gla_ssm.cuh"

namespace gla {
namespace {

constexpr int kStepT = 8;            // the longest call that gla_ssm_step takes
constexpr int kMaxSegments = 1024;

size_t align_up(size_t x) { return (x + 255) / 256 * 256; }

gla_status check(const gla_ssm_params* p)
{
    if (!p || p->B <= 0 || p->T < 0 || p->D <= 0 || p->G <= 0 || p->N <= 0) return GLA_ERR_INVALID_ARG;
    if (p->D % p->G != 0 || p->D / p->G % 8 != 0) return GLA_ERR_INVALID_ARG;
    if (p->dtype != GLA_BF16 && p->dtype != GLA_FP32) return GLA_ERR_INVALID_ARG;
    if (p->force_segments < 0 || !p->A) return GLA_ERR_INVALID_ARG;
    if (p->T > 0 && (!p->x || !p->dt || !p->Bm || !p->Cm)) return GLA_ERR_INVALID_ARG;
    const size_t e = p->dtype == GLA_BF16 ? 2 : 4;
    for (const long long* s : {p->x_stride, p->dt_stride, p->z_stride, p->B_stride, p->C_stride})
        for (int i = 0; i < 2; ++i)
            if (s[i] * (long long)e % 16 != 0) return GLA_ERR_INVALID_ARG;   // every row starts on 16 bytes
    for (const void* x : {p->x, p->dt, p->z, p->Bm, p->Cm, (const void*)p->A, (const void*)p->S0})
        if (!aligned(x, 16)) return GLA_ERR_INVALID_ARG;
    if (!aligned(p->D_skip, 4) || !aligned(p->dt_bias, 4)) return GLA_ERR_INVALID_ARG;
    if (p->N != 8 && p->N != 16 && p->N != 32 && p->N != 64) return GLA_ERR_UNSUPPORTED;
    if (p->D > (1 << 20) || p->T > (1 << 30) || (long long)p->B * p->D > (1LL << 30) ||
        (long long)p->B * p->T > (1LL << 40) / p->D)
        return GLA_ERR_UNSUPPORTED;
    return GLA_OK;
}

struct SsmPlan {
    int nseg = 1, seg = 0;
    size_t off_sumd = 0, off_s0 = 0, off_segG = 0, off_keep = 0, off_bc = 0, off_p = 0, ws = 0;
};

// Segments of the sequence. A walk is serial over its tokens, so few blocks leave SMs idle; cut, they fill the chip evenly, but
// the tokens are walked twice (backward: three times more in part). Uncut, a walk of up to 1.7 blocks an SM takes 0.08 us a token, 0.107 at
// 2.5, 0.11 at 3.4; cut so that there are twenty blocks an SM in all, 2.6e-4 us a block: equal at 2.7 an SM (rows of
// 4096 channels of 16 states: one of 16421 tokens 1292 us uncut, 582 in 8 segments, 562 in 23; three of 4096 439
// uncut, 404 in 8). The backward's larger blocks take 0.28 us a token up to one an SM and 0.42 up to two, and 2e-3 us each when
// cut so that there are seven an SM: equal at 1.4 an SM (one row of 2048 tokens 567 us uncut, 295 in 16; two 600 and 519). Segments
// are four tiles or more (two rows of 2048 tokens of 1536 channels of 8 states: 52 us in 32 segments, 60 in 64), two where the chip
// is not filled otherwise (one row of 256 tokens of 1024 channels: 24 us uncut, 13 in 8, 15 in 16).
void split(const gla_ssm_params* p, int sms, bool bwd, SsmPlan& pl)
{
    const int CB = bwd ? ssm_bwd_channels(p->N) : ssm_walk_channels(p->N);
    const long long blocks = (long long)p->B * p->G * ((p->D / p->G + CB - 1) / CB);
    const long long tiles = ((long long)p->T + kSsmTile - 1) / kSsmTile;
    long long n = p->force_segments;
    if (n == 0) {
        const long long units = bwd ? blocks : blocks * ssm_walk_warps(p->N) / 2;    // (blocks of two warps)
        n = 10 * units < (bwd ? 14LL : 27LL) * sms ? (bwd ? 7LL : 20LL) * sms / units : 1;
        const long long filled = 7LL * sms / units, most = tiles / 2 < filled ? tiles / 2 : filled;
        if (n > tiles / 4) n = most > tiles / 4 ? most : tiles / 4;
    }
    if (n > kMaxSegments) n = kMaxSegments;
    if (n > tiles) n = tiles;
    if (n < 1) n = 1;
    long long per = (tiles + n - 1) / n;
    if (per > 1 && per < tiles) per += per % 2;      // (the walks load two tiles at a time)
    pl.nseg = per > 0 ? (int)((tiles + per - 1) / per) : 1;
    if (pl.nseg < 1) pl.nseg = 1;
    pl.seg = per > 0 ? (int)(per * kSsmTile) : kSsmTile;
    const size_t states = (size_t)p->B * p->D * p->N * 4;
    if (pl.nseg > 1) {
        pl.off_sumd = pl.ws + align_up((pl.nseg - 1) * states);
        pl.ws = pl.off_sumd + align_up((size_t)(pl.nseg - 1) * p->B * p->D * 4);
    }
    if (!bwd && pl.nseg > 1) {
        pl.off_s0 = pl.ws;
        pl.ws += align_up(states);
    }
    if (bwd) {
        pl.off_segG = pl.ws;
        if (pl.nseg > 1) pl.ws += align_up((pl.nseg - 1) * states);
        pl.off_keep = pl.ws;
        pl.ws += align_up((size_t)tiles * states);
        pl.off_bc = pl.ws;
        pl.ws += align_up((size_t)((p->D / p->G + CB - 1) / CB) * p->B * p->T * p->G * 2 * p->N * 4);
        pl.off_p = pl.ws;
        pl.ws += align_up((size_t)p->B * pl.nseg * ((size_t)p->D * p->N + 2 * p->D) * 4);
    }
}

SsmArgs common(const gla_ssm_params* p, const SsmPlan& pl, void* ws)
{
    SsmArgs a;
    std::memset(&a, 0, sizeof(a));
    a.x = p->x; a.dt = p->dt; a.z = p->z; a.Bm = p->Bm; a.Cm = p->Cm;
    for (int i = 0; i < 2; ++i) {
        a.sx[i] = p->x_stride[i]; a.sdt[i] = p->dt_stride[i]; a.sz[i] = p->z_stride[i];
        a.sB[i] = p->B_stride[i]; a.sC[i] = p->C_stride[i];
    }
    a.A = p->A; a.Dk = p->D_skip; a.bias = p->dt_bias; a.S0 = p->S0;
    a.B = p->B; a.T = p->T; a.D = p->D; a.G = p->G; a.N = p->N; a.softplus = p->softplus != 0;
    a.nseg = pl.nseg; a.seg = pl.seg;
    char* w = static_cast<char*>(ws);
    a.segS = reinterpret_cast<float*>(w);
    a.sumd = reinterpret_cast<float*>(w + pl.off_sumd);
    return a;
}

struct Inputs { Span s[9]; };
Inputs inputs_of(const gla_ssm_params* p)
{
    const size_t e = p->dtype == GLA_BF16 ? 2 : 4;
    auto rows = [&](const void* q, const long long* st, int n) {
        const long long s[3] = {st[0], 0, st[1]};
        return span(q, s, p->B, 1, p->T, n, e);
    };
    return Inputs{{rows(p->x, p->x_stride, p->D), rows(p->dt, p->dt_stride, p->D), rows(p->z, p->z_stride, p->D),
                   rows(p->Bm, p->B_stride, p->G * p->N), rows(p->Cm, p->C_stride, p->G * p->N),
                   flat(p->A, (size_t)p->D * p->N * 4), flat(p->D_skip, (size_t)p->D * 4), flat(p->dt_bias, (size_t)p->D * 4),
                   flat(p->S0, (size_t)p->B * p->D * p->N * 4)}};
}

gla_status cuda(cudaError_t r) { return r == cudaSuccess ? GLA_OK : GLA_ERR_CUDA; }

}  // namespace
}  // namespace gla

using namespace gla;

extern "C" {

size_t gla_ssm_fwd_workspace_size(const gla_ssm_params* p)
{
    int sms = 0;
    if (check(p) != GLA_OK) return 0;
    if (device_ready(&sms) != GLA_OK) sms = 152;
    SsmPlan pl;
    split(p, sms, false, pl);
    return p->T <= kStepT && p->force_segments == 0 ? 0 : pl.ws;
}

gla_status gla_ssm_fwd(const gla_ssm_params* p, void* y, float* ST, void* workspace, size_t workspace_bytes, cudaStream_t stream)
{
    gla_status st = check(p);
    if (st != GLA_OK) return st;
    if ((p->T > 0 && !y) || !aligned(y, 16) || !aligned(ST, 16) || !aligned(workspace, 256)) return GLA_ERR_INVALID_ARG;
    const size_t e = p->dtype == GLA_BF16 ? 2 : 4, states = (size_t)p->B * p->D * p->N * 4;
    const Inputs in = inputs_of(p);
    const Span yo = flat(y, (size_t)p->B * p->T * p->D * e), so = flat(ST, states);
    for (int i = 0; i < 9; ++i)
        if (overlap(yo, in.s[i]) || (overlap(so, in.s[i]) && !(i == 8 && ST == p->S0))) return GLA_ERR_INVALID_ARG;
    if (overlap(yo, so)) return GLA_ERR_INVALID_ARG;
    int sms = 0;
    st = device_ready(&sms);
    if (st != GLA_OK) return st;
    if (p->T == 0) {
        if (!ST || ST == p->S0) return GLA_OK;
        return cuda(p->S0 ? cudaMemcpyAsync(ST, p->S0, states, cudaMemcpyDeviceToDevice, stream) : cudaMemsetAsync(ST, 0, states, stream));
    }
    SsmPlan pl;
    split(p, sms, false, pl);
    const bool step = p->T <= kStepT && p->force_segments == 0;
    if (!step && pl.ws > 0 && (!workspace || workspace_bytes < pl.ws)) return GLA_ERR_WORKSPACE;
    SsmArgs a = common(p, pl, workspace);
    a.y = y; a.ST = ST;
    if (step) return cuda(launch_ssm_step(a, p->dtype, sms, stream));
    cudaError_t r = cudaSuccess;
    if (pl.nseg > 1) {
        if (ST && ST == p->S0) {     // the last segment's blocks write ST beside the first's, that read S0: those get a copy
            float* s0 = reinterpret_cast<float*>(static_cast<char*>(workspace) + pl.off_s0);
            r = cudaMemcpyAsync(s0, p->S0, states, cudaMemcpyDeviceToDevice, stream);
            a.S0 = s0;
        }
        if (r == cudaSuccess) r = launch_ssm_walk(a, kSsmState, p->dtype, stream);
        if (r == cudaSuccess && pl.nseg > 2) r = launch_ssm_scan(a, false, sms, stream);
    }
    if (r == cudaSuccess) r = launch_ssm_walk(a, kSsmOut, p->dtype, stream);
    return cuda(r);
}

size_t gla_ssm_bwd_workspace_size(const gla_ssm_params* p)
{
    int sms = 0;
    if (check(p) != GLA_OK || p->T == 0) return 0;
    if (device_ready(&sms) != GLA_OK) sms = 152;
    SsmPlan pl;
    split(p, sms, true, pl);
    return pl.ws;
}

gla_status gla_ssm_bwd(const gla_ssm_params* p, const gla_ssm_grads* g, void* workspace, size_t workspace_bytes,
                       cudaStream_t stream)
{
    gla_status st = check(p);
    if (st != GLA_OK) return st;
    if (!g || !g->grad_A) return GLA_ERR_INVALID_ARG;
    if (p->T > 0 && (!g->grad_y || !g->grad_x || !g->grad_dt || !g->grad_B || !g->grad_C || (p->z && !g->grad_z)))
        return GLA_ERR_INVALID_ARG;
    if ((g->grad_z && !p->z) || (g->grad_D && !p->D_skip) || (g->grad_dt_bias && !p->dt_bias)) return GLA_ERR_INVALID_ARG;
    for (const void* x : {g->grad_y, (const void*)g->grad_ST, (const void*)g->grad_x, (const void*)g->grad_dt, (const void*)g->grad_z,
                          (const void*)g->grad_B, (const void*)g->grad_C, (const void*)g->grad_S0})
        if (!aligned(x, 16)) return GLA_ERR_INVALID_ARG;
    if (!aligned(g->grad_A, 4) || !aligned(g->grad_D, 4) || !aligned(g->grad_dt_bias, 4) || !aligned(workspace, 256))
        return GLA_ERR_INVALID_ARG;
    const size_t e = p->dtype == GLA_BF16 ? 2 : 4, states = (size_t)p->B * p->D * p->N * 4, row = (size_t)p->B * p->T * p->D * e,
                 bc = (size_t)p->B * p->T * p->G * p->N * e;
    const Inputs in = inputs_of(p);
    const Span gy = flat(g->grad_y, row), gst = flat(g->grad_ST, states);
    const Span out[] = {flat(g->grad_x, row), flat(g->grad_dt, row), flat(g->grad_z, row), flat(g->grad_B, bc), flat(g->grad_C, bc),
                        flat(g->grad_A, (size_t)p->D * p->N * 4), flat(g->grad_D, (size_t)p->D * 4),
                        flat(g->grad_dt_bias, (size_t)p->D * 4), flat(g->grad_S0, states)};
    for (int i = 0; i < 9; ++i) {
        for (const Span& s : in.s)
            if (overlap(out[i], s)) return GLA_ERR_INVALID_ARG;
        if (overlap(out[i], gy) || overlap(out[i], gst)) return GLA_ERR_INVALID_ARG;
        for (int j = i + 1; j < 9; ++j)
            if (overlap(out[i], out[j])) return GLA_ERR_INVALID_ARG;
    }
    int sms = 0;
    st = device_ready(&sms);
    if (st != GLA_OK) return st;
    cudaError_t r = cudaSuccess;
    if (p->T == 0) {
        r = cudaMemsetAsync(g->grad_A, 0, (size_t)p->D * p->N * 4, stream);
        if (r == cudaSuccess && g->grad_D) r = cudaMemsetAsync(g->grad_D, 0, (size_t)p->D * 4, stream);
        if (r == cudaSuccess && g->grad_dt_bias) r = cudaMemsetAsync(g->grad_dt_bias, 0, (size_t)p->D * 4, stream);
        if (r == cudaSuccess && g->grad_S0)
            r = g->grad_ST ? cudaMemcpyAsync(g->grad_S0, g->grad_ST, states, cudaMemcpyDeviceToDevice, stream)
                           : cudaMemsetAsync(g->grad_S0, 0, states, stream);
        return cuda(r);
    }
    SsmPlan pl;
    split(p, sms, true, pl);
    if (!workspace || workspace_bytes < pl.ws) return GLA_ERR_WORKSPACE;
    SsmArgs a = common(p, pl, workspace);
    char* w = static_cast<char*>(workspace);
    a.keep = reinterpret_cast<float*>(w + pl.off_keep);
    a.part_bc = reinterpret_cast<float*>(w + pl.off_bc);
    a.part_p = reinterpret_cast<float*>(w + pl.off_p);
    a.segG = reinterpret_cast<float*>(w + pl.off_segG);
    a.dy = g->grad_y; a.dST = g->grad_ST;
    a.dx = g->grad_x; a.ddt = g->grad_dt; a.dz = g->grad_z; a.dS0 = g->grad_S0;
    if (pl.nseg > 1) {
        r = launch_ssm_walk(a, kSsmState, p->dtype, stream);
        if (r == cudaSuccess && pl.nseg > 2) r = launch_ssm_scan(a, false, sms, stream);
        if (r == cudaSuccess) r = launch_ssm_walk(a, kSsmRev, p->dtype, stream);
        if (r == cudaSuccess && pl.nseg > 2) r = launch_ssm_scan(a, true, sms, stream);
    }
    if (r == cudaSuccess) r = launch_ssm_walk(a, kSsmKeep, p->dtype, stream);
    if (r == cudaSuccess) r = launch_ssm_bwd(a, p->dtype, stream);
    if (r == cudaSuccess) r = launch_ssm_bc_sum(a, g->grad_B, g->grad_C, p->dtype, sms, stream);
    if (r == cudaSuccess)
        r = launch_column_sum(a.part_p, (long long)p->B * pl.nseg, (long long)p->D * p->N + 2LL * p->D,
                              ColumnOuts{{{g->grad_A, (long long)p->D * p->N}, {g->grad_D, p->D}, {g->grad_dt_bias, p->D}}}, stream);
    return cuda(r);
}

}  // extern "C"
