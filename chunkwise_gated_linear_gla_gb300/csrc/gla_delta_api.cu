// The C ABI of the gated delta rule: argument checks, the choice of form, workspace layout and
// launch order. No arithmetic of the method happens here.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "gla_delta_internal.h"

namespace gla {
namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
size_t align_up(size_t x) { return (x + 255) / 256 * 256; }

struct Range { uintptr_t lo, hi; };
Range rng(const void* p, size_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return p ? Range{a, a + bytes} : Range{0, 0};
}
bool overlap(Range a, Range b) {
    if (a.lo == a.hi || b.lo == b.hi) return false;
    return a.lo < b.hi && b.lo < a.hi;
}

gla_status check_sizes(int B, int H, int Hk, int T, int dk, int dv, float scale, int dtype, int path)
{
    if (B <= 0 || H <= 0 || Hk <= 0 || T < 0 || dk <= 0 || dv <= 0) return GLA_ERR_INVALID_ARG;
    if (H % Hk != 0 || dk % 16 != 0 || dv % 16 != 0) return GLA_ERR_INVALID_ARG;
    if (dtype != GLA_BF16 && dtype != GLA_FP32) return GLA_ERR_INVALID_ARG;
    if (path != GLA_PATH_AUTO && path != GLA_PATH_TENSOR && path != GLA_PATH_SIMT) return GLA_ERR_INVALID_ARG;
    if (!std::isfinite(scale)) return GLA_ERR_INVALID_ARG;
    if ((long long)B * H > (1LL << 30)) return GLA_ERR_INVALID_ARG;
    if (dk > kDeltaMaxDk || dv > (1 << 20) || T > kDeltaMaxT) return GLA_ERR_UNSUPPORTED;
    return GLA_OK;
}

// Whether the chunk form takes these sizes: bf16, keys of one or two 64-key slabs, dv in halves
// of its 128-column tile; grid dimensions and TMA coordinates within their types.
bool chunk_shape_ok(int B, int H, int T, int dk, int dv, int dtype)
{
    const long long nch = ((long long)T + kChunk - 1) / kChunk;
    return dtype == GLA_BF16 && T <= kDeltaChunkMaxT && (dk == 64 || dk == 128) && dv % 64 == 0 && (long long)B * H <= 65535 &&
           (long long)B * H * nch < (1LL << 31) && (long long)B * H * T < (1LL << 40);
}

struct DeltaPlan {
    int path = GLA_PATH_SIMT;
    int nch = 0, cps = 0, nseg = 1, per = 1;
    size_t off_pair = 0, off_in = 0;
    size_t ws = 0;
};

// Segments of the sequence. The pass is serial over the chunks of a head's 128 dv columns, so few
// heads leave SMs idle. Cut into n segments the pass takes two walks of nch / n chunks (the first, of
// all segments but the last, has one more tile per head for the transitions; 2.4 and 3.3 us a chunk with all
// SMs busy) and a scan of 3.5 us per segment and wave of its blocks (16 columns each). Where one wave does not
// hold the first walk's segments, its CTAs take two each, one after the other, if it holds them so.
int segments_per_cta(int n, int units, int trans, int sms)
{
    const long long u = (long long)units + trans;
    return (n - 1) * u > sms && n / 2 * u <= sms ? 2 : 1;
}
// The best n of those that take one wave each time, by these rates and 12 us of launches (16384 tokens,
// dk = dv = 128, caches flushed, one head: uncut 736 us, 5 segments 296, 20 140, 40 158; 16 heads: uncut 728,
// 5 segments 300, 9, two to a CTA, 267, 12 in several waves 347). With 64-wide keys both are cheaper and n is
// taken by the same rates: one head 97 us at the rule's 20 against 87 at 32 and 105 at 64; 16 heads 212 at its 9, the
// best of 1 to 32.
int choose_segments(int units, int trans, int dv, int nch, int sms)
{
    const int most = std::min(sms / units, nch / 4);
    const long long waves = ((long long)trans * (dv / 16) + sms - 1) / sms;
    int best = 1;
    long long least = 29LL * nch - 120;
    for (int n = 3; n <= most; ++n) {
        const int per = segments_per_cta(n, units, trans, sms);
        if ((long long)(per == 2 ? n / 2 : n - 1) * (units + trans) > sms) continue;
        const long long cost = (24LL * per + 33) * ((nch + n - 1) / n) + 35 * waves * n;
        if (cost < least) { least = cost; best = n; }
    }
    return best;
}

gla_status plan_fwd(const gla_delta_params* p, DeltaPlan& pl)
{
    if (!p) return GLA_ERR_INVALID_ARG;
    gla_status st = check_sizes(p->B, p->H, p->Hk, p->T, p->dk, p->dv, p->scale, p->dtype, p->path);
    if (st != GLA_OK) return st;
    if (p->force_segments < 0) return GLA_ERR_INVALID_ARG;
    const bool ok = chunk_shape_ok(p->B, p->H, p->T, p->dk, p->dv, p->dtype);
    if (p->path == GLA_PATH_TENSOR && !ok) return GLA_ERR_UNSUPPORTED;
    if (p->T == 0 || !ok || p->path == GLA_PATH_SIMT) return GLA_OK;
    const long long units = (long long)p->B * p->H * ((p->dv + kDvTile - 1) / kDvTile);
    if (p->path == GLA_PATH_AUTO && p->T < (units < kDeltaFewTiles ? kDeltaChunkMinTFew : kDeltaChunkMinT)) return GLA_OK;
    pl.path = GLA_PATH_TENSOR;
    pl.nch = (p->T + kChunk - 1) / kChunk;
    int sms = 0;
    if (device_ready(&sms) != GLA_OK) sms = 152;
    const int BH = p->B * p->H;
    int n = p->force_segments > 0 ? p->force_segments
                                  : choose_segments((int)units, BH, p->dv, pl.nch, sms);
    if (n > pl.nch) n = pl.nch;
    if (n > 65535) n = 65535;
    pl.cps = (pl.nch + n - 1) / n;
    pl.nseg = (pl.nch + pl.cps - 1) / pl.cps;
    pl.per = segments_per_cta(pl.nseg, (int)units, BH, sms);
    if (pl.nseg > 1) {
        const size_t st4 = (size_t)p->dk * p->dv * 4, m4 = (size_t)p->dk * p->dk * 4;
        size_t off = 0;
        auto take = [&](size_t bytes) { const size_t at = off; off = align_up(off + bytes); return at; };
        pl.off_pair = take((size_t)BH * (pl.nseg - 1) * (st4 + m4));
        pl.off_in = take((size_t)BH * pl.nseg * st4);
        pl.ws = off;
    }
    return GLA_OK;
}

gla_status check_fwd(const gla_delta_params* p)
{
    if (p->T > 0 && (!p->q || !p->k || !p->v || !p->beta || !p->O)) return GLA_ERR_INVALID_ARG;
    for (const void* x : {p->q, p->k, p->v, (const void*)p->O, (const void*)p->S0, (const void*)p->ST})
        if (!aligned(x, 16)) return GLA_ERR_INVALID_ARG;
    const size_t e = p->dtype == GLA_BF16 ? 2 : 4;
    if (!aligned(p->log_g, 4) || !aligned(p->beta, e) || !aligned(p->workspace, 256)) return GLA_ERR_INVALID_ARG;
    const size_t BHT = (size_t)p->B * p->H * p->T, nk = (size_t)p->B * p->Hk * p->T * p->dk * e;
    const size_t ns = (size_t)p->B * p->H * p->dk * p->dv * 4;
    const Range O = rng(p->O, BHT * p->dv * e), ST = rng(p->ST, ns), S0 = rng(p->S0, ns);
    const Range in[] = {rng(p->q, nk), rng(p->k, nk), rng(p->v, BHT * p->dv * e), rng(p->log_g, BHT * 4),
                        rng(p->beta, BHT * e)};
    for (const Range& r : in)
        if (overlap(O, r) || overlap(ST, r)) return GLA_ERR_INVALID_ARG;
    if (overlap(O, S0) || overlap(O, ST)) return GLA_ERR_INVALID_ARG;
    if (overlap(ST, S0) && (const void*)p->ST != (const void*)p->S0) return GLA_ERR_INVALID_ARG;
    return GLA_OK;
}

struct DeltaBwdPlan {
    int path = GLA_PATH_SIMT;
    int tiles = 0;
    int nch = 0;
    // chunk form: prep's T and P in two parts, gates; the sweeps' states, U and what dV's rounding left
    size_t off_t = 0, off_p = 0, off_g = 0, off_sh = 0, off_sl = 0, off_uh = 0, off_ul = 0,
           off_dh = 0, off_dl = 0, off_xl = 0;
    // recurrent form; part_q and part_k also serve the chunk form when heads share keys
    size_t off_keep = 0, off_pq = 0, off_pk = 0, off_pg = 0, off_pb = 0, off_scr = 0;
    size_t ws = 0;
};

gla_status plan_bwd(const gla_delta_bwd_params* p, DeltaBwdPlan& pl)
{
    if (!p) return GLA_ERR_INVALID_ARG;
    gla_status st = check_sizes(p->B, p->H, p->Hk, p->T, p->dk, p->dv, p->scale, p->dtype, p->path);
    if (st != GLA_OK) return st;
    const bool ok = chunk_shape_ok(p->B, p->H, p->T, p->dk, p->dv, p->dtype);
    if (p->path == GLA_PATH_TENSOR && !ok) return GLA_ERR_UNSUPPORTED;
    if (p->T == 0) return GLA_OK;
    const size_t BH = (size_t)p->B * p->H, T = p->T;
    const size_t dkp = p->dk <= 64 ? 64 : p->dk <= 128 ? 128 : 256;
    size_t off = 0;
    auto take = [&](size_t bytes) { const size_t at = off; off = align_up(off + bytes); return at; };
    if (ok && p->path != GLA_PATH_SIMT) {
        pl.path = GLA_PATH_TENSOR;
        pl.nch = (p->T + kChunk - 1) / kChunk;
        const size_t nc = BH * pl.nch, cc = nc * 2 * kChunk * kChunk * 2, st = nc * p->dk * p->dv * 2, u = nc * kChunk * p->dv * 2;
        pl.off_t = take(cc); pl.off_p = take(cc);
        pl.off_g = take(nc * 8 * kChunk * 4);
        pl.off_sh = take(st); pl.off_sl = take(st); pl.off_dh = take(st); pl.off_dl = take(st);
        pl.off_uh = take(u); pl.off_ul = take(u);
        pl.off_xl = take(BH * T * p->dv * 2);
        if (p->H != p->Hk) {
            pl.tiles = 1;
            pl.off_pq = take(BH * T * p->dk * 4);
            pl.off_pk = take(BH * T * p->dk * 4);
        }
        pl.ws = off;
        return GLA_OK;
    }
    pl.tiles = (p->dv + kDeltaBwdTile - 1) / kDeltaBwdTile;
    pl.off_keep = take(BH * ((T + kDeltaKeep - 1) / kDeltaKeep) * p->dk * p->dv * 4);
    pl.off_pq = take(pl.tiles * BH * T * p->dk * 4);
    pl.off_pk = take(pl.tiles * BH * T * p->dk * 4);
    pl.off_pg = take(pl.tiles * BH * T * 4);
    pl.off_pb = take(pl.tiles * BH * T * 4);
    pl.off_scr = take(pl.tiles * BH * kDeltaKeep * dkp * kDeltaBwdTile * 4);
    pl.ws = off;
    return GLA_OK;
}

gla_status check_bwd(const gla_delta_bwd_params* p)
{
    if (p->T > 0 && (!p->q || !p->k || !p->v || !p->beta || !p->grad_O || !p->grad_q || !p->grad_k || !p->grad_v))
        return GLA_ERR_INVALID_ARG;
    if (p->grad_log_g && !p->log_g && p->T > 0) return GLA_ERR_INVALID_ARG;
    for (const void* x : {p->q, p->k, p->v, p->grad_O, (const void*)p->S0, (const void*)p->grad_ST,
                          (const void*)p->grad_q, (const void*)p->grad_k, (const void*)p->grad_v,
                          (const void*)p->grad_S0})
        if (!aligned(x, 16)) return GLA_ERR_INVALID_ARG;
    const size_t e = p->dtype == GLA_BF16 ? 2 : 4;
    if (!aligned(p->log_g, 4) || !aligned(p->grad_log_g, 4) || !aligned(p->beta, e) || !aligned(p->grad_beta, e) ||
        !aligned(p->workspace, 256))
        return GLA_ERR_INVALID_ARG;
    const size_t BHT = (size_t)p->B * p->H * p->T, nk = (size_t)p->B * p->Hk * p->T * p->dk * e;
    const size_t nv = BHT * p->dv * e, ns = (size_t)p->B * p->H * p->dk * p->dv * 4;
    const Range in[] = {rng(p->q, nk), rng(p->k, nk), rng(p->v, nv), rng(p->log_g, BHT * 4), rng(p->beta, BHT * e),
                        rng(p->S0, ns), rng(p->grad_O, nv), rng(p->grad_ST, ns)};
    const Range out[] = {rng(p->grad_q, nk), rng(p->grad_k, nk), rng(p->grad_v, nv), rng(p->grad_log_g, BHT * 4),
                         rng(p->grad_beta, BHT * e), rng(p->grad_S0, ns)};
    const int no = sizeof(out) / sizeof(out[0]);
    for (int i = 0; i < no; ++i) {
        for (const Range& r : in)
            if (overlap(out[i], r)) return GLA_ERR_INVALID_ARG;
        for (int j = i + 1; j < no; ++j)
            if (overlap(out[i], out[j])) return GLA_ERR_INVALID_ARG;
    }
    return GLA_OK;
}

DeltaStep step_args(const gla_delta_params* p, int sms)
{
    DeltaStep a;
    a.q = p->q; a.k = p->k; a.v = p->v; a.log_g = p->log_g; a.beta = p->beta;
    a.S0 = p->S0; a.O = p->O; a.ST = p->ST; a.keep = nullptr;
    a.B = p->B; a.H = p->H; a.Hk = p->Hk; a.T = p->T; a.dk = p->dk; a.dv = p->dv;
    a.scale = p->scale; a.dtype = p->dtype; a.sms = sms;
    return a;
}

// The chunk form of the backward: prep, the two sweeps, the gradients, and the sum over heads
// that share keys.
gla_status bwd_chunks(const gla_delta_bwd_params* p, const DeltaBwdPlan& pl, int sms, cudaStream_t stream)
{
    uint8_t* ws = static_cast<uint8_t*>(p->workspace);
    int* status = device_status_ptr();
    if (!status) return GLA_ERR_CUDA;
    float* gates = reinterpret_cast<float*>(ws + pl.off_g);
    DeltaPrep a;
    a.q = p->q; a.k = p->k; a.log_g = p->log_g; a.beta = p->beta;
    a.t = ws + pl.off_t; a.p = ws + pl.off_p; a.gates = gates;
    a.B = p->B; a.H = p->H; a.Hk = p->Hk; a.T = p->T; a.dk = p->dk; a.nch = pl.nch; a.scale = p->scale;
    a.beta_floor = 0x1p-40f;
    cudaError_t e = launch_delta_prep(a, status, stream);
    DeltaSweep w;
    w.q = p->q; w.k = p->k; w.v = p->v;
    w.t = a.t; w.p = a.p; w.gates = gates;
    w.S_in = p->S0; w.S_out = nullptr;
    w.s_hi = ws + pl.off_sh; w.s_lo = ws + pl.off_sl; w.u_hi = ws + pl.off_uh; w.u_lo = ws + pl.off_ul;
    w.x_hi = p->grad_v; w.x_lo = ws + pl.off_xl;
    w.B = p->B; w.H = p->H; w.Hk = p->Hk; w.T = p->T; w.dk = p->dk; w.dv = p->dv; w.nch = pl.nch;
    w.scale = p->scale; w.reverse = false;
    if (e == cudaSuccess) e = launch_delta_sweep(w, status, stream);
    w.v = p->grad_O; w.S_in = p->grad_ST; w.S_out = p->grad_S0;
    w.s_hi = ws + pl.off_dh; w.s_lo = ws + pl.off_dl; w.reverse = true;
    if (e == cudaSuccess) e = launch_delta_sweep(w, status, stream);
    const bool shared = p->H != p->Hk;
    DeltaGrads g;
    g.q = p->q; g.k = p->k; g.dO = p->grad_O;
    g.s_hi = ws + pl.off_sh; g.s_lo = ws + pl.off_sl; g.u_hi = w.u_hi; g.u_lo = w.u_lo;
    g.d_hi = w.s_hi; g.d_lo = w.s_lo; g.x_hi = p->grad_v; g.x_lo = w.x_lo;
    g.log_g = p->log_g; g.gates = gates;
    g.dq = p->grad_q; g.dk_out = p->grad_k;
    g.part_q = shared ? reinterpret_cast<float*>(ws + pl.off_pq) : nullptr;
    g.part_k = shared ? reinterpret_cast<float*>(ws + pl.off_pk) : nullptr;
    g.dlog_g = p->grad_log_g; g.dbeta = p->grad_beta;
    g.B = p->B; g.H = p->H; g.Hk = p->Hk; g.T = p->T; g.dk = p->dk; g.dv = p->dv; g.nch = pl.nch; g.sms = sms; g.scale = p->scale;
    if (e == cudaSuccess) e = launch_delta_grads(g, status, stream);
    if (e == cudaSuccess && shared) {
        DeltaBwdSum u;
        u.part_q = g.part_q; u.part_k = g.part_k; u.part_g = nullptr; u.part_b = nullptr;
        u.dq = p->grad_q; u.dk_out = p->grad_k; u.dlog_g = nullptr; u.dbeta = nullptr;
        u.tiles = 1; u.B = p->B; u.H = p->H; u.Hk = p->Hk; u.T = p->T; u.dk = p->dk;
        u.dtype = p->dtype; u.sms = sms;
        e = launch_delta_bwd_sum(u, stream);
    }
    return e == cudaSuccess ? GLA_OK : GLA_ERR_CUDA;
}

}  // namespace
}  // namespace gla

using namespace gla;

extern "C" {

size_t gla_delta_fwd_workspace_size(const gla_delta_params* p)
{
    DeltaPlan pl;
    return plan_fwd(p, pl) == GLA_OK ? pl.ws : 0;
}

gla_status gla_delta_fwd(const gla_delta_params* p, cudaStream_t stream)
{
    DeltaPlan pl;
    gla_status st = plan_fwd(p, pl);
    if (st != GLA_OK) return st;
    st = check_fwd(p);
    if (st != GLA_OK) return st;
    int sms = 0;
    st = device_ready(&sms);
    if (st != GLA_OK) return st;
    if (pl.ws > 0 && (!p->workspace || p->workspace_bytes < pl.ws)) return GLA_ERR_WORKSPACE;
    cudaError_t e = cudaSuccess;
    if (p->T == 0) {
        const size_t ns = (size_t)p->B * p->H * p->dk * p->dv * 4;
        if (p->ST && p->ST != p->S0)
            e = p->S0 ? cudaMemcpyAsync(p->ST, p->S0, ns, cudaMemcpyDeviceToDevice, stream)
                      : cudaMemsetAsync(p->ST, 0, ns, stream);
    } else if (pl.path == GLA_PATH_TENSOR) {
        uint8_t* ws = static_cast<uint8_t*>(p->workspace);
        int* status = device_status_ptr();
        if (!status) return GLA_ERR_CUDA;
        DeltaChunks a;
        a.q = p->q; a.k = p->k; a.v = p->v; a.log_g = p->log_g; a.beta = p->beta;
        a.S0 = p->S0; a.O = p->O; a.ST = p->ST;
        a.pair = pl.ws ? reinterpret_cast<float*>(ws + pl.off_pair) : nullptr;
        a.seg_in = pl.ws ? reinterpret_cast<float*>(ws + pl.off_in) : nullptr;
        a.B = p->B; a.H = p->H; a.Hk = p->Hk; a.T = p->T; a.dk = p->dk; a.dv = p->dv;
        a.nch = pl.nch; a.cps = pl.cps; a.nseg = pl.nseg; a.per = pl.per; a.scale = p->scale;
        e = launch_delta_chunks(a, status, stream);
    } else {
        e = launch_delta_step(step_args(p, sms), stream);
    }
    return e == cudaSuccess ? GLA_OK : GLA_ERR_CUDA;
}

size_t gla_delta_bwd_workspace_size(const gla_delta_bwd_params* p)
{
    DeltaBwdPlan pl;
    return plan_bwd(p, pl) == GLA_OK ? pl.ws : 0;
}

gla_status gla_delta_bwd(const gla_delta_bwd_params* p, cudaStream_t stream)
{
    DeltaBwdPlan pl;
    gla_status st = plan_bwd(p, pl);
    if (st != GLA_OK) return st;
    st = check_bwd(p);
    if (st != GLA_OK) return st;
    int sms = 0;
    st = device_ready(&sms);
    if (st != GLA_OK) return st;
    if (pl.ws > 0 && (!p->workspace || p->workspace_bytes < pl.ws)) return GLA_ERR_WORKSPACE;
    cudaError_t e = cudaSuccess;
    if (p->T == 0) {
        const size_t ns = (size_t)p->B * p->H * p->dk * p->dv * 4;
        if (p->grad_S0)
            e = p->grad_ST ? cudaMemcpyAsync(p->grad_S0, p->grad_ST, ns, cudaMemcpyDeviceToDevice, stream)
                           : cudaMemsetAsync(p->grad_S0, 0, ns, stream);
        return e == cudaSuccess ? GLA_OK : GLA_ERR_CUDA;
    }
    uint8_t* ws = static_cast<uint8_t*>(p->workspace);
    auto f = [&](size_t off) { return reinterpret_cast<float*>(ws + off); };
    if (pl.path == GLA_PATH_TENSOR) return bwd_chunks(p, pl, sms, stream);
    DeltaStep a;
    std::memset(&a, 0, sizeof(a));
    a.q = p->q; a.k = p->k; a.v = p->v; a.log_g = p->log_g; a.beta = p->beta; a.S0 = p->S0;
    a.keep = f(pl.off_keep);
    a.B = p->B; a.H = p->H; a.Hk = p->Hk; a.T = p->T; a.dk = p->dk; a.dv = p->dv;
    a.scale = p->scale; a.dtype = p->dtype; a.sms = sms;
    e = launch_delta_step(a, stream);
    if (e == cudaSuccess) {
        DeltaBwdStep w;
        w.q = p->q; w.k = p->k; w.v = p->v; w.log_g = p->log_g; w.beta = p->beta;
        w.keep = f(pl.off_keep); w.dO = p->grad_O; w.dST = p->grad_ST; w.dv_out = p->grad_v; w.dS0 = p->grad_S0;
        w.part_q = f(pl.off_pq); w.part_k = f(pl.off_pk); w.part_g = f(pl.off_pg); w.part_b = f(pl.off_pb);
        w.scratch = f(pl.off_scr);
        w.B = p->B; w.H = p->H; w.Hk = p->Hk; w.T = p->T; w.dk = p->dk; w.dv = p->dv;
        w.scale = p->scale; w.dtype = p->dtype;
        e = launch_delta_bwd_step(w, stream);
    }
    if (e == cudaSuccess) {
        DeltaBwdSum w;
        w.part_q = f(pl.off_pq); w.part_k = f(pl.off_pk); w.part_g = f(pl.off_pg); w.part_b = f(pl.off_pb);
        w.dq = p->grad_q; w.dk_out = p->grad_k; w.dlog_g = p->grad_log_g; w.dbeta = p->grad_beta;
        w.tiles = pl.tiles; w.B = p->B; w.H = p->H; w.Hk = p->Hk; w.T = p->T; w.dk = p->dk;
        w.dtype = p->dtype; w.sms = sms;
        e = launch_delta_bwd_sum(w, stream);
    }
    return e == cudaSuccess ? GLA_OK : GLA_ERR_CUDA;
}

}  // extern "C"
