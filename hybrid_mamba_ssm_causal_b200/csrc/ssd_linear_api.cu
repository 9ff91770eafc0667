// ssd_linear_api.cu -- the C ABI of linear attention with a decay per head (include/ssd_mixer.h):
// argument checks, workspace carving and dispatch. Nothing is allocated, no state is kept.
#include <math.h>

#include "../../include/ssd_mixer.h"
#include "ssd_linear.h"

namespace {

size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }
bool pow2_16_128(int v) { return v >= 16 && v <= 128 && (v & (v - 1)) == 0; }

ssd_status check_linear(const ssd_linear_dims* d)
{
    if (!d) return SSD_ERR_INVALID_ARG;
    if (d->batch < 0 || d->seqlen < 0 || d->nheads <= 0 || d->ngroups <= 0 || d->dk <= 0 || d->dv <= 0 ||
        !isfinite(d->scale))
        return SSD_ERR_INVALID_ARG;
    if (d->nheads % d->ngroups != 0) return SSD_ERR_INVALID_ARG;
    if (d->act != SSD_F32 && d->act != SSD_BF16) return SSD_ERR_UNSUPPORTED;
    if (!pow2_16_128(d->dk) || !pow2_16_128(d->dv)) return SSD_ERR_UNSUPPORTED;
    if (d->nheads > 65535 || d->batch > 65535) return SSD_ERR_UNSUPPORTED;
    // token rows and (segment, head) pairs are counted in 31 bits
    const int64_t tokens = d->batch > 0 && d->seqlen > 0x7fffff00LL / d->batch ? -1 : d->batch * d->seqlen;
    if (tokens < 0 || (tokens / 128 + 2 * d->batch + 1) * d->nheads > 0x7fffffffLL) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}
// The same for a packed call, whose seqlen counts all token rows.
ssd_status check_linear_packed(const ssd_linear_dims* d)
{
    if (!d) return SSD_ERR_INVALID_ARG;
    ssd_linear_dims one = *d;
    one.batch = d->batch < 0 ? d->batch : 1;
    const ssd_status st = check_linear(&one);
    if (st != SSD_OK) return st;
    if (d->batch > 65535) return SSD_ERR_UNSUPPORTED;
    if ((d->seqlen / 128 + 2 * d->batch + 1) * d->nheads > 0x7fffffffLL) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

size_t elem(const ssd_linear_dims* d) { return d->act == SSD_BF16 ? 2 : 4; }
bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
// One operand's rows: 16-byte aligned, at least `width` elements apart.
bool row_ok(const void* p, int64_t ld, int64_t width, size_t es)
{
    return aligned16(p) && ld >= width && ((size_t)ld * es) % 16 == 0;
}

struct Layout {
    size_t status, list, seg, part_k, part_v, total;   // seg: one region per scan
    size_t seg_each;
};

bool on_tensor_cores(const ssd_linear_dims* d)
{
    ssd::LinearScan s{};
    s.DK = d->dk;
    s.DV = d->dv;
    return ssd::linear_tc_supported(s, d->act);
}

// The split of a call's rows, which depends on the sizes and the SM count alone.
void plan(ssd::LinearCall* c, const ssd_linear_dims* d, bool packed, int nscans)
{
    c->b = d->batch;
    c->T = packed ? d->seqlen : d->batch * d->seqlen;
    c->L = d->seqlen;
    c->H = d->nheads;
    c->act = d->act;
    c->seg_tokens = ssd::linear_segment_tokens(on_tensor_cores(d), d->batch, c->L, c->T, packed, d->nheads,
                                               nscans, d->dk, d->dv, ssd::device_sm_count(), &c->sub);
    if (packed) {
        c->nseg = 0;
        c->items = d->batch > 0 ? d->batch + c->T / c->seg_tokens : 0;
        c->split = c->T > c->seg_tokens;
    } else {
        c->nseg = c->L > 0 ? (c->L + c->seg_tokens - 1) / c->seg_tokens : 1;
        c->items = d->batch * c->nseg;
        c->split = c->nseg > 1;
    }
}

Layout layout(const ssd_linear_dims* d, const ssd::LinearCall& c, int nscans)
{
    Layout w{};
    size_t off = 256;
    w.list = off;
    if (c.nseg == 0 && on_tensor_cores(d)) off = align256(off + (size_t)c.items * 2 * sizeof(int2));   // a packed call's segments
    w.seg = off;
    w.seg_each = c.split ? align256((size_t)ssd::linear_pieces(c).items * d->nheads * d->dk * d->dv * 4) : 0;
    off += nscans * w.seg_each;
    w.part_k = off;
    if (nscans == 3 && d->nheads != d->ngroups) off = align256(off + (size_t)c.T * d->nheads * d->dk * 4);
    w.part_v = off;
    if (nscans == 3 && d->nheads != d->ngroups) off = align256(off + (size_t)c.T * d->nheads * d->dv * 4);
    w.total = off;
    return w;
}

ssd::LinearScan prefill_scan(const ssd_linear_dims* d, const void* q, int64_t q_ld, const void* k, int64_t k_ld,
                             const void* v, int64_t v_ld, const float* init, void* o, int64_t o_ld, float* final_state,
                             char* ws, const Layout& w)
{
    ssd::LinearScan s{};
    const int r = d->nheads / d->ngroups;
    s.q = q; s.k = k; s.v = v; s.o = o;
    s.q_ld = q_ld; s.k_ld = k_ld; s.v_ld = v_ld; s.o_ld = o_ld;
    s.q_share = 1; s.k_share = r; s.v_share = r;
    s.DK = d->dk; s.DV = d->dv;
    s.u_scale = 1.0f; s.out_scale = d->scale;
    s.init = init; s.init_rs = d->dk; s.init_cs = 1;
    s.final_state = final_state;
    s.seg_states = (float*)(ws + w.seg);
    return s;
}

ssd_status run(const ssd::LinearCall& c, const ssd::LinearScan* s, int n, cudaStream_t st)
{
    if (ssd::linear_tc_supported(s[0], c.act))
        return ssd::launch_linear_tc(c, s, n, st) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
    return ssd::launch_linear_simt(c, s, n, st) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t ssd_mixer_linear_prefill_workspace_size(const ssd_linear_dims* d)
{
    if (check_linear(d) != SSD_OK) return 0;
    ssd::LinearCall c{};
    plan(&c, d, false, 1);
    return layout(d, c, 1).total;
}

size_t ssd_mixer_linear_prefill_varlen_workspace_size(const ssd_linear_dims* d)
{
    if (check_linear_packed(d) != SSD_OK) return 0;
    ssd::LinearCall c{};
    plan(&c, d, true, 1);
    return layout(d, c, 1).total;
}

size_t ssd_mixer_linear_backward_workspace_size(const ssd_linear_dims* d)
{
    if (check_linear(d) != SSD_OK) return 0;
    ssd::LinearCall c{};
    plan(&c, d, false, 3);
    return layout(d, c, 3).total;
}

ssd_status ssd_mixer_linear_prefill(const ssd_linear_dims* d, const void* q, int64_t q_ld, const void* k, int64_t k_ld,
                                    const void* v, int64_t v_ld, const float* log_decay, const float* init_state, void* o,
                                    int64_t o_ld, float* final_state, void* workspace, size_t workspace_bytes, void* stream)
{
    const ssd_status ds = check_linear(d);
    if (ds != SSD_OK) return ds;
    if (!log_decay || !final_state) return SSD_ERR_INVALID_ARG;
    if (!aligned16(final_state) || (init_state && !aligned16(init_state)) || ((uintptr_t)log_decay & 3u))
        return SSD_ERR_UNSUPPORTED;
    ssd::LinearCall c{};
    plan(&c, d, false, 1);
    const Layout w = layout(d, c, 1);
    if (!workspace || workspace_bytes < w.total || ((uintptr_t)workspace & 255u)) return SSD_ERR_INVALID_ARG;
    if (c.T > 0) {
        const size_t es = elem(d);
        if (!q || !k || !v || !o) return SSD_ERR_INVALID_ARG;
        if (!row_ok(q, q_ld, (int64_t)d->nheads * d->dk, es) || !row_ok(k, k_ld, (int64_t)d->ngroups * d->dk, es) ||
            !row_ok(v, v_ld, (int64_t)d->ngroups * d->dv, es) || !row_ok(o, o_ld, (int64_t)d->nheads * d->dv, es))
            return SSD_ERR_UNSUPPORTED;
    }
    if (d->batch == 0) return SSD_OK;
    c.log_decay = log_decay;
    c.nslots = d->batch;
    c.status = (int*)workspace;
    cudaStream_t st = (cudaStream_t)stream;
    c.taken = c.status + 1;
    if (ssd::set_clear_status(&c, st) != cudaSuccess) return SSD_ERR_CUDA;
    const ssd::LinearScan s = prefill_scan(d, q, q_ld, k, k_ld, v, v_ld, init_state, o, o_ld, final_state, (char*)workspace, w);
    if (d->seqlen <= ssd::kLinearShort)
        return ssd::launch_linear_short(c, s, false, false, st) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
    return run(c, &s, 1, st);
}

ssd_status ssd_mixer_linear_prefill_varlen(const ssd_linear_dims* d, const int32_t* cu_seqlens, const int32_t* slot_idx,
                                           const uint8_t* has_init, const void* q, int64_t q_ld, const void* k, int64_t k_ld,
                                           const void* v, int64_t v_ld, const float* log_decay, float* state, int64_t nslots,
                                           void* o, int64_t o_ld, void* workspace, size_t workspace_bytes, void* stream)
{
    const ssd_status ds = check_linear_packed(d);
    if (ds != SSD_OK) return ds;
    if (!cu_seqlens || !log_decay || !state || nslots < 0) return SSD_ERR_INVALID_ARG;
    if (!slot_idx && nslots < d->batch) return SSD_ERR_INVALID_ARG;
    if (!aligned16(state) || ((uintptr_t)cu_seqlens & 3u) || ((uintptr_t)slot_idx & 3u) || ((uintptr_t)log_decay & 3u))
        return SSD_ERR_UNSUPPORTED;
    ssd::LinearCall c{};
    plan(&c, d, true, 1);
    const Layout w = layout(d, c, 1);
    if (!workspace || workspace_bytes < w.total || ((uintptr_t)workspace & 255u)) return SSD_ERR_INVALID_ARG;
    if (c.T > 0) {
        const size_t es = elem(d);
        if (!q || !k || !v || !o) return SSD_ERR_INVALID_ARG;
        if (!row_ok(q, q_ld, (int64_t)d->nheads * d->dk, es) || !row_ok(k, k_ld, (int64_t)d->ngroups * d->dk, es) ||
            !row_ok(v, v_ld, (int64_t)d->ngroups * d->dv, es) || !row_ok(o, o_ld, (int64_t)d->nheads * d->dv, es))
            return SSD_ERR_UNSUPPORTED;
    }
    if (d->batch == 0) return SSD_OK;
    c.log_decay = log_decay;
    c.cu_seqlens = cu_seqlens;
    c.slot_idx = slot_idx;
    if (on_tensor_cores(d)) {
        c.list = (int2*)((char*)workspace + w.list);
        c.counts = (int*)workspace + 32;
    }
    c.has_init = has_init;
    c.nslots = nslots;
    c.status = (int*)workspace;
    cudaStream_t st = (cudaStream_t)stream;
    c.taken = c.status + 1;
    if (ssd::set_clear_status(&c, st) != cudaSuccess) return SSD_ERR_CUDA;
    const ssd::LinearScan s = prefill_scan(d, q, q_ld, k, k_ld, v, v_ld, state, o, o_ld, state, (char*)workspace, w);
    return run(c, &s, 1, st);
}

ssd_status ssd_mixer_linear_decode_step(const ssd_linear_dims* d, const void* q, int64_t q_ld, const void* k, int64_t k_ld,
                                        const void* v, int64_t v_ld, const float* log_decay, float* state, int64_t nslots,
                                        const int32_t* slot_idx, void* o, int64_t o_ld, void* stream)
{
    const ssd_status ds = check_linear(d);
    if (ds != SSD_OK) return ds;
    if (d->seqlen != 1 || nslots < 0) return SSD_ERR_INVALID_ARG;
    if (d->batch == 0) return SSD_OK;
    if (!slot_idx && nslots < d->batch) return SSD_ERR_INVALID_ARG;
    if (!q || !k || !v || !o || !log_decay || !state) return SSD_ERR_INVALID_ARG;
    const size_t es = elem(d);
    if (!aligned16(state) || ((uintptr_t)slot_idx & 3u) || ((uintptr_t)log_decay & 3u) ||
        !row_ok(q, q_ld, (int64_t)d->nheads * d->dk, es) || !row_ok(k, k_ld, (int64_t)d->ngroups * d->dk, es) ||
        !row_ok(v, v_ld, (int64_t)d->ngroups * d->dv, es) || !row_ok(o, o_ld, (int64_t)d->nheads * d->dv, es))
        return SSD_ERR_UNSUPPORTED;
    ssd::LinearCall c{};
    c.b = d->batch; c.L = c.T = 1;
    c.H = d->nheads; c.act = d->act;
    c.log_decay = log_decay;
    c.slot_idx = slot_idx; c.nslots = nslots;
    const ssd::LinearScan s = prefill_scan(d, q, q_ld, k, k_ld, v, v_ld, state, o, o_ld, state, nullptr, Layout{});
    return ssd::launch_linear_short(c, s, true, false, (cudaStream_t)stream) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

ssd_status ssd_mixer_linear_backward(const ssd_linear_dims* d, const void* q, int64_t q_ld, const void* k, int64_t k_ld,
                                     const void* v, int64_t v_ld, const float* log_decay, const float* init_state,
                                     const void* dout, int64_t dout_ld, const float* dfinal_state, void* dq, int64_t dq_ld,
                                     void* dk, int64_t dk_ld, void* dv, int64_t dv_ld, float* dinit_state, void* workspace,
                                     size_t workspace_bytes, void* stream)
{
    const ssd_status ds = check_linear(d);
    if (ds != SSD_OK) return ds;
    if (!log_decay) return SSD_ERR_INVALID_ARG;
    if ((init_state && !aligned16(init_state)) || (dfinal_state && !aligned16(dfinal_state)) ||
        (dinit_state && !aligned16(dinit_state)) || ((uintptr_t)log_decay & 3u))
        return SSD_ERR_UNSUPPORTED;
    ssd::LinearCall c{};
    plan(&c, d, false, 3);
    const Layout w = layout(d, c, 3);
    if (!workspace || workspace_bytes < w.total || ((uintptr_t)workspace & 255u)) return SSD_ERR_INVALID_ARG;
    const int r = d->nheads / d->ngroups;
    const int64_t HK = (int64_t)d->nheads * d->dk, HV = (int64_t)d->nheads * d->dv;
    const int64_t GK = (int64_t)d->ngroups * d->dk, GV = (int64_t)d->ngroups * d->dv;
    if (c.T > 0) {
        const size_t es = elem(d);
        if (!q || !k || !v || !dout || !dq || !dk || !dv) return SSD_ERR_INVALID_ARG;
        if (!row_ok(q, q_ld, HK, es) || !row_ok(k, k_ld, GK, es) || !row_ok(v, v_ld, GV, es) || !row_ok(dout, dout_ld, HV, es) ||
            !row_ok(dq, dq_ld, HK, es) || !row_ok(dk, dk_ld, GK, es) || !row_ok(dv, dv_ld, GV, es))
            return SSD_ERR_UNSUPPORTED;
    }
    if (d->batch == 0) return SSD_OK;
    c.log_decay = log_decay;
    c.nslots = d->batch;
    c.status = (int*)workspace;
    char* ws = (char*)workspace;
    cudaStream_t st = (cudaStream_t)stream;

    ssd::LinearScan s[3] = {};
    ssd::LinearScan &sq = s[0], &sv = s[1], &sk = s[2];
    // dq: forwards on (do, v, k), the state transposed
    sq.q = dout; sq.q_ld = dout_ld; sq.q_share = 1;
    sq.k = v; sq.k_ld = v_ld; sq.k_share = r;
    sq.v = k; sq.v_ld = k_ld; sq.v_share = r;
    sq.o = dq; sq.o_ld = dq_ld;
    sq.DK = d->dv; sq.DV = d->dk;
    sq.u_scale = 1.0f; sq.out_scale = d->scale;
    sq.init = init_state; sq.init_rs = 1; sq.init_cs = d->dk;
    // dv: backwards on (k, q, do); its state is the gradient of the state
    sv.q = k; sv.q_ld = k_ld; sv.q_share = r;
    sv.k = q; sv.k_ld = q_ld; sv.k_share = 1;
    sv.v = dout; sv.v_ld = dout_ld; sv.v_share = 1;
    sv.DK = d->dk; sv.DV = d->dv;
    sv.u_scale = d->scale; sv.out_scale = 1.0f;
    sv.init = dfinal_state; sv.init_rs = d->dk; sv.init_cs = 1;
    sv.final_state = dinit_state;
    sv.reverse = true;
    // dk: backwards on (v, do, q), that state transposed
    sk.q = v; sk.q_ld = v_ld; sk.q_share = r;
    sk.k = dout; sk.k_ld = dout_ld; sk.k_share = 1;
    sk.v = q; sk.v_ld = q_ld; sk.v_share = 1;
    sk.DK = d->dv; sk.DV = d->dk;
    sk.u_scale = d->scale; sk.out_scale = 1.0f;
    sk.init = dfinal_state; sk.init_rs = 1; sk.init_cs = d->dk;
    sk.reverse = true;
    if (r == 1) {
        sv.o = dv; sv.o_ld = dv_ld;
        sk.o = dk; sk.o_ld = dk_ld;
    } else {   // each head's own share in fp32, summed over the group below
        sv.o = ws + w.part_v; sv.o_ld = HV; sv.o_f32 = true;
        sk.o = ws + w.part_k; sk.o_ld = HK; sk.o_f32 = true;
    }
    for (int i = 0; i < 3; ++i) s[i].seg_states = (float*)(ws + w.seg + i * w.seg_each);
    c.taken = c.status + 1;
    if (ssd::set_clear_status(&c, st) != cudaSuccess) return SSD_ERR_CUDA;
    const ssd_status rs = run(c, s, 3, st);
    if (rs != SSD_OK || r == 1) return rs;
    if (ssd::launch_linear_group_sum((const float*)(ws + w.part_k), dk, dk_ld, c.T, d->ngroups, r, d->dk, d->act, st) != cudaSuccess ||
        ssd::launch_linear_group_sum((const float*)(ws + w.part_v), dv, dv_ld, c.T, d->ngroups, r, d->dv, d->act, st) != cudaSuccess)
        return SSD_ERR_CUDA;
    return SSD_OK;
}

}  // extern "C"
