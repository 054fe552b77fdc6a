// C ABI of the gated delta rule (declared in include/ssd.h): argument checks, workspace
// layout and launch order. Host-only; allocates nothing and does not synchronise.
#include <hip/hip_runtime.h>

#include <initializer_list>

#include "../../include/ssd.h"
#include "ssd_launch.h"

using ssd::DeltaArgs;
using ssd::Dims;

namespace {

size_t round_up(size_t v) { return (v + 255) / 256 * 256; }

bool aligned16(std::initializer_list<const void*> ps) {
    for (const void* p : ps)
        if ((uintptr_t)p & 15u) return false;
    return true;
}
bool given(std::initializer_list<const void*> ps) {
    for (const void* p : ps)
        if (!p) return false;
    return true;
}
bool one_of(int64_t v, std::initializer_list<int64_t> set) {
    for (int64_t s : set)
        if (v == s) return true;
    return false;
}

double nchunks(const ssd_shape* s) { return (double)((s->seqlen + ssd::kDeltaChunk - 1) / ssd::kDeltaChunk); }

ssd_status check(const ssd_shape* s, bool out_used) {
    if (!s) return SSD_ERR_NULL;
    if (s->batch < 1 || s->seqlen < 0 || s->nheads < 1 || s->headdim < 1 || s->dstate < 1 || s->ngroups < 1 ||
        s->nheads % s->ngroups != 0)
        return SSD_ERR_SHAPE;
    if (!one_of(s->in_dtype, {SSD_F32, SSD_BF16}) || (out_used && !one_of(s->out_dtype, {SSD_F32, SSD_BF16})))
        return SSD_ERR_DTYPE;
    if (out_used && s->out_dtype == SSD_BF16 && s->in_dtype != SSD_BF16) return SSD_ERR_UNSUPPORTED;
    if (!one_of(s->headdim, {16, 32, 64, 128}) || !one_of(s->dstate, {16, 32, 64, 128, 256}))
        return SSD_ERR_UNSUPPORTED;
    // sizes as doubles first: products of int64 sizes may not fit
    const double tokens = (double)s->batch * s->seqlen, heads = (double)s->batch * s->nheads;
    if ((double)s->seqlen > 2.0e9 || tokens * s->nheads * s->headdim > 2.0e9 ||
        tokens * s->ngroups * s->dstate > 2.0e9 || heads * s->headdim * s->dstate > 2.0e9 ||
        heads * nchunks(s) * s->headdim > 2.0e9)
        return SSD_ERR_UNSUPPORTED;
    // a chunk's rows lie within one buffer descriptor, and a grid has fewer than 2^32 threads
    if ((double)s->nheads * s->headdim * ssd::kDeltaChunk * 4 >= 2147483648.0 ||
        (double)s->ngroups * s->dstate * ssd::kDeltaChunk * 4 >= 2147483648.0 || heads * nchunks(s) > 1.6e7)
        return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

Dims dims_of(const ssd_shape* s) {
    Dims d;
    d.batch = (int)s->batch;
    d.seqlen = (int)s->seqlen;
    d.nheads = (int)s->nheads;
    d.headdim = (int)s->headdim;
    d.dstate = (int)s->dstate;
    d.ngroups = (int)s->ngroups;
    d.chunk = ssd::kDeltaChunk;
    return d;
}

struct Sizes {
    size_t scal, mat, state, rows, part, ends, starts, total;
};
Sizes sizes(const ssd_shape* s, bool backward) {
    Sizes z = {};
    const Dims d = dims_of(s);
    if (d.seqlen == 0 || (!backward && ssd::delta_recurrent_preferred(s->in_dtype, d))) return z;
    const size_t n = (size_t)d.batch * d.nheads * d.nchunks();
    z.scal = round_up(n * ssd::kDeltaScal * sizeof(float));
    z.mat = round_up(n * ssd::kDeltaMatBytes);
    z.total = z.scal + 2 * z.mat;
    if (!backward) {
        const ssd::DeltaSegs sg = ssd::delta_segments(s->in_dtype, d);
        if (sg.nseg > 1) {
            const size_t heads = (size_t)d.batch * d.nheads;
            z.ends = round_up(heads * (sg.nseg - 1) * (d.headdim + d.dstate) * d.dstate * sizeof(float));
            z.starts = round_up(heads * sg.nseg * d.headdim * d.dstate * sizeof(float));
            z.total += z.ends + z.starts;
        }
    } else {
        z.state = round_up(n * d.headdim * d.dstate * sizeof(float));
        z.rows = round_up(n * ssd::kDeltaChunk * d.headdim * sizeof(float));
        const int parts = ssd::delta_bwd_parts(d);
        z.part = parts > 1 ? round_up((size_t)parts * d.batch * d.seqlen * d.ngroups * d.dstate * sizeof(float)) : 0;
        z.total += z.mat + 2 * z.state + 3 * z.rows + 2 * z.part;
    }
    return z;
}

struct Carver {
    char* at;
    template <typename T> void take(T*& p, size_t n) {
        p = n ? (T*)at : nullptr;
        at += n;
    }
};

hipError_t walk(const ssd_shape* s, bool save, const DeltaArgs& a, const Dims& d, hipStream_t stream) {
    return s->in_dtype == SSD_BF16 ? ssd::launch_delta_walk_bf16(s->out_dtype, save, a, d, stream)
                                   : ssd::launch_delta_walk_f32(save, a, d, stream);
}
hipError_t reverse(const ssd_shape* s, const DeltaArgs& a, const Dims& d, hipStream_t stream) {
    return s->in_dtype == SSD_BF16 ? ssd::launch_delta_reverse_bf16(a, d, stream)
                                   : ssd::launch_delta_reverse_f32(a, d, stream);
}

ssd_status status_of(hipError_t e) { return e == hipSuccess ? SSD_OK : SSD_ERR_HIP; }

#define SSD_REQUIRE(cond, code) \
    do {                        \
        if (!(cond)) return code; \
    } while (0)

}  // namespace

extern "C" {

ssd_status ssd_delta_forward_workspace_bytes(const ssd_shape* shape, size_t* bytes) {
    SSD_REQUIRE(bytes, SSD_ERR_NULL);
    const ssd_status st = check(shape, true);
    if (st != SSD_OK) return st;
    *bytes = sizes(shape, false).total;
    return SSD_OK;
}

ssd_status ssd_delta_forward(const ssd_shape* shape, const void* v, const float* g, const void* beta,
                             const void* k, const void* q, const float* h0, float scale, void* y,
                             float* final_state, void* workspace, size_t workspace_bytes, void* stream) {
    const ssd_status st = check(shape, true);
    if (st != SSD_OK) return st;
    const bool empty = shape->seqlen == 0;  // only the final state (= h0) is written
    SSD_REQUIRE(empty || given({v, g, beta, k, q, y}), SSD_ERR_NULL);
    SSD_REQUIRE(aligned16({v, g, beta, k, q, h0, y, final_state}), SSD_ERR_ALIGN);
    const Sizes z = sizes(shape, false);
    SSD_REQUIRE(workspace_bytes >= z.total && (z.total == 0 || workspace), SSD_ERR_WORKSPACE);
    SSD_REQUIRE(aligned16({workspace}), SSD_ERR_ALIGN);
    const Dims d = dims_of(shape);
    hipStream_t s = (hipStream_t)stream;
    if (empty) return final_state ? status_of(ssd::launch_state_init(h0, final_state, d, s)) : SSD_OK;
    DeltaArgs a = {};
    a.v = v; a.g = g; a.beta = beta; a.k = k; a.q = q; a.h0 = h0; a.scale = scale;
    a.y = y; a.final_state = final_state;
    if (z.total == 0) return status_of(ssd::launch_delta_recurrent(shape->in_dtype, shape->out_dtype, a, d, s));
    Carver w = {(char*)workspace};
    w.take(a.scal, z.scal);
    w.take(a.matT, z.mat);
    w.take(a.matM, z.mat);
    w.take(a.seg_ends, z.ends);
    w.take(a.seg_starts, z.starts);
    hipError_t e = ssd::launch_delta_prep(shape->in_dtype, false, a, d, s);
    if (e == hipSuccess) e = walk(shape, false, a, d, s);
    return status_of(e);
}

ssd_status ssd_delta_forward_plan(const ssd_shape* shape, int32_t* segments, int32_t* waves,
                                  int32_t* first_waves, int32_t* prep_heads) {
    const ssd_status st = check(shape, true);
    if (st != SSD_OK) return st;
    const Dims d = dims_of(shape);
    int n = 0, w = 0, first = 0, hb = 0;
    if (sizes(shape, false).total > 0) {
        const long heads = (long)d.batch * d.nheads;
        n = ssd::delta_segments(shape->in_dtype, d).nseg;
        w = ssd::delta_waves(heads * n, d.headdim);
        first = n > 1 ? ssd::delta_waves(heads * (n - 1), ssd::delta_first_rows(d)) : 0;
        hb = ssd::delta_prep_heads(d);
    }
    if (segments) *segments = n;
    if (waves) *waves = w;
    if (first_waves) *first_waves = first;
    if (prep_heads) *prep_heads = hb;
    return SSD_OK;
}

ssd_status ssd_delta_decode_step(const ssd_shape* shape, const void* v, const float* g, const void* beta,
                                 const void* k, const void* q, const float* state, float scale,
                                 float* state_out, float* y, void* stream) {
    const ssd_status st = check(shape, false);
    if (st != SSD_OK) return st;
    SSD_REQUIRE(shape->seqlen == 1, SSD_ERR_SHAPE);
    SSD_REQUIRE(given({v, g, beta, k, q, state, state_out, y}), SSD_ERR_NULL);
    SSD_REQUIRE(aligned16({v, g, beta, k, q, state, state_out, y}), SSD_ERR_ALIGN);
    DeltaArgs a = {};
    a.v = v; a.g = g; a.beta = beta; a.k = k; a.q = q; a.h0 = state; a.scale = scale;
    a.y = y; a.final_state = state_out;
    return status_of(ssd::launch_delta_recurrent(shape->in_dtype, SSD_F32, a, dims_of(shape), (hipStream_t)stream));
}

ssd_status ssd_delta_backward_workspace_bytes(const ssd_shape* shape, size_t* bytes) {
    SSD_REQUIRE(bytes, SSD_ERR_NULL);
    const ssd_status st = check(shape, false);
    if (st != SSD_OK) return st;
    *bytes = sizes(shape, true).total;
    return SSD_OK;
}

ssd_status ssd_delta_backward_plan(const ssd_shape* shape, int32_t* waves, int32_t* prep_heads,
                                   int32_t* grad_heads) {
    const ssd_status st = check(shape, false);
    if (st != SSD_OK) return st;
    const Dims d = dims_of(shape);
    const bool empty = d.seqlen == 0;
    const int hpg = d.nheads / d.ngroups, parts = ssd::delta_bwd_parts(d);
    if (waves) *waves = empty ? 0 : ssd::delta_waves((long)d.batch * d.nheads, d.headdim);
    if (prep_heads) *prep_heads = empty ? 0 : ssd::delta_prep_heads(d);
    if (grad_heads) *grad_heads = empty ? 0 : (hpg + parts - 1) / parts;
    return SSD_OK;
}

ssd_status ssd_delta_backward(const ssd_shape* shape, const void* v, const float* g, const void* beta,
                              const void* k, const void* q, const float* h0, const float* dy,
                              const float* dfinal, float scale, float* dv, float* dg, float* dbeta,
                              float* dk, float* dq, float* dh0, void* workspace, size_t workspace_bytes,
                              void* stream) {
    const ssd_status st = check(shape, false);
    if (st != SSD_OK) return st;
    const bool empty = shape->seqlen == 0;  // only dh0 (= dfinal) is written
    SSD_REQUIRE(empty || given({v, g, beta, k, q, dy, dv, dg, dbeta, dk, dq}), SSD_ERR_NULL);
    SSD_REQUIRE(aligned16({v, g, beta, k, q, h0, dy, dfinal, dv, dg, dbeta, dk, dq, dh0}), SSD_ERR_ALIGN);
    const Sizes z = sizes(shape, true);
    SSD_REQUIRE(workspace_bytes >= z.total && (z.total == 0 || workspace), SSD_ERR_WORKSPACE);
    SSD_REQUIRE(aligned16({workspace}), SSD_ERR_ALIGN);
    const Dims d = dims_of(shape);
    hipStream_t s = (hipStream_t)stream;
    if (empty) return dh0 ? status_of(ssd::launch_state_init(dfinal, dh0, d, s)) : SSD_OK;
    DeltaArgs a = {};
    a.v = v; a.g = g; a.beta = beta; a.k = k; a.q = q; a.h0 = h0; a.scale = scale;
    a.dy = dy; a.dfinal = dfinal; a.dv = dv; a.dg = dg; a.dbeta = dbeta; a.dk = dk; a.dq = dq; a.dh0 = dh0;
    Carver w = {(char*)workspace};
    w.take(a.scal, z.scal);
    w.take(a.matT, z.mat);
    w.take(a.matM, z.mat);
    w.take(a.matTt, z.mat);
    w.take(a.Hc, z.state);
    w.take(a.Ec, z.state);
    w.take(a.Ut, z.rows);
    w.take(a.Nt, z.rows);
    w.take(a.Zt, z.rows);
    w.take(a.dkp, z.part);
    w.take(a.dqp, z.part);
    hipError_t e = ssd::launch_delta_prep(shape->in_dtype, true, a, d, s);
    if (e == hipSuccess) e = walk(shape, true, a, d, s);
    if (e == hipSuccess) e = reverse(shape, a, d, s);
    if (e == hipSuccess) e = ssd::launch_delta_grads(shape->in_dtype, a, d, s);
    return status_of(e);
}

}  // extern "C"
