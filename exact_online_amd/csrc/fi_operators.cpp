// fi_operators.cpp -- host side of the operators around the mixers
// (fi_lattn_*, fi_dense_*, fi_scores_*, fi_delta_*, fi_rotary_*, fi_verify_* of
// include/fi.h): argument checks, workspaces and launches.
#include "fi_operators.h"

#include <hip/hip_runtime_api.h>

#include <cmath>
#include <new>
#include <vector>

#include "fi.h"
#include "fi_host.h"

using namespace fi;

struct fi_lattn {
    fi_lattn_config cfg;
    hipStream_t stream;
    float *ld;     // [Hkv] log decay, device
    float *ws;     // entry states of a split prompt's segments
};

struct fi_dense {
    fi_dense_config cfg;
    hipStream_t stream;
    float *part;   // partial sums of products split over K
};

struct fi_scores {
    fi_scores_config cfg;
    hipStream_t stream;
    float *pst;                  // partial sums and alternatives of rows' parts
    unsigned long long *pkey;
};

struct fi_delta {
    fi_delta_config cfg;
    hipStream_t stream;
    int device;
    float *ws;       // chunks' systems, segments' states
};

struct fi_rotary {
    fi_rotary_config cfg;
    hipStream_t stream;
    int device;
    double *turns;   // [rot / 2], device
};

struct fi_verify {
    fi_verify_config cfg;
    hipStream_t stream;
    int device;
    double *ws;      // sums of rows' parts
};

namespace {

constexpr int64_t kLim = (int64_t)1 << 31;
constexpr int64_t kMaxHead = 256;            // largest head size of fi_lattn
constexpr int64_t kMaxCount = (int64_t)1 << 46;   // elements of one array

#define FI_HIP(expr)                                      \
    do {                                                  \
        hipError_t e_ = (expr);                           \
        if (e_ != hipSuccess) return fi::hip_fail(e_);    \
    } while (0)

bool dtype_ok(int v) { return v == FI_F32 || v == FI_BF16; }
int esize(int dt) { return dt == FI_BF16 ? 2 : 4; }
bool aligned(const void *p, int64_t to) { return reinterpret_cast<uintptr_t>(p) % (uintptr_t)to == 0; }

// a * b * ... of factors >= 1 within `most`
bool fits(std::initializer_list<int64_t> f, int64_t most) {
    int64_t n = 1;
    for (int64_t v : f) {
        if (v > most / n) return false;
        n *= v;
    }
    return true;
}

// The handle's device is the current one as long as this lives.
struct OnDevice {
    int before = -1;
    hipError_t error;
    explicit OnDevice(int device) {
        error = hipGetDevice(&before);
        if (error != hipSuccess || before == device) before = -1;
        else error = hipSetDevice(device);
    }
    ~OnDevice() {
        if (before >= 0) (void)hipSetDevice(before);
    }
};

}  // namespace

extern "C" {

// ------------------------------------------------------------ linear attention
int fi_lattn_create(const fi_lattn_config *cfg, const float *log_decay, fi_lattn **out) {
    if (out) *out = nullptr;
    if (!cfg || !log_decay || !out) return FI_ERR_INVALID;
    if (cfg->B < 1 || cfg->L < 1 || cfg->H < 1 || cfg->Hkv < 1 || cfg->dk < 1 || cfg->dv < 1) return FI_ERR_INVALID;
    if (cfg->B >= kLim || cfg->L >= kLim || cfg->H >= kLim) return FI_ERR_INVALID;
    if (cfg->H % cfg->Hkv != 0 || !std::isfinite(cfg->scale) || !dtype_ok(raw_int(cfg->io_dtype))) return FI_ERR_INVALID;
    if (!fits({cfg->B, cfg->L, cfg->H, cfg->dk}, kMaxCount) || !fits({cfg->B, cfg->L, cfg->H, cfg->dv}, kMaxCount))
        return FI_ERR_INVALID;
    if (cfg->dk > kMaxHead || cfg->dv > kMaxHead || cfg->L > FI_MAX_L || cfg->B > kLattnMaxRows / cfg->Hkv)
        return FI_ERR_UNSUPPORTED;
    int rc = check_device();
    if (rc != FI_OK) return rc;
    fi_lattn *s = new (std::nothrow) fi_lattn();
    if (!s) return FI_ERR_NOMEM;
    s->cfg = *cfg;
    s->stream = static_cast<hipStream_t>(cfg->stream);
    s->ld = s->ws = nullptr;
    const size_t bytes = (size_t)cfg->Hkv * sizeof(float);
    float *host = new (std::nothrow) float[(size_t)cfg->Hkv];
    hipError_t e = host ? dalloc(&s->ld, bytes) : hipErrorOutOfMemory;
    if (e == hipSuccess) e = hipMemcpyAsync(s->ld, log_decay, bytes, hipMemcpyDeviceToDevice, s->stream);
    if (e == hipSuccess) e = hipMemcpyAsync(host, log_decay, bytes, hipMemcpyDeviceToHost, s->stream);
    if (e == hipSuccess) e = hipStreamSynchronize(s->stream);
    const size_t ws = lattn_ws_bytes(cfg->B, cfg->L, (int)cfg->H, (int)cfg->Hkv, (int)cfg->dk, (int)cfg->dv,
                                     raw_int(cfg->io_dtype) == FI_BF16);
    if (e == hipSuccess && ws > 0) e = dalloc(&s->ws, ws);
    bool ok = e == hipSuccess;
    for (int64_t n = 0; ok && n < cfg->Hkv; ++n) ok = host[n] <= 0.f;   // false for NaN
    delete[] host;
    if (e != hipSuccess || !ok) {
        fi_lattn_destroy(s);
        return e != hipSuccess ? hip_fail(e) : FI_ERR_INVALID;
    }
    *out = s;
    return FI_OK;
}

void fi_lattn_destroy(fi_lattn *s) {
    if (!s) return;
    (void)hipStreamSynchronize(s->stream);
    if (s->ld) (void)hipFree(s->ld);
    if (s->ws) (void)hipFree(s->ws);
    delete s;
}

}  // extern "C"

namespace {

// a view's whole heads load in 16-byte units, and the rows of a chunk (at most
// 64) span less than 2^31 bytes
bool view_vec(const fi_view &v, int64_t d, int es) {
    const int64_t u = 16 / es;
    return v.pos >= 0 && v.pos < ((int64_t)1 << 22) && aligned(v.p, 16) && v.row % u == 0 && v.pos % u == 0 && v.head % u == 0 && d % u == 0;
}

int lattn_call(const fi_lattn *s, const fi_lattn_args *a, LattnCall &c) {
    if (!s || !a) return FI_ERR_INVALID;
    const fi_lattn_config &f = s->cfg;
    if (a->B < 0 || a->B > f.B || a->L < 0 || a->L > f.L) return FI_ERR_INVALID;
    const int dt = raw_int(f.io_dtype), es = esize(dt);
    const bool some = a->B > 0 && a->L > 0;   // an empty call's arrays may be NULL
    for (const fi_view *v : {&a->q, &a->k, &a->v, &a->o})
        if ((some && !v->p) || !aligned(v->p, es)) return FI_ERR_INVALID;
    if ((!a->state && !a->fresh) || !aligned(a->state, 16) || !aligned(a->lens, 4) || !aligned(a->slots, 4))
        return FI_ERR_INVALID;
    if (a->n_slots < 0 || a->n_slots >= kLim || (!a->slots && a->state && a->n_slots < a->B)) return FI_ERR_INVALID;
    c.B = a->B;
    c.L = (int)a->L;
    c.H = (int)f.H;
    c.Hkv = (int)f.Hkv;
    c.G = (int)(f.H / f.Hkv);
    c.dk = (int)f.dk;
    c.dv = (int)f.dv;
    c.scale = f.scale;
    c.io_bf16 = dt == FI_BF16;
    c.fresh = a->fresh != 0;
    c.vec = view_vec(a->q, f.dk, es) && view_vec(a->k, f.dk, es) && view_vec(a->v, f.dv, es) && view_vec(a->o, f.dv, es);
    c.ld = s->ld;
    auto view = [](const fi_view &v) { return View{v.p, v.row, v.pos, v.head}; };
    c.q = view(a->q);
    c.k = view(a->k);
    c.v = view(a->v);
    c.o = view(a->o);
    c.lens = a->lens;
    c.slots = a->slots;
    c.n_slots = a->state ? a->n_slots : kLim;   // without states every slot is fine
    c.state = a->state;
    c.ws = s->ws;
    c.nseg = 1;
    c.seg_chunks = 0;
    return FI_OK;
}

}  // namespace

extern "C" {

int fi_lattn_prompt(fi_lattn *s, const fi_lattn_args *a) {
    LattnCall c;
    const int rc = lattn_call(s, a, c);
    if (rc != FI_OK || c.B == 0) return rc;
    // a single position: the recurrent form, which needs no chunk (5 us for 7 to 12)
    FI_HIP(c.L == 1 && c.state ? launch_lattn_step(c, s->stream) : launch_lattn_chunk(c, s->stream));
    return FI_OK;
}

int fi_lattn_step(fi_lattn *s, const fi_lattn_args *a) {
    LattnCall c;
    const int rc = lattn_call(s, a, c);
    if (rc != FI_OK) return rc;
    if (a->L != 1 || a->lens) return FI_ERR_INVALID;
    if (c.B == 0) return FI_OK;
    if (!c.state) return FI_ERR_INVALID;   // every step leaves its state behind
    FI_HIP(launch_lattn_step(c, s->stream));
    return FI_OK;
}

// ------------------------------------------------------------ dense product
int fi_dense_create(const fi_dense_config *cfg, fi_dense **out) {
    if (out) *out = nullptr;
    if (!cfg || !out) return FI_ERR_INVALID;
    if (cfg->M < 1 || cfg->N < 1 || cfg->K < 1 || cfg->M >= kLim || cfg->N >= kLim || cfg->K >= kLim) return FI_ERR_INVALID;
    const int act = raw_int(cfg->act);
    if (!dtype_ok(raw_int(cfg->io_dtype)) || !dtype_ok(raw_int(cfg->out_dtype))) return FI_ERR_INVALID;
    if (act != FI_ACT_GELU && act != FI_ACT_TANH && act != FI_ACT_IDENTITY) return FI_ERR_INVALID;
    if (cfg->M > kDenseMaxRows || cfg->N > kDenseMaxRows) return FI_ERR_UNSUPPORTED;
    const int rc = check_device();
    if (rc != FI_OK) return rc;
    fi_dense *s = new (std::nothrow) fi_dense();
    if (!s) return FI_ERR_NOMEM;
    s->cfg = *cfg;
    s->stream = static_cast<hipStream_t>(cfg->stream);
    s->part = nullptr;
    const size_t ws = dense_ws_bytes(cfg->M, cfg->N, cfg->K, raw_int(cfg->io_dtype) == FI_BF16);
    const hipError_t e = ws > 0 ? dalloc(&s->part, ws) : hipSuccess;
    if (e != hipSuccess) {
        delete s;
        return hip_fail(e);
    }
    *out = s;
    return FI_OK;
}

int fi_dense_run(fi_dense *s, const fi_dense_args *a) {
    if (!s || !a || a->M < 0 || a->M > s->cfg.M) return FI_ERR_INVALID;
    if (a->M == 0) return FI_OK;   // no rows: their arrays may be NULL
    if (!a->x || !a->w || !a->y) return FI_ERR_INVALID;
    const fi_dense_config &f = s->cfg;
    if (a->ldx < f.K || a->ldw < f.K || a->ldy < f.N || (a->res && a->ldr < f.N)) return FI_ERR_INVALID;
    if (!fits({a->ldx, f.M}, kMaxCount) || !fits({a->ldw, f.N}, kMaxCount) || !fits({a->ldy, f.M}, kMaxCount) ||
        (a->res && !fits({a->ldr, f.M}, kMaxCount)))
        return FI_ERR_INVALID;
    const int io = raw_int(f.io_dtype), od = raw_int(f.out_dtype);
    if (!aligned(a->x, esize(io)) || !aligned(a->w, esize(io)) || !aligned(a->bias, esize(io)) ||
        !aligned(a->res, esize(od)) || !aligned(a->y, esize(od)))
        return FI_ERR_INVALID;
    const DenseCall c{a->M, f.N, f.K, io == FI_BF16, od == FI_BF16, raw_int(f.act), a->x, a->w, a->bias, a->res, a->y,
                      a->ldx, a->ldw, a->ldr, a->ldy, s->part, 0, 0, 1};
    FI_HIP(launch_dense(c, s->stream));
    return FI_OK;
}

void fi_dense_destroy(fi_dense *s) {
    if (!s) return;
    (void)hipStreamSynchronize(s->stream);
    if (s->part) (void)hipFree(s->part);
    delete s;
}

// ------------------------------------------------------------ token scores
int fi_scores_create(const fi_scores_config *cfg, fi_scores **out) {
    if (out) *out = nullptr;
    if (!cfg || !out) return FI_ERR_INVALID;
    if (cfg->rows < 1 || cfg->V < 1 || cfg->rows >= kLim || cfg->V >= kLim) return FI_ERR_INVALID;
    if (cfg->k < 0 || cfg->k > FI_SCORES_MAX_K || !dtype_ok(raw_int(cfg->io_dtype))) return FI_ERR_INVALID;
    if (!(cfg->scale > 0.f) || !std::isfinite(cfg->scale)) return FI_ERR_INVALID;
    const int rc = check_device();
    if (rc != FI_OK) return rc;
    fi_scores *s = new (std::nothrow) fi_scores();
    if (!s) return FI_ERR_NOMEM;
    s->cfg = *cfg;
    s->stream = static_cast<hipStream_t>(cfg->stream);
    s->pst = nullptr;
    s->pkey = nullptr;
    const size_t parts = scores_ws_parts(cfg->rows, cfg->V, raw_int(cfg->io_dtype) == FI_BF16);
    hipError_t e = hipSuccess;
    if (parts > 0) e = dalloc(&s->pst, parts * 3 * sizeof(float));
    if (e == hipSuccess && parts > 0 && cfg->k > 0) e = dalloc(&s->pkey, parts * cfg->k * sizeof(unsigned long long));
    if (e != hipSuccess) {
        fi_scores_destroy(s);
        return hip_fail(e);
    }
    *out = s;
    return FI_OK;
}

int fi_scores_run(fi_scores *s, const fi_scores_args *a) {
    if (!s || !a || a->rows < 0 || a->rows > s->cfg.rows) return FI_ERR_INVALID;
    if (a->rows == 0) return FI_OK;   // no rows: their arrays may be NULL
    const fi_scores_config &f = s->cfg;
    if (!a->logits || a->ld < f.V || !fits({a->ld, f.rows}, kMaxCount)) return FI_ERR_INVALID;
    if (!a->targets != !a->logprob || (f.k > 0 && (!a->top || !a->top_id))) return FI_ERR_INVALID;
    const int io = raw_int(f.io_dtype);
    if (!aligned(a->logits, esize(io)) || !aligned(a->targets, 8) || !aligned(a->top_id, 8)) return FI_ERR_INVALID;
    for (const float *p : {a->logprob, a->entropy, a->lse, a->top})
        if (!aligned(p, 4)) return FI_ERR_INVALID;
    const ScoresCall c{a->rows, f.V, a->ld, f.k, io == FI_BF16, f.scale, a->logits, a->targets, a->logprob, a->entropy,
                       a->lse, f.k > 0 ? a->top : nullptr, f.k > 0 ? a->top_id : nullptr, 1, 0, s->pst, s->pkey};
    FI_HIP(launch_scores(c, s->stream));
    return FI_OK;
}

void fi_scores_destroy(fi_scores *s) {
    if (!s) return;
    (void)hipStreamSynchronize(s->stream);
    if (s->pst) (void)hipFree(s->pst);
    if (s->pkey) (void)hipFree(s->pkey);
    delete s;
}

// ------------------------------------------------------------ gated delta rule
int fi_delta_create(const fi_delta_config *cfg, fi_delta **out) {
    if (out) *out = nullptr;
    if (!cfg || !out) return FI_ERR_INVALID;
    if (cfg->B < 1 || cfg->L < 1 || cfg->Hk < 1 || cfg->Hv < 1 || cfg->dk < 1 || cfg->dv < 1) return FI_ERR_INVALID;
    if (cfg->B >= kLim || cfg->L >= kLim || cfg->Hv >= kLim) return FI_ERR_INVALID;
    if (cfg->Hv % cfg->Hk != 0 || !std::isfinite(cfg->scale) || !dtype_ok(raw_int(cfg->io_dtype))) return FI_ERR_INVALID;
    if (!fits({cfg->B, cfg->L, cfg->Hv, cfg->dk}, kMaxCount) || !fits({cfg->B, cfg->L, cfg->Hv, cfg->dv}, kMaxCount))
        return FI_ERR_INVALID;
    if (cfg->dk > kMaxHead || cfg->dv > kMaxHead || cfg->L > FI_MAX_L || cfg->B > kLattnMaxRows / cfg->Hv)
        return FI_ERR_UNSUPPORTED;
    const int rc = check_device();
    if (rc != FI_OK) return rc;
    fi_delta *s = new (std::nothrow) fi_delta();
    if (!s) return FI_ERR_NOMEM;
    s->cfg = *cfg;
    s->stream = static_cast<hipStream_t>(cfg->stream);
    s->ws = nullptr;
    hipError_t e = hipGetDevice(&s->device);
    const size_t ws = delta_ws_bytes(cfg->B, cfg->L, (int)cfg->Hv, (int)cfg->dk, (int)cfg->dv, raw_int(cfg->io_dtype) == FI_BF16);
    if (e == hipSuccess && ws > 0) e = dalloc(&s->ws, ws);
    if (e != hipSuccess) {
        fi_delta_destroy(s);
        return hip_fail(e);
    }
    *out = s;
    return FI_OK;
}

void fi_delta_destroy(fi_delta *s) {
    if (!s) return;
    const OnDevice here(s->device);
    (void)hipStreamSynchronize(s->stream);
    if (s->ws) (void)hipFree(s->ws);
    delete s;
}

}  // extern "C"

namespace {

int delta_call(const fi_delta *s, const fi_delta_args *a, DeltaCall &c) {
    if (!s || !a) return FI_ERR_INVALID;
    const fi_delta_config &f = s->cfg;
    if (a->B < 0 || a->B > f.B || a->L < 0 || a->L > f.L) return FI_ERR_INVALID;
    const int dt = raw_int(f.io_dtype), es = esize(dt);
    const bool some = a->B > 0 && a->L > 0;   // an empty call's arrays may be NULL
    for (const fi_view *v : {&a->q, &a->k, &a->v, &a->o})
        if ((some && !v->p) || !aligned(v->p, es)) return FI_ERR_INVALID;
    for (const fi_view *v : {&a->log_decay, &a->beta})
        if ((some && !v->p) || !aligned(v->p, 4)) return FI_ERR_INVALID;
    if ((!a->state && !a->fresh) || !aligned(a->state, 16) || !aligned(a->lens, 4) || !aligned(a->slots, 4))
        return FI_ERR_INVALID;
    if (a->n_slots < 0 || a->n_slots >= kLim || (!a->slots && a->state && a->n_slots < a->B)) return FI_ERR_INVALID;
    c = {};
    c.B = a->B;
    c.L = (int)a->L;
    c.Hk = (int)f.Hk;
    c.Hv = (int)f.Hv;
    c.G = (int)(f.Hv / f.Hk);
    c.dk = (int)f.dk;
    c.dv = (int)f.dv;
    c.scale = f.scale;
    c.io_bf16 = dt == FI_BF16;
    c.fresh = a->fresh != 0;
    c.hold = a->hold != 0;
    c.vec = view_vec(a->q, f.dk, es) && view_vec(a->k, f.dk, es) && view_vec(a->v, f.dv, es) && view_vec(a->o, f.dv, es);
    auto view = [](const fi_view &v) { return View{v.p, v.row, v.pos, v.head}; };
    c.q = view(a->q);
    c.k = view(a->k);
    c.v = view(a->v);
    c.o = view(a->o);
    c.ld = view(a->log_decay);
    c.beta = view(a->beta);
    c.lens = a->lens;
    c.slots = a->slots;
    c.n_slots = a->state ? a->n_slots : kLim;   // without states every slot is fine
    c.state = a->state;
    return FI_OK;
}

}  // namespace

extern "C" {

int fi_delta_prompt(fi_delta *s, const fi_delta_args *a) {
    DeltaCall c;
    const int rc = delta_call(s, a, c);
    if (rc != FI_OK || c.B == 0) return rc;
    const OnDevice here(s->device);
    FI_HIP(here.error);
    FI_HIP(launch_delta_prompt(c, s->ws, s->stream));
    return FI_OK;
}

int fi_delta_step(fi_delta *s, const fi_delta_args *a) {
    DeltaCall c;
    const int rc = delta_call(s, a, c);
    if (rc != FI_OK) return rc;
    if (a->L != 1 || a->lens) return FI_ERR_INVALID;
    if (c.B == 0) return FI_OK;
    if (!c.state) return FI_ERR_INVALID;   // every step leaves its state behind
    const OnDevice here(s->device);
    FI_HIP(here.error);
    FI_HIP(launch_delta_step(c, s->stream));
    return FI_OK;
}

// ------------------------------------------------------------ normed and turned heads
int fi_rotary_create(const fi_rotary_config *cfg, const float *inv_freq, fi_rotary **out) {
    if (out) *out = nullptr;
    if (!cfg || !out || (!inv_freq && cfg->rot > 0)) return FI_ERR_INVALID;
    if (cfg->B < 1 || cfg->L < 1 || cfg->Hq < 1 || cfg->Hk < 0 || cfg->d < 1) return FI_ERR_INVALID;
    if (cfg->B >= kLim || cfg->L >= kLim || cfg->Hq >= kLim || cfg->Hk >= kLim) return FI_ERR_INVALID;
    if (cfg->rot < 0 || cfg->rot > cfg->d || cfg->rot % 2 != 0 || !(cfg->eps >= 0.f) || !std::isfinite(cfg->eps)) return FI_ERR_INVALID;
    const int norm = raw_int(cfg->norm), pairs = raw_int(cfg->pairs);
    if (norm != FI_NORM_NONE && norm != FI_NORM_RMS && norm != FI_NORM_L2) return FI_ERR_INVALID;
    if (pairs != FI_PAIRS_HALVES && pairs != FI_PAIRS_ADJACENT) return FI_ERR_INVALID;
    if (!dtype_ok(raw_int(cfg->io_dtype)) || !fits({cfg->B, cfg->L, cfg->Hq + cfg->Hk, cfg->d}, kMaxCount)) return FI_ERR_INVALID;
    if (cfg->d > kMaxHead) return FI_ERR_UNSUPPORTED;
    const int rc = check_device();
    if (rc != FI_OK) return rc;
    fi_rotary *s = new (std::nothrow) fi_rotary();
    if (!s) return FI_ERR_NOMEM;
    s->cfg = *cfg;
    s->stream = static_cast<hipStream_t>(cfg->stream);
    s->turns = nullptr;
    hipError_t e = hipGetDevice(&s->device);
    bool ok = true;
    if (cfg->rot > 0 && e == hipSuccess) {
        float freq[kMaxHead / 2];
        double turns[kMaxHead / 2];
        const int n = (int)cfg->rot / 2;
        e = hipMemcpyAsync(freq, inv_freq, n * sizeof(float), hipMemcpyDeviceToHost, s->stream);
        if (e == hipSuccess) e = hipStreamSynchronize(s->stream);
        for (int i = 0; e == hipSuccess && i < n; ++i) {
            ok = ok && std::isfinite(freq[i]);
            turns[i] = (double)freq[i] / 6.283185307179586476925;
        }
        if (e == hipSuccess) e = dalloc(&s->turns, n * sizeof(double));
        if (e == hipSuccess) e = hipMemcpyAsync(s->turns, turns, n * sizeof(double), hipMemcpyHostToDevice, s->stream);
        if (e == hipSuccess) e = hipStreamSynchronize(s->stream);
    }
    if (e != hipSuccess || !ok) {
        fi_rotary_destroy(s);
        return e != hipSuccess ? hip_fail(e) : FI_ERR_INVALID;
    }
    *out = s;
    return FI_OK;
}

void fi_rotary_destroy(fi_rotary *s) {
    if (!s) return;
    const OnDevice here(s->device);
    (void)hipStreamSynchronize(s->stream);
    if (s->turns) (void)hipFree(s->turns);
    delete s;
}

int fi_rotary_run(fi_rotary *s, const fi_rotary_args *a) {
    if (!s || !a) return FI_ERR_INVALID;
    const fi_rotary_config &f = s->cfg;
    if (a->B < 0 || a->B > f.B || a->L < 0 || a->L > f.L) return FI_ERR_INVALID;
    if (a->B == 0 || a->L == 0) return FI_OK;   // their arrays may be NULL
    const int dt = raw_int(f.io_dtype), es = esize(dt);
    if (!a->q.p || !a->qo.p || (f.Hk > 0 && (!a->k.p || !a->ko.p)) || (a->first && a->positions)) return FI_ERR_INVALID;
    const bool keys = f.Hk > 0;
    int unit = 16 / es;   // elements that load at once
    const auto narrow = [&](int64_t n) {
        while (n % unit) unit /= 2;
    };
    for (const fi_view *v : {&a->q, &a->qo, &a->k, &a->ko}) {
        if (!keys && (v == &a->k || v == &a->ko)) continue;
        if (!aligned(v->p, es)) return FI_ERR_INVALID;
        while (!aligned(v->p, (int64_t)unit * es)) unit /= 2;
        narrow(v->row);
        narrow(v->pos);
        narrow(v->head);
    }
    for (const void *w : {a->wq, keys ? a->wk : nullptr}) {
        if (!aligned(w, es)) return FI_ERR_INVALID;
        while (!aligned(w, (int64_t)unit * es)) unit /= 2;
    }
    if (!aligned(a->first, 4) || !aligned(a->positions, 4)) return FI_ERR_INVALID;
    narrow(f.d);
    if (raw_int(f.pairs) == FI_PAIRS_HALVES) narrow(f.rot / 2);
    auto view = [](const fi_view &v) { return View{v.p, v.row, v.pos, v.head}; };
    const RotaryCall c{a->B, (int)a->L, (int)f.Hq, (int)f.Hk, (int)f.d, (int)f.rot, raw_int(f.norm), raw_int(f.pairs), dt == FI_BF16,
                       f.eps, s->turns, view(a->q), view(a->k), view(a->qo), view(a->ko), a->wq, a->wk, a->first, a->positions,
                       unit, 1};
    const OnDevice here(s->device);
    FI_HIP(here.error);
    FI_HIP(launch_rotary(c, s->stream));
    return FI_OK;
}

// ------------------------------------------------------------ drafted tokens
int fi_verify_create(const fi_verify_config *cfg, fi_verify **out) {
    if (out) *out = nullptr;
    if (!cfg || !out) return FI_ERR_INVALID;
    if (cfg->B < 1 || cfg->N < 0 || cfg->V < 1 || cfg->B >= kLim || cfg->N > FI_VERIFY_MAX_DRAFTS || cfg->V >= kLim) return FI_ERR_INVALID;
    if (!dtype_ok(raw_int(cfg->io_dtype))) return FI_ERR_INVALID;
    for (float x : {cfg->scale, cfg->draft_scale})
        if (!(x > 0.f) || !std::isfinite(x)) return FI_ERR_INVALID;
    if (cfg->B > kVerifyMaxRows / (2 * cfg->N + 1)) return FI_ERR_UNSUPPORTED;
    const int rc = check_device();
    if (rc != FI_OK) return rc;
    fi_verify *s = new (std::nothrow) fi_verify();
    if (!s) return FI_ERR_NOMEM;
    s->cfg = *cfg;
    s->stream = static_cast<hipStream_t>(cfg->stream);
    s->ws = nullptr;
    hipError_t e = hipGetDevice(&s->device);
    const size_t n = verify_ws_doubles(cfg->B, (int)cfg->N, cfg->V);
    if (e == hipSuccess) e = dalloc(&s->ws, n * sizeof(double));
    if (e != hipSuccess) {
        fi_verify_destroy(s);
        return hip_fail(e);
    }
    *out = s;
    return FI_OK;
}

void fi_verify_destroy(fi_verify *s) {
    if (!s) return;
    const OnDevice here(s->device);
    (void)hipStreamSynchronize(s->stream);
    if (s->ws) (void)hipFree(s->ws);
    delete s;
}

int fi_verify_run(fi_verify *s, const fi_verify_args *a) {
    if (!s || !a) return FI_ERR_INVALID;
    const fi_verify_config &f = s->cfg;
    if (a->B < 0 || a->B > f.B || a->N < 0 || a->N > f.N) return FI_ERR_INVALID;
    if (a->B == 0) return FI_OK;   // no rows: their arrays may be NULL
    if (!a->target || !a->r || !a->out || !a->kept || (a->N > 0 && (!a->tokens || !a->u))) return FI_ERR_INVALID;
    if (a->target_row < 0 || a->target_ld < 0 || a->draft_row < 0 || a->draft_ld < 0) return FI_ERR_INVALID;
    const int io = raw_int(f.io_dtype);
    const bool draft = a->draft && a->N > 0;
    const auto within = [&](int64_t n, int64_t stride) { return stride <= kMaxCount / n; };
    if (!within(a->B, a->target_row) || !within(a->N + 1, a->target_ld) || (draft && (!within(a->B, a->draft_row) || !within(a->N, a->draft_ld))))
        return FI_ERR_INVALID;
    if (!aligned(a->target, esize(io)) || !aligned(a->draft, esize(io)) || !aligned(a->tokens, 8) || !aligned(a->out, 8)) return FI_ERR_INVALID;
    for (const void *p : {(const void *)a->lens, (const void *)a->u, (const void *)a->r, (const void *)a->kept, (const void *)a->logprob})
        if (!aligned(p, 4)) return FI_ERR_INVALID;
    VerifyCall c{};
    c.B = a->B;
    c.V = f.V;
    c.N = (int)a->N;
    c.io_bf16 = io == FI_BF16;
    c.scale = (double)f.scale * kVerifyOctave;
    c.draft_scale = (double)f.draft_scale * kVerifyOctave;
    c.target = a->target;
    c.target_row = a->target_row;
    c.target_ld = a->target_ld;
    c.draft = draft ? a->draft : nullptr;
    c.draft_row = a->draft_row;
    c.draft_ld = a->draft_ld;
    c.tokens = a->tokens;
    c.lens = a->lens;
    c.u = a->u;
    c.r = a->r;
    c.out = a->out;
    c.kept = a->kept;
    c.logprob = a->logprob;
    c.sums = s->ws;
    const OnDevice here(s->device);
    FI_HIP(here.error);
    FI_HIP(launch_verify(c, s->stream));
    return FI_OK;
}

}  // extern "C"
