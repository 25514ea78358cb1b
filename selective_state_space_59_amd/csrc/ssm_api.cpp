// ssm_api.cpp -- the C ABI declared in include/ssm.h: argument checking,
// dispatch to the kernel launchers, status strings.  Nothing here allocates
// device memory or keeps state between calls (apart from the per-thread text
// of the last error and the block plans the caller creates and destroys).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdarg>
#include <cstdio>
#include <cstdint>
#include <climits>

#include "ssm_internal.h"

namespace {

thread_local char g_last_error[512] = "";

ssm_status_t fail(ssm_status_t s, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_last_error, sizeof(g_last_error), fmt, ap);
    va_end(ap);
    return s;
}

ssm_status_t ok() {
    g_last_error[0] = '\0';
    return SSM_OK;
}

struct Range {
    uintptr_t lo, hi;  // [lo, hi)
    const char *name;
};

Range range(const void *p, int64_t count, int64_t elem, const char *name) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return Range{lo, p ? lo + (uintptr_t)(count * elem) : lo, name};
}

bool overlaps(const Range &a, const Range &b) {
    if (a.lo == a.hi || b.lo == b.hi) return false;  // empty or absent
    return a.lo < b.hi && b.lo < a.hi;
}

int64_t io_bytes(int32_t dt) { return dt == SSM_BF16 ? 2 : 4; }

bool aligned(const void *p, int64_t a) { return (reinterpret_cast<uintptr_t>(p) % (uintptr_t)a) == 0; }

// Products of non-negative sizes that must stay far from int64 overflow.
bool mul_ok(int64_t a, int64_t b, int64_t c = 1) {
    const int64_t lim = (int64_t)1 << 60;
    if (a == 0 || b == 0 || c == 0) return true;
    if (a > lim / b) return false;
    const int64_t ab = a * b;
    return ab <= lim / c;
}

// Elements of a checkpoint buffer, (ceil(L / SSM_SCAN_BLOCK), B, D, SSM_MAX_DSTATE),
// or -1 where that product is too large.
int64_t checkpoint_elems(int64_t B, int64_t L, int64_t D) {
    const int64_t nblk = (L + SSM_SCAN_BLOCK - 1) / SSM_SCAN_BLOCK;
    if (!mul_ok(B, D) || !mul_ok(nblk, B * D, SSM_MAX_DSTATE)) return -1;
    return nblk * B * D * SSM_MAX_DSTATE;
}

ssm_status_t check_scan_sizes(const ssm_scan_args_t *a) {
    if (!a) return fail(SSM_ERR_NULL_ARG, "args is NULL");
    if (a->io_dtype != SSM_F32 && a->io_dtype != SSM_BF16)
        return fail(SSM_ERR_BAD_DTYPE, "io_dtype %d is not SSM_F32 or SSM_BF16", a->io_dtype);
    if (a->batch < 0 || a->seqlen < 0)
        return fail(SSM_ERR_BAD_SHAPE, "negative batch (%lld) or seqlen (%lld)",
                    (long long)a->batch, (long long)a->seqlen);
    if (a->dim < 1) return fail(SSM_ERR_BAD_SHAPE, "dim must be >= 1 (got %lld)", (long long)a->dim);
    if (a->dstate < 1) return fail(SSM_ERR_BAD_SHAPE, "dstate must be >= 1 (got %lld)", (long long)a->dstate);
    if (a->dstate > SSM_MAX_DSTATE)
        return fail(SSM_ERR_UNSUPPORTED, "dstate %lld exceeds SSM_MAX_DSTATE (%d)",
                    (long long)a->dstate, SSM_MAX_DSTATE);
    if (a->conv_k < 0) return fail(SSM_ERR_BAD_SHAPE, "conv_k must be >= 0");
    if (a->conv_k > SSM_MAX_CONV_K)
        return fail(SSM_ERR_UNSUPPORTED, "conv_k %lld exceeds SSM_MAX_CONV_K (%d)",
                    (long long)a->conv_k, SSM_MAX_CONV_K);
    if (a->delta_softplus != 0 && a->delta_softplus != 1)
        return fail(SSM_ERR_UNSUPPORTED, "delta_softplus must be 0 or 1");
    if (!mul_ok(a->batch, a->seqlen, a->dim) || !mul_ok(a->batch, a->seqlen, a->dstate) ||
        !mul_ok(a->batch, a->dim, a->dstate))
        return fail(SSM_ERR_BAD_SHAPE, "sizes overflow");
    if (a->checkpoints && checkpoint_elems(a->batch, a->seqlen, a->dim) < 0)
        return fail(SSM_ERR_BAD_SHAPE, "checkpoint sizes overflow");
    return SSM_OK;
}

}  // namespace

extern "C" {

int ssm_abi_version(void) { return SSM_ABI_VERSION; }

const char *ssm_last_error_message(void) { return g_last_error; }

const char *ssm_status_string(ssm_status_t s) {
    switch (s) {
        case SSM_OK: return "SSM_OK: success";
        case SSM_ERR_NULL_ARG: return "SSM_ERR_NULL_ARG: a required pointer is NULL";
        case SSM_ERR_BAD_SHAPE: return "SSM_ERR_BAD_SHAPE: a size is negative or inconsistent";
        case SSM_ERR_BAD_DTYPE: return "SSM_ERR_BAD_DTYPE: unknown io_dtype";
        case SSM_ERR_UNSUPPORTED: return "SSM_ERR_UNSUPPORTED: size or option beyond what the kernels support";
        case SSM_ERR_ALIAS: return "SSM_ERR_ALIAS: an output overlaps another argument";
        case SSM_ERR_WORKSPACE: return "SSM_ERR_WORKSPACE: workspace missing, too small or misaligned";
        case SSM_ERR_HIP: return "SSM_ERR_HIP: the HIP runtime reported an error";
        case SSM_ERR_ALIGN: return "SSM_ERR_ALIGN: a pointer is not aligned to its element size";
    }
    return "unknown ssm_status_t";
}

size_t ssm_selective_scan_workspace_size(const ssm_scan_args_t *a) {
    if (check_scan_sizes(a) != SSM_OK) return (size_t)-1;
    if (a->batch == 0 || a->seqlen == 0) return 0;
    return ssm::scan_workspace_bytes(*a);
}

}  // extern "C"

namespace {

// The checks and launch of both scan entry points.  With `noalloc` the
// workspace comes from the library's scratch array and the caller passes none.
ssm_status_t scan_fwd(const ssm_scan_args_t *a, void *stream, bool noalloc) {
    ssm_status_t s = check_scan_sizes(a);
    if (s != SSM_OK) return s;
    const int64_t B = a->batch, L = a->seqlen, D = a->dim, N = a->dstate, K = a->conv_k;
    const int64_t es = io_bytes(a->io_dtype);
    const bool work = B > 0 && L > 0;
    if (work) {
        if (!a->x) return fail(SSM_ERR_NULL_ARG, "x is NULL");
        if (!a->delta) return fail(SSM_ERR_NULL_ARG, "delta is NULL");
        if (!a->Bm) return fail(SSM_ERR_NULL_ARG, "Bm is NULL");
        if (!a->Cm) return fail(SSM_ERR_NULL_ARG, "Cm is NULL");
        if (!a->A) return fail(SSM_ERR_NULL_ARG, "A is NULL");
        if (!a->y) return fail(SSM_ERR_NULL_ARG, "y is NULL");
        if (K > 0 && !a->conv_w) return fail(SSM_ERR_NULL_ARG, "conv_w is NULL but conv_k > 0");
    }
    if (K == 0 && (a->conv_w || a->conv_b || a->conv_state_in || a->conv_state_out))
        return fail(SSM_ERR_BAD_SHAPE, "conv_w/conv_b/conv state given but conv_k == 0");
    const void *io_ptrs[] = {a->x, a->delta, a->Bm, a->Cm, a->z, a->y, a->conv_state_in,
                             a->conv_state_out};
    for (const void *p : io_ptrs)
        if (!aligned(p, es)) return fail(SSM_ERR_ALIGN, "an io_dtype pointer is not %lld-byte aligned", (long long)es);
    const void *f_ptrs[] = {a->A, a->Dskip, a->delta_bias, a->conv_w, a->conv_b, a->h0, a->h_final,
                            a->checkpoints};
    for (const void *p : f_ptrs)
        if (!aligned(p, 4)) return fail(SSM_ERR_ALIGN, "an fp32 pointer is not 4-byte aligned");

    const int64_t csn = B * (K > 0 ? K - 1 : 0) * D;  // elements of a conv state
    const Range csi = range(a->conv_state_in, csn, es, "conv_state_in");
    const Range inputs[] = {
        range(a->x, B * L * D, es, "x"),          range(a->delta, B * L * D, es, "delta"),
        range(a->Bm, B * L * N, es, "Bm"),        range(a->Cm, B * L * N, es, "Cm"),
        range(a->z, B * L * D, es, "z"),          range(a->A, D * N, 4, "A"),
        range(a->Dskip, D, 4, "Dskip"),           range(a->delta_bias, D, 4, "delta_bias"),
        range(a->conv_w, D * K, 4, "conv_w"),     range(a->conv_b, D, 4, "conv_b"),
        range(a->h0, B * D * N, 4, "h0"),
        csi,
    };
    const Range y = range(a->y, B * L * D, es, "y");
    const Range hf = range(a->h_final, B * D * N, 4, "h_final");
    const Range cso = range(a->conv_state_out, csn, es, "conv_state_out");
    // The conv state may be updated in place (the same tensor in and out).
    const bool cs_in_place = a->conv_state_out != nullptr && a->conv_state_out == a->conv_state_in;
    for (const Range &r : inputs) {
        if (overlaps(y, r)) return fail(SSM_ERR_ALIAS, "y overlaps %s", r.name);
        if (overlaps(hf, r)) return fail(SSM_ERR_ALIAS, "h_final overlaps %s", r.name);
        if (!(cs_in_place && &r == &inputs[sizeof(inputs) / sizeof(inputs[0]) - 1]) && overlaps(cso, r))
            return fail(SSM_ERR_ALIAS, "conv_state_out overlaps %s", r.name);
    }
    if (overlaps(y, hf)) return fail(SSM_ERR_ALIAS, "y overlaps h_final");
    if (overlaps(cso, y) || overlaps(cso, hf)) return fail(SSM_ERR_ALIAS, "conv_state_out overlaps an output");
    const int64_t nck = a->checkpoints ? checkpoint_elems(B, L, D) : 0;  // >= 0 (checked above)
    const Range ck = range(a->checkpoints, nck, 4, "checkpoints");
    for (const Range &r : inputs)
        if (overlaps(ck, r)) return fail(SSM_ERR_ALIAS, "checkpoints overlap %s", r.name);
    if (overlaps(ck, y) || overlaps(ck, hf) || overlaps(ck, cso))
        return fail(SSM_ERR_ALIAS, "checkpoints overlap an output");

    const size_t need = work ? ssm::scan_workspace_bytes(*a) : 0;
    if (noalloc) {
        if (a->workspace || a->workspace_bytes)
            return fail(SSM_ERR_WORKSPACE, "the no-allocation scan takes no workspace (use its scratch array)");
        if (need > (size_t)SSM_NOALLOC_SCRATCH_BYTES)
            return fail(SSM_ERR_WORKSPACE, "these sizes need %zu bytes of workspace; the no-allocation "
                        "scan has %zu (use ssm_selective_scan_fwd with a workspace)",
                        need, (size_t)SSM_NOALLOC_SCRATCH_BYTES);
    } else if (need > 0) {
        if (!a->workspace) return fail(SSM_ERR_WORKSPACE, "workspace of %zu bytes required", need);
        if (a->workspace_bytes < need)
            return fail(SSM_ERR_WORKSPACE, "workspace has %zu bytes, %zu required", a->workspace_bytes, need);
        if (!aligned(a->workspace, 256)) return fail(SSM_ERR_WORKSPACE, "workspace is not 256-byte aligned");
        const Range ws = range(a->workspace, (int64_t)need, 1, "workspace");
        for (const Range &r : inputs)
            if (overlaps(ws, r)) return fail(SSM_ERR_ALIAS, "workspace overlaps %s", r.name);
        if (overlaps(ws, y) || overlaps(ws, hf) || overlaps(ws, cso) || overlaps(ws, ck))
            return fail(SSM_ERR_ALIAS, "workspace overlaps an output");
    }

    hipStream_t st = static_cast<hipStream_t>(stream);
    hipError_t e = hipSuccess;
    if (B == 0) return ok();
    if (L == 0) {
        e = ssm::launch_empty_scan_state(*a, st);
    } else if (noalloc && need > 0) {
        ssm_scan_args_t b = *a;
        e = ssm::noalloc_scratch(st, &b.workspace);
        if (e != hipSuccess)
            return fail(SSM_ERR_HIP, "scratch array address: %s", hipGetErrorString(e));
        b.workspace_bytes = SSM_NOALLOC_SCRATCH_BYTES;
        e = ssm::launch_scan_fwd(b, st);
    } else {
        e = ssm::launch_scan_fwd(*a, st);
    }
    if (e != hipSuccess) return fail(SSM_ERR_HIP, "HIP error: %s", hipGetErrorString(e));
    return ok();
}

}  // namespace

extern "C" {

ssm_status_t ssm_selective_scan_fwd(const ssm_scan_args_t *a, void *stream) {
    return scan_fwd(a, stream, false);
}

ssm_status_t ssm_selective_scan_fwd_noalloc(const ssm_scan_args_t *a, void *stream) {
    return scan_fwd(a, stream, true);
}

ssm_status_t ssm_causal_conv1d_silu(int64_t B, int64_t L, int64_t D, int64_t K, int32_t io_dtype,
                                    const void *x, const float *w, const float *bias, void *u,
                                    void *stream) {
    if (io_dtype != SSM_F32 && io_dtype != SSM_BF16)
        return fail(SSM_ERR_BAD_DTYPE, "io_dtype %d is not SSM_F32 or SSM_BF16", io_dtype);
    if (B < 0 || L < 0) return fail(SSM_ERR_BAD_SHAPE, "negative batch or seqlen");
    if (D < 1) return fail(SSM_ERR_BAD_SHAPE, "dim must be >= 1");
    if (K < 1) return fail(SSM_ERR_BAD_SHAPE, "k must be >= 1");
    if (K > SSM_MAX_CONV_K) return fail(SSM_ERR_UNSUPPORTED, "k %lld exceeds SSM_MAX_CONV_K (%d)", (long long)K, SSM_MAX_CONV_K);
    if (!mul_ok(B, L, D)) return fail(SSM_ERR_BAD_SHAPE, "sizes overflow");
    const int64_t es = io_bytes(io_dtype);
    if (B == 0 || L == 0) return ok();
    if (!x) return fail(SSM_ERR_NULL_ARG, "x is NULL");
    if (!w) return fail(SSM_ERR_NULL_ARG, "w is NULL");
    if (!u) return fail(SSM_ERR_NULL_ARG, "u is NULL");
    if (!aligned(x, es) || !aligned(u, es) || !aligned(w, 4) || !aligned(bias, 4))
        return fail(SSM_ERR_ALIGN, "a pointer is not aligned to its element size");
    const Range ur = range(u, B * L * D, es, "u");
    if (overlaps(ur, range(x, B * L * D, es, "x")) || overlaps(ur, range(w, D * K, 4, "w")) ||
        overlaps(ur, range(bias, D, 4, "bias")))
        return fail(SSM_ERR_ALIAS, "u overlaps an input");
    hipError_t e = ssm::launch_conv1d_silu(B, L, D, (int)K, io_dtype, x, w, bias, u,
                                           static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return fail(SSM_ERR_HIP, "HIP error: %s", hipGetErrorString(e));
    return ok();
}

ssm_status_t ssm_state_update(const ssm_state_update_args_t *a, void *stream) {
    if (!a) return fail(SSM_ERR_NULL_ARG, "args is NULL");
    if (a->io_dtype != SSM_F32 && a->io_dtype != SSM_BF16)
        return fail(SSM_ERR_BAD_DTYPE, "io_dtype %d is not SSM_F32 or SSM_BF16", a->io_dtype);
    if (a->batch < 0) return fail(SSM_ERR_BAD_SHAPE, "negative batch");
    if (a->dim < 1) return fail(SSM_ERR_BAD_SHAPE, "dim must be >= 1");
    if (a->dstate < 1) return fail(SSM_ERR_BAD_SHAPE, "dstate must be >= 1");
    if (a->dstate > SSM_MAX_DSTATE)
        return fail(SSM_ERR_UNSUPPORTED, "dstate %lld exceeds SSM_MAX_DSTATE (%d)", (long long)a->dstate, SSM_MAX_DSTATE);
    if (a->delta_softplus != 0 && a->delta_softplus != 1)
        return fail(SSM_ERR_UNSUPPORTED, "delta_softplus must be 0 or 1");
    if (!mul_ok(a->batch, a->dim, a->dstate)) return fail(SSM_ERR_BAD_SHAPE, "sizes overflow");
    if (a->conv_k < 0) return fail(SSM_ERR_BAD_SHAPE, "conv_k must be >= 0");
    if (a->conv_k > SSM_MAX_CONV_K)
        return fail(SSM_ERR_UNSUPPORTED, "conv_k %lld exceeds SSM_MAX_CONV_K (%d)", (long long)a->conv_k, SSM_MAX_CONV_K);
    if (a->conv_k == 0 && (a->conv_w || a->conv_b || a->conv_state))
        return fail(SSM_ERR_BAD_SHAPE, "conv_w/conv_b/conv_state given but conv_k == 0");
    if (a->conv_k > 0 && a->dim > ((int64_t)1 << 28))
        return fail(SSM_ERR_UNSUPPORTED, "dim %lld with a conv window exceeds 2^28", (long long)a->dim);
    const int64_t B = a->batch, D = a->dim, N = a->dstate, K = a->conv_k;
    const int64_t es = io_bytes(a->io_dtype);
    if (B == 0) return ok();
    if (!a->state) return fail(SSM_ERR_NULL_ARG, "state is NULL");
    if (!a->x) return fail(SSM_ERR_NULL_ARG, "x is NULL");
    if (!a->delta) return fail(SSM_ERR_NULL_ARG, "delta is NULL");
    if (!a->Bm) return fail(SSM_ERR_NULL_ARG, "Bm is NULL");
    if (!a->Cm) return fail(SSM_ERR_NULL_ARG, "Cm is NULL");
    if (!a->A) return fail(SSM_ERR_NULL_ARG, "A is NULL");
    if (!a->y) return fail(SSM_ERR_NULL_ARG, "y is NULL");
    if (K > 0 && !a->conv_w) return fail(SSM_ERR_NULL_ARG, "conv_w is NULL but conv_k > 0");
    if (K > 1 && !a->conv_state) return fail(SSM_ERR_NULL_ARG, "conv_state is NULL but conv_k > 1");
    const void *io_ptrs[] = {a->x, a->delta, a->z, a->Bm, a->Cm, a->y, a->conv_state};
    for (const void *p : io_ptrs)
        if (!aligned(p, es)) return fail(SSM_ERR_ALIGN, "an io_dtype pointer is not %lld-byte aligned", (long long)es);
    const void *f_ptrs[] = {a->state, a->A, a->Dskip, a->delta_bias, a->conv_w, a->conv_b};
    for (const void *p : f_ptrs)
        if (!aligned(p, 4)) return fail(SSM_ERR_ALIGN, "an fp32 pointer is not 4-byte aligned");
    const Range st = range(a->state, B * D * N, 4, "state");
    const Range y = range(a->y, B * D, es, "y");
    const Range inputs[] = {
        range(a->x, B * D, es, "x"),   range(a->delta, B * D, es, "delta"),
        range(a->z, B * D, es, "z"),   range(a->Bm, B * N, es, "Bm"),
        range(a->Cm, B * N, es, "Cm"), range(a->A, D * N, 4, "A"),
        range(a->Dskip, D, 4, "Dskip"), range(a->delta_bias, D, 4, "delta_bias"),
        range(a->conv_w, D * K, 4, "conv_w"), range(a->conv_b, D, 4, "conv_b"),
    };
    const Range cs = range(K > 1 ? a->conv_state : nullptr, B * (K > 0 ? K - 1 : 0) * D, es, "conv_state");
    for (const Range &r : inputs) {
        if (overlaps(y, r)) return fail(SSM_ERR_ALIAS, "y overlaps %s", r.name);
        if (overlaps(st, r)) return fail(SSM_ERR_ALIAS, "state overlaps %s", r.name);
        if (overlaps(cs, r)) return fail(SSM_ERR_ALIAS, "conv_state overlaps %s", r.name);
    }
    if (overlaps(y, st)) return fail(SSM_ERR_ALIAS, "y overlaps state");
    if (overlaps(cs, y) || overlaps(cs, st)) return fail(SSM_ERR_ALIAS, "conv_state overlaps an output");
    hipError_t e = ssm::launch_state_update(*a, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return fail(SSM_ERR_HIP, "HIP error: %s", hipGetErrorString(e));
    return ok();
}

static ssm_status_t check_bwd(const ssm_scan_bwd_args_t *a, size_t *need_out) {
    if (!a) return fail(SSM_ERR_NULL_ARG, "args is NULL");
    if (a->io_dtype != SSM_F32 && a->io_dtype != SSM_BF16)
        return fail(SSM_ERR_BAD_DTYPE, "io_dtype %d is not SSM_F32 or SSM_BF16", a->io_dtype);
    if (a->batch < 0 || a->seqlen < 0)
        return fail(SSM_ERR_BAD_SHAPE, "negative batch (%lld) or seqlen (%lld)", (long long)a->batch,
                    (long long)a->seqlen);
    if (a->dim < 1) return fail(SSM_ERR_BAD_SHAPE, "dim must be >= 1");
    if (a->dstate < 1) return fail(SSM_ERR_BAD_SHAPE, "dstate must be >= 1");
    if (a->dstate > SSM_MAX_DSTATE)
        return fail(SSM_ERR_UNSUPPORTED, "dstate %lld exceeds SSM_MAX_DSTATE (%d)", (long long)a->dstate,
                    SSM_MAX_DSTATE);
    if (a->conv_k < 0) return fail(SSM_ERR_BAD_SHAPE, "conv_k must be >= 0");
    if (a->conv_k > SSM_MAX_CONV_K)
        return fail(SSM_ERR_UNSUPPORTED, "conv_k %lld exceeds SSM_MAX_CONV_K (%d)", (long long)a->conv_k, SSM_MAX_CONV_K);
    if (a->conv_k == 0 && (a->conv_w || a->conv_b || a->dconv_w || a->dconv_b))
        return fail(SSM_ERR_BAD_SHAPE, "conv weights or their gradients given but conv_k == 0");
    if (a->conv_k < 2 && (a->conv_state_in || a->dconv_state_in))
        return fail(SSM_ERR_BAD_SHAPE, "a conv state or its gradient given but conv_k < 2");
    if (a->delta_softplus != 0 && a->delta_softplus != 1)
        return fail(SSM_ERR_UNSUPPORTED, "delta_softplus must be 0 or 1");
    // (the backward's checkpoints, in its workspace or the caller's, must be addressable too)
    if (!mul_ok(a->batch, a->seqlen, a->dim) || !mul_ok(a->batch, a->seqlen, a->dstate) ||
        !mul_ok(a->batch, a->dim, a->dstate) || checkpoint_elems(a->batch, a->seqlen, a->dim) < 0)
        return fail(SSM_ERR_BAD_SHAPE, "sizes overflow");
    const int64_t B = a->batch, L = a->seqlen, D = a->dim, N = a->dstate, K = a->conv_k;
    const int64_t es = io_bytes(a->io_dtype);
    *need_out = (B > 0) ? ssm::scan_bwd_workspace_bytes(*a) : 0;
    if (B == 0) return SSM_OK;
    if (!a->A) return fail(SSM_ERR_NULL_ARG, "A is NULL");
    if (!a->dA) return fail(SSM_ERR_NULL_ARG, "dA is NULL");
    if (K > 0 && !a->conv_w) return fail(SSM_ERR_NULL_ARG, "conv_w is NULL but conv_k > 0");
    if (K > 0 && !a->dconv_w) return fail(SSM_ERR_NULL_ARG, "dconv_w is NULL but conv_k > 0");
    if (L > 0) {
        const struct { const void *p; const char *name; } req[] = {
            {a->x, "x"}, {a->delta, "delta"}, {a->Bm, "Bm"}, {a->Cm, "Cm"}, {a->dy, "dy"},
            {a->dx, "dx"}, {a->ddelta, "ddelta"}, {a->dBm, "dBm"}, {a->dCm, "dCm"}};
        for (const auto &r : req)
            if (!r.p) return fail(SSM_ERR_NULL_ARG, "%s is NULL", r.name);
        if (a->z && !a->dz) return fail(SSM_ERR_NULL_ARG, "dz is NULL but z is given");
    }
    if (!a->z && a->dz) return fail(SSM_ERR_BAD_SHAPE, "dz given without z");
    const void *io_ptrs[] = {a->x, a->delta, a->Bm, a->Cm, a->z, a->dy, a->dx, a->ddelta, a->dz,
                             a->conv_state_in, a->dconv_state_in};
    for (const void *p : io_ptrs)
        if (!aligned(p, es)) return fail(SSM_ERR_ALIGN, "an io_dtype pointer is not %lld-byte aligned", (long long)es);
    const void *f_ptrs[] = {a->A, a->Dskip, a->delta_bias, a->h0, a->dh_final, a->dA, a->dBm, a->dCm,
                            a->dDskip, a->ddelta_bias, a->dh0, a->conv_w, a->conv_b, a->dconv_w, a->dconv_b,
                            a->checkpoints};
    for (const void *p : f_ptrs)
        if (!aligned(p, 4)) return fail(SSM_ERR_ALIGN, "an fp32 pointer is not 4-byte aligned");
    const int64_t nck = a->checkpoints ? checkpoint_elems(B, L, D) : 0;
    if (nck < 0) return fail(SSM_ERR_BAD_SHAPE, "checkpoint sizes overflow");
    const Range inputs[] = {
        range(a->x, B * L * D, es, "x"),          range(a->delta, B * L * D, es, "delta"),
        range(a->Bm, B * L * N, es, "Bm"),        range(a->Cm, B * L * N, es, "Cm"),
        range(a->z, B * L * D, es, "z"),          range(a->dy, B * L * D, es, "dy"),
        range(a->A, D * N, 4, "A"),               range(a->Dskip, D, 4, "Dskip"),
        range(a->delta_bias, D, 4, "delta_bias"), range(a->h0, B * D * N, 4, "h0"),
        range(a->dh_final, B * D * N, 4, "dh_final"), range(a->conv_w, D * K, 4, "conv_w"),
        range(a->conv_b, D, 4, "conv_b"),
        range(a->conv_state_in, B * (K > 0 ? K - 1 : 0) * D, es, "conv_state_in"),
        range(a->checkpoints, nck, 4, "checkpoints"),
    };
    const Range outputs[] = {
        range(a->dx, B * L * D, es, "dx"),        range(a->ddelta, B * L * D, es, "ddelta"),
        range(a->dz, B * L * D, es, "dz"),        range(a->dA, D * N, 4, "dA"),
        range(a->dBm, B * L * N, 4, "dBm"),       range(a->dCm, B * L * N, 4, "dCm"),
        range(a->dDskip, D, 4, "dDskip"),         range(a->ddelta_bias, D, 4, "ddelta_bias"),
        range(a->dh0, B * D * N, 4, "dh0"),         range(a->dconv_w, D * K, 4, "dconv_w"),
        range(a->dconv_b, D, 4, "dconv_b"),
        range(a->dconv_state_in, B * (K > 0 ? K - 1 : 0) * D, es, "dconv_state_in"),
    };
    const int nout = (int)(sizeof(outputs) / sizeof(outputs[0]));
    for (int i = 0; i < nout; ++i) {
        for (const Range &r : inputs)
            if (overlaps(outputs[i], r)) return fail(SSM_ERR_ALIAS, "%s overlaps %s", outputs[i].name, r.name);
        for (int k = i + 1; k < nout; ++k)
            if (overlaps(outputs[i], outputs[k]))
                return fail(SSM_ERR_ALIAS, "%s overlaps %s", outputs[i].name, outputs[k].name);
    }
    if (*need_out > 0) {
        if (!a->workspace) return fail(SSM_ERR_WORKSPACE, "workspace of %zu bytes required", *need_out);
        if (a->workspace_bytes < *need_out)
            return fail(SSM_ERR_WORKSPACE, "workspace has %zu bytes, %zu required", a->workspace_bytes, *need_out);
        if (!aligned(a->workspace, 256)) return fail(SSM_ERR_WORKSPACE, "workspace is not 256-byte aligned");
        const Range ws = range(a->workspace, (int64_t)*need_out, 1, "workspace");
        for (const Range &r : inputs)
            if (overlaps(ws, r)) return fail(SSM_ERR_ALIAS, "workspace overlaps %s", r.name);
        for (const Range &r : outputs)
            if (overlaps(ws, r)) return fail(SSM_ERR_ALIAS, "workspace overlaps %s", r.name);
    }
    return SSM_OK;
}

size_t ssm_selective_scan_bwd_workspace_size(const ssm_scan_bwd_args_t *a) {
    if (!a || a->batch < 0 || a->seqlen < 0 || a->dim < 1 || a->dstate < 1 || a->dstate > SSM_MAX_DSTATE ||
        !mul_ok(a->batch, a->seqlen, a->dim) || !mul_ok(a->batch, a->dim, a->dstate) ||
        checkpoint_elems(a->batch, a->seqlen, a->dim) < 0)
        return (size_t)-1;
    return a->batch > 0 ? ssm::scan_bwd_workspace_bytes(*a) : 0;
}

ssm_status_t ssm_selective_scan_bwd(const ssm_scan_bwd_args_t *a, void *stream) {
    size_t need = 0;
    const ssm_status_t s = check_bwd(a, &need);
    if (s != SSM_OK) return s;
    if (a->batch == 0) return ok();
    const hipError_t e = ssm::launch_scan_bwd(*a, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return fail(SSM_ERR_HIP, "HIP error: %s", hipGetErrorString(e));
    return ok();
}

ssm_status_t ssm_block_plan_create(const ssm_block_dims_t *d, ssm_block_plan_t **plan) {
    if (!plan) return fail(SSM_ERR_NULL_ARG, "plan is NULL");
    *plan = nullptr;
    if (!d) return fail(SSM_ERR_NULL_ARG, "dims is NULL");
    if (d->batch < 1 || d->seqlen < 1 || d->d_model < 1 || d->d_inner < 1 || d->dstate < 1 || d->dt_rank < 1)
        return fail(SSM_ERR_BAD_SHAPE, "block sizes must all be >= 1");
    if (d->dstate > SSM_MAX_DSTATE)
        return fail(SSM_ERR_UNSUPPORTED, "dstate %lld exceeds SSM_MAX_DSTATE (%d)", (long long)d->dstate,
                    SSM_MAX_DSTATE);
    if (d->d_model % 8 != 0 || d->d_inner % 8 != 0)
        return fail(SSM_ERR_UNSUPPORTED, "d_model and d_inner must be multiples of 8 (got %lld, %lld)",
                    (long long)d->d_model, (long long)d->d_inner);
    if (d->conv_k < 1 || d->conv_k > SSM_MAX_CONV_K)
        return fail(SSM_ERR_UNSUPPORTED, "conv_k must be 1..%d (got %lld)", SSM_MAX_CONV_K, (long long)d->conv_k);
    // hipBLASLt takes 32-bit sizes; the largest operands stay well inside them.
    const int64_t M = d->batch * d->seqlen;
    if (!mul_ok(d->batch, d->seqlen, 4 * (d->d_model + d->d_inner)) || M >= ((int64_t)1 << 30) ||
        d->d_model > INT32_MAX / 4 || d->d_inner > INT32_MAX / 4 || d->dt_rank > d->d_inner)
        return fail(SSM_ERR_BAD_SHAPE, "block sizes out of range (dt_rank <= d_inner, B*L < 2^30)");
    ssm_block_plan *p = nullptr;
    const ssm_status_t s = ssm::block_plan_create(*d, &p);
    if (s != SSM_OK) return fail(s, "could not set up the block's GEMMs (hipBLASLt handle or algorithm)");
    *plan = p;
    return ok();
}

size_t ssm_block_workspace_size(const ssm_block_plan_t *plan) {
    return plan ? ssm::block_workspace_bytes(*plan) : 0;
}

void ssm_block_plan_destroy(ssm_block_plan_t *plan) { ssm::block_plan_destroy(plan); }

ssm_status_t ssm_block_fwd(const ssm_block_plan_t *plan, const ssm_block_weights_t *w, const void *h_in,
                           void *h_out, void *workspace, size_t workspace_bytes, void *stream) {
    if (!plan || !w || !h_in || !h_out) return fail(SSM_ERR_NULL_ARG, "plan, weights, h_in and h_out are required");
    if (!w->norm_w || !w->w_in || !w->conv_w || !w->w_x || !w->w_dt || !w->dt_bias || !w->A || !w->w_out)
        return fail(SSM_ERR_NULL_ARG, "a required weight is NULL (only conv_b and Dskip are optional)");
    if (!(w->norm_eps > 0.0f) || !(w->norm_eps < 1e30f)) return fail(SSM_ERR_BAD_SHAPE, "norm_eps must be > 0");
    const ssm_block_dims_t &d = ssm::block_dims(*plan);
    const int64_t M = d.batch * d.seqlen, D = d.d_inner, N = d.dstate, R = d.dt_rank, dm = d.d_model;
    const void *bf[] = {w->w_in, w->w_x, w->w_dt, w->w_out, h_in, h_out, w->norm_w, w->dt_bias};
    for (const void *v : bf)
        if (!aligned(v, 16))
            return fail(SSM_ERR_ALIGN, "bf16 tensors, norm_w and dt_bias must be 16-byte aligned");
    const void *f4[] = {w->norm_w, w->conv_w, w->conv_b, w->dt_bias, w->A, w->Dskip};
    for (const void *v : f4)
        if (!aligned(v, 4)) return fail(SSM_ERR_ALIGN, "fp32 tensors must be 4-byte aligned");
    const size_t need = ssm::block_workspace_bytes(*plan);
    if (!workspace) return fail(SSM_ERR_WORKSPACE, "workspace of %zu bytes required", need);
    if (workspace_bytes < need)
        return fail(SSM_ERR_WORKSPACE, "workspace has %zu bytes, %zu required", workspace_bytes, need);
    if (!aligned(workspace, 256)) return fail(SSM_ERR_WORKSPACE, "workspace is not 256-byte aligned");
    const Range hi = range(h_in, M * dm, 2, "h_in"), ho = range(h_out, M * dm, 2, "h_out");
    if (h_in != h_out && overlaps(hi, ho)) return fail(SSM_ERR_ALIAS, "h_out overlaps h_in (other than in place)");
    const Range inputs[] = {hi,
                            range(w->norm_w, dm, 4, "norm_w"),
                            range(w->w_in, 2 * D * dm, 2, "w_in"),
                            range(w->conv_w, D * d.conv_k, 4, "conv_w"),
                            range(w->conv_b, D, 4, "conv_b"),
                            range(w->w_x, (R + 2 * N) * D, 2, "w_x"),
                            range(w->w_dt, D * R, 2, "w_dt"),
                            range(w->dt_bias, D, 4, "dt_bias"),
                            range(w->A, D * N, 4, "A"),
                            range(w->Dskip, D, 4, "Dskip"),
                            range(w->w_out, dm * D, 2, "w_out")};
    const Range ws = range(workspace, (int64_t)need, 1, "workspace");
    for (const Range &r : inputs) {
        if (overlaps(ws, r)) return fail(SSM_ERR_ALIAS, "workspace overlaps %s", r.name);
        if (&r != &inputs[0] && overlaps(ho, r)) return fail(SSM_ERR_ALIAS, "h_out overlaps %s", r.name);
    }
    if (overlaps(ws, ho)) return fail(SSM_ERR_ALIAS, "workspace overlaps h_out");
    const hipError_t e = ssm::launch_block_fwd(*plan, *w, h_in, h_out, workspace, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return fail(SSM_ERR_HIP, "HIP error: %s", hipGetErrorString(e));
    return ok();
}

namespace {
ssm_status_t check_ssd_sizes(const ssm_ssd_args_t *a) {
    if (!a) return fail(SSM_ERR_NULL_ARG, "args is NULL");
    if (a->io_dtype != SSM_F32 && a->io_dtype != SSM_BF16)
        return fail(SSM_ERR_BAD_DTYPE, "io_dtype %d is not SSM_F32 or SSM_BF16", a->io_dtype);
    if (a->batch < 0 || a->seqlen < 0) return fail(SSM_ERR_BAD_SHAPE, "negative batch or seqlen");
    if (a->nheads < 1 || a->headdim < 1 || a->ngroups < 1 || a->dstate < 1)
        return fail(SSM_ERR_BAD_SHAPE, "nheads, headdim, ngroups and dstate must be >= 1");
    if (a->nheads % a->ngroups != 0)
        return fail(SSM_ERR_BAD_SHAPE, "ngroups (%lld) must divide nheads (%lld)", (long long)a->ngroups,
                    (long long)a->nheads);
    if (!ssm::ssd_supported(a->headdim, a->dstate))
        return fail(SSM_ERR_UNSUPPORTED,
                    "SSD needs headdim a multiple of 32 up to 4096 and dstate 16, 32, 64 or 128 (got %lld, %lld)",
                    (long long)a->headdim, (long long)a->dstate);
    if (a->delta_softplus != 0 && a->delta_softplus != 1)
        return fail(SSM_ERR_UNSUPPORTED, "delta_softplus must be 0 or 1");
    const int64_t B = a->batch, L = a->seqlen, H = a->nheads, P = a->headdim, G = a->ngroups, N = a->dstate;
    if (!mul_ok(B, L, H * P) || !mul_ok(B, L, G * N) || !mul_ok(B, H, P * N))
        return fail(SSM_ERR_BAD_SHAPE, "sizes overflow");
    // one workgroup of 256 threads per (batch, head, 32 channels): the launch holds < 2^32 threads
    if (B * H * (P / 32) > ((int64_t)1 << 23))
        return fail(SSM_ERR_UNSUPPORTED, "batch * nheads * headdim / 32 (%lld) exceeds 2^23",
                    (long long)(B * H * (P / 32)));
    return SSM_OK;
}
}  // namespace

size_t ssm_ssd_workspace_size(const ssm_ssd_args_t *a) {
    if (check_ssd_sizes(a) != SSM_OK) return (size_t)-1;
    if (a->batch == 0 || a->seqlen == 0) return 0;
    return ssm::ssd_workspace_bytes(*a);
}

ssm_status_t ssm_ssd_fwd(const ssm_ssd_args_t *a, void *stream) {
    {
        const ssm_status_t s = check_ssd_sizes(a);
        if (s != SSM_OK) return s;
    }
    const int64_t B = a->batch, L = a->seqlen, H = a->nheads, P = a->headdim, G = a->ngroups, N = a->dstate;
    if (!a->A) return fail(SSM_ERR_NULL_ARG, "A is required");
    if (B * L > 0 && (!a->x || !a->delta || !a->Bm || !a->Cm || !a->y))
        return fail(SSM_ERR_NULL_ARG, "x, delta, Bm, Cm and y are required");
    const int64_t es = io_bytes(a->io_dtype);
    if (a->io_dtype == SSM_BF16) {
        const void *a16[] = {a->x, a->Bm, a->Cm, a->z, a->y};
        for (const void *v : a16)
            if (!aligned(v, 16)) return fail(SSM_ERR_ALIGN, "x, Bm, Cm, z and y must be 16-byte aligned");
        if (!aligned(a->delta, 2)) return fail(SSM_ERR_ALIGN, "delta must be 2-byte aligned");
    } else {
        // fp32: the B and C rows are read as 16-byte groups of 4 entries
        if (!aligned(a->Bm, 16) || !aligned(a->Cm, 16))
            return fail(SSM_ERR_ALIGN, "fp32 Bm and Cm must be 16-byte aligned");
        const void *a4io[] = {a->x, a->z, a->y, a->delta};
        for (const void *v : a4io)
            if (!aligned(v, 4)) return fail(SSM_ERR_ALIGN, "fp32 x, z, y and delta must be 4-byte aligned");
    }
    const void *a4[] = {a->A, a->Dskip, a->delta_bias, a->h0, a->h_final};
    for (const void *v : a4)
        if (!aligned(v, 4)) return fail(SSM_ERR_ALIGN, "fp32 tensors must be 4-byte aligned");
    if (a->io_dtype == SSM_F32 && (!aligned(a->h0, 16) || !aligned(a->h_final, 16)))
        return fail(SSM_ERR_ALIGN, "with fp32 I/O h0 and h_final must be 16-byte aligned");
    const Range inputs[] = {range(a->x, B * L * H * P, es, "x"), range(a->delta, B * L * H, es, "delta"),
                            range(a->A, H, 4, "A"), range(a->Bm, B * L * G * N, es, "Bm"),
                            range(a->Cm, B * L * G * N, es, "Cm"), range(a->Dskip, H, 4, "Dskip"),
                            range(a->z, B * L * H * P, es, "z"), range(a->delta_bias, H, 4, "delta_bias"),
                            range(a->h0, B * H * P * N, 4, "h0")};
    const Range y = range(a->y, B * L * H * P, es, "y"), hf = range(a->h_final, B * H * P * N, 4, "h_final");
    for (const Range &r : inputs) {
        if (overlaps(y, r)) return fail(SSM_ERR_ALIAS, "y overlaps %s", r.name);
        if (overlaps(hf, r)) return fail(SSM_ERR_ALIAS, "h_final overlaps %s", r.name);
    }
    if (overlaps(y, hf)) return fail(SSM_ERR_ALIAS, "h_final overlaps y");
    if (B == 0) return ok();
    const size_t need = L > 0 ? ssm::ssd_workspace_bytes(*a) : 0;
    if (need > 0) {
        if (!a->workspace) return fail(SSM_ERR_WORKSPACE, "workspace of %zu bytes required", need);
        if (a->workspace_bytes < need)
            return fail(SSM_ERR_WORKSPACE, "workspace has %zu bytes, %zu required", a->workspace_bytes, need);
        if (!aligned(a->workspace, 256)) return fail(SSM_ERR_WORKSPACE, "workspace is not 256-byte aligned");
        const Range ws = range(a->workspace, (int64_t)need, 1, "workspace");
        for (const Range &r : inputs)
            if (overlaps(ws, r)) return fail(SSM_ERR_ALIAS, "workspace overlaps %s", r.name);
        if (overlaps(ws, y) || overlaps(ws, hf)) return fail(SSM_ERR_ALIAS, "workspace overlaps an output");
    }
    const hipError_t e = ssm::launch_ssd_fwd(*a, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return fail(SSM_ERR_HIP, "HIP error: %s", hipGetErrorString(e));
    return ok();
}

ssm_status_t ssm_ssd_step(const ssm_ssd_step_args_t *a, void *stream) {
    if (!a) return fail(SSM_ERR_NULL_ARG, "args is NULL");
    if (a->io_dtype != SSM_F32 && a->io_dtype != SSM_BF16)
        return fail(SSM_ERR_BAD_DTYPE, "io_dtype %d is not SSM_F32 or SSM_BF16", a->io_dtype);
    if (a->batch < 0) return fail(SSM_ERR_BAD_SHAPE, "negative batch");
    if (a->nheads < 1 || a->headdim < 1 || a->ngroups < 1 || a->dstate < 1)
        return fail(SSM_ERR_BAD_SHAPE, "nheads, headdim, ngroups and dstate must be >= 1");
    if (a->nheads % a->ngroups != 0) return fail(SSM_ERR_BAD_SHAPE, "ngroups must divide nheads");
    if (a->io_dtype != SSM_BF16) return fail(SSM_ERR_UNSUPPORTED, "the SSD step takes bf16 I/O");
    if (!ssm::ssd_step_supported(a->dstate))
        return fail(SSM_ERR_UNSUPPORTED, "dstate must be a power of two from 4 to 256 (got %lld)",
                    (long long)a->dstate);
    if (a->delta_softplus != 0 && a->delta_softplus != 1)
        return fail(SSM_ERR_UNSUPPORTED, "delta_softplus must be 0 or 1");
    const int64_t B = a->batch, H = a->nheads, P = a->headdim, G = a->ngroups, N = a->dstate;
    if (!mul_ok(B, H, P * N) || B * H * P * (N / 4) > ((int64_t)1 << 31))
        return fail(SSM_ERR_BAD_SHAPE, "sizes out of range (B*H*P*N/4 <= 2^31)");
    if (B == 0) return ok();
    if (!a->state || !a->x || !a->delta || !a->A || !a->Bm || !a->Cm || !a->y)
        return fail(SSM_ERR_NULL_ARG, "state, x, delta, A, Bm, Cm and y are required");
    if (!aligned(a->state, 16)) return fail(SSM_ERR_ALIGN, "state must be 16-byte aligned");
    if (!aligned(a->Bm, 8) || !aligned(a->Cm, 8)) return fail(SSM_ERR_ALIGN, "Bm and Cm must be 8-byte aligned");
    const void *a2[] = {a->x, a->delta, a->z, a->y};
    for (const void *v : a2)
        if (!aligned(v, 2)) return fail(SSM_ERR_ALIGN, "bf16 tensors must be 2-byte aligned");
    const void *a4[] = {a->A, a->Dskip, a->delta_bias};
    for (const void *v : a4)
        if (!aligned(v, 4)) return fail(SSM_ERR_ALIGN, "fp32 tensors must be 4-byte aligned");
    const Range inputs[] = {range(a->x, B * H * P, 2, "x"), range(a->delta, B * H, 2, "delta"),
                            range(a->A, H, 4, "A"), range(a->Bm, B * G * N, 2, "Bm"),
                            range(a->Cm, B * G * N, 2, "Cm"), range(a->Dskip, H, 4, "Dskip"),
                            range(a->z, B * H * P, 2, "z"), range(a->delta_bias, H, 4, "delta_bias")};
    const Range st = range(a->state, B * H * P * N, 4, "state"), y = range(a->y, B * H * P, 2, "y");
    for (const Range &r : inputs) {
        if (overlaps(st, r)) return fail(SSM_ERR_ALIAS, "state overlaps %s", r.name);
        if (overlaps(y, r)) return fail(SSM_ERR_ALIAS, "y overlaps %s", r.name);
    }
    if (overlaps(y, st)) return fail(SSM_ERR_ALIAS, "y overlaps the state");
    const hipError_t e = ssm::launch_ssd_step(*a, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return fail(SSM_ERR_HIP, "HIP error: %s", hipGetErrorString(e));
    return ok();
}

}  // extern "C"

// ------------------------------------------------- gated recurrence and fused norms
namespace {

// Grids and lane offsets of the gated scan and the norms stay in 32 bits up to this width.
constexpr int64_t kMaxWidth = (int64_t)1 << 20;

bool io_ok(int32_t dt) { return dt == SSM_F32 || dt == SSM_BF16; }

// Every output against every input, the other outputs and the workspace.  `same_ok`: pairs
// (output, input) that may be the very same tensor.
struct SameOk {
    const void *out, *in;
};

ssm_status_t check_overlaps(const Range *in, int nin, const Range *out, int nout, const Range &ws,
                            SameOk s0 = SameOk{nullptr, nullptr}, SameOk s1 = SameOk{nullptr, nullptr}) {
    for (int i = 0; i < nout; ++i) {
        for (int k = 0; k < nin; ++k) {
            const bool same = out[i].lo == in[k].lo && out[i].hi == in[k].hi;
            const uintptr_t o = out[i].lo, n = in[k].lo;
            if (same && ((o == (uintptr_t)s0.out && n == (uintptr_t)s0.in) ||
                         (o == (uintptr_t)s1.out && n == (uintptr_t)s1.in)))
                continue;
            if (overlaps(out[i], in[k])) return fail(SSM_ERR_ALIAS, "%s overlaps %s", out[i].name, in[k].name);
        }
        for (int k = i + 1; k < nout; ++k)
            if (overlaps(out[i], out[k])) return fail(SSM_ERR_ALIAS, "%s overlaps %s", out[i].name, out[k].name);
        if (overlaps(ws, out[i])) return fail(SSM_ERR_ALIAS, "workspace overlaps %s", out[i].name);
    }
    for (int k = 0; k < nin; ++k)
        if (overlaps(ws, in[k])) return fail(SSM_ERR_ALIAS, "workspace overlaps %s", in[k].name);
    return SSM_OK;
}

ssm_status_t check_workspace(const void *ws, size_t have, size_t need) {
    if (need == 0) return SSM_OK;
    if (!ws) return fail(SSM_ERR_WORKSPACE, "workspace of %zu bytes required", need);
    if (have < need) return fail(SSM_ERR_WORKSPACE, "workspace has %zu bytes, %zu required", have, need);
    if (!aligned(ws, 256)) return fail(SSM_ERR_WORKSPACE, "workspace is not 256-byte aligned");
    return SSM_OK;
}

ssm_status_t check_align(const void *const *io, int nio, int64_t es, const void *const *f, int nf) {
    for (int i = 0; i < nio; ++i)
        if (!aligned(io[i], es))
            return fail(SSM_ERR_ALIGN, "an io_dtype pointer is not %lld-byte aligned", (long long)es);
    for (int i = 0; i < nf; ++i)
        if (!aligned(f[i], 4)) return fail(SSM_ERR_ALIGN, "an fp32 pointer is not 4-byte aligned");
    return SSM_OK;
}

#define COUNT(a) ((int)(sizeof(a) / sizeof((a)[0])))

// Sizes, types and the pairing of options shared by the gated scan, its backward and its step.
ssm_status_t check_gated(int64_t B, int64_t L, int64_t D, int32_t io, int32_t mode, const void *in_gate,
                         const float *A, const float *gate_bias, const float *in_bias) {
    if (!io_ok(io)) return fail(SSM_ERR_BAD_DTYPE, "io_dtype %d is not SSM_F32 or SSM_BF16", io);
    if (B < 0 || L < 0)
        return fail(SSM_ERR_BAD_SHAPE, "negative batch (%lld) or seqlen (%lld)", (long long)B, (long long)L);
    if (D < 1) return fail(SSM_ERR_BAD_SHAPE, "dim must be >= 1 (got %lld)", (long long)D);
    if (D > kMaxWidth) return fail(SSM_ERR_UNSUPPORTED, "dim %lld exceeds 2^20", (long long)D);
    if (mode != SSM_GATE_DECAY && mode != SSM_GATE_SIGMOID && mode != SSM_GATE_RATE)
        return fail(SSM_ERR_UNSUPPORTED, "mode %d is not one of ssm_gate_mode_t", mode);
    if (!mul_ok(B, L, 4 * D)) return fail(SSM_ERR_BAD_SHAPE, "sizes overflow");
    // a workgroup of up to 512 threads per 128 steps of 32 channels, fewer than 2^32 threads a launch
    const int64_t blocks = (std::max<int64_t>(L, 1) + SSM_GATED_BLOCK - 1) / SSM_GATED_BLOCK, strips = (D + 31) / 32;
    if (!mul_ok(B, blocks, strips) || B * blocks * strips >= (int64_t)1 << 23)
        return fail(SSM_ERR_UNSUPPORTED, "batch * ceil(seqlen / 128) * ceil(dim / 32) is not below 2^23");
    if (mode != SSM_GATE_RATE && (in_gate || A))
        return fail(SSM_ERR_BAD_SHAPE, "in_gate and A are for SSM_GATE_RATE only");
    if (mode == SSM_GATE_DECAY && gate_bias) return fail(SSM_ERR_BAD_SHAPE, "SSM_GATE_DECAY takes no gate_bias");
    // (an empty in_gate has no address)
    if (B > 0 && L > 0 && in_bias && !in_gate) return fail(SSM_ERR_BAD_SHAPE, "in_bias given without in_gate");
    return SSM_OK;
}

int64_t gated_blocks(int64_t L) { return (L + SSM_GATED_BLOCK - 1) / SSM_GATED_BLOCK; }

}  // namespace

extern "C" {

size_t ssm_gated_scan_workspace_size(const ssm_gated_scan_args_t *a) {
    if (!a || check_gated(a->batch, a->seqlen, a->dim, a->io_dtype, SSM_GATE_DECAY, nullptr, nullptr, nullptr,
                          nullptr) != SSM_OK)
        return (size_t)-1;
    return a->batch > 0 && a->seqlen > 0 ? ssm::gated_scan_workspace_bytes(*a) : 0;
}

ssm_status_t ssm_gated_scan_fwd(const ssm_gated_scan_args_t *a, void *stream) {
    if (!a) return fail(SSM_ERR_NULL_ARG, "args is NULL");
    ssm_status_t s = check_gated(a->batch, a->seqlen, a->dim, a->io_dtype, a->mode, a->in_gate, a->A, a->gate_bias,
                                 a->in_bias);
    if (s != SSM_OK) return s;
    const int64_t B = a->batch, L = a->seqlen, D = a->dim, es = io_bytes(a->io_dtype), n = B * L * D;
    const bool work = B > 0 && L > 0;
    if (work) {
        if (!a->x) return fail(SSM_ERR_NULL_ARG, "x is NULL");
        if (!a->gate) return fail(SSM_ERR_NULL_ARG, "gate is NULL");
        if (!a->y) return fail(SSM_ERR_NULL_ARG, "y is NULL");
        if (a->mode == SSM_GATE_RATE && !a->A) return fail(SSM_ERR_NULL_ARG, "A is NULL");
    }
    const void *io[] = {a->x, a->gate, a->in_gate, a->y};
    const void *f[] = {a->A, a->gate_bias, a->in_bias, a->h0, a->h_final, a->checkpoints};
    if ((s = check_align(io, COUNT(io), es, f, COUNT(f))) != SSM_OK) return s;
    const size_t need = work ? ssm::gated_scan_workspace_bytes(*a) : 0;
    if ((s = check_workspace(a->workspace, a->workspace_bytes, need)) != SSM_OK) return s;
    const Range in[] = {range(a->x, n, es, "x"), range(a->gate, n, es, "gate"), range(a->in_gate, n, es, "in_gate"),
                        range(a->A, D, 4, "A"), range(a->gate_bias, D, 4, "gate_bias"),
                        range(a->in_bias, D, 4, "in_bias"), range(a->reset, B * L, 1, "reset"),
                        range(a->h0, B * D, 4, "h0")};
    const Range out[] = {range(a->y, n, es, "y"), range(a->h_final, B * D, 4, "h_final"),
                         range(a->checkpoints, gated_blocks(L) * B * D, 4, "checkpoints")};
    const Range ws = range(need ? a->workspace : nullptr, (int64_t)need, 1, "workspace");
    if ((s = check_overlaps(in, COUNT(in), out, COUNT(out), ws)) != SSM_OK) return s;
    if (B == 0) return ok();
    hipStream_t st = static_cast<hipStream_t>(stream);
    hipError_t e = hipSuccess;
    if (L > 0)
        e = ssm::launch_gated_scan_fwd(*a, st);
    else if (a->h_final)
        e = ssm::launch_copy_or_zero(a->h_final, a->h0, B * D, st);
    if (e != hipSuccess) return fail(SSM_ERR_HIP, "HIP error: %s", hipGetErrorString(e));
    return ok();
}

size_t ssm_gated_scan_bwd_workspace_size(const ssm_gated_scan_bwd_args_t *a) {
    if (!a || check_gated(a->batch, a->seqlen, a->dim, a->io_dtype, a->mode, nullptr, nullptr, nullptr, nullptr) !=
                  SSM_OK)
        return (size_t)-1;
    return a->batch > 0 && a->seqlen > 0 ? ssm::gated_scan_bwd_workspace_bytes(*a) : 0;
}

ssm_status_t ssm_gated_scan_bwd(const ssm_gated_scan_bwd_args_t *a, void *stream) {
    if (!a) return fail(SSM_ERR_NULL_ARG, "args is NULL");
    ssm_status_t s = check_gated(a->batch, a->seqlen, a->dim, a->io_dtype, a->mode, a->in_gate, a->A, a->gate_bias,
                                 a->in_bias);
    if (s != SSM_OK) return s;
    const int64_t B = a->batch, L = a->seqlen, D = a->dim, es = io_bytes(a->io_dtype), n = B * L * D;
    const bool work = B > 0 && L > 0;
    if (work) {
        const struct { const void *p; const char *name; } req[] = {
            {a->x, "x"}, {a->gate, "gate"}, {a->dy, "dy"}, {a->dx, "dx"}, {a->dgate, "dgate"}};
        for (const auto &r : req)
            if (!r.p) return fail(SSM_ERR_NULL_ARG, "%s is NULL", r.name);
        if (a->mode == SSM_GATE_RATE && !a->A) return fail(SSM_ERR_NULL_ARG, "A is NULL");
        if (a->in_gate && !a->din_gate) return fail(SSM_ERR_NULL_ARG, "din_gate is NULL but in_gate is given");
    }
    if (a->mode == SSM_GATE_RATE && !a->dA) return fail(SSM_ERR_NULL_ARG, "dA is NULL");
    if (a->mode != SSM_GATE_RATE && a->dA) return fail(SSM_ERR_BAD_SHAPE, "dA is for SSM_GATE_RATE only");
    if (a->mode == SSM_GATE_DECAY && a->dgate_bias) return fail(SSM_ERR_BAD_SHAPE, "SSM_GATE_DECAY has no gate_bias");
    // (with B == 0 or L == 0 the (B,L,D) inputs may be absent)
    if (work && !a->in_gate && (a->din_gate || a->din_bias))
        return fail(SSM_ERR_BAD_SHAPE, "din_gate or din_bias given without in_gate");
    if (a->mode != SSM_GATE_RATE && (a->din_gate || a->din_bias))
        return fail(SSM_ERR_BAD_SHAPE, "din_gate and din_bias are for SSM_GATE_RATE only");
    const void *io[] = {a->x, a->gate, a->in_gate, a->dy, a->dx, a->dgate, a->din_gate};
    const void *f[] = {a->A, a->gate_bias, a->in_bias, a->h0, a->dh_final, a->checkpoints, a->dA, a->dgate_bias,
                       a->din_bias, a->dh0};
    if ((s = check_align(io, COUNT(io), es, f, COUNT(f))) != SSM_OK) return s;
    const size_t need = work ? ssm::gated_scan_bwd_workspace_bytes(*a) : 0;
    if ((s = check_workspace(a->workspace, a->workspace_bytes, need)) != SSM_OK) return s;
    const Range in[] = {range(a->x, n, es, "x"), range(a->gate, n, es, "gate"), range(a->in_gate, n, es, "in_gate"),
                        range(a->A, D, 4, "A"), range(a->gate_bias, D, 4, "gate_bias"),
                        range(a->in_bias, D, 4, "in_bias"), range(a->reset, B * L, 1, "reset"),
                        range(a->h0, B * D, 4, "h0"), range(a->dy, n, es, "dy"),
                        range(a->dh_final, B * D, 4, "dh_final"),
                        range(a->checkpoints, gated_blocks(L) * B * D, 4, "checkpoints")};
    const Range out[] = {range(a->dx, n, es, "dx"), range(a->dgate, n, es, "dgate"),
                         range(a->din_gate, n, es, "din_gate"), range(a->dA, D, 4, "dA"),
                         range(a->dgate_bias, D, 4, "dgate_bias"), range(a->din_bias, D, 4, "din_bias"),
                         range(a->dh0, B * D, 4, "dh0")};
    const Range ws = range(need ? a->workspace : nullptr, (int64_t)need, 1, "workspace");
    if ((s = check_overlaps(in, COUNT(in), out, COUNT(out), ws)) != SSM_OK) return s;
    hipStream_t st = static_cast<hipStream_t>(stream);
    hipError_t e = hipSuccess;
    if (work) {
        e = ssm::launch_gated_scan_bwd(*a, st);
    } else {
        float *sums[] = {a->dA, a->dgate_bias, a->din_bias};
        for (float *p : sums)
            if (e == hipSuccess && p) e = ssm::launch_copy_or_zero(p, nullptr, D, st);
        if (e == hipSuccess && a->dh0 && B > 0) e = ssm::launch_copy_or_zero(a->dh0, a->dh_final, B * D, st);
    }
    if (e != hipSuccess) return fail(SSM_ERR_HIP, "HIP error: %s", hipGetErrorString(e));
    return ok();
}

ssm_status_t ssm_gated_scan_step(const ssm_gated_step_args_t *a, void *stream) {
    if (!a) return fail(SSM_ERR_NULL_ARG, "args is NULL");
    ssm_status_t s = check_gated(a->batch, 1, a->dim, a->io_dtype, a->mode, a->in_gate, a->A, a->gate_bias,
                                 a->in_bias);
    if (s != SSM_OK) return s;
    const int64_t B = a->batch, D = a->dim, es = io_bytes(a->io_dtype), n = B * D;
    if (B == 0) return ok();
    const struct { const void *p; const char *name; } req[] = {
        {a->state, "state"}, {a->x, "x"}, {a->gate, "gate"}, {a->y, "y"}};
    for (const auto &r : req)
        if (!r.p) return fail(SSM_ERR_NULL_ARG, "%s is NULL", r.name);
    if (a->mode == SSM_GATE_RATE && !a->A) return fail(SSM_ERR_NULL_ARG, "A is NULL");
    const void *io[] = {a->x, a->gate, a->in_gate, a->y};
    const void *f[] = {a->A, a->gate_bias, a->in_bias, a->state};
    if ((s = check_align(io, COUNT(io), es, f, COUNT(f))) != SSM_OK) return s;
    const Range in[] = {range(a->x, n, es, "x"), range(a->gate, n, es, "gate"), range(a->in_gate, n, es, "in_gate"),
                        range(a->A, D, 4, "A"), range(a->gate_bias, D, 4, "gate_bias"),
                        range(a->in_bias, D, 4, "in_bias"), range(a->reset, B, 1, "reset")};
    const Range out[] = {range(a->state, n, 4, "state"), range(a->y, n, es, "y")};
    if ((s = check_overlaps(in, COUNT(in), out, COUNT(out), range(nullptr, 0, 1, ""))) != SSM_OK) return s;
    const hipError_t e = ssm::launch_gated_step(*a, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return fail(SSM_ERR_HIP, "HIP error: %s", hipGetErrorString(e));
    return ok();
}

static ssm_status_t check_norm(int64_t rows, int64_t D, float eps) {
    if (rows < 0) return fail(SSM_ERR_BAD_SHAPE, "negative rows (%lld)", (long long)rows);
    if (D < 1) return fail(SSM_ERR_BAD_SHAPE, "dim must be >= 1 (got %lld)", (long long)D);
    if (D > kMaxWidth) return fail(SSM_ERR_UNSUPPORTED, "dim %lld exceeds 2^20", (long long)D);
    if (!mul_ok(rows, 4 * D)) return fail(SSM_ERR_BAD_SHAPE, "sizes overflow");
    if (!(eps > 0.0f) || !(eps < 1e30f)) return fail(SSM_ERR_BAD_SHAPE, "eps must be > 0");
    return SSM_OK;
}

ssm_status_t ssm_add_rmsnorm_fwd(const ssm_add_norm_args_t *a, void *stream) {
    if (!a) return fail(SSM_ERR_NULL_ARG, "args is NULL");
    if (!io_ok(a->io_dtype) || !io_ok(a->res_dtype))
        return fail(SSM_ERR_BAD_DTYPE, "io_dtype (%d) and res_dtype (%d) must be SSM_F32 or SSM_BF16", a->io_dtype,
                    a->res_dtype);
    ssm_status_t s = check_norm(a->rows, a->dim, a->eps);
    if (s != SSM_OK) return s;
    if (a->rows == 0) return ok();
    if (!a->x) return fail(SSM_ERR_NULL_ARG, "x is NULL");
    if (!a->w) return fail(SSM_ERR_NULL_ARG, "w is NULL");
    if (!a->y) return fail(SSM_ERR_NULL_ARG, "y is NULL");
    const int64_t D = a->dim, n = a->rows * D, es = io_bytes(a->io_dtype), rs = io_bytes(a->res_dtype);
    const void *io[] = {a->x, a->y}, *res[] = {a->residual, a->res_out}, *f[] = {a->scale, a->post_w, a->w};
    if ((s = check_align(io, COUNT(io), es, f, COUNT(f))) != SSM_OK) return s;
    if ((s = check_align(res, COUNT(res), rs, nullptr, 0)) != SSM_OK) return s;
    const Range in[] = {range(a->x, n, es, "x"), range(a->residual, n, rs, "residual"),
                        range(a->scale, D, 4, "scale"), range(a->post_w, D, 4, "post_w"), range(a->w, D, 4, "w")};
    const Range out[] = {range(a->res_out, n, rs, "res_out"), range(a->y, n, es, "y")};
    s = check_overlaps(in, COUNT(in), out, COUNT(out), range(nullptr, 0, 1, ""), SameOk{a->res_out, a->residual});
    if (s != SSM_OK) return s;
    const hipError_t e = ssm::launch_add_norm_fwd(*a, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return fail(SSM_ERR_HIP, "HIP error: %s", hipGetErrorString(e));
    return ok();
}

size_t ssm_add_rmsnorm_bwd_workspace_size(const ssm_add_norm_bwd_args_t *a) {
    if (!a || !io_ok(a->io_dtype) || !io_ok(a->res_dtype) || check_norm(a->rows, a->dim, 1.0f) != SSM_OK)
        return (size_t)-1;
    return a->rows > 0 ? ssm::add_norm_bwd_workspace_bytes(*a) : 0;
}

ssm_status_t ssm_add_rmsnorm_bwd(const ssm_add_norm_bwd_args_t *a, void *stream) {
    if (!a) return fail(SSM_ERR_NULL_ARG, "args is NULL");
    if (!io_ok(a->io_dtype) || !io_ok(a->res_dtype))
        return fail(SSM_ERR_BAD_DTYPE, "io_dtype (%d) and res_dtype (%d) must be SSM_F32 or SSM_BF16", a->io_dtype,
                    a->res_dtype);
    ssm_status_t s = check_norm(a->rows, a->dim, a->eps);
    if (s != SSM_OK) return s;
    const bool work = a->rows > 0;
    if (work) {
        const struct { const void *p; const char *name; } req[] = {
            {a->x, "x"}, {a->w, "w"}, {a->dy, "dy"}, {a->dx, "dx"}};
        for (const auto &r : req)
            if (!r.p) return fail(SSM_ERR_NULL_ARG, "%s is NULL", r.name);
        if (a->dresidual && !a->residual) return fail(SSM_ERR_BAD_SHAPE, "dresidual given without residual");
    }
    if (!a->dw) return fail(SSM_ERR_NULL_ARG, "dw is NULL");
    if (a->dscale && !a->scale) return fail(SSM_ERR_BAD_SHAPE, "dscale given without scale");
    if (a->dpost_w && !a->post_w) return fail(SSM_ERR_BAD_SHAPE, "dpost_w given without post_w");
    const int64_t D = a->dim, n = a->rows * D, es = io_bytes(a->io_dtype), rs = io_bytes(a->res_dtype);
    const void *io[] = {a->x, a->dy, a->dx}, *res[] = {a->residual, a->dres_out, a->dresidual};
    const void *f[] = {a->scale, a->post_w, a->w, a->dw, a->dscale, a->dpost_w};
    if ((s = check_align(io, COUNT(io), es, f, COUNT(f))) != SSM_OK) return s;
    if ((s = check_align(res, COUNT(res), rs, nullptr, 0)) != SSM_OK) return s;
    const size_t need = work ? ssm::add_norm_bwd_workspace_bytes(*a) : 0;
    if ((s = check_workspace(a->workspace, a->workspace_bytes, need)) != SSM_OK) return s;
    const Range in[] = {range(a->x, n, es, "x"), range(a->residual, n, rs, "residual"),
                        range(a->scale, D, 4, "scale"), range(a->post_w, D, 4, "post_w"), range(a->w, D, 4, "w"),
                        range(a->dy, n, es, "dy"), range(a->dres_out, n, rs, "dres_out")};
    const Range out[] = {range(a->dx, n, es, "dx"), range(a->dresidual, n, rs, "dresidual"),
                         range(a->dw, D, 4, "dw"), range(a->dscale, D, 4, "dscale"),
                         range(a->dpost_w, D, 4, "dpost_w")};
    const Range ws = range(need ? a->workspace : nullptr, (int64_t)need, 1, "workspace");
    s = check_overlaps(in, COUNT(in), out, COUNT(out), ws, SameOk{a->dresidual, a->dres_out});
    if (s != SSM_OK) return s;
    hipStream_t st = static_cast<hipStream_t>(stream);
    hipError_t e = hipSuccess;
    if (work) {
        e = ssm::launch_add_norm_bwd(*a, st);
    } else {
        float *sums[] = {a->dw, a->dscale, a->dpost_w};
        for (float *p : sums)
            if (e == hipSuccess && p) e = ssm::launch_copy_or_zero(p, nullptr, D, st);
    }
    if (e != hipSuccess) return fail(SSM_ERR_HIP, "HIP error: %s", hipGetErrorString(e));
    return ok();
}

static ssm_status_t check_gated_norm(int64_t rows, int64_t D, int64_t G, int32_t io, int32_t gate_first, float eps) {
    if (!io_ok(io)) return fail(SSM_ERR_BAD_DTYPE, "io_dtype %d is not SSM_F32 or SSM_BF16", io);
    const ssm_status_t s = check_norm(rows, D, eps);
    if (s != SSM_OK) return s;
    if (G < 1 || D % G != 0)
        return fail(SSM_ERR_BAD_SHAPE, "groups (%lld) must divide dim (%lld)", (long long)G, (long long)D);
    if (gate_first != 0 && gate_first != 1) return fail(SSM_ERR_UNSUPPORTED, "gate_first must be 0 or 1");
    return SSM_OK;
}

ssm_status_t ssm_gated_rmsnorm_fwd(const ssm_gated_norm_args_t *a, void *stream) {
    if (!a) return fail(SSM_ERR_NULL_ARG, "args is NULL");
    ssm_status_t s = check_gated_norm(a->rows, a->dim, a->groups, a->io_dtype, a->gate_first, a->eps);
    if (s != SSM_OK) return s;
    if (a->rows == 0) return ok();
    if (!a->x) return fail(SSM_ERR_NULL_ARG, "x is NULL");
    if (!a->z) return fail(SSM_ERR_NULL_ARG, "z is NULL");
    if (!a->w) return fail(SSM_ERR_NULL_ARG, "w is NULL");
    if (!a->y) return fail(SSM_ERR_NULL_ARG, "y is NULL");
    const int64_t D = a->dim, n = a->rows * D, es = io_bytes(a->io_dtype);
    const void *io[] = {a->x, a->z, a->y}, *f[] = {a->w};
    if ((s = check_align(io, COUNT(io), es, f, COUNT(f))) != SSM_OK) return s;
    const Range in[] = {range(a->x, n, es, "x"), range(a->z, n, es, "z"), range(a->w, D, 4, "w")};
    const Range out[] = {range(a->y, n, es, "y")};
    s = check_overlaps(in, COUNT(in), out, COUNT(out), range(nullptr, 0, 1, ""), SameOk{a->y, a->x}, SameOk{a->y, a->z});
    if (s != SSM_OK) return s;
    const hipError_t e = ssm::launch_gated_norm_fwd(*a, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return fail(SSM_ERR_HIP, "HIP error: %s", hipGetErrorString(e));
    return ok();
}

size_t ssm_gated_rmsnorm_bwd_workspace_size(const ssm_gated_norm_bwd_args_t *a) {
    if (!a || check_gated_norm(a->rows, a->dim, a->groups, a->io_dtype, 0, 1.0f) != SSM_OK) return (size_t)-1;
    return a->rows > 0 ? ssm::gated_norm_bwd_workspace_bytes(*a) : 0;
}

ssm_status_t ssm_gated_rmsnorm_bwd(const ssm_gated_norm_bwd_args_t *a, void *stream) {
    if (!a) return fail(SSM_ERR_NULL_ARG, "args is NULL");
    ssm_status_t s = check_gated_norm(a->rows, a->dim, a->groups, a->io_dtype, a->gate_first, a->eps);
    if (s != SSM_OK) return s;
    const bool work = a->rows > 0;
    if (work) {
        const struct { const void *p; const char *name; } req[] = {
            {a->x, "x"}, {a->z, "z"}, {a->w, "w"}, {a->dy, "dy"}, {a->dx, "dx"}, {a->dz, "dz"}};
        for (const auto &r : req)
            if (!r.p) return fail(SSM_ERR_NULL_ARG, "%s is NULL", r.name);
    }
    if (!a->dw) return fail(SSM_ERR_NULL_ARG, "dw is NULL");
    const int64_t D = a->dim, n = a->rows * D, es = io_bytes(a->io_dtype);
    const void *io[] = {a->x, a->z, a->dy, a->dx, a->dz}, *f[] = {a->w, a->dw};
    if ((s = check_align(io, COUNT(io), es, f, COUNT(f))) != SSM_OK) return s;
    const size_t need = work ? ssm::gated_norm_bwd_workspace_bytes(*a) : 0;
    if ((s = check_workspace(a->workspace, a->workspace_bytes, need)) != SSM_OK) return s;
    const Range in[] = {range(a->x, n, es, "x"), range(a->z, n, es, "z"), range(a->w, D, 4, "w"),
                        range(a->dy, n, es, "dy")};
    const Range out[] = {range(a->dx, n, es, "dx"), range(a->dz, n, es, "dz"), range(a->dw, D, 4, "dw")};
    const Range ws = range(need ? a->workspace : nullptr, (int64_t)need, 1, "workspace");
    if ((s = check_overlaps(in, COUNT(in), out, COUNT(out), ws)) != SSM_OK) return s;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const hipError_t e = work ? ssm::launch_gated_norm_bwd(*a, st) : ssm::launch_copy_or_zero(a->dw, nullptr, D, st);
    if (e != hipSuccess) return fail(SSM_ERR_HIP, "HIP error: %s", hipGetErrorString(e));
    return ok();
}

}  // extern "C"

// --------------------------------------------------------------------- gated delta rule
namespace {

struct DeltaSizes {
    int64_t B, L, Hk, H, K, V;
    int32_t io, l2norm;
    float scale;
};

ssm_status_t check_delta(const DeltaSizes &z) {
    if (!io_ok(z.io)) return fail(SSM_ERR_BAD_DTYPE, "io_dtype %d is not SSM_F32 or SSM_BF16", z.io);
    if (z.B < 0 || z.L < 0)
        return fail(SSM_ERR_BAD_SHAPE, "negative batch (%lld) or seqlen (%lld)", (long long)z.B, (long long)z.L);
    if (z.Hk < 1 || z.H < 1 || z.K < 1 || z.V < 1)
        return fail(SSM_ERR_BAD_SHAPE, "kheads, heads, kdim and vdim must be >= 1");
    if (z.H % z.Hk != 0)
        return fail(SSM_ERR_BAD_SHAPE, "kheads (%lld) must divide heads (%lld)", (long long)z.Hk, (long long)z.H);
    if (z.K > SSM_DELTA_MAX_KDIM || z.K % 8 != 0)
        return fail(SSM_ERR_UNSUPPORTED, "kdim %lld is not a multiple of 8 up to %d", (long long)z.K,
                    SSM_DELTA_MAX_KDIM);
    if (z.V > SSM_DELTA_MAX_VDIM || z.V % 8 != 0)
        return fail(SSM_ERR_UNSUPPORTED, "vdim %lld is not a multiple of 8 up to %d", (long long)z.V,
                    SSM_DELTA_MAX_VDIM);
    if (z.H > 65535 || z.B > 65535)
        return fail(SSM_ERR_UNSUPPORTED, "heads (%lld) and batch (%lld) go up to 65535", (long long)z.H, (long long)z.B);
    if (z.L >= (int64_t)1 << 30) return fail(SSM_ERR_UNSUPPORTED, "seqlen %lld is not below 2^30", (long long)z.L);
    if (z.H * z.V >= (int64_t)1 << 24 || z.Hk * z.K >= (int64_t)1 << 24)
        return fail(SSM_ERR_UNSUPPORTED, "heads * vdim and kheads * kdim have to be below 2^24");
    // 512 threads for each 16 channels of a head, fewer than 2^32 threads a launch
    if ((z.B * z.H + 8) * ((z.V + 15) / 16) >= (int64_t)1 << 23)
        return fail(SSM_ERR_UNSUPPORTED, "batch * heads * ceil(vdim / 16) is not below 2^23");
    if (z.l2norm != 0 && z.l2norm != 1) return fail(SSM_ERR_UNSUPPORTED, "l2norm must be 0 or 1");
    if (!(z.scale - z.scale == 0.0f)) return fail(SSM_ERR_BAD_SHAPE, "scale must be finite");
    // the largest arrays: checkpoints and the backward's workspace, below 2^60 bytes
    const int64_t chunks = z.L / SSM_DELTA_CHUNK + 1;
    if (!mul_ok(z.B * z.H, chunks, ((int64_t)1 << 21))) return fail(SSM_ERR_BAD_SHAPE, "sizes overflow");
    return SSM_OK;
}

int64_t delta_chunks(int64_t L) { return (L + SSM_DELTA_CHUNK - 1) / SSM_DELTA_CHUNK; }

// The tensor of one of q, k, v: B x L steps of `width` consecutive elements.
struct Steps {
    const void *p;
    int64_t token, batch, width, es;
    const char *name;
    bool wide;  // read 16 bytes at a time
};

// Fills in the strides of a dense tensor and checks those given; `out`: what the tensor spans.
ssm_status_t check_steps(Steps s, int64_t B, int64_t L, Range &out) {
    if (s.token == 0) {
        s.token = s.width;
        s.batch = L * s.width;
    }
    // (a lane's way to its step of a chunk, up to 63 steps of 4 bytes an element, is a number of 32 bits)
    if (s.token < 0 || s.batch < 0 || s.token >= (int64_t)1 << 24 || s.batch > (int64_t)1 << 40)
        return fail(SSM_ERR_BAD_SHAPE, "%s has a stride that is negative, 2^24 or more (steps) or above 2^40 (rows)",
                    s.name);
    if (!mul_ok(L, s.token, 16) || !mul_ok(B, s.batch, 16)) return fail(SSM_ERR_BAD_SHAPE, "sizes overflow");
    if (s.wide && (!aligned(s.p, 16) || (L > 1 && s.token * s.es % 16 != 0) || (B > 1 && s.batch * s.es % 16 != 0)))
        return fail(SSM_ERR_ALIGN, "%s does not lie at 16-byte boundaries", s.name);
    out = range(s.p, B > 0 && L > 0 ? (B - 1) * s.batch + (L - 1) * s.token + s.width : 0, s.es, s.name);
    return SSM_OK;
}

template <typename A>
DeltaSizes delta_sizes(const A &a, int64_t L) {
    return {a.batch, L, a.kheads, a.heads, a.kdim, a.vdim, a.io_dtype, a.l2norm, a.scale};
}

struct Named {
    const void *p;
    const char *name;
};

ssm_status_t check_required(const Named *req, int n) {
    for (int i = 0; i < n; ++i)
        if (!req[i].p) return fail(SSM_ERR_NULL_ARG, "%s is NULL", req[i].name);
    return SSM_OK;
}

}  // namespace

extern "C" {

size_t ssm_gated_delta_workspace_size(const ssm_gated_delta_args_t *a) {
    if (!a) return (size_t)-1;
    DeltaSizes z = delta_sizes(*a, a->seqlen);
    z.scale = 1.0f;
    z.l2norm = 0;
    if (check_delta(z) != SSM_OK) return (size_t)-1;
    return a->batch > 0 && a->seqlen > 0 ? ssm::gated_delta_workspace_bytes(*a) : 0;
}

ssm_status_t ssm_gated_delta_fwd(const ssm_gated_delta_args_t *a, void *stream) {
    if (!a) return fail(SSM_ERR_NULL_ARG, "args is NULL");
    ssm_status_t s = check_delta(delta_sizes(*a, a->seqlen));
    if (s != SSM_OK) return s;
    const int64_t B = a->batch, L = a->seqlen, H = a->heads, K = a->kdim, V = a->vdim, es = io_bytes(a->io_dtype);
    const bool work = B > 0 && L > 0;
    if (work) {
        const Named req[] = {{a->q, "q"}, {a->k, "k"}, {a->v, "v"}, {a->g, "g"}, {a->beta, "beta"}, {a->o, "o"}};
        if ((s = check_required(req, COUNT(req))) != SSM_OK) return s;
    }
    const void *io[] = {a->q, a->k, a->v, a->beta, a->o};
    const void *f[] = {a->g, a->h0, a->h_final, a->checkpoints};
    if ((s = check_align(io, COUNT(io), es, f, COUNT(f))) != SSM_OK) return s;
    if (!aligned(a->checkpoints, 16)) return fail(SSM_ERR_ALIGN, "checkpoints are not 16-byte aligned");
    Range rq, rk, rv;
    if ((s = check_steps({a->q, a->q_token, a->q_batch, a->kheads * K, es, "q", true}, B, L, rq)) != SSM_OK ||
        (s = check_steps({a->k, a->k_token, a->k_batch, a->kheads * K, es, "k", true}, B, L, rk)) != SSM_OK ||
        (s = check_steps({a->v, a->v_token, a->v_batch, H * V, es, "v", false}, B, L, rv)) != SSM_OK)
        return s;
    const size_t need = work ? ssm::gated_delta_workspace_bytes(*a) : 0;
    if ((s = check_workspace(a->workspace, a->workspace_bytes, need)) != SSM_OK) return s;
    const int64_t state = B * H * K * V;
    const Range in[] = {rq, rk, rv, range(a->g, B * L * H, 4, "g"), range(a->beta, B * L * H, es, "beta"),
                        range(a->reset, B * L, 1, "reset"), range(a->h0, state, 4, "h0")};
    const Range out[] = {range(a->o, B * L * H * V, es, "o"), range(a->h_final, state, 4, "h_final"),
                         range(a->checkpoints, delta_chunks(L) * B * H * (K + SSM_DELTA_CHUNK) * V, 4, "checkpoints")};
    const Range ws = range(need ? a->workspace : nullptr, (int64_t)need, 1, "workspace");
    if ((s = check_overlaps(in, COUNT(in), out, COUNT(out), ws)) != SSM_OK) return s;
    if (B == 0) return ok();
    hipStream_t st = static_cast<hipStream_t>(stream);
    hipError_t e = hipSuccess;
    if (L > 0)
        e = ssm::launch_gated_delta_fwd(*a, st);
    else if (a->h_final)
        e = ssm::launch_copy_or_zero(a->h_final, a->h0, state, st);
    if (e != hipSuccess) return fail(SSM_ERR_HIP, "HIP error: %s", hipGetErrorString(e));
    return ok();
}

size_t ssm_gated_delta_bwd_workspace_size(const ssm_gated_delta_bwd_args_t *a) {
    if (!a) return (size_t)-1;
    DeltaSizes z = delta_sizes(*a, a->seqlen);
    z.scale = 1.0f;
    z.l2norm = 0;
    if (check_delta(z) != SSM_OK) return (size_t)-1;
    return a->batch > 0 && a->seqlen > 0 ? ssm::gated_delta_bwd_workspace_bytes(*a) : 0;
}

ssm_status_t ssm_gated_delta_bwd(const ssm_gated_delta_bwd_args_t *a, void *stream) {
    if (!a) return fail(SSM_ERR_NULL_ARG, "args is NULL");
    ssm_status_t s = check_delta(delta_sizes(*a, a->seqlen));
    if (s != SSM_OK) return s;
    const int64_t B = a->batch, L = a->seqlen, H = a->heads, K = a->kdim, V = a->vdim, es = io_bytes(a->io_dtype);
    const bool work = B > 0 && L > 0;
    if (work) {
        const Named req[] = {{a->q, "q"}, {a->k, "k"}, {a->v, "v"}, {a->g, "g"}, {a->beta, "beta"}, {a->dout, "dout"},
                             {a->dq, "dq"}, {a->dk, "dk"}, {a->dv, "dv"}, {a->dg, "dg"}, {a->dbeta, "dbeta"}};
        if ((s = check_required(req, COUNT(req))) != SSM_OK) return s;
    }
    const void *io[] = {a->q, a->k, a->v, a->beta, a->dout, a->dq, a->dk, a->dv, a->dbeta};
    const void *f[] = {a->g, a->h0, a->dh_final, a->checkpoints, a->dg, a->dh0};
    if ((s = check_align(io, COUNT(io), es, f, COUNT(f))) != SSM_OK) return s;
    if (!aligned(a->checkpoints, 16)) return fail(SSM_ERR_ALIGN, "checkpoints are not 16-byte aligned");
    Range rq, rk, rv;
    if ((s = check_steps({a->q, a->q_token, a->q_batch, a->kheads * K, es, "q", true}, B, L, rq)) != SSM_OK ||
        (s = check_steps({a->k, a->k_token, a->k_batch, a->kheads * K, es, "k", true}, B, L, rk)) != SSM_OK ||
        (s = check_steps({a->v, a->v_token, a->v_batch, H * V, es, "v", false}, B, L, rv)) != SSM_OK)
        return s;
    const size_t need = work ? ssm::gated_delta_bwd_workspace_bytes(*a) : 0;
    if ((s = check_workspace(a->workspace, a->workspace_bytes, need)) != SSM_OK) return s;
    const int64_t state = B * H * K * V, steps = B * L;
    const Range in[] = {rq, rk, rv, range(a->g, steps * H, 4, "g"), range(a->beta, steps * H, es, "beta"),
                        range(a->reset, steps, 1, "reset"), range(a->h0, state, 4, "h0"),
                        range(a->dout, steps * H * V, es, "dout"), range(a->dh_final, state, 4, "dh_final"),
                        range(a->checkpoints, delta_chunks(L) * B * H * (K + SSM_DELTA_CHUNK) * V, 4, "checkpoints")};
    const Range out[] = {range(a->dq, steps * a->kheads * K, es, "dq"), range(a->dk, steps * a->kheads * K, es, "dk"),
                         range(a->dv, steps * H * V, es, "dv"), range(a->dg, steps * H, 4, "dg"),
                         range(a->dbeta, steps * H, es, "dbeta"), range(a->dh0, state, 4, "dh0")};
    const Range ws = range(need ? a->workspace : nullptr, (int64_t)need, 1, "workspace");
    if ((s = check_overlaps(in, COUNT(in), out, COUNT(out), ws)) != SSM_OK) return s;
    if (B == 0) return ok();
    hipStream_t st = static_cast<hipStream_t>(stream);
    hipError_t e = hipSuccess;
    if (L > 0)
        e = ssm::launch_gated_delta_bwd(*a, st);
    else if (a->dh0)
        e = ssm::launch_copy_or_zero(a->dh0, a->dh_final, state, st);
    if (e != hipSuccess) return fail(SSM_ERR_HIP, "HIP error: %s", hipGetErrorString(e));
    return ok();
}

ssm_status_t ssm_gated_delta_step(const ssm_gated_delta_step_args_t *a, void *stream) {
    if (!a) return fail(SSM_ERR_NULL_ARG, "args is NULL");
    ssm_status_t s = check_delta(delta_sizes(*a, 1));
    if (s != SSM_OK) return s;
    const int64_t B = a->batch, Hk = a->kheads, H = a->heads, K = a->kdim, V = a->vdim, es = io_bytes(a->io_dtype);
    if (B == 0) return ok();
    const Named req[] = {{a->state, "state"}, {a->q, "q"}, {a->k, "k"}, {a->v, "v"},
                         {a->g, "g"}, {a->beta, "beta"}, {a->o, "o"}};
    if ((s = check_required(req, COUNT(req))) != SSM_OK) return s;
    const void *io[] = {a->q, a->k, a->v, a->beta, a->o};
    const void *f[] = {a->g};
    if ((s = check_align(io, COUNT(io), es, f, COUNT(f))) != SSM_OK) return s;
    if (!aligned(a->state, 16)) return fail(SSM_ERR_ALIGN, "state is not 16-byte aligned");
    Range rq, rk, rv;  // each batch row is a step here
    if ((s = check_steps({a->q, a->q_batch, 0, Hk * K, es, "q", false}, 1, B, rq)) != SSM_OK ||
        (s = check_steps({a->k, a->k_batch, 0, Hk * K, es, "k", false}, 1, B, rk)) != SSM_OK ||
        (s = check_steps({a->v, a->v_batch, 0, H * V, es, "v", false}, 1, B, rv)) != SSM_OK)
        return s;
    const Range in[] = {rq, rk, rv, range(a->g, B * H, 4, "g"), range(a->beta, B * H, es, "beta"),
                        range(a->reset, B, 1, "reset")};
    const Range out[] = {range(a->state, B * H * K * V, 4, "state"), range(a->o, B * H * V, es, "o")};
    if ((s = check_overlaps(in, COUNT(in), out, COUNT(out), range(nullptr, 0, 1, ""))) != SSM_OK) return s;
    const hipError_t e = ssm::launch_gated_delta_step(*a, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return fail(SSM_ERR_HIP, "HIP error: %s", hipGetErrorString(e));
    return ok();
}

// ------------------------------------------------------------------------------ e4m3
static ssm_status_t check_fp8_width(int64_t rows, int64_t D) {
    if (rows < 0) return fail(SSM_ERR_BAD_SHAPE, "negative rows (%lld)", (long long)rows);
    if (D < 1) return fail(SSM_ERR_BAD_SHAPE, "dim must be >= 1 (got %lld)", (long long)D);
    if (D > kMaxWidth || D % 16 != 0)
        return fail(SSM_ERR_UNSUPPORTED, "dim %lld is not a multiple of 16 up to 2^20", (long long)D);
    // 16 blocks a workgroup of 256 threads, fewer than 2^32 threads a launch
    const int64_t blocks = (D + SSM_FP8_BLOCK - 1) / SSM_FP8_BLOCK;
    if (rows >= ((int64_t)1 << 28) / blocks)
        return fail(SSM_ERR_UNSUPPORTED, "rows * ceil(dim / 128) is not below 2^28");
    return SSM_OK;
}

ssm_status_t ssm_quantize_fp8(const ssm_quantize_fp8_args_t *a, void *stream) {
    if (!a) return fail(SSM_ERR_NULL_ARG, "args is NULL");
    if (!io_ok(a->io_dtype)) return fail(SSM_ERR_BAD_DTYPE, "io_dtype %d is not SSM_F32 or SSM_BF16", a->io_dtype);
    ssm_status_t s = check_fp8_width(a->rows, a->dim);
    if (s != SSM_OK) return s;
    if (a->block_rows != 1 && a->block_rows != SSM_FP8_BLOCK)
        return fail(SSM_ERR_UNSUPPORTED, "block_rows must be 1 or %d", SSM_FP8_BLOCK);
    if (a->rows == 0) return ok();
    const Named req[] = {{a->x, "x"}, {a->q, "q"}, {a->scales, "scales"}};
    if ((s = check_required(req, COUNT(req))) != SSM_OK) return s;
    const int64_t n = a->rows * a->dim, es = io_bytes(a->io_dtype);
    const void *io[] = {a->x}, *f[] = {a->scales};
    if ((s = check_align(io, 1, es, f, 1)) != SSM_OK) return s;
    if (!aligned(a->q, 16)) return fail(SSM_ERR_ALIGN, "q is not 16-byte aligned");
    const Range in[] = {range(a->x, n, es, "x")};
    const int64_t blocks = (a->rows + a->block_rows - 1) / a->block_rows * ((a->dim + 127) / 128);
    const Range out[] = {range(a->q, n, 1, "q"), range(a->scales, blocks, 4, "scales")};
    if ((s = check_overlaps(in, 1, out, COUNT(out), range(nullptr, 0, 1, ""))) != SSM_OK) return s;
    const hipError_t e = ssm::launch_quantize_fp8(*a, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return fail(SSM_ERR_HIP, "HIP error: %s", hipGetErrorString(e));
    return ok();
}

ssm_status_t ssm_add_rmsnorm_fp8(const ssm_add_norm_fp8_args_t *p, void *stream) {
    if (!p) return fail(SSM_ERR_NULL_ARG, "args is NULL");
    const ssm_add_norm_args_t *a = &p->norm;
    if (!io_ok(a->io_dtype) || !io_ok(a->res_dtype))
        return fail(SSM_ERR_BAD_DTYPE, "io_dtype (%d) and res_dtype (%d) must be SSM_F32 or SSM_BF16", a->io_dtype,
                    a->res_dtype);
    ssm_status_t s = check_norm(a->rows, a->dim, a->eps);
    if (s == SSM_OK) s = check_fp8_width(a->rows, a->dim);
    if (s != SSM_OK) return s;
    if (a->y) return fail(SSM_ERR_BAD_SHAPE, "y must be NULL: the norm's output is q");
    if (a->rows == 0) return ok();
    const Named req[] = {{a->x, "x"}, {a->w, "w"}, {p->q, "q"}, {p->scales, "scales"}};
    if ((s = check_required(req, COUNT(req))) != SSM_OK) return s;
    const int64_t D = a->dim, n = a->rows * D, es = io_bytes(a->io_dtype), rs = io_bytes(a->res_dtype);
    const void *io[] = {a->x}, *res[] = {a->residual, a->res_out}, *f[] = {a->scale, a->post_w, a->w, p->scales};
    if ((s = check_align(io, COUNT(io), es, f, COUNT(f))) != SSM_OK) return s;
    if ((s = check_align(res, COUNT(res), rs, nullptr, 0)) != SSM_OK) return s;
    if (!aligned(p->q, 16)) return fail(SSM_ERR_ALIGN, "q is not 16-byte aligned");
    const Range in[] = {range(a->x, n, es, "x"), range(a->residual, n, rs, "residual"),
                        range(a->scale, D, 4, "scale"), range(a->post_w, D, 4, "post_w"), range(a->w, D, 4, "w")};
    const Range out[] = {range(a->res_out, n, rs, "res_out"), range(p->q, n, 1, "q"),
                         range(p->scales, a->rows * ((D + 127) / 128), 4, "scales")};
    s = check_overlaps(in, COUNT(in), out, COUNT(out), range(nullptr, 0, 1, ""), SameOk{a->res_out, a->residual});
    if (s != SSM_OK) return s;
    const hipError_t e = ssm::launch_add_norm_fp8(*p, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return fail(SSM_ERR_HIP, "HIP error: %s", hipGetErrorString(e));
    return ok();
}

ssm_status_t ssm_matmul_fp8(const ssm_matmul_fp8_args_t *a, void *stream) {
    if (!a) return fail(SSM_ERR_NULL_ARG, "args is NULL");
    if (!io_ok(a->out_dtype)) return fail(SSM_ERR_BAD_DTYPE, "out_dtype %d is not SSM_F32 or SSM_BF16", a->out_dtype);
    const int64_t M = a->m, N = a->n, K = a->k;
    if (M < 0 || N < 1 || K < 1)
        return fail(SSM_ERR_BAD_SHAPE, "sizes m %lld, n %lld, k %lld", (long long)M, (long long)N, (long long)K);
    if (K % 16 != 0 || K > kMaxWidth)
        return fail(SSM_ERR_UNSUPPORTED, "k %lld is not a multiple of 16 up to 2^20", (long long)K);
    // a workgroup of 512 threads per 256 x 256 of y, fewer than 2^32 threads a launch
    if (N >= (int64_t)1 << 24 || M >= (int64_t)1 << 31 || !mul_ok(M + 256, N + 256) ||
        (M + 255) / 256 * ((N + 255) / 256) >= (int64_t)1 << 22)
        return fail(SSM_ERR_UNSUPPORTED, "n is not below 2^24, or ceil(m / 256) * ceil(n / 256) not below 2^22");
    if (M == 0) return ok();
    ssm_status_t s;
    const Named req[] = {{a->xq, "xq"}, {a->x_scales, "x_scales"}, {a->wq, "wq"}, {a->w_scales, "w_scales"}, {a->y, "y"}};
    if ((s = check_required(req, COUNT(req))) != SSM_OK) return s;
    const int64_t es = io_bytes(a->out_dtype), blocks = (K + 127) / 128;
    const void *io[] = {a->y}, *f[] = {a->x_scales, a->w_scales};
    if ((s = check_align(io, 1, es, f, COUNT(f))) != SSM_OK) return s;
    if (!aligned(a->xq, 16) || !aligned(a->wq, 16)) return fail(SSM_ERR_ALIGN, "xq or wq is not 16-byte aligned");
    const Range in[] = {range(a->xq, M * K, 1, "xq"), range(a->x_scales, M * blocks, 4, "x_scales"),
                        range(a->wq, N * K, 1, "wq"), range(a->w_scales, (N + 127) / 128 * blocks, 4, "w_scales")};
    const Range out[] = {range(a->y, M * N, es, "y")};
    if ((s = check_overlaps(in, COUNT(in), out, 1, range(nullptr, 0, 1, ""))) != SSM_OK) return s;
    const hipError_t e = ssm::launch_matmul_fp8(*a, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return fail(SSM_ERR_HIP, "HIP error: %s", hipGetErrorString(e));
    return ok();
}

}  // extern "C"
