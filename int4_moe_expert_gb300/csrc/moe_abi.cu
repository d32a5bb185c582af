// C-ABI layer of the int4 routed-MoE FFN library: argument validation,
// workspace ownership, error reporting.  All compute is in moe_kernels.cu.
#include <cuda_runtime.h>
#include <math.h>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>
#include <exception>
#include <new>
#include <numeric>
#include <vector>

#include "moe_internal.h"

struct moe_handle {
    moe::Params p;
    void *ws_base;
    size_t ws_bytes;
    void *tables;        // device copies of the per-expert pointer arrays
    void *tmaps;         // tcgen05 path: tensor maps of the weights and activations (or NULL)
    float *x_stage;      // device staging for moe_forward_host
    float *y_stage;
    int device;
    cudaEvent_t *prof_ev;   // [prof_max][kStages + 1]
    int prof_max;           // calls to record
    int prof_n;             // calls recorded so far
    int last_T;             // tokens of the last call, and whether it built buckets (checks)
    bool last_buckets;
};

namespace {

thread_local char g_err[512] = "";

moe_status fail(moe_status s, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof(g_err), fmt, ap);
    va_end(ap);
    return s;
}

moe_status cuda_fail(cudaError_t e, const char *what) {
    const moe_status s = (e == cudaErrorMemoryAllocation) ? MOE_ERR_NOMEM : MOE_ERR_CUDA;
    return fail(s, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

bool aligned16(const void *ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }

constexpr int kMaxTokens = 1 << 16;

moe_status check_config(const moe_config *c, int32_t max_tokens, moe::Dims *d) {
    if (!c) return fail(MOE_ERR_INVALID, "config is NULL");
    if (c->hidden < 32 || c->hidden > 16384 || c->hidden % 32)
        return fail(MOE_ERR_UNSUPPORTED, "hidden=%d: need a multiple of 32 in [32, 16384]", c->hidden);
    if (c->n_experts < 1 || c->n_experts > 1024)
        return fail(MOE_ERR_UNSUPPORTED, "n_experts=%d: need 1..1024", c->n_experts);
    if (c->top_k < 1 || c->top_k > c->n_experts || c->top_k > 32)
        return fail(MOE_ERR_INVALID, "top_k=%d: need 1..min(n_experts, 32)", c->top_k);
    if (c->moe_inter < 32 || c->moe_inter > 16384 || c->moe_inter % 32)
        return fail(MOE_ERR_UNSUPPORTED, "moe_inter=%d: need a multiple of 32 in [32, 16384]", c->moe_inter);
    if (c->n_shared != 0 && c->n_shared != 1)
        return fail(MOE_ERR_UNSUPPORTED, "n_shared=%d: need 0 or 1", c->n_shared);
    if (c->n_shared == 1 &&
        (c->shared_inter < 32 || c->shared_inter > 16384 || c->shared_inter % 32))
        return fail(MOE_ERR_UNSUPPORTED, "shared_inter=%d: need a multiple of 32 in [32, 16384]",
                    c->shared_inter);
    if (c->expert_format < MOE_FORMAT_INT4 || c->expert_format > MOE_FORMAT_G64 ||
        c->shared_format < MOE_FORMAT_INT4 || c->shared_format > MOE_FORMAT_G64)
        return fail(MOE_ERR_INVALID, "expert_format / shared_format: need a MOE_FORMAT_* value");
    if (c->expert_format != MOE_FORMAT_INT4 || (c->n_shared && c->shared_format != MOE_FORMAT_INT4)) {
        if (c->hidden % 128 || c->moe_inter % 128 || (c->n_shared && c->shared_inter % 128))
            return fail(MOE_ERR_UNSUPPORTED, "int8 / group-64 experts need H, I and I_shared multiples of 128");
        if (c->flags & MOE_FLAG_CUDA_CORES)
            return fail(MOE_ERR_UNSUPPORTED, "int8 / group-64 experts run on the tensor-core kernels only");
    }
    if (c->score_func != MOE_SCORE_SIGMOID && c->score_func != MOE_SCORE_SOFTMAX)
        return fail(MOE_ERR_INVALID, "score_func=%d: need MOE_SCORE_SIGMOID or MOE_SCORE_SOFTMAX", c->score_func);
    if (c->n_group < 1 || c->n_group > 32 || c->n_experts % c->n_group)
        return fail(MOE_ERR_INVALID, "n_group=%d: need 1..32 dividing n_experts", c->n_group);
    if (c->n_group > 1) {
        if (c->score_func != MOE_SCORE_SIGMOID)
            return fail(MOE_ERR_INVALID, "n_group > 1 needs the sigmoid score");
        if (c->topk_group < 1 || c->topk_group > c->n_group)
            return fail(MOE_ERR_INVALID, "topk_group=%d: need 1..n_group", c->topk_group);
        if (c->top_k > c->topk_group * (c->n_experts / c->n_group))
            return fail(MOE_ERR_INVALID, "top_k=%d exceeds the experts of the kept groups", c->top_k);
    }
    if (c->norm_topk != 0 && c->norm_topk != 1)
        return fail(MOE_ERR_INVALID, "norm_topk=%d: need 0 or 1", c->norm_topk);
    if (!isfinite(c->routed_scale)) return fail(MOE_ERR_INVALID, "routed_scale is not finite");
    if (c->flags & ~(MOE_FLAG_PRENORM_RESIDUAL | MOE_FLAG_TRACE | MOE_FLAG_CUDA_CORES | MOE_FLAG_DEBUG_CHECKS))
        return fail(MOE_ERR_INVALID, "unknown flags 0x%x", c->flags);
    if ((c->flags & MOE_FLAG_PRENORM_RESIDUAL) && !(c->rms_eps >= 0.0f && isfinite(c->rms_eps)))
        return fail(MOE_ERR_INVALID, "rms_eps must be finite and >= 0");
    if (max_tokens < 1 || max_tokens > kMaxTokens)
        return fail(MOE_ERR_INVALID, "max_tokens=%d: need 1..%d", max_tokens, kMaxTokens);
    const int ep = c->ep_size == 0 ? 1 : c->ep_size;
    if (ep < 1 || ep > c->n_experts || c->ep_rank < 0 || c->ep_rank >= ep)
        return fail(MOE_ERR_INVALID, "ep_size=%d, ep_rank=%d: need 1 <= ep_size <= n_experts, 0 <= ep_rank < ep_size",
                    c->ep_size, c->ep_rank);
    d->H = c->hidden;
    d->E = c->n_experts;
    d->K = c->top_k;
    d->I = c->moe_inter;
    d->n_shared = (c->n_shared && c->ep_rank == 0) ? 1 : 0;   // the shared expert is rank 0's
    d->I_sh = d->n_shared ? c->shared_inter : 0;
    d->I_max = d->I > d->I_sh ? d->I : d->I_sh;
    d->norm_topk = c->norm_topk;
    d->n_group = c->n_group;
    d->topk_group = c->n_group > 1 ? c->topk_group : 1;
    d->score_func = c->score_func;
    d->expert_fmt = c->expert_format;
    d->shared_fmt = d->n_shared ? c->shared_format : MOE_FORMAT_INT4;
    d->mma_fmt = (d->expert_fmt != MOE_FORMAT_INT4 || d->shared_fmt != MOE_FORMAT_INT4) ? 1 : 0;
    d->tc = moe::tc_supported(*d) ? 1 : 0;
    d->prenorm = (c->flags & MOE_FLAG_PRENORM_RESIDUAL) ? 1 : 0;
    d->ep_lo = (int)((long long)c->ep_rank * c->n_experts / ep);
    d->ep_hi = (int)((long long)(c->ep_rank + 1) * c->n_experts / ep);
    d->resid = (d->prenorm && c->ep_rank == 0) ? 1 : 0;
    d->scale = c->routed_scale;
    d->eps = c->rms_eps;
    d->max_tokens = max_tokens;
    d->fast_decode = (ep == 1 && moe::decode_fast_supported(*d)) ? 1 : 0;
    d->mma = (moe::mma_supported(*d) && !(c->flags & MOE_FLAG_CUDA_CORES)) ? 1 : 0;
    d->trace = (c->flags & MOE_FLAG_TRACE) ? 1 : 0;
    d->debug_checks = (c->flags & MOE_FLAG_DEBUG_CHECKS) ? 1 : 0;
    return MOE_OK;
}

bool is_device_ptr(const void *ptr) {
    cudaPointerAttributes a;
    if (cudaPointerGetAttributes(&a, ptr) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    return a.type == cudaMemoryTypeDevice || a.type == cudaMemoryTypeManaged;
}

moe_status check_weights(const moe::Dims &d, const moe_weights *w) {
    if (!w) return fail(MOE_ERR_INVALID, "weights is NULL");
    if (!w->router_w || !w->router_bias) return fail(MOE_ERR_INVALID, "router_w / router_bias is NULL");
    if (!aligned16(w->router_w)) return fail(MOE_ERR_INVALID, "router_w must be 16-byte aligned");
    if (!is_device_ptr(w->router_w) || !is_device_ptr(w->router_bias))
        return fail(MOE_ERR_INVALID, "router_w / router_bias are not device pointers");
    if (!w->expert_slab || !w->expert_scale) return fail(MOE_ERR_INVALID, "expert pointer arrays are NULL");
    for (int e = d.ep_lo; e < d.ep_hi; e++) {     // the experts this handle computes
        const void *s = w->expert_slab[e], *c = w->expert_scale[e];
        if (!s || !c) return fail(MOE_ERR_INVALID, "expert %d: NULL slab or scale", e);
        if (!aligned16(s) || !aligned16(c))
            return fail(MOE_ERR_INVALID, "expert %d: slab and scale must be 16-byte aligned", e);
        if (!is_device_ptr(s) || !is_device_ptr(c))
            return fail(MOE_ERR_INVALID, "expert %d: slab / scale are not device pointers", e);
    }
    if (d.n_shared) {
        if (!w->shared_slab || !w->shared_scale) return fail(MOE_ERR_INVALID, "shared expert pointers are NULL");
        if (!aligned16(w->shared_slab) || !aligned16(w->shared_scale))
            return fail(MOE_ERR_INVALID, "shared slab and scale must be 16-byte aligned");
        if (!is_device_ptr(w->shared_slab) || !is_device_ptr(w->shared_scale))
            return fail(MOE_ERR_INVALID, "shared slab / scale are not device pointers");
    }
    return MOE_OK;
}

void free_events(moe_handle *h) {
    if (h->prof_ev) {
        for (int i = 0; i < h->prof_max * (moe::kStages + 1); i++)
            if (h->prof_ev[i]) cudaEventDestroy(h->prof_ev[i]);
        delete[] h->prof_ev;
    }
    h->prof_ev = nullptr;
    h->prof_max = 0;
    h->prof_n = 0;
}

void free_handle(moe_handle *h) {
    if (!h) return;
    free_events(h);
    if (h->ws_base) cudaFree(h->ws_base);
    if (h->tables) cudaFree(h->tables);
    if (h->tmaps) cudaFree(h->tmaps);
    if (h->x_stage) cudaFree(h->x_stage);
    if (h->y_stage) cudaFree(h->y_stage);
    delete h;
}

bool ranges_overlap(const void *a, const void *b, size_t n) {
    const char *pa = static_cast<const char *>(a), *pb = static_cast<const char *>(b);
    return pa < pb + n && pb < pa + n;
}

moe_status run(moe_handle *h, const float *x, int32_t T, float *y, int32_t *topk_idx,
               float *topk_w, int32_t *counts, void *stream, bool debug) {
    if (!h) return fail(MOE_ERR_INVALID, "handle is NULL");
    if (T < 0 || T > h->p.d.max_tokens)
        return fail(MOE_ERR_INVALID, "T=%d: need 0..max_tokens=%d", T, h->p.d.max_tokens);
    if (T == 0) return MOE_OK;
    if (!x || !y) return fail(MOE_ERR_INVALID, "x / y is NULL");
    if (!aligned16(x) || !aligned16(y)) return fail(MOE_ERR_INVALID, "x and y must be 16-byte aligned");
    const size_t bytes = (size_t)T * h->p.d.H * sizeof(float);
    if (ranges_overlap(x, y, bytes)) return fail(MOE_ERR_INVALID, "x and y overlap");
    if (debug && (!topk_idx || !topk_w)) return fail(MOE_ERR_INVALID, "topk_idx / topk_w is NULL");
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    if (dev != h->device)
        return fail(MOE_ERR_INVALID, "current device %d is not the handle's device %d", dev, h->device);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaEvent_t *ev = nullptr;
    if (h->prof_ev && h->prof_n < h->prof_max) ev = h->prof_ev + (size_t)(h->prof_n++) * (moe::kStages + 1);
    e = moe::launch_forward(h->p, x, T, y, st, counts != nullptr, ev);
    if (e != cudaSuccess) return cuda_fail(e, "kernel launch");
    h->last_T = T;
    h->last_buckets = moe::buckets_built(h->p.d, T, counts != nullptr);
    if (h->p.d.debug_checks) {
        e = moe::launch_checks(h->p, T, h->last_buckets, st);
        if (e != cudaSuccess) return cuda_fail(e, "check kernel launch");
    }
    if (debug) {
        const size_t nk = (size_t)T * h->p.d.K;
        e = cudaMemcpyAsync(topk_idx, h->p.ws.topk_idx, nk * sizeof(int32_t), cudaMemcpyDeviceToDevice, st);
        if (e == cudaSuccess)
            e = cudaMemcpyAsync(topk_w, h->p.ws.topk_w, nk * sizeof(float), cudaMemcpyDeviceToDevice, st);
        if (e == cudaSuccess && counts)
            e = cudaMemcpyAsync(counts, h->p.ws.cnt, (size_t)h->p.d.E * sizeof(int32_t),
                                cudaMemcpyDeviceToDevice, st);
        if (e != cudaSuccess) return cuda_fail(e, "debug copy");
    }
    return MOE_OK;
}

}  // namespace

extern "C" {

int32_t moe_abi_version(void) { return MOE_ABI_VERSION; }

const char *moe_last_error(void) { return g_err; }

size_t moe_workspace_bytes(const moe_config *cfg, int32_t max_tokens) {
    moe::Dims d;
    if (check_config(cfg, max_tokens, &d) != MOE_OK) return 0;
    return moe::workspace_bytes(d);
}

moe_status moe_init(const moe_config *cfg, const moe_weights *w, int32_t max_tokens, moe_handle **out) {
    if (!out) return fail(MOE_ERR_INVALID, "out is NULL");
    *out = nullptr;
    g_err[0] = '\0';
    moe::Dims d;
    moe_status s = check_config(cfg, max_tokens, &d);
    if (s != MOE_OK) return s;
    s = check_weights(d, w);
    if (s != MOE_OK) return s;

    moe_handle *h = new (std::nothrow) moe_handle();
    if (!h) return fail(MOE_ERR_NOMEM, "host allocation failed");
    cudaError_t e = cudaGetDevice(&h->device);
    if (e != cudaSuccess) { free_handle(h); return cuda_fail(e, "cudaGetDevice"); }

    h->ws_bytes = moe::workspace_bytes(d);
    e = cudaMalloc(&h->ws_base, h->ws_bytes);
    if (e != cudaSuccess) { h->ws_base = nullptr; free_handle(h); return cuda_fail(e, "workspace cudaMalloc"); }
    const size_t tbytes = 2 * (size_t)d.E * sizeof(void *);
    e = cudaMalloc(&h->tables, tbytes);
    if (e != cudaSuccess) { h->tables = nullptr; free_handle(h); return cuda_fail(e, "table cudaMalloc"); }
    const size_t stage = (size_t)max_tokens * d.H * sizeof(float);
    e = cudaMalloc(reinterpret_cast<void **>(&h->x_stage), stage);
    if (e == cudaSuccess) e = cudaMalloc(reinterpret_cast<void **>(&h->y_stage), stage);
    if (e != cudaSuccess) { free_handle(h); return cuda_fail(e, "staging cudaMalloc"); }

    void **host_tab = new (std::nothrow) void *[2 * (size_t)d.E];
    if (!host_tab) { free_handle(h); return fail(MOE_ERR_NOMEM, "host allocation failed"); }
    for (int i = 0; i < d.E; i++) {      // experts another rank computes: NULL (never read)
        const bool own = i >= d.ep_lo && i < d.ep_hi;
        host_tab[i] = own ? const_cast<uint8_t *>(w->expert_slab[i]) : nullptr;
        host_tab[d.E + i] = own ? const_cast<float *>(w->expert_scale[i]) : nullptr;
    }
    e = cudaMemcpy(h->tables, host_tab, tbytes, cudaMemcpyHostToDevice);
    if (e != cudaSuccess) { delete[] host_tab; free_handle(h); return cuda_fail(e, "table upload"); }

    moe::Params &p = h->p;
    p.d = d;
    p.router_w = w->router_w;
    p.router_b = w->router_bias;
    p.slabs = static_cast<const uint8_t *const *>(h->tables);
    p.scales = reinterpret_cast<const float *const *>(static_cast<void **>(h->tables) + d.E);
    p.sh_slab = d.n_shared ? w->shared_slab : nullptr;
    p.sh_scale = d.n_shared ? w->shared_scale : nullptr;
    moe::carve_workspace(d, h->ws_base, &p.ws);
    const size_t nmaps = moe::tc_map_count(d);
    if (nmaps) {
        e = cudaMalloc(&h->tmaps, nmaps * moe::kTmapBytes);
        if (e != cudaSuccess) { h->tmaps = nullptr; delete[] host_tab; free_handle(h); return cuda_fail(e, "tensor-map cudaMalloc"); }
        p.tmaps = h->tmaps;
        e = moe::upload_tc_maps(p, reinterpret_cast<const uint8_t *const *>(host_tab), h->tmaps);
        if (e != cudaSuccess) { delete[] host_tab; free_handle(h); return cuda_fail(e, "tensor-map encoding"); }
    } else {
        p.tmaps = nullptr;
    }
    delete[] host_tab;
    e = cudaMemset(h->ws_base, 0, h->ws_bytes);
    if (e == cudaSuccess) e = moe::prepare_kernels(p.d);
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e != cudaSuccess) { free_handle(h); return cuda_fail(e, "workspace init"); }
    *out = h;
    return MOE_OK;
}

moe_status moe_forward(moe_handle *h, const float *x, int32_t T, float *y, void *stream) {
    return run(h, x, T, y, nullptr, nullptr, nullptr, stream, false);
}

moe_status moe_forward_debug(moe_handle *h, const float *x, int32_t T, float *y, int32_t *topk_idx,
                             float *topk_w, int32_t *expert_counts, void *stream) {
    return run(h, x, T, y, topk_idx, topk_w, expert_counts, stream, true);
}

moe_status moe_forward_host(moe_handle *h, const float *x_host, int32_t T, float *y_host, void *stream) {
    if (!h) return fail(MOE_ERR_INVALID, "handle is NULL");
    if (T < 0 || T > h->p.d.max_tokens)
        return fail(MOE_ERR_INVALID, "T=%d: need 0..max_tokens=%d", T, h->p.d.max_tokens);
    if (T == 0) return MOE_OK;
    if (!x_host || !y_host) return fail(MOE_ERR_INVALID, "x_host / y_host is NULL");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const size_t bytes = (size_t)T * h->p.d.H * sizeof(float);
    cudaError_t e = cudaMemcpyAsync(h->x_stage, x_host, bytes, cudaMemcpyHostToDevice, st);
    if (e != cudaSuccess) return cuda_fail(e, "input copy");
    moe_status s = run(h, h->x_stage, T, h->y_stage, nullptr, nullptr, nullptr, stream, false);
    if (s != MOE_OK) return s;
    e = cudaMemcpyAsync(y_host, h->y_stage, bytes, cudaMemcpyDeviceToHost, st);
    if (e != cudaSuccess) return cuda_fail(e, "output copy");
    e = cudaStreamSynchronize(st);
    if (e != cudaSuccess) return cuda_fail(e, "stream synchronize");
    return MOE_OK;
}

moe_status moe_profile_start(moe_handle *h, int32_t max_calls) {
    if (!h) return fail(MOE_ERR_INVALID, "handle is NULL");
    if (max_calls < 0 || max_calls > 4096) return fail(MOE_ERR_INVALID, "max_calls=%d: need 0..4096", max_calls);
    cudaError_t e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return cuda_fail(e, "device synchronize");
    free_events(h);
    if (max_calls == 0) return MOE_OK;
    const int n = max_calls * (moe::kStages + 1);
    h->prof_ev = new (std::nothrow) cudaEvent_t[n]();
    if (!h->prof_ev) return fail(MOE_ERR_NOMEM, "host allocation failed");
    h->prof_max = max_calls;
    for (int i = 0; i < n; i++) {
        e = cudaEventCreate(&h->prof_ev[i]);
        if (e != cudaSuccess) { free_events(h); return cuda_fail(e, "cudaEventCreate"); }
    }
    return MOE_OK;
}

moe_status moe_profile_read(moe_handle *h, int32_t *n_calls, float *stage_ms) {
    if (!h || !n_calls || !stage_ms) return fail(MOE_ERR_INVALID, "NULL argument");
    *n_calls = h->prof_n;
    for (int s = 0; s < moe::kStages; s++) stage_ms[s] = 0.0f;
    if (!h->prof_ev || h->prof_n == 0) return MOE_OK;
    double sum[moe::kStages] = {0, 0, 0, 0};
    for (int c = 0; c < h->prof_n; c++) {
        cudaEvent_t *ev = h->prof_ev + (size_t)c * (moe::kStages + 1);
        cudaError_t e = cudaEventSynchronize(ev[moe::kStages]);
        if (e != cudaSuccess) return cuda_fail(e, "cudaEventSynchronize");
        for (int s = 0; s < moe::kStages; s++) {
            float ms = 0.0f;
            e = cudaEventElapsedTime(&ms, ev[s], ev[s + 1]);
            if (e != cudaSuccess) return cuda_fail(e, "cudaEventElapsedTime");
            sum[s] += ms;
        }
    }
    for (int s = 0; s < moe::kStages; s++) stage_ms[s] = (float)(sum[s] / h->prof_n);
    return MOE_OK;
}

moe_status moe_device_error(moe_handle *h, uint32_t *flags) {
    if (!h || !flags) return fail(MOE_ERR_INVALID, "NULL argument");
    unsigned v = 0;
    cudaError_t e = cudaDeviceSynchronize();
    if (e == cudaSuccess) e = cudaMemcpy(&v, h->p.ws.err, sizeof(v), cudaMemcpyDeviceToHost);
    if (e == cudaSuccess && v) {
        // a kernel gave up part-way: start the barrier counters and the call
        // counter afresh so that the next call is consistent again (until this
        // reset, every call on the handle is invalid)
        e = cudaMemset(h->p.ws.counters, 0, 16 * sizeof(unsigned));
        if (e == cudaSuccess) e = cudaMemset(h->p.ws.err, 0, 4 * sizeof(unsigned));
        if (e == cudaSuccess) e = cudaDeviceSynchronize();
    }
    if (e != cudaSuccess) return cuda_fail(e, "reading the device error word");
    *flags = v;
    if (v) return fail(MOE_ERR_CUDA, "a kernel gave up waiting (flags 0x%x)", v);
    return MOE_OK;
}

moe_status moe_debug_check(moe_handle *h, int32_t T) {
    if (!h) return fail(MOE_ERR_INVALID, "handle is NULL");
    if (T < 1 || T > h->p.d.max_tokens) return fail(MOE_ERR_INVALID, "T=%d: need 1..max_tokens", T);
    cudaError_t e = cudaDeviceSynchronize();
    if (e == cudaSuccess) e = moe::launch_checks(h->p, T, T == h->last_T && h->last_buckets, nullptr);
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return cuda_fail(e, "check kernel");
    return MOE_OK;
}

moe_status moe_debug_set_topk(moe_handle *h, int32_t pair, int32_t expert) {
    if (!h) return fail(MOE_ERR_INVALID, "handle is NULL");
    if (pair < 0 || (long long)pair >= (long long)h->p.d.max_tokens * h->p.d.K)
        return fail(MOE_ERR_INVALID, "pair=%d: need 0..max_tokens*K-1", pair);
    cudaError_t e = cudaDeviceSynchronize();
    if (e == cudaSuccess) e = cudaMemcpy(h->p.ws.topk_idx + pair, &expert, sizeof(expert), cudaMemcpyHostToDevice);
    if (e != cudaSuccess) return cuda_fail(e, "writing the top-K index");
    return MOE_OK;
}

moe_status moe_debug_check_result(moe_handle *h, int32_t *pair, int32_t *code) {
    if (!h || !pair || !code) return fail(MOE_ERR_INVALID, "NULL argument");
    unsigned v[4] = {0, 0, 0, 0};
    cudaError_t e = cudaDeviceSynchronize();
    if (e == cudaSuccess) e = cudaMemcpy(v, h->p.ws.err, sizeof(v), cudaMemcpyDeviceToHost);
    if (e != cudaSuccess) return cuda_fail(e, "reading the check record");
    *pair = v[1] ? (int32_t)(v[1] - 1) : -1;
    *code = v[1] ? (int32_t)v[2] : 0;
    return MOE_OK;
}

moe_status moe_debug_stall_next_call(moe_handle *h) {
    if (!h) return fail(MOE_ERR_INVALID, "handle is NULL");
    if (!h->p.d.fast_decode) return fail(MOE_ERR_UNSUPPORTED, "T == 1 calls on this handle do not use the decode kernel");
    // counters[7] is the number of the handle's last call; every barrier target of the next
    // call is that number + 1 times the grid, which the barrier counters (at most the calls
    // so far times the grid) then cannot reach
    unsigned calls = 0;
    cudaError_t e = cudaDeviceSynchronize();
    if (e == cudaSuccess) e = cudaMemcpy(&calls, h->p.ws.counters + 7, sizeof(calls), cudaMemcpyDeviceToHost);
    calls += 1000u;
    if (e == cudaSuccess) e = cudaMemcpy(h->p.ws.counters + 7, &calls, sizeof(calls), cudaMemcpyHostToDevice);
    if (e != cudaSuccess) return cuda_fail(e, "moving the call counter");
    return MOE_OK;
}

int32_t moe_uses_streaming_decode(const moe_handle *h) { return h ? h->p.d.fast_decode : 0; }

int32_t moe_streaming_decode_max_tokens(const moe_handle *h) {
    return (h && h->p.d.fast_decode) ? moe::decode_loop_max_tokens() : 0;
}

int32_t moe_uses_tensor_cores(const moe_handle *h) { return h ? h->p.d.mma : 0; }

moe_status moe_trace_read(moe_handle *h, uint64_t *out, int32_t capacity_blocks, int32_t *n_blocks) {
    if (!h || !out || !n_blocks || capacity_blocks < 0) return fail(MOE_ERR_INVALID, "NULL argument or negative capacity");
    if (!h->p.d.trace || !h->p.d.fast_decode)
        return fail(MOE_ERR_UNSUPPORTED, "the handle records no trace (MOE_FLAG_TRACE and the decode kernel needed)");
    const int g = moe::decode_grid_blocks(h->p.d);
    const int n = g < capacity_blocks ? g : capacity_blocks;
    cudaError_t e = cudaDeviceSynchronize();
    if (e == cudaSuccess && n > 0)
        e = cudaMemcpy(out, h->p.ws.trace, (size_t)n * MOE_TRACE_SLOTS * sizeof(uint64_t), cudaMemcpyDeviceToHost);
    if (e != cudaSuccess) return cuda_fail(e, "reading the trace");
    *n_blocks = g;
    return MOE_OK;
}

moe_status moe_destroy(moe_handle *h) {
    if (!h) return MOE_OK;
    int cur = -1;
    cudaGetDevice(&cur);
    const int dev = h->device;
    if (cur != dev) cudaSetDevice(dev);
    const cudaError_t e = cudaDeviceSynchronize();
    free_handle(h);
    if (cur >= 0 && cur != dev) cudaSetDevice(cur);
    if (e != cudaSuccess) return cuda_fail(e, "device synchronize before free");
    return MOE_OK;
}


// --- operators around the router and its experts (no handle) ---------------

#define MOE_NEED(cond, status, ...) \
    do { if (!(cond)) return fail(status, __VA_ARGS__); } while (0)

static bool dtype_ok(int32_t d) { return d == MOE_DTYPE_F32 || d == MOE_DTYPE_F16 || d == MOE_DTYPE_BF16; }
static bool aligned4(const void *ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 3u) == 0; }
static bool aligned_el(const void *ptr, int32_t dtype) {
    return (reinterpret_cast<uintptr_t>(ptr) & (dtype == MOE_DTYPE_F32 ? 3u : 1u)) == 0;
}
static moe_status launched(cudaError_t e, const char *what) { return e == cudaSuccess ? MOE_OK : cuda_fail(e, what); }

int64_t moe_expert_lists_rows(int32_t T, int32_t top_k, int32_t n_experts, int32_t align) {
    if (T < 0 || top_k < 1 || n_experts < 1 || align < 1) return -1;
    const int64_t pairs = (int64_t)T * top_k, most = pairs < n_experts ? pairs : n_experts;
    return (pairs + most * (align - 1) + align - 1) / align * align;
}

size_t moe_expert_lists_workspace(int32_t T, int32_t top_k, int32_t n_experts) {
    if (T < 0 || top_k < 1 || n_experts < 1) return 0;
    return moe::lists_workspace((long long)T * top_k, n_experts);
}

moe_status moe_expert_lists(const int32_t *topk_idx, int32_t T, int32_t top_k, int32_t n_experts, int32_t align,
                            int32_t *counts, int32_t *offsets, int32_t *rows, int32_t *pos, void *workspace,
                            size_t workspace_bytes, void *stream) {
    MOE_NEED(T >= 0, MOE_ERR_INVALID, "T=%d is negative", T);
    MOE_NEED(n_experts >= 1 && n_experts <= 1024, MOE_ERR_UNSUPPORTED, "n_experts=%d: need 1..1024", n_experts);
    MOE_NEED(top_k >= 1 && top_k <= 1024, MOE_ERR_UNSUPPORTED, "top_k=%d: need 1..1024", top_k);
    MOE_NEED(align >= 1 && align <= 4096, MOE_ERR_UNSUPPORTED, "align=%d: need 1..4096", align);
    const int64_t room = moe_expert_lists_rows(T, top_k, n_experts, align);
    MOE_NEED(room < (1ll << 31), MOE_ERR_UNSUPPORTED, "%lld rows: need fewer than 2^31", (long long)room);
    MOE_NEED(counts && offsets, MOE_ERR_INVALID, "counts / offsets is NULL");
    MOE_NEED(T == 0 || (topk_idx && rows && pos), MOE_ERR_INVALID, "topk_idx / rows / pos is NULL");
    MOE_NEED(aligned4(topk_idx) && aligned4(counts) && aligned4(offsets) && aligned4(rows) && aligned4(pos),
             MOE_ERR_INVALID, "int32 buffers must be 4-byte aligned");
    const size_t need = moe_expert_lists_workspace(T, top_k, n_experts);
    MOE_NEED(need == 0 || (workspace && aligned16(workspace) && workspace_bytes >= need), MOE_ERR_INVALID,
             "workspace: need %zu bytes, 16-byte aligned", need);
    return launched(moe::launch_lists(topk_idx, T, top_k, n_experts, align, room, counts, offsets, rows, pos, workspace,
                                      static_cast<cudaStream_t>(stream)), "moe_expert_lists");
}

static moe_status check_balance(const void *logits, int32_t dtype, int64_t ld, int32_t T, int32_t E, int32_t top_k,
                                int32_t score_func, float coef, const int32_t *seq, int32_t n_seq) {
    MOE_NEED(dtype_ok(dtype), MOE_ERR_INVALID, "dtype=%d: need a MOE_DTYPE_* value", dtype);
    MOE_NEED(T >= 0, MOE_ERR_INVALID, "T=%d is negative", T);
    MOE_NEED(T <= MOE_BALANCE_MAX_TOKENS, MOE_ERR_UNSUPPORTED, "T=%d: need %d or fewer", T, MOE_BALANCE_MAX_TOKENS);
    MOE_NEED(E >= 1 && E <= 1024, MOE_ERR_UNSUPPORTED, "n_experts=%d: need 1..1024", E);
    MOE_NEED(top_k >= 1 && top_k <= E, MOE_ERR_INVALID, "top_k=%d: need 1..n_experts", top_k);
    MOE_NEED(ld >= E, MOE_ERR_INVALID, "ld=%lld: need n_experts or more", (long long)ld);
    MOE_NEED(score_func == MOE_SCORE_SIGMOID || score_func == MOE_SCORE_SOFTMAX, MOE_ERR_INVALID,
             "score_func=%d: need MOE_SCORE_SIGMOID or MOE_SCORE_SOFTMAX", score_func);
    MOE_NEED(isfinite(coef), MOE_ERR_INVALID, "coef is not finite");
    MOE_NEED(n_seq >= 1 && n_seq <= 65535, MOE_ERR_UNSUPPORTED, "n_seq=%d: need 1..65535", n_seq);
    MOE_NEED(seq || n_seq == 1, MOE_ERR_INVALID, "n_seq=%d without seq_offsets", n_seq);
    MOE_NEED(T == 0 || logits, MOE_ERR_INVALID, "logits is NULL");
    MOE_NEED(aligned_el(logits, dtype) && aligned4(seq), MOE_ERR_INVALID, "logits / seq_offsets are not aligned to their elements");
    return MOE_OK;
}

size_t moe_balance_workspace(int32_t T, int32_t n_experts, int32_t n_seq) {
    if (T < 0 || T > MOE_BALANCE_MAX_TOKENS || n_experts < 1 || n_seq < 1) return 0;
    return moe::balance_workspace(T, n_experts, n_seq);
}

moe_status moe_balance_forward(const void *logits, int32_t dtype, int64_t ld, int32_t T, int32_t n_experts,
                               const int32_t *topk_idx, int32_t top_k, int32_t score_func, float coef,
                               const int32_t *seq_offsets, int32_t n_seq, const uint8_t *mask, float *loss,
                               int32_t *counts, float *prob_sums, int32_t *tokens, void *workspace,
                               size_t workspace_bytes, void *stream) {
    const moe_status s = check_balance(logits, dtype, ld, T, n_experts, top_k, score_func, coef, seq_offsets, n_seq);
    if (s != MOE_OK) return s;
    MOE_NEED(T == 0 || topk_idx, MOE_ERR_INVALID, "topk_idx is NULL");
    MOE_NEED(loss && counts && prob_sums && tokens, MOE_ERR_INVALID, "an output is NULL");
    MOE_NEED(aligned4(topk_idx) && aligned4(loss) && aligned4(counts) && aligned4(prob_sums) && aligned4(tokens),
             MOE_ERR_INVALID, "int32 / float32 buffers must be 4-byte aligned");
    const size_t need = moe_balance_workspace(T, n_experts, n_seq);
    MOE_NEED(workspace && aligned16(workspace) && workspace_bytes >= need, MOE_ERR_INVALID,
             "workspace: need %zu bytes, 16-byte aligned", need);
    return launched(moe::launch_balance_forward(logits, dtype, ld, T, n_experts, topk_idx, top_k, score_func == MOE_SCORE_SOFTMAX,
                                                coef, seq_offsets, n_seq, mask, loss, counts, prob_sums, tokens, workspace,
                                                static_cast<cudaStream_t>(stream)), "moe_balance_forward");
}

moe_status moe_balance_backward(const void *logits, int32_t dtype, int64_t ld, int32_t T, int32_t n_experts, int32_t top_k,
                                int32_t score_func, float coef, const int32_t *counts, const int32_t *tokens,
                                const int32_t *seq_offsets, int32_t n_seq, const uint8_t *mask, const float *grad_loss,
                                void *dlogits, int64_t ldd, int32_t zero_rest, void *stream) {
    const moe_status s = check_balance(logits, dtype, ld, T, n_experts, top_k, score_func, coef, seq_offsets, n_seq);
    if (s != MOE_OK) return s;
    MOE_NEED(counts && tokens, MOE_ERR_INVALID, "counts / tokens is NULL");
    MOE_NEED(ldd >= n_experts, MOE_ERR_INVALID, "ldd=%lld: need n_experts or more", (long long)ldd);
    MOE_NEED(aligned4(counts) && aligned4(tokens) && aligned4(grad_loss) && aligned_el(dlogits, dtype), MOE_ERR_INVALID,
             "a buffer is not aligned to its elements");
    if (T == 0) return MOE_OK;
    MOE_NEED(dlogits, MOE_ERR_INVALID, "dlogits is NULL");
    return launched(moe::launch_balance_backward(logits, dtype, ld, T, n_experts, top_k, score_func == MOE_SCORE_SOFTMAX, coef,
                                                 counts, tokens, seq_offsets, n_seq, mask, grad_loss, dlogits, ldd, zero_rest != 0,
                                                 static_cast<cudaStream_t>(stream)), "moe_balance_backward");
}

static const int32_t kMaxWidth = 131072, kMaxRows = 65535 * 128;

moe_status moe_fp8_quantize(const void *x, int32_t dtype, int64_t ld, int32_t n_tokens, int32_t width, const int32_t *rows,
                            int32_t R, uint8_t *codes, float *scales, uint8_t *codes_t, float *scales_t, void *stream) {
    MOE_NEED(dtype_ok(dtype), MOE_ERR_INVALID, "dtype=%d: need a MOE_DTYPE_* value", dtype);
    MOE_NEED(n_tokens >= 0 && R >= 0, MOE_ERR_INVALID, "n_tokens=%d, R=%d: negative", n_tokens, R);
    MOE_NEED(rows || R == n_tokens, MOE_ERR_INVALID, "R=%d without rows: need n_tokens=%d", R, n_tokens);
    MOE_NEED(width >= 16 && width <= kMaxWidth && width % 16 == 0, MOE_ERR_UNSUPPORTED,
             "width=%d: need a multiple of 16 in 16..%d", width, kMaxWidth);
    MOE_NEED(R <= kMaxRows, MOE_ERR_UNSUPPORTED, "R=%d: need %d or fewer", R, kMaxRows);
    MOE_NEED(ld >= width, MOE_ERR_INVALID, "ld=%lld: need width or more", (long long)ld);
    MOE_NEED((codes_t == nullptr) == (scales_t == nullptr), MOE_ERR_INVALID, "codes_t and scales_t: give both or neither");
    if (R == 0) return MOE_OK;
    MOE_NEED((x || n_tokens == 0) && codes && scales, MOE_ERR_INVALID, "x / codes / scales is NULL");
    MOE_NEED(aligned16(x) && ld * (dtype == MOE_DTYPE_F32 ? 4 : 2) % 16 == 0, MOE_ERR_INVALID,
             "every row of x must start on a 16-byte boundary");
    MOE_NEED(aligned16(codes) && aligned16(codes_t) && aligned4(scales) && aligned4(scales_t) && aligned4(rows), MOE_ERR_INVALID,
             "code buffers must be 16-byte aligned, scales and rows 4-byte aligned");
    return launched(moe::launch_quantize(x, dtype, ld, n_tokens, width, rows, R, codes, scales, codes_t, scales_t,
                                         static_cast<cudaStream_t>(stream)), "moe_fp8_quantize");
}

moe_status moe_fp8_quantize_weights(const void *w, int32_t dtype, int32_t E, int32_t N, int32_t K, uint8_t *codes, float *scales,
                                    uint8_t *codes_t, float *scales_t, void *stream) {
    MOE_NEED(dtype_ok(dtype), MOE_ERR_INVALID, "dtype=%d: need a MOE_DTYPE_* value", dtype);
    MOE_NEED(E >= 1 && E <= 65535, MOE_ERR_UNSUPPORTED, "E=%d: need 1..65535", E);
    MOE_NEED(N >= 1 && N <= kMaxWidth, MOE_ERR_UNSUPPORTED, "N=%d: need 1..%d", N, kMaxWidth);
    MOE_NEED(K >= 16 && K <= kMaxWidth && K % 16 == 0, MOE_ERR_UNSUPPORTED, "K=%d: need a multiple of 16 in 16..%d", K, kMaxWidth);
    MOE_NEED((codes_t == nullptr) == (scales_t == nullptr), MOE_ERR_INVALID, "codes_t and scales_t: give both or neither");
    MOE_NEED(w && codes && scales, MOE_ERR_INVALID, "w / codes / scales is NULL");
    MOE_NEED(aligned16(w) && aligned16(codes) && aligned16(codes_t) && aligned4(scales) && aligned4(scales_t), MOE_ERR_INVALID,
             "w and the code buffers must be 16-byte aligned, scales 4-byte aligned");
    return launched(moe::launch_quantize_weights(w, dtype, E, N, K, codes, scales, codes_t, scales_t,
                                                 static_cast<cudaStream_t>(stream)), "moe_fp8_quantize_weights");
}

moe_status moe_fp8_matmul(const uint8_t *x, const float *x_scale, int32_t R, const uint8_t *w, const float *w_scale, int32_t E,
                          int32_t N, int32_t K, const int32_t *offsets, void *y, int32_t y_dtype, int64_t ldy, void *stream) {
    MOE_NEED(dtype_ok(y_dtype), MOE_ERR_INVALID, "y_dtype=%d: need a MOE_DTYPE_* value", y_dtype);
    MOE_NEED(R >= 0, MOE_ERR_INVALID, "R=%d is negative", R);
    MOE_NEED(R <= kMaxRows, MOE_ERR_UNSUPPORTED, "R=%d: need %d or fewer", R, kMaxRows);
    MOE_NEED(E >= 1 && E <= 1024, MOE_ERR_UNSUPPORTED, "E=%d: need 1..1024", E);
    MOE_NEED(offsets || E == 1, MOE_ERR_INVALID, "E=%d without offsets", E);
    MOE_NEED(N >= 1 && N <= kMaxWidth, MOE_ERR_UNSUPPORTED, "N=%d: need 1..%d", N, kMaxWidth);
    MOE_NEED(K >= 16 && K <= kMaxWidth && K % 16 == 0, MOE_ERR_UNSUPPORTED, "K=%d: need a multiple of 16 in 16..%d", K, kMaxWidth);
    MOE_NEED(ldy >= N, MOE_ERR_INVALID, "ldy=%lld: need N or more", (long long)ldy);
    if (R == 0) return MOE_OK;
    MOE_NEED(x && x_scale && w && w_scale && y, MOE_ERR_INVALID, "a pointer is NULL");
    MOE_NEED(aligned16(x) && aligned16(w) && aligned4(x_scale) && aligned4(w_scale) && aligned4(offsets) && aligned_el(y, y_dtype),
             MOE_ERR_INVALID, "codes must be 16-byte aligned, the other buffers to their elements");
    return launched(moe::launch_fp8_matmul(x, x_scale, R, w, w_scale, E, N, K, offsets, y, y_dtype, ldy,
                                           static_cast<cudaStream_t>(stream)), "moe_fp8_matmul");
}

moe_status moe_fp8_wgrad(const uint8_t *xt, const float *xt_scale, const uint8_t *dyt, const float *dyt_scale, int32_t R,
                         int32_t N, int32_t K, int32_t E, const int32_t *offsets, void *dw, int32_t dw_dtype, void *stream) {
    MOE_NEED(dtype_ok(dw_dtype), MOE_ERR_INVALID, "dw_dtype=%d: need a MOE_DTYPE_* value", dw_dtype);
    MOE_NEED(R >= 0 && R % 128 == 0, MOE_ERR_INVALID, "R=%d: need a multiple of 128", R);
    MOE_NEED(R <= kMaxRows, MOE_ERR_UNSUPPORTED, "R=%d: need %d or fewer", R, kMaxRows);
    MOE_NEED(E >= 1 && E <= 1024, MOE_ERR_UNSUPPORTED, "E=%d: need 1..1024", E);
    MOE_NEED(offsets || E == 1, MOE_ERR_INVALID, "E=%d without offsets", E);
    MOE_NEED(N >= 1 && N <= kMaxWidth && K >= 1 && K <= kMaxWidth, MOE_ERR_UNSUPPORTED, "N=%d, K=%d: need 1..%d", N, K, kMaxWidth);
    MOE_NEED(dw && aligned_el(dw, dw_dtype), MOE_ERR_INVALID, "dw is NULL or not aligned to its elements");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (R == 0)
        return launched(cudaMemsetAsync(dw, 0, (size_t)E * N * K * (dw_dtype == MOE_DTYPE_F32 ? 4 : 2), st), "moe_fp8_wgrad");
    MOE_NEED(xt && xt_scale && dyt && dyt_scale, MOE_ERR_INVALID, "a pointer is NULL");
    MOE_NEED(aligned16(xt) && aligned16(dyt) && aligned4(xt_scale) && aligned4(dyt_scale) && aligned4(offsets), MOE_ERR_INVALID,
             "codes must be 16-byte aligned, scales and offsets 4-byte aligned");
    return launched(moe::launch_fp8_wgrad(xt, xt_scale, dyt, dyt_scale, R, N, K, E, offsets, dw, dw_dtype, st), "moe_fp8_wgrad");
}

static bool aligned_rows(const void *p, int64_t ld, int32_t dtype) {
    return aligned16(p) && ld * (dtype == MOE_DTYPE_F32 ? 4 : 2) % 16 == 0;
}

// A tensor in memory: rows of `width` bytes, `pitch` bytes apart, from `at` to `end` (none: both 0).
struct Rows {
    uintptr_t at = 0, end = 0;
    int64_t rows = 0, pitch = 0, width = 0;
    Rows(const void *p, int64_t n, int64_t ld, int64_t elements, int64_t el) {
        if (!p || n < 1) return;
        int64_t bytes;
        at = reinterpret_cast<uintptr_t>(p);
        rows = n;
        width = elements * el;
        if (__builtin_mul_overflow(ld, el, &pitch) || __builtin_mul_overflow(n - 1, pitch, &bytes)) pitch = bytes = n > 1 ? INT64_MAX / 2 : 0;
        end = at + (uintptr_t)bytes + (uintptr_t)width;
    }
    Rows(const void *p, int64_t bytes) {
        if (!p || bytes < 1) return;
        at = reinterpret_cast<uintptr_t>(p);
        end = at + (uintptr_t)bytes;
        rows = 1;
        pitch = width = bytes;
    }
};
static int64_t el_size(int32_t dtype) { return dtype == MOE_DTYPE_F32 ? 4 : 2; }
// Whether the two have bytes in common: slices of other columns of one buffer's rows have none.
static bool overlap(const Rows &a, const Rows &b) {
    if (a.at >= b.end || b.at >= a.end) return false;
    if (a.rows < 2 && b.rows < 2) return true;
    const int64_t g = a.rows < 2 ? b.pitch : b.rows < 2 ? a.pitch : std::gcd(a.pitch, b.pitch), d = (int64_t)(b.at - a.at) % g, r = d < 0 ? d + g : d;
    return r < a.width || r + b.width > g;
}
// The same, but rows on top of one another: each is read by who writes it, before it does.
static bool askew(const Rows &a, const Rows &b) {
    return overlap(a, b) && !(a.at == b.at && a.rows == b.rows && a.width == b.width && (a.rows < 2 || a.pitch == b.pitch));
}

static moe_status check_route(const void *logits, int32_t dtype, int64_t ld, int32_t T, int32_t E, int32_t top_k, int32_t score_func,
                              int32_t norm_topk, float scale) {
    MOE_NEED(dtype_ok(dtype), MOE_ERR_INVALID, "dtype=%d: need a MOE_DTYPE_* value", dtype);
    MOE_NEED(T >= 0, MOE_ERR_INVALID, "T=%d is negative", T);
    MOE_NEED(E >= 1 && E <= 1024, MOE_ERR_UNSUPPORTED, "n_experts=%d: need 1..1024", E);
    MOE_NEED(top_k >= 1 && top_k <= E && top_k <= 32, MOE_ERR_INVALID, "top_k=%d: need 1..min(n_experts, 32)", top_k);
    MOE_NEED(ld >= E, MOE_ERR_INVALID, "ld=%lld: need n_experts or more", (long long)ld);
    MOE_NEED(score_func == MOE_SCORE_SIGMOID || score_func == MOE_SCORE_SOFTMAX, MOE_ERR_INVALID,
             "score_func=%d: need MOE_SCORE_SIGMOID or MOE_SCORE_SOFTMAX", score_func);
    MOE_NEED(norm_topk == 0 || norm_topk == 1, MOE_ERR_INVALID, "norm_topk=%d: need 0 or 1", norm_topk);
    MOE_NEED(isfinite(scale), MOE_ERR_INVALID, "routed_scale is not finite");
    MOE_NEED(T == 0 || logits, MOE_ERR_INVALID, "logits is NULL");
    MOE_NEED(aligned_el(logits, dtype), MOE_ERR_INVALID, "logits is not aligned to its elements");
    return MOE_OK;
}

moe_status moe_route_forward(const void *logits, int32_t dtype, int64_t ld, int32_t T, int32_t n_experts, const float *bias,
                             int32_t top_k, int32_t score_func, int32_t n_group, int32_t topk_group, int32_t norm_topk,
                             float routed_scale, const uint8_t *mask, int32_t *topk_idx, float *topk_w, void *stream) {
    const moe_status s = check_route(logits, dtype, ld, T, n_experts, top_k, score_func, norm_topk, routed_scale);
    if (s != MOE_OK) return s;
    MOE_NEED(n_group >= 1 && n_group <= 32 && n_experts % n_group == 0, MOE_ERR_INVALID,
             "n_group=%d: need 1..32, a divisor of n_experts", n_group);
    MOE_NEED(score_func == MOE_SCORE_SIGMOID || (n_group == 1 && !bias), MOE_ERR_INVALID, "groups and bias go with the sigmoid score alone");
    MOE_NEED(n_group == 1 || (topk_group >= 1 && topk_group <= n_group), MOE_ERR_INVALID, "topk_group=%d: need 1..n_group", topk_group);
    MOE_NEED(n_group == 1 || top_k <= topk_group * (n_experts / n_group), MOE_ERR_INVALID,
             "top_k=%d: need topk_group * n_experts / n_group or fewer", top_k);
    MOE_NEED(T == 0 || (topk_idx && topk_w), MOE_ERR_INVALID, "topk_idx / topk_w is NULL");
    MOE_NEED(aligned4(bias) && aligned4(topk_idx) && aligned4(topk_w), MOE_ERR_INVALID, "int32 / float32 buffers must be 4-byte aligned");
    if (T == 0) return MOE_OK;
    const Rows rx(logits, T, ld, n_experts, el_size(dtype)), ri(topk_idx, (int64_t)T * top_k * 4), rw(topk_w, (int64_t)T * top_k * 4),
        rb(bias, (int64_t)n_experts * 4), rm(mask, T);
    for (const Rows *o : {&ri, &rw})
        MOE_NEED(!overlap(*o, rx) && !overlap(*o, rb) && !overlap(*o, rm), MOE_ERR_INVALID, "topk_idx or topk_w overlaps logits, bias or mask");
    MOE_NEED(!overlap(ri, rw), MOE_ERR_INVALID, "topk_idx and topk_w overlap");
    return launched(moe::launch_route_forward(logits, dtype, ld, T, n_experts, bias, top_k, score_func == MOE_SCORE_SOFTMAX, n_group,
                                              n_group > 1 ? topk_group : 1, norm_topk, routed_scale, mask, topk_idx, topk_w,
                                              static_cast<cudaStream_t>(stream)), "moe_route_forward");
}

moe_status moe_route_backward(const void *logits, int32_t dtype, int64_t ld, int32_t T, int32_t n_experts, const int32_t *topk_idx,
                              int32_t top_k, int32_t score_func, int32_t norm_topk, float routed_scale, const float *grad_w,
                              void *dlogits, int64_t ldd, int32_t accumulate, void *stream) {
    const moe_status s = check_route(logits, dtype, ld, T, n_experts, top_k, score_func, norm_topk, routed_scale);
    if (s != MOE_OK) return s;
    MOE_NEED(ldd >= n_experts, MOE_ERR_INVALID, "ldd=%lld: need n_experts or more", (long long)ldd);
    MOE_NEED(T == 0 || (topk_idx && grad_w && dlogits), MOE_ERR_INVALID, "topk_idx / grad_w / dlogits is NULL");
    MOE_NEED(aligned4(topk_idx) && aligned4(grad_w) && aligned_el(dlogits, dtype), MOE_ERR_INVALID, "a buffer is not aligned to its elements");
    if (T == 0) return MOE_OK;
    const Rows ro(dlogits, T, ldd, n_experts, el_size(dtype));
    MOE_NEED(!overlap(ro, Rows(logits, T, ld, n_experts, el_size(dtype))) && !overlap(ro, Rows(topk_idx, (int64_t)T * top_k * 4)) &&
             !overlap(ro, Rows(grad_w, (int64_t)T * top_k * 4)), MOE_ERR_INVALID, "dlogits overlaps logits, topk_idx or grad_w");
    return launched(moe::launch_route_backward(logits, dtype, ld, T, n_experts, topk_idx, top_k, score_func == MOE_SCORE_SOFTMAX, norm_topk,
                                               routed_scale, grad_w, dlogits, ldd, accumulate != 0, static_cast<cudaStream_t>(stream)),
                    "moe_route_backward");
}

static const int32_t kMaxNorm = 16384;

static moe_status check_norm(int32_t dtype, int32_t stream_dtype, const void *weight, int32_t weight_dtype, int32_t T, int32_t width) {
    MOE_NEED(dtype_ok(dtype), MOE_ERR_INVALID, "dtype=%d: need a MOE_DTYPE_* value", dtype);
    MOE_NEED(stream_dtype == dtype || stream_dtype == MOE_DTYPE_F32, MOE_ERR_INVALID, "stream_dtype=%d: need dtype or MOE_DTYPE_F32", stream_dtype);
    MOE_NEED(!weight || weight_dtype == dtype || weight_dtype == MOE_DTYPE_F32, MOE_ERR_INVALID,
             "weight_dtype=%d: need dtype or MOE_DTYPE_F32", weight_dtype);
    MOE_NEED(T >= 0, MOE_ERR_INVALID, "T=%d is negative", T);
    MOE_NEED(width >= 1 && width <= kMaxNorm, MOE_ERR_UNSUPPORTED, "width=%d: need 1..%d", width, kMaxNorm);
    MOE_NEED(!weight || aligned_el(weight, weight_dtype), MOE_ERR_INVALID, "weight is not aligned to its elements");
    return MOE_OK;
}

moe_status moe_norm_forward(const void *x, int32_t dtype, int64_t ldx, const void *residual, int32_t stream_dtype, int64_t ldr,
                            const void *weight, int32_t weight_dtype, int32_t T, int32_t width, double eps, void *h, int64_t ldh,
                            void *y, int64_t ldy, float *rstd, uint8_t *codes, float *scales, void *stream) {
    if (!residual) stream_dtype = dtype;
    const moe_status s = check_norm(dtype, stream_dtype, weight, weight_dtype, T, width);
    if (s != MOE_OK) return s;
    MOE_NEED(isfinite(eps) && eps >= 0, MOE_ERR_INVALID, "eps: need a finite value, 0 or more");
    MOE_NEED((codes == nullptr) == (scales == nullptr), MOE_ERR_INVALID, "codes and scales: give both or neither");
    MOE_NEED(ldx >= width && (!residual || (ldr >= width && ldh >= width)) && (!y || ldy >= width), MOE_ERR_INVALID,
             "a row stride is less than width=%d", width);
    MOE_NEED(!codes || width % 16 == 0, MOE_ERR_UNSUPPORTED, "width=%d: need a multiple of 16 for codes", width);
    if (T == 0) return MOE_OK;
    MOE_NEED(x && (!residual || h), MOE_ERR_INVALID, "x / h is NULL");
    MOE_NEED(aligned_el(x, dtype) && aligned_el(residual, stream_dtype) && aligned_el(h, stream_dtype) && aligned_el(y, dtype) &&
             aligned4(rstd) && aligned4(scales), MOE_ERR_INVALID, "a buffer is not aligned to its elements");
    MOE_NEED(!codes || (aligned16(codes) && aligned_rows(x, ldx, dtype) && (!y || aligned_rows(y, ldy, dtype)) && aligned16(weight) &&
             (!residual || (aligned_rows(residual, ldr, stream_dtype) && aligned_rows(h, ldh, stream_dtype)))),
             MOE_ERR_INVALID, "with codes every row, weight and codes must start on a 16-byte boundary");
    const int64_t el = el_size(dtype), es = el_size(stream_dtype);
    const Rows rx(x, T, ldx, width, el), rr(residual, T, ldr, width, es), rh(residual ? h : nullptr, T, ldh, width, es), ry(y, T, ldy, width, el),
        rw(weight, width * el_size(weight_dtype)), rs(rstd, (int64_t)T * 4), rc(codes, (int64_t)T * width), rb(scales, (width + 127) / 128 * (int64_t)T * 4);
    // a row next to a scale's step is read again, from h or x, while others write y
    MOE_NEED(!askew(rh, rr) && !askew(rh, rx) && !askew(ry, rx) && !askew(ry, rr) && !askew(ry, rh) && (!codes || !overlap(ry, residual ? rh : rx)),
             MOE_ERR_INVALID, "h or y overlaps another tensor");
    for (const Rows *o : {&rs, &rc, &rb})
        for (const Rows *i : {&rx, &rr, &rh, &ry, &rw}) MOE_NEED(!overlap(*o, *i), MOE_ERR_INVALID, "rstd, codes or scales overlap another tensor");
    MOE_NEED(!overlap(rs, rc) && !overlap(rs, rb) && !overlap(rc, rb) && !overlap(rw, rh) && !overlap(rw, ry), MOE_ERR_INVALID, "two outputs, or weight and one, overlap");
    return launched(moe::launch_norm_forward(x, dtype, ldx, residual, stream_dtype, ldr, weight, weight_dtype, T, width, eps, h, ldh, y, ldy,
                                             rstd, codes, scales, static_cast<cudaStream_t>(stream)), "moe_norm_forward");
}

size_t moe_norm_workspace(int32_t T, int32_t width) {
    return T < 0 || width < 1 || width > kMaxNorm ? 0 : moe::norm_grad_workspace(T, width);
}

moe_status moe_norm_backward(const void *dy, int32_t dtype, int64_t lddy, const void *h, int32_t stream_dtype, int64_t ldh,
                             const float *rstd, const void *weight, int32_t weight_dtype, const void *grad_h, int64_t ldg, int32_t T,
                             int32_t width, void *dh, int64_t ldd, float *dweight, void *workspace, size_t workspace_bytes, void *stream) {
    const moe_status s = check_norm(dtype, stream_dtype, weight, weight_dtype, T, width);
    if (s != MOE_OK) return s;
    MOE_NEED(lddy >= width && ldh >= width && (!grad_h || ldg >= width) && ldd >= width, MOE_ERR_INVALID,
             "a row stride is less than width=%d", width);
    MOE_NEED(aligned4(dweight), MOE_ERR_INVALID, "dweight must be 4-byte aligned");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T == 0) return dweight ? launched(cudaMemsetAsync(dweight, 0, (size_t)width * 4, st), "moe_norm_backward") : MOE_OK;
    MOE_NEED(dy && h && rstd && dh, MOE_ERR_INVALID, "dy / h / rstd / dh is NULL");
    MOE_NEED(aligned_el(dy, dtype) && aligned_el(h, stream_dtype) && aligned_el(grad_h, stream_dtype) && aligned_el(dh, stream_dtype) &&
             aligned4(rstd), MOE_ERR_INVALID, "a buffer is not aligned to its elements");
    const size_t need = dweight ? moe_norm_workspace(T, width) : 0;
    MOE_NEED(need == 0 || (workspace && aligned16(workspace) && workspace_bytes >= need), MOE_ERR_INVALID,
             "workspace: need %zu bytes, 16-byte aligned", need);
    const int64_t el = el_size(dtype), es = el_size(stream_dtype);
    const Rows rd(dy, T, lddy, width, el), rh(h, T, ldh, width, es), rg(grad_h, T, ldg, width, es), ro(dh, T, ldd, width, es), rs(rstd, (int64_t)T * 4),
        rw(weight, width * el_size(weight_dtype)), rdw(dweight, (int64_t)width * 4), ws(need ? workspace : nullptr, (int64_t)need);
    MOE_NEED(!askew(ro, rd) && !askew(ro, rh) && !askew(ro, rg) && !overlap(ro, rs) && !overlap(ro, rw), MOE_ERR_INVALID, "dh overlaps another tensor");
    for (const Rows *i : {&rd, &rh, &rg, &ro, &rs, &rw, &rdw}) MOE_NEED(!overlap(ws, *i), MOE_ERR_INVALID, "workspace overlaps a tensor");
    MOE_NEED(!overlap(rdw, ro), MOE_ERR_INVALID, "dweight overlaps dh");
    return launched(moe::launch_norm_backward(dy, dtype, lddy, h, stream_dtype, ldh, rstd, weight, weight_dtype, grad_h, ldg, T, width, dh, ldd,
                                              dweight, workspace, st), "moe_norm_backward");
}

static moe_status check_combine(int32_t dtype, int64_t ld, int32_t R, int32_t N, int32_t T, int32_t top_k) {
    MOE_NEED(dtype_ok(dtype), MOE_ERR_INVALID, "dtype=%d: need a MOE_DTYPE_* value", dtype);
    MOE_NEED(T >= 0 && R >= 0, MOE_ERR_INVALID, "T=%d, R=%d: negative", T, R);
    MOE_NEED(N >= 1 && N <= kMaxWidth, MOE_ERR_UNSUPPORTED, "N=%d: need 1..%d", N, kMaxWidth);
    MOE_NEED(top_k >= 1 && top_k <= 32, MOE_ERR_UNSUPPORTED, "top_k=%d: need 1..32", top_k);
    MOE_NEED(ld >= N, MOE_ERR_INVALID, "ld=%lld: need N or more", (long long)ld);
    return MOE_OK;
}

moe_status moe_combine_forward(const void *rows, int32_t dtype, int64_t ld, int32_t R, int32_t N, const int32_t *pos, int32_t T,
                               int32_t top_k, const float *topk_w, const void *add, int64_t ldadd, void *y, int32_t y_dtype,
                               int64_t ldy, void *stream) {
    const moe_status s = check_combine(dtype, ld, R, N, T, top_k);
    if (s != MOE_OK) return s;
    MOE_NEED(dtype_ok(y_dtype), MOE_ERR_INVALID, "y_dtype=%d: need a MOE_DTYPE_* value", y_dtype);
    // a warp has 124 columns at least, seven before the row's first boundary among them: 2^30 blocks of 8 warps
    MOE_NEED((int64_t)T * ((N + 7 + 123) / 124) <= 1ll << 33, MOE_ERR_UNSUPPORTED, "T=%d: need 2^33 / ceil((N + 7) / 124) or fewer", T);
    MOE_NEED(ldy >= N && (!add || ldadd >= N), MOE_ERR_INVALID, "a row stride is less than N=%d", N);
    if (T == 0) return MOE_OK;
    MOE_NEED((rows || R == 0) && pos && y, MOE_ERR_INVALID, "rows / pos / y is NULL");
    MOE_NEED(aligned_el(rows, dtype) && aligned_el(add, y_dtype) && aligned_el(y, y_dtype) && aligned4(pos) && aligned4(topk_w),
             MOE_ERR_INVALID, "a buffer is not aligned to its elements");
    const Rows ry(y, T, ldy, N, el_size(y_dtype));
    MOE_NEED(!overlap(ry, Rows(rows, R, ld, N, el_size(dtype))) && !askew(ry, Rows(add, T, ldadd, N, el_size(y_dtype))) &&
             !overlap(ry, Rows(pos, (int64_t)T * top_k * 4)) && !overlap(ry, Rows(topk_w, (int64_t)T * top_k * 4)),
             MOE_ERR_INVALID, "y overlaps another tensor");
    return launched(moe::launch_combine_forward(rows, dtype, ld, R, N, pos, T, top_k, topk_w, add, ldadd, y, y_dtype, ldy,
                                                static_cast<cudaStream_t>(stream)), "moe_combine_forward");
}

moe_status moe_combine_backward(const void *dy, int32_t dtype, int64_t lddy, const void *rows, int64_t ld, int32_t R, int32_t N,
                                const int32_t *pos, int32_t T, int32_t top_k, const int32_t *tokens, const float *topk_w,
                                void *drows, int64_t ldd, float *dtopk_w, void *stream) {
    const moe_status s = check_combine(dtype, dtopk_w ? ld : N, R, N, T, top_k);
    if (s != MOE_OK) return s;
    MOE_NEED(T <= 1 << 30, MOE_ERR_UNSUPPORTED, "T=%d: need 2^30 or fewer", T);
    MOE_NEED(lddy >= N && (!drows || ldd >= N), MOE_ERR_INVALID, "a row stride is less than N=%d", N);
    MOE_NEED(T == 0 || (dy && pos), MOE_ERR_INVALID, "dy / pos is NULL");
    MOE_NEED(R == 0 || (tokens && (rows || !dtopk_w)), MOE_ERR_INVALID, "tokens / rows is NULL");
    MOE_NEED(aligned_el(dy, dtype) && aligned_el(rows, dtype) && aligned_el(drows, dtype) && aligned4(pos) && aligned4(tokens) &&
             aligned4(topk_w) && aligned4(dtopk_w), MOE_ERR_INVALID, "a buffer is not aligned to its elements");
    if ((T == 0 && (R == 0 || !drows)) || (!drows && !dtopk_w)) return MOE_OK;
    const int64_t el = el_size(dtype), pairs = (int64_t)T * top_k * 4;
    const Rows ro(drows, R, ldd, N, el), rdy(dy, T, lddy, N, el), rr(dtopk_w ? rows : nullptr, R, ld, N, el), rp(pos, pairs), rt(tokens, (int64_t)R * 4),
        rw(topk_w, pairs), rdw(dtopk_w, pairs);
    for (const Rows *i : {&rdy, &rr, &rp, &rt}) MOE_NEED(!overlap(ro, *i) && !overlap(rdw, *i), MOE_ERR_INVALID, "drows or dtopk_w overlaps another tensor");
    MOE_NEED(!overlap(ro, rw) && !overlap(ro, rdw) && !askew(rdw, rw), MOE_ERR_INVALID, "drows or dtopk_w overlaps another tensor");
    return launched(moe::launch_combine_backward(dy, dtype, lddy, rows, ld, R, N, pos, T, top_k, tokens, topk_w, drows, ldd, dtopk_w,
                                                 static_cast<cudaStream_t>(stream)), "moe_combine_backward");
}

static moe_status check_grads(int32_t n, const void *const *grads, const int32_t *dtypes, const int64_t *sizes, const float *norm) {
    MOE_NEED(n >= 0, MOE_ERR_INVALID, "n_tensors=%d is negative", n);
    MOE_NEED(n <= 65536, MOE_ERR_UNSUPPORTED, "n_tensors=%d: need 65536 or fewer", n);
    MOE_NEED(norm && aligned4(norm), MOE_ERR_INVALID, "norm is NULL or not 4-byte aligned");
    MOE_NEED(n == 0 || (grads && dtypes && sizes), MOE_ERR_INVALID, "grads / dtypes / sizes is NULL");
    int64_t all = 0;
    for (int32_t i = 0; i < n; i++) {
        MOE_NEED(dtype_ok(dtypes[i]), MOE_ERR_INVALID, "tensor %d: dtype=%d: need a MOE_DTYPE_* value", i, dtypes[i]);
        MOE_NEED(sizes[i] >= 0, MOE_ERR_INVALID, "tensor %d: size=%lld is negative", i, (long long)sizes[i]);
        MOE_NEED(sizes[i] <= (1ll << 45) - all, MOE_ERR_UNSUPPORTED, "more than 2^45 elements");
        MOE_NEED(sizes[i] == 0 || (grads[i] && aligned_el(grads[i], dtypes[i])), MOE_ERR_INVALID,
                 "tensor %d: NULL or not aligned to its elements", i);
        all += sizes[i];
    }
    return MOE_OK;
}

size_t moe_grad_norm_workspace(int32_t n_tensors) { return n_tensors < 0 || n_tensors > 65536 ? 0 : moe::grad_norm_workspace(n_tensors); }

moe_status moe_grad_norm(int32_t n_tensors, const void *const *grads, const int32_t *dtypes, const int64_t *sizes, float *norm,
                         void *workspace, size_t workspace_bytes, void *stream) {
    const moe_status s = check_grads(n_tensors, grads, dtypes, sizes, norm);
    if (s != MOE_OK) return s;
    const size_t need = moe_grad_norm_workspace(n_tensors);
    MOE_NEED(workspace && aligned16(workspace) && workspace_bytes >= need, MOE_ERR_INVALID, "workspace: need %zu bytes, 16-byte aligned", need);
    const Rows rn(norm, 4), rw(workspace, (int64_t)need);
    MOE_NEED(!overlap(rn, rw), MOE_ERR_INVALID, "norm and workspace overlap");
    for (int32_t i = 0; i < n_tensors; i++) {
        const Rows g(grads[i], sizes[i] * el_size(dtypes[i]));
        MOE_NEED(!overlap(g, rn) && !overlap(g, rw), MOE_ERR_INVALID, "norm or workspace overlaps tensor %d", i);
    }
    return launched(moe::launch_grad_norm(n_tensors, grads, dtypes, sizes, norm, workspace, static_cast<cudaStream_t>(stream)), "moe_grad_norm");
}

moe_status moe_grad_clip(int32_t n_tensors, const void *const *grads, const int32_t *dtypes, const int64_t *sizes, const float *norm,
                         float max_norm, void *const *out, void *stream) {
    const moe_status s = check_grads(n_tensors, grads, dtypes, sizes, norm);
    if (s != MOE_OK) return s;
    MOE_NEED(isfinite(max_norm) && max_norm >= 0, MOE_ERR_INVALID, "max_norm: need a finite value, 0 or more");
    void *const *to = out ? out : const_cast<void *const *>(reinterpret_cast<const void *const *>(grads));
    // no output on top of another tensor: ranges in order of their addresses, the written ones against all
    struct Range {
        uintptr_t a, b;
        int32_t tensor;
        bool written;
    };
    try {
        std::vector<Range> r;
        r.reserve(2 * (size_t)n_tensors + 1);
        const uintptr_t at = reinterpret_cast<uintptr_t>(norm);       // read by every block
        r.push_back({at, at + 4, n_tensors, false});
        for (int32_t i = 0; i < n_tensors; i++) {
            if (sizes[i] == 0) continue;
            const uintptr_t bytes = (uintptr_t)sizes[i] * (dtypes[i] == MOE_DTYPE_F32 ? 4 : 2);
            MOE_NEED(to[i] && aligned_el(to[i], dtypes[i]), MOE_ERR_INVALID, "output %d: NULL or not aligned to its elements", i);
            const uintptr_t a = reinterpret_cast<uintptr_t>(grads[i]), b = reinterpret_cast<uintptr_t>(to[i]);
            if (a != b) r.push_back({a, a + bytes, i, false});
            r.push_back({b, b + bytes, i, true});
        }
        std::sort(r.begin(), r.end(), [](const Range &x, const Range &y) { return x.a < y.a; });
        const Range *far = nullptr, *far_written = nullptr;       // the furthest end so far, of all and of the written ones
        for (const Range &q : r) {
            const Range *other = q.written ? far : far_written;
            MOE_NEED(!other || other->b <= q.a, MOE_ERR_INVALID, "tensors %d and %d overlap, and one of them is written (%d: norm)", other->tensor,
                     q.tensor, n_tensors);
            if (!far || q.b > far->b) far = &q;
            if (q.written && (!far_written || q.b > far_written->b)) far_written = &q;
        }
    } catch (const std::exception &) {
        return fail(MOE_ERR_NOMEM, "no host memory for %d tensors", n_tensors);
    }
    return launched(moe::launch_grad_clip(n_tensors, grads, dtypes, sizes, norm, max_norm, to, static_cast<cudaStream_t>(stream)), "moe_grad_clip");
}

moe_status moe_fp8_debug_stall_next_call(int32_t stages, int32_t block) {
    MOE_NEED(stages >= 0, MOE_ERR_INVALID, "stages=%d is negative", stages);
    MOE_NEED(block >= 0 && block < 8, MOE_ERR_INVALID, "block=%d: need 0..7", block);
    moe::fp8_stall_next(stages, block);
    return MOE_OK;
}

moe_status moe_fp8_device_error(uint32_t *flags) {
    MOE_NEED(flags, MOE_ERR_INVALID, "flags is NULL");
    *flags = 0;
    unsigned f = 0;
    const cudaError_t e = moe::fp8_error_read(&f);
    if (e != cudaSuccess) return cuda_fail(e, "reading the device error word");
    *flags = f;
    MOE_NEED(f == 0, MOE_ERR_CUDA, "device error word 0x%x: a pipeline wait of a block-scaled product ran out", f);
    return MOE_OK;
}

#undef MOE_NEED

}  // extern "C"
