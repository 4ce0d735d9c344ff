// C ABI of the selective-scan library: argument validation, launch planning
// and dispatch. Declarations and the contract are in include/mambascan.h.
#include <cuda_runtime.h>

#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <numeric>

#include <nvtx3/nvToolsExt.h>

#include "launch.h"
#include "mambascan.h"

namespace {

// An NVTX range named after the entry point for the duration of the call, so
// that profilers (ncu --nvtx, nsys) can attribute the launches; without a
// profiler attached the push and pop return at once.
struct CallRange {
    explicit CallRange(const char *name) { nvtxRangePushA(name); }
    ~CallRange() { nvtxRangePop(); }
    CallRange(const CallRange &) = delete;
    CallRange &operator=(const CallRange &) = delete;
};

thread_local char g_last_error[512] = "";

void set_error(const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_last_error, sizeof g_last_error, fmt, ap);
    va_end(ap);
}

ms_status invalid(const char *what) {
    set_error("invalid argument: %s", what);
    return MS_ERR_INVALID_ARG;
}

ms_status cuda_fail(cudaError_t e, const char *where) {
    set_error("%s: %s", where, cudaGetErrorString(e));
    return MS_ERR_CUDA;
}

// Number of SMs of the current device, cached per device.
constexpr int kMaxDevices = 64;
int g_sms[kMaxDevices] = {0};
std::mutex g_sms_mu;

ms_status device_sms(int *out) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    if (dev >= 0 && dev < kMaxDevices) {
        std::lock_guard<std::mutex> lk(g_sms_mu);
        if (g_sms[dev] == 0) {
            int sms = 0;
            e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
            if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute");
            g_sms[dev] = sms;
        }
        *out = g_sms[dev];
        return MS_OK;
    }
    int sms = 0;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute");
    *out = sms;
    return MS_OK;
}

bool elem_aligned(const void *ptr, int eb) {
    return (reinterpret_cast<uintptr_t>(ptr) % static_cast<uintptr_t>(eb)) == 0;
}

ms_status check_scan(const ms_scan_args *a) {
    if (!a) return invalid("args is NULL");
    if (a->batch <= 0 || a->dim <= 0 || a->dstate <= 0 || a->seqlen <= 0)
        return invalid("batch, dim, dstate and seqlen must be positive");
    if (a->in_dtype != MS_F32 && a->in_dtype != MS_BF16) return invalid("in_dtype");
    if (a->reserved != 0) return invalid("reserved must be 0");
    if (a->force_segments < 0) return invalid("force_segments must be >= 0");
    if (!a->u || !a->delta || !a->B || !a->C || !a->A || !a->y)
        return invalid("u, delta, B, C, A and y are required");
    if (a->u_batch_stride < 0 || a->u_dim_stride < 0 || a->delta_batch_stride < 0 ||
        a->delta_dim_stride < 0 || a->B_batch_stride < 0 || a->B_state_stride < 0 ||
        a->C_batch_stride < 0 || a->C_state_stride < 0 || a->y_batch_stride < 0 ||
        a->y_dim_stride < 0 || (a->z && (a->z_batch_stride < 0 || a->z_dim_stride < 0)))
        return invalid("strides must be non-negative");
    if (a->dstate > MS_MAX_DSTATE) {
        set_error("dstate %lld exceeds the supported maximum %d", static_cast<long long>(a->dstate),
                  MS_MAX_DSTATE);
        return MS_ERR_UNSUPPORTED;
    }
    if (a->batch > 65535) {
        set_error("batch %lld exceeds 65535", static_cast<long long>(a->batch));
        return MS_ERR_UNSUPPORTED;
    }
    const int eb = a->in_dtype == MS_F32 ? 4 : 2;
    if (!elem_aligned(a->u, eb) || !elem_aligned(a->delta, eb) || !elem_aligned(a->B, eb) ||
        !elem_aligned(a->C, eb) || !elem_aligned(a->y, eb) || (a->z && !elem_aligned(a->z, eb)) ||
        !elem_aligned(a->A, 4) || (a->D && !elem_aligned(a->D, 4)) ||
        (a->delta_bias && !elem_aligned(a->delta_bias, 4)) ||
        (a->initial_state && !elem_aligned(a->initial_state, 4)) ||
        (a->final_state && !elem_aligned(a->final_state, 4))) {
        set_error("a pointer is not aligned to its element size");
        return MS_ERR_ALIGNMENT;
    }
    return MS_OK;
}

ms::ScanParams to_params(const ms_scan_args *a) {
    ms::ScanParams p{};
    p.batch = a->batch; p.dim = a->dim; p.dstate = a->dstate; p.seqlen = a->seqlen;
    p.u = a->u; p.u_sb = a->u_batch_stride; p.u_sd = a->u_dim_stride;
    p.delta = a->delta; p.dl_sb = a->delta_batch_stride; p.dl_sd = a->delta_dim_stride;
    p.B = a->B; p.B_sb = a->B_batch_stride; p.B_sn = a->B_state_stride;
    p.C = a->C; p.C_sb = a->C_batch_stride; p.C_sn = a->C_state_stride;
    p.z = a->z; p.z_sb = a->z_batch_stride; p.z_sd = a->z_dim_stride;
    p.y = a->y; p.y_sb = a->y_batch_stride; p.y_sd = a->y_dim_stride;
    p.A = a->A; p.D = a->D; p.delta_bias = a->delta_bias;
    p.h0 = a->initial_state; p.hT = a->final_state;
    p.softplus = a->delta_softplus ? 1 : 0;
    return p;
}

ms_status check_conv(const ms_conv1d_args *c) {
    if (!c) return invalid("conv is NULL");
    if (!c->weight) return invalid("conv weight is required");
    if (c->silu != 0 && c->silu != 1) return invalid("conv silu must be 0 or 1");
    if (c->width < 1) return invalid("conv width must be >= 1");
    if (c->width > MS_MAX_CONV_WIDTH) {
        set_error("conv width %d exceeds the supported maximum %d", c->width, MS_MAX_CONV_WIDTH);
        return MS_ERR_UNSUPPORTED;
    }
    if (!elem_aligned(c->weight, 4) || (c->bias && !elem_aligned(c->bias, 4))) {
        set_error("conv weight or bias is not aligned to 4 bytes");
        return MS_ERR_ALIGNMENT;
    }
    return MS_OK;
}

// Validate a decode call and fill its kernel parameters.
ms_status update_params(const ms_update_args *a, ms::UpdateParams *p) {
    if (!a) return invalid("args is NULL");
    if (a->batch <= 0 || a->dim <= 0 || a->dstate <= 0)
        return invalid("batch, dim and dstate must be positive");
    if (a->in_dtype != MS_F32 && a->in_dtype != MS_BF16) return invalid("in_dtype");
    if (!a->state || !a->x || !a->delta || !a->B || !a->C || !a->A || !a->y)
        return invalid("state, x, delta, B, C, A and y are required");
    if (a->state_batch_stride < 0 || a->state_dim_stride < 0 || a->x_batch_stride < 0 ||
        a->delta_batch_stride < 0 || a->B_batch_stride < 0 || a->C_batch_stride < 0 ||
        a->y_batch_stride < 0 || (a->z && a->z_batch_stride < 0))
        return invalid("strides must be non-negative");
    if (a->dstate > MS_MAX_DSTATE) {
        set_error("dstate %lld exceeds the supported maximum %d", static_cast<long long>(a->dstate),
                  MS_MAX_DSTATE);
        return MS_ERR_UNSUPPORTED;
    }
    if (a->batch > 65535) {
        set_error("batch %lld exceeds 65535", static_cast<long long>(a->batch));
        return MS_ERR_UNSUPPORTED;
    }
    const int eb = a->in_dtype == MS_F32 ? 4 : 2;
    if (!elem_aligned(a->state, 4) || !elem_aligned(a->x, eb) || !elem_aligned(a->delta, eb) ||
        !elem_aligned(a->B, eb) || !elem_aligned(a->C, eb) || !elem_aligned(a->y, eb) ||
        (a->z && !elem_aligned(a->z, eb)) || !elem_aligned(a->A, 4) ||
        (a->D && !elem_aligned(a->D, 4)) || (a->delta_bias && !elem_aligned(a->delta_bias, 4))) {
        set_error("a pointer is not aligned to its element size");
        return MS_ERR_ALIGNMENT;
    }
    *p = ms::UpdateParams{};
    p->batch = a->batch; p->dim = a->dim; p->dstate = a->dstate;
    p->state = a->state; p->s_sb = a->state_batch_stride; p->s_sd = a->state_dim_stride;
    p->x = a->x; p->x_sb = a->x_batch_stride;
    p->delta = a->delta; p->dl_sb = a->delta_batch_stride;
    p->B = a->B; p->B_sb = a->B_batch_stride;
    p->C = a->C; p->C_sb = a->C_batch_stride;
    p->z = a->z; p->z_sb = a->z_batch_stride;
    p->y = a->y; p->y_sb = a->y_batch_stride;
    p->A = a->A; p->D = a->D; p->delta_bias = a->delta_bias;
    p->softplus = a->delta_softplus ? 1 : 0;
    return MS_OK;
}

ms_status run_plan(ms::ScanParams p, const ms::ScanPlan &plan, int in_dtype, void *workspace,
                   size_t workspace_bytes, void *stream) {
    if (plan.ws_bytes > 0) {
        if (!workspace || workspace_bytes < plan.ws_bytes) {
            set_error("workspace of %zu bytes needed, %zu given", plan.ws_bytes,
                      workspace ? workspace_bytes : static_cast<size_t>(0));
            return MS_ERR_WORKSPACE;
        }
        if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) {
            set_error("workspace must be 256-byte aligned");
            return MS_ERR_ALIGNMENT;
        }
    }
    ms::bind_workspace(p, plan, workspace);
    const cudaError_t e = ms::launch_scan(p, plan, in_dtype, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "scan kernel launch");
    return MS_OK;
}

}  // namespace

namespace ms {
void record_error(const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_last_error, sizeof g_last_error, fmt, ap);
    va_end(ap);
}
}  // namespace ms

extern "C" {

const char *mamba_status_string(int status) {
    switch (status) {
        case MS_OK: return "MS_OK";
        case MS_ERR_INVALID_ARG: return "MS_ERR_INVALID_ARG";
        case MS_ERR_UNSUPPORTED: return "MS_ERR_UNSUPPORTED";
        case MS_ERR_ALIGNMENT: return "MS_ERR_ALIGNMENT";
        case MS_ERR_CUDA: return "MS_ERR_CUDA";
        case MS_ERR_TIMEOUT: return "MS_ERR_TIMEOUT";
        case MS_ERR_WORKSPACE: return "MS_ERR_WORKSPACE";
        default: return "MS_UNKNOWN_STATUS";
    }
}

const char *mamba_last_error(void) { return g_last_error; }

int mamba_abi_version(void) { return MAMBASCAN_ABI_VERSION; }

ms_status mamba_scan_workspace_size(const ms_scan_args *args, size_t *bytes) {
    if (!bytes) return invalid("bytes is NULL");
    *bytes = 0;
    ms_status st = check_scan(args);
    if (st != MS_OK) return st;
    int sms = 0;
    st = device_sms(&sms);
    if (st != MS_OK) return st;
    const ms::ScanParams p = to_params(args);
    *bytes = ms::plan_scan(p, args->in_dtype, args->force_segments, sms).ws_bytes;
    return MS_OK;
}

ms_status mamba_scan_fwd(const ms_scan_args *args, void *workspace, size_t workspace_bytes,
                         void *stream) {
    const CallRange range("mamba_scan_fwd");
    ms_status st = check_scan(args);
    if (st != MS_OK) return st;
    int sms = 0;
    st = device_sms(&sms);
    if (st != MS_OK) return st;
    const ms::ScanParams p = to_params(args);
    const ms::ScanPlan plan = ms::plan_scan(p, args->in_dtype, args->force_segments, sms);
    return run_plan(p, plan, args->in_dtype, workspace, workspace_bytes, stream);
}

int mamba_scan_num_configs(void) { return ms::scan_num_configs(); }

ms_status mamba_scan_config_info(int config, int *lanes, int *states_per_pass, int *max_warps) {
    if (!ms::scan_config_info(config, lanes, states_per_pass, max_warps)) return invalid("unknown config");
    return MS_OK;
}

ms_status mamba_scan_config_kind(int config, int *kind) {
    if (!kind) return invalid("kind is NULL");
    *kind = ms::scan_config_kind(config);
    if (*kind < 0) return invalid("unknown config");
    return MS_OK;
}

ms_status mamba_scan_plan_query(const ms_scan_args *args, ms_scan_plan *plan) {
    if (!plan) return invalid("plan is NULL");
    ms_status st = check_scan(args);
    if (st != MS_OK) return st;
    int sms = 0;
    st = device_sms(&sms);
    if (st != MS_OK) return st;
    const ms::ScanPlan pl = ms::plan_scan(to_params(args), args->in_dtype, args->force_segments, sms);
    plan->config = pl.config;
    plan->warps_per_cta = pl.warps;
    plan->segments = pl.nseg;
    plan->lanes = pl.lg;
    plan->segment_len = pl.seg_len;
    plan->workspace_bytes = pl.ws_bytes;
    plan->ctas = pl.ctas;
    plan->reserved = 0;
    return MS_OK;
}

ms_status mamba_scan_plan_workspace_size(const ms_scan_args *args, const ms_scan_plan *plan, size_t *bytes) {
    if (!bytes) return invalid("bytes is NULL");
    *bytes = 0;
    if (!plan) return invalid("plan is NULL");
    ms_status st = check_scan(args);
    if (st != MS_OK) return st;
    int sms = 0;
    st = device_sms(&sms);
    if (st != MS_OK) return st;
    ms::ScanPlan pl{};
    if (!ms::make_plan(to_params(args), args->in_dtype, plan->config, plan->warps_per_cta, plan->segments,
                       plan->ctas, sms, &pl)) {
        set_error("plan (config %d, %d warps, %d segments, %d CTAs) cannot run these arguments", plan->config,
                  plan->warps_per_cta, plan->segments, plan->ctas);
        return MS_ERR_UNSUPPORTED;
    }
    *bytes = pl.ws_bytes;
    return MS_OK;
}

ms_status mamba_scan_fwd_with_plan(const ms_scan_args *args, const ms_scan_plan *plan, void *workspace,
                                   size_t workspace_bytes, void *stream) {
    const CallRange range("mamba_scan_fwd_with_plan");
    if (!plan) return invalid("plan is NULL");
    ms_status st = check_scan(args);
    if (st != MS_OK) return st;
    const ms::ScanParams p = to_params(args);
    int sms = 0;
    st = device_sms(&sms);
    if (st != MS_OK) return st;
    ms::ScanPlan pl{};
    if (plan->reserved != 0 ||
        !ms::make_plan(p, args->in_dtype, plan->config, plan->warps_per_cta, plan->segments, plan->ctas, sms, &pl)) {
        set_error("plan (config %d, %d warps, %d segments, %d CTAs) cannot run these arguments", plan->config,
                  plan->warps_per_cta, plan->segments, plan->ctas);
        return MS_ERR_UNSUPPORTED;
    }
    return run_plan(p, pl, args->in_dtype, workspace, workspace_bytes, stream);
}

ms_status mamba_state_update(const ms_update_args *a, void *stream) {
    const CallRange range("mamba_state_update");
    ms::UpdateParams p;
    const ms_status st = update_params(a, &p);
    if (st != MS_OK) return st;
    const cudaError_t e = ms::launch_state_update(p, a->in_dtype, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "state update kernel launch");
    return MS_OK;
}

ms_status mamba_conv_state_update(const ms_update_args *a, const ms_conv1d_args *conv, void *conv_state,
                                  int64_t conv_state_batch_stride, int64_t conv_state_dim_stride,
                                  void *stream) {
    const CallRange range("mamba_conv_state_update");
    ms::UpdateParams p;
    ms_status st = update_params(a, &p);
    if (st != MS_OK) return st;
    st = check_conv(conv);
    if (st != MS_OK) return st;
    if (!conv_state) return invalid("conv_state is required");
    if (conv_state_batch_stride < 0 || conv_state_dim_stride < 0)
        return invalid("conv_state strides must be non-negative");
    if (!elem_aligned(conv_state, a->in_dtype == MS_F32 ? 4 : 2)) {
        set_error("conv_state is not aligned to its element size");
        return MS_ERR_ALIGNMENT;
    }
    p.conv_state = conv_state;
    p.cs_sb = conv_state_batch_stride;
    p.cs_sd = conv_state_dim_stride;
    p.conv_w = conv->weight;
    p.conv_b = conv->bias;
    p.conv_width = conv->width;
    p.conv_silu = conv->silu;
    const cudaError_t e = ms::launch_state_update(p, a->in_dtype, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "state update kernel launch");
    return MS_OK;
}

static ms_status conv_scan_impl(const ms_scan_args *args, const ms_conv1d_args *conv, const ms_scan_plan *plan,
                                void *workspace, size_t workspace_bytes, void *stream, bool with_workspace,
                                size_t *query) {
    ms_status st = check_scan(args);
    if (st != MS_OK) return st;
    st = check_conv(conv);
    if (st != MS_OK) return st;
    if (args->force_segments > 1) {
        set_error("the convolution prologue runs in one segment (force_segments %d)", args->force_segments);
        return MS_ERR_UNSUPPORTED;
    }
    ms::ScanParams p = to_params(args);
    p.conv_w = conv->weight;
    p.conv_b = conv->bias;
    p.conv_width = conv->width;
    p.conv_silu = conv->silu;
    int sms = 0;
    st = device_sms(&sms);
    if (st != MS_OK) return st;
    ms::ScanPlan pl{};
    if (plan) {
        if ((!with_workspace && plan->ctas != 0) || plan->reserved != 0 ||
            !ms::make_plan(p, args->in_dtype, plan->config, plan->warps_per_cta, plan->segments, plan->ctas, sms,
                           &pl)) {
            set_error("plan (config %d, %d warps, %d segments, %d CTAs) cannot run the convolution prologue",
                      plan->config, plan->warps_per_cta, plan->segments, plan->ctas);
            return MS_ERR_UNSUPPORTED;
        }
    } else {
        pl = ms::plan_scan(p, args->in_dtype, 0, sms, with_workspace);
        if (pl.kind != 1) {
            set_error("no kernel configuration fuses the convolution prologue for these arguments");
            return MS_ERR_UNSUPPORTED;
        }
    }
    if (query) {
        *query = pl.ws_bytes;
        return MS_OK;
    }
    return run_plan(p, pl, args->in_dtype, workspace, workspace_bytes, stream);
}

ms_status mamba_conv_scan_fwd(const ms_scan_args *args, const ms_conv1d_args *conv, const ms_scan_plan *plan,
                              void *stream) {
    const CallRange range("mamba_conv_scan_fwd");
    return conv_scan_impl(args, conv, plan, nullptr, 0, stream, false, nullptr);
}

ms_status mamba_conv_scan_workspace_size(const ms_scan_args *args, const ms_conv1d_args *conv,
                                         const ms_scan_plan *plan, size_t *bytes) {
    if (!bytes) return invalid("bytes is NULL");
    *bytes = 0;
    return conv_scan_impl(args, conv, plan, nullptr, 0, nullptr, true, bytes);
}

ms_status mamba_conv_scan_fwd_ws(const ms_scan_args *args, const ms_conv1d_args *conv, const ms_scan_plan *plan,
                                 void *workspace, size_t workspace_bytes, void *stream) {
    const CallRange range("mamba_conv_scan_fwd_ws");
    return conv_scan_impl(args, conv, plan, workspace, workspace_bytes, stream, true, nullptr);
}

static ms_status trap_scan_impl(const ms_scan_args *args, const void *lambda_raw, int64_t lambda_batch_stride,
                                int64_t lambda_dim_stride, const ms_scan_plan *plan, void *workspace,
                                size_t workspace_bytes, void *stream, bool with_workspace, size_t *query) {
    ms_status st = check_scan(args);
    if (st != MS_OK) return st;
    if (!lambda_raw) return invalid("lambda_raw is required");
    if (lambda_batch_stride < 0 || lambda_dim_stride < 0) return invalid("lambda strides must be non-negative");
    if (!elem_aligned(lambda_raw, args->in_dtype == MS_F32 ? 4 : 2)) {
        set_error("lambda_raw is not aligned to its element size");
        return MS_ERR_ALIGNMENT;
    }
    if (args->force_segments > 1) {
        set_error("the trapezoidal rule runs in one segment (force_segments %d)", args->force_segments);
        return MS_ERR_UNSUPPORTED;
    }
    ms::ScanParams p = to_params(args);
    p.lambda_raw = lambda_raw;
    p.lm_sb = lambda_batch_stride;
    p.lm_sd = lambda_dim_stride;
    int sms = 0;
    st = device_sms(&sms);
    if (st != MS_OK) return st;
    ms::ScanPlan pl{};
    if (plan) {
        if ((!with_workspace && plan->ctas != 0) || plan->reserved != 0 ||
            !ms::make_plan(p, args->in_dtype, plan->config, plan->warps_per_cta, plan->segments, plan->ctas, sms,
                           &pl)) {
            set_error("plan (config %d, %d warps, %d segments, %d CTAs) cannot run the trapezoidal rule",
                      plan->config, plan->warps_per_cta, plan->segments, plan->ctas);
            return MS_ERR_UNSUPPORTED;
        }
    } else {
        pl = ms::plan_scan(p, args->in_dtype, 0, sms, with_workspace);
        if (pl.kind != 1) {
            set_error("no kernel configuration runs the trapezoidal rule for these arguments");
            return MS_ERR_UNSUPPORTED;
        }
    }
    if (query) {
        *query = pl.ws_bytes;
        return MS_OK;
    }
    return run_plan(p, pl, args->in_dtype, workspace, workspace_bytes, stream);
}

ms_status mamba_trap_scan_fwd(const ms_scan_args *args, const void *lambda_raw, int64_t lambda_batch_stride,
                              int64_t lambda_dim_stride, const ms_scan_plan *plan, void *stream) {
    const CallRange range("mamba_trap_scan_fwd");
    return trap_scan_impl(args, lambda_raw, lambda_batch_stride, lambda_dim_stride, plan, nullptr, 0, stream, false,
                          nullptr);
}

ms_status mamba_trap_scan_workspace_size(const ms_scan_args *args, const void *lambda_raw,
                                         int64_t lambda_batch_stride, int64_t lambda_dim_stride,
                                         const ms_scan_plan *plan, size_t *bytes) {
    if (!bytes) return invalid("bytes is NULL");
    *bytes = 0;
    return trap_scan_impl(args, lambda_raw, lambda_batch_stride, lambda_dim_stride, plan, nullptr, 0, nullptr, true,
                          bytes);
}

ms_status mamba_trap_scan_fwd_ws(const ms_scan_args *args, const void *lambda_raw, int64_t lambda_batch_stride,
                                 int64_t lambda_dim_stride, const ms_scan_plan *plan, void *workspace,
                                 size_t workspace_bytes, void *stream) {
    const CallRange range("mamba_trap_scan_fwd_ws");
    return trap_scan_impl(args, lambda_raw, lambda_batch_stride, lambda_dim_stride, plan, workspace,
                          workspace_bytes, stream, true, nullptr);
}

ms_status mamba_scan_bwd_workspace_size(const ms_scan_args *args, size_t *bytes) {
    if (!bytes) return invalid("bytes is NULL");
    *bytes = 0;
    const ms_status st = check_scan(args);
    if (st != MS_OK) return st;
    *bytes = ms::bwd_workspace_bytes(to_params(args));
    return MS_OK;
}

static ms_status scan_bwd_impl(const ms_scan_args *args, const ms_scan_bwd_args *g, void *workspace,
                               size_t workspace_bytes, void *stream, int ckpt_ready) {
    ms_status st = check_scan(args);
    if (st != MS_OK) return st;
    if (!g) return invalid("bwd is NULL");
    if (args->seqlen > (int64_t(1) << 30)) return invalid("seqlen above 2^30 is not supported by the backward");
    if (!g->dy || !g->du || !g->ddelta || !g->dA || !g->dB || !g->dC)
        return invalid("dy, du, ddelta, dA, dB and dC are required");
    if ((args->z && !g->dz) || (args->D && !g->dD) || (args->delta_bias && !g->ddelta_bias))
        return invalid("dz, dD and ddelta_bias are required when z, D and delta_bias are given");
    if (g->dy_batch_stride < 0 || g->dy_dim_stride < 0 || g->du_batch_stride < 0 || g->du_dim_stride < 0 ||
        g->ddelta_batch_stride < 0 || g->ddelta_dim_stride < 0 ||
        (g->dz && (g->dz_batch_stride < 0 || g->dz_dim_stride < 0)))
        return invalid("gradient strides must be non-negative");
    const int eb = args->in_dtype == MS_F32 ? 4 : 2;
    if (!elem_aligned(g->dy, eb) || !elem_aligned(g->du, eb) || !elem_aligned(g->ddelta, eb) ||
        (g->dz && !elem_aligned(g->dz, eb)) || !elem_aligned(g->dA, 4) || !elem_aligned(g->dB, 4) ||
        !elem_aligned(g->dC, 4) || (g->dD && !elem_aligned(g->dD, 4)) ||
        (g->ddelta_bias && !elem_aligned(g->ddelta_bias, 4)) ||
        (g->dfinal_state && !elem_aligned(g->dfinal_state, 4)) ||
        (g->dinitial_state && !elem_aligned(g->dinitial_state, 4))) {
        set_error("a gradient pointer is not aligned to its element size");
        return MS_ERR_ALIGNMENT;
    }
    const ms::ScanParams p = to_params(args);
    const size_t need = ms::bwd_workspace_bytes(p);
    if (!workspace || workspace_bytes < need) {
        set_error("%s of %zu bytes needed, %zu given", ckpt_ready ? "checkpoints" : "workspace", need,
                  workspace ? workspace_bytes : static_cast<size_t>(0));
        return MS_ERR_WORKSPACE;
    }
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) {
        set_error("workspace must be 256-byte aligned");
        return MS_ERR_ALIGNMENT;
    }
    ms::BwdParams q{};
    q.dy = g->dy; q.dy_sb = g->dy_batch_stride; q.dy_sd = g->dy_dim_stride;
    q.dhT = g->dfinal_state;
    q.du = g->du; q.du_sb = g->du_batch_stride; q.du_sd = g->du_dim_stride;
    q.ddelta = g->ddelta; q.dd_sb = g->ddelta_batch_stride; q.dd_sd = g->ddelta_dim_stride;
    q.dz = g->dz; q.dz_sb = g->dz_batch_stride; q.dz_sd = g->dz_dim_stride;
    q.dA = g->dA; q.dB = g->dB; q.dC = g->dC; q.dD = g->dD; q.dbias = g->ddelta_bias;
    q.dh0 = g->dinitial_state;
    q.ckpt = static_cast<float *>(workspace);
    q.ckpt_ready = ckpt_ready;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const size_t bc = static_cast<size_t>(args->batch * args->dstate * args->seqlen) * sizeof(float);
    cudaError_t e = cudaMemsetAsync(g->dA, 0, static_cast<size_t>(args->dim * args->dstate) * sizeof(float), s);
    if (e == cudaSuccess) e = cudaMemsetAsync(g->dB, 0, bc, s);
    if (e == cudaSuccess) e = cudaMemsetAsync(g->dC, 0, bc, s);
    if (e == cudaSuccess && g->dD) e = cudaMemsetAsync(g->dD, 0, static_cast<size_t>(args->dim) * sizeof(float), s);
    if (e == cudaSuccess && g->ddelta_bias)
        e = cudaMemsetAsync(g->ddelta_bias, 0, static_cast<size_t>(args->dim) * sizeof(float), s);
    if (e != cudaSuccess) return cuda_fail(e, "clearing the gradient accumulators");
    e = ms::launch_bwd(p, q, args->in_dtype, s);
    if (e != cudaSuccess) return cuda_fail(e, "backward kernel launch");
    return MS_OK;
}

ms_status mamba_scan_bwd(const ms_scan_args *args, const ms_scan_bwd_args *g, void *workspace,
                         size_t workspace_bytes, void *stream) {
    const CallRange range("mamba_scan_bwd");
    return scan_bwd_impl(args, g, workspace, workspace_bytes, stream, 0);
}

ms_status mamba_scan_bwd_checkpointed(const ms_scan_args *args, const ms_scan_bwd_args *g,
                                      const float *checkpoints, size_t checkpoint_bytes, void *stream) {
    const CallRange range("mamba_scan_bwd_checkpointed");
    if (!checkpoints) return invalid("checkpoints is NULL");
    return scan_bwd_impl(args, g, const_cast<float *>(checkpoints), checkpoint_bytes, stream, 1);
}

ms_status mamba_scan_fwd_checkpointed(const ms_scan_args *args, float *checkpoints, size_t checkpoint_bytes,
                                      void *workspace, size_t workspace_bytes, void *stream) {
    const CallRange range("mamba_scan_fwd_checkpointed");
    ms_status st = check_scan(args);
    if (st != MS_OK) return st;
    if (!checkpoints) return invalid("checkpoints is NULL");
    const ms::ScanParams p0 = to_params(args);
    const size_t need = ms::bwd_workspace_bytes(p0);
    if (checkpoint_bytes < need) {
        set_error("checkpoints of %zu bytes needed, %zu given", need, checkpoint_bytes);
        return MS_ERR_WORKSPACE;
    }
    if ((reinterpret_cast<uintptr_t>(checkpoints) & 255u) != 0) {
        set_error("checkpoints must be 256-byte aligned");
        return MS_ERR_ALIGNMENT;
    }
    int sms = 0;
    st = device_sms(&sms);
    if (st != MS_OK) return st;
    ms::ScanParams p = p0;
    p.ckpt = checkpoints;   // (the planner then considers the sequential kernels only)
    const ms::ScanPlan plan = ms::plan_scan(p, args->in_dtype, args->force_segments, sms);
    if (plan.kind != 1) {
        set_error("checkpoints are written by the sequential kernels only, which run no forced segments");
        return MS_ERR_UNSUPPORTED;
    }
    return run_plan(p, plan, args->in_dtype, workspace, workspace_bytes, stream);
}

static ms_status check_ssd(const ms_ssd_args *a) {
    if (!a) return invalid("args is NULL");
    if (a->batch <= 0 || a->seqlen <= 0 || a->nheads <= 0 || a->ngroups <= 0)
        return invalid("batch, seqlen, nheads and ngroups must be positive");
    if (a->nheads % a->ngroups != 0) return invalid("nheads must be a multiple of ngroups");
    if (!a->x || !a->dt || !a->B || !a->C || !a->y || !a->A) return invalid("x, dt, B, C, y and A are required");
    if (a->in_dtype != MS_BF16) {
        if (a->in_dtype != MS_F32) return invalid("unknown in_dtype");
        set_error("the SSD kernel takes bf16 inputs only");
        return MS_ERR_UNSUPPORTED;
    }
    if (a->seqlen > (int64_t(1) << 30) || a->batch * a->nheads > (int64_t(1) << 30))
        return invalid("seqlen or batch * nheads too large");
    const int64_t strides[] = {a->x_batch_stride, a->x_token_stride, a->dt_batch_stride, a->dt_token_stride,
                               a->B_batch_stride, a->B_token_stride, a->C_batch_stride, a->C_token_stride,
                               a->y_batch_stride, a->y_token_stride, a->z_batch_stride, a->z_token_stride};
    for (int i = 0; i < (a->z ? 12 : 10); ++i)
        if (strides[i] < 0) return invalid("strides must be non-negative");
    if (a->x_token_stride < a->nheads * MS_SSD_HEADDIM || a->y_token_stride < a->nheads * MS_SSD_HEADDIM ||
        (a->z && a->z_token_stride < a->nheads * MS_SSD_HEADDIM))
        return invalid("the token stride of x, y and z must cover nheads * 64 elements");
    if (a->B_token_stride < a->ngroups * MS_SSD_DSTATE || a->C_token_stride < a->ngroups * MS_SSD_DSTATE)
        return invalid("the token stride of B and C must cover ngroups * 128 elements");
    if (a->dt_token_stride < a->nheads) return invalid("the token stride of dt must cover nheads elements");
    for (int i : {0, 1, 4, 5, 6, 7, 8, 9}) {
        if (strides[i] % 8 != 0) {
            set_error("batch and token strides of x, y, B, C (and z) must be multiples of 8 elements");
            return MS_ERR_ALIGNMENT;
        }
    }
    if (a->z && (a->z_batch_stride % 8 != 0 || a->z_token_stride % 8 != 0)) {
        set_error("batch and token strides of x, y, B, C (and z) must be multiples of 8 elements");
        return MS_ERR_ALIGNMENT;
    }
    if (!elem_aligned(a->x, 16) || !elem_aligned(a->B, 16) || !elem_aligned(a->C, 16) || !elem_aligned(a->y, 16) ||
        (a->z && !elem_aligned(a->z, 16)) || !elem_aligned(a->dt, 2) || !elem_aligned(a->A, 4) ||
        (a->D && !elem_aligned(a->D, 4)) || (a->dt_bias && !elem_aligned(a->dt_bias, 4)) ||
        (a->initial_state && !elem_aligned(a->initial_state, 4)) ||
        (a->final_state && !elem_aligned(a->final_state, 4))) {
        set_error("x, y, B, C and z must be 16-byte aligned, the other pointers aligned to their elements");
        return MS_ERR_ALIGNMENT;
    }
    if (a->withhold_block < 0) return invalid("withhold_block must be >= 0");
    return MS_OK;
}

// CTAs of the persistent schedule the call would take (0: one CTA per (batch, head)).
static ms_status ssd_plan_ctas(const ms_ssd_args *a, int *ctas) {
    int sms = 0;
    const ms_status st = device_sms(&sms);
    if (st != MS_OK) return st;
    *ctas = ms::ssd_persistent_ctas(a->batch, a->nheads, a->seqlen, sms);
    return MS_OK;
}

ms_status mamba_ssd_workspace_size(const ms_ssd_args *a, size_t *bytes) {
    if (!bytes) return invalid("bytes is NULL");
    *bytes = 0;
    ms_status st = check_ssd(a);
    if (st != MS_OK) return st;
    int ctas = 0;
    st = ssd_plan_ctas(a, &ctas);
    if (st != MS_OK) return st;
    *bytes = ctas ? ms::ssd_persistent_ws_bytes(ctas) : static_cast<size_t>(MS_SSD_WORKSPACE_BYTES);
    return MS_OK;
}

ms_status mamba_ssd_fwd(const ms_ssd_args *a, void *workspace, size_t workspace_bytes, void *stream) {
    const CallRange range("mamba_ssd_fwd");
    ms_status st = check_ssd(a);
    if (st != MS_OK) return st;
    if (!workspace || workspace_bytes < MS_SSD_WORKSPACE_BYTES) {
        set_error("workspace of %d bytes needed, %zu given", MS_SSD_WORKSPACE_BYTES,
                  workspace ? workspace_bytes : static_cast<size_t>(0));
        return MS_ERR_WORKSPACE;
    }
    if (!elem_aligned(workspace, 16)) {
        set_error("workspace must be 16-byte aligned");
        return MS_ERR_ALIGNMENT;
    }
    ms::SsdParams p{};
    p.x = a->x; p.x_sb = a->x_batch_stride; p.x_st = a->x_token_stride;
    p.dt = a->dt; p.dt_sb = a->dt_batch_stride; p.dt_st = a->dt_token_stride;
    p.B = a->B; p.B_sb = a->B_batch_stride; p.B_st = a->B_token_stride;
    p.C = a->C; p.C_sb = a->C_batch_stride; p.C_st = a->C_token_stride;
    p.z = a->z; p.z_sb = a->z_batch_stride; p.z_st = a->z_token_stride;
    p.y = a->y; p.y_sb = a->y_batch_stride; p.y_st = a->y_token_stride;
    p.A = a->A; p.D = a->D; p.dt_bias = a->dt_bias; p.h0 = a->initial_state; p.hT = a->final_state;
    p.batch = a->batch; p.seqlen = a->seqlen; p.nheads = a->nheads; p.ngroups = a->ngroups;
    p.softplus = a->dt_softplus ? 1 : 0;
    p.status = static_cast<int *>(workspace);
    p.wait_limit_ns = a->wait_limit_us ? 1000ull * a->wait_limit_us : 1000000000ull;
    p.withhold_block = a->withhold_block;
    int ctas = 0;
    st = ssd_plan_ctas(a, &ctas);
    if (st != MS_OK) return st;
    if (ctas > 0 && workspace_bytes >= ms::ssd_persistent_ws_bytes(ctas)) {
        p.sk_ctas = ctas;
        p.sk_flag = reinterpret_cast<int *>(static_cast<char *>(workspace) + ms::ssd_flag_offset());
        p.sk_carry = reinterpret_cast<float *>(static_cast<char *>(workspace) + ms::ssd_carry_offset(ctas));
    }
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = ms::launch_ssd(p, s);
    if (e == cudaErrorNotSupported) {
        set_error("the driver offers no tensor-map encoder");
        return MS_ERR_UNSUPPORTED;
    }
    if (e != cudaSuccess) return cuda_fail(e, "SSD kernel launch");
    return MS_OK;
}

// ---- Mamba-2 serving operators and norms --------------------------------------

static ms_status misaligned(const char *what) {
    set_error("%s", what);
    return MS_ERR_ALIGNMENT;
}

static ms_status unsupported(const char *what) {
    set_error("%s", what);
    return MS_ERR_UNSUPPORTED;
}

// Element size of an ms_dtype, 0 for an unknown one.
static int dtype_bytes(int dtype) { return dtype == MS_F32 ? 4 : dtype == MS_BF16 ? 2 : 0; }

// Rows of packed tensors and cache slots are counted in 32 bits on the device.
static const int64_t kMaxRows = (int64_t(1) << 31) - 1;

// Whether two tensors of `rows` rows of `width` elements of eb bytes share an element; row strides in elements.
// Exact for one stride (and one row); with two, rows that lie apart only by their numbers count as shared.
static bool rows_overlap(const void *a, int64_t sa, const void *b, int64_t sb, int64_t rows, int64_t width, int eb) {
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
    const __int128 d = (static_cast<__int128>(pb) - static_cast<__int128>(pa)), last = rows - 1;
    if (d >= (last * sa + width) * eb || -d >= (last * sb + width) * eb) return false;   // one behind the other
    if (rows == 1) return true;
    // where the rows begin, modulo what both strides are multiples of
    const __int128 period = static_cast<__int128>(std::gcd(sa, sb)) * eb, w = static_cast<__int128>(width) * eb;
    const __int128 r = ((d % period) + period) % period;
    return r < w || period - r < w;
}

// The checks that the packed calls share: counts, the cache and its index table.
static ms_status check_slots(int64_t nseq, int64_t slots, const void *state, const int32_t *idx,
                             const uint8_t *has_init, bool need_state) {
    if (nseq < 0 || slots < 0 || nseq > kMaxRows || slots > kMaxRows) return invalid("nseq or slots out of range");
    if (!state && need_state && (idx || has_init))
        return invalid("state_indices and has_initial_state need a state");
    if (state && !idx && slots < nseq) return invalid("without state_indices there must be a slot for every sequence");
    if (idx && !elem_aligned(idx, 4)) return misaligned("state_indices is not aligned to 4 bytes");
    return MS_OK;
}

ms_status mamba_conv_packed_fwd(const ms_conv_packed_args *a, const ms_conv1d_args *c, void *stream) {
    const CallRange range("mamba_conv_packed_fwd");
    if (!a) return invalid("args is NULL");
    ms_status st = check_conv(c);
    if (st != MS_OK) return st;
    const int eb = dtype_bytes(a->in_dtype);
    if (!eb) return invalid("in_dtype");
    if (a->reserved != 0) return invalid("reserved must be 0");
    if (a->tokens < 0 || a->tokens > kMaxRows - 64 || a->channels <= 0 || a->channels > (int64_t(1) << 22))
        return invalid("tokens must be in [0, 2^31 - 65] and channels in [1, 2^22]");
    const bool stateful = a->state != nullptr && c->width > 1;
    st = check_slots(a->nseq, a->slots, a->state, a->state_indices, a->has_initial_state, c->width > 1);
    if (st != MS_OK) return st;
    if (!a->cu_seqlens && (a->tokens != a->nseq || a->has_initial_state))
        return invalid("single tokens: tokens must equal nseq and has_initial_state be NULL");
    if (!a->cu_seqlens && c->width > 1 && !a->state) return invalid("single tokens need a state");
    if (a->nseq > (int64_t(1) << 30)) return invalid("nseq above 2^30");
    if (a->tokens > 0 && (!a->x || !a->y)) return invalid("x and y are required");
    if (a->tokens > 0 && a->x == a->y) return invalid("the convolution is not computed in place: y must not be x");
    if (a->x_token_stride < 0 || a->y_token_stride < a->channels ||
        (stateful && (a->state_slot_stride < 0 || a->state_row_stride < a->channels)))
        return invalid("strides must be non-negative and those of y and the state rows cover the channels");
    if (a->tokens > 0 &&
        rows_overlap(a->x, a->x_token_stride, a->y, a->y_token_stride, a->tokens, a->channels, eb))
        return invalid("y must not overlap x");
    if (stateful && a->slots > 1 && a->state_slot_stride < a->state_row_stride * (c->width - 1))
        return invalid("the state's slot stride must cover its rows");
    if (!elem_aligned(a->x, eb) || !elem_aligned(a->y, eb) || (stateful && !elem_aligned(a->state, eb)) ||
        !elem_aligned(a->cu_seqlens, 4))
        return misaligned("a pointer is not aligned to its element size");
    if (a->nseq == 0) return MS_OK;   // nothing to read or write
    int sms = 0;
    st = device_sms(&sms);
    if (st != MS_OK) return st;
    ms::ConvPackedParams p{};
    p.tokens = a->tokens; p.channels = a->channels; p.nseq = a->nseq;
    p.slots = a->state || a->state_indices ? a->slots : a->nseq;
    p.x = a->x; p.x_st = a->x_token_stride;
    p.y = a->y; p.y_st = a->y_token_stride;
    if (stateful) { p.state = a->state; p.st_slot = a->state_slot_stride; p.st_row = a->state_row_stride; }
    p.cu = a->cu_seqlens; p.idx = a->state_indices; p.has_init = a->has_initial_state;
    p.weight = c->weight; p.bias = c->bias; p.width = c->width; p.silu = c->silu;
    const cudaError_t e = ms::launch_conv_packed(p, a->in_dtype, sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MS_OK : cuda_fail(e, "packed convolution launch");
}

ms_status mamba_ssd_state_update(const ms_ssd_update_args *a, void *stream) {
    const CallRange range("mamba_ssd_state_update");
    if (!a) return invalid("args is NULL");
    const int eb = dtype_bytes(a->in_dtype);
    if (!eb) return invalid("in_dtype");
    if (a->batch < 0 || a->nheads <= 0 || a->ngroups <= 0 || a->headdim <= 0 || a->dstate <= 0)
        return invalid("batch must not be negative, nheads, ngroups, headdim and dstate must be positive");
    if (a->nheads % a->ngroups != 0) return invalid("nheads must be a multiple of ngroups");
    if (a->dstate > MS_SSD_UPDATE_MAX_DSTATE) return unsupported("dstate above 256");
    if (a->batch > 65535) return unsupported("batch above 65535");
    if (a->nheads > 65535 || a->headdim > 65535 || a->nheads * a->headdim > (int64_t(1) << 30))
        return unsupported("nheads or headdim above 65535, or their product above 2^30");
    ms_status st = check_slots(a->batch, a->slots, a->state, a->state_indices, nullptr, true);
    if (st != MS_OK) return st;
    if (a->batch == 0) return MS_OK;
    if (!a->state || !a->x || !a->dt || !a->B || !a->C || !a->y || !a->A)
        return invalid("state, x, dt, B, C, y and A are required");
    const int64_t per = a->nheads * a->headdim;
    if (a->x_batch_stride < 0 || a->dt_batch_stride < 0 || a->B_batch_stride < 0 || a->C_batch_stride < 0 ||
        (a->z && a->z_batch_stride < 0))
        return invalid("strides must be non-negative");
    if ((a->batch > 1 && a->y_batch_stride < per) || (a->slots > 1 && a->state_slot_stride < per * a->dstate))
        return invalid("the strides of y and of the state's slots must cover their entries");
    if (!elem_aligned(a->x, eb) || !elem_aligned(a->dt, eb) || !elem_aligned(a->B, eb) || !elem_aligned(a->C, eb) ||
        (a->z && !elem_aligned(a->z, eb)) || !elem_aligned(a->y, eb) || !elem_aligned(a->state, 4) ||
        !elem_aligned(a->A, 4) || (a->D && !elem_aligned(a->D, 4)) || (a->dt_bias && !elem_aligned(a->dt_bias, 4)))
        return misaligned("a pointer is not aligned to its element size");
    ms::SsdUpdateParams p{};
    p.batch = a->batch; p.slots = a->slots;
    p.nheads = static_cast<int>(a->nheads); p.hpg = static_cast<int>(a->nheads / a->ngroups);
    p.headdim = static_cast<int>(a->headdim); p.dstate = static_cast<int>(a->dstate);
    p.state = a->state; p.s_slot = a->state_slot_stride;
    p.x = a->x; p.x_sb = a->x_batch_stride;
    p.dt = a->dt; p.dt_sb = a->dt_batch_stride;
    p.B = a->B; p.B_sb = a->B_batch_stride;
    p.C = a->C; p.C_sb = a->C_batch_stride;
    p.z = a->z; p.z_sb = a->z_batch_stride;
    p.y = a->y; p.y_sb = a->y_batch_stride;
    p.A = a->A; p.D = a->D; p.dt_bias = a->dt_bias;
    p.idx = a->state_indices;
    p.softplus = a->dt_softplus ? 1 : 0;
    const cudaError_t e = ms::launch_ssd_update(p, a->in_dtype, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MS_OK : cuda_fail(e, "SSD state update launch");
}

static ms_status check_ssd_packed(const ms_ssd_packed_args *a) {
    if (!a) return invalid("args is NULL");
    if (a->nheads <= 0 || a->ngroups <= 0) return invalid("nheads and ngroups must be positive");
    if (a->nheads % a->ngroups != 0) return invalid("nheads must be a multiple of ngroups");
    if (a->reserved != 0) return invalid("reserved must be 0");
    if (a->in_dtype != MS_BF16) {
        if (a->in_dtype != MS_F32) return invalid("unknown in_dtype");
        return unsupported("the SSD kernel takes bf16 inputs only");
    }
    if (a->tokens < 0 || a->tokens > kMaxRows - 64 * 1024 || a->max_seqlen < 0)
        return invalid("tokens must be in [0, 2^31 - 2^16) and max_seqlen not negative");
    if (a->nheads > 65535) return unsupported("nheads above 65535");
    const ms_status st = check_slots(a->nseq, a->slots, a->state, a->state_indices, a->has_initial_state, true);
    if (st != MS_OK) return st;
    if (a->nseq > (int64_t(1) << 27) || a->nseq * a->nheads > (int64_t(1) << 27) ||
        (a->tokens / 256 + a->nseq) * a->nheads > kMaxRows)
        return unsupported("too many sequences or segments times heads for one launch");
    if (a->nseq == 0) return MS_OK;
    if (!a->cu_seqlens || !a->A) return invalid("cu_seqlens and A are required");
    if (a->tokens > 0 && (!a->x || !a->dt || !a->B || !a->C || !a->y)) return invalid("x, dt, B, C and y are required");
    if (a->tokens > 0) {
        const int64_t xi = a->nheads * MS_SSD_HEADDIM, bi = a->ngroups * MS_SSD_DSTATE;
        if (a->x_token_stride < xi || a->y_token_stride < xi || (a->z && a->z_token_stride < xi))
            return invalid("the token stride of x, y and z must cover nheads * 64 elements");
        if (a->B_token_stride < bi || a->C_token_stride < bi)
            return invalid("the token stride of B and C must cover ngroups * 128 elements");
        if (a->dt_token_stride < a->nheads) return invalid("the token stride of dt must cover nheads elements");
        if (a->x_token_stride % 8 || a->y_token_stride % 8 || a->B_token_stride % 8 || a->C_token_stride % 8 ||
            (a->z && a->z_token_stride % 8))
            return misaligned("token strides of x, y, B, C (and z) must be multiples of 8 elements");
        if (a->x_token_stride >= (int64_t(1) << 38) || a->B_token_stride >= (int64_t(1) << 38) ||
            a->C_token_stride >= (int64_t(1) << 38))
            return unsupported("a token stride of 2^38 elements or more");
    }
    if (a->state && (a->state_slot_stride < 0 ||
                     (a->slots > 1 && a->state_slot_stride < a->nheads * MS_SSD_HEADDIM * MS_SSD_DSTATE)))
        return invalid("the state's slot stride must cover its heads");
    if (!elem_aligned(a->x, 16) || !elem_aligned(a->B, 16) || !elem_aligned(a->C, 16) || !elem_aligned(a->y, 16) ||
        (a->z && !elem_aligned(a->z, 16)) || !elem_aligned(a->dt, 2) || !elem_aligned(a->A, 4) ||
        (a->D && !elem_aligned(a->D, 4)) || (a->dt_bias && !elem_aligned(a->dt_bias, 4)) ||
        (a->state && !elem_aligned(a->state, 4)) || !elem_aligned(a->cu_seqlens, 4))
        return misaligned("x, y, B, C and z must be 16-byte aligned, the other pointers aligned to their elements");
    return MS_OK;
}

static ms_status ssd_packed_plan(const ms_ssd_packed_args *a, ms::SsdPackedPlan *plan) {
    int sms = 0;
    const ms_status st = device_sms(&sms);
    if (st != MS_OK) return st;
    *plan = ms::ssd_packed_plan(a->tokens, a->nseq, a->nheads, a->ngroups, a->max_seqlen, sms);
    return MS_OK;
}

ms_status mamba_ssd_packed_workspace_size(const ms_ssd_packed_args *a, size_t *bytes) {
    if (!bytes) return invalid("bytes is NULL");
    *bytes = 0;
    ms_status st = check_ssd_packed(a);
    if (st != MS_OK) return st;
    ms::SsdPackedPlan plan{};
    st = ssd_packed_plan(a, &plan);
    if (st != MS_OK) return st;
    *bytes = ms::ssd_packed_ws_bytes(a->tokens, a->nseq, a->nheads, plan.seg_chunks);
    return MS_OK;
}

ms_status mamba_ssd_packed_fwd(const ms_ssd_packed_args *a, void *workspace, size_t workspace_bytes, void *stream) {
    const CallRange range("mamba_ssd_packed_fwd");
    ms_status st = check_ssd_packed(a);
    if (st != MS_OK) return st;
    ms::SsdPackedPlan plan{};
    st = ssd_packed_plan(a, &plan);
    if (st != MS_OK) return st;
    const size_t need = ms::ssd_packed_ws_bytes(a->tokens, a->nseq, a->nheads, plan.seg_chunks);
    if (!workspace || workspace_bytes < need) {
        set_error("workspace of %zu bytes needed, %zu given", need, workspace ? workspace_bytes : static_cast<size_t>(0));
        return MS_ERR_WORKSPACE;
    }
    if (!elem_aligned(workspace, 256)) return misaligned("workspace must be 256-byte aligned");
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (a->nseq == 0) {
        const cudaError_t e = cudaMemsetAsync(workspace, 0, sizeof(int), s);
        return e == cudaSuccess ? MS_OK : cuda_fail(e, "clearing the status word");
    }
    ms::SsdPackedParams p{};
    p.tokens = a->tokens; p.nseq = a->nseq; p.nheads = a->nheads; p.ngroups = a->ngroups; p.slots = a->slots;
    p.x = a->x; p.x_st = a->x_token_stride;
    p.dt = a->dt; p.dt_st = a->dt_token_stride;
    p.B = a->B; p.B_st = a->B_token_stride;
    p.C = a->C; p.C_st = a->C_token_stride;
    p.z = a->z; p.z_st = a->z_token_stride;
    p.y = a->y; p.y_st = a->y_token_stride;
    p.A = a->A; p.D = a->D; p.dt_bias = a->dt_bias;
    p.state = a->state; p.s_slot = a->state_slot_stride;
    p.cu = a->cu_seqlens; p.idx = a->state_indices; p.has_init = a->has_initial_state;
    p.softplus = a->dt_softplus ? 1 : 0;
    p.wait_limit_ns = a->wait_limit_us ? 1000ull * a->wait_limit_us : 1000000000ull;
    p.seg_chunks = plan.seg_chunks; p.each = plan.each;
    ms::ssd_packed_bind(p, workspace);
    const cudaError_t e = ms::launch_ssd_packed(p, s);
    if (e == cudaErrorNotSupported) return unsupported("the driver offers no tensor-map encoder");
    return e == cudaSuccess ? MS_OK : cuda_fail(e, "packed SSD launch");
}

ms_status mamba_ssd_packed_failures(uint64_t *count, void *stream) {
    if (!count) return invalid("count is NULL");
    unsigned long long n = 0;
    const cudaError_t e = ms::ssd_packed_failures(&n, static_cast<cudaStream_t>(stream));
    *count = n;
    return e == cudaSuccess ? MS_OK : cuda_fail(e, "reading the count of failures");
}

// What the forward and the backward norm share.
static ms_status check_norm(const ms_norm_args *a) {
    if (!a) return invalid("args is NULL");
    if (!dtype_bytes(a->in_dtype)) return invalid("in_dtype");
    if (a->reserved != 0) return invalid("reserved must be 0");
    if (a->rows < 0 || a->dim <= 0 || a->group_size <= 0) return invalid("rows, dim or group_size out of range");
    if (a->dim % a->group_size != 0) return invalid("dim must be a multiple of group_size");
    if (a->dim > (int64_t(1) << 30) || a->rows > kMaxRows || a->rows * (a->dim / a->group_size) > kMaxRows)
        return unsupported("dim above 2^30 or rows times groups above 2^31 - 1");
    if (!(a->eps >= 0.f) || a->eps > 3e38f) return invalid("eps must be finite and not negative");
    if (a->gate_first != 0 && a->gate_first != 1) return invalid("gate_first must be 0 or 1");
    if ((a->residual || a->residual_out) &&
        (!dtype_bytes(a->residual_dtype) || (a->in_dtype == MS_F32 && a->residual_dtype != MS_F32)))
        return invalid("residual_dtype must be in_dtype or MS_F32");
    if (a->x_row_stride < 0 || (a->z && a->z_row_stride < 0) || (a->residual && a->residual_row_stride < 0))
        return invalid("strides must be non-negative");
    const int eb = dtype_bytes(a->in_dtype), rb = dtype_bytes(a->residual_dtype);
    if ((a->x && !elem_aligned(a->x, eb)) || (a->z && !elem_aligned(a->z, eb)) ||
        (a->residual && !elem_aligned(a->residual, rb)) || (a->residual_out && !elem_aligned(a->residual_out, rb)) ||
        (a->weight && !elem_aligned(a->weight, 4)))
        return misaligned("a pointer is not aligned to its element size");
    return MS_OK;
}

static ms::NormParams norm_params(const ms_norm_args *a) {
    ms::NormParams p{};
    p.rows = a->rows; p.dim = a->dim; p.gs = a->group_size; p.groups = a->dim / a->group_size;
    p.x = a->x; p.x_sr = a->x_row_stride;
    p.z = a->z; p.z_sr = a->z_row_stride;
    p.res = a->residual; p.res_sr = a->residual_row_stride;
    p.ro = a->residual_out; p.ro_sr = a->residual_out_row_stride;
    p.y = a->y; p.y_sr = a->y_row_stride;
    p.w = a->weight;
    p.eps = a->eps; p.scale = a->residual_scale;
    p.inv_gs = 1.f / static_cast<float>(a->group_size);
    p.gate_first = a->gate_first;
    return p;
}

ms_status mamba_norm_fwd(const ms_norm_args *a, void *stream) {
    const CallRange range("mamba_norm_fwd");
    ms_status st = check_norm(a);
    if (st != MS_OK) return st;
    if (a->rows == 0) return MS_OK;
    if (!a->x || !a->y) return invalid("x and y are required");
    if ((a->residual != nullptr) != (a->residual_out != nullptr))
        return invalid("residual and residual_out are given together");
    if (a->rows > 1 && (a->y_row_stride < a->dim || (a->residual_out && a->residual_out_row_stride < a->dim)))
        return invalid("the row strides of y and residual_out must cover dim elements");
    if (!elem_aligned(a->y, dtype_bytes(a->in_dtype))) return misaligned("a pointer is not aligned to its element size");
    const cudaError_t e = ms::launch_norm_fwd(norm_params(a), a->in_dtype,
                                              a->residual ? a->residual_dtype : a->in_dtype,
                                              static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MS_OK : cuda_fail(e, "norm launch");
}

static ms_status norm_slabs(const ms_norm_args *a, int64_t *slabs) {
    int sms = 0;
    const ms_status st = device_sms(&sms);
    if (st != MS_OK) return st;
    *slabs = ms::norm_bwd_slabs(a->rows, a->dim, a->group_size, sms);
    return MS_OK;
}

ms_status mamba_norm_bwd_workspace_size(const ms_norm_args *a, size_t *bytes) {
    if (!bytes) return invalid("bytes is NULL");
    *bytes = 0;
    ms_status st = check_norm(a);
    if (st != MS_OK) return st;
    if (a->rows == 0) return MS_OK;
    int64_t slabs = 0;
    st = norm_slabs(a, &slabs);
    if (st != MS_OK) return st;
    *bytes = slabs > 1 ? static_cast<size_t>(slabs) * static_cast<size_t>(a->dim) * sizeof(float) : 0;
    return MS_OK;
}

ms_status mamba_norm_bwd(const ms_norm_args *a, const ms_norm_bwd_args *g, void *workspace, size_t workspace_bytes,
                         void *stream) {
    const CallRange range("mamba_norm_bwd");
    ms_status st = check_norm(a);
    if (st != MS_OK) return st;
    if (!g) return invalid("bwd is NULL");
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (g->dweight && !elem_aligned(g->dweight, 4)) return misaligned("dweight is not aligned to 4 bytes");
    if (a->rows == 0) {
        if (!g->dweight) return MS_OK;
        const cudaError_t e = cudaMemsetAsync(g->dweight, 0, static_cast<size_t>(a->dim) * sizeof(float), s);
        return e == cudaSuccess ? MS_OK : cuda_fail(e, "clearing dweight");
    }
    const bool res = a->residual_out != nullptr;
    const int eb = dtype_bytes(a->in_dtype), rb = res ? dtype_bytes(a->residual_dtype) : 4;
    const bool need_x = !res || (a->z && a->gate_first);
    if (!g->dy || !g->dx || (need_x && !a->x) || (a->z && !g->dz) || (res && !g->dresidual))
        return invalid("dy and dx are required, x, dz with z and dresidual with a residual too");
    if (!res && (g->dresidual || g->dresidual_out)) return invalid("residual gradients need residual_out");
    if (g->dy_row_stride < 0 || (g->dresidual_out && g->dresidual_out_row_stride < 0) ||
        (res && a->residual_out_row_stride < 0))
        return invalid("strides must be non-negative");
    if (a->rows > 1 && (g->dx_row_stride < a->dim || (a->z && g->dz_row_stride < a->dim) ||
                        (res && g->dresidual_row_stride < a->dim)))
        return invalid("the row strides of dx, dz and dresidual must cover dim elements");
    if (!elem_aligned(g->dy, eb) || !elem_aligned(g->dx, eb) || (a->z && !elem_aligned(g->dz, eb)) ||
        (res && !elem_aligned(g->dresidual, rb)) || (g->dresidual_out && !elem_aligned(g->dresidual_out, rb)))
        return misaligned("a gradient pointer is not aligned to its element size");
    int64_t slabs = 0;
    st = norm_slabs(a, &slabs);
    if (st != MS_OK) return st;
    ms::NormBwdParams q{};
    q.dy = g->dy; q.dy_sr = g->dy_row_stride;
    q.dro = g->dresidual_out; q.dro_sr = g->dresidual_out_row_stride;
    q.dx = g->dx; q.dx_sr = g->dx_row_stride;
    q.dz = a->z ? g->dz : nullptr; q.dz_sr = g->dz_row_stride;
    q.dres = g->dresidual; q.dres_sr = g->dresidual_row_stride;
    q.dw = g->dweight;
    q.slabs = slabs;
    if (g->dweight) {
        if (slabs == 1) {
            q.partial = g->dweight;
        } else {
            const size_t need = static_cast<size_t>(slabs) * static_cast<size_t>(a->dim) * sizeof(float);
            if (!workspace || workspace_bytes < need) {
                set_error("workspace of %zu bytes needed, %zu given", need,
                          workspace ? workspace_bytes : static_cast<size_t>(0));
                return MS_ERR_WORKSPACE;
            }
            if (!elem_aligned(workspace, 16)) return misaligned("workspace must be 16-byte aligned");
            q.partial = static_cast<float *>(workspace);
        }
    }
    const cudaError_t e = ms::launch_norm_bwd(norm_params(a), q, a->in_dtype, res ? a->residual_dtype : a->in_dtype, s);
    return e == cudaSuccess ? MS_OK : cuda_fail(e, "norm backward launch");
}

}  // extern "C"
