// Host side of the paged-cache calls declared in include/fadkv.h: argument
// checks and launches.  No device memory is allocated.
#include <math.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <atomic>

#include "paged.cuh"

using namespace fadkv;

namespace {

std::atomic<uint64_t> g_wait_ns{0};    // fadkv_debug_paged_wait_limit

bool aligned(const void* ptr, size_t a) { return ((uintptr_t)ptr % a) == 0; }

fadkv_status cuda_error(const char* where, cudaError_t e)
{
    char msg[256];
    snprintf(msg, sizeof(msg), "%s: %s (%d)", where, cudaGetErrorString(e), (int)e);
    set_last_error(msg);
    return FADKV_ERR_CUDA;
}

// FADKV_FAULT=cuda: as for the other calls, fails before anything is launched.
bool fault_injected()
{
    const char* f = getenv("FADKV_FAULT");
    return f && strcmp(f, "cuda") == 0;
}

int log2_exact(int v)
{
    int s = 0;
    while ((1 << s) < v && s < 30) ++s;
    return s;
}

bool page_size_ok(int ps) { return ps >= 8 && ps <= 1024 && (ps & (ps - 1)) == 0; }

bool stride_ok(int64_t s, int64_t least) { return s >= least && s % 8 == 0 && s < ((int64_t)1 << 38); }

// Pool shape: sizes and strides.
fadkv_status check_pool(int page_size, int num_pages, int d, int64_t page_stride, int64_t head_stride,
                        int64_t token_stride)
{
    if (num_pages < 0) return FADKV_ERR_INVALID_ARG;
    if (!page_size_ok(page_size) || (int64_t)num_pages * page_size > 0x7fffffffll) return FADKV_ERR_UNSUPPORTED;
    if (num_pages > 0 && (!stride_ok(page_stride, d) || !stride_ok(head_stride, d) || !stride_ok(token_stride, d)))
        return FADKV_ERR_INVALID_ARG;
    return FADKV_OK;
}

fadkv_status check_paged(const fadkv_paged_params* p)
{
    if (!p) return FADKV_ERR_INVALID_ARG;
    if (p->B < 0 || p->T < 0 || p->Hq < 1 || p->Hkv < 1 || p->Hq % p->Hkv != 0 || p->max_pages < 1 ||
        p->num_pages < 1 ||
        p->window < 0 || p->sinks < 0 || !isfinite(p->scale))
        return FADKV_ERR_INVALID_ARG;
    if (p->dtype != FADKV_F16 && p->dtype != FADKV_F32 && p->dtype != FADKV_BF16) return FADKV_ERR_INVALID_ARG;
    if (p->dtype == FADKV_F32 || (p->d != 64 && p->d != 128) || p->B > FADKV_MAX_REQUESTS || p->Hq > 4096)
        return FADKV_ERR_UNSUPPORTED;
    const fadkv_status st =
        check_pool(p->page_size, p->num_pages, p->d, p->page_stride, p->head_stride, p->token_stride);
    if (st != FADKV_OK) return st;
    if ((int64_t)p->max_pages * p->page_size > 0x7fffffffll - 4096) return FADKV_ERR_UNSUPPORTED;
    if (!stride_ok(p->q_stride, (int64_t)p->Hq * p->d) || !stride_ok(p->out_stride, (int64_t)p->Hq * p->d))
        return FADKV_ERR_INVALID_ARG;
    return FADKV_OK;
}

PagedArgs paged_args(const fadkv_paged_params& p, const void* k, const void* v, const int32_t* table,
                     const int32_t* lengths, const int32_t* starts, const int32_t* positions, const void* q, void* out,
                     float* lse, void* ws)
{
    PagedArgs a;
    a.p = p;
    a.shift = log2_exact(p.page_size);
    a.grp = p.Hq / p.Hkv;
    a.split = 0;
    a.wait_ns = g_wait_ns.load(std::memory_order_relaxed);
    a.tile_ns = 0;
    a.scale_log2 = p.scale * 1.44269504088896f;
    a.k = k;
    a.v = v;
    a.table = table;
    a.lengths = lengths;
    a.starts = starts;
    a.positions = positions;
    a.q = q;
    a.out = out;
    a.lse = lse;
    a.ws = ws;
    return a;
}

bool dtype_ok(int t) { return t == FADKV_F16 || t == FADKV_F32 || t == FADKV_BF16; }

}  // namespace

extern "C" {

fadkv_status fadkv_page_plan(const fadkv_page_params* p, const int32_t* add, const int32_t* lengths,
                             int32_t* block_table, int32_t* free_pages, const int32_t* free_count,
                             int32_t* lengths_out, int32_t* free_count_out, int32_t* starts, int32_t* positions,
                             int32_t* slots, int32_t* refused, void* stream)
{
    if (!p || p->B < 0 || p->num_pages < 0 || p->max_pages < 1 || p->max_tokens < 0) return FADKV_ERR_INVALID_ARG;
    if (!page_size_ok(p->page_size) || (int64_t)p->num_pages * p->page_size > 0x7fffffffll ||
        (int64_t)p->max_pages * p->page_size > 0x7fffffffll - 4096 || p->B > FADKV_MAX_REQUESTS)
        return FADKV_ERR_UNSUPPORTED;
    if (!free_count || !free_count_out || !starts || !refused || (p->num_pages > 0 && !free_pages) ||
        (p->max_tokens > 0 && (!positions || !slots)) ||
        (p->B > 0 && (!add || !lengths || !block_table || !lengths_out)))
        return FADKV_ERR_INVALID_ARG;
    const void* all[] = {add, lengths, block_table, free_pages, free_count, lengths_out, free_count_out, starts,
                         positions, slots, refused};
    for (const void* ptr : all)
        if (!aligned(ptr, 4)) return FADKV_ERR_INVALID_ARG;
    if (fault_injected()) return cuda_error("fadkv_page_plan", cudaErrorLaunchFailure);
    PlanArgs a;
    a.B = p->B;
    a.shift = log2_exact(p->page_size);
    a.num_pages = p->num_pages;
    a.max_pages = p->max_pages;
    a.max_tokens = p->max_tokens;
    a.add = add;
    a.lengths = lengths;
    a.table = block_table;
    a.free_pages = free_pages;
    a.free_count = free_count;
    a.lengths_out = lengths_out;
    a.free_count_out = free_count_out;
    a.starts = starts;
    a.positions = positions;
    a.slots = slots;
    a.refused = refused;
    const cudaError_t e = launch_page_plan(a, (cudaStream_t)stream);
    return e == cudaSuccess ? FADKV_OK : cuda_error("fadkv_page_plan", e);
}

fadkv_status fadkv_rope_init(const fadkv_rope_params* p, fadkv_rope* out)
{
    if (!p || !out) return FADKV_ERR_INVALID_ARG;
    if (p->rotary_dim < 0 || p->rotary_dim > p->d || !(p->base > 1.0) || !isfinite(p->base) ||
        !isfinite((float)p->amplitude) || p->scaling < FADKV_ROPE_PLAIN || p->scaling > FADKV_ROPE_PARTS)
        return FADKV_ERR_INVALID_ARG;
    if ((p->d != 64 && p->d != 128) || p->rotary_dim % 16 != 0) return FADKV_ERR_UNSUPPORTED;
    if (p->scaling != FADKV_ROPE_PLAIN && !(p->factor >= 1.0 && isfinite(p->factor))) return FADKV_ERR_INVALID_ARG;
    if (p->scaling == FADKV_ROPE_PARTS &&
        !(p->original > 0.0 && isfinite(p->original) && p->slow < p->fast && isfinite(p->slow) && isfinite(p->fast)))
        return FADKV_ERR_INVALID_ARG;
    memset(out, 0, sizeof(*out));
    out->d = p->d;
    out->rotary_dim = p->rotary_dim;
    out->interleaved = p->interleaved != 0;
    out->amplitude = (float)p->amplitude;
    const double two_pi = 6.283185307179586476925;
    const int rd = p->rotary_dim;
    double base = p->base;
    if (p->scaling == FADKV_ROPE_STRETCH && rd > 2) base *= pow(p->factor, (double)rd / (rd - 2));
    for (int i = 0; i < rd / 2; ++i) {
        double f = pow(base, -2.0 * i / rd);
        if (p->scaling == FADKV_ROPE_LINEAR) f /= p->factor;
        if (p->scaling == FADKV_ROPE_PARTS) {
            double g = (p->original * f / two_pi - p->slow) / (p->fast - p->slow);
            g = g < 0.0 ? 0.0 : (g > 1.0 ? 1.0 : g);
            f *= g + (1.0 - g) / p->factor;
        }
        out->turns[i] = (uint64_t)ldexp(f / two_pi, 64);   // f <= 1: less than a sixth of a turn
    }
    return FADKV_OK;
}

fadkv_status fadkv_qk_norm_rope(const fadkv_qk_params* p, const fadkv_rope* rope, const void* q, const void* k,
                                const void* v, const void* wq, const void* wk, const int32_t* positions,
                                const int32_t* slots, void* q_out, void* k_out, void* k_pages, void* v_pages,
                                void* stream)
{
    if (!p || !rope) return FADKV_ERR_INVALID_ARG;
    if (p->T < 0 || p->Hq < 1 || p->Hkv < 1 || !(p->eps >= 0.f) || !dtype_ok(p->dtype) || !dtype_ok(p->q_dtype) ||
        !dtype_ok(p->kv_dtype))
        return FADKV_ERR_INVALID_ARG;
    if ((p->d != 64 && p->d != 128) || p->Hq > 4096 || p->Hkv > 4096) return FADKV_ERR_UNSUPPORTED;
    if (rope->d != p->d || rope->rotary_dim < 0 || rope->rotary_dim > p->d || rope->rotary_dim % 16 != 0)
        return FADKV_ERR_INVALID_ARG;
    if (!stride_ok(p->q_stride, (int64_t)p->Hq * p->d) || !stride_ok(p->k_stride, (int64_t)p->Hkv * p->d) ||
        !stride_ok(p->v_stride, (int64_t)p->Hkv * p->d))
        return FADKV_ERR_INVALID_ARG;
    if (slots) {
        const fadkv_status st =
            check_pool(p->page_size, p->num_pages, p->d, p->page_stride, p->head_stride, p->token_stride);
        if (st != FADKV_OK) return st;
    }
    if (p->T > 0) {
        if (!q || !k || !v || !positions || !q_out || (slots && (!k_pages || !v_pages))) return FADKV_ERR_INVALID_ARG;
        const void* all[] = {q, k, v, wq, wk, q_out, k_out, k_pages, v_pages};
        for (const void* ptr : all)
            if (!aligned(ptr, 16)) return FADKV_ERR_INVALID_ARG;
        if (!aligned(positions, 4) || !aligned(slots, 4)) return FADKV_ERR_INVALID_ARG;
    }
    if (fault_injected()) return cuda_error("fadkv_qk_norm_rope", cudaErrorLaunchFailure);
    QkArgs a;
    a.p = *p;
    a.rope = *rope;
    a.shift = slots ? log2_exact(p->page_size) : 0;
    a.q = q;
    a.k = k;
    a.v = v;
    a.wq = wq;
    a.wk = wk;
    a.positions = positions;
    a.slots = slots;
    a.q_out = q_out;
    a.k_out = k_out;
    a.k_pages = k_pages;
    a.v_pages = v_pages;
    const cudaError_t e = launch_qk_norm_rope(a, (cudaStream_t)stream);
    return e == cudaSuccess ? FADKV_OK : cuda_error("fadkv_qk_norm_rope", e);
}

fadkv_status fadkv_paged_attend_workspace_bytes(const fadkv_paged_params* p, size_t* bytes)
{
    const fadkv_status st = check_paged(p);
    if (st != FADKV_OK) return st;
    if (!bytes) return FADKV_ERR_INVALID_ARG;
    *bytes = paged_attend_workspace(*p);
    return FADKV_OK;
}

fadkv_status fadkv_paged_prefill_workspace_bytes(const fadkv_paged_params* p, size_t* bytes)
{
    const fadkv_status st = check_paged(p);
    if (st != FADKV_OK) return st;
    if (!bytes) return FADKV_ERR_INVALID_ARG;
    *bytes = paged_prefill_workspace(*p);
    return FADKV_OK;
}

fadkv_status fadkv_paged_status(void* workspace, uint64_t* host_out, int32_t clear, void* stream)
{
    if (!workspace || !aligned(workspace, 256) || !host_out) return FADKV_ERR_INVALID_ARG;
    if (fault_injected()) return cuda_error("fadkv_paged_status", cudaErrorLaunchFailure);
    cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e = cudaMemcpyAsync(host_out, workspace, sizeof(uint64_t), cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess && clear) e = cudaMemsetAsync(workspace, 0, sizeof(uint64_t), st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    return e == cudaSuccess ? FADKV_OK : cuda_error("fadkv_paged_status", e);
}

fadkv_status fadkv_debug_paged_wait_limit(uint64_t limit_ns)
{
    g_wait_ns.store(limit_ns, std::memory_order_relaxed);
    return FADKV_OK;
}

}  // extern "C"

namespace {

fadkv_status paged_call(const char* name, bool prefill, const fadkv_paged_params* p, const void* k_pages,
                        const void* v_pages, const int32_t* block_table, const int32_t* lengths,
                        const int32_t* starts, const int32_t* positions, const void* q, void* out, float* lse,
                        void* workspace, size_t workspace_bytes, void* stream)
{
    const fadkv_status st = check_paged(p);
    if (st != FADKV_OK) return st;
    if (!prefill && p->T != p->B) return FADKV_ERR_INVALID_ARG;
    const size_t need = prefill ? paged_prefill_workspace(*p) : paged_attend_workspace(*p);
    if (workspace_bytes < need || (need > 0 && !workspace)) return FADKV_ERR_WORKSPACE;
    if (need > 0 && !aligned(workspace, 256)) return FADKV_ERR_INVALID_ARG;
    if (p->B > 0 && p->T > 0) {
        if ((p->num_pages > 0 && (!k_pages || !v_pages)) || !block_table || !lengths || !q || !out ||
            (prefill && !starts))
            return FADKV_ERR_INVALID_ARG;
        if (!aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(block_table, 4) || !aligned(lengths, 4) ||
            !aligned(starts, 4) || !aligned(positions, 4) || !aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4))
            return FADKV_ERR_INVALID_ARG;
    }
    if (fault_injected()) return cuda_error(name, cudaErrorLaunchFailure);
    const PagedArgs a = paged_args(*p, k_pages, v_pages, block_table, lengths, starts, positions, q, out, lse, workspace);
    const cudaError_t e = prefill ? launch_paged_prefill(a, (cudaStream_t)stream)
                                  : launch_paged_attend(a, (cudaStream_t)stream);
    return e == cudaSuccess ? FADKV_OK : cuda_error(name, e);
}

}  // namespace

extern "C" {

fadkv_status fadkv_paged_attend(const fadkv_paged_params* p, const void* k_pages, const void* v_pages,
                                const int32_t* block_table, const int32_t* lengths, const void* q, void* out,
                                float* lse, void* workspace, size_t workspace_bytes, void* stream)
{
    return paged_call("fadkv_paged_attend", false, p, k_pages, v_pages, block_table, lengths, nullptr, nullptr, q, out,
                      lse, workspace, workspace_bytes, stream);
}

fadkv_status fadkv_paged_attend_planned(const fadkv_paged_params* p, const void* k_pages, const void* v_pages,
                                        const int32_t* block_table, const int32_t* lengths, const int32_t* positions,
                                        const void* q, void* out, float* lse, void* workspace,
                                        size_t workspace_bytes, void* stream)
{
    return paged_call("fadkv_paged_attend_planned", false, p, k_pages, v_pages, block_table, lengths, nullptr,
                      positions, q, out, lse, workspace, workspace_bytes, stream);
}

fadkv_status fadkv_paged_prefill(const fadkv_paged_params* p, const void* k_pages, const void* v_pages,
                                 const int32_t* block_table, const int32_t* lengths, const int32_t* starts,
                                 const void* q, void* out, float* lse, void* workspace, size_t workspace_bytes,
                                 void* stream)
{
    return paged_call("fadkv_paged_prefill", true, p, k_pages, v_pages, block_table, lengths, starts, nullptr, q, out,
                      lse, workspace, workspace_bytes, stream);
}

fadkv_status fadkv_paged_prefill_planned(const fadkv_paged_params* p, const void* k_pages, const void* v_pages,
                                         const int32_t* block_table, const int32_t* lengths, const int32_t* starts,
                                         const int32_t* positions, const void* q, void* out, float* lse,
                                         void* workspace, size_t workspace_bytes, void* stream)
{
    return paged_call("fadkv_paged_prefill_planned", true, p, k_pages, v_pages, block_table, lengths, starts,
                      positions, q, out, lse, workspace, workspace_bytes, stream);
}

}  // extern "C"
