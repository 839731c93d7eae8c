// C ABI of the generation path (declared in include/rlhead.h): host-side argument checks
// and dispatch.  Nothing here allocates device memory or synchronises.
#include <cmath>

#include "internal.h"

using namespace rl;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int fail(int code, const char* msg) {
    set_last_error(msg);
    return code;
}

int check_device() {
    int dev = 0, major = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess || major != 10)
        return fail(RL_ERR_UNSUPPORTED, "needs an sm_100-family GPU");
    return RL_OK;
}

// Whether n and m elements of 4 bytes at p and q share memory.
bool overlap(const void* p, int64_t n, const void* q, int64_t m) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return n > 0 && m > 0 && a < b + 4 * static_cast<uintptr_t>(m) && b < a + 4 * static_cast<uintptr_t>(n);
}

bool page_size_ok(int32_t p) { return p == 16 || p == 32 || p == 64 || p == 128; }

constexpr int64_t kMaxVocab = int64_t(1) << 20;
constexpr int64_t kMax31 = int64_t(1) << 31;

int check_attn_sizes(const rl_prefix_attn_args* a) {
    if (!a) return fail(RL_ERR_ARG, "args is NULL");
    if (a->T < 0 || a->R < 0 || a->G < 0 || a->n_pages < 0 || a->table_width < 0 || a->prefix_width < 0 || a->max_q < 0 ||
        a->max_kv < 0 || a->max_prefix < 0)
        return fail(RL_ERR_ARG, "negative size");
    if (a->Hkv <= 0 || a->Hq <= 0 || a->Hq % a->Hkv != 0) return fail(RL_ERR_ARG, "Hq must be a positive multiple of Hkv");
    if (a->D != 64 && a->D != 128) return fail(RL_ERR_UNSUPPORTED, "D must be 64 or 128");
    if (!page_size_ok(a->page_size)) return fail(RL_ERR_UNSUPPORTED, "page_size must be 16, 32, 64 or 128");
    if (a->dtype != RL_DTYPE_BF16 && a->dtype != RL_DTYPE_F16) return fail(RL_ERR_UNSUPPORTED, "dtype must be bf16 or fp16");
    if (a->T >= kMax31 || a->R >= kMax31 || a->G >= kMax31 || a->Hq > 4096 || a->T * a->Hq >= kMax31 || a->n_pages >= kMax31 ||
        a->n_pages * a->Hkv * a->page_size >= kMax31 || a->max_q >= kMax31 || a->max_kv >= kMax31 || a->max_prefix >= kMax31)
        return fail(RL_ERR_UNSUPPORTED, "sizes too large (rows of queries and rows of the cache below 2^31)");
    if (a->T > 0 && a->R > 0 && a->max_q < 1) return fail(RL_ERR_ARG, "max_q must bound the step's lengths");
    if (!(a->scale >= 0.f) || !std::isfinite(a->scale * 1.5f)) return fail(RL_ERR_ARG, "scale is negative, not finite or too large");
    return RL_OK;
}

}  // namespace

extern "C" {

int rl_page_plan(const rl_page_plan_args* a, int32_t* dev_status, void* stream) {
    if (!a || !dev_status) return fail(RL_ERR_ARG, "args/dev_status is NULL");
    if (a->R < 0 || a->T < 0 || a->G < 0 || a->n_free < 0 || a->n_pages < 0 || a->table_width < 0)
        return fail(RL_ERR_ARG, "negative size");
    if (!page_size_ok(a->page_size)) return fail(RL_ERR_UNSUPPORTED, "page_size must be 16, 32, 64 or 128");
    if (a->R >= kMax31 || a->T >= kMax31 || a->G >= kMax31 || a->n_free >= kMax31 || a->n_pages >= kMax31 || a->table_width >= kMax31)
        return fail(RL_ERR_UNSUPPORTED, "R, T, G, n_free, n_pages or table_width too large");
    if (!a->cu_q || !a->free_used_out || (a->R > 0 && (!a->q_lens || !a->ctx_lens || !a->kv_lens)) ||
        (a->T > 0 && !a->slot_map) || (a->R > 0 && a->table_width > 0 && !a->block_table) ||
        (a->n_free > 0 && !a->free_pages))
        return fail(RL_ERR_ARG, "required pointer is NULL");
    if (a->G > 0 && (!a->group_offsets || !a->prefix_lens))
        return fail(RL_ERR_ARG, "group_offsets/prefix_lens NULL with G > 0");
    if (a->free_used == a->free_used_out) return fail(RL_ERR_ARG, "free_used_out must not be free_used");
    if (overlap(a->cu_q, a->R + 1, a->q_lens, a->R) || overlap(a->cu_q, a->R + 1, a->ctx_lens, a->R) ||
        overlap(a->kv_lens, a->R, a->q_lens, a->R) || (a->kv_lens != a->ctx_lens && overlap(a->kv_lens, a->R, a->ctx_lens, a->R)))
        return fail(RL_ERR_ARG, "cu_q/kv_lens share memory with q_lens/ctx_lens");
    int rc = check_device();
    return rc != RL_OK ? rc : page_plan_impl(a, dev_status, static_cast<cudaStream_t>(stream));
}

int rl_kv_append(const rl_kv_append_args* a, int32_t* dev_status, void* stream) {
    if (!a || !dev_status) return fail(RL_ERR_ARG, "args/dev_status is NULL");
    if (a->T < 0 || a->n_pages < 0 || a->Hkv <= 0 || a->D <= 0) return fail(RL_ERR_ARG, "negative or zero size");
    if (!page_size_ok(a->page_size)) return fail(RL_ERR_UNSUPPORTED, "page_size must be 16, 32, 64 or 128");
    if (a->dtype != RL_DTYPE_BF16 && a->dtype != RL_DTYPE_F16) return fail(RL_ERR_UNSUPPORTED, "dtype must be bf16 or fp16");
    if (a->T >= kMax31 || a->n_pages >= kMax31 || int64_t(a->Hkv) * a->D >= (int64_t(1) << 24))
        return fail(RL_ERR_UNSUPPORTED, "T, n_pages or Hkv * D too large");
    if (a->T > 0 && (!a->k || !a->v || !a->slot_map)) return fail(RL_ERR_ARG, "k/v/slot_map is NULL");
    if (a->T > 0 && a->n_pages > 0 && (!a->k_cache || !a->v_cache)) return fail(RL_ERR_ARG, "cache is NULL");
    if (!aligned(a->k_cache, 16) || !aligned(a->v_cache, 16)) return fail(RL_ERR_ARG, "cache not 16-byte aligned");
    int rc = check_device();
    return rc != RL_OK ? rc : kv_append_impl(a, dev_status, static_cast<cudaStream_t>(stream));
}

size_t rl_prefix_attn_workspace_bytes(const rl_prefix_attn_args* a) {
    if (check_attn_sizes(a) != RL_OK) return 0;
    return prefix_attn_ws_bytes(a);
}

int rl_prefix_attn(const rl_prefix_attn_args* a, void* ws, size_t ws_bytes, int32_t* dev_status, void* stream) {
    int rc = check_attn_sizes(a);
    if (rc != RL_OK) return rc;
    if (!dev_status) return fail(RL_ERR_ARG, "dev_status is NULL");
    if (a->T > 0) {
        if (!a->q || !a->out || !a->cu_q) return fail(RL_ERR_ARG, "q/out/cu_q is NULL");
        if (a->R > 0 && (!a->kv_lens || (a->table_width > 0 && !a->block_table))) return fail(RL_ERR_ARG, "kv_lens/block_table is NULL");
        if (a->G > 0 && (!a->group_offsets || !a->prefix_lens || (a->prefix_width > 0 && !a->prefix_table)))
            return fail(RL_ERR_ARG, "group_offsets/prefix_lens/prefix_table NULL with G > 0");
        if (!a->k_cache || !a->v_cache || a->n_pages == 0) return fail(RL_ERR_ARG, "the cache is missing");
        if (!aligned(a->k_cache, 16) || !aligned(a->v_cache, 16) || !aligned(a->out, 16)) return fail(RL_ERR_ARG, "cache/out not 16-byte aligned");
        // (the stride of an axis of one entry means nothing)
        if (!aligned(a->q, 16) || (a->T > 1 && a->q_stride_t % 8 != 0) || (a->Hq > 1 && a->q_stride_h % 8 != 0))
            return fail(RL_ERR_ARG, "q rows not 16-byte aligned");
        const size_t need = prefix_attn_ws_bytes(a);
        if (ws_bytes < need) return fail(RL_ERR_WORKSPACE, "attention workspace too small");
        if (need > 0 && (!ws || !aligned(ws, 16))) return fail(RL_ERR_ARG, "ws is NULL or not 16-byte aligned");
    }
    rc = check_device();
    return rc != RL_OK ? rc : prefix_attn_impl(a, ws, dev_status, static_cast<cudaStream_t>(stream));
}

size_t rl_sample_workspace_bytes(int64_t N, int64_t V, int32_t K) {
    if (N < 0 || V <= 0 || V > kMaxVocab || K <= 0) return 0;
    return sample_ws_bytes(N, V);
}

int rl_sample(const rl_sample_args* a, void* ws, size_t ws_bytes, int32_t* dev_status, void* stream) {
    if (!a || !dev_status) return fail(RL_ERR_ARG, "args/dev_status is NULL");
    if (a->N < 0 || a->V <= 0 || a->K <= 0 || a->capacity < 0) return fail(RL_ERR_ARG, "negative or zero size");
    if (a->dtype != RL_DTYPE_F32 && a->dtype != RL_DTYPE_BF16 && a->dtype != RL_DTYPE_F16)
        return fail(RL_ERR_UNSUPPORTED, "dtype must be fp32, bf16 or fp16");
    if (a->V > kMaxVocab || a->N >= kMax31 || a->K > 1024) return fail(RL_ERR_UNSUPPORTED, "N, V or K too large");
    if (a->N > 1 && a->row_stride < a->V) return fail(RL_ERR_ARG, "row_stride smaller than V");
    if (a->N > 0 && (!a->logits || !a->u || !a->tokens)) return fail(RL_ERR_ARG, "logits/u/tokens is NULL");
    if (a->offsets && a->capacity > 0 && (!a->ids || !a->support_logq))
        return fail(RL_ERR_ARG, "ids/support_logq NULL with capacity > 0");
    if (!aligned(a->logits, a->dtype == RL_DTYPE_F32 ? 4 : 2)) return fail(RL_ERR_ARG, "logits not aligned to their type");
    if (ws_bytes < rl_sample_workspace_bytes(a->N, a->V, a->K)) return fail(RL_ERR_WORKSPACE, "sampling workspace too small");
    if (!ws || !aligned(ws, 16)) return fail(RL_ERR_ARG, "ws is NULL or not 16-byte aligned");
    int rc = check_device();
    if (rc != RL_OK) return rc;
    if (a->N == 0) {
        if (a->offsets && cudaMemsetAsync(a->offsets, 0, sizeof(int64_t), static_cast<cudaStream_t>(stream)) != cudaSuccess)
            return fail(RL_ERR_CUDA, "cudaMemsetAsync failed");
        return RL_OK;
    }
    return sample_impl(a, ws, dev_status, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
