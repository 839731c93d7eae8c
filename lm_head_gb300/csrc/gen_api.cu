// C ABI of the generation path and of distillation (declared in include/rlhead.h): host-side
// argument checks and dispatch.  Nothing here allocates device memory or synchronises.
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

// n pieces of `bytes` bytes, `stride` bytes apart.
struct Pieces {
    const void* p;
    int64_t n, bytes, stride;
};
Pieces whole(const void* p, int64_t n, int64_t size) { return {p, p && n > 0 ? 1 : 0, n * size, 0}; }
// Whether they share memory.  Pieces of b may lie between those of a where both are as far apart, or b is one.
bool share(const Pieces& a, const Pieces& b) {
    using I = __int128;
    if (!a.p || !b.p || a.n <= 0 || b.n <= 0) return false;
    const I x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    if (x >= y + I(b.n - 1) * b.stride + b.bytes || y >= x + I(a.n - 1) * a.stride + a.bytes) return false;
    if (a.n == 1) return b.n == 1 || share(b, a);
    if (b.n > 1 && b.stride != a.stride) return true;
    const I k = (y < x ? y - x - (a.stride - 1) : y - x) / a.stride, d = y - x - k * a.stride;      // b begins d bytes after the piece k of a
    if (b.n > 1) return d < a.bytes || a.stride - d < b.bytes;
    return (k >= 0 && k < a.n && d < a.bytes) || (k + 1 >= 0 && k + 1 < a.n && a.stride - d < b.bytes);
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

int check_dist(const rl_dist* d, int32_t dtype, int64_t V, bool needed) {
    if (!d->logits && !d->offsets) return needed ? fail(RL_ERR_ARG, "a distribution has neither logits nor support rows") : RL_OK;
    if (d->n_rows < 0 || d->nnz < 0) return fail(RL_ERR_ARG, "negative size");
    if (d->n_rows >= kMax31) return fail(RL_ERR_UNSUPPORTED, "n_rows too large");
    if (d->logits) {
        if (dtype != RL_DTYPE_F32 && dtype != RL_DTYPE_BF16 && dtype != RL_DTYPE_F16)
            return fail(RL_ERR_UNSUPPORTED, "dtype must be fp32, bf16 or fp16");
        if (!aligned(d->logits, dtype == RL_DTYPE_F32 ? 4 : 2)) return fail(RL_ERR_ARG, "logits not aligned to their type");
        if (d->n_rows > 1 && d->row_stride < V) return fail(RL_ERR_ARG, "row_stride smaller than V");
    }
    if (d->offsets && d->nnz > 0 && (!d->ids || !d->logq)) return fail(RL_ERR_ARG, "ids/logq NULL with support rows");
    if (d->logits && d->offsets && !d->replayed) return fail(RL_ERR_ARG, "replayed NULL with logits and support rows");
    return RL_OK;
}

int check_verify_sizes(const rl_verify_args* a) {
    if (!a) return fail(RL_ERR_ARG, "args is NULL");
    if (a->R < 0 || a->T < 0 || a->V <= 0) return fail(RL_ERR_ARG, "negative or zero size");
    if (a->V > kMaxVocab || a->R >= (int64_t(1) << 28) || a->T >= kMax31) return fail(RL_ERR_UNSUPPORTED, "R, T or V too large");
    const int rc = check_dist(&a->target, a->target_dtype, a->V, true);
    return rc != RL_OK ? rc : check_dist(&a->draft, a->draft_dtype, a->V, false);
}

int check_distill(const rl_distill_args* a, const void* saved, const int32_t* dev_status, int pass) {
    if (!a || !dev_status) return fail(RL_ERR_ARG, "args/dev_status is NULL");
    if (a->N < 0 || a->V <= 0 || a->nnz < 0) return fail(RL_ERR_ARG, "negative or zero size");
    if (a->dtype != RL_DTYPE_F32 && a->dtype != RL_DTYPE_BF16 && a->dtype != RL_DTYPE_F16)
        return fail(RL_ERR_UNSUPPORTED, "dtype must be fp32, bf16 or fp16");
    const int64_t size = a->dtype == RL_DTYPE_F32 ? 4 : 2;
    if (a->kind < RL_DISTILL_FORWARD || a->kind > RL_DISTILL_JSD || a->tail < 0 || a->tail > 1 || a->reserved != 0)
        return fail(RL_ERR_ARG, "kind, tail or reserved out of range");
    if (!a->tail && a->kind != RL_DISTILL_FORWARD) return fail(RL_ERR_ARG, "the reverse and JSD kinds need tail = 1");
    if (!(a->temperature >= 0x1p-20f) || !(a->temperature <= 0x1p20f)) return fail(RL_ERR_ARG, "temperature out of range");
    if (a->kind == RL_DISTILL_JSD && (!(a->beta > 0.f) || !(a->beta < 1.f))) return fail(RL_ERR_ARG, "beta must lie between 0 and 1");
    if (a->V > kDistillRowBytes / size || a->N >= kMax31) return fail(RL_ERR_UNSUPPORTED, "N or V too large");
    if (a->N > 1 && a->row_stride < a->V) return fail(RL_ERR_ARG, "row_stride smaller than V");
    if (a->N == 0) return RL_OK;
    if (!a->logits || !a->offsets || (a->nnz > 0 && (!a->ids || !a->logq))) return fail(RL_ERR_ARG, "logits/offsets/ids/logq is NULL");
    if (!aligned(a->logits, size)) return fail(RL_ERR_ARG, "logits not aligned to their type");
    if (pass != kDistillBwd && !a->loss) return fail(RL_ERR_ARG, "loss is NULL");
    if (pass != kDistillFwd) {
        if (!a->dloss || !a->dlogits) return fail(RL_ERR_ARG, "dloss/dlogits is NULL");
        if (!aligned(a->dlogits, size)) return fail(RL_ERR_ARG, "dlogits not aligned to their type");
        if (a->N > 1 && a->grad_stride < a->V) return fail(RL_ERR_ARG, "grad_stride smaller than V");
        const bool in_place = a->logits == a->dlogits && (a->N == 1 || a->row_stride == a->grad_stride);
        const Pieces z = {a->logits, a->N, a->V * size, a->row_stride * size}, d = {a->dlogits, a->N, a->V * size, a->grad_stride * size};
        if (!in_place && share(z, d)) return fail(RL_ERR_ARG, "dlogits shares memory with logits");
    }
    // (the support rows are read until the loss and the gradients are written; dloss before the loss is)
    const Pieces none = {nullptr, 0, 0, 0}, state = whole(saved, 1, static_cast<int64_t>(distill_saved_bytes(a->N, a->nnz)));
    const Pieces d = pass == kDistillFwd ? none : Pieces{a->dlogits, a->N, a->V * size, a->grad_stride * size};
    const Pieces out[] = {pass == kDistillBwd ? none : whole(a->loss, a->N, 4), pass == kDistillBwd ? none : whole(a->mass, a->N, 4), d, state};
    const Pieces in[] = {whole(a->offsets, a->N + 1, 8), whole(a->ids, a->nnz, 4), whole(a->logq, a->nnz, 4)};
    for (const Pieces& y : out) {
        for (const Pieces& x : in)
            if (share(x, y)) return fail(RL_ERR_ARG, "an output shares memory with a support row");
        if (&y != out + 2 && share({a->logits, a->N, a->V * size, a->row_stride * size}, y))
            return fail(RL_ERR_ARG, "an output shares memory with logits");
    }
    if (share(state, out[0]) || share(state, out[1]) || share(state, d) || share(d, out[0]) || share(d, out[1]) || share(out[0], out[1]))
        return fail(RL_ERR_ARG, "outputs share memory with each other");
    if (pass != kDistillFwd && (share(whole(a->dloss, a->N, 4), d) || share(whole(a->dloss, a->N, 4), state)))
        return fail(RL_ERR_ARG, "an output shares memory with dloss");
    return check_device();
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

// ---- verification of drafts ------------------------------------------------------------
size_t rl_verify_workspace_bytes(const rl_verify_args* a) { return check_verify_sizes(a) != RL_OK ? 0 : verify_ws_bytes(a); }

int rl_verify(const rl_verify_args* a, void* ws, size_t ws_bytes, int32_t* dev_status, void* stream) {
    int rc = check_verify_sizes(a);
    if (rc != RL_OK) return rc;
    if (!dev_status) return fail(RL_ERR_ARG, "dev_status is NULL");
    if ((a->R > 0 && (!a->cu_q || !a->u_next || !a->accepted)) || (a->T > 0 && (!a->step_tokens || !a->u || !a->tokens)))
        return fail(RL_ERR_ARG, "required pointer is NULL");
    if (a->keep_lens && a->keep_lens != a->ctx_lens && overlap(a->keep_lens, a->R, a->ctx_lens, a->ctx_lens ? a->R : 0))
        return fail(RL_ERR_ARG, "keep_lens shares memory with ctx_lens");
    const size_t need = verify_ws_bytes(a);
    if (ws_bytes < need) return fail(RL_ERR_WORKSPACE, "verification workspace too small");
    if (need > 0 && (!ws || !aligned(ws, 16))) return fail(RL_ERR_ARG, "ws is NULL or not 16-byte aligned");
    // (outputs are written before the last request has read its inputs)
    const Pieces out[] = {whole(a->tokens, a->T, 4), whole(a->logq, a->T, 4), whole(a->accepted, a->R, 4), whole(a->keep_lens, a->R, 4)};
    const auto shared = [&](const Pieces& in, int n) {
        for (int k = 0; k < n; ++k)
            if (share(in, out[k])) return true;
        return false;
    };
    if (shared(whole(a->cu_q, a->R + 1, 4), 4) || shared(whole(a->step_tokens, a->T, 4), 4) || shared(whole(a->u, a->T, 4), 4) ||
        shared(whole(a->u_next, a->R, 4), 4) || shared(whole(a->ctx_lens, a->R, 4), 3))
        return fail(RL_ERR_ARG, "an output shares memory with an input");
    const struct { const rl_dist& d; int64_t size; } sides[] = {{a->target, a->target_dtype == RL_DTYPE_F32 ? 4 : 2}, {a->draft, a->draft_dtype == RL_DTYPE_F32 ? 4 : 2}};
    for (const auto& s : sides) {
        if (!s.d.logits && !s.d.offsets) continue;
        if (shared({s.d.logits, s.d.n_rows, a->V * s.size, s.d.row_stride * s.size}, 4) || shared(whole(s.d.temperature, s.d.n_rows, 4), 4) ||
            shared(whole(s.d.rows, a->T, 4), 4) || shared(whole(s.d.replayed, s.d.logits && s.d.offsets ? s.d.n_rows : 0, 1), 4) ||
            (s.d.offsets && (shared(whole(s.d.offsets, s.d.n_rows + 1, 8), 4) || shared(whole(s.d.ids, s.d.nnz, 4), 4) || shared(whole(s.d.logq, s.d.nnz, 4), 4))))
            return fail(RL_ERR_ARG, "an output shares memory with a distribution");
    }
    rc = check_device();
    return rc != RL_OK ? rc : verify_impl(a, ws, dev_status, static_cast<cudaStream_t>(stream));
}

// ---- pages of a rollout's life ---------------------------------------------------------
size_t rl_page_release_workspace_bytes(int64_t n_pages) {
    return n_pages < 0 || n_pages >= kMax31 ? 0 : page_release_ws_bytes(n_pages);
}

int rl_page_release(const rl_page_release_args* a, void* ws, size_t ws_bytes, int32_t* dev_status, void* stream) {
    if (!a || !dev_status) return fail(RL_ERR_ARG, "args/dev_status is NULL");
    if (a->R < 0 || a->G < 0 || a->n_free < 0 || a->n_pages < 0 || a->table_width < 0 || a->held_width < 0)
        return fail(RL_ERR_ARG, "negative size");
    if (!page_size_ok(a->page_size)) return fail(RL_ERR_UNSUPPORTED, "page_size must be 16, 32, 64 or 128");
    if (a->R >= kMax31 || a->G >= kMax31 || a->n_free >= kMax31 || a->n_pages >= kMax31 || a->table_width >= kMax31 || a->held_width >= kMax31)
        return fail(RL_ERR_UNSUPPORTED, "R, G, n_free, n_pages or a table's width too large");
    if (!a->free_used || !a->free_used_out || (a->R > 0 && (!a->kv_lens || !a->keep_lens)) ||
        (a->R > 0 && a->table_width > 0 && !a->block_table) || (a->n_free > 0 && !a->free_pages))
        return fail(RL_ERR_ARG, "required pointer is NULL");
    if (a->G > 0 && (!a->held_lens || (a->held_width > 0 && !a->held_table)))
        return fail(RL_ERR_ARG, "held_lens/held_table NULL with G > 0");
    if (a->free_used == a->free_used_out) return fail(RL_ERR_ARG, "free_used_out must not be free_used");
    if (ws_bytes < page_release_ws_bytes(a->n_pages)) return fail(RL_ERR_WORKSPACE, "release workspace too small");
    if (a->n_pages > 0 && (!ws || !aligned(ws, 16))) return fail(RL_ERR_ARG, "ws is NULL or not 16-byte aligned");
    int rc = check_device();
    return rc != RL_OK ? rc : page_release_impl(a, ws, dev_status, static_cast<cudaStream_t>(stream));
}

size_t rl_page_fork_workspace_bytes(int64_t R, int64_t C) {
    return R < 0 || C < 0 || R >= kMax31 || C >= kMax31 ? 0 : page_fork_ws_bytes(R, C);
}

int rl_page_fork(const rl_page_fork_args* a, void* ws, size_t ws_bytes, int32_t* dev_status, void* stream) {
    if (!a || !dev_status) return fail(RL_ERR_ARG, "args/dev_status is NULL");
    if (a->R < 0 || a->C < 0 || a->n_free < 0 || a->n_pages < 0 || a->table_width < 0) return fail(RL_ERR_ARG, "negative size");
    if (!page_size_ok(a->page_size)) return fail(RL_ERR_UNSUPPORTED, "page_size must be 16, 32, 64 or 128");
    if (a->R >= kMax31 || a->C >= kMax31 || a->n_free >= kMax31 || a->n_pages >= kMax31 || a->table_width >= kMax31)
        return fail(RL_ERR_UNSUPPORTED, "R, C, n_free, n_pages or table_width too large");
    if (!a->free_used || !a->free_used_out || (a->C > 0 && (!a->parents || !a->children || !a->lens || !a->src || !a->dst || !a->tokens)) ||
        (a->C > 0 && a->R > 0 && (!a->kv_lens || (a->table_width > 0 && !a->block_table))) || (a->n_free > 0 && !a->free_pages))
        return fail(RL_ERR_ARG, "required pointer is NULL");
    if (a->free_used == a->free_used_out) return fail(RL_ERR_ARG, "free_used_out must not be free_used");
    if (ws_bytes < page_fork_ws_bytes(a->R, a->C)) return fail(RL_ERR_WORKSPACE, "fork workspace too small");
    if (a->C > 0 && (!ws || !aligned(ws, 16))) return fail(RL_ERR_ARG, "ws is NULL or not 16-byte aligned");
    // (the rows are written after the lists)
    for (const int32_t* in : {a->parents, a->children, a->lens}) {
        if (overlap(in, a->C, a->kv_lens, a->R)) return fail(RL_ERR_ARG, "an input shares memory with kv_lens");
        for (const int32_t* out : {a->src, a->dst, a->tokens})
            if (overlap(in, a->C, out, a->C)) return fail(RL_ERR_ARG, "an input shares memory with an output");
    }
    int rc = check_device();
    return rc != RL_OK ? rc : page_fork_impl(a, ws, dev_status, static_cast<cudaStream_t>(stream));
}

size_t rl_page_compact_workspace_bytes(int64_t n_pages) {
    return n_pages < 0 || n_pages >= kMax31 ? 0 : page_compact_ws_bytes(n_pages);
}

int rl_page_compact(const rl_page_compact_args* a, void* ws, size_t ws_bytes, int32_t* dev_status, void* stream) {
    if (!a || !dev_status) return fail(RL_ERR_ARG, "args/dev_status is NULL");
    if (a->R < 0 || a->G < 0 || a->n_pages < 0 || a->table_width < 0 || a->prefix_width < 0) return fail(RL_ERR_ARG, "negative size");
    if (!page_size_ok(a->page_size)) return fail(RL_ERR_UNSUPPORTED, "page_size must be 16, 32, 64 or 128");
    if (a->R >= kMax31 || a->G >= kMax31 || a->n_pages >= kMax31 || a->table_width >= kMax31 || a->prefix_width >= kMax31)
        return fail(RL_ERR_UNSUPPORTED, "R, G, n_pages or a table's width too large");
    if (!a->free_used_out || (a->R > 0 && !a->kv_lens) || (a->R > 0 && a->table_width > 0 && (!a->block_table || !a->block_table_out)) ||
        (a->n_pages > 0 && !a->free_pages) || (a->n_pages > 1 && (!a->src || !a->dst)))
        return fail(RL_ERR_ARG, "required pointer is NULL");
    if (a->G > 0 && (!a->prefix_lens || (a->prefix_width > 0 && (!a->prefix_table || !a->prefix_table_out))))
        return fail(RL_ERR_ARG, "prefix_lens/prefix_table NULL with G > 0");
    const auto apart = [](const int32_t* x, const int32_t* y, int64_t n) { return x == y || !overlap(x, n, y, n); };
    if (!apart(a->block_table, a->block_table_out, a->R * a->table_width) || !apart(a->prefix_table, a->prefix_table_out, a->G * a->prefix_width))
        return fail(RL_ERR_ARG, "a table's output shares memory with it and is not it");
    if (ws_bytes < page_compact_ws_bytes(a->n_pages)) return fail(RL_ERR_WORKSPACE, "compact workspace too small");
    if (a->n_pages > 0 && (!ws || !aligned(ws, 16))) return fail(RL_ERR_ARG, "ws is NULL or not 16-byte aligned");
    int rc = check_device();
    return rc != RL_OK ? rc : page_compact_impl(a, ws, dev_status, static_cast<cudaStream_t>(stream));
}

int rl_page_copy(const rl_page_copy_args* a, int32_t* dev_status, void* stream) {
    if (!a || !dev_status) return fail(RL_ERR_ARG, "args/dev_status is NULL");
    if (a->n < 0 || a->n_pages < 0 || a->layers < 0 || a->Hkv <= 0 || a->D <= 0) return fail(RL_ERR_ARG, "negative or zero size");
    if (!page_size_ok(a->page_size)) return fail(RL_ERR_UNSUPPORTED, "page_size must be 16, 32, 64 or 128");
    if (a->dtype != RL_DTYPE_F32 && a->dtype != RL_DTYPE_BF16 && a->dtype != RL_DTYPE_F16)
        return fail(RL_ERR_UNSUPPORTED, "dtype must be fp32, bf16 or fp16");
    if (a->n >= kMax31 || a->n_pages >= kMax31 || int64_t(a->Hkv) * a->D >= (int64_t(1) << 24) || a->layers > 65536 ||
        int64_t(a->layers) * a->Hkv >= (int64_t(1) << 30))
        return fail(RL_ERR_UNSUPPORTED, "n, n_pages, layers or Hkv * D too large");
    if (a->layers > 1 && (a->layer_stride < 0 || a->layer_stride < a->n_pages * a->Hkv * a->page_size * a->D))
        return fail(RL_ERR_ARG, "layer_stride smaller than a layer");
    if (a->n > 0 && (!a->src || !a->dst)) return fail(RL_ERR_ARG, "src/dst is NULL");
    if (a->n > 0 && a->layers > 0 && a->n_pages > 0 && (!a->k_cache || !a->v_cache)) return fail(RL_ERR_ARG, "cache is NULL");
    if (!aligned(a->k_cache, 16) || !aligned(a->v_cache, 16)) return fail(RL_ERR_ARG, "cache not 16-byte aligned");
    int rc = check_device();
    return rc != RL_OK ? rc : page_copy_impl(a, dev_status, static_cast<cudaStream_t>(stream));
}

// ---- distillation ------------------------------------------------------------------------
size_t rl_distill_saved_bytes(int64_t N, int64_t nnz) { return N < 0 || nnz < 0 ? 0 : distill_saved_bytes(N, nnz); }

int rl_distill_fwd(const rl_distill_args* a, void* saved, int32_t* dev_status, void* stream) {
    if (!saved || !aligned(saved, 16)) return fail(RL_ERR_ARG, "saved is NULL or not 16-byte aligned");
    const int rc = check_distill(a, saved, dev_status, kDistillFwd);
    return rc != RL_OK ? rc : distill_impl(a, kDistillFwd, saved, dev_status, static_cast<cudaStream_t>(stream));
}

int rl_distill_bwd(const rl_distill_args* a, const void* saved, int32_t* dev_status, void* stream) {
    if (!saved || !aligned(saved, 16)) return fail(RL_ERR_ARG, "saved is NULL or not 16-byte aligned");
    const int rc = check_distill(a, saved, dev_status, kDistillBwd);
    return rc != RL_OK ? rc : distill_impl(a, kDistillBwd, const_cast<void*>(saved), dev_status, static_cast<cudaStream_t>(stream));
}

int rl_distill_fwd_bwd(const rl_distill_args* a, void* saved, int32_t* dev_status, void* stream) {
    if (!saved || !aligned(saved, 16)) return fail(RL_ERR_ARG, "saved is NULL or not 16-byte aligned");
    const int rc = check_distill(a, saved, dev_status, kDistillBoth);
    return rc != RL_OK ? rc : distill_impl(a, kDistillBoth, saved, dev_status, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
