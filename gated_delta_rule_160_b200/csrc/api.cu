// api.cu -- the C ABI of libgdn2 (include/gdn2.h): argument checks and kernel dispatch.
//
// Every check runs on the host before anything is queued; a rejected call queues
// nothing. Error text is kept per calling thread.
#include <stdarg.h>
#include <stdio.h>

#include <atomic>

#include "internal.cuh"

namespace gdn2 {
namespace {

thread_local char g_err[512] = "";

// Testing hook (gdn2_testing_set_wait_limit): limit of the prefill's bounded waits, and
// whether its producer withholds the first loads.
std::atomic<unsigned long long> g_wait_ns{kDefaultWaitNs};
std::atomic<int> g_withhold{0};

gdn2_status fail(gdn2_status st, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof g_err, fmt, ap);
    va_end(ap);
    return st;
}

gdn2_status ok() {
    g_err[0] = '\0';
    return GDN2_OK;
}

// A pointer the GPU can dereference as device memory (plain or managed allocations).
bool is_device_ptr(const void* ptr) {
    cudaPointerAttributes attr;
    if (cudaPointerGetAttributes(&attr, ptr) != cudaSuccess) {
        cudaGetLastError();  // clear the sticky-free error this query may leave
        return false;
    }
    return attr.type == cudaMemoryTypeDevice || attr.type == cudaMemoryTypeManaged;
}

gdn2_status check_shape(const gdn2_shape* sh) {
    if (!sh) return fail(GDN2_ERR_INVALID_ARG, "shape is NULL");
    if (sh->n_seq < 1 || sh->n_seq > 65535)
        return fail(GDN2_ERR_INVALID_ARG, "n_seq = %d outside [1, 65535]", sh->n_seq);
    if (sh->T_total < 0) return fail(GDN2_ERR_INVALID_ARG, "T_total = %d is negative", sh->T_total);
    if (sh->h_qk < 1 || sh->h_v < 1)
        return fail(GDN2_ERR_INVALID_ARG, "head counts must be positive (h_qk=%d, h_v=%d)", sh->h_qk, sh->h_v);
    if (sh->h_v % sh->h_qk != 0)
        return fail(GDN2_ERR_INVALID_ARG, "h_v = %d is not a multiple of h_qk = %d", sh->h_v, sh->h_qk);
    if (sh->h_v > 65535) return fail(GDN2_ERR_UNSUPPORTED, "h_v = %d above 65535", sh->h_v);
    if ((long long)sh->n_seq * sh->h_v > 0x7fffffffLL)  // one CTA per (sequence, value head)
        return fail(GDN2_ERR_UNSUPPORTED, "n_seq * h_v = %lld (sequence, head) pairs above 2^31 - 1",
                    (long long)sh->n_seq * sh->h_v);
    if (sh->dtype != GDN2_F32 && sh->dtype != GDN2_BF16)
        return fail(GDN2_ERR_INVALID_ARG, "unknown dtype %d", (int)sh->dtype);
    if (sh->o_dtype != GDN2_F32 && sh->o_dtype != GDN2_BF16)
        return fail(GDN2_ERR_INVALID_ARG, "unknown o_dtype %d", (int)sh->o_dtype);
    if ((sh->dk != 64 && sh->dk != 128) || (sh->dv != 64 && sh->dv != 128))
        return fail(GDN2_ERR_UNSUPPORTED, "dk = %d, dv = %d: only 64 and 128 are supported", sh->dk, sh->dv);
    return GDN2_OK;
}

struct NamedPtr {
    const char* name;
    const void* ptr;
    bool required;
    unsigned align = 16;
};

gdn2_status check_ptrs(const NamedPtr* ps, int n) {
    for (int i = 0; i < n; ++i) {
        if (!ps[i].ptr) {
            if (ps[i].required) return fail(GDN2_ERR_INVALID_ARG, "%s is NULL", ps[i].name);
            continue;
        }
        if (reinterpret_cast<uintptr_t>(ps[i].ptr) & (ps[i].align - 1u))
            return fail(GDN2_ERR_INVALID_ARG, "%s = %p is not %u-byte aligned", ps[i].name, ps[i].ptr, ps[i].align);
        if (!is_device_ptr(ps[i].ptr))
            return fail(GDN2_ERR_INVALID_ARG, "%s = %p is not device memory", ps[i].name, ps[i].ptr);
    }
    return GDN2_OK;
}

Params make_params(const gdn2_shape* sh, const void* q, const void* k, const void* v,
                   const float* la, const void* b, const void* w, const float* S0,
                   const int32_t* cu, void* o, float* S_T) {
    Params p{};
    p.n_seq = sh->n_seq;
    p.T_total = sh->T_total;
    p.h_qk = sh->h_qk;
    p.h_v = sh->h_v;
    p.dk = sh->dk;
    p.dv = sh->dv;
    p.T_fixed = cu ? 0 : sh->T_total / sh->n_seq;
    p.q = q; p.k = k; p.v = v; p.log_alpha = la; p.b = b; p.w = w;
    p.S0 = S0; p.cu_seqlens = cu; p.o = o; p.S_T = S_T; p.order = nullptr;
    p.n_tok = 1; p.slots = nullptr; p.n_slots = sh->n_seq; p.S_steps = nullptr;
    p.wait_ns = g_wait_ns.load(std::memory_order_relaxed);
    p.test_withhold_loads = g_withhold.load(std::memory_order_relaxed);
    return p;
}

}  // namespace

gdn2_status report_error(gdn2_status st, const char* msg) { return fail(st, "%s", msg); }

}  // namespace gdn2

using namespace gdn2;

extern "C" {

const char* gdn2_last_error_string(void) { return g_err; }

int gdn2_version(void) { return 210; }

gdn2_status gdn2_device_status(unsigned int* flags, gdn2_stream_t stream) {
    if (!flags) return fail(GDN2_ERR_INVALID_ARG, "flags is NULL");
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    unsigned int w[5] = {0u, 0u, 0u, 0u, 0u};
    cudaError_t e = cudaStreamSynchronize(s);  // the work queued so far has run
    if (e == cudaSuccess) e = read_clear_status_chunk_tc(&w[0], s);
    if (e == cudaSuccess) e = read_clear_status_recurrent(&w[1], s);
    if (e == cudaSuccess) e = read_clear_status_schedule(&w[2], s);
    if (e == cudaSuccess) e = read_clear_status_decode(&w[3], s);
    if (e == cudaSuccess) e = read_clear_status_decode_q8(&w[4], s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);  // the reads have landed in w
    if (e != cudaSuccess) return fail(GDN2_ERR_CUDA, "device status: %s", cudaGetErrorString(e));
    *flags = w[0] | w[1] | w[2] | w[3] | w[4];
    return ok();
}

void gdn2_testing_set_wait_limit(unsigned long long wait_ns, int withhold_first_load) {
    g_wait_ns.store(wait_ns ? wait_ns : kDefaultWaitNs, std::memory_order_relaxed);
    g_withhold.store(withhold_first_load ? 1 : 0, std::memory_order_relaxed);
}

size_t gdn2_chunk_fwd_workspace_size(const gdn2_shape* shape, int varlen) {
    if (!shape || !varlen || shape->n_seq < 1) return 0;
    // the longest-first order of the sequences, 256-byte rounded
    return ((size_t)shape->n_seq * sizeof(int32_t) + 255) & ~(size_t)255;
}

}  // extern "C"

namespace {

// gdn2_chunk_fwd and gdn2_chunk_fwd_prologue: with prologue, la is the dtype decay
// pre-activation instead of fp32 log_alpha.
gdn2_status chunk_fwd(bool prologue, const gdn2_shape* shape, const void* q, const void* k, const void* v,
                      const void* la, const void* b, const void* w, const float* S0, const int32_t* cu_seqlens,
                      void* o, float* S_T, void* workspace, size_t workspace_bytes, gdn2_stream_t stream) {
    gdn2_status st = check_shape(shape);
    if (st != GDN2_OK) return st;
    const bool any_tokens = shape->T_total > 0;
    const NamedPtr ps[] = {
        {"q", q, any_tokens}, {"k", k, any_tokens}, {"v", v, any_tokens},
        {prologue ? "a" : "log_alpha", la, any_tokens}, {"b", b, any_tokens}, {"w", w, any_tokens},
        {"o", o, any_tokens}, {"S0", S0, false}, {"S_T", S_T, false},
        {"cu_seqlens", cu_seqlens, false}, {"workspace", workspace, false},
    };
    st = check_ptrs(ps, (int)(sizeof ps / sizeof ps[0]));
    if (st != GDN2_OK) return st;
    if (!cu_seqlens && shape->T_total % shape->n_seq != 0)
        return fail(GDN2_ERR_INVALID_ARG, "T_total = %d is not a multiple of n_seq = %d (and no cu_seqlens)",
                    shape->T_total, shape->n_seq);
    const size_t need = gdn2_chunk_fwd_workspace_size(shape, cu_seqlens != nullptr);
    if (need && (!workspace || workspace_bytes < need))
        return fail(GDN2_ERR_INVALID_ARG, "workspace of %zu bytes needed, %zu given", need,
                    workspace ? workspace_bytes : (size_t)0);
    if (workspace && (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return fail(GDN2_ERR_INVALID_ARG, "workspace is not 256-byte aligned");

    Params p = make_params(shape, q, k, v, prologue ? nullptr : static_cast<const float*>(la), b, w, S0,
                           cu_seqlens, o, S_T);
    p.prologue = prologue;
    p.a_raw = prologue ? la : nullptr;
    if (prologue && any_tokens && !chunk_tc_supported(p, shape->dtype))
        return fail(GDN2_ERR_UNSUPPORTED, "the fused pre-processing needs bf16 inputs with dk = dv = 128");
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (cu_seqlens) {
        int32_t* order = static_cast<int32_t*>(workspace);
        cudaError_t e = launch_varlen_order(p, order, s);
        if (e != cudaSuccess) return fail(GDN2_ERR_CUDA, "order kernel: %s", cudaGetErrorString(e));
        p.order = order;
    }
    cudaError_t e = chunk_tc_supported(p, shape->dtype) ? launch_chunk_tc(p, shape->o_dtype, s)
                                                        : launch_recurrent(p, shape->dtype, shape->o_dtype, s);
    if (e != cudaSuccess) return fail(GDN2_ERR_CUDA, "chunk kernel launch: %s", cudaGetErrorString(e));
    return ok();
}

}  // namespace

extern "C" {

gdn2_status gdn2_chunk_fwd(const gdn2_shape* shape, const void* q, const void* k, const void* v,
                           const float* log_alpha, const void* b, const void* w, const float* S0,
                           const int32_t* cu_seqlens, void* o, float* S_T, void* workspace,
                           size_t workspace_bytes, gdn2_stream_t stream) {
    return chunk_fwd(false, shape, q, k, v, log_alpha, b, w, S0, cu_seqlens, o, S_T, workspace, workspace_bytes,
                     stream);
}

gdn2_status gdn2_chunk_fwd_prologue(const gdn2_shape* shape, const void* q_raw, const void* k_raw, const void* v,
                                    const void* a_raw, const void* b_raw, const void* w_raw, const float* S0,
                                    const int32_t* cu_seqlens, void* o, float* S_T, void* workspace,
                                    size_t workspace_bytes, gdn2_stream_t stream) {
    return chunk_fwd(true, shape, q_raw, k_raw, v, a_raw, b_raw, w_raw, S0, cu_seqlens, o, S_T, workspace,
                     workspace_bytes, stream);
}

gdn2_status gdn2_decode_step(const gdn2_shape* shape, const void* q, const void* k, const void* v,
                             const float* log_alpha, const void* b, const void* w, float* S, void* o,
                             gdn2_stream_t stream) {
    gdn2_status st = check_shape(shape);
    if (st != GDN2_OK) return st;
    if (shape->T_total != shape->n_seq)
        return fail(GDN2_ERR_INVALID_ARG, "decode takes one token per sequence: T_total = %d, n_seq = %d",
                    shape->T_total, shape->n_seq);
    if ((long long)shape->n_seq * shape->h_v > 0x7fffffffLL)
        return fail(GDN2_ERR_UNSUPPORTED, "n_seq * h_v too large for one launch");
    const NamedPtr ps[] = {
        {"q", q, true}, {"k", k, true}, {"v", v, true}, {"log_alpha", log_alpha, true},
        {"b", b, true}, {"w", w, true}, {"S", S, true}, {"o", o, true},
    };
    st = check_ptrs(ps, (int)(sizeof ps / sizeof ps[0]));
    if (st != GDN2_OK) return st;
    Params p = make_params(shape, q, k, v, log_alpha, b, w, nullptr, nullptr, o, S);
    cudaError_t e = launch_decode(p, shape->dtype, shape->o_dtype, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return fail(GDN2_ERR_CUDA, "decode kernel launch: %s", cudaGetErrorString(e));
    return ok();
}

}  // extern "C"

namespace {

// What the serving decodes ask of their shape, token count and pool.
gdn2_status check_serving(const gdn2_shape* shape, int n_tok, const int32_t* slots, int n_slots) {
    gdn2_status st = check_shape(shape);
    if (st != GDN2_OK) return st;
    if (n_tok < 1 || n_tok > GDN2_DECODE_MAX_TOKENS)
        return fail(GDN2_ERR_INVALID_ARG, "n_tok = %d outside 1..%d", n_tok, GDN2_DECODE_MAX_TOKENS);
    if ((long long)shape->n_seq * n_tok != shape->T_total)
        return fail(GDN2_ERR_INVALID_ARG, "T_total = %d is not n_seq * n_tok = %d * %d", shape->T_total,
                    shape->n_seq, n_tok);
    if (n_slots < 1 || (!slots && n_slots < shape->n_seq))
        return fail(GDN2_ERR_INVALID_ARG, "n_slots = %d too small (n_seq = %d, slots %s)", n_slots, shape->n_seq,
                    slots ? "given" : "NULL");
    // the kernels go from pair to pair by adding their grid (a few CTAs per SM) in 32 bits
    if ((long long)shape->n_seq * shape->h_v > 0x7fffffffLL - 0xffff)
        return fail(GDN2_ERR_UNSUPPORTED, "n_seq * h_v = %lld (sequence, head) pairs above 2^31 - 2^16",
                    (long long)shape->n_seq * shape->h_v);
    return GDN2_OK;
}

gdn2_status decode_multi(bool prologue, const gdn2_shape* shape, int n_tok, const int32_t* slots, const void* q,
                         const void* k, const void* v, const void* la, const void* b, const void* w, float* S_pool,
                         int n_slots, void* o, float* S_steps, gdn2_stream_t stream) {
    gdn2_status st = check_serving(shape, n_tok, slots, n_slots);
    if (st != GDN2_OK) return st;
    if ((long long)shape->n_seq * shape->h_v > 0x7fffffffLL || (long long)n_slots * shape->h_v > 0x7fffffffLL)
        return fail(GDN2_ERR_UNSUPPORTED, "n_seq * h_v or n_slots * h_v too large for one launch");
    if ((long long)n_slots * shape->h_v * shape->dk > 0x7fffffffLL)  // state rows, addressed by TMA
        return fail(GDN2_ERR_UNSUPPORTED, "n_slots * h_v * dk = %lld state rows, above 2^31 - 1",
                    (long long)n_slots * shape->h_v * shape->dk);
    const NamedPtr ps[] = {
        {"q", q, true}, {"k", k, true}, {"v", v, true}, {prologue ? "a" : "log_alpha", la, true}, {"b", b, true},
        {"w", w, true}, {"S_pool", S_pool, true}, {"o", o, true}, {"slots", slots, false},
        {"S_steps", S_steps, false},
    };
    st = check_ptrs(ps, (int)(sizeof ps / sizeof ps[0]));
    if (st != GDN2_OK) return st;
    Params p = make_params(shape, q, k, v, prologue ? nullptr : static_cast<const float*>(la), b, w, nullptr,
                           nullptr, o, S_pool);
    p.prologue = prologue;
    p.a_raw = prologue ? la : nullptr;
    p.n_tok = n_tok;
    p.slots = slots;
    p.n_slots = n_slots;
    p.S_steps = S_steps;
    cudaError_t e = launch_decode(p, shape->dtype, shape->o_dtype, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return fail(GDN2_ERR_CUDA, "decode kernel launch: %s", cudaGetErrorString(e));
    return ok();
}

}  // namespace

extern "C" {

gdn2_status gdn2_decode_multi(const gdn2_shape* shape, int n_tok, const int32_t* slots, const void* q,
                              const void* k, const void* v, const float* log_alpha, const void* b, const void* w,
                              float* S_pool, int n_slots, void* o, float* S_steps, gdn2_stream_t stream) {
    return decode_multi(false, shape, n_tok, slots, q, k, v, log_alpha, b, w, S_pool, n_slots, o, S_steps, stream);
}

gdn2_status gdn2_decode_multi_prologue(const gdn2_shape* shape, int n_tok, const int32_t* slots, const void* q_raw,
                                       const void* k_raw, const void* v, const void* a_raw, const void* b_raw,
                                       const void* w_raw, float* S_pool, int n_slots, void* o, float* S_steps,
                                       gdn2_stream_t stream) {
    return decode_multi(true, shape, n_tok, slots, q_raw, k_raw, v, a_raw, b_raw, w_raw, S_pool, n_slots, o, S_steps,
                        stream);
}

size_t gdn2_chunk_bwd_workspace_size(const gdn2_shape* shape) {
    if (!shape || shape->n_seq < 1 || shape->T_total < 0 || shape->h_v < 1 || shape->dk < 1 || shape->dv < 1) return 0;
    return (bwd_workspace_bytes(shape) + 255) & ~(size_t)255;
}

gdn2_status gdn2_chunk_bwd(const gdn2_shape* shape, const void* q, const void* k, const void* v,
                           const float* log_alpha, const void* b, const void* w, const float* S0,
                           const int32_t* cu_seqlens, const float* dO, const float* dS_T, float* dq, float* dk,
                           float* dv, float* dlog_alpha, float* db, float* dw, float* dS0, void* workspace,
                           size_t workspace_bytes, gdn2_stream_t stream) {
    gdn2_status st = check_shape(shape);
    if (st != GDN2_OK) return st;
    const bool any = shape->T_total > 0;
    const NamedPtr ps[] = {
        {"q", q, any}, {"k", k, any}, {"v", v, any}, {"log_alpha", log_alpha, any}, {"b", b, any},
        {"w", w, any}, {"dO", dO, any}, {"dq", dq, any}, {"dk", dk, any}, {"dv", dv, any},
        {"dlog_alpha", dlog_alpha, any}, {"db", db, any}, {"dw", dw, any}, {"S0", S0, false},
        {"cu_seqlens", cu_seqlens, false}, {"dS_T", dS_T, false}, {"dS0", dS0, false},
        {"workspace", workspace, false},
    };
    st = check_ptrs(ps, (int)(sizeof ps / sizeof ps[0]));
    if (st != GDN2_OK) return st;
    if (!cu_seqlens && shape->T_total % shape->n_seq != 0)
        return fail(GDN2_ERR_INVALID_ARG, "T_total = %d is not a multiple of n_seq = %d (and no cu_seqlens)",
                    shape->T_total, shape->n_seq);
    const size_t need = gdn2_chunk_bwd_workspace_size(shape);
    if (!workspace || workspace_bytes < need)
        return fail(GDN2_ERR_INVALID_ARG, "workspace of %zu bytes needed, %zu given", need,
                    workspace ? workspace_bytes : (size_t)0);
    if (reinterpret_cast<uintptr_t>(workspace) & 255u)
        return fail(GDN2_ERR_INVALID_ARG, "workspace is not 256-byte aligned");
    Params p = make_params(shape, q, k, v, log_alpha, b, w, S0, cu_seqlens, nullptr, nullptr);
    if (cu_seqlens) {
        cudaError_t ec = launch_check_seqlens(p, reinterpret_cast<cudaStream_t>(stream));
        if (ec != cudaSuccess) return fail(GDN2_ERR_CUDA, "cu_seqlens check kernel: %s", cudaGetErrorString(ec));
    }
    cudaError_t e = launch_bwd(p, shape->dtype, dO, dS_T, dq, dk, dv, dlog_alpha, db, dw, dS0, workspace,
                               reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return fail(GDN2_ERR_CUDA, "backward kernel launch: %s", cudaGetErrorString(e));
    return ok();
}

}  // extern "C"

// ---------------------------------------------------------------- around the state pool
namespace {

gdn2_status check_states(int n_seq, int h_v, int dk, int dv, const int32_t* slots, int n_slots) {
    const gdn2_shape sh{n_seq, 0, 1, h_v, dk, dv, GDN2_F32, GDN2_F32};
    gdn2_status st = check_shape(&sh);
    if (st != GDN2_OK) return st;
    if (n_slots < 1 || (!slots && n_slots < n_seq))
        return fail(GDN2_ERR_INVALID_ARG, "n_slots = %d too small (n_seq = %d, slots %s)", n_slots, n_seq,
                    slots ? "given" : "NULL");
    return GDN2_OK;
}

gdn2_status check_format(gdn2_q8_format fmt) {
    if (fmt != GDN2_Q8_INT8 && fmt != GDN2_Q8_E4M3) return fail(GDN2_ERR_INVALID_ARG, "unknown 8-bit format %d", (int)fmt);
    return GDN2_OK;
}

gdn2_status state_cache(bool store, int n_seq, int h_v, int dk, int dv, gdn2_q8_format fmt, float* S, const int32_t* slots,
                        void* codes, float* scales, int n_slots, gdn2_stream_t stream) {
    gdn2_status st = check_states(n_seq, h_v, dk, dv, slots, n_slots);
    if (st == GDN2_OK) st = check_format(fmt);
    if (st != GDN2_OK) return st;
    if ((long long)n_seq * h_v > 0x3fffffffLL)  // two CTAs per state
        return fail(GDN2_ERR_UNSUPPORTED, "n_seq * h_v = %lld states, above 2^30 - 1", (long long)n_seq * h_v);
    const NamedPtr ps[] = {{"S", S, true}, {"codes", codes, true}, {"scales", scales, true}, {"slots", slots, false, 4}};
    st = check_ptrs(ps, (int)(sizeof ps / sizeof ps[0]));
    if (st != GDN2_OK) return st;
    const StateCacheArgs a{n_seq, h_v, dk, dv, n_slots, S, slots, codes, scales};
    cudaError_t e = launch_state_cache(store, a, fmt, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return fail(GDN2_ERR_CUDA, "state %s kernel launch: %s", store ? "store" : "load", cudaGetErrorString(e));
    return ok();
}

gdn2_status state_commit(bool q8, int n_seq, int h_v, int dk, int dv, int n_tok, const void* steps, const float* step_scales,
                         const int32_t* index, const int32_t* slots, void* pool, float* scales, int n_slots,
                         gdn2_stream_t stream) {
    gdn2_status st = check_states(n_seq, h_v, dk, dv, slots, n_slots);
    if (st != GDN2_OK) return st;
    if (n_tok < 1 || n_tok > GDN2_DECODE_MAX_TOKENS)
        return fail(GDN2_ERR_INVALID_ARG, "n_tok = %d outside 1..%d", n_tok, GDN2_DECODE_MAX_TOKENS);
    const NamedPtr ps[] = {{q8 ? "code_steps" : "S_steps", steps, true}, {"scale_steps", step_scales, q8}, {"index", index, true, 4},
                           {"slots", slots, false, 4}, {q8 ? "codes" : "S_pool", pool, true}, {"scales", scales, q8}};
    st = check_ptrs(ps, (int)(sizeof ps / sizeof ps[0]));
    if (st != GDN2_OK) return st;
    const size_t elts = (size_t)h_v * dk * dv, rows = (size_t)h_v * dk;
    cudaError_t e = launch_state_commit(steps, step_scales, index, slots, pool, scales, n_seq, n_tok, n_slots, q8 ? elts : 4 * elts,
                                        q8 ? 4 * rows : 0, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return fail(GDN2_ERR_CUDA, "state commit kernel launch: %s", cudaGetErrorString(e));
    return ok();
}

gdn2_status decode_multi_q8(bool prologue, const gdn2_shape* shape, gdn2_q8_format fmt, int n_tok, const int32_t* slots,
                            const int32_t* slots_out, const void* q, const void* k, const void* v, const void* la,
                            const void* b, const void* w, void* codes, float* scales, int n_slots, void* o,
                            void* code_steps, float* scale_steps, gdn2_stream_t stream) {
    gdn2_status st = check_serving(shape, n_tok, slots, n_slots);
    if (st == GDN2_OK) st = check_format(fmt);
    if (st != GDN2_OK) return st;
    if ((code_steps == nullptr) != (scale_steps == nullptr))
        return fail(GDN2_ERR_INVALID_ARG, "code_steps and scale_steps are given together or not at all");
    const NamedPtr ps[] = {
        {"q", q, true}, {"k", k, true}, {"v", v, true}, {prologue ? "a" : "log_alpha", la, true}, {"b", b, true},
        {"w", w, true}, {"codes", codes, true}, {"scales", scales, true}, {"o", o, true}, {"slots", slots, false, 4},
        {"slots_out", slots_out, false, 4}, {"code_steps", code_steps, false}, {"scale_steps", scale_steps, false},
    };
    st = check_ptrs(ps, (int)(sizeof ps / sizeof ps[0]));
    if (st != GDN2_OK) return st;
    Params p = make_params(shape, q, k, v, prologue ? nullptr : static_cast<const float*>(la), b, w, nullptr, nullptr, o,
                           nullptr);
    p.prologue = prologue;
    p.a_raw = prologue ? la : nullptr;
    p.n_tok = n_tok;
    p.slots = slots;
    p.n_slots = n_slots;
    const Q8Args a{fmt, shape->dtype == GDN2_BF16, shape->o_dtype == GDN2_BF16, slots_out, codes, scales, code_steps, scale_steps};
    cudaError_t e = launch_decode_q8(p, a, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return fail(GDN2_ERR_CUDA, "8-bit decode kernel launch: %s", cudaGetErrorString(e));
    return ok();
}

}  // namespace

extern "C" {

gdn2_status gdn2_state_store(int n_seq, int h_v, int dk, int dv, gdn2_q8_format format, const float* S, const int32_t* slots,
                             void* codes, float* scales, int n_slots, gdn2_stream_t stream) {
    return state_cache(true, n_seq, h_v, dk, dv, format, const_cast<float*>(S), slots, codes, scales, n_slots, stream);
}

gdn2_status gdn2_state_load(int n_seq, int h_v, int dk, int dv, gdn2_q8_format format, const void* codes, const float* scales,
                            int n_slots, const int32_t* slots, float* S, gdn2_stream_t stream) {
    return state_cache(false, n_seq, h_v, dk, dv, format, S, slots, const_cast<void*>(codes), const_cast<float*>(scales), n_slots,
                       stream);
}

gdn2_status gdn2_decode_multi_q8(const gdn2_shape* shape, gdn2_q8_format format, int n_tok, const int32_t* slots,
                                 const int32_t* slots_out, const void* q, const void* k, const void* v, const float* log_alpha,
                                 const void* b, const void* w, void* codes, float* scales, int n_slots, void* o,
                                 void* code_steps, float* scale_steps, gdn2_stream_t stream) {
    return decode_multi_q8(false, shape, format, n_tok, slots, slots_out, q, k, v, log_alpha, b, w, codes, scales, n_slots, o,
                           code_steps, scale_steps, stream);
}

gdn2_status gdn2_decode_multi_q8_prologue(const gdn2_shape* shape, gdn2_q8_format format, int n_tok, const int32_t* slots,
                                          const int32_t* slots_out, const void* q_raw, const void* k_raw, const void* v,
                                          const void* a_raw, const void* b_raw, const void* w_raw, void* codes, float* scales,
                                          int n_slots, void* o, void* code_steps, float* scale_steps, gdn2_stream_t stream) {
    return decode_multi_q8(true, shape, format, n_tok, slots, slots_out, q_raw, k_raw, v, a_raw, b_raw, w_raw, codes, scales,
                           n_slots, o, code_steps, scale_steps, stream);
}

gdn2_status gdn2_state_commit(int n_seq, int h_v, int dk, int dv, int n_tok, const float* S_steps, const int32_t* index,
                              const int32_t* slots, float* S_pool, int n_slots, gdn2_stream_t stream) {
    return state_commit(false, n_seq, h_v, dk, dv, n_tok, S_steps, nullptr, index, slots, S_pool, nullptr, n_slots, stream);
}

gdn2_status gdn2_state_commit_q8(int n_seq, int h_v, int dk, int dv, int n_tok, const void* code_steps, const float* scale_steps,
                                 const int32_t* index, const int32_t* slots, void* codes, float* scales, int n_slots,
                                 gdn2_stream_t stream) {
    return state_commit(true, n_seq, h_v, dk, dv, n_tok, code_steps, scale_steps, index, slots, codes, scales, n_slots, stream);
}

gdn2_status gdn2_verify_drafts(int n_seq, int n_draft, int vocab, gdn2_dtype dtype, const void* target_probs, const void* draft_probs,
                               const int32_t* draft_tokens, const int32_t* n_drafted, const float* u_accept,
                               const float* u_sample, int32_t* n_accepted, int32_t* tokens, gdn2_stream_t stream) {
    if (n_seq < 1 || n_seq > 65535) return fail(GDN2_ERR_INVALID_ARG, "n_seq = %d outside [1, 65535]", n_seq);
    if (n_draft < 0) return fail(GDN2_ERR_INVALID_ARG, "n_draft = %d is negative", n_draft);
    if (n_draft > GDN2_VERIFY_MAX_DRAFTS)
        return fail(GDN2_ERR_UNSUPPORTED, "n_draft = %d above %d", n_draft, GDN2_VERIFY_MAX_DRAFTS);
    if (vocab < 1) return fail(GDN2_ERR_INVALID_ARG, "vocab = %d must be positive", vocab);
    if (vocab > GDN2_VERIFY_MAX_VOCAB) return fail(GDN2_ERR_UNSUPPORTED, "vocab = %d above %d", vocab, GDN2_VERIFY_MAX_VOCAB);
    if (dtype != GDN2_F32 && dtype != GDN2_BF16) return fail(GDN2_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    const bool drafts = n_draft > 0;
    const unsigned es = dtype == GDN2_F32 ? 4 : 2;
    const NamedPtr ps[] = {
        {"target_probs", target_probs, true, es}, {"draft_probs", drafts ? draft_probs : nullptr, false, es},
        {"draft_tokens", drafts ? draft_tokens : nullptr, drafts, 4}, {"n_drafted", n_drafted, false, 4},
        {"u_accept", drafts ? u_accept : nullptr, drafts, 4}, {"u_sample", u_sample, true, 4},
        {"n_accepted", n_accepted, true, 4}, {"tokens", tokens, true, 4},
    };
    gdn2_status st = check_ptrs(ps, (int)(sizeof ps / sizeof ps[0]));
    if (st != GDN2_OK) return st;
    const VerifyArgs a{n_seq, n_draft, vocab, target_probs, drafts ? draft_probs : nullptr, draft_tokens, n_drafted, u_accept,
                       u_sample, n_accepted, tokens};
    cudaError_t e = launch_verify(a, dtype, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return fail(GDN2_ERR_CUDA, "verification kernel launch: %s", cudaGetErrorString(e));
    return ok();
}

}  // extern "C"
