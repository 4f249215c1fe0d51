// state_cache.cu -- states moved between fp32 buffers, per-token states and the slots of a pool:
// quantised on the way into an 8-bit pool (gdn2_state_store), read back (gdn2_state_load), and
// the state after the last accepted token put back (gdn2_state_commit, gdn2_state_commit_q8).
//
// All of these are bound by HBM: 5 bytes a state element for store and load, twice the state's
// own bytes for commit; nothing is read twice. Measured on B200: 256 x 32 states of 128 x 128
// stored and loaded in 206 us (1.35 GB, 6.56 TB/s), 185 x 32 fp32 states committed in 120 us
// (0.78 GB, 6.46 TB/s).
#include "q8.cuh"

namespace gdn2 {
namespace {

constexpr int kThreads = 256;
constexpr int kParts = 2;  // CTAs per state (store, load)

// ---------------------------------------------------------------- store, load
// A CTA per half of a (sequence, value head)'s key rows: 61 x 16 states take 25.2 us stored and loaded, 27.4
// with a whole state per CTA (fewer, longer waves), 26.5 with a quarter. (The halves are neighbours in
// the grid: half a grid apart, 256 x 32 states take 215 us instead of 206.) A thread holds four
// neighbouring columns (a float4, four codes) of its rows, so a warp's access covers whole rows: 512
// bytes of state, 128 of codes. All loads are issued before the first use. The row's
// largest magnitude is taken over the 16 or 32 lanes that share the row: shuffles and quotients are
// repeated in each of them, which the memory time hides.
template <int DK, int DV, int kFmt>
__global__ void __launch_bounds__(kThreads) state_store_kernel(const float* __restrict__ S, const int32_t* __restrict__ slots,
                                                               uint32_t* __restrict__ codes, float* __restrict__ scales,
                                                               int n_slots, int h_v) {
    constexpr int TPR = DV / 4, RG = kThreads / TPR, ROWS = DK / kParts, RPT = ROWS / RG;
    const int item = blockIdx.x / kParts, first = blockIdx.x % kParts * ROWS, n = item / h_v, h = item % h_v;
    const int slot = slots ? slots[n] : n;
    if (slot < 0 || slot >= n_slots) return;  // no slot: nothing to keep
    const int cg = threadIdx.x % TPR, rg = threadIdx.x / TPR;
    const float4* src = reinterpret_cast<const float4*>(S) + ((size_t)item * DK + first) * TPR + cg;
    const size_t row0 = ((size_t)slot * h_v + h) * DK + first;
    float4 s[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i) s[i] = __ldcs(src + (rg + RG * i) * TPR);
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        uint32_t m = max(max(mag_bits(s[i].x), mag_bits(s[i].y)), max(mag_bits(s[i].z), mag_bits(s[i].w)));
#pragma unroll
        for (int off = TPR / 2; off > 0; off >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
        float scale, inv;
        q8_scale<kFmt>(__uint_as_float(m), scale, inv);
        const size_t row = row0 + rg + RG * i;
        codes[row * TPR + cg] = q8_pack<kFmt>(s[i], inv);
        if (cg == 0) scales[row] = scale;
    }
}

template <int DK, int DV, int kFmt>
__global__ void __launch_bounds__(kThreads) state_load_kernel(const uint32_t* __restrict__ codes, const float* __restrict__ scales,
                                                              const int32_t* __restrict__ slots, float* __restrict__ S,
                                                              int n_slots, int h_v) {
    constexpr int TPR = DV / 4, RG = kThreads / TPR, ROWS = DK / kParts, RPT = ROWS / RG;
    const int item = blockIdx.x / kParts, first = blockIdx.x % kParts * ROWS, n = item / h_v, h = item % h_v;
    const int slot = slots ? slots[n] : n;
    const int cg = threadIdx.x % TPR, rg = threadIdx.x / TPR;
    float4* dst = reinterpret_cast<float4*>(S) + ((size_t)item * DK + first) * TPR + cg;
    if (slot < 0 || slot >= n_slots) {  // nothing kept: the sequence starts from the zero state
#pragma unroll
        for (int i = 0; i < RPT; ++i) __stcs(dst + (rg + RG * i) * TPR, make_float4(0.f, 0.f, 0.f, 0.f));
        return;
    }
    const size_t row0 = ((size_t)slot * h_v + h) * DK + first;
    uint32_t c[RPT];
    float sc[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        c[i] = __ldcs(codes + (row0 + rg + RG * i) * TPR + cg);
        sc[i] = __ldcs(scales + row0 + rg + RG * i);
    }
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const float4 x = q8_unpack<kFmt>(c[i]);
        __stcs(dst + (rg + RG * i) * TPR, make_float4(x.x * sc[i], x.y * sc[i], x.z * sc[i], x.w * sc[i]));
    }
}

// ---------------------------------------------------------------- commit
// A sequence's heads are contiguous in the pool and in the per-token states, so this is a copy of
// one block a sequence (two with 8-bit states: codes, scales), cut into pieces of kPiece bytes.
constexpr int kPiece = kThreads * 16 * 8;  // 8 16-byte loads in flight per thread

__global__ void __launch_bounds__(kThreads) state_commit_kernel(const char* __restrict__ steps, const char* __restrict__ step_scales,
                                                                const int32_t* __restrict__ index, const int32_t* __restrict__ slots,
                                                                char* __restrict__ pool, char* __restrict__ scales, int n_tok,
                                                                int n_slots, size_t bytes, size_t scale_bytes, int pieces) {
    const int n = blockIdx.y;
    const int slot = slots ? slots[n] : n, t = index[n];
    if (slot < 0 || slot >= n_slots || t < 0 || t >= n_tok) return;  // the slot stays as it is
    const bool second = (int)blockIdx.x >= pieces;  // the scales' pieces come after the states'
    const size_t total = second ? scale_bytes : bytes;
    const size_t off = (size_t)(blockIdx.x - (second ? pieces : 0)) * kPiece;
    const char* src = (second ? step_scales : steps) + ((size_t)n * n_tok + t) * total + off;
    char* dst = (second ? scales : pool) + (size_t)slot * total + off;
    const int left = (int)min((size_t)kPiece, total - off) / 16;
    uint4 x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if ((int)threadIdx.x + i * kThreads < left) x[i] = __ldcs(reinterpret_cast<const uint4*>(src) + threadIdx.x + i * kThreads);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if ((int)threadIdx.x + i * kThreads < left) reinterpret_cast<uint4*>(dst)[threadIdx.x + i * kThreads] = x[i];
}

template <int DK, int DV, int kFmt>
cudaError_t launch_cache_t(bool store, const StateCacheArgs& a, cudaStream_t st) {
    const int grid = kParts * a.n_seq * a.h_v;
    if (store)
        state_store_kernel<DK, DV, kFmt><<<grid, kThreads, 0, st>>>(a.S, a.slots, static_cast<uint32_t*>(a.codes), a.scales, a.n_slots, a.h_v);
    else
        state_load_kernel<DK, DV, kFmt><<<grid, kThreads, 0, st>>>(static_cast<const uint32_t*>(a.codes), a.scales, a.slots, a.S, a.n_slots, a.h_v);
    return cudaGetLastError();
}

template <int kFmt>
cudaError_t launch_cache_f(bool store, const StateCacheArgs& a, cudaStream_t st) {
    if (a.dk == 128) return a.dv == 128 ? launch_cache_t<128, 128, kFmt>(store, a, st) : launch_cache_t<128, 64, kFmt>(store, a, st);
    return a.dv == 128 ? launch_cache_t<64, 128, kFmt>(store, a, st) : launch_cache_t<64, 64, kFmt>(store, a, st);
}

}  // namespace

cudaError_t launch_state_cache(bool store, const StateCacheArgs& a, gdn2_q8_format fmt, cudaStream_t st) {
    return fmt == GDN2_Q8_INT8 ? launch_cache_f<GDN2_Q8_INT8>(store, a, st) : launch_cache_f<GDN2_Q8_E4M3>(store, a, st);
}

cudaError_t launch_state_commit(const void* steps, const float* step_scales, const int32_t* index, const int32_t* slots, void* pool,
                                float* scales, int n_seq, int n_tok, int n_slots, size_t bytes, size_t scale_bytes, cudaStream_t st) {
    const int pieces = (int)((bytes + kPiece - 1) / kPiece), more = (int)((scale_bytes + kPiece - 1) / kPiece);
    state_commit_kernel<<<dim3(pieces + more, n_seq), kThreads, 0, st>>>(
        static_cast<const char*>(steps), reinterpret_cast<const char*>(step_scales), index, slots, static_cast<char*>(pool),
        reinterpret_cast<char*>(scales), n_tok, n_slots, bytes, scale_bytes, pieces);
    return cudaGetLastError();
}

}  // namespace gdn2
