// verify.cu -- verification of drafted tokens against the target's probabilities, from given
// random numbers (gdn2_verify_drafts).
//
// Of sequence n's drafted tokens t_0 .. t_{m-1}, token i is accepted while u_i q_i(t_i) < p_i(t_i).
// The first one that is not is replaced by a token of the residual r = max(p_i - q_i, 0) (of p_i
// where r is empty); with all accepted one more token comes from p_m. Tokens are drawn by inverse
// CDF: the lowest j with r_0 + .. + r_j > u (r_0 + .. + r_{V-1}).
//
// Everything is computed in fp64 from the exact values of the inputs: u q is exact (24 + 24 bits), and a
// sum's rounding, ~1e-16, all but never crosses a border of the CDF, so the order of the sums does not show
// in the tokens.
//
// The work is one row of p and one of q a sequence.
#include "internal.cuh"

namespace gdn2 {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kSeg = 1024;                                 // values per segment of the CDF
constexpr int kMaxSeg = GDN2_VERIFY_MAX_VOCAB / kSeg;

enum Mode { kPlain, kResidual, kOneHot };

__device__ __forceinline__ double clean(float x) { return x > 0.f && x <= 3.402823466e38f ? (double)x : 0.0; }

// The weight of token j in the row that the token is drawn from.
template <typename T>
struct Row {
    const T* p;
    const T* q;
    int t, mode;
    __device__ __forceinline__ double at(int j) const {
        const double x = clean(to_f32(p[j]));
        if (mode == kResidual) return fmax(x - clean(to_f32(q[j])), 0.0);
        return mode == kOneHot && j == t ? 0.0 : x;
    }
};

__device__ __forceinline__ double warp_sum(double x) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}
__device__ __forceinline__ double warp_scan(double x, int lane) {  // inclusive
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
    }
    return x;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) verify_kernel(const __grid_constant__ VerifyArgs a) {
    __shared__ double seg_sum[kMaxSeg];
    __shared__ double wsum[kWarps];
    __shared__ int s_taken, s_mode, s_found, s_last;
    __shared__ double s_total;
    const int n = blockIdx.x, tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int V = a.vocab, k = a.n_draft;
    int m = a.n_drafted ? a.n_drafted[n] : k;
    int* tokens = a.tokens + (size_t)n * (k + 1);
    if (m < 0) {  // an inactive sequence
        for (int i = tid; i <= k; i += kThreads) tokens[i] = -1;
        if (tid == 0) a.n_accepted[n] = -1;
        return;
    }
    m = min(m, k);
    const T* P = static_cast<const T*>(a.p) + (size_t)n * (k + 1) * V;
    const T* Q = a.q ? static_cast<const T*>(a.q) + (size_t)n * k * V : nullptr;
    const int* drafts = a.drafts + (size_t)n * k;
    if (warp == 0) {  // lane i: drafted token i
        bool yes = false;
        if (lane < m) {
            const int t = drafts[lane];
            if (t >= 0 && t < V) {
                const double pt = clean(to_f32(P[(size_t)lane * V + t])), qt = Q ? clean(to_f32(Q[(size_t)lane * V + t])) : 1.0;
                yes = (double)a.u_accept[(size_t)n * k + lane] * qt < pt;
            }
        }
        const unsigned no = ~__ballot_sync(0xffffffffu, yes);  // lane m's bit is set: m <= 31
        if (lane == 0) s_taken = __ffs(no) - 1;
    }
    __syncthreads();
    const int taken = s_taken;
    const bool refused = taken < m;
    Row<T> row{P + (size_t)taken * V, refused && Q ? Q + (size_t)taken * V : nullptr, refused ? drafts[taken] : -1,
               !refused ? kPlain : (Q ? kResidual : kOneHot)};
    const int segs = (V + kSeg - 1) / kSeg;
    double total;
    for (;;) {
        for (int s = warp; s < segs; s += kWarps) {
            double x = 0.0;
            const int end = min(V, (s + 1) * kSeg);
            for (int j = s * kSeg + lane; j < end; j += 32) x += row.at(j);
            x = warp_sum(x);
            if (lane == 0) seg_sum[s] = x;
        }
        __syncthreads();
        if (warp == 0) {
            double x = 0.0;
            for (int s = lane; s < segs; s += 32) x += seg_sum[s];
            x = warp_sum(x);
            if (lane == 0) s_total = x;
        }
        __syncthreads();
        total = s_total;
        if (total > 0.0 || row.mode == kPlain) break;
        row.mode = kPlain;  // nothing is left of the row: its own probabilities
    }
    int token = -1;
    if (total > 0.0) {
        const double u = fmin(fmax((double)a.u_sample[n], 0.0), 1.0);
        const double target = u * total;
        // the segment that the border falls into: the first whose running sum passes the target, else the last
        // that is not empty
        if (warp == 0) {
            double before = 0.0, at = 0.0;
            int found = -1, last = -1;
            double last_before = 0.0;
            for (int s0 = 0; s0 < segs && found < 0; s0 += 32) {
                const double x = s0 + lane < segs ? seg_sum[s0 + lane] : 0.0;
                const double c = before + warp_scan(x, lane);
                const unsigned hit = __ballot_sync(0xffffffffu, x > 0.0 && c > target);
                const unsigned some = __ballot_sync(0xffffffffu, x > 0.0);
                if (hit) {
                    const int l = __ffs(hit) - 1;
                    found = s0 + l;
                    at = __shfl_sync(0xffffffffu, c - x, l);
                } else if (some) {
                    const int l = 31 - __clz(some);
                    last = s0 + l;
                    last_before = __shfl_sync(0xffffffffu, c - x, l);
                }
                before = __shfl_sync(0xffffffffu, c, 31);
            }
            if (lane == 0) {
                s_mode = found >= 0 ? found : last;
                s_total = found >= 0 ? at : last_before;
                s_found = 0x7fffffff;
                s_last = -1;
            }
        }
        __syncthreads();
        // the token within the segment
        const int j0 = s_mode * kSeg + tid * (kSeg / kThreads);
        double x[kSeg / kThreads], mine = 0.0;
#pragma unroll
        for (int i = 0; i < kSeg / kThreads; ++i) {
            x[i] = j0 + i < V ? row.at(j0 + i) : 0.0;
            mine += x[i];
        }
        const double c = warp_scan(mine, lane);
        if (lane == 31) wsum[warp] = c;
        __syncthreads();
        double run = s_total + c - mine;
        for (int w = 0; w < warp; ++w) run += wsum[w];
        int found = 0x7fffffff, last = -1;
#pragma unroll
        for (int i = 0; i < kSeg / kThreads; ++i) {
            run += x[i];
            if (x[i] > 0.0) {
                if (run > target) found = min(found, j0 + i);
                last = j0 + i;
            }
        }
        if (found != 0x7fffffff) atomicMin(&s_found, found);
        if (last >= 0) atomicMax(&s_last, last);
        __syncthreads();
        token = s_found != 0x7fffffff ? s_found : s_last;
    }
    for (int i = tid; i <= k; i += kThreads) tokens[i] = i < taken ? drafts[i] : (i == taken ? token : -1);
    if (tid == 0) a.n_accepted[n] = taken;
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a, gdn2_dtype dt, cudaStream_t st) {
    if (dt == GDN2_F32)
        verify_kernel<float><<<a.n_seq, kThreads, 0, st>>>(a);
    else
        verify_kernel<__nv_bfloat16><<<a.n_seq, kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace gdn2
